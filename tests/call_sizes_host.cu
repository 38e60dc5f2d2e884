// What the older cache calls' kernels take holds nothing of the prefixes' arguments: a launch of a single token is
// short enough for them to show. Prints "ok".
#include <cstdio>
#include <type_traits>

#include "mp_cache.cuh"
#include "mp_prefix.h"

using namespace mp;

template <typename T, typename = void>
struct Grouped : std::false_type {};
template <typename T>
struct Grouped<T, std::void_t<decltype(T::cu_group)>> : std::true_type {};
template <typename T, typename = void>
struct Sums : std::false_type {};
template <typename T>
struct Sums<T, std::void_t<decltype(T::state)>> : std::true_type {};

int main() {
  // 8 numbers, 3 addresses, 3 numbers, 1 address; with 5 addresses, 2 numbers and 3 addresses behind them
  static_assert(sizeof(decltype(ChunkArgs::c)) == 80 && sizeof(ChunkArgs) == 80 + 40 + 8 + 24);
  static_assert(!Grouped<decltype(ChunkArgs::c)>::value && !Sums<ChunkArgs>::value);
  static_assert(!Grouped<decltype(WeightsArgs::c)>::value && !Grouped<decltype(AppendArgs::c)>::value && !Grouped<decltype(EvictArgs::c)>::value);
  static_assert(Grouped<decltype(PrefixFew::own.c)>::value && Sums<decltype(PrefixFew::own)>::value);  // the test sees what it looks for
  std::printf("ok\n");
  return 0;
}
