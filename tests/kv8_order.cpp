// Prints what a product warp of the attention tiles does, in its order, from the header that the kernel is made from.
// Arguments: BY, group, then the segments' steps.  A line an operation; "products" with its step and the scores issued behind it.
#include <cstdio>
#include <cstdlib>

#include "kv8_order.h"

template <int BY>
void print(int grp, int segments, char** steps) {
  int step = 0;
  for (int i = 0; i < segments; ++i) {
    const int n = std::atoi(steps[i]);
    csa2::product_order<BY>(
        grp, step, n, [&] { std::printf("query %d\n", i); }, [](int st) { std::printf("keys %d\n", st); },
        [](int st) { std::printf("scores %d\n", st); }, [](int st) { std::printf("values %d\n", st); },
        [] { std::printf("turn\n"); }, [] { std::printf("weights\n"); },
        [](int st, bool, bool on) {
          std::printf("products %d\n", st);
          if (on) std::printf("scores %d\n", st + BY);
          std::printf("pass\n");
        },
        [] { std::printf("pass\n"); });
    step += n;
  }
}

int main(int argc, char** argv) {
  if (argc < 4) return 1;
  if (std::atoi(argv[1]) == 1) print<1>(std::atoi(argv[2]), argc - 3, argv + 3);
  else print<2>(std::atoi(argv[2]), argc - 3, argv + 3);
  return 0;
}
