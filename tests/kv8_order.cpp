// Prints what a product warp of the attention tiles does, in its order, from the header that the kernel is made from.
// Arguments: BY, RUN, group, then the segments' steps.  A line an operation; "products" with its step and whether it adds to the
// sum, "out" behind the last of a run, then the scores issued behind it.
#include <cstdio>
#include <cstdlib>

#include "kv8_order.h"

template <int BY, int RUN>
void print(int grp, int segments, char** steps) {
  int step = 0;
  for (int i = 0; i < segments; ++i) {
    const int n = std::atoi(steps[i]);
    csa2::product_order<BY, RUN>(
        grp, step, n, [&] { std::printf("query %d\n", i); }, [](int st) { std::printf("keys %d\n", st); },
        [](int st) { std::printf("scores %d\n", st); }, [](int st) { std::printf("values %d\n", st); },
        [] { std::printf("turn\n"); }, [] { std::printf("weights\n"); },
        [](int st, bool add, bool out, bool on) {
          std::printf("products %d %d\n", st, add);
          if (out) std::printf("out\n");
          if (on) std::printf("scores %d\n", st + BY);
          std::printf("pass\n");
        },
        [] { std::printf("pass\n"); });
    step += n;
  }
}

int main(int argc, char** argv) {
  if (argc < 5) return 1;
  const bool both = std::atoi(argv[1]) == 1, two = std::atoi(argv[2]) == 2;
  const auto run = both ? (two ? print<1, 2> : print<1, 128>) : two ? print<2, 2> : print<2, 128>;
  run(std::atoi(argv[3]), argc - 4, argv + 4);
  return 0;
}
