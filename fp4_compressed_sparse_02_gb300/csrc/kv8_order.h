// The order in which a product warp of k_kv8_tile (kv8_tile.cu) waits and issues, for one segment of steps.  The kernel
// and, on the host, a model of its barriers (tests/kv8_order.cpp) are both made from it.
#pragma once

#ifdef __CUDACC__
#define CSA2_ORDER __device__ __forceinline__
#else
#define CSA2_ORDER inline
#endif

namespace csa2 {

// Group grp's part of the steps step .. step + n.  BY = 1: both groups have every step; 2: group 0 has the first, third, ...
// and group 1 the others.  The operations:
//   query()                 wait until Q is there, and with it all of the earlier segments is done
//   keys(st), values(st)    wait for the step's keys, for its values in fp16
//   scores(st)              issue the product of Q with the step's keys
//   turn(), pass()          wait for this group's turn; give it to the other group
//   weights()               wait for the weights of the group's next step
//   products(st, add, out, on)
//                           issue the product of the weights with the values (add: to what is there; out: the sum is read
//                           after it), then, if `on`, the scores of step st + BY; pass
// A sum has up to RUN steps of the group.  Who makes the weights reads it before it hands out the next step's.
//
// A wait by parity tells a phase from the one before it, not from the one two before or two after: it may stand only where
// the phase before the awaited one is known to be over, and the one after it to be still to come.  The keys of step st and
// of st - 3 come through one barrier, and with BY = 2 the two steps belong to different groups.  In a segment of one step
// the second group has none, and the next segment's Q does not wait for it: it only takes its turn, which is behind
// the first group's wait for Q.
template <int BY, int RUN, class Query, class Keys, class Scores, class Values, class Turn, class Weights, class Products, class Pass>
CSA2_ORDER void product_order(int grp, int step, int n, Query query, Keys keys, Scores scores, Values values, Turn turn,
                              Weights weights, Products products, Pass pass) {
  const int first = BY == 2 ? grp : 0;
  if (first < n) {
    query();
    keys(step + first);
    scores(step + first);
  }
  for (int j = first; j < n; j += BY) {
    const int st = step + j;
    const bool on = j + BY < n;
    if (BY == 1 && on) keys(st + 1);
    values(st);
    turn();                              // the other group's products of step st - 1 are issued, so its keys have been there
    if (BY == 2 && on) keys(st + 2);
    weights();
    const int i = j / BY % RUN;
    products(st, i > 0, i == RUN - 1 || !on, on);
  }
  if (BY == 2 && grp == 1 && (n & 1)) {  // the first group had a step more
    turn();
    pass();
  }
}

}  // namespace csa2
