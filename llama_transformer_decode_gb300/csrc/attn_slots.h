// The order in which the issuing warp of one slot of the 16-bit tensor-core role (attn_pages_tc.cuh) meets the tiles of an
// item, and the barriers it meets them at.  Plain C++, so that a simulation on the CPU runs the same code as the kernel.
//
// A wait by parity cannot tell a phase from the one two before it, so whoever waits at a barrier must have seen its last phase.
// Tiles alternate between the slots inside an item, but their numbers run on from item to item and items of many pairs
// give every tile to both slots, so a stage's last tile may have been either slot's.  Hence a stage has three barriers that a
// tile's arrival completes: one for tiles of slot 0, one for tiles of slot 1, one for tiles of both.  Each is then
// awaited, phase after phase, by all who ever wait at it.  (One barrier at which both slots await every tile: 104 us in place of
// 101 for 32 KV heads of 64 pairs and 16384 keys, since neither slot then gets ahead of the other.)
#pragma once
#ifdef __CUDACC__
#define L2_SLOTS_FN __host__ __device__ __forceinline__
#else
#define L2_SLOTS_FN inline
#endif

namespace l2 {

constexpr int kTakers = 3;
// Who takes tile i of an item: slot 0 or 1, or 2 for both.
L2_SLOTS_FN int taker_of(int i, bool both) { return both ? 2 : i & 1; }

// The parities of the phases that a slot awaits next, a bit for each barrier of one ring.
template <int STAGES>
struct Phases {
    unsigned bits = 0;
    static_assert(kTakers * STAGES <= 32, "a bit for each barrier");
    L2_SLOTS_FN int next(int taker, int stage) {
        const int b = taker * STAGES + stage, parity = (int)(bits >> b & 1u);
        bits ^= 1u << b;
        return parity;
    }
};

// Slot s, tiles t0 .. t0 + n - 1 of the block.  `both`: both slots take every tile, else slot s takes tiles t0 + s, t0 + s + 2, ..
//   queries()            waits for the item's queries; a slot without tiles has none
//   see_k(t), see_v(t)   waits until K or V of tile t is there
//   scores(t)            issues the first product
//   weights()            waits for the weights of the first half of the last scores' keys
//   products(t, first)   issues the second product, for those keys and, once their weights are there, for the others
//   drained()            waits until it is complete
// All but scores return whether to go on.  The weights lie over their scores, so the next scores wait for the product that reads them.
template <class Queries, class SeeK, class SeeV, class Scores, class Weights, class Products, class Drained>
L2_SLOTS_FN bool slot_item(int s, int t0, int n, bool both, Queries &queries, SeeK &see_k, SeeV &see_v, Scores &scores, Weights &weights,
                           Products &products, Drained &drained) {
    const int step = both ? 1 : 2, end = t0 + n, begin = t0 + (both ? 0 : s);
    auto score = [&](int t) {
        if (!see_k(t)) return false;
        scores(t);
        return true;
    };
    if (begin < end && (!queries() || !score(begin))) return false;
    for (int t = begin; t < end; t += step) {
        if (!weights() || !see_v(t) || !products(t, t == begin)) return false;
        if (t + step < end && !(drained() && score(t + step))) return false;
    }
    return true;
}

}  // namespace l2
