// Index arithmetic of the tensor-core kernel for runs of rows (pages_prompt.cu), compiled for the host as well, so that the
// order of its waits is stepped through on the CPU: a wait that is missed ends in its time limit on the GPU.
#pragma once

#include "pages_index.cuh"

namespace polykv {
namespace rows {

// The ring that keys and values arrive in: a stage holds a tile's keys or its values.
POLYKV_HD constexpr int ring_stages(int d) { return d == 128 ? 5 : 11; }

// A tile's values and the next one's keys have one barrier turn together, a pair (a unit's first keys and its last values one
// each to themselves), and pairs take the barriers in turn. A wait tells a turn from the next one only, so no barrier may come
// two turns ahead of it: the producer, about to fill a stage, waits for the pair that filled it ring_stages stages ago, and
// as a pair has a stage at least, the pair being filled is at most ring_stages pairs on. With as many barriers as stages it is no
// later turn of the barrier waited for than the next one, and that cannot have been released.
constexpr int kPairs = 16;
static_assert(kPairs >= ring_stages(64) && kPairs >= ring_stages(128), "a stage's last pair and the one being filled share a barrier");
POLYKV_HD uint32_t pair_barrier(uint32_t pair) { return pair % kPairs; }
POLYKV_HD uint32_t pair_parity(uint32_t pair) { return pair / kPairs & 1u; }

// A row tile's key tiles of a unit, counted from its first: every other one, or a range (with what it cannot see inside). Where
// it has none, its sums are not announced: such an announcement would depend on nothing that the tile's softmax does, and the barrier
// could come two turns ahead of a warp that is still behind the sums of the unit before.
struct Turns {
    int lo, hi, by;
    POLYKV_HD bool has(int j) const { return j >= lo && j < hi && !((j - lo) & by); }
    POLYKV_HD bool any() const { return lo < hi; }
};
// Where both row tiles hold the same rows, they take a unit's nj key tiles in turn.
POLYKV_HD Turns every_other(int nj, int i) { return Turns{i, nj > i ? nj - ((nj - 1 - i) & 1) : i, 1}; }

}  // namespace rows
}  // namespace polykv
