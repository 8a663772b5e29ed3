// How an attention call's work is laid on a line and cut into equal shares.  Plain integer
// arithmetic shared by the kernels, the launch code and a host test.
//
// A unit is (layer, sequence, kv head, block of tile_rows rows); its cost is the slots its last row
// sees, times the query heads of the kv head so that it grows linearly from block to block, plus a
// constant for the work of starting and ending it.  Units stand on a line, layer by layer, sequence
// by sequence, head by head, block by block, and workgroup w takes [w Q, (w + 1) Q) of it, Q the
// total over the number of workgroups.  Lengths are read on the device, so shares are equal whatever
// they are, ragged batches and causal prompts included, and a captured call adapts to new lengths.
#pragma once

#include <cstdint>

#include "kv_layout.h"

namespace gdn {

// Cost of starting and ending a unit, in slots: what a workgroup's four waves walk in that time.
constexpr int64_t kUnitSlots = 256;

// A length as the calls read it: 0 to the capacity (2^30 at most), past which no slot is there.
GDN_HD int length_of(int64_t length, int64_t capacity) {
    return int(length < 0 ? 0 : length < capacity ? length : capacity);
}

// Slots that new token `node` sees of a causal sequence, or the slots in use if it is the last.
GDN_HD int slots_upto(int past, int node, int64_t capacity) {
    const int64_t n = int64_t(past) + node + 1;
    return int(n < capacity ? n : capacity);
}

struct SeqWork {
    int64_t a, b;    // cost of block k: a + b k
    int64_t blocks;
    int64_t cost;    // of one head: all blocks
};

GDN_HD SeqWork seq_work(int64_t past, int64_t n_new, int64_t group, int64_t tile_rows, bool tree,
                        int64_t capacity) {
    SeqWork s;
    past = length_of(past, capacity);
    const int64_t total = past + n_new < capacity ? past + n_new : capacity;
    s.blocks = n_new > 0 ? (n_new * group + tile_rows - 1) / tile_rows : 0;
    s.a = (tree ? total * group : past * group + tile_rows) + kUnitSlots * group;
    s.b = tree ? 0 : tile_rows;
    s.cost = s.blocks * s.a + s.b * (s.blocks * (s.blocks - 1) / 2);
    return s;
}

// Cost of the blocks before block k.
GDN_HD int64_t cost_before(const SeqWork &s, int64_t k) { return k * s.a + s.b * (k * (k - 1) / 2); }

// a / b, a >= 0, b > 0: one fp64 division and a correction, a few times faster on the device than
// the 64-bit integer division it has no instruction for.
GDN_HD int64_t quotient(int64_t a, int64_t b) {
    int64_t q = int64_t(double(a) / double(b));
    while (q * b > a) --q;
    while ((q + 1) * b <= a) ++q;
    return q;
}

// Block that holds position rem (0 <= rem < s.cost) of a head's blocks.
GDN_HD int64_t block_at(const SeqWork &s, int64_t rem) {
    int64_t k;
    if (s.b == 0) {
        k = quotient(rem, s.a);
    } else {  // root of b k^2 / 2 + (a - b / 2) k = rem, then exact
        const double p = double(s.a) / double(s.b) - 0.5;
        k = int64_t(__builtin_sqrt(p * p + 2.0 * double(rem) / double(s.b)) - p);
    }
    k = k < 0 ? 0 : k >= s.blocks ? s.blocks - 1 : k;
    while (k > 0 && cost_before(s, k) > rem) --k;
    while (k + 1 < s.blocks && cost_before(s, k + 1) <= rem) ++k;
    return k;
}

// Tile at position x of a unit of cost v (0 <= x <= v), rising with x: the same for the end of one
// share and the start of the next.
GDN_HD int tile_at(int64_t x, int64_t v, int tiles) {
    const int t = int(double(x) * double(tiles) / double(v));
    return x >= v || t > tiles ? tiles : t;
}

// A run of a unit that one workgroup walks: [x, x + length) of its cost.  `begins`: the unit's first,
// which says where its fragments are.  That goes by the run's number, not by x == 0: a unit may cost
// less than it has parts (256 G + 32 and up to 768), and several of them then start at 0.
struct Run {
    int64_t x, length;
    bool begins;
};
GDN_HD Run part_of(int64_t cost, int part, int parts) {
    const int64_t x = cost * part / parts;
    return Run{x, cost * (part + 1) / parts - x, part == 0};
}

// Fragment of a unit cut between workgroups: a share holds two at most, the end of a unit that began
// in an earlier share and the beginning of one that ends in a later.
GDN_HD int64_t fragment_at(int64_t share, bool begins) { return share * 2 + (begins ? 1 : 0); }

}  // namespace gdn
