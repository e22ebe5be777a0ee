// Decode over shared prefixes: groups of rows, the units of their shared pages
// and where the partial results lie.
//
// A group that shares npg pages has nb = ceil(npg / 2) blocks of 128 keys (two
// pages).  Its rows are cut into tiles of tile_tokens; the units (block, kv
// head, tile) of all groups, blocks fastest, are cut into equal runs of `share`
// units, one per CTA, and a run's part of one (tile, kv head) is a piece.
#pragma once

#include "internal.h"

namespace pdattn {

// Groups that save fewer page reads are attended row by row: (rows - 1) pages.
// (256 rows in 128 groups of 8 pages: 129 us shared, 116 row by row; in 64
// groups 107 and 108; in 16 groups 84 and 105; two rows of 16 pages 14 and 19.)
constexpr int kSharedMinPages = 6;
constexpr int kSharedMinSaved = 24;

// Most CTAs that nb units in a row can belong to, at `share` units a CTA.
__host__ __device__ __forceinline__ int shared_pieces(int nb, int share) { return (nb + share - 2) / share + 1; }

// The group that holds a row (or, by_unit, a unit of the shared pages), and
// what all groups have.
struct GroupAt {
    int index, row0, rows, npg;
    int unit0;              // units of the groups before
    int s1, s2;             // sums over the groups before that share: rows * kv_heads * nb, rows * kv_heads
    int units, halves;      // of all groups: units; the same, counted twice where a tile has rows in both halves
    int covered;            // of all groups: rows * shared pages
    bool bad;               // the list is no partition of the rows
    // First partial slot.  The group needs rows * kv_heads * shared_pieces(nb, share)
    // <= rows * kv_heads * (nb / share + 2) of them, and rounding s1 / share
    // down loses less than the one that `index` adds per group.
    __device__ int slot0(int share) const { return s1 / share + 2 * s2 + index; }
};

// Whole warp; reads the call's inputs only.
template <bool by_unit>
__device__ GroupAt find_group(const SharedScan& a, int key, int lane) {
    const int Hk = a.kv_heads, Tt = a.tile_tokens;
    GroupAt f = {};
    bool bad = false;
    int carry1 = 0, carry2 = 0;
    #pragma unroll 1
    for (int b = 0; b < a.n_groups; b += 32) {
        const int i = b + lane;
        int s0 = 0, rows = 0, npg = 0;
        if (i < a.n_groups) {
            s0 = __ldg(a.start + i);
            const int s1 = __ldg(a.start + i + 1), n = __ldg(a.pages + i);
            bad = bad || (i == 0 && s0 != 0) || (i == a.n_groups - 1 && s1 != a.rows) || s0 > s1 || n < 0;
            rows = s1 - s0;
            npg = n >= kSharedMinPages && n <= a.pages_per_row && (long long)(rows - 1) * n >= kSharedMinSaved ? n : 0;
        }
        if (a.window > 0) {
            // a group of which the window hides some position from some row does not share
            for (uint32_t todo = __ballot_sync(0xffffffffu, npg > 0); todo; todo &= todo - 1) {
                const int l = __ffs(todo) - 1;
                const int r0 = max(__shfl_sync(0xffffffffu, s0, l), 0);
                const int r1 = min(__shfl_sync(0xffffffffu, s0 + rows, l), a.rows);
                bool hidden = false;
                #pragma unroll 4
                for (int v = r0 + lane; v < r1; v += 32) {
                    const int pos = __ldg(a.positions + v);
                    hidden = hidden || (pos >= 0 && pos < a.max_pos && row_lo(pos, a.window) > 0);
                }
                if (__any_sync(0xffffffffu, hidden) && lane == l) npg = 0;
            }
        }
        const int nb = (npg + 1) / 2, mine = npg ? (rows + Tt - 1) / Tt * nb * Hk : 0;
        const int m1 = rows * Hk * nb, m2 = npg ? rows * Hk : 0;
        int u = mine, t1 = m1, t2 = m2;
        #pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int pu = __shfl_up_sync(0xffffffffu, u, d), p1 = __shfl_up_sync(0xffffffffu, t1, d);
            const int p2 = __shfl_up_sync(0xffffffffu, t2, d);
            if (lane >= d) {
                u += pu;
                t1 += p1;
                t2 += p2;
            }
        }
        const int unit0 = f.units + u - mine;
        const bool here = by_unit ? mine > 0 && unit0 <= key && key < unit0 + mine : s0 <= key && key < s0 + rows;
        const uint32_t hit = __ballot_sync(0xffffffffu, here);
        if (hit) {
            const int l = __ffs(hit) - 1;
            f.index = b + l;
            f.row0 = __shfl_sync(0xffffffffu, s0, l);
            f.rows = __shfl_sync(0xffffffffu, rows, l);
            f.npg = __shfl_sync(0xffffffffu, npg, l);
            f.unit0 = __shfl_sync(0xffffffffu, unit0, l);
            f.s1 = carry1 + __shfl_sync(0xffffffffu, t1 - m1, l);
            f.s2 = carry2 + __shfl_sync(0xffffffffu, t2 - m2, l);
        }
        // (a group's last tile may be a small one)
        const int two = npg ? (rows + Tt / 2 - 1) / Tt * nb * Hk : 0;
        f.halves += (int)__reduce_add_sync(0xffffffffu, (unsigned)(mine + two));
        f.covered += (int)__reduce_add_sync(0xffffffffu, (unsigned)(rows * npg));
        f.units += __shfl_sync(0xffffffffu, u, 31);
        carry1 += __shfl_sync(0xffffffffu, t1, 31);
        carry2 += __shfl_sync(0xffffffffu, t2, 31);
    }
    f.bad = __any_sync(0xffffffffu, bad);
    return f;
}

}  // namespace pdattn
