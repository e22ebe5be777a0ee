// Attention of a decode step over the pages that the rows of a group share,
// on the fifth-generation tensor cores (tcgen05).
//
// Rows whose tables begin with the same pages (a common system prompt, samples
// of one prompt, beams) attend those pages together: with R rows of g query
// heads per kv head the product is [R g, D] x [D, keys], and a page is read
// once for the group where a decode over each row alone reads it R times.
// Softmax splits over the keys,
//   out = sum_c e^(m_c - M) O_c / sum_c e^(m_c - M) l_c,
// so the CTAs that take the shared pages leave (m, l, O) of their share of the
// keys, those that take the rows' own pages (attend_kernel.cuh) do the same,
// and a last launch joins them into the outputs.
//
// Work.  Tiles of up to 256 / g rows of a group (two halves of 128 MMA rows)
// times kv heads, each over blocks of 128 keys (two pages).  All (tile, kv
// head, block) units in order are cut into equal runs, one per CTA, so that
// every CTA works equally long whatever the groups' sizes are; a run that
// covers part of a (tile, kv head) is one piece, and a CTA's first and last
// pieces are the only ones cut.  There is no plan: every CTA finds its run from
// the group list, and loads keys and values (which no launch of the call
// writes) before the rope launch is over, whose queries it then waits for.
// Every key of a block is visible to every row
// of its tile (shared pages are full, and a window that hides some of them
// keeps the group from being shared), so there is no mask but the missing
// second page of an odd count.
//
// Halves.  The two halves keep the tensor core busy in turn: one's softmax runs
// under the other's MMAs.  In a tile of at most 128 MMA rows they take every
// other block of keys for the same rows, and each adds its half of the columns
// of both outputs up at the end; in a larger one half B holds the rows past
// 128 / g.
//
// Per block and half: S = Q K^T into tensor memory, one softmax thread per MMA
// row (running maximum, raised lazily past 2^8; exp2; sums), P as bf16 over
// S's columns, O += P V with P read from tensor memory.  Each half's S follows
// the PV of its block before (P lies in S's columns).  bf16 weights are summed as rounded, so that the
// normalised weights stay a convex combination.
//
// Warpgroups: 0 = warp 0 TMA producer, warp 1 tensor-memory owner and MMA
// issuer; 1 and 2 = softmax and partial results of halves A and B.  Every
// wait is bounded; on a timeout the kernel sets the error flag, drains its own
// copies and MMAs, frees tensor memory and returns.
#include "attend_kernel.cuh"
#include "shared.cuh"

namespace pdattn {
namespace {

constexpr int kShThreads = 384;
constexpr float kRescaleLog2 = 8.0f;    // lazy rescale threshold (log2 units)
// Up to here (log2 units) a score's product with the scale and the subtraction
// of the running maximum are one FMA.  The maximum is a rounded product, so the
// FMA leaves the largest score up to 2^-24 of itself above or below it: past
// 2^31 a weight of 2^128 or of nothing, and beside the own pages' weights, whose
// products are rounded, a factor of 2^(2^-24 |score|).  Past kFar, where that
// factor reaches 2^-12, products are rounded here too.  (That the case is looked
// for takes a call of 64 rows 44.6 instead of 43.8 us and one of 256 rows 156.7
// instead of 156.2, graph replays 41.4 and 41.3, 154.0 and 153.8; as a loop of its
// own over S in tensor memory calls took 45.7 and 156.4.)
constexpr float kFar = 4096.f;
constexpr int kPieceSlots = 4;
constexpr int kPieceReaders = 9;        // the issuing warp and the eight softmax warps

// Registers per thread after the hand-over (the launch gives 384 threads 168
// each): 128 x 80 + 256 x 208 = 63488 of 64512.
constexpr uint32_t kRegsIssue = 80, kRegsSoftmax = 208;
static_assert(128 * kRegsIssue + 256 * kRegsSoftmax <= 384 * 168, "register hand-over exceeds the launch");

struct ShBars {
    uint64_t q_full[2], q_empty[2];   // [half]: Q loaded / every S of the piece reading it done
    uint64_t piece_full[kPieceSlots], piece_empty[kPieceSlots];
    uint64_t s_full[2];               // [half]: S of the block done (its previous PV too)
    uint64_t p_full[2];               // [half]: P of the block written (one arrival per warp of the half)
    uint64_t o_done[2];               // [half]: the piece's last PV done
    uint64_t both;                    // the halves of a small tile exchange their sums, then have read both outputs
    uint64_t mma_done;
};

// Blocks of one (tile, kv head); nblk 0: no more work.
struct __align__(32) Piece {
    int ntok;           // rows of the tile: at most tile_tokens / 2 where the halves take every other block
    int nblk;
    int pages;          // shared pages from the first block on
    int slot, stride;   // partial of the tile's first row, and from one row to the next
    int pad[3];
};

// What lies after the ring.  (The launch has no other shared variables: its
// dynamic memory then begins where swizzled tiles may, at a multiple of 1024.)
constexpr int kMaxSlots = 10;

struct ShSmem {
    float2 sums[2][128];                    // small tiles: (maximum, sum) of each half's rows
    Piece ring[kPieceSlots];
    ShBars bars;
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint32_t tmem;
    int abort;
};

template <int D>
struct ShCfg {
    static constexpr int kBoxes = D / 64;                 // 64-element column boxes
    static constexpr int kQBytes = kBoxes * 16384;        // one half: 128 rows x 128 B per box
    static constexpr int kKBytes = kBoxes * 16384;        // K (or V) of a block: 128 keys x 128 B per box
    static constexpr int kPageBytes = 8192;               // one page's 64 rows of a box
    // K and V of successive blocks take the slots of one ring in turn: 160 KiB
    // in flight, which HBM under load needs (a block's K and V as one stage, two
    // of them: 24 rows over 65472 positions 68.5 instead of 66.6 us)
    static constexpr int kSlots = D == 128 ? 5 : 10;
    static constexpr int kOffRing = 2 * kQBytes;
    static constexpr int kSmem = kOffRing + kSlots * kKBytes + (int)sizeof(ShSmem);
    // Tensor memory: S of half h at column 128 h (the first 64 then hold P as
    // bf16 pairs); O of half h at 256 + h D.
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kColO = 256;
    static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

// Whole warp: the next piece; false on abort.
__device__ __forceinline__ bool take_piece(ShBars& bars, const Piece* ring, uint32_t k, int lane, volatile int* abort,
                                           Ctrl* ctrl, Piece& p) {
    const int slot = k % kPieceSlots;
    if (!warp_wait(smem_u32(&bars.piece_full[slot]), (k / kPieceSlots) & 1, abort, ctrl)) return false;
    const volatile int4* src = reinterpret_cast<const volatile int4*>(&ring[slot]);
    p.ntok = src[0].x; p.nblk = src[0].y; p.pages = src[0].z; p.slot = src[0].w;
    p.stride = src[1].x;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars.piece_empty[slot]));
    return true;
}

// Softmax and partial results of one half (128 threads, one MMA row each).
template <int D>
__device__ __forceinline__ void softmax_half(const SharedArgs& a, int half, int quarter, int lane, uint32_t tmem,
                                             ShBars& bars, const Piece* ring, float2 (*s_sums)[128],
                                             volatile int* abort, Ctrl* ctrl) {
    using C = ShCfg<D>;
    const int g = a.group, Tq = a.sc.tile_tokens / 2;
    const int m = quarter * 32 + lane;                    // MMA row = TMEM lane
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + 128u * half, o_addr = tmem + lane_base + C::kColO + half * D;
    const int tq = m / g, jh = m % g;
    const float sl2 = a.scale_log2;
    const uint32_t s_full = smem_u32(&bars.s_full[half]), p_full = smem_u32(&bars.p_full[half]);
    uint32_t ch = 0, uh = 0, xh = 0;                      // blocks and pieces of this half; exchanges
    Piece p;
    for (uint32_t k = 0; take_piece(bars, ring, k, lane, abort, ctrl, p) && p.nblk > 0; ++k) {
        const bool small = p.ntok <= Tq;
        const int tok = small ? tq : half * Tq + tq;      // row of the tile
        const int slot = tq < Tq && tok < p.ntok ? p.slot + tok * p.stride : -1;
        const int nblk = small ? (p.nblk + 1 - half) / 2 : p.nblk;
        // whether this half's last block lacks its second page
        const int odd = p.pages < 2 * p.nblk && (!small || ((p.nblk - 1) & 1) == half) ? nblk - 1 : -1;
        float m_run = -INFINITY, l = 0.f;
        bool ok = true;
        for (int b = 0; b < nblk; ++b) {
            ok = pf_wait(s_full, (ch + b) & 1, abort, ctrl);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            uint32_t s[128];
            #pragma unroll
            for (int q4 = 0; q4 < 4; ++q4)
                tmem_ld32(s_addr + 32 * q4, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * q4]));
            tmem_wait_ld();
            if (b == odd) {
                #pragma unroll
                for (int c = 64; c < 128; ++c) s[c] = __float_as_uint(-INFINITY);
            }
            const float mx = __fmul_rn(max128(s), sl2);    // scale > 0: the max commutes with it
            const bool need = mx > m_run + kRescaleLog2;
            float alpha = 1.f;
            if (need) {
                alpha = exp2_approx(m_run - mx);           // 0 while m_run is -inf
                m_run = mx;
                l *= alpha;
            }
            const float neg_mu = m_run == -INFINITY ? 0.f : -m_run;
            // (one vote for both rare cases)
            const bool far = fabsf(neg_mu) > kFar, moved = b > 0 && need && alpha != 1.f;
            float factor = sl2;
            if (__any_sync(0xffffffffu, far || moved)) {
                if (__any_sync(0xffffffffu, moved)) {
                    #pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[32];
                        tmem_ld32(o_addr + c0, o);
                        tmem_wait_ld();
                        #pragma unroll
                        for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                        tmem_st32(o_addr + c0, o);
                    }
                }
                if (__any_sync(0xffffffffu, far)) {
                    // (x + -0 is x: the other lanes' scores stay as they are)
                    const float f = far ? sl2 : 1.f;
                    factor = far ? 1.f : sl2;
                    #pragma unroll
                    for (int c = 0; c < 128; c += 2) {
                        float x0, x1;
                        ffma2(x0, x1, __uint_as_float(s[c]), __uint_as_float(s[c + 1]), f, -0.f);
                        s[c] = __float_as_uint(x0);
                        s[c + 1] = __float_as_uint(x1);
                    }
                }
            }
            uint32_t pk[64];
            float acc[8] = {};
            #pragma unroll
            for (int h64 = 0; h64 < 2; ++h64) {
                #pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    const int cc = 64 * h64 + c, q = (cc >> 1) & 3;
                    float x0, x1;
                    ffma2(x0, x1, __uint_as_float(s[cc]), __uint_as_float(s[cc + 1]), factor, neg_mu);
                    pk[cc >> 1] = pack_bf16x2(exp2_approx(x0), exp2_approx(x1));
                    add_bf16x2_f32(acc[2 * q], acc[2 * q + 1], pk[cc >> 1]);
                }
                tmem_st32(s_addr + 32 * h64, *reinterpret_cast<const uint32_t(*)[32]>(&pk[32 * h64]));
            }
            // every lane's stores are complete and fenced before its warp's
            // one arrival
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
            l += ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
        }
        if (!ok) return;
        ch += nblk;
        if (nblk > 0) {
            if (!warp_wait(smem_u32(&bars.o_done[half]), uh & 1, abort, ctrl)) return;
            ++uh;
        }
        tc_fence_after();
        const size_t at = (size_t)max(slot, 0) * g + jh;
        float2* ml = reinterpret_cast<float2*>(a.ws + a.S.pre_ml) + at;
        float* orow = reinterpret_cast<float*>(a.ws + a.S.pre_o) + at * D;
        // O of this half's columns of its own rows, or of both halves' blocks
        auto store = [&](int c0, const uint32_t (&o)[32]) {
            #pragma unroll
            for (int v = 0; v < 4; ++v)
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                             ::"l"(orow + c0 + 8 * v), "r"(o[8 * v]), "r"(o[8 * v + 1]), "r"(o[8 * v + 2]),
                               "r"(o[8 * v + 3]), "r"(o[8 * v + 4]), "r"(o[8 * v + 5]), "r"(o[8 * v + 6]),
                               "r"(o[8 * v + 7])
                             : "memory");
        };
        if (!small) {
            if (slot >= 0) *ml = make_float2(m_run, l);
            #pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t o[32];
                tmem_ld32(o_addr + c0, o);
                tmem_wait_ld();
                if (slot >= 0) store(c0, o);
            }
            // The next piece's first PV overwrites O only after this read (its
            // p_full arrival follows in program order).
            tc_fence_before();
            continue;
        }
        auto meet = [&]() -> bool {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars.both));
            const bool met = warp_wait(smem_u32(&bars.both), xh++ & 1, abort, ctrl);
            tc_fence_after();
            return met;
        };
        s_sums[half][m] = make_float2(m_run, l);
        if (!meet()) return;
        const float2 other = s_sums[half ^ 1][m];
        const bool has_other = half == 1 || p.nblk > 1;
        const float M = fmaxf(m_run, other.x);
        const float f0 = m_run == -INFINITY ? 0.f : exp2_approx(m_run - M);
        const float f1 = other.x == -INFINITY ? 0.f : exp2_approx(other.x - M);
        if (slot >= 0 && half == 0) *ml = make_float2(M, l * f0 + other.y * f1);
        const uint32_t x_addr = o_addr + (half ? -D : D);
        #pragma unroll 1
        for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {
            // (a half without blocks holds old values, which are not used)
            uint32_t o[32], x[32];
            tmem_ld32(o_addr + c0, o);
            tmem_ld32(x_addr + c0, x);
            tmem_wait_ld();
            #pragma unroll
            for (int c = 0; c < 32; ++c) {
                float y = nblk > 0 ? __uint_as_float(o[c]) * f0 : 0.f;
                if (has_other) y += __uint_as_float(x[c]) * f1;
                o[c] = __float_as_uint(y);
            }
            if (slot >= 0) store(c0, o);
        }
        // Both halves have read before either's next PV.
        if (!meet()) return;
    }
}

// CTA `cta` of `n_ctas` that attend the shared pages; `total` units in all.
template <int D>
__device__ __forceinline__ void prefix_cta(const CUtensorMap& q_map, const CUtensorMap& k_map, const CUtensorMap& v_map,
                                           const SharedArgs& a, const int cta, const int n_ctas, const int total) {
    using C = ShCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* sm = smem_raw;
    ShSmem& m = *reinterpret_cast<ShSmem*>(sm + C::kOffRing + C::kSlots * C::kKBytes);
    ShBars& bars = m.bars;
    Piece* ring = m.ring;
    const uint32_t q_s = smem_u32(sm), st_s = q_s + C::kOffRing;
    const uint32_t full = smem_u32(m.full), empty = smem_u32(m.empty);     // of slot s: + 8 s
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(a.ws);
    volatile int* abort = &m.abort;

    // Rows of the Q tiles that no query fills stay zero.
    for (int i = tid; i < 2 * C::kQBytes / 16; i += kShThreads) reinterpret_cast<uint4*>(sm)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) {
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int k = 0; k < kPieceSlots; ++k) {
            mbar_init(smem_u32(&bars.piece_full[k]), 1);
            mbar_init(smem_u32(&bars.piece_empty[k]), kPieceReaders);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(smem_u32(&bars.q_full[h]), 1);
            mbar_init(smem_u32(&bars.q_empty[h]), 1);
            mbar_init(smem_u32(&bars.s_full[h]), 1);
            mbar_init(smem_u32(&bars.p_full[h]), 4);
            mbar_init(smem_u32(&bars.o_done[h]), 1);
        }
        mbar_init(smem_u32(&bars.both), 8);
        mbar_init(smem_u32(&bars.mma_done), 1);
        m.abort = 0;
        fence_barrier_init();
        prefetch_tensormap(&q_map);
        prefetch_tensormap(&k_map);
        prefetch_tensormap(&v_map);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&m.tmem)), "r"(C::kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_proxy_async_shared();     // zeroed Q rows, before any MMA reads them
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m.tmem;

    // The issuing warpgroup hands registers to the softmax warpgroups.
    if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        softmax_half<D>(a, (warp - 4) >> 2, warp & 3, lane, tmem, bars, ring, m.sums, abort, ctrl);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
      if (warp == 0) {
        // ---------------- TMA producer (whole warp, one lane issues) ----------------
        const int Hk = a.sc.kv_heads, g = a.group, Tt = a.sc.tile_tokens, Tq = Tt / 2;
        uint32_t it = 0, uq0 = 0, uq1 = 0;            // slots filled (K, V, K, ...); pieces whose Q halves were loaded
        bool ok = true, waited = false;
        const int share = (total + n_ctas - 1) / n_ctas;
        int x = cta * share;
        const int xe = min(total, x + share);
        if (cta == 0 && lane == 0) ctrl->sh_share = share;
        int row0 = 0, rows = 0, npg = 0, unit0 = 0, slot0 = 0;        // the group that unit x lies in
        int left = 0;                                                 // its units from x on
        for (uint32_t k = 0; ok; ++k) {
            const int slot = k % kPieceSlots;
            int t0 = 0, ntok = 0, h = 0, nblk = 0, first = 0, pages = 0, part = 0, stride = 0;
            if (x < xe) {
                if (left == 0) {
                    const GroupAt f = find_group<true>(a.sc, x, lane);
                    row0 = f.row0;
                    rows = f.rows;
                    npg = f.npg;
                    unit0 = f.unit0;
                    slot0 = f.slot0(share);
                }
                const int nb = (npg + 1) / 2, tile = (x - unit0) / (nb * Hk), rel = x - unit0 - tile * nb * Hk;
                const int pair0 = x - rel % nb, most = shared_pieces(nb, share);
                h = rel / nb;
                nblk = min(pair0 + nb, xe) - x;
                first = 2 * (x - pair0);
                pages = min(npg - first, 2 * nblk);
                t0 = row0 + tile * Tt;
                ntok = min(rows - tile * Tt, Tt);
                stride = Hk * most;
                part = slot0 + tile * Tt * stride + h * most + cta - pair0 / share;
                x += nblk;
                left = unit0 + (rows + Tt - 1) / Tt * nb * Hk - x;
            }
            ok = warp_wait(smem_u32(&bars.piece_empty[slot]), ((k / kPieceSlots) & 1) ^ 1, abort, ctrl);
            if (!ok) break;
            if (lane == 0) {
                int4* dst = reinterpret_cast<int4*>(&ring[slot]);
                dst[0] = make_int4(ntok, nblk, pages, part);
                dst[1] = make_int4(stride, 0, 0, 0);
                mbar_arrive(smem_u32(&bars.piece_full[slot]));
            }
            __syncwarp();
            if (nblk == 0) break;
            const int nh = ntok > Tq ? 2 : 1;
            const int* trow = a.table + (size_t)t0 * a.sc.pages_per_row + first;
            // The piece's page ids, 32 at a time: lane l holds page pid_base + l
            // (pid_cur) and the next window's (pid_nxt, read a window ahead).
            int pid_base = -32, pid_cur = 0, pid_nxt = 0;
            auto page_of = [&](int pi) -> int {
                if (pi - pid_base >= 32) {
                    if (pid_base < 0) pid_cur = lane < pages ? __ldg(trow + lane) : 0;
                    else pid_cur = pid_nxt;
                    pid_base += 32;
                    pid_nxt = pid_base + 32 + lane < pages ? __ldg(trow + pid_base + 32 + lane) : 0;
                }
                int page = __shfl_sync(0xffffffffu, pid_cur, pi & 31);
                if (page < 0 || page >= a.num_pages) {
                    if (lane == 0) set_error(ctrl, kErrBadPage);
                    page = 0;
                }
                return (page * Hk + h) * kPageSize;
            };
            // One block's K or V: pages y0 and, unless it is the missing one
            // of an odd count, y1.
            auto load = [&](const CUtensorMap* map, int y0, int y1) -> bool {
                const int s = it % C::kSlots;
                const uint32_t dst = st_s + s * C::kKBytes, bar = full + 8 * s;
                if (!warp_wait(empty + 8 * s, ((it / C::kSlots) & 1) ^ 1, abort, ctrl)) return false;
                elect_arrive_expect_tx(bar, (y1 >= 0 ? 2 : 1) * C::kBoxes * C::kPageBytes);
                #pragma unroll
                for (int b = 0; b < C::kBoxes; ++b) {
                    elect_tma_2d(dst + b * 16384, map, b * 64, y0, bar);
                    if (y1 >= 0) elect_tma_2d(dst + b * 16384 + C::kPageBytes, map, b * 64, y1, bar);
                }
                ++it;
                return true;
            };
            for (int bk = 0; bk < nblk && ok; ++bk) {
                const int y0 = page_of(2 * bk), y1 = 2 * bk + 1 < pages ? page_of(2 * bk + 1) : -1;
                ok = load(&k_map, y0, y1);
                if (!ok) break;
                if (bk == 0) {
                    // K of the first block goes first: its stage frees before the
                    // previous piece's last S is done, which is what Q waits for.
                    // The queries come from the rope launch.
                    if (!waited) griddep_wait();
                    waited = true;
                    #pragma unroll 1
                    for (int hf = 0; hf < nh; ++hf) {
                        const uint32_t n = hf ? uq1 : uq0;
                        ok = warp_wait(smem_u32(&bars.q_empty[hf]), (n & 1) ^ 1, abort, ctrl);
                        if (!ok) break;
                        const uint32_t qf = smem_u32(&bars.q_full[hf]);
                        elect_arrive_expect_tx(qf, C::kBoxes * 128 * g * Tq);
                        #pragma unroll
                        for (int b = 0; b < C::kBoxes; ++b)
                            elect_tma_3d(q_s + hf * C::kQBytes + b * 16384, &q_map, b * 64, h * g, t0 + hf * Tq, qf);
                        if (hf) ++uq1;
                        else ++uq0;
                    }
                }
                ok = ok && load(&v_map, y0, y1);
            }
        }
        // The launches after this one take its end for the rope launch's too.
        if (!waited) griddep_wait();
        // Drain: every load issued has landed before exit.
        for (uint32_t k = 0; k < (uint32_t)C::kSlots && k < it; ++k) {
            const uint32_t j = it - 1 - k;
            mbar_wait(full + 8 * (j % C::kSlots), (j / C::kSlots) & 1, kPfTimeoutNs);
        }
        if (uq0 > 0) mbar_wait(smem_u32(&bars.q_full[0]), (uq0 - 1) & 1, kPfTimeoutNs);
        if (uq1 > 0) mbar_wait(smem_u32(&bars.q_full[1]), (uq1 - 1) & 1, kPfTimeoutNs);
      } else if (warp == 1) {
        // ---------------- MMA issuer (whole warp, one lane issues) ----------------
        constexpr uint32_t idesc_s = instr_desc(128, 128, 0, 0);
        constexpr uint32_t idesc_s64 = instr_desc(128, 64, 0, 0);    // a block of one page
        constexpr uint32_t idesc_o = instr_desc(128, D, 0, 1);
        bool issued = false, ok = true;
        // The start-address field of a descriptor (bits 0..13, address >> 4) is
        // linear, so every operand is a base descriptor plus a constant.
        const uint64_t dq = smem_desc(q_s, 16, 1024), dk = smem_desc(st_s, 16, 1024), dv = smem_desc(st_s, 16384, 1024);
        auto qk = [&](int h, int qh, int s, bool one_page) {
            const uint32_t idesc = one_page ? idesc_s64 : idesc_s;
            const uint64_t a0 = dq + (uint64_t)(qh * (C::kQBytes >> 4));
            const uint64_t b0 = dk + (uint64_t)(s * (C::kKBytes >> 4));
            #pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                umma_f16kind(tmem + 128u * h, a0 + (uint64_t)((ks >> 2) * 1024 + (ks & 3) * 2),
                             b0 + (uint64_t)((ks >> 2) * 1024 + (ks & 3) * 2), idesc, ks > 0 ? 1u : 0u);
            umma_commit(smem_u32(&bars.s_full[h]));
        };
        // Blocks of successive pieces form one stream.  A half's step is the PV
        // of its pending block (possibly of the piece before), then its S of
        // this one.  The half loop stays rolled so that each MMA sequence is
        // issued from one place; per-half state is selected by value.
        // (pend: the pending block's index and flags.)
        constexpr uint32_t kFirst = 1u << 28, kLast = 1u << 29, kOne = 1u << 30, kFree = 1u << 31;
        constexpr uint32_t kIndex = kFirst - 1, kNone = kIndex;
        uint32_t it = 0, uq0 = 0, uq1 = 0, cs0 = 0, cs1 = 0;          // blocks; pieces per Q half / S per half
        uint32_t pend0 = kNone, pend1 = kNone;
        int nblk = 0, bk = 0, pages = 0;                              // the current piece and block
        bool small = false;
        for (uint32_t k = 0; ok;) {
            if (bk >= nblk) {                                         // the piece is done: the next one
                if (nblk > 0) {
                    ++uq0;
                    if (!small) ++uq1;
                }
                Piece p;
                ok = take_piece(bars, ring, k++, lane, abort, ctrl, p);
                if (!ok) break;
                nblk = uni(p.nblk);
                small = uni(p.ntok) <= a.sc.tile_tokens / 2;
                pages = uni(p.pages);
                bk = 0;
            }
            const uint32_t s = 2 * it % C::kSlots;                     // K's slot; V of a block follows its K
            const bool one = pages - 2 * bk == 1, last = bk + 1 >= nblk;
            #pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const bool mine = nblk > 0 && (!small || (bk & 1) == h);
                const uint32_t pend = h ? pend1 : pend0;
                // (at a piece's start both halves' last blocks are finished)
                if (pend != kNone && (mine || bk == 0)) {
                    const uint32_t j = pend & kIndex;
                    const uint32_t sv = (2 * j + 1) % C::kSlots;
                    ok = warp_wait(full + 8 * sv, ((2 * j + 1) / C::kSlots) & 1, abort, ctrl) &&
                         warp_wait(smem_u32(&bars.p_full[h]), ((h ? cs1 : cs0) - 1) & 1, abort, ctrl);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t b0 = dv + (uint64_t)(sv * (C::kKBytes >> 4));
                    #pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        if (ks < 4 || !(pend & kOne))
                            umma_f16kind_ts(tmem + C::kColO + h * D, tmem + 128u * h + ks * 8, b0 + (uint64_t)(ks * 128),
                                            idesc_o, (pend & kFirst) && ks == 0 ? 0u : 1u);
                    if (pend & kLast) umma_commit(smem_u32(&bars.o_done[h]));
                    if (pend & kFree) umma_commit(empty + 8 * sv);
                    if (h) pend1 = kNone;
                    else pend0 = kNone;
                }
                if (!mine) continue;
                ok = warp_wait(full + 8 * s, (2 * it / C::kSlots) & 1, abort, ctrl);
                if (ok && bk == 0) ok = warp_wait(smem_u32(&bars.q_full[h]), (h ? uq1 : uq0) & 1, abort, ctrl);
                if (!ok) break;
                tc_fence_after();
                issued = true;
                qk(h, small ? 0 : h, s, one);
                const uint32_t f = it | (bk < (small ? 2 : 1) ? kFirst : 0) | (bk + (small ? 2 : 1) >= nblk ? kLast : 0) |
                                   (one ? kOne : 0) | (small || h == 1 ? kFree : 0);
                if (h) {
                    pend1 = f;
                    ++cs1;
                } else {
                    pend0 = f;
                    ++cs0;
                }
            }
            if (!ok || nblk == 0) break;
            umma_commit(empty + 8 * s);                       // this block's S issued
            if (last) {
                umma_commit(smem_u32(&bars.q_empty[0]));
                if (!small) umma_commit(smem_u32(&bars.q_empty[1]));
            }
            ++it;
            ++bk;
        }
        // Drain: every MMA issued has finished before TMEM is freed.
        if (issued) {
            umma_commit(smem_u32(&bars.mma_done));
            mbar_wait(smem_u32(&bars.mma_done), 0, kPfTimeoutNs);
        }
      }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols)
                     : "memory");
    }
}

// One launch attends both kinds of pages: the shared ones are bound by the
// tensor cores and their softmax, the rows' own ones by HBM, so that side by
// side each takes what the other leaves.  The number of CTAs of each kind goes
// by what a block of 128 keys for one half of a tile and an own page take on an
// SM (10 ns).  Graph replays, us: at head dim 128 a unit at 105, 118, 130 and 135,
// 256 rows in six groups 155.1, 152.3, 153.7 and 154.5; 40 rows under 200 pages
// 35.8, 37.1, 39.5 and 39.4.  Head dim 64 at 80, 90, 100 and 120, 64 rows under 32
// pages 50.0, 41.9, 42.0 and 46.3; 128 rows under 100 69.6, 68.5, 67.3 and 64.8.
// (The costs differ by what else the launch does; the shared pages have no
// cursor that would make up for it.)
constexpr int kUnitCost[2] = {100, 118};    // head dim 64, 128
constexpr int kPageCost[2] = {40, 36};
constexpr int kItemPages = 3;               // what a pair's start and end cost, in pages

template <int D>
__global__ void __launch_bounds__(kShThreads, 1)
    shared_attend_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map, const __grid_constant__ SharedArgs a,
                         const __grid_constant__ AttendArgs own) {
    // (the dynamic memory's start, before either kind of CTA uses it)
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    int& s_pages = reinterpret_cast<int*>(smem_raw)[0];
    int& s_units = reinterpret_cast<int*>(smem_raw)[1];
    int& s_halves = reinterpret_cast<int*>(smem_raw)[2];
    int& s_covered = reinterpret_cast<int*>(smem_raw)[3];
    griddep_launch_dependents();
    if (threadIdx.x == 0) s_pages = 0;
    __syncthreads();
    // From the call's inputs alone, so that no CTA waits for the rope launch here.
    int pages = 0;
    for (int r = threadIdx.x; r < a.sc.rows; r += kShThreads) {
        const int pos = __ldg(a.sc.positions + r);
        if (pos >= 0 && pos < a.sc.max_pos) pages += pos / kPageSize - row_lo(pos, a.sc.window) / kPageSize + 1;
    }
    pages = (int)__reduce_add_sync(0xffffffffu, (unsigned)pages);
    if ((threadIdx.x & 31) == 0) atomicAdd(&s_pages, pages);
    if (threadIdx.x < 32) {
        const GroupAt f = find_group<true>(a.sc, -1, threadIdx.x);
        if (threadIdx.x == 0) {
            s_units = f.bad ? 0 : f.units;
            s_halves = f.halves;
            s_covered = f.covered;
        }
    }
    __syncthreads();
    const int grid = a.grid, units = s_units, b = blockIdx.x;
    int n_pre = 0;
    if (units > 0) {
        const long long u = (long long)s_halves * kUnitCost[D / 128];
        const long long o = (max(s_pages - s_covered, 0) + (long long)kItemPages * a.sc.rows) * a.sc.kv_heads * kPageCost[D / 128];
        n_pre = max(1, min((int)((u * grid + (u + o) / 2) / (u + o)), grid - 1));
    }
    __syncthreads();
    if (b < n_pre) {
        prefix_cta<D>(q_map, k_map, v_map, a, b, n_pre, units);
    } else {
        const AttendShared sh = {a.S.pairs};
        attend_cta<__nv_bfloat16, D, kMaxGroup>(k_map, v_map, own, sh, b - n_pre, grid - n_pre);
    }
}

// The outputs of rows that share pages, and of pairs that were cut, from their
// partials: four dimensions of one query head per thread.  It is bound by
// latency: the loads of a batch of kBatch partials go out together, and where
// there are more blocks than fit at once, batches are small and more do.  Few
// rows are cut into many pieces, which kLanes lanes then share (24 rows of 19
// pieces and two own ones: a graph replay 63.4 us with four, 64.2 with two, 66.3
// with one; batches of 12 and 24 instead: 65.8, 69.7).
constexpr int kJoinThreads = 128;
constexpr int kJoinWide = 6;         // blocks per SM that fit with batches of 8
constexpr int kJoinFew = 2;          // blocks per SM that leave room for four times as many
constexpr int kJoinLanes = 4;

template <int kBatch, int kLanes>
__global__ void __launch_bounds__(kJoinThreads, kBatch == 4 ? 9 : kJoinWide)
    shared_join_kernel(const __grid_constant__ SharedArgs a) {
    const int D = a.head_dim, g = a.group, Hk = a.sc.kv_heads, per = D / 4, r = blockIdx.x;
    // (a warp's units are dimensions of one head)
    constexpr int kUnits = 32 / kLanes;
    const int part = threadIdx.x % 32 / kUnits;
    const int u = (blockIdx.y * (kJoinThreads / 32) + threadIdx.x / 32) * kUnits + threadIdx.x % kUnits;
    const int hq = u / per, h = hq / g, j = hq - h * g, d0 = (u - hq * per) * 4;
    griddep_wait();
    if (hq >= a.heads) return;
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(a.ws);
    const int4 ri = __ldcg(reinterpret_cast<const int4*>(a.ws + a.S.w.row_info) + r);
    const int4 rp = __ldcg(reinterpret_cast<const int4*>(a.ws + a.S.row_pre) + r);
    const int2 pair = __ldcg(reinterpret_cast<const int2*>(a.ws + a.S.pairs) + (size_t)r * Hk + h);
    const int share = max(__ldcg(&ctrl->sh_share), 1), runs = __ldcg(&ctrl->sh_runs);
    if (ri.x < 0 || pair.x < -1) return;        // skipped, or the output is written
    const int nb = (ri.z + 1) / 2, unit = rp.x + h * nb;
    const int n_pre = ri.z ? (unit + nb - 1) / share - unit / share + 1 : 0, n = n_pre + pair.y;
    const int pre0 = rp.y / share + rp.z + (rp.w * Hk + h) * shared_pieces(nb, share);
    // Where a wait of the attention ran out, some of this was not written in
    // this call: nothing is read past the partials then.
    if (runs < 0 || runs > kSharedRuns * a.grid || pair.y < 1 || pair.y > runs || pair.x > runs - pair.y ||
        (ri.z && (n_pre < 0 || pre0 < 0 || pre0 > a.S.pre_slots - n_pre))) {
        set_error(ctrl, kErrBadPlan);
        return;
    }
    float M = -1.0e30f, L = 0.f, O[4] = {};
    #pragma unroll 1
    for (int c0 = part; c0 < n; c0 += kBatch * kLanes) {
        float2 x[kBatch];
        float4 p[kBatch];
        #pragma unroll
        for (int c = 0; c < kBatch; ++c) {
            const int i = c0 + c * kLanes, o = i - n_pre;
            x[c] = make_float2(-1.0e30f, 0.f);
            if (i >= n) continue;
            // a cut pair's first piece is its run's second slot, the others are the first ones of the runs that follow
            const size_t at = (size_t)(o < 0 ? pre0 + i : pair.x < 0 ? 2 * runs + r * Hk + h : 2 * (pair.x + o) + (o == 0)) * g + j;
            x[c] = __ldcg(reinterpret_cast<const float2*>(a.ws + (o < 0 ? a.S.pre_ml : a.S.w.part_ml)) + at);
            p[c] = __ldcg(reinterpret_cast<const float4*>(
                reinterpret_cast<const float*>(a.ws + (o < 0 ? a.S.pre_o : a.S.w.part_o)) + at * D + d0));
        }
        float Mn = M;
        #pragma unroll
        for (int c = 0; c < kBatch; ++c) Mn = fmaxf(Mn, x[c].x);
        const float fa = exp2_approx(M - Mn);
        M = Mn;
        L *= fa;
        #pragma unroll
        for (int e = 0; e < 4; ++e) O[e] *= fa;
        #pragma unroll
        for (int c = 0; c < kBatch; ++c) {
            if (c0 + c * kLanes >= n) break;
            const float f = exp2_approx(x[c].x - M);
            L += f * x[c].y;
            O[0] += f * p[c].x;
            O[1] += f * p[c].y;
            O[2] += f * p[c].z;
            O[3] += f * p[c].w;
        }
    }
    if constexpr (kLanes > 1) {
        #pragma unroll
        for (int d = kUnits; d < 32; d *= 2) {
            const float Mo = __shfl_xor_sync(0xffffffffu, M, d), Lo = __shfl_xor_sync(0xffffffffu, L, d);
            const float Mn = fmaxf(M, Mo), f = exp2_approx(M - Mn), fo = exp2_approx(Mo - Mn);
            M = Mn;
            L = L * f + Lo * fo;
            #pragma unroll
            for (int e = 0; e < 4; ++e) O[e] = O[e] * f + __shfl_xor_sync(0xffffffffu, O[e], d) * fo;
        }
        if (part != 0) return;
    }
    const bool has_sink = a.sinks != nullptr;
    const float sk = has_sink ? load_f32<__nv_bfloat16>(a.sinks, hq) * 1.4426950408889634f : 0.f;
    const float inv = out_scale(M, L, has_sink, sk);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + ((size_t)r * a.heads + hq) * D + d0) =
        make_uint2(pack_bf16x2(O[0] * inv, O[1] * inv), pack_bf16x2(O[2] * inv, O[3] * inv));
}

template <int D>
cudaError_t launch_d(const SharedArgs& a, const AttendArgs& own, const CUtensorMap& q_map, const CUtensorMap& k_map,
                     const CUtensorMap& v_map, cudaStream_t stream) {
    constexpr int own_smem = Cfg<__nv_bfloat16, D, kMaxGroup, Uncoded, kWideOwn<D>>::kSmem;
    constexpr int smem = ShCfg<D>::kSmem > own_smem ? ShCfg<D>::kSmem : own_smem;
    auto kern = shared_attend_kernel<D>;
    static int configured_mask = 0;   // bit per device id < 31
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 31 || !(__atomic_load_n(&configured_mask, __ATOMIC_ACQUIRE) & (1 << dev))) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 31) __atomic_fetch_or(&configured_mask, 1 << dev, __ATOMIC_ACQ_REL);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.grid);
    cfg.blockDim = dim3(kShThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, q_map, k_map, v_map, a, own);
}

}  // namespace

cudaError_t launch_shared_attend(const SharedArgs& a, const AttendArgs& own, const CUtensorMap& q_map,
                                 const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
    if (a.head_dim == 128) return launch_d<128>(a, own, q_map, k_map, v_map, stream);
    if (a.head_dim == 64) return launch_d<64>(a, own, q_map, k_map, v_map, stream);
    return cudaErrorInvalidValue;
}

cudaError_t launch_shared_join(const SharedArgs& a, cudaStream_t stream) {
    const int per_row = (a.heads * (a.head_dim / 4) + kJoinThreads - 1) / kJoinThreads;
    const long long blocks = (long long)a.sc.rows * per_row;
    const bool few = blocks <= (long long)a.grid * kJoinFew;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.sc.rows, few ? kJoinLanes * per_row : per_row);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (few) return cudaLaunchKernelEx(&cfg, shared_join_kernel<8, kJoinLanes>, a);
    return blocks <= (long long)a.grid * kJoinWide ? cudaLaunchKernelEx(&cfg, shared_join_kernel<8, 1>, a)
                                                   : cudaLaunchKernelEx(&cfg, shared_join_kernel<4, 1>, a);
}

}  // namespace pdattn
