// Attention of a decode step over the pages that the rows of a group share,
// on the fifth-generation tensor cores (tcgen05).
//
// Rows whose tables begin with the same pages (a common system prompt, samples
// of one prompt, beams) attend those pages together: with R rows of g query
// heads per kv head the product is [R g, D] x [D, keys], and a page is read
// once for the group where a decode over each row alone reads it R times.
// Softmax splits over the keys,
//   out = sum_c e^(m_c - M) O_c / sum_c e^(m_c - M) l_c,
// so this kernel leaves (m, l, O) of its share of the keys as one more chunk
// of each row, and the decode kernel, which attends the row's own pages,
// merges them all.
//
// Work.  Tiles of up to 256 / g rows of a group (two halves of 128 MMA rows)
// times kv heads, each over blocks of 128 keys (two pages).  All (tile, kv
// head, block) units in order are cut into equal runs, one per CTA, so that
// every CTA works equally long whatever the groups' sizes are; a run that
// covers part of a (tile, kv head) is one piece, and a CTA's first and last
// pieces are the only ones cut.  Every key of a block is visible to every row
// of its tile (shared pages are full, and a window that hides some of them
// keeps the group from being shared), so there is no mask but the missing
// second page of an odd count.
//
// Per block and half: S = Q K^T into tensor memory, one softmax thread per MMA
// row (running maximum, raised lazily past 2^8; exp2; sums), P as bf16 over
// S's columns, O += P V with P read from tensor memory.  The issuer runs
// PV_A(j-1) S_A(j) PV_B(j-1) S_B(j), so each half's softmax runs under the
// other half's MMAs.  bf16 weights are summed as rounded, so that the
// normalised weights stay a convex combination.
//
// Warpgroups: 0 = warp 0 TMA producer, warp 1 tensor-memory owner and MMA
// issuer; 1 and 2 = softmax and partial results of halves A and B.  Every
// wait is bounded; on a timeout the kernel sets the error flag, drains its own
// copies and MMAs, frees tensor memory and returns.
#include "internal.h"
#include "umma.cuh"

namespace pdattn {
namespace {

constexpr int kShThreads = 384;
constexpr float kRescaleLog2 = 8.0f;    // lazy rescale threshold (log2 units)
constexpr int kPieceSlots = 4;
constexpr int kPieceReaders = 9;        // the issuing warp and the eight softmax warps

// Registers per thread after the hand-over (the launch gives 384 threads 168
// each): 128 x 80 + 256 x 208 = 63488 of 64512.
constexpr uint32_t kRegsIssue = 80, kRegsSoftmax = 208;
static_assert(128 * kRegsIssue + 256 * kRegsSoftmax <= 384 * 168, "register hand-over exceeds the launch");

template <int D>
struct ShCfg {
    static constexpr int kBoxes = D / 64;                 // 64-element column boxes
    static constexpr int kQBytes = kBoxes * 16384;        // one half: 128 rows x 128 B per box
    static constexpr int kKBytes = kBoxes * 16384;        // K (or V) of a block: 128 keys x 128 B per box
    static constexpr int kPageBytes = 8192;               // one page's 64 rows of a box
    static constexpr int kStageBytes = 2 * kKBytes;       // K then V of one block
    static constexpr int kStages = D == 128 ? 2 : 5;
    static constexpr int kOffStage = 2 * kQBytes;
    static constexpr int kSmem = kOffStage + kStages * kStageBytes + 1024;   // + alignment slack
    // Tensor memory: S of half h at column 128 h (the first 64 then hold P as
    // bf16 pairs); O of half h at 256 + h D.
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kColO = 256;
    static_assert(kSmem <= 227 * 1024 - 1024, "shared memory budget");
};

struct ShBars {
    uint64_t q_full[2], q_empty[2];   // [half]: Q loaded / every S of the piece reading it done
    uint64_t piece_full[kPieceSlots], piece_empty[kPieceSlots];
    uint64_t s_full[2];               // [half]: S of the block done (its previous PV too)
    uint64_t p_full[2];               // [half]: P of the block written (one arrival per warp of the half)
    uint64_t o_done[2];               // [half]: the piece's last PV done
    uint64_t mma_done;
};

// Blocks [k0, k0 + nblk) of one (tile, kv head); nblk 0: no more work.
struct __align__(32) Piece {
    int t0, ntok;       // the tile's rows
    int npg;            // shared pages of the group
    int h;              // kv head
    int k0, nblk;
    int piece;          // of this (tile, kv head)
    int pad;
};

// Whole warp: the next piece; false on abort.
__device__ __forceinline__ bool take_piece(ShBars& bars, const Piece* ring, uint32_t k, int lane, volatile int* abort,
                                           Ctrl* ctrl, Piece& p) {
    const int slot = k % kPieceSlots;
    if (!warp_wait(smem_u32(&bars.piece_full[slot]), (k / kPieceSlots) & 1, abort, ctrl)) return false;
    const volatile int4* src = reinterpret_cast<const volatile int4*>(&ring[slot]);
    p.t0 = src[0].x; p.ntok = src[0].y; p.npg = src[0].z; p.h = src[0].w;
    p.k0 = src[1].x; p.nblk = src[1].y; p.piece = src[1].z;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars.piece_empty[slot]));
    return true;
}

// Softmax and partial results of one half (128 threads, one MMA row each).
template <int D>
__device__ __forceinline__ void softmax_half(const SharedArgs& a, int half, int quarter, int lane, uint32_t tmem,
                                             ShBars& bars, const Piece* ring, volatile int* abort, Ctrl* ctrl) {
    using C = ShCfg<D>;
    const int g = a.group, Tq = a.tile_tokens / 2;
    const int m = quarter * 32 + lane;                    // MMA row = TMEM lane
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + 128u * half, o_addr = tmem + lane_base + C::kColO + half * D;
    const int tq = m / g, jh = m % g;
    const int tok = half * Tq + tq;                       // row of the tile
    const float sl2 = a.scale_log2;
    const int4* row_info = reinterpret_cast<const int4*>(a.ws + a.L.row_info);
    const uint32_t s_full = smem_u32(&bars.s_full[half]), p_full = smem_u32(&bars.p_full[half]);
    uint32_t ch = 0, uh = 0;                              // blocks and pieces of this half
    Piece p;
    for (uint32_t k = 0; take_piece(bars, ring, k, lane, abort, ctrl, p) && p.nblk > 0; ++k) {
        if (half == 1 && p.ntok <= Tq) continue;
        // The row's partial goes to chunk (own chunks + piece) of its kv head;
        // -1: no row, or one that is skipped.
        int slot = -1;
        if (tq < Tq && tok < p.ntok) {
            const int4 ri = __ldcg(row_info + p.t0 + tok);
            const int most = shared_pieces((p.npg + 1) / 2, __ldcg(&ctrl->sh_share));
            if (ri.x >= 0) slot = ri.w + p.h * (ri.z + most) + ri.z + p.piece;
        }
        const int nblk = p.nblk, pages = p.npg - 2 * p.k0;
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
            if (pages - 2 * b < 2) {
                #pragma unroll
                for (int c = 64; c < 128; ++c) s[c] = __float_as_uint(-INFINITY);
            }
            const float mx = max128(s) * sl2;              // scale > 0: the max commutes with it
            const bool need = mx > m_run + kRescaleLog2;
            float alpha = 1.f;
            if (need) {
                alpha = exp2_approx(m_run - mx);           // 0 while m_run is -inf
                m_run = mx;
                l *= alpha;
            }
            const float neg_mu = m_run == -INFINITY ? 0.f : -m_run;
            if (b > 0 && __any_sync(0xffffffffu, need && alpha != 1.f)) {
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
            uint32_t pk[64];
            float acc[8] = {};
            #pragma unroll
            for (int h64 = 0; h64 < 2; ++h64) {
                #pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    const int cc = 64 * h64 + c, q = (cc >> 1) & 3;
                    float x0, x1;
                    ffma2(x0, x1, __uint_as_float(s[cc]), __uint_as_float(s[cc + 1]), sl2, neg_mu);
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
        if (!warp_wait(smem_u32(&bars.o_done[half]), uh & 1, abort, ctrl)) return;
        tc_fence_after();
        const size_t at = (size_t)max(slot, 0) * g + jh;
        float* orow = reinterpret_cast<float*>(a.ws + a.L.part_o) + at * D;
        if (slot >= 0) reinterpret_cast<float2*>(a.ws + a.L.part_ml)[at] = make_float2(m_run, l);
        #pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[32];
            tmem_ld32(o_addr + c0, o);
            tmem_wait_ld();
            if (slot >= 0) {
                #pragma unroll
                for (int v = 0; v < 4; ++v)
                    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                                 ::"l"(orow + c0 + 8 * v), "r"(o[8 * v]), "r"(o[8 * v + 1]), "r"(o[8 * v + 2]),
                                   "r"(o[8 * v + 3]), "r"(o[8 * v + 4]), "r"(o[8 * v + 5]), "r"(o[8 * v + 6]),
                                   "r"(o[8 * v + 7])
                                 : "memory");
            }
        }
        // The next piece's first PV overwrites O only after this read (its
        // p_full arrival follows in program order).
        tc_fence_before();
        ch += nblk;
        ++uh;
    }
}

template <int D>
__global__ void __launch_bounds__(kShThreads, 1)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map, const __grid_constant__ SharedArgs a) {
    using C = ShCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // K and V of a stage fill and drain separately: K is free once the
    // block's S is done, V once its PV is
    __shared__ __align__(8) uint64_t k_full[C::kStages], k_empty[C::kStages];
    __shared__ __align__(8) uint64_t v_full[C::kStages], v_empty[C::kStages];
    __shared__ __align__(8) ShBars bars;
    __shared__ Piece ring[kPieceSlots];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t q_s = smem_u32(sm), st_s = q_s + C::kOffStage;
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(a.ws + a.L.ctrl);
    volatile int* abort = &s_abort;

    griddep_launch_dependents();
    // Rows of the Q tiles that no query fills stay zero.
    for (int i = tid; i < 2 * C::kQBytes / 16; i += kShThreads) reinterpret_cast<uint4*>(sm)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&k_full[s]), 1);
            mbar_init(smem_u32(&k_empty[s]), 1);
            mbar_init(smem_u32(&v_full[s]), 1);
            mbar_init(smem_u32(&v_empty[s]), 1);
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
        mbar_init(smem_u32(&bars.mma_done), 1);
        s_abort = 0;
        fence_barrier_init();
        prefetch_tensormap(&q_map);
        prefetch_tensormap(&k_map);
        prefetch_tensormap(&v_map);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&s_tmem)), "r"(C::kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_proxy_async_shared();     // zeroed Q rows, before any MMA reads them
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    // Everything below reads what the planner and the rope launch wrote.
    griddep_wait();
    // The issuing warpgroup hands registers to the softmax warpgroups.
    if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        softmax_half<D>(a, (warp - 4) >> 2, warp & 3, lane, tmem, bars, ring, abort, ctrl);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
      if (warp == 0) {
        // ---------------- TMA producer (whole warp, one lane issues) ----------------
        const int Hk = a.kv_heads, g = a.group, Tq = a.tile_tokens / 2;
        const SharedTile* tiles = reinterpret_cast<const SharedTile*>(a.ws + a.tiles);
        const int n_tiles = __ldcg(&ctrl->magic) == kSharedPlanMagic ? __ldcg(&ctrl->sh_tiles) : 0;
        const int share = __ldcg(&ctrl->sh_share);
        uint32_t it = 0, kit = 0, uq0 = 0, uq1 = 0;   // blocks loaded, K of them; pieces whose Q halves were loaded
        bool ok = true;
        int x = n_tiles > 0 ? (int)blockIdx.x * share : 0;
        const int xe = n_tiles > 0 ? min(__ldcg(&ctrl->sh_blocks), x + share) : 0;
        // The tile that unit x lies in: the last one that starts at or before it.
        int ti = 0;
        for (int n = x < xe ? n_tiles : 0; n > 1;) {
            const int step = (n + 31) / 32;
            const bool le = lane * step < n && __ldcg(&tiles[ti + lane * step].start) <= x;
            const int q = 31 - __clz(__ballot_sync(0xffffffffu, le));
            ti += q * step;
            n = min(step, n - q * step);
        }
        for (uint32_t k = 0; ok; ++k) {
            const int slot = k % kPieceSlots;
            int t0 = 0, ntok = 0, npg = 0, h = 0, k0 = 0, nblk = 0, piece = 0;
            if (x < xe) {
                const int4 d0 = __ldcg(reinterpret_cast<const int4*>(tiles + ti));
                npg = uni(__ldcg(&tiles[ti].npg));
                t0 = uni(d0.x);
                ntok = uni(d0.y);
                const int start = uni(d0.z), nb = uni(d0.w);
                h = (x - start) / nb;
                k0 = x - start - h * nb;
                nblk = min(nb - k0, xe - x);
                piece = (int)blockIdx.x - (start + h * nb) / share;
                x += nblk;
                if (x == start + nb * Hk) ++ti;
            }
            ok = warp_wait(smem_u32(&bars.piece_empty[slot]), ((k / kPieceSlots) & 1) ^ 1, abort, ctrl);
            if (!ok) break;
            if (lane == 0) {
                int4* dst = reinterpret_cast<int4*>(&ring[slot]);
                dst[0] = make_int4(t0, ntok, npg, h);
                dst[1] = make_int4(k0, nblk, piece, 0);
                mbar_arrive(smem_u32(&bars.piece_full[slot]));
            }
            __syncwarp();
            if (nblk == 0) break;
            const int nh = ntok > Tq ? 2 : 1, first = 2 * k0, pages = min(npg, first + 2 * nblk) - first;
            const int* trow = a.table + (size_t)t0 * a.pages_per_row + first;
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
            auto load = [&](const CUtensorMap* map, uint32_t full, uint32_t empty, uint32_t dst, uint32_t par, int y0,
                            int y1) -> bool {
                if (!warp_wait(empty, par ^ 1, abort, ctrl)) return false;
                elect_arrive_expect_tx(full, (y1 >= 0 ? 2 : 1) * C::kBoxes * C::kPageBytes);
                #pragma unroll
                for (int b = 0; b < C::kBoxes; ++b) {
                    elect_tma_2d(dst + b * 16384, map, b * 64, y0, full);
                    if (y1 >= 0) elect_tma_2d(dst + b * 16384 + C::kPageBytes, map, b * 64, y1, full);
                }
                return true;
            };
            for (int bk = 0; bk < nblk && ok; ++bk) {
                const int y0 = page_of(2 * bk), y1 = 2 * bk + 1 < pages ? page_of(2 * bk + 1) : -1;
                const int s = it % C::kStages;
                const uint32_t par = (it / C::kStages) & 1, dst = st_s + s * C::kStageBytes;
                ok = load(&k_map, smem_u32(&k_full[s]), smem_u32(&k_empty[s]), dst, par, y0, y1);
                if (!ok) break;
                kit = it + 1;
                if (bk == 0) {
                    // K of the first block goes first: its stage frees before the
                    // previous piece's last S is done, which is what Q waits for.
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
                ok = ok && load(&v_map, smem_u32(&v_full[s]), smem_u32(&v_empty[s]), dst + C::kKBytes, par, y0, y1);
                if (ok) ++it;
            }
        }
        // Drain: every load issued has landed before exit.
        for (uint32_t k = 0; k < (uint32_t)C::kStages && k < kit; ++k) {
            const uint32_t j = kit - 1 - k;
            mbar_wait(smem_u32(&k_full[j % C::kStages]), (j / C::kStages) & 1, kPfTimeoutNs);
        }
        for (uint32_t k = 0; k < (uint32_t)C::kStages && k < it; ++k) {
            const uint32_t j = it - 1 - k;
            mbar_wait(smem_u32(&v_full[j % C::kStages]), (j / C::kStages) & 1, kPfTimeoutNs);
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
        const uint64_t dq = smem_desc(q_s, 16, 1024), dk = smem_desc(st_s, 16, 1024);
        const uint64_t dv = smem_desc(st_s + C::kKBytes, 16384, 1024);
        auto qk = [&](int h, int s, bool one_page) {
            const uint32_t idesc = one_page ? idesc_s64 : idesc_s;
            const uint64_t a0 = dq + (uint64_t)(h * (C::kQBytes >> 4));
            const uint64_t b0 = dk + (uint64_t)(s * (C::kStageBytes >> 4));
            #pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                umma_f16kind(tmem + 128u * h, a0 + (uint64_t)((ks >> 2) * 1024 + (ks & 3) * 2),
                             b0 + (uint64_t)((ks >> 2) * 1024 + (ks & 3) * 2), idesc, ks > 0 ? 1u : 0u);
            umma_commit(smem_u32(&bars.s_full[h]));
        };
        auto pv = [&](int h, uint32_t j, int s, bool first, bool one_page) -> bool {
            if (!warp_wait(smem_u32(&bars.p_full[h]), j & 1, abort, ctrl)) return false;
            tc_fence_after();
            const uint64_t b0 = dv + (uint64_t)(s * (C::kStageBytes >> 4));
            #pragma unroll
            for (int ks = 0; ks < 8; ++ks)
                if (ks < 4 || !one_page)
                    umma_f16kind_ts(tmem + C::kColO + h * D, tmem + 128u * h + ks * 8, b0 + (uint64_t)(ks * 128),
                                    idesc_o, (first && ks == 0) ? 0u : 1u);
            return true;
        };
        // Blocks of successive pieces form one stream, one step per block (and
        // a last one for the end): for each half, the PV of the pending block
        // (possibly the previous piece's last), then the S of this one.
        constexpr uint32_t kPend = 1, kPendFirst = 2, kPendLast = 4, kPendOne = 8, kPendB = 16, kEnd = 32;
        uint32_t it = 0, uq0 = 0, uq1 = 0, cs0 = 0, cs1 = 0, f = 0;   // blocks; pieces / S per half; flags
        int nh = 0, nblk = 0, bk = 0, pages = 0;                      // the current piece and block
        for (uint32_t k = 0; ok;) {
            if (bk >= nblk) {                                         // the piece is done: the next one
                if (nblk > 0) {
                    ++uq0;
                    if (nh == 2) ++uq1;
                }
                Piece p;
                ok = take_piece(bars, ring, k++, lane, abort, ctrl, p);
                if (!ok) break;
                nblk = uni(p.nblk);
                nh = nblk > 0 ? uni(p.ntok > a.tile_tokens / 2 ? 2 : 1) : 0;
                pages = uni(p.npg - 2 * p.k0);
                bk = 0;
                if (nblk == 0) f |= kEnd;
            }
            const int s = it % C::kStages;
            const bool one = pages - 2 * bk == 1;
            #pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                if ((f & kPend) && (h == 0 || (f & kPendB))) {
                    if (h == 0) {
                        ok = warp_wait(smem_u32(&v_full[(it - 1) % C::kStages]), ((it - 1) / C::kStages) & 1, abort, ctrl);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    ok = pv(h, (h ? cs1 : cs0) - 1, (it - 1) % C::kStages, f & kPendFirst, f & kPendOne);
                    if (!ok) break;
                    if (f & kPendLast) umma_commit(smem_u32(&bars.o_done[h]));
                }
                if (h < nh) {
                    if (h == 0) {
                        ok = warp_wait(smem_u32(&k_full[s]), (it / C::kStages) & 1, abort, ctrl);
                        if (!ok) break;
                    }
                    if (bk == 0) {
                        ok = warp_wait(smem_u32(&bars.q_full[h]), (h ? uq1 : uq0) & 1, abort, ctrl);
                        if (!ok) break;
                    }
                    tc_fence_after();
                    issued = true;
                    qk(h, s, one);
                }
            }
            if (!ok) break;
            if (f & kPend) umma_commit(smem_u32(&v_empty[(it - 1) % C::kStages]));   // the pending block's PV issued
            if (f & kEnd) break;
            umma_commit(smem_u32(&k_empty[s]));                                       // this block's S issued
            const bool last = bk + 1 >= nblk;
            if (last) {
                umma_commit(smem_u32(&bars.q_empty[0]));
                if (nh == 2) umma_commit(smem_u32(&bars.q_empty[1]));
            }
            f = kPend | (bk == 0 ? kPendFirst : 0) | (last ? kPendLast : 0) | (one ? kPendOne : 0) |
                (nh == 2 ? kPendB : 0);
            ++cs0;
            if (nh == 2) ++cs1;
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

template <int D>
cudaError_t launch_d(const SharedArgs& a, const CUtensorMap& q_map, const CUtensorMap& k_map, const CUtensorMap& v_map,
                     int grid, cudaStream_t stream) {
    using C = ShCfg<D>;
    auto kern = shared_prefix_kernel<D>;
    static int configured_mask = 0;   // bit per device id < 31
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 31 || !(__atomic_load_n(&configured_mask, __ATOMIC_ACQUIRE) & (1 << dev))) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 31) __atomic_fetch_or(&configured_mask, 1 << dev, __ATOMIC_ACQ_REL);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kShThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, q_map, k_map, v_map, a);
}

}  // namespace

cudaError_t launch_shared_prefix(const SharedArgs& a, const CUtensorMap& q_map, const CUtensorMap& k_map,
                                 const CUtensorMap& v_map, int grid, cudaStream_t stream) {
    if (a.head_dim == 128) return launch_d<128>(a, q_map, k_map, v_map, grid, stream);
    if (a.head_dim == 64) return launch_d<64>(a, q_map, k_map, v_map, grid, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pdattn
