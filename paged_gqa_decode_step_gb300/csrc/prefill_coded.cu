// Prefill attention over a coded (8-bit) paged cache on the tensor cores.
//
// The dataflow is prefill.cu's: a unit is a tile of up to 256 / g tokens of
// one row times one kv head, in two halves of 128 MMA rows; per block of 128
// keys S = Q K^T, softmax with one thread per row, P over S's columns in
// tensor memory, O += P V.  What differs:
//
//   * Codes.  Four converter warps read a block's codes straight from the
//     cache (contiguous pages, one block ahead, in registers) and store
//     K' = code * r as f16 where the MMA reads it; r = scale / ref in (0, 2^7]
//     with ref a power of two (448 * 2^7 is an f16).  The block's scores are
//     multiplied by K's ref; a row's O is in units of V's, which seldom changes
//     along a unit (O is rescaled when it grows).  r and code * r round to
//     f16's 11 bits (2^-12 of the value, against 2^-9 for bf16).  Converting
//     once per unit and block costs each SM 12 codes per clock at full MMA
//     rate.  Multiplying the scales into S and P instead would put two more
//     instructions per score into the softmax, which bounds the kernel.
//   * Blocks with a scale further than 2^kSpread below its ref do just that
//     (wide_block): ratios to one ref would run out of f16's exponents, and a
//     key that a query does not see must not take bits off those it sees.
//     There K' and V' are the codes (V' times 2^7), and a row takes its V ref
//     from the keys it sees.  Rows that come to a block of a lower V ref than
//     their own, or whose scores may be too large for the exponent's FMA
//     (kFarFactor), go the same way.
//   * Types.  Q comes as f16 rows with a factor each (code_kernel), P is f16
//     kept 2^7 above the usual scale: f16's 11 bits hold all weights above
//     2^-21 of the largest.
//   * Long rows in few tiles are split along their keys (the planner's
//     sub-tiles): a piece writes its own output, maximum and sum, and a
//     second kernel merges them.
//   * A tile that fits one half (up to 128 / g tokens: drafted tokens, the
//     end of a prompt) alternates: both halves hold its queries, half A takes
//     the even blocks and half B the odd ones, so that one softmax still runs
//     under the other half's MMAs; half A's epilogue merges the two sums.
//   * What the coding launch writes (codes, scales, query factors) is read past
//     L1: this grid may have started before that launch ended, so the data is
//     not constant while it runs.
//   * A key or value that stands for NaN makes its K' row NaN and its V' row
//     zero: the weights of exactly the queries that see it become NaN.
//
// Warps: 0 takes units (with their page ids, some blocks ahead), 1 issues
// MMAs, 2 loads Q (TMA), 3 describes the blocks (pages, refs, ratios) a few
// ahead of their use; 4 to 7 convert; 8 to 11 and 12 to 15 are the softmax and
// epilogue of the halves.  Waits are bounded as in prefill.cu.
#include <cfloat>
#include <climits>

#include "coded.cuh"
#include "internal.h"
#include "umma.cuh"

namespace pdattn {
namespace {

constexpr int kCpThreads = 512;
constexpr float kRescale = 8.0f;    // lazy rescale threshold (log2 units)
constexpr float kPBias = 7.0f;      // weights are kept 2^7 up: at most 2^(kRescale + kPBias) = 2^15
// A product of f16 query and K' is below 2^24 (elements below 2 and 448 * 2^7, D
// up to 128), so a score is below 2^23 for factors up to this.  Beyond, an FMA
// with the rounded maximum could leave more than the half by which a weight's
// exponent may grow (2^16 is no f16).
constexpr float kFarFactor = 0.5f;
constexpr int kDescs = 8;           // ring of block descriptors, longer than any stage ring
// A scale's exponent below its block's ref, at most: f16 has 14 below 1.  (8 x 1024
// tokens 550 us; with tokens of log-normal sizes, sigma 1, 576; with every block
// past the spread 2.73 ms.)
constexpr int kSpread = 13;
constexpr int kUp = 7;              // ratios reach 2^kUp
constexpr float kVWide = 128.f;     // V ratio of a wide block, so that its rows' refs are like those of others
constexpr int kRoom = 3;            // room that a unit's first V ref leaves, in exponents

template <int D>
struct CpCfg {
    static constexpr int kBoxes = D / 64;                 // 64-element column boxes
    static constexpr int kQBytes = kBoxes * 16384;        // one half: 128 rows x 128 B per box
    static constexpr int kKBytes = kBoxes * 16384;        // K' (or V') of a block: 128 keys x 128 B per box
    static constexpr int kStageBytes = 2 * kKBytes;
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int kOffStage = 2 * kQBytes;
    static constexpr int kSmem = kOffStage + kStages * kStageBytes + 1024;   // + alignment slack
    static constexpr uint32_t kTmemCols = 512;            // S of half h at 128 h, O at 256 + h D
    static constexpr uint32_t kColO = 256;
    static_assert(kStages < kDescs, "a block's descriptor outlives its stage");
};

constexpr int kUnitSlots = 4;
constexpr int kUnitReaders = 11;     // the issuing, the Q and the block warp, and eight softmax warps
// Blocks queued before the next unit is taken: short units queue up, long ones do
// not hold back work that other CTAs could take.  (2, 6 and 12: drafted tokens
// 110.3, 108.2 and 107.6 us, four prompts of 50 to 300 tokens 51.1, 55.3 and 55.0.)
constexpr int kBlocksAhead = 6;

// warp_wait with its polling loop out of line: some thirty waits with the loop
// in place would crowd the instruction cache.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, Ctrl* ctrl) {
    return warp_wait(bar, parity, abort, ctrl);
}

__device__ __forceinline__ bool cwait(uint32_t bar, uint32_t parity, volatile int* abort, Ctrl* ctrl) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    return wait_slow(bar, parity, abort, ctrl);
}

struct CpBars {
    uint64_t alt_full, alt_free;     // alternating units: half B's sums written / half A has merged them
    uint64_t q_full[2], q_empty[2];
    uint64_t mma_done;
    uint64_t unit_full[kUnitSlots], unit_empty[kUnitSlots];
    uint64_t s_full[2], p_full[2], o_done[2];
    uint64_t k_ready[4], k_empty[4], v_ready[4], v_empty[4];   // [stage]
    uint64_t desc_full[kDescs], desc_empty[kDescs];
};

struct __align__(32) UnitSlot {
    PfTile t;
    int u;
    int pad[7];
    int pids[32];                    // the unit's first page ids
};

// A block of 128 keys: the first rows of its two pages in the pools (y1 -1: one
// page; y0 -1: the end of the work), whether the tile sees every key, the refs,
// whether the softmax applies each key's scales (wide) in their place, and per
// key the K ratio (low half) and the V ratio.
struct __align__(16) BlockDesc {
    int y0, y1, all_in, pad;
    float k_ref, v_ref;
    int wide, pad2;
    uint32_t ratio[128];
};

// Half B's (maximum, sum, V ref) of an alternating unit, by row.
struct AltSums {
    float mu[128], l[128], v_ref[128];
};

// Blocks and halves of a unit: an alternating unit's half h takes blocks h,
// h + 2, ...; otherwise each present half takes all of them.
__device__ __forceinline__ bool alternates(const PfTile& t, int Tq) { return t.ntok <= Tq && t.npg > 2; }

// The next unit from the producer's ring (whole warp) and its tile: -1 once
// there is no more work, -2 on abort.
__device__ __forceinline__ int take_unit(CpBars& bars, const UnitSlot* s_unit, uint32_t k, int lane,
                                         volatile int* abort, Ctrl* ctrl, PfTile& t, int* pid = nullptr) {
    const int slot = k % kUnitSlots;
    if (!cwait(smem_u32(&bars.unit_full[slot]), (k / kUnitSlots) & 1, abort, ctrl)) return -2;
    const volatile int4* src = reinterpret_cast<const volatile int4*>(&s_unit[slot]);
    const int4 t0 = make_int4(src[0].x, src[0].y, src[0].z, src[0].w);
    const int4 t1 = make_int4(src[1].x, src[1].y, src[1].z, src[1].w);
    const int u = src[2].x;
    t.t0 = t0.x; t.ntok = t0.y; t.row = t0.z; t.first_page = t0.w;
    t.npg = t1.x; t.lo_min = t1.y; t.pos_max = t1.z; t.pad = t1.w;
    if (pid) *pid = reinterpret_cast<const volatile int*>(s_unit[slot].pids)[lane];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars.unit_empty[slot]));
    return u;
}

// ---------------------------------------------------------------------------
// MMA sequences.  The issuing warp bounds short and long rows alike, and with
// four code streams per scheduler an instruction of it costs some ten clocks:
// a block's MMAs and their commits are one run of code under one elected lane,
// with conditions as predicates and descriptors whose upper words (constant,
// see smem_desc) need no carry.
// ---------------------------------------------------------------------------
#define PDATTN_MMA_SS(off, pred, acc)                                                                       \
    "add.u32 x, %1, " off ";\n add.u32 y, %2, " off ";\n mov.b64 a, {x, %5};\n mov.b64 b, {y, %5};\n"       \
    "@" pred " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, " acc ";\n"
#define PDATTN_MMA_TS(aoff, boff, pred, acc)                                                                \
    "add.u32 x, %1, " aoff ";\n add.u32 y, %2, " boff ";\n mov.b64 b, {y, %5};\n"                          \
    "@" pred " tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, " acc ";\n"
#define PDATTN_COMMIT(pred, bar)                                                                            \
    "@" pred " tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [" bar "];\n"

// Upper word of the descriptors: stride 1024 bytes, version 1, 128-byte swizzle.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;

// S = Q K^T over D dimensions; then the commits of S, and if so flagged of the
// Q tile (bit 0) and of K's stage (bit 1).
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t s_tmem, uint32_t q_lo, uint32_t k_lo, uint32_t idesc, uint32_t s_full,
                                         uint32_t q_empty, uint32_t k_empty, uint32_t flags) {
    if constexpr (D == 128)
        asm volatile(
            "{\n .reg .pred e, f, t, c0, c1;\n .reg .b32 x, y;\n .reg .b64 a, b;\n elect.sync _|e, 0xffffffff;\n"
            " setp.ne.u32 t, 0, 0;\n not.pred f, t;\n and.b32 x, %4, 1;\n setp.ne.and.u32 c0, x, 0, e;\n"
            " and.b32 y, %4, 2;\n setp.ne.and.u32 c1, y, 0, e;\n"
            PDATTN_MMA_SS("0", "e", "t") PDATTN_MMA_SS("2", "e", "f") PDATTN_MMA_SS("4", "e", "f")
            PDATTN_MMA_SS("6", "e", "f") PDATTN_MMA_SS("1024", "e", "f") PDATTN_MMA_SS("1026", "e", "f")
            PDATTN_MMA_SS("1028", "e", "f") PDATTN_MMA_SS("1030", "e", "f")
            PDATTN_COMMIT("e", "%6") PDATTN_COMMIT("c0", "%7") PDATTN_COMMIT("c1", "%8") "}"
            ::"r"(s_tmem), "r"(q_lo), "r"(k_lo), "r"(idesc), "r"(flags), "n"(kDescHi), "r"(s_full), "r"(q_empty),
              "r"(k_empty)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred e, f, t, c0, c1;\n .reg .b32 x, y;\n .reg .b64 a, b;\n elect.sync _|e, 0xffffffff;\n"
            " setp.ne.u32 t, 0, 0;\n not.pred f, t;\n and.b32 x, %4, 1;\n setp.ne.and.u32 c0, x, 0, e;\n"
            " and.b32 y, %4, 2;\n setp.ne.and.u32 c1, y, 0, e;\n"
            PDATTN_MMA_SS("0", "e", "t") PDATTN_MMA_SS("2", "e", "f") PDATTN_MMA_SS("4", "e", "f")
            PDATTN_MMA_SS("6", "e", "f")
            PDATTN_COMMIT("e", "%6") PDATTN_COMMIT("c0", "%7") PDATTN_COMMIT("c1", "%8") "}"
            ::"r"(s_tmem), "r"(q_lo), "r"(k_lo), "r"(idesc), "r"(flags), "n"(kDescHi), "r"(s_full), "r"(q_empty),
              "r"(k_empty)
            : "memory");
}

// O (+)= P V over a block's keys, one page of them with kOne; then the commits
// that the flags ask for.
constexpr uint32_t kPend = 1, kFirst = 2, kLast = 4, kOne = 8, kFrees = 16;
__device__ __forceinline__ void issue_pv(uint32_t o_tmem, uint32_t p_tmem, uint32_t v_lo, uint32_t idesc,
                                         uint32_t v_empty, uint32_t o_done, uint32_t flags) {
    asm volatile(
        "{\n .reg .pred e, f, t, two, c0, c1;\n .reg .b32 x, y;\n .reg .b64 b;\n elect.sync _|e, 0xffffffff;\n"
        " and.b32 x, %4, 2;\n setp.eq.u32 t, x, 0;\n setp.eq.u32 f, 0, 0;\n"
        " and.b32 y, %4, 8;\n setp.eq.and.u32 two, y, 0, e;\n and.b32 x, %4, 16;\n setp.ne.and.u32 c0, x, 0, e;\n"
        " and.b32 y, %4, 4;\n setp.ne.and.u32 c1, y, 0, e;\n"
        PDATTN_MMA_TS("0", "0", "e", "t") PDATTN_MMA_TS("8", "128", "e", "f") PDATTN_MMA_TS("16", "256", "e", "f")
        PDATTN_MMA_TS("24", "384", "e", "f") PDATTN_MMA_TS("32", "512", "two", "f") PDATTN_MMA_TS("40", "640", "two", "f")
        PDATTN_MMA_TS("48", "768", "two", "f") PDATTN_MMA_TS("56", "896", "two", "f")
        PDATTN_COMMIT("c0", "%6") PDATTN_COMMIT("c1", "%7") "}"
        ::"r"(o_tmem), "r"(p_tmem), "r"(v_lo), "r"(idesc), "r"(flags), "n"(kDescHi), "r"(v_empty), "r"(o_done)
        : "memory");
}
#undef PDATTN_MMA_SS
#undef PDATTN_MMA_TS
#undef PDATTN_COMMIT

// ---------------------------------------------------------------------------
// The block warp: descriptors of the unit stream's blocks.
// ---------------------------------------------------------------------------
constexpr uint32_t kAboveZeros = 0x00800001u;   // the scale after 2^-126
constexpr uint32_t kScaleEnd = 0x7e000000u;     // 2^125: no scale of a finite key or value reaches it

// The lowest ref for a scale, 2^-kUp of the power of two at or above it, as a
// biased exponent in [1, 243] (finite keys and values have scales of at most
// 2^122).
__device__ __forceinline__ int ref_exp(uint32_t bits) {
    const int e = (int)(bits >> 23) + ((bits & 0x7fffffu) != 0);
    return min(max(e - kUp, 1), 243);
}

template <int D>
__device__ __forceinline__ void block_warp(const CodedPrefillArgs& ca, int lane, CpBars& bars, const UnitSlot* s_unit,
                                           BlockDesc* s_desc, volatile int* abort, Ctrl* ctrl) {
    // Descriptor n goes where n - kDescs was.  The softmax may read that one
    // until its block's PV is issued, which the conversion of the V kStages
    // blocks later has waited for.
    constexpr uint32_t kAhead = kDescs - CpCfg<D>::kStages;
    const PrefillArgs& a = ca.a;
    const int Hk = a.kv_heads;
    uint32_t n = 0;
    for (uint32_t k = 0;; ++k) {
        PfTile t;
        int pid_cur = 0;
        const int u = take_unit(bars, s_unit, k, lane, abort, ctrl, t, &pid_cur);
        if (u == -2) return;
        const int npg = u < 0 ? 1 : t.npg, kvh = u < 0 ? 0 : u % Hk;
        const int* trow = u < 0 ? nullptr : a.table + (size_t)t.row * a.pages_per_row + t.first_page;
        int pid_base = 0, pid_nxt = u >= 0 && 32 + lane < npg ? __ldg(trow + 32 + lane) : 0;
        auto page_row = [&](int pi) -> int {
            if (pi - pid_base >= 32) {          // pages are visited in order, 32 ids at a time
                pid_cur = pid_nxt;
                pid_base += 32;
                pid_nxt = pid_base + 32 + lane < npg ? __ldg(trow + pid_base + 32 + lane) : 0;
            }
            int page = __shfl_sync(0xffffffffu, pid_cur, pi & 31);
            if (page < 0 || page >= a.num_pages) {
                if (lane == 0) set_error(ctrl, kErrBadPage);
                page = 0;
            }
            return (page * Hk + kvh) * kPageSize;
        };
        int v_run = 1;                          // biased exponent of the V ref before
        #pragma unroll 1
        for (int bk = 0; 2 * bk < npg; ++bk, ++n) {
            int y0 = -1, y1 = -1;
            float ks[4] = {}, vs[4] = {};
            if (u >= 0) {
                y0 = page_row(2 * bk);
                if (2 * bk + 1 < npg) y1 = page_row(2 * bk + 1);
                const int y = lane < 16 ? y0 : y1;
                if (y >= 0) {
                    const float4 kq = __ldcg(reinterpret_cast<const float4*>(ca.k_scale + y) + (lane & 15));
                    const float4 vq = __ldcg(reinterpret_cast<const float4*>(ca.v_scale + y) + (lane & 15));
                    ks[0] = kq.x; ks[1] = kq.y; ks[2] = kq.z; ks[3] = kq.w;
                    vs[0] = vq.x; vs[1] = vq.y; vs[2] = vq.z; vs[3] = vq.w;
                }
            }
            if (n >= kAhead) {
                const uint32_t m = n - kAhead;
                if (!cwait(smem_u32(&bars.desc_empty[m % kDescs]), (m / kDescs) & 1, abort, ctrl)) return;
            }
            const int key0 = (t.first_page + 2 * bk) * kPageSize, key_end = key0 + (y1 >= 0 ? 128 : 64);
            const bool all_in = key0 >= t.lo_min && key_end - 1 <= t.pos_max && y1 >= 0;
            uint32_t kb[4], vb[4];
            #pragma unroll
            for (int e = 0; e < 4; ++e) {
                kb[e] = __float_as_uint(ks[e]);
                vb[e] = __float_as_uint(vs[e]);
            }
            uint32_t outside = 0, bad = 0;          // bits: this lane's keys out of range, and of no finite scale
            if (!all_in) {
                #pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = key0 + 4 * lane + e;
                    if (key < t.lo_min || key > t.pos_max) {
                        outside |= 1u << e;
                        kb[e] = vb[e] = 0u;
                    }
                }
            }
            // largest scales, and smallest ones above 2^-126, which zeros have (they
            // lose nothing): the difference wraps for that and for 0
            uint32_t kmax, vmax;
            #pragma unroll 1
            while (true) {
                kmax = __reduce_max_sync(0xffffffffu, max(max(kb[0], kb[1]), max(kb[2], kb[3])));
                vmax = __reduce_max_sync(0xffffffffu, max(max(vb[0], vb[1]), max(vb[2], vb[3])));
                if (__builtin_expect(max(kmax, vmax) < kScaleEnd, 1)) break;
                #pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (max(kb[e], vb[e]) >= kScaleEnd) {
                        bad |= 1u << e;
                        kb[e] = vb[e] = 0u;
                    }
            }
            const uint32_t kmin = min(min(kb[0] - kAboveZeros, kb[1] - kAboveZeros), min(kb[2] - kAboveZeros, kb[3] - kAboveZeros));
            const uint32_t vmin = min(min(vb[0] - kAboveZeros, vb[1] - kAboveZeros), min(vb[2] - kAboveZeros, vb[3] - kAboveZeros));
            const int k_exp = ref_exp(kmax);
            // V keeps the ref of the block before unless its own scales are larger or
            // the smallest much smaller; a new ref leaves them room to grow
            const int v_own = ref_exp(vmax);
            int v_exp = v_run >= v_own ? v_run : v_own + kRoom;
            auto far_below = [&](uint32_t least, int ref) { return least < (uint32_t)max(ref - kSpread - 1, 0) << 23; };
            bool wide = __any_sync(0xffffffffu, far_below(kmin, k_exp) || far_below(vmin, v_exp));
            if (__builtin_expect(wide, 0)) {
                // the highest ref that V's smallest scale allows, if it serves the largest
                const int most = (int)((__reduce_min_sync(0xffffffffu, vmin) + kAboveZeros) >> 23) + kSpread - 1;
                if (most >= v_own) v_exp = min(v_exp, most);
                wide = __any_sync(0xffffffffu, far_below(kmin, k_exp) || far_below(vmin, v_exp));
            }
            v_run = v_exp;
            const float k_down = __uint_as_float((uint32_t)(254 - k_exp) << 23);
            const float v_down = __uint_as_float((uint32_t)(254 - v_exp) << 23);
            uint32_t own[4];
            #pragma unroll
            for (int e = 0; e < 4; ++e)
                own[e] = pack_f16x2(__uint_as_float(kb[e]) * k_down, __uint_as_float(vb[e]) * v_down);
            if (__builtin_expect(wide, 0)) {
                #pragma unroll
                for (int e = 0; e < 4; ++e) own[e] = outside >> e & 1 ? 0u : 0x58003c00u;   // K 1, V kVWide
            }
            if (__builtin_expect(bad != 0, 0)) {
                #pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (bad >> e & 1) own[e] = 0x7e00u;               // K ratio NaN, V ratio 0
            }
            // The converters load one operand ahead, 16 KB: enough for L2's
            // latency but not for HBM's, so the pages go to L2 from here.
            if (lane < 4) {
                const int y = lane & 1 ? y1 : y0;
                if (y >= 0) prefetch_l2_bulk((lane < 2 ? ca.k : ca.v) + (size_t)y * D, kPageSize * D);
            }
            BlockDesc& d = s_desc[n % kDescs];
            *reinterpret_cast<uint4*>(d.ratio + 4 * lane) = make_uint4(own[0], own[1], own[2], own[3]);
            if (lane == 0) {
                *reinterpret_cast<int4*>(&d) = make_int4(y0, y1, all_in ? 1 : 0, 0);
                *reinterpret_cast<int4*>(&d.k_ref) = make_int4(k_exp << 23, v_exp << 23, wide ? 1 : 0, 0);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars.desc_full[n % kDescs]));
        }
        if (u < 0) return;
    }
}

// ---------------------------------------------------------------------------
// Converters: codes of the unit stream's blocks to f16, K by two warps and V
// by two.  (Four warps that take K and V in turn meet twice the barriers:
// drafted tokens 116 us against 111.)
// ---------------------------------------------------------------------------
template <int D, typename Code>
__device__ __forceinline__ void convert_warp(const CodedPrefillArgs& ca, int cw, int lane, uint8_t* stages, CpBars& bars,
                                             const BlockDesc* s_desc, volatile int* s_blocks, volatile int* abort,
                                             Ctrl* ctrl) {
    using C = CpCfg<D>;
    // A thread takes 16 codes of four keys (32 j + 16 w + 8 part + lane / 4,
    // j = 0..3) from each 64-column box, in two parts: eight lanes then store
    // the even 16-byte chunks of one key and the odd ones of the next, which
    // fill the eight bank groups, and every address is a constant away from two
    // bases.
    constexpr int kKeys = 4, kPer = kKeys * C::kBoxes;
    const bool is_k = cw < 2;
    const int kx = lane >> 2, w16 = (cw & 1) * 16;
    const uint8_t* pool = (is_k ? ca.k : ca.v) + (size_t)(w16 + kx) * D + (lane & 3) * 16;
    const uint32_t pick = is_k ? 0x1010 : 0x3232;
    uint64_t* ready = is_k ? bars.k_ready : bars.v_ready;
    uint64_t* empty = is_k ? bars.k_empty : bars.v_empty;
    stages += (is_k ? 0 : C::kKBytes) + w16 * 128 + kx * 128;
    const int dst0 = ((2 * (lane & 3)) ^ kx) << 4, dst1 = ((2 * (lane & 3) + 1) ^ kx) << 4;
    uint4 r[kPer];                              // the next part's codes: key i / boxes, box i % boxes
    auto fetch = [&](int i, const uint8_t* p0, const uint8_t* p1, bool two) {
        const int j = i / C::kBoxes;
        if (j < kKeys / 2 || two)
            r[i] = __ldcg(reinterpret_cast<const uint4*>((j < kKeys / 2 ? p0 : p1) + (j & 1) * 32 * D + (i % C::kBoxes) * 64));
    };
    if (!cwait(smem_u32(&bars.desc_full[0]), 0, abort, ctrl)) return;
    uint4 d = lds128(smem_u32(&s_desc[0]));     // y0, y1, all_in
    if ((int)d.x < 0) return;
    #pragma unroll
    for (int i = 0; i < kPer; ++i)
        fetch(i, pool + (size_t)d.x * D, pool + (size_t)max((int)d.y, 0) * D, (int)d.y >= 0);
    #pragma unroll 1
    for (uint32_t it = 0;; ++it) {
        const int st = it % C::kStages;
        const bool two = (int)d.y >= 0, all_in = d.z != 0;
        bool more = true;
        #pragma unroll 1
        for (int part = 0; part < 2; ++part) {
            uint32_t r2[kKeys];
            #pragma unroll
            for (int j = 0; j < kKeys; ++j) {
                const uint32_t rr = s_desc[it % kDescs].ratio[32 * j + w16 + 8 * part + kx];
                r2[j] = __byte_perm(rr, rr, pick);
            }
            if (part == 0) {
                if (!cwait(smem_u32(&empty[st]), (it / C::kStages + 1) & 1, abort, ctrl)) return;
            } else {
                // the next part is the next block's first
                if (!cwait(smem_u32(&bars.desc_full[(it + 1) % kDescs]), ((it + 1) / kDescs) & 1, abort, ctrl)) return;
                d = lds128(smem_u32(&s_desc[(it + 1) % kDescs]));
                more = (int)d.x >= 0;
            }
            if (!all_in) {
                // a row outside the tile's keys (ratio 0) may hold any codes, e4m3's NaN among them
                #pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (r2[i / C::kBoxes] == 0) r[i] = make_uint4(0, 0, 0, 0);
            }
            const uint8_t* p0 = pool + (size_t)d.x * D + (part == 0 ? 8 * D : 0);
            const uint8_t* p1 = pool + (size_t)max((int)d.y, 0) * D + (part == 0 ? 8 * D : 0);
            const bool next_two = (int)d.y >= 0;
            uint8_t* base = stages + st * C::kStageBytes + part * 1024;
            // each register is refilled as soon as it is converted
            #pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int j = i / C::kBoxes;
                if (j < kKeys / 2 || two) {
                    const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
                    uint32_t h[8];
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        widen4<Code>(w[e], h[2 * e], h[2 * e + 1]);
                        h[2 * e] = mul_f16x2(h[2 * e], r2[j]);
                        h[2 * e + 1] = mul_f16x2(h[2 * e + 1], r2[j]);
                    }
                    uint8_t* to = base + (i % C::kBoxes) * 16384 + j * 4096;
                    *reinterpret_cast<uint4*>(to + dst0) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4*>(to + dst1) = make_uint4(h[4], h[5], h[6], h[7]);
                }
                if (more) fetch(i, p0, p1, next_two);
            }
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(smem_u32(&ready[st]));
            mbar_arrive(smem_u32(&bars.desc_empty[it % kDescs]));
            if (cw == 2) *s_blocks = (int)it + 1;   // progress, for the scheduler
        }
        if (!more) return;
    }
}

// ---------------------------------------------------------------------------
// Softmax and epilogue of one half (128 threads, one MMA row each).
// ---------------------------------------------------------------------------
// Max of 32 values as four short independent chains.
__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
    float acc[4];
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float* v = reinterpret_cast<const float*>(&s[8 * k]);
        float x = fmax3(v[0], v[1], v[2]);
        x = fmax3(x, v[3], v[4]);
        x = fmax3(x, v[5], v[6]);
        acc[k] = fmaxf(x, v[7]);
    }
    return fmaxf(fmax3(acc[0], acc[1], acc[2]), acc[3]);
}

__device__ __forceinline__ float sink_scale(float mu, float l, bool has_sink, float sk) {
    if (!has_sink) return l == 0.f ? 0.f : 1.f / l;
    const float Mp = fmaxf(mu, sk);
    const float f = exp2_approx(mu - Mp);
    return f / (l * f + exp2_approx(sk - Mp));
}

// A row's softmax state: maximum and sum (as softmax_half keeps them) and the
// V ref that its O is in units of.
struct RowState {
    float m, l, v_ref;
};

// Multiplies the rows' O by a factor each, where that seldom comes (whole warp).
template <int D>
__device__ __noinline__ void scale_o(uint32_t o_addr, float f) {
    #pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 8) {
        uint32_t o[8];
        tmem_ld8_wait(o_addr + c0, o);
        #pragma unroll
        for (int c = 0; c < 8; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
        tmem_st8(o_addr + c0, o);
    }
    tmem_wait_st();
}

// The softmax of a block with the scales applied here (whole warp).  Wide: S
// holds the products of queries and K codes, and every key's scales are read
// from the cache, by one lane for its column; otherwise all keys have the
// block's refs for scales.  Scores take K's in f32; a weight takes V's relative
// to the row's V ref, at least what every V scale that the row has seen takes, on
// its way to f16.  Out of line and of 8 columns at a time: it must not
// crowd the loops that other blocks run in, and a call's first such block finds
// none of it in the caches.
template <int D>
__device__ __noinline__ RowState wide_block(uint32_t s_addr, uint32_t o_addr, const float* k_scale,
                                            const float* v_scale, const BlockDesc* desc, float qf, int c_lo, int c_hi,
                                            bool has_o, int lane, RowState st) {
    const uint4 dy = lds128(smem_u32(desc)), dq = lds128(smem_u32(&desc->k_ref));   // y0, y1; k_ref, v_ref, wide
    // the scales of columns 32 q4 + lane
    const float k_blk = __uint_as_float(dq.x), v_blk = __uint_as_float(dq.y) * kVWide;
    auto scale_of = [&](const float* scales, float ref, int q4) {
        const int y = (int)(q4 < 2 ? dy.x : dy.y);
        return dq.z == 0 ? ref : y >= 0 ? __ldcg(scales + y + (q4 & 1) * 32 + lane) : 0.f;
    };
    float ks = 0.f, vs = 0.f, top = -INFINITY, big = 0.f;
    #pragma unroll 1
    for (int c0 = 0; c0 < 128; c0 += 8) {
        if (c0 % 32 == 0) {
            ks = scale_of(k_scale, k_blk, c0 / 32);
            vs = scale_of(v_scale, v_blk, c0 / 32);
        }
        uint32_t x[8];
        tmem_ld8_wait(s_addr + c0, x);
        #pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float f = fminf(qf * __shfl_sync(0xffffffffu, ks, c0 + c), FLT_MAX);
            const float v = __shfl_sync(0xffffffffu, vs, c0 + c);
            if (c0 + c >= c_lo && c0 + c <= c_hi) {
                top = fmaxf(top, __fmul_rn(__uint_as_float(x[c]), f));
                big = fmaxf(big, v);
            }
        }
    }
    float alpha = 1.f;
    if (top > st.m + kRescale) {
        alpha = exp2_approx(st.m - top);
        st.m = top;
        st.l *= alpha;
    }
    const float ref = fmaxf(st.v_ref, __uint_as_float((uint32_t)ref_exp(__float_as_uint(big)) << 23));
    alpha *= st.v_ref / ref;
    st.v_ref = ref;
    if (has_o && __any_sync(0xffffffffu, alpha != 1.f)) scale_o<D>(o_addr, alpha);
    const float down = 1.f / (ref * kVWide);
    #pragma unroll 1
    for (int c0 = 0; c0 < 128; c0 += 8) {
        if (c0 % 32 == 0) {
            ks = scale_of(k_scale, k_blk, c0 / 32);
            vs = scale_of(v_scale, v_blk, c0 / 32);
        }
        uint32_t x[8];
        float w[8];
        tmem_ld8_wait(s_addr + c0, x);
        #pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float f = fminf(qf * __shfl_sync(0xffffffffu, ks, c0 + c), FLT_MAX);
            const float v = __shfl_sync(0xffffffffu, vs, c0 + c);
            w[c] = 0.f;
            if (c0 + c >= c_lo && c0 + c <= c_hi) {
                // (rounded like the maximum, which then differs from itself by nothing)
                const float p = exp2_approx(__fadd_rn(__fmul_rn(__uint_as_float(x[c]), f), -st.m) + kPBias);
                st.l += p;
                w[c] = p * (v * down);
            }
        }
        // over columns of S that have been read
        tmem_st4(s_addr + c0 / 2, pack_f16x2(w[0], w[1]), pack_f16x2(w[2], w[3]), pack_f16x2(w[4], w[5]),
                 pack_f16x2(w[6], w[7]));
    }
    return st;
}

template <int D>
__device__ __forceinline__ void softmax_half(const CodedPrefillArgs& ca, int half, int quarter, int lane, uint32_t tmem,
                                             CpBars& bars, const BlockDesc* s_desc, volatile AltSums& s_alt,
                                             const UnitSlot* s_unit, volatile int* abort, Ctrl* ctrl) {
    using C = CpCfg<D>;
    const PrefillArgs& a = ca.a;
    const int W = a.window, Hk = a.kv_heads, g = a.group, Tq = a.tile_tokens / 2;
    const int m = quarter * 32 + lane;                    // MMA row = TMEM lane
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + 128u * half, o_addr = tmem + lane_base + C::kColO + half * D;
    const int tq = m / g, jh = m % g;
    const __nv_bfloat16* sinks = static_cast<const __nv_bfloat16*>(a.sinks);
    const bool out_wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
    const uint32_t s_full = smem_u32(&bars.s_full[half]), p_full = smem_u32(&bars.p_full[half]);
    uint32_t it = 0, ch = 0, uh = 0, uh_b = 0, ua = 0, k = 0;   // blocks; this half's blocks, units; half B's units; alternating units
    bool ok = true;
    PfTile t;
    int u = take_unit(bars, s_unit, k++, lane, abort, ctrl, t);
    int pos_next = -1;
    float f_next = 1.f;
    auto token_of = [&](const PfTile& tt) { return alternates(tt, Tq) ? tq : half * Tq + tq; };
    auto row_inputs = [&](const PfTile& tt, int uu) {
        const int tok = token_of(tt);
        pos_next = -1;
        if (tq < Tq && tok < tt.ntok) {
            pos_next = __ldg(a.positions + tt.t0 + tok);
            f_next = __ldcg(ca.q_factor + (size_t)(tt.t0 + tok) * a.heads + (uu % Hk) * g + jh);
        }
    };
    if (u >= 0) row_inputs(t, u);
    while (u >= 0) {
        const int kvh = u % Hk, nb = (t.npg + 1) / 2;
        const bool alt = alternates(t, Tq);
        if (half == 1 && t.ntok <= Tq && !alt) {
            it += nb;
            u = take_unit(bars, s_unit, k++, lane, abort, ctrl, t);
            if (u >= 0) row_inputs(t, u);
            continue;
        }
        const int tok = token_of(t);
        const bool active = tq < Tq && tok < t.ntok;
        const bool warp_active = __any_sync(0xffffffffu, active);
        // (a row that holds no query must not keep its warp from skipping masks)
        const int pos = active ? max(pos_next, 0) : INT_MAX;
        const int lo = active && W > 0 && pos - W + 1 > 0 ? pos - W + 1 : 0;
        const float qf = active ? f_next : 0.f;
        float m_run = -INFINITY, l = 0.f, v_ref = kScaleMin;
        const int first = alt ? half : 0, stride = alt ? 2 : 1;
        for (int b = first; b < nb; b += stride) {
            ok = cwait(s_full, ch & 1, abort, ctrl);
            if (!ok) break;
            ++ch;
            tc_fence_after();
            if (!warp_active) {                            // none of this warp's rows is a query
                tc_fence_before();
                if (lane == 0) mbar_arrive(p_full);
                continue;
            }
            const int di = (it + b) % kDescs;
            ok = cwait(smem_u32(&bars.desc_full[di]), ((it + b) / kDescs) & 1, abort, ctrl);
            if (!ok) break;
            const uint4 dq = lds128(smem_u32(&s_desc[di].k_ref));      // k_ref, v_ref, wide
            // a factor that underflows keeps -inf times it at -inf
            const float f = fmaxf(qf * __uint_as_float(dq.x), kScaleMin), v_blk = __uint_as_float(dq.y);
            const int pg0 = t.first_page + 2 * b, key0 = pg0 * kPageSize, npb = min(2, t.npg - 2 * b);
            // keys c of this block visible to the row: c_lo <= c <= c_hi;
            // 32-column chunks visible to every row of the warp skip the test, and
            // those visible to none the exponentials too
            const int c_lo = lo - key0, c_hi = min(pos - key0, npb * kPageSize - 1);
            // (per chunk: 0 wholly visible to the warp, 1 not, 2 wholly hidden)
            int state = 0;
            if (!__all_sync(0xffffffffu, c_lo <= 0 && c_hi >= 2 * kPageSize - 1 && dq.z == 0 && v_ref == v_blk && f <= kFarFactor)) {
                const bool sees = active && c_hi >= max(c_lo, 0);
                // a row takes the V ref of its first keys (its O is zero)
                if (dq.z == 0 && (!active || (sees && m_run == -INFINITY))) v_ref = v_blk;
                const bool apply = dq.z != 0 || f > kFarFactor, other = sees && v_ref != v_blk;
                if (__any_sync(0xffffffffu, apply || other)) {
                    if (__any_sync(0xffffffffu, apply || (other && v_ref > v_blk))) {
                        const RowState st = wide_block<D>(s_addr, o_addr, ca.k_scale, ca.v_scale, &s_desc[di], qf, c_lo,
                                                          c_hi, b > first, lane, RowState{m_run, l, v_ref});
                        m_run = st.m;
                        l = st.l;
                        v_ref = st.v_ref;
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(p_full);
                        continue;
                    }
                    if (b > first) scale_o<D>(o_addr, other ? v_ref / v_blk : 1.f);   // powers of two: exact
                    if (other) v_ref = v_blk;
                }
                #pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                    const int b0 = 32 * q4;
                    const bool in = __all_sync(0xffffffffu, c_lo <= b0 && c_hi >= b0 + 31);
                    const bool out = __all_sync(0xffffffffu, !active || c_lo > b0 + 31 || c_hi < b0);
                    state |= (out ? 2 : in ? 0 : 1) << (2 * q4);
                }
            }
            auto mask = [&](uint32_t (&y)[32], int q4) {
                if (state >> (2 * q4) & 1) {
                    const int from = min(max(c_lo - 32 * q4, 0), 32), to = min(max(c_hi + 1 - 32 * q4, 0), 32);
                    const uint32_t vis = (uint32_t)((1ull << to) - 1) & ~(uint32_t)((1ull << from) - 1);
                    #pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!(vis >> c & 1)) y[c] = __float_as_uint(-INFINITY);
                }
            };
            // Both passes are rolled loops over 32 columns: a scheduler's warps
            // run two softmax halves and a converter, and code that outgrows
            // its instruction cache cost 7 to 15 clocks per instruction
            // (unrolled passes: 1.5 times the kernel's time).  Reading S twice
            // costs 30 clocks per chunk.
            float top = -INFINITY;
            if (state == 0) {
                // the load brings the maximum along
                #pragma unroll 1
                for (int q2 = 0; q2 < 2; ++q2) {
                    uint32_t x[32], y[32];
                    float mx, my;
                    tmem_ld32_max(s_addr + 64 * q2, x, mx);
                    tmem_ld32_max(s_addr + 64 * q2 + 32, y, my);
                    tmem_wait_ld();
                    asm volatile("" : "+f"(mx), "+f"(my));   // no use of them ahead of the wait
                    top = fmax3(top, mx, my);
                }
            } else {
                #pragma unroll 1
                for (int q4 = 0; q4 < 4; ++q4) {
                    if (state >> (2 * q4) & 2) continue;
                    uint32_t x[32];
                    tmem_ld32(s_addr + 32 * q4, x);
                    tmem_wait_ld();
                    mask(x, q4);
                    top = fmaxf(top, max32(x));
                }
            }
            const float mx = top * f;
            const bool need = mx > m_run + kRescale;
            float alpha = 1.f;
            if (need) {
                alpha = exp2_approx(m_run - mx);
                m_run = mx;
                l *= alpha;
            }
            if (b > first && __any_sync(0xffffffffu, alpha != 1.f)) {
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
            const float neg_mu = m_run == -INFINITY ? 0.f : kPBias - m_run;
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            // weights of 32 columns over the first 64 columns of S: chunk q's go
            // over columns that chunks 0 .. q / 2 held, which have been read
            auto weights = [&](const uint32_t (&y)[32], int q4) {
                uint32_t pk[16];
                #pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    float p0, p1;
                    ffma2(p0, p1, __uint_as_float(y[c]), __uint_as_float(y[c + 1]), f, neg_mu);
                    p0 = exp2_approx(p0);
                    p1 = exp2_approx(p1);
                    pk[c >> 1] = pack_f16x2(p0, p1);
                    fadd2(acc[c & 2], acc[(c & 2) + 1], p0, p1);
                }
                tmem_st16(s_addr + 16 * q4, pk);
            };
            #pragma unroll 1
            for (int q4 = 0; q4 < 4; ++q4) {
                uint32_t x[32];
                if (state >> (2 * q4) & 2) {
                    #pragma unroll
                    for (int c = 0; c < 16; ++c) x[c] = 0;
                    tmem_st16(s_addr + 16 * q4, *reinterpret_cast<const uint32_t(*)[16]>(&x[0]));
                    continue;
                }
                tmem_ld32(s_addr + 32 * q4, x);
                tmem_wait_ld();
                if (state != 0) mask(x, q4);
                weights(x, q4);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
            l += (acc[0] + acc[1]) + (acc[2] + acc[3]);
        }
        if (!ok) break;
        PfTile tn;
        const int un = take_unit(bars, s_unit, k++, lane, abort, ctrl, tn);
        if (un >= 0) row_inputs(tn, un);
        ok = cwait(smem_u32(&bars.o_done[half]), uh & 1, abort, ctrl);
        if (!ok) break;
        tc_fence_after();
        const float mu = m_run == -INFINITY ? -1.0e30f : m_run - kPBias;
        if (alt && half == 1) {
            // hand the sums to half A, whose epilogue merges both; O stays
            // until it has (this half's next weights come after alt_free)
            s_alt.mu[m] = mu;
            s_alt.l[m] = l;
            s_alt.v_ref[m] = v_ref;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars.alt_full));
            ok = cwait(smem_u32(&bars.alt_free), ua & 1, abort, ctrl);
            if (!ok) break;
        } else {
            float M = mu, L = l, fa = v_ref, fb = 0.f;     // O = fa O_A + fb O_B
            if (alt) {
                ok = cwait(smem_u32(&bars.o_done[1]), uh_b & 1, abort, ctrl) &&
                     cwait(smem_u32(&bars.alt_full), ua & 1, abort, ctrl);
                if (!ok) break;
                tc_fence_after();
                const float mu_b = s_alt.mu[m];
                M = fmaxf(mu, mu_b);
                const float ea = exp2_approx(mu - M), eb = exp2_approx(mu_b - M);
                L = l * ea + s_alt.l[m] * eb;
                fa = v_ref * ea;
                fb = s_alt.v_ref[m] * eb;
            }
            if (warp_active) {
                const int h = kvh * g + jh;
                float sk = 0.f;
                if (sinks != nullptr && active && t.pad == 0) sk = __bfloat162float(sinks[h]) * 1.4426950408889634f;
                // a piece of a split tile leaves its own output (an unnormalised one
                // could leave f32), maximum and sum
                const float inv = sink_scale(M, L, t.pad == 0 && sinks != nullptr, sk);
                fa *= inv;
                fb *= inv;
                const size_t at = ((size_t)(t.pad - 1) * Hk + kvh) * ca.slot_rows + tok * g + jh;
                if (t.pad != 0 && active) ca.part_ml[at] = make_float2(M, L);
                __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.out) + ((size_t)(t.t0 + tok) * a.heads + h) * D;
                #pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(o_addr + c0, o);
                    tmem_wait_ld();
                    #pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * fa);
                    if (alt) {
                        uint32_t ob[32];
                        tmem_ld32(o_addr + D + c0, ob);
                        tmem_wait_ld();
                        #pragma unroll
                        for (int c = 0; c < 32; ++c)
                            o[c] = __float_as_uint(fmaf(__uint_as_float(ob[c]), fb, __uint_as_float(o[c])));
                    }
                    if (!active) continue;
                    if (t.pad != 0) {
                        float4* dst = reinterpret_cast<float4*>(ca.part_o + at * D + c0);
                        #pragma unroll
                        for (int c = 0; c < 32; c += 4)
                            dst[c / 4] = make_float4(__uint_as_float(o[c]), __uint_as_float(o[c + 1]),
                                                     __uint_as_float(o[c + 2]), __uint_as_float(o[c + 3]));
                        continue;
                    }
                    #pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        uint32_t w[8];
                        #pragma unroll
                        for (int e = 0; e < 8; ++e)
                            w[e] = pack_bf16x2(__uint_as_float(o[16 * v + 2 * e]), __uint_as_float(o[16 * v + 2 * e + 1]));
                        __nv_bfloat16* dst = orow + c0 + 16 * v;
                        if (out_wide) {
                            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                                         ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                                           "r"(w[5]), "r"(w[6]), "r"(w[7])
                                         : "memory");
                        } else {
                            reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                }
            }
            // The next unit's first PV overwrites O only after this read (its
            // p_full arrival follows in program order; half B's, after alt_free).
            tc_fence_before();
            if (alt) {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.alt_free));
            }
        }
        it += nb;
        ++uh;
        if (alt) ++ua;
        if (alt || t.ntok > Tq) ++uh_b;
        u = un;
        t = tn;
    }
}

template <int D, typename Code>
__global__ void __launch_bounds__(kCpThreads, 1)
    prefill_coded_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CodedPrefillArgs ca) {
    using C = CpCfg<D>;
    const PrefillArgs& a = ca.a;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) CpBars bars;
    __shared__ BlockDesc s_desc[kDescs];
    __shared__ UnitSlot s_unit[kUnitSlots];
    __shared__ AltSums s_alt;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_blocks;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    const uint32_t q_s = sb, st_s = sb + C::kOffStage;
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(a.ws + a.L.ctrl);
    volatile int* abort = &s_abort;

    // Rows of the Q tiles that no token fills stay zero.
    for (int i = tid; i < 2 * C::kQBytes / 16; i += kCpThreads) reinterpret_cast<uint4*>(sm)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) {
        for (int s = 0; s < 4; ++s) {
            mbar_init(smem_u32(&bars.k_ready[s]), 2);
            mbar_init(smem_u32(&bars.k_empty[s]), 1);
            mbar_init(smem_u32(&bars.v_ready[s]), 2);
            mbar_init(smem_u32(&bars.v_empty[s]), 1);
        }
        for (int r = 0; r < kDescs; ++r) {
            mbar_init(smem_u32(&bars.desc_full[r]), 1);
            mbar_init(smem_u32(&bars.desc_empty[r]), 4);
        }
        mbar_init(smem_u32(&bars.mma_done), 1);
        for (int k = 0; k < kUnitSlots; ++k) {
            mbar_init(smem_u32(&bars.unit_full[k]), 1);
            mbar_init(smem_u32(&bars.unit_empty[k]), kUnitReaders);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(smem_u32(&bars.q_full[h]), 1);
            mbar_init(smem_u32(&bars.q_empty[h]), 1);
            mbar_init(smem_u32(&bars.s_full[h]), 1);
            mbar_init(smem_u32(&bars.p_full[h]), 4);
            mbar_init(smem_u32(&bars.o_done[h]), 1);
        }
        mbar_init(smem_u32(&bars.alt_full), 4);
        mbar_init(smem_u32(&bars.alt_free), 4);
        s_abort = 0;
        s_blocks = 0;
        fence_barrier_init();
        prefetch_tensormap(&q_map);
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

    // Everything below reads what the planner and the coding launch wrote.
    griddep_launch_dependents();
    griddep_wait();
    const int Hk = a.kv_heads, g = a.group, Tq = a.tile_tokens / 2;
    const int n_units = (ctrl->magic == kCodedPlanMagic ? ctrl->n_items : 0) * Hk;
    const PfTile* tiles = reinterpret_cast<const PfTile*>(a.ws + ca.units);

    if (warp >= 8) {
        softmax_half<D>(ca, (warp - 8) >> 2, warp & 3, lane, tmem, bars, s_desc, s_alt, s_unit, abort, ctrl);
    } else if (warp >= 4) {
        convert_warp<D, Code>(ca, warp - 4, lane, sm + C::kOffStage, bars, s_desc, &s_blocks, abort, ctrl);
    } else {
      if (warp == 0) {
        // ---------------- units ----------------
        bool ok = true;
        int u = blockIdx.x, queued = 0;
        for (uint32_t k = 0; ok; ++k) {
            if (k > 0) {
                int v = 0;
                if (lane == 0) {
                    uint64_t t0 = 0;
                    while (queued - *reinterpret_cast<volatile int*>(&s_blocks) > kBlocksAhead && !*abort) {
                        __nanosleep(256);
                        const uint64_t now = globaltimer_ns();
                        if (t0 == 0) {
                            t0 = now;
                        } else if (now - t0 > kPfTimeoutNs) {
                            *abort = 1;
                            set_error(ctrl, kErrTimeout);
                        }
                    }
                    v = (int)gridDim.x + atomicAdd(&ctrl->next_item, 1);
                }
                u = __shfl_sync(0xffffffffu, v, 0);
            }
            const int slot = k % kUnitSlots;
            PfTile t = {};
            int pid = 0;
            if (u < n_units) {
                t = tiles[u / Hk];
                if (lane < t.npg) pid = __ldg(a.table + (size_t)t.row * a.pages_per_row + t.first_page + lane);
            }
            ok = cwait(smem_u32(&bars.unit_empty[slot]), ((k / kUnitSlots) & 1) ^ 1, abort, ctrl);
            if (!ok) break;
            if (lane == 0) {
                int4* dst = reinterpret_cast<int4*>(&s_unit[slot]);
                dst[0] = make_int4(t.t0, t.ntok, t.row, t.first_page);
                dst[1] = make_int4(t.npg, t.lo_min, t.pos_max, t.pad);
                dst[2] = make_int4(u < n_units ? u : -1, 0, 0, 0);
            }
            s_unit[slot].pids[lane] = pid;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars.unit_full[slot]));
            if (u >= n_units) break;
            queued += (t.npg + 1) / 2;
        }
      } else if (warp == 3) {
        block_warp<D>(ca, lane, bars, s_unit, s_desc, abort, ctrl);
      } else if (warp == 2) {
        // ---------------- Q (whole warp, one lane issues) ----------------
        uint32_t uq[2] = {0, 0};     // units whose Q half h was loaded
        bool ok = true;
        for (uint32_t k = 0; ok; ++k) {
            PfTile t;
            const int u = take_unit(bars, s_unit, k, lane, abort, ctrl, t);
            if (u < 0) break;
            const bool alt = alternates(t, Tq);
            const int kvh = uni(u % Hk), nh = uni(alt || t.ntok > Tq ? 2 : 1), t0 = uni(t.t0), step = uni(alt ? 0 : Tq);
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!ok || h >= nh) break;
                ok = cwait(smem_u32(&bars.q_empty[h]), (uq[h] & 1) ^ 1, abort, ctrl);
                if (!ok) break;
                const uint32_t qf = smem_u32(&bars.q_full[h]);
                elect_arrive_expect_tx(qf, C::kBoxes * 128 * g * Tq);
                for (int b = 0; b < C::kBoxes; ++b)
                    elect_tma_3d(q_s + h * C::kQBytes + b * 16384, &q_map, b * 64, kvh * g, t0 + h * step, qf);
                ++uq[h];
            }
        }
        // Drain: every load issued has landed before exit.
        #pragma unroll
        for (int h = 0; h < 2; ++h)
            if (uq[h] > 0) mbar_wait(smem_u32(&bars.q_full[h]), (uq[h] - 1) & 1, kPfTimeoutNs);
      } else if (warp == 1) {
        // ---------------- MMA issuer (as in prefill.cu) ----------------
        constexpr uint32_t idesc_s = instr_desc(128, 128, 0, 0, 0);
        constexpr uint32_t idesc_s64 = instr_desc(128, 64, 0, 0, 0);    // a block of one page
        constexpr uint32_t idesc_o = instr_desc(128, D, 0, 1, 0);
        bool issued = false;
        bool ok = true;
        const uint32_t q_lo = (uint32_t)smem_desc(q_s, 16, 1024), k_lo = (uint32_t)smem_desc(st_s, 16, 1024);
        const uint32_t v_lo = (uint32_t)smem_desc(st_s + C::kKBytes, 16384, 1024);
        // Blocks of successive units form one stream.  A step takes one block:
        // for each half that works on it, the half's pending PV (of its
        // previous block), then S of this block.  A pending PV of the unit
        // before goes out at the next unit's first step in any case.  The
        // half loop stays rolled so that each MMA sequence is issued from one
        // place; per-half state is selected by value.
        uint32_t it = 0, uq0 = 0, uq1 = 0;               // blocks; units per half
        uint32_t cs0 = 0, cs1 = 0, f0 = 0, f1 = 0;       // S issued per half; flags of the pending PV
        uint32_t pit0 = 0, pit1 = 0;                     // its block
        int nh = 0, npg = 0, bk = 0;                     // the current unit and block
        bool alt = false, end = false;
        for (uint32_t k = 0; ok;) {
            if (2 * bk >= npg) {                         // the unit is done: the next one
                if (npg > 0) {
                    ++uq0;
                    if (nh == 2) ++uq1;
                }
                PfTile t;
                const int u = take_unit(bars, s_unit, k++, lane, abort, ctrl, t);
                if (u == -2) {
                    ok = false;
                    break;
                }
                nh = 0;
                npg = 0;
                bk = 0;
                alt = false;
                end = u < 0;
                if (u >= 0) {
                    alt = uni(alternates(t, Tq) ? 1 : 0);
                    nh = uni(alt || t.ntok > Tq ? 2 : 1);
                    npg = uni(t.npg);
                }
            }
            const int s = it % C::kStages;
            const bool one = npg - 2 * bk == 1;
            bool k_waited = false;
            const bool one_half = alt && bk > 0;         // the other half has nothing to issue
            const int h_from = one_half ? bk & 1 : 0, h_to = one_half ? h_from + 1 : 2;
            #pragma unroll 1
            for (int h = h_from; h < h_to; ++h) {
                const bool here = alt ? h == (bk & 1) : h < nh;
                const uint32_t f = h ? f1 : f0;
                if ((f & kPend) && (here || bk == 0)) {
                    const uint32_t pit = h ? pit1 : pit0;
                    ok = cwait(smem_u32(&bars.v_ready[pit % C::kStages]), (pit / C::kStages) & 1, abort, ctrl);
                    if (!ok) break;
                    ok = cwait(smem_u32(&bars.p_full[h]), ((h ? cs1 : cs0) - 1) & 1, abort, ctrl);
                    if (!ok) break;
                    tc_fence_after();
                    issued = true;
                    issue_pv(tmem + C::kColO + h * D, tmem + 128u * h,
                             v_lo + (pit % C::kStages) * (C::kStageBytes >> 4), idesc_o,
                             smem_u32(&bars.v_empty[pit % C::kStages]), smem_u32(&bars.o_done[h]), f);
                    if (h) f1 = 0;
                    else f0 = 0;
                }
                if (here) {
                    if (!k_waited) {
                        ok = cwait(smem_u32(&bars.k_ready[s]), (it / C::kStages) & 1, abort, ctrl);
                        if (!ok) break;
                        k_waited = true;
                    }
                    const bool first = alt ? bk < 2 : bk == 0;
                    if (first) {
                        ok = cwait(smem_u32(&bars.q_full[h]), (h ? uq1 : uq0) & 1, abort, ctrl);
                        if (!ok) break;
                    }
                    tc_fence_after();
                    issued = true;
                    // the half's last block of the unit; the block's last half frees K
                    const bool last = 2 * (bk + (alt ? 2 : 1)) >= npg;
                    issue_qk<D>(tmem + 128u * h, q_lo + h * (C::kQBytes >> 4), k_lo + s * (C::kStageBytes >> 4),
                                one ? idesc_s64 : idesc_s, smem_u32(&bars.s_full[h]), smem_u32(&bars.q_empty[h]),
                                smem_u32(&bars.k_empty[s]), (last ? 1u : 0u) | (alt || h == nh - 1 ? 2u : 0u));
                    const uint32_t nf = kPend | (first ? kFirst : 0) | (last ? kLast : 0) | (one ? kOne : 0) |
                                        (alt || h == nh - 1 ? kFrees : 0);
                    if (h) {
                        f1 = nf;
                        pit1 = it;
                        ++cs1;
                    } else {
                        f0 = nf;
                        pit0 = it;
                        ++cs0;
                    }
                }
            }
            if (!ok || end) break;
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
    if (tid == 0) {
        // The last CTA out rewinds the unit cursor.
        __threadfence();
        if (atomicAdd(&ctrl->done_ctas, 1) == (int)gridDim.x - 1) {
            ctrl->next_item = 0;
            ctrl->done_ctas = 0;
        }
    }
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols)
                     : "memory");
    }
}

// ---------------------------------------------------------------------------
// Merge of split tiles: out = sum_c w_c o_c / sum_c w_c, w_c = 2^(mu_c - M) l_c,
// over a tile's pieces, with the sink's share of the denominator.  A warp
// takes a row of a (tile, kv head), a lane D / 32 dimensions.
// ---------------------------------------------------------------------------
constexpr int kMergeBlocksPerSm = 4;

template <int D>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ CodedPrefillArgs ca) {
    constexpr int N = D / 32;
    const PrefillArgs& a = ca.a;
    const Ctrl* ctrl = reinterpret_cast<const Ctrl*>(a.ws + a.L.ctrl);
    griddep_wait();
    const int lane = threadIdx.x & 31, g = a.group, Hk = a.kv_heads;
    const __nv_bfloat16* sinks = static_cast<const __nv_bfloat16*>(a.sinks);
    // tiles up to the last split one (of 0 units none), rows of the fullest of them
    const int most = ctrl->chunk_pages * g;
    const int rows = ctrl->n_items == 0 ? 0 : ctrl->max_items * Hk * most;
    for (int w = blockIdx.x * 8 + (threadIdx.x >> 5); w < rows; w += gridDim.x * 8) {
        const int r = w % most, kvh = w / most % Hk, j = w / most / Hk;
        const PfTile t = reinterpret_cast<const PfTile*>(a.ws + a.L.tiles)[j];
        const int nch = t.pad & 4095, slot0 = t.pad >> 12;
        if (nch == 0 || r >= t.ntok * g) continue;
        const size_t at0 = ((size_t)slot0 * a.kv_heads + kvh) * ca.slot_rows + r;
        const size_t step = (size_t)a.kv_heads * ca.slot_rows;
        float M = -1.0e30f, L = 0.f, O[N] = {};
        #pragma unroll 4
        for (int c = 0; c < nch; ++c) {
            const float2 ml = __ldcg(ca.part_ml + at0 + c * step);
            const float* src = ca.part_o + (at0 + c * step) * D + lane * N;
            float x[N];
            if constexpr (N == 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
                x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
            } else {
                const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
                x[0] = v.x; x[1] = v.y;
            }
            const float Mn = fmaxf(M, ml.x);
            const float fa = exp2_approx(M - Mn), fc = exp2_approx(ml.x - Mn) * ml.y;
            const float fo = L * fa;
            M = Mn;
            L = fo + fc;
            const float inv = L == 0.f ? 0.f : 1.f / L;      // O stays an average
            #pragma unroll
            for (int e = 0; e < N; ++e) O[e] = O[e] * (fo * inv) + x[e] * (fc * inv);
        }
        const int h = kvh * g + r % g;
        const float sk = sinks != nullptr ? __bfloat162float(sinks[h]) * 1.4426950408889634f : 0.f;
        const float inv = L * sink_scale(M, L, sinks != nullptr, sk);
        __nv_bfloat16* dst =
            static_cast<__nv_bfloat16*>(a.out) + ((size_t)(t.t0 + r / g) * a.heads + h) * D + lane * N;
        if constexpr (N == 4)
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(O[0] * inv, O[1] * inv),
                                                        pack_bf16x2(O[2] * inv, O[3] * inv));
        else
            *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(O[0] * inv, O[1] * inv);
    }
}

template <int D, typename Code>
cudaError_t launch_d(const CodedPrefillArgs& ca, const CUtensorMap& q_map, int grid, bool merge, cudaStream_t stream) {
    using C = CpCfg<D>;
    auto kern = prefill_coded_kernel<D, Code>;
    static int configured_mask = 0;   // bit per device id < 31
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 31 || !(__atomic_load_n(&configured_mask, __ATOMIC_ACQUIRE) & (1 << dev))) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 31) __atomic_fetch_or(&configured_mask, 1 << dev, __ATOMIC_ACQ_REL);
    }
    // Both are programmatic dependents: their start-up runs under the launch
    // before, and they wait before they read what it wrote.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kCpThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, q_map, ca);
    if (e != cudaSuccess || !merge) return e;
    cfg.gridDim = dim3((unsigned)(grid * kMergeBlocksPerSm));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, merge_kernel<D>, ca);
}

}  // namespace

cudaError_t launch_prefill_coded(const CodedPrefillArgs& ca, const CUtensorMap& q_map, int code, int grid,
                                 bool merge, cudaStream_t stream) {
    if (ca.a.head_dim == 128)
        return code == 0 ? launch_d<128, E4m3>(ca, q_map, grid, merge, stream)
                         : launch_d<128, Int8>(ca, q_map, grid, merge, stream);
    return code == 0 ? launch_d<64, E4m3>(ca, q_map, grid, merge, stream)
                     : launch_d<64, Int8>(ca, q_map, grid, merge, stream);
}

}  // namespace pdattn
