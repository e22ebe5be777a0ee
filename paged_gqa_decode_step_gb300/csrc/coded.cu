// Writing a coded KV cache and reading it back.
//
// The write rotates keys as rope_write_kernel does (Llama example page,
// "src/rope.linnet": separate f32 products and one f32 add) but codes the f32
// value itself, with no rounding to T in between.  A group of D / 16 lanes
// holds one head vector (8 elements of each half per lane, so a lane has both
// elements of every pair it rotates), finds max|x| with shuffles and
// divides by the scale (IEEE division: the codes are those of the formula in
// coded.cuh, bit for bit).
//
// The attention calls rotate their queries here too: each query head becomes
// an f16 row q * 2^-e with the largest element in [1, 2), and the factor
// 2^e * scale * log2 e that its scores are multiplied with.  f16 keeps 11
// bits of every element above 2^-14 of the largest; for f32 inputs a second
// f16 row holds what the first one rounds off.
//
// Bound by the latency of the loads: position, slot and rope row one after the
// other (8192 tokens, 8 kv heads of 128, bf16: 55 MB in 17.8 us, of measured
// copy bandwidth 0.45; issue slots half used).  48 registers a thread, for five
// blocks per SM, spill some (24 bytes stored for bf16, 120 for f32).
#include <type_traits>

#include "coded.cuh"

namespace pdattn {

constexpr int kCodeThreads = 256;
constexpr float kEdge = 8.67361738e-19f;       // 2^-60

// Pairs of f32 as one instruction's operand.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n"
        " mul.rn.f32x2 rd, ra, rb;\n mov.b64 {%0, %1}, rd;\n}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n"
        " sub.rn.f32x2 rd, ra, rb;\n mov.b64 {%0, %1}, rd;\n}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 ra, rb, rc, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n mov.b64 rc, {%6, %7};\n"
        " fma.rn.f32x2 rd, ra, rb, rc;\n mov.b64 {%0, %1}, rd;\n}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// The larger magnitude of three; a NaN wins.
__device__ __forceinline__ float top3(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Eight consecutive elements as loaded, and as pairs of f32.
template <typename T>
struct Raw8 {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
        #pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k) v[k] = __ldg(reinterpret_cast<const uint4*>(p) + k);
    }
    __device__ __forceinline__ float2 pair(int k) const {
        if constexpr (sizeof(T) == 2) {
            const uint32_t w = k == 0 ? v[0].x : k == 1 ? v[0].y : k == 2 ? v[0].z : v[0].w;
            return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
        } else {
            const uint4& q = v[k / 2];
            return k & 1 ? make_float2(__uint_as_float(q.z), __uint_as_float(q.w))
                         : make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
        }
    }
};

// x becomes -x / s, rounded to nearest, with s = max(top / qmax, 2^-126) of
// the finite vector's largest magnitude `top`; returns s.
//
// For many x of one s: with r = RN(1 / s) and q0 = RN(x r), the remainder
// x - s q0 is exact in one FMA and q0 + r * rem rounds to the quotient
// (Markstein, IBM J. Res. Dev. 34, 1990); top / qmax the same way.  That needs
// quotient, remainder and s clear of the ends of the exponent range, so a
// vector whose top lies outside [2^-60, 2^60] is scaled by a power of two
// first.  (A remainder of a quotient below 2^-11 may still be inexact, and its
// x rounded by the scaling; such a quotient is under half of any code's
// smallest step.)  The quotients are negated so that a zero keeps its sign: a
// remainder of nothing is +0, and -r times it leaves a zero of either sign.
template <typename Code>
__device__ __forceinline__ float divide_by_scale(float2 (&x)[8], float top) {
    constexpr float kBig = 18446744073709551616.f, kSmall = 1.f / kBig;    // 2^64, 2^-64
    constexpr float kRq = 1.f / Code::kQMax;
    float up = 1.f, down = 1.f;
    if (top < kEdge || top > 1.f / kEdge) {
        up = top < 1.f ? kBig : kSmall;
        down = top < 1.f ? kSmall : kBig;
        #pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = mul2(x[k], make_float2(up, up));
    }
    const float t = top * up;
    const float t0 = __fmul_rn(t, kRq);
    const float s = fmaxf(__fmaf_rn(__fmaf_rn(-Code::kQMax, t0, t), kRq, t0), kScaleMin * up);
    const float r = __frcp_rn(s);
    const float2 nr = make_float2(-r, -r), s2 = make_float2(s, s);
    #pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float2 n0 = mul2(x[k], nr);
        x[k] = fma2(fma2(s2, n0, x[k]), nr, n0);
    }
    return s * down;
}

// Block = one token; its vectors (`heads` queries in attention calls, then
// keys, then values) are dealt to groups of D / 16 lanes, so that every lane
// moves 16 bytes of bf16 at a time and position, slot and table rows are
// found once per block.
template <typename T, int D, typename Code>
__global__ void __launch_bounds__(kCodeThreads, 5) code_kernel(const __grid_constant__ CodeArgs a) {
    griddep_launch_dependents();
    constexpr int kLanes = D / 16, kHalf = D / 2;
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(a.ws);
    const int Hk = a.kv_heads, Hq = a.q ? a.heads : 0, per = Hq + 2 * Hk, i = blockIdx.x;
    const int lane = threadIdx.x % kLanes, e0 = 8 * lane;
    if (a.merge_cnt) {
        for (int h = threadIdx.x; h < Hk; h += blockDim.x) a.merge_cnt[(size_t)i * Hk + h] = 0;
        // a plan left here by another call is overwritten by this one
        if (i == 0 && threadIdx.x == 0) ctrl->magic = 0;
    }
    // a vector's loads are under way before the position and slot are known, or
    // while the vector before it is coded (8192 cold tokens: 22.4 -> 20.4 us)
    Raw8<T> raw_lo, raw_hi;
    auto load = [&](int j) {
        const T* src = j < Hq ? static_cast<const T*>(a.q) + ((size_t)i * Hq + j) * D
                              : static_cast<const T*>(j < Hq + Hk ? a.k_new : a.v_new) +
                                    ((size_t)i * Hk + (j < Hq + Hk ? j - Hq : j - Hq - Hk)) * D;
        raw_lo.load(src + e0);
        raw_hi.load(src + kHalf + e0);
    };
    const int j0 = threadIdx.x / kLanes, step = blockDim.x / kLanes;
    if (j0 < per) load(j0);
    const int pos = __ldg(a.positions + i);
    const bool pos_ok = pos >= 0 && pos <= a.last_pos;
    int slot = -1;
    if (pos_ok) {
        if (a.slots) {
            slot = __ldg(a.slots + i);
        } else {
            const int page = __ldg(a.table + (size_t)i * a.pages_per_row + pos / kPageSize);
            slot = page >= 0 && page < a.num_pages ? page * kPageSize + pos % kPageSize : -1;
        }
    }
    const bool slot_ok = slot >= 0 && slot / kPageSize < a.num_pages;
    if (threadIdx.x == 0) {
        if (!pos_ok) set_error(ctrl, kErrBadPos);
        else if (!slot_ok) set_error(ctrl, kErrBadPage);
    }
    const int end = !pos_ok ? 0 : slot_ok ? per : Hq;
    const uint32_t group = ((1u << kLanes) - 1) << ((threadIdx.x & 31) / kLanes * kLanes);
    #pragma unroll 1
    for (int j = j0; j < end; j += step) {
        const bool is_q = j < Hq, is_v = j >= Hq + Hk;
        const int h = is_q ? j : (is_v ? j - Hq - Hk : j - Hq);
        float2 x[8];                        // four pairs of the lower half, four of the upper
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[k] = raw_lo.pair(k);
            x[4 + k] = raw_hi.pair(k);
        }
        if (j + step < end) load(j + step);
        if (a.rope_cos && !is_v) {
            const T* cr = static_cast<const T*>(a.rope_cos) + (size_t)pos * D + e0;
            const T* sr = static_cast<const T*>(a.rope_sin) + (size_t)pos * D + e0;
            Raw8<T> cos_lo, cos_hi, sin_lo, sin_hi;
            cos_lo.load(cr);
            cos_hi.load(cr + kHalf);
            sin_lo.load(sr);
            sin_hi.load(sr + kHalf);
            // (not packed: packed products came out fused with the sums)
            auto rotate = [](float u, float c, float v, float t, bool minus) {
                return minus ? __fsub_rn(__fmul_rn(u, c), __fmul_rn(v, t)) : __fadd_rn(__fmul_rn(u, c), __fmul_rn(v, t));
            };
            #pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 u = x[k], v = x[4 + k], cl = cos_lo.pair(k), ch = cos_hi.pair(k), sl = sin_lo.pair(k),
                             sh = sin_hi.pair(k);
                x[k] = make_float2(rotate(u.x, cl.x, v.x, sl.x, true), rotate(u.y, cl.y, v.y, sl.y, true));
                x[4 + k] = make_float2(rotate(v.x, ch.x, u.x, sh.x, false), rotate(v.y, ch.y, u.y, sh.y, false));
            }
        }
        // the largest magnitude as its bits (they order like the value), so
        // that an infinity or a NaN anywhere shows in the result
        float top_a = 0.f, top_b = 0.f;
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
            top_a = top3(top_a, x[k].x, x[k].y);
            top_b = top3(top_b, x[4 + k].x, x[4 + k].y);
        }
        uint32_t top = __float_as_uint(top3(top_a, top_b, 0.f));
        #pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) top = max(top, __shfl_xor_sync(group, top, d));
        const bool finite = top < 0x7f800000u;
        if (is_q) {
            // 2^-e scales the largest element into [1, 2)
            const int ex = min(max((int)(top >> 23), 1), 253);      // biased exponent
            const float down = finite ? __uint_as_float((uint32_t)(254 - ex) << 23) : __uint_as_float(0x7fc00000u);
            const float factor = (finite ? __uint_as_float((uint32_t)ex << 23) : 1.f) * a.scale_log2;
            uint8_t* row = a.q_out + ((size_t)i * Hq + h) * a.q_row_bytes;
            uint32_t w[8], r[8];
            #pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 y = mul2(x[k], make_float2(down, down));
                w[k] = pack_f16x2(y.x, y.y);
                const float2 rest = sub2(y, __half22float2(*reinterpret_cast<const __half2*>(&w[k])));
                r[k] = pack_f16x2(rest.x, rest.y);
            }
            *reinterpret_cast<uint4*>(row + e0 * 2) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(row + (kHalf + e0) * 2) = make_uint4(w[4], w[5], w[6], w[7]);
            if (sizeof(T) == 4) {     // f32: the second row (see attend_kernel.cuh)
                *reinterpret_cast<uint4*>(row + 2 * D + e0 * 2) = make_uint4(r[0], r[1], r[2], r[3]);
                *reinterpret_cast<uint4*>(row + 2 * D + (kHalf + e0) * 2) = make_uint4(r[4], r[5], r[6], r[7]);
            }
            if (lane == 0) {
                if (a.q_factor) a.q_factor[(size_t)i * Hq + h] = factor;
                else *reinterpret_cast<float*>(row + (int)sizeof(T) * D) = factor;
            }
        } else {
            // a vector that holds an infinity or a NaN stands for NaN throughout
            float scale = __uint_as_float(0x7fc00000u);
            if (finite) {
                scale = divide_by_scale<Code>(x, __uint_as_float(top));
            } else {
                #pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = make_float2(-0.f, -0.f);
            }
            const size_t at = ((size_t)(slot / kPageSize) * Hk + h) * kPageSize + slot % kPageSize;
            uint8_t* dst = (is_v ? a.v : a.k) + at * D;
            *reinterpret_cast<uint2*>(dst + e0) = make_uint2(encode4<Code>(x[0], x[1]), encode4<Code>(x[2], x[3]));
            *reinterpret_cast<uint2*>(dst + kHalf + e0) = make_uint2(encode4<Code>(x[4], x[5]), encode4<Code>(x[6], x[7]));
            if (lane == 0) (is_v ? a.v_scale : a.k_scale)[at] = scale;
        }
    }
    // With a planner launched before it, the last block exits only after the
    // planner has finished: the attention waits for this grid alone.
    if (a.after_plan && blockIdx.x == gridDim.x - 1) griddep_wait();
}

// 16 codes of one head vector of K and of V per thread, widened, scaled in
// f32 and rounded once to T.
template <typename T, int D, typename Code>
__global__ void __launch_bounds__(kCodeThreads) read_kernel(const __grid_constant__ ReadArgs a) {
    constexpr int kPieces = D / 16;
    const int Hk = a.kv_heads;
    const long long u = (long long)blockIdx.x * kCodeThreads + threadIdx.x;
    if (u >= (long long)a.n_tokens * Hk * kPieces) return;
    const int piece = (int)(u % kPieces);
    const long long vec = u / kPieces;
    const int h = (int)(vec % Hk), i = (int)(vec / Hk);
    const int slot = __ldg(a.slots + i);
    if (slot < 0 || slot / kPageSize >= a.num_pages) {
        if (piece == 0 && h == 0) set_error(reinterpret_cast<Ctrl*>(a.ws), kErrBadPage);
        return;
    }
    const size_t at = ((size_t)(slot / kPageSize) * Hk + h) * kPageSize + slot % kPageSize;
    const uint4 kc = __ldg(reinterpret_cast<const uint4*>(a.k + at * D) + piece);
    const uint4 vc = __ldg(reinterpret_cast<const uint4*>(a.v + at * D) + piece);
    const float ks = __ldg(a.k_scale + at), vs = __ldg(a.v_scale + at);
    auto put = [&](const uint4& c, float s, void* out) {
        T* dst = static_cast<T*>(out) + (size_t)vec * D + piece * 16;
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        float f[16];
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t lo, hi;
            widen4<Code>(w[k], lo, hi);
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
            f[4 * k] = x.x * s; f[4 * k + 1] = x.y * s; f[4 * k + 2] = y.x * s; f[4 * k + 3] = y.y * s;
        }
        constexpr int kWords = 4 * sizeof(T);
        uint32_t u[kWords];
        #pragma unroll
        for (int k = 0; k < kWords; ++k) {
            if constexpr (sizeof(T) == 2) u[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
            else u[k] = __float_as_uint(f[k]);
        }
        // whole 32-byte sectors where the outputs' alignment allows them
        #pragma unroll
        for (int k = 0; k < kWords; k += 8) {
            uint32_t* to = reinterpret_cast<uint32_t*>(dst) + k;
            if (a.wide) {
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                             ::"l"(to), "r"(u[k]), "r"(u[k + 1]), "r"(u[k + 2]), "r"(u[k + 3]), "r"(u[k + 4]),
                               "r"(u[k + 5]), "r"(u[k + 6]), "r"(u[k + 7])
                             : "memory");
            } else {
                reinterpret_cast<uint4*>(to)[0] = make_uint4(u[k], u[k + 1], u[k + 2], u[k + 3]);
                reinterpret_cast<uint4*>(to)[1] = make_uint4(u[k + 4], u[k + 5], u[k + 6], u[k + 7]);
            }
        }
    };
    put(kc, ks, a.k_out);
    put(vc, vs, a.v_out);
}

// ---------------------------------------------------------------------------
// Host launchers
// ---------------------------------------------------------------------------
// f(T, D, Code) for the call's types: head dim 64 or 128, bf16 or f32, e4m3 or int8.
template <typename F>
static cudaError_t by_types(int dtype, int D, int code, F f) {
    auto with_code = [&](auto t, auto d) {
        return code == 0 ? f(t, d, E4m3{}) : f(t, d, Int8{});
    };
    auto with_dim = [&](auto t) {
        return D == 128 ? with_code(t, std::integral_constant<int, 128>{}) : with_code(t, std::integral_constant<int, 64>{});
    };
    return dtype == 0 ? with_dim(__nv_bfloat16{}) : with_dim(float{});
}

cudaError_t launch_code(const CodeArgs& a, int dtype, int code, cudaStream_t stream) {
    // As many lanes as the token's vectors can use, in whole warps; with many
    // tokens blocks of 64 threads, which come and go one by one, with few all of
    // the token's vectors at once.  Up to 2048 tokens the call hides the
    // difference (8 kv heads of 128, bf16: 512 tokens 8.3 us with 64 threads and
    // 8.5 with 256, 2048 tokens 8.1 and 8.8); 8192 take 17.8 and 20.2 us.  For
    // f32 it is the other way round (4096 tokens of 12 heads of 64: 12.3 and
    // 10.3 us).
    const long long most = a.n_tokens >= 1024 ? 64 : kCodeThreads;
    const long long lanes = (long long)((a.q ? a.heads : 0) + 2 * a.kv_heads) * (a.head_dim / 16);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.n_tokens);
    cfg.blockDim = dim3((unsigned)(lanes >= most ? most : (lanes + 31) / 32 * 32));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.after_plan ? 1 : 0;
    return by_types(dtype, a.head_dim, code, [&](auto t, auto d, auto c) {
        return cudaLaunchKernelEx(&cfg, code_kernel<decltype(t), decltype(d)::value, decltype(c)>, a);
    });
}

cudaError_t launch_read(const ReadArgs& a, int dtype, int code, cudaStream_t stream) {
    const long long units = (long long)a.n_tokens * a.kv_heads * (a.head_dim / 16);
    const unsigned grid = (unsigned)((units + kCodeThreads - 1) / kCodeThreads);
    return by_types(dtype, a.head_dim, code, [&](auto t, auto d, auto c) {
        read_kernel<decltype(t), decltype(d)::value, decltype(c)><<<grid, kCodeThreads, 0, stream>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace pdattn
