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
// Bound by the loads and stores of T (the codes are a third of the bytes for
// bf16).
#include <type_traits>

#include "coded.cuh"

namespace pdattn {

constexpr int kCodeThreads = 256;

// Eight consecutive elements as f32.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[8]) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&f)[8]) {
    #pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p) + k);
        f[4 * k] = v.x; f[4 * k + 1] = v.y; f[4 * k + 2] = v.z; f[4 * k + 3] = v.w;
    }
}

// x / s rounded to nearest, for many x of one s: with r = RN(1 / s) and
// q0 = RN(x r), the remainder x - s q0 is exact in one FMA and q0 + r * rem
// rounds to the quotient (Markstein, IBM J. Res. Dev. 34, 1990).  Needs
// quotient, remainder and s clear of the ends of the exponent range; a vector
// whose largest magnitude lies outside [2^-60, 2^60] divides directly.  (The
// remainder of a quotient below 2^-11 may then still be inexact; such a
// quotient is under half of any code's smallest step.)
struct Divider {
    float s, r;
    bool direct;
    __device__ __forceinline__ Divider(float scale, uint32_t top) {
        s = scale;
        r = __fdiv_rn(1.f, scale);
        direct = top < (uint32_t)(127 - 60) << 23 || top > (uint32_t)(127 + 60) << 23;
    }
    __device__ void apply(float (&x)[8]) const {
        if (direct) {
            #pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = __fdiv_rn(x[k], s);
        } else {
            #pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float q0 = __fmul_rn(x[k], r);
                x[k] = __fmaf_rn(__fmaf_rn(-s, q0, x[k]), r, q0);
            }
        }
    }
};

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
    const int pos = __ldg(a.positions + i);
    // a token's position must lie in the rope table, and for the attention
    // calls in the page table
    const bool pos_ok = pos >= 0 && (!a.rope_cos || pos < a.rope_len) && (!a.q || pos < a.pages_per_row * kPageSize);
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
    for (int j = threadIdx.x / kLanes; j < end; j += blockDim.x / kLanes) {
        const bool is_q = j < Hq, is_v = j >= Hq + Hk;
        const int h = is_q ? j : (is_v ? j - Hq - Hk : j - Hq);
        const T* src = static_cast<const T*>(is_q ? a.q : (is_v ? a.v_new : a.k_new)) +
                       ((size_t)i * (is_q ? Hq : Hk) + h) * D;
        float lo[8], hi[8];
        load8<T>(src + e0, lo);
        load8<T>(src + kHalf + e0, hi);
        if (a.rope_cos && !is_v) {
            const T* cr = static_cast<const T*>(a.rope_cos) + (size_t)pos * D;
            const T* sr = static_cast<const T*>(a.rope_sin) + (size_t)pos * D;
            float cl[8], ch[8], sl[8], sh[8];
            load8<T>(cr + e0, cl);
            load8<T>(cr + kHalf + e0, ch);
            load8<T>(sr + e0, sl);
            load8<T>(sr + kHalf + e0, sh);
            #pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float x = lo[k], y = hi[k];
                lo[k] = __fsub_rn(__fmul_rn(x, cl[k]), __fmul_rn(y, sl[k]));
                hi[k] = __fadd_rn(__fmul_rn(y, ch[k]), __fmul_rn(x, sh[k]));
            }
        }
        // the largest magnitude as its bits (they order like the value), so
        // that an infinity or a NaN anywhere shows in the result
        uint32_t top = 0;
        #pragma unroll
        for (int k = 0; k < 8; ++k)
            top = max(top, max(__float_as_uint(lo[k]) & 0x7fffffffu, __float_as_uint(hi[k]) & 0x7fffffffu));
        const uint32_t group = ((1u << kLanes) - 1) << ((threadIdx.x & 31) / kLanes * kLanes);
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
                const float x0 = (k < 4 ? lo : hi)[2 * (k & 3)] * down, x1 = (k < 4 ? lo : hi)[2 * (k & 3) + 1] * down;
                w[k] = pack_f16x2(x0, x1);
                const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                r[k] = pack_f16x2(x0 - back.x, x1 - back.y);
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
            float scale = fmaxf(__fdiv_rn(__uint_as_float(top), Code::kQMax), kScaleMin);
            if (finite) {
                const Divider by(scale, top);
                by.apply(lo);
                by.apply(hi);
            } else {
                scale = __uint_as_float(0x7fc00000u);
                #pragma unroll
                for (int k = 0; k < 8; ++k) lo[k] = hi[k] = 0.f;
            }
            const size_t at = ((size_t)(slot / kPageSize) * Hk + h) * kPageSize + slot % kPageSize;
            uint8_t* dst = (is_v ? a.v : a.k) + at * D;
            *reinterpret_cast<uint2*>(dst + e0) = make_uint2(encode4<Code>(lo[0], lo[1], lo[2], lo[3]),
                                                             encode4<Code>(lo[4], lo[5], lo[6], lo[7]));
            *reinterpret_cast<uint2*>(dst + kHalf + e0) = make_uint2(encode4<Code>(hi[0], hi[1], hi[2], hi[3]),
                                                                     encode4<Code>(hi[4], hi[5], hi[6], hi[7]));
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
    // tokens blocks of 64 threads, which come and go one by one (8192 tokens
    // of 16 vectors: 64 threads 18.5 us, 128 22, 256 24.6), with few all of
    // the token's vectors at once.
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
