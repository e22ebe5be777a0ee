// Writing a coded KV cache and reading it back.
//
// The write rotates keys as rope_write_kernel does (Llama example page,
// "src/rope.linnet": separate f32 products and one f32 add) but codes the f32
// value itself, with no rounding to T in between.  A group of D / 8 lanes
// holds one head vector (4 elements of each half per lane, so a lane has
// both elements of every pair it rotates), finds max|x| with shuffles and
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

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&f)[4]);
template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[4]) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xffff0000u);
}
template <>
__device__ __forceinline__ void load4<float>(const float* p, float (&f)[4]) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}

// One head vector per group of D / 8 lanes: vector v of token v / per, where
// a token has `heads` query vectors (attention calls only), then its key and
// its value vectors.
template <typename T, int D, typename Code>
__global__ void __launch_bounds__(kCodeThreads) code_kernel(const __grid_constant__ CodeArgs a) {
    griddep_launch_dependents();
    constexpr int kLanes = D / 8, kHalf = D / 2;
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(a.ws);
    const int Hk = a.kv_heads, Hq = a.q ? a.heads : 0, per = Hq + 2 * Hk;
    const long long v = (long long)blockIdx.x * (kCodeThreads / kLanes) + threadIdx.x / kLanes;
    const int lane = threadIdx.x % kLanes, e0 = 4 * lane;
    if (v < (long long)a.n_tokens * per) {
        const int i = (int)(v / per), j = (int)(v - (long long)i * per);
        const bool is_q = j < Hq, is_v = j >= Hq + Hk;
        const int h = is_q ? j : (is_v ? j - Hq - Hk : j - Hq);
        const int pos = __ldg(a.positions + i);
        // a token's position must lie in the rope table, and for the
        // attention calls in the page table
        const bool pos_ok = pos >= 0 && (!a.rope_cos || pos < a.rope_len) && (!a.q || pos < a.pages_per_row * kPageSize);
        int slot = -1;
        if (pos_ok && !is_q) {
            if (a.slots) {
                slot = __ldg(a.slots + i);
            } else {
                const int page = __ldg(a.table + (size_t)i * a.pages_per_row + pos / kPageSize);
                slot = page >= 0 && page < a.num_pages ? page * kPageSize + pos % kPageSize : -1;
            }
        }
        const bool slot_ok = slot >= 0 && slot / kPageSize < a.num_pages;
        if (lane == 0) {
            if (!pos_ok) set_error(ctrl, kErrBadPos);
            else if (!is_q && !slot_ok) set_error(ctrl, kErrBadPage);
        }
        if (pos_ok && (is_q || slot_ok)) {
            const T* src = static_cast<const T*>(is_q ? a.q : (is_v ? a.v_new : a.k_new)) +
                           ((size_t)i * (is_q ? Hq : Hk) + h) * D;
            float lo[4], hi[4];
            load4<T>(src + e0, lo);
            load4<T>(src + kHalf + e0, hi);
            if (a.rope_cos && !is_v) {
                const T* cr = static_cast<const T*>(a.rope_cos) + (size_t)pos * D;
                const T* sr = static_cast<const T*>(a.rope_sin) + (size_t)pos * D;
                float cl[4], ch[4], sl[4], sh[4];
                load4<T>(cr + e0, cl);
                load4<T>(cr + kHalf + e0, ch);
                load4<T>(sr + e0, sl);
                load4<T>(sr + kHalf + e0, sh);
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x = lo[k], y = hi[k];
                    lo[k] = __fsub_rn(__fmul_rn(x, cl[k]), __fmul_rn(y, sl[k]));
                    hi[k] = __fadd_rn(__fmul_rn(y, ch[k]), __fmul_rn(x, sh[k]));
                }
            }
            // the largest magnitude as its bits (they order like the value),
            // so that an infinity or a NaN anywhere shows in the result
            uint32_t top = 0;
            #pragma unroll
            for (int k = 0; k < 4; ++k)
                top = max(top, max(__float_as_uint(lo[k]) & 0x7fffffffu, __float_as_uint(hi[k]) & 0x7fffffffu));
            const uint32_t group = kLanes == 32 ? 0xffffffffu
                                                : ((1u << kLanes) - 1) << ((threadIdx.x & 31) / kLanes * kLanes);
            #pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) top = max(top, __shfl_xor_sync(group, top, d));
            const bool finite = top < 0x7f800000u;
            if (is_q) {
                // 2^-e scales the largest element into [1, 2)
                const int ex = min(max((int)(top >> 23), 1), 253);      // biased exponent
                const float down = finite ? __uint_as_float((uint32_t)(254 - ex) << 23) : __uint_as_float(0x7fc00000u);
                const float factor = (finite ? __uint_as_float((uint32_t)ex << 23) : 1.f) * a.scale_log2;
                uint8_t* row = a.q_out + ((size_t)i * Hq + h) * a.q_row_bytes;
                uint32_t w[4], r[4];
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float* x = k < 2 ? lo : hi;
                    const int o = 2 * (k & 1);
                    const float x0 = x[o] * down, x1 = x[o + 1] * down;
                    w[k] = pack_f16x2(x0, x1);
                    const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                    r[k] = pack_f16x2(x0 - back.x, x1 - back.y);
                }
                *reinterpret_cast<uint2*>(row + e0 * 2) = make_uint2(w[0], w[1]);
                *reinterpret_cast<uint2*>(row + (kHalf + e0) * 2) = make_uint2(w[2], w[3]);
                if (a.q_split) {
                    *reinterpret_cast<uint2*>(row + 2 * D + e0 * 2) = make_uint2(r[0], r[1]);
                    *reinterpret_cast<uint2*>(row + 2 * D + (kHalf + e0) * 2) = make_uint2(r[2], r[3]);
                }
                if (lane == 0) {
                    if (a.q_factor) a.q_factor[(size_t)i * Hq + h] = factor;
                    else *reinterpret_cast<float*>(row + (a.q_split ? 4 : 2) * D) = factor;
                }
            } else {
                // a vector that holds an infinity or a NaN stands for NaN throughout
                const float scale = finite ? fmaxf(__fdiv_rn(__uint_as_float(top), Code::kQMax), kScaleMin)
                                           : __uint_as_float(0x7fc00000u);
                if (!finite) {
                    #pragma unroll
                    for (int k = 0; k < 4; ++k) lo[k] = hi[k] = 0.f;
                }
                const float by = finite ? scale : 1.f;
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    lo[k] = __fdiv_rn(lo[k], by);
                    hi[k] = __fdiv_rn(hi[k], by);
                }
                const size_t at = ((size_t)(slot / kPageSize) * Hk + h) * kPageSize + slot % kPageSize;
                uint8_t* dst = (is_v ? a.v : a.k) + at * D;
                *reinterpret_cast<uint32_t*>(dst + e0) = encode4<Code>(lo[0], lo[1], lo[2], lo[3]);
                *reinterpret_cast<uint32_t*>(dst + kHalf + e0) = encode4<Code>(hi[0], hi[1], hi[2], hi[3]);
                if (lane == 0) (is_v ? a.v_scale : a.k_scale)[at] = scale;
            }
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
        if constexpr (sizeof(T) == 2) {
            #pragma unroll
            for (int k = 0; k < 2; ++k)
                reinterpret_cast<uint4*>(dst)[k] =
                    make_uint4(pack_bf16x2(f[8 * k], f[8 * k + 1]), pack_bf16x2(f[8 * k + 2], f[8 * k + 3]),
                               pack_bf16x2(f[8 * k + 4], f[8 * k + 5]), pack_bf16x2(f[8 * k + 6], f[8 * k + 7]));
        } else {
            #pragma unroll
            for (int k = 0; k < 4; ++k)
                reinterpret_cast<float4*>(dst)[k] = make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
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
    const long long vectors = (long long)a.n_tokens * ((a.q ? a.heads : 0) + 2 * a.kv_heads);
    const long long lanes = vectors * (a.head_dim / 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((lanes + kCodeThreads - 1) / kCodeThreads));
    cfg.blockDim = dim3(kCodeThreads);
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
