// Rotary positions for long contexts: frequency tables, and the rotation of q
// and k by it (or back, which is the gradient).
//
// Pair i of a head vector turns by angle(pos, i) = pos * w_i:
//   y0 = x0 cos - x1 sin,  y1 = x1 cos + x0 sin   (sin negated for the inverse)
// with cos and sin times the frequencies' gain.  A rotation's inverse is its
// transpose, so the inverse call on an output's gradient is the input's.
//
// Angles.  The host holds w_i / (2 pi) in turns as a fraction of 2^64
// (pdattn_rotary.turns).  pos * turns mod 2^64 is the angle's exact place in
// its turn: one integer product, whose overflow drops the whole turns, where a
// product in f32 is off by 2^-24 of the angle (0.004 rad at position 131072).
// The top 32 bits are cut into a quarter turn and a signed rest of at most an
// eighth of a turn, so that the rest is an f32 to 2^-25 of an eighth of a turn.
#include "internal.h"

namespace pdattn {
namespace {

// cos and sin of the angle t / 2^64 turns, times gain.
__device__ __forceinline__ void cos_sin(uint64_t t, float gain, float& c, float& s) {
    const uint32_t u = (uint32_t)(t >> 32) + 0x20000000u;              // + an eighth of a turn
    const int rest = (int)(u & 0x3fffffffu) - 0x20000000;              // [-1/8, 1/8) turns in 2^-32
    float a, b;
    sincospif((float)rest * 4.656612873077393e-10f, &a, &b);           // in half turns: 2^-31
    const uint32_t q = u >> 30;                                        // quarter turns
    const float cc = q & 1 ? a : b, ss = q & 1 ? b : a;
    c = (q == 1 || q == 2 ? -cc : cc) * gain;
    s = (q >= 2 ? -ss : ss) * gain;
}

// cos and sin [length, D] of T for half pairs over the whole head: both halves
// of a row hold the same values.
//
// f32: every value by cos_sin; the stores bound it.  bf16, half the bytes, was
// bound by the arithmetic (131072 rows of 128: 21 us against 10 of stores), so
// where there are rows enough (kSums: 12.9 us, 14.1 with runs of 8; 4096 rows of
// 64 take twice as long so) a thread takes N pairs (one 16-byte vector) at kRun positions in a row: the first
// by cos_sin, the others by the sum formulas with cos and sin of 1 .. kRun - 1
// positions, which the block computes once.  A sum is off by at most
// |c| e + |s| e on either side, 2 sqrt(2) e in all with e what cos_sin is off by,
// and two roundings: far below bf16's.
constexpr int kRun = 4;

template <typename T, bool kSums>
__global__ void __launch_bounds__(256) rotary_tables_kernel(const __grid_constant__ RotaryArgs a, int length,
                                                            T* __restrict__ cos_out, T* __restrict__ sin_out) {
    using V = Vec16<T>;
    constexpr int N = V::N;
    __shared__ float s_cos[kSums ? kRun : 1][kRotaryPairs], s_sin[kSums ? kRun : 1][kRotaryPairs];
    const int D = a.head_dim, half = D / 2, vecs = half / N;           // a power of two
    const int e0 = (threadIdx.x % vecs) * N, per = 256 / vecs;         // runs (f32: positions) a block covers at once
    uint64_t w[N];
    #pragma unroll
    for (int k = 0; k < N; ++k) w[k] = a.turns[e0 + k];
    auto put = [&](int pos, const float (&c)[N], const float (&s)[N]) {
        const uint4 vc = V::from_f32(c), vs = V::from_f32(s);
        T* co = cos_out + (size_t)pos * D + e0;
        T* so = sin_out + (size_t)pos * D + e0;
        *reinterpret_cast<uint4*>(co) = vc;
        *reinterpret_cast<uint4*>(co + half) = vc;
        *reinterpret_cast<uint4*>(so) = vs;
        *reinterpret_cast<uint4*>(so + half) = vs;
    };
    if constexpr (kSums) {
        for (int i = threadIdx.x; i < kRun * half; i += 256)
            cos_sin((uint64_t)(i / half) * a.turns[i % half], 1.f, s_cos[i / half][i % half], s_sin[i / half][i % half]);
        __syncthreads();
        const int runs = (length + kRun - 1) / kRun;
        for (int run = blockIdx.x * per + threadIdx.x / vecs; run < runs; run += gridDim.x * per) {
            float c0[N], s0[N], c[N], s[N];
            #pragma unroll
            for (int k = 0; k < N; ++k) cos_sin((uint64_t)run * kRun * w[k], a.gain, c0[k], s0[k]);
            const int n = min(kRun, length - run * kRun);
            for (int j = 0; j < n; ++j) {
                #pragma unroll
                for (int k = 0; k < N; ++k) {
                    const float cj = s_cos[j][e0 + k], sj = s_sin[j][e0 + k];
                    c[k] = c0[k] * cj - s0[k] * sj;
                    s[k] = s0[k] * cj + c0[k] * sj;
                }
                put(run * kRun + j, c, s);
            }
        }
    } else {
        for (int pos = blockIdx.x * per + threadIdx.x / vecs; pos < length; pos += gridDim.x * per) {
            float c[N], s[N];
            #pragma unroll
            for (int k = 0; k < N; ++k) cos_sin((uint64_t)pos * w[k], a.gain, c[k], s[k]);
            put(pos, c, s);
        }
    }
}

// One token per block: its pairs' cos and sin go to shared memory once for all
// heads while the first vectors of the token load.  A unit is the two 16-byte
// vectors of N half pairs, or one vector of interleaved pairs or of dimensions
// past rot_dim.
constexpr int kRotaryThreads = 128;
template <bool kInterleaved>
constexpr int kRotaryAhead = kInterleaved ? 4 : 3;     // units a thread loads before it needs the angles

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
    using V = Vec16<T>;
    constexpr int N = V::N;
    __shared__ float s_cos[kRotaryPairs], s_sin[kRotaryPairs];
    const int tok = blockIdx.x, tid = threadIdx.x;
    const int D = a.head_dim, rot = a.rot_dim, half = rot / 2;
    const int turned = kInterleaved ? rot / N : half / N;              // units of a head that turn
    const int per = turned + (D - rot) / N, units = per * (a.heads + a.kv_heads);
    const T* qi = static_cast<const T*>(a.q) + (size_t)tok * a.q_stride;
    const T* ki = static_cast<const T*>(a.k) + (size_t)tok * a.k_stride;
    T* qo = static_cast<T*>(a.q_out) + (size_t)tok * a.q_out_stride;
    T* ko = static_cast<T*>(a.k_out) + (size_t)tok * a.k_out_stride;
    // unit u: its head's vector and first element
    auto place = [&](int u, const T*& src, T*& dst, int& e) {
        const int h = u / per, v = u - h * per;
        e = v < turned ? v * N : rot + (v - turned) * N;
        const bool is_q = h < a.heads;
        const size_t at = (size_t)(is_q ? h : h - a.heads) * D + e;
        src = (is_q ? qi : ki) + at;
        dst = (is_q ? qo : ko) + at;
    };
    constexpr int kAhead = kRotaryAhead<kInterleaved>;
    uint4 x[kAhead][2];
    auto load = [&](int u, uint4 (&r)[2]) {
        const T* src;
        T* dst;
        int e;
        place(u, src, dst, e);
        r[0] = *reinterpret_cast<const uint4*>(src);
        if (!kInterleaved && e < rot) r[1] = *reinterpret_cast<const uint4*>(src + half);
    };
    #pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if (tid + k * kRotaryThreads < units) load(tid + k * kRotaryThreads, x[k]);
    const int pos = __ldg(a.positions + tok);
    if (pos < 0) {
        if (tid == 0) set_error(reinterpret_cast<Ctrl*>(a.ws), kErrBadPos);
        return;
    }
    for (int i = tid; i < half; i += kRotaryThreads) {
        float c, s;
        cos_sin((uint64_t)pos * a.turns[i], a.gain, c, s);
        s_cos[i] = c;
        s_sin[i] = a.inverse ? -s : s;
    }
    __syncthreads();
    auto turn = [&](int u, const uint4 (&r)[2]) {
        const T* src;
        T* dst;
        int e;
        place(u, src, dst, e);
        if (e >= rot) {
            *reinterpret_cast<uint4*>(dst) = r[0];
            return;
        }
        float f[N], y[N];
        V::to_f32(r[0], f);
        if constexpr (kInterleaved) {
            #pragma unroll
            for (int k = 0; k < N; k += 2) {
                const float c = s_cos[(e + k) / 2], s = s_sin[(e + k) / 2];
                y[k] = f[k] * c - f[k + 1] * s;
                y[k + 1] = f[k + 1] * c + f[k] * s;
            }
            *reinterpret_cast<uint4*>(dst) = V::from_f32(y);
        } else {
            float g[N], z[N];
            V::to_f32(r[1], g);
            #pragma unroll
            for (int k = 0; k < N; ++k) {
                const float c = s_cos[e + k], s = s_sin[e + k];
                y[k] = f[k] * c - g[k] * s;
                z[k] = g[k] * c + f[k] * s;
            }
            *reinterpret_cast<uint4*>(dst) = V::from_f32(y);
            *reinterpret_cast<uint4*>(dst + half) = V::from_f32(z);
        }
    };
    #pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if (tid + k * kRotaryThreads < units) turn(tid + k * kRotaryThreads, x[k]);
    for (int u = tid + kAhead * kRotaryThreads; u < units; u += kRotaryThreads) {
        uint4 r[2];
        load(u, r);
        turn(u, r);
    }
}

}  // namespace

cudaError_t launch_rotary_tables(const RotaryArgs& a, int length, int dtype, void* cos_out, void* sin_out,
                                 cudaStream_t stream) {
    // sums: when the runs make a block for every SM
    const int runs = kRun * 256 / (a.head_dim / 16), each = 256 / (a.head_dim / (dtype == 0 ? 16 : 8));
    const bool sums = dtype == 0 && length >= 148 * runs;
    const long long blocks = ((long long)length + (sums ? runs : each) - 1) / (sums ? runs : each);
    const int grid = (int)(blocks < 8192 ? blocks : 8192);
    __nv_bfloat16 *cb = static_cast<__nv_bfloat16*>(cos_out), *sb = static_cast<__nv_bfloat16*>(sin_out);
    if (sums)
        rotary_tables_kernel<__nv_bfloat16, true><<<grid, 256, 0, stream>>>(a, length, cb, sb);
    else if (dtype == 0)
        rotary_tables_kernel<__nv_bfloat16, false><<<grid, 256, 0, stream>>>(a, length, cb, sb);
    else
        rotary_tables_kernel<float, false><<<grid, 256, 0, stream>>>(a, length, static_cast<float*>(cos_out),
                                                                    static_cast<float*>(sin_out));
    return cudaGetLastError();
}

cudaError_t launch_rotary(const RotaryArgs& a, int n_tokens, int dtype, cudaStream_t stream) {
    if (dtype == 0) {
        if (a.interleaved) rotary_kernel<__nv_bfloat16, true><<<n_tokens, kRotaryThreads, 0, stream>>>(a);
        else rotary_kernel<__nv_bfloat16, false><<<n_tokens, kRotaryThreads, 0, stream>>>(a);
    } else {
        if (a.interleaved) rotary_kernel<float, true><<<n_tokens, kRotaryThreads, 0, stream>>>(a);
        else rotary_kernel<float, false><<<n_tokens, kRotaryThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace pdattn
