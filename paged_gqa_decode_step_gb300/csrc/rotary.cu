// Rotary positions for long contexts: frequency tables, and the rotation of q
// and k by it (or back, which is the gradient).
//
// Pair i of a head vector turns by angle(pos, i) = pos * w_i:
//   y0 = x0 cos - x1 sin,  y1 = x1 cos + x0 sin   (sin negated for the inverse)
// with cos and sin times the frequencies' gain.  A rotation's inverse is its
// transpose, so the inverse call on an output's gradient is the input's.
//
// Angles.  The host holds w_i / (2 pi) in turns as a fraction of 2^64
// (pdattn_rotary.turns), to half a unit or a little more, which is 2^-33 turns at
// position 2^31.  pos * turns mod 2^64 is then the angle's place in its turn:
// one integer product, whose overflow drops the whole turns, where a product
// in f32 is off by 2^-24 of the angle (0.004 rad at position 131072).
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
// heads while the first vectors of the token load.
constexpr int kRotaryThreads = 128;

// The angles of the block's token into shared memory; false if it has none.
__device__ __forceinline__ bool token_angles(const RotaryArgs& a, float* s_cos, float* s_sin) {
    const int pos = __ldg(a.positions + blockIdx.x);
    if (pos < 0) {
        if (threadIdx.x == 0) set_error(reinterpret_cast<Ctrl*>(a.ws), kErrBadPos);
        return false;
    }
    for (int i = threadIdx.x; i < a.rot_dim / 2; i += kRotaryThreads) {
        float c, s;
        cos_sin((uint64_t)pos * a.turns[i], a.gain, c, s);
        s_cos[i] = c;
        s_sin[i] = a.inverse ? -s : s;
    }
    __syncthreads();
    return true;
}

// Half pairs.  A unit is the two vectors of N pairs, or one vector of
// dimensions past rot_dim.  (A division by `per` and 2 N shared reads of 4 bytes
// a unit: 8192 tokens of 40 heads of 128 26.5 us, half of each turned 31.4;
// now 26.2 and 27.5.  A thread that keeps to one unit of every head, as below,
// has too few heads of 8 vectors: 31.5 and 38.5.)
constexpr int kHalfAhead = 3;            // units a thread loads before it needs the angles (2: 26.7, 28.1)

template <typename T>
__global__ void __launch_bounds__(kRotaryThreads) rotary_half_kernel(const __grid_constant__ RotaryArgs a) {
    using V = Vec16<T>;
    constexpr int N = V::N;
    __shared__ __align__(16) float s_cos[kRotaryPairs], s_sin[kRotaryPairs];
    const int tok = blockIdx.x, tid = threadIdx.x;
    const int D = a.head_dim, rot = a.rot_dim, half = rot / 2, turned = half / N;
    const int per = turned + (D - rot) / N, units = per * (a.heads + a.kv_heads);
    const uint32_t magic = 0xffffffffu / per + 1;                      // u / per for u < 2^27
    const T* qi = static_cast<const T*>(a.q) + (size_t)tok * a.q_stride;
    const T* ki = static_cast<const T*>(a.k) + (size_t)tok * a.k_stride;
    T* qo = static_cast<T*>(a.q_out) + (size_t)tok * a.q_out_stride;
    T* ko = static_cast<T*>(a.k_out) + (size_t)tok * a.k_out_stride;
    // unit u: whether it is q's, its vector's place in a token and its first element
    auto place = [&](int u, bool& is_q, int& at, int& e) {
        const int h = (int)__umulhi((uint32_t)u, magic), v = u - h * per;
        e = v < turned ? v * N : rot + (v - turned) * N;
        is_q = h < a.heads;
        at = (is_q ? h : h - a.heads) * D + e;
    };
    uint4 x[kHalfAhead][2];
    auto load = [&](int u, uint4 (&r)[2]) {
        bool is_q;
        int at, e;
        place(u, is_q, at, e);
        const T* src = (is_q ? qi : ki) + at;
        r[0] = *reinterpret_cast<const uint4*>(src);
        if (e < rot) r[1] = *reinterpret_cast<const uint4*>(src + half);
    };
    #pragma unroll
    for (int k = 0; k < kHalfAhead; ++k)
        if (tid + k * kRotaryThreads < units) load(tid + k * kRotaryThreads, x[k]);
    if (!token_angles(a, s_cos, s_sin)) return;
    auto turn = [&](int u, const uint4 (&r)[2]) {
        bool is_q;
        int at, e;
        place(u, is_q, at, e);
        T* dst = (is_q ? qo : ko) + at;
        if (e >= rot) {
            *reinterpret_cast<uint4*>(dst) = r[0];
            return;
        }
        float f[N], g[N], y[N], z[N];
        V::to_f32(r[0], f);
        V::to_f32(r[1], g);
        float cc[N], ss[N];
        #pragma unroll
        for (int k = 0; k < N; k += 4) {
            *reinterpret_cast<float4*>(cc + k) = *reinterpret_cast<const float4*>(s_cos + e + k);
            *reinterpret_cast<float4*>(ss + k) = *reinterpret_cast<const float4*>(s_sin + e + k);
        }
        #pragma unroll
        for (int k = 0; k < N; ++k) {
            const float c = cc[k], s = ss[k];
            y[k] = f[k] * c - g[k] * s;
            z[k] = g[k] * c + f[k] * s;
        }
        *reinterpret_cast<uint4*>(dst) = V::from_f32(y);
        *reinterpret_cast<uint4*>(dst + half) = V::from_f32(z);
    };
    #pragma unroll
    for (int k = 0; k < kHalfAhead; ++k)
        if (tid + k * kRotaryThreads < units) turn(tid + k * kRotaryThreads, x[k]);
    for (int u = tid + kHalfAhead * kRotaryThreads; u < units; u += kRotaryThreads) {
        uint4 r[2];
        load(u, r);
        turn(u, r);
    }
}

// Interleaved pairs.  A thread takes the same vector of every H-th head (D / N
// divides the threads), so that it keeps its cos and sin in registers: with
// vectors in order and 2 N shared reads for each the schedulers were 80 % busy
// (8192 tokens of 40 heads of 128, half of each turned, 31.2 us; so 26.5).
constexpr int kPairAhead = 5;            // heads a thread has in flight (4: 28.4 us, 6: 27.9)

template <typename T>
__global__ void __launch_bounds__(kRotaryThreads) rotary_pair_kernel(const __grid_constant__ RotaryArgs a) {
    using V = Vec16<T>;
    constexpr int N = V::N;
    __shared__ __align__(16) float s_cos[kRotaryPairs], s_sin[kRotaryPairs];
    const int tok = blockIdx.x, tid = threadIdx.x, D = a.head_dim;
    const int per = D / N, H = kRotaryThreads / per, h0 = tid / per, e = (tid - h0 * per) * N;
    const int heads = a.heads + a.kv_heads;
    const T* qi = static_cast<const T*>(a.q) + (size_t)tok * a.q_stride + e;
    const T* ki = static_cast<const T*>(a.k) + (size_t)tok * a.k_stride + e;
    T* qo = static_cast<T*>(a.q_out) + (size_t)tok * a.q_out_stride + e;
    T* ko = static_cast<T*>(a.k_out) + (size_t)tok * a.k_out_stride + e;
    uint4 x[kPairAhead];
    auto load = [&](int hb) {
        #pragma unroll
        for (int k = 0; k < kPairAhead; ++k) {
            const int h = hb + k * H;
            if (h < heads) x[k] = *reinterpret_cast<const uint4*>(h < a.heads ? qi + h * D : ki + (h - a.heads) * D);
        }
    };
    load(h0);
    if (!token_angles(a, s_cos, s_sin)) return;
    const bool turns = e < a.rot_dim;
    float c[N / 2] = {}, s[N / 2] = {};
    if (turns) {
        #pragma unroll
        for (int k = 0; k < N / 2; ++k) {
            c[k] = s_cos[e / 2 + k];
            s[k] = s_sin[e / 2 + k];
        }
    }
    for (int hb = h0; hb < heads;) {
        #pragma unroll
        for (int k = 0; k < kPairAhead; ++k) {
            const int h = hb + k * H;
            if (h >= heads) continue;
            uint4 out = x[k];
            if (turns) {
                float f[N], y[N];
                V::to_f32(x[k], f);
                #pragma unroll
                for (int t = 0; t < N; t += 2) {
                    y[t] = f[t] * c[t / 2] - f[t + 1] * s[t / 2];
                    y[t + 1] = f[t + 1] * c[t / 2] + f[t] * s[t / 2];
                }
                out = V::from_f32(y);
            }
            *reinterpret_cast<uint4*>(h < a.heads ? qo + h * D : ko + (h - a.heads) * D) = out;
        }
        hb += kPairAhead * H;
        load(hb);
    }
}

}  // namespace

cudaError_t launch_rotary_tables(const RotaryArgs& a, int length, int dtype, void* cos_out, void* sin_out, int sms,
                                 cudaStream_t stream) {
    // sums: when the runs make a block for every SM
    const int runs = kRun * 256 / (a.head_dim / 16), each = 256 / (a.head_dim / (dtype == 0 ? 16 : 8));
    const bool sums = dtype == 0 && length >= (long long)sms * runs;
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
        if (a.interleaved) rotary_pair_kernel<__nv_bfloat16><<<n_tokens, kRotaryThreads, 0, stream>>>(a);
        else rotary_half_kernel<__nv_bfloat16><<<n_tokens, kRotaryThreads, 0, stream>>>(a);
    } else {
        if (a.interleaved) rotary_pair_kernel<float><<<n_tokens, kRotaryThreads, 0, stream>>>(a);
        else rotary_half_kernel<float><<<n_tokens, kRotaryThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace pdattn
