// k6_rope.cu -- rotary positions of queries and keys in one launch.
//
// Pair i of token t turns by pos_t * f_i.  In fp32 that product loses the
// angle at far positions, and fp64 is slow here, so the angle is kept as a
// 64-bit fraction of a turn: F_i = f_i / 2 pi mod 1 in units of 2^-64, and
// pos * F mod 2^64 is the angle's fraction (integer products wrap by themselves),
// off by pos units at most: 2^-33 of a turn.  F needs more digits than one fp64
// product has (2^-55 of a turn off, times 2^31), so it is the sum of a product, of
// what that lost (one fma) and of f times the next digits of 1 / 2 pi.  Sine and
// cosine are taken of the top 32 bits, rounded to fp32: 2^-26 of a turn.
//
// Bound by HBM: every element is read and written once.  A CTA takes a few
// tokens at a time, computes their R / 2 sines and cosines once for all heads
// into shared memory, then walks the heads with 16-byte loads: one work item is
// the pairs of two vectors of one head, so that both halves of a pair are in
// one thread for either layout.  16416 tokens of 72 heads of 128: 97 us, 6.2 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sdv_layer.h"

namespace sdv {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;          // tokens of a CTA's step

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f(float x) { return x; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

template <typename T> struct alignas(16) Vec { T x[16 / sizeof(T)]; };

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
    extern __shared__ float2 cs[];                  // [kTokens][R / 2] (cos, sin) * factor
    const int half = a.R / 2, heads = a.Hq + a.Hk;
    constexpr int E = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;   // elements of a vector
    const int turn_items = VEC ? a.R / (2 * E) : half;      // items of pairs per head
    const int copy_items = VEC ? (a.D - a.R) / E : a.D - a.R;
    const bool in_place = a.q == a.oq && (a.k == a.ok || !a.Hk);
    const int items = turn_items + (in_place ? 0 : copy_items);

    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens; t0 < a.T;
         t0 += static_cast<int64_t>(gridDim.x) * kTokens) {
        const int nt = static_cast<int>(a.T - t0 < kTokens ? a.T - t0 : kTokens);
        for (int i = threadIdx.x; i < half; i += kThreads) {
            const float f = a.freq[i];
            constexpr double kInv = 0.15915494309189535, kInvLow = -9.839338337591243e-18;   // 1 / (2 pi)
            constexpr double kUnits = 18446744073709551616.0;
            const double d = f, turns = d * kInv, low = fma(d, kInv, -turns) + d * kInvLow;
            const unsigned long long F = static_cast<unsigned long long>(__double2ll_rn((turns - rint(turns)) * kUnits)) +
                                         static_cast<unsigned long long>(__double2ll_rn(low * kUnits));
            for (int t = 0; t < nt; ++t) {
                const long long p = a.pos[t0 + t];
                const int frac = static_cast<int>((static_cast<unsigned long long>(p) * F) >> 32);
                float s, c;
                sincospif(static_cast<float>(frac) * 4.656612873077393e-10f, &s, &c);   // 2^-31
                if (!(fabsf(f) < INFINITY)) s = c = __int_as_float(0x7fc00000);
                cs[t * half + i] = make_float2(c * a.factor, s * a.factor);
            }
        }
        __syncthreads();
        const int total = nt * heads * items;
        for (int w = threadIdx.x; w < total; w += kThreads) {
            const int item = w % items, th = w / items;
            const int head = th % heads, t = th / heads;
            const bool isq = head < a.Hq;
            const int hh = isq ? head : head - a.Hq;
            const char* src = static_cast<const char*>(isq ? a.q : a.k) +
                              (t0 + t) * (isq ? a.q_st : a.k_st) + hh * (isq ? a.q_sh : a.k_sh);
            char* dst = static_cast<char*>(isq ? a.oq : a.ok) +
                        (t0 + t) * (isq ? a.oq_st : a.ok_st) + hh * (isq ? a.oq_sh : a.ok_sh);
            using V = Vec<T>;
            if (item >= turn_items) {               // past the rotated part: copied
                const int e = a.R + (item - turn_items) * E;
                if constexpr (VEC)
                    reinterpret_cast<V*>(dst)[e / E] = reinterpret_cast<const V*>(src)[e / E];
                else
                    reinterpret_cast<T*>(dst)[e] = reinterpret_cast<const T*>(src)[e];
                continue;
            }
            const int i0 = item * E;                // first pair of the item
            const float2* ang = cs + t * half + i0;
            const int ea = a.interleaved ? 2 * i0 : i0, eb = a.interleaved ? 2 * i0 + E : i0 + half;
            if constexpr (VEC) {
                const V va = reinterpret_cast<const V*>(src)[ea / E];
                const V vb = reinterpret_cast<const V*>(src)[eb / E];
                V ra, rb;
                if (a.interleaved) {
#pragma unroll
                    for (int j = 0; j < E / 2; ++j) {
                        const float2 u = ang[j], v = ang[j + E / 2];
                        const float x0 = to_f(va.x[2 * j]), y0 = to_f(va.x[2 * j + 1]);
                        const float x1 = to_f(vb.x[2 * j]), y1 = to_f(vb.x[2 * j + 1]);
                        ra.x[2 * j] = from_f<T>(x0 * u.x - y0 * u.y);
                        ra.x[2 * j + 1] = from_f<T>(y0 * u.x + x0 * u.y);
                        rb.x[2 * j] = from_f<T>(x1 * v.x - y1 * v.y);
                        rb.x[2 * j + 1] = from_f<T>(y1 * v.x + x1 * v.y);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < E; ++j) {
                        const float2 u = ang[j];
                        const float x = to_f(va.x[j]), y = to_f(vb.x[j]);
                        ra.x[j] = from_f<T>(x * u.x - y * u.y);
                        rb.x[j] = from_f<T>(y * u.x + x * u.y);
                    }
                }
                reinterpret_cast<V*>(dst)[ea / E] = ra;
                reinterpret_cast<V*>(dst)[eb / E] = rb;
            } else {
                const int e1 = a.interleaved ? 2 * i0 + 1 : i0 + half;
                const float x = to_f(reinterpret_cast<const T*>(src)[ea]);
                const float y = to_f(reinterpret_cast<const T*>(src)[e1]);
                reinterpret_cast<T*>(dst)[ea] = from_f<T>(x * ang->x - y * ang->y);
                reinterpret_cast<T*>(dst)[e1] = from_f<T>(y * ang->x + x * ang->y);
            }
        }
        __syncthreads();
    }
}

template <typename T>
cudaError_t launch(const RopeArgs& a, bool vec, int nsm, cudaStream_t s) {
    const int64_t steps = (a.T + kTokens - 1) / kTokens, most = static_cast<int64_t>(nsm) * 8;
    const unsigned grid = static_cast<unsigned>(steps < most ? steps : most);
    const size_t smem = static_cast<size_t>(kTokens) * (a.R / 2) * sizeof(float2);
    if (vec)
        rope_kernel<T, true><<<grid, kThreads, smem, s>>>(a);
    else
        rope_kernel<T, false><<<grid, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int type, bool vec, int nsm, cudaStream_t s) {
    if (type == kTypeBf16) return launch<__nv_bfloat16>(a, vec, nsm, s);
    if (type == kTypeF16) return launch<__half>(a, vec, nsm, s);
    return launch<float>(a, vec, nsm, s);
}

}  // namespace sdv
