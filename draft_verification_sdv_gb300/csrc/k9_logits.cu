// k9_logits.cu -- sampling parameters (penalties for repeated tokens, biases,
// grammar masks) on the logits of every draft position, and the update of the
// token counts after a step.
//
// Row (b, k, j) counts the history of sequence b and the first j tokens of
// draft k, so the rows of one draft differ by one token from one to the next.
// A CTA therefore owns a slice of the vocabulary and walks the rows of one
// sequence, draft by draft: the counts, prompt bits and biases of its slice stay
// with their threads (in registers, but for one array that the compiler keeps in
// local memory; the counts are read again at each draft's start), and the thread
// that owns draft token j counts it after row j.
//
// Bound by HBM: each logit is read and written once (2 + 2 bytes in bf16, and a
// bit of the grammar mask).  Four rows are in flight per thread.  32 sequences of
// 8 drafts of 16 tokens, 152064 logits a row under a grammar: 512 us, 5.2 TB/s.
// What is left: four rows are loaded, then worked on, and nothing is in flight
// meanwhile (issue slots 58 % and DRAM 51 % of the time on a quarter of the rows).
#include <cuda_bf16.h>

#include "sdv_device.cuh"
#include "sdv_layer.h"
#include "sdv_plan.h"

namespace sdv {
namespace {

constexpr int kThreads = 256;
constexpr int kFlight = 4;            // rows in flight per thread
constexpr int kBiasPass = 1024;       // biases sorted at a time
constexpr int kRowsMost = 1024;       // rows of a CTA

template <bool BF16>
__global__ void __launch_bounds__(kThreads) logits_kernel(const LogitsArgs a) {
    constexpr int E = BF16 ? 8 : 4;                 // logits of a 16-byte vector
    constexpr int kSlice = kThreads * E;
    __shared__ int s_n;
    __shared__ int2 s_raw[kBiasPass];               // (place in the list, id)
    __shared__ int2 s_bias[kBiasPass];              // (id, value) in the list's order
    __shared__ int2 s_row[kRowsMost];               // source row, the draft token after it (-1: none)
    const unsigned slices = (static_cast<unsigned>(a.V) + kSlice - 1) / kSlice;
    const int b = static_cast<int>(blockIdx.x / slices);
    const int slice0 = static_cast<int>(blockIdx.x % slices) * kSlice;
    const int v0 = slice0 + threadIdx.x * E;        // this thread's first token
    const bool live = v0 < a.V;                     // V is a multiple of E
    const int rows = a.G + 1;                       // of a draft
    const int64_t all = static_cast<int64_t>(a.K) * rows;
    const int r0 = static_cast<int>(blockIdx.y * all / a.row_splits);
    const int r1 = static_cast<int>((blockIdx.y + 1) * all / a.row_splits);

    for (int i = threadIdx.x; i < r1 - r0; i += kThreads) {
        const int r = r0 + i, k = r / rows, j = r - k * rows;
        const int64_t at = b * all + r;
        int src = r;
        if (a.rows) {
            src = a.rows[at];
            if (src < 0 || src >= a.nsrc) {
                src = -1;
                if (slice0 == 0 && a.status) atomicOr(a.status, kStatusBadLength);
            }
        }
        s_row[i] = make_int2(src, j < a.G ? a.drafts[(static_cast<int64_t>(b) * a.K + k) * a.G + j] : -1);
    }
    __syncthreads();
    const float rep = a.rep ? a.rep[b] : 1.0f;
    // bf16 logits are multiplied by 1 / rep, a rounding of fp32 more before the one to
    // bf16 (where rep or its reciprocal leaves fp32's normal numbers, by that of rep in
    // units of 2^64); fp32 logits get the quotient itself.  (The quotient for bf16 too:
    // 664 us in the place of 536; the product for fp32 too, half the sequences: 507 us
    // in the place of 527.)
    const float unit = fabsf(rep) > 4.25e37f ? 1.8446744e19f : fabsf(rep) < 2.35e-38f ? 5.4210109e-20f : 1.0f;
    const float inv = unit == 1.0f ? 1.0f / rep : 1.0f / (rep / unit), by = 1.0f / unit;
    const float freq = a.freq ? a.freq[b] : 0.0f, pres = a.pres ? a.pres[b] : 0.0f;
    int c[E];
    float bias[E], add[E];
    unsigned prompt = 0, seen = 0;                  // bit e: in the prompt; the repetition penalty applies
#pragma unroll
    for (int e = 0; e < E; ++e) bias[e] = 0.0f;
    if (live && a.prompt)
        prompt = static_cast<unsigned>(__ldg(a.prompt + static_cast<int64_t>(b) * a.W + (v0 >> 5))) >> (v0 & 31);
    for (int m0 = 0; m0 < a.M; m0 += kBiasPass) {   // the biases that fall into the slice
        if (threadIdx.x == 0) s_n = 0;
        __syncthreads();
        for (int m = m0 + threadIdx.x; m < min(m0 + kBiasPass, a.M); m += kThreads) {
            const int id = a.bias_ids[static_cast<int64_t>(b) * a.M + m];
            if (id >= slice0 && id < slice0 + kSlice && id < a.V)
                s_raw[atomicAdd(&s_n, 1)] = make_int2(m, id);
        }
        __syncthreads();
        const int n = s_n;
        for (int i = threadIdx.x; i < n; i += kThreads) {     // in the list's order
            int at = 0;
            for (int x = 0; x < n; ++x) at += s_raw[x].x < s_raw[i].x;
            s_bias[at] = make_int2(s_raw[i].y, __float_as_int(
                a.bias[static_cast<int64_t>(b) * a.M + s_raw[i].x]));
        }
        __syncthreads();
        for (int i = 0; i < n; ++i) {
            const int off = s_bias[i].x - v0;
            if (off >= 0 && off < E) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (e == off) bias[e] += __int_as_float(s_bias[i].y);
            }
        }
        __syncthreads();
    }
    if (!live) return;

    auto history = [&] {                            // the counts before a draft's first token
#pragma unroll
        for (int e = 0; e < E; ++e) c[e] = 0;
        if (a.counts) {
            const int4* p = reinterpret_cast<const int4*>(a.counts + static_cast<int64_t>(b) * a.V + v0);
#pragma unroll
            for (int u = 0; u < E / 4; ++u) {
                const int4 x = __ldg(p + u);
                c[4 * u] = x.x, c[4 * u + 1] = x.y, c[4 * u + 2] = x.z, c[4 * u + 3] = x.w;
            }
        }
    };
    auto count_token = [&](int tok) {
        if (tok < v0 || tok >= v0 + E) return false;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e == tok - v0) ++c[e];
        return true;
    };
    auto settle = [&] {                             // what the counts come to
        seen = prompt;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (c[e] > 0) seen |= 1u << e;
            add[e] = (bias[e] - freq * static_cast<float>(c[e])) - (c[e] > 0 ? pres : 0.0f);
        }
    };
    const int32_t* dr = a.drafts + static_cast<int64_t>(b) * a.K * a.G;
    const int k0 = r0 / rows;
    int j = r0 - k0 * rows;                         // the next row's place in its draft
    history();
    for (int i = 0; i < j; ++i) count_token(dr[k0 * a.G + i]);
    settle();

    const int64_t row0 = b * all, nvec = a.V / E;
    const uint4* in = static_cast<const uint4*>(a.logits) + (a.rows ? static_cast<int64_t>(b) * a.nsrc : row0) * nvec + v0 / E;
    uint4* out = static_cast<uint4*>(a.out) + row0 * nvec + v0 / E;
    const int32_t* allow = a.allow ? a.allow + row0 * a.W + (v0 >> 5) : nullptr;

    for (int r = r0; r < r1; r += kFlight) {
        uint4 x[kFlight];
        unsigned ok[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            if (r + u >= r1) break;
            const int src = s_row[r + u - r0].x;
            ok[u] = allow ? static_cast<unsigned>(__ldg(allow + static_cast<int64_t>(r + u) * a.W)) >> (v0 & 31)
                          : 0xffffffffu;
            if (src >= 0)
                x[u] = __ldcs(in + src * nvec);
            else                                    // NaN in either type
                x[u] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u), ok[u] = ~0u;
        }
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            if (r + u >= r1) break;
            if (j == rows) {                        // the next draft
                j = 0;
                history();
                settle();
            }
            const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            float f[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                f[e] = BF16 ? ((e & 1) ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2])) : __uint_as_float(w[e % 4]);
            }
            if (!BF16) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (seen >> e & 1) f[e] = f[e] > 0.0f ? f[e] / rep : f[e] * rep;
            } else if (by == 1.0f) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (seen >> e & 1) f[e] *= f[e] > 0.0f ? inv : rep;
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (seen >> e & 1) f[e] = f[e] > 0.0f ? f[e] * inv * by : f[e] * rep;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                f[e] += add[e];
                if (!(ok[u] >> e & 1)) f[e] = -INFINITY;
            }
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (BF16) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                    o[i] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                    o[i] = __float_as_uint(f[i]);
                }
            }
            __stcs(out + static_cast<int64_t>(r + u) * nvec, make_uint4(o[0], o[1], o[2], o[3]));
            if (count_token(s_row[r + u - r0].y)) settle();
            ++j;
        }
    }
}

__global__ void __launch_bounds__(128) counts_kernel(const CountsArgs a) {
    const int b = blockIdx.x;
    const int sel = a.sel[b], acc = a.acc[b];
    if (sel == -1) return;
    if (sel < 0 || sel >= a.K || acc < 0 || acc > a.G) {
        if (threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadLength);
        return;
    }
    for (int i = threadIdx.x; i <= acc; i += blockDim.x) {
        const int tok = i < acc ? a.drafts[(static_cast<int64_t>(b) * a.K + sel) * a.G + i] : a.next[b];
        if (tok >= 0 && tok < a.V)
            atomicAdd(a.counts + static_cast<int64_t>(b) * a.V + tok, 1);   // whole numbers: any order
        else if (a.status)
            atomicOr(a.status, kStatusBadDraft);
    }
}

}  // namespace

cudaError_t launch_logits(const LogitsArgs& args, bool bf16, int nsm, cudaStream_t s) {
    LogitsArgs a = args;
    const int slice = kThreads * (bf16 ? 8 : 4);
    const int64_t base = static_cast<int64_t>((a.V + slice - 1) / slice) * a.B;
    // Few sequences: their rows are shared out until every SM has about eight
    // CTAs, a CTA keeping four rows at least (its counts and biases serve those).
    // One sequence of 4 x 17 rows: 31 us against 43 us in one share; two of 8 x 17:
    // 51 against 72; eight of 4 x 17: 78 against 74.
    const int64_t all = static_cast<int64_t>(a.K) * (a.G + 1);
    int64_t split = (static_cast<int64_t>(nsm) * 8 + base - 1) / base;
    const int64_t most = (all + kFlight - 1) / kFlight;
    split = split > most ? most : split;
    const int64_t least = (all + kRowsMost - 1) / kRowsMost;
    a.row_splits = static_cast<int>(split < least ? least : split);
    const dim3 grid(static_cast<unsigned>(base), static_cast<unsigned>(a.row_splits));
    if (bf16)
        logits_kernel<true><<<grid, kThreads, 0, s>>>(a);
    else
        logits_kernel<false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_counts_commit(const CountsArgs& a, cudaStream_t s) {
    counts_kernel<<<static_cast<unsigned>(a.B), 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace sdv
