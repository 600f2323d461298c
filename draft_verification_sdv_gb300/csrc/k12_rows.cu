// k12_rows.cu -- draws from rows of logits and their truncation (sdv_sample,
// sdv_logits_truncate); k12_rows.cuh has the order and the weights.
//
// A CTA takes a row at a time and reads it in passes: the largest logit; a
// histogram of counts and weights over 4096 bins of equal width in (max - x) / T,
// which keeps the order; then, for each of the places that are asked for (the last
// token that min-p and top-k keep, the last that top-p keeps, the one that is
// drawn), the bin that holds it is split by keys until one logit is left.
#include "k12_rows.cuh"

namespace sdv {
namespace {

using namespace rows;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 4096, kPerThread = kBins / kThreads;
constexpr float kBinsPerHalving = 64.0f;

struct Hist {
    uint64_t mass[kBins];
    uint32_t count[kBins];
};

struct Smem {
    Tables tables;
    Hist first, next;
    uint64_t sum[2][kWarps];
    uint32_t word[kWarps];
    // what `locate` has found
    uint64_t before_w, at_w;
    uint32_t before_n, at_n;
    int bin;
};

// Where in the order a place lies: the logit there, and what comes before it.
struct Place {
    uint32_t key;
    uint32_t before_n, at_n;         // tokens of larger logits, and of this one
    uint64_t before_w;               // weight of the former
};

template <bool BF16> constexpr int kStep = BF16 ? 8 : 4;         // logits of 16 bytes

// Logits i0 .. of a row; past its end, -infinity (which no row counts).
template <bool BF16>
__device__ __forceinline__ void load_step(const unsigned char* row, int i0, int V, bool vec, float (&x)[kStep<BF16>]) {
    constexpr int E = kStep<BF16>;
    if (vec && i0 + E <= V) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + static_cast<int64_t>(i0) * (16 / E));
        if constexpr (BF16) {
            x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
            x[4] = bf16_lo(v.z), x[5] = bf16_hi(v.z), x[6] = bf16_lo(v.w), x[7] = bf16_hi(v.w);
        } else {
            x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
        }
    } else {
#pragma unroll
        for (int y = 0; y < E; ++y) x[y] = i0 + y < V ? load_logit(row, i0 + y, BF16) : -INFINITY;
    }
}

template <bool BF16>
__device__ __forceinline__ void store_step(unsigned char* row, int i0, int V, bool vec, const float (&x)[kStep<BF16>]) {
    constexpr int E = kStep<BF16>;
    uint32_t w[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        if constexpr (BF16)                          // (they come from bf16: nothing is rounded)
            w[y] = __byte_perm(__float_as_uint(x[2 * y]), __float_as_uint(x[2 * y + 1]), 0x7632);
        else
            w[y] = __float_as_uint(x[y]);
    }
    if (vec && i0 + E <= V) {
        *reinterpret_cast<uint4*>(row + static_cast<int64_t>(i0) * (16 / E)) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int y = 0; y < E; ++y) {
            if (i0 + y >= V) break;
            if constexpr (BF16)
                reinterpret_cast<unsigned short*>(row)[i0 + y] = static_cast<unsigned short>(w[y / 2] >> (16 * (y % 2)));
            else
                reinterpret_cast<uint32_t*>(row)[i0 + y] = w[y];
        }
    }
}

__device__ __forceinline__ uint32_t block_sum(uint32_t x, uint32_t* sm) {
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
    __syncthreads();
    uint32_t s = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sm[w];
    return s;
}

// The bin of a histogram where the running count (or weight) passes `target`:
// into sm.bin and what comes before it and lies in it.
__device__ __forceinline__ void pick(Smem& sm, const Hist& h, bool by_weight, uint64_t target) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t n = 0, w = 0;
    for (int i = 0; i < kPerThread; ++i) n += h.count[tid * kPerThread + i], w += h.mass[tid * kPerThread + i];
    uint64_t un = n, uw = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t a = __shfl_up_sync(0xffffffffu, un, o), b = __shfl_up_sync(0xffffffffu, uw, o);
        if (lane >= o) un += a, uw += b;
    }
    __syncthreads();
    if (lane == 31) sm.sum[0][warp] = un, sm.sum[1][warp] = uw;
    __syncthreads();
    un -= n, uw -= w;
    for (int i = 0; i < warp; ++i) un += sm.sum[0][i], uw += sm.sum[1][i];
    const uint64_t at = by_weight ? uw : un, own = by_weight ? w : n;
    if (at <= target && target < at + own) {
        for (int i = 0; i < kPerThread; ++i) {
            const uint32_t c = h.count[tid * kPerThread + i];
            const uint64_t m = h.mass[tid * kPerThread + i];
            if (target < (by_weight ? uw + m : un + c)) {
                sm.bin = tid * kPerThread + i;
                sm.before_n = static_cast<uint32_t>(un), sm.before_w = uw;
                sm.at_n = c, sm.at_w = m;
                break;
            }
            un += c, uw += m;
        }
    }
    __syncthreads();
}

template <bool BF16> struct Row {
    const unsigned char* at;
    int V;
    bool vec;
    Scale scale;
    float bins;                      // per unit of logit
    uint32_t low;                    // key of the smallest finite logit
    __device__ __forceinline__ int bin_of(float x) const {
        return static_cast<int>(fminf((scale.top - x) * bins, static_cast<float>(kBins - 1)));
    }
    template <class F> __device__ __forceinline__ void each(F f) const {
        constexpr int E = kStep<BF16>;
        for (int i0 = threadIdx.x * E; i0 < V; i0 += kThreads * E) {
            float x[E];
            load_step<BF16>(at, i0, V, vec, x);
#pragma unroll
            for (int y = 0; y < E; ++y) f(x[y]);
        }
    }
    // The place where the running count (weight) of the order passes `target`
    // (which lies below its total).
    __device__ Place locate(Smem& sm, bool by_weight, uint64_t target) const {
        pick(sm, sm.first, by_weight, target);
        Place p{0, sm.before_n, sm.at_n, sm.before_w};
        const int bin = sm.bin;
        // keys of the bin: the order of bins is that of keys, turned round
        uint32_t lo = low, hi = key_of(scale.top);
        for (uint32_t a = lo, b = hi; a < b;) {      // the smallest key whose bin is no later
            const uint32_t m = a + (b - a) / 2;
            if (bin_of(of_key(m)) <= bin)
                b = m;
            else
                a = m + 1;
            lo = b;
        }
        for (uint32_t a = lo, b = hi; a < b;) {      // the largest whose bin is no earlier
            const uint32_t m = b - (b - a) / 2;
            if (bin_of(of_key(m)) >= bin)
                a = m;
            else
                b = m - 1;
            hi = a;
        }
        for (int level = 0; level < 3 && lo != hi; ++level) {    // (a level settles 12 bits)
            int shift = 0;
            while ((hi - lo) >> shift >= kBins) ++shift;
            __syncthreads();
            for (int i = threadIdx.x; i < kBins; i += kThreads) sm.next.count[i] = 0, sm.next.mass[i] = 0;
            __syncthreads();
            each([&](float x) {
                const uint32_t k = key_of(x);
                if (k < lo || k > hi) return;
                atomicAdd(&sm.next.count[(hi - k) >> shift], 1u);
                atomicAdd(reinterpret_cast<unsigned long long*>(&sm.next.mass[(hi - k) >> shift]),
                          static_cast<unsigned long long>(weight_of(scale, x, sm.tables)));
            });
            __syncthreads();
            pick(sm, sm.next, by_weight, target - (by_weight ? p.before_w : p.before_n));
            p.before_n += sm.before_n, p.before_w += sm.before_w, p.at_n = sm.at_n;
            const uint32_t top = hi - (static_cast<uint32_t>(sm.bin) << shift), span = (1u << shift) - 1;
            lo = top - lo > span ? top - span : lo;
            hi = top;
        }
        p.key = lo;
        return p;
    }
};

// One row's parameters, checked.
struct Ask {
    float T, top_p, min_p, u;
    int top_k;
    bool bad;
};

__device__ __forceinline__ Ask ask_of(const RowsArgs& a, int64_t row) {
    const int64_t g = row / a.per;
    Ask q;
    q.T = a.temperature ? a.temperature[g] : 1.0f;
    q.top_k = a.top_k ? a.top_k[g] : 0;
    q.top_p = a.top_p ? a.top_p[g] : 1.0f;
    q.min_p = a.min_p ? a.min_p[g] : 0.0f;
    q.u = a.uniform ? a.uniform[row] : 0.0f;
    q.bad = !(q.T == 0.0f || (q.T >= 0x1p-64f && q.T <= 0x1p64f)) || q.top_k < 0 || !(q.top_p > 0.0f && q.top_p <= 1.0f) ||
            !(q.min_p >= 0.0f && q.min_p <= 1.0f) || !(q.u >= 0.0f && q.u < 1.0f);
    return q;
}

template <bool BF16, bool DRAW> __global__ void __launch_bounds__(kThreads) rows_kernel(const RowsArgs a) {
    constexpr int E = kStep<BF16>;
    extern __shared__ __align__(16) unsigned char raw[];
    Smem& sm = *reinterpret_cast<Smem*>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float nan = __int_as_float(0x7fc00000);
    for (int i = tid; i < 129; i += kThreads) sm.tables.coarse[i] = kTables.coarse[i], sm.tables.fine[i] = kTables.fine[i];
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const Ask q = ask_of(a, r);
        Row<BF16> row;
        row.at = static_cast<const unsigned char*>(a.logits) + r * a.in_stride;
        row.V = a.V;
        row.vec = (reinterpret_cast<uintptr_t>(row.at) & 15) == 0;
        unsigned char* out = static_cast<unsigned char*>(a.out) + r * a.out_stride;
        const bool out_vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0;

        // ---- the largest and the smallest logit, and how many there are ----
        uint32_t high = kKeyLow, low = kKeyHigh, finite = 0, odd = 0;
        row.each([&](float x) {
            const uint32_t k = key_of(x);
            odd |= x != x || x == INFINITY;
            if (x > -INFINITY) high = max(high, k), low = min(low, k), ++finite;
        });
        __syncthreads();
        high = __reduce_max_sync(0xffffffffu, high);
        low = __reduce_min_sync(0xffffffffu, low);
        if (lane == 0) sm.sum[0][warp] = high, sm.sum[1][warp] = low;
        for (int i = tid; i < kBins; i += kThreads) sm.first.count[i] = 0, sm.first.mass[i] = 0;
        odd = __syncthreads_or(odd);
        for (int i = 0; i < kWarps; ++i) high = max(high, static_cast<uint32_t>(sm.sum[0][i])), low = min(low, static_cast<uint32_t>(sm.sum[1][i]));
        finite = block_sum(finite, sm.word);
        if (q.bad || odd || finite == 0) {
            if (tid == 0) {
                if (a.status) atomicOr(a.status, q.bad ? kStatusBadTemp : kStatusBadRow);
                if (a.kept) a.kept[r] = 0;
                if (DRAW) a.tokens[r] = -1;
                if (DRAW && a.logprob) a.logprob[r] = nan;
            }
            if (!DRAW) {
                float x[E];
#pragma unroll
                for (int y = 0; y < E; ++y) x[y] = nan;
                for (int i0 = tid * E; i0 < a.V; i0 += kThreads * E) store_step<BF16>(out, i0, a.V, out_vec, x);
            }
            continue;
        }

        // ---- what is kept: the order up to `last` and the first `share` of its tokens ----
        const float top = of_key(high);
        row.low = low;
        Place last{low, 0, 0, 0};
        uint32_t kept = finite, share = 0;           // (share: of last.key's; unused while all are kept)
        uint64_t weight = 0;                         // of the kept
        Place drawn{high, 0, 0, 0};
        uint64_t aim = 0, unit = 0;
        if (q.T == 0.0f) {
            row.scale = Scale{top, 0.0f, 0.0f};
            kept = 1, share = 1, last.key = high;
            weight = unit = uint64_t(1) << kOneBits;
        } else {
            row.scale = scale_of(top, q.T);
            row.bins = kBinsPerHalving * 0.5f * row.scale.hi;
            const float floor = q.min_p > 0.0f ? __double2float_ru(static_cast<double>(top) + static_cast<double>(q.T) * log(static_cast<double>(q.min_p)))
                                               : -INFINITY;
            uint32_t over = 0;
            uint64_t sum = 0;
            row.each([&](float x) {
                if (!(x > -INFINITY)) return;
                const uint64_t w = weight_of(row.scale, x, sm.tables);
                const int b = row.bin_of(x);
                atomicAdd(&sm.first.count[b], 1u);
                atomicAdd(reinterpret_cast<unsigned long long*>(&sm.first.mass[b]), static_cast<unsigned long long>(w));
                over += x >= floor;
                sum += w;
            });
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            __syncthreads();
            if (lane == 0) sm.sum[0][warp] = sum;
            over = block_sum(over, sm.word);
            for (int i = 0; i < kWarps; ++i) weight += sm.sum[0][i];
            __syncthreads();
            uint32_t most = min(finite, over);
            if (q.top_k > 0) most = min(most, static_cast<uint32_t>(q.top_k));
            auto cut = [&](const Place& p, uint32_t n) {         // keeps n of the logits at p
                last = p;
                share = n;
                kept = p.before_n + n;
                weight = p.before_w + n * weight_of(row.scale, of_key(p.key), sm.tables);
            };
            if (most < finite) {
                const Place p = row.locate(sm, false, most - 1);
                cut(p, most - p.before_n);
            }
            if (q.top_p < 1.0f) {
                // tokens while what comes before them weighs less than this
                const uint64_t need = __double2ull_ru(static_cast<double>(q.top_p) * static_cast<double>(weight));
                const Place p = row.locate(sm, true, need - 1);
                cut(p, static_cast<uint32_t>((need - 1 - p.before_w) / weight_of(row.scale, of_key(p.key), sm.tables)) + 1);
            }
            if (DRAW) {
                aim = static_cast<uint64_t>(static_cast<double>(q.u) * static_cast<double>(weight));
                drawn = row.locate(sm, true, aim);
                unit = weight_of(row.scale, of_key(drawn.key), sm.tables);
            }
        }
        if (a.kept && tid == 0) a.kept[r] = static_cast<int32_t>(kept);

        // ---- tokens of one logit, counted in the order of their index ----
        // A warp looks after a run of the row, so that counts of runs place it.
        const uint32_t key = DRAW ? drawn.key : last.key;
        const uint32_t rank = DRAW ? static_cast<uint32_t>((aim - drawn.before_w) / unit) : share;
        const int steps = (a.V + 32 * E - 1) / (32 * E), run = (steps + kWarps - 1) / kWarps;
        const int s0 = min(warp * run, steps), s1 = min(s0 + run, steps);
        auto equals = [&](int s, float (&x)[E]) {    // of this lane's logits of step s
            load_step<BF16>(row.at, (s * 32 + lane) * E, a.V, row.vec, x);
            uint32_t m = 0;
#pragma unroll
            for (int y = 0; y < E; ++y) m |= (key_of(x[y]) == key && (s * 32 + lane) * E + y < a.V ? 1u : 0u) << y;
            return m;
        };
        const bool ranked = DRAW || (kept < finite);
        uint32_t mine = 0;
        if (ranked)
            for (int s = s0; s < s1; ++s) {
                float x[E];
                mine += __popc(equals(s, x));
            }
        mine = __reduce_add_sync(0xffffffffu, mine);
        __syncthreads();
        if (lane == 0) sm.word[warp] = mine;
        __syncthreads();
        uint32_t before = 0;
        for (int i = 0; i < warp; ++i) before += sm.word[i];
        if (!DRAW || (before <= rank && rank < before + mine)) {
            for (int s = s0; s < s1; ++s) {
                float x[E];
                const uint32_t m = equals(s, x), n = __popc(m);
                uint32_t upto = n;
                if (ranked && __any_sync(0xffffffffu, n)) {
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
                        if (lane >= o) upto += y;
                    }
                }
                uint32_t at = before + upto - n;
                before += __shfl_sync(0xffffffffu, upto, 31);
                if constexpr (DRAW) {
#pragma unroll
                    for (int y = 0; y < E; ++y)
                        if (m >> y & 1) {
                            if (at == rank) {
                                a.tokens[r] = (s * 32 + lane) * E + y;
                                if (a.logprob) {
                                    const uint64_t rest = weight - unit;
                                    const double part = rest < unit ? static_cast<double>(rest) : static_cast<double>(unit);
                                    const float f = static_cast<float>(part / static_cast<double>(weight));
                                    a.logprob[r] = rest < unit ? log1pf(-f) : logf(f);
                                }
                            }
                            ++at;
                        }
                } else {
                    if (ranked) {
#pragma unroll
                        for (int y = 0; y < E; ++y) {
                            const uint32_t k = key_of(x[y]);
                            if (k < key || (k == key && at >= rank)) x[y] = -INFINITY;
                            at += k == key;
                        }
                    }
                    store_step<BF16>(out, (s * 32 + lane) * E, a.V, out_vec, x);
                }
            }
        }
        __syncthreads();
    }
}

template <bool BF16, bool DRAW> cudaError_t launch(const RowsArgs& a, int nsm, cudaStream_t s) {
    const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(rows_kernel<BF16, DRAW>), sizeof(Smem));
    if (e != cudaSuccess) return e;
    const int64_t ctas = a.rows < 2 * nsm ? a.rows : 2 * nsm;
    rows_kernel<BF16, DRAW><<<static_cast<unsigned>(ctas), kThreads, sizeof(Smem), s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows(const RowsArgs& a, bool bf16, bool draw, int nsm, cudaStream_t s) {
    if (draw) return bf16 ? launch<true, true>(a, nsm, s) : launch<false, true>(a, nsm, s);
    return bf16 ? launch<true, false>(a, nsm, s) : launch<false, false>(a, nsm, s);
}

}  // namespace sdv
