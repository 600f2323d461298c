// k12_rows.cuh -- what the kernels that draw from rows of logits share: whole
// weights, the order of a row's tokens, block sums.
//
// A row's tokens are ordered by falling logit, equal ones by index.  Token i weighs
//   w_i = 2^44 e^((x_i - max) / T)
// as a whole number, so that sums of weights are exact, the same in any order, and
// fit 64 bits (V <= 2^19).  Their products with u and top_p are exact too (times_down,
// times_up): what is kept and drawn does not depend on how the row was shared out.  What a
// row keeps is then a first part of that order (min-p, top-k and top-p each cut its
// end), and a draw is the token where the running sum of weights passes u times the
// sum of those kept.
//
// 2^44 e^(-d / T) is computed in pairs of fp32 numbers: p = d log2(e) / T to 2^-47
// of itself, 2^(frac p) as a product of two table entries (7 bits each) and
// 1 + z + z^2 / 2 + z^3 / 6 with |z| < 2^-14.9, in 62-bit fixed point: off by less
// than a unit.  Weights below 2^20 are fp32's, off by up to 0.7 units there (their
// exponent is rounded to 2^-20), but for a drawn token's logarithm.
#pragma once

#include "sdv_device.cuh"
#include "sdv_layer.h"
#include "sdv_plan.h"

namespace sdv {
namespace rows {

constexpr int kManyLogits = 1 << 16;         // from here on the bound of a head is taken from maxima of more logits
constexpr int kOneBits = 44;                 // the largest weight is 2^44
constexpr float kFallMost = 45.5f;           // a fall (in halvings) from which on a weight is 0
constexpr float kFallLight = 24.0f;          // ... and from which on fp32 gives it

// 2^(i / 128) and 2^(i / 2^14) for i = -64 .. 64, in units of 2^-62.
constexpr double exp_series(double x) {
    double term = 1.0, sum = 1.0;
    for (int i = 1; i < 24; ++i) {
        term *= x / i;
        sum += term;
    }
    return sum;
}
struct Tables {
    uint64_t coarse[129], fine[129];
};
constexpr Tables make_tables() {
    Tables t{};
    for (int i = 0; i < 129; ++i) {
        const double ln2 = 0.693147180559945309417;
        t.coarse[i] = static_cast<uint64_t>(exp_series((i - 64) / 128.0 * ln2) * 4611686018427387904.0);
        t.fine[i] = static_cast<uint64_t>(exp_series((i - 64) / 16384.0 * ln2) * 4611686018427387904.0);
    }
    return t;
}
__device__ constexpr Tables kTables = make_tables();

__device__ __forceinline__ void load_tables(Tables& t, int tid, int threads) {
    for (int i = tid; i < 129; i += threads) t.coarse[i] = kTables.coarse[i], t.fine[i] = kTables.fine[i];
}

// What turns a row's logits into weights.
struct Scale {
    float top;               // the row's largest logit
    float hi, lo;            // 2 log2(e) / T
};

// What one thread works out in 64 bits, of which an SM has few lanes: the factor,
// and how far below the largest logit min-p reaches (T ln(min_p)).
struct Factors {
    float hi, lo;
    double reach;
};
__device__ __forceinline__ Factors factors_of(float T, float min_p) {
    Factors f;
    const double c = 2.8853900817779268147 / static_cast<double>(T);
    f.hi = static_cast<float>(c);
    f.lo = static_cast<float>(c - static_cast<double>(f.hi));
    f.reach = min_p > 0.0f ? static_cast<double>(T) * log(static_cast<double>(min_p)) : 0.0;
    return f;
}
__device__ __forceinline__ float floor_of(float top, double reach) { return __double2float_ru(static_cast<double>(top) + reach); }

// How far x lies below the largest, in halvings of the weight, as an fp32
// number; `low` is what it lacks.
__device__ __forceinline__ float fall_of(const Scale& s, float x, float& low) {
    // the halves' difference does not overflow; what its rounding loses is exact
    const float a = 0.5f * s.top, b = -0.5f * x;
    const float d = a + b, bb = d - a;
    const float e = (a - (d - bb)) + (b - bb);
    const float p = __fmul_rn(d, s.hi);
    low = __fmaf_rn(d, s.hi, -p) + __fmaf_rn(d, s.lo, __fmul_rn(e, s.hi));
    return p;
}

// 2^(44 - p - low) to the next whole number, for p up to kFallMost.
__device__ __forceinline__ uint64_t weight_of_fall(float p, float low, const Tables& t) {
    const float k = rintf(p), f = k - p;                         // exact; 2^-p = 2^-k 2^f
    const int i = __float2int_rn(f * 128.0f);
    const float g = __fmaf_rn(static_cast<float>(i), -0x1p-7f, f);
    const int j = __float2int_rn(g * 16384.0f);
    const float h = __fmaf_rn(static_cast<float>(j), -0x1p-14f, g);
    const float z = h - low, zl = (h - z) - low;                 // |z| < 2^-14.9
    const float y = __fmul_rn(z, 0.693147182f);                  // z ln 2, and what that lacks
    const float yl = __fmaf_rn(z, 0.693147182f, -y) + __fmaf_rn(z, -1.90465421e-9f, __fmul_rn(zl, 0.693147182f));
    const float more = yl + __fmul_rn(__fmul_rn(y, y), __fmaf_rn(y, 0.166666667f, 0.5f));
    // (32-bit conversions: 64-bit ones share the few 64-bit lanes)
    const int32_t frac = __float2int_rn(y * 0x1p46f) + __float2int_rn(more * 0x1p46f);
    const uint64_t ab = __umul64hi(t.coarse[i + 64], t.fine[j + 64]) << 2;
    const uint64_t w = ab + static_cast<uint64_t>((static_cast<int64_t>(static_cast<uint32_t>(ab >> 31)) * frac) >> 15);   // 2^f in units of 2^-62
    const int shift = 62 - kOneBits + static_cast<int>(k);       // 18 .. 64
    return ((w >> (shift - 1)) + 1) >> 1;
}

// The whole weight of a logit that is at most the largest.  Most logits of a row weigh
// less than 2^20, which fp32 gives to a unit (the exponent is rounded to 2^-20).
__device__ __forceinline__ uint64_t weight_of(const Scale& s, float x, const Tables& t) {
    float low;
    const float p = fmaxf(fall_of(s, x, low), 0.0f);
    if (p >= kFallLight) return p < kFallMost ? __float2uint_rn(ex2((static_cast<float>(kOneBits) - p) - low)) : 0u;
    if (x == s.top) return uint64_t(1) << kOneBits;
    return weight_of_fall(p, low, t);
}

// a / b, less than 2^20: off by one at most in fp32.
__device__ __forceinline__ uint32_t quotient(uint64_t a, uint64_t b) {
    uint32_t q = __float2uint_rz(__fdividef(__ull2float_rn(a), __ull2float_rn(b)));
    while (q * b > a) --q;
    while ((q + 1) * b <= a) ++q;
    return q;
}

// The same place in another CTA of the cluster.
template <int C, class T> __device__ __forceinline__ T* of_rank(T* p, uint32_t rank) {
    if constexpr (C == 1) return p;
    T* r;
    asm volatile("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(p), "r"(rank));
    return r;
}
template <int C> __device__ __forceinline__ void sync_all() {
    if constexpr (C == 1) {
        __syncthreads();
    } else {
        __syncwarp();
        cluster_sync();
    }
}

// The first look at a row leaves its lines in L2 as any read does, the last one and the results
// do not.  (Lines marked to stay, evict_last, made no call faster, 1088 rows of 152064 truncated in
// 209 us either way, and a kernel behind it that reads 100 MB over and over slower for good, 25.6 us
// against 19.5.  Reads without a policy: 226 us.)
__device__ __forceinline__ uint64_t first_policy() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t drop_policy() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint4 ld_hint(const unsigned char* p, uint64_t policy) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p), "l"(policy));
    return v;
}
__device__ __forceinline__ void st_hint(unsigned char* p, const uint4& v, uint64_t policy) {
    asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "l"(policy) : "memory");
}
__device__ __forceinline__ uint4 ld_row(const unsigned char* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// The fourth smallest of N numbers in shared memory, equal ones taken as one (the smallest
// of 16 differ much).  A whole warp.
template <int N> __device__ __forceinline__ uint32_t fourth_smallest(const uint32_t* words) {
    const int lane = threadIdx.x & 31;
    uint32_t mine[(N + 31) / 32], found = 0;
#pragma unroll
    for (int x = 0; x < (N + 31) / 32; ++x) mine[x] = x * 32 + lane < N ? words[x * 32 + lane] : 0xffffffffu;
#pragma unroll
    for (int turn = 0; turn < 4; ++turn) {
        uint32_t m = 0xffffffffu;
#pragma unroll
        for (int x = 0; x < (N + 31) / 32; ++x) m = min(m, mine[x]);
        found = __reduce_min_sync(0xffffffffu, m);
#pragma unroll
        for (int x = 0; x < (N + 31) / 32; ++x) mine[x] = mine[x] == found ? 0xffffffffu : mine[x];
    }
    return found;
}

// u * w and p * w for an fp32 number in [0, 1), exact but for the last step: rounded
// down, or up.
__device__ __forceinline__ uint64_t times_down(float u, uint64_t w) {
    const int e = static_cast<int>(__float_as_uint(u) >> 23);                  // u = m 2^(max(e, 1) - 150)
    const uint64_t m = (__float_as_uint(u) & 0x7fffffu) | (e > 0 ? 0x800000u : 0u);
    const int shift = 150 - (e > 0 ? e : 1);                     // 24 .. 149
    const uint64_t lo = m * w, hi = __umul64hi(m, w);
    if (shift >= 128) return 0;
    return shift >= 64 ? hi >> (shift - 64) : (lo >> shift) | (hi << (64 - shift));
}
__device__ __forceinline__ uint64_t times_up(float p, uint64_t w) {
    const int e = static_cast<int>(__float_as_uint(p) >> 23);
    const uint64_t m = (__float_as_uint(p) & 0x7fffffu) | (e > 0 ? 0x800000u : 0u);
    const int shift = 150 - (e > 0 ? e : 1);
    const uint64_t lo = m * w, hi = __umul64hi(m, w);
    if (shift >= 128) return 1;                                  // (neither is 0)
    const uint64_t down = shift >= 64 ? hi >> (shift - 64) : (lo >> shift) | (hi << (64 - shift));
    const bool left = shift >= 64 ? lo != 0 || (hi & ((uint64_t(1) << (shift - 64)) - 1)) != 0 : (lo & ((uint64_t(1) << shift) - 1)) != 0;
    return down + left;
}

// ln(w / weight) for a drawn logit of weight `unit`.  A light one's is worked out again:
// being off by one would show in the logarithm (5e-6 at 2^17.5).
static __device__ __noinline__ float log_share(const Scale& s, float x, uint64_t unit, uint64_t weight, const Tables& t) {
    if (unit < uint64_t(1) << 21) {                  // (2^20 and the one after among them)
        float low;
        const float p = fall_of(s, x, low);
        if (p >= kFallLight && p < kFallMost) unit = max(weight_of_fall(p, low, t), uint64_t(1));
    }
    const uint64_t rest = weight - unit;
    const float f = __ull2float_rn(rest < unit ? rest : unit) / __ull2float_rn(weight);
    return rest < unit ? log1pf(-f) : logf(f);
}

// Logits in order: a larger one has a larger key, and both zeros the same.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = x == 0.0f ? 0u : __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
constexpr uint32_t kKeyLow = 0x007fffffu;    // -infinity
constexpr uint32_t kKeyHigh = 0xff800000u;   // +infinity; keys outside the two are not numbers


template <int BINS> struct Hist {
    uint64_t mass[BINS];
    uint32_t count[BINS];
};

// A weight into a shared sum, in 32-bit steps: 64-bit ones go round a loop.
__device__ __forceinline__ void add_weight(uint64_t* sum, uint64_t w) {
    uint32_t* at = reinterpret_cast<uint32_t*>(sum);
    const uint32_t lo = static_cast<uint32_t>(w);
    uint32_t hi = static_cast<uint32_t>(w >> 32);
    if (lo && atomicAdd(at, lo) > ~lo) ++hi;         // (it ran over)
    if (hi) atomicAdd(at + 1, hi);
}

// What `pick` finds, and its room.
template <int THREADS> struct Picked {
    uint64_t sum[2][THREADS / 32];
    uint64_t before_w, at_w;
    uint32_t before_n, at_n;
    int bin;
};

template <int THREADS, int BINS> struct PassSmem : Picked<THREADS> {
    Tables tables;
    Hist<BINS> first, next;
    uint32_t word[THREADS / 32];
    Factors factors;
    float floor;
};

// Where in the order a place lies: the logit there, and what comes before it.
struct Place {
    uint32_t key;
    uint32_t before_n, at_n;         // tokens of larger logits, and of this one
    uint64_t before_w;               // weight of the former
};

// A row in 16-byte vectors: the logits before the first that lies on 16 bytes, the
// vectors, and those after the last.  Loose ones are counted through: first the former.
struct Span {
    int head, vectors, loose, width;
    __device__ __forceinline__ int index_of(int v) const { return head + v * width; }
    __device__ __forceinline__ int loose_at(int i) const { return i < head ? i : i + vectors * width; }
};
__device__ __forceinline__ Span span_of(const unsigned char* row, int V, int bytes) {
    Span s;
    s.width = 16 / bytes;
    s.head = static_cast<int>((0u - static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row))) & 15u) / bytes;
    s.head = s.head < V ? s.head : V;
    s.vectors = (V - s.head) / s.width;
    s.loose = V - s.vectors * s.width;
    return s;
}

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

template <int THREADS> __device__ __forceinline__ uint32_t block_sum(uint32_t x, uint32_t* sm) {
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
    __syncthreads();
    uint32_t s = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) s += sm[w];
    return s;
}

// The bin of a histogram where the running count (or weight) passes `target`:
// into sm.bin and what comes before it and lies in it.
template <int THREADS, int BINS>
__device__ __forceinline__ void pick(Picked<THREADS>& sm, const Hist<BINS>& h, bool by_weight, uint64_t target) {
    constexpr int kPerThread = BINS / THREADS;
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

template <bool BF16, int THREADS, int BINS> struct Row {
    const unsigned char* at;
    int V;
    bool vec;
    Scale scale;
    float bins;                      // per unit of logit
    uint32_t low;                    // key of the smallest finite logit
    __device__ __forceinline__ int bin_of(float x) const {
        return static_cast<int>(fminf((scale.top - x) * bins, static_cast<float>(BINS - 1)));
    }
    template <class F> __device__ __forceinline__ void each(F f) const {
        constexpr int E = kStep<BF16>;
        for (int i0 = threadIdx.x * E; i0 < V; i0 += THREADS * E) {
            float x[E];
            load_step<BF16>(at, i0, V, vec, x);
#pragma unroll
            for (int y = 0; y < E; ++y) f(x[y]);
        }
    }
    // The place where the running count (weight) of the order passes `target`
    // (which lies below its total).
    __device__ Place locate(PassSmem<THREADS, BINS>& sm, bool by_weight, uint64_t target) const {
        pick<THREADS, BINS>(sm, sm.first, by_weight, target);
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
        for (int level = 0; level < 4 && lo != hi; ++level) {    // (a level settles 10 bits or more)
            int shift = 0;
            while ((hi - lo) >> shift >= BINS) ++shift;
            __syncthreads();
            for (int i = threadIdx.x; i < BINS; i += THREADS) sm.next.count[i] = 0, sm.next.mass[i] = 0;
            __syncthreads();
            each([&](float x) {
                const uint32_t k = key_of(x);
                if (k < lo || k > hi) return;
                atomicAdd(&sm.next.count[(hi - k) >> shift], 1u);
                add_weight(&sm.next.mass[(hi - k) >> shift], weight_of(scale, x, sm.tables));
            });
            __syncthreads();
            pick<THREADS, BINS>(sm, sm.next, by_weight, target - (by_weight ? p.before_w : p.before_n));
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
    const uint32_t g = a.per == 1 ? static_cast<uint32_t>(row) : static_cast<uint32_t>(row) / static_cast<uint32_t>(a.per);
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

// One row, in passes: for rows in 32 bits, and for those in 16 whose counts do not fit
// k12_rows_bf16.cu's.  All threads of the CTA; sm.tables is filled.
template <bool BF16, bool DRAW, int THREADS, int BINS>
__device__ __noinline__ void row_in_passes(const RowsArgs& a, int64_t r, PassSmem<THREADS, BINS>& sm) {
    constexpr int E = kStep<BF16>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float nan = __int_as_float(0x7fc00000);
    const Ask q = ask_of(a, r);
    Row<BF16, THREADS, BINS> row;
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
    for (int i = tid; i < BINS; i += THREADS) sm.first.count[i] = 0, sm.first.mass[i] = 0;
    odd = __syncthreads_or(odd);
    for (int i = 0; i < (THREADS / 32); ++i) high = max(high, static_cast<uint32_t>(sm.sum[0][i])), low = min(low, static_cast<uint32_t>(sm.sum[1][i]));
    finite = block_sum<THREADS>(finite, sm.word);
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
            for (int i0 = tid * E; i0 < a.V; i0 += THREADS * E) store_step<BF16>(out, i0, a.V, out_vec, x);
        }
        return;
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
        if (tid == 0) {
            sm.factors = factors_of(q.T, q.min_p);
            sm.floor = q.min_p > 0.0f ? floor_of(top, sm.factors.reach) : -INFINITY;
        }
        __syncthreads();
        row.scale = Scale{top, sm.factors.hi, sm.factors.lo};
        row.bins = (BINS / 64) * 0.5f * row.scale.hi;
        const float floor = sm.floor;
        uint32_t over = 0;
        uint64_t sum = 0;
        row.each([&](float x) {
            if (!(x > -INFINITY)) return;
            const uint64_t w = weight_of(row.scale, x, sm.tables);
            const int b = row.bin_of(x);
            atomicAdd(&sm.first.count[b], 1u);
            add_weight(&sm.first.mass[b], w);
            over += x >= floor;
            sum += w;
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        __syncthreads();
        if (lane == 0) sm.sum[0][warp] = sum;
        over = block_sum<THREADS>(over, sm.word);
        for (int i = 0; i < (THREADS / 32); ++i) weight += sm.sum[0][i];
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
            const uint64_t need = times_up(q.top_p, weight);
            const Place p = row.locate(sm, true, need - 1);
            cut(p, quotient(need - 1 - p.before_w, weight_of(row.scale, of_key(p.key), sm.tables)) + 1);
        }
        if (DRAW) {
            aim = times_down(q.u, weight);
            drawn = row.locate(sm, true, aim);
            unit = weight_of(row.scale, of_key(drawn.key), sm.tables);
        }
    }
    if (a.kept && tid == 0) a.kept[r] = static_cast<int32_t>(kept);

    // ---- tokens of one logit, counted in the order of their index ----
    // A warp looks after a run of the row, so that counts of runs place it.
    const uint32_t key = DRAW ? drawn.key : last.key;
    const uint32_t rank = DRAW ? quotient(aim - drawn.before_w, unit) : share;
    const int steps = (a.V + 32 * E - 1) / (32 * E), run = (steps + (THREADS / 32) - 1) / (THREADS / 32);
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
                            if (a.logprob) a.logprob[r] = log_share(row.scale, of_key(key), unit, weight, sm.tables);
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

}  // namespace rows

cudaError_t launch_rows_bf16(const RowsArgs& a, bool draw, int nsm, cudaStream_t s);
}  // namespace sdv
