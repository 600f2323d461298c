// k12_rows_bf16.cu -- draws from rows of logits and their truncation (sdv_sample,
// sdv_logits_truncate): rows in bf16.
//
// A bf16 logit is one of 2^16 values, so a row is counted once into a histogram
// of all of them, and everything that is asked for follows from the counts: the
// sum of count times weight over the few thousand values that occur, the last
// value that top-k, min-p and top-p keep, the one that a draw meets.  Only which
// token of that value it is takes a second look at the row, which is in L2 by then.
//
// The histogram holds 2^15 words in shared memory, one to a magnitude: its low
// half counts positive logits, its high half negative ones.  A half holds
// 65535; that none ran over shows in the sum of all counts, and a row where one did
// goes the long way (row_in_passes).
//
// An octave is the 128 magnitudes of one exponent.  A warp takes octaves in turn
// and sums counts and weights of those that are not empty; warp 0 adds up the
// 512 sums in the order of the logits and finds places in them, octave first.
#include <cuda_bf16.h>

#include "k12_rows.cuh"

namespace sdv {
namespace {

using namespace rows;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kWords = 1 << 15, kOctaves = 256, kSteps = 2 * kOctaves;     // steps: octaves of either sign
constexpr int kListed = 256;             // tokens of one value that are kept in a list

struct Sums {
    uint64_t mass[kSteps];               // step s < 256: positive octave 255 - s; else negative octave s - 256
    uint32_t count[kSteps];
    Tables tables;
    double inv_T, floor;                 // 2 log2(e) / T, T ln(min_p)
    uint32_t word[kWarps], word2[kWarps];
    uint32_t high;                       // how the largest logit stands in the order: its step and place
    uint32_t infinities;
    // what warp 0 has found
    uint32_t kept, key, share, at_n, rank;       // key: bits of a bf16
    uint64_t weight, unit;
    uint32_t listed, found;
    uint32_t list[kListed];
};

struct Smem {
    uint32_t count[kWords];              // or a PassSmem
    Sums s;
};
static_assert(sizeof(PassSmem<kThreads>) <= sizeof(uint32_t) * kWords, "the long way uses the histogram's place");
static_assert(sizeof(Smem) <= 227 * 1024, "one CTA per SM");

__device__ __forceinline__ uint4 ld_row(const unsigned char* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Counts one word's two logits: the magnitude's word, the sign's half of it.
__device__ __forceinline__ void count_two(uint32_t* h, uint32_t w) {
    unsigned char* at = reinterpret_cast<unsigned char*>(h);
    atomicAdd(reinterpret_cast<uint32_t*>(at + ((w << 2) & 0x1fffcu)), 1u << ((w >> 11) & 16u));
    atomicAdd(reinterpret_cast<uint32_t*>(at + ((w >> 14) & 0x1fffcu)), 1u << ((w >> 27) & 16u));
}
__device__ __forceinline__ void count_one(uint32_t* h, uint32_t bits) { atomicAdd(h + (bits & 0x7fffu), 1u << ((bits >> 11) & 16u)); }

__device__ __forceinline__ float value_of(uint32_t bits) { return __uint_as_float(bits << 16); }

__device__ __forceinline__ uint64_t warp_sum64(uint64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Four values of a step, in the order of the logits, that a lane looks after.
struct Four {
    uint32_t bits[4], count[4];
    uint64_t mass[4];
};
__device__ __forceinline__ Four four_of(const uint32_t* h, int step, int lane) {
    Four f;
    const bool neg = step >= kOctaves;
    const int first = neg ? (step - kOctaves) * 128 + 4 * lane : (kOctaves - 1 - step) * 128 + 124 - 4 * lane;
    const uint4 v = *reinterpret_cast<const uint4*>(h + first);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = neg ? w[i] : w[3 - i];
        f.count[i] = neg ? x >> 16 : x & 0xffffu;
        f.bits[i] = neg ? 0x8000u | static_cast<uint32_t>(first + i) : static_cast<uint32_t>(first + 3 - i);
    }
    return f;
}
__device__ __forceinline__ void weigh(Four& f, const Scale& scale, const Tables& t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f.mass[i] = f.count[i] ? f.count[i] * weight_of(scale, value_of(f.bits[i]), t) : 0;
}

// A lane's 16 steps: what comes before them, and what they hold.
struct Chunk {
    uint64_t before_w, own_w;
    uint32_t before_n, own_n;
};

struct Found {
    uint32_t bits, at_n, before_n;
    uint64_t before_w;
};

// The value where the running count (weight) of the order passes `target`.  Warp 0.
__device__ __forceinline__ Found find(const Smem& sm, const Chunk& c, const Scale& scale, bool by_weight, uint64_t target) {
    const int lane = threadIdx.x & 31;
    // the chunk, the step in it, the value in that
    const uint64_t at = by_weight ? c.before_w : c.before_n, own = by_weight ? c.own_w : c.own_n;
    const int src = __ffs(__ballot_sync(0xffffffffu, at <= target && target < at + own)) - 1;
    uint64_t bw = __shfl_sync(0xffffffffu, c.before_w, src);
    uint32_t bn = __shfl_sync(0xffffffffu, c.before_n, src);
    {
        const int s = src * 16 + (lane & 15);
        const uint64_t w = sm.s.mass[s];
        const uint32_t n = sm.s.count[s];
        uint64_t uw = w;
        uint32_t un = n;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
            const uint64_t x = __shfl_up_sync(0xffffffffu, uw, o, 16);
            const uint32_t y = __shfl_up_sync(0xffffffffu, un, o, 16);
            if ((lane & 15) >= o) uw += x, un += y;
        }
        const uint64_t upto = by_weight ? bw + uw : bn + un;
        const int in = __ffs(__ballot_sync(0xffffffffu, target < upto) | 0x8000u) - 1;
        bw += __shfl_sync(0xffffffffu, uw - w, in);
        bn += __shfl_sync(0xffffffffu, un - n, in);
        Four f = four_of(sm.count, src * 16 + in, lane);
        weigh(f, scale, sm.s.tables);
        uint64_t fw = (f.mass[0] + f.mass[1]) + (f.mass[2] + f.mass[3]);
        uint32_t fn = (f.count[0] + f.count[1]) + (f.count[2] + f.count[3]);
        uint64_t aw = fw;
        uint32_t an = fn;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t x = __shfl_up_sync(0xffffffffu, aw, o);
            const uint32_t y = __shfl_up_sync(0xffffffffu, an, o);
            if (lane >= o) aw += x, an += y;
        }
        const int who = __ffs(__ballot_sync(0xffffffffu, target < (by_weight ? bw + aw : bn + an)) | 0x80000000u) - 1;
        bw += aw - fw;                               // before this lane's four
        bn += an - fn;
        Found r{f.bits[3], f.count[3], bn, bw};
        bool done = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!done) r = Found{f.bits[i], f.count[i], bn, bw};
            done = done || target < (by_weight ? bw + f.mass[i] : static_cast<uint64_t>(bn) + f.count[i]);
            bw += f.mass[i], bn += f.count[i];
        }
        r.bits = __shfl_sync(0xffffffffu, r.bits, who);
        r.at_n = __shfl_sync(0xffffffffu, r.at_n, who);
        r.before_n = __shfl_sync(0xffffffffu, r.before_n, who);
        r.before_w = __shfl_sync(0xffffffffu, r.before_w, who);
        return r;
    }
}

// How many logits are at least `floor`.  Warp 0.
__device__ __forceinline__ uint32_t count_from(const Smem& sm, const Chunk& c, float floor) {
    const int lane = threadIdx.x & 31;
    // the last value of the order that is no smaller
    const uint32_t u = __float_as_uint(floor), mag = (u & 0x7fffffffu) >> 16;
    const bool neg = (u >> 31) != 0 && mag > 0;
    const uint32_t least = neg ? mag : (u >> 31) ? 0u : mag + ((u & 0xffffu) != 0);      // (of negative ones: the largest magnitude)
    const int step = neg ? kOctaves + static_cast<int>(least >> 7) : kOctaves - 1 - static_cast<int>(least >> 7);
    const int s = (step & ~15) + (lane & 15);
    uint32_t n = lane < 16 && s < step ? sm.s.count[s] : 0u;
    const Four f = four_of(sm.count, step, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t m = f.bits[i] & 0x7fffu;
        if (neg ? m <= least : m >= least) n += f.count[i];
    }
    return __reduce_add_sync(0xffffffffu, n) + __shfl_sync(0xffffffffu, c.before_n, step >> 4);
}

// Which halves of a word are this value (both zeros are one).
__device__ __forceinline__ uint32_t halves_of(uint32_t w, uint32_t pair, uint32_t sign) {
    const uint32_t t = (w & ~sign) ^ pair;
    return (t & 0xffffu ? 0u : 1u) | (t >> 16 ? 0u : 2u);
}

template <bool DRAW> __global__ void __launch_bounds__(kThreads) rows_bf16_kernel(const RowsArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    Smem& sm = *reinterpret_cast<Smem*>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float nan = __int_as_float(0x7fc00000);
    load_tables(sm.s.tables, tid, kThreads);
    for (int i = tid; i < kWords / 4; i += kThreads) reinterpret_cast<uint4*>(sm.count)[i] = make_uint4(0, 0, 0, 0);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const Ask q = ask_of(a, r);
        const unsigned char* row = static_cast<const unsigned char*>(a.logits) + r * a.in_stride;
        unsigned char* out = static_cast<unsigned char*>(a.out) + r * a.out_stride;
        const bool vec = (reinterpret_cast<uintptr_t>(row) & 15) == 0, out_vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
        const int vectors = vec ? a.V / 8 : 0;
        if (tid == kThreads - 1) {                   // (64-bit divisions take long: they are done by the time the row is counted)
            sm.s.listed = sm.s.found = 0;
            sm.s.inv_T = 2.8853900817779268147 / static_cast<double>(q.T);
            sm.s.floor = q.min_p > 0.0f ? static_cast<double>(q.T) * log(static_cast<double>(q.min_p)) : 0.0;
        }
        __syncthreads();

        // ---- every logit is counted ----
        constexpr int U = 4;
        int i = tid;
        for (; i + (U - 1) * kThreads < vectors; i += U * kThreads) {
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = ld_row(row + static_cast<int64_t>(i + u * kThreads) * 16);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                count_two(sm.count, v[u].x), count_two(sm.count, v[u].y);
                count_two(sm.count, v[u].z), count_two(sm.count, v[u].w);
            }
        }
        for (; i < vectors; i += kThreads) {
            const uint4 v = ld_row(row + static_cast<int64_t>(i) * 16);
            count_two(sm.count, v.x), count_two(sm.count, v.y), count_two(sm.count, v.z), count_two(sm.count, v.w);
        }
        for (int y = vectors * 8 + tid; y < a.V; y += kThreads) count_one(sm.count, reinterpret_cast<const unsigned short*>(row)[y]);
        __syncthreads();

        // ---- which octaves hold something, how much in all, the largest ----
        // (octave x * 32 + warp, a lane to four magnitudes)
        uint32_t some[2] = {0, 0}, total = 0, high = 0;      // high: 1 + the order turned round
        bool odd = false;
#pragma unroll
        for (int x = 0; x < kOctaves / kWarps; ++x) {
            const int o = x * kWarps + warp;
            uint4 v = reinterpret_cast<const uint4*>(sm.count)[o * 32 + lane];
            if (o == kOctaves - 1) {                 // infinities and what is not a number
                odd |= (v.y | v.z | v.w) != 0 || (lane == 0 ? (v.x & 0xffffu) != 0 : v.x != 0);
                if (lane == 0) sm.s.infinities = v.x >> 16;
                continue;
            }
            if (o == 0 && lane == 0) {               // both zeros count as the positive one
                const uint32_t zeros = (v.x & 0xffffu) + (v.x >> 16);
                if (zeros > 0xffffu)
                    total = 1u << 30;                // (as if a half had run over)
                else
                    sm.count[0] = v.x = zeros;
            }
            const uint32_t any = v.x | v.y | v.z | v.w;
            total += (v.x & 0xffffu) + (v.x >> 16) + (v.y & 0xffffu) + (v.y >> 16) + (v.z & 0xffffu) + (v.z >> 16) + (v.w & 0xffffu) + (v.w >> 16);
            if (__ballot_sync(0xffffffffu, (any & 0xffffu) != 0)) {
                some[0] |= 1u << x;
                const uint32_t top = v.w & 0xffffu ? 3 : v.z & 0xffffu ? 2 : v.y & 0xffffu ? 1 : 0;
                if (any & 0xffffu) high = max(high, 0x10000u + (o * 128 + lane * 4 + top));
            }
            if (__ballot_sync(0xffffffffu, (any >> 16) != 0)) {
                some[1] |= 1u << x;
                const uint32_t top = v.x >> 16 ? 0 : v.y >> 16 ? 1 : v.z >> 16 ? 2 : 3;
                if (any >> 16) high = max(high, 0x8000u - (o * 128 + lane * 4 + top));
            }
        }
        high = __reduce_max_sync(0xffffffffu, high);
        total = __reduce_add_sync(0xffffffffu, total);
        if (lane == 0) sm.s.word[warp] = high, sm.s.word2[warp] = total;
        odd = __syncthreads_or(odd);
        high = sm.s.word[lane], total = sm.s.word2[lane];
        high = __reduce_max_sync(0xffffffffu, high);
        total = __reduce_add_sync(0xffffffffu, total);
        // -infinities are counted modulo 2^16, which is their number if that is all that is missing
        bool over = total > static_cast<uint32_t>(a.V) || a.V - total != sm.s.infinities;
        if (over && total <= static_cast<uint32_t>(a.V) && !odd) {
            uint32_t n = 0;
            for (int y = tid; y < a.V; y += kThreads) n += reinterpret_cast<const unsigned short*>(row)[y] == 0xff80u;
            n = __reduce_add_sync(0xffffffffu, n);
            __syncthreads();
            if (lane == 0) sm.s.word2[warp] = n;
            __syncthreads();
            n = __reduce_add_sync(0xffffffffu, sm.s.word2[lane]);
            over = a.V - total != n;
        }
        const bool bad = q.bad || odd || (!over && total == 0);
        if (bad || over) {
            __syncthreads();
            if (!bad) {
                PassSmem<kThreads>& ps = *reinterpret_cast<PassSmem<kThreads>*>(raw);
                load_tables(ps.tables, tid, kThreads);
                __syncthreads();
                row_in_passes<true, DRAW, kThreads>(a, r, ps);
            } else {
                if (tid == 0) {
                    if (a.status) atomicOr(a.status, q.bad ? kStatusBadTemp : kStatusBadRow);
                    if (a.kept) a.kept[r] = 0;
                    if (DRAW) a.tokens[r] = -1;
                    if (DRAW && a.logprob) a.logprob[r] = nan;
                }
                if (!DRAW) {
                    float x[8];
#pragma unroll
                    for (int y = 0; y < 8; ++y) x[y] = nan;
                    for (int i0 = tid * 8; i0 < a.V; i0 += kThreads * 8) store_step<true>(out, i0, a.V, out_vec, x);
                }
            }
            __syncthreads();
            for (int x = tid; x < kWords / 4; x += kThreads) reinterpret_cast<uint4*>(sm.count)[x] = make_uint4(0, 0, 0, 0);
            continue;
        }

        // ---- weights ----
        Scale scale;
        scale.top = value_of(high >= 0x10000u ? high - 0x10000u : 0x8000u | (0x8000u - high));
        scale.hi = static_cast<float>(sm.s.inv_T);
        scale.lo = static_cast<float>(sm.s.inv_T - static_cast<double>(scale.hi));
        if (q.T != 0.0f) {
#pragma unroll 1
            for (int x = 0; x < 2 * (kOctaves / kWarps); ++x) {
                const int o = (x >> 1) * kWarps + warp, step = x & 1 ? kOctaves + o : kOctaves - 1 - o;
                uint64_t mass = 0;
                uint32_t n = 0;
                if (some[x & 1] >> (x >> 1) & 1) {
                    Four f = four_of(sm.count, step, lane);
                    weigh(f, scale, sm.s.tables);
                    mass = warp_sum64((f.mass[0] + f.mass[1]) + (f.mass[2] + f.mass[3]));
                    n = __reduce_add_sync(0xffffffffu, (f.count[0] + f.count[1]) + (f.count[2] + f.count[3]));
                }
                if (lane == 0) sm.s.mass[step] = mass, sm.s.count[step] = n;
            }
        }
        __syncthreads();

        // ---- what is kept, what is drawn ----
        if (warp == 0) {
            uint32_t kept = 1, share = 1, key = 0, at_n = 0, rank = 0;
            uint64_t weight = uint64_t(1) << kOneBits, unit = weight;
            const uint32_t best = __float_as_uint(scale.top) >> 16;
            if (q.T == 0.0f) {
                key = best;
                const uint32_t w = sm.count[best & 0x7fffu];
                at_n = best & 0x8000u ? w >> 16 : w & 0xffffu;
            } else {
                Chunk c{0, 0, 0, 0};
#pragma unroll
                for (int x = 0; x < 16; ++x) c.own_w += sm.s.mass[lane * 16 + x], c.own_n += sm.s.count[lane * 16 + x];
                c.before_w = c.own_w, c.before_n = c.own_n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t y = __shfl_up_sync(0xffffffffu, c.before_w, o);
                    const uint32_t z = __shfl_up_sync(0xffffffffu, c.before_n, o);
                    if (lane >= o) c.before_w += y, c.before_n += z;
                }
                weight = __shfl_sync(0xffffffffu, c.before_w, 31);
                c.before_w -= c.own_w, c.before_n -= c.own_n;
                uint32_t most = total;
                if (q.min_p > 0.0f) most = count_from(sm, c, __double2float_ru(static_cast<double>(scale.top) + sm.s.floor));
                if (q.top_k > 0) most = min(most, static_cast<uint32_t>(q.top_k));
                kept = total, share = 0;
                if (most < total) {
                    const Found f = find(sm, c, scale, false, most - 1);
                    key = f.bits, at_n = f.at_n, share = most - f.before_n, kept = most;
                    weight = f.before_w + share * weight_of(scale, value_of(key), sm.s.tables);
                }
                if (q.top_p < 1.0f) {
                    // tokens while what comes before them weighs less than this
                    const uint64_t need = __double2ull_ru(static_cast<double>(q.top_p) * static_cast<double>(weight));
                    const Found f = find(sm, c, scale, true, need - 1);
                    const uint64_t w = weight_of(scale, value_of(f.bits), sm.s.tables);
                    key = f.bits, at_n = f.at_n, share = static_cast<uint32_t>((need - 1 - f.before_w) / w) + 1;
                    kept = f.before_n + share;
                    weight = f.before_w + share * w;
                }
                if (DRAW) {
                    const uint64_t aim = static_cast<uint64_t>(static_cast<double>(q.u) * static_cast<double>(weight));
                    const Found f = find(sm, c, scale, true, aim);
                    key = f.bits, at_n = f.at_n;
                    unit = weight_of(scale, value_of(key), sm.s.tables);
                    rank = static_cast<uint32_t>((aim - f.before_w) / unit);
                }
            }
            if (lane == 0) {
                sm.s.kept = kept, sm.s.key = key, sm.s.share = share, sm.s.at_n = at_n, sm.s.rank = rank;
                if (a.kept) a.kept[r] = static_cast<int32_t>(kept);
                if (DRAW && a.logprob) {
                    const uint64_t rest = weight - unit;
                    const double part = rest < unit ? static_cast<double>(rest) : static_cast<double>(unit);
                    const float f = static_cast<float>(part / static_cast<double>(weight));
                    a.logprob[r] = rest < unit ? log1pf(-f) : logf(f);
                }
            }
        }
        __syncthreads();
        // the histogram is done with
#pragma unroll
        for (int x = 0; x < kOctaves / kWarps; ++x)
            if ((some[0] | some[1]) >> x & 1) reinterpret_cast<uint4*>(sm.count)[(x * kWarps + warp) * 32 + lane] = make_uint4(0, 0, 0, 0);
        if (warp == kWarps - 1) reinterpret_cast<uint4*>(sm.count)[(kOctaves - 1) * 32 + lane] = make_uint4(0, 0, 0, 0);

        // ---- the tokens of one value, by index ----
        const uint32_t key = sm.s.key, at_n = sm.s.at_n, rank = DRAW ? sm.s.rank : sm.s.share;
        const bool all = !DRAW && sm.s.kept == total;                // nothing is cut
        const uint32_t sign = (key & 0x7fffu) == 0 ? 0x80008000u : 0u, pair = (key & ~sign & 0xffffu) * 0x10001u;
        const bool some_stay = !DRAW && rank < at_n;                 // of the last value, the first `rank` stay
        if (DRAW && at_n <= kListed) {
            auto put = [&](uint32_t index) {
                const uint32_t n = atomicAdd(&sm.s.listed, 1u);
                if (n < kListed) sm.s.list[n] = index;
            };
            for (int v0 = tid; v0 < vectors; v0 += kThreads) {
                const uint4 v = ld_row(row + static_cast<int64_t>(v0) * 16);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const uint32_t m = halves_of(w[y], pair, sign);
                    if (m & 1) put(v0 * 8 + 2 * y);
                    if (m & 2) put(v0 * 8 + 2 * y + 1);
                }
                if (*reinterpret_cast<volatile uint32_t*>(&sm.s.listed) >= at_n) break;    // that was all of them
            }
            for (int y = vectors * 8 + tid; y < a.V; y += kThreads)
                if (halves_of(reinterpret_cast<const unsigned short*>(row)[y] | ~pair << 16, pair, sign) & 1) put(y);
            __syncthreads();
        }
        uint32_t last = 0;                                           // index of the token of that rank (a truncation: the first that goes)
        if (DRAW || some_stay) {
            if (at_n <= kListed) {
                if (DRAW && tid < static_cast<int>(at_n)) {
                    const uint32_t mine = sm.s.list[tid];
                    uint32_t before = 0;
                    for (uint32_t x = 0; x < at_n; ++x) before += sm.s.list[x] < mine;
                    if (before == rank) a.tokens[r] = static_cast<int32_t>(mine);
                }
            } else {
                // by runs of the row, a warp to each: counted, then the one that holds it
                const int run = (a.V + kWarps - 1) / kWarps, y0 = min(warp * run, a.V), y1 = min(y0 + run, a.V);
                auto is = [&](int y) { return y < y1 && (halves_of(reinterpret_cast<const unsigned short*>(row)[y] | ~pair << 16, pair, sign) & 1); };
                uint32_t n = 0;
                for (int y = y0 + lane; y < y1; y += 32) n += is(y);
                n = __reduce_add_sync(0xffffffffu, n);
                if (lane == 0) sm.s.word[warp] = n;
                __syncthreads();
                uint32_t before = 0;
                for (int x = 0; x < warp; ++x) before += sm.s.word[x];
                if (before <= rank && rank < before + n) {
                    for (int y = y0; y < y1; y += 32) {
                        const uint32_t m = __ballot_sync(0xffffffffu, is(y + lane));
                        const uint32_t here = __popc(m);
                        if (rank < before + here) {
                            if ((m >> lane & 1) && before + __popc(m & ((1u << lane) - 1u)) == rank) sm.s.found = y + lane;
                            break;
                        }
                        before += here;
                    }
                }
                __syncthreads();
                last = sm.s.found;
                if (DRAW && tid == 0) a.tokens[r] = static_cast<int32_t>(last);
            }
        }
        if constexpr (!DRAW) {
            // kept: above the last value, and of that one the first (by index) that stay
            const float least = all ? -INFINITY : value_of(key);
            const bool by_list = some_stay && at_n <= kListed, by_index = some_stay && !by_list;
            const __nv_bfloat162 bound = __floats2bfloat162_rn(least, least);
            auto cut = [&](uint32_t w, uint32_t index) {             // two logits, the first of this index
                const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w);
                uint32_t stay = by_list ? __hgt2_mask(x, bound) : __hge2_mask(x, bound);
                if (by_list || by_index) {
                    const uint32_t m = halves_of(w, pair, sign);
                    if (m & 1) {
                        if (by_index) stay = index < last ? stay : stay & 0xffff0000u;
                        else sm.s.list[atomicAdd(&sm.s.listed, 1u)] = index | (w & 0x8000u) << 16;
                    }
                    if (m & 2) {
                        if (by_index) stay = index + 1 < last ? stay : stay & 0x0000ffffu;
                        else sm.s.list[atomicAdd(&sm.s.listed, 1u)] = (index + 1) | (w & 0x80000000u);
                    }
                }
                return (w & stay) | (~stay & 0xff80ff80u);
            };
            if (out_vec) {
                for (int v0 = tid; v0 < vectors; v0 += kThreads) {
                    const uint4 v = ld_row(row + static_cast<int64_t>(v0) * 16);
                    *reinterpret_cast<uint4*>(out + static_cast<int64_t>(v0) * 16) =
                        make_uint4(cut(v.x, v0 * 8), cut(v.y, v0 * 8 + 2), cut(v.z, v0 * 8 + 4), cut(v.w, v0 * 8 + 6));
                }
            }
            for (int y = (out_vec ? vectors * 8 : 0) + tid; y < a.V; y += kThreads) {
                const uint32_t w = cut(reinterpret_cast<const unsigned short*>(row)[y] | ~pair << 16, y);
                reinterpret_cast<unsigned short*>(out)[y] = static_cast<unsigned short>(w);
            }
            if (by_list) {                                           // those that stay go back
                __syncthreads();
                if (tid < static_cast<int>(at_n)) {
                    const uint32_t mine = sm.s.list[tid], index = mine & 0x7fffffffu;
                    uint32_t before = 0;
                    for (uint32_t x = 0; x < at_n; ++x) before += (sm.s.list[x] & 0x7fffffffu) < index;
                    if (before < rank) reinterpret_cast<unsigned short*>(out)[index] = static_cast<unsigned short>(key | (mine >> 31) << 15);
                }
            }
        }
        __syncthreads();
    }
}

template <bool DRAW> cudaError_t launch(const RowsArgs& a, int nsm, cudaStream_t s) {
    const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(rows_bf16_kernel<DRAW>), sizeof(Smem));
    if (e != cudaSuccess) return e;
    const int64_t ctas = a.rows < nsm ? a.rows : nsm;
    rows_bf16_kernel<DRAW><<<static_cast<unsigned>(ctas), kThreads, sizeof(Smem), s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows_bf16(const RowsArgs& a, bool draw, int nsm, cudaStream_t s) {
    return draw ? launch<true>(a, nsm, s) : launch<false>(a, nsm, s);
}

}  // namespace sdv
