// k12_rows_bf16.cu -- draws from rows of logits and their truncation (sdv_sample,
// sdv_logits_truncate): rows in bf16.
//
// A bf16 logit is one of few values, so a row is counted once into a histogram of
// all of them, and everything that is asked for follows from the counts: the sum
// of count times weight over the few thousand values that occur, the last value
// that top-k, min-p and top-p keep, the one that a draw meets.  Only which token of
// that value it is takes a second look at the row, which is in L2 by then.
//
// The histogram has a word for each magnitude from 2^-40 to 2^24, 64 octaves of 128
// (32 KB, so that two CTAs share an SM and one counts while the other looks for
// its places); its low half counts positive logits, its high half negative ones.
// Zeros and -infinity are counted in registers.  A row that holds something else, or
// more of one value than a half can count (which shows in the sum of all counts)
// goes the long way, row_in_passes.
//
// Few rows are shared by a cluster of C CTAs, each of which counts a C-th of the
// row; octave o is looked after by CTA o % C, which adds up the C counts.  A warp
// takes an octave at a time and sums its counts and weights; warp 0 of the first CTA
// adds up the 129 sums (octaves of either sign, zeros between them) in the order
// of the logits and finds places in them, octave first.
#include <cuda_bf16.h>

#include "k12_rows.cuh"

namespace sdv {
namespace {

using namespace rows;

constexpr int kThreads = 512, kWarps = kThreads / 32, kPassBins = 1024;
constexpr int kOctaves = 64, kFirstOctave = 127 - 40, kWords = kOctaves * 128, kBase = kFirstOctave * 128;
constexpr int kZeroStep = kOctaves, kSteps = 2 * kOctaves + 1;   // step s < 64: positive octave 63 - s; s > 64: negative octave s - 65
constexpr int kChunk = 5, kPadded = 32 * kChunk;                 // steps of a lane of warp 0
static_assert(kPadded >= kSteps, "a lane holds five steps");
constexpr int kListed = 256;             // tokens of one value that are kept in a list

// What a CTA says of its part of a row, or of its octaves.
struct Note {
    uint32_t total, zeros, infinities, odd, high;
};
enum : uint32_t { kOddNan = 1u, kOddFar = 2u };

struct Smem {
    uint32_t count[kWords];              // or a PassSmem
    uint64_t mass[kPadded];
    uint32_t steps[kPadded];             // counts
    Tables tables;
    Factors factors;
    Note part[8], whole[8];              // of each CTA of the cluster
    uint32_t word[8 * kWarps];
    // what warp 0 has found
    uint32_t kept, key, share, at_n, rank;       // key: bits of a bf16
    uint32_t listed, found;
    uint32_t list[kListed];
};
static_assert(sizeof(PassSmem<kThreads, kPassBins>) <= sizeof(uint32_t) * kWords, "the long way uses the histogram's place");
static_assert(2 * (sizeof(Smem) + 1024) <= 227 * 1024, "two CTAs per SM");

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

__device__ __forceinline__ uint4 ld_row(const unsigned char* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ float value_of(uint32_t bits) { return __uint_as_float(bits << 16); }

// A thread's counts of what has no word.
struct Rest {
    uint32_t zeros, infinities, odd;
};

// Counts a logit, given as its magnitude's distance from the first word and its sign's half.
__device__ __forceinline__ void count_one(uint32_t* h, Rest& rest, uint32_t mag, uint32_t one) {
    const uint32_t at = mag - kBase;
    if (at < kWords) {
        atomicAdd(h + at, one);
    } else {
        const bool zero = mag == 0, inf = mag == 0x7f80u && one != 1u;
        rest.zeros += zero;
        rest.infinities += inf;
        rest.odd |= zero || inf ? 0u : mag >= 0x7f80u ? kOddNan : kOddFar;
    }
}
__device__ __forceinline__ void count_two(uint32_t* h, Rest& rest, uint32_t w) {
    count_one(h, rest, w & 0x7fffu, 1u << ((w >> 11) & 16u));
    count_one(h, rest, (w >> 16) & 0x7fffu, 1u << ((w >> 27) & 16u));
}

__device__ __forceinline__ uint64_t warp_sum64(uint64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Four values of a step (not the zeros'), in the order of the logits, that a lane looks after.
struct Four {
    uint32_t bits[4], count[4];
    uint64_t mass[4];
};
template <int C> __device__ __forceinline__ Four four_of(const uint32_t* h, int step, int lane) {
    Four f;
    const bool neg = step > kZeroStep;
    const int first = neg ? (step - kZeroStep - 1) * 128 + 4 * lane : (kOctaves - 1 - step) * 128 + 124 - 4 * lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f.count[i] = 0;
        f.bits[i] = neg ? 0x8000u | static_cast<uint32_t>(kBase + first + i) : static_cast<uint32_t>(kBase + first + 3 - i);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(of_rank<C>(h + first, c));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f.count[i] += neg ? w[i] >> 16 : w[3 - i] & 0xffffu;
    }
    return f;
}
__device__ __forceinline__ void weigh(Four& f, const Scale& scale, const Tables& t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f.mass[i] = 0;
        if (__any_sync(0xffffffffu, f.count[i] != 0)) f.mass[i] = f.count[i] * weight_of(scale, value_of(f.bits[i]), t);
    }
}

// A lane's steps: what comes before them, and what they hold.
struct Chunk {
    uint64_t before_w, own_w;
    uint32_t before_n, own_n;
};

struct Found {
    uint32_t bits, at_n, before_n;
    uint64_t before_w;
};

// The value where the running count (weight) of the order passes `target`.  Warp 0.
template <int C>
__device__ __forceinline__ Found find(const Smem& sm, const Chunk& c, const Scale& scale, bool by_weight, uint64_t target) {
    const int lane = threadIdx.x & 31;
    // the chunk, the step in it, the value in that
    const uint64_t at = by_weight ? c.before_w : c.before_n, own = by_weight ? c.own_w : c.own_n;
    const int src = __ffs(__ballot_sync(0xffffffffu, at <= target && target < at + own) | 0x80000000u) - 1;
    uint64_t bw = __shfl_sync(0xffffffffu, c.before_w, src);
    uint32_t bn = __shfl_sync(0xffffffffu, c.before_n, src);
    int step = src * kChunk;
#pragma unroll
    for (int i = 0; i < kChunk - 1; ++i) {
        const uint64_t w = sm.mass[step];
        const uint32_t n = sm.steps[step];
        if (target < (by_weight ? bw + w : static_cast<uint64_t>(bn) + n)) break;
        bw += w, bn += n, ++step;
    }
    step = min(step, kSteps - 1);
    if (step == kZeroStep) return Found{0, sm.steps[step], bn, bw};
    Four f = four_of<C>(sm.count, step, lane);
    weigh(f, scale, sm.tables);
    const uint64_t fw = (f.mass[0] + f.mass[1]) + (f.mass[2] + f.mass[3]);
    const uint32_t fn = (f.count[0] + f.count[1]) + (f.count[2] + f.count[3]);
    uint64_t aw = fw;
    uint32_t an = fn;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, aw, o);
        const uint32_t y = __shfl_up_sync(0xffffffffu, an, o);
        if (lane >= o) aw += x, an += y;
    }
    const int who = __ffs(__ballot_sync(0xffffffffu, target < (by_weight ? bw + aw : static_cast<uint64_t>(bn) + an)) | 0x80000000u) - 1;
    bw += aw - fw;                                   // before this lane's four
    bn += an - fn;
    Found r{0, 0, 0, 0};
    bool done = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (!done) r = Found{f.bits[i], f.count[i], bn, bw};
        bw += f.mass[i], bn += f.count[i];
        done = done || target < (by_weight ? bw : static_cast<uint64_t>(bn));
    }
    r.bits = __shfl_sync(0xffffffffu, r.bits, who);
    r.at_n = __shfl_sync(0xffffffffu, r.at_n, who);
    r.before_n = __shfl_sync(0xffffffffu, r.before_n, who);
    r.before_w = __shfl_sync(0xffffffffu, r.before_w, who);
    return r;
}

// How many logits are at least `floor` (no larger than the largest).  Warp 0.
template <int C> __device__ __forceinline__ uint32_t count_from(const Smem& sm, float floor) {
    const int lane = threadIdx.x & 31;
    const uint32_t u = __float_as_uint(floor), cut = (u & 0x7fffffffu) >> 16;
    const bool neg = (u >> 31) != 0;
    // a negative floor: magnitudes up to `edge` of the negative ones; else those from it on
    const uint32_t edge = neg ? cut : cut + ((u & 0xffffu) != 0);
    const int o = static_cast<int>(edge >> 7) - kFirstOctave;
    // whole steps before `step`, and part of that one (none where it is past the octaves)
    int step = neg ? (floor == 0.0f || o < 0 ? kZeroStep + 1 : kZeroStep + 1 + min(o, kOctaves)) : o < 0 ? (floor == 0.0f ? kZeroStep + 1 : kZeroStep) : kOctaves - 1 - o;
    step = max(step, 0);
    const bool part = !(neg && floor == 0.0f) && o >= 0 && o < kOctaves;
    uint32_t n = 0;
    for (int s = lane; s < step; s += 32) n += sm.steps[s];
    if (part) {
        const Four f = four_of<C>(sm.count, step, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t m = f.bits[i] & 0x7fffu;
            if (neg ? m <= edge : m >= edge) n += f.count[i];
        }
    }
    return __reduce_add_sync(0xffffffffu, n);
}

// Which halves of a word are this value (both zeros are one).
__device__ __forceinline__ uint32_t halves_of(uint32_t w, uint32_t pair, uint32_t sign) {
    const uint32_t t = (w & ~sign) ^ pair;
    return (t & 0xffffu ? 0u : 1u) | (t >> 16 ? 0u : 2u);
}

template <bool DRAW, int C> __global__ void __launch_bounds__(kThreads, 2) rows_bf16_kernel(const RowsArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    Smem& sm = *reinterpret_cast<Smem*>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int me = rank * kThreads + tid;            // among the cluster's threads
    constexpr int kAll = C * kThreads;
    const float nan = __int_as_float(0x7fc00000);
    Smem* const lead = of_rank<C>(&sm, 0);
    load_tables(sm.tables, tid, kThreads);
    for (int i = tid; i < kWords / 4; i += kThreads) reinterpret_cast<uint4*>(sm.count)[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < kPadded; i += kThreads) sm.mass[i] = 0, sm.steps[i] = 0;
    if (tid == 0) sm.listed = 0;
    for (int64_t r = blockIdx.x / C; r < a.rows; r += gridDim.x / C) {
        const Ask q = ask_of(a, r);
        const unsigned char* row = static_cast<const unsigned char*>(a.logits) + r * a.in_stride;
        unsigned char* out = static_cast<unsigned char*>(a.out) + r * a.out_stride;
        const bool vec = (reinterpret_cast<uintptr_t>(row) & 15) == 0, out_vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
        const int vectors = vec ? a.V / 8 : 0;
        const unsigned short* cells = reinterpret_cast<const unsigned short*>(row);
        sync_all<C>();                               // (the row before is done with shared memory)
        if (tid == kThreads - 1) sm.factors = factors_of(q.T, q.min_p);

        // ---- every logit is counted ----
        Rest rest{0, 0, 0};
        constexpr int U = 4;
        int i = me;
        for (; i + (U - 1) * kAll < vectors; i += U * kAll) {
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = ld_row(row + static_cast<int64_t>(i + u * kAll) * 16);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                count_two(sm.count, rest, v[u].x), count_two(sm.count, rest, v[u].y);
                count_two(sm.count, rest, v[u].z), count_two(sm.count, rest, v[u].w);
            }
        }
        for (; i < vectors; i += kAll) {
            const uint4 v = ld_row(row + static_cast<int64_t>(i) * 16);
            count_two(sm.count, rest, v.x), count_two(sm.count, rest, v.y);
            count_two(sm.count, rest, v.z), count_two(sm.count, rest, v.w);
        }
        for (int y = vectors * 8 + me; y < a.V; y += kAll) count_one(sm.count, rest, cells[y] & 0x7fffu, 1u << ((cells[y] >> 11) & 16u));
        rest.zeros = __reduce_add_sync(0xffffffffu, rest.zeros);
        rest.infinities = __reduce_add_sync(0xffffffffu, rest.infinities);
        rest.odd = __reduce_or_sync(0xffffffffu, rest.odd);
        if (lane == 0) sm.list[warp] = rest.zeros, sm.list[kWarps + warp] = rest.infinities, sm.list[2 * kWarps + warp] = rest.odd;
        sync_all<C>();

        // ---- which octaves hold something, how much in all, the largest ----
        // (octaves of this CTA, a warp to each, a lane to four magnitudes)
        constexpr int kMine = kOctaves / (C * kWarps) > 0 ? kOctaves / (C * kWarps) : 1;
        uint32_t some[2] = {0, 0}, total = 0, high = 0;      // high: 0x8000 and how far the largest lies above zero
#pragma unroll
        for (int x = 0; x < kMine; ++x) {
            const int o = (x * kWarps + warp) * C + rank;
            if (o >= kOctaves) break;
            uint32_t any = 0, top[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const uint4 v = reinterpret_cast<const uint4*>(of_rank<C>(sm.count, c))[o * 32 + lane];
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    total += (w[y] & 0xffffu) + (w[y] >> 16);
                    any |= w[y];
                    if (w[y] & 0xffffu) top[0] = max(top[0], static_cast<uint32_t>(y));
                    if (w[y] >> 16) top[1] = max(top[1], static_cast<uint32_t>(3 - y));
                }
            }
            if (any & 0xffffu) high = max(high, 0x8000u + kBase + o * 128 + lane * 4 + top[0]);
            if (any >> 16) high = max(high, 0x8000u - (kBase + o * 128 + lane * 4 + 3 - top[1]));
            some[0] |= (__ballot_sync(0xffffffffu, (any & 0xffffu) != 0) != 0 ? 1u : 0u) << x;
            some[1] |= (__ballot_sync(0xffffffffu, (any >> 16) != 0) != 0 ? 1u : 0u) << x;
        }
        high = __reduce_max_sync(0xffffffffu, high);
        total = __reduce_add_sync(0xffffffffu, total);
        if (lane == 0) sm.word[warp] = high, sm.word[kWarps + warp] = total;
        __syncthreads();
        if (warp == 0) {
            const int w = lane % kWarps;
            Note n;
            n.high = __reduce_max_sync(0xffffffffu, sm.word[w]);
            n.odd = __reduce_or_sync(0xffffffffu, sm.list[2 * kWarps + w]);
            n.total = __reduce_add_sync(0xffffffffu, lane < kWarps ? sm.word[kWarps + w] : 0u);
            n.zeros = __reduce_add_sync(0xffffffffu, lane < kWarps ? sm.list[w] : 0u);
            n.infinities = __reduce_add_sync(0xffffffffu, lane < kWarps ? sm.list[kWarps + w] : 0u);
            if (lane < C) *of_rank<C>(&sm.part[rank], lane) = n;
        }
        sync_all<C>();
        Note all = sm.part[0];
#pragma unroll
        for (int c = 1; c < C; ++c) {
            const Note n = sm.part[c];
            all.total += n.total, all.zeros += n.zeros, all.infinities += n.infinities;
            all.odd |= n.odd, all.high = max(all.high, n.high);
        }
        if (all.zeros) all.high = max(all.high, 0x8000u);
        total = all.total + all.zeros;               // finite logits
        const bool over = (all.odd & kOddFar) || total + all.infinities != static_cast<uint32_t>(a.V);
        const bool bad = q.bad || (all.odd & kOddNan) || (!over && total == 0);
        if (bad || over) {
            sync_all<C>();                           // (nobody reads another's counts any more)
            if (!bad) {
                if (rank == 0) {
                    PassSmem<kThreads, kPassBins>& ps = *reinterpret_cast<PassSmem<kThreads, kPassBins>*>(raw);
                    load_tables(ps.tables, tid, kThreads);
                    __syncthreads();
                    row_in_passes<true, DRAW, kThreads, kPassBins>(a, r, ps);
                    __syncthreads();
                }
            } else {
                if (me == 0) {
                    if (a.status) atomicOr(a.status, q.bad ? kStatusBadTemp : kStatusBadRow);
                    if (a.kept) a.kept[r] = 0;
                    if (DRAW) a.tokens[r] = -1;
                    if (DRAW && a.logprob) a.logprob[r] = nan;
                }
                if (!DRAW) {
                    float x[8];
#pragma unroll
                    for (int y = 0; y < 8; ++y) x[y] = nan;
                    for (int i0 = me * 8; i0 < a.V; i0 += kAll * 8) store_step<true>(out, i0, a.V, out_vec, x);
                }
            }
            for (int x = tid; x < kWords / 4; x += kThreads) reinterpret_cast<uint4*>(sm.count)[x] = make_uint4(0, 0, 0, 0);
            continue;
        }

        // ---- weights ----
        const uint32_t best = all.high >= 0x8000u ? all.high - 0x8000u : 0x8000u | (0x8000u - all.high);
        const Scale scale{value_of(best), sm.factors.hi, sm.factors.lo};
        if (q.T != 0.0f) {
#pragma unroll 1
            for (int x = 0; x < 2 * kMine; ++x) {
                const int o = ((x >> 1) * kWarps + warp) * C + rank, step = x & 1 ? kZeroStep + 1 + o : kOctaves - 1 - o;
                if (o >= kOctaves) break;
                uint64_t mass = 0;
                uint32_t n = 0;
                if (some[x & 1] >> (x >> 1) & 1) {
                    Four f = four_of<C>(sm.count, step, lane);
                    weigh(f, scale, sm.tables);
                    mass = warp_sum64((f.mass[0] + f.mass[1]) + (f.mass[2] + f.mass[3]));
                    n = __reduce_add_sync(0xffffffffu, (f.count[0] + f.count[1]) + (f.count[2] + f.count[3]));
                }
                if (lane == 0) lead->mass[step] = mass, lead->steps[step] = n;
            }
        }
        sync_all<C>();

        // ---- what is kept, what is drawn ----
        if (rank == 0 && warp == 0) {
            uint32_t kept = 1, share = 1, key = best, at_n = 0, place = 0;
            uint64_t weight = uint64_t(1) << kOneBits, unit = weight;
            if (q.T == 0.0f) {
                at_n = best == 0 ? all.zeros : 0;
                if (best != 0)
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const uint32_t w = *of_rank<C>(&sm.count[(best & 0x7fffu) - kBase], c);
                        at_n += best & 0x8000u ? w >> 16 : w & 0xffffu;
                    }
            } else {
                if (lane == 0) {
                    sm.steps[kZeroStep] = all.zeros;
                    sm.mass[kZeroStep] = all.zeros ? all.zeros * weight_of(scale, 0.0f, sm.tables) : 0;
                }
                __syncwarp();
                Chunk c{0, 0, 0, 0};
#pragma unroll
                for (int x = 0; x < kChunk; ++x) c.own_w += sm.mass[lane * kChunk + x], c.own_n += sm.steps[lane * kChunk + x];
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
                if (q.min_p > 0.0f) most = count_from<C>(sm, floor_of(scale.top, sm.factors.reach));
                if (q.top_k > 0) most = min(most, static_cast<uint32_t>(q.top_k));
                kept = total, share = 0;
                if (most < total) {
                    const Found f = find<C>(sm, c, scale, false, most - 1);
                    key = f.bits, at_n = f.at_n, share = most - f.before_n, kept = most;
                    weight = f.before_w + share * weight_of(scale, value_of(key), sm.tables);
                }
                if (q.top_p < 1.0f) {
                    // tokens while what comes before them weighs less than this
                    const uint64_t need = times_up(q.top_p, weight);
                    const Found f = find<C>(sm, c, scale, true, need - 1);
                    const uint64_t w = weight_of(scale, value_of(f.bits), sm.tables);
                    key = f.bits, at_n = f.at_n, share = static_cast<uint32_t>((need - 1 - f.before_w) / w) + 1;
                    kept = f.before_n + share;
                    weight = f.before_w + share * w;
                }
                if (DRAW) {
                    const uint64_t aim = times_down(q.u, weight);
                    const Found f = find<C>(sm, c, scale, true, aim);
                    key = f.bits, at_n = f.at_n;
                    unit = weight_of(scale, value_of(key), sm.tables);
                    place = static_cast<uint32_t>((aim - f.before_w) / unit);
                }
            }
            if (lane < C) {
                Smem* to = of_rank<C>(&sm, lane);
                to->kept = kept, to->key = key, to->share = share, to->at_n = at_n, to->rank = place;
            }
            if (lane == 0) {
                if (a.kept) a.kept[r] = static_cast<int32_t>(kept);
                if (DRAW && a.logprob) a.logprob[r] = log_share(unit, weight);
            }
        }
        sync_all<C>();
        // the histogram is done with
        for (int x = tid; x < kWords / 4; x += kThreads) reinterpret_cast<uint4*>(sm.count)[x] = make_uint4(0, 0, 0, 0);

        // ---- the tokens of one value, by index ----
        const uint32_t key = sm.key, at_n = sm.at_n, place = DRAW ? sm.rank : sm.share;
        const bool uncut = !DRAW && sm.kept == total;                // nothing goes
        const uint32_t sign = (key & 0x7fffu) == 0 ? 0x80008000u : 0u, pair = (key & ~sign & 0xffffu) * 0x10001u;
        const uint32_t other = ~pair << 16;                          // beside a logit alone: not that value
        const bool some_stay = !DRAW && place < at_n && !uncut;      // of the last value, the first `place` stay
        const bool by_list = (DRAW || some_stay) && at_n <= kListed, by_index = (DRAW || some_stay) && !by_list;
        auto put = [&](uint32_t token) { lead->list[atomicAdd(&lead->listed, 1u)] = token; };
        if (DRAW && by_list) {
            for (int v0 = me; v0 < vectors; v0 += kAll) {
                const uint4 v = ld_row(row + static_cast<int64_t>(v0) * 16);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const uint32_t m = halves_of(w[y], pair, sign);
                    if (m & 1) put(v0 * 8 + 2 * y);
                    if (m & 2) put(v0 * 8 + 2 * y + 1);
                }
                if (C == 1 && *reinterpret_cast<volatile uint32_t*>(&sm.listed) >= at_n) break;      // that was all of them
            }
            for (int y = vectors * 8 + me; y < a.V; y += kAll)
                if (halves_of(cells[y] | other, pair, sign) & 1) put(y);
        }
        uint32_t last = 0;                                           // index of the token of that place (a truncation: the first that goes)
        if (by_index) {
            // by runs of the row, a warp to each: counted, then the one that holds it
            constexpr int kRuns = C * kWarps;
            const int run = (a.V + kRuns - 1) / kRuns, mine = rank * kWarps + warp, y0 = min(mine * run, a.V), y1 = min(y0 + run, a.V);
            auto is = [&](int y) { return y < y1 && (halves_of(cells[y] | other, pair, sign) & 1); };
            uint32_t n = 0;
            for (int y = y0 + lane; y < y1; y += 32) n += is(y);
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane < C) of_rank<C>(&sm, lane)->word[mine] = n;
            sync_all<C>();
            uint32_t before = 0;
            for (int x = lane; x < mine; x += 32) before += sm.word[x];
            before = __reduce_add_sync(0xffffffffu, before);
            if (before <= place && place < before + n) {
                for (int y = y0; y < y1; y += 32) {
                    const uint32_t m = __ballot_sync(0xffffffffu, is(y + lane)), here = __popc(m);
                    if (place < before + here) {
                        if ((m >> lane & 1) && before + __popc(m & ((1u << lane) - 1u)) == place)
                            for (int c = 0; c < C; ++c) of_rank<C>(&sm, c)->found = y + lane;
                        break;
                    }
                    before += here;
                }
            }
            sync_all<C>();
            last = sm.found;
            if (DRAW && me == 0) a.tokens[r] = static_cast<int32_t>(last);
        }
        if constexpr (!DRAW) {
            // kept: above the last value, and of that one the first (by index) that stay
            const float least = uncut ? -INFINITY : value_of(key);
            const __nv_bfloat162 bound = __floats2bfloat162_rn(least, least);
            auto cut = [&](uint32_t w, uint32_t index) {             // two logits, the first of this index
                const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w);
                uint32_t stay = by_list ? __hgt2_mask(x, bound) : __hge2_mask(x, bound);
                if (some_stay) {
                    const uint32_t m = halves_of(w, pair, sign);
                    if (m & 1) {
                        if (by_index) stay = index < last ? stay : stay & 0xffff0000u;
                        else put(index | (w & 0x8000u) << 16);
                    }
                    if (m & 2) {
                        if (by_index) stay = index + 1 < last ? stay : stay & 0x0000ffffu;
                        else put((index + 1) | (w & 0x80000000u));
                    }
                }
                return (w & stay) | (~stay & 0xff80ff80u);
            };
            if (out_vec)
                for (int v0 = me; v0 < vectors; v0 += kAll) {
                    const uint4 v = ld_row(row + static_cast<int64_t>(v0) * 16);
                    *reinterpret_cast<uint4*>(out + static_cast<int64_t>(v0) * 16) =
                        make_uint4(cut(v.x, v0 * 8), cut(v.y, v0 * 8 + 2), cut(v.z, v0 * 8 + 4), cut(v.w, v0 * 8 + 6));
                }
            for (int y = (out_vec ? vectors * 8 : 0) + me; y < a.V; y += kAll)
                reinterpret_cast<unsigned short*>(out)[y] = static_cast<unsigned short>(cut(cells[y] | other, y));
        }
        if (by_list) {
            sync_all<C>();
            if (rank == 0) {
                if (tid < static_cast<int>(at_n)) {
                    const uint32_t mine = sm.list[tid], index = mine & 0x7fffffffu;
                    uint32_t before = 0;
                    for (uint32_t x = 0; x < at_n; ++x) before += (sm.list[x] & 0x7fffffffu) < index;
                    if (DRAW) {
                        if (before == place) a.tokens[r] = static_cast<int32_t>(mine);
                    } else if (before < place) {                     // one that stays goes back, with its sign if it is a zero
                        reinterpret_cast<unsigned short*>(out)[index] = static_cast<unsigned short>(key | (mine >> 31) << 15);
                    }
                }
                __syncthreads();
                if (tid == 0) sm.listed = 0;
            }
        }
    }
    sync_all<C>();                                   // no CTA goes while another may still write to it
}

template <bool DRAW, int C> cudaError_t launch_one(const RowsArgs& a, int slots, cudaStream_t s) {
    const void* f = reinterpret_cast<const void*>(rows_bf16_kernel<DRAW, C>);
    const cudaError_t e = raise_smem_limit(f, sizeof(Smem));
    if (e != cudaSuccess) return e;
    const int64_t rows = a.rows < slots / C ? a.rows : slots / C;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, rows_bf16_kernel<DRAW, C>, a);
}

template <bool DRAW> cudaError_t launch(const RowsArgs& a, int nsm, cudaStream_t s) {
    // a row to a cluster, of as many CTAs as the machine has places for
    const int slots = 2 * nsm;
    if (a.rows * 8 <= slots) return launch_one<DRAW, 8>(a, slots, s);
    if (a.rows * 4 <= slots) return launch_one<DRAW, 4>(a, slots, s);
    if (a.rows * 2 <= slots) return launch_one<DRAW, 2>(a, slots, s);
    return launch_one<DRAW, 1>(a, slots, s);
}

}  // namespace

cudaError_t launch_rows_bf16(const RowsArgs& a, bool draw, int nsm, cudaStream_t s) {
    return draw ? launch<true>(a, nsm, s) : launch<false>(a, nsm, s);
}

}  // namespace sdv
