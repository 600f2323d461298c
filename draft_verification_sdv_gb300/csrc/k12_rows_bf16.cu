// k12_rows_bf16.cu -- draws from rows of logits and their truncation (sdv_sample,
// sdv_logits_truncate): rows in bf16.
//
// A bf16 logit is one of few values, so a row is counted once into a histogram of
// all of them, and everything that is asked for follows from the counts: the sum
// of count times weight over the few thousand values that occur, the last value
// that top-k, min-p and top-p keep, the one that a draw meets.  Only which token of
// that value it is takes a second look at the row, which is in L2 by then.
//
// The histogram has a word for each value whose magnitude lies from 2^-39 to 2^23,
// 62 octaves of 128 of either sign (64 KB: two CTAs share an SM, and one counts
// while the other looks for its places).  Smaller and larger magnitudes go to a word
// at either end; a row where the sum of the counts shows such logits is looked
// through once more for zeros and infinities, and one that holds other ones goes the
// long way (row_in_passes).
//
// Where top-k (up to 256), min-p or temperature 0 limits a row, what it keeps is
// nearly always among a few hundred logits.  A sample gives a bound that so many
// reach; one look at the row writes down the vectors that hold such a one, the head,
// and only its logits are counted.  If it turns out not to hold all that is asked for,
// the row is counted as a whole.  A truncation whose last value lies in the head
// fills the row with -infinity and writes the head's vectors over it, so that the
// row is read once.
//
// Few rows are shared by a cluster of C CTAs, each of which counts a C-th of the
// row; octave o is looked after by CTA o % C, which adds up the C counts.  A warp
// takes an octave at a time and sums its counts and weights; warp 0 of the first CTA
// adds up the 125 sums (octaves of either sign, zeros between them) in the order
// of the logits and finds places in them, octave first.
//
// What bounds it.  Counting a whole row: the banks that 32 lanes' words lie in (3.5 of
// them in one; 17 000 clocks for 152064 logits, of 20 000 to 25 000 that it takes).  A
// head: the reads (36 000 clocks where two rows share an SM; 24 000 at HBM's rate),
// then a chain of steps of one CTA and of one warp, some 16 000 clocks (octaves 3500,
// weights 3900, places 8400).  256 rows of 152064 under top-k, top-p and min-p: 42 us,
// 1.9 TB/s (518 when each place was looked for in passes, 65 with a histogram that
// took a whole SM, 58 before heads); 1088 rows truncated: 207 us, 3.9 TB/s with what
// rows without top-k read twice (1693, 320 and 213); one row, eight CTAs: 22 us.
// Reading the next row into L2 ahead of time makes it slower (229 us): rows in
// flight push one another out.
#include <cuda_bf16.h>

#include "k12_rows.cuh"

namespace sdv {
namespace {

using namespace rows;

constexpr int kThreads = 512, kCtas = 1024 / kThreads, kWarps = kThreads / 32, kPassBins = 1024;
constexpr int kOctaves = 62, kFirstOctave = 127 - 39, kBase = kFirstOctave * 128, kAbove = kBase + kOctaves * 128;
// words: a magnitude m stands at m - kBase + 128, smaller ones at 127, larger ones at kLarge; negative ones kHalf further
constexpr int kHalf = 8192, kSmall = 127, kLarge = 128 + kOctaves * 128, kWords = 2 * kHalf;
static_assert(kLarge < kHalf, "a sign's words and the two at their ends");
constexpr int kZeroStep = kOctaves, kSteps = 2 * kOctaves + 1;   // step s < 62: positive octave 61 - s; s > 62: negative octave s - 63
constexpr int kChunk = 4, kPadded = 32 * kChunk;                 // steps of a lane of warp 0
static_assert(kPadded >= kSteps, "a lane holds four steps");
constexpr int kListed = 256;             // tokens of one value that are kept in a list
constexpr int kHeads = 2048;             // vectors that hold a logit of the head
constexpr int kHeadK = 256;              // top-k up to which a row is first looked through for its head alone (which
                                         // has some 400 logits or more; where it fails, the row is read twice)

// What a CTA says of its part of a row and of its octaves.
struct Note {
    uint32_t total, high;                // logits in the octaves, the largest
    uint32_t head, heads, odd, beyond;   // the head's bound (a key), its vectors; kOdd* bits; counts beyond the octaves
};
struct Rest {
    uint32_t zeros, odd;
};
enum : uint32_t { kOddNan = 1u, kOddFar = 2u };

struct Smem {
    uint32_t count[kWords];              // or a PassSmem
    uint64_t mass[kPadded];
    uint32_t steps[kPadded];             // counts
    Tables tables;
    Factors factors;
    Note note[8];                        // of each CTA of the cluster
    Rest rest[8];
    uint32_t word[8 * kWarps];
    // what warp 0 has found
    uint32_t kept, key, share, at_n, rank;       // key: bits of a bf16
    uint32_t listed, found, heads, odd;
    uint32_t list[kListed], head[kHeads];
};
static_assert(sizeof(PassSmem<kThreads, kPassBins>) <= sizeof(uint32_t) * kWords, "the long way uses the histogram's place");
static_assert(kCtas * (sizeof(Smem) + 1024) <= 227 * 1024, "two CTAs per SM");

// (Functions that are called find it for themselves: the compiler then knows that it
// is shared memory.)
__device__ __forceinline__ Smem& smem() {
    extern __shared__ __align__(16) unsigned char raw[];
    return *reinterpret_cast<Smem*>(raw);
}

__device__ __forceinline__ float value_of(uint32_t bits) { return __uint_as_float(bits << 16); }

// Counts a word's two logits.  Both halves at once: the magnitude, kept within the
// octaves and the words at their ends, as a byte offset; the sign on top of it.
// (Lanes that hit one word cost one pass: masked rows are no slower.)
__device__ __forceinline__ void count_two(uint32_t counts, uint32_t w) {
    constexpr uint32_t kTwo = 0x00010001u;
    const uint32_t m = __vminu2(__vmaxu2(w & 0x7fff7fffu, (kBase - 1) * kTwo), static_cast<uint32_t>(kAbove) * kTwo);
    const uint32_t p = (m * 4 - (kBase - 128) * 4 * kTwo) | (w & 0x80008000u);
    asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(counts + (p & 0xffffu)) : "memory");
    asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(counts + (p >> 16)) : "memory");
}
__device__ __forceinline__ void count_one(uint32_t* h, uint32_t bits) {
    const uint32_t m = min(max(bits & 0x7fffu, static_cast<uint32_t>(kBase - 1)), static_cast<uint32_t>(kAbove));
    atomicAdd(h + (m - (kBase - 128) + (bits & 0x8000u ? kHalf : 0)), 1u);
}
__device__ __forceinline__ void look_at(Rest& rest, uint32_t bits) {
    const uint32_t m = bits & 0x7fffu;
    if (m - kBase < static_cast<uint32_t>(kAbove - kBase)) return;
    const bool zero = m == 0, inf = bits == 0xff80u;
    rest.zeros += zero;
    rest.odd |= zero || inf ? 0u : m >= 0x7f80u ? kOddNan : kOddFar;
}

// Key of the largest of eight logits (0: none above -infinity).
__device__ __forceinline__ uint32_t largest_of(const uint4& v) {
    const uint32_t m = bf16x2_max(bf16x2_max(v.x, v.y), bf16x2_max(v.z, v.w));
    const float f = fmaxf(bf16_lo(m), bf16_hi(m));
    return f > -INFINITY ? key_of(f) : 0u;
}
__device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ void count_above(uint32_t* h, uint32_t w, float least) {
    if (bf16_lo(w) >= least) count_one(h, w & 0xffffu);
    if (bf16_hi(w) >= least) count_one(h, w >> 16);
}
// Whether one of them is at least `above`.
__device__ __forceinline__ bool at_least(const uint4& v, __nv_bfloat162 above) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int y = 0; y < 4; ++y) m |= __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[y]), above);
    return m != 0;
}

__device__ __forceinline__ uint64_t warp_sum64(uint64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Four values of a step (not the zeros'), in the order of the logits, that a lane looks after.
struct Four {
    uint32_t bits[4], count[4];
    uint64_t weight[4];                  // of one
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
        const uint4 v = *reinterpret_cast<const uint4*>(of_rank<C>(h + (neg ? kHalf : 0) + 128 + first, c));
        f.count[0] += neg ? v.x : v.w, f.count[1] += neg ? v.y : v.z;
        f.count[2] += neg ? v.z : v.y, f.count[3] += neg ? v.w : v.x;
    }
    return f;
}
__device__ __forceinline__ void weigh(Four& f, const Scale& scale, const Tables& t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f.weight[i] = weight_of(scale, value_of(f.bits[i]), t);
}

// A lane's steps: what comes before them, and what they hold.
struct Chunk {
    uint64_t before_w, own_w;
    uint32_t before_n, own_n;
};

struct Found {
    uint32_t bits, at_n, before_n;
    uint64_t before_w, weight;           // weight: of one of them
};

// The step that was looked into last.
struct Look {
    int step;
    Four f;
    uint32_t n;                          // counts and weights of the lanes before, within it
    uint64_t w;
};

// The value where the running count (weight) of the order passes `target`.  Warp 0.
template <int C>
__device__ __forceinline__ Found find(const Smem& sm, const Chunk& c, Look& look, const Scale& scale, bool by_weight, uint64_t target) {
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
    if (step == kZeroStep) return Found{0, sm.steps[step], bn, bw, weight_of(scale, 0.0f, sm.tables)};
    if (look.step != step) {
        look.step = step;
        look.f = four_of<C>(sm.count, step, lane);
        weigh(look.f, scale, sm.tables);
        uint64_t own_w = 0;
        uint32_t own_n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) own_w += look.f.count[i] * look.f.weight[i], own_n += look.f.count[i];
        look.w = own_w, look.n = own_n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t x = __shfl_up_sync(0xffffffffu, look.w, o);
            const uint32_t y = __shfl_up_sync(0xffffffffu, look.n, o);
            if (lane >= o) look.w += x, look.n += y;
        }
        look.w -= own_w, look.n -= own_n;
    }
    bw += look.w;                                    // before this lane's four
    bn += look.n;
    // the lane and the value where it is passed: the first past the target
    Found r{0, 0, 0, 0, 0};
    bool passed = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (!passed) r = Found{look.f.bits[i], look.f.count[i], bn, bw, look.f.weight[i]};
        bw += look.f.count[i] * look.f.weight[i], bn += look.f.count[i];
        passed = passed || target < (by_weight ? bw : static_cast<uint64_t>(bn));
    }
    const int who = __ffs(__ballot_sync(0xffffffffu, passed) | 0x80000000u) - 1;
    r.bits = __shfl_sync(0xffffffffu, r.bits, who);
    r.at_n = __shfl_sync(0xffffffffu, r.at_n, who);
    r.before_n = __shfl_sync(0xffffffffu, r.before_n, who);
    r.before_w = __shfl_sync(0xffffffffu, r.before_w, who);
    r.weight = __shfl_sync(0xffffffffu, r.weight, who);
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

// Counts and weights of this CTA's octaves, a warp to each: some[x] tells which of the
// positive (negative) ones are not empty.
template <int C> constexpr int kMine = (kOctaves + C * kWarps - 1) / (C * kWarps);
template <int C> __device__ __noinline__ void weigh_octaves(const Scale scale, uint32_t positive, uint32_t negative, int rank) {
    Smem& sm = smem();
    Smem* const lead = of_rank<C>(&sm, 0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 1
    for (int x = 0; x < 2 * kMine<C>; ++x) {
        const int o = ((x >> 1) * kWarps + warp) * C + rank, step = x & 1 ? kZeroStep + 1 + o : kOctaves - 1 - o;
        if (o >= kOctaves) break;
        uint64_t mass = 0;
        uint32_t n = 0;
        if ((x & 1 ? negative : positive) >> (x >> 1) & 1) {
            Four f = four_of<C>(sm.count, step, lane);
            weigh(f, scale, sm.tables);
            mass = warp_sum64((f.count[0] * f.weight[0] + f.count[1] * f.weight[1]) + (f.count[2] * f.weight[2] + f.count[3] * f.weight[3]));
            n = __reduce_add_sync(0xffffffffu, (f.count[0] + f.count[1]) + (f.count[2] + f.count[3]));
        }
        if (lane == 0) lead->mass[step] = mass, lead->steps[step] = n;
    }
}

// What a row keeps and what is drawn (total: logits counted, finite: of how many): told to every CTA of the cluster.  Warp 0 of the first.
template <bool DRAW, int C>
__device__ __noinline__ void settle(const RowsArgs& a, int r, const Ask q, const Scale scale, uint32_t best, uint32_t total, uint32_t finite, uint32_t zeros) {
    Smem& sm = smem();
    const int lane = threadIdx.x & 31;
    uint32_t kept = 1, share = 1, key = best, at_n = 0, place = 0;
    uint64_t weight = uint64_t(1) << kOneBits, unit = weight;
    if (q.T == 0.0f) {
        at_n = best == 0 ? zeros : 0;
        if (best != 0)
#pragma unroll
            for (int c = 0; c < C; ++c)
                at_n += *of_rank<C>(&sm.count[(best & 0x7fffu) - kBase + 128 + (best & 0x8000u ? kHalf : 0)], c);
    } else {
        if (lane == 0) {
            sm.steps[kZeroStep] = zeros;
            sm.mass[kZeroStep] = zeros ? zeros * weight_of(scale, 0.0f, sm.tables) : 0;
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
        Look look;
        look.step = -1;
        uint32_t most = total;
        if (q.min_p > 0.0f) most = count_from<C>(sm, floor_of(scale.top, sm.factors.reach));
        if (q.top_k > 0) most = min(most, static_cast<uint32_t>(q.top_k));
        kept = total, share = 0;
        // the last of the first `most`; the last before which less than top_p of their
        // weight lies; the one that is drawn
#pragma unroll 1
        for (int ask = 0; ask < 3; ++ask) {
            if (ask == 0 ? most >= finite : ask == 1 ? !(q.top_p < 1.0f) : !DRAW) continue;
            const uint64_t target = ask == 0 ? most - 1 : ask == 1 ? times_up(q.top_p, weight) - 1 : times_down(q.u, weight);
            const Found f = find<C>(sm, c, look, scale, ask != 0, target);
            key = f.bits, at_n = f.at_n;
            const uint32_t nth = ask == 0 ? most - 1 - f.before_n : quotient(target - f.before_w, f.weight);
            if (ask < 2) {
                share = nth + 1;
                kept = f.before_n + share;
                weight = f.before_w + share * f.weight;
            } else {
                place = nth;
                unit = f.weight;
            }
        }
    }
    if (lane < C) {
        Smem* to = of_rank<C>(&sm, lane);
        to->kept = kept, to->key = key, to->share = share, to->at_n = at_n, to->rank = place;
    }
    if (lane == 0) {
        if (a.kept) a.kept[r] = static_cast<int32_t>(kept);
        if (DRAW && a.logprob) a.logprob[r] = log_share(scale, value_of(key), unit, weight, sm.tables);
    }
}

// Counts this CTA's vectors of a row.  A sample, 32 vectors here and there, gives a bound
// that some hundred logits of the row reach; vectors with such a one, the head, are
// written down; without COUNT only those are counted.  Returns the bound, a key.  (A function of its own, as the other steps
// are: a row's other numbers would take the registers of its loads.)
template <int C, bool COUNT> __device__ __noinline__ uint32_t count_row(const unsigned char* cells, int V, const Span span, int rank) {
    const unsigned char* row = cells + span.head * 2;            // the first vector
    const int vectors = span.vectors;
    constexpr int U = 4, kAll = C * kThreads, kSamples = C * kWarps * 2;
    Smem& sm = smem();
    const uint32_t counts = smem_u32(sm.count);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t policy = first_policy();
    const int chunks = (vectors + 31) / 32;
    uint32_t least = 0xffffffffu, most = 0;
    {
        uint4 v[2];
        bool there[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int n = (rank * kWarps + warp) * 2 + u;
            const int at = (chunks >= kSamples ? static_cast<int>(static_cast<uint32_t>(n) * chunks / kSamples) : n) * 32 + lane;
            there[u] = at < vectors;
            if (there[u]) v[u] = ld_hint(row + static_cast<int64_t>(at) * 16, policy);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, there[u] ? largest_of(v[u]) : 0u);
            if (top) least = min(least, top);
            most = max(most, top);
        }
    }
    if (lane < C) of_rank<C>(&sm, lane)->word[rank * kWarps + warp] = V < kManyLogits || most == 0 ? least : most;
    int i = rank * kThreads + threadIdx.x;
    uint4 v[U];
    const bool full = i + (U - 1) * kAll < vectors;
    if (full)                                        // (on their way while the bound is agreed upon)
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = ld_hint(row + static_cast<int64_t>(i + u * kAll) * 16, policy);
    sync_all<C>();
    uint32_t bound = kKeyLow + 1;                    // (a short row is head as a whole)
    if (vectors > kHeads) bound = min(fourth_smallest<C * kWarps>(sm.word), kKeyHigh);
    const float f = of_key(bound);
    const __nv_bfloat162 above = __floats2bfloat162_rn(f, f);
    uint32_t most2 = 0xff80ff80u;                    // of both halves; a NaN stays
    auto take = [&](const uint4& x, int index) {
        if constexpr (COUNT)
            count_two(counts, x.x), count_two(counts, x.y), count_two(counts, x.z), count_two(counts, x.w);
        else
            most2 = max_nan(most2, max_nan(max_nan(x.x, x.y), max_nan(x.z, x.w)));
        if (at_least(x, above)) {
            const uint32_t n = atomicAdd(&sm.heads, 1u);
            if (n < kHeads) sm.head[n] = index;
        }
    };
    if (full) {
        for (;;) {
#pragma unroll
            for (int u = 0; u < U; ++u) take(v[u], i + u * kAll);
            i += U * kAll;
            if (i + (U - 1) * kAll >= vectors) break;
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = ld_hint(row + static_cast<int64_t>(i + u * kAll) * 16, policy);
        }
    }
    for (; i < vectors; i += kAll) take(ld_hint(row + static_cast<int64_t>(i) * 16, policy), i);
    if constexpr (!COUNT) {
        const bool odd = !(fmaxf(bf16_lo(most2), bf16_hi(most2)) < INFINITY) || bf16_lo(most2) != bf16_lo(most2) || bf16_hi(most2) != bf16_hi(most2);
        if (odd) atomicOr(&sm.odd, kOddNan);
        // of the vectors written down, what reaches the bound is counted
        __syncthreads();
        if (sm.heads <= kHeads)
            for (uint32_t x = threadIdx.x; x < sm.heads; x += kThreads) {
                const uint4 w = ld_hint(row + static_cast<int64_t>(sm.head[x]) * 16, policy);
                count_above(sm.count, w.x, f), count_above(sm.count, w.y, f), count_above(sm.count, w.z, f), count_above(sm.count, w.w, f);
            }
        if (rank * kThreads + static_cast<int>(threadIdx.x) < span.loose) {
            const uint32_t x = reinterpret_cast<const unsigned short*>(cells)[span.loose_at(rank * kThreads + threadIdx.x)];
            if (value_of(x) >= f) count_one(sm.count, x);
            if (!(value_of(x) < INFINITY)) atomicOr(&sm.odd, kOddNan);
        }
    }
    return bound;
}

// The index of the token of one value that stands at `place` among them, into sm.found of
// every CTA of the cluster.
template <int C>
__device__ __noinline__ void find_by_index(const unsigned short* cells, int V, const Span span, int rank, uint32_t pair, uint32_t sign, uint32_t place) {
    constexpr int U = 4;
    Smem& sm = smem();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t other = ~pair << 16;
    // by runs of the row, a warp to each: counted, then the one that holds it
    constexpr int kRuns = C * kWarps;
    // eights of the row: whole vectors, but for the first (where a vector does not begin the
    // row) and the last
    const int shift = (8 - span.head) & 7;
    auto eight_at = [&](int e) { return e * 8 - shift; };
    auto is_vector = [&](int e) { const int v = e - (shift ? 1 : 0); return v >= 0 && v < span.vectors; };
    const int steps = (V + shift + 255) / 256, run = (steps + kRuns - 1) / kRuns, mine = rank * kWarps + warp;
    const int s0 = min(mine * run, steps), s1 = min(s0 + run, steps);
    auto load = [&](int s, uint4 (&v)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (is_vector((s + u) * 32 + lane)) v[u] = ld_row(reinterpret_cast<const unsigned char*>(cells + eight_at((s + u) * 32 + lane)));
    };
    auto matches = [&](int s, const uint4& v) {          // among the lane's eight logits of step s, as bits
        const int at = eight_at(s * 32 + lane);
        if (s >= s1 || at >= V) return 0u;
        if (is_vector(s * 32 + lane))
            return halves_of(v.x, pair, sign) | halves_of(v.y, pair, sign) << 2 | halves_of(v.z, pair, sign) << 4 | halves_of(v.w, pair, sign) << 6;
        uint32_t m = 0;
        for (int y = 0; y < 8; ++y)
            if (at + y >= 0 && at + y < V) m |= (halves_of(cells[at + y] | other, pair, sign) & 1u) << y;
        return m;
    };
    uint32_t n = 0;
    for (int s = s0; s < s1; s += U) {
        uint4 v[U];
        load(s, v);
#pragma unroll
        for (int u = 0; u < U; ++u) n += __popc(matches(s + u, v[u]));
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane < C) of_rank<C>(&sm, lane)->word[mine] = n;
    sync_all<C>();
    uint32_t before = 0;
    for (int x = lane; x < mine; x += 32) before += sm.word[x];
    before = __reduce_add_sync(0xffffffffu, before);
    if (before <= place && place < before + n) {
        bool done = false;
        for (int s = s0; s < s1 && !done; s += U) {
            uint4 v[U];
            load(s, v);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t m = matches(s + u, v[u]), own = __popc(m), here = __reduce_add_sync(0xffffffffu, own);
                if (!done && place < before + here) {
                    done = true;
                    uint32_t upto = own;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
                        if (lane >= o) upto += x;
                    }
                    const uint32_t first = before + upto - own;
                    if (first <= place && place < first + own)
                        for (int c = 0; c < C; ++c)
                            of_rank<C>(&sm, c)->found = eight_at((s + u) * 32 + lane) + __fns(m, 0, static_cast<int>(place - first) + 1);
                }
                before += here;
            }
        }
    }
    sync_all<C>();
}

template <bool DRAW, int C> __global__ void __launch_bounds__(kThreads, kCtas) rows_bf16_kernel(const RowsArgs a) {
    Smem& sm = smem();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int me = rank * kThreads + tid;            // among the cluster's threads
    constexpr int kAll = C * kThreads;
    const float nan = __int_as_float(0x7fc00000);
    Smem* const lead = of_rank<C>(&sm, 0);
    const uint64_t drop = drop_policy();
    load_tables(sm.tables, tid, kThreads);
    for (int i = tid; i < kWords / 4; i += kThreads) reinterpret_cast<uint4*>(sm.count)[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < kPadded; i += kThreads) sm.mass[i] = 0, sm.steps[i] = 0;
    if (tid == 0) sm.listed = sm.heads = sm.odd = 0;
    for (int64_t r = blockIdx.x / C; r < a.rows; r += gridDim.x / C) {
        const Ask q = ask_of(a, r);
        const unsigned char* row = static_cast<const unsigned char*>(a.logits) + r * a.in_stride;
        unsigned char* out = static_cast<unsigned char*>(a.out) + r * a.out_stride;
        const Span span = span_of(row, a.V, 2);
        const int vectors = span.vectors;
        const unsigned char* first = row + span.head * 2;        // vector
        unsigned char* out_first = out + span.head * 2;
        const bool out_vec = (reinterpret_cast<uintptr_t>(out_first) & 15) == 0;
        const unsigned short* cells = reinterpret_cast<const unsigned short*>(row);
        sync_all<C>();                               // (the row before is done with shared memory)
        if (tid == kThreads - 1) sm.factors = factors_of(q.T, q.min_p);

        // ---- every logit is counted ----
        constexpr int U = 4;
        // Where few tokens are asked for, they are in the head as a rule: the first look is for
        // that alone, at HBM's rate, and a second one counts all where it does not do.
        const bool brief = vectors > 0 && (q.T == 0.0f || (q.top_k > 0 && q.top_k <= kHeadK) || q.min_p >= 0x1p-10f);
        uint32_t some[2] = {0, 0}, total = 0;
        Note all;
        bool whole = !brief;                         // all logits are counted
#pragma unroll 1
        for (;; whole = true) {
            uint32_t bound = kKeyHigh;
            if (vectors > 0) bound = whole ? count_row<C, true>(row, a.V, span, rank) : count_row<C, false>(row, a.V, span, rank);
            if (whole && me < span.loose) count_one(sm.count, cells[span.loose_at(me)]);
            sync_all<C>();

            // ---- which octaves hold something, how much in all, the largest ----
            // (octaves of this CTA, a warp to each, a lane to four magnitudes)
            some[0] = some[1] = 0;
            total = 0;
            uint32_t high = 0;                       // high: 0x8000 and how far the largest lies above zero
#pragma unroll
            for (int x = 0; x < 2 * kMine<C>; ++x) {
                const int o = ((x >> 1) * kWarps + warp) * C + rank;
                if (o >= kOctaves) break;
                uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const uint4 v = reinterpret_cast<const uint4*>(of_rank<C>(sm.count, c))[((x & 1) * kHalf + 128) / 4 + o * 32 + lane];
                    w[0] += v.x, w[1] += v.y, w[2] += v.z, w[3] += v.w;
                }
                const uint32_t n = (w[0] + w[1]) + (w[2] + w[3]);
                total += n;
                if (!__any_sync(0xffffffffu, n != 0)) continue;
                some[x & 1] |= 1u << (x >> 1);
                const uint32_t at = kBase + o * 128 + lane * 4;
                if (n) high = max(high, x & 1 ? 0x8000u - (at + (w[0] ? 0 : w[1] ? 1 : w[2] ? 2 : 3)) : 0x8000u + at + (w[3] ? 3 : w[2] ? 2 : w[1] ? 1 : 0));
            }
            high = __reduce_max_sync(0xffffffffu, high);
            total = __reduce_add_sync(0xffffffffu, total);
            if (lane == 0) sm.word[warp] = high, sm.word[kWarps + warp] = total;
            __syncthreads();
            if (warp == 0) {
                Note n;
                n.high = __reduce_max_sync(0xffffffffu, sm.word[lane % kWarps]);
                n.total = __reduce_add_sync(0xffffffffu, lane < kWarps ? sm.word[kWarps + lane] : 0u);
                n.head = bound, n.heads = sm.heads, n.odd = sm.odd;
                n.beyond = sm.count[kSmall] + sm.count[kLarge] + sm.count[kHalf + kSmall] + sm.count[kHalf + kLarge];
                if (lane < C) *of_rank<C>(&sm.note[rank], lane) = n;
            }
            sync_all<C>();
            all = sm.note[0];
#pragma unroll
            for (int c = 1; c < C; ++c) {
                const Note n = sm.note[c];
                all.total += n.total, all.high = max(all.high, n.high);
                all.head = max(all.head, n.head), all.heads = max(all.heads, n.heads);
                all.odd |= n.odd, all.beyond += n.beyond;
            }
            if (whole || q.bad) break;
            // does the head hold all that is asked for?
            const float top = value_of(all.high >= 0x8000u ? all.high - 0x8000u : 0x8000u | (0x8000u - all.high));
            const float back = q.min_p > 0.0f ? q.T * logf(q.min_p) : -INFINITY;                 // min-p reaches to top + back
            const bool first = q.T == 0.0f || (q.top_k > 0 && static_cast<uint32_t>(q.top_k) <= all.total);
            const bool near = top + back - 1e-5f * (fabsf(top) + fabsf(back)) >= of_key(all.head);       // (with room for what it is off by)
            const bool enough = all.total > 0 && all.heads <= kHeads && all.beyond == 0 && (first || near);
            if (enough || (all.odd & kOddNan)) break;
            sync_all<C>();                           // (nobody reads another's counts any more)
            for (int x = tid; x < kWords / 4; x += kThreads) reinterpret_cast<uint4*>(sm.count)[x] = make_uint4(0, 0, 0, 0);
            if (tid == 0) sm.heads = 0;
            sync_all<C>();
        }
        Rest rest{0, 0};
        if (whole && all.total != static_cast<uint32_t>(a.V)) {  // some logits are not in the octaves: which
            for (int x = me; x < vectors; x += kAll) {
                const uint4 v = ld_row(first + static_cast<int64_t>(x) * 16);
                look_at(rest, v.x & 0xffffu), look_at(rest, v.x >> 16), look_at(rest, v.y & 0xffffu), look_at(rest, v.y >> 16);
                look_at(rest, v.z & 0xffffu), look_at(rest, v.z >> 16), look_at(rest, v.w & 0xffffu), look_at(rest, v.w >> 16);
            }
            if (me < span.loose) look_at(rest, cells[span.loose_at(me)]);
            rest.zeros = __reduce_add_sync(0xffffffffu, rest.zeros);
            rest.odd = __reduce_or_sync(0xffffffffu, rest.odd);
            if (lane == 0) sm.word[warp] = rest.zeros, sm.word[kWarps + warp] = rest.odd;
            __syncthreads();
            if (warp == 0) {
                rest.zeros = __reduce_add_sync(0xffffffffu, lane < kWarps ? sm.word[lane] : 0u);
                rest.odd = __reduce_or_sync(0xffffffffu, sm.word[kWarps + lane % kWarps]);
                if (lane < C) *of_rank<C>(&sm.rest[rank], lane) = rest;
            }
            sync_all<C>();
            rest = sm.rest[0];
#pragma unroll
            for (int c = 1; c < C; ++c) rest.zeros += sm.rest[c].zeros, rest.odd |= sm.rest[c].odd;
            if (rest.zeros) all.high = max(all.high, 0x8000u);
        }
        total = all.total + rest.zeros;              // finite logits
        const bool over = rest.odd & kOddFar;
        const bool bad = q.bad || ((rest.odd | all.odd) & kOddNan) || (!over && total == 0);
        if (bad || over) {
            sync_all<C>();                           // (nobody reads another's counts any more)
            if (!bad) {
                if (rank == 0) {
                    PassSmem<kThreads, kPassBins>& ps = *reinterpret_cast<PassSmem<kThreads, kPassBins>*>(sm.count);
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
                    for (int i0 = me * 8; i0 < a.V; i0 += kAll * 8) store_step<true>(out, i0, a.V, (reinterpret_cast<uintptr_t>(out) & 15) == 0, x);
                }
            }
            for (int x = tid; x < kWords / 4; x += kThreads) reinterpret_cast<uint4*>(sm.count)[x] = make_uint4(0, 0, 0, 0);
            if (tid == 0) sm.heads = sm.odd = 0;
            continue;
        }

        // ---- weights ----
        const uint32_t best = all.high >= 0x8000u ? all.high - 0x8000u : 0x8000u | (0x8000u - all.high);
        const Scale scale{value_of(best), sm.factors.hi, sm.factors.lo};
        if (q.T != 0.0f) {
            weigh_octaves<C>(scale, some[0], some[1], rank);
        }
        sync_all<C>();

        // ---- what is kept, what is drawn ----
        if (rank == 0 && warp == 0) {
            settle<DRAW, C>(a, static_cast<int>(r), q, scale, best, total, whole ? total : 0xffffffffu, rest.zeros);
        }
        sync_all<C>();
        // the histogram is done with
        for (int x = tid; x < kWords / 4; x += kThreads) reinterpret_cast<uint4*>(sm.count)[x] = make_uint4(0, 0, 0, 0);

        // ---- the tokens of one value, by index ----
        const uint32_t key = sm.key, at_n = sm.at_n, place = DRAW ? sm.rank : sm.share;
        const bool uncut = !DRAW && whole && sm.kept == total;       // nothing goes
        const uint32_t sign = (key & 0x7fffu) == 0 ? 0x80008000u : 0u, pair = (key & ~sign & 0xffffu) * 0x10001u;
        const uint32_t other = ~pair << 16;                          // beside a logit alone: not that value
        const bool some_stay = !DRAW && place < at_n && !uncut;      // of the last value, the first `place` stay
        const bool by_list = (DRAW || some_stay) && at_n <= kListed, by_index = (DRAW || some_stay) && !by_list;
        // the head holds every logit from the last value on
        const bool by_head = vectors > 0 && !uncut && !by_index && all.heads <= kHeads && key_of(value_of(key)) >= all.head;
        const uint32_t heads = min(sm.heads, static_cast<uint32_t>(kHeads));
        auto put = [&](uint32_t token) {                             // (once for each of the at_n)
            const uint32_t n = atomicAdd(&lead->listed, 1u);
            if (n < kListed) lead->list[n] = token;
        };
        if (DRAW && by_list) {
            auto look_for = [&](const uint4& v, int v0) {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const uint32_t m = halves_of(w[y], pair, sign);
                    if (m & 1) put(span.index_of(v0) + 2 * y);
                    if (m & 2) put(span.index_of(v0) + 2 * y + 1);
                }
            };
            if (by_head)
                for (uint32_t x = tid; x < heads; x += kThreads) look_for(ld_row(first + static_cast<int64_t>(sm.head[x]) * 16), sm.head[x]);
            int v0 = by_head ? vectors : me;
            for (; v0 + (U - 1) * kAll < vectors; v0 += U * kAll) {
                uint4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) v[u] = ld_row(first + static_cast<int64_t>(v0 + u * kAll) * 16);
#pragma unroll
                for (int u = 0; u < U; ++u) look_for(v[u], v0 + u * kAll);
                if (C == 1 && *reinterpret_cast<volatile uint32_t*>(&sm.listed) >= at_n) {           // that was all of them
                    v0 = vectors;
                    break;
                }
            }
            for (; v0 < vectors; v0 += kAll) look_for(ld_row(first + static_cast<int64_t>(v0) * 16), v0);
            if (me < span.loose && (halves_of(cells[span.loose_at(me)] | other, pair, sign) & 1)) put(span.loose_at(me));
        }
        uint32_t last = 0;                                           // index of the token of that place (a truncation: the first that goes)
        if (by_index) {
            find_by_index<C>(cells, a.V, span, rank, pair, sign, place);
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
            auto write = [&](const uint4& v, int v0) {
                st_hint(out_first + static_cast<int64_t>(v0) * 16,
                        make_uint4(cut(v.x, span.index_of(v0)), cut(v.y, span.index_of(v0) + 2), cut(v.z, span.index_of(v0) + 4), cut(v.w, span.index_of(v0) + 6)), drop);
            };
            if (by_head) {
                // the head is taken up, all becomes -infinity, and what the head keeps comes back
                constexpr int kOwn = kHeads / kThreads;
                uint4 v[kOwn];
#pragma unroll
                for (int x = 0; x < kOwn; ++x)
                    if (tid + x * kThreads < heads) v[x] = ld_row(first + static_cast<int64_t>(sm.head[tid + x * kThreads]) * 16);
                sync_all<C>();
                const uint4 none = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
                for (int v0 = me; v0 < vectors; v0 += kAll) {
                    if (out_vec)
                        st_hint(out_first + static_cast<int64_t>(v0) * 16, none, drop);
                    else
                        for (int y = 0; y < 8; ++y) reinterpret_cast<unsigned short*>(out_first)[v0 * 8 + y] = 0xff80u;
                }
                sync_all<C>();
#pragma unroll
                for (int x = 0; x < kOwn; ++x)
                    if (tid + x * kThreads < heads) {
                        const int at = static_cast<int>(sm.head[tid + x * kThreads]);
                        const uint32_t w[4] = {cut(v[x].x, span.index_of(at)), cut(v[x].y, span.index_of(at) + 2), cut(v[x].z, span.index_of(at) + 4), cut(v[x].w, span.index_of(at) + 6)};
                        if (out_vec)
                            *reinterpret_cast<uint4*>(out_first + static_cast<int64_t>(at) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                        else
#pragma unroll
                            for (int y = 0; y < 8; ++y)
                                reinterpret_cast<unsigned short*>(out_first)[at * 8 + y] = static_cast<unsigned short>(w[y / 2] >> (16 * (y % 2)));
                    }
            } else if (out_vec) {
                int v0 = me;
                for (; v0 + (U - 1) * kAll < vectors; v0 += U * kAll) {
                    uint4 v[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) v[u] = ld_hint(first + static_cast<int64_t>(v0 + u * kAll) * 16, drop);
#pragma unroll
                    for (int u = 0; u < U; ++u) write(v[u], v0 + u * kAll);
                }
                for (; v0 < vectors; v0 += kAll) write(ld_hint(first + static_cast<int64_t>(v0) * 16, drop), v0);
            }
            // the loose ones; and where the result lies otherwise than the row, all of them
            const int singles = out_vec || by_head ? span.loose : a.V;
            for (int l = me; l < singles; l += kAll) {
                const int y = singles == a.V ? l : span.loose_at(l);
                reinterpret_cast<unsigned short*>(out)[y] = static_cast<unsigned short>(cut(cells[y] | other, y));
            }
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
        __syncthreads();
        if (tid == 0) sm.heads = 0;
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
    // a row to a cluster, of as many CTAs as the machine has places for (one row of 152064: 37
    // us with one CTA, 27 with four, 22 with eight; 256 rows 65 us with one, 90 with two)
    const int slots = kCtas * nsm;
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
