// k12_rows.cu -- draws from rows of logits and their truncation (sdv_sample,
// sdv_logits_truncate): rows in 32 bits.
//
// What a row keeps or draws is nearly always among the few hundred largest logits.  A
// sample gives a bound that so many reach; one look at the row writes those, the
// head, into a list, which is sorted by logit and index.  There top-k, min-p, top-p
// and the draw are places of running sums.  Where only top-p or the draw limits the
// row, a second look adds up all weights (whole numbers: the sum is the one that
// any other order gives), and the head's share of them tells whether the place lies in
// it, unless it is plain that it does not.  Other rows are counted and weighed into bins of equal width in (max - x) / T,
// which keep the order, and the bin that holds a place is listed and sorted in turn
// (row_by_bins); rows with too many logits in one bin go the long way, in passes over
// histograms of keys (row_in_passes).
//
// A row is shared by a cluster of C CTAs where there are few; the first one has the list.
// What bounds it: for a row that its head settles, the latency of its steps (13 000
// clocks to list 32001 logits, 9000 to sort 1000 of them, 6500 for the places); a
// second look takes 35 000 to 50 000 clocks for the instructions of the weights, and
// bins 50 000 to 70 000.  168 rows of 32001 under top-p or min-p: 60 to 80 us, as many
// rows need bins (166 when all went in passes, 109 before bins, 96 with both for a row).
#include "k12_rows.cuh"

namespace sdv {
namespace {

using namespace rows;

constexpr int kThreads = 512, kWarps = kThreads / 32, kBins = 4096;
constexpr int kList = 2048, kOwn = kList / kThreads;
constexpr uint32_t kOddNan = 1u;
// What a logit behind the head is taken to weigh, in units of the head's least, where it is
// guessed whether the place lies there (normal logits: 0.2 for a deviation of 1, 0.02 for 6;
// the answer does not depend on it).
constexpr float kRest = 0.125f;

struct Head {
    uint64_t list[kList];                // key << 32 | ~index, 0: none
    uint64_t before[kList];              // weight of those before
    Tables tables;
    Factors factors;
    float floor;
    uint64_t sum[kWarps], total;
    uint32_t word[8 * kWarps];
    uint32_t listed, odd, finite, over, at;
    uint64_t part[8];                    // weights and counts of the CTAs' parts
    uint32_t count[8], strange[8];
    // what the first CTA has found
    uint32_t verdict, kept;
};
struct Bins {
    Head head;
    Hist<kBins> hist;
    Picked<kThreads> picked;
};
union Smem {
    Head head;
    Bins bins;
    PassSmem<kThreads, kBins> passes;
};
static_assert(2 * (sizeof(Smem) + 1024) <= 227 * 1024, "two CTAs per SM");
enum : uint32_t { kDone, kCopy, kBad, kLongWay };        // verdicts: kept ones are the list's first; all are kept

__device__ __forceinline__ Smem& smem() {
    extern __shared__ __align__(16) unsigned char raw[];
    return *reinterpret_cast<Smem*>(raw);
}

__device__ __forceinline__ float largest_of(const uint4& v) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
}

// Writes the logits of this CTA's part of a row that reach the bound into the first CTA's
// list; whether there is a NaN or +infinity into `odd`.  Returns the bound, a key.
template <int C> __device__ __noinline__ uint32_t list_head(const unsigned char* row, int V, const Span span, int rank) {
    constexpr int U = 4, kAll = C * kThreads, kSamples = C * kWarps * 2;
    Head& sm = smem().head;
    Head* const lead = of_rank<C>(&sm, 0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, me = rank * kThreads + threadIdx.x;
    const uint64_t policy = first_policy();
    const unsigned char* first = row + span.head * 4;
    uint32_t bound = kKeyLow + 1;                    // (a short row is head as a whole)
    if (V > kList) {
        const int chunks = (span.vectors + 31) / 32;
        uint32_t least = 0xffffffffu, most = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int n = (rank * kWarps + warp) * 2 + u;
            const int at = (chunks >= kSamples ? static_cast<int>(static_cast<uint32_t>(n) * chunks / kSamples) : n) * 32 + lane;
            float x = -INFINITY;
            if (at < span.vectors) x = largest_of(ld_hint(first + static_cast<int64_t>(at) * 16, policy));
            const uint32_t top = __reduce_max_sync(0xffffffffu, x > -INFINITY ? key_of(x) : 0u);
            if (top) least = min(least, top);
            most = max(most, top);
        }
        if (lane < C) of_rank<C>(&sm, lane)->word[rank * kWarps + warp] = V < kManyLogits || most == 0 ? least : most;
        sync_all<C>();
        bound = min(fourth_smallest<C * kWarps>(sm.word), kKeyHigh);
    }
    const float f = of_key(bound);
    float most = -INFINITY;
    bool odd = false;
    auto put = [&](float x, int index) {
        if (!(x >= f)) return;
        const uint32_t n = atomicAdd(&lead->listed, 1u);
        if (n < kList) lead->list[n] = static_cast<uint64_t>(key_of(x)) << 32 | static_cast<uint32_t>(~index);
    };
    auto take = [&](const uint4& v, int index) {
        const float x = __uint_as_float(v.x), y = __uint_as_float(v.y), z = __uint_as_float(v.z), w = __uint_as_float(v.w);
        const float top = fmaxf(fmaxf(x, y), fmaxf(z, w));
        most = fmaxf(most, top);
        odd |= !((x + y) + (z + w) < INFINITY) && (x != x || y != y || z != z || w != w);
        if (top >= f) put(x, index), put(y, index + 1), put(z, index + 2), put(w, index + 3);
    };
    int i = me;
    for (; i + (U - 1) * kAll < span.vectors; i += U * kAll) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = ld_hint(first + static_cast<int64_t>(i + u * kAll) * 16, policy);
#pragma unroll
        for (int u = 0; u < U; ++u) take(v[u], span.index_of(i + u * kAll));
    }
    for (; i < span.vectors; i += kAll) take(ld_hint(first + static_cast<int64_t>(i) * 16, policy), span.index_of(i));
    if (me < span.loose) {                           // (six at most)
        const int y = span.loose_at(me);
        const float x = reinterpret_cast<const float*>(row)[y];
        odd |= x != x;
        most = fmaxf(most, x);
        put(x, y);
    }
    odd |= most == INFINITY;
    if (__any_sync(0xffffffffu, odd) && lane == 0) atomicOr(&sm.odd, kOddNan);
    return bound;
}

// Weights and number of the finite logits of this CTA's part, told to every CTA.
template <int C> __device__ __noinline__ void sum_all(const unsigned char* row, const Span span, int rank, const Scale scale) {
    constexpr int U = 2, kAll = C * kThreads;
    Head& sm = smem().head;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, me = rank * kThreads + threadIdx.x;
    uint64_t sum = 0;
    uint32_t n = 0;
    auto add = [&](float x) {
        sum += weight_of(scale, x, sm.tables);
        n += x > -INFINITY;
    };
    auto take = [&](const uint4& v) {
        add(__uint_as_float(v.x)), add(__uint_as_float(v.y)), add(__uint_as_float(v.z)), add(__uint_as_float(v.w));
    };
    const unsigned char* first = row + span.head * 4;
    int i = me;
    for (; i + (U - 1) * kAll < span.vectors; i += U * kAll) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = ld_row(first + static_cast<int64_t>(i + u * kAll) * 16);
#pragma unroll
        for (int u = 0; u < U; ++u) take(v[u]);
    }
    for (; i < span.vectors; i += kAll) take(ld_row(first + static_cast<int64_t>(i) * 16));
    if (me < span.loose) add(reinterpret_cast<const float*>(row)[span.loose_at(me)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    n = __reduce_add_sync(0xffffffffu, n);
    __syncthreads();
    if (lane == 0) sm.sum[warp] = sum, sm.word[warp] = n;
    __syncthreads();
    if (threadIdx.x < C) {
        uint64_t s = 0;
        uint32_t c = 0;
        for (int w = 0; w < kWarps; ++w) s += sm.sum[w], c += sm.word[w];
        Head* to = of_rank<C>(&sm, threadIdx.x);
        to->part[rank] = s, to->count[rank] = c;
    }
}

// The list's first `size` entries in falling order (a power of two, 64 at least).  Merges of
// alternating runs; each warp holds 64 entries in registers, two to a lane (i and
// i + 32), so that only exchanges over 64 entries and more go through shared memory.
__device__ __noinline__ void sort_list(int size) {
    Head& sm = smem().head;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto within = [&](int base, int k, int top) {    // the steps top, top / 2, ... 1 of merges to runs of k
        uint64_t a = sm.list[base + lane], b = sm.list[base + 32 + lane];
        if (top == 32) {
            if ((a < b) == (((base + lane) & k) == 0)) {
                const uint64_t x = a;
                a = b, b = x;
            }
            top = 16;
        }
        for (int j = top; j > 0; j >>= 1) {
            const uint64_t x = __shfl_xor_sync(0xffffffffu, a, j), y = __shfl_xor_sync(0xffffffffu, b, j);
            const bool first = (lane & j) == 0;
            // (a falling run keeps the larger one first)
            const bool fa = ((base + lane) & k) == 0, fb = ((base + 32 + lane) & k) == 0;
            a = (a > x) == (first == fa) ? a : x;
            b = (b > y) == (first == fb) ? b : y;
        }
        sm.list[base + lane] = a, sm.list[base + 32 + lane] = b;
    };
    __syncthreads();
    for (int base = warp * 64; base < size; base += kWarps * 64)
        for (int k = 2; k <= 64; k <<= 1) {
            within(base, k, k >> 1);
            __syncwarp();
        }
    for (int k = 128; k <= size; k <<= 1) {
        for (int j = k >> 1; j >= 64; j >>= 1) {
            __syncthreads();
            for (int x = threadIdx.x; x < size / 2; x += kThreads) {
                const int lo = 2 * x - (x & (j - 1)), hi = lo + j;   // pairs j apart
                const uint64_t a = sm.list[lo], b = sm.list[hi];
                if ((a < b) == ((lo & k) == 0)) sm.list[lo] = b, sm.list[hi] = a;
            }
        }
        __syncthreads();
        for (int base = warp * 64; base < size; base += kWarps * 64) within(base, k, 32);
    }
    __syncthreads();
}

// The weights before each of the list's n entries, and their total.
__device__ __noinline__ void sum_list(int n, const Scale scale) {
    Head& sm = smem().head;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t w[kOwn], own = 0;
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
        const int i = tid * kOwn + x;
        w[x] = i < n ? weight_of(scale, of_key(static_cast<uint32_t>(sm.list[i] >> 32)), sm.tables) : 0;
        own += w[x];
    }
    uint64_t upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    if (lane == 31) sm.sum[warp] = upto;
    __syncthreads();
    uint64_t before = upto - own;
    for (int x = 0; x < warp; ++x) before += sm.sum[x];
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
        sm.before[tid * kOwn + x] = before;
        before += w[x];
    }
    if (tid == kThreads - 1) sm.total = before;
    __syncthreads();
}

// The entry where the running weight passes `target` (less than the total): into sm.at.
__device__ __forceinline__ int find(Head& sm, int n, uint64_t target) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t end = i + 1 < n ? sm.before[i + 1] : sm.total;
        if (sm.before[i] <= target && target < end) sm.at = i;
    }
    __syncthreads();
    const int at = static_cast<int>(sm.at);
    __syncthreads();
    return at;
}

// Bins of equal width in (max - x) / T, which keep the order.
struct Binned {
    float top, wide;                     // bins per unit of logit
    __device__ __forceinline__ explicit Binned(const Scale& s) : top(s.top), wide((kBins / 64) * 0.5f * s.hi) {}
    __device__ __forceinline__ int of(float x) const { return static_cast<int>(fminf((top - x) * wide, static_cast<float>(kBins - 1))); }
};

// work(x, index) for each logit of a row, by one CTA.
template <typename Work> __device__ __forceinline__ void each_logit(const unsigned char* row, int V, Work work) {
    constexpr int U = 2;
    const int tid = threadIdx.x;
    const Span span = span_of(row, V, 4);
    const unsigned char* first = row + span.head * 4;
    auto four = [&](const uint4& v, int at) {
        work(__uint_as_float(v.x), at), work(__uint_as_float(v.y), at + 1);
        work(__uint_as_float(v.z), at + 2), work(__uint_as_float(v.w), at + 3);
    };
    int i = tid;
    for (; i + (U - 1) * kThreads < span.vectors; i += U * kThreads) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = ld_row(first + static_cast<int64_t>(i + u * kThreads) * 16);
#pragma unroll
        for (int u = 0; u < U; ++u) four(v[u], span.index_of(i + u * kThreads));
    }
    for (; i < span.vectors; i += kThreads) four(ld_row(first + static_cast<int64_t>(i) * 16), span.index_of(i));
    if (tid < span.loose) work(reinterpret_cast<const float*>(row)[span.loose_at(tid)], span.loose_at(tid));
}

// All of a row's logits into bins, by one CTA: their weight (head.part[0]), how many are
// finite (head.count[0]) and reach the floor (head.over).
__device__ __noinline__ void weigh_bins(const unsigned char* row, int V, const Scale scale, float floor) {
    Bins& sm = smem().bins;
    Head& head = sm.head;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Binned bins(scale);
    for (int x = tid; x < kBins; x += kThreads) sm.hist.count[x] = 0, sm.hist.mass[x] = 0;
    if (tid == 0) head.over = 0;
    __syncthreads();
    uint64_t weight = 0;
    uint32_t finite = 0, over = 0;
    each_logit(row, V, [&](float x, int) {
        if (!(x > -INFINITY)) return;
        const uint64_t w = weight_of(scale, x, head.tables);
        const int b = bins.of(x);
        atomicAdd(&sm.hist.count[b], 1u);
        add_weight(&sm.hist.mass[b], w);
        weight += w;
        ++finite;
        over += x >= floor;
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) weight += __shfl_xor_sync(0xffffffffu, weight, o);
    finite = __reduce_add_sync(0xffffffffu, finite);
    over = __reduce_add_sync(0xffffffffu, over);
    if (lane == 0) head.sum[warp] = weight, head.word[warp] = finite, atomicAdd(&head.over, over);
    __syncthreads();
    if (tid == 0) {
        weight = 0, finite = 0;
        for (int w = 0; w < kWarps; ++w) weight += head.sum[w], finite += head.word[w];
        head.part[0] = weight, head.count[0] = finite;
    }
    __syncthreads();
}

// A row whose places do not lie in its head; the largest logit and the factors are known,
// and the bins are filled (weigh_bins).  The first CTA; false: a bin does not fit the list,
// and nothing is written.
template <bool DRAW> __device__ __noinline__ bool row_by_bins(const RowsArgs& a, int r, const Ask q, const Scale scale) {
    Bins& sm = smem().bins;
    Head& head = sm.head;
    const int tid = threadIdx.x;
    const unsigned char* row = static_cast<const unsigned char*>(a.logits) + r * a.in_stride;
    const Binned bins(scale);
    uint64_t weight = head.part[0];
    const uint32_t finite = head.count[0];
    uint32_t kept = finite, most = min(finite, head.over);
    if (q.top_k > 0) most = min(most, static_cast<uint32_t>(q.top_k));
    // the last of the first `most`; the last before which less than top_p of their weight
    // lies; the one that is drawn
    uint64_t last = 0, unit = 0;                     // (an entry, as the list has them: what is not less is kept)
    int listed = -1;
#pragma unroll 1
    for (int ask = 0; ask < 3; ++ask) {
        if (ask == 0 ? most >= finite : ask == 1 ? !(q.top_p < 1.0f) : !DRAW) continue;
        const uint64_t target = ask == 0 ? most - 1 : ask == 1 ? times_up(q.top_p, weight) - 1 : times_down(q.u, weight);
        pick<kThreads, kBins>(sm.picked, sm.hist, ask != 0, target);
        const int bin = sm.picked.bin, n = static_cast<int>(sm.picked.at_n);
        if (n > kList) return false;
        if (bin != listed) {
            listed = bin;
            if (tid == 0) head.listed = 0;
            int size = 64;
            while (size < n) size <<= 1;
            for (int x = n + tid; x < size; x += kThreads) head.list[x] = 0;
            __syncthreads();
            each_logit(row, a.V, [&](float x, int index) {
                if (x > -INFINITY && bins.of(x) == bin)
                    head.list[atomicAdd(&head.listed, 1u)] = static_cast<uint64_t>(key_of(x)) << 32 | static_cast<uint32_t>(~index);
            });
            sort_list(size);
            sum_list(n, scale);
        }
        const int at = ask == 0 ? static_cast<int>(target) - static_cast<int>(sm.picked.before_n) : find(head, n, target - sm.picked.before_w);
        const uint64_t end = sm.picked.before_w + (at + 1 < n ? head.before[at + 1] : head.total);
        if (ask < 2) {
            kept = sm.picked.before_n + at + 1;
            weight = end;
            last = head.list[at];
        } else {
            unit = end - sm.picked.before_w - head.before[at];
            if (tid == 0) {
                a.tokens[r] = static_cast<int32_t>(~static_cast<uint32_t>(head.list[at]));
                if (a.logprob) a.logprob[r] = log_share(scale, of_key(static_cast<uint32_t>(head.list[at] >> 32)), unit, weight, head.tables);
            }
        }
        __syncthreads();
    }
    if (tid == 0 && a.kept) a.kept[r] = static_cast<int32_t>(kept);
    if constexpr (!DRAW) {
        float* out = reinterpret_cast<float*>(static_cast<unsigned char*>(a.out) + r * a.out_stride);
        each_logit(row, a.V, [&](float x, int index) {
            out[index] = (static_cast<uint64_t>(key_of(x)) << 32 | static_cast<uint32_t>(~index)) >= last ? x : -INFINITY;
        });
    }
    return true;
}

template <bool DRAW, int C> __global__ void __launch_bounds__(kThreads, 2) rows_f32_kernel(const RowsArgs a) {
    Head& sm = smem().head;
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int me = rank * kThreads + tid;
    constexpr int kAll = C * kThreads;
    const float nan = __int_as_float(0x7fc00000);
    bool tables = false;
    for (int64_t r = blockIdx.x / C; r < a.rows; r += gridDim.x / C) {
        const Ask q = ask_of(a, r);
        const unsigned char* row = static_cast<const unsigned char*>(a.logits) + r * a.in_stride;
        float* out = reinterpret_cast<float*>(static_cast<unsigned char*>(a.out) + r * a.out_stride);
        const Span span = span_of(row, a.V, 4);
        sync_all<C>();                               // (the row before is done with shared memory)
        if (!tables) load_tables(sm.tables, tid, kThreads);
        tables = true;
        if (tid == 0) sm.listed = sm.odd = 0;
        if (tid == kThreads - 1) sm.factors = factors_of(q.T, q.min_p);
        sync_all<C>();
        const uint32_t bound = list_head<C>(row, a.V, span, rank);
        __syncthreads();
        if (tid < C) of_rank<C>(&sm, tid)->strange[rank] = sm.odd;
        sync_all<C>();
        uint32_t odd = 0;
        for (int c = 0; c < C; ++c) odd |= sm.strange[c];
        const uint32_t listed = of_rank<C>(&sm, 0)->listed;

        // ---- the head, sorted ----
        const int n = static_cast<int>(min(listed, static_cast<uint32_t>(kList)));
        const bool usable = !q.bad && !odd && listed > 0 && listed <= kList;
        int size = 64;
        while (size < n) size <<= 1;
        if (rank == 0 && usable) {
            for (int i = n + tid; i < size; i += kThreads) sm.list[i] = 0;
            sort_list(size);
        }
        sync_all<C>();
        const float top = usable ? of_key(static_cast<uint32_t>(of_rank<C>(&sm, 0)->list[0] >> 32)) : 0.0f;
        const Scale scale{top, sm.factors.hi, sm.factors.lo};
        // does it hold what top-k and min-p keep, or do all weights have to be known?
        if (tid == 0) sm.floor = usable && q.min_p > 0.0f ? floor_of(top, sm.factors.reach) : -INFINITY;
        __syncthreads();
        const float floor = sm.floor;
        const bool by_floor = q.min_p > 0.0f && floor >= of_key(bound), by_k = q.top_k > 0 && q.top_k <= n;
        const bool limited = q.T == 0.0f || by_floor || by_k;
        const bool whole = bound == kKeyLow + 1;     // the list holds every finite logit
        const bool sums = usable && !limited && !whole && q.top_k == 0 && q.min_p == 0.0f && (DRAW || q.top_p < 1.0f || a.kept);
        if (rank == 0 && usable && q.T != 0.0f) sum_list(n, scale);
        // A place that is likely not to lie in the head is looked for in bins at once, which
        // saves weighing all logits twice.  32001 normal logits under top-p 0.95, 168 rows:
        // 96 us against 125 with a second look first (deviation 3); 1088 rows 352 against 470,
        // and where the head does, 227 against 260 with bins for every row (deviation 6).
        bool binned = false;
        if (C == 1 && sums) {
            const float held = static_cast<float>(sm.total), least = static_cast<float>(weight_of(scale, of_key(bound), sm.tables));
            const float part = q.top_p < 1.0f ? q.top_p : DRAW ? q.u : 0.0f;
            binned = part * (held + kRest * least * static_cast<float>(a.V - n)) >= held;
        }
        if (binned) {
            weigh_bins(row, a.V, scale, floor);
        } else if (sums) {
            sum_all<C>(row, span, rank, scale);
            sync_all<C>();
        }
        if (rank == 0) {
            uint32_t verdict = kDone;
            uint64_t weight = uint64_t(1) << kOneBits, unit = weight;
            int kept = 1, drawn = 0, all = 0;        // all: finite logits, where they are known
            if (q.bad || odd) {
                verdict = kBad;
            } else if (!usable) {
                verdict = kLongWay;                  // (a row without finite logits too)
            } else if (q.T != 0.0f) {
                kept = n, weight = sm.total;
                if (whole) all = n;
                if (sums) {
                    weight = 0;
                    for (int c = 0; c < C; ++c) weight += sm.part[c], all += static_cast<int>(sm.count[c]);
                    kept = all;
                } else if (!limited && !whole) {
                    verdict = !DRAW && q.top_k == 0 && q.min_p == 0.0f ? kCopy : kLongWay;       // (the former: nothing cuts it)
                }
                if (by_floor || (whole && q.min_p > 0.0f)) {
                    if (tid == 0) sm.over = 0;
                    __syncthreads();
                    uint32_t c = 0;
                    for (int i = tid; i < n; i += kThreads) c += of_key(static_cast<uint32_t>(sm.list[i] >> 32)) >= floor;
                    c = __reduce_add_sync(0xffffffffu, c);
                    if (lane == 0) atomicAdd(&sm.over, c);
                    __syncthreads();
                    kept = min(kept, static_cast<int>(sm.over));
                }
                if (q.top_k > 0) kept = min(kept, q.top_k);
                if (!sums && kept < n) weight = sm.before[kept];
                if (verdict == kDone && q.top_p < 1.0f) {
                    // tokens while what comes before them weighs less than this
                    const uint64_t need = times_up(q.top_p, weight);
                    if (need > sm.total) {
                        verdict = kLongWay;
                    } else {
                        kept = find(sm, n, need - 1) + 1;
                        weight = kept < n ? sm.before[kept] : sm.total;
                    }
                }
                if (verdict == kDone && DRAW) {
                    const uint64_t aim = times_down(q.u, weight);
                    if (aim >= sm.total) {
                        verdict = kLongWay;
                    } else {
                        drawn = find(sm, n, aim);
                        unit = (drawn + 1 < n ? sm.before[drawn + 1] : sm.total) - sm.before[drawn];
                    }
                }
                if (verdict == kDone && !DRAW && kept > n) verdict = kCopy;
            }
            if (tid == 0) {
                if (verdict == kBad) {
                    if (a.status) atomicOr(a.status, q.bad ? kStatusBadTemp : kStatusBadRow);
                    if (DRAW) a.tokens[r] = -1;
                    if (DRAW && a.logprob) a.logprob[r] = nan;
                } else if (DRAW && verdict == kDone) {
                    a.tokens[r] = static_cast<int32_t>(~static_cast<uint32_t>(sm.list[drawn]));
                    if (a.logprob) a.logprob[r] = log_share(scale, of_key(static_cast<uint32_t>(sm.list[drawn] >> 32)), unit, weight, sm.tables);
                }
                if (a.kept && verdict != kLongWay) a.kept[r] = verdict == kBad ? 0 : kept;
            }
            __syncthreads();
            if (tid < C) {
                Head* to = of_rank<C>(&sm, tid);
                to->verdict = verdict, to->kept = static_cast<uint32_t>(kept);
            }
        }
        sync_all<C>();
        const uint32_t verdict = sm.verdict;
        if (verdict == kLongWay) {
            if (rank == 0 && usable && !binned) weigh_bins(row, a.V, scale, floor);
            if (rank == 0 && !(usable && row_by_bins<DRAW>(a, static_cast<int>(r), q, scale))) {
                PassSmem<kThreads, kBins>& ps = smem().passes;
                __syncthreads();
                load_tables(ps.tables, tid, kThreads);
                __syncthreads();
                row_in_passes<false, DRAW, kThreads, kBins>(a, r, ps);
                tables = false;
            }
        } else if constexpr (!DRAW) {
            if (verdict == kCopy) {
                const float* from = reinterpret_cast<const float*>(row);
                if (from != out)
                    for (int y = me; y < a.V; y += kAll) out[y] = from[y];
            } else {
                // all becomes -infinity (or NaN), and what is kept comes back
                const float none = verdict == kBad ? nan : -INFINITY;
                float mine[kOwn];                    // (with their signs, if they are zeros)
                uint32_t index[kOwn];
                if (rank == 0)
#pragma unroll
                    for (int x = 0; x < kOwn; ++x) {
                        const uint32_t i = tid + x * kThreads;
                        index[x] = verdict == kDone && i < sm.kept ? ~static_cast<uint32_t>(sm.list[i]) : 0xffffffffu;
                        if (index[x] != 0xffffffffu) mine[x] = reinterpret_cast<const float*>(row)[index[x]];
                    }
                sync_all<C>();
                const Span to = span_of(reinterpret_cast<const unsigned char*>(out), a.V, 4);
                const uint32_t bits = __float_as_uint(none);
                const uint64_t drop = drop_policy();
                for (int y = me; y < to.vectors; y += kAll)
                    st_hint(reinterpret_cast<unsigned char*>(out + to.index_of(y)), make_uint4(bits, bits, bits, bits), drop);
                if (me < to.loose) out[to.loose_at(me)] = none;
                sync_all<C>();
                if (rank == 0)
#pragma unroll
                    for (int x = 0; x < kOwn; ++x)
                        if (index[x] != 0xffffffffu) out[index[x]] = mine[x];
            }
        }
    }
    sync_all<C>();                                   // no CTA goes while another may still write to it
}

template <bool DRAW, int C> cudaError_t launch_one(const RowsArgs& a, int slots, cudaStream_t s) {
    const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(rows_f32_kernel<DRAW, C>), sizeof(Smem));
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
    return cudaLaunchKernelEx(&cfg, rows_f32_kernel<DRAW, C>, a);
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

cudaError_t launch_rows(const RowsArgs& a, bool bf16, bool draw, int nsm, cudaStream_t s) {
    if (bf16) return launch_rows_bf16(a, draw, nsm, s);
    return draw ? launch<true>(a, nsm, s) : launch<false>(a, nsm, s);
}

}  // namespace sdv
