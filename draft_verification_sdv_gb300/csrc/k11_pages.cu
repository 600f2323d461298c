// k11_pages.cu -- the cache's pages from request lengths (sdv_pages_extend,
// sdv_pages_release): a stack of free pages, each sequence's table row.
//
// A sequence that is to hold `end` positions needs ceil(end / P) pages and takes
// those it lacks.  Where its pages lie on the stack is the sum of what the
// sequences before it take, so that every CTA adds those up for itself (a few
// kilobytes, out of L2) and fills its own sequences' rows at once; nothing is
// decided by the order in which threads run.  Each page is read from the list
// and written to a table once, each token's position and slot written once.
// What all of them read, the stack's height and the pages held, changes in a
// kernel after, or behind a barrier where one CTA does it all.
//
// Small calls are bound by their launches and a chain of five reads (64 sequences of one
// token: 4.7 us; 48 trees of 129 nodes: 4.3 and 2.3 us).  Large ones issue for 60 % of
// the time (300 prompts of up to 8191 tokens: 9.7 us, 3.0 TB/s of positions and slots;
// 13.4 us with two divisions a token, which small calls liked better by 0.4); pages that
// go back wait at barriers behind such chains (154 000: 4.8 us, 7.7 with a warp to a
// sequence).
#include "sdv_device.cuh"
#include "sdv_layer.h"
#include "sdv_plan.h"

namespace sdv {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;

struct Want {                // one sequence's
    int held, pages;         // pages it holds, and that it takes or (release) gives back
    bool bad;
};

template <bool EXTEND> __device__ __forceinline__ Want want_of(const PagesArgs& a, int b) {
    Want w;
    w.held = a.held[b];
    const int at = a.start[b], count = EXTEND ? (a.count ? a.count[b] : a.N) : 0;
    const int64_t room = static_cast<int64_t>(a.max_pages) * a.P;
    w.bad = w.held < 0 || w.held > a.max_pages || at < 0 || (EXTEND && (count < 0 || count > a.N || static_cast<int64_t>(at) + count > room));
    const int need = w.bad ? 0 : static_cast<int>((static_cast<int64_t>(at) + count + a.P - 1) / a.P);
    const int more = EXTEND ? need - w.held : w.held - need;
    w.pages = w.bad || more < 0 ? 0 : more;
    return w;
}

// Sum over the block; every thread gets it.
__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t* sm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
    __syncthreads();
    int64_t sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sm[w];
    return sum;
}

// Sum of the threads before this one; `total` of all.
__device__ __forceinline__ int64_t block_before(int64_t x, int64_t* sm, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t upto = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    __syncthreads();
    if (lane == 31) sm[warp] = upto;
    __syncthreads();
    int64_t before = upto - x;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sm[w];
        total += sm[w];
    }
    return before;
}

// The stack's height; out of range: nothing is taken or given back.
__device__ __forceinline__ int height_of(const PagesArgs& a) {
    const int h = *a.free_count;
    return h < 0 || h > a.pages ? -1 : h;
}

struct Seq { int held, pages, at, count; int64_t before; };

// The new height and what each sequence holds, once every row is filled.
template <bool EXTEND> __device__ __forceinline__ void finish(const PagesArgs& a, int height, int64_t* sm) {
    int64_t carry = 0, done = 0;
    if (height < 0) return;
    int64_t all = 0;
    if (!EXTEND) {
        for (int b = threadIdx.x; b < a.B; b += kThreads) all += want_of<false>(a, b).pages;
        all = block_sum(all, sm);
        if (all + height > a.pages) return;
    }
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        const Want w = b < a.B ? want_of<EXTEND>(a, b) : Want{0, 0, false};
        int64_t total;
        const int64_t before = carry + block_before(w.pages, sm, total);
        carry += total;
        if (b < a.B && w.pages > 0 && (!EXTEND || before + w.pages <= height)) {
            a.held[b] = EXTEND ? w.held + w.pages : w.held - w.pages;
            done += w.pages;
        }
    }
    done = block_sum(done, sm);
    if (threadIdx.x == 0) *a.free_count = static_cast<int>(EXTEND ? height - done : height + done);
}

// Sequences blockIdx.x * each .. + each - 1; blockIdx.y shares out their tokens and pages.
template <bool EXTEND> __global__ void __launch_bounds__(kThreads) pages_kernel(const PagesArgs a, int each, int columns) {
    __shared__ int64_t sm[kWarps];
    __shared__ Seq s_seq[kThreads];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int first = blockIdx.x * each, last = min(first + each, a.B);
    const int height = height_of(a);
    // pages of the sequences before these; those of all, when they go back
    int64_t sum = 0, all = 0;
    for (int b = tid; b < (EXTEND ? first : a.B); b += kThreads) {
        const int n = want_of<EXTEND>(a, b).pages;
        if (b < first) sum += n;
        all += n;
    }
    int64_t carry = block_sum(sum, sm);
    if (!EXTEND) all = block_sum(all, sm);
    unsigned bad = height < 0 || (!EXTEND && all + height > a.pages) ? kStatusBadLength : 0u;
    const bool stuck = bad != 0;
    const int n0 = blockIdx.y * columns, n1 = min(n0 + columns, a.N);
    for (int b0 = first; b0 < last; b0 += kThreads) {
        const int b = b0 + tid, seqs = min(kThreads, last - b0);
        Want w{0, 0, false};
        if (b < last) w = want_of<EXTEND>(a, b);
        int64_t total;
        const int64_t before = carry + block_before(w.pages, sm, total);
        carry += total;
        if (w.bad) bad |= kStatusBadLength;
        if (EXTEND && !stuck && w.pages > 0 && before + w.pages > height) bad |= kStatusNoPages;
        const bool served = !stuck && w.pages > 0 && (!EXTEND || before + w.pages <= height);
        if (tid < seqs)
            s_seq[tid] = Seq{w.held, served ? w.pages : 0, a.start[b], w.bad || !EXTEND ? 0 : a.count ? a.count[b] : a.N, before};
        __syncthreads();
        // rows of the table: a warp to a sequence, or all of them to one where there are few
        const bool many = seqs >= kWarps;
        const int own = many ? lane : tid, all_own = many ? 32 : kThreads;
        for (int i = many ? warp : 0; i < seqs; i += many ? kWarps : 1) {
            const Seq q = s_seq[i];
            int32_t* row = a.table + static_cast<int64_t>(b0 + i) * a.max_pages;
            for (int x = own + all_own * blockIdx.y; x < q.pages; x += all_own * gridDim.y) {
                if (EXTEND) {
                    const int page = a.list[height - 1 - (q.before + x)];
                    if (page < 0 || page >= a.pages) bad |= kStatusBadPage;
                    row[q.held + x] = page;
                } else {
                    const int at = q.held - q.pages + x, page = row[at];
                    if (page < 0 || page >= a.pages) bad |= kStatusBadPage;
                    a.list[height + all - 1 - (q.before + x)] = page;
                    row[at] = -1;
                }
            }
        }
        if (EXTEND && n1 > n0) {                     // positions and slots
            // a power of two of threads to a sequence, and one division for all its tokens
            const int shift = min(n1 - n0 > 1 ? 32 - __clz(n1 - n0 - 1) : 0, 31 - __clz(kThreads)), group = 1 << shift;
            const int step_pages = group / a.P, step_in = group - step_pages * a.P;
            for (int i = tid >> shift; i < seqs; i += kThreads >> shift) {
                const Seq q = s_seq[i];
                const int32_t* row = a.table + static_cast<int64_t>(b0 + i) * a.max_pages;
                const int offset = a.base ? a.base[b0 + i] : 0, has = q.held + q.pages;
                int n = n0 + (tid & (group - 1)), place = 0, in = 0;
                if (n < q.count) {
                    place = (q.at + n) / a.P;
                    in = q.at + n - place * a.P;
                }
                for (; n < n1; n += group) {
                    const int64_t o = static_cast<int64_t>(b0 + i) * a.N + n;
                    int64_t slot = -1;
                    int position = 0;
                    if (n < q.count) {
                        int page = -1;               // a new page comes from the list: its row is being filled
                        if (place < q.held)
                            page = row[place];
                        else if (place < has)
                            page = a.list[height - 1 - (q.before + place - q.held)];
                        if (page >= 0 && page < a.pages)
                            slot = static_cast<int64_t>(page) * a.P + in;
                        else if (place < has)
                            bad |= kStatusBadPage;
                        position = q.at + (a.depth ? a.depth[o] : n) + offset;
                        place += step_pages, in += step_in;
                        if (in >= a.P) in -= a.P, ++place;
                    }
                    if (a.positions) a.positions[o] = position;
                    if (a.slots) a.slots[o] = slot;
                }
            }
        }
        __syncthreads();
    }
    if (bad && a.status) atomicOr(a.status, bad);
    if (gridDim.x * gridDim.y == 1) finish<EXTEND>(a, height, sm);
}

template <bool EXTEND> __global__ void __launch_bounds__(kThreads) finish_kernel(const PagesArgs a) {
    __shared__ int64_t sm[kWarps];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    finish<EXTEND>(a, height_of(a), sm);
}

template <bool EXTEND> cudaError_t launch(const PagesArgs& a, int nsm, cudaStream_t s) {
    // one CTA does it all where there is little: 64 tokens take 4.7 us, and a second launch 2.5
    const int64_t items = static_cast<int64_t>(a.B) * (EXTEND ? a.N : a.max_pages);
    const bool small = items <= 4 * kThreads;
    int each = a.B, columns = a.N > 0 ? a.N : 1;
    dim3 grid(1, 1);
    if (!small) {
        const int want = 2 * nsm;
        each = (a.B + want - 1) / want;
        grid.x = static_cast<unsigned>((a.B + each - 1) / each);
        int split = static_cast<int>(want / grid.x);
        const int most = EXTEND ? (a.N + kThreads - 1) / kThreads : (a.max_pages + kThreads - 1) / kThreads;
        split = split > most ? most : split < 1 ? 1 : split;
        if (EXTEND) {
            columns = (a.N + split - 1) / split;
            split = (a.N + columns - 1) / columns;
        }
        grid.y = static_cast<unsigned>(split);
    }
    pages_kernel<EXTEND><<<grid, kThreads, 0, s>>>(a, each, columns);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || grid.x * grid.y == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, finish_kernel<EXTEND>, a);
}

}  // namespace

cudaError_t launch_pages_extend(const PagesArgs& a, int nsm, cudaStream_t s) { return launch<true>(a, nsm, s); }
cudaError_t launch_pages_release(const PagesArgs& a, int nsm, cudaStream_t s) { return launch<false>(a, nsm, s); }

}  // namespace sdv
