// k8_attn.cuh -- what the tree-attention kernels share: how the work is cut,
// where partial results go, visibility.
//
// A unit is (sequence b, kv head h, row tile mt): MT of the N * g query rows
// that read kv head h (row = node * g + head within the group), against all
// positions that the tile's nodes can see, BN positions at a time.  All units'
// key tiles form one long line, b outermost, and CTA i of n takes the i-th n-th
// of it (so ragged lengths need no tuning: every CTA streams the same number of
// tiles).  A unit cut by the end of a CTA's part gives partial results, one per
// CTA: normalised fp32 outputs and the base-2 log of their sum, joined by
// combine_kernel.  A CTA has at most two: a unit begun before it (slot 0) and
// one that goes on after it (slot 1).
#pragma once

#include "sdv_device.cuh"
#include "sdv_layer.h"
#include "sdv_plan.h"

namespace sdv {
namespace attn {

struct Cut {                 // one sequence
    int ctx, cnt;            // committed positions and nodes (bad: both 0)
    bool bad;
};

__device__ __forceinline__ Cut cut_of(const AttnArgs& a, int b) {
    Cut c;
    c.ctx = __ldg(a.ctx + b);
    c.cnt = a.count ? __ldg(a.count + b) : a.N;
    c.bad = c.ctx < 0 || c.cnt < 0 || c.cnt > a.N ||
            static_cast<int64_t>(c.ctx) + c.cnt > static_cast<int64_t>(a.max_pages) * a.c.P;
    if (c.bad) c.ctx = c.cnt = 0;
    return c;
}

// Positions that row tile mt of a sequence reads.
template <int MT> __device__ __forceinline__ int tile_len(const AttnArgs& a, const Cut& c, int mt) {
    const int first = mt * MT / a.g;
    if (first >= c.cnt) return 0;
    if (a.mask) return c.ctx + c.cnt;
    const int last = (mt * MT + MT - 1) / a.g;
    return c.ctx + min(c.cnt, last + 1);
}

template <int BN> __device__ __forceinline__ int tiles_of(int len) {
    return len > 0 ? (len + BN - 1) / BN : 1;       // an empty unit still writes its rows
}

// Tiles of all row tiles of one head of a sequence.
template <int MT, int BN>
__device__ __forceinline__ int64_t head_tiles(const AttnArgs& a, const Cut& c, int mts) {
    if (a.mask) {
        const int live = min(mts, (c.cnt * a.g + MT - 1) / MT);
        return static_cast<int64_t>(live) * tiles_of<BN>(c.ctx + c.cnt) + (mts - live);
    }
    int64_t n = 0;
    for (int mt = 0; mt < mts; ++mt) n += tiles_of<BN>(tile_len<MT>(a, c, mt));
    return n;
}

struct Part {                // a CTA's part of the line
    int64_t begin, end, total;
    int ctas;                // CTAs that have a part
    int b;                   // sequence of `begin`, and where its tiles begin
    int64_t seq0;
};

__device__ __forceinline__ int64_t part_begin(int64_t total, int n, int i) { return total * i / n; }
__device__ __forceinline__ int part_owner(int64_t total, int n, int64_t tile) {
    return static_cast<int>(((tile + 1) * n - 1) / total);
}

// Every thread of the CTA calls this; `sm` holds 40 int64.
template <int MT, int BN, int THREADS>
__device__ __forceinline__ Part find_part(const AttnArgs& a, int mts, int64_t* sm) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t mine = 0;
    for (int b = tid; b < a.B; b += THREADS)
        mine += head_tiles<MT, BN>(a, cut_of(a, b), mts) * a.c.H;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) sm[warp] = mine;
    __syncthreads();
    Part p;
    p.total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) p.total += sm[w];
    p.ctas = static_cast<int>(p.total < a.ctas ? p.total : a.ctas);
    const int i = blockIdx.x;
    if (i >= p.ctas) {
        p.begin = p.end = p.total;
        p.b = a.B;
        p.seq0 = p.total;
        return p;
    }
    p.begin = part_begin(p.total, p.ctas, i);
    p.end = part_begin(p.total, p.ctas, i + 1);
    if (warp == 0) {
        int64_t base = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + lane;
            const int64_t n = b < a.B ? head_tiles<MT, BN>(a, cut_of(a, b), mts) * a.c.H : 0;
            int64_t upto = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            const bool here = b < a.B && base + upto > p.begin && base + upto - n <= p.begin;
            if (here) sm[32] = b, sm[33] = base + upto - n;
            if (__ballot_sync(0xffffffffu, here)) break;
            base += __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    __syncthreads();
    p.b = static_cast<int>(sm[32]);
    p.seq0 = sm[33];
    return p;
}

struct Unit {
    int b, h, mt;
    Cut cut;
    int len;                 // positions it reads
    int t0, t1;              // this CTA's of its tiles
    bool whole;              // that is all of them
};

// Walks the units of a CTA's part: the first is found by division, the others
// follow one another.
template <int MT, int BN> struct Walk {
    int left, rest;          // tiles left of the part; tiles of the unit before it
    int b, h, mt;
    Cut cut;
    __device__ __forceinline__ void start(const AttnArgs& a, const Part& p, int mts) {
        left = static_cast<int>(p.end - p.begin);
        rest = 0;
        b = p.b;
        h = mt = 0;
        if (b >= a.B) return;
        cut = cut_of(a, b);
        const int64_t in_seq = p.begin - p.seq0, per_head = head_tiles<MT, BN>(a, cut, mts);
        h = static_cast<int>(in_seq / per_head);
        int64_t before = in_seq - h * per_head;
        if (a.mask) {
            const int t = tiles_of<BN>(cut.ctx + cut.cnt);
            const int live = min(mts, (cut.cnt * a.g + MT - 1) / MT);
            if (before < static_cast<int64_t>(live) * t) {
                mt = static_cast<int>(before / t);
                before -= static_cast<int64_t>(mt) * t;
            } else {
                mt = live + static_cast<int>(before - static_cast<int64_t>(live) * t);
                before = 0;
            }
        } else {
            while (true) {
                const int t = tiles_of<BN>(tile_len<MT>(a, cut, mt));
                if (before < t) break;
                before -= t;
                ++mt;
            }
        }
        rest = static_cast<int>(before);
    }
    __device__ __forceinline__ bool next(const AttnArgs& a, int mts, Unit& u) {
        if (left <= 0) return false;
        u.b = b;
        u.h = h;
        u.mt = mt;
        u.cut = cut;
        u.len = tile_len<MT>(a, cut, mt);
        const int tiles = tiles_of<BN>(u.len);
        u.t0 = rest;
        u.t1 = min(tiles, rest + left);
        u.whole = u.t0 == 0 && u.t1 == tiles;
        left -= u.t1 - u.t0;
        rest = 0;
        if (++mt == mts) {
            mt = 0;
            if (++h == a.c.H) {
                h = 0;
                if (++b < a.B) cut = cut_of(a, b);
            }
        }
        return true;
    }
};

// Partial results: [cta][slot] of MT rows of D fp32, then MT logs.
__device__ __forceinline__ float* part_rows(const AttnArgs& a, int cta, int slot, int mt_rows) {
    return a.part + (static_cast<int64_t>(cta) * 2 + slot) * mt_rows * (a.c.D + 1);
}

// desc[2 i] = the unit that CTA i's part begins within, if CTA i is the first
// to go on with it: (b, h, mt, first CTA); the last CTA in desc[2 i + 1].  One
// thread writes it, from a walk that has just started.
template <int MT, int BN> __device__ __forceinline__ void write_desc(const AttnArgs& a, const Part& p, const Walk<MT, BN>& w) {
    const int i = blockIdx.x;
    int4 d = make_int4(-1, 0, 0, 0);
    if (w.left > 0 && w.rest > 0) {
        const int64_t first = p.begin - w.rest;
        const int owner = part_owner(p.total, p.ctas, first);
        const int tiles = tiles_of<BN>(tile_len<MT>(a, w.cut, w.mt));
        if (owner == i - 1) d = make_int4(w.b, w.h, w.mt, owner);
        a.desc[2 * i + 1] = make_int4(part_owner(p.total, p.ctas, first + tiles - 1), 0, 0, 0);
    }
    a.desc[2 * i] = d;
}

template <bool F16> __device__ __forceinline__ uint32_t pack2(float x, float y) {   // x in the low half
    uint32_t r;
    if constexpr (F16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    return r;
}

}  // namespace attn

// mma.sync kernels for head dimensions up to 64, 128 and 256 (a.ctas, a.part
// and a.desc set by the launcher); `rows`: query rows per kv head.
cudaError_t launch_attn_mma64(const AttnArgs& a, bool f16, bool e4m3, int rows, int nsm, cudaStream_t s);
cudaError_t launch_attn_mma128(const AttnArgs& a, bool f16, bool e4m3, int rows, int nsm, cudaStream_t s);
cudaError_t launch_attn_mma256(const AttnArgs& a, bool f16, bool e4m3, int rows, int nsm, cudaStream_t s);
// tcgen05 kernel, and whether it takes this head dimension and page size.
bool attn_tc_takes(const AttnArgs& a);
cudaError_t launch_attn_tc(const AttnArgs& a, bool f16, bool e4m3, int nsm, cudaStream_t s);
// Joins the partial results of the kernel just launched with row tiles of MT.
cudaError_t launch_attn_combine(const AttnArgs& a, bool f16, int MT, cudaStream_t s);

}  // namespace sdv
