// k8_attn.cuh -- what the tree-attention kernels share: how the work is cut,
// where partial results go, visibility.
//
// A unit is (sequence b, kv head h, row tile mt): MT of the N * g query rows
// that read kv head h (row = node * g + head within the group), against all
// positions that the tile's nodes can see, BN positions at a time.  Units are
// numbered b outermost, mt innermost.
//
// Where several row tiles read the same keys and values (mts > 1), CTA i first
// takes units i, i + n, i + 2 n, ... for `rounds` rounds, so that the row tiles
// of one head run side by side and its keys and values come from HBM once (all
// heads at once would not fit the L2: 784 us against 869 us on 16 trees of 513
// nodes and some 200 MB of cache, 232 against 260 us on 3 chunks of 1900 tokens).  The key tiles of the other units (of all, where
// there is one row tile) form one line, cut into one part per CTA, longer for
// those whose rounds were shorter: ragged lengths need no tuning.  A unit cut
// by the end of a part gives partial results, one per CTA: normalised fp32
// outputs and the base-2 log of their sum, joined by combine_kernel.  A CTA has
// at most two: a unit begun before it (slot 0) and one that goes on after it
// (slot 1).
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

// Positions, from the first on, that every row of the tile sees (if it has any).
template <int MT> __device__ __forceinline__ int seen_by_all(const AttnArgs& a, const Cut& c, int mt) {
    return a.mask ? c.ctx : c.ctx + mt * MT / a.g + 1;
}

template <int BN> __device__ __forceinline__ int tiles_of(int len) {
    return len > 0 ? (len + BN - 1) / BN : 1;       // an empty unit still writes its rows
}

// Tiles of the first mts row tiles of one head of a causal chain: a tile's last
// node, (mt * MT + MT - 1) / g, is carried along rather than divided for.
template <int MT, int BN> __device__ __forceinline__ int64_t chain_tiles(const AttnArgs& a, const Cut& c, int mts) {
    const int dq = MT / a.g, dr = MT - dq * a.g;
    int first = 0, fr = 0;                           // the tile's first node, and its row's head
    int64_t n = 0;
    for (int mt = 0; mt < mts; ++mt) {
        int next = first + dq, nr = fr + dr;
        if (nr >= a.g) nr -= a.g, ++next;
        const int last = nr == 0 ? next - 1 : next;
        n += first >= c.cnt ? 1 : tiles_of<BN>(c.ctx + min(c.cnt, last + 1));
        first = next, fr = nr;
    }
    return n;
}

// Tiles of all row tiles of one head of a sequence.
template <int MT, int BN>
__device__ __forceinline__ int64_t head_tiles(const AttnArgs& a, const Cut& c, int mts) {
    if (a.mask) {
        const int live = min(mts, (c.cnt * a.g + MT - 1) / MT);
        return static_cast<int64_t>(live) * tiles_of<BN>(c.ctx + c.cnt) + (mts - live);
    }
    return chain_tiles<MT, BN>(a, c, mts);
}

// a / b of numbers that are not negative: 64 bits only where they are needed.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return (a | b) >> 32 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

struct Part {                // a CTA's part of the line
    int64_t begin, end;      // tiles, counted from the line's first unit
    int64_t total;
    int64_t each;            // (total - ctas) / ctas, and what is left of it
    int rest;
    int ctas;                // CTAs that have a part
    int b;                   // sequence of `begin`, and where its first unit would be
    int64_t seq0;
    const int64_t* begins;   // rounds > 0: every CTA's begin (valid until shared memory is reused)
};

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// How many of the units j .. (all heads, of a sequence) are row tile mt's.
__device__ __forceinline__ int units_from(int heads, int mts, int j, int mt) {
    return heads - (j > mt ? (j - mt + mts - 1) / mts : 0);
}

// Tiles of row tile mt of a sequence.
template <int MT, int BN> __device__ __forceinline__ int unit_tiles(const AttnArgs& a, const Cut& c, int mt) {
    return tiles_of<BN>(tile_len<MT>(a, c, mt));
}

// Where CTA i's part begins: every CTA has a tile at least.
__device__ __forceinline__ int64_t part_begin(const Part& p, int i) {
    if (p.begins) return p.begins[i];
    return i + p.each * i + static_cast<uint32_t>(p.rest) * static_cast<uint32_t>(i) / static_cast<uint32_t>(p.ctas);
}

// Every thread of the CTA calls this; `sm` holds 48 + 3 * ctas int64.
template <int MT, int BN, int THREADS>
__device__ __forceinline__ Part find_part(const AttnArgs& a, int mts, int64_t* sm) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per_seq = a.c.H * mts, n = a.ctas;
    const int first = a.rounds * n;                  // the line's first unit
    const int b0 = first / per_seq, j0 = first - b0 * per_seq;
    int64_t* begins = sm + 48;
    int64_t* done = begins + n + 1;
    if (a.rounds > 0)
        for (int i = tid; i < n; i += THREADS) done[i] = 0;
    // a thread takes row tiles of the line's sequences
    int64_t mine = 0;
    const int64_t pairs = static_cast<int64_t>(a.B - b0) * mts;
    for (int64_t i = tid; i < pairs; i += THREADS) {
        const int b = static_cast<int>(quotient(i, mts)), mt = static_cast<int>(i - static_cast<int64_t>(b) * mts);
        mine += static_cast<int64_t>(unit_tiles<MT, BN>(a, cut_of(a, b0 + b), mt)) * units_from(a.c.H, mts, b == 0 ? j0 : 0, mt);
    }
    mine = warp_sum(mine);
    if (lane == 0) sm[warp] = mine;
    if (a.rounds > 0) {
        __syncthreads();
        for (int j = tid; j < first; j += THREADS) { // the tiles of each CTA's rounds
            const int b = j / per_seq;
            const int tiles = unit_tiles<MT, BN>(a, cut_of(a, b), (j - b * per_seq) % mts);
            atomicAdd(reinterpret_cast<unsigned long long*>(done + j % n), static_cast<unsigned long long>(tiles));
        }
    }
    __syncthreads();
    Part p;
    p.total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) p.total += sm[w];
    p.ctas = static_cast<int>(p.total < n ? p.total : n);
    p.begins = nullptr;
    p.each = quotient(p.total - p.ctas, p.ctas > 0 ? p.ctas : 1);
    p.rest = static_cast<int>(p.total - p.ctas - p.each * p.ctas);
    if (a.rounds > 0) {
        // shares of the line: what a CTA's rounds lack of the mean
        if (warp == 0) {
            int64_t sum = 0;
            for (int i = lane; i < n; i += 32) sum += done[i];
            sum = warp_sum(sum);
            const int64_t mean = quotient(sum + p.total, n) + 1;
            int64_t base = 0;
            for (int i0 = 0; i0 < p.ctas; i0 += 32) {
                const int i = i0 + lane;
                const int64_t w = i < p.ctas ? (mean > done[i] ? mean - done[i] : 0) : 0;
                int64_t upto = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += x;
                }
                if (i < p.ctas) begins[i] = base + upto - w;
                base += __shfl_sync(0xffffffffu, upto, 31);
            }
            __syncwarp();
            for (int i = lane; i <= p.ctas; i += 32)
                begins[i] = i == p.ctas ? p.total
                                        : i + (base > 0 ? static_cast<int64_t>(static_cast<double>(p.total - p.ctas) * begins[i] / base) : 0);
        }
        p.begins = begins;
        __syncthreads();
    }
    const int i = blockIdx.x;
    p.b = a.B;
    if (i >= p.ctas) {
        p.begin = p.end = p.seq0 = p.total;
        return p;
    }
    p.begin = part_begin(p, i);
    p.end = i + 1 == p.ctas ? p.total : part_begin(p, i + 1);
    if (warp == 0) {
        int64_t base = 0;                            // tiles of sequence b0 that come before the line
        if (j0 > 0 && b0 < a.B)
            for (int mt = lane; mt < mts; mt += 32)
                base -= static_cast<int64_t>(unit_tiles<MT, BN>(a, cut_of(a, b0), mt)) * (a.c.H - units_from(a.c.H, mts, j0, mt));
        base = warp_sum(base);
        for (int bb = b0; bb < a.B; bb += 32) {
            const int b = bb + lane;
            const int64_t n_b = b < a.B ? head_tiles<MT, BN>(a, cut_of(a, b), mts) * a.c.H : 0;
            int64_t upto = n_b;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            const bool here = b < a.B && base + upto > p.begin && base + upto - n_b <= p.begin;
            if (here) sm[32] = b, sm[33] = base + upto - n_b;
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

// Walks a CTA's units: those of its rounds, then those of its part, of which the
// first is found by division and the others follow one another.  Whole warps
// begin together; what goes on from a copy may be a single thread.
template <int MT, int BN> struct Walk {
    int round;               // the next one
    int left, rest;          // tiles left of the part; tiles of the unit before it
    int b, h, mt;
    Cut cut;
    __device__ __forceinline__ void begin(const AttnArgs& a, const Part& p, int mts) {
        round = 0;
        left = static_cast<int>(p.end - p.begin);
        rest = 0;
        b = p.b;
        h = mt = 0;
        if (b >= a.B) return;
        cut = cut_of(a, b);
        const int lane = threadIdx.x & 31;
        const int64_t in_seq = p.begin - p.seq0;
        if (a.mask) {
            const int64_t per_head = head_tiles<MT, BN>(a, cut, mts);
            h = static_cast<int>(quotient(in_seq, per_head));
            int64_t before = in_seq - h * per_head;
            const int t = tiles_of<BN>(cut.ctx + cut.cnt);
            const int live = min(mts, (cut.cnt * a.g + MT - 1) / MT);
            if (before < static_cast<int64_t>(live) * t) {
                mt = static_cast<int>(quotient(before, t));
                before -= static_cast<int64_t>(mt) * t;
            } else {
                mt = live + static_cast<int>(before - static_cast<int64_t>(live) * t);
                before = 0;
            }
            rest = static_cast<int>(before);
        } else {
            // a lane to a row tile, 32 at a time
            int64_t per_head = 0;
            for (int i = lane; i < mts; i += 32) per_head += unit_tiles<MT, BN>(a, cut, i);
            per_head = warp_sum(per_head);
            h = static_cast<int>(quotient(in_seq, per_head));
            int64_t before = in_seq - h * per_head;
            for (int i0 = 0; i0 < mts; i0 += 32) {
                const int own = i0 + lane < mts ? unit_tiles<MT, BN>(a, cut, i0 + lane) : 0;
                int upto = own;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += x;
                }
                const uint32_t past = __ballot_sync(0xffffffffu, upto > before);
                if (past) {
                    const int at = __ffs(past) - 1;
                    mt = i0 + at;
                    rest = static_cast<int>(before - __shfl_sync(0xffffffffu, upto - own, at));
                    break;
                }
                before -= __shfl_sync(0xffffffffu, upto, 31);
            }
        }
    }
    __device__ __forceinline__ bool next(const AttnArgs& a, const Part& p, int mts, Unit& u) {
        if (round < a.rounds) {
            const int j = blockIdx.x + round * a.ctas, per_seq = a.c.H * mts;
            u.b = j / per_seq;
            u.h = (j - u.b * per_seq) / mts;
            u.mt = (j - u.b * per_seq) - u.h * mts;
            u.cut = cut_of(a, u.b);
            u.len = tile_len<MT>(a, u.cut, u.mt);
            u.t0 = 0;
            u.t1 = tiles_of<BN>(u.len);
            u.whole = true;
            ++round;
            return true;
        }
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
// thread writes it.
template <int MT, int BN>
__device__ __forceinline__ void write_desc(const AttnArgs& a, const Part& p, const Walk<MT, BN>& w) {    // w: begun, not gone on
    const int i = blockIdx.x;
    int4 d = make_int4(-1, 0, 0, 0);
    if (w.left > 0 && w.rest > 0) {
        const int64_t first = p.begin - w.rest, end = first + tiles_of<BN>(tile_len<MT>(a, w.cut, w.mt));
        if (part_begin(p, i - 1) <= first) d = make_int4(w.b, w.h, w.mt, i - 1);
        int last = i;
        while (last + 1 < p.ctas && part_begin(p, last + 1) < end) ++last;
        a.desc[2 * i + 1] = make_int4(last, 0, 0, 0);
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
// Kernels whose tiles come by tile copies, for few rows per kv head and for
// many (tcgen05), and whether they take this head dimension and page size.
bool attn_tma_takes(const AttnArgs& a);
cudaError_t launch_attn_dec(const AttnArgs& a, bool f16, bool e4m3, int nsm, cudaStream_t s);
cudaError_t launch_attn_tc(const AttnArgs& a, bool f16, bool e4m3, int nsm, cudaStream_t s);
// After launch_attn_tc with fp16 queries on an e4m3 cache: does the call again, in
// units of 16 rows, if a block has met rows that fp16 does not hold (a.beyond);
// otherwise its blocks end at once, 3 us later.  8 trees of 65 nodes behind 4000
// positions, 8 x 8 heads of 128: 258 us, and 754 us with such a row in each.
cudaError_t launch_attn_redo(const AttnArgs& a, int nsm, cudaStream_t s);
// Joins the partial results of the kernel just launched with row tiles of MT.
cudaError_t launch_attn_combine(const AttnArgs& a, bool f16, int MT, cudaStream_t s);

}  // namespace sdv
