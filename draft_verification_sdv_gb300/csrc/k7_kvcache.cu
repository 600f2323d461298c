// k7_kvcache.cu -- the paged cache: writing new keys and values (quantising
// them on the way), reading them back, and keeping the accepted path's.
//
// An e4m3 row (one position, one head) is held in units of a power of two of
// its own, so both directions are exact but for the one rounding to e4m3: the
// product by a power of two rounds nothing, neither here nor where attention
// takes the row back to 16 bits.  Against a free scale (largest value at 448) a
// row loses at most one binade of e4m3's range at its small end and none of its
// relative precision.
//
// Bound by HBM: each row is read once and written once.  D / 8 lanes (the next
// power of two of them) hold a row, eight elements each (half as many, sixteen
// each, where many rows are quantised), find its largest magnitude with shuffles and write it back.  A CTA covers the heads of a few
// positions, so that its reads of one position's heads are contiguous.  8 prompts
// of up to 4099 positions, 8 heads of 128, to e4m3: 37 us, 4.5 TB/s; 2000 positions of
// each read back: 23 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sdv_layer.h"
#include "sdv_plan.h"

namespace sdv {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float pow2f(int e) {        // 2^e, -126 <= e <= 127
    return __int_as_float((e + 127) << 23);
}

template <int TYPE> __device__ __forceinline__ void widen(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f;
        if constexpr (TYPE == kTypeBf16) {
            f = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
            f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        }
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <int TYPE> __device__ __forceinline__ uint32_t narrow2(float x, float y) {
    if constexpr (TYPE == kTypeBf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// Eight consecutive 16-bit elements, with or without 16-byte alignment.
template <bool VEC> __device__ __forceinline__ uint4 load8(const unsigned char* p) {
    if constexpr (VEC) {
        return __ldcs(reinterpret_cast<const uint4*>(p));
    } else {
        const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = h[2 * i] | (static_cast<uint32_t>(h[2 * i + 1]) << 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// A thread's work: R positions from n on, one head of the keys or the values.
struct Rows {
    int b, n, h, cnt, start;
    bool isv, live;
};

// Item w of the grid: (b, block of R positions, k or v, h), heads fastest.
template <int R> __device__ __forceinline__ Rows rows_of(const CellsArgs& a, int64_t w) {
    Rows r;
    const unsigned hv = 2u * a.c.H, blocks = static_cast<unsigned>((a.N + R - 1) / R);
    const int64_t all = static_cast<int64_t>(a.B) * blocks * hv;
    r.live = w < all;
    if (!r.live) w = 0;
    int x;
    if (all >> 32 == 0) {                           // divisions of 64 bits only where they are needed
        const unsigned bn = static_cast<unsigned>(w) / hv;
        x = static_cast<int>(static_cast<unsigned>(w) - bn * hv);
        r.b = static_cast<int>(bn / blocks);
        r.n = static_cast<int>(bn - static_cast<unsigned>(r.b) * blocks) * R;
    } else {
        const unsigned long long bn = static_cast<unsigned long long>(w) / hv;
        x = static_cast<int>(static_cast<unsigned long long>(w) - bn * hv);
        r.b = static_cast<int>(bn / blocks);
        r.n = static_cast<int>(bn - static_cast<unsigned long long>(r.b) * blocks) * R;
    }
    r.isv = x >= a.c.H;
    r.h = r.isv ? x - a.c.H : x;
    r.cnt = a.count ? __ldg(a.count + r.b) : a.N;
    r.start = __ldg(a.start + r.b);
    return r;
}

// Where position n of the item sits: its page (or -1, with the status set, or
// -2: there is no such row) and its row within the page.
__device__ __forceinline__ int place_of(const CellsArgs& a, const Rows& r, int n, int64_t* cell, unsigned* st) {
    if (!r.live || n >= a.N) return -2;
    if (r.cnt < 0 || r.cnt > a.N) {
        *st |= kStatusBadLength;
        return -1;
    }
    if (n >= r.cnt) return -2;
    const int64_t pos = static_cast<int64_t>(r.start) + n;
    if (pos < 0 || pos >= static_cast<int64_t>(a.max_pages) * a.c.P) {
        *st |= kStatusBadLength;
        return -1;
    }
    const int p = static_cast<int>(pos), i = p / a.c.P;          // at most 2^30 positions
    *cell = static_cast<int64_t>(r.h) * a.c.P + (p - i * a.c.P);
    const int page = __ldg(a.table + static_cast<int64_t>(r.b) * a.max_pages + i);
    if (page < 0 || page >= a.c.pages) {
        *st |= kStatusBadPage;
        return -1;
    }
    return page;
}

// The places of an item's R rows, one lane of it looking up each; the status is
// set for those that have none.
template <int LANES, int R>
__device__ __forceinline__ void places_of(const CellsArgs& a, const Rows& r, int lane, int (&page)[R], int64_t (&cell)[R]) {
    unsigned st = 0;
    int64_t c = 0;
    const int p = lane < R ? place_of(a, r, r.n + lane, &c, &st) : -2;
    if (st && a.status) atomicOr(a.status, st);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        page[i] = __shfl_sync(0xffffffffu, p, i, LANES);
        cell[i] = __shfl_sync(0xffffffffu, static_cast<int>(c), i, LANES);      // rows of a page: fewer than 2^30
    }
}

// U: vectors of eight values of a row that a lane has, LANES apart.
template <int TYPE, bool E4M3, bool VEC, int LANES, int R, int U>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const CellsArgs a) {
    const int lane = threadIdx.x % LANES;
    const Rows r = rows_of<R>(a, (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / LANES);
    const unsigned char* src = (r.isv ? a.v + r.b * a.v_sb + r.h * a.v_sh : a.k + r.b * a.k_sb + r.h * a.k_sh) + lane * 16;
    const int64_t sn = r.isv ? a.v_sn : a.k_sn;
    uint4 x[R][U];
#pragma unroll
    for (int i = 0; i < R; ++i)                     // whatever becomes of a row, it may be read
#pragma unroll
        for (int u = 0; u < U; ++u)
            x[i][u] = r.live && (lane + u * LANES) * 8 < a.c.D && r.n + i < a.N ? load8<VEC>(src + (r.n + i) * sn + u * LANES * 16)
                                                                                : make_uint4(0, 0, 0, 0);
    int page[R];
    int64_t cell[R];
    places_of<LANES, R>(a, r, lane, page, cell);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const bool go = page[i] >= 0;
        unsigned char* dst = (r.isv ? a.c.v : a.c.k) + (go ? page[i] * a.c.page_stride : 0);
        if constexpr (!E4M3) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (go && (lane + u * LANES) * 8 < a.c.D)
                    *reinterpret_cast<uint4*>(dst + cell[i] * a.c.D * 2 + (lane + u * LANES) * 16) = x[i][u];
        } else {
            // magnitudes order as their bits do, infinities and NaN last
            unsigned top = 0;
#pragma unroll
            for (int u = 0; u < U; ++u)
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[i][u].x & 0x7fff7fffu, x[i][u].y & 0x7fff7fffu),
                                             __vmaxu2(x[i][u].z & 0x7fff7fffu, x[i][u].w & 0x7fff7fffu)));
            top = max(top >> 16, top & 0xffffu);
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const bool bad = top >= (TYPE == kTypeBf16 ? 0x7f80u : 0x7c00u);
            const unsigned bits = TYPE == kTypeBf16 ? top << 16 : __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(top))));
            // top = 1.m 2^x <= 448 2^e: e = x - 8 while 1.m <= 1.75, else x - 7
            // (a subnormal or zero top has x = -127 and ends at the floor as well)
            int e = static_cast<int>(bits >> 23) - 127 - ((bits & 0x7fffff) <= 0x600000 ? 8 : 7);
            e = bad ? 0 : e < -126 ? -126 : e;
            const float inv = pow2f(-e);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[8];
                widen<TYPE>(x[i][u], f);
                uint32_t o[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
                        make_float2(f[4 * y] * inv, f[4 * y + 1] * inv), __NV_SATFINITE, __NV_E4M3);
                    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
                        make_float2(f[4 * y + 2] * inv, f[4 * y + 3] * inv), __NV_SATFINITE, __NV_E4M3);
                    o[y] = bad ? 0x7f7f7f7fu : static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
                }
                if (go && (lane + u * LANES) * 8 < a.c.D)
                    *reinterpret_cast<uint2*>(dst + cell[i] * a.c.D + (lane + u * LANES) * 8) = make_uint2(o[0], o[1]);
            }
            if (go && lane == 0)
                (r.isv ? a.c.ve : a.c.ke)[page[i] * a.c.exp_page_stride + cell[i]] = static_cast<unsigned char>(bad ? 255 : e + 127);
        }
    }
}

template <int TYPE, bool E4M3, int LANES, int R>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const CellsArgs a) {
    const int lane = threadIdx.x % LANES;
    const Rows r = rows_of<R>(a, (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / LANES);
    int page[R], ex[R];
    int64_t cell[R];
    places_of<LANES, R>(a, r, lane, page, cell);
    if (!r.live || lane * 8 >= a.c.D) return;
    uint4 x[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        ex[i] = 127;
        x[i] = make_uint4(0, 0, 0, 0);
        if (page[i] >= 0) {
            const unsigned char* src = (r.isv ? a.c.v : a.c.k) + page[i] * a.c.page_stride;
            if constexpr (E4M3) {
                const uint2 q = __ldcs(reinterpret_cast<const uint2*>(src + cell[i] * a.c.D + lane * 8));
                x[i].x = q.x, x[i].y = q.y;
                ex[i] = __ldg((r.isv ? a.c.ve : a.c.ke) + page[i] * a.c.exp_page_stride + cell[i]);
            } else {
                x[i] = __ldcs(reinterpret_cast<const uint4*>(src + cell[i] * a.c.D * 2 + lane * 16));
            }
        }
    }
    unsigned char* dst = static_cast<unsigned char*>(r.isv ? a.ov : a.ok);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (r.n + i >= a.N) break;
        uint4 o = x[i];
        if (page[i] == -1) {
            o = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);   // NaN in either type
        } else if constexpr (E4M3) {
            // 2^(ex - 127) (0 stands for 2^-127, a subnormal), 255: not a number
            const float unit = ex[i] == 255 ? __int_as_float(0x7fc00000)
                               : ex[i] == 0 ? __int_as_float(0x00400000) : __int_as_float(ex[i] << 23);
            const uint32_t w[2] = {x[i].x, x[i].y};
            uint32_t out[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                    static_cast<__nv_fp8x2_storage_t>(w[y / 2] >> (16 * (y % 2))), __NV_E4M3);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
                out[y] = narrow2<TYPE>(f.x * unit, f.y * unit);
            }
            o = make_uint4(out[0], out[1], out[2], out[3]);
        }
        const int64_t row = (static_cast<int64_t>(r.b) * a.N + r.n + i) * a.c.H + r.h;
        __stcs(reinterpret_cast<uint4*>(dst + row * a.c.D * 2 + lane * 16), o);
    }
}

// One CTA per sequence; a thread moves one piece of a row (or one exponent) of
// every accepted token, in the path's order.  Nodes grow along the path from 1
// on, so token j' sits at place j' + 1 or later: its cell is read before the
// moves overwrite it, and within a thread nothing is reordered.
__global__ void __launch_bounds__(kThreads) kv_commit_kernel(const CommitArgs a) {
    const int b = blockIdx.x;
    const int start = a.start[b], sel = a.sel[b], acc = a.acc[b];
    const int64_t places = static_cast<int64_t>(a.max_pages) * a.c.P;
    __shared__ unsigned s_bad;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    const bool skip = sel == -1;
    const bool ok = !skip && sel >= 0 && sel < a.K && acc >= 0 && acc <= a.G && start >= 0 &&
                    start + static_cast<int64_t>(acc) < places;
    if (ok) {
        const int32_t* path = a.nodes + (static_cast<int64_t>(b) * a.K + sel) * a.G;
        const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_pages;
        const int piece = a.cell == 1 ? 8 : 16;            // bytes a thread moves at a time
        const int per_row = a.c.D * a.cell / piece;
        const int pieces = 2 * a.c.H * per_row, exps = a.cell == 1 ? 2 * a.c.H : 0;
        for (int w = threadIdx.x; w < pieces + exps; w += kThreads) {
            const bool isx = w >= pieces;
            const int x = isx ? w - pieces : w / per_row;
            const int off = isx ? 0 : (w % per_row) * piece;
            const bool isv = x >= a.c.H;
            const int h = isv ? x - a.c.H : x;
            unsigned char* base = isx ? (isv ? a.c.ve : a.c.ke) : (isv ? a.c.v : a.c.k);
            const int64_t stride = isx ? a.c.exp_page_stride : a.c.page_stride;
            const int row_bytes = isx ? 1 : a.c.D * a.cell;
            int last = 0;
            for (int j = 0; j < acc; ++j) {
                const int node = path[j];
                const int64_t from = static_cast<int64_t>(start) + node, to = static_cast<int64_t>(start) + 1 + j;
                if (node <= last || from >= places) {      // not a path of this tree
                    atomicOr(&s_bad, kStatusBadLength);
                    break;
                }
                last = node;
                const int pf = table[from / a.c.P], pt = table[to / a.c.P];
                if (pf < 0 || pf >= a.c.pages || pt < 0 || pt >= a.c.pages) {
                    atomicOr(&s_bad, kStatusBadPage);
                    break;
                }
                if (from == to) continue;
                const unsigned char* src = base + pf * stride + (static_cast<int64_t>(h) * a.c.P + from % a.c.P) * row_bytes + off;
                unsigned char* dst = base + pt * stride + (static_cast<int64_t>(h) * a.c.P + to % a.c.P) * row_bytes + off;
                if (isx)
                    *dst = *src;
                else if (a.cell == 1)
                    *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(src);
                else
                    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        const unsigned st = ok ? s_bad : skip ? 0u : static_cast<unsigned>(kStatusBadLength);
        if (st && a.status) atomicOr(a.status, st);
        if (a.out_len) a.out_len[b] = ok && !st ? start + 1 + acc : start;
    }
}

// Positions a thread takes: several where there are many, for loads in flight.
// Four against one: 64 x 65 bf16 positions of 8 heads of 128 written in 10.2 and
// 14.3 us, 64 x 32 in 8.2 and 10.2; 64 x 16 the same, 64 x 8 to e4m3 read in 10.2
// and 8.2 us.
constexpr int kMany = 4, kManyFrom = 32;

template <int LANES, int R> dim3 grid_of(const CellsArgs& a) {
    const int64_t items = static_cast<int64_t>(a.B) * ((a.N + R - 1) / R) * 2 * a.c.H;
    return dim3(static_cast<unsigned>((items * LANES + kThreads - 1) / kThreads));
}

template <int TYPE, bool E4M3, int LANES, int R, int U>
cudaError_t write_rows(const CellsArgs& a, bool vec, cudaStream_t s) {
    if (vec)
        kv_write_kernel<TYPE, E4M3, true, LANES, R, U><<<grid_of<LANES, R>(a), kThreads, 0, s>>>(a);
    else
        kv_write_kernel<TYPE, E4M3, false, LANES, R, U><<<grid_of<LANES, R>(a), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <int TYPE, bool E4M3, int LANES>
cudaError_t write_lanes(const CellsArgs& a, bool vec, cudaStream_t s) {
    if (a.N < kManyFrom) return write_rows<TYPE, E4M3, LANES, 1, 1>(a, vec, s);
    // quantising is bound by instructions: two vectors a lane share a row's maximum,
    // its power of two and its place (8 prompts of 4099: 37 us against 45 us)
    if constexpr (E4M3)
        return write_rows<TYPE, E4M3, LANES / 2, kMany, 2>(a, vec, s);
    else
        return write_rows<TYPE, E4M3, LANES, kMany, 1>(a, vec, s);
}

template <int TYPE, bool E4M3>
cudaError_t write_typed(const CellsArgs& a, bool vec, cudaStream_t s) {
    if (a.c.D <= 64) return write_lanes<TYPE, E4M3, 8>(a, vec, s);
    if (a.c.D <= 128) return write_lanes<TYPE, E4M3, 16>(a, vec, s);
    return write_lanes<TYPE, E4M3, 32>(a, vec, s);
}

template <int TYPE, bool E4M3, int LANES> cudaError_t read_lanes(const CellsArgs& a, cudaStream_t s) {
    if (a.N >= kManyFrom)
        kv_read_kernel<TYPE, E4M3, LANES, kMany><<<grid_of<LANES, kMany>(a), kThreads, 0, s>>>(a);
    else
        kv_read_kernel<TYPE, E4M3, LANES, 1><<<grid_of<LANES, 1>(a), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <int TYPE, bool E4M3>
cudaError_t read_typed(const CellsArgs& a, cudaStream_t s) {
    if (a.c.D <= 64) return read_lanes<TYPE, E4M3, 8>(a, s);
    if (a.c.D <= 128) return read_lanes<TYPE, E4M3, 16>(a, s);
    return read_lanes<TYPE, E4M3, 32>(a, s);
}

}  // namespace

cudaError_t launch_kv_write(const CellsArgs& a, int type, bool e4m3, bool vec, cudaStream_t s) {
    if (!e4m3) return write_typed<kTypeBf16, false>(a, vec, s);      // 16-bit cells: moved as they are
    return type == kTypeBf16 ? write_typed<kTypeBf16, true>(a, vec, s) : write_typed<kTypeF16, true>(a, vec, s);
}

cudaError_t launch_kv_read(const CellsArgs& a, int type, bool e4m3, cudaStream_t s) {
    if (!e4m3) return read_typed<kTypeBf16, false>(a, s);
    return type == kTypeBf16 ? read_typed<kTypeBf16, true>(a, s) : read_typed<kTypeF16, true>(a, s);
}

cudaError_t launch_kv_commit(const CommitArgs& a, cudaStream_t s) {
    kv_commit_kernel<<<static_cast<unsigned>(a.B), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace sdv
