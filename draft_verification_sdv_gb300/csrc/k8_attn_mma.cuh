// k8_attn_mma.cuh -- tree attention for head dimensions above 128 and for pages
// of any size (sdv_tree_attn), where the kernels that load by tile copies do not
// go; one translation unit per head dimension includes this.
//
// A tile of BN positions may begin and end anywhere in a page, so its rows come
// in by 16-byte asynchronous copies, each with an address of its own, several
// tiles ahead, swizzled so that the fragments are read without bank conflicts.
// The contractions run on mma.sync m16n8k16, whose 16 rows waste less on 8 query
// heads than a 128-row instruction would.  For few rows the cache's bytes and
// the copies' instructions bound it (32 sequences of 4000 positions, 8 kv heads,
// 8 rows each: heads of 256, 321 us, 3.3 TB/s; heads of 128 on pages of 12, 128
// us, 4.1 TB/s), for many the matrix instructions.
//
// MT = 16 WM rows; the WN = 4 / WM warps that share rows split each tile's
// positions and keep their own running maximum, sum and output, which are
// joined at the end of the unit.
//
// e4m3 cells stay 8 bits wide in shared memory and are widened to fp16 (exact)
// as fragments are read.  The order of the contraction's index is free, so a
// lane takes 16 consecutive cells of a key row as its share of four
// instructions, and four consecutive cells of each of four value rows as its
// share of four output columns, transposed by byte permutes.  The rows' powers
// of two stay out of the products: a key's multiplies its score; a value's is
// added to the exponent, x' = x + e_v, with a running maximum of x' for the
// outputs beside the one of x for the sum, so that neither can overflow.  These
// weights of the values have digits down to 2^-14, and some down to 2^-25, so the
// largest so far is 2^14: a row of values up to 2^-28 of the largest in probability
// times power counts with all its digits, one below 2^-39 not at all.  bf16 queries
// are brought to fp16 in units of a power of two per row.
#pragma once

#include "k8_attn.cuh"

namespace sdv {
namespace {

using namespace attn;

constexpr int kThreads = 128;
constexpr float kUp = 14.0f;             // e4m3: log2 of the largest weight of a value

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&x)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}
// Two e4m3 cells (the low 16 bits) as two fp16, exactly.
__device__ __forceinline__ uint32_t widen2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr) : "memory");
    return r;
}

template <int DP, bool E4> struct Shape {
    static constexpr int ROW = DP * (E4 ? 1 : 2);               // bytes of a cell row
    static constexpr int BN = DP == 256 || ROW == 256 ? 64 : 128;   // positions of a tile
    static constexpr int TILE = BN * ROW;
    static constexpr int FIT = 96 * 1024 / (2 * TILE);          // two CTAs per SM
    static constexpr int STAGES = FIT > 4 ? 4 : FIT < 2 ? 2 : FIT;
};

// Byte offset of 16-byte chunk c of row r in a tile.
template <int ROW, bool E4, bool VALUE> __device__ __forceinline__ int chunk_at(int r, int c) {
    constexpr int N = ROW / 16;
    if constexpr (!E4)
        c ^= r & 7;
    else if constexpr (VALUE)
        c ^= (((r >> 1) & 3) << 1) & (N - 1);
    else
        c ^= ((r & 1) << 2) & (N - 1);
    return r * ROW + c * 16;
}

// Shared memory of a CTA, in bytes from its start.
template <int DP, bool E4, int WM> struct Layout {
    using S = Shape<DP, E4>;
    static constexpr int MT = 16 * WM;
    static constexpr int tiles = S::STAGES * 2 * S::TILE, join = 4 * 16 * DP * 4;
    static constexpr int q = tiles > join ? tiles : join;       // the join's outputs lie over the tiles
    static constexpr int off = q + MT * DP * 2;                 // int64 [2][BN] page of a row
    static constexpr int cell = off + 2 * S::BN * 8;            // int [2][BN] row within its page (< 0: none)
    static constexpr int ke = cell + 2 * S::BN * 4;             // float [STAGES][BN] keys' powers of two
    static constexpr int ve = ke + (E4 ? S::STAGES * S::BN * 4 : 0);    // float [STAGES][BN] values' exponents
    static constexpr int qe = ve + (E4 ? S::STAGES * S::BN * 4 : 0);    // float [MT] the rows' score factors
    static constexpr int any = qe + MT * 4;                     // int [STAGES] 1 + the last tile here with a flagged column
    static constexpr int flag = any + S::STAGES * 4;            // bytes [STAGES][BN] the column is not a number
    static constexpr int bytes = (flag + S::STAGES * S::BN + 15) / 16 * 16;
};

template <int DP, bool E4, bool F16, int WM>
__global__ void __launch_bounds__(kThreads) attn_mma_kernel(const AttnArgs a) {
    using S = Shape<DP, E4>;
    using L = Layout<DP, E4, WM>;
    constexpr int WN = 4 / WM, MT = 16 * WM, BN = S::BN, NW = BN / WN, NT = NW / 8;
    constexpr int STAGES = S::STAGES, ROW = S::ROW, TILE = S::TILE, CH = ROW / 16;
    constexpr int CELL = E4 ? 1 : 2;
    constexpr bool M16 = F16 || E4;                 // the products' type is fp16
    static_assert(NT % 2 == 0 && BN <= kThreads, "a warp takes pairs of column tiles, a thread one row");
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* s_kv = smem;                                  // [STAGES][K, V] tiles
    unsigned char* s_q = smem + L::q;                            // [MT][DP] 16-bit, swizzled
    int64_t* s_off = reinterpret_cast<int64_t*>(smem + L::off);
    int* s_cell = reinterpret_cast<int*>(smem + L::cell);
    float* s_ke = reinterpret_cast<float*>(smem + L::ke);
    float* s_ve = reinterpret_cast<float*>(smem + L::ve);
    float* s_qe = reinterpret_cast<float*>(smem + L::qe);
    int* s_any = reinterpret_cast<int*>(smem + L::any);
    unsigned char* s_flag = smem + L::flag;
    __shared__ int64_t s_part[40];
    __shared__ float s_m[4][16], s_l[4][16];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wm = warp / WN, wn = warp % WN;
    const int g4 = lane >> 2, t4 = lane & 3;
    const int mts = (a.N * a.g + MT - 1) / MT;
    const Part part = find_part<MT, BN, kThreads>(a, mts, s_part);

    Walk<MT, BN> walk;
    walk.begin(a, part, mts);
    if (tid == 0) write_desc(a, part, walk);
    Unit u;
    while (walk.next(a, part, mts, u)) {
        __syncthreads();                            // the unit before is done with shared memory
        if (tid == 0 && u.cut.bad && a.status) atomicOr(a.status, kStatusBadLength);
        const int32_t* table = a.table + static_cast<int64_t>(u.b) * a.max_pages;
        const int nt = u.len > 0 ? u.t1 - u.t0 : 0;

        // ---- queries: MT rows into shared memory ----
        for (int w = tid; w < MT * (DP / 8); w += kThreads) {
            const int r = w / (DP / 8), c = w % (DP / 8);
            const int row = u.mt * MT + r, node = row / a.g;
            uint32_t v[4] = {0, 0, 0, 0};
            if (node < u.cut.cnt && c * 8 < a.c.D) {
                const unsigned char* p = q_of(a, u.b, node) + (static_cast<int64_t>(u.h) * a.g + row % a.g) * a.q_sh + c * 16;
                if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
                    const uint4 x = *reinterpret_cast<const uint4*>(p);
                    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
                } else {
                    const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = h[2 * i] | (static_cast<uint32_t>(h[2 * i + 1]) << 16);
                }
            }
            if constexpr (E4 && !F16) {             // bf16 to fp16 in units of a power of two per row
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top = fmaxf(top, fmaxf(fabsf(bf16_lo(v[i])), fabsf(bf16_hi(v[i]))));
#pragma unroll
                for (int o = DP / 16; o > 0; o >>= 1)   // the DP / 8 lanes of a row
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                int e = (__float_as_int(top) >> 23) - 127 - 14;  // the largest ends in [2^14, 2^15)
                e = e < -126 ? -126 : e;
                const float inv = __int_as_float((127 - e) << 23);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = pack2<true>(bf16_lo(v[i]) * inv, bf16_hi(v[i]) * inv);
                if (c == 0) s_qe[r] = __int_as_float((e + 127) << 23) * a.scale_log2;
            } else if (c == 0) {
                s_qe[r] = a.scale_log2;
            }
            if constexpr (E4) {
                // cell d = 64 x + 16 t + 4 s + e is element 2 t + (e & 1) + 8 (e >> 1) of step 4 x + s
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = c * 8 + 2 * i, t = d >> 4 & 3, s = d >> 2 & 3, hi = d >> 1 & 1;
                    const int to = (d & ~63) + s * 16 + 2 * t + 8 * hi;
                    *reinterpret_cast<uint32_t*>(s_q + r * DP * 2 + (((to >> 3) ^ (r & 7)) << 4) + (to & 7) * 2) = v[i];
                }
            } else {
                *reinterpret_cast<uint4*>(s_q + r * DP * 2 + ((c ^ (r & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
            }
        }

        // ---- loading, a thread per row: its page is asked for (fetch) one step
        // before the row's place is set down (place), and the copies of a tile
        // (load) begin after that; the exponents that load asks for are set down
        // (settle) a step later.  No step waits for its own reads.
        int page = 0, ke = 127, ve = 127, cell_now = -1;
        auto fetch = [&](int t) {                   // tile t of this CTA's part of the unit
            const int pos = (u.t0 + t) * BN + tid;
            page = tid < BN && t < nt && pos < u.len ? __ldg(table + pos / a.c.P) : -1;
        };
        auto place = [&](int t, int slot) {
            if (tid >= BN) return;
            const int pos = (u.t0 + t) * BN + tid;
            int cell = -1;                          // past the end: zeros
            if (t < nt && pos < u.len) {
                if (page >= 0 && page < a.c.pages) {
                    cell = u.h * a.c.P + pos % a.c.P;
                } else {
                    cell = -2;
                    if (a.status) atomicOr(a.status, kStatusBadPage);
                }
            }
            s_off[slot * BN + tid] = page;
            s_cell[slot * BN + tid] = cell;
        };
        auto load = [&](int t, int slot) {
            if (t < nt) {
                const uint32_t k0 = smem_u32(s_kv + (t % STAGES) * 2 * TILE), v0 = k0 + TILE;
                const int used = a.c.D * CELL / 16;
#pragma unroll 4
                for (int w = tid; w < BN * CH; w += kThreads) {
                    const int r = w / CH, c = w % CH;
                    const int cell = s_cell[slot * BN + r];
                    const bool live = cell >= 0 && c < used;
                    const int64_t o = live ? s_off[slot * BN + r] * a.c.page_stride + (static_cast<int64_t>(cell) * a.c.D * CELL + c * 16) : 0;
                    cp16(k0 + chunk_at<ROW, E4, false>(r, c), a.c.k + o, live);
                    cp16(v0 + chunk_at<ROW, E4, true>(r, c), a.c.v + o, live);
                }
                if (tid < BN) {
                    cell_now = s_cell[slot * BN + tid];
                    if constexpr (E4) {
                        ke = ve = 127;
                        if (cell_now >= 0) {
                            const int64_t o = s_off[slot * BN + tid] * a.c.exp_page_stride + cell_now;
                            ke = a.c.ke[o];
                            ve = a.c.ve[o];
                        }
                    }
                }
            }
            cp_commit();
        };
        auto settle = [&](int t) {
            if (tid >= BN || t >= nt) return;
            const int st = t % STAGES;
            bool nan = cell_now == -2;
            if constexpr (E4) {
                nan |= ke == 255 || ve == 255;
                s_ke[st * BN + tid] = ke == 0 ? __int_as_float(0x00400000) : __int_as_float(ke << 23);
                s_ve[st * BN + tid] = static_cast<float>(ve - 127);
            }
            s_flag[st * BN + tid] = nan;
            if (nan) s_any[st] = t + 1;
        };

        float o[DP / 8][4];
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, mv[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
        const int row0 = u.mt * MT + wm * 16 + g4;
        const int node[2] = {row0 / a.g, (row0 + 8) / a.g};

        if (tid < STAGES) s_any[tid] = 0;
        fetch(0);
        place(0, 0);
        fetch(1);
        __syncthreads();
        for (int t = 0; t < STAGES - 1; ++t) {
            load(t, t & 1);
            settle(t);
            place(t + 1, (t + 1) & 1);
            fetch(t + 2);
            __syncthreads();
        }
        const float rowf[2] = {s_qe[wm * 16 + g4], s_qe[wm * 16 + g4 + 8]};

        for (int t = 0; t < nt; ++t) {
            const int st = t % STAGES;
            // tile t has come in, and every warp is done with the one before it
            cp_wait<STAGES - 2>();
            settle(t + STAGES - 2);
            __syncthreads();
            load(t + STAGES - 1, (t + STAGES - 1) & 1);
            place(t + STAGES, (t + STAGES) & 1);
            fetch(t + STAGES + 1);

            const uint32_t k0 = smem_u32(s_kv + st * 2 * TILE), v0 = k0 + TILE;
            const int pos0 = (u.t0 + t) * BN;
            // columns that are nodes: some rows see them and some do not
            const bool mixed = pos0 + BN > u.cut.ctx;
            if (mixed) {                            // values that are not numbers are kept out of the products
                constexpr int TR = kThreads / BN;   // threads of a row
                const int r = tid / TR, part_c = tid % TR;
                int bad = 0;
                if (pos0 + r >= u.cut.ctx) {
                    for (int c = part_c; c < CH; c += TR) {
                        const uint4 x = lds128(v0 + chunk_at<ROW, E4, true>(r, c));
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if constexpr (E4) {
#pragma unroll
                                for (int y = 0; y < 4; ++y) bad |= (w[i] >> (8 * y) & 0x7f) == 0x7f;
                            } else {
                                constexpr uint32_t top = F16 ? 0x7c00u : 0x7f80u;
                                bad |= (w[i] & top) == top || (w[i] >> 16 & top) == top;
                            }
                        }
                    }
                }
                if constexpr (TR > 1) bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
                if (bad) {
                    for (int c = part_c; c < CH; c += TR)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v0 + chunk_at<ROW, E4, true>(r, c)), "r"(0) : "memory");
                    s_flag[st * BN + r] = 1;
                    s_any[st] = t + 1;
                }
                __syncthreads();
            }

            // ---- scores ----
            float s[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
            const uint32_t q0 = smem_u32(s_q) + (wm * 16 + (lane & 15)) * DP * 2;
            if constexpr (!E4) {
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks) {
                    uint32_t q[4];
                    ldsm4(q, q0 + (((ks * 2 + (lane >> 4)) ^ (lane & 7)) << 4));
#pragma unroll
                    for (int i = 0; i < NT; i += 2) {
                        uint32_t k[4];              // two column tiles: lane >> 4 picks one, lane >> 3 & 1 the half of the step
                        const int r = wn * NW + i * 8 + (lane >> 4) * 8 + (lane & 7);
                        ldsm4(k, k0 + chunk_at<ROW, false, false>(r, ks * 2 + (lane >> 3 & 1)));
                        mma<M16>(s[i], q, k[0], k[1]);
                        mma<M16>(s[i + 1], q, k[2], k[3]);
                    }
                }
            } else {
#pragma unroll
                for (int x = 0; x < DP / 64; ++x) {
                    uint32_t q[4][4];
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        ldsm4(q[ks], q0 + ((((x * 4 + ks) * 2 + (lane >> 4)) ^ (lane & 7)) << 4));
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const uint4 w = lds128(k0 + chunk_at<ROW, true, false>(wn * NW + i * 8 + g4, x * 4 + t4));
                        mma<true>(s[i], q[0], widen2(w.x), widen2(w.x >> 16));
                        mma<true>(s[i], q[1], widen2(w.y), widen2(w.y >> 16));
                        mma<true>(s[i], q[2], widen2(w.z), widen2(w.z >> 16));
                        mma<true>(s[i], q[3], widen2(w.w), widen2(w.w >> 16));
                    }
                }
            }

            // ---- scale, mask, running maxima ----
            const bool any = s_any[st] == t + 1;
            float top[2] = {m[0], m[1]}, topv[2] = {mv[0], mv[1]};
#pragma unroll
            for (int i = 0; i < NT; ++i) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int rr = x >> 1, col = wn * NW + i * 8 + 2 * t4 + (x & 1);
                    float v = s[i][x] * rowf[rr];
                    if constexpr (E4) v *= s_ke[st * BN + col];
                    if (any && s_flag[st * BN + col]) v = __int_as_float(0x7fc00000);
                    if (mixed) {
                        const int nm = pos0 + col - u.cut.ctx;      // which node the column is
                        bool see = pos0 + col < u.len;
                        if (see && nm >= 0) {
                            if (a.mask)
                                see = node[rr] < u.cut.cnt &&
                                      (__ldg(a.mask + u.b * a.mask_sb + static_cast<int64_t>(node[rr]) * a.W + (nm >> 5)) >> (nm & 31) & 1);
                            else
                                see = nm <= node[rr];
                        }
                        if (!see) v = -INFINITY;
                    }
                    s[i][x] = v;
                    top[rr] = fmaxf(top[rr], v);
                    if constexpr (E4) topv[rr] = fmaxf(topv[rr], v + s_ve[st * BN + col]);
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int x = 1; x < 4; x <<= 1) {
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], x));
                    if constexpr (E4) topv[r] = fmaxf(topv[r], __shfl_xor_sync(0xffffffffu, topv[r], x));
                }
                if constexpr (!E4) topv[r] = top[r];
            }
            float by[2], sub[2], subv[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                sub[r] = top[r] == -INFINITY ? 0.0f : top[r];       // nothing seen yet: 2^-inf = 0
                subv[r] = topv[r] == -INFINITY ? 0.0f : topv[r];
                l[r] *= ex2(m[r] - sub[r]);
                by[r] = ex2(mv[r] - subv[r]);
                m[r] = top[r];
                mv[r] = topv[r];
            }
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) {
                o[i][0] *= by[0], o[i][1] *= by[0];
                o[i][2] *= by[1], o[i][3] *= by[1];
            }

            // ---- probabilities (fp32 into the sum, 16 bits into the product) and outputs ----
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
                uint32_t p[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {       // registers a0..a3: column tile y >> 1, row y & 1
                    const int i = 2 * j + (y >> 1), r = y & 1;
                    const float x0 = s[i][2 * r], x1 = s[i][2 * r + 1];
                    const float e0 = ex2(x0 - sub[r]), e1 = ex2(x1 - sub[r]);
                    l[r] += e0 + e1;
                    if constexpr (E4) {
                        const float2 ev = *reinterpret_cast<const float2*>(s_ve + st * BN + wn * NW + i * 8 + 2 * t4);
                        p[y] = pack2<true>(ex2(x0 + ev.x - (subv[r] - kUp)), ex2(x1 + ev.y - (subv[r] - kUp)));
                    } else {
                        p[y] = pack2<F16>(e0, e1);
                    }
                }
                const int r0 = wn * NW + j * 16;
                if constexpr (!E4) {
#pragma unroll
                    for (int i = 0; i < DP / 8; i += 2) {
                        uint32_t v[4];              // 16 positions x 16 columns
                        ldsm4t(v, v0 + chunk_at<ROW, false, true>(r0 + (lane & 15), i + (lane >> 4)));
                        mma<M16>(o[i], p, v[0], v[1]);
                        mma<M16>(o[i + 1], p, v[2], v[3]);
                    }
                } else {
#pragma unroll
                    for (int y = 0; y < DP / 32; ++y) {
                        uint32_t w[4];              // cells 32 y + 4 g4 .. + 3 of rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int r = r0 + 2 * t4 + (x & 1) + 8 * (x >> 1);
                            w[x] = lds32(v0 + chunk_at<ROW, true, true>(r, 2 * y + (g4 >> 2)) + (g4 & 3) * 4);
                        }
                        const uint32_t lo01 = __byte_perm(w[0], w[1], 0x5140), lo23 = __byte_perm(w[0], w[1], 0x7362);
                        const uint32_t hi01 = __byte_perm(w[2], w[3], 0x5140), hi23 = __byte_perm(w[2], w[3], 0x7362);
                        mma<true>(o[4 * y + 0], p, widen2(lo01), widen2(hi01));
                        mma<true>(o[4 * y + 1], p, widen2(lo01 >> 16), widen2(hi01 >> 16));
                        mma<true>(o[4 * y + 2], p, widen2(lo23), widen2(hi23));
                        mma<true>(o[4 * y + 3], p, widen2(lo23 >> 16), widen2(hi23 >> 16));
                    }
                }
            }
        }

        // ---- the unit's rows: join the warps, write outputs or partials ----
        cp_wait<0>();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        }
        __syncthreads();
        float* s_o = reinterpret_cast<float*>(smem);        // [4 warps][16][DP]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            // the warp's own outputs in units of 2^m: o * 2^(mv - m)
            const float up = E4 ? (m[r] == -INFINITY ? 0.0f : ex2(mv[r] - kUp - m[r])) : 1.0f;
            if (t4 == 0) s_m[warp][g4 + 8 * r] = m[r], s_l[warp][g4 + 8 * r] = l[r];
            float* dst = s_o + (warp * 16 + g4 + 8 * r) * DP;
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) {
                if constexpr (E4) {
                    const int d = (i >> 2) * 32 + 8 * t4 + (i & 3);
                    dst[d] = o[i][2 * r] * up;
                    dst[d + 4] = o[i][2 * r + 1] * up;
                } else {
                    *reinterpret_cast<float2*>(dst + i * 8 + 2 * t4) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
                }
            }
        }
        __syncthreads();
        const int slot = u.t0 > 0 ? 0 : 1;
        float* prow = part_rows(a, blockIdx.x, slot, MT);
        for (int w = tid; w < MT * (DP / 4); w += kThreads) {
            const int r = w / (DP / 4), d = (w % (DP / 4)) * 4;
            const int row = u.mt * MT + r, nd = row / a.g;
            if (nd >= a.N || d >= a.c.D) continue;
            const int w0 = (r / 16) * WN, rr = r & 15;
            float mx = -INFINITY;
#pragma unroll
            for (int x = 0; x < WN; ++x) mx = fmaxf(mx, s_m[w0 + x][rr]);
            const float base = mx == -INFINITY ? 0.0f : mx;
            float sum = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int x = 0; x < WN; ++x) {
                const float f = ex2(s_m[w0 + x][rr] - base);
                sum += s_l[w0 + x][rr] * f;
                const float4 v = *reinterpret_cast<const float4*>(s_o + ((w0 + x) * 16 + rr) * DP + d);
                acc[0] += v.x * f, acc[1] += v.y * f, acc[2] += v.z * f, acc[3] += v.w * f;
            }
            const float nan = __int_as_float(0x7fc00000);
            const bool empty = !u.cut.bad && (sum == 0.0f || nd >= u.cut.cnt);
            const float inv = u.cut.bad ? nan : 1.0f / sum;
            const float log2sum = u.cut.bad ? nan : empty ? -INFINITY : mx + log2f(sum);
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[x] = empty ? 0.0f : acc[x] * inv;
            if (u.whole) {
                const int64_t orow = (static_cast<int64_t>(u.b) * a.N + nd) * a.Hq + u.h * a.g + row % a.g;
                store_row4<F16>(a, orow, d, acc, log2sum);
            } else {
                *reinterpret_cast<float4*>(prow + r * a.c.D + d) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                if (d == 0) prow[MT * a.c.D + r] = log2sum;
            }
        }
    }
}

template <int DP, bool E4, bool F16, int WM>
cudaError_t launch_one(AttnArgs a, int nsm, cudaStream_t s) {
    constexpr size_t smem = Layout<DP, E4, WM>::bytes;
    const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(attn_mma_kernel<DP, E4, F16, WM>), smem);
    if (e != cudaSuccess) return e;
    a.ctas = nsm * (smem > 112 * 1024 ? 1 : 2);
    a.rounds = 0;
    attn_mma_kernel<DP, E4, F16, WM><<<static_cast<unsigned>(a.ctas), kThreads, smem, s>>>(a);
    const cudaError_t e2 = cudaGetLastError();
    return e2 != cudaSuccess ? e2 : launch_attn_combine(a, F16, 16 * WM, s);
}

// Units of 16 rows read the cache once per 16 rows, units of 64 compute for 64
// however many there are.  32 sequences of 4000 positions, 8 kv heads, 16-bit cache:
// heads of 256, 16 rows 328 and 658 us, 32 rows 636 and 673, 40 rows 936 and 677
// (heads of 128 on pages of 12: 32 rows 243 and 425, 48 rows 355 and 432, 56 rows 465
// and 433); e4m3: heads of 128, 48 rows 308 and 646, heads of 64, 48 rows 228 and
// 267, 64 rows 295 and 269.
template <int DP, bool E4, bool F16> cudaError_t launch_rows(const AttnArgs& a, int rows, int nsm, cudaStream_t s) {
    return rows <= (E4 ? 48 : 32) ? launch_one<DP, E4, F16, 1>(a, nsm, s) : launch_one<DP, E4, F16, 4>(a, nsm, s);
}

template <int DP>
cudaError_t launch_dim(const AttnArgs& a, bool f16, bool e4m3, int rows, int nsm, cudaStream_t s) {
    if (e4m3) return f16 ? launch_rows<DP, true, true>(a, rows, nsm, s) : launch_rows<DP, true, false>(a, rows, nsm, s);
    return f16 ? launch_rows<DP, false, true>(a, rows, nsm, s) : launch_rows<DP, false, false>(a, rows, nsm, s);
}

}  // namespace
}  // namespace sdv
