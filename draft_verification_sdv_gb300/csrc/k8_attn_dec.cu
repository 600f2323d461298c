// k8_attn_dec.cu -- tree attention for few query rows per kv head, such as one new
// token's (sdv_tree_attn), in units of 16 rows.
//
// The whole cache is read for a handful of rows, so HBM bounds the step, and the
// work per byte has to be small: a producer warp brings tiles of 32 KB (keys and
// values of BN positions) by tile copies, two ahead, and four warps
// split each tile's positions.  Each keeps its own running maximum, sum and
// output, so no warp waits for another until the unit's end; the products run on
// mma.sync m16n8k16, whose 16 rows waste less on 8 query heads than a
// tcgen05.mma of 128 would.
//
// e4m3 cells stay 8 bits wide in shared memory and are widened to fp16 (exact)
// as fragments are read.  The order of the contraction's index is free, so a
// lane takes 16 consecutive cells of a key row as its share of four
// instructions, and four consecutive cells of each of four value rows as its
// share of four output columns, transposed by byte permutes; under the copies'
// 128-byte swizzle neither has a bank conflict.  The rows' powers of two stay
// out of the products: a key's multiplies its score; a value's is added to the
// exponent, x' = x + e_v, with a running reference of x' for the outputs beside
// the one of x for the sum, so that neither can overflow.  These weights of the
// values have digits down to 2^-14, and some down to 2^-25; so the largest is kept
// within 2^6 .. 2^14: a row of values up to 2^-20 of the largest in probability
// times power counts with all its digits, one below 2^-31 not at all (with the
// largest at 1, channels beside one of 65000 were off by 2^-9).  bf16 queries are
// brought to fp16 in units of a power of two per row.
//
// 64 ragged sequences of up to 32000 positions, 8 kv heads of 128, e4m3: 457 us,
// 5.3 TB/s (the widening and the products then take the warps' time); 32 of 4000,
// 16 bits: 95 us, 5.6 TB/s.  Two CTAs of three stages per SM, where e4m3 heads of
// 128 spill 30 to 60 bytes a thread; with three CTAs of two stages it is far more
// (657 us).
#include "k8_attn_mma.cuh"
#include "k8_attn_tma.cuh"

namespace sdv {
namespace {

constexpr int kDecWarps = 4, kDecThreads = 32 * (kDecWarps + 1);
constexpr int kDecTile = 16 * 1024;          // of keys or of values
constexpr float kDecSlack = 8.0f;            // how far (log2) scores may pass their reference
constexpr float kDecUp = 14.0f - kDecSlack;  // e4m3: weights of values may reach 2^14

// DP: head dimension's room, 64 or 128; H: halves of the 16 rows in use.
template <int DP, bool E4> struct DecShape {
    static constexpr int NB = !E4 && DP == 128 ? 2 : 1;     // blocks of 128 bytes of a row
    static constexpr int BN = kDecTile / (128 * NB), NW = BN / kDecWarps, NT = NW / 8;
};

template <int DP, bool E4, int H> struct DecSmem {
    static constexpr int kStages = 3;                       // two CTAs per SM
    static constexpr int q = kStages * 2 * kDecTile;        // [16][DP] 16-bit, swizzled
    static constexpr int join = q + 16 * DP * 2;            // float [8 H][DP]
    static constexpr int ke = join + 8 * H * DP * 4;        // float [warps][2][NW] keys' powers of two, values' exponents
    static constexpr int qe = ke + (E4 ? 2 * DecShape<DP, E4>::BN * 4 : 0);
    static constexpr int ml = qe + 16 * 4;                  // float [2][warps][16] maxima and sums
    static constexpr int bar = ml + 2 * kDecWarps * 16 * 4;         // full, empty [kStages]
    static constexpr int dead = bar + 2 * kStages * 8;
    static constexpr int bytes = (dead + 4 + 15) / 16 * 16 + 1024;
};

// ONE: a kv head has one unit (16 rows at most).  REDO: launch_attn_redo; whole
// units, dealt out in turn.
template <int DP, bool E4, bool F16, int H, bool ONE, bool REDO>
__global__ void __launch_bounds__(kDecThreads, 2) attn_dec_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
                                                               const __grid_constant__ CUtensorMap map_v, int run_rows) {
    using S = DecShape<DP, E4>;
    using M = DecSmem<DP, E4, H>;
    constexpr int BN = S::BN, NW = S::NW, NT = S::NT, NB = S::NB, MT = 16, kStages = M::kStages;
    constexpr bool M16 = F16 || E4;                  // the products' type is fp16
    static_assert(NT % 2 == 0 && NW <= 32, "a warp takes pairs of column tiles, a lane one position");
    extern __shared__ unsigned char raw[];
    unsigned char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::bar);
    __shared__ int64_t s_part[40];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Sync sync{smem_u32(bars), smem_u32(smem + M::dead), a.status, a.hooks ? kHookPolls : kPolls};
    if (tid == 0) {
        *reinterpret_cast<int*>(smem + M::dead) = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bars + i, 1);
            mbar_init(bars + kStages + i, kDecWarps);
        }
    }
    const int mts = ONE ? 1 : (a.N * a.g + MT - 1) / MT;
    Part part{};
    Walk<MT, BN> walk{};
    if constexpr (REDO) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        unsigned beyond = 0;
        for (int i = tid; i < static_cast<int>(gridDim.x) / 2; i += kDecThreads) beyond |= a.beyond[i];
        if (!__syncthreads_or(beyond != 0)) return;
    } else {
        part = find_part<MT, BN, kDecThreads>(a, mts, s_part);            // holds barriers of the CTA
        walk.begin(a, part, mts);
        if (tid == 0) write_desc(a, part, walk);
    }
    auto next_unit = [&](Walk<MT, BN>& w, Unit& u) {
        if constexpr (REDO)
            if (static_cast<int>(blockIdx.x) + w.round * a.ctas >= a.B * a.c.H * mts) return false;
        return w.next(a, part, mts, u);
    };
    Unit u;
    uint32_t n = 0;                                  // tiles so far

    if (warp == kDecWarps) {
        // ---------------- loads ----------------
        // a lane to each copy of a tile's keys or values (32 at most), in turn
        const int copies = BN / run_rows, copy = lane / NB, block = lane - copy * NB;
        bool ok = true;
        while (ok && next_unit(walk, u)) {
            const int nt = u.len > 0 ? u.t1 - u.t0 : 0;
            const int32_t* table = a.table + static_cast<int64_t>(u.b) * a.max_pages;
            int off = 0, noff = 0;
            auto page_at = [&](int t, int& o) {
                const int pos = (u.t0 + t) * BN + copy * run_rows;
                if (copy >= copies || t >= nt || pos >= u.len) return -1;
                const int i = pos / a.c.P;
                o = u.h * a.c.P + pos - i * a.c.P;
                return __ldg(table + i);
            };
            int page = -1, npage = page_at(0, noff);
            for (int t = 0; t < nt; ++t, ++n) {
                page = npage, off = noff;
                npage = page_at(t + 1, noff);
                const uint32_t st = n % kStages;
                ok = sync.wait(kStages + st, (n / kStages & 1) ^ 1) && !sync.is_dead();
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if ((a.hooks & kHookAttnNoCopy) && blockIdx.x == 0 && n == 1) continue;     // a test: a tile that never comes
                const bool good = page >= 0 && page < a.c.pages;
                const uint32_t many = __popc(__ballot_sync(0xffffffffu, good));
                const uint32_t dst = smem_u32(smem + st * 2 * kDecTile) + block * BN * 128 + copy * run_rows * 128;
                if (elected()) mbar_arrive_expect_tx(bars + st, many * run_rows * 128 * 2);
                __syncwarp();
                if (good) {
                    tma_load(dst, &map_k, bars + st, block * 64, off, page);
                    tma_load(dst + kDecTile, &map_v, bars + st, block * 64, off, page);
                }
                __syncwarp();
            }
        }
        // what is still under way lands before the CTA goes (a dead one's too)
        for (uint32_t i = n > kStages ? n - kStages : 0; i < n; ++i) sync.landed(i % kStages, i / kStages & 1);
        return;
    }

    // ---------------- four warps of products and softmax ----------------
    unsigned char* s_q = smem + M::q;
    float* s_join = reinterpret_cast<float*>(smem + M::join);
    float* s_ke = reinterpret_cast<float*>(smem + M::ke) + warp * 2 * NW;
    float* s_ve = s_ke + NW;
    float* s_qe = reinterpret_cast<float*>(smem + M::qe);
    float* s_m = reinterpret_cast<float*>(smem + M::ml);
    float* s_l = s_m + kDecWarps * 16;
    const int g4 = lane >> 2, t4 = lane & 3;
    const int CW = warp * NW;                        // this warp's first position of a tile
    auto chunk_of = [](int r, int c) { return (c >> 3) * (BN * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4); };
    constexpr int kAll = 32 * kDecWarps;

    // where the warp is among its units waits in shared memory: registers are short
    __shared__ Walk<MT, BN> s_walk[kDecWarps];
    if (lane == 0) s_walk[warp] = walk;
    __syncwarp();
    auto next = [&]() {
        Walk<MT, BN> w = s_walk[warp];
        __syncwarp();
        const bool more = next_unit(w, u);
        if (lane == 0) s_walk[warp] = w;
        __syncwarp();
        return more;
    };

    while (next()) {
        if (tid == 0 && u.cut.bad && a.status) atomicOr(a.status, kStatusBadLength);
        const int32_t* table = a.table + static_cast<int64_t>(u.b) * a.max_pages;
        const int nt = u.len > 0 ? u.t1 - u.t0 : 0;
        bool alive = true;
        const int first = ONE ? 0 : u.mt * MT;       // of the unit's rows

        // ---- queries ----
        for (int w = tid; w < 16 * (DP / 8); w += kAll) {
            const int r = w / (DP / 8), c = w % (DP / 8);
            const int row = first + r, node = row / a.g;
            uint32_t v[4] = {0, 0, 0, 0};
            if (node < u.cut.cnt && c * 8 < a.c.D) {
                const unsigned char* p = a.q + u.b * a.q_sb + node * a.q_sn +
                                         (static_cast<int64_t>(u.h) * a.g + row % a.g) * a.q_sh + c * 16;
                if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
                    const uint4 x = *reinterpret_cast<const uint4*>(p);
                    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
                } else {
                    const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = h[2 * i] | (static_cast<uint32_t>(h[2 * i + 1]) << 16);
                }
            }
            if constexpr (E4 && !F16) {              // bf16 to fp16 in units of a power of two per row
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top = fmaxf(top, fmaxf(fabsf(bf16_lo(v[i])), fabsf(bf16_hi(v[i]))));
#pragma unroll
                for (int o = DP / 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
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
                // cell d is in chunk d >> 4, which lane t = chunk >> 1 reads in turn x = chunk & 1 (64
                // cells: t = chunk), and there element 2 t + (d & 1) + 8 (d >> 1 & 1) of step 4 x + (d >> 2 & 3)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = c * 8 + 2 * i, ch = d >> 4, x = DP == 128 ? ch & 1 : 0, t = DP == 128 ? ch >> 1 : ch;
                    const int to = (x * 4 + (d >> 2 & 3)) * 16 + 2 * t + 8 * (d >> 1 & 1);
                    *reinterpret_cast<uint32_t*>(s_q + r * DP * 2 + (((to >> 3) ^ (r & 7)) << 4) + (to & 7) * 2) = v[i];
                }
            } else {
                *reinterpret_cast<uint4*>(s_q + r * DP * 2 + ((c ^ (r & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
        bar_sync(1, kAll);

        float o[DP / 8][2 * H];
#pragma unroll
        for (int i = 0; i < DP / 8; ++i)
#pragma unroll
            for (int x = 0; x < 2 * H; ++x) o[i][x] = 0.0f;
        float m[H], mv[H], l[H], rowf[H];
        int node[H];
#pragma unroll
        for (int r = 0; r < H; ++r) {
            m[r] = mv[r] = -INFINITY, l[r] = 0.0f;
            rowf[r] = s_qe[g4 + 8 * r];
            node[r] = (first + g4 + 8 * r) / a.g;
        }

        // a lane looks after one of the warp's positions: its page is read two
        // tiles ahead, its exponents one
        auto page_at = [&](int t) {
            const int pos = (u.t0 + t) * BN + CW + lane;
            return lane < NW && t < nt && pos < u.len ? __ldg(table + pos / a.c.P) : 0;
        };
        int ke = 127, ve = 127;
        auto exps_at = [&](int t, int pg) {
            const int pos = (u.t0 + t) * BN + CW + lane;
            ke = ve = 127;
            if (lane < NW && t < nt && pos < u.len && pg >= 0 && pg < a.c.pages) {
                const int64_t at = pg * a.c.exp_page_stride + static_cast<int64_t>(u.h) * a.c.P + pos % a.c.P;
                ke = a.c.ke[at];
                ve = a.c.ve[at];
            }
        };
        int page0 = page_at(0), page1 = page_at(1);
        if constexpr (E4) exps_at(0, page0);

        for (int t = 0; t < nt; ++t, ++n) {
            const uint32_t st = n % kStages;
            const int pos0 = (u.t0 + t) * BN;        // of the tile
            bool odd = page0 < 0 || page0 >= a.c.pages;     // the lane's position is not a number
            if (odd && a.status) atomicOr(a.status, kStatusBadPage);
            if constexpr (E4) {
                odd |= ke == 255 || ve == 255;
                if (lane < NW) {
                    s_ke[lane] = ke == 0 ? __int_as_float(0x00400000) : __int_as_float(ke << 23);
                    s_ve[lane] = static_cast<float>(ve - 127);
                }
            }
            uint32_t flags = __ballot_sync(0xffffffffu, odd);   // also orders the exponents' stores
            page0 = page1;
            page1 = page_at(t + 2);
            if constexpr (E4) exps_at(t + 1, page0);
            alive &= sync.wait(st, n / kStages & 1);
            __syncwarp();
            const uint32_t k0 = smem_u32(smem + st * 2 * kDecTile), v0 = k0 + kDecTile;
            const bool mixed = pos0 + CW + NW > u.cut.ctx;
            if (mixed) {                             // values that are not numbers are kept out of the products
                constexpr int LR = E4 ? 8 : DP / 8, CH = LR;    // chunks, and lanes, of a row
                for (int r0 = 0; r0 < NW; r0 += 32 / LR) {
                    const int r = CW + r0 + lane / LR, c = lane % LR;
                    bool bad = false;
                    if (pos0 + r >= u.cut.ctx && c < CH) {
                        const uint4 x = lds128(v0 + chunk_of(r, c));
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if constexpr (E4) {
                                bad |= (((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
                            } else {
                                constexpr uint32_t ones = F16 ? 0x7c007c00u : 0x7f807f80u, unit = F16 ? 0x04000400u : 0x00800080u;
                                bad |= (((w[i] & ones) + unit) & 0x80008000u) != 0;
                            }
                        }
                    }
                    const uint32_t who = __ballot_sync(0xffffffffu, bad);
                    if (who) {
                        const bool row_bad = (who >> (lane / LR * LR) & (LR == 32 ? ~0u : (1u << LR) - 1u)) != 0;
                        if (row_bad) {
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v0 + chunk_of(r, c)), "r"(0) : "memory");
                            fence_async();           // before the copy that takes the slot next
                        }
#pragma unroll
                        for (int i = 0; i < 32 / LR; ++i)
                            if (who >> (i * LR) & (LR == 32 ? ~0u : (1u << LR) - 1u)) flags |= 1u << (r0 + i);
                        __syncwarp();
                    }
                }
            }

            // ---- scores ----
            float s[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
            const uint32_t q0 = smem_u32(s_q) + (lane & 15) * DP * 2;
            if constexpr (!E4) {
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks) {
                    uint32_t q[4];
                    ldsm4(q, q0 + (((ks * 2 + (lane >> 4)) ^ (lane & 7)) << 4));
#pragma unroll
                    for (int i = 0; i < NT; i += 2) {
                        uint32_t k[4];
                        ldsm4(k, k0 + chunk_of(CW + i * 8 + (lane >> 4) * 8 + (lane & 7), ks * 2 + (lane >> 3 & 1)));
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
                        const uint4 w = lds128(k0 + chunk_of(CW + i * 8 + g4, DP == 128 ? 2 * t4 + x : t4));
                        mma<true>(s[i], q[0], widen2(w.x), widen2(w.x >> 16));
                        mma<true>(s[i], q[1], widen2(w.y), widen2(w.y >> 16));
                        mma<true>(s[i], q[2], widen2(w.z), widen2(w.z >> 16));
                        mma<true>(s[i], q[3], widen2(w.w), widen2(w.w >> 16));
                    }
                }
            }

            // ---- scale, mask, references ----
            float ev[NT][2];
            float top[H], topv[H];
#pragma unroll
            for (int r = 0; r < H; ++r) top[r] = topv[r] = -INFINITY;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                float kf[2] = {1.0f, 1.0f};
                if constexpr (E4) {
                    const float2 x = *reinterpret_cast<const float2*>(s_ke + i * 8 + 2 * t4);
                    const float2 y = *reinterpret_cast<const float2*>(s_ve + i * 8 + 2 * t4);
                    kf[0] = x.x, kf[1] = x.y, ev[i][0] = y.x, ev[i][1] = y.y;
                }
#pragma unroll
                for (int x = 0; x < 2 * H; ++x) {
                    const int rr = x >> 1;
                    float v = s[i][x] * rowf[rr];
                    if constexpr (E4) v *= kf[x & 1];
                    s[i][x] = v;
                }
            }
            if (mixed || flags) {
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int x = 0; x < 2 * H; ++x) {
                        const int rr = x >> 1, col = i * 8 + 2 * t4 + (x & 1), pos = pos0 + CW + col;
                        if (flags >> col & 1) s[i][x] = __int_as_float(0x7fc00000);
                        const int nm = pos - u.cut.ctx;      // which node the column is
                        bool see = pos < u.len;
                        if (see && nm >= 0) {
                            if (a.mask)
                                see = node[rr] < u.cut.cnt &&
                                      (__ldg(a.mask + u.b * a.mask_sb + static_cast<int64_t>(node[rr]) * a.W + (nm >> 5)) >> (nm & 31) & 1);
                            else
                                see = nm <= node[rr];
                        }
                        if (!see) s[i][x] = -INFINITY;
                    }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int x = 0; x < 2 * H; ++x) {
                    const int rr = x >> 1;
                    top[rr] = fmaxf(top[rr], s[i][x]);
                    if constexpr (E4) topv[rr] = fmaxf(topv[rr], s[i][x] + ev[i][x & 1]);
                }
            bool move = false;
#pragma unroll
            for (int r = 0; r < H; ++r) {
#pragma unroll
                for (int x = 1; x < 4; x <<= 1) {
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], x));
                    if constexpr (E4) topv[r] = fmaxf(topv[r], __shfl_xor_sync(0xffffffffu, topv[r], x));
                }
                if constexpr (!E4) topv[r] = top[r];
                move |= top[r] > m[r] + kDecSlack || topv[r] > mv[r] + kDecSlack || (m[r] == -INFINITY && top[r] != -INFINITY);
            }
            if (__any_sync(0xffffffffu, move)) {     // the references follow the scores
#pragma unroll
                for (int r = 0; r < H; ++r) {
                    const float to = fmaxf(m[r], top[r]), tov = fmaxf(mv[r], topv[r]);
                    l[r] *= ex2(m[r] - (to == -INFINITY ? 0.0f : to));
                    const float by = ex2(mv[r] - (tov == -INFINITY ? 0.0f : tov));
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i) o[i][2 * r] *= by, o[i][2 * r + 1] *= by;
                    m[r] = to;
                    mv[r] = tov;
                }
            }
            float sub[H], subv[H];
#pragma unroll
            for (int r = 0; r < H; ++r) {
                sub[r] = m[r] == -INFINITY ? 0.0f : m[r];    // nothing seen yet: 2^-inf = 0
                subv[r] = mv[r] == -INFINITY ? 0.0f : mv[r] - kDecUp;
            }

            // ---- probabilities (fp32 into the sum, 16 bits into the product) and outputs ----
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
                uint32_t p[4] = {0, 0, 0, 0};
#pragma unroll
                for (int y = 0; y < 4; ++y) {        // registers a0..a3: column tile y >> 1, row y & 1
                    const int i = 2 * j + (y >> 1), r = y & 1;
                    if (r >= H) continue;
                    const float x0 = s[i][2 * r], x1 = s[i][2 * r + 1];
                    const float e0 = ex2(x0 - sub[r]), e1 = ex2(x1 - sub[r]);
                    l[r] += e0 + e1;
                    if constexpr (E4)
                        p[y] = pack2<true>(ex2(x0 + ev[i][0] - subv[r]), ex2(x1 + ev[i][1] - subv[r]));
                    else
                        p[y] = pack2<F16>(e0, e1);
                }
                const int r0 = CW + j * 16;
                // (with one half in use the other rows' outputs are not kept)
                auto add = [&](int i, uint32_t b0, uint32_t b1) {
                    if constexpr (H == 2) {
                        mma<M16>(reinterpret_cast<float(&)[4]>(o[i]), p, b0, b1);
                    } else {
                        float d[4] = {o[i][0], o[i][1], 0.0f, 0.0f};
                        mma<M16>(d, p, b0, b1);
                        o[i][0] = d[0], o[i][1] = d[1];
                    }
                };
                if constexpr (!E4) {
#pragma unroll
                    for (int i = 0; i < DP / 8; i += 2) {
                        uint32_t v[4];               // 16 positions x 16 columns
                        ldsm4t(v, v0 + chunk_of(r0 + (lane & 15), i + (lane >> 4)));
                        add(i, v[0], v[1]);
                        add(i + 1, v[2], v[3]);
                    }
                } else {
#pragma unroll
                    for (int y = 0; y < DP / 32; ++y) {
                        uint32_t w[4];               // cells 32 y + 4 g4 .. + 3 of rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int r = r0 + 2 * t4 + (x & 1) + 8 * (x >> 1);
                            w[x] = lds32(v0 + chunk_of(r, 2 * y + (g4 >> 2)) + (g4 & 3) * 4);
                        }
                        const uint32_t lo01 = __byte_perm(w[0], w[1], 0x5140), lo23 = __byte_perm(w[0], w[1], 0x7362);
                        const uint32_t hi01 = __byte_perm(w[2], w[3], 0x5140), hi23 = __byte_perm(w[2], w[3], 0x7362);
                        add(4 * y + 0, widen2(lo01), widen2(hi01));
                        add(4 * y + 1, widen2(lo01 >> 16), widen2(hi01 >> 16));
                        add(4 * y + 2, widen2(lo23), widen2(hi23));
                        add(4 * y + 3, widen2(lo23 >> 16), widen2(hi23 >> 16));
                    }
                }
            }
            __syncwarp();
            if (lane == 0) sync.arrive(kStages + st);
        }

        // ---- the unit's rows: the warps' outputs join one after another ----
        const bool dead = !alive || sync.is_dead();
        float base[H];
#pragma unroll
        for (int r = 0; r < H; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (dead) l[r] = __int_as_float(0x7fc00000);
            if (t4 == 0) s_m[warp * 16 + g4 + 8 * r] = m[r], s_l[warp * 16 + g4 + 8 * r] = l[r];
        }
        bar_sync(1, kAll);
#pragma unroll
        for (int r = 0; r < H; ++r) {
            float mx = -INFINITY;
#pragma unroll
            for (int x = 0; x < kDecWarps; ++x) mx = fmaxf(mx, s_m[x * 16 + g4 + 8 * r]);
            base[r] = mx == -INFINITY ? 0.0f : mx;
            // in units of 2^base: o * 2^(mv - base)
            const float up = mv[r] == -INFINITY ? 0.0f : ex2(mv[r] - (E4 ? kDecUp : 0.0f) - base[r]);
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) o[i][2 * r] *= up, o[i][2 * r + 1] *= up;
        }
        for (int turn = 0; turn < kDecWarps; ++turn) {
            if (warp == turn) {
#pragma unroll
                for (int r = 0; r < H; ++r) {
                    float* dst = s_join + (g4 + 8 * r) * DP;
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int d = E4 ? (i >> 2) * 32 + 8 * t4 + 4 * x + (i & 3) : i * 8 + 2 * t4 + x;
                            dst[d] = turn == 0 ? o[i][2 * r + x] : dst[d] + o[i][2 * r + x];
                        }
                }
            }
            bar_sync(1, kAll);
        }
        float* prow = part_rows(a, blockIdx.x, u.t0 > 0 ? 0 : 1, MT);
        for (int w = tid; w < 8 * H * (DP / 4); w += kAll) {
            const int r = w / (DP / 4), d = (w % (DP / 4)) * 4;
            const int nd = (first + r) / a.g;
            if (nd >= a.N || d >= a.c.D) continue;
            float mx = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int x = 0; x < kDecWarps; ++x) mx = fmaxf(mx, s_m[x * 16 + r]);
            const float b0 = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
            for (int x = 0; x < kDecWarps; ++x) sum += s_l[x * 16 + r] * ex2(s_m[x * 16 + r] - b0);
            const float4 v = *reinterpret_cast<const float4*>(s_join + r * DP + d);
            const float nan = __int_as_float(0x7fc00000);
            const bool empty = !u.cut.bad && (sum == 0.0f || nd >= u.cut.cnt);
            const float inv = u.cut.bad ? nan : empty ? 0.0f : 1.0f / sum;
            const float log2sum = u.cut.bad ? nan : empty ? -INFINITY : b0 + log2f(sum);
            const float acc[4] = {empty ? 0.0f : v.x * inv, empty ? 0.0f : v.y * inv, empty ? 0.0f : v.z * inv, empty ? 0.0f : v.w * inv};
            if (u.whole) {
                const int64_t orow = (static_cast<int64_t>(u.b) * a.N + nd) * a.Hq + u.h * a.g + (first + r) % a.g;
                unsigned short* dst = static_cast<unsigned short*>(a.out) + orow * a.c.D + d;
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<F16>(acc[0], acc[1]), pack2<F16>(acc[2], acc[3]));
                if (d == 0 && a.lse) a.lse[orow] = log2sum * kLn2;
            } else {
                *reinterpret_cast<float4*>(prow + r * a.c.D + d) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                if (d == 0) prow[MT * a.c.D + r] = log2sum;
            }
        }
        bar_sync(1, kAll);                           // before the next unit's queries and joins
    }
}

template <int DP, bool E4, bool F16, int H, bool ONE, bool REDO = false>
cudaError_t dec_one(AttnArgs a, int nsm, cudaStream_t s) {
    constexpr int bytes = DecSmem<DP, E4, H>::bytes, BN = DecShape<DP, E4>::BN;
    const int rows = min(a.c.P & -a.c.P, BN);        // of one copy: sure to lie in one page
    CUtensorMap k, v;
    if (!encode_cells(&k, a, a.c.k, E4, rows, true) || !encode_cells(&v, a, a.c.v, E4, rows, true)) return cudaErrorInvalidValue;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(attn_dec_kernel<DP, E4, F16, H, ONE, REDO>), bytes);
    if (e != cudaSuccess) return e;
    a.ctas = nsm * 2;
    a.rounds = REDO ? 1 << 30 : 0;
    if constexpr (REDO) {                            // its launch is on its way while the kernel before ends
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(a.ctas));
        cfg.blockDim = dim3(kDecThreads);
        cfg.dynamicSmemBytes = bytes;
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, attn_dec_kernel<DP, E4, F16, H, ONE, REDO>, a, k, v, rows);
    } else {
        attn_dec_kernel<DP, E4, F16, H, ONE, REDO><<<static_cast<unsigned>(a.ctas), kDecThreads, bytes, s>>>(a, k, v, rows);
        e = cudaGetLastError();
        return e != cudaSuccess ? e : launch_attn_combine(a, F16, 16, s);
    }
}

// With 8 rows or fewer the other half of the instructions' 16 is not carried
// along: 64 ragged sequences of 8 rows, e4m3, 457 us against 533 us.
template <int DP, bool E4, bool F16> cudaError_t dec_rows(const AttnArgs& a, int nsm, cudaStream_t s) {
    const int rows = a.N * a.g;
    if (rows <= 8) return dec_one<DP, E4, F16, 1, true>(a, nsm, s);
    if (rows <= 16) return dec_one<DP, E4, F16, 2, true>(a, nsm, s);
    // (e4m3 alone comes here with more rows)
    if constexpr (E4) return dec_one<DP, E4, F16, 2, false>(a, nsm, s);
    return cudaErrorInvalidValue;
}

template <int DP> cudaError_t dec_types(const AttnArgs& a, bool f16, bool e4m3, int nsm, cudaStream_t s) {
    if (e4m3) return f16 ? dec_rows<DP, true, true>(a, nsm, s) : dec_rows<DP, true, false>(a, nsm, s);
    return f16 ? dec_rows<DP, false, true>(a, nsm, s) : dec_rows<DP, false, false>(a, nsm, s);
}

}  // namespace

cudaError_t launch_attn_dec(const AttnArgs& a, bool f16, bool e4m3, int nsm, cudaStream_t s) {
    return a.c.D <= 64 ? dec_types<64>(a, f16, e4m3, nsm, s) : dec_types<128>(a, f16, e4m3, nsm, s);
}

cudaError_t launch_attn_redo(const AttnArgs& a, int nsm, cudaStream_t s) {
    return a.c.D <= 64 ? dec_one<64, true, true, 2, false, true>(a, nsm, s) : dec_one<128, true, true, 2, false, true>(a, nsm, s);
}

}  // namespace sdv
