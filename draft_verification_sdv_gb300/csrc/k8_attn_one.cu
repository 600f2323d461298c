// k8_attn_one.cu -- what single tokens add behind a shared prefix (sdv_prefix_attn
// with N = 1): attention over each sequence's own, mostly short, positions.
//
// A unit is a sequence and a kv head.  Its positions are few, and there are many
// units, so what costs is a unit's beginning and end.  A CTA of four warps takes one
// unit (or one of `splits` parts of it, where there are few), and many CTAs on an SM
// keep the reads going; nothing is staged: a lane reads keys and values as the
// operands of mma.sync m16n8k16 want them, 16 bytes at a time.
//   S = Q K^T   the contraction's index is taken in an order in which a lane's
//               share of a key row is 8 consecutive 16-bit cells (16 of e4m3) of each
//               64 bytes; the queries are read in the same order
//   O = P V     a lane takes the same 8 (16) columns of its four value rows, and
//               byte permutes pair up the rows; so column tile (p, e) has the columns
//               64 p + 8 n + e (16 n + e)
// Each warp takes every fourth tile of 16 positions and keeps its own maxima, sums and
// outputs; e4m3 rows' powers of two are kept out of the products as in
// k8_attn_dec.cu.  The warps' outputs join in shared memory, and with the prefix's
// row, where nothing was split.
//
// What bounds it: the latency of a unit's chain of reads (length, page, cells) and the
// cells in flight, of which three CTAs an SM (168 registers) hold 8 KB a warp (e4m3: 4).  One
// token each of 128 sequences with 1 to 700 own positions, 8 x 8 heads of 128, 16 bits:
// 56 us, 3.2 TB/s (104 us and two joins in units of k8_attn_dec.cu, of which each costs 9
// us); 96 sequences of up to 500, e4m3: 29 us (71).
#include "k8_attn_mma.cuh"

namespace sdv {
namespace {

using namespace attn;

constexpr int kOneWarps = 4, kOneThreads = 32 * kOneWarps, kOneTile = 16;
constexpr float kOneSlack = 8.0f;           // how far (log2) scores may pass their reference
constexpr float kOneUp = 14.0f - kOneSlack; // e4m3: weights of values may reach 2^14

__device__ __forceinline__ uint4 ld_cells(const unsigned char* p, bool there) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (there) v = ld_stream(reinterpret_cast<const uint4*>(p));
    return v;
}

// H: halves of the 16 rows in use.
template <int DP, bool E4, bool F16, int H>
__global__ void __launch_bounds__(kOneThreads, DP == 64 ? 4 : H == 1 ? 3 : 2) attn_one_kernel(const AttnArgs a, const float* far, const float* far_log, int splits) {
    constexpr bool M16 = F16 || E4;                  // the products' type is fp16
    constexpr int KL = E4 ? DP / 64 : DP / 32;       // 16-byte loads of a lane from a key row
    constexpr int VL = E4 ? 1 : DP / 64;             // ... from a value row (e4m3 heads of 64: half of one)
    constexpr int CT = DP / 8;                       // column tiles
    __shared__ float s_o[kOneWarps][8 * H][DP + 4];
    __shared__ float s_m[kOneWarps][8 * H], s_l[kOneWarps][8 * H];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g4 = lane >> 2, t4 = lane & 3;
    const int b = blockIdx.x / a.c.H, h = blockIdx.x - b * a.c.H;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Cut cut = cut_of(a, b);
    const int own = cut.cnt > 0 && (!a.mask || (a.mask[b * a.mask_sb] & 1)) ? 1 : 0;     // does the token see itself
    const int len = cut.cnt > 0 ? cut.ctx + own : 0;
    // (parts of what is held: the table may be far wider)
    constexpr int kRound = kOneWarps * kOneTile;
    const int chunk = ((len + kRound - 1) / kRound + splits - 1) / splits * kRound;
    const int begin = blockIdx.y * chunk, end = min(len, begin + chunk);
    if (tid == 0 && blockIdx.y == 0 && cut.bad && a.status) atomicOr(a.status, kStatusBadLength);

    // ---- queries ----
    uint32_t q[H][KL][E4 ? 8 : 4];
    float rowf[H];
#pragma unroll
    for (int r = 0; r < H; ++r) {
        const int head = g4 + 8 * r;
        const unsigned char* p = a.q + b * a.q_sb + (static_cast<int64_t>(h) * a.g + head) * a.q_sh;
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < KL; ++j)
#pragma unroll
            for (int x = 0; x < (E4 ? 2 : 1); ++x) {
                const unsigned char* at = p + (E4 ? j * 128 + t4 * 32 + x * 16 : j * 64 + t4 * 16);
                uint4 v = make_uint4(0, 0, 0, 0);
                if (head < a.g && begin < end) {
                    if ((reinterpret_cast<uintptr_t>(at) & 15) == 0) {
                        v = *reinterpret_cast<const uint4*>(at);
                    } else {
                        const unsigned short* e = reinterpret_cast<const unsigned short*>(at);
                        v = make_uint4(e[0] | static_cast<uint32_t>(e[1]) << 16, e[2] | static_cast<uint32_t>(e[3]) << 16,
                                       e[4] | static_cast<uint32_t>(e[5]) << 16, e[6] | static_cast<uint32_t>(e[7]) << 16);
                    }
                }
                q[r][j][4 * x] = v.x, q[r][j][4 * x + 1] = v.y, q[r][j][4 * x + 2] = v.z, q[r][j][4 * x + 3] = v.w;
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    if constexpr (E4 && !F16) top = fmaxf(top, fmaxf(fabsf(bf16_lo(q[r][j][4 * x + y])), fabsf(bf16_hi(q[r][j][4 * x + y]))));
            }
        rowf[r] = a.scale_log2;
        if constexpr (E4 && !F16) {                  // bf16 to fp16 in units of a power of two per row
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            int e = (__float_as_int(top) >> 23) - 127 - 14;      // the largest ends in [2^14, 2^15)
            e = e < -126 ? -126 : e;
            const float inv = __int_as_float((127 - e) << 23);
#pragma unroll
            for (int j = 0; j < KL; ++j)
#pragma unroll
                for (int y = 0; y < 8; ++y) q[r][j][y] = pack2<true>(bf16_lo(q[r][j][y]) * inv, bf16_hi(q[r][j][y]) * inv);
            rowf[r] *= __int_as_float((e + 127) << 23);
        }
    }

    float o[CT][2 * H], m[H], mv[H], l[H];
#pragma unroll
    for (int i = 0; i < CT; ++i)
#pragma unroll
        for (int x = 0; x < 2 * H; ++x) o[i][x] = 0.0f;
#pragma unroll
    for (int r = 0; r < H; ++r) m[r] = mv[r] = -INFINITY, l[r] = 0.0f;

    // a lane looks after one of the tile's positions: its page is asked for two tiles ahead,
    // its cells one; keys (values) are read as soon as those before them are used
    const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_pages;
    auto page_at = [&](int pos) { return lane < kOneTile && pos + lane < end ? __ldg(table + (pos + lane) / a.c.P) : 0; };
    struct Place {
        int64_t at;                                  // the cells' offset, -1: none
        int ke, ve;
        bool bad;                                    // a page that is not the cache's
    };
    auto place_at = [&](int pos0, int page) {
        Place p{-1, 127, 127, false};
        const int pos = pos0 + lane;
        if (lane >= kOneTile || pos >= end) return p;
        p.bad = page < 0 || page >= a.c.pages;
        if (p.bad) return p;
        const int cell = h * a.c.P + pos % a.c.P;    // within the page
        p.at = page * a.c.page_stride + static_cast<int64_t>(cell) * (a.c.D * (E4 ? 1 : 2));
        if constexpr (E4) p.ke = a.c.ke[page * a.c.exp_page_stride + cell], p.ve = a.c.ve[page * a.c.exp_page_stride + cell];
        return p;
    };
    // keys g4 and 8 + g4; values 2 t4, 2 t4 + 1, 2 t4 + 8 and 2 t4 + 9
    uint4 k[2][KL], v[4][VL];
    auto load_keys = [&](const Place& p) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t row = __shfl_sync(0xffffffffu, p.at, i * 8 + g4);
#pragma unroll
            for (int j = 0; j < KL; ++j) k[i][j] = ld_cells(a.c.k + row + j * 64 + t4 * 16, row >= 0);
        }
    };
    auto load_values = [&](const Place& p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = __shfl_sync(0xffffffffu, p.at, 2 * t4 + (i & 1) + 8 * (i >> 1));
#pragma unroll
            for (int j = 0; j < VL; ++j) {
                if constexpr (E4 && DP == 64) {
                    uint2 x = make_uint2(0, 0);
                    if (row >= 0) x = __ldg(reinterpret_cast<const uint2*>(a.c.v + row + g4 * 8));
                    v[i][j] = make_uint4(x.x, x.y, 0, 0);
                } else {
                    v[i][j] = ld_cells(a.c.v + row + j * 128 + g4 * 16, row >= 0);
                }
            }
        }
    };
    bool nan_row = false;
    int pos0 = begin + warp * kOneTile;
    int page = page_at(pos0 + kRound);
    Place here = place_at(pos0, page_at(pos0));
    load_keys(here);
    load_values(here);
    for (; pos0 < end; pos0 += kRound) {
        const Place next = place_at(pos0 + kRound, page);
        page = page_at(pos0 + 2 * kRound);
        if (here.bad && a.status) atomicOr(a.status, kStatusBadPage);

        // ---- scores ----
        float s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll
            for (int j = 0; j < KL; ++j) {
                const uint32_t w[4] = {k[i][j].x, k[i][j].y, k[i][j].z, k[i][j].w};
                if constexpr (E4) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t qa[4] = {q[0][j][2 * y], H > 1 ? q[H - 1][j][2 * y] : 0u, q[0][j][2 * y + 1], H > 1 ? q[H - 1][j][2 * y + 1] : 0u};
                        mma<true>(s[i], qa, widen2(w[y]), widen2(w[y] >> 16));
                    }
                } else {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t qa[4] = {q[0][j][2 * y], H > 1 ? q[H - 1][j][2 * y] : 0u, q[0][j][2 * y + 1], H > 1 ? q[H - 1][j][2 * y + 1] : 0u};
                        mma<M16>(s[i], qa, w[2 * y], w[2 * y + 1]);
                    }
                }
            }
        }

        load_keys(next);

        // ---- scale, what lies past the end, references ----
        float ev[2][2] = {};
        const uint32_t odd = __ballot_sync(0xffffffffu, here.bad || (E4 && here.at >= 0 && (here.ke == 255 || here.ve == 255)));
        nan_row |= odd != 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int col = i * 8 + 2 * t4 + x;
                float kf = 1.0f;
                if constexpr (E4) {
                    const int e = __shfl_sync(0xffffffffu, here.ke, col);
                    kf = e == 0 ? __int_as_float(0x00400000) : __int_as_float(e << 23);
                    ev[i][x] = static_cast<float>(__shfl_sync(0xffffffffu, here.ve, col) - 127);
                }
#pragma unroll
                for (int r = 0; r < H; ++r) s[i][2 * r + x] = pos0 + col < end ? s[i][2 * r + x] * rowf[r] * kf : -INFINITY;
            }
        float top[H], topv[H];
        bool move = false;
#pragma unroll
        for (int r = 0; r < H; ++r) {
            top[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
            topv[r] = top[r];
            if constexpr (E4)
                topv[r] = fmaxf(fmaxf(s[0][2 * r] + ev[0][0], s[0][2 * r + 1] + ev[0][1]), fmaxf(s[1][2 * r] + ev[1][0], s[1][2 * r + 1] + ev[1][1]));
#pragma unroll
            for (int x = 1; x < 4; x <<= 1) {
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], x));
                if constexpr (E4) topv[r] = fmaxf(topv[r], __shfl_xor_sync(0xffffffffu, topv[r], x));
            }
            if constexpr (!E4) topv[r] = top[r];
            move |= top[r] > m[r] + kOneSlack || topv[r] > mv[r] + kOneSlack || (m[r] == -INFINITY && top[r] != -INFINITY);
        }
        if (__any_sync(0xffffffffu, move)) {         // the references follow the scores
#pragma unroll
            for (int r = 0; r < H; ++r) {
                const float to = fmaxf(m[r], top[r]), tov = fmaxf(mv[r], topv[r]);
                l[r] *= ex2(m[r] - (to == -INFINITY ? 0.0f : to));
                const float by = ex2(mv[r] - (tov == -INFINITY ? 0.0f : tov));
#pragma unroll
                for (int i = 0; i < CT; ++i) o[i][2 * r] *= by, o[i][2 * r + 1] *= by;
                m[r] = to;
                mv[r] = tov;
            }
        }

        // ---- probabilities (fp32 into the sum, 16 bits into the product) and outputs ----
        // (mma.sync takes 16-bit operands, as the other attention kernels' products do; outputs are off by
        // 0.0023 rms relative in bf16, and rounding them alone makes 0.0017)
        uint32_t p[4] = {0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < H; ++r) {
            const float sub = m[r] == -INFINITY ? 0.0f : m[r], subv = mv[r] == -INFINITY ? 0.0f : mv[r] - kOneUp;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x0 = s[i][2 * r], x1 = s[i][2 * r + 1], e0 = ex2(x0 - sub), e1 = ex2(x1 - sub);
                l[r] += e0 + e1;
                if constexpr (E4)
                    p[2 * i + r] = pack2<true>(ex2(x0 + ev[i][0] - subv), ex2(x1 + ev[i][1] - subv));
                else
                    p[2 * i + r] = pack2<F16>(e0, e1);
            }
        }
        auto add = [&](int i, uint32_t b0, uint32_t b1) {
            if constexpr (H == 2) {
                mma<M16>(reinterpret_cast<float(&)[4]>(o[i]), p, b0, b1);
            } else {
                float d[4] = {o[i][0], o[i][1], 0.0f, 0.0f};
                mma<M16>(d, p, b0, b1);
                o[i][0] = d[0], o[i][1] = d[1];
            }
        };
#pragma unroll
        for (int j = 0; j < VL; ++j) {
            const uint32_t w[4][4] = {{v[0][j].x, v[0][j].y, v[0][j].z, v[0][j].w}, {v[1][j].x, v[1][j].y, v[1][j].z, v[1][j].w},
                                      {v[2][j].x, v[2][j].y, v[2][j].z, v[2][j].w}, {v[3][j].x, v[3][j].y, v[3][j].z, v[3][j].w}};
            if constexpr (E4) {
#pragma unroll
                for (int y = 0; y < CT / 4; ++y) {   // four columns: pairs of rows byte by byte
                    const uint32_t lo01 = __byte_perm(w[0][y], w[1][y], 0x5140), lo23 = __byte_perm(w[0][y], w[1][y], 0x7362);
                    const uint32_t hi01 = __byte_perm(w[2][y], w[3][y], 0x5140), hi23 = __byte_perm(w[2][y], w[3][y], 0x7362);
                    add(4 * y, widen2(lo01), widen2(hi01));
                    add(4 * y + 1, widen2(lo01 >> 16), widen2(hi01 >> 16));
                    add(4 * y + 2, widen2(lo23), widen2(hi23));
                    add(4 * y + 3, widen2(lo23 >> 16), widen2(hi23 >> 16));
                }
            } else {
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    add(j * 8 + 2 * y, __byte_perm(w[0][y], w[1][y], 0x5410), __byte_perm(w[2][y], w[3][y], 0x5410));
                    add(j * 8 + 2 * y + 1, __byte_perm(w[0][y], w[1][y], 0x7632), __byte_perm(w[2][y], w[3][y], 0x7632));
                }
            }
        }
        load_values(next);
        here = next;
    }

    // ---- the warps' outputs join, and then the prefix's ----
#pragma unroll
    for (int r = 0; r < H; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if (nan_row) l[r] = __int_as_float(0x7fc00000);
        if (t4 == 0) s_m[warp][g4 + 8 * r] = m[r], s_l[warp][g4 + 8 * r] = l[r];
        // in units of 2^m: o * 2^(mv - m)
        const float up = m[r] == -INFINITY ? 0.0f : E4 ? ex2(mv[r] - kOneUp - m[r]) : 1.0f;
        float* row = s_o[warp][g4 + 8 * r];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < CT; i += 4) {
                const int d = E4 ? (2 * t4 + x) * CT + i : (i >> 3) * 64 + (2 * t4 + x) * 8 + (i & 7);
                *reinterpret_cast<float4*>(row + d) = make_float4(o[i][2 * r + x] * up, o[i + 1][2 * r + x] * up, o[i + 2][2 * r + x] * up, o[i + 3][2 * r + x] * up);
            }
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");       // (the prefix's rows, and what this writes over)
    const float nan = __int_as_float(0x7fc00000);
    for (int w = tid; w < a.g * (DP / 4); w += kOneThreads) {
        const int r = w / (DP / 4), d = (w % (DP / 4)) * 4;
        const int64_t orow = static_cast<int64_t>(b) * a.Hq + h * a.g + r;
        float top = -INFINITY;
#pragma unroll
        for (int x = 0; x < kOneWarps; ++x) top = fmaxf(top, s_m[x][r]);
        float base = top == -INFINITY ? 0.0f : top, sum = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int x = 0; x < kOneWarps; ++x) {
            const float f = ex2(s_m[x][r] - base);
            sum += s_l[x][r] * f;
            const float4 y = *reinterpret_cast<const float4*>(&s_o[x][r][d]);
            acc[0] += y.x * f, acc[1] += y.y * f, acc[2] += y.z * f, acc[3] += y.w * f;
        }
        if (splits > 1) {                            // a part: normalised, with its log
            const int64_t part = static_cast<int64_t>(blockIdx.y) * a.B * a.Hq + orow;
            const float log2sum = cut.bad ? nan : sum == 0.0f ? -INFINITY : base + log2f(sum);
            if (d == 0) a.raw_log[part] = log2sum;
            if (log2sum != -INFINITY) {
                const float inv = cut.bad ? nan : 1.0f / sum;
                *reinterpret_cast<float4*>(a.raw + part * DP + d) = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
            }
            continue;
        }
        const bool dead = !cut.bad && cut.cnt == 0;
        const float L = far_log[orow];
        if (!dead && L != -INFINITY) {               // the prefix's row weighs 2^L
            const float4 y = *reinterpret_cast<const float4*>(far + orow * DP + d);
            const float to = fmaxf(base, L), was = sum == 0.0f ? 0.0f : ex2(base - to);
            const float mine = sum == 0.0f ? 1.0f : ex2(L - to);
            sum = sum == 0.0f ? 1.0f : sum * was + mine;
            acc[0] = acc[0] * was + y.x * mine, acc[1] = acc[1] * was + y.y * mine;
            acc[2] = acc[2] * was + y.z * mine, acc[3] = acc[3] * was + y.w * mine;
            base = was == 0.0f && mine == 1.0f ? L : to;
        }
        const bool bad = cut.bad || L != L, empty = dead || (!bad && sum == 0.0f);
        const float inv = bad && !dead ? nan : empty ? 0.0f : 1.0f / sum;
        const float x[4] = {empty ? 0.0f : acc[0] * inv, empty ? 0.0f : acc[1] * inv, empty ? 0.0f : acc[2] * inv, empty ? 0.0f : acc[3] * inv};
        *reinterpret_cast<uint2*>(static_cast<unsigned short*>(a.out) + orow * DP + d) = make_uint2(pack2<F16>(x[0], x[1]), pack2<F16>(x[2], x[3]));
        if (d == 0 && a.lse) a.lse[orow] = empty ? -INFINITY : bad ? nan : (base + log2f(sum)) * kLn2;
    }
}

template <int DP, bool E4, bool F16, int H>
cudaError_t one(const AttnArgs& a, const float* far, const float* far_log, int splits, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B * a.c.H), static_cast<unsigned>(splits));
    cfg.blockDim = dim3(kOneThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_one_kernel<DP, E4, F16, H>, a, far, far_log, splits);
}

template <int DP, bool E4>
cudaError_t one_types(const AttnArgs& a, bool f16, const float* far, const float* far_log, int splits, cudaStream_t s) {
    if (a.g <= 8)
        return f16 ? one<DP, E4, true, 1>(a, far, far_log, splits, s) : one<DP, E4, false, 1>(a, far, far_log, splits, s);
    return f16 ? one<DP, E4, true, 2>(a, far, far_log, splits, s) : one<DP, E4, false, 2>(a, far, far_log, splits, s);
}

}  // namespace

bool attn_one_takes(const AttnArgs& a) { return a.N == 1 && a.g <= 16 && (a.c.D == 64 || a.c.D == 128); }

cudaError_t launch_attn_one(const AttnArgs& a, bool f16, bool e4m3, const float* far, const float* far_log, int splits, cudaStream_t s) {
    if (a.c.D == 64)
        return e4m3 ? one_types<64, true>(a, f16, far, far_log, splits, s) : one_types<64, false>(a, f16, far, far_log, splits, s);
    return e4m3 ? one_types<128, true>(a, f16, far, far_log, splits, s) : one_types<128, false>(a, f16, far, far_log, splits, s);
}

}  // namespace sdv
