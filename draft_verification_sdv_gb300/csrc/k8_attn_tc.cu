// k8_attn_tc.cu -- tree attention for many query rows (sdv_tree_attn) on the
// 5th-generation tensor cores.
//
// A tree of N nodes has N * g query rows per kv head; from a few dozen rows on
// the two contractions bound the step, not the cache's bytes.  A CTA works on
// 256 rows as two streams of 128 (the rows of one tcgen05.mma), so that while
// the softmax of one stream runs, the tensor cores multiply for the other:
//   S_s = Q_s K^T        both operands in shared memory, accumulator in TMEM
//   P_s = 2^(c S_s - m)  a thread per row reads S_s from TMEM and writes P_s,
//                        16 bits wide, over S_s
//   O_s += P_s V         P_s from TMEM, V from shared memory, O_s in TMEM
// TMEM holds S_0, S_1, O_0, O_1: 4 x 128 columns, all 512.
//
// O is not rescaled each time the maximum grows: the running reference m only
// moves when a row's scores pass it by 2^8 (fp32 sums and 16-bit probabilities
// keep their relative precision below that), and then the row's warp rescales.
//
// Warps 0-3 and 4-7: softmax of stream 0 and 1; 8-11: loads; 12: one thread
// that issues the products.  Keys and values have two slots each in shared
// memory, rows of 128 bytes in the 128-byte swizzle, [D / 64][128 rows]: the K
// operand is read K-major, and V, whose contraction index is the row, MN-major.
// Rows come from pages of any size, so they are brought by 16-byte asynchronous
// copies rather than by tile copies.
//
// Every wait is bounded: a wait that gives up marks the CTA dead, after which
// no wait waits, no product is issued, and every row that is still written is
// not a number (SDV_STATUS_TIMEOUT).
#include "k8_attn.cuh"

namespace sdv {
namespace {

using namespace attn;

constexpr int kThreads = 416;
constexpr int kRows = 128;               // rows of a stream
constexpr int MT = 2 * kRows, BN = 128;
constexpr int kBlock = BN * 128;         // bytes of 128 rows of 64 16-bit cells
constexpr int kTile = 2 * kBlock;        // ... of 128
constexpr uint32_t kPolls = 1u << 22;
constexpr float kSlack = 8.0f;           // how far (log2) scores may pass the reference

// Shared memory, bytes from its 1024-aligned start.
constexpr int kOffK = 0, kOffV = 2 * kTile, kOffQ = 4 * kTile;
constexpr int kOffRow = kOffQ + 2 * kTile;              // int64 [2][BN] byte offset of a row (-1: zeros)
constexpr int kOffFlag = kOffRow + 2 * BN * 8;          // uint32 [2][4] values that are not numbers
constexpr int kOffBar = kOffFlag + 2 * 4 * 4;
constexpr int kBars = 18;
constexpr int kSmem = kOffBar + kBars * 8 + 1024;

enum Bar { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kQFull = 8, kSFull = 10, kPFull = 12, kOFull = 14, kEnd = 16 };

struct Sync {
    uint64_t* bar;
    volatile int* dead;
    unsigned* status;
    __device__ __forceinline__ void wait(int i, uint32_t parity) const {
        const uint32_t addr = smem_u32(bar + i);
        for (uint32_t n = 0; n < kPolls; ++n) {
            uint32_t done;
            asm volatile(
                "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(done) : "r"(addr), "r"(parity) : "memory");
            if (done) return;
            if (*dead) return;
        }
        *dead = 1;
        if (status) atomicOr(status, kStatusTimeout);
    }
    __device__ __forceinline__ void arrive(int i) const {
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar + i)) : "memory");
    }
    __device__ __forceinline__ void commit(int i) const {
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar + i)) : "memory");
    }
};

__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// 32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(float (&x)[32], uint32_t addr) {
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_ld16(float (&x)[16], uint32_t addr) {
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const float (&x)[32]) {
    const uint32_t* r = reinterpret_cast<const uint32_t*>(x);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand: 128-byte swizzle, `lbo` / `sbo` bytes between 64-cell
// column blocks (MN-major) and between groups of eight rows.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
           (static_cast<uint64_t>(sbo >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t x, uint64_t y, uint32_t idesc, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(x), "l"(y), "r"(idesc),
                 "r"(static_cast<uint32_t>(add)) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t x, uint64_t y, uint32_t idesc, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(x), "l"(y), "r"(idesc),
                 "r"(static_cast<uint32_t>(add)) : "memory");
}

// Byte offset of 16-byte chunk c of row r in a tile.
__device__ __forceinline__ int chunk_at(int r, int c) { return (c >> 3) * kBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4); }

// Which of the 32 positions from pos0 on a live row sees, as bits.
__device__ __forceinline__ uint32_t sees(const AttnArgs& a, const Unit& u, int node, const int32_t* row, int pos0) {
    const int base = pos0 - u.cut.ctx;               // node of the first one
    if (base + 32 <= 0) return 0xffffffffu;
    uint32_t bits;
    if (!row) {
        const int n = node - base + 1;
        bits = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
    } else if (base < 0) {
        bits = (static_cast<uint32_t>(__ldg(row)) << -base) | ((1u << -base) - 1u);
    } else {
        const int w = base >> 5;
        const uint32_t lo = w < a.W ? static_cast<uint32_t>(__ldg(row + w)) : 0u;
        const uint32_t hi = w + 1 < a.W ? static_cast<uint32_t>(__ldg(row + w + 1)) : 0u;
        bits = __funnelshift_r(lo, hi, base & 31);
    }
    const int left = u.cut.cnt - base;               // nodes from the first one on
    if (left < 32) bits &= left <= 0 ? 0u : (1u << left) - 1u;
    return bits;
}

template <bool F16>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const AttnArgs a) {
    extern __shared__ unsigned char raw[];
    unsigned char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    int64_t* s_row = reinterpret_cast<int64_t*>(smem + kOffRow);
    uint32_t* s_flag = reinterpret_cast<uint32_t*>(smem + kOffFlag);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
    __shared__ int64_t s_part[40];
    __shared__ uint32_t s_tmem;
    __shared__ int s_dead;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mts = (a.N * a.g + MT - 1) / MT;
    const int D = a.c.D;
    const Sync sync{bars, &s_dead, a.status};
    if (tid == 0) {
        s_dead = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + kKFull + i, 4);
            mbar_init(bars + kKEmpty + i, 1);
            mbar_init(bars + kVFull + i, 4);
            mbar_init(bars + kVEmpty + i, 1);
            mbar_init(bars + kQFull + i, kRows);
            mbar_init(bars + kSFull + i, 1);
            mbar_init(bars + kPFull + i, kRows);
            mbar_init(bars + kOFull + i, 1);
        }
        mbar_init(bars + kEnd, 1);
        a.desc[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    if (tid < 8) s_flag[tid] = 0;
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const Part part = find_part<MT, BN, kThreads>(a, mts, s_part);      // holds barriers of the CTA
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;
    Walk<MT, BN> walk;
    walk.start(a, part, mts);
    Unit u;

    if (warp < 8) {
        // ---------------- softmax of one stream, a thread per row ----------------
        const int st = warp >> 2, r = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + st * 128, tO = tmem + lanes + 256 + st * 128;
        const float c = fabsf(a.scale_log2);
        const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
        uint32_t n = 0;                              // tiles of this stream so far
        uint32_t nv = 0;                             // tiles of the CTA so far
        while (walk.next(a, part, u)) {
            const int nt = u.len > 0 ? u.t1 - u.t0 : 0;
            const int first_row = u.mt * MT + st * kRows;
            const int row = first_row + r, node = row / a.g;
            const bool live = node < u.cut.cnt;
            const bool run = nt > 0 && first_row / a.g < u.cut.cnt;     // the stream has a live row
            if (tid == 0) {
                if (u.t0 > 0) write_desc(a, part, u);
                if (u.cut.bad && a.status) atomicOr(a.status, kStatusBadLength);
            }
            float m = -INFINITY, l = 0.0f;
            bool nan_row = false;
            if (run) {
                unsigned char* qs = smem + kOffQ + st * kTile;
                const unsigned char* p = a.q + u.b * a.q_sb + node * a.q_sn +
                                         (static_cast<int64_t>(u.h) * a.g + row % a.g) * a.q_sh;
                const bool aligned = (reinterpret_cast<uintptr_t>(p) & 15) == 0;
                for (int ch = 0; ch < D / 8; ++ch) {
                    uint32_t v[4] = {0, 0, 0, 0};
                    if (live && aligned) {
                        const uint4 x = *reinterpret_cast<const uint4*>(p + ch * 16);
                        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
                    } else if (live) {
                        const unsigned short* hp = reinterpret_cast<const unsigned short*>(p + ch * 16);
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = hp[2 * i] | (static_cast<uint32_t>(hp[2 * i + 1]) << 16);
                    }
                    *reinterpret_cast<uint4*>(qs + chunk_at(r, ch)) = make_uint4(v[0] ^ flip, v[1] ^ flip, v[2] ^ flip, v[3] ^ flip);
                }
                fence_async();
                sync.arrive(kQFull + st);
                // pages that are not the cache's: looked for once, a slow path if there are any
                const int32_t* table = a.table + static_cast<int64_t>(u.b) * a.max_pages;
                const int pos_end = min(u.t1 * BN, u.len);
                int bad = 0;
                for (int pg = u.t0 * BN / a.c.P + r; pg <= (pos_end - 1) / a.c.P; pg += kRows) {
                    const int x = __ldg(table + pg);
                    bad |= x < 0 || x >= a.c.pages;
                }
                int any_bad;
                asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.red.or.pred q, %2, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
                             : "=r"(any_bad) : "r"(bad), "r"(2 + st) : "memory");
                if (any_bad && r == 0 && a.status) atomicOr(a.status, kStatusBadPage);
                const int32_t* mrow = a.mask && live ? a.mask + u.b * a.mask_sb + static_cast<int64_t>(node) * a.W : nullptr;

                for (int t = 0; t < nt; ++t, ++n) {
                    const int pos0 = (u.t0 + t) * BN;
                    const bool mixed = pos0 + BN > u.cut.ctx;       // some rows see a column and some do not
                    uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
                    if (mixed) {
                        sync.wait(kVFull + ((nv + t) & 1), (nv + t) >> 1 & 1);
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            see[i] = live ? sees(a, u, node, mrow, pos0 + 32 * i) : 0u;
                            if (see[i] & s_flag[((nv + t) & 1) * 4 + i]) nan_row = true;
                        }
                    }
                    if (any_bad) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            for (int y = 0; y < 32; ++y) {
                                const int pos = pos0 + 32 * i + y;
                                if (pos >= u.len || !(see[i] >> y & 1)) continue;
                                const int pg = __ldg(table + pos / a.c.P);
                                nan_row |= pg < 0 || pg >= a.c.pages;
                            }
                    }
                    sync.wait(kSFull + st, n & 1);
                    __syncwarp();
                    fence_after();
                    float x[32];
                    float top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        tmem_ld32(x, tS + 32 * i);
                        if (mixed) {
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                if (see[i] >> y & 1) top = fmaxf(top, x[y]);
                        } else {
                            float t4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                            for (int y = 4; y < 32; ++y) t4[y & 3] = fmaxf(t4[y & 3], x[y]);
                            top = fmaxf(top, fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])));
                        }
                    }
                    top = top == -INFINITY ? top : top * c;
                    // the reference moves when the scores pass it by far
                    const bool move = top > m + kSlack || (m == -INFINITY && top != -INFINITY);
                    if (t > 0 && __any_sync(0xffffffffu, move)) {
                        const float by = move ? ex2(m - top) : 1.0f;
                        sync.wait(kOFull + st, (n - 1) & 1);        // the product before has been added
                        __syncwarp();
                        fence_after();
                        l *= by;
                        for (int i = 0; i < D; i += 32) {           // columns past D hold nothing of use
                            float o[32];
                            tmem_ld32(o, tO + i);
#pragma unroll
                            for (int y = 0; y < 32; ++y) o[y] *= by;
                            tmem_st32(tO + i, o);
                        }
                        tmem_wait_st();
                    }
                    if (move) m = top;
                    const float sub = m == -INFINITY ? 0.0f : m;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        tmem_ld32(x, tS + 32 * i);
                        uint32_t p2[16];
                        float sum0 = 0.0f, sum1 = 0.0f;
                        if (mixed) {
#pragma unroll
                            for (int y = 0; y < 32; ++y) x[y] = see[i] >> y & 1 ? ex2(fmaf(x[y], c, -sub)) : 0.0f;
                        } else {
#pragma unroll
                            for (int y = 0; y < 32; ++y) x[y] = ex2(fmaf(x[y], c, -sub));
                        }
#pragma unroll
                        for (int y = 0; y < 16; ++y) {
                            sum0 += x[2 * y], sum1 += x[2 * y + 1];
                            p2[y] = pack2<F16>(x[2 * y], x[2 * y + 1]);
                        }
                        l += sum0 + sum1;
                        tmem_st16(tS + 16 * i, p2);                  // over columns that have been read
                    }
                    tmem_wait_st();
                    fence_before();
                    sync.arrive(kPFull + st);
                }
                sync.wait(kOFull + st, (n - 1) & 1);
                __syncwarp();
                fence_after();
                if (*sync.dead) nan_row = true;
            }
            nv += nt;

            // the row: its output, or its part of one (the TMEM reads are the warp's)
            const float nanv = __int_as_float(0x7fc00000);
            if (nan_row || u.cut.bad) l = nanv;
            const bool empty = l == 0.0f || (!live && !u.cut.bad);
            const float inv = empty ? 0.0f : 1.0f / l;
            const float log2sum = u.cut.bad ? nanv : empty ? -INFINITY : m + log2f(l);
            const bool whole = u.t0 == 0 && u.t1 == u.tiles, mine = node < a.N;
            const int64_t orow = (static_cast<int64_t>(u.b) * a.N + node) * a.Hq + u.h * a.g + row % a.g;
            float* prow = part_rows(a, blockIdx.x, u.t0 > 0 ? 0 : 1, MT);
            if (mine && whole && a.lse) a.lse[orow] = log2sum * kLn2;
            if (mine && !whole) prow[MT * D + st * kRows + r] = log2sum;
            unsigned short* dst = static_cast<unsigned short*>(a.out) + orow * D;
            float* pdst = prow + (st * kRows + r) * D;
            for (int i = 0; i < D; i += 16) {
                float o[16];
#pragma unroll
                for (int y = 0; y < 16; ++y) o[y] = 0.0f;
                __syncwarp();
                if (run) tmem_ld16(o, tO + i);
                if (!mine) continue;
#pragma unroll
                for (int y = 0; y < 16; ++y) o[y] = empty ? 0.0f : o[y] * inv;
                if (whole) {
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        reinterpret_cast<uint4*>(dst + i)[y] =
                            make_uint4(pack2<F16>(o[8 * y], o[8 * y + 1]), pack2<F16>(o[8 * y + 2], o[8 * y + 3]),
                                       pack2<F16>(o[8 * y + 4], o[8 * y + 5]), pack2<F16>(o[8 * y + 6], o[8 * y + 7]));
                } else {
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        reinterpret_cast<float4*>(pdst + i)[y] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
                }
            }
            __syncwarp();
            fence_before();
        }
    } else if (warp < 12) {
        // ---------------- loads ----------------
        const int p = tid - 256;                     // row of a tile, and thread of the copies
        const int CH = D / 8;                        // 16-byte chunks of a row
        uint32_t tiles = 0;                          // tiles of the CTA so far
        const int pr = p / 16, pc = p % 16;          // chunk pc of rows pr, pr + 8, ...
        // what the copies under way hold, for when they are in: is it V, its slot,
        // and the first row that some rows do not see
        bool pend_v = false;
        int pend_slot = 0, pend_from = BN;
        bool pending = false;
        auto settle = [&]() {                        // the pending copies are in: look at them, hand them over
            if (!pending) return;
            if (pend_v && pend_from < BN) {          // values that are not numbers are kept out of the products
                for (int i = 0; i < BN / 8; ++i) {
                    const int r = pr + 8 * i;
                    unsigned char* at = smem + kOffV + pend_slot * kTile + chunk_at(r, pc);
                    bool bad = false;
                    if (r >= pend_from && pc < CH) {
                        const uint4 v = *reinterpret_cast<const uint4*>(at);
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                        constexpr uint32_t top = F16 ? 0x7c00u : 0x7f80u;
#pragma unroll
                        for (int y = 0; y < 4; ++y) bad |= (w[y] & top) == top || (w[y] >> 16 & top) == top;
                    }
                    const uint32_t who = __ballot_sync(0xffffffffu, bad) & (0xffffu << (lane & 16));
                    if (who) {
                        if (pc < CH) *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
                        if (pc == 0) atomicOr(s_flag + pend_slot * 4 + (r >> 5), 1u << (r & 31));
                    }
                }
            }
            fence_async();
            __syncwarp();
            if (lane == 0) sync.arrive((pend_v ? kVFull : kKFull) + pend_slot);
            pending = false;
        };
        while (walk.next(a, part, u)) {
            const int nt = u.len > 0 ? u.t1 - u.t0 : 0;
            const int32_t* table = a.table + static_cast<int64_t>(u.b) * a.max_pages;
            auto fetch = [&](int t) {
                const int pos = (u.t0 + t) * BN + p;
                return t < nt && pos < u.len ? __ldg(table + pos / a.c.P) : -1;
            };
            int page = fetch(0);
            for (int t = 0; t < nt; ++t, ++tiles) {
                const int pos0 = (u.t0 + t) * BN, pos = pos0 + p, slot = tiles & 1;
                s_row[slot * BN + p] =
                    page >= 0 && page < a.c.pages
                        ? page * a.c.page_stride + (static_cast<int64_t>(u.h) * a.c.P + pos % a.c.P) * D * 2 : -1;
                page = fetch(t + 1);
                bar_sync(1, 128);
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv) {
                    sync.wait((kv ? kVEmpty : kKEmpty) + slot, (tiles >> 1 & 1) ^ 1);
                    __syncwarp();
                    if (kv && pos0 + BN > u.cut.ctx) {              // flags are looked at in such tiles only
                        if (p < 4) s_flag[slot * 4 + p] = 0;
                        bar_sync(1, 128);
                    }
                    const unsigned char* src = kv ? a.c.v : a.c.k;
                    const uint32_t dst = smem_u32(smem + (kv ? kOffV : kOffK) + slot * kTile);
                    if (pc < CH) {
#pragma unroll 4
                        for (int i = 0; i < BN / 8; ++i) {
                            const int r = pr + 8 * i;
                            const int64_t off = s_row[slot * BN + r];
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + chunk_at(r, pc)),
                                         "l"(src + (off < 0 ? 0 : off + pc * 16)), "r"(off < 0 ? 0 : 16) : "memory");
                        }
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    if (pending) {
                        asm volatile("cp.async.wait_group 1;" ::: "memory");
                        settle();
                    }
                    pending = true;
                    pend_v = kv != 0;
                    pend_slot = slot;
                    pend_from = min(max(u.cut.ctx - pos0, 0), BN);
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        settle();
    } else if (lane == 0) {
        // ---------------- products ----------------
        constexpr uint32_t type = F16 ? 0u : 1u;
        const uint32_t common = (1u << 4) | (type << 7) | (type << 10) | (8u << 24);    // fp32 += 16 bits, 128 rows
        const uint32_t idesc_s = common | (static_cast<uint32_t>(BN / 8) << 17);
        const uint32_t idesc_o = common | (1u << 16) | (static_cast<uint32_t>(D / 8) << 17);    // V is MN-major
        const uint32_t k0 = smem_u32(smem + kOffK), v0 = smem_u32(smem + kOffV), q0 = smem_u32(smem + kOffQ);
        uint32_t n[2] = {0, 0}, q[2] = {0, 0}, tiles = 0;
        auto scores = [&](int s, uint32_t tile) {
            if (*sync.dead) return;
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = (ks >> 2) * kBlock + (ks & 3) * 32;
                mma_ss(tmem + s * 128, operand(q0 + s * kTile + off, 16, 1024),
                       operand(k0 + (tile & 1) * kTile + off, 16, 1024), idesc_s, ks > 0);
            }
        };
        while (walk.next(a, part, u)) {
            const int nt = u.len > 0 ? u.t1 - u.t0 : 0;
            if (nt == 0) continue;
            // stream s has a live row (stream 0 has one in every unit with tiles)
            const int streams = (u.mt * MT + kRows) / a.g < u.cut.cnt ? 2 : 1;
            sync.wait(kKFull + (tiles & 1), tiles >> 1 & 1);
            for (int s = 0; s < streams; ++s) {
                sync.wait(kQFull + s, q[s]++ & 1);
                fence_after();
                scores(s, tiles);
                sync.commit(kSFull + s);
            }
            sync.commit(kKEmpty + (tiles & 1));
            for (int t = 0; t < nt; ++t, ++tiles) {
                const bool more = t + 1 < nt;
                for (int s = 0; s < streams; ++s) {
                    sync.wait(kPFull + s, n[s]++ & 1);
                    if (s == 0) sync.wait(kVFull + (tiles & 1), tiles >> 1 & 1);
                    fence_after();
                    if (!*sync.dead) {
                        for (int ks = 0; ks < BN / 16; ++ks)
                            mma_ts(tmem + 256 + s * 128, tmem + s * 128 + ks * 8,
                                   operand(v0 + (tiles & 1) * kTile + ks * 2048, kBlock, 1024), idesc_o, t > 0 || ks > 0);
                    }
                    sync.commit(kOFull + s);
                    if (more) {
                        if (s == 0) {
                            sync.wait(kKFull + ((tiles + 1) & 1), (tiles + 1) >> 1 & 1);
                            fence_after();
                        }
                        scores(s, tiles + 1);
                        sync.commit(kSFull + s);
                    }
                }
                sync.commit(kVEmpty + (tiles & 1));
                if (more) sync.commit(kKEmpty + ((tiles + 1) & 1));
            }
        }
        sync.commit(kEnd);                           // nothing is under way any more
        sync.wait(kEnd, 0);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 12) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <bool F16> cudaError_t launch(AttnArgs a, int nsm, cudaStream_t s) {
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(attn_tc_kernel<F16>), kSmem);
    if (e != cudaSuccess) return e;
    a.ctas = nsm;
    attn_tc_kernel<F16><<<static_cast<unsigned>(nsm), kThreads, kSmem, s>>>(a);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_attn_combine(a, F16, MT, s);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs& a, bool f16, int nsm, cudaStream_t s) {
    return f16 ? launch<true>(a, nsm, s) : launch<false>(a, nsm, s);
}

}  // namespace sdv
