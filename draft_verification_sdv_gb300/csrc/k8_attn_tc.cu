// k8_attn_tc.cu -- tree attention for many query rows (sdv_tree_attn) on the
// 5th-generation tensor cores.
//
// A tree of N nodes has N * g query rows per kv head; from a few dozen rows on
// the two contractions bound the step, not the cache's bytes.  A CTA works on
// 256 rows as two streams of 128 (the rows of one tcgen05.mma), so that while
// the softmax of one stream runs, the tensor cores multiply for the other:
//   S_s = Q_s K^T        operands in shared memory, accumulator in TMEM
//   P_s = 2^(c S_s - m)  a thread per row takes its 128 scores into registers
//                        and writes P_s over S_s, 16 bits wide as the products
//                        want it (half a step of that type off, relative; the sum
//                        of the row adds them up in fp32 as they were)
//   O_s += P_s V         P_s from TMEM, V from shared memory, O_s in TMEM
// TMEM holds S_0, S_1, O_0, O_1: 4 x 128 columns, all 512.  P could go through
// shared memory, where a product takes 65 clocks instead of 100; but two
// operands there use all of the shared memory's bandwidth, and every barrier
// and store of the other warps then waits (1547 us against 1276 us for 16 trees
// of 513 nodes, when both were built).
//
// O is not rescaled each time the maximum grows: the running reference m only
// moves when a row's scores pass it by 2^8 (fp32 sums and 16-bit probabilities
// keep their relative precision below that), and then the row's warp rescales.
//
// Warps 0-3 and 4-7: softmax of stream 0 and 1; 8-10: loads; 11: one thread
// that issues the products.  Tiles of 128 positions, keys and values in turn,
// go through a ring of slots in shared memory, as rows of 128 bytes in the
// 128-byte swizzle, [D / 64][128 rows]: the K operand is read K-major, and V,
// whose contraction index is the row, MN-major.  They come by tile copies (TMA),
// one per page and column block and a lane to each, so that pages may be of any
// size that is a multiple of 8 rows: warp 8 brings the keys and warp 9 the
// values, and warp 10 hands a tile over, after a look at the values of rows that
// some queries do not see (what is not a number there must not meet a zero
// probability in a product).  e4m3 rows land as they are in the upper half of
// their slot; then warp 8 brings both, and all three hand over, after widening
// the rows in place to the queries' type, times their power of two.  bf16 holds that
// as it is; fp16 does not where a power is far from 1.  A block that meets such a
// row says so, and launch_attn_redo then takes the call's place, with the powers
// outside the products.
//
// What bounds it: the chain of one stream's step, softmax (2230 clocks for two
// streams' tiles, a third of them the 2^x), P V (430) and S (640) and the waits
// between them (440), 3740 clocks for two tiles where the products alone take
// 2100 (counted when 16 trees took 840 us).  16 trees of 513 nodes over 1500 to
// 3500 positions, 8 x 8 heads of 128: 780 us, 855 TFLOP/s; 3 chunks of 1900 tokens,
// 8 x 4 heads of 64: 232 us.  e4m3 rows: 2700 clocks and more to widen a tile (682 us
// against 280 us for 4 chains of 513 nodes behind 4000 positions).  Seven warps for
// it have too few registers, and rows that land beside their slots leave too few
// slots: both were slower.  Short units: some 11000 clocks from one to the next, of
// which the rows' way to memory is 4000.
//
// Every wait is bounded: a wait that gives up marks the CTA dead, after which
// no wait waits, no copy is begun, and every row with something to see that is
// still written is not a number (SDV_STATUS_TIMEOUT).
#include "k8_attn_tma.cuh"

namespace sdv {
namespace {

using namespace attn;

constexpr int kThreads = 384;
constexpr int kRegs = 168;               // per thread at launch
constexpr int kRows = 128;               // rows of a stream
constexpr int MT = 2 * kRows, BN = 128;
constexpr int kBlock = BN * 128;         // bytes of 128 rows of 64 16-bit cells
constexpr int kTile = 2 * kBlock;        // ... of 128
constexpr int kLoadWarps = 3, kLoadThreads = 32 * kLoadWarps;
constexpr float kSlack = 8.0f;           // how far (log2) scores may pass the reference

// Shared memory, bytes from its 1024-aligned start.
constexpr int kKeySlots = 3, kValueSlots = 2, kSlots = kKeySlots + kValueSlots;

// Where a softmax warp is: kept in shared memory, its registers hold scores.
struct SoftmaxState {
    Walk<MT, BN> walk;
    Unit u;
};

struct Smem {
    static constexpr int q = kSlots * kTile;
    static constexpr int exps = q + 2 * kTile;                  // bytes [3 tiles][keys, values][BN] (e4m3)
    static constexpr int flag = exps + 6 * BN;                  // uint32 [4 tiles][3 warps][4] values that are not numbers
    static constexpr int bar = flag + 4 * kLoadWarps * 4 * 4;
    static constexpr int word = bar + 20 * 8;                   // TMEM address, dead, rows that fp16 does not hold
    static constexpr int state = word + 16;                     // SoftmaxState [8 warps]
    static constexpr int bytes = state + 8 * static_cast<int>(sizeof(SoftmaxState)) + 1024;
};
static_assert(Smem::bytes <= 227 * 1024, "one CTA per SM");

// Barriers: two per stream of each kind, one for the end, and the tiles'.  Tile T
// (of the CTA's, through all its units) has its keys in slot T % 3 and its
// values in slot 3 + T % 2.  The values of a tile and the keys of the next one
// are used and freed together: full(T) says that K(T) and V(T - 1) are there,
// free(T) that S(T + 1) and the outputs of tile T are done, so that V(T + 2) and
// K(T + 3) may come.  Few barriers, because each is a round trip through a
// shared memory that the products keep busy (200 clocks and more).
enum Bar { kQFull = 0, kQEmpty = 2, kSFull = 4, kPFull = 6, kOFull = 8, kEnd = 10, kFull = 11, kFree = 13, kLand = 15,
           kBars = kLand + kSlots };

static_assert(Smem::word == Smem::bar + kBars * 8, "a place for each barrier");

__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tma_load_q(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int head, int node, int b) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(head), "r"(node), "r"(b) : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

#define SDV_R4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define SDV_R16(r, i) SDV_R4(r, i), SDV_R4(r, i + 4), SDV_R4(r, i + 8), SDV_R4(r, i + 12)
#define SDV_I4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
#define SDV_I16(r, i) SDV_I4(r, i), SDV_I4(r, i + 4), SDV_I4(r, i + 8), SDV_I4(r, i + 12)

// 128 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld128(float (&x)[128], uint32_t addr) {
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%128];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,%80,%81,"
        "%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,"
        "%108,%109,%110,%111,%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%129];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : SDV_R16(r, 0), SDV_R16(r, 16), SDV_R16(r, 32), SDV_R16(r, 48), SDV_R16(r, 64), SDV_R16(r, 80), SDV_R16(r, 96),
          SDV_R16(r, 112) : "r"(addr), "r"(addr + 64) : "memory");
}
__device__ __forceinline__ void tmem_ld16(float (&x)[16], uint32_t addr) {
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : SDV_R16(r, 0) : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        SDV_I16(r, 0) : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand: 128-byte swizzle, `lbo` bytes between 64-cell column
// blocks (MN-major), 1024 between groups of eight rows.  Moving it by a number
// of bytes adds a sixteenth of them to the low word.
__device__ __forceinline__ uint32_t operand_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); }
constexpr uint32_t kOperandHi = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t x, uint32_t y, uint32_t idesc, uint32_t add) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d), "r"(x), "r"(y), "r"(idesc), "r"(add),
                 "r"(kOperandHi) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t x, uint32_t y, uint32_t idesc, uint32_t add) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.u32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d), "r"(x), "r"(y), "r"(idesc), "r"(add),
                 "r"(kOperandHi) : "memory");
}

// Two fp32 operations at once.
struct F2 { float x, y; };
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Byte offset of 16-byte chunk c of row r in a tile.
__device__ __forceinline__ int chunk_at(int r, int c) { return (c >> 3) * kBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4); }

// A whole sector at once: the rows of a warp lie apart, and each store of it
// takes a turn per row at a memory pipe that the products keep busy.
__device__ __forceinline__ void store32(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f, uint32_t g,
                                        uint32_t h) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(f),
                 "r"(g), "r"(h) : "memory");
}

// The mask words that hold nodes base .. base + 127 of a row.
__device__ __forceinline__ void mask_words(const AttnArgs& a, const int32_t* row, int base, uint32_t (&w)[5]) {
    const int w0 = base >> 5;                        // floor
#pragma unroll
    for (int i = 0; i < 5; ++i)
        w[i] = w0 + i < 0 ? 0xffffffffu : w0 + i < a.W ? static_cast<uint32_t>(__ldg(row + w0 + i)) : 0u;
}

// Which of the positions pos0 + 32 i .. + 31 a live row sees, as bits: all
// committed ones (word 0xffffffff before the mask's first), then its mask's.
__device__ __forceinline__ uint32_t sees(const Unit& u, bool tree, int node, const uint32_t (&w)[5], int pos0, int i) {
    const int base = pos0 - u.cut.ctx, b = base + 32 * i;
    uint32_t bits;
    if (tree) {
        bits = __funnelshift_r(w[i], w[i + 1], base & 31);
    } else {
        const int n = node - b + 1;
        bits = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
    }
    const int left = u.cut.cnt - b;                  // nodes from the first position on
    if (left < 32) bits &= left <= 0 ? 0u : (1u << left) - 1u;
    return bits;
}

// A thread's row of queries into its place, with the sign turned where flip is
// set: copies that are still under way if it lies on 16 bytes.
__device__ __noinline__ void copy_row(const unsigned char* src, bool there, uint32_t flip, unsigned char* qs, int r, int chunks) {
    const bool plain = flip == 0 && (reinterpret_cast<uintptr_t>(src) & 15) == 0;
    for (int c = 0; c < chunks; ++c, src += 16) {
        unsigned char* dst = qs + chunk_at(r, c);
        if (!there) {
            *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
        } else if (plain) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
        } else {
            const unsigned short* e = reinterpret_cast<const unsigned short*>(src);
            *reinterpret_cast<uint4*>(dst) =
                make_uint4((e[0] | static_cast<uint32_t>(e[1]) << 16) ^ flip, (e[2] | static_cast<uint32_t>(e[3]) << 16) ^ flip,
                           (e[4] | static_cast<uint32_t>(e[5]) << 16) ^ flip, (e[6] | static_cast<uint32_t>(e[7]) << 16) ^ flip);
        }
    }
}

// Whether a row sees a position on a page that is not the cache's.
__device__ __noinline__ bool sees_bad_page(const int32_t* table, int pages, int P, uint4 see, int pos0, int len) {
    bool bad = false;
    for (int i = 0; i < BN && pos0 + i < len; ++i) {
        const int pg = __ldg(table + (pos0 + i) / P);
        const uint32_t w = i < 32 ? see.x : i < 64 ? see.y : i < 96 ? see.z : see.w;
        bad |= (w >> (i & 31) & 1) && (pg < 0 || pg >= pages);
    }
    return bad;
}

// Sixteen e4m3 cells times 2^(e - 127), in the queries' type; `beyond` is set where
// that is fp16, which does not hold them as they are.
template <bool F16> __device__ __forceinline__ void widen16(const uint4& raw, int e, uint32_t (&o)[8], bool& beyond) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    // a cell that is not a number takes its chunk with it
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= ((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    if (bad) e = 255;
    if constexpr (F16) {
        // 2^(e - 127) as the product of two fp16 powers (its range is smaller)
        int h = e - 127;
        // (beyond 2^30 every cell but zero is infinite, below 2^-34 none is left)
        h = h < -34 ? -34 : h > 30 ? 30 : h;
        const int h1 = h / 2, h2 = h - h1;
        uint32_t s1 = static_cast<uint32_t>(h1 + 15) << 10, s2 = static_cast<uint32_t>(h2 + 15) << 10;
        if (h1 < -14) s1 = 0x0400u >> (-14 - h1);
        if (h2 < -14) s2 = 0x0400u >> (-14 - h2);
        if (e == 255) s1 = 0x7e00u;
        s1 |= s1 << 16, s2 |= s2 << 16;
        // the way back (to 2^15 a step) gives the cells, unless digits went missing
        const uint32_t r1 = (h1 < -15 ? 30u : 15u - h1) << 10, r2 = (h2 < -15 ? 30u : 15u - h2) << 10;
        uint32_t off = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t lost;
            asm("{\n\t.reg .b16 lo, hi;\n\t.reg .b32 t, u;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 t, lo;\n\t"
                "mul.rn.f16x2 u, t, %3;\n\tmul.rn.f16x2 %0, u, %4;\n\t"
                "mul.rn.f16x2 u, %0, %5;\n\tmul.rn.f16x2 u, u, %6;\n\txor.b32 %1, t, u;\n\t}"
                : "=&r"(o[i]), "=r"(lost)
                : "r"(w[i / 2] >> (16 * (i % 2))), "r"(s1), "r"(s2), "r"(r1 | r1 << 16), "r"(r2 | r2 << 16));
            off |= lost;
        }
        beyond |= e != 255 && off != 0;
    } else {
        // the cell's exponent and digits in bf16's places are its value times 2^-120
        uint32_t s = e == 255 ? 0x7fc0u : e == 0 ? 0x0040u : static_cast<uint32_t>(e) << 7;
        s |= s << 16;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t t = __byte_perm(w[i / 2], 0, i % 2 ? 0x3424 : 0x1404);    // the bytes on top of 16 bits
            const uint32_t v = (t & 0x80008000u) | ((t >> 4) & 0x07f007f0u);
            asm("{\n\t.reg .b32 t;\n\tmul.rn.bf16x2 t, %1, %2;\n\tmul.rn.bf16x2 %0, t, %3;\n\t}"
                : "=r"(o[i]) : "r"(v), "r"(0x7b807b80u), "r"(s));
        }
    }
}

// The same for the usual powers, those that one 16-bit factor holds: half the work.
template <bool F16> __device__ __forceinline__ bool usual_power(int e) { return F16 ? e >= 113 && e <= 134 : e <= 134; }
__device__ __forceinline__ bool has_nan(const uint4& v) {
    return ((((v.x & 0x7f7f7f7fu) + 0x01010101u) | ((v.y & 0x7f7f7f7fu) + 0x01010101u) | ((v.z & 0x7f7f7f7fu) + 0x01010101u) |
             ((v.w & 0x7f7f7f7fu) + 0x01010101u)) & 0x80808080u) != 0;
}
template <bool F16> __device__ __forceinline__ void widen16_usual(const uint4& raw, int e, uint32_t (&o)[8]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= ((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    uint32_t s = F16 ? static_cast<uint32_t>(e - 112) << 10 : static_cast<uint32_t>(e + 120) << 7;
    if (bad) s = F16 ? 0x7e00u : 0x7fc0u;
    s = __byte_perm(s, 0, 0x1010);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F16) {
            asm("{\n\t.reg .b16 lo, hi;\n\t.reg .b32 t, u;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 t, lo;\n\t"
                "cvt.rn.f16x2.e4m3x2 u, hi;\n\tmul.rn.f16x2 %0, t, %3;\n\tmul.rn.f16x2 %1, u, %3;\n\t}"
                : "=r"(o[2 * i]), "=r"(o[2 * i + 1]) : "r"(w[i]), "r"(s));
        } else {
            // high and low bytes of the cells' bits in bf16's places
            const uint32_t hi = (w[i] & 0x80808080u) | ((w[i] >> 4) & 0x07070707u), lo = (w[i] << 4) & 0xf0f0f0f0u;
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o[2 * i]) : "r"(__byte_perm(lo, hi, 0x5140)), "r"(s));
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o[2 * i + 1]) : "r"(__byte_perm(lo, hi, 0x7362)), "r"(s));
        }
    }
}

// Whether rows from `from` on of a tile of 16-bit cells hold what is not a number:
// times zero, it adds one that stays.  A warp reads the rows as they lie: the
// swizzle keeps a row's chunks in the row, and columns past D are zeros.
template <bool F16> __device__ __forceinline__ bool odd_values(const unsigned char* base, int from, int blocks, int lane) {
    uint32_t acc[4] = {0, 0, 0, 0};
    for (int b = 0; b < blocks; ++b) {
        const unsigned char* at = base + b * kBlock + lane * 16;
#pragma unroll 4
        for (int i = from >> 2; i < BN / 4; ++i) {
            uint4 v = *reinterpret_cast<const uint4*>(at + i * 512);
            if (4 * i + (lane >> 3) < from) v = make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                if constexpr (F16)
                    asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc[y]) : "r"(w[y]), "r"(0));
                else
                    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[y]) : "r"(w[y]), "r"(0));
            }
        }
    }
    // (zeros of either sign otherwise)
    return __any_sync(0xffffffffu, ((acc[0] | acc[1] | acc[2] | acc[3]) & 0x7fff7fffu) != 0);
}

// BOXES: queries come by tile copies.  PARTS: rows may go out as fp32, or go on from others'
// (a.raw, a.far: shared prefixes); a kernel of its own, the others would be 3 % slower.
template <bool E4, bool F16, bool BOXES, bool PARTS>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
                                                              const __grid_constant__ CUtensorMap map_v,
                                                              const __grid_constant__ CUtensorMap map_q, int run_rows) {
    using M = Smem;
    extern __shared__ unsigned char raw[];
    unsigned char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint32_t* s_flag = reinterpret_cast<uint32_t*>(smem + M::flag);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::bar);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + M::word);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mts = (a.N * a.g + MT - 1) / MT;
    const int D = a.c.D;
    const Sync sync{smem_u32(bars), smem_u32(smem + M::word + 4), a.status, a.hooks ? kHookPolls : kPolls};
    if (tid == 0) {
        s_tmem[1] = s_tmem[2] = 0;                   // not dead, no such row
        for (int i = 0; i < 4 * kLoadWarps * 4; ++i) s_flag[i] = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + kQFull + i, BOXES ? 1 : kRows / 32);
            mbar_init(bars + kQEmpty + i, 1);
            mbar_init(bars + kSFull + i, 1);
            mbar_init(bars + kPFull + i, kRows / 32);    // a warp arrives once: 32 arrivals take turns
            mbar_init(bars + kOFull + i, 1);
        }
        mbar_init(bars + kEnd, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + kFull + i, E4 ? kLoadWarps : 1);
            mbar_init(bars + kFree + i, 1);
        }
        for (int i = 0; i < kSlots; ++i) mbar_init(bars + kLand + i, 1);
    }
    if (tid == 32) {                                 // on its way while the work is shared out
        prefetch_map(&map_k);
        prefetch_map(&map_v);
        if (BOXES) prefetch_map(&map_q);
    }
    if (warp == 11) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // the ring is not in use yet: its first bytes serve the search
    const Part part = find_part<MT, BN, kThreads>(a, mts, reinterpret_cast<int64_t*>(smem));
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *s_tmem;
    Walk<MT, BN> walk;
    walk.begin(a, part, mts);
    if (a.rounds > 0 && tid == 0) write_desc(a, part, walk);    // (its begins are in the ring)
    fence_async();                                   // what the search kept there comes before the tiles
    __syncthreads();                                 // the ring may be used

    // the softmax warps hold a row of scores: they take registers that the others
    // do not need (256 * kMore + 128 * kLess = 384 * 168, the launch's own; the
    // warps that bring e4m3 rows to 16 bits need some themselves)
    constexpr int kMore = E4 ? 184 : 200, kLess = E4 ? 136 : 104;
    static_assert(256 * kMore + 128 * kLess == kThreads * kRegs, "no more than the launch has");
    if (warp < 8)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMore) : "memory");
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLess) : "memory");
    if (warp < 8) {
        // ---------------- softmax of one stream, a thread per row ----------------
        const int st = warp >> 2, r = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + st * 128, tO = tmem + lanes + 256 + st * 128;
        // (a negative scale has turned the queries round); c > 0 so that -inf stays -inf
        const float c = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);
        uint32_t n = 0;                              // tiles of this stream so far
        uint32_t nv = 0, units = 0;                  // tiles of the CTA, units of this stream so far
        int seq = -1, any_bad = 0;
        SoftmaxState& state = reinterpret_cast<SoftmaxState*>(smem + M::state)[warp];
        Unit& u = state.u;
        if (lane == 0) state.walk = walk;
        if (a.rounds == 0 && tid == 0) write_desc(a, part, walk);
        // the next unit; and for a new sequence a look for pages that are not the
        // cache's: a slow path if there are any
        auto prepare = [&]() {
            int more = 0;
            if (lane == 0) more = state.walk.next(a, part, mts, u);
            __syncwarp();
            if (!__shfl_sync(0xffffffffu, more, 0)) return false;
            if (u.b != seq) {
                seq = u.b;
                const int32_t* table = a.table + static_cast<int64_t>(u.b) * a.max_pages;
                const int pages = (held_of(a, u.cut) + a.c.P - 1) / a.c.P;
                int bad = 0;
                for (int pg = r; pg < pages; pg += kRows) {
                    const int x = __ldg(table + pg);
                    bad |= x < 0 || x >= a.c.pages;
                }
                asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.red.or.pred q, %2, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
                             : "=r"(any_bad) : "r"(bad), "r"(2 + st) : "memory");
                if (any_bad && r == 0 && a.status) atomicOr(a.status, kStatusBadPage);
            }
            return true;
        };
        // queries that no box takes: each thread brings its row of the next unit (the
        // scores of the one before are done with theirs: their last tile was read)
        auto begin_queries = [&]() {
            const int first_row = u.mt * MT + st * kRows, row = first_row + r, node = row / a.g;
            if (u.len <= 0 || u.t1 <= u.t0 || first_row / a.g >= u.cut.cnt) return false;
            copy_row(q_of(a, u.b, node) + (static_cast<int64_t>(u.h) * a.g + row - node * a.g) * a.q_sh, node < u.cut.cnt,
                     a.scale_log2 < 0.0f ? 0x80008000u : 0u, smem + M::q + st * kTile, r, D / 8);
            return true;
        };
        auto end_queries = [&]() {
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async();
            __syncwarp();
            if (lane == 0) sync.arrive(kQFull + st);
        };
        bool more = prepare();
        if constexpr (!BOXES) {
            if (more && begin_queries()) end_queries();
        }
        while (more) {
            const int nt = u.len > 0 ? u.t1 - u.t0 : 0;
            const int first_row = u.mt * MT + st * kRows;
            const int row = first_row + r, node = row / a.g;
            const bool live = node < u.cut.cnt;
            const bool run = nt > 0 && first_row / a.g < u.cut.cnt;     // the stream has a live row
            if (tid == 0 && u.cut.bad && a.status) atomicOr(a.status, kStatusBadLength);
            float m = -INFINITY, l = 0.0f;
            bool nan_row = false;
            const bool begun = PARTS && a.far != nullptr && u.t0 == 0;    // rows go on from others' outputs
            if (PARTS && run && begun) {
                const int64_t from = (static_cast<int64_t>(u.b) * a.N + (live ? node : 0)) * a.Hq + u.h * a.g + row % a.g;
                const float L = live ? a.far_log[from] : -INFINITY;
                nan_row = L != L;
                const bool some = L > -INFINITY;     // (normalised: of a sum of 1 in units of 2^L)
                if (some) m = L, l = 1.0f;
                const float* src = a.far + from * D;
#pragma unroll 1
                for (int i = 0; i < D; i += 16) {
                    uint32_t o[16];
#pragma unroll
                    for (int y = 0; y < 16; y += 4) {
                        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (some) x = *reinterpret_cast<const float4*>(src + i + y);
                        o[y] = __float_as_uint(x.x), o[y + 1] = __float_as_uint(x.y), o[y + 2] = __float_as_uint(x.z), o[y + 3] = __float_as_uint(x.w);
                    }
                    __syncwarp();
                    tmem_st16(tO + i, o);
                }
                tmem_wait_st();
            }
            if (run) {
                const int32_t* table = a.table + static_cast<int64_t>(u.b) * a.max_pages;
                const int32_t* mrow = a.mask ? a.mask + u.b * a.mask_sb + static_cast<int64_t>(live ? node : 0) * a.W : nullptr;
                uint32_t words[5] = {0, 0, 0, 0, 0};
                // tiles from `plain` on hold positions that some rows see and some do not
                // (all of them go the long way where a page is bad)
                const int plain = any_bad ? 0 : min(max(min(seen_by_all<MT>(a, u.cut, u.mt), held_of(a, u.cut)) / BN - u.t0, 0), nt);
                if (mrow && plain == 0) mask_words(a, mrow, u.t0 * BN - u.cut.ctx, words);
                // scores to probabilities: the running maximum and sum, P over S
                auto weigh = [&](const float (&x)[128], bool first) {
                    float t4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int y = 4; y < 124; y += 8)
#pragma unroll
                        for (int z = 0; z < 4; ++z) t4[z] = max3(t4[z], x[y + z], x[y + 4 + z]);
                    float top = max3(max3(t4[0], x[124], x[125]), max3(t4[1], x[126], x[127]), fmaxf(t4[2], t4[3]));
                    top *= c;                        // (c > 0: -inf stays)
                    // the reference moves when the scores pass it by far
                    const bool move = top > m + kSlack || (m == -INFINITY && top != -INFINITY);
                    if (__any_sync(0xffffffffu, move)) {
                        if (!first) {
                            // (these scores were multiplied after the outputs of the tile before: both are done)
                            const float by = move ? ex2(m - top) : 1.0f;
                            l *= by;
#pragma unroll 1
                            for (int i = 0; i < D; i += 16) {
                                float o[16];
                                uint32_t o2[16];
                                tmem_ld16(o, tO + i);
#pragma unroll
                                for (int y = 0; y < 16; ++y) o2[y] = __float_as_uint(o[y] * by);
                                tmem_st16(tO + i, o2);
                            }
                        }
                        if (move) m = top;
                    }
                    const float sub = m == -INFINITY ? 0.0f : -m;
                    const F2 c2{c, c}, sub2{sub, sub};
                    float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        uint32_t pk[16];
#pragma unroll
                        for (int y = 0; y < 16; y += 2) {
                            const int z = 32 * h + 2 * y;
                            F2 v = fma2(F2{x[z], x[z + 1]}, c2, sub2);
                            F2 w = fma2(F2{x[z + 2], x[z + 3]}, c2, sub2);
                            v.x = ex2(v.x), v.y = ex2(v.y), w.x = ex2(w.x), w.y = ex2(w.y);
                            s4[0] += v.x, s4[1] += v.y, s4[2] += w.x, s4[3] += w.y;
                            pk[y] = pack2<F16>(v.x, v.y);
                            pk[y + 1] = pack2<F16>(w.x, w.y);
                        }
                        tmem_st16(tS + 16 * h, pk);
                    }
                    l += (s4[0] + s4[1]) + (s4[2] + s4[3]);
                };
                auto hand_over = [&]() {
                    tmem_wait_st();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) sync.arrive(kPFull + st);
                };
#pragma unroll 1
                for (int t = 0; t < nt; ++t, ++n) {
                    const bool mixed = t >= plain;
                    const int pos0 = (u.t0 + t) * BN;
                    uint32_t see[4] = {0, 0, 0, 0};
                    if (mixed) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) see[i] = live ? sees(u, mrow != nullptr, node, words, pos0, i) : 0u;
                        if (any_bad) nan_row |= sees_bad_page(table, a.c.pages, a.c.P, make_uint4(see[0], see[1], see[2], see[3]), pos0, u.len);
                    }
                    if (mrow && t + 1 >= plain && t + 1 < nt) mask_words(a, mrow, pos0 + BN - u.cut.ctx, words);
                    sync.wait(kSFull + st, n & 1);
                    __syncwarp();
                    fence_after();
                    float x[128];
                    tmem_ld128(x, tS);
                    if (mixed) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int y = 0; y < 32; ++y) x[32 * i + y] = see[i] >> y & 1 ? x[32 * i + y] : -INFINITY;
                    }
                    weigh(x, t == 0 && !begun);
                    if (mixed) {                     // values that are not numbers, among those that the row sees
                        const uint32_t T = nv + t;
                        sync.wait(kFull + ((T + 1) & 1), (T + 1) >> 1 & 1);
                        const uint32_t* f = s_flag + (T & 3) * (kLoadWarps * 4);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (see[i] & (f[i] | f[4 + i] | f[8 + i])) nan_row = true;
                        __syncwarp();
                    }
                    hand_over();
                }
            }
            nv += nt;

            // the row: its output, or its part of one.  What comes next is looked up
            // while the last products run; the TMEM reads are the warp's.
            const float nanv = __int_as_float(0x7fc00000);
            const bool whole = u.whole, ubad = u.cut.bad, mine = node < a.N;
            const int64_t orow = (static_cast<int64_t>(u.b) * a.N + node) * a.Hq + u.h * a.g + row % a.g;
            float* prow = part_rows(a, blockIdx.x, u.t0 > 0 ? 0 : 1, MT);
            __syncwarp();                            // every lane has read the unit
            more = prepare();
            bool coming = false;
            if constexpr (!BOXES) coming = more && begin_queries();
            if (run) {
                const bool done = sync.wait(kOFull + st, units++ & 1);
                __syncwarp();
                fence_after();
                if (!done || sync.is_dead()) nan_row = true;
            }
            if (coming) end_queries();
            if (nan_row || ubad) l = nanv;
            const bool empty = l == 0.0f || (!live && !ubad);
            const float inv = empty ? 0.0f : 1.0f / l;
            const float log2sum = ubad ? nanv : empty ? -INFINITY : m + log2f(l);
            const bool half = whole && !(PARTS && a.raw);      // 16-bit outputs
            if (mine && half && a.lse) a.lse[orow] = log2sum * kLn2;
            if (PARTS && mine && whole && a.raw) a.raw_log[orow] = log2sum;
            if (mine && !whole) prow[MT * D + st * kRows + r] = log2sum;
            unsigned short* dst = static_cast<unsigned short*>(a.out) + orow * D;
            float* pdst = PARTS && whole ? a.raw + orow * D : prow + (st * kRows + r) * D;
            for (int i = 0; i < D; i += 16) {
                float o[16];
#pragma unroll
                for (int y = 0; y < 16; ++y) o[y] = 0.0f;
                __syncwarp();
                if (run) tmem_ld16(o, tO + i);
                if (!mine) continue;
#pragma unroll
                for (int y = 0; y < 16; ++y) o[y] = empty ? 0.0f : o[y] * inv;
                if (half) {
                    store32(dst + i, pack2<F16>(o[0], o[1]), pack2<F16>(o[2], o[3]), pack2<F16>(o[4], o[5]), pack2<F16>(o[6], o[7]),
                            pack2<F16>(o[8], o[9]), pack2<F16>(o[10], o[11]), pack2<F16>(o[12], o[13]), pack2<F16>(o[14], o[15]));
                } else {
                    const uint32_t* q = reinterpret_cast<const uint32_t*>(o);
                    store32(pdst + i, q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7]);
                    store32(pdst + i + 8, q[8], q[9], q[10], q[11], q[12], q[13], q[14], q[15]);
                }
            }
            __syncwarp();
            fence_before();
        }
    } else if (warp < 11) {
        // ---------------- loads ----------------
        const int p = tid - 256, w = warp - 8;
        constexpr int kFirst = E4 ? 0 : 2, kSettle = kLoadWarps - kFirst;   // warps that hand tiles over
        constexpr int kBatch = E4 ? 6 : 1;
        const int CH = D / (E4 ? 16 : 8);            // 16-byte chunks of a row as it comes
        const int LR = CH > 8 ? 16 : CH > 4 ? 8 : 4; // lanes of a row
        const int RP = 32 / LR, lr = lane / LR, lc = lane % LR;     // rows of a warp's step
        const uint32_t group = ((1u << LR) - 1u) << (lr * LR);

        // warp 8: begins the copies of the next step; a walk of its own, ahead
        Walk<MT, BN> lead = walk;
        Unit lu{};
        int lt = 0, lnt = 0;                         // tile of the unit, its tiles
        int lpage = -1, loff = 0, npage = -1, noff = 0;     // this lane's rows of the tile and of the next one
        uint32_t lstep = 0;
        bool more = w < (E4 ? 1 : 2);
        const int blocks = !E4 && D > 64 ? 2 : 1, copies = BN / run_rows;      // 32 at most, a lane to each
        const int copy = lane / blocks, column = lane - copy * blocks;
        auto lead_page = [&](int t, int& off) {
            const int pos = (lu.t0 + t) * BN + copy * run_rows;
            if (copy >= copies || t >= lnt || pos >= lu.len) return -1;
            const int i = pos / a.c.P;
            off = lu.h * a.c.P + pos - i * a.c.P;
            return __ldg(a.table + static_cast<int64_t>(lu.b) * a.max_pages + i);
        };
        // step 2 T: the keys of tile T, 2 T + 1: its values; false: not yet
        auto begin = [&](bool block) {
            if (!more) return false;
            const bool isv = lstep & 1;
            const uint32_t T = lstep >> 1;
            // (values wait for free(T - 2); with it the keys of tile T + 1 may come)
            const bool mine = E4 || isv == (w == 1);
            if (isv && T >= 2) {
                const int bar = kFree + (T & 1);
                const uint32_t parity = (T - 2) >> 1 & 1;
                if (block) {
                    more = sync.wait(bar, parity);
                    more = __all_sync(0xffffffffu, more);
                } else if (!__all_sync(0xffffffffu, sync.test(bar, parity))) {
                    return false;
                }
                more = more && !__any_sync(0xffffffffu, sync.is_dead());
                if (!more) return false;
            }
            if (!isv && lt == lnt) {                 // the next unit with tiles
                do {
                    more = lead.next(a, part, mts, lu);
                    lnt = more && lu.len > 0 ? lu.t1 - lu.t0 : 0;
                } while (more && lnt == 0);
                if (!more) return false;
                lt = 0;
                npage = lead_page(0, noff);
            }
            if (!isv) {
                lpage = npage, loff = noff;
                npage = lead_page(lt + 1, noff);
            }
            const uint32_t slot = isv ? kKeySlots + (T & 1) : T % kKeySlots;
            const bool good = lpage >= 0 && lpage < a.c.pages;
            const uint32_t n = __popc(__ballot_sync(0xffffffffu, good));
            // (a test: the values of the second tile never come)
            const bool skip = (a.hooks & kHookAttnNoCopy) && blockIdx.x == 0 && lstep == 3;
            if (mine && !skip && elected()) mbar_arrive_expect_tx(bars + kLand + slot, n * run_rows * 128);
            __syncwarp();
            if (mine && good && !skip)                       // e4m3 lands in the slot's upper half
                tma_load(smem_u32(smem + slot * kTile + (E4 ? kBlock : column * kBlock) + copy * run_rows * 128), isv ? &map_v : &map_k,
                         bars + kLand + slot, column * 64, loff, lpage);
            __syncwarp();
            ++lstep;
            if (isv) ++lt;
            return true;
        };
        if (!E4 && w < kFirst)
            while (begin(true)) {}                   // nothing else to do

        Unit u;
        uint32_t tiles = 0, step = 0, nq[2] = {0, 0};
        while (w >= kFirst && walk.next(a, part, mts, u)) {
            const int nt = u.len > 0 ? u.t1 - u.t0 : 0;
            const int all_see = min(seen_by_all<MT>(a, u.cut, u.mt), held_of(a, u.cut));
            // e4m3: a thread looks after the exponents of rows p and p + 96 of a
            // tile; a row's page is read two tiles ahead, its exponents one
            const int32_t* table = a.table + static_cast<int64_t>(u.b) * a.max_pages;
            int page[2][2], ke[2] = {127, 127}, ve[2] = {127, 127};
            auto page_at = [&](int t, int i) {
                const int rr = p + i * kLoadThreads, pos = (u.t0 + t) * BN + rr;
                return rr < BN && t < nt && pos < u.len ? __ldg(table + pos / a.c.P) : -1;
            };
            auto exps_at = [&](int t, int i, int pg) {
                ke[i] = ve[i] = 127;
                if (pg >= 0 && pg < a.c.pages) {
                    const int64_t o = pg * a.c.exp_page_stride + static_cast<int64_t>(u.h) * a.c.P +
                                      ((u.t0 + t) * BN + p + i * kLoadThreads) % a.c.P;
                    ke[i] = a.c.ke[o];
                    ve[i] = a.c.ve[o];
                }
            };
            if constexpr (E4) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    page[0][i] = page_at(0, i);
                    page[1][i] = page_at(1, i);
                    exps_at(0, i, page[0][i]);
                }
            }
#pragma unroll 1
            for (int j = 0; j < 2 * nt; ++j, ++step) {
                const bool isv = j & 1;
                const int t = j >> 1;
                const uint32_t tile = tiles + t, slot = isv ? kKeySlots + (tile & 1) : tile % kKeySlots;
                if constexpr (E4) {                  // copies as far ahead as there is room
                    if (w == 0) {
                        while (begin(false)) {}
                        while (lstep <= step && begin(true)) {}
                    }
                }
                const int from = min(max(all_see - (u.t0 + t) * BN, 0), BN);    // first row that some do not see
                if (E4 && !isv) {                    // the exponents of tile t
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int rr = p + i * kLoadThreads;
                        if (rr < BN) {
                            smem[M::exps + tile % 3 * 2 * BN + rr] = static_cast<unsigned char>(ke[i]);
                            smem[M::exps + tile % 3 * 2 * BN + BN + rr] = static_cast<unsigned char>(ve[i]);
                        }
                        page[0][i] = page[1][i];
                        page[1][i] = page_at(t + 2, i);
                        exps_at(t + 1, i, page[0][i]);
                    }
                    bar_sync(1, kLoadThreads);
                }
                sync.wait(kLand + slot, (isv ? tile >> 1 : tile / kKeySlots) & 1);
                __syncwarp();
                unsigned char* base = smem + slot * kTile;
                const bool check = isv && from < BN;
                if (isv) {                           // (read for other tiles too, where a page is bad)
                    if (lane < 4) s_flag[(tile & 3) * (kLoadWarps * 4) + w * 4 + lane] = 0;
                    __syncwarp();
                }
                if (E4 || (check && odd_values<F16>(base, from, D > 64 ? 2 : 1, lane))) {
                    uint32_t* flags = s_flag + (tile & 3) * (kLoadWarps * 4) + w * 4;
                    const unsigned char* ex = smem + M::exps + (tile % 3 * 2 + isv) * BN;
                    // several of its rows read before the first is written: a read
                    // waits hundreds of clocks behind the products' operands
                    for (int q0 = w - kFirst; q0 < BN / RP; q0 += kBatch * kSettle) {
                        uint4 in[kBatch];
                        int e[kBatch];
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) {
                            const int q = q0 + i * kSettle, r = q * RP + lr;
                            in[i] = make_uint4(0, 0, 0, 0), e[i] = 127;
                            if (q < BN / RP && lc < CH) {
                                in[i] = *reinterpret_cast<const uint4*>(base + (E4 ? kBlock + r * 128 + lc * 16 : chunk_at(r, lc)));
                                e[i] = E4 ? ex[r] : 127;
                            }
                        }
                        __syncwarp();                // a row's lanes have read it before it is written over
                        if constexpr (E4) {
                            // (the usual powers make no infinity)
                            bool usual = true;
#pragma unroll
                            for (int i = 0; i < kBatch; ++i) usual = usual && usual_power<F16>(e[i]);
                            if (check)
#pragma unroll
                                for (int i = 0; i < kBatch; ++i) usual = usual && !has_nan(in[i]);
                            if (__all_sync(0xffffffffu, usual)) {
                                // (no branch between the rows: their steps overlap)
#pragma unroll
                                for (int i = 0; i < kBatch; ++i) {
                                    const int q = q0 + i * kSettle, r = q * RP + lr;
                                    uint32_t o[8];
                                    widen16_usual<F16>(in[i], e[i], o);
                                    if (q < BN / RP && lc < CH) {
                                        *reinterpret_cast<uint4*>(base + chunk_at(r, 2 * lc)) = make_uint4(o[0], o[1], o[2], o[3]);
                                        *reinterpret_cast<uint4*>(base + chunk_at(r, 2 * lc + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                                    }
                                }
                                continue;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) {
                            const int q = q0 + i * kSettle, r = q * RP + lr;
                            if (q >= BN / RP) break;
                            uint32_t o[8];
                            if constexpr (E4) {
                                bool beyond = false;
                                widen16<F16>(in[i], e[i], o, beyond);
                                if (F16 && beyond) s_tmem[2] = 1;
                            } else {
                                o[0] = in[i].x, o[1] = in[i].y, o[2] = in[i].z, o[3] = in[i].w;
                            }
                            bool row_bad = false;
                            if (check) {
                                constexpr uint32_t top = F16 ? 0x7c00u : 0x7f80u;
                                bool bad = false;
                                if (lc < CH && r >= from)
#pragma unroll
                                    for (int y = 0; y < (E4 ? 8 : 4); ++y)
                                        bad |= (o[y] & top) == top || (o[y] >> 16 & top) == top;
                                row_bad = (__ballot_sync(0xffffffffu, bad) & group) != 0;
                                if (row_bad && lc == 0) atomicOr(flags + (r >> 5), 1u << (r & 31));
                            }
                            if (lc < CH && (E4 || row_bad)) {
#pragma unroll
                                for (int y = 0; y < (E4 ? 8 : 4); y += 4)
                                    *reinterpret_cast<uint4*>(base + chunk_at(r, E4 ? 2 * lc + y / 4 : lc)) =
                                        row_bad ? make_uint4(0, 0, 0, 0) : make_uint4(o[y], o[y + 1], o[y + 2], o[y + 3]);
                            }
                        }
                    }
                }
                fence_async();
                __syncwarp();
                if (!isv && lane == 0) sync.arrive(kFull + (tile & 1));
                if (BOXES && j == 0 && w == kFirst) {
                    // the queries, once the scores of the unit before are done with theirs
                    const int streams = nt == 0 ? 0 : (u.mt * MT + kRows) / a.g < u.cut.cnt ? 2 : 1;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (s >= streams) break;
                        sync.wait(kQEmpty + s, (nq[s] & 1) ^ 1);
                        __syncwarp();
                        if (__any_sync(0xffffffffu, sync.is_dead())) break;
                        ++nq[s];
                        // the 128 rows are the group's heads of whole nodes
                        unsigned char* qs = smem + M::q + s * kTile;
                        const int q_blocks = D > 64 ? 2 : 1;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(bars + kQFull + s, q_blocks * kBlock);
                            for (int i = 0; i < q_blocks; ++i)
                                tma_load_q(smem_u32(qs + i * kBlock), &map_q, bars + kQFull + s, i * 64, u.h * a.g, (u.mt * MT + s * kRows) / a.g, u.b);
                        }
                    }
                }
            }
            tiles += nt;
        }
        if (w >= kFirst && lane == 0) sync.arrive(kFull + (tiles & 1));       // the last values
        if (BOXES && w == kFirst)                  // a dead CTA too waits for the copies it has begun
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (nq[s] > 0) sync.landed(kQFull + s, (nq[s] - 1) & 1);
        if (w == 0 || (!E4 && w == 1))
            // (two tiles' values and the keys of three at most; those before have been used)
            for (uint32_t i = lstep > 5 ? lstep - 4 - (lstep & 1) : 0; i < lstep; ++i) {
                const uint32_t T = i >> 1;
                const int bar = kLand + (i & 1 ? kKeySlots + (T & 1) : T % kKeySlots);
                sync.landed(bar, (i & 1 ? T >> 1 : T / kKeySlots) & 1);
            }
    } else {
        // ---------------- products ----------------
        // The whole warp walks and waits, so that the operands stay uniform; one
        // elected thread issues.
        constexpr uint32_t type = F16 ? 0u : 1u;
        const uint32_t common = (1u << 4) | (type << 7) | (type << 10) | (8u << 24);    // fp32 += 16 bits, 128 rows
        const uint32_t idesc_s = common | (static_cast<uint32_t>(BN / 8) << 17);
        const uint32_t idesc_o = common | (1u << 16) | (static_cast<uint32_t>(D / 8) << 17);    // V is MN-major
        const uint32_t ring_k = operand_lo(smem_u32(smem), 16), ring_v = operand_lo(smem_u32(smem), kBlock);
        const uint32_t q0 = operand_lo(smem_u32(smem + M::q), 16);
        const int nks = D / 16;
        Unit u;
        uint32_t n[2] = {0, 0}, q[2] = {0, 0}, T = 0;           // tiles and queries of each stream, tiles of the CTA
        bool ok = true;                              // while no wait has given up
        const uint32_t tm = uniform(tmem);
        auto scores = [&](int s, uint32_t key_slot, bool last) {
            if (elected()) {
                if (ok) {
                    const uint32_t x = q0 + s * (kTile >> 4), y = ring_k + key_slot * (kTile >> 4), d = tm + s * 128;
                    if (nks == 8) {
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            const uint32_t off = ((ks >> 2) * kBlock + (ks & 3) * 32) >> 4;
                            mma_ss(d, x + off, y + off, idesc_s, ks > 0);
                        }
                    } else {
                        for (int ks = 0; ks < nks; ++ks) {
                            const uint32_t off = ((ks >> 2) * kBlock + (ks & 3) * 32) >> 4;
                            mma_ss(d, x + off, y + off, idesc_s, ks > 0);
                        }
                    }
                }
                sync.commit(kSFull + s);
                if (last) sync.commit(kQEmpty + s);
            }
        };
        while (walk.next(a, part, mts, u)) {
            const int nt = u.len > 0 ? u.t1 - u.t0 : 0;
            if (nt == 0) continue;
            // stream s has a live row (stream 0 has one in every unit with tiles)
            const int streams = (u.mt * MT + kRows) / a.g < u.cut.cnt ? 2 : 1;
            const bool begun = PARTS && a.far != nullptr && u.t0 == 0;    // the softmax warps have set the outputs
            // (the unit before has waited for these keys with its last values)
            if (T == 0) ok = sync.wait(kFull, 0) && ok;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (s >= streams) break;
                ok = sync.wait(kQFull + s, q[s]++ & 1) && ok;
                __syncwarp();
                fence_after();
                scores(s, T % kKeySlots, nt == 1);
            }
            if (T > 0 && elected()) sync.commit(kFree + ((T - 1) & 1));
            uint32_t key_slot = T % kKeySlots;
            for (int t = 0; t < nt; ++t, ++T) {
                const bool more = t + 1 < nt;
                key_slot = key_slot + 1 == kKeySlots ? 0 : key_slot + 1;
                ok = sync.wait(kFull + ((T + 1) & 1), (T + 1) >> 1 & 1) && ok;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (s >= streams) break;
                    ok = sync.wait(kPFull + s, n[s]++ & 1) && ok;
                    __syncwarp();
                    fence_after();
                    if (elected()) {
                        if (ok) {
                            const uint32_t x = tm + s * 128, y = ring_v + (kKeySlots + (T & 1)) * (kTile >> 4), d = tm + 256 + s * 128;
#pragma unroll
                            for (int ks = 0; ks < BN / 16; ++ks) mma_ts(d, x + ks * 8, y + ks * (2048 >> 4), idesc_o, t > 0 || ks > 0 || begun);
                        }
                        if (!more) sync.commit(kOFull + s);
                    }
                    if (more) scores(s, key_slot, t + 2 == nt);
                }
                if (more && elected()) sync.commit(kFree + (T & 1));
                __syncwarp();
            }
        }
        if (elected()) sync.commit(kEnd);            // nothing is under way any more
        __syncwarp();
        sync.landed(kEnd, 0);                        // (in a dead CTA too: TMEM is given back next)
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if constexpr (E4 && F16)
        if (tid == 0) a.beyond[blockIdx.x] = s_tmem[2];
    if (warp == 11) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// Queries as [B][N][Hq][D]: a box is the group's heads of 128 / g nodes.  Not
// for every group and stride: the kernel then copies the rows itself.
bool encode_q(CUtensorMap* map, const AttnArgs& a) {
    const EncodeTiled f = encode_tiled();
    const int64_t strides_in[3] = {a.q_sh, a.q_sn, a.q_sb};
    if (!f || kRows % a.g || a.q_n > 0 || (reinterpret_cast<uintptr_t>(a.q) & 15)) return false;
    for (int i = 0; i < 3; ++i)
        if (strides_in[i] <= 0 || strides_in[i] % 16 || strides_in[i] >= (int64_t(1) << 40)) return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.c.D), static_cast<cuuint64_t>(a.Hq), static_cast<cuuint64_t>(a.N),
                                static_cast<cuuint64_t>(a.B)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(a.q_sh), static_cast<cuuint64_t>(a.q_sn), static_cast<cuuint64_t>(a.q_sb)};
    const cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(a.g), static_cast<cuuint32_t>(kRows / a.g), 1u}, one[4] = {1u, 1u, 1u, 1u};
    return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<unsigned char*>(a.q), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool E4, bool F16, bool BOXES, bool PARTS>
cudaError_t launch_one(AttnArgs a, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& q, int rows, int nsm, cudaStream_t s) {
    constexpr int bytes = Smem::bytes;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(attn_tc_kernel<E4, F16, BOXES, PARTS>), bytes);
    if (e != cudaSuccess) return e;
    // the exchange of registers needs a launch that has them
    static const int regs = [] {
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, reinterpret_cast<const void*>(attn_tc_kernel<E4, F16, BOXES, PARTS>)) == cudaSuccess ? at.numRegs : 0;
    }();
    if (regs != kRegs) return cudaErrorInvalidKernelImage;
    a.ctas = nsm;
    const int mts = (a.N * a.g + MT - 1) / MT;
    const int64_t units = static_cast<int64_t>(a.B) * a.c.H * mts;
    a.rounds = mts > 1 && units >= 2 * nsm ? static_cast<int>(units / nsm - 1) : 0;
    attn_tc_kernel<E4, F16, BOXES, PARTS><<<static_cast<unsigned>(nsm), kThreads, bytes, s>>>(a, k, v, q, rows);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_attn_combine(a, F16, MT, s);
}

template <bool E4, bool F16>
cudaError_t launch(const AttnArgs& a, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& q, bool boxes, int rows, int nsm,
                   cudaStream_t s) {
    if (a.raw || a.far)
        return boxes ? launch_one<E4, F16, true, true>(a, k, v, q, rows, nsm, s) : launch_one<E4, F16, false, true>(a, k, v, q, rows, nsm, s);
    return boxes ? launch_one<E4, F16, true, false>(a, k, v, q, rows, nsm, s) : launch_one<E4, F16, false, false>(a, k, v, q, rows, nsm, s);
}

}  // namespace

bool attn_tma_takes(const AttnArgs& a) { return a.c.D <= 128 && a.c.P % 8 == 0 && encode_tiled() != nullptr; }

cudaError_t launch_attn_tc(const AttnArgs& a, bool f16, bool e4m3, int nsm, cudaStream_t s) {
    // rows of one copy: those of a tile that are sure to lie in one page
    const int rows = min(a.c.P & -a.c.P, BN);
    CUtensorMap k, v, q = {};
    if (!encode_cells(&k, a, a.c.k, e4m3, rows, !e4m3) || !encode_cells(&v, a, a.c.v, e4m3, rows, !e4m3)) return cudaErrorInvalidValue;
    // (a negative scale is the queries' sign, which a copy by boxes leaves alone)
    const bool boxes = a.scale_log2 >= 0.0f && encode_q(&q, a);
    if (e4m3) return f16 ? launch<true, true>(a, k, v, q, boxes, rows, nsm, s) : launch<true, false>(a, k, v, q, boxes, rows, nsm, s);
    return f16 ? launch<false, true>(a, k, v, q, boxes, rows, nsm, s) : launch<false, false>(a, k, v, q, boxes, rows, nsm, s);
}

}  // namespace sdv
