// k8_attn_prefix.cu -- attention of sequences that share prefixes
// (sdv_prefix_attn).
//
// The nodes of a group's sequences are to its prefix what the nodes of one
// sequence are to theirs: one batch of S * N nodes that all see the prefix and
// nothing of one another.  So the attention kernels run over the prefixes with a
// group for a sequence, which reads a prefix once for all its sequences, and leave
// normalised fp32 rows and the base-2 logs L of their sums.  What the sequences have
// added comes from the same kernels, or for single tokens from k8_attn_one.cu.  A
// row's results join as
//   out = sum_i 2^(L_i - L) o_i,   L = log2 sum_i 2^(L_i),
// in the kernel of single tokens; in the kernel of many rows, which goes on from the
// prefix's; or in one of its own.
//
// 128 tokens behind 8191 shared positions, 8 x 8 heads of 128: 119 us (prefix 51, joins
// of its parts 10, own positions 56) where attention of each sequence over all of it
// reads 4.3 GB; 16 trees of 257 nodes behind 6001: 900 us, 0.94 PFLOP/s, of which the
// prefix's kernel takes three quarters.
#include "k8_attn.cuh"

namespace sdv {
namespace {

constexpr int kThreads = 256;

// Parts of single tokens' own positions, where there are few heads to share out.  With 64
// heads: 4 sequences of 4000 positions 52 us in 8 parts and 142 in one, 16 of them 99 and
// 152; 48 sequences of 600 positions 70 us in two parts and 62 in one, of 4000 189 and 181.
// (Each sequence's held positions are cut, however wide the table.)
constexpr int kMaxSplits = 8;
int splits_of(int64_t rows, int N) {
    const int64_t n = N > 1 ? 1 : 6000 / rows;
    return static_cast<int>(n < 1 ? 1 : n > kMaxSplits ? kMaxSplits : n);
}

// Four elements of a row to a thread; near: `parts` of [rows][D], whose rows are only
// there where their log is not -infinity.
template <bool F16, int MOST>
__global__ void __launch_bounds__(kThreads) join_kernel(const AttnArgs a, const float* far, const float* far_log, const float* near,
                                                        const float* near_log, int parts, int64_t rows) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int vec = a.c.D / 4;
    const int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    const int64_t row = i / vec;
    if (row >= rows) return;
    const int d = static_cast<int>(i - row * vec) * 4;
    const float nan = __int_as_float(0x7fc00000);
    float L[MOST + 1];
    L[0] = far_log[row];
#pragma unroll
    for (int p = 0; p < MOST; ++p) L[p + 1] = p < parts ? near_log[p * rows + row] : -INFINITY;
    const int64_t node = row / a.Hq;
    const int b = static_cast<int>(node / a.N);
    float top = -INFINITY;
    bool bad = false, bad_near = false;
#pragma unroll
    for (int p = 0; p <= MOST; ++p) {
        top = fmaxf(top, L[p]);
        bad |= L[p] != L[p];
        bad_near |= p > 0 && L[p] != L[p];
    }
    // (a bad sequence's own result is not a number; nodes that are not there see nothing)
    const bool there = !a.count || node - static_cast<int64_t>(b) * a.N < a.count[b] || bad_near;
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p <= MOST; ++p) {
        if (L[p] == -INFINITY) continue;
        const float4 x = *reinterpret_cast<const float4*>((p == 0 ? far : near + (p - 1) * rows * a.c.D) + row * a.c.D + d);
        const float f = ex2(L[p] - base);
        sum += f;
        o[0] += x.x * f, o[1] += x.y * f, o[2] += x.z * f, o[3] += x.w * f;
    }
    const bool empty = !there || (!bad && sum == 0.0f);
    const float inv = empty ? 0.0f : bad ? nan : 1.0f / sum;
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] = empty ? 0.0f : o[x] * inv;
    attn::store_row4<F16, false>(a, row, d, o, empty ? -INFINITY : bad ? nan : base + log2f(sum));
}

// from: rows and logs of the prefix, rows and logs of the parts.
template <bool F16, int MOST>
cudaError_t launch_join(const AttnArgs& a, const float* const (&from)[4], int64_t rows, cudaStream_t s, int parts = 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((rows * (a.c.D / 4) + kThreads - 1) / kThreads));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<F16, MOST>, a, from[0], from[1], from[2], from[3], parts, rows);
}

}  // namespace

// (The second set of rows is not used by calls that go on from the prefix's: which do depends on the
// cache's type and pages, which the size is asked for without.)
size_t prefix_workspace_bytes(int B, int N, int Hq, int D, int nsm) {
    const int64_t rows = static_cast<int64_t>(B) * N * Hq;
    const size_t one = static_cast<size_t>(rows) * (D + 1) * sizeof(float);
    return (attn_workspace_bytes(nsm) + 31) / 32 * 32 + (1 + splits_of(rows, N)) * ((one + 31) / 32 * 32);
}

cudaError_t launch_prefix_attn(const AttnArgs& a, const PrefixArgs& p, int type, bool e4m3, void* workspace, int nsm, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(a.B) * a.N * a.Hq, cells = rows * a.c.D;
    const bool f16 = type == kTypeF16;
    float* far_rows = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + (attn_workspace_bytes(nsm) + 31) / 32 * 32);
    float* near_rows = far_rows + (cells + rows + 7) / 8 * 8;
    const bool single = attn_one_takes(a);
    const int parts = single ? splits_of(rows, a.N) : 1;

    AttnArgs far = a, near = a;
    const int each = a.B / p.groups;
    far.B = p.groups;
    far.N = each * a.N;
    far.q_sb = each * a.q_sb;
    if (a.N == 1) {
        far.q_sn = a.q_sb;
    } else if (each > 1 && a.q_sb != a.N * a.q_sn) {
        far.q_n = a.N;
        far.q_s2 = a.q_sb;
    }
    far.table = p.table, far.max_pages = p.max_pages, far.ctx = p.len;
    far.count = nullptr;
    far.mask = p.table, far.mask_sb = 0, far.W = far.own = 0;     // (a mask without words: no node sees another)
    far.raw = far_rows, far.raw_log = far_rows + cells;
    cudaError_t e = launch_tree_attn(far, type, e4m3, workspace, nsm, s);
    if (e != cudaSuccess) return e;
    // many rows go on from the prefix's outputs themselves (16 trees of 257 nodes: 907 us, and
    // 930 with a join of 270 MB; not where fp16 queries may make them be done again)
    if (attn_goes_on(near, f16, e4m3)) {
        near.far = far.raw, near.far_log = far.raw_log;
        return launch_tree_attn(near, type, e4m3, workspace, nsm, s);
    }
    near.raw = near_rows, near.raw_log = near_rows + parts * cells;
    e = single ? launch_attn_one(near, f16, e4m3, far.raw, far.raw_log, parts, s) : launch_tree_attn(near, type, e4m3, workspace, nsm, s);
    if (e != cudaSuccess || (single && parts == 1)) return e;
    const float* rows_of[4] = {far.raw, far.raw_log, near.raw, near.raw_log};
    if (parts == 1) return f16 ? launch_join<true, 1>(a, rows_of, rows, s) : launch_join<false, 1>(a, rows_of, rows, s);
    return f16 ? launch_join<true, kMaxSplits>(a, rows_of, rows, s, parts) : launch_join<false, kMaxSplits>(a, rows_of, rows, s, parts);
}

}  // namespace sdv
