// k8_attn_prefix.cu -- attention of sequences that share prefixes
// (sdv_prefix_attn).
//
// The nodes of a group's sequences are to its prefix what the nodes of one
// sequence are to theirs: one batch of S * N nodes that all see the prefix and
// nothing of one another.  So the attention kernels run twice, over the prefixes
// with a group for a sequence, which reads a prefix once for all its sequences,
// and over the sequences' own pages; each time they leave normalised fp32 rows
// and the base-2 logs L of their sums.  A row's two results join as
//   out = (2^(L1 - L) o1 + 2^(L2 - L) o2),   L = log2(2^L1 + 2^L2).
#include "k8_attn.cuh"

namespace sdv {
namespace {

constexpr int kThreads = 256;

// Four elements of a row to a thread.
template <bool F16>
__global__ void __launch_bounds__(kThreads) join_kernel(const AttnArgs a, const float* far, const float* far_log, const float* near,
                                                        const float* near_log, int64_t rows) {
    const int vec = a.c.D / 4;
    const int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    const int64_t row = i / vec;
    if (row >= rows) return;
    const int d = static_cast<int>(i - row * vec) * 4;
    const float nan = __int_as_float(0x7fc00000);
    const float L1 = far_log[row], L2 = near_log[row];
    const float4 x = *reinterpret_cast<const float4*>(far + row * a.c.D + d);
    const float4 y = *reinterpret_cast<const float4*>(near + row * a.c.D + d);
    const int64_t node = row / a.Hq;
    const int b = static_cast<int>(node / a.N);
    // (a bad sequence's second result is not a number; nodes that are not there see nothing)
    const bool there = !a.count || node - static_cast<int64_t>(b) * a.N < a.count[b] || L2 != L2;
    const float top = fmaxf(L1, L2), base = top == -INFINITY ? 0.0f : top;
    const float f1 = ex2(L1 - base), f2 = ex2(L2 - base), sum = f1 + f2;
    const bool bad = L1 != L1 || L2 != L2, empty = !there || (!bad && top == -INFINITY);
    const float g1 = empty ? 0.0f : bad ? nan : f1 / sum, g2 = empty ? 0.0f : bad ? nan : f2 / sum;
    float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (!empty) {
        // (an empty side's row is 0, and its factor too)
        o[0] = x.x * g1 + y.x * g2, o[1] = x.y * g1 + y.y * g2;
        o[2] = x.z * g1 + y.z * g2, o[3] = x.w * g1 + y.w * g2;
    }
    attn::store_row4<F16>(a, row, d, o, empty ? -INFINITY : bad ? nan : base + log2f(sum));
}

}  // namespace

size_t prefix_workspace_bytes(int64_t rows, int D, int nsm) {
    const size_t one = static_cast<size_t>(rows) * (D + 1) * sizeof(float);
    return (attn_workspace_bytes(nsm) + 31) / 32 * 32 + 2 * ((one + 31) / 32 * 32);
}

cudaError_t launch_prefix_attn(const AttnArgs& a, const PrefixArgs& p, int type, bool e4m3, void* workspace, int nsm, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(a.B) * a.N * a.Hq;
    unsigned char* at = static_cast<unsigned char*>(workspace) + (attn_workspace_bytes(nsm) + 31) / 32 * 32;
    const size_t one = (static_cast<size_t>(rows) * (a.c.D + 1) * sizeof(float) + 31) / 32 * 32;
    float* raw[2] = {reinterpret_cast<float*>(at), reinterpret_cast<float*>(at + one)};

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
    far.mask = p.table, far.mask_sb = 0, far.W = 0;  // (a mask without words: no node sees another)
    far.raw = raw[0], far.raw_log = raw[0] + rows * a.c.D;
    near.raw = raw[1], near.raw_log = raw[1] + rows * a.c.D;
    cudaError_t e = launch_tree_attn(far, type, e4m3, workspace, nsm, s);
    if (e == cudaSuccess) e = launch_tree_attn(near, type, e4m3, workspace, nsm, s);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (rows * (a.c.D / 4) + kThreads - 1) / kThreads;
    if (type == kTypeF16)
        join_kernel<true><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a, far.raw, far.raw_log, near.raw, near.raw_log, rows);
    else
        join_kernel<false><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a, far.raw, far.raw_log, near.raw, near.raw_log, rows);
    return cudaGetLastError();
}

}  // namespace sdv
