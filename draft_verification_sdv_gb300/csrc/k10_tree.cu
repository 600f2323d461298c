// k10_tree.cu -- the tree of K drafts (sdv_tree_build): whole numbers only, one
// CTA per sequence.
//
// Draft k's token j shares the node of the first draft whose tokens 0..j are
// the same.  Nodes are numbered draft by draft: draft k adds the nodes past the
// longest beginning that it shares with an earlier draft, and its other nodes
// are that draft's.
#include "sdv_layer.h"
#include "sdv_plan.h"

namespace sdv {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) tree_kernel(const TreeArgs a) {
    extern __shared__ int32_t sm[];
    int32_t* tok = sm;                       // [K][G] tokens
    int32_t* node = tok + a.K * a.G;         // [K][G] nodes
    __shared__ int share[kTreeMaxDrafts];    // tokens shared with an earlier draft
    __shared__ int from[kTreeMaxDrafts];     // ... the first one that shares as many
    __shared__ int base[kTreeMaxDrafts];     // node of the draft's first own token
    const int b = blockIdx.x, KG = a.K * a.G;
    const int64_t b64 = b;
    int len = a.draft_len ? a.draft_len[b] : a.G;
    if (len < 0 || len > a.G) {
        if (threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadLength);
        len = 0;
    }
    for (int i = threadIdx.x; i < KG; i += kThreads) tok[i] = a.drafts[b64 * KG + i];
    __syncthreads();
    for (int k = threadIdx.x; k < a.K; k += kThreads) {
        int best = 0, who = 0;
        for (int o = 0; o < k; ++o) {
            int n = 0;
            while (n < len && tok[k * a.G + n] == tok[o * a.G + n]) ++n;
            if (n > best) best = n, who = o;
        }
        share[k] = best;
        from[k] = who;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int next = 1;
        for (int k = 0; k < a.K; ++k) base[k] = next, next += len - share[k];
        a.count[b] = next;
    }
    __syncthreads();
    const int count = base[a.K - 1] + len - share[a.K - 1];
    for (int i = threadIdx.x; i < KG; i += kThreads) {
        const int j = i % a.G;
        int k = i / a.G;
        while (j < share[k]) k = from[k];    // the draft that owns the node: always an earlier one
        node[i] = j < len ? base[k] + j - share[k] : -1;
        a.nodes[b64 * KG + i] = node[i];
    }
    for (int n = threadIdx.x; n < a.N; n += kThreads)
        if (n == 0 || n >= count) {
            a.tokens[b64 * a.N + n] = n == 0 ? a.root[b] : -1;
            a.depth[b64 * a.N + n] = 0;
        }
    int32_t* mask = a.mask + b64 * a.N * a.W;
    for (int64_t w = threadIdx.x; w < static_cast<int64_t>(a.N) * a.W; w += kThreads) {
        const int n = static_cast<int>(w / a.W);
        if (n == 0 || n >= count) mask[w] = w == 0 ? 1 : 0;     // the others are written below
    }
    __syncthreads();
    int32_t* rows = a.rows + b64 * a.K * (a.G + 1);
    for (int i = threadIdx.x; i < KG; i += kThreads) {
        const int k = i / a.G, j = i % a.G;
        rows[k * (a.G + 1) + j + 1] = j < len ? node[i] : 0;
        if (j == 0) rows[k * (a.G + 1)] = 0;
        if (j >= len || j < share[k]) continue;
        const int n = node[i];
        a.tokens[b64 * a.N + n] = tok[i];
        a.depth[b64 * a.N + n] = j + 1;
        // the path's nodes grow with j, so the words come in order
        int32_t* row = mask + static_cast<int64_t>(n) * a.W;
        uint32_t bits = 1u;                  // the root
        int word = 0;
        for (int at = 0; at <= j; ++at) {
            const int m = node[k * a.G + at];
            while (m / 32 > word) row[word++] = static_cast<int32_t>(bits), bits = 0;
            bits |= 1u << (m & 31);
        }
        while (word < a.W) row[word++] = static_cast<int32_t>(bits), bits = 0;
    }
}

}  // namespace

cudaError_t launch_tree_build(const TreeArgs& a, cudaStream_t s) {
    const size_t smem = static_cast<size_t>(2) * a.K * a.G * sizeof(int32_t);    // 64 KB at most
    if (smem > 40 * 1024) {
        const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(tree_kernel), smem);
        if (e != cudaSuccess) return e;
    }
    tree_kernel<<<static_cast<unsigned>(a.B), kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace sdv
