// sdv_layer.h -- arguments and launchers of the verifier's-layer operators:
// draft tree, rotary positions, paged cache, tree attention, sampling
// parameters (the entry points of include/sdv.h that take no context).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace sdv {

constexpr int kTypeBf16 = 0, kTypeF32 = 1, kTypeF16 = 2, kTypeE4m3 = 3;
constexpr unsigned kStatusBadPage = 64u;     // a page id outside the cache
constexpr unsigned kStatusNoPages = 128u;    // the free pages ran out

constexpr int kTreeMaxDrafts = 64;
constexpr int kTreeMaxGamma = 128;
constexpr int kRopeMaxDim = 512;
constexpr int kCacheMaxDim = 256;

struct TreeArgs {
    const int32_t *root, *drafts, *draft_len;
    int32_t *tokens, *depth, *mask, *nodes, *rows, *count;
    unsigned* status;
    int B, K, G, N, W;
};
cudaError_t launch_tree_build(const TreeArgs& a, cudaStream_t s);

struct RopeArgs {
    const void *q, *k;
    void *oq, *ok;
    int64_t q_st, q_sh, k_st, k_sh, oq_st, oq_sh, ok_st, ok_sh;   // bytes
    const int32_t* pos;
    const float* freq;
    float factor;
    int64_t T;
    int Hq, Hk, D, R, interleaved;
};
// `vec`: rows are made of whole, aligned 16-byte vectors, two to a work item
cudaError_t launch_rope(const RopeArgs& a, int type, bool vec, int nsm, cudaStream_t s);

// A paged cache, strides in bytes.
struct CacheView {
    unsigned char *k, *v;
    unsigned char *ke, *ve;
    int64_t page_stride, exp_page_stride;
    int pages, P, H, D;
};

struct CellsArgs {
    CacheView c;
    const unsigned char *k, *v;       // kv_write: sources
    int64_t k_sb, k_sn, k_sh, v_sb, v_sn, v_sh;   // bytes
    void *ok, *ov;                    // kv_read: outputs
    const int32_t *table, *start, *count;
    unsigned* status;
    int B, N, max_pages;
};
cudaError_t launch_kv_write(const CellsArgs& a, int type, bool e4m3, bool vec, cudaStream_t s);
cudaError_t launch_kv_read(const CellsArgs& a, int type, bool e4m3, cudaStream_t s);

struct CommitArgs {
    CacheView c;
    int cell;                         // bytes of a cell
    const int32_t *table, *start, *nodes, *sel, *acc;
    int32_t* out_len;
    unsigned* status;
    int B, K, G, max_pages;
};
cudaError_t launch_kv_commit(const CommitArgs& a, cudaStream_t s);

struct AttnArgs {
    CacheView c;
    const unsigned char* q;
    int64_t q_sb, q_sn, q_sh;         // bytes
    int q_n;                          // > 0: nodes q_n apart are q_s2 bytes apart, those between q_sn
    int64_t q_s2;
    const int32_t *table, *ctx, *count, *mask;
    int64_t mask_sb;                  // words
    void* out;
    float* lse;
    float *raw, *raw_log;             // not NULL: rows go here as fp32, with the base-2 logs of their sums
    const float *far, *far_log;       // not NULL: rows to go on from (launch_attn_tc alone, without a raw)
    unsigned* status;
    float* part;                      // partial outputs (see part_rows)
    int4* desc;                       // two per CTA: the unit that its start splits
    unsigned* beyond;                 // one per SM: see launch_attn_redo
    int B, N, Hq, g, max_pages;
    int W;                            // words of a mask row
    int own;                          // -1; 0 (with W = 0, and a mask that is not read): no node's keys are in the cache
    float scale_log2;                 // scale * log2(e)
    int ctas, rounds;                 // see k8_attn.cuh
    unsigned hooks;                   // kHook* bits (tests of the waits)
};
// The first CTA's second tile (its values) never comes, and waits give up soon:
// nothing is in flight for the wait that runs out (the public SDV_HOOK_ATTN_NO_COPY).
constexpr unsigned kHookAttnNoCopy = 2u;
size_t attn_workspace_bytes(int nsm);
cudaError_t launch_tree_attn(AttnArgs a, int type, bool e4m3, void* workspace, int nsm,
                             cudaStream_t s);

// The prefixes of `groups` groups of sequences (the groups' sequences are a.B / groups).
struct PrefixArgs {
    const int32_t *table, *len;
    int max_pages, groups;
};
size_t prefix_workspace_bytes(int B, int N, int Hq, int D, int nsm);
cudaError_t launch_prefix_attn(const AttnArgs& a, const PrefixArgs& p, int type, bool e4m3, void* workspace, int nsm,
                               cudaStream_t s);

struct LogitsArgs {
    const void* logits;
    void* out;
    const int32_t *rows, *drafts, *counts, *prompt, *bias_ids, *allow;
    const float *rep, *freq, *pres, *bias;
    unsigned* status;
    int B, K, G, V, nsrc, M, W;
    int row_splits;                   // CTAs that share the rows of one draft
};
cudaError_t launch_logits(const LogitsArgs& a, bool bf16, int nsm, cudaStream_t s);

struct CountsArgs {
    const int32_t *drafts, *sel, *acc, *next;
    int32_t* counts;
    unsigned* status;
    int B, K, G, V;
};
cudaError_t launch_counts_commit(const CountsArgs& a, cudaStream_t s);

struct PagesArgs {
    int32_t *list, *free_count, *table, *held;
    const int32_t *start, *count, *depth, *base;      // (release: start is what is kept)
    int32_t* positions;
    int64_t* slots;
    unsigned* status;
    int B, N, pages, P, max_pages;
};
cudaError_t launch_pages_extend(const PagesArgs& a, int nsm, cudaStream_t s);
cudaError_t launch_pages_release(const PagesArgs& a, int nsm, cudaStream_t s);

constexpr int kRowsMaxVocab = 1 << 19;       // sums of that many weights fit 64 bits
struct RowsArgs {
    const void* logits;
    int64_t in_stride, out_stride;            // bytes
    const float *temperature, *top_p, *min_p, *uniform;
    const int32_t* top_k;
    void* out;
    int32_t *tokens, *kept;
    float* logprob;
    unsigned* status;
    int64_t rows;
    int per, V;
};
cudaError_t launch_rows(const RowsArgs& a, bool bf16, bool draw, int nsm, cudaStream_t s);

}  // namespace sdv
