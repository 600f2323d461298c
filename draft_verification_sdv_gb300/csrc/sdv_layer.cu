// sdv_layer.cu -- the C ABI of the verifier's-layer operators (declared in
// include/sdv.h): argument checks, strides to bytes, which variant runs.
#include <cmath>

#include "../../include/sdv.h"
#include "sdv_layer.h"
#include "sdv_plan.h"

using namespace sdv;

static_assert(SDV_BF16 == kTypeBf16 && SDV_F32 == kTypeF32 && SDV_F16 == kTypeF16 && SDV_E4M3 == kTypeE4m3,
              "public and kernel types must agree");
static_assert(SDV_STATUS_BAD_TOKEN == kStatusBadDraft && SDV_STATUS_TIMEOUT == kStatusTimeout &&
                  SDV_STATUS_BAD_PAGE == kStatusBadPage && SDV_STATUS_BAD_LENGTH == kStatusBadLength,
              "public and kernel status bits must agree");
static_assert(SDV_HOOK_ATTN_NO_COPY == kHookAttnNoCopy, "public test hooks and kernel hooks must agree");

namespace {

// Whether each is NULL or memory of the current device, which the call runs on.
template <int N> bool all_device(const void* const (&p)[N]) {
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    for (const void* x : p) {
        cudaPointerAttributes at;
        if (!x) continue;
        if (cudaPointerGetAttributes(&at, x) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        if (!memory_of(at, device)) return false;
    }
    return true;
}

bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

sdv_status done(cudaError_t e) { return e == cudaSuccess ? SDV_OK : SDV_ERR_CUDA; }

unsigned test_hooks = 0;      // sdv_set_attn_test_hooks

cudaStream_t stream_of(void* s) { return static_cast<cudaStream_t>(s); }

// SM count of the current device (asked once per device), 0 on failure.
int sm_count() {
    constexpr int kDevices = 64;
    static int known[kDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) {
        cudaGetLastError();
        return 0;
    }
    int n = __atomic_load_n(&known[dev], __ATOMIC_RELAXED);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        __atomic_store_n(&known[dev], n, __ATOMIC_RELAXED);
    }
    return n;
}

// A cache's own checks; `dtype` is the type of what is written, read or asked.
bool cache_ok(const sdv_kv_cache* c, sdv_dtype dtype, bool any_type, CacheView* v) {
    if (!c || !c->k || !c->v) return false;
    const bool e4m3 = c->dtype == SDV_E4M3;
    if (!e4m3 && c->dtype != SDV_BF16 && c->dtype != SDV_F16) return false;
    if (!any_type && dtype != SDV_BF16 && dtype != SDV_F16) return false;
    if (!any_type && !e4m3 && dtype != c->dtype) return false;
    if (c->pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->kv_heads > 4096) return false;
    if (c->head_dim < 16 || c->head_dim > kCacheMaxDim || c->head_dim % 16) return false;
    const int64_t rows = static_cast<int64_t>(c->kv_heads) * c->page_size;      // of a page
    if (rows > (int64_t(1) << 30)) return false;
    const int cell = e4m3 ? 1 : 2;
    if (c->page_stride < rows * c->head_dim || c->page_stride > (int64_t(1) << 40)) return false;
    if ((c->page_stride * cell) % 16 || misaligned(c->k, 16) || misaligned(c->v, 16)) return false;
    if (e4m3 ? !c->k_exp || !c->v_exp || c->exp_page_stride < rows || c->exp_page_stride > (int64_t(1) << 40)
             : c->k_exp || c->v_exp)
        return false;
    const void* ptrs[4] = {c->k, c->v, c->k_exp, c->v_exp};
    if (!all_device(ptrs)) return false;
    v->k = static_cast<unsigned char*>(c->k);
    v->v = static_cast<unsigned char*>(c->v);
    v->ke = c->k_exp;
    v->ve = c->v_exp;
    v->page_stride = c->page_stride * cell;
    v->exp_page_stride = c->exp_page_stride;
    v->pages = c->pages;
    v->P = c->page_size;
    v->H = c->kv_heads;
    v->D = c->head_dim;
    return true;
}

// B sequences of N positions each, and the table of their pages.
bool spans_ok(const CacheView& v, int B, int N, const int32_t* table, int max_pages) {
    if (B < 1 || N < 1 || max_pages < 1 || !table || misaligned(table, 4)) return false;
    if (static_cast<int64_t>(max_pages) * v.P > (int64_t(1) << 30)) return false;
    return static_cast<int64_t>(B) * N <= (int64_t(1) << 36) / (2 * v.H * 32);
}

}  // namespace

extern "C" {

sdv_status sdv_tree_build(int B, int K, int gamma, void* stream, const int32_t* root,
                          const int32_t* drafts, const int32_t* draft_len, int32_t* tokens,
                          int32_t* depth, int32_t* mask, int32_t* nodes, int32_t* rows,
                          int32_t* count, int32_t* status) {
    if (B < 1 || K < 1 || K > kTreeMaxDrafts || gamma < 1 || gamma > kTreeMaxGamma) return SDV_ERR_ARG;
    if (!root || !drafts || !tokens || !depth || !mask || !nodes || !rows || !count) return SDV_ERR_ARG;
    const void* ptrs[10] = {root, drafts, draft_len, tokens, depth, mask, nodes, rows, count, status};
    for (const void* p : ptrs)
        if (misaligned(p, 4)) return SDV_ERR_ARG;
    if (!all_device(ptrs)) return SDV_ERR_ARG;
    TreeArgs a{};
    a.root = root, a.drafts = drafts, a.draft_len = draft_len;
    a.tokens = tokens, a.depth = depth, a.mask = mask, a.nodes = nodes, a.rows = rows, a.count = count;
    a.status = reinterpret_cast<unsigned*>(status);
    a.B = B, a.K = K, a.G = gamma, a.N = 1 + K * gamma, a.W = (a.N + 31) / 32;
    return done(launch_tree_build(a, stream_of(stream)));
}

sdv_status sdv_rope_freqs(int R, double base, int scaling, double factor, double original,
                          double fast, double slow, float* inv_freq, float* attn_factor) {
    if (R < 2 || R > kRopeMaxDim || R % 2 || !inv_freq || !(base > 0.0) || !std::isfinite(base)) return SDV_ERR_ARG;
    if (scaling < SDV_ROPE_PLAIN || scaling > SDV_ROPE_PARTS) return SDV_ERR_ARG;
    if (scaling != SDV_ROPE_PLAIN && !(factor >= 1.0 && std::isfinite(factor))) return SDV_ERR_ARG;
    if (scaling == SDV_ROPE_BASE && R < 4) return SDV_ERR_ARG;
    if (scaling == SDV_ROPE_PARTS &&
        !(fast > slow && slow >= 0.0 && std::isfinite(fast) && original >= 1.0 && std::isfinite(original)))
        return SDV_ERR_ARG;
    if (scaling == SDV_ROPE_BASE) base *= std::pow(factor, static_cast<double>(R) / (R - 2));
    for (int i = 0; i < R / 2; ++i) {
        double f = std::pow(base, -2.0 * i / R);
        if (scaling == SDV_ROPE_LINEAR) f /= factor;
        if (scaling == SDV_ROPE_PARTS) {
            const double turns = original * f / 6.283185307179586477;
            double keep = (turns - slow) / (fast - slow);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = f * keep + f / factor * (1.0 - keep);
        }
        inv_freq[i] = static_cast<float>(f);
    }
    if (attn_factor)
        *attn_factor = scaling == SDV_ROPE_PARTS ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return SDV_OK;
}

sdv_status sdv_rope(int64_t T, int Hq, int Hk, int D, int R, int interleaved, sdv_dtype dtype,
                    void* stream, const void* q, int64_t q_st, int64_t q_sh, const void* k,
                    int64_t k_st, int64_t k_sh, const int32_t* positions, const float* inv_freq,
                    float factor, void* out_q, int64_t oq_st, int64_t oq_sh, void* out_k,
                    int64_t ok_st, int64_t ok_sh) {
    if (dtype != SDV_BF16 && dtype != SDV_F16 && dtype != SDV_F32) return SDV_ERR_ARG;
    if (T < 0 || T > (int64_t(1) << 40) || Hq < 1 || Hk < 0 || Hq > 4096 || Hq + Hk > 4096) return SDV_ERR_ARG;
    if (D < 2 || D > 4096 || R < 2 || R > D || R > kRopeMaxDim || R % 2) return SDV_ERR_ARG;
    if (T == 0) return SDV_OK;
    if (!q || !out_q || !positions || !inv_freq || (Hk > 0 && (!k || !out_k)) || (Hk == 0 && (k || out_k)))
        return SDV_ERR_ARG;
    const int elt = dtype == SDV_F32 ? 4 : 2;
    const void* ptrs[6] = {q, k, out_q, out_k, positions, inv_freq};
    for (int i = 0; i < 6; ++i)
        if (misaligned(ptrs[i], i < 4 ? elt : 4)) return SDV_ERR_ARG;
    // in place means the same rows: anything else would read what it has written
    if ((q == out_q && (q_st != oq_st || q_sh != oq_sh)) || (k && k == out_k && (k_st != ok_st || k_sh != ok_sh)))
        return SDV_ERR_ARG;
    if (!all_device(ptrs)) return SDV_ERR_ARG;
    const int nsm = sm_count();
    if (nsm < 1) return SDV_ERR_CUDA;
    RopeArgs a{};
    a.q = q, a.k = k, a.oq = out_q, a.ok = out_k;
    a.q_st = q_st * elt, a.q_sh = q_sh * elt, a.k_st = k_st * elt, a.k_sh = k_sh * elt;
    a.oq_st = oq_st * elt, a.oq_sh = oq_sh * elt, a.ok_st = ok_st * elt, a.ok_sh = ok_sh * elt;
    a.pos = positions, a.freq = inv_freq, a.factor = factor;
    a.T = T, a.Hq = Hq, a.Hk = Hk, a.D = D, a.R = R, a.interleaved = interleaved != 0;
    // 16-byte vectors when every row starts on one and holds whole pairs of them
    const int E = 16 / elt;
    const int64_t steps = a.q_st | a.q_sh | a.oq_st | a.oq_sh | a.k_st | a.k_sh | a.ok_st | a.ok_sh;
    bool vec = R % (2 * E) == 0 && D % E == 0 && (steps & 15) == 0;
    for (int i = 0; i < 4; ++i) vec = vec && !misaligned(ptrs[i], 16);
    return done(launch_rope(a, dtype, vec, nsm, stream_of(stream)));
}

sdv_status sdv_kv_write(const sdv_kv_cache* cache, int B, int N, sdv_dtype dtype, void* stream,
                        const void* k, int64_t k_sb, int64_t k_sn, int64_t k_sh, const void* v,
                        int64_t v_sb, int64_t v_sn, int64_t v_sh, const int32_t* block_table,
                        int max_pages, const int32_t* start, const int32_t* count,
                        int32_t* status) {
    CellsArgs a{};
    if (!cache_ok(cache, dtype, false, &a.c) || !spans_ok(a.c, B, N, block_table, max_pages)) return SDV_ERR_ARG;
    if (!k || !v || !start || misaligned(k, 2) || misaligned(v, 2) || misaligned(start, 4) ||
        misaligned(count, 4) || misaligned(status, 4))
        return SDV_ERR_ARG;
    const void* ptrs[6] = {k, v, block_table, start, count, status};
    if (!all_device(ptrs)) return SDV_ERR_ARG;
    a.k = static_cast<const unsigned char*>(k);
    a.v = static_cast<const unsigned char*>(v);
    a.k_sb = k_sb * 2, a.k_sn = k_sn * 2, a.k_sh = k_sh * 2;
    a.v_sb = v_sb * 2, a.v_sn = v_sn * 2, a.v_sh = v_sh * 2;
    a.table = block_table, a.start = start, a.count = count;
    a.status = reinterpret_cast<unsigned*>(status);
    a.B = B, a.N = N, a.max_pages = max_pages;
    const bool vec = !misaligned(k, 16) && !misaligned(v, 16) &&
                     ((a.k_sb | a.k_sn | a.k_sh | a.v_sb | a.v_sn | a.v_sh) & 15) == 0;
    return done(launch_kv_write(a, dtype, cache->dtype == SDV_E4M3, vec, stream_of(stream)));
}

sdv_status sdv_kv_read(const sdv_kv_cache* cache, int B, int N, sdv_dtype dtype, void* stream,
                       void* out_k, void* out_v, const int32_t* block_table, int max_pages,
                       const int32_t* start, const int32_t* count, int32_t* status) {
    CellsArgs a{};
    if (!cache_ok(cache, dtype, false, &a.c) || !spans_ok(a.c, B, N, block_table, max_pages)) return SDV_ERR_ARG;
    if (!out_k || !out_v || !start || misaligned(out_k, 16) || misaligned(out_v, 16) || misaligned(start, 4) ||
        misaligned(count, 4) || misaligned(status, 4))
        return SDV_ERR_ARG;
    const void* ptrs[6] = {out_k, out_v, block_table, start, count, status};
    if (!all_device(ptrs)) return SDV_ERR_ARG;
    a.ok = out_k, a.ov = out_v;
    a.table = block_table, a.start = start, a.count = count;
    a.status = reinterpret_cast<unsigned*>(status);
    a.B = B, a.N = N, a.max_pages = max_pages;
    return done(launch_kv_read(a, dtype, cache->dtype == SDV_E4M3, stream_of(stream)));
}

sdv_status sdv_kv_commit(const sdv_kv_cache* cache, int B, int K, int gamma, void* stream,
                         const int32_t* block_table, int max_pages, const int32_t* start,
                         const int32_t* nodes, const int32_t* sel, const int32_t* accept_len,
                         int32_t* out_len, int32_t* status) {
    CommitArgs a{};
    if (K < 1 || gamma < 1 || static_cast<int64_t>(K) * gamma > (int64_t(1) << 24)) return SDV_ERR_ARG;
    if (!cache_ok(cache, SDV_BF16, true, &a.c) || !spans_ok(a.c, B, 1, block_table, max_pages)) return SDV_ERR_ARG;
    if (!start || !nodes || !sel || !accept_len) return SDV_ERR_ARG;
    const void* ptrs[7] = {block_table, start, nodes, sel, accept_len, out_len, status};
    for (const void* p : ptrs)
        if (misaligned(p, 4)) return SDV_ERR_ARG;
    if (!all_device(ptrs)) return SDV_ERR_ARG;
    a.cell = cache->dtype == SDV_E4M3 ? 1 : 2;
    a.table = block_table, a.start = start, a.nodes = nodes, a.sel = sel, a.acc = accept_len;
    a.out_len = out_len;
    a.status = reinterpret_cast<unsigned*>(status);
    a.B = B, a.K = K, a.G = gamma, a.max_pages = max_pages;
    return done(launch_kv_commit(a, stream_of(stream)));
}

sdv_status sdv_logits_process(int B, int K, int gamma, int V, sdv_dtype dtype, void* stream,
                              const void* logits, int nsrc, const int32_t* rows,
                              const int32_t* drafts, const int32_t* counts, const int32_t* prompt,
                              const float* repetition, const float* frequency,
                              const float* presence, int M, const int32_t* bias_ids,
                              const float* bias, const int32_t* allow, void* out,
                              int32_t* status) {
    if (dtype != SDV_BF16 && dtype != SDV_F32) return SDV_ERR_ARG;
    if (B < 1 || K < 1 || gamma < 1 || V < 1 || M < 0 || M > (1 << 24)) return SDV_ERR_ARG;
    const int elt = dtype == SDV_BF16 ? 2 : 4;
    if ((static_cast<int64_t>(V) * elt) % 16 || V > (1 << 28)) return SDV_ERR_ARG;
    if (static_cast<int64_t>(B) * K * (gamma + 1) > (int64_t(1) << 27)) return SDV_ERR_ARG;
    if (static_cast<int64_t>(B) * K * (V / 1024 + 1) >= (int64_t(1) << 31) || gamma > 65535 ||
        static_cast<int64_t>(K) * (gamma + 1) > (int64_t(1) << 25))
        return SDV_ERR_ARG;
    if (!logits || !drafts || !out || misaligned(logits, 16) || misaligned(out, 16) || misaligned(counts, 16))
        return SDV_ERR_ARG;
    if (rows ? nsrc < 1 || out == logits : false) return SDV_ERR_ARG;
    if (M > 0 ? !bias_ids || !bias : bias_ids || bias) return SDV_ERR_ARG;
    const void* ptrs[13] = {rows, drafts, prompt, repetition, frequency, presence, bias_ids, bias, allow, status,
                            logits, counts, out};
    for (const void* p : ptrs)
        if (misaligned(p, 4)) return SDV_ERR_ARG;
    if (!all_device(ptrs)) return SDV_ERR_ARG;
    const int nsm = sm_count();
    if (nsm < 1) return SDV_ERR_CUDA;
    LogitsArgs a{};
    a.logits = logits, a.out = out, a.rows = rows, a.drafts = drafts, a.counts = counts, a.prompt = prompt;
    a.bias_ids = bias_ids, a.allow = allow, a.rep = repetition, a.freq = frequency, a.pres = presence, a.bias = bias;
    a.status = reinterpret_cast<unsigned*>(status);
    a.B = B, a.K = K, a.G = gamma, a.V = V, a.nsrc = nsrc, a.M = M, a.W = (V + 31) / 32;
    return done(launch_logits(a, dtype == SDV_BF16, nsm, stream_of(stream)));
}

sdv_status sdv_counts_commit(int B, int K, int gamma, int V, void* stream, const int32_t* drafts,
                             const int32_t* sel, const int32_t* accept_len,
                             const int32_t* next_token, int32_t* counts, int32_t* status) {
    if (B < 1 || K < 1 || gamma < 1 || V < 1) return SDV_ERR_ARG;
    if (!drafts || !sel || !accept_len || !next_token || !counts) return SDV_ERR_ARG;
    const void* ptrs[6] = {drafts, sel, accept_len, next_token, counts, status};
    for (const void* p : ptrs)
        if (misaligned(p, 4)) return SDV_ERR_ARG;
    if (!all_device(ptrs)) return SDV_ERR_ARG;
    CountsArgs a{};
    a.drafts = drafts, a.sel = sel, a.acc = accept_len, a.next = next_token, a.counts = counts;
    a.status = reinterpret_cast<unsigned*>(status);
    a.B = B, a.K = K, a.G = gamma, a.V = V;
    return done(launch_counts_commit(a, stream_of(stream)));
}

sdv_status sdv_set_attn_test_hooks(unsigned hooks) {
    if (hooks & ~kHookAttnNoCopy) return SDV_ERR_ARG;
    __atomic_store_n(&test_hooks, hooks, __ATOMIC_RELAXED);
    return SDV_OK;
}

size_t sdv_tree_attn_workspace(void) {
    const int nsm = sm_count();
    return nsm > 0 ? attn_workspace_bytes(nsm) : 0;
}

sdv_status sdv_tree_attn(const sdv_kv_cache* cache, int B, int N, int Hq, sdv_dtype dtype,
                         void* stream, const void* q, int64_t q_sb, int64_t q_sn, int64_t q_sh,
                         const int32_t* block_table, int max_pages, const int32_t* ctx_len,
                         const int32_t* count, const int32_t* mask, int64_t mask_sb, float scale,
                         void* out, float* lse, void* workspace, size_t workspace_bytes,
                         int32_t* status) {
    AttnArgs a{};
    if (!cache_ok(cache, dtype, false, &a.c) || !spans_ok(a.c, B, N, block_table, max_pages)) return SDV_ERR_ARG;
    if (Hq < 1 || Hq % a.c.H || N > (1 << 20) || !std::isfinite(scale)) return SDV_ERR_ARG;
    a.g = Hq / a.c.H;
    if (static_cast<int64_t>(N) * a.g > (int64_t(1) << 28)) return SDV_ERR_ARG;
    if (!q || !ctx_len || !out || !workspace) return SDV_ERR_ARG;
    if (misaligned(q, 2) || misaligned(out, 32) || misaligned(workspace, 32)) return SDV_ERR_ARG;
    const void* ptrs[9] = {ctx_len, count, mask, lse, status, block_table, q, out, workspace};
    for (int i = 0; i < 6; ++i)
        if (misaligned(ptrs[i], 4)) return SDV_ERR_ARG;
    if (!all_device(ptrs)) return SDV_ERR_ARG;
    const int nsm = sm_count();
    if (nsm < 1) return SDV_ERR_CUDA;
    if (workspace_bytes < attn_workspace_bytes(nsm)) return SDV_ERR_SCRATCH;
    a.q = static_cast<const unsigned char*>(q);
    a.q_sb = q_sb * 2, a.q_sn = q_sn * 2, a.q_sh = q_sh * 2;
    a.table = block_table, a.ctx = ctx_len, a.count = count, a.mask = mask, a.mask_sb = mask_sb;
    a.out = out, a.lse = lse;
    a.status = reinterpret_cast<unsigned*>(status);
    a.B = B, a.N = N, a.Hq = Hq, a.W = (N + 31) / 32, a.max_pages = max_pages;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.hooks = __atomic_load_n(&test_hooks, __ATOMIC_RELAXED);
    return done(launch_tree_attn(a, dtype, cache->dtype == SDV_E4M3, workspace, nsm, stream_of(stream)));
}

}  // extern "C"
