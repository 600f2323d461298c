// k8_attn.cu -- tree attention (sdv_tree_attn): which kernel runs, and the join
// of the partial results of units that several CTAs share.
#include "k8_attn.cuh"

namespace sdv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxCtasPerSm = 2;

// Query rows per kv head up to which k8_attn_dec.cu runs, in units of 16 rows;
// above, k8_attn_tc.cu, whose time hardly depends on the rows up to 256.  Times
// for 32 sequences of 4000 positions, 8 kv heads of 128: 16-bit caches, 16 rows
// 100 and 117 us, 24 rows 178 (when the first took them) and 118 us; e4m3 caches,
// which the second has to widen in shared memory first, 48 rows 207 and 322 us, 80
// rows 326 and 330, 128 rows 495 and 342.  (Heads of 64, 16 bits: 16 rows 59 and 96
// us, 48 rows 139 and 97; e4m3: 80 rows 220 and 262 us, 128 rows 339 and 265.)  Two
// sequences of 100000: 16 bits, 16 rows 143 and 161 us; e4m3, 80 rows 405 and 476 us,
// 128 rows 626 and 478; one of 20000: e4m3, 80 rows 70 and 68 us, 128 rows 91 and 68.
constexpr int kDecRows = 16, kDecRowsE4m3 = 80;

// out = sum_i 2^(L_i - L) out_i with L = log2 sum_i 2^(L_i), over the CTAs that
// share a unit, in the CTAs' order.  One column of the grid per CTA of the kernel
// before, most of which find nothing to do; up to 16 blocks deep, so that the
// round trips of a unit's parts are shared (2 chains of 177 nodes, 13 parts a
// unit: 21 us in 16, 38 us in 8 that read twice; 32 gain nothing more).
// RAW: rows go out as fp32, for the kernel that this one lets begin (shared prefixes).
template <bool F16, bool RAW>
__global__ void __launch_bounds__(kThreads) combine_kernel(const AttnArgs a, int MT) {
    if (RAW) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 d0 = a.desc[2 * blockIdx.x];
    if (d0.x < 0) return;
    const int b = d0.x, h = d0.y, mt = d0.z, first = d0.w, last = a.desc[2 * blockIdx.x + 1].x;
    const int D = a.c.D, vec = D / 4;
    const float nan_value = __int_as_float(0x7fc00000);
    for (int w = threadIdx.x + blockIdx.y * kThreads; w < MT * vec; w += kThreads * gridDim.y) {
        const int r = w / vec, d = (w % vec) * 4;
        const int row = mt * MT + r, node = row / a.g;
        if (node >= a.N) continue;
        // eight parts' loads at once, their sum in units of the largest so far
        float top = -INFINITY, sum = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        bool nan = false;
        for (int i0 = first; i0 <= last; i0 += 8) {
            float L[8];
            float4 v[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                L[y] = -INFINITY, v[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (i0 + y > last) continue;
                const float* p = attn::part_rows(a, i0 + y, i0 + y == first, MT);
                L[y] = p[MT * D + r];
                v[y] = *reinterpret_cast<const float4*>(p + r * D + d);
            }
            float to = top;
#pragma unroll
            for (int y = 0; y < 8; ++y) to = fmaxf(to, L[y]), nan |= L[y] != L[y];
            const float base = to == -INFINITY ? 0.0f : to, by = ex2(top - base);
            top = to;
            sum *= by, acc[0] *= by, acc[1] *= by, acc[2] *= by, acc[3] *= by;
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const float f = ex2(L[y] - base);
                sum += f;
                acc[0] += v[y].x * f, acc[1] += v[y].y * f, acc[2] += v[y].z * f, acc[3] += v[y].w * f;
            }
        }
        const float inv = nan ? nan_value : sum == 0.0f ? 0.0f : 1.0f / sum;
        const int64_t orow = (static_cast<int64_t>(b) * a.N + node) * a.Hq + h * a.g + row % a.g;
        const float x[4] = {acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv};
        attn::store_row4<F16, RAW>(a, orow, d, x, nan ? nan_value : sum == 0.0f ? -INFINITY : top + log2f(sum));
    }
}

}  // namespace

cudaError_t launch_attn_combine(const AttnArgs& a, bool f16, int MT, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    const int blocks = (MT * (a.c.D / 4) + kThreads - 1) / kThreads;        // 16 rows of 128: two
    cfg.gridDim = dim3(static_cast<unsigned>(a.ctas), static_cast<unsigned>(blocks < 16 ? blocks : 16));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (a.raw)
        return f16 ? cudaLaunchKernelEx(&cfg, combine_kernel<true, true>, a, MT) : cudaLaunchKernelEx(&cfg, combine_kernel<false, true>, a, MT);
    return f16 ? cudaLaunchKernelEx(&cfg, combine_kernel<true, false>, a, MT) : cudaLaunchKernelEx(&cfg, combine_kernel<false, false>, a, MT);
}

size_t attn_workspace_bytes(int nsm) {
    // two partial results per CTA: 256 rows of up to 128 (one CTA per SM), 64
    // rows of up to 256 (two), which covers 16 rows of up to 128 (two)
    const size_t tc = size_t(1) * 256 * (128 + 1), mma = size_t(2) * 64 * (kCacheMaxDim + 1);
    const size_t most = tc > mma ? tc : mma;
    return nsm * (kMaxCtasPerSm * 2 * sizeof(int4) + 2 * most * sizeof(float) + sizeof(unsigned));
}

bool attn_goes_on(const AttnArgs& a, bool f16, bool e4m3) {
    return attn_tma_takes(a) && a.N * a.g > (e4m3 ? kDecRowsE4m3 : kDecRows) && !(f16 && e4m3);
}

cudaError_t launch_tree_attn(AttnArgs a, int type, bool e4m3, void* workspace, int nsm, cudaStream_t s) {
    a.desc = static_cast<int4*>(workspace);
    a.part = reinterpret_cast<float*>(a.desc + 2 * kMaxCtasPerSm * nsm);
    a.beyond = reinterpret_cast<unsigned*>(static_cast<unsigned char*>(workspace) + attn_workspace_bytes(nsm)) - nsm;
    const bool f16 = type == kTypeF16;
    const int rows = a.N * a.g;
    if (attn_tma_takes(a)) {
        if (rows <= (e4m3 ? kDecRowsE4m3 : kDecRows)) return launch_attn_dec(a, f16, e4m3, nsm, s);
        const cudaError_t e = launch_attn_tc(a, f16, e4m3, nsm, s);
        return e == cudaSuccess && f16 && e4m3 ? launch_attn_redo(a, nsm, s) : e;
    }
    if (a.c.D <= 64) return launch_attn_mma64(a, f16, e4m3, rows, nsm, s);
    if (a.c.D <= 128) return launch_attn_mma128(a, f16, e4m3, rows, nsm, s);
    return launch_attn_mma256(a, f16, e4m3, rows, nsm, s);
}

}  // namespace sdv
