// k12_rows.cu -- draws from rows of logits and their truncation (sdv_sample,
// sdv_logits_truncate): rows in 32 bits.
//
// A CTA takes a row at a time and reads it in passes (row_in_passes): the largest
// logit; a histogram of counts and weights over 4096 bins of equal width in
// (max - x) / T, which keeps the order; then, for each of the places that are asked
// for (the last token that min-p and top-k keep, the last that top-p keeps, the one
// that is drawn), the bin that holds it is split by keys until one logit is left.
#include "k12_rows.cuh"

namespace sdv {
namespace {

using namespace rows;

constexpr int kThreads = 512, kBins = 4096;

template <bool DRAW> __global__ void __launch_bounds__(kThreads, 2) rows_f32_kernel(const RowsArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    PassSmem<kThreads, kBins>& sm = *reinterpret_cast<PassSmem<kThreads, kBins>*>(raw);
    load_tables(sm.tables, threadIdx.x, kThreads);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        row_in_passes<false, DRAW, kThreads, kBins>(a, r, sm);
        __syncthreads();
    }
}

template <bool DRAW> cudaError_t launch(const RowsArgs& a, int nsm, cudaStream_t s) {
    constexpr size_t bytes = sizeof(PassSmem<kThreads, kBins>);
    const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(rows_f32_kernel<DRAW>), bytes);
    if (e != cudaSuccess) return e;
    const int64_t ctas = a.rows < 2 * nsm ? a.rows : 2 * nsm;
    rows_f32_kernel<DRAW><<<static_cast<unsigned>(ctas), kThreads, bytes, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows(const RowsArgs& a, bool bf16, bool draw, int nsm, cudaStream_t s) {
    if (bf16) return launch_rows_bf16(a, draw, nsm, s);
    return draw ? launch<true>(a, nsm, s) : launch<false>(a, nsm, s);
}

}  // namespace sdv
