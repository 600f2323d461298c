// k8_attn_tma.cuh -- what the attention kernels that bring tiles by tile copies
// share: bounded barrier waits, the copies, their tensor maps.
#pragma once

#include <cuda.h>

#include "k8_attn.cuh"

namespace sdv {
namespace {

constexpr uint32_t kPolls = 1u << 17, kPollNs = 20000;     // a wait's limit: so many polls, each sleeping that long at most
constexpr uint32_t kHookPolls = 1u << 12;                  // ... under the test hook

// A wait that gives up marks its CTA dead.  From then on no wait waits and no
// copy is begun.  Phases may then be out of step, so that a later wait finds its
// phase over although nothing came: whatever is handed on is only good if the
// CTA is not dead when it is written, which `is_dead` is asked then.  (The mark is
// set before the arrivals that what was not waited for leads to.)
struct Sync {
    uint32_t bar, dead;      // shared-memory addresses
    unsigned* status;
    uint32_t polls;
    __device__ __forceinline__ bool is_dead() const {
        uint32_t d;
        asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(d) : "r"(dead) : "memory");
        return d != 0;
    }
    __device__ __forceinline__ bool test(int i, uint32_t parity) const {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done) : "r"(bar + i * 8), "r"(parity) : "memory");
        return done != 0;
    }
    // sleeps until the phase is over or for some time: a warp that keeps asking
    // holds up the shared-memory accesses of the others
    __device__ __forceinline__ bool poll(int i, uint32_t parity) const {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done) : "r"(bar + i * 8), "r"(parity), "r"(kPollNs) : "memory");
        return done != 0;
    }
    // false: the CTA is dead
    __device__ __forceinline__ bool wait(int i, uint32_t parity) const {
        for (uint32_t n = 0; n < polls; ++n) {
            if (poll(i, parity)) return true;
            if (is_dead()) return false;
        }
        asm volatile("st.volatile.shared.u32 [%0], 1;" ::"r"(dead) : "memory");
        if (status) atomicOr(status, kStatusTimeout);
        return false;
    }
    // The copies that complete phase `parity` have landed (or the limit is over).
    __device__ __forceinline__ void landed(int i, uint32_t parity) const {
        for (uint32_t n = 0; n < polls && !poll(i, parity); ++n) {}
    }
    __device__ __forceinline__ void arrive(int i) const {
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar + i * 8) : "memory");
    }
    __device__ __forceinline__ void commit(int i) const {
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar + i * 8) : "memory");
    }
};

// Tile copy of the box at (x, row, page) into shared memory.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int row, int page) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(row), "r"(page) : "memory");
}
// This thread's ordinary accesses to shared memory come before the copies (and
// products) that a barrier after this lets begin.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
// One thread of a converged warp, and a value that is the same in all of them.
__device__ __forceinline__ bool elected() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

// Cells as [pages][kv_heads * page_size][head_dim]; boxes of `rows` rows of 64
// 16-bit or 128 e4m3 cells, in the 128-byte swizzle or not; what lies past
// head_dim is 0.
bool encode_cells(CUtensorMap* map, const AttnArgs& a, unsigned char* cells, bool e4m3, int rows, bool swizzle) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const int cell = e4m3 ? 1 : 2;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.c.D), static_cast<cuuint64_t>(a.c.H) * a.c.P,
                                static_cast<cuuint64_t>(a.c.pages)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.c.D) * cell, static_cast<cuuint64_t>(a.c.page_stride)};
    const cuuint32_t box[3] = {e4m3 ? 128u : 64u, static_cast<cuuint32_t>(rows), 1u}, one[3] = {1u, 1u, 1u};
    return f(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, cells, dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace sdv
