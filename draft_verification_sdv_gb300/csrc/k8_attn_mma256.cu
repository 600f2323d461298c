// k8_attn_mma256.cu -- tree attention on mma.sync for head dimensions up to 256.
#include "k8_attn_mma.cuh"

namespace sdv {

cudaError_t launch_attn_mma256(const AttnArgs& a, bool f16, bool e4m3, int rows, int nsm, cudaStream_t s) {
    return launch_dim<256>(a, f16, e4m3, rows, nsm, s);
}

}  // namespace sdv
