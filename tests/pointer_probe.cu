// Host-only probe of memory_of in sdv_plan.h (no GPU, no kernel): for each input
// line "type device current" it prints 1 where the library takes such a pointer.
// Built and run by tests/test_pointer_host.py.
#include <cstdio>

#include "../draft_verification_sdv_gb300/csrc/sdv_plan.h"

int main() {
    int type, device, current;
    while (std::scanf("%d %d %d", &type, &device, &current) == 3) {
        cudaPointerAttributes at = {};
        at.type = static_cast<cudaMemoryType>(type);
        at.device = device;
        std::printf("%d\n", sdv::memory_of(at, current) ? 1 : 0);
    }
    return 0;
}
