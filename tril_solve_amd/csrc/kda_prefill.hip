// Gated delta rule over whole prompts for gfx950.
#include <hip/hip_runtime.h>

#include "kda_layer.h"

namespace kda {

// Token by token, as the recurrent form does.
hipError_t launch_prefill(const DeltaProblem &p, int in_dt, hipStream_t stream) {
    return launch_recurrent(p, in_dt, stream);
}

}  // namespace kda
