// Launch of the gated delta rule over whole prompts.
#include "kda_prefill.h"

namespace kda {

hipError_t launch_prefill(const DeltaProblem &p, int in_dt, hipStream_t stream) {
    return in_dt == 0   ? launch_prefill_f32(p, stream)
           : in_dt == 1 ? launch_prefill_bf16(p, stream)
                        : launch_prefill_f16(p, stream);
}

}  // namespace kda
