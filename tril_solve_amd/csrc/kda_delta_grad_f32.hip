// The delta rule's gradients for f32 inputs (a file per input type: they compile
// side by side).
#include "kda_delta_grad.h"

namespace kda {

hipError_t launch_delta_grad_f32(const DeltaGradProblem &p, int dout_dt, hipStream_t stream) {
    return launch_delta_grad_of<F32>(p, dout_dt, stream);
}

hipError_t launch_delta_grad_bf16(const DeltaGradProblem &p, int dout_dt, hipStream_t stream);
hipError_t launch_delta_grad_f16(const DeltaGradProblem &p, int dout_dt, hipStream_t stream);

hipError_t launch_delta_grad(const DeltaGradProblem &p, int in_dt, int dout_dt,
                             hipStream_t stream) {
    return in_dt == 0   ? launch_delta_grad_f32(p, dout_dt, stream)
           : in_dt == 1 ? launch_delta_grad_bf16(p, dout_dt, stream)
                        : launch_delta_grad_f16(p, dout_dt, stream);
}

}  // namespace kda
