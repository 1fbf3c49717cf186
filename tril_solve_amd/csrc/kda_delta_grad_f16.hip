// The delta rule's gradients for f16 inputs (a file per input type: they compile
// side by side).
#include "kda_delta_grad.h"

namespace kda {

hipError_t launch_delta_grad_f16(const DeltaGradProblem &p, int dout_dt, hipStream_t stream) {
    return launch_delta_grad_of<F16>(p, dout_dt, stream);
}

}  // namespace kda
