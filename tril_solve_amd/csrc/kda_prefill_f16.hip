// The prefill kernels for f16 inputs (a file per input type: they compile side
// by side).
#include "kda_prefill.h"

namespace kda {

hipError_t launch_prefill_f16(const DeltaProblem &p, PrePass pass, hipStream_t stream) {
    return launch_prefill_of<F16>(p, pass, stream);
}

}  // namespace kda
