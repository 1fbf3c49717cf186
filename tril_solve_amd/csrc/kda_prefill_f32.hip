// The prefill kernels for f32 inputs (a file per input type: they compile side
// by side).
#include "kda_prefill.h"

namespace kda {

hipError_t launch_prefill_f32(const DeltaProblem &p, PrePass pass, hipStream_t stream) {
    return launch_prefill_of<F32>(p, pass, stream);
}

}  // namespace kda
