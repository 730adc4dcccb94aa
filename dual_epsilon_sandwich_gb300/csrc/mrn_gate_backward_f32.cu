// mrn_gate_backward_f32.cu -- the gradient of the gated tail over f32 rows.
#include "mrn_gate_backward.cuh"

namespace mrn {

cudaError_t launch_gate_backward_f32(const GateBackwardArgs &a, int sms, bool pdl, cudaStream_t stream,
                                     uint64_t *launches) {
    return launch_gate_backward_typed<F32>(a, sms, pdl, stream, launches);
}

int take_wait_timeouts_gate_backward_f32() { return take_wait_timeouts<kOpGateBackwardF32Timeouts>(); }

}  // namespace mrn
