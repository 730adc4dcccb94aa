// mrn_gate_backward_bf16.cu -- the gradient of the gated tail over bf16 rows.
#include "mrn_gate_backward.cuh"

namespace mrn {

cudaError_t launch_gate_backward_bf16(const GateBackwardArgs &a, int sms, bool pdl, cudaStream_t stream,
                                     uint64_t *launches) {
    return launch_gate_backward_typed<BF16>(a, sms, pdl, stream, launches);
}

int take_wait_timeouts_gate_backward_bf16() { return take_wait_timeouts<kOpGateBackwardBF16Timeouts>(); }

}  // namespace mrn
