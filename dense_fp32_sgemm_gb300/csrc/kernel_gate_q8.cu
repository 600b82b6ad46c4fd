// The gate that leaves in 8 bits, and plain rows: row_kernel.cuh.
#include "row_kernel.cuh"

namespace sgemm {

cudaError_t launch_gate_q8(const RowParams &p, int type, bool vec, int num_sms, cudaStream_t stream) {
    if (!p.b) return launch_rows_of<kRowGateQ8, -1>(p, type, vec, num_sms, stream);
    switch (p.act) {
        case kGateSilu: return launch_rows_of<kRowGateQ8, kGateSilu>(p, type, vec, num_sms, stream);
        case kGateGelu: return launch_rows_of<kRowGateQ8, kGateGelu>(p, type, vec, num_sms, stream);
        default: return launch_rows_of<kRowGateQ8, kGateRelu>(p, type, vec, num_sms, stream);
    }
}

}  // namespace sgemm
