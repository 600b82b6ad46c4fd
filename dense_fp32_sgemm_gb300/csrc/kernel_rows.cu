// The root-mean-square norm, and the norm that leaves in 8 bits: row_kernel.cuh.
#include "row_kernel.cuh"

namespace sgemm {

cudaError_t launch_norm(const RowParams &p, int type, bool q8, bool vec, int num_sms,
                        cudaStream_t stream) {
    return q8 ? launch_rows_of<kRowNormQ8, -1>(p, type, vec, num_sms, stream)
              : launch_rows_of<kRowNorm, -1>(p, type, vec, num_sms, stream);
}

}  // namespace sgemm
