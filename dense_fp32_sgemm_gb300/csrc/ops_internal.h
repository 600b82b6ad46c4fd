// What api.cu lends the translation units of the operators around it: its
// lock, the per-device state, a workspace per (device, stream) and the TMA
// descriptor encoder.  Host-visible only.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "../../include/sgemm.h"

namespace sgemm {

struct OpDevice {
    int index;    // device ordinal
    int num_sms;
    int *err;     // device error word (sgemm_device_status reads and clears it)
    unsigned long long timeout_ns;
    int skip_loads_from;  // testing hook, -1 = off
};

// Held for the whole of an entry point: guards the state the others return.
std::mutex &api_mutex();

// The current device's state, created on first use.
sgemm_status_t op_device(OpDevice *out);

// Grow-only workspace of the current device and `stream`, kept until
// sgemm_release_workspace().  The buffer's contents do not survive a call.
sgemm_status_t op_workspace(cudaStream_t stream, size_t bytes, void **out);

// Arrival counters of the current device and `stream`, zero at rest (and
// cleared by sgemm_device_status() after a wait that gave up).
sgemm_status_t op_counters(cudaStream_t stream, size_t count, int **out);

// `planes` row-major rows x cols matrices of 16-bit elements (bf16 or fp16),
// rows ld and planes plane_stride elements apart; boxes of box_planes planes,
// box_rows x 64 of each, 128-byte swizzle, zero outside.
sgemm_status_t op_encode_16(CUtensorMap *map, bool bf16, const void *base, int64_t rows,
                            int64_t cols, int64_t ld, int64_t planes, int64_t plane_stride,
                            int box_rows, int box_planes = 1);

// Row-major rows x cols matrix of 32-bit words, rows ld words apart; boxes of
// box_rows x box_cols, 128-byte swizzle, zero outside.
sgemm_status_t op_encode_words(CUtensorMap *map, const uint32_t *base, int64_t rows, int64_t cols,
                               int64_t ld, int box_cols, int box_rows);

// Row-major rows x cols matrix of bytes, rows ld bytes apart (a multiple of 16);
// boxes of box_rows x 128, 128-byte swizzle, zero outside.
sgemm_status_t op_encode_bytes(CUtensorMap *map, const void *base, int64_t rows, int64_t cols,
                               int64_t ld, int box_rows);

}  // namespace sgemm
