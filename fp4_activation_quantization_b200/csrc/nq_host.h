// nq_host.h — host helpers of the library that more than one translation unit
// uses; defined in nq_host.cu.  Not installed.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "nq.h"

namespace nq {
namespace host {

// Records the message that nq_last_error returns on this thread; returns st.
nq_status error(nq_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Launches `kernel` (nullptr: NQ_ERR_UNSUPPORTED).
nq_status launch(const char* fn, const void* kernel, unsigned grid, unsigned block, size_t smem, void** args, bool pdl,
                 cudaStream_t stream);
// The current device's error word (nullptr: no device).
uint32_t* error_word();
// Opts `kernel` in to `bytes` of dynamic shared memory on the current device.
bool allow_smem(const void* kernel, size_t bytes);
// CTAs of `kernel` that the current device holds at once (0: unknown).
int64_t resident_ctas(const void* kernel, int block, size_t smem);

}  // namespace host
}  // namespace nq
