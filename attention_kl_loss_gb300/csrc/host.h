// Host helpers shared by the C-ABI files; defined in api.cu.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "streamkl.h"

namespace skl {
namespace host {

// This thread's detail message (streamkl_last_error): cleared at the start of
// a call, set by fail() / cuda_fail(), which return the status given.
void clear_error();
streamkl_status fail(streamkl_status s, const char* fmt, ...);
streamkl_status cuda_fail(cudaError_t e, const char* what);

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // null when the driver has none
uint64_t wait_timeout_ns();                     // limit of one wait inside a kernel
int num_sms();                                  // of the current device
bool aligned16(const void* p);

}  // namespace host
}  // namespace skl
