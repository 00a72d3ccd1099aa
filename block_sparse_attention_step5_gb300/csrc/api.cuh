// api.cuh -- host-side helpers shared by the files that implement the C ABI.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "step5_sparse_attn.h"

namespace step5 {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

step5_status check_geometry(const step5_geometry* g);
uint32_t* status_ptr();  // the current device's status word, or null
int num_sms();           // of the current device
PFN_cuTensorMapEncodeTiled_v12000 get_encode();

}  // namespace step5
