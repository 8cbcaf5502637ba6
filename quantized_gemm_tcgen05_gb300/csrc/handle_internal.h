// Internal accessors of the opaque gemm handle for other translation units of
// the library.
#pragma once
#include <cuda.h>
#include <stddef.h>
#include <stdint.h>

#include "gemm.h"

namespace qg {
// CUDA device ordinal the handle is bound to, or -1 for a NULL handle.
int handle_device(gemm_handle_t h);
// Makes the handle's device current (GEMM_OK or GEMM_ERR_CUDA).
int handle_bind(gemm_handle_t h);
// Whether p is device (or managed) memory; remembers recent answers.
bool handle_device_pointer(gemm_handle_t h, const void* p);
// cuTensorMapEncodeTiled through the handle's map cache: byte-typed or 8-byte
// elements, zero fill out of bounds.  GEMM_OK or GEMM_ERR_CUDA.
int handle_encode(gemm_handle_t h, CUtensorMap* m, CUtensorMapDataType type, uint32_t rank, const void* ptr,
                  const uint64_t* dims, const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swizzle);
int handle_sm_count(gemm_handle_t h);
uint32_t* handle_status(gemm_handle_t h);
uint64_t handle_timeout_ns(gemm_handle_t h);
// Records the kernel chosen for the call (gemm_last_choice; logged with GEMM_LOG=1).
void handle_set_choice(gemm_handle_t h, const char* name, int64_t m, int64_t n, int64_t k);
}  // namespace qg
