// api_internal.h -- host helpers shared by the C ABI translation units
// (api.cu, decode_api.cu): the thread's error string, the per-device set-up,
// tensor-map encoding and argument checks.  Not part of the public interface.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

// Records the message moe_last_error_string() returns; yields `code`.
int fail(int code, const char* fmt, ...);
int cuda_fail(cudaError_t e, const char* what);

constexpr int kMaxDevices = 64;

// Sets the current device up on its first use (attributes of moe.h's kernels,
// the tensor-map encoder) and yields its SM count.
int device_setup(int* sms);

// Tensor map of `rank` dimensions, zero fill out of bounds.  Needs a
// device_setup() that succeeded.
int encode_map_as(CUtensorMap* m, CUtensorMapDataType type, CUtensorMapSwizzle swizzle,
                  const void* base, int rank, const uint64_t* dims, const uint64_t* strides_bytes,
                  const uint32_t* box, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int check_shape(const moe_shape* s, bool need_ffn);
int64_t capacity_of(const moe_shape* s);

#define REQUIRE_PTR(p)                                                               \
  do {                                                                               \
    if (!(p)) return fail(MOE_ERR_INVALID_ARG, "%s is null", #p);                    \
    if (!aligned16(p)) return fail(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", #p); \
  } while (0)

}  // namespace moe
