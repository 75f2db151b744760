// api.h -- what the translation units of the C ABI share (api.cu, api_paged.cu): error
// text, the current device and its error word, pointer checks and the driver's tensor-map
// encoder.  Not part of the public ABI.
#pragma once
#include <cstddef>
#include <cstdint>
#include <initializer_list>
#include <cuda.h>
#include <cuda_runtime.h>

#include "neattn.h"

namespace ne {
namespace api {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Records the calling thread's error text and returns `s`.
ne_status fail(ne_status s, const char* fmt, ...);
ne_status cuda_fail(cudaError_t e, const char* what);
void clear_error();

// The current device, which must be an sm_103 one.
ne_status current_device(int* dev);
// Device error word of device `dev`, the current one (allocated once).
ne_status error_word(int dev, int** out);
// Whether that word exists already.
bool have_error_word(int dev);
// Wall-clock limit of the kernels' bounded waits.
unsigned long long timeout_ns();
// cuTensorMapEncodeTiled, from the driver.
ne_status encode_fn(EncodeTiledFn* out);

bool aligned16(const void* p);
// Every pointer non-null and 16-byte aligned.
ne_status check_ptrs(std::initializer_list<const void*> ps);

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

}  // namespace api
}  // namespace ne
