// host.h -- host-side state of the library that its sources share (defined in attn_fwd.cu).
#pragma once
#include <cuda.h>

#include <cstddef>
#include <cstdint>
#include <mutex>

#include "attn.h"

namespace attn {

// Bits of a stream's status word.
constexpr unsigned int STATUS_TIMEOUT = 1u, STATUS_PAGE = 2u;

// The current device and its SM count; ATTN_ERR_DEVICE unless it is an sm_103 GPU.
int host_device(int& sms, int& dev);

// The longest a kernel may wait on one barrier, in microseconds.
uint32_t host_timeout_us();

// The armed state of attn_debug_inject, which one launch takes.
int host_take_inject();

// 5-D tensor map of fp16 / bf16 with 128-byte swizzle, from the library's cache: extents and box in
// elements, strides of dimensions 1-4 in bytes.  What lies outside reads as zeros.
struct Map5 {
  long long dims[5], strides[4];
  int box[5], pad;  // (pad: so that maps compare byte by byte)
};
int host_map5(CUtensorMap* m, const void* ptr, bool bf16, const Map5& t);

// Device address of the status word of `stream` (what attn_check reads and clears).
int host_status_word(int dev, void* stream, unsigned int** word);

// The workspace that the library keeps for `stream`, grown to `bytes` where needed (stream-ordered).  `hold`
// keeps other calls on the stream from it until the caller has enqueued what uses it.
int host_workspace(int dev, void* stream, size_t bytes, std::unique_lock<std::mutex>& hold, void** ws);

// A C entry's body: what it throws (host memory that has run out, a mutex that fails) becomes a status.
template <class F>
int entry(F body) noexcept {
  try {
    return body();
  } catch (...) {
    return ATTN_ERR_CUDA;
  }
}

}  // namespace attn
