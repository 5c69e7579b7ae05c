// host.h -- host-side state of the library that its sources share (defined in attn_fwd.cu).
#pragma once

namespace attn {

// Bits of a stream's status word.
constexpr unsigned int STATUS_TIMEOUT = 1u, STATUS_PAGE = 2u;

// The current device and its SM count; ATTN_ERR_DEVICE unless it is an sm_103 GPU.
int host_device(int& sms, int& dev);

// Device address of the status word of `stream` (what attn_check reads and clears).
int host_status_word(int dev, void* stream, unsigned int** word);

}  // namespace attn
