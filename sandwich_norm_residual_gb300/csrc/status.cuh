// The device's status word, read by beam_sync_status. One translation unit holds
// it; the others get its address.
#pragma once

namespace beam {

__device__ unsigned int g_status_word;  // bit 0: a bounded wait gave up; bit 1: a bad value on the device
__device__ __forceinline__ void report_timeout() { atomicOr(&g_status_word, 1u); }

}  // namespace beam
