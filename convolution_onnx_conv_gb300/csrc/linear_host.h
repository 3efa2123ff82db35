// Host-side checks shared by the entry points of the 8-bit operators (linear.cu, rows.cu).
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "api_internal.h"
#include "linear_internal.h"

namespace convf {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// whether `rows` rows `ld` elements apart pass the address space (their products then pass 64 bits)
inline bool too_far(long long rows, long long ld, int esz) { return ld > ((1LL << 48) / esz) / (rows > 1 ? rows : 1); }

// the largest power of two that divides v, up to 32: bytes on which rows begin
inline int common_alignment(uintptr_t v) { return static_cast<int>((v | 32) & (~(v | 32) + 1)); }

// SMs of the current device (looked up once per device), or an error
inline convf_status current_device(int* dev, int* num_sms) {
  static int sms[kMaxDevices];   // 0 = not looked up; every writer stores the same value
  if (cudaGetDevice(dev) != cudaSuccess) return record_error(CONVF_ERR_CUDA, "no current CUDA device");
  const bool known = *dev >= 0 && *dev < kMaxDevices;
  *num_sms = known ? sms[*dev] : 0;
  if (*num_sms == 0) {
    if (cudaDeviceGetAttribute(num_sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess || *num_sms < 1)
      return record_error(CONVF_ERR_CUDA, "the SM count of device %d could not be read", *dev);
    if (known) sms[*dev] = *num_sms;
  }
  return CONVF_OK;
}

}  // namespace convf
