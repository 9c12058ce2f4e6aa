// internal.h -- host-side helpers shared by the C entry points (api.cu,
// mx_api.cu, noalloc.cu, selftest.cu): launch counting, validation of a
// quantized weight's descriptor, the device's properties and tensor maps.  Not
// part of the public ABI.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "codec.h"
#include "nf4_tables.h"
#include "qlora.h"

namespace qlora {

constexpr int64_t kMaxDim = int64_t(1) << 31;

struct DeviceInfo {
  bool ready = false;
  bool sm100 = false;
  int num_sms = 0;
  uint32_t* err = nullptr;     // the library's error flag on the device
};

// Properties of the current device; QLORA_ERR_UNSUPPORTED on a non-sm_100 device.
qlora_status device_info(DeviceInfo* out);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Tensor maps (after device_info): 2-D bf16 with 128-byte swizzle and box
// {64, box_outer}; 2-D uint8 with the given box and swizzle.
bool make_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t pitch_bytes,
              uint32_t box_outer);
bool make_map_u8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t pitch_bytes,
                 uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swz);
// Scale tiles (512 bytes each, `tiles` of them) as 32-bit words, box {128, box_outer}, no swizzle.
bool make_map_scales(CUtensorMap* m, const void* base, uint64_t tiles, uint32_t box_outer);

// Returns e; when it is cudaSuccess, adds n to the process-wide count of
// kernels the library has launched (qlora_kernel_launches).
cudaError_t counted(cudaError_t e, int n = 1);

// Checks a quantized-weight descriptor before any launch: NULL descriptor,
// shape range (0 <= rows, cols <= 2^31), block sizes, then (for a non-empty
// weight) NULL buffers and 16-byte alignment, in that order.
qlora_status check_tensor(const qlora_nf4_tensor* t);

// The encode kernel's bucket tables (kernel parameter) of one type's tables.
EncodeTables encode_tables(const Nf4Tables& tabs);

// Device address of the library's error flag on the current device (the flag
// qlora_read_device_errors reads); QLORA_ERR_UNSUPPORTED on a non-sm_100 device.
qlora_status device_error_flag(uint32_t** flag);

}  // namespace qlora
