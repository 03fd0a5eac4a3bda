// api_util.hpp -- host helpers shared by the translation units of the C ABI:
// element sizes, alignment checks and the per-device architecture check.
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/mcg.h"

namespace mcg {
namespace host {

// MCG_SUCCESS when the current device is gfx950 (api.cpp).
int check_arch();
// Compute units of the current device, 256 when none is visible (api.cpp).
int current_num_cu();

inline int elem_bytes(int dt) {
  switch (dt) {
    case MCG_BF16:
    case MCG_F16: return 2;
    case MCG_I8:
    case MCG_FP8_E4M3:
    case MCG_FP8_E5M2: return 1;
    case MCG_F32:
    case MCG_I32: return 4;
    case MCG_F64: return 8;
    default: return 0;
  }
}
inline bool aligned_to(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
inline bool valid_layout(int l) { return l == MCG_K_CONTIG || l == MCG_MN_CONTIG; }
inline bool float_out(int dt) { return dt == MCG_F32 || dt == MCG_BF16 || dt == MCG_F16; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? MCG_SUCCESS : MCG_ERR_HIP; }

}  // namespace host
}  // namespace mcg
