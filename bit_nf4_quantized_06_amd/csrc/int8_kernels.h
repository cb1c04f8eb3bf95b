// Launchers of the 8-bit linear layer's kernels (int8.hip).
#pragma once

#include <hip/hip_runtime_api.h>

#include "int8.h"

namespace qlora {

hipError_t launch_int8_quantize(const Int8QuantArgs& a, int x_type, hipStream_t stream);
// X16: the 16-bit tokens of a kInt8Fused plan (otherwise not read).
hipError_t launch_int8_product(const Int8Args& a, const uint16_t* X16, const Int8Plan& p, bool f16,
                               hipStream_t stream);

}  // namespace qlora
