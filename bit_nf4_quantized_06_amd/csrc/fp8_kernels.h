// Launchers of the kernels of the linear layer in 8-bit floating point (fp8.hip).
#pragma once

#include <hip/hip_runtime_api.h>

#include "fp8.h"

namespace qlora {

hipError_t launch_fp8_quantize(const Fp8QuantArgs& a, int x_type, hipStream_t stream);
hipError_t launch_fp8_quantize_weight(const Fp8QuantArgs& a, int w_type, hipStream_t stream);
hipError_t launch_fp8_product(const Fp8Args& a, const Fp8Plan& p, bool gated, bool f16,
                              hipStream_t stream);

}  // namespace qlora
