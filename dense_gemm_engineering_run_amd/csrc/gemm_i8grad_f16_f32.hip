// Products with 8-bit values scaled along k, dtype f16_f32 (A F16, output F32).
#include "gemm_i8grad.hpp"

namespace mg {

hipError_t i8grad_f16_f32(const GradCall& c, hipStream_t s) { return GradInst<In::F16, Out::F32>::launch(c, s); }

}  // namespace mg
