// Products with 8-bit values scaled along k, dtype f16_f16 (A F16, output F16).
#include "gemm_i8grad.hpp"

namespace mg {

hipError_t i8grad_f16_f16(const GradCall& c, hipStream_t s) { return GradInst<In::F16, Out::F16>::launch(c, s); }

}  // namespace mg
