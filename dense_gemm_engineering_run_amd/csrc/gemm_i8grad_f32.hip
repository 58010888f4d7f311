// Products with 8-bit values scaled along k, dtype f32 (A F32, output F32).
#include "gemm_i8grad.hpp"

namespace mg {

hipError_t i8grad_f32(const GradCall& c, hipStream_t s) { return GradInst<In::F32, Out::F32>::launch(c, s); }

}  // namespace mg
