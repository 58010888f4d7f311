// Products with 8-bit values scaled along k, dtype bf16_bf16 (A BF16, output BF16).
#include "gemm_i8grad.hpp"

namespace mg {

hipError_t i8grad_bf16_bf16(const GradCall& c, hipStream_t s) { return GradInst<In::BF16, Out::BF16>::launch(c, s); }

}  // namespace mg
