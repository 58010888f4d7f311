// 8-bit integer products with output BF16.
#include "gemm_i8.hpp"

namespace mg {

hipError_t i8_bf16(const I8Call& c, hipStream_t s) { return I8Inst<Out::BF16>::launch(c, s); }

}  // namespace mg
