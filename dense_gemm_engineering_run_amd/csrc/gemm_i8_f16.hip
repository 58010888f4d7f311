// 8-bit integer products with output F16.
#include "gemm_i8.hpp"

namespace mg {

hipError_t i8_f16(const I8Call& c, hipStream_t s) { return I8Inst<Out::F16>::launch(c, s); }

}  // namespace mg
