// 8-bit integer products with output F32.
#include "gemm_i8.hpp"

namespace mg {

hipError_t i8_f32(const I8Call& c, hipStream_t s) { return I8Inst<Out::F32>::launch(c, s); }

}  // namespace mg
