// Grouped-product kernels for dtype f16_f16 (inputs F16, output F16).
#include "gemm_ragged.hpp"

namespace mg {

hipError_t ragged_f16_f16(const RaggedCall& c, hipStream_t s) { return RaggedInst<In::F16, Out::F16>::launch(c, s); }

}  // namespace mg
