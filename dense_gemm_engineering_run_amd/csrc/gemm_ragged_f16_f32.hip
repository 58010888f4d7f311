// Grouped-product kernels for dtype f16_f32 (inputs F16, output F32).
#include "gemm_ragged.hpp"

namespace mg {

hipError_t ragged_f16_f32(const RaggedCall& c, hipStream_t s) { return RaggedInst<In::F16, Out::F32>::launch(c, s); }

}  // namespace mg
