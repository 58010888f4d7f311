// Grouped-product kernels for dtype f32 (inputs F32, output F32).
#include "gemm_ragged.hpp"

namespace mg {

hipError_t ragged_f32(const RaggedCall& c, hipStream_t s) { return RaggedInst<In::F32, Out::F32>::launch(c, s); }

}  // namespace mg
