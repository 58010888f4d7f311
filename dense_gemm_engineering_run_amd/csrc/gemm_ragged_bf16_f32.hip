// Grouped-product kernels for dtype bf16_f32 (inputs BF16, output F32).
#include "gemm_ragged.hpp"

namespace mg {

hipError_t ragged_bf16_f32(const RaggedCall& c, hipStream_t s) { return RaggedInst<In::BF16, Out::F32>::launch(c, s); }

}  // namespace mg
