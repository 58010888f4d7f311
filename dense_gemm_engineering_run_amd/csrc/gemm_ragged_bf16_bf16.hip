// Grouped-product kernels for dtype bf16_bf16 (inputs BF16, output BF16).
#include "gemm_ragged.hpp"

namespace mg {

hipError_t ragged_bf16_bf16(const RaggedCall& c, hipStream_t s) { return RaggedInst<In::BF16, Out::BF16>::launch(c, s); }

}  // namespace mg
