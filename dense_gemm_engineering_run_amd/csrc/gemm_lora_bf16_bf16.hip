// Adapter kernels for dtype bf16_bf16 (inputs BF16, output BF16).
#include "gemm_lora.hpp"

namespace mg {

hipError_t lora_bf16_bf16(const LoraCall& c, hipStream_t s) { return LoraInst<In::BF16, Out::BF16>::launch(c, s); }

}  // namespace mg
