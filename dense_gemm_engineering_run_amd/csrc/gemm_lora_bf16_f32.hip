// Adapter kernels for dtype bf16_f32 (inputs BF16, output F32).
#include "gemm_lora.hpp"

namespace mg {

hipError_t lora_bf16_f32(const LoraCall& c, hipStream_t s) { return LoraInst<In::BF16, Out::F32>::launch(c, s); }

}  // namespace mg
