// Adapter kernels for dtype f16_f32 (inputs F16, output F32).
#include "gemm_lora.hpp"

namespace mg {

hipError_t lora_f16_f32(const LoraCall& c, hipStream_t s) { return LoraInst<In::F16, Out::F32>::launch(c, s); }

}  // namespace mg
