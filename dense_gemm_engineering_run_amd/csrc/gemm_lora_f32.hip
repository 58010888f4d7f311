// Adapter kernels for dtype f32 (inputs F32, output F32).
#include "gemm_lora.hpp"

namespace mg {

hipError_t lora_f32(const LoraCall& c, hipStream_t s) { return LoraInst<In::F32, Out::F32>::launch(c, s); }

}  // namespace mg
