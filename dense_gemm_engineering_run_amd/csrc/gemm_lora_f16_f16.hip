// Adapter kernels for dtype f16_f16 (inputs F16, output F16).
#include "gemm_lora.hpp"

namespace mg {

hipError_t lora_f16_f16(const LoraCall& c, hipStream_t s) { return LoraInst<In::F16, Out::F16>::launch(c, s); }

}  // namespace mg
