// lora_up.cuh for adapters in bf16.
#include "lora_up.cuh"

namespace ft {

int launch_lora_up_bf16(const LoraUp& j, const LoraPlan& p, cudaStream_t s) { return launch_up<__nv_bfloat16>(j, p, s); }

}  // namespace ft
