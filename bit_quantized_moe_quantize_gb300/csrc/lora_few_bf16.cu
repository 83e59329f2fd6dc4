// lora_few.cuh for adapters in bf16.
#include "lora_few.cuh"

namespace ft {

int launch_lora_few_bf16(const LoraFew& f, const LoraPlan& p, cudaStream_t s) { return launch_few<__nv_bfloat16>(f, p, s); }

}  // namespace ft
