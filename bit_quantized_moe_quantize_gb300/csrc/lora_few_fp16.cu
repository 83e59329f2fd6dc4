// lora_few.cuh for adapters in fp16, and the choice between the two types.
#include "lora_few.cuh"

namespace ft {

int launch_lora_few(const LoraFew& f, const LoraPlan& p, int dtype, cudaStream_t s) {
    return dtype == FT_DTYPE_F16 ? launch_few<__half>(f, p, s) : launch_lora_few_bf16(f, p, s);
}

}  // namespace ft
