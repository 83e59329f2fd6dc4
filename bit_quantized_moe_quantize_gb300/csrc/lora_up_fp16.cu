// lora_up.cuh for adapters in fp16, and the choice between the two types.
#include "lora_up.cuh"

namespace ft {

int launch_lora_up(const LoraUp& j, const LoraPlan& p, int dtype, cudaStream_t s) {
    return dtype == FT_DTYPE_F16 ? launch_up<__half>(j, p, s) : launch_lora_up_bf16(j, p, s);
}

}  // namespace ft
