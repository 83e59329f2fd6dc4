// What the two kernels of the adapters' gradients share: their arguments, and the chunks of slots.  They may come up under the
// tail of the second product (lora_up.cuh), whose results they do not read, and end behind it.  What they do read, the order
// and the first products, is made by the grids before that one, and they read it without a wait of their own: that is sound
// because they start only once every CTA of the second product has let them or has ended, and its first CTA, as every one with a
// tile, waits for all that came before.  A change there that takes this wait out needs one here.
#pragma once

#include "gemm_common.cuh"
#include "lora.cuh"
#include "ft_internal.h"
#include "launch.cuh"

namespace ft {

constexpr int kGradThreads = 256;

template <typename T>
struct GradJob {
    const T* z;
    const float* w;         // [slots][R] (fp16)
    const uint8_t* w_parts; // lines of the scaled sums' parts (bf16, lora.cuh)
    float *out, *parts;     // [adapters][size], [chunks][size]
    int32_t cols, div;      // of z; row of slot s: s / div
    bool turned;            // out is [cols][R], else [R][cols]
};

template <typename T>
struct GradArgs {
    GradJob<T> job[2];
    LoraSlots slots;
    const float* scales;
    uint32_t* err;
    int32_t rank, per, blocks0;      // per: slots of a chunk; blocks0: blocks of columns of the first job
};

// Chunk number b: its adapter, whether it has others, its first slot in order and its slots (0: none).
struct Chunk {
    int32_t adapter, first, n;
    bool alone;
};

template <int THREADS>
__device__ __forceinline__ Chunk find_chunk(const LoraSlots& s, int32_t b, int32_t per) {
    __shared__ Chunk found;
    const int32_t tid = static_cast<int32_t>(threadIdx.x);
    if (tid == 0) found = Chunk{0, 0, 0, true};
    __syncthreads();
    for (int32_t e = tid; e < s.n_adapters; e += THREADS) {
        const int32_t o0 = __ldg(s.offsets + e), o1 = __ldg(s.offsets + e + 1), j = b - (o0 / per + e);
        // j * per stays small where it is looked at: numbers rise with the slots
        if (j >= 0 && j <= (o1 - o0) / per && j * per < o1 - o0) found = Chunk{e, o0 + j * per, min(per, o1 - o0 - j * per), o1 - o0 <= per};
    }
    __syncthreads();
    return found;
}

template <typename T>
GradArgs<T> grad_args(const LoraGrad* jobs, const LoraPlan& p, int32_t columns, int64_t* blocks) {
    GradArgs<T> a{};
    int n = 0;
    *blocks = 0;
    for (int i = 0; i < 2; ++i) {
        if (!jobs[i].out) continue;
        a.job[n++] = GradJob<T>{static_cast<const T*>(jobs[i].z), jobs[i].w, static_cast<const uint8_t*>(jobs[i].w_parts), jobs[i].out, jobs[i].parts, jobs[i].cols, jobs[i].div,
                                jobs[i].turned};
        if (n == 1) a.blocks0 = (jobs[i].cols + columns - 1) / columns;
        *blocks += (jobs[i].cols + columns - 1) / columns;
    }
    a.slots = LoraSlots{p.ids, p.offsets, p.tiles, p.perm, p.n_slots, p.n_adapters, p.width};
    a.scales = p.scales;
    a.err = p.err;
    a.rank = p.rank;
    a.per = p.chunk;
    return a;
}

// The kernel for bf16 adapters (lora_grad_tc.cu).
int launch_lora_grad_tc(const LoraGrad* jobs, const LoraPlan& p, cudaStream_t s);

}  // namespace ft
