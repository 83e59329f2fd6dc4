// Router of a mixture-of-experts layer: logits -> the top_k experts of each
// token and their weights.
//
//   s   = softmax(l) or sigmoid(l) over the E experts of a token; an expert
//         whose logit is -inf or NaN is masked: s = 0, and it is never chosen
//   key = l where there is no bias and one group (the order of l is the order
//         of s, without its rounding), else s + bias
//   groups of E / n_groups neighbouring experts: a group's score is the sum of
//         its group_top largest keys (of those not masked); only experts of
//         the topk_groups best groups can be chosen
//   ids = the top_k largest keys, equal keys by lowest index; -1 with weight 0
//         where no expert is left
//   w   = s[ids], renormalised by max(sum, 1e-30) if asked, times `scale`
//
// Up to 512 experts in one group, or in groups of 16, 32, 64, ..: 2, 8, 16 or 32 lanes per token,
// 16 neighbouring experts each, in registers (few_experts has when).  A key and the complement of its
// expert make one integer (32 bits where 16-bit logits are the keys, else 64), whose maximum over the
// lanes is the choice with its tie rule: a round is a few shuffles, and the lane that held the
// maximum looks again.  Up to eight choices come from sorting networks instead.  65536 tokens of 128 bf16
// logits, 8 choices: 16 us (21 MB: 3 us at the copy's rate); fp32 33 us, by rounds 48.  A warp's four tokens take 604
// instructions, mostly integer maxima and minima, whose pipe the warps wait for.
//
// Otherwise one warp per token (65535 tokens of 1024 experts: 191 us).  The keys lie in shared
// memory; each lane keeps the best key of its experts (every 32nd), and one round per chosen
// expert takes the warp's best of those with two integer warp reductions (largest key, then the
// lowest index that has it) and lets the lane that held it look again.
#include "fp8_common.cuh"
#include "ft_internal.h"

namespace ft {

constexpr int kGateWarps = 4;
constexpr float kGateTiny = 1e-30f;   // smallest sum that weights are divided by

struct GateArgs {
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* weights;
    int64_t tokens, stride;
    int32_t n_experts, top_k, score, n_groups, topk_groups, group_top, renormalize;
    float scale;
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// exp(l - top) with the limits top = +inf (those experts share the weight) and
// a masked l taken as 0.
__device__ __forceinline__ float gate_exp(float l, float top) {
    if (!(l > -INFINITY)) return 0.0f;
    return l == top ? 1.0f : expf(l - top);
}

__device__ __forceinline__ float gate_score(float l, float top, float sum, int32_t score) {
    if (!(l > -INFINITY)) return 0.0f;
    if (score == FT_SCORE_SIGMOID) return __fdiv_rn(1.0f, 1.0f + expf(-l));
    return __fdiv_rn(gate_exp(l, top), fmaxf(sum, kGateTiny));
}

// A lane's own largest key (an order integer, 0: none left) and its index.
struct Best {
    uint32_t key;
    int32_t at;
};

__device__ __forceinline__ Best lane_best(const uint32_t* keys, int32_t n) {
    Best b{0u, -1};
    for (int32_t e = static_cast<int32_t>(lane_id()); e < n; e += 32)
        if (keys[e] > b.key) b = Best{keys[e], e};
    return b;
}

// Removes the largest key of keys[0..n) and returns its index, -1 if none is left.  b: kept from call to call.
__device__ __forceinline__ int32_t take_best(uint32_t* keys, int32_t n, Best& b) {
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, b.key);
    if (top == 0u) return -1;
    const uint32_t at = __reduce_min_sync(0xFFFFFFFFu, b.key == top ? static_cast<uint32_t>(b.at) : 0xFFFFFFFFu);
    if (b.at == static_cast<int32_t>(at)) {
        keys[at] = 0u;
        b = lane_best(keys, n);
    }
    return static_cast<int32_t>(at);
}

template <typename T>
__global__ void __launch_bounds__(32 * kGateWarps) moe_gate_kernel(const GateArgs a) {
    extern __shared__ uint32_t gate_smem[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");      // a kernel launched to overlap may come up
    const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp;
    if (t >= a.tokens) return;
    const int32_t E = a.n_experts;
    uint32_t* keys = gate_smem + static_cast<size_t>(warp) * (E + a.n_groups);
    const T* row = static_cast<const T*>(a.logits) + t * a.stride;

    float top = -INFINITY, sum = 0.0f;
    if (a.score == FT_SCORE_SOFTMAX) {
        for (int32_t e = lane; e < E; e += 32) top = fmaxf(top, to_f32<T>(row[e]));   // fmaxf leaves NaN out
        top = warp_max(top);
        for (int32_t e = lane; e < E; e += 32) sum += gate_exp(to_f32<T>(row[e]), top);
        sum = warp_sum(sum);
    }
    const bool by_logit = a.bias == nullptr && a.n_groups == 1;
    for (int32_t e = lane; e < E; e += 32) {
        const float l = to_f32<T>(row[e]);
        float key = l;
        if (!by_logit) {
            key = gate_score(l, top, sum, a.score);
            if (a.bias) key += a.bias[e];
        }
        keys[e] = l > -INFINITY && key > -INFINITY ? float_order(key) : 0u;
    }
    __syncwarp();

    if (a.n_groups > 1) {
        const int32_t per = E / a.n_groups;
        uint32_t* score = keys + E;
        for (int32_t g = lane; g < a.n_groups; g += 32) {
            uint32_t k1 = 0u, k2 = 0u;      // the group's two largest keys
            for (int32_t i = 0; i < per; ++i) {
                const uint32_t k = keys[g * per + i];
                k2 = max(k2, min(k, k1));
                k1 = max(k1, k);
            }
            auto value = [](uint32_t k) {   // inverse of float_order
                return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
            };
            float v = k1 ? value(k1) : -INFINITY;
            if (a.group_top == 2 && k2) v += value(k2);
            score[g] = k1 ? float_order(v) : 0u;
        }
        __syncwarp();
        // each chosen group's score becomes the mark ~0
        Best b = lane_best(score, a.n_groups);
        for (int32_t i = 0; i < a.topk_groups; ++i) {
            const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, b.key);
            if (best == 0u) break;
            const uint32_t at =
                __reduce_min_sync(0xFFFFFFFFu, b.key == best ? static_cast<uint32_t>(b.at) : 0xFFFFFFFFu);
            if (b.at == static_cast<int32_t>(at)) {
                score[at] = 0xFFFFFFFFu;
                b = Best{0u, -1};
                for (int32_t g = lane; g < a.n_groups; g += 32)
                    if (score[g] != 0xFFFFFFFFu && score[g] > b.key) b = Best{score[g], g};
            }
        }
        __syncwarp();
        for (int32_t e = lane; e < E; e += 32)
            if (score[e / per] != 0xFFFFFFFFu) keys[e] = 0u;
        __syncwarp();
    }

    Best b = lane_best(keys, E);
    int32_t* ids = a.ids + t * a.top_k;
    float* weights = a.weights + t * a.top_k;
    float total = 0.0f, mine = 0.0f;      // mine: weight `lane` of the current 32
    for (int32_t j0 = 0; j0 < a.top_k; j0 += 32) {
        const int32_t n = min(32, a.top_k - j0);
        for (int32_t j = 0; j < n; ++j) {
            const int32_t at = take_best(keys, E, b);
            const float w = at < 0 ? 0.0f : gate_score(to_f32<T>(row[at]), top, sum, a.score);
            total += w;
            if (lane == static_cast<uint32_t>(j)) {
                mine = w;
                ids[j0 + j] = at;
            }
        }
        if (static_cast<int32_t>(lane) < n && (!a.renormalize || a.top_k > 32))
            weights[j0 + lane] = a.renormalize ? mine : mine * a.scale;
    }
    if (!a.renormalize) return;
    total = fmaxf(total, kGateTiny);
    if (a.top_k <= 32) {
        if (lane < static_cast<uint32_t>(a.top_k)) weights[lane] = __fdiv_rn(mine, total) * a.scale;
    } else {      // each lane rereads what it wrote
        for (int32_t j = lane; j < a.top_k; j += 32) weights[j] = __fdiv_rn(weights[j], total) * a.scale;
    }
}

// ------------------------------------------------------------ few experts
constexpr int kGateThreads = 128, kGatePer = 16;      // experts per lane

// 16-bit float bits -> order-preserving 16-bit integer, zeros of both signs alike.
__device__ __forceinline__ uint32_t order16(uint32_t b) {
    b = b == 0x8000u ? 0u : b;
    return (b & 0x8000u) ? (~b & 0xFFFFu) : (b | 0x8000u);
}

template <typename T>
__device__ __forceinline__ float order16_value(uint32_t o) {
    const uint16_t b = static_cast<uint16_t>((o & 0x8000u) ? (o ^ 0x8000u) : (~o & 0xFFFFu));
    return to_f32<T>(*reinterpret_cast<const T*>(&b));
}

__device__ __forceinline__ float order32_value(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}

template <typename K>
__device__ __forceinline__ void order_pair(K& a, K& b) {
    if constexpr (sizeof(K) == 4) {
        const uint32_t x = max(a, b), y = min(a, b);
        a = x;
        b = y;
    } else {
        const bool turn = a < b;
        const K x = turn ? b : a, y = turn ? a : b;
        a = x;
        b = y;
    }
}

// Sorts eight keys, largest first (odd-even merges: 19 exchanges).
template <typename K>
__device__ __forceinline__ void sort8(K (&k)[8]) {
    order_pair(k[0], k[1]);
    order_pair(k[2], k[3]);
    order_pair(k[4], k[5]);
    order_pair(k[6], k[7]);
    order_pair(k[0], k[2]);
    order_pair(k[1], k[3]);
    order_pair(k[4], k[6]);
    order_pair(k[5], k[7]);
    order_pair(k[1], k[2]);
    order_pair(k[5], k[6]);
    order_pair(k[0], k[4]);
    order_pair(k[1], k[5]);
    order_pair(k[2], k[6]);
    order_pair(k[3], k[7]);
    order_pair(k[2], k[4]);
    order_pair(k[3], k[5]);
    order_pair(k[1], k[2]);
    order_pair(k[3], k[4]);
    order_pair(k[5], k[6]);
}

// a := the eight largest of two sorted lists of eight, sorted.  Largest of a against smallest
// of b, and so on, leaves them as a bitonic list; three halvings sort that.
template <typename K>
__device__ __forceinline__ void merge8(K (&a)[8], const K (&b)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = a[i] > b[7 - i] ? a[i] : b[7 - i];
#pragma unroll
    for (int d = 4; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & d)) order_pair(a[i], a[i + d]);
}

// K: uint32_t (T is 16-bit and the keys are logits) or uint64_t.  WIDE: rows start at whole
// 16-byte words.
template <typename T, int LANES, typename K, bool WIDE>
__global__ void __launch_bounds__(kGateThreads) moe_gate_few_kernel(const GateArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");      // a kernel launched to overlap may come up
    constexpr bool PACKED = sizeof(K) == 4;
    const uint32_t sub = threadIdx.x & (LANES - 1);
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * (kGateThreads / LANES) + threadIdx.x / LANES;
    const bool there = t0 < a.tokens;
    const int64_t t = there ? t0 : a.tokens - 1;
    const int32_t E = a.n_experts, e0 = static_cast<int32_t>(sub) * kGatePer;
    const T* row = static_cast<const T*>(a.logits) + t * a.stride;
    const bool by_logit = PACKED || (a.bias == nullptr && a.n_groups == 1);
    T raw[kGatePer];
    if (WIDE && e0 + kGatePer <= E) {
        constexpr int WORDS = kGatePer * static_cast<int>(sizeof(T)) / 16;
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
            reinterpret_cast<uint4*>(raw)[i] = __ldg(reinterpret_cast<const uint4*>(row + e0) + i);
    } else {
#pragma unroll
        for (int i = 0; i < kGatePer; ++i) raw[i] = e0 + i < E ? row[e0 + i] : from_f32<T>(-INFINITY);
    }
    float top = -INFINITY, sum = 0.0f;
    if (a.score == FT_SCORE_SOFTMAX) {
#pragma unroll
        for (int i = 0; i < kGatePer; ++i) top = fmaxf(top, to_f32<T>(raw[i]));
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        // renormalised weights of the largest logits need no sum over all: it cancels
        if (!(by_logit && a.renormalize)) {
#pragma unroll
            for (int i = 0; i < kGatePer; ++i) sum += gate_exp(to_f32<T>(raw[i]), top);
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        }
    }
    K key[kGatePer], best = 0;
#pragma unroll
    for (int i = 0; i < kGatePer; ++i) {
        const float l = to_f32<T>(raw[i]);
        bool ok = l > -INFINITY;
        if constexpr (PACKED) {
            key[i] = (order16(*reinterpret_cast<const uint16_t*>(&raw[i])) << 16) | (0xFFFFu - static_cast<uint32_t>(e0 + i));
        } else {
            float x = l;
            if (!by_logit) {
                if (e0 + i < E) x = gate_score(l, top, sum, a.score) + (a.bias ? __ldg(a.bias + e0 + i) : 0.0f);
                else x = -INFINITY;
                ok = ok && x > -INFINITY;
            }
            key[i] = (static_cast<uint64_t>(float_order(x)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(e0 + i));
        }
        if (!ok) key[i] = 0;
        best = key[i] > best ? key[i] : best;
    }
    if constexpr (!PACKED) {
        if (a.n_groups > 1) {      // a group's experts are those of 1, 2, 4, .. whole lanes
            const int32_t per = E / a.n_groups / kGatePer, mine = static_cast<int32_t>(sub) / per;
            uint32_t k1 = 0u, k2 = 0u;      // the group's two largest keys
#pragma unroll
            for (int i = 0; i < kGatePer; ++i) {
                const uint32_t k = static_cast<uint32_t>(key[i] >> 32);
                k2 = max(k2, min(k, k1));
                k1 = max(k1, k);
            }
            for (int o = 1; o < per; o <<= 1) {
                const uint32_t o1 = __shfl_xor_sync(0xFFFFFFFFu, k1, o), o2 = __shfl_xor_sync(0xFFFFFFFFu, k2, o);
                k2 = max(max(k2, o2), min(k1, o1));
                k1 = max(k1, o1);
            }
            float v = order32_value(k1);
            if (a.group_top == 2 && k2) v += order32_value(k2);
            const uint32_t score = k1 ? float_order(v) : 0u;
            int32_t better = 0;
            for (int32_t g = 0; g < a.n_groups; ++g) {
                const uint32_t other = __shfl_sync(0xFFFFFFFFu, score, g * per, LANES);
                better += other > score || (other == score && g < mine) ? 1 : 0;
            }
            if (better >= a.topk_groups) {
                best = 0;
#pragma unroll
                for (int i = 0; i < kGatePer; ++i) key[i] = 0;
            }
        }
    }
    int32_t* ids = a.ids + t * a.top_k;
    float* weights = a.weights + t * a.top_k;
    // softmax weights of the largest logits, renormalised, need no sum over all
    const bool cancel = by_logit && a.renormalize && a.score == FT_SCORE_SOFTMAX;
    auto chosen = [&](K m, int32_t& at) {      // a choice's expert and logit
        if constexpr (PACKED) {
            at = static_cast<int32_t>(0xFFFFu - (m & 0xFFFFu));
            return order16_value<T>(static_cast<uint32_t>(m) >> 16);
        } else {
            at = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(m));
            return by_logit ? order32_value(static_cast<uint32_t>(m >> 32)) : to_f32<T>(row[at]);
        }
    };
    if constexpr (LANES >= 8) {
        // up to eight choices: every lane's eight largest by sorting networks, then the lanes' lists
        // merged pairwise; the rounds below take three times the instructions
        if (a.top_k <= 8) {
            K k8[8], l8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                k8[i] = key[i];
                l8[i] = key[8 + i];
            }
            sort8(k8);
            sort8(l8);
            merge8(k8, l8);
#pragma unroll
            for (int o = 1; o < LANES; o <<= 1) {
#pragma unroll
                for (int i = 0; i < 8; ++i) l8[i] = __shfl_xor_sync(0xFFFFFFFFu, k8[i], o);
                merge8(k8, l8);
            }
            K m = k8[0];      // lane j takes choice j
#pragma unroll
            for (int i = 1; i < 8; ++i) m = sub == static_cast<uint32_t>(i) ? k8[i] : m;
            const bool mine = sub < static_cast<uint32_t>(a.top_k);
            int32_t at = -1;
            float w = 0.0f;
            if (mine && m != 0) {
                const float l = chosen(m, at);
                w = cancel ? gate_exp(l, top) : gate_score(l, top, sum, a.score);
            }
            float total = w;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
            if (there && mine) {
                ids[sub] = at;
                weights[sub] = (a.renormalize ? __fdiv_rn(w, fmaxf(total, kGateTiny)) : w) * a.scale;
            }
            return;
        }
    }
    float total = 0.0f, mine = 0.0f;      // mine: weight `sub` (of the first LANES)
    const bool few = a.top_k <= LANES;
    for (int32_t j = 0; j < a.top_k; ++j) {
        K m = best;
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) {
            const K other = __shfl_xor_sync(0xFFFFFFFFu, m, o);
            m = other > m ? other : m;
        }
        if (m != 0 && best == m) {
            best = 0;
#pragma unroll
            for (int i = 0; i < kGatePer; ++i) {
                key[i] = key[i] == m ? 0 : key[i];
                best = key[i] > best ? key[i] : best;
            }
        }
        int32_t at = -1;
        float w = 0.0f;
        if (m != 0) {
            const float l = chosen(m, at);
            w = cancel ? gate_exp(l, top) : gate_score(l, top, sum, a.score);
        }
        total += w;
        if (there && sub == static_cast<uint32_t>(j & (LANES - 1))) {
            mine = w;
            ids[j] = at;
            if (!few) weights[j] = a.renormalize ? w : w * a.scale;
        }
    }
    if (!there) return;
    total = fmaxf(total, kGateTiny);
    if (few) {
        if (sub < static_cast<uint32_t>(a.top_k)) weights[sub] = (a.renormalize ? __fdiv_rn(mine, total) : mine) * a.scale;
    } else if (a.renormalize) {
        for (int32_t j = static_cast<int32_t>(sub); j < a.top_k; j += LANES)      // each lane rereads what it wrote
            weights[j] = __fdiv_rn(weights[j], total) * a.scale;
    }
}

template <typename T, int LANES, typename K>
static int launch_few(const GateArgs& a, cudaStream_t s) {
    const int64_t per = kGateThreads / LANES, ctas = (a.tokens + per - 1) / per;
    if (ctas > 0x7FFFFFFF) return fail(FT_ERR_SIZE, "too many tokens for one launch");
    const dim3 grid(static_cast<unsigned>(ctas)), block(kGateThreads);
    const bool wide = a.stride * static_cast<int64_t>(sizeof(T)) % 16 == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
    if (wide) moe_gate_few_kernel<T, LANES, K, true><<<grid, block, 0, s>>>(a);
    else moe_gate_few_kernel<T, LANES, K, false><<<grid, block, 0, s>>>(a);
    return check_launch("moe_gate_few_kernel", grid, block, 0);
}

template <typename T>
static int launch_few_typed(const GateArgs& a, cudaStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (a.bias == nullptr && a.n_groups == 1) {
            if (a.n_experts <= 2 * kGatePer) return launch_few<T, 2, uint32_t>(a, s);
            if (a.n_experts <= 8 * kGatePer) return launch_few<T, 8, uint32_t>(a, s);
            if (a.n_experts <= 16 * kGatePer) return launch_few<T, 16, uint32_t>(a, s);
            return launch_few<T, 32, uint32_t>(a, s);
        }
    }
    if (a.n_experts <= 2 * kGatePer) return launch_few<T, 2, uint64_t>(a, s);
    if (a.n_experts <= 8 * kGatePer) return launch_few<T, 8, uint64_t>(a, s);
    if (a.n_experts <= 16 * kGatePer) return launch_few<T, 16, uint64_t>(a, s);
    return launch_few<T, 32, uint64_t>(a, s);
}

// Whether a batch goes to moe_gate_few_kernel.  It takes up to 512 experts, and groups that are 1, 2,
// 4, .. whole lanes; where it takes a batch, both kernels' times decide (us with cold caches, registers /
// shared memory):
//   16-bit logits as keys: 65535 tokens of 512, 8 choices 63 / 126, 32 choices 281 / 331
//   64-bit keys, 65535 tokens by 2, 8, 16 choices
//     128 experts       fp32 logits 39/46, 39/82, 87/132     sigmoid with a bias 51/47, 51/81, 97/131
//     256               75/54, 75/93, 169/147                97/64, 97/100, 185/150
//     512               151/74, 151/125, 331/192             198/101, 199/145, 364/206
//     256 in 8 groups   -                                    106/112, 106/146, 196/194, and 339/299 by 32
//     512 in 8 groups   -                                    216/189, 216/227, 389/285
//   8192 tokens of 512  29/20, 29/27, 53/36                  34/29, 33/35, 58/43
//   777 tokens of 512   12/11, 12/14, 19/17                  15/18, 16/19, 21/23
// so 64-bit keys of many tokens stay in registers up to 128 experts, up to 256 where the sorting
// networks' time, the same for one choice as for eight, is made use of, and in groups while there are
// networks for them.
static bool few_experts(const GateParams& p, int dtype) {
    const int32_t lanes = p.n_experts / p.n_groups / kGatePer;
    const bool whole = p.n_groups == 1 || (lanes > 0 && p.n_experts == lanes * kGatePer * p.n_groups && (lanes & (lanes - 1)) == 0);
    if (!whole || p.n_experts > 32 * kGatePer) return false;
    const bool packed = dtype != FT_DTYPE_F32 && p.bias == nullptr && p.n_groups == 1;
    if (packed || p.tokens < 8192 || p.n_experts <= 8 * kGatePer) return true;
    if (p.n_groups > 1) return p.top_k <= 8 || p.n_experts <= 16 * kGatePer;
    return p.n_experts <= 16 * kGatePer && p.top_k > 5 && p.top_k <= 8;
}

int launch_gate(const GateParams& p, const void* logits, int dtype, int64_t stride, int32_t* ids, float* weights,
                cudaStream_t s) {
    if (p.tokens == 0) return FT_OK;
    GateArgs a{};
    a.logits = logits;
    a.bias = p.bias;
    a.ids = ids;
    a.weights = weights;
    a.tokens = p.tokens;
    a.stride = stride;
    a.n_experts = p.n_experts;
    a.top_k = p.top_k;
    a.score = p.score;
    a.n_groups = p.n_groups;
    a.topk_groups = p.topk_groups;
    a.group_top = p.group_top;
    a.renormalize = p.renormalize;
    a.scale = p.scale;
    if (few_experts(p, dtype))
        return dtype == FT_DTYPE_F32   ? launch_few_typed<float>(a, s)
               : dtype == FT_DTYPE_F16 ? launch_few_typed<__half>(a, s)
                                       : launch_few_typed<__nv_bfloat16>(a, s);
    const int64_t ctas = (p.tokens + kGateWarps - 1) / kGateWarps;
    if (ctas > 0x7FFFFFFF) return fail(FT_ERR_SIZE, "too many tokens for one launch");
    const dim3 grid(static_cast<unsigned>(ctas)), block(32 * kGateWarps);
    const size_t sm = static_cast<size_t>(kGateWarps) * (p.n_experts + p.n_groups) * sizeof(uint32_t);
    const void* k = dtype == FT_DTYPE_F32   ? reinterpret_cast<const void*>(moe_gate_kernel<float>)
                    : dtype == FT_DTYPE_F16 ? reinterpret_cast<const void*>(moe_gate_kernel<__half>)
                                            : reinterpret_cast<const void*>(moe_gate_kernel<__nv_bfloat16>);
    if (sm > 48 * 1024)
        if (int st = set_smem_limit(k, static_cast<int>(sm))) return st;
    if (dtype == FT_DTYPE_F32) moe_gate_kernel<float><<<grid, block, sm, s>>>(a);
    else if (dtype == FT_DTYPE_F16) moe_gate_kernel<__half><<<grid, block, sm, s>>>(a);
    else moe_gate_kernel<__nv_bfloat16><<<grid, block, sm, s>>>(a);
    return check_launch("moe_gate_kernel", grid, block, sm);
}

}  // namespace ft
