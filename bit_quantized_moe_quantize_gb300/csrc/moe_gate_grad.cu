// Gradient of the router: of its weights, and of the load-balance loss, to the logits in one pass.
//
//   s   scores of a row (softmax or sigmoid; 0 where masked), W = sum_j s[id_j], gw_j the weights' gradients
//   h_j scale gw_j; with renormalised weights scale / max(W, 1e-30) (gw_j - [W > 1e-30] sum_i gw_i s[id_i] / W)
//   a_e grad_loss seq_scale c_se, the loss' gradient to p_te
//   softmax:  d l_e = p_e (H_e + a_e - sum_j h_j s[id_j] - sum_i a_i p_i),  H_e = sum of h_j over id_j = e
//             (the sum of h_j s[id_j] is 0 where the weights are renormalised)
//   sigmoid:  d l_e = s_e (1 - s_e) H_e + p_e (1 - s_e) (a_e - sum_i a_i p_i),  p = s / max(sum, 1e-30)
//
// A row is read once, by the lanes that hold its experts, and written once.  The slots' parts lie in a row of
// shared memory that their lanes write to and the experts' lanes read.  Ids that repeat in a row, found by
// whose mark stays, are added in the order of the slots.  65536 rows of 128 bf16, top-8 of them, move 38 MB in
// 15.4 us (2.5 TB/s), 10 million instructions of a warp: with 24 warps of an SM neither the issue slots (47 %) nor memory are
// full, and waits for loads, for shared memory and for arithmetic weigh alike.  777 rows of 256 take 5.8 us, a chain of loads
// and sums.  Rows are read whole for the weights' gradient alone, too (from a graph 17.6 us, with the loss 19.6): softmax
// scores, and whether the weights' sum passes the smallest divisor, need them; sigmoid scores would not (21 us).
#include <type_traits>

#include "router_rows.cuh"
#include "ft_internal.h"
#include "launch.cuh"

namespace ft {

namespace {

// CTAs per SM, which take their rows in turn: three are resident (held to 80 registers: 65536 x 128 fp32 24 us from a graph,
// 26 with two), so that six end together (bf16: 19.6 us; with four, or a CTA for each set of rows, 21.7; a run of
// neighbouring rows for each, which would keep their sequence, 21.6).
constexpr int kGateGradCtas = 6;

struct GateGradArgs {
    const void* logits;
    const int32_t* ids;
    const float* grad_weights;   // null: no gradient arrives at the weights
    const int32_t* counts;       // null: none at the loss
    const float* seq_scale;
    const float* grad_loss;
    const int32_t* offsets;
    void* out;
    uint32_t* err;
    int64_t tokens, stride;
    int32_t n_experts, top_k, score, renormalize, n_seqs;
    float scale;
    bool wide, wide_out, wide_counts;
};

// ONE: no more slots than lanes that share them, so that each has one.
template <typename T, int L, int STEPS, bool ONE, bool SOFT>
__global__ void __launch_bounds__(kRowThreads, 3) gate_grad_kernel(const GateGradArgs a) {
    using G = RowGroup<L>;
    constexpr int WIDTH = 8 * L * STEPS, LANES = L < 32 ? L : 32;      // LANES: lanes that share the slots
    __shared__ __align__(16) float extra_all[G::kRows * WIDTH];
    __shared__ float part[kRowThreads / 32];
    const G g{part};
    const int32_t E = a.n_experts, k = a.top_k;
    float* extra = extra_all + G::row() * WIDTH;
    // the first LANES lanes of the group take a slot each (a whole CTA's other warps take none)
    const bool mine = L <= 32 || threadIdx.x < 32;
    const int32_t lane = static_cast<int32_t>(G::lane());
    struct Slot {
        int32_t e;        // expert, -1: takes no part
        float l, gw;      // its logit, the weight's gradient
    };
    // A run of rows after another: the next one's logits and slots are on their way while this one's are worked on.
    RowAhead<T, L, STEPS> ahead;
    int32_t ahead_e = -1;
    float ahead_gw = 0.0f;
    auto fetch = [&](int64_t first) {
        const int64_t t = first + G::row();
        ahead.fetch(static_cast<const T*>(a.logits) + (t < a.tokens ? t : a.tokens - 1) * a.stride, E, a.wide);
        if (ONE && a.grad_weights) {
            const bool in = mine && t < a.tokens && lane < k;
            ahead_e = in ? __ldg(a.ids + t * k + lane) : -1;
            ahead_gw = in ? __ldg(a.grad_weights + t * k + lane) : 0.0f;
        }
    };
    fetch(static_cast<int64_t>(blockIdx.x) * G::kRows);
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * G::kRows; first < a.tokens; first += static_cast<int64_t>(gridDim.x) * G::kRows) {
        const int64_t t0 = first + G::row();
        const bool there = t0 < a.tokens;
        const int64_t t = there ? t0 : a.tokens - 1;
        const T* row = static_cast<const T*>(a.logits) + t * a.stride;
        auto slot_at = [&](int32_t e, float gw) {
            Slot x{-1, 0.0f, 0.0f};
            if (e < -1 || e >= E) atomicOr(a.err, FT_DEVERR_BAD_EXPERT_ID);
            else if (e >= 0) {
                x.l = to_f32<T>(row[e]);
                if (x.l > -INFINITY) {      // not masked, which has no part in anything
                    x.e = e;
                    x.gw = gw;
                }
            }
            return x;
        };
        auto slot = [&](int32_t j) {
            if (!mine || !there || j >= k) return Slot{-1, 0.0f, 0.0f};
            return slot_at(__ldg(a.ids + t * k + j), __ldg(a.grad_weights + t * k + j));
        };
        Slot x{-1, 0.0f, 0.0f};
        if (ONE) x = slot_at(ahead_e, ahead_gw);
        float p[STEPS][8], rest[SOFT ? 1 : STEPS][8];              // rest: 1 - score
        ahead.take(row, E, a.wide, p);
        if (first + static_cast<int64_t>(gridDim.x) * G::kRows < a.tokens) fetch(first + static_cast<int64_t>(gridDim.x) * G::kRows);
        RowScale sc;
        if constexpr (SOFT) sc = row_softmax<L, STEPS>(g, p);
        else sc = row_sigmoid<L, STEPS>(g, p, rest);
        float dots = 0.0f;         // softmax: sum over slots of h_j s[id_j]

        if (a.grad_weights) {
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                float4* z = reinterpret_cast<float4*>(extra + first_expert<L>(i));
                z[0] = z[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            g.sync();
            auto score_of = [&](const Slot& x, float& s, float& r) {      // score and 1 - score (softmax: 1)
                s = r = 0.0f;
                if (x.e < 0) return;
                if (SOFT) {
                    s = soft_exp(x.l, sc.top) * sc.inv;      // +inf at the top: 1, others 0
                    r = 1.0f;
                } else {
                    sigmoid_pair(x.l, s, r);
                }
            };
            float W = 0.0f, m = 0.0f, s = 0.0f, r = 0.0f;
            if (ONE) score_of(x, s, r);
            if (a.renormalize) {
                if (ONE) {
                    W = s;
                    m = x.gw * s;
                } else {
                    for (int32_t j0 = 0; j0 < k; j0 += LANES) {
                        x = slot(j0 + lane);
                        score_of(x, s, r);
                        W += s;
                        m = fmaf(x.gw, s, m);
                    }
                }
                W = g.sum(W);
                m = g.sum(m);
            }
            const bool spread = a.renormalize && W > kScoreTiny;
            const float c = a.renormalize ? __fdividef(a.scale, fmaxf(W, kScoreTiny)) : a.scale;
            const float mean = spread ? __fdividef(m, W) : 0.0f;
            for (int32_t j0 = 0; j0 < k; j0 += LANES) {
                if (!ONE) {
                    x = slot(j0 + lane);
                    score_of(x, s, r);
                }
                // the score meets the divisor before the gradient: c alone may be 1e30, and 0 times what that makes of a
                // large gradient would be no number
                const float q = c * s * (x.gw - mean), d = r * q;
                if (x.e >= 0) dots += q;
                if (mine) {
                    // every lane marks its expert; where all marks stay, no id repeats
                    int32_t* mark = reinterpret_cast<int32_t*>(extra);
                    const float was = !ONE && x.e >= 0 ? extra[x.e] : 0.0f;
                    __syncwarp();
                    if (x.e >= 0) mark[x.e] = static_cast<int32_t>(lane_id());
                    __syncwarp();
                    const bool alone = x.e < 0 || mark[x.e] == static_cast<int32_t>(lane_id());
                    if (__all_sync(0xFFFFFFFFu, alone)) {
                        if (x.e >= 0) extra[x.e] = was + d;
                    } else {
                        __syncwarp();
                        if (x.e >= 0) extra[x.e] = was;
                        __syncwarp();
                        // lanes of this row with the same expert add in turn, lowest first
                        const uint32_t same = __match_any_sync(0xFFFFFFFFu, x.e < 0 ? -1 - static_cast<int32_t>(lane_id())
                                                                                     : x.e * G::kRows + static_cast<int32_t>(G::row()));
                        const int32_t turn = __popc(same & ((1u << lane_id()) - 1u));
                        const int32_t turns = static_cast<int32_t>(__reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(turn)));
                        for (int32_t i = 0; i <= turns; ++i) {
                            if (x.e >= 0 && turn == i) extra[x.e] += d;
                            __syncwarp();
                        }
                    }
                    __syncwarp();
                }
            }
            // by all lanes where it is one row's affair: rows of a warp may differ
            if (SOFT && __any_sync(0xFFFFFFFFu, !spread)) dots = g.sum(dots);
            if (!SOFT || spread) dots = 0.0f;
            g.sync();
        }

        float coef = 0.0f, mean = 0.0f;      // the loss' part
        const int32_t* count = nullptr;
        if (a.counts) {
            int32_t seq = 0;
            bool inside = true;
            if (a.offsets) {
                seq = seq_of(a.offsets, a.n_seqs, t);
                inside = seq_start(a.offsets, seq, a.tokens) <= t && t < seq_start(a.offsets, seq + 1, a.tokens);
            }
            // a row of padding has no part, whatever arrives
            coef = inside && sc.any ? __ldg(a.grad_loss) * __ldg(a.seq_scale + seq) : 0.0f;
            if constexpr (SOFT) coef *= sc.inv;
            count = a.counts + static_cast<int64_t>(seq) * E;
        }
        float c[STEPS][8] = {};
        if (count) {
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int32_t e0 = first_expert<L>(i);
                if (a.wide_counts && e0 + 8 <= E) {
                    const int4 x0 = __ldg(reinterpret_cast<const int4*>(count + e0)), x1 = __ldg(reinterpret_cast<const int4*>(count + e0) + 1);
                    c[i][0] = static_cast<float>(x0.x), c[i][1] = static_cast<float>(x0.y), c[i][2] = static_cast<float>(x0.z);
                    c[i][3] = static_cast<float>(x0.w), c[i][4] = static_cast<float>(x1.x), c[i][5] = static_cast<float>(x1.y);
                    c[i][6] = static_cast<float>(x1.z), c[i][7] = static_cast<float>(x1.w);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) c[i][j] = e0 + j < E ? static_cast<float>(__ldg(count + e0 + j)) : 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) mean = fmaf(c[i][j], p[i][j], mean);
            }
            mean = g.sum(mean);
            mean = SOFT ? mean * sc.inv : sc.sum > kScoreTiny ? __fdividef(mean, sc.sum) : 0.0f;
        }
        if (!there) continue;      // (the last run)
        // sigmoid: scores become p before they meet the loss' gradient, which 1e30 would put out of range
        const float inv = SOFT || !count ? 1.0f : __fdividef(1.0f, fmaxf(sc.sum, kScoreTiny));
        // with softmax, p holds exponentials: what multiplies them carries the reciprocal of their sum
        if (SOFT) dots *= sc.inv;
        T* out = static_cast<T*>(a.out) + t * E;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int32_t e0 = first_expert<L>(i);
            if (e0 >= E) break;
            __align__(16) T o[8];
            float x[8] = {};      // the slots' part
            if (a.grad_weights) {
                const float4 x0 = reinterpret_cast<const float4*>(extra + e0)[0], x1 = reinterpret_cast<const float4*>(extra + e0)[1];
                x[0] = x0.x, x[1] = x0.y, x[2] = x0.z, x[3] = x0.w;
                x[4] = x1.x, x[5] = x1.y, x[6] = x1.z, x[7] = x1.w;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float v, of = p[i][j];
                if constexpr (SOFT) {
                    v = fmaf(coef, c[i][j] - mean, -dots);
                } else {
                    v = coef * (c[i][j] - mean);
                    of *= inv * rest[i][j];
                }
                o[j] = from_f32<T>(fmaf(of, v, x[j]));
            }
            if (a.wide_out && e0 + 8 <= E) {
#pragma unroll
                for (int w = 0; w < static_cast<int>(sizeof(o) / 16); ++w)
                    reinterpret_cast<uint4*>(out + e0)[w] = reinterpret_cast<const uint4*>(o)[w];
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (e0 + j < E) out[e0 + j] = o[j];
            }
        }
    }
}

}  // namespace

int launch_gate_grad(const GateGradParams& p, const void* logits, int dtype, int64_t stride, void* out, uint32_t* err,
                     cudaStream_t s) {
    GateGradArgs a{};
    a.logits = logits;
    a.ids = p.ids;
    a.grad_weights = p.grad_weights;
    a.counts = p.counts;
    a.seq_scale = p.seq_scale;
    a.grad_loss = p.grad_loss;
    a.offsets = p.offsets;
    a.out = out;
    a.err = err;
    a.tokens = p.tokens;
    a.stride = stride;
    a.n_experts = p.n_experts;
    a.top_k = p.top_k;
    a.score = p.score;
    a.renormalize = p.renormalize;
    a.n_seqs = p.n_seqs;
    a.scale = p.scale;
    const int size = dtype == FT_DTYPE_F32 ? 4 : 2;
    a.wide = stride * size % 16 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0;
    a.wide_out = static_cast<int64_t>(p.n_experts) * size % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
    a.wide_counts = p.n_experts % 4 == 0 && reinterpret_cast<uintptr_t>(p.counts) % 16 == 0;
    auto launch = [&](auto lanes, auto steps) {
        constexpr int L = decltype(lanes)::value, N = decltype(steps)::value, ROWS = kRowThreads / L;
        const int64_t runs = (p.tokens + ROWS - 1) / ROWS, most = kGateGradCtas * static_cast<int64_t>(sm_count());
        const dim3 grid(static_cast<unsigned>(runs < most ? runs : most)), block(kRowThreads);
        auto go = [&](auto type) {
            using T = decltype(type);
            const bool one = p.top_k <= (L < 32 ? L : 32);
            if (p.score == FT_SCORE_SOFTMAX) {
                if (one) gate_grad_kernel<T, L, N, true, true><<<grid, block, 0, s>>>(a);
                else gate_grad_kernel<T, L, N, false, true><<<grid, block, 0, s>>>(a);
            } else {
                if (one) gate_grad_kernel<T, L, N, true, false><<<grid, block, 0, s>>>(a);
                else gate_grad_kernel<T, L, N, false, false><<<grid, block, 0, s>>>(a);
            }
        };
        if (dtype == FT_DTYPE_F32) go(float());
        else if (dtype == FT_DTYPE_F16) go(__half());
        else go(__nv_bfloat16());
        return check_launch("gate_grad_kernel", grid, block, 0);
    };
    // many rows: half the lanes, with twice the experts each, take fewer instructions (65536 x 128 from a graph: 19.6 us,
    // 23.7 with all); few rows: all of them are sooner done (777 x 256: 9.3 us against 11.4)
    return p.tokens >= 8192 ? with_row_lanes<true>(p.n_experts, launch) : with_row_lanes<false>(p.n_experts, launch);
}

}  // namespace ft
