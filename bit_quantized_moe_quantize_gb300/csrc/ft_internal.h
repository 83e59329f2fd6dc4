// Host-side internals shared by the translation units of libft_moe.so.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace ft {

// Status plus a message recorded for ft_last_error().
int fail(int status, const char* fmt, ...);

// Multiprocessor count of the current device (cached per device).
int sm_count();

// Clears the message of ft_last_error() at the start of an entry point.
void clear_error();

// Device word that the FP8 operators raise FT_DEVERR_* flags in (one per
// device, fixed for the life of the process; ft_moe_read_device_error reads it).
// only_if_used: null where no call of this process has asked for it before.
int fp8_error_word(uint32_t** word, bool only_if_used = false);

// Sets the dynamic shared-memory limit of a kernel once per device and size.
int set_smem_limit(const void* kernel, int bytes);

// Profiling hooks (no-ops unless ft_profile_enable is active).
enum ProfPoint { kProfQuantBegin, kProfQuantEnd, kProfRouteBegin, kProfMatmulBegin, kProfMatmulEnd };
void prof_mark(ProfPoint p, cudaStream_t s);
void prof_count_launch();

// Checks cudaGetLastError() after a launch; on failure records the kernel
// name and geometry and returns FT_ERR_LAUNCH.
int check_launch(const char* kernel, dim3 grid, dim3 block, size_t smem);

// Test hook: a kernel whose bounded wait must give up after limit_ns.
int launch_wait_timeout_probe(uint32_t* err, int64_t limit_ns, cudaStream_t s);
// Measurement hook: a plain streaming read of n16 16-byte words of buf.
int launch_stream_read(const void* buf, int64_t n16, uint32_t* sink, cudaStream_t s);

// ------------------------------------------------------------ quantizer
int launch_quantize_q8_1(const void* x, void* act, int64_t tokens, int64_t ncols, cudaStream_t s);
int launch_act_mul_quantize_q8_1(const float* h, void* act, int64_t rows, int64_t n_inter, int kind, cudaStream_t s);
int launch_repack_q4_0_soa(const void* blocks, void* qs, void* d, int64_t n_blocks, cudaStream_t s);

// ---------------------------------------------------------------- router
constexpr int kRouteChunk = 256;          // slots per warp-chunk
constexpr int kRouteWarps = 8;            // warp-chunks per CTA

struct RouteBuffers {
    int32_t* counts;       // [E]
    int32_t* offsets;      // [E+1]
    int32_t* perm;         // [S]
    int32_t* hist;         // [nchunks][E] scratch
    int32_t* tiles_gemv;   // [E+1] or nullptr
    int32_t* tiles_gemm;   // [E+1] or nullptr
    uint32_t* err;
    // Expert-parallel shard: ids are global, the routed experts are
    // [expert_start, expert_start + n_experts) of n_global (0 = n_experts);
    // other valid ids are left out (zero rows, no error), ids outside
    // [0, n_global) raise FT_DEVERR_BAD_EXPERT_ID.
    int32_t expert_start;
    int32_t n_global;
};

inline int64_t route_chunks(int64_t n_slots) { return (n_slots + kRouteChunk - 1) / kRouteChunk; }

// Launches the three routing kernels.  When zero_rows != nullptr the rows of
// slots with a bad expert id are zeroed there (row_words 4-byte words each).
int launch_route(const int32_t* ids, int64_t n_slots, int32_t n_experts, const RouteBuffers& b,
                 int32_t gemv_group, int32_t gemm_group, uint32_t* zero_rows, int64_t row_words, cudaStream_t s);

// ------------------------------------------------------------------ GEMV
struct GemvPlan {
    int group;            // slots per tile (1, 2, 4 or 8)
    int row_warps;        // row-per-lane kernel: row groups of 32 per CTA (0: the block-per-lane kernel)
    int ksplit;           // row-per-lane kernel: warps that share a row group
    int64_t min_tiles;    // slot tiles the batch has at least (ceil(S / group))
    int rows;             // weight rows per stage (8 * rows per warp)
    int lanes_per_row;    // rows per warp per stage (1, 2 or 4)
    int stages;           // depth of the bulk-copy ring
    int64_t grid_x;       // slot-tile upper bound
    int64_t row_tiles;    // grid.y: CTAs per slot tile
    int64_t rows_per_cta;
    size_t smem;
    // Q4_0 tiles of `mma` groups of 8 slots on mma.sync (moe_gemv_mma.cu; 0:
    // the dp4a kernels); row_warps (warps of 16 rows there), stages and smem
    // then describe that kernel
    int mma;
};

// mean: routed slots per expert on average (decides the slots per tile);
// mma: Q4_0 tiles with more than 4 slots may run on the mma.sync kernel
GemvPlan plan_gemv(int64_t n_slots, int32_t n_experts, int64_t nrows, int64_t ncols, double mean,
                   int wtype = FT_TYPE_Q4_0, bool mma = true);
// bytes of one stored block of a FT_TYPE_* weight type (0: unknown type) and
// the weights it holds (32, or 256 for the K-quant super-blocks)
int weight_block_bytes(int wtype);
int weight_block_values(int wtype);
// Row-per-lane GEMV kernel: bytes of a row's 256 weights of a FT_TYPE_* type
// and their pitch in a shared-memory box (0: the type does not run there).
int row_box_bytes(int wtype);
int row_box_pitch(int wtype);

int launch_gemv(const GemvPlan& plan, const uint8_t* weights, const uint8_t* act, const int32_t* perm,
                const int32_t* offsets, const int32_t* tiles, float* out, int32_t* dots, uint32_t* err,
                int64_t n_slots, int32_t top_k, int32_t n_experts, int64_t nrows, int64_t ncols, cudaStream_t s,
                int wtype = FT_TYPE_Q4_0);

// The decode step in one launch (moe_decode.cu): the row-per-lane GEMV with
// the routing and the activation quantizer done per CTA, from fp16 x
// [tokens][ncols] and the ids; Q4_0 weights.  gemv_fused_ok: whether the plan
// and sizes allow it (and it pays off).
bool gemv_fused_ok(const GemvPlan& plan, int64_t n_slots, int32_t n_experts, int64_t ncols);
int launch_gemv_fused(const GemvPlan& plan, const uint8_t* weights, const uint16_t* x, const int32_t* ids,
                      float* out, uint32_t* err, int64_t n_slots, int32_t top_k, int32_t n_experts, int64_t nrows,
                      int64_t ncols, cudaStream_t s);

// ------------------------------------------------------------------ GEMM
constexpr int kGemmBN = 128;   // slots per tile
constexpr int kGemmBM = 128;   // weight rows per tile

// Slot-tile width (32 or 128) the tensor-core path uses for this batch; the
// router's GEMM tile prefix must be built with the same width.
int gemm_tile_width(double mean_slots_per_expert);

inline int64_t gemm_rows(int64_t n_slots) { return (n_slots + kGemmBN - 1) / kGemmBN * kGemmBN; }

// xh: [S_pad][ncols] fp16 and da: [S_pad][ncols/32] fp16 workspace for the
// routed activations in router order, S_pad = gemm_rows(S): written by
// launch_gather (zero past the routed slots), then read by the GEMM's TMA.
// sa != nullptr (Q4_K weights): also the exact d_a * sum(q_a) of every block, [S_pad][ncols/32] fp32.
int launch_gather(const uint8_t* act, const int32_t* perm, const int32_t* offsets, int32_t n_experts, int32_t top_k,
                  int64_t nb, int64_t n_slots, uint16_t* xh, uint16_t* da, cudaStream_t s, float* sa = nullptr);
// Layer 1 with the gated activation fused into the epilogue: the weights
// hold n_inter gate rows then n_inter up rows per expert (nrows = 2 n_inter),
// and instead of out the kernel writes act_mid [S][n_inter / 32] Q8_1 rows of
// act(gate) * up (kind: FT_ACT_*).
struct ActFuse {
    uint8_t* act_mid;
    int64_t n_inter;
    int32_t kind;
};

int launch_gemm(const uint8_t* weights, const uint8_t* act, const int32_t* perm, const int32_t* offsets,
                const int32_t* tiles, float* out, int32_t* dots, uint32_t* err, int64_t n_slots, int32_t top_k,
                int32_t n_experts, int64_t nrows, int64_t ncols, uint16_t* xh, uint16_t* da, int tile_width,
                cudaStream_t s, const ActFuse* af = nullptr, const float* sa = nullptr);


// ------------------------------------------------- FP8 expert-layer operators
struct GateParams {
    int64_t tokens;
    int32_t n_experts, top_k, score, n_groups, topk_groups, group_top, renormalize;
    float scale;
    const float* bias;
};
// stride: elements between the rows of logits (dtype FT_DTYPE_*)
int launch_gate(const GateParams& p, const void* logits, int dtype, int64_t stride, int32_t* ids, float* weights,
                cudaStream_t s);

// gated: x holds rows of 2 ncols values (gate, up), and act(gate) * up is quantized
int launch_quantize_fp8(const void* x, int dtype, uint8_t* codes, float* scales, int64_t rows, int64_t ncols,
                        bool gated, int kind, cudaStream_t s);

int launch_combine(const void* rows, int rows_dtype, const float* weights, const void* add, void* y, int y_dtype,
                   int64_t tokens, int32_t top_k, int64_t ncols, cudaStream_t s);

// The same into router order: row r of x goes to rows pos[r * k .. r * k + k - 1] (-1:
// none) of codes and scales (rows of scales `pitch` apart).  x fp16 or bf16, or gated fp32.
int launch_quantize_fp8_spread(const void* x, int dtype, uint8_t* codes, float* scales, int64_t rows, int64_t ncols,
                               bool gated, int kind, const int32_t* pos, int32_t k, int32_t pitch, cudaStream_t s);

// Router order (fp8_route.cu); fp8_route_ok: sizes that it takes.  pos may be null.
constexpr int64_t kFastRouteSlots = 256 * 1024;
bool fp8_route_ok(int64_t n_slots, int32_t n_experts);
size_t fp8_route_scratch(int64_t n_slots, int32_t n_experts);
int launch_fp8_route(const int32_t* ids, int64_t n_slots, int32_t n_experts, int32_t tile, int32_t* hist, int32_t* offsets,
                     int32_t* tiles, int32_t* perm, int32_t* pos, cudaStream_t s);
int launch_fp8_invert(const int32_t* perm, const int32_t* n_routed, int64_t n_slots, int32_t* pos, cudaStream_t s);

// Slots in router order, in the caller's workspace.
struct Fp8Order {
    int32_t *offsets, *tiles, *perm, *pos, *hist, *counts;
    uint32_t* err;        // the general router's own flags: ids of -1 are no error here
};
size_t fp8_order_layout(uint8_t* base, int64_t n_slots, int32_t n_experts, bool with_pos, Fp8Order* o);   // bytes
int launch_fp8_order(const int32_t* ids, int64_t n_slots, int32_t n_experts, int width, const Fp8Order& o, cudaStream_t s);

struct Fp8Product {
    const uint8_t* weights;     // [n_experts][nrows][ncols] e4m3
    const float* w_scales;      // [n_experts][ceil(nrows / 128)][ceil(ncols / 128)]
    const uint8_t* act;         // [act_rows][ncols] e4m3
    const float* act_scales;    // [act_rows], rows scale_pitch apart
    const int32_t* ids;         // [n_slots] expert of each slot, -1: none; nullptr: dense (one matrix)
    const Fp8Order* order;      // router order of ids (nullptr: dense)
    int64_t n_slots, act_rows, nrows, ncols;
    int32_t act_div;            // activation row of slot s: s / act_div (not `ordered`)
    int32_t n_experts, scale_pitch;
    bool ordered;               // act rows and scales lie in router order
    // gated (nrows = 2 n_inter, n_inter % 128 == 0): instead of out, the e4m3 codes
    // [routed][n_inter] and scales (rows mid_pitch apart) of act(gate) * up, in router order
    uint8_t* mid;
    float* mid_scales;
    int32_t mid_pitch, act_kind;
};
// Slots per tile for a batch (1: moe_fp8_gemv.cu; 16 or 32: moe_fp8_narrow.cu; 256:
// moe_fp8.cu); the order's tiles must be of that width.  fp8_orders_itself: the product needs no launch_fp8_order before it.
// Tiles of 256 take rows in router order only.
constexpr int kWideTile = 256;
// Slots per expert on average up to which a batch's slots are matrix-vector products of
// their own, go by tiles of 16 and of 32.  Measured (us, experts' matrices 768 x 2048 of 128,
// and 14336 x 4096 of 8): one slot each / 16 / 32 / 256 at
//   0.25: 8.1 / 15.5 / 17.2 / 26.4    25.5 / 28.1 / 29.9 / 40.5
//   0.5:  16.9 / 16.2 / 17.7 / 35.7   41.4 / 41.6 / 42.3 / 62.6
//   1:    32 / 27 / 28 / 48           78 / 60 / 61 / 92
//   8:    - / 38.4 / 39.0 / 61.9      - / 74.3 / 75.0 / 104.8
//   16:   - / 45.7 / 45.8 / 66.6      - / 90.9 / 77.4 / 103.5
//   32:   - / 60.0 / 53.7 / 70.2      (768 x 2048)
// and tiles of 32 / 256, one product (1536 x 2048 of 128, 1312 x 1040 of 60, 7168 x 4096 of 8) and
// the whole layer around it:
//   40: 101 / 131, 47 / 56, 67 / 79;    185 / 209, 85 / 96, 112 / 117
//   48: 107 / 134, 50 / 57, 69 / 78;    192 / 210, 87 / 97, 114 / 116
//   64: 122 / 134, 53 / 58, 77 / 78;    233 / 213, 97 / 97, 131 / 115
// One expert (a dense matrix) of 2048 x 7168, 4096 x 4096, 7168 x 2048, 14336 x 4096:
//   64:  28.4 / 32.1, 22.4 / 24.4, 18.0 / 18.7, 30.0 / 29.0
//   128: 28.9 / 33.0, 22.7 / 24.3, 19.0 / 19.2, 40.4 / 29.2
//   512: 33.0 / 34.4, 37.1 / 24.8, 32.4 / 20.0, 94.9 / 45.7
// and 16 experts of 768 x 2048, 4 of 1024 x 2048 (up to 1024 slots order themselves with the narrow tiles):
//   56: 21.5 / 29.0, 19.4 / 26.7    96: 33.1 / 32.1, 20.9 / 27.5    256: 42.4 / 34.8, 22.1 / 27.4    400: 55.1 / 44.6, 32.6 / 30.7
// so few experts of few rows would stay with 32 slots for longer; by slots per expert alone, 52 is between.
constexpr double kGemvMean = 0.5, kMean16 = 12, kMean32 = 52;
int fp8_tile_width(int64_t n_slots, int32_t n_experts);
bool fp8_orders_itself(int64_t n_slots, int32_t n_experts, int width);
int launch_fp8_product(const Fp8Product& p, int width, void* out, int out_dtype, uint32_t* err, cudaStream_t s);
int launch_fp8_gemv(const Fp8Product& p, void* out, int out_dtype, uint32_t* err, cudaStream_t s);
int launch_fp8_narrow(const Fp8Product& p, int width, void* out, int out_dtype, uint32_t* err, cudaStream_t s);
// Copies the rows of p to router order (codes, scales: room for n_slots rows) and makes p `ordered`.
int launch_fp8_order_rows(Fp8Product* p, uint8_t* codes, float* scales, cudaStream_t s);
// A layer of few tokens after its router (moe_fp8_token.cu); mid: room for n_slots * n_inter floats.
bool fp8_token_ok(int64_t n_slots, int64_t tokens, int32_t top_k, int64_t hidden, int64_t n_inter);
int launch_fp8_token_layer(const void* x, int x_dtype, const uint8_t* w13, const float* s13, const uint8_t* w2, const float* s2,
                           const int32_t* ids, const float* weights, float* mid, void* y, int64_t tokens, int32_t top_k,
                           int32_t n_experts, int64_t hidden, int64_t n_inter, int kind, cudaStream_t s);
// Pitch of rows of scales in router order.
inline int32_t fp8_scale_pitch(int64_t ncols) { return static_cast<int32_t>(((ncols + 127) / 128 + 3) / 4 * 4); }


// ------------------------------------------------- training the router
struct BalanceParams {
    int64_t tokens;
    int32_t n_experts, top_k, score, n_seqs;
};
constexpr int64_t kBalanceCtas = 1024;      // CTAs of the loss' first launch at most
size_t balance_workspace(int64_t tokens, int32_t n_experts, int32_t n_seqs);
int launch_balance(const BalanceParams& p, const void* logits, int dtype, int64_t stride, const int32_t* ids,
                   const int32_t* offsets, float* loss, int32_t* counts, float* seq_scale, uint8_t* ws, uint32_t* err,
                   cudaStream_t s);

struct GateGradParams {
    int64_t tokens;
    int32_t n_experts, top_k, score, renormalize, n_seqs;
    float scale;
    const int32_t* ids;
    const float* grad_weights;      // null: none arrives at the weights
    const int32_t* counts;          // null: none at the loss
    const float *seq_scale, *grad_loss;
    const int32_t* offsets;         // null: one sequence
};
int launch_gate_grad(const GateGradParams& p, const void* logits, int dtype, int64_t stride, void* out, uint32_t* err,
                     cudaStream_t s);

// grad_rows or grad_weights may be null
int launch_combine_grad(const void* dy, int dy_dtype, const void* rows, int rows_dtype, const float* weights, void* grad_rows,
                        float* grad_weights, int64_t tokens, int32_t top_k, int64_t ncols, cudaStream_t s);

// ------------------------------------------------- low-rank adapters
// Slots by adapter, and what the kernels of a call share.
struct LoraPlan {
    const int32_t *ids, *offsets, *tiles, *perm;
    const float* scales;                              // per adapter, or null: 1
    int32_t n_slots, n_adapters, rank;
    int width;               // slots of a tile: 128, 64 or 16
    int64_t n_tiles;         // tiles at most
    int32_t chunk;           // slots of a chunk of the matrices' gradients
    uint32_t* err;           // raised by launch_lora_down for ids that are no adapter
    bool overlap_grad;       // launch_lora_up directly before launch_lora_grad, which takes what came before that for done (lora_grad.cuh)
    int32_t down_jobs, down_cols;      // first products that a call of this kind can have, their longest rows
};
int32_t lora_part_kinds(int32_t rank);      // lines of 128 bytes of a slot's parts (lora.cuh)
// Numbers of chunks that lora_grad.cu gives out at most.
inline int64_t lora_chunks(int64_t n_slots, int32_t n_adapters, int32_t chunk) { return n_slots / chunk + n_adapters; }

// Slots by adapter: o's offsets, tiles and perm.
int launch_lora_order(const int32_t* ids, int64_t n_slots, int32_t n_adapters, int width, const Fp8Order& o, cudaStream_t s);

struct LoraDown {      // u[s] = W z[s / div]
    const void *z, *w;
    float* u;          // [slots][rank], or null
    void* parts;       // lines of the bf16 parts of scale u, whose sum it is (lora.cuh); or null
    int32_t cols, div;
    bool trans;        // W is [cols][rank], else [rank][cols]
};
int launch_lora_down(const LoraDown* jobs, int n_jobs, const LoraPlan& p, int dtype, cudaStream_t s);

struct LoraUp {        // out[s] = add[s] + scale W u[s]; launched to overlap launch_lora_down's tail
    const float* u;
    const void *w, *add;
    void* out;         // fp32 (out_f32) or the adapters' type
    float* present;    // [slots] 1 or 0, instead of passing rows without an adapter on; or null
    int32_t cols;
    bool trans, out_f32;      // trans: W is [rank][cols], else [cols][rank]
};
int launch_lora_up(const LoraUp& j, const LoraPlan& p, int dtype, cudaStream_t s);
int launch_lora_up_bf16(const LoraUp& j, const LoraPlan& p, cudaStream_t s);

struct LoraFew {       // the whole of ft_lora_add for up to kLoraFewSlots slots (plan: ids, scales, sizes)
    const void *x, *a, *b, *add;
    void* out;         // fp32 (out_f32) or the adapters' type
    int32_t ncols, nrows, div;
    bool out_f32;
};
// One launch against order, first and second product, from a graph: 128 slots of 64 adapters 18 against 26 us, 256 22
// against 26, 512 30 against 28: the search for a tile's slots among all ids and A read for each 16 of them cost what it saves.
constexpr int64_t kLoraFewSlots = 256;
int launch_lora_few(const LoraFew& f, const LoraPlan& p, int dtype, cudaStream_t s);
int launch_lora_few_bf16(const LoraFew& f, const LoraPlan& p, cudaStream_t s);

struct LoraGrad {      // out[e] = sum over its slots of scale w[s] z[s / div]; out null: not wanted
    const void* z;
    const float* w;       // fp16
    const void* w_parts;  // bf16: LoraDown's
    float *out, *parts;
    int32_t cols, div;
    bool turned;       // out is [cols][rank], else [rank][cols]
};
int launch_lora_grad(const LoraGrad* jobs, const LoraPlan& p, int dtype, cudaStream_t s);

}  // namespace ft
