// Gradients of bf16 adapters' matrices (lora_grad.cu has the formulas) on the tensor cores by tcgen05.
//
// D[m][c] = sum over slots of W[m][s] z[s][c]: a CTA takes a chunk of an adapter's slots and 256 columns of z.  The rows m are
// the narrow side's ranks, each three times: an fp32 value is the sum of three bf16 parts (24 bits), whose products with
// z's bf16 are exact.  Up to rank 40 all three parts fit the 128 rows of one MMA; up to 64 two, and the third
// is a second MMA onto the first part's rows; above, each part is an MMA of its own.
//
// Both operands lie as they come, a slot's neighbours side by side (M- and N-major), in lines of 128 bytes whose 16-byte
// words are exchanged by word ^ slot % 8 (the 128-byte swizzle), two to four stages of 64 slots.  lora_down.cu has left the
// parts as such lines, which bulk copies bring; z's rows come by TMA where a stage's are neighbours, in four boxes of 64
// columns, else by cp.async.  One warp does nothing but issue MMAs, which holds it for as long as they take; the others have
// the copies made, one each, and empty the accumulators.
//
// The tensor cores cut what they add off at the accumulator's last bit, so that a sum of n products is too small by some
// n 2^-25 of itself.  Every 128 slots the sums move on to the other half of the tensor memory, and the first are added to
// registers by rounding to nearest: 4096 x 4096, rank 64, 8192 slots: 2e-7 of the gradients' norm off.
//
// Those take 51 us: 134 MB of x and dy at 2.5 TB/s, 17 GFLOP.  A stage of an SM has 32 KB of z and 24 KB of parts to take in, and each of the
// 32 blocks of columns its own copy of the parts: the SMs' intake, 32 bytes a clock, is 40 us of it.
#include "fp8_tc.cuh"
#include "lora_grad.cuh"

namespace ft {

namespace {

constexpr int kTcThreads = 512, kTcAll = kTcThreads + 64, kTcSlots = 64, kTcCols = 256, kTcRing = 8, kTcWindow = 2;      // kTcWindow: stages of an accumulator
constexpr uint32_t kTcGroup = 1024, kTcAtom = kTcSlots / 8 * kTcGroup;       // bytes of eight slots' lines, of 64 columns or ranks
constexpr uint32_t kTcZStage = kTcCols / 64 * kTcAtom, kTcWPass = 128 / 64 * kTcAtom;

__host__ __device__ inline int32_t tc_stages(int32_t passes) { return 5 - passes; }
__host__ __device__ inline uint32_t tc_stage_bytes(int32_t passes) { return kTcZStage + static_cast<uint32_t>(passes) * kTcWPass; }

// Shared-memory descriptor of an M- or N-major operand with the 128-byte swizzle.
__device__ __forceinline__ uint64_t tc_desc(uint32_t at) {
    return static_cast<uint64_t>((at & 0x3FFFFu) >> 4) | static_cast<uint64_t>(kTcAtom >> 4) << 16 |
           static_cast<uint64_t>(kTcGroup >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

struct TcArgs {
    CUtensorMap zmap[2];      // boxes of 64 columns of 64 rows
    bool tma[2];
    GradArgs<__nv_bfloat16> grad;
};

__global__ void __launch_bounds__(kTcAll, 1) lora_grad_tc_kernel(const __grid_constant__ TcArgs t) {
    using T = __nv_bfloat16;
    const GradArgs<T>& a = t.grad;
    extern __shared__ uint8_t tc_smem_raw[];
    uint8_t* tc_smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tc_smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ int32_t row_ring[kTcRing][kTcSlots];      // rows of z of the stages ahead
    __shared__ __align__(8) uint64_t done[4], full[4];      // full: a stage's rows by TMA, or nothing to wait for
    __shared__ uint32_t tmem_at;
    const int32_t tid = static_cast<int32_t>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const bool second = static_cast<int32_t>(blockIdx.y) >= a.blocks0;
    const GradJob<T>& job = a.job[second ? 1 : 0];
    const int32_t col0 = (static_cast<int32_t>(blockIdx.y) - (second ? a.blocks0 : 0)) * kTcCols, cols = job.cols;
    const Chunk ck = find_chunk<kTcThreads>(a.slots, static_cast<int32_t>(blockIdx.x), a.per);
    if (ck.n == 0) {
        wait_for_prior_grid();
        return;
    }
    const int32_t R = a.rank, passes = part_passes(R), stages = tc_stages(passes), used = passes == 3 ? R : (4 - passes) * R;
    const uint32_t stage_bytes = tc_stage_bytes(passes);
    const int32_t* perm = a.slots.perm + ck.first;
    const int32_t steps = (ck.n + kTcSlots - 1) / kTcSlots;

    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&done[i], 1);
            mbar_init(&full[i], 1);
        }
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&tmem_at, 512);
        tmem_relinquish();
    }
    // with two passes, zeros in the third part's upper atom: its MMA adds to the second part's rows, too
    if (passes == 2) {
        constexpr int32_t WORDS = static_cast<int32_t>(kTcAtom / 16);
        for (int32_t i = tid; i < stages * WORDS; i += kTcAll)
            reinterpret_cast<uint4*>(tc_smem + static_cast<uint32_t>(i / WORDS) * stage_bytes + kTcZStage + kTcWPass + kTcAtom)[i % WORDS] = make_uint4(0u, 0u, 0u, 0u);
    }

    // the slots are asked for stages ahead of the rows they name
    constexpr int AHEAD = 5;
    for (int32_t i = tid; i < AHEAD * kTcSlots && i < ck.n; i += kTcAll) row_ring[i / kTcSlots][i % kTcSlots] = __ldg(perm + i) / job.div;
    auto slot_of = [&](int32_t i) { return tid < kTcSlots && i * kTcSlots + tid < ck.n ? __ldg(perm + i * kTcSlots + tid) : 0; };
    int32_t next = slot_of(AHEAD);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_at;

    // words of z: column block `lane` of slots warp, warp + 16, ..
    constexpr int WARPS = kTcThreads / 32, ZJ = kTcSlots / WARPS;
    const bool in = col0 + lane * 8 < cols, tma = t.tma[second ? 1 : 0] && job.div == 1;
    const T* z_base = job.z + (in ? col0 + lane * 8 : 0);
    const uint32_t z_to = smem_u32(tc_smem) + static_cast<uint32_t>(lane / 8) * kTcAtom + static_cast<uint32_t>(warp) * 128 + (lane % 8 ^ warp % 8) * 16;
    // lines of the parts: every kind's run of the workspace goes to the atom of its rows
    const int32_t kinds = part_kinds(R), first_lines = part_lines(R, 0);
    const uint8_t* w_src = job.w_parts + static_cast<int64_t>(ck.first) * 128;
    auto kind_to = [&](int32_t kind) {      // bytes into a stage
        const int32_t lines = passes == 3 ? first_lines : 1 << 30, pass = passes == 3 ? kind / lines : kind >= first_lines, atom = kind - pass * first_lines;
        return kTcZStage + static_cast<uint32_t>(pass) * kTcWPass + static_cast<uint32_t>(atom) * kTcAtom;
    };
    constexpr int BOXES = kTcCols / 64;
    const uint32_t my_kind_to = kind_to(warp >= BOXES && warp < BOXES + kinds ? warp - BOXES : 0);
    auto load = [&](int32_t i) {      // stages in turn
        const uint32_t stage = static_cast<uint32_t>(i % stages) * stage_bytes;
        const int32_t left = ck.n - i * kTcSlots;
        const int32_t* rows = row_ring[i % kTcRing];
        const bool run = tma && left >= kTcSlots && rows[kTcSlots - 1] - rows[0] == kTcSlots - 1;
        if (lane == 0) {      // a box or a run of lines for each warp, the count for the last
            uint64_t* bar = &full[i % stages];
            const uint32_t bytes = static_cast<uint32_t>(min(left, kTcSlots)) * 128;
            if (warp == kTcAll / 32 - 1) mbar_arrive_expect_tx(bar, (run ? kTcZStage : 0u) + static_cast<uint32_t>(kinds) * bytes);
            else if (run && warp < BOXES) tma_load_2d(tc_smem + stage + static_cast<uint32_t>(warp) * kTcAtom, &t.zmap[second ? 1 : 0], col0 + warp * 64, rows[0], bar);
            else if (warp >= BOXES && warp < BOXES + kinds)
                bulk_g2s(tc_smem + stage + my_kind_to, w_src + (static_cast<int64_t>(warp - BOXES) * a.slots.n_slots + i * kTcSlots) * 128, bytes, bar);
        }
        __syncwarp();
        if (warp >= WARPS) return;
        if (!run) {
#pragma unroll
            for (int j = 0; j < ZJ; ++j) {
                const int32_t s = warp + j * WARPS;
                const bool there = in && s < left;
                const T* src = there ? z_base + static_cast<int64_t>(rows[s]) * cols : job.z;
                copy16_at(z_to + stage + j * WARPS * 128, src, there);
            }
        }
        // a last stage's lines that are no slot's: zeros, as z has there
        for (int32_t x = left * 8 + tid; x < kTcSlots * 8; x += kTcThreads)
            for (int32_t q = 0; q < kinds; ++q) reinterpret_cast<uint4*>(tc_smem + stage + kind_to(q))[x] = make_uint4(0u, 0u, 0u, 0u);
    };

    constexpr int TC = kTcCols * 128 / kTcThreads;      // sums of a thread: row 32 (warp % 4) + lane, columns TC (warp / 4) ..
    float total[TC] = {};
    const uint32_t mine = tmem + (static_cast<uint32_t>(warp % 4 * 32) << 16) + static_cast<uint32_t>(warp / 4 * TC);
    auto drain = [&](int32_t window) {
        if (warp % 4 * 32 < used) {
#pragma unroll
            for (int q = 0; q < TC / 16; ++q) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(mine + static_cast<uint32_t>(window & 1) * kTcCols + q * 16, v);
                tmem_wait_ld_regs(v);
#pragma unroll
                for (int i = 0; i < 16; ++i) total[q * 16 + i] += __uint_as_float(v[i]);
            }
        }
        tc_fence_before();      // the accumulator is written again after the next barrier
    };

    for (int32_t i = 0; i < stages - 1; ++i) {
        if (i < steps) load(i);
        copies_commit();
    }
    bool ok = true;
    for (int32_t i = 0; i < steps; ++i) {
        if (stages == 4) copies_wait<2>();
        else if (stages == 3) copies_wait<1>();
        else copies_wait<0>();
        ok = mbar_wait_warp(&full[i % stages], static_cast<uint32_t>(i / stages & 1), a.err) && ok;
        fence_proxy_async_smem();
        ok = __syncthreads_and(ok);
        if (!ok) {      // what is under way ends before the CTA's memory goes
            for (int32_t q = i; q < steps && q < i + stages - 1; ++q)
                mbar_wait_warp(&full[q % stages], static_cast<uint32_t>(q / stages & 1), a.err, kLastWaitNs);
            if (i > 0) mbar_wait_warp(&done[(i - 1) % 4], static_cast<uint32_t>((i - 1) / 4 & 1), a.err, kLastWaitNs);
            break;
        }
        if (tid == kTcThreads) {
            tc_fence_after();
            // bf16 operands, fp32 sums, both M- or N-major, 128 x 256
            constexpr uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | 1u << 15 | 1u << 16 | (kTcCols >> 3) << 17 | (128u >> 4) << 24;
            const uint32_t zs = smem_u32(tc_smem) + static_cast<uint32_t>(i % stages) * stage_bytes, ws = zs + kTcZStage;
            const uint32_t d = tmem + static_cast<uint32_t>(i / kTcWindow & 1) * kTcCols;
            for (int32_t p = 0; p < passes; ++p)
#pragma unroll
                for (int k = 0; k < kTcSlots / 16; ++k)
                    tc_mma_f16(d, tc_desc(ws + static_cast<uint32_t>(p) * kTcWPass + k * 2 * kTcGroup), tc_desc(zs + k * 2 * kTcGroup), idesc,
                               i % kTcWindow || p || k);
            tc_commit(&done[i % 4]);
        }
        if (i > 0 && warp != WARPS) ok = mbar_wait_warp(&done[(i - 1) % 4], static_cast<uint32_t>((i - 1) / 4 & 1), a.err);
        if (warp != WARPS && i + stages - 1 < steps) load(i + stages - 1);      // where the MMAs just waited for read
        copies_commit();
        if (ok && warp < WARPS && i > 0 && i % kTcWindow == 0) {
            tc_fence_after();
            drain(i / kTcWindow - 1);
        }
        if (tid < kTcSlots) row_ring[(i + AHEAD) % kTcRing][tid] = next / job.div;
        next = slot_of(i + AHEAD + 1);
    }
    copies_wait<0>();
    if (ok) ok = mbar_wait_warp(&done[(steps - 1) % 4], static_cast<uint32_t>((steps - 1) / 4 & 1), a.err);
    ok = __syncthreads_and(ok);
    if (ok) {
        tc_fence_after();
        if (warp < WARPS) drain((steps - 1) / kTcWindow);
        const int64_t size = static_cast<int64_t>(R) * cols;
        float* out = ck.alone ? job.out + ck.adapter * size : job.parts + blockIdx.x * size;
        // the parts' rows meet in shared memory
        constexpr int PITCH = kTcCols + 1;
        float* tile = reinterpret_cast<float*>(tc_smem);
        const int32_t m = warp % 4 * 32 + lane;
        if (warp < WARPS && m < used) {
#pragma unroll
            for (int c = 0; c < TC; ++c) tile[m * PITCH + warp / 4 * TC + c] = total[c];
        }
        __syncthreads();
        auto sum = [&](int32_t r, int32_t c) {
            float v = tile[r * PITCH + c];
            if (passes < 3) v += tile[(R + r) * PITCH + c];
            if (passes < 2) v += tile[(2 * R + r) * PITCH + c];
            return v;
        };
        const int32_t width = min(kTcCols, cols - col0);
        if (job.turned) {
            for (int32_t c = warp; c < width; c += kTcAll / 32)
                for (int32_t r = lane; r < R; r += 32) out[static_cast<int64_t>(col0 + c) * R + r] = sum(r, c);
        } else {
            for (int32_t r = warp; r < R; r += kTcAll / 32)
                for (int32_t c = lane; c < width; c += 32) out[static_cast<int64_t>(r) * cols + col0 + c] = sum(r, c);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
    wait_for_prior_grid();
}

}  // namespace

int32_t lora_part_kinds(int32_t rank) { return part_kinds(rank); }

int launch_lora_grad_tc(const LoraGrad* jobs, const LoraPlan& p, cudaStream_t s) {
    int64_t blocks;
    TcArgs a{};
    a.grad = grad_args<__nv_bfloat16>(jobs, p, kTcCols, &blocks);
    int n = 0;
    for (int i = 0; i < 2; ++i) {
        if (!jobs[i].out) continue;
        a.tma[n] = jobs[i].div == 1 && jobs[i].cols >= 64;
        if (a.tma[n])
            if (int st = encode_2d(&a.zmap[n], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, jobs[i].z, static_cast<uint64_t>(jobs[i].cols),
                                   static_cast<uint64_t>(p.n_slots), static_cast<uint64_t>(jobs[i].cols) * 2, 64, kTcSlots, CU_TENSOR_MAP_SWIZZLE_128B,
                                   "rows of an adapter"))
                return st;
        ++n;
    }
    const dim3 grid(static_cast<unsigned>(lora_chunks(p.n_slots, p.n_adapters, p.chunk)), static_cast<unsigned>(blocks)), block(kTcAll);
    const int32_t passes = part_passes(p.rank);
    const size_t sm = static_cast<size_t>(tc_stages(passes)) * tc_stage_bytes(passes) + 1024;
    auto go = [&](auto k) { return launch_with(k, "lora_grad_tc_kernel", grid, block, sm, p.overlap_grad, 1, s, a); };
    return go(lora_grad_tc_kernel);
}

}  // namespace ft
