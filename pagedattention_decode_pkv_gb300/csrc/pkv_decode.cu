// Paged decode attention: one query token per sequence, GQA, split-K over the
// context with a log-sum-exp combine.
//
// "Paged KV Cache - AI infra interview lesson", "Step 2: paged_attention_decode":
// n_blk = ceil(ctx / bs) block ids are taken from the sequence's table row
// (later entries may be -1); K and V are gathered through them, the unused
// tail of the last block is cut, query head h reads KV head h // (Hq / H_kv),
// and the result is softmax(q K^T * scale) V.
//
// Design (GB300, sm_103a)
// -----------------------
// The kernel is HBM-bound: every cached K/V byte of a sequence is read once.
// Work unit = (sequence b, group of HPC KV heads, partition j of the context).
// One CTA per unit runs a TMA -> shared-memory pipeline:
//   * a producer warp issues, per 16-token stage, two cp.async.bulk.tensor
//     loads (K and V) of the box [HPC heads x 2 halves x 16 tokens x 64 dims]
//     out of a 3-D tensor map over the pool viewed as
//     (64 elements, num_slots rows, 2 * H_kv half-rows), 128-byte swizzled, so
//     that the 16 tokens of one head are consecutive 128-byte rows in shared
//     memory and every ldmatrix below is bank-conflict free;
//   * one consumer warp per KV head keeps all G = Hq / H_kv query heads of its
//     group in registers (as the B operand of mma.m16n8k16, G <= 8 padded to
//     n = 8) and computes S^T = K Q^T for the 16 tokens with 8 MMAs, an online
//     softmax on the accumulator fragment (max/sum over tokens via 3 shuffles),
//     transposes P in registers with movmatrix and accumulates O^T += V^T P^T
//     with 8 more MMAs (V read with ldmatrix.trans).  Each K/V byte therefore
//     costs a handful of instructions instead of G FMAs + conversions, which
//     keeps the SMs far from the issue limit at HBM speed.
// mbarrier full/empty pairs hand stages between producer and consumers; all
// waits are bounded and report PKV_ERRBIT_TIMEOUT instead of hanging.
// A partition's output is written directly when the sequence fits in one
// partition, otherwise as an unnormalised fp32 partial (o, max, sum) that the
// combine kernel merges.  Shapes outside the fast path (fp32, other head
// dims, G > 8, block sizes not a multiple of 16) run a plain CUDA-core kernel
// with the same partitioning and the same combine.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdlib>
#include <type_traits>

#include "pkv_decode.cuh"

namespace pkv {
namespace {

// ----------------------------------------------------------------------------- plan
int env_partition_override() {
    static int v = [] {
        const char *s = std::getenv("PKV_DECODE_PARTITION_TOKENS");
        return s ? std::atoi(s) : 0;
    }();
    return v;
}

// generic_only: plan the CUDA-core kernel (used when the fast path's pointer
// alignment does not hold at call time); max_parts > 0 caps the partitions so
// that the partials fit a workspace sized for another plan; grouped: more than
// kMaxStreamSeqs sequences run as groups of the work-balanced kernel (8-bit caches
// and score rules, which the fixed-partition kernel does not have).
Plan make_plan(int B, int Hq, int Hkv, int d, int bs, int max_ctx, pkv_dtype dt, bool generic_only = false,
               int64_t max_parts = 0, bool grouped = false) {
    Plan p;
    const int G = Hq / Hkv;
    p.fast = !generic_only && (dt == PKV_F16 || dt == PKV_BF16) && d == kFastHeadDim && G >= 1 && G <= 8 &&
             bs % kStageTokens == 0 && bs <= 32768;
    p.hpc = (Hkv % 4 == 0) ? 4 : (Hkv % 2 == 0) ? 2 : 1;
    const int stage_bytes = p.hpc * 2 * kStageTokens * kFastHeadDim * 2;
    p.stages = 98304 / stage_bytes;
    if (p.stages > 8) p.stages = 8;
    if (p.stages < 2) p.stages = 2;
    // Past kMaxStreamSeqs sequences, 16-bit caches take the fixed-partition
    // kernel (a many-wave grid: measured 7.33 TB/s on 1024 Qwen3-shaped
    // sequences); 8-bit caches and score rules, which only the work-balanced
    // kernel has, run it as consecutive launches over groups of near-equal size that reuse
    // one scratch region in stream order (each launch's first global access
    // waits for the previous grid to complete).
    p.stream = p.fast && (B <= kMaxStreamSeqs || grouped);
    if (p.stream) {
        p.groups = B > kMaxStreamSeqs ? (B + kMaxStreamSeqs - 1) / kMaxStreamSeqs : 1;
        p.group_seqs = (B + p.groups - 1) / p.groups;
        // Pieces: at most one per (unit, segment) boundary; segments are the
        // static slices (at most kMaxStreamCtas) and the dynamic-tail chunks.
        const int64_t HG = Hkv / p.hpc, HU = Hq / HG;
        p.units = static_cast<int64_t>(p.group_seqs) * HG;
        const int64_t w_max = p.units * ((static_cast<int64_t>(max_ctx) + kStageTokens - 1) / kStageTokens);
        p.max_chunks = w_max / kTailDenominator / kChunkStages + 1;
        // static slots [0, kMaxStreamCtas + units), dynamic slots after them
        p.max_segments = 2 * p.units + kMaxStreamCtas + p.max_chunks;  // piece slots
        const size_t pieces = static_cast<size_t>(p.max_segments);
        p.o_bytes = (pieces * HU * d * sizeof(float) + 255) / 256 * 256;
        p.ml_bytes = (pieces * HU * sizeof(float2) + 255) / 256 * 256;
        p.unit_bytes = (static_cast<size_t>(p.units) * sizeof(int4) + 255) / 256 * 256;
        p.ws_bytes = p.o_bytes + p.ml_bytes + p.unit_bytes + 256;  // + Cw and the chunk counter
        p.partition = 0;
        p.nparts = 0;
        return p;
    }
    const int64_t units = static_cast<int64_t>(B) * (p.fast ? Hkv / p.hpc : Hq);
    // Aim for ~8 waves of 2 CTAs per SM; partitions are multiples of 64 tokens.
    const int64_t target = static_cast<int64_t>(kTargetSms) * 2 * 8;
    int64_t P = (static_cast<int64_t>(max_ctx) * units + target - 1) / target;
    P = ((P + 63) / 64) * 64;
    if (P < 256) P = 256;
    if (env_partition_override() > 0) P = ((env_partition_override() + 15) / 16) * 16;
    if (max_parts > 0 && (static_cast<int64_t>(max_ctx) + P - 1) / P > max_parts)
        P = ((static_cast<int64_t>(max_ctx) + max_parts - 1) / max_parts + 15) / 16 * 16;
    if (P > kMaxPartition) P = kMaxPartition;
    if (P >= max_ctx) P = ((max_ctx > 0 ? max_ctx : 1) + 15) / 16 * 16;
    if (P > kMaxPartition) P = kMaxPartition;
    p.partition = static_cast<int>(P);
    p.nparts = max_ctx > 0 ? static_cast<int>((max_ctx + P - 1) / P) : 0;
    if (p.nparts > 1) {
        const size_t rows = static_cast<size_t>(B) * Hq * p.nparts;
        p.o_bytes = (rows * d * sizeof(float) + 255) / 256 * 256;
        p.ml_bytes = (rows * sizeof(float2) + 255) / 256 * 256;
        p.ws_bytes = p.o_bytes + p.ml_bytes;
    }
    return p;
}

// ----------------------------------------------------------------------------- fast kernel
template <int HPC, int STAGES>
struct FastSmem {
    static constexpr int kTileBytes = HPC * 2 * kStageTokens * 128;  // one of K / V per stage
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kTilesBytes = STAGES * kStageBytes;
    static constexpr int kBlkOffset = kTilesBytes;
    static constexpr int kBarOffset = kBlkOffset + kMaxStagesPerPartition * 4;
    static constexpr int kFlagOffset = kBarOffset + 2 * STAGES * 8;
    static constexpr int kBytes = kFlagOffset + 16;
    static constexpr int kAlloc = kBytes + 1024;  // slack for 1024-byte alignment
};

template <typename T, int HPC, int STAGES>
__global__ void __launch_bounds__((HPC + 1) * 32)
decode_fast_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   T *__restrict__ out, const T *__restrict__ q,
                   const int32_t *__restrict__ block_tables, int32_t max_blocks,
                   const int32_t *__restrict__ context_lens, int32_t Hq, int32_t G, int32_t bs,
                   int32_t num_blocks, int32_t max_ctx, int32_t partition, int32_t nparts,
                   float scale_log2, float *__restrict__ o_part, float2 *__restrict__ ml_part,
                   int32_t *__restrict__ err_flag) {
    using L = FastSmem<HPC, STAGES>;
    using H = Half16<T>;
    pdl_wait();
    pdl_trigger();
    const int j = blockIdx.x, hg = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ctx = context_lens[b];
    const int heads_per_cta = HPC * G;
    if (!context_ok(ctx, max_ctx, bs, max_blocks) || ctx == 0) {
        if (j == 0) {
            if (ctx != 0 && threadIdx.x == 0 && err_flag) atomicOr(err_flag, PKV_ERRBIT_CONTEXT);
            T *o = out + (static_cast<int64_t>(b) * Hq + static_cast<int64_t>(hg) * heads_per_cta) * kFastHeadDim;
            for (int i = threadIdx.x; i < heads_per_cta * kFastHeadDim; i += blockDim.x) o[i] = from_f32<T>(0.f);
        }
        return;
    }
    const int t0 = j * partition;
    if (t0 >= ctx) return;
    // Once any CTA has reported a broken pipeline, the rest of the launch stops early.
    if (err_flag && (*reinterpret_cast<volatile int32_t *>(err_flag) & PKV_ERRBIT_TIMEOUT)) return;
    const uint64_t deadline = global_ns() + kCtaDeadlineNs;
    const int t1 = min(t0 + partition, ctx);
    const int nstage = (t1 - t0 + kStageTokens - 1) / kStageTokens;
    const bool single = ctx <= partition;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int32_t *sblk = reinterpret_cast<int32_t *>(smem + L::kBlkOffset);
    const uint32_t bar0 = smem_u32(smem + L::kBarOffset);  // full[s] = bar0 + 8s, empty[s] = bar0 + 8(STAGES+s)
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kFlagOffset);
    const uint32_t tiles = smem_u32(smem);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar0 + 8 * s, 1);
            mbar_init(bar0 + 8 * (STAGES + s), HPC);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == HPC) {  // producer warp: resolve this partition's block ids once
        const int32_t *row = block_tables + static_cast<int64_t>(b) * max_blocks;
        bool bad = false;
        for (int s = lane; s < nstage; s += 32) {
            const int pos = t0 + s * kStageTokens;
            int32_t id = row[pos / bs];
            if (id < 0 || id >= num_blocks) { id = -1; bad = true; }
            sblk[s] = id;
        }
        if (bad && err_flag) atomicOr(err_flag, PKV_ERRBIT_BLOCK_RANGE);
    }
    __syncthreads();

    if (warp == HPC) {
        if (lane == 0) {
            int issued = 0;
            for (int s = 0; s < nstage; ++s) {
                const int slot = s % STAGES;
                const uint32_t full = bar0 + 8 * slot, empty = bar0 + 8 * (STAGES + slot);
                if (s >= STAGES && !mbar_wait(empty, ((s / STAGES) - 1) & 1, deadline)) {
                    *abort_flag = 1;
                    if (err_flag) atomicOr(err_flag, PKV_ERRBIT_TIMEOUT);
                    break;
                }
                const int id = sblk[s];
                if (id >= 0) {
                    const int slot_row = id * bs + (t0 + s * kStageTokens) % bs;
                    const uint32_t dst = tiles + slot * L::kStageBytes;
                    mbar_arrive_expect_tx(full, L::kStageBytes);
                    tma_load_3d(dst, &tm_k, 0, slot_row, 2 * hg * HPC, full);
                    tma_load_3d(dst + L::kTileBytes, &tm_v, 0, slot_row, 2 * hg * HPC, full);
                } else {
                    mbar_arrive(full);  // nothing to load: consumers mask the whole stage
                }
                issued = s + 1;
            }
            // Drain: no bulk copy may still be writing shared memory when the CTA exits.
            for (int s = issued - STAGES > 0 ? issued - STAGES : 0; s < issued; ++s)
                if (!mbar_wait(bar0 + 8 * (s % STAGES), (s / STAGES) & 1, deadline) && err_flag)
                    atomicOr(err_flag, PKV_ERRBIT_TIMEOUT);
        }
        return;
    }

    // ---------------------------------------------------------------- consumer warp
    const int g = lane >> 2, t = lane & 3;
    const int hk = hg * HPC + warp;  // KV head of this warp
    uint32_t qf[8][2];
    {
        const bool live = g < G;
        const T *qrow = q + (static_cast<int64_t>(b) * Hq + static_cast<int64_t>(hk) * G + (live ? g : 0)) * kFastHeadDim;
        const uint32_t *q32 = reinterpret_cast<const uint32_t *>(qrow);
#pragma unroll
        for (int kc = 0; kc < 8; ++kc) {
            qf[kc][0] = live ? __ldg(q32 + kc * 8 + t) : 0u;
            qf[kc][1] = live ? __ldg(q32 + kc * 8 + 4 + t) : 0u;
        }
    }
    float o[8][4];
#pragma unroll
    for (int dc = 0; dc < 8; ++dc)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[dc][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    // Per-lane ldmatrix row offsets inside this warp's head (rows of 128 B,
    // row R = (2 * warp + half) * 16 + token, chunk swizzled with R & 7).
    const int mi = lane >> 3, r = lane & 7;
    const uint32_t head_off = static_cast<uint32_t>(warp) * 2 * kStageTokens * 128;
    uint32_t k_off[8], v_off[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        {   // QK: A = K[16 tokens x 16 dims]; matrices (tok 0-7|8-15) x (dims 0-7|8-15)
            const int tok = r + 8 * (mi & 1);
            const int c16 = 2 * c + (mi >> 1);
            const int R = ((c16 >> 3)) * kStageTokens + tok;
            k_off[c] = head_off + R * 128 + (((c16 & 7) ^ r) << 4);
        }
        {   // PV: A = V^T[16 dims x 16 tokens] via .trans; matrices (dims 0-7|8-15) x (tok 0-7|8-15)
            const int tok = r + 8 * (mi >> 1);
            const int c16 = 2 * c + (mi & 1);
            const int R = ((c16 >> 3)) * kStageTokens + tok;
            v_off[c] = head_off + R * 128 + (((c16 & 7) ^ r) << 4);
        }
    }

    for (int s = 0; s < nstage; ++s) {
        const int slot = s % STAGES;
        if (!mbar_wait(bar0 + 8 * slot, (s / STAGES) & 1, deadline) || *abort_flag) {
            if (lane == 0 && err_flag) atomicOr(err_flag, PKV_ERRBIT_TIMEOUT);
            return;
        }
        const uint32_t kt = tiles + slot * L::kStageBytes;
        const uint32_t vt = kt + L::kTileBytes;
        const int id = sblk[s];
        const int pos0 = t0 + s * kStageTokens;
        const int nvalid = id < 0 ? 0 : min(kStageTokens, t1 - pos0);
        if (nvalid < kStageTokens) {
            // Rows past the context (or of a skipped block) may hold anything,
            // NaN included: zero this head's V rows so 0 * row stays 0.
            const int nbad = kStageTokens - nvalid;
            for (int idx = lane; idx < nbad * 16; idx += 32) {
                const int tok = nvalid + (idx >> 4);
                const int half = (idx >> 3) & 1;
                const int chunk = idx & 7;
                const uint32_t addr = vt + head_off + (half * kStageTokens + tok) * 128 + chunk * 16;
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
            }
            __syncwarp();
        }
        float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kc = 0; kc < 8; ++kc) {
            uint32_t a[4];
            ldsm_x4(kt + k_off[kc], a);
            H::mma(sc, a, qf[kc][0], qf[kc][1]);
        }
        // scores in log2 units; masked tokens -> -inf
        const bool vg = g < nvalid, vg8 = g + 8 < nvalid;
        const float x0 = vg ? sc[0] * scale_log2 : -INFINITY;
        const float x1 = vg ? sc[1] * scale_log2 : -INFINITY;
        const float x2 = vg8 ? sc[2] * scale_log2 : -INFINITY;
        const float x3 = vg8 ? sc[3] * scale_log2 : -INFINITY;
        float mx0 = fmaxf(x0, x2), mx1 = fmaxf(x1, x3);
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, sh));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, sh));
        }
        const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
        const float base0 = mn0 == -INFINITY ? 0.f : mn0;
        const float base1 = mn1 == -INFINITY ? 0.f : mn1;
        const float p0 = fast_exp2(x0 - base0), p1 = fast_exp2(x1 - base1);
        const float p2 = fast_exp2(x2 - base0), p3 = fast_exp2(x3 - base1);
        const float a0 = fast_exp2(m0 - base0), a1 = fast_exp2(m1 - base1);
        m0 = mn0;
        m1 = mn1;
        l0 = l0 * a0 + (p0 + p2);
        l1 = l1 * a1 + (p1 + p3);
#pragma unroll
        for (int dc = 0; dc < 8; ++dc) {
            o[dc][0] *= a0;
            o[dc][1] *= a1;
            o[dc][2] *= a0;
            o[dc][3] *= a1;
        }
        const uint32_t pb0 = movmatrix_trans(H::pack(p0, p1));
        const uint32_t pb1 = movmatrix_trans(H::pack(p2, p3));
#pragma unroll
        for (int dc = 0; dc < 8; ++dc) {
            uint32_t a[4];
            ldsm_x4_trans(vt + v_off[dc], a);
            H::mma(o[dc], a, pb0, pb1);
        }
        if (nvalid < kStageTokens) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar0 + 8 * (STAGES + slot));
    }

    // row sums over the 16 token lanes of each head column
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, sh);
        l1 += __shfl_xor_sync(0xffffffffu, l1, sh);
    }
    const int hA = 2 * t, hB = 2 * t + 1;  // head columns of this lane
    const int64_t qhead0 = static_cast<int64_t>(b) * Hq + static_cast<int64_t>(hk) * G;
    if (single) {
        const float inv0 = l0 > 0.f ? 1.f / l0 : 0.f, inv1 = l1 > 0.f ? 1.f / l1 : 0.f;
#pragma unroll
        for (int dc = 0; dc < 8; ++dc) {
            const int d0 = dc * 16 + g;
            if (hA < G) {
                T *dst = out + (qhead0 + hA) * kFastHeadDim;
                dst[d0] = from_f32<T>(o[dc][0] * inv0);
                dst[d0 + 8] = from_f32<T>(o[dc][2] * inv0);
            }
            if (hB < G) {
                T *dst = out + (qhead0 + hB) * kFastHeadDim;
                dst[d0] = from_f32<T>(o[dc][1] * inv1);
                dst[d0 + 8] = from_f32<T>(o[dc][3] * inv1);
            }
        }
    } else {
#pragma unroll
        for (int dc = 0; dc < 8; ++dc) {
            const int d0 = dc * 16 + g;
            if (hA < G) {
                float *dst = o_part + ((qhead0 + hA) * nparts + j) * kFastHeadDim;
                dst[d0] = o[dc][0];
                dst[d0 + 8] = o[dc][2];
            }
            if (hB < G) {
                float *dst = o_part + ((qhead0 + hB) * nparts + j) * kFastHeadDim;
                dst[d0] = o[dc][1];
                dst[d0 + 8] = o[dc][3];
            }
        }
        if (g == 0) {
            if (hA < G) ml_part[(qhead0 + hA) * nparts + j] = make_float2(m0, l0);
            if (hB < G) ml_part[(qhead0 + hB) * nparts + j] = make_float2(m1, l1);
        }
    }
}

// ----------------------------------------------------------------------------- append (other paths)
// The step's new K/V rows for the paths that do not append inside the
// attention kernel: row ctx - 1 of every sequence with a valid, non-empty
// context receives key[b] / value[b] (the slot rule of "Step 1: slot_mapping
// and store_kvcache").  One warp per (sequence, segment of 32 x 4 vectors).
constexpr int kAppendThreads = 256;

template <typename V>
__global__ void __launch_bounds__(kAppendThreads)
append_kv_kernel(const char *__restrict__ key, const char *__restrict__ value, char *__restrict__ k_cache,
                 char *__restrict__ v_cache, const int32_t *__restrict__ block_tables, int32_t max_blocks,
                 const int32_t *__restrict__ context_lens, int32_t B, int32_t bs, int32_t num_blocks,
                 int32_t max_ctx, int64_t row_bytes, int32_t *__restrict__ err_flag) {
    pdl_wait();
    pdl_trigger();
    constexpr int64_t kSeg = 32 * 4 * static_cast<int64_t>(sizeof(V));
    const int lane = threadIdx.x & 31;
    const int64_t nseg = (row_bytes + kSeg - 1) / kSeg;
    const int64_t items = static_cast<int64_t>(B) * nseg;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kAppendThreads / 32);
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5); it < items;
         it += warps) {
        const int b = static_cast<int>(it / nseg);
        const int64_t seg = it - static_cast<int64_t>(b) * nseg;
        const int ctx = context_lens[b];
        if (ctx <= 0 || !context_ok(ctx, max_ctx, bs, max_blocks)) continue;  // the attention flags it
        const int p = ctx - 1;
        const int32_t blk = block_tables[static_cast<int64_t>(b) * max_blocks + p / bs];
        if (blk < 0 || blk >= num_blocks) {
            if (lane == 0 && seg == 0 && err_flag) atomicOr(err_flag, PKV_ERRBIT_BLOCK_RANGE);
            continue;
        }
        const int64_t src = static_cast<int64_t>(b) * row_bytes + seg * kSeg;
        const int64_t dst = (static_cast<int64_t>(blk) * bs + p % bs) * row_bytes + seg * kSeg;
        V kv[4], vv[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t off = (static_cast<int64_t>(u) * 32 + lane) * static_cast<int64_t>(sizeof(V));
            if (seg * kSeg + off < row_bytes) {
                kv[u] = *reinterpret_cast<const V *>(key + src + off);
                vv[u] = *reinterpret_cast<const V *>(value + src + off);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t off = (static_cast<int64_t>(u) * 32 + lane) * static_cast<int64_t>(sizeof(V));
            if (seg * kSeg + off < row_bytes) {
                *reinterpret_cast<V *>(k_cache + dst + off) = kv[u];
                *reinterpret_cast<V *>(v_cache + dst + off) = vv[u];
            }
        }
    }
}

// ----------------------------------------------------------------------------- host side
pkv_status launch_append(const DecodeArgs &a, int64_t es) {
    const int64_t row_bytes = static_cast<int64_t>(a.Hkv) * a.d * es;
    auto kc = static_cast<char *>(const_cast<void *>(a.k_cache));
    auto vc = static_cast<char *>(const_cast<void *>(a.v_cache));
    auto kk = static_cast<const char *>(a.new_k);
    auto vv = static_cast<const char *>(a.new_v);
    const bool v16 = row_bytes % 16 == 0 && aligned(kc, 16) && aligned(vc, 16) && aligned(kk, 16) && aligned(vv, 16);
    const bool v8 = row_bytes % 8 == 0 && aligned(kc, 8) && aligned(vc, 8) && aligned(kk, 8) && aligned(vv, 8);
    const int64_t vec = v16 ? 16 : v8 ? 8 : es;
    const int64_t items = static_cast<int64_t>(a.B) * ((row_bytes + 128 * vec - 1) / (128 * vec));
    int64_t grid = (items + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
    if (grid > 1024) grid = 1024;
    if (grid < 1) grid = 1;
    cudaError_t e;
#define PKV_APPEND(V) \
    launch_pdl(kPdlStore, append_kv_kernel<V>, dim3(static_cast<unsigned>(grid)), dim3(kAppendThreads), 0, a.stream, kk, \
               vv, kc, vc, a.block_tables, a.max_blocks, a.context_lens, a.B, a.bs, a.num_blocks, a.max_ctx, row_bytes, a.err)
    switch (vec) {
    case 16: e = PKV_APPEND(int4); break;
    case 8: e = PKV_APPEND(int2); break;
    case 4: e = PKV_APPEND(int); break;
    default: e = PKV_APPEND(short); break;
    }
#undef PKV_APPEND
    if (e != cudaSuccess) return set_error(PKV_ERR_CUDA, "append launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}

int stream_grid_for(pkv_dtype dt, int hpc) {
    if (dt == PKV_BF16) {
        switch (hpc) {
        case 4: return StreamLaunch<__nv_bfloat16, 4, 3, kCode16, false>::grid();
        case 2: return StreamLaunch<__nv_bfloat16, 2, 6, kCode16, false>::grid();
        default: return StreamLaunch<__nv_bfloat16, 1, 8, kCode16, false>::grid();
        }
    }
    switch (hpc) {
    case 4: return StreamLaunch<__half, 4, 3, kCode16, false>::grid();
    case 2: return StreamLaunch<__half, 2, 6, kCode16, false>::grid();
    default: return StreamLaunch<__half, 1, 8, kCode16, false>::grid();
    }
}

template <typename T, int HPC, int STAGES>
pkv_status launch_fast(const DecodeArgs &a, const Plan &p) {
    using L = FastSmem<HPC, STAGES>;
    CUtensorMap mk, mv;
    pkv_status st = make_kv_map(&mk, a.k_cache, Half16<T>::kTmaType, static_cast<int64_t>(a.num_blocks) * a.bs, a.Hkv, HPC);
    if (st != PKV_OK) return st;
    st = make_kv_map(&mv, a.v_cache, Half16<T>::kTmaType, static_cast<int64_t>(a.num_blocks) * a.bs, a.Hkv, HPC);
    if (st != PKV_OK) return st;
    auto kern = decode_fast_kernel<T, HPC, STAGES>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = ensure_smem(kern, L::kAlloc, configured);
    if (e != cudaSuccess) return set_error(PKV_ERR_CUDA, "decode: smem attribute: %s", cudaGetErrorString(e));
    // At least one partition, so that zero-length contexts still get their zero rows.
    dim3 grid(p.nparts > 0 ? p.nparts : 1, a.Hkv / HPC, a.B);
    e = launch_pdl(kPdlDecode, kern, grid, dim3((HPC + 1) * 32), L::kAlloc, a.stream, mk, mv, static_cast<T *>(a.out),
                   static_cast<const T *>(a.q), a.block_tables, a.max_blocks, a.context_lens, a.Hq, a.Hq / a.Hkv,
                   a.bs, a.num_blocks, a.max_ctx, p.partition, p.nparts, a.scale * kLog2e, a.o_part, a.ml_part,
                   a.err);
    if (e != cudaSuccess) return set_error(PKV_ERR_CUDA, "decode launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}

template <typename T>
pkv_status launch_fast_any(const DecodeArgs &a, const Plan &p) {
    switch (p.hpc) {
    case 4: return launch_fast<T, 4, 3>(a, p);
    case 2: return launch_fast<T, 2, 6>(a, p);
    default: return launch_fast<T, 1, 8>(a, p);
    }
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_paged_attention_decode_workspace_size(int32_t num_seqs, int32_t num_q_heads,
                                                            int32_t num_kv_heads, int32_t head_dim,
                                                            int32_t block_size, int32_t max_context_len,
                                                            pkv_dtype dtype) {
    if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
        head_dim <= 0 || block_size <= 0 || max_context_len < 0 || dtype_bytes(dtype) == 0)
        return 0;
    // one size for 16-bit and 8-bit caches (their plans differ past 512 sequences)
    const size_t a = make_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, dtype).ws_bytes;
    const size_t b = make_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, dtype,
                               false, 0, true).ws_bytes;
    return a > b ? a : b;
}

extern "C" pkv_status pkv_paged_attention_decode_plan(int32_t num_seqs, int32_t num_q_heads,
                                                      int32_t num_kv_heads, int32_t head_dim,
                                                      int32_t block_size, int32_t max_context_len,
                                                      pkv_dtype dtype, int32_t *partition_tokens,
                                                      int32_t *num_partitions, int32_t *fast_path) {
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
        head_dim <= 0 || block_size <= 0 || max_context_len < 0 || dtype_bytes(dtype) == 0)
        return set_error(PKV_ERR_INVALID_ARG, "decode plan: bad sizes");
    Plan p = make_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, dtype);
    if (partition_tokens) *partition_tokens = p.partition;
    if (num_partitions) *num_partitions = p.stream ? stream_grid_for(dtype, p.hpc) : p.nparts;
    if (fast_path) *fast_path = p.fast ? 1 : 0;
    return ok();
}

namespace pkv {
namespace {

// Sizes, dtype and pointers of a decode call, checked before anything else
// (the workspace is checked later, against the plan these sizes give).
pkv_status check_decode_args(const void *out, const void *q, const void *k_cache, const void *v_cache,
                             const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *context_lens,
                             int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                             int32_t block_size, int32_t num_blocks, int32_t max_context_len, pkv_dtype dtype) {
    if (dtype_bytes(dtype) == 0) return set_error(PKV_ERR_INVALID_ARG, "decode: unknown dtype %d", (int)dtype);
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        num_blocks < 0 || max_context_len < 0 || max_blocks_per_seq < 0)
        return set_error(PKV_ERR_INVALID_ARG, "decode: bad sizes");
    if (num_q_heads % num_kv_heads)
        return set_error(PKV_ERR_INVALID_ARG, "decode: num_q_heads (%d) is not a multiple of num_kv_heads (%d)",
                         num_q_heads, num_kv_heads);
    if (head_dim > 1024) return set_error(PKV_ERR_UNSUPPORTED, "decode: head_dim > 1024");
    if (static_cast<int64_t>(num_blocks) * block_size > INT32_MAX)
        return set_error(PKV_ERR_INVALID_ARG, "decode: num_blocks * block_size >= 2^31");
    if (num_seqs > 65535) return set_error(PKV_ERR_UNSUPPORTED, "decode: more than 65535 sequences in one call");
    if (num_seqs > 0 && (!out || !q || !context_lens || (max_blocks_per_seq > 0 && !block_tables) ||
                         (num_blocks > 0 && (!k_cache || !v_cache))))
        return set_error(PKV_ERR_INVALID_ARG, "decode: NULL pointer");
    return PKV_OK;
}

// Decode attention, with the step's new K/V rows appended first when new_k is
// not null (the fused decode step).
pkv_status decode_entry(void *out, const void *q, const void *k_cache, const void *v_cache,
                        const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *context_lens,
                        int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                        int32_t block_size, int32_t num_blocks, int32_t max_context_len, float scale,
                        pkv_dtype dtype, void *workspace, size_t workspace_bytes, int32_t *err_flag, void *stream,
                        const void *new_k, const void *new_v, const float *k_scale = nullptr,
                        const float *v_scale = nullptr, int32_t codes = kCode16, const DecodeMod *mod = nullptr) {
    const int64_t es = dtype_bytes(dtype);
    const bool c8 = codes != kCode16;  // 8-bit caches with per-(block, head) scales
    const char *fmt = codes == kCodeInt8 ? "int8" : "fp8";
    pkv_status chk = check_decode_args(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                                       num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                                       max_context_len, dtype);
    if (chk != PKV_OK) return chk;
    if (num_seqs == 0) return ok();
    const bool append = new_k != nullptr || new_v != nullptr;
    if (append && (!new_k || !new_v || !aligned(new_k, es) || !aligned(new_v, es)))
        return set_error(PKV_ERR_INVALID_ARG, "decode append: key/value NULL or not aligned to the element size");
    Plan p = make_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, dtype, false, 0,
                       c8 || mod);
    if (p.ws_bytes > 0 && (!workspace || workspace_bytes < p.ws_bytes || !aligned(workspace, 256)))
        return set_error(PKV_ERR_WORKSPACE, "decode: workspace needs %zu bytes (256-byte aligned), got %zu",
                         p.ws_bytes, workspace_bytes);
    if (!aligned(out, es) || !aligned(q, es) || (k_cache && !aligned(k_cache, es)) || (v_cache && !aligned(v_cache, es)))
        return set_error(PKV_ERR_INVALID_ARG, "decode: buffers not aligned to the element size");
    // The fast path additionally wants 16-byte aligned pools (TMA) and 4-byte aligned q.
    const bool fast = p.fast && num_blocks > 0 && aligned(k_cache, 16) && aligned(v_cache, 16) && aligned(q, 4);
    if (c8) {
        if (!fast || !p.stream || !aligned(q, 16) || (append && (!aligned(new_k, 8) || !aligned(new_v, 8))))
            return set_error(PKV_ERR_UNSUPPORTED,
                             "decode %s: needs fp16/bf16 q, head_dim 128, Hq/Hkv <= 8, block_size a multiple of "
                             "16, 16-byte aligned q and code pools (and 8-byte aligned key/value to append)",
                             fmt);
        if (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4))
            return set_error(PKV_ERR_INVALID_ARG, "decode %s: scales NULL or not 4-byte aligned", fmt);
    }
    if (p.fast && !fast) {
        // CUDA-core fallback with partitions that fit the workspace sized for the fast plan.
        const int64_t per_part = static_cast<int64_t>(num_seqs) * num_q_heads * (head_dim * 4 + 8);
        const int64_t max_parts = p.ws_bytes > 512 ? (static_cast<int64_t>(p.ws_bytes) - 512) / per_part : 1;
        p = make_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, dtype, true,
                      max_parts > 0 ? max_parts : 1);
        if (p.ws_bytes > workspace_bytes)
            return set_error(PKV_ERR_WORKSPACE, "decode: unaligned pools need the CUDA-core path, whose partials "
                                                "(%zu bytes) do not fit the workspace (%zu bytes)",
                             p.ws_bytes, workspace_bytes);
    }
    char *ws = static_cast<char *>(workspace);
    DecodeArgs a{out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, num_q_heads,
                 num_kv_heads, head_dim, block_size, num_blocks, max_context_len, scale,
                 p.ws_bytes ? reinterpret_cast<float *>(ws) : nullptr,
                 p.ws_bytes ? reinterpret_cast<float2 *>(ws + p.o_bytes) : nullptr,
                 p.stream ? reinterpret_cast<int4 *>(ws + p.o_bytes + p.ml_bytes) : nullptr,
                 p.stream ? reinterpret_cast<int32_t *>(ws + p.o_bytes + p.ml_bytes + p.unit_bytes) : nullptr,
                 p.stream ? reinterpret_cast<uint32_t *>(ws + p.o_bytes + p.ml_bytes + p.unit_bytes + 8) : nullptr,
                 nullptr, nullptr, nullptr, nullptr, err_flag, static_cast<cudaStream_t>(stream)};
    pkv_status st;
    // The work-balanced kernel appends in its producer warp (8-byte copies);
    // every other path runs the append kernel first, in stream order.
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.codes = codes;
    if (mod) a.mod = *mod;
    const bool fused = append && fast && p.stream && aligned(new_k, 8) && aligned(new_v, 8);
    if (fused) {
        a.new_k = new_k;
        a.new_v = new_v;
    } else if (append && num_blocks > 0 && max_blocks_per_seq > 0) {
        a.new_k = new_k;
        a.new_v = new_v;
        st = launch_append(a, es);
        if (st != PKV_OK) return st;
        a.new_k = a.new_v = nullptr;
    }
    if (fast && p.stream) {
        // one work-balanced launch (and merge) per group of sequences
        const int64_t q_row = static_cast<int64_t>(num_q_heads) * head_dim * es;
        const int64_t kv_row = static_cast<int64_t>(num_kv_heads) * head_dim * es;
        for (int g = 0; g < p.groups; ++g) {
            const int b0 = g * p.group_seqs;
            DecodeArgs ag = a;
            ag.B = min(p.group_seqs, num_seqs - b0);
            ag.out = static_cast<char *>(out) + b0 * q_row;
            ag.q = static_cast<const char *>(q) + b0 * q_row;
            ag.block_tables = block_tables ? block_tables + static_cast<int64_t>(b0) * max_blocks_per_seq : nullptr;
            ag.context_lens = context_lens + b0;
            if (ag.mod.key_starts) ag.mod.key_starts += b0;
            if (a.new_k) {
                ag.new_k = static_cast<const char *>(a.new_k) + b0 * kv_row;
                ag.new_v = static_cast<const char *>(a.new_v) + b0 * kv_row;
            }
            st = mod                 ? launch_stream_mod(ag, p, dtype)
                 : dtype == PKV_BF16 ? launch_stream_any<__nv_bfloat16, false>(ag, p)
                                     : launch_stream_any<__half, false>(ag, p);
            if (st != PKV_OK) return st;
        }
    } else if (fast) {
        st = dtype == PKV_BF16 ? launch_fast_any<__nv_bfloat16>(a, p) : launch_fast_any<__half>(a, p);
        if (st != PKV_OK) return st;
        st = dtype == PKV_BF16 ? launch_generic_and_combine<__nv_bfloat16, false>(a, p, false)
                               : launch_generic_and_combine<__half, false>(a, p, false);
    } else if (mod) {
        st = launch_generic_mod(a, p, dtype);
    } else {
        switch (dtype) {
        case PKV_BF16: st = launch_generic_and_combine<__nv_bfloat16, false>(a, p, true); break;
        case PKV_F16: st = launch_generic_and_combine<__half, false>(a, p, true); break;
        default: st = launch_generic_and_combine<float, false>(a, p, true); break;
        }
    }
    if (st != PKV_OK) return st;
    return ok();
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_paged_attention_decode(void *out, const void *q, const void *k_cache,
                                                 const void *v_cache, const int32_t *block_tables,
                                                 int32_t max_blocks_per_seq, const int32_t *context_lens,
                                                 int32_t num_seqs, int32_t num_q_heads,
                                                 int32_t num_kv_heads, int32_t head_dim,
                                                 int32_t block_size, int32_t num_blocks,
                                                 int32_t max_context_len, float scale, pkv_dtype dtype,
                                                 void *workspace, size_t workspace_bytes,
                                                 int32_t *err_flag, void *stream) {
    return decode_entry(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs,
                        num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, max_context_len, scale, dtype,
                        workspace, workspace_bytes, err_flag, stream, nullptr, nullptr);
}

extern "C" pkv_status pkv_paged_attention_decode_append(void *out, const void *q, const void *key,
                                                        const void *value, void *k_cache, void *v_cache,
                                                        const int32_t *block_tables, int32_t max_blocks_per_seq,
                                                        const int32_t *context_lens, int32_t num_seqs,
                                                        int32_t num_q_heads, int32_t num_kv_heads,
                                                        int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                                        int32_t max_context_len, float scale, pkv_dtype dtype,
                                                        void *workspace, size_t workspace_bytes,
                                                        int32_t *err_flag, void *stream) {
    if (num_seqs > 0 && (!key || !value))
        return set_error(PKV_ERR_INVALID_ARG, "decode append: NULL key or value");
    return decode_entry(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs,
                        num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, max_context_len, scale, dtype,
                        workspace, workspace_bytes, err_flag, stream, key, value);
}

extern "C" pkv_status pkv_paged_attention_decode_fp8(void *out, const void *q, const void *k_cache,
                                                     const void *v_cache, const float *k_scale, const float *v_scale,
                                                     const int32_t *block_tables, int32_t max_blocks_per_seq,
                                                     const int32_t *context_lens, int32_t num_seqs,
                                                     int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                                     int32_t block_size, int32_t num_blocks, int32_t max_context_len,
                                                     float scale, pkv_dtype dtype, void *workspace,
                                                     size_t workspace_bytes, int32_t *err_flag, void *stream) {
    if (num_seqs > 0 && (!k_scale || !v_scale))
        return set_error(PKV_ERR_INVALID_ARG, "decode fp8: NULL scales");
    if (dtype == PKV_F32) return set_error(PKV_ERR_UNSUPPORTED, "decode fp8: q/out must be fp16 or bf16");
    return decode_entry(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs,
                        num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, max_context_len, scale, dtype,
                        workspace, workspace_bytes, err_flag, stream, nullptr, nullptr, k_scale, v_scale, kCodeE4M3);
}

extern "C" pkv_status pkv_paged_attention_decode_int8(void *out, const void *q, const void *k_cache,
                                                      const void *v_cache, const float *k_scale, const float *v_scale,
                                                      const int32_t *block_tables, int32_t max_blocks_per_seq,
                                                      const int32_t *context_lens, int32_t num_seqs,
                                                      int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                                      int32_t block_size, int32_t num_blocks, int32_t max_context_len,
                                                      float scale, pkv_dtype dtype, void *workspace,
                                                      size_t workspace_bytes, int32_t *err_flag, void *stream) {
    if (num_seqs > 0 && (!k_scale || !v_scale))
        return set_error(PKV_ERR_INVALID_ARG, "decode int8: NULL scales");
    if (dtype == PKV_F32) return set_error(PKV_ERR_UNSUPPORTED, "decode int8: q/out must be fp16 or bf16");
    return decode_entry(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs,
                        num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, max_context_len, scale, dtype,
                        workspace, workspace_bytes, err_flag, stream, nullptr, nullptr, k_scale, v_scale, kCodeInt8);
}

// Decode attention with score rules over any cache format, with the step's new row
// appended first when key / value are given.
extern "C" pkv_status pkv_paged_attention_decode_mod(
    void *out, const void *q, const void *key, const void *value, void *k_cache, void *v_cache, const float *k_scale,
    const float *v_scale, pkv_cache_format format, const int32_t *block_tables, int32_t max_blocks_per_seq,
    const int32_t *context_lens, int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t block_size, int32_t num_blocks, int32_t max_context_len, float scale, const pkv_score_mod *mod,
    pkv_dtype dtype, void *workspace, size_t workspace_bytes, int32_t *err_flag, void *stream) {
    if (format != PKV_CACHE_DTYPE && format != PKV_CACHE_E4M3 && format != PKV_CACHE_INT8)
        return set_error(PKV_ERR_INVALID_ARG, "decode: unknown cache format %d", (int)format);
    const bool c8 = format != PKV_CACHE_DTYPE;
    if (num_seqs > 0 && (key == nullptr) != (value == nullptr))
        return set_error(PKV_ERR_INVALID_ARG, "decode: key and value go together");
    if (num_seqs > 0 && c8 && (!k_scale || !v_scale)) return set_error(PKV_ERR_INVALID_ARG, "decode: NULL scales");
    if (c8 && dtype == PKV_F32)
        return set_error(PKV_ERR_UNSUPPORTED, "decode: q/out over 8-bit caches must be fp16 or bf16");
    DecodeMod m;
    if (mod) {
        if (!(mod->softcap >= 0.f) || mod->softcap > 1e30f || (mod->softcap > 0.f && mod->softcap < 1e-30f))
            return set_error(PKV_ERR_INVALID_ARG, "decode: softcap must be 0, or from 1e-30 to 1e30");
        m.softcap = mod->softcap;
        m.slopes = mod->alibi_slopes;
        m.key_starts = mod->key_starts;
    }
    return decode_entry(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs,
                        num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, max_context_len, scale, dtype,
                        workspace, workspace_bytes, err_flag, stream, key, value, c8 ? k_scale : nullptr,
                        c8 ? v_scale : nullptr,
                        format == PKV_CACHE_E4M3 ? kCodeE4M3 : format == PKV_CACHE_INT8 ? kCodeInt8 : kCode16, &m);
}

// The fused decode step over 8-bit caches: key[b] / value[b] are encoded
// under the (block, head) scales already in k_scale / v_scale and written to
// the cache row of position context_lens[b] - 1 by the attention kernel's
// producer warp, then the attention runs over the whole context.
namespace pkv {
namespace {
pkv_status decode_append_q8(void *out, const void *q, const void *key, const void *value, void *k_cache,
                            void *v_cache, const float *k_scale, const float *v_scale, const int32_t *block_tables,
                            int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t num_seqs,
                            int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                            int32_t num_blocks, int32_t max_context_len, float scale, pkv_dtype dtype, void *workspace,
                            size_t workspace_bytes, int32_t *err_flag, void *stream, int32_t codes) {
    const char *fmt = codes == kCodeInt8 ? "int8" : "fp8";
    if (num_seqs > 0 && (!k_scale || !v_scale || !key || !value))
        return set_error(PKV_ERR_INVALID_ARG, "decode append %s: NULL key, value or scales", fmt);
    if (dtype == PKV_F32) return set_error(PKV_ERR_UNSUPPORTED, "decode append %s: q/out must be fp16 or bf16", fmt);
    return decode_entry(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs,
                        num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, max_context_len, scale, dtype,
                        workspace, workspace_bytes, err_flag, stream, key, value, k_scale, v_scale, codes);
}
}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_paged_attention_decode_append_fp8(
    void *out, const void *q, const void *key, const void *value, void *k_cache, void *v_cache, const float *k_scale,
    const float *v_scale, const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *context_lens,
    int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
    int32_t num_blocks, int32_t max_context_len, float scale, pkv_dtype dtype, void *workspace,
    size_t workspace_bytes, int32_t *err_flag, void *stream) {
    return decode_append_q8(out, q, key, value, k_cache, v_cache, k_scale, v_scale, block_tables, max_blocks_per_seq,
                            context_lens, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                            max_context_len, scale, dtype, workspace, workspace_bytes, err_flag, stream, kCodeE4M3);
}

extern "C" pkv_status pkv_paged_attention_decode_append_int8(
    void *out, const void *q, const void *key, const void *value, void *k_cache, void *v_cache, const float *k_scale,
    const float *v_scale, const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *context_lens,
    int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
    int32_t num_blocks, int32_t max_context_len, float scale, pkv_dtype dtype, void *workspace,
    size_t workspace_bytes, int32_t *err_flag, void *stream) {
    return decode_append_q8(out, q, key, value, k_cache, v_cache, k_scale, v_scale, block_tables, max_blocks_per_seq,
                            context_lens, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                            max_context_len, scale, dtype, workspace, workspace_bytes, err_flag, stream, kCodeInt8);
}

// ----------------------------------------------------------------------------- no-allocation variant
// Decode attention for callers that cannot allocate device memory where they
// run (an engine plugin that may only use memory it was handed, a service with
// a fixed budget reserved at start-up).  The split-K scratch lives in this
// fixed region instead of a caller workspace; every GPU that loads the library
// holds it until exit.  All calls share it: nothing in it must start at zero
// (each call writes every scratch value before reading it), and calls whose GPU
// work overlaps race on it.
static __device__ __align__(256) unsigned char g_pkv_static_workspace[PKV_STATIC_WORKSPACE_BYTES];

namespace pkv {
namespace {

// Device address of the region on the current device.  Host code cannot use
// the symbol itself (it names a host-side shadow), so the address is looked up
// with the device current, on every call: the lookup allocates nothing, and a
// fresh one stays right after a cudaDeviceReset reloads the module.
pkv_status static_workspace_address(void **addr) {
    void *p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_pkv_static_workspace);
    if (e != cudaSuccess || !p)
        return set_error(PKV_ERR_CUDA, "static workspace: cudaGetSymbolAddress: %s", cudaGetErrorString(e));
    *addr = p;
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_paged_attention_decode_static_ws(
    void *out, const void *q, const void *k_cache, const void *v_cache, const int32_t *block_tables,
    int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t num_seqs, int32_t num_q_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks, int32_t max_context_len,
    float scale, pkv_dtype dtype, int32_t *err_flag, void *stream) {
    // the same argument errors as the workspace variant, before the size check
    const pkv_status chk = check_decode_args(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                                             context_lens, num_seqs, num_q_heads, num_kv_heads, head_dim,
                                             block_size, num_blocks, max_context_len, dtype);
    if (chk != PKV_OK) return chk;
    const size_t need = pkv_paged_attention_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                                  block_size, max_context_len, dtype);
    if (need > PKV_STATIC_WORKSPACE_BYTES)
        return set_error(PKV_ERR_WORKSPACE,
                         "decode (static workspace): these sizes need %zu bytes of scratch, more than the "
                         "library's built-in %u bytes; call pkv_paged_attention_decode with a workspace",
                         need, (unsigned)PKV_STATIC_WORKSPACE_BYTES);
    void *ws = nullptr;
    if (need > 0) {
        pkv_status st = static_workspace_address(&ws);
        if (st != PKV_OK) return st;
    }
    return pkv_paged_attention_decode(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                                      num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                                      max_context_len, scale, dtype, ws, need > 0 ? PKV_STATIC_WORKSPACE_BYTES : 0,
                                      err_flag, stream);
}
