// Causal varlen / chunked prefill attention over the paged cache with score
// rules and over 8-bit and 4-bit caches.
//
// Query i of sequence b sits at position p = starts[b] + i.  Its score for key t
// (query head h reading KV head h / G) is
//     s = scale q . K_t,   s <- c tanh(s / c) (softcap c > 0),
//     s <- s - slope_h |p - t| (alibi slopes),
// over the visible keys  lo <= t < hi,  lo = key_starts[row] (0 without),
// hi = min(total, max(p + 1, prefix_lens[b])): one interval per row, so a document
// mask, a window and a prefix cost two comparisons, and only in the blocks that
// hold a boundary; blocks that no row of the CTA sees are never loaded.  Then the
// softmax and the sum over V_t; a row that sees nothing is zero.
//
// tanh(u), |u| <= 0.7 (35 of a cap of 50), is u times a polynomial of degree 4 in u^2,
// the minimax fit in relative error (linear programming on a Chebyshev grid): 3e-7, at
// seven packed FMA-unit operations a pair of scores.  Larger scores take c tanh(u) =
// c - 2 c / (1 + e^{2u}), one exponential and one reciprocal, off by a few 2^-23 c, in
// the 64-key steps of a warp that have one: two more trips through the special-function
// unit, which the softmax needs as well (8 prompts of 4k, cap 50: 1432 us with that
// alone, 1279 with the polynomial, at that step of the kernel).  Both errors are far
// below the rounding of P; the one-instruction tanh (relative 2^-11) is not.  A capped
// score is bounded, so over bf16 caches P = 2^s needs no reference maximum (kFreeCap).
//
// 8-bit caches: K_t = ks code, V_t = vs code, one scale per (block, KV head).  Both
// code formats are exact in f16, so K and V codes are widened to f16 tiles by
// converter warps and never rounded; ks multiplies the score, in f32.  P enters
// its product as f16(p vs), and the row's reference maximum follows s + log2 vs,
// which keeps p vs in f16's range whatever the scales; the row sum adds p itself.
// bf16 queries become f16 under a power of two per row (undone in the score's factor), so
// no bf16 magnitude overflows; elements from 2^-30 of their row's largest on are exact,
// smaller ones off by at most 2^-38 of it.
//
// 4-bit caches (pkv_int4.cuh): a scale per 32 dims of a row goes into the f16 tile with its
// codes, exactly (its eight significant bits and a code's three fit f16's eleven), so scores and
// P take no factor; P is rounded once and its row sum adds what was rounded, as over 16-bit caches.
// A lane of the converter warps takes a group: 16 bytes of codes, five operations for eight codes
// to f16 1024 + u, four to u - 8, four times the scale.
//
// The CTA.  Two tiles of 128 query rows (128 / G positions x G heads) of one KV
// head, accumulators in tensor memory: eight softmax warps hold one query row per
// thread, one producer warp copies pages by TMA, two warps issue the tcgen05.mma, one
// for each tile, and over 8-bit caches four widen codes.  K and V come in blocks of 128
// keys through one ring of 32 KB tiles in order K_0 V_0 K_1 V_1 ..; the work goes by
// half blocks of 64 keys.  Per tile and half block h: S_h = Q K_h^T, softmax, P_h (16
// bit, over S_h's columns), O += P_h V_h.  A tile has two S buffers of 64 columns and
// QK_{h+2} follows PV_h into the buffer that P_h leaves, so that S_{h+1} is there when
// the softmax of h ends and its warps never wait for the tensor core's round trip.
//
// What bounds it.  Plain scores, 8 prompts of 4k (32 heads, 8 KV heads): 908 us, 1093
// TFLOP/s.  A step of 64 keys of both tiles is 1240 clk of products alone: Q K^T at 64
// keys reads its operands from shared memory at 386 clk where the arithmetic takes 256
// (128 keys at once, one S buffer a tile, read less and ran 976 us: both tiles then sit
// in their softmax together).  With the copies into the ring the step is 1534, with the
// softmax warps beside it 1834.  Cap 50: 1049 us; the polynomial's operations come on
// top.  With a bias 1236.  E4M3 and int8: 1264 and 1297; widening writes every tile once
// more.  4-bit codes: 1231 (fp16, prompts of 3700 to 4096), where the 16-bit kernel over the
// same rows widened beforehand takes 988 with the widening.  Short spans: of a CTA's ~13k clk
// of setup, first products and output nothing overlaps, for both tiles do them together (2 x
// 8k rows of packed documents of 60 to 2500 rows: 150 us, 664 TFLOP/s).
//
// Few rows over a long context (a small chunk, few sequences) leave most SMs idle,
// so the blocks of a tile pair are cut into up to nsplit runs, one CTA each, whose
// (O, m, l) a second kernel joins (prefill_plan).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "pkv_int4.cuh"
#include "pkv_internal.h"
#include "pkv_mod.h"
#include "pkv_pack.cuh"
#include "pkv_pdl.cuh"
#include "pkv_tc.cuh"
#include "pkv_tma.cuh"

namespace pkv {
namespace {

constexpr int kModRows = 128;   // query rows per tile (MMA M, TMEM lanes)
constexpr int kModKeys = 128;   // keys per block
// Threads: eight softmax warps, a producer, an MMA warp per tile, and over 8-bit
// caches four converter warps.  384 threads have 168 registers each.  512 have 128,
// of which the service warps give up 40 so that the softmax warps get theirs:
// 256 x 168 + 256 x 88 = 512 x 128.
template <int FMT> constexpr bool kCoded = FMT != kCode16 && FMT != kCodeF16;
template <bool C8> constexpr int kModThreads = C8 ? 512 : 384;
constexpr int kModLaunchRegs = 128, kModSoftRegs = 168, kModServiceRegs = 88;  // 8-bit caches
static_assert(256 * (kModSoftRegs + kModServiceRegs) <= 512 * kModLaunchRegs, "the split draws on the launch's registers");
constexpr int kConvWarps = 4;
constexpr int kHalfKeys = kModKeys / 2;  // keys per step of the softmax and the products
constexpr int kModTile = 32768;       // a 128 x 128 tile of 16-bit values: two 64-column halves
constexpr int kModHalf = kModTile / 2;
constexpr int kModScales4 = kModKeys * 64;  // where a 4-bit code tile's scales begin, 8 bytes a key
constexpr uint64_t kModDeadlineNs = 2000000000ull;
constexpr float kModRescale = 8.f;    // log2 units a block may exceed the reference maximum by before O is rescaled
// CAP: no cap, a cap, or a cap that bounds the scores so far that no reference
// maximum is needed: P = 2^s itself, |s| <= kFreeCap, is in bf16's range with all its
// bits, and its sums times V are in f32's as long as keys x max |V| < 2^54 (at the other
// end, V below 2^-53 under P = 2^-73, products leave f32's normal range). Without the
// maximum and the rescaling 8 prompts of 4096 rows (32 heads, 8 KV heads, cap 50) take
// 1049 us; with both (f16, or a cap of 51) 1180.
enum { kNoCap = 0, kCap = 1, kCapBounded = 2 };
constexpr float kFreeCap = 73.f;
constexpr int kMaxGridPairs = 32768;  // grid.y
constexpr int kMinSplitBlocks = 2;    // blocks of a split at least

// Scores of a block of keys as every consumer needs them.
struct ModInfo {
    int32_t miss;  // bit g: the page of keys 16 g .. 16 g + 15 is out of range
    int32_t fix;   // some V rows of the block hold nothing valid and must read as zero (8-bit caches)
    int32_t neg;   // a K scale is negative or NaN
    int32_t pad;
    float ks[8], vs[8], lv[8];  // scales of each 16 keys, and log2 of the V scale (at least -100)
};
static_assert(sizeof(ModInfo) <= 128, "info slot");

// 4-bit code tiles are small enough for a fourth ring tile beside them (8 prompts of 3700 to 4096,
// fp16: 1231 us with two code tiles, 1251 with three, 1268 with three ring tiles and four).
template <int FMT>
struct ModLayout {
    static constexpr bool C8 = kCoded<FMT>, C4 = FMT == kCodeInt4;
    static constexpr int kRing = C8 && !C4 ? 3 : 4;      // 32 KB tiles
    static constexpr int kStage = C4 ? 2 : C8 ? 4 : 0;   // code tiles
    static constexpr int kCodeTile = C4 ? kModScales4 + kModKeys * 8 : 16384;
    static constexpr int kQ = 0;
    static constexpr int kRingOff = 2 * kModTile;
    static constexpr int kStageOff = kRingOff + kRing * kModTile;
    static constexpr int kInfoOff = kStageOff + kStage * kCodeTile;
    static constexpr int kRangeOff = kInfoOff + 4 * 128;
    static constexpr int kBarOff = kRangeOff + 64;
    static constexpr int kTmemSlot = kBarOff + 320;
    static constexpr int kBytes = kTmemSlot + 16;
    static constexpr int kAlloc = kBytes + 1024;
    static_assert(kAlloc <= 227 * 1024, "shared memory per CTA");
    // mbarriers
    static constexpr int kFull = 0;                     // [kRing] tile landed (copy bytes) or widened (every converter warp)
    static constexpr int kEmpty = kFull + kRing;        // [kRing] MMA commits: each query tile is done with it
    static constexpr int kStFull = kEmpty + kRing;      // [kStage] codes landed
    static constexpr int kStEmpty = kStFull + kStage;   // [kStage] codes read by every converter warp
    static constexpr int kInfo = kStEmpty + kStage;     // [4] the block's ModInfo is written
    static constexpr int kVLand = kInfo + 4;            // 16-bit: a V tile landed that the producer goes over first
    static constexpr int kSFull = kVLand + 1;           // [2][2] S of a tile's buffer ready, and every earlier MMA done
    static constexpr int kPFull = kSFull + 4;           // [2][2] P written by the tile's four warps
    static constexpr int kQFull = kPFull + 4;           // [2] Q rows written
    static constexpr int kOPrev = kQFull + 2;           // [2] the tile's last PV but one is done
    static constexpr int kOLast = kOPrev + 2;           // [2] the tile's last PV is done
    static constexpr int kFinal = kOLast + 2;           // every MMA of the CTA is done
    static constexpr int kNumBars = kFinal + 1;
    static_assert(kNumBars * 8 <= 320, "mbarriers");
};

struct ModArgs {
    void *out;
    const void *q;
    const int32_t *block_tables, *starts, *cu_q;
    const float *k_scale, *v_scale;
    const uint8_t *codes[2];    // 4-bit caches: K, V
    const uint16_t *scales[2];
    const float *slopes;
    const int32_t *key_starts, *prefix_lens;
    int32_t max_blocks, Hq, Hkv, lg_g, bs, num_blocks, box_lg, max_q_len, pairs, nsplit;
    int32_t pair_grids;  // grids of kMaxGridPairs items that hold pairs * nsplit
    float sl;     // scale log2 e: raw score -> log2 units
    float sa;     // softcap: raw score -> scale / c
    float su;     // softcap: raw score -> 2 log2 e scale / c
    float tanh_poly[5];  // softcap in log2 units times the fit's coefficients
    float capl2;  // softcap in log2 units
    float *o_part;
    float2 *ml_part;
    int32_t *split_used;  // [B * pairs]
    int32_t *err_flag;
};

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t (&x)[4]) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(addr)
                 : "memory");
}

template <typename T, int FMT, int CAP, bool ALIBI>
__global__ void __launch_bounds__(kModThreads<kCoded<FMT>>, 1)
prefill_mod_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ ModArgs A) {
    constexpr bool C8 = kCoded<FMT>;        // codes, which converter warps widen
    constexpr bool C4 = FMT == kCodeInt4;  // with their scales, row by row
    constexpr bool BS = C8 && !C4;         // a scale per block, kept out of the tiles
    constexpr bool HQ = FMT != kCode16;    // f16 products, whatever the queries' type
    constexpr bool RQ = HQ && !BS;         // the queries' power of two is the scores' only factor
    constexpr bool RAW = !CAP && !ALIBI;  // the score's factor goes into the exponent's FMA
    using L = ModLayout<FMT>;
    using M16 = typename std::conditional<HQ, __half, T>::type;  // operand type of the products
    using H = Half16<M16>;
    constexpr bool kBf16 = std::is_same<M16, __nv_bfloat16>::value;
    constexpr bool kFree = CAP == kCapBounded;
    static_assert(!kFree || (kBf16 && !ALIBI), "P = 2^s needs bf16's range and bounded scores");
    constexpr int kRing = L::kRing;
    // CTAs start in grid order: every KV head's last pair of a sequence first, the shortest pairs
    // last, so that the launch's end is short (heads slower than pairs: 8 prompts
    // of 4k, cap 50, 1049 us against 1037, packed documents 155 against 150)
    const int kh = blockIdx.x, b = A.pair_grids == 1 ? blockIdx.z : blockIdx.z / A.pair_grids;
    const int item = (blockIdx.z - b * A.pair_grids) * kMaxGridPairs + blockIdx.y;
    if (item >= A.pairs * A.nsplit) return;
    const int pair = A.nsplit == 1 ? item : item / A.nsplit, split = item - pair * A.nsplit;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lg_g = A.lg_g, G = 1 << lg_g, Hq = A.Hq, bs = A.bs;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // [0, 1]: the lowest key that a row of the CTA sees, the highest + 1.  [2, 3]: the sequence's
    // first row and row count, which the epilogue reads again: kept in registers over the loop
    // they cost its warps more (E4M3 chunks 547 us against 541).
    volatile int32_t *cta = reinterpret_cast<volatile int32_t *>(smem + L::kRangeOff);
    int raw0 = 0, raw1 = 0;  // producer: table entries of the first two blocks
    auto info = [&](int jj) { return reinterpret_cast<ModInfo *>(smem + L::kInfoOff + (jj & 3) * 128); };
    const uint32_t bar0 = smem_u32(smem + L::kBarOff);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    const uint32_t sQ = smem_u32(smem + L::kQ), sRing = smem_u32(smem + L::kRingOff);
    const uint32_t sStage = smem_u32(smem + L::kStageOff);
    if (warp == 8 && lane == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(bar(L::kFull + i), C8 ? kConvWarps : 1);
        }
        for (int i = 0; i < L::kStage; ++i) {
            mbar_init(bar(L::kStFull + i), 1);
            mbar_init(bar(L::kStEmpty + i), kConvWarps);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(L::kInfo + i), 1);
            mbar_init(bar(L::kSFull + i), 1);
            mbar_init(bar(L::kPFull + i), 4);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(L::kQFull + t), 4);
            mbar_init(bar(L::kOPrev + t), 1);
            mbar_init(bar(L::kOLast + t), 1);
        }
        mbar_init(bar(L::kVLand), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if constexpr (!C4) {
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
        }
    }
    pdl_wait();
    pdl_trigger();
    const int q_begin = A.cu_q[b], n = A.cu_q[b + 1] - q_begin, start = A.starts[b];
    const bool first = pair == 0 && split == 0 && kh == 0;  // the CTA that reports the sequence's errors
    if (n <= 0 || n > A.max_q_len) {  // nothing to do, or not what was declared: the rows stay as they are
        if (n != 0 && first && threadIdx.x == 0 && A.err_flag) atomicOr(A.err_flag, PKV_ERRBIT_CONTEXT);
        return;
    }
    const int positions = kModRows >> lg_g;
    const int tile0 = ((n + positions - 1) >> (7 - lg_g)) - 1 - 2 * pair;  // the CTA's tiles: tile0, tile0 - 1
    if (tile0 < 0) return;
    const int64_t total64 = static_cast<int64_t>(start) + n;
    T *out = static_cast<T *>(A.out);
    if (start < 0 || total64 > static_cast<int64_t>(A.max_blocks) * bs || total64 > INT32_MAX - 4 * kModKeys) {
        if (split != 0) return;  // a bad span: zero rows and a flag
        if (first && threadIdx.x == 0 && A.err_flag) atomicOr(A.err_flag, PKV_ERRBIT_CONTEXT);
        if (A.nsplit > 1 && kh == 0 && threadIdx.x == 0) A.split_used[static_cast<int64_t>(b) * A.pairs + pair] = 1;
        const int p0 = max(tile0 - 1, 0) * positions, p1 = min(n, (tile0 + 1) * positions);
        for (int i = threadIdx.x; i < (p1 - p0) * G * kFastHeadDim; i += kModThreads<C8>) {
            const int pi = i / (G * kFastHeadDim), rem = i - pi * G * kFastHeadDim;
            out[(static_cast<int64_t>(q_begin + p0 + pi) * Hq + kh * G) * kFastHeadDim + rem] = from_f32<T>(0.f);
        }
        return;
    }
    const int total = static_cast<int>(total64);
    // From here on every path goes to the common exit (the CTA holds TMEM).
    const int ntiles = tile0 > 0 ? 2 : 1;
    if (warp == 8 && lane == 0) {  // barriers that count tiles
        for (int i = 0; i < kRing; ++i) mbar_init(bar(L::kEmpty + i), ntiles);
        mbar_init(bar(L::kFinal), ntiles);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) tmem_alloc(smem_u32(smem + L::kTmemSlot), 512);

    // Softmax threads: tile t = warp / 4, query row r of it: position r / G, head r % G.
    const int t = warp >> 2;  // 2 and more: service warps
    const int r = threadIdx.x & (kModRows - 1);
    const int q0 = (tile0 - t) * positions;
    const int pi = r >> lg_g;
    const int64_t tile_row = (static_cast<int64_t>(q_begin) + q0) * Hq + kh * G;  // the tile's first q / out row
    bool live = false;
    int pos = 0;  // the row's position
    // The warp's 32 Q rows, two rows of 16 chunks at a time (zeros past the sequence).  Over
    // 16-bit caches they are in flight over the barrier; the 8-bit kernels have no registers for
    // that before their split.  Row and head of r0 + 2 i are those of r0 plus those of 2 i (their
    // bits are apart), so what depends on i is uniform: a CTA's first instructions are fetched
    // anew, and cost more than they do.
    uint4 qv[16];
    auto load_q = [&] {
        const int r0 = (warp & 3) * 32 + (lane >> 4), pr = r0 >> lg_g;
        const uint4 *src = static_cast<const uint4 *>(A.q) + (tile_row + pr * Hq + (r0 & (G - 1))) * 16 + (lane & 15);
        const int left = t < ntiles ? n - q0 - pr : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int up = (2 * i) >> lg_g;
            qv[i] = up < left ? __ldg(src + (up * Hq + ((2 * i) & (G - 1))) * 16) : make_uint4(0, 0, 0, 0);
        }
    };
    // The sequence's table entry for this lane's 16 keys of block j (0: none).  Only a chunk of
    // 2^box_lg keys (all of one page) that reaches the CTA's keys [lo, hi) is looked up: pages that
    // nobody sees may be missing.
    const int32_t *table = A.block_tables + static_cast<int64_t>(b) * A.max_blocks;
    auto owned = [&](int j, int lo, int hi) {
        const int box = 1 << A.box_lg, last = (j * kModKeys + 16 * lane) | (box - 1);
        return lane < 8 && last >= lo && last - box < hi - 1;
    };
    auto entry = [&](int j, int lo, int hi) -> int {  // hi <= total: key / bs < ceil(total / bs) <= max_blocks
        return owned(j, lo, hi) ? table[(j * kModKeys + 16 * lane) / bs] : 0;
    };
    if (t < 2) {
        if constexpr (!C8) load_q();
        live = t < ntiles && q0 + pi < n;
        pos = start + q0 + pi;
    } else if (warp == 8) {
        // What the first copy waits for is a chain of loads (offsets, key starts, table entries):
        // the producer goes through it alone, beside the loads of Q, which take longer.  (Key
        // starts by every row, behind its Q, and the table entries behind the barrier: the first
        // S 1800 clk later, 8 prompts of 4k, cap 50, 1071 us against 1052, packed documents 163
        // against 156.)
        const int prefix = A.prefix_lens ? A.prefix_lens[b] : 0;
        const int p0 = (tile0 - ntiles + 1) * positions, p1 = min(n, (tile0 + 1) * positions);
        int key_lo = 0, key_hi = min(total, max(start + p1, prefix));
        if (A.key_starts) {
            int lo = INT32_MAX, hi = 0;
#pragma unroll
            for (int i = 0; i < 2 * kModRows / 32; ++i) {
                const int p = p0 + 32 * i + lane;
                const int from = p < p1 ? max(A.key_starts[q_begin + p], 0) : INT32_MAX;
                const int to = min(total, max(start + p + 1, prefix));
                if (from < to) {
                    lo = min(lo, from);
                    hi = max(hi, to);
                }
            }
            key_hi = __reduce_max_sync(0xffffffffu, hi);
            key_lo = key_hi > 0 ? __reduce_min_sync(0xffffffffu, lo) : 0;  // 0 where no row sees a key
        }
        if (lane == 0) {
            cta[0] = key_lo;
            cta[1] = key_hi;
            cta[2] = q_begin;
            cta[3] = n;
        }
        raw0 = entry(key_lo / kModKeys, key_lo, key_hi);
        raw1 = entry(key_lo / kModKeys + 1, key_lo, key_hi);
    }
    tc_fence_before();
    __syncthreads();  // the barriers, the range and the TMEM address are there
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::kTmemSlot);
    // Half blocks [h0, h1) that a row of the CTA sees any key of, cut to this split.  Both
    // tiles go through all of them: their ranges differ by a few halves at most, and every
    // barrier then passes through the same phases for everybody.
    const int key_lo = cta[0], key_hi = cta[1];
    int h0 = key_hi > 0 ? key_lo / kHalfKeys : 0, h1 = key_hi > 0 ? (key_hi - 1) / kHalfKeys + 1 : 0;
    bool partial = false;
    if (A.nsplit > 1) {
        const int j0 = h0 >> 1, blocks = ((h1 + 1) >> 1) - j0;
        const int per = max((blocks + A.nsplit - 1) / A.nsplit, kMinSplitBlocks);
        const int used = blocks > 0 ? (blocks + per - 1) / per : 1;
        if (split == 0 && kh == 0 && threadIdx.x == 0) A.split_used[static_cast<int64_t>(b) * A.pairs + pair] = used;
        partial = used > 1;
        if (split >= used) live = false;
        const int s0 = 2 * (j0 + split * per), s1 = s0 + 2 * per;
        h0 = min(max(h0, s0), h1);
        h1 = max(min(h1, s1), h0);
    }
    const int j0 = h0 >> 1, j1 = (h1 + 1) >> 1;  // the blocks to load
    const int nb = h1 > h0 ? j1 - j0 : 0;
    const uint64_t deadline = global_ns() + kModDeadlineNs;
    bool timed_out = false;

    if (warp >= 8) {
        if constexpr (C8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kModServiceRegs));
        if (warp == 8) {
            // ------------------------------------------------------------ producer warp
            // Lane g < 8 owns keys 16 g .. 16 g + 15 of the block; the first lane of each
            // chunk of 2^box_lg keys (consecutive in one page) copies it.  Table entries are
            // loaded two blocks ahead and scales one, so that no copy waits for them.
            const int box_rows = 1 << A.box_lg;
            bool bad = false;
            // a page id, -1 where nobody sees a key, -2 out of range
            auto page = [&](int j, int raw) -> int {
                if (!owned(j, key_lo, key_hi)) return -1;
                if (raw >= 0 && raw < A.num_blocks) return raw;
                bad = true;
                return -2;
            };
            auto scale_of = [&](const float *scales, int page_id) -> float {
                if constexpr (!BS) return 1.f;
                return page_id >= 0 ? __ldg(scales + static_cast<int64_t>(page_id) * A.Hkv + kh) : 1.f;
            };
            auto wait_bar = [&](int i, uint32_t parity) -> bool {
                int ok = 1;
                if (lane == 0) ok = mbar_wait(bar(i), parity, deadline);
                return __shfl_sync(0xffffffffu, ok, 0) != 0;
            };
            constexpr int kSlots = C8 ? L::kStage : kRing;
            constexpr int kSlotBytes = C8 ? L::kCodeTile : kModTile;
            constexpr int kSlotFull = C8 ? L::kStFull : L::kFull, kSlotEmpty = C8 ? L::kStEmpty : L::kEmpty;
            const uint32_t sDst = C8 ? sStage : sRing;
            int issued = 0;
            int fix_jj = -1;  // a block whose V rows are still to be zeroed
            unsigned fix_miss = 0;
            uint32_t lands = 0;  // blocks that went through kVLand
            // V rows that no row of the CTA sees (in front of the lowest key, from the highest
            // on: later tokens, past the sequence) or of a missing page read as zero (0 x NaN
            // would stay): such a tile lands on a barrier of its own, and its full barrier is
            // arrived on when the rows are zero.
            auto zero_v = [&]() -> bool {
                if (!wait_bar(L::kVLand, lands & 1)) return false;
                ++lands;
                __syncwarp();
                const int slot = (2 * fix_jj + 1) % kRing;
                const uint32_t vt = sRing + static_cast<uint32_t>(slot) * kModTile;
                for (int i = lane; i < kModKeys * 16; i += 32) {
                    const int rr = i >> 4, c = i & 15, key = (j0 + fix_jj) * kModKeys + rr;
                    if (key < key_lo || key >= key_hi || (fix_miss >> (rr >> 4) & 1))
                        st_shared_v4(vt + (c >> 3) * kModHalf + rr * 128 + (c & 7) * 16, 0, 0, 0, 0);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::kFull + slot));
                fix_jj = -1;
                return true;
            };
            int id = -1, next_raw = 0;
            float ks = 1.f, vs = 1.f;
            if (nb > 0) {
                if (split != 0) {  // the first split starts at the lowest key's block
                    raw0 = entry(j0, key_lo, key_hi);
                    raw1 = entry(j0 + 1, key_lo, key_hi);
                }
                id = page(j0, raw0);
                next_raw = raw1;
                ks = scale_of(A.k_scale, id);
                vs = scale_of(A.v_scale, id);
            }
            for (int jj = 0; jj < nb && !timed_out; ++jj) {
                const int key = (j0 + jj) * kModKeys + 16 * lane;
                const unsigned miss = __ballot_sync(0xffffffffu, id == -2);
                const unsigned neg = __ballot_sync(0xffffffffu, BS && id >= 0 && !(ks >= 0.f));
                const unsigned chunks = __ballot_sync(0xffffffffu, id >= 0 && (key & (box_rows - 1)) == 0);
                const uint32_t chunk_bytes = static_cast<uint32_t>(box_rows) * (C4 ? 72 : C8 ? 128 : 256);
                const bool mine = (chunks >> lane) & 1;
                const int slot_row = mine ? id * bs + key % bs : 0;
                int next_id = -1;
                float next_ks = 1.f, next_vs = 1.f;
                const bool fix = miss || (j0 + jj) * kModKeys < key_lo || (j0 + jj + 1) * kModKeys > key_hi;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const int item = 2 * jj + kv, slot = item % kSlots;
                    if (item >= kSlots && !wait_bar(kSlotEmpty + slot, ((item / kSlots) - 1) & 1)) {
                        timed_out = true;
                        break;
                    }
                    if (kv == 0) {
                        // The slot of info jj held block jj - 4, whose readers are done: the wait
                        // above was for MMAs (or conversions) that come after its softmax.
                        ModInfo *f = info(jj);
                        if (lane == 0) {
                            f->miss = static_cast<int32_t>(miss);
                            f->fix = fix;
                            f->neg = neg != 0;
                        }
                        if (BS && lane < 8) {
                            f->ks[lane] = ks;
                            f->vs[lane] = vs;
                            f->lv[lane] = fmaxf(__log2f(vs), -100.f);  // also a scale of 0
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(L::kInfo + (jj & 3)));
                    }
                    const uint32_t landed = bar(!C8 && kv == 1 && fix ? L::kVLand : kSlotFull + slot);
                    if (lane == 0) mbar_arrive_expect_tx(landed, __popc(chunks) * chunk_bytes);
                    __syncwarp();
                    if (mine) {
                        const CUtensorMap *tm = kv ? &tm_v : &tm_k;
                        const uint32_t dst = sDst + static_cast<uint32_t>(slot) * kSlotBytes + (16 * lane) * (C4 ? 64 : 128);
                        if constexpr (C4) {
                            const int64_t row = (static_cast<int64_t>(id) * A.Hkv + kh) * bs + key % bs;
                            bulk_load(dst, A.codes[kv] + row * 64, box_rows * 64, landed);
                            bulk_load(sDst + static_cast<uint32_t>(slot) * kSlotBytes + kModScales4 + 16 * lane * 8,
                                      A.scales[kv] + row * 4, box_rows * 8, landed);
                        } else if constexpr (C8) {
                            tma_load_3d(dst, tm, 0, slot_row, kh, landed);
                        } else {
                            tma_load_3d(dst, tm, 0, slot_row, 2 * kh, landed);
                            tma_load_3d(dst + kModHalf, tm, 0, slot_row, 2 * kh + 1, landed);
                        }
                    }
                    issued = item + 1;
                    if (kv == 0 && jj + 1 < nb) {
                        next_id = page(j0 + jj + 1, next_raw);
                        next_ks = scale_of(A.k_scale, next_id);
                        next_vs = scale_of(A.v_scale, next_id);
                        next_raw = entry(j0 + jj + 2, key_lo, key_hi);
                    }
                    if (!C8 && kv == 0 && fix_jj >= 0 && !zero_v()) {
                        timed_out = true;
                        break;
                    }
                }
                if (!C8 && fix && issued == 2 * jj + 2) {
                    fix_jj = jj;
                    fix_miss = miss;
                }
                id = next_id;
                ks = next_ks;
                vs = next_vs;
            }
            if (!C8 && fix_jj >= 0 && !zero_v()) timed_out = true;  // on the way out of a broken pipeline too: the copy must land
            bad = __any_sync(0xffffffffu, bad);
            if (lane == 0) {
                if (bad && A.err_flag) atomicOr(A.err_flag, PKV_ERRBIT_BLOCK_RANGE);
                // no bulk copy may still be writing shared memory when the CTA exits
                for (int i = max(issued - kSlots, 0); i < issued; ++i)
                    if (!mbar_wait(bar(kSlotFull + i % kSlots), (i / kSlots) & 1, deadline)) timed_out = true;
            }
        } else if (warp < 11) {
            // ------------------------------------------------------------ MMA warps
            // One per tile that exists.  The tensor core's queue is short: what an issuer does
            // between two products (waits, descriptors) is lost unless another issuer's products
            // run meanwhile (64 keys of both tiles, products alone: 1240 clk; one issuer 1700).
            // The loop's values are made warp-uniform first: operands in per-thread registers
            // took longer to move than the product to run.
            auto uni = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
            const int uh0 = uni(h0), uh1 = uni(h1), uj0 = uh0 >> 1, uitems = uni(2 * nb);
            const uint32_t utmem = static_cast<uint32_t>(uni(static_cast<int>(tmem)));
            const uint32_t ubar = static_cast<uint32_t>(uni(static_cast<int>(bar0)));
            auto mbar = [&](int i) { return ubar + 8u * static_cast<uint32_t>(i); };
            const uint32_t ring16 = static_cast<uint32_t>(uni(static_cast<int>(sRing))) >> 4;
            const uint32_t q16 = static_cast<uint32_t>(uni(static_cast<int>(sQ))) >> 4;
            const int tt = uni(warp) - 9;
            const uint32_t tc = utmem + tt * 256;
            if (tt < uni(ntiles) && elect_one()) {
                constexpr uint32_t kIdescS = umma_idesc_f16(kBf16, kModRows, kHalfKeys, false);
                constexpr uint32_t kIdescO = umma_idesc_f16(kBf16, kModRows, kFastHeadDim, true);
                const uint64_t kmajor = umma_desc_sw128(0, 16, 1024), vmajor = umma_desc_sw128(0, kModHalf, 1024);
                // Operations of one thread run in order: a QK may be issued right behind the PV
                // that reads P from the columns it writes, and a commit stands for everything
                // before it.  Step h issues PV_h and QK_{h+2} (the first two steps no PV); the
                // tiles release a K tile with the QKs of its second half, a V tile with the PVs
                // of its second half, where the producer fills the slot again.  One copy of the
                // code, as short as it gets: its warp shares the instruction cache with the
                // softmax warps.
                bool ok = true;
#pragma unroll 1
                for (int h = uh0 - 2; ok && h < uh1; ++h) {
                    const bool second = h & 1;  // second half of its block
                    const int vitem = 2 * ((h >> 1) - uj0) + 1, kitem = vitem + 1;  // V of h, K of h + 2
                    const int vslot = vitem % kRing, vuse = vitem / kRing, kslot = kitem % kRing, kuse = kitem / kRing;
                    if (h >= uh0) {
                        // O += P_h V_h
                        if (!second || h == uh0) ok = mbar_wait(mbar(L::kFull + vslot), vuse & 1, deadline);
                        ok = ok && mbar_wait(mbar(L::kPFull + 2 * tt + (h & 1)), ((h - uh0) >> 1) & 1, deadline);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t vd = vmajor + (ring16 + (vslot * kModTile + (h & 1) * (kHalfKeys * 128)) / 16);
                        const uint32_t pc = tc + (h & 1) * kHalfKeys;
                        umma_f16_tmem_a(tc + 128, pc, vd, kIdescO, h > uh0 ? 1u : 0u);
#pragma unroll
                        for (int k = 1; k < kHalfKeys / 16; ++k)  // 16 keys per step: 8 P columns, two 8-row V groups
                            umma_f16_tmem_a(tc + 128, pc + 8 * k, vd + k * 128, kIdescO, 1u);
                        if (h == uh1 - 2) umma_commit(mbar(L::kOPrev + tt));
                        if (h == uh1 - 1) umma_commit(mbar(L::kOLast + tt));
                        if (second && vitem + kRing < uitems) umma_commit(mbar(L::kEmpty + vslot));
                    }
                    if (h + 2 < uh1) {
                        // S_{h+2} = Q K_{h+2}^T
                        if (h + 2 == uh0) ok = mbar_wait(mbar(L::kQFull + tt), 0, deadline);
                        if (ok && (!second || h + 2 == uh0)) ok = mbar_wait(mbar(L::kFull + kslot), kuse & 1, deadline);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t kd = kmajor + (ring16 + (kslot * kModTile + (h & 1) * (kHalfKeys * 128)) / 16);
                        const uint64_t qd = kmajor + (q16 + tt * kModTile / 16);
                        const uint32_t sc = tc + (h & 1) * kHalfKeys;
#pragma unroll
                        for (int k = 0; k < kFastHeadDim / 16; ++k) {  // 16 dims (32 bytes) per step
                            const uint32_t off = ((k >> 2) * kModHalf + (k & 3) * 32) / 16;
                            umma_f16(sc, qd + off, kd + off, kIdescS, k > 0);
                        }
                        umma_commit(mbar(L::kSFull + 2 * tt + (h & 1)));
                        if (second && kitem + kRing < uitems) umma_commit(mbar(L::kEmpty + kslot));
                    }
                }
                if (!ok) timed_out = true;
                umma_commit(mbar(L::kFinal));  // arrives once every MMA of this thread has completed
                if (!mbar_wait(mbar(L::kFinal), 0, deadline)) timed_out = true;
            }
            __syncwarp();
        } else if constexpr (C8) {
            // ------------------------------------------------------------ converter warps
            // Warp w widens rows 32 w .. 32 w + 31 of every code tile.  A lane takes 16 codes
            // (one 16-byte chunk) and writes two chunks; lanes 4 .. 7 of each eight take the
            // row four below and write their second chunk first, so that neither the reads
            // nor the writes (both 128-byte swizzled) meet a bank twice.
            const int w = warp - 11;
            const int l8 = lane & 7, hi = l8 >> 2;
            const int row0 = 32 * w + (lane >> 3) + 4 * hi;
            for (int item = 0; item < 2 * nb && w < kConvWarps; ++item) {
                const int st = item % L::kStage, slot = item % kRing;
                bool ok = mbar_wait(bar(L::kStFull + st), (item / L::kStage) & 1, deadline) &&
                          (item < kRing || mbar_wait(bar(L::kEmpty + slot), ((item / kRing) - 1) & 1, deadline));
                if (!__all_sync(0xffffffffu, ok)) {
                    timed_out = true;
                    break;
                }
                const ModInfo *f = info(item >> 1);
                const bool fix = (item & 1) && f->fix;
                const int miss = f->miss, key0 = (j0 + (item >> 1)) * kModKeys;
                const uint32_t src = sStage + static_cast<uint32_t>(st) * L::kCodeTile;
                const uint32_t dst = sRing + static_cast<uint32_t>(slot) * kModTile;
                if constexpr (C4) {
                    // A lane takes a group: 16 bytes of codes, one scale, four chunks of eight
                    // dims.  Eight lanes are two rows of four groups (their reads are 128
                    // consecutive bytes), and groups 2 and 3 write their chunks in the order 2 3 0 1,
                    // so that the eight writes of a step are in eight different places.
                    const int c = lane & 3, flip = c & 2;
                    const uint32_t d0 = dst + (c >> 1) * kModHalf;
#pragma unroll 2
                    for (int i = 0; i < 4; ++i) {
                        const int rr = 32 * w + 8 * i + (lane >> 2);
                        uint32_t x[4], s;
                        ld_shared_v4(src + rr * 64 + c * 16, x);
                        asm volatile("{\n\t.reg .b16 h;\n\tld.shared.b16 h, [%1];\n\tmov.b32 %0, {h, h};\n\t}"
                                     : "=r"(s)
                                     : "r"(src + kModScales4 + rr * 8 + c * 2)
                                     : "memory");
                        bool none = false;
                        if (fix) {
                            const int key = key0 + rr;
                            none = key < key_lo || key >= key_hi || (miss >> (rr >> 4) & 1);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t y[4];
                            int4_widen(flip ? x[e ^ 2] : x[e], y);
#pragma unroll
                            for (int k = 0; k < 4; ++k) y[k] = none ? 0u : mul_f16x2(y[k], s);
                            st_shared_v4(d0 + rr * 128 + (((4 * (c & 1) + (e ^ flip)) ^ (rr & 7)) << 4), y[0], y[1], y[2], y[3]);
                        }
                    }
                } else {
#pragma unroll 2  // more (4: -6 % with int8) costs the other warps their instruction cache
                    for (int i = 0; i < 8; ++i) {
                        const int rr = row0 + 8 * (i >> 1), c4 = l8 & 3;
                        const int c = c4 + 4 * (i & 1);
                        uint32_t x[4];
                        ld_shared_v4(src + rr * 128 + ((c ^ (rr & 7)) << 4), x);
                        uint32_t y[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) codes4_to_f16x4<FMT, false>(x[e], y[2 * e], y[2 * e + 1]);
                        if (fix) {
                            const int key = key0 + rr;
                            if (key < key_lo || key >= key_hi || (miss >> (rr >> 4) & 1)) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) y[e] = 0;
                            }
                        }
                        const uint32_t d = dst + (i & 1) * kModHalf + rr * 128;
                        const uint32_t d0 = d + (((2 * c4 + hi) ^ (rr & 7)) << 4), d1 = d + (((2 * c4 + (hi ^ 1)) ^ (rr & 7)) << 4);
                        st_shared_v4(d0, hi ? y[4] : y[0], hi ? y[5] : y[1], hi ? y[6] : y[2], hi ? y[7] : y[3]);
                        st_shared_v4(d1, hi ? y[0] : y[4], hi ? y[1] : y[5], hi ? y[2] : y[6], hi ? y[3] : y[7]);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(L::kStEmpty + st));
                    mbar_arrive(bar(L::kFull + slot));
                }
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax warps
        if constexpr (C8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kModSoftRegs));
        const bool on = t < ntiles && h0 < h1;  // the tile exists and sees a key
        const int hd = r & (G - 1);
        // The row's visible keys [lo_r, hi_r).  A row that is not written must not make its warp mask.
        int lo_r = 0, hi_r = INT32_MAX;
        if (live) {
            lo_r = A.key_starts ? max(A.key_starts[q_begin + q0 + pi], 0) : 0;
            hi_r = min(total, max(pos + 1, A.prefix_lens ? A.prefix_lens[b] : 0));
            if (lo_r >= hi_r) lo_r = hi_r = 0;
        }
        float rq = 1.f;  // HQ: what the row's scores are multiplied by, a power of two
        if (on) {
            const uint32_t sQt = sQ + static_cast<uint32_t>(t) * kModTile;
            if constexpr (C8) load_q();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int rr = (warp & 3) * 32 + 2 * i + (lane >> 4), c = lane & 15;
                st_shared_v4(sQt + (c >> 3) * kModHalf + rr * 128 + (((c & 7) ^ (rr & 7)) << 4), qv[i].x, qv[i].y, qv[i].z, qv[i].w);
            }
            if constexpr (HQ && std::is_same<T, __nv_bfloat16>::value) {
                // bf16 becomes f16 with the row's largest value moved to [2^13, 2^14), a row per
                // thread in place (rolled loops: unrolled over the loads above they cost every CTA
                // more in instruction fetches than they save)
                __syncwarp();
                const uint32_t mine = sQt + r * 128;
                auto chunk = [&](int i) { return mine + (i >> 3) * kModHalf + (((i & 7) ^ (r & 7)) << 4); };
                uint32_t top = 0;
#pragma unroll 4
                for (int i = 0; i < 16; ++i) {
                    uint32_t x[4];
                    ld_shared_v4(chunk(i), x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = max(top, max((x[e] & 0x7fffu) << 16, x[e] & 0x7fff0000u));
                }
                const int e = static_cast<int>(top >> 23);  // biased exponent of the largest value
                const int k = top == 0 || e == 255 ? 0 : min(max(13 - (e - 127), -120), 120);
                const float f = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
                rq = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll 4
                for (int i = 0; i < 16; ++i) {
                    uint32_t x[4];
                    ld_shared_v4(chunk(i), x);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[e] = H::pack(__uint_as_float(x[e] << 16) * f, __uint_as_float(x[e] & 0xffff0000u) * f);
                    st_shared_v4(chunk(i), x[0], x[1], x[2], x[3]);
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kQFull + t));
        }
        // The scores' factor f of this row where rq is all of it: finite, so that a score of 0 stays 0.
        auto by_row = [&](float f) {
            const float v = f * rq;
            return fabsf(v) > 3e38f ? copysignf(3e38f, v) : v;
        };
        // RAW: not 0 either, since it meets masked scores, which are -inf
        const float raw_sl = RQ ? fmaxf(by_row(A.sl), 1.17549435e-38f) : A.sl;
        const float nslope = ALIBI && A.slopes && live ? -A.slopes[kh * G + hd] * 1.4426950408889634f : 0.f;
        // this warp's TMEM lanes (32 (warp % 4) ..) in the tile's columns: S / P at 0 and 64, O at 128
        const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + t * 256;
        float m_ref = kFree ? 0.f : -INFINITY, l_sum = 0.f;
        for (int h = h0; on && h < h1; ++h) {
            const int jj = (h >> 1) - j0, g0 = (h & 1) * 4;  // the half's first group of 16 keys
            const uint32_t scol = trow + (h & 1) * kHalfKeys;
            bool ok = mbar_wait(bar(L::kInfo + (jj & 3)), (jj >> 2) & 1, deadline) &&
                      mbar_wait(bar(L::kSFull + 2 * t + (h & 1)), ((h - h0) >> 1) & 1, deadline);
            if (!__all_sync(0xffffffffu, ok)) {
                timed_out = true;
                break;
            }
            tc_fence_after();
            // Keys a <= k < z of the half are visible to this row, but for missing pages.
            const int a = lo_r - h * kHalfKeys, z = hi_r - h * kHalfKeys;
            // A warp that sees none of them (the other tile's keys, rows past the sequence) is
            // done: P = 0.  Packed documents 162 us against 169; the capped and the 8-bit kernels
            // lose 2 % by the longer loop (1071 us to 1097, 547 to 560) and go without.
            if (!CAP && !C8 && __all_sync(0xffffffffu, !live || a >= kHalfKeys || z <= 0)) {
                const uint32_t none[32] = {};
                tmem_st32(scol, none);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::kPFull + 2 * t + (h & 1)));
                continue;
            }
            const ModInfo *f = info(jj);
            float x[kHalfKeys];
            {
                uint32_t v[64];
                tmem_ld64(scol, v);
#pragma unroll
                for (int i = 0; i < 64; ++i) x[i] = __uint_as_float(v[i]);
            }
            const int miss = f->miss >> g0 & 15;
            const bool open = __all_sync(0xffffffffu, a <= 0 && z >= kHalfKeys && miss == 0);
            // 1. scores in log2 units (RAW: left as they are, factor `mul` below)
            bool scaled = !RAW;  // whether x holds final scores
            if constexpr (CAP) {
                uint64_t c[5];
#pragma unroll
                for (int i = 0; i < 5; ++i) c[i] = splat2(A.tanh_poly[i]);
                float top = 0.f;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const uint64_t sa = splat2(BS ? A.sa * f->ks[g0 + g] * rq : RQ ? by_row(A.sa) : A.sa);
#pragma unroll
                    for (int k = 16 * g; k < 16 * g + 16; k += 2) {
                        const uint64_t u = mul2(pack2(x[k], x[k + 1]), sa), u2 = mul2(u, u);
                        float z0, z1;
                        unpack2(u2, z0, z1);
                        top = max3f(top, z0, z1);
                        unpack2(mul2(u, fma2(u2, fma2(u2, fma2(u2, fma2(u2, c[4], c[3]), c[2]), c[1]), c[0])), x[k], x[k + 1]);
                    }
                }
                if (!__all_sync(0xffffffffu, top <= kTanhLimit * kTanhLimit)) {  // S is still there: once more for the large ones
#pragma unroll
                    for (int c0 = 0; c0 < kHalfKeys; c0 += 32) {
                        uint32_t v[32];
                        tmem_ld32(scol + c0, v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float su = BS ? A.su * f->ks[g0 + (c0 + i) / 16] * rq : RQ ? by_row(A.su) : A.su;
                            const float e = __uint_as_float(v[i]) * su;  // 2 log2 e score / cap
                            const float big = fmaf(fast_rcp(1.f + fast_exp2(e)), -2.f * A.capl2, A.capl2);
                            // each score by its own size: a row's bits are its own
                            x[c0 + i] = fabsf(e) > kTanhLimit * 2.8853900817779268f ? big : x[c0 + i];
                        }
                    }
                }
            }
            if constexpr (ALIBI) {
                // bias nslope |k - c|, c the row's own key in the half's coordinates
                const float c = static_cast<float>(pos - h * kHalfKeys);
                // On one side of every row's own key the bias is linear: by (c - k).  The seldom
                // half with keys on both sides is corrected afterwards: |c - k| in a branch of its own
                // lengthened the loop (8 prompts of 4k 1330 us against 1235).
                const bool past = __all_sync(0xffffffffu, pos - h * kHalfKeys >= kHalfKeys - 1);
                const bool ahead = __all_sync(0xffffffffu, pos - h * kHalfKeys <= 0);
                const float by = ahead ? -nslope : nslope;
                const uint64_t on = splat2(-2.f * by);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const uint64_t sl = splat2(CAP ? 1.f : BS ? A.sl * f->ks[g0 + g] * rq : RQ ? by_row(A.sl) : A.sl);
                    uint64_t bias = pack2(by * (c - 16 * g), by * (c - 16 * g - 1));  // two keys on by one addition
#pragma unroll
                    for (int k = 16 * g; k < 16 * g + 16; k += 2) {
                        const uint64_t s = pack2(x[k], x[k + 1]);
                        unpack2(CAP ? add2(s, bias) : fma2(s, sl, bias), x[k], x[k + 1]);
                        bias = add2(bias, on);
                    }
                }
                if (!past && !ahead) {  // keys behind the row's own: from nslope (c - k) to nslope (k - c)
#pragma unroll
                    for (int k = 0; k < kHalfKeys; ++k) x[k] = fmaf(fmaxf(k - c, 0.f), 2.f * nslope, x[k]);
                }
            }
            // 2. masked keys
            if constexpr (RAW && BS) {
                if (!open || f->neg) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float s = A.sl * f->ks[g0 + g] * rq;
#pragma unroll
                        for (int k = 16 * g; k < 16 * g + 16; ++k) x[k] *= s;
                    }
                    scaled = true;
                }
            }
            if (!open) {  // one boundary at a time: seldom more than one of them is in a warp's half
                if (__any_sync(0xffffffffu, z < kHalfKeys)) {
#pragma unroll
                    for (int k = 0; k < kHalfKeys; ++k) x[k] = k < z ? x[k] : -INFINITY;
                }
                if (__any_sync(0xffffffffu, a > 0)) {
#pragma unroll
                    for (int k = 0; k < kHalfKeys; ++k) x[k] = k >= a ? x[k] : -INFINITY;
                }
                if (miss) {
#pragma unroll
                    for (int k = 0; k < kHalfKeys; ++k) x[k] = miss >> (k >> 4) & 1 ? -INFINITY : x[k];
                }
            }
            // 3. the half's maximum, of s + log2 vs for 8-bit caches
            float mx, resc = 1.f;
            bool moved = false;
            if constexpr (kFree) {
                mx = 0.f;
            } else if constexpr (BS) {
                mx = -INFINITY;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float m = max3f(x[16 * g], x[16 * g + 1], x[16 * g + 2]);
#pragma unroll
                    for (int k = 16 * g + 3; k < 16 * g + 15; k += 2) m = max3f(m, x[k], x[k + 1]);
                    m = fmaxf(m, x[16 * g + 15]);
                    if (RAW && !scaled) m *= A.sl * f->ks[g0 + g] * rq;
                    mx = fmaxf(mx, m + f->lv[g0 + g]);
                }
            } else {
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // four independent chains
#pragma unroll
                for (int k = 0; k < kHalfKeys; k += 2) m4[(k >> 1) & 3] = max3f(m4[(k >> 1) & 3], x[k], x[k + 1]);
                mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                if (RAW) mx *= raw_sl;
            }
            if (!kFree && mx > m_ref + kModRescale) {  // also the row's first visible key (m_ref = -inf)
                if (m_ref != -INFINITY) {
                    resc = fast_exp2(m_ref - mx);
                    moved = true;
                }
                m_ref = mx;
            }
            // O moves with the reference, once the PV before this half's is done: the next S
            // stands for it, or its own barrier in the tile's last half.  (A row has no
            // reference to move in the tile's first half.)
            if (!kFree && __any_sync(0xffffffffu, moved)) {  // TMEM access is warp-wide; a factor of 1 leaves a row as it is
                ok = h + 1 < h1 ? mbar_wait(bar(L::kSFull + 2 * t + ((h + 1) & 1)), ((h + 1 - h0) >> 1) & 1, deadline)
                                  : mbar_wait(bar(L::kOPrev + t), 0, deadline);
                if (!__all_sync(0xffffffffu, ok)) {
                    timed_out = true;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int c0 = 0; c0 < kFastHeadDim; c0 += 32) {
                    uint32_t v[32];
                    tmem_ld32(trow + 128 + c0, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * resc);
                    tmem_st32(trow + 128 + c0, v);
                }
            }
            // 4. P = 2^(s - m) over the S columns it came from
            const uint64_t nb2 = splat2(m_ref == -INFINITY ? 0.f : -m_ref);
            float s4[4] = {0.f, 0.f, 0.f, 0.f};
            uint64_t l2[2] = {0, 0};
            uint32_t pk[32];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint64_t mul = splat2(RAW ? (BS ? (scaled ? 1.f : A.sl * f->ks[g0 + g] * rq) : raw_sl) : 1.f);
                const uint64_t sv = splat2(BS ? f->vs[g0 + g] : 1.f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int k = 16 * g + 2 * i, o = 8 * g + i;
                    float e0, e1;
                    const uint64_t s = pack2(x[k], x[k + 1]);
                    unpack2(RAW ? fma2(s, mul, nb2) : kFree ? s : add2(s, nb2), e0, e1);
                    e0 = fast_exp2(e0);
                    e1 = fast_exp2(e1);
                    if constexpr (BS) {
                        const uint64_t p = pack2(e0, e1);
                        l2[i & 1] = add2(l2[i & 1], p);
                        unpack2(mul2(p, sv), e0, e1);
                        pk[o] = H::pack(e0, e1);
                    } else {
                        pk[o] = H::pack(e0, e1);
                        pair_acc<M16>(pk[o], s4[i & 1], s4[2 + (i & 1)]);  // the rounded P: weights sum to 1
                    }
                }
            }
            tmem_st32(scol, pk);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kPFull + 2 * t + (h & 1)));
            if constexpr (BS) unpack2(add2(l2[0], l2[1]), s4[0], s4[1]);
            l_sum = l_sum * resc + ((s4[0] + s4[1]) + (s4[2] + s4[3]));
        }
        // Epilogue: O row / row sum, or the split's share of both.
        bool ok = !timed_out && (!on || mbar_wait(bar(L::kOLast + t), 0, deadline));
        if (!__all_sync(0xffffffffu, ok)) {
            timed_out = true;
        } else if (__any_sync(0xffffffffu, live)) {
            tc_fence_after();
            const int q_begin = cta[2], n = cta[3];
            const int q0 = (((n + positions - 1) >> (7 - lg_g)) - 1 - 2 * pair - t) * positions, pi = r >> lg_g, hd = r & (G - 1);
            const int64_t tile_row = (static_cast<int64_t>(q_begin) + q0) * Hq + kh * G;
            const float inv = l_sum > 0.f ? 1.f / l_sum : (l_sum == l_sum ? 0.f : l_sum);
            const int64_t prow = ((static_cast<int64_t>(b) * A.max_q_len + q0 + pi) * Hq + kh * G + hd) * A.nsplit + split;
            if (partial && live) A.ml_part[prow] = make_float2(m_ref, l_sum);
            float *po = A.o_part + prow * kFastHeadDim;
            // 16-bit rows go through the tile's Q rows in shared memory (its last QK is done),
            // so that they leave as whole lines.
            const uint32_t sOt = sQ + static_cast<uint32_t>(t) * kModTile;
#pragma unroll 1
            for (int c0 = 0; c0 < kFastHeadDim; c0 += 32) {
                uint32_t v[32];
                if (on) {
                    tmem_ld32(trow + 128 + c0, v);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0;
                }
                if (partial) {
                    if (live) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4 *>(po + c0 + 4 * i) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = Half16<T>::pack(__uint_as_float(v[8 * i + 2 * e]) * inv, __uint_as_float(v[8 * i + 2 * e + 1]) * inv);
                        const int c = c0 / 8 + i;
                        st_shared_v4(sOt + (c >> 3) * kModHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
                    }
                }
            }
            if (!partial) {
                __syncwarp();
                const int c = lane & 15;
                uint4 *dst = static_cast<uint4 *>(A.out) + tile_row * 16 + c;
#pragma unroll 4
                for (int i = 0; i < 16; ++i) {
                    const int rr = (warp & 3) * 32 + 2 * i + (lane >> 4), pr = rr >> lg_g;
                    if (q0 + pr >= n) continue;
                    uint32_t o[4];
                    ld_shared_v4(sOt + (c >> 3) * kModHalf + rr * 128 + (((c & 7) ^ (rr & 7)) << 4), o);
                    dst[(pr * Hq + (rr & (G - 1))) * 16] = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
    }
    // Common exit: copies landed (producer), MMAs completed (MMA warp), TMEM reads done.
    if (timed_out && A.err_flag) atomicOr(A.err_flag, PKV_ERRBIT_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, 512);
}

// Joins the splits of a row: out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s.
// One warp per (sequence, query, head), lanes over the dims.  Splits without a
// visible key carry m = -inf and l = 0, and their O is not read.
constexpr int kModMergeThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kModMergeThreads)
prefill_mod_merge_kernel(const __grid_constant__ ModArgs A, int64_t rows) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kModMergeThreads / 32) + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int h = static_cast<int>(row % A.Hq);
    const int64_t bi = row / A.Hq;
    const int b = static_cast<int>(bi / A.max_q_len), i = static_cast<int>(bi - static_cast<int64_t>(b) * A.max_q_len);
    const int q_begin = A.cu_q[b], n = A.cu_q[b + 1] - q_begin;
    if (i >= n || n > A.max_q_len) return;
    const int lg_p = 7 - A.lg_g;  // log2 of the positions of a tile
    const int pair = (((n + (1 << lg_p) - 1) >> lg_p) - 1 - (i >> lg_p)) >> 1;
    const int used = min(A.split_used[static_cast<int64_t>(b) * A.pairs + pair], A.nsplit);
    if (used <= 1) return;  // written by the main kernel
    const float2 *ml = A.ml_part + row * A.nsplit;
    float M = -INFINITY;
    for (int s = 0; s < used; ++s) M = fmaxf(M, ml[s].x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int s = 0; s < used; ++s) {
        const float2 v = ml[s];
        if (v.x == -INFINITY && v.y == 0.f) continue;  // (scores that are all NaN leave the maximum there, and a NaN sum)
        const float w = exp2f(v.x - M);
        const float4 o = __ldg(reinterpret_cast<const float4 *>(A.o_part + (row * A.nsplit + s) * kFastHeadDim) + lane);
        acc.x = fmaf(w, o.x, acc.x);
        acc.y = fmaf(w, o.y, acc.y);
        acc.z = fmaf(w, o.z, acc.z);
        acc.w = fmaf(w, o.w, acc.w);
        l = fmaf(w, v.y, l);
    }
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    uint2 o;
    o.x = Half16<T>::pack(acc.x * inv, acc.y * inv);
    o.y = Half16<T>::pack(acc.z * inv, acc.w * inv);
    *(reinterpret_cast<uint2 *>(static_cast<T *>(A.out) + ((static_cast<int64_t>(q_begin) + i) * A.Hq + h) * kFastHeadDim) + lane) = o;
}

// ----------------------------------------------------------------------------- host side
// The shared-memory attribute and a check of the build, once per (kernel, device):
// with fewer registers than its split draws on, an 8-bit kernel would wait for ever.
template <typename T, int FMT, int CAP, bool ALIBI>
pkv_status prefill_mod_configure() {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (e == cudaSuccess && (done.load(std::memory_order_acquire) & bit)) return PKV_OK;
    auto kern = prefill_mod_kernel<T, FMT, CAP, ALIBI>;
    cudaFuncAttributes attr;
    if (kCoded<FMT> && e == cudaSuccess) e = cudaFuncGetAttributes(&attr, kern);
    if (kCoded<FMT> && e == cudaSuccess && attr.numRegs < kModLaunchRegs)
        return set_error(PKV_ERR_CUDA, "prefill: the kernel was built with %d registers, not %d", attr.numRegs, kModLaunchRegs);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ModLayout<FMT>::kAlloc);
    if (e != cudaSuccess) return set_error(PKV_ERR_CUDA, "prefill: kernel attributes: %s", cudaGetErrorString(e));
    done.fetch_or(bit, std::memory_order_acq_rel);
    return PKV_OK;
}

template <typename T, int FMT, int CAP, bool ALIBI>
pkv_status prefill_mod_launch(const PrefillCall &c) {
    int box_rows = kModKeys;  // chunk: gcd(block_size, 128) keys, consecutive in a page
    while (c.block_size % box_rows) box_rows >>= 1;
    CUtensorMap mk, mv;
    const int64_t slots = static_cast<int64_t>(c.num_blocks) * c.block_size;
    pkv_status st;
    if constexpr (FMT == kCodeInt4) {
        mk = mv = CUtensorMap{};  // its copies are whole runs of a (block, head)
        st = PKV_OK;
    } else if constexpr (kCoded<FMT>) {
        st = make_kv_map_8bit(&mk, c.k_cache, slots, c.Hkv, box_rows, 1);
        if (st == PKV_OK) st = make_kv_map_8bit(&mv, c.v_cache, slots, c.Hkv, box_rows, 1);
    } else {
        using M16 = typename std::conditional<FMT == kCodeF16, __half, T>::type;
        st = make_kv_map_box(&mk, c.k_cache, Half16<M16>::kTmaType, slots, c.Hkv, box_rows, 1);
        if (st == PKV_OK) st = make_kv_map_box(&mv, c.v_cache, Half16<M16>::kTmaType, slots, c.Hkv, box_rows, 1);
    }
    if (st == PKV_OK) st = prefill_mod_configure<T, FMT, CAP, ALIBI>();
    if (st != PKV_OK) return st;
    const float log2e = 1.4426950408889634f;
    ModArgs a{};
    a.out = c.out;
    a.q = c.q;
    a.block_tables = c.block_tables;
    a.starts = c.starts;
    a.cu_q = c.cu_q;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    a.codes[0] = static_cast<const uint8_t *>(c.k_cache);
    a.codes[1] = static_cast<const uint8_t *>(c.v_cache);
    a.scales[0] = c.k_scale4;
    a.scales[1] = c.v_scale4;
    a.slopes = c.mod.alibi_slopes;
    a.key_starts = c.mod.key_starts;
    a.prefix_lens = c.mod.prefix_lens;
    a.max_blocks = c.max_blocks;
    a.Hq = c.Hq;
    a.Hkv = c.Hkv;
    a.lg_g = __builtin_ctz(c.Hq / c.Hkv);  // 1, 2, 4 or 8
    a.bs = c.block_size;
    a.num_blocks = c.num_blocks;
    a.box_lg = __builtin_ctz(box_rows);
    a.max_q_len = c.max_q_len;
    a.pairs = c.plan.pairs;
    a.nsplit = c.plan.nsplit;
    a.sl = c.scale * log2e;
    a.sa = CAP ? c.scale / c.mod.softcap : 0.f;
    for (int i = 0; i < 5; ++i) a.tanh_poly[i] = static_cast<float>(kTanhFit[i] * c.mod.softcap * 1.4426950408889634);
    a.su = CAP ? 2.f * log2e * c.scale / c.mod.softcap : 0.f;
    a.capl2 = CAP ? c.mod.softcap * log2e : 0.f;
    a.o_part = reinterpret_cast<float *>(c.workspace);
    a.ml_part = reinterpret_cast<float2 *>(c.workspace + c.plan.o_bytes);
    a.split_used = reinterpret_cast<int32_t *>(c.workspace + c.plan.o_bytes + c.plan.ml_bytes);
    a.err_flag = c.err_flag;
    const int items = a.pairs * a.nsplit;
    a.pair_grids = (items + kMaxGridPairs - 1) / kMaxGridPairs;
    cudaError_t e = launch_pdl(kPdlDecode, prefill_mod_kernel<T, FMT, CAP, ALIBI>,
                               dim3(c.Hkv, items < kMaxGridPairs ? items : kMaxGridPairs, c.num_seqs * a.pair_grids), dim3(kModThreads<kCoded<FMT>>),
                               ModLayout<FMT>::kAlloc, c.stream, mk, mv, a);
    if (e == cudaSuccess && a.nsplit > 1) {
        const int64_t rows = static_cast<int64_t>(c.num_seqs) * c.max_q_len * c.Hq;
        constexpr int kRows = kModMergeThreads / 32;
        e = launch_pdl(kPdlCombine, prefill_mod_merge_kernel<T>, dim3(static_cast<unsigned>((rows + kRows - 1) / kRows)),
                       dim3(kModMergeThreads), 0, c.stream, a, rows);
    }
    if (e != cudaSuccess) return set_error(PKV_ERR_CUDA, "prefill launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}

template <int FMT>
pkv_status prefill_mod_format(const PrefillCall &c) {
    const bool cap = c.mod.softcap > 0.f;
    // Without a cap or a bias the score's factor goes into the exponent, which
    // wants it positive; other scales take the bias kernel with a bias of 0.
    const bool bias = c.mod.alibi_slopes || (!cap && !(c.scale > 1e-30f));
#define PKV_MOD(T) \
    (cap ? (bias ? prefill_mod_launch<T, FMT, kCap, true>(c) : prefill_mod_launch<T, FMT, kCap, false>(c)) \
         : (bias ? prefill_mod_launch<T, FMT, kNoCap, true>(c) : prefill_mod_launch<T, FMT, kNoCap, false>(c)))
    if constexpr (FMT == kCode16)
        if (c.dtype == PKV_BF16 && cap && !bias && c.mod.softcap * 1.4426950408889634f <= kFreeCap)
            return prefill_mod_launch<__nv_bfloat16, FMT, kCapBounded, false>(c);
    if constexpr (FMT == kCodeF16) return PKV_MOD(__nv_bfloat16);  // f16 queries over f16 pools are kCode16
    else return c.dtype == PKV_BF16 ? PKV_MOD(__nv_bfloat16) : PKV_MOD(__half);
#undef PKV_MOD
}

}  // namespace
}  // namespace pkv
