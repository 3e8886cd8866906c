// Decode attention over the 4-bit paged cache (pkv_int4.cuh has the format).
//
// With codes c and scales s of 32-dim groups g, per query head
//     S_t = scale sum_g ks_{t,g} (q_g . kc_{t,g}),   out = sum_t p_t vs_{t,g} vc_t / sum_t p_t,
// p the softmax of S (after the score rules), kept as a running maximum, sum and accumulator.
//
// A KV head of a token is 144 bytes of K and V at head_dim 128 where 16 bits take 512, so the
// arithmetic that a byte feeds is 3.6 times that of the 16-bit kernel and the kernel is built
// to keep it small:
//   * K enters the products as it unpacks: a nibble in the low byte of a half is the f16 number
//     u 2^-24, or 16 u 2^-24 (under q / 16), exactly.  Five operations for eight codes; the 8 that a code
//     is too large by is a constant per query and group, the accumulator's start.  (As 1024 + u, which
//     costs the same, the start is 128 times larger and the score as much less exact.)
//   * A group's scale multiplies its partial score in f32 (two products of 16 dims each).
//   * V codes are widened exactly to u - 8.  A group's scale goes into P: p rounded to f16, times
//     the scale, rounded again, each by 2^-12 of it at most on average, which is what the rounding
//     of an fp16 output amounts to.  (The scales on V are exact, but 64 more half-pair products
//     for 32 tokens: 64 sequences of up to 4096 tokens 132 us against 123, 8 x 32768 61.7 against
//     59.4, when this was chosen.)
//   * f16 has its bits above 2^-14 only, and a key far below the largest score may be one of many:
//     P stands as high as the scales of V let it (kI4Slack), so that small values keep their weights
//     (11 binades more than with the largest P at 1; 3 % of the time: 125 to 128 us, 57.9 to 59.5).
//   * The transposed fragments of V come from ldmatrix.trans on 16-bit units: four dims of a
//     token each, two tokens in a register, which is the pair the product wants.
//   * The offset of V could be taken out by a further product, 8 times the weights' sum, as for K: fewer
//     operations, but no faster (8 x 32768 59.5 us both ways, more registers), and the rounding of p
//     then counts for 8 of every code.
//
// A warp works alone: it takes its own slice of the launch's (unit, step of 64 tokens) list, a unit
// being a (sequence, KV head, up to 8 of its query heads), copies its steps by cp.async into tiles
// of its own (K of the next step while P V of this one runs, V while Q K does) and never meets
// another warp.  The list is cut evenly, whatever the mix of lengths; a unit that several warps
// share leaves a piece (max, sum, accumulator) each, which a second kernel joins.
//
// Measured with heads of 128 dims, on the GPU: 8 x 32768 tokens, 32 heads over 8 KV heads, 59.5 us, 5.1 TB/s;
// 64 sequences of up to 4096 tokens, 32 heads each with its own K and V, 126 us, 4.2 TB/s; 4 of up to 500,
// 16 heads over 8, 8.3 us, its launch and one chain of loads.
// Long contexts are bound by the issue of what a byte feeds, 544 warp instructions for 32 tokens of a KV
// head at 0.6 a clock and scheduler, 43 % of them on the integer pipe; the copies alone would keep HBM
// busy.  Three warps a scheduler at 168 registers: 16 warps of 128 spill (8 x 32768 67 us, when that was
// tried), steps of 32 tokens pay the rescaling and the table look-ups twice.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "pkv_int4.cuh"
#include "pkv_internal.h"
#include "pkv_pack.cuh"
#include "pkv_pdl.cuh"
#include "pkv_tma.cuh"

namespace pkv {
namespace {

constexpr int kI4MaxSeqs = 512;      // sequences of a launch (shared-memory prefix)
constexpr int kI4MaxWarps = 152 * 16;  // working warps of a launch (sizes the workspace)
constexpr int kI4Heads = 8;          // query heads of a unit
// Few units (one wave) of short contexts: a CTA each, its warps meeting in shared memory, in one
// launch without a workspace.  Against slices and the join, 32 heads over 8 KV heads, bf16, on the
// GPU: 1 sequence of 500 tokens 8.3 us / 10.3, 16 of up to 1000 10.3 / 14.4, 36 of up to 1000 14.4 /
// 16.5; 4 of up to 2000, where more SMs help, 15.6 / 12.4.
constexpr int kI4DirectCtas = 3, kI4DirectLen = 1024;  // CTAs an SM (2 at head_dim 256)
constexpr float kI4Log2e = 1.4426950408889634f;
constexpr float kI4Unit = 5.9604644775390625e-8f;  // 2^-24, f16's smallest
// P, and P times a V scale, stay below 2^15, and as near to it as they can, since f16 has few bits
// below 2^-14: P is 2^room at the score of its reference, and may pass that by kI4Slack binades.
constexpr float kI4Slack = 4.f;
constexpr int kI4TopExp = 14;  // exponent field of f16 scales below 1, the least that lowers room
__device__ __forceinline__ uint32_t i4_top_scale(int exp) { return static_cast<uint32_t>((exp << 10) + 1023) * 0x10001u; }
__device__ __forceinline__ int i4_exp(uint32_t scale) { return static_cast<int>(scale >> 10 & 63); }  // (a sign would count as a large one)
__device__ __forceinline__ float i4_room(int top_exp) { return 29.f - kI4Slack - static_cast<float>(top_exp); }  // scales below 2^(top_exp - 14)

struct I4Args {
    void *out;
    const void *q;
    const uint8_t *k_cache, *v_cache;
    const __half *k_scale, *v_scale;
    const int32_t *block_tables, *context_lens, *key_starts;
    const float *slopes;
    int32_t max_blocks, B, Hq, Hkv, G, subs, bs, num_blocks, max_ctx;
    float scale_log2, softcap;
    int32_t rows;      // query heads of a unit, at most
    float *o_piece;    // [slots][rows][D], slot warp + unit
    float2 *ml_piece;  // [slots][rows]
    int2 *unit_info;   // [units]: first and last warp
    int32_t *err_flag;
};

__device__ __forceinline__ int64_t i4_div(int64_t a, int64_t b) {  // a >= 0, b > 0
    if (((a | b) >> 32) == 0) return static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
    return a / b;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 16 bytes from global to shared memory.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// N consecutive 32-bit words of shared memory.
template <int N> __device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&x)[N]) {
    if constexpr (N == 1) {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x[0]) : "r"(addr));
    } else if constexpr (N == 2) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(addr));
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3])
                         : "r"(addr + 4 * i));
    }
}

// d = a b + c, the columns of c alike in both rows.
__device__ __forceinline__ void mma_start(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0, float c1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %10, %11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

// A warp's shared memory: K codes and scales of a step, V's, and queries.  K of the next step is
// copied while P V runs, V while Q K does, a unit's queries with the step before its first.
template <int D, int STEP> struct I4Tile {
    static constexpr int NG = D / 32;  // groups, and 16-byte chunks of a row
    static constexpr int kCodes = STEP * D / 2;
    static constexpr int kHalf = kCodes + STEP * NG * 2;
    static constexpr int kQ = kI4Heads * D * 2;  // a unit's queries, of two units
    static constexpr int kWarp = 2 * kHalf + 2 * kQ;
};

template <typename T, int D, int STEP, int WARPS, int CTAS, bool MOD, bool DIRECT>
__global__ void __launch_bounds__(WARPS * 32, CTAS)
decode_int4_kernel(const __grid_constant__ I4Args A) {
    using R = I4Tile<D, STEP>;
    using H = Half16<__half>;
    constexpr int NG = R::NG, TILES = STEP / 16;  // tiles of 16 tokens, each inside one block
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int B = A.B, bs = A.bs;
    // Context length (0: nothing visible) and first visible key of sequence b.
    auto first_of = [&](int b) -> int { return MOD && A.key_starts ? max(__ldg(A.key_starts + b), 0) : 0; };
    auto context_of = [&](int b, int first) -> int {
        const int ctx = __ldg(A.context_lens + b);
        return ctx > first && ctx <= A.max_ctx && static_cast<int64_t>(ctx) <= static_cast<int64_t>(A.max_blocks) * bs ? ctx : 0;
    };
    auto steps_of = [&](int b) -> int {
        const int first = first_of(b), ctx = context_of(b, first);
        return ctx > 0 ? (ctx + STEP - 1) / STEP - first / STEP : 0;
    };
    const int HU = A.Hkv * A.subs;  // units of a sequence
    struct Cursor { int b, hu, st, n; };  // step st of the n of unit hu of sequence b
    Cursor cur;
    int64_t me = 0;
    int count = 0;  // steps of this warp's slice
    if constexpr (DIRECT) {
        // The CTA's one unit: its warps take every WARPS-th step.
        cur.b = static_cast<int>(blockIdx.x / HU);
        cur.hu = static_cast<int>(blockIdx.x) - cur.b * HU;
        cur.st = warp;
        cur.n = steps_of(cur.b);
        count = cur.n > warp ? (cur.n - 1 - warp) / WARPS + 1 : 0;
        if (cur.n == 0 && threadIdx.x == 0) {
            const int ctx = A.context_lens[cur.b];
            if ((ctx < 0 || ctx > A.max_ctx || static_cast<int64_t>(ctx) > static_cast<int64_t>(A.max_blocks) * bs) && A.err_flag)
                atomicOr(A.err_flag, PKV_ERRBIT_CONTEXT);
        }
    } else {
        // The prefix of steps over the sequences (of one unit each), in what holds the tiles later.
        int64_t *pref = reinterpret_cast<int64_t *>(smem);  // [B + 1]
        int32_t *ns = reinterpret_cast<int32_t *>(pref + kI4MaxSeqs + 1);
        for (int b = threadIdx.x; b < B; b += WARPS * 32) {
            const int n = steps_of(b);
            ns[b] = n;
            if (n == 0 && b % gridDim.x == blockIdx.x) {  // a row of zeros
                const int ctx = A.context_lens[b];
                if ((ctx < 0 || ctx > A.max_ctx || static_cast<int64_t>(ctx) > static_cast<int64_t>(A.max_blocks) * bs) && A.err_flag)
                    atomicOr(A.err_flag, PKV_ERRBIT_CONTEXT);
                uint4 *o = reinterpret_cast<uint4 *>(static_cast<T *>(A.out) + static_cast<int64_t>(b) * A.Hq * D);
                for (int i = 0; i < A.Hq * D / 8; ++i) o[i] = make_uint4(0, 0, 0, 0);
            }
        }
        __syncthreads();
        if (warp == 0) {
            const int chunk = (B + 31) / 32, lo = min(lane * chunk, B), hi = min(lo + chunk, B);
            int64_t sum = 0;
            for (int b = lo; b < hi; ++b) sum += ns[b];
            int64_t incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            int64_t run = incl - sum;
            for (int b = lo; b < hi; ++b) {
                pref[b] = run;
                run += ns[b];
            }
            if (lane == 31) pref[B] = incl;
        }
        __syncthreads();
        const int64_t W = pref[B] * HU;
        const int64_t all = static_cast<int64_t>(gridDim.x) * WARPS;
        const int64_t Cw = W > all ? all : W < 1 ? 1 : W;  // working warps, a step each at least
        // neighbouring slices go to different SMs, so that a launch of few slices uses them all
        me = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
        if (me < Cw && W > 0) {
            const int64_t s0 = i4_div(W * me, Cw), s1 = i4_div(W * (me + 1), Cw);
            count = static_cast<int>(s1 - s0);
            int lo = 0, hi = B - 1;  // the largest b with HU pref[b] <= s0
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (pref[mid] * HU <= s0) lo = mid; else hi = mid - 1;
            }
            const int64_t off = s0 - pref[lo] * HU;
            cur.b = lo;
            cur.n = ns[lo];
            cur.hu = static_cast<int>(i4_div(off, cur.n));
            cur.st = static_cast<int>(off - static_cast<int64_t>(cur.hu) * cur.n);
        }
        __syncthreads();  // the prefix has been read: the tiles may be filled
    }
    if (!DIRECT && count == 0) return;
    constexpr int kStride = DIRECT ? WARPS : 1;  // steps from one of the warp's to the next
    auto next_unit = [&](Cursor &c) {  // the first step of the next unit (b == B: there is none)
        c.st = 0;
        if (++c.hu == HU) {
            c.hu = 0;
            do {
                ++c.b;
                c.n = c.b < B ? steps_of(c.b) : 1;
            } while (c.n == 0);
        }
    };

    // ---- copies.  Lanes 0 .. TILES - 1 keep the table column and the row of their tile and load
    // its entry a step ahead; of a tile's codes every lane takes the same chunk of rows r, r +
    // 32 / NG, .., so that all addresses but the tile's first row are constants of the lane.
    const uint32_t k_tile = smem_u32(smem) + static_cast<uint32_t>(warp) * R::kWarp, v_tile = k_tile + R::kHalf;
    const uint32_t q_tile = k_tile + 2 * R::kHalf;
    constexpr int kRowsPer = 32 / NG;        // rows that one copy instruction covers
    constexpr int kCopies = 16 / kRowsPer;   // of a tile
    constexpr int kChunks = 2 * NG;          // 16-byte chunks of a tile's scales
    constexpr int kScaleTiles = 32 / kChunks < TILES ? 32 / kChunks : TILES;  // tiles whose scales one instruction copies
    static_assert(kRowsPer <= 16 && kChunks <= 32, "lanes of the copies");
    auto swizzled = [](int row, int c) { return (c ^ ((row * NG / 8) & (NG - 1))) << 4; };  // the same for rows 8 apart
    const uint32_t code_src = (lane / NG) * (D / 2) + (lane & (NG - 1)) * 16;
    uint32_t code_dst[kRowsPer < 8 ? 2 : 1];
    code_dst[0] = (lane / NG) * (D / 2) + swizzled(lane / NG, lane & (NG - 1));
    if constexpr (kRowsPer < 8) code_dst[1] = (lane / NG) * (D / 2) + swizzled(lane / NG + kRowsPer, lane & (NG - 1));
    Cursor ld = cur;
    uint32_t col = 0, in = 0;  // table column, and row of 16 inside the block, of tile lane % TILES
    int next_id = -2;          // its entry (-2: nothing of the tile is seen)
    bool bad = false;
    const uint32_t bs16 = static_cast<uint32_t>(bs) >> 4;
    const uint32_t col_by = kStride * TILES / bs16, in_by = kStride * TILES - col_by * bs16;  // the warp's next step
    int ld_pos = 0, ld_ctx = 0, ld_first = 0;  // of ld's step: position of this lane's tile
    uint32_t ld_head = 0;
    const int32_t *ld_table = nullptr;
    auto look_up = [&] {
        next_id = -2;
        if (lane < TILES && ld_pos < ld_ctx && (!MOD || ld_pos + 16 > ld_first)) next_id = __ldg(ld_table + col);
    };
    int ld_b = -1, ld_unit = 0;  // the sequence that ld_ctx is of, units begun
    auto start_unit = [&] {
        next_id = -2;
        if (ld.b >= B) return;
        if (ld.b != ld_b) {
            ld_b = ld.b;
            ld_first = first_of(ld.b);
            ld_ctx = context_of(ld.b, ld_first);
            ld_table = A.block_tables + static_cast<int64_t>(ld.b) * A.max_blocks;
        }
        const int kh = ld.hu / A.subs, sub = ld.hu - kh * A.subs;
        ld_head = static_cast<uint32_t>(kh);
        ld_pos = (ld_first / STEP + ld.st) * STEP + 16 * (lane & (TILES - 1));
        col = static_cast<uint32_t>(ld_pos >> 4) / bs16;
        in = static_cast<uint32_t>(ld_pos >> 4) - col * bs16;
        look_up();
        const int live = min(kI4Heads, A.G - sub * kI4Heads);
        const uint8_t *src = static_cast<const uint8_t *>(A.q) +
                             (static_cast<int64_t>(ld.b) * A.Hq + kh * A.G + sub * kI4Heads) * (D * 2) + 16 * lane;
        for (int i = lane; i < live * (D / 8); i += 32, src += 512) cp16(q_tile + (ld_unit & 1) * R::kQ + 16 * i, src);
        ++ld_unit;  // committed with the next copy
    };
    uint32_t at = 0, here = 0;  // of the step copied last: a tile's first row, in rows of 16 (lane h: tile h); the tiles that are there
    auto copy = [&](uint32_t dst, const uint8_t *codes, const __half *scales) {
#pragma unroll
        for (int h = 0; h < TILES; ++h) {
            const uint32_t row16 = __shfl_sync(0xffffffffu, at, h);
            if (!(here >> h & 1)) continue;  // what is not there is masked, its stale rows too
            const uint8_t *src = codes + (static_cast<uint64_t>(row16) * (8 * D) + code_src);
#pragma unroll
            for (int i = 0; i < kCopies; ++i)
                cp16(dst + code_dst[kRowsPer < 8 ? i & 1 : 0] + (16 * h + i * kRowsPer) * (D / 2), src + i * kRowsPer * (D / 2));
        }
#pragma unroll
        for (int h = 0; h < TILES; h += kScaleTiles) {
            const int mt = h + lane / kChunks;  // this lane's tile
            const uint32_t row16 = __shfl_sync(0xffffffffu, at, mt & (TILES - 1));
            if (lane < kScaleTiles * kChunks && (here >> mt & 1))
                cp16(dst + R::kCodes + 16 * (h * kChunks + lane), scales + (static_cast<uint64_t>(row16) * (16 * NG) + 8 * (lane % kChunks)));
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto copy_k = [&] {  // of the next step, whose entries have been looked up; then those of the one behind it are
        const bool mine = next_id >= 0 && next_id < A.num_blocks;
        bad = bad || (!mine && next_id != -2);
        // a pool that fits the memory has less than 2^32 rows of 16
        at = mine ? (static_cast<uint32_t>(next_id) * A.Hkv + ld_head) * bs16 + in : 0u;
        here = __ballot_sync(0xffffffffu, mine) & ((1u << TILES) - 1);
        copy(k_tile, A.k_cache, A.k_scale);
        ld.st += kStride;
        if (DIRECT || ld.st < ld.n) {
            const bool over = in + in_by >= bs16;
            in = in + in_by - (over ? bs16 : 0u);
            col += col_by + (over ? 1u : 0u);
            ld_pos += kStride * STEP;
            look_up();
        } else {
            next_unit(ld);
            start_unit();
        }
    };
    if (count > 0) start_unit();
    // ---- a unit's queries: lane (g = head, t): dims 8 t .. 8 t + 7 of every group, f16 under a power of two
    const int g = lane >> 2, t = lane & 3, mi = lane >> 3, r8 = lane & 7;
    const uint32_t frag_at = (r8 + 8 * (mi & 1)) * (D / 2), frag_sw = swizzled(r8, 0);  // this lane's row of the ldmatrix tiles
    uint32_t qf[NG][4];
    float off[NG][2];            // start of the group's accumulator, heads 2 t and 2 t + 1
    float sl0 = 0.f, sl1 = 0.f;  // scores to log2 units, of heads 2 t, 2 t + 1
    float slope0 = 0.f, slope1 = 0.f;
    int heads = 0;
    int64_t head0 = 0;  // first query head's row of q and out
    int unit = 0;  // units begun
    auto load_q = [&](const Cursor &c) {
        const int kh = c.hu / A.subs, sub = c.hu - kh * A.subs;
        heads = min(kI4Heads, A.G - sub * kI4Heads);
        head0 = static_cast<int64_t>(c.b) * A.Hq + kh * A.G + sub * kI4Heads;
        const bool live = g < heads;
        const uint32_t src = q_tile + (unit & 1) * R::kQ + g * (D * 2) + t * 16;
        ++unit;
        uint32_t x[NG][4];
        float top = 0.f;
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
            lds_words(src + gg * 64, x[gg]);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[gg][k] = live ? x[gg][k] : 0u;
        }
        auto get = [&](int gg, int k) -> float {
            const T *e = reinterpret_cast<const T *>(&x[gg]);
            return to_f32<T>(e[k]);
        };
#pragma unroll
        for (int gg = 0; gg < NG; ++gg)
#pragma unroll
            for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(get(gg, k)));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the largest value to [2^13, 2^14): all of a 16-bit type's bits down to 2^-23 of it, q / 16 included
        const int e = static_cast<int>(__float_as_uint(top) >> 23);
        const int k2 = e == 0 || e == 255 ? 0 : min(max(140 - e, -120), 120);
        const float f = __uint_as_float(static_cast<uint32_t>(k2 + 127) << 23);
        const float back = __uint_as_float(static_cast<uint32_t>(127 - k2) << 23);
        float start[NG];
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
            float a = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w = j & 1 ? 0.0625f * f : f;
                const uint32_t p = H::pack(get(gg, 2 * j) * w, get(gg, 2 * j + 1) * w);
                qf[gg][j] = p;
                const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&p));
                a = fmaf(v.x + v.y, j & 1 ? -128.f * kI4Unit : -8.f * kI4Unit, a);
            }
            a += __shfl_xor_sync(0xffffffffu, a, 1);
            a += __shfl_xor_sync(0xffffffffu, a, 2);
            start[gg] = a;
        }
        const float whole_sl = A.scale_log2 * back * (1.f / kI4Unit);
        // finite, and without rules not 0 either: times a score of 0, or of -inf (a masked one), it is a number
        const float top_sl = fabsf(whole_sl) > 3e38f ? copysignf(3e38f, whole_sl) : whole_sl;
        const float sl = MOD ? top_sl : fmaxf(top_sl, 1.17549435e-38f);
        // from the lanes of head g to those of columns 2 t, 2 t + 1
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
            off[gg][0] = __shfl_sync(0xffffffffu, start[gg], 8 * t);
            off[gg][1] = __shfl_sync(0xffffffffu, start[gg], 8 * t + 4);
        }
        sl0 = __shfl_sync(0xffffffffu, sl, 8 * t);
        sl1 = __shfl_sync(0xffffffffu, sl, 8 * t + 4);
        if (MOD && A.slopes) {
            const int h = kh * A.G + sub * kI4Heads + 2 * t;
            slope0 = 2 * t < heads ? A.slopes[h] * kI4Log2e : 0.f;
            slope1 = 2 * t + 1 < heads ? A.slopes[h + 1] * kI4Log2e : 0.f;
        }
    };

    float o[NG][2][4];  // rows: dims 32 gg + 8 (g / 2) + g % 2 + 4 e (+ 2), columns: heads 2 t, 2 t + 1
    float m0, m1, l0, l1, b0, b1;  // references (b = room - m, 0 before there is one) and sums
    uint32_t top_scale = i4_top_scale(kI4TopExp);  // twice the largest f16 with the exponent field that room is for
    int pos = 0, ctx = 0, first = 0, cur_b = -1;  // of cur's step, and the sequence they are of
    bool fresh = true;                // the next step starts a unit
    bool whole = false;               // the unit began in this slice
    if (count > 0) {
        copy_k();
        copy(v_tile, A.v_cache, A.v_scale);
    }
    for (int s = 0; s < count; ++s) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");  // K: V, committed after it, may be under way
        __syncwarp();
        if (fresh) {
            load_q(cur);
            if (cur.b != cur_b) {
                cur_b = cur.b;
                first = first_of(cur.b);
                ctx = context_of(cur.b, first);
            }
            pos = (first / STEP + cur.st) * STEP;
#pragma unroll
            for (int gg = 0; gg < NG; ++gg)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[gg][e][c] = 0.f;
            m0 = m1 = -INFINITY;
            l0 = l1 = b0 = b1 = 0.f;
            top_scale = i4_top_scale(kI4TopExp);
            whole = cur.st == 0;
            if (!DIRECT && lane == 0 && whole) A.unit_info[static_cast<int64_t>(cur.b) * HU + cur.hu].x = static_cast<int>(me);
            fresh = false;
        }
        const uint32_t now = here;
        const bool partial = pos + STEP > ctx || (MOD && pos < first) || now != (1u << TILES) - 1;
        auto seen = [&](int k) {  // token k of the step
            return pos + k < ctx && (!MOD || pos + k >= first) && (now >> (k >> 4) & 1);
        };
        // 1. scores, tiles of 16 tokens: rows (tokens) g and g + 8, columns (heads) 2 t, 2 t + 1
        float y[TILES][4];
#pragma unroll
        for (int tile = 0; tile < TILES; ++tile) {
            uint32_t w[NG][2];  // word t of group gg, of tokens g and g + 8
#pragma unroll
            for (int gg = 0; gg < NG; gg += 2) {
                uint32_t x[4];
                ldsm_x4(k_tile + frag_at + 16 * tile * (D / 2) + (((gg + (mi >> 1)) << 4) ^ frag_sw), x);
                w[gg][0] = x[0];
                w[gg][1] = x[1];
                w[gg + 1][0] = x[2];
                w[gg + 1][1] = x[3];
            }
            uint32_t sa[NG / 2], sb[NG / 2];  // scales of tokens g and g + 8
            const uint32_t ks = k_tile + R::kCodes + (16 * tile + g) * (NG * 2);
            lds_words(ks, sa);
            lds_words(ks + 8 * NG * 2, sb);
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) {
                float acc[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t a[4];
                    const uint32_t x0 = e ? w[gg][0] >> 8 : w[gg][0], x1 = e ? w[gg][1] >> 8 : w[gg][1];
                    a[0] = x0 & 0x000f000fu;
                    a[1] = x1 & 0x000f000fu;
                    a[2] = x0 & 0x00f000f0u;
                    a[3] = x1 & 0x00f000f0u;
                    if (e == 0) mma_start(acc, a, qf[gg][0], qf[gg][1], off[gg][0], off[gg][1]);
                    else H::mma(acc, a, qf[gg][2], qf[gg][3]);
                }
                const float2 fa = __half22float2(*reinterpret_cast<const __half2 *>(&sa[gg / 2]));
                const float2 fb = __half22float2(*reinterpret_cast<const __half2 *>(&sb[gg / 2]));
                const float s_a = gg & 1 ? fa.y : fa.x, s_b = gg & 1 ? fb.y : fb.x;
                y[tile][0] = gg ? fmaf(s_a, acc[0], y[tile][0]) : s_a * acc[0];
                y[tile][1] = gg ? fmaf(s_a, acc[1], y[tile][1]) : s_a * acc[1];
                y[tile][2] = gg ? fmaf(s_b, acc[2], y[tile][2]) : s_b * acc[2];
                y[tile][3] = gg ? fmaf(s_b, acc[3], y[tile][3]) : s_b * acc[3];
            }
        }
        __syncwarp();
        const bool more = s + 1 < count;
        if (more) copy_k();
        else asm volatile("cp.async.commit_group;" ::: "memory");  // (the group that the waits count)
        asm volatile("cp.async.wait_group 1;" ::: "memory");  // V: the next K may be under way
        __syncwarp();
        if (partial) {  // V scales of rows that are not seen may be anything, and P there is 0: their product must be 0
            for (int k = lane; k < STEP; k += 32)
                if (!seen(k)) {
#pragma unroll
                    for (int i = 0; i < NG / 2; ++i)
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(v_tile + R::kCodes + k * (NG * 2) + 4 * i), "r"(0) : "memory");
                }
            __syncwarp();
        }
        uint32_t vmax;  // the largest of this lane's share of V's scales, by halves
        {
            constexpr int kWords = STEP * NG / 64;  // pairs of scales of a lane
            static_assert(kWords == 2 || kWords == 4, "a vector of scales a lane");
            uint32_t x[kWords];
            lds_words(v_tile + R::kCodes + lane * (4 * kWords), x);
            vmax = x[0];
#pragma unroll
            for (int i = 1; i < kWords; ++i) vmax = max_u16x2(vmax, x[i]);
        }
        // 2. score rules, in log2 units (without them the factors sl0, sl1 > 0 wait for the exponent), and masks
        if constexpr (MOD) {
#pragma unroll
            for (int tile = 0; tile < TILES; ++tile) {
                y[tile][0] *= sl0;
                y[tile][1] *= sl1;
                y[tile][2] *= sl0;
                y[tile][3] *= sl1;
                if (A.softcap > 0.f) {
                    // c tanh(s / c): the fit where |s / c| is small, else by the exponential
                    const float cap = A.softcap * kI4Log2e, inv = 1.f / cap, u2 = 2.f / A.softcap;
                    constexpr float f0 = kTanhFit[0], f1 = kTanhFit[1], f2 = kTanhFit[2], f3 = kTanhFit[3], f4 = kTanhFit[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float v = y[tile][c], u = v * inv, z = u * u;
                        const float p = fmaf(fmaf(fmaf(fmaf(f4, z, f3), z, f2), z, f1), z, f0);
                        y[tile][c] = fabsf(u) > kTanhLimit ? fmaf(fast_rcp(1.f + fast_exp2(v * u2)), -2.f * cap, cap) : v * p;
                    }
                }
                const float d0 = static_cast<float>(ctx - 1 - (pos + 16 * tile + g)), d8 = d0 - 8.f;
                y[tile][0] = fmaf(-slope0, d0, y[tile][0]);
                y[tile][1] = fmaf(-slope1, d0, y[tile][1]);
                y[tile][2] = fmaf(-slope0, d8, y[tile][2]);
                y[tile][3] = fmaf(-slope1, d8, y[tile][3]);
            }
        }
        if (partial) {
#pragma unroll
            for (int tile = 0; tile < TILES; ++tile) {
                const bool a = seen(16 * tile + g), b = seen(16 * tile + g + 8);
                y[tile][0] = a ? y[tile][0] : -INFINITY;
                y[tile][1] = a ? y[tile][1] : -INFINITY;
                y[tile][2] = b ? y[tile][2] : -INFINITY;
                y[tile][3] = b ? y[tile][3] : -INFINITY;
            }
        }
        // 3. The reference m of a head is a maximum of some step; P = 2^(y - m + room) may pass 2^room
        // by kI4Slack binades before it is moved, and the sum and accumulator with it; so they are where
        // scales of V leave P less room.
        float mx0 = fmaxf(y[0][0], y[0][2]), mx1 = fmaxf(y[0][1], y[0][3]);
#pragma unroll
        for (int tile = 1; tile < TILES; ++tile) {
            mx0 = max3f(mx0, y[tile][0], y[tile][2]);
            mx1 = max3f(mx1, y[tile][1], y[tile][3]);
        }
        if constexpr (!MOD) {
            mx0 *= sl0;
            mx1 *= sl1;
        }
        if (__any_sync(0xffffffffu, mx0 > m0 + kI4Slack || mx1 > m1 + kI4Slack || max_u16x2(vmax, top_scale) != top_scale)) {
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, sh));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, sh));
            }
            const int from = i4_exp(top_scale);
            const int top = __reduce_max_sync(0xffffffffu, max(from, max(i4_exp(vmax), i4_exp(vmax >> 16))));
            top_scale = i4_top_scale(top);
            const float room = i4_room(top), less = fast_exp2(static_cast<float>(from - top));
            const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
            const float a0 = n0 == -INFINITY ? 1.f : less * fast_exp2(m0 - n0), a1 = n1 == -INFINITY ? 1.f : less * fast_exp2(m1 - n1);
            m0 = n0;
            m1 = n1;
            b0 = n0 == -INFINITY ? 0.f : room - n0;
            b1 = n1 == -INFINITY ? 0.f : room - n1;
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int gg = 0; gg < NG; ++gg)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    o[gg][e][0] *= a0;
                    o[gg][e][1] *= a1;
                    o[gg][e][2] *= a0;
                    o[gg][e][3] *= a1;
                }
        }
        // 4. P and O += P V
#pragma unroll
        for (int tile = 0; tile < TILES; ++tile) {
            const float f0 = MOD ? 1.f : sl0, f1 = MOD ? 1.f : sl1;
            const float p0 = fast_exp2(fmaf(y[tile][0], f0, b0)), p1 = fast_exp2(fmaf(y[tile][1], f1, b1));
            const float p2 = fast_exp2(fmaf(y[tile][2], f0, b0)), p3 = fast_exp2(fmaf(y[tile][3], f1, b1));
            l0 += p0 + p2;
            l1 += p1 + p3;
            const uint32_t pb0 = movmatrix_trans(H::pack(p0, p1)), pb1 = movmatrix_trans(H::pack(p2, p3));
            // scales of tokens 2 t, 2 t + 1 (words 0 .. NG - 1) and of those 8 further
            uint32_t va[NG], vb[NG];
            const uint32_t vs = v_tile + R::kCodes + (16 * tile + 2 * t) * (NG * 2);
            lds_words(vs, va);
            lds_words(vs + 8 * NG * 2, vb);
#pragma unroll
            for (int gg = 0; gg < NG; gg += 2) {
                uint32_t w[4];  // (tokens 0 .. 7 | 8 .. 15) of groups gg, gg + 1
                ldsm_x4_trans(v_tile + frag_at + 16 * tile * (D / 2) + (((gg + (mi >> 1)) << 4) ^ frag_sw), w);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t sel = h ? 0x7632 : 0x5410;  // (scale of token 2 t, of 2 t + 1)
                    const uint32_t s_a = __byte_perm(va[gg / 2], va[NG / 2 + gg / 2], sel);
                    const uint32_t s_b = __byte_perm(vb[gg / 2], vb[NG / 2 + gg / 2], sel);
                    const uint32_t q0 = mul_f16x2(pb0, s_a), q1 = mul_f16x2(pb1, s_b);
                    uint32_t xa[4], xb[4];
                    int4_widen(w[2 * h], xa);
                    int4_widen(w[2 * h + 1], xb);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t a[4] = {xa[2 * e], xa[2 * e + 1], xb[2 * e], xb[2 * e + 1]};
                        H::mma(o[gg + h][e], a, q0, q1);
                    }
                }
            }
        }
        __syncwarp();
        if (more) copy(v_tile, A.v_cache, A.v_scale);
        pos += kStride * STEP;
        if constexpr (DIRECT) continue;
        if (++cur.st == cur.n || s + 1 == count) {
            // the unit ends, or the slice does
            fresh = true;
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, sh);
                l1 += __shfl_xor_sync(0xffffffffu, l1, sh);
            }
            const bool ends = cur.st == cur.n;
            const int64_t u = static_cast<int64_t>(cur.b) * HU + cur.hu;
            if (ends && lane == 0) A.unit_info[u].y = static_cast<int>(me);
            const int hA = 2 * t, hB = 2 * t + 1;
            if (whole && ends) {
                const float i0 = l0 > 0.f ? 1.f / l0 : (l0 == l0 ? 0.f : l0), i1 = l1 > 0.f ? 1.f / l1 : (l1 == l1 ? 0.f : l1);
                T *out = static_cast<T *>(A.out) + head0 * D;
#pragma unroll
                for (int gg = 0; gg < NG; ++gg)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int d = 32 * gg + 8 * (g >> 1) + (g & 1) + 4 * e;
                        if (hA < heads) {
                            out[hA * D + d] = from_f32<T>(o[gg][e][0] * i0);
                            out[hA * D + d + 2] = from_f32<T>(o[gg][e][2] * i0);
                        }
                        if (hB < heads) {
                            out[hB * D + d] = from_f32<T>(o[gg][e][1] * i1);
                            out[hB * D + d + 2] = from_f32<T>(o[gg][e][3] * i1);
                        }
                    }
            } else {
                const int64_t piece = (me + u) * A.rows;
                float *po = A.o_piece + piece * D;
#pragma unroll
                for (int gg = 0; gg < NG; ++gg)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int d = 32 * gg + 8 * (g >> 1) + (g & 1) + 4 * e;
                        if (hA < heads) {
                            po[hA * D + d] = o[gg][e][0];
                            po[hA * D + d + 2] = o[gg][e][2];
                        }
                        if (hB < heads) {
                            po[hB * D + d] = o[gg][e][1];
                            po[hB * D + d + 2] = o[gg][e][3];
                        }
                    }
                const float room = i4_room(i4_exp(top_scale));
                if (g == 0 && hA < heads) A.ml_piece[piece + hA] = make_float2(m0 - room, l0);
                if (g == 0 && hB < heads) A.ml_piece[piece + hB] = make_float2(m1 - room, l1);
            }
            if (ends) next_unit(cur);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (bad && A.err_flag) atomicOr(A.err_flag, PKV_ERRBIT_BLOCK_RANGE);
    if constexpr (DIRECT) {
        // The warps' accumulators meet in shared memory, each in its own tiles.
        __shared__ float2 warp_ml[WARPS][kI4Heads];
        const int kh = cur.hu / A.subs, sub = cur.hu - kh * A.subs, live = min(kI4Heads, A.G - sub * kI4Heads);
        constexpr int kFloats = R::kWarp / 4;
        static_assert(kFloats >= kI4Heads * D, "a unit's accumulator fits the warp's tiles");
        float *mine = reinterpret_cast<float *>(smem) + warp * kFloats;
        __syncwarp();
        if (count == 0) {
            if (lane < kI4Heads) warp_ml[warp][lane] = make_float2(-INFINITY, 0.f);
        } else {
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, sh);
                l1 += __shfl_xor_sync(0xffffffffu, l1, sh);
            }
            if (g == 0) {
                const float room = i4_room(i4_exp(top_scale));
                warp_ml[warp][2 * t] = make_float2(m0 - room, l0);
                warp_ml[warp][2 * t + 1] = make_float2(m1 - room, l1);
            }
#pragma unroll
            for (int gg = 0; gg < NG; ++gg)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int d = 32 * gg + 8 * (g >> 1) + (g & 1) + 4 * e;
                    mine[2 * t * D + d] = o[gg][e][0];
                    mine[2 * t * D + d + 2] = o[gg][e][2];
                    mine[(2 * t + 1) * D + d] = o[gg][e][1];
                    mine[(2 * t + 1) * D + d + 2] = o[gg][e][3];
                }
        }
        __syncthreads();
        uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<T *>(A.out) + (static_cast<int64_t>(cur.b) * A.Hq + kh * A.G + sub * kI4Heads) * D);
        for (int i = threadIdx.x; i < live * (D / 2); i += WARPS * 32) {
            const int h = i / (D / 2);
            float M = -INFINITY, L = 0.f, a = 0.f, c = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) M = fmaxf(M, warp_ml[w][h].x);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float2 ml = warp_ml[w][h];
                if (ml.x == -INFINITY && ml.y == 0.f) continue;  // (scores that are all NaN leave the maximum there, and a NaN sum)
                const float f = exp2f(ml.x - (M == -INFINITY ? 0.f : M));
                const float2 v = reinterpret_cast<const float2 *>(smem)[w * (kFloats / 2) + i];
                L = fmaf(f, ml.y, L);
                a = fmaf(f, v.x, a);
                c = fmaf(f, v.y, c);
            }
            const float inv = L > 0.f ? 1.f / L : (L == L ? 0.f : L);
            out[i] = Half16<T>::pack(a * inv, c * inv);
        }
    }
}

// Joins a unit's pieces: out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k.  WPR warps take a
// row (a unit's query head), lanes the dims, eight pieces in flight a warp; the host spreads few
// rows over more warps.
constexpr int kI4JoinWarps = 8;
constexpr int kI4JoinTarget = 4096;  // warps of a launch, about

template <typename T, int D, int WPR>
__global__ void __launch_bounds__(kI4JoinWarps * 32)
decode_int4_join_kernel(const __grid_constant__ I4Args A, int64_t rows) {
    constexpr int V = D / 32;  // dims of a lane
    constexpr int U = D == 256 ? 4 : 8;
    using F = typename std::conditional<V == 2, float2, float4>::type;
    constexpr int FW = sizeof(F) / 4, FN = V / FW;
    __shared__ float part[WPR > 1 ? kI4JoinWarps : 1][D];
    __shared__ float2 part_ml[kI4JoinWarps];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub_warp = warp % WPR;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kI4JoinWarps / WPR) + warp / WPR;
    const int HU = A.Hkv * A.subs;
    int64_t u = 0, out_row = 0;
    int r = 0, from = 0, to = -1;  // the row's pieces are those of warps from .. to
    if (row < rows) {
        u = i4_div(row, A.rows);
        r = static_cast<int>(row - u * A.rows);
        const int b = static_cast<int>(i4_div(u, HU)), hu = static_cast<int>(u - static_cast<int64_t>(b) * HU);
        const int kh = hu / A.subs, head = (hu - kh * A.subs) * kI4Heads + r;
        const int ctx = A.context_lens[b], first = A.key_starts ? max(A.key_starts[b], 0) : 0;
        const int2 ui = A.unit_info[u];
        out_row = static_cast<int64_t>(b) * A.Hq + kh * A.G + head;
        // Nothing to do: a row of zeros already, or one piece (the main kernel wrote the output).
        // Ranges outside the launch's warps are never left behind; none would be followed.
        if (head < A.G && ctx > first && ctx <= A.max_ctx && static_cast<int64_t>(ctx) <= static_cast<int64_t>(A.max_blocks) * A.bs &&
            ui.x >= 0 && ui.x < ui.y && ui.y < kI4MaxWarps) {
            from = ui.x;
            to = ui.y;
        }
    }
    float M = -INFINITY, L = 0.f, acc[V] = {};
    for (int w = from + sub_warp; w <= to; w += U * WPR) {
        F v[U][FN];
        float2 ml[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const bool in = w + i * WPR <= to;
            const int64_t piece = (w + i * WPR + u) * A.rows + r;
            ml[i] = in ? __ldg(A.ml_piece + piece) : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int k = 0; k < FN; ++k) v[i][k] = in ? __ldg(reinterpret_cast<const F *>(A.o_piece + piece * D) + lane * FN + k) : F{};
        }
        float n = M;
#pragma unroll
        for (int i = 0; i < U; ++i) n = fmaxf(n, ml[i].x);
        const float base = n == -INFINITY ? 0.f : n, a = exp2f(M - base);
        M = n;
        L *= a;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] *= a;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const float f = exp2f(ml[i].x - base);
            L = fmaf(f, ml[i].y, L);
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = fmaf(f, reinterpret_cast<const float *>(v[i])[k], acc[k]);
        }
    }
    if constexpr (WPR > 1) {
#pragma unroll
        for (int k = 0; k < V; ++k) part[warp][lane * V + k] = acc[k];
        if (lane == 0) part_ml[warp] = make_float2(M, L);
        __syncthreads();
        if (sub_warp != 0) return;
        M = -INFINITY;
#pragma unroll
        for (int i = 0; i < WPR; ++i) M = fmaxf(M, part_ml[warp + i].x);
        const float base = M == -INFINITY ? 0.f : M;
        L = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.f;
#pragma unroll
        for (int i = 0; i < WPR; ++i) {
            const float f = exp2f(part_ml[warp + i].x - base);
            L = fmaf(f, part_ml[warp + i].y, L);
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = fmaf(f, part[warp + i][lane * V + k], acc[k]);
        }
    }
    if (to < from) return;
    const float inv = L > 0.f ? 1.f / L : (L == L ? 0.f : L);
    uint32_t o[V / 2];
#pragma unroll
    for (int k = 0; k < V / 2; ++k) o[k] = Half16<T>::pack(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<T *>(A.out) + out_row * D) + lane * (V / 2);
#pragma unroll
    for (int k = 0; k < V / 2; ++k) dst[k] = o[k];
}

// ----------------------------------------------------------------------------- host side
struct I4Plan {
    int32_t subs = 1, rows = 0, group = 0;  // units of a KV head, query heads of a unit at most, sequences of a launch
    int64_t units = 0;            // of a launch
    bool direct = false;          // a CTA per unit, nothing to join
    size_t o_bytes = 0, ml_bytes = 0, ws_bytes = 0;
};

bool i4_shape(int32_t d) { return d == 64 || d == 128 || d == 256; }

I4Plan i4_plan(int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int32_t max_ctx) {
    I4Plan p;
    p.subs = (Hq / Hkv + kI4Heads - 1) / kI4Heads;
    p.rows = Hq / Hkv < kI4Heads ? Hq / Hkv : kI4Heads;
    p.group = B < kI4MaxSeqs ? B : kI4MaxSeqs;
    p.units = static_cast<int64_t>(p.group) * Hkv * p.subs;
    p.direct = B <= kI4MaxSeqs && p.units <= 152 * (d == 256 ? 2 : kI4DirectCtas) && max_ctx <= kI4DirectLen;
    if (p.direct) return p;
    const int64_t slots = kI4MaxWarps + p.units;
    p.o_bytes = static_cast<size_t>(slots) * p.rows * d * sizeof(float);
    p.ml_bytes = (static_cast<size_t>(slots) * p.rows * sizeof(float2) + 255) / 256 * 256;
    p.ws_bytes = p.o_bytes + p.ml_bytes + (static_cast<size_t>(p.units) * sizeof(int2) + 255) / 256 * 256;
    return p;
}

template <typename T, int D, bool MOD, bool DIRECT>
cudaError_t i4_launch(const I4Args &a, const I4Plan &p, cudaStream_t stream) {
    // 8, 12 or 16 warps an SM (255, 168 or 128 registers a thread): as one CTA, whose prefix of the
    // lengths serves them all (8 x 32768 tokens 57.8 us, as three CTAs 59.5), or direct CTAs of four.
    constexpr int STEP = D == 256 ? 32 : 64, kSmWarps = D == 256 ? 8 : D == 128 ? 12 : 16;
    constexpr int WARPS = DIRECT ? 4 : kSmWarps, CTAS = kSmWarps / WARPS;
    constexpr int smem = WARPS * I4Tile<D, STEP>::kWarp;
    static_assert(smem >= (kI4MaxSeqs + 1) * 8 + kI4MaxSeqs * 4, "the prefix lies in the tiles");
    auto kern = decode_int4_kernel<T, D, STEP, WARPS, CTAS, MOD, DIRECT>;
    static std::atomic<int> grids[64];  // resident CTAs, per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int grid = grids[dev & 63].load(std::memory_order_acquire);
    if (grid == 0) {
        int per_sm = 0, sms = 0;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, WARPS * 32, smem);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        grid = per_sm * sms;
        if (grid > kI4MaxWarps / WARPS) grid = kI4MaxWarps / WARPS;
        if (grid < 1) return cudaErrorInvalidConfiguration;
        grids[dev & 63].store(grid, std::memory_order_release);
    }
    if (DIRECT) return launch_pdl(kPdlDecode, kern, dim3(static_cast<unsigned>(p.units)), dim3(WARPS * 32), smem, stream, a);
    e = launch_pdl(kPdlDecode, kern, dim3(grid), dim3(WARPS * 32), smem, stream, a);
    if (e != cudaSuccess) return e;
    const int64_t rows = static_cast<int64_t>(a.B) * a.Hkv * a.subs * a.rows;
    int wpr = kI4JoinWarps;
    while (wpr > 1 && rows * wpr > kI4JoinTarget) wpr >>= 1;
    const int64_t per = kI4JoinWarps / wpr;
    auto join = wpr == 8 ? decode_int4_join_kernel<T, D, 8> : wpr == 4 ? decode_int4_join_kernel<T, D, 4>
              : wpr == 2 ? decode_int4_join_kernel<T, D, 2> : decode_int4_join_kernel<T, D, 1>;
    return launch_pdl(kPdlCombine, join, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(kI4JoinWarps * 32), 0, stream, a, rows);
}

template <typename T, bool MOD, bool DIRECT>
cudaError_t i4_launch_d(const I4Args &a, const I4Plan &p, int32_t d, cudaStream_t s) {
    return d == 64 ? i4_launch<T, 64, MOD, DIRECT>(a, p, s) : d == 128 ? i4_launch<T, 128, MOD, DIRECT>(a, p, s)
                                                                      : i4_launch<T, 256, MOD, DIRECT>(a, p, s);
}

template <typename T>
cudaError_t i4_launch_any(const I4Args &a, const I4Plan &p, int32_t d, bool rules, cudaStream_t s) {
    if (p.direct) return rules ? i4_launch_d<T, true, true>(a, p, d, s) : i4_launch_d<T, false, true>(a, p, d, s);
    return rules ? i4_launch_d<T, true, false>(a, p, d, s) : i4_launch_d<T, false, false>(a, p, d, s);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_paged_attention_decode_int4_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                                                 int32_t head_dim, int32_t max_context_len) {
    if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || !i4_shape(head_dim)) return 0;
    return i4_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len).ws_bytes;
}

extern "C" pkv_status pkv_paged_attention_decode_int4(
    void *out, const void *q, const void *k_cache, const void *v_cache, const uint16_t *k_scale, const uint16_t *v_scale,
    const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t num_seqs, int32_t num_q_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks, int32_t max_context_len, float scale,
    const pkv_score_mod *mod, pkv_dtype dtype, void *workspace, size_t workspace_bytes, int32_t *err_flag, void *stream) {
    if (dtype_bytes(dtype) == 0) return set_error(PKV_ERR_INVALID_ARG, "int4 decode: unknown dtype %d", (int)dtype);
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks < 0 ||
        max_blocks_per_seq < 0 || max_context_len < 0)
        return set_error(PKV_ERR_INVALID_ARG, "int4 decode: bad sizes");
    if (num_q_heads % num_kv_heads)
        return set_error(PKV_ERR_INVALID_ARG, "int4 decode: num_q_heads (%d) is not a multiple of num_kv_heads (%d)", num_q_heads, num_kv_heads);
    if (static_cast<int64_t>(num_blocks) * block_size > INT32_MAX)
        return set_error(PKV_ERR_INVALID_ARG, "int4 decode: num_blocks * block_size >= 2^31");
    if (max_context_len > INT32_MAX - 64) return set_error(PKV_ERR_INVALID_ARG, "int4 decode: max_context_len is too long");
    const pkv_score_mod none{};
    const pkv_score_mod m = mod ? *mod : none;
    if (!(m.softcap >= 0.f) || m.softcap > 1e30f || (m.softcap > 0.f && m.softcap < 1e-30f))
        return set_error(PKV_ERR_INVALID_ARG, "int4 decode: softcap must be 0, or from 1e-30 to 1e30");
    if (num_q_heads > (1 << 20)) return set_error(PKV_ERR_UNSUPPORTED, "int4 decode: more than 2^20 query heads");
    if (num_seqs == 0) return ok();
    if ((dtype != PKV_F16 && dtype != PKV_BF16) || !i4_shape(head_dim) || block_size % 16)
        return set_error(PKV_ERR_UNSUPPORTED, "int4 decode: needs fp16/bf16, head_dim 64, 128 or 256 and block_size a multiple of 16");
    if (!out || !q || !context_lens || (max_blocks_per_seq > 0 && !block_tables) || !k_cache || !v_cache || !k_scale || !v_scale ||
        num_blocks == 0)
        return set_error(PKV_ERR_INVALID_ARG, "int4 decode: NULL pointer or empty pool");
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 16) ||
        !aligned(v_scale, 16))
        return set_error(PKV_ERR_UNSUPPORTED, "int4 decode: caches, scales, q and out must be 16-byte aligned");
    const I4Plan p = i4_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len);
    if (p.ws_bytes > 0 && (!workspace || workspace_bytes < p.ws_bytes || !aligned(workspace, 256)))
        return set_error(PKV_ERR_WORKSPACE, "int4 decode: workspace needs %zu bytes (256-byte aligned), got %zu", p.ws_bytes, workspace_bytes);
    I4Args a{};
    a.k_cache = static_cast<const uint8_t *>(k_cache);
    a.v_cache = static_cast<const uint8_t *>(v_cache);
    a.k_scale = reinterpret_cast<const __half *>(k_scale);
    a.v_scale = reinterpret_cast<const __half *>(v_scale);
    a.slopes = m.alibi_slopes;
    a.max_blocks = max_blocks_per_seq;
    a.Hq = num_q_heads;
    a.Hkv = num_kv_heads;
    a.G = num_q_heads / num_kv_heads;
    a.subs = p.subs;
    a.rows = p.rows;
    a.bs = block_size;
    a.num_blocks = num_blocks;
    a.max_ctx = max_context_len;
    a.scale_log2 = scale * kI4Log2e;
    a.softcap = m.softcap;
    char *ws = static_cast<char *>(workspace);
    a.o_piece = reinterpret_cast<float *>(ws);
    a.ml_piece = reinterpret_cast<float2 *>(ws + p.o_bytes);
    a.unit_info = reinterpret_cast<int2 *>(ws + p.o_bytes + p.ml_bytes);
    a.err_flag = err_flag;
    // without rules the score's factor goes into the exponent, which wants it positive
    const bool rules = m.softcap > 0.f || m.alibi_slopes || m.key_starts || !(scale > 1e-30f);
    for (int32_t b0 = 0; b0 < num_seqs; b0 += p.group) {  // consecutive launches, one workspace
        const int64_t at = static_cast<int64_t>(b0) * num_q_heads * head_dim * 2;
        a.out = static_cast<char *>(out) + at;
        a.q = static_cast<const char *>(q) + at;
        a.block_tables = block_tables + static_cast<int64_t>(b0) * max_blocks_per_seq;
        a.context_lens = context_lens + b0;
        a.key_starts = m.key_starts ? m.key_starts + b0 : nullptr;
        a.B = num_seqs - b0 < p.group ? num_seqs - b0 : p.group;
        auto s = static_cast<cudaStream_t>(stream);
        const cudaError_t e = dtype == PKV_BF16 ? i4_launch_any<__nv_bfloat16>(a, p, head_dim, rules, s) : i4_launch_any<__half>(a, p, head_dim, rules, s);
        if (e != cudaSuccess) return set_error(PKV_ERR_CUDA, "int4 decode launch: %s", cudaGetErrorString(e));
    }
    return ok();
}
