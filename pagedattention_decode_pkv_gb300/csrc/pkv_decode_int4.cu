// Decode attention over the 4-bit paged cache (pkv_int4.cuh has the format).
//
// With codes c and scales s of 32-dim groups g, per query head
//     S_t = scale sum_g ks_{t,g} (q_g . kc_{t,g}),   out = sum_t p_t vs_{t,g} vc_t / sum_t p_t,
// p the softmax of S (after the score rules), kept as a running maximum, sum and accumulator.
//
// A KV head of a token is 144 bytes of K and V at head_dim 128 where 16 bits take 512, so the
// arithmetic that a byte feeds is 3.6 times that of the 16-bit kernel and the kernel is built
// to keep it small:
//   * K enters the products as it unpacks, f16 1024 + u (and 1024 + 16 u under q / 16): five
//     operations for eight codes.  What 1024 + 8 adds is a constant per query and group, the
//     accumulator's start, so the codes are never corrected; f32 sums of some 2^12 |q| carry
//     it with an error of 2^-12 of a code step.
//   * A group's scale multiplies its partial score in f32 (two products of 16 dims each).
//   * V codes are widened exactly and multiplied by their scales, which is exact in f16 too
//     (eight significant bits), so that P, rounded once to f16, is the only rounding.
//   * The transposed fragments of V come from ldmatrix.trans on 16-bit units: four dims of a
//     token each, two tokens in a register, which is the pair the product wants.
//
// A warp works alone: it takes its own slice of the launch's (unit, 32-token step) list, a unit
// being a (sequence, KV head, up to 8 of its query heads), copies its steps by cp.async into a
// ring of its own and never meets another warp.  The list is cut evenly, whatever the mix of
// lengths; a unit that several warps share leaves a piece (max, sum, accumulator) each, which a
// second kernel joins.
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

constexpr int kI4Step = 32;          // tokens of a step
constexpr int kI4MaxSeqs = 512;      // sequences of a launch (shared-memory prefix)
constexpr int kI4MaxWarps = 152 * 16;  // working warps of a launch (sizes the workspace)
constexpr int kI4MinSteps = 2;       // steps that a working warp takes at least
constexpr int kI4Heads = 8;          // query heads of a unit
constexpr float kI4Log2e = 1.4426950408889634f;

struct I4Args {
    void *out;
    const void *q;
    const uint8_t *k_cache, *v_cache;
    const __half *k_scale, *v_scale;
    const int32_t *block_tables, *context_lens, *key_starts;
    const float *slopes;
    int32_t max_blocks, B, Hq, Hkv, G, subs, bs, num_blocks, max_ctx;
    float scale_log2, softcap;
    float *o_piece;    // [slots][NG * 8][32]
    float2 *ml_piece;  // [slots][8]
    int2 *unit_info;   // [units]: first and last warp
    int32_t *err_flag;
};

__device__ __forceinline__ int64_t i4_div(int64_t a, int64_t b) {  // a >= 0, b > 0
    if (((a | b) >> 32) == 0) return static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
    return a / b;
}

// 16 bytes from global to shared memory, zeros when `bytes` is 0 (nothing is read then).
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

template <int D> struct I4Ring {
    static constexpr int NG = D / 32;              // groups, and 16-byte chunks of a row
    static constexpr int kCodes = kI4Step * D / 2;
    static constexpr int kScales = kI4Step * NG * 2;
    static constexpr int kStage = 2 * (kCodes + kScales);  // K codes, V codes, K scales, V scales
};

template <typename T, int D, int WARPS, int STAGES, int CTAS, bool MOD>
__global__ void __launch_bounds__(WARPS * 32, CTAS)
decode_int4_kernel(const __grid_constant__ I4Args A) {
    using R = I4Ring<D>;
    using H = Half16<__half>;
    constexpr int NG = R::NG;
    extern __shared__ __align__(128) uint8_t smem[];
    int64_t *pref = reinterpret_cast<int64_t *>(smem + WARPS * STAGES * R::kStage);  // [B + 1] steps of a head's sequences before b
    int32_t *cx = reinterpret_cast<int32_t *>(pref + kI4MaxSeqs + 1);                // context length (0: nothing visible)
    int32_t *fk = cx + kI4MaxSeqs;                                                   // MOD: first visible key
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int B = A.B, bs = A.bs;
    for (int b = threadIdx.x; b < B; b += WARPS * 32) {
        const int ctx = A.context_lens[b];
        const bool good = ctx >= 0 && ctx <= A.max_ctx && static_cast<int64_t>(ctx) <= static_cast<int64_t>(A.max_blocks) * bs;
        const int first = MOD && A.key_starts ? max(A.key_starts[b], 0) : 0;
        const bool any = good && ctx > first;
        cx[b] = any ? ctx : 0;
        if (MOD) fk[b] = any ? first : 0;
        if (!any && b % gridDim.x == blockIdx.x) {  // a row of zeros
            if (!good && A.err_flag) atomicOr(A.err_flag, PKV_ERRBIT_CONTEXT);
            uint4 *o = reinterpret_cast<uint4 *>(static_cast<T *>(A.out) + static_cast<int64_t>(b) * A.Hq * D);
            for (int i = 0; i < A.Hq * D / 8; ++i) o[i] = make_uint4(0, 0, 0, 0);
        }
    }
    __syncthreads();
    auto steps_of = [&](int b) -> int64_t {
        return (cx[b] + kI4Step - 1) / kI4Step - (MOD ? fk[b] / kI4Step : 0);
    };
    if (warp == 0) {
        const int chunk = (B + 31) / 32, lo = min(lane * chunk, B), hi = min(lo + chunk, B);
        int64_t sum = 0;
        for (int b = lo; b < hi; ++b) sum += steps_of(b);
        int64_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        int64_t run = incl - sum;
        for (int b = lo; b < hi; ++b) {
            pref[b] = run;
            run += steps_of(b);
        }
        if (lane == 31) pref[B] = incl;
    }
    __syncthreads();
    const int HU = A.Hkv * A.subs;  // units of a sequence
    const int64_t W = pref[B] * HU;
    int64_t Cw = W / kI4MinSteps;
    const int64_t all = static_cast<int64_t>(gridDim.x) * WARPS;
    Cw = Cw > all ? all : Cw < 1 ? 1 : Cw;
    // neighbouring slices go to different SMs, so that a launch of few slices uses them all
    const int64_t me = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
    if (me >= Cw || W == 0) return;
    const int64_t s0 = i4_div(W * me, Cw), s1 = i4_div(W * (me + 1), Cw);

    // Cursor: sequence b, unit hu of it, step st of n.
    struct Cursor { int b, hu, st, n; };
    Cursor cur;
    {
        int lo = 0, hi = B - 1;  // the largest b with HU pref[b] <= s0
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pref[mid] * HU <= s0) lo = mid; else hi = mid - 1;
        }
        const int64_t n = pref[lo + 1] - pref[lo], off = s0 - pref[lo] * HU;
        cur.b = lo;
        cur.n = static_cast<int>(n);
        cur.hu = static_cast<int>(i4_div(off, n));
        cur.st = static_cast<int>(off - cur.hu * n);
    }
    auto advance = [&](Cursor &c) {  // true at the start of a unit
        if (++c.st < c.n) return false;
        c.st = 0;
        if (++c.hu == HU) {
            c.hu = 0;
            do {
                ++c.b;
                c.n = c.b < B ? static_cast<int>(pref[c.b + 1] - pref[c.b]) : 1;
            } while (c.b < B && c.n == 0);
        }
        return true;
    };

    // ---- copies: lane l takes 16-byte chunks of codes and one of scales; the table entries of
    // a step's two halves of 16 tokens (one block each) are loaded a step ahead
    const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(warp) * STAGES * R::kStage;
    Cursor ld = cur;
    int next_id = -1;
    bool bad = false;
    auto position = [&](const Cursor &c) { return (c.st + (MOD ? fk[c.b] / kI4Step : 0)) * kI4Step; };
    auto fetch_id = [&](const Cursor &c) {  // lane h < 2: half h
        next_id = -2;                       // behind the context
        if (lane < 2 && c.b < B) {
            const int pos = position(c) + 16 * lane;
            const bool seen = pos < cx[c.b] && (!MOD || pos + 16 > fk[c.b]);
            if (seen) next_id = A.block_tables[static_cast<int64_t>(c.b) * A.max_blocks + pos / bs];
        }
    };
    constexpr int kRowsPer = 32 / NG;                 // rows that one copy instruction covers
    constexpr int kCopies = kI4Step / kRowsPer;
    static_assert(kRowsPer <= 16 && kI4Step * NG * 2 / 16 <= 32, "lanes of the copies");
    auto swizzled = [](int row, int c) { return (c ^ ((row * NG / 8) & (NG - 1))) << 4; };
    auto issue = [&](int slot) {
        const int kh = ld.hu / A.subs, pos = position(ld);
        const uint32_t dst = ring + static_cast<uint32_t>(slot) * R::kStage;
        int64_t row[2];
        bool ok[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int id = __shfl_sync(0xffffffffu, next_id, h);
            ok[h] = id >= 0 && id < A.num_blocks;
            bad = bad || (!ok[h] && id != -2);
            const int p = pos + 16 * h;
            row[h] = ok[h] ? (static_cast<int64_t>(id) * A.Hkv + kh) * bs + p % bs : 0;
        }
        const int c = lane & (NG - 1), r0 = lane / NG;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int h = i * kRowsPer / 16, r = i * kRowsPer + r0;
            const int64_t src = (row[h] + (r - 16 * h)) * (D / 2) + 16 * c;
            const uint32_t d = dst + r * (D / 2) + swizzled(r, c), bytes = ok[h] ? 16 : 0;
            cp16(d, A.k_cache + (ok[h] ? src : 0), bytes);
            cp16(d + R::kCodes, A.v_cache + (ok[h] ? src : 0), bytes);
        }
        // scales: 16 tokens x NG x 2 bytes of a half are NG * 2 chunks
        constexpr int kChunks = kI4Step * NG * 2 / 16;  // both halves
        if (lane < kChunks) {
            const int h = lane / (kChunks / 2), k = lane - h * (kChunks / 2);
            const int64_t src = (h ? row[1] : row[0]) * NG + 8 * k;
            const bool o = h ? ok[1] : ok[0];
            cp16(dst + 2 * R::kCodes + 16 * lane, A.k_scale + (o ? src : 0), o ? 16 : 0);
            cp16(dst + 2 * R::kCodes + R::kScales + 16 * lane, A.v_scale + (o ? src : 0), o ? 16 : 0);
        }
        advance(ld);
        fetch_id(ld);
        return (ok[0] ? 1 : 0) | (ok[1] ? 2 : 0);
    };
    uint32_t oks = 0;  // two bits a ring slot: the halves that were there
    fetch_id(ld);
    int64_t issued = s0;
    auto issue_next = [&] {
        if (issued < s1) {
            const int slot = static_cast<int>((issued - s0) % STAGES);
            oks = (oks & ~(3u << 2 * slot)) | static_cast<uint32_t>(issue(slot)) << 2 * slot;
        }
        ++issued;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue_next();

    // ---- a unit's queries: lane (g = head, t): dims 8 t .. 8 t + 7 of every group, f16 under a power of two
    const int g = lane >> 2, t = lane & 3, mi = lane >> 3, r8 = lane & 7;
    uint32_t qf[NG][4];
    float off[NG][2];            // start of the group's accumulator, heads 2 t and 2 t + 1
    float sl0 = 0.f, sl1 = 0.f;  // scores to log2 units, of heads 2 t, 2 t + 1
    float slope0 = 0.f, slope1 = 0.f;
    int heads = 0;
    int64_t head0 = 0;  // first query head's row of q and out
    auto load_q = [&](const Cursor &c) {
        const int kh = c.hu / A.subs, sub = c.hu - kh * A.subs;
        heads = min(kI4Heads, A.G - sub * kI4Heads);
        head0 = static_cast<int64_t>(c.b) * A.Hq + kh * A.G + sub * kI4Heads;
        const bool live = g < heads;
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(A.q) + (head0 + (live ? g : 0)) * D) + t;
        uint4 x[NG];
        float top = 0.f;
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) x[gg] = live ? __ldg(src + 4 * gg) : make_uint4(0, 0, 0, 0);
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
        // the largest value to [8, 16): all of a 16-bit type's bits down to 2^-17 of it, q / 16 included
        const int e = static_cast<int>(__float_as_uint(top) >> 23);
        const int k2 = e == 0 || e == 255 ? 0 : min(max(130 - e, -120), 120);
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
                a = fmaf(v.x + v.y, j & 1 ? -1152.f : -1032.f, a);
            }
            a += __shfl_xor_sync(0xffffffffu, a, 1);
            a += __shfl_xor_sync(0xffffffffu, a, 2);
            start[gg] = a;
        }
        const float sl = A.scale_log2 * back;
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
    float m0, m1, l0, l1;
    bool fresh = true;   // the next step starts a unit
    bool whole = false;  // the unit began in this slice
    for (int64_t s = s0; s < s1; ++s) {
        if (fresh) {
            load_q(cur);
#pragma unroll
            for (int gg = 0; gg < NG; ++gg)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[gg][e][c] = 0.f;
            m0 = m1 = -INFINITY;
            l0 = l1 = 0.f;
            whole = cur.st == 0;
            if (lane == 0 && whole) A.unit_info[static_cast<int64_t>(cur.b) * HU + cur.hu].x = static_cast<int>(me);
            fresh = false;
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
        __syncwarp();
        issue_next();  // into the slot of the step before this one
        const int slot = static_cast<int>((s - s0) % STAGES);
        const uint32_t base = ring + static_cast<uint32_t>(slot) * R::kStage;
        const int pos = position(cur), ctx = cx[cur.b], first = MOD ? fk[cur.b] : 0;
        const uint32_t here = oks >> 2 * slot & 3;
        const bool partial = pos + kI4Step > ctx || (MOD && pos < first) || here != 3;
        auto seen = [&](int k) {  // token k of the step
            return pos + k < ctx && (!MOD || pos + k >= first) && (here >> (k >> 4) & 1);
        };

        // 1. scores, two tiles of 16 tokens: rows (tokens) g and g + 8, columns (heads) 2 t, 2 t + 1
        float y[2][4];
#pragma unroll
        for (int tile = 0; tile < 2; ++tile) {
            uint32_t w[NG][2];  // word t of group gg, of tokens g and g + 8
#pragma unroll
            for (int gg = 0; gg < NG; gg += 2) {
                const int row = 16 * tile + r8 + 8 * (mi & 1);
                uint32_t x[4];
                ldsm_x4(base + row * (D / 2) + swizzled(row, gg + (mi >> 1)), x);
                w[gg][0] = x[0];
                w[gg][1] = x[1];
                w[gg + 1][0] = x[2];
                w[gg + 1][1] = x[3];
            }
            uint32_t sa[NG / 2], sb[NG / 2];  // scales of tokens g and g + 8
            const uint32_t ks = base + 2 * R::kCodes + (16 * tile + g) * (NG * 2);
#pragma unroll
            for (int i = 0; i < NG / 2; ++i) {
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sa[i]) : "r"(ks + 4 * i));
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sb[i]) : "r"(ks + 8 * NG * 2 + 4 * i));
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) y[tile][c] = 0.f;
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) {
                float acc[4] = {off[gg][0], off[gg][1], off[gg][0], off[gg][1]};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t a[4];
                    const uint32_t x0 = e ? w[gg][0] >> 8 : w[gg][0], x1 = e ? w[gg][1] >> 8 : w[gg][1];
                    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(a[0]) : "r"(x0));
                    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(a[1]) : "r"(x1));
                    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(a[2]) : "r"(x0));
                    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(a[3]) : "r"(x1));
                    H::mma(acc, a, qf[gg][2 * e], qf[gg][2 * e + 1]);
                }
                const float2 fa = __half22float2(*reinterpret_cast<const __half2 *>(&sa[gg / 2]));
                const float2 fb = __half22float2(*reinterpret_cast<const __half2 *>(&sb[gg / 2]));
                const float s_a = gg & 1 ? fa.y : fa.x, s_b = gg & 1 ? fb.y : fb.x;
                y[tile][0] = fmaf(s_a, acc[0], y[tile][0]);
                y[tile][1] = fmaf(s_a, acc[1], y[tile][1]);
                y[tile][2] = fmaf(s_b, acc[2], y[tile][2]);
                y[tile][3] = fmaf(s_b, acc[3], y[tile][3]);
            }
        }
        // 2. log2 units, score rules, masks
#pragma unroll
        for (int tile = 0; tile < 2; ++tile) {
            y[tile][0] *= sl0;
            y[tile][1] *= sl1;
            y[tile][2] *= sl0;
            y[tile][3] *= sl1;
            if constexpr (MOD) {
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
            for (int tile = 0; tile < 2; ++tile) {
                const bool a = seen(16 * tile + g), b = seen(16 * tile + g + 8);
                y[tile][0] = a ? y[tile][0] : -INFINITY;
                y[tile][1] = a ? y[tile][1] : -INFINITY;
                y[tile][2] = b ? y[tile][2] : -INFINITY;
                y[tile][3] = b ? y[tile][3] : -INFINITY;
            }
        }
        // 3. running maximum; the accumulator moves when it does
        float mx0 = fmaxf(fmaxf(y[0][0], y[0][2]), fmaxf(y[1][0], y[1][2]));
        float mx1 = fmaxf(fmaxf(y[0][1], y[0][3]), fmaxf(y[1][1], y[1][3]));
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, sh));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, sh));
        }
        if (__any_sync(0xffffffffu, mx0 > m0 || mx1 > m1)) {
            const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
            const float a0 = n0 == -INFINITY ? 1.f : fast_exp2(m0 - n0), a1 = n1 == -INFINITY ? 1.f : fast_exp2(m1 - n1);
            m0 = n0;
            m1 = n1;
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
        const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
        // 4. P and O += P V
#pragma unroll
        for (int tile = 0; tile < 2; ++tile) {
            const float p0 = fast_exp2(y[tile][0] - b0), p1 = fast_exp2(y[tile][1] - b1);
            const float p2 = fast_exp2(y[tile][2] - b0), p3 = fast_exp2(y[tile][3] - b1);
            l0 += p0 + p2;
            l1 += p1 + p3;
            const uint32_t pb0 = movmatrix_trans(H::pack(p0, p1)), pb1 = movmatrix_trans(H::pack(p2, p3));
            // scales of tokens 2 t, 2 t + 1 (words 0 .. NG - 1) and of those 8 further
            uint32_t va[NG], vb[NG];
            const uint32_t vs = base + 2 * R::kCodes + R::kScales + (16 * tile + 2 * t) * (NG * 2);
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(va[i]) : "r"(vs + 4 * i));
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(vb[i]) : "r"(vs + 8 * NG * 2 + 4 * i));
            }
            if (partial) {  // scales of rows that are not seen may be anything, P there is 0: their product must be 0
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    const int k = 16 * tile + 2 * t + (i >= NG / 2 ? 1 : 0);
                    va[i] = seen(k) ? va[i] : 0u;
                    vb[i] = seen(k + 8) ? vb[i] : 0u;
                }
            }
#pragma unroll
            for (int gg = 0; gg < NG; gg += 2) {
                uint32_t w[4];  // (tokens 0 .. 7 | 8 .. 15) of groups gg, gg + 1
                const int row = 16 * tile + r8 + 8 * (mi & 1);
                ldsm_x4_trans(base + R::kCodes + row * (D / 2) + swizzled(row, gg + (mi >> 1)), w);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t sel = h ? 0x7632 : 0x5410;  // (scale of token 2 t, of 2 t + 1)
                    const uint32_t s_a = __byte_perm(va[gg / 2], va[NG / 2 + gg / 2], sel);
                    const uint32_t s_b = __byte_perm(vb[gg / 2], vb[NG / 2 + gg / 2], sel);
                    uint32_t xa[4], xb[4];
                    int4_widen(w[2 * h], xa);
                    int4_widen(w[2 * h + 1], xb);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t a[4] = {mul_f16x2(xa[2 * e], s_a), mul_f16x2(xa[2 * e + 1], s_a),
                                               mul_f16x2(xb[2 * e], s_b), mul_f16x2(xb[2 * e + 1], s_b)};
                        H::mma(o[gg + h][e], a, pb0, pb1);
                    }
                }
            }
        }
        const Cursor at = cur;
        if (advance(cur) || s + 1 == s1) {
            // the unit ends, or the slice does
            fresh = true;
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, sh);
                l1 += __shfl_xor_sync(0xffffffffu, l1, sh);
            }
            const bool ends = at.st == at.n - 1;
            const int64_t u = static_cast<int64_t>(at.b) * HU + at.hu;
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
            } else if (hA < heads) {
                const int64_t piece = me + u;
                float *po = A.o_piece + piece * (NG * 8 * 32) + lane;
#pragma unroll
                for (int gg = 0; gg < NG; ++gg)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int c = 0; c < 4; ++c) po[((gg * 2 + e) * 4 + c) * 32] = o[gg][e][c];
                if (g == 0) {
                    A.ml_piece[piece * kI4Heads + hA] = make_float2(m0, l0);
                    A.ml_piece[piece * kI4Heads + hB] = make_float2(m1, l1);
                }
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (bad && A.err_flag) atomicOr(A.err_flag, PKV_ERRBIT_BLOCK_RANGE);
}

// Joins a unit's pieces: out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k.  A warp takes one
// (unit, group, half) of the accumulator in the layout the pieces are in.
constexpr int kI4JoinWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kI4JoinWarps * 32)
decode_int4_join_kernel(const __grid_constant__ I4Args A, int64_t units) {
    constexpr int NG = D / 32, kParts = NG * 2;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kI4JoinWarps + (threadIdx.x >> 5);
    const int64_t u = item / kParts;
    const int part = static_cast<int>(item - u * kParts);
    if (u >= units) return;
    const int HU = A.Hkv * A.subs;
    const int b = static_cast<int>(u / HU), hu = static_cast<int>(u - static_cast<int64_t>(b) * HU);
    const int kh = hu / A.subs, sub = hu - kh * A.subs, heads = min(kI4Heads, A.G - sub * kI4Heads);
    const int ctx = A.context_lens[b], first = A.key_starts ? max(A.key_starts[b], 0) : 0;
    const int2 ui = A.unit_info[u];
    if (ctx <= first || ctx > A.max_ctx || static_cast<int64_t>(ctx) > static_cast<int64_t>(A.max_blocks) * A.bs) return;  // zeros already
    if (ui.x >= ui.y || 2 * t >= heads) return;  // one piece: written by the main kernel
    constexpr int U = 8;
    float M0 = -INFINITY, M1 = -INFINITY, L0 = 0.f, L1 = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int w = ui.x; w <= ui.y; w += U) {
        float v[U][4];
        float4 ml[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t piece = w + i + u;
            const bool in = w + i <= ui.y;
            ml[i] = in ? __ldg(reinterpret_cast<const float4 *>(A.ml_piece + piece * kI4Heads + 2 * t)) : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
#pragma unroll
            for (int c = 0; c < 4; ++c) v[i][c] = in ? __ldg(A.o_piece + piece * (NG * 8 * 32) + (part * 4 + c) * 32 + lane) : 0.f;
        }
        float n0 = M0, n1 = M1;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            n0 = fmaxf(n0, ml[i].x);
            n1 = fmaxf(n1, ml[i].z);
        }
        const float r0 = n0 == -INFINITY ? 0.f : n0, r1 = n1 == -INFINITY ? 0.f : n1;
        const float a0 = exp2f(M0 - r0), a1 = exp2f(M1 - r1);
        M0 = n0;
        M1 = n1;
        L0 *= a0;
        L1 *= a1;
        acc[0] *= a0;
        acc[1] *= a1;
        acc[2] *= a0;
        acc[3] *= a1;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const float w0 = exp2f(ml[i].x - r0), w1 = exp2f(ml[i].z - r1);
            L0 = fmaf(w0, ml[i].y, L0);
            L1 = fmaf(w1, ml[i].w, L1);
            acc[0] = fmaf(w0, v[i][0], acc[0]);
            acc[1] = fmaf(w1, v[i][1], acc[1]);
            acc[2] = fmaf(w0, v[i][2], acc[2]);
            acc[3] = fmaf(w1, v[i][3], acc[3]);
        }
    }
    const float i0 = L0 > 0.f ? 1.f / L0 : (L0 == L0 ? 0.f : L0), i1 = L1 > 0.f ? 1.f / L1 : (L1 == L1 ? 0.f : L1);
    const int gg = part >> 1, e = part & 1, d = 32 * gg + 8 * (g >> 1) + (g & 1) + 4 * e, hA = 2 * t;
    T *out = static_cast<T *>(A.out) + (static_cast<int64_t>(b) * A.Hq + kh * A.G + sub * kI4Heads + hA) * D + d;
    out[0] = from_f32<T>(acc[0] * i0);
    out[2] = from_f32<T>(acc[2] * i0);
    if (hA + 1 < heads) {
        out[D] = from_f32<T>(acc[1] * i1);
        out[D + 2] = from_f32<T>(acc[3] * i1);
    }
}

// ----------------------------------------------------------------------------- host side
struct I4Plan {
    int32_t subs = 1, group = 0;  // units of a KV head, sequences of a launch
    int64_t units = 0;            // of a launch
    size_t o_bytes = 0, ml_bytes = 0, ws_bytes = 0;
};

bool i4_shape(int32_t d) { return d == 64 || d == 128 || d == 256; }

I4Plan i4_plan(int32_t B, int32_t Hq, int32_t Hkv, int32_t d) {
    I4Plan p;
    p.subs = (Hq / Hkv + kI4Heads - 1) / kI4Heads;
    p.group = B < kI4MaxSeqs ? B : kI4MaxSeqs;
    p.units = static_cast<int64_t>(p.group) * Hkv * p.subs;
    const int64_t slots = kI4MaxWarps + p.units;
    p.o_bytes = static_cast<size_t>(slots) * d * kI4Heads * sizeof(float);
    p.ml_bytes = static_cast<size_t>(slots) * kI4Heads * sizeof(float2);
    p.ws_bytes = p.o_bytes + p.ml_bytes + (static_cast<size_t>(p.units) * sizeof(int2) + 255) / 256 * 256;
    return p;
}

template <typename T, int D, bool MOD>
cudaError_t i4_launch(const I4Args &a, const I4Plan &p, cudaStream_t stream) {
    constexpr int WARPS = 4, STAGES = D == 256 ? 2 : 3, CTAS = D == 256 ? 2 : 3;
    constexpr int smem = WARPS * STAGES * I4Ring<D>::kStage + (kI4MaxSeqs + 1) * 8 + kI4MaxSeqs * 8;
    auto kern = decode_int4_kernel<T, D, WARPS, STAGES, CTAS, MOD>;
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
    e = launch_pdl(kPdlDecode, kern, dim3(grid), dim3(WARPS * 32), smem, stream, a);
    if (e != cudaSuccess) return e;
    const int64_t units = static_cast<int64_t>(a.B) * a.Hkv * a.subs, items = units * (D / 16);
    return launch_pdl(kPdlCombine, decode_int4_join_kernel<T, D>, dim3(static_cast<unsigned>((items + kI4JoinWarps - 1) / kI4JoinWarps)),
                      dim3(kI4JoinWarps * 32), 0, stream, a, units);
}

template <typename T, bool MOD>
cudaError_t i4_launch_d(const I4Args &a, const I4Plan &p, int32_t d, cudaStream_t s) {
    return d == 64 ? i4_launch<T, 64, MOD>(a, p, s) : d == 128 ? i4_launch<T, 128, MOD>(a, p, s) : i4_launch<T, 256, MOD>(a, p, s);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_paged_attention_decode_int4_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                                                 int32_t head_dim) {
    if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || !i4_shape(head_dim)) return 0;
    return i4_plan(num_seqs, num_q_heads, num_kv_heads, head_dim).ws_bytes;
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
    if (max_context_len > INT32_MAX - kI4Step) return set_error(PKV_ERR_INVALID_ARG, "int4 decode: max_context_len is too long");
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
    const I4Plan p = i4_plan(num_seqs, num_q_heads, num_kv_heads, head_dim);
    if (!workspace || workspace_bytes < p.ws_bytes || !aligned(workspace, 256))
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
    const bool rules = m.softcap > 0.f || m.alibi_slopes || m.key_starts;
    for (int32_t b0 = 0; b0 < num_seqs; b0 += p.group) {  // consecutive launches, one workspace
        const int64_t at = static_cast<int64_t>(b0) * num_q_heads * head_dim * 2;
        a.out = static_cast<char *>(out) + at;
        a.q = static_cast<const char *>(q) + at;
        a.block_tables = block_tables + static_cast<int64_t>(b0) * max_blocks_per_seq;
        a.context_lens = context_lens + b0;
        a.key_starts = m.key_starts ? m.key_starts + b0 : nullptr;
        a.B = num_seqs - b0 < p.group ? num_seqs - b0 : p.group;
        auto s = static_cast<cudaStream_t>(stream);
        const cudaError_t e = dtype == PKV_BF16 ? (rules ? i4_launch_d<__nv_bfloat16, true>(a, p, head_dim, s) : i4_launch_d<__nv_bfloat16, false>(a, p, head_dim, s))
                                                : (rules ? i4_launch_d<__half, true>(a, p, head_dim, s) : i4_launch_d<__half, false>(a, p, head_dim, s));
        if (e != cudaSuccess) return set_error(PKV_ERR_CUDA, "int4 decode launch: %s", cudaGetErrorString(e));
    }
    return ok();
}
