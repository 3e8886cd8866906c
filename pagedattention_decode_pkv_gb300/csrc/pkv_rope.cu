// Rotary positions with the cache write, and the 4-bit cache written and read back.
//
// Pair i of a head, (x_a, x_b) at dims (i, i + r/2) or (2 i, 2 i + 1) of the first r, turns by
// the angle position * f_i:
//     y_a = A (x_a cos - x_b sin),   y_b = A (x_b cos + x_a sin),
// the other dims pass.  One call rotates the step's queries, and rotates and stores its keys
// with the values beside them: what a step writes is read once and written once.
//
// Angles.  f_i comes as turns per position in 64-bit fixed point, so position * f_i modulo one
// turn is an integer product that loses nothing, however far the position; its upper half, cut
// to the nearest quarter turn, is at most 2^-24 of an eighth off as an f32 (an f32 product
// would be off by 2^-24 of the position in radians).  Then one sincospif a pair, shared by all
// heads of the token.
//
// 4-bit rows (pkv_int4.cuh) are quantised from the rotated values themselves.  The definition
// rounds exact values; the f32 rotation is off by at most kRotError (|x_a| + |x_b|) A, so a
// pair with a value (or a group maximum) that close to a rounding border is turned again in
// f64, a few of a thousand.
//
// A warp takes a token's heads, a lane 16 dims of a head.  Measured with heads of 128 dims, on the GPU:
//   * 16-bit rows are bound by HBM, four steps of heads loaded before the first is used: 16381 tokens of
//     32 + 2 x 8 heads 66 us, 6.1 TB/s.
//   * 4-bit rows are bound by the chain and the issue of the quantisation (55 % of the issue slots, 14
//     warps an SM at 128 registers): 32700 tokens of 32 + 2 x 8 heads, bf16, 150 us, 4.7 TB/s; 5003 rows of
//     32 heads, not rotated, 35 us, 3.0 TB/s.
//   * A step of 64 tokens is its launch and one chain of loads, 6.3 us.
//   * Reading back is bound by HBM, and by where the rows lie: 131001 tokens of 8 heads, bf16, by whole
//     blocks 107 us, 6.4 TB/s; anywhere in the pool 137 us, for DRAM reads 361 MB where the rows are 151.
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "pkv_int4.cuh"
#include "pkv_internal.h"
#include "pkv_pack.cuh"
#include "pkv_pdl.cuh"

namespace pkv {
namespace {

constexpr int kRopeThreads = 128, kRopeWarps = kRopeThreads / 32;
constexpr int kRopeMaxDim = 512;           // fast kernels: head_dim / 16 lanes a head
constexpr int kRopeGenericMaxDim = 1024;   // generic kernel: a row in shared memory
constexpr int64_t kRopeMaxCtas = 1 << 20;  // of a grid; the rest is looped over
constexpr int64_t kRopeFullWarps = 152 * 64;  // warps that fill the GPU
// Largest error of a rotated f32 value over (|x_a| + |x_b|) A: sincospif 2 ulp, the angle one
// rounding, A, two products and a sum: below 7 x 2^-24, taken as 16.
constexpr float kRotError = 9.5367431640625e-7f;

struct RopeArgs {
    const void *q, *key, *value;
    void *q_out, *k_cache, *v_cache;
    __half *k_scale, *v_scale;
    const int32_t *positions, *slots;
    const uint64_t *turns;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    int64_t num_tokens, num_slots;
    double amplitude;
    float amp;
    int32_t Hq, Hkv, d, r, bs, inter;
    int32_t parts, steps_per_part;
    int32_t *err_flag;
};

template <typename T> __device__ __forceinline__ float widen(T x);
template <> __device__ __forceinline__ float widen<float>(float x) { return x; }
template <> __device__ __forceinline__ float widen<__half>(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T narrow(float x);
template <> __device__ __forceinline__ float narrow<float>(float x) { return x; }
template <> __device__ __forceinline__ __half narrow<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Eight consecutive elements, as 16-byte words.
template <typename T> struct Eight {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) w[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) reinterpret_cast<uint4 *>(p)[i] = w[i];
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) w[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const T *e = reinterpret_cast<const T *>(w);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = widen<T>(e[k]);
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
        T *e = reinterpret_cast<T *>(w);
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = narrow<T>(x[k]);
    }
};

// (cos, sin) of `position` times a frequency in turns, to f32.
__device__ __forceinline__ float2 turn_cos_sin(int32_t position, uint64_t turns) {
    const uint64_t p = static_cast<uint64_t>(static_cast<int64_t>(position)) * turns;
    const uint32_t u = static_cast<uint32_t>(p >> 32);
    const uint32_t quarter = (u + (1u << 29)) >> 30;
    const float half_turns = static_cast<float>(static_cast<int32_t>(u - (quarter << 30))) * 4.656612873077393e-10f;  // 2^-31
    float s, c;
    sincospif(half_turns, &s, &c);
    const float cc = quarter & 1 ? -s : c, ss = quarter & 1 ? c : s;
    return quarter & 2 ? make_float2(-cc, -ss) : make_float2(cc, ss);
}

// The rotated pair in f64, for values next to a border.
__device__ __noinline__ double2 rotate_exact(int32_t position, uint64_t turns, double amplitude, float a, float b) {
    const int64_t p = static_cast<int64_t>(static_cast<uint64_t>(static_cast<int64_t>(position)) * turns);
    double s, c;
    sincospi(static_cast<double>(p) * 1.0842021724855044e-19, &s, &c);  // 2^-63: half turns
    s *= amplitude;
    c *= amplitude;
    return make_double2(a * c - b * s, b * c + a * s);
}

// int4_scale of an f64 maximum.
__device__ __forceinline__ __half int4_scale_f64(double top) {
    if (!(top < kInt4TopInput)) return __float2half_rn(kInt4TopScale);
    float mid;
    int4_seventh_bf16(static_cast<float>(top), mid);
    const uint32_t lo = __float_as_uint(mid) & 0xffff0000u;
    const double side = fma(-7.0, static_cast<double>(mid), top);
    const bool up = side > 0.0 || (side == 0.0 && (lo & 0x10000u));
    return __float2half_rn(fminf(__uint_as_float(up ? lo + 0x10000u : lo), kInt4TopScale));
}

__device__ __forceinline__ int int4_code_f64(double x, float s) {
    if (x != x) return 0;
    return static_cast<int>(fmin(fmax(rint(x / static_cast<double>(s)), -7.0), 7.0));
}

// The largest magnitude of eight values, NaN if one is.
__device__ __forceinline__ float max_abs8(const float (&x)[8]) {
    float m = fabsf(x[0]);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(x[1])));
#pragma unroll
    for (int k = 2; k < 8; k += 2) asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(x[k])), "f"(fabsf(x[k + 1])));
    return m;
}

// The word of eight values (no NaN, none beyond 7 s) under the scale s (inv = 1 / s, 0 for a zero
// scale), two values an operation.  `snap` 384 rounds x inv to multiples of 2^-15 first: of 16-bit
// values (11 bits over the scale's 8) a quotient is a tie or 2^-13 away from one, and a tie may
// come out of the rounded inv a little off it; then it is one again and goes to even.  With 0 a
// product next to a border may fall to either side: `near` becomes the smallest distance of
// |x - c s| from half a step.
template <bool NEAR>
__device__ __forceinline__ uint32_t int4_word(const float (&x)[8], float s, float inv, float snap, float &near) {
    const uint64_t inv2 = splat2(inv), on = splat2(snap), off = splat2(-snap);
    const uint64_t magic = splat2(12582912.f), back = splat2(-12582912.f);  // 1.5 x 2^23: a sum with it is an integer
    uint64_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint64_t v = pack2(x[2 * j], x[2 * j + 1]);
        c[j] = add2(add2(add2(fma2(v, inv2, on), off), magic), back);
        if constexpr (NEAR) {
            float r0, r1;
            unpack2(fma2(c[j], splat2(-s), v), r0, r1);
            near = fminf(near, fminf(fabsf(fabsf(r0) - 0.5f * s), fabsf(fabsf(r1) - 0.5f * s)));
        }
    }
    // both halves of the word at once: nibble j is dim 2 j below and dim 2 j + 1 above; 2^23 + 0x8888: all
    // + 8, and the integer in the low bits
    const uint64_t sum = fma2(c[3], splat2(4096.f), fma2(c[2], splat2(256.f), fma2(c[1], splat2(16.f), c[0])));
    float lo, hi;
    unpack2(add2(sum, splat2(8423560.f)), lo, hi);
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410);
}

// w with the nibble at `shift` as the code of z under s > 0: next to z / s to f32, then by the exact
// remainder.  (Of a pair that cancels, the f32 rotation may have been off by any number of codes.)
__device__ __noinline__ uint32_t int4_settled(uint32_t w, int shift, double z, float s) {
    float c = rintf(fminf(fmaxf(static_cast<float>(z) * __frcp_rn(s), -8.f), 8.f));
    const double r = fma(-static_cast<double>(c), static_cast<double>(s), z), h = 0.5 * s;
    if (fabs(r) > h || (fabs(r) == h && (static_cast<int>(c) & 1))) c += r > 0.0 ? 1.f : -1.f;
    const int to = z == z ? static_cast<int>(fminf(fmaxf(c, -7.f), 7.f)) : 0;
    return w + (static_cast<uint32_t>(to + 8 - static_cast<int>(w >> shift & 15)) << shift);
}

// Whether x lies within `err` of the border between two codes under s.
__device__ __forceinline__ bool int4_near_border(float x, float s, int code, float err) {
    const float r = fmaf(-static_cast<float>(code), s, x);
    return fabsf(fabsf(r) - 0.5f * s) <= err;
}

// ----------------------------------------------------------------------------- fast kernel
// A head is d / 16 lanes of two chunks of eight dims: lane l has chunks 2 l and 2 l + 1 where
// pairs lie side by side, else l and l + r / 16 (a pair's two halves) among the rotated and
// two of the others past them.  Either way its pairs are 8 l .. 8 l + 7 and its groups of 32
// dims are 2 lanes or twice 4 lanes, so a rotation never leaves a lane and a group's maximum
// takes one or two shuffles.
template <typename T, bool INTER, bool Q4>
__global__ void __launch_bounds__(kRopeThreads, Q4 && !INTER ? 4 : 5)
rope_store_kernel(const __grid_constant__ RopeArgs A) {
    constexpr int U = sizeof(T) == 2 ? 4 : 2;  // steps in flight of the queries
    __shared__ __align__(16) float2 table[kRopeWarps][kRopeMaxDim / 2];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d = A.d, r = A.r, lph = d >> 4, hpw = 32 / lph;
    const int hl = lane / lph, l = lane - hl * lph;
    const bool on = hl < hpw;
    int c0, c1;
    if (INTER) {
        c0 = 2 * l;
        c1 = c0 + 1;
    } else {
        const int nr = r >> 4;
        c0 = l < nr ? l : (r >> 3) + l - nr;
        c1 = c0 + (l < nr ? nr : lph - nr);
    }
    const bool rot0 = 8 * c0 < r, rot1 = 8 * c1 < r;
    const int nq = (A.Hq + hpw - 1) / hpw, nk = (A.Hkv + hpw - 1) / hpw, total = nq + 2 * nk;
    const int64_t items = A.num_tokens * A.parts;
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp; item < items;
         item += static_cast<int64_t>(gridDim.x) * kRopeWarps) {
        const int64_t i = item / A.parts;
        const int part = static_cast<int>(item - i * A.parts);
        const int s0 = part * A.steps_per_part, s1 = min(s0 + A.steps_per_part, total);
        const int32_t slot = A.slots[i];
        const int32_t position = r > 0 ? A.positions[i] : 0;
        float cs[8], sn[8];  // of pairs 8 l + k
        bool have = false;
        auto angles = [&] {  // the token's, while the first loads are under way
            if (have || r == 0 || s0 >= nq + nk) return;
            have = true;
            __syncwarp();
            for (int p = lane; 2 * p < r; p += 32) {
                const float2 t = turn_cos_sin(position, A.turns[p]);
                table[warp][p] = make_float2(t.x * A.amp, t.y * A.amp);
            }
            __syncwarp();
            if (rot0 && on) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 t = table[warp][8 * l + k];  // past the last pair (r / 2 not whole lanes): not used
                    cs[k] = t.x;
                    sn[k] = t.y;
                }
            }
        };
        // (a, b), the lane's two chunks, -> (y0, y1)
        auto turn = [&](const float (&a)[8], const float (&b)[8], bool turned, float (&y0)[8], float (&y1)[8]) {
            if (turned) {
                if constexpr (INTER) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        y0[2 * k] = fmaf(a[2 * k], cs[k], -(a[2 * k + 1] * sn[k]));
                        y0[2 * k + 1] = fmaf(a[2 * k + 1], cs[k], a[2 * k] * sn[k]);
                        y1[2 * k] = rot1 ? fmaf(b[2 * k], cs[4 + k], -(b[2 * k + 1] * sn[4 + k])) : b[2 * k];
                        y1[2 * k + 1] = rot1 ? fmaf(b[2 * k + 1], cs[4 + k], b[2 * k] * sn[4 + k]) : b[2 * k + 1];
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {  // two pairs an operation
                        const uint64_t va = pack2(a[k], a[k + 1]), vb = pack2(b[k], b[k + 1]);
                        const uint64_t c = pack2(cs[k], cs[k + 1]), n = pack2(sn[k], sn[k + 1]);
                        unpack2(fma2(va, c, mul2(vb, pack2(-sn[k], -sn[k + 1]))), y0[k], y0[k + 1]);
                        unpack2(fma2(vb, c, mul2(va, n)), y1[k], y1[k + 1]);
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    y0[k] = a[k];
                    y1[k] = b[k];
                }
            }
        };
        const int64_t lane_at = static_cast<int64_t>(hl) * d;  // the lane's head of a step of hpw heads
        const int hop = hpw * d;
        // Steps [from, to) of a token's `heads` heads from src to dst, rotated or as they are.
        auto stream = [&](const T *src, T *dst, int heads, int from, int to, bool turned) {
            // steps of this lane: its head of a step exists
            const int end = on ? min(to, hl < heads ? (heads - 1 - hl) / hpw + 1 : 0) : from;
            src += static_cast<int64_t>(from) * hop;
            dst += static_cast<int64_t>(from) * hop;
            for (int sb = from; sb < to; sb += U) {
                Eight<T> x0[U], x1[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (sb + u < end) {
                        x0[u].load(src + u * hop + 8 * c0);
                        x1[u].load(src + u * hop + 8 * c1);
                    } else {
                        x0[u].clear();
                        x1[u].clear();
                    }
                }
                src += U * hop;
                angles();
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (turned) {  // (in halves both of the lane's chunks)
                        float a[8], b[8], y0[8], y1[8];
                        x0[u].get(a);
                        x1[u].get(b);
                        turn(a, b, true, y0, y1);
                        x0[u].put(y0);
                        x1[u].put(y1);
                    }
                    if (sb + u < end) {
                        x0[u].store(dst + u * hop + 8 * c0);
                        x1[u].store(dst + u * hop + 8 * c1);
                    }
                }
                dst += U * hop;
            }
        };
        const T *key = static_cast<const T *>(A.key) + i * A.k_stride + lane_at;
        const T *value = static_cast<const T *>(A.value) + i * A.v_stride + lane_at;
        Eight<T> n0, n1;
        auto load = [&](int e) {  // step e of the keys, then of the values
            const int step = e < nk ? e : e - nk;
            if (on && step * hpw + hl < A.Hkv) {
                const T *p = (e < nk ? key : value) + static_cast<int64_t>(step) * hop;
                n0.load(p + 8 * c0);
                n1.load(p + 8 * c1);
            } else {
                n0.clear();
                n1.clear();
            }
        };
        if (Q4 && nq < s1) load(max(s0 - nq, 0));  // on its way beside the queries
        if (s0 < nq)
            stream(static_cast<const T *>(A.q) + i * A.q_stride + lane_at, static_cast<T *>(A.q_out) + i * A.Hq * d + lane_at, A.Hq, s0,
                   min(s1, nq), rot0);
        const bool stored = slot >= 0 && slot < A.num_slots;
        if (slot != -1 && !stored && s0 <= nq && nq < s1 && lane == 0 && A.err_flag) atomicOr(A.err_flag, PKV_ERRBIT_SLOT_RANGE);
        if (!stored || s1 <= nq) continue;
        if constexpr (!Q4) {
            const int64_t at = static_cast<int64_t>(slot) * A.Hkv * d + lane_at;
            stream(key, static_cast<T *>(A.k_cache) + at, A.Hkv, max(s0 - nq, 0), min(s1 - nq, nk), rot0);
            stream(value, static_cast<T *>(A.v_cache) + at, A.Hkv, max(s0 - nq - nk, 0), s1 - nq - nk, false);
        } else {
            // Keys and values into codes, the next step's loads under way.  One copy of the code:
            // unrolled over steps it outgrows the instruction caches (32700 tokens of 32 + 2 x 8
            // heads: four copies 394 us with the rows read back, two 274, at that step).
            const int64_t block = slot / A.bs, row0 = block * A.Hkv * A.bs + (slot - block * A.bs);
            const int last = s1 - nq;
            angles();
#pragma unroll 1
            for (int e = max(s0 - nq, 0); e < last; ++e) {
                const int role = e < nk ? 1 : 2, h = (e < nk ? e : e - nk) * hpw + hl;
                const bool live = on && h < A.Hkv, turned = role == 1 && rot0;
                float a[8], b[8], y0[8], y1[8];
                n0.get(a);
                n1.get(b);
                if (e + 1 < last) load(e + 1);
                turn(a, b, turned, y0, y1);
                constexpr int kReach = INTER ? 2 : 4;  // lanes of a group
                const bool loose0 = turned, loose1 = turned && rot1;  // rotated: off by up to err
                // largest magnitudes; NaN are zeros (seldom there: the maximum keeps them)
                float top0 = max_abs8(y0), top1 = max_abs8(y1);
                if (__any_sync(0xffffffffu, top0 != top0 || top1 != top1)) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        y0[k] = y0[k] == y0[k] ? y0[k] : 0.f;
                        y1[k] = y1[k] == y1[k] ? y1[k] : 0.f;
                    }
                    top0 = max_abs8(y0);
                    top1 = max_abs8(y1);
                }
                if constexpr (INTER) top0 = top1 = fmaxf(top0, top1);
#pragma unroll
                for (int o = 1; o < kReach; o <<= 1) {
                    top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, o));
                    if (!INTER) top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, o));
                }
                if (INTER) top1 = top0;
                // |x_a| + |x_b| of a pair is at most sqrt(2) times its norm, which the turn keeps
                // and which the groups' maxima bound; A is in them
                const bool turns = role == 1 && r > 0;  // of a whole warp
                float err = 0.f, far = 0.f;             // far: of the group
                float m0, m1;
                __half h0 = int4_scale(top0, m0), h1 = h0;
                if (INTER) m1 = m0;
                else h1 = int4_scale(top1, m1);
                bool unsure0 = false, unsure1 = false;
                if (turns) {
                    far = err = turned ? 1.42f * kRotError * (top0 + top1) : 0.f;
                    if (INTER) far = fmaxf(far, __shfl_xor_sync(0xffffffffu, far, 1));
                    // a maximum beyond int4_scale's range is far beyond the largest scale, and top - 2 far below
                    // would not be a number
                    unsure0 = far > 0.f && top0 < kInt4TopInput && fabsf(fmaf(-7.f, m0, top0)) <= far;
                    unsure1 = !INTER && far > 0.f && top1 < kInt4TopInput && fabsf(fmaf(-7.f, m1, top1)) <= far;
                }
                // The pair k of the lane (its elements in y0, y1) in f64.
                auto exact = [&](int k) -> double2 {
                    const float xa = !INTER ? a[k] : k < 4 ? a[2 * (k & 3)] : b[2 * (k & 3)];
                    const float xb = !INTER ? b[k] : k < 4 ? a[2 * (k & 3) + 1] : b[2 * (k & 3) + 1];
                    return (INTER && k >= 4 ? loose1 : loose0) ? rotate_exact(position, A.turns[8 * l + k], A.amplitude, xa, xb)
                                                               : make_double2(xa, xb);
                };
                if (turns && __any_sync(0xffffffffu, unsure0 || unsure1)) {  // a maximum next to the border of two scales
                    double g0 = 0.0, g1 = 0.0;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float ya = !INTER ? y0[k] : k < 4 ? y0[2 * (k & 3)] : y1[2 * (k & 3)];
                        const float yb = !INTER ? y1[k] : k < 4 ? y0[2 * (k & 3) + 1] : y1[2 * (k & 3) + 1];
                        const bool pa = unsure0 && fabsf(ya) >= top0 - 2.f * far;
                        const bool pb = INTER ? unsure0 && fabsf(yb) >= top0 - 2.f * far : unsure1 && fabsf(yb) >= top1 - 2.f * far;
                        if (__any_sync(0xffffffffu, pa || pb)) {
                            const double2 z = exact(k);
                            if (pa) g0 = fmax(g0, fabs(z.x));
                            if (pb && INTER) g0 = fmax(g0, fabs(z.y));
                            if (pb && !INTER) g1 = fmax(g1, fabs(z.y));
                        }
                    }
#pragma unroll
                    for (int o = 1; o < kReach; o <<= 1) {
                        g0 = fmax(g0, __shfl_xor_sync(0xffffffffu, g0, o));
                        if (!INTER) g1 = fmax(g1, __shfl_xor_sync(0xffffffffu, g1, o));
                    }
                    if (unsure0) h0 = int4_scale_f64(g0);
                    if (unsure1) h1 = int4_scale_f64(g1);
                    if (INTER) h1 = h0;
                }
                const float t0 = __half2float(h0), t1 = __half2float(h1);
                // Saturated groups, or too small for a scale, or under a subnormal one, coarse enough that the largest
                // value is 7.5 of them and would round to 8; under a normal scale it is at most 7 (1 + 2^-8).
                if (__any_sync(0xffffffffu, top0 > 7.25f * t0 || top1 > 7.25f * t1)) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        y0[k] = fminf(fmaxf(y0[k], -7.f * t0), 7.f * t0);
                        y1[k] = fminf(fmaxf(y1[k], -7.f * t1), 7.f * t1);
                    }
                }
                const float i0 = t0 > 0.f ? __frcp_rn(t0) : 0.f, i1 = t1 > 0.f ? __frcp_rn(t1) : 0.f;
                float gap0 = 3e38f, gap1 = 3e38f;
                uint32_t w0, w1;
                constexpr bool kWide = sizeof(T) == 4;
                if (kWide || turns) {
                    w0 = int4_word<true>(y0, t0, i0, kWide || loose0 ? 0.f : 384.f, gap0);
                    w1 = int4_word<true>(y1, t1, i1, kWide || loose1 ? 0.f : 384.f, gap1);
                } else {
                    w0 = int4_word<false>(y0, t0, i0, 384.f, gap0);
                    w1 = int4_word<false>(y1, t1, i1, 384.f, gap1);
                }
                // rotated (and f32) values next to the border of two codes: 2^-18 s for x inv
                const float e0 = fmaf(t0, 3.8e-6f, loose0 ? err : 0.f), e1 = fmaf(t1, 3.8e-6f, loose1 ? err : 0.f);
                const bool border0 = (kWide || loose0) && t0 > 0.f && gap0 <= e0, border1 = (kWide || loose1) && t1 > 0.f && gap1 <= e1;
                if ((kWide || turns) && __any_sync(0xffffffffu, border0 || border1)) {
                    uint32_t near0 = 0, near1 = 0;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (border0 && int4_near_border(y0[k], t0, static_cast<int>(w0 >> int4_shift(k) & 15) - 8, e0)) near0 |= 1u << k;
                        if (border1 && int4_near_border(y1[k], t1, static_cast<int>(w1 >> int4_shift(k) & 15) - 8, e1)) near1 |= 1u << k;
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        // bits of the pair's two elements
                        const int ea = !INTER ? k : 2 * (k & 3), eb = !INTER ? k : ea + 1;
                        const uint32_t na = !INTER || k < 4 ? near0 : near1, nb = !INTER ? near1 : na;
                        if (__any_sync(0xffffffffu, (na >> ea & 1) || (nb >> eb & 1))) {
                            const double2 z = exact(k);
                            const bool second = INTER && k >= 4;
                            uint32_t &wa = second ? w1 : w0, &wb = !INTER || second ? w1 : w0;
                            if (na >> ea & 1) wa = int4_settled(wa, int4_shift(ea), z.x, second ? t1 : t0);
                            if (nb >> eb & 1) wb = int4_settled(wb, int4_shift(eb), z.y, !INTER || second ? t1 : t0);
                        }
                    }
                }
                if (live) {
                    const int64_t row = row0 + static_cast<int64_t>(h) * A.bs;
                    uint32_t *codes = static_cast<uint32_t *>(role == 1 ? A.k_cache : A.v_cache) + row * (d >> 3);
                    __half *scales = (role == 1 ? A.k_scale : A.v_scale) + row * (d >> 5);
                    if (INTER) {
                        *reinterpret_cast<uint2 *>(codes + c0) = make_uint2(w0, w1);
                    } else {
                        codes[c0] = w0;
                        codes[c1] = w1;
                    }
                    if ((c0 & 3) == 0) scales[c0 >> 2] = h0;
                    if (!INTER && (c1 & 3) == 0) scales[c1 >> 2] = h1;
                }
            }
        }
    }
}

// ----------------------------------------------------------------------------- generic kernel
// Any even r, stride and alignment: a warp takes one head's row, an element a lane, the row
// first copied to shared memory (the queries may be rotated in place).
template <typename T, bool Q4>
__global__ void __launch_bounds__(kRopeThreads)
rope_store_generic_kernel(const __grid_constant__ RopeArgs A) {
    __shared__ float stage[kRopeWarps][kRopeGenericMaxDim];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d = A.d, r = A.r, heads = A.Hq + 2 * A.Hkv;
    float *x = stage[warp];
    const int64_t rows = A.num_tokens * heads;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp; row < rows;
         row += static_cast<int64_t>(gridDim.x) * kRopeWarps) {
        const int64_t i = row / heads;
        int h = static_cast<int>(row - i * heads);
        const int role = h < A.Hq ? 0 : h < A.Hq + A.Hkv ? 1 : 2;
        h -= role == 0 ? 0 : role == 1 ? A.Hq : A.Hq + A.Hkv;
        const int32_t slot = A.slots[i];
        const bool stored = slot >= 0 && slot < A.num_slots;
        if (role != 0 && !stored) {
            if (slot != -1 && role == 1 && h == 0 && lane == 0 && A.err_flag) atomicOr(A.err_flag, PKV_ERRBIT_SLOT_RANGE);
            continue;
        }
        const T *src = (role == 0 ? static_cast<const T *>(A.q) + i * A.q_stride
                      : role == 1 ? static_cast<const T *>(A.key) + i * A.k_stride
                                  : static_cast<const T *>(A.value) + i * A.v_stride) + static_cast<int64_t>(h) * d;
        __syncwarp();
        for (int j = lane; j < d; j += 32) x[j] = widen<T>(src[j]);
        __syncwarp();
        const int32_t position = r > 0 && role != 2 ? A.positions[i] : 0;
        const int64_t block = Q4 ? slot / A.bs : 0;
        const int64_t out_row = Q4 ? (block * A.Hkv + h) * A.bs + (slot - block * A.bs) : static_cast<int64_t>(slot) * A.Hkv + h;
        T *dst = role == 0 ? static_cast<T *>(A.q_out) + (i * A.Hq + h) * d
                           : static_cast<T *>(role == 1 ? A.k_cache : A.v_cache) + (Q4 ? 0 : out_row * d);
        for (int j0 = 0; j0 < d; j0 += 32) {
            const int j = j0 + lane;  // d is a multiple of 32 where it is quantised
            const bool spin = role != 2 && j < r;
            const int pair = A.inter ? j >> 1 : j < (r >> 1) ? j : j - (r >> 1);
            const bool second = A.inter ? j & 1 : j >= (r >> 1);
            float y = j < d ? x[j] : 0.f, a = 0.f, b = 0.f, err = 0.f;
            if (spin) {
                a = x[A.inter ? 2 * pair : pair];
                b = x[A.inter ? 2 * pair + 1 : pair + (r >> 1)];
                const float2 t = turn_cos_sin(position, A.turns[pair]);
                const float c = t.x * A.amp, s = t.y * A.amp;
                y = second ? fmaf(b, c, a * s) : fmaf(a, c, -(b * s));
                err = (fabsf(a) + fabsf(b)) * fabsf(A.amp) * kRotError;
            }
            if (!Q4 || role == 0) {
                if (j < d) dst[j] = narrow<T>(y);
                continue;
            }
            float top = fmaxf(fabsf(y), 0.f), far = err;  // fmaxf leaves NaN out
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                far = fmaxf(far, __shfl_xor_sync(0xffffffffu, far, o));
            }
            float mid;
            __half hs = int4_scale(top, mid);
            float s = __half2float(hs);
            int code = s > 0.f ? int4_code(y, s, 1.f / s) : 0;
            const bool unsure = far > 0.f && (fabsf(fmaf(-7.f, mid, top)) <= far || int4_near_border(y, s, code, far));
            if (__any_sync(0xffffffffu, unsure)) {
                double z = y;
                if (spin) {
                    const double2 p = rotate_exact(position, A.turns[pair], A.amplitude, a, b);
                    z = second ? p.y : p.x;
                }
                double g = fmax(fabs(z), 0.0);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) g = fmax(g, __shfl_xor_sync(0xffffffffu, g, o));
                hs = int4_scale_f64(g);
                s = __half2float(hs);
                code = s > 0.f ? int4_code_f64(z, s) : 0;
            }
            // lanes 8 e .. 8 e + 7 are one word
            uint32_t w = static_cast<uint32_t>(code + 8) << int4_shift(lane & 7);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) w |= __shfl_xor_sync(0xffffffffu, w, o);
            uint8_t *codes = static_cast<uint8_t *>(role == 1 ? A.k_cache : A.v_cache) + out_row * (d >> 1) + (j0 >> 1);
            if ((lane & 1) == 0) codes[lane >> 1] = static_cast<uint8_t>(w >> (lane & 6) * 4);
            if (lane == 0) (role == 1 ? A.k_scale : A.v_scale)[out_row * (d >> 5) + (j0 >> 5)] = hs;
        }
    }
}

// ----------------------------------------------------------------------------- read back
// Rows of both caches through a slot map: a word of eight codes a lane, widened, times its
// scale (exact in f16), as 16 bytes; bf16 rounds once.  A warp takes 128 words of a token.  CTAs in
// the order of the tokens: as many as fit the GPU, each going from token to token, keep the
// writes less together (131001 tokens of 8 heads, bf16, whole blocks: 105 us, 117 so).
constexpr int kLoadThreads = 128, kLoadCtas = 1 << 20;

// A word's codes as the bf16 pairs of u - 8, times a scale that bf16 holds.
__device__ __forceinline__ uint4 int4_bf16(uint32_t w, uint32_t scale) {
    uint32_t p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // 128 + u - 136
        asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(p[j]) : "r"(w >> 4 * j));
        asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(p[j]) : "r"(0x43084308u));
        asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(p[j]) : "r"(scale));
    }
    return make_uint4(p[0], p[1], p[2], p[3]);
}

template <typename T>
__device__ __forceinline__ void store_eight(T *dst, uint32_t w, __half scale, bool short_scale) {
    const float t = __half2float(scale);
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        if (short_scale) {
            *reinterpret_cast<uint4 *>(dst) = int4_bf16(w, __byte_perm(__float_as_uint(t), 0, 0x3232));
            return;
        }
    }
    uint32_t p[4];
    int4_widen(w, p);
    if constexpr (sizeof(T) == 4) {
        // a scale that this library did not write may have 11 bits: exact in f32
        float4 v[2];
        float *f = reinterpret_cast<float *>(v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 c = __half22float2(*reinterpret_cast<__half2 *>(&p[j]));
            f[2 * j] = c.x * t;
            f[2 * j + 1] = c.y * t;
        }
        reinterpret_cast<float4 *>(dst)[0] = v[0];
        reinterpret_cast<float4 *>(dst)[1] = v[1];
    } else {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __half2 c = *reinterpret_cast<__half2 *>(&p[j]);
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 y = __hmul2(c, __half2half2(scale));
                o[j] = *reinterpret_cast<const uint32_t *>(&y);
            } else {
                const float2 f = __half22float2(c);
                const __nv_bfloat162 y = __floats2bfloat162_rn(f.x * t, f.y * t);
                o[j] = *reinterpret_cast<const uint32_t *>(&y);
            }
        }
        *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <typename T>
__global__ void __launch_bounds__(kLoadThreads)
load_int4_kernel(T *__restrict__ key, T *__restrict__ value, const uint32_t *__restrict__ k_cache,
                 const uint32_t *__restrict__ v_cache, const __half *__restrict__ k_scale,
                 const __half *__restrict__ v_scale, const int32_t *__restrict__ slots, int64_t num_tokens,
                 int64_t num_slots, int32_t Hkv, int32_t d, int32_t bs, int32_t *__restrict__ err_flag) {
    constexpr int U = 4;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int wph = d >> 3, words = Hkv * wph;  // words of a head, of a token
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kLoadThreads / 32);
    for (int seg = blockIdx.y; seg * (32 * U) < words; seg += gridDim.y) {
        const int w0 = seg * (32 * U) + lane;
        int64_t i = static_cast<int64_t>(blockIdx.x) * (kLoadThreads / 32) + (threadIdx.x >> 5);
        int32_t next = i < num_tokens ? slots[i] : -1;  // on its way beside the divisions
        int64_t code_at[U];
        int32_t ends = 0;  // of the lane's words, how many there are
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int w = w0 + 32 * u, h = w / wph;
            code_at[u] = static_cast<int64_t>(h) * bs * wph + (w - h * wph);
            ends += w < words ? 1 : 0;
        }
        for (; i < num_tokens; i += step) {
            const int32_t slot = next;
            if (i + step < num_tokens) next = slots[i + step];
            const bool live = slot >= 0 && slot < num_slots;
            if (!live && slot != -1 && w0 == 0 && err_flag) atomicOr(err_flag, PKV_ERRBIT_SLOT_RANGE);
            const int block = live ? slot / bs : 0;
            // the slot's row of head 0, in words
            const int64_t row = (static_cast<int64_t>(block) * Hkv * bs + (live ? slot - block * bs : 0)) * wph;
            uint32_t kw[U], vw[U];
            __half ks[U], vs[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                kw[u] = vw[u] = 0x88888888u;  // zeros
                ks[u] = vs[u] = __float2half_rn(0.f);
                if (live && u < ends) {
                    const int64_t at = row + code_at[u];  // a scale for every four words
                    kw[u] = __ldg(k_cache + at);
                    vw[u] = __ldg(v_cache + at);
                    ks[u] = __ldg(k_scale + (at >> 2));
                    vs[u] = __ldg(v_scale + (at >> 2));
                }
            }
            // scales of eight bits, as the store writes them, are bf16 values too
            uint32_t low = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) low |= __float_as_uint(__half2float(ks[u])) | __float_as_uint(__half2float(vs[u]));
            const bool short_scales = __all_sync(0xffffffffu, (low & 0xffffu) == 0);
            const int64_t out = (i * words + w0) * 8;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u < ends) {
                    store_eight<T>(key + out + 256 * u, kw[u], ks[u], short_scales);
                    store_eight<T>(value + out + 256 * u, vw[u], vs[u], short_scales);
                }
            }
        }
    }
}

// ----------------------------------------------------------------------------- host side
uint64_t turns_of(double radians) {
    double t = radians / 6.283185307179586476925286766559;
    t -= std::floor(t);
    const double scaled = std::ldexp(t, 64);
    return scaled >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(scaled);  // t rounded up to a whole turn
}

template <typename T, bool INTER, bool Q4>
cudaError_t launch_fast(RopeArgs a, cudaStream_t stream) {
    const int hpw = 32 / (a.d / 16);
    const int steps = (a.Hq + hpw - 1) / hpw + 2 * ((a.Hkv + hpw - 1) / hpw);
    // A warp per token once there are warps enough; before that a token's steps are spread over several.
    int64_t per = a.num_tokens * steps / kRopeFullWarps;
    per = per < 1 ? 1 : per > steps ? steps : per;
    a.steps_per_part = static_cast<int32_t>(per);
    a.parts = (steps + a.steps_per_part - 1) / a.steps_per_part;
    const int64_t ctas = (a.num_tokens * a.parts + kRopeWarps - 1) / kRopeWarps;
    return launch_pdl(kPdlStore, rope_store_kernel<T, INTER, Q4>, dim3(static_cast<unsigned>(ctas < kRopeMaxCtas ? ctas : kRopeMaxCtas)),
                      dim3(kRopeThreads), 0, stream, a);
}

template <typename T, bool Q4>
cudaError_t launch_rope(const RopeArgs &a, bool vectors, cudaStream_t stream) {
    const int r = a.r, d = a.d;
    const bool base = vectors && d % 16 == 0 && d <= kRopeMaxDim && r % 8 == 0;
    // pairs side by side (and rows that are not rotated); pairs in halves
    if (base && (a.inter || r == 0) && (!Q4 || d % 32 == 0)) return launch_fast<T, true, Q4>(a, stream);
    if (base && !a.inter && r % 16 == 0 && (!Q4 || (r % 64 == 0 && d % 64 == 0))) return launch_fast<T, false, Q4>(a, stream);
    const int64_t ctas = (a.num_tokens * (a.Hq + 2 * a.Hkv) + kRopeWarps - 1) / kRopeWarps;
    return launch_pdl(kPdlStore, rope_store_generic_kernel<T, Q4>, dim3(static_cast<unsigned>(ctas < kRopeMaxCtas ? ctas : kRopeMaxCtas)),
                      dim3(kRopeThreads), 0, stream, a);
}

pkv_status rope_store(const char *what, bool q4, void *q_out, const void *q, int64_t q_stride, const void *key, int64_t key_stride,
                      const void *value, int64_t value_stride, const int32_t *positions, const pkv_rope *rope, void *k_cache,
                      void *v_cache, uint16_t *k_scale, uint16_t *v_scale, const int32_t *slot_mapping, int64_t num_tokens,
                      int32_t Hq, int32_t Hkv, int32_t d, int32_t bs, int64_t num_slots, pkv_dtype dtype, int32_t *err_flag,
                      void *stream) {
    const int64_t es = dtype_bytes(dtype);
    if (es == 0) return set_error(PKV_ERR_INVALID_ARG, "%s: unknown dtype %d", what, (int)dtype);
    if (num_tokens < 0 || Hq < 0 || Hkv <= 0 || d <= 0 || bs <= 0 || num_slots < 0)
        return set_error(PKV_ERR_INVALID_ARG, "%s: bad sizes", what);
    if (static_cast<int64_t>(Hq) * d > INT32_MAX || static_cast<int64_t>(Hkv) * d > INT32_MAX)
        return set_error(PKV_ERR_INVALID_ARG, "%s: a token's heads hold 2^31 elements or more", what);
    if (num_slots > INT32_MAX) return set_error(PKV_ERR_INVALID_ARG, "%s: num_blocks * block_size >= 2^31", what);
    const int32_t r = rope ? rope->rotary_dim : 0;
    if (r < 0 || r > d || r % 2) return set_error(PKV_ERR_INVALID_ARG, "%s: rotary_dim must be even, from 0 to head_dim (%d)", what, d);
    if (r > 0 && !(std::fabs(rope->amplitude) <= 1e6)) return set_error(PKV_ERR_INVALID_ARG, "%s: amplitude must be finite, at most 1e6", what);
    if (r > 0 && rope->interleaved != 0 && rope->interleaved != 1)
        return set_error(PKV_ERR_INVALID_ARG, "%s: interleaved must be 0 or 1", what);
    const int64_t q_row = static_cast<int64_t>(Hq) * d, kv_row = static_cast<int64_t>(Hkv) * d;
    if (num_tokens > 1 && ((Hq > 0 && q_stride < q_row) || key_stride < kv_row || value_stride < kv_row))
        return set_error(PKV_ERR_INVALID_ARG, "%s: token strides are shorter than a token's heads", what);
    if (q4 && d % kInt4Group) return set_error(PKV_ERR_UNSUPPORTED, "%s: head_dim must be a multiple of %d", what, kInt4Group);
    if (d > kRopeGenericMaxDim) return set_error(PKV_ERR_UNSUPPORTED, "%s: head_dim above %d", what, kRopeGenericMaxDim);
    if (num_tokens == 0) return ok();
    if (!key || !value || !k_cache || !v_cache || !slot_mapping || (Hq > 0 && (!q || !q_out)) ||
        (r > 0 && (!positions || !rope->turns)) || (q4 && (!k_scale || !v_scale)))
        return set_error(PKV_ERR_INVALID_ARG, "%s: NULL pointer", what);
    if (Hq > 0 && q_out == q && q_stride != q_row && num_tokens > 1)
        return set_error(PKV_ERR_INVALID_ARG, "%s: rotating in place needs contiguous queries", what);
    if (!aligned(q, es) || !aligned(key, es) || !aligned(value, es) || !aligned(q_out, es) || !aligned(slot_mapping, 4) ||
        !aligned(positions, 4) || (r > 0 && !aligned(rope->turns, 8)) ||
        (q4 ? !aligned(k_cache, 4) || !aligned(v_cache, 4) || !aligned(k_scale, 2) || !aligned(v_scale, 2)
            : !aligned(k_cache, es) || !aligned(v_cache, es)))
        return set_error(PKV_ERR_INVALID_ARG, "%s: buffers not aligned to their elements (codes: 4 bytes)", what);
    RopeArgs a{};
    a.q = q;
    a.key = key;
    a.value = value;
    a.q_out = q_out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = reinterpret_cast<__half *>(k_scale);
    a.v_scale = reinterpret_cast<__half *>(v_scale);
    a.positions = positions;
    a.slots = slot_mapping;
    a.q_stride = q_stride;
    a.k_stride = key_stride;
    a.v_stride = value_stride;
    a.num_tokens = num_tokens;
    a.num_slots = num_slots;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.d = d;
    a.r = r;
    a.bs = bs;
    a.err_flag = err_flag;
    if (r > 0) {
        a.turns = rope->turns;
        a.amplitude = rope->amplitude;
        a.amp = static_cast<float>(rope->amplitude);
        a.inter = rope->interleaved;
    }
    auto whole = [&](const void *p, int64_t stride) { return aligned(p, 16) && (num_tokens == 1 || stride * es % 16 == 0); };
    const bool vectors = whole(key, key_stride) && whole(value, value_stride) && (Hq == 0 || (whole(q, q_stride) && aligned(q_out, 16))) &&
                         (q4 ? aligned(k_cache, 8) && aligned(v_cache, 8) : aligned(k_cache, 16) && aligned(v_cache, 16));
    auto s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == PKV_F32) e = q4 ? launch_rope<float, true>(a, vectors, s) : launch_rope<float, false>(a, vectors, s);
    else if (dtype == PKV_F16) e = q4 ? launch_rope<__half, true>(a, vectors, s) : launch_rope<__half, false>(a, vectors, s);
    else e = q4 ? launch_rope<__nv_bfloat16, true>(a, vectors, s) : launch_rope<__nv_bfloat16, false>(a, vectors, s);
    if (e != cudaSuccess) return set_error(PKV_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    return ok();
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_rope_turns(const double *inv_freq, int32_t num_pairs, uint64_t *turns) {
    if (num_pairs < 0 || (num_pairs > 0 && (!inv_freq || !turns))) return set_error(PKV_ERR_INVALID_ARG, "rope: bad sizes or NULL pointer");
    for (int32_t i = 0; i < num_pairs; ++i)
        if (!(std::fabs(inv_freq[i]) <= 1e15)) return set_error(PKV_ERR_INVALID_ARG, "rope: frequency %d is not finite", i);
    for (int32_t i = 0; i < num_pairs; ++i) turns[i] = turns_of(inv_freq[i]);
    return ok();
}

extern "C" pkv_status pkv_rope_frequencies(int32_t rotary_dim, double base, pkv_rope_scaling scaling, double factor,
                                           double original_len, double beta_fast, double beta_slow, uint64_t *turns,
                                           double *amplitude) {
    if (rotary_dim < 0 || rotary_dim % 2 || !(base > 1.0) || !(base <= 1e15))
        return set_error(PKV_ERR_INVALID_ARG, "rope: rotary_dim must be even and base above 1");
    if (scaling != PKV_ROPE_NONE && scaling != PKV_ROPE_LINEAR && scaling != PKV_ROPE_NTK && scaling != PKV_ROPE_YARN)
        return set_error(PKV_ERR_INVALID_ARG, "rope: unknown scaling %d", (int)scaling);
    if (scaling != PKV_ROPE_NONE && !(factor >= 1.0 && factor <= 1e9))
        return set_error(PKV_ERR_INVALID_ARG, "rope: factor must be from 1 to 1e9");
    if (scaling == PKV_ROPE_YARN && !(original_len > 0.0 && original_len <= 1e15 && beta_slow >= 0.0 && beta_fast > beta_slow && beta_fast <= 1e15))
        return set_error(PKV_ERR_INVALID_ARG, "rope: yarn needs original_len > 0 and beta_fast > beta_slow >= 0");
    if (!amplitude || (rotary_dim > 0 && !turns)) return set_error(PKV_ERR_INVALID_ARG, "rope: NULL pointer");
    const double r = rotary_dim, two_pi = 6.283185307179586476925286766559;
    if (scaling == PKV_ROPE_NTK && rotary_dim > 2) base *= std::pow(factor, r / (r - 2.0));
    for (int32_t i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / r);
        if (scaling == PKV_ROPE_LINEAR) f /= factor;
        if (scaling == PKV_ROPE_YARN) {
            double keep = (original_len * f / two_pi - beta_slow) / (beta_fast - beta_slow);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = f * keep + f / factor * (1.0 - keep);
        }
        turns[i] = turns_of(f);
    }
    *amplitude = scaling == PKV_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return ok();
}

extern "C" pkv_status pkv_rope_store_kvcache(void *q_out, const void *q, int64_t q_stride, const void *key, int64_t key_stride,
                                             const void *value, int64_t value_stride, const int32_t *positions,
                                             const pkv_rope *rope, void *k_cache, void *v_cache, const int32_t *slot_mapping,
                                             int64_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                             int64_t num_slots, pkv_dtype dtype, int32_t *err_flag, void *stream) {
    return rope_store("rope store", false, q_out, q, q_stride, key, key_stride, value, value_stride, positions, rope, k_cache, v_cache,
                      nullptr, nullptr, slot_mapping, num_tokens, num_q_heads, num_kv_heads, head_dim, 1, num_slots, dtype, err_flag,
                      stream);
}

extern "C" pkv_status pkv_rope_store_kvcache_int4(void *q_out, const void *q, int64_t q_stride, const void *key, int64_t key_stride,
                                                  const void *value, int64_t value_stride, const int32_t *positions,
                                                  const pkv_rope *rope, void *k_cache, void *v_cache, uint16_t *k_scale,
                                                  uint16_t *v_scale, const int32_t *slot_mapping, int64_t num_tokens,
                                                  int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                                  int32_t num_blocks, pkv_dtype dtype, int32_t *err_flag, void *stream) {
    if (num_blocks < 0 || block_size <= 0) return set_error(PKV_ERR_INVALID_ARG, "int4 store: bad sizes");
    return rope_store("int4 store", true, q_out, q, q_stride, key, key_stride, value, value_stride, positions, rope, k_cache, v_cache,
                      k_scale, v_scale, slot_mapping, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size,
                      static_cast<int64_t>(num_blocks) * block_size, dtype, err_flag, stream);
}

extern "C" pkv_status pkv_store_kvcache_int4(const void *key, int64_t key_stride, const void *value, int64_t value_stride, void *k_cache,
                                             void *v_cache, uint16_t *k_scale, uint16_t *v_scale, const int32_t *slot_mapping,
                                             int64_t num_tokens, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                             int32_t num_blocks, pkv_dtype dtype, int32_t *err_flag, void *stream) {
    return pkv_rope_store_kvcache_int4(nullptr, nullptr, 0, key, key_stride, value, value_stride, nullptr, nullptr, k_cache, v_cache,
                                       k_scale, v_scale, slot_mapping, num_tokens, 0, num_kv_heads, head_dim, block_size, num_blocks,
                                       dtype, err_flag, stream);
}

extern "C" pkv_status pkv_load_kvcache_int4(void *key, void *value, const void *k_cache, const void *v_cache, const uint16_t *k_scale,
                                            const uint16_t *v_scale, const int32_t *slot_mapping, int64_t num_tokens,
                                            int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                            pkv_dtype dtype, int32_t *err_flag, void *stream) {
    if (dtype_bytes(dtype) == 0) return set_error(PKV_ERR_INVALID_ARG, "int4 load: unknown dtype %d", (int)dtype);
    if (num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks < 0)
        return set_error(PKV_ERR_INVALID_ARG, "int4 load: bad sizes");
    const int64_t num_slots = static_cast<int64_t>(num_blocks) * block_size;
    if (num_slots > INT32_MAX) return set_error(PKV_ERR_INVALID_ARG, "int4 load: num_blocks * block_size >= 2^31");
    if (head_dim % kInt4Group || static_cast<int64_t>(num_kv_heads) * head_dim > (1 << 30))
        return set_error(PKV_ERR_UNSUPPORTED, "int4 load: head_dim must be a multiple of %d", kInt4Group);
    if (num_tokens == 0) return ok();
    if (!key || !value || !k_cache || !v_cache || !k_scale || !v_scale || !slot_mapping)
        return set_error(PKV_ERR_INVALID_ARG, "int4 load: NULL pointer");
    if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 4) || !aligned(v_cache, 4) || !aligned(k_scale, 2) ||
        !aligned(v_scale, 2) || !aligned(slot_mapping, 4))
        return set_error(PKV_ERR_INVALID_ARG, "int4 load: key and value must be 16-byte aligned, codes 4-byte aligned");
    const int64_t segs = (static_cast<int64_t>(num_kv_heads) * head_dim / 8 + 127) / 128;
    const int64_t y = segs < 64 ? segs : 64, x = (num_tokens + kLoadThreads / 32 - 1) / (kLoadThreads / 32);
    const int64_t most = (kLoadCtas + y - 1) / y;
    const dim3 grid(static_cast<unsigned>(x < most ? x : most), static_cast<unsigned>(y));
    auto s = static_cast<cudaStream_t>(stream);
    auto kc = static_cast<const uint32_t *>(k_cache), vc = static_cast<const uint32_t *>(v_cache);
    auto ks = reinterpret_cast<const __half *>(k_scale), vs = reinterpret_cast<const __half *>(v_scale);
    auto go = [&](auto *kp, auto *vp) {
        using T = std::remove_pointer_t<decltype(kp)>;
        return launch_pdl(kPdlStore, load_int4_kernel<T>, grid, dim3(kLoadThreads), 0, s, kp, vp, kc, vc, ks, vs, slot_mapping, num_tokens,
                          num_slots, num_kv_heads, head_dim, block_size, err_flag);
    };
    const cudaError_t e = dtype == PKV_F32 ? go(static_cast<float *>(key), static_cast<float *>(value))
                        : dtype == PKV_F16 ? go(static_cast<__half *>(key), static_cast<__half *>(value))
                                           : go(static_cast<__nv_bfloat16 *>(key), static_cast<__nv_bfloat16 *>(value));
    if (e != cudaSuccess) return set_error(PKV_ERR_CUDA, "int4 load launch: %s", cudaGetErrorString(e));
    return ok();
}
