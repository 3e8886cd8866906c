// Prefill over 4-bit caches: the score-rule kernels that widen codes as they go, the widening into
// f16 for calls of many rows, and the entry point.
//
// A tile pair (256 / G positions of a KV head) reads every key its rows see, and the fused kernels
// widen all of them anew: 512 new positions at G = 4 are 8 pairs.  Widened once into the workspace
// and read by the 16-bit kernel the same call takes the 16-bit kernel's time and a pass over the
// contexts, bound by HBM (144 bytes read and 512 written a token and KV head): 8 prompts of 3700 to
// 4096 tokens, 32 heads over 8 KV heads, fp16, 988 us against 1231; 8 x 512 behind 3000 to 7680,
// bf16, 472 against 512.  Fewer rows read too little of it again: 8 x 128 behind 4000 104 / 90, 8 x 192
// 170 / 170, 8 x 256 174 / 175, 8 x 512 318 / 349; one head a KV head, 8 x 512 111 / 96, 8 x 1024 198 /
// 198.
#include "pkv_prefill_mod.cuh"

namespace pkv {
namespace {

constexpr int kWideRows = 1024;                   // rows of a KV head from which on a call is widened
constexpr size_t kWideLimit = size_t(1) << 30;    // bytes of workspace it may take
constexpr int kWidenWarps = 8;

// One warp per (sequence, 16 tokens, KV head): 256 words of codes of K and of V, eight dims each;
// 16 lanes write a row of 256 bytes.  Blocks out of range get no entry in the new table, which the
// attention then treats as it would have treated theirs.
__global__ void __launch_bounds__(kWidenWarps * 32)
widen_int4_kernel(__half *__restrict__ k_out, __half *__restrict__ v_out, int32_t *__restrict__ table_out, int32_t stride,
                  const uint32_t *__restrict__ k_codes, const uint32_t *__restrict__ v_codes, const __half *__restrict__ k_scale,
                  const __half *__restrict__ v_scale, const int32_t *__restrict__ tables, int32_t max_blocks,
                  const int32_t *__restrict__ starts, const int32_t *__restrict__ cu_q, int32_t max_q_len, int32_t Hkv, int32_t bs,
                  int32_t num_blocks, int64_t items) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int tiles = stride * (bs >> 4);  // of a sequence
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWidenWarps + (threadIdx.x >> 5); item < items;
         item += static_cast<int64_t>(gridDim.x) * kWidenWarps) {
        const int64_t bt = item / Hkv;
        const int kh = static_cast<int>(item - bt * Hkv), b = static_cast<int>(bt / tiles), tile = static_cast<int>(bt - static_cast<int64_t>(b) * tiles);
        const int n = cu_q[b + 1] - cu_q[b], start = starts[b];
        const int64_t total = static_cast<int64_t>(start) + n, pos = static_cast<int64_t>(tile) * 16;
        // a sequence that the attention does not run has nothing to widen
        if (n <= 0 || n > max_q_len || start < 0 || total > static_cast<int64_t>(stride) * bs || pos >= total) continue;
        const int block = static_cast<int>(pos / bs), in = static_cast<int>(pos - static_cast<int64_t>(block) * bs);
        const int id = tables[static_cast<int64_t>(b) * max_blocks + block];
        const bool there = id >= 0 && id < num_blocks;
        if (kh == 0 && in == 0 && lane == 0) table_out[static_cast<int64_t>(b) * stride + block] = there ? b * stride + block : -1;
        if (!there) continue;
        const int64_t from = (static_cast<int64_t>(id) * Hkv + kh) * bs + in;                                   // row of codes
        const int64_t to = (static_cast<int64_t>(b) * stride + block) * bs + in;                                // token of the pool
        const int c = lane & 15, r0 = lane >> 4;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint32_t *src = (kv ? v_codes : k_codes) + from * 16 + lane;
            const __half *scale = (kv ? v_scale : k_scale) + from * 4 + r0 * 4 + (c >> 2);
            uint4 *dst = reinterpret_cast<uint4 *>(kv ? v_out : k_out) + ((to + r0) * Hkv + kh) * 16 + c;
            uint32_t w[8];
            uint16_t s[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // rows 2 i + r0
                w[i] = __ldg(src + 32 * i);
                s[i] = __ldg(reinterpret_cast<const uint16_t *>(scale) + 8 * i);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t p[4];
                int4_widen(w[i], p);
                const uint32_t s2 = s[i] | static_cast<uint32_t>(s[i]) << 16;
                dst[static_cast<int64_t>(2 * i) * Hkv * 16] =
                    make_uint4(mul_f16x2(p[0], s2), mul_f16x2(p[1], s2), mul_f16x2(p[2], s2), mul_f16x2(p[3], s2));
            }
        }
    }
}

}  // namespace

pkv_status prefill_mod_int4(const PrefillCall &c) { return prefill_mod_format<kCodeInt4>(c); }

WidePlan wide_plan(int32_t B, int32_t Hq, int32_t Hkv, int32_t bs, int32_t max_q_len, int32_t max_blocks, int32_t max_total_len) {
    WidePlan w;
    if (static_cast<int64_t>(max_q_len) * (Hq / Hkv) < kWideRows || max_blocks == 0) return w;
    const int64_t width = static_cast<int64_t>(max_blocks) * bs;
    const int64_t total = max_total_len > 0 && max_total_len < width ? max_total_len : width;
    const int64_t stride = (total + bs - 1) / bs, tokens = B * stride * bs;
    const size_t row = static_cast<size_t>(Hkv) * kFastHeadDim * sizeof(__half);
    if (tokens > INT32_MAX || static_cast<size_t>(tokens) > kWideLimit / (2 * row)) return w;
    w.stride = static_cast<int32_t>(stride);
    w.pool_bytes = tokens * row;  // a multiple of 256
    w.bytes = 2 * w.pool_bytes + (static_cast<size_t>(B) * stride * sizeof(int32_t) + 255) / 256 * 256;
    return w;
}

pkv_status widen_int4(PrefillCall &c, const WidePlan &w, char *workspace) {
    __half *k = reinterpret_cast<__half *>(workspace), *v = reinterpret_cast<__half *>(workspace + w.pool_bytes);
    int32_t *table = reinterpret_cast<int32_t *>(workspace + 2 * w.pool_bytes);
    const int64_t items = static_cast<int64_t>(c.num_seqs) * w.stride * (c.block_size / 16) * c.Hkv;
    const int64_t ctas = (items + kWidenWarps - 1) / kWidenWarps;
    const cudaError_t e = launch_pdl(kPdlStore, widen_int4_kernel, dim3(static_cast<unsigned>(ctas < (1 << 20) ? ctas : 1 << 20)),
                                     dim3(kWidenWarps * 32), 0, c.stream, k, v, table, w.stride, static_cast<const uint32_t *>(c.k_cache),
                                     static_cast<const uint32_t *>(c.v_cache), reinterpret_cast<const __half *>(c.k_scale4),
                                     reinterpret_cast<const __half *>(c.v_scale4), c.block_tables, c.max_blocks, c.starts, c.cu_q,
                                     c.max_q_len, c.Hkv, c.block_size, c.num_blocks, items);
    if (e != cudaSuccess) return set_error(PKV_ERR_CUDA, "prefill: widening launch: %s", cudaGetErrorString(e));
    c.k_cache = k;
    c.v_cache = v;
    c.block_tables = table;
    c.max_blocks = w.stride;
    c.num_blocks = c.num_seqs * w.stride;
    return PKV_OK;
}

}  // namespace pkv

extern "C" pkv_status pkv_paged_attention_prefill_int4(
    void *out, const void *q, const void *k_cache, const void *v_cache, const uint16_t *k_scale, const uint16_t *v_scale,
    const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *starts, const int32_t *cu_q, int32_t num_seqs,
    int32_t max_q_len, int32_t max_total_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
    int32_t num_blocks, float scale, const pkv_score_mod *mod, pkv_dtype dtype, void *workspace, size_t workspace_bytes,
    int32_t *err_flag, void *stream) {
    pkv::PrefillCall c{};
    c.out = out;
    c.q = q;
    c.k_cache = k_cache;
    c.v_cache = v_cache;
    c.k_scale4 = k_scale;
    c.v_scale4 = v_scale;
    c.block_tables = block_tables;
    c.max_blocks = max_blocks_per_seq;
    c.starts = starts;
    c.cu_q = cu_q;
    c.num_seqs = num_seqs;
    c.max_q_len = max_q_len;
    c.max_total_len = max_total_len;
    c.Hq = num_q_heads;
    c.Hkv = num_kv_heads;
    c.block_size = block_size;
    c.num_blocks = num_blocks;
    c.scale = scale;
    if (mod) c.mod = *mod;
    c.dtype = dtype;
    c.err_flag = err_flag;
    c.stream = static_cast<cudaStream_t>(stream);
    return pkv::prefill_mod_run(c, pkv::kCodeInt4, head_dim, workspace, workspace_bytes);
}
