// Entry points of the score-rule and 8-bit prefill, and its kernels over 16-bit
// caches (pkv_prefill_mod.cuh has the method).
#include "pkv_prefill_mod.cuh"

#include <cmath>

namespace pkv {

pkv_status prefill_mod_16bit(const PrefillCall &c) { return prefill_mod_format<kCode16>(c); }

namespace {

constexpr int kModSms = 152;  // GB300; fixed so that the plan is device independent
constexpr int kMaxSplits = 32;

// Splits: one CTA runs per SM, so a launch of fewer than half as many CTAs as SMs
// cuts its key blocks until it fills one wave, in runs of kMinSplitBlocks blocks at
// least; longer launches gain nothing from it.  Cap 50, 32 heads over 8 KV heads, bf16,
// with the joining kernel against one CTA a pair, on the GPU: 16 rows over 512 keys
// 11.6 us / 11.9 (from Python, with the workspace and the second launch, 24 / 18), over
// 2048 13.8 / 33.5 (24 / 34); 64 over 8k 33 / 145; 4 x 16 over 32k 128 / 472; 8 x 64 over
// 4k 53 / 78; 512 over 64k 581 / 1127.
PrefillPlan prefill_plan(int32_t B, int32_t Hq, int32_t Hkv, int32_t max_q_len, int32_t max_blocks, int32_t bs) {
    PrefillPlan p;
    const int G = Hq / Hkv, positions = kModRows / G;
    const int64_t tiles = (static_cast<int64_t>(max_q_len) + positions - 1) / positions;
    p.pairs = static_cast<int32_t>((tiles + 1) / 2);
    const int64_t ctas = static_cast<int64_t>(p.pairs) * Hkv * B;
    const int64_t blocks = (static_cast<int64_t>(max_blocks) * bs + kModKeys - 1) / kModKeys;
    int64_t s = kModSms / ctas;
    if (s > blocks / kMinSplitBlocks) s = blocks / kMinSplitBlocks;
    if (s > kMaxSplits) s = kMaxSplits;
    p.nsplit = static_cast<int32_t>(s < 1 ? 1 : s);
    if (p.nsplit > 1) {
        const size_t rows = static_cast<size_t>(B) * max_q_len * Hq * p.nsplit;
        p.o_bytes = rows * kFastHeadDim * sizeof(float);
        p.ml_bytes = (rows * sizeof(float2) + 255) / 256 * 256;
        p.ws_bytes = p.o_bytes + p.ml_bytes + (static_cast<size_t>(B) * p.pairs * 4 + 255) / 256 * 256;
    }
    return p;
}

bool supported_shape(int32_t Hq, int32_t Hkv, int32_t d, int32_t bs) {
    const int G = Hq / Hkv;
    return d == kFastHeadDim && (G == 1 || G == 2 || G == 4 || G == 8) && bs % kStageTokens == 0;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_paged_attention_prefill_mod_workspace_size(int32_t num_seqs, int32_t num_q_heads,
                                                                 int32_t num_kv_heads, int32_t head_dim,
                                                                 int32_t block_size, int32_t max_q_len,
                                                                 int32_t max_blocks_per_seq) {
    if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || block_size <= 0 ||
        max_q_len <= 0 || max_blocks_per_seq < 0 || !supported_shape(num_q_heads, num_kv_heads, head_dim, block_size))
        return 0;
    return prefill_plan(num_seqs, num_q_heads, num_kv_heads, max_q_len, max_blocks_per_seq, block_size).ws_bytes;
}

extern "C" pkv_status pkv_paged_attention_prefill_mod(
    void *out, const void *q, const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
    pkv_cache_format format, const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *starts,
    const int32_t *cu_q, int32_t num_seqs, int32_t max_q_len, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int32_t num_blocks, float scale, const pkv_score_mod *mod, pkv_dtype dtype,
    void *workspace, size_t workspace_bytes, int32_t *err_flag, void *stream) {
    if (dtype_bytes(dtype) == 0) return set_error(PKV_ERR_INVALID_ARG, "prefill: unknown dtype %d", (int)dtype);
    if (format != PKV_CACHE_DTYPE && format != PKV_CACHE_E4M3 && format != PKV_CACHE_INT8)
        return set_error(PKV_ERR_INVALID_ARG, "prefill: unknown cache format %d", (int)format);
    if (num_seqs < 0 || max_q_len < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        num_blocks < 0 || max_blocks_per_seq < 0)
        return set_error(PKV_ERR_INVALID_ARG, "prefill: bad sizes");
    if (num_q_heads % num_kv_heads)
        return set_error(PKV_ERR_INVALID_ARG, "prefill: num_q_heads (%d) is not a multiple of num_kv_heads (%d)",
                         num_q_heads, num_kv_heads);
    if (static_cast<int64_t>(num_blocks) * block_size > INT32_MAX)
        return set_error(PKV_ERR_INVALID_ARG, "prefill: num_blocks * block_size >= 2^31");
    const pkv_score_mod none{};
    const pkv_score_mod m = mod ? *mod : none;
    if (!(m.softcap >= 0.f) || m.softcap > 1e30f || (m.softcap > 0.f && m.softcap < 1e-30f))
        return set_error(PKV_ERR_INVALID_ARG, "prefill: softcap must be 0, or from 1e-30 to 1e30");
    if (num_seqs > 65535 || num_kv_heads > 65535)
        return set_error(PKV_ERR_UNSUPPORTED, "prefill: more than 65535 sequences or KV heads");
    if (num_seqs == 0 || max_q_len == 0) return ok();
    if ((dtype != PKV_F16 && dtype != PKV_BF16) || !supported_shape(num_q_heads, num_kv_heads, head_dim, block_size))
        return set_error(PKV_ERR_UNSUPPORTED, "prefill: needs fp16/bf16, head_dim 128, Hq/Hkv in {1, 2, 4, 8} and "
                                              "block_size a multiple of 16");
    if (!out || !q || !starts || !cu_q || !block_tables || !k_cache || !v_cache || num_blocks == 0)
        return set_error(PKV_ERR_INVALID_ARG, "prefill: NULL pointer or empty pool");
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q, 16) || !aligned(out, 16))
        return set_error(PKV_ERR_UNSUPPORTED, "prefill: pools, q and out must be 16-byte aligned");
    if (format != PKV_CACHE_DTYPE && (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4)))
        return set_error(PKV_ERR_INVALID_ARG, "prefill: scales of an 8-bit cache NULL or not 4-byte aligned");
    PrefillCall c{};
    c.plan = prefill_plan(num_seqs, num_q_heads, num_kv_heads, max_q_len, max_blocks_per_seq, block_size);
    if (c.plan.ws_bytes > 0 && (!workspace || workspace_bytes < c.plan.ws_bytes || !aligned(workspace, 256)))
        return set_error(PKV_ERR_WORKSPACE, "prefill: workspace needs %zu bytes (256-byte aligned), got %zu",
                         c.plan.ws_bytes, workspace_bytes);
    c.out = out;
    c.q = q;
    c.k_cache = k_cache;
    c.v_cache = v_cache;
    c.k_scale = k_scale;
    c.v_scale = v_scale;
    c.block_tables = block_tables;
    c.max_blocks = max_blocks_per_seq;
    c.starts = starts;
    c.cu_q = cu_q;
    c.num_seqs = num_seqs;
    c.max_q_len = max_q_len;
    c.Hq = num_q_heads;
    c.Hkv = num_kv_heads;
    c.block_size = block_size;
    c.num_blocks = num_blocks;
    c.scale = scale;
    c.mod = m;
    c.dtype = dtype;
    c.workspace = static_cast<char *>(workspace);
    c.err_flag = err_flag;
    c.stream = static_cast<cudaStream_t>(stream);
    const pkv_status st = format == PKV_CACHE_E4M3   ? prefill_mod_e4m3(c)
                          : format == PKV_CACHE_INT8 ? prefill_mod_int8(c)
                                                     : prefill_mod_16bit(c);
    return st == PKV_OK ? ok() : st;
}
