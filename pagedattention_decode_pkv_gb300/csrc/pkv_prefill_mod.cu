// Entry points of the score-rule and 8-bit prefill, the checks of every call, and the
// kernels over 16-bit caches (pkv_prefill_mod.cuh has the method).
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

pkv_status pkv::prefill_mod_run(PrefillCall c, int format, int32_t head_dim, void *workspace, size_t workspace_bytes) {
    if (dtype_bytes(c.dtype) == 0) return set_error(PKV_ERR_INVALID_ARG, "prefill: unknown dtype %d", (int)c.dtype);
    if (format != kCode16 && format != kCodeE4M3 && format != kCodeInt8 && format != kCodeInt4)
        return set_error(PKV_ERR_INVALID_ARG, "prefill: unknown cache format %d", format);
    if (c.num_seqs < 0 || c.max_q_len < 0 || c.Hq <= 0 || c.Hkv <= 0 || head_dim <= 0 || c.block_size <= 0 ||
        c.num_blocks < 0 || c.max_blocks < 0 || c.max_total_len < 0)
        return set_error(PKV_ERR_INVALID_ARG, "prefill: bad sizes");
    if (c.Hq % c.Hkv)
        return set_error(PKV_ERR_INVALID_ARG, "prefill: num_q_heads (%d) is not a multiple of num_kv_heads (%d)", c.Hq, c.Hkv);
    if (static_cast<int64_t>(c.num_blocks) * c.block_size > INT32_MAX)
        return set_error(PKV_ERR_INVALID_ARG, "prefill: num_blocks * block_size >= 2^31");
    const float cap = c.mod.softcap;
    if (!(cap >= 0.f) || cap > 1e30f || (cap > 0.f && cap < 1e-30f))
        return set_error(PKV_ERR_INVALID_ARG, "prefill: softcap must be 0, or from 1e-30 to 1e30");
    if (c.num_seqs > 65535 || c.Hkv > 65535)
        return set_error(PKV_ERR_UNSUPPORTED, "prefill: more than 65535 sequences or KV heads");
    if (c.num_seqs == 0 || c.max_q_len == 0) return ok();
    if ((c.dtype != PKV_F16 && c.dtype != PKV_BF16) || !supported_shape(c.Hq, c.Hkv, head_dim, c.block_size))
        return set_error(PKV_ERR_UNSUPPORTED, "prefill: needs fp16/bf16, head_dim 128, Hq/Hkv in {1, 2, 4, 8} and "
                                              "block_size a multiple of 16");
    if (!c.out || !c.q || !c.starts || !c.cu_q || !c.block_tables || !c.k_cache || !c.v_cache || c.num_blocks == 0)
        return set_error(PKV_ERR_INVALID_ARG, "prefill: NULL pointer or empty pool");
    if (!aligned(c.k_cache, 16) || !aligned(c.v_cache, 16) || !aligned(c.q, 16) || !aligned(c.out, 16))
        return set_error(PKV_ERR_UNSUPPORTED, "prefill: pools, q and out must be 16-byte aligned");
    if ((format == kCodeE4M3 || format == kCodeInt8) &&
        (!c.k_scale || !c.v_scale || !aligned(c.k_scale, 4) || !aligned(c.v_scale, 4)))
        return set_error(PKV_ERR_INVALID_ARG, "prefill: scales of an 8-bit cache NULL or not 4-byte aligned");
    if (format == kCodeInt4) {
        if (!c.k_scale4 || !c.v_scale4) return set_error(PKV_ERR_INVALID_ARG, "prefill: scales of a 4-bit cache NULL");
        if (!aligned(c.k_scale4, 16) || !aligned(c.v_scale4, 16))
            return set_error(PKV_ERR_UNSUPPORTED, "prefill: scales of a 4-bit cache must be 16-byte aligned");
    }
    WidePlan w;
    if (format == kCodeInt4) {
        w = wide_plan(c.num_seqs, c.Hq, c.Hkv, c.block_size, c.max_q_len, c.max_blocks, c.max_total_len);
    }
    c.plan = prefill_plan(c.num_seqs, c.Hq, c.Hkv, c.max_q_len, w.bytes ? w.stride : c.max_blocks, c.block_size);
    const size_t need = c.plan.ws_bytes + w.bytes;
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return set_error(PKV_ERR_WORKSPACE, "prefill: workspace needs %zu bytes (256-byte aligned), got %zu", need, workspace_bytes);
    const int64_t grids = (static_cast<int64_t>(c.plan.pairs) * c.plan.nsplit + kMaxGridPairs - 1) / kMaxGridPairs;
    if (c.num_seqs * grids > 65535)
        return set_error(PKV_ERR_UNSUPPORTED, "prefill: max_q_len is too long for so many sequences");
    c.workspace = static_cast<char *>(workspace);
    if (w.bytes) {
        const pkv_status st = widen_int4(c, w, c.workspace + c.plan.ws_bytes);
        if (st != PKV_OK) return st;
        format = c.dtype == PKV_F16 ? kCode16 : kCodeF16;
    }
    const pkv_status st = format == kCodeE4M3   ? prefill_mod_e4m3(c)
                          : format == kCodeInt8 ? prefill_mod_int8(c)
                          : format == kCodeInt4 ? prefill_mod_int4(c)
                          : format == kCodeF16  ? prefill_mod_f16(c)
                                                : prefill_mod_16bit(c);
    return st == PKV_OK ? ok() : st;
}

extern "C" size_t pkv_paged_attention_prefill_int4_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                                                  int32_t head_dim, int32_t block_size, int32_t max_q_len,
                                                                  int32_t max_blocks_per_seq, int32_t max_total_len) {
    if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || block_size <= 0 ||
        max_q_len <= 0 || max_blocks_per_seq < 0 || max_total_len < 0 ||
        !supported_shape(num_q_heads, num_kv_heads, head_dim, block_size))
        return 0;
    const WidePlan w = wide_plan(num_seqs, num_q_heads, num_kv_heads, block_size, max_q_len, max_blocks_per_seq, max_total_len);
    return w.bytes + prefill_plan(num_seqs, num_q_heads, num_kv_heads, max_q_len, w.bytes ? w.stride : max_blocks_per_seq,
                                  block_size).ws_bytes;
}

extern "C" pkv_status pkv_paged_attention_prefill_mod(
    void *out, const void *q, const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
    pkv_cache_format format, const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *starts,
    const int32_t *cu_q, int32_t num_seqs, int32_t max_q_len, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int32_t num_blocks, float scale, const pkv_score_mod *mod, pkv_dtype dtype,
    void *workspace, size_t workspace_bytes, int32_t *err_flag, void *stream) {
    if (format != PKV_CACHE_DTYPE && format != PKV_CACHE_E4M3 && format != PKV_CACHE_INT8)
        return set_error(PKV_ERR_INVALID_ARG, "prefill: unknown cache format %d", (int)format);
    PrefillCall c{};
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
    if (mod) c.mod = *mod;
    c.dtype = dtype;
    c.err_flag = err_flag;
    c.stream = static_cast<cudaStream_t>(stream);
    return prefill_mod_run(c, format, head_dim, workspace, workspace_bytes);
}
