// The score-rule prefill kernels over 4-bit caches, and their entry point.
#include "pkv_prefill_mod.cuh"

pkv_status pkv::prefill_mod_int4(const PrefillCall &c) { return prefill_mod_format<kCodeInt4>(c); }

extern "C" pkv_status pkv_paged_attention_prefill_int4(
    void *out, const void *q, const void *k_cache, const void *v_cache, const uint16_t *k_scale, const uint16_t *v_scale,
    const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *starts, const int32_t *cu_q, int32_t num_seqs,
    int32_t max_q_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks,
    float scale, const pkv_score_mod *mod, pkv_dtype dtype, void *workspace, size_t workspace_bytes, int32_t *err_flag,
    void *stream) {
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
