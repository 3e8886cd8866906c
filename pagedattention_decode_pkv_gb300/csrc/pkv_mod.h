// What the translation units of the score-rule prefill share: the checked call
// and its plan.
#pragma once

#include <cuda_runtime.h>

#include "pkv_internal.h"

namespace pkv {

// Tile pairs per (sequence, KV head), the splits of their key blocks, and the
// workspace of the splits' partial results.
struct PrefillPlan {
    int32_t pairs = 0, nsplit = 1;
    size_t o_bytes = 0, ml_bytes = 0, ws_bytes = 0;
};

struct PrefillCall {
    void *out;
    const void *q, *k_cache, *v_cache;
    const float *k_scale, *v_scale;  // 8-bit caches
    const uint16_t *k_scale4, *v_scale4;  // 4-bit caches, f16 bits
    const int32_t *block_tables;
    int32_t max_blocks;
    const int32_t *starts, *cu_q;
    int32_t num_seqs, max_q_len, Hq, Hkv, block_size, num_blocks;
    int32_t max_total_len;  // 4-bit caches: bound on a sequence's positions, 0: the table's width
    float scale;
    pkv_score_mod mod;
    pkv_dtype dtype;
    PrefillPlan plan;
    char *workspace;
    int32_t *err_flag;
    cudaStream_t stream;
};

// One translation unit per cache format.
pkv_status prefill_mod_16bit(const PrefillCall &c);
pkv_status prefill_mod_e4m3(const PrefillCall &c);
pkv_status prefill_mod_int8(const PrefillCall &c);
pkv_status prefill_mod_int4(const PrefillCall &c);
pkv_status prefill_mod_f16(const PrefillCall &c);  // a pool of f16 values under bf16 queries

// 4-bit prefill through f16: the sequences' blocks widened once into the workspace, `stride` a
// sequence, instead of by every tile pair that reads them.  bytes 0: not for these sizes.
struct WidePlan {
    int32_t stride = 0;
    size_t pool_bytes = 0, bytes = 0;
};
WidePlan wide_plan(int32_t B, int32_t Hq, int32_t Hkv, int32_t bs, int32_t max_q_len, int32_t max_blocks, int32_t max_total_len);
// Enqueues the widening and points c at its result.
pkv_status widen_int4(PrefillCall &c, const WidePlan &w, char *workspace);

// Checks the call (whose plan and workspace are still to be set) and enqueues it; `format` is a CacheCode.
pkv_status prefill_mod_run(PrefillCall c, int format, int32_t head_dim, void *workspace, size_t workspace_bytes);

}  // namespace pkv
