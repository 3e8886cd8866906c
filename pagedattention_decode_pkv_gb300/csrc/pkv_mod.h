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
    const int32_t *block_tables;
    int32_t max_blocks;
    const int32_t *starts, *cu_q;
    int32_t num_seqs, max_q_len, Hq, Hkv, block_size, num_blocks;
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

}  // namespace pkv
