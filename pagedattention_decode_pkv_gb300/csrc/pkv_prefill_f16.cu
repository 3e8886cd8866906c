// The score-rule prefill kernels over f16 pools under bf16 queries (4-bit caches, widened).
#include "pkv_prefill_mod.cuh"

pkv_status pkv::prefill_mod_f16(const PrefillCall &c) { return prefill_mod_format<kCodeF16>(c); }
