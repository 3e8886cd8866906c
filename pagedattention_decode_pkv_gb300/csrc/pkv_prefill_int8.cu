// The score-rule prefill kernels over int8 caches.
#include "pkv_prefill_mod.cuh"

pkv_status pkv::prefill_mod_int8(const PrefillCall &c) { return prefill_mod_format<kCodeInt8>(c); }
