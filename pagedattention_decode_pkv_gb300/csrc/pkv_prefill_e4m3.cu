// The score-rule prefill kernels over E4M3 caches.
#include "pkv_prefill_mod.cuh"

pkv_status pkv::prefill_mod_e4m3(const PrefillCall &c) { return prefill_mod_format<kCodeE4M3>(c); }
