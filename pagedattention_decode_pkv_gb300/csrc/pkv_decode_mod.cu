// Decode attention with score rules: the MOD instances of the decode kernels.
#include "pkv_decode.cuh"

namespace pkv {

pkv_status launch_stream_mod(const DecodeArgs &a, const Plan &p, pkv_dtype dtype) {
    return dtype == PKV_BF16 ? launch_stream_any<__nv_bfloat16, true>(a, p) : launch_stream_any<__half, true>(a, p);
}

pkv_status launch_generic_mod(const DecodeArgs &a, const Plan &p, pkv_dtype dtype) {
    switch (dtype) {
    case PKV_BF16: return launch_generic_and_combine<__nv_bfloat16, true>(a, p, true);
    case PKV_F16: return launch_generic_and_combine<__half, true>(a, p, true);
    default: return launch_generic_and_combine<float, true>(a, p, true);
    }
}

}  // namespace pkv
