// Paged decode over 8-bit K/V caches (E4M3 or E5M2, torch.float8_e4m3fn /
// torch.float8_e5m2 in flashinfer_backend.py should_use_tensor_core): the kernels of
// pkv_decode_kernel.cuh instantiated for one-byte elements. K and V tiles are
// widened to f16 in registers right before their MMAs; k_scale and v_scale
// dequantise through the logit scale and the output factor.
#include "pkv_decode_kernel.cuh"

namespace pkv {
cudaError_t launch_decode_kv8(const DecodeParams &p, int head_dim, int num_items, cudaStream_t s, int tile,
                              bool tma, const CUtensorMap &tk, const CUtensorMap &tv, bool overlap_prev)
{
    if (p.kv_dtype == PKV_FP8_E4M3)
        return dec::launch_decode_kv<PKV_FP8_E4M3, false>(p, head_dim, num_items, s, tile, tma, tk, tv, overlap_prev);
    if (p.kv_dtype == PKV_FP8_E5M2)
        return dec::launch_decode_kv<PKV_FP8_E5M2, false>(p, head_dim, num_items, s, tile, tma, tk, tv, overlap_prev);
    return cudaErrorInvalidValue;
}

}  // namespace pkv
