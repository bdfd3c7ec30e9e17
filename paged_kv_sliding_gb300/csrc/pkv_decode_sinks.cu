// Paged decode under a window with sinks (the first keys stay visible): the kernels of
// pkv_decode_kernel.cuh instantiated for items of two key ranges, over every cache type.
#include "pkv_decode_kernel.cuh"

namespace pkv {

cudaError_t launch_decode_sinks(const DecodeParams &p, int head_dim, int num_items, cudaStream_t s, int tile,
                                bool tma, const CUtensorMap &tk, const CUtensorMap &tv, bool overlap_prev)
{
    switch (p.kv_dtype) {
    case PKV_BF16:
        return dec::launch_decode_kv<PKV_BF16, true>(p, head_dim, num_items, s, tile, tma, tk, tv, overlap_prev);
    case PKV_FP8_E4M3:
        return dec::launch_decode_kv<PKV_FP8_E4M3, true>(p, head_dim, num_items, s, tile, tma, tk, tv, overlap_prev);
    case PKV_FP8_E5M2:
        return dec::launch_decode_kv<PKV_FP8_E5M2, true>(p, head_dim, num_items, s, tile, tma, tk, tv, overlap_prev);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkv
