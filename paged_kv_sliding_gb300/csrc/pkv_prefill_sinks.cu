// Prefill under a window with sinks (the first keys stay visible), bf16 K/V: the kernels
// of pkv_prefill_kernel.cuh for the two mask modes with sinks, over paged (TMA boxes or
// cp.async gathers) and ragged K/V.
#include "pkv_prefill_kernel.cuh"

namespace pkv {
namespace {

template <int D>
cudaError_t launch_d(const PrefillParams &p, int mask_mode, bool tma_kv, const CUtensorMap &tq, const CUtensorMap &tk,
                     const CUtensorMap &tv, const CUtensorMap &to, int num_ctas, cudaStream_t s)
{
    if (p.ragged)
        return pp::launch_pp_dt_sinks<D, true, true, PKV_BF16>(p, mask_mode, tq, tk, tv, to, num_ctas, s);
    return tma_kv ? pp::launch_pp_dt_sinks<D, true, false, PKV_BF16>(p, mask_mode, tq, tk, tv, to, num_ctas, s)
                  : pp::launch_pp_dt_sinks<D, false, false, PKV_BF16>(p, mask_mode, tq, tk, tv, to, num_ctas, s);
}

}  // namespace

cudaError_t launch_prefill_pp_sinks(const PrefillParams &p, int head_dim, int mask_mode, bool tma_kv,
                                    const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                                    const CUtensorMap &to, int num_ctas, cudaStream_t s)
{
    switch (head_dim) {
    case 64: return launch_d<64>(p, mask_mode, tma_kv, tq, tk, tv, to, num_ctas, s);
    case 128: return launch_d<128>(p, mask_mode, tma_kv, tq, tk, tv, to, num_ctas, s);
    case 256: return launch_d<256>(p, mask_mode, tma_kv, tq, tk, tv, to, num_ctas, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkv
