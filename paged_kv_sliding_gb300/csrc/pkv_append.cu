// What comes between the projections and attention, in one pass over q, k and v: each
// head of q and k divided by its root mean square and weighed, its first columns rotated
// by the token's position, q written for the attention run, k and v written into their
// slots of the paged cache (bf16 or 8-bit).
//
//   y = x / sqrt(mean(x^2) + eps) * (w + weight_offset)          (no w: y = x)
//   (a, b) -> (a cos - b sin, b cos + a sin) for the column pairs (i, i + r/2), or
//   (2i, 2i + 1) when interleaved, of the first r = rotary_dim columns
//   cache[slot] = y / scale
// Everything between the loaded bf16 and the stored value is fp32, rounded once; an 8-bit
// store takes the nearest finite value.
//
// Bound by memory: every row is read once and written once, and the pass does about one
// flop a byte. A head's row belongs to d / 8 adjacent lanes (16 bytes apiece), the sum of
// squares and the far column of a pair travel by shuffles. A lane group takes HPG heads of
// one token, whose rows are all in flight before the first is needed: HPG = 1 for few rows
// (latency: a decode step of 64 tokens x 48 heads spreads over all SMs), HPG = 4 otherwise
// (the token's cos and sin, four times a row's bytes, are then loaded once for four heads).
#include <cmath>
#include <string>

#include <cuda_fp8.h>

#include "pkv_internal.h"
#include "pkv_nvtx.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;

struct AppendParams {
    const uint16_t *q, *k, *v;
    const uint16_t *q_weight, *k_weight;
    const float *cos_sin;
    const int32_t *positions;
    const int64_t *slots;
    uint16_t *q_out, *k_out;
    void *k_cache, *v_cache;
    int32_t *status;
    int64_t q_stride, k_stride, v_stride;
    int64_t num_slots;
    int32_t num_tokens;
    int32_t num_qo_heads, num_kv_heads;
    int32_t num_heads;  // rows of a token: q heads, k heads and, with a cache, v heads
    int32_t chunks;     // lane groups of a token
    int32_t rotary_dim, max_position;
    float eps, weight_offset;
    float k_inv, v_inv;  // 1 / k_scale, 1 / v_scale
};

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Eight values of a row into the cache, `at` elements from its start.
template <int KV>
__device__ __forceinline__ void store_cache(void *cache, int64_t at, const float (&y)[8], float inv)
{
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = y[i] * inv;
    if (KV == PKV_BF16) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(cache) + at) = pack8(x);
    } else {
        constexpr __nv_fp8_interpretation_t F = KV == PKV_FP8_E4M3 ? __NV_E4M3 : __NV_E5M2;
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, F) |
                   (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, F) << 16;
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(cache) + at) = make_uint2(w[0], w[1]);
    }
}

template <int D, int HPG, int KV, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p)
{
    constexpr int G = D / 8;  // lanes of a row
    grid_dependency_wait();
    grid_launch_dependents();
    const int chunk = blockIdx.x % (unsigned)p.chunks;
    const int64_t tok = (int64_t)(blockIdx.x / (unsigned)p.chunks) * (kThreads / G) + threadIdx.x / G;
    const int l = threadIdx.x % G;  // columns 8l .. 8l + 7 of a row
    // Every lane stays for the shuffles; a row that is not there is neither read nor written.
    bool live = tok < p.num_tokens;
    int64_t slot = 0;
    if (live && p.slots) {
        slot = p.slots[tok];
        live = slot >= 0;  // a padding row
        if (slot >= p.num_slots) {
            live = false;
            if (p.status && l == 0)
                record_status(p.status, PKV_ERR_DEVICE_BOUNDS);
        }
    }
    const bool turned = 8 * l < p.rotary_dim;
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        cs[i] = sn[i] = 0.f;
    if (live && p.rotary_dim > 0) {
        const int pos = p.positions[tok];
        if ((unsigned)pos >= (unsigned)p.max_position) {
            live = false;
            if (p.status && l == 0)
                record_status(p.status, PKV_ERR_DEVICE_BOUNDS);
        } else if (turned) {
            const int half = p.rotary_dim / 2;
            const float *c = p.cos_sin + (int64_t)pos * p.rotary_dim;
            if (INTERLEAVED) {
                *reinterpret_cast<float4 *>(cs) = __ldg(reinterpret_cast<const float4 *>(c + 4 * l));
                *reinterpret_cast<float4 *>(sn) = __ldg(reinterpret_cast<const float4 *>(c + half + 4 * l));
            } else {
                const int at = 8 * l < half ? 8 * l : 8 * l - half;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    reinterpret_cast<float4 *>(cs)[i] = __ldg(reinterpret_cast<const float4 *>(c + at) + i);
                    reinterpret_cast<float4 *>(sn)[i] = __ldg(reinterpret_cast<const float4 *>(c + half + at) + i);
                }
            }
        }
    }

    const int hq = p.num_qo_heads, hkv = p.num_kv_heads;
    const int h0 = chunk * HPG;
    uint4 raw[HPG];
#pragma unroll
    for (int j = 0; j < HPG; ++j) {
        const int h = h0 + j;
        raw[j] = make_uint4(0u, 0u, 0u, 0u);
        if (live && h < p.num_heads) {
            const uint16_t *row = h < hq         ? p.q + tok * p.q_stride + h * D
                                  : h < hq + hkv ? p.k + tok * p.k_stride + (h - hq) * D
                                                 : p.v + tok * p.v_stride + (h - hq - hkv) * D;
            raw[j] = *reinterpret_cast<const uint4 *>(row + 8 * l);
        }
    }
#pragma unroll
    for (int j = 0; j < HPG; ++j) {
        const int h = h0 + j;
        if (h >= p.num_heads)
            break;  // the same for every lane
        float x[8];
        unpack8(raw[j], x);
        if (h >= hq + hkv) {  // v
            if (live)
                store_cache<KV>(p.v_cache, (slot * hkv + h - hq - hkv) * D + 8 * l, x, p.v_inv);
            continue;
        }
        const uint16_t *weight = h < hq ? p.q_weight : p.k_weight;
        if (weight) {
            float w[8], ss = 0.f;
            unpack8(__ldg(reinterpret_cast<const uint4 *>(weight) + l), w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ss += x[i] * x[i];
#pragma unroll
            for (int o = G / 2; o >= 1; o >>= 1)
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = x[i] * r * (w[i] + p.weight_offset);
        }
        if (INTERLEAVED) {
            if (turned) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = x[2 * i], b = x[2 * i + 1];
                    x[2 * i] = a * cs[i] - b * sn[i];
                    x[2 * i + 1] = b * cs[i] + a * sn[i];
                }
            }
        } else if (p.rotary_dim > 0) {
            // the other column of a pair sits rotary_dim / 16 lanes up or down
            const int step = p.rotary_dim / 16;
            const bool low = l < step;
            const int src = turned ? (low ? l + step : l - step) : l;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float other = __shfl_sync(0xffffffffu, x[i], src, G);
                if (turned)
                    x[i] = low ? x[i] * cs[i] - other * sn[i] : x[i] * cs[i] + other * sn[i];
            }
        }
        if (!live)
            continue;
        if (h < hq) {
            *reinterpret_cast<uint4 *>(p.q_out + (tok * hq + h) * D + 8 * l) = pack8(x);
        } else {
            if (p.k_out)
                *reinterpret_cast<uint4 *>(p.k_out + (tok * hkv + h - hq) * D + 8 * l) = pack8(x);
            if (p.k_cache)
                store_cache<KV>(p.k_cache, (slot * hkv + h - hq) * D + 8 * l, x, p.k_inv);
        }
    }
}

// Rows (token, head) above which a lane group takes four heads.
constexpr int64_t kFewRows = 16384;

template <int D, int KV, bool INTERLEAVED>
cudaError_t launch_di(AppendParams p, cudaStream_t s)
{
    const bool few = (int64_t)p.num_tokens * p.num_heads <= kFewRows;
    const int hpg = few ? 1 : 4;
    p.chunks = (p.num_heads + hpg - 1) / hpg;
    constexpr int kTokens = kThreads / (D / 8);  // tokens of a block
    const int64_t blocks = (((int64_t)p.num_tokens + kTokens - 1) / kTokens) * p.chunks;
    if (blocks > INT32_MAX)
        return cudaErrorInvalidConfiguration;
    // The launch may overlap the end of the kernel before it, which it waits for first thing.
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return few ? cudaLaunchKernelEx(&cfg, append_kernel<D, 1, KV, INTERLEAVED>, p)
               : cudaLaunchKernelEx(&cfg, append_kernel<D, 4, KV, INTERLEAVED>, p);
}

template <int D>
cudaError_t launch_d(const AppendParams &p, int kv_dtype, bool interleaved, cudaStream_t s)
{
    switch (kv_dtype) {
    case PKV_BF16: return interleaved ? launch_di<D, PKV_BF16, true>(p, s) : launch_di<D, PKV_BF16, false>(p, s);
    case PKV_FP8_E4M3:
        return interleaved ? launch_di<D, PKV_FP8_E4M3, true>(p, s) : launch_di<D, PKV_FP8_E4M3, false>(p, s);
    case PKV_FP8_E5M2:
        return interleaved ? launch_di<D, PKV_FP8_E5M2, true>(p, s) : launch_di<D, PKV_FP8_E5M2, false>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

int refuse(int status, const char *what)
{
    set_last_error((std::string("pkv_norm_rope_append: ") + what).c_str());
    return status;
}

bool misaligned(const void *p, uintptr_t a) { return (uintptr_t)p % a != 0; }

}  // namespace
}  // namespace pkv

extern "C" PKV_API int pkv_norm_rope_append(const pkv_append_desc *desc, const void *q, const void *k, const void *v,
                                            const void *q_weight, const void *k_weight, const float *cos_sin,
                                            const int32_t *positions, const int64_t *slots, void *q_out, void *k_out,
                                            void *k_cache, void *v_cache, int32_t *status, void *stream_)
{
    using namespace pkv;
    NvtxRange range("pkv_norm_rope_append");
    set_last_error("");
    if (!desc)
        return refuse(PKV_ERR_INVALID_ARG, "desc is NULL");
    const pkv_append_desc &d = *desc;
    if (d.num_tokens < 0 || d.num_qo_heads < 0 || d.num_kv_heads < 0 || d.num_qo_heads + (int64_t)d.num_kv_heads == 0)
        return refuse(PKV_ERR_INVALID_ARG, "negative size, or no heads");
    if (d.num_tokens > INT32_MAX || d.num_qo_heads > 65535 || d.num_kv_heads > 65535)
        return refuse(PKV_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens or 65535 heads");
    if (d.head_dim != 64 && d.head_dim != 128 && d.head_dim != 256)
        return refuse(PKV_ERR_UNSUPPORTED, "head_dim not in {64, 128, 256}");
    if (d.kv_dtype != PKV_BF16 && d.kv_dtype != PKV_FP8_E4M3 && d.kv_dtype != PKV_FP8_E5M2)
        return refuse(PKV_ERR_INVALID_ARG, "kv_dtype is not PKV_BF16, PKV_FP8_E4M3 or PKV_FP8_E5M2");
    if (d.rotary_dim < 0 || d.rotary_dim > d.head_dim)
        return refuse(PKV_ERR_INVALID_ARG, "rotary_dim outside [0, head_dim]");
    if (d.rotary_dim % 16)
        return refuse(PKV_ERR_UNSUPPORTED, "rotary_dim is not a multiple of 16");
    for (float x : {d.weight_offset, d.k_scale, d.v_scale})
        if (!std::isfinite(x))
            return refuse(PKV_ERR_INVALID_ARG, "weight_offset, k_scale and v_scale must be finite");
    if (!(d.eps >= 0.f) || !std::isfinite(d.eps))
        return refuse(PKV_ERR_INVALID_ARG, "eps must be finite and not negative");
    const bool cache = k_cache || v_cache;
    if (cache && (!k_cache || !v_cache || !slots || d.num_kv_heads == 0))
        return refuse(PKV_ERR_INVALID_ARG, "k_cache, v_cache, slots and KV heads come together");
    if (cache && (d.page_size <= 0 || d.num_pages < 0))
        return refuse(PKV_ERR_INVALID_ARG, "page_size or num_pages");
    if (d.num_tokens == 0)
        return PKV_OK;
    if (d.num_qo_heads > 0 && (!q || !q_out))
        return refuse(PKV_ERR_INVALID_ARG, "q and q_out are required");
    if (d.num_kv_heads > 0 && (!k || (!k_out && !cache) || (cache && !v)))
        return refuse(PKV_ERR_INVALID_ARG, "k (and v with a cache) and somewhere to put them are required");
    if (d.rotary_dim > 0 && (!cos_sin || !positions || d.max_position <= 0))
        return refuse(PKV_ERR_INVALID_ARG, "a rotation needs cos_sin, positions and max_position");
    if (d.q_stride < 0 || d.k_stride < 0 || d.v_stride < 0 || d.q_stride % 8 || d.k_stride % 8 || d.v_stride % 8)
        return refuse(PKV_ERR_UNSUPPORTED, "token strides must be multiples of 8 elements");
    for (const void *p : {q, k, v, q_weight, k_weight, (const void *)cos_sin, (const void *)q_out, (const void *)k_out,
                          (const void *)k_cache, (const void *)v_cache})
        if (misaligned(p, 16))
            return refuse(PKV_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
    if (misaligned(positions, 4) || misaligned(slots, 8) || misaligned(status, 4))
        return refuse(PKV_ERR_INVALID_ARG, "positions, slots or status are misaligned");
    AppendParams p{};
    p.q = (const uint16_t *)q;
    p.k = (const uint16_t *)k;
    p.v = (const uint16_t *)v;
    p.q_weight = (const uint16_t *)q_weight;
    p.k_weight = (const uint16_t *)k_weight;
    p.cos_sin = cos_sin;
    p.positions = positions;
    p.slots = slots;
    p.q_out = (uint16_t *)q_out;
    p.k_out = (uint16_t *)k_out;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.status = status;
    p.q_stride = d.q_stride;
    p.k_stride = d.k_stride;
    p.v_stride = d.v_stride;
    p.num_slots = cache ? (int64_t)d.num_pages * d.page_size : INT64_MAX;
    p.num_tokens = (int32_t)d.num_tokens;
    p.num_qo_heads = d.num_qo_heads;
    p.num_kv_heads = d.num_kv_heads;
    p.num_heads = d.num_qo_heads + (cache ? 2 : 1) * d.num_kv_heads;
    p.rotary_dim = d.rotary_dim;
    p.max_position = d.max_position;
    p.eps = d.eps;
    p.weight_offset = d.weight_offset;
    p.k_inv = 1.f / (d.k_scale > 0.f ? d.k_scale : 1.f);
    p.v_inv = 1.f / (d.v_scale > 0.f ? d.v_scale : 1.f);
    const cudaStream_t stream = (cudaStream_t)stream_;
    const cudaError_t ce = d.head_dim == 64    ? launch_d<64>(p, d.kv_dtype, d.interleaved != 0, stream)
                           : d.head_dim == 128 ? launch_d<128>(p, d.kv_dtype, d.interleaved != 0, stream)
                                               : launch_d<256>(p, d.kv_dtype, d.interleaved != 0, stream);
    if (ce != cudaSuccess)
        return refuse(PKV_ERR_CUDA, cudaGetErrorString(ce));
    return PKV_OK;
}
