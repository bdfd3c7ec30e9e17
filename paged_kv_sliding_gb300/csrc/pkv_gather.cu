// Cached keys and values read back: the rows of requests' pages, in order, as contiguous bf16
// K and V, which a ragged prefill takes (the way of a prefill over a 4-bit cache), or a move
// of a cache to another type.
//
//   out[out_indptr[b] + i] = scale * cache[row kv_start[b] + i of request b]
//
// Values of every cache type are exact in fp32 (and in bf16: E4M3 and E5M2 have at most 4
// significant bits, a 4-bit value times its block scale at most 6), so that the one rounding
// is that of the product with the tensor's scale to fp32 and then to bf16; with a scale of 1,
// or a power of two, there is none.
//
// Bound by memory: every byte is read once and written once, most of them written (2 bytes a
// value, from 2, 1 or 0.5625). A block takes a few tokens: its first threads find their
// requests (a binary search in out_indptr) and pages, then all threads walk the tokens' rows,
// sixteen columns a thread (one 32-byte store, whole lines for a warp), kUnroll of them loaded
// before the first is stored. Measured: 62.7 thousand rows of 8 heads of 128 as bf16 (257 MB written)
// from 4 bits 53.6 us, 0.91 of the copy rate, from E4M3 61 us (0.93), from bf16 79 us (0.96): the
// writes alone take 64-70 us as one fill of that size. Eight columns a thread, with fp32 products for
// every value, took 70 us from 4 bits, 76% of the issue slots.
#include <cmath>
#include <string>

#include "pkv_internal.h"
#include "pkv_nvtx.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kMaxTokens = 16;  // tokens of a block

struct GatherParams {
    const uint8_t *k_cache, *v_cache;
    const uint8_t *k_block_scales, *v_block_scales;
    const int32_t *kv_indptr, *kv_indices, *kv_start, *out_indptr;
    uint4 *k_out, *v_out;
    int32_t *status;
    int64_t total, num_indices;
    int32_t batch, page_size, num_pages;
    int32_t units;   // of sixteen columns of a token: num_kv_heads * head_dim / 16
    int32_t tokens;  // tokens of a block
    uint32_t magic;  // e / units = the high word of e magic for every unit e of a block's tokens; 0: divide
    bool wide;       // both outputs are 32-byte aligned
    float k_scale, v_scale;
    bool k_shifted, v_shifted;  // (see to_bf16)
    uint32_t k_factor, v_factor;
};

// Sixteen columns of a row as they lie in the cache.
template <int KV>
struct Raw {
    uint32_t w[KV == PKV_BF16 ? 8 : KV == PKV_FP4_E2M1 ? 2 : 4];
    uint8_t s;  // 4 bits: the block's scale
};

// Unit `at` of sixteen columns (of the whole cache).
template <int KV>
__device__ __forceinline__ void load16(Raw<KV> &r, const uint8_t *cache, const uint8_t *scales, int64_t at)
{
    if constexpr (KV == PKV_FP4_E2M1) {
        const uint2 v = reinterpret_cast<const uint2 *>(cache)[at];
        r.w[0] = v.x;
        r.w[1] = v.y;
        r.s = scales[at];
    } else {
#pragma unroll
        for (int i = 0; i < (KV == PKV_BF16 ? 2 : 1); ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(cache)[at * (KV == PKV_BF16 ? 2 : 1) + i];
            r.w[4 * i] = v.x;
            r.w[4 * i + 1] = v.y;
            r.w[4 * i + 2] = v.z;
            r.w[4 * i + 3] = v.w;
        }
    }
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// The unit's values times `scale` as sixteen bf16. `shifted`: scale is a power of two and
// `factor` = 2^112 scale, as two bf16. A 4-bit value times its block's scale is then a normal f16 of
// at most 6 significant bits (or 0), whose bits moved down by 3 are a bf16 2^112 times
// smaller; the product with the factor is exact, and takes half the instructions.
template <int KV>
__device__ __forceinline__ void to_bf16(const Raw<KV> &r, float scale, bool shifted, uint32_t factor, uint32_t (&out)[8])
{
    uint32_t h[8];
    if constexpr (KV == PKV_FP4_E2M1) {
        uint32_t s;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(s) : "h"((uint16_t)(r.s | r.s << 8)));
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n"
                " cvt.rn.f16x2.e2m1x2 %1, b;\n cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
                : "=r"(h[4 * i]), "=r"(h[4 * i + 1]), "=r"(h[4 * i + 2]), "=r"(h[4 * i + 3])
                : "r"(r.w[i]));
#pragma unroll
        for (int i = 0; i < 8; ++i)  // (exact)
            asm("mul.rn.f16x2 %0, %0, %1;\n" : "+r"(h[i]) : "r"(s));
        if (shifted) {
            factor = (r.s & 0x7f) == 0x7f ? 0x7fff7fffu : factor;  // a NaN of a scale
#pragma unroll
            for (int i = 0; i < 8; ++i)
                asm("mul.rn.bf16x2 %0, %1, %2;\n"
                    : "=r"(out[i])
                    : "r"((h[i] & 0x80008000u) | (h[i] >> 3 & 0x0fff0fffu)), "r"(factor));
            return;
        }
    } else if constexpr (KV == PKV_BF16) {
        if (scale == 1.f) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                out[i] = r.w[i];
            return;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            fp8x4_widen_f16<KV == PKV_FP8_E5M2>(r.w[i], h[2 * i], h[2 * i + 1]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float2 x;
        if constexpr (KV == PKV_BF16)
            x = make_float2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xffff0000u));
        else
            x = f16x2_to_float2(h[i]);
        out[i] = pack_bf16(x.x * scale, x.y * scale);
    }
}

template <int KV>
__global__ void __launch_bounds__(kThreads) gather_kernel(const GatherParams p)
{
    __shared__ int64_t slot_s[kMaxTokens];  // the token's row in the cache; -1: zeros; -2: left as it is
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t tok0 = (int64_t)blockIdx.x * p.tokens;
    const int ntok = (int)min((int64_t)p.tokens, p.total - tok0);
    if ((int)threadIdx.x < ntok) {
        const int64_t t = tok0 + threadIdx.x;
        // the last request whose rows begin at or before t
        int lo = -1, hi = p.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.out_indptr[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        int64_t slot = -2;
        if (lo >= 0 && t < p.out_indptr[lo + 1]) {
            slot = -1;
            const int64_t j = t - p.out_indptr[lo] + (p.kv_start ? p.kv_start[lo] : 0);
            const int64_t first = p.kv_indptr[lo];
            const int64_t at = j < 0 ? -1 : first + j / p.page_size;
            if (first >= 0 && at >= first && at < p.kv_indptr[lo + 1] && at < p.num_indices) {
                const int page = p.kv_indices[at];
                if ((unsigned)page < (unsigned)p.num_pages)
                    slot = (int64_t)page * p.page_size + j % p.page_size;
            }
            if (slot < 0 && p.status)
                record_status(p.status, PKV_ERR_DEVICE_BOUNDS);
        }
        slot_s[threadIdx.x] = slot;
    }
    __syncthreads();
    // items: K's units of every token of the block, then V's
    const int half = ntok * p.units;
    for (int i0 = threadIdx.x; i0 < 2 * half; i0 += kUnroll * kThreads) {
        Raw<KV> raw[kUnroll];
        int64_t slot[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kThreads;
            slot[u] = -2;
            if (i < 2 * half) {
                const bool is_v = i >= half;
                const int e = is_v ? i - half : i;
                const int t = p.magic ? (int)__umulhi((uint32_t)e, p.magic) : e / p.units;
                slot[u] = slot_s[t];
                if (slot[u] >= 0)
                    load16<KV>(raw[u], is_v ? p.v_cache : p.k_cache, is_v ? p.v_block_scales : p.k_block_scales,
                               slot[u] * p.units + (e - t * p.units));
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kThreads;
            if (slot[u] == -2)
                continue;
            const bool is_v = i >= half;
            uint32_t x[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
            if (slot[u] >= 0)
                to_bf16<KV>(raw[u], is_v ? p.v_scale : p.k_scale, is_v ? p.v_shifted : p.k_shifted,
                            is_v ? p.v_factor : p.k_factor, x);
            uint4 *dst = (is_v ? p.v_out : p.k_out) + 2 * (tok0 * p.units + (is_v ? i - half : i));
            if (p.wide) {
                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(dst), "r"(x[0]), "r"(x[1]),
                             "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                             : "memory");
            } else {
                dst[0] = make_uint4(x[0], x[1], x[2], x[3]);
                dst[1] = make_uint4(x[4], x[5], x[6], x[7]);
            }
        }
    }
}

template <int KV>
cudaError_t launch(GatherParams p, int n_sm, cudaStream_t s)
{
    // enough blocks for every SM before a block takes more tokens
    p.tokens = (int)std::min<int64_t>(kMaxTokens, std::max<int64_t>(1, p.total / (4LL * n_sm)));
    // with m = ceil(2^32 / units), e m / 2^32 exceeds e / units by less than e / 2^32, which is less
    // than the 1 / units that it has to the next whole number while e units < 2^32
    if (p.units > 1 && (uint64_t)p.tokens * p.units * p.units < (1ull << 32))
        p.magic = (uint32_t)(((1ull << 32) + p.units - 1) / p.units);
    const int64_t blocks = (p.total + p.tokens - 1) / p.tokens;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gather_kernel<KV>, p);
}

int refuse(int status, const char *what)
{
    set_last_error((std::string("pkv_gather_kv: ") + what).c_str());
    return status;
}

// 2^112 scale as two bf16, where scale is a power of two, the factor finite, and 2^-10 scale, the
// least 4-bit value, normal.
bool shift_factor(float scale, uint32_t &factor)
{
    int e;
    if (std::frexp(scale, &e) != 0.5f || e < -100 || e > 15)
        return false;
    const uint32_t bf16 = (uint32_t)(e - 1 + 112 + 127) << 7;
    factor = bf16 | bf16 << 16;
    return true;
}

bool misaligned(const void *p, uintptr_t a) { return (uintptr_t)p % a != 0; }

}  // namespace
}  // namespace pkv

extern "C" PKV_API int pkv_gather_kv(const pkv_gather_desc *desc, const void *k_cache, const void *v_cache,
                                     const void *k_block_scales, const void *v_block_scales, const int32_t *kv_indptr,
                                     const int32_t *kv_indices, const int32_t *kv_start, const int32_t *out_indptr,
                                     void *k_out, void *v_out, int32_t *status, void *stream_)
{
    using namespace pkv;
    NvtxRange range("pkv_gather_kv");
    set_last_error("");
    if (!desc)
        return refuse(PKV_ERR_INVALID_ARG, "desc is NULL");
    const pkv_gather_desc &d = *desc;
    if (d.batch_size < 0 || d.total < 0 || d.num_indices < 0 || d.num_kv_heads <= 0 || d.num_pages < 0 || d.page_size <= 0)
        return refuse(PKV_ERR_INVALID_ARG, "negative size, no heads or no page_size");
    if (d.head_dim != 64 && d.head_dim != 128 && d.head_dim != 256)
        return refuse(PKV_ERR_UNSUPPORTED, "head_dim not in {64, 128, 256}");
    if (d.kv_dtype != PKV_BF16 && d.kv_dtype != PKV_FP8_E4M3 && d.kv_dtype != PKV_FP8_E5M2 && d.kv_dtype != PKV_FP4_E2M1)
        return refuse(PKV_ERR_INVALID_ARG, "kv_dtype is not PKV_BF16, PKV_FP8_E4M3, PKV_FP8_E5M2 or PKV_FP4_E2M1");
    if (d.total > INT32_MAX || d.num_kv_heads > 65535)
        return refuse(PKV_ERR_UNSUPPORTED, "more than 2^31 - 1 rows or 65535 heads");
    if (!std::isfinite(d.k_scale) || !std::isfinite(d.v_scale))
        return refuse(PKV_ERR_INVALID_ARG, "k_scale and v_scale must be finite");
    if (d.total == 0 || d.batch_size == 0)
        return PKV_OK;
    const bool blocks = d.kv_dtype == PKV_FP4_E2M1;
    // (arrays of no pages or entries may be NULL: every row is then one that the pages do not hold)
    if ((d.num_pages > 0 && (!k_cache || !v_cache)) || !kv_indptr || (d.num_indices > 0 && !kv_indices) || !out_indptr ||
        !k_out || !v_out)
        return refuse(PKV_ERR_INVALID_ARG, "caches, kv_indptr, kv_indices, out_indptr, k_out and v_out are required");
    if (blocks ? d.num_pages > 0 && (!k_block_scales || !v_block_scales) : k_block_scales || v_block_scales)
        return refuse(PKV_ERR_INVALID_ARG, "block scales come with 4-bit caches, and these with them");
    for (const void *p : {k_cache, v_cache, k_block_scales, v_block_scales, (const void *)k_out, (const void *)v_out})
        if (misaligned(p, 16))
            return refuse(PKV_ERR_INVALID_ARG, "caches, block scales and outputs must be 16-byte aligned");
    for (const void *p : {(const void *)kv_indptr, (const void *)kv_indices, (const void *)kv_start,
                          (const void *)out_indptr, (const void *)status})
        if (misaligned(p, 4))
            return refuse(PKV_ERR_INVALID_ARG, "index arrays and status must be 4-byte aligned");
    GatherParams p{};
    p.k_cache = (const uint8_t *)k_cache;
    p.v_cache = (const uint8_t *)v_cache;
    p.k_block_scales = (const uint8_t *)k_block_scales;
    p.v_block_scales = (const uint8_t *)v_block_scales;
    p.kv_indptr = kv_indptr;
    p.kv_indices = kv_indices;
    p.kv_start = kv_start;
    p.out_indptr = out_indptr;
    p.k_out = (uint4 *)k_out;
    p.v_out = (uint4 *)v_out;
    p.status = status;
    p.total = d.total;
    p.num_indices = d.num_indices;
    p.batch = d.batch_size;
    p.page_size = d.page_size;
    p.num_pages = d.num_pages;
    p.units = d.num_kv_heads * (d.head_dim / 16);
    p.wide = !misaligned(k_out, 32) && !misaligned(v_out, 32);
    p.k_scale = d.k_scale > 0.f ? d.k_scale : 1.f;
    p.v_scale = d.v_scale > 0.f ? d.v_scale : 1.f;
    p.k_shifted = shift_factor(p.k_scale, p.k_factor);
    p.v_shifted = shift_factor(p.v_scale, p.v_factor);
    const cudaStream_t stream = (cudaStream_t)stream_;
    int dev = 0, n_sm = 0;
    cudaError_t ce = cudaGetDevice(&dev);
    if (ce == cudaSuccess)
        ce = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
    if (ce == cudaSuccess)
        ce = d.kv_dtype == PKV_BF16       ? launch<PKV_BF16>(p, n_sm, stream)
             : d.kv_dtype == PKV_FP8_E4M3 ? launch<PKV_FP8_E4M3>(p, n_sm, stream)
             : d.kv_dtype == PKV_FP8_E5M2 ? launch<PKV_FP8_E5M2>(p, n_sm, stream)
                                          : launch<PKV_FP4_E2M1>(p, n_sm, stream);
    if (ce != cudaSuccess)
        return refuse(PKV_ERR_CUDA, cudaGetErrorString(ce));
    return PKV_OK;
}
