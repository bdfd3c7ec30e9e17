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
// flop a byte; what stands in its way is the number of instructions, so that
//   - a head's row belongs to d / 8 adjacent lanes of two 8-byte pieces each, chosen so that
//     both columns of a pair are one lane's (columns 4l.. and r/2 + 4l.. for the split
//     pairs): the rotation takes no shuffle, and cos and sin are loaded once per pair;
//   - the arithmetic is on packed pairs (f32x2), four of them to a lane and row;
//   - a lane group takes HPG heads of one token and one tensor: rows, slot and position are
//     all in flight at once, and weights, cos and sin are loaded once for HPG rows.
// HPG = 1 for few rows (latency: a decode step of 64 tokens x 48 heads spreads over all
// SMs, 2.1 us), HPG = 4 otherwise. Measured on 16384 tokens x 48 heads of 128, bf16: 64.5 us
// = 6.37 TB/s, 0.94 of the copy rate; 8191 tokens of 8 + 2 x 4 heads of 256 into E4M3 22.5 us
// (with products by one rounded reciprocal 22.15; eight heads to a group, measured with
// those, 62 and 23.4 us: on the second they stay half empty).
#include <cmath>
#include <string>

#include <cuda_fp8.h>

#include "pkv_internal.h"
#include "pkv_nvtx.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;

// What a value is divided by: the divisor and its reciprocal in two parts, hi + lo, lo > 0, or
// hi alone (lo = 0) where that is exact.
struct Divisor {
    float value, hi, lo;
};

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
    int32_t chunks;  // lane groups of a token
    int32_t rotary_dim, max_position;
    float eps, weight_offset;
    Divisor k_scale, v_scale;
};

// Four bf16 values (two words) as two packed pairs of floats.
struct Quad {
    float2 a, b;
};

__device__ __forceinline__ Quad widen(uint2 w)
{
    return {make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u)),
            make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u))};
}

__device__ __forceinline__ uint2 narrow(const Quad &x)
{
    return make_uint2(pack_bf16(x.a.x, x.a.y), pack_bf16(x.b.x, x.b.y));
}

__device__ __forceinline__ float2 mul2(float2 x, float2 y)
{
    float2 r;
    asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n mul.rn.f32x2 rd, ra, rb;\n"
        " mov.b64 {%0, %1}, rd;\n}\n"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}

__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z)
{
    float2 r;
    pkv::fma2(r.x, r.y, x.x, x.y, y.x, y.y, z.x, z.y);
    return r;
}

__device__ __forceinline__ Quad scaled(const Quad &x, float f)
{
    return {mul2(x.a, make_float2(f, f)), mul2(x.b, make_float2(f, f))};
}

// a / b to nearest, subnormals kept (the build's fast division is neither).
__device__ __forceinline__ float divide(float a, float b)
{
    float r;
    asm("div.rn.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// x / s. A product with the rounded reciprocal alone is off by up to 1.5 steps of fp32, which
// moves a quotient halfway between two stored values (bf16 inputs give many) to either
// side. x hi + x lo, the small product rounded and the sum of a fused multiply-add (the
// multiplication by a constant of Brisebarre and Muller, 2008), is off by a relative
// 2^-47 before its one rounding: every quotient that is a float comes out as it is, those
// halves among them, and another as the nearest float unless it lies that close to the
// middle of two. (Not below 2^-100, where x lo loses bits; an 8-bit type holds nothing there.)
// With lo > 0 an infinity stays one. DIVIDE, the division instruction, is for the rest: bf16
// stores, and divisors whose parts would leave the normal floats. On 16384 tokens of bf16
// it takes 74.6 us against 64.5 with the products; in one kernel with them its registers
// alone cost 6%, so that it has kernels of its own.
template <int KV, bool DIVIDE>
__device__ __forceinline__ Quad over(const Quad &x, const Divisor &s)
{
    if (DIVIDE)
        return {make_float2(divide(x.a.x, s.value), divide(x.a.y, s.value)),
                make_float2(divide(x.b.x, s.value), divide(x.b.y, s.value))};
    if (KV == PKV_BF16 || s.lo == 0.f)
        return scaled(x, s.hi);
    const float2 hi = make_float2(s.hi, s.hi);
    const Quad low = scaled(x, s.lo);
    return {fma2(x.a, hi, low.a), fma2(x.b, hi, low.b)};
}

// The lane's two pieces of a row, at columns c0 and c1; ONE: c1 = c0 + 4, one access.
template <bool ONE>
__device__ __forceinline__ void load_row(const uint16_t *row, int c0, int c1, uint2 (&raw)[2])
{
    if (ONE) {
        const uint4 v = *reinterpret_cast<const uint4 *>(row + c0);
        raw[0] = make_uint2(v.x, v.y);
        raw[1] = make_uint2(v.z, v.w);
    } else {
        raw[0] = *reinterpret_cast<const uint2 *>(row + c0);
        raw[1] = *reinterpret_cast<const uint2 *>(row + c1);
    }
}

template <int KV, bool ONE>
__device__ __forceinline__ void store_row(void *base, int64_t at, int c0, int c1, const Quad &x0, const Quad &x1)
{
    if (KV == PKV_BF16) {
        uint16_t *row = static_cast<uint16_t *>(base) + at;
        const uint2 w0 = narrow(x0), w1 = narrow(x1);
        if (ONE) {
            *reinterpret_cast<uint4 *>(row + c0) = make_uint4(w0.x, w0.y, w1.x, w1.y);
        } else {
            *reinterpret_cast<uint2 *>(row + c0) = w0;
            *reinterpret_cast<uint2 *>(row + c1) = w1;
        }
    } else {
        constexpr __nv_fp8_interpretation_t F = KV == PKV_FP8_E4M3 ? __NV_E4M3 : __NV_E5M2;
        uint8_t *row = static_cast<uint8_t *>(base) + at;
        const uint32_t w0 = __nv_cvt_float2_to_fp8x2(x0.a, __NV_SATFINITE, F) |
                            (uint32_t)__nv_cvt_float2_to_fp8x2(x0.b, __NV_SATFINITE, F) << 16;
        const uint32_t w1 = __nv_cvt_float2_to_fp8x2(x1.a, __NV_SATFINITE, F) |
                            (uint32_t)__nv_cvt_float2_to_fp8x2(x1.b, __NV_SATFINITE, F) << 16;
        if (ONE) {
            *reinterpret_cast<uint2 *>(row + c0) = make_uint2(w0, w1);
        } else {
            *reinterpret_cast<uint32_t *>(row + c0) = w0;
            *reinterpret_cast<uint32_t *>(row + c1) = w1;
        }
    }
}

template <int D, int HPG, int KV, bool INTERLEAVED, bool DIVIDE>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p)
{
    constexpr int G = D / 8;  // lanes of a row
    grid_dependency_wait();
    grid_launch_dependents();
    // The block's tensor and heads: q's chunks first, then k's, then v's.
    int chunk = blockIdx.x % (unsigned)p.chunks;
    const int64_t tok = (int64_t)(blockIdx.x / (unsigned)p.chunks) * (kThreads / G) + threadIdx.x / G;
    const int l = threadIdx.x % G;
    const int hq = p.num_qo_heads, hkv = p.num_kv_heads;
    const int q_chunks = (hq + HPG - 1) / HPG, kv_chunks = (hkv + HPG - 1) / HPG;
    const bool is_q = chunk < q_chunks, is_v = chunk >= q_chunks + kv_chunks;
    chunk -= is_q ? 0 : is_v ? q_chunks + kv_chunks : q_chunks;
    const int heads = is_q ? hq : hkv, h0 = chunk * HPG;
    // First columns of the lane's two pieces. Lanes past the rotated columns, and all of
    // them for adjacent pairs, hold eight columns in a row.
    const bool turned = 8 * l < p.rotary_dim && !is_v;
    const bool split = !INTERLEAVED && turned;
    const int c0 = split ? 4 * l : 8 * l, c1 = split ? p.rotary_dim / 2 + 4 * l : 8 * l + 4;

    // Every lane stays for the shuffles; a row that is not there is neither read nor written.
    // The token's slot and position and the rows themselves are all loaded at once.
    const bool there = tok < p.num_tokens;
    const int64_t slot = !there ? -1 : p.slots ? p.slots[tok] : 0;
    const int pos = there && p.rotary_dim > 0 ? p.positions[tok] : 0;
    const uint16_t *row = (is_q ? p.q + tok * p.q_stride : is_v ? p.v + tok * p.v_stride : p.k + tok * p.k_stride) + h0 * D;
    uint2 raw[HPG][2];
#pragma unroll
    for (int j = 0; j < HPG; ++j) {
        raw[j][0] = raw[j][1] = make_uint2(0u, 0u);
        if (there && h0 + j < heads) {
            // (one form for every tensor: a branch here keeps the loads apart, 64.7 -> 70.9 us)
            load_row<INTERLEAVED>(row + j * D, c0, c1, raw[j]);
        }
    }
    bool live = slot >= 0;  // negative: a padding row
    if (slot >= p.num_slots || (live && p.rotary_dim > 0 && (unsigned)pos >= (unsigned)p.max_position)) {
        live = false;
        if (p.status && l == 0)
            record_status(p.status, PKV_ERR_DEVICE_BOUNDS);
    }
    if (is_v) {
#pragma unroll
        for (int j = 0; j < HPG; ++j) {
            if (live && h0 + j < heads)
                store_row<KV, true>(p.v_cache, (slot * hkv + h0 + j) * D, c0, c1,
                                    over<KV, DIVIDE>(widen(raw[j][0]), p.v_scale),
                                    over<KV, DIVIDE>(widen(raw[j][1]), p.v_scale));
        }
        return;
    }
    // cos and sin of the lane's four pairs
    Quad cs{}, sn{};
    if (live && turned) {
        const float *c = p.cos_sin + (int64_t)pos * p.rotary_dim + 4 * l;
        const float4 x = *reinterpret_cast<const float4 *>(c);
        const float4 y = *reinterpret_cast<const float4 *>(c + p.rotary_dim / 2);
        cs = {make_float2(x.x, x.y), make_float2(x.z, x.w)};
        sn = {make_float2(y.x, y.y), make_float2(y.z, y.w)};
    }
    const uint16_t *weight = is_q ? p.q_weight : p.k_weight;
    Quad w0{}, w1{};
    if (weight) {
        w0 = widen(*reinterpret_cast<const uint2 *>(weight + c0));
        w1 = widen(*reinterpret_cast<const uint2 *>(weight + c1));
        for (float2 *w : {&w0.a, &w0.b, &w1.a, &w1.b})
            *w = make_float2(w->x + p.weight_offset, w->y + p.weight_offset);
    }
#pragma unroll
    for (int j = 0; j < HPG; ++j) {
        if (h0 + j >= heads)
            break;  // the same for every lane
        Quad x0 = widen(raw[j][0]), x1 = widen(raw[j][1]);
        if (weight) {
            float2 s2 = fma2(x1.b, x1.b, fma2(x1.a, x1.a, fma2(x0.b, x0.b, mul2(x0.a, x0.a))));
            float ss = s2.x + s2.y;
#pragma unroll
            for (int o = G / 2; o >= 1; o >>= 1)
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = rsqrtf(ss * (1.f / D) + p.eps);
            x0 = scaled(x0, r);
            x1 = scaled(x1, r);
            x0 = {mul2(x0.a, w0.a), mul2(x0.b, w0.b)};
            x1 = {mul2(x1.a, w1.a), mul2(x1.b, w1.b)};
        }
        if (!live)
            continue;
        if (turned) {
            // the first and second columns of the four pairs
            Quad a = x0, b = x1;
            if (INTERLEAVED) {
                a = {make_float2(x0.a.x, x0.b.x), make_float2(x1.a.x, x1.b.x)};
                b = {make_float2(x0.a.y, x0.b.y), make_float2(x1.a.y, x1.b.y)};
            }
            const Quad neg = scaled(sn, -1.f);
            const Quad ra{fma2(a.a, cs.a, mul2(b.a, neg.a)), fma2(a.b, cs.b, mul2(b.b, neg.b))};
            const Quad rb{fma2(b.a, cs.a, mul2(a.a, sn.a)), fma2(b.b, cs.b, mul2(a.b, sn.b))};
            if (INTERLEAVED) {
                x0 = {make_float2(ra.a.x, rb.a.x), make_float2(ra.a.y, rb.a.y)};
                x1 = {make_float2(ra.b.x, rb.b.x), make_float2(ra.b.y, rb.b.y)};
            } else {
                x0 = ra;
                x1 = rb;
            }
        }
        uint16_t *out = is_q ? p.q_out : p.k_out;
        if (out)
            store_row<PKV_BF16, INTERLEAVED>(out, (tok * heads + h0 + j) * D, c0, c1, x0, x1);
        if (!is_q && p.k_cache)
            store_row<KV, INTERLEAVED>(p.k_cache, (slot * hkv + h0 + j) * D, c0, c1, over<KV, DIVIDE>(x0, p.k_scale),
                                       over<KV, DIVIDE>(x1, p.k_scale));
    }
}

// Values of q, k and v below which a lane group takes one head, otherwise kManyHeads; a call
// without two heads in any tensor, whose groups of four would stay three quarters empty,
// takes one at any size. Measured in us, one head against four, bf16: 32 + 2 x 8 heads of
// 64, 12288 rows 2.12 / 2.49, 16384 2.83 / 2.49, 24576 2.93 / 2.70; of 128, 4096 rows 1.97 /
// 2.39, 8192 2.79 / 2.57; of 256, 4096 rows 2.81 / 2.58, 65536 17.8 / 9.6; 1 + 2 x 1 heads of
// 128, 8192 rows 2.68 / 2.77, 196608 26.4 / 30.4. Heads that fill half of their groups lose
// between 1.4 and 2.1 million values (5 + 2 x 1 of 64, 24576 rows 2.89 / 3.50; 32768 3.29 /
// 3.54) and gain on either side (2 + 2 x 2, 16384 rows 2.67 / 2.27, 49152 4.11 / 3.52).
constexpr int kManyHeads = 4;
constexpr int64_t kFewValues = 1 << 20;

template <int D, int KV, bool INTERLEAVED>
cudaError_t launch_di(AppendParams p, cudaStream_t s)
{
    const bool few = (p.num_qo_heads <= 1 && p.num_kv_heads <= 1) ||
                     (int64_t)p.num_tokens * (p.num_qo_heads + 2 * p.num_kv_heads) * D < kFewValues;
    const int hpg = few ? 1 : kManyHeads;
    const int kv_chunks = (p.num_kv_heads + hpg - 1) / hpg;
    p.chunks = (p.num_qo_heads + hpg - 1) / hpg + (p.k_cache ? 2 : 1) * kv_chunks;
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
    bool divide = false;
    for (const Divisor &s : {p.k_scale, p.v_scale})
        divide |= s.hi == 0.f || (KV == PKV_BF16 && s.lo != 0.f);
    return cudaLaunchKernelEx(&cfg,
                              few ? divide ? append_kernel<D, 1, KV, INTERLEAVED, true>
                                           : append_kernel<D, 1, KV, INTERLEAVED, false>
                              : divide ? append_kernel<D, kManyHeads, KV, INTERLEAVED, true>
                                       : append_kernel<D, kManyHeads, KV, INTERLEAVED, false>,
                              p);
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

// The divisor of a descriptor's scale. hi = 0: its reciprocal is not finite, or it is no power
// of two and outside [2^-64, 2^64), where lo (at least 2^-49 of hi) would not stay normal.
Divisor divisor(float scale)
{
    const float x = scale > 0.f ? scale : 1.f;
    int e;
    if (std::frexp(x, &e) == 0.5f) {
        const float r = std::ldexp(1.f, 1 - e);
        return {x, std::isfinite(r) ? r : 0.f, 0.f};
    }
    if (e < -63 || e > 64)
        return {x, 0.f, 0.f};
    float hi = (float)(1.0 / x);
    if ((double)hi * x > 1.0)  // (a product of two floats is exact in double)
        hi = std::nextafter(hi, 0.f);
    return {x, hi, (float)((1.0 - (double)hi * x) / x)};
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
    if (d.num_tokens == 0)
        return PKV_OK;
    const bool cache = k_cache || v_cache;
    if (cache && (!k_cache || !v_cache || !slots || d.num_kv_heads == 0))
        return refuse(PKV_ERR_INVALID_ARG, "k_cache, v_cache, slots and KV heads come together");
    if (cache && (d.page_size <= 0 || d.num_pages < 0))
        return refuse(PKV_ERR_INVALID_ARG, "page_size or num_pages");
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
    p.rotary_dim = d.rotary_dim;
    p.max_position = d.max_position;
    p.eps = d.eps;
    p.weight_offset = d.weight_offset;
    p.k_scale = divisor(d.k_scale);
    p.v_scale = divisor(d.v_scale);
    const cudaStream_t stream = (cudaStream_t)stream_;
    const cudaError_t ce = d.head_dim == 64    ? launch_d<64>(p, d.kv_dtype, d.interleaved != 0, stream)
                           : d.head_dim == 128 ? launch_d<128>(p, d.kv_dtype, d.interleaved != 0, stream)
                                               : launch_d<256>(p, d.kv_dtype, d.interleaved != 0, stream);
    if (ce != cudaSuccess)
        return refuse(PKV_ERR_CUDA, cudaGetErrorString(ce));
    return PKV_OK;
}
