// Internal declarations shared by the host plan code and the kernels of libpkv.
// Not part of the C ABI (include/pkv.h is).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "pkv.h"

namespace pkv {

// Per-request facts the kernels need, computed once by the plan.
struct RequestInfo {
    int32_t qo_begin;       // first global query row (qo_indptr[b])
    int32_t qo_len;         // query rows of the request
    int32_t kv_len;         // valid tokens in its pages
    int32_t kv_page_begin;  // kv_indptr[b]
    int32_t q_start;        // position of its first query row
    int32_t pad0, pad1, pad2;
};

// One work item of the prefill kernel: one or two tiles of packed query rows (query
// tokens x the KV head's query-head group) of one request against the kv_tiles KV
// tiles from key kv_start on, which cover every key its positions can see.
struct PrefillItem {
    int32_t req;
    int32_t kv_head;
    int32_t tok0;        // first query token of the tile, within the request
    int32_t ntok;        // query tokens in the tile
    int32_t kv_start;    // first key of the item's first KV tile (aligned for the loader)
    int32_t kv_tiles;    // KV tiles of the item (0: no visible key)
    int32_t kv_tile_rot; // tiles are visited from tile kv_tile_rot on, wrapping around
    int32_t join;        // plans with sinks: packed rows below it are the first keys themselves
};

// First row of the KV tile visited at step j (0 <= j < kv_tiles) of a prefill item
// whose tiles hold T keys. Softmax accumulation is order-independent; staggering the
// start keeps the items that run at the same time on one KV head from all missing L2
// on the same tile. Rows are keys, counted from the item's first key; in a plan with
// sinks they are packed: the pages of the sinks, then directly those of the window.
template <bool SINK = false>
__host__ __device__ inline int prefill_kv_row_at(const PrefillItem &it, int j, int T)
{
    const int k = j + it.kv_tile_rot;
    return (SINK ? 0 : it.kv_start) + (k < it.kv_tiles ? k : k - it.kv_tiles) * T;
}

// The key of a row: rows at and above `join` lie kv_start keys further on (sinks).
template <bool SINK = false>
__host__ __device__ inline int prefill_row_key(const PrefillItem &it, int row)
{
    return SINK && row >= it.join ? row + it.kv_start : row;
}

// One CTA of the decode kernel: up to kDecodeRows query heads of one request's
// single row against the key range [j0, j1) of one KV head (and, in a plan with sinks,
// the first keys [0, sink_end) before it).
struct DecodeItem {
    int32_t req;
    int32_t kv_head;
    int32_t head0;    // first query head handled
    int32_t nheads;   // query heads handled (<= kDecodeRows)
    int32_t j0, j1;   // key range, already clipped to the visible interval
    int32_t partial;  // -1: write out/lse directly; else partial slot of this split
    int32_t pbase;    // first partial slot of the request (split items)
    int32_t nsplit;   // splits of the request (split items)
    int32_t counter;  // arrival counter of this (request, KV head, head block) group
    // The request's facts the kernel needs, carried here so that a CTA's first
    // page-table read does not wait behind a second dependent load.
    int32_t row;            // the request's query row (its qo_begin)
    int32_t kv_len;         // keys in the request's cache
    int32_t kv_page_begin;  // the request's first entry in kv_indices
    int32_t sink_end;       // keys [0, sink_end) are visible too (sink plans; <= j0)
};

// Merge of a request's split-KV partial states into its output row.
struct MergeItem {
    int32_t row;            // global query row
    int32_t partial_begin;  // first partial slot
    int32_t num_partials;   // splits to combine
    int32_t pad;
};

constexpr int kDecodeRows = 16;   // query heads per decode CTA (one m16 MMA tile)
constexpr int kPrefillRows = 128; // packed query rows per prefill CTA (UMMA M)

enum MaskMode : int32_t {
    kMaskNone = 0,
    kMaskCausal = 1,
    kMaskCausalWindow = 2,
    kMaskWindow = 3,
    kMaskCausalWindowSinks = 4,
    kMaskWindowSinks = 5
};

struct DecodeParams {
    const DecodeItem *items;
    const int32_t *live_items;  // non-NULL: CTAs at or above *live_items have no work
    const RequestInfo *reqs;
    const int32_t *kv_indices;
    const uint16_t *q;
    const uint16_t *k_cache;
    const uint16_t *v_cache;
    uint16_t *out;
    float *lse;          // may be null
    float *partial_o;    // [num_partials, num_qo_heads, head_dim]
    float *partial_lse;  // [num_partials, num_qo_heads]
    int32_t *merge_counters;  // non-null: the last split CTA of a group merges its partials
    int32_t *status;
    int32_t num_qo_heads;
    int32_t num_kv_heads;
    int32_t page_size;
    int32_t page_shift;  // log2(page_size) when a power of two, else -1
    int32_t num_pages;
    float sm_scale_log2; // sm_scale * k_scale * log2(e)
    float cap_in;        // soft cap: dot -> cap_out * tanh(dot * cap_in); cap_in = 0: none
    float cap_out;
    float v_scale;       // multiplies the final output
    int32_t kv_dtype;    // element type of the caches (pkv_dtype: bf16 or an 8-bit float)
    int32_t wait_probe;  // nonzero: each CTA's first consuming wait is on a barrier nothing completes
    int32_t sinks;       // nonzero: the items may see sinks (the kernels for two key ranges)
    long long wait_ns;   // bound of every wait (globaltimer nanoseconds)
};

struct MergePartialsParams {
    const MergeItem *items;
    const float *partial_o;
    const float *partial_lse;
    uint16_t *out;
    float *lse;
    int32_t num_items;
    int32_t num_qo_heads;
    float v_scale;  // multiplies the merged output
};

struct PrefillParams {
    const PrefillItem *items;    // grouped by CTA
    const int32_t *cta_items;    // CTA c runs items [cta_items[c], cta_items[c + 1])
    const RequestInfo *reqs;
    const int32_t *kv_indices;
    const uint16_t *q;
    const uint16_t *k_cache;
    const uint16_t *v_cache;
    uint16_t *out;
    float *lse;
    int32_t *status;
    int32_t num_qo_heads;
    int32_t num_kv_heads;
    int32_t group;           // num_qo_heads / num_kv_heads
    int32_t tokens_per_tile; // query tokens per CTA = floor(128 / group)
    int32_t page_size;
    int32_t page_shift;
    int32_t num_pages;
    int32_t window_left;
    int32_t sinks;           // keys [0, sinks) stay visible under the window (0: none)
    int32_t total_q;         // rows of q (bound of the query tensor map)
    float sm_scale_log2;     // sm_scale * k_scale * log2(e)
    float cap_in;            // soft cap, as in DecodeParams
    float cap_out;
    float v_scale;
    int32_t ragged;          // 1: K/V are contiguous [total_kv, H_kv, d], kv_page_begin = token offset
    int32_t total_kv;        // ragged: rows of K/V (bound of their tensor maps)
    int32_t kv_dtype;        // element type of the caches (pkv_dtype: bf16 or an 8-bit float)
    int32_t wait_probe;      // as in DecodeParams
    long long wait_ns;       // as in DecodeParams
};

// Bound of every wait inside the kernels: the descriptor's wait_limit_us, or 2 s.
constexpr long long kDefaultWaitNs = 2000000000LL;
inline long long wait_ns_of(const pkv_plan_desc &d)
{
    return d.wait_limit_us > 0 ? (long long)d.wait_limit_us * 1000LL : kDefaultWaitNs;
}

// The logit and output factors of a plan descriptor (k_scale folded into the logit
// scale; scales <= 0 mean 1; a soft cap <= 0 means none).
struct LogitFactors {
    float sm_scale_log2, cap_in, cap_out, v_scale;
};
inline LogitFactors logit_factors(const pkv_plan_desc &d)
{
    const float ks = d.k_scale > 0.f ? d.k_scale : 1.f;
    const float vs = d.v_scale > 0.f ? d.v_scale : 1.f;
    const float s = d.sm_scale * ks;
    LogitFactors f;
    f.sm_scale_log2 = s * 1.4426950408889634f;
    f.cap_in = d.logits_soft_cap > 0.f ? s / d.logits_soft_cap : 0.f;
    f.cap_out = d.logits_soft_cap > 0.f ? d.logits_soft_cap / s : 0.f;
    f.v_scale = vs;
    return f;
}

// Launchers (one per kernel family); return cudaGetLastError() of the launch.
// tile: KV tokens per stage, 64 or (head_dim <= 128) 32. overlap_prev: the kernel's
// set-up may overlap the previous kernel in the stream (programmatic dependent
// launch); false when that kernel writes the work list the decode reads first.
cudaError_t launch_decode(const DecodeParams &p, int head_dim, int num_items, cudaStream_t s, int tile,
                          bool overlap_prev = true);
// KV tile of the decode kernel (head_dim <= 128): 32 tokens (4 CTAs per SM) for
// short key ranges, which are latency-bound, and for medium ones (<= 1024 keys)
// whose CTAs need more than one wave at 2 per SM but fit in one at 4; otherwise 64
// (twice the bytes in flight per CTA, which long ranges need).
inline int decode_tile_for(int head_dim, int64_t max_keys, int64_t n_items, int n_sm)
{
    if (head_dim > 128)
        return 64;
    if (max_keys <= 192)
        return 32;
    if (max_keys <= 1024 && n_items > 2LL * n_sm && n_items <= 4LL * n_sm)
        return 32;
    return 64;
}

// The same for plans with sinks, whose kernels are others: 64 while the items fit in one wave
// of such CTAs (2 on an SM at head_dim 128, 3 at 64), 32, of which an SM holds twice as many,
// beyond, for ranges of up to 1536 keys (640 just above one wave). Measured, 32 against 64 in
// us, 8 KV heads, pages of 16, bf16 (or E4M3): d 128, 8 items of 132 keys 5.65 / 4.81, 304
// of 132 6.82 / 6.06, 512 of 132 7.45 / 11.33, 312 of 505 15.3 / 16.7, of 1028 28.3 / 26.8,
// 512 of 1028 41.1 / 45.9 (26.1 / 32.2), of 2005 63.0 / 61.6; d 64, 352 of 1028 23.7 / 17.1
// (448: 18.8 / 15.1), 512 of 505 14.4 / 18.3, 608 of 1028 26.9 / 34.8. Over 1684 measured
// batches (1 to 200 requests, 9 to 2005 keys, pages of 1, 5, 16 and 64) the choice is within
// 5% of the better one in 1532 and 1.3% slower in the mean; it loses most where lengths
// happen to fill the other's waves (384 items of 1405 keys, E4M3: 29.5 / 24.1), on E4M3 ranges
// of some 20 keys (3.7 / 4.5 at d 64) and beyond 1536 keys with gathered pages (d 64, E4M3,
// pages of 5, 608 items of 1705 keys: 46.9 / 73.6).
inline int decode_sinks_tile_for(int head_dim, int64_t max_keys, int64_t n_items, int n_sm)
{
    const int wave = head_dim == 64 ? 3 : 2;  // items per SM
    if (head_dim > 128 || n_items <= (int64_t)wave * n_sm)
        return 64;
    return max_keys <= (4 * n_items > (4LL * wave + 1) * n_sm ? 1536 : 640) ? 32 : 64;
}

// KV tokens per stage of the decode kernel that runs a plan's tile variant (32: short
// key ranges; 64: the rest): 8-bit caches at head_dim <= 128 run both variants with
// two 16-token sub-blocks per compute warp, so their stages are twice as long (64 and
// 128 tokens).
inline int decode_kernel_tile(int tile, int head_dim, int kv_dtype)
{
    return (kv_dtype != PKV_BF16 && head_dim <= 128) ? 2 * tile : tile;
}
// Page sizes whose pages the decode kernel loads with TMA boxes of a `tile`-token stage.
bool decode_tma_page_size(int page_size, int tile);
// Tensor map over a cache of kv_dtype elements for the decode kernel's TMA page boxes:
// bf16, 5-D [8-row blocks][KV head][128-byte plane][row in block][64], one box = box_rows
// rows of one KV head with every plane (the group-major stage layout); 8-bit, 4-D
// [page, slot, KV head, d], one box = one 128-byte plane (64 bytes at d 64) x box_rows.
bool encode_kv_map(CUtensorMap *m, const void *base, int head_dim, int num_kv_heads, int page_size,
                   int num_pages, int box_rows, int kv_dtype);
// The 8-bit-cache decode kernels (p.kv_dtype = PKV_FP8_E4M3 or PKV_FP8_E5M2).
cudaError_t launch_decode_kv8(const DecodeParams &p, int head_dim, int num_items, cudaStream_t s, int tile,
                              bool tma, const CUtensorMap &tk, const CUtensorMap &tv, bool overlap_prev);
// The decode kernels of plans with sinks, over any cache type.
cudaError_t launch_decode_sinks(const DecodeParams &p, int head_dim, int num_items, cudaStream_t s, int tile,
                                bool tma, const CUtensorMap &tk, const CUtensorMap &tv, bool overlap_prev);
cudaError_t launch_merge_partials(const MergePartialsParams &p, int head_dim, cudaStream_t s);
cudaError_t launch_merge_state(const void *v_a, const float *s_a, const void *v_b,
                               const float *s_b, void *v_out, float *s_out, int64_t rows,
                               int head_dim, int dtype, cudaStream_t s);
// One persistent CTA per entry of cta_items (num_ctas + 1 offsets).
cudaError_t launch_prefill_pp(const PrefillParams &p, int head_dim, int mask_mode, int num_ctas,
                              cudaStream_t s);
// Page sizes whose pages the prefill kernel loads with TMA boxes.
bool prefill_pp_tma_page_size(int page_size, int head_dim);
// The prefill kernels over 8-bit caches (p.kv_dtype = PKV_FP8_E4M3 or PKV_FP8_E5M2).
cudaError_t launch_prefill_pp_kv8(const PrefillParams &p, int head_dim, int mask_mode, int num_ctas,
                                  cudaStream_t s);
// The prefill kernels of plans with sinks (mask modes kMaskCausalWindowSinks and
// kMaskWindowSinks): bf16 caches with the launch's tensor maps, and 8-bit caches.
cudaError_t launch_prefill_pp_sinks(const PrefillParams &p, int head_dim, int mask_mode, bool tma_kv,
                                    const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                                    const CUtensorMap &to, int num_ctas, cudaStream_t s);
cudaError_t launch_prefill_pp_kv8_sinks(const PrefillParams &p, int head_dim, int mask_mode, int num_ctas,
                                        cudaStream_t s);

// Allow `kernel` its dynamic shared memory on the current device; `done` holds the devices
// (a bit each) on which that was said before, by any thread.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)))
        return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64)
        done.fetch_or(1ull << dev, std::memory_order_relaxed);
    return e;
}

// Set the calling thread's pkv_last_error() text.
void set_last_error(const char *msg);

// KV tile (tokens) of the prefill kernels for a head_dim.
int prefill_kv_tile(int head_dim);
// Query tokens per prefill CTA: one 128-row tile (head_dim 256) or two (64, 128).
inline int prefill_tokens_per_cta(int head_dim, int group)
{
    const int tq = group < kPrefillRows ? kPrefillRows / group : 1;
    return head_dim <= 128 ? 2 * tq : tq;
}

}  // namespace pkv
