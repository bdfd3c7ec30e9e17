// Host side of libpkv: argument validation, the plan (work decomposition with the
// window fixed at plan time), run dispatch and error reporting.
//
// The plan follows the shape of the pages' plan/run split (sglang
// flashinfer_backend.py page: in section fast_prefill_plan the schedule comes from
// host-known query and KV layouts without a device-to-host read; in section
// call_begin_forward the plan receives kv_indptr, kv_indices and kv_last_page_len)
// with the change sglang PR #31501 asks for: window_left and causal are given to the
// plan, and the run cannot override them.
#include <algorithm>
#include <cfloat>
#include <cstdarg>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <exception>
#include <functional>
#include <new>
#include <numeric>
#include <queue>
#include <string>
#include <vector>

#include "pkv_internal.h"
#include "pkv_nvtx.h"

using namespace pkv;

namespace {

thread_local std::string g_last_error;

int fail(int status, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int status, const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return status;
}

int cuda_fail(cudaError_t e, const char *what)
{
    return fail(e == cudaErrorMemoryAllocation ? PKV_ERR_OOM : PKV_ERR_CUDA, "%s: %s", what,
                cudaGetErrorString(e));
}

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

}  // namespace

void pkv::set_last_error(const char *msg) { g_last_error = msg ? msg : ""; }

struct pkv_plan {
    pkv_plan_desc desc{};  // host pointers cleared after planning
    int device = 0;
    int mask_mode = kMaskNone;
    int num_items = 0;
    int num_partials = 0;
    int num_ctas = 0;  // prefill: persistent CTAs (lists)
    int n_sm = 0;
    // Capturable plans: launch shapes and workspace sized by the declared capacity,
    // re-planned in place by pkv_plan_update through two pinned staging images.
    bool capturable = false;
    int64_t cap_items = 0, cap_total_q = 0, cap_batch = 0;
    size_t upload_bytes = 0;
    void *staging[2] = {nullptr, nullptr};
    cudaEvent_t staging_done[2] = {nullptr, nullptr};
    int staging_next = 0;
    int32_t *d_live = nullptr;  // live work items (capturable decode launches exit above it)
    int64_t total_kv = 0;       // ragged prefill: rows of the contiguous K/V
    int sinks = 0;              // keys [0, sinks) stay visible under the window (0: none)
    int decode_tile = 64;  // decode: KV tokens per stage of the kernel
    bool shared = false;   // decode with shared prefixes: the prefix kernel runs before the decode
    int num_shared_ctas = 0;
    SharedItem *d_shared_items = nullptr;
    int32_t *d_shared_cta = nullptr;
    SharedRow *d_shared_rows = nullptr;
    SharedMerge *d_shared_merges = nullptr;  // null: the decode kernel merges
    int64_t total_q = 0;
    const int32_t *kv_indices = nullptr;  // borrowed device pointer
    void *workspace = nullptr;
    size_t workspace_bytes = 0;
    RequestInfo *d_reqs = nullptr;
    void *d_items = nullptr;
    int32_t *d_cta_items = nullptr;
    float *d_partial_o = nullptr;
    float *d_partial_lse = nullptr;
    int32_t *d_status = nullptr;
    int32_t *d_counters = nullptr;  // split-KV arrival counters (fused merge)
    cudaEvent_t ev_begin = nullptr;  // optional timing events around the main kernel
    cudaEvent_t ev_end = nullptr;
};

namespace {

struct HostRequest {
    int64_t qo_begin, qo_len, kv_len, kv_page_begin, q_start;
};

int validate(const pkv_plan_desc *d, std::vector<HostRequest> &reqs)
{
    if (!d)
        return fail(PKV_ERR_INVALID_ARG, "desc is NULL");
    if (d->kind != PKV_PREFILL && d->kind != PKV_DECODE && d->kind != PKV_PREFILL_RAGGED)
        return fail(PKV_ERR_INVALID_ARG, "kind %d is not a pkv_kind", d->kind);
    const bool ragged = d->kind == PKV_PREFILL_RAGGED;
    if (d->batch_size < 0)
        return fail(PKV_ERR_INVALID_ARG, "batch_size %d < 0", d->batch_size);
    const int B = d->batch_size;
    if (!d->kv_indptr || (!ragged && !d->kv_last_page_len))
        return fail(PKV_ERR_INVALID_ARG, "kv_indptr%s required", ragged ? " is" : " and kv_last_page_len are");
    if (d->kind != PKV_DECODE && !d->qo_indptr)
        return fail(PKV_ERR_INVALID_ARG, "prefill plans need qo_indptr");
    if (d->num_qo_heads <= 0 || d->num_kv_heads <= 0)
        return fail(PKV_ERR_INVALID_ARG, "head counts must be positive (%d, %d)", d->num_qo_heads,
                    d->num_kv_heads);
    if (d->num_qo_heads % d->num_kv_heads != 0)
        return fail(PKV_ERR_UNSUPPORTED, "num_qo_heads %d is not a multiple of num_kv_heads %d",
                    d->num_qo_heads, d->num_kv_heads);
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
        return fail(PKV_ERR_UNSUPPORTED, "head_dim %d not in {64, 128, 256}", d->head_dim);
    if (!ragged && d->page_size <= 0)
        return fail(PKV_ERR_INVALID_ARG, "page_size %d <= 0", d->page_size);
    if (d->num_pages < 0)
        return fail(PKV_ERR_INVALID_ARG, "num_pages %d < 0", d->num_pages);
    if (d->dtype != PKV_BF16)
        return fail(PKV_ERR_UNSUPPORTED, "dtype %d: only PKV_BF16 q/out are supported", d->dtype);
    if (d->kv_dtype != PKV_BF16 && d->kv_dtype != PKV_FP8_E4M3 && d->kv_dtype != PKV_FP8_E5M2 &&
        d->kv_dtype != PKV_FP4_E2M1)
        return fail(PKV_ERR_INVALID_ARG,
                    "kv_dtype %d is not PKV_BF16, PKV_FP8_E4M3, PKV_FP8_E5M2 or PKV_FP4_E2M1", d->kv_dtype);
    if (d->kv_dtype == PKV_FP4_E2M1 && d->kind != PKV_DECODE)
        return fail(PKV_ERR_UNSUPPORTED,
                    "4-bit caches are for decode plans; prefill reads them through pkv_gather_kv and a ragged plan");
    if (d->kv_dtype == PKV_FP4_E2M1 && (int64_t)d->num_pages * d->page_size >= (1LL << 32))
        return fail(PKV_ERR_UNSUPPORTED, "num_pages %d x page_size %d: 4-bit caches of 2^32 rows or more", d->num_pages,
                    d->page_size);
    if (d->kv_dtype != PKV_BF16 && d->kind == PKV_PREFILL_RAGGED)
        return fail(PKV_ERR_UNSUPPORTED, "8-bit K/V are supported in paged caches only");
    if (!(d->sm_scale == d->sm_scale) || std::isinf(d->sm_scale))
        return fail(PKV_ERR_INVALID_ARG, "sm_scale is not finite");
    if (!(d->sm_scale > 0.f))
        return fail(PKV_ERR_UNSUPPORTED, "sm_scale must be positive");
    for (float x : {d->logits_soft_cap, d->k_scale, d->v_scale})
        if (!(x == x) || std::isinf(x))
            return fail(PKV_ERR_INVALID_ARG, "logits_soft_cap, k_scale and v_scale must be finite");
    if (d->kind != PKV_DECODE &&
        d->num_qo_heads / d->num_kv_heads > kPrefillRows)
        return fail(PKV_ERR_UNSUPPORTED, "query-head group %d exceeds %d",
                    d->num_qo_heads / d->num_kv_heads, kPrefillRows);
    if (d->kv_indptr[0] != 0)
        return fail(PKV_ERR_INVALID_ARG, "kv_indptr[0] = %d, expected 0", d->kv_indptr[0]);
    if (d->kind != PKV_DECODE && d->qo_indptr[0] != 0)
        return fail(PKV_ERR_INVALID_ARG, "qo_indptr[0] = %d, expected 0", d->qo_indptr[0]);
    if (!ragged && B > 0 && d->kv_indptr[B] > 0 && !d->kv_indices)
        return fail(PKV_ERR_INVALID_ARG, "kv_indices is NULL but the batch holds pages");
    reqs.resize(B);
    for (int b = 0; b < B; ++b) {
        int64_t np = (int64_t)d->kv_indptr[b + 1] - d->kv_indptr[b];
        if (np < 0)
            return fail(PKV_ERR_INVALID_ARG, "kv_indptr decreases at request %d", b);
        int64_t kv_len = np;  // ragged: kv_indptr counts tokens
        if (!ragged) {
            int64_t last = d->kv_last_page_len[b];
            if (np > 0 && (last < 1 || last > d->page_size))
                return fail(PKV_ERR_INVALID_ARG, "kv_last_page_len[%d] = %lld outside [1, %d]", b,
                            (long long)last, d->page_size);
            kv_len = np > 0 ? (np - 1) * d->page_size + last : 0;
        }
        if (kv_len > INT32_MAX / 2)
            return fail(PKV_ERR_UNSUPPORTED, "request %d holds %lld tokens", b, (long long)kv_len);
        int64_t qo_begin, qo_len;
        if (d->kind != PKV_DECODE) {
            qo_begin = d->qo_indptr[b];
            qo_len = (int64_t)d->qo_indptr[b + 1] - d->qo_indptr[b];
            if (qo_len < 0)
                return fail(PKV_ERR_INVALID_ARG, "qo_indptr decreases at request %d", b);
        } else {
            qo_begin = b;
            qo_len = 1;
        }
        int64_t q_start = d->q_start ? (int64_t)d->q_start[b] : kv_len - qo_len;
        if (std::llabs(q_start) > INT32_MAX / 2)
            return fail(PKV_ERR_INVALID_ARG, "q_start[%d] out of range", b);
        reqs[b] = {qo_begin, qo_len, kv_len, (int64_t)d->kv_indptr[b], q_start};
    }
    return PKV_OK;
}

// Visible key interval [lo, hi] (inclusive; empty when hi < lo) of the query
// positions [p_min, p_max] taken together, for a request of kv_len keys.
void visible_interval(int64_t p_min, int64_t p_max, int64_t kv_len, int window_left, bool causal,
                      int64_t &lo, int64_t &hi)
{
    lo = window_left >= 0 ? std::max<int64_t>(0, p_min - window_left) : 0;
    hi = causal ? std::min<int64_t>(kv_len - 1, p_max) : kv_len - 1;
}

// Clip `sinks` to the keys before the visible interval [lo, hi] of the positions up to
// p_max. When they touch it, or it is empty, one range is left: [lo, hi] then holds it
// and 0 is returned.
int64_t separate_sinks(int64_t sinks, int64_t p_max, int64_t kv_len, bool causal, int64_t &lo, int64_t &hi)
{
    int64_t s = std::min(sinks, kv_len);
    if (causal)
        s = std::min(s, p_max + 1);
    if (s <= 0)
        return 0;
    if (hi < lo) {  // the sinks alone
        lo = 0;
        hi = s - 1;
        return 0;
    }
    if (s >= lo) {
        lo = 0;
        return 0;
    }
    return s;
}

// A split of a decode request: keys [0, sink_end) and [j0, j1).
struct DecodePiece {
    int64_t sink_end, j0, j1;
};

// Pieces of `per` visible keys each of the keys [0, s) and [lo, lo + n): the key ranges of
// one request's splits. A piece across the gap keeps both ranges if it starts at key 0
// and is cut there otherwise.
std::vector<DecodePiece> cut_pieces(int64_t s, int64_t lo, int64_t n, int64_t per)
{
    std::vector<DecodePiece> out;
    for (int64_t v0 = 0; v0 < s + n; v0 += per) {
        const int64_t v1 = std::min(s + n, v0 + per);
        if (v1 <= s) {
            out.push_back({0, v0, v1});
        } else if (v0 >= s) {
            out.push_back({0, lo + v0 - s, lo + v1 - s});
        } else if (v0 == 0) {
            out.push_back({s, lo, lo + v1 - s});
        } else {
            out.push_back({0, v0, s});
            out.push_back({0, lo, lo + v1 - s});
        }
    }
    return out;
}

// Greedy longest-first assignment of item costs to `slots` equal workers; returns
// the finishing time of the busiest worker.
double simulate_makespan(std::vector<double> costs, int slots)
{
    std::sort(costs.begin(), costs.end(), std::greater<double>());
    std::priority_queue<double, std::vector<double>, std::greater<double>> load;
    for (int i = 0; i < slots; ++i)
        load.push(0.0);
    for (double c : costs) {
        double t = load.top();
        load.pop();
        load.push(t + c);
    }
    double mx = 0;
    while (!load.empty()) {
        mx = std::max(mx, load.top());
        load.pop();
    }
    return mx;
}

int device_sm_count(int device)
{
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n <= 0)
        n = 148;
    return n;
}

// Decode: pick the KV tokens per split. A pure function of the plan inputs and the
// SM count: every candidate split size (no split first, then from 256 tokens up
// in steps of 1.25x) is scored by a simulated longest-first makespan of its CTAs
// over the SM slots (each CTA costing its tokens plus a fixed start-up cost, plus
// the partial-state traffic when split) plus a fixed cost for the merge pass
// when any request splits; a candidate must beat the best so far by 2% to win,
// which keeps splits rare unless they clearly pay (measured on GB300: a second
// pass and many short CTAs cost more than the tail they remove on 64-request
// batches).
int64_t choose_decode_chunk(const std::vector<int64_t> &lens, int head_blocks, int sms,
                            int ctas_per_sm)
{
    int64_t max_len = 0;
    for (int64_t l : lens)
        max_len = std::max(max_len, l);
    if (max_len <= 256)
        return std::max<int64_t>(max_len, 1);
    const int slots = sms * ctas_per_sm;
    const double kCtaOverhead = 96.0;   // token-row equivalents per CTA
    const double kPartialCost = 32.0;   // token-row equivalents per partial (write + merge read)
    const double kMergeFixed = 512.0;   // the merge pass (launch and drain), per slot
    std::vector<int64_t> cands{max_len};
    for (int64_t c = 256; c < max_len; c = round_up((int64_t)(c * 1.25), 64))
        cands.push_back(c);
    int64_t best_chunk = max_len;
    double best = 0;
    bool have = false;
    for (int64_t chunk : cands) {
        std::vector<double> costs;
        costs.reserve(lens.size() * 8);
        double merge = 0;
        bool any_split = false;
        for (int64_t l : lens) {
            if (l <= 0) {
                costs.push_back(kCtaOverhead);
                continue;
            }
            int64_t n = (l + chunk - 1) / chunk;
            int64_t per = round_up((l + n - 1) / n, 16);
            for (int64_t s = 0; s < n; ++s) {
                int64_t t = std::min(per, l - s * per);
                if (t <= 0)
                    break;
                for (int h = 0; h < head_blocks; ++h)
                    costs.push_back((double)t + kCtaOverhead + (n > 1 ? kPartialCost : 0.0));
            }
            if (n > 1) {
                merge += (double)n * head_blocks * kPartialCost / slots;
                any_split = true;
            }
        }
        double score = simulate_makespan(costs, slots) + merge + (any_split ? kMergeFixed : 0.0);
        if (!have || score < best * 0.98) {
            best = score;
            best_chunk = chunk;
            have = true;
        }
    }
    return best_chunk;
}

// Keys of each of n splits of `len`, a multiple of `align` (the last may have fewer).
int64_t split_length(int64_t len, int64_t n, int align) { return round_up((len + n - 1) / n, align); }

// 4-bit decode: KV heads to a CTA and KV tokens per split, by an estimate of the time in us: CTAs
// start longest first in 3 slots an SM, each has `keys` and a start-up to do, and what all of
// them do in a microsecond depends on how many there are. Measured at head_dim 128, in tokens of a
// CTA of 4 heads an SM and us: 20 with a CTA on every other SM, 33 with one on each, 43, 49.5 and
// 64 with 1.5, 2 and 3; CTAs of 2 heads and 1 do 0.95 and 0.88 of that in heads x tokens. A start-up
// is worth 80 of these tokens; a merge costs 1.5 us and 0.06 for each state and head. Over the
// batches that it was made from (1 to 64 requests of 300 to 4096 keys, 256 of 4224) the choice takes
// 7% longer in the mean than the best of 14 split sizes, the worst 20%.
struct Fp4Choice {
    int heads;
    int64_t chunk;
};

double fp4_decode_time(const std::vector<int64_t> &lens, int copies, int heads, int64_t chunk, int head_dim, int n_sm)
{
    static const double kAt[] = {0.0, 0.5, 1.0, 1.5, 2.0, 3.0}, kRate[] = {0.0, 20.0, 33.0, 43.0, 49.5, 64.0};
    const double per_head = heads == 4 ? 1.0 : heads == 2 ? 0.95 : 0.88;
    const double unit = heads / 4.0 * head_dim / 128.0 / per_head;  // a key, in tokens of 4 heads of 128
    std::vector<std::pair<double, int>> items;                     // work, how many CTAs of it
    int64_t most = 1;
    for (int64_t len : lens) {
        int64_t n = len > 0 ? (len + chunk - 1) / chunk : 1;
        const int64_t per = len > 0 ? split_length(len, n, fp4_decode_tile(heads)) : 1;
        n = std::max<int64_t>(1, (len + per - 1) / per);
        most = std::max(most, n);
        if (n > 1)
            items.push_back({per * unit + 80.0, (int)((n - 1) * copies)});
        items.push_back({(len - (n - 1) * per) * unit + 80.0, copies});
    }
    std::sort(items.begin(), items.end(), std::greater<>());
    // All CTAs that run advance alike: `done` is what each has got through so far, a CTA that starts
    // at `done` ends at done + work.
    std::priority_queue<std::pair<double, int>, std::vector<std::pair<double, int>>, std::greater<>> running;
    double done = 0, us = 0;
    int64_t active = 0;
    for (size_t i = 0; i < items.size() || active > 0;) {
        while (i < items.size() && active < 3LL * n_sm) {
            const int n = (int)std::min<int64_t>(items[i].second, 3LL * n_sm - active);
            running.push({done + items[i].first, n});
            active += n;
            if ((items[i].second -= n) == 0)
                ++i;
        }
        const auto [end, n] = running.top();
        running.pop();
        const double at = (double)active / n_sm;
        int k = 1;
        while (k < 5 && at > kAt[k])
            ++k;
        const double rate = kRate[k - 1] + (kRate[k] - kRate[k - 1]) * (at - kAt[k - 1]) / (kAt[k] - kAt[k - 1]);
        us += (end - done) * at / rate;
        done = end;
        active -= n;
    }
    return us + (most > 1 ? 1.5 + 0.06 * heads * (double)most : 0.0);
}

// lens: the keys that each request sees; only_heads, only_chunk > 0: given.
Fp4Choice choose_fp4_decode(const std::vector<int64_t> &lens, int num_kv_heads, int head_blocks, int head_dim, int n_sm,
                            int only_heads, int64_t only_chunk)
{
    int64_t max_len = 1;
    for (int64_t l : lens)
        max_len = std::max(max_len, l);
    Fp4Choice best{1, max_len};
    double best_us = -1;
    for (int heads : {4, 2, 1}) {
        if (only_heads > 0 ? heads != only_heads : !fp4_decode_heads(heads, head_dim, num_kv_heads))
            continue;
        const int copies = num_kv_heads / heads * head_blocks;
        for (int64_t chunk = max_len; chunk > 0; chunk = chunk <= 128 ? 0 : std::max<int64_t>(128, (int64_t)(chunk / 1.2))) {
            if (only_chunk > 0)
                chunk = only_chunk;
            int64_t n = 0;
            for (int64_t l : lens)
                n += copies * std::max<int64_t>(1, (l + chunk - 1) / chunk);
            if (best_us >= 0 && only_chunk <= 0 && chunk < max_len && n > 16LL * n_sm)
                break;  // many short CTAs: their start-ups outweigh the balance
            const double us = fp4_decode_time(lens, copies, heads, chunk, head_dim, n_sm);
            if (best_us < 0 || us < best_us * 0.98) {
                best_us = us;
                best = {heads, chunk};
            }
            if (only_chunk > 0)
                break;
        }
    }
    return best;
}

}  // namespace

namespace {

// The work schedule of a batch, built on the host from the host arrays alone.
struct Schedule {
    std::vector<RequestInfo> reqs;
    std::vector<PrefillItem> p_items;
    std::vector<DecodeItem> d_items;
    std::vector<int32_t> cta_items;  // prefill: list offsets (lists + 1 entries)
    std::vector<SharedItem> s_items;   // shared prefixes: items of the prefix kernel, CTA after CTA
    std::vector<int32_t> s_cta_items;  // their list offsets
    std::vector<SharedRow> s_rows;
    std::vector<SharedMerge> s_merges;  // empty: the decode kernel merges
    int num_partials = 0;
    int num_counters = 0;
    int mask_mode = kMaskNone;
    int decode_tile = 64;
    int64_t total_q = 0;
};

// Largest num_sinks: packed rows and the keys they stand for then stay below 2^31.
constexpr int kMaxSinks = 1 << 24;

// Splits per request that a capturable decode plan's workspace holds.
constexpr int kCapturableMaxSplits = 4;

// capturable: one prefill list per SM and at most kCapturableMaxSplits decode splits
// per request; fixed_tile > 0: the decode tile to use (a captured launch's variant).
// sinks: keys [0, sinks) stay visible under the window (0: none).
void build_schedule(const pkv_plan_desc &d, const std::vector<HostRequest> &reqs, int device, bool capturable,
                    int fixed_tile, int sinks, Schedule &sc)
{
    const int B = d.batch_size;
    const int group = d.num_qo_heads / d.num_kv_heads;
    const bool causal = d.causal != 0;
    const int W = d.window_left < 0 ? -1 : d.window_left;
    std::vector<RequestInfo> &h_reqs = sc.reqs;
    h_reqs.assign(B, RequestInfo{});
    int64_t total_q = 0;
    for (int b = 0; b < B; ++b) {
        const HostRequest &r = reqs[b];
        h_reqs[b] = {(int32_t)r.qo_begin, (int32_t)r.qo_len, (int32_t)r.kv_len,
                     (int32_t)r.kv_page_begin, (int32_t)r.q_start, 0, 0, 0};
        total_q = std::max<int64_t>(total_q, r.qo_begin + r.qo_len);
    }

    std::vector<PrefillItem> &p_items = sc.p_items;
    std::vector<DecodeItem> &d_items = sc.d_items;
    std::vector<int32_t> &cta_items = sc.cta_items;  // prefill: per-list item offsets
    int decode_tile = 64;
    int num_partials = 0;
    int num_counters = 0;
    int mask_mode = causal ? (W >= 0 ? kMaskCausalWindow : kMaskCausal)
                           : (W >= 0 ? kMaskWindow : kMaskNone);
    if (sinks > 0)
        mask_mode = causal ? kMaskCausalWindowSinks : kMaskWindowSinks;

    if (d.kind != PKV_DECODE) {
        const int T = prefill_kv_tile(d.head_dim);
        const int tq = prefill_tokens_per_cta(d.head_dim, group);
        // Ragged K/V: a TMA box may start at any row. Pages: at a page (TMA page
        // boxes) or anywhere (cp.async gathers).
        // 8-bit caches are gathered row by row.
        const int64_t kv_align = d.kind == PKV_PREFILL_RAGGED || d.kv_dtype != PKV_BF16 ? 1
                                 : prefill_pp_tma_page_size(d.page_size, d.head_dim)    ? std::min(d.page_size, T)
                                                                                        : 1;
        // Rows the window's tiles may follow the sinks at: a ragged box is a whole tile.
        const int64_t join_align = d.kind == PKV_PREFILL_RAGGED ? T : kv_align;
        for (int b = 0; b < B; ++b) {
            const HostRequest &r = reqs[b];
            for (int64_t t0 = 0; t0 < r.qo_len; t0 += tq) {
                int64_t nt = std::min<int64_t>(tq, r.qo_len - t0);
                int64_t lo, hi;
                const int64_t p_max = r.q_start + t0 + nt - 1;
                visible_interval(r.q_start + t0, p_max, r.kv_len, W, causal, lo, hi);
                const bool no_window = hi < lo;
                const int64_t s = sinks > 0 ? separate_sinks(sinks, p_max, r.kv_len, causal, lo, hi) : 0;
                // The item's KV tiles start at its first visible key, rounded down
                // only as far as the loader needs (a page for TMA page boxes), not
                // to a multiple of the tile: the window then spans the fewest tiles.
                // Sinks come before it in packed rows, the window's following at `join`
                // (sinks alone: no row from there on is a key of the request).
                int32_t start = 0, ntl = 0, join = 0;
                if (hi >= lo && no_window) {
                    join = (int32_t)round_up(hi + 1, join_align);
                    start = INT32_MAX / 2 + 1;
                    ntl = (int32_t)(hi / T + 1);
                } else if (hi >= lo) {
                    const int64_t base = lo / kv_align * kv_align;
                    if (round_up(s, join_align) < base) {
                        join = (int32_t)round_up(s, join_align);
                        start = (int32_t)(base - join);
                    }
                    ntl = (int32_t)((hi - start) / T + 1);
                }
                // Start tile: the query block's index times the golden ratio,
                // modulo the tile count, so that neighbouring blocks (which run at
                // the same time over nearly the same KV tiles) start far apart.
                const double frac = std::fmod((double)(t0 / tq) * 0.6180339887498949, 1.0);
                const int32_t rot = ntl > 1 ? std::min<int32_t>(ntl - 1, (int32_t)(frac * ntl)) : 0;
                for (int hk = 0; hk < d.num_kv_heads; ++hk)
                    p_items.push_back({b, hk, (int32_t)t0, (int32_t)nt, start, ntl, rot, join});
            }
        }
        // Persistent CTAs, one per SM: longest-processing-time-first assignment of
        // the items to the least loaded CTA. Cost of an item in KV-tile steps: a
        // single query tile runs its softmax-bound chain alone (about 0.8 of the
        // two-tile ping-pong step, as measured through the schedule it yields),
        // plus a fixed cost per item (pipeline fill and epilogue).
        const int tq_tile = std::max(1, kPrefillRows / group);
        auto cost = [&](const PrefillItem &it) {
            const int nq = (d.head_dim <= 128 && it.ntok > tq_tile) ? 2 : 1;
            return it.kv_tiles * (nq == 2 ? 1.0 : 0.8) + 1.5;
        };
        std::stable_sort(p_items.begin(), p_items.end(),
                         [&](const PrefillItem &a, const PrefillItem &b) { return cost(a) > cost(b); });
        const int n_sm = device_sm_count(device);
        // A capturable plan keeps one list per SM (some may be empty): the launch's
        // grid is fixed when it is captured.
        const int G = capturable ? n_sm : (int)std::min<size_t>(p_items.size(), (size_t)n_sm);
        std::vector<std::vector<PrefillItem>> per_cta(G);
        std::priority_queue<std::pair<double, int>, std::vector<std::pair<double, int>>,
                            std::greater<std::pair<double, int>>>
            heap;
        for (int c = 0; c < G; ++c)
            heap.push({0.0, c});
        for (const PrefillItem &it : p_items) {
            auto [load, c] = heap.top();
            heap.pop();
            per_cta[c].push_back(it);
            heap.push({load + cost(it), c});
        }
        p_items.clear();
        cta_items.assign(1, 0);
        for (int c = 0; c < G; ++c) {
            p_items.insert(p_items.end(), per_cta[c].begin(), per_cta[c].end());
            cta_items.push_back((int32_t)p_items.size());
        }
    } else {
        const int rows = decode_rows(d.kv_dtype);
        const int head_blocks = (group + rows - 1) / rows;
        std::vector<int64_t> lens(B), los(B), sink_lens(B);
        for (int b = 0; b < B; ++b) {
            int64_t lo, hi;
            const HostRequest &r = reqs[b];
            visible_interval(r.q_start, r.q_start, r.kv_len, W, causal, lo, hi);
            sink_lens[b] = sinks > 0 ? separate_sinks(sinks, r.q_start, r.kv_len, causal, lo, hi) : 0;
            los[b] = lo;
            lens[b] = sink_lens[b] + std::max<int64_t>(0, hi - lo + 1);
        }
        int64_t chunk;
        int heads = 1;  // KV heads of a CTA
        if (d.kv_dtype == PKV_FP4_E2M1) {
            const Fp4Choice c = choose_fp4_decode(lens, d.num_kv_heads, head_blocks, d.head_dim, device_sm_count(device),
                                                  fixed_tile, d.disable_split_kv ? INT32_MAX : d.fixed_split_size);
            chunk = c.chunk;
            heads = c.heads;
        } else if (d.disable_split_kv) {
            chunk = INT32_MAX;
        } else if (d.fixed_split_size > 0) {
            chunk = d.fixed_split_size;
        } else {
            const int ctas_per_sm = d.head_dim <= 128 ? 2 : 1;
            chunk = choose_decode_chunk(lens, head_blocks * d.num_kv_heads,
                                        device_sm_count(device), ctas_per_sm);
        }
        // (4-bit: whole stages)
        const int split_align = d.kv_dtype == PKV_FP4_E2M1 ? fp4_decode_tile(heads) : 16;
        for (int b = 0; b < B; ++b) {
            int64_t L = lens[b];
            int64_t n = L > 0 ? (L + chunk - 1) / chunk : 1;
            int64_t per = L > 0 ? (d.fixed_split_size > 0 && !d.disable_split_kv
                                       ? chunk
                                       : split_length(L, n, split_align))
                                : 0;
            const int64_t sl = sink_lens[b];
            std::vector<DecodePiece> pieces{{0, los[b], los[b]}};
            if (L > 0)
                pieces = cut_pieces(sl, los[b], L - sl, per);
            // the workspace of a capturable plan holds this many splits per request (a
            // piece cut at the end of the sinks is one more)
            for (int k = kCapturableMaxSplits; capturable && (int)pieces.size() > kCapturableMaxSplits; --k)
                pieces = cut_pieces(sl, los[b], L - sl, split_length(L, k, split_align));
            n = (int64_t)pieces.size();
            int32_t pbase = -1, cbase = -1;
            if (n > 1) {
                pbase = num_partials;
                num_partials += (int32_t)n;
                cbase = num_counters;  // one arrival counter per (KV head, head block)
                num_counters += d.num_kv_heads * head_blocks;
            }
            for (int64_t s = 0; s < n; ++s) {
                const DecodePiece &pc = pieces[s];
                for (int hk = 0; hk < d.num_kv_heads; hk += heads)
                    for (int h0 = 0; h0 < group; h0 += rows)
                        d_items.push_back({b, hk, hk * group + h0, std::min(rows, group - h0),
                                           (int32_t)pc.j0, (int32_t)pc.j1, n > 1 ? (int32_t)(pbase + s) : -1,
                                           pbase, (int32_t)n,
                                           n > 1 ? cbase + hk * head_blocks + h0 / rows : -1,
                                           h_reqs[b].qo_begin, h_reqs[b].kv_len, h_reqs[b].kv_page_begin,
                                           (int32_t)pc.sink_end, 0u});
            }
        }
        auto keys = [](const DecodeItem &it) { return it.sink_end + it.j1 - it.j0; };
        std::stable_sort(d_items.begin(), d_items.end(),
                         [&](const DecodeItem &a, const DecodeItem &b) { return keys(a) > keys(b); });
        const auto tile_for = sinks > 0 ? decode_sinks_tile_for : decode_tile_for;
        decode_tile = d.kv_dtype == PKV_FP4_E2M1 ? heads
                      : fixed_tile > 0           ? fixed_tile
                                     : tile_for(d.head_dim, d_items.empty() ? 0 : keys(d_items.front()),
                                                (int64_t)d_items.size(), device_sm_count(device));
    }
    sc.num_partials = num_partials;
    sc.num_counters = num_counters;
    sc.mask_mode = mask_mode;
    sc.decode_tile = decode_tile;
    sc.total_q = total_q;

}

// A group of requests (rows) b0 .. b1 - 1 whose first `keys` keys are the same pages.
struct Group {
    int b0, b1;
    int64_t keys;
};

// The groups of a plan of shared prefixes, checked. A prefix ends at the shortest of its group's
// requests.
int validate_groups(const pkv_plan_desc &d, const std::vector<HostRequest> &reqs, const pkv_plan_groups &gr,
                    std::vector<Group> &groups)
{
    if (d.kind != PKV_DECODE)
        return fail(PKV_ERR_UNSUPPORTED, "shared prefixes are for decode plans");
    if (gr.num_groups < 0 || (gr.num_groups > 0 && (!gr.group_indptr || !gr.shared_pages)))
        return fail(PKV_ERR_INVALID_ARG, "num_groups %d, or no group_indptr or shared_pages", gr.num_groups);
    if (gr.num_groups > 0 && (gr.group_indptr[0] != 0 || gr.group_indptr[gr.num_groups] != d.batch_size))
        return fail(PKV_ERR_INVALID_ARG, "group_indptr must go from 0 to the batch's %d requests", d.batch_size);
    for (int g = 0; g < gr.num_groups; ++g)
        if (gr.group_indptr[g + 1] < gr.group_indptr[g])
            return fail(PKV_ERR_INVALID_ARG, "group_indptr decreases at group %d", g);
    for (int g = 0; g < gr.num_groups; ++g) {
        const int b0 = gr.group_indptr[g], b1 = gr.group_indptr[g + 1];
        if (gr.shared_pages[g] < 0)
            return fail(PKV_ERR_INVALID_ARG, "shared_pages[%d] = %d < 0", g, gr.shared_pages[g]);
        int64_t keys = (int64_t)gr.shared_pages[g] * d.page_size;
        for (int b = b0; b < b1; ++b) {
            if (gr.shared_pages[g] > d.kv_indptr[b + 1] - d.kv_indptr[b])
                return fail(PKV_ERR_INVALID_ARG, "shared_pages[%d] = %d, but request %d holds %d pages", g,
                            gr.shared_pages[g], b, d.kv_indptr[b + 1] - d.kv_indptr[b]);
            keys = std::min(keys, reqs[b].kv_len);
        }
        if (b1 > b0)
            groups.push_back({b0, b1, keys});
    }
    return PKV_OK;
}

// Fewest prefix keys that a group's requests see together for which the prefix is computed apart: a
// floor for what is a few tiles at most, and no comparison with the ordinary plan, which is faster for
// short prefixes and for few requests over narrow caches. Measured, ordinary / shared in us, 8 KV
// heads of 128, 32 query heads, 100 keys of each request's own:
//                                 80 keys      256          1024         4096
//     1 group of 4, bf16          6.1 / 12.2   7.1 / 8.8    10.2 / 9.1   14.4 / 10.9
//     1 group of 16, bf16         6.3 / 12.8   7.5 / 9.2    16.4 / 9.7   33.4 / 17.2
//     1 group of 4, E4M3          5.6 / 12.6   6.3 / 10.0   10.5 / 10.1  13.8 / 12.0
//     1 group of 4, 4 bits        4.9 / 12.8   6.0 / 10.6   8.4 / 10.7   11.8 / 12.5
//     8 groups of 2, bf16         6.3 / 12.5   7.5 / 9.1    18.6 / 17.8  34.5 / 32.1
//     8 groups of 8, bf16         9.2 / 16.4   14.7 / 18.7  38.6 / 23.4  114 / 38.5
//     8 groups of 2, 4 bits       4.9 / 12.7   6.1 / 10.9   11.2 / 15.8  22.9 / 40.2
//     8 groups of 8, 4 bits       7.6 / 14.0   11.3 / 11.7  24.1 / 20.8  69.9 / 40.3
// The caller says which groups are shared (pkv.h has the rule of thumb).
constexpr int64_t kMinSharedKeys = 64;
// Fewest tiles of an item list: below, fewer CTAs share the work.
constexpr int64_t kMinSharedTiles = 2;

// CTAs of the prefix kernel: the more, the sooner it ends, but the fewer SMs the decode kernel has
// beside it meanwhile. Both are estimated in us: a list of n tiles in k pieces takes
// 7 + 7 k + c n, with c = 0.96 for a tile of 64 KB (K and V) by TMA and 1.4 where rows are
// copied or widened; the decode kernel its bytes at 6.8 TB/s, plus the SMs' share that the
// prefix has. The prefix is to end in 0.85 of the whole time, as its states are merged last.
// Measured, with as many CTAs as there are SMs and the choice, in us: 128 requests behind 8192 keys,
// 8 KV heads of 128, bf16 87.6 / 72.0, in pages of 5 118 / 111, E4M3 80.2 / 74.9, 4 bits 62.2 / 61.1;
// 6 groups of up to 48 behind up to 6000, bf16 104.6 / 95.4, E4M3 96.6 / 92.6, 4 bits 78.0 / 78.4; 128
// behind 4096, 4 heads of 256, bf16 82.5 / 64.0, E4M3 73.3 / 64.4, 4 bits 54.4 / 44.7. The one 1.4
// stands for tiles of 1.2 us (rows copied), 1.6 (8 bits) and 1.8 (4 bits): with these in its
// place every one of 31 batches was within 1%. Nor does it matter that the 4-bit decode keeps to 0.75 of
// the 6.8 TB/s, and that states are not counted: one KV head with 16 requests behind 60000 keys,
// in 150 pieces, takes 31.1 us, an ordinary plan 59.0.
int64_t choose_prefix_ctas(const pkv_plan_desc &d, const std::vector<int64_t> &units, int64_t total, int64_t own_keys,
                           int n_sm)
{
    const int64_t most = std::min<int64_t>(std::min(n_sm, kMaxPrefixPieces - 1), total / kMinSharedTiles);
    if (most <= 1)
        return total > 0;
    const int T = prefill_kv_tile(d.head_dim);
    const bool tma = d.kv_dtype == PKV_BF16 && prefill_pp_tma_page_size(d.page_size, d.head_dim);
    const double tile_us = (tma ? 0.96 : 1.4) * T * d.head_dim / 16384;
    const double bits = d.kv_dtype == PKV_BF16 ? 16 : d.kv_dtype == PKV_FP4_E2M1 ? 4.5 : 8;
    const double own_us = (double)own_keys * d.num_kv_heads * d.head_dim * 2 * bits / 8 / 6.8e6;
    int64_t best = most;
    double best_us = DBL_MAX;
    for (int64_t n = most; n >= 1; n -= n > 16 ? 8 : 1) {
        double prefix_us = 0;
        int64_t cta = 0, at = 0, pieces = 0, begin = 0;
        for (const int64_t u : units)
            for (int64_t left = u; left > 0;) {
                const int64_t end = (cta + 1) * total / n, k = std::min(left, end - at);
                left -= k;
                at += k;
                pieces += k > 0;
                if (at == end) {
                    prefix_us = std::max(prefix_us, 7 + 7.0 * pieces + tile_us * (at - begin));
                    begin = at;
                    pieces = 0;
                    ++cta;
                }
            }
        const double us = std::max(prefix_us / 0.85, own_us + prefix_us * n / n_sm);
        if (us < best_us) {
            best_us = us;
            best = n;
        }
    }
    return best;
}

// The schedule of a decode batch with shared prefixes: the prefix kernel's items, and decode items
// for what each request sees behind its group's prefix. Partial slots of a request: its own
// pieces, then the prefix's.
void build_shared_schedule(const pkv_plan_desc &d, const std::vector<HostRequest> &reqs,
                           const std::vector<Group> &groups, int n_sm, int sinks, Schedule &sc)
{
    const int B = d.batch_size, H = d.num_kv_heads, group = d.num_qo_heads / d.num_kv_heads;
    const bool causal = d.causal != 0;
    const int W = d.window_left < 0 ? -1 : d.window_left;
    const int T = prefill_kv_tile(d.head_dim);
    const int tq = group <= kPrefillRows ? kPrefillRows / group : 1;  // requests of an item
    const int64_t align =
        d.kv_dtype == PKV_BF16 && prefill_pp_tma_page_size(d.page_size, d.head_dim) ? std::min(d.page_size, T) : 1;
    sc.total_q = B;
    sc.mask_mode = sinks > 0 ? (causal ? kMaskCausalWindowSinks : kMaskWindowSinks)
                   : W >= 0  ? (causal ? kMaskCausalWindow : kMaskWindow)
                             : (causal ? kMaskCausal : kMaskNone);
    struct Seen {
        int64_t lo, hi, sink;  // keys [lo, hi] and [0, sink)
    };
    std::vector<Seen> seen(B);
    std::vector<int64_t> prefix(B, 0);  // keys computed by the prefix kernel
    for (int b = 0; b < B; ++b) {
        const HostRequest &r = reqs[b];
        sc.reqs.push_back({(int32_t)r.qo_begin, (int32_t)r.qo_len, (int32_t)r.kv_len, (int32_t)r.kv_page_begin,
                           (int32_t)r.q_start, 0, 0, 0});
        Seen &s = seen[b];
        visible_interval(r.q_start, r.q_start, r.kv_len, W, causal, s.lo, s.hi);
        s.sink = sinks > 0 ? separate_sinks(sinks, r.q_start, r.kv_len, causal, s.lo, s.hi) : 0;
    }
    // Units: a run of tiles of one (group, KV head, block of requests).
    struct Unit {
        int group, kv_head, row0, ntok;
        int64_t key0, tiles, kv_end;
        bool first;  // of its (group, KV head, block)
    };
    std::vector<Unit> units;
    int64_t total = 0;
    for (size_t g = 0; g < groups.size(); ++g) {
        const Group &gr = groups[g];
        if (gr.b1 - gr.b0 < 2 || group > kPrefillRows)
            continue;
        int64_t lo = INT64_MAX, hi = -1, sink = 0;  // what any of the requests sees of the prefix
        for (int b = gr.b0; b < gr.b1; ++b) {
            const int64_t h = std::min(seen[b].hi, gr.keys - 1);
            if (seen[b].lo <= h) {
                lo = std::min(lo, seen[b].lo);
                hi = std::max(hi, h);
            }
            sink = std::max(sink, std::min(seen[b].sink, gr.keys));
        }
        const int64_t keys = (hi >= 0 ? hi - lo + 1 : 0) + sink;
        if (keys < kMinSharedKeys)
            continue;
        // the window's tiles, and the sinks' before them where no page joins them: pages that none of
        // the requests sees are not read
        struct Run {
            int64_t key0, tiles, kv_end;
        };
        std::vector<Run> runs;
        int64_t base = hi >= 0 ? lo / align * align : 0;
        const bool apart = hi >= 0 && sink > 0 && sink <= base;
        if (apart || hi < 0)
            runs.push_back({0, round_up(sink, T) / T, sink});
        else if (sink > 0)
            base = 0;
        if (hi >= 0) {
            const int64_t end = std::max(hi + 1, apart ? 0 : sink);
            runs.push_back({base, (end - base + T - 1) / T, end});
        }
        for (int b = gr.b0; b < gr.b1; ++b)
            prefix[b] = gr.keys;
        for (int hk = 0; hk < H; ++hk)
            for (int b = gr.b0; b < gr.b1; b += tq) {
                bool first = true;
                for (const Run &r : runs) {
                    units.push_back({(int)g, hk, b, std::min(tq, gr.b1 - b), r.key0, r.tiles, r.kv_end, first});
                    total += r.tiles;
                    first = false;
                }
            }
    }
    // What each request sees behind its prefix.
    const int rows = decode_rows(d.kv_dtype);
    const int head_blocks = (group + rows - 1) / rows;
    auto own = [&](int b) {  // key ranges, sinks beyond the prefix first
        std::vector<std::pair<int64_t, int64_t>> r;
        if (seen[b].sink > prefix[b])
            r.push_back({prefix[b], seen[b].sink});
        if (std::max(seen[b].lo, prefix[b]) <= seen[b].hi)
            r.push_back({std::max(seen[b].lo, prefix[b]), seen[b].hi + 1});
        return r;
    };
    std::vector<int64_t> lens(B, 0);
    for (int b = 0; b < B; ++b)
        for (const auto &r : own(b))
            lens[b] += r.second - r.first;
    // Cut the sequence of all tiles into one list a CTA, of equal lengths.
    // (a unit of two runs is cut into one piece more than it has lists)
    std::vector<int64_t> unit_tiles;
    for (const Unit &u : units)
        unit_tiles.push_back(u.tiles);
    const int64_t own_keys = std::accumulate(lens.begin(), lens.end(), int64_t(0));
    const int64_t n_cta = choose_prefix_ctas(d, unit_tiles, total, own_keys, n_sm);
    std::vector<int32_t> pieces((size_t)B * H, 0);  // prefix pieces of a request's KV head
    sc.s_cta_items.assign(1, 0);
    int64_t cta = 0, at = 0;  // `at`: tiles before this one
    int32_t piece = 0;
    for (const Unit &u : units) {
        if (u.first)
            piece = 0;
        for (int64_t t = 0; t < u.tiles;) {
            const int64_t end = (cta + 1) * total / n_cta;  // where this CTA's list ends
            const int64_t n = std::min(u.tiles - t, end - at);
            if (n > 0) {
                sc.s_items.push_back({u.row0, u.ntok, u.kv_head, (int32_t)reqs[groups[u.group].b0].kv_page_begin,
                                      (int32_t)(u.key0 + t * T), (int32_t)n, (int32_t)u.kv_end, piece++});
                t += n;
                at += n;
            }
            if (at == end) {
                sc.s_cta_items.push_back((int32_t)sc.s_items.size());
                ++cta;
            }
        }
        for (int b = u.row0; b < u.row0 + u.ntok; ++b)
            pieces[(size_t)b * H + u.kv_head] = piece;
    }
    int64_t chunk = d.disable_split_kv ? INT32_MAX : d.fixed_split_size;
    int heads = 1;
    if (d.kv_dtype == PKV_FP4_E2M1) {
        const Fp4Choice c = choose_fp4_decode(lens, H, head_blocks, d.head_dim, n_sm, 0, chunk);
        chunk = c.chunk;
        heads = c.heads;
    } else if (chunk <= 0) {
        chunk = choose_decode_chunk(lens, head_blocks * H, n_sm, d.head_dim <= 128 ? 2 : 1);
    }
    sc.s_rows.resize(B);
    std::vector<SharedMerge> merges((size_t)B * H, SharedMerge{0, 0});
    for (int b = 0; b < B; ++b) {
        std::vector<DecodePiece> own_pieces;
        for (const auto &r : own(b)) {
            const int64_t len = r.second - r.first, n = (len + chunk - 1) / chunk;
            const int64_t per = d.fixed_split_size > 0 && !d.disable_split_kv
                                    ? chunk
                                    : split_length(len, n, d.kv_dtype == PKV_FP4_E2M1 ? fp4_decode_tile(heads) : 16);
            for (int64_t k = r.first; k < r.second; k += per)
                own_pieces.push_back({0, k, std::min(r.second, k + per)});
        }
        if (own_pieces.empty())
            own_pieces.push_back({0, prefix[b], prefix[b]});
        const int n = (int)own_pieces.size();
        const int32_t most = *std::max_element(pieces.begin() + (size_t)b * H, pieces.begin() + (size_t)(b + 1) * H);
        const bool merge = n > 1 || most > 0;
        const int32_t pbase = merge ? sc.num_partials : -1, cbase = merge ? sc.num_counters : -1;
        if (merge) {
            sc.num_partials += n + most;
            sc.num_counters += H * head_blocks;
        }
        sc.s_rows[b] = {(int32_t)seen[b].lo, (int32_t)std::min(seen[b].hi, prefix[b] - 1),
                        (int32_t)std::min(seen[b].sink, prefix[b]), merge ? pbase + n : 0};
        if (merge)
            for (int hk = 0; hk < H; ++hk)
                merges[(size_t)b * H + hk] = {pbase, n + pieces[(size_t)b * H + hk]};
        for (int s = 0; s < n; ++s)
            for (int hk = 0; hk < H; hk += heads)
                for (int h0 = 0; h0 < group; h0 += rows) {
                    uint32_t prefix_pieces = 0;
                    for (int x = 0; x < heads; ++x)
                        prefix_pieces |= (uint32_t)pieces[(size_t)b * H + hk + x] << (8 * x);
                    sc.d_items.push_back({b, hk, hk * group + h0, std::min(rows, group - h0), (int32_t)own_pieces[s].j0,
                                          (int32_t)own_pieces[s].j1, merge ? pbase + s : -1, pbase, n,
                                          merge ? cbase + hk * head_blocks + h0 / rows : -1, sc.reqs[b].qo_begin,
                                          sc.reqs[b].kv_len, sc.reqs[b].kv_page_begin, 0, prefix_pieces});
                }
    }
    // CTAs that wait for the prefix keep others out where not all of them fit beside it: two to an SM
    // taken for every kernel, of which one (head_dim 256, bf16) to four fit. Measured, with 1, 2 and 4 in
    // its place: heads of 256, 24 requests behind 4096 keys 27.1 / 26.2 / 26.1 us, 64 37.5 / 37.5 / 39.6,
    // 128 64.0 / 64.0 / 84.5; 28 more batches of every type within 4% of each other.
    if ((int64_t)sc.d_items.size() > 2 * (n_sm - n_cta))
        sc.s_merges = std::move(merges);
    auto keys = [](const DecodeItem &it) { return it.j1 - it.j0; };
    std::stable_sort(sc.d_items.begin(), sc.d_items.end(),
                     [&](const DecodeItem &a, const DecodeItem &b) { return keys(a) > keys(b); });
    sc.decode_tile = d.kv_dtype == PKV_FP4_E2M1 ? heads : decode_tile_for(d.head_dim, sc.d_items.empty() ? 0 : keys(sc.d_items.front()),
                                     (int64_t)sc.d_items.size(), n_sm);
}

// Sizes of a plan's device workspace: the live schedule for an ordinary plan, the
// declared capacity for a capturable one.
struct Caps {
    int64_t batch = 0, total_q = 0, items = 0, lists = 0, partials = 0, counters = 0;
    int64_t shared_items = 0, shared_lists = 0, shared_rows = 0, shared_merges = 0;  // plans of shared prefixes
};

Caps caps_of(const pkv_plan_desc &d, const Schedule &sc)
{
    Caps c;
    c.batch = d.batch_size;
    c.total_q = sc.total_q;
    c.items = d.kind != PKV_DECODE ? (int64_t)sc.p_items.size() : (int64_t)sc.d_items.size();
    c.lists = sc.cta_items.empty() ? 0 : (int64_t)sc.cta_items.size() - 1;
    c.partials = sc.num_partials;
    c.counters = sc.num_counters;
    c.shared_items = (int64_t)sc.s_items.size();
    c.shared_lists = (int64_t)sc.s_cta_items.size();
    c.shared_rows = (int64_t)sc.s_rows.size();
    c.shared_merges = (int64_t)sc.s_merges.size();
    return c;
}

Caps caps_for_capacity(const pkv_plan_desc &d, const pkv_plan_caps &cap, int n_sm, int decode_tile)
{
    const int group = d.num_qo_heads / d.num_kv_heads;
    Caps c;
    c.batch = cap.max_batch;
    if (d.kind != PKV_DECODE) {
        const int64_t tq = prefill_tokens_per_cta(d.head_dim, group);
        c.total_q = cap.max_total_q;
        c.items = (int64_t)d.num_kv_heads * ((cap.max_total_q + tq - 1) / tq + cap.max_batch);
        c.lists = n_sm;
    } else {
        const int64_t head_blocks = (group + decode_rows(d.kv_dtype) - 1) / decode_rows(d.kv_dtype);
        const int heads = d.kv_dtype == PKV_FP4_E2M1 ? decode_tile : 1;
        c.total_q = cap.max_batch;
        c.items = (int64_t)cap.max_batch * (d.num_kv_heads / heads) * head_blocks * kCapturableMaxSplits;
        c.partials = (int64_t)cap.max_batch * kCapturableMaxSplits;
        c.counters = (int64_t)cap.max_batch * d.num_kv_heads * head_blocks;
    }
    return c;
}

// requests | items | list offsets | live item count | shared prefixes: items, list offsets, rows
// (uploaded) | partial o | partial lse | arrival counters | status.
struct Layout {
    size_t reqs, items, cta, live, s_items, s_cta, s_rows, s_merges, po, pl, cnt, status, bytes, upload;
};

Layout layout_for(const pkv_plan_desc &d, const Caps &c)
{
    const size_t item_bytes = d.kind != PKV_DECODE ? sizeof(PrefillItem) : sizeof(DecodeItem);
    size_t off = 0;
    auto carve = [&](size_t bytes) {
        size_t at = off;
        off = (size_t)round_up((int64_t)(off + bytes), 256);
        return at;
    };
    Layout l{};
    l.reqs = carve(sizeof(RequestInfo) * std::max<int64_t>(1, c.batch));
    l.items = carve(item_bytes * std::max<int64_t>(1, c.items));
    l.cta = carve(sizeof(int32_t) * (std::max<int64_t>(0, c.lists) + 1));
    l.live = carve(sizeof(int32_t) * 4);
    l.s_items = carve(sizeof(SharedItem) * (size_t)c.shared_items);
    l.s_cta = carve(sizeof(int32_t) * (size_t)c.shared_lists);
    l.s_rows = carve(sizeof(SharedRow) * (size_t)c.shared_rows);
    l.s_merges = carve(sizeof(SharedMerge) * (size_t)c.shared_merges);
    l.po = carve(sizeof(float) * (size_t)c.partials * d.num_qo_heads * d.head_dim);
    l.pl = carve(sizeof(float) * (size_t)c.partials * d.num_qo_heads);
    l.cnt = carve(sizeof(int32_t) * std::max<int64_t>(1, c.counters));
    l.status = carve(sizeof(int32_t) * 4);
    l.bytes = off;
    l.upload = l.po;
    return l;
}

// The uploaded part of the workspace image of a schedule.
void fill_image(const pkv_plan_desc &d, const Schedule &sc, const Layout &l, uint8_t *img)
{
    std::memset(img, 0, l.upload);
    std::memcpy(img + l.reqs, sc.reqs.data(), sizeof(RequestInfo) * sc.reqs.size());
    if (d.kind != PKV_DECODE)
        std::memcpy(img + l.items, sc.p_items.data(), sizeof(PrefillItem) * sc.p_items.size());
    else
        std::memcpy(img + l.items, sc.d_items.data(), sizeof(DecodeItem) * sc.d_items.size());
    std::memcpy(img + l.cta, sc.cta_items.data(), sizeof(int32_t) * sc.cta_items.size());
    const int32_t live = d.kind != PKV_DECODE ? (int32_t)sc.p_items.size() : (int32_t)sc.d_items.size();
    std::memcpy(img + l.live, &live, sizeof(live));
    if (!sc.s_items.empty()) {
        std::memcpy(img + l.s_items, sc.s_items.data(), sizeof(SharedItem) * sc.s_items.size());
        std::memcpy(img + l.s_cta, sc.s_cta_items.data(), sizeof(int32_t) * sc.s_cta_items.size());
        std::memcpy(img + l.s_rows, sc.s_rows.data(), sizeof(SharedRow) * sc.s_rows.size());
        std::memcpy(img + l.s_merges, sc.s_merges.data(), sizeof(SharedMerge) * sc.s_merges.size());
    }
}

// No exception of the host containers leaves a C entry: a batch too large for them is out
// of memory.
template <typename F>
int guarded(F &&body)
{
    try {
        return body();
    } catch (const std::exception &) {
        return fail(PKV_ERR_OOM, "host allocation of the schedule failed");
    }
}

}  // namespace

extern "C" {

const char *pkv_status_string(int status)
{
    switch (status) {
    case PKV_OK: return "PKV_OK";
    case PKV_ERR_INVALID_ARG: return "PKV_ERR_INVALID_ARG";
    case PKV_ERR_UNSUPPORTED: return "PKV_ERR_UNSUPPORTED";
    case PKV_ERR_CUDA: return "PKV_ERR_CUDA";
    case PKV_ERR_OOM: return "PKV_ERR_OOM";
    case PKV_ERR_DEVICE_BOUNDS: return "PKV_ERR_DEVICE_BOUNDS";
    case PKV_ERR_TIMEOUT: return "PKV_ERR_TIMEOUT";
    default: return "PKV_ERR_UNKNOWN";
    }
}

const char *pkv_last_error(void) { return g_last_error.c_str(); }

int pkv_abi_version(void) { return PKV_ABI_VERSION; }

namespace {

int create_plan(pkv_plan **out, const pkv_plan_desc *desc, const pkv_plan_caps *capacity, int32_t num_sinks,
                void *stream_, const pkv_plan_groups *shared = nullptr)
{
    g_last_error.clear();
    if (!out)
        return fail(PKV_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    std::vector<HostRequest> reqs;
    int st = validate(desc, reqs);
    if (st != PKV_OK)
        return st;
    const pkv_plan_desc &d = *desc;
    if (num_sinks < 0)
        return fail(PKV_ERR_INVALID_ARG, "num_sinks %d < 0", num_sinks);
    if (num_sinks > kMaxSinks)
        return fail(PKV_ERR_UNSUPPORTED, "num_sinks %d exceeds %d", num_sinks, kMaxSinks);
    // without a window nothing is hidden from the sinks' queries: a plain plan
    const int sinks = d.window_left < 0 ? 0 : num_sinks;
    const bool capturable = capacity != nullptr;
    if (capturable && d.kind == PKV_PREFILL_RAGGED)
        return fail(PKV_ERR_UNSUPPORTED, "ragged plans are not capturable (the K/V row count is baked into a launch)");
    if (capturable && (capacity->max_batch < d.batch_size || capacity->max_batch < 1 ||
                       (d.kind != PKV_DECODE && capacity->max_total_q < 1)))
        return fail(PKV_ERR_INVALID_ARG, "capacity: max_batch must be >= 1 and >= batch_size%s",
                    d.kind != PKV_DECODE ? ", max_total_q >= 1" : "");
    std::vector<Group> groups;
    if (shared && (st = validate_groups(d, reqs, *shared, groups)) != PKV_OK)
        return st;
    cudaStream_t stream = (cudaStream_t)stream_;
    int device = 0;
    cudaError_t ce = cudaGetDevice(&device);
    if (ce != cudaSuccess)
        return cuda_fail(ce, "cudaGetDevice");
    const int n_sm = device_sm_count(device);

    Schedule sc;
    if (shared) {
        build_shared_schedule(d, reqs, groups, n_sm, sinks, sc);
        if (sc.s_items.empty())  // nothing to share: the plain plan
            sc = Schedule{};
    }
    const bool with_prefix = !sc.s_items.empty();
    if (!with_prefix)
        build_schedule(d, reqs, device, capturable, 0, sinks, sc);
    const Caps caps = capturable ? caps_for_capacity(d, *capacity, n_sm, sc.decode_tile) : caps_of(d, sc);
    if (capturable && (sc.total_q > caps.total_q))
        return fail(PKV_ERR_UNSUPPORTED, "the batch has %lld query rows, the capacity %lld",
                    (long long)sc.total_q, (long long)caps.total_q);
    const Layout lay = layout_for(d, caps);

    std::vector<uint8_t> image(lay.upload, 0);
    fill_image(d, sc, lay, image.data());
    pkv_plan *plan = new (std::nothrow) pkv_plan();
    if (!plan)
        return fail(PKV_ERR_OOM, "host allocation of the plan failed");
    ce = cudaMalloc(&plan->workspace, lay.bytes);
    if (ce != cudaSuccess) {
        delete plan;
        return cuda_fail(ce, "cudaMalloc(plan workspace)");
    }
    uint8_t *base = (uint8_t *)plan->workspace;
    ce = cudaMemcpyAsync(base, image.data(), lay.upload, cudaMemcpyHostToDevice, stream);
    if (ce == cudaSuccess)
        ce = cudaMemsetAsync(base + lay.status, 0, sizeof(int32_t) * 4, stream);
    if (ce == cudaSuccess)  // arrival counters start at zero; each merge resets its own
        ce = cudaMemsetAsync(base + lay.cnt, 0, lay.status - lay.cnt, stream);
    if (ce == cudaSuccess)
        ce = cudaStreamSynchronize(stream);  // the host image is freed on return
    if (ce == cudaSuccess && capturable) {
        for (int k = 0; k < 2 && ce == cudaSuccess; ++k) {
            ce = cudaHostAlloc(&plan->staging[k], lay.upload, cudaHostAllocDefault);
            if (ce == cudaSuccess)
                ce = cudaEventCreateWithFlags(&plan->staging_done[k], cudaEventDisableTiming);
        }
    }
    if (ce != cudaSuccess) {
        for (int k = 0; k < 2; ++k) {
            if (plan->staging[k])
                cudaFreeHost(plan->staging[k]);
            if (plan->staging_done[k])
                cudaEventDestroy(plan->staging_done[k]);
        }
        cudaFree(plan->workspace);
        delete plan;
        return cuda_fail(ce, "uploading the plan");
    }
    plan->desc = d;
    plan->desc.qo_indptr = plan->desc.kv_indptr = plan->desc.kv_last_page_len = nullptr;
    plan->desc.q_start = nullptr;
    plan->desc.window_left = d.window_left < 0 ? -1 : d.window_left;
    plan->device = device;
    plan->n_sm = n_sm;
    plan->capturable = capturable;
    plan->mask_mode = sc.mask_mode;
    plan->sinks = sinks;
    plan->num_items = (int)(d.kind != PKV_DECODE ? sc.p_items.size() : sc.d_items.size());
    plan->num_partials = sc.num_partials;
    plan->num_ctas = sc.cta_items.empty() ? 0 : (int)sc.cta_items.size() - 1;
    plan->decode_tile = sc.decode_tile;
    plan->total_q = sc.total_q;
    plan->total_kv = d.batch_size > 0 ? d.kv_indptr[d.batch_size] : 0;
    plan->cap_items = caps.items;
    plan->cap_total_q = caps.total_q;
    plan->cap_batch = caps.batch;
    plan->upload_bytes = lay.upload;
    plan->kv_indices = d.kv_indices;
    plan->workspace_bytes = lay.bytes;
    plan->d_reqs = (RequestInfo *)(base + lay.reqs);
    plan->d_items = base + lay.items;
    plan->d_cta_items = (int32_t *)(base + lay.cta);
    plan->d_live = (int32_t *)(base + lay.live);
    plan->d_partial_o = (float *)(base + lay.po);
    plan->d_partial_lse = (float *)(base + lay.pl);
    plan->d_status = (int32_t *)(base + lay.status);
    plan->d_counters = (int32_t *)(base + lay.cnt);
    plan->shared = with_prefix;
    plan->num_shared_ctas = with_prefix ? (int)sc.s_cta_items.size() - 1 : 0;
    plan->d_shared_items = (SharedItem *)(base + lay.s_items);
    plan->d_shared_cta = (int32_t *)(base + lay.s_cta);
    plan->d_shared_rows = (SharedRow *)(base + lay.s_rows);
    plan->d_shared_merges = sc.s_merges.empty() ? nullptr : (SharedMerge *)(base + lay.s_merges);
    *out = plan;
    return PKV_OK;
}

}  // namespace

int pkv_plan_create(pkv_plan **out, const pkv_plan_desc *desc, void *stream)
{
    NvtxRange range("pkv_plan_create");
    return guarded([&] { return create_plan(out, desc, nullptr, 0, stream); });
}

int pkv_plan_create_sinks(pkv_plan **out, const pkv_plan_desc *desc, int32_t num_sinks, const pkv_plan_caps *caps,
                          void *stream)
{
    NvtxRange range("pkv_plan_create_sinks");
    return guarded([&] { return create_plan(out, desc, caps, num_sinks, stream); });
}

int pkv_plan_create_shared(pkv_plan **out, const pkv_plan_desc *desc, const pkv_plan_groups *groups,
                           int32_t num_sinks, void *stream)
{
    NvtxRange range("pkv_plan_create_shared");
    if (!groups) {
        g_last_error.clear();
        if (out)
            *out = nullptr;
        return fail(PKV_ERR_INVALID_ARG, "groups is NULL");
    }
    return guarded([&] { return create_plan(out, desc, nullptr, num_sinks, stream, groups); });
}

int pkv_plan_create_capturable(pkv_plan **out, const pkv_plan_desc *desc, const pkv_plan_caps *caps,
                               void *stream)
{
    NvtxRange range("pkv_plan_create_capturable");
    if (!caps) {
        g_last_error.clear();
        if (out)
            *out = nullptr;
        return fail(PKV_ERR_INVALID_ARG, "caps is NULL");
    }
    return guarded([&] { return create_plan(out, desc, caps, 0, stream); });
}

static int update_plan(pkv_plan *plan, const pkv_plan_desc *desc, void *stream_)
{
    if (!plan)
        return fail(PKV_ERR_INVALID_ARG, "plan is NULL");
    if (!plan->capturable)
        return fail(PKV_ERR_INVALID_ARG, "pkv_plan_update needs a plan from pkv_plan_create_capturable");
    std::vector<HostRequest> reqs;
    int st = validate(desc, reqs);
    if (st != PKV_OK)
        return st;
    const pkv_plan_desc &d = *desc, &o = plan->desc;
    const int W = d.window_left < 0 ? -1 : d.window_left;
    // What the captured launches bake in must not change.
    if (d.kind != o.kind || d.num_qo_heads != o.num_qo_heads || d.num_kv_heads != o.num_kv_heads ||
        d.head_dim != o.head_dim || d.page_size != o.page_size || W != o.window_left ||
        (d.causal != 0) != (o.causal != 0) || d.sm_scale != o.sm_scale || d.dtype != o.dtype ||
        d.logits_soft_cap != o.logits_soft_cap || d.k_scale != o.k_scale || d.v_scale != o.v_scale ||
        d.kv_dtype != o.kv_dtype || d.wait_limit_us != o.wait_limit_us || d.wait_probe != o.wait_probe ||
        d.num_pages != o.num_pages || d.kv_indices != o.kv_indices)
        return fail(PKV_ERR_INVALID_ARG,
                    "update must keep kind, heads, head_dim, page_size, window_left, causal, sm_scale, "
                    "dtype, kv_dtype, soft cap, scales, wait bound and probe, num_pages and the kv_indices "
                    "pointer of the plan");
    if (d.batch_size > plan->cap_batch)
        return fail(PKV_ERR_UNSUPPORTED, "batch %d exceeds the plan's capacity %lld", d.batch_size,
                    (long long)plan->cap_batch);
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess || cur != plan->device)
        return fail(PKV_ERR_INVALID_ARG, "plan was made on device %d, current device is %d", plan->device, cur);
    Schedule sc;
    build_schedule(d, reqs, plan->device, true, plan->decode_tile, plan->sinks, sc);
    const int64_t items = d.kind != PKV_DECODE ? (int64_t)sc.p_items.size() : (int64_t)sc.d_items.size();
    if (sc.total_q > plan->cap_total_q || items > plan->cap_items)
        return fail(PKV_ERR_UNSUPPORTED, "the batch needs %lld query rows and %lld work items, the capacity is %lld "
                    "and %lld", (long long)sc.total_q, (long long)items, (long long)plan->cap_total_q,
                    (long long)plan->cap_items);
    pkv_plan_caps cap{};
    cap.max_batch = (int32_t)plan->cap_batch;
    cap.max_total_q = plan->cap_total_q;
    const Layout lay = layout_for(plan->desc, caps_for_capacity(plan->desc, cap, plan->n_sm, plan->decode_tile));
    cudaStream_t stream = (cudaStream_t)stream_;
    // Two pinned staging images, each reused only once its previous upload is done
    // (an event wait that is normally already satisfied; nothing else waits).
    const int k = plan->staging_next;
    cudaError_t ce = cudaEventSynchronize(plan->staging_done[k]);
    if (ce != cudaSuccess)
        return cuda_fail(ce, "waiting for the staging image");
    fill_image(plan->desc, sc, lay, (uint8_t *)plan->staging[k]);
    ce = cudaMemcpyAsync(plan->workspace, plan->staging[k], lay.upload, cudaMemcpyHostToDevice, stream);
    if (ce == cudaSuccess)
        ce = cudaEventRecord(plan->staging_done[k], stream);
    if (ce != cudaSuccess)
        return cuda_fail(ce, "uploading the updated plan");
    plan->staging_next = k ^ 1;
    plan->num_items = (int)items;
    plan->num_partials = sc.num_partials;
    plan->num_ctas = sc.cta_items.empty() ? 0 : (int)sc.cta_items.size() - 1;
    plan->total_q = sc.total_q;
    plan->desc.batch_size = d.batch_size;
    plan->desc.fixed_split_size = d.fixed_split_size;
    plan->desc.disable_split_kv = d.disable_split_kv;
    return PKV_OK;
}

int pkv_plan_update(pkv_plan *plan, const pkv_plan_desc *desc, void *stream)
{
    NvtxRange range("pkv_plan_update");
    g_last_error.clear();
    return guarded([&] { return update_plan(plan, desc, stream); });
}

int pkv_plan_destroy(pkv_plan *plan)
{
    if (!plan)
        return PKV_OK;
    for (int k = 0; k < 2; ++k) {
        if (plan->staging_done[k]) {
            cudaEventSynchronize(plan->staging_done[k]);
            cudaEventDestroy(plan->staging_done[k]);
        }
        if (plan->staging[k])
            cudaFreeHost(plan->staging[k]);
    }
    cudaError_t ce = cudaFree(plan->workspace);
    delete plan;
    if (ce != cudaSuccess)
        return cuda_fail(ce, "cudaFree(plan workspace)");
    return PKV_OK;
}

int pkv_plan_get_info(const pkv_plan *plan, pkv_plan_info *info)
{
    if (!plan || !info)
        return fail(PKV_ERR_INVALID_ARG, "plan and info are required");
    std::memset(info, 0, sizeof *info);
    info->kind = plan->desc.kind;
    info->num_work_items = plan->num_items;
    info->num_partials = plan->num_partials;
    info->mask_mode = plan->mask_mode;
    info->workspace_bytes = (int64_t)plan->workspace_bytes;
    info->total_q = plan->total_q;
    info->kernels_per_run = ((plan->num_items > 0 || plan->capturable) ? 1 : 0) + (plan->shared ? 1 : 0) +
                            (plan->d_shared_merges ? 1 : 0);
    info->kv_tile = plan->desc.kind == PKV_DECODE
                        ? decode_kernel_tile(plan->decode_tile, plan->desc.head_dim, plan->desc.kv_dtype)
                        : prefill_kv_tile(plan->desc.head_dim);
    return PKV_OK;
}

int pkv_plan_set_timing_events(pkv_plan *plan, void *ev_begin, void *ev_end)
{
    if (!plan)
        return fail(PKV_ERR_INVALID_ARG, "plan is NULL");
    plan->ev_begin = (cudaEvent_t)ev_begin;
    plan->ev_end = (cudaEvent_t)ev_end;
    return PKV_OK;
}

int pkv_plan_device_status(const pkv_plan *plan, int32_t *status)
{
    if (!plan || !status)
        return fail(PKV_ERR_INVALID_ARG, "plan and status are required");
    int32_t h = 0;
    cudaError_t ce = cudaDeviceSynchronize();
    if (ce == cudaSuccess)
        ce = cudaMemcpy(&h, plan->d_status, sizeof h, cudaMemcpyDeviceToHost);
    // cleared before the next run, on whatever stream, can record anything
    if (ce == cudaSuccess)
        ce = cudaMemset(plan->d_status, 0, sizeof(int32_t));
    if (ce == cudaSuccess)
        ce = cudaDeviceSynchronize();
    if (ce != cudaSuccess)
        return cuda_fail(ce, "reading the device status");
    *status = h;
    return PKV_OK;
}

static int page_shift_of(int page_size)
{
    if (page_size <= 0 || (page_size & (page_size - 1)))
        return -1;
    int s = 0;
    while ((1 << s) < page_size)
        ++s;
    return s;
}

static bool misaligned(const void *p, uintptr_t a) { return ((uintptr_t)p) % a != 0; }

static int run_plan(const pkv_plan *plan, const void *q, const void *k_cache, const void *k_block_scales,
                    const void *v_cache, const void *v_block_scales, void *out, float *lse, void *stream_)
{
    const bool blocks = plan->desc.kv_dtype == PKV_FP4_E2M1;
    if (blocks && (plan->num_items > 0 || plan->capturable) && (!k_block_scales || !v_block_scales))
        return fail(PKV_ERR_INVALID_ARG, "a 4-bit cache needs its block scales (pkv_run_blocks)");
    if (!blocks && (k_block_scales || v_block_scales))
        return fail(PKV_ERR_INVALID_ARG, "block scales belong to 4-bit caches");
    if (misaligned(k_block_scales, 16) || misaligned(v_block_scales, 16))
        return fail(PKV_ERR_INVALID_ARG, "block scales must be 16-byte aligned");
    if ((plan->total_q > 0 || plan->capturable) && (!q || !out))
        return fail(PKV_ERR_INVALID_ARG, "q and out are required");
    if ((plan->num_items > 0 || plan->capturable) && (!k_cache || !v_cache))
        return fail(PKV_ERR_INVALID_ARG, "k_cache and v_cache are required");
    if (misaligned(q, 16) || misaligned(k_cache, 16) || misaligned(v_cache, 16) ||
        misaligned(out, 16) || misaligned(lse, 4))
        return fail(PKV_ERR_INVALID_ARG, "q, caches and out must be 16-byte aligned, lse 4-byte");
    int cur = -1;
    if (cudaGetDevice(&cur) == cudaSuccess && cur != plan->device)
        return fail(PKV_ERR_INVALID_ARG, "plan was made on device %d, current device is %d",
                    plan->device, cur);
    // A capturable plan always launches (its launch may be captured and replayed
    // after pkv_plan_update); its decode grid is the capacity, its prefill grid one
    // CTA per SM, and CTAs without work leave at once.
    if (plan->num_items == 0 && !plan->capturable)
        return PKV_OK;
    cudaStream_t stream = (cudaStream_t)stream_;
    const pkv_plan_desc &d = plan->desc;
    cudaError_t ce;
    if (d.kind == PKV_DECODE) {
        DecodeParams p{};
        p.items = (const DecodeItem *)plan->d_items;
        p.reqs = plan->d_reqs;
        p.kv_indices = plan->kv_indices;
        p.q = (const uint16_t *)q;
        p.k_cache = (const uint16_t *)k_cache;
        p.v_cache = (const uint16_t *)v_cache;
        p.out = (uint16_t *)out;
        p.lse = lse;
        p.partial_o = plan->d_partial_o;
        p.partial_lse = plan->d_partial_lse;
        p.merge_counters = plan->d_shared_merges ? nullptr : plan->d_counters;
        p.live_items = plan->capturable ? plan->d_live : nullptr;
        p.status = plan->d_status;
        p.num_qo_heads = d.num_qo_heads;
        p.num_kv_heads = d.num_kv_heads;
        p.page_size = d.page_size;
        p.page_shift = page_shift_of(d.page_size);
        p.num_pages = d.num_pages;
        const LogitFactors lf = logit_factors(d);
        p.sm_scale_log2 = lf.sm_scale_log2;
        p.cap_in = lf.cap_in;
        p.cap_out = lf.cap_out;
        p.v_scale = lf.v_scale;
        p.kv_dtype = d.kv_dtype;
        p.wait_probe = d.wait_probe;
        p.sinks = plan->sinks > 0;
        p.wait_ns = wait_ns_of(d);
        p.k_block_scales = (const uint8_t *)k_block_scales;
        p.v_block_scales = (const uint8_t *)v_block_scales;
        p.shared = plan->shared;
        if (plan->ev_begin && (ce = cudaEventRecord(plan->ev_begin, stream)) != cudaSuccess)
            return cuda_fail(ce, "cudaEventRecord");
        if (plan->shared) {
            SharedParams sp{};
            sp.items = plan->d_shared_items;
            sp.cta_items = plan->d_shared_cta;
            sp.rows = plan->d_shared_rows;
            sp.kv_indices = p.kv_indices;
            sp.q = p.q;
            sp.k_cache = (const uint8_t *)k_cache;
            sp.v_cache = (const uint8_t *)v_cache;
            sp.k_block_scales = p.k_block_scales;
            sp.v_block_scales = p.v_block_scales;
            sp.partial_o = p.partial_o;
            sp.partial_lse = p.partial_lse;
            sp.status = p.status;
            sp.num_qo_heads = p.num_qo_heads;
            sp.num_kv_heads = p.num_kv_heads;
            sp.group = d.num_qo_heads / d.num_kv_heads;
            sp.page_size = p.page_size;
            sp.page_shift = p.page_shift;
            sp.num_pages = p.num_pages;
            sp.sm_scale_log2 = p.sm_scale_log2;
            sp.cap_in = p.cap_in;
            sp.cap_out = p.cap_out;
            sp.wait_probe = p.wait_probe;
            sp.wait_ns = p.wait_ns;
            ce = launch_shared_prefix(sp, d.head_dim, d.kv_dtype, plan->num_shared_ctas, stream);
            if (ce != cudaSuccess)
                return cuda_fail(ce, "shared prefix kernel launch");
        }
        ce = launch_decode(p, d.head_dim, plan->capturable ? (int)plan->cap_items : plan->num_items, stream,
                           plan->decode_tile);
        if (ce != cudaSuccess)
            return cuda_fail(ce, "decode kernel launch");
        if (plan->d_shared_merges) {
            ce = launch_shared_merge(p, plan->d_shared_merges, d.batch_size, d.head_dim, stream);
            if (ce != cudaSuccess)
                return cuda_fail(ce, "merge kernel launch");
        }
        if (plan->ev_end && (ce = cudaEventRecord(plan->ev_end, stream)) != cudaSuccess)
            return cuda_fail(ce, "cudaEventRecord");
        return PKV_OK;
    }
    PrefillParams p{};
    p.items = (const PrefillItem *)plan->d_items;
    p.cta_items = plan->d_cta_items;
    p.reqs = plan->d_reqs;
    p.kv_indices = plan->kv_indices;
    p.q = (const uint16_t *)q;
    p.k_cache = (const uint16_t *)k_cache;
    p.v_cache = (const uint16_t *)v_cache;
    p.out = (uint16_t *)out;
    p.lse = lse;
    p.status = plan->d_status;
    p.num_qo_heads = d.num_qo_heads;
    p.num_kv_heads = d.num_kv_heads;
    p.group = d.num_qo_heads / d.num_kv_heads;
    p.tokens_per_tile = std::max(1, kPrefillRows / p.group);
    p.total_q = (int32_t)(plan->capturable ? plan->cap_total_q : plan->total_q);
    p.page_size = d.page_size;
    p.page_shift = page_shift_of(d.page_size);
    p.num_pages = d.num_pages;
    p.window_left = d.window_left;
    p.sinks = plan->sinks;
    const LogitFactors lf = logit_factors(d);
    p.sm_scale_log2 = lf.sm_scale_log2;
    p.cap_in = lf.cap_in;
    p.cap_out = lf.cap_out;
    p.v_scale = lf.v_scale;
    p.ragged = d.kind == PKV_PREFILL_RAGGED ? 1 : 0;
    p.kv_dtype = d.kv_dtype;
    p.wait_probe = d.wait_probe;
    p.wait_ns = wait_ns_of(d);
    p.total_kv = (int32_t)plan->total_kv;
    if (p.ragged) {
        p.page_size = 1;
        p.page_shift = 0;
        p.num_pages = (int32_t)plan->total_kv;
    }
    if (plan->ev_begin && (ce = cudaEventRecord(plan->ev_begin, stream)) != cudaSuccess)
        return cuda_fail(ce, "cudaEventRecord");
    ce = launch_prefill_pp(p, d.head_dim, plan->mask_mode, plan->capturable ? plan->n_sm : plan->num_ctas, stream);
    if (ce != cudaSuccess)
        return cuda_fail(ce, "prefill kernel launch");
    if (plan->ev_end && (ce = cudaEventRecord(plan->ev_end, stream)) != cudaSuccess)
        return cuda_fail(ce, "cudaEventRecord");
    return PKV_OK;
}

int pkv_run(const pkv_plan *plan, const void *q, const void *k_cache, const void *v_cache, void *out,
            float *lse, void *stream)
{
    NvtxRange range(plan && plan->desc.kind == PKV_DECODE ? "pkv_run decode" : "pkv_run prefill");
    g_last_error.clear();
    if (!plan)
        return fail(PKV_ERR_INVALID_ARG, "plan is NULL");
    return run_plan(plan, q, k_cache, nullptr, v_cache, nullptr, out, lse, stream);
}

int pkv_run_blocks(const pkv_plan *plan, const void *q, const void *k_cache, const void *k_block_scales,
                   const void *v_cache, const void *v_block_scales, void *out, float *lse, void *stream)
{
    NvtxRange range("pkv_run_blocks");
    g_last_error.clear();
    if (!plan)
        return fail(PKV_ERR_INVALID_ARG, "plan is NULL");
    return run_plan(plan, q, k_cache, k_block_scales, v_cache, v_block_scales, out, lse, stream);
}

int pkv_merge_state(const void *v_a, const float *s_a, const void *v_b, const float *s_b, void *v_out,
                    float *s_out, int64_t n_tokens, int32_t n_heads, int32_t head_dim, int32_t dtype,
                    void *stream)
{
    NvtxRange range("pkv_merge_state");
    g_last_error.clear();
    if (n_tokens < 0 || n_heads < 0)
        return fail(PKV_ERR_INVALID_ARG, "negative size");
    if (dtype != PKV_BF16 && dtype != PKV_F32)
        return fail(PKV_ERR_UNSUPPORTED, "merge_state dtype %d", dtype);
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return fail(PKV_ERR_UNSUPPORTED, "head_dim %d not in {64, 128, 256}", head_dim);
    const int64_t rows = n_tokens * (int64_t)n_heads;
    if (rows == 0)
        return PKV_OK;
    if (!v_a || !s_a || !v_b || !s_b || !v_out || !s_out)
        return fail(PKV_ERR_INVALID_ARG, "null pointer");
    if (misaligned(v_a, 16) || misaligned(v_b, 16) || misaligned(v_out, 16))
        return fail(PKV_ERR_INVALID_ARG, "value pointers must be 16-byte aligned");
    cudaError_t ce = launch_merge_state(v_a, s_a, v_b, s_b, v_out, s_out, rows, head_dim, dtype,
                                        (cudaStream_t)stream);
    if (ce != cudaSuccess)
        return cuda_fail(ce, "merge_state launch");
    return PKV_OK;
}

}  // extern "C"
