// Split-KV paged decode over 4-bit caches: e2m1 values, two to a byte (the even column in
// the low half), and an e4m3 scale for every 16 columns of a token's head,
//     K = k_scale * s * e2m1,
// 0.5625 bytes a value. The work items, windows, sinks, splits and the merge of partial
// states are those of pkv_decode_kernel.cuh; the inner loop is another, because at this
// size a key is bound by the instructions that widen it and not by its bytes:
//   - the products are turned over, S^T = K Q^T and O^T = V^T P^T with mma.sync m16n8k16: K and
//     V are the 16-row operand and the query heads (8 to a CTA) the 8 columns, so that an
//     MMA takes 256 values of the cache (128 with the heads as rows), and a lane holds half
//     the accumulators and half the softmax that it would for 16 rows of which 8 are used;
//   - S^T comes out with a token to a row and is the B operand of O^T after one movmatrix per
//     8 tokens;
//   - a 32-bit word of a K row is eight columns: k-slots take them in the order in which they
//     lie (a dot product has no order), and a transposed load of V gives two tokens of four
//     columns each;
//   - s * e2m1 has at most six significant bits and lies in [2^-10, 2688]: exact in f16. q is
//     scaled by a power of two to fit f16 (as for 8-bit caches), P is rounded to f16.
// A CTA takes HP neighbouring KV heads of a request, a warp each for its own head and tokens:
// the heads' rows of a token lie side by side in the cache, so that one TMA box brings whole lines
// of a page for all of them, and another the page's block scales in whole sectors. The copies'
// number and the producer's instructions matter as much as the bytes: boxes of two heads were
// 14% slower on long ranges, and copies of each row's scales by the lanes as much again. Where
// the work is little, fewer heads a CTA (and more warps for the tokens of each) finish it
// sooner; the plan picks (choose_fp4_decode in pkv_api.cpp).
// The running maximum moves only where a score exceeds it by 2^8 (P stays below 2^8, far
// from f16's largest value), so that most stages take one vote instead of the shuffles of a
// maximum; sums are fp32.
// V rows that are not visible take block scales of 0, so that whatever their 4-bit values are,
// which are all finite, their products are 0.
//
// Measured, 8 KV heads of 128: 256 requests of 16384 keys 226 us, 0.80 of the time that their bytes
// take at the copy rate; without the copies, the instructions alone 200 us. 64 requests of
// 256-4096 keys 39.7 us (0.57: CTAs of unequal length, 193 partial states), 256 requests of
// 6000-8192 keys under a window of 4095 with 128 sinks 246 us (0.75), one of 4001 keys 8.6 us.
#pragma once

#include <cfloat>

#include "pkv_decode_merge.cuh"
#include "pkv_internal.h"
#include "pkv_sm100.cuh"

namespace pkv {
namespace dec4 {

constexpr int kRows = kFp4DecodeRows;  // query heads of a CTA

// NWH compute warps of 32 tokens (two 16-token sub-blocks) for each of HP KV heads.
template <int D, int HP, int NWH>
struct Traits {
    static constexpr int kTPW = 32;
    static constexpr int kWarps = HP * NWH;
    static constexpr int kTile = NWH * kTPW;
    static constexpr int kThreads = 32 * (kWarps + 1);
    static constexpr int kRowBytes = D / 2;            // one head's row
    static constexpr int kLine = HP * kRowBytes < 128 ? HP * kRowBytes : 128;  // bytes of a line
    static constexpr int kLines = HP * kRowBytes / kLine;                      // lines of a token
    static constexpr int kGran = kRowBytes / 16;       // 16-byte granules (32 columns) of a row
    static constexpr int kScales = D / 16;             // scale bytes of a row
    static constexpr int kScaleLine = HP * kScales;
    static constexpr int kTileBytes = kTile * HP * kRowBytes;
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kScaleBytes = 2 * kTile * kScaleLine;  // K's, then V's
    static constexpr int kStages = D == 256 ? 3 : 4;
    static constexpr int kORow = D + 4;                // floats of a row of the combine buffer
    static constexpr int kRingBytes = kStages * (kStageBytes + kScaleBytes);
    static constexpr int kCombineBytes = kWarps * kRows * kORow * 4;
    static constexpr int kDynSmem = (kRingBytes > kCombineBytes ? kRingBytes : kCombineBytes) + 1024;
    // as many CTAs to an SM as shared memory (228 KB, 1 KB of it and 1 KB of static each) and
    // about 112 registers a thread (160 at head_dim 256) allow
    static constexpr int kFitSmem = 228 * 1024 / (kDynSmem + 2048);
    static constexpr int kFitRegs = 65536 / (kThreads * (D == 256 ? 168 : 128));
    static constexpr int kMinBlocks = kFitSmem < kFitRegs ? kFitSmem : kFitRegs;
};

// A tile is [8-token groups][N lines][8 tokens][R bytes], each group of a line as a TMA box with
// the swizzle of R bytes stores it: the granules of 128 / R neighbouring rows form one 128-byte
// line, and these turn by R / 16 granules. Byte offset of granule c of line l of token r:
template <int R, int N>
__device__ __forceinline__ uint32_t row_off(int r, int l, int c)
{
    return (uint32_t)(((r >> 3) * N + l) * (8 * R) + (r & 7) * R +
                      ((c ^ (R == 128 ? r & 7 : R == 64 ? (r >> 1) & 3 : (r >> 2) & 1)) << 4));
}

// Copy n = 4, 8 or 16 bytes global -> shared (zeros for src_bytes = 0).
template <int N>
__device__ __forceinline__ void cp_async_n(uint32_t dst, const void *src, uint32_t src_bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(dst), "l"(src), "n"(N), "r"(src_bytes) : "memory");
}

// Eight e2m1 values (a 32-bit word, lowest half byte first) as four f16x2 words.
__device__ __forceinline__ void widen8(uint32_t w, uint32_t (&x)[4])
{
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n"
        " cvt.rn.f16x2.e2m1x2 %1, b;\n cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
        : "r"(w));
}

__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// D = A B of m16n8k16 (f16 in, fp32 out).
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Two f16 values times one half of s.
template <bool HIGH>
__device__ __forceinline__ uint32_t times_half(uint32_t x, uint32_t s)
{
    const __half2 v = *reinterpret_cast<const __half2 *>(&s);
    const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&x), HIGH ? __high2half2(v) : __low2half2(v));
    return *reinterpret_cast<const uint32_t *>(&y);
}

// The transpose of an 8 x 8 matrix of 16-bit values (a row's pairs to four lanes).
__device__ __forceinline__ uint32_t movmatrix(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(a));
    return d;
}

template <int W>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&w)[W])
{
    static_assert(W == 1 || W == 2 || W == 4, "words");
    if (W == 1)
        asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(w[0]) : "r"(addr));
    else if (W == 2)
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];\n" : "=r"(w[0]), "=r"(w[W > 1 ? 1 : 0]) : "r"(addr));
    else
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                     : "=r"(w[0]), "=r"(w[W > 1 ? 1 : 0]), "=r"(w[W > 2 ? 2 : 0]), "=r"(w[W > 3 ? 3 : 0])
                     : "r"(addr));
}

// Every other byte of two words, from byte h on: the scales of one 16-column half of four
// granules.
__device__ __forceinline__ uint32_t half_scales(uint32_t a, uint32_t b, int h)
{
    return __byte_perm(a, b, h ? 0x7531 : 0x6420);
}

// Tensor maps of the caches and, where a token's are 16 bytes, of the block scales.
struct Maps {
    CUtensorMap k, v, ks, vs;
};

template <int D, int HP, bool TMA_KV, int NWH, bool SINK, bool SHARED>
__global__ void __launch_bounds__(Traits<D, HP, NWH>::kThreads, Traits<D, HP, NWH>::kMinBlocks)
    decode_fp4_kernel(const DecodeParams p, const __grid_constant__ Maps tm)
{
    using Tr = Traits<D, HP, NWH>;
    constexpr int TT = Tr::kTile, S = Tr::kStages, SB = Tr::kScales, TPW = Tr::kTPW, NW = Tr::kWarps;
    constexpr int LINE = Tr::kLine, NL = Tr::kLines, TOKEN = LINE * NL, SL = Tr::kScaleLine;
    constexpr bool TMA_S = TMA_KV && SL >= 16;  // scales by TMA
    constexpr int NG = Tr::kGran;  // granules of 32 columns
    constexpr int NT = 32 * NW;    // compute threads
    extern __shared__ uint8_t dsmem_raw[];
    __shared__ __align__(8) uint64_t full_bar[S];
    __shared__ __align__(8) uint64_t empty_bar[S];
    __shared__ float red_m[NW][kRows];
    __shared__ float red_l[NW][kRows];
    __shared__ float row_m[HP * kRows];  // of KV head hp's query heads, from kRows hp on
    __shared__ float row_inv_l[HP * kRows];
    __shared__ float row_lse[SHARED ? HP * kRows : 1];  // of this CTA's own keys
    __shared__ __align__(8) uint64_t never_bar;  // the wait probe's barrier: nothing completes it
    __shared__ int abort_flag;
    __shared__ int no_abort;

    const uint32_t ring = (smem_u32(dsmem_raw) + 1023u) & ~1023u;
    uint8_t *ring_gen = dsmem_raw + (ring - smem_u32(dsmem_raw));
    const uint32_t scale_ring = ring + S * Tr::kStageBytes;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (p.live_items && (int)blockIdx.x >= *p.live_items) {
        grid_dependency_wait();  // (see pkv_decode_kernel.cuh)
        return;
    }
    const DecodeItem it = p.items[blockIdx.x];
    // Packed rows u of an item with sinks: those of the sinks, then those of the window.
    int u_sink = 0, u_lo = it.j0, u_hi = it.j1, join = 0, shift = 0;
    if (SINK) {
        const int A = !TMA_KV ? 1 : (p.page_size < TT ? p.page_size : TT);
        const int base = it.j0 / A * A;
        u_sink = it.sink_end;
        join = min((u_sink + A - 1) / A * A, base);
        shift = base - join;
        u_lo = it.j0 - shift;
        u_hi = it.j1 - shift;
    }
    auto key_of = [&](int u) { return SINK && u >= join ? u + shift : u; };
    auto visible = [&](int u) { return (u >= u_lo && u < u_hi) || (SINK && u < u_sink); };
    const int tb = SINK ? 0 : (it.j1 > it.j0 ? (it.j0 / TT) * TT : it.j0);  // first tile start
    const int ntiles = it.j1 > it.j0 ? (u_hi - tb + TT - 1) / TT : 0;
    const volatile int *abort_v = &abort_flag;

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&full_bar[s]), TMA_S ? 1 : TMA_KV ? 33 : 32);  // (copies by the lanes)
            mbar_init(smem_u32(&empty_bar[s]), NW);
        }
        mbar_init(smem_u32(&never_bar), 1);
        abort_flag = 0;
        no_abort = 0;
        fence_mbarrier_init();
        fence_proxy_async_smem();
    }
    __syncthreads();
    if (!SHARED)  // (see Shared prefixes in pkv_decode_kernel.cuh)
        grid_dependency_wait();

    if (warp == NW) {
        // ------------------------------------------------------------ producer
        // Rows of a tile are handed out as lane + 32 k (k < KR); a row of the cache, page *
        // page_size + slot, is below 2^32 - 1 (larger caches are refused).
        constexpr int KR = TT / 32;
        constexpr uint32_t kNone = 0xffffffffu;
        const int P = p.page_size, H = p.num_kv_heads;
        int issued = 0;
        bool ok = true;
        const uint8_t *ks = p.k_block_scales + (size_t)it.kv_head * SB, *vs = p.v_block_scales + (size_t)it.kv_head * SB;
        const size_t scale_row = (size_t)H * SB;  // bytes from a token's scales to the next one's
        const int rows_box = P < TT ? P : TT;
        const int npg = TMA_KV ? TT / rows_box : 0;
        const int n_pages_req = (it.kv_len + P - 1) / P;
        auto page_of = [&](int lp) -> int {
            const int pg = p.kv_indices[it.kv_page_begin + lp];
            if ((unsigned)pg >= (unsigned)p.num_pages) {
                record_status(p.status, PKV_ERR_DEVICE_BOUNDS);
                return -1;
            }
            return pg;
        };
        // TMA: boxes of whole pages, or of TT rows of one. In units of A rows (A = min(P, TT)) the
        // first tile starts at unit u0, packed units from `join_u` on lie `shift_u` further.
        const int A = TMA_KV ? rows_box : 1;
        const int u0 = TMA_KV ? tb / A : 0, join_u = SINK && TMA_KV ? join / A : 0, shift_u = SINK && TMA_KV ? shift / A : 0;
        const int per = TMA_KV && P > TT ? P / TT : 1;  // units of a page
        int box[KR], in_box[KR];
        if (TMA_KV && !TMA_S) {
#pragma unroll
            for (int k = 0; k < KR; ++k) {
                box[k] = (lane + 32 * k) / rows_box;
                in_box[k] = lane + 32 * k - box[k] * rows_box;
            }
        }
        int slot0 = 0;  // first slot of this tile's box and of the next one's (P > TT)
        auto load_id = [&](int t, int &slot) -> int {
            // (one box of a larger page, the same for all lanes)
            const int u = u0 + t * npg + (per > 1 ? 0 : lane), first = u * A;
            int lp = SINK && u >= join_u ? u + shift_u : u;
            slot = 0;
            if (per > 1) {
                const int q = lp / per;
                slot = (lp - q * per) * TT;
                lp = q;
            }
            if (lane >= npg || lp >= n_pages_req || ((first >= u_hi || first + rows_box <= u_lo) && !(SINK && first < u_sink)))
                return -1;
            return page_of(lp);
        };
        // gather: the cache row of this lane's k-th row of tile t
        auto load_row = [&](int t, int k) -> uint32_t {
            const int u = tb + t * TT + lane + 32 * k;
            if (!visible(u))
                return kNone;
            const int j = key_of(u), lp = p.page_shift >= 0 ? (j >> p.page_shift) : j / P;
            const int pg = page_of(lp);
            return pg < 0 ? kNone : (uint32_t)pg * (uint32_t)P + (uint32_t)(j - lp * P);
        };
        if (TMA_KV && lane == 0) {
            tma_prefetch_desc(&tm.k);
            tma_prefetch_desc(&tm.v);
            if (TMA_S) {
                tma_prefetch_desc(&tm.ks);
                tma_prefetch_desc(&tm.vs);
            }
        }
        int pg = -1;
        uint32_t row_id[KR];
        if (ntiles > 0) {
            if (TMA_KV) {
                pg = load_id(0, slot0);
            } else {
#pragma unroll
                for (int k = 0; k < KR; ++k)
                    row_id[k] = load_row(0, k);
            }
        }
        for (int t = 0; t < ntiles; ++t) {
            const int s = t % S;
            int pg_next = -1, slot_next = 0;
            uint32_t row_next[KR];
            if (TMA_KV) {
                if (t + 1 < ntiles)
                    pg_next = load_id(t + 1, slot_next);
            } else {
#pragma unroll
                for (int k = 0; k < KR; ++k)
                    row_next[k] = t + 1 < ntiles ? load_row(t + 1, k) : kNone;
            }
            if (t >= S) {
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&empty_bar[s]), ((t / S) - 1) & 1, abort_v, p.wait_ns));
                if (!ok)
                    break;
            }
            const int ts = tb + t * TT;
            const uint32_t kb = ring + s * Tr::kStageBytes, vb = kb + Tr::kTileBytes;
            const uint32_t ksb = scale_ring + s * Tr::kScaleBytes, vsb = ksb + TT * SL;
            const uint32_t full = smem_u32(&full_bar[s]);
            if (TMA_KV) {
                const unsigned valid = __ballot_sync(0xffffffffu, pg >= 0);
                if (lane == 0)
                    mbar_arrive_expect_tx(full, (uint32_t)__popc(valid) * rows_box * (TOKEN + (TMA_S ? SL : 0)) * 2);
                __syncwarp();
                if (pg >= 0) {
                    // (rows pass 31 bits, their blocks of 8 do not)
                    const int x = it.kv_head / HP, block = (int)(((uint32_t)pg * (uint32_t)P + (uint32_t)slot0) >> 3);
                    tma_load_4d(kb + lane * rows_box * TOKEN, &tm.k, 0, 0, x * NL, block, full);
                    tma_load_4d(vb + lane * rows_box * TOKEN, &tm.v, 0, 0, x * NL, block, full);
                    if (TMA_S) {
                        tma_load_4d(ksb + lane * rows_box * SL, &tm.ks, 0, 0, x, block, full);
                        tma_load_4d(vsb + lane * rows_box * SL, &tm.vs, 0, 0, x, block, full);
                    }
                }
                const bool edge = !(ts >= u_lo && ts + TT <= u_hi);
#pragma unroll
                for (int k = 0; !TMA_S && k < KR; ++k) {
                    const int page = __shfl_sync(0xffffffffu, pg, box[k]);
                    row_id[k] = page < 0 || (edge && !visible(ts + lane + 32 * k))
                                    ? kNone
                                    : (uint32_t)page * (uint32_t)P + (uint32_t)(slot0 + in_box[k]);
                }
            } else {
                // TOKEN / 16 lanes copy a token's rows
                constexpr int LPR = TOKEN / 16, RPI = 32 / LPR;
                const int l = lane % LPR / (LINE / 16), c = lane % (LINE / 16);
#pragma unroll
                for (int i = 0; i < TT / RPI; ++i) {
                    const int row = i * RPI + lane / LPR;
                    const uint32_t id = __shfl_sync(0xffffffffu, row_id[i * RPI / 32], row & 31);
                    const uint32_t bytes = id == kNone ? 0 : 16;
                    const size_t at = id == kNone ? 0 : ((size_t)id * H + it.kv_head) * Tr::kRowBytes + (lane % LPR) * 16;
                    cp_async_16(kb + row_off<LINE, NL>(row, l, c), reinterpret_cast<const uint8_t *>(p.k_cache) + at, bytes);
                    cp_async_16(vb + row_off<LINE, NL>(row, l, c), reinterpret_cast<const uint8_t *>(p.v_cache) + at, bytes);
                }
            }
#pragma unroll
            for (int k = 0; !TMA_S && k < KR; ++k) {
                const size_t at = row_id[k] == kNone ? 0 : row_id[k] * scale_row;
                const uint32_t bytes = row_id[k] == kNone ? 0 : 1, row = lane + 32 * k;
                constexpr int N = SL < 16 ? SL : 16;
#pragma unroll
                for (int e = 0; e < SL; e += N) {
                    cp_async_n<N>(ksb + row * SL + e, ks + at + e, bytes ? N : 0);
                    cp_async_n<N>(vsb + row * SL + e, vs + at + e, bytes ? N : 0);
                }
            }
            if (!TMA_S)
                cp_async_mbar_arrive(full);
            issued = t + 1;
            pg = pg_next;
            slot0 = slot_next;
            if (!TMA_KV) {
#pragma unroll
                for (int k = 0; k < KR; ++k)
                    row_id[k] = row_next[k];
            }
        }
        if (!ok && lane == 0) {
            record_status(p.status, PKV_ERR_TIMEOUT);
            abort_flag = 1;
        }
        // Never leave with copies in flight: wait for the last stages issued.
        for (int t = issued - S < 0 ? 0 : issued - S; t < issued; ++t)
            mbar_wait(smem_u32(&full_bar[t % S]), (t / S) & 1, &no_abort, p.wait_ns);
        asm volatile("cp.async.wait_all;\n" ::: "memory");
    } else {
        // ------------------------------------------------------------ compute
        const int n = lane >> 2, c = lane & 3;
        const int hp = warp / NWH, head0 = it.head0 + hp * (p.num_qo_heads / p.num_kv_heads);  // this warp's KV and query heads
        // Q as the B operand: head n's columns 32g + 8c .. 8c + 7, the k-slots of two k-steps.
        uint32_t qf[NG][4];
        float q_unscale;
        {
            const uint4 *q = reinterpret_cast<const uint4 *>(
                p.q + ((size_t)it.row * p.num_qo_heads + head0 + (n < it.nheads ? n : 0)) * D);
            float amax = 0.f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint4 x = n < it.nheads ? q[4 * g + c] : make_uint4(0u, 0u, 0u, 0u);
                qf[g][0] = x.x; qf[g][1] = x.y; qf[g][2] = x.z; qf[g][3] = x.w;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    amax = max3f(amax, fabsf(__uint_as_float(qf[g][r] << 16)), fabsf(__uint_as_float(qf[g][r] & 0xffff0000u)));
            }
            // q * 2^qe with max |q| * 2^qe in [2^13, 2^14): exact in f16 above 2^-28 of the largest
#pragma unroll
            for (int sh = 16; sh >= 1; sh >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, sh));
            int qe = 13 - ((int)((__float_as_uint(amax) >> 23) & 0xff) - 127);
            qe = qe < -100 ? -100 : (qe > 100 ? 100 : qe);
            const float up = __uint_as_float((uint32_t)(127 + qe) << 23);
            q_unscale = __uint_as_float((uint32_t)(127 - qe) << 23);
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    qf[g][r] = pack_f16(__uint_as_float(qf[g][r] << 16) * up, __uint_as_float(qf[g][r] & 0xffff0000u) * up);
        }
        // heads 2c and 2c + 1: running maximum (the same in all lanes of a c), this lane's sum
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        // o[2g + t]: columns 32g + 4n + 2t, + 1 of heads 2c, 2c + 1 (column, head)
        float o[2 * NG][4];
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i)
            o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        const float cap_in = p.cap_in * q_unscale;  // raw MMA dot -> tanh argument
        // raw MMA dot, or tanh, -> log2-domain logit
        const float unit = p.cap_in > 0.f ? p.cap_out * p.sm_scale_log2 : p.sm_scale_log2 * q_unscale;
        bool ok = true;
        // This lane's address in an x4 matrix load (matrix mi: tokens 8 (mi & 1).., granule + (mi >> 1)),
        // within a tile and for the warp's first token: the swizzle depends on the token's lowest
        // three bits, which are the lane's, so that granules 2 gp differ from it by one XOR.
        const int w0 = (warp % NWH) * TPW;  // first token of this warp
        const uint32_t mat = row_off<LINE, NL>(w0 + (((lane >> 3) & 1) << 3) + (lane & 7), hp * Tr::kRowBytes / LINE,
                                               hp * NG % (LINE / 16) + (lane >> 4));

        for (int t = 0; t < ntiles; ++t) {
            const int s = t % S;
            const uint32_t fb = (p.wait_probe && t == 0) ? smem_u32(&never_bar) : smem_u32(&full_bar[s]);
            ok = __all_sync(0xffffffffu, mbar_wait(fb, (t / S) & 1, abort_v, p.wait_ns));
            if (!ok)
                break;
            const uint32_t kb = ring + s * Tr::kStageBytes, vb = kb + Tr::kTileBytes;
            const uint32_t ksb = scale_ring + s * Tr::kScaleBytes + hp * SB, vsb = ksb + TT * SL;
            const int wt0 = tb + t * TT + w0;
            const bool partial = (wt0 < u_lo || wt0 + TPW > u_hi) && !(SINK && wt0 + TPW <= u_sink);
            if (TMA_S && partial) {  // (copies by the lanes fill these rows with zeros)
                if (!visible(wt0 + lane)) {
#pragma unroll
                    for (int k = 0; k < SB; k += 4)
                        asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(vsb + (w0 + lane) * SL + k), "r"(0) : "memory");
                }
                __syncwarp();
            }

            // S^T of each 16-token sub-block: rows tokens n, n + 8, columns heads 2c, 2c + 1
            float sc[2][4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int row0 = w0 + 16 * b;
                float acc[2][4];
                // scales of tokens n and n + 8 for this lane's half (c >> 1) of each granule
                uint32_t sl[NG / 2], sh[NG / 2];
                {
                    uint32_t a[SB / 4], z[SB / 4];
                    lds<SB / 4>(ksb + (row0 + n) * SL, a);
                    lds<SB / 4>(ksb + (row0 + n + 8) * SL, z);
#pragma unroll
                    for (int k = 0; k < SB / 4; k += 2) {
                        uint32_t unused;
                        const uint32_t x = half_scales(a[k], SB > 4 ? a[SB > 4 ? k + 1 : 0] : 0u, c >> 1);
                        const uint32_t y = half_scales(z[k], SB > 4 ? z[SB > 4 ? k + 1 : 0] : 0u, c >> 1);
                        if (SB > 4) {
                            e4m3x4_to_f16x2(x, sl[k], sl[SB > 4 ? k + 1 : 0]);
                            e4m3x4_to_f16x2(y, sh[k], sh[SB > 4 ? k + 1 : 0]);
                        } else {
                            e4m3x4_to_f16x2(x, sl[0], unused);
                            e4m3x4_to_f16x2(y, sh[0], unused);
                        }
                    }
                }
#pragma unroll
                for (int gp = 0; gp < NG / 2; ++gp) {
                    uint32_t w[4];
                    ldmatrix_x4(kb + 16 * b * TOKEN + (mat ^ (gp << 5)), w[0], w[1], w[2], w[3]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int g = 2 * gp + h;
                        uint32_t x[4], y[4];
                        widen8(w[2 * h], x);
                        widen8(w[2 * h + 1], y);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[e] = h ? times_half<true>(x[e], sl[gp]) : times_half<false>(x[e], sl[gp]);
                            y[e] = h ? times_half<true>(y[e], sh[gp]) : times_half<false>(y[e], sh[gp]);
                        }
                        const uint32_t a0[4] = {x[0], y[0], x[1], y[1]}, a1[4] = {x[2], y[2], x[3], y[3]};
                        if (g == 0) {
                            mma_first(acc[0], a0, qf[g][0], qf[g][1]);
                            mma_first(acc[1], a1, qf[g][2], qf[g][3]);
                        } else {
                            mma_f16_16816(acc[0], a0, qf[g][0], qf[g][1]);
                            mma_f16_16816(acc[1], a1, qf[g][2], qf[g][3]);
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sc[b][e] = acc[0][e] + acc[1][e];
            }
            // scores in units of `unit` (> 0) of the log2 domain
            if (p.cap_in > 0.f) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[b][e] = soft_cap_tanh(sc[b][e] * cap_in);
            }
            if (partial) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!visible(wt0 + 16 * b + n + (e >> 1) * 8))
                            sc[b][e] = -INFINITY;
            }
            float mx0 = unit * fmaxf(fmaxf(sc[0][0], sc[0][2]), fmaxf(sc[1][0], sc[1][2]));
            float mx1 = unit * fmaxf(fmaxf(sc[0][1], sc[0][3]), fmaxf(sc[1][1], sc[1][3]));
            if (__any_sync(0xffffffffu, mx0 > m[0] + 8.f || mx1 > m[1] + 8.f)) {
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, x));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, x));
                }
                const float m0 = fmaxf(m[0], mx0), m1 = fmaxf(m[1], mx1);
                const float a0 = m[0] == -INFINITY ? 0.f : fast_exp2(m[0] - m0);
                const float a1 = m[1] == -INFINITY ? 0.f : fast_exp2(m[1] - m1);
                m[0] = m0;
                m[1] = m1;
                l[0] *= a0;
                l[1] *= a1;
#pragma unroll
                for (int i = 0; i < 2 * NG; ++i) {
                    o[i][0] *= a0;
                    o[i][1] *= a1;
                    o[i][2] *= a0;
                    o[i][3] *= a1;
                }
            }
            const float ref0 = m[0] == -INFINITY ? 0.f : m[0], ref1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                sc[b][0] = fast_exp2(fmaf(sc[b][0], unit, -ref0));
                sc[b][1] = fast_exp2(fmaf(sc[b][1], unit, -ref1));
                sc[b][2] = fast_exp2(fmaf(sc[b][2], unit, -ref0));
                sc[b][3] = fast_exp2(fmaf(sc[b][3], unit, -ref1));
                l[0] += sc[b][0] + sc[b][2];
                l[1] += sc[b][1] + sc[b][3];
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int row0 = w0 + 16 * b;
                const uint32_t b0 = movmatrix(pack_f16(sc[b][0], sc[b][1]));
                const uint32_t b1 = movmatrix(pack_f16(sc[b][2], sc[b][3]));
                // scales of token pairs 2c, 2c + 1 and 2c + 8, 2c + 9 for this lane's half (n >> 2)
                uint32_t vl[NG], vh[NG];
                {
                    uint32_t a[4][SB / 4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        lds<SB / 4>(vsb + (row0 + 2 * c + (k & 1) + (k >> 1) * 8) * SL, a[k]);
                    const uint32_t sel = n >> 2 ? 0x7351 : 0x6240;
#pragma unroll
                    for (int k = 0; k < SB / 4; ++k) {
                        e4m3x4_to_f16x2(__byte_perm(a[0][k], a[1][k], sel), vl[2 * k], vl[2 * k + 1]);
                        e4m3x4_to_f16x2(__byte_perm(a[2][k], a[3][k], sel), vh[2 * k], vh[2 * k + 1]);
                    }
                }
#pragma unroll
                for (int gp = 0; gp < NG / 2; ++gp) {
                    uint32_t w[4];
                    ldmatrix_x4_trans(vb + 16 * b * TOKEN + (mat ^ (gp << 5)), w[0], w[1], w[2], w[3]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int g = 2 * gp + h;
                        // x[0], x[1]: columns 4n, +1 and +2, +3 of token 2c; x[2], x[3] of 2c + 1
                        uint32_t x[4], y[4];
                        widen8(w[2 * h], x);
                        widen8(w[2 * h + 1], y);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t a[4] = {hmul2(__byte_perm(x[e], x[e + 2], 0x5410), vl[g]),
                                                   hmul2(__byte_perm(x[e], x[e + 2], 0x7632), vl[g]),
                                                   hmul2(__byte_perm(y[e], y[e + 2], 0x5410), vh[g]),
                                                   hmul2(__byte_perm(y[e], y[e + 2], 0x7632), vh[g])};
                            mma_f16_16816(o[2 * g + e], a, b0, b1);
                        }
                    }
                }
            }
            if (TMA_S && partial)
                fence_proxy_async_smem();  // the zeros precede the next copy into this stage
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&empty_bar[s]));
        }
        if (!ok && lane == 0) {
            record_status(p.status, PKV_ERR_TIMEOUT);
            abort_flag = 1;
        }

        grid_launch_dependents();
        if (SHARED && p.merge_counters)  // (see pkv_decode_kernel.cuh)
            grid_dependency_wait();
        const bool from_registers = SHARED && p.merge_counters && it.partial >= 0 && it.nsplit == 1;
        // Merge the compute warps' states (named barrier 1 over the compute threads).
#pragma unroll
        for (int x = 4; x <= 16; x <<= 1) {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], x);
            l[1] += __shfl_xor_sync(0xffffffffu, l[1], x);
        }
        if (n == 0) {
            red_m[warp][2 * c] = m[0];
            red_m[warp][2 * c + 1] = m[1];
            red_l[warp][2 * c] = l[0];
            red_l[warp][2 * c + 1] = l[1];
        }
        asm volatile("bar.sync 1, %0;\n" ::"n"(NT) : "memory");
        const int group = p.num_qo_heads / p.num_kv_heads;
        if (tid < HP * kRows) {
            const int x = tid / kRows, r = tid % kRows;
            float M = red_m[x * NWH][r];
#pragma unroll
            for (int w = 1; w < NWH; ++w)
                M = fmaxf(M, red_m[x * NWH + w][r]);
            const float ref = M == -INFINITY ? 0.f : M;
            float L = 0.f;
#pragma unroll
            for (int w = 0; w < NWH; ++w)
                L += red_l[x * NWH + w][r] * fast_exp2(red_m[x * NWH + w][r] - ref);
            row_m[tid] = M;
            row_inv_l[tid] = L > 0.f ? (it.partial >= 0 ? 1.f : p.v_scale) / L : 0.f;
            if (r < it.nheads && !abort_flag) {
                const float lse_v = L > 0.f ? (M + __log2f(L)) * 0.6931471805599453f : -INFINITY;
                const int h = it.head0 + x * group + r;
                if (SHARED)
                    row_lse[tid] = lse_v;
                if (from_registers)
                    ;
                else if (it.partial >= 0)
                    p.partial_lse[(size_t)it.partial * p.num_qo_heads + h] = lse_v;
                else if (p.lse)
                    p.lse[(size_t)it.row * p.num_qo_heads + h] = lse_v;
            }
        }
        // The ring's stages have been consumed: it becomes the combine buffer.
        asm volatile("bar.sync 1, %0;\n" ::"n"(NT) : "memory");
        float *sO = reinterpret_cast<float *>(ring_gen);
        {
            const int r = hp * kRows + 2 * c;
            const float M0 = row_m[r], M1 = row_m[r + 1];
            const float f0 = fast_exp2(m[0] - (M0 == -INFINITY ? 0.f : M0)) * row_inv_l[r];
            const float f1 = fast_exp2(m[1] - (M1 == -INFINITY ? 0.f : M1)) * row_inv_l[r + 1];
            float *d0 = sO + (warp * kRows + 2 * c) * Tr::kORow + 4 * n, *d1 = d0 + Tr::kORow;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                *reinterpret_cast<float4 *>(d0 + 32 * g) =
                    make_float4(o[2 * g][0] * f0, o[2 * g][2] * f0, o[2 * g + 1][0] * f0, o[2 * g + 1][2] * f0);
                *reinterpret_cast<float4 *>(d1 + 32 * g) =
                    make_float4(o[2 * g][1] * f1, o[2 * g][3] * f1, o[2 * g + 1][1] * f1, o[2 * g + 1][3] * f1);
            }
        }
        asm volatile("bar.sync 1, %0;\n" ::"n"(NT) : "memory");
        if (!abort_flag) {
            for (int idx = tid; idx < HP * kRows * (D / 8); idx += NT) {
                const int x = idx / (kRows * (D / 8)), r = idx / (D / 8) % kRows, col = (idx % (D / 8)) * 8;
                if (r >= it.nheads)
                    continue;
                float acc[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    acc[e] = 0.f;
#pragma unroll
                for (int w = 0; w < NWH; ++w) {
                    const float4 *src = reinterpret_cast<const float4 *>(sO + ((x * NWH + w) * kRows + r) * Tr::kORow + col);
                    const float4 x = src[0], y = src[1];
                    acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
                    acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
                }
                const int h = it.head0 + x * group + r;
                if (from_registers) {
                    merge_own<D>(p, it.pbase + 1, (int)(it.prefix_pieces >> (8 * x) & 0xff), it.row, h, col, acc,
                                 row_lse[x * kRows + r]);
                } else if (it.partial >= 0) {
                    float4 *dst = reinterpret_cast<float4 *>(p.partial_o + ((size_t)it.partial * p.num_qo_heads + h) * D + col);
                    dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
                } else {
                    *reinterpret_cast<uint4 *>(p.out + ((size_t)it.row * p.num_qo_heads + h) * D + col) =
                        make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]), pack_bf16(acc[4], acc[5]),
                                   pack_bf16(acc[6], acc[7]));
                }
            }
        }
        if (it.partial >= 0 && !from_registers && p.merge_counters) {
            // The last CTA of the split group merges its partial states through their LSE.
            __shared__ int last_flag;
            asm volatile("bar.sync 1, %0;\n" ::"n"(NT) : "memory");
            if (tid == 0) {
                __threadfence();
                last_flag = atomicAdd(p.merge_counters + it.counter, 1) == it.nsplit - 1;
            }
            asm volatile("bar.sync 1, %0;\n" ::"n"(NT) : "memory");
            if (last_flag) {
                __threadfence();
                for (int idx = tid; idx < HP * it.nheads * (D / 8); idx += NT) {
                    const int x = idx / (it.nheads * (D / 8)), r = idx / (D / 8) - x * it.nheads;
                    const int h = it.head0 + x * group + r, col = (idx % (D / 8)) * 8;
                    const int prefix = SHARED ? (int)(it.prefix_pieces >> (8 * x) & 0xff) : 0;
                    merge_partials<D>(p, it.pbase, it.nsplit + prefix, it.row, h, col);
                }
                if (tid == 0)
                    atomicExch(p.merge_counters + it.counter, 0);
            }
        }
    }
    if (SHARED && blockIdx.x == gridDim.x - 1)
        grid_dependency_wait();
}

template <int D, int HP, bool TMA_KV, int NWH, bool SINK, bool SHARED>
cudaError_t launch(const DecodeParams &p, const Maps &tm, int num_items, cudaStream_t s)
{
    using Tr = Traits<D, HP, NWH>;
    const auto kernel = decode_fp4_kernel<D, HP, TMA_KV, NWH, SINK, SHARED>;
    static std::atomic<uint64_t> configured{0};
    const cudaError_t e = allow_smem(kernel, Tr::kDynSmem, configured);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)num_items);
    cfg.blockDim = dim3(Tr::kThreads);
    cfg.dynamicSmemBytes = Tr::kDynSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, tm);
}

template <int D, int HP, int NWH, bool SINK, bool SHARED>
cudaError_t launch_t(const DecodeParams &p, bool tma, const Maps &tm, int num_items, cudaStream_t s)
{
    return tma ? launch<D, HP, true, NWH, SINK, SHARED>(p, tm, num_items, s)
               : launch<D, HP, false, NWH, SINK, SHARED>(p, tm, num_items, s);
}

template <bool SINK, bool SHARED = false>
cudaError_t launch_all(const DecodeParams &p, int head_dim, int num_items, cudaStream_t s, int heads, bool tma,
                       const Maps &tm)
{
    // (32 tokens a warp: fp4_decode_tile)
    switch (head_dim) {
    case 64:
        return heads == 4 ? launch_t<64, 4, 1, SINK, SHARED>(p, tma, tm, num_items, s)
                          : launch_t<64, 1, 4, SINK, SHARED>(p, tma, tm, num_items, s);
    case 128:
        return heads == 4   ? launch_t<128, 4, 1, SINK, SHARED>(p, tma, tm, num_items, s)
               : heads == 2 ? launch_t<128, 2, 2, SINK, SHARED>(p, tma, tm, num_items, s)
                            : launch_t<128, 1, 4, SINK, SHARED>(p, tma, tm, num_items, s);
    case 256:
        return heads == 4   ? launch_t<256, 4, 1, SINK, SHARED>(p, tma, tm, num_items, s)
               : heads == 2 ? launch_t<256, 2, 2, SINK, SHARED>(p, tma, tm, num_items, s)
                            : launch_t<256, 1, 4, SINK, SHARED>(p, tma, tm, num_items, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace dec4

// Units of their own, for the build: plans with sinks, and of shared prefixes.
cudaError_t launch_decode_fp4_sinks(const DecodeParams &p, int head_dim, int num_items, cudaStream_t s, int heads,
                                    bool tma, const dec4::Maps &tm);
cudaError_t launch_decode_fp4_shared(const DecodeParams &p, int head_dim, int num_items, cudaStream_t s, int heads,
                                     bool tma, const dec4::Maps &tm);

}  // namespace pkv
