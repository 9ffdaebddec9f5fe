// append_sm100.cu -- new tokens into the paged cache with the norm and the
// position rotation on the way: into bf16 pages (fa_append_paged_rope) and
// into 8-bit pages with a scale for each block of tokens and head
// (fa_append_paged_fp8).
//
// The cache is the page pool of the page "“Flash”不是那个被时代淘汰的插件"
// (0539edu.com), section 2, whose section 3 rotates queries and keys from a
// precomputed table as they are made.  One launch takes the projections'
// output to what attention reads: queries rotated, keys rotated and stored,
// values stored.  Each row is read and written once.
//
// Each CTA finds its own sequence: its threads look at the sequences' offsets
// and lengths together, one sequence a thread, and the block sums the pages
// before it.  That is one round trip to L2, overlapped with the loads of the
// rows, where a plan kernel before it would be a launch of its own.
#include <cuda_fp8.h>

#include <cmath>

#include "fa_internal.h"
#include "rope_row.cuh"

namespace fa {
namespace {

constexpr int kPage = 256;
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

struct Append {
    const __nv_bfloat16 *q, *k, *v;  // new rows, `stride` elements a token apart
    __nv_bfloat16* qo;               // [total, H, D]
    int64_t sq, sk, sv;
    const int32_t *cu, *table, *lens;
    int table_len, max_pages;  // max_pages 0: packed table
    void *kp, *vp;             // pages
    float *ks, *vs;            // 8-bit pages: scales [P, Hk, kPage / block]
    int block_log2;
    NormWeight wq, wk;
    RopeTable t;
    int B, H, Hk, total, num_pages;
    int units;  // 8-bit: (sequence, block) pairs with new rows, at most
    float eps;
    unsigned int* err;
};

// A sequence as the offsets and lengths give it; `bad`: nothing of it is
// touched (reported once).
struct Seq {
    int b, row0, n, len;
    int64_t page_base;
    bool found, bad;
};

// Lengths may be anything up to 2^31 - 1, and so may their sums be wrong: page
// counts are added in 64 bits.
__device__ __forceinline__ int pages_of(int len) {
    return len <= 0 ? 0 : len / kPage + (len % kPage != 0);
}

// The rows of sequence b: cu[b] .. cu[b + 1] - 1, cut to [0, total].
__device__ __forceinline__ void rows_of(const Append& p, int b, int& r0, int& n, bool& bad) {
    const int lo = __ldg(p.cu + b), hi = __ldg(p.cu + b + 1);
    bad = lo < 0 || hi > p.total || hi < lo;
    r0 = min(max(lo, 0), p.total);
    n = bad ? 0 : hi - lo;
}

// Sum over the block (every thread gets it).
__device__ __forceinline__ int64_t block_sum(int64_t a, int64_t* sh /*[kWarps]*/) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = a;
    __syncthreads();
    int64_t s = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s += sh[i];
    __syncthreads();
    return s;
}

// Whether the sequence's new rows fit it, its table row and the rotation's
// table (page_base: packed tables' entries before it).
__device__ __forceinline__ bool seq_bad(const Append& p, int n, int len,
                                        int64_t page_base) {
    if (n > len || (p.t.half > 0 && len > p.t.max_pos)) return true;
    const int np = pages_of(len);
    return p.max_pages ? np > p.max_pages : page_base + np > p.table_len;
}

// The page of position pos, or -1 (reported) where its index is outside the pool.
__device__ __forceinline__ int page_at(const Append& p, const Seq& s, int pos) {
    const int64_t at = p.max_pages ? static_cast<int64_t>(s.b) * p.max_pages + pos / kPage
                                   : s.page_base + pos / kPage;
    const int page = __ldg(p.table + at);
    if (page < 0 || page >= p.num_pages) {
        if (threadIdx.x == 0) record_error(p.err, FA_DEVERR_BAD_INPUT);
        return -1;
    }
    return page;
}

struct Shared {
    int64_t units[kWarps], pages[kWarps];
    int64_t page_base;
    int b, blk;
};

// The sequence that holds row r, found by the whole CTA.
__device__ __forceinline__ Seq find_row(const Append& p, int r, Shared& sh) {
    if (threadIdx.x == 0) sh.b = -1;
    __syncthreads();
    int mine = -1;
    for (int i = threadIdx.x; i < p.B; i += kThreads) {
        int r0, n;
        bool bad;
        rows_of(p, i, r0, n, bad);
        if (r >= r0 && r < r0 + n) mine = i;
        if (bad) record_error(p.err, FA_DEVERR_BAD_INPUT);
    }
    if (mine >= 0) atomicMax(&sh.b, mine);  // offsets that overlap: the last one
    __syncthreads();
    Seq s{};
    s.b = sh.b;
    s.found = s.b >= 0;
    int64_t pages = 0;
    if (!p.max_pages)
        for (int i = threadIdx.x; i < s.b; i += kThreads) pages += pages_of(__ldg(p.lens + i));
    s.page_base = block_sum(pages, sh.pages);
    if (!s.found) return s;
    rows_of(p, s.b, s.row0, s.n, s.bad);
    s.len = __ldg(p.lens + s.b);
    s.bad = s.bad || seq_bad(p, s.n, s.len, s.page_base);
    if (s.bad && threadIdx.x == 0) record_error(p.err, FA_DEVERR_BAD_INPUT);
    return s;
}

// ---------------------------------------------------------------------------
// bf16 pages: a CTA takes one token; D / 8 lanes a row of it, the H query
// rows, H_kv key rows and H_kv value rows in turn.
// ---------------------------------------------------------------------------
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) fa_append_rope_kernel(const Append p) {
    constexpr int LPR = D / 8, SL = kThreads / LPR;
    __shared__ Shared sh;
    const int r = blockIdx.x;
    const int my = threadIdx.x / LPR;
    const Seq s = find_row(p, r, sh);
    if (!s.found) return;
    const int pos = s.bad ? 0 : s.len - s.n + (r - s.row0);
    const int page = s.bad ? -1 : page_at(p, s, pos);
    const Lane<D, INTER> lane(p.t.half);
    Rotation<D, INTER> rot;
    rot.load(p.t, pos, lane);
    __nv_bfloat16* kp = static_cast<__nv_bfloat16*>(p.kp);
    __nv_bfloat16* vp = static_cast<__nv_bfloat16*>(p.vp);
    const int rows = p.H + 2 * p.Hk;
    for (int i = my; i - my < rows; i += SL) {
        const bool live = i < rows;
        const bool is_q = i < p.H, is_k = !is_q && i < p.H + p.Hk;
        const int h = is_q ? i : is_k ? i - p.H : min(i - p.H - p.Hk, p.Hk - 1);
        const __nv_bfloat16* x = is_q ? p.q + r * p.sq : is_k ? p.k + r * p.sk : p.v + r * p.sv;
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (live) raw = lane.load(x + static_cast<int64_t>(h) * D);
        Vec8 y = lane.unpack(raw);
        if (p.wq.w || p.wk.w) {
            const float rs = row_rstd<D>(y, p.eps);
            const NormWeight nw = is_q ? p.wq : p.wk;
            if (nw.w && (is_q || is_k)) y = mul8(y, scale8(lane.weights(nw), rs));
        }
        rot.apply(y);
        if (!live) continue;
        if (is_q) {
            lane.store(p.qo + (static_cast<int64_t>(r) * p.H + h) * D,
                       s.bad ? make_uint4(0, 0, 0, 0) : lane.pack(y));
        } else if (page >= 0) {
            const int64_t at = ((static_cast<int64_t>(page) * p.Hk + h) * kPage + pos % kPage) * D;
            if (is_k) lane.store(kp + at, lane.pack(y));
            else lane.store(vp + at, raw);  // values as they are
        }
    }
}

// ---------------------------------------------------------------------------
// 8-bit pages.  A block of `block` tokens of one head shares one scale, a
// power of two, so that a scale that grows only shifts the exponents of the
// codes already there: they are rounded again only where they fall below the
// format's normal range.  With a the largest finite magnitude of the block's
// new values, the scale is the least 2^e with a <= 448 * 2^e (e in [-64, 64]),
// or the block's present scale where it holds earlier tokens and that is
// larger.  A CTA takes one (sequence, block) and one head of K or of V.
// ---------------------------------------------------------------------------
constexpr float kMaxCode = 448.f;

// The least e in [-64, 64] with a <= 448 * 2^e (448 = 0.875 * 2^9).
__device__ __forceinline__ int scale_exponent(float a) {
    int e;
    const float m = frexpf(a, &e);
    return a > 0.f ? min(max(e - 9 + (m > 0.875f), -64), 64) : -64;
}

// y / scale.  The inverse of a power of two is exact (2^-64 .. 2^64), so the
// product is the quotient; a caller's other scale divides.
__device__ __forceinline__ void divide8(float (&y)[8], float scale) {
    if ((__float_as_uint(scale) & 0x7fffffu) == 0) {  // the same for the CTA
        const float inv = 1.f / scale;
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= inv;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = __fdiv_rn(y[j], scale);
    }
}

// 8-bit codes of values already divided by the scale: to nearest even; what
// the format cannot hold is stored as NaN, so that it shows.
__device__ __forceinline__ float codable(float v) {
    return fabsf(v) <= kMaxCode ? v : __int_as_float(0x7fffffff);
}

__device__ __forceinline__ uint2 encode8(const float (&y)[8]) {
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        h[j] = __nv_cvt_float2_to_fp8x2(make_float2(codable(y[2 * j]), codable(y[2 * j + 1])),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ void decode8(const uint2& u, float (&y)[8]) {
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>((w[j >> 1] >> (16 * (j & 1))) & 0xffffu), __NV_E4M3);
        const float2 f = __half22float2(__half2(hr));
        y[2 * j] = f.x;
        y[2 * j + 1] = f.y;
    }
}

// The new tokens of (sequence, block) number `unit`: the blocks that hold new
// rows are counted over the sequences.
__device__ __forceinline__ bool find_unit(const Append& p, int unit, Shared& sh, Seq& s,
                                          int& blk) {
    const int lg = p.block_log2;
    int64_t before = 0, pages = 0;  // of the sequences scanned
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) sh.b = -1;
    for (int base = 0; base < p.B; base += kThreads) {
        const int i = base + threadIdx.x;
        int c = 0, np = 0, r0 = 0, n = 0, len = 0;
        bool bad = false;
        if (i < p.B) {
            rows_of(p, i, r0, n, bad);
            len = __ldg(p.lens + i);
            np = pages_of(len);
            if (bad || n > len) {  // no units, but its pages count
                record_error(p.err, FA_DEVERR_BAD_INPUT);
            } else if (n > 0) {
                c = ((len - 1) >> lg) - ((len - n) >> lg) + 1;
            }
        }
        int64_t ci = c, pi = np;  // inclusive prefixes over the block
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t a = __shfl_up_sync(0xffffffffu, ci, o);
            const int64_t b = __shfl_up_sync(0xffffffffu, pi, o);
            if (lane >= o) {
                ci += a;
                pi += b;
            }
        }
        if (lane == 31) {
            sh.units[warp] = ci;
            sh.pages[warp] = pi;
        }
        __syncthreads();
        int64_t all_units = 0, all_pages = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) {
                ci += sh.units[w];
                pi += sh.pages[w];
            }
            all_units += sh.units[w];
            all_pages += sh.pages[w];
        }
        if (unit >= before + ci - c && unit < before + ci) {
            sh.b = i;
            sh.blk = static_cast<int>(unit - (before + ci - c));
            sh.page_base = pages + pi - np;
        }
        before += all_units;
        pages += all_pages;
        __syncthreads();
        if (before > unit) break;
    }
    s = Seq{};
    s.b = sh.b;
    s.found = s.b >= 0;
    if (!s.found) return false;
    rows_of(p, s.b, s.row0, s.n, s.bad);
    s.len = __ldg(p.lens + s.b);
    s.page_base = sh.page_base;
    s.bad = s.bad || seq_bad(p, s.n, s.len, s.page_base);
    blk = ((s.len - s.n) >> lg) + sh.blk;
    if (s.bad && threadIdx.x == 0) record_error(p.err, FA_DEVERR_BAD_INPUT);
    return !s.bad;
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) fa_append_fp8_kernel(const Append p) {
    constexpr int LPR = D / 8, SL = kThreads / LPR;
    __shared__ Shared sh;
    __shared__ float red[kWarps];
    const int my = threadIdx.x / LPR;
    const Lane<D, INTER> lane(p.t.half);
    const int kv_ctas = p.units * 2 * p.Hk;
    if (static_cast<int>(blockIdx.x) >= kv_ctas) {
        // query rows: one token's heads over a CTA's slots
        const int r = blockIdx.x - kv_ctas;
        const Seq s = find_row(p, r, sh);
        if (!s.found) return;
        const int pos = s.bad ? 0 : s.len - s.n + (r - s.row0);
        Rotation<D, INTER> rot;
        rot.load(p.t, pos, lane);
        Vec8 w = {};
        if (p.wq.w) w = lane.weights(p.wq);
        for (int h = my; h - my < p.H; h += SL) {
            const bool live = h < p.H;
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (live) raw = lane.load(p.q + r * p.sq + static_cast<int64_t>(h) * D);
            Vec8 y = lane.unpack(raw);
            if (p.wq.w) y = norm_row<D>(y, w, p.eps);
            rot.apply(y);
            if (live)
                lane.store(p.qo + (static_cast<int64_t>(r) * p.H + h) * D,
                           s.bad ? make_uint4(0, 0, 0, 0) : lane.pack(y));
        }
        return;
    }
    const int unit = blockIdx.x / (2 * p.Hk), sub = blockIdx.x - unit * 2 * p.Hk;
    const bool is_k = sub < p.Hk;
    const int h = is_k ? sub : sub - p.Hk;
    Seq s;
    int blk = 0;
    if (!find_unit(p, unit, sh, s, blk)) return;
    const int lg = p.block_log2, start = s.len - s.n;
    const int lo = blk << lg;                              // the block's first position
    const int first = max(lo, start), last = min(lo + (1 << lg), s.len);
    const int page = page_at(p, s, lo);
    if (page < 0) return;
    const __nv_bfloat16* x = (is_k ? p.k : p.v) + static_cast<int64_t>(h) * D;
    const int64_t sx = is_k ? p.sk : p.sv;
    const bool norms = is_k && p.wk.w;
    Vec8 w = {};
    if (norms) w = lane.weights(p.wk);
    // row `pos` of the new tokens, normed and rotated
    auto row = [&](int pos, float (&y)[8]) {
        Vec8 v = lane.unpack(lane.load(x + (s.row0 + (pos - start)) * sx));
        if (norms) v = norm_row<D>(v, w, p.eps);
        if (is_k) {
            Rotation<D, INTER> rot;
            rot.load(p.t, pos, lane);
            rot.apply(v);
        }
        lane.in_order(v, y);
    };
    float amax = 0.f;
    for (int i = first + my; i - my < last; i += SL) {
        float y[8];
        row(min(i, last - 1), y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float a = fabsf(y[j]);
            if (a < INFINITY) amax = fmaxf(amax, a);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
    const int64_t slice = static_cast<int64_t>(page) * p.Hk + h;
    float* scale = (is_k ? p.ks : p.vs) + slice * (kPage >> lg) + ((lo % kPage) >> lg);
    const float was = first > lo ? *scale : 0.f;
    __syncthreads();  // every thread has read the old scale
#pragma unroll
    for (int i = 0; i < kWarps; ++i) amax = fmaxf(amax, red[i]);
    const int e = scale_exponent(amax);
    const float now = fmaxf(was, ldexpf(1.f, e));
    uint8_t* dst = static_cast<uint8_t*>(is_k ? p.kp : p.vp) +
                   (slice * kPage + lo % kPage) * D;
    if (threadIdx.x == 0) *scale = now;
    if (first > lo && now != was) {  // earlier tokens under the larger scale
        const float ratio = was / now;  // now is a power of two
        for (int i = my; i < first - lo; i += SL) {
            float y[8];
            uint8_t* c = dst + static_cast<int64_t>(i) * D;
            decode8(lane.load(c), y);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= ratio;
            lane.store(c, encode8(y));
        }
    }
    for (int i = first + my; i - my < last; i += SL) {
        float y[8];
        row(min(i, last - 1), y);
        divide8(y, now);
        if (i < last) lane.store(dst + static_cast<int64_t>(i - lo) * D, encode8(y));
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int stride_of(int stride, int heads, int d, int64_t* out) {
    *out = stride == 0 ? static_cast<int64_t>(heads) * d : stride;
    if (*out < static_cast<int64_t>(heads) * d) return FA_ERR_SHAPE;
    return *out % 8 == 0 ? FA_OK : FA_ERR_ALIGN;
}

// The arguments that both appends share.
int fill(Append& p, const void* q_new, const void* k_new, const void* v_new,
         const int32_t* cu_new, void* q_out, void* k_pages, void* v_pages,
         const int32_t* page_table, int table_len, int max_pages, const int32_t* seq_lens,
         const void* q_weight, const void* k_weight, int weight_type, const float* rope_cos,
         const float* rope_sin, int max_pos, int rotary_dim, int B, int H, int H_kv,
         int total_new, int num_pages, int d, int page_size, int q_stride, int k_stride,
         int v_stride, float eps) {
    if (!k_new || !v_new || !cu_new || !k_pages || !v_pages || !page_table || !seq_lens)
        return FA_ERR_NULL;
    if ((q_new == nullptr) != (q_out == nullptr)) return FA_ERR_NULL;
    if (rotary_dim > 0 && (!rope_cos || !rope_sin)) return FA_ERR_NULL;
    if (B < 1 || H < 0 || H_kv < 1 || total_new < 0 || num_pages < 1 || max_pages < 0 ||
        table_len < 0 || rotary_dim < 0 || (q_new && H < 1))
        return FA_ERR_SHAPE;
    if (max_pages > 0 && static_cast<int64_t>(B) * max_pages > table_len) return FA_ERR_SHAPE;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (page_size != kPage) return FA_ERR_UNSUPPORTED;
    if (rotary_dim % 16 != 0) return FA_ERR_UNSUPPORTED;
    if (rotary_dim > d || (rotary_dim > 0 && max_pos < 1)) return FA_ERR_SHAPE;
    if (weight_type != FA_WEIGHT_BF16 && weight_type != FA_WEIGHT_FP32) return FA_ERR_UNSUPPORTED;
    if (!std::isfinite(eps) || eps < 0.f) return FA_ERR_SHAPE;
    int rc;
    if ((rc = stride_of(q_stride, H, d, &p.sq)) != FA_OK) return rc;
    if ((rc = stride_of(k_stride, H_kv, d, &p.sk)) != FA_OK) return rc;
    if ((rc = stride_of(v_stride, H_kv, d, &p.sv)) != FA_OK) return rc;
    const void* wide[] = {q_new, k_new, v_new, q_out, k_pages, v_pages, q_weight, k_weight,
                          rope_cos, rope_sin};
    for (const void* w : wide)
        if (!aligned16(w)) return FA_ERR_ALIGN;
    p.q = static_cast<const __nv_bfloat16*>(q_new);
    p.k = static_cast<const __nv_bfloat16*>(k_new);
    p.v = static_cast<const __nv_bfloat16*>(v_new);
    p.qo = static_cast<__nv_bfloat16*>(q_out);
    p.cu = cu_new;
    p.table = page_table;
    p.lens = seq_lens;
    p.table_len = table_len;
    p.max_pages = max_pages;
    p.kp = k_pages;
    p.vp = v_pages;
    p.wq = NormWeight{q_new ? q_weight : nullptr, weight_type == FA_WEIGHT_FP32};
    p.wk = NormWeight{k_weight, weight_type == FA_WEIGHT_FP32};
    p.t = RopeTable{rope_cos, rope_sin, max_pos, rotary_dim / 2};
    p.B = B;
    p.H = q_new ? H : 0;
    p.Hk = H_kv;
    p.total = total_new;
    p.num_pages = num_pages;
    p.eps = eps;
    return FA_OK;
}

template <int D, bool INTER>
int launch_rope(const Append& p, cudaStream_t st) {
    fa_append_rope_kernel<D, INTER><<<p.total, kThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D, bool INTER>
int launch_fp8(const Append& p, cudaStream_t st) {
    const int64_t ctas = static_cast<int64_t>(p.units) * 2 * p.Hk + (p.q ? p.total : 0);
    fa_append_fp8_kernel<D, INTER><<<static_cast<unsigned>(ctas), kThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

extern "C" {

int fa_append_paged_rope(const void* q_new, const void* k_new, const void* v_new,
                         const int32_t* cu_new, void* q_out, void* k_pages, void* v_pages,
                         const int32_t* page_table, int table_len, int max_pages,
                         const int32_t* seq_lens, const void* q_weight, const void* k_weight,
                         int weight_type, const float* rope_cos, const float* rope_sin,
                         int max_pos, int rotary_dim, int interleaved, int B, int H, int H_kv,
                         int total_new, int num_pages, int d, int page_size, int q_stride,
                         int k_stride, int v_stride, float eps, fa_stream_t stream) {
    fa::Append p{};
    int rc = fa::fill(p, q_new, k_new, v_new, cu_new, q_out, k_pages, v_pages, page_table,
                      table_len, max_pages, seq_lens, q_weight, k_weight, weight_type, rope_cos,
                      rope_sin, max_pos, rotary_dim, B, H, H_kv, total_new, num_pages, d,
                      page_size, q_stride, k_stride, v_stride, eps);
    int num_sms = 0;
    if (rc != FA_OK || (rc = fa::device_error_word(&p.err, &num_sms)) != FA_OK) return rc;
    if (total_new == 0) return FA_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d == 64)
        return interleaved ? fa::launch_rope<64, true>(p, st) : fa::launch_rope<64, false>(p, st);
    return interleaved ? fa::launch_rope<128, true>(p, st) : fa::launch_rope<128, false>(p, st);
}

int fa_append_paged_fp8(const void* q_new, const void* k_new, const void* v_new,
                        const int32_t* cu_new, void* q_out, void* k_pages, void* v_pages,
                        float* k_scales, float* v_scales, int block,
                        const int32_t* page_table, int table_len, int max_pages,
                        const int32_t* seq_lens, const void* q_weight, const void* k_weight,
                        int weight_type, const float* rope_cos, const float* rope_sin,
                        int max_pos, int rotary_dim, int interleaved, int B, int H, int H_kv,
                        int total_new, int num_pages, int d, int page_size, int q_stride,
                        int k_stride, int v_stride, float eps, fa_stream_t stream) {
    if (!k_scales || !v_scales) return FA_ERR_NULL;
    if (block < 16 || block > fa::kPage || (block & (block - 1)) != 0) return FA_ERR_UNSUPPORTED;
    fa::Append p{};
    int rc = fa::fill(p, q_new, k_new, v_new, cu_new, q_out, k_pages, v_pages, page_table,
                      table_len, max_pages, seq_lens, q_weight, k_weight, weight_type, rope_cos,
                      rope_sin, max_pos, rotary_dim, B, H, H_kv, total_new, num_pages, d,
                      page_size, q_stride, k_stride, v_stride, eps);
    if (rc != FA_OK) return rc;
    // scales are read one by one
    if ((reinterpret_cast<uintptr_t>(k_scales) | reinterpret_cast<uintptr_t>(v_scales)) & 3u)
        return FA_ERR_ALIGN;
    p.ks = k_scales;
    p.vs = v_scales;
    while ((1 << p.block_log2) < block) ++p.block_log2;
    // a sequence with n new rows touches at most (n - 1) / block + 2 blocks,
    // and no more than n
    const int64_t seqs = B < total_new ? B : total_new;
    const int64_t most = static_cast<int64_t>(total_new) / block + 2 * seqs;
    p.units = static_cast<int>(most < total_new ? most : total_new);
    if (static_cast<int64_t>(p.units) * 2 * H_kv + total_new > 0x7fffffff) return FA_ERR_SHAPE;
    int num_sms = 0;
    if ((rc = fa::device_error_word(&p.err, &num_sms)) != FA_OK) return rc;
    if (total_new == 0) return FA_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d == 64)
        return interleaved ? fa::launch_fp8<64, true>(p, st) : fa::launch_fp8<64, false>(p, st);
    return interleaved ? fa::launch_fp8<128, true>(p, st) : fa::launch_fp8<128, false>(p, st);
}

}  // extern "C"
