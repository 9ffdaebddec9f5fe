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
// Each CTA finds its own sequences: its threads look at all offsets and
// lengths together, one sequence a thread, and scan the pages before them.
// That is one round trip to L2, overlapped with the loads of the rows and
// shared by the CTA's tokens, where a plan kernel would be a launch of its own.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fa_internal.h"
#include "rope_row.cuh"

namespace fa {
namespace {

constexpr int kPage = 256;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 16;  // of a CTA, at most, where rows are taken one by one
constexpr int kRows = 4;     // of a thread at a time
constexpr int kStages = 3;   // 8-bit pages: chunks of new rows on their way, less one
constexpr int kRing = kStages * kRows * kThreads * 16;  // bytes of shared memory

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
    int tokens;  // of a CTA that takes rows
    int units;   // 8-bit: (sequence, block) pairs with new rows, at most
    int unit_heads, unit_ctas;  // heads of a CTA that takes a unit; such CTAs
    float eps;
    unsigned int* err;
};

// A sequence as the offsets and lengths give it; `bad`: nothing of it is
// touched (reported once).
struct Seq {
    int b, row0, n, len;
    int64_t page_base;
    bool bad;
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

// Whether the sequence's new rows fit it, its table row and the rotation's
// table (page_base: packed tables' entries before it).
__device__ __forceinline__ bool seq_bad(const Append& p, int n, int len,
                                        int64_t page_base) {
    if (n > len || (p.t.half > 0 && len > p.t.max_pos)) return true;
    const int np = pages_of(len);
    return p.max_pages ? np > p.max_pages : page_base + np > p.table_len;
}

// The page of position pos, or -1 where its index is outside the pool (reported
// by threads that `tell`).
__device__ __forceinline__ int page_at(const Append& p, const Seq& s, int pos, bool tell) {
    const int64_t at = p.max_pages ? static_cast<int64_t>(s.b) * p.max_pages + pos / kPage
                                   : s.page_base + pos / kPage;
    const int page = __ldg(p.table + at);
    if (page < 0 || page >= p.num_pages) {
        if (tell) record_error(p.err, FA_DEVERR_BAD_INPUT);
        return -1;
    }
    return page;
}

struct Shared {
    int64_t units[kWarps], pages[kWarps];
    Seq seq_of_unit;
    int blk;
    // rows: of each token, its sequence; position and page
    int seq[kTokens];
    Seq of[kTokens];
    int pos[kTokens], page[kTokens];
};

// Exclusive prefix over the block; `total` of it.
__device__ __forceinline__ int64_t block_prefix(int64_t v, int64_t* sh /*[kWarps]*/,
                                                int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t n = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += n;
    }
    if (lane == 31) sh[warp] = inc;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) inc += sh[w];
        total += sh[w];
    }
    __syncthreads();
    return inc - v;
}

// Where rows first .. first + count - 1 belong: sh.pos (-1: of a sequence that
// cannot be taken) and sh.page (-1: nothing is stored); sh.seq -1: a row of no
// sequence, left alone.
__device__ __forceinline__ void place_rows(const Append& p, int first, int count, Shared& sh) {
    if (threadIdx.x < kTokens) sh.seq[threadIdx.x] = -1;
    __syncthreads();
    int64_t pages = 0;
    for (int at = 0; at < p.B; at += kThreads) {
        const int i = at + threadIdx.x;
        int r0 = 0, n = 0, len = 0;
        if (i < p.B) {
            bool bad;
            len = __ldg(p.lens + i);
            rows_of(p, i, r0, n, bad);
            if (bad || n > len) record_error(p.err, FA_DEVERR_BAD_INPUT);
        }
        const int lo = max(r0, first), hi = min(r0 + n, first + count);
        for (int r = lo; r < hi; ++r) atomicMax(&sh.seq[r - first], i);  // overlapping: the last
        int64_t base = 0, total = 0;
        if (p.max_pages) {
            __syncthreads();
        } else {
            base = pages + block_prefix(pages_of(len), sh.pages, total);
            pages += total;
        }
        for (int r = lo; r < hi; ++r)
            if (sh.seq[r - first] == i)
                sh.of[r - first] = Seq{i, r0, n, len, base, seq_bad(p, n, len, base)};
    }
    __syncthreads();
    if (threadIdx.x < count && sh.seq[threadIdx.x] >= 0) {
        const Seq s = sh.of[threadIdx.x];
        int pos = -1, page = -1;
        if (s.bad) {
            record_error(p.err, FA_DEVERR_BAD_INPUT);
        } else {
            pos = s.len - s.n + (first + static_cast<int>(threadIdx.x) - s.row0);
            page = page_at(p, s, pos, true);
        }
        sh.pos[threadIdx.x] = pos;
        sh.page[threadIdx.x] = page;
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------
// Rows one by one: the queries, and into bf16 pages the keys and values.  A
// slot is kRows heads of one token and kind, taken by D / 8 lanes; the next
// slot's rows are on their way while one is worked on, the first ones while
// the CTA looks for its sequences.
//
// 31.8K prompt tokens of 32 + 2 * 8 heads into bf16 pages: 142 us, 5.5 TB/s, 0.85
// of a copy (a CTA a token, each with its own search: 159; 32 tokens a CTA: 155).
// A step of 64 tokens 4.5 us: launch, lengths, page table, row.
// ---------------------------------------------------------------------------
template <int D, bool INTER, bool KV>
__device__ __forceinline__ void append_rows(const Append& p, int cta, Shared& sh) {
    constexpr int LPR = D / 8, SL = kThreads / LPR;
    const Lane<D, INTER> lane(p.t.half);
    const int my = threadIdx.x / LPR;
    const int first = cta * p.tokens, count = min(p.tokens, p.total - first);
    const int gq = (p.H + kRows - 1) / kRows, gk = KV ? (p.Hk + kRows - 1) / kRows : 0;
    const int groups = gq + 2 * gk, slots = count * groups;
    struct Where {
        int tok, kind, h0, rows;  // kind 0: query, 1: key, 2: value
    };
    int tok_ = my / groups, g_ = my - tok_ * groups;
    const int step_tok = SL / groups, step_g = SL - step_tok * groups;
    auto next_slot = [&]() {  // this thread's next one; no rows behind the last
        Where w;
        w.tok = tok_;
        w.kind = g_ < gq ? 0 : g_ < gq + gk ? 1 : 2;
        w.h0 = (w.kind == 0 ? g_ : w.kind == 1 ? g_ - gq : g_ - gq - gk) * kRows;
        w.rows = tok_ < count ? min(kRows, (w.kind == 0 ? p.H : p.Hk) - w.h0) : 0;
        tok_ += step_tok;
        g_ += step_g;
        if (g_ >= groups) {
            g_ -= groups;
            ++tok_;
        }
        return w;
    };
    uint4 next[kRows];
    auto fetch = [&](const Where& w) {
        const int64_t r = first + w.tok;
        const __nv_bfloat16* x = (w.kind == 0   ? p.q + r * p.sq
                                  : w.kind == 1 ? p.k + r * p.sk
                                                : p.v + r * p.sv) + static_cast<int64_t>(w.h0) * D;
#pragma unroll
        for (int u = 0; u < kRows; ++u)
            if (u < w.rows) next[u] = lane.load(x + u * D);
    };
    Where w = next_slot();
    fetch(w);
    place_rows(p, first, count, sh);
    const bool norms = p.wq.w || p.wk.w;
    for (int i = my; i - my < slots; i += SL) {  // all lanes of a warp together
        uint4 raw[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) raw[u] = next[u];
        const Where now = w;
        w = next_slot();
        fetch(w);
        if (now.rows == 0 && !norms) continue;
        const int tok = min(now.tok, count - 1);
        const bool mine = sh.seq[tok] >= 0;
        const int pos = mine ? sh.pos[tok] : -1, page = mine ? sh.page[tok] : -1;
        Rotation<D, INTER> rot;
        rot.load(p.t, max(pos, 0), lane);
        const NormWeight nw = now.kind == 0 ? p.wq : now.kind == 1 ? p.wk : NormWeight{nullptr, 0};
        Vec8 weight = {};
        if (nw.w) weight = lane.weights(nw);
        __nv_bfloat16* y;
        int64_t step;
        bool store = mine;
        if (now.kind == 0) {
            y = p.qo + (static_cast<int64_t>(first + tok) * p.H + now.h0) * D;
            step = D;
        } else {
            y = static_cast<__nv_bfloat16*>(now.kind == 1 ? p.kp : p.vp) +
                ((static_cast<int64_t>(page) * p.Hk + now.h0) * kPage + pos % kPage) * D;
            step = kPage * D;
            store = page >= 0;
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            if (u >= now.rows) raw[u] = make_uint4(0, 0, 0, 0);
            Vec8 v = lane.unpack(raw[u]);
            if (norms) {  // the same for the launch; a warp's slots may be of two kinds
                const float r = row_rstd<D>(v, p.eps);
                if (nw.w) v = mul8(v, scale8(weight, r));
            }
            rot.apply(v);
            const uint4 out = now.kind == 2 ? raw[u]  // values as they are
                              : pos < 0     ? make_uint4(0, 0, 0, 0)
                                            : lane.pack(v);
            if (store && u < now.rows) lane.store(y + u * step, out);
        }
    }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 3)
    fa_append_rope_kernel(const __grid_constant__ Append p) {
    __shared__ Shared sh;
    append_rows<D, INTER, true>(p, blockIdx.x, sh);
}

// ---------------------------------------------------------------------------
// 8-bit pages.  A block of `block` tokens of one head shares one scale, a
// power of two, so that a scale that grows only shifts the exponents of the
// codes already there: they are rounded again only where they fall below the
// format's normal range.  With a the largest finite magnitude of the block's
// new values, the scale is the least 2^e with a <= 448 * 2^e (e in [-64, 64]),
// or the block's present scale where it holds earlier tokens and that is
// larger.
//
// A CTA takes one (sequence, block) of K or of V and some of its heads, one
// after the other.  Each thread keeps its rows' values in registers between
// the maximum and the rounding (4 rows: 64 tokens of 128 values a CTA; larger
// blocks are read twice); the next heads' rows are on their way into shared memory
// meanwhile.  The positions' rotations are read from L1 again for each head (kept in
// registers, 32 of them, blocks of 128 took 105 us instead of 93).
//
// 8 x 1024 tokens of 32 + 2 * 32 heads, blocks of 64: 76 us, 4.5 TB/s, 0.69 of a
// copy; of it the queries 23 us (at their floor) and keys and values some 54 (31).
// Those are bound by latency: a barrier a head, two CTAs of 128 registers an SM
// (three spill: 109 us without the queries), the scheduler 46 % busy.  With the
// rows read twice instead of kept, 132 us; with them fetched into registers one
// head ahead instead of the ring of copies, 102.  A ring of 2 chunks 84, of 6 94.
// ---------------------------------------------------------------------------
constexpr float kMaxCode = 448.f;

// The least power of two s in [2^-64, 2^64] with a <= 448 s, a finite.  With
// a = m 2^E, m in [1, 2), and 448 = 1.75 * 2^8 it is 2^(E - 8), or the next one
// where m > 1.75: a quarter less one ulp, added to the bits, carries just then.
__device__ __forceinline__ float least_scale(float a) {
    const int f = static_cast<int>((__float_as_uint(a) + 0x1fffffu) >> 23) - 8;
    return __uint_as_float(static_cast<uint32_t>(min(max(f, 63), 191)) << 23);
}

// 1 / s of a power of two in that range.
__device__ __forceinline__ float inverse_power(float s) {
    return __uint_as_float((254u << 23) - __float_as_uint(s));
}

// 8-bit codes of values already divided by the scale: to nearest even.
__device__ __forceinline__ uint2 encode8(const float (&y)[8]) {
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        h[j] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * j], y[2 * j + 1]), __NV_SATFINITE,
                                        __NV_E4M3);
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
// rows are counted over the sequences.  One CTA of a launch without queries (whose
// rows' CTAs look at all sequences) looks at those behind its unit too, so that what
// is wrong with them is reported.
__device__ __forceinline__ bool find_unit(const Append& p, int unit, Shared& sh, Seq& s,
                                          int& blk) {
    const int lg = p.block_log2;
    int64_t before = 0, pages = 0;  // of the sequences scanned
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool all = blockIdx.x == 0 && !p.q;
    if (threadIdx.x == 0) sh.blk = -1;
    for (int base = 0; base < p.B; base += kThreads) {
        const int i = base + threadIdx.x;
        int c = 0, np = 0, r0 = 0, n = 0, len = 0;
        if (i < p.B) {
            bool bad;
            len = __ldg(p.lens + i);
            rows_of(p, i, r0, n, bad);
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
            const int64_t first_page = pages + pi - np;
            sh.blk = ((len - n) >> lg) + static_cast<int>(unit - (before + ci - c));
            sh.seq_of_unit = Seq{i, r0, n, len, first_page, seq_bad(p, n, len, first_page)};
        }
        before += all_units;
        pages += all_pages;
        __syncthreads();
        if (before > unit && !all) break;
    }
    blk = sh.blk;
    if (blk < 0) return false;
    s = sh.seq_of_unit;
    if (s.bad && threadIdx.x == 0) record_error(p.err, FA_DEVERR_BAD_INPUT);
    return !s.bad;
}

// Largest magnitude of a lane's values, infinities among them, NaN not.
__device__ __forceinline__ float largest8(const Vec8& v) {
    float m = fmaxf(fabsf(f2_lo(v.a[0])), fabsf(f2_hi(v.a[0])));
    m = max3f(m, fabsf(f2_lo(v.a[1])), fabsf(f2_hi(v.a[1])));
    m = max3f(m, fabsf(f2_lo(v.b[0])), fabsf(f2_hi(v.b[0])));
    return max3f(m, fabsf(f2_lo(v.b[1])), fabsf(f2_hi(v.b[1])));
}

// The largest finite magnitude of R of a lane's rows; `odd`: infinities too.
template <int D, bool INTER, int R>
__device__ __forceinline__ float finite_max(const Vec8* v, float& odd) {
    float m = 0.f;
#pragma unroll
    for (int u = 0; u < R; ++u) m = fmaxf(m, largest8(v[u]));
    odd = m;
    if (m == INFINITY) {  // rare: once more without them
        m = 0.f;
#pragma unroll
        for (int u = 0; u < R; ++u) {
            float y[8];
            Lane<D, INTER>::in_order(v[u], y);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (fabsf(y[j]) < INFINITY) m = fmaxf(m, fabsf(y[j]));
        }
    }
    return m;
}

// A lane's codes of v / scale.  The inverse of a power of two is exact, so the
// product is the quotient, and where the lane's largest magnitude `odd` is in
// reach of the format there is no more to it (`simple`); a caller's other scale
// divides, and what the format cannot hold is stored as NaN, so that it shows.
__device__ __forceinline__ bool simple_scale(float scale, float odd) {
    return (__float_as_uint(scale) & 0x7fffffu) == 0 && odd <= kMaxCode * scale;
}

template <int D, bool INTER>
__device__ __forceinline__ uint2 codes8(const Vec8& v, float scale, bool simple) {
    float y[8];
    if (simple) {
        Lane<D, INTER>::in_order(scale8(v, inverse_power(scale)), y);
    } else {
        Lane<D, INTER>::in_order(v, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            y[j] = __fdiv_rn(y[j], scale);
            if (!(fabsf(y[j]) <= kMaxCode)) y[j] = __int_as_float(0x7fffffff);
        }
    }
    return encode8(y);
}

// Codes under a scale 1 / `ratio` times the old one.
template <int D, bool INTER>
__device__ __forceinline__ uint2 rescaled(const uint2& codes, float ratio) {
    float y[8];
    decode8(codes, y);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] *= ratio;
    return encode8(y);
}

// A block's `rows` earlier tokens under it, by `slots` slots, of which this is
// number `slot`.
template <int D, bool INTER>
__device__ __forceinline__ void rescale_rows(uint8_t* dst, int rows, float ratio, int slot,
                                             int slots, const Lane<D, INTER>& lane) {
    for (int i = slot; i < rows; i += slots * kRows) {
        uint2 c[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u)
            if (i + u * slots < rows) c[u] = lane.load(dst + (i + u * slots) * D);
#pragma unroll
        for (int u = 0; u < kRows; ++u)
            if (i + u * slots < rows)
                lane.store(dst + (i + u * slots) * D, rescaled<D, INTER>(c[u], ratio));
    }
}

// A block with new tokens: where it is.
struct Block {
    int64_t slice0;            // page * heads
    int lo, first, last, row;  // positions; the row of `first`
    int at;                    // the block's first slot in its page
};

// 16 bytes from global into shared memory without a register; zeros where
// `take` is false.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(take ? 16 : 0)
                 : "memory");
}

// The CTA's slots times kRows are CH rows: a head's CH tokens at a time (larger
// blocks, MANY, in chunks), or the block's tokens of CH / block heads at once.  A
// thread's rows are of NH = kRows / UH heads, UH rows each, UH = block / slots;
// where a block has half as many tokens as there are slots (16 tokens of 64
// values), PARTS = 2: the first half of the warps and the second take heads of
// their own.  Row u is token tok + (u % UH) * slots of the chunk, of head
// h + part + (u / UH) * PARTS.
template <int D, bool INTER, int UH, int PARTS, bool MANY>
__device__ __forceinline__ void append_block(const Append& p, const Block& b, bool is_k,
                                             int h_begin, int h_end, uint4* ring) {
    constexpr int LPR = D / 8, SL = kThreads / LPR, CH = SL * kRows, NH = kRows / UH;
    constexpr int HEADS = NH * PARTS;  // at once
    __shared__ float red[2][NH][kWarps];
    const Lane<D, INTER> lane(p.t.half);
    const int my = threadIdx.x / LPR;
    const int part = PARTS > 1 ? my / (SL / PARTS) : 0, tok = PARTS > 1 ? my % (SL / PARTS) : my;
    const int rows = b.last - b.first, chunks = MANY ? (rows + CH - 1) / CH : 1;
    const bool norms = is_k && p.wk.w;
    Vec8 w = {};
    if (norms) w = lane.weights(p.wk);
    int pos[UH];  // of the thread's tokens
    // Where the thread's tokens of chunk c lie, and which of them there are: rows
    // behind the last are that one again, and are not stored.
    const int64_t sx = is_k ? p.sk : p.sv;
    const __nv_bfloat16* x0 = (is_k ? p.k : p.v) + b.row * sx;
    const __nv_bfloat16* src[UH];
    uint32_t there = 0;
    auto aim = [&](int c, int h) {
#pragma unroll
        for (int i = 0; i < UH; ++i)
            src[i] = x0 + min(c * CH + i * SL + tok, rows - 1) * sx + h * D;
    };
    auto place = [&](int c) {
        there = 0;
#pragma unroll
        for (int i = 0; i < UH; ++i) {
            if (c * CH + i * SL + tok < rows) there |= 1u << i;
            pos[i] = b.first + min(c * CH + i * SL + tok, rows - 1);
        }
    };
    // A ring of chunks on their way: a slot's rows are copied, and read, by its
    // own lanes, so that a warp waits for nothing but its own copies.
    int ask_h = h_begin, ask_c = 0, ask_at = 0, at = 0;
    uint4* const mine_in_ring = ring + threadIdx.x;
    auto ask = [&]() {
        if (ask_h < h_end) {
            uint4* dst = mine_in_ring + ask_at * (kRows * kThreads);
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const __nv_bfloat16* x = src[u % UH] + (u / UH) * PARTS * D + 8 * lane.chunk;
                const bool head = HEADS == 1 || ask_h + part + (u / UH) * PARTS < h_end;
                copy16(dst + u * kThreads, head ? x : p.k, head);
            }
            if (MANY) {  // a head's chunks up to the last one, and back to the first
                if (++ask_c == 2 * chunks - 1) {
                    ask_c = 0;
                    ask_h += HEADS;
                }
                aim(min(ask_c, 2 * chunks - 2 - ask_c), ask_h + part);
            } else {
                ask_h += HEADS;
#pragma unroll
                for (int i = 0; i < UH; ++i) src[i] += HEADS * D;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ask_at = ask_at + 1 == kStages ? 0 : ask_at + 1;
    };
    Vec8 v[kRows];
    auto turn = [&]() {  // v's rows normed and rotated
        if (norms) {
#pragma unroll
            for (int u = 0; u < kRows; ++u) v[u] = norm_row<D>(v[u], w, p.eps);
        }
        if (is_k && lane.turns) {
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                Rotation<D, INTER> rot;
                rot.load(p.t, pos[u % UH], lane);
                rot.turn(v[u]);
            }
        }
    };
    const uint4* const slot_in_ring = ring + my * LPR;
    auto take = [&]() {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncwarp();
        const uint4* stage = slot_in_ring + at * (kRows * kThreads);
        const __nv_bfloat16* lo = reinterpret_cast<const __nv_bfloat16*>(stage) + lane.lo;
        const __nv_bfloat16* hi = reinterpret_cast<const __nv_bfloat16*>(stage) + lane.hi;
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const uint2 l = *reinterpret_cast<const uint2*>(lo + u * (kThreads * 8));
            const uint2 h = *reinterpret_cast<const uint2*>(hi + u * (kThreads * 8));
            v[u] = lane.unpack(make_uint4(l.x, l.y, h.x, h.y));
        }
        at = at + 1 == kStages ? 0 : at + 1;
        turn();
        ask();  // into the stage read before this one
    };
    const int per_page = kPage >> p.block_log2;
    float* scale = (is_k ? p.ks : p.vs) + (b.slice0 + h_begin + part) * per_page +
                   (b.at >> p.block_log2);
    uint8_t* const codes = static_cast<uint8_t*>(is_k ? p.kp : p.vp);
    uint8_t* dst =
        codes + ((b.slice0 + h_begin + part) * kPage + b.at + (b.first - b.lo) + tok) * D;
    aim(0, h_begin + part);
    place(0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) ask();
    for (int h = h_begin; h < h_end; h += HEADS) {
        float was[NH], amax[NH], odd[NH];
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            const bool head = HEADS == 1 || h + part + n * PARTS < h_end;
            was[n] = b.first > b.lo && head ? scale[n * PARTS * per_page] : 0.f;
            amax[n] = odd[n] = 0.f;
        }
        for (int c = 0; c < chunks; ++c) {
            if (MANY) place(c);
            take();
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                float o;
                amax[n] = fmaxf(amax[n], finite_max<D, INTER, UH>(v + n * UH, o));
                odd[n] = fmaxf(odd[n], o);
            }
        }
        float(&mine)[NH][kWarps] = red[(h - h_begin) / HEADS & 1];  // two: one barrier will do
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            // (bits of non-negative floats are in their order)
            const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(amax[n]));
            if ((threadIdx.x & 31) == 0) mine[n][threadIdx.x >> 5] = __uint_as_float(top);
        }
        __syncthreads();  // every thread has read the old scales
        bool simple = true;
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            constexpr int warps = kWarps / PARTS;
            const bool head = HEADS == 1 || h + part + n * PARTS < h_end;
#pragma unroll
            for (int i = 0; i < warps; ++i) amax[n] = fmaxf(amax[n], mine[n][part * warps + i]);
            const float now = fmaxf(was[n], least_scale(amax[n]));
            if (head && tok == 0 && lane.chunk == 0) scale[n * PARTS * per_page] = now;
            amax[n] = now;  // the scale from here on
            simple = simple && simple_scale(now, odd[n]);
            if (b.first > b.lo && head && now != was[n])  // now is a power of two
                rescale_rows<D, INTER>(
                    codes + ((b.slice0 + h + part + n * PARTS) * kPage + b.at) * D,
                    b.first - b.lo, was[n] * inverse_power(now), tok, SL / PARTS, lane);
        }
        // the new tokens: the last chunk's values are still there
        for (int c = chunks - 1; c >= 0; --c) {
            if (MANY && c < chunks - 1) {
                place(c);
                take();
            }
            uint2 out[kRows];
            if (simple) {
#pragma unroll
                for (int u = 0; u < kRows; ++u) out[u] = codes8<D, INTER>(v[u], amax[u / UH], true);
            } else {
#pragma unroll
                for (int u = 0; u < kRows; ++u)
                    out[u] = codes8<D, INTER>(v[u], amax[u / UH],
                                              simple_scale(amax[u / UH], odd[u / UH]));
            }
            uint8_t *lo = dst + c * CH * D + lane.lo, *hi = dst + c * CH * D + lane.hi;
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                constexpr int kHead = PARTS * kPage * D;
                const int off = (u % UH) * SL * D + (u / UH) * kHead;
                if ((there >> (u % UH) & 1) &&
                    (HEADS == 1 || h + part + (u / UH) * PARTS < h_end)) {
                    if (INTER) {
                        *reinterpret_cast<uint2*>(lo + off) = out[u];
                    } else {
                        *reinterpret_cast<uint32_t*>(lo + off) = out[u].x;
                        *reinterpret_cast<uint32_t*>(hi + off) = out[u].y;
                    }
                }
            }
        }
        scale += HEADS * per_page;
        dst += HEADS * kPage * D;
    }
}

// A block where sequences have a few new tokens each, as in a decode step: each
// slot takes one head of K or of V (pairs pair_begin .. pair_end - 1, the keys
// first), R tokens at a time, and finds its scale alone; where scales grow,
// the CTA rounds the earlier tokens of those heads together.  A step of 64 tokens
// with 32 + 2 * 8 heads takes 4.5 to 5.1 us, into bf16 pages 4.5.  (A longer prompt
// among so many single tokens that their mean is small goes R rows at a time through
// one CTA for each of its blocks and heads: 190 tokens beside 63 single ones 60 us in
// blocks of 64, 150 in blocks of 256.)
template <int D, bool INTER, int R>
__device__ __forceinline__ void append_few(const Append& p, const Seq& s, Block b, int pair_begin,
                                           int pair_end) {
    constexpr int LPR = D / 8, SL = kThreads / LPR;
    __shared__ float ratio[SL];  // of each slot's head; 0: nothing to round again
    const Lane<D, INTER> lane(p.t.half);
    const int my = threadIdx.x / LPR;
    const int rows = b.last - b.first, chunks = (rows + R - 1) / R;
    const int per_page = kPage >> p.block_log2;
    Vec8 w = {};
    if (p.wk.w) w = lane.weights(p.wk);
    // the first rows and positions, on their way while the page is looked up
    auto rows_at = [&](int pair) {
        return (pair < p.Hk ? p.k + b.row * p.sk + pair * D
                            : p.v + b.row * p.sv + (pair - p.Hk) * D);
    };
    uint4 raw[R];
    Rotation<D, INTER> rot[R];
    auto fetch = [&](int pair, int c) {
        const __nv_bfloat16* x = rows_at(pair);
        const int64_t sx = pair < p.Hk ? p.sk : p.sv;
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const int r = c * R + u;
            raw[u] = make_uint4(0, 0, 0, 0);
            if (r < rows) {
                raw[u] = lane.load(x + r * sx);
                rot[u].load(p.t, b.first + r, lane);
            }
        }
    };
    fetch(min(pair_begin + my, pair_end - 1), 0);
    const int page = page_at(p, s, b.lo, threadIdx.x == 0);
    if (page < 0) return;
    b.slice0 = static_cast<int64_t>(page) * p.Hk;
    for (int base = pair_begin; base < pair_end; base += SL) {
        const bool live = base + my < pair_end;
        const int pair = live ? base + my : pair_end - 1;
        const bool is_k = pair < p.Hk;
        const int h = is_k ? pair : pair - p.Hk;
        float* scale = (is_k ? p.ks : p.vs) + (b.slice0 + h) * per_page + (b.at >> p.block_log2);
        float was = 0.f;
        if (b.first > b.lo && lane.chunk == 0) was = *scale;
        was = __shfl_sync(0xffffffffu, was, threadIdx.x & 31 & ~(LPR - 1));
        Vec8 v[R];
        auto take = [&](int c) {
            if (c > 0 || base > pair_begin) fetch(pair, c);
#pragma unroll
            for (int u = 0; u < R; ++u) {
                v[u] = lane.unpack(raw[u]);
                if (p.wk.w) {  // a warp's slots may be of keys and of values
                    const Vec8 n = norm_row<D>(v[u], w, p.eps);
                    if (is_k) v[u] = n;
                }
                if (is_k && c * R + u < rows) rot[u].apply(v[u]);
            }
        };
        float amax = 0.f, odd = 0.f;
        for (int c = 0; c < chunks; ++c) {
            take(c);
            float o;
            amax = fmaxf(amax, finite_max<D, INTER, R>(v, o));
            odd = fmaxf(odd, o);
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float now = fmaxf(was, least_scale(amax));
        uint8_t* dst = static_cast<uint8_t*>(is_k ? p.kp : p.vp) +
                       ((b.slice0 + h) * kPage + b.at) * D;
        if (live && lane.chunk == 0) *scale = now;
        for (int c = chunks - 1; c >= 0; --c) {
            if (c < chunks - 1) {
                if (c == 0 && base == pair_begin) fetch(pair, c);  // (take has the others)
                take(c);
            }
#pragma unroll
            for (int u = 0; u < R; ++u) {
                const int r = c * R + u;
                if (live && r < rows)
                    lane.store(dst + (b.first - b.lo + r) * D,
                               codes8<D, INTER>(v[u], now, simple_scale(now, odd)));
            }
        }
        if (b.first == b.lo) continue;  // the same for the CTA
        const bool grows = live && now != was;
        if (lane.chunk == 0) ratio[my] = grows ? was * inverse_power(now) : 0.f;
        if (!__syncthreads_or(grows)) continue;
        // rows of all the slots' heads, kFew of them in flight for each slot
        constexpr int kFew = 8;
        const int old = b.first - b.lo, all = min(SL, pair_end - base) * old;
        for (int i = my; i < all; i += SL * kFew) {
            uint8_t* row[kFew];
            uint2 c[kFew];
            float f[kFew];
#pragma unroll
            for (int u = 0; u < kFew; ++u) {
                const int at = i + u * SL, slot = at / old;
                f[u] = at < all ? ratio[slot] : 0.f;
                if (f[u] == 0.f) continue;
                const int pr = base + slot, hh = pr < p.Hk ? pr : pr - p.Hk;
                row[u] = static_cast<uint8_t*>(pr < p.Hk ? p.kp : p.vp) +
                         ((b.slice0 + hh) * kPage + b.at + at - slot * old) * D;
                c[u] = lane.load(row[u]);
            }
#pragma unroll
            for (int u = 0; u < kFew; ++u)
                if (f[u] != 0.f) lane.store(row[u], rescaled<D, INTER>(c[u], f[u]));
        }
        __syncthreads();
    }
}

// The block of unit `unit` (without its page); false: none that can be taken.
__device__ __forceinline__ bool find_block(const Append& p, int unit, Shared& sh, Seq& s,
                                           Block& b) {
    int blk = 0;
    if (!find_unit(p, unit, sh, s, blk)) return false;
    const int start = s.len - s.n;
    b.lo = blk << p.block_log2;
    b.first = max(b.lo, start);
    b.last = b.lo + min(1 << p.block_log2, s.len - b.lo);  // (lo + a block may pass 2^31)
    b.row = s.row0 + (b.first - start);
    b.at = b.lo % kPage;
    return true;
}

// unit_ctas CTAs take units: for each unit as many as cover the heads of K and then
// those of V, unit_heads each (FEW: the heads of both together).  The others take
// the queries' rows: after them, as the lighter work, or (FEW, where all run at
// once) before them, as the longer one.
template <int D, bool INTER, bool FEW>
__global__ void __launch_bounds__(kThreads, 2)
    fa_append_fp8_kernel(const __grid_constant__ Append p) {
    __shared__ Shared sh;
    extern __shared__ uint4 ring[];
    const int block = blockIdx.x, row_ctas = gridDim.x - p.unit_ctas;
    const int cta = FEW ? block - row_ctas : block;
    if (FEW ? cta < 0 : cta >= p.unit_ctas) {
        append_rows<D, INTER, false>(p, FEW ? block : cta - p.unit_ctas, sh);
        return;
    }
    const int hgroups = (p.Hk + p.unit_heads - 1) / p.unit_heads;
    const int per_unit = FEW ? (2 * p.Hk + p.unit_heads - 1) / p.unit_heads : 2 * hgroups;
    const int unit = cta / per_unit, sub = cta - unit * per_unit;
    Seq s;
    Block b;
    if (!find_block(p, unit, sh, s, b)) return;
    if constexpr (FEW) {
        const int first = sub * p.unit_heads;
        const int end = min(first + p.unit_heads, 2 * p.Hk);
        if (b.last - b.first == 1) append_few<D, INTER, 1>(p, s, b, first, end);
        else append_few<D, INTER, kRows>(p, s, b, first, end);
    } else {
        const int page = page_at(p, s, b.lo, threadIdx.x == 0);
        if (page < 0) return;
        b.slice0 = static_cast<int64_t>(page) * p.Hk;
        const bool is_k = sub < hgroups;
        const int first = (is_k ? sub : sub - hgroups) * p.unit_heads;
        const int end = min(first + p.unit_heads, p.Hk);
        constexpr int SL = kThreads / (D / 8);
        const int width = 1 << p.block_log2;
        auto run = [&](auto uh, auto parts, auto many) {
            append_block<D, INTER, decltype(uh)::value, decltype(parts)::value,
                         decltype(many)::value>(p, b, is_k, first, end, ring);
        };
        using std::integral_constant;
        if (D == 64 && width < SL)
            run(integral_constant<int, 1>{}, integral_constant<int, D == 64 ? 2 : 1>{},
                std::false_type{});
        else if (width == SL)
            run(integral_constant<int, 1>{}, integral_constant<int, 1>{}, std::false_type{});
        else if (width == 2 * SL)
            run(integral_constant<int, 2>{}, integral_constant<int, 1>{}, std::false_type{});
        else if (width == 4 * SL)
            run(integral_constant<int, 4>{}, integral_constant<int, 1>{}, std::false_type{});
        else
            run(integral_constant<int, 4>{}, integral_constant<int, 1>{}, std::true_type{});
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

// Tokens of a CTA that takes rows: at most kTokens, and fewer where that would
// leave SMs without one.
int tokens_of(int total, int num_sms) {
    const int t = total / (num_sms * 4);
    return t < 1 ? 1 : t > kTokens ? kTokens : t;
}

template <int D, bool INTER>
int launch_rope(const Append& p, cudaStream_t st) {
    fa_append_rope_kernel<D, INTER>
        <<<(p.total + p.tokens - 1) / p.tokens, kThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D, bool INTER>
int launch_fp8(Append& p, int num_sms, cudaStream_t st) {
    // Sequences with a few tokens each: a slot takes a head, and a unit's heads go
    // to as many CTAs as make two an SM, the rows' CTAs among them (a step of 64
    // tokens 4.5 us, with one CTA more an SM 6.2).  Else up to 16 heads of a
    // unit one after the other, and fewer where SMs would be short of CTAs.
    const int row_ctas = p.q ? (p.total + p.tokens - 1) / p.tokens : 0;
    const bool few = p.total <= static_cast<int64_t>(p.B) * kRows;
    int64_t each;
    if (few) {
        const int per_unit = std::max(1, std::max(num_sms, 2 * num_sms - row_ctas) / p.units);
        each = std::max(1, (2 * p.Hk + per_unit - 1) / per_unit);
    } else {
        // (a CTA takes 64 rows of 128 values, or 128 of 64, at once)
        const int at_once = std::max(1, kThreads * kRows * 8 / D >> p.block_log2);
        each = static_cast<int64_t>(p.units) * 2 * p.Hk / (num_sms * 3);
        each = std::min<int64_t>(std::max<int64_t>(each, 1), 16);
        each = std::min<int64_t>((each + at_once - 1) / at_once * at_once, p.Hk);
    }
    p.unit_heads = static_cast<int>(each);
    p.unit_ctas = p.units * static_cast<int>(few ? (2 * p.Hk + each - 1) / each
                                                 : 2 * ((p.Hk + each - 1) / each));
    const int ctas = p.unit_ctas + row_ctas;
    if (few) {
        fa_append_fp8_kernel<D, INTER, true><<<ctas, kThreads, 0, st>>>(p);
    } else {
        auto kernel = fa_append_fp8_kernel<D, INTER, false>;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing) !=
            cudaSuccess)
            return FA_ERR_CUDA;
        kernel<<<ctas, kThreads, kRing, st>>>(p);
    }
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
    p.tokens = fa::tokens_of(total_new, num_sms);
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
    p.tokens = fa::tokens_of(total_new, num_sms);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d == 64)
        return interleaved ? fa::launch_fp8<64, true>(p, num_sms, st)
                           : fa::launch_fp8<64, false>(p, num_sms, st);
    return interleaved ? fa::launch_fp8<128, true>(p, num_sms, st)
                       : fa::launch_fp8<128, false>(p, num_sms, st);
}

}  // extern "C"
