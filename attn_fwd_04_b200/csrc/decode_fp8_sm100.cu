// decode_fp8_sm100.cu -- single-token decode over a paged cache of 8-bit
// values (e4m3) with one scale for each block of tokens and head.
//
// The cache is the page pool of the page "“Flash”不是那个被时代淘汰的插件"
// (0539edu.com), section 2, which notes that decode is bound by memory
// traffic: at 8 bits there is half of it, and twice the arithmetic for each
// byte.  For one sequence and K/V head, with the G query heads that share it,
//     s[g, l] = scale * q[g] . kcode[l] * kscale(l),   p = 2^(s log2 e - m),
//     o[g] = sum_l p[g, l] vscale(l) vcode[l] / sum_l p[g, l],
// the running maximum m as in the page "Flash Attention 是什么", section
// 关键术语解析, item 4.
//
// Two launches: split and merge.  The tokens of all sequences and K/V heads
// form one stream of tiles of 32 tokens (64 at d = 64), and each warp of a grid that fills the
// GPU takes an equal, contiguous piece of it, whatever the lengths.  A warp
// that holds all of a sequence's head writes the output; pieces of one that is
// cut are written as normalised partial outputs with their log-sum-exp, which
// the second launch joins.  There is no plan kernel: each warp (each CTA, where
// there are many sequences) sums the lengths itself while it starts.
//
// With up to 8 query heads a K/V head nothing goes through shared memory but the
// query (with more, tiles do: below).  The matrix
// instruction's first operand is the cache: S^T[tokens, heads] = K Q^T and
// O^T[d, heads] += V^T P^T, m16n8k16 in fp16 with fp32 sums, to which the
// conversion from e4m3 is exact.  The order of d in the first product and of d
// in the rows of the second is free, and is chosen so that each lane's share
// of a fragment is 16 consecutive bytes of a token: K and V go from global
// memory to registers in whole 128-byte rows, 8 KB a warp in flight, and only
// V's bytes are paired across two tokens (a byte permute).  S^T's accumulators
// are P^T's operand after one 8 x 8 transpose in registers.  8 query heads
// fill an instruction's 8 columns; up to 24 take two or three of them, more are
// split into groups, a warp each, over the same tokens.
// (With the heads in the 16 rows instead, 8 heads would leave half of every
// instruction and half of the accumulators empty.)
//
// 64 sequences of 1K to 32K tokens, 8 K/V heads and 32 query heads: 354 us, 6.4
// TB/s, 0.98 of a copy, every byte read once; with 32 K/V heads and up to 16K tokens
// 718 us, 6.5 TB/s.  Run on end for seconds the board's 1000 W bound it instead: 385
// and 776 us at 1.6 GHz.  The scheduler is 40 % busy, the tensor pipe 28 %.  A stream of
// few tiles is bound by latency: 14 us for 8 x 2048 tokens, of which a copy would
// take 5.
//
// Rounding: each query row is scaled by a power of two into fp16, which holds
// its 8 bits exactly down to 2^-31 of the row's largest; scores, maxima and sums
// are fp32.  Weights p * vscale are held relative to the largest of them so far, for
// each query head: the running maximum m is that of the scores with log2 vscale
// added, so that a block of large values that the softmax hardly sees does not
// push the others out of fp16's range, whatever the scales.  A weight is the sum of
// two fp16 values (22 bits, or 2^-40 of the largest), each with a product of its own:
// with one alone an output differed by 1e-3 of its size from that of fp32 weights, now
// by 2e-4, which is what bf16 makes of fp32 sums in another order.  It costs 2 % of the
// time above, and 14 to 36 % where more than 8 query heads share a K/V head (below).
#include <algorithm>
#include <cmath>

#include "fa_internal.h"
#include "rope_row.cuh"

namespace fa {
namespace {

constexpr int kPage = 256;
// Tokens a step of a warp: 8 KB of keys and values.
constexpr int tile_tokens(int d) { return d == 64 ? 64 : 32; }
constexpr int kWarps = 4;  // a CTA
constexpr int kThreads = kWarps * 32;
constexpr int kWarpSeqs = 128;  // sequences that a warp looks through by itself, at most

struct DecodeFp8 {
    const __nv_bfloat16* q;
    const uint8_t *kp, *vp;
    const float *ks, *vs;
    const int32_t *table, *lens;
    __nv_bfloat16* o;
    float* lse;
    float *part_o, *part_lse;  // [2 * warps, 8 * NT (, D)] pieces
    int64_t* seqs;             // [1 + B, 2]: the stream's tiles; for each sequence the
                               // tiles before it and its length (B > kWarpSeqs)
    int B, H, Hk, G, num_pages, table_len, max_pages, block_log2;
    int groups, group_heads;  // groups of query heads of one K/V head
    int ranges;               // warps of each group: the stream's ranges, at most
    int cluster;              // CTAs of a sequence's head, where it has CTAs of its own
    float scale_log2;
    unsigned int* err;
};

// ---- the stream of tiles ------------------------------------------------------
// Sequence b's cached tokens as its length and its table's entries give them,
// the first entry at `base` (lengths may be anything: 64-bit sums).
__device__ __forceinline__ int usable_len(const DecodeFp8& p, int len, int64_t base, bool& bad) {
    bad = len < 0;
    if (len <= 0) return 0;
    const int64_t room = p.max_pages ? p.max_pages : max(int64_t{0}, p.table_len - base);
    if (len > room * kPage) {
        bad = true;
        len = static_cast<int>(room * kPage);
    }
    return len;
}
__device__ __forceinline__ int pages_of(int len) {
    return len <= 0 ? 0 : len / kPage + (len % kPage != 0);
}
template <int TILE>
__device__ __forceinline__ int tiles_of(int len) {
    return len / TILE + (len % TILE != 0);
}

// A sequence's table base, usable length and the tiles before it.
struct Slice {
    int64_t base, tiles_before;
    int len;
};

// Inclusive prefix over a warp's lanes.
__device__ __forceinline__ int64_t warp_prefix(int64_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t n = __shfl_up_sync(0xffffffffu, v, o);
        if ((threadIdx.x & 31) >= o) v += n;
    }
    return v;
}

// Sequences first .. first + 31, one a lane, with the pages and tiles before them:
// up to kWarpSeqs are looked at by every warp for itself, without a barrier
// between a short batch's lengths and its first loads.
template <int TILE>
__device__ __forceinline__ Slice scan_lanes(const DecodeFp8& p, int first, int64_t& pages,
                                            int64_t& tiles) {
    const int i = first + (threadIdx.x & 31);
    const int len = i < p.B ? __ldg(p.lens + i) : 0;
    Slice s;
    s.base = static_cast<int64_t>(i) * p.max_pages;
    if (p.max_pages == 0) {
        const int64_t upto = pages + warp_prefix(pages_of(len));
        s.base = upto - pages_of(len);
        pages = __shfl_sync(0xffffffffu, upto, 31);
    }
    bool bad;
    s.len = usable_len(p, len, s.base, bad);
    if (bad) record_error(p.err, FA_DEVERR_BAD_INPUT);
    const int64_t upto = tiles + warp_prefix(tiles_of<TILE>(s.len));
    s.tiles_before = upto - tiles_of<TILE>(s.len);
    tiles = __shfl_sync(0xffffffffu, upto, 31);
    return s;
}

// Lane `from`'s, in every lane.
__device__ __forceinline__ Slice of_lane(const Slice& s, int from) {
    return Slice{__shfl_sync(0xffffffffu, s.base, from),
                 __shfl_sync(0xffffffffu, s.tiles_before, from),
                 __shfl_sync(0xffffffffu, s.len, from)};
}

struct ScanShared {
    int64_t sum[kWarps];
};

// Exclusive prefix over the block of one value a thread; `total` of the block.
__device__ __forceinline__ int64_t block_prefix(int64_t v, ScanShared& sh, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc = warp_prefix(v);
    if (lane == 31) sh.sum[warp] = inc;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) inc += sh.sum[w];
        total += sh.sum[w];
    }
    __syncthreads();
    return inc - v;
}

// More of them: sequences first .. first + kThreads - 1, one a thread, with the
// pages and tiles before them.
template <int TILE>
__device__ __forceinline__ Slice scan_chunk(const DecodeFp8& p, int first, int64_t& pages,
                                            int64_t& tiles, ScanShared& sh) {
    const int i = first + threadIdx.x;
    const int len = i < p.B ? __ldg(p.lens + i) : 0;
    Slice s;
    int64_t total = 0;
    if (p.max_pages) {
        s.base = static_cast<int64_t>(i) * p.max_pages;
    } else {
        s.base = pages + block_prefix(pages_of(len), sh, total);
        pages += total;
    }
    bool bad;
    s.len = usable_len(p, len, s.base, bad);
    if (bad) record_error(p.err, FA_DEVERR_BAD_INPUT);
    s.tiles_before = tiles + block_prefix(tiles_of<TILE>(s.len), sh, total);
    tiles += total;
    return s;
}

// a / b, by a 32-bit division where that will do (a short stream's latency).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// The stream is cut into as many ranges as there are warps, but no empty ones.
__device__ __forceinline__ int ranges_of(const DecodeFp8& p, int64_t T) {
    return static_cast<int>(min(static_cast<int64_t>(p.ranges), T));
}
// Range r of `ranges` equal ones of T tiles, and the range that holds tile t.
__device__ __forceinline__ int64_t range_start(int64_t r, int64_t T, int ranges) {
    return quotient(r * T, ranges);
}
__device__ __forceinline__ int64_t range_of(int64_t t, int64_t T, int ranges) {
    return quotient((t + 1) * ranges - 1, T);
}

// ---- fragments ------------------------------------------------------------------
__device__ __forceinline__ void cvt4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// (lo, hi) as the sum of two fp16 pairs.
__device__ __forceinline__ void split_f16x2(float lo, float hi, uint32_t& a, uint32_t& b) {
    a = pack_f16x2(lo, hi);
    float back_lo, back_hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(back_lo), "=f"(back_hi)
        : "r"(a));
    b = pack_f16x2(lo - back_lo, hi - back_hi);
}

// 2^x down to the least subnormal: where a weight below 2^-126 may meet a value that
// is larger than the others' by more than that.
__device__ __forceinline__ float ex2_gradual(float x) {
    const float y = ex2_approx(0.5f * x);
    return y * y;
}

__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Cache bytes are read once: kept out of L1, and in the order written here.
template <int N>
__device__ __forceinline__ void load_bytes(uint32_t (&r)[N], const uint8_t* p) {
    static_assert(N == 4 || N == 2, "16 or 8 bytes");
    if constexpr (N == 4)
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "l"(p));
    else
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                     : "=r"(r[0]), "=r"(r[1])
                     : "l"(p));
}

// Shared memory of a CTA of the cluster.
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

// Where a warp is in the stream.
struct Cursor {
    int b, hk, len, tile, tiles;
    int64_t base;   // of the sequence's table entries
    int64_t slice;  // (page, head) of the tile, in slices of kPage tokens
    int ahead;      // the next page's index
};

__device__ __forceinline__ int page_index(const DecodeFp8& p, const Cursor& c, int k) {
    int page = __ldg(p.table + c.base + k);
    if (page < 0 || page >= p.num_pages) {
        record_error(p.err, FA_DEVERR_BAD_INPUT);
        page = 0;
    }
    return page;
}

// The cursor's page, and the one after it (of the same sequence) on its way.
template <int TILE>
__device__ __forceinline__ void enter_head(const DecodeFp8& p, Cursor& c) {
    const int k = c.tile / (kPage / TILE);
    c.slice = static_cast<int64_t>(page_index(p, c, k)) * p.Hk + c.hk;
    c.ahead = k < (c.len - 1) / kPage ? page_index(p, c, k + 1) : 0;
}

// The next tile; PAGES: and its page.
template <int TILE, bool PAGES = true>
__device__ __forceinline__ void advance(const DecodeFp8& p, Cursor& c) {
    if (++c.tile < c.tiles) {
        if (PAGES && c.tile % (kPage / TILE) == 0) {
            c.slice = static_cast<int64_t>(c.ahead) * p.Hk + c.hk;
            const int k = c.tile / (kPage / TILE);
            c.ahead = k < (c.len - 1) / kPage ? page_index(p, c, k + 1) : 0;
        }
        return;
    }
    c.tile = 0;
    if (++c.hk == p.Hk) {
        c.hk = 0;
        do {  // the caller has tiles left, so there is such a sequence
            c.base = p.max_pages ? c.base + p.max_pages : c.base + pages_of(__ldg(p.lens + c.b));
            ++c.b;
            bool bad;
            c.len = usable_len(p, __ldg(p.lens + c.b), c.base, bad);
        } while (c.len == 0 && c.b + 1 < p.B);
        c.tiles = tiles_of<TILE>(c.len);
    }
    if (PAGES) enter_head<TILE>(p, c);
}

// ---- more than 8 query heads: tiles by way of shared memory --------------------------
// A warp's accumulators (16 registers for every 8 heads, at d = 128 32) then leave no
// room for a tile on its way, so each warp has a ring of two tiles of its own,
// filled by asynchronous copies of 16 bytes one tile ahead.  Where the pieces go is
// permuted within 128-byte lines so that the 8 lanes of a phase of a fragment's load
// find 8 different ones.  Up to 24 heads share a warp, and so one conversion of the
// tile's bytes.
//
// 64 sequences of 8K to 16K tokens, 4 K/V heads of 16 query heads: 169 us, 0.74 of a
// copy; of 24 229, of 32 (two groups of 16) 326: the products bound them, some 75 us
// for every 8 heads.  (With one product for the weights 148, 188, and 240 for 32 in one
// group.)
constexpr int kStages = 2;  // (three leave room for one CTA an SM only)
constexpr int stage_bytes(int d) { return 2 * tile_tokens(d) * d + 128; }  // K, V, scales
constexpr int ring_bytes(int d) { return kWarps * kStages * stage_bytes(d); }

template <int D>
__device__ __forceinline__ int k_place(int row, int u) {  // of 16-byte piece u of a row
    const int at = row * (D / 16) + u;
    return D == 128 ? at ^ ((row & 1) << 2) : at;
}
template <int D>
__device__ __forceinline__ int v_place(int row, int u) {
    return (row * (D / 16) + u) ^ ((row >> 1 & 3) << 1);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// CTAs of four warps an SM, by their registers.
constexpr int resident_ctas(int nt) { return nt == 1 ? 3 : 2; }

// SOLO > 0: short sequences, whose table rows hold a few pages.  A CTA of SOLO
// warps, or a cluster of such CTAs, takes all of a sequence's head, an equal part
// of its tiles a warp, joins the warps' results in shared memory and writes the
// output: one launch, and no length but its own sequence's (and those before it,
// in a packed table).
// RING: tiles by way of shared memory.
template <int D, int NT, int SOLO, bool RING>
__global__ void __launch_bounds__((SOLO ? SOLO : kWarps) * 32,
                                  SOLO == 8 ? 1 : resident_ctas(NT))
    fa_decode_fp8_split_kernel(const __grid_constant__ DecodeFp8 p) {
    constexpr int KJ = D / 64;   // 16-byte loads of a token's K for each lane
    constexpr int VW = D / 32;   // words of a token's V for each lane
    constexpr int MT = D / 16;   // 16-row tiles of O^T
    constexpr int TILE = tile_tokens(D), M = TILE / 16;
    extern __shared__ uint4 ring[];
    __shared__ ScanShared scan;
    __shared__ Slice found[kWarps];
    __shared__ int found_b[kWarps];
    __shared__ uint4 qs[SOLO ? 1 : kWarps][NT][2 * KJ][32];  // query fragments, a lane's own
    __shared__ float acc_sh[SOLO ? SOLO : 1][SOLO ? 8 * NT : 1][D];  // the warps' results
    __shared__ float lse_sh[SOLO ? SOLO : 1][8 * NT], cta_lse[SOLO ? 8 * NT : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    Cursor c;
    int group, wid = 0;
    int64_t left;
    const int ctas = SOLO ? p.cluster : 1, rank = SOLO ? blockIdx.x % ctas : 0;
    if constexpr (SOLO > 0) {
        const int part = blockIdx.x / ctas, head = part / p.groups;
        group = part - head * p.groups;
        c.b = head / p.Hk;
        c.hk = head - c.b * p.Hk;
        c.base = static_cast<int64_t>(c.b) * p.max_pages;
        if (p.max_pages == 0) {
            int64_t before = 0;
            for (int i = lane; i < c.b; i += 32) before += pages_of(__ldg(p.lens + i));
            c.base = __shfl_sync(0xffffffffu, warp_prefix(before), 31);
        }
        bool bad;
        c.len = usable_len(p, __ldg(p.lens + c.b), c.base, bad);
        if (bad && threadIdx.x == 0) record_error(p.err, FA_DEVERR_BAD_INPUT);
        c.tiles = tiles_of<TILE>(c.len);
        const int w = rank * SOLO + warp;
        c.tile = w * c.tiles / (SOLO * ctas);
        left = (w + 1) * c.tiles / (SOLO * ctas) - c.tile;
        if (left > 0) enter_head<TILE>(p, c);
    } else {
    asm volatile("griddepcontrol.launch_dependents;");
    // consecutive ranges on different CTAs, so that a few spread over the SMs
    wid = warp * gridDim.x + blockIdx.x;
    const int r = wid / p.groups;
    group = wid - r * p.groups;
    int64_t T, start;
    int ranges;
    Slice mine;  // the sequence in which this warp's range begins
    if (p.B <= kWarpSeqs) {
        int64_t pages = 0, tiles = 0;
        mine = scan_lanes<TILE>(p, 0, pages, tiles);
        for (int first = 32; first < p.B; first += 32) scan_lanes<TILE>(p, first, pages, tiles);
        T = tiles * p.Hk;
        ranges = ranges_of(p, T);
        if (r >= ranges) return;
        start = range_start(r, T, ranges);
        pages = tiles = 0;
        for (int first = 0;; first += 32) {  // some sequence holds tile `start`
            if (p.B > 32) mine = scan_lanes<TILE>(p, first, pages, tiles);
            const uint32_t here = __ballot_sync(
                0xffffffffu, start >= mine.tiles_before * p.Hk &&
                                 start < (mine.tiles_before + tiles_of<TILE>(mine.len)) * p.Hk);
            if (here == 0 && first + 32 < p.B) continue;
            c.b = first + __ffs(here) - 1;
            mine = of_lane(mine, c.b - first);
            break;
        }
    } else {
        int64_t pages = 0, tiles = 0;
        Slice s = scan_chunk<TILE>(p, 0, pages, tiles, scan);
        for (int first = kThreads; first < p.B; first += kThreads)
            scan_chunk<TILE>(p, first, pages, tiles, scan);
        T = tiles * p.Hk;
        ranges = ranges_of(p, T);
        if (blockIdx.x == 0 && threadIdx.x == 0) p.seqs[0] = tiles;
        pages = tiles = 0;
        for (int first = 0; first < p.B; first += kThreads) {
            s = scan_chunk<TILE>(p, first, pages, tiles, scan);
            const int i = first + threadIdx.x;
            if (blockIdx.x == 0 && i < p.B) {  // for the merge
                p.seqs[2 + 2 * static_cast<int64_t>(i)] = s.tiles_before;
                p.seqs[3 + 2 * static_cast<int64_t>(i)] = s.len;
            }
            if (T == 0) continue;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const int64_t at =
                    range_start((w * gridDim.x + blockIdx.x) / p.groups, T, ranges);
                if (at >= s.tiles_before * p.Hk &&
                    at < (s.tiles_before + tiles_of<TILE>(s.len)) * p.Hk) {
                    found[w] = s;
                    found_b[w] = first + threadIdx.x;
                }
            }
        }
        __syncthreads();
        if (r >= ranges) return;
        start = range_start(r, T, ranges);
        mine = found[warp];
        c.b = found_b[warp];
    }
    left = range_start(r + 1, T, ranges) - start;
    c.len = mine.len;
    c.base = mine.base;
    c.tiles = tiles_of<TILE>(c.len);
    const int64_t in_seq = start - mine.tiles_before * p.Hk;
    c.hk = static_cast<int>(quotient(in_seq, c.tiles));
    c.tile = static_cast<int>(in_seq - static_cast<int64_t>(c.hk) * c.tiles);
    enter_head<TILE>(p, c);
    }

    const int heads = min(p.group_heads, p.G - group * p.group_heads);  // of this group
    const int nb_log2 = 8 - p.block_log2;  // blocks of a page
    uint32_t kr[M][2][RING ? 1 : KJ][4], vr[RING ? 1 : M][4][VW];  // (a ring's part by part)
    float ks[M], vs[M];
    auto load_k = [&](const Cursor& x) {
        const int slot0 = (x.tile * TILE) % kPage, last = slot0 + x.len - 1 - x.tile * TILE;
        const uint8_t* base = p.kp + x.slice * (kPage * D) + 16 * t;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            // (both scales: the softmax wants V's with the scores)
            const int64_t scale =
                (x.slice << nb_log2) + (min(slot0 + 16 * m, last) >> p.block_log2);
            ks[m] = __ldg(p.ks + scale);
            vs[m] = __ldg(p.vs + scale);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // behind the last token: that token again
                const uint8_t* row = base + min(slot0 + 16 * m + 8 * h + g, last) * D;
#pragma unroll
                for (int j = 0; j < KJ; ++j) load_bytes(kr[m][h][RING ? 0 : j], row + 64 * j);
            }
        }
    };
    auto load_v = [&](const Cursor& x) {
        const int slot0 = (x.tile * TILE) % kPage, last = slot0 + x.len - 1 - x.tile * TILE;
        const uint8_t* base = p.vp + x.slice * (kPage * D) + D / 8 * g;
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                load_bytes(vr[RING ? 0 : m][i],
                           base + min(slot0 + 16 * m + 2 * t + (i & 1) + 8 * (i >> 1), last) * D);
    };

    // the same by way of the ring: tiles asked for, and taken, in turn
    const uint32_t stages = smem_u32(ring) + warp * (kStages * stage_bytes(D));
    Cursor asked = c;
    int64_t to_ask = left;
    int ask_at = 0, at = 0;
    auto ask = [&]() {
        if (to_ask > 0) {
            const int slot0 = (asked.tile * TILE) % kPage;
            const int last = slot0 + asked.len - 1 - asked.tile * TILE;
            const uint32_t dst = stages + ask_at * stage_bytes(D);
            const uint8_t* kb = p.kp + asked.slice * (kPage * D);
            const uint8_t* vb = p.vp + asked.slice * (kPage * D);
#pragma unroll
            for (int i = 0; i < TILE * D / 16 / 32; ++i) {
                const int piece = i * 32 + lane, row = piece / (D / 16), u = piece % (D / 16);
                const int off = min(slot0 + row, last) * D + 16 * u;
                copy16(dst + 16 * k_place<D>(row, u), kb + off);
                copy16(dst + TILE * D + 16 * v_place<D>(row, u), vb + off);
            }
            if (lane < 2 * M) {
                const int m = lane % M;
                copy4(dst + 2 * TILE * D + 4 * lane,
                      (lane < M ? p.ks : p.vs) + (asked.slice << nb_log2) +
                          (min(slot0 + 16 * m, last) >> p.block_log2));
            }
            if (--to_ask > 0) advance<TILE>(p, asked);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ask_at ^= 1;
    };
    auto stage = [&]() {
        return reinterpret_cast<const uint8_t*>(ring) + (warp * kStages + at) * stage_bytes(D);
    };
    auto take_k = [&](int j) {  // the tokens' 64 values from 64 j on
        const uint4* base = reinterpret_cast<const uint4*>(stage());
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 x = base[k_place<D>(16 * m + 8 * h + g, t + 4 * j)];
                kr[m][h][0][0] = x.x;
                kr[m][h][0][1] = x.y;
                kr[m][h][0][2] = x.z;
                kr[m][h][0][3] = x.w;
            }
    };
    auto take_v = [&](int m) {  // of 16 tokens
        const uint8_t* base = stage() + TILE * D;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 16 * m + 2 * t + (i & 1) + 8 * (i >> 1);
            if constexpr (D == 128) {
                const uint4 x = reinterpret_cast<const uint4*>(base)[v_place<D>(row, g)];
                vr[0][i][0] = x.x;
                vr[0][i][1] = x.y;
                vr[0][i][2] = x.z;
                vr[0][i][3] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(
                    base + 16 * v_place<D>(row, g >> 1) + 8 * (g & 1));
                vr[0][i][0] = x.x;
                vr[0][i][1] = x.y;
            }
        }
    };

    float o[NT][MT][4], m_run[NT][2], l_run[NT][2], fac[NT][2];
    // A new head of a sequence: its queries as fragments, and an empty state.
    auto begin = [&](int b, int hk) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int hh = nt * 8 + g;
            const bool real = hh < heads;
            const __nv_bfloat16* row =
                p.q + (static_cast<int64_t>(b) * p.H + hk * p.G +
                       (real ? group * p.group_heads + hh : 0)) * D;
            float x[KJ][16], top = 0.f;
#pragma unroll
            for (int j = 0; j < KJ; ++j) {
                const uint4* src = reinterpret_cast<const uint4*>(row + 64 * j + 16 * t);
                float y[8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    unpack8(__ldg(src + h), y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[j][8 * h + i] = real ? y[i] : 0.f;
                        top = fmaxf(top, fabsf(x[j][8 * h + i]));
                    }
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // times 2^(14 - floor(log2 top)), no more than 2^126
            const uint32_t e = min(268u - (__float_as_uint(top) >> 23), 253u);
            const float up = __uint_as_float(e << 23);
            const float f = p.scale_log2 * __uint_as_float((254u - e) << 23);
            fac[nt][0] = __shfl_sync(0xffffffffu, f, 8 * t);
            fac[nt][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
            for (int j = 0; j < KJ && (SOLO == 0 || warp == 0); ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    qs[SOLO ? 0 : warp][nt][2 * j + h][lane] =
                        make_uint4(pack_f16x2(x[j][8 * h] * up, x[j][8 * h + 1] * up),
                                   pack_f16x2(x[j][8 * h + 2] * up, x[j][8 * h + 3] * up),
                                   pack_f16x2(x[j][8 * h + 4] * up, x[j][8 * h + 5] * up),
                                   pack_f16x2(x[j][8 * h + 6] * up, x[j][8 * h + 7] * up));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m_run[nt][i] = -INFINITY;
                l_run[nt][i] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][mt][i] = 0.f;
        }
    };

    if constexpr (RING) {
        ask();
    } else if (SOLO == 0 || left > 0) {
        load_k(c);
        load_v(c);
    }
    begin(c.b, c.hk);
    if (SOLO > 0) __syncthreads();
    bool whole = c.tile == 0, first_piece = true;
    while (SOLO == 0 || left > 0) {
        const int b = c.b, hk = c.hk, tok0 = c.tile * TILE, len = c.len;
        const bool seg_end = c.tile + 1 == c.tiles, more = left > 1;
        --left;
        if (more) advance<TILE, !RING>(p, c);
        if constexpr (RING) {
            // the tile's copies, by all lanes, are there; all are done with the one before
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();
            ask();
#pragma unroll
            for (int m = 0; m < M; ++m) {
                ks[m] = reinterpret_cast<const float*>(stage() + 2 * TILE * D)[m];
                vs[m] = reinterpret_cast<const float*>(stage() + 2 * TILE * D)[M + m];
            }
        }
        // ---- S^T = K Q^T -------------------------------------------------------
        float sc[NT][M][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[nt][m][i] = 0.f;
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            if (RING) take_k(j);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 qf[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) qf[nt] = qs[SOLO ? 0 : warp][nt][2 * j + h][lane];
#pragma unroll
                for (int s2 = 0; s2 < 2; ++s2) {
#pragma unroll
                    for (int m = 0; m < M; ++m) {
                        uint32_t a0, a1, a2, a3;
                        cvt4(kr[m][0][RING ? 0 : j][2 * h + s2], a0, a2);
                        cvt4(kr[m][1][RING ? 0 : j][2 * h + s2], a1, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16(sc[nt][m], a0, a1, a2, a3, s2 ? qf[nt].z : qf[nt].x,
                                    s2 ? qf[nt].w : qf[nt].y);
                    }
                }
            }
        }
        float k_scale[M], v_weight[M], v_log[M];
#pragma unroll
        for (int m = 0; m < M; ++m) {
            k_scale[m] = ks[m];
            v_weight[m] = vs[m] * 0x1p15f;
            v_log[m] = fmaxf(lg2_approx(vs[m]), -64.f);
        }
        if (!RING && more) load_k(c);
        // ---- softmax over the tile's tokens ---------------------------------------
        bool moved = false;
        float keep[NT][2];
        uint32_t pf[NT][M][2], pr[NT][M][2];  // weights, and what fp16 leaves of them
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // (in this order neither product leaves fp32 where the score does not)
                    sc[nt][m][i] = sc[nt][m][i] * k_scale[m] * fac[nt][i & 1];
                    if (tok0 + 16 * m + 8 * (i >> 1) + g >= len) sc[nt][m][i] = -INFINITY;
                }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float top = fmaxf(sc[nt][0][i], sc[nt][0][i + 2]) + v_log[0];
#pragma unroll
                for (int m = 1; m < M; ++m)
                    top = fmaxf(top, fmaxf(sc[nt][m][i], sc[nt][m][i + 2]) + v_log[m]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                const float m_new = fmaxf(m_run[nt][i], top);
                const float base = m_new == -INFINITY ? 0.f : m_new;
                keep[nt][i] = ex2_gradual(m_run[nt][i] - base);
                moved = moved || m_new != m_run[nt][i];
                m_run[nt][i] = m_new;
                float sum = 0.f;
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float& x = sc[nt][m][i + 2 * h];
                        x = ex2_approx(x - base);
                        sum += x;
                    }
                l_run[nt][i] = l_run[nt][i] * keep[nt][i] + sum;
            }
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a, b;
                    split_f16x2(sc[nt][m][2 * h] * v_weight[m],
                                sc[nt][m][2 * h + 1] * v_weight[m], a, b);
                    pf[nt][m][h] = transpose8x8(a);
                    pr[nt][m][h] = transpose8x8(b);
                }
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    o[nt][mt][0] *= keep[nt][0];
                    o[nt][mt][1] *= keep[nt][1];
                    o[nt][mt][2] *= keep[nt][0];
                    o[nt][mt][3] *= keep[nt][1];
                }
            }
        }
        // ---- O^T += V^T P^T ----------------------------------------------------------
#pragma unroll
        for (int m = 0; m < M; ++m) {
            if (RING) take_v(m);
            const int from = RING ? 0 : m;
#pragma unroll
            for (int w = 0; w < VW; ++w) {
#pragma unroll
                for (int hi = 0; hi < 2; ++hi) {
                    uint32_t a0, a1, a2, a3;
                    cvt4(__byte_perm(vr[from][0][w], vr[from][1][w], hi ? 0x7362 : 0x5140), a0, a1);
                    cvt4(__byte_perm(vr[from][2][w], vr[from][3][w], hi ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16(o[nt][2 * w + hi], a0, a1, a2, a3, pf[nt][m][0], pf[nt][m][1]);
                        mma_f16(o[nt][2 * w + hi], a0, a1, a2, a3, pr[nt][m][0], pr[nt][m][1]);
                    }
                }
            }
        }
        if (RING) at ^= 1;
        if (!RING && more) load_v(c);
        if (SOLO > 0 || (!seg_end && more)) continue;
        // ---- the end of a head, or of the warp's range ------------------------------
        whole = whole && seg_end;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float l = l_run[nt][i];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const int hh = nt * 8 + 2 * t + i;
                if (hh >= heads) continue;
                const float lse2 = m_run[nt][i] + log2f(l);
                const float inv = l == 0.f ? 0.f : 0x1p-15f / l;
                if (whole) {
                    const int64_t row =
                        static_cast<int64_t>(b) * p.H + hk * p.G + group * p.group_heads + hh;
                    if (p.lse && g == 0) p.lse[row] = lse2 * 0.69314718055994531f;
                    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D + D / 8 * g);
#pragma unroll
                    for (int mt = 0; mt < MT; mt += 4)
                        *reinterpret_cast<uint4*>(dst + mt) = make_uint4(
                            pack_bf16x2(o[nt][mt][i] * inv, o[nt][mt][i + 2] * inv),
                            pack_bf16x2(o[nt][mt + 1][i] * inv, o[nt][mt + 1][i + 2] * inv),
                            pack_bf16x2(o[nt][mt + 2][i] * inv, o[nt][mt + 2][i + 2] * inv),
                            pack_bf16x2(o[nt][mt + 3][i] * inv, o[nt][mt + 3][i + 2] * inv));
                } else {
                    const int64_t slot =
                        (2 * static_cast<int64_t>(wid) + !first_piece) * (8 * NT) + hh;
                    if (g == 0) p.part_lse[slot] = lse2;
                    float* dst = p.part_o + slot * D + D / 8 * g;
#pragma unroll
                    for (int mt = 0; mt < MT; mt += 2)
                        *reinterpret_cast<float4*>(dst + 2 * mt) =
                            make_float4(o[nt][mt][i] * inv, o[nt][mt][i + 2] * inv,
                                        o[nt][mt + 1][i] * inv, o[nt][mt + 1][i + 2] * inv);
                }
            }
        }
        if (!more) return;
        whole = true;
        first_piece = false;
        begin(c.b, c.hk);
    }
    if constexpr (SOLO > 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float l = l_run[nt][i];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const int hh = nt * 8 + 2 * t + i;
                const float inv = l == 0.f ? 0.f : 0x1p-15f / l;
                if (g == 0) lse_sh[warp][hh] = m_run[nt][i] + log2f(l);
                float* dst = &acc_sh[warp][hh][D / 8 * g];
#pragma unroll
                for (int mt = 0; mt < MT; mt += 2)
                    *reinterpret_cast<float4*>(dst + 2 * mt) =
                        make_float4(o[nt][mt][i] * inv, o[nt][mt][i + 2] * inv,
                                    o[nt][mt + 1][i] * inv, o[nt][mt + 1][i + 2] * inv);
            }
        }
        __syncthreads();
        // the warps' results joined, in place of the first warp's; with a cluster
        // the CTAs' after that, a part of the head by each
        struct Joined {
            float4 a;
            float lse2;
        };
        auto join = [&](int n, auto lse_of, auto value_of) {
            float top = -INFINITY, sum = 0.f;
            for (int w = 0; w < n; ++w) top = fmaxf(top, lse_of(w));
            const float base = top == -INFINITY ? 0.f : top;
            Joined j{make_float4(0.f, 0.f, 0.f, 0.f), 0.f};
            for (int w = 0; w < n; ++w) {
                const float f = ex2_gradual(lse_of(w) - base);
                const float4 x = value_of(w);
                sum += f;
                j.a.x = fmaf(f, x.x, j.a.x);
                j.a.y = fmaf(f, x.y, j.a.y);
                j.a.z = fmaf(f, x.z, j.a.z);
                j.a.w = fmaf(f, x.w, j.a.w);
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            j.a.x *= inv;
            j.a.y *= inv;
            j.a.z *= inv;
            j.a.w *= inv;
            j.lse2 = top + log2f(sum);
            return j;
        };
        auto write = [&](int hh, int d, const Joined& j) {
            const int64_t row =
                static_cast<int64_t>(c.b) * p.H + c.hk * p.G + group * p.group_heads + hh;
            *reinterpret_cast<uint2*>(p.o + row * D + d) =
                make_uint2(pack_bf16x2(j.a.x, j.a.y), pack_bf16x2(j.a.z, j.a.w));
            if (d == 0 && p.lse) p.lse[row] = j.lse2 * 0.69314718055994531f;
        };
        for (int at = threadIdx.x; at < heads * (D / 4); at += SOLO * 32) {
            const int hh = at / (D / 4), d = at % (D / 4) * 4;
            const Joined j = join(
                SOLO, [&](int w) { return lse_sh[w][hh]; },
                [&](int w) { return *reinterpret_cast<const float4*>(&acc_sh[w][hh][d]); });
            if (ctas == 1) {
                write(hh, d, j);
            } else {
                *reinterpret_cast<float4*>(&acc_sh[0][hh][d]) = j.a;
                if (d == 0) cta_lse[hh] = j.lse2;
            }
        }
        if (ctas > 1) {
            __syncwarp();
            cluster_sync_all();
            for (int at = rank * SOLO * 32 + threadIdx.x; at < heads * (D / 4);
                 at += ctas * SOLO * 32) {
                const int hh = at / (D / 4), d = at % (D / 4) * 4;
                write(hh, d,
                      join(
                          ctas,
                          [&](int w) {
                              return ld_cluster(mapa_rank(smem_u32(&cta_lse[hh]), w));
                          },
                          [&](int w) {
                              return ld_cluster4(mapa_rank(smem_u32(&acc_sh[0][hh][d]), w));
                          }));
            }
            __syncwarp();
            cluster_sync_all();  // the others may still read this CTA's
        }
    }
}

// The pieces of a (sequence, query head) that the ranges cut,
// o = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M); and what has no tokens.
// ROW warps take a row's pieces in turn, kBatch of them in flight with their
// sums, each warp with a running maximum of its own; the CTA's other warps take
// other rows.
constexpr int merge_warps(int row) { return row > 4 ? row : 4; }
template <int D, int ROW>
__global__ void __launch_bounds__(merge_warps(ROW) * 32)
    fa_decode_fp8_merge_kernel(const __grid_constant__ DecodeFp8 p, int slots) {
    constexpr int V = D / 32, kBatch = 8, kMergeWarps = merge_warps(ROW);
    constexpr int TILE = tile_tokens(D);
    static_assert(kMergeWarps == ROW || ROW == 1, "a row's warps are the CTA's, or one");
    __shared__ float acc_sh[ROW][D], top_sh[ROW], sum_sh[ROW];
    const int lane = threadIdx.x & 31;
    // (B * H is below 2^26)
    const uint32_t at = (blockIdx.x * kMergeWarps + (threadIdx.x >> 5)) / ROW;
    const int part = (threadIdx.x >> 5) % ROW;
    if (at >= static_cast<uint32_t>(p.B) * p.H) return;  // a whole row's warps
    const int b = static_cast<int>(at / static_cast<uint32_t>(p.H));
    const int h = static_cast<int>(at - static_cast<uint32_t>(b) * p.H);
    const int64_t row = at;
    int64_t T, before;
    int len;
    if (p.B <= kWarpSeqs) {
        int64_t pages = 0;
        T = 0;
        Slice mine{};
        for (int first = 0; first < p.B; first += 32) {
            const Slice s = of_lane(scan_lanes<TILE>(p, first, pages, T), b % 32);
            if (first == b / 32 * 32) mine = s;
        }
        before = mine.tiles_before;
        len = mine.len;
    } else {
        asm volatile("griddepcontrol.wait;" ::: "memory");  // the split kernel's
        T = p.seqs[0];
        before = p.seqs[2 + 2 * static_cast<int64_t>(b)];
        len = static_cast<int>(p.seqs[3 + 2 * static_cast<int64_t>(b)]);
    }
    const int n = tiles_of<TILE>(len);
    const int hk = h / p.G, hg = h - hk * p.G, group = hg / p.group_heads;
    const int hh = hg - group * p.group_heads;
    T *= p.Hk;
    const int64_t t0 = before * p.Hk + static_cast<int64_t>(hk) * n;
    const int ranges = ranges_of(p, T);
    int64_t r0 = 0, r1 = 0;
    bool from_start = true;
    if (n > 0) {
        r0 = range_of(t0, T, ranges);
        r1 = range_of(t0 + n - 1, T, ranges);
        from_start = range_start(r0, T, ranges) == t0;
    }
    // (what is above is of this call's inputs alone; nothing is written before this)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (n == 0) {
        if (part == 0) {
            for (int i = lane; i < D; i += 32) p.o[row * D + i] = __float2bfloat16(0.f);
            if (lane == 0 && p.lse) p.lse[row] = -INFINITY;
        }
        return;
    }
    if (r0 == r1) return;  // the warp wrote it
    const int pieces = static_cast<int>(r1 - r0) + 1;
    float top = -INFINITY, sum = 0.f, acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    for (int i0 = part; i0 < pieces; i0 += ROW * kBatch) {
        float lse[kBatch], x[kBatch][V];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = i0 + k * ROW;
            lse[k] = -INFINITY;
#pragma unroll
            for (int j = 0; j < V; ++j) x[k][j] = 0.f;
            if (i >= pieces) continue;
            const int64_t w = (r0 + i) * p.groups + group;
            const int64_t s = (2 * w + (i == 0 && !from_start)) * slots + hh;
            lse[k] = p.part_lse[s];
            const float* src = p.part_o + s * D + V * lane;
            if constexpr (V == 4) {
                const float4 y = *reinterpret_cast<const float4*>(src);
                x[k][0] = y.x;
                x[k][1] = y.y;
                x[k][2] = y.z;
                x[k][3] = y.w;
            } else {
                const float2 y = *reinterpret_cast<const float2*>(src);
                x[k][0] = y.x;
                x[k][1] = y.y;
            }
        }
        float m = top;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) m = fmaxf(m, lse[k]);
        const float base = m == -INFINITY ? 0.f : m, keep = ex2_gradual(top - base);
        top = m;
        sum *= keep;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] *= keep;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const float w = ex2_gradual(lse[k] - base);
            sum += w;
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] = fmaf(w, x[k][j], acc[j]);
        }
    }
    if constexpr (ROW > 1) {
#pragma unroll
        for (int j = 0; j < V; ++j) acc_sh[part][V * lane + j] = acc[j];
        if (lane == 0) {
            top_sh[part] = top;
            sum_sh[part] = sum;
        }
        __syncthreads();
        if (part > 0) return;
        top = top_sh[0];
#pragma unroll
        for (int w = 1; w < ROW; ++w) top = fmaxf(top, top_sh[w]);
        const float base = top == -INFINITY ? 0.f : top;
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = 0.f;
#pragma unroll
        for (int w = 0; w < ROW; ++w) {
            const float f = ex2_gradual(top_sh[w] - base);
            sum = fmaf(f, sum_sh[w], sum);
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] = fmaf(f, acc_sh[w][V * lane + j], acc[j]);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D) + lane * (V / 2);
#pragma unroll
    for (int j = 0; j < V; j += 2) dst[j / 2] = pack_bf16x2(acc[j] * inv, acc[j + 1] * inv);
    if (lane == 0 && p.lse) p.lse[row] = (top + log2f(sum)) * 0.69314718055994531f;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// How the query heads of a K/V head and the warps are cut: up to kMostHeads of them
// to a warp, kFewHeads where the stream is short or a sequence's head has CTAs of its
// own, and more warps are worth more than fewer products and conversions.
// (64 sequences of 8K to 16K tokens, 24 heads for each of 4 K/V heads 229 us in one
// group, 324 in two; 32 heads in one group of 32, whose registers spill, 310 and 102 for
// one K/V head, in two of 16 326 and 96.)
constexpr int kMostHeads = 24, kFewHeads = 16;
struct Shape {
    int groups, group_heads, nt, ctas, ranges;
    size_t seqs_bytes, lse_bytes, bytes;  // of the workspace: sequences, sums, pieces
};

// (most: query heads of a group)
Shape shape_of(int B, int H, int H_kv, int d, int num_sms, int most) {
    Shape s;
    const int G = H / H_kv;
    s.groups = (G + most - 1) / most;
    s.group_heads = (G + s.groups - 1) / s.groups;
    s.nt = (s.group_heads + 7) / 8;
    s.ctas = num_sms * resident_ctas(s.nt);
    const int min_ctas = (s.groups + kWarps - 1) / kWarps;
    if (s.ctas < min_ctas) s.ctas = min_ctas;  // a warp for each group
    s.ranges = s.ctas * kWarps / s.groups;
    const size_t rows = static_cast<size_t>(s.ctas) * kWarps * 2 * 8 * s.nt;
    s.lse_bytes = (rows * sizeof(float) + 255) & ~size_t{255};
    s.seqs_bytes = B > kWarpSeqs ? ((2 + 2 * static_cast<size_t>(B)) * 8 + 255) & ~size_t{255} : 0;
    s.bytes = s.seqs_bytes + s.lse_bytes + rows * d * sizeof(float);
    return s;
}

// Scratch of a call, whichever way it takes.
size_t scratch_bytes(int B, int H, int H_kv, int d, int num_sms) {
    return std::max(shape_of(B, H, H_kv, d, num_sms, kFewHeads).bytes,
                    shape_of(B, H, H_kv, d, num_sms, kMostHeads).bytes);
}

// Up to four tiles a warp, as far as the table tells (one sequence of 32K tokens with
// one K/V head of 48: 18 us in groups of 16 heads, 25 in groups of 24; 64 sequences of 2K
// to 4K tokens, seven tiles a warp, with one of 24 36 and 33).
bool is_short(const Shape& s, int B, int H_kv, int d, int max_pages, int table_len) {
    const int64_t entries = max_pages ? static_cast<int64_t>(B) * max_pages : table_len;
    return entries * (kPage / tile_tokens(d)) * H_kv <= 4 * static_cast<int64_t>(s.ranges);
}

// CTAs of its own for each sequence's head, where a table row holds a few pages (a
// packed table may hold them all for one sequence): up to 8 where each head can
// have an SM and more, up to 2 with a few heads an SM.  Against the even ranges, on
// the GPU alone: 16 sequences of 400 tokens, 8 K/V heads 7.5 us and 9.5, of 1600
// 15.5 and 15.5; 64 of 400 16.6 and 17.0, of 800 29.1 and 25.7; 64 with 32 K/V heads
// 48.5 and 41.8.  The launch saved is 2 us of the host's time besides.
bool is_solo(int64_t heads, int max_pages, int table_len, int num_sms) {
    const int pages = max_pages ? max_pages : table_len;
    return heads <= num_sms ? pages <= 8 : heads <= 4 * num_sms && pages <= 2;
}

template <int D>
int launch_solo(DecodeFp8& p, const Shape& s, int num_sms, cudaStream_t st) {
    const int heads = p.B * p.Hk * p.groups;
    const bool wide = s.nt == 1 && heads <= num_sms;
    // (clusters of 8 would not all find room at once: 16 of them took 12 us and not 9)
    p.cluster = 4;
    while (p.cluster > 1 && heads * p.cluster > num_sms) p.cluster /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(heads) * p.cluster);
    cfg.blockDim = dim3(wide ? 256 : 128);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(p.cluster);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.cluster > 1 ? 1 : 0;
    auto kernel = s.nt == 2 ? fa_decode_fp8_split_kernel<D, 2, 4, false>
                  : wide    ? fa_decode_fp8_split_kernel<D, 1, 8, false>
                            : fa_decode_fp8_split_kernel<D, 1, 4, false>;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D>
int launch(const DecodeFp8& p, const Shape& s, cudaStream_t st) {
    auto split = s.nt == 1   ? fa_decode_fp8_split_kernel<D, 1, 0, false>
                 : s.nt == 2 ? fa_decode_fp8_split_kernel<D, 2, 0, true>
                             : fa_decode_fp8_split_kernel<D, 3, 0, true>;
    const int ring = s.nt > 1 ? ring_bytes(D) : 0;
    if (ring && cudaFuncSetAttribute(split, cudaFuncAttributeMaxDynamicSharedMemorySize, ring) !=
                    cudaSuccess)
        return FA_ERR_CUDA;
    split<<<s.ctas, kThreads, ring, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    // Pieces of a head, at most on average: the ranges, or the tiles that the table
    // has room for.  Rows of a few pieces take a warp each (2048 rows of 4: 18.4 us
    // in all, with 4 warps a row 22.3), others 4 (1024 rows of 19: 22.2, with one
    // 26.0) or 16.
    const int64_t heads = static_cast<int64_t>(p.B) * p.Hk;
    const int64_t entries = p.max_pages ? static_cast<int64_t>(p.B) * p.max_pages : p.table_len;
    const int64_t pieces =
        std::min<int64_t>(p.ranges, entries * (kPage / tile_tokens(D)) * p.Hk) / heads + 1;
    const int each = pieces <= 8 ? 1 : pieces <= 48 ? 4 : 16;  // warps of a row
    const int64_t warps = static_cast<int64_t>(p.B) * p.H * each;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim =
        dim3(static_cast<unsigned>((warps + merge_warps(each) - 1) / merge_warps(each)));
    cfg.blockDim = dim3(merge_warps(each) * 32);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    auto merge = each == 1   ? fa_decode_fp8_merge_kernel<D, 1>
                 : each == 4 ? fa_decode_fp8_merge_kernel<D, 4>
                             : fa_decode_fp8_merge_kernel<D, 16>;
    return cudaLaunchKernelEx(&cfg, merge, p, 8 * s.nt) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

extern "C" {

int fa_decode_paged_fp8_workspace(int B, int H, int H_kv, int d, int* bytes) {
    if (!bytes) return FA_ERR_NULL;
    if (B < 1 || H < 1 || H_kv < 1 || H % H_kv != 0) return FA_ERR_SHAPE;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    unsigned int* err = nullptr;
    int num_sms = 0, rc;
    if ((rc = fa::device_error_word(&err, &num_sms)) != FA_OK) return rc;
    const size_t most = fa::scratch_bytes(B, H, H_kv, d, num_sms);
    if (most > 0x7fffffff) return FA_ERR_SHAPE;
    *bytes = static_cast<int>(most);
    return FA_OK;
}

int fa_decode_paged_fp8(const void* q, const void* k_pages, const void* v_pages,
                        const float* k_scales, const float* v_scales, int block,
                        const int32_t* page_table, int table_len, int max_pages,
                        const int32_t* seq_lens, void* o, float* lse, int B, int H, int H_kv,
                        int num_pages, int d, int page_size, float scale, void* workspace,
                        int workspace_bytes, fa_stream_t stream) {
    if (!q || !k_pages || !v_pages || !k_scales || !v_scales || !page_table || !seq_lens || !o)
        return FA_ERR_NULL;
    if (B < 1 || H < 1 || H_kv < 1 || H % H_kv != 0 || num_pages < 1 || table_len < 0 ||
        max_pages < 0 || workspace_bytes < 0)
        return FA_ERR_SHAPE;
    if (max_pages > 0 && (static_cast<int64_t>(B) * max_pages > table_len ||
                          static_cast<int64_t>(max_pages) * page_size > 0x7fffffff))
        return FA_ERR_SHAPE;
    if (static_cast<int64_t>(B) * H > 0x7fffffff / 64) return FA_ERR_SHAPE;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (page_size != fa::kPage) return FA_ERR_UNSUPPORTED;
    if (block < 16 || block > fa::kPage || (block & (block - 1)) != 0) return FA_ERR_UNSUPPORTED;
    if (!std::isfinite(scale)) return FA_ERR_SHAPE;
    const void* wide[] = {q, k_pages, v_pages, o, workspace};
    for (const void* w : wide)
        if (!fa::aligned16(w)) return FA_ERR_ALIGN;
    // read or written one by one
    if ((reinterpret_cast<uintptr_t>(k_scales) | reinterpret_cast<uintptr_t>(v_scales) |
         reinterpret_cast<uintptr_t>(lse)) & 3u)
        return FA_ERR_ALIGN;
    fa::DecodeFp8 p{};
    int num_sms = 0, rc;
    if ((rc = fa::device_error_word(&p.err, &num_sms)) != FA_OK) return rc;
    const fa::Shape few = fa::shape_of(B, H, H_kv, d, num_sms, fa::kFewHeads);
    const fa::Shape most = fa::shape_of(B, H, H_kv, d, num_sms, fa::kMostHeads);
    const bool solo = fa::is_solo(static_cast<int64_t>(B) * H_kv * few.groups, max_pages, table_len,
                                  num_sms);
    const fa::Shape& s =
        solo || fa::is_short(few, B, H_kv, d, max_pages, table_len) ? few : most;
    const size_t need = fa::scratch_bytes(B, H, H_kv, d, num_sms);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    fa::WorkspaceHold hold;
    if (!solo) {
        void* ws = nullptr;
        if ((rc = fa::call_workspace(workspace, workspace_bytes, need, st, &ws, &hold)) != FA_OK)
            return rc;
        p.seqs = static_cast<int64_t*>(ws);
        p.part_lse = reinterpret_cast<float*>(static_cast<char*>(ws) + s.seqs_bytes);
        p.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + s.seqs_bytes + s.lse_bytes);
    } else if (workspace && static_cast<size_t>(workspace_bytes) < need) {
        return FA_ERR_SHAPE;  // as for any other table
    }
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.kp = static_cast<const uint8_t*>(k_pages);
    p.vp = static_cast<const uint8_t*>(v_pages);
    p.ks = k_scales;
    p.vs = v_scales;
    p.table = page_table;
    p.lens = seq_lens;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.B = B;
    p.H = H;
    p.Hk = H_kv;
    p.G = H / H_kv;
    p.num_pages = num_pages;
    p.table_len = table_len;
    p.max_pages = max_pages;
    p.groups = s.groups;
    p.group_heads = s.group_heads;
    p.ranges = s.ranges;
    while ((1 << p.block_log2) < block) ++p.block_log2;
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    if (solo)
        return d == 64 ? fa::launch_solo<64>(p, s, num_sms, st)
                       : fa::launch_solo<128>(p, s, num_sms, st);
    return d == 64 ? fa::launch<64>(p, s, st) : fa::launch<128>(p, s, st);
}

}  // extern "C"
