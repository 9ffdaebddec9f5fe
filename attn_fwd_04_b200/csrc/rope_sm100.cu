// rope_sm100.cu -- rotary tables scaled for long contexts, and the per-head
// norms of queries and keys with the rotation in the same pass, forward and
// backward.
//
// The page "“Flash”不是那个被时代淘汰的插件" (0539edu.com), sections 2 and 3,
// keeps the rotation's sines and cosines in a precomputed table; so do these
// calls.  Everything here moves a few bytes for each operation, so all of it
// is written for memory: every row is read once and written once, in 16-byte
// pieces, several of them in flight for each thread.
#include <algorithm>
#include <cmath>

#include "fa_internal.h"
#include "rope_row.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kFwdHeads = 4;  // heads a slot takes
constexpr int kBwdHeads = 4;
constexpr int kFwdCtas = 32;  // CTAs per SM of the grids, at most
// The backward grid is what is resident: 3 CTAs of 80 registers an SM (figures at the
// kernel).
constexpr int kBwdCtas = 3;
constexpr double kTwoPi = 6.283185307179586476925286766559;

// ---------------------------------------------------------------------------
// tables: cos and sin of p * w_i, w_i handed over in turns (w_i / 2 pi) in
// fp64.  A thread takes one pair and a run of positions: one fp64 sine and
// cosine where the run begins (the angle of a far position is many turns:
// p * w_i is formed and reduced in fp64), and from there
//     (c, s) -> (c cos w - s sin w, s cos w + c sin w)
// in fp64, whose rounding over a run of 16 stays below 2^-47.  Two products and
// two multiply-adds a pair instead of a sine and a cosine: 131072 positions of
// 64 pairs in 11.9 us (5.6 TB/s written, which bounds it), where an fp32 sine
// and cosine of the reduced angle for each took 23.3; runs of 64 12.8 us.
// ---------------------------------------------------------------------------
struct Turns {
    double w[kRopeMaxPairs];
};

__global__ void __launch_bounds__(kThreads)
    fa_rope_table_kernel(float* __restrict__ cos_t, float* __restrict__ sin_t, int max_pos,
                         int half, int run, double mscale, const __grid_constant__ Turns turns) {
    const int64_t thread = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t first = thread / half * run;
    if (first >= max_pos) return;
    const int i = static_cast<int>(thread % half);
    const double w = turns.w[i];
    double at = static_cast<double>(first) * w, c, s, cw, sw;
    at -= rint(at);
    sincospi(2.0 * at, &s, &c);
    sincospi(2.0 * (w - rint(w)), &sw, &cw);
    c *= mscale;
    s *= mscale;
    const int n = static_cast<int>(min(static_cast<int64_t>(run), max_pos - first));
    float* pc = cos_t + first * half + i;
    float* ps = sin_t + first * half + i;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
        *pc = static_cast<float>(c);
        *ps = static_cast<float>(s);
        pc += half;
        ps += half;
        const double t = c * cw - s * sw;
        s = s * cw + c * sw;
        c = t;
    }
}

// ---------------------------------------------------------------------------
// norm and rotation
// ---------------------------------------------------------------------------
// Where the rows of one tensor lie: token t = (b, n), head h at
// b * batch + n * token + h * head (elements).
struct Rows {
    int64_t batch, token, head;
    __device__ __forceinline__ int64_t at(int b, int n, int h) const {
        return b * batch + n * token + h * head;
    }
};

// i / d for i < 2^31 by a multiplication (Granlund and Montgomery, "Division by
// Invariant Integers using Multiplication", 1994): with l = ceil(log2 d) and
// m = floor(2^32 (2^l - d) / d) + 1, it is (floor(m i / 2^32) + i) >> l.
struct Divisor {
    uint32_t d, m, l;
    static Divisor of(uint32_t d) {
        uint32_t l = 0;
        while ((uint64_t{1} << l) < d) ++l;
        const uint64_t m = ((uint64_t{1} << 32) * ((uint64_t{1} << l) - d)) / d + 1;
        return Divisor{d, static_cast<uint32_t>(m), l};
    }
    __device__ __forceinline__ uint32_t quotient(uint32_t i) const {
        return (__umulhi(m, i) + i) >> l;
    }
};

// One of the two tensors of a call: queries or keys.
struct Side {
    const __nv_bfloat16* x;  // the rows to norm
    const __nv_bfloat16* g;  // backward: gradients of the outputs
    __nv_bfloat16* y;        // outputs, or gradients of the rows
    Rows rx, rg, ry;
    NormWeight w;
    int heads;
    Divisor groups;  // groups of U heads
    uint32_t slots;  // tokens * groups
    int ctas;        // CTAs of the grid that take this side
};

struct NormRope {
    Side q, k;
    RopeTable t;
    const int32_t* positions;
    Divisor N;
    bool heads_first;
    float eps;
    float* part;  // backward: [CTAs, D] partial weight gradients
    unsigned int* err;
};

// A slot is U heads of one token, taken by D / 8 lanes: the token's table
// entries are read once for U rows, and U loads are in flight.  Slots next to
// each other are next to each other in memory: the groups of heads of a token
// where tokens come first, the tokens of a group where heads do.
struct Slot {
    int b, n, h0;
    __device__ __forceinline__ Slot(const NormRope& p, const Side& s, uint32_t i, int U,
                                    bool heads_first) {
        if (heads_first) {
            const uint32_t outer = p.N.quotient(i);
            n = static_cast<int>(i - outer * p.N.d);
            b = static_cast<int>(s.groups.quotient(outer));
            h0 = static_cast<int>(outer - static_cast<uint32_t>(b) * s.groups.d) * U;
        } else {
            b = 0;
            n = static_cast<int>(s.groups.quotient(i));
            h0 = static_cast<int>(i - static_cast<uint32_t>(n) * s.groups.d) * U;
        }
    }
    // The token's position in the tables; out of them: 0, and bad.
    __device__ __forceinline__ int position(const NormRope& p, bool& bad) const {
        const int pos =
            p.positions ? __ldg(p.positions + static_cast<int64_t>(b) * p.N.d + n) : n;
        bad = p.t.half > 0 && (pos < 0 || pos >= p.t.max_pos);
        return bad ? 0 : pos;
    }
};

// The grid's first CTAs take the queries, the others the keys, each in equal
// strides over its slots: a CTA's weights stay in registers.
//
// 16384 tokens of 32 + 8 heads (heads first, fp32 weights): 58.7 us, 5.86 TB/s,
// 0.91 of a copy; 64 tokens 3.0 us, launch and two round trips to memory.  Bound by
// memory, with the scheduler 70 % busy: 4 CTAs of 64 registers an SM keep 64 KB of
// rows in flight (72 registers and 3 CTAs: 68.5 us; 2 heads a slot instead of 4,
// half the bytes in flight and twice the table reads: 71.7 us).
// (HEADS: heads first; else the heads of a token are D apart, which makes every
// row's address a constant offset.)
template <int D, bool INTER, bool HEADS, int U>
__global__ void __launch_bounds__(kThreads, 4)
    fa_norm_rope_kernel(const __grid_constant__ NormRope p) {
    constexpr int LPR = D / 8, SL = kThreads / LPR;
    const Lane<D, INTER> lane(p.t.half);
    const bool is_q = static_cast<int>(blockIdx.x) < p.q.ctas;
    const Side& s = is_q ? p.q : p.k;
    const uint32_t stride = static_cast<uint32_t>(s.ctas) * SL;
    const bool norms = s.w.w != nullptr;
    Vec8 w = {};
    if (norms) w = lane.weights(s.w);
    // all lanes of a warp stay together: the last slot stands in for those behind it
    for (uint32_t base = (blockIdx.x - (is_q ? 0 : p.q.ctas)) * SL; base < s.slots;
         base += stride) {
        const uint32_t i = base + threadIdx.x / LPR;
        const bool live = i < s.slots;
        const Slot at(p, s, live ? i : s.slots - 1, U, HEADS);
        const int count = s.heads - at.h0;  // of rows, U at most
        uint4 raw[U];
        const __nv_bfloat16* x = s.x + s.rx.at(at.b, at.n, at.h0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            raw[u] = make_uint4(0, 0, 0, 0);
            if (u < count) raw[u] = lane.load(x + u * (HEADS ? s.rx.head : D));
        }
        bool bad;
        const int pos = at.position(p, bad);
        if (bad && live && lane.chunk == 0) record_error(p.err, FA_DEVERR_BAD_INPUT);
        Rotation<D, INTER> rot;
        rot.load(p.t, pos, lane);
        __nv_bfloat16* y = s.y + s.ry.at(at.b, at.n, at.h0);
        Vec8 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = lane.unpack(raw[u]);
        if (norms) {
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = norm_row<D>(v[u], w, p.eps);
        }
        if (lane.turns) {
#pragma unroll
            for (int u = 0; u < U; ++u) rot.turn(v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (live && u < count)
                lane.store(y + u * (HEADS ? s.ry.head : D),
                           bad ? make_uint4(0, 0, 0, 0) : lane.pack(v[u]));
        }
    }
}

// With g = the output's gradient turned back (the rotation's transpose),
//     dw = sum over rows of g * x * r,   dx = r (g w - x r^2 mean(g w x)).
// x is read again and normed again: cheaper than a saved statistic.  Each
// thread sums dw over its rows in registers, the CTA over its threads in
// shared memory, and a second kernel over the CTAs in fp64: a fixed order.
// 36800 packed tokens of 32 + 8 heads: 196 to 203 us with the second kernel (of
// several machines), 5.6 to 5.8 TB/s, up to 0.90 of a copy; memory latency leads the stalls, with the scheduler over half
// busy (3 heads a slot 208 us, 2 heads and 4 CTAs an SM 210, 6 and 2 242).
template <int D, bool INTER, bool HEADS, int U>
__global__ void __launch_bounds__(kThreads, kBwdCtas)
    fa_norm_rope_bwd_kernel(const __grid_constant__ NormRope p) {
    constexpr int LPR = D / 8, SL = kThreads / LPR;
    __shared__ float red[SL][D];
    const Lane<D, INTER> lane(p.t.half);
    asm volatile("griddepcontrol.launch_dependents;");
    const bool is_q = static_cast<int>(blockIdx.x) < p.q.ctas;
    const Side& s = is_q ? p.q : p.k;
    const uint32_t stride = static_cast<uint32_t>(s.ctas) * SL;
    const bool norms = s.w.w != nullptr;
    Vec8 w = {}, acc = {};
    if (norms) w = lane.weights(s.w);
    for (uint32_t base = (blockIdx.x - (is_q ? 0 : p.q.ctas)) * SL; base < s.slots;
         base += stride) {
        const uint32_t i = base + threadIdx.x / LPR;
        const bool live = i < s.slots;
        const Slot at(p, s, live ? i : s.slots - 1, U, HEADS);
        const int count = live ? s.heads - at.h0 : 0;  // rows that are not there: zeros
        uint4 gr[U], xr[U];
        const __nv_bfloat16* g = s.g + s.rg.at(at.b, at.n, at.h0);
        const __nv_bfloat16* x = s.x + s.rx.at(at.b, at.n, at.h0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            gr[u] = xr[u] = make_uint4(0, 0, 0, 0);
            if (u < count) {
                gr[u] = lane.load(g + u * (HEADS ? s.rg.head : D));
                if (norms) xr[u] = lane.load(x + u * (HEADS ? s.rx.head : D));
            }
        }
        bool bad;
        const int pos = at.position(p, bad);
        if (bad && live && lane.chunk == 0) record_error(p.err, FA_DEVERR_BAD_INPUT);
        if (bad) {  // zero gradients of the row, nothing to the weights'
#pragma unroll
            for (int u = 0; u < U; ++u) gr[u] = xr[u] = make_uint4(0, 0, 0, 0);
        }
        Rotation<D, INTER> rot;
        rot.template load<true>(p.t, pos, lane);
        __nv_bfloat16* y = s.y + s.ry.at(at.b, at.n, at.h0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Vec8 gv = lane.unpack(gr[u]);
            rot.apply(gv);
            if (norms) {
                // with g' = g r:  dw += g' x,  dx = g' w - x r^2 mean(g' w x)
                const Vec8 xv = lane.unpack(xr[u]);
                float r = row_rstd<D>(xv, p.eps);
                if (u >= count || bad) r = 0.f;  // (of zeros it is infinite where eps is 0)
                gv = scale8(gv, r);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    acc.a[j] = f2_fma(gv.a[j], xv.a[j], acc.a[j]);
                    acc.b[j] = f2_fma(gv.b[j], xv.b[j], acc.b[j]);
                }
                gv = mul8(gv, w);
                const float m = row_sum<D>(dot8(gv, xv)) * (-1.f / D) * (r * r);
                const uint64_t mm = f2_pack(m, m);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    gv.a[j] = f2_fma(xv.a[j], mm, gv.a[j]);
                    gv.b[j] = f2_fma(xv.b[j], mm, gv.b[j]);
                }
            }
            if (u < count) lane.store(y + u * (HEADS ? s.ry.head : D), lane.pack(gv));
        }
    }
    if (!norms) return;  // the whole CTA
    float sums[8];
    lane.in_order(acc, sums);
    const int my = threadIdx.x / LPR;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        red[my][lane.lo + j] = sums[j];
        red[my][lane.hi + j] = sums[4 + j];
    }
    __syncthreads();
    if (threadIdx.x < D) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < SL; ++i) sum += red[i][threadIdx.x];
        p.part[static_cast<int64_t>(blockIdx.x) * D + threadIdx.x] = sum;
    }
}

// dw, kSumCols values of it a block, q's first: the CTAs' partial sums added in
// fp64.  Launched while the last CTAs of the kernel before it still run.
constexpr int kSumCols = 32, kSumRows = 32;
template <int D>
__global__ void __launch_bounds__(kSumCols* kSumRows)
    fa_norm_rope_dw_kernel(const float* part, int q_ctas, int ctas, float* __restrict__ dwq,
                           float* __restrict__ dwk) {
    __shared__ double red[kSumRows][kSumCols];
    const bool is_q = blockIdx.x < D / kSumCols;
    float* dst = is_q ? dwq : dwk;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (dst == nullptr) return;
    const int col = blockIdx.x % (D / kSumCols) * kSumCols + threadIdx.x;
    const int end = is_q ? q_ctas : ctas;
    double s = 0.0;
#pragma unroll 8
    for (int i = (is_q ? 0 : q_ctas) + threadIdx.y; i < end; i += kSumRows)
        s += part[static_cast<int64_t>(i) * D + col];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0) {
#pragma unroll
        for (int i = 1; i < kSumRows; ++i) s += red[i][threadIdx.x];
        dst[col] = static_cast<float>(s);
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The rows of a tensor with `heads` heads: packed tokens `stride` apart (0:
// back to back), or [B, heads, N, d].
int rows_of(int layout, int heads, int N, int d, int stride, Rows* r) {
    if (layout == FA_LAYOUT_HEADS) {
        if (stride != 0) return FA_ERR_SHAPE;
        *r = Rows{static_cast<int64_t>(heads) * N * d, d, static_cast<int64_t>(N) * d};
        return FA_OK;
    }
    const int64_t st = stride == 0 ? static_cast<int64_t>(heads) * d : stride;
    if (st < static_cast<int64_t>(heads) * d) return FA_ERR_SHAPE;
    if (st % 8 != 0) return FA_ERR_ALIGN;
    *r = Rows{st * N, st, d};
    return FA_OK;
}

// What both directions take and check alike.
int fill(NormRope& p, const void* q, const void* k, void* qo, void* ko, const void* wq,
         const void* wk, int weight_type, const float* rope_cos, const float* rope_sin,
         int max_pos, int rotary_dim, const int32_t* positions, int layout, int B, int N, int H,
         int H_kv, int d, int q_stride, int k_stride, int qo_stride, int ko_stride, float eps) {
    if (!q || !k || !qo || !ko) return FA_ERR_NULL;
    if (rotary_dim < 0 || (rotary_dim > 0 && (!rope_cos || !rope_sin)))
        return rotary_dim < 0 ? FA_ERR_SHAPE : FA_ERR_NULL;
    if (layout != FA_LAYOUT_PACKED && layout != FA_LAYOUT_HEADS) return FA_ERR_UNSUPPORTED;
    if (B < 1 || N < 1 || H < 1 || H_kv < 1 || (layout == FA_LAYOUT_PACKED && B != 1))
        return FA_ERR_SHAPE;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (rotary_dim % 16 != 0) return FA_ERR_UNSUPPORTED;
    if (rotary_dim > d) return FA_ERR_SHAPE;
    if (weight_type != FA_WEIGHT_BF16 && weight_type != FA_WEIGHT_FP32) return FA_ERR_UNSUPPORTED;
    if (!std::isfinite(eps) || eps < 0.f) return FA_ERR_SHAPE;
    if (rotary_dim > 0 && (max_pos < 1 || (!positions && max_pos < N))) return FA_ERR_SHAPE;
    // rows are counted in 32 bits: 2^31 of them would fill 256 GB and more
    if (static_cast<int64_t>(B) * N > 0x7fffffff / (static_cast<int64_t>(H) + H_kv))
        return FA_ERR_SHAPE;
    int rc;
    if ((rc = rows_of(layout, H, N, d, q_stride, &p.q.rx)) != FA_OK) return rc;
    if ((rc = rows_of(layout, H_kv, N, d, k_stride, &p.k.rx)) != FA_OK) return rc;
    if ((rc = rows_of(layout, H, N, d, qo_stride, &p.q.ry)) != FA_OK) return rc;
    if ((rc = rows_of(layout, H_kv, N, d, ko_stride, &p.k.ry)) != FA_OK) return rc;
    if (!aligned16(q) || !aligned16(k) || !aligned16(qo) || !aligned16(ko) ||
        (wq && !aligned16(wq)) || (wk && !aligned16(wk)) ||
        (rotary_dim > 0 && (!aligned16(rope_cos) || !aligned16(rope_sin))))
        return FA_ERR_ALIGN;
    p.q.x = static_cast<const __nv_bfloat16*>(q);
    p.k.x = static_cast<const __nv_bfloat16*>(k);
    p.q.y = static_cast<__nv_bfloat16*>(qo);
    p.k.y = static_cast<__nv_bfloat16*>(ko);
    p.q.w = NormWeight{wq, weight_type == FA_WEIGHT_FP32};
    p.k.w = NormWeight{wk, weight_type == FA_WEIGHT_FP32};
    p.q.heads = H;
    p.k.heads = H_kv;
    p.t = RopeTable{rope_cos, rope_sin, max_pos, rotary_dim / 2};
    p.positions = positions;
    p.N = Divisor::of(static_cast<uint32_t>(N));
    p.heads_first = layout == FA_LAYOUT_HEADS;
    p.eps = eps;
    return FA_OK;
}

// Slots of U heads, and CTAs for them: as many as there is work for, up to
// `per_sm` for each SM, shared between the sides as their slots are.
int set_grid(NormRope& p, int64_t tokens, int d, int heads_per_slot, int per_sm, int num_sms) {
    const int64_t per = kThreads / (d / 8);
    Side* sides[] = {&p.q, &p.k};
    int64_t want[2];
    for (int i = 0; i < 2; ++i) {
        const int groups = (sides[i]->heads + heads_per_slot - 1) / heads_per_slot;
        sides[i]->groups = Divisor::of(static_cast<uint32_t>(groups));
        const int64_t slots = tokens * groups;
        sides[i]->slots = static_cast<uint32_t>(slots);
        want[i] = (slots + per - 1) / per;
    }
    const int64_t most = static_cast<int64_t>(num_sms) * per_sm, all = want[0] + want[1];
    if (all > most) {
        int64_t k = (want[1] * most + all / 2) / all;
        k = k < 1 ? 1 : k > most - 1 ? most - 1 : k;
        want[1] = k;
        want[0] = most - k;
    }
    p.q.ctas = static_cast<int>(want[0]);
    p.k.ctas = static_cast<int>(want[1]);
    return p.q.ctas + p.k.ctas;
}

template <int D, bool INTER>
int launch_norm(const NormRope& p, int ctas, cudaStream_t st) {
    if (p.heads_first) fa_norm_rope_kernel<D, INTER, true, kFwdHeads><<<ctas, kThreads, 0, st>>>(p);
    else fa_norm_rope_kernel<D, INTER, false, kFwdHeads><<<ctas, kThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D, bool INTER>
int launch_norm_bwd(const NormRope& p, int ctas, float* dwq, float* dwk, cudaStream_t st) {
    if (p.heads_first)
        fa_norm_rope_bwd_kernel<D, INTER, true, kBwdHeads><<<ctas, kThreads, 0, st>>>(p);
    else
        fa_norm_rope_bwd_kernel<D, INTER, false, kBwdHeads><<<ctas, kThreads, 0, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    if (!p.part) return FA_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * D / kSumCols);
    cfg.blockDim = dim3(kSumCols, kSumRows);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fa_norm_rope_dw_kernel<D>, static_cast<const float*>(p.part),
                              p.q.ctas, ctas, dwq, dwk) == cudaSuccess
               ? FA_OK
               : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

extern "C" {

int fa_rope_table(float* rope_cos, float* rope_sin, int max_pos, int rotary_dim, double base,
                  int scaling, double factor, int original_len, double low, double high,
                  double mscale, fa_stream_t stream) {
    if (!rope_cos || !rope_sin) return FA_ERR_NULL;
    if (max_pos < 1 || rotary_dim < 2 || rotary_dim % 2 != 0 ||
        rotary_dim > 2 * fa::kRopeMaxPairs)
        return FA_ERR_SHAPE;
    if (!std::isfinite(base) || base <= 1.0 || !std::isfinite(mscale)) return FA_ERR_SHAPE;
    if (scaling < FA_ROPE_PLAIN || scaling > FA_ROPE_YARN) return FA_ERR_UNSUPPORTED;
    if (scaling != FA_ROPE_PLAIN && (!std::isfinite(factor) || factor <= 0.0))
        return FA_ERR_SHAPE;
    if (scaling == FA_ROPE_NTK && rotary_dim <= 2) return FA_ERR_SHAPE;
    if ((scaling == FA_ROPE_TURNS || scaling == FA_ROPE_YARN) &&
        (original_len < 1 || !std::isfinite(low) || !std::isfinite(high) || high <= low ||
         (scaling == FA_ROPE_YARN && low <= 0.0)))
        return FA_ERR_SHAPE;
    if (!fa::aligned16(rope_cos) || !fa::aligned16(rope_sin)) return FA_ERR_ALIGN;
    const int R = rotary_dim, half = R / 2;
    if (scaling == FA_ROPE_NTK) base *= std::pow(factor, R / (R - 2.0));
    double first = 0.0, last = 0.0;  // the pairs between which the frequencies blend
    if (scaling == FA_ROPE_YARN) {
        auto pair_of = [&](double turns) {
            return R * std::log(original_len / (turns * fa::kTwoPi)) / (2.0 * std::log(base));
        };
        first = std::fmax(std::floor(pair_of(high)), 0.0);
        last = std::fmin(std::ceil(pair_of(low)), R - 1.0);
    }
    fa::Turns t;
    const double log2_step = -2.0 * std::log2(base) / R;
    for (int i = 0; i < half; ++i) {
        double w = std::exp2(log2_step * i);
        double slow = 0.0;  // the share of the stretched frequency
        if (scaling == FA_ROPE_LINEAR) slow = 1.0;
        if (scaling == FA_ROPE_TURNS) {
            const double made = original_len * w / fa::kTwoPi;
            slow = 1.0 - std::fmin(1.0, std::fmax(0.0, (made - low) / (high - low)));
        }
        if (scaling == FA_ROPE_YARN)
            slow = std::fmin(1.0, std::fmax(0.0, (i - first) / std::fmax(last - first, 0.001)));
        if (slow > 0.0) w = w * (1.0 - slow) + w / factor * slow;
        t.w[i] = w / fa::kTwoPi;
        if (!std::isfinite(t.w[i] * max_pos)) return FA_ERR_SHAPE;  // no angle
    }
    unsigned int* err = nullptr;
    int num_sms = 0, rc;
    if ((rc = fa::device_error_word(&err, &num_sms)) != FA_OK) return rc;
    // runs of up to 16 positions, and shorter ones where SMs would be short of
    // threads
    const int64_t n = static_cast<int64_t>(max_pos) * half;
    const int64_t run =
        std::min<int64_t>(std::max<int64_t>(n / (static_cast<int64_t>(num_sms) * 512), 4), 16);
    const int64_t threads = (max_pos + run - 1) / run * half;
    fa::fa_rope_table_kernel<<<static_cast<unsigned>((threads + fa::kThreads - 1) / fa::kThreads),
                               fa::kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        rope_cos, rope_sin, max_pos, half, static_cast<int>(run), mscale, t);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int fa_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const void* q_weight,
                    const void* k_weight, int weight_type, const float* rope_cos,
                    const float* rope_sin, int max_pos, int rotary_dim, int interleaved,
                    const int32_t* positions, int layout, int B, int N, int H, int H_kv, int d,
                    int q_stride, int k_stride, int q_out_stride, int k_out_stride, float eps,
                    fa_stream_t stream) {
    fa::NormRope p{};
    int rc = fa::fill(p, q, k, q_out, k_out, q_weight, k_weight, weight_type, rope_cos, rope_sin,
                      max_pos, rotary_dim, positions, layout, B, N, H, H_kv, d, q_stride,
                      k_stride, q_out_stride, k_out_stride, eps);
    if (rc != FA_OK) return rc;
    int num_sms = 0;
    if ((rc = fa::device_error_word(&p.err, &num_sms)) != FA_OK) return rc;
    const int ctas = fa::set_grid(p, static_cast<int64_t>(B) * N, d, fa::kFwdHeads, fa::kFwdCtas,
                                  num_sms);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d == 64)
        return interleaved ? fa::launch_norm<64, true>(p, ctas, st)
                           : fa::launch_norm<64, false>(p, ctas, st);
    return interleaved ? fa::launch_norm<128, true>(p, ctas, st)
                       : fa::launch_norm<128, false>(p, ctas, st);
}

int fa_qk_norm_rope_bwd_workspace(int B, int N, int H, int H_kv, int d, int* bytes) {
    if (!bytes) return FA_ERR_NULL;
    if (B < 1 || N < 1 || H < 1 || H_kv < 1) return FA_ERR_SHAPE;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    unsigned int* err = nullptr;
    int num_sms = 0, rc;
    if ((rc = fa::device_error_word(&err, &num_sms)) != FA_OK) return rc;
    fa::NormRope p{};
    p.q.heads = H;
    p.k.heads = H_kv;
    *bytes = fa::set_grid(p, static_cast<int64_t>(B) * N, d, fa::kBwdHeads, fa::kBwdCtas,
                          num_sms) * d * static_cast<int>(sizeof(float));
    return FA_OK;
}

int fa_qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out,
                        void* dq, void* dk, float* dq_weight, float* dk_weight,
                        const void* q_weight, const void* k_weight, int weight_type,
                        const float* rope_cos, const float* rope_sin, int max_pos,
                        int rotary_dim, int interleaved, const int32_t* positions, int layout,
                        int B, int N, int H, int H_kv, int d, int q_stride, int k_stride,
                        int dq_out_stride, int dk_out_stride, int dq_stride, int dk_stride,
                        float eps, void* workspace, int workspace_bytes, fa_stream_t stream) {
    if (!dq_out || !dk_out) return FA_ERR_NULL;
    // a weight and its gradient come together
    if ((q_weight == nullptr) != (dq_weight == nullptr) ||
        (k_weight == nullptr) != (dk_weight == nullptr))
        return FA_ERR_NULL;
    fa::NormRope p{};
    int rc = fa::fill(p, q, k, dq, dk, q_weight, k_weight, weight_type, rope_cos, rope_sin,
                      max_pos, rotary_dim, positions, layout, B, N, H, H_kv, d, q_stride,
                      k_stride, dq_stride, dk_stride, eps);
    if (rc != FA_OK) return rc;
    if ((rc = fa::rows_of(layout, H, N, d, dq_out_stride, &p.q.rg)) != FA_OK) return rc;
    if ((rc = fa::rows_of(layout, H_kv, N, d, dk_out_stride, &p.k.rg)) != FA_OK) return rc;
    if (workspace_bytes < 0) return FA_ERR_SHAPE;
    if (!fa::aligned16(dq_out) || !fa::aligned16(dk_out) || !fa::aligned16(workspace))
        return FA_ERR_ALIGN;
    p.q.g = static_cast<const __nv_bfloat16*>(dq_out);
    p.k.g = static_cast<const __nv_bfloat16*>(dk_out);
    int num_sms = 0;
    if ((rc = fa::device_error_word(&p.err, &num_sms)) != FA_OK) return rc;
    const int ctas = fa::set_grid(p, static_cast<int64_t>(B) * N, d, fa::kBwdHeads, fa::kBwdCtas,
                                  num_sms);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    fa::WorkspaceHold hold;
    if (q_weight || k_weight) {
        void* ws = nullptr;
        const size_t need = sizeof(float) * static_cast<size_t>(ctas) * d;
        if ((rc = fa::call_workspace(workspace, workspace_bytes, need, st, &ws, &hold)) != FA_OK)
            return rc;
        p.part = static_cast<float*>(ws);
    }
    if (d == 64)
        return interleaved ? fa::launch_norm_bwd<64, true>(p, ctas, dq_weight, dk_weight, st)
                           : fa::launch_norm_bwd<64, false>(p, ctas, dq_weight, dk_weight, st);
    return interleaved ? fa::launch_norm_bwd<128, true>(p, ctas, dq_weight, dk_weight, st)
                       : fa::launch_norm_bwd<128, false>(p, ctas, dq_weight, dk_weight, st);
}

}  // extern "C"
