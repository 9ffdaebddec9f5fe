// rope_sm100.cu -- rotary tables scaled for long contexts, and the per-head
// norms of queries and keys with the rotation in the same pass, forward and
// backward.
//
// The page "“Flash”不是那个被时代淘汰的插件" (0539edu.com), sections 2 and 3,
// keeps the rotation's sines and cosines in a precomputed table; so do these
// calls.  Everything here moves a few bytes for each operation, so all of it
// is written for memory: every row is read once and written once, in 16-byte
// pieces, several of them in flight for each thread.
#include <cmath>

#include "fa_internal.h"
#include "rope_row.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr double kTwoPi = 6.283185307179586476925286766559;

// ---------------------------------------------------------------------------
// tables: cos and sin of p * w_i, w_i handed over in turns (w_i / 2 pi) in
// fp64.  The angle of a far position is many turns: p * w_i is formed in fp64
// and reduced there to an eighth of a turn either way, exactly, before one
// fp32 sine and cosine of it; the octant swaps and signs them.  Written in
// 16-byte stores; at 131072 positions the writes are the bound.
// ---------------------------------------------------------------------------
struct Turns {
    double w[kRopeMaxPairs];
};

__global__ void __launch_bounds__(kThreads)
    fa_rope_table_kernel(float* __restrict__ cos_t, float* __restrict__ sin_t, int64_t n,
                         int half, float mscale, const __grid_constant__ Turns turns) {
    __shared__ double w[kRopeMaxPairs];  // the threads of a warp read different pairs
    for (int i = threadIdx.x; i < half; i += kThreads) w[i] = turns.w[i];
    __syncthreads();
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads * 4;
    for (int64_t e = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 4; e < n;
         e += step) {
        int64_t p = e / half;
        int i = static_cast<int>(e - p * half);
        float c[4], s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const double q = static_cast<double>(p) * w[i] * 4.0;  // quarter turns
            const double whole = rint(q);
            const int quarter = static_cast<int>(static_cast<int64_t>(whole)) & 3;
            float sv, cv;
            sincospif(static_cast<float>(q - whole) * 0.5f, &sv, &cv);
            const float a = (quarter & 1) ? sv : cv, b = (quarter & 1) ? cv : sv;
            c[j] = ((quarter + 1) & 2 ? -a : a) * mscale;
            s[j] = (quarter & 2 ? -b : b) * mscale;
            if (++i == half) {
                i = 0;
                ++p;
            }
        }
        if (e + 4 <= n) {
            *reinterpret_cast<float4*>(cos_t + e) = make_float4(c[0], c[1], c[2], c[3]);
            *reinterpret_cast<float4*>(sin_t + e) = make_float4(s[0], s[1], s[2], s[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (e + j < n) {
                    cos_t[e + j] = c[j];
                    sin_t[e + j] = s[j];
                }
            }
        }
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

struct NormRope {
    const __nv_bfloat16 *q, *k;    // the rows to norm
    const __nv_bfloat16 *gq, *gk;  // backward: gradients of the outputs
    __nv_bfloat16 *qo, *ko;        // outputs, or gradients of the rows
    Rows rq, rk, rgq, rgk, rqo, rko;
    NormWeight wq, wk;
    RopeTable t;
    const int32_t* positions;
    int N, H, Hk;
    int gq_groups, groups;  // groups of U heads of one token: of queries, of both
    int64_t slots;          // tokens * groups
    float eps;
    float* part;  // backward: [grid, 2, D] partial weight gradients
    unsigned int* err;
};

// D / 8 lanes take U heads of one token, so that the token's table entries are
// read once for U rows and U loads are in flight.
template <int D, bool INTER, int U>
__global__ void __launch_bounds__(kThreads) fa_norm_rope_kernel(const NormRope p) {
    constexpr int LPR = D / 8;
    const int lane = threadIdx.x & 31, chunk = threadIdx.x % LPR;
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * (kThreads / LPR) + threadIdx.x / LPR;
    const bool live = slot < p.slots;
    const int64_t sl = live ? slot : p.slots - 1;
    const int64_t token = sl / p.groups;
    const int group = static_cast<int>(sl - token * p.groups);
    const int b = static_cast<int>(token / p.N), n = static_cast<int>(token - static_cast<int64_t>(b) * p.N);
    const bool is_q = group < p.gq_groups;
    const int heads = is_q ? p.H : p.Hk;
    const int h0 = (is_q ? group : group - p.gq_groups) * U;
    const __nv_bfloat16* x = is_q ? p.q : p.k;
    const Rows& rx = is_q ? p.rq : p.rk;
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        raw[u] = __ldcs(reinterpret_cast<const uint4*>(
            x + rx.at(b, n, min(h0 + u, heads - 1)) + chunk * 8));
    int pos = p.positions ? __ldg(p.positions + token) : n;
    const bool bad = p.t.half > 0 && (pos < 0 || pos >= p.t.max_pos);
    if (bad) pos = 0;
    if (bad && live && chunk == 0) record_error(p.err, FA_DEVERR_BAD_INPUT);
    Rotation<D, INTER> rot;
    rot.load(p.t, pos, lane, 1.f);
    const NormWeight nw = is_q ? p.wq : p.wk;
    const bool norms = p.wq.w || p.wk.w;
    float w[8];
    if (nw.w) load_weight8(nw, chunk, w);
    __nv_bfloat16* y = is_q ? p.qo : p.ko;
    const Rows& ry = is_q ? p.rqo : p.rko;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float v[8];
        unpack8(raw[u], v);
        // the lanes of a warp may hold rows of q and of k: all take the sum
        const float r = norms ? row_rstd<D>(v, p.eps) : 1.f;
        if (nw.w) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= r * w[j];
        }
        rot.apply(v);
        if (live && h0 + u < heads) {
            const uint4 out = bad ? make_uint4(0, 0, 0, 0) : pack8(v);
            *reinterpret_cast<uint4*>(y + ry.at(b, n, h0 + u) + chunk * 8) = out;
        }
    }
}

// With g = the output's gradient turned back (the rotation's transpose),
//     dw = sum over rows of g * x * r,   dx = r (g w - x r^2 mean(g w x)).
// x is read again and normed again: cheaper than a saved statistic.  Each
// thread sums dw over its rows in registers, the CTA over its threads in
// shared memory, and a second kernel over the CTAs in fp64: a fixed order.
template <int D, bool INTER, int U>
__global__ void __launch_bounds__(kThreads) fa_norm_rope_bwd_kernel(const NormRope p) {
    constexpr int LPR = D / 8, SL = kThreads / LPR;
    __shared__ float red[SL][D];
    const int lane = threadIdx.x & 31, chunk = threadIdx.x % LPR, my = threadIdx.x / LPR;
    const bool norms = p.wq.w || p.wk.w;
    float accq[8], acck[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) accq[j] = acck[j] = 0.f;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * SL; base < p.slots;
         base += static_cast<int64_t>(gridDim.x) * SL) {
        const int64_t slot = base + my;
        const bool live = slot < p.slots;
        const int64_t sl = live ? slot : p.slots - 1;
        const int64_t token = sl / p.groups;
        const int group = static_cast<int>(sl - token * p.groups);
        const int b = static_cast<int>(token / p.N), n = static_cast<int>(token - static_cast<int64_t>(b) * p.N);
        const bool is_q = group < p.gq_groups;
        const int heads = is_q ? p.H : p.Hk;
        const int h0 = (is_q ? group : group - p.gq_groups) * U;
        const NormWeight nw = is_q ? p.wq : p.wk;
        const __nv_bfloat16* x = is_q ? p.q : p.k;
        const __nv_bfloat16* g = is_q ? p.gq : p.gk;
        const Rows& rx = is_q ? p.rq : p.rk;
        const Rows& rg = is_q ? p.rgq : p.rgk;
        uint4 gr[U], xr[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = min(h0 + u, heads - 1);
            gr[u] = __ldcs(reinterpret_cast<const uint4*>(g + rg.at(b, n, h) + chunk * 8));
            xr[u] = make_uint4(0, 0, 0, 0);
            if (nw.w)
                xr[u] = __ldcs(reinterpret_cast<const uint4*>(x + rx.at(b, n, h) + chunk * 8));
        }
        int pos = p.positions ? __ldg(p.positions + token) : n;
        const bool bad = p.t.half > 0 && (pos < 0 || pos >= p.t.max_pos);
        if (bad) pos = 0;
        if (bad && live && chunk == 0) record_error(p.err, FA_DEVERR_BAD_INPUT);
        Rotation<D, INTER> rot;
        rot.load(p.t, pos, lane, -1.f);
        float w[8];
        if (nw.w) load_weight8(nw, chunk, w);
        __nv_bfloat16* y = is_q ? p.qo : p.ko;
        const Rows& ry = is_q ? p.rqo : p.rko;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float gv[8], xv[8];
            unpack8(gr[u], gv);
            unpack8(xr[u], xv);
            rot.apply(gv);
            const bool mine = live && h0 + u < heads;
            const float r = norms ? row_rstd<D>(xv, p.eps) : 1.f;
            float dot = 0.f;
            if (nw.w) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float hat = xv[j] * r;
                    if (mine && !bad) {
                        if (is_q) accq[j] = fmaf(gv[j], hat, accq[j]);
                        else acck[j] = fmaf(gv[j], hat, acck[j]);
                    }
                    xv[j] = hat;
                    gv[j] *= w[j];
                    dot = fmaf(gv[j], hat, dot);
                }
            }
            if (norms) dot = row_sum<D>(dot) * (1.f / D);
            if (nw.w) {
#pragma unroll
                for (int j = 0; j < 8; ++j) gv[j] = r * (gv[j] - xv[j] * dot);
            }
            if (mine) {
                const uint4 out = bad ? make_uint4(0, 0, 0, 0) : pack8(gv);
                *reinterpret_cast<uint4*>(y + ry.at(b, n, h0 + u) + chunk * 8) = out;
            }
        }
    }
    if (p.part == nullptr) return;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int j = 0; j < 8; ++j) red[my][chunk * 8 + j] = which ? acck[j] : accq[j];
        __syncthreads();
        if (threadIdx.x < D) {
            float s = 0.f;
            for (int i = 0; i < SL; ++i) s += red[i][threadIdx.x];
            p.part[(static_cast<int64_t>(blockIdx.x) * 2 + which) * D + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

// dw of q (block 0) and of k (block 1): the CTAs' partial sums added in fp64.
constexpr int kSumRows = 8;
template <int D>
__global__ void __launch_bounds__(D* kSumRows)
    fa_norm_rope_dw_kernel(const float* __restrict__ part, int ctas, float* __restrict__ dwq,
                           float* __restrict__ dwk) {
    __shared__ double red[kSumRows][D];
    const int col = threadIdx.x % D, row = threadIdx.x / D;
    float* dst = blockIdx.x == 0 ? dwq : dwk;
    double s = 0.0;
    if (dst)
        for (int i = row; i < ctas; i += kSumRows)
            s += part[(static_cast<int64_t>(i) * 2 + blockIdx.x) * D + col];
    red[row][col] = s;
    __syncthreads();
    if (row == 0 && dst) {
        for (int i = 1; i < kSumRows; ++i) s += red[i][col];
        dst[col] = static_cast<float>(s);
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kFwdHeads = 4;  // heads a slot takes
constexpr int kBwdHeads = 2;
constexpr int kBwdCtas = 4;  // CTAs per SM of the backward kernel's grid

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
    // one slot of a CTA takes at least one row; the grid's x has 2^31 - 1 CTAs
    const int64_t tokens = static_cast<int64_t>(B) * N;
    if (tokens > (int64_t{1} << 34) / (static_cast<int64_t>(H) + H_kv)) return FA_ERR_SHAPE;
    int rc;
    if ((rc = rows_of(layout, H, N, d, q_stride, &p.rq)) != FA_OK) return rc;
    if ((rc = rows_of(layout, H_kv, N, d, k_stride, &p.rk)) != FA_OK) return rc;
    if ((rc = rows_of(layout, H, N, d, qo_stride, &p.rqo)) != FA_OK) return rc;
    if ((rc = rows_of(layout, H_kv, N, d, ko_stride, &p.rko)) != FA_OK) return rc;
    if (!aligned16(q) || !aligned16(k) || !aligned16(qo) || !aligned16(ko) ||
        (wq && !aligned16(wq)) || (wk && !aligned16(wk)) ||
        (rotary_dim > 0 && (!aligned16(rope_cos) || !aligned16(rope_sin))))
        return FA_ERR_ALIGN;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.qo = static_cast<__nv_bfloat16*>(qo);
    p.ko = static_cast<__nv_bfloat16*>(ko);
    p.wq = NormWeight{wq, weight_type == FA_WEIGHT_FP32};
    p.wk = NormWeight{wk, weight_type == FA_WEIGHT_FP32};
    p.t = RopeTable{rope_cos, rope_sin, max_pos, rotary_dim / 2};
    p.positions = positions;
    p.N = N;
    p.H = H;
    p.Hk = H_kv;
    p.eps = eps;
    return FA_OK;
}

void set_groups(NormRope& p, int64_t tokens, int heads_per_slot) {
    p.gq_groups = (p.H + heads_per_slot - 1) / heads_per_slot;
    p.groups = p.gq_groups + (p.Hk + heads_per_slot - 1) / heads_per_slot;
    p.slots = tokens * p.groups;
}

// Workspace of the backward pass: [CTAs, 2, d] partial weight gradients.
int bwd_ctas(int64_t slots, int d, int num_sms) {
    const int64_t per = kThreads / (d / 8);
    const int64_t want = (slots + per - 1) / per, most = static_cast<int64_t>(num_sms) * kBwdCtas;
    return static_cast<int>(want < most ? want : most);
}

template <int D, bool INTER>
int launch_norm(NormRope& p, int64_t tokens, cudaStream_t st) {
    constexpr int per = kThreads / (D / 8);
    set_groups(p, tokens, kFwdHeads);
    const int64_t ctas = (p.slots + per - 1) / per;
    fa_norm_rope_kernel<D, INTER, kFwdHeads>
        <<<static_cast<unsigned>(ctas), kThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D, bool INTER>
int launch_norm_bwd(NormRope& p, int ctas, float* dwq, float* dwk, cudaStream_t st) {
    fa_norm_rope_bwd_kernel<D, INTER, kBwdHeads><<<ctas, kThreads, 0, st>>>(p);
    if (p.part)
        fa_norm_rope_dw_kernel<D><<<2, D * kSumRows, 0, st>>>(p.part, ctas, dwq, dwk);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
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
    for (int i = 0; i < half; ++i) {
        double w = std::pow(base, -2.0 * i / R);
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
    }
    unsigned int* err = nullptr;
    int num_sms = 0, rc;
    if ((rc = fa::device_error_word(&err, &num_sms)) != FA_OK) return rc;
    const int64_t n = static_cast<int64_t>(max_pos) * half;
    const int64_t want = (n + fa::kThreads * 4 - 1) / (fa::kThreads * 4);
    const int64_t most = static_cast<int64_t>(num_sms) * 8;
    fa::fa_rope_table_kernel<<<static_cast<unsigned>(want < most ? want : most), fa::kThreads, 0,
                               reinterpret_cast<cudaStream_t>(stream)>>>(
        rope_cos, rope_sin, n, half, static_cast<float>(mscale), t);
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
    const int64_t tokens = static_cast<int64_t>(B) * N;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d == 64)
        return interleaved ? fa::launch_norm<64, true>(p, tokens, st)
                           : fa::launch_norm<64, false>(p, tokens, st);
    return interleaved ? fa::launch_norm<128, true>(p, tokens, st)
                       : fa::launch_norm<128, false>(p, tokens, st);
}

int fa_qk_norm_rope_bwd_workspace(int B, int N, int H, int H_kv, int d, int* bytes) {
    if (!bytes) return FA_ERR_NULL;
    if (B < 1 || N < 1 || H < 1 || H_kv < 1) return FA_ERR_SHAPE;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    unsigned int* err = nullptr;
    int num_sms = 0, rc;
    if ((rc = fa::device_error_word(&err, &num_sms)) != FA_OK) return rc;
    fa::NormRope p{};
    p.H = H;
    p.Hk = H_kv;
    fa::set_groups(p, static_cast<int64_t>(B) * N, fa::kBwdHeads);
    *bytes = fa::bwd_ctas(p.slots, d, num_sms) * 2 * d * static_cast<int>(sizeof(float));
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
    if ((rc = fa::rows_of(layout, H, N, d, dq_out_stride, &p.rgq)) != FA_OK) return rc;
    if ((rc = fa::rows_of(layout, H_kv, N, d, dk_out_stride, &p.rgk)) != FA_OK) return rc;
    if (workspace_bytes < 0) return FA_ERR_SHAPE;
    if (!fa::aligned16(dq_out) || !fa::aligned16(dk_out) || !fa::aligned16(workspace))
        return FA_ERR_ALIGN;
    p.gq = static_cast<const __nv_bfloat16*>(dq_out);
    p.gk = static_cast<const __nv_bfloat16*>(dk_out);
    int num_sms = 0;
    if ((rc = fa::device_error_word(&p.err, &num_sms)) != FA_OK) return rc;
    fa::set_groups(p, static_cast<int64_t>(B) * N, fa::kBwdHeads);
    const int ctas = fa::bwd_ctas(p.slots, d, num_sms);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (q_weight || k_weight) {
        void* ws = nullptr;
        const size_t need = sizeof(float) * 2 * static_cast<size_t>(ctas) * d;
        if ((rc = fa::call_workspace(workspace, workspace_bytes, need, st, &ws)) != FA_OK)
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
