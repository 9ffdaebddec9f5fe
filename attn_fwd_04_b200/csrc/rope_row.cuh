// rope_row.cuh -- one head row (D values) normed and rotated by D/8 lanes of a
// warp, 8 values (16 bytes of bf16) each: shared by the kernels that norm and
// rotate queries and keys and by the cache appends.
//
// With x the row, w its weight, R the rotated part and (c_i, s_i) the table's
// entries of the row's position,
//     y  = x * rsqrt(mean(x^2) + eps) * w            (y = x without a weight)
//     (y_a, y_b) -> (y_a c_i - y_b s_i, y_b c_i + y_a s_i)   for the R/2 pairs
// where pair i is (i, i + R/2) (halves) or (2i, 2i + 1) (interleaved), and the
// values from R on stay.  R is a multiple of 16, so that a lane's 8 values lie
// in one half and its partner's 8 in one other lane: the exchange is one
// shuffle per value, and no value passes through shared memory.  The rotation
// rounds each product and then their sum (no fused multiply-add): the same
// rounding as the rotation inside fa_fwd_rope, so that the two agree bit for
// bit where there is no norm.
#pragma once
#include <cuda_bf16.h>

#include "fa_ptx.cuh"

namespace fa {

// The rotation's arguments as every entry point takes them.
struct RopeTable {
    const float* cos_t;
    const float* sin_t;
    int max_pos;
    int half;  // R / 2 pairs; 0: no rotation
};

// Norm weights: bf16 or fp32 [D], or null.
struct NormWeight {
    const void* w;
    int fp32;
};

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    x[0] = bf16_lo(v.x);
    x[1] = bf16_hi(v.x);
    x[2] = bf16_lo(v.y);
    x[3] = bf16_hi(v.y);
    x[4] = bf16_lo(v.z);
    x[5] = bf16_hi(v.z);
    x[6] = bf16_lo(v.w);
    x[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// 8 weights of lane chunk c.
__device__ __forceinline__ void load_weight8(const NormWeight& nw, int c, float (&w)[8]) {
    if (nw.fp32) {
        const float4* p = reinterpret_cast<const float4*>(nw.w) + 2 * c;
        const float4 a = __ldg(p), b = __ldg(p + 1);
        w[0] = a.x;
        w[1] = a.y;
        w[2] = a.z;
        w[3] = a.w;
        w[4] = b.x;
        w[5] = b.y;
        w[6] = b.z;
        w[7] = b.w;
    } else {
        unpack8(__ldg(reinterpret_cast<const uint4*>(nw.w) + c), w);
    }
}

// One lane's share of a position's rotation: cosines and signed sines of its
// values, and the lane its partners are in.
template <int D, bool INTER>
struct Rotation {
    static constexpr int kPairs = INTER ? 4 : 8;
    float c[kPairs], s[kPairs];
    int src;
    bool on;

    // pos in [0, max_pos); `sign` -1 turns back (the transpose, for gradients)
    __device__ __forceinline__ void load(const RopeTable& t, int pos, int lane, float sign) {
        const int chunk = lane % (D / 8);
        on = chunk * 8 < 2 * t.half;
        src = lane;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) c[j] = 1.f, s[j] = 0.f;
        if (!on) return;
        int i = chunk * 4;  // interleaved: the pairs 4 chunk .. 4 chunk + 3
        if (!INTER) {
            const int hc = t.half / 8;  // chunks in a half
            const bool lower = chunk < hc;
            src = lower ? lane + hc : lane - hc;
            i = (lower ? chunk : chunk - hc) * 8;
            if (lower) sign = -sign;
        }
        const int64_t at = static_cast<int64_t>(pos) * t.half + i;
#pragma unroll
        for (int j = 0; j < kPairs; j += 4) {
            const float4 cv = __ldg(reinterpret_cast<const float4*>(t.cos_t + at + j));
            const float4 sv = __ldg(reinterpret_cast<const float4*>(t.sin_t + at + j));
            c[j] = cv.x;
            c[j + 1] = cv.y;
            c[j + 2] = cv.z;
            c[j + 3] = cv.w;
            s[j] = sign * sv.x;
            s[j + 1] = sign * sv.y;
            s[j + 2] = sign * sv.z;
            s[j + 3] = sign * sv.w;
        }
    }

    // every lane of the warp calls this together
    __device__ __forceinline__ void apply(float (&y)[8]) const {
        if (INTER) {
            if (on) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a = y[2 * j], b = y[2 * j + 1];
                    y[2 * j] = __fsub_rn(__fmul_rn(a, c[j]), __fmul_rn(b, s[j]));
                    y[2 * j + 1] = __fadd_rn(__fmul_rn(b, c[j]), __fmul_rn(a, s[j]));
                }
            }
        } else {
            float p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = __shfl_sync(0xffffffffu, y[j], src);
            if (on) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = __fadd_rn(__fmul_rn(y[j], c[j % kPairs]), __fmul_rn(p[j], s[j % kPairs]));
            }
        }
    }
};

// Sum over the D/8 lanes of a row, the same in each of them.
template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// 1 / sqrt(mean(x^2) + eps) of a row.
template <int D>
__device__ __forceinline__ float row_rstd(const float (&x)[8], float eps) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
    return rsqrtf(row_sum<D>(ss) * (1.f / D) + eps);
}

// x normed by weight nw (skipped where it is null), in place.
template <int D>
__device__ __forceinline__ void norm_row(float (&x)[8], const NormWeight& nw, int chunk,
                                         float eps) {
    if (nw.w == nullptr) return;  // the same for the whole launch
    const float r = row_rstd<D>(x, eps);
    float w[8];
    load_weight8(nw, chunk, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= r * w[j];
}

}  // namespace fa
