// rope_row.cuh -- one head row (D values) normed and rotated by D/8 lanes of a
// warp, 8 values each: shared by the kernels that norm and rotate queries and
// keys and by the cache appends.
//
// With x the row, w its weight, R the rotated part and (c_i, s_i) the table's
// entries of the row's position,
//     y  = x * rsqrt(mean(x^2) + eps) * w            (y = x without a weight)
//     (y_a, y_b) -> (y_a c_i - y_b s_i, y_b c_i + y_a s_i)   for the R/2 pairs
// where pair i is (i, i + R/2) (halves) or (2i, 2i + 1) (interleaved), and the
// values from R on stay.  A lane holds 4 whole pairs: 8 consecutive values
// where the pairs are interleaved, 4 from each half where they are not (two
// 8-byte loads instead of one of 16), so a rotation needs no exchange between
// lanes and each lane reads 4 cosines and 4 sines only.  (With 8 consecutive
// values of the halves layout in a lane, the exchange was 8 shuffles a row and
// the table's reads twice as many: 88 us instead of 62 for 16384 tokens of 40
// heads.)  R is a multiple of 16, so the 4 lie in one half.  The rotation
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

// Which 8 values of a row a lane holds: 4 from `lo` on and 4 from `hi` on; and
// whether they are 4 pairs of the rotated part.
template <int D, bool INTER>
struct Lane {
    int chunk, lo, hi;
    bool turns;

    __device__ __forceinline__ explicit Lane(int half) {
        chunk = threadIdx.x % (D / 8);
        turns = 4 * chunk < half;
        lo = !INTER && turns ? 4 * chunk : 8 * chunk;
        hi = !INTER && turns ? 4 * chunk + half : 8 * chunk + 4;
    }

    // raw bf16 of a row (read once)
    __device__ __forceinline__ uint4 load(const __nv_bfloat16* row) const {
        if (INTER) return __ldcs(reinterpret_cast<const uint4*>(row + lo));
        const uint2 a = __ldcs(reinterpret_cast<const uint2*>(row + lo));
        const uint2 b = __ldcs(reinterpret_cast<const uint2*>(row + hi));
        return make_uint4(a.x, a.y, b.x, b.y);
    }
    __device__ __forceinline__ void store(__nv_bfloat16* row, const uint4& v) const {
        if (INTER) {
            *reinterpret_cast<uint4*>(row + lo) = v;
        } else {
            *reinterpret_cast<uint2*>(row + lo) = make_uint2(v.x, v.y);
            *reinterpret_cast<uint2*>(row + hi) = make_uint2(v.z, v.w);
        }
    }
    // 8-bit values of a row
    __device__ __forceinline__ uint2 load(const uint8_t* row) const {
        if (INTER) return *reinterpret_cast<const uint2*>(row + lo);
        return make_uint2(*reinterpret_cast<const uint32_t*>(row + lo),
                          *reinterpret_cast<const uint32_t*>(row + hi));
    }
    __device__ __forceinline__ void store(uint8_t* row, const uint2& v) const {
        if (INTER) {
            *reinterpret_cast<uint2*>(row + lo) = v;
        } else {
            *reinterpret_cast<uint32_t*>(row + lo) = v.x;
            *reinterpret_cast<uint32_t*>(row + hi) = v.y;
        }
    }
    // the lane's weights
    __device__ __forceinline__ void weights(const NormWeight& nw, float (&w)[8]) const {
        if (nw.fp32) {
            const float* p = static_cast<const float*>(nw.w);
            const float4 a = __ldg(reinterpret_cast<const float4*>(p + lo));
            const float4 b = __ldg(reinterpret_cast<const float4*>(p + hi));
            w[0] = a.x;
            w[1] = a.y;
            w[2] = a.z;
            w[3] = a.w;
            w[4] = b.x;
            w[5] = b.y;
            w[6] = b.z;
            w[7] = b.w;
        } else {
            const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(nw.w);
            const uint2 a = __ldg(reinterpret_cast<const uint2*>(p + lo));
            const uint2 b = __ldg(reinterpret_cast<const uint2*>(p + hi));
            unpack8(make_uint4(a.x, a.y, b.x, b.y), w);
        }
    }
};

// A position's rotation of a lane's 4 pairs.
template <int D, bool INTER>
struct Rotation {
    float c[4], s[4];
    bool on;

    // pos in [0, max_pos); BACK turns back (the transpose, for gradients)
    template <bool BACK = false>
    __device__ __forceinline__ void load(const RopeTable& t, int pos,
                                         const Lane<D, INTER>& lane) {
        on = lane.turns;
        float4 cv = make_float4(1.f, 1.f, 1.f, 1.f), sv = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on) {
            const int64_t at = static_cast<int64_t>(pos) * t.half + 4 * lane.chunk;
            cv = __ldg(reinterpret_cast<const float4*>(t.cos_t + at));
            sv = __ldg(reinterpret_cast<const float4*>(t.sin_t + at));
        }
        c[0] = cv.x;
        c[1] = cv.y;
        c[2] = cv.z;
        c[3] = cv.w;
        s[0] = BACK ? -sv.x : sv.x;
        s[1] = BACK ? -sv.y : sv.y;
        s[2] = BACK ? -sv.z : sv.z;
        s[3] = BACK ? -sv.w : sv.w;
    }

    __device__ __forceinline__ void apply(float (&y)[8]) const {
        if (!on) return;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float &a = y[INTER ? 2 * j : j], &b = y[INTER ? 2 * j + 1 : j + 4];
            const float ra = __fsub_rn(__fmul_rn(a, c[j]), __fmul_rn(b, s[j]));
            b = __fadd_rn(__fmul_rn(b, c[j]), __fmul_rn(a, s[j]));
            a = ra;
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

// x normed by the lane's weights, in place (every lane of the row together).
template <int D>
__device__ __forceinline__ void norm_row(float (&x)[8], const float (&w)[8], float eps) {
    const float r = row_rstd<D>(x, eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= r * w[j];
}

}  // namespace fa
