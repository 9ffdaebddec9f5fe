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
// the table's reads twice as many: 88 us instead of 69 for 16384 tokens of 40
// heads.)  Values are held in pairs for the instructions that take two at a time,
// which with slots found without a division made that 60.  R is a multiple of 16,
// so the 4 lie in one half.  The rotation
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

// A lane's 8 values of a row as 4 pairs of fp32, for the instructions that take
// two at a time: where the lane is rotated, a[0], a[1] are the first values of
// its 4 rotation pairs and b[0], b[1] the second.
struct Vec8 {
    uint64_t a[2], b[2];
};

// Which 8 values of a row a lane holds: 4 from `lo` on and 4 from `hi` on
// (interleaved: 8 from `lo` on); and whether they are 4 pairs of the rotated part.
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

    static __device__ __forceinline__ Vec8 unpack(const uint4& v) {
        Vec8 x;
        if (INTER) {
            x.a[0] = f2_pack(bf16_lo(v.x), bf16_lo(v.y));
            x.a[1] = f2_pack(bf16_lo(v.z), bf16_lo(v.w));
            x.b[0] = f2_pack(bf16_hi(v.x), bf16_hi(v.y));
            x.b[1] = f2_pack(bf16_hi(v.z), bf16_hi(v.w));
        } else {
            x.a[0] = f2_pack(bf16_lo(v.x), bf16_hi(v.x));
            x.a[1] = f2_pack(bf16_lo(v.y), bf16_hi(v.y));
            x.b[0] = f2_pack(bf16_lo(v.z), bf16_hi(v.z));
            x.b[1] = f2_pack(bf16_lo(v.w), bf16_hi(v.w));
        }
        return x;
    }
    // The values in the order of the row: `lo` .. lo + 3, then `hi` .. hi + 3.
    static __device__ __forceinline__ void in_order(const Vec8& x, float (&y)[8]) {
        if (INTER) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                y[4 * j] = f2_lo(x.a[j]);
                y[4 * j + 1] = f2_lo(x.b[j]);
                y[4 * j + 2] = f2_hi(x.a[j]);
                y[4 * j + 3] = f2_hi(x.b[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                y[2 * j] = f2_lo(x.a[j]);
                y[2 * j + 1] = f2_hi(x.a[j]);
                y[4 + 2 * j] = f2_lo(x.b[j]);
                y[5 + 2 * j] = f2_hi(x.b[j]);
            }
        }
    }
    static __device__ __forceinline__ Vec8 of(const float (&y)[8]) {
        Vec8 x;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x.a[j] = INTER ? f2_pack(y[4 * j], y[4 * j + 2]) : f2_pack(y[2 * j], y[2 * j + 1]);
            x.b[j] =
                INTER ? f2_pack(y[4 * j + 1], y[4 * j + 3]) : f2_pack(y[4 + 2 * j], y[5 + 2 * j]);
        }
        return x;
    }
    static __device__ __forceinline__ uint4 pack(const Vec8& x) {
        float y[8];
        in_order(x, y);
        return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                          pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    }

    // the lane's weights
    __device__ __forceinline__ Vec8 weights(const NormWeight& nw) const {
        if (!nw.fp32) {
            const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(nw.w);
            const uint2 a = __ldg(reinterpret_cast<const uint2*>(p + lo));
            const uint2 b = __ldg(reinterpret_cast<const uint2*>(p + hi));
            return unpack(make_uint4(a.x, a.y, b.x, b.y));
        }
        const float* p = static_cast<const float*>(nw.w);
        const float4 a = __ldg(reinterpret_cast<const float4*>(p + lo));
        const float4 b = __ldg(reinterpret_cast<const float4*>(p + hi));
        const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        return of(y);
    }
};

// A position's rotation of a lane's 4 pairs.
template <int D, bool INTER>
struct Rotation {
    uint64_t c[2], s[2];
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
        c[0] = f2_pack(cv.x, cv.y);
        c[1] = f2_pack(cv.z, cv.w);
        s[0] = BACK ? f2_pack(-sv.x, -sv.y) : f2_pack(sv.x, sv.y);
        s[1] = BACK ? f2_pack(-sv.z, -sv.w) : f2_pack(sv.z, sv.w);
    }

    __device__ __forceinline__ void apply(Vec8& y) const {
        if (on) turn(y);
    }
    // (of a lane that `on` holds for)
    __device__ __forceinline__ void turn(Vec8& y) const {
        const uint64_t minus = f2_pack(-1.f, -1.f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint64_t a = y.a[j], b = y.b[j];
            // products rounded, then their difference (exact times -1) and sum
            // (one by one: ptxas contracts a packed sum of packed products)
            y.a[j] = f2_fma(f2_mul(b, s[j]), minus, f2_mul(a, c[j]));
            const uint64_t bc = f2_mul(b, c[j]), as = f2_mul(a, s[j]);
            y.b[j] = f2_pack(__fadd_rn(f2_lo(bc), f2_lo(as)), __fadd_rn(f2_hi(bc), f2_hi(as)));
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

__device__ __forceinline__ float dot8(const Vec8& x, const Vec8& y) {
    uint64_t d = f2_mul(x.a[0], y.a[0]);
    d = f2_fma(x.a[1], y.a[1], d);
    d = f2_fma(x.b[0], y.b[0], d);
    d = f2_fma(x.b[1], y.b[1], d);
    return f2_lo(d) + f2_hi(d);
}

__device__ __forceinline__ Vec8 mul8(const Vec8& x, const Vec8& y) {
    Vec8 z;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        z.a[j] = f2_mul(x.a[j], y.a[j]);
        z.b[j] = f2_mul(x.b[j], y.b[j]);
    }
    return z;
}

__device__ __forceinline__ Vec8 scale8(const Vec8& x, float r) {
    const uint64_t rr = f2_pack(r, r);
    Vec8 z;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        z.a[j] = f2_mul(x.a[j], rr);
        z.b[j] = f2_mul(x.b[j], rr);
    }
    return z;
}

// 1 / sqrt(mean(x^2) + eps) of a row.
template <int D>
__device__ __forceinline__ float row_rstd(const Vec8& x, float eps) {
    return rsqrtf(fmaf(row_sum<D>(dot8(x, x)), 1.f / D, eps));
}

// x normed by the lane's weights (every lane of the row together).
template <int D>
__device__ __forceinline__ Vec8 norm_row(const Vec8& x, const Vec8& w, float eps) {
    return mul8(x, scale8(w, row_rstd<D>(x, eps)));
}

}  // namespace fa
