// decode_fp8_sm100.cu -- single-token decode over a paged cache of 8-bit
// values (e4m3) with one scale for each block of tokens and head.
#include <cuda_fp8.h>

#include <cmath>

#include "fa_internal.h"
#include "rope_row.cuh"

namespace fa {
namespace {

constexpr int kPage = 256;
constexpr int kThreads = 128;

struct DecodeFp8 {
    const __nv_bfloat16* q;
    const uint8_t *kp, *vp;
    const float *ks, *vs;
    const int32_t *table, *lens;
    __nv_bfloat16* o;
    float* lse;
    int B, H, Hk, num_pages, table_len, max_pages, block_log2;
    float scale_log2;
    unsigned int* err;
};

__device__ __forceinline__ float code_value(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// One CTA per (sequence, query head); 128 tokens at a time: a thread scores
// one token, then sums one output column (two threads' share for D = 64).
template <int D>
__global__ void __launch_bounds__(kThreads) fa_decode_fp8_kernel(const DecodeFp8 p) {
    __shared__ float q[D], prob[kThreads], red[kThreads / 32];
    __shared__ unsigned long long base_sh;
    const int b = blockIdx.x / p.H, h = blockIdx.x - b * p.H, hk = h / (p.H / p.Hk);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < D) q[tid] = __bfloat162float(p.q[(static_cast<int64_t>(b) * p.H + h) * D + tid]) * p.scale_log2;
    if (tid == 0) base_sh = 0;
    __syncthreads();
    int len = max(p.lens[b], 0);
    if (p.max_pages == 0) {
        unsigned long long mine = 0;
        for (int i = tid; i < b; i += kThreads) {
            const int n = max(p.lens[i], 0);
            mine += n / kPage + (n % kPage != 0);
        }
        if (mine) atomicAdd(&base_sh, mine);
    }
    if (p.lens[b] < 0 && tid == 0) record_error(p.err, FA_DEVERR_BAD_INPUT);
    __syncthreads();
    const int64_t base = p.max_pages ? static_cast<int64_t>(b) * p.max_pages
                                     : static_cast<int64_t>(base_sh);
    const int64_t room = p.max_pages ? p.max_pages : p.table_len > base ? p.table_len - base : 0;
    if (len > room * kPage) {
        if (tid == 0) record_error(p.err, FA_DEVERR_BAD_INPUT);
        len = static_cast<int>(room * kPage);
    }
    float m = -INFINITY, l = 0.f, acc = 0.f;
    for (int t0 = 0; t0 < len; t0 += kThreads) {
        int page = p.table[base + t0 / kPage];
        if (page < 0 || page >= p.num_pages) {
            if (tid == 0) record_error(p.err, FA_DEVERR_BAD_INPUT);
            page = 0;
        }
        const int64_t slice = static_cast<int64_t>(page) * p.Hk + hk;
        const int t = t0 + tid, slot = t % kPage, nb = kPage >> p.block_log2;
        float s = -INFINITY;
        if (t < len) {
            s = 0.f;
            const uint8_t* k = p.kp + (slice * kPage + slot) * D;
            for (int c = 0; c < D; ++c) s += q[c] * code_value(k[c]);
            s *= p.ks[slice * nb + (slot >> p.block_log2)];
        }
        float top = s;
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) red[warp] = top;
        __syncthreads();
        for (int i = 0; i < kThreads / 32; ++i) top = fmaxf(top, red[i]);
        const float m2 = fmaxf(m, top), old = exp2f(m - m2);
        m = m2;
        prob[tid] = t < len ? exp2f(s - m2) : 0.f;
        __syncthreads();
        acc *= old;
        l *= old;
        const int n = min(kThreads, len - t0);
        for (int i = 0; i < n; ++i) {
            l += prob[i];
            if (tid < D) {
                const int sl = (t0 + i) % kPage;
                acc += prob[i] * p.vs[slice * nb + (sl >> p.block_log2)] *
                       code_value(p.vp[(slice * kPage + sl) * D + tid]);
            }
        }
        __syncthreads();
    }
    const int64_t row = static_cast<int64_t>(b) * p.H + h;
    if (tid < D) p.o[row * D + tid] = __float2bfloat16(len > 0 ? acc / l : 0.f);
    if (tid == 0 && p.lse) p.lse[row] = len > 0 ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace fa

extern "C" {

int fa_decode_paged_fp8_workspace(int B, int H, int H_kv, int d, int* bytes) {
    if (!bytes) return FA_ERR_NULL;
    if (B < 1 || H < 1 || H_kv < 1 || H % H_kv != 0) return FA_ERR_SHAPE;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    *bytes = 0;
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
    p.num_pages = num_pages;
    p.table_len = table_len;
    p.max_pages = max_pages;
    while ((1 << p.block_log2) < block) ++p.block_log2;
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d == 64) fa::fa_decode_fp8_kernel<64><<<B * H, fa::kThreads, 0, st>>>(p);
    else fa::fa_decode_fp8_kernel<128><<<B * H, fa::kThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
