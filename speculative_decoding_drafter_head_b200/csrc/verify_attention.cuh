// verify_attention.cuh -- attention of a verification batch's rows over the paged cache.
//
// Row r_b + i of request b stands at position context[b] + i and sees keys 0 .. context[b]+i:
//     out[r, h] = sum_j softmax_j(scale q[r, h] . k[j, h / g]) v[j, h / g]
// with j running over the request's block table and g = Hq / Hkv query heads to a key head.
//
// One CTA per (row, query head): each thread scores one key of a tile of 128, the softmax's
// maximum and sum run along the tiles (fp32), and each thread then adds up one channel.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"

namespace dspark {
namespace vattn {

constexpr int kThreads = 128;
constexpr int kMaxB = 4096;

struct Params {
    const uint16_t *q, *k_cache, *v_cache;
    const int32_t *pages, *context, *row_start;
    int B, row_capacity, Hq, Hkv, ps, max_pages, num_pages;
    float scale;
    uint16_t *out;
};

template <int D>
__global__ void __launch_bounds__(kThreads) verify_attention_kernel(const Params p)
{
    __shared__ float q_s[D], p_s[kThreads], red[4];
    __shared__ const uint16_t *v_s[kThreads];
    const int row = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
    if (row >= min(max(p.row_start[p.B], 0), p.row_capacity)) return;
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.row_start[mid] <= row) lo = mid;
        else hi = mid - 1;
    }
    const int b = lo;
    const size_t at = (static_cast<size_t>(row) * p.Hq + h) * D;
    if (tid < D) q_s[tid] = __uint_as_float(static_cast<uint32_t>(p.q[at + tid]) << 16);
    __syncthreads();
    const int kvh = h / (p.Hq / p.Hkv);
    const long long room = static_cast<long long>(p.max_pages) * p.ps;
    const long long wants = static_cast<long long>(max(p.context[b], 0)) + row - p.row_start[b] + 1;
    if (wants > room) record_error(DSPARK_INVALID_TOKEN);
    const int len = static_cast<int>(min(wants, room));
    float m = -INFINITY, l = 0.0f, acc = 0.0f;
    for (int j0 = 0; j0 < len; j0 += kThreads) {
        const int j = j0 + tid;
        float s = -INFINITY;
        if (j < len) {
            int page = p.pages[static_cast<size_t>(b) * p.max_pages + j / p.ps];
            if (page < 0 || page >= p.num_pages) {
                record_error(DSPARK_INVALID_PAGE);
                page = 0;
            }
            const size_t off = ((static_cast<size_t>(page) * p.Hkv + kvh) * p.ps + j % p.ps) * D;
            const uint4 *k = reinterpret_cast<const uint4 *>(p.k_cache + off);
            v_s[tid] = p.v_cache + off;
            s = 0.0f;
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
                const uint4 w = k[c];
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s = fmaf(bf16lo_to_f32(u[e]), q_s[8 * c + 2 * e], s);
                    s = fmaf(bf16hi_to_f32(u[e]), q_s[8 * c + 2 * e + 1], s);
                }
            }
            s *= p.scale;
        }
        float t = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
        if ((tid & 31) == 0) red[tid >> 5] = t;
        __syncthreads();
        t = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        const float f = m == -INFINITY ? 0.0f : expf(m - t);
        m = t;
        const float e = j < len ? expf(s - m) : 0.0f;
        p_s[tid] = e;
        const float w = warp_sum(e);
        __syncthreads();
        if ((tid & 31) == 0) red[tid >> 5] = w;
        __syncthreads();
        l = l * f + (red[0] + red[1]) + (red[2] + red[3]);
        if (tid < D) {
            acc *= f;
            for (int i = 0; i < min(kThreads, len - j0); ++i)
                acc = fmaf(p_s[i], __uint_as_float(static_cast<uint32_t>(v_s[i][tid]) << 16), acc);
        }
        __syncthreads();
    }
    if (tid < D) {
        const __nv_bfloat16 o = __float2bfloat16_rn(acc / l);
        p.out[at + tid] = *reinterpret_cast<const uint16_t *>(&o);
    }
}

}  // namespace vattn
}  // namespace dspark
