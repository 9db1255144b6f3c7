// qk_norm_rope.cuh -- queries and keys normalised and rotated, keys and values stored.
//
// For row t of a verification batch (position m, cache slot s) and each query or key head x
// of D channels:
//     y = x / sqrt(mean(x^2) + eps) w                         (when a weight is given)
//     (a, b) -> c (a cos - b sin, a sin + b cos),  angle = m inv_freq[j]
// over the pairs (j, j + R/2), or (2j, 2j + 1) when interleaved, of the first R channels;
// c = rope_scale.  Queries go to q_out, keys and values into the paged cache at slot s.
//
// Numerics: everything between the bf16 input and the one rounding of the bf16 output is
// fp32.  The angle is the exact fp64 product of the position and the fp32 frequency, and is
// reduced to a fraction of a turn in fp64 before the fp32 sine and cosine: an fp32 product
// would be off by 2^-24 m radians (0.06 at a position of a million).
//
// What bounds it: HBM, every channel read and written once.  A thread holds 8 channels (one
// 16-byte load and store), so a head is D / 8 neighbouring lanes and its mean and its
// rotation partners are shuffles.  The sines of a row are formed once per CTA, in shared
// memory, and serve all its heads.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"

namespace dspark {
namespace qknorm {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 64;                     // R / 2 <= 64
constexpr int kMaxTile = 4;                       // rows per CTA

struct Params {
    const uint16_t *qkv;          // [rows][stride], heads Hq + Hkv + Hkv
    long long stride;
    const uint16_t *q_weight, *k_weight;
    float eps;
    const float *inv_freq;
    int rot, interleaved;
    float rope_scale;
    const int32_t *position, *slot, *n_rows;
    int row_capacity, tile;       // rows per CTA
    int Hq, Hkv, ps, num_pages;
    uint16_t *q_out, *k_cache, *v_cache;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <int D>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_store_kernel(const Params p)
{
    constexpr int kLanes = D / 8;                 // lanes of a head
    constexpr int kHeadsPerWarp = 32 / kLanes;
    __shared__ float2 turn[kMaxTile][kMaxPairs];  // (cos, sin) of the tile's rows

    const int n = min(max(*p.n_rows, 0), p.row_capacity);
    const int row0 = blockIdx.x * p.tile;
    const int rows = min(p.tile, n - row0);
    if (rows <= 0) return;
    const int pairs = p.rot / 2;
    for (int i = threadIdx.x; i < rows * pairs; i += kThreads) {
        const int r = i / pairs, j = i - r * pairs;
        // angle / pi in (-1, 1]: fraction of a turn, times two
        const double turns = static_cast<double>(p.position[row0 + r]) *
                             static_cast<double>(p.inv_freq[j]) * 0.15915494309189533577;
        const float half = 2.0f * static_cast<float>(turns - rint(turns));
        float s, c;
        sincospif(half, &s, &c);
        turn[r][j] = make_float2(c * p.rope_scale, s * p.rope_scale);
    }
    __syncthreads();

    const int lane = threadIdx.x & 31;
    const int sub = lane % kLanes, ch = sub * 8;  // this lane's place in its head
    const int heads = p.Hq + 2 * p.Hkv;
    const int groups = (heads + kHeadsPerWarp - 1) / kHeadsPerWarp;
    for (int u = threadIdx.x >> 5; u < rows * groups; u += kWarps) {
        const int r = u / groups;
        const int head = (u - r * groups) * kHeadsPerWarp + lane / kLanes;
        const bool live = head < heads;
        const int row = row0 + r;
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (live)
            raw = __ldg(reinterpret_cast<const uint4 *>(p.qkv + row * p.stride +
                                                        static_cast<long long>(head) * D + ch));
        const bool is_q = head < p.Hq, is_v = head >= p.Hq + p.Hkv;
        float y[8] = {bf16lo_to_f32(raw.x), bf16hi_to_f32(raw.x), bf16lo_to_f32(raw.y),
                      bf16hi_to_f32(raw.y), bf16lo_to_f32(raw.z), bf16hi_to_f32(raw.z),
                      bf16lo_to_f32(raw.w), bf16hi_to_f32(raw.w)};
        // the mean and the partners of every lane, values included: shuffles need all lanes
        float sq = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fmaf(y[i], y[i], sq);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, o);
        const uint16_t *w = is_q ? p.q_weight : p.k_weight;
        if (w && !is_v) {
            const float inv = rsqrtf(sq * (1.0f / D) + p.eps);
            const uint4 ww = __ldg(reinterpret_cast<const uint4 *>(w + ch));
            const float wf[8] = {bf16lo_to_f32(ww.x), bf16hi_to_f32(ww.x), bf16lo_to_f32(ww.y),
                                 bf16hi_to_f32(ww.y), bf16lo_to_f32(ww.z), bf16hi_to_f32(ww.z),
                                 bf16lo_to_f32(ww.w), bf16hi_to_f32(ww.w)};
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = y[i] * inv * wf[i];
        }
        if (p.rot) {
            if (p.interleaved) {
                if (!is_v && ch < p.rot) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 t = turn[r][(ch + i) >> 1];
                        const float a = y[i], b = y[i + 1];
                        y[i] = a * t.x - b * t.y;
                        y[i + 1] = a * t.y + b * t.x;
                    }
                }
            } else {
                // channels j and j + R/2 stand R/16 lanes apart
                const bool low = ch < pairs;
                const int from = low ? lane + pairs / 8 : lane - pairs / 8;
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xFFFFFFFFu, y[i], from & 31);
                if (!is_v && ch < p.rot) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 t = turn[r][low ? ch + i : ch + i - pairs];
                        y[i] = low ? y[i] * t.x - o[i] * t.y : o[i] * t.y + y[i] * t.x;
                    }
                }
            }
        }
        if (!live) continue;
        const uint4 out = is_v ? raw
                               : make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]),
                                            pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
        if (is_q) {
            *reinterpret_cast<uint4 *>(p.q_out + (static_cast<size_t>(row) * p.Hq + head) * D +
                                       ch) = out;
            continue;
        }
        const int slot = p.slot[row];
        const int page = slot / p.ps;
        if (slot < 0 || page >= p.num_pages) {
            record_error(DSPARK_INVALID_PAGE);
            continue;
        }
        const int h = head - p.Hq - (is_v ? p.Hkv : 0);
        uint16_t *cache = is_v ? p.v_cache : p.k_cache;
        *reinterpret_cast<uint4 *>(
            cache + ((static_cast<size_t>(page) * p.Hkv + h) * p.ps + (slot - page * p.ps)) * D +
            ch) = out;
    }
}

}  // namespace qknorm
}  // namespace dspark
