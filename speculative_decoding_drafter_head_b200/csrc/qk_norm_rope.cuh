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
// What bounds it: HBM, every channel read and written once; but 8 channels a lane leave room for
// some 100 instructions only.  So a lane holds whole rotation pairs (4 channels from each half,
// or 8 neighbours when interleaved) and needs no exchange for them, and the weights times
// cosines and sines of its channels stay in registers for all heads of a row:
//     y_a = inv (w_a c x_a - w_b s x_b),  y_b = inv (w_a s x_a + w_b c x_b)
// (13000 rows of 48 heads of 128: 104 us with 16-byte chunks, shuffled partners and factors
// from shared memory).  One warp takes a row, four units of two (D = 128) heads in flight; with
// few rows the 8 warps of a CTA share one.  Measured (B200, device time): the 13000 rows 62 us,
// 5.2 TB/s of the 6.47 a copy reaches; 550 rows of the same heads 5.5 us, one row 3.7 us, which
// are a launch and two dependent loads.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace dspark {
namespace qknorm {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 64;                     // R / 2 <= 64
constexpr int kBlocks = 3;                        // CTAs to an SM, at least
constexpr int kInFlight = 2;                      // units a warp works on at once

struct Params {
    const uint16_t *qkv;          // [rows][stride], heads Hq + Hkv + Hkv
    long long stride;
    const uint16_t *q_weight, *k_weight;
    float eps;
    const float *inv_freq;
    int rot, interleaved;
    float rope_scale;
    const int32_t *position, *slot, *n_rows;
    int row_capacity, share;      // warps that share a row: 1 or 8
    int Hq, Hkv, ps, num_pages;
    uint16_t *q_out, *k_cache, *v_cache;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Factors of a lane's four pairs for queries or keys: y_a = ac x_a - bs x_b, y_b = as x_a + bc x_b.
struct Factors {
    float ac[4], bs[4], as[4], bc[4];
};

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kBlocks) qk_norm_rope_store_kernel(const Params p)
{
    constexpr int kLanes = D / 8;                 // lanes of a head
    constexpr int kHeads = 32 / kLanes;           // heads of a unit
    __shared__ float2 turn[kWarps][kMaxPairs];    // (cos, sin) of the CTA's rows

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    launch_dependents();
    wait_for_prior_kernels();
    const int n = min(max(*p.n_rows, 0), p.row_capacity);
    const int per_cta = kWarps / p.share;
    const int row0 = blockIdx.x * per_cta;
    const int rows = min(per_cta, n - row0);
    if (rows <= 0) return;
    const int pairs = p.rot / 2;
    const int r = warp / p.share, row = row0 + r;
    const bool live = r < rows;

    // the lane's channels: ca .. ca + 3 and cb .. cb + 3; pair i is (a_i, b_i) of its factors
    const int sub = lane % kLanes;
    const bool halves = !kInterleaved && 8 * sub < p.rot;
    const int ca = halves ? 4 * sub : 8 * sub, cb = halves ? pairs + 4 * sub : 8 * sub + 4;
    const bool turns = 8 * sub < p.rot;
    const int heads = p.Hq + 2 * p.Hkv;
    const int step = p.share * kHeads;            // heads from a warp's unit to its next
    const uint16_t *from = p.qkv + row * p.stride + ca;
    const int gap = cb - ca, first = (warp - r * p.share) * kHeads;

    // the next units' channels are on their way while these are worked on, the first ones
    // while the sines are
    uint2 na[kInFlight], nb[kInFlight];
    auto fetch = [&](int h0) {
#pragma unroll
        for (int f = 0; f < kInFlight; ++f) {
            const int head = h0 + f * step + lane / kLanes;
            na[f] = nb[f] = make_uint2(0, 0);
            if (head < heads) {
                const uint16_t *x = from + static_cast<size_t>(head) * D;
                na[f] = __ldg(reinterpret_cast<const uint2 *>(x));
                nb[f] = __ldg(reinterpret_cast<const uint2 *>(x + gap));
            }
        }
    };
    int slot = -1;
    if (live) {
        fetch(first);
        slot = p.slot[row];
    }
    for (int i = threadIdx.x; i < rows * pairs; i += kThreads) {
        const int t = i / pairs, j = i - t * pairs;
        // angle / pi in [-1, 1]: fraction of a turn, times two
        const double turned = static_cast<double>(p.position[row0 + t]) *
                              static_cast<double>(p.inv_freq[j]) * 0.15915494309189533577;
        float s, c;
        sincospif(2.0f * static_cast<float>(turned - rint(turned)), &s, &c);
        turn[t][j] = make_float2(c * p.rope_scale, s * p.rope_scale);
    }
    __syncthreads();
    if (!live) return;

    Factors fq, fk;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int xa = kInterleaved ? 8 * sub + 2 * i : ca + i;
        const int xb = kInterleaved ? xa + 1 : cb + i;
        float2 t = make_float2(1.0f, 0.0f);
        if (turns) t = turn[r][kInterleaved ? xa / 2 : xa];
        auto weight = [](const uint16_t *w, int ch) {
            return w ? __uint_as_float(static_cast<uint32_t>(__ldg(w + ch)) << 16) : 1.0f;
        };
        const float qa = weight(p.q_weight, xa), qb = weight(p.q_weight, xb);
        const float ka = weight(p.k_weight, xa), kb = weight(p.k_weight, xb);
        fq.ac[i] = qa * t.x, fq.bs[i] = qb * t.y, fq.as[i] = qa * t.y, fq.bc[i] = qb * t.x;
        fk.ac[i] = ka * t.x, fk.bs[i] = kb * t.y, fk.as[i] = ka * t.y, fk.bc[i] = kb * t.x;
    }
    const int page = slot / p.ps;
    const bool stored = slot >= 0 && page < p.num_pages;
    if (!stored && lane == 0) record_error(DSPARK_INVALID_PAGE);
    const size_t place =
        stored ? (static_cast<size_t>(page) * p.Hkv * p.ps + (slot - page * p.ps)) * D : 0;
    for (int u0 = first; u0 < heads; u0 += kInFlight * step) {
        const int h0 = u0 + lane / kLanes;
        uint2 xa[kInFlight], xb[kInFlight];
#pragma unroll
        for (int f = 0; f < kInFlight; ++f) xa[f] = na[f], xb[f] = nb[f];
        fetch(u0 + kInFlight * step);
#pragma unroll
        for (int f = 0; f < kInFlight; ++f) {
            const int head = h0 + f * step;
            if (u0 + f * step >= heads) break;
            float a[4] = {bf16lo_to_f32(xa[f].x), bf16hi_to_f32(xa[f].x), bf16lo_to_f32(xa[f].y),
                          bf16hi_to_f32(xa[f].y)};
            float b[4] = {bf16lo_to_f32(xb[f].x), bf16hi_to_f32(xb[f].x), bf16lo_to_f32(xb[f].y),
                          bf16hi_to_f32(xb[f].y)};
            float sq = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) sq = fmaf(a[i], a[i], fmaf(b[i], b[i], sq));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, o);
            if (kInterleaved) {                   // neighbours are the pairs
                const float t0 = a[1], t1 = a[3], t2 = b[0], t3 = b[2];
                a[1] = a[2], a[2] = t2, a[3] = t3;
                b[0] = t0, b[2] = b[1], b[1] = t1;
            }
            uint2 ya = xa[f], yb = xb[f];
            // queries or keys; values stay as they are
            auto turned = [&](const Factors &w, bool normed) {
                const float inv = normed ? rsqrtf(sq * (1.0f / D) + p.eps) : 1.0f;
                float u[4], v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (turns) {
                        u[i] = inv * (w.ac[i] * a[i] - w.bs[i] * b[i]);
                        v[i] = inv * (w.as[i] * a[i] + w.bc[i] * b[i]);
                    } else {                      // no zero times infinity
                        u[i] = inv * (w.ac[i] * a[i]);
                        v[i] = inv * (w.bc[i] * b[i]);
                    }
                }
                if (kInterleaved) {
                    ya = make_uint2(pack_bf16(u[0], v[0]), pack_bf16(u[1], v[1]));
                    yb = make_uint2(pack_bf16(u[2], v[2]), pack_bf16(u[3], v[3]));
                } else {
                    ya = make_uint2(pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3]));
                    yb = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
                }
            };
            uint16_t *to;
            if (head < p.Hq) {
                turned(fq, p.q_weight != nullptr);
                to = p.q_out + (static_cast<size_t>(row) * p.Hq + head) * D;
            } else {
                const bool key = head < p.Hq + p.Hkv;
                if (key) turned(fk, p.k_weight != nullptr);
                to = (key ? p.k_cache : p.v_cache) + place +
                     static_cast<size_t>(head - p.Hq - (key ? 0 : p.Hkv)) * p.ps * D;
                if (!stored) continue;
            }
            if (head < heads) {
                *reinterpret_cast<uint2 *>(to + ca) = ya;
                *reinterpret_cast<uint2 *>(to + cb) = yb;
            }
        }
    }
}

}  // namespace qknorm
}  // namespace dspark
