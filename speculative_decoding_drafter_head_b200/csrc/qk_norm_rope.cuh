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
// What bounds it: HBM, every channel read and written once, which takes some 70 KB on their way
// to each SM: more than registers hold beside the arithmetic, so channels go to shared memory
// first (13000 rows of 48 heads of 128: 62.4 us with two units of 512 bytes ahead in registers,
// 55.6 with six in shared memory, 56.3 with four, 57.5 with ten).  8 channels a lane leave room for
// some 100 instructions.  So a lane holds whole rotation pairs (4 channels from each half,
// or 8 neighbours when interleaved) and needs no exchange for them, and the weights times
// cosines and sines of its channels stay in registers for all heads of a row:
//     y_a = inv (w_a c x_a - w_b s x_b),  y_b = inv (w_a s x_a + w_b c x_b)
// (the same rows: 104 us with 16-byte chunks, shuffled partners and factors from shared memory).
// One warp takes a row, by units of two (D = 128) heads; with few rows up to 8 warps share one.
// Measured (B200, device time): the 13000 rows 56 us, 5.8 TB/s of the 6.47 a copy reaches; 550
// rows of the same heads 5.7 us, one row 2.9 us, which are a launch and two dependent loads.
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
constexpr int kAhead = 3;                         // and so many times that on their way

struct Params {
    const uint16_t *qkv;          // [rows][stride], heads Hq + Hkv + Hkv
    long long stride;
    const uint16_t *q_weight, *k_weight;
    float eps;
    const float *inv_freq;
    int rot, interleaved;
    float rope_scale;
    const int32_t *position, *slot, *n_rows;
    int row_capacity, share;      // warps that share a row: 1, 2, 4 or 8
    int Hq, Hkv, ps, num_pages;
    uint16_t *q_out, *k_cache, *v_cache;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The lane's four pairs (a_i, b_i) from its channels ca .. ca + 3 and cb .. cb + 3.
template <bool kInterleaved>
__device__ __forceinline__ void pairs_of(uint2 x, uint2 y, float (&a)[4], float (&b)[4])
{
    const float u[4] = {bf16lo_to_f32(x.x), bf16hi_to_f32(x.x), bf16lo_to_f32(x.y),
                        bf16hi_to_f32(x.y)};
    const float v[4] = {bf16lo_to_f32(y.x), bf16hi_to_f32(y.x), bf16lo_to_f32(y.y),
                        bf16hi_to_f32(y.y)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = !kInterleaved ? u[i] : i < 2 ? u[2 * i] : v[2 * i - 4];   // neighbours are the pairs
        b[i] = !kInterleaved ? v[i] : i < 2 ? u[2 * i + 1] : v[2 * i - 3];
    }
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
    __shared__ uint2 ring[kWarps][kAhead][kInFlight][2][32];   // channels, each lane's own

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

    // the next units' channels are on their way to shared memory while these are worked on, the
    // first ones while the sines are; a lane reads what it copied itself, so nobody else waits
    auto fetch = [&](int u, int at) {
#pragma unroll
        for (int f = 0; f < kInFlight; ++f) {
            const int head = u + f * step + lane / kLanes;
            if (head < heads) {
                const uint16_t *x = from + static_cast<size_t>(head) * D;
                cp_async_8(smem_u32(&ring[warp][at][f][0][lane]), x);
                cp_async_8(smem_u32(&ring[warp][at][f][1][lane]), x + gap);
            }
        }
        cp_async_commit();
    };
    int slot = -1;
    uint2 wq[2], wk[2];                           // weights of the lane's channels, or ones
    wq[0] = wq[1] = wk[0] = wk[1] = make_uint2(0x3F803F80u, 0x3F803F80u);
    if (live) {
        if (p.q_weight) {
            wq[0] = *reinterpret_cast<const uint2 *>(p.q_weight + ca);
            wq[1] = *reinterpret_cast<const uint2 *>(p.q_weight + cb);
        }
        if (p.k_weight) {
            wk[0] = *reinterpret_cast<const uint2 *>(p.k_weight + ca);
            wk[1] = *reinterpret_cast<const uint2 *>(p.k_weight + cb);
        }
#pragma unroll
        for (int at = 0; at < kAhead; ++at) fetch(first + at * kInFlight * step, at);
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
    float qa[4], qb[4], ka[4], kb[4];
    pairs_of<kInterleaved>(wq[0], wq[1], qa, qb);
    pairs_of<kInterleaved>(wk[0], wk[1], ka, kb);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = turns ? turn[r][4 * sub + i] : make_float2(1.0f, 0.0f);
        fq.ac[i] = qa[i] * t.x, fq.bs[i] = qb[i] * t.y, fq.as[i] = qa[i] * t.y, fq.bc[i] = qb[i] * t.x;
        fk.ac[i] = ka[i] * t.x, fk.bs[i] = kb[i] * t.y, fk.as[i] = ka[i] * t.y, fk.bc[i] = kb[i] * t.x;
    }
    const int page = slot / p.ps;
    const bool stored = slot >= 0 && page < p.num_pages;
    if (!stored && lane == 0) record_error(DSPARK_INVALID_PAGE);
    const size_t place =
        stored ? (static_cast<size_t>(page) * p.Hkv * p.ps + (slot - page * p.ps)) * D : 0;
    int at = 0;
    for (int u0 = first; u0 < heads; u0 += kInFlight * step) {
        const int h0 = u0 + lane / kLanes;
        uint2 xa[kInFlight], xb[kInFlight];
        cp_async_wait<kAhead - 1>();
#pragma unroll
        for (int f = 0; f < kInFlight; ++f)
            xa[f] = ring[warp][at][f][0][lane], xb[f] = ring[warp][at][f][1][lane];
        fetch(u0 + kAhead * kInFlight * step, at);
        if (++at == kAhead) at = 0;
#pragma unroll
        for (int f = 0; f < kInFlight; ++f) {
            const int head = h0 + f * step;
            if (u0 + f * step >= heads) break;
            float a[4], b[4];
            pairs_of<kInterleaved>(xa[f], xb[f], a, b);
            float sq = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) sq = fmaf(a[i], a[i], fmaf(b[i], b[i], sq));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, o);
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
