// verify_attention.cuh -- attention of a verification batch's rows over the paged cache.
//
// Row r_b + i of request b stands at position context[b] + i and sees keys 0 .. context[b]+i:
//     out[r, h] = sum_j softmax_j(scale q[r, h] . k[j, h / g]) v[j, h / g]
// with j running over the request's block table and g = Hq / Hkv query heads to a key head.
//
// What bounds it: HBM.  The cache is read once, 4 D bytes for a key and its value, and serves
// the n = (L + 1) g rows that share a key head (17 x 4 at most at the benchmark's shapes): n
// flops a byte, far below the tensor cores' 250.  So the keys, not the rows, fill the 128
// lanes of an MMA, and no lane is padding whatever n is:
//     S^T [128 keys x n] = K Q^T         A = K tile (K-major), B = Q (K-major)
//     O^T [D x n] += V^T P               A = V tile (M-major), B = P [keys x n] (N-major)
//     l [n]       += 1^T P               A = ones (64 x 16), the softmax's sum
// n is rounded up to 16 for each unit of work.  The sum comes from the tensor core for the
// price of A's rows, in fp32, of the same rounded weights as O; no thread adds up anything.
//
// Softmax: a thread owns one key and all n rows.  exp2 needs a reference m per row that keeps
// the weights in range, not the maximum itself: m is the maximum over the unit's first key
// tile, and stays until some score exceeds it by more than 2^24 in weight; then m rises to the
// new maximum and O and l are scaled (one vote a tile, folded into the barrier that a tile
// needs anyway).  bf16 weights keep their 8 bits at any magnitude, and O and l are fp32, so
// a stale m costs no accuracy.  A row without a finite score so far has an m below any, so that
// its first one raises it.  A weight's exponent is one fma, score scale - m; but m is a rounded
// product itself, by up to 16 and more from |m| = 2^28 on, so there the product is rounded as m
// was and the maximum's exponent is zero again (a step's other rows, which lose nothing that counts
// by it, go the same way).  The weights are rounded to bf16 (by 2^-8 of each at most, as the
// output itself), which is what the tensor core's second product asks for: against 64 bits the
// output is off by 0.0021 to 0.0024 of its norm, where rounding it alone makes 0.0017.
//
// Masks: key j is seen by the rows from (j - context) g on, so a thread compares the row's
// number with one number of its own.  Values behind the last key are cleared in shared memory
// (0 x NaN is NaN); values of the step's own rows that are not finite are cleared as well and
// added at the end to the rows that see them, so that they reach no row that does not.
//
// Work: key tiles in one line, an equal share for each of 148 CTAs (verify_plan.h), because
// lengths are known to the device alone and differ by orders of magnitude.  Units cut by a
// border leave (m, l, O) in the workspace, and verify_join_kernel adds the parts up, in
// order, so results do not depend on timing.  It is launched to overlap with this kernel's end.
//
// Warps: 0-3 and 4-7 softmax and output (thread = key of the tile, then channel of the output),
// the groups taking tiles in turn, 8 and 9 copy K and V pages into rings of 32 KB tiles by TMA
// (one box a page and 64 channels; one warp for both took 90 cycles a box, 3000 of a tile's
// 2800 with pages of 16), 10 issues the MMAs, 11 copies Q.  S is double-buffered and P at least
// (three buffers where rows are 64), so S of the next tiles and O of the last run beside the
// softmax.
//
// Measured (B200, device time): 64 requests, 32/8 heads of 128, 500-8000 keys, up to 17 rows
// each 177 us, 6.2 TB/s of the 6.47 a copy reaches; 256 requests of one row, 32/4 heads 304 us,
// 6.7 TB/s; one request of 131 thousand keys 90 us, 6.0 TB/s; one token over 700 keys 10.6 us,
// of which 4 go before the first tile has come (launch, lengths, this CTA's share, page ids, the tile).
// With few keys to a unit its start and end are the bound: 2 us a unit of one tile and 4 rows,
// 2.6 of 32, 5.4 of 112 (Q in, the reference, the output), which overlap the other group's.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>

#include <cfloat>

#include "common.cuh"
#include "ptx.cuh"
#include "verify_plan.h"

namespace dspark {
namespace vattn {

using vplan::kTileKeys;

constexpr int kMaxB = 4096;
constexpr int kMaxCtas = 160;                     // grid: one CTA per SM, at most this many
constexpr int kMaxRows = vplan::kMostRows;        // rows of a query tile
constexpr int kThreads = 384;
constexpr int kSoftThreads = 128;               // of each of the two softmax groups
constexpr int kWarpK = 8, kWarpV = 9, kWarpMma = 10, kWarpQ = 11;
constexpr int kQThreads = 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kWaitHintNs = 20000;
constexpr int kLooks = 4096;                      // at two barriers in turn, before a wait for one
constexpr float kRaise = 24.0f;                   // log2 of the weight at which m rises
constexpr float kUnset = -FLT_MAX;                // m of a row that has met no finite score yet
// From this size of m on, half a step of an fp32 score is more than a weight's range.
constexpr float kFar = 0x1p28f;
constexpr int kOnesBytes = 1152;                  // 8 x 2 core matrices of 128 B, one apart
constexpr int kJoinThreads = 256;
constexpr int kJoinAhead = 8;                     // parts whose O a row has in flight

struct Params {
    const uint16_t *q, *k_cache, *v_cache;
    const int32_t *pages, *context, *row_start;
    int B, row_capacity, Hq, Hkv, group, tokens, ps, ps_log2, max_pages, num_pages;
    uint32_t group_inv;                           // r / group = r group_inv >> 16, r < 112
    float scale_log2;                             // scale log2(e)
    uint16_t *out;
    int4 *desc;                                   // [ctas] the unit that starts a join
    float2 *part_ml;                              // [ctas][2][kMaxRows] (m, l)
    float *part_o;                                // [ctas][2][kMaxRows][D]
    unsigned long long timeout_ns;
    int barrier_extra;                            // test hook: arrivals that never come
};

// Workspace: descriptors, then (m, l), then O, two parts a CTA.
struct Layout {
    size_t ml, o, total;
};
__host__ __device__ inline Layout workspace_layout(int D)
{
    Layout w;
    w.ml = (kMaxCtas * sizeof(int4) + 255) / 256 * 256;
    w.o = w.ml + static_cast<size_t>(kMaxCtas) * 2 * kMaxRows * sizeof(float2);
    w.total = w.o + static_cast<size_t>(kMaxCtas) * 2 * kMaxRows * D * sizeof(float);
    return w;
}

// kN: rows of a query tile at most.  Beside 64 rows fit two buffers of Q and of O; beside 112,
// one of each.
template <int D, int kN>
struct Cfg {
    static constexpr int kQBufs = kN == 64 ? 2 : 1;
    static constexpr int kOBufs = kN == 64 ? 2 : 1;
    static constexpr int kPBufs = kN == 64 ? 3 : 2;
    static constexpr int kMBufs = kN == 64 ? 8 : 4;          // references m, by segment
    static constexpr int kTileBytes = kTileKeys * D * 2;
    static constexpr int kHalfBytes = kTileKeys * 128;       // 64 channels of a tile
    static constexpr int kSlots = 2 * (128 / D);             // K tiles, and V tiles, in the ring
    static constexpr int kQBytes = kN * D * 2;
    static constexpr int kPBytes = (kN + 63) / 64 * kTileKeys * 128;
    static constexpr int kRing = 0;
    static constexpr int kRingV = kRing + kSlots * kTileBytes;
    static constexpr int kQ = kRingV + kSlots * kTileBytes;
    static constexpr int kP = kQ + kQBufs * kQBytes;
    static constexpr int kOnes = kP + kPBufs * kPBytes;
    static constexpr int kM = kOnes + kOnesBytes;            // float [kMBufs][kN]
    static constexpr int kRed = kM + kMBufs * kN * 4;             // float [2 groups][4][kN]
    static constexpr int kCtl = kRed + 2 * 4 * kN * 4;
    static constexpr uint32_t kColS = 0, kColO = 2 * kN, kColL = kColO + kOBufs * kN;
    static_assert(kColL + kOBufs * kN <= kTmemCols, "tensor memory");
};

// Barriers of the tiles, four of a kind whatever the ring's depth.  A wait by parity cannot tell a
// phase from the one two back or two ahead, so nobody may wait for a tile's phase while the
// fourth tile before it is still open or once the fourth after it is done.  Who has seen S of
// tile i knows that the values of tile i - 3 have been added, and S and O of tile i + 4 need
// the weights of tile i + 2, of the same softmax group: waits for tiles i - 4 to i are safe.
constexpr uint32_t kTileBars = 4;
__device__ __forceinline__ uint32_t tile_bar(uint32_t bars, uint32_t t)
{
    return bars + 8 * (t % kTileBars);
}
__device__ __forceinline__ uint32_t tile_phase(uint32_t t) { return t / kTileBars & 1u; }

constexpr int kMaxBoxes = kTileKeys / 16;         // pages of a tile at most

struct Ctl {
    // by tile: K copied, V copied, S made (and K's slot free), O added to (and V's slot free)
    unsigned long long k_full[kTileBars], v_full[kTileBars], s_full[kTileBars], o_done[kTileBars];
    unsigned long long p_full[2], m_full[2];
    unsigned long long q_full[2], q_empty[2], o_empty[2], drain;
    struct {
        int b, ctx, rows, start, h, qt, at;       // the CTA's first place
    } first;
    unsigned long long sums[kThreads / 32];
    uint32_t tmem;
    int abort;
    int epoch;                                    // times that a reference m rose
    int odd[8];                                   // a cleared value, by segment as for m
    int far[8];                                   // an m of kFar or more, likewise
    int seg_n[2], seg_tiles[2];                   // the segment of a Q buffer; no tiles: the end
};

template <int D, int kN>
constexpr int smem_bytes()
{
    static_assert(Cfg<D, kN>::kCtl + sizeof(Ctl) <= 227 * 1024, "shared memory of a CTA");
    return Cfg<D, kN>::kCtl + static_cast<int>(sizeof(Ctl));
}

// Rows and context of request b, inside the arrays and the block table.
__device__ __forceinline__ void load_request(const Params &p, int b, int &ctx, int &rows, int &start,
                                             bool &bad)
{
    const int s0 = p.row_start[b], s1 = p.row_start[b + 1], c = p.context[b];
    start = min(max(s0, 0), p.row_capacity);
    rows = min(max(s1, start), p.row_capacity) - start;
    const int room = static_cast<int>(
        min(static_cast<long long>(p.max_pages) * p.ps, static_cast<long long>(INT32_MAX)));
    bad = s0 != start || s1 != start + rows || (rows > 0 && c < 0);
    ctx = max(c, 0);
    if (rows > 0 && (rows > room || ctx > room - rows)) {
        bad = true;
        rows = min(rows, room);
        ctx = room - rows;
    }
}

// A wait that does not succeed at once; a call, to keep the loops that make it short.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, int *abort,
                                       unsigned long long timeout_ns)
{
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (mbar_try_wait_sleep(bar, parity, kWaitHintNs)) return true;
        if (*reinterpret_cast<volatile int *>(abort)) return false;
        if (globaltimer_ns() - t0 > timeout_ns) {
            record_error(DSPARK_TIMEOUT);
            *reinterpret_cast<volatile int *>(abort) = 1;
            return false;
        }
    }
}

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, Ctl &ctl, const Params &p)
{
    return mbar_try_wait(bar, parity) || wait_long(bar, parity, &ctl.abort, p.timeout_ns);
}

// The same for a whole warp, which goes on only if every lane may.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, Ctl &ctl, const Params &p)
{
    return __all_sync(0xFFFFFFFFu, wait(bar, parity, ctl, p));
}

// Bounded wait for this CTA's own copies and MMAs before it ends, whatever the abort flag and
// for a second at least.
__device__ __noinline__ void wait_drain(uint32_t bar, uint32_t parity, const Params &p)
{
    const uint64_t t0 = globaltimer_ns();
    const unsigned long long limit = max(p.timeout_ns, 1000000000ull);
    while (!mbar_try_wait_sleep(bar, parity, kWaitHintNs))
        if (globaltimer_ns() - t0 > limit) {
            record_error(DSPARK_TIMEOUT);
            return;
        }
}

// A CTA's way along its tiles, segment (part of a unit) by segment.  Every role walks it by
// itself, a whole warp at a time: the lanes hold the next 32 requests' lengths.
struct Walk {
    int base, l_ctx, l_rows, l_start;             // request base + lane
    int b, ctx, rows, start;
    int h, qt, kt, kt_end, tiles;                 // segment [kt, kt_end) of the unit's tiles
    int all;                                      // places of the unit
    long long left, unit;                         // places left, and the first of the unit

    __device__ __forceinline__ void load(const Params &p)
    {
        const int r = base + static_cast<int>(threadIdx.x & 31);
        l_ctx = l_rows = l_start = 0;
        bool bad;
        if (r < p.B) load_request(p, r, l_ctx, l_rows, l_start, bad);
    }
    __device__ __forceinline__ void take(int request)
    {
        b = request;
        ctx = __shfl_sync(0xFFFFFFFFu, l_ctx, b - base);
        rows = __shfl_sync(0xFFFFFFFFu, l_rows, b - base);
        start = __shfl_sync(0xFFFFFFFFu, l_start, b - base);
    }
    __device__ __forceinline__ vplan::Request request(const Params &p) const
    {
        return vplan::Request{ctx, rows, p.tokens, p.group};
    }
    // From place `at` of the unit on; false when the CTA's share ends before a key tile starts.
    __device__ __forceinline__ bool segment(const Params &p, int at)
    {
        const vplan::Request r = request(p);
        tiles = r.key_tiles(qt);
        const int per = r.tile_places(qt);
        all = vplan::kUnitPlaces + tiles * per;
        kt = vplan::tile_at(at, per);
        if (all - at <= left) {
            left -= all - at;
            kt_end = tiles;
        } else {
            kt_end = min(vplan::tile_at(at + left, per), tiles);
            left = 0;
        }
        return kt_end > kt;
    }
    __device__ __forceinline__ long long last_place(const Params &p) const
    {
        return unit + vplan::kUnitPlaces + static_cast<long long>(tiles - 1) *
                                               request(p).tile_places(qt);
    }
    // The first segment of the `count` places from `first` on; false when there is none.
    __device__ __forceinline__ bool begin(const Params &p, const Ctl &ctl, long long first,
                                          long long count)
    {
        left = count;
        if (count <= 0) return false;
        b = ctl.first.b, ctx = ctl.first.ctx, rows = ctl.first.rows, start = ctl.first.start;
        h = ctl.first.h, qt = ctl.first.qt;
        base = -1;                                // nothing loaded yet
        unit = first - ctl.first.at;
        return segment(p, ctl.first.at) || next(p);
    }
    __device__ __forceinline__ bool next(const Params &p)
    {
        if (left <= 0) return false;
        unit += all;
        if (++qt == request(p).query_tiles()) {
            qt = 0;
            if (++h == p.Hkv) {
                h = 0;
                if (base < 0) {
                    base = b;
                    load(p);
                }
                unsigned more = __ballot_sync(
                    0xFFFFFFFFu, l_rows > 0 && base + static_cast<int>(threadIdx.x & 31) > b);
                while (!more) {
                    base += 32;
                    if (base >= p.B) return false;
                    load(p);
                    more = __ballot_sync(0xFFFFFFFFu, l_rows > 0);
                }
                take(base + __ffs(more) - 1);
            }
        }
        return segment(p, 0);
    }
    __device__ __forceinline__ int first_token(const Params &p) const { return qt * p.tokens; }
    // rows of the unit (tokens times query heads) and keys that it sees
    __device__ __forceinline__ int unit_rows(const Params &p) const
    {
        return min(rows - qt * p.tokens, p.tokens) * p.group;
    }
    __device__ __forceinline__ int keys(const Params &p) const { return request(p).keys(qt); }
};

// Barrier of a softmax group's 128 threads (named barriers 2 and 3).
__device__ __forceinline__ void group_sync(int group)
{
    asm volatile("bar.sync %0, 128;" ::"r"(2 + group) : "memory");
}

__device__ __forceinline__ bool group_any(int group, bool v)
{
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(static_cast<uint32_t>(v)), "r"(2 + group)
        : "memory");
    return any != 0;
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// t = s scale - m for two rows (fma.rn.f32x2)
__device__ __forceinline__ void scaled2(float &t0, float &t1, uint32_t s0, uint32_t s1, float scale,
                                        float m0, float m1)
{
    asm("{\n\t.reg .b64 rs, rc, rm, rt;\n\t"
        "mov.b64 rs, {%2, %3};\n\t"
        "mov.b64 rc, {%4, %4};\n\t"
        "mov.b64 rm, {%5, %6};\n\t"
        "fma.rn.f32x2 rt, rs, rc, rm;\n\t"
        "mov.b64 {%0, %1}, rt;\n\t}"
        : "=f"(t0), "=f"(t1)
        : "f"(__uint_as_float(s0)), "f"(__uint_as_float(s1)), "f"(scale), "f"(-m0), "f"(-m1));
}

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c,
                                       uint32_t &d)
{
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(addr)
                 : "memory");
}

// Maximum of each of 16 columns over the warp's 32 lanes, halving the columns that a lane
// holds at every exchange: 16 shuffles.  Lane t ends with column t / 2.
__device__ __forceinline__ float column_max(float (&v)[16])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) {
        const int bit = 2 * w;
        const bool up = lane & bit;
#pragma unroll
        for (int k = 0; k < w; ++k) {
            const float keep = up ? v[k + w] : v[k], send = up ? v[k] : v[k + w];
            v[k] = fmaxf(keep, __shfl_xor_sync(0xFFFFFFFFu, send, bit));
        }
    }
    return fmaxf(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 1));
}

// sum += 0 x, of two bf16 each: NaN from a value that is not finite on, else zero
__device__ __forceinline__ void add_zero_times(uint32_t &sum, uint32_t x)
{
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(x), "r"(0u));
}
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w)
{
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
    return w;
}

// The weights of a thread's key against a tile's n rows, from S in tensor memory to P in shared
// memory; returns the largest log2 of one.  Rows below `from` do not see the key.
template <bool kIsFar>
__device__ __forceinline__ float make_weights(uint32_t col, int n, const float *m_row, float sl,
                                              bool masked, int from, uint32_t prow)
{
    const int at = threadIdx.x & 127;
    float top = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < n; c += 16) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(col + c, r);
        float4 m[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) m[q] = *reinterpret_cast<const float4 *>(m_row + c + 4 * q);
        tmem_wait_ld16(r);
        float t[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (!kIsFar) {
                scaled2(t[4 * q], t[4 * q + 1], r[4 * q], r[4 * q + 1], sl, m[q].x, m[q].y);
                scaled2(t[4 * q + 2], t[4 * q + 3], r[4 * q + 2], r[4 * q + 3], sl, m[q].z, m[q].w);
            } else {
                const float f[4] = {m[q].x, m[q].y, m[q].z, m[q].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    t[4 * q + e] =
                        __fsub_rn(__fmul_rn(__uint_as_float(r[4 * q + e]), sl), f[e]);
            }
        }
        if (masked) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (c + j < from) t[j] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < 16; j += 2) top = max3(top, t[j], t[j + 1]);
        uint32_t word[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            word[j] = pack2_bf16(exp2_approx(t[2 * j]), exp2_approx(t[2 * j + 1]));
        const uint32_t to = prow + (c >> 6) * (kTileKeys * 128);
        const int u = (c >> 3) & 7;
        sts128(to + ((u ^ (at & 7)) << 4), word[0], word[1], word[2], word[3]);
        sts128(to + (((u + 1) ^ (at & 7)) << 4), word[4], word[5], word[6], word[7]);
    }
    return top;
}

// The same where an m is kFar or more: a call, to keep the loop that makes it short (the choice
// inside the loop made tiles of 112 rows 4% slower).
__device__ __noinline__ float make_far_weights(uint32_t col, int n, const float *m_row, float sl,
                                               int from, uint32_t prow)
{
    return make_weights<true>(col, n, m_row, sl, true, from, prow);
}

template <int D, int kN>
__global__ void __launch_bounds__(kThreads, 1)
    verify_attention_kernel(const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const Params p)
{
    using C = Cfg<D, kN>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t s0 = smem_u32(smem);
    Ctl &ctl = *reinterpret_cast<Ctl *>(smem + C::kCtl);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    launch_dependents();
    if (s0 % 1024 != 0) {                         // the swizzled tiles need it
        wait_for_prior_kernels();
        if (tid == 0) record_error(DSPARK_BAD_LAUNCH);
        if (tid == 0) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }

    for (int i = tid; i < kOnesBytes / 4; i += kThreads)
        reinterpret_cast<uint32_t *>(smem + C::kOnes)[i] = 0x3F803F80u;
    const uint32_t k_full = smem_u32(ctl.k_full), v_full = smem_u32(ctl.v_full);
    const uint32_t s_full = smem_u32(ctl.s_full), o_done = smem_u32(ctl.o_done);
    const uint32_t p_full = smem_u32(ctl.p_full), m_full = smem_u32(ctl.m_full);
    const uint32_t q_full = smem_u32(ctl.q_full);
    const uint32_t q_empty = smem_u32(ctl.q_empty);
    const uint32_t o_empty = smem_u32(ctl.o_empty), drain = smem_u32(&ctl.drain);
    if (tid >= 32 && tid < 40) ctl.odd[tid - 32] = ctl.far[tid - 32] = 0;
    if (tid == 0) {
        for (uint32_t i = 0; i < kTileBars; ++i) {
            mbar_init(k_full + 8 * i, 1);
            mbar_init(v_full + 8 * i, 1);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(o_done + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(p_full + 8 * i, kSoftThreads + p.barrier_extra);
            mbar_init(m_full + 8 * i, kSoftThreads);
            mbar_init(q_full + 8 * i, kQThreads);
            mbar_init(q_empty + 8 * i, 1);
            mbar_init(o_empty + 8 * i, kSoftThreads);
        }
        mbar_init(drain, 1);
        mbar_fence_init();
        ctl.abort = 0;
        ctl.epoch = 0;
    }
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(&ctl.tmem), kTmemCols);
        tmem_relinquish();
    }
    // what the CTAs need first, into L2 while the kernel before ends: lengths, and page ids (of a
    // table of up to a line a thread)
    {
        const int at = static_cast<int>(blockIdx.x) * kThreads + tid;
        if (at <= (p.B * p.max_pages - 1) / 32) prefetch_l2(p.pages + 32 * at);
        if (at <= (p.B - 1) / 32) {
            prefetch_l2(p.context + 32 * at);
            prefetch_l2(p.row_start + 32 * at);
        }
    }
    wait_for_prior_kernels();

    // ------------------------------------------------ this CTA's share of the tiles
    long long mine = 0;
    const int per = (p.B + kThreads - 1) / kThreads, r0 = tid * per;
    int ctx = 0, rows = 0, start = 0;             // of this thread's last request
    for (int r = r0; r < min(r0 + per, p.B); ++r) {
        bool bad;
        load_request(p, r, ctx, rows, start, bad);
        if (bad && blockIdx.x == 0) record_error(DSPARK_INVALID_TOKEN);
        if (rows > 0) mine += vplan::Request{ctx, rows, p.tokens, p.group}.per_head() * p.Hkv;
    }
    long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += u;
    }
    if (lane == 31) ctl.sums[warp] = sum;
    __syncthreads();
    long long T = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += ctl.sums[w];
        T += ctl.sums[w];
    }
    before += sum - mine;
    const vplan::Split split(T, gridDim.x);
    const int cta = blockIdx.x;
    const long long t0 = cta < split.G ? split.first(cta) : 0;
    const long long t1 = cta < split.G ? split.first(cta + 1) : 0;
    if (t1 > t0 && before <= t0 && t0 < before + mine) {
        // one thread finds the CTA's first place
        long long at = before;
        for (int r = r0;; ++r) {
            if (per > 1) {                        // else it is what this thread holds already
                bool bad;
                load_request(p, r, ctx, rows, start, bad);
                if (rows == 0) continue;
            }
            const vplan::Request q{ctx, rows, p.tokens, p.group};
            const long long n = per > 1 ? q.per_head() * p.Hkv : mine;
            if (t0 < at + n) {
                int h, qt, in_unit;
                place(q, t0 - at, h, qt, in_unit);
                ctl.first.b = r, ctl.first.ctx = ctx, ctl.first.rows = rows;
                ctl.first.start = start, ctl.first.h = h, ctl.first.qt = qt;
                ctl.first.at = in_unit;
                break;
            }
            at += n;
        }
    }
    fence_proxy_async_smem();                     // the ones
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    Walk w = {};
    bool more = w.begin(p, ctl, t0, t1 - t0);

    if (warp == kWarpK || warp == kWarpV) {
        // ---------------------------------------------------- K or V pages into the ring
        const int boxes = kTileKeys >> p.ps_log2;   // pages of a tile
        const bool is_k = warp == kWarpK;
        const void *map = is_k ? &tm_k : &tm_v;
        const uint32_t full = is_k ? k_full : v_full, empty = is_k ? s_full : o_done;
        const uint32_t ring = s0 + (is_k ? C::kRing : C::kRingV);
        uint32_t i = 0;
        bool ok = true;
        // A segment, and page ids 32 at a time, those after them and the next segment's first
        // on their way meanwhile: a table's line comes from HBM, which is most of a tile's time.
        struct Seg {
            int b, h, kt, kt_end, pages;
        };
        auto segment = [&]() {
            return Seg{w.b, w.h, w.kt, w.kt_end, ((w.keys(p) - 1) >> p.ps_log2) + 1};
        };
        auto ids_at = [&](const Seg &s, int at) {
            return at + lane < s.pages
                       ? p.pages[static_cast<size_t>(s.b) * p.max_pages + at + lane]
                       : 0;
        };
        Seg nxt = {};
        int nids = 0;
        if (more) {
            nxt = segment();
            nids = ids_at(nxt, nxt.kt * boxes);
        }
        while (more && ok) {
            const Seg cur = nxt;
            int base = cur.kt * boxes, ids = nids, ids2 = ids_at(cur, base + 32);
            for (int kt = cur.kt; kt < cur.kt_end; ++kt) {
                if (kt * boxes == base + 32) {
                    base += 32;
                    ids = ids2;
                    ids2 = ids_at(cur, base + 32);
                }
                const int n = min(boxes, cur.pages - kt * boxes);   // live pages, the first ones
                int id = __shfl_sync(0xFFFFFFFFu, ids, (kt * boxes - base + lane) & 31);
                if (lane < n && (id < 0 || id >= p.num_pages)) {
                    record_error(DSPARK_INVALID_PAGE);
                    id = 0;
                }
                id = (id * p.Hkv + cur.h) * p.ps;   // the page's first row of the cache
                int row[kMaxBoxes];
#pragma unroll
                for (int j = 0; j < kMaxBoxes; ++j) row[j] = __shfl_sync(0xFFFFFFFFu, id, j);
                const uint32_t slot = i % C::kSlots;
                if (i >= C::kSlots)
                    ok = warp_wait(tile_bar(empty, i - C::kSlots), tile_phase(i - C::kSlots), ctl, p);
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t bar = tile_bar(full, i);
                    uint32_t dst = ring + slot * C::kTileBytes;
                    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(n) * p.ps * D * 2);
#pragma unroll
                    for (int j = 0; j < kMaxBoxes; ++j)
                        if (j < n) {
                            tma_load_2d_plain(dst, map, bar, 0, row[j]);
                            if (D == 128)
                                tma_load_2d_plain(dst + C::kHalfBytes, map, bar, 64, row[j]);
                            dst += p.ps * 128;
                        }
                }
                __syncwarp();
                ++i;
                if (kt == cur.kt) {
                    more = w.next(p);
                    if (more) {
                        nxt = segment();
                        nids = ids_at(nxt, nxt.kt * boxes);
                    }
                }
            }
        }
        // copies land before the CTA ends
        for (uint32_t back = 1; back <= C::kSlots && back <= i; ++back)
            wait_drain(tile_bar(full, i - back), tile_phase(i - back), p);
    } else if (warp == kWarpMma) {
        // ---------------------------------------------------- S^T = K Q^T, O^T += V^T P
        // One thread, from start to end: votes and walks of a whole warp took longer than the
        // MMAs themselves (800 of 1900 cycles a tile with D = 64).
        if (elect_one()) {
            // descriptors: high halves, and low halves of the first buffers
            const uint64_t dk = smem_desc(s0 + C::kRing, 16, 1024, kSwizzle128B);
            const uint64_t dv = smem_desc(s0 + C::kRingV, C::kHalfBytes, 1024, kSwizzle128B);
            const uint64_t dp = smem_desc(s0 + C::kP, kTileKeys * 128, 1024, kSwizzle128B);
            const uint64_t d1 = smem_desc(s0 + C::kOnes, 128, 128, kSwizzleNone);
            const uint32_t k_hi = dk >> 32, v_hi = dv >> 32, p_hi = dp >> 32, ones_hi = d1 >> 32;
            const uint32_t k_lo = dk, v_lo = dv, p_lo = dp, ones_lo = d1;
            const uint32_t q_lo = k_lo + ((C::kQ - C::kRing) >> 4);
            // S runs two tiles ahead of O: once the weights of tile i are there, S of tile i + 2
            // goes first, since its softmax waits for it, and the values of tile i after it; or
            // the other way round while keys or queries are still on their way.
            struct Tile {
                uint32_t id_o, id_l, seg;
                bool first;                       // of its segment
            } t0 = {}, t1 = {};
            uint32_t ahead = 0;                   // tiles in t0, t1
            // tile, ring slot and P buffer: of the next S, and of the next values
            uint32_t i = 0, slot = 0, j = 0, jslot = 0, jbuf = 0;
            bool ok = true;
            auto weights_there = [&]() { return wait(p_full + 8 * (j & 1), (j >> 1) & 1u, ctl, p); };
            auto values_ready = [&]() {
                return mbar_test_wait(p_full + 8 * (j & 1), (j >> 1) & 1u) &&
                       mbar_test_wait(tile_bar(v_full, j), tile_phase(j)) &&
                       (!t0.first || mbar_test_wait(o_empty + 8 * (t0.seg % C::kOBufs),
                                                    ((t0.seg / C::kOBufs) & 1u) ^ 1u));
            };
            auto values = [&]() {
                const uint32_t ob = t0.seg % C::kOBufs;
                ok = wait(tile_bar(v_full, j), tile_phase(j), ctl, p) &&
                     (!t0.first ||
                      wait(o_empty + 8 * ob, ((t0.seg / C::kOBufs) & 1u) ^ 1u, ctl, p));
                if (!ok) return;
                tc_fence_after();
                const uint32_t a = v_lo + jslot * (C::kTileBytes >> 4);
                const uint32_t b = p_lo + jbuf * (C::kPBytes >> 4);
                const uint32_t to = tmem + C::kColO + ob * kN, tl = tmem + C::kColL + ob * kN;
#pragma unroll
                for (int k = 0; k < kTileKeys / 16; ++k) {
                    const bool acc = k > 0 || !t0.first;
                    umma_bf16(to, a + k * 128, v_hi, b + k * 128, p_hi, t0.id_o, acc);
                    umma_bf16(tl, ones_lo, ones_hi, b + k * 128, p_hi, t0.id_l, acc);
                }
                umma_commit(tile_bar(o_done, j));
                ++j;
                if (++jslot == C::kSlots) jslot = 0;
                if (++jbuf == C::kPBufs) jbuf = 0;
                t0 = t1;
                --ahead;
            };
            for (uint32_t seg = 0; ok; ++seg) {
                const uint32_t qb = seg % C::kQBufs;
                const uint32_t turn = (seg / C::kQBufs) & 1u;
                // values or queries, whichever are there first (a bounded wait after so many looks)
                for (int looks = 0; ok && ahead > 0 && !mbar_test_wait(q_full + 8 * qb, turn);) {
                    if (++looks < kLooks && !values_ready()) continue;
                    looks = 0;
                    ok = weights_there();
                    if (ok) values();
                }
                ok = ok && wait(q_full + 8 * qb, turn, ctl, p);
                if (!ok) break;
                const uint32_t n = ctl.seg_n[qb];
                const int tiles = ctl.seg_tiles[qb];
                if (tiles == 0) break;
                const uint32_t id = idesc_bf16_f32(kTileKeys, n, 0, 0);
                const uint32_t q = q_lo + qb * (C::kQBytes >> 4);
                for (int t = 0; t < tiles; ++t) {
                    if (ahead == 2) {             // S's buffer is free once they are
                        ok = weights_there();
                        if (ok && !mbar_test_wait(tile_bar(k_full, i), tile_phase(i))) values();
                    }
                    ok = ok && wait(tile_bar(k_full, i), tile_phase(i), ctl, p);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a = k_lo + slot * (C::kTileBytes >> 4);
                    const uint32_t to = tmem + C::kColS + (i & 1) * kN;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        umma_bf16(to, a + (k >> 2) * (C::kHalfBytes >> 4) + (k & 3) * 2, k_hi,
                                  q + (k >> 2) * (kN * 128 >> 4) + (k & 3) * 2, k_hi, id, k > 0);
                    umma_commit(tile_bar(s_full, i));
                    if (t + 1 == tiles) umma_commit(q_empty + 8 * qb);
                    ++i;
                    if (++slot == C::kSlots) slot = 0;
                    if (ahead == 2) values();
                    if (!ok) break;
                    const Tile cur = {idesc_bf16_f32(D, n, 1, 1), idesc_bf16_f32(64, n, 0, 1), seg,
                                      t == 0};
                    if (ahead == 0) t0 = cur;
                    else t1 = cur;
                    ++ahead;
                }
            }
            while (ok && ahead > 0) {
                ok = weights_there();
                if (ok) values();
            }
            umma_commit(drain);                   // MMAs finish before the CTA ends
            wait_drain(drain, 0, p);
        }
        __syncwarp();
    } else if (warp >= kWarpQ) {
        // ---------------------------------------------------- Q rows of each segment
        const int t = tid - kWarpQ * 32;
        uint32_t seg = 0;
        for (;;) {
            const uint32_t qb = seg % C::kQBufs;
            const int rows = more ? w.unit_rows(p) : 0, n = (rows + 15) & ~15;
            if (!warp_wait(q_empty + 8 * qb, ((seg / C::kQBufs) & 1u) ^ 1u, ctl, p))
                break;
            const uint32_t dst = s0 + C::kQ + qb * C::kQBytes;
            const size_t row0 = static_cast<size_t>(w.start + w.first_token(p)) * p.Hq +
                                static_cast<size_t>(w.h) * p.group;
            constexpr int kStep = kQThreads / (D / 8);   // rows between a thread's
            const int u = t % (D / 8);
            const uint16_t *from = p.q + row0 * D + u * 8;
            const long long token = static_cast<long long>(p.Hq - p.group) * D;   // past a token's rows
#pragma unroll 4
            for (int r = t / (D / 8); r < n; r += kStep) {
                const uint32_t to = dst + (u >> 3) * (kN * 128) + r * 128 +
                                    (((u & 7) ^ (r & 7)) << 4);
                if (r < rows)
                    cp_async_16(to, from + r * D + (r * p.group_inv >> 16) * token);
                else
                    sts128(to, 0, 0, 0, 0);
            }
            cp_async_wait_all();
            fence_proxy_async_smem();
            if (lane == 0) {
                ctl.seg_n[qb] = n;
                ctl.seg_tiles[qb] = more ? w.kt_end - w.kt : 0;
            }
            mbar_arrive(q_full + 8 * qb);
            if (!more) break;
            ++seg;
            more = w.next(p);
        }
    } else {
        // ---------------------------------------------------- softmax and output
        // Group 0 takes the CTA's even tiles, group 1 the odd ones, so that one's exponentials
        // run beside the other's waits and barriers (both on one tile, half of the rows each,
        // took as long as one alone).  They share m and O, so tiles are handed to the MMA in
        // their order: a group waits for the one before its own, and makes its weights anew
        // if m rose meanwhile.
        const int wg = warp >> 2, quad = warp & 3, at = tid & 127;
        float *m_s = reinterpret_cast<float *>(smem + C::kM);
        float *red = reinterpret_cast<float *>(smem + C::kRed) + wg * 4 * kN;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        // the output's channel of this thread (M = 64 puts 16 rows in each warp's lanes)
        const int d = D == 128 ? at : quad * 16 + (lane & 15);
        const bool has_d = D == 128 || lane < 16;
        const float sl = p.scale_log2;
        struct Seg {
            int row0, rows, h, kt, kt_end, keys, hidden, b;   // hidden: keys that row 0 sees
            bool starts, ends;
        } cur = {}, late = {};
        bool owed = false;                        // the output of `late` is still to be written
        uint32_t late_seg = 0, late_tile = 0;
        int4 desc = make_int4(0, 0, 0, 0);

        // after a wait that ran out the warps go on without waiting, so that they meet at the
        // same barriers until the end (the results are unspecified then)
        bool dead = false;
        auto await = [&](uint32_t bar, uint32_t parity) {
            if (!dead && !wait(bar, parity, ctl, p)) dead = true;
        };
        // l, O -> out, or to the workspace when the unit has other parts
        auto output = [&](const Seg &s, uint32_t seg, uint32_t last_tile) {
            const uint32_t ob = seg % C::kOBufs;
            await(tile_bar(o_done, last_tile), tile_phase(last_tile));
            __syncwarp();
            tc_fence_after();
            const bool direct = s.starts && s.ends;
            const int part = 2 * blockIdx.x + (s.starts ? 1 : 0);
            const bool odd = *reinterpret_cast<volatile int *>(&ctl.odd[seg % C::kMBufs]);
            // a thread per row: 1 / l and the row's place in the output, or (m, l)
            for (int c0 = 16 * quad; c0 < s.rows; c0 += 64) {
                uint32_t l[16];
                tmem_ld_32x32b_x16(lane_base + C::kColL + ob * kN + c0, l);
                tmem_wait_ld16(l);
                if (lane == 0)
#pragma unroll
                    for (int j = 0; j < 16; ++j) red[c0 + j] = __uint_as_float(l[j]);
            }
            group_sync(wg);
            if (at < s.rows) {
                const float l = red[at];
                if (direct) {
                    const int i = at * p.group_inv >> 16;
                    red[kN + at] = __int_as_float(i * p.Hq + at - i * p.group);
                    red[at] = 1.0f / l;
                } else {
                    p.part_ml[static_cast<size_t>(part) * kMaxRows + at] =
                        make_float2(m_s[seg % C::kMBufs * kN + at], l);
                }
            }
            group_sync(wg);
            const size_t row0 = static_cast<size_t>(s.row0) * p.Hq + static_cast<size_t>(s.h) * p.group;
            uint32_t o[16];
            tmem_ld_32x32b_x16(lane_base + C::kColO + ob * kN, o);
            for (int c0 = 0; c0 < s.rows; c0 += 16) {
                float v[16];
                tmem_wait_ld16(o);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float4 f = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                    if (direct) f = *reinterpret_cast<const float4 *>(red + c0 + 4 * q);
                    v[4 * q] = __uint_as_float(o[4 * q]) * f.x;
                    v[4 * q + 1] = __uint_as_float(o[4 * q + 1]) * f.y;
                    v[4 * q + 2] = __uint_as_float(o[4 * q + 2]) * f.z;
                    v[4 * q + 3] = __uint_as_float(o[4 * q + 3]) * f.w;
                }
                if (c0 + 16 < s.rows) tmem_ld_32x32b_x16(lane_base + C::kColO + ob * kN + c0 + 16, o);
                if (odd && has_d) {               // values that are not finite, to who sees them
                    const int end = s.ends ? s.keys : s.kt_end * kTileKeys;
                    for (int j = max(s.kt * kTileKeys, s.hidden); j < end; ++j) {
                        int page = p.pages[static_cast<size_t>(s.b) * p.max_pages + j / p.ps];
                        if (page < 0 || page >= p.num_pages) page = 0;
                        const uint32_t x =
                            p.v_cache[((static_cast<size_t>(page) * p.Hkv + s.h) * p.ps +
                                       j % p.ps) * D + d];
                        if ((x & 0x7F80u) == 0x7F80u) {
                            const int from = (j - s.hidden + 1) * p.group;
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (c0 + e >= from) v[e] += __uint_as_float(x << 16);
                        }
                    }
                }
                if (direct) {
                    // neighbouring lanes hold neighbouring channels: the even lane stores row
                    // j's pair, the odd lane row j + 1's
                    const bool up = lane & 1;
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float got = __shfl_xor_sync(0xFFFFFFFFu, up ? v[j] : v[j + 1], 1);
                        const uint32_t word =
                            up ? pack2_bf16(got, v[j + 1]) : pack2_bf16(v[j], got);
                        const int r = c0 + j + (up ? 1 : 0);
                        if (r < s.rows && has_d)
                            *reinterpret_cast<uint32_t *>(
                                p.out + (row0 + __float_as_int(red[kN + r])) * D + (d & ~1)) = word;
                    }
                } else if (has_d) {
                    float *to = p.part_o + (static_cast<size_t>(part) * kMaxRows + c0) * D + d;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c0 + j < s.rows) to[j * D] = v[j];
                }
            }
            group_sync(wg);                       // red is free again
            if (at == 0) ctl.odd[seg % C::kMBufs] = ctl.far[seg % C::kMBufs] = 0;
            tc_fence_before();
            mbar_arrive(o_empty + 8 * ob);
        };

        // the tile's scores times scale log2(e), hidden ones -inf
        auto scores = [&](uint32_t (&r)[16], float (&t)[16], int c0, int from) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                t[j] = __uint_as_float(r[j]) * sl;
                if (c0 + j < from) t[j] = -INFINITY;
            }
        };
        // red[q][row] = the tile's maximum in the keys of warp q; `share`: in that of one warp
        auto reduce = [&](uint32_t col, int n, int from, bool share) {
            for (int c0 = share ? 16 * quad : 0; c0 < n; c0 += share ? 64 : 16) {
                uint32_t r[16];
                float t[16];
                tmem_ld_32x32b_x16(col + c0, r);
                tmem_wait_ld16(r);
                scores(r, t, c0, from);
                const float m = column_max(t);
                if ((lane & 1) == 0) red[quad * kN + c0 + (lane >> 1)] = m;
            }
        };
        auto max_of = [&](int r) {
            return fmaxf(fmaxf(red[r], red[kN + r]), fmaxf(red[2 * kN + r], red[3 * kN + r]));
        };

        uint32_t i = 0, seg = 0;
        while (more) {
            const int tok0 = w.first_token(p);
            cur.row0 = w.start + tok0;
            cur.rows = w.unit_rows(p);
            cur.h = w.h;
            cur.b = w.b;
            cur.kt = w.kt;
            cur.kt_end = w.kt_end;
            cur.keys = w.keys(p);
            cur.hidden = w.ctx + tok0 + 1;
            cur.starts = w.kt == 0;
            cur.ends = w.kt_end == w.tiles;
            if (cur.starts && !cur.ends)
                desc = make_int4(cur.row0, cur.h, cur.rows,
                                 split.cta_of(w.last_place(p)) - cta + 1);
            const int n = (cur.rows + 15) & ~15;
            float *m_row = m_s + seg % C::kMBufs * kN;
            int kt = cur.kt + ((i & 1) == static_cast<uint32_t>(wg) ? 0 : 1);
            i += kt - cur.kt;
            for (; kt < cur.kt_end; kt += 2, i += 2) {
                const uint32_t col = lane_base + C::kColS + wg * kN;
                const int key = kt * kTileKeys + at;
                // rows from `from` on see this thread's key
                int from = 0;
                if (key >= cur.keys) from = kMaxRows;
                else if (key >= cur.hidden) from = (key - cur.hidden + 1) * p.group;
                // (a tile's end may be past 32 bits)
                const bool masked = kt * kTileKeys > cur.hidden - kTileKeys;
                const bool first = kt == cur.kt;
                const uint32_t before = p_full + 8 * (wg ^ 1), before_phase = ((i - 1) >> 1) & 1u;
                await(tile_bar(s_full, i), tile_phase(i));
                // m of this segment: to be set here, or set by the other group.  S of this tile
                // came after the other had handed over tile i - 2 at least, so what it may still
                // read belongs to one of the last kMBufs - 1 segments.
                if (!first) await(m_full + 8 * (seg & 1), (seg >> 1) & 1u);
                __syncwarp();
                tc_fence_after();
                // With three P buffers this one is free: its last product, three tiles ago, came
                // before this S in the tensor core's order.  With two it is waited for.
                const uint32_t prow = s0 + C::kP + i % C::kPBufs * C::kPBytes + at * 128;
                if (C::kPBufs == 2 && i >= 2) await(tile_bar(o_done, i - 2), tile_phase(i - 2));
                __syncwarp();
                // 1: m has to be set, 2: to be raised.  m is the maximum over the first tile, or,
                // where every row sees all of it, over one warp's 32 keys, which does as well and
                // is one exchange for a warp.
                int task = first ? 1 : 0;
                for (int tries = 0; tries < 8; ++tries) {
                    if (task) {
                        const bool share = task == 1 && !masked;
                        reduce(col, n, from, share);
                        group_sync(wg);
                        if (at < n) {
                            const float m = share ? red[((at >> 4) & 3) * kN + at] : max_of(at);
                            if (fabsf(m) >= kFar && m != -INFINITY)
                                *reinterpret_cast<volatile int *>(&ctl.far[seg % C::kMBufs]) = 1;
                            if (task == 1) {
                                m_row[at] = m == -INFINITY ? kUnset : m;
                            } else {
                                const float old = m_row[at], now = fmaxf(old, m);
                                m_row[at] = now;
                                red[at] = exp2_approx(old - now);
                            }
                        }
                        group_sync(wg);
                        if (task == 1) {
                            mbar_arrive(m_full + 8 * (seg & 1));
                        } else {                  // the new m first, then word of it
                            if (at == 0)
                                *reinterpret_cast<volatile int *>(&ctl.epoch) = ctl.epoch + 1;
                            group_sync(wg);
                        }
                    }
                    if (task == 2 && !first) {
                        // O and l of the tiles before are scaled
                        const uint32_t ob = seg % C::kOBufs;
                        await(tile_bar(o_done, i - 1), tile_phase(i - 1));
                        __syncwarp();
                        tc_fence_after();
                        for (int c0 = 0; c0 < n; c0 += 16) {
                            for (uint32_t base : {C::kColO, C::kColL}) {
                                uint32_t r[16];
                                tmem_ld_32x32b_x16(lane_base + base + ob * kN + c0, r);
                                tmem_wait_ld16(r);
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    r[j] = __float_as_uint(__uint_as_float(r[j]) * red[c0 + j]);
                                tmem_st_32x32b_x16(lane_base + base + ob * kN + c0, r);
                            }
                        }
                        tmem_wait_st();
                    }
                    // weights to shared memory; the largest log2 of one
                    const int epoch = *reinterpret_cast<volatile int *>(&ctl.epoch);
                    // (the whole warp takes the same way; the other group may be raising m meanwhile,
                    // and then these weights are stale)
                    const bool far = __any_sync(
                        0xFFFFFFFFu, *reinterpret_cast<volatile int *>(&ctl.far[seg % C::kMBufs]));
                    const float top =
                        far ? make_far_weights(col, n, m_row, sl, from, prow)
                            : make_weights<false>(col, n, m_row, sl, masked, from, prow);
                    if (masked && tries == 0) {
                        // values behind the last key, and those that are not finite: the last
                        // thing, since the values come after the keys
                        const uint32_t slot = i % C::kSlots;
                        await(tile_bar(v_full, i), tile_phase(i));
                        // 16-byte chunks in an order of the lane's own, so that neighbouring rows,
                        // 128 bytes apart, meet different banks
                        const uint32_t v = s0 + C::kRingV + slot * C::kTileBytes + at * 128;
                        auto chunk = [&](int u) {
                            return v + (u >> 3) * C::kHalfBytes + (((u ^ at) & 7) << 4);
                        };
                        if (key >= cur.keys) {
#pragma unroll
                            for (int u = 0; u < D / 8; ++u) sts128(chunk(u), 0, 0, 0, 0);
                        } else if (from > 0) {
                            uint32_t sum[4] = {};          // of zero times each value
#pragma unroll
                            for (int u = 0; u < D / 8; ++u) {
                                uint32_t x[4];
                                lds128(chunk(u), x[0], x[1], x[2], x[3]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) add_zero_times(sum[e], x[e]);
                            }
                            if (((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7FFF7FFFu) != 0) {
#pragma unroll 1
                                for (int u = 0; u < D / 8; ++u) {
                                    uint32_t x0, x1, x2, x3;
                                    lds128(chunk(u), x0, x1, x2, x3);
                                    sts128(chunk(u), finite_or_zero(x0), finite_or_zero(x1),
                                           finite_or_zero(x2), finite_or_zero(x3));
                                }
                                *reinterpret_cast<volatile int *>(&ctl.odd[seg % C::kMBufs]) = 1;
                            }
                        }
                    }
                    // this tile's turn, and what has become of m
                    if (i > 0) await(before, before_phase);
                    __syncwarp();
                    const bool stale = *reinterpret_cast<volatile int *>(&ctl.epoch) != epoch;
                    if (!group_any(wg, stale || top > kRaise)) break;
                    task = group_any(wg, stale) ? 0 : 2;
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(p_full + 8 * wg);
                // a unit's output: at once, since the next unit's O waits for it, or, with a
                // second O buffer, after the group's next tile, when the last product is done
                if (owed) {
                    output(late, late_seg, late_tile);
                    owed = false;
                }
                if (kt + 1 == cur.kt_end) {
                    late = cur;
                    late_seg = seg;
                    late_tile = i;
                    if (C::kOBufs == 1) output(late, late_seg, late_tile);
                    else owed = true;
                }
            }
            i -= kt - cur.kt_end;                 // the next segment's first tile
            ++seg;
            more = w.next(p);
        }
        if (owed) output(late, late_seg, late_tile);
        if (tid == 0) p.desc[blockIdx.x] = desc;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) tmem_dealloc(tmem, kTmemCols);
}

// Adds up the parts of the unit that starts in CTA blockIdx.x and ends in a later one: with
// M = max m over the parts,  out = sum 2^(m - M) O / sum 2^(m - M) l.  What bounds it: latency, of
// three loads that need one another if nothing is done about it.  So two rows at most have a warp
// of their own (gridDim.y CTAs to a unit; 17 tokens of 4 heads over 131 thousand keys: 96.6 us a
// call with one, 93.1 with two, 91.8 with four, 89.9 with six or more), lane i holds part i's
// (m, l), and O is fetched beside them.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) verify_join_kernel(const Params p)
{
    constexpr int kPer = D / 32;
    launch_dependents();
    wait_for_prior_kernels();
    const int4 unit = p.desc[blockIdx.x];
    const int row0 = unit.x, h = unit.y, rows = unit.z, parts = unit.w;
    if (parts < 2) return;
    const int lane = threadIdx.x & 31;
    for (int r = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5); r < rows;
         r += gridDim.y * (kJoinThreads / 32)) {
        // part 0 is its CTA's last, the others their CTAs' first
        auto part = [&](int i) {
            return static_cast<size_t>(2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * kMaxRows + r;
        };
        auto fetch = [&](int i, float (&v)[kPer]) {
            const float *o = p.part_o + part(i) * D + lane * kPer;
            if constexpr (kPer == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(o);
                v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2 *>(o);
                v[0] = x.x, v[1] = x.y;
            }
        };
        float v[kJoinAhead][kPer];
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i)
            if (i < parts) fetch(i, v[i]);
        // M over all parts; a part without l saw no key, or none of a finite score
        float2 ml = make_float2(0.0f, 0.0f);
        if (lane < parts) ml = p.part_ml[part(lane)];
        float m = ml.y != 0.0f ? ml.x : -INFINITY;
        for (int i = 32 + lane; i < parts; i += 32) {
            const float2 x = p.part_ml[part(i)];
            if (x.y != 0.0f) m = fmaxf(m, x.x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        float l = 0.0f, acc[kPer] = {};
        for (int i0 = 0; i0 < parts; i0 += 32) {
            if (i0 > 0) {
                ml = make_float2(0.0f, 0.0f);
                if (i0 + lane < parts) ml = p.part_ml[part(i0 + lane)];
            }
            // a weight of nothing still multiplies: zero times a value that is not finite is NaN,
            // as it is within a part (a row that saw no key of a part left zeros there)
            const float f = ml.y != 0.0f ? exp2_approx(ml.x - m) : 0.0f;
            l += ml.y * f;
            for (int g = i0; g < min(i0 + 32, parts); g += kJoinAhead) {
#pragma unroll
                for (int e = 0; e < kJoinAhead; ++e) {
                    const float w = __shfl_sync(0xFFFFFFFFu, f, g + e - i0);
                    if (g + e < parts)
#pragma unroll
                        for (int j = 0; j < kPer; ++j) acc[j] = fmaf(v[e][j], w, acc[j]);
                    if (g + e + kJoinAhead < parts) fetch(g + e + kJoinAhead, v[e]);
                }
            }
        }
        l = warp_sum(l);
        const float inv = 1.0f / l;
        uint32_t *to = reinterpret_cast<uint32_t *>(
            p.out + (static_cast<size_t>(row0 + r / p.group) * p.Hq +
                     static_cast<size_t>(h) * p.group + r % p.group) * D + lane * kPer);
#pragma unroll
        for (int j = 0; j < kPer; j += 2) to[j / 2] = pack2_bf16(acc[j] * inv, acc[j + 1] * inv);
    }
}

}  // namespace vattn
}  // namespace dspark
