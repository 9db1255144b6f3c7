// verify_layout.cuh -- the ragged batch of one verification step over a paged cache.
//
// Request b has context[b] tokens in the cache (-1: idle slot) and sends L[b] + 1 more
// (its anchor and L[b] drafts).  With ps tokens to a page,
//     want = L + 1 (0 when idle),  need = ceil((context + want) / ps),
// pages held beyond `need` go back on the free stack, in request order, then the pages that
// requests miss are popped from its top, in request order; rows = what the pages held
// hold of `want`, and row_start is the running sum of rows.
//
// Everything follows from two running sums over the requests (pages returned and asked
// for, in one 64-bit word; then rows), so no request waits for another: with F pages on
// the stack, R returned in all and A_b asked for before request b, its share is
// clamp(F + R - A_b, 0, asked), and its j-th page stands at F + R - 1 - A_b - j.
//
// What bounds it: latency.  One cluster of up to 8 CTAs runs it in one launch; every CTA
// forms the sums for all requests (they are a few KB) instead of exchanging them, and the
// rows are spread over all threads of the cluster by a binary search in the sums, since a
// request's rows number from none to a whole prompt.  The state is updated in place, so a
// cluster barrier stands between the last read of the old state and the first write.
// Measured (B200, device time): 64 requests with up to 17 rows 3.8 us where no page moves, 5.4
// where a third of them return or take one; 1024 with up to 25 rows 7.8, and 9.8 with pages
// moved by a quarter.  A page that moves costs a second cluster barrier and the loads after it.
// Where every 32nd request ends or starts with all its pages as well: 8.9 and 15.9.
#pragma once
#include "common.cuh"
#include "ptx.cuh"

namespace dspark {
namespace layout {

constexpr int kThreadsFew = 128, kThreadsMany = 1024;   // to a CTA, for up to 128 requests or more
constexpr int kMaxB = 4096;
constexpr int kWordsPerRequest = 6;

struct Params {
    int32_t *L;                   // [B] in; cut where the pages ran out
    const int32_t *anchor, *x;    // [B], [B][gamma]; null without tokens
    const int32_t *accepted;      // [B], or null
    int32_t *context;             // [B] in; grown by `accepted`
    int32_t *rows;                // [B] in (with accepted), out
    int32_t *pages;               // [B][max_pages]
    int32_t *held;                // [B]
    int32_t *free_pages;          // [num_pages], free_count of them in use
    int32_t *free_count;          // [1]
    int B, gamma, ps, max_pages, num_pages;
    int32_t *row_start, *position, *slot, *token;
};

// Exclusive running sum of one 64-bit value per thread; `total` is the sum of all.
template <int kThreads>
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v,
                                                         unsigned long long *warp_sums,
                                                         unsigned long long &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += u;
    }
    __syncthreads();                              // the last round's sums have been read
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    // the warps' sums: read by every thread where they are few, else summed as the threads' were
    // (of 32, one by one: 9.6 us a call for 1024 requests instead of 7.9)
    unsigned long long before = 0;
    total = 0;
    if (kThreads <= 128) {
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const unsigned long long t = warp_sums[w];
            if (w < warp) before += t;
            total += t;
        }
    } else {
        unsigned long long t = lane < kThreads / 32 ? warp_sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < kThreads / 32; o <<= 1) {
            const unsigned long long u = __shfl_up_sync(0xFFFFFFFFu, t, o);
            if (lane >= o) t += u;
        }
        total = __shfl_sync(0xFFFFFFFFu, t, kThreads / 32 - 1);
        before = __shfl_sync(0xFFFFFFFFu, t, max(warp - 1, 0));
        if (warp == 0) before = 0;
    }
    return before + s - v;
}

// Value in [lo, hi], recording one that lies outside.
__device__ __forceinline__ int checked_length(int v, int lo, int hi)
{
    if (v < lo || v > hi) {
        record_error(DSPARK_INVALID_TOKEN);
        return min(max(v, lo), hi);
    }
    return v;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) verify_layout_kernel(const Params p)
{
    constexpr int kWarps = kThreads / 32;
    extern __shared__ int32_t words[];
    __shared__ unsigned long long warp_sums[kWarps];
    int32_t *s_ctx = words, *s_want = words + p.B, *s_held = words + 2 * p.B;
    int32_t *s_back = words + 3 * p.B, *s_ask = words + 4 * p.B, *s_row = words + 5 * p.B;
    const int tid = threadIdx.x;
    const int cta = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(cluster_nctarank());
    launch_dependents();
    wait_for_prior_kernels();
    // the state is updated in place, and the cluster barriers are all that keeps one CTA's update
    // from another's reads: a grid that is not one cluster (a tool re-issuing the launch without
    // it, say) stops here, before it touches memory
    if (cluster_nctarank() != gridDim.x || blockDim.x != kThreads) {
        if (tid == 0) record_error(DSPARK_BAD_LAUNCH);
        return;
    }
    const int room = static_cast<int>(
        min(static_cast<long long>(p.max_pages) * p.ps, static_cast<long long>(INT32_MAX)));

    const int free_count = *p.free_count;         // used after the first sums
    unsigned long long carry = 0;                 // pages returned << 32 | pages asked for
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + tid;
        int back = 0, ask = 0, ctx = -1, want = 0, held = 0;
        if (b < p.B) {
            // all loads first: none waits for another's value
            ctx = p.context[b];
            const int len = p.L[b], had = p.held[b];
            const int accepted = p.accepted ? p.accepted[b] : -1;
            const int sent_before = p.accepted ? p.rows[b] : 0;
            if (ctx >= 0) {
                const int grown = min(checked_length(accepted, -1, INT32_MAX - 1) + 1,
                                      max(sent_before, 0));
                ctx = static_cast<int>(min(static_cast<long long>(ctx) + grown,
                                           static_cast<long long>(INT32_MAX)));
            }
            ctx = checked_length(ctx, -1, room);
            if (ctx >= 0) want = checked_length(len, 0, p.gamma) + 1;
            held = checked_length(had, 0, p.max_pages);
            const int sent = min(want, room - max(ctx, 0));   // what the block table has room for
            const int need = ctx < 0 ? 0 : static_cast<int>((static_cast<long long>(ctx) + sent +
                                                             p.ps - 1) / p.ps);
            back = max(held - need, 0);
            ask = max(need - held, 0);
            held = min(held, need);
        }
        unsigned long long total;
        const unsigned long long at =
            carry + block_scan<kThreads>(static_cast<unsigned long long>(back) << 32 |
                                   static_cast<unsigned>(ask), warp_sums, total);
        carry += total;
        if (b < p.B) {
            s_ctx[b] = ctx;
            s_want[b] = want;
            s_held[b] = held;
            s_back[b] = static_cast<int>(at >> 32);
            s_ask[b] = static_cast<int>(at);
        }
    }
    const int F = checked_length(free_count, 0, p.num_pages);
    const int returned = static_cast<int>(carry >> 32);
    const unsigned asked = static_cast<unsigned>(carry);
    // the stack after the returns; pages past the array's end (a caller's page that stands
    // in two tables) are lost rather than written out of bounds
    const int top = static_cast<int>(min(static_cast<long long>(F) + returned,
                                         static_cast<long long>(p.num_pages)));
    if (static_cast<long long>(F) + returned > p.num_pages) record_error(DSPARK_INVALID_PAGE);

    // a request's pages asked for and returned are differences of the running sums
    auto ask_of = [&](int b) {
        return static_cast<int>((b + 1 < p.B ? static_cast<unsigned>(s_ask[b + 1]) : asked) -
                                static_cast<unsigned>(s_ask[b]));
    };
    auto back_of = [&](int b) { return (b + 1 < p.B ? s_back[b + 1] : returned) - s_back[b]; };
    auto grant_of = [&](int b) { return min(ask_of(b), max(top - s_ask[b], 0)); };
    __syncthreads();

    unsigned long long rows_before = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + tid;
        int n = 0;
        if (b < p.B && s_ctx[b] >= 0) {
            const long long have = static_cast<long long>(s_held[b] + grant_of(b)) * p.ps;
            n = static_cast<int>(
                min(static_cast<long long>(s_want[b]), max(have - s_ctx[b], 0ll)));
        }
        unsigned long long total;
        const unsigned long long at =
            rows_before + block_scan<kThreads>(static_cast<unsigned>(n), warp_sums, total);
        rows_before += total;
        if (b < p.B) s_row[b] = static_cast<int>(at);
    }
    const int total_rows = static_cast<int>(rows_before);

    cluster_sync();                               // the old state has been read everywhere

    // returned pages go on the stack
    const int warp = cta * kWarps + (tid >> 5), warps = ctas * kWarps, lane = tid & 31;
    if (returned) {
        for (int b = warp; b < p.B; b += warps) {
            const int n = back_of(b);
            const int32_t *from = p.pages + static_cast<size_t>(b) * p.max_pages + s_held[b];
            for (int i = lane; i < n; i += 32)
                if (F + s_back[b] + i < p.num_pages) p.free_pages[F + s_back[b] + i] = from[i];
        }
        if (asked) cluster_sync();                // and are on it before any is popped
    }

    // popped pages go into the tables, and the requests' state is written
    for (int b = warp; b < p.B; b += warps) {
        const int n = grant_of(b);
        int32_t *to = p.pages + static_cast<size_t>(b) * p.max_pages + s_held[b];
        for (int i = lane; i < n; i += 32) to[i] = __ldcg(p.free_pages + top - 1 - s_ask[b] - i);
        if (lane == 0) {
            const int rows = (b + 1 < p.B ? s_row[b + 1] : total_rows) - s_row[b];
            p.row_start[b] = s_row[b];
            p.rows[b] = rows;
            p.held[b] = s_held[b] + n;
            if (p.accepted) p.context[b] = s_ctx[b];
            if (rows < s_want[b]) {
                p.L[b] = max(rows - 1, 0);
                record_error(DSPARK_OUT_OF_PAGES);
            }
        }
    }
    if (cta == 0 && tid == 0) {
        p.row_start[p.B] = total_rows;
        *p.free_count = top - static_cast<int>(min(asked, static_cast<unsigned>(top)));
    }

    // the rows, in order, over all threads of the cluster
    for (int r = cta * kThreads + tid; r < total_rows; r += ctas * kThreads) {
        int lo = 0, hi = p.B - 1;                 // the last request that starts at or before r
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_row[mid] <= r) lo = mid;
            else hi = mid - 1;
        }
        const int b = lo, i = r - s_row[b];
        const int pos = s_ctx[b] + i, at = pos / p.ps;
        const int page = at < s_held[b]
                             ? p.pages[static_cast<size_t>(b) * p.max_pages + at]
                             : __ldcg(p.free_pages + top - 1 - s_ask[b] - (at - s_held[b]));
        p.position[r] = pos;
        if (page < 0 || page >= p.num_pages) {
            record_error(DSPARK_INVALID_PAGE);
            p.slot[r] = -1;
        } else {
            p.slot[r] = page * p.ps + (pos - at * p.ps);
        }
        if (p.token)
            p.token[r] = i == 0 ? p.anchor[b] : p.x[static_cast<size_t>(b) * p.gamma + i - 1];
    }
}

}  // namespace layout
}  // namespace dspark
