// verify_plan.h -- how the attention of a verification batch is cut into work for the CTAs.
//
// A unit is (request, key head, query tile): up to `tokens` of the request's rows, all the
// query heads of one key head, against the keys that the tile's last row sees, in key tiles
// of 128.  All units stand in one line (requests, then key heads, then query tiles), each as
// kUnitPlaces places, what starting and ending it costs, and then tile_places() a key tile, what
// a tile costs; a tile belongs to where its first place is.  Every CTA takes as many places as
// the others, to one: equal work whatever the lengths, a function of the lengths alone.  A unit
// whose tiles are cut by a border is joined from its parts.
//
// A tile's cost is its 64 KB and, a little, its rows: tiles of 16 rows took 2430 cycles, of 48
// 2680 and of 80 2860 where all of them shared the memory's rate.  A unit's own: 64 requests of
// 100 to 3000 keys took 82.8 us with places for three tiles of 16 rows, 81.5 with two, 81.7 with
// one and a half.
//
// Plain integer arithmetic, the same on the host and the device.
#pragma once

#ifdef __CUDACC__
#define DSPARK_HD __host__ __device__ __forceinline__
#define DSPARK_HD_CALL __host__ __device__ __noinline__
#else
#define DSPARK_HD inline
#define DSPARK_HD_CALL inline
#endif

namespace dspark {
namespace vplan {

constexpr int kTileKeys = 128;
constexpr int kTilePlaces = 24;                   // of a tile, and one for each 16 rows
constexpr int kUnitPlaces = 50;                   // of a unit: two tiles of 16 rows
constexpr int kMostRows = 112;
constexpr int kMostPlaces = kTilePlaces + kMostRows / 16;

// a / b, both at least 0: a 64-bit division takes the device several times a 32-bit one's time,
// and the kernel's first copies wait for these
DSPARK_HD long long quotient(long long a, long long b)
{
    if ((a | b) >> 31 == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
    return a / b;
}

// Key tiles of query tiles 0 .. n - 1, all of them full: the sum of floor(e / 128) over the ends
// e = b, b + a, ..., b + (n - 1) a (a, b >= 0).
//
// An end's place in its key tile, e mod 128, comes back after 128 query tiles, in which the ends
// have moved by a whole key tiles.  So with n = 128 u + v the u whole rounds follow from the first:
// its places run through the classes r, r + g, r + 2 g, ... below 128 (g = gcd(a, 128), a power
// of two; r = b mod g) g times each, so they add up to 64 (128 - g + 2 r), and what is left of the
// ends' sum is 128 times their tiles'.  The v ends behind the last round are added up one by one:
// 127 at most, of an addition and a shift each, where divisions by the step take longer.
// (a call: only requests of three query tiles or more come here, and inlined where it is used it
// is most of what a CTA fetches as instructions before its first copy)
DSPARK_HD_CALL long long tiles_of(long long n, int a, long long b)
{
    static_assert(kTileKeys == 128, "the shifts below");
    const long long u = n >> 7;
    const int v = static_cast<int>(n & 127);
    const int g = (a | 128) & -(a | 128);             // gcd(a, 128)
    const int r = static_cast<int>(b & (g - 1));
    // tiles of the first round: (sum of its ends - sum of their places) / 128
    const long long round = b + ((127ll * a - (128 - g + 2 * r)) >> 1);
    long long sum = u * round + 64 * a * u * (u - 1);
    const long long from = b + 128 * a * u;           // the first end behind the rounds
    int e = static_cast<int>(from & 127), part = 0;
    for (int i = 0; i < v; ++i, e += a) part += e >> 7;
    return sum + v * (from >> 7) + part;
}

struct Request {
    int ctx, rows;     // rows > 0
    int tokens;        // tokens of a query tile
    int group;         // rows (query heads) of a token

    DSPARK_HD int query_tiles() const
    {
        return rows <= tokens ? 1 : (rows + tokens - 1) / tokens;
    }
    // keys that query tile qt sees, and its key tiles
    DSPARK_HD int keys(int qt) const
    {
        const long long end = (static_cast<long long>(qt) + 1) * tokens;
        return ctx + static_cast<int>(end < rows ? end : rows);
    }
    DSPARK_HD int key_tiles(int qt) const { return (keys(qt) - 1) / kTileKeys + 1; }
    DSPARK_HD int unit_rows(int qt) const
    {
        const long long left = rows - static_cast<long long>(qt) * tokens;
        return static_cast<int>(left < tokens ? left : tokens) * group;
    }
    DSPARK_HD int tile_places(int qt) const { return kTilePlaces + (unit_rows(qt) + 15) / 16; }
    // places of query tiles 0 .. qt - 1, all but the last of which may be full
    DSPARK_HD long long before(int qt) const
    {
        if (qt <= 0) return 0;
        const int full = qt < query_tiles() ? qt : query_tiles() - 1;
        long long sum = 0;
        if (full > 0)
            sum = tiles_of(full, tokens, static_cast<long long>(ctx) + tokens + kTileKeys - 1) *
                  tile_places(0);
        if (full < qt) sum += static_cast<long long>(key_tiles(full)) * tile_places(full);
        return sum + static_cast<long long>(qt) * kUnitPlaces;
    }
    DSPARK_HD long long per_head() const { return before(query_tiles()); }
};

// T places over G CTAs: the first `more` of them take `each` + 1, the others `each`.
struct Split {
    long long each, more;
    int G;

    // Each CTA that takes part has as many places as the largest tile at least, so that no CTA
    // between a unit's first and last is without a tile of it.
    DSPARK_HD Split(long long T, int most)
    {
        G = T >= static_cast<long long>(most) * kMostPlaces ? most
            : T < kMostPlaces                               ? (T > 0)
                                                            : static_cast<int>(T / kMostPlaces);
        each = G > 0 ? quotient(T, G) : 0;
        more = T - each * G;
    }
    // first place of CTA c
    DSPARK_HD long long first(int c) const { return each * c + (c < more ? c : more); }
    // the CTA that holds place t
    DSPARK_HD int cta_of(long long t) const
    {
        const long long cut = (each + 1) * more;
        return static_cast<int>(t < cut ? quotient(t, each + 1) : more + quotient(t - cut, each));
    }
};
// the first key tile that starts at place `at` of a unit or later
DSPARK_HD int tile_at(long long at, int tile_places)
{
    return at <= kUnitPlaces
               ? 0
               : static_cast<int>(quotient(at - kUnitPlaces + tile_places - 1, tile_places));
}

// Place `at` of a request with per_head() * heads places: key head, query tile, place in the unit.
DSPARK_HD void place(const Request &r, long long at, int &h, int &qt, int &in_unit)
{
    const long long per = r.per_head();
    h = static_cast<int>(quotient(at, per));
    const long long rest = at - h * per;
    int lo = 0, hi = r.query_tiles() - 1;
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (r.before(mid) <= rest) lo = mid;
        else hi = mid - 1;
    }
    qt = lo;
    in_unit = static_cast<int>(rest - r.before(lo));
}

}  // namespace vplan
}  // namespace dspark
