"""The attention's work split (csrc/verify_plan.h), compiled for the host: closed forms against
sums, and every key tile of every unit in exactly one CTA, in parts that join in order."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_drafter_head_b200", "csrc")

PROGRAM = r"""
#include "verify_plan.h"
#include <algorithm>
#include <cstdio>
#include <random>
#include <vector>
using namespace dspark::vplan;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main()
{
    std::mt19937 rng(7);
    auto in = [&](int lo, int hi) { return lo + static_cast<int>(rng() % (hi - lo + 1)); };
    for (int it = 0; it < 3000; ++it) {                    // closed forms, far contexts
        const int group = in(1, 20);
        Request r{in(0, it % 2 ? 3000 : 2000000000), in(1, it % 3 ? 25 : 900), in(1, 112 / group),
                  group};
        long long sum = 0;
        for (int q = 0; q < r.query_tiles(); ++q) {
            CHECK(r.before(q) == sum);
            const long long end = std::min<long long>(r.rows, (q + 1LL) * r.tokens);
            CHECK(r.keys(q) == r.ctx + end);
            CHECK(r.key_tiles(q) == (r.ctx + end + kTileKeys - 1) / kTileKeys);
            const int rows = static_cast<int>(end - static_cast<long long>(q) * r.tokens) * group;
            CHECK(r.unit_rows(q) == rows && rows >= 1 && rows <= kMostRows);
            CHECK(r.tile_places(q) == kTilePlaces + (rows + 15) / 16);
            CHECK(r.tile_places(q) <= kMostPlaces);
            sum += kUnitPlaces + static_cast<long long>(r.key_tiles(q)) * r.tile_places(q);
        }
        CHECK(r.per_head() == sum);
        const int heads = in(1, 8);
        const long long at = static_cast<long long>(rng()) % (sum * heads);
        int h, qt, in_unit;
        place(r, at, h, qt, in_unit);
        CHECK(h * sum + r.before(qt) + in_unit == at);
        const int per = r.tile_places(qt), tiles = r.key_tiles(qt);
        CHECK(in_unit >= 0 && in_unit < kUnitPlaces + static_cast<long long>(tiles) * per);
        const int t = tile_at(in_unit, per);
        CHECK(t <= tiles && (t == 0 || kUnitPlaces + (t - 1LL) * per < in_unit));
        CHECK(t == tiles || kUnitPlaces + static_cast<long long>(t) * per >= in_unit);
    }
    for (int it = 0; it < 400; ++it) {                     // whole batches
        const int B = in(1, 40), heads = in(1, 4), most = 148, group = in(1, 8);
        const int tokens = in(1, 112 / group);
        std::vector<Request> req;
        long long T = 0;
        for (int b = 0; b < B; ++b) {
            req.push_back(Request{in(0, it % 4 ? 900 : 30000), in(1, 25), tokens, group});
            T += req.back().per_head() * heads;
        }
        const Split split(T, most);
        const int G = split.G;
        CHECK(G >= 1 && G <= most && (G == 1 || T / G >= kMostPlaces));
        CHECK(split.first(0) == 0 && split.first(G) == T);
        // the line, place by place: the unit, and the tile that starts there or -1
        std::vector<int> unit_of, tile_of, tiles;
        for (auto &r : req)
            for (int h = 0; h < heads; ++h)
                for (int q = 0; q < r.query_tiles(); ++q) {
                    const int per = r.tile_places(q);
                    for (int c = 0; c < kUnitPlaces + r.key_tiles(q) * per; ++c) {
                        const int in_tiles = c - kUnitPlaces;
                        unit_of.push_back(static_cast<int>(tiles.size()));
                        tile_of.push_back(in_tiles >= 0 && in_tiles % per == 0 ? in_tiles / per
                                                                               : -1);
                    }
                    tiles.push_back(r.key_tiles(q));
                }
        CHECK(static_cast<long long>(unit_of.size()) == T);
        std::vector<std::vector<int>> parts(tiles.size());
        std::vector<int> seen(tiles.size(), 0);
        for (int c = 0; c < G; ++c) {
            const long long a = split.first(c), e = split.first(c + 1);
            CHECK(a < e && e <= T && e - a >= T / G && e - a <= T / G + 1);
            for (long long t = a; t < e; ++t) {
                CHECK(split.cta_of(t) == c);
                if (tile_of[t] < 0) continue;
                const int u = unit_of[t];
                CHECK(tile_of[t] == seen[u]);
                ++seen[u];
                if (parts[u].empty() || parts[u].back() != c) parts[u].push_back(c);
            }
        }
        for (size_t u = 0; u < tiles.size(); ++u) {
            CHECK(seen[u] == tiles[u]);
            for (size_t i = 0; i < parts[u].size(); ++i)   // consecutive CTAs
                CHECK(parts[u][i] == parts[u][0] + static_cast<int>(i));
        }
        // a CTA holds at most one part that started before it and one that goes on after it
        for (int c = 0; c < G; ++c) {
            int before = 0, after = 0;
            for (auto &p : parts) {
                for (size_t i = 0; i < p.size(); ++i)
                    if (p[i] == c) before += i > 0, after += i == 0 && p.size() > 1;
            }
            CHECK(before <= 1 && after <= 1);
        }
    }
    std::puts("ok");
    return 0;
}
"""


def test_work_split(tmp_path):
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined",
                           "-fno-sanitize-recover", "-I", CSRC, "-o", str(exe), str(src)])
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr
