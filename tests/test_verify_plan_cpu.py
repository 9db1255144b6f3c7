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
        Request r{in(0, it % 2 ? 3000 : 2000000000), in(1, it % 3 ? 25 : 900), in(1, 112)};
        long long sum = 0;
        for (int q = 0; q < r.query_tiles(); ++q) {
            CHECK(r.before(q) == sum);
            const long long keys = r.ctx + std::min<long long>(r.rows, (q + 1LL) * r.tokens);
            CHECK(r.keys(q) == keys);
            CHECK(r.key_tiles(q) == (keys + kTileKeys - 1) / kTileKeys);
            sum += kUnitCost + r.key_tiles(q);
        }
        CHECK(r.per_head() == sum);
        const int heads = in(1, 8);
        const long long at = static_cast<long long>(rng()) % (sum * heads);
        int h, qt, in_unit;
        place(r, at, h, qt, in_unit);
        CHECK(h * sum + r.before(qt) + in_unit == at);
        CHECK(in_unit >= 0 && in_unit < kUnitCost + r.key_tiles(qt));
    }
    for (int it = 0; it < 400; ++it) {                     // whole batches
        const int B = in(1, 40), heads = in(1, 4), tokens = in(1, 30), most = 148;
        std::vector<Request> req;
        long long T = 0;
        for (int b = 0; b < B; ++b) {
            req.push_back(Request{in(0, it % 4 ? 900 : 30000), in(1, 25), tokens});
            T += req.back().per_head() * heads;
        }
        const int G = ctas(T, most);
        // the line, place by place: (unit, tile) or overhead
        std::vector<int> unit_of, tile_of, tiles;
        for (auto &r : req)
            for (int h = 0; h < heads; ++h)
                for (int q = 0; q < r.query_tiles(); ++q) {
                    for (int c = 0; c < kUnitCost + r.key_tiles(q); ++c) {
                        unit_of.push_back(static_cast<int>(tiles.size()));
                        tile_of.push_back(c - kUnitCost);
                    }
                    tiles.push_back(r.key_tiles(q));
                }
        CHECK(static_cast<long long>(unit_of.size()) == T);
        std::vector<std::vector<int>> parts(tiles.size());
        std::vector<int> seen(tiles.size(), 0);
        for (int c = 0; c < G; ++c) {
            const long long a = first_place(T, c, G), e = first_place(T, c + 1, G);
            CHECK(a < e && e <= T);
            for (long long t = a; t < e; ++t) {
                CHECK(cta_of(T, t, G) == c);
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
