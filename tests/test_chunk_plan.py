"""The division of gdn_attn_chunk's work (csrc/gdn_chunk_plan.h, host code as well): every tile of every unit has one worker, the
parts of a unit follow one another, and what the join takes for granted holds (CPU only)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <tuple>
#include <vector>
#include "gdn_chunk_plan.h"
using namespace gdn::chunk;
#define NEED(x) do { if (!(x)) { std::printf("%s\n", #x); return 1; } } while (0)

int main() {
    std::srand(1);
    for (int it = 0; it < 6000; ++it) {
        const int G = 1 + std::rand() % 16, RT = std::rand() % 2 ? 256 : 64, costs[4] = {1, 64, 200, 700};
        const Line ln{RT / G, std::rand() % 2 ? 7 : 6, costs[std::rand() % 4]};
        const int B = 1 + std::rand() % 6, Hkv = 1 + std::rand() % 3;
        std::vector<Rows> rs;
        std::vector<long long> start;
        long long total = 0;
        for (int b = 0, row = 0; b < B; ++b) {
            const int n = std::rand() % 4 == 0 ? 0 : std::rand() % (std::rand() % 2 ? 5 : 600);
            const int len = std::rand() % 8 == 0 ? std::rand() % (n + 1) : n + (std::rand() % 3 ? std::rand() % 3000 : 0);
            const Rows r{row, n, len};
            long long h = 0;
            for (int i = 0; n > 0 && i < ln.units(r); ++i) {
                NEED(ln.before(r, i) == h);
                h += ln.cost + ln.seen(r, i);
            }
            NEED(h == ln.head(r));
            start.push_back(total);
            rs.push_back(r);
            total += h * Hkv;
            row += n;
        }
        if (total == 0) continue;
        const int W = workers_of(total, 1 + std::rand() % 500, (std::rand() % 2 ? 1 : 2) * ln.keys());
        std::map<std::tuple<int, int, int>, std::vector<std::pair<int, Part>>> got;
        auto rows = [&](int b) { return rs[b]; };
        for (int w = 0; w < W; ++w) {
            const Share sh = Share::of(total, W, w);
            int b = 0, begins = 0, goes_on = 0;
            while (b + 1 < B && start[b + 1] <= sh.first) ++b;
            Part c{};
            c.b = b;
            c.r = rs[b];
            for (bool ok = first_part(ln, sh, start[b], c) || next_part(ln, sh, B, Hkv, c, rows); ok; ok = next_part(ln, sh, B, Hkv, c, rows)) {
                got[std::make_tuple(c.b, c.hk, c.i)].push_back({w, c});
                if (!c.whole()) ++(c.t0 == 0 ? begins : goes_on);
            }
            NEED(begins <= 1 && goes_on <= 1);   // the two places of a worker
        }
        size_t units = 0;
        for (int b = 0; b < B; ++b)
            for (int h = 0; h < Hkv; ++h)
                for (int i = 0; rs[b].n > 0 && i < ln.units(rs[b]); ++i, ++units) {
                    const auto& v = got[std::make_tuple(b, h, i)];
                    NEED(!v.empty());
                    int t = 0;
                    for (const auto& x : v) {
                        NEED(x.second.t0 == t && x.second.t1 >= t);
                        t = x.second.t1;
                    }
                    const Part c = v[0].second;
                    NEED(t == c.tiles && (c.tiles > 0 || v.size() == 1));
                    if (c.tiles == 0) continue;
                    const Share sh = Share::of(total, W, 0);
                    const long long base = c.at + ln.cost;
                    const int w0 = sh.owner(base), w1 = sh.owner(base + static_cast<long long>(ln.keys()) * (c.tiles - 1));
                    NEED(w0 == v.front().first && w1 == v.back().first && w1 - w0 + 1 == static_cast<int>(v.size()));
                }
        NEED(units == got.size());
    }
    std::printf("ok\n");
    return 0;
}
"""


def test_every_tile_has_one_worker(tmp_path):
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(DRIVER)
    csrc = os.path.join(ROOT, "gated_deltanet_linear_decode_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I", csrc, str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
