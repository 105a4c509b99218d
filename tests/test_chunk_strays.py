"""How a pair's CTAs agree on a part's infinite and NaN values (csrc/gdn_chunk_strays.h): a model of the softmax warps of both CTAs with
the header's own code, their barriers, and steps in a random order, some warps far slower than others (CPU only)."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_deltanet_linear_decode_gb300", "csrc")

DRIVER = r"""
#include <coroutine>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "gdn_chunk_strays.h"
using gdn::chunk::Strays;

struct Task {
    struct promise_type {
        Task get_return_object() { return {std::coroutine_handle<promise_type>::from_promise(*this)}; }
        std::suspend_always initial_suspend() { return {}; }
        std::suspend_always final_suspend() noexcept { return {}; }
        void return_void() {}
        void unhandled_exception() { std::abort(); }
    };
    std::coroutine_handle<promise_type> h;
};
#define STEP co_await std::suspend_always{}
#define UNTIL(x) while (!(x)) STEP

constexpr int kWarps = 2;            // of a group
struct Barrier {                     // of a CTA's softmax warps
    int n = 0, phase = 0;
};
struct Part {
    int tiles;
    std::vector<int> finders;        // by tile: bit 4 * cta + warp of the tile's group: that warp finds strays
};
struct World {
    bool f32, live;                  // live: the mistake that this is about, warps that go by the marks themselves
    int ns;                          // places of scores
    std::vector<Part> parts;
    Strays cta[2];
    bool ever[2] = {false, false};
    Barrier bar[2];
    std::vector<int> p_ready, given[2][kWarps];
    std::vector<char> pv_done;
    int wrong = 0, done = 0;
};

Task warp(World& w, int cta, int half, int id) {
    auto& bar = w.bar[cta];
    int g = 0;
#define SYNC do { const int ph = bar.phase; if (++bar.n == 2 * kWarps) { bar.n = 0; ++bar.phase; } UNTIL(bar.phase != ph); } while (0)
    for (size_t i = 0; i < w.parts.size(); ++i) {
        const Part& pt = w.parts[i];
        const int g0 = g;
        for (int t = 0; t < pt.tiles; ++t, ++g) {
            if ((g & 1) != half) continue;
            UNTIL(g < w.ns || w.pv_done[g - w.ns]);   // its scores are there
            STEP;
            if (!w.f32 && g > 0) UNTIL(w.given[cta][id][g - 1]);
            if (!w.f32) w.given[cta][id][g] = 1;
            STEP;
            if ((pt.finders[t] >> (4 * cta + id)) & 1) {
                volatile int* const mark = w.cta[cta].mark();
                *mark = 1;
                w.ever[cta] = true;
                STEP;
                *(w.cta[cta ^ 1].found + (mark - w.cta[cta].found)) = 1;   // the same place in the other CTA
                w.ever[cta ^ 1] = true;
                STEP;
            }
            ++w.p_ready[g];
            STEP;
        }
        const bool any = pt.tiles > 0;
        const int mine = w.f32 ? ((g - 1 - half) & 1 ? g - 2 : g - 1) : g - 1;
        if (any && mine >= g0) UNTIL(w.pv_done[mine]);
        STEP;
        if (((g - 1) & 1) == half && id == 0) w.cta[cta].take_over(any);
        STEP;
        SYNC;
        STEP;
        bool truth = false;
        for (int f : pt.finders) truth |= f != 0;
        const bool strays = w.live ? w.ever[cta] : w.cta[cta].now != 0;
        if (!w.live && strays != truth) ++w.wrong;
        STEP;
        if (strays) SYNC;
        STEP;
        SYNC;
    }
    ++w.done;
}

// true: all warps have come to the end, and none went wrong
bool run(unsigned seed, bool live) {
    std::mt19937 rng(seed);
    auto pick = [&](int n) { return static_cast<int>(rng() % n); };
    World w;
    w.live = live;
    w.f32 = pick(2);
    w.ns = w.f32 ? 2 : 2 + pick(2);
    for (Strays& s : w.cta) s.clear();
    int tiles = 0;
    for (int i = 0, n = 2 + pick(7); i < n; ++i) {
        Part p{pick(3) ? 1 + pick(4) : 0, {}};
        for (int t = 0; t < p.tiles; ++t) {
            const int f = pick(3) ? 0 : rng() & 0xff;
            p.finders.push_back(f & 0x33);
        }
        tiles += p.tiles;
        w.parts.push_back(p);
    }
    w.p_ready.assign(tiles, 0);
    w.pv_done.assign(tiles, 0);
    for (auto& c : w.given)
        for (auto& v : c) v.assign(tiles, 0);
    std::vector<Task> tasks;
    std::vector<int> weight;
    for (int cta = 0; cta < 2; ++cta)
        for (int half = 0; half < 2; ++half)
            for (int id = 0; id < kWarps; ++id) {
                tasks.push_back(warp(w, cta, half, id));
                weight.push_back(pick(2) ? 1 : 40);
            }
    int next = 0;   // products, in order
    bool ok = false;
    for (long it = 0; it < 200000 && !ok; ++it) {
        const int i = pick(static_cast<int>(tasks.size()) + 1);
        if (i == static_cast<int>(tasks.size())) {
            if (next < tiles && w.p_ready[next] == 2 * kWarps && pick(2)) w.pv_done[next++] = 1;
        } else if (!tasks[i].h.done() && pick(weight[i]) == 0) {
            tasks[i].h.resume();
        }
        ok = w.done == static_cast<int>(tasks.size());
    }
    for (Task& t : tasks) t.h.destroy();
    return ok && w.wrong == 0;
}

int main(int argc, char** argv) {
    const bool live = argc > 1;
    int bad = 0;
    for (unsigned s = 0; s < 3000 && (!live || !bad); ++s) bad += !run(s, live);
    std::printf("%d\n", bad);
    return 0;
}
"""


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    d = tmp_path_factory.mktemp("strays")
    (d / "strays.cpp").write_text(DRIVER)
    subprocess.run(["g++", "-std=c++20", "-O1", "-I", CSRC, str(d / "strays.cpp"), "-o", str(d / "strays")], check=True)
    return lambda *a: int(subprocess.run([str(d / "strays"), *a], capture_output=True, text=True, check=True, timeout=600).stdout)


def test_both_ctas_agree_whatever_the_order_of_their_steps(model):
    assert model() == 0


def test_the_model_sees_warps_that_go_by_the_other_ctas_mark(model):
    assert model("live") > 0


def test_no_warp_branches_on_what_the_other_cta_writes():
    """In the kernel, what a remote store reaches is never asked in a condition: barriers lie behind those."""
    src = re.sub(r"//.*", "", open(os.path.join(CSRC, "gdn_chunk_tc.cu")).read())
    stores = re.findall(r"st\.shared::cluster\.u32[^;]*;\"[^;]*in_cta\(smem_u32\(([^;]*?)\), rank", src)
    assert len(stores) == 1 and "mark" in stores[0], stores
    assert "sm.strays.found" not in src
    uses = set(re.findall(r"sm\.strays\.(\w+)", src)) | {"bare" for _ in re.findall(r"sm\.strays\b(?!\.)", src)}
    assert uses == {"clear", "mark", "take_over", "now"}, uses
