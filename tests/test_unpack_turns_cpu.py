"""The rings of the tiled packed-weight products under random schedules, compiled as plain C++ (no GPU).

csrc/unpack_turns.h says which set of unpacking warps takes which half of a step. The program runs the roles of k_matmul_tc as fibers over barriers that know a phase by its
parity alone, as an mbarrier does: the warps that copy words and rows, the three unpacking sets, the
warp that issues the products, and the units that complete copies and products. Each schedule holds some
roles back for long stretches. Every piece of a stage carries the number of the step it was made for:
  - a set reads the words of its step, also at the end of its reading;
  - nothing is written into an operand stage that a product has yet to read;
  - a product reads both halves and the rows of its own step;
  - every role comes to its end.
"""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_weight_quantization_solve_b200", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <deque>
#include <functional>
#include <memory>
#include <random>
#include <string>
#include <vector>
#include <ucontext.h>
#include "unpack_turns.h"
using namespace gptq;

// ---- fibers --------------------------------------------------------------------------------
struct Fiber { ucontext_t ctx; std::function<void()> body; bool done = false; int held = 0; std::vector<char> stack; };
static ucontext_t main_ctx;
static std::vector<std::unique_ptr<Fiber>> fibers;
static Fiber *current;
static long progress;                       // barrier completions and steps: a standstill has none
static void start() { current->body(); current->done = true; swapcontext(&current->ctx, &main_ctx); }
static void yield() { swapcontext(&current->ctx, &main_ctx); }
static void spawn(std::function<void()> f) {
    auto p = std::make_unique<Fiber>();
    p->body = std::move(f);
    p->stack.resize(64 * 1024);
    getcontext(&p->ctx);
    p->ctx.uc_stack.ss_sp = p->stack.data();
    p->ctx.uc_stack.ss_size = p->stack.size();
    p->ctx.uc_link = &main_ctx;
    makecontext(&p->ctx, start, 0);
    fibers.push_back(std::move(p));
}

struct RingPos {
    int stage = 0;
    uint32_t phase = 0;
    void advance(int n) { if (++stage == n) { stage = 0; phase ^= 1u; } }
    void to(int steps, int n) { for (; steps > 0; --steps) advance(n); }
};

struct Bar {
    int count = 1, left = 1;
    unsigned phase = 0;
    void init(int n) { count = left = n; phase = 0; }
    bool test(uint32_t parity) const { return (phase & 1u) != parity; }
    void arrive() { if (--left == 0) { left = count; ++phase; ++progress; } }
};
static void wait(const Bar &b, uint32_t parity) { while (!b.test(parity)) yield(); }

// halves: a stage of words is half a step's. restart: the adapters' halves from the first set again for
// each tile
struct Config { int stages, ring, main_steps, tiles; bool adapters, halves, restart, copies_in_order; };
static std::string fault;
static void blame(const char *what) { if (fault.empty()) fault = what; }

static std::string run(const Config &c, unsigned seed) {
    std::mt19937 rng(seed);
    auto pick = [&](int n) { return (int)(rng() % (unsigned)n); };
    fibers.clear();
    fault.clear();
    progress = 0;
    std::vector<int> extra(c.tiles);                    // adapters' steps of each tile
    for (int &e : extra) e = c.adapters ? pick(3) * (1 + pick(2)) : 0;

    Bar wfull[8], wempty[8], full[4], empty[4];
    int words[8], half[4][2], rows[4], unread[4] = {0, 0, 0, 0};
    for (int i = 0; i < 8; ++i) { wfull[i].init(1); wempty[i].init(c.halves ? 1 : 2); words[i] = -1; }
    for (int i = 0; i < 4; ++i) { full[i].init(3); empty[i].init(1); half[i][0] = half[i][1] = rows[i] = -1; }
    std::deque<std::function<void()>> copies;
    std::deque<std::pair<int, int>> products;           // stage, step
    int left = 6;                                       // roles at work

    spawn([&] {                                         // words
        RingPos p;
        for (int t = 0, s = 0; t < c.tiles; ++t)
            for (int i = 0; i < c.main_steps * (c.halves ? 2 : 1); ++i, ++s) {
                wait(wempty[p.stage], p.phase ^ 1);
                const int at = p.stage;
                copies.push_back([&, at, s] { words[at] = s; wfull[at].arrive(); });
                p.advance(c.ring);
            }
        --left;
    });
    spawn([&] {                                         // rows
        RingPos p;
        for (int t = 0, s = 0; t < c.tiles; ++t)
            for (int i = 0; i < c.main_steps + extra[t]; ++i, ++s) {
                wait(empty[p.stage], p.phase ^ 1);
                const int at = p.stage;
                auto land = [&, at, s] { rows[at] = s; full[at].arrive(); };
                if (i < c.main_steps) copies.push_back(land);
                else land();
                p.advance(c.stages);
            }
        --left;
    });
    for (int set = 0; set < 3; ++set)
        spawn([&, set] {
            RingPos ops, in;
            int ops_step = 0, in_step = 0, first_step = 0, first_words = 0, turn = 0;
            auto put = [&](int side, int step) {
                ops.to(step - ops_step, c.stages);
                ops_step = step;
                const int at = ops.stage;
                wait(empty[at], ops.phase ^ 1);
                if (unread[at] & (1 << side)) blame("a stage overwritten");
                unread[at] |= 1 << side;
                half[at][side] = step;
                yield();
                full[at].arrive();
            };
            for (int t = 0; t < c.tiles; ++t) {
                for (int h = unpack_first_half(set, turn); h < 2 * c.main_steps; h += UNPACK_SETS) {
                    const int w = first_words + (c.halves ? h : h >> 1);
                    in.to(w - in_step, c.ring);
                    in_step = w;
                    const int at = in.stage;
                    wait(wfull[at], in.phase);
                    if (words[at] != w) blame("words of another step");
                    yield();
                    if (words[at] != w) blame("words changed while read");
                    wempty[at].arrive();
                    put(h & 1, first_step + (h >> 1));
                }
                turn = unpack_next_turn(turn, 2 * c.main_steps);
                first_words += c.main_steps * (c.halves ? 2 : 1);
                first_step += c.main_steps;
                for (int h = 0; h < 2 * extra[t]; ++h)
                    if ((c.restart ? h % 3 : unpack_adapter_set(turn, h, 2 * extra[t])) == set)
                        put(h & 1, first_step + (h >> 1));
                first_step += extra[t];
            }
            --left;
        });
    spawn([&] {                                         // issue of the products
        RingPos p;
        for (int t = 0, s = 0; t < c.tiles; ++t)
            for (int i = 0; i < c.main_steps + extra[t]; ++i, ++s) {
                wait(full[p.stage], p.phase);
                products.push_back({p.stage, s});
                p.advance(c.stages);
            }
        --left;
    });
    spawn([&] {                                         // copies land
        while (left > 0 || !copies.empty()) {
            if (!copies.empty()) {
                const int i = c.copies_in_order ? 0 : pick((int)copies.size());
                auto f = copies[i];
                copies.erase(copies.begin() + i);
                f();
            }
            yield();
        }
    });
    spawn([&] {                                         // products complete, in order
        while (left > 0 || !products.empty()) {
            if (!products.empty()) {
                const auto [at, s] = products.front();
                yield();
                if (half[at][0] != s || half[at][1] != s || rows[at] != s) blame("a product of another step's operands");
                products.pop_front();
                unread[at] = 0;
                empty[at].arrive();
            }
            yield();
        }
    });

    long seen = 0, idle = 0;
    while (fault.empty()) {
        bool any = false;
        const int n = (int)fibers.size(), from = pick(n);
        for (int i = 0; i < n; ++i) {
            Fiber &f = *fibers[(from + i) % n];
            if (f.done) continue;
            any = true;
            if (f.held > 0) { --f.held; continue; }
            if (pick(24) == 0) { f.held = pick(60); continue; }
            current = &f;
            swapcontext(&main_ctx, &f.ctx);
        }
        if (!any) break;
        if (progress != seen) { seen = progress; idle = 0; }
        else if (++idle > 20000) blame("a standstill");
    }
    return fault;
}

static int faults(Config c, const std::vector<int> &rings, int seeds) {
    int bad = 0;
    for (int seed = 0; seed < seeds && bad < 3; ++seed) {
        std::mt19937 r(seed * 7919 + 13);
        c.stages = 2 + (int)(r() % 3u);
        c.ring = rings[r() % rings.size()];
        c.main_steps = 1 + (int)(r() % 9u);
        c.tiles = 1 + (int)(r() % 5u);
        const std::string f = run(c, seed);
        if (!f.empty()) {
            std::fprintf(stderr, "%s: stages %d ring %d steps %d tiles %d seed %d\n", f.c_str(), c.stages, c.ring,
                         c.main_steps, c.tiles, seed);
            ++bad;
        }
    }
    return bad;
}

int main(int argc, char **argv) {
    const std::string what = argv[1];
    Config c{};
    c.adapters = what.find("main") == std::string::npos;
    c.halves = what.find("halves") != std::string::npos;
    c.restart = what == "restart";
    std::vector<int> rings = {3, 6};
    if (what.find("two stages") != std::string::npos) rings = {2};
    if (what.find("four stages") != std::string::npos) rings = {4};
    std::printf("%d\n", faults(c, rings, 4000));
}
"""


@pytest.fixture(scope="module")
def faults(tmp_path_factory):
    folder = tmp_path_factory.mktemp("ring")
    src, exe = folder / "ring.cpp", folder / "ring"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def count(what):
        r = subprocess.run([str(exe), what], capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr
        return int(r.stdout), r.stderr

    return count


@pytest.mark.parametrize("what", ["main", "adapters", "main halves", "adapters halves"])
def test_rings(faults, what):
    n, first = faults(what)
    assert n == 0, first


def test_the_program_sees_a_set_that_falls_behind(faults):
    # the adapters' halves from the first set again for each tile: a set may pass over three steps
    n, first = faults("restart")
    assert n > 0 and "standstill" not in first


@pytest.mark.parametrize("what", ["main two stages", "main halves four stages"])
def test_the_program_sees_words_that_land_late(faults, what):
    # a stage that a set meets every other time, filled by copies that land in any order
    n, first = faults(what)
    assert n > 0 and "words" in first


def test_any_two_steps_hold_every_set(tmp_path):
    src, exe = tmp_path / "turns.cpp", tmp_path / "turns"
    src.write_text(r"""
#include <cstdio>
#include <vector>
#include "unpack_turns.h"
using namespace gptq;
int main() {
    int bad = 0;
    for (int steps = 1; steps <= 7; ++steps)
        for (int extra = 0; extra < 4096; ++extra) {                // adapters' steps of four tiles
            std::vector<int> owner;
            int turn = 0;
            for (int t = 0; t < 4; ++t) {
                std::vector<int> tile(2 * steps, -1);
                for (int set = 0; set < UNPACK_SETS; ++set)
                    for (int h = unpack_first_half(set, turn); h < 2 * steps; h += UNPACK_SETS) tile[h] = set;
                owner.insert(owner.end(), tile.begin(), tile.end());
                turn = unpack_next_turn(turn, 2 * steps);
                const int n = 2 * ((extra >> (3 * t)) & 7);
                for (int i = 0; i < n; ++i) owner.push_back(unpack_adapter_set(turn, i, n));
            }
            for (size_t h = 0; h + 4 <= owner.size(); h += 2) {
                int seen = 0;
                for (int i = 0; i < 4; ++i) seen |= 1 << owner[h + i];
                bad += seen != 7 || owner[h] == owner[h + 1];
            }
        }
    std::printf("%d\n", bad);
}
""")
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, timeout=600).stdout.strip() == "0"
