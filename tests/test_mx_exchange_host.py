"""How the CTAs of a K-split cluster exchange partial tiles and leave
(csrc/mx_exchange.h), run on the CPU against a model of the cluster: CTAs as
threads that take turns in a random order, announcements and copies that land
at random times, waits that may run out, main loops that gave up.  In every
run nothing may address a CTA that has left, nor be in flight from or to one,
nor be copied into a ring in use, and every CTA has to end; without a failure
every share has to arrive."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

MODEL = r'''
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <random>
#include <thread>
#include <vector>

#include "mx_exchange.h"

struct Flight { int src, dst; bool share; };

struct Cluster {
    int n, chance;                 // CTAs; a wait runs out with 1 in `chance` looks (0: never)
    std::mt19937 rng;
    std::mutex m;
    std::condition_variable cv;
    int turn = -1, ended = 0, looks = 0;
    const char* wrong = nullptr;
    std::vector<int> alive, announced, shares, expecting, arrived, warned, got;
    std::vector<Flight> flying;

    Cluster(int n, int chance, unsigned seed)
        : n(n), chance(chance), rng(seed), alive(n, 1), announced(n), shares(n), expecting(n), arrived(n), warned(n), got(n) {}
    int pick(int k) { return (int)(rng() % (unsigned)k); }
    void fault(const char* what) { if (!wrong) wrong = what; }
    void touch(int z) { if (!alive[z]) fault("addressed a CTA that has left"); }
    // lets copies land, then somebody else run
    void pass() {
        while (!flying.empty() && pick(3) == 0) {
            const int i = pick((int)flying.size());
            const Flight f = flying[i];
            flying.erase(flying.begin() + i);
            touch(f.dst);
            if (f.share) {
                touch(f.src);
                ++shares[f.dst];
            } else {
                ++announced[f.dst];
            }
        }
        if (++looks > 4000000) { printf("does not end\n"); exit(1); }
        std::vector<int> up;
        for (int i = 0; i < n; ++i) if (alive[i]) up.push_back(i);
        turn = up.empty() ? -1 : up[pick((int)up.size())];
        cv.notify_all();
    }
    void yield(int me, std::unique_lock<std::mutex>& l) {
        pass();
        cv.wait(l, [&] { return turn == me; });
    }
};

struct Link {
    Cluster& c;
    int me;
    std::unique_lock<std::mutex>& l;
    void step() { c.yield(me, l); }
    template <typename F> bool until(F f, bool bounded) {
        for (;;) {
            step();
            if (f()) return true;
            if (bounded && c.chance && c.pick(c.chance) == 0) return false;
        }
    }
    void expect() { step(); c.expecting[me] = 1; }
    void announce(int z) { step(); c.touch(z); c.flying.push_back({me, z, false}); }
    bool await_announced() { return until([&] { return c.announced[me] == c.n; }, true); }
    void send(int z) {
        step();
        c.touch(z);
        if (!c.expecting[z]) c.fault("copied into a ring in use");
        c.flying.push_back({me, z, true});
    }
    bool await_shares() { return until([&] { return c.shares[me] == c.n; }, true); }
    void warn(int z) { step(); c.touch(z); c.warned[z] = 1; }
    void arrive() { step(); c.arrived[me] = 1; }
    void wait() {
        until([&] { for (int a : c.arrived) if (!a) return false; return true; }, false);
    }
    bool warned() { step(); return c.warned[me]; }
    void settle() {
        until([&] { for (const Flight& f : c.flying) if (f.src == me || f.dst == me) return false; return true; }, false);
    }
};

int main() {
    int late = 0;
    for (unsigned seed = 0; seed < 1500; ++seed) {
        const int n = 2 << seed % 3, chance = (int[]){0, 40, 400, 8}[seed / 3 % 4];
        Cluster c(n, chance, seed);
        std::vector<int> delay(n);
        // one CTA's main loop is slow, or gave up long after the others were through
        for (int i = 0; i < n; ++i) delay[i] = c.pick(i == (int)seed % n ? 60 : 5);
        std::vector<std::thread> ts;
        for (int me = 0; me < n; ++me)
            ts.emplace_back([&, me] {
                std::unique_lock<std::mutex> l(c.m);
                c.cv.wait(l, [&] { return c.turn == me; });
                Link k{c, me, l};
                for (int i = 0; i < delay[me]; ++i) k.step();
                c.got[me] = qg::mx_exchange(k, n, true);
                for (int i = c.pick(4); i > 0; --i) k.step();  // the epilogue
                qg::mx_exchange_leave(k);
                c.alive[me] = 0;
                ++c.ended;
                c.pass();
            });
        {
            std::unique_lock<std::mutex> l(c.m);
            c.turn = c.pick(n);
            c.cv.notify_all();
        }
        for (auto& t : ts) t.join();
        for (const Flight& f : c.flying) {
            c.touch(f.dst);
            if (f.share) c.touch(f.src);
        }
        int lost = 0;
        for (int g : c.got) lost += !g;
        if (!chance && lost) c.fault("a share was lost without a failure");
        if (c.wrong) { printf("seed %u, %d CTAs: %s\n", seed, n, c.wrong); return 1; }
        late += lost > 0;
    }
    printf("%d runs with a wait that ran out\n", late);
    return late < 300;
}
'''


def test_nothing_addresses_a_cta_that_has_left(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no host C++ compiler")
    src, exe = tmp_path / "model.cpp", tmp_path / "model"
    src.write_text(MODEL)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-pthread", "-I",
                           os.path.join(ROOT, "quantized_gemm_tcgen05_gb300", "csrc"), str(src), "-o", str(exe)])
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
