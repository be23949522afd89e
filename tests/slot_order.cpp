// A simulation, on the CPU, of the barriers of one block of the 16-bit tensor-core role: csrc/attn_slots.h is the code the
// kernel's issuing warps run.  Actors are threads of control that one scheduler steps in a random order, so a schedule is
// repeatable by its seed:
//   the copying warp   arms a stage once it is released, and starts its copy (K runs a tile ahead of V inside an item)
//   the copies         land at any later time, each in its own
//   two issuing warps  slot_item; products read their stage from issue to completion
//   the products       complete at any later time, a slot's in order, and then arrive at the barriers committed behind them
//   two softmaxes      queries, weights
// A barrier is what an mbarrier is: pending arrivals (and bytes) of the current phase; a wait by parity passes when the
// parity differs from the current phase's.  Checked: whoever passes a wait for a tile finds that tile in the stage; nothing is
// copied into a stage that a product still reads, or that holds a tile somebody still waits for; everything ends.
#include <condition_variable>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <deque>
#include <functional>
#include <memory>
#include <mutex>
#include <random>
#include <thread>
#include <vector>

#include "attn_slots.h"

namespace {

struct Bar {
    int count = 1, pending = 1, bytes = 0;
    unsigned phase = 0;
    void init(int c) {
        count = pending = c;
        bytes = 0;
        phase = 0;
    }
    void turn() {
        if (pending == 0 && bytes == 0) {
            ++phase;
            pending = count;
        }
    }
    void arrive() {
        --pending;
        turn();
    }
    bool passed(int parity) const { return (phase & 1u) != ((unsigned)parity & 1u); }
};

// Actors as threads of which one runs at a time, handed on at every wait and event.
struct Sim {
    std::mutex m;
    std::condition_variable cv;
    std::vector<bool> done;
    std::vector<std::function<bool()>> ready;  // what an actor waits for
    int turn = -1;
    std::mt19937 rng;
    std::deque<std::pair<int, std::function<void()>>> later;  // (queue, event): events of one queue come in order
    bool dead = false;

    explicit Sim(unsigned seed) : rng(seed) {}

    // Called by the actor that runs: lets the scheduler pick; returns when this actor is picked again and `r` holds.
    bool yield(int me, std::function<bool()> r) {
        std::unique_lock<std::mutex> l(m);
        ready[me] = std::move(r);
        turn = -1;
        cv.notify_all();
        cv.wait(l, [&] { return turn == me || dead; });
        return !dead;
    }
    void run(const std::vector<std::function<void(int)>> &actors, int lazy) {
        const int n = (int)actors.size();
        done.assign(n, false);
        ready.assign(n, [] { return true; });
        std::vector<std::thread> th;
        for (int i = 0; i < n; ++i)
            th.emplace_back([&, i] {
                {
                    std::unique_lock<std::mutex> l(m);
                    cv.wait(l, [&] { return turn == i || dead; });
                    if (dead) return;
                }
                actors[i](i);
                std::unique_lock<std::mutex> l(m);
                done[i] = true;
                turn = -1;
                cv.notify_all();
            });
        std::unique_lock<std::mutex> l(m);
        for (;;) {
            cv.wait(l, [&] { return turn == -1; });
            std::vector<int> can;
            for (int i = 0; i < n; ++i)
                if (!done[i] && ready[i]()) can.push_back(i);
            std::vector<int> ev;  // the first event of each queue
            std::vector<int> seen;
            for (int i = 0; i < (int)later.size(); ++i) {
                bool first = true;
                for (int q : seen) first &= q != later[i].first;
                if (first) ev.push_back(i), seen.push_back(later[i].first);
            }
            const bool event = !ev.empty() && (can.empty() || (int)(rng() % 100) >= lazy);
            if (event) {
                const int i = ev[rng() % ev.size()];
                auto f = later[i].second;
                later.erase(later.begin() + i);
                f();
                continue;
            }
            if (can.empty()) {
                for (int i = 0; i < n; ++i)
                    if (!done[i]) dead = true;
                break;
            }
            turn = can[rng() % can.size()];
            cv.notify_all();
        }
        cv.notify_all();
        l.unlock();
        for (auto &t : th) t.join();
    }
};

struct Item {
    int n;
    bool both;
};

struct Block {
    int ns;
    std::vector<Bar> full[2], empty[2];  // K, V; a full barrier for each taker and stage
    Bar q_full[2], s_full[2], p_half[2], p_full[2], pv_done[2];
    std::vector<int> holds[2], readers[2];  // tile that has landed in a stage (-1: none), products reading it
    const char *fault = nullptr;
    void bad(const char *what) {
        if (!fault) fault = what;
    }
};

template <int NS>
const char *simulate(const std::vector<Item> &items, unsigned seed, int lazy) {
    constexpr int ns = NS;
    Sim sim(seed);
    Block b;
    b.ns = ns;
    for (int kv = 0; kv < 2; ++kv) {
        b.full[kv].resize(l2::kTakers * ns);
        b.empty[kv].resize(ns);
        for (auto &x : b.full[kv]) x.init(1);
        for (auto &x : b.empty[kv]) x.init(2);
        b.holds[kv].assign(ns, -1);
        b.readers[kv].assign(ns, 0);
    }
    for (int s = 0; s < 2; ++s)
        for (Bar *x : {&b.q_full[s], &b.s_full[s], &b.p_half[s], &b.p_full[s], &b.pv_done[s]}) x->init(1);

    auto wait = [&](int me, Bar &bar, int parity) { return sim.yield(me, [&bar, parity] { return bar.passed(parity); }); };
    auto copier = [&](int me) {
        int t = 0;
        auto copy = [&](int kv, int tt, int taker) {
            const int st = tt % ns;
            if (tt >= ns && !wait(me, b.empty[kv][st], tt / ns - 1)) return false;
            if (b.readers[kv][st]) b.bad("a stage is copied into while a product reads it");
            b.holds[kv][st] = -1;
            Bar &f = b.full[kv][taker * ns + st];
            f.bytes += 1;
            f.arrive();
            sim.later.emplace_back(2 + kv * ns + st, [&b, &f, kv, st, tt] {
                b.holds[kv][st] = tt;
                f.bytes -= 1;
                f.turn();
            });
            return true;
        };
        for (const Item &g : items) {
            for (int i = 0; i <= g.n; ++i) {
                if (i < g.n && !copy(0, t + i, l2::taker_of(i, g.both))) return;
                if (i > 0 && !copy(1, t + i - 1, l2::taker_of(i - 1, g.both))) return;
            }
            t += g.n;
        }
        for (int tt = t > ns ? t - ns : 0; tt < t; ++tt)
            for (int kv = 0; kv < 2; ++kv)
                if (!wait(me, b.empty[kv][tt % ns], tt / ns)) return;
    };
    auto issuer = [&](int s) {
        return [&, s](int me) {
            int t0 = 0, n_p = 0, nq = 0;
            l2::Phases<NS> phases[2];
            for (const Item &g : items) {
                auto queries = [&]() { return wait(me, b.q_full[s], nq++); };
                auto see = [&](int kv, int t) {
                    const int st = t % ns, taker = l2::taker_of(t - t0, g.both);
                    if (!wait(me, b.full[kv][taker * ns + st], phases[kv].next(taker, st))) return false;
                    if (b.holds[kv][st] != t) b.bad("a wait for a tile passed before it was there");
                    return true;
                };
                // queue s: this slot's products complete in order, and their commits arrive behind them
                auto start = [&](int kv, int t) {
                    const int st = t % ns;
                    if (b.holds[kv][st] != t) b.bad("a product reads a stage that does not hold its tile");
                    ++b.readers[kv][st];
                };
                auto commit = [&](int kv, int t, Bar &after) {
                    const int st = t % ns;
                    sim.later.emplace_back(s, [&b, kv, st, &after, both = g.both] {
                        --b.readers[kv][st];
                        after.arrive();
                        b.empty[kv][st].arrive();
                        if (!both) b.empty[kv][st].arrive();  // for the slot that does not use it
                    });
                };
                auto see_k = [&](int t) { return see(0, t); };
                auto see_v = [&](int t) { return see(1, t); };
                auto scores = [&](int t) {
                    start(0, t);
                    commit(0, t, b.s_full[s]);
                };
                auto weights = [&]() { return wait(me, b.p_half[s], n_p++); };
                auto products = [&](int t, bool) {
                    start(1, t);
                    if (!wait(me, b.p_full[s], n_p - 1)) return false;
                    commit(1, t, b.pv_done[s]);
                    return true;
                };
                auto drained = [&]() { return wait(me, b.pv_done[s], n_p - 1); };
                if (!l2::slot_item(s, t0, g.n, g.both, queries, see_k, see_v, scores, weights, products, drained)) return;
                t0 += g.n;
            }
        };
    };
    auto softmax = [&](int s) {
        return [&, s](int me) {
            int done = 0;
            for (const Item &g : items) {
                const int n = g.both ? g.n : (g.n + 1 - s) >> 1;
                if (n) b.q_full[s].arrive();
                for (int i = 0; i < n; ++i, ++done) {
                    if (!wait(me, b.s_full[s], done)) return;
                    b.p_half[s].arrive();
                    if (!sim.yield(me, [] { return true; })) return;
                    b.p_full[s].arrive();
                }
                if (n) {
                    if (!wait(me, b.pv_done[s], done - 1)) return;
                }
            }
        };
    };
    sim.run({copier, issuer(0), issuer(1), softmax(0), softmax(1)}, lazy);
    if (!b.fault && sim.dead) b.bad("a wait never ends");
    return b.fault;
}

}  // namespace

// stages, seeds, then items as n or -n (both slots): prints the first fault, or "ok".  Several lists: separated by 0.
int main(int argc, char **argv) {
    if (argc < 4) return 2;
    const int ns = atoi(argv[1]), seeds = atoi(argv[2]);
    std::vector<std::vector<Item>> lists(1);
    for (int i = 3; i < argc; ++i) {
        const int n = atoi(argv[i]);
        if (n)
            lists.back().push_back({abs(n), n < 0});
        else
            lists.emplace_back();
    }
    int faults = 0;
    for (auto &items : lists)
        for (int seed = 0; seed < seeds; ++seed) {
            // events only when nothing else can go on, or now and then, or early
            const int lazy = seed % 3 == 0 ? 100 : seed % 3 == 1 ? 80 : 20;
            const char *f = ns == 4 ? simulate<4>(items, seed, lazy) : ns == 3 ? simulate<3>(items, seed, lazy) : simulate<2>(items, seed, lazy);
            if (!f) continue;
            if (!faults++) {
                printf("%s: seed %d, tiles", f, seed);
                for (auto &g : items) printf(" %d%s", g.n, g.both ? " (both slots)" : "");
                printf("\n");
            }
        }
    printf(faults ? "%d schedules fail\n" : "ok\n", faults);
    return faults != 0;
}
