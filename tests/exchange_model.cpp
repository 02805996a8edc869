// The turns of a cluster's exchange, as kda_exchange.cuh tells them, on threads: CTAs that stall at random,
// so that waits of the others give up, messages that come late and in any order, and barriers that keep the
// rules of the GPU's.  Prints what went wrong, and how many CTAs were lost.
//   exchange_model K turns seeds wait_rounds
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <random>
#include <thread>
#include <vector>

#include "kda_exchange.cuh"

namespace {

constexpr int kMost = (1 << 20) / 512;   // messages that a barrier can count

struct Barrier {            // one arrival a phase, and as many messages as it said
    int pending = 1, messages = 0, phase = 0;
};
struct Message {
    int from, to, turn;
    bool late;              // comes when no other is on its way
};
struct World {
    int K, turns, wait_rounds;
    std::mutex lock;
    std::condition_variable all;
    int here = 0, generation = 0;
    std::vector<Barrier> bars;                 // [cta][2]
    std::vector<int> holds;                    // [cta][2][r] turn of the message there
    std::vector<bool> ended;
    std::vector<Message> flying;
    long long wrong = 0, mixed = 0, lost = 0;
    bool gave_up = false;                      // a wait, of any CTA

    void fault(const char* what) {
        if (wrong++ < 5) std::printf("%s\n", what);
    }
    void complete(Barrier& b) {
        if (b.pending == 0 && b.messages == 0) {
            ++b.phase;
            b.pending = 1;
        }
    }
    void land(size_t i) {
        const Message m = flying[i];
        flying[i] = flying.back();
        flying.pop_back();
        if (ended[m.to]) return fault("a message came to a CTA that had ended");
        holds[(m.to * 2 + m.turn % 2) * K + m.from] = m.turn;
        Barrier& b = bars[m.to * 2 + m.turn % 2];
        --b.messages;
        if (b.messages <= -kMost || b.messages >= kMost) fault("a barrier's count out of range");
        complete(b);
    }
    void sync() {
        std::unique_lock<std::mutex> hold(lock);
        const int g = generation;
        if (++here == K) {
            here = 0;
            ++generation;
            all.notify_all();
        } else {
            all.wait(hold, [&] { return generation != g; });
        }
    }
};
struct Port {
    World& w;
    int rank;
    std::mt19937& gen;
    bool late = false, last_wait = false;

    void send(int turn) {
        for (int r = 0; r < w.K; ++r) {
            std::lock_guard<std::mutex> hold(w.lock);
            w.flying.push_back({rank, r, turn, late && gen() % 16 == 0});
        }
    }
    bool wait(int turn) {
        for (int i = 0; i < (last_wait ? 1 << 30 : w.wait_rounds); ++i) {
            {
                std::lock_guard<std::mutex> hold(w.lock);
                if (w.bars[rank * 2 + turn % 2].phase > turn / 2) return true;
            }
            std::this_thread::yield();
        }
        return false;
    }
    void arrive(int turn) {
        std::lock_guard<std::mutex> hold(w.lock);
        Barrier& b = w.bars[rank * 2 + turn % 2];
        if (b.pending != 1) w.fault("an arrival that its phase does not expect");
        b.pending = 0;
        w.complete(b);
    }
    void pause() { w.fault("too few turns for a pause"); }
    void expect(int turn, int n) {
        std::lock_guard<std::mutex> hold(w.lock);
        Barrier& b = w.bars[rank * 2 + turn % 2];
        b.messages += n * w.K;
        if (b.messages >= kMost) w.fault("a barrier's count out of range");
        w.complete(b);
    }
    void arm(int turn) {   // both at once
        std::lock_guard<std::mutex> hold(w.lock);
        Barrier& b = w.bars[rank * 2 + turn % 2];
        if (b.pending != 1 || b.phase != turn / 2) w.fault("an arrival that its phase does not expect");
        b.messages += w.K;
        b.pending = 0;
        w.complete(b);
    }
};

void cta(World& w, int rank, unsigned seed) {
    std::mt19937 gen(seed * 31 + rank);
    Port port{w, rank, gen};
    for (int t = 0; t < 2; ++t) port.arm(t);
    w.sync();
    port.late = gen() % 3 == 0;
    const int stall = gen() % 3 ? -1 : (int)(gen() % w.turns);
    int lost = -1;
    for (int t = 0; t < w.turns; ++t) {
        if (t == stall) {
            std::this_thread::sleep_for(std::chrono::milliseconds(gen() % 4));
            // (on a busy machine the others' waits may take longer than that)
            for (int i = 0; i < 10000 && w.wait_rounds < 1 << 30 && w.K > 1; ++i) {
                std::this_thread::sleep_for(std::chrono::microseconds(100));
                std::lock_guard<std::mutex> hold(w.lock);
                if (w.gave_up) break;
            }
        }
        port.send(t);
        if (lost < 0 && !port.wait(t)) {
            lost = t;
            std::lock_guard<std::mutex> hold(w.lock);
            w.gave_up = true;
        }
        if (lost >= 0) continue;
        port.arm(t + 2);
        if (gen() % 4 == 0) std::this_thread::yield();
        std::lock_guard<std::mutex> hold(w.lock);   // all messages of the turn, none of a later one
        for (int r = 0; r < w.K; ++r) w.mixed += w.holds[(rank * 2 + t % 2) * w.K + r] != t;
    }
    w.sync();
    port.last_wait = true;
    if (lost >= 0) kda::exchange_drain(port, w.K, w.turns, lost);
    std::lock_guard<std::mutex> hold(w.lock);
    w.ended[rank] = true;
    w.lost += lost >= 0;
}

}  // namespace

int main(int argc, char** argv) {
    if (argc != 5) return 2;
    const int K = std::atoi(argv[1]), turns = std::atoi(argv[2]), seeds = std::atoi(argv[3]);
    long long wrong = 0, lost = 0;
    for (int seed = 0; seed < seeds; ++seed) {
        World w;
        w.K = K, w.turns = turns, w.wait_rounds = std::atoi(argv[4]);
        w.bars.resize(K * 2);
        w.holds.assign(K * 2 * K, -1);
        w.ended.assign(K, false);
        std::vector<std::thread> ctas;
        for (int r = 0; r < K; ++r) ctas.emplace_back(cta, std::ref(w), r, seed);
        std::mt19937 gen(seed);
        for (bool done = false; !done;) {   // the network
            bool idle = true;
            {
                std::lock_guard<std::mutex> hold(w.lock);
                std::vector<size_t> next;
                for (size_t i = 0; i < w.flying.size(); ++i)
                    if (!w.flying[i].late) next.push_back(i);
                if (!next.empty()) idle = false;
                if (next.empty() && !w.flying.empty() && gen() % 8 == 0) next.push_back(gen() % w.flying.size());
                if (!next.empty()) w.land(next[gen() % next.size()]);
                done = w.flying.empty();
                for (bool e : w.ended) done = done && e;
            }
            if (idle) std::this_thread::sleep_for(std::chrono::microseconds(200));
        }
        for (auto& c : ctas) c.join();
        if (w.mixed && !w.lost) w.fault("a message of another turn, and no CTA was lost");
        wrong += w.wrong;
        lost += w.lost;
    }
    std::printf("wrong %lld lost %lld\n", wrong, lost);
    return wrong != 0;
}
