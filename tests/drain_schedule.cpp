// CPU model of a product's stage barriers, driven by the schedule the kernel follows
// when it winds down (ebin_gemm_drain.h).  See test_drain_schedule.py.
#include <cstdint>
#include <vector>

#include "ebin_gemm_drain.h"

namespace {

struct Rng {
    uint64_t s;
    uint32_t next() {
        s = s * 6364136223846793005ull + 1442695040888963407ull;
        return (uint32_t)(s >> 33);
    }
    int below(int n) { return (int)(next() % (uint32_t)n); }
};

// A barrier of one arrival: its phase ends when the arrival is in and the bytes are level.
struct Bar {
    int phase = 0, pending = 1;
    long tx = 0;
    void settle() {
        if (pending == 0 && tx == 0) {
            ++phase;
            pending = 1;
        }
    }
    void arrive_expect(long bytes) {
        tx += bytes;
        --pending;
        settle();
    }
    void complete(long bytes) {
        tx -= bytes;
        settle();
    }
    // a parity wait for the phase of index i, of which only i and i + 1 can be met
    bool over(int i) const { return ((i & 1) ^ (phase & 1)) != 0; }
};

struct Copy {
    int step;
    bool landed;
};

struct Model {
    int stages, ctas;
    long bytes;
    std::vector<Bar> full;
    std::vector<Copy> fly;
    int issued[2] = {0, 0}, consumed = 0;

    Model(int stages, int ctas, long bytes) : stages(stages), ctas(ctas), bytes(bytes), full(stages) {}

    void land_some(Rng &r, int chance) {
        for (Copy &c : fly)
            if (!c.landed && r.below(100) < chance) {
                c.landed = true;
                full[c.step % stages].complete(bytes);
            }
    }
    bool may_issue(int cta) const { return issued[cta] < consumed + stages; }
    void issue(int cta) {
        const int j = issued[cta]++;
        if (cta == 0) full[j % stages].arrive_expect(ctas * bytes);
        fly.push_back({j, false});
    }
    bool step_over(int j) const { return full[j % stages].over(j / stages); }
    bool consume() {
        if (consumed >= issued[0] || !step_over(consumed)) return false;
        ++consumed;
        return true;
    }
    int open() const {
        int n = 0;
        for (const Copy &c : fly) n += !c.landed;
        return n;
    }
};

}  // namespace

// Random walks that stop at a random point; then the drain, with copies landing meanwhile.
// rule 0: the schedule; 1: no drain unless warp 0's own wait ran out (none is open then);
// 2: plain waits for the leader's own steps.  Returns walks that left a copy open, or in
// which a wait would never have ended though every copy landed (counted in *stuck).
extern "C" int drain_check(uint64_t seed, int walks, int ctas, int rule, int *stuck, int *uneven) {
    Rng r{seed * 2654435761u + 1};
    int left = 0;
    *stuck = *uneven = 0;
    for (int w = 0; w < walks; ++w) {
        Model m(1 + r.below(12), ctas, 16 + 16 * r.below(8));
        const int steps = 1 + r.below(40), events = r.below(400);
        bool stopped[2] = {false, ctas == 1}, dead = false;
        for (int e = 0; e < events; ++e) {
            const int what = r.below(8);
            if (what < 4) {
                const int cta = ctas == 2 ? what & 1 : 0;
                if (!stopped[cta] && m.issued[cta] < steps && m.may_issue(cta)) m.issue(cta);
            } else if (what == 4) {
                m.land_some(r, 40);
            } else if (what < 7) {
                if (!dead) m.consume();
            } else if (r.below(30) == 0) {
                const int who = r.below(3);   // a wait ran out
                if (who == 2) dead = true;
                else stopped[who % ctas] = true;
            }
        }
        const int own = m.issued[0], peer = ctas == 2 ? m.issued[1] : own;
        *uneven += own != peer;
        bool hung = false;
        auto wait = [&](int j) {
            for (int i = 0; i < 64 && !m.step_over(j); ++i) m.land_some(r, 50);
            if (!m.step_over(j)) {
                m.land_some(r, 100);
                hung |= !m.step_over(j);
            }
        };
        if (rule == 0) {
            const int end = ebin::tc_drain_end(own, peer);
            for (int j = ebin::tc_drain_first(own, peer, m.stages); j < end; ++j) {
                const ebin::TcDrain todo = ebin::tc_drain_step(j, own, peer);
                if (todo == ebin::TC_DRAIN_EXPECT) m.full[j % m.stages].arrive_expect(m.bytes);
                if (todo == ebin::TC_DRAIN_COUNT_OFF) m.full[j % m.stages].complete(m.bytes);
                wait(j);
            }
        } else if (rule == 2) {
            for (int j = own > m.stages ? own - m.stages : 0; j < own; ++j) wait(j);
        }
        left += m.open() > 0;
        *stuck += hung;
    }
    return left;
}
