// s4::delta::last_parity on the host, against a model of the barrier that a
// stage's copies complete: the wait for it lasts as long as the last copy does.
#include <cstdio>

#include "delta.cuh"

struct Barrier {
    int phase = 0;   // completed ones
    bool done(int parity) const { return (phase & 1) != parity; }   // of the phase with that parity, as mbarrier.try_wait
};

int main() {
    int bad = 0;
    for (int stages = 1; stages <= 3; ++stages)
        for (int count = 0; count <= 12; ++count) {
            int copies[3] = {}, seen = 0;
            for (int n = 0; n < count; ++n) ++copies[n % stages];
            for (int i = 0; i < stages; ++i) {
                const int parity = s4::delta::last_parity(count, stages, i);
                seen += copies[i];
                if (copies[i] == 0) {
                    bad |= parity != -1;
                    continue;
                }
                Barrier b;
                b.phase = copies[i] - 1;   // all but the last one have arrived
                const bool early = b.done(parity);
                ++b.phase;
                if (early || !b.done(parity)) {
                    std::printf("%d copies, %d stages: stage %d's last is %s\n", count, stages, i, early ? "not waited for" : "missed");
                    bad = 1;
                }
            }
            bad |= seen != count;
        }
    return bad;
}
