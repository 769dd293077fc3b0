// The rule for clusters that a device has no place for, run by test_cluster_fit_cpu.py.
#include <cstdio>
#include <vector>

#include "cluster_fit.h"

int main() {
    struct {
        int want, most, got;
        std::vector<int> asked;
    } cases[] = {{1, 0, 1, {}}, {8, 0, 8, {}}, {16, 16, 16, {16}}, {16, 15, 8, {16}}, {16, 0, 8, {16}}, {2, 1, 2, {}}};
    int bad = 0;
    for (auto &c : cases) {
        std::vector<int> asked;
        const int got = hm::placeable_cluster(c.want, [&](int n) {
            asked.push_back(n);
            return n <= c.most;
        });
        if (got != c.got || asked != c.asked) std::printf("%d of at most %d: %d\n", c.want, c.most, got), ++bad;
    }
    std::printf("%d failures\n", bad);
    return bad != 0;
}
