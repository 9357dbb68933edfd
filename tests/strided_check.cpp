// ks_strided.h against counting bytes, on small random tensors: none that share a byte come out apart;
// those of equal steps and axes that nest come out as they are. Prints how many of each it saw.
#include <cstdio>
#include <random>
#include <vector>

#include "ks_strided.h"

using ks::Strided;

static std::vector<int64_t> bytes(const Strided &v, int64_t base) {
    std::vector<int64_t> b;
    for (int64_t i = 0; i < v.count[0]; ++i)
        for (int64_t j = 0; j < v.count[1]; ++j)
            for (int64_t k = 0; k < v.count[2]; ++k)
                for (int64_t r = 0; r < v.run; ++r)
                    b.push_back(base + i * v.stride[0] + j * v.stride[1] + k * v.stride[2] + r);
    return b;
}

int main() {
    std::mt19937 rng(1);
    auto pick = [&](int lo, int hi) { return (int64_t)(lo + rng() % (unsigned)(hi - lo + 1)); };
    static char memory[1 << 16];
    long shared = 0, apart = 0, alternating = 0, wrong = 0;
    for (int trial = 0; trial < 400000; ++trial) {
        Strided x, y;
        const bool alike = trial % 4 != 0;
        x.run = pick(1, 4);
        y.run = alike && pick(0, 1) ? x.run : pick(1, 4);
        int axes[3] = {0, 1, 2};
        for (int i = 2; i > 0; --i) std::swap(axes[i], axes[pick(0, i)]);
        int64_t inner = 2 * (x.run > y.run ? x.run : y.run);  // axes that nest, with room for both
        for (int k : axes) {
            x.count[k] = pick(1, 4);
            y.count[k] = pick(0, 2) ? x.count[k] : pick(1, 4);
            x.stride[k] = inner + pick(0, 3) * pick(0, 2);
            y.stride[k] = alike ? x.stride[k] : pick(0, 12);
            if (alike && pick(0, 15) == 0) x.stride[k] = 0;  // broadcast
            const int64_t most = x.count[k] > y.count[k] ? x.count[k] : y.count[k];
            inner = (alike ? y.stride[k] : inner) * (most - 1) + inner;
        }
        const int64_t at = pick(0, 60) - 30;
        x.p = memory + 20000;
        y.p = memory + 20000 + at;
        std::vector<char> hit(60000, 0);
        for (int64_t b : bytes(x, 20000)) hit[b] = 1;
        bool truth = false;
        for (int64_t b : bytes(y, 20000 + at)) truth |= hit[b] != 0;
        const bool said = ks::strided_cross(x, y);
        if (said != ks::strided_cross(y, x)) ++wrong;
        if (truth && !said) ++wrong;
        if (alike && said != truth) ++wrong;
        if (alike && !truth && at >= 0 && at < ks::strided_span(x, ks::StridedOrder(x, y))) ++alternating;
        ++(truth ? shared : apart);
        // a tensor's own runs
        std::vector<char> seen(60000, 0);
        bool twice = false;
        for (int64_t b : bytes(x, 20000)) {
            twice |= seen[b] != 0;
            seen[b] = 1;
        }
        bool zero = false;
        for (int k = 0; k < 3; ++k) zero |= x.stride[k] == 0 && x.count[k] > 1;
        if (alike ? ks::strided_rows_apart(x) == twice && !zero : ks::strided_rows_apart(x) && twice) ++wrong;
        if (zero && ks::strided_rows_apart(x)) ++wrong;
    }
    std::printf("%ld shared, %ld apart, %ld of them alternating, %ld wrong\n", shared, apart, alternating, wrong);
    return wrong == 0 && shared > 10000 && alternating > 10000 ? 0 : 1;
}
