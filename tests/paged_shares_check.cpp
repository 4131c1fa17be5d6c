// Reads "ctas n_pairs units units ..." per line: the units of the pairs in list order. Prints the shares, and the most
// of them that hold units of one pair, by the decode's rule (paged_shares.cuh): share c starts at base c + min(c, more).
#include <cstdio>
#include <iostream>
#include <sstream>
#include <string>
#include <vector>

#include "paged_shares.cuh"

int main() {
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        int ctas, n;
        in >> ctas >> n;
        std::vector<int> units(n);
        int64_t total = 0;
        int longest = 0;
        for (int& u : units) {
            in >> u;
            total += u;
            if (u > longest) longest = u;
        }
        const int shares = duo::share_count(total, longest, ctas);
        const int64_t base = shares ? total / shares : 0, more = shares ? total % shares : 0;
        auto of = [&](int64_t u) {
            const int64_t large = (base + 1) * more;
            return u < large ? u / (base + 1) : more + (u - large) / base;
        };
        int64_t first = 0, most = 0;
        for (int u : units) {
            const int64_t parts = u ? of(first + u - 1) - of(first) + 1 : 0;
            if (parts > most) most = parts;
            first += u;
        }
        std::printf("%d %lld\n", shares, static_cast<long long>(most));
    }
    return 0;
}
