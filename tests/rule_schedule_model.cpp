// Walks the requests of the rule's scans (tree_masked_gated_amd/csrc/rule_schedule.hpp) as the kernels do, for
// sequences of given lengths, and prints every row of a sequence that is requested and is not one of its rows.
//
//   model forward|back LENGTH...
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "rule_schedule.hpp"

namespace {

struct Lanes {                               // the rows that a workgroup's lanes keep
    int n, off[gdn::kC], faults = 0, requests = 0;
    explicit Lanes(int n_) : n(n_) {
        for (int i = 0; i < gdn::kC; ++i) off[i] = i;
    }
    void places(int rows) {
        for (int i = 0; i < gdn::kC; ++i) off[i] = gdn::row_in(i, rows);
    }
    void load(int c) {
        ++requests;
        for (int i = 0; i < gdn::kC; ++i) {
            const int row = c * gdn::kC + off[i];
            if (row >= 0 && row < n) continue;
            if (!faults++) printf("%d rows: row %d requested with chunk %d\n", n, row, c);
        }
    }
};

}  // namespace

int main(int argc, char** argv) {
    int faults = 0;
    for (int a = 2; a < argc; ++a) {
        const int n = atoi(argv[a]), chunks = gdn::chunks_of(n);
        Lanes x(n);
        auto places = [&](int rows) { x.places(rows); };
        auto load = [&](int c) { x.load(c); };
        if (chunks > 0 && !strcmp(argv[1], "forward")) {
            gdn::request_forward(n, 0, places, load);
            for (int c = 0; c < chunks; ++c) gdn::request_forward(n, gdn::after(n, c), places, load);
        } else if (chunks > 0) {
            gdn::request_back_first(n, places, load);
            for (int c = chunks - 1; c >= 0; --c) load(gdn::before(c));
        }
        if (x.requests != (chunks ? chunks + 1 : 0)) printf("%d rows: %d requests\n", n, x.requests), ++faults;
        faults += x.faults;
    }
    printf("%d lengths, %d faults\n", argc - 2, faults);
    return faults != 0;
}
