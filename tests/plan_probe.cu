// Host-only probe for tests/test_kv_plan_host.py: for small tables, every length (beyond the table too), number of rows
// and entry of a plan, the columns that a sequence counts as shared, one line of numbers each.
#include <algorithm>
#include <cstdio>

#include "kv_attention.cuh"

int main() {
    for (int log2p = 4; log2p <= 5; ++log2p) {
        const int page = 1 << log2p;
        for (int width = 1; width <= 4; ++width) {
            const int most = width * page;
            for (int held = -1; held <= 3 * most; held += held % page == page - 1 || held % page == 0 ? 1 : page / 2 - 1)
                for (int n : {0, 1, 2, page, page + 1, 3 * most})
                    for (int skip = -page; skip <= 3 * most; skip += page / 2) {
                        const int len = std::min(std::max(held, 0), most);  // as the kernels cut it
                        std::printf("%d %d %d %d %d %d\n", log2p, width, held, n, skip, qg::columns_shared(skip, n, len, log2p));
                    }
        }
    }
}
