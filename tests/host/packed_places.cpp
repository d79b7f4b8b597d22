// A packed batch's places as the kernels find them, on the host.  Reads the sequences, the
// rows of q and of k, and both offsets; goes over the sequences in the
// searches' order with the kernels' spans, counts and bounds.  Writes the room for tiles of
// queries, the last one that a sequence would use unbounded and as it is bounded, the least
// count that a place has, and whether a span left the tensors.
#include <cstdio>
#include <vector>

#include "packed.cuh"

int main()
{
    using namespace gbssim;
    int n, q_rows, k_rows;
    if (std::scanf("%d %d %d", &n, &q_rows, &k_rows) != 3) return 1;
    std::vector<int> q(n + 1), k(n + 1);
    for (auto *v : {&q, &k})
        for (int &x : *v)
            if (std::scanf("%d", &x) != 1) return 1;
    const int room = q_rows / kAttnTile + n + 1;
    long long exact = 0, loose = 0, tight = 0;
    int before = 0, least = 0, left = 0;
    for (int s = 0; s <= n; ++s) {
        int first, queries, k_first, keys;
        packed_span(q.data(), n, q_rows, s, first, queries);
        packed_span(k.data(), n, k_rows, s, k_first, keys);
        left |= first < 0 || queries < 0 || first + (long long)queries > q_rows || k_first < 0 || keys < 0 ||
                k_first + (long long)keys > k_rows;
        const int tiles = (queries + kAttnTile - 1) / kAttnTile;
        const int some = tiles_within(room, before, tiles);
        const long long end = some ? before + (long long)some : 0;
        if (exact + tiles > loose) loose = exact + tiles;
        if (end > tight) tight = end;
        if (before < least || some < least) least = before < some ? before : some;
        exact += tiles;
        if (exact <= room && (before != exact - tiles || some != tiles)) left |= 2;
        before = add_tiles(before, tiles);
    }
    std::printf("%d %lld %lld %d %d\n", room, loose, tight, least, left);
}
