// The rows and tiles of a packed batch's sequences; on the host too, where tests hold
// them to the tensors' bounds.
#pragma once

#include <algorithm>
#include <cuda_runtime.h>

namespace gbssim {

// Tiles of 128 rows, the lanes of tensor memory.
constexpr int kAttnTile = 128;

// Offsets that do not ascend or leave the tensors are brought into range, so that
// no row outside them is read or written whatever they hold.  Behind the last
// sequence comes one more, of the rows that are left and without a partner: its
// outputs are zeros.
__host__ __device__ inline void packed_span(const int *offsets, int sequences, int rows, int s, int &first, int &count)
{
#ifdef __CUDA_ARCH__
    const auto at = [&](int i) { return __ldg(offsets + i); };
#else
    const auto at = [&](int i) { return offsets[i]; };
#endif
    first = s == 0 ? 0 : std::min(std::max(at(s), 0), rows);
    const int end = s >= sequences ? rows : std::min(std::max(at(s + 1), first), rows);
    count = end - first;
}

// Sequences whose offsets do not ascend may share rows, and then have more tiles together
// than there is room for in the row sums, or in an int.  Counts stop far above what
// ascending ones come to (2^22 tiles of 128 rows, 2^29 sequences), ...
constexpr int kMostTiles = (1 << 30) - 1;

__host__ __device__ inline int add_tiles(int a, int b) { return a + b < kMostTiles ? a + b : kMostTiles; }

// ... and of a sequence's tiles of queries those count that there is room for, `room` in
// all, behind the ones before it.
__host__ __device__ inline int tiles_within(int room, int before, int tiles)
{
    const int left = room - before;
    return left < 0 ? 0 : left < tiles ? left : tiles;
}

}  // namespace gbssim
