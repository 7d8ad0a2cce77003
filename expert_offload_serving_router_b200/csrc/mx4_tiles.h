// How the MXFP4 product cuts its groups into row tiles (plain integer code, also compiled for the host by its test).
//
// A group of n rows takes ceil(n / BN) tiles of nearly equal size, a multiple of 16 rows each but the last:
// per <= BN, and all tiles but the last fill (tiles - 1) * per < n.  Counts are unsigned on the way: n is an
// int32, and n + BN - 1 or n + tiles - 1 is not once a group passes some 2^31 * 32 / 33 rows.
#pragma once
#include <stdint.h>
#ifndef __CUDACC__
#define __host__
#define __device__
#define __forceinline__ inline
#endif

namespace ftmoe {

struct PxTile { int g, m, row0, nvalid; };

template <int BN>
__host__ __device__ __forceinline__ int px_row_tiles(int n) { return int((uint32_t(n) + BN - 1) / BN); }

// tile t -> group, 128-row weight tile m (fastest, so CTAs that share rows of `a` run together), rows.
// ntile: first row tile of each group, off: its first row, [G + 1] each.
template <int BN>
__host__ __device__ __forceinline__ PxTile px_tile(int t, const int* ntile, const int* off, int G, int m_tiles) {
    PxTile r;
    const int u = t / m_tiles;
    r.m = t - u * m_tiles;
    int lo = 0, hi = G;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ntile[mid] <= u) lo = mid; else hi = mid;
    }
    r.g = lo;
    const int n = off[lo + 1] - off[lo], nt = ntile[lo + 1] - ntile[lo];
    const int per = int(((uint32_t(n) + uint32_t(nt) - 1) / uint32_t(nt) + 15) & ~15u);
    const int i = u - ntile[lo];
    r.row0 = off[lo] + i * per;
    r.nvalid = per < n - i * per ? per : n - i * per;
    return r;
}

}  // namespace ftmoe
