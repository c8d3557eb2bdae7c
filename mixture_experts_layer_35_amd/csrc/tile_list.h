// tile_list.h -- the tiles of a product grouped by expert, found on the device from the experts' row offsets (gfx950, wave64).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "parts.h"

namespace moe {
namespace {

// The list of tiles: experts in order, an expert's feature tiles, a feature tile's row blocks.  Every
// wave works with it by itself: lane l adds up the tiles of experts l*P .. l*P + P-1.  The experts' ends
// (offsets[1] on) lie in LDS, so that looking a tile up does not wait for the loads under way.
struct TileList {
    const int32_t *ends;
    int P, bm, ftiles;
    int base, count;             // this lane's first tile and tiles
    int total;
    __device__ void init(const int32_t *o, int n, int bm_, int ftiles_, int lane) {
        ends = o;
        bm = bm_;
        ftiles = ftiles_;
        P = (n + 63) / 64;
        count = 0;
        for (int e = lane * P; e < min(n, lane * P + P); ++e) count += blocks(e) * ftiles;
        int run = count;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int up = __shfl_up(run, m, 64);
            if (lane >= m) run += up;
        }
        base = run - count;
        total = __builtin_amdgcn_readlane(run, 63);
    }
    __device__ int start(int e) const { return e ? ends[e - 1] : 0; }
    __device__ int blocks(int e) const { return parts_of(ends[e] - start(e), bm); }
    // Tile t < total (the same in all lanes): expert, feature tile, first row and number of rows.  An expert's
    // token blocks of `unit` rows are split evenly over its row blocks, so that at most one is part empty.
    __device__ void find(int t, int lane, int &e, int &ft, int &row0, int &valid) const {
        const uint64_t started = __ballot(count > 0 && base <= t);
        const int owner = 63 - __builtin_clzll(started);
        int le = 0, rest = t - base;
        if (lane == owner) {
            le = lane * P;
            for (int k = blocks(le) * ftiles; rest >= k; k = blocks(le) * ftiles) {
                rest -= k;
                ++le;
            }
        }
        e = __builtin_amdgcn_readlane(le, owner);
        rest = __builtin_amdgcn_readlane(rest, owner);
        const int first = __builtin_amdgcn_readfirstlane(start(e));
        const int m = __builtin_amdgcn_readfirstlane(ends[e]) - first;
        const int mt = parts_of(m, bm);
        // quotients are vector instructions: back to scalars, which the descriptors have to be
        ft = __builtin_amdgcn_readfirstlane(rest / mt);
        const int unit = min(bm, 32), units = parts_of(m, unit);
        const int block = rest - ft * mt, uq = __builtin_amdgcn_readfirstlane(units / mt), ur = units - uq * mt;
        const int r = (block * uq + min(block, ur)) * unit;
        row0 = first + r;
        valid = min((uq + (block < ur ? 1 : 0)) * unit, m - r);
    }
};

// A value of a kernel's read-only arrays at an address that all lanes share, by a scalar load: it does not wait behind the
// vector loads under way.
__device__ __forceinline__ int scalar_load(const int32_t *p, int64_t i) {
    typedef const __attribute__((address_space(4))) int32_t constant_int;
    return ((constant_int *)(uintptr_t)p)[i];
}

}  // namespace
}  // namespace moe
