// Tiles of a product's output and the order in which a launch takes them, shared by the products of the expert layers.
//
// A launch's arguments P have mode (MUON_PRODUCT_*), m, n, k, groups, offsets and, from count_tiles, tiles_m, tiles_n, tiles.
// The depth k counts in units of UNIT values.  With PAIR = 2 a launch makes two products of one shape, each group's one
// after the other.
#pragma once

#include <cstdint>

#include "device_common.h"
#include "muon.h"

namespace muon {
namespace tiles {

constexpr int NUM_XCD = 8, CUS = 256;

// Bands of BAND tile rows, each walked column by column: the tiles an XCD runs at once share panels.
constexpr int BAND = 8;
__device__ __forceinline__ void band_decode(int t, int tm, int tn, int& ti, int& tj) {
    const int band = t / (BAND * tn);
    const int r0 = band * BAND;
    const int rows = min(BAND, tm - r0);
    const int w = t - band * BAND * tn;
    tj = w / rows;
    ti = r0 + (w - tj * rows);
}

__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
    const uint64_t v = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (const uint8_t*)(((uint64_t)hi << 32) | lo);
}

struct Tile {
    int64_t m0, n0;            // first row of a, of b
    int rows_a, rows_b;        // rows of either inside the tile
    int group, kb0, kb1;       // units of k [kb0, kb1)
    int which;                 // of the pair's two products
};

// Whether a depth-grouped launch deals every group's tiles to all XCDs (see Walk): where that leaves an XCD 8 of them,
// which share operand panels, and workgroups have several tiles.
template <class P>
__device__ __forceinline__ bool in_parts(const P& p) {
    return p.mode == MUON_PRODUCT_DEPTH && p.tiles_m * p.tiles_n >= 8 * NUM_XCD && p.tiles > (int)gridDim.x;
}

// The segments' bounds, clamped to the operand, and in ends how many tile rows lie before each segment (rows-grouped),
// or the groups in the order of falling depth (depth-grouped), into LDS, by the whole workgroup.
constexpr int SORT_MAX_GROUPS = 256;      // each thread compares with every group; many groups even out by themselves
template <int UNIT, int THREADS, class P>
__device__ __forceinline__ void read_segments(const P& p, int tile_rows, int* bounds, int* ends, int64_t* wave_tot) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t limit = p.mode == MUON_PRODUCT_ROWS ? p.m : (p.k + UNIT - 1) / UNIT * UNIT;
    for (int g = tid; g <= p.groups; g += THREADS) bounds[g] = (int)min(max((int64_t)p.offsets[g], (int64_t)0), limit);
    if (tid == 0 && p.mode == MUON_PRODUCT_ROWS) ends[0] = 0;
    __syncthreads();
    if (p.mode != MUON_PRODUCT_ROWS) {
        auto depth = [&](int g) { return bounds[g + 1] / UNIT - bounds[g] / UNIT; };
        for (int g = tid; g < p.groups; g += THREADS) {
            int before = g;
            if (in_parts(p) && p.groups <= SORT_MAX_GROUPS) {
                before = 0;
                const int mine = depth(g);
                for (int h = 0; h < p.groups; ++h) {
                    const int other = depth(h);
                    before += other > mine || (other == mine && h < g);
                }
            }
            ends[before] = g;
        }
        __syncthreads();
        return;
    }
    // sums in 64 bits and capped: falling offsets, which are not allowed, must not lead outside the operand either
    int64_t before = 0;
    for (int g0 = 0; g0 < p.groups; g0 += THREADS) {
        const int g = g0 + tid;
        int64_t inc = g < p.groups ? ((int64_t)max(bounds[g + 1] - bounds[g], 0) + tile_rows - 1) / tile_rows : 0;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int64_t o = __shfl_up(inc, off, 64);
            if (lane >= off) inc += o;
        }
        if (lane == 63) wave_tot[wave] = inc;
        __syncthreads();
        int64_t total = 0;
        for (int w = 0; w < THREADS / 64; ++w) {
            if (w < wave) inc += wave_tot[w];
            total += wave_tot[w];
        }
        if (g < p.groups) ends[g + 1] = (int)min(before + inc, (int64_t)1 << 30);
        before += total;
        __syncthreads();
    }
}

// Tile t of the launch, of up to tile_rows x tile_cols.
template <int UNIT, int PAIR, class P>
__device__ __forceinline__ Tile decode(const P& p, int t, int tile_rows, int tile_cols, const int* bounds,
                                       const int* ends) {
    auto at = [](const int* v) { return __builtin_amdgcn_readfirstlane(*v); };
    Tile r;
    r.group = r.which = 0;
    r.kb0 = 0;
    r.kb1 = (int)((p.k + UNIT - 1) / UNIT);
    int64_t m1 = p.m;
    int tm, tn;
    if (p.mode == MUON_PRODUCT_ROWS) {
        tm = t / p.tiles_n;
        tn = t - tm * p.tiles_n;
        int lo = 0, hi = p.groups;                         // the last g with ends[g] <= tm
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (at(ends + mid) <= tm) lo = mid;
            else hi = mid;
        }
        r.group = lo;
        r.m0 = at(bounds + lo) + (int64_t)(tm - at(ends + lo)) * tile_rows;
        m1 = at(bounds + lo + 1);
    } else {
        if (p.mode == MUON_PRODUCT_DEPTH) {
            const int per = p.tiles_m * p.tiles_n, nth = t / per;
            t -= nth * per;
            r.group = at(ends + nth / PAIR);
            r.which = nth % PAIR;
            r.kb0 = at(bounds + r.group) / UNIT;
            r.kb1 = max(at(bounds + r.group + 1) / UNIT, r.kb0);
        } else if (PAIR > 1) {
            const int per = p.tiles_m * p.tiles_n;
            r.which = t / per;
            t -= r.which * per;
        }
        band_decode(t, p.tiles_m, p.tiles_n, tm, tn);
        r.m0 = (int64_t)tm * tile_rows;
    }
    r.n0 = (int64_t)tn * tile_cols;
    r.rows_a = (int)min(m1 - r.m0, (int64_t)tile_rows);
    r.rows_b = (int)min(p.n - r.n0, (int64_t)tile_cols);
    return r;
}

// A workgroup's tiles.  Workgroups are dealt to the XCDs in turn.  Each XCD takes a contiguous share of the tiles and its
// workgroups walk it together, so that the tiles that run at once share operand panels in its L2.
//
// Depth-grouped, tiles of different groups take different times.  In parts, each XCD takes an eighth of every group's
// tiles, the deepest group first, and its workgroups walk them to and fro: 8 groups of 1024 x 4096 over 9000 in
// float32 82 us against 104, 64 groups 390 against 406; with one tile in a part the shared panels are lost (128 groups of
// 512 x 1024: 57 us against 42).
struct Walk {
    int pos, last, step, turn; // tile or place in the XCD's share, its end, step; to and fro: a step's other length
    int chunk, chunks;         // tiles of a group in a part, parts of a group; 0 without parts
};
template <int PAIR, class P>
__device__ __forceinline__ Walk walk(const P& p, const int* ends) {
    const int xcd = blockIdx.x % NUM_XCD, nth = blockIdx.x / NUM_XCD, all = gridDim.x / NUM_XCD;
    if (in_parts(p)) {
        const int per = p.tiles_m * p.tiles_n;
        const int chunk = (per + NUM_XCD - 1) / NUM_XCD, chunks = (per + chunk - 1) / chunk;
        const int mine = (p.groups * PAIR * chunks - xcd + NUM_XCD - 1) / NUM_XCD;
        return {nth, mine * chunk, 2 * (all - nth) - 1, 2 * nth + 1, chunk, chunks};
    }
    int total = p.tiles;
    if (p.mode == MUON_PRODUCT_ROWS)
        total = (int)min((int64_t)__builtin_amdgcn_readfirstlane(ends[p.groups]) * p.tiles_n, (int64_t)p.tiles);
    const int share = total / NUM_XCD, rest = total % NUM_XCD;
    const int first = xcd * share + min(xcd, rest);
    return {first + nth, first + share + (xcd < rest ? 1 : 0), all, all, 0, 0};
}
// The tile at the walk's place or the next one that has one, which the walk is put past; -1 at the end.
template <class P>
__device__ __forceinline__ int next_tile(const P& p, Walk& w) {
    while (w.pos < w.last) {
        const int at = w.pos, step = w.step;
        w.pos += step;
        w.step = w.turn;
        w.turn = step;
        if (w.chunk == 0) return at;
        // part q of all groups' parts is the XCD's q / 8-th; the last part of a group may be short
        const int q = at / w.chunk * NUM_XCD + blockIdx.x % NUM_XCD, group = q / w.chunks;
        const int t = (q - group * w.chunks) * w.chunk + at % w.chunk, per = p.tiles_m * p.tiles_n;
        if (t < per) return group * per + t;
    }
    return -1;
}

// Tiles of a launch, at most; -1 for too many.
template <int PAIR, class P>
inline int64_t count_tiles(P& a, int tile_rows, int tile_cols) {
    a.tiles_n = (int32_t)((a.n + tile_cols - 1) / tile_cols);
    a.tiles_m = (int32_t)((a.m + tile_rows - 1) / tile_rows);
    // every segment may end inside a tile, but not more of them than there are rows
    int64_t rows = a.tiles_m;
    if (a.mode == MUON_PRODUCT_ROWS) rows = a.m / tile_rows + (a.m < a.groups ? a.m : (int64_t)a.groups);
    if (a.mode == MUON_PRODUCT_DEPTH) rows *= a.groups;
    rows *= PAIR;
    const int64_t total = rows * a.tiles_n;
    if (total >= ((int64_t)1 << 31) - 2 * CUS) return -1;   // a workgroup's step past its last tile stays an int
    a.tiles = (int32_t)total;
    return total;
}

}  // namespace tiles
}  // namespace muon
