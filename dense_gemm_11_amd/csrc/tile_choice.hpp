// What the calls over ragged rows share on the host: the sizes they take and the
// choice of a tile.
#pragma once

#include <algorithm>
#include <climits>

#include "handle.hpp"
#include "ragged_variants.hpp"

namespace dg {

constexpr int MAX_GROUPS = 1 << 16;

// The kernels form row, column and step numbers in 32 bits up to a tile or a
// batch of steps past the end (a last tile of 192 rows would pass 2^31 from M =
// 2^31 - 128), and twice the padded rank.
constexpr int64_t MAX_EXTENT = INT_MAX - 512;

// Byte offsets inside a panel of `rows` rows of `ld` elements and `cols` more
// stay below 2^32.
inline bool panel_fits(int64_t rows, int64_t ld, int64_t cols, int64_t es)
{
    return (rows * ld + cols) * es < ((int64_t)1 << 32) - 64;
}

// A launch has fewer than 2^32 threads along its first axis.
inline bool grid_fits(int64_t grid, int threads) { return grid * threads < (int64_t)1 << 32; }

// C against D: the same matrix with the same strides, or disjoint.
inline bool c_d_ok(const void* C, int64_t span_c, const void* D, int64_t span_d, bool same_strides)
{
    return C == D ? same_strides : !ranges_overlap(C, span_c, D, span_d);
}

// A call's tiles, tallest first: the direct-to-LDS ones, then the streaming
// ones.
template <class Tile>
struct TileList {
    const Tile* dma;
    const Tile* stream;
    int n_dma, n;
    const Tile& operator[](int i) const { return i < n_dma ? dma[i] : stream[i - n_dma]; }
};
template <class Tile>
TileList<Tile> tile_list(const Tile* (*dma)(int*), const Tile* (*stream)(int*))
{
    TileList<Tile> l{};
    int n_stream = 0;
    l.dma = dma(&l.n_dma);
    l.stream = stream(&n_stream);
    l.n = l.n_dma + n_stream;
    return l;
}

// Number of tile i among those of its height.
template <class Tile>
int nth_of_height(const TileList<Tile>& t, int i)
{
    int n = 0;
    for (int j = 0; j < i; ++j) n += t[j].bm == t[i].bm;
    return n;
}

// The forced tile (gemm_set_group_tile_nth), else the one of least expected
// time among those whose grid fits; tiles(t) is the number of output tiles of t a
// call has, or expects, grid(t) its workgroups, and `bytes` what it reads and
// writes at the least.
template <class Tile, class F, class G>
const Tile& pick_tile(gemm_handle_t h, const TileList<Tile>& t, bool b_kc, int64_t K, double bytes, F tiles,
                      G grid)
{
    int best = t.n - 1;
    if (h->forced_rows > 0) {
        int height = t[best].bm;
        for (int i = 0; i < t.n; ++i)
            if (t[i].bm <= h->forced_rows && t[i].bm > height) height = t[i].bm;
        for (int i = 0; i < t.n; ++i)
            if (t[i].bm == height) {
                best = i;
                if (nth_of_height(t, i) == h->forced_nth) break;
            }
        return t[best];
    }
    double best_us = 0.0;
    const int cus = device_cus();
    for (int i = 0; i < t.n; ++i) {
        if (!grid_fits(grid(t[i]), t[i].threads)) continue;
        const double us = expected_us(t[i], b_kc, (double)tiles(t[i]), (double)K, bytes, cus);
        if (best_us == 0.0 || us < best_us) {
            best = i;
            best_us = us;
        }
    }
    return t[best];
}

// Rows of tiles of height bm in `busy` groups of avg rows on average: the last
// tile of a group is half full.
inline double row_tiles(double busy, double avg, int bm)
{
    return busy * std::max(1.0, avg / bm + 0.5);
}

}  // namespace dg
