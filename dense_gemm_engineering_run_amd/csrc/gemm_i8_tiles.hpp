// gemm_i8_tiles.hpp -- which kernel a product of 8-bit values runs, and the size
// of its grid (host only; no HIP).
#pragma once

#include <initializer_list>

#include "gemm_tiles.hpp"

namespace mg {

// bk counts pairs of 8-bit values.
enum class I8Tile : int {
    Stream16x16, Stream16x32, Stream32x32, Dma32x64, Dma64x64, Dma64x128, Dma128x128, Dma128x256, PingPong,
    OddStream16x16, OddStream32x32, Odd32x32, Odd64x64, Odd128x128, Odd128x256,
    Count
};
constexpr Tile kI8Tiles[] = {
    {"stream 16x16", 16, 16, 0, 1, 1, 16, 4, 8, 512},
    {"stream 16x32", 16, 32, 0, 1, 2, 16, 3, 8, 512},
    {"stream 32x32", 32, 32, 0, 2, 2, 16, 2, 8, 512},
    {"32x64", 32, 64, 128, 1, 4, 16, 3, 0, 256},
    {"64x64", 64, 64, 128, 2, 4, 16, 3, 0, 512},
    {"64x128", 64, 128, 64, 2, 4, 16, 4, 0, 512},
    {"128x128", 128, 128, 64, 2, 4, 16, 4, 0, 512},
    {"128x256", 128, 256, 64, 2, 4, 16, 3, 0, 512},
    {"ping-pong 256x256", 256, 256, 64, 4, 2, 16, 3, 0, 512},
    {"unaligned stream 16x16", 16, 16, 0, 1, 1, 16, 4, 8, 512},
    {"unaligned stream 32x32", 32, 32, 0, 1, 1, 16, 2, 8, 512},
    {"unaligned 32x32", 32, 32, 128, 2, 2, 16, 2, 0, 256},
    {"unaligned 64x64", 64, 64, 64, 2, 4, 16, 2, 0, 512},
    {"unaligned 128x128", 128, 128, 64, 2, 4, 16, 2, 0, 512},
    {"unaligned 128x256", 128, 256, 64, 4, 4, 16, 2, 0, 1024},
};
static_assert(sizeof(kI8Tiles) / sizeof(Tile) == (int)I8Tile::Count, "one entry a tile");
constexpr Tile tile_of(I8Tile t) { return kI8Tiles[(int)t]; }

struct I8Shape {
    bool vec;             // A and B allow 16-byte loads
    int64_t M, N, K;
};

// The smallest tile that makes no more than one for each of the 256 CUs, else
// the largest, or one as narrow as C.  us, bf16 outputs, N = K = 4096 unless given:
//   rows               16x16  16x32  32x32  32x64  64x64  64x128 128x128 128x256 256x256
//      1                 6.0    6.1    6.3    8.9   10.2
//     16                 6.2    6.3    6.5    9.1
//     32                        6.5    7.1    9.3   10.7
//     64                               7.4    9.3   10.8   14.7
//     64  N 8192 K 2048                9.9    7.1    7.9    9.8
//    128                                     10.0   11.1   14.8   20.4
//    256                                     13.8   12.5   15.6   20.7    31.0
//   1000  N 1024 K 2048                       9.2    8.3   10.1   13.8    19.6    27.0
//    512                                            23.7   18.4   22.9    32.0    45.3
//   1024                                                   33.9   25.9    34.4    45.9
//   2048                                                          47.3    39.6    48.0
//   8192  K 1024                                                          56.0    53.4
//   8192                                                                 147.7   125.3
//      1  N 131072      138    109    121    102    114    112     123     128     147
//     64  N 65536 K 2048                       41     37     30      33      30      40
//  65536  N 64 K 2048                          40     38     42      36      46      41
// (The first three stream: the waves share a tile's k.)
// Unaligned, us:              16x16 str. 32x32 str.  32x32   64x64  128x128  128x256
//      1 of 4095 x 4095           7.8      10.1       14.4    26.1    35.4
//     40 of 4095 x 4095          16.6       9.8       14.8    26.3
//    300 of 1023 x 2047          19.5      14.5       10.1    15.2    23.8
//   1500 of 1025 x 4095                               50.7    39.3    37.1     52.4
//   4095 of 2048 x 1028                                       44.8    25.0     23.2
//   2048 of 4096 x 4096                                               65.7     57.6
//   3000 of 4095 x 2047                              156      87.0    53.8     60.2
//   8192 of 4096 x 1024                                               71.4     73.1
//   8192 of 4096 x 4096                                              241.4    215.1
// Two 128x128 tiles share a CU, a 128x256 tile has one for itself: the wide ones
// lose where their last round would be half a round or less of the others, and
// for short K.  Times of 128x256 to 128x128, by how many tiles the last round has
// (2048 columns, 4224 to 16384 rows; bf16 / fp32 outputs):
//   K          up to 128 of 256    160 to 224        256
//    512         1.13-1.15/1.22   .97-.99/1.03-1.06  1.04/1.01
//   1000, 1500   1.12-1.18/1.19   .95-.97/.98-1.03   1.02/1.00
//   2000, 2500   1.09-1.17/1.19   .93-.97/.95-1.00   .94-.98/.97
//   4096         1.04-1.16/1.16   .90-.92/.92-.94    .85-.92/.92
inline I8Tile i8_tile(const I8Shape& s)
{
    auto tiles = [&](int bm, int bn) { return ceil_div(s.M, bm) * ceil_div(s.N, bn); };
    if (!s.vec) {
        if (tiles(16, 16) <= 256) return I8Tile::OddStream16x16;
        if (tiles(32, 32) <= 256) return I8Tile::OddStream32x32;
        if (tiles(32, 32) <= 512) return I8Tile::Odd32x32;
        if (tiles(64, 64) <= 512) return I8Tile::Odd64x64;
        if (tiles(128, 128) <= 256) return I8Tile::Odd128x128;
        const int64_t wide = tiles(128, 256);
        return wide <= 256 || (s.K >= 2048 && (wide - 1) % 256 >= 128) ? I8Tile::Odd128x256 : I8Tile::Odd128x128;
    }
    if (tiles(16, 16) <= 256) return I8Tile::Stream16x16;
    if (tiles(16, 32) <= 256) return I8Tile::Stream16x32;
    if (tiles(32, 32) <= 256) return I8Tile::Stream32x32;
    if (s.M <= 32 || tiles(32, 64) <= 256) return I8Tile::Dma32x64;
    if (tiles(64, 64) <= 256) return I8Tile::Dma64x64;
    if (s.M <= 64 || tiles(64, 128) <= 256) return I8Tile::Dma64x128;
    if (s.N <= 128 || tiles(128, 128) <= 256) return I8Tile::Dma128x128;
    return s.M <= 128 || tiles(128, 256) <= 256 ? I8Tile::Dma128x256 : I8Tile::PingPong;
}

inline int64_t i8_grid(const I8Shape& s, const Tile& t) { return ceil_div(s.M, t.bm) * ceil_div(s.N, t.bn); }

// C's last columns and rows, up to 16 past a multiple of 128, can go to calls of
// their own behind the rest, where that saves the CUs a round of tiles or lets a
// smaller tile do.  Costs in products of one CU, about 4 * 2^20 a us: rounds of
// tiles (an unaligned 128x128 tile shares its CU where there are more than 256),
// and for an edge's call 16 * 2^20 for being one, with its own rounds or, where
// that is more, the bytes that it reads (an edge of a long C reads the long
// operand once more; 1 us is as many).  us, in brackets without the cut: 8193 x
// 4096 x 4096 135 (167); 2049 rows of it 45.4 (49.9); 4100 x 4104 x 2048 55 (68);
// unaligned 2049 x 4096 x 4096 61 (87), 4095 x 2049 x 1028 into fp32 31 (39).  Left
// whole: 65536 x 144 x 2048 87 (51), 130 x 65536 x 2048 67 (50), unaligned 16384 x
// 130 x 4096 60 (43).  Of 328 such sizes the worst is 9 % off its better way.
inline int64_t i8_cost(const I8Shape& s)
{
    const Tile& t = kI8Tiles[(int)i8_tile(s)];
    const int64_t grid = i8_grid(s, t), a_cu = !s.vec && t.bm == 128 && t.bn == 128 && grid > 256 ? 2 : 1;
    return ceil_div(grid, 256 * a_cu) * a_cu * t.bm * t.bn * s.K;
}
inline int64_t i8_edge_cost(const I8Shape& s)
{
    if (s.M == 0 || s.N == 0) return 0;
    const int64_t cost = i8_cost(s), bytes = (s.M + s.N) * s.K;
    return (16 << 20) + (cost > bytes ? cost : bytes);
}
// A launch can have its grid.
inline bool i8_fits(const I8Shape& s)
{
    const Tile& t = kI8Tiles[(int)i8_tile(s)];
    return i8_grid(s, t) <= kMaxGridThreads / t.threads;
}
struct I8Edges {
    int64_t rows, cols;
};
inline I8Edges i8_edges(const I8Shape& s)
{
    const int64_t m = s.M > 128 && s.M % 128 <= 16 ? s.M % 128 : 0, n = s.N > 128 && s.N % 128 <= 16 ? s.N % 128 : 0;
    I8Edges best = {0, 0};
    int64_t least = i8_cost(s);
    for (const I8Edges e : {I8Edges{0, n}, I8Edges{m, 0}, I8Edges{m, n}}) {
        const I8Shape rest = {s.vec, s.M - e.rows, s.N - e.cols, s.K}, rows = {s.vec, e.rows, s.N, s.K},
                      cols = {s.vec, s.M - e.rows, e.cols, s.K};
        if (!i8_fits(rest) || !i8_fits(rows) || !i8_fits(cols)) continue;
        const int64_t cost = i8_cost(rest) + i8_edge_cost(rows) + i8_edge_cost(cols);
        if (cost < least) {
            least = cost;
            best = e;
        }
    }
    return best;
}

// ------------------------------------------------------------ gradients from 8-bit values

// bk: k of a tile; stages: tiles of loads in flight (streaming: a wave's);
// extra: waves that stream, else waves a SIMD that the registers leave room for.
// (The deep 128x128 tile here is one of three: deep_tile.)
enum class GradTile : int {
    Stream32x32, Stream32x64, T64x64, T64x128, T64x128Two, T128x128Deep, T128x128, T256x256, Tall256x128, Wide128x256, Count
};
constexpr Tile kGradTiles[] = {
    {"stream 32x32", 32, 32, 64, 1, 1, 16, 1, 8, 512},
    {"stream 32x64", 32, 64, 32, 1, 1, 16, 2, 8, 512},
    {"64x64", 64, 64, 128, 2, 4, 16, 2, 2, 512},
    {"64x128", 64, 128, 64, 2, 4, 16, 2, 2, 512},
    {"64x128, two a CU", 64, 128, 64, 2, 4, 16, 1, 4, 512},
    {"128x128, deep", 128, 128, 64, 4, 4, 16, 1, 4, 1024},
    {"128x128", 128, 128, 32, 2, 4, 16, 2, 2, 512},
    {"256x256", 256, 256, 32, 4, 2, 16, 1, 2, 512},
    {"256x128", 256, 128, 64, 4, 4, 16, 1, 4, 1024},
    {"128x256", 128, 256, 64, 4, 4, 16, 1, 4, 1024},
};
static_assert(sizeof(kGradTiles) / sizeof(Tile) == (int)GradTile::Count, "one entry a tile");
constexpr Tile tile_of(GradTile t) { return kGradTiles[(int)t]; }
// The deep 128x128 tile of each kind of call.  Sixteen waves of 32x32 convert fast,
// but read 16 fragments of LDS for the products of three terms where eight of 32x64
// read 10.  us, this | as in the table, m-major A (k-major):
//   16-bit C   2048 x 2048, 4096 k - | 77 (- | 78), 2049 x 1028, 4095 k - | 76 (- | 75)
//     (on 4 x 2 waves 78 (87) and 84 (91), on 2 x 4 86 (90) and 90 (93))
//   Q's terms                      93 | 103 (94 | 100),                  94 | 96 (93 | 93)
//   A's terms into fp32           104 | 113,                             96 | 102
constexpr Tile deep_tile(bool wide, bool split_a, bool a_kmajor)
{
    if (!split_a) return {"", 128, 128, 64, 2, 4, 16, 1, 2, 512};
    return !wide || a_kmajor ? kGradTiles[(int)GradTile::T128x128Deep] : Tile{"", 128, 128, 64, 4, 2, 16, 1, 2, 512};
}
// What runs as tile t in a kind of call.
constexpr Tile tile_of(GradTile t, bool wide, bool split_a, bool a_kmajor)
{
    return t == GradTile::T128x128Deep ? deep_tile(wide, split_a, a_kmajor) : tile_of(t);
}
// The kinds of calls that each tile has a kernel for.
constexpr bool has_kernel(GradTile t, bool vec, bool wide, bool split_a, bool a_kmajor)
{
    switch (t) {
    case GradTile::T64x128Two: return split_a && !vec && (wide || a_kmajor);
    case GradTile::T128x128: return wide ? !split_a : vec || !a_kmajor;
    case GradTile::T256x256: return !wide && vec;
    case GradTile::Tall256x128: return wide && !split_a && vec;
    case GradTile::Wide128x256: return split_a && vec;
    default: return true;
    }
}

struct GradShape {
    bool vec;             // A and Q allow 16-byte loads
    bool wide;            // fp32 C: three MFMAs a product (else two)
    bool split_a;         // the terms are A's (else Q's: bf16 into fp32)
    int64_t M, N, K;
    bool a_kmajor;
};

// The smallest tile that makes no more than one for each of the 256 CUs; past that:
//
// 16-bit C: 128x256, where one for each CU does, else 256x256; as narrow as C.  us,
// bf16 into bf16, A m-major (k-major; fp16 is within a few percent):
//   M x N, K              32x32 str.   32x64 str.    64x64        64x128      128x128, deep
//    512 x  256, 1000       7.6          8.6         12.7         14.9
//     32 x 4096, 4096      16.9         19.7         38.2         48.8
//   1024 x  512, 1024      12.9          8.9         13.0         15.3
//   1024 x 1024, 4096      62           34           39           49           82 (2 x 4 waves)
//   2048 x 1024, 4096                                77 (79)      50 (51)      69 (70)
//   2048 x 2048, 4096                               157 (165)     87 (86)      77 (78)
//                          64x128      128x128      128x256      256x256
//   2304 x 1952,   64     10.7          9.3          9.5
//   2304 x 1952,  256     16.4         15.8         15.0
//   2304 x 1952, 2048     72           77           65          105
//   3008 x 2000, 3008     95 (96)     101 (103)      87 (86)    141 (146)
//   4096 x 2048, 1024     47 (46)      39 (42)       36 (36)     52 (54)
//   3300 x 3104, 2048    137          126          132          108
//   4096 x 4096, 2048    166 (165)    145 (151)     128 (127)   110 (115)
//   8192 x 4096, 4096    636 (635)    561 (597)     492 (498)   420 (436)
//  65536 x   64, 2048    101 (99)      87 (93)      144 (145)    -         64x64: 89 (94)
//  65536 x  128, 1024     55 (53)      47 (50)       80 (76)     65 (68)
//     64 x 65536, 2048    52 (49)      83 (78)       73 (65)     -
//    128 x 65536, 1024    48 (47)      40 (42)       36 (36)     57 (54)
// Unaligned        64x128     two a CU     128x128, deep   128x128
//   2049 x 1028, 4095      86 (107)    91  (82)       76  (75)       109 (107)
//   2304 x 1950, 2048      71  (85)    74  (71)       81  (81)        77 (106)
//   3000 x 2000, 3001     106 (123)   110 (106)      116 (116)       111 (155)
//   8192 x 4096, 4096     713 (846)   752 (719)      656 (665)       627 (840)
//     64 x 65536, 2048     58  (62)    60  (55)       90  (83)        88 (110)
//
// fp32 C: the largest that fills most of the CUs, but for a narrow C.  us, bf16 into
// fp32 / fp32, A m-major (k-major in brackets, else within a few percent):
//   M x N, K              32x32 str.   32x64 str.    64x64        64x128       128x128, deep
//    512 x  256, 1000      7.2/7.7       10/9.6      13/16         21/19
//     32 x 4096, 4096       16/18        26/22       42/50
//   1024 x  512, 1024       14/16        11/10       14/16
//   1024 x 1024, 4096       64/77        52/44       44/50         71/65         88/ -
//   2048 x 1024, 4096                                83/97         71/66         - /92
//   2048 x 2048, 4096                               165/192       142/113        95/104
//                          64x128        128x128     256x128 | 128x256 (Q's terms, A's terms)
//   4096 x 2048, 1024       80/61         50/74       49/54
//   2304 x 1952,   64       13/9.8 (12/12) 8.1/12     8.5/8.4 (8.7/8.5)
//   2304 x 1952, 2048      110/83 (105/97) 81/131     77/80 (74/76)
//   2600 x 1952, 2048      113/87 (107/99) 83/132     78/82 (74/78)
//   3008 x 2000, 3008      158/126       123/197     113/118
//   4096 x 4096, 2048       - /225       181/ -      176/179
//   8192 x 2048, 1024       - /115        94/ -       98/94
//     64 x 65536, 2048      81/67 (78/72) 101/ -     182/101 (145/88)
//    128 x 65536, 1024      81/64 (78/73)  50/ -      92/52 (79/50)
//  65536 x   64, 2048      155/144       107/150     101/206; 64x64: 101/128
//  65536 x  128, 1024       85/78 (87/88)  56/81      56/111; 128x128, deep: 60/70 (62/76)
// Unaligned                64x128     two a CU    128x128, deep  128x128
//   2049 x 1028, 4095      141/135     146/111        95/96      113/137
//   2304 x 1950, 2048      111/107     115/92         98/100      84/139
//   3000 x 2000, 3001      161/155     169/138       141/144     127/201
//     64 x 65536, 2048      82/76       84/67        110/113     101/141
//    128 x 65536, 1024      81/78       83/68         57/59       51/75
//  65536 x   64, 2048      162/161     162/149       115/134     109/155; 64x64: 106/135
//  65536 x  128, 1024       87/88       89/79         62/72       60/84
// (For 129 to 159 tiles of 256x128, or of 128x256 with m-major A, the smaller ones
// take 4 % longer from K = 512 on; at K = 64 128x128 5 % less, 64x128 14 % more.)
inline GradTile grad_tile(const GradShape& s)
{
    auto tiles = [&](int bm, int bn) { return ceil_div(s.M, bm) * ceil_div(s.N, bn); };
    if (tiles(32, 32) <= 256) return GradTile::Stream32x32;
    if (tiles(32, 64) <= 256) return GradTile::Stream32x64;
    if (tiles(64, 64) <= 256) return GradTile::T64x64;
    if (tiles(64, 128) <= 256) return GradTile::T64x128;
    if (tiles(128, 128) <= 256) return GradTile::T128x128Deep;
    if (s.M <= 64) return s.wide && s.split_a && !s.vec ? GradTile::T64x128Two : GradTile::T64x128;
    if (!s.wide) {
        if (!s.vec) return s.a_kmajor ? GradTile::T64x128Two : GradTile::T128x128;
        if (s.N <= 64) return GradTile::T64x64;
        if (s.N <= 128) return GradTile::T128x128;
        if (s.M > 128 && tiles(128, 256) > 256) return GradTile::T256x256;
        return s.K <= 128 && !s.a_kmajor ? GradTile::T128x128 : GradTile::Wide128x256;
    }
    if (s.split_a) {
        if (s.N <= 64) return GradTile::T64x64;
        if (s.N <= 128 || (!s.vec && s.M <= 128)) return GradTile::T128x128Deep;
        if (!s.vec) return GradTile::T64x128Two;
        return s.a_kmajor || tiles(128, 256) >= 160 ? GradTile::Wide128x256 : GradTile::T64x128;
    }
    if (!s.vec || s.M <= 128) return GradTile::T128x128;
    return tiles(256, 128) >= 160 ? GradTile::Tall256x128 : GradTile::T128x128;
}

inline int64_t grad_grid(const GradShape& s, const Tile& t) { return ceil_div(s.M, t.bm) * ceil_div(s.N, t.bn); }

}  // namespace mg
