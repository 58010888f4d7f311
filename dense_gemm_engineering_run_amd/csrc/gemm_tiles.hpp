// gemm_tiles.hpp -- which kernel a grouped or adapter call runs, and the size
// of its grid (host only; no HIP).  The launchers take their template arguments
// from the tables here, the entry points refuse grids from them.
#pragma once

#include <stdint.h>

namespace mg {

// A tile of C and how a workgroup goes about it: k of a tile (0: a streaming
// adapter product, its own), waves (streaming: 16x16 MFMA tiles) along m and
// n, MFMA size, stages in LDS (unaligned operands: tiles in flight).
// `extra`: waves that stream; of the other adapter products, adapters at a time
// (0: shared by a workgroup through LDS).
struct Tile {
    const char* name;
    int bm, bn, bk, wm, wn, mi, stages, extra, threads;
};

// Threads along one axis of a grid that a launch can have.
constexpr int64_t kMaxGridThreads = ((int64_t)1 << 32) - 1;

constexpr int64_t ceil_div(int64_t n, int64_t d) { return (n + d - 1) / d; }

// ------------------------------------------------------------ grouped products

enum class RaggedTile : int {
    Rows32x64, Rows64x128, Rows128x64, Rows128x128, Rows128x128Two, Rows128x256, PingPong,
    K64x64, K128x128, K128x128Two,
    Odd32x64, Odd64x128, Odd128x128, OddK64x64, OddK128x128,
    F32Stream16x32, F32Stream32x64, F32Stream32x32, F32Rows64x64, F32Rows64x128, F32Two64x64, F32K128x128,
    Count
};
constexpr Tile kRaggedTiles[] = {
    {"rows 32x64", 32, 64, 128, 1, 4, 16, 3, 0, 256},
    {"rows 64x128", 64, 128, 64, 2, 2, 16, 3, 0, 256},
    {"rows 128x64", 128, 64, 64, 2, 2, 16, 4, 0, 256},
    {"rows 128x128", 128, 128, 64, 2, 2, 16, 4, 0, 256},
    {"rows 128x128 in two stages", 128, 128, 64, 2, 2, 32, 2, 0, 256},
    {"rows 128x256", 128, 256, 64, 2, 4, 16, 3, 0, 512},
    {"ping-pong 256x256", 256, 256, 64, 4, 2, 16, 3, 0, 512},
    {"k 64x64", 64, 64, 64, 2, 2, 32, 4, 0, 256},
    {"k 128x128", 128, 128, 64, 2, 4, 16, 4, 0, 512},
    {"k 128x128 in two stages", 128, 128, 64, 2, 2, 32, 2, 0, 256},
    {"unaligned rows 32x64", 32, 64, 128, 2, 4, 16, 2, 0, 512},
    {"unaligned rows 64x128", 64, 128, 64, 2, 4, 16, 2, 0, 512},
    {"unaligned rows 128x128", 128, 128, 64, 2, 4, 16, 2, 0, 512},
    {"unaligned k 64x64", 64, 64, 128, 2, 4, 16, 2, 0, 512},
    {"unaligned k 128x128", 128, 128, 64, 4, 2, 16, 2, 0, 512},
    {"fp32 stream 16x32", 16, 32, 32, 1, 2, 16, 3, 4, 256},
    {"fp32 stream 32x64", 32, 64, 32, 2, 4, 16, 2, 4, 256},
    {"fp32 stream 32x32", 32, 32, 32, 2, 2, 16, 2, 4, 256},
    {"fp32 rows 64x64", 64, 64, 32, 2, 2, 32, 3, 0, 256},
    {"fp32 rows 64x128", 64, 128, 32, 2, 2, 32, 2, 0, 256},
    {"fp32 64x64 in two stages", 64, 64, 32, 2, 2, 32, 2, 0, 256},
    {"fp32 k 128x128", 128, 128, 32, 2, 2, 32, 2, 0, 256},
};
static_assert(sizeof(kRaggedTiles) / sizeof(Tile) == (int)RaggedTile::Count, "one entry a tile");
constexpr Tile tile_of(RaggedTile t) { return kRaggedTiles[(int)t]; }

// What the choice looks at.  By rows M is the rows of all groups; by k M and N
// are C's (exchanged where C is m-major).
struct RaggedShape {
    bool f32, by_rows, vec, b_kmajor;      // vec: operands allow 16-byte loads
    int64_t M, N, groups;
};

// By rows the tile height follows the rows a group has on average (the host
// knows no more), then how many tiles that makes.  The limits stand between
// sizes that were measured on both sides.
//
// 16-bit, measured in bf16, B k-major (n-major in brackets where it differs), us:
//   rows/group  groups  N x K       16-row 32     64     128x128 128x256 256x256
//       1         8     4096 x 4096   39.7  38.6 [44.9] 42.0 [36.7] 41.6  61.7  75
//      16         8     4096 x 4096   55.9  53.2 [62.8] 61.8 [47.5] 62.5  74.1  75
//      16        64     2048 x 1024   60.3  56.9   51.5   61.1   59.0   85
//      64         8     4096 x 4096  100    77.4   67.3   90.4   78.7   88.9
//     128         8     4096 x 4096  168   118     95.6   89.0   80.2   89.2
//     128        32     2048 x 4096                155    143    153    194
//     256         8     4096 x 4096               132    121    126     90.9
//     256         8     2048 x 1024                21.1   25.7   20.2   23.5
//    1024         8     4096 x 2048               206    190    175    140
//    4096         8     4096 x 4096                      1270   1150    847
// (128x256 on eight waves of 16x16 MFMAs; on four of 32x32: 82.8 and 160 at
// 128 rows.)  Too few tiles of 128x256: 128x128, from 192 rows on in two
// stages, two workgroups a CU (22.9 us at 256 rows in 8 groups of 2048 x
// 1024, 24.6 in four stages).
// Products too small to fill the chip with those take the tile that spreads
// them further: 1 group of 48 rows of 1024 x 4096 14.6 on 32x64 (25.8 on
// 64x128), 4 groups of 128 20.2 (34.3 on 128x128), 4 groups of 300 28.0 on
// 128x64 (37.1 on 128x128).
// At the limits (K = 2048 unless given; the tile above a limit second):
//   320 tiles of 32x64: 5 groups of 32 rows, N = 4096, 18.4 and 17.2 (4 groups
//     13.8 and 16.8); 5 of 64, N = 2048, 14.0 and 16.3; 2 of 128 rows, N = 2560,
//     13.4 and 15.5 on 128x64.
//   192 tiles of 128x64: 4 groups of 128 rows, N = 3008, 16.3 and 21.8 on
//     128x128; 4 of 256, N = 1536, 16.3 and 21.2.
//   24 rows: 16 groups, N = 2048, 23.8 and 24.5; 8 of 4096 x 4096 55.4 and 65.9
//     (32 rows 57.0 and 66.1); n-major 26.1 and 23.3 at 16.
//   80 rows: 16 groups, N = 2048, 30.1 and 26.2 (64 rows 25.3 and 25.8).
//   192 rows: 16 groups, N = 2048, 37.4 on 128x256 and 45.2 on 256x256 (224
//     rows 40.9 and 47.0); 100 tiles of 256x256: 6 groups of 256 rows, N = 4096,
//     32.4 and 39.4 (128 tiles 40.7 and 46.8).
//   100 tiles of 128x256: 7 groups of 128 rows, N = 3500, 23.7 on 128x128 and
//     31.2; 9 of 256, N = 1536, 28.4 and 29.6.
//
// Unaligned 16-bit operands, eight waves a tile.  Measured in bf16, B k-major
// (n-major in brackets where it differs), us, in brackets behind the 128x128
// tile: on four waves:
//   rows/group  groups  N x K         32x64   64x128       128x128           256x128
//       2         8     4095 x 4095    54.8    70.6         72.7 ( 90.4)      98.3
//      16        64     1023 x 2047    72.0    67.4 [58.4]  72.0 ( 99.7)     107
//      50         2     4095 x 1023    10.9    17.0         20.2 ( 26.7)      28.4
//      64        32     2047 x 2047   117      97.5 [86.8] 110   (149)       116
//     128        32     2047 x 2047   189     142          116   (160)       168
//     512        16     4095 x 2047   635     397          298   (446) [278] 345 [350]
// Loads element by element took 181, 190, -, -, -, 1657 us.
// At the limits (K = 2048): 8 rows in 16 groups, N = 2048, 26.8 and 34.4; 320
// tiles, 5 groups of 40, N = 2048, 24.0 and 29.1; 80 rows in 16 groups 52.5 and
// 40.9 (64 rows 39.1 and 40.5).
//
// fp32, us (K = 1024; 64x64 in three stages, 64x128 in two, 128x128 in two):
//           64 rows in  4 groups of 1024     24.2    41.9   66.9
//         1024 rows in 16 groups of 2048     60.1    70.6  126
//         4096 rows in 16 groups of 2048    178     165    196
//        16384 rows in 16 groups of 2048    577     549    562
// Few rows stream (16x32, 32x64 and 32x32 tiles; B k-major, n-major in
// brackets), against 64x64, us:
//        1 row  in 122 groups of  384 x 4224   86.7 [ 95.8]    95.1          94.9   157
//       16 rows in   8 groups of 4096 x 4096  109   [121]     113           110     164
//       22 rows in  14 groups of 7192 x 5264  569   [632]     455   [441]   505     611
//       48 rows in  16 groups of 2048 x 2048   99.5 [107]      92.7          91.8   112
//       64 rows in  16 groups of 2048 x 1024                   69.3          68.9    62.9
//      300 rows in   1 group  of 1024 x 4096                   40.8          39.8    83.6
// (Four waves that share a row's k-tiles also round less than one.)
// At the limits: 16 rows in 8 groups of 4096 x 4096 104 and 112 on 32x64 (20
// rows 128 and 113); 48 rows in 16 groups of 2048 x 2048 101 on 32x64, 95 on
// 32x32, 79 on 64x64; 192 tiles of 64x64, 12 groups of 64 rows of 1024 x 2048,
// 36.8 and 45.1; 1024 tiles of 64x128, 16 groups of 256 rows of 2048 x 1024, 146
// on 64x64 and 169 (18 groups 165 and 170).
inline RaggedTile rows_tile(const RaggedShape& s)
{
    const int64_t avg = ceil_div(s.M, s.groups);
    auto tiles = [&](int bm, int bn) { return s.groups * ceil_div(avg, bm) * ceil_div(s.N, bn); };
    if (s.f32) {
        if (avg <= 16) return RaggedTile::F32Stream16x32;
        if (avg <= 48) return RaggedTile::F32Stream32x64;
        if (tiles(64, 64) <= 192) return RaggedTile::F32Stream32x32;
        if (!s.vec) return RaggedTile::F32Two64x64;
        return tiles(64, 128) >= 1024 ? RaggedTile::F32Rows64x128 : RaggedTile::F32Rows64x64;
    }
    if (!s.vec) {
        if (avg <= 8 || tiles(32, 64) <= 320) return RaggedTile::Odd32x64;
        return avg <= 80 ? RaggedTile::Odd64x128 : RaggedTile::Odd128x128;
    }
    if (tiles(32, 64) <= 320) return RaggedTile::Rows32x64;
    if (avg > 80 && tiles(128, 64) <= 192) return RaggedTile::Rows128x64;
    if (avg <= 24) return s.b_kmajor ? RaggedTile::Rows32x64 : RaggedTile::Rows64x128;
    if (avg <= 80) return RaggedTile::Rows64x128;
    if (avg >= 192 && tiles(256, 256) >= 100) return RaggedTile::PingPong;
    if (tiles(128, 256) >= 100) return RaggedTile::Rows128x256;
    return avg < 192 ? RaggedTile::Rows128x128 : RaggedTile::Rows128x128Two;
}

// By k, 16-bit: 256x256 tiles from three quarters of a CU's share of them up
// (bf16 -> fp32, 8 groups: 4096 x 2048 of 8192 k 161 us against 197 on 128x128;
// 4 groups of 2048 x 2048 of 4096 k, 256 tiles, 43.2 against 48.1), then
// 128x128 in two stages, two workgroups a CU (8 groups of 1024 x 1024, 128
// tiles of 256x256: 36.4 against 47.1), up to one a CU in four (4 groups of
// 1024 x 1024: 19.5 against 24.4), and 64x64 where even those leave CUs idle
// (8 groups of 512 x 512 of 8192 k: 19.9 against 22.1; in 4 groups of 256 x
// 256 19.7 against 29.3).
// Unaligned, bf16 -> fp32, us: 8192 k in 16 groups of 4095 x 2047 402 (on 64x64
// tiles 561); 4096 k in 4 groups of 1023 x 1023, 256 tiles, 30.0 (38.2 on 64x64
// with 128 k at a time); 8192 k in 8 groups of 511 x 511, 128 tiles, 34.6
// (26.7); in 4 groups of 255 x 255 47.1 (29.8).
// fp32, us (64x64 in two stages, 128x128 in two), 4096 k:
//        16 groups of 512 x 512              28.1           43.4
//         4 groups of 1024 x 1024            75.7           98.6
//         4 groups of 4096 x 2048           550            503
// At the limits (1024 k a group; the tile above a limit second): 192 tiles of
// 256x256, 6 groups of 2048 x 1024, 36.8 on 128x128 and 37.7 (into bf16 35.4 and
// 33.4); 256 tiles of 128x128, 4 groups of 1024 x 1024, 16.5 on eight waves and
// 17.3 (5 groups 27.1 and 20.5); 192, 4 groups of 1024 x 768, 19.6 on 64x64 and
// 15.5.  Unaligned, 8 groups of 512 x 512 21.9 and 21.5 (10 groups 29.7 and
// 21.8).  fp32, 512 tiles, 8 groups of 1024 x 1024 of 512 k 75.6 and 69.9.
inline RaggedTile k_tile(const RaggedShape& s)
{
    auto tiles = [&](int t) { return ceil_div(s.M, t) * ceil_div(s.N, t) * s.groups; };
    if (s.f32) return tiles(128) >= 512 ? RaggedTile::F32K128x128 : RaggedTile::F32Two64x64;
    if (!s.vec) return tiles(128) <= 128 ? RaggedTile::OddK64x64 : RaggedTile::OddK128x128;
    if (tiles(256) >= 192) return RaggedTile::PingPong;
    if (tiles(128) > 256) return RaggedTile::K128x128Two;
    return tiles(128) >= 192 ? RaggedTile::K128x128 : RaggedTile::K64x64;
}

inline RaggedTile ragged_tile(const RaggedShape& s) { return s.by_rows ? rows_tile(s) : k_tile(s); }

// Workgroups along x.  By rows, ceil(len_g / bm) tiles of bm rows summed over
// the groups are at most (rows + groups * (bm - 1)) / bm, and no more than rows.
// (By k the groups lie along y.)
inline int64_t ragged_grid(const RaggedShape& s, const Tile& t)
{
    const int64_t n = ceil_div(s.N, t.bn);
    if (!s.by_rows) return ceil_div(s.M, t.bm) * n;
    const int64_t m = (s.M + s.groups * (t.bm - 1)) / t.bm;
    return (m < s.M ? m : s.M) * n;
}

// ------------------------------------------------------------ adapter products

enum class LoraTile : int {
    Stream16x16, Stream16x32, Stream32x32,
    Few16x32, Few32x32, Shared32x32, Shared64x64, Shared64x64Four, Shared128x128, PingPong,
    Odd32x32, Odd64x64, Odd128x128, Odd256x128,
    F32Rows64x64, F32Rows64x128, F32Odd64x64,
    Count
};
constexpr Tile kLoraTiles[] = {
    {"stream 16x16", 16, 16, 0, 1, 1, 16, 4, 8, 768},
    {"stream 16x32", 16, 32, 0, 1, 2, 16, 3, 8, 768},
    {"stream 32x32", 32, 32, 0, 2, 2, 16, 2, 8, 768},
    {"16x32", 16, 32, 256, 1, 2, 16, 4, 4, 128},
    {"32x32", 32, 32, 128, 2, 2, 16, 4, 4, 256},
    {"shared 32x32", 32, 32, 128, 2, 2, 16, 4, 0, 256},
    {"shared 64x64", 64, 64, 128, 2, 4, 16, 3, 0, 512},
    {"shared 64x64 in four stages", 64, 64, 64, 2, 4, 16, 4, 0, 512},
    {"shared 128x128", 128, 128, 64, 2, 4, 16, 4, 0, 512},
    {"shared ping-pong 256x256", 256, 256, 64, 4, 2, 16, 3, 0, 512},
    {"unaligned 32x32", 32, 32, 256, 2, 2, 16, 2, 1, 256},
    {"unaligned 64x64", 64, 64, 128, 2, 4, 16, 2, 1, 512},
    {"unaligned 128x128", 128, 128, 64, 4, 2, 16, 2, 1, 512},
    {"unaligned 256x128", 256, 128, 64, 4, 2, 16, 2, 1, 512},
    {"fp32 64x64", 64, 64, 32, 2, 2, 32, 3, 2, 256},
    {"fp32 64x128", 64, 128, 32, 2, 2, 32, 2, 2, 256},
    {"unaligned fp32 64x64", 64, 64, 32, 2, 2, 32, 2, 2, 256},
};
static_assert(sizeof(kLoraTiles) / sizeof(Tile) == (int)LoraTile::Count, "one entry a tile");
constexpr Tile tile_of(LoraTile t) { return kLoraTiles[(int)t]; }

struct LoraShape {
    bool f32, vec, b_kmajor;      // vec: A, B and down allow 16-byte loads
    int64_t M, N;
};

// The limits stand between sizes that were measured on both sides, rows with an
// adapter each up to 64 rows and packed prompts above, at N = 4096.  (Those by M
// alone suit N up to that: 144 rows at N = 14336, K = 4096 take 97 us on 32x32
// and 58 on 128x128.)
//
// fp32, N = K = 4096, us for both kernels (rows: one adapter each of 16 up to
// 64, packed above; B n-major in brackets):
//   rows rank  16x16 str.    16x32 str.    32x32 str.    64x64        64x128
//      1  16    24.2 [31.3]   26.2 [28.5]   31.6 [31.6]    94 [ 95]
//     16 128    47.1 [61.1]   54.3 [68.3]   65.6 [78.9]   146 [182]
//     32  16    40.2 [55.4]   31.9 [37.0]   39.6 [44.8]   107 [113]
//     64  16    65.1 [86.8]   48.8 [58.8]   40.6 [43.5]   108 [113]
//    128  16    96.2 [141]    69.4 [94.0]   56.6 [70.3]    96 [110]
//    256 128                               158  [224]     130 [146]     238 [238]
//   1024  16                               419  [429]     298 [303]     283 [284]
//   4096  16                              1344           1110          1065
// At the limits: 16 rows 27.1 and 29.9 (24 rows 35.2 and 30.9), 32 rows 30.5 and
// 40.9 (48 rows 44.2 and 44.1), 192 tiles of 64x64 73.8 and 96.0 (256 tiles 92.0
// and 96.5), 512 tiles of 64x128 296 and 275.
//
// Unaligned 16-bit operands, bf16, N = 4096, K = 4095, us for both kernels
// (rows: one adapter each of 16 up to 64, packed above):
//   rows rank  32x32   64x64   128x128  256x128
//      1  16    29.4    41.5     71.4    104
//     64  16    38.3    58.2    105      154
//    128  64    45.2    54.4    100      127
//    256  64    77.7    55.6     98.0    143
//   1024  64   297     182      115      171
//   4096  64   971     517      383      315
// (Loads element by element: 123 at one row, 1853 at 4096.)
// At the limits: 128 rows 41.7 and 49.4, 144 rows 61.5 and 50.4; 512 tiles of
// 64x64 78.8 and 89.7 (576 107 and 92); 256 tiles of 256x128 175 on 128x128 and
// 149 (2304 rows 251 and 271).
//
// 16-bit, bf16, N = K = 4096, us for both kernels (rows: one adapter each up to
// 64, packed above; rank):
//   rows rank  16x16 str. 16x32 str. 32x16 str. 32x32   32x32 sh. 64x64 sh. 128x128 sh. 256x256 sh.
//      1  16   15.2                  17.3       19.4
//     16  16   20.2                  22.9       25.5
//     32  16   30.4       23.4       23.8       27.2
//     32 128              42.6       57.2
//     64  16   53.3       35.4       38.3       30.5    34.5      65.6
//    128  64                                    42.9    31.9      37.4      62.6        100
//    256  64                                    43.3    48.9      33.9      56.1        103
//    512  64                                                      49.5      55.0        103
//   1024  64                                                      86.4      59.5        102
//   2048  64                                                     151       109          107
//   8192  64                                                     482       367          234
// (str.: the streaming kernel for few rows, B k-major only; sh.: adapters
// through LDS for the whole workgroup, of eight waves from 64x64 on: 1024 rows
// 66.5 on four.)  64x64 tiles that the chip holds at once take 128 of k at a
// time in three stages (33.9 us at 256 rows, 36.6 with 64 in four; at 512 rows
// 56.9 and 49.5).
// At the limits (rank 16 up to 40 rows, 64 above): 16 rows 21.5 and 24.8 (20
// rows 30.4 and 24.4); 32 rows 25.0 and 29.4 (40 rows 36.2 and 30.3), B n-major
// 28.8 and 29.9 (44.8 and 30.7); 96 rows packed 28.0 on 32x32 and 27.8 shared,
// an adapter each 43.1 and 53.9; 128 rows 27.7 and 30.8 on 64x64, 144 rows 40.5
// and 32.2; 256 tiles of 64x64 30.6 and 34.9 (320 51.1 and 45.9), 512 45.5 and
// 47.6 on 128x128 (576 66.1 and 49.5); 100 tiles of 256x256 (1664 rows are 112)
// 94.0 on 128x128 and 95.4, 1792 rows 94.5 and 93.8.
inline LoraTile lora_tile(const LoraShape& s)
{
    auto tiles = [&](int bm, int bn) { return ceil_div(s.M, bm) * ceil_div(s.N, bn); };
    if (s.f32) {
        if (s.M <= 16) return LoraTile::Stream16x16;
        if (s.M <= 32) return LoraTile::Stream16x32;
        if (tiles(64, 64) <= 192) return LoraTile::Stream32x32;
        if (!s.vec) return LoraTile::F32Odd64x64;
        return tiles(64, 128) >= 512 ? LoraTile::F32Rows64x128 : LoraTile::F32Rows64x64;
    }
    if (!s.vec) {
        if (s.M <= 144) return LoraTile::Odd32x32;
        if (tiles(64, 64) <= 512) return LoraTile::Odd64x64;
        return tiles(256, 128) >= 256 ? LoraTile::Odd256x128 : LoraTile::Odd128x128;
    }
    if (s.b_kmajor && s.M <= 32) return s.M <= 16 ? LoraTile::Stream16x16 : LoraTile::Stream16x32;
    if (s.M <= 32) return LoraTile::Few16x32;
    if (s.M <= 96) return LoraTile::Few32x32;
    if (s.M <= 144) return LoraTile::Shared32x32;
    if (tiles(256, 256) >= 100) return LoraTile::PingPong;
    if (tiles(64, 64) <= 256) return LoraTile::Shared64x64;
    return tiles(64, 64) <= 512 ? LoraTile::Shared64x64Four : LoraTile::Shared128x128;
}

// Workgroups of the product; the streaming kernel's column tiles stand in chunks
// of 8, one per XCD.
inline int64_t lora_grid(const LoraShape& s, const Tile& t)
{
    const int64_t n = ceil_div(s.N, t.bn);
    return ceil_div(s.M, t.bm) * (t.bk ? n : ceil_div(n, 8) * 8);
}

}  // namespace mg
