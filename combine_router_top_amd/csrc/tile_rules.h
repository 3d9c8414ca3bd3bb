// Which kernels a training or 8-bit call takes: rules on sizes and the number of
// compute units alone, without device code, so that any host compiler can evaluate
// them.  The launchers do what a plan says and decide nothing themselves.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace moe {

// ---------------------------------------------------------------------------
// tiles of seg_tile.h
// ---------------------------------------------------------------------------
constexpr int ST_KB = 128;     // bytes of K per stage

// Height (in units of 64 rows) of the tiles for segments of about `mean` rows of
// n experts: the one whose rounds of workgroups take the least time.  A stage of
// a tile costs the copies of its rows and columns, at the 38 GB/s that a compute
// unit sustains from L2, but at least about half a microsecond; a tile costs
// about 4 us more (first loads, epilogue).  Segments are taken a quarter longer
// than the mean unless there is one alone: a segment that does not fit its tile
// reads all its columns again.  ntn[h]: column blocks for height h, each of
// bn[h] operand columns; 0: no such tile.
inline int st_height(int64_t cus, int64_t n, int64_t mean, int stages, const int (&ntn)[5], const int (&bn)[5]) {
  const int64_t seg = std::max<int64_t>(1, n > 1 ? mean + mean / 4 : mean);
  int best = 0;
  double least = 0;
  for (int h = 4; h >= 1; --h) {
    if (!ntn[h]) continue;
    const int64_t tiles = n * ((seg + 64 * h - 1) / (64 * h)) * ntn[h];
    const double stage = std::max(0.5, (64 * h + bn[h]) * 128 / 38e3);
    const double us = (double)((tiles + cus - 1) / cus) * (stages * stage + 4.0);
    if (!best || us < least) {
      best = h;
      least = us;
    }
  }
  return best;
}
// The same for tiles of 256 columns and, at height 1, `small` columns.
inline int st_height(int64_t cus, int64_t n, int64_t mean, int64_t kbytes, int N, int small) {
  const int wide = (N + 255) / 256;
  return st_height(cus, n, mean, (int)((kbytes + ST_KB - 1) / ST_KB), {0, (N + small - 1) / small, wide, wide, wide},
                   {0, small, 256, 256, 256});
}

// ---------------------------------------------------------------------------
// training, bf16: tk assignments to E experts, n of them here
// ---------------------------------------------------------------------------
struct TrainPlan {
  int up, down;   // tile heights
};
inline TrainPlan train_plan(int64_t cus, int64_t tk, int E, int n, int d, int f) {
  const int64_t seg = std::max<int64_t>(1, tk / E);   // expected rows of a segment
  const int nup = (f + 127) / 128;
  return TrainPlan{st_height(cus, n, seg, (d + 63) / 64, {0, nup, nup, nup, nup}, {0, 256, 256, 256, 256}),
                   st_height(cus, n, seg, (int64_t)f * 2, d, 256)};
}

// How the weight gradients run: whole segments by st_run, short ones by
// st_run_short, or long segments of few tiles split along their rows.
enum { WG_LONG = 0, WG_SHORT = 1, WG_SPLIT = 2 };
constexpr int WG_SHORT_ROWS = 512;   // expected rows up to which the weight gradients take st_run_short

// Parts that the rows of the weight gradients are split into: as many as make
// the least time by the rule of st_height, the fp32 parts written and read at
// about 4 TB/s, at most 256 MB of them.  1: not split.
inline int weight_parts(int64_t cus, int64_t tk, int E, int n, int d, int f) {
  const int64_t mean = tk / E, stages = (mean + 63) / 64;
  const int64_t tiles = 3 * (int64_t)n * ((d + 255) / 256) * ((f + 255) / 256);
  const double elems = 3.0 * n * d * f;
  int best = 1;
  double least = 0;
  for (int s = 1; s <= 32 && (s == 1 || (s * elems * 4 <= 256e6 && stages >= 4 * s)); ++s) {
    const double us = (double)((tiles * s + cus - 1) / cus) * ((stages + s - 1) / s * 1.72 + 4) +
                      (s > 1 ? 4 + elems * (8.0 * s + 2) / 4e6 : 0);
    if (s == 1 || us < least) {
      best = s;
      least = us;
    }
  }
  return best;
}

struct BackwardPlan {
  int gate, input;   // tile heights
  int mode;          // WG_*
  int div;           // WG_SPLIT: parts; WG_SHORT: row blocks of a unit at most
  int64_t units;     // tiles (WG_SPLIT: of all parts) of the weight gradients
  bool apart;        // input and weight gradients in a launch each
};
// input: dx is wanted; wants: weight gradients that are (each has the same number
// of tiles).
inline BackwardPlan backward_plan(int64_t cus, int64_t tk, int E, int n, int d, int f, bool input, int wants) {
  const int64_t mean = tk / E;   // expected rows of a segment
  const int64_t tiles = (int64_t)wants * ((d + 255) / 256) * ((f + 255) / 256) * n;
  BackwardPlan p;
  p.gate = st_height(cus, n, mean, (int64_t)d * 2, f, 128);
  p.input = input ? st_height(cus, n, mean, (int64_t)f * 4, d, 128) : 4;
  const int parts = weight_parts(cus, tk, E, n, d, f);
  if (wants && parts > 1) {
    p.mode = WG_SPLIT;
    p.div = parts;
    p.units = tiles * parts;
  } else if (mean <= WG_SHORT_ROWS) {
    // runs of row blocks that share their columns: up to 4 (8, 2 and 1 measured
    // 864, 813 and 839 us against 808 on 32 experts of about 128 rows), fewer where that
    // would leave less than four units for each compute unit
    p.mode = WG_SHORT;
    p.div = (int)std::min<int64_t>(4, std::max<int64_t>(1, tiles / (4 * cus)));
    p.units = tiles;
  } else {
    p.mode = WG_LONG;
    p.div = 1;
    p.units = tiles;
  }
  // Apart where both have many rounds of long tiles: workgroups that finish the
  // first walk at different times no longer share operands in an L2 in the
  // second (8 dense experts: 18.62 ms against 18.87 in one launch).
  p.apart = input && wants && p.mode == WG_LONG && p.units >= 8 * cus;
  return p;
}

// ---------------------------------------------------------------------------
// 8-bit products
// ---------------------------------------------------------------------------
constexpr int I8_THIN = 32;        // rows up to which a segment may stream beside a launch of tiles
constexpr int I8_THIN_MEAN = 64;   // expected rows of a segment from which all of them take tiles
constexpr int I8_THIN_MOST = 128;  // longest possible segment for which all of them stream

// A product of rows with packed weights [n][K][N] (gated: two of them side by side),
// kt blocks of 64 K.
struct I8Shape {
  bool gated, segments;   // segments: rows of n experts; else one segment of `most` rows
  int n, N, kt;
  int64_t mean, all, most;   // expected rows of a segment and of all; bound of one segment's rows
};
struct I8Plan {
  bool stream;   // i8_stream, for all segments or for those of at most I8_THIN rows
  bool tiles;    // i8_tile, for all segments or for those that do not stream
  bool wide;     // stream: four tiles of 16 columns a workgroup, else one (gated: of each matrix)
  bool low;      // stream: up to 16 rows
  int blocks;    // stream: workgroups that a segment's blocks of 32 rows are dealt out to
  int height;    // tiles
};

// Output columns of a tile of height h.
constexpr int i8_cols(bool gated, int h) { return (h == 1 ? 128 : 256) / (gated ? 2 : 1); }

// Whether the stream takes less time than the tiles, by what both measured: a
// round of tiles about 4 us and 0.36 for each stage of 128 K; a round of narrow
// stream workgroups, one for each 16 columns and 32 rows, about 4 us and 0.05 for
// each 64 K; weights in bulk 4.7 and 6 TB/s.  5 us for a second launch.  E.g.
// (K x N, rows: tiles, stream in us) 5824 x 368, 128: 20.4, 9.1; 7168 x 2048, 64:
// 24.8, 12.2; 512 x 512, 64: 5.0, 7.8; 4096 x 14336, 64: 18.5, 44.2.
inline bool i8_streams(int64_t cus, const I8Shape& p, bool wide, bool alone) {
  const int64_t rows = std::max<int64_t>(1, p.mean), act = std::min<int64_t>(p.n, std::max<int64_t>(1, p.all));
  const int ntiles = (p.N + 15) / 16;
  auto rounds = [&](int64_t wgs) { return (double)((wgs + cus - 1) / cus); };
  const double mb = act * (p.kt * 1024e-6) * ntiles * (p.gated ? 2 : 1);   // act: experts with rows
  const int64_t cols = (p.N + i8_cols(p.gated, 1) - 1) / i8_cols(p.gated, 1);
  const double tiles = std::max(mb / 4.7, rounds(act * ((rows + 63) / 64) * cols) * (4 + 0.18 * p.kt));
  const int64_t blocks = (rows + 31) / 32;
  const double stream =
      wide ? 2 + blocks * mb / 6 : std::max(mb / 6, 2 + rounds(act * blocks * ntiles) * (4 + 0.05 * p.kt));
  return stream + (alone ? 0 : 5) <= tiles;
}

inline I8Plan i8_plan(int64_t cus, const I8Shape& p) {
  I8Plan r{};
  // four tiles of 16 columns a workgroup where that still makes a workgroup
  // per compute unit, else one
  r.wide = (int64_t)((p.N + (p.gated ? 31 : 63)) / (p.gated ? 32 : 64)) * p.n >= cus;
  // a second launch for the segments that do not fit costs about 5 us even if
  // there are none; short batches stream them in blocks of 32 rows instead (32
  // experts, 128 tokens: 246 -> 241 us, with skewed routing 247 -> 203 us; with
  // 256 tokens and skewed routing the tiles are faster, 75 against 123 us)
  const bool alone = !p.segments || p.most <= I8_THIN_MOST;
  r.stream = (!p.segments || p.mean <= I8_THIN_MEAN) && i8_streams(cus, p, r.wide, alone);
  r.tiles = !(r.stream && alone);
  r.low = p.most <= 16;
  // A segment's blocks of 32 rows go to workgroups of their own: all of them for a
  // single product, up to 4 for segments (100 tokens, skewed over 16 experts of
  // 2048 x 768: whole call 53.7 -> 42.4 us; 128 even rows over 32 experts 243.8,
  // 243.7).  Beside tiles a segment that streams has one block.
  r.blocks = r.tiles ? 1 : (int)std::min<int64_t>((p.most + 31) / 32, p.segments ? 4 : 1024);
  auto cols = [&](int h) { return (p.N + i8_cols(p.gated, h) - 1) / i8_cols(p.gated, h); };
  const int ncol = cols(2);
  if (r.tiles)
    r.height = st_height(cus, p.n, p.mean, (p.kt + 1) / 2, {0, cols(1), ncol, ncol, ncol}, {0, 128, 256, 256, 256});
  return r;
}

}  // namespace moe
