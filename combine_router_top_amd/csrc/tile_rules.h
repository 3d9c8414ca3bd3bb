// Which kernels a training call, the router's gradients or an 8- or 4-bit call takes: rules
// on sizes and the number of compute units alone, without device code, so that any host
// compiler can evaluate them.  The launchers do what a plan says and decide nothing
// themselves.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace moe {

// ---------------------------------------------------------------------------
// tiles of seg_tile.h
// ---------------------------------------------------------------------------
constexpr int ST_KB = 128;     // bytes of K per stage

// The scalar offset of a load from a buffer of `size` bytes.  What lies past the end (blocks
// ahead of the last, groups that the last block has not, absent zero points, rows that a
// share has not) is asked for at the end, where the range check drops every lane: it
// compares lane offsets with the size less the scalar offset, which is not to pass zero.
constexpr uint32_t st_offset(uint32_t off, uint32_t size) { return off < size ? off : size; }
// The block or step of n that a copy ahead of its use takes: past the last one, that again.
constexpr int st_upto(int i, int n) { return i < n ? i : n - 1; }

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
// the router's gradients, bf16
// ---------------------------------------------------------------------------
// Tiles of dx are 64 x 128 where 256 x 256 ones would make less than half a round.
inline bool route_few(int64_t cus, int64_t T, int d) { return (T + 255) / 256 * ((d + 255) / 256) < cus / 2; }
// Shares of the tokens that the units of dWg are split into: as many as give every
// compute unit one, each of at least four stages.
inline int route_shares(int64_t cus, int64_t T, int d, int E) {
  const int64_t tiles = (int64_t)((d + 127) / 128) * ((E + 255) / 256), stages = (T + 63) / 64;
  return (int)std::max<int64_t>(1, std::min<int64_t>(cus / tiles, stages / 4));
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

// ---------------------------------------------------------------------------
// 4-bit products
// ---------------------------------------------------------------------------
// A product of rows with packed 4-bit weights [n][K][N] (gated: two of them side by
// side), kb blocks of 128 K; rows as in I8Shape.
struct W4Shape {
  bool gated, segments;
  int n, N, kb;
  int64_t mean, all, most;
};
struct W4Plan {
  bool tiles;        // w4_tile, else w4_stream
  int bm;            // tiles: rows of a block, a multiple of 64 up to 192
  int parts, per;    // tiles of a single product: parts of K, blocks of 128 K in each
  bool wide;         // stream: four column tiles of 16 a workgroup, else one (gated: of each matrix)
  bool low;          // stream: 16 rows at a time, else 32
  int blocks;        // stream: workgroups that a segment's blocks of rows are dealt out to
  int waves;         // stream: waves of a workgroup, among which K is dealt out
  bool ahead;        // stream: a wave loads its next block of K before it multiplies one
};

// What the kernels take, in us, by what they measured (K x N, rows: us of either side):
//   - wide stream: 2.4, and a workgroup 0.6 and, for each 4 blocks of 128 K, 0.6 or 0.034 a row;
//     narrow: 1.3, and 0.9 and, for each 8 blocks, 0.4 + 0.047 a row.  One workgroup at a time on
//     a compute unit; weights in bulk 5.2 and 4 TB/s.  Wide, narrow: 4096 x 14336, 1: 9.5, 13.4;
//     16: 9.9, 20.6; 32: 13.7, 36.6; 7168 x 2048, 1: 11.2, 5.9; 32: 18.1, 16.7; 2048 x 7168, 1: 5.6,
//     4.9; 16: 5.8, 7.5; 14336 x 4096, 64: 34, 58; 32 experts of 7168 x 2048 with 2 rows each, the
//     whole call: 111, 137.
//   - tiles: 0.72 + 0.5 h for each block of a tile of 64 h rows and 2.5 more; the rows'
//     preparation 6 and its bytes.  64, 128, 192 rows: 4096 x 14336, 256: 50, 62, 71; 512: 91,
//     67, 75; 2048: 288, 238, 233.  Wide stream and tiles: 1024 x 1024, 2048: 15, 22; 4096: 26,
//     25; 8192: 47, 33; 368 x 5824, 256: 9.9, 12.4; 512: 15.4, 13.1.
//   - K in parts: 3 more and the bytes of their sums.  One part, several: 7168 x 2048, 256: 74,
//     19; 512: 75, 33.
inline W4Plan w4_plan(int64_t cus, const W4Shape& p) {
  W4Plan r{};
  const int64_t act = std::min<int64_t>(p.n, std::max<int64_t>(1, p.all));   // experts with rows
  const int64_t seg = std::max<int64_t>(1, p.segments && p.n > 1 ? p.mean + p.mean / 4 : p.mean);
  const double mb = act * (p.kb * 1024e-6) * ((p.N + 15) / 16) * (p.gated ? 2 : 1);
  const double kept = std::max<double>(1, p.segments ? (double)p.all : (double)p.mean);   // rows in all
  const int64_t cols = (p.N + (p.gated ? 127 : 255)) / (p.gated ? 128 : 256);
  auto rounds = [&](int64_t wgs) { return (double)((wgs + cus - 1) / cus); };
  double tiles = 0;
  const double rows_us = 6 + kept * p.kb * (128 * 4e-6 / 4);
  for (int h = 3; h >= 1; --h) {
    const int64_t full = seg / (64 * h), rest = (seg % (64 * h) + 63) / 64;
    const int64_t wgs = act * (full + (rest ? 1 : 0)) * cols;
    for (int parts = 1; parts <= 16; parts *= 2) {
      if (parts > 1 && (p.segments || wgs * parts > cus || p.kb < 4 * parts)) break;
      const int per = (p.kb + parts - 1) / parts, used = (p.kb + per - 1) / per;
      double us = std::max(mb / 5.2, rounds(wgs * used) * (per * (0.72 + 0.5 * h) + 2.5)) + rows_us;
      if (used > 1) us += 3 + (used + 1) * kept * p.N * (4e-6 / 4);
      if (!r.bm || us < tiles) {
        r.bm = 64 * h;
        r.parts = used;
        r.per = per;
        tiles = us;
      }
    }
  }
  // stream: passes of 32 rows, the last of up to 16 or 32
  r.low = p.most <= 16 || p.mean <= 8;
  const int64_t pass = r.low ? 16 : 32, passes = (seg + pass - 1) / pass;
  r.blocks = (int)std::min<int64_t>((p.most + pass - 1) / pass, p.segments ? 4 : 1024);
  auto stream = [&](bool wide) {
    const int64_t per = wide ? (p.gated ? 32 : 64) : 16, wgs = act * ((p.N + per - 1) / per);
    const int64_t last = seg - (passes - 1) * pass;
    auto block = [&](int64_t rows) { return wide ? std::max(0.6, 0.034 * (double)rows) : 0.4 + 0.047 * (double)rows; };
    const double steps = (double)((p.kb + (wide ? 3 : 7)) / (wide ? 4 : 8)), more = wide ? 0.6 : 0.9;
    const double work = ((passes - 1) * block(pass) + block(last)) * steps + more * (double)passes;
    const double one = block(std::min(seg, pass)) * steps + more;
    return (wide ? 2.4 : 1.3) + std::max(mb / (wide ? 5.2 : 4), std::max(one, work * (double)wgs / (double)cus));
  };
  const double narrow = stream(false), wide = stream(true);
  r.wide = wide < narrow;
  r.tiles = std::min(wide, narrow) > tiles;
  // With several workgroups for each compute unit the waves beside one another hide its
  // loads, and registers for a block in advance only keep waves out (32 experts of 7168 x 2048,
  // 4 rows each: 4 waves with it 140 us, 8 without 126; 24 rows: 224, 222; 16 of 2048 x 768, 24 rows:
  // 25.6, 23.5); with one it pays (4096 x 14336, 8 rows: 9.5, 12.5; 24 rows: 12.6, 18.8).
  const int64_t wgs = (p.N + 63) / 64 * (int64_t)r.blocks;
  r.ahead = r.wide && !p.segments && wgs <= cus && p.kb > 4;
  // narrow ones for up to 16 rows take 16 waves where K lasts (7168 x 2048, one row: 8 waves 6.4 us, 16
  // 5.6; 8 experts of 512 x 512: 8.0, 8.9)
  r.waves = r.wide ? (r.low && !r.ahead ? 8 : 4) : r.low && p.kb >= 32 ? 16 : 8;
  return r;
}

}  // namespace moe
