// share_out.h -- how many CTAs of attention over shared prefixes take the rows'
// own keys and how many the prefixes (attn_prefix.cu): the arithmetic, for the
// device and for a host.
#pragma once

#include <math.h>
#include <string.h>

#ifdef __CUDACC__
#define GQA_BOTH __host__ __device__ __forceinline__
#else
#define GQA_BOTH inline
#endif

namespace gqa {

// So that both parts end at the same time, by what they were measured to take (ns).
//   Two tiles of query rows a CTA: the MMAs bound a prefix, kPair a block of 128 keys.  Beside it an SM streams own keys
//   at kOwnTile a tile of 8 KB, all SMs together at kOwnTileAll.
//   One tile of rows, held by both: the memory bounds both parts, and an SM gets its share of it: kByte a byte.
// 64 rows over 8192 keys and 32768 own ones, CTAs of own keys 64 / 72 / 80 / 88 / 96: 43.4, 42.5, 42.0, 41.6, 44.5 us;
// 256 rows over 32768, 32 / 34 / 36 / 38: 132.3, 130.0, 129.9, 132.4.  (These two sizes are what the constants were
// fitted on.)
constexpr float kOwnStart = 6000.f, kOwnTile = 94.f, kOwnTileAll = 1.25f;
constexpr float kOwnUnit = 2000.f;    // a unit, of one of a CTA's warps: its queries and its output
constexpr float kPreStart = 10000.f, kPair = 1350.f, kByte = 1.f / 41.f;
constexpr float kPiece = 5000.f;      // a second piece: its queries, the first one's drain and partial

// What is to be shared out between `ctas` CTAs.
struct ShareWork {
  int ctas;
  int width, runs, prefixes;   // CTAs of a team; (K/V head, outer row block) pairs; prefixes
  int blocks;                  // key blocks of all prefixes' runs
  bool split;                  // one tile of rows, held by both tiles of a CTA
  int heads;                   // (K/V head, row block) pairs of the own keys
  int tiles, rows;             // of own keys: tiles of 8 KB a pair, batch rows that have any
  int warps;                   // that take own keys, of a CTA
  int D;
};

// Estimated time of the call if `own` CTAs take the own keys, 1 <= own <= ctas - width.  Counts are multiplied as floats:
// 2^30 blocks of 2^10 runs pass 32 bits.
GQA_BOTH float share_time(const ShareWork& s, int own) {
  const float tile = s.split ? 8192 * kByte : kOwnTile, block = s.split ? 4 * 128 * s.D * kByte : kPair;
  const float start = s.split ? kOwnStart : kPreStart;
  const float one = (s.tiles * tile + s.rows * (kOwnUnit / s.warps)) * (float)s.heads, all = s.tiles * kOwnTileAll * (float)s.heads;
  const float t_own = kOwnStart + fmaxf(one / own, all);
  const int teams = (s.ctas - own) / s.width;
  // one prefix: no CTA crosses from a unit to the next if the teams are a multiple of its runs, or the reverse
  const bool whole = s.prefixes == 1 && (teams % s.runs == 0 || s.runs % teams == 0);
  const int most = (s.blocks + teams - 1) / teams;
  const float crossed = floorf((float)most * s.runs * s.prefixes / s.blocks);
  return fmaxf(t_own, start + most * block + (whole ? 0.f : kPiece * (1.f + crossed)));
}

// (t, own), t > 0 and own < 256, as one number, the least of which is the choice: positive floats lie in the order of their
// bits, so the upper 24 of t's, whatever its size, and own below them.  What is cut off is 2^-15 of t.
GQA_BOTH unsigned share_rank(float t, int own) {
  unsigned bits;
  memcpy(&bits, &t, 4);
  return (bits & ~255u) | (unsigned)own;
}

}  // namespace gqa
