// attn_decode_q4.cu -- cached attention over a 4-bit KV cache (E2M1 codes, an
// E4M3 scale per 16 features, one f32 scale per cache).
//
// A few query rows meet a long stream of keys, as in attn_decode.cu, but at
// 4.5 bits an element the HBM stream carries 3.5 times the elements of a bf16
// cache: at 6.8 TB/s an SM receives about 40 elements a clock.  Every one has
// to become a 16-bit operand.  An operand tile in shared memory for tcgen05
// would cost 2 bytes written and 2 read there for each 0.56 byte of cache;
// instead the codes are converted in registers straight into the fragments of
// warp-level MMAs, whose rate (0.5 m16n8k16 a clock and SM, 128 elements) is
// three times what the stream needs, with the long side as M and the query
// rows as N:
//
//   S^T[key][row]  = sum_d K[key][d] Q[row][d]        m16 = keys, k16 = features
//   O^T[d][row]   += sum_key V[key][d] P[row][key]     m16 = features, k16 = keys
//
// e2m1 * e4m3 has 6 significant bits between 2^-10 and 2688 or is 0: exact in
// f16, so one conversion and one f16 multiplication a pair of elements give
// the operand.  Which feature or key a contraction index stands for is free as
// long as both operands agree, and each fragment is arranged so that a thread
// gets its elements from consecutive bytes of the cache's rows:
//   K: thread (g, t) = (lane / 4, lane % 4) takes features [tD/4, (t+1)D/4) of
//      keys pi(g) and pi(g + 8) of a group of 16, four features an MMA;
//   V: features [gD/8, (g+1)D/8) of the four keys pi(2t), pi(2t+1), pi(2t+8),
//      pi(2t+9); the half bytes of two keys are interleaved so that one
//      conversion gives a pair along the keys.
// S^T's fragment has rows 2t, 2t+1 as columns, and so has O^T's: the running
// maximum and the rescaling stay in the thread.  P goes from S^T's fragment to
// the second product's by two 8x8 transpositions (movmatrix).  It is rounded to
// f16: its weights are at most 2^15, so an error is 2^-11 of the weight, and
// 2^-24 below 2^-14, 2^-31 of the row's largest.  Scores, sums and O stay f32.
//
// Work: units (batch row, K/V head, block of 8*NT query rows) of 32-key tiles
// form one stream that is shared out evenly over the grid's warps, each unit
// counting kUnitCost tiles more than it has (its queries have to be loaded,
// its output written).  Each warp has a ring of its own in shared memory that
// it fills by cp.async, kStages - 1 tiles ahead, across units.  No warp waits
// for another until the end: a unit inside one warp's share is written
// directly; pieces of a unit cut between warps of a CTA are combined through
// shared memory, those of a unit cut between CTAs through the workspace by
// decode_q4_merge.  Few units of short rows go to a cluster of CTAs each
// instead, whose pieces meet in distributed shared memory (see cluster_of).
//
// Bound: long rows by the chain of instructions that turns codes into operands,
// which three warps a scheduler do not hide.  A tile of 32 keys and 128 features
// takes a warp some 570, and per SM sub-partition a conversion (F2FP) or byte
// operation takes 2 cycles, an f16 multiplication 2, an MMA 8, which overlap
// only in part; no unit is full (issue slots 60%, ALU 47%, tensor 27%).  In a
// captured graph 226.6 MB of cache, queries, outputs and tables take 45 to 46 us,
// 5.0 TB/s, 74% of a copy's rate; 8 rows of 8192 keys, 8 heads of 128, 22.4 us,
// twice their floor, of which 7 to 9 are start, tail and merge.  Short rows by
// latency: 8 rows of 2048 keys of 2 heads of 64, 2.4 MB, take 6.4 us in clusters
// (8.4 as a stream, of which 3 lie between the last warp's end and the merge's).
#include <math_constants.h>

#include <atomic>

#include "cache_ops.h"
#include "fp4.cuh"
#include "kernels.h"

namespace gqa {

namespace {

constexpr int kTK = 32;        // keys per tile
constexpr int kMaxCtas = 160;  // CTAs the workspace holds pieces for
constexpr int kUnitCost = 2;   // what a unit costs beside its tiles, in tiles (1 and 4 measure within 0.3 us of it)
// Warps a CTA uses before work goes to another SM: pieces met in a CTA cost less than those that go through the
// workspace, but a few warps on every SM convert faster than many on a few.  One row of 2048 keys, 2 K/V heads of
// 128 (as a stream): 1 warp 9.1 us, 4 8.4, 8 8.8, 12 9.6; 8192 keys: 9.4, 9.4, 9.5,
// 10.1.
constexpr int kMinWarps = 4;
constexpr int kMaxCluster = 8; // CTAs of a cluster
constexpr float kLazy = 8.f;   // the maximum moves when it would grow by more than 2^8 ...
constexpr float kOff = 7.f;    // ... and P is scaled by 2^7, so P <= 2^15 and f16's smallest step is 2^-31 of a row's largest P

template <int D, int NT>
struct Q4Cfg {
  static constexpr int kWarps = NT == 2 ? 8 : D == 128 ? 12 : 16;
  static constexpr int kStages = NT == 1 && D == 128 ? 3 : 4;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kMT = D / 16;                // 16-feature tiles of O^T
  static constexpr int kCodes = kTK * D / 2;        // bytes of a tile's K (or V) codes
  static constexpr int kSf = kTK * D / 16;          // bytes of its block scales
  static constexpr int kStage = 2 * kCodes + 2 * kSf;
  static constexpr int kRing = kStages * kStage;    // per warp
  static constexpr int kRec = NT * (kMT + 1);       // float4 of a piece per lane: per 8 rows O^T's fragments, maxima and sums
  static constexpr int kSmem = kWarps * (kRing + kRec * 512);   // rings, then a piece per warp
  static_assert(kRec * 512 <= kRing, "a warp's last piece goes into its drained ring");
  static_assert(kSmem <= 227 * 1024 - 4096, "shared memory");
};

// A thread's part of a piece: O^T fragments and, for its two columns of each
// 8-row tile, the maximum (log2 units, the same in all lanes of a column) and
// its own keys' sum.  Stored per 8 rows as kPer float4 a lane: a tile's
// fragment each, then both maxima and sums.
template <int D, int NT>
struct Piece4 {
  static constexpr int kPer = D / 16 + 1;
  float acc[NT][D / 16][4];
  float m[NT][2], l[NT][2];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[n][i][j] = 0.f;
      m[n][0] = m[n][1] = -CUDART_INF_F;
      l[n][0] = l[n][1] = 0.f;
    }
  }
  __device__ __forceinline__ void store(float4* p, int lane) const {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float4* q = p + n * kPer * 32 + lane;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) q[32 * i] = make_float4(acc[n][i][0], acc[n][i][1], acc[n][i][2], acc[n][i][3]);
      q[32 * (D / 16)] = make_float4(m[n][0], m[n][1], l[n][0], l[n][1]);
    }
  }
};

// TILES 16-feature tiles of 8 rows of a unit, combined from stored pieces with
// a running maximum.
template <int D, int TILES>
struct Combined {
  float acc[TILES][4], m[2], l[2];
  __device__ __forceinline__ void clear() {
    m[0] = m[1] = -CUDART_INF_F;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < TILES; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  }
  // a piece: its first tile at p, its maxima and sums `stat` tiles on
  __device__ __forceinline__ void add(const float4* p, int stat) {
    float4 x[TILES];
    const float4 ml = p[32 * stat];
#pragma unroll
    for (int j = 0; j < TILES; ++j) x[j] = p[32 * j];
    scale_to(0, fmaxf(m[0], ml.x));
    scale_to(1, fmaxf(m[1], ml.y));
    accumulate(ml, x);
  }
  __device__ __forceinline__ void scale_to(int c, float top) {
    const float f = m[c] == -CUDART_INF_F ? 1.f : ex2_approx(m[c] - top);   // zeros so far (or NaN, which is kept)
    m[c] = top;
    l[c] *= f;
#pragma unroll
    for (int i = 0; i < TILES; ++i) acc[i][c] *= f, acc[i][2 + c] *= f;
  }
  __device__ __forceinline__ void accumulate(const float4& ml, const float4* x) {   // ml's maxima <= m
    const float f0 = ml.x == -CUDART_INF_F ? 1.f : ex2_approx(ml.x - m[0]);
    const float f1 = ml.y == -CUDART_INF_F ? 1.f : ex2_approx(ml.y - m[1]);
    l[0] = fmaf(ml.z, f0, l[0]);
    l[1] = fmaf(ml.w, f1, l[1]);
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      acc[i][0] = fmaf(x[i].x, f0, acc[i][0]);
      acc[i][1] = fmaf(x[i].y, f1, acc[i][1]);
      acc[i][2] = fmaf(x[i].z, f0, acc[i][2]);
      acc[i][3] = fmaf(x[i].w, f1, acc[i][3]);
    }
  }
};

// Tiles of batch row b: a row without keys has one (all masked), a row with an
// invalid length none.
__device__ __forceinline__ int row_tiles(const DecodeQ4Args& a, int b, int& len) {
  len = a.cache_lens[b];
  return len < 0 || len > a.S ? 0 : len == 0 ? 1 : (len + kTK - 1) / kTK;
}

// The stream's positions: each unit has kUnitCost that stand for no tile, then
// one a tile.  All C of them (C < 2^31) are shared out: warps 0..G-1 take C / G
// each, the first C % G one more.
struct Shares {
  int q, r;
  __device__ __forceinline__ Shares(int C, int G) : q(C / G), r(C - C / G * G) {}
  __device__ __forceinline__ int begin(int w) const { return w * q + min(w, r); }
  __device__ __forceinline__ int owner(int g) const {
    const int cut = r * (q + 1);
    return g < cut ? g / (q + 1) : r + (g - cut) / q;
  }
};

// A unit of the stream.
struct Unit {
  int P;           // position of its first tile
  int nb;          // its tiles
  int b, k;        // batch row, unit within it (hkv * nrb + row block)
  int len;         // keys of the row
  __device__ __forceinline__ void next(const DecodeQ4Args& a) {
    P += nb + kUnitCost;
    if (++k < a.Hkv * a.nrb) return;
    k = 0;
    do {
      if (++b >= a.B) {             // past the last unit
        P = 0x7fffffff;
        return;
      }
      nb = row_tiles(a, b, len);
    } while (nb == 0);
  }
};

// Where slot s of a CTA's 2 * kWarps stored pieces lies: 2w is warp w's first
// piece, 2w + 1 its last, which replaces the ring.
template <int D, int NT>
__device__ __forceinline__ float4* piece_at(uint8_t* smem, int s) {
  using C = Q4Cfg<D, NT>;
  return reinterpret_cast<float4*>(s & 1 ? smem + (s >> 1) * C::kRing
                                         : smem + C::kWarps * C::kRing + (s >> 1) * C::kRec * 512);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(ok ? N : 0) : "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The low half bytes of a and the high ones of b: one three-input operation
// (two, written with masks).
__device__ __forceinline__ uint32_t half_bytes(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(r) : "r"(a), "r"(b), "n"(0x0F0F0F0F));
  return r;
}
// Both halves of a times one half of s.
__device__ __forceinline__ uint32_t hmul2_half(uint32_t a, uint32_t s, bool high) {
  const __half2 h = *reinterpret_cast<const __half2*>(&s);
  const __half2 r = __hmul2_rn(*reinterpret_cast<const __half2*>(&a), high ? __high2half2(h) : __low2half2(h));
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int N>
__device__ __forceinline__ uint32_t lds(uint32_t addr) {
  uint32_t v;
  if constexpr (N == 1) asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  else if constexpr (N == 2) asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  else asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void lds64(uint32_t addr, uint32_t* v) {
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr) : "memory");
}

// The key (of 16) that contraction row rho stands for: pairs 2t, 2t+1 are
// swapped for odd t, so that both the K loads (pairs of lanes take rho, rho+1)
// and the V loads (lanes t take 2t) meet rows of either parity -- with the
// row placement of row_at, no two lanes of a shared-memory phase share a bank.
__device__ __forceinline__ int key_of(int rho) { return rho ^ ((rho >> 1) & 1); }

// Byte offset of 16-byte chunk c of key k's codes in a tile (rows of D/2 bytes).
template <int D>
__device__ __forceinline__ int row_at(int k, int c) {
  const int s = (k >> 2) & 1;
  return D == 128 ? k * 64 + ((c ^ (2 * s)) * 16) : (k ^ s) * 32 + c * 16;
}

// The last key that rows r0 + 8n + 2t (+ 1) of a unit see, for a thread's columns of 8-row tile n: key
// len - Tq + (row % Tq); below 0: none.
__device__ __forceinline__ void row_limits(const DecodeQ4Args& a, int len, int r, int* lim) {
  const int q = r % a.Tq;
  lim[0] = len - a.Tq + q;
  lim[1] = q + 1 == a.Tq ? len - a.Tq : lim[0] + 1;
}

// How the queries reach the score MMA, whose columns are 8 query rows: their
// bf16 values (exact in f16 after scaling while 8 bits end above f16's smallest
// step: from 2^-31 of the row's largest on; below, off by half that step, 2^-39
// of the largest at most); rotated, the f16 value and the f16 remainder (22
// bits), each an MMA of its own; or rotated and at most 4 rows, the values
// in columns 0-3 and the remainders in columns 4-7 of the same MMA, added after
// it (8 rows of 8192 keys, 8 K/V heads of 128, 4 query heads each: 24.0 us, 25.9 with two MMAs).
enum { kPlain = 0, kRotated = 1, kStacked = 2 };

// A unit's query rows as B fragments; rows are scaled by a power of two so that
// their largest element lies in [2^14, 2^15); fac undoes it and applies the
// softmax scale.
template <int D, int NT, int MODE, int PARTS>
__device__ __forceinline__ void load_queries(const DecodeQ4Args& a, const Unit& w, int lane, uint32_t (*qf)[PARTS][D / 16][2],
                                             float (*fac)[2]) {
  // A thread's features of its row: [tD/4, (t+1)D/4); stacked, where lanes g and g + 4 have the same row, half of
  // them each, and then one exchanges its remainders for the other's values.
  constexpr int F = D / 4, N = MODE == kStacked ? F / 2 : F;
  const int g = lane >> 2, t = lane & 3;
  const bool upper = MODE == kStacked && g >= 4;
  const int f0 = upper ? N : 0;
  const int hkv = w.k / a.nrb, r0 = (w.k - hkv * a.nrb) * 8 * NT;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = r0 + n * 8 + (MODE == kStacked ? g & 3 : g);
    const long row = ((long)w.b * a.Hq + hkv * a.G) * a.Tq + r;
    float x[N];
    const bool live = r < a.R;
    uint32_t u[N / 2];
#pragma unroll
    for (int c = 0; c < N / 8; ++c) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (live) v = __ldg(reinterpret_cast<const uint4*>(a.q + row * D + t * F + f0) + c);
      u[4 * c] = v.x, u[4 * c + 1] = v.y, u[4 * c + 2] = v.z, u[4 * c + 3] = v.w;
    }
    if constexpr (MODE != kPlain) {
      // features t F.. pair with those of lane t ^ 2; a row at a negative position sees no key: any angle will do
      const int pos = max(w.len - a.Tq + r % a.Tq, 0);
      const float4* cs = reinterpret_cast<const float4*>(a.rope_cs + (long)pos * D + (t & 1) * F + f0);
      const float sign = t < 2 ? -1.f : 1.f;
#pragma unroll
      for (int c = 0; c < N / 4; ++c) {
        const float4 co = __ldg(cs + c), si = __ldg(cs + D / 8 + c);
        const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t y = __shfl_xor_sync(~0u, u[2 * c + i], 2);
          x[4 * c + 2 * i] = fmaf(__uint_as_float(u[2 * c + i] << 16), cc[2 * i], sign * ss[2 * i] * __uint_as_float(y << 16));
          x[4 * c + 2 * i + 1] = fmaf(__uint_as_float(u[2 * c + i] & 0xFFFF0000u), cc[2 * i + 1],
                                      sign * ss[2 * i + 1] * __uint_as_float(y & 0xFFFF0000u));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) amax = fmaxf(amax, fabsf(x[i]));
    amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
    if constexpr (MODE == kStacked) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 16));
    const int ex = (int)(__float_as_uint(amax) >> 23);          // biased exponent: 0 zero, 255 not finite
    const int sh = ex == 0 || ex == 255 ? 0 : 14 - (ex - 127);  // x * 2^sh, in two steps within f32's range
    const float s1 = __uint_as_float((uint32_t)(127 + sh / 2) << 23), s2 = __uint_as_float((uint32_t)(127 + sh - sh / 2) << 23);
    const float i1 = __uint_as_float((uint32_t)(127 - sh / 2) << 23), i2 = __uint_as_float((uint32_t)(127 - sh + sh / 2) << 23);
#pragma unroll
    for (int j = 0; j < N / 4; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float lo = x[4 * j + 2 * h] * s1 * s2, hi = x[4 * j + 2 * h + 1] * s1 * s2;
        const uint32_t v = pack_f16x2(lo, hi);
        uint32_t rest = 0;
        if constexpr (MODE != kPlain) {
          const float2 b = f16x2_to_f32(v);
          rest = pack_f16x2(lo - b.x, hi - b.y);
        }
        if constexpr (MODE == kStacked) {
          const uint32_t mine = upper ? rest : v, other = __shfl_xor_sync(~0u, upper ? v : rest, 16);
          qf[n][0][j][h] = upper ? other : mine;
          qf[n][0][j + N / 4][h] = upper ? mine : other;
        } else {
          qf[n][0][j][h] = v;
          if constexpr (MODE == kRotated) qf[n][PARTS - 1][j][h] = rest;
        }
      }
    // the columns of S^T are rows 2t and 2t+1: their factors come from the lanes that hold those rows
    const float mine = a.scale_log2 * i1 * i2;
    fac[n][0] = __shfl_sync(~0u, mine, 8 * t);
    fac[n][1] = __shfl_sync(~0u, mine, 8 * t + 4);
  }
}

// O and LSE of two rows (2t, 2t+1 of the 8 from r0 on) from their sums and
// a run of O^T's tiles: tile i holds features 2i, 2i+1 of the gD/8.. that a lane group has.  APPROX, in the merge and in
// a cluster's join, whose every instruction is waited for: quotient and logarithm to 2 ulp of f32 (0.2 us less), far
// below the bf16 step of O.
template <int D, int TILES, bool APPROX>
__device__ __forceinline__ void write_rows(const DecodeQ4Args& a, int b, int hkv, int r0, const int* lim, int tile0,
                                           const float (*acc)[4], const float* m, const float* lsum, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float l = lsum[c];
    l += __shfl_xor_sync(~0u, l, 4);
    l += __shfl_xor_sync(~0u, l, 8);
    l += __shfl_xor_sync(~0u, l, 16);
    const int r = r0 + 2 * t + c;
    if (r >= a.R) continue;
    const long row = ((long)b * a.Hq + hkv * a.G) * a.Tq + r;
    const bool empty = lim[c] < 0;      // the row sees no key
    const float inv = APPROX ? __fdividef(a.v_scale, l) : a.v_scale / l;
    if (!GQA_CHECK(row >= 0 && row < (long)a.B * a.Hq * a.Tq, a.status, a.dbg_line)) continue;
    __nv_bfloat16* o = a.o + row * D + g * (D / 8) + 2 * tile0;
    uint32_t w[TILES];
#pragma unroll
    for (int i = 0; i < TILES; ++i) w[i] = empty ? 0u : pack_bf16x2(acc[i][c] * inv, acc[i][2 + c] * inv);
    if constexpr (TILES == 1) {
      *reinterpret_cast<uint32_t*>(o) = w[0];
    } else {
#pragma unroll
      for (int i = 0; i < TILES / 4; ++i)
        reinterpret_cast<uint4*>(o)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    if (g == 0 && tile0 == 0) a.lse[row] = empty ? -CUDART_INF_F : (m[c] - kOff + (APPROX ? __log2f(l) : log2f(l))) * 0.69314718055994531f;
  }
}

template <int D, int NT, int TILES>
__device__ __forceinline__ void write_tiles(const DecodeQ4Args& a, int b, int k, int len, int n, int tile,
                                            const Combined<D, TILES>& x, int lane) {
  const int hkv = k / a.nrb, r0 = (k - hkv * a.nrb) * 8 * NT + n * 8;
  int lim[2];
  row_limits(a, len, r0 + 2 * (lane & 3), lim);
  write_rows<D, TILES, TILES == 1>(a, b, hkv, r0, lim, tile, x.acc, x.m, x.l, lane);
}

// Workspace: a header per CTA, then two pieces a CTA (kRec * 32 float4 each): 0 of
// the unit begun before the CTA's share, 1 of the one that goes on after it.
struct Q4Head {
  int b, k, len;   // the unit begun before the CTA's share
  int first, last; // CTAs that hold pieces of it; first = -1: there is none
  int pad[3];
};

// Copies tiles of a share (CLUSTER: within one unit) into a warp's ring.
template <int D, int NT, bool CLUSTER>
struct Loader {
  using C = Q4Cfg<D, NT>;
  static constexpr int kHalf = 16 * D / 2;   // bytes of 16 keys' codes
  Unit u;
  int end;             // end of the share
  bool more;           // tiles left to issue
  int tiles;           // of the unit's tiles in the share, those from the current one on
  int keys;            // keys from the current tile on
  int inpg;            // row of the tile in its page (contiguous caches: a page of S rows)
  int pidx, pbase;     // its page's block-table index; lane i holds entries pbase + i and pbase + 32 + i
  int entry[2];
  bool ok[2];          // the pages of its two 16-key halves are pages of the pool
  long off[2];         // offsets of their codes
  long head;           // offset of the K/V head in a page
  const uint8_t *kb, *vb, *ksb, *vsb;   // the lane's 16 bytes of a half tile at offset 0; its key's scales

  __device__ __forceinline__ void begin(const DecodeQ4Args& a, int lane) {
    kb = a.k4 + lane * 16;
    vb = a.v4 + lane * 16;
    ksb = a.ksf + (lane & 15) * (D / 16);
    vsb = a.vsf + (lane & 15) * (D / 16);
  }
  __device__ __forceinline__ int load_entry(const DecodeQ4Args& a, int e) const {   // only pages that hold keys are looked up
    return (long)e * a.page_size < u.len ? __ldg(a.block_table + (long)u.b * a.max_pages + e) : 0;
  }
  // the halves of a tile that begins at row inpg of block-table entry pidx (pages of 16: the second half in the next)
  __device__ __forceinline__ void to_page(const DecodeQ4Args& a) {
    const long page_bytes = (long)a.Hkv * a.page_size * (D / 2);
    const int p0 = __shfl_sync(~0u, entry[0], pidx - pbase);
    ok[0] = ok[1] = (unsigned)p0 < (unsigned)a.num_pages;
    off[0] = (ok[0] ? p0 : 0) * page_bytes + head + (long)inpg * (D / 2);
    off[1] = off[0] + kHalf;
    if (a.page_size == 16) {
      const int p1 = __shfl_sync(~0u, entry[0], pidx - pbase + 1);
      ok[1] = (unsigned)p1 < (unsigned)a.num_pages || keys <= 16;
      off[1] = (ok[1] ? p1 : 0) * page_bytes + head;
    }
  }
  // the unit's tile `tile`, if the share reaches it
  __device__ __forceinline__ void enter(const DecodeQ4Args& a, int tile, int lane) {
    tiles = min(u.nb, end - u.P) - tile;
    more = tiles > 0;
    if (!more) return;
    const int j = tile * kTK;
    keys = u.len - j;
    const int hkv = u.k / a.nrb;
    head = (long)hkv * a.page_size * (D / 2);
    // its queries, and the rotary rows of their positions, towards L2 (before the wait for the block table)
    const int r0 = (u.k - hkv * a.nrb) * 8 * NT, n = min(8 * NT, a.R - r0) * D * 2;
    const char* q = reinterpret_cast<const char*>(a.q + (((long)u.b * a.Hq + hkv * a.G) * a.Tq + r0) * D);
    if (lane * 128 < n) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + lane * 128));
    const int pos = u.len - a.Tq + (lane >> 2);
    if (a.rope_cs && (lane >> 2) < a.Tq && pos >= 0 && (lane & 3) < D / 32)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.rope_cs + (long)pos * D + (lane & 3) * 32));
    if (a.block_table) {
      pidx = pbase = j / a.page_size;
      inpg = j - pidx * a.page_size;
      entry[0] = load_entry(a, pbase + lane);
      entry[1] = load_entry(a, pbase + 32 + lane);
      to_page(a);
    } else {
      inpg = j;
      off[0] = (long)u.b * a.Hkv * a.S * (D / 2) + head + (long)j * (D / 2);
      off[1] = off[0] + kHalf;
      ok[0] = ok[1] = true;
    }
  }
  // Copies the current tile to stage s.  lane_dst: where the lane's 16 bytes of a half tile go.
  __device__ __forceinline__ void issue(const DecodeQ4Args& a, uint32_t s, int lane, uint32_t lane_dst) {
    if (more) {
      bool there = keys >= kTK;
      if (!(ok[0] && ok[1])) {
        if (keys > 0 && (threadIdx.x & 31) == 0) atomicCAS(a.status, 0, kDevBadPage);
        there = false;
      }
      // the scales' offset is an eighth of the codes': 1 byte to 8
      const long f = (lane < 16 ? off[0] : off[1]) >> 3;
      const uint32_t d = s + lane_dst, ds = s + 2 * C::kCodes + lane * (D / 16);
#ifdef GQA_DEBUG
      const long bytes = (a.block_table ? (long)a.num_pages * a.Hkv * a.page_size : (long)a.B * a.Hkv * a.S) * (D / 2);
      for (int h = 0; h < 2; ++h)
        if (min(keys - 16 * h, 16) > 0 && ok[h] &&
            !GQA_CHECK(off[h] >= 0 && off[h] + min(keys - 16 * h, 16) * (D / 2) <= bytes, a.status, a.dbg_line))
          there = ok[h] = false;
#endif
      if (there) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t *k = kb + off[h], *v = vb + off[h];
#pragma unroll
          for (int i = 0; i < kHalf; i += 512) {
            cp_async16(d + h * kHalf + i, k + i);
            cp_async16(d + C::kCodes + h * kHalf + i, v + i);
          }
        }
        cp_async_small<D / 16>(ds, ksb + f);
        cp_async_small<D / 16>(ds + C::kSf, vsb + f);
      } else {                              // the row's last tile, or a page outside the pool: zeros for what is not there
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < kHalf; i += 512) {
            const bool valid = ok[h] && 16 * h + (i + lane * 16) / (D / 2) < keys;
            const long o = valid ? off[h] + i : -(long)lane * 16;
            cp_async16(d + h * kHalf + i, kb + o, valid);
            cp_async16(d + C::kCodes + h * kHalf + i, vb + o, valid);
          }
        const bool valid = lane < keys && (lane < 16 ? ok[0] : ok[1]);
        const long o = valid ? f : -(long)(lane & 15) * (D / 16);
        cp_async_small<D / 16>(ds, ksb + o, valid);
        cp_async_small<D / 16>(ds + C::kSf, vsb + o, valid);
      }
      if (--tiles > 0) {
        keys -= kTK;
        inpg += kTK;
        off[0] += 2 * kHalf;
        off[1] += 2 * kHalf;
        if (inpg >= a.page_size) {          // not in contiguous caches: the row goes on
          pidx += a.page_size == 16 ? 2 : 1;
          inpg = 0;
          if (pidx >= pbase + 32) {
            pbase += 32;
            entry[0] = entry[1];
            entry[1] = load_entry(a, pbase + 32 + lane);
          }
          to_page(a);
        }
      } else if constexpr (CLUSTER) {
        more = false;
      } else {
        u.next(a);
        enter(a, 0, lane);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
};

constexpr int kStored = 1, kFirst = 2, kLast = 4;

__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// A float4 of CTA `rank` of the cluster, at the place that p is in this one's shared memory.
__device__ __forceinline__ float4 load_of(const float4* p, int rank) {
  uint32_t at;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

// Joins the pieces of a cluster's unit: each CTA its own, 8 rows a warp, and then
// the CTAs and warps share out the unit's 16-feature tiles and read one another's.
template <int D, int NT>
__device__ __forceinline__ void join_cluster(const DecodeQ4Args& a, const Unit& u, uint8_t* smem, const int* rec_kind, int warp,
                                             int lane) {
  using C = Q4Cfg<D, NT>;
  constexpr int kPer = Piece4<D, NT>::kPer;
  if (u.nb > 1) {          // else nothing, or written already
    const int kind = lane < 2 * C::kWarps ? rec_kind[lane] : 0;
    const unsigned slots = __ballot_sync(~0u, kind);
    float4* own = piece_at<D, NT>(smem, 0) + lane;   // what the CTA has, over warp 0's piece: a lane reads its part before
    for (int n = warp; n < NT; n += C::kWarps) {
      Combined<D, C::kMT> x;
      x.clear();
      for (unsigned left = slots; left; left &= left - 1)
        x.add(piece_at<D, NT>(smem, __ffs(left) - 1) + n * kPer * 32 + lane, C::kMT);
#pragma unroll
      for (int j = 0; j < C::kMT; ++j) own[(n * kPer + j) * 32] = make_float4(x.acc[j][0], x.acc[j][1], x.acc[j][2], x.acc[j][3]);
      own[(n * kPer + C::kMT) * 32] = make_float4(x.m[0], x.m[1], x.l[0], x.l[1]);
    }
    cluster_barrier();
    for (int tile = warp * a.cluster + blockIdx.x % a.cluster; tile < NT * C::kMT; tile += C::kWarps * a.cluster) {
      const int n = tile / C::kMT, i = tile % C::kMT;
      float4 y[kMaxCluster], ml[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < a.cluster) {
          y[r] = load_of(own + (n * kPer + i) * 32, r);
          ml[r] = load_of(own + (n * kPer + C::kMT) * 32, r);
        }
      Combined<D, 1> x;
      x.clear();
      float top[2] = {x.m[0], x.m[1]};
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < a.cluster) top[0] = fmaxf(top[0], ml[r].x), top[1] = fmaxf(top[1], ml[r].y);
      x.scale_to(0, top[0]);
      x.scale_to(1, top[1]);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < a.cluster) x.accumulate(ml[r], &y[r]);
      write_tiles<D, NT>(a, u.b, u.k, u.len, n, i, x, lane);
    }
    cluster_barrier();     // no CTA leaves while its pieces are read
  }
}

template <int D, int NT, int MODE, bool CLUSTER>
__global__ void __launch_bounds__(Q4Cfg<D, NT>::kThreads, 1) decode_q4_kernel(const DecodeQ4Args a) {
  using C = Q4Cfg<D, NT>;
  constexpr int PARTS = MODE == kRotated ? 2 : 1;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int sums[C::kWarps];
  __shared__ int prefix[C::kThreads];
  __shared__ Unit rec_unit[2 * C::kWarps];   // unit of each stored piece
  __shared__ int rec_kind[2 * C::kWarps];    // kStored, with kFirst / kLast if it has the unit's first / last tile; 0: none
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(~0u, tid >> 5, 0);   // the same in a warp, told so
  const int g = lane >> 2, t = lane & 3;
  const int upb = a.Hkv * a.nrb;

  griddep_wait();                            // launched while the kernel before drains
  griddep_launch();                          // the merge waits for this grid's end in any case
  // a warp's own entries, by the thread that sets them: in a cluster no barrier stands between this and the pieces
  if (lane == 0) rec_kind[2 * warp] = rec_kind[2 * warp + 1] = 0;
  // The positions of all units, and the batch row that holds the share's first:
  // inclusive sums over the rows, kThreads rows at a time (more rows: a pass for the total first).
  int total = 0, Wn = 0, wpc = 1, v0 = 0, v1 = 0, before = 0;
  Unit cu{0, 0, -1, 0, 0};
  auto positions = [&](int b) {
    int len;
    const int nb = row_tiles(a, b, len);
    return nb ? nb + kUnitCost : 0;
  };
  auto take_share = [&](int sum) {
    total = sum * upb;
    wpc = min(max((total + (int)gridDim.x - 1) / (int)gridDim.x, kMinWarps), C::kWarps);
    Wn = min(total, (int)gridDim.x * wpc);
    const int gw = blockIdx.x * wpc + warp;
    if (warp < wpc && gw < Wn) {
      const Shares sh(total, Wn);
      v0 = sh.begin(gw), v1 = sh.begin(gw + 1);
    }
  };
  if constexpr (CLUSTER) {
    const int unit = blockIdx.x / a.cluster;
    cu.b = unit / upb;
    cu.k = unit - cu.b * upb;
    cu.nb = row_tiles(a, cu.b, cu.len);
    if (cu.nb == 0 && cu.k == 0 && tid == 0) atomicCAS(a.status, 0, kDevBadSeqlens);
    // neighbouring shares go to different CTAs, so that few tiles still use all of them
    const int gw = warp * a.cluster + blockIdx.x - unit * a.cluster;
    Wn = min(cu.nb, a.cluster * C::kWarps);
    if (gw < Wn) {
      const Shares sh(cu.nb, Wn);
      v0 = sh.begin(gw), v1 = sh.begin(gw + 1);
    }
  }
  if (!CLUSTER && a.B > C::kThreads) {
    int mine = 0;
    for (int b = tid; b < a.B; b += C::kThreads) mine += positions(b);
    mine = __reduce_add_sync(~0u, mine);
    if (lane == 0) sums[warp] = mine;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) all += sums[w];
    take_share(all);
  }
  for (int b0 = 0; !CLUSTER && b0 < a.B; b0 += C::kThreads) {
    int inc = 0;
    if (b0 + tid < a.B) {
      inc = positions(b0 + tid);
      if (inc == 0 && blockIdx.x == 0) atomicCAS(a.status, 0, kDevBadSeqlens);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(~0u, inc, d);
      if (lane >= d) inc += x;
    }
    if (b0 > 0 || a.B > C::kThreads) __syncthreads();   // the sums before are read
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
      if (w < warp) inc += sums[w];
      all += sums[w];
    }
    prefix[tid] = inc;
    __syncthreads();
    if (a.B <= C::kThreads) take_share(all);
    if (v0 < v1 && cu.b < 0 && v0 < (before + all) * upb) {
      const int x = v0 - before * upb;   // row i of these: prefix[i - 1] * upb <= x < prefix[i] * upb
      int lo = 0, hi = min(C::kThreads, a.B - b0) - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] * upb > x) hi = mid;
        else lo = mid + 1;
      }
      cu.b = b0 + lo;
      cu.nb = row_tiles(a, cu.b, cu.len);
      const int P = (before + (lo ? prefix[lo - 1] : 0)) * upb;
      cu.k = (v0 - P) / (cu.nb + kUnitCost);
      cu.P = P + cu.k * (cu.nb + kUnitCost) + kUnitCost;
    }
    before += all;
  }

  // all of a warp's lanes found the same: told so, the loops below need no divergence handling
  v0 = __shfl_sync(~0u, v0, 0), v1 = __shfl_sync(~0u, v1, 0);
  cu.P = __shfl_sync(~0u, cu.P, 0), cu.nb = __shfl_sync(~0u, cu.nb, 0), cu.b = __shfl_sync(~0u, cu.b, 0);
  cu.k = __shfl_sync(~0u, cu.k, 0), cu.len = __shfl_sync(~0u, cu.len, 0);
  // the share's tiles [ct, te) of its first unit
  int ct = max(v0 - cu.P, 0), te = min(cu.nb, v1 - cu.P);
  if (v0 < v1 && ct < te) {
    const uint32_t ring = smem_u32(smem + warp * C::kRing);
    Loader<D, NT, CLUSTER> ld;
    ld.u = cu;
    ld.end = v1;
    ld.begin(a, lane);
    ld.enter(a, ct, lane);
    const uint32_t lane_dst = row_at<D>(lane / (D / 32), lane % (D / 32));
    // the lane's bytes in a stage: of K rows pi(g) (+ 8, 16, 24) and of V rows pi(2t), pi(2t + 1)
    const uint32_t k_at = row_at<D>(key_of(g), D == 128 ? t : 0) + (D == 128 ? 0 : 8 * t);
    const uint32_t ks_at = 2 * C::kCodes + key_of(g) * (D / 16) + (D == 128 ? 2 * t : t);
    uint32_t v_at[2], vs_at[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int key = key_of(2 * t + e);
      v_at[e] = C::kCodes + row_at<D>(key, D == 128 ? g >> 1 : 0) + (D == 128 ? 8 * (g & 1) : 4 * g);
      vs_at[e] = 2 * C::kCodes + C::kSf + key * (D / 16) + (D == 128 ? g : g >> 1);
    }
    Piece4<D, NT> p;
    uint32_t qf[NT][PARTS][D / 16][2];
    float fac[NT][2], bias[NT][2];
    int lim[NT][2];                      // last key each of the thread's rows sees
    int r0 = 0;
    uint32_t s = ring;                   // stage of the current tile, and the one to fill
    uint32_t fill = ring;
    int ta = ct;                         // the current piece: unit cu's tiles [ta, te)
    bool fresh = true;
    // a round issues the copies of the tile kStages - 1 ahead, then takes a tile
    for (int lead = C::kStages - 1;;) {
      if (fresh && lead < C::kStages - 1) {   // before all copies but the first tile's: these loads would queue behind them
        load_queries<D, NT, MODE, PARTS>(a, cu, lane, qf, fac);
        p.clear();
        r0 = (cu.k % a.nrb) * 8 * NT;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          row_limits(a, cu.len, r0 + n * 8 + 2 * t, lim[n]);
          bias[n][0] = bias[n][1] = CUDART_INF_F;     // kOff - m: any visible score makes the maximum move
        }
        fresh = false;
      }
      __syncwarp();                      // the stage to fill is read
      ld.issue(a, fill, lane, lane_dst);
      fill = fill == ring + (C::kStages - 1) * C::kStage ? ring : fill + C::kStage;
      if (lead > 0) {
        --lead;
        continue;
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 1) : "memory");
      __syncwarp();                      // every lane's copies of tile i have landed
      const int j0 = ct * kTK;
      {
        // S^T of both 16-key groups
        float sc[2][NT][4];
#pragma unroll
        for (int G = 0; G < 2; ++G) {
#pragma unroll
          for (int n = 0; n < NT; ++n) sc[G][n][0] = sc[G][n][1] = sc[G][n][2] = sc[G][n][3] = 0.f;
          // row_at's swizzle repeats every 8 keys: the rows 8 and 16 further on are at fixed distances
          const uint32_t ka = s + k_at + G * 16 * (D / 2), kb = ka + 8 * (D / 2);
          const uint32_t fa_at = s + ks_at + G * D, fb_at = fa_at + D / 2;
          uint32_t wa[D / 32], wb[D / 32];
          uint32_t sa, sb;               // block scales as f16 pairs: (first, second) 16 features, D = 64: one
          if constexpr (D == 128) {
            const uint4 u = ld_shared_v4(ka), v = ld_shared_v4(kb);
            wa[0] = u.x, wa[1] = u.y, wa[2] = u.z, wa[3] = u.w;
            wb[0] = v.x, wb[1] = v.y, wb[2] = v.z, wb[3] = v.w;
            sa = e4m3x2_to_f16(lds<2>(fa_at));
            sb = e4m3x2_to_f16(lds<2>(fb_at));
          } else {
            lds64(ka, wa);
            lds64(kb, wb);
            sa = e4m3x2_to_f16(lds<1>(fa_at));
            sb = e4m3x2_to_f16(lds<1>(fb_at));
          }
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {     // 8 features: two MMAs
            uint32_t ra[4], rb[4];
            e2m1x8_to_f16(wa[w], ra);
            e2m1x8_to_f16(wb[w], rb);
            const bool high = D == 128 && w >= 2;
#pragma unroll
            for (int i = 0; i < 4; ++i) ra[i] = hmul2_half(ra[i], sa, high), rb[i] = hmul2_half(rb[i], sb, high);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int q = 0; q < PARTS; ++q)
                  mma_f16(sc[G][n], ra[2 * i], rb[2 * i], ra[2 * i + 1], rb[2 * i + 1], qf[n][q][2 * w + i][0],
                          qf[n][q][2 * w + i][1]);
          }
        }
        if constexpr (MODE == kStacked) {   // rows' values and remainders: columns c and c + 4 are lanes t and t ^ 2
#pragma unroll
          for (int G = 0; G < 2; ++G)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[G][0][i] += __shfl_xor_sync(~0u, sc[G][0][i], 2);
        }
        // y = s - m + kOff in log2 units, hidden keys out; the maximum moves when some y is above kOff + kLazy
        const bool edge = j0 + kTK > cu.len - a.Tq + 1;   // some key of the tile is hidden from some row
        float y[2][NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int G = 0; G < 2; ++G)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[G][n][i] = fmaf(sc[G][n][i], fac[n][i & 1], bias[n][i & 1]);
        if (edge) {
          const int key = j0 + key_of(g);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int G = 0; G < 2; ++G)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (key + 16 * G + 8 * (i >> 1) > lim[n][i & 1]) y[G][n][i] = sc[G][n][i] = -CUDART_INF_F;
        }
        float top = -CUDART_INF_F;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int G = 0; G < 2; ++G) top = max3f(max3f(top, y[G][n][0], y[G][n][1]), y[G][n][2], y[G][n][3]);
        if (__any_sync(~0u, top > kOff + kLazy)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float mx = -CUDART_INF_F;
#pragma unroll
              for (int G = 0; G < 2; ++G)
#pragma unroll
                for (int h = 0; h < 2; ++h) {   // a hidden key's score is -infinity whatever the factor's sign
                  const float x = sc[G][n][2 * h + c];
                  mx = fmaxf(mx, x == -CUDART_INF_F ? x : x * fac[n][c]);
                }
              mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
              mx = fmaxf(mx, p.m[n][c]);
              const float f = p.m[n][c] == -CUDART_INF_F ? 1.f : ex2_approx(p.m[n][c] - mx);
              p.m[n][c] = mx;
              bias[n][c] = kOff - mx;
              p.l[n][c] *= f;
#pragma unroll
              for (int i = 0; i < C::kMT; ++i) p.acc[n][i][c] *= f, p.acc[n][i][2 + c] *= f;
#pragma unroll
              for (int G = 0; G < 2; ++G)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float x = sc[G][n][2 * h + c];
                  y[G][n][2 * h + c] = x == -CUDART_INF_F ? x : fmaf(x, fac[n][c], bias[n][c]);
                }
            }
        }
        // P, its sums, and its fragments
        uint32_t pf[2][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int G = 0; G < 2; ++G) {
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[i] = ex2_approx(y[G][n][i]);
              p.l[n][i & 1] += x[i];
            }
            pf[G][n][0] = transpose8x8(pack_f16x2(x[0], x[1]));
            pf[G][n][1] = transpose8x8(pack_f16x2(x[2], x[3]));
          }
        // O^T: the block scales of the thread's keys pi(2t), pi(2t+1), pi(2t+8), pi(2t+9) of each group
        uint32_t vsf[2][4];
#pragma unroll
        for (int G = 0; G < 2; ++G)
#pragma unroll
          for (int i = 0; i < 4; ++i) vsf[G][i] = lds<1>(s + vs_at[i & 1] + (16 * G + 8 * (i >> 1)) * (D / 16));
        if (edge && a.Tq > 1) {
          // a NaN block at a key that some rows do not see: 0 * NaN would reach them through the MMA, so it is
          // taken out here and put into the rows that do see it
          bool bad = false;
#pragma unroll
          for (int G = 0; G < 2; ++G)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((vsf[G][i] & 0x7f) == 0x7f) bad = true, vsf[G][i] = 0;
          if (__any_sync(~0u, bad)) {
#pragma unroll 1
            for (int k = 0; k < kTK; ++k) {
              const uint32_t v = lds<1>(s + 2 * C::kCodes + C::kSf + k * (D / 16) + (D == 128 ? g : g >> 1));
              if ((v & 0x7f) != 0x7f) continue;
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  if (j0 + k <= lim[n][c]) {
#pragma unroll
                    for (int i = 0; i < C::kMT; ++i) p.acc[n][i][c] = p.acc[n][i][2 + c] = CUDART_NAN_F;
                  }
            }
          }
        }
#pragma unroll
        for (int G = 0; G < 2; ++G) {
          constexpr int VW = D / 64;                 // words of a thread's features of one key
          uint32_t w[4][VW];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t at_v = s + v_at[i & 1] + (16 * G + 8 * (i >> 1)) * (D / 2);
            if constexpr (D == 128) lds64(at_v, w[i]);
            else w[i][0] = lds<4>(at_v);
          }
          const uint32_t* sb = vsf[G];
          const uint32_t f01 = e4m3x2_to_f16(__byte_perm(sb[0], sb[1], 0x0040)), f23 = e4m3x2_to_f16(__byte_perm(sb[2], sb[3], 0x0040));
#pragma unroll
          for (int v = 0; v < VW; ++v) {
            // half bytes of two keys side by side: byte i of e.. is feature 2i of both, of o.. feature 2i+1
            uint32_t e01[4], o01[4], e23[4], o23[4];
            e2m1x8_to_f16(half_bytes(w[0][v], w[1][v] << 4), e01);
            e2m1x8_to_f16(half_bytes(w[0][v] >> 4, w[1][v]), o01);
            e2m1x8_to_f16(half_bytes(w[2][v], w[3][v] << 4), e23);
            e2m1x8_to_f16(half_bytes(w[2][v] >> 4, w[3][v]), o23);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t a0 = hmul2_u(e01[i], f01), a1 = hmul2_u(o01[i], f01);
              const uint32_t a2 = hmul2_u(e23[i], f23), a3 = hmul2_u(o23[i], f23);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16(p.acc[n][4 * v + i], a0, a1, a2, a3, pf[G][n][0], pf[G][n][1]);
            }
          }
        }
        s = s == ring + (C::kStages - 1) * C::kStage ? ring : s + C::kStage;
      }
      if (++ct < te) continue;

      // the piece is done: written if it is its whole unit, else stored
      if (ta == 0 && te == cu.nb) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
          write_rows<D, C::kMT, false>(a, cu.b, cu.k / a.nrb, r0 + 8 * n, lim[n], 0, p.acc[n], p.m[n], p.l[n], lane);
      } else {
        const int slot = 2 * warp + (ta == 0);   // a unit begun before the share, or continued after it
        if (slot & 1) {   // the share ends here: no copy is in flight, and every lane has read the last tile
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          __syncwarp();
        }
        p.store(piece_at<D, NT>(smem, slot), lane);
        if (lane == 0) {
          rec_unit[slot] = cu;
          rec_kind[slot] = kStored | (ta == 0 ? kFirst : 0) | (te == cu.nb ? kLast : 0);
        }
      }
      if constexpr (CLUSTER) break;
      cu.next(a);
      fresh = true;
      ct = ta = 0;
      te = min(cu.nb, v1 - cu.P);
      if (te <= 0) break;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  __syncthreads();
  if constexpr (CLUSTER) {
    join_cluster<D, NT>(a, cu, smem, rec_kind, warp, lane);
    return;
  }

  // Combine the stored pieces of each unit, in stream order: a warp per 8 rows of a unit (shared out by its feature
  // tiles among more warps, a unit's chain of dependent steps is as long, and there are more of them)
  static_assert(2 * C::kWarps <= 32, "a lane per slot");   // lane s looks after slot s
  const int kind = lane < 2 * C::kWarps ? rec_kind[lane] : 0;
  const unsigned taken = __ballot_sync(~0u, kind);
  const unsigned earlier = taken & ((1u << lane) - 1);
  const int my_P = kind ? rec_unit[lane].P : -1;
  const int prev_P = __shfl_sync(~0u, my_P, earlier ? 31 - __clz(earlier) : lane);
  const unsigned begins = __ballot_sync(~0u, kind && (!earlier || prev_P != my_P));
  Q4Head* heads = static_cast<Q4Head*>(a.ws);
  float4* pieces = reinterpret_cast<float4*>(heads + kMaxCtas);
  const int unit_of = begins >> lane & 1 ? __popc(begins & ((1u << lane) - 1)) : -1;   // the unit that begins with the lane's slot
#pragma unroll 1
  for (int item = warp; item < __popc(begins) * NT; item += C::kWarps) {
    const int n = item % NT, s0 = __ffs(__ballot_sync(~0u, unit_of == item / NT)) - 1;
    const unsigned later = begins & ~((2u << s0) - 1);
    const unsigned slots = taken & ~((1u << s0) - 1) & (later ? (later & -later) - 1 : ~0u);   // up to the next unit's
    const bool first = __shfl_sync(~0u, kind, s0) & kFirst, last = __shfl_sync(~0u, kind, 31 - __clz(slots)) & kLast;
    Combined<D, C::kMT> x;
    x.clear();
    for (unsigned left = slots; left; left &= left - 1)
      x.add(piece_at<D, NT>(smem, __ffs(left) - 1) + n * Piece4<D, NT>::kPer * 32 + lane, C::kMT);
    if (first && last) {
      const Unit u = rec_unit[s0];
      write_tiles<D, NT>(a, u.b, u.k, u.len, n, 0, x, lane);
    } else {
      float4* q = pieces + ((long)blockIdx.x * 2 + first) * C::kRec * 32 + n * Piece4<D, NT>::kPer * 32 + lane;
#pragma unroll
      for (int j = 0; j < C::kMT; ++j) q[32 * j] = make_float4(x.acc[j][0], x.acc[j][1], x.acc[j][2], x.acc[j][3]);
      q[32 * C::kMT] = make_float4(x.m[0], x.m[1], x.l[0], x.l[1]);
    }
  }
  if (tid == C::kThreads - 32) {   // of the warp that gets an item last
    Q4Head head{};
    head.first = -1;
    const int s0 = __ffs(begins) - 1;
    if (begins && !(rec_kind[s0] & kFirst)) {
      const Unit u = rec_unit[s0];
      const Shares sh(total, Wn);
      head = Q4Head{u.b, u.k, u.len, sh.owner(u.P) / wpc, sh.owner(u.P + u.nb - 1) / wpc, {}};
    }
    heads[blockIdx.x] = head;
  }
}

// Units cut between CTAs.  A warp combines a 16-feature tile of up to
// kMergePieces pieces (their loads in flight together); with more pieces, 2, 4,
// 8 or 16 groups of warps share them and meet in shared memory, and the tiles
// go to several blocks: those of the CTAs from the second on that hold a piece
// (there are more of them than blocks needed).  Beyond 64 pieces, where there
// are no more groups to take, a warp has up to 10, in two rounds of loads.  One row of 8192 keys, 2 K/V
// heads of 128: 9.4 us; one block a unit took 4.8 more.
constexpr int kMergeLog = 4, kMergeWarps = 1 << kMergeLog;
constexpr int kMergePieces = 4;

template <int D, int NT>
__global__ void __launch_bounds__(kMergeWarps * 32) decode_q4_merge(const DecodeQ4Args a) {
  using C = Q4Cfg<D, NT>;
  constexpr int kTilesLog = NT * C::kMT == 16 ? 4 : NT * C::kMT == 8 ? 3 : 2, kPer = Piece4<D, NT>::kPer;
  __shared__ float4 part[kMergeWarps][2][32];   // per warp: a tile's fragment, maxima and sums
  griddep_wait();
  griddep_launch();
  const Q4Head* heads = static_cast<const Q4Head*>(a.ws);
  const float4* pieces = reinterpret_cast<const float4*>(heads + kMaxCtas);
  const Q4Head h = heads[blockIdx.x];
  if (h.first < 0) return;
  const int count = h.last - h.first + 1;
  const int groups_log = min(count <= kMergePieces ? 0 : 32 - __clz((count - 1) / kMergePieces), kMergeLog);
  const int tiles_log = min(kMergeLog - groups_log, kTilesLog), groups = 1 << groups_log;
  const int block = blockIdx.x - h.first - 1;
  if (block >> (kTilesLog - tiles_log)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tt = warp & ((1 << tiles_log) - 1), group = warp >> tiles_log;
  const int tile = (block << tiles_log) + tt, n = tile / C::kMT, i = tile % C::kMT;
  Combined<D, 1> x;
  x.clear();
  constexpr int kBatch = 8;
  if (group < groups)
    for (int j0 = group; j0 < count; j0 += kBatch * groups) {   // up to kBatch pieces' loads in flight
      float4 y[kBatch], ml[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int j = j0 + u * groups;
        if (j < count) {
          const float4* p = pieces + (((long)(h.first + j) * 2 + (j == 0)) * C::kRec + n * kPer) * 32 + lane;
          y[u] = p[32 * i];
          ml[u] = p[32 * C::kMT];
        }
      }
      float top[2] = {x.m[0], x.m[1]};
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (j0 + u * groups < count) top[0] = fmaxf(top[0], ml[u].x), top[1] = fmaxf(top[1], ml[u].y);
      x.scale_to(0, top[0]);
      x.scale_to(1, top[1]);
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (j0 + u * groups < count) x.accumulate(ml[u], &y[u]);
    }
  if (groups > 1) {
    part[warp][0][lane] = make_float4(x.acc[0][0], x.acc[0][1], x.acc[0][2], x.acc[0][3]);
    part[warp][1][lane] = make_float4(x.m[0], x.m[1], x.l[0], x.l[1]);
    __syncthreads();
  }
  if (group > 0) return;
#pragma unroll 3
  for (int q = 1; q < groups; ++q) x.add(&part[(q << tiles_log) + tt][0][lane], 1);
  write_tiles<D, NT>(a, h.b, h.k, h.len, n, i, x, lane);
}

constexpr int kMaxDevices = 64;
int device() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && dev < kMaxDevices ? dev : -1;
}

// The kernel's shared memory allowed, once per device: the call costs a microsecond.
template <int D, int NT, int MODE, bool CLUSTER>
cudaError_t allow_smem(int dev) {
  static std::atomic<unsigned long long> done{0};
  const unsigned long long bit = 1ull << dev;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(decode_q4_kernel<D, NT, MODE, CLUSTER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Q4Cfg<D, NT>::kSmem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Clusters of c CTAs that run at once (a cluster's SMs are of one part of the chip, so fewer than SMs / c).
template <int D, int NT, int MODE>
int clusters_at_once(int dev, int c) {
  static std::atomic<int> known[kMaxDevices][kMaxCluster + 1];   // one more than that; 0: not asked yet
  int n = known[dev][c].load(std::memory_order_relaxed);
  if (n == 0) {
    if (allow_smem<D, NT, MODE, true>(dev) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(Q4Cfg<D, NT>::kThreads);
    cfg.dynamicSmemBytes = Q4Cfg<D, NT>::kSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = c;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, decode_q4_kernel<D, NT, MODE, true>, &cfg) != cudaSuccess || n < 0) n = 0;
    known[dev][c].store(++n, std::memory_order_relaxed);
  }
  return n - 1;
}

// CTAs of a unit's cluster, 0: the units are one stream.  A cluster each saves
// the scan of the lengths, the second launch and the way through the workspace,
// 2.5 us, but gives a unit the same share whatever its row's length, and leaves
// SMs idle: taken where all clusters run at once, a row of S keys is at most 3
// tiles a warp, and at most 2 more than its part of the stream.  8 K/V heads of
// 128, 4 queries each, clusters against the stream: 1 row of 1024 keys 6.0 us,
// 8.4; 4 rows of 2048 8.3, 11.3; 16 of 1024 9.1, 11.4.  2 heads: 1 row of 2048
// keys 6.7, 8.0; of 4096 8.2, 8.6; of 8192 9.8, 9.3.
template <int D, int NT, int MODE>
int cluster_of(const DecodeQ4Args& a, int dev, int ctas) {
  constexpr int kWarps = Q4Cfg<D, NT>::kWarps;
  const long units = (long)a.B * a.Hkv * a.nrb, tiles = ((long)a.S + kTK - 1) / kTK;
  if (units > ctas || tiles > 3 * kMaxCluster * kWarps) return 0;
  for (int c = kMaxCluster; c > 0; --c) {
    if (units * c > ctas || units > clusters_at_once<D, NT, MODE>(dev, c)) continue;
    const float own = (float)tiles / (float)(kWarps * c), even = (float)(units * tiles) / (float)(kWarps * ctas);
    return own <= 3.f && own - even <= 2.f ? c : 0;
  }
  return 0;
}

template <int D, int NT, int MODE, bool CLUSTER>
cudaError_t run_kernel(const DecodeQ4Args& a, int dev, int ctas, cudaStream_t stream) {
  cudaError_t e = allow_smem<D, NT, MODE, CLUSTER>(dev);
  if (e != cudaSuccess) return e;
  prof_begin(kProfDecode, stream);
  e = launch_programmatic_clusters(decode_q4_kernel<D, NT, MODE, CLUSTER>, CLUSTER ? a.cluster : 1, dim3(ctas),
                                   dim3(Q4Cfg<D, NT>::kThreads), Q4Cfg<D, NT>::kSmem, stream, a);
  prof_end(stream);
  return e;
}

template <int D, int NT, int MODE>
cudaError_t run(DecodeQ4Args a, int ctas, cudaStream_t stream) {
  const int dev = device();
  if (dev < 0) return cudaErrorInvalidDevice;
  a.cluster = cluster_of<D, NT, MODE>(a, dev, ctas);
  if (a.cluster) return run_kernel<D, NT, MODE, true>(a, dev, a.B * a.Hkv * a.nrb * a.cluster, stream);
  cudaError_t e = run_kernel<D, NT, MODE, false>(a, dev, ctas, stream);
  if (e != cudaSuccess) return e;
  prof_begin(kProfDecodeMerge, stream);
  e = launch_programmatic(decode_q4_merge<D, NT>, dim3(ctas), dim3(kMergeWarps * 32), 0, stream, a);
  prof_end(stream);
  return e;
}

}  // namespace

// Rows go in blocks of 16 (two 8-row tiles, one conversion of the cache for
// both) unless one tile of 8 holds them all: 8 rows of 8192 keys, 8 K/V heads,
// blocks of 16 against 8: 16 query rows a head 27.1 us against 33.2 (D = 64:
// 20.3, 23.0), 8 query rows 26.9 against 22.3 (20.3, 16.2).
static int row_tiles_of(int R) { return R <= 8 ? 1 : 2; }

size_t decode_q4_ws_bytes(int, int Hq, int Hkv, int Tq, int, int D) {
  const int nt = row_tiles_of(Hq / Hkv * Tq);
  return sizeof(Q4Head) * kMaxCtas + (size_t)kMaxCtas * 2 * nt * (D / 16 + 1) * 512;
}

template <int D>
static cudaError_t run_as(const DecodeQ4Args& a, int nt, int mode, int ctas, cudaStream_t stream) {
  if (mode == kStacked) return run<D, 1, kStacked>(a, ctas, stream);
  if (nt == 1) return mode ? run<D, 1, kRotated>(a, ctas, stream) : run<D, 1, kPlain>(a, ctas, stream);
  return mode ? run<D, 2, kRotated>(a, ctas, stream) : run<D, 2, kPlain>(a, ctas, stream);
}

cudaError_t launch_decode_q4(const DecodeQ4Args& args, int sms, cudaStream_t stream) {
  DecodeQ4Args a = args;
  const int nt = row_tiles_of(a.R);
  a.nrb = (a.R + 8 * nt - 1) / (8 * nt);
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  const int mode = !a.rope_cs ? kPlain : a.R <= 4 ? kStacked : kRotated;
  return a.D == 128 ? run_as<128>(a, nt, mode, ctas, stream) : run_as<64>(a, nt, mode, ctas, stream);
}

}  // namespace gqa
