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
// the second product's by two 8x8 transpositions (movmatrix).
//
// Work: units (batch row, K/V head, block of 8*NT query rows) of 32-key tiles
// form one stream; warp w of all W takes tiles [wC/W, (w+1)C/W), each with a
// ring of its own in shared memory that it fills by cp.async, kStages - 1
// tiles ahead, across units.  No warp waits for another until the end: a unit
// inside one warp's share is written directly; pieces of a unit cut between
// warps of a CTA are combined through shared memory, those of a unit cut
// between CTAs through the workspace by decode_q4_merge.
#include <math_constants.h>

#include "cache_ops.h"
#include "fp4.cuh"
#include "kernels.h"

namespace gqa {

namespace {

constexpr int kTK = 32;        // keys per tile
constexpr int kMaxCtas = 160;  // CTAs the workspace holds pieces for
constexpr float kLazy = 8.f;   // the maximum moves when it would grow by more than 2^8 ...
constexpr float kOff = 7.f;    // ... and P is scaled by 2^7, so P <= 2^15 and f16's smallest step is 2^-31 of a row's largest P

template <int D, int NT>
struct Q4Cfg {
  static constexpr int kWarps = 8;
  static constexpr int kStages = 4;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kMT = D / 16;                // 16-feature tiles of O^T
  static constexpr int kCodes = kTK * D / 2;        // bytes of a tile's K (or V) codes
  static constexpr int kSf = kTK * D / 16;          // bytes of its block scales
  static constexpr int kStage = 2 * kCodes + 2 * kSf;
  static constexpr int kRing = kStages * kStage;    // per warp
  static constexpr int kRec = NT * (kMT * 4 + 4);   // f32 of a piece per lane: O^T fragment, maxima, sums
  static constexpr int kSmem = kWarps * (kRing + kRec * 128);   // rings, then a piece per warp
  static_assert(kRec * 128 <= kRing, "a warp's last piece goes into its drained ring");
  static_assert(kSmem <= 227 * 1024 - 2048, "shared memory");
};

// A thread's part of a piece: O^T fragments and, for its two columns of each
// 8-row tile, the maximum (log2 units, the same in all lanes of a column) and
// its own keys' sum.
template <int D, int NT>
struct Piece4 {
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
  // [register][lane] f32: coalesced in global memory, free of conflicts in shared memory
  __device__ __forceinline__ void store(float* p, int lane) const {
    int r = 0;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) p[32 * r++ + lane] = acc[n][i][j];
#pragma unroll
      for (int c = 0; c < 2; ++c) p[32 * r++ + lane] = m[n][c];
#pragma unroll
      for (int c = 0; c < 2; ++c) p[32 * r++ + lane] = l[n][c];
    }
  }
  // combine with a stored piece of the same unit
  __device__ __forceinline__ void add(const float* p, int lane) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float* q = p + n * (D / 16 * 4 + 4) * 32 + lane;
      float a[2], b[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float m2 = q[(D / 16 * 4 + c) * 32], l2 = q[(D / 16 * 4 + 2 + c) * 32];
        const float mn = fmaxf(m[n][c], m2);
        a[c] = m[n][c] == -CUDART_INF_F ? 0.f : ex2_approx(m[n][c] - mn);
        b[c] = m2 == -CUDART_INF_F ? 0.f : ex2_approx(m2 - mn);
        // a NaN sum must survive a piece whose maximum is -infinity
        l[n][c] = (m[n][c] == -CUDART_INF_F ? l[n][c] : l[n][c] * a[c]) + (m2 == -CUDART_INF_F ? l2 : l2 * b[c]);
        if (m[n][c] == -CUDART_INF_F) a[c] = 1.f;
        if (m2 == -CUDART_INF_F) b[c] = 1.f;
        m[n][c] = mn;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[n][i][j] = acc[n][i][j] * a[j & 1] + q[(i * 4 + j) * 32] * b[j & 1];
    }
  }
};

// Where slot s of a CTA's 2 * kWarps stored pieces lies: 2w is warp w's first
// piece, 2w + 1 its last, which replaces the ring.
template <int D, int NT>
__device__ __forceinline__ float* piece_at(uint8_t* smem, int s) {
  using C = Q4Cfg<D, NT>;
  return reinterpret_cast<float*>(s & 1 ? smem + (s >> 1) * C::kRing
                                        : smem + C::kWarps * C::kRing + (s >> 1) * C::kRec * 128);
}

// Tiles of batch row b: a row without keys has one (all masked), a row with an
// invalid length none.
__device__ __forceinline__ int row_tiles(const DecodeQ4Args& a, int b, int& len) {
  len = a.cache_lens[b];
  return len < 0 || len > a.S ? 0 : len == 0 ? 1 : (len + kTK - 1) / kTK;
}

// The share of all tiles: warps 0..G-1 of the grid, warp w takes [wC/G, (w+1)C/G).
__device__ __forceinline__ int owner_of(long g, long C, int G) { return (int)(((g + 1) * G - 1) / C); }

// A position in the stream.
struct Walk {
  long g;          // stream index of the tile
  long Pu;         // stream index of its unit's first tile
  int b, k;        // batch row, unit within it (hkv * nrb + row block)
  int len, nb;     // keys of the row, tiles per unit
  __device__ __forceinline__ int tile() const { return (int)(g - Pu); }
  __device__ __forceinline__ void next(const DecodeQ4Args& a, long end) {
    ++g;
    if (g - Pu < nb || g >= end) return;
    Pu += nb;
    if (++k < a.Hkv * a.nrb) return;
    k = 0;
    do {
      if (++b >= a.B) return;     // not reached before `end`
      nb = row_tiles(a, b, len);
    } while (nb == 0);
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(ok ? N : 0) : "memory");
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

// One piece's query rows as B fragments: part 0 the f16 value, part 1 (rotary
// queries) the remainder; rows are scaled by a power of two so that their
// largest element lies in [2^14, 2^15); fac undoes it and applies the softmax scale.
template <int D, int NT, int PARTS>
__device__ __forceinline__ void load_queries(const DecodeQ4Args& a, const Walk& w, int lane, uint32_t (*qf)[PARTS][D / 16][2],
                                             float (*fac)[2]) {
  constexpr int F = D / 4;            // features of a thread
  const int g = lane >> 2, t = lane & 3;
  const int hkv = w.k / a.nrb, r0 = (w.k - hkv * a.nrb) * 8 * NT;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = r0 + n * 8 + g;
    const long row = ((long)w.b * a.Hq + hkv * a.G) * a.Tq + r;
    const int pos = w.len - a.Tq + r % a.Tq;
    float x[F];
    float amax = 0.f;
    const bool live = r < a.R;
#pragma unroll
    for (int c = 0; c < F / 8; ++c) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (live) u = __ldg(reinterpret_cast<const uint4*>(a.q + row * D + t * F) + c);
      bf16x8_to_f32(u, x + 8 * c);
    }
    if constexpr (PARTS == 2) {
      if (live && pos >= 0) {
        const bool second = t >= 2;   // features D/2.. pair with features 0..
        const int f0 = t * F;
        const float* cs = a.rope_cs + (long)pos * D + (second ? f0 - D / 2 : f0);
#pragma unroll
        for (int c = 0; c < F / 8; ++c) {
          float y[8];
          bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(a.q + row * D + (second ? f0 - D / 2 : f0 + D / 2)) + c), y);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float co = __ldg(cs + 8 * c + i), si = __ldg(cs + D / 2 + 8 * c + i);
            x[8 * c + i] = second ? fmaf(x[8 * c + i], co, y[i] * si) : fmaf(x[8 * c + i], co, -y[i] * si);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < F; ++i) amax = fmaxf(amax, fabsf(x[i]));
    amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
    const int ex = (int)(__float_as_uint(amax) >> 23);          // biased exponent: 0 zero, 255 not finite
    const int sh = ex == 0 || ex == 255 ? 0 : 14 - (ex - 127);  // x * 2^sh, in two steps within f32's range
    const float s1 = __uint_as_float((uint32_t)(127 + sh / 2) << 23), s2 = __uint_as_float((uint32_t)(127 + sh - sh / 2) << 23);
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float lo = x[4 * j + 2 * h] * s1 * s2, hi = x[4 * j + 2 * h + 1] * s1 * s2;
        const uint32_t v = pack_f16x2(lo, hi);
        qf[n][0][j][h] = v;
        if constexpr (PARTS == 2) {
          const float2 b = f16x2_to_f32(v);
          qf[n][1][j][h] = pack_f16x2(lo - b.x, hi - b.y);
        }
      }
    // the columns of S^T are rows 2t and 2t+1: their factors come from the lanes that hold those rows
    const float mine = a.scale_log2 * (1.f / s1) * (1.f / s2);
    fac[n][0] = __shfl_sync(~0u, mine, 8 * t);
    fac[n][1] = __shfl_sync(~0u, mine, 8 * t + 4);
  }
}

// O and LSE of a unit from its complete piece.
template <int D, int NT>
__device__ __forceinline__ void write_unit(const DecodeQ4Args& a, int b, int k, int len, Piece4<D, NT>& p, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const int hkv = k / a.nrb, r0 = (k - hkv * a.nrb) * 8 * NT;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float l = p.l[n][c];
      l += __shfl_xor_sync(~0u, l, 4);
      l += __shfl_xor_sync(~0u, l, 8);
      l += __shfl_xor_sync(~0u, l, 16);
      const int r = r0 + n * 8 + 2 * t + c;
      if (r >= a.R) continue;
      const long row = ((long)b * a.Hq + hkv * a.G) * a.Tq + r;
      const bool empty = len - a.Tq + r % a.Tq < 0;      // the row sees no key
      const float inv = empty ? 0.f : a.v_scale / l;
      if (!GQA_CHECK(row >= 0 && row < (long)a.B * a.Hq * a.Tq, a.status, a.dbg_line)) continue;
      // features gD/8 ..: tile i holds features 2i, 2i+1 of them
      __nv_bfloat16* o = a.o + row * D + g * (D / 8);
      uint32_t w[D / 16];
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        w[i] = empty ? 0u : pack_bf16x2(p.acc[n][i][c] * inv, p.acc[n][i][2 + c] * inv);
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        reinterpret_cast<uint4*>(o)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      if (g == 0) a.lse[row] = empty ? -CUDART_INF_F : (p.m[n][c] - kOff + log2f(l)) * 0.69314718055994531f;
    }
}

// Workspace: a header per CTA, then two pieces per CTA (kRec * 32 f32 each).
struct Q4Head {
  int b, k, len;   // unit of the CTA's first piece
  int first, last; // CTAs that hold pieces of it, -1: not cut before this CTA
  int pad[3];
};

template <int D, int NT, int PARTS>
__global__ void __launch_bounds__(Q4Cfg<D, NT>::kThreads, 1) decode_q4_kernel(const DecodeQ4Args a) {
  using C = Q4Cfg<D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long sums[C::kWarps];
  __shared__ int prefix[C::kThreads];
  __shared__ Walk rec_walk[2 * C::kWarps];   // unit of each stored piece, its first and last tile
  __shared__ long rec_end[2 * C::kWarps];    // stream index after the piece; 0: none
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int upb = a.Hkv * a.nrb;

  if (tid < 2 * C::kWarps) rec_end[tid] = 0;
  // C: tiles of all units
  long mine = 0;
  for (int b = tid; b < a.B; b += C::kThreads) {
    int len;
    const int nb = row_tiles(a, b, len);
    if (nb == 0 && blockIdx.x == 0) atomicCAS(a.status, 0, kDevBadSeqlens);
    mine += nb;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) mine += __shfl_xor_sync(~0u, mine, d);
  if (lane == 0) sums[warp] = mine;
  __syncthreads();
  long total = 0;
#pragma unroll
  for (int w = 0; w < C::kWarps; ++w) total += sums[w];
  total *= upb;
  const int Wn = (int)(total < (long)gridDim.x * C::kWarps ? total : (long)gridDim.x * C::kWarps);
  const int gw = blockIdx.x * C::kWarps + warp;
  const long g0 = Wn == 0 || gw >= Wn ? 0 : gw * total / Wn, g1 = Wn == 0 || gw >= Wn ? 0 : (gw + 1) * total / Wn;

  // the batch row that holds tile g0: inclusive sums of the rows' tiles, kThreads rows at a time
  Walk cw{g0, 0, -1, 0, 0, 0};
  long before = 0;
  for (int b0 = 0; b0 < a.B; b0 += C::kThreads) {
    int len = 0, nb = b0 + tid < a.B ? row_tiles(a, b0 + tid, len) : 0;
    int inc = nb;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(~0u, inc, d);
      if (lane >= d) inc += x;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    long all = 0;
    for (int w = 0; w < C::kWarps; ++w) {
      if (w < warp) inc += (int)sums[w];
      all += sums[w];
    }
    prefix[tid] = inc;
    __syncthreads();
    if (g0 < g1 && cw.b < 0 && g0 < (before + all) * upb) {
      const long x = g0 - before * upb;   // row i of these: prefix[i - 1] * upb <= x < prefix[i] * upb
      int lo = 0, hi = C::kThreads - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((long)prefix[mid] * upb > x) hi = mid;
        else lo = mid + 1;
      }
      cw.b = b0 + lo;
      cw.nb = row_tiles(a, cw.b, cw.len);
      const long P = (before + (lo ? prefix[lo - 1] : 0)) * upb;
      cw.k = (int)((g0 - P) / cw.nb);
      cw.Pu = P + (long)cw.k * cw.nb;
    }
    before += all;
  }

  if (g0 < g1) {
    uint8_t* ring = smem + warp * C::kRing;
    const uint32_t ring_s = smem_u32(ring);
    Walk lw = cw;
    int page[2] = {0, 0};
    auto look_up = [&]() {   // pages of the two halves of the tile at lw
      if (a.block_table && lw.g < g1) {
        const int j = lw.tile() * kTK;
        const int* bt = a.block_table + (long)lw.b * a.max_pages;
        const int p = j / a.page_size;
        page[0] = j < lw.len ? __ldg(bt + p) : 0;
        page[1] = a.page_size == 16 ? (j + 16 < lw.len ? __ldg(bt + p + 1) : 0) : page[0];
      }
    };
    auto issue = [&](int stage) {
      if (lw.g < g1) {
        const int j = lw.tile() * kTK, n = lw.len - j;   // keys of the tile
        const int hkv = lw.k / a.nrb;
        long row[2];
        bool ok[2] = {true, true};
        if (a.block_table) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (page[h] < 0 || page[h] >= a.num_pages) {
              if (lane == 0 && j + 16 * h < lw.len) atomicCAS(a.status, 0, kDevBadPage);
              ok[h] = false;
              page[h] = 0;
            }
            const int off = a.page_size == 16 ? -16 * h : j % a.page_size;   // so that row + key is the key's row
            row[h] = ((long)page[h] * a.Hkv + hkv) * a.page_size + off;
          }
        } else {
          row[0] = row[1] = ((long)lw.b * a.Hkv + hkv) * a.S + j;
        }
        [[maybe_unused]] const long rows = a.block_table ? (long)a.num_pages * a.Hkv * a.page_size : (long)a.B * a.Hkv * a.S;
        const uint32_t s = ring_s + stage * C::kStage;
        constexpr int CH = D / 32;    // 16-byte chunks of a key's codes
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int key = (i * 32 + lane) / CH, c = lane % CH, h = key >> 4;
          const bool valid = key < n && ok[h] && GQA_CHECK(row[h] + key < rows, a.status, a.dbg_line);
          const long at = valid ? (row[h] + key) * (D / 2) + c * 16 : 0;
          const uint32_t d = s + row_at<D>(key, c);
          cp_async16(d, a.k4 + at, valid);
          cp_async16(d + C::kCodes, a.v4 + at, valid);
        }
        const int h = lane >> 4;
        const bool valid = lane < n && ok[h] && GQA_CHECK(row[h] + lane < rows, a.status, a.dbg_line);
        const long at = valid ? (row[h] + lane) * (D / 16) : 0;
        const uint32_t d = s + 2 * C::kCodes + lane * (D / 16);
        cp_async_small<D / 16>(d, a.ksf + at, valid);
        cp_async_small<D / 16>(d + C::kSf, a.vsf + at, valid);
        lw.next(a, g1);
        look_up();
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look_up();
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) issue(i);

    Piece4<D, NT> p;
    uint32_t qf[NT][PARTS][D / 16][2];
    float fac[NT][2];
    int lim[NT][2];               // last key each of the thread's rows sees
    bool fresh = true;
    int stage = 0;
    while (cw.g < g1) {
      if (fresh) {
        load_queries<D, NT, PARTS>(a, cw, lane, qf, fac);
        p.clear();
        const int r0 = (cw.k % a.nrb) * 8 * NT;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) lim[n][c] = cw.len - a.Tq + (r0 + n * 8 + 2 * t + c) % a.Tq;
        fresh = false;
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
      __syncwarp();               // every lane's copies have landed; the stage before is read
      issue(stage == 0 ? C::kStages - 1 : stage - 1);
      const uint32_t s = ring_s + stage * C::kStage;
      const int j0 = cw.tile() * kTK;

      // S^T of both 16-key groups
      float sc[2][NT][4];
#pragma unroll
      for (int G = 0; G < 2; ++G) {
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[G][n][0] = sc[G][n][1] = sc[G][n][2] = sc[G][n][3] = 0.f;
        const int ka = 16 * G + key_of(g), kb = ka + 8;
        uint32_t wa[D / 32], wb[D / 32];
        uint32_t sa, sb;             // block scales as f16 pairs: (first, second) 16 features, D = 64: one
        if constexpr (D == 128) {
          const uint4 u = ld_shared_v4(s + row_at<D>(ka, t)), v = ld_shared_v4(s + row_at<D>(kb, t));
          wa[0] = u.x, wa[1] = u.y, wa[2] = u.z, wa[3] = u.w;
          wb[0] = v.x, wb[1] = v.y, wb[2] = v.z, wb[3] = v.w;
          sa = e4m3x2_to_f16(lds<2>(s + 2 * C::kCodes + ka * 8 + 2 * t));
          sb = e4m3x2_to_f16(lds<2>(s + 2 * C::kCodes + kb * 8 + 2 * t));
        } else {
          lds64(s + row_at<D>(ka, 0) + 8 * t, wa);
          lds64(s + row_at<D>(kb, 0) + 8 * t, wb);
          sa = e4m3x2_to_f16(lds<1>(s + 2 * C::kCodes + ka * 4 + t));
          sb = e4m3x2_to_f16(lds<1>(s + 2 * C::kCodes + kb * 4 + t));
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {     // 8 features: two MMAs
          uint32_t ra[4], rb[4];
          e2m1x8_to_f16(wa[w], ra);
          e2m1x8_to_f16(wb[w], rb);
          const uint32_t sel = D == 128 && w >= 2 ? 0x3232u : 0x1010u;
          const uint32_t fa = __byte_perm(sa, 0, sel), fb = __byte_perm(sb, 0, sel);
#pragma unroll
          for (int i = 0; i < 4; ++i) ra[i] = hmul2_u(ra[i], fa), rb[i] = hmul2_u(rb[i], fb);
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
      // scale, mask, running maximum
      const bool edge = j0 + kTK > cw.len - a.Tq + 1;   // some key of the tile is hidden from some row
      bool grow = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = -CUDART_INF_F;
#pragma unroll
          for (int G = 0; G < 2; ++G)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float& x = sc[G][n][2 * h + c];
              x *= fac[n][c];
              if (edge && j0 + 16 * G + 8 * h + key_of(g) > lim[n][c]) x = -CUDART_INF_F;
              mx = fmaxf(mx, x);
            }
          grow |= mx > p.m[n][c] + kLazy;
        }
      if (__any_sync(~0u, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = fmaxf(fmaxf(sc[0][n][c], sc[0][n][2 + c]), fmaxf(sc[1][n][c], sc[1][n][2 + c]));
            mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
            mx = fmaxf(mx, p.m[n][c]);
            const float f = p.m[n][c] == -CUDART_INF_F ? 1.f : ex2_approx(p.m[n][c] - mx);
            p.m[n][c] = mx;
            p.l[n][c] *= f;
#pragma unroll
            for (int i = 0; i < C::kMT; ++i) p.acc[n][i][c] *= f, p.acc[n][i][2 + c] *= f;
          }
      }
      // P, its sums, and its fragments
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float bias[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) bias[c] = p.m[n][c] == -CUDART_INF_F ? 0.f : kOff - p.m[n][c];
#pragma unroll
        for (int G = 0; G < 2; ++G) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = ex2_approx(sc[G][n][i] + bias[i & 1]);
            p.l[n][i & 1] += x[i];
          }
          pf[G][n][0] = transpose8x8(pack_f16x2(x[0], x[1]));
          pf[G][n][1] = transpose8x8(pack_f16x2(x[2], x[3]));
        }
      }
      // O^T
#pragma unroll
      for (int G = 0; G < 2; ++G) {
        uint32_t sb[4];
        constexpr int VW = D / 64;                 // words of a thread's features of one key
        uint32_t w[4][VW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {              // keys pi(2t), pi(2t+1), pi(2t+8), pi(2t+9)
          const int key = 16 * G + 8 * (i >> 1) + key_of(2 * t + (i & 1));
          if constexpr (D == 128) lds64(s + C::kCodes + row_at<D>(key, g >> 1) + 8 * (g & 1), w[i]);
          else w[i][0] = lds<4>(s + C::kCodes + row_at<D>(key, 0) + 4 * g);
          sb[i] = lds<1>(s + 2 * C::kCodes + C::kSf + key * (D / 16) + (D == 128 ? g : g >> 1));
        }
        if (edge && a.Tq > 1) {
          // a NaN block at a key that some rows do not see: 0 * NaN would reach them through the MMA, so it is
          // taken out here and put into the rows that do see it
          bool bad = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if ((sb[i] & 0x7f) == 0x7f) bad = true, sb[i] = 0;
          }
          if (__any_sync(~0u, bad)) {
            for (int k = 0; k < 16; ++k) {
              const uint32_t v = lds<1>(s + 2 * C::kCodes + C::kSf + (16 * G + k) * (D / 16) + (D == 128 ? g : g >> 1));
              if ((v & 0x7f) != 0x7f) continue;
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  if (j0 + 16 * G + k <= lim[n][c]) {
#pragma unroll
                    for (int i = 0; i < C::kMT; ++i) p.acc[n][i][c] = p.acc[n][i][2 + c] = CUDART_NAN_F;
                  }
            }
          }
        }
        const uint32_t f01 = e4m3x2_to_f16(sb[0] | sb[1] << 8), f23 = e4m3x2_to_f16(sb[2] | sb[3] << 8);
#pragma unroll
        for (int v = 0; v < VW; ++v) {
          // half bytes of two keys side by side: byte i of `even` is feature 2i of both, of `odd` feature 2i+1
          uint32_t e01[4], o01[4], e23[4], o23[4];
          e2m1x8_to_f16((w[0][v] & 0x0F0F0F0Fu) | ((w[1][v] << 4) & 0xF0F0F0F0u), e01);
          e2m1x8_to_f16(((w[0][v] >> 4) & 0x0F0F0F0Fu) | (w[1][v] & 0xF0F0F0F0u), o01);
          e2m1x8_to_f16((w[2][v] & 0x0F0F0F0Fu) | ((w[3][v] << 4) & 0xF0F0F0F0u), e23);
          e2m1x8_to_f16(((w[2][v] >> 4) & 0x0F0F0F0Fu) | (w[3][v] & 0xF0F0F0F0u), o23);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = hmul2_u(e01[i], f01), a1 = hmul2_u(o01[i], f01);
            const uint32_t a2 = hmul2_u(e23[i], f23), a3 = hmul2_u(o23[i], f23);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(p.acc[n][4 * v + i], a0, a1, a2, a3, pf[G][n][0], pf[G][n][1]);
          }
        }
      }
      stage = stage == C::kStages - 1 ? 0 : stage + 1;

      // end of the unit, or of the share
      const long at = cw.g;
      const bool unit_end = cw.tile() == cw.nb - 1;
      if (unit_end || at == g1 - 1) {
        if (unit_end && cw.Pu >= g0) {
          write_unit<D, NT>(a, cw.b, cw.k, cw.len, p, lane);
        } else {
          const int slot = 2 * warp + (cw.Pu < g0 ? 0 : 1);   // a unit begun before the share, or continued after it
          if (slot & 1) {   // the share ends here: no copy is in flight, and every lane has read the last tile
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();
          }
          p.store(piece_at<D, NT>(smem, slot), lane);
          if (lane == 0) {
            rec_walk[slot] = cw;
            rec_end[slot] = at + 1;
          }
        }
        fresh = true;
      }
      cw.next(a, g1);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  __syncthreads();
  griddep_launch();

  // combine the stored pieces of each unit, in stream order; a warp takes the
  // units whose first piece here is its own
  const long c0 = Wn == 0 ? 0 : (long)min((int)blockIdx.x * C::kWarps, Wn) * total / Wn;   // the CTA's share
  Q4Head* heads = static_cast<Q4Head*>(a.ws);
  float* parts = reinterpret_cast<float*>(heads + kMaxCtas);
  bool cut_before = false;
  for (int s = 2 * warp; s < 2 * warp + 2; ++s) {
    if (rec_end[s] == 0) continue;
    const Walk w = rec_walk[s];
    int prev = s - 1;
    while (prev >= 0 && rec_end[prev] == 0) --prev;
    if (prev >= 0 && rec_walk[prev].Pu == w.Pu) continue;   // not the unit's first piece here
    Piece4<D, NT> p;
    p.clear();
    long end = 0;
    for (int i = s; i < 2 * C::kWarps; ++i) {
      if (rec_end[i] == 0) continue;
      if (rec_walk[i].Pu != w.Pu) break;
      p.add(piece_at<D, NT>(smem, i), lane);
      end = rec_end[i];
    }
    if (w.Pu >= c0 && end == w.Pu + w.nb) {
      write_unit<D, NT>(a, w.b, w.k, w.len, p, lane);
      continue;
    }
    const int slot = w.Pu < c0 ? 0 : 1;   // begun before the CTA's share, or in it
    p.store(parts + ((long)blockIdx.x * 2 + slot) * C::kRec * 32, lane);
    if (slot == 0) {
      cut_before = true;
      if (lane == 0) {
        Q4Head h{};
        h.b = w.b;
        h.k = w.k;
        h.len = w.len;
        h.first = owner_of(w.Pu, total, Wn) / C::kWarps;
        h.last = owner_of(w.Pu + w.nb - 1, total, Wn) / C::kWarps;
        heads[blockIdx.x] = h;
      }
    }
  }
  // slot 0 belongs to the warp with the CTA's first tile: warp 0
  if (warp == 0 && lane == 0 && !cut_before) heads[blockIdx.x].first = -1;
}

// Units cut between CTAs: the block of the second CTA that holds a piece of a
// unit combines all of them.
template <int D, int NT>
__global__ void __launch_bounds__(32) decode_q4_merge(const DecodeQ4Args a) {
  using C = Q4Cfg<D, NT>;
  griddep_wait();
  const Q4Head* heads = static_cast<const Q4Head*>(a.ws);
  const float* parts = reinterpret_cast<const float*>(heads + kMaxCtas);
  const Q4Head h = heads[blockIdx.x];
  if (h.first < 0 || (int)blockIdx.x != h.first + 1) return;
  const int lane = threadIdx.x;
  Piece4<D, NT> p;
  p.clear();
  p.add(parts + ((long)h.first * 2 + 1) * C::kRec * 32, lane);
  for (int c = h.first + 1; c <= h.last; ++c) p.add(parts + (long)c * 2 * C::kRec * 32, lane);
  write_unit<D, NT>(a, h.b, h.k, h.len, p, lane);
}

template <int D, int NT, int PARTS>
cudaError_t run(const DecodeQ4Args& a, int ctas, cudaStream_t stream) {
  using C = Q4Cfg<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(decode_q4_kernel<D, NT, PARTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  prof_begin(kProfDecode, stream);
  decode_q4_kernel<D, NT, PARTS><<<ctas, C::kThreads, C::kSmem, stream>>>(a);
  prof_end(stream);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  prof_begin(kProfDecodeMerge, stream);
  e = launch_programmatic(decode_q4_merge<D, NT>, dim3(ctas), dim3(32), 0, stream, a);
  prof_end(stream);
  return e;
}

}  // namespace

// Rows go in blocks of 16 (two 8-row tiles, one conversion of the cache for
// both) unless one tile of 8 holds them all.
static int row_tiles_of(int R) { return R <= 8 ? 1 : 2; }

size_t decode_q4_ws_bytes(int, int Hq, int Hkv, int Tq, int, int D) {
  const int nt = row_tiles_of(Hq / Hkv * Tq);
  return sizeof(Q4Head) * kMaxCtas + (size_t)kMaxCtas * 2 * nt * (D / 16 * 4 + 4) * 128;
}

cudaError_t launch_decode_q4(const DecodeQ4Args& args, int sms, cudaStream_t stream) {
  DecodeQ4Args a = args;
  const int nt = row_tiles_of(a.R);
  a.nrb = (a.R + 8 * nt - 1) / (8 * nt);
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  const bool rope = a.rope_cs != nullptr;
  if (a.D == 128) {
    if (nt == 1) return rope ? run<128, 1, 2>(a, ctas, stream) : run<128, 1, 1>(a, ctas, stream);
    return rope ? run<128, 2, 2>(a, ctas, stream) : run<128, 2, 1>(a, ctas, stream);
  }
  if (nt == 1) return rope ? run<64, 1, 2>(a, ctas, stream) : run<64, 1, 1>(a, ctas, stream);
  return rope ? run<64, 2, 2>(a, ctas, stream) : run<64, 2, 1>(a, ctas, stream);
}

}  // namespace gqa
