// cache_evict.cu -- the attention weight that cached keys receive, and cutting
// a cache down to the keys that received most, for sm_103a.
//
// cache_weights  w_j += sum over a step's queries that see key j of
//   exp(scale q . k_j - lse), from w_j = 0 for its Tq new keys: K is read once
//   (memory bounds it for few queries), the scores are warp-level MMAs with 16
//   keys as M and 8 query rows as N.  A dot product does not care for the order of its terms, so a lane
//   takes whole 16-byte parts of a key row as its share of the k index and
//   needs neither shared memory nor shuffles to bring them into place; the
//   query fragments follow the same order.  E4M3 and 4-bit codes are widened to
//   f16 in registers (exactly: e2m1 * e4m3 has 6 significant bits); query rows
//   then are f16 too, scaled by a power of two a row, exact down to 2^-31 of
//   the row's largest feature.  One lane group adds up a key's weight in a
//   fixed order: the same call gives the same bits.
//
//   A long window of queries is GEMM-shaped: tcgen05 (cache_weights_window).
//   Many keys: 32 of them a tile, all in one stream that the grid's warps share
//   (cache_weights_kernel); 8 long rows of 8 heads of 128, 61 us at the copy
//   rate: bf16 keys 67 us; 4-bit ones (18) 32: the chain that widens a tile's keys
//   and multiplies them (issue slots 63% active, no unit full).
//
// evict  a cluster of CTAs a (row, K/V head): each keeps a run of the weights in
//   shared memory (short rows: each all of them, and no exchange); the budget-th
//   largest by radix selection over the weights' bits (11, 11, 10, histograms
//   added up through distributed shared memory), then the kept positions in
//   order, then the rows of every plane to the front.
//   Row i comes from position src_i >= i, and src grows, so going up in phases a
//   phase's rows are read before any is overwritten.
//   Bound: the chain of passes and barriers (some 10 us), then the moves.
#include <cuda_fp16.h>

#include "cache_ops.h"
#include "fp4.cuh"
#include "kernels.h"
#include "sm103.cuh"
#include "stream.cuh"

namespace gqa {

namespace {

constexpr int kWWarps = 8;
constexpr int kWKeys = 32 * kWWarps;   // keys a CTA takes at once
constexpr int kWRows = 64;             // query rows in shared memory at once
constexpr int kScanRows = 128;

__device__ __forceinline__ void mma_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1, bool f16) {
  if (f16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A lane's share of a key row: D/4 features, in parts of E consecutive ones,
// part i at feature E (tig + 4 i).  Step s (16 features of the row, 4 of them
// the lane's) takes its features 4 s .. 4 s + 3.
template <int D, CacheFmt F>
struct KeyPart {
  static constexpr int E = F == kCacheBf16 ? 8 : F == kCacheE4m3 ? 16 : D / 4;
  static constexpr int kParts = D / 4 / E;
  static constexpr int kBytes = F == kCacheBf16 ? 16 : F == kCacheE4m3 ? 16 : E / 2;   // of a part
  static constexpr int kRowBytes = F == kCacheBf16 ? 2 * D : F == kCacheE4m3 ? D : D / 2;
  static constexpr int kWords = kParts * kBytes / 4;
  __device__ static int feature(int s, int tig) { return E * (tig + 4 * (4 * s / E)) + 4 * s % E; }
};

// A lane's share of one key row.
template <int D, CacheFmt F>
struct KeyRow {
  using P = KeyPart<D, F>;
  uint32_t w[P::kWords];
  uint32_t sf;      // 4-bit: the block scales of the lane's features
  // The 16-bit pairs of steps 2 s (r[0], r[1]: its features 0, 1 and 2, 3) and 2 s + 1 (r[2], r[3]).
  __device__ __forceinline__ void steps(int s, uint32_t* r) const {
    if constexpr (F == kCacheBf16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = w[4 * s + i];
    } else if constexpr (F == kCacheE4m3) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        r[2 * i] = e4m3x2_to_f16(w[2 * s + i] & 0xffffu);
        r[2 * i + 1] = e4m3x2_to_f16(w[2 * s + i] >> 16);
      }
    } else {
      const uint32_t both = e4m3x2_to_f16(sf);      // of features 0-15 and (D = 128) 16-31
      const uint32_t two = __byte_perm(both, both, s / 2 ? 0x3232 : 0x1010);
      e2m1x8_to_f16(w[s], r);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = hmul2_u(r[i], two);
    }
  }
};

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}

// A tile of 32 keys on its way into shared memory, by bulk copies of the rows that lie side by side (a page's), with their
// block scales, weights and slots: any number of tiles can be under way without registers, and a warp spends some tens of
// instructions on one.  Rows of 128 or 256 bytes are read back two lanes a bank, which the time does not show.
template <int D, CacheFmt F>
struct KeyStage {
  using P = KeyPart<D, F>;
  static constexpr int kKeys = 32 * P::kRowBytes;
  static constexpr int kSfRow = F == kCacheQ4 ? D / 16 : 0;
  static constexpr int kWeights = kKeys + 32 * kSfRow, kSlots = kWeights + 32 * 4;
  static constexpr int kBytes = kSlots + 32 * 8;

  // The block table's entry for this lane's key (row b itself in a contiguous cache): looked up a tile ahead, for what it
  // takes to come is time that the warp stands still.
  __device__ static int page_of(const WeightsArgs& a, int b, int t, int len, int lane) {
    const int j = 32 * t + lane;
    return a.block_table && j < len ? a.block_table[(long)b * a.max_pages + a.page(j)] : b;
  }
  // Keys 32 t .. of head h of a row of len keys: the copies complete on `bar` (one phase) and as one group of this lane's
  // own.  Returns whether a page was bad.
  __device__ static bool issue(const WeightsArgs& a, uint8_t* st, uint64_t* bar, int page, int h, int t, int len, int lane) {
    const int j = 32 * t + lane, ps = a.page.d;
    const int in_page = a.block_table ? j - a.page(j) * ps : j;               // 0: another page begins
    const int run = a.block_table ? min(ps - in_page, 32 - lane) : 32;
    const bool there = j < len && page >= 0 && page < a.num_pages;
    const long slot = there ? ((long)page * a.Hkv + h) * ps + in_page : -1;
    const int bytes = slot >= 0 && (lane == 0 || in_page == 0) ? min(run, len - j) * P::kRowBytes : 0;
    const int all = __reduce_add_sync(~0u, bytes);
    if (lane == 0) mbar_expect_tx(bar, all);
    __syncwarp();
    if (bytes)
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                       smem_u32(st + lane * P::kRowBytes)),
                   "l"(a.k + slot * P::kRowBytes), "r"(bytes), "r"(smem_u32(bar))
                   : "memory");
    if (slot >= 0) {
      if constexpr (F == kCacheQ4) copy_async<kSfRow>(smem_u32(st + kKeys + lane * kSfRow), a.ksf + slot * kSfRow);
      copy_async<4>(smem_u32(st + kWeights + lane * 4), a.weights + slot);
    }
    *reinterpret_cast<long*>(st + kSlots + lane * 8) = slot;
    copies_commit();
    return j < len && slot < 0;
  }
  // Row `row` of the tile (8 m + g), the lane's share of it.
  __device__ static void row(const uint8_t* st, int row, int tig, KeyRow<D, F>& k) {
    const uint8_t* p = st + row * P::kRowBytes + tig * P::kBytes;
#pragma unroll
    for (int i = 0; i < P::kParts; ++i) {
      if constexpr (P::kBytes == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i * P::kBytes);
        k.w[4 * i] = v.x, k.w[4 * i + 1] = v.y, k.w[4 * i + 2] = v.z, k.w[4 * i + 3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        k.w[0] = v.x, k.w[1] = v.y;
      }
    }
    if constexpr (F == kCacheQ4) {
      const uint8_t* f = st + kKeys + row * kSfRow;
      if constexpr (D == 128) k.sf = *reinterpret_cast<const uint16_t*>(f + 2 * tig);
      else k.sf = f[tig];
    }
  }
  __device__ static float weight(const uint8_t* st, int row) { return *reinterpret_cast<const float*>(st + kWeights + row * 4); }
  __device__ static long slot(const uint8_t* st, int row) { return *reinterpret_cast<const long*>(st + kSlots + row * 8); }
};

// The lane's share of query row `row` (-1: none) in fragments q[s] of step s; f16: scaled by 2^e, which it returns.
template <int D, CacheFmt F>
__device__ __forceinline__ int query_fragments(const WeightsArgs& a, long row, int tig, uint2* q) {
  using P = KeyPart<D, F>;
  constexpr int kSteps = D / 16;
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
    q[s] = row >= 0 ? __ldg(reinterpret_cast<const uint2*>(a.q + row * D + P::feature(s, tig))) : make_uint2(0, 0);
  int e = 0;
  if constexpr (F != kCacheBf16) {
    float mx = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const float2 x = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&q[s].x));
      const float2 y = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&q[s].y));
      mx = fmaxf(fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y))), mx);
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    if (mx > 0.f && mx < INFINITY) e = 14 - ilogbf(mx);     // the largest feature goes to [2^14, 2^15)
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const float2 x = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&q[s].x));
      const float2 y = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&q[s].y));
      q[s].x = pack_f16x2(ldexpf(x.x, e), ldexpf(x.y, e));
      q[s].y = pack_f16x2(ldexpf(y.x, e), ldexpf(y.y, e));
    }
  }
  return e;
}

// Score factor and -lse of a query row, in log2 units, and the last key that it sees (none: no key, nor does a query
// that the caller's attention found to see none).
struct RowConstants {
  float c, l;
  int lim;
};
__device__ __forceinline__ RowConstants row_constants(const WeightsArgs& a, long row, int e, int lim) {
  const float lse = row >= 0 ? __ldg(a.lse + row) : -INFINITY;
  return {ldexpf(a.scale_log2, -e), -lse * 1.4426950408889634f, lse == -INFINITY ? -1 : lim};
}

// ------------------------------------------------ at most 8 NT query rows a key: one stream of tiles over all warps
// Warps: what registers leave; 4-bit keys, with a longer chain a tile, more of them (20 and 16; 12, 16, 24: slower).
template <int D, CacheFmt F, int NT>
struct NarrowCfg {
  static constexpr int kWarps = F == kCacheQ4 ? (NT == 1 ? 20 : 16) : 12;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kFit = (216 << 10) / (kWarps * KeyStage<D, F>::kBytes);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kSmemBytes = kWarps * kStages * KeyStage<D, F>::kBytes;
  static_assert(kStages >= 2, "two tiles on the way");
};

template <int D, CacheFmt F, int NT>
__global__ void __launch_bounds__(NarrowCfg<D, F, NT>::kThreads, 1) cache_weights_kernel(const WeightsArgs a) {
  using C = NarrowCfg<D, F, NT>;
  using St = KeyStage<D, F>;
  constexpr int kSteps = D / 16;
  constexpr bool f16 = F != kCacheBf16;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_sum[C::kWarps], s_pre[C::kThreads], s_abort;
  __shared__ uint64_t s_full[C::kWarps][C::kStages];
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31, g = lane >> 2, tig = lane & 3;
  if (tid == 0) s_abort = 0;
  if (lane == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(&s_full[warp][i], 1);
    fence_barrier_init();
  }
  const Guard guard{&s_abort, a.status};
  griddep_wait();
  griddep_launch();
  auto tiles_of = [&](int b, int& len) {
    len = a.cache_lens[b];
    return len > 0 && len <= a.S ? (len + 31) / 32 : 0;
  };
  auto positions = [&](int b) {
    int len;
    const int nb = tiles_of(b, len);
    if (nb == 0 && len != 0) atomicCAS(a.status, 0, kDevBadSeqlens);
    return nb * a.Hkv;
  };
  const int gw = warp * gridDim.x + blockIdx.x;
  const StreamShare sh = stream_share<C::kThreads>(a.B, gw, gridDim.x * C::kWarps, 1, s_sum, s_pre, positions);
  int left = sh.v1 - sh.v0;
  if (sh.row < 0 || left <= 0) return;
  // where the loads and the scores stand: tile t of (row b, head h)
  struct At {
    int b, h, len, nb, t;
  };
  At ld{sh.row, 0, 0, 0, 0};
  ld.nb = tiles_of(ld.b, ld.len);
  ld.h = (sh.v0 - sh.at) / ld.nb;
  ld.t = (sh.v0 - sh.at) % ld.nb;
  auto next = [&](At& x) {
    if (++x.t < x.nb) return;
    x.t = 0;
    if (++x.h < a.Hkv) return;
    x.h = 0;
    do x.nb = tiles_of(++x.b, x.len);
    while (x.nb == 0);
  };
  uint8_t* ring = smem + warp * (C::kStages * St::kBytes);
  int to_load = left, page = St::page_of(a, ld.b, ld.t, ld.len, lane);
  bool bad = false, ok = true;
  auto issue = [&](int st) {
    if (to_load > 0) {
      bad |= St::issue(a, ring + st * St::kBytes, &s_full[warp][st], page, ld.h, ld.t, ld.len, lane);
      if (--to_load > 0) {
        next(ld);
        page = St::page_of(a, ld.b, ld.t, ld.len, lane);
      }
    } else {
      copies_commit();
    }
  };
  At at = ld;
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) issue(i);
  uint2 q[NT][kSteps];
  RowConstants c[NT][2];      // of rows 8 n + 2 tig + i
  bool fresh = true;
  uint32_t phase = 0;
  int st = 0;
  for (; left > 0; --left) {
    __syncwarp();        // the stage before is read
    issue(st == 0 ? C::kStages - 1 : st - 1);
    if (fresh) {
      const long row0 = ((long)at.b * a.Hkv + at.h) * a.R;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int e = query_fragments<D, F>(a, 8 * n + g < a.R ? row0 + 8 * n + g : -1, tig, q[n]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 8 * n + 2 * tig + i;
          const int er = __shfl_sync(~0u, e, 4 * (2 * tig + i));
          c[n][i] = row_constants(a, r < a.R ? row0 + r : -1, er, at.len - a.Tq + r % a.Tq);
        }
      }
      fresh = false;
    }
    copies_wait<C::kStages - 1>();
    ok = __all_sync(~0u, mbar_wait(&s_full[warp][st], phase, guard));
    if (!ok) break;
    __syncwarp();        // the other lanes' copies have landed too
    const uint8_t* sp = ring + st * St::kBytes;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      KeyRow<D, F> k0, k1;      // keys 16 m + g and 16 m + 8 + g
      St::row(sp, 16 * m + g, tig, k0);
      St::row(sp, 16 * m + 8 + g, tig, k1);
      float acc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
      for (int s = 0; s < kSteps / 2; ++s) {
        uint32_t f0[4], f1[4];
        k0.steps(s, f0);
        k1.steps(s, f1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t f[4] = {f0[2 * i], f1[2 * i], f0[2 * i + 1], f1[2 * i + 1]};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_16816(acc[n], f, q[n][2 * s + i].x, q[n][2 * s + i].y, f16);
        }
      }
      const int j = 32 * at.t + 16 * m + g;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float p0 = ex2_approx(fmaf(acc[n][i], c[n][i].c, c[n][i].l));
          const float p1 = ex2_approx(fmaf(acc[n][2 + i], c[n][i].c, c[n][i].l));
          if (j <= c[n][i].lim) sum[2 * m] += p0;
          if (j + 8 <= c[n][i].lim) sum[2 * m + 1] += p1;
        }
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      sum[m] += __shfl_xor_sync(~0u, sum[m], 1);
      sum[m] += __shfl_xor_sync(~0u, sum[m], 2);
    }
    const float mine = tig == 0 ? sum[0] : tig == 1 ? sum[1] : tig == 2 ? sum[2] : sum[3];
    const int r = 8 * tig + g;
    const long slot = St::slot(sp, r);
    // the step's new keys had no weight before
    if (slot >= 0) a.weights[slot] = mine + (32 * at.t + r < at.len - a.Tq ? St::weight(sp, r) : 0.f);
    if (left > 1) {
      fresh = at.t + 1 == at.nb;
      next(at);
    }
    if (++st == C::kStages) {
      st = 0;
      phase ^= 1;
    }
  }
  // never leave with copies in flight (after a wait that gave up)
  copies_wait<0>();
  if (lane == 0)
    for (int i = left - to_load; i > 0; --i) {
      mbar_wait_drain(&s_full[warp][st], phase);
      if (++st == C::kStages) st = 0, phase ^= 1;
    }
  __syncwarp();
  if (bad) atomicCAS(a.status, 0, kDevBadPage);
}

// The chunk of kWKeys keys that this CTA takes: from key c0 on of head hkv of row b.
struct Chunk {
  int b, hkv, c0, len;
};

// All warps together.  a.scan: the chunks that hold keys, one CTA after another, found by a scan of the lengths in each
// warp, so that none of the CTAs that start together is one that its row has no keys for.  For grids that do not fit at
// once (5 rows of 301-7001 keys, 16 queries, 560 CTAs: 7.3 us, otherwise 8.9; where all have keys it costs 2-5%) and up to
// kScanRows rows.  Otherwise a CTA has its place in the capacity.
__device__ __forceinline__ bool find_chunk(const WeightsArgs& a, Chunk& c) {
  const int lane = threadIdx.x & 31, at = (int)blockIdx.x;
  if (!a.scan) {
    const int bh = at % (a.B * a.Hkv);
    c.b = bh / a.Hkv, c.hkv = bh % a.Hkv, c.c0 = at / (a.B * a.Hkv) * kWKeys;
    c.len = a.cache_lens[c.b];
    if (c.len >= 0 && c.len <= a.S) return c.c0 < c.len;
    if (c.c0 == 0 && threadIdx.x == 0) atomicCAS(a.status, 0, kDevBadSeqlens);
    return false;
  }
  int before = 0;
  bool found = false;
  for (int b0 = 0; b0 < a.B && (!found || at == 0); b0 += 32) {
    int len = b0 + lane < a.B ? a.cache_lens[b0 + lane] : 0;
    if (len < 0 || len > a.S) {
      if (at == 0) atomicCAS(a.status, 0, kDevBadSeqlens);
      len = 0;
    }
    const int n = (len + kWKeys - 1) / kWKeys * a.Hkv;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned hit = __ballot_sync(~0u, before + incl > at);
    if (hit && !found) {
      const int l = __ffs(hit) - 1, k = at - before - __shfl_sync(~0u, incl - n, l);
      found = true;
      c.b = b0 + l, c.hkv = k % a.Hkv, c.c0 = k / a.Hkv * kWKeys;
      c.len = __shfl_sync(~0u, len, l);
    }
    before += __shfl_sync(~0u, incl, 31);
  }
  return found;
}

// ------------------------------------------------ more query rows (a window of a prompt), or few keys: a CTA a chunk of keys
// Each warp holds the fragments of 32 keys in registers and takes the query rows, kWRows at a time, from shared memory.
template <int D, CacheFmt F>
__global__ void __launch_bounds__(32 * kWWarps) cache_weights_wide_kernel(const WeightsArgs a) {
  using St = KeyStage<D, F>;
  constexpr int kSteps = D / 16;
  constexpr bool f16 = F != kCacheBf16;
  extern __shared__ __align__(128) uint8_t smem[];  // a stage a warp
  __shared__ uint64_t s_full[kWWarps];
  __shared__ int s_abort;
  __shared__ uint2 s_q[kWRows / 8][kSteps][32];     // query fragments, by lane
  __shared__ RowConstants s_c[kWRows];
  griddep_wait();
  griddep_launch();
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  Chunk chunk;
  if (!find_chunk(a, chunk)) return;
  const int b = chunk.b, hkv = chunk.hkv, c0 = chunk.c0, len = chunk.len, bh = b * a.Hkv + hkv;
  if (threadIdx.x == 0) s_abort = 0;
  if (lane == 0) {
    mbar_init(&s_full[warp], 1);
    fence_barrier_init();
  }
  __syncthreads();
  const Guard guard{&s_abort, a.status};
  const int k0 = c0 + warp * 32;
  uint8_t* sp = smem + warp * St::kBytes;
  if (St::issue(a, sp, &s_full[warp], St::page_of(a, b, k0 / 32, len, lane), hkv, k0 / 32, len, lane))
    atomicCAS(a.status, 0, kDevBadPage);
  bool ok = true;
  uint32_t f[2][kSteps][4];
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  for (int r0 = 0; r0 < a.R; r0 += kWRows) {
    const int nt = min(kWRows, (a.R - r0 + 7) & ~7) / 8;
    if (r0) __syncthreads();
    for (int t = warp; t < nt; t += kWWarps) {      // eight query rows a warp
      const long row0 = (long)bh * a.R + r0;
      const int r = 8 * t + g;
      uint2 q[kSteps];
      const long row = r0 + r < a.R ? row0 + r : -1;
      const int e = query_fragments<D, F>(a, row, tig, q);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) s_q[t][s][lane] = q[s];
      if (tig == 0) {
        s_c[r] = row_constants(a, row, e, len - a.Tq + (r0 + r) % a.Tq);
      }
    }
    if (r0 == 0) {
      copies_wait<0>();
      ok = __all_sync(~0u, mbar_wait(&s_full[warp], 0, guard));      // and, as a barrier, the other lanes' copies
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        KeyRow<D, F> x, y;
        St::row(sp, 16 * m + g, tig, x);
        St::row(sp, 16 * m + 8 + g, tig, y);
#pragma unroll
        for (int s = 0; s < kSteps / 2; ++s) {
          uint32_t f0[4], f1[4];
          x.steps(s, f0);
          y.steps(s, f1);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            f[m][2 * s + i][0] = f0[2 * i], f[m][2 * s + i][1] = f1[2 * i], f[m][2 * s + i][2] = f0[2 * i + 1],
                            f[m][2 * s + i][3] = f1[2 * i + 1];
        }
      }
    }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      float acc[2][4] = {};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const uint2 q = s_q[t][s][lane];
        mma_16816(acc[0], f[0][s], q.x, q.y, f16);
        mma_16816(acc[1], f[1][s], q.x, q.y, f16);
      }
      // acc[m][0, 1]: key 16 m + g, rows 2 tig, 2 tig + 1; [2, 3]: key 16 m + 8 + g
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * t + 2 * tig + i;
        const RowConstants c = s_c[r];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float p = ex2_approx(fmaf(acc[m / 2][2 * (m & 1) + i], c.c, c.l));
          if (k0 + 8 * m + g <= c.lim) sum[m] += p;
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    sum[m] += __shfl_xor_sync(0xffffffffu, sum[m], 1);
    sum[m] += __shfl_xor_sync(0xffffffffu, sum[m], 2);
  }
  const float mine = tig == 0 ? sum[0] : tig == 1 ? sum[1] : tig == 2 ? sum[2] : sum[3];
  const int r = 8 * tig + g;
  const long slot = St::slot(sp, r);
  // the step's new keys had no weight before
  if (ok && slot >= 0) a.weights[slot] = mine + (k0 + r < len - a.Tq ? St::weight(sp, r) : 0.f);
  if (!ok) mbar_wait_drain(&s_full[warp], 0);        // never leave with copies in flight
}

// ------------------------------------------------ a long window: S^T = K Q^T on tcgen05
// A CTA a chunk of 256 keys, in shared memory as two tiles of 128 (M); the query rows (N) go by 64, and while a block's
// weights are formed the next one's products run.  A thread has one key's scores and adds its weights up by itself.
// Bound: latency of a block's chain (128 rows: issue slots 45% active, XU and tensor pipe 26% each); for 8- and 4-bit keys
// also the query rows' conversion to f16, which every CTA does for itself.  512 rows over 2^20 keys: bf16 of 128 221 us, of 64 174 (3.1e12 exponentials a second), E4M3 of 128 340.
template <int D>
struct WindowCfg {
  static constexpr int kRows = 64, kKeys = kWKeys;
  static constexpr int kBoxes = D / 64;             // of 64 features, 128 bytes a row
  static constexpr int kKeyBox = 128 * 128, kRowBox = kRows * 128;
  static constexpr int kSmemBytes = kBoxes * (2 * kKeyBox + 2 * kRowBox) + 1024;
};

// Part c (16 bytes) of row r of a tile whose boxes are `box` bytes apart, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_at(uint32_t tile, int box, int r, int c) {
  return tile + (c >> 3) * box + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

template <int D, CacheFmt F>
__global__ void __launch_bounds__(WindowCfg<D>::kKeys, 2) cache_weights_window_kernel(const WeightsArgs a) {
  using C = WindowCfg<D>;
  using P = KeyPart<D, F>;
  constexpr int kParts = D / 8, kAt = C::kRows * kParts / C::kKeys;
  extern __shared__ uint8_t smem_raw[];
  // RowConstants of the block before, this and the next: c, l side by side (bf16 keys: c is the same for all)
  constexpr int kEach = F == kCacheBf16 ? 1 : 2;
  __shared__ __align__(16) float s_c[3][C::kRows * kEach];
  __shared__ int s_lim[3][C::kRows], s_whole[3][2];      // s_whole: 32 rows that see all of the chunk's keys
  __shared__ uint64_t s_done[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31, x = warp >> 2;
  griddep_wait();
  Chunk chunk;
  if (!find_chunk(a, chunk)) return;
  const int b = chunk.b, hkv = chunk.hkv, c0 = chunk.c0, len = chunk.len, bh = b * a.Hkv + hkv;
  const uint32_t s_k = (smem_u32(smem_raw) + 1023) & ~1023u, s_q = s_k + 2 * C::kBoxes * C::kKeyBox;
  const uint32_t tile = s_k + x * C::kBoxes * C::kKeyBox;
  if (tid == 0) {
    s_abort = 0;
    mbar_init(&s_done[0], 1);
    mbar_init(&s_done[1], 1);
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(&s_tmem, 4 * C::kRows);
    tmem_relinquish();
  }
  const Guard guard{&s_abort, a.status};
  // ---------------------------------------------------------- query rows, D / 8 lanes each; on their way a block ahead
  uint4 q[kAt];
  float lse = -INFINITY;                                 // of row tid
  auto load_q = [&](int r0) {
    const int rows = min(C::kRows, a.R - r0);
    const long row0 = (long)bh * a.R + r0;
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      const int at = tid + i * C::kKeys;
      q[i] = at < rows * kParts ? __ldg(reinterpret_cast<const uint4*>(a.q + row0 * D) + at) : make_uint4(0, 0, 0, 0);
    }
    lse = tid < rows ? __ldg(a.lse + row0 + tid) : -INFINITY;
  };
  auto store_q = [&](int blk) {
    const int r0 = blk * C::kRows, buf = blk & 1, cbuf = blk % 3;
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      const int at = tid + i * C::kKeys, r = at / kParts, c = at % kParts;
      uint4 v = q[i];
      int e = 0;
      if constexpr (F != kCacheBf16) {
        float f[8];
        bf16x8_to_f32(v, f);
        float mx = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(f[k]));
#pragma unroll
        for (int o = 1; o < kParts; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
        if (mx > 0.f && mx < INFINITY) e = 14 - ilogbf(mx);     // the largest feature goes to [2^14, 2^15)
        // 2^e in two factors, each a normal number; what the first makes subnormal is below f16's least by far
        const float e0 = __int_as_float((127 + (e >> 1)) << 23), e1 = __int_as_float((127 + e - (e >> 1)) << 23);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = f[k] * e0 * e1;
        v = make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]), pack_f16x2(f[6], f[7]));
      }
      st_shared_v4(tile_at(s_q + buf * C::kBoxes * C::kRowBox, C::kRowBox, r, c), v.x, v.y, v.z, v.w);
      if (kEach == 2 && c == 0) s_c[cbuf][2 * r] = ldexpf(a.scale_log2, -e);
    }
    if (tid < C::kRows) {
      s_c[cbuf][kEach * tid + kEach - 1] = -lse * 1.4426950408889634f;
      s_lim[cbuf][tid] = lse == -INFINITY ? -1 : len - a.Tq + (r0 + tid) % a.Tq;
      const bool all = __all_sync(~0u, c0 + C::kKeys - 1 <= len - a.Tq && lse > -INFINITY && r0 + tid < a.R);
      if (lane == 0) s_whole[cbuf][warp] = all;
    }
    fence_proxy_async_smem();
    tc_fence_before();
  };
  // warp 0: both tiles' scores of the block in buffer `buf`
  auto issue = [&](int buf) {
    constexpr uint32_t kIdesc =
        F == kCacheBf16 ? idesc_bf16(128, C::kRows, false, false) : idesc_f16(128, C::kRows, false, false);
    tc_fence_after();
    const uint64_t kd = sdesc_sw128(s_k, 16, 1024), qd = sdesc_sw128(s_q + buf * C::kBoxes * C::kRowBox, 16, 1024);
    if (elect_one()) {
#pragma unroll 1
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          mma_ss(s_tmem + (2 * buf + t) * C::kRows, sdesc_add(kd, (t * C::kBoxes + (s >> 2)) * C::kKeyBox + (s & 3) * 32),
                 sdesc_add(qd, (s >> 2) * C::kRowBox + (s & 3) * 32), kIdesc, s > 0);
    }
    __syncwarp();
    tc_commit_warp(&s_done[buf]);
  };
  load_q(0);
  // ---------------------------------------------------------- keys: thread = key, then lanes side by side along its row
  const int j = c0 + tid;
  long slot = -1;
  if (j < len) {
    const int i = a.block_table ? a.page(j) : 0, page = a.block_table ? a.block_table[(long)b * a.max_pages + i] : b;
    if (page >= 0 && page < a.num_pages) slot = ((long)page * a.Hkv + hkv) * a.page.d + (j - i * a.page.d);
    else atomicCAS(a.status, 0, kDevBadPage);
  }
  {
    constexpr int kLanes = P::kRowBytes / 16, kPer = 32 / kLanes, kSteps = 32 / kPer;
    const int part = lane % kLanes, row0 = lane / kLanes, r0 = (warp & 3) * 32;
    if constexpr (F == kCacheBf16) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = i * kPer + row0;
        const long s = __shfl_sync(~0u, slot, r);
        if (s >= 0) copy_async<16>(tile_at(tile, C::kKeyBox, r0 + r, part), a.k + s * P::kRowBytes + part * 16);
      }
      copies_commit();
      store_q(0);
      copies_wait<0>();
      fence_proxy_async_smem();
    } else {
      uint4 v[kSteps];
      uint32_t sf[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const long s = __shfl_sync(~0u, slot, i * kPer + row0);
        v[i] = make_uint4(0, 0, 0, 0);
        sf[i] = 0;
        if (s >= 0) {
          v[i] = __ldg(reinterpret_cast<const uint4*>(a.k + s * P::kRowBytes + part * 16));
          if constexpr (F == kCacheQ4) sf[i] = __ldg(reinterpret_cast<const uint16_t*>(a.ksf + s * (D / 16) + part * 2));
        }
      }
      store_q(0);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = r0 + i * kPer + row0;
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        if constexpr (F == kCacheE4m3) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            st_shared_v4(tile_at(tile, C::kKeyBox, r, 2 * part + c), e4m3x2_to_f16(w[2 * c] & 0xffffu),
                         e4m3x2_to_f16(w[2 * c] >> 16), e4m3x2_to_f16(w[2 * c + 1] & 0xffffu), e4m3x2_to_f16(w[2 * c + 1] >> 16));
        } else {
          const uint32_t both = e4m3x2_to_f16(sf[i]);      // the scales of 16 features each
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t f[4];
            const uint32_t two = __byte_perm(both, both, c / 2 ? 0x3232 : 0x1010);
            e2m1x8_to_f16(w[c], f);
            st_shared_v4(tile_at(tile, C::kKeyBox, r, 4 * part + c), hmul2_u(f[0], two), hmul2_u(f[1], two),
                         hmul2_u(f[2], two), hmul2_u(f[3], two));
          }
        }
      }
      fence_proxy_async_smem();
    }
  }
  // the step's new keys had no weight before
  const float old = slot >= 0 && j < len - a.Tq ? a.weights[slot] : 0.f;
  __syncthreads();
  griddep_launch();      // not before this CTA has its TMEM: the next kernel's CTAs may take theirs before they wait
  if (warp == 0) issue(0);
  if (C::kRows < a.R) load_q(C::kRows);
  const uint32_t mine = s_tmem + ((uint32_t)(warp & 3) * 32 << 16) + x * C::kRows;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  bool ok = true;
  const int blocks = (a.R + C::kRows - 1) / C::kRows;
  int issued = 1;
  for (int i = 0; i < blocks; ++i) {
    const int buf = i & 1;
    if (i + 1 < blocks) {
      // its rows' place is free: this warp has waited for block i - 1's products
      store_q(i + 1);
      ok = __syncthreads_and(ok);      // and all warps have read block i - 1's scores
      if (!ok) break;
      if (warp == 0) issue(buf ^ 1);
      ++issued;
      if (i + 2 < blocks) load_q((i + 2) * C::kRows);
    }
    ok = __all_sync(~0u, mbar_wait(&s_done[buf], (i >> 1) & 1, guard));
    if (ok) {
      tc_fence_after();
      const float* cs = s_c[i % 3];
#pragma unroll 1
      for (int n0 = 0; n0 < C::kRows; n0 += 32) {
        uint32_t s[32];
        tmem_ld_x32(mine + 2 * buf * C::kRows + n0, s);
        tmem_ld_wait();
        reg_fence<32>(s);
        if (s_whole[i % 3][n0 / 32]) {
          // a shared-memory word serves 32 lanes at once, but a 16-byte one takes four times as long as a 4-byte one: 16 a
          // row (c, l, the last key seen) would take longer than the exponentials
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            float c[4], l[4];
            if constexpr (kEach == 1) {
              const float4 v = *reinterpret_cast<const float4*>(cs + n0 + k);
              c[0] = c[1] = c[2] = c[3] = a.scale_log2;
              l[0] = v.x, l[1] = v.y, l[2] = v.z, l[3] = v.w;
            } else {
              const float4 v = *reinterpret_cast<const float4*>(cs + 2 * (n0 + k));
              const float4 w = *reinterpret_cast<const float4*>(cs + 2 * (n0 + k) + 4);
              c[0] = v.x, c[1] = v.z, c[2] = w.x, c[3] = w.z;
              l[0] = v.y, l[1] = v.w, l[2] = w.y, l[3] = w.w;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += ex2_approx(fmaf(__uint_as_float(s[k + e]), c[e], l[e]));
          }
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float c = kEach == 1 ? a.scale_log2 : cs[2 * (n0 + k)], l = cs[kEach * (n0 + k) + kEach - 1];
            const float p = ex2_approx(fmaf(__uint_as_float(s[k]), c, l));
            if (j <= s_lim[i % 3][n0 + k]) sum[k & 3] += p;
          }
        }
      }
    }
  }
  if (ok && slot >= 0) a.weights[slot] = (sum[0] + sum[1]) + (sum[2] + sum[3]) + old;
  // never leave with MMAs in flight (after a wait that gave up): the last block's, and the one's before
  if (!ok)
    for (int i = max(issued - 2, 0); i < issued; ++i) mbar_wait_drain(&s_done[i & 1], (i >> 1) & 1);
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(s_tmem, 4 * C::kRows);
  }
}

// Once a device.
template <auto KERNEL>
cudaError_t allow_smem(int bytes) {
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && attr_set[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) attr_set[dev] = true;
  return e;
}

template <int D, CacheFmt F, int NT>
cudaError_t launch_narrow(const WeightsArgs& a, int sms, cudaStream_t stream) {
  using C = NarrowCfg<D, F, NT>;
  const cudaError_t e = allow_smem<cache_weights_kernel<D, F, NT>>(C::kSmemBytes);
  return e != cudaSuccess ? e
                          : launch_programmatic(cache_weights_kernel<D, F, NT>, dim3(sms), dim3(C::kThreads),
                                                (size_t)C::kSmemBytes, stream, a);
}

template <int D, CacheFmt F>
cudaError_t launch_weights_df(WeightsArgs a, int sms, cudaStream_t stream) {
  // The stream is for many keys: where a CTA a chunk of the capacity are resident together (two an SM, heads of 64 three),
  // they have no shares to work out.  us, CTAs / stream, 8 rows: bf16 keys of 128, 32768: 3.4 / 4.1, 65536: 4.3 / 5.4,
  // 98304: 7.0 / 6.5; keys of 64, 98304: 4.1 / 5.0, 131072: 5.9 / 5.6; E4M3 of 128, 65536: 4.1 / 5.5, 131072: 6.8 / 6.7;
  // 4-bit of 128, 65536: 3.8 / 6.0, 131072: 6.3 / 7.3, 262144: 11.2 / 9.4.  (Lengths equal to the capacity, which is what
  // a host knows: 8 rows of 2048 keys, 2 heads of 64, tables of 2048 / 8192 / 131072 positions: 3.0 / 3.5 / 3.6.)
  const long ctas = (long)a.B * a.Hkv * ((a.S + (long)kWKeys - 1) / kWKeys);
  const bool at_once = ctas <= (D == 128 ? 2L : 3L) * sms;
  if (a.R <= 16 && !at_once)
    return a.R <= 8 ? launch_narrow<D, F, 1>(a, sms, stream) : launch_narrow<D, F, 2>(a, sms, stream);
  const dim3 grid((unsigned)ctas);
  a.scan = a.B <= kScanRows && !at_once;
  // Warp MMAs keep up with few rows only, but need no tiles in shared memory.  us, this / those: bf16 keys of 128, 131072
  // of them: 32 rows 9.0 / 9.9, 64: 9.1 / 13.8, 128: 12.6 / 22.9, 512: 34 / 75; 2^20, 512 rows: 221 / 490; keys of 64,
  // 2^20: 48 rows 50 / 45, 64: 50 / 51, 128: 69 / 82.  E4M3 of 128, 262144: 64 rows 21 / 21, 96: 31 / 29, 128: 31 / 34,
  // 512: 93 / 119; 4-bit: 96 rows 31 / 32, 512: 93 / 130.
  if (a.R > (F != kCacheBf16 ? 96 : D == 128 ? 32 : 48)) {
    using C = WindowCfg<D>;
    const cudaError_t e = allow_smem<cache_weights_window_kernel<D, F>>(C::kSmemBytes);
    return e != cudaSuccess ? e
                            : launch_programmatic(cache_weights_window_kernel<D, F>, grid, dim3(C::kKeys),
                                                  (size_t)C::kSmemBytes, stream, a);
  }
  constexpr int kSmem = kWWarps * KeyStage<D, F>::kBytes;
  const cudaError_t e = allow_smem<cache_weights_wide_kernel<D, F>>(kSmem);
  return e != cudaSuccess ? e
                          : launch_programmatic(cache_weights_wide_kernel<D, F>, grid, dim3(32 * kWWarps), (size_t)kSmem,
                                                stream, a);
}

template <CacheFmt F>
cudaError_t launch_weights_f(const WeightsArgs& a, int sms, cudaStream_t stream) {
  return a.D == 128 ? launch_weights_df<128, F>(a, sms, stream) : launch_weights_df<64, F>(a, sms, stream);
}

}  // namespace

cudaError_t launch_cache_weights(WeightsArgs a, CacheFmt fmt, int sms, cudaStream_t stream) {
  a.page = FastDiv::of(a.page_size);
  prof_begin(kProfWeights, stream);
  const cudaError_t e = fmt == kCacheBf16   ? launch_weights_f<kCacheBf16>(a, sms, stream)
                        : fmt == kCacheE4m3 ? launch_weights_f<kCacheE4m3>(a, sms, stream)
                                            : launch_weights_f<kCacheQ4>(a, sms, stream);
  prof_end(stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

namespace {

constexpr int kEvThreads = 512;      // two CTAs an SM at 64 registers
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kBins = 2048;          // of a pass over 11 bits (the last: 10)
constexpr int kPlaceBytes = 4096;    // of rows that a warp has on the way between reading and writing
constexpr int kPlaces = kEvWarps * kPlaceBytes;
constexpr int kKeyBytes = 80 << 10;  // weights a CTA keeps in shared memory; a longer share is read again each pass
// Positions up to which each CTA of a cluster selects by itself, without the cluster's barriers (us, alone / together,
// 16 units: 2048 positions 11.8 / 12.7, 4096: 20.6 / 18.0, 8192: 29.8 / 25.0).
constexpr int kAlone = 2048;
// The most that a launch asks for: a share of the weights, or places and (CTAs that select alone) a list behind them.
constexpr int kEvMaxSmem = kKeyBytes > kPlaces + 4 * kAlone ? kKeyBytes : kPlaces + 4 * kAlone;
static_assert(4 * kAlone <= kPlaces && kKeyBytes % 16 == 0, "the list lies behind the places");

// Whole numbers in the weights' order: NaN above all, -0 = 0; 0 is below all of them.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ int4 peer_int4(const void* p, int rank) {
  int4 v;
  asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
               "ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [a];\n\t}"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(smem_u32(p)), "r"(rank)
               : "memory");
  return v;
}

// A run of `cnt` rows, list[d0 + i] -> d0 + i, of one plane, by one warp through its place in shared memory.  Lane i finds
// where row i comes from and goes to; the warp then moves the rows' parts side by side.
struct Task {
  uint8_t* base;
  int row_bytes, size, parts, cnt;
  long from, to;      // slots of row `lane`; -1: it stays, or is in a page outside the pool
  __device__ __forceinline__ void find(const EvictPlane& pl, const Slots& slot_of, const int* list, int d0, int rows, int S,
                                       int lane) {
    base = static_cast<uint8_t*>(pl.p);
    row_bytes = pl.row_bytes;
    size = pl.size;
    parts = pl.parts;
    cnt = rows;
    const int src = lane < cnt ? list[d0 + lane] : -1;
    from = to = -1;
    if (src > d0 + lane && src < S) {
      from = slot_of(src);
      to = from >= 0 ? slot_of(d0 + lane) : -1;
      if (to < 0) from = -1;
    }
  }
  // f(byte in the run, address of that part of its row), for all parts of rows whose slot is not -1
  template <class F>
  __device__ __forceinline__ void each(long slot, int lane, F f) const {
    const int n = min(parts, 32), rpw = 32 / n;           // rows at once
    const int sub = lane / n, part = lane - sub * n;
    for (int r0 = 0; r0 < cnt; r0 += rpw) {
      const int r = r0 + sub;
      const long s = __shfl_sync(~0u, slot, r & 31);
      if (sub < rpw && r < cnt && s >= 0)
        for (int p = part; p < parts; p += 32) f(r * row_bytes + p * size, base + s * row_bytes + p * size);
    }
  }
  __device__ __forceinline__ void read(uint8_t* place, int lane) const {
    each(from, lane, [&](int at, const uint8_t* p) {
      const uint32_t to_smem = smem_u32(place + at);
      if (size == 16) copy_async<16>(to_smem, p);
      else if (size == 8) copy_async<8>(to_smem, p);
      else copy_async<4>(to_smem, p);
    });
    copies_commit();
    copies_wait<0>();
    __syncwarp();
  }
  __device__ __forceinline__ void write(const uint8_t* place, int lane) const {
    each(to, lane, [&](int at, uint8_t* p) {
      if (size == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(place + at);
      else if (size == 8) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(place + at);
      else *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(place + at);
    });
    __syncwarp();         // the place is free again
  }
};

// Moves the rows list[d] -> d, d in [first, budget), of every plane, runs of rows by the cluster's warps.  Row d may be
// written once whatever is kept of position d has been read, that is all rows i with list[i] <= d.  So the rows go in
// phases [c0, c1): if list[c0] lies `hold` rows or more behind c0, all rows up to position list[c0] are free to go one
// run after another, for every source in front of that position belongs to an earlier phase; otherwise as many as the
// warps' places hold are read before any is written.
__device__ __forceinline__ void move_rows(const EvictArgs& a, const Slots& slot_of, const int* list, uint8_t* places, int rank,
                                          int ranks) {
  const int lane = threadIdx.x & 31, warp = __shfl_sync(~0u, threadIdx.x >> 5, 0);
  uint8_t* place = places + warp * kPlaceBytes;
  const int me = warp * ranks + rank, all = kEvWarps * ranks;
  // the first row that moves: list[d] - d never falls
  int d_lo = a.first, d_hi = a.budget;
  while (d_lo < d_hi) {
    const int step = (d_hi - d_lo + 31) / 32, d = d_lo + lane * step;
    const unsigned in = __ballot_sync(~0u, d < d_hi), moves = __ballot_sync(~0u, d < d_hi && list[d] > d);
    const int i = moves ? __ffs(moves) - 1 : __popc(in);     // the first of the lanes whose row moves
    if (moves) d_hi = d_lo + i * step;
    d_lo = i ? d_lo + (i - 1) * step + 1 : d_hi;
  }
  for (int c0 = d_lo; c0 < a.budget;) {
    const int free_to = min(list[c0], a.budget);
    const bool held = free_to < c0 + a.hold && free_to < a.budget;
    const int c1 = held ? min(c0 + a.hold, a.budget) : free_to;
    for (int k = me;; k += all) {          // held: no warp has more than one run
      int i = 0, t = k, runs = 0;
      for (; i < a.n_planes; ++i) {
        runs = (c1 - c0 + a.planes[i].run - 1) / a.planes[i].run;
        if (t < runs) break;
        t -= runs;
      }
      const bool mine = i < a.n_planes;
      if (!mine && !held) break;
      Task task;
      if (mine) {
        const int d0 = c0 + t * a.planes[i].run;
        task.find(a.planes[i], slot_of, list, d0, min(a.planes[i].run, c1 - d0), a.S, lane);
        task.read(place, lane);
      }
      if (held) cluster_sync();
      if (mine) task.write(place, lane);
      if (held) break;
    }
    if (!held && c1 < a.budget) cluster_sync();       // the phase's rows are read before later ones are written over them
    c0 = c1;
  }
}

__global__ void __launch_bounds__(kEvThreads, 2) evict_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint32_t s_keys[];   // order_of this CTA's share of the weights
  __shared__ __align__(16) int s_hist[3][kBins];
  __shared__ __align__(16) int s_coarse[3][kEvWarps];  // sums over 128 bins
  __shared__ int s_gt[kEvWarps], s_eq[kEvWarps];
  __shared__ __align__(16) int s_tot[4];               // the CTA's keys above the threshold, and equal to it
  __shared__ uint32_t s_pre;
  __shared__ int s_need, s_all;
  const int ranks = a.cluster, rank = blockIdx.x % ranks, unit = blockIdx.x / ranks, b = unit / a.Hkv, h = unit % a.Hkv;
  // the warp's number told to be the same in all lanes: votes and shuffles under conditions on it take 100 ns each otherwise
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
  griddep_wait();
  griddep_launch();
  const int n = __shfl_sync(~0u, a.cache_lens[b], 0);
  int* kept = a.kept + (long)unit * a.budget;
  const bool valid = n >= 0 && n <= a.S;
  if (h == 0 && rank == 0 && tid == 0) {
    if (!valid) atomicCAS(a.status, 0, kDevBadSeqlens);
    a.lens_out[b] = valid ? min(n, a.budget) : n;
  }
  if (!valid || n <= a.budget) {                        // the same in the whole cluster
    for (int i = rank * kEvThreads + tid; i < a.budget; i += ranks * kEvThreads) kept[i] = valid && i < n ? i : -1;
    return;
  }
  // n > budget >= first + recent: of the positions [first, n - recent) the `need` largest are kept.  Each CTA selects
  // among all of them by itself, or (a.shared_select) the cluster together, a CTA a run, so that the runs follow one
  // another in the list.
  const int sr = a.shared_select ? rank : 0, srs = a.shared_select ? ranks : 1;
  const int m = n - a.recent - a.first, run = (m + srs - 1) / srs;
  const int lo = a.first + min(sr * run, m), hi = a.first + min((sr + 1) * run, m);
  int need = a.budget - a.first - a.recent;
  const bool cached = run * 4 <= a.key_bytes;
  // shared memory: the weights, in whose place rows are on the way later; the list
  int* list = a.shared_select ? kept : reinterpret_cast<int*>(s_keys) + max(a.key_bytes, kPlaces) / 4;
  bool bad = false;
  const Slots slot_of{a.block_table ? a.block_table + (long)b * a.max_pages : nullptr, a.num_pages, b, a.page, a.Hkv, h};
  auto load_key = [&](int j) {
    const long s = slot_of(j);
    bad |= s < 0;
    return s < 0 ? 0u : order_of(a.weights[s]);
  };
  auto key = [&](int j) { return cached ? s_keys[j - lo] : load_key(j); };
  uint32_t thr = 0xffffffffu, mask = 0xffffffffu;       // kept: (key & mask) > thr, and the first `need` equal to it
  if (need > 0) {
    for (int i = tid; i < 3 * kBins / 4; i += kEvThreads) reinterpret_cast<int4*>(&s_hist[0][0])[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    thr = mask = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t bins = pass == 2 ? 1023u : 2047u;
      int* hist = s_hist[pass];
      if (pass == 0 && cached) {
        for (int j0 = lo + tid; j0 < hi; j0 += 8 * kEvThreads) {
          uint32_t k[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) k[u] = j0 + u * kEvThreads < hi ? load_key(j0 + u * kEvThreads) : 0u;
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (j0 + u * kEvThreads < hi) {
              s_keys[j0 + u * kEvThreads - lo] = k[u];
              atomicAdd(&hist[k[u] >> shift], 1);
            }
        }
      } else if (cached) {
#pragma unroll 8
        for (int i = tid; i < hi - lo; i += kEvThreads) {
          const uint32_t k = s_keys[i];
          if ((k & mask) == thr) atomicAdd(&hist[(k >> shift) & bins], 1);
        }
      } else {
        for (int j = lo + tid; j < hi; j += kEvThreads) {
          const uint32_t k = load_key(j);
          if ((k & mask) == thr) atomicAdd(&hist[(k >> shift) & bins], 1);
        }
      }
      __syncthreads();
      const int4 own = *reinterpret_cast<const int4*>(&hist[4 * tid]);
      const int sum = __reduce_add_sync(0xffffffffu, own.x + own.y + own.z + own.w);
      if (lane == 0) s_coarse[pass][warp] = sum;
      if (srs > 1) cluster_sync();
      else __syncthreads();
      if (warp == 0) {
        // Of 16 x 128 bins, from above until `need` keys are reached: the sums of 128, then the bins of one of them.
        // Lane 4 r + k has rank r's sums 4 k .. 4 k + 3, then all ranks' together.
        int4 c = make_int4(0, 0, 0, 0);
        if (lane / 4 < srs) c = srs > 1 ? peer_int4(&s_coarse[pass][4 * (lane & 3)], lane / 4)
                                        : *reinterpret_cast<const int4*>(&s_coarse[pass][4 * (lane & 3)]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          c.x += __shfl_xor_sync(0xffffffffu, c.x, o);
          c.y += __shfl_xor_sync(0xffffffffu, c.y, o);
          c.z += __shfl_xor_sync(0xffffffffu, c.z, o);
          c.w += __shfl_xor_sync(0xffffffffu, c.w, o);
        }
        const int t = c.x + c.y + c.z + c.w;
        int from = 0;
#pragma unroll
        for (int k = 1; k < 4; ++k) {
          const int y = __shfl_sync(0xffffffffu, t, k);
          if (k > (lane & 3)) from += y;
        }
        int hit = -1, base = 0;
        const int cc[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          if (from < need && need <= from + cc[i]) hit = 4 * (lane & 3) + i, base = from;
          from += cc[i];
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, hit >= 0)) - 1;
        hit = __shfl_sync(0xffffffffu, hit, src);
        base = __shfl_sync(0xffffffffu, base, src);
        const int* fine = &hist[128 * hit + 4 * lane];
        int4 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          v[r] = r >= srs ? make_int4(0, 0, 0, 0) : srs > 1 ? peer_int4(fine, r) : *reinterpret_cast<const int4*>(fine);
        int f[4] = {0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < 8; ++r) f[0] += v[r].x, f[1] += v[r].y, f[2] += v[r].z, f[3] += v[r].w;
        const int mine = f[0] + f[1] + f[2] + f[3];
        int above = mine;                               // keys in bins of this and higher lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_down_sync(0xffffffffu, above, o);
          if (lane + o < 32) above += y;
        }
        from = base + above - mine;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          if (from < need && need <= from + f[i]) {
            s_pre = thr | (uint32_t)(128 * hit + 4 * lane + i) << shift;
            s_need = need - from;
            s_all = need - from == f[i];
          }
          from += f[i];
        }
      }
      __syncthreads();
      thr = s_pre;
      need = s_need;
      mask |= bins << shift;
      if (s_all) break;                                 // the whole bin is kept: its keys need no order
      __syncthreads();
    }
  }
  // Count, then write: a warp takes a run of the CTA's.
  const bool any = a.budget > a.first + a.recent;
  const int wrun = ((hi - lo + kEvWarps - 1) / kEvWarps + 31) & ~31;
  const int w0 = min(lo + warp * wrun, hi), w1 = min(w0 + wrun, hi);
  int gt = 0, eq = 0;
  if (any && cached) {
#pragma unroll 4
    for (int j = w0 + lane; j < w1; j += 32) {
      const uint32_t k = s_keys[j - lo] & mask;
      gt += k > thr;
      eq += k == thr;
    }
  } else if (any) {
    for (int j = w0 + lane; j < w1; j += 32) {
      const uint32_t k = load_key(j) & mask;
      gt += k > thr;
      eq += k == thr;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  if (srs > 1) {
    if (warp == 0) {
      const int g = __reduce_add_sync(0xffffffffu, lane < kEvWarps ? s_gt[lane] : 0);
      const int e = __reduce_add_sync(0xffffffffu, lane < kEvWarps ? s_eq[lane] : 0);
      if (lane == 0) s_tot[0] = g, s_tot[1] = e;
    }
    cluster_sync();
  }
  // what lies before this warp's run: lane r adds up rank r's, lane 8 + i warp i's
  gt = eq = 0;
  if (lane < sr) {
    const int4 v = peer_int4(s_tot, lane);
    gt = v.x, eq = v.y;
  } else if (lane >= 8 && lane - 8 < warp) {
    gt = s_gt[lane - 8], eq = s_eq[lane - 8];
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  for (int j0 = w0; j0 < w1 && any; j0 += 32) {
    const int j = j0 + lane;
    const uint32_t k = j < w1 ? key(j) & mask : 0u;
    const unsigned bg = __ballot_sync(0xffffffffu, j < w1 && k > thr), be = __ballot_sync(0xffffffffu, j < w1 && k == thr);
    const unsigned below = (1u << lane) - 1u;
    const int g = gt + __popc(bg & below), e = eq + __popc(be & below);
    // (in bounds whatever happens: weights read again each pass may be another row's too, against the contract)
    const int at = a.first + g + min(e, need);
    if (((bg >> lane & 1u) || ((be >> lane & 1u) && e < need)) && at < a.budget) list[at] = j;
    gt += __popc(bg);
    eq += __popc(be);
  }
  for (int i = sr * kEvThreads + tid; i < a.first; i += srs * kEvThreads) list[i] = i;
  for (int i = sr * kEvThreads + tid; i < a.recent; i += srs * kEvThreads) list[a.budget - a.recent + i] = n - a.recent + i;
  if (bad) atomicCAS(a.status, 0, kDevBadPage);
  // the list is written, and every weight is read (and every peer's shared memory), before rows move
  cluster_sync();
  if (!a.shared_select)
    for (int i = rank * kEvThreads + tid; i < a.budget; i += ranks * kEvThreads) kept[i] = list[i];
  move_rows(a, slot_of, list, reinterpret_cast<uint8_t*>(s_keys), rank, ranks);
}

}  // namespace

cudaError_t launch_cache_evict(EvictArgs a, cudaStream_t stream) {
  a.page = FastDiv::of(a.page_size);
  const long units = (long)a.B * a.Hkv;
  // a cluster a unit, as large as leaves all CTAs resident (two an SM) and 256 positions a CTA
  a.cluster = 8;
  while (a.cluster > 1 && (units * a.cluster > 304 || a.S < 256L * a.cluster)) a.cluster /= 2;
  a.shared_select = a.cluster > 1 && a.S > kAlone;
  const long run = a.shared_select ? ((long)a.S + a.cluster - 1) / a.cluster : a.S;
  a.key_bytes = run * 4 <= kKeyBytes ? (int)(run * 4 + 15) / 16 * 16 : 0;
  int smem = a.key_bytes > kPlaces ? a.key_bytes : kPlaces;
  if (!a.shared_select) {      // the list beside the weights; rows too long for that: one CTA, the list in memory
    if (a.S <= kAlone) smem += (a.budget < a.S ? a.budget : a.S) * 4;
    else a.shared_select = 1;
  }
  // runs of rows that fill a warp's place, 32 at most; as many rows as the cluster's warps hold with a run each
  for (int i = 0; i < a.n_planes; ++i) {
    EvictPlane& p = a.planes[i];
    p.size = p.row_bytes % 16 == 0 ? 16 : p.row_bytes % 8 == 0 ? 8 : 4;
    p.parts = p.row_bytes / p.size;
    p.run = kPlaceBytes / p.row_bytes < 32 ? kPlaceBytes / p.row_bytes : 32;
  }
  auto runs = [&](int rows) {
    int n = 0;
    for (int i = 0; i < a.n_planes; ++i) n += (rows + a.planes[i].run - 1) / a.planes[i].run;
    return n;
  };
  a.hold = 1;
  for (int step = 1 << 12; step > 0; step /= 2)
    if (runs(a.hold + step) <= kEvWarps * a.cluster) a.hold += step;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvMaxSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[dev] = true;
  }
  prof_begin(kProfEvict, stream);
  const cudaError_t e = launch_programmatic_clusters(evict_kernel, a.cluster, dim3((unsigned)(units * a.cluster)),
                                                     dim3(kEvThreads), (size_t)smem, stream, a);
  prof_end(stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gqa
