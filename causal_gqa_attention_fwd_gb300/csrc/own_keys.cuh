// own_keys.cuh -- the rows' own keys in attention over a shared prefix, and the
// prefix itself where few rows share it, for sm_103a: unnormalised partials
// (O, M, L) of cached attention of few query rows over ragged bf16 caches.
//
// A few query rows (G * Tq of a (batch row, K/V head)) meet each key once: the
// stream of keys and values bounds it, and with rows of a few hundred keys what
// a unit costs beside its stream -- first loads, the drain of the last tile,
// the output -- counts as much.  So every warp runs alone: all units' tiles in
// one stream, each warp a contiguous share of it (a unit counting kUnitCost
// tiles more than it has), its tiles by TMA through a ring of its own that runs
// on across unit boundaries, no barrier between warps.  Both products are
// warp-level MMAs with the cache as the M side:
//   S^T[16 keys][8 rows] = K Q^T,   O^T[16 features][8 rows] += V^T P^T,
// K and V^T fragments by ldmatrix from the 128-byte-swizzled tiles, P^T from the
// score fragments by a register transpose.  (tcgen05 needs 128 keys or features
// as M and a CTA's warps in step; measured on these rows, the decode kernel
// built so streams at a quarter of the copy rate.)
//   A piece (a warp's run of one unit's tiles) is number warp + unit among the
// pieces, so that those of a unit follow one another and the workspace needs
// warps + units entries whatever the lengths are.
#pragma once

#include "kernels.h"
#include "sm103.cuh"
#include "stream.cuh"

namespace gqa {

namespace {

constexpr int kUnitCost = 2;        // tiles that a unit counts more than it has
constexpr int kMinShare = 2;        // least tiles (so counted) a warp takes
constexpr float kRescale = 8.0f;    // log2 units: the maximum in use moves when a score exceeds it by more
constexpr int kDevPages = 11;       // ATTN_ERR_PAGES
constexpr int kOwnIdle = 1 << 30;   // share number of a warp that takes none

template <int D, int NT>
struct OwnCfg {
  static constexpr int KT = D == 128 ? 16 : 32;       // keys a tile: 4 KB of K and of V
  static constexpr int kStage = 8192;
  static constexpr int kWarps = NT == 1 ? 12 : 8;     // registers: 64 a row tile for O and Q
  static constexpr int kStages = NT == 1 ? 2 : 3;
  static constexpr int kSmemBytes = kWarps * kStages * kStage + 1024;
};

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int NT, int THREADS>
struct OwnShared {
  uint64_t full[OwnCfg<D, NT>::kWarps][OwnCfg<D, NT>::kStages];
  int sum[THREADS / 32], pre[THREADS];
};

// The stream's rows are the prefixes it holds (a.P of them, query rows of all their batch rows), then the batch rows.
// A unit in it, and the warp's run of the unit's tiles.
struct Run {
  int i, k;          // row of the stream; unit within it (K/V head, row block)
  int len, nb;       // the row's keys, tiles
  int P;             // stream position of the unit's first tile
  int t, te;         // tiles [t, te)
};

template <int KT>
__device__ __forceinline__ int row_tiles(const OwnArgs& a, int i, int& len) {
  len = i < a.P ? a.prefix_lens[i] : a.cache_lens[i - a.P];
  return len > 0 && len <= (i < a.P ? a.Sp : a.S) ? (len + KT - 1) / KT : 0;
}

__device__ __forceinline__ int blocks_of(const OwnArgs& a, int i) { return i < a.P ? a.nrbp : a.nrb; }

// The next unit's run; te <= t: the share is done.
template <int KT>
__device__ __forceinline__ void next_run(const OwnArgs& a, Run& u, int end) {
  u.P += u.nb + kUnitCost;
  u.t = 0;
  u.te = 0;
  if (u.P >= end) return;
  if (++u.k == a.Hkv * blocks_of(a, u.i)) {
    u.k = 0;
    do {
      ++u.i;
      u.nb = row_tiles<KT>(a, u.i, u.len);
    } while (u.nb == 0);
  }
  u.te = min(u.nb, end - u.P);
}

// All THREADS threads of a block call this; the first kWarps warps take the shares gw, the others kOwnIdle.  smem: 1024-byte
// aligned, kWarps * kStages * kStage bytes.  `warps`: of all blocks.
template <int D, bool PAGED, int NT, int THREADS>
__device__ __forceinline__ void own_keys(uint8_t* smem, OwnShared<D, NT, THREADS>& sh_mem, const CUtensorMap& tm_k,
                                         const CUtensorMap& tm_v, const CUtensorMap& tm_pk, const CUtensorMap& tm_pv,
                                         const OwnArgs& a, int gw, int warps, const Guard& guard) {
  using C = OwnCfg<D, NT>;
  constexpr int KT = C::KT, NB = D / 64, kSteps = D / 16, kMT = D / 16;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(~0u, tid >> 5, 0), g = lane >> 2, tig = lane & 3;
  if (lane == 0 && warp < C::kWarps) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(&sh_mem.full[warp][i], 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  auto positions = [&](int i) {
    int len;
    const int nb = row_tiles<KT>(a, i, len);
    return nb ? (nb + kUnitCost) * (a.Hkv * blocks_of(a, i)) : 0;
  };
  const StreamShare sh = stream_share<THREADS>(a.P + a.B, gw, warps, kMinShare, sh_mem.sum, sh_mem.pre, positions);
  if constexpr (32 * C::kWarps < THREADS) {
    // 8 of 12 warps work, with registers that the others give up: 256 * 232 + 128 * 24 = 62464 of 384 * 168 = 64512.
    // Here, past the code that all of them run with 168.
    static_assert(C::kWarps == 8 && THREADS == 384, "register split");
    if (warp >= C::kWarps) {
      regs_dec<24>();
      return;
    }
    regs_inc<232>();
  }
  Run u{sh.row, 0, 0, 0, 0, 0, 0};
  const int v1 = sh.v1;
  if (u.i >= 0) {
    u.nb = row_tiles<KT>(a, u.i, u.len);
    u.k = (sh.v0 - sh.at) / (u.nb + kUnitCost);
    u.P = sh.at + u.k * (u.nb + kUnitCost) + kUnitCost;
    u.t = max(sh.v0 - u.P, 0);
    u.te = min(u.nb, v1 - u.P);
  }
  if (u.i < 0 || u.t >= u.te) return;
  const uint32_t ring = smem_u32(smem) + warp * (C::kStages * C::kStage);
  uint8_t* ring_p = smem + warp * (C::kStages * C::kStage);
  uint64_t* full = sh_mem.full[warp];
  // ---------------------------------------------------------- loads
  Run ld = u;
  int page0 = -1, ids = -1, loaded = 0;      // paged: lane i holds the id of the row's page page0 + i
  auto issue = [&]() {
    if (ld.t >= ld.te) return;
    const bool pre = ld.i < a.P;
    const int st = loaded % C::kStages, k0 = ld.t * KT, row = pre ? ld.i : ld.i - a.P, hkv = ld.k / blocks_of(a, ld.i);
    uint8_t* dst = ring_p + st * C::kStage;
    uint64_t* bar = &full[st];
    if constexpr (PAGED) {
      const int psz = a.page_size, used = (ld.len - 1) / psz + 1;      // (len + psz may pass 32 bits)
      const int box = min(KT, psz), n = KT / box;
      if (page0 < 0 || (k0 + KT - 1) / psz >= page0 + 32) {
        page0 = k0 / psz;
        ids = -1;
        if (page0 + lane < used) {
          const int e = pre ? a.prefix_table[(long)row * a.max_prefix_pages + page0 + lane]
                            : a.block_table[(long)row * a.max_pages + page0 + lane];
          if (e >= 0 && e < a.num_pages) ids = e;
          else atomicCAS(a.status, 0, kDevPages);
        }
      }
      if (lane == 0) mbar_expect_tx(bar, C::kStage);
      for (int i = 0; i < n; ++i) {
        const int j = k0 + i * box, id = __shfl_sync(~0u, ids, j / psz - page0);
        // no page, or none that holds a key of the row: past the tensor, which gives zeros
        const int z = id >= 0 ? id * a.Hkv + hkv : a.num_pages * a.Hkv;
        if (lane == 0) {
#pragma unroll
          for (int x = 0; x < NB; ++x) {
            tma_load_3d(dst + x * (KT * 128) + i * box * 128, &tm_k, bar, x * 64, j % psz, z);
            tma_load_3d(dst + 4096 + x * (KT * 128) + i * box * 128, &tm_v, bar, x * 64, j % psz, z);
          }
        }
      }
    } else if (lane == 0) {
      mbar_expect_tx(bar, C::kStage);
      const CUtensorMap *mk = pre ? &tm_pk : &tm_k, *mv = pre ? &tm_pv : &tm_v;
#pragma unroll
      for (int x = 0; x < NB; ++x) {
        tma_load_3d(dst + x * (KT * 128), mk, bar, x * 64, k0, row * a.Hkv + hkv);
        tma_load_3d(dst + 4096 + x * (KT * 128), mv, bar, x * 64, k0, row * a.Hkv + hkv);
      }
    }
    ++loaded;
    if (++ld.t == ld.te) {
      next_run<KT>(a, ld, v1);
      page0 = -1;
    }
  };
  for (int i = 0; i < C::kStages; ++i) issue();

  // query fragments of a unit: rows 8 n + g of its block, features 16 s + 2 tig (+1, +8, +9)
  auto load_q = [&](const Run& r, uint32_t (*q)[NT][2]) {
    const int nrb = blocks_of(a, r.i), hkv = r.k / nrb, r0 = r.k % nrb * (8 * NT);
    const int b0 = r.i < a.P ? r.i * a.W : r.i - a.P, n_rows = r.i < a.P ? a.W * a.R : a.R;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = r0 + 8 * n + g, b = b0 + row / a.R;
      const uint32_t* p = reinterpret_cast<const uint32_t*>(a.q + (((long)b * a.Hkv + hkv) * a.R + row % a.R) * D) + tig;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        q[s][n][0] = row < n_rows ? __ldg(p + 8 * s) : 0u;
        q[s][n][1] = row < n_rows ? __ldg(p + 8 * s + 4) : 0u;
      }
    }
  };
  uint32_t q[kSteps][NT][2], qn[kSteps][NT][2];
  load_q(u, qn);
  int done = 0;
  bool ok = true;
  // ldmatrix rows: K, matrices (keys 0-7, 8-15) x (features 0-7, 8-15); V, transposed, (features) x (keys)
  const int krow = lane & 15, kch = lane >> 4, vrow = (lane & 7) + 8 * (lane >> 4), vch = (lane >> 3) & 1;
  while (u.t < u.te && ok) {
    Run nx = u;
    next_run<KT>(a, nx, v1);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int n = 0; n < NT; ++n) q[s][n][0] = qn[s][n][0], q[s][n][1] = qn[s][n][1];
    if (nx.t < nx.te) load_q(nx, qn);      // one unit ahead
    float acc[kMT][NT][4];
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
    float mx[NT][2], l[NT][2];
    int lim[NT][2];                        // last key the row sees
    const bool pre = u.i < a.P;
    const int r0 = u.k % blocks_of(a, u.i) * (8 * NT), n_rows = pre ? a.W * a.R : a.R;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[n][i] = -INFINITY;
        l[n][i] = 0.f;
        lim[n][i] = pre ? u.len - 1 : u.len - a.Tq + (r0 + 8 * n + 2 * tig + i) % a.Tq;
      }
    const int all_see = pre ? u.len - 1 : u.len - a.Tq;      // keys up to here are seen by every row
    for (int t = u.t; t < u.te; ++t) {
      const int st = done % C::kStages;
      ok = __all_sync(~0u, mbar_wait(&full[st], (done / C::kStages) & 1, guard));
      if (!ok) break;
      const uint32_t kb = ring + st * C::kStage, vb = kb + 4096;
#pragma unroll
      for (int sub = 0; sub < KT / 16; ++sub) {
        const int k0 = t * KT + sub * 16;
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        const int kr = sub * 16 + krow;
#pragma unroll
        for (int st2 = 0; st2 < kSteps; ++st2) {
          uint32_t f[4];
          const int ch = 2 * st2 + kch;    // 16-byte part of the row
          ldsm4(f, kb + (ch >> 3) * (KT * 128) + kr * 128 + (((ch & 7) ^ (kr & 7)) << 4));
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_bf16(s[n], f, q[st2][n][0], q[st2][n][1]);
        }
        // s[n]: key g rows 2 tig, 2 tig + 1; key g + 8 the same
        bool over = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] *= a.scale_log2;
          if (k0 + 15 > all_see) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (k0 + g + 8 * (e >> 1) > lim[n][e & 1]) s[n][e] = -INFINITY;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) over |= s[n][e] > mx[n][e & 1] + kRescale;
        }
        if (__any_sync(~0u, over)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float v = fmaxf(s[n][i], s[n][i + 2]);
              v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
              v = fmaxf(v, __shfl_xor_sync(~0u, v, 8));
              v = fmaxf(v, __shfl_xor_sync(~0u, v, 16));
              if (v > mx[n][i] + kRescale) {
                const float al = ex2_approx(mx[n][i] - v);
                mx[n][i] = v;
                l[n][i] *= al;
#pragma unroll
                for (int m = 0; m < kMT; ++m) acc[m][n][i] *= al, acc[m][n][i + 2] *= al;
              }
            }
        }
        uint32_t p[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float u0 = mx[n][0] == -INFINITY ? 0.f : mx[n][0], u1 = mx[n][1] == -INFINITY ? 0.f : mx[n][1];
          const float p0 = ex2_approx(s[n][0] - u0), p1 = ex2_approx(s[n][1] - u1);
          const float p2 = ex2_approx(s[n][2] - u0), p3 = ex2_approx(s[n][3] - u1);
          l[n][0] += p0 + p2;
          l[n][1] += p1 + p3;
          // rounded to bf16 (2^-8 of each weight), V's type, for the MMA
          p[n][0] = transpose8x8(pack_bf16x2(p0, p1));
          p[n][1] = transpose8x8(pack_bf16x2(p2, p3));
        }
        // V rows past the cache may hold anything: zeros, so that 0 * V stays 0
        uint32_t keep[2] = {~0u, ~0u};     // of the keys 2 tig, +1 and 2 tig + 8, +9
        const bool tail = k0 + 16 > u.len;
        if (tail) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int j = k0 + 2 * tig + 8 * i;
            keep[i] = (j < u.len ? 0xffffu : 0u) | (j + 1 < u.len ? 0xffff0000u : 0u);
          }
        }
        const int vr = sub * 16 + vrow;
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
          uint32_t f[4];
          const int ch = 2 * m + vch;
          ldsm4_t(f, vb + (ch >> 3) * (KT * 128) + vr * 128 + (((ch & 7) ^ (vr & 7)) << 4));
          if (tail) f[0] &= keep[0], f[1] &= keep[0], f[2] &= keep[1], f[3] &= keep[1];
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_bf16(acc[m][n], f, p[n][0], p[n][1]);
        }
      }
      ++done;
      __syncwarp();      // the stage is read
      issue();
    }
    if (!ok) break;
    // ------------------------------------------------------- the piece
    const int unit = (pre ? u.i * a.nrbp : a.P * a.nrbp + (u.i - a.P) * a.nrb) * a.Hkv + u.k;
    const long base = ((long)gw + unit) * a.rows_ws;
    if (u.t == 0 && lane == 0) {
      a.counts[unit] = make_int2(gw + unit, sh.split.owner(u.P + u.nb - 1) - gw + 1);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = l[n][i];
        sum += __shfl_xor_sync(~0u, sum, 4);
        sum += __shfl_xor_sync(~0u, sum, 8);
        sum += __shfl_xor_sync(~0u, sum, 16);
        const int row = 8 * n + 2 * tig + i;
        if (row < a.rows_ws && r0 + row < n_rows) {
          if (g == 0) a.ws_ml[base + row] = make_float2(mx[n][i], sum);
          float* o = a.ws_o + (base + row) * D + g;
#pragma unroll
          for (int m = 0; m < kMT; ++m) {
            o[16 * m] = acc[m][n][i];
            o[16 * m + 8] = acc[m][n][i + 2];
          }
        }
      }
    u = nx;
  }
  // never leave with copies in flight
  if (lane == 0)
    for (; done < loaded; ++done) mbar_wait_drain(&full[done % C::kStages], (done / C::kStages) & 1);
  __syncwarp();
}

}  // namespace

}  // namespace gqa
