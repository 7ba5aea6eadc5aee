// attn_prefix.cu -- cached attention of a batch whose rows share a prefix, for
// sm_103a: the prefix's keys and values are read once for all of its rows.
//
// Row b of prefix p holds the prefix's m_p keys and n_b keys of its own; with
// S_j = scale q k_j the softmax over both is the two softmaxes joined,
//   M = max(M_p, M_o),  L = L_p 2^(M_p - M) + L_o 2^(M_o - M),
//   O = (O_p 2^(M_p - M) + O_o 2^(M_o - M)) / L,   LSE = ln 2 (M + log2 L),
// so the two parts run apart, in one launch: some CTAs of attn_prefix leave
// unnormalised partials (O, M, L) of the prefixes, the others those of the rows'
// own caches (own_keys.cuh), and prefix_merge joins them.  (Where few rows share
// a prefix attn_own.cu takes both parts as one stream instead.)
//
// attn_prefix  Which CTAs take the own keys is settled on the device, by the
//   lengths (share_out).  The W * G * Tq query rows that meet a (prefix, K/V
//   head) are a matrix, and both products are GEMM-shaped: tiles of 128 query
//   rows as M, 128 keys as N of the score MMA, on tcgen05 with the accumulators
//   in TMEM (S_A, S_B, O_A, O_B; P in bf16 over its S), as the prefill kernel
//   has them.  One CTA holds two tiles.  A unit of more than 128 rows fills both
//   and each reads every key block; one of at most 128 rows is held by both
//   tiles, which then take the key blocks in turn, so that one's exponentials
//   run beside the other's MMAs (two partials a piece).
//   Persistent CTAs in teams (kernels.h, PrefixArgs) share the key blocks
//   evenly; a piece is a run of one unit's blocks.
//   Roles (384 threads): warp 0 TMA producer (K and V blocks, one box a page
//   where a page is shorter than a block), warp 1 MMA issuer, warps 4-7 and
//   8-11 softmax of a tile each, thread = row; they also gather the query rows
//   (a tile's rows lie in runs of G * Tq in memory) and write the partials.
//   Bound: many rows, the MMAs (a pair of tiles' two products are 1.35 us a
//   block of 128 keys at the rate of a large library product); few rows, the
//   stream of keys and values.  A CTA's start takes some 10 us beside the own
//   keys' loads, much of it code that it meets for the first time: the softmax
//   takes 64 scores at a time rather than 128 for that.  64 rows over 8192 keys and ~32000
//   own ones 41 us (25 at the copy rate), 256 rows over 32768 keys and ~70000
//   own ones 130 us (74).
#include "own_keys.cuh"
#include "share_out.h"

namespace gqa {

namespace {

constexpr int kBM = 128;                   // query rows per tile
constexpr int kBN = 128;                   // keys per block
constexpr int kCh = 64;                    // scores of a row in registers at once
constexpr float kRescaleThreshold = 8.0f;  // log2 units: lazy O rescale

template <int D>
struct PreCfg {
  static constexpr int kTileBytes = kBM * D * 2;
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kBM * 128;
  static constexpr int kStages = D == 128 ? 5 : 10;    // K and V blocks in flight: what shared memory holds
  static constexpr int kSmemBytes = 2 * kTileBytes + kStages * kTileBytes + 1024;
  static constexpr uint32_t kIdescQK = idesc_bf16(kBM, kBN, false, false);
  static constexpr uint32_t kIdescPV = idesc_bf16(kBM, D, false, true);
  __device__ static constexpr uint32_t col_s(int x) { return (uint32_t)x * 128u; }
  __device__ static constexpr uint32_t col_o(int x) { return 256u + (uint32_t)x * 128u; }
  static_assert(kSmemBytes + 1024 <= 232448, "shared memory");
};

struct __align__(8) PreBarriers {
  uint64_t q_full[2];
  uint64_t kv_full[10], kv_empty[10];
  uint64_t s_full[2];
  uint64_t p_half[2], p_full[2];   // keys 0-63 of P are in TMEM; all of them
  uint64_t o_done[2];
  uint64_t teardown;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ int prefix_blocks(const PrefixArgs& a, int p) {
  const int m = a.prefix_lens[p];
  return m > 0 && m <= a.Sp ? (m + kBN - 1) / kBN : 0;
}

// Scores kCh q .. of a row, -infinity from column nvis on.
__device__ __forceinline__ void load_scores(uint32_t tS, int q, int nvis, uint32_t* s) {
#pragma unroll
  for (int k = 0; k < kCh / 32; ++k) tmem_ld_x32(tS + q * kCh + k * 32, s + k * 32);
  tmem_ld_wait();
  reg_fence<kCh>(s);
  if (nvis < kBN) {
#pragma unroll
    for (int k = 0; k < kCh; ++k)
      if (q * kCh + k >= nvis) s[k] = 0xff800000u;
  }
}

// A piece: blocks [kb, kb + n) of unit (p, hkv, mt).
struct Piece {
  int p, hkv, mt;
  int kb, n;
  int len;             // keys of the prefix
  int rows;            // query rows of the unit
  int split;           // the two tiles take the blocks in turn
};

// Where a CTA's walk over its share stands.  Every role walks it.
struct Walk {
  Piece it;
  EvenSplit split;     // of the stream between the teams with a share
  int g, g1;           // stream position of the piece's first block; end of the share
  int p, nb;           // prefix of the piece, its blocks
  int Pb;              // stream position of prefix p's first block
  int team, inner;
  bool valid;
};

__device__ __forceinline__ void walk_piece(const PrefixArgs& a, Walk& w) {
  const int off = w.g - w.Pb, group = off / w.nb, kb = off - group * w.nb;   // (hkv, outer), block
  Piece& it = w.it;
  it.p = w.p;
  it.hkv = group / a.outer;
  it.mt = (group - it.hkv * a.outer) * a.width + w.inner;
  it.kb = kb;
  it.n = min(w.nb - kb, w.g1 - w.g);
  it.len = a.prefix_lens[w.p];
  it.rows = min(kPrefixRows, a.Rp - it.mt * kPrefixRows);
  it.split = it.rows <= kBM;
  w.valid = true;
}

__device__ __forceinline__ void walk_next(const PrefixArgs& a, Walk& w) {
  w.g += w.it.n;
  if (w.g >= w.g1) {
    w.valid = false;
    return;
  }
  const int gpp = a.Hkv * a.outer;
  while (w.g >= w.Pb + gpp * w.nb) {
    w.Pb += gpp * w.nb;
    ++w.p;
    w.nb = prefix_blocks(a, w.p);
  }
  walk_piece(a, w);
}

// The walk of CTA `cta` of `ctas` from its start (one warp); total: blocks of all groups.
__device__ Walk walk_begin(const PrefixArgs& a, int cta, int ctas, int total) {
  const int lane = threadIdx.x & 31, gpp = a.Hkv * a.outer;
  Walk w{};
  w.split = EvenSplit::of(total, min(ctas / a.width, total));
  w.team = cta / a.width;
  w.inner = cta - w.team * a.width;
  w.valid = false;
  if (w.team >= w.split.parts) return w;
  w.g = w.split.begin(w.team);
  w.g1 = w.split.begin(w.team + 1);
  int P = 0;
  for (int p0 = 0; p0 < a.P; p0 += 32) {
    const int n = p0 + lane < a.P ? prefix_blocks(a, p0 + lane) : 0;
    int incl = gpp * n;   // inclusive sums over the 32 prefixes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, P + incl > w.g);
    if (hit) {
      const int l = __ffs(hit) - 1;
      w.p = p0 + l;
      w.nb = __shfl_sync(0xffffffffu, n, l);
      w.Pb = P + __shfl_sync(0xffffffffu, incl - gpp * n, l);
      break;
    }
    P += __shfl_sync(0xffffffffu, incl, 31);
  }
  walk_piece(a, w);
  return w;
}

}  // namespace

// What the lengths make of the grid's G CTAs (share_out.h).
struct Parts {
  int own;         // CTAs of the rows' own keys, the others take the prefixes
  int blocks;      // key blocks of all prefixes' groups
};

template <int KT, int WARPS>
__device__ Parts share_out(const PrefixArgs& p, const OwnArgs& a, int G, int* s_red) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int tiles = 0, blocks = 0, rows = 0;
  for (int b = tid; b < a.B; b += 384) {
    int len;
    const int nb = row_tiles<KT>(a, b, len);
    if (nb == 0 && len != 0 && blockIdx.x == 0) atomicCAS(a.status, 0, kDevBadSeqlens);
    tiles += nb;
    rows += nb > 0;
  }
  for (int i = tid; i < p.P; i += 384) {
    const int m = p.prefix_lens[i];
    if ((m < 0 || m > p.Sp) && blockIdx.x == 0) atomicCAS(a.status, 0, kDevBadSeqlens);
    blocks += prefix_blocks(p, i);
  }
  tiles = __reduce_add_sync(~0u, tiles);
  blocks = __reduce_add_sync(~0u, blocks);
  rows = __reduce_add_sync(~0u, rows);
  if (lane == 0) s_red[warp] = tiles, s_red[12 + warp] = blocks, s_red[24 + warp] = rows;
  __syncthreads();
  tiles = blocks = rows = 0;
#pragma unroll
  for (int w = 0; w < 12; ++w) tiles += s_red[w], blocks += s_red[12 + w], rows += s_red[24 + w];
  const int runs = p.Hkv * p.outer;
  blocks *= runs;
  if (tiles == 0) return {0, blocks};
  if (blocks == 0) return {G, 0};
  // (a single unit of at most a tile's rows: `split`)
  const ShareWork work{G, p.width, runs, p.P, blocks, p.nrt == 1 && p.Rp <= kBM, a.Hkv * a.nrb, tiles, rows, WARPS, a.D};
  unsigned best = ~0u;
  if (tid >= 1 && tid <= G - p.width) best = share_rank(share_time(work, tid), tid);
  best = __reduce_min_sync(~0u, best);
  __syncthreads();
  if (lane == 0) s_red[warp] = (int)best;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 12; ++w) best = min(best, (unsigned)s_red[w]);
  return {(int)(best & 255u), blocks};
}

template <int D, bool PAGED, int NT>
__global__ void __launch_bounds__(384, 1)
    attn_prefix_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_ok, const __grid_constant__ CUtensorMap tm_ov,
                       const PrefixArgs a, const OwnArgs own) {
  using C = PreCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                          // 2 tiles
  uint8_t* sRing = smem + 2 * C::kTileBytes;   // kStages tiles: K_0, V_0, K_1, ...
  __shared__ PreBarriers bars;
  __shared__ Walk s_walk;
  __shared__ int s_red[36];

  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // the same in a warp, told so
  Guard guard{&bars.abort, a.status};
  if (threadIdx.x == 0) bars.abort = 0;
  griddep_wait();
  griddep_launch();

  // ------------------------------------------------ this CTA's part: own keys (spread evenly over the grid) or prefixes
  const Parts parts = share_out<OwnCfg<D, NT>::KT, OwnCfg<D, NT>::kWarps>(a, own, gridDim.x, s_red);
  const int G = gridDim.x, X = __shfl_sync(~0u, parts.own, 0);
  const int before = blockIdx.x * X / G;       // own-key CTAs of lower number
  if ((blockIdx.x + 1) * X / G > before) {
    using O = OwnCfg<D, NT>;
    auto& shared = *reinterpret_cast<OwnShared<D, NT, 384>*>(smem + O::kWarps * O::kStages * O::kStage);   // behind the rings
    const int gw = warp < O::kWarps ? warp * X + before : kOwnIdle;
    own_keys<D, PAGED, NT, 384>(smem, shared, tm_ok, tm_ov, tm_ok, tm_ov, own, gw, X * O::kWarps, guard);
    return;
  }
  const int cta = blockIdx.x - before, ctas = G - X;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 4);     // one arrive per softmax warp
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_half[i], 4);
      mbar_init(&bars.p_full[i], 4);
      mbar_init(&bars.o_done[i], 1);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bars.kv_full[s], 1);
      mbar_init(&bars.kv_empty[s], 1);
    }
    mbar_init(&bars.teardown, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars.tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == 0) {
    const Walk w0 = walk_begin(a, cta, ctas, parts.blocks);
    if (lane == 0) s_walk = w0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;

  if (warp == 0) {
    // ======================================================== TMA producer
    regs_dec<64>();
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    int stage = 0, fill = 0;
    int last_fill[C::kStages];
#pragma unroll
    for (int i = 0; i < C::kStages; ++i) last_fill[i] = -1;
    bool ok = true;
    for (Walk w = s_walk; w.valid && ok; walk_next(a, w)) {
      for (int j = 0; j < w.it.n && ok; ++j) {
        const int k0 = (w.it.kb + j) * kBN;
        // Paged: lane i looks up the block's i-th page; pages without a key of the prefix and invalid entries
        // (reported) get a coordinate past the tensor, which the TMA fills with zeros.
        int pg = -1, npc = 1;
        if constexpr (PAGED) {
          const int psz = a.page_size;
          npc = psz >= kBN ? 1 : kBN / psz;
          const int idx = k0 / psz + lane;
          bool bad = false;
          if (lane < npc && idx <= (w.it.len - 1) / psz) {
            const int e = a.table[(long)w.it.p * a.max_pages + idx];
            if (e >= 0 && e < a.num_pages) pg = e;
            else bad = true;
          }
          if (__any_sync(0xffffffffu, bad) && lane == 0) atomicCAS(a.status, 0, kDevPages);
        }
        for (int kv = 0; kv < 2 && ok; ++kv) {
          if (fill >= 1) ok = __all_sync(0xffffffffu, mbar_wait(&bars.kv_empty[stage], (fill - 1) & 1, guard));
          if (!ok) break;
          uint8_t* dst = sRing + stage * C::kTileBytes;
          uint64_t* bar = &bars.kv_full[stage];
          const CUtensorMap* tm = kv == 0 ? &tm_k : &tm_v;
          if (lane == 0) mbar_expect_tx(bar, C::kTileBytes);
          __syncwarp();
          if constexpr (PAGED) {
            const int psz = a.page_size;
            const int row = psz >= kBN ? k0 % psz : 0;
            // lane i loads the i-th page's boxes
            if (lane < npc) {
              const int z = pg >= 0 ? pg * a.Hkv + w.it.hkv : a.num_pages * a.Hkv;
#pragma unroll
              for (int x = 0; x < C::kBoxes; ++x)
                tma_load_3d(dst + x * C::kBoxBytes + lane * psz * 128, tm, bar, x * 64, row, z);
            }
          } else if (lane == 0) {
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x)
              tma_load_3d(dst + x * C::kBoxBytes, tm, bar, x * 64, k0, w.it.p * a.Hkv + w.it.hkv);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < C::kStages; ++i)
            if (i == stage) last_fill[i] = fill;
          if (++stage == C::kStages) {
            stage = 0;
            ++fill;
          }
        }
      }
    }
    // never leave the CTA with copies in flight
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < C::kStages; ++i)
        if (last_fill[i] >= 0) mbar_wait_drain(&bars.kv_full[i], (uint32_t)last_fill[i] & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ============================================ MMA issuer (whole warp, one lane issues)
    regs_dec<64>();
    // One loop for both kinds of unit and both tiles: a CTA sees few blocks, and code that runs for the first time costs
    // 0.5 us for every 50 instructions (a loop for each kind with both tiles unrolled: 20 us at 8192 keys and 100 at 32768
    // where this takes 15 and 87; the products rolled too: 17 and 112).
    const uint32_t sq_addr = smem_u32(sQ), ring_addr = smem_u32(sRing);
    bool ok = true;
    uint32_t pc[2] = {0, 0};   // P blocks taken from each tile
    int base = 0, uses = 0;    // ring index of the piece's K_0 (V_j follows K_j); pieces before
    for (Walk w = s_walk; w.valid && ok; walk_next(a, w), ++uses) {
      const int n = w.it.n;
      const bool split = w.it.split;
      for (int x = 0; x < 2 && ok; ++x) ok = __all_sync(0xffffffffu, mbar_wait(&bars.q_full[x], uses & 1, guard));
      // Step t is tile t & 1's: P V of its block j, then the scores of its next one.  Tiles that read every block:
      // j = t / 2 - 1 and j + 1; tiles that take them in turn: j = t - 2 and j + 2.
      const int steps = split ? n + 2 : 2 * n + 2;
#pragma unroll 1
      for (int t = 0; t < steps && ok; ++t) {
        const int x = t & 1, nj = split ? t : t >> 1, j = split ? t - 2 : (t >> 1) - 1;
        const bool last_reader = split || x == 1;
        if (j >= 0) {
          const int vi = base + 2 * j + 1, st = vi % C::kStages;
          ok = __all_sync(0xffffffffu, mbar_wait(&bars.kv_full[st], (vi / C::kStages) & 1, guard));
          if (!ok) break;
          const uint64_t vd = sdesc_sw128(ring_addr + st * C::kTileBytes, C::kBoxBytes, 1024);
          const uint32_t par = (x ? pc[1] : pc[0]) & 1;
          const bool acc = j >= (split ? 2 : 1);
          // P comes in two halves, so that the first half's P V runs while the softmax forms the second
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            ok = __all_sync(0xffffffffu, mbar_wait(half ? &bars.p_full[x] : &bars.p_half[x], par, guard));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t hd = sdesc_add(vd, half * (kBN / 32) * 2048);
              const uint32_t p = tmem + C::col_s(x) + half * (kBN / 4);
#pragma unroll
              for (int kk = 0; kk < kBN / 32; ++kk)
                mma_ts(tmem + C::col_o(x), p + kk * 8, sdesc_add(hd, kk * 2048), C::kIdescPV, acc || half || kk > 0);
            }
            __syncwarp();
          }
          if (!ok) break;
          if (x) ++pc[1];
          else ++pc[0];
          if (last_reader) tc_commit_warp(&bars.kv_empty[st]);
        }
        if (nj < n) {
          const int ki = base + 2 * nj, st = ki % C::kStages;
          ok = __all_sync(0xffffffffu, mbar_wait(&bars.kv_full[st], (ki / C::kStages) & 1, guard));
          if (!ok) break;
          tc_fence_after();
          const uint64_t qd = sdesc_sw128(sq_addr + x * C::kTileBytes, 16, 1024);
          const uint64_t kd = sdesc_sw128(ring_addr + st * C::kTileBytes, 16, 1024);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * C::kBoxBytes + (kk & 3) * 32;
              mma_ss(tmem + C::col_s(x), sdesc_add(qd, off), sdesc_add(kd, off), C::kIdescQK, kk > 0);
            }
          }
          __syncwarp();
          tc_commit_warp(&bars.s_full[x]);
          if (last_reader) tc_commit_warp(&bars.kv_empty[st]);
        } else if (j >= 0 || n == 1) {
          tc_commit_warp(&bars.o_done[x]);     // also of a tile without blocks, which is not a piece ahead either
        }
      }
      base += 2 * n;
    }
    // every issued MMA finishes before TMEM and shared memory are released
    tc_commit_warp(&bars.teardown);
    mbar_wait_drain(&bars.teardown, 0);
  } else if (warp < 4) {
    regs_dec<64>();                         // idle: registers go to the softmax warpgroups
  } else {
    // ============================================================ softmax
    // Register split (launched 384 x 168 = 64512): 128 * 64 + 256 * 216 = 63488.
    regs_inc<216>();
    const int x = (warp - 4) >> 2;          // tile
    const int r = threadIdx.x & 127;        // row within the tile
    const int wrow = (warp & 3) * 32;       // first row of the warp
    const uint32_t lane_base = (uint32_t)wrow << 16;
    const uint32_t tS = tmem + lane_base + C::col_s(x);
    const uint32_t tO = tmem + lane_base + C::col_o(x);
    // a negative scale is its absolute value on negated queries; one of 0 the least that keeps a masked score's -infinity
    const uint32_t sign = a.scale_log2 < 0.f ? 0x80008000u : 0u;
    const float c = fmaxf(fabsf(a.scale_log2), 1e-37f);
    uint32_t sc = 0, od = 0;                // S blocks and outputs taken so far
    int base = 0;
    bool ok = true;
    for (Walk w = s_walk; w.valid && ok; walk_next(a, w)) {
      const Piece& it = w.it;
      const int row0 = it.mt * kPrefixRows + (it.split ? 0 : x * kBM);   // first row of the tile within the unit's head
      const int rows = min(kBM, it.rows - (it.split ? 0 : x * kBM));
      const int nx = it.split ? (it.n + 1 - x) / 2 : it.n;               // blocks of this tile
      int piece, pieces;
      // ------------------------------------------------ the tile's query rows
      // (shared memory is free: the previous piece's MMAs were done before its output was read)
      {
        constexpr int kC = D / 8;                 // 16-byte parts of a row
        constexpr int kPer = 32 / kC;             // rows a warp takes at once
        const int part = lane % kC;
        // the row's place within its batch row moves on by kPer a step: one division
        int gr = row0 + wrow + lane / kC, b = it.p * a.W + gr / a.R, in = gr % a.R;
        uint4 v[kC];
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          const bool real = wrow + i * kPer + lane / kC < rows;
          const long qr = ((long)b * a.Hkv + it.hkv) * a.R + in;
          v[i] = real ? __ldg(reinterpret_cast<const uint4*>(a.q + qr * D + part * 8)) : make_uint4(0, 0, 0, 0);
          for (in += kPer; in >= a.R; in -= a.R) ++b;
        }
        // while they are on their way: which of the unit's pieces this is
        const int Pg = w.g - it.kb, first = w.split.owner(Pg);
        piece = w.team - first;
        pieces = w.split.owner(Pg + w.nb - 1) - first + 1;
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          const int rr = wrow + i * kPer + lane / kC;
          v[i].x ^= sign, v[i].y ^= sign, v[i].z ^= sign, v[i].w ^= sign;
          *reinterpret_cast<uint4*>(sQ + x * C::kTileBytes + (part >> 3) * C::kBoxBytes + rr * 128 +
                                    (((part & 7) ^ (rr & 7)) << 4)) = v[i];
        }
        fence_proxy_async_smem();
        mbar_arrive_warp(&bars.q_full[x]);
      }
      const bool live = wrow < rows;        // a warp without rows only answers the barriers
      float m_run = -INFINITY;              // running max, log2 units (scale folded in)
      float l_run = 0.f;
      for (int i = 0; i < nx; ++i, ++sc) {
        const int j = it.split ? 2 * i + x : i;
        ok = __all_sync(0xffffffffu, mbar_wait(&bars.s_full[x], sc & 1, guard));
        if (!ok) break;
        tc_fence_after();
        const int nvis = it.len - (it.kb + j) * kBN;    // visible keys of the block
        if (nvis < kBN) {
          // V rows past the prefix may hold anything: zeros, so that 0 * V stays 0 in the MMA
          const int vi = base + 2 * j + 1;
          ok = __all_sync(0xffffffffu, mbar_wait(&bars.kv_full[vi % C::kStages], (vi / C::kStages) & 1, guard));
          if (!ok) break;
          if (r >= nvis) {
            uint8_t* vs = sRing + (vi % C::kStages) * C::kTileBytes + r * 128;
#pragma unroll
            for (int b = 0; b < C::kBoxes; ++b)
#pragma unroll
              for (int q = 0; q < 8; ++q) *reinterpret_cast<uint4*>(vs + b * C::kBoxBytes + q * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();         // P V waits for all four warps' P
        }
        if (!live) {
          tc_fence_before();
          mbar_arrive_warp(&bars.p_half[x]);
          mbar_arrive_warp(&bars.p_full[x]);
          continue;
        }
        float mx = -INFINITY;
#pragma unroll 1
        for (int q = 0; q < kBN / kCh; ++q) {
          uint32_t s[kCh];
          load_scores(tS, q, nvis, s);
          const float* sf = reinterpret_cast<const float*>(s);
          float m8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) m8[e] = fmaxf(sf[e], sf[e + 8]);
#pragma unroll
          for (int k = 16; k < kCh; k += 16)
#pragma unroll
            for (int e = 0; e < 8; ++e) m8[e] = max3f(m8[e], sf[k + e], sf[k + 8 + e]);
          mx = max3f(mx, max3f(max3f(m8[0], m8[1], m8[2]), max3f(m8[3], m8[4], m8[5]), m8[6]), m8[7]);
        }
        const float mn = mx * c;
        float alpha = 1.f;
        bool resc = false;
        if (i == 0) {
          m_run = mn;
        } else if (mn > m_run + kRescaleThreshold) {
          alpha = ex2_approx(m_run - mn);
          m_run = mn;
          resc = true;
        }
        const float m_use = m_run == -INFINITY ? 0.f : m_run;
        // O is rescaled first (the commit of S covered the P V before), then P goes out in two halves
        if (__any_sync(0xffffffffu, resc)) {
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld_x32(tO + q * 32, o);
            tmem_ld_wait();
            reg_fence<32>(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st_x32(tO + q * 32, o);
          }
        }
        const uint64_t c2 = f2(c, c), nm2 = f2(-m_use, -m_use);
        uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll 1
        for (int h = 0; h < kBN / kCh; ++h) {
          uint32_t s[kCh];
          load_scores(tS, h, nvis, s);
          const float* sf = reinterpret_cast<const float*>(s);
#pragma unroll
          for (int q = 0; q < kCh / 32; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float t0, t1;
              f2_split(fma2(f2(sf[q * 32 + 2 * k], sf[q * 32 + 2 * k + 1]), c2, nm2), t0, t1);
              const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
              acc[k & 3] = add2(acc[k & 3], f2(p0, p1));
              pk[k] = pack_bf16x2(p0, p1);   // rounded to bf16 (2^-8 of each weight): the type of V, for the MMA
            }
            tmem_st_x16(tS + h * (kCh / 2) + q * 16, pk);
          }
          if (h == kBN / kCh / 2 - 1) {
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive_warp(&bars.p_half[x]);
          }
        }
        float rs0, rs1;
        f2_split(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), rs0, rs1);
        l_run = l_run * alpha + (rs0 + rs1);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(&bars.p_full[x]);
      }
      if (!ok) break;
      base += 2 * it.n;
      // ------------------------------------------------------- the partial
      ok = __all_sync(0xffffffffu, mbar_wait(&bars.o_done[x], od & 1, guard));
      if (!ok) break;
      ++od;
      tc_fence_after();
      const int slot = it.split ? 2 * piece + x : piece;
      const long wr = (((long)it.p * a.Hkv + it.hkv) * a.Rp + row0 + r) * a.slots + slot;
      const bool mine = r < rows && GQA_CHECK(slot >= 0 && slot < a.slots && row0 + r < a.Rp, a.status, a.dbg_line);
      if (nx > 0 && live) {
        // by way of this warp's rows of the query tile (free: the piece's MMAs are done), 32 features at a time, so that
        // a row's 128 bytes go out together
        const long wr0 = wr - (long)lane * a.slots;      // of the warp's first row
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tmem_ld_x32(tO + q * 32, o);
          tmem_ld_wait();
          reg_fence<32>(o);
          const uint32_t buf = smem_u32(sQ + x * C::kTileBytes + (q & (C::kBoxes - 1)) * C::kBoxBytes + wrow * 128);
          if (C::kBoxes == 1) __syncwarp();              // the buffer before is read
#pragma unroll
          for (int k = 0; k < 8; ++k)
            st_shared_v4(buf + lane * 128 + ((k ^ (lane & 7)) << 4), o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int rr = 4 * k + (lane >> 3);
            const uint4 v = ld_shared_v4(buf + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
            if (wrow + rr < rows && GQA_CHECK(slot >= 0 && slot < a.slots && row0 + wrow + rr < a.Rp, a.status, a.dbg_line))
              *reinterpret_cast<uint4*>(a.ws_o + (wr0 + (long)rr * a.slots) * D + q * 32 + (lane & 7) * 4) = v;
          }
        }
        __syncwarp();        // all lanes have read before the next piece's queries go into these rows
        tc_fence_before();   // O is read before the next piece's P V (after its q_full) writes it
      }
      if (mine) a.ws_ml[wr] = make_float2(m_run, l_run);
      if (piece == 0 && x == 0 && r == 0)
        a.counts[((long)it.p * a.Hkv + it.hkv) * a.nrt + it.mt] = it.split ? 2 * pieces : pieces;
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// WPR warps per output row, warp w with the row's pieces w, w + WPR, ...: the weights 2^(M_s - M) under a running
// maximum M, and the weighted sums of the partials and of their L.  What a row costs is a chain of loads (lengths; which
// pieces; their statistics and partials, kAt pieces at a time).
template <int D, int WPR, int kAt>
__global__ void __launch_bounds__(WPR > 8 ? 32 * WPR : 256)
    prefix_merge_kernel(const PrefixArgs p, const OwnArgs a, __nv_bfloat16* o, float* lse) {
  constexpr int V = D / 32;     // features a lane holds
  constexpr int kW = WPR > 8 ? WPR : 8;
  __shared__ float s_acc[WPR > 1 ? kW : 1][D], s_m[kW], s_l[kW];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), part = warp % WPR;
  const long row = (long)blockIdx.x * (kW / WPR) + warp / WPR;   // (b * Hq + h) * Tq + t = (b * Hkv + hkv) * R + rr
  const bool in = row < (long)a.B * a.Hkv * p.R;
  const int rr = (int)(row % p.R), bh = (int)(row / p.R), hkv = bh % a.Hkv, b = bh / a.Hkv, pre = b / p.W;
  const int gr = b % p.W * p.R + rr;
  const long hp = (long)pre * a.Hkv + hkv;
  // the lengths are older than the kernels whose partials are waited for
  const int len = in ? a.cache_lens[b] : -1, m = in ? p.prefix_lens[pre] : -1;
  const bool valid = len >= 0 && len <= a.S && m >= 0 && m <= p.Sp;      // others: reported by the kernels before
  const bool query = valid && len - a.Tq + rr % a.Tq >= 0;
  griddep_wait();               // the kernel that leaves the pieces has ended
  float acc[V] = {};
  float M = -INFINITY, L = 0.f;
  if (query) {
    // the prefix's pieces: attn_prefix's, or pieces of the stream
    const float* po;
    const float2* pml;
    int np = 0, pstep;
    // a kernel that gave up (reported) has not written all of its counts
    const unsigned entries = kOwnMaxWarps + a.Hkv * (a.B * a.nrb + a.P * a.nrbp);
    auto pieces = [&](int2 c) {
      return (unsigned)c.x < entries && (unsigned)c.y <= (unsigned)kOwnMaxWarps && (unsigned)(c.x + c.y) <= entries ? c.y : 0;
    };
    const int2 own = a.counts[(long)a.P * a.Hkv * a.nrbp + (long)bh * a.nrb + rr / a.block];
    if (a.P == 0) {
      pstep = 1;
      const long at = (hp * p.Rp + gr) * p.slots;
      po = p.ws_o + at * D;
      pml = p.ws_ml + at;
      if (m > 0) np = min(max(p.counts[hp * p.nrt + gr / kPrefixRows], 0), p.slots);
    } else {
      pstep = a.rows_ws;
      const int2 c = m > 0 ? a.counts[hp * a.nrbp + gr / a.block] : make_int2(0, 0);
      const long at = (long)c.x * a.rows_ws + gr % a.block;
      po = a.ws_o + at * D;
      pml = a.ws_ml + at;
      np = pieces(c);
    }
    const int n = np + pieces(own);
    const long obase = (long)own.x * a.rows_ws + rr % a.block;
    for (int s0 = part; s0 < n; s0 += WPR * kAt) {
      float2 ml[kAt];
      float v[kAt][V];
#pragma unroll
      for (int k = 0; k < kAt; ++k) {
        const int s = s0 + WPR * k;
        const long at = s < np ? (long)s * pstep : obase + (long)(s - np) * a.rows_ws;
        ml[k] = make_float2(-INFINITY, 0.f);
        if (s >= n) continue;
        ml[k] = (s < np ? pml : a.ws_ml)[at];
        const float* src = (s < np ? po : a.ws_o) + at * D + lane * V;
        if constexpr (V == 4) {
          const float4 x = *reinterpret_cast<const float4*>(src);
          v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(src);
          v[k][0] = x.x, v[k][1] = x.y;
        }
      }
      float top = M;
#pragma unroll
      for (int k = 0; k < kAt; ++k) top = fmaxf(top, ml[k].x);
      // No finite maximum yet: the weights are 0 (2^-inf, not of -inf - -inf).  An L is then 0, of a piece that the row sees
      // nothing of, or NaN, of one whose scores are NaN: those have no part in a maximum, but their L counts.
      const float use = top == -INFINITY ? 0.f : top;
      const float scale = ex2_approx(M - use);
      M = top;
      L *= scale;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] *= scale;
#pragma unroll
      for (int k = 0; k < kAt; ++k) {
        // a piece of weight 0 holds no key that the row sees, and its partial may be anything
        const float w = ex2_approx(ml[k].x - use);
        const bool any = ml[k].x > -INFINITY || ml[k].x != ml[k].x;
        L = fmaf(ml[k].y, w, L);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = any ? fmaf(v[k][e], w, acc[e]) : acc[e];
      }
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int k = 0; k < V; ++k) s_acc[warp][lane * V + k] = acc[k];
    if (lane == 0) {
      s_m[warp] = M;
      s_l[warp] = L;
    }
    __syncthreads();
    if (part > 0) return;
    float top = M;
#pragma unroll
    for (int w = 1; w < WPR; ++w) top = fmaxf(top, s_m[warp + w]);
    const float use = top == -INFINITY ? 0.f : top;
    L = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      const float wk = ex2_approx(s_m[warp + w] - use);     // of a warp without pieces: 0, and so are its sums
      L = fmaf(s_l[warp + w], wk, L);
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] = fmaf(s_acc[warp + w][lane * V + k], wk, acc[k]);
    }
    M = top;
  }
  if (!valid) return;
  const float inv = query ? 1.f / L : 0.f;
  __nv_bfloat16* out = o + row * D + lane * V;
  if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(out) =
        make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  } else {
    *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  }
  if (lane == 0) lse[row] = query ? (M + __log2f(L)) * 0.69314718055994531f : -INFINITY;
}

template <int D, bool PAGED, int NT>
static cudaError_t launch_prefix_dp(const CUtensorMap& k, const CUtensorMap& v, const PrefixArgs& p, const OwnMaps& m,
                                    const OwnArgs& a, cudaStream_t stream) {
  constexpr int kOwn = OwnCfg<D, NT>::kSmemBytes + (int)sizeof(OwnShared<D, NT, 384>);
  constexpr int kSmem = PreCfg<D>::kSmemBytes > kOwn ? PreCfg<D>::kSmemBytes : kOwn;
  static_assert(kSmem + 1024 <= 232448, "shared memory");
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(attn_prefix_kernel<D, PAGED, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[dev] = true;
  }
  prof_begin(kProfPrefix, stream);
  const cudaError_t e = launch_programmatic(attn_prefix_kernel<D, PAGED, NT>, dim3(p.ctas), dim3(384), kSmem, stream, k, v,
                                            m.k, m.v, p, a);
  prof_end(stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D>
static cudaError_t launch_prefix_d(const CUtensorMap& k, const CUtensorMap& v, const PrefixArgs& p, const OwnMaps& m,
                                   const OwnArgs& a, cudaStream_t stream) {
  if (a.block == 8)
    return p.table ? launch_prefix_dp<D, true, 1>(k, v, p, m, a, stream) : launch_prefix_dp<D, false, 1>(k, v, p, m, a, stream);
  return p.table ? launch_prefix_dp<D, true, 2>(k, v, p, m, a, stream) : launch_prefix_dp<D, false, 2>(k, v, p, m, a, stream);
}

cudaError_t launch_attn_prefix(const CUtensorMap& k, const CUtensorMap& v, const PrefixArgs& p, const OwnMaps& m,
                               const OwnArgs& a, cudaStream_t stream) {
  return a.D == 128 ? launch_prefix_d<128>(k, v, p, m, a, stream) : launch_prefix_d<64>(k, v, p, m, a, stream);
}

template <int D>
static cudaError_t launch_merge_d(const PrefixArgs& p, const OwnArgs& a, __nv_bfloat16* o, float* lse, cudaStream_t stream) {
  const long rows = (long)a.B * a.Hkv * p.R;
  // about as many pieces as a row has, if all its keys are there (a host knows the capacities alone)
  constexpr int KT = OwnCfg<D, 1>::KT;
  auto tiles = [](int keys) { return (keys + KT - 1) / KT + kUnitCost; };
  const long total = (long)a.B * a.Hkv * a.nrb * tiles(a.S) + (long)a.P * a.Hkv * a.nrbp * tiles(a.Sp);
  const long share = total / kOwnMaxWarps > kMinShare ? total / kOwnMaxWarps : kMinShare;
  long n = tiles(a.S) / share;
  if (a.P > 0) {
    n += tiles(a.Sp) / share;
  } else {
    const long per = 1 + p.ctas / p.width / ((long)p.P * p.Hkv * p.outer), most = (p.Sp + kBN - 1) / kBN;
    n += (per < most ? per : most) * (p.Rp <= kPrefixRows / 2 ? 2 : 1);
  }
  auto blocks = [&](int per_block) { return dim3((unsigned)((rows + per_block - 1) / per_block)); };
  // Warps a row, as many as leave the blocks in about a wave.  Whole calls, us, 16 / 8 / 4 / 1 warps: 32 rows of 70 pieces
  // 8.0 / 8.9 / 9.0 / 18.6, 128 rows 9.6 / 10.4 / 10.4 / 21.3, 112 rows of 40 (heads of 64) 10.1 / 9.3 / 9.2 / 13.6,
  // 256 rows 13.8 / 11.9 / 11.9 / 23.0, 512 rows 21.0 / 15.9 / 15.9 / 19.3, 1024 rows of 20 31 / 23 / 17.1 / 18.8, 896 rows
  // of 40 (heads of 64) 22.9 / 17.6 / 20.7 / 19.0 and 1024 of 23 - / 19.4 / 15.7 / -, 2048 rows 49 / 31 / 18.9
  // / 18.1, 8192 rows of 7 245 / 195 / 142 / 132.  Heads of 64, 8 warps / 4 for up to 1024 rows where n is above 40: 640
  // rows (32 / 8 heads) over 4096 and 8192 keys 16.6 / 18.5, 17.7 / 19.6; 768 (8 / 2) over 8192 20.4 / 26.4; 896 (14 / 2)
  // 19.8 / 22.4; 1024 (8 / 1) 20.7 / 22.2, (32 / 8) 21.7 / 21.3; where the table is far wider than the prefix (2048 keys of
  // 65536) n tells nothing: 15.5 / 17.1, 18.0 / 20.2, 18.1 / 18.2, 19.0 / 18.2, 17.9 / 15.8.
  if (rows <= 128 && n > 64)
    return launch_programmatic(prefix_merge_kernel<D, 16, 8>, blocks(1), dim3(512), 0, stream, p, a, o, lse);
  if (rows <= 512 || (D == 64 && rows <= 1024 && n > 40))
    return launch_programmatic(prefix_merge_kernel<D, 8, 8>, blocks(1), dim3(256), 0, stream, p, a, o, lse);
  if (rows <= 1536) return launch_programmatic(prefix_merge_kernel<D, 4, 4>, blocks(2), dim3(256), 0, stream, p, a, o, lse);
  return launch_programmatic(prefix_merge_kernel<D, 1, 8>, blocks(8), dim3(256), 0, stream, p, a, o, lse);
}

cudaError_t launch_prefix_merge(const PrefixArgs& p, const OwnArgs& a, __nv_bfloat16* o, float* lse, cudaStream_t stream) {
  prof_begin(kProfPrefixMerge, stream);
  const cudaError_t e = a.D == 128 ? launch_merge_d<128>(p, a, o, lse, stream) : launch_merge_d<64>(p, a, o, lse, stream);
  prof_end(stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gqa
