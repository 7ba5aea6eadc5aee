// cache_evict.cu -- the attention weight that cached keys receive, and cutting
// a cache down to the keys that received most, for sm_103a.
//
// cache_weights  w_j += sum over a step's queries that see key j of
//   exp(scale q . k_j - lse), from w_j = 0 for its Tq new keys: K is read once (memory bounds it for few
//   queries), the scores are warp-level MMAs with 16 keys as M and 8 query rows
//   as N.  A dot product does not care for the order of its terms, so a lane
//   takes whole 16-byte parts of a key row as its share of the k index and
//   needs neither shared memory nor shuffles to bring them into place; the
//   query fragments follow the same order.  E4M3 and 4-bit codes are widened to
//   f16 in registers (exactly: e2m1 * e4m3 has 6 significant bits); query rows
//   then are f16 too, scaled by a power of two a row, exact down to 2^-31 of
//   the row's largest feature.  One lane group adds up a key's weight in a
//   fixed order: the same call gives the same bits.
//
// evict_select   one CTA a (row, K/V head): the budget-th largest weight by
//   radix selection over the weights' bits, then the kept positions in order.
// evict_move     the kept rows of every plane to the front.  Row i comes from
//   position src_i >= i, and src grows, so going up in chunks a chunk's rows
//   are read before any is overwritten; planes and column slices of a row are
//   independent of each other and go to CTAs of their own.
#include <cuda_fp16.h>

#include "cache_ops.h"
#include "fp4.cuh"
#include "kernels.h"
#include "sm103.cuh"

namespace gqa {

namespace {

constexpr int kWWarps = 8;
constexpr int kWKeys = 32 * kWWarps;   // keys a CTA takes at once
constexpr int kWRows = 64;             // query rows in shared memory at once

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

template <int D, CacheFmt F>
struct KeyRow {
  using P = KeyPart<D, F>;
  uint32_t w[P::kWords];
  uint32_t sf;      // 4-bit: the block scales of the lane's features
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < P::kWords; ++i) w[i] = 0;
    sf = 0;
  }
  __device__ __forceinline__ void load(const WeightsArgs& a, long row, int tig) {
    const uint8_t* p = a.k + row * P::kRowBytes;
#pragma unroll
    for (int i = 0; i < P::kParts; ++i) {
      if constexpr (P::kBytes == 16) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + (tig + 4 * i) * 16));
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p + tig * 8));
        w[0] = v.x, w[1] = v.y;
      }
    }
    if constexpr (F == kCacheQ4) {
      if constexpr (D == 128) sf = __ldg(reinterpret_cast<const uint16_t*>(a.ksf + row * 8) + tig);
      else sf = __ldg(a.ksf + row * 4 + tig);
    }
  }
  // The 16-bit pairs (features 4 s, +1) and (+2, +3) of step s.
  __device__ __forceinline__ void step(int s, uint32_t& lo, uint32_t& hi) const {
    if constexpr (F == kCacheBf16) {
      lo = w[2 * s];
      hi = w[2 * s + 1];
    } else if constexpr (F == kCacheE4m3) {
      lo = e4m3x2_to_f16(w[s] & 0xffffu);
      hi = e4m3x2_to_f16(w[s] >> 16);
    } else {
      uint32_t h[4];      // 8 codes: steps 2 s', 2 s' + 1; the unused half is dropped by the compiler
      e2m1x8_to_f16(w[s / 2], h);
      const uint32_t byte = (sf >> (s / 4 * 8)) & 0xffu, two = e4m3x2_to_f16(byte | byte << 8);
      lo = hmul2_u(h[2 * (s & 1)], two);
      hi = hmul2_u(h[2 * (s & 1) + 1], two);
    }
  }
};

// The page of position j of batch row b, -1 where the table names none.
__device__ __forceinline__ int page_of(const int* table, int max_pages, int num_pages, int b, int page) {
  if (!table) return b;
  const int e = table[(long)b * max_pages + page];
  return e >= 0 && e < num_pages ? e : -1;
}

template <int D, CacheFmt F>
__global__ void __launch_bounds__(32 * kWWarps) cache_weights_kernel(const WeightsArgs a) {
  using P = KeyPart<D, F>;
  constexpr int kSteps = D / 16;
  constexpr bool f16 = F != kCacheBf16;
  __shared__ uint2 s_q[kWRows / 8][kSteps][32];     // query fragments, by lane
  __shared__ float2 s_c[kWRows];                    // score factor and -lse, in log2 units; factor NaN: no query
  __shared__ int s_t[kWRows];                       // query position of the row
  griddep_wait();
  griddep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const int bh = (int)(blockIdx.x % (unsigned)(a.B * a.Hkv)), b = bh / a.Hkv, hkv = bh % a.Hkv;
  const int c0 = (int)(blockIdx.x / (unsigned)(a.B * a.Hkv)) * kWKeys;
  const int len = a.cache_lens[b];
  if (len < 0 || len > a.S) {
    if (c0 == 0 && threadIdx.x == 0) atomicCAS(a.status, 0, kDevBadSeqlens);
    return;
  }
  if (c0 >= len) return;
  // the lane's four keys: 8 m + g of the warp's 32, m = 0..3
  const int k0 = c0 + warp * 32;
  KeyRow<D, F> kr[4];
  bool bad = false;
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int j = k0 + 8 * m + g;
    kr[m].zero();
    if (j < len) {
      const int page = page_of(a.block_table, a.max_pages, a.num_pages, b, j / a.page_size);
      bad |= page < 0;
      if (page >= 0) kr[m].load(a, ((long)page * a.Hkv + hkv) * a.page_size + j % a.page_size, tig);
    }
  }
  if (bad) atomicCAS(a.status, 0, kDevBadPage);
  // the key whose weight this lane writes
  const int jw = k0 + 8 * tig + g;
  float* wp = nullptr;
  float w = 0.f;
  if (jw < len) {
    const int page = page_of(a.block_table, a.max_pages, a.num_pages, b, jw / a.page_size);
    if (page >= 0) {
      wp = a.weights + ((long)page * a.Hkv + hkv) * a.page_size + jw % a.page_size;
      w = jw < len - a.Tq ? *wp : 0.f;     // the step's new keys had no weight before
    }
  }
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  for (int r0 = 0; r0 < a.R; r0 += kWRows) {
    const int nt = min(kWRows, (a.R - r0 + 7) & ~7) / 8;
    if (r0) __syncthreads();
    // query rows r0 .. into fragments, a warp a row
    for (int r = warp; r < 8 * nt; r += kWWarps) {
      const bool real = r0 + r < a.R;
      const long qrow = (long)bh * a.R + r0 + r;
      int e = 0;
      if (real && f16) {
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) mx = fmaxf(mx, fabsf(__bfloat162float(a.q[qrow * D + i * 32 + lane])));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (mx > 0.f && mx < INFINITY) e = 15 - ilogbf(mx) - 1;     // the largest feature goes to [2^14, 2^15)
      }
      for (int i = lane; i < kSteps * 4; i += 32) {
        const int s = i / 4, t = i % 4;
        uint2 v = make_uint2(0, 0);
        if (real) {
          v = *reinterpret_cast<const uint2*>(a.q + qrow * D + P::feature(s, t));
          if constexpr (f16) {
            const float2 x = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&v.x));
            const float2 y = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&v.y));
            v.x = pack_f16x2(ldexpf(x.x, e), ldexpf(x.y, e));
            v.y = pack_f16x2(ldexpf(y.x, e), ldexpf(y.y, e));
          }
        }
        s_q[r / 8][s][r % 8 * 4 + t] = v;
      }
      if (lane == 0) {
        const float lse = real ? a.lse[qrow] : -INFINITY;
        s_c[r] = lse == -INFINITY ? make_float2(NAN, 0.f)
                                  : make_float2(ldexpf(a.scale_log2, -e), -lse * 1.4426950408889634f);
        s_t[r] = (r0 + r) % a.Tq;
      }
    }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      float acc[2][4] = {};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const uint2 q = s_q[t][s][lane];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t f[4];
          kr[2 * m].step(s, f[0], f[2]);
          kr[2 * m + 1].step(s, f[1], f[3]);
          mma_16816(acc[m], f, q.x, q.y, f16);
        }
      }
      // acc[m][0, 1]: key 16 m + g, rows 2 tig, 2 tig + 1; [2, 3]: key 16 m + 8 + g
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * t + 2 * tig + i;
        const float2 c = s_c[r];
        const bool query = !(c.x != c.x);
        const int lim = len - a.Tq + s_t[r] - k0;      // last key the row sees
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float p = ex2_approx(fmaf(acc[m / 2][2 * (m & 1) + i], c.x, c.y));
          sum[m] += query && 8 * m + g <= lim ? p : 0.f;
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
  if (wp) *wp = w + mine;
}

}  // namespace

cudaError_t launch_cache_weights(const WeightsArgs& a, CacheFmt fmt, int sms, cudaStream_t stream) {
  (void)sms;
  const dim3 grid((unsigned)((long)a.B * a.Hkv * ((a.S + (long)kWKeys - 1) / kWKeys))), block(32 * kWWarps);
  prof_begin(kProfWeights, stream);
  cudaError_t e;
#define GQA_WEIGHTS(F)                                                                              \
  (a.D == 128 ? launch_programmatic(cache_weights_kernel<128, F>, grid, block, 0, stream, a)        \
              : launch_programmatic(cache_weights_kernel<64, F>, grid, block, 0, stream, a))
  e = fmt == kCacheBf16 ? GQA_WEIGHTS(kCacheBf16) : fmt == kCacheE4m3 ? GQA_WEIGHTS(kCacheE4m3) : GQA_WEIGHTS(kCacheQ4);
#undef GQA_WEIGHTS
  prof_end(stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

namespace {

constexpr int kSelThreads = 1024;

// Whole numbers in the weights' order: NaN above all, -0 = 0.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ int s_hist[256];
  __shared__ int s_gt[32], s_eq[32];
  __shared__ uint32_t s_pre;
  __shared__ int s_need;
  griddep_wait();
  griddep_launch();
  const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = a.cache_lens[b];
  int* kept = a.kept + (long)blockIdx.x * a.budget;
  const bool valid = n >= 0 && n <= a.S;
  if (h == 0 && tid == 0) {
    if (!valid) atomicCAS(a.status, 0, kDevBadSeqlens);
    a.lens_out[b] = valid ? min(n, a.budget) : n;
  }
  if (!valid || n <= a.budget) {
    for (int i = tid; i < a.budget; i += kSelThreads) kept[i] = valid && i < n ? i : -1;
    return;
  }
  // n > budget >= first + recent: of the positions [lo, hi) the `need` largest are kept
  const int lo = a.first, hi = n - a.recent;
  int need = a.budget - a.first - a.recent;
  bool bad = false;
  auto key = [&](int j) {
    const int page = page_of(a.block_table, a.max_pages, a.num_pages, b, j / a.page_size);
    bad |= page < 0;
    return page < 0 ? 0u : order_of(a.weights[((long)page * a.Hkv + h) * a.page_size + j % a.page_size]);
  };
  uint32_t pre = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) s_hist[tid] = 0;
    __syncthreads();
    const uint32_t above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int j = lo + tid; j < hi; j += kSelThreads) {
      const uint32_t k = key(j);
      if ((k & above) == pre) atomicAdd(&s_hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // bins 8 lane .. 8 lane + 7; the bin where the count from the top reaches `need`
      int c[8], t = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) t += c[i] = s_hist[8 * lane + i];
      int above_lane = t;     // keys in bins of this and higher lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_down_sync(0xffffffffu, above_lane, o);
        if (lane + o < 32) above_lane += y;
      }
      int from = above_lane - t;
#pragma unroll
      for (int i = 7; i >= 0; --i) {
        if (from < need && need <= from + c[i]) {
          s_pre = pre | (uint32_t)(8 * lane + i) << shift;
          s_need = need - from;
        }
        from += c[i];
      }
      if (need == 0 && lane == 0) {
        s_pre = 0xffffffffu;
        s_need = 0;
      }
    }
    __syncthreads();
    pre = s_pre;
    need = s_need;
    if (need == 0) break;
  }
  // kept: keys above `pre`, and the first `need` equal to it.  A warp takes a run of positions: count, then write.
  const bool none = a.budget == a.first + a.recent;
  const int run = ((hi - lo + 31) / 32 + 31) & ~31, w0 = lo + warp * run, w1 = min(w0 + run, hi);
  int gt = 0, eq = 0;
  for (int j0 = w0; j0 < w1; j0 += 32) {
    const int j = j0 + lane;
    const uint32_t k = j < w1 ? key(j) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, j < w1 && !none && k > pre));
    eq += __popc(__ballot_sync(0xffffffffu, j < w1 && !none && k == pre));
  }
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  gt = eq = 0;
  for (int i = 0; i < warp; ++i) {
    gt += s_gt[i];
    eq += s_eq[i];
  }
  for (int j0 = w0; j0 < w1; j0 += 32) {
    const int j = j0 + lane;
    const uint32_t k = j < w1 ? key(j) : 0u;
    const unsigned bg = __ballot_sync(0xffffffffu, j < w1 && !none && k > pre);
    const unsigned be = __ballot_sync(0xffffffffu, j < w1 && !none && k == pre);
    const unsigned below = (1u << lane) - 1u;
    const int g = gt + __popc(bg & below), e = eq + __popc(be & below);
    if ((bg >> lane & 1u) || ((be >> lane & 1u) && e < need)) kept[a.first + g + min(e, need)] = j;
    gt += __popc(bg);
    eq += __popc(be);
  }
  for (int i = tid; i < a.first; i += kSelThreads) kept[i] = i;
  for (int i = tid; i < a.recent; i += kSelThreads) kept[a.budget - a.recent + i] = n - a.recent + i;
  if (bad) atomicCAS(a.status, 0, kDevBadPage);
}

constexpr int kMoveThreads = 256, kMoveRows = 4;   // rows a thread moves a piece of at once

template <typename V>
__device__ __forceinline__ void move_rows(const EvictArgs& a, const EvictPlane& pl, int slice, int b, int h) {
  const int tpr = pl.slice_bytes / (int)sizeof(V), rpi = kMoveThreads / tpr;
  const int sub = threadIdx.x / tpr;
  const bool active = sub < rpi;
  const long col = (long)slice * pl.slice_bytes + (threadIdx.x % tpr) * (long)sizeof(V);
  const int* kept = a.kept + ((long)b * a.Hkv + h) * a.budget;
  uint8_t* base = static_cast<uint8_t*>(pl.p) + col;
  auto at = [&](int j) -> V* {
    const int page = page_of(a.block_table, a.max_pages, a.num_pages, b, j / a.page_size);
    return page < 0 ? nullptr
                    : reinterpret_cast<V*>(base + (((long)page * a.Hkv + h) * a.page_size + j % a.page_size) * pl.row_bytes);
  };
  for (int c0 = a.first; c0 < a.budget; c0 += rpi * kMoveRows) {
    V v[kMoveRows];
    bool go[kMoveRows];
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const int d = c0 + u * rpi + sub;
      go[u] = false;
      if (active && d < a.budget) {
        const int src = kept[d];
        const V* s = src > d ? at(src) : nullptr;
        if (s) {
          v[u] = *s;
          go[u] = true;
        }
      }
    }
    __syncthreads();      // the chunk's rows are read before any of them is overwritten
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      if (!go[u]) continue;
      V* d = at(c0 + u * rpi + sub);
      if (d) *d = v[u];
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
  griddep_wait();
  griddep_launch();
  const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
  const int n = a.cache_lens[b];
  if (n <= a.budget || n > a.S) return;
  int slice = blockIdx.y, i = 0;
  while (slice >= a.planes[i].slices) slice -= a.planes[i++].slices;
  const EvictPlane& pl = a.planes[i];
  if (pl.piece == 16) move_rows<uint4>(a, pl, slice, b, h);
  else if (pl.piece == 8) move_rows<uint2>(a, pl, slice, b, h);
  else move_rows<uint32_t>(a, pl, slice, b, h);
}

}  // namespace

cudaError_t launch_cache_evict(EvictArgs a, cudaStream_t stream) {
  int slices = 0;
  for (int i = 0; i < a.n_planes; ++i) {
    EvictPlane& p = a.planes[i];
    p.piece = p.row_bytes % 16 == 0 ? 16 : p.row_bytes % 8 == 0 ? 8 : 4;
    const int pieces = p.row_bytes / p.piece;
    int t = 1;                                   // pieces of a row that a CTA moves: at most 8
    for (int d = 1; d <= 8; ++d)
      if (pieces % d == 0) t = d;
    p.slice_bytes = t * p.piece;
    p.slices = pieces / t;
    slices += p.slices;
  }
  const dim3 grid((unsigned)(a.B * a.Hkv));
  prof_begin(kProfEvictSelect, stream);
  cudaError_t e = launch_programmatic(evict_select_kernel, grid, dim3(kSelThreads), 0, stream, a);
  prof_end(stream);
  if (e != cudaSuccess) return e;
  prof_begin(kProfEvictMove, stream);
  e = launch_programmatic(evict_move_kernel, dim3(grid.x, (unsigned)slices), dim3(kMoveThreads), 0, stream, a);
  prof_end(stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gqa
