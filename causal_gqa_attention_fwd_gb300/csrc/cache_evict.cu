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
// evict  a cluster of CTAs a (row, K/V head): each keeps a run of the weights in
//   shared memory; the budget-th largest by radix selection over the weights'
//   bits (11, 11, 10, histograms added up through distributed shared memory),
//   then the kept positions in order, then the rows of every plane to the front.
//   Row i comes from position src_i >= i, and src grows, so going up in chunks a
//   chunk's rows are read before any is overwritten.
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

constexpr int kEvThreads = 512;      // two CTAs an SM at 64 registers
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kBins = 2048;          // of a pass over 11 bits (the last: 10)
constexpr int kMoveRows = 6;         // rows a thread has parts of on the way between reading and writing
constexpr int kPlaceBytes = kMoveRows * kEvThreads * 16;
constexpr int kKeyBytes = 80 << 10;  // weights a CTA keeps in shared memory; a longer share is read again each pass
constexpr int kAlone = 8192;         // positions up to which each CTA selects by itself (weights and list in 64 KB)

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

// Where position j of (row b, head h) is: the number of its slot row in a plane, -1 in a page outside the pool.
struct Slots {
  const int* table;      // of row b, nullptr: contiguous
  int num_pages, page_size, b;
  unsigned mul, shift;   // j / page_size = umulhi(j, mul) >> shift, page_size > 1
  long heads, h;
  __device__ __forceinline__ long operator()(int j) const {
    int page = b, r = j;
    if (table) {
      const int i = page_size == 1 ? j : (int)(__umulhi((unsigned)j, mul) >> shift);
      r = j - i * page_size;
      page = table[i];
      if (page < 0 || page >= num_pages) return -1;
    }
    return ((long)page * heads + h) * page_size + r;
  }
};

// A thread's part of every row that it moves: 16, 8 or 4 bytes of one plane, by way of its place in shared memory.
struct Part {
  uint8_t* base;      // of the plane, at the part
  int row_bytes, size;
  __device__ __forceinline__ void load(uint32_t to, long slot) const {
    const uint8_t* p = base + slot * row_bytes;
    if (size == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p) : "memory");
    else if (size == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(p) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(p) : "memory");
  }
  __device__ __forceinline__ void store(const uint4* from, long slot) const {
    uint8_t* p = base + slot * row_bytes;
    if (size == 16) *reinterpret_cast<uint4*>(p) = *from;
    else if (size == 8) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(from);
    else *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(from);
  }
};
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Moves the rows list[d] -> d, d in [first, budget), of every plane.  A thread has one part of a row (a row's parts of all
// planes lie on neighbouring threads), kMoveRows of them on the way at a time.  Row d may be written once whatever is kept
// of position d has been read, that is all rows i with list[i] <= d.  So the rows go in phases [c0, c1): if list[c0] lies
// further behind c0 than the threads' places reach, all rows up to position list[c0] are free to go one by one, for every
// source in front of that position belongs to an earlier phase; otherwise as many as there are places are read before any
// is written.
__device__ __forceinline__ void move_rows(const EvictArgs& a, const Slots& slot_of, const int* list, uint4* places, int rank,
                                          int ranks) {
  // the first row that moves: list[d] - d never falls
  int d_lo = a.first, d_hi = a.budget;
  while (d_lo < d_hi) {
    const int mid = (d_lo + d_hi) >> 1;
    if (list[mid] > mid) d_hi = mid;
    else d_lo = mid + 1;
  }
  for (int p0 = 0; p0 < a.parts; p0 += kEvThreads) {     // more parts than threads: some of each row's at a time
    const int ppr = min(a.parts - p0, kEvThreads), rpi = kEvThreads / ppr, sub = threadIdx.x / ppr;
    Part part{nullptr, 0, 0};
    int q = p0 + threadIdx.x % ppr;
    for (int i = 0; i < a.n_planes; ++i) {
      const EvictPlane& pl = a.planes[i];
      const int size = pl.row_bytes % 16 == 0 ? 16 : pl.row_bytes % 8 == 0 ? 8 : 4, n = pl.row_bytes / size;
      if (q >= 0 && q < n) part = Part{static_cast<uint8_t*>(pl.p) + q * size, pl.row_bytes, size};
      q -= n;
    }
    const int step = ranks * rpi, hold = step * kMoveRows;
    uint4* mine = places + threadIdx.x;                  // place u: kEvThreads further on
    auto source = [&](int d, int c1) { return sub < rpi && d < c1 ? list[d] : -1; };
    auto read = [&](int u, int src) {
      const long s = src >= 0 ? slot_of(src) : -1;
      if (s >= 0) part.load(smem_u32(mine + u * kEvThreads), s);
      copies_commit();
      return s >= 0;
    };
    auto write = [&](int u, int d) {
      const long t = slot_of(d);
      if (t >= 0) part.store(mine + u * kEvThreads, t);
    };
    for (int c0 = d_lo; c0 < a.budget;) {
      const int free_to = min(list[c0], a.budget);
      const bool held = free_to < c0 + hold && free_to < a.budget;
      const int c1 = held ? min(c0 + hold, a.budget) : free_to;
      int d = c0 + rank * rpi + sub, src[kMoveRows];
      unsigned go = 0;
#pragma unroll
      for (int u = 0; u < kMoveRows; ++u) src[u] = source(d + u * step, c1);
#pragma unroll
      for (int u = 0; u < kMoveRows; ++u) go |= (unsigned)read(u, src[u]) << u;
      if (held) {
        copies_wait<0>();
        cluster_sync();
#pragma unroll
        for (int u = 0; u < kMoveRows; ++u)
          if (go >> u & 1u) write(u, d + u * step);
      } else {
#pragma unroll
        for (int u = 0; u < kMoveRows; ++u) src[u] = source(d + hold + u * step, c1);
        while (go) {
          unsigned next = 0;
#pragma unroll
          for (int u = 0; u < kMoveRows; ++u) {
            copies_wait<kMoveRows - 1>();                 // the oldest has landed
            if (go >> u & 1u) write(u, d + u * step);
            next |= (unsigned)read(u, src[u]) << u;
            src[u] = source(d + 2 * hold + u * step, c1);
          }
          d += hold;
          go = next;
        }
        copies_wait<0>();
        if (c1 < a.budget) cluster_sync();   // the phase's rows are read before later ones are written over them
      }
      c0 = c1;
    }
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
  int* list = a.shared_select ? kept : reinterpret_cast<int*>(s_keys) + max(a.key_bytes, kPlaceBytes) / 4;
  bool bad = false;
  const Slots slot_of{a.block_table ? a.block_table + (long)b * a.max_pages : nullptr, a.num_pages, a.page_size, b,
                      a.div_mul, a.div_shift, a.Hkv, h};
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
  if (any) {
#pragma unroll 4
    for (int j0 = w0; j0 < w1; j0 += 32) {
      const int j = j0 + lane;
      const uint32_t k = j < w1 ? key(j) & mask : 0u;
      gt += j < w1 && k > thr;
      eq += j < w1 && k == thr;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
  }
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
    if ((bg >> lane & 1u) || ((be >> lane & 1u) && e < need)) list[a.first + g + min(e, need)] = j;
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
  move_rows(a, slot_of, list, reinterpret_cast<uint4*>(s_keys), rank, ranks);
}

}  // namespace

cudaError_t launch_cache_evict(EvictArgs a, cudaStream_t stream) {
  const long units = (long)a.B * a.Hkv;
  // a cluster a unit, as large as leaves all CTAs resident (two an SM) and 256 positions a CTA
  a.cluster = 8;
  while (a.cluster > 1 && (units * a.cluster > 304 || a.S < 256L * a.cluster)) a.cluster /= 2;
  a.shared_select = a.cluster > 1 && a.S > kAlone;
  const long run = a.shared_select ? ((long)a.S + a.cluster - 1) / a.cluster : a.S;
  a.key_bytes = run * 4 <= kKeyBytes ? (int)(run * 4 + 15) / 16 * 16 : 0;
  int smem = a.key_bytes > kPlaceBytes ? a.key_bytes : kPlaceBytes;
  if (!a.shared_select) {      // the list beside the weights; rows too long for that: one CTA, the list in memory
    if (a.S <= kAlone) smem += (a.budget < a.S ? a.budget : a.S) * 4;
    else a.shared_select = 1;
  }
  // j / page_size for 0 <= j < 2^31 by a multiplication: with s = ceil(log2 p) and m = ceil(2^(31+s) / p) < 2^32 the error
  // m p - 2^(31+s) is below p <= 2^s, so floor(j m / 2^(31+s)) is exact; umulhi takes 32 of the bits
  a.div_shift = 0;
  while ((1L << a.div_shift) < a.page_size) ++a.div_shift;
  a.div_mul = a.page_size > 1 ? (unsigned)(((1ULL << (31 + a.div_shift)) + a.page_size - 1) / a.page_size) : 0;
  a.div_shift -= a.page_size > 1;
  a.parts = 0;
  for (int i = 0; i < a.n_planes; ++i) {
    const int rb = a.planes[i].row_bytes;
    a.parts += rb / (rb % 16 == 0 ? 16 : rb % 8 == 0 ? 8 : 4);
  }
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeyBytes + 8192);
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
