// stream.cuh -- one stream of tiles, shared out evenly between a grid's warps:
// the rows of a batch, each contributing positions(row) to the stream, and the
// part of it that a warp takes.
#pragma once

#include "sm103.cuh"

namespace gqa {

// j / d for 0 <= j < 2^31 and d >= 1 by a multiplication: with s = ceil(log2 d) and m = ceil(2^(31+s) / d) < 2^32 the
// error m d - 2^(31+s) is below d <= 2^s, so floor(j m / 2^(31+s)) is exact; umulhi takes 32 of the 31 + s bits.
struct FastDiv {
  int d;
  unsigned mul, shift;
  __host__ static FastDiv of(int d) {
    FastDiv f{d, 0, 0};
    if (d <= 1) return f;
    while ((1L << f.shift) < d) ++f.shift;
    f.mul = (unsigned)(((1ULL << (31 + f.shift)) + d - 1) / d);
    --f.shift;
    return f;
  }
  __device__ __forceinline__ int operator()(int j) const { return d == 1 ? j : (int)(__umulhi((unsigned)j, mul) >> shift); }
};

// Where position j of a batch row is: the number of its row in the planes [pages, heads, page_size] of a cache, -1 in a
// page outside the pool.
struct Slots {
  const int* table;      // of the batch row, nullptr: contiguous
  int num_pages, b;
  FastDiv page;
  long heads, h;
  __device__ __forceinline__ long operator()(int j) const {
    int pg = b, r = j;
    if (table) {
      const int i = page(j);
      r = j - i * page.d;
      pg = table[i];
      if (pg < 0 || pg >= num_pages) return -1;
    }
    return ((long)pg * heads + h) * page.d + r;
  }
};

// `total` positions in `parts` runs, run i from floor(i total / parts) on, so that the runs of equal parts of the whole
// end with them.  32-bit divisions only (a 64-bit one takes as long as a load): with total = q parts + r that is
// i q + floor(i r / parts), parts < 2^15.
struct EvenSplit {
  int total, parts, q, r;
  __device__ __forceinline__ static EvenSplit of(int total, int parts) {
    EvenSplit e{total, parts, 0, 0};
    if (parts > 0) e.q = total / parts, e.r = total - e.q * parts;
    return e;
  }
  __device__ __forceinline__ int begin(int i) const { return i * q + (int)((unsigned)(i * r) / (unsigned)parts); }
  // The run that has position x: an estimate, off by one at most, then exactly.
  __device__ __forceinline__ int owner(int x) const {
    int i = min(parts - 1, (int)((float)x / (float)total * (float)parts));
    while (begin(i) > x) --i;
    while (begin(i + 1) <= x) ++i;
    return i;
  }
};

// Positions [v0, v1) are warp gw's; `row` holds v0 and begins at position `at`.  v1 <= v0: none.
struct StreamShare {
  EvenSplit split;      // between the warps in use
  int v0, v1, row, at;
};

// All threads of a block of THREADS call this; s_sum [THREADS / 32], s_pre [THREADS] in shared memory.  A warp takes at
// least min_share positions, if there are fewer than `warps` times that.  The total is below 2^31 - 2^12.
template <int THREADS, class Positions>
__device__ __forceinline__ StreamShare stream_share(int rows, int gw, int warps, int min_share, int* s_sum, int* s_pre,
                                                    Positions positions) {
  constexpr int kWarps = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(~0u, tid >> 5, 0);
  StreamShare sh{{}, 0, 0, -1, 0};
  auto take = [&](int total) {
    sh.split = EvenSplit::of(total, min(warps, (total + min_share - 1) / min_share));
    if (gw < sh.split.parts) {
      sh.v0 = sh.split.begin(gw);
      sh.v1 = sh.split.begin(gw + 1);
    }
  };
  if (rows > THREADS) {     // a pass for the total first
    int mine = 0;
    for (int i = tid; i < rows; i += THREADS) mine += positions(i);
    mine = __reduce_add_sync(~0u, mine);
    if (lane == 0) s_sum[warp] = mine;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += s_sum[w];
    take(total);
  }
  int before = 0;
  for (int i0 = 0; i0 < rows; i0 += THREADS) {
    int inc = i0 + tid < rows ? positions(i0 + tid) : 0;      // inclusive sums of THREADS rows
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(~0u, inc, d);
      if (lane >= d) inc += x;
    }
    if (rows > THREADS) __syncthreads();     // the sums before are read
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int x = s_sum[w];
      if (w < warp) inc += x;
      all += x;
    }
    s_pre[tid] = inc;
    __syncthreads();
    if (rows <= THREADS) take(all);
    if (sh.v0 < sh.v1 && sh.row < 0 && sh.v0 < before + all) {
      const int x = sh.v0 - before;      // the first row whose inclusive sum is above
      int lo = 0, hi = min(THREADS, rows - i0) - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_pre[mid] > x) hi = mid;
        else lo = mid + 1;
      }
      sh.row = i0 + lo;
      sh.at = before + (lo ? s_pre[lo - 1] : 0);
    }
    before += all;
  }
  // the same in a warp, told so
  sh.v0 = __shfl_sync(~0u, sh.v0, 0);
  sh.v1 = __shfl_sync(~0u, sh.v1, 0);
  sh.row = __shfl_sync(~0u, sh.row, 0);
  sh.at = __shfl_sync(~0u, sh.at, 0);
  return sh;
}

}  // namespace gqa
