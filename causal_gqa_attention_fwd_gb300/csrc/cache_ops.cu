// cache_ops.cu -- the operators around a KV cache other than attention itself:
// the cache plan (block tables, slots, positions), rotary rows and tables,
// appending keys and values, reading 4-bit slots back.  All of them move a few
// bytes per element and compute little: what bounds them is memory traffic at
// prompt sizes and the launch at decode sizes.
#include "cache_ops.h"
#include "fp4.cuh"
#include "kernels.h"
#include "sm103.cuh"

namespace gqa {

namespace {

// ------------------------------------------------------------- cache plan
// slot = page * page_size + row of each new token, by integer arithmetic: a scan
// over the requests, then a search per token.  Bound by the launch and a few
// dependent loads: in a captured graph 64 requests of one token 4.3 us, 512 with
// 256k tokens in all (2.2 MB) 6.5 us; called from Python 6.0 and 7.7.
// One launch and no exchange between CTAs: every CTA scans all B requests
// (pages needed, new tokens) into shared memory, then fills its share of the
// tokens and of the block-table rows.  Slots come from the free list directly
// rather than from the table entries another CTA may be writing.
constexpr int kPlanThreads = 512;

struct PlanReq {
  long len, add;   // valid request: keys held, tokens added
  bool valid;
};

__device__ __forceinline__ PlanReq plan_req(const PlanArgs& a, int b) {
  PlanReq r;
  r.len = a.cache_lens[b];
  r.add = a.new_lens[b];
  r.valid = r.len >= 0 && r.add >= 0 && r.len + r.add <= (long)a.max_pages * a.page_size;
  return r;
}

// Pages of the keys of a valid request (below 2^31, as page_size is).
__device__ __forceinline__ int pages_of(long keys, int page_size) {
  return (int)(((unsigned)keys + (unsigned)page_size - 1u) / (unsigned)page_size);
}

// kPer: tokens a thread takes, kPlanThreads apart, so that their searches and
// look-ups overlap.
template <int kPer>
__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const PlanArgs a) {
  extern __shared__ int plan_smem[];
  int* cu = plan_smem;              // [B + 1] first token of each request
  int* first = plan_smem + a.B + 1; // [B] its first page's index in free_pages, -1: refused
  __shared__ long warp_need[kPlanThreads / 32], warp_add[kPlanThreads / 32];
  __shared__ int end_cursor;
  griddep_wait();     // launched while the kernel before drains, as all kernels here
  griddep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cursor = a.cursor ? *a.cursor : 0;
  const bool cursor_ok = cursor >= 0 && cursor <= a.num_free;
  if (tid == 0) end_cursor = cursor;
  long need_before = 0, add_before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    PlanReq r{0, 0, false};
    long need = 0, add = 0;
    if (b < a.B) {
      r = plan_req(a, b);
      add = r.add > 0 ? r.add : 0;
      if (r.valid) need = pages_of(r.len + r.add, a.page_size) - pages_of(r.len, a.page_size);
    }
    long in = need, ia = add;   // inclusive sums over the warp, then over the warps
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long x = __shfl_up_sync(~0u, in, d), y = __shfl_up_sync(~0u, ia, d);
      if (lane >= d) in += x, ia += y;
    }
    __syncthreads();            // the previous round's sums are read
    if (lane == 31) warp_need[warp] = in, warp_add[warp] = ia;
    __syncthreads();
    long all_need = 0, all_add = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) in += warp_need[w], ia += warp_add[w];
      all_need += warp_need[w], all_add += warp_add[w];
    }
    in += need_before, ia += add_before;
    need_before += all_need, add_before += all_add;
    if (b < a.B) {
      const bool tokens_fit = ia <= a.total;
      const bool pages_fit = in == 0 || (cursor_ok && in <= (long)a.num_free - cursor);
      const bool ok = r.valid && tokens_fit && pages_fit;
      const long at = ia - add;
      cu[b] = (int)(at < a.total ? at : a.total);
      first[b] = !ok ? -1 : in == 0 ? 0 : (int)(cursor + in - need);
      if (ok && need > 0) atomicMax(&end_cursor, (int)(cursor + in));
      if (blockIdx.x == 0) {
        a.cu_seqlens[b] = cu[b];
        a.lens_out[b] = ok ? (int)(r.len + r.add) : a.cache_lens[b];
        if (!r.valid || !tokens_fit) atomicCAS(a.status, 0, kDevBadSeqlens);
        else if (!ok) atomicCAS(a.status, 0, kDevBadPage);
      }
    }
  }
  if (tid == 0) cu[a.B] = (int)(add_before < a.total ? add_before : a.total);
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    a.cu_seqlens[a.B] = cu[a.B];
    *a.cursor_out = end_cursor;
  }
  // block-table rows: a warp per request
  const int warps = gridDim.x * (kPlanThreads / 32);
  for (int b = blockIdx.x * (kPlanThreads / 32) + warp; b < a.B; b += warps) {
    const int f = first[b];
    if (f < 0) continue;
    const PlanReq r = plan_req(a, b);
    const int have = pages_of(r.len, a.page_size), want = pages_of(r.len + r.add, a.page_size);
    for (int p = have + lane; p < want; p += 32) a.block_table[(long)b * a.max_pages + p] = a.free_pages[f + p - have];
  }
  // tokens
  const int live = cu[a.B];
  bool bad_page = false;
  for (long n0 = (long)blockIdx.x * kPlanThreads * kPer + tid; n0 < a.total; n0 += (long)gridDim.x * kPlanThreads * kPer) {
    int slot[kPer], pos[kPer], req[kPer], page[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const long n = n0 + i * kPlanThreads;
      int lo = 0, hi = a.B - 1;   // the last request that starts at or before n
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= n) lo = mid;
        else hi = mid - 1;
      }
      req[i] = n < live && first[lo] >= 0 ? lo : -1;
      slot[i] = -1;
      pos[i] = page[i] = 0;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (req[i] >= 0) {
        const int len = a.cache_lens[req[i]];
        pos[i] = len + (int)(n0 + i * kPlanThreads - cu[req[i]]);
        const int p = (int)((unsigned)pos[i] / (unsigned)a.page_size), have = pages_of(len, a.page_size);
        page[i] = p < have ? a.block_table[(long)req[i] * a.max_pages + p] : a.free_pages[first[req[i]] + p - have];
        slot[i] = pos[i] - p * a.page_size;
      }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const long n = n0 + i * kPlanThreads;
      if (n >= a.total) break;
      if (req[i] >= 0) {
        const long s = (long)page[i] * a.page_size + slot[i];
        const bool ok = page[i] >= 0 && s <= 0x7fffffffL;
        slot[i] = ok ? (int)s : -1;
        bad_page |= !ok;
      }
      a.slots[n] = slot[i];
      a.positions[n] = pos[i];
    }
  }
  if (bad_page) atomicCAS(a.status, 0, kDevBadPage);
}

// ------------------------------------------------------------ rotary rows
// Products and sums are rounded one by one (no fused multiply-add): the values
// are the elementary ones, whoever computes them.
__device__ __forceinline__ float rot_first(float x, float y, float c, float s) {
  return __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
}
__device__ __forceinline__ float rot_second(float x, float y, float c, float s) {   // x: the pair's second
  return __fadd_rn(__fmul_rn(x, c), __fmul_rn(y, s));
}

__device__ __forceinline__ void load8f(const float* p, float* x) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// Bound by memory: each row is read and written once.  A thread takes one part
// of a token's heads, HC of them: 8 features (4 neighbouring pairs, or features
// past rotary_dim), or in the half layout the two groups of 8 that are paired.
// Neighbouring threads take neighbouring 16 bytes, the table row is read once
// for HC heads, and all HC heads' loads are in flight together.  2 x 4096 tokens
// of 32 + 8 heads of 128 (172 MB): 28.1 us, 6.1 TB/s, 90% of a copy's rate (29.5
// with the loads one head after another); 64 of 128 features interleaved, 16411
// tokens of 16 + 8 heads (204 MB): 32.6 us, 92%.  f32 throughout, one rounding
// to the bf16 that the output is.
template <int HC, bool INTER>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a) {
  griddep_wait();
  griddep_launch();
  const int rotated = a.R / (INTER ? 8 : 16), U = rotated + (a.D - a.R) / 8;
  const long idx = (long)blockIdx.x * 256 + threadIdx.x;
  const long n = idx / U;
  if (n >= (long)a.B * a.T) return;
  const int u = (int)(idx - n * U);
  const long b = a.B == 1 ? 0 : n / a.T, t = n - b * a.T;
  const int pos = a.positions[b * a.pos_stride + t];
  const bool ok = pos >= 0 && pos < a.n_table;
  const bool rot = u < rotated, two = rot && !INTER;   // two: features fa.. are paired with fb..
  const int fa = rot ? 8 * u : a.R + 8 * (u - rotated), fb = a.R / 2 + 8 * u;
  const int h0 = blockIdx.y * HC;
  const int H = a.Hq + a.Hkv;
  uint4 wa[HC], wb[HC];
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    const int hh = h0 + i;
    const bool is_q = hh < a.Hq;
    const __nv_bfloat16* x = is_q ? a.q.p + b * a.q.sb + t * a.q.st + hh * a.q.sh
                                  : a.k.p + b * a.k.sb + t * a.k.st + (hh - a.Hq) * a.k.sh;
    wa[i] = wb[i] = make_uint4(0, 0, 0, 0);
    if (ok && hh < H) {
      wa[i] = *reinterpret_cast<const uint4*>(x + fa);
      if (two) wb[i] = *reinterpret_cast<const uint4*>(x + fb);
    }
  }
  if (!ok && u == 0 && h0 == 0) atomicCAS(a.status, 0, kDevBadSeqlens);
  float c[8], s[8];
  if (rot && ok) {
    const float* cs = a.cs + (long)pos * a.R + (INTER ? 4 * u : 8 * u);
    if constexpr (INTER) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(cs)), y = __ldg(reinterpret_cast<const float4*>(cs + a.R / 2));
      c[0] = x.x, c[1] = x.y, c[2] = x.z, c[3] = x.w;
      s[0] = y.x, s[1] = y.y, s[2] = y.z, s[3] = y.w;
    } else {
      load8f(cs, c);
      load8f(cs + a.R / 2, s);
    }
#pragma unroll
    for (int i = 0; i < (INTER ? 4 : 8); ++i) s[i] *= a.sign;
  }
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    const int hh = h0 + i;
    if (hh >= H) break;
    if (rot && ok) {
      float x[8];
      bf16x8_to_f32(wa[i], x);
      if constexpr (INTER) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[2 * j] = rot_first(x[2 * j], x[2 * j + 1], c[j], s[j]);
          y[2 * j + 1] = rot_second(x[2 * j + 1], x[2 * j], c[j], s[j]);
        }
        wa[i] = f32_to_bf16x8(y);
      } else {
        float y[8], x2[8], y2[8];
        bf16x8_to_f32(wb[i], x2);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          y[j] = rot_first(x[j], x2[j], c[j], s[j]);
          y2[j] = rot_second(x2[j], x[j], c[j], s[j]);
        }
        wa[i] = f32_to_bf16x8(y);
        wb[i] = f32_to_bf16x8(y2);
      }
    }
    const bool is_q = hh < a.Hq;
    __nv_bfloat16* y = const_cast<__nv_bfloat16*>(is_q ? a.qo.p + b * a.qo.sb + t * a.qo.st + hh * a.qo.sh
                                                       : a.ko.p + b * a.ko.sb + t * a.ko.st + (hh - a.Hq) * a.ko.sh);
    *reinterpret_cast<uint4*>(y + fa) = wa[i];
    if (two) *reinterpret_cast<uint4*>(y + fb) = wb[i];
  }
}

// ----------------------------------------------------------- rotary table
// w_i, the turns pair i makes per position as a 64-bit fraction, comes from
// the host in double; p * w_i modulo 2^64 is then the position's phase, exact
// to 2^-64 p turns however far p is.  Its top two bits (rounded) are the
// quadrant, what is left an angle a in [-pi/4, pi/4], and sin and cos of that are
// their Taylor polynomials of degree 9 and 10 (remainders below a^11/11! and
// a^12/12!: 2e-9).  Errors: a is rounded to 24 bits and once more by the factor
// pi 2^-31 (8e-8 in all), the sums to 6e-8; the largest found over 4e7 phases is
// 1.0e-7, three times that of the correctly rounded value.  A thread keeps one pair: its w is
// read once (a constant indexed by the lane is fetched once per lane) and its
// phase advances by an addition.  131072 rows of 128: 16.6 us with sincospif,
// whose conversions bound it, 12.4 us now; the stores alone would take 9.9 us.
constexpr int kMaxPairs = 256;
struct TurnsTable {
  unsigned long long w[kMaxPairs];
};

__global__ void __launch_bounds__(256) rope_table_kernel(float* out, int n, int R, float mscale, const TurnsTable tt) {
  griddep_wait();
  griddep_launch();
  const int H = R / 2, rows = blockDim.x / H, i = threadIdx.x % H, step = rows * gridDim.x;
  const int p0 = blockIdx.x * rows + threadIdx.x / H;
  const unsigned long long w = tt.w[i], dw = w * step;
  unsigned long long ph = w * p0 + (1ull << 61);     // an eighth of a turn ahead: the quadrant is rounded
  float* o = out + (long)p0 * R + i;
  const long stride = (long)step * R;
#pragma unroll 2
  for (long p = p0; p < n; p += step, ph += dw, o += stride) {
    const unsigned top = (unsigned)(ph >> 32);
    const float a = (float)((int)(top & 0x3FFFFFFFu) - 0x20000000) * (3.14159265358979f * 0x1p-31f);
    const float a2 = a * a;
    float s = fmaf(a2, 1.f / 362880.f, -1.f / 5040.f), c = fmaf(a2, -1.f / 3628800.f, 1.f / 40320.f);
    s = fmaf(a2, s, 1.f / 120.f);
    c = fmaf(a2, c, -1.f / 720.f);
    s = fmaf(a2, s, -1.f / 6.f);
    c = fmaf(a2, c, 1.f / 24.f);
    s = fmaf(a2 * a, s, a);
    c = fmaf(a2, c, -0.5f);
    c = fmaf(a2, c, 1.f);
    // quadrant q: (cos, sin) = (c, s), (-s, c), (-c, -s), (s, -c)
    const unsigned q = top >> 30;
    const float x = q & 1 ? s : c, y = q & 1 ? c : s;
    o[0] = ((q + 1) & 2 ? -x : x) * mscale;
    o[H] = (q & 2 ? -y : y) * mscale;
  }
}

// ------------------------------------------------------------------ append
// Bound by memory, or for 4 bits by its latency: 8 features are one 16-byte load
// and some 100 instructions to scale, round and pack, and each head's loads are
// waited for before them (issue slots 50%, ALU 42%).  A thread takes one part of
// a token's row, or two paired ones, of k and of v, in HC heads one after
// another: what depends on the token alone (its place in the cache) is found
// once.  A part is 8 features, so that neighbouring threads write neighbouring
// 16 (8) bytes, or for 4-bit caches a whole block of 16: its scale then stays in
// the thread.  The cosines and sines are loaded anew for each head: a thread then
// fits 64 registers, and the 8 warps a scheduler that this allows hide more
// latency than the table's row and the next head's loads kept in registers did
// (105 of them; 4 bits, 16411 tokens of 8 heads of 128, 64 features rotated:
// 20.4 us against 18.2, 71% of a copy's rate).  All 128 rotated in halves, 16384
// tokens: bf16 23.1 us (88%; one part a thread 28.5), E4M3 19.8 (78%; 24.4), 4
// bits 24.4 (54%: the paired features and table rows are loaded twice; two parts
// a thread 23 to 26, but 2.9 against 2.5 for 1000 tokens).  64 tokens and their
// gather: 4.1 us, two launches; called from Python 9.5.  Times in captured
// graphs but for the last.  All arithmetic is f32, each
// element rounded once to the cache's type.
__device__ __forceinline__ uint32_t e4m3_of(float x) { return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3); }

// A part at p (of a 4-bit row: codes at p, the block's scale at sf).  to_scale:
// E4M3 1 / scale, 4 bits 1 / (6 scale); inv: of each E4M3 code, 1 / (its value * scale).
template <int FMT>
__device__ __forceinline__ void store_part(uint8_t* p, uint8_t* sf, const float* x, float to_scale, const float* inv) {
  if constexpr (FMT == kCacheBf16) {
    *reinterpret_cast<uint4*>(p) = f32_to_bf16x8(x);
  } else if constexpr (FMT == kCacheE4m3) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = e4m3_of(__fmul_rn(x[4 * i], to_scale)) | e4m3_of(__fmul_rn(x[4 * i + 1], to_scale)) << 8 |
             e4m3_of(__fmul_rn(x[4 * i + 2], to_scale)) << 16 | e4m3_of(__fmul_rn(x[4 * i + 3], to_scale)) << 24;
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
    uint32_t m = 0;   // the largest magnitude's bits; NaN and infinity are the largest of all
#pragma unroll
    for (int i = 0; i < 16; i += 2)
      m = __vimax3_u32(m, __float_as_uint(x[i]) & 0x7fffffffu, __float_as_uint(x[i + 1]) & 0x7fffffffu);
    // not finite: the NaN code, and codes 0
    const bool fin = m < 0x7f800000u;
    const uint32_t sf8 = fin ? e4m3_of(fminf(__fmul_rn(__uint_as_float(m), to_scale), 448.f)) : 0x7fu;
    const float r = inv[sf8];
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(x[i], r);
    const uint32_t lo = f32x8_to_e2m1(y), hi = f32x8_to_e2m1(y + 8);
    *reinterpret_cast<uint2*>(p) = make_uint2(fin ? lo : 0u, fin ? hi : 0u);
    *sf = (uint8_t)sf8;
  }
}

// Loaded where it stands: a plain load would be moved out of the loop over the heads, into registers.
__device__ __forceinline__ void load4_here(const float* p, float* x) {
  asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "l"(p));
}

enum { kNoRope = 0, kHalf = 1, kInter = 2 };

// Parts a thread takes: in the half layout the two that are paired, but for 4 bits (two blocks' values at once do not
// fit its registers), where the paired features are loaded beside its own.
template <int FMT, int ROT>
constexpr int kParts = ROT == kHalf && FMT != kCacheQ4 ? 2 : 1;

template <int FMT, int HC, int ROT>
__global__ void __launch_bounds__(256, 4) cache_append_kernel(const AppendArgs a) {
  constexpr int G = FMT == kCacheQ4 ? 2 : 1;         // groups of 8 features of a part
  constexpr int P = kParts<FMT, ROT>;
  // 1 / (sf * scale) for every block scale: rounded reciprocals, one a thread instead of one a block of features
  __shared__ float inv[2][128];
  if constexpr (FMT == kCacheQ4) {
    const uint32_t code = threadIdx.x & 127;
    const float sf = f16x2_to_f32(e4m3x2_to_f16(code)).x;
    inv[threadIdx.x >> 7][code] = code == 0 || code == 127 ? 0.f : __frcp_rn(__fmul_rn(sf, threadIdx.x < 128 ? a.k_scale : a.v_scale));
    __syncthreads();
  }
  griddep_wait();
  griddep_launch();
  const int u_log = (a.D == 128 ? 4 : 3) - (G - 1) - (P - 1);  // threads of a row, as a power of two
  const long idx = (long)blockIdx.x * 256 + threadIdx.x, n = idx >> u_log;
  if (n >= (long)a.B * a.T) return;
  const int u = (int)idx & ((1 << u_log) - 1), h0 = blockIdx.y * HC, R2 = a.R / 2;
  const bool rotated = ROT != kNoRope && 8 * G * P * u < a.R;
  // the part's first feature; with two parts, the pairs' first and second ones, or neighbours past rotary_dim
  const int f0 = 8 * G * u * (P == 1 || rotated ? 1 : 2), f1 = rotated ? f0 + R2 : f0 + 8 * G;
  const int slot = a.slots[n];
  int pos = 0;
  if constexpr (ROT != kNoRope) pos = a.positions[n];
  const int heads = min(HC, a.H - h0);
  const long b = a.B == 1 ? 0 : n / a.T, t = n - b * a.T;
  const __nv_bfloat16* kr = a.k.p + b * a.k.sb + t * a.k.st + h0 * a.k.sh + f0;
  const __nv_bfloat16* vr = a.v.p + b * a.v.sb + t * a.v.st + h0 * a.v.sh + f0;
  bool second[G];                                    // a group of 8 is the second of its pairs
#pragma unroll
  for (int g = 0; g < G; ++g) second[g] = P == 1 && ROT == kHalf && f0 + 8 * g >= R2;
  if (slot < 0 || slot >= (long)a.num_pages * a.page_size) {
    if (slot != -1 && u == 0 && h0 == 0) atomicCAS(a.status, 0, kDevBadPage);
    return;
  }
  if constexpr (ROT != kNoRope)
    if (pos < 0 || pos >= a.n_table) {
      if (u == 0 && h0 == 0) atomicCAS(a.status, 0, kDevBadSeqlens);
      return;
    }
  const float* cs = a.cs + (long)pos * a.R;
  auto rotation = [&](int g, float* c, float* s) {   // of group g's features
    const int f = f0 + 8 * g;
    if constexpr (ROT == kHalf) {
      const int p = second[g] ? f - R2 : f;
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        load4_here(cs + p + j, c + j);
        load4_here(cs + R2 + p + j, s + j);
      }
    } else {
      load4_here(cs + f / 2, c);
      load4_here(cs + R2 + f / 2, s);
    }
  };
  // the part's place in the first head's row; the heads of a page are page_size rows apart
  constexpr int kNum = FMT == kCacheBf16 ? 4 : FMT == kCacheE4m3 ? 2 : 1;   // half bytes a feature
  const int page = slot / a.page_size, width = a.D * kNum / 2;
  const long row = ((long)page * a.H + h0) * a.page_size + (slot - page * a.page_size);
  if (!GQA_CHECK(row >= 0 && row + (long)(heads - 1) * a.page_size < (long)a.num_pages * a.H * a.page_size, a.status, a.dbg_line))
    return;
  const long at = row * width + f0 * kNum / 2, sf_at = row * (a.D / 16) + f0 / 16;
  uint8_t *kp = static_cast<uint8_t*>(a.kc) + at, *vp = static_cast<uint8_t*>(a.vc) + at;
  uint8_t *kf = a.ksf + sf_at, *vf = a.vsf + sf_at;
  const int to1 = (f1 - f0) * kNum / 2, sf_to1 = (f1 - f0) / 16;
  const long step = (long)a.page_size * width, sf_step = (long)a.page_size * (a.D / 16);
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    if (i >= heads) break;
    uint4 wk[P][G], wp[G], wv[P][G];                 // the row's parts, and with one part the one paired with k's
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const __nv_bfloat16 *k = kr + i * a.k.sh + 8 * g, *v = vr + i * a.v.sh + 8 * g;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        wk[p][g] = __ldg(reinterpret_cast<const uint4*>(k + (p ? f1 - f0 : 0)));
        wv[p][g] = __ldg(reinterpret_cast<const uint4*>(v + (p ? f1 - f0 : 0)));
      }
      if (P == 1 && ROT == kHalf && rotated) wp[g] = __ldg(reinterpret_cast<const uint4*>(k + (second[g] ? -R2 : R2)));
    }
    float x[P][8 * G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
      for (int p = 0; p < P; ++p) bf16x8_to_f32(wk[p][g], x[p] + 8 * g);
      if constexpr (ROT != kNoRope) {
        if (!rotated) continue;
        float c[8], s[8];
        rotation(g, c, s);
        if constexpr (P == 2) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float y = x[0][8 * g + j], z = x[1][8 * g + j];
            x[0][8 * g + j] = rot_first(y, z, c[j], s[j]);
            x[1][8 * g + j] = rot_second(z, y, c[j], s[j]);
          }
        } else if constexpr (ROT == kHalf) {
          const uint32_t sign = second[g] ? 0x80008000u : 0u;   // x c + y s as x c - (-y) s: the same rounding
          float y[8];
          bf16x8_to_f32(make_uint4(wp[g].x ^ sign, wp[g].y ^ sign, wp[g].z ^ sign, wp[g].w ^ sign), y);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[0][8 * g + j] = rot_first(x[0][8 * g + j], y[j], c[j], s[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float e = x[0][8 * g + 2 * j], o = x[0][8 * g + 2 * j + 1];
            x[0][8 * g + 2 * j] = rot_first(e, o, c[j], s[j]);
            x[0][8 * g + 2 * j + 1] = rot_second(o, e, c[j], s[j]);
          }
        }
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) store_part<FMT>(kp + p * to1, kf + p * sf_to1, x[p], a.k_inv, inv[0]);
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int g = 0; g < G; ++g) bf16x8_to_f32(wv[p][g], x[p] + 8 * g);
      store_part<FMT>(vp + p * to1, vf + p * sf_to1, x[p], a.v_inv, inv[1]);
    }
    kp += step, vp += step, kf += sf_step, vf += sf_step;
  }
}

// ------------------------------------------------------------------ gather
// A thread takes 8 features of HC heads of a token.
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t sf8, float scale) {
  const uint32_t s = e4m3x2_to_f16(sf8 | sf8 << 8);
  uint32_t r[4];
  e2m1x8_to_f16(codes, r);
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = f16x2_to_f32(hmul2_u(r[i], s));   // exact: 6 significant bits within f16's range
    x[2 * i] = v.x * scale;
    x[2 * i + 1] = v.y * scale;
  }
  return f32_to_bf16x8(x);
}

template <int HC>
__global__ void __launch_bounds__(256) cache_gather_kernel(const GatherArgs a) {
  griddep_wait();
  griddep_launch();
  const int U = a.D / 8, u_log = a.D == 128 ? 4 : 3;
  const long idx = (long)blockIdx.x * 256 + threadIdx.x, n = idx >> u_log;
  if (n >= a.tokens) return;
  const int u = (int)(idx & (U - 1)), h0 = blockIdx.y * HC;
  const int slot = a.slots[n];
  const bool live = slot >= 0 && slot < (long)a.num_pages * a.page_size;
  if (!live && slot != -1 && u == 0 && h0 == 0) atomicCAS(a.status, 0, kDevBadPage);
  const int page = live ? slot / a.page_size : 0;
  const long row0 = ((long)page * a.H + h0) * a.page_size + (live ? slot - page * a.page_size : 0);
  uint32_t kc[HC], vc[HC], ks[HC], vs[HC];
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    kc[i] = vc[i] = ks[i] = vs[i] = 0;
    if (live && h0 + i < a.H) {
      const long row = row0 + (long)i * a.page_size;
      kc[i] = __ldg(reinterpret_cast<const uint32_t*>(a.k4 + row * (a.D / 2)) + u);
      vc[i] = __ldg(reinterpret_cast<const uint32_t*>(a.v4 + row * (a.D / 2)) + u);
      ks[i] = __ldg(a.ksf + row * (a.D / 16) + u / 2);
      vs[i] = __ldg(a.vsf + row * (a.D / 16) + u / 2);
    }
  }
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    if (h0 + i >= a.H) break;
    const long out = (n * a.H + h0 + i) * U + u;
    reinterpret_cast<uint4*>(a.k)[out] = values8(kc[i], ks[i], a.k_scale);
    reinterpret_cast<uint4*>(a.v)[out] = values8(vc[i], vs[i], a.v_scale);
  }
}

bool grid_of(long threads, unsigned* blocks) {
  const long g = (threads + 255) / 256;
  *blocks = (unsigned)g;
  return g >= 1 && g <= 0x7fffffffL;
}

}  // namespace

template <int kPer>
static cudaError_t launch_plan_as(const PlanArgs& a, long grid, cudaStream_t stream) {
  const size_t smem = (size_t)(2 * a.B + 1) * sizeof(int);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(cache_plan_kernel<kPer>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (2 * kPlanMaxB + 1) * 4);
    if (e != cudaSuccess) return e;
  }
  prof_begin(kProfPlan, stream);
  const cudaError_t e = launch_programmatic(cache_plan_kernel<kPer>, dim3((unsigned)grid), dim3(kPlanThreads), smem, stream, a);
  prof_end(stream);
  return e;
}

// One token a thread while that needs no more blocks than there are SMs (each
// scans all requests anew), else four.  64 requests of 600 tokens: one 3.9 us,
// four 5.5; 512 of 500: 6.9, 6.4; 512 of 4000: 27.0, 24.2.
cudaError_t launch_cache_plan(const PlanArgs& a, int sms, cudaStream_t stream) {
  const long one = ((long)a.total + kPlanThreads - 1) / kPlanThreads;
  if (one <= sms) return launch_plan_as<1>(a, one < 1 ? 1 : one, stream);
  const long four = (one + 3) / 4;
  return launch_plan_as<4>(a, four < sms ? four : sms, stream);
}

// Heads a thread takes: `most` if that leaves every SM two blocks or more, else
// one, so that few tokens still spread over the SMs.  Rotary rows of 40 heads of
// 128: 256 tokens 3.4 us with 8 heads a thread, 2.6 with one; 1024: 4.9, 4.8;
// 8192: 28.4, 31.9.  Append (and gather, 4 bits, 8 heads of 128) of 1024 tokens:
// 8.7 with 4, 5.5 with one; 4096: 12.7, 11.6; 16384: 38.5, 43.7.
static bool many_heads(unsigned gx, int H, int most, int sms) { return (long)gx * ((H + most - 1) / most) >= 2L * sms; }

template <bool INTER>
static cudaError_t launch_rope_as(const RopeArgs& a, int sms, cudaStream_t stream) {
  constexpr int kHeads = 8;
  const int H = a.Hq + a.Hkv, U = a.R / (INTER ? 8 : 16) + (a.D - a.R) / 8;
  unsigned gx;
  if (!grid_of((long)a.B * a.T * U, &gx)) return cudaErrorInvalidValue;
  const bool wide = many_heads(gx, H, kHeads, sms);
  const dim3 grid(gx, (unsigned)(wide ? (H + kHeads - 1) / kHeads : H));
  prof_begin(kProfRope, stream);
  const cudaError_t e = wide ? launch_programmatic(rope_kernel<kHeads, INTER>, grid, dim3(256), 0, stream, a)
                             : launch_programmatic(rope_kernel<1, INTER>, grid, dim3(256), 0, stream, a);
  prof_end(stream);
  return e;
}

cudaError_t launch_rope(const RopeArgs& a, int sms, cudaStream_t stream) {
  return a.interleaved ? launch_rope_as<true>(a, sms, stream) : launch_rope_as<false>(a, sms, stream);
}

cudaError_t launch_rope_table(const RopeTableArgs& a, int sms, cudaStream_t stream) {
  TurnsTable tt{};
  for (int i = 0; i < a.R / 2; ++i) {
    double theta = exp2(-2.0 * i / a.R * log2(a.base));
    if (a.turns > 0.0) {
      double g = (a.turns * theta - a.low) / (a.high - a.low);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      theta = theta * g + theta / a.factor * (1.0 - g);
    } else {
      theta /= a.factor;
    }
    double f = theta * 0.15915494309189533576888;   // turns: 1 / (2 pi)
    f -= floor(f);
    tt.w[i] = f < 1.0 ? (unsigned long long)ldexp(f, 64) : 0ull;
  }
  const int H = a.R / 2, rows = 256 / H;   // positions a block takes at a time
  long g = ((long)a.n + rows - 1) / rows;
  if (g > 8L * sms) g = 8L * sms;
  prof_begin(kProfRopeTable, stream);
  const cudaError_t e = launch_programmatic(rope_table_kernel, dim3((unsigned)g), dim3(rows * H), 0, stream, a.out, a.n, a.R,
                                            a.mscale, tt);
  prof_end(stream);
  return e;
}

template <int FMT, int ROT>
static cudaError_t launch_append_as(const AppendArgs& a, int sms, cudaStream_t stream) {
  constexpr int kHeads = 4 / kParts<FMT, ROT>;
  unsigned gx;
  if (!grid_of((long)a.B * a.T * (a.D / ((FMT == kCacheQ4 ? 16 : 8) * kParts<FMT, ROT>)), &gx))
    return cudaErrorInvalidValue;
  const bool wide = many_heads(gx, a.H, kHeads, sms);
  const dim3 grid(gx, (unsigned)(wide ? (a.H + kHeads - 1) / kHeads : a.H));
  prof_begin(kProfAppend, stream);
  const cudaError_t e = wide ? launch_programmatic(cache_append_kernel<FMT, kHeads, ROT>, grid, dim3(256), 0, stream, a)
                             : launch_programmatic(cache_append_kernel<FMT, 1, ROT>, grid, dim3(256), 0, stream, a);
  prof_end(stream);
  return e;
}

template <int FMT>
static cudaError_t launch_append_rot(const AppendArgs& a, int sms, cudaStream_t stream) {
  if (!a.cs) return launch_append_as<FMT, kNoRope>(a, sms, stream);
  return a.interleaved ? launch_append_as<FMT, kInter>(a, sms, stream) : launch_append_as<FMT, kHalf>(a, sms, stream);
}

cudaError_t launch_cache_append(const AppendArgs& a, CacheFmt fmt, int sms, cudaStream_t stream) {
  if (fmt == kCacheBf16) return launch_append_rot<kCacheBf16>(a, sms, stream);
  if (fmt == kCacheE4m3) return launch_append_rot<kCacheE4m3>(a, sms, stream);
  return launch_append_rot<kCacheQ4>(a, sms, stream);
}

cudaError_t launch_cache_gather(const GatherArgs& a, int sms, cudaStream_t stream) {
  constexpr int kHeads = 4;
  unsigned gx;
  if (!grid_of((long)a.tokens * (a.D / 8), &gx)) return cudaErrorInvalidValue;
  const bool wide = many_heads(gx, a.H, kHeads, sms);
  const dim3 grid(gx, (unsigned)(wide ? (a.H + kHeads - 1) / kHeads : a.H));
  prof_begin(kProfGather, stream);
  const cudaError_t e = wide ? launch_programmatic(cache_gather_kernel<kHeads>, grid, dim3(256), 0, stream, a)
                             : launch_programmatic(cache_gather_kernel<1>, grid, dim3(256), 0, stream, a);
  prof_end(stream);
  return e;
}

}  // namespace gqa
