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

__device__ __forceinline__ long pages_of(long keys, int page_size) { return (keys + page_size - 1) / page_size; }

__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const PlanArgs a) {
  extern __shared__ int plan_smem[];
  int* cu = plan_smem;              // [B + 1] first token of each request
  int* first = plan_smem + a.B + 1; // [B] its first page's index in free_pages, -1: refused
  __shared__ long warp_need[kPlanThreads / 32], warp_add[kPlanThreads / 32];
  __shared__ int end_cursor;
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
    const int have = (int)pages_of(r.len, a.page_size), want = (int)pages_of(r.len + r.add, a.page_size);
    for (int p = have + lane; p < want; p += 32) a.block_table[(long)b * a.max_pages + p] = a.free_pages[f + p - have];
  }
  // tokens
  bool bad_page = false;
  for (int n = blockIdx.x * kPlanThreads + tid; n < a.total; n += gridDim.x * kPlanThreads) {
    int slot = -1, pos = 0;
    if (n < cu[a.B]) {
      int lo = 0, hi = a.B - 1;   // the last request that starts at or before n
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= n) lo = mid;
        else hi = mid - 1;
      }
      const int f = first[lo];
      if (f >= 0) {
        const int len = a.cache_lens[lo];
        pos = len + (n - cu[lo]);
        const int p = pos / a.page_size, have = (int)pages_of(len, a.page_size);
        const int page = p < have ? a.block_table[(long)lo * a.max_pages + p] : a.free_pages[f + p - have];
        const long s = (long)page * a.page_size + (pos - p * a.page_size);
        if (page >= 0 && s <= 0x7fffffffL) slot = (int)s;
        else bad_page = true;
      }
    }
    a.slots[n] = slot;
    a.positions[n] = pos;
    if (n > 0x7fffffff - (int)(gridDim.x * kPlanThreads)) break;
  }
  if (bad_page) atomicCAS(a.status, 0, kDevBadPage);
}

// ------------------------------------------------------------ rotary rows
// A thread takes 16 features of a token: 8 rotated pairs (both layouts use
// the same 8 cosines and sines) or 16 features past rotary_dim, for HC heads,
// so the table row is read once per HC heads.  Products and sums are rounded
// one by one (no fused multiply-add): the values are the elementary ones.
__device__ __forceinline__ void rotate8(const float* x, const float* y, const float* c, const float* s, float* xo,
                                        float* yo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    xo[i] = __fsub_rn(__fmul_rn(x[i], c[i]), __fmul_rn(y[i], s[i]));
    yo[i] = __fadd_rn(__fmul_rn(y[i], c[i]), __fmul_rn(x[i], s[i]));
  }
}

__device__ __forceinline__ void load8f(const float* p, float* x) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

template <int HC>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a) {
  const int U = a.D / 16;
  const long idx = (long)blockIdx.x * 256 + threadIdx.x;
  const long n = idx / U;
  if (n >= (long)a.B * a.T) return;
  const int u = (int)(idx - n * U);
  const long b = n / a.T, t = n - b * a.T;
  const int pos = a.positions[b * a.pos_stride + t];
  const bool ok = pos >= 0 && pos < a.n_table;
  if (!ok && u == 0 && blockIdx.y == 0) atomicCAS(a.status, 0, kDevBadSeqlens);
  const bool rot = u < a.R / 16;
  // features of the thread: [fa, fa + 8) and [fb, fb + 8)
  const int fa = rot && !a.interleaved ? 8 * u : 16 * u;
  const int fb = rot && !a.interleaved ? a.R / 2 + 8 * u : 16 * u + 8;
  float c[8], s[8];
  if (rot && ok) {
    const float* cs = a.cs + (long)pos * a.R + 8 * u;
    load8f(cs, c);
    load8f(cs + a.R / 2, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] *= a.sign;
  }
  const int h0 = blockIdx.y * HC;
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    const int hh = h0 + i;
    if (hh >= a.Hq + a.Hkv) break;
    const bool is_q = hh < a.Hq;
    const RowView& in = is_q ? a.q : a.k;
    const RowView& out = is_q ? a.qo : a.ko;
    const int h = is_q ? hh : hh - a.Hq;
    const __nv_bfloat16* x = in.p + b * in.sb + t * in.st + h * in.sh;
    __nv_bfloat16* y = const_cast<__nv_bfloat16*>(out.p) + b * out.sb + t * out.st + h * out.sh;
    uint4 wa = make_uint4(0, 0, 0, 0), wb = wa;
    if (ok) {
      wa = *reinterpret_cast<const uint4*>(x + fa);
      wb = *reinterpret_cast<const uint4*>(x + fb);
      if (rot) {
        float va[8], vb[8], oa[8], ob[8];
        bf16x8_to_f32(wa, va);
        bf16x8_to_f32(wb, vb);
        if (a.interleaved) {   // pairs (0,1), (2,3), ...: split, rotate, put back
          float e[8], o[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) e[j] = va[2 * j], o[j] = va[2 * j + 1], e[4 + j] = vb[2 * j], o[4 + j] = vb[2 * j + 1];
          float re[8], ro[8];
          rotate8(e, o, c, s, re, ro);
#pragma unroll
          for (int j = 0; j < 4; ++j) oa[2 * j] = re[j], oa[2 * j + 1] = ro[j], ob[2 * j] = re[4 + j], ob[2 * j + 1] = ro[4 + j];
        } else {
          rotate8(va, vb, c, s, oa, ob);
        }
        wa = f32_to_bf16x8(oa);
        wb = f32_to_bf16x8(ob);
      }
    }
    *reinterpret_cast<uint4*>(y + fa) = wa;
    *reinterpret_cast<uint4*>(y + fb) = wb;
  }
}

// ----------------------------------------------------------- rotary table
// w_i, the turns pair i makes per position as a 64-bit fraction, comes from
// the host in double; p * w_i modulo 2^64 is then the position's phase, exact
// to 2^-64 p turns however far p is.  Its upper 24 bits are an f32 half-turn
// count for sincospif; the next 24 are a correction of first order (below
// 2^-23 pi, its square is lost in f32).
constexpr int kMaxPairs = 256;
struct TurnsTable {
  unsigned long long w[kMaxPairs];
};

__global__ void __launch_bounds__(256) rope_table_kernel(float* out, int n, int R, float mscale, const TurnsTable tt) {
  const int H = R / 2;
  const long total = (long)n * H, step = (long)gridDim.x * 256;
  for (long e = (long)blockIdx.x * 256 + threadIdx.x; e < total; e += step) {
    const int p = (int)(e / H), i = (int)(e - (long)p * H);
    const unsigned long long ph = (unsigned long long)p * tt.w[i];
    const float half_turns = (float)(int)((long long)ph >> 40) * 0x1p-23f;
    const float d = (float)(unsigned)((ph >> 16) & 0xFFFFFFull) * (0x1p-47f * 3.14159265358979f);
    float s, c;
    sincospif(half_turns, &s, &c);
    out[(long)p * R + i] = fmaf(-s, d, c) * mscale;
    out[(long)p * R + H + i] = fmaf(c, d, s) * mscale;
  }
}

// ------------------------------------------------------------------ append
// A thread takes one 16-feature block of one head of one token, of k and of
// v: the unit that shares a 4-bit scale, so nothing crosses threads.  With
// half-layout rotation it also loads the 16 features its own are paired with
// (they come from L1: a neighbouring thread's own block).
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float* x) {
  bf16x8_to_f32(*reinterpret_cast<const uint4*>(p), x);
  bf16x8_to_f32(*reinterpret_cast<const uint4*>(p + 8), x + 8);
}

// Features [f0, f0 + 16) of one k row, rotated by table row cs.
__device__ __forceinline__ void rotate_block(const AppendArgs& a, const __nv_bfloat16* row, const float* cs, int f0,
                                             float* x) {
  const int H = a.R / 2;
  if (a.interleaved) {
    float c[8], s[8];
    load8f(cs + f0 / 2, c);
    load8f(cs + H + f0 / 2, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float e = x[2 * i], o = x[2 * i + 1];
      x[2 * i] = __fsub_rn(__fmul_rn(e, c[i]), __fmul_rn(o, s[i]));
      x[2 * i + 1] = __fadd_rn(__fmul_rn(o, c[i]), __fmul_rn(e, s[i]));
    }
    return;
  }
#pragma unroll
  for (int g = 0; g < 2; ++g) {   // 8 features at a time: H is a multiple of 8
    const int f = f0 + 8 * g;
    const bool second = f >= H;
    const int i0 = second ? f - H : f;
    float c[8], s[8], y[8];
    load8f(cs + i0, c);
    load8f(cs + H + i0, s);
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(row + (second ? f - H : f + H)), y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = __fmul_rn(x[8 * g + i], c[i]), q = __fmul_rn(y[i], s[i]);
      x[8 * g + i] = second ? __fadd_rn(p, q) : __fsub_rn(p, q);
    }
  }
}

__device__ __forceinline__ uint32_t e4m3_of(float x) { return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3); }

// One 16-feature block into a 4-bit cache: its codes and its scale byte.
__device__ __forceinline__ void quantise_block(const float* x, float scale, uint2& codes, uint8_t& sf8) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
  if (m >= 0x7f800000u) {   // a NaN or an infinity: the whole block reads as NaN
    sf8 = 0x7f;
    codes = make_uint2(0, 0);
    return;
  }
  const float rc = __fdiv_rn(1.f, __fmul_rn(6.f, scale));
  sf8 = (uint8_t)e4m3_of(fminf(__fmul_rn(__uint_as_float(m), rc), 448.f));
  const float sf = f16x2_to_f32(e4m3x2_to_f16(sf8)).x;
  const float inv = sf > 0.f ? __fdiv_rn(1.f, __fmul_rn(sf, scale)) : 0.f;
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(x[i], inv);
  codes = make_uint2(f32x8_to_e2m1(y), f32x8_to_e2m1(y + 8));
}

template <int FMT>
__device__ __forceinline__ void store_block(const AppendArgs& a, bool is_k, long row, int f0, const float* x) {
  void* cache = is_k ? a.kc : a.vc;
  const float scale = is_k ? a.k_scale : a.v_scale;
  if constexpr (FMT == kCacheBf16) {
    uint4* y = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(cache) + row * a.D + f0);
    y[0] = f32_to_bf16x8(x);
    y[1] = f32_to_bf16x8(x + 8);
  } else if constexpr (FMT == kCacheE4m3) {
    const float r = __fdiv_rn(1.f, scale);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = e4m3_of(__fmul_rn(x[4 * i], r)) | e4m3_of(__fmul_rn(x[4 * i + 1], r)) << 8 |
             e4m3_of(__fmul_rn(x[4 * i + 2], r)) << 16 | e4m3_of(__fmul_rn(x[4 * i + 3], r)) << 24;
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(cache) + row * a.D + f0) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint2 codes;
    uint8_t sf;
    quantise_block(x, scale, codes, sf);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + row * (a.D / 2) + f0 / 2) = codes;
    (is_k ? a.ksf : a.vsf)[row * (a.D / 16) + f0 / 16] = sf;
  }
}

template <int FMT>
__global__ void __launch_bounds__(256) cache_append_kernel(const AppendArgs a) {
  const int NB = a.D / 16;
  const long idx = (long)blockIdx.x * 256 + threadIdx.x;
  const long rowi = idx / NB, n = rowi / a.H;
  if (n >= (long)a.B * a.T) return;
  const int f0 = (int)(idx - rowi * NB) * 16, h = (int)(rowi - n * a.H);
  const int slot = a.slots[n];
  if (slot < 0 || slot >= (long)a.num_pages * a.page_size) {
    if (slot != -1 && f0 == 0 && h == 0) atomicCAS(a.status, 0, kDevBadPage);
    return;
  }
  const float* cs = nullptr;
  if (a.cs) {
    const int pos = a.positions[n];
    if (pos < 0 || pos >= a.n_table) {
      if (f0 == 0 && h == 0) atomicCAS(a.status, 0, kDevBadSeqlens);
      return;
    }
    cs = a.cs + (long)pos * a.R;
  }
  const long b = n / a.T, t = n - b * a.T;
  const int page = slot / a.page_size;
  const long row = ((long)page * a.H + h) * a.page_size + (slot - page * a.page_size);
  const __nv_bfloat16* kr = a.k.p + b * a.k.sb + t * a.k.st + h * a.k.sh;
  const __nv_bfloat16* vr = a.v.p + b * a.v.sb + t * a.v.st + h * a.v.sh;
  if (!GQA_CHECK(row >= 0 && row < (long)a.num_pages * a.H * a.page_size, a.status, a.dbg_line)) return;
  float x[16];
  load16(kr + f0, x);
  if (cs && f0 < a.R) rotate_block(a, kr, cs, f0, x);
  store_block<FMT>(a, true, row, f0, x);
  load16(vr + f0, x);
  store_block<FMT>(a, false, row, f0, x);
}

// ------------------------------------------------------------------ gather
__device__ __forceinline__ void block_values(const uint8_t* c4, const uint8_t* sf8, float scale, float* x) {
  const uint2 w = *reinterpret_cast<const uint2*>(c4);
  const uint32_t s = e4m3x2_to_f16(*sf8 | (uint32_t)*sf8 << 8);
  uint32_t r[8];
  e2m1x8_to_f16(w.x, r);
  e2m1x8_to_f16(w.y, r + 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = f16x2_to_f32(hmul2_u(r[i], s));   // exact: 6 significant bits within f16's range
    x[2 * i] = v.x * scale;
    x[2 * i + 1] = v.y * scale;
  }
}

__global__ void __launch_bounds__(256) cache_gather_kernel(const GatherArgs a) {
  const int NB = a.D / 16;
  const long idx = (long)blockIdx.x * 256 + threadIdx.x;
  const long rowi = idx / NB, n = rowi / a.H;
  if (n >= a.tokens) return;
  const int blk = (int)(idx - rowi * NB), h = (int)(rowi - n * a.H);
  const int slot = a.slots[n];
  uint4* ko = reinterpret_cast<uint4*>(a.k + rowi * a.D + blk * 16);
  uint4* vo = reinterpret_cast<uint4*>(a.v + rowi * a.D + blk * 16);
  if (slot < 0 || slot >= (long)a.num_pages * a.page_size) {
    if (slot != -1 && blk == 0 && h == 0) atomicCAS(a.status, 0, kDevBadPage);
    ko[0] = ko[1] = vo[0] = vo[1] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int page = slot / a.page_size;
  const long row = ((long)page * a.H + h) * a.page_size + (slot - page * a.page_size);
  const long c = row * (a.D / 2) + blk * 8, s = row * NB + blk;
  float x[16];
  block_values(a.k4 + c, a.ksf + s, a.k_scale, x);
  ko[0] = f32_to_bf16x8(x);
  ko[1] = f32_to_bf16x8(x + 8);
  block_values(a.v4 + c, a.vsf + s, a.v_scale, x);
  vo[0] = f32_to_bf16x8(x);
  vo[1] = f32_to_bf16x8(x + 8);
}

bool grid_of(long threads, unsigned* blocks) {
  const long g = (threads + 255) / 256;
  *blocks = (unsigned)g;
  return g >= 1 && g <= 0x7fffffffL;
}

}  // namespace

cudaError_t launch_cache_plan(const PlanArgs& a, int sms, cudaStream_t stream) {
  const size_t smem = (size_t)(2 * a.B + 1) * sizeof(int);
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(cache_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (2 * kPlanMaxB + 1) * 4);
    if (e != cudaSuccess) return e;
  }
  long g = ((long)a.total + 2 * kPlanThreads - 1) / (2 * kPlanThreads);
  if (g > sms) g = sms;
  if (g < 1) g = 1;
  prof_begin(kProfPlan, stream);
  cache_plan_kernel<<<(unsigned)g, kPlanThreads, smem, stream>>>(a);
  prof_end(stream);
  return cudaGetLastError();
}

cudaError_t launch_rope(const RopeArgs& a, int sms, cudaStream_t stream) {
  const int H = a.Hq + a.Hkv;
  unsigned gx;
  if (!grid_of((long)a.B * a.T * (a.D / 16), &gx)) return cudaErrorInvalidValue;
  // 8 heads a thread when that still leaves every SM several blocks, else one
  const bool wide = (long)gx * ((H + 7) / 8) >= 4L * sms;
  const unsigned gy = (unsigned)(wide ? (H + 7) / 8 : H);
  if (gy > 65535u) return cudaErrorInvalidValue;
  prof_begin(kProfRope, stream);
  if (wide) rope_kernel<8><<<dim3(gx, gy), 256, 0, stream>>>(a);
  else rope_kernel<1><<<dim3(gx, gy), 256, 0, stream>>>(a);
  prof_end(stream);
  return cudaGetLastError();
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
  const long total = (long)a.n * (a.R / 2);
  long g = (total + 1023) / 1024;
  if (g > 8L * sms) g = 8L * sms;
  if (g < 1) g = 1;
  prof_begin(kProfRopeTable, stream);
  rope_table_kernel<<<(unsigned)g, 256, 0, stream>>>(a.out, a.n, a.R, a.mscale, tt);
  prof_end(stream);
  return cudaGetLastError();
}

cudaError_t launch_cache_append(const AppendArgs& a, CacheFmt fmt, cudaStream_t stream) {
  unsigned g;
  if (!grid_of((long)a.B * a.T * a.H * (a.D / 16), &g)) return cudaErrorInvalidValue;
  prof_begin(kProfAppend, stream);
  if (fmt == kCacheBf16) cache_append_kernel<kCacheBf16><<<g, 256, 0, stream>>>(a);
  else if (fmt == kCacheE4m3) cache_append_kernel<kCacheE4m3><<<g, 256, 0, stream>>>(a);
  else cache_append_kernel<kCacheQ4><<<g, 256, 0, stream>>>(a);
  prof_end(stream);
  return cudaGetLastError();
}

cudaError_t launch_cache_gather(const GatherArgs& a, cudaStream_t stream) {
  unsigned g;
  if (!grid_of((long)a.tokens * a.H * (a.D / 16), &g)) return cudaErrorInvalidValue;
  prof_begin(kProfGather, stream);
  cache_gather_kernel<<<g, 256, 0, stream>>>(a);
  prof_end(stream);
  return cudaGetLastError();
}

}  // namespace gqa
