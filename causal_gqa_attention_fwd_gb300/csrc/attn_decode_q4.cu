// attn_decode_q4.cu -- cached attention over a 4-bit KV cache (E2M1 codes, an
// E4M3 scale per 16 features, one f32 scale per cache).
#include <math_constants.h>

#include "cache_ops.h"
#include "fp4.cuh"
#include "kernels.h"

namespace gqa {

namespace {

// One CTA per query row, a warp per key, a lane per D/32 features.
template <int D>
__global__ void __launch_bounds__(128) decode_q4_kernel(const DecodeQ4Args a) {
  constexpr int F = D / 32;
  __shared__ float part[4][D];
  __shared__ float2 ml[4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long row = blockIdx.x;                 // (b * Hq + h) * Tq + t
  const int t = (int)(row % a.Tq);
  const int h = (int)(row / a.Tq % a.Hq), b = (int)(row / a.Tq / a.Hq);
  const int len = a.cache_lens[b], hkv = h / a.G;
  if (len < 0 || len > a.S) {
    if (tid == 0) atomicCAS(a.status, 0, kDevBadSeqlens);
    return;
  }
  const int pos = len - a.Tq + t;              // keys 0..pos are visible
  float q[F], acc[F] = {}, m = -CUDART_INF_F, l = 0.f;
  for (int i = 0; i < F; ++i) {
    const int d = lane * F + i;
    float x = __bfloat162float(a.q[row * D + d]);
    if (a.rope_cs && pos >= 0) {
      const bool second = d >= D / 2;
      const float y = __bfloat162float(a.q[row * D + (second ? d - D / 2 : d + D / 2)]);
      const float* cs = a.rope_cs + (long)pos * D + (second ? d - D / 2 : d);
      x = second ? x * cs[0] + y * cs[D / 2] : x * cs[0] - y * cs[D / 2];
    }
    q[i] = x;
  }
  for (int j = warp; j <= pos; j += 4) {
    long r;
    if (a.block_table) {
      const int page = a.block_table[(long)b * a.max_pages + j / a.page_size];
      if (page < 0 || page >= a.num_pages) {
        if (lane == 0) atomicCAS(a.status, 0, kDevBadPage);
        r = -1;
      } else {
        r = ((long)page * a.Hkv + hkv) * a.page_size + j % a.page_size;
      }
    } else {
      r = ((long)b * a.Hkv + hkv) * a.S + j;
    }
    float kk[F] = {}, vv[F] = {};
    if (r >= 0) {
      uint32_t k4[4], v4[4];
      const long c = r * (D / 2) + lane * (F / 2), f = r * (D / 16) + lane * F / 16;
      uint32_t kw = 0, vw = 0;
      for (int i = 0; i < F / 2; ++i) kw |= a.k4[c + i] << (8 * i), vw |= a.v4[c + i] << (8 * i);
      e2m1x8_to_f16(kw, k4);
      e2m1x8_to_f16(vw, v4);
      const float ks = f16x2_to_f32(e4m3x2_to_f16(a.ksf[f])).x, vs = f16x2_to_f32(e4m3x2_to_f16(a.vsf[f])).x;
      for (int i = 0; i < F / 2; ++i) {
        const float2 x = f16x2_to_f32(k4[i]), y = f16x2_to_f32(v4[i]);
        kk[2 * i] = x.x * ks, kk[2 * i + 1] = x.y * ks;
        vv[2 * i] = y.x * vs, vv[2 * i + 1] = y.y * vs;
      }
    }
    float s = 0.f;
    for (int i = 0; i < F; ++i) s += q[i] * kk[i];
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s), w = exp2f(m - mn), p = exp2f(s - mn);
    l = l * w + p;
    for (int i = 0; i < F; ++i) acc[i] = acc[i] * w + p * vv[i];
    m = mn;
  }
  for (int i = 0; i < F; ++i) part[warp][lane * F + i] = acc[i];
  if (lane == 0) ml[warp] = make_float2(m, l);
  __syncthreads();
  float mm = -CUDART_INF_F, ll = 0.f;
  for (int w = 0; w < 4; ++w) mm = fmaxf(mm, ml[w].x);
  const float base = mm == -CUDART_INF_F ? 0.f : mm;
  for (int w = 0; w < 4; ++w) ll += ml[w].y * exp2f(ml[w].x - base);
  if (tid < D) {
    float o = 0.f;
    for (int w = 0; w < 4; ++w) o += part[w][tid] * exp2f(ml[w].x - base);
    a.o[row * D + tid] = __float2bfloat16(pos < 0 ? 0.f : o / ll * a.v_scale);
  }
  if (tid == 0) a.lse[row] = pos < 0 ? -CUDART_INF_F : (mm + log2f(ll)) * 0.69314718055994531f;
}

}  // namespace

size_t decode_q4_ws_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t launch_decode_q4(const DecodeQ4Args& a, int, cudaStream_t stream) {
  const long g = (long)a.B * a.Hq * a.Tq;
  prof_begin(kProfDecode, stream);
  if (a.D == 128) decode_q4_kernel<128><<<(unsigned)g, 128, 0, stream>>>(a);
  else decode_q4_kernel<64><<<(unsigned)g, 128, 0, stream>>>(a);
  prof_end(stream);
  return cudaGetLastError();
}

}  // namespace gqa
