// cache_ops.h -- internal launch interface of the cache operators: the cache
// plan, rotary positions, appending and gathering, 4-bit cached attention.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "stream.cuh"

namespace gqa {

struct PlanArgs {
  const int *cache_lens, *new_lens, *free_pages, *cursor;
  int* block_table;
  int *slots, *positions, *cu_seqlens, *lens_out, *cursor_out;
  int B, page_size, max_pages, num_free, total;
  int* status;
};
constexpr int kPlanMaxB = 8192;  // requests whose offsets fit a CTA's shared memory
cudaError_t launch_cache_plan(const PlanArgs& a, int sms, cudaStream_t stream);

// A [B, T, H, D] bf16 tensor: element (b, t, h, d) at b*sb + t*st + h*sh + d.
struct RowView {
  const __nv_bfloat16* p;
  long sb, st, sh;
};

// Rotary rows: x rotated by R(pos) (sign +1) or its transpose (sign -1).
struct RopeArgs {
  RowView q, k, qo, ko;      // qo.p and ko.p are written
  const int* positions;
  int pos_stride;            // positions[b * pos_stride + t]
  const float* cs;           // [n_table, R]
  int n_table, R, interleaved;
  float sign;
  int B, T, Hq, Hkv, D;
  int* status;
};
cudaError_t launch_rope(const RopeArgs& a, int sms, cudaStream_t stream);

struct RopeTableArgs {
  float* out;
  int n, R;
  double base, factor, turns;  // turns: original context length / (2 pi), 0 = none
  double low, high;
  float mscale;
};
cudaError_t launch_rope_table(const RopeTableArgs& a, int sms, cudaStream_t stream);

enum CacheFmt { kCacheBf16 = 0, kCacheE4m3 = 1, kCacheQ4 = 2 };

struct AppendArgs {
  RowView k, v;
  const int* slots;
  const int* positions;      // rotary: of token n, nullptr = none
  const float* cs;
  int n_table, R, interleaved;
  void *kc, *vc;             // caches; 4-bit: codes
  uint8_t *ksf, *vsf;        // 4-bit: block scales
  float k_scale, v_scale;
  float k_inv, v_inv;        // E4M3: 1 / scale; 4-bit: 1 / (6 scale), in f32
  int B, T, H, D, page_size, num_pages;
  int* status;
  int* dbg_line;
};
cudaError_t launch_cache_append(const AppendArgs& a, CacheFmt fmt, int sms, cudaStream_t stream);

struct GatherArgs {
  const int* slots;
  const uint8_t *k4, *ksf, *v4, *vsf;
  float k_scale, v_scale;
  __nv_bfloat16 *k, *v;
  int tokens, H, D, page_size, num_pages;
  int* status;
};
cudaError_t launch_cache_gather(const GatherArgs& a, int sms, cudaStream_t stream);

// 4-bit cached attention.  Codes [N, Hkv, P, D/2], block scales
// [N, Hkv, P, D/16]; contiguous caches: N = B, P = S, no block table.
struct DecodeQ4Args {
  const __nv_bfloat16* q;    // [B, Hq, Tq, D]
  const uint8_t *k4, *ksf, *v4, *vsf;
  const int* block_table;    // [B, max_pages] or nullptr
  const int* cache_lens;
  __nv_bfloat16* o;
  float* lse;
  void* ws;
  const float* rope_cs;      // [positions, D] or nullptr
  int B, Hq, Hkv, G, Tq, R, nrb, S, D;
  int cluster;               // CTAs of a unit, 0: units in one stream
  int page_size, max_pages, num_pages;
  float scale_log2;          // softmax scale * k_scale * log2(e)
  float v_scale;
  int* status;
  int* dbg_line;
};
size_t decode_q4_ws_bytes(int B, int Hq, int Hkv, int Tq, int S, int D);
cudaError_t launch_decode_q4(const DecodeQ4Args& a, int sms, cudaStream_t stream);

// Attention weight of cached keys, added to weights [N, Hkv, P] f32 (contiguous
// caches: N = B, P = S, no block table).
struct WeightsArgs {
  const __nv_bfloat16* q;    // [B, Hkv, R, D], R = G * Tq
  const uint8_t *k, *ksf;    // keys (any format), 4-bit: their block scales
  const float* lse;          // [B, Hkv, R]
  const int* block_table;    // [B, max_pages] or nullptr
  const int* cache_lens;
  float* weights;
  int B, Hkv, Tq, R, S, D, page_size, max_pages, num_pages;
  float scale_log2;          // softmax scale * k_scale * log2(e)
  FastDiv page;              // page_size (set by the launch)
  int scan;                  // CTAs look for their keys by the lengths (set by the launch)
  int* status;
};
cudaError_t launch_cache_weights(WeightsArgs a, CacheFmt fmt, int sms, cudaStream_t stream);

// Eviction.  The planes [N, Hkv, P, row_bytes] of a cache, the weights among them.
constexpr int kEvictPlanes = 8;
struct EvictPlane {
  void* p;
  int row_bytes;
  int size, parts, run;      // bytes a lane moves, such parts of a row, rows a warp moves at once (set by the launch)
};
struct EvictArgs {
  const float* weights;
  EvictPlane planes[kEvictPlanes + 1];
  int n_planes;
  const int* block_table;    // [B, max_pages] or nullptr
  const int* cache_lens;
  int *kept, *lens_out;      // [B, Hkv, budget], [B]
  int B, Hkv, S, page_size, max_pages, num_pages;
  int budget, recent, first;
  // set by the launch: CTAs of a unit; shared memory for a CTA's weights, 0: they do not fit; rows the cluster holds at once
  int cluster, key_bytes, hold;
  FastDiv page;              // page_size
  int shared_select;         // the cluster selects together and the list is `kept`; otherwise each CTA does, into its own
  int* status;
};
cudaError_t launch_cache_evict(EvictArgs a, cudaStream_t stream);

}  // namespace gqa
