// cache_api.cu -- C entry points of the cache operators (include/gqa_attn.h):
// argument checks and launches.  Every host-detectable error is returned
// before anything is launched.
#include <math.h>
#include <stdint.h>

#include "api_util.h"
#include "cache_ops.h"
#include "gqa_attn.h"

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
cudaStream_t st_of(void* stream) { return static_cast<cudaStream_t>(stream); }
// (as launch_status in api.cu: an error that was returned is not left for the next launch to find)
attn_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return ATTN_OK;
  cudaGetLastError();
  return ATTN_ERR_CUDA;
}

// A token view: strides not negative and multiples of 8 elements, so that every
// row of a 16-byte aligned tensor is 16-byte aligned.
attn_status view(gqa::RowView* r, const void* p, const long long* s) {
  if (!aligned(p, 16)) return ATTN_ERR_ALIGN;
  for (int i = 0; i < 3; ++i) {
    if (s[i] < 0) return ATTN_ERR_SHAPE;
    if (s[i] % 8) return ATTN_ERR_ALIGN;
  }
  r->p = static_cast<const __nv_bfloat16*>(p);
  r->sb = (long)s[0];
  r->st = (long)s[1];
  r->sh = (long)s[2];
  return ATTN_OK;
}

bool scale_ok(float s) { return s >= 1e-20f && s <= 1e20f; }

attn_status rope(const void* q, const void* k, void* qo, void* ko, const int* positions, int pos_stride,
                 const float* cs, int n_table, int B, int T, int Hq, int Hkv, int D, int R, int interleaved,
                 const long long* strides, void* stream, float sign) {
  if (B < 0 || T < 0 || Hq < 0 || Hkv < 0 || Hq + (long)Hkv > 65535 || n_table < 0 || (long)B * T > 0x7fffffffL)
    return ATTN_ERR_SHAPE;
  if (D < 16 || D > 512 || D % 16) return ATTN_ERR_HEADDIM;
  if (R < 16 || R > D || R % 16 || (pos_stride != 0 && pos_stride != T)) return ATTN_ERR_SHAPE;
  if (B == 0 || T == 0 || Hq + Hkv == 0) return ATTN_OK;
  if (!positions || !cs || !strides || (Hq && (!q || !qo)) || (Hkv && (!k || !ko))) return ATTN_ERR_NULL;
  if (!aligned(positions, 4) || !aligned(cs, 16)) return ATTN_ERR_ALIGN;
  gqa::RopeArgs a{};
  attn_status st;
  if (Hq && ((st = view(&a.q, q, strides)) != ATTN_OK || (st = view(&a.qo, qo, strides + 6)) != ATTN_OK)) return st;
  if (Hkv && ((st = view(&a.k, k, strides + 3)) != ATTN_OK || (st = view(&a.ko, ko, strides + 9)) != ATTN_OK))
    return st;
  if ((st = gqa::api_check_arch()) != ATTN_OK) return st;
  a.positions = positions;
  a.pos_stride = pos_stride;
  a.cs = cs;
  a.n_table = n_table;
  a.R = R;
  a.interleaved = interleaved != 0;
  a.sign = sign;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.status = gqa::api_status_word();
  const int sms = gqa::api_sm_count();
  if (!a.status || sms < 1) return ATTN_ERR_CUDA;
  return status_of(gqa::launch_rope(a, sms, st_of(stream)));
}

// What the three append entry points share: everything but the caches' scales.
attn_status append(const void* k, const void* v, const int* slots, const int* positions, const float* cs, int n_table,
                   int R, int interleaved, void* kc, void* ksf, void* vc, void* vsf, float k_scale, float v_scale,
                   int B, int T, int H, int D, int page_size, int num_pages, const long long* strides, void* stream,
                   gqa::CacheFmt fmt) {
  if (B < 0 || T < 0 || page_size < 0 || num_pages < 0 || (long)B * T > 0x7fffffffL) return ATTN_ERR_SHAPE;
  attn_status st = gqa::api_check_heads(H, H, D);
  if (st != ATTN_OK) return st;
  if ((long)page_size * num_pages > 0x7fffffffL) return ATTN_ERR_SHAPE;
  if (cs && (R < 16 || R > D || R % 16 || n_table < 0)) return ATTN_ERR_SHAPE;
  if (fmt != gqa::kCacheBf16 && (!scale_ok(k_scale) || !scale_ok(v_scale))) return ATTN_ERR_SHAPE;
  if (B == 0 || T == 0) return ATTN_OK;
  if ((long)B * T * H * (D / 16) > 0x7fffffffL * 256) return ATTN_ERR_SHAPE;
  if (page_size < 1 || num_pages < 1) return ATTN_ERR_SHAPE;
  if (!k || !v || !slots || !kc || !vc || !strides || (cs && !positions)) return ATTN_ERR_NULL;
  if (fmt == gqa::kCacheQ4 && (!ksf || !vsf)) return ATTN_ERR_NULL;
  if (!aligned(slots, 4) || !aligned(positions, 4) || !aligned(cs, 16) || !aligned(kc, 16) || !aligned(vc, 16) ||
      !aligned(ksf, 16) || !aligned(vsf, 16))
    return ATTN_ERR_ALIGN;
  gqa::AppendArgs a{};
  if ((st = view(&a.k, k, strides)) != ATTN_OK || (st = view(&a.v, v, strides + 3)) != ATTN_OK) return st;
  if ((st = gqa::api_check_arch()) != ATTN_OK) return st;
  a.slots = slots;
  a.positions = positions;
  a.cs = cs;
  a.n_table = n_table;
  a.R = cs ? R : 0;
  a.interleaved = interleaved != 0;
  a.kc = kc;
  a.vc = vc;
  a.ksf = static_cast<uint8_t*>(ksf);
  a.vsf = static_cast<uint8_t*>(vsf);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.k_inv = 1.f / (fmt == gqa::kCacheQ4 ? 6.f * k_scale : k_scale);
  a.v_inv = 1.f / (fmt == gqa::kCacheQ4 ? 6.f * v_scale : v_scale);
  a.B = B;
  a.T = T;
  a.H = H;
  a.D = D;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.status = gqa::api_status_word();
  a.dbg_line = gqa::api_check_line();
  const int sms = gqa::api_sm_count();
  if (!a.status || sms < 1) return ATTN_ERR_CUDA;
  return status_of(gqa::launch_cache_append(a, fmt, sms, st_of(stream)));
}

attn_status decode_q4_check(int B, int Hq, int Hkv, int Tq, int S, int D) {
  if (B < 0 || Tq < 0 || S < 0) return ATTN_ERR_SHAPE;
  const attn_status st = gqa::api_check_heads(Hq, Hkv, D);
  if (st != ATTN_OK) return st;
  if (B == 0 || Tq == 0) return ATTN_OK;
  if (Tq > S) return ATTN_ERR_SHAPE;
  if (S > 0x7fffffff - 32) return ATTN_ERR_SHAPE;   // a row's last 32-key tile ends within 32 bits
  if ((long)B * Hq * Tq > 0x7fffffffL) return ATTN_ERR_SHAPE;
  // the kernel numbers the 32-key tiles (and three more) of all (row, K/V head, block of 8 or 16 query rows) units
  const long blocks = ((long)Hq / Hkv * Tq + 7) / 8;
  if ((long)B * Hkv * blocks > 0x7fffffffL / (S / 32 + 4L)) return ATTN_ERR_SHAPE;
  return ATTN_OK;
}

attn_status decode_q4(const void* q, const void* k4, const void* ksf, const void* v4, const void* vsf, float k_scale,
                      float v_scale, const int* block_table, const int* cache_lens, void* o, float* lse, void* ws,
                      size_t ws_bytes, int B, int Hq, int Hkv, int Tq, int S, int D, int page_size, int num_pages,
                      int max_pages, float scale, const float* cs, int n_table, void* stream) {
  const float scale_log2 = scale * k_scale * 1.4426950408889634f;
  if (!isfinite(scale_log2) || !isfinite(scale) || !isfinite(k_scale) || !isfinite(v_scale)) return ATTN_ERR_SHAPE;
  if (!q || !k4 || !ksf || !v4 || !vsf || !cache_lens || !o || !lse) return ATTN_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k4, 16) || !aligned(ksf, 16) || !aligned(v4, 16) || !aligned(vsf, 16) ||
      !aligned(o, 16) || !aligned(lse, 16) || !aligned(cache_lens, 4) || !aligned(block_table, 4))
    return ATTN_ERR_ALIGN;
  if (cs) {
    if (!aligned(cs, 16)) return ATTN_ERR_ALIGN;
    if (n_table < S) return ATTN_ERR_SHAPE;
  }
  const size_t need = gqa::decode_q4_ws_bytes(B, Hq, Hkv, Tq, S, D);
  if (need > 0 && (!ws || ws_bytes < need || !aligned(ws, 256))) return ATTN_ERR_WORKSPACE;
  const attn_status st = gqa::api_check_arch();
  if (st != ATTN_OK) return st;
  gqa::DecodeQ4Args a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k4 = static_cast<const uint8_t*>(k4);
  a.ksf = static_cast<const uint8_t*>(ksf);
  a.v4 = static_cast<const uint8_t*>(v4);
  a.vsf = static_cast<const uint8_t*>(vsf);
  a.block_table = block_table;
  a.cache_lens = cache_lens;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.ws = ws;
  a.rope_cs = cs;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.Tq = Tq;
  a.R = a.G * Tq;
  a.S = S;
  a.D = D;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.scale_log2 = scale_log2;
  a.v_scale = v_scale;
  a.status = gqa::api_status_word();
  a.dbg_line = gqa::api_check_line();
  const int sms = gqa::api_sm_count();
  if (!a.status || sms < 1) return ATTN_ERR_CUDA;
  return status_of(gqa::launch_decode_q4(a, sms, st_of(stream)));
}

// What the three entry points share.  Contiguous caches: no block table, page_size = S, num_pages = B.
attn_status cache_weights(const void* q, const void* k, const void* ksf, float k_scale, const float* lse,
                          const int* block_table, const int* cache_lens, float* weights, int B, int Hq, int Hkv, int Tq,
                          int page_size, int num_pages, int max_pages, int D, float scale, void* stream,
                          gqa::CacheFmt fmt) {
  if (B < 0 || Tq < 0 || page_size < 0 || num_pages < 0 || max_pages < 0) return ATTN_ERR_SHAPE;
  attn_status st = gqa::api_check_heads(Hq, Hkv, D);
  if (st != ATTN_OK) return st;
  const long S = block_table ? (long)page_size * max_pages : page_size;
  const float scale_log2 = scale * k_scale * 1.4426950408889634f;
  if (S > 0x7fffffffL - 512 || (long)page_size * num_pages > 0x7fffffffL || !isfinite(scale_log2) || !isfinite(scale) ||
      !isfinite(k_scale) || (Tq > 0 && (long)B * Hq > 0x3fffffffL / Tq) || (long)B * max_pages > 0x7fffffffL ||
      (long)B * Hkv > 0x7fffffffL / ((S + 31) / 32 + 1))
    return ATTN_ERR_SHAPE;
  if (B == 0) return ATTN_OK;      // (a block table without rows may be NULL)
  if (!block_table && num_pages != B) return ATTN_ERR_SHAPE;
  if (Tq == 0 || S == 0) return ATTN_OK;
  if (num_pages < 1) return ATTN_ERR_SHAPE;
  if (!q || !k || !lse || !cache_lens || !weights || (fmt == gqa::kCacheQ4 && !ksf)) return ATTN_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(ksf, 16) || !aligned(lse, 16) || !aligned(weights, 16) ||
      !aligned(cache_lens, 4) || !aligned(block_table, 4))
    return ATTN_ERR_ALIGN;
  if ((st = gqa::api_check_arch()) != ATTN_OK) return st;
  gqa::WeightsArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const uint8_t*>(k);
  a.ksf = static_cast<const uint8_t*>(ksf);
  a.lse = lse;
  a.block_table = block_table;
  a.cache_lens = cache_lens;
  a.weights = weights;
  a.B = B;
  a.Hkv = Hkv;
  a.Tq = Tq;
  a.R = Hq / Hkv * Tq;
  a.S = (int)S;
  a.D = D;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.scale_log2 = scale_log2;
  a.status = gqa::api_status_word();
  const int sms = gqa::api_sm_count();
  if (!a.status || sms < 1) return ATTN_ERR_CUDA;
  return status_of(gqa::launch_cache_weights(a, fmt, sms, st_of(stream)));
}

// Whether [p, p + n) and [q, q + m) (bytes) share one.
bool overlap(const void* p, long n, const void* q, long m) {
  const char *a = static_cast<const char*>(p), *b = static_cast<const char*>(q);
  return a && b && n > 0 && m > 0 && a < b + m && b < a + n;
}

}  // namespace

extern "C" {

attn_status attn_cache_weights(const void* q, const void* k_cache, const float* lse, const int* block_table,
                               const int* cache_lens, float* weights, int B, int Hq, int Hkv, int Tq, int page_size,
                               int num_pages, int max_pages, int D, float scale, void* stream) {
  return cache_weights(q, k_cache, nullptr, 1.f, lse, block_table, cache_lens, weights, B, Hq, Hkv, Tq, page_size,
                       num_pages, max_pages, D, scale, stream, gqa::kCacheBf16);
}

attn_status attn_cache_weights_fp8(const void* q, const void* k8, float k_scale, const float* lse, const int* block_table,
                                   const int* cache_lens, float* weights, int B, int Hq, int Hkv, int Tq, int page_size,
                                   int num_pages, int max_pages, int D, float scale, void* stream) {
  return cache_weights(q, k8, nullptr, k_scale, lse, block_table, cache_lens, weights, B, Hq, Hkv, Tq, page_size,
                       num_pages, max_pages, D, scale, stream, gqa::kCacheE4m3);
}

attn_status attn_cache_weights_q4(const void* q, const void* k4, const void* k4_sf, float k_scale, const float* lse,
                                  const int* block_table, const int* cache_lens, float* weights, int B, int Hq, int Hkv,
                                  int Tq, int page_size, int num_pages, int max_pages, int D, float scale, void* stream) {
  return cache_weights(q, k4, k4_sf, k_scale, lse, block_table, cache_lens, weights, B, Hq, Hkv, Tq, page_size, num_pages,
                       max_pages, D, scale, stream, gqa::kCacheQ4);
}

attn_status attn_cache_evict(float* weights, void* const* planes, const int* row_bytes, int num_planes,
                             const int* block_table, const int* cache_lens, int budget, int recent, int first, int* kept,
                             int* lens_out, int B, int Hkv, int page_size, int num_pages, int max_pages, void* stream) {
  if (B < 0 || Hkv < 1 || Hkv > 65535 || page_size < 0 || num_pages < 0 || max_pages < 0 || num_planes < 0 ||
      num_planes > gqa::kEvictPlanes || budget < 1 || recent < 0 || first < 0 || (long)first + recent > budget)
    return ATTN_ERR_SHAPE;
  const long S = block_table ? (long)page_size * max_pages : page_size;
  if (S > 0x7fffffffL - 2048 || (long)page_size * num_pages > 0x7fffffffL || (long)B * Hkv > 0x7fffffffL ||
      (long)B * max_pages > 0x7fffffffL || budget > 0x7fffffff - 4096)
    return ATTN_ERR_SHAPE;
  if (B > 0 && !block_table && num_pages != B) return ATTN_ERR_SHAPE;      // (one without rows may be NULL)
  if (num_planes > 0 && (!planes || !row_bytes)) return ATTN_ERR_NULL;
  for (int i = 0; i < num_planes; ++i)
    if (row_bytes[i] < 4 || row_bytes[i] % 4 || row_bytes[i] > 4096) return ATTN_ERR_SHAPE;
  if (B == 0) return ATTN_OK;
  if (!cache_lens || !kept || !lens_out) return ATTN_ERR_NULL;
  const long slots = (long)num_pages * Hkv * page_size;
  if (slots > 0) {
    if (!weights) return ATTN_ERR_NULL;
    for (int i = 0; i < num_planes; ++i)
      if (!planes[i]) return ATTN_ERR_NULL;
  }
  if (!aligned(weights, 16) || !aligned(cache_lens, 4) || !aligned(block_table, 4) || !aligned(kept, 4) ||
      !aligned(lens_out, 4))
    return ATTN_ERR_ALIGN;
  for (int i = 0; i < num_planes; ++i)
    if (!aligned(planes[i], 16)) return ATTN_ERR_ALIGN;
  // the lengths and the table are read while rows move and the outputs are written, and no plane may be another's
  gqa::EvictArgs a{};
  a.planes[num_planes].p = weights;      // the smallest rows last
  a.planes[num_planes].row_bytes = 4;
  for (int i = 0; i < num_planes; ++i) {
    a.planes[i].p = planes[i];
    a.planes[i].row_bytes = row_bytes[i];
  }
  const struct { const void* p; long n; } io[] = {{cache_lens, 4L * B}, {block_table, 4L * B * max_pages},
                                                  {kept, 4L * B * Hkv * budget}, {lens_out, 4L * B}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 2; j < 4; ++j)
      if (i != j && overlap(io[i].p, io[i].n, io[j].p, io[j].n)) return ATTN_ERR_SHAPE;
    for (int j = 0; j <= num_planes; ++j)
      if (overlap(io[i].p, io[i].n, a.planes[j].p, slots * a.planes[j].row_bytes)) return ATTN_ERR_SHAPE;
  }
  for (int i = 0; i <= num_planes; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(a.planes[i].p, slots * a.planes[i].row_bytes, a.planes[j].p, slots * a.planes[j].row_bytes))
        return ATTN_ERR_SHAPE;
  const attn_status st = gqa::api_check_arch();
  if (st != ATTN_OK) return st;
  a.weights = weights;
  a.n_planes = num_planes + 1;
  a.block_table = block_table;
  a.cache_lens = cache_lens;
  a.kept = kept;
  a.lens_out = lens_out;
  a.B = B;
  a.Hkv = Hkv;
  a.S = (int)S;
  a.page_size = page_size > 0 ? page_size : 1;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.budget = budget;
  a.recent = recent;
  a.first = first;
  a.status = gqa::api_status_word();
  if (!a.status) return ATTN_ERR_CUDA;
  return status_of(gqa::launch_cache_evict(a, st_of(stream)));
}

attn_status attn_cache_plan(const int* cache_lens, const int* new_lens, int* block_table, const int* free_pages,
                            const int* cursor, int* slots, int* positions, int* cu_seqlens, int* lens_out,
                            int* cursor_out, int B, int page_size, int max_pages, int num_free, int total_tokens,
                            void* stream) {
  if (B < 0 || B > gqa::kPlanMaxB || page_size < 1 || max_pages < 0 || num_free < 0 || total_tokens < 0 ||
      (long)B * max_pages > 0x7fffffffL || (long)max_pages * page_size > 0x7fffffffL)
    return ATTN_ERR_SHAPE;
  if (!cu_seqlens || !cursor_out || (total_tokens > 0 && (!slots || !positions)) ||
      (B > 0 && (!cache_lens || !new_lens || !lens_out)) || ((long)B * max_pages > 0 && !block_table) ||
      (num_free > 0 && !free_pages))
    return ATTN_ERR_NULL;
  const void* all[] = {cache_lens, new_lens, block_table, free_pages, cursor, slots, positions, cu_seqlens, lens_out,
                       cursor_out};
  for (const void* p : all)
    if (!aligned(p, 4)) return ATTN_ERR_ALIGN;
  // several CTAs read the inputs while others write: no output may replace an entry of them
  const struct { const int* p; long n; } in[] = {{cache_lens, B}, {new_lens, B}, {cursor, 1}, {free_pages, num_free},
                                                 {block_table, (long)B * max_pages}},
      out[] = {{slots, total_tokens}, {positions, total_tokens}, {cu_seqlens, B + 1L}, {lens_out, B}, {cursor_out, 1}};
  for (const auto& i : in)
    for (const auto& o : out)
      if (i.p && o.p && i.n > 0 && o.n > 0 && i.p < o.p + o.n && o.p < i.p + i.n) return ATTN_ERR_SHAPE;
  const attn_status st = gqa::api_check_arch();
  if (st != ATTN_OK) return st;
  gqa::PlanArgs a{cache_lens, new_lens, free_pages, cursor,    block_table, slots, positions,    cu_seqlens,
                  lens_out,   cursor_out, B,        page_size, max_pages,   num_free, total_tokens, gqa::api_status_word()};
  const int sms = gqa::api_sm_count();
  if (!a.status || sms < 1) return ATTN_ERR_CUDA;
  return status_of(gqa::launch_cache_plan(a, sms, st_of(stream)));
}

attn_status attn_rope_table(float* rope_cos_sin, int n, int rotary_dim, double base, double factor,
                            int original_positions, double low_turns, double high_turns, double mscale,
                            void* stream) {
  if (n < 0 || rotary_dim < 16 || rotary_dim > 512 || rotary_dim % 16 || original_positions < 0) return ATTN_ERR_SHAPE;
  if (!isfinite(base) || !isfinite(factor) || !isfinite(low_turns) || !isfinite(high_turns) || !isfinite(mscale) ||
      base <= 1.0 || factor <= 0.0 || low_turns >= high_turns || !isfinite((float)mscale) || !isfinite(1.0 / factor))
    return ATTN_ERR_SHAPE;
  if (n == 0) return ATTN_OK;
  if (!rope_cos_sin) return ATTN_ERR_NULL;
  if (!aligned(rope_cos_sin, 16)) return ATTN_ERR_ALIGN;
  const attn_status st = gqa::api_check_arch();
  if (st != ATTN_OK) return st;
  gqa::RopeTableArgs a{};
  a.out = rope_cos_sin;
  a.n = n;
  a.R = rotary_dim;
  a.base = base;
  a.factor = factor;
  a.turns = original_positions * 0.15915494309189533576888;
  a.low = low_turns;
  a.high = high_turns;
  a.mscale = (float)mscale;
  const int sms = gqa::api_sm_count();
  if (sms < 1) return ATTN_ERR_CUDA;
  return status_of(gqa::launch_rope_table(a, sms, st_of(stream)));
}

attn_status attn_rope(const void* q, const void* k, void* q_out, void* k_out, const int* positions,
                      int positions_stride, const float* rope_cos_sin, int rope_positions, int B, int T, int Hq,
                      int Hkv, int D, int rotary_dim, int interleaved, const long long* strides, void* stream) {
  return rope(q, k, q_out, k_out, positions, positions_stride, rope_cos_sin, rope_positions, B, T, Hq, Hkv, D,
              rotary_dim, interleaved, strides, stream, 1.f);
}

attn_status attn_rope_bwd(const void* dq_out, const void* dk_out, void* dq, void* dk, const int* positions,
                          int positions_stride, const float* rope_cos_sin, int rope_positions, int B, int T, int Hq,
                          int Hkv, int D, int rotary_dim, int interleaved, const long long* strides, void* stream) {
  return rope(dq_out, dk_out, dq, dk, positions, positions_stride, rope_cos_sin, rope_positions, B, T, Hq, Hkv, D,
              rotary_dim, interleaved, strides, stream, -1.f);
}

attn_status attn_cache_append(const void* k, const void* v, const int* slots, const int* positions,
                              const float* rope_cos_sin, int rope_positions, int rotary_dim, int interleaved,
                              void* k_cache, void* v_cache, int B, int T, int Hkv, int D, int page_size,
                              int num_pages, const long long* strides, void* stream) {
  return append(k, v, slots, positions, rope_cos_sin, rope_positions, rotary_dim, interleaved, k_cache, nullptr,
                v_cache, nullptr, 1.f, 1.f, B, T, Hkv, D, page_size, num_pages, strides, stream, gqa::kCacheBf16);
}

attn_status attn_cache_append_fp8(const void* k, const void* v, const int* slots, const int* positions,
                                  const float* rope_cos_sin, int rope_positions, int rotary_dim, int interleaved,
                                  void* k8, void* v8, float k_scale, float v_scale, int B, int T, int Hkv, int D,
                                  int page_size, int num_pages, const long long* strides, void* stream) {
  return append(k, v, slots, positions, rope_cos_sin, rope_positions, rotary_dim, interleaved, k8, nullptr, v8,
                nullptr, k_scale, v_scale, B, T, Hkv, D, page_size, num_pages, strides, stream, gqa::kCacheE4m3);
}

attn_status attn_cache_append_q4(const void* k, const void* v, const int* slots, const int* positions,
                                 const float* rope_cos_sin, int rope_positions, int rotary_dim, int interleaved,
                                 void* k4, void* k4_sf, void* v4, void* v4_sf, float k_scale, float v_scale, int B,
                                 int T, int Hkv, int D, int page_size, int num_pages, const long long* strides,
                                 void* stream) {
  return append(k, v, slots, positions, rope_cos_sin, rope_positions, rotary_dim, interleaved, k4, k4_sf, v4, v4_sf,
                k_scale, v_scale, B, T, Hkv, D, page_size, num_pages, strides, stream, gqa::kCacheQ4);
}

attn_status attn_cache_gather_q4(const int* slots, const void* k4, const void* k4_sf, const void* v4,
                                 const void* v4_sf, float k_scale, float v_scale, void* k, void* v, int tokens,
                                 int Hkv, int D, int page_size, int num_pages, void* stream) {
  if (tokens < 0 || page_size < 0 || num_pages < 0) return ATTN_ERR_SHAPE;
  attn_status st = gqa::api_check_heads(Hkv, Hkv, D);
  if (st != ATTN_OK) return st;
  if ((long)page_size * num_pages > 0x7fffffffL || !isfinite(k_scale) || !isfinite(v_scale)) return ATTN_ERR_SHAPE;
  if (tokens == 0) return ATTN_OK;
  if ((long)tokens * Hkv * (D / 16) > 0x7fffffffL * 256 || page_size < 1 || num_pages < 1) return ATTN_ERR_SHAPE;
  if (!slots || !k4 || !k4_sf || !v4 || !v4_sf || !k || !v) return ATTN_ERR_NULL;
  if (!aligned(slots, 4) || !aligned(k4, 16) || !aligned(k4_sf, 16) || !aligned(v4, 16) || !aligned(v4_sf, 16) ||
      !aligned(k, 16) || !aligned(v, 16))
    return ATTN_ERR_ALIGN;
  if ((st = gqa::api_check_arch()) != ATTN_OK) return st;
  gqa::GatherArgs a{};
  a.slots = slots;
  a.k4 = static_cast<const uint8_t*>(k4);
  a.ksf = static_cast<const uint8_t*>(k4_sf);
  a.v4 = static_cast<const uint8_t*>(v4);
  a.vsf = static_cast<const uint8_t*>(v4_sf);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.k = static_cast<__nv_bfloat16*>(k);
  a.v = static_cast<__nv_bfloat16*>(v);
  a.tokens = tokens;
  a.H = Hkv;
  a.D = D;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.status = gqa::api_status_word();
  const int sms = gqa::api_sm_count();
  if (!a.status || sms < 1) return ATTN_ERR_CUDA;
  return status_of(gqa::launch_cache_gather(a, sms, st_of(stream)));
}

size_t attn_decode_q4_workspace_size(int B, int Hq, int Hkv, int Tq, int S, int D) {
  if (decode_q4_check(B, Hq, Hkv, Tq, S, D) != ATTN_OK || B == 0 || Tq == 0) return 0;
  return gqa::decode_q4_ws_bytes(B, Hq, Hkv, Tq, S, D);
}

attn_status attn_decode_q4_fwd(const void* q, const void* k4, const void* k4_sf, const void* v4, const void* v4_sf,
                               float k_scale, float v_scale, const int* cache_lens, void* o, float* lse,
                               void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv, int Tq, int S, int D,
                               float scale, const float* rope_cos_sin, int rope_positions, void* stream) {
  const attn_status st = decode_q4_check(B, Hq, Hkv, Tq, S, D);
  if (st != ATTN_OK) return st;
  if (B == 0 || Tq == 0) return ATTN_OK;
  return decode_q4(q, k4, k4_sf, v4, v4_sf, k_scale, v_scale, nullptr, cache_lens, o, lse, workspace,
                   workspace_bytes, B, Hq, Hkv, Tq, S, D, S, B, 1, scale, rope_cos_sin, rope_positions, stream);
}

attn_status attn_decode_paged_q4_fwd(const void* q, const void* k4_pages, const void* k4_sf_pages,
                                     const void* v4_pages, const void* v4_sf_pages, float k_scale, float v_scale,
                                     const int* block_table, const int* cache_lens, void* o, float* lse,
                                     void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv, int Tq,
                                     int page_size, int num_pages, int max_pages, int D, float scale,
                                     const float* rope_cos_sin, int rope_positions, void* stream) {
  if (page_size < 0 || num_pages < 0 || max_pages < 0) return ATTN_ERR_SHAPE;
  const long S = (long)page_size * max_pages;
  if (S > 0x7fffffffL) return ATTN_ERR_SHAPE;
  const attn_status st = decode_q4_check(B, Hq, Hkv, Tq, (int)S, D);
  if (st != ATTN_OK) return st;
  if (B == 0 || Tq == 0) return ATTN_OK;
  const bool size_ok = page_size == 16 || page_size == 32 || page_size == 64 || (page_size > 0 && page_size % 128 == 0);
  if (!size_ok || num_pages < 1 || (long)B * max_pages > 0x7fffffffL) return ATTN_ERR_SHAPE;
  if (!block_table) return ATTN_ERR_NULL;
  return decode_q4(q, k4_pages, k4_sf_pages, v4_pages, v4_sf_pages, k_scale, v_scale, block_table, cache_lens, o, lse,
                   workspace, workspace_bytes, B, Hq, Hkv, Tq, (int)S, D, page_size, num_pages, max_pages, scale,
                   rope_cos_sin, rope_positions, stream);
}

}  // extern "C"
