// kernels.h -- internal launch interface between the C-ABI layer (api.cu) and
// the kernel translation units.  Not part of the public header.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace gqa {

// Forward.  Dense layout: Q,O [B,Hq,T,D], K,V [B,Hkv,T,D], LSE [B,Hq,T]
// (num_seqs = B).  Packed layout (varlen = 1): Q,O [total,Hq,D],
// K,V [total,Hkv,D], LSE [Hq,total], sequences [cu[s], cu[s+1]).
struct FwdArgs {
  __nv_bfloat16* o;
  float* lse;
  const int* cu_seqlens;  // device, varlen only
  int* status;            // device status word
  int num_seqs;           // B for the dense layout
  int T;                  // dense sequence length (unused for varlen)
  int total;              // varlen total tokens
  int Hq, Hkv, G;
  int causal;
  int varlen;
  int pair_heads;         // 1: a CTA's two tiles are heads 2p, 2p+1; 0: row blocks 2m, 2m+1
  int pairs_per_seq;      // head pairs (pair_heads) or heads
  int m_items;            // row-block items per sequence
  float scale_log2;       // scale * log2(e)
  // failure-path test only (attn_test_inject_timeout): when inject_step >= 0,
  // CTA 0's producer stops before the load of that step and every wait of
  // the launch gives up after wait_ns
  int inject_step;
  uint64_t wait_ns;
  int* dbg_line;          // debug builds: source line of the first failed bounds check
};

cudaError_t launch_attn_fwd(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const FwdArgs& a,
                            int D, int grid, cudaStream_t stream);

// Backward.  Same layouts; the workspace holds -Delta and -LSE*log2(e) per
// query row (row-padded to whole 128-row tiles).
struct BwdArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* o;
  const __nv_bfloat16* dout;
  const float* lse;
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  float* delta;           // workspace: -Delta, [B,Hq,T_pad] or [Hq,total_pad]
  float* lse_log2;        // workspace: -LSE * log2(e), same layout as delta
  int* tile_counter;      // workspace: the dQ kernel's next tile (zeroed by the preprocess)
  const int* cu_seqlens;
  int* status;
  int num_seqs;
  int T;                  // dense sequence length; varlen: the longest sequence
  int T_pad;              // dense rows per head in the f32 workspaces
  int total;
  int total_pad;          // varlen rows per head in the f32 workspaces
  int Hq, Hkv, G;
  int D;
  int causal;
  int varlen;
  int n_items;            // key-block items per sequence (max)
  float scale;
  float scale_log2;
  // rotary backward (f16 Q/K copies): [positions, D] cos/sin table; dK and
  // dQ rows get the transposed rotation at their positions
  const float* rope_cs;
  // failure-path test only (attn_test_inject_timeout): in the kernel named by
  // inject_kernel (1 dK/dV, 2 dQ), the producer of CTA 0 (dK/dV) or of the
  // CTA that takes the first tile (dQ) stops before the load of step
  // inject_step, and every wait gives up after wait_ns
  int inject_kernel;
  int inject_step;
  uint64_t wait_ns;
  long ws_rows;           // rows of each workspace section (bounds of the debug build)
  int n_table;            // rows of rope_cs
  int* dbg_line;          // debug builds: source line of the first failed bounds check
};

// The preprocess, then the dK/dV and dQ kernels.  f16qk: q and k are the f16
// rotated copies (the rotary backward).
cudaError_t launch_attn_bwd(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            const CUtensorMap& dout, const BwdArgs& a, cudaStream_t stream, bool f16qk = false);

// After the preprocess: the key/value-stationary dK/dV kernel and the
// query-stationary dQ kernel (attn_bwd_split.cu).  f16qk: q and k are the
// f16 rotated copies (the rotary backward).
cudaError_t launch_attn_bwd_split(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                  const CUtensorMap& dout, const BwdArgs& a, bool f16qk, cudaStream_t stream);


// Cached (decode) attention.  Q, O [B,Hq,Tq,D]; K/V cache [B,Hkv,S,D];
// LSE [B,Hq,Tq]; cache_lens [B].  The R = G*Tq query rows of a (row, K/V
// head) pair are processed in nrb blocks of 16; a (row, K/V head, block) is
// a unit, u = (b*Hkv + hkv)*nrb + block.  The ctas CTAs share the stream of
// the units' 128-key chunks evenly; a unit cut between CTAs leaves one
// partial per piece in ws_o / ws_ml ([unit][slot][rows_ws]) and a merge
// kernel produces its O and LSE.
constexpr int kDecodeMaxSlots = 160;  // pieces per unit the workspace holds (>= CTAs launched)

struct DecodeArgs {
  const __nv_bfloat16* q;
  const int* cache_lens;  // device
  __nv_bfloat16* o;
  float* lse;
  float* ws_o;            // [units * slots * rows_ws, D] f32 (slots > 1)
  float2* ws_ml;          // [units * slots * rows_ws] (max in log2 units, sum)
  int* status;
  int B, Hq, Hkv, G, Tq, S, D, R;
  int nrb;                // row blocks per (row, K/V head)
  int slots;              // workspace slots per unit: min(chunks at capacity S, kDecodeMaxSlots)
  int rows_ws;            // rows per slot: min(R, 16)
  int ctas;               // CTAs of the partial kernel
  float scale_log2;
  // paged caches (k, v maps over [num_pages * Hkv, page_size, D]): key
  // position j of row b is row j % page_size of page block_table[b * max_pages + j / page_size]
  const int* block_table; // device, nullptr for contiguous caches
  int page_size, max_pages, num_pages;
  // rotary queries: rope_cs [positions, D] f32 (cos half, then sin half), nullptr = none
  const float* rope_cs;
  // FP8 (E4M3) caches: the k, v maps are 8-bit ([.., D] rows, 128-key
  // boxes, no swizzle); K's scale is folded into scale_log2, V's applied to O
  int fp8;
  float v_scale;          // 1 for 16-bit caches
};

// k, v: dense maps over the caches ([B*Hkv, S, D], 64 x 128 boxes) or, paged,
// over the pages ([num_pages*Hkv, page_size, D], 64 x min(page_size, 128)
// boxes); q: 2-D map over the query rows ([B*Hq*Tq, D], 64 x 16 boxes).
cudaError_t launch_attn_decode(const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& q, const DecodeArgs& a,
                               int grid, cudaStream_t stream);

// Attention of a batch over prefixes that its rows share: prefix p (p < P) belongs to rows p*W .. p*W + W - 1.  The
// Rp = W*R query rows (R = G*Tq a batch row) of a (prefix, K/V head) go in nrt blocks of 256; a (prefix, K/V head,
// block) is a unit.  CTAs work in teams of `width`: a team takes a share of the stream of 128-key blocks of its
// groups (prefix, K/V head, outer), CTA i of it the unit of row block outer*width + i, so that the CTAs that read the
// same keys read them at the same time.
constexpr int kPrefixRows = 256;
struct PrefixArgs {
  const __nv_bfloat16* q;   // [B, Hkv, R, D]
  const int* prefix_lens;   // [P] device
  const int* table;         // [P, max_pages] device, nullptr for contiguous prefixes
  float* ws_o;              // [P * Hkv * Rp, slots, D]
  float2* ws_ml;            // [P * Hkv * Rp, slots] (max in log2 units, sum)
  int* counts;              // [units] slots in use
  int* status;
  int* dbg_line;
  int P, W, Hkv, R, Rp, nrt, width, outer, ctas, Sp, slots;
  int page_size, max_pages, num_pages;
  float scale_log2;
};

// Few query rows a key: the rows' own keys, R = G*Tq query rows a (batch row, K/V head), and, where few rows share a
// prefix (P > 0), the prefixes, W*R query rows a (prefix, K/V head).  They go in nrb (nrbp) blocks of `block` rows; a
// (row or prefix, K/V head, block) is a unit, the prefixes' units first.  Piece i of the stream (attn_own.cu) leaves
// rows_ws rows at i * rows_ws.
constexpr int kOwnMaxWarps = 160 * 12;
struct OwnArgs {
  const __nv_bfloat16* q;   // [B, Hkv, R, D]
  const int *cache_lens, *prefix_lens;     // [B], [P] device
  const int *block_table, *prefix_table;   // [B, max_pages], [P, max_prefix_pages] device, nullptr for contiguous caches
  float* ws_o;              // [(kOwnMaxWarps + units) * rows_ws, D]
  float2* ws_ml;            // [(kOwnMaxWarps + units) * rows_ws] (max in log2 units, sum)
  int2* counts;             // [units] (first piece, pieces)
  int* status;
  int B, P, W, Hkv, Tq, R, nrb, nrbp, block, rows_ws, S, Sp, D;
  int page_size, max_pages, max_prefix_pages, num_pages;
  int ctas;                 // CTAs of the launch
  float scale_log2;
};
// Maps over the caches or pages with boxes of 64 features x own_box_rows(); pk, pv: of contiguous prefixes.
struct OwnMaps {
  CUtensorMap k, v, pk, pv;
};
// Whether prefixes of Sp keys, Rp query rows each, go into the stream: it reads them again for every 16 rows, from L2,
// where attn_prefix needs some microseconds for its pipeline of large tiles.  Measured (us, stream / attn_prefix; 8 heads
// of 128): 2048 keys, 96 rows 16.4 / 15.9, 128 rows 17.6 / 16.9; 8192 keys, 16 rows 13.7 / 13.7, 32 rows 17.7 / 14.9, 48
// rows 22.0 / 17.4; 3001 keys, 4 heads, 80 rows 15.0 / 16.4; 8 prefixes of 2048, 24 rows 28.5 / 27.8, 48 rows 37.5 / 29.5;
// 8 heads of 64, 32 rows 20.7 / 22.0, 48 rows 25.9 / 25.1; 2 heads, 32768 keys, 56 rows 18.3 / 17.1: about 24 MB read again
// is where they meet; about 96 MB where the units are nearly as many as the CTAs or more, each of which then pays for one
// unit's queries and partials after the other (5 prefixes, 8 heads of 64, 520 rows, 120 units: 128 keys, 41 MB, 34 / 45,
// 384, 124 MB, 42 / 44, 768 56 / 48; 16 prefixes, 8 heads of 128, 32 rows, 128 units: 384 keys, 48 MB, 22.4 / 23.6, 1536,
// 192 MB, 38 / 37; 32 units, 256 rows, 384 keys, 96 MB: 35 / 30).
// Sp is the capacity, all that the host knows; the figures are at lengths equal to it.  A table far wider than its prefix
// sends it to the large tiles: 2048 keys, 2 heads of 64, 56 rows, tables of 2048 / 8192 / 32768 / 131072 positions: 9.9 /
// 9.8 / 11.0 / 11.1 us.
inline bool prefix_in_stream(int Rp, int P, int Hkv, int Sp, int D) {
  const long again = ((long)(Rp + 15) / 16 - 1) * P * Hkv * Sp * D * 4;
  return again <= ((long)P * Hkv * ((Rp + kPrefixRows - 1) / kPrefixRows) < 96 ? 24L << 20 : 96L << 20);
}
inline int own_box_rows(int D, int page_size) {   // page_size 0: contiguous
  const int tile = D == 128 ? 16 : 32;
  return page_size > 0 && page_size < tile ? page_size : tile;
}
// Both as one stream (a.P > 0).
cudaError_t launch_attn_own(const OwnMaps& m, const OwnArgs& a, cudaStream_t stream);
// The prefixes by large tiles (maps k, v with boxes of 128 rows), and beside them, on SMs of its own, the stream of the
// rows' own keys (a.P = 0).
cudaError_t launch_attn_prefix(const CUtensorMap& k, const CUtensorMap& v, const PrefixArgs& p, const OwnMaps& m,
                               const OwnArgs& a, cudaStream_t stream);

// Joins the prefix's partials with those of the rows' own caches: O and LSE of every row.
cudaError_t launch_prefix_merge(const PrefixArgs& p, const OwnArgs& a, __nv_bfloat16* o, float* lse, cudaStream_t stream);

// Kernel-level timing (opt-in instrumentation, api.cu): event pairs recorded
// on the launch stream around each kernel.
enum ProfKind {
  kProfFwd = 0,
  kProfBwdPre = 1,
  kProfBwdDkdv = 2,
  kProfUnused3 = 3,
  kProfDecode = 4,
  kProfDecodeMerge = 5,
  kProfBwdDq = 6,
  kProfPlan = 7,
  kProfRope = 8,
  kProfRopeTable = 9,
  kProfAppend = 10,
  kProfGather = 11,
  kProfPrefix = 12,
  kProfPrefixMerge = 13,
  kProfWeights = 14,
  kProfEvict = 15,
  kProfOwn = 16,
  kProfKinds = 17
};
// Launch with programmatic stream serialization (see griddep_wait in
// sm103.cuh): the kernel's CTAs may be scheduled, and run their set-up, while
// the previous kernel in the stream drains.
template <typename... KArgs, typename... Args>
cudaError_t launch_programmatic_clusters(void (*kernel)(KArgs...), int cluster, dim3 grid, dim3 block, size_t smem,
                                         cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;   // CTAs that neighbour in x
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}
template <typename... KArgs, typename... Args>
cudaError_t launch_programmatic(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                                Args&&... args) {
  return launch_programmatic_clusters(kernel, 1, grid, block, smem, stream, static_cast<Args&&>(args)...);
}

void prof_begin(int kind, cudaStream_t s);
void prof_end(cudaStream_t s);

}  // namespace gqa
