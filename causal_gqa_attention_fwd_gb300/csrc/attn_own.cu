// attn_own.cu -- attention over shared prefixes where few rows share one: the
// prefixes and the rows' own keys as one stream of tiles (own_keys.cuh).
#include "own_keys.cuh"

namespace gqa {

template <int D, bool PAGED, int NT>
__global__ void __launch_bounds__(32 * OwnCfg<D, NT>::kWarps, 1)
    attn_own_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_pk, const __grid_constant__ CUtensorMap tm_pv, const OwnArgs a) {
  constexpr int kThreads = 32 * OwnCfg<D, NT>::kWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ OwnShared<D, NT, kThreads> shared;
  __shared__ int s_abort;
  const Guard guard{&s_abort, a.status};
  if (threadIdx.x == 0) s_abort = 0;
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.P + a.B; i += kThreads) {
      int len;
      if (row_tiles<OwnCfg<D, NT>::KT>(a, i, len) == 0 && len != 0) atomicCAS(a.status, 0, kDevBadSeqlens);
    }
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0);
  // neighbouring shares go to different SMs
  own_keys<D, PAGED, NT, kThreads>(smem, shared, tm_k, tm_v, tm_pk, tm_pv, a, warp * gridDim.x + blockIdx.x,
                                   gridDim.x * OwnCfg<D, NT>::kWarps, guard);
}

template <int D, bool PAGED, int NT>
static cudaError_t launch_own_n(const OwnMaps& m, const OwnArgs& a, cudaStream_t stream) {
  using C = OwnCfg<D, NT>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(attn_own_kernel<D, PAGED, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[dev] = true;
  }
  prof_begin(kProfOwn, stream);
  const cudaError_t e = launch_programmatic(attn_own_kernel<D, PAGED, NT>, dim3(a.ctas), dim3(32 * C::kWarps),
                                            C::kSmemBytes, stream, m.k, m.v, m.pk, m.pv, a);
  prof_end(stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D>
static cudaError_t launch_own_d(const OwnMaps& m, const OwnArgs& a, cudaStream_t stream) {
  const bool paged = a.block_table != nullptr;
  if (a.block == 8) return paged ? launch_own_n<D, true, 1>(m, a, stream) : launch_own_n<D, false, 1>(m, a, stream);
  return paged ? launch_own_n<D, true, 2>(m, a, stream) : launch_own_n<D, false, 2>(m, a, stream);
}

cudaError_t launch_attn_own(const OwnMaps& m, const OwnArgs& a, cudaStream_t stream) {
  return a.D == 128 ? launch_own_d<128>(m, a, stream) : launch_own_d<64>(m, a, stream);
}

}  // namespace gqa
