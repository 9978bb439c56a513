// The attention kernels of one head size, chosen by -DQMM_HEAD_DIM.
#include "qmm_paged.cuh"

#ifndef QMM_HEAD_DIM
#error "QMM_HEAD_DIM must be defined"
#endif

namespace qmm {

template <int D, bool E8, int RG>
cudaError_t launch_rows(const AttentionArgs& a, cudaStream_t stream) {
  using Cfg = AttnCfg<D, E8, RG>;
  auto kern = attention_kernel<D, E8, RG>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(a.parts), kAttnThreads, Cfg::SMEM, stream, a);
}

template <int D>
cudaError_t launch_attention(AttentionArgs a, bool e8, cudaStream_t stream) {
  const cudaError_t e = a.RB == 16   ? (e8 ? launch_rows<D, true, 1>(a, stream) : launch_rows<D, false, 1>(a, stream))
                        : a.RB == 32 ? (e8 ? launch_rows<D, true, 2>(a, stream) : launch_rows<D, false, 2>(a, stream))
                                     : (e8 ? launch_rows<D, true, 4>(a, stream) : launch_rows<D, false, 4>(a, stream));
  if (e != cudaSuccess) return e;
  const int64_t blocks = static_cast<int64_t>(a.B) * a.c.heads * a.RT * (a.RB / 4);
  return launch_dependent(join_kernel<D>, dim3(static_cast<unsigned>(blocks)), kAttnThreads, 0, stream, a);
}

template <int D>
unsigned int read_attention_status(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_qmm_status, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (clear && v != 0) {
    const unsigned int zero = 0;
    cudaMemcpyToSymbol(g_qmm_status, &zero, sizeof(zero));
  }
  return v;
}

template cudaError_t launch_attention<QMM_HEAD_DIM>(AttentionArgs, bool, cudaStream_t);
template unsigned int read_attention_status<QMM_HEAD_DIM>(int);

}  // namespace qmm
