// Launcher of the sliding-window extend: the extend pipeline (extend_dev.cuh)
// over the keys each CTA's queries see.
#include "extend_dev.cuh"
#include "launch.h"

namespace sgl {

using namespace ext;

namespace {

template <int D, bool kFp8>
sgl_status run(const Params& prm, int32_t batch, int32_t max_extend, cudaStream_t stream) {
  constexpr int kThreads = Roles<kFp8>::kThreads;
  constexpr int kSmem = smem_bytes<D, kFp8>();
  if (kernel_blocks_per_sm<extend_kernel<D, kFp8, true>>(kSmem, kThreads) < 0) return SGL_ERR_CUDA;
  if (Roles<kFp8>::kSplitRegs && !kernel_regs_at_least<extend_kernel<D, kFp8, true>>(Roles<kFp8>::kLaunchRegs))
    return SGL_ERR_UNSUPPORTED;
  const int per_cta = 2 * prm.tpt;
  const dim3 grid((unsigned)((max_extend + per_cta - 1) / per_cta), (unsigned)prm.Hkv, (unsigned)batch);
  extend_kernel<D, kFp8, true><<<grid, kThreads, kSmem, stream>>>(prm);
  return cudaGetLastError() == cudaSuccess ? SGL_OK : SGL_ERR_CUDA;
}

}  // namespace

sgl_status launch_extend_window(const ExtendArgs& a, cudaStream_t stream) {
  if (a.batch == 0 || a.total_extend == 0 || a.max_extend == 0) return SGL_OK;
  Params prm;
  const sgl_status st = make_extend_params(a, &prm);
  if (st != SGL_OK) return st;
  if (a.head_dim == 128)
    return a.kv_fp8 ? run<128, true>(prm, a.batch, a.max_extend, stream)
                    : run<128, false>(prm, a.batch, a.max_extend, stream);
  if (a.head_dim == 64)
    return a.kv_fp8 ? run<64, true>(prm, a.batch, a.max_extend, stream)
                    : run<64, false>(prm, a.batch, a.max_extend, stream);
  return SGL_ERR_UNSUPPORTED;
}

}  // namespace sgl
