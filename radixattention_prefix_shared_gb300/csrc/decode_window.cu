// Launchers of the sliding-window decode: the split kernel's work loop
// (decode_dev.cuh) over each request's visible keys, one run of them a CTA,
// and the combine of requests with more than one run.
//
// A request's visible keys number at most sinks + window whatever its length,
// so the host knows every CTA's share from its own arguments: no plan kernel
// and no work counters, one launch where a run holds a whole request.
#include "decode_dev.cuh"
#include "launch.h"

namespace sgl {

using namespace dec;

namespace {

// Runs are made as short as it takes to give the part kFillUnits units of
// work, but no shorter than kMinRun keys and no longer than kItemMax (the
// slot run buffer).
constexpr int kFillUnits = 1824;
constexpr int kMinRun = 128;

int32_t splits_for(int64_t units, int32_t keys) {
  const int32_t fill = (int32_t)((kFillUnits + units - 1) / units);
  const int32_t most = (keys + kMinRun - 1) / kMinRun;
  const int32_t least = (keys + kItemMax - 1) / kItemMax;
  const int32_t s = fill < most ? fill : most;
  return s > least ? s : least;
}

// Virtual KV heads, their grid groups, and the runs a request is cut into.
struct Shape {
  int32_t split, Hkv, G;
  int32_t keys, n_splits, chunk;
  Shape(int32_t batch, int32_t max_seq_len, int32_t window, int32_t sinks, int32_t Hq, int32_t Hkv_pool) {
    split = kv_split_for(Hq / Hkv_pool);
    Hkv = Hkv_pool * split;
    G = Hq / Hkv;
    const int64_t seen = (int64_t)window + sinks;
    keys = (int32_t)(seen < max_seq_len ? seen : max_seq_len);
    n_splits = splits_for((int64_t)batch * Hkv, keys);
    chunk = (keys + n_splits - 1) / n_splits;
  }
};

size_t ws_bytes(int32_t batch, const Shape& s, int32_t D, void* base, Ws* ws) {
  const size_t n = s.n_splits > 1 ? (size_t)batch * s.n_splits * s.Hkv * s.G : 0;
  const size_t o_acc = align256(sizeof(float2) * n);
  if (ws != nullptr) {
    char* b = static_cast<char*>(base);
    ws->part_ml = reinterpret_cast<float2*>(b);
    ws->part_acc = reinterpret_cast<float*>(b + o_acc);
  }
  return o_acc + sizeof(float) * n * D;
}

template <int D, int G, int LPT, typename KV, bool kSpans>
__global__ void __launch_bounds__(kThreads, (split_min_blocks<D, G, LPT, KV>())) decode_window_kernel(Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int32_t s_item[2];
  grid_dep_launch();
  // KV heads fastest: the CTAs of a run gather the heads of the same slots
  const int32_t heads = kSpans ? p.Hkv / kWarps : p.Hkv;
  const int32_t unit = (int32_t)(blockIdx.x / (unsigned)heads), y = (int32_t)(blockIdx.x % (unsigned)heads);
  bool taken = false;
  split_units<D, G, LPT, KV, 0, kSpans, true>(
      p, smem, s_item, threadIdx.x, 1, [] { __syncthreads(); },
      [&] {
        const int32_t u = taken ? 1 : 0;
        taken = true;
        return u;
      },
      [&](int32_t) { return kSpans ? kWarps * y : y; }, [&](int32_t) { return unit; });
}

template <int D, int G, int LPT, typename KV, bool kSpans>
sgl_status launch(const Params& prm, cudaStream_t stream) {
  constexpr size_t smem = SplitRing<KV, G>::template bytes<D>() + kItemMax * sizeof(int32_t);
  static_assert(kWarps * G * (D + 2) * sizeof(float) <= SplitRing<KV, G>::template bytes<D>(),
                "reduction scratch must fit in the ring");
  if (kernel_blocks_per_sm<decode_window_kernel<D, G, LPT, KV, kSpans>>((int)smem, kThreads) < 0) return SGL_ERR_CUDA;
  const int64_t heads = kSpans ? prm.Hkv / kWarps : prm.Hkv;
  const int64_t units = (int64_t)prm.batch * prm.win.n_splits * heads;
  if (units > 0x7fffffff) return SGL_ERR_UNSUPPORTED;
  decode_window_kernel<D, G, LPT, KV, kSpans><<<(unsigned)units, kThreads, smem, stream>>>(prm);
  if (prm.win.n_splits > 1) {
    const int64_t warps = (int64_t)prm.batch * prm.Hq;
    if (launch_dependent(decode_combine_kernel<D, true>, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, stream,
                         prm) != cudaSuccess)
      return SGL_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? SGL_OK : SGL_ERR_CUDA;
}

template <int D, int G, typename KV>
sgl_status run(const Params& prm, cudaStream_t stream) {
  constexpr int LPT = (D == 128 && G >= 4) ? 16 : 8;
  if constexpr (sizeof(KV) == 1) {
    if (spans_for(prm.Hkv, prm.kv_split, true)) return launch<D, G, LPT, KV, true>(prm, stream);
  }
  return launch<D, G, LPT, KV, false>(prm, stream);
}

template <int D, typename KV>
sgl_status run_g(int G, const Params& prm, cudaStream_t stream) {
  switch (G) {
    case 1: return run<D, 1, KV>(prm, stream);
    case 2: return run<D, 2, KV>(prm, stream);
    case 3: return run<D, 3, KV>(prm, stream);
    case 4: return run<D, 4, KV>(prm, stream);
    case 5: return run<D, 5, KV>(prm, stream);
    case 6: return run<D, 6, KV>(prm, stream);
    case 7: return run<D, 7, KV>(prm, stream);
    case 8: return run<D, 8, KV>(prm, stream);
    case 9: return run<D, 9, KV>(prm, stream);
    case 10: return run<D, 10, KV>(prm, stream);
    case 11: return run<D, 11, KV>(prm, stream);
    case 12: return run<D, 12, KV>(prm, stream);
    case 13: return run<D, 13, KV>(prm, stream);
    case 14: return run<D, 14, KV>(prm, stream);
    case 15: return run<D, 15, KV>(prm, stream);
    case 16: return run<D, 16, KV>(prm, stream);
    default: return SGL_ERR_UNSUPPORTED;
  }
}

}  // namespace

size_t decode_window_workspace_bytes(int32_t batch, int32_t max_seq_len, int32_t window, int32_t sinks, int32_t Hq,
                                     int32_t Hkv, int32_t D) {
  if (batch <= 0 || max_seq_len <= 0 || window <= 0 || sinks < 0 || Hkv <= 0 || Hq < Hkv) return 256;
  const Shape s(batch, max_seq_len, window, sinks, Hq, Hkv);
  return 256 + ws_bytes(batch, s, D, nullptr, nullptr);
}

sgl_status launch_decode_window(const DecodeArgs& a, cudaStream_t stream) {
  if (a.batch == 0) return SGL_OK;
  if (decode_shape_supported(a.num_q_heads, a.num_kv_heads) != SGL_OK) return SGL_ERR_UNSUPPORTED;
  const Shape s(a.batch, a.max_seq_len, a.window, a.sinks, a.num_q_heads, a.num_kv_heads);
  Params prm = {};
  if (ws_bytes(a.batch, s, a.head_dim, a.workspace, &prm.ws) > a.workspace_bytes) return SGL_ERR_WORKSPACE;
  prm.q = static_cast<const __nv_bfloat16*>(a.q);
  prm.pool_k = static_cast<const uint8_t*>(a.pool_k);
  prm.pool_v = static_cast<const uint8_t*>(a.pool_v);
  prm.req_to_token = a.req_to_token;
  prm.rtt_stride = a.rtt_stride;
  prm.req_pool_idx = a.req_pool_idx;
  prm.seq_lens = a.seq_lens;
  prm.out = static_cast<__nv_bfloat16*>(a.out);
  prm.batch = a.batch;
  prm.Hq = a.num_q_heads;
  prm.Hkv = s.Hkv;
  prm.kv_split = s.split;
  prm.Hkv_pool = a.num_kv_heads;
  prm.chunk = s.chunk;
  prm.scale_log2 = a.sm_scale * 1.4426950408889634f * (a.kv_fp8 ? a.k_scale : 1.f);
  prm.v_scale = a.kv_fp8 ? a.v_scale : 1.f;
  prm.win = Window{a.sinks, s.keys, a.max_seq_len, s.n_splits};
  if (a.head_dim == 128)
    return a.kv_fp8 ? run_g<128, uint8_t>(s.G, prm, stream) : run_g<128, __nv_bfloat16>(s.G, prm, stream);
  if (a.head_dim == 64)
    return a.kv_fp8 ? run_g<64, uint8_t>(s.G, prm, stream) : run_g<64, __nv_bfloat16>(s.G, prm, stream);
  return SGL_ERR_UNSUPPORTED;
}

}  // namespace sgl
