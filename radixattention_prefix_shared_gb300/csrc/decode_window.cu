// Launchers of the sliding-window decode: the split kernel's work loop
// (decode_dev.cuh) over each request's visible keys, one run of them a CTA,
// and the combine of requests with more than one run.
//
// A request's visible keys number at most sinks + window whatever its length,
// so the host knows every CTA's share from its own arguments: no plan kernel
// and no work counters, one launch where a run holds a whole request.
//
// Bound by HBM where there is work for every SM: 248 requests, 16 query and 8 KV
// heads of 128, window 4,096: 509 us, 6.78 TB/s, the measured copy rate; 64
// requests of 32 e4m3 KV heads, window 1,024: 91 us, 5.5 TB/s (0.81), bound by
// the conversions of the codes.  Small calls are bound by latency: one request
// of window 4,096 takes 11.9 us (three dependent loads, 8 stages a run, the
// combine) for 16.8 MB.
#include "decode_dev.cuh"
#include "launch.h"

namespace sgl {

using namespace dec;

namespace {

// Runs are made as short as it takes to give the part kFillUnits CTAs (four
// waves: the runs' lengths vary and a CTA lasts as long as its run), but no
// shorter than kMinRun keys and no longer than kItemMax (the slot run buffer).
// Measured: 64 requests of 32 KV heads over an e4m3 pool, window 1,024: 102 us
// at 456 CTAs, 96.9 at 912, 93.2 at 1,824; 93.2 us with runs of 256 keys, 95.1
// with 512; one request of 8 KV heads, window 4,096: 12.6 us with runs of 256
// keys or 128, 16.3 with 512.  Runs merged by clusters of up to 8 CTAs
// through distributed shared memory took as long as the combine (12.6 us).
constexpr int kFillUnits = 1824;
constexpr int kMinRun = 256;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int32_t most_runs(int32_t keys) { return (int32_t)ceil_div(keys, kMinRun); }
int32_t least_runs(int32_t keys) { return (int32_t)ceil_div(keys, kItemMax); }

// Rows of at most 128 bytes (an e4m3 pool's, and bf16 ones of 64 elements)
// are gathered in spans of kWarps KV heads, a CTA a run of all of them, where
// that leaves kSpanUnits CTAs of the shortest runs: a span is read at a higher
// rate than as many rows, but with few CTAs a quarter of them is what counts.
// Spans and rows: one request of 8 query and 8 e4m3 KV heads of 128, window
// 4,096 (32 CTAs): 17.5 us, 8.8; 16 x 1,000 (128): 18.2, 13.0; 96 x 511
// (384): 26.2, 28.7; 32 x 2,048 (512): 30.2, 35.5; 200 x 4,096: 269, 285.
// bf16 of 64, 16 query and 8 KV heads: 21.2, 9.7; 22.0, 13.0; 27.8, 28.1; 29.8,
// 33.3; 276, 286; 96 requests of 4 KV heads, 511 (192): 18.7, 11.1; 64 query
// heads on 8: 128 x 100 (256): 11.8, 14.7.
constexpr int kSpanUnits = 256;
constexpr bool short_rows(int32_t D, bool kv_fp8) { return kv_fp8 || D == 64; }

// Virtual KV heads, whether their rows are gathered in spans, and the runs a
// request is cut into.
struct Shape {
  int32_t split, Hkv, G;
  bool spans;
  int32_t keys, n_splits, chunk;
  Shape(int32_t batch, int32_t max_seq_len, int32_t window, int32_t sinks, int32_t Hq, int32_t Hkv_pool,
        int32_t D, bool kv_fp8) {
    split = kv_split_for(Hq / Hkv_pool);
    Hkv = Hkv_pool * split;
    G = Hq / Hkv;
    const int64_t seen = (int64_t)window + sinks;
    keys = (int32_t)(seen < max_seq_len ? seen : max_seq_len);
    spans = short_rows(D, kv_fp8) && spans_possible(Hkv, split) &&
            (int64_t)batch * (Hkv / kWarps) * most_runs(keys) >= kSpanUnits;
    const int64_t fill = ceil_div(kFillUnits, (int64_t)batch * (spans ? Hkv / kWarps : Hkv));
    n_splits = fill < most_runs(keys) ? (int32_t)fill : most_runs(keys);
    if (n_splits < least_runs(keys)) n_splits = least_runs(keys);
    chunk = (int32_t)ceil_div(keys, n_splits);
  }
};

// Bytes in front of the states that a decode leaves as they are: a workspace
// may serve the window's extend too, whose wait status is its first word.
constexpr size_t kStatusBytes = 256;

// (max, sum) and P.V row of every (request, run, query head), behind them
size_t ws_bytes(int64_t entries, int32_t D, void* base, Ws* ws) {
  const size_t o_acc = kStatusBytes + align256(sizeof(float2) * (size_t)entries);
  if (ws != nullptr) {
    char* b = static_cast<char*>(base);
    ws->part_ml = reinterpret_cast<float2*>(b + kStatusBytes);
    ws->part_acc = reinterpret_cast<float*>(b + o_acc);
  }
  return o_acc + sizeof(float) * (size_t)entries * D;
}

// Ring stages: the split kernel's, but four on the CUDA-core path over an e4m3
// pool, whose conversions want the fifth CTA on an SM more than the deeper
// ring (64 requests of 32 KV heads, window 1,024: 95.0 us with 6 stages, 94.2
// with 5, 90.4 with 4, 93.5 with 3).
template <int G, typename KV>
constexpr int ring_depth() {
  return !use_mma<KV, G>() && sizeof(KV) == 1 ? 4 : SplitRing<KV, G>::kDepth;
}
template <int D, int G, typename KV>
constexpr size_t ring_bytes() {
  return SplitRing<KV, G>::template bytes<D>() / SplitRing<KV, G>::kDepth * ring_depth<G, KV>();
}

template <int D, int G, int LPT, typename KV, bool kSpans>
__global__ void __launch_bounds__(kThreads, (split_min_blocks<D, G, LPT, KV>())) decode_window_kernel(Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int32_t s_item[2];
  grid_dep_launch();
  // KV heads fastest: the CTAs next to each other gather the heads of the same
  // slots
  const uint32_t heads = kSpans ? p.Hkv / kWarps : p.Hkv;
  const int32_t item = (int32_t)(blockIdx.x / heads), y = (int32_t)(blockIdx.x % heads);
  bool taken = false;
  split_units<D, G, LPT, KV, ring_depth<G, KV>(), kSpans, true>(
      p, smem, s_item, threadIdx.x, 1, [] { __syncthreads(); },
      [&] {
        const int32_t u = taken ? 1 : 0;
        taken = true;
        return u;
      },
      [&](int32_t) { return kSpans ? kWarps * y : y; }, [&](int32_t) { return item; });
}

// Merges the states of requests with more than one run: a block a (request,
// query head), its warps taking the runs in turn, four loads of each in flight
// (one warp reading 33 runs one after the other took 14 us, longer than the
// split kernel).
template <int D>
__global__ void __launch_bounds__(128) window_combine_kernel(Params p) {
  constexpr int E = D / 32, kBatch = 4;
  __shared__ float s_m[4], s_l[4];
  __shared__ float s_acc[4][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq;
  const int32_t ns = WindowRun(p.win, p.chunk, p.seq_lens[r]).ns;
  // launched dependent on the split kernel; every block waits, so that this
  // grid never ends (and what follows it never starts) before that one
  grid_dep_wait();
  if (ns <= 1) return;  // a single run wrote the output (none: no keys)
  const int64_t first = (int64_t)r * p.win.n_splits * p.Hq + h, step = p.Hq;
  float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int32_t s0 = warp; s0 < ns; s0 += 4 * kBatch) {
    float2 ml[kBatch];
    float a[kBatch][E];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t slot = first + (int64_t)min(s0 + 4 * u, ns - 1) * step;
      ml[u] = p.ws.part_ml[slot];
#pragma unroll
      for (int e = 0; e < E; ++e) a[u][e] = p.ws.part_acc[slot * D + lane + 32 * e];
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (s0 + 4 * u >= ns) break;
      const float m = fmaxf(M, ml[u].x);
      const float f = ex2(M - m), w = ex2(ml[u].x - m);
      M = m;
      L = L * f + ml[u].y * w;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + a[u][e] * w;
    }
  }
  if (lane == 0) s_m[warp] = M, s_l[warp] = L;
#pragma unroll
  for (int e = 0; e < E; ++e) s_acc[warp][lane + 32 * e] = acc[e];
  __syncthreads();
  M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  float f[4];
  L = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = ex2(s_m[w] - M);  // 0 for a warp without a run (-inf)
    L += s_l[w] * f[w];
  }
  const int d = threadIdx.x;
  if (d < D) {
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) o += s_acc[w][d] * f[w];
    p.out[((int64_t)r * p.Hq + h) * D + d] = __float2bfloat16_rn(o * (p.v_scale / L));
  }
}

template <int D, int G, int LPT, typename KV, bool kSpans>
sgl_status launch(const Params& prm, cudaStream_t stream) {
  constexpr size_t smem = ring_bytes<D, G, KV>() + kItemMax * sizeof(int32_t);
  static_assert(kWarps * G * (D + 2) * sizeof(float) <= ring_bytes<D, G, KV>(),
                "reduction scratch must fit in the ring");
  if (kernel_blocks_per_sm<decode_window_kernel<D, G, LPT, KV, kSpans>>((int)smem, kThreads) < 0) return SGL_ERR_CUDA;
  const int64_t heads = kSpans ? prm.Hkv / kWarps : prm.Hkv;
  const int64_t ctas = (int64_t)prm.batch * prm.win.n_splits * heads;
  const int64_t rows = (int64_t)prm.batch * prm.Hq;
  if (ctas > 0x7fffffff || rows > 0x7fffffff) return SGL_ERR_UNSUPPORTED;
  decode_window_kernel<D, G, LPT, KV, kSpans><<<(unsigned)ctas, kThreads, smem, stream>>>(prm);
  if (prm.win.n_splits > 1) {
    if (launch_dependent(window_combine_kernel<D>, dim3((unsigned)rows), dim3(128), 0, stream, prm) != cudaSuccess)
      return SGL_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? SGL_OK : SGL_ERR_CUDA;
}

template <int D, int G, typename KV>
sgl_status run(const Params& prm, bool spans, cudaStream_t stream) {
  constexpr int LPT = (D == 128 && G >= 4) ? 16 : 8;
  if constexpr (short_rows(D, sizeof(KV) == 1)) {
    if (spans) return launch<D, G, LPT, KV, true>(prm, stream);
  }
  return launch<D, G, LPT, KV, false>(prm, stream);
}

template <int D, typename KV>
sgl_status run_g(int G, const Params& prm, bool spans, cudaStream_t stream) {
  switch (G) {
    case 1: return run<D, 1, KV>(prm, spans, stream);
    case 2: return run<D, 2, KV>(prm, spans, stream);
    case 3: return run<D, 3, KV>(prm, spans, stream);
    case 4: return run<D, 4, KV>(prm, spans, stream);
    case 5: return run<D, 5, KV>(prm, spans, stream);
    case 6: return run<D, 6, KV>(prm, spans, stream);
    case 7: return run<D, 7, KV>(prm, spans, stream);
    case 8: return run<D, 8, KV>(prm, spans, stream);
    case 9: return run<D, 9, KV>(prm, spans, stream);
    case 10: return run<D, 10, KV>(prm, spans, stream);
    case 11: return run<D, 11, KV>(prm, spans, stream);
    case 12: return run<D, 12, KV>(prm, spans, stream);
    case 13: return run<D, 13, KV>(prm, spans, stream);
    case 14: return run<D, 14, KV>(prm, spans, stream);
    case 15: return run<D, 15, KV>(prm, spans, stream);
    case 16: return run<D, 16, KV>(prm, spans, stream);
    default: return SGL_ERR_UNSUPPORTED;
  }
}

}  // namespace

size_t decode_window_workspace_bytes(int32_t batch, int32_t max_seq_len, int32_t window, int32_t sinks, int32_t Hq,
                                     int32_t Hkv, int32_t D) {
  if (batch <= 0 || max_seq_len <= 0 || window <= 0 || sinks < 0 || Hkv <= 0 || Hq < Hkv) return kStatusBytes;
  // A bound that grows with every argument, so that a workspace for a server's
  // largest call serves its smaller ones: fewer requests are cut into more runs
  // each, and batch x runs is at most the larger of the runs that kItemMax
  // asks for and of kFillUnits CTAs' over the call's head groups (those of
  // the gather in spans, which takes fewer) plus one a request, and never past runs of
  // kMinRun keys.
  const int64_t seen = (int64_t)window + sinks;
  const int32_t keys = (int32_t)(seen < max_seq_len ? seen : max_seq_len);
  if (most_runs(keys) <= 1) return kStatusBytes;
  const int32_t split = kv_split_for(Hq / Hkv), heads = Hkv * split;
  const int64_t fill = ceil_div(kFillUnits, spans_possible(heads, split) ? heads / kWarps : heads) + batch;
  int64_t runs = (int64_t)batch * least_runs(keys);
  if (runs < fill) runs = fill;
  if (runs > (int64_t)batch * most_runs(keys)) runs = (int64_t)batch * most_runs(keys);
  return ws_bytes(runs * Hq, D, nullptr, nullptr);
}

sgl_status launch_decode_window(const DecodeArgs& a, cudaStream_t stream) {
  if (a.batch == 0) return SGL_OK;
  if (decode_shape_supported(a.num_q_heads, a.num_kv_heads) != SGL_OK) return SGL_ERR_UNSUPPORTED;
  const Shape s(a.batch, a.max_seq_len, a.window, a.sinks, a.num_q_heads, a.num_kv_heads, a.head_dim,
                a.kv_fp8);
  Params prm = {};
  const int64_t entries = s.n_splits > 1 ? (int64_t)a.batch * s.n_splits * a.num_q_heads : 0;
  if (ws_bytes(entries, a.head_dim, a.workspace, &prm.ws) > a.workspace_bytes) return SGL_ERR_WORKSPACE;
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
  // (positions past the rows of req_to_token are left out as well)
  const int32_t max_seq = a.max_seq_len < a.rtt_stride ? a.max_seq_len : a.rtt_stride;
  prm.win = Window{a.sinks, a.window, max_seq, s.n_splits};
  if (a.head_dim == 128)
    return a.kv_fp8 ? run_g<128, uint8_t>(s.G, prm, s.spans, stream)
                    : run_g<128, __nv_bfloat16>(s.G, prm, s.spans, stream);
  if (a.head_dim == 64)
    return a.kv_fp8 ? run_g<64, uint8_t>(s.G, prm, s.spans, stream)
                    : run_g<64, __nv_bfloat16>(s.G, prm, s.spans, stream);
  return SGL_ERR_UNSUPPORTED;
}

}  // namespace sgl
