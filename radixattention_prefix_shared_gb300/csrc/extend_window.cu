// Launchers of the sliding-window extend: the extend pipeline (extend_dev.cuh)
// over the keys each CTA's queries see, and the combine of tiles whose keys
// were dealt to several CTAs.
//
// A query's softmax runs over positions j <= P with j < sinks or j > P -
// window; a CTA walks the union over its queries, whose ends are masked row by
// row (window_mask), so of each 4,096-key window some 4,350 key columns are
// multiplied.  Long chunks are bound by the pipeline's chain from one block's
// softmax to the next block's scores (8 chunks of 2,048 tokens, 16 query and 8
// KV heads of 128, window 4,096: 473 us, 1,160 TFLOP/s, 0.61 of the measured
// peak), e4m3 pools also by the instructions that widen the codes (64 x 256
// tokens, 32 query heads, window 2,048: 583 us, 943 TFLOP/s); short extends by
// the latency of one CTA, some 8 us with one key block.
#include "extend_dev.cuh"
#include "launch.h"

namespace sgl {

using namespace ext;

namespace {

// A call with fewer tile pairs than this part has SMs deals each pair's key
// blocks to as many CTAs as fill them (one CTA of two Q tiles an SM).
constexpr int kFillCtas = 152;
constexpr int kMaxRuns = 32;  // a lane each in the combine
// Key blocks from which dealing them out pays for the combine: a block takes a
// CTA 1.6 us, the combine 2 us and its launch as much of the host's time.
constexpr int kMinBlocks = 4;
// bf16 pools: up to this many key blocks, more CTAs than SMs hold one Q tile
// each, two on an SM, so that one's start and end overlap the other's work;
// longer lists are bound by the K/V copies, which one-tile CTAs make twice.
// 17 requests of up to 700 tokens, 4 query heads of 64 a KV head: 16.3 -> 15.5
// us with 2 blocks, 23.3 -> 19.6 with 3, 34.1 -> 35.5 with 8; 16 of 300 tokens,
// 2 heads of 128: 33.6 -> 26.9, 39.4 -> 40.0 with 3, 44.8 -> 47.9 with 4.
// Requests that never fill a second tile always take one (40 of 3 to 30
// tokens: 22.3 -> 15.4 us with 1 block, 57.1 -> 51.5 with 7).
constexpr int kOneTileBlocks = 3;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Key blocks of a pair of tiles of `tpt` tokens each: its queries' positions,
// the window before them, the sinks.
int64_t key_blocks(int32_t tpt, int32_t max_extend, int32_t max_prefix, int32_t window, int32_t sinks) {
  int64_t keys = (int64_t)window - 1 + (max_extend < 2 * tpt ? max_extend : 2 * tpt) + sinks;
  if (keys > (int64_t)max_prefix + max_extend) keys = (int64_t)max_prefix + max_extend;
  return ceil_div(keys, BN);
}

int64_t query_rows(int32_t batch, int32_t total_extend, int32_t max_extend) {
  const int64_t most = (int64_t)batch * max_extend;
  return total_extend < most ? total_extend : most;
}

struct Shape {
  bool one_tile;
  int32_t tiles;   // CTAs along x for the longest request, without runs
  int32_t n_runs;
  int64_t rows;    // tokens that can have queries (total_extend may count padding)
  Shape(int32_t batch, int32_t total_extend, int32_t max_extend, int32_t max_prefix, int32_t window, int32_t sinks,
        int32_t Hq, int32_t Hkv, bool kv_fp8) {
    const int32_t tpt = BM / (Hq / Hkv), pair = 2 * tpt;
    rows = query_rows(batch, total_extend, max_extend);
    // CTAs with queries: every request's last one may be short
    int64_t live = rows / pair + batch;
    const int64_t most = ceil_div(max_extend, pair) * batch;
    if (live > most) live = most;
    live *= Hkv;
    const int64_t blocks = key_blocks(tpt, max_extend, max_prefix, window, sinks);
    int64_t runs = live > 0 && blocks >= kMinBlocks ? kFillCtas / live : 1;
    if (runs > blocks) runs = blocks;
    if (runs > kMaxRuns) runs = kMaxRuns;
    n_runs = runs < 1 ? 1 : (int32_t)runs;
    one_tile = !kv_fp8 && n_runs == 1 && (max_extend <= tpt || (blocks <= kOneTileBlocks && live > kFillCtas));
    tiles = (int32_t)ceil_div(max_extend, one_tile ? tpt : pair);
  }
};

// status word (256 bytes), then (max, sum) and P.V row of every (token, query
// head, run)
size_t layout(int64_t entries, int32_t D, void* base, Params* prm) {
  const size_t o_ml = extend_workspace_bytes();
  const size_t o_acc = o_ml + ((size_t)entries * sizeof(float2) + 255) / 256 * 256;
  if (prm != nullptr) {
    prm->part_ml = reinterpret_cast<float2*>(static_cast<char*>(base) + o_ml);
    prm->part_acc = reinterpret_cast<float*>(static_cast<char*>(base) + o_acc);
  }
  return o_acc + (size_t)entries * D * sizeof(float);
}

// A warp a (token, query head): lane i holds run i's (max, sum); rows past
// the last request's are left alone.
template <int D>
__global__ void __launch_bounds__(128) extend_window_combine_kernel(Params p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  int64_t tokens = 0;
  for (int i = lane; i < p.batch; i += 32) tokens += p.extend_lens[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) tokens += __shfl_xor_sync(0xffffffffu, tokens, o);
  // launched dependent on the extend kernel; every warp waits, so that this
  // grid never ends (and what follows it never starts) before that one
  grid_dep_wait();
  if (row >= tokens * p.Hq || row >= p.state_rows) return;
  float2 ml = make_float2(-INFINITY, 0.f);
  if (lane < p.n_runs) ml = p.part_ml[row * p.n_runs + lane];
  float M = ml.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float w = ml.y > 0.f ? ex2(ml.x - M) : 0.f;
  float L = ml.y * w;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  const float* a = p.part_acc + row * p.n_runs * D;
#pragma unroll 8
  for (int s = 0; s < p.n_runs; ++s) {
    const float f = __shfl_sync(0xffffffffu, w, s);
    if (f != 0.f) {  // (a run without keys left its rows unwritten)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(f, a[s * D + lane + 32 * e], acc[e]);
    }
  }
  const float inv = p.o_scale / L;
  __nv_bfloat16* o = p.out + row * D;
#pragma unroll
  for (int e = 0; e < E; ++e) o[lane + 32 * e] = __float2bfloat16_rn(acc[e] * inv);
}

template <int D, bool kFp8, bool kRuns, int kTiles>
sgl_status launch(const Params& prm, const ExtendArgs& a, const Shape& s, cudaStream_t stream) {
  constexpr int kThreads = Roles<kFp8, kTiles>::kThreads;
  constexpr int kSmem = smem_bytes<D, kFp8, kTiles>();
  auto kern = extend_window_kernel<D, kFp8, kRuns, kTiles>;
  if (kernel_blocks_per_sm<extend_window_kernel<D, kFp8, kRuns, kTiles>>(kSmem, kThreads) < 0) return SGL_ERR_CUDA;
  if (Roles<kFp8, kTiles>::kSplitRegs &&
      !kernel_regs_at_least<extend_window_kernel<D, kFp8, kRuns, kTiles>>(Roles<kFp8, kTiles>::kLaunchRegs))
    return SGL_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(s.tiles * s.n_runs), (unsigned)prm.Hkv, (unsigned)a.batch);
  kern<<<grid, kThreads, kSmem, stream>>>(prm);
  if (kRuns) {
    const dim3 blocks((unsigned)ceil_div(prm.state_rows, 4));
    if (launch_dependent(extend_window_combine_kernel<D>, blocks, dim3(128), 0, stream, prm) != cudaSuccess)
      return SGL_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? SGL_OK : SGL_ERR_CUDA;
}

template <int D, bool kFp8>
sgl_status run(const Params& prm, const ExtendArgs& a, const Shape& s, cudaStream_t stream) {
  if (s.n_runs > 1) return launch<D, kFp8, true, 2>(prm, a, s, stream);
  if constexpr (!kFp8) {
    if (s.one_tile) return launch<D, kFp8, false, 1>(prm, a, s, stream);
  }
  return launch<D, kFp8, false, 2>(prm, a, s, stream);
}

}  // namespace

size_t extend_window_workspace_bytes(int32_t batch, int32_t total_extend, int32_t max_extend, int32_t max_prefix,
                                     int32_t window, int32_t sinks, int32_t Hq, int32_t Hkv, int32_t D) {
  if (batch <= 0 || total_extend <= 0 || max_extend <= 0 || max_prefix < 0 || window <= 0 || sinks < 0 || Hkv <= 0 ||
      Hq < Hkv || Hq / Hkv > BM)
    return extend_workspace_bytes();
  // A bound that grows with every argument, so that a workspace for a server's
  // largest call serves its smaller ones (fewer tiles are dealt to more CTAs
  // each): live x runs <= kFillCtas, and a pair of tiles has 2 BM rows.
  const int64_t blocks = key_blocks(BM / (Hq / Hkv), max_extend, max_prefix, window, sinks);
  if (blocks < kMinBlocks) return extend_workspace_bytes();
  int64_t entries = query_rows(batch, total_extend, max_extend) * Hq * (blocks < kMaxRuns ? blocks : kMaxRuns);
  if (entries > (int64_t)kFillCtas * 2 * BM) entries = (int64_t)kFillCtas * 2 * BM;
  return layout(entries, D, nullptr, nullptr);
}

sgl_status launch_extend_window(const ExtendArgs& a, cudaStream_t stream) {
  if (a.batch == 0 || a.total_extend == 0 || a.max_extend == 0) return SGL_OK;
  Params prm;
  const sgl_status st = make_extend_params(a, &prm);
  if (st != SGL_OK) return st;
  const Shape s(a.batch, a.total_extend, a.max_extend, a.max_prefix, a.window, a.sinks, a.num_q_heads,
                a.num_kv_heads, a.kv_fp8);
  prm.batch = a.batch;
  prm.n_runs = s.n_runs;
  prm.state_rows = s.rows * a.num_q_heads;
  if (layout(s.n_runs > 1 ? prm.state_rows * s.n_runs : 0, a.head_dim, a.workspace, &prm) > a.workspace_bytes)
    return SGL_ERR_WORKSPACE;
  if (a.head_dim == 128)
    return a.kv_fp8 ? run<128, true>(prm, a, s, stream) : run<128, false>(prm, a, s, stream);
  if (a.head_dim == 64)
    return a.kv_fp8 ? run<64, true>(prm, a, s, stream) : run<64, false>(prm, a, s, stream);
  return SGL_ERR_UNSUPPORTED;
}

}  // namespace sgl
