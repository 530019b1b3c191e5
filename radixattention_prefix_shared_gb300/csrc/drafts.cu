// The walk down each request's tree of drafted tokens, and what becomes of the
// tokens' slots (speculative decoding).
//
// sgl_verify_drafts: the walk starts at the root (node 0) with R = the root's
// target row and m = 1.  Nodes come in index order; node i is asked when its
// parent is the last accepted node c:
//     accepted iff R(x_i) > 0 and u_i q(x_i) m < R(x_i),
// q = c's draft row, or 1 where drafts were picked and not drawn.  Accepted:
// c = i, R = i's target row, m = 1.  Rejected: R <- max(R / m - q, 0), m <- sum R;
// or, without draft rows, R(x_i) <- 0, m <- m - R(x_i).  Where the walk ends the
// next token is the first v with sum_{w <= v} R(w) > u sum R.
//
// Work: a cluster of CTAs a request, the vocabulary dealt out in contiguous spans
// to the CTAs and their warps.  All weights that the walk can ask for are gathered
// at once (one dependent load after the tokens); every CTA then walks by itself
// and they meet only for sums over a row: one a second child that is asked (with
// draft rows), one at the end.  R is never stored: a pass recomputes it from the
// target and the draft row.  The CTA and the warp in whose span the drawn token
// lies read that span once more.
//
// Bound: HBM (one row, two with draft rows) for large batches, a chain of some
// six dependent loads and two cluster barriers for small ones.
//
// Sums: up to 256 values are added in fp32 (a weight's own rounding included,
// some 2^-22 of the sum), all else in fp64, whose adds this part makes at 1 / 64 of
// the fp32 rate.
#include <cooperative_groups.h>

#include "common.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace sgl {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;

struct Row {
  const float* p;  // aligned to 16 bytes, `shift` values before the row
  int shift;
};
SGL_DEV Row row_at(const float* base, int64_t stride, int64_t r) {
  const float* p = base + r * stride;
  const int shift = (int)((reinterpret_cast<uintptr_t>(p) >> 2) & 3);
  return Row{p - shift, shift};
}
// Values 4 k - shift .. + 3 of a row of V (those outside it are 0).
SGL_DEV float4 load4(const Row& r, int k, int V) {
  const int at = 4 * k - r.shift;
  if (at >= 0 && at + 3 < V) return __ldg(reinterpret_cast<const float4*>(r.p) + k);
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (at >= 0 && at < V) v.x = __ldg(r.p + 4 * k);
  if (at + 1 >= 0 && at + 1 < V) v.y = __ldg(r.p + 4 * k + 1);
  if (at + 2 >= 0 && at + 2 < V) v.z = __ldg(r.p + 4 * k + 2);
  if (at + 3 >= 0 && at + 3 < V) v.w = __ldg(r.p + 4 * k + 3);
  return v;
}
// The same values of a row that lies otherwise against 16 bytes (`shift` of the
// first row's).
SGL_DEV float4 load4_at(const float* row, int at, int V) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (at >= 0 && at < V) v.x = __ldg(row + at);
  if (at + 1 >= 0 && at + 1 < V) v.y = __ldg(row + at + 1);
  if (at + 2 >= 0 && at + 2 < V) v.z = __ldg(row + at + 2);
  if (at + 3 >= 0 && at + 3 < V) v.w = __ldg(row + at + 3);
  return v;
}

// What is not a positive finite weight counts as none.
SGL_DEV float weight(float x) { return x > 0.f && x <= 3.402823466e38f ? x : 0.f; }

struct Shared {
  int parent[kMaxDraft], token[kMaxDraft];
  float coin[kMaxDraft];
  float px[kMaxDraft], qx[kMaxDraft];  // target and draft weight of a node's token at its parent
  double mass[kMaxDraft + 1];          // m after j rejections at the node
  int gone[kMaxDraft];                 // tokens rejected there (without draft rows)
  int path[kMaxDraft];
  int at, next, rejected, accepted, asks;  // asks: the walk stands before a sum
  int part[kWarps];
  double warp_sum[kWarps];
  double cta_sum[2][kMaxCluster];  // by pass parity: the cluster's CTAs write here
};

// Four values of R at vector k of a row.
template <bool kDraft>
SGL_DEV float4 residual4(const Row& t, const Row& d, bool same, const float* drow, int k, int V, int rej, float inv1,
                         const Shared* s) {
  float4 v = load4(t, k, V);
  v = make_float4(weight(v.x), weight(v.y), weight(v.z), weight(v.w));
  if (rej == 0) return v;
  if constexpr (kDraft) {
    float4 q = same ? load4(d, k, V) : load4_at(drow, 4 * k - t.shift, V);
    q = make_float4(weight(q.x), weight(q.y), weight(q.z), weight(q.w));
    v = make_float4(fmaxf(v.x - q.x, 0.f), fmaxf(v.y - q.y, 0.f), fmaxf(v.z - q.z, 0.f), fmaxf(v.w - q.w, 0.f));
    for (int j = 1; j < rej; ++j) {
      const float inv = j == 1 ? inv1 : (float)(1.0 / s->mass[j]);
      v = make_float4(fmaxf(fmaf(v.x, inv, -q.x), 0.f), fmaxf(fmaf(v.y, inv, -q.y), 0.f),
                      fmaxf(fmaf(v.z, inv, -q.z), 0.f), fmaxf(fmaf(v.w, inv, -q.w), 0.f));
    }
  } else {
    const int at = 4 * k - t.shift;
    for (int j = 0; j < rej; ++j) {
      const int g = s->gone[j] - at;
      if (g == 0) v.x = 0.f;
      if (g == 1) v.y = 0.f;
      if (g == 2) v.z = 0.f;
      if (g == 3) v.w = 0.f;
    }
  }
  return v;
}

// One CTA of a request's cluster.  kDraft: drafts were drawn from draft_probs.
template <bool kDraft>
__global__ void __launch_bounds__(kThreads) verify_drafts_kernel(const DraftArgs a, int cluster) {
  __shared__ Shared s;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / cluster, rank = blockIdx.x % cluster;
  const int V = a.vocab;

  // where the request's nodes start
  int64_t before = 0;
  for (int i = tid; i < r; i += kThreads) before += max(0, min(__ldg(a.draft_lens + i), a.max_draft));
  int n = max(0, min(__ldg(a.draft_lens + r), a.max_draft));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  if (lane == 0) s.part[warp] = (int)min(before, (int64_t)a.total_draft);
  __syncthreads();
  int64_t off = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) off += s.part[w];
  n = (int)max((int64_t)0, min((int64_t)n, a.total_draft - off));
  if (n == 0) {  // padding
    if (rank == 0) {
      for (int k = tid; k < a.max_draft; k += kThreads) a.accepted[(int64_t)r * a.max_draft + k] = -1;
      if (tid == 0) a.num_accepted[r] = 0, a.next_tokens[r] = -1;
    }
    return;  // (the whole cluster)
  }
  cl.barrier_arrive();  // waited for before the first write into another CTA's memory
  if (tid < n) {
    const int64_t t = off + tid;
    int par = __ldg(a.parents + t);
    if (tid == 0 || par < 0 || par >= tid) par = -1;
    const int tok = __ldg(a.draft_tokens + t);
    float px = 0.f, qx = 1.f;
    if (par >= 0) {
      if (tok >= 0 && tok < V) {
        px = weight(__ldg(a.target_probs + (off + par) * a.target_stride + tok));
        if (kDraft) qx = weight(__ldg(a.draft_probs + (off + par) * a.draft_stride + tok));
      }
    }
    s.parent[tid] = par;
    s.token[tid] = tok;
    s.coin[tid] = __ldg(a.coins + t);
    s.px[tid] = px;
    s.qx[tid] = qx;
  }
  if (tid == 0) s.at = 0, s.next = 1, s.rejected = 0, s.accepted = 1, s.path[0] = 0, s.mass[0] = 1.0, s.asks = 0;
  __syncthreads();

  // a cluster-wide sum of R: pass after pass into alternating slots
  const int per = ((((V + 3 + 3) / 4 + cluster * kWarps - 1) / (cluster * kWarps)) + 31) / 32 * 32;
  int pass = 0;
  auto rows = [&](int node, Row* t, Row* d, const float** drow, bool* same) {
    *t = row_at(a.target_probs, a.target_stride, off + node);
    *d = *t;
    *drow = nullptr;
    *same = true;
    if (kDraft) {
      *drow = a.draft_probs + (off + node) * a.draft_stride;
      *d = row_at(a.draft_probs, a.draft_stride, off + node);
      *same = d->shift == t->shift;
    }
  };
  auto sum = [&](int node, int rej) {
    Row t, d;
    const float* drow;
    bool same;
    rows(node, &t, &d, &drow, &same);
    const int K = (V + t.shift + 3) / 4, k0 = (rank * kWarps + warp) * per, k1 = min(K, k0 + per);
    const float inv1 = rej > 1 ? (float)(1.0 / s.mass[1]) : 1.f;
    double total = 0.0;
    for (int kb = k0; kb < k1; kb += 8 * 32) {
      float part = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = kb + 32 * i + lane;
        if (k < k1) {
          const float4 v = residual4<kDraft>(t, d, same, drow, k, V, rej, inv1, &s);
          part += (v.x + v.y) + (v.z + v.w);
        }
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      total += (double)part;
    }
    total += __shfl_xor_sync(0xffffffffu, total, 8);
    total += __shfl_xor_sync(0xffffffffu, total, 16);
    __syncthreads();  // the last pass's warp sums have been read
    if (lane == 0) s.warp_sum[warp] = total;
    __syncthreads();
    if (pass == 0) cl.barrier_wait();
    if (tid < cluster) {
      double mine = 0.0;
      for (int w = 0; w < kWarps; ++w) mine += s.warp_sum[w];
      *cl.map_shared_rank(&s.cta_sum[pass & 1][rank], tid) = mine;
    }
    cl.sync();
    double all = 0.0;
    for (int c = 0; c < cluster; ++c) all += s.cta_sum[pass & 1][c];
    ++pass;
    return all;
  };

  // the walk; every CTA takes the same steps
  while (true) {
    if (tid == 0) {
      int at = s.at, i = s.next, rej = s.rejected, acc = s.accepted;
      bool asks = s.asks != 0;
      s.asks = 0;
      for (; i < n; ++i) {
        if (s.parent[i] != at) continue;
        if (kDraft && rej > 0 && !asks) {  // the sum of R is not known yet
          s.asks = 1;
          break;
        }
        double m = 1.0, w = s.px[i], q = s.qx[i];
        if (kDraft) {
          for (int j = 0; j < rej; ++j) w = fmax(w / s.mass[j] - q, 0.0);
          m = s.mass[rej];
        } else {
          m = s.mass[rej];
          for (int j = 0; j < rej; ++j)
            if (s.gone[j] == s.token[i]) w = 0.0;
        }
        if (w > 0.0 && (double)s.coin[i] * q * m < w) {
          at = i, rej = 0;
          s.path[acc++] = i;
        } else {
          if (!kDraft) {
            s.gone[rej] = s.token[i];
            s.mass[rej + 1] = s.mass[rej] - w;
          }
          ++rej;
        }
        asks = false;
      }
      s.at = at, s.next = i, s.rejected = rej, s.accepted = acc;
    }
    __syncthreads();
    if (!s.asks) break;
    const double m = sum(s.at, s.rejected);
    __syncthreads();
    if (tid == 0) s.mass[s.rejected] = m;
    __syncthreads();
  }

  const int at = s.at;
  int rej = s.rejected;
  double total = sum(at, rej);
  if (!(total > 0.0) && rej > 0) {  // nothing is left: draw from the row itself
    rej = 0;
    total = sum(at, 0);
  }
  if (rank == 0) {
    for (int k = tid; k < a.max_draft; k += kThreads)
      a.accepted[(int64_t)r * a.max_draft + k] = k < s.accepted ? s.path[k] : -1;
    if (tid == 0) {
      a.num_accepted[r] = s.accepted;
      if (!(total > 0.0)) a.next_tokens[r] = -1;  // a row without weights
    }
  }
  if (!(total > 0.0)) return;

  // the CTA, the warp and the values among which the sum passes u of the total; a
  // bound that rounding (or a u of 1) puts past the end is the last weight's
  const double bound = (double)__ldg(a.final_coins + r) * total;
  const double* cta = s.cta_sum[(pass - 1) & 1];
  double cum = 0.0;
  int found = -1;
  for (int c = 0; c < cluster; ++c) {
    if (cum + cta[c] > bound) {
      found = c;
      break;
    }
    cum += cta[c];
  }
  bool past = false;
  if (found < 0) {
    past = true;
    for (int c = 0; c < cluster; ++c)
      if (cta[c] > 0.0) found = c;
  }
  if (found != rank) return;
  int fw = -1;
  if (!past) {
    for (int w = 0; w < kWarps; ++w) {
      if (cum + s.warp_sum[w] > bound) {
        fw = w;
        break;
      }
      cum += s.warp_sum[w];
    }
  }
  if (fw < 0) {
    past = true;
    for (int w = 0; w < kWarps; ++w)
      if (s.warp_sum[w] > 0.0) fw = w;
  }
  if (fw != warp) return;
  Row t, d;
  const float* drow;
  bool same;
  rows(at, &t, &d, &drow, &same);
  const int K = (V + t.shift + 3) / 4, k0 = (rank * kWarps + warp) * per, k1 = min(K, k0 + per);
  const float inv1 = rej > 1 ? (float)(1.0 / s.mass[1]) : 1.f;
  int last = -1, token = -1;
  for (int kb = k0; kb < k1 && token < 0; kb += 32) {
    const int k = kb + lane;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (k < k1) v = residual4<kDraft>(t, d, same, drow, k, V, rej, inv1, &s);
    const float x[4] = {v.x, v.y, v.z, v.w};
    const double mine = ((double)x[0] + (double)x[1]) + ((double)x[2] + (double)x[3]);
    double incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    int top = -1, hit = -1;
    double c = cum + (incl - mine);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c += (double)x[j];
      if (x[j] > 0.f) {
        top = 4 * k - t.shift + j;
        if (!past && hit < 0 && c > bound) hit = top;
      }
    }
    const uint32_t hits = __ballot_sync(0xffffffffu, hit >= 0), tops = __ballot_sync(0xffffffffu, top >= 0);
    if (hits != 0) token = __shfl_sync(0xffffffffu, hit, __ffs(hits) - 1);
    if (tops != 0) last = __shfl_sync(0xffffffffu, top, 31 - __clz(tops));
    cum += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) a.next_tokens[r] = token >= 0 ? token : last;
}

// A warp a request: the accepted nodes' slots into its row of req_to_token, the
// others into the list of freed ones, in order over the batch.
__global__ void __launch_bounds__(128) commit_drafts_kernel(const CommitArgs a) {
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (r >= a.batch) return;
  // tokens and freed tokens before the request's (a warp adds up the batch: 512
  // requests are 16 loads a lane)
  int64_t off = 0, free_at = 0;
#pragma unroll 4
  for (int i = lane; i < r; i += 32) {
    const int n = max(0, min(__ldg(a.draft_lens + i), a.max_draft));
    off += n;
    free_at += n - max(0, min(__ldg(a.num_accepted + i), n));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    off += __shfl_xor_sync(0xffffffffu, off, o);
    free_at += __shfl_xor_sync(0xffffffffu, free_at, o);
  }
  const int n = max(0, min(__ldg(a.draft_lens + r), a.max_draft));
  const int count = max(0, min(__ldg(a.num_accepted + r), n));
  const int prefix = __ldg(a.prefix_lens + r);
  if (lane == 0) {
    a.seq_lens[r] = prefix + count;
    if (r == a.batch - 1) *a.num_freed = (int32_t)(free_at + n - count);
  }
  if (n == 0) return;  // padding: its row of the table is not looked at
  const int row = __ldg(a.req_pool_idx + r);
  uint32_t kept[2] = {0u, 0u};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = lane + 32 * h;
    if (k >= count) continue;
    const int node = __ldg(a.accepted + (int64_t)r * a.max_draft + k);
    if (node < 0 || node >= n || off + node >= a.total_draft) continue;
    if (node < 32) kept[0] |= 1u << node;
    else kept[1] |= 1u << (node - 32);
    const int64_t pos = (int64_t)prefix + k;
    if (row >= 0 && row < a.rtt_rows && pos >= 0 && pos < a.rtt_stride)
      a.req_to_token[(int64_t)row * a.rtt_stride + pos] = __ldg(a.slots + off + node);
  }
  kept[0] = __reduce_or_sync(0xffffffffu, kept[0]);
  kept[1] = __reduce_or_sync(0xffffffffu, kept[1]);
  const uint64_t free_nodes = ~((uint64_t)kept[1] << 32 | kept[0]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    if (i >= n || off + i >= a.total_draft || !(free_nodes >> i & 1)) continue;
    const int pos = __popcll(free_nodes & ((1ull << i) - 1));
    if (pos < n - count && free_at + pos < a.total_draft) a.freed[free_at + pos] = __ldg(a.slots + off + i);
  }
}

}  // namespace

sgl_status launch_verify_drafts(const DraftArgs& a, cudaStream_t stream) {
  // the spans of a cluster's warps hold 128 values at the least
  int cluster = kMaxCluster;
  while (cluster > 1 && a.vocab < cluster * kWarps * 128) cluster /= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.batch * (unsigned)cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = a.draft_probs != nullptr ? cudaLaunchKernelEx(&cfg, verify_drafts_kernel<true>, a, cluster)
                                                 : cudaLaunchKernelEx(&cfg, verify_drafts_kernel<false>, a, cluster);
  return e == cudaSuccess ? SGL_OK : SGL_ERR_CUDA;
}

sgl_status launch_commit_drafts(const CommitArgs& a, cudaStream_t stream) {
  commit_drafts_kernel<<<(unsigned)((a.batch + 3) / 4), 128, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? SGL_OK : SGL_ERR_CUDA;
}

}  // namespace sgl
