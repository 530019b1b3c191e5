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
// at once (one dependent load after the tokens); each CTA's first warp then walks,
// nodes in its lanes, and the cluster meets only for sums over a row: one a second
// child that is asked (with draft rows), one at the end.  R is never stored: a pass
// recomputes it from the target and the draft row.  The warp in whose span the
// drawn token lies reads that span once more.
//
// Bound: by latency everywhere measured (2 to 3 CTAs an SM).  One chain of 5 over
// 32,000 tokens 9.0 us: five dependent loads, the scans, two cluster barriers; 64
// chains of 6 over 131,072 tokens 29.9 us, 2.2 TB/s of the 67 MB that the rows hold; 200
// trees of up to 8 picked drafts 47.5 us, 2.2 TB/s; 24 trees of up to 24 drawn drafts over
// 50,257 tokens 35 us, some five sums after one another.
//
// Sums: most of a vocabulary's weights are some 1e-8 of the sum, so an error of that
// size moves the drawn token; but this part makes fp64 sums at 1 / 64 of the fp32
// rate.  Values of R and their sums are held as two fp32 numbers (the second what
// the first has lost), some 45 bits, up to a warp's sum, and in fp64 from there on, in
// one warp of a CTA (all eight of them: 20 us of 82, 64 chains over 131,072 tokens).
#include <cooperative_groups.h>

#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace sgl {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;
// 16-byte vectors of a row that a lane holds at a time.  8: the unrolled arithmetic
// with draft rows outgrows the instruction cache (64 chains over 131,072 tokens 75 us
// against 45), without them the registers (one chain over 32,000 11.3 us against 8.9).
constexpr int kVecs = 4;
// CTAs an SM that the registers are cut for
template <bool kDraft>
constexpr int ctas_per_sm() { return kDraft ? 2 : 3; }
constexpr int kParts = 8;  // of a warp's span, whose sums are kept for the draw

// A row as 16-byte vectors: vector k is values 4 k - shift .. + 3.
struct Row {
  const float* p;
  int shift;
};
SGL_DEV Row row_at(const float* base, int64_t stride, int64_t r) {
  const float* p = base + r * stride;
  const int shift = (int)((reinterpret_cast<uintptr_t>(p) >> 2) & 3);
  return Row{p - shift, shift};
}
// Values at .. at + 3 of a row, one by one; 0 outside it.
__device__ __noinline__ float4 load_each(const float* row, int at, int V) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (at >= 0 && at < V) v.x = __ldg(row + at);
  if (at + 1 >= 0 && at + 1 < V) v.y = __ldg(row + at + 1);
  if (at + 2 >= 0 && at + 2 < V) v.z = __ldg(row + at + 2);
  if (at + 3 >= 0 && at + 3 < V) v.w = __ldg(row + at + 3);
  return v;
}

// What is not a positive finite weight counts as none.
SGL_DEV float weight(float x) {
  x = fmaxf(x, 0.f);  // NaN, too
  return x <= 3.402823466e38f ? x : 0.f;
}

// h + l, l what h has lost: Knuth's two-sum, whose error term is exact.  (No contraction or
// reordering.)
struct Pair {
  float h = 0.f, l = 0.f;
  SGL_DEV void add(float h2, float l2) {
    const float s = __fadd_rn(h, h2), b = __fsub_rn(s, h);
    const float e = __fadd_rn(__fsub_rn(h, __fsub_rn(s, b)), __fsub_rn(h2, b));
    h = s, l = __fadd_rn(l, __fadd_rn(e, l2));
  }
  SGL_DEV void tidy() {  // |l| below a step of h again
    const float s = __fadd_rn(h, l);
    l = __fsub_rn(l, __fsub_rn(s, h)), h = s;
  }
  SGL_DEV double value() const { return (double)h + (double)l; }
};
// Two such sums side by side, in packed arithmetic (a - b as a + (-1) b: exact).
struct Pair2 {
  float2 h = make_float2(0.f, 0.f), l = make_float2(0.f, 0.f);
  SGL_DEV void add(float2 x, float2 y) {
    const float2 minus = make_float2(-1.f, -1.f);
    const float2 s = fadd2(h, x), b = ffma2(h, minus, s);
    const float2 e = fadd2(ffma2(ffma2(b, minus, s), minus, h), ffma2(b, minus, x));
    h = s, l = fadd2(l, fadd2(e, y));
  }
};
SGL_DEV Pair warp_total(Pair p) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    p.tidy();
    p.add(__shfl_xor_sync(0xffffffffu, p.h, o), __shfl_xor_sync(0xffffffffu, p.l, o));
  }
  return p;
}

SGL_DEV int pick(const int (&x)[2], int i) {
  const int a = __shfl_sync(0xffffffffu, x[0], i & 31), b = __shfl_sync(0xffffffffu, x[1], i & 31);
  return i < 32 ? a : b;
}
SGL_DEV float pick(const float (&x)[2], int i) {
  const float a = __shfl_sync(0xffffffffu, x[0], i & 31), b = __shfl_sync(0xffffffffu, x[1], i & 31);
  return i < 32 ? a : b;
}
SGL_DEV double pick(const double (&x)[2], int i) {
  const double a = __shfl_sync(0xffffffffu, x[0], i & 31), b = __shfl_sync(0xffffffffu, x[1], i & 31);
  return i < 32 ? a : b;
}
// Bit i: node i (lane i % 32's) has it.
SGL_DEV uint64_t nodes(bool lo, bool hi) {
  return (uint64_t)__ballot_sync(0xffffffffu, hi) << 32 | __ballot_sync(0xffffffffu, lo);
}

struct Shared {
  // what the warps go by in a pass: the node, its rejections, which nodes those were
  int at, rej, more;  // more: another pass follows this one
  uint64_t gone;
  int token[kMaxDraft];
  float inv_h[kMaxDraft], inv_l[kMaxDraft];  // 1 / m after j rejections, j >= 1
  double warp_sum[kWarps];
  float2 part_sum[kWarps][kParts];  // the latest pass's, part by part of a span (a Pair each: a
                                    // conversion to fp64 in the loop costs as much as its loads)
  double cta_sum[2][kMaxCluster];  // by pass parity: the cluster's CTAs write here
  // where the drawn token lies: the warp (below 0: not in this CTA), what lies before
  int found, past;
  double cum, bound;
};

// Of `count` sums in the first lanes: the first whose inclusive sum from `cum` on
// passes the bound (cum becomes what lies before it), else (past) the last one
// above 0.
SGL_DEV int find(double x, int count, double* cum, double bound, bool* past) {
  const int lane = threadIdx.x & 31;
  double incl = lane < count ? x : 0.0;
#pragma unroll
  for (int o = 1; o < kMaxCluster; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  const uint32_t some = __ballot_sync(0xffffffffu, lane < count && x > 0.0);
  const uint32_t hits = *past ? 0u : __ballot_sync(0xffffffffu, lane < count && x > 0.0 && *cum + incl > bound);
  if (hits == 0) *past = true;
  const int at = hits != 0 ? __ffs(hits) - 1 : 31 - __clz(some);
  *cum += __shfl_sync(0xffffffffu, incl - x, at & 31);
  return at;
}
static_assert(kWarps <= kMaxCluster && kParts <= kMaxCluster, "find() scans that many");

// One CTA of a request's cluster.  kDraft: drafts were drawn from draft_probs.
template <bool kDraft>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<kDraft>()) verify_drafts_kernel(const DraftArgs a, int cluster) {
  __shared__ Shared s;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / cluster, rank = blockIdx.x % cluster;
  const int V = a.vocab;

  // where the request's nodes start
  int64_t off = 0;
#pragma unroll 4
  for (int i = lane; i < r; i += 32) off += max(0, min(__ldg(a.draft_lens + i), a.max_draft));
  int n = max(0, min(__ldg(a.draft_lens + r), a.max_draft));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) off += __shfl_xor_sync(0xffffffffu, off, o);
  n = (int)max((int64_t)0, min((int64_t)n, a.total_draft - off));
  const bool first = rank == 0 && warp == 0;
  int32_t* path = a.accepted + (int64_t)r * a.max_draft;
  if (n == 0) {  // padding
    if (first) {
      for (int k = lane; k < a.max_draft; k += 32) path[k] = -1;
      if (lane == 0) a.num_accepted[r] = 0, a.next_tokens[r] = -1;
    }
    return;  // (the whole cluster)
  }
  cl.barrier_arrive();  // waited for before the first write into another CTA's memory

  // the first warp: nodes lane and lane + 32, their parent, token, coin, weights of
  // the token at the parent
  int parent[2], token[2];
  float coin[2], px[2], qx[2], final_coin = 0.f;
  uint64_t keep_first = 0;
  if (warp == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = lane + 32 * h;
      parent[h] = -1, token[h] = -1, coin[h] = 0.f, px[h] = 0.f, qx[h] = 1.f;
      if (i > 0 && i < n) {
        const int par = __ldg(a.parents + off + i);
        token[h] = __ldg(a.draft_tokens + off + i);
        coin[h] = __ldg(a.coins + off + i);
        if (par >= 0 && par < i) {
          parent[h] = par;
          if (token[h] >= 0 && token[h] < V) {
            px[h] = weight(__ldg(a.target_probs + (off + par) * a.target_stride + token[h]));
            if (kDraft) qx[h] = weight(__ldg(a.draft_probs + (off + par) * a.draft_stride + token[h]));
          }
        }
      }
      s.token[i] = token[h];
    }
    // kept if asked before any sibling (R is the target row, m is 1)
    keep_first = nodes(px[0] > 0.f && (double)coin[0] * (double)qx[0] < (double)px[0],
                       px[1] > 0.f && (double)coin[1] * (double)qx[1] < (double)px[1]);
    __syncwarp();
    final_coin = __ldg(a.final_coins + r);
  }
  double mass[2] = {1.0, 1.0};  // lane j % 32's: m after j rejections at the node (j >= 1, with draft rows)
  double m = 1.0;               // after the latest
  int at = 0, rej = 0, kept = 1, next = 0;
  uint64_t gone = 0;  // nodes rejected there
  if (first && lane == 0) path[0] = 0;

  // The walk, from node `next` on, as far as it goes without a sum: true where it
  // stands before one (`next` the child that asks), false at its end.  summed: that
  // sum is m.
  auto walk = [&](bool summed) {
    for (;;) {
      if (!summed) {
        const uint64_t open = nodes(parent[0] == at, parent[1] == at) & ~((2ull << next) - 1);  // c's children behind
        if (open == 0) return false;
        next = __ffsll(open) - 1;
        if (kDraft && rej > 0) return true;
      }
      summed = false;
      const int i = next;
      bool keep = keep_first >> i & 1;
      double w = 0.0;
      if (kDraft) {
        if (rej > 0) {
          const double q = pick(qx, i);
          w = pick(px, i);
          for (int j = 0; j < rej; ++j) w = fmax((j == 0 ? w : w / pick(mass, j)) - q, 0.0);
          keep = w > 0.0 && (double)pick(coin, i) * q * m < w;
        }
      } else if (rej > 0 || !keep) {
        const int x = pick(token, i);
        if ((nodes(token[0] == x, token[1] == x) & gone) == 0) w = pick(px, i);
        keep = w > 0.0 && (double)pick(coin, i) * m < w;
      }
      if (keep) {
        if (first && lane == 0) path[kept] = i;
        at = i, ++kept, rej = 0, gone = 0, m = 1.0;
      } else {
        ++rej, gone |= 1ull << i;
        if (!kDraft) m -= w;
      }
    }
  };

  // spans: vectors of a row, `vecs` a lane at a time
  const int vecs = min(kVecs, max(1, ((V + 6) / 4 + 32 * kWarps * cluster - 1) / (32 * kWarps * cluster)));
  const int step = 32 * vecs, chunks = ((V + 6) / 4 + step - 1) / step;
  const int per = (chunks + kWarps * cluster - 1) / (kWarps * cluster) * step;
  const int k_begin = (rank * kWarps + warp) * per;
  const int part_vecs = (per / step + kParts - 1) / kParts * step;  // vectors of a part
  // R of node `at` after `rej` rejections (every warp's, by now): take(i, h, l) with
  // the values of the lane's vector kb + 32 i + lane, i < count <= kN
  auto residual = [&](auto most, int kb, int count, auto&& take) {
    constexpr int kN = decltype(most)::value;
    const Row t = row_at(a.target_probs, a.target_stride, off + at);
    const int K = (V + t.shift + 3) / 4;
    auto load = [&](const Row& row, float4 (&x)[kN]) {  // lies against 16 bytes as t does, or value by value
      const bool same = row.shift == t.shift;
      bool full[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int k = kb + 32 * i + lane;
        full[i] = same && i < count && 4 * k >= t.shift && 4 * k - t.shift + 3 < V;
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (full[i]) x[i] = __ldg(reinterpret_cast<const float4*>(row.p) + k);
      }
#pragma unroll
      for (int i = 0; i < kN; ++i) {  // a row's ends
        const int k = kb + 32 * i + lane;
        if (i < count && k < K && !full[i]) x[i] = load_each(row.p + row.shift, 4 * k - t.shift, V);
      }
    };
    float4 v[kN];
    if constexpr (kDraft) {
      float4 q[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) q[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      load(t, v);
      if (rej > 0) load(row_at(a.draft_probs, a.draft_stride, off + at), q);
      // the first rejection's difference is exact; each further one multiplies by
      // 1 / m, two numbers too, and takes q off
      auto value = [&](float x, float y) {
        x = weight(x), y = weight(y);
        Pair r;
        if (x > y) r.h = __fsub_rn(x, y), r.l = __fsub_rn(__fsub_rn(x, r.h), y);
#pragma unroll 1
        for (int j = 1; j < rej; ++j) {
          const float ih = s.inv_h[j], il = s.inv_l[j];
          const float ph = __fmul_rn(r.h, ih);
          const float pl = __fmaf_rn(r.l, ih, __fmaf_rn(r.h, il, __fmaf_rn(r.h, ih, -ph)));
          r.h = ph, r.l = 0.f;
          r.add(-y, pl);
          r.tidy();
          if (!(r.h > 0.f)) r.h = r.l = 0.f;
        }
        return r;
      };
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const Pair a0 = value(v[i].x, q[i].x), a1 = value(v[i].y, q[i].y), a2 = value(v[i].z, q[i].z),
                   a3 = value(v[i].w, q[i].w);
        take(i, make_float4(a0.h, a1.h, a2.h, a3.h), make_float4(a0.l, a1.l, a2.l, a3.l));
      }
    } else {
      load(t, v);
#pragma unroll 1
      for (uint64_t left = gone; left != 0; left &= left - 1) {
        const int g = s.token[__ffsll(left) - 1];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const int e = g - (4 * (kb + 32 * i + lane) - t.shift);
          if (e == 0) v[i].x = 0.f;
          if (e == 1) v[i].y = 0.f;
          if (e == 2) v[i].z = 0.f;
          if (e == 3) v[i].w = 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        take(i, make_float4(weight(v[i].x), weight(v[i].y), weight(v[i].z), weight(v[i].w)),
             make_float4(0.f, 0.f, 0.f, 0.f));
      }
    }
  };
  const std::integral_constant<int, kVecs> all_vecs;
  const std::integral_constant<int, 1> one_vec;
  auto end_of = [&]() { return min(k_begin + per, (V + row_at(a.target_probs, a.target_stride, off + at).shift + 3) / 4); };

  // Passes over the vocabulary: the sum of R, for the walk or for the draw.
  double total = 0.0;
  bool drawing = false, again = false;
  for (int pass = 0;; ++pass) {
    if (warp == 0) {
      if (!again) drawing = !walk(pass > 0);
      if (lane == 0) s.at = at, s.rej = rej, s.gone = gone, s.more = !drawing;
    }
    __syncthreads();
    at = s.at, rej = s.rej, gone = s.gone;
    const bool more = s.more;
    const int k_end = end_of();
    Pair mine, span;
    for (int kb = k_begin, j = 0; kb < k_end; kb += step) {
      Pair2 part[2];
      residual(all_vecs, kb, vecs, [&](int, const float4& h, const float4& l) {
        part[0].add(make_float2(h.x, h.y), make_float2(l.x, l.y));
        part[1].add(make_float2(h.z, h.w), make_float2(l.z, l.w));
      });
      part[0].add(part[1].h, part[1].l);
      mine.add(part[0].h.x, part[0].l.x);
      mine.add(part[0].h.y, part[0].l.y);
      if ((kb - k_begin + step) % part_vecs == 0 || kb + step >= k_end) {
        const Pair sum = warp_total(mine);
        if (lane == 0) s.part_sum[warp][j] = make_float2(sum.h, sum.l);
        span.tidy(), span.add(sum.h, sum.l);
        ++j, mine = Pair();
      }
    }
    if (lane == 0) s.warp_sum[warp] = span.value();
    __syncthreads();
    if (pass == 0) cl.barrier_wait();
    if (warp == 0) {
      double sum = lane < kWarps ? s.warp_sum[lane] : 0.0;
#pragma unroll
      for (int o = 1; o < kWarps; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane < cluster) *cl.map_shared_rank(&s.cta_sum[pass & 1][rank], lane) = sum;
    }
    cl.sync();
    if (warp == 0) {
      // (in every CTA the same lanes add the same sums)
      const double x = lane < cluster ? s.cta_sum[pass & 1][lane] : 0.0;
      double sum = x;
#pragma unroll
      for (int o = 1; o < kMaxCluster; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      total = __shfl_sync(0xffffffffu, sum, 0);
      again = false;
      if (more) {
        m = total;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (lane + 32 * h == rej) {
            const double inv = m > 0.0 ? 1.0 / m : 0.0;  // (m of 0: nothing is left of R)
            mass[h] = m, s.inv_h[rej] = (float)inv, s.inv_l[rej] = (float)(inv - (double)(float)inv);
          }
      } else if (!(total > 0.0) && rej > 0) {  // nothing is left: draw from the row itself
        again = true, rej = 0, gone = 0;
      } else {
        // where the sum passes u of the total; a bound that rounding (or a u of 1)
        // puts past the end is the last weight's
        int where = -1;
        double cum = 0.0;
        const double bound = (double)final_coin * total;
        bool past = false;
        if (total > 0.0 && find(x, cluster, &cum, bound, &past) == rank)
          where = find(lane < kWarps ? s.warp_sum[lane] : 0.0, kWarps, &cum, bound, &past);
        if (lane == 0) s.found = where, s.cum = cum, s.past = past, s.bound = bound;
      }
      if (lane == 0) s.more = more || again;
      __syncwarp();
    }
    __syncthreads();
    if (!s.more) break;
    __syncthreads();  // all have read it
  }
  if (first) {
    for (int k = kept + lane; k < a.max_draft; k += 32) path[k] = -1;
    if (lane == 0) {
      a.num_accepted[r] = kept;
      if (!(total > 0.0)) a.next_tokens[r] = -1;  // a row without weights
    }
  }
  if (warp != s.found) return;

  // the span's vectors among which the sum passes the bound, or (past, or by a
  // rounding apart) its last ones above 0; then the value among those
  bool past = s.past != 0;
  const double bound = s.bound;
  double cum = s.cum, before = cum;
  const int shift = row_at(a.target_probs, a.target_stride, off + at).shift, k_end = end_of();
  int k_hit = -1;
  bool found = false;
  const int parts = (k_end - k_begin + part_vecs - 1) / part_vecs;
  const float2 mine = lane < parts ? s.part_sum[warp][lane] : make_float2(0.f, 0.f);
  const int k_from = k_begin + find((double)mine.x + (double)mine.y, parts, &cum, bound, &past) * part_vecs;
  for (int kb = k_from; kb < min(k_end, k_from + part_vecs) && !found; kb += step) {
    Pair part[kVecs];
    residual(all_vecs, kb, vecs, [&](int i, const float4& h, const float4& l) {
      part[i].add(h.x, l.x), part[i].add(h.y, l.y), part[i].add(h.z, l.z), part[i].add(h.w, l.w);
    });
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const double sum = warp_total(part[i]).value();
      if (!found && sum > 0.0) {
        k_hit = kb + 32 * i, before = cum;
        found = !past && cum + sum > bound;
        cum += sum;
      }
    }
  }
  past = !found;
  double x[4];
  residual(one_vec, k_hit, 1, [&](int, const float4& h, const float4& l) {
    x[0] = (double)h.x + (double)l.x, x[1] = (double)h.y + (double)l.y;
    x[2] = (double)h.z + (double)l.z, x[3] = (double)h.w + (double)l.w;
  });
  const double four = (x[0] + x[1]) + (x[2] + x[3]);
  double incl = four;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  int top = -1, hit = -1;
  double c = before + (incl - four);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    c += x[e];
    if (x[e] > 0.0) {
      top = 4 * (k_hit + lane) - shift + e;
      if (!past && hit < 0 && c > bound) hit = top;
    }
  }
  const uint32_t hits = __ballot_sync(0xffffffffu, hit >= 0), tops = __ballot_sync(0xffffffffu, top >= 0);
  const int token_at = hits != 0 ? __shfl_sync(0xffffffffu, hit, __ffs(hits) - 1)
                                 : __shfl_sync(0xffffffffu, top, 31 - __clz(tops));
  if (lane == 0) a.next_tokens[r] = token_at;
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
  int prefix = 0;
  if (lane == 0) {
    prefix = a.prefix_lens[r];  // (seq_lens may be the same array)
    a.seq_lens[r] = prefix + count;
    if (r == a.batch - 1) *a.num_freed = (int32_t)(free_at + n - count);
  }
  prefix = __shfl_sync(0xffffffffu, prefix, 0);
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
  // As many CTAs as run at once: half of one's time is a chain of loads, sums and
  // barriers that its span does not shorten.  Its warps take 128 values at the least.
  const int at_once = num_sms() * (a.draft_probs != nullptr ? ctas_per_sm<true>() : ctas_per_sm<false>());
  int cluster = kMaxCluster;
  while (cluster > 1 && ((int64_t)a.batch * cluster > at_once || a.vocab < cluster * kWarps * 128)) cluster /= 2;
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
