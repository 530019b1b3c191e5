// Attention of drafted tokens (speculative decoding) on tcgen05 tensor cores.
//
// A request holds a prefix of p cached tokens and a tree of n drafted ones, all
// stored in the pool.  Node t's query sees the prefix and, of the tree, itself
// and the nodes above it:
//     out[t, h] = softmax_j(scale q[t, h] . K_j) V over j < p and j = p + i,
//     i in {t, parent(t), parent(parent(t)), ...}.
//
// The n g query rows that share a KV head (g = Hq / Hkv) are too few to fill the
// 128 rows of a tensor-core tile, and the keys are many, so the keys take the
// tile's rows and the queries its columns:
//     S^T [128 keys x N] = K Q^T,   O^T [D x N] += V^T P^T,
// N = 16, 32, 64 or 128 columns.  A tile costs the tensor core what its columns
// need, K and V enter it as they lie in shared memory (K as a K-major operand,
// V^T as an MN-major one), and up to 128 query rows read each key once: the call
// is bound by HBM.  A thread owns a key's row of S^T: it exponentiates N columns
// and stores them as 16-byte pieces of an MN-major P^T.
//
// Softmax: all keys of a block use one reference per column, the maximum of the
// segment's first block; a later block is accepted while no weight exceeds 2^30
// (bf16; 2^15 in f16), so maxima over the keys, which lie across the threads, are
// rare: a butterfly that leaves one column a lane.  Sums are held by column in
// each thread, in fp32, and added up at the segment's end.
//
// Work: (KV head, request, tile of columns) are units of 128-key blocks, laid
// one after another; every CTA, one an SM, takes an equal run of blocks.  A
// unit that one CTA holds whole is written as it ends; the pieces of the others
// leave fp32 states that a second kernel merges.  KV heads are the outermost
// index, so the CTAs of neighbouring heads walk the same slots at about the same
// time and their rows share DRAM pages.
//
// A prefix that the whole batch shares (shared_len) is a unit of its own, whose
// columns are the rows of all requests: a launch before that of the rest.
//
// Roles: softmax warps (a warpgroup for 32 columns), four epilogue warps, which also
// list the CTA's units ahead for the others, producer warps (16-byte copies into the
// swizzled rings; over e4m3 pools they widen the codes to f16 in place), one thread
// that issues MMAs as their operands arrive.  S is held three times (twice with 128
// columns), P, O and (but for 128 columns) Q twice, so that the roles meet neither at
// a block's end nor at a unit's.  Waits are bounded as in the extend kernels.
//
// What it measured (of the copy benchmark's 6.78 TB/s, 32 query heads of 128 on 8): 128
// requests of 1,024 to 32,768 tokens, 8 drafts, 16 query heads on 8: 711 to 741 us, 6.5 to
// 6.8 TB/s, 0.96 to 1.00.  64 requests of 4,000 tokens: 4, 8, 16 and 32 drafts (16 to 128
// columns) 174, 177, 209 and 326 us, 0.89 to 0.49: beyond 32 columns by what the warps
// issue and wait for (128 columns: 10,400 warp instructions a block, issue slots busy 52%,
// DRAM 46%, tensor pipe 20%).  e4m3: 207, 213, 306 and 592 us, 0.38 and less: shared memory
// carries each code as a copy, a load, stores of twice its size and the MMAs' reads, and
// with 64 columns (the most) the ring has room for two tiles on their way.  One request of
// 16,384 tokens, 5 drafts: 25 us, six blocks a CTA between start and merge.  A chain of
// more than 64 query rows a KV head is faster as an extend where requests are many (64
// x 32 drafts: 266 us).
#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.h"

namespace sgl {
namespace vfy {
namespace {

constexpr int BN = 128;         // keys of a block
constexpr int kMaxCtas = 160;   // of a launch (sizes the workspace)
constexpr int kMaxStages = 12;

template <int D, int N, bool kFp8>
struct Cfg {
  static_assert(N <= (kFp8 ? 64 : 128), "columns");
  static constexpr int kCols = N < 32 ? N : 32;  // columns of a softmax warpgroup
  // of which a thread holds the scores of so many at a time (and the sums of all)
  static constexpr int kHeld = N == 128 ? 16 : kCols;
  static constexpr int kWgs = N / kCols;
  // warps: softmax, epilogue (4), producers, MMA
  static constexpr int kSoftWarps = 4 * kWgs;
  static constexpr int kProdWarp = kSoftWarps + 4;
  static constexpr int kProdWarps = kFp8 ? 11 : 7;
  static constexpr int kProdThreads = 32 * kProdWarps;
  static constexpr int kMmaWarp = kProdWarp + kProdWarps;
  static constexpr int kThreads = 32 * (kMmaWarp + 1);
  // Registers.  16 warps are launched with 128 a thread; with more, the softmax
  // warps take some of the others' (setmaxnreg; the shares add up to the launch's
  // registers at most).  A register that does not fit costs much here: its load waits
  // behind the copies.  The softmax needs 104, the epilogue 80 and the producers 72
  // without one; 24 warps (e4m3, 64 columns) leave 96, 72 and 72, 28 warps (128 columns)
  // 80, 64 and 56.
  static constexpr int kWarps = kThreads / 32;
  static constexpr bool kSplitRegs = kWarps > 16;
  static constexpr int kLaunchRegs = kWarps == 28 ? 72 : kWarps == 24 ? 80 : 96;
  static constexpr int kSoftRegs = kWarps == 28 ? 80 : kWarps == 24 ? 96 : 104;
  static constexpr int kEpiRegs = kWarps == 28 ? 64 : kWarps == 24 ? 72 : 80;
  static constexpr int kProdRegs = kWarps == 28 ? 56 : kWarps == 24 ? 72 : 96;
  static_assert(!kSplitRegs || kWarps * kLaunchRegs >= kSoftWarps * kSoftRegs + 4 * kEpiRegs +
                                                           (kProdWarps + 1) * kProdRegs,
                "register split within the launch's registers");
  static constexpr int kChunks = D / 64;         // 128-byte pieces of a row of 16-bit values
  static constexpr int kChunkBytes = 128 * 128;  // 128 rows of one
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  static constexpr int kQChunkBytes = N * 128;
  static constexpr int kQBytes = kChunks * kQChunkBytes;
  static constexpr int kQBufs = N == 128 ? 1 : 2;
  // P^T: a key's row is min(N, 64) values, swizzled over as many bytes
  static constexpr int kPRow = N >= 64 ? 128 : 2 * N;
  static constexpr int kPChunkBytes = 128 * kPRow;
  static constexpr int kPBytes = (N + 63) / 64 * kPChunkBytes;
  static constexpr uint64_t kPLayout = N >= 64 ? 2 : N == 32 ? 4 : 6;  // 128-, 64-, 32-byte swizzle
  static constexpr int kMiscBytes = 3 * 1024;
  static constexpr int kFit = (227 * 1024 - kMiscBytes - kQBufs * kQBytes - 2 * kPBytes) / kTileBytes;
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kK = (kStages + 1) / 2, kV = kStages / 2;  // the K and the V ring
  static constexpr int kSmem = kQBufs * kQBytes + 2 * kPBytes + kStages * kTileBytes + kMiscBytes;
  // S^T is held so often; a K slot's barrier tells its readers of S too, so there
  // are no more of those than K slots
  static constexpr int kSBufs = N == 128 ? 2 : 3;
  static constexpr int kTmemCols = N == 128 ? 512 : 8 * N;
  static constexpr int kColO = kSBufs * N;
  // largest accepted exponent of a weight, and where the reference puts a
  // segment's largest: f16 weights start at 2^8, so that they reach down to 2^-32
  // of it before they round to nothing
  static constexpr float kAccept = kFp8 ? 15.f : 30.f;
  static constexpr float kShift = kFp8 ? 8.f : 0.f;
  static_assert(kV >= 2 && kK >= kSBufs && kStages <= kMaxStages && kSmem <= 227 * 1024, "shared memory");
  static_assert(kColO + 2 * N <= kTmemCols && kTmemCols <= 512, "tensor memory");
};

// A CTA's first block (found by one warp) and what all roles go by.
struct Start {
  int32_t kvh, r, tile, off, b, blocks;  // blocks: how many the CTA takes
  int32_t first_req;                     // first request with tokens
  int32_t tokens;                        // of the batch
  int32_t ctas;                          // that have blocks, each of them at least one
  int64_t pos, total;                    // first block, blocks of the launch
};

// What the softmax and the epilogue go by in a segment (the blocks of a unit that
// a CTA takes).  The epilogue's first warp writes it, two segments ahead, so that
// no softmax warp waits for a load from global memory.
struct Segment {
  int32_t b0, take, nb;      // first block, blocks of it; blocks of the unit
  int32_t vis, n_tree;       // keys that all see; the tree's nodes behind them
  int32_t t0, h0, live;      // token and head of the tile's first column, columns of it
  int32_t off, kvh;          // the request's first token among the step's
  int8_t up[kMaxDraft];      // parents (below 0: none)
};

struct Misc {
  uint64_t q_full[2], q_empty[2], p_ready[2], o_full[2], o_free[2], u_full[2], l_full, l_free, drain;
  // a slot's copies have landed; it has been read (the MMA that reads it is done,
  // so what waits for S^T or for P^T's buffer waits for this too)
  uint64_t k_full[kMaxStages / 2], k_done[kMaxStages / 2], v_full[kMaxStages / 2], v_done[kMaxStages / 2];
  int32_t k_last[kMaxStages / 2];  // the slot's block is its segment's last
  uint32_t tmem_base;
  int abort;
  Start start;
  Segment seg[2];
  alignas(16) float mcol[128];  // a column's reference (read four at a time)
  int32_t mxcol[128];  // its block maximum, as an ordered integer; then (as a float) its rescaling;
                       // at a segment's end a warp's sums
  float lcol[2][128];  // at a segment's end: sums over the keys, references (then output factors)
};
static_assert(sizeof(Misc) <= 3 * 1024, "barriers and column states");

struct Params {
  const __nv_bfloat16* q;
  const void* pool_k;
  const void* pool_v;
  const int32_t* rtt;
  int64_t rtt_stride;
  const int32_t* req_pool_idx;
  const int32_t* prefix_lens;
  const int32_t* draft_lens;
  const int32_t* parents;
  __nv_bfloat16* out;
  int32_t Hq, Hkv, g, cols;
  int32_t batch, total, max_draft, max_prefix, shared;
  bool shared_pass;  // the launch over the batch's shared prefix
  float scale_log2, o_scale;
  int* status;  // word 0: the bounded waits' status; word 1: tokens of the batch
  uint64_t wait_ns;
  // states: CTA c's piece of a unit goes to slot 2c + 1 (the unit's first piece)
  // or 2c, N rows each; whole units' rows go to row_ml / row_acc (nullptr: their
  // output is written)
  int4* info;  // per row: first CTA, last CTA, column
  float2* slot_ml;
  float* slot_acc;
  float2* row_ml;
  float* row_acc;
};

SGL_DEV int32_t drafts_of(const Params& p, int r) { return max(0, min(__ldg(p.draft_lens + r), p.max_draft)); }
SGL_DEV int32_t prefix_of(const Params& p, int r) { return max(0, min(__ldg(p.prefix_lens + r), p.max_prefix)); }

// The requests that a CTA comes to, in order, from the one it starts with: a warp
// holds the lengths of 64 (lane l those of numbers base + l and base + 32 + l), the
// later half on its way while the first is used: a load that waits behind the
// copies takes 2 us.
struct Requests {
  int32_t n[2], pre[2], row[2], base, first;
  SGL_DEV void fill(const Params& p, int h) {
    const int r = (int)(((int64_t)first + base + 32 * h + (threadIdx.x & 31)) % p.batch);
    n[h] = drafts_of(p, r), pre[h] = prefix_of(p, r), row[h] = __ldg(p.req_pool_idx + r);
  }
  SGL_DEV Requests(const Params& p, const Start& s) : base(0), first(s.r) {
    fill(p, 0);
    fill(p, 1);
  }
  SGL_DEV void get(const Params& p, int u, int32_t* nn, int32_t* pp, int32_t* rr) {
    while (u - base >= 32) {
      n[0] = n[1], pre[0] = pre[1], row[0] = row[1];
      base += 32;
      fill(p, 1);
    }
    *nn = __shfl_sync(0xffffffffu, n[0], u - base);
    *pp = __shfl_sync(0xffffffffu, pre[0], u - base);
    *rr = __shfl_sync(0xffffffffu, row[0], u - base);
  }
};

// One block after another of a CTA's run.  keys [0, vis) of a unit are seen by
// every column, keys [vis, vis + n_tree) are its request's tree.
struct Cursor {
  int32_t kvh, r, u, tile, off, n, b, nb, tiles;
  int32_t k0, vis, n_tree, row;  // first position; keys; row of the table
  SGL_DEV void lens(const Params& p, int32_t n_, int32_t pre, int32_t row_) {
    n = n_, row = row_;
    n_tree = (int32_t)min((int64_t)n, p.rtt_stride - pre);  // positions end with the row
    k0 = min(p.shared, pre);
    vis = pre - k0;
    tiles = (n * p.g + p.cols - 1) / p.cols;
    nb = n > 0 ? (vis + n_tree + BN - 1) / BN : 0;
  }
  SGL_DEV Cursor() {}
  SGL_DEV Cursor(const Params& p, const Start& s, Requests& q) {
    kvh = s.kvh, r = s.r, u = 0, tile = s.tile, off = s.off, b = s.b;
    if (p.shared_pass) {
      n = s.tokens;
      k0 = 0, vis = p.shared, n_tree = 0;
      row = __ldg(p.req_pool_idx + s.first_req);
      tiles = (n * p.g + p.cols - 1) / p.cols;
      nb = (vis + BN - 1) / BN;
    } else {
      int32_t n_, pre, row_;
      q.get(p, 0, &n_, &pre, &row_);
      lens(p, n_, pre, row_);
    }
  }
  // the first block of the next unit (there is one: the caller counts blocks)
  SGL_DEV void next_unit(const Params& p, Requests& q) {
    b = 0;
    if (++tile < tiles) return;
    tile = 0;
    if (p.shared_pass) {
      ++kvh;
      return;
    }
    do {
      off += n;
      ++u;
      if (++r >= p.batch) r = 0, off = 0, ++kvh;
      int32_t n_, pre, row_;
      q.get(p, u, &n_, &pre, &row_);
      lens(p, n_, pre, row_);
    } while (nb == 0);
  }
  SGL_DEV void advance(const Params& p, Requests& q) {
    if (++b == nb) next_unit(p, q);
  }
};

// The CTA whose run of blocks holds block x: runs start at c * total / ctas.
SGL_DEV int32_t owner(int64_t x, int64_t total, int32_t ctas) { return (int32_t)(((x + 1) * ctas - 1) / total); }

// Finds the CTA's run of blocks (one warp).
SGL_DEV void find_start(const Params& p, Start* out) {
  const int lane = threadIdx.x & 31;
  int64_t blocks = 0;
  int32_t tokens = 0, first = p.batch;
  for (int r = lane; r < p.batch; r += 32) {
    Cursor c;
    c.lens(p, drafts_of(p, r), prefix_of(p, r), 0);
    if (!p.shared_pass) blocks += (int64_t)c.nb * c.tiles;
    tokens += c.n;
    if (c.n > 0) first = min(first, r);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    blocks += __shfl_xor_sync(0xffffffffu, blocks, o);
    tokens += __shfl_xor_sync(0xffffffffu, tokens, o);
    first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
  }
  tokens = min(tokens, p.total);
  Start s = {};
  s.tokens = tokens;
  s.first_req = first;
  if (p.shared_pass) blocks = (int64_t)((tokens * p.g + p.cols - 1) / p.cols) * ((p.shared + BN - 1) / BN);
  const int64_t total = blocks * p.Hkv;
  s.total = total;
  // (a CTA without blocks would leave a state of an earlier call in the middle of a
  // unit's pieces)
  s.ctas = (int32_t)min((int64_t)gridDim.x, total);
  if ((int)blockIdx.x < s.ctas) {
    s.pos = total * blockIdx.x / s.ctas;
    s.blocks = (int32_t)(total * (blockIdx.x + 1) / s.ctas - s.pos);
  }
  if (s.blocks > 0) {
    s.kvh = (int32_t)(s.pos / blocks);
    int64_t rem = s.pos % blocks;
    if (p.shared_pass) {
      const int32_t nb = (p.shared + BN - 1) / BN;
      s.r = first;
      s.tile = (int32_t)(rem / nb);
      s.b = (int32_t)(rem % nb);
    } else {
      int32_t off = 0;
      for (int r0 = 0;; r0 += 32) {
        const int r = r0 + lane;
        int64_t mine = 0;
        int32_t n = 0, nb = 1;
        if (r < p.batch) {
          Cursor c;
          c.lens(p, drafts_of(p, r), prefix_of(p, r), 0);
          n = c.n, nb = max(1, c.nb);
          mine = (int64_t)c.nb * c.tiles;
        }
        int64_t cum = mine;
        int32_t at = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t a = __shfl_up_sync(0xffffffffu, cum, o);
          const int32_t t = __shfl_up_sync(0xffffffffu, at, o);
          if (lane >= o) cum += a, at += t;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, cum > rem);
        if (hit != 0) {
          const int w = __ffs(hit) - 1;
          const int64_t in = rem - __shfl_sync(0xffffffffu, cum - mine, w);
          const int32_t nbw = __shfl_sync(0xffffffffu, nb, w);
          s.r = r0 + w;
          s.off = off + __shfl_sync(0xffffffffu, at - n, w);
          s.tile = (int32_t)(in / nbw);
          s.b = (int32_t)(in % nbw);
          break;
        }
        if (r0 + 32 >= p.batch) break;  // (not reached: rem < blocks)
        rem -= __shfl_sync(0xffffffffu, cum, 31);
        off += __shfl_sync(0xffffffffu, at, 31);
      }
    }
  }
  if (lane == 0) *out = s;
}

SGL_DEV uint32_t sw128(int row, int ci) { return row * 128 + ((ci ^ (row & 7)) << 4); }

SGL_DEV bool warp_wait(uint64_t* bar, uint32_t parity, Misc* m, const Params& p) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait_bounded(bar, parity, &m->abort, p.status, p.wait_ns);
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

// floats as integers of the same order
SGL_DEV int32_t ordered(float x) {
  const int32_t i = __float_as_int(x);
  return i < 0 ? i ^ 0x7fffffff : i;
}
SGL_DEV float unordered(int32_t i) { return __int_as_float(i < 0 ? i ^ 0x7fffffff : i); }

// v[c] of every lane combined over the warp; lane l is left with column l % W.
template <int W, typename Op>
SGL_DEV float columns(float (&v)[W], Op op) {
  const int lane = threadIdx.x & 31;
  if constexpr (W == 16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = op(v[i], __shfl_xor_sync(0xffffffffu, v[i], 16));
  }
#pragma unroll
  for (int s = W / 2; s > 0; s >>= 1) {
    const bool upper = lane & s;
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float keep = upper ? v[i + s] : v[i], send = upper ? v[i] : v[i + s];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, s));
    }
  }
  return v[0];
}

SGL_DEV void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
template <int W>
SGL_DEV void tmem_ld(uint32_t taddr, uint32_t (&r)[W]) {
  if constexpr (W == 32) tmem_ld32(taddr, r);
  else tmem_ld16(taddr, r);
  tmem_wait_ld();
}
template <int W>
SGL_DEV void tmem_st(uint32_t taddr, const uint32_t (&r)[W]) {
  if constexpr (W == 32) tmem_st32(taddr, r);
  else tmem_st16(taddr, r);
}

// Instruction descriptor, kind::f16, fp32 accumulator, M = 128; S^T = K Q^T has
// both operands K-major, O^T = V^T P^T both MN-major.
template <int N, bool kFp8>
constexpr uint32_t idesc(bool mn_major) {
  return make_idesc_bf16(128, N, mn_major, kFp8) | ((mn_major ? 1u : 0u) << 15);
}

// ----------------------------------------------------------------- producers

// A unit's query rows into its Q tile: a request's rows are (token, head of the KV
// head's group), tile t holds rows t N .. t N + N - 1.
template <int D, int N, bool kFp8>
SGL_DEV void copy_q(const Params& p, const Segment& g, uint32_t sQ, int ptid) {
  using C = Cfg<D, N, kFp8>;
  const int ci = ptid & 7;
  const int64_t row0 = (int64_t)(g.off + g.t0) * p.Hq + (int64_t)g.kvh * p.g;
  for (int row = ptid >> 3; row < N; row += C::kProdThreads / 8) {
    const bool valid = row < g.live;
    const int r = g.h0 + row;
    const __nv_bfloat16* src = p.q + (valid ? (row0 + (int64_t)(r / p.g) * p.Hq + r % p.g) * D : 0) + ci * 8;
#pragma unroll
    for (int h = 0; h < C::kChunks; ++h)
      cp_async_16(sQ + h * C::kQChunkBytes + sw128(row, ci), src + 64 * h, valid ? 16u : 0u);
  }
}
// The thread's own pieces of it, landed, from bf16 to f16 (e4m3 pools).
template <int D, int N>
SGL_DEV void widen_q(uint32_t sQ, int ptid) {
  using C = Cfg<D, N, true>;
  const int ci = ptid & 7;
  for (int row = ptid >> 3; row < N; row += C::kProdThreads / 8) {
#pragma unroll
    for (int h = 0; h < C::kChunks; ++h) {
      const uint32_t at = sQ + h * C::kQChunkBytes + sw128(row, ci);
      float f[8];
      bf16x8_to_f32(ld_shared_v4(at), f);
      st_shared_v4(at, pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]),
                   pack_f16x2(f[6], f[7]));
    }
  }
}

// The slots of a block's rows first, first + step, ...; -1 where there is no key.
// Those of later blocks are called into the L2: behind a ring full of copies a load
// that goes to memory takes as long as the ring lasts.
constexpr int kSlotsAhead = 6;
template <int kRows>
SGL_DEV void load_slots(const Params& p, const Cursor& c, int first, int step, int32_t (&slot)[kRows]) {
  const int32_t at = c.b * BN;
  const int32_t* t = p.rtt + c.row * p.rtt_stride + c.k0;
  const int32_t all = c.vis + c.n_tree, keys = min(all - at, BN);
#pragma unroll
  for (int i = 0; i < kRows; ++i) slot[i] = first + step * i < keys ? __ldg(t + at + first + step * i) : -1;
  // one warp's threads, a line of 32 slots each: at a unit's start kSlotsAhead blocks
  const int ahead = at + (c.b == 0 ? first * 32 : kSlotsAhead * BN + first * 32);
  if (first < (c.b == 0 ? 4 * (kSlotsAhead + 1) : 4) && ahead < all)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(t + ahead));
}

// Where the producers are in the segments (every thread for itself).
struct Place {
  int seg = -1, left = 0;
  bool opens;
  SGL_DEV bool step(Misc* m, const Params& p) {
    opens = left == 0;
    if (opens) {
      ++seg;
      if (!warp_wait(&m->u_full[seg & 1], (seg >> 1) & 1, m, p)) return false;
      left = m->seg[seg & 1].take;
    }
    --left;
    return true;
  }
};

template <int D, int N>
SGL_DEV void produce(const Params& p, const Start& s, Misc* m, uint32_t sQ, uint32_t sKV, int ptid) {
  using C = Cfg<D, N, false>;
  constexpr int kStep = C::kProdThreads / 8, kRows = (BN + kStep - 1) / kStep;
  const int ci = ptid & 7, rb = ptid >> 3;
  Requests req(p, s);
  Cursor c(p, s, req);  // one block ahead: its slots are on their way
  int32_t slot[kRows], next[kRows];
  load_slots(p, c, rb, kStep, slot);
  Place at;
  auto query = [&]() {
    const int qb = at.seg % C::kQBufs, round = at.seg / C::kQBufs;
    if (round > 0 && !warp_wait(&m->q_empty[qb], (round - 1) & 1, m, p)) return false;
    copy_q<D, N, false>(p, m->seg[at.seg & 1], sQ + qb * C::kQBytes, ptid);
    cp_async_mbar_arrive(&m->q_full[qb]);
    return true;
  };
  for (int i = 0; i < s.blocks; ++i) {
    if (!at.step(m, p)) return;
    const int32_t kvh = m->seg[at.seg & 1].kvh;
    if (i + 1 < s.blocks) {
      c.advance(p, req);
      load_slots(p, c, rb, kStep, next);
    }
    if (at.opens && C::kQBufs == 2 && !query()) return;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const int ring = kv ? C::kV : C::kK, st = i % ring, round = i / ring;
      uint64_t* full = kv ? m->v_full : m->k_full;
      uint64_t* done = kv ? m->v_done : m->k_done;
      if (round > 0 && !warp_wait(&done[st], (round - 1) & 1, m, p)) return;
      const __nv_bfloat16* pool = static_cast<const __nv_bfloat16*>(kv ? p.pool_v : p.pool_k);
      const uint32_t dst = sKV + (kv ? C::kK + st : st) * C::kTileBytes;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int row = rb + kStep * r;
        if (row >= BN) break;
        const bool valid = slot[r] >= 0;
        const __nv_bfloat16* src = pool + ((int64_t)(valid ? slot[r] : 0) * p.Hkv + kvh) * D + ci * 8;
#pragma unroll
        for (int h = 0; h < C::kChunks; ++h)
          cp_async_16(dst + h * C::kChunkBytes + sw128(row, ci), src + 64 * h, valid ? 16u : 0u);
      }
      cp_async_mbar_arrive(&full[st]);
      if (kv == 0 && ptid == 0) {
        m->k_last[st] = at.left == 0;
        mbar_arrive(&full[st]);
      }
    }
    // one Q tile alone: the next unit's waits for the last scores of this one,
    // and its first keys go ahead of it
    if (at.opens && C::kQBufs == 1 && !query()) return;
#pragma unroll
    for (int r = 0; r < kRows; ++r) slot[r] = next[r];
  }
}

// e4m3 pool: a row's codes are copied into the second half of its place in the slot
// and widened to f16 from there, by the threads of the warp that copied them, so
// every free slot has codes on their way and no staging of its own.  Tiles (K and V
// in turn) are copied kLag ahead of the one that is widened: as many as leave the
// MMAs slots besides.  (Codes held in registers instead, one block
// ahead: 1,328 us on 48 requests of up to 16,000 tokens, 32 drafts, 32 heads on 8.)
template <int D, int N>
SGL_DEV void produce_fp8(const Params& p, const Start& s, Misc* m, uint32_t sQ, uint32_t sKV, int ptid) {
  using C = Cfg<D, N, true>;
  constexpr int kPieces = D / 16;  // 16-byte pieces of a row of codes
  constexpr int kStep = C::kProdThreads / kPieces, kRows = (BN + kStep - 1) / kStep;
  // A wait ends as long as what it waits for can be widened before: V's slot the
  // tile 2 kV before it, and with units of one block the segment (listed once the
  // scores of the one two before are through) and its Q tile K two blocks before.
  constexpr int kLag = C::kV == 2 ? 2 : 3;
  static_assert(kLag <= 2 * C::kV - 1 && kLag <= 3, "a producer waits for what it has not widened");
  const int rc = ptid % kPieces, rb = ptid / kPieces;
  const int raw = (D == 128 ? C::kChunkBytes : 64) + rc * 16;  // the thread's codes in a row's place
  Requests req(p, s);
  Cursor c(p, s, req);  // one block ahead of the copies
  int32_t slot[kRows], next[kRows];
  load_slots(p, c, rb, kStep, slot);
  Place at;
  int seg_w = 0;
  int32_t kvh = 0;
  uint32_t firsts = 0, lasts = 0;  // bit b % 32: block b is its segment's first, last
  auto copy = [&](int i, int kv) {
    const int ring = kv ? C::kV : C::kK, st = i % ring, round = i / ring;
    if (!kv) {
      if (!at.step(m, p)) return false;
      const uint32_t bit = 1u << (i & 31);
      firsts = at.opens ? firsts | bit : firsts & ~bit;
      lasts = at.left == 0 ? lasts | bit : lasts & ~bit;
      if (i + 1 < s.blocks) {
        c.advance(p, req);
        load_slots(p, c, rb, kStep, next);
      }
      if (at.opens) {
        const int seg = at.seg;
        kvh = m->seg[seg & 1].kvh;
        if (seg >= 2 && !warp_wait(&m->q_empty[seg & 1], ((seg >> 1) - 1) & 1, m, p)) return false;
        copy_q<D, N, true>(p, m->seg[seg & 1], sQ + (seg & 1) * C::kQBytes, ptid);
      }
    }
    if (round > 0 && !warp_wait(kv ? &m->v_done[st] : &m->k_done[st], (round - 1) & 1, m, p)) return false;
    const uint8_t* pool = static_cast<const uint8_t*>(kv ? p.pool_v : p.pool_k);
    const uint32_t dst = sKV + (kv ? C::kK + st : st) * C::kTileBytes + raw;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int row = rb + kStep * r;
      if (row >= BN) break;
      const bool valid = slot[r] >= 0;
      cp_async_16(dst + row * 128, pool + ((int64_t)(valid ? slot[r] : 0) * p.Hkv + kvh) * D + rc * 16,
                  valid ? 16u : 0u);
    }
    if (kv) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) slot[r] = next[r];
    }
    return true;
  };
  auto widen = [&](int i, int kv) {
    const int st = i % (kv ? C::kV : C::kK);
    const uint32_t tile = sKV + (kv ? C::kK + st : st) * C::kTileBytes;
    uint4 w[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int row = rb + kStep * r;
      if (row < BN) w[r] = ld_shared_v4(tile + raw + row * 128);
    }
    __syncwarp();  // a row's codes have been read by all its threads
    const uint32_t dst = tile + (rc >> 2) * C::kChunkBytes;
    const int piece = 2 * (rc & 3);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int row = rb + kStep * r;
      if (row >= BN) break;
      const uint32_t x[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x[j] & 0xffffu), __NV_E4M3);
        const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x[j] >> 16), __NV_E4M3);
        o[2 * j] = *reinterpret_cast<const uint32_t*>(&a);
        o[2 * j + 1] = *reinterpret_cast<const uint32_t*>(&b);
      }
      // (a row's two halves lie 16 KB apart, on the same banks: their threads store
      // their pieces in opposite order)
      const int swap = rc >> 2;
      st_shared_v4(dst + sw128(row, piece + swap), swap ? o[4] : o[0], swap ? o[5] : o[1], swap ? o[6] : o[2],
                   swap ? o[7] : o[3]);
      st_shared_v4(dst + sw128(row, piece + 1 - swap), swap ? o[0] : o[4], swap ? o[1] : o[5], swap ? o[2] : o[6],
                   swap ? o[3] : o[7]);
    }
    const bool first = !kv && (firsts >> (i & 31) & 1);
    if (first) widen_q<D, N>(sQ + (seg_w & 1) * C::kQBytes, ptid);
    fence_proxy_async_smem();
    if (first) mbar_arrive(&m->q_full[seg_w & 1]), ++seg_w;
    uint64_t* full = kv ? &m->v_full[st] : &m->k_full[st];
    if (!kv && ptid == 0) {
      m->k_last[st] = lasts >> (i & 31) & 1;
      mbar_arrive(full);
    }
    mbar_arrive(full);
  };
  const int tiles = 2 * s.blocks;
  for (int t = 0; t < tiles + kLag; ++t) {
    if (t < tiles && !copy(t >> 1, t & 1)) return;
    cp_async_commit();  // one group a tile (an empty one past the last)
    if (t >= kLag) {
      cp_async_wait<kLag>();  // the thread's copies of tile t - kLag have landed
      widen((t - kLag) >> 1, (t - kLag) & 1);
    }
  }
}

// ----------------------------------------------------------------- MMA

// The next scores or the next P V, whichever's operands are there first.
template <int D, int N, bool kFp8>
SGL_DEV void issue(const Params& p, const Start& s, Misc* m, uint32_t tmem, uint32_t sQ, uint32_t sP, uint32_t sKV) {
  using C = Cfg<D, N, kFp8>;
  auto there = [&](uint64_t* bar, uint32_t parity) { return mbar_try_wait(bar, parity, 20u); };
  int i = 0, j = 0;  // next block of S^T, of O^T
  uint32_t lasts = 0;  // bit b % 32: block b is its segment's last
  int seg = 0, seg_v = 0;
  bool opens = true, opens_v = true;
  uint32_t idle = 0;
  uint64_t since = 0;
  while (j < s.blocks) {
    bool moved = false;
    if (i < s.blocks && i < j + C::kSBufs) {
      const int st = i % C::kK, qb = seg % C::kQBufs;
      if (there(&m->k_full[st], (i / C::kK) & 1) && (!opens || there(&m->q_full[qb], (seg / C::kQBufs) & 1))) {
        fence_proxy_async_smem();
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t a = make_sw128_desc(sKV + st * C::kTileBytes + (kk >> 2) * C::kChunkBytes + (kk & 3) * 32, 16, 1024);
          const uint64_t b = make_sw128_desc(sQ + qb * C::kQBytes + (kk >> 2) * C::kQChunkBytes + (kk & 3) * 32, 16, 1024);
          umma_ss(tmem + (i % C::kSBufs) * N, a, b, idesc<N, kFp8>(false), kk > 0 ? 1u : 0u);
        }
        opens = m->k_last[st] != 0;
        lasts = (lasts & ~(1u << (i & 31))) | ((opens ? 1u : 0u) << (i & 31));
        umma_commit(&m->k_done[st]);
        if (opens) umma_commit(&m->q_empty[qb]), ++seg;
        ++i;
        moved = true;
      }
    }
    if (j < i) {
      const int st = j % C::kV, ob = seg_v & 1;
      if (there(&m->p_ready[j & 1], (j >> 1) & 1) && there(&m->v_full[st], (j / C::kV) & 1) &&
          (!opens_v || seg_v < 2 || there(&m->o_free[ob], ((seg_v >> 1) - 1) & 1))) {
        fence_proxy_async_smem();
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk) {
          // 16 keys are 16 rows in V as in P; 64 dims (or columns) further on lies the
          // next chunk.  D = 64: the tile's rows 64.. repeat the others.
          const uint64_t a = make_sw128_desc(sKV + (C::kK + st) * C::kTileBytes + kk * 2048, D == 128 ? C::kChunkBytes : 0, 1024);
          const uint64_t b = (make_sw128_desc(sP + (j & 1) * C::kPBytes + kk * 16 * C::kPRow, C::kPChunkBytes, 8 * C::kPRow) &
                              ~((uint64_t)7 << 61)) | (C::kPLayout << 61);
          umma_ss(tmem + C::kColO + ob * N, a, b, idesc<N, kFp8>(true), (opens_v && kk == 0) ? 0u : 1u);
        }
        umma_commit(&m->v_done[st]);
        opens_v = lasts >> (j & 31) & 1;
        if (opens_v) umma_commit(&m->o_full[ob]), ++seg_v;
        ++j;
        moved = true;
      }
    }
    if (moved) {
      idle = 0;
    } else if ((++idle & 63u) == 0) {  // bounded, as every wait
      const uint64_t now = global_timer_ns();
      if (idle == 64u) since = now;
      if (m->abort) return;
      if (now - since > p.wait_ns) {
        m->abort = 1;
        atomicExch(p.status, (int)kDevWaitTimeout);
        return;
      }
    }
  }
}

// ----------------------------------------------------------------- softmax

// Which of the W columns from col0 on see the thread's key, node `node` of the
// tree (below 0: a key that all see): bit e for column col0 + e, whose token has
// that node among itself and those above it.  Lanes hold the ancestor sets of
// nodes lane and lane + 32, which grow by doubling: each round adds what the node
// reached last has reached.
template <int W>
SGL_DEV uint32_t seen_by(const Params& p, const Segment& g, int node, int col0) {
  const int lane = threadIdx.x & 31;
  if (g.n_tree == 0) return node < 0 ? 0xffffffffu : 0u;
  uint64_t anc[2] = {1ull << lane, 1ull << (lane + 32)};
  int at[2] = {g.up[lane], g.up[lane + 32]};
  for (int span = 1; span < g.n_tree; span *= 2) {
    uint64_t a[2];
    int u[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int src = at[h] & 31;
      const uint64_t a0 = __shfl_sync(0xffffffffu, anc[0], src), a1 = __shfl_sync(0xffffffffu, anc[1], src);
      const int u0 = __shfl_sync(0xffffffffu, at[0], src), u1 = __shfl_sync(0xffffffffu, at[1], src);
      a[h] = at[h] < 0 ? 0ull : at[h] < 32 ? a0 : a1;
      u[h] = at[h] < 0 ? -1 : at[h] < 32 ? u0 : u1;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) anc[h] |= a[h], at[h] = u[h];
  }
  uint32_t bits = 0;
  int t = g.t0 + (g.h0 + col0) / p.g, lo = -((g.h0 + col0) % p.g);  // token, its first column
  for (; lo < W && t < 64; ++t, lo += p.g) {  // (columns past the tile's are not used)
    const uint64_t a = __shfl_sync(0xffffffffu, t < 32 ? anc[0] : anc[1], t & 31);
    const int c0 = max(0, lo), c1 = min(W, lo + p.g);
    const uint32_t span = (c1 - c0 >= 32 ? 0xffffffffu : (1u << (c1 - c0)) - 1u) << c0;
    if (node < 0 || (node < g.n_tree && (a >> node & 1))) bits |= span;
  }
  return bits;
}

// Byte of P^T at (key, column col, a multiple of 8): rows of kPRow bytes whose
// 16-byte pieces are swizzled.
template <int N>
SGL_DEV uint32_t p_at(int key, int col) {
  if constexpr (N == 16) return key * 32 + (((col >> 3) ^ ((key >> 2) & 1)) << 4);
  else if constexpr (N == 32) return key * 64 + (((col >> 3) ^ ((key >> 1) & 3)) << 4);
  else return (col >> 6) * (128 * 128) + sw128(key, (col & 63) >> 3);
}

template <int D, int N, bool kFp8>
SGL_DEV void softmax(const Params& p, const Start& s, Misc* m, uint32_t tmem, uint32_t sP) {
  using C = Cfg<D, N, kFp8>;
  constexpr int W = C::kCols, H = C::kHeld, kParts = W / H;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wg = warp >> 2, q = warp & 3, key = q * 32 + lane, col0 = wg * W, wt = tid & 127;
  const uint32_t bar = 1 + wg;
  const uint32_t lanes = (uint32_t)(q * 32) << 16;
  const float sc = p.scale_log2;
  int i = 0;
  bool ok = true;
  float l[W];
  for (int seg = 0; i < s.blocks; ++seg) {
    const Segment& g = m->seg[seg & 1];
    ok = warp_wait(&m->u_full[seg & 1], (seg >> 1) & 1, m, p) && ok;
    if (bar_red_or(bar, 128, !ok)) return;
    const int take = g.take;
    int node = g.b0 * BN + key - g.vis;  // of the tree; below 0 a key that all see
    const bool first_masked = (g.b0 + 1) * BN > g.vis;
    const int hidden_from = g.vis / BN - g.b0;  // first block of the segment with keys that some do not see
    const uint32_t tO = tmem + lanes + C::kColO + (seg & 1) * N + col0;
#pragma unroll
    for (int e = 0; e < W; ++e) l[e] = 0.f;
    for (int b = 0; b < take; ++b, ++i, node += BN) {
      const bool masked = b >= hidden_from, opens = b == 0;
      uint32_t bits = 0;
      if (masked) bits = seen_by<W>(p, g, node, col0);
      ok = warp_wait(&m->k_done[i % C::kK], (i / C::kK) & 1, m, p) && ok;  // S^T is there
      tc_fence_after();
      const uint32_t tS = tmem + lanes + (i % C::kSBufs) * N + col0;
      uint32_t x[H];
      auto load = [&](int part) {
        tmem_ld<H>(tS + part * H, x);
        if (masked) {
#pragma unroll
          for (int e = 0; e < H; ++e)
            if (!(bits >> (part * H + e) & 1)) x[e] = __float_as_uint(-INFINITY);
        }
      };
      // scores against their columns' references, in units of log 2
      auto relative = [&](int part) {
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        const float2 s2 = make_float2(sc, sc);
#pragma unroll
        for (int e = 0; e < H; e += 4) {
          const float4 r = *reinterpret_cast<const float4*>(&m->mcol[col0 + part * H + e]);
          const float2 a = ffma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), s2, make_float2(-r.x, -r.y));
          const float2 c = ffma2(make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), s2, make_float2(-r.z, -r.w));
          x[e] = __float_as_uint(a.x), x[e + 1] = __float_as_uint(a.y);
          x[e + 2] = __float_as_uint(c.x), x[e + 3] = __float_as_uint(c.y);
          top[(e >> 1) & 3] = fmax3(top[(e >> 1) & 3], a.x, a.y);
          top[((e >> 1) + 1) & 3] = fmax3(top[((e >> 1) + 1) & 3], c.x, c.y);
        }
        return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      };
      // a segment's first block sets the references; one whose first block hides
      // keys (columns may have seen none yet) sets them block by block
      bool redo = opens || (masked && first_masked);
      if (!redo) {
        float top = -INFINITY;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          load(part);
          top = fmaxf(top, relative(part));
        }
        redo = top > C::kAccept;
      }
      // the warpgroup agrees: lane 0 votes to move the references, lanes 1 to 8
      // that the warp gave up waiting
      const bool redo_w = __any_sync(0xffffffffu, redo);
      const uint32_t votes = bar_red_popc(bar, 128, (lane == 0 && redo_w) || (lane >= 1 && lane <= 8 && !ok));
      if (votes >= 8) return;
      if (votes != 0) {
        if (wt < W) m->mxcol[col0 + wt] = ordered(-INFINITY);
        named_bar_sync(bar, 128);
#pragma unroll 1
        for (int part = 0; part < kParts; ++part) {
          load(part);
          const float top = columns<H>(*reinterpret_cast<float(*)[H]>(&x), [](float a, float c) { return fmaxf(a, c); });
          atomicMax(&m->mxcol[col0 + part * H + (lane & (H - 1))], ordered(top));
        }
        named_bar_sync(bar, 128);
        if (wt < W) {
          const int col = col0 + wt;
          const float before = opens ? -INFINITY : m->mcol[col];
          const float now = fmaxf(before, unordered(m->mxcol[col]) * sc - C::kShift);
          m->mcol[col] = now;
          m->mxcol[col] = __float_as_int(before == -INFINITY ? 0.f : ex2(before - now));
        }
        named_bar_sync(bar, 128);
        if (!opens) {
          // O^T of the blocks before comes to the new references
          ok = warp_wait(&m->v_done[(i - 1) % C::kV], ((i - 1) / C::kV) & 1, m, p) && ok;
          tc_fence_after();
#pragma unroll
          for (int part = 0; part < kParts; ++part) {
            tmem_ld<H>(tO + part * H, x);
#pragma unroll
            for (int e = 0; e < H; ++e) {
              const float a = __int_as_float(m->mxcol[col0 + part * H + e]);
              l[part * H + e] *= a;
              x[e] = __float_as_uint(__uint_as_float(x[e]) * a);
            }
            tmem_st<H>(tO + part * H, x);
          }
          tmem_wait_st();
          named_bar_sync(bar, 128);  // all have read the factors: the segment's end writes sums there
        }
      }
      // P^T: this key's row, 8 columns a 16-byte piece; its buffer was last read
      // with block i - 2
      if (i >= 2) ok = warp_wait(&m->v_done[(i - 2) % C::kV], ((i - 2) / C::kV) & 1, m, p) && ok;
      const uint32_t pbuf = sP + (i & 1) * C::kPBytes;
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        if (kParts > 1 || votes != 0) {
          load(part);
          relative(part);
        }
        if (votes != 0) {
#pragma unroll
          for (int e = 0; e < H; ++e)  // a column that has seen no key yet
            if (m->mcol[col0 + part * H + e] == -INFINITY) x[e] = __float_as_uint(-INFINITY);
        }
#pragma unroll
        for (int e = 0; e < H; e += 8) {
          uint32_t o[4];
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const int at = e + 2 * d, c = part * H + at;
            const float2 w = make_float2(ex2(__uint_as_float(x[at])), ex2(__uint_as_float(x[at + 1])));
            const float2 sum = fadd2(make_float2(l[c], l[c + 1]), w);
            l[c] = sum.x, l[c + 1] = sum.y;
            o[d] = kFp8 ? pack_f16x2(w.x, w.y) : pack_bf16x2(w.x, w.y);
          }
          st_shared_v4(pbuf + p_at<N>(key, col0 + part * H + e), o[0], o[1], o[2], o[3]);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&m->p_ready[i & 1]);
    }
    // the segment's sums and references go to the epilogue warps
    if (seg > 0) ok = warp_wait(&m->l_free, (seg - 1) & 1, m, p) && ok;
    float sum = columns<W>(l, [](float a, float c) { return a + c; });
    const int col = col0 + lane;
    if (q > 0 && lane < W) (q == 1 ? m->lcol[0] : q == 2 ? m->lcol[1] : reinterpret_cast<float*>(m->mxcol))[col] = sum;
    if (bar_red_or(bar, 128, !ok)) return;
    if (q == 0) {
      if (lane < W) {
        m->lcol[0][col] = (sum + m->lcol[0][col]) + (m->lcol[1][col] + __int_as_float(m->mxcol[col]));
        m->lcol[1][col] = m->mcol[col];
      }
      mbar_arrive(&m->l_full);
    }
  }
}

// ----------------------------------------------------------------- epilogue

// A segment's O^T: lane d of warp q holds dim 32 q + d of every column.
template <int D, int N, bool kFp8>
SGL_DEV void epilogue(const Params& p, const Start& s, Misc* m, uint32_t tmem, int et) {
  using C = Cfg<D, N, kFp8>;
  constexpr int W = 16;
  const int q = et >> 5, lane = et & 31;
  const uint32_t bar = 1 + C::kWgs;
  // the first warp lists the segments; the parents of the one after next are on
  // their way meanwhile
  Requests req(p, s);
  Cursor c(p, s, req);
  int listed = 0, n_listed = 0;  // blocks, segments
  auto list = [&]() {
    if (listed >= s.blocks) return;
    Segment& g = m->seg[n_listed & 1];
    const int take = min(c.nb - c.b, s.blocks - listed), r0 = c.tile * N;
    int up[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = lane + 32 * h;
      up[h] = t < c.n_tree && c.off + t < p.total ? __ldg(p.parents + c.off + t) : -1;
      if (up[h] < 0 || up[h] >= t) up[h] = -1;  // a parent lies before its child
      g.up[t] = (int8_t)up[h];
    }
    if (lane == 0) {
      g.b0 = c.b, g.take = take, g.nb = c.nb, g.vis = c.vis, g.n_tree = c.n_tree, g.kvh = c.kvh;
      g.t0 = r0 / p.g, g.h0 = r0 % p.g, g.off = c.off;
      g.live = min(N, min(c.n, p.total - c.off) * p.g - r0);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&m->u_full[n_listed & 1]);
    listed += take;
    ++n_listed;
    if (listed < s.blocks) c.next_unit(p, req);
  };
  if (q == 0) {
    list();
    list();
  }
  int i = 0;
  for (int seg = 0; i < s.blocks; ++seg) {
    bool ok = q == 0 || warp_wait(&m->u_full[seg & 1], (seg >> 1) & 1, m, p);
    const Segment& g = m->seg[seg & 1];
    const int b0 = g.b0, take = g.take, nb = g.nb, live = g.live, h0 = g.h0;
    const int64_t row0 = (int64_t)(g.off + g.t0) * p.Hq + (int64_t)g.kvh * p.g;  // of the token's first head
    const bool whole = take == nb, direct = whole && p.row_ml == nullptr;
    const int64_t slot = (int64_t)(2 * blockIdx.x + (b0 == 0 ? 1 : 0)) * N;
    ok = warp_wait(&m->l_full, seg & 1, m, p) && ok;
    if (bar_red_or(bar, 128, !ok)) return;  // (and all have read the segment)
    if (q == 0) list();
    if (et < N) {
      const float sum = m->lcol[0][et], ref = m->lcol[1][et];
      m->lcol[1][et] = p.o_scale / sum;
      if (et < live) {
        const int64_t row = row0 + (int64_t)((h0 + et) / p.g) * p.Hq + (h0 + et) % p.g;
        const float2 ml = make_float2(ref, sum);
        if (!whole) p.slot_ml[slot + et] = ml;
        else if (!direct) p.row_ml[row] = ml;
        // (pos + i - b0 + nb - 1: the unit's last block)
        if (b0 == 0)
          p.info[row] = make_int4(blockIdx.x, whole ? (int)blockIdx.x : owner(s.pos + i + nb - 1, s.total, s.ctas), et, 0);
      }
    }
    ok = warp_wait(&m->o_full[seg & 1], (seg >> 1) & 1, m, p);
    tc_fence_after();
    if (bar_red_or(bar, 128, !ok)) return;
    const uint32_t tO = tmem + ((uint32_t)(q * 32) << 16) + C::kColO + (seg & 1) * N;
    int h = h0;
    int64_t row = row0 + h0;
#pragma unroll 1
    for (int w = 0; w < N / W; ++w) {
      if (w * W >= live) break;
      uint32_t x[W];
      tmem_ld<W>(tO + w * W, x);
      if (et >= D) continue;  // (a warp's lanes alike)
      if (whole) {  // rows of a token's heads
#pragma unroll
        for (int e = 0; e < W; ++e) {
          if (w * W + e < live) {
            const float o = __uint_as_float(x[e]);
            if (direct) p.out[row * D + et] = __float2bfloat16_rn(o * m->lcol[1][w * W + e]);
            else p.row_acc[row * D + et] = o;
          }
          ++row;
          if (++h == p.g) h = 0, row += p.Hq - p.g;
        }
      } else {
        float* to = p.slot_acc + (slot + w * W) * D + et;
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (w * W + e < live) to[e * D] = __uint_as_float(x[e]);
      }
    }
    tc_fence_before();
    mbar_arrive(&m->o_free[seg & 1]);
    mbar_arrive(&m->l_free);
    i += take;
  }
}

// ----------------------------------------------------------------- kernels

template <int D, int N, bool kFp8>
__global__ void __launch_bounds__(Cfg<D, N, kFp8>::kThreads, 1) verify_kernel(const Params p) {
  using C = Cfg<D, N, kFp8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sP = sQ + C::kQBufs * C::kQBytes;
  uint8_t* sKV = sP + 2 * C::kPBytes;
  Misc* m = reinterpret_cast<Misc*>(sKV + C::kStages * C::kTileBytes);
  const int tid = threadIdx.x, warp = tid >> 5;
  grid_dep_launch();  // what follows waits for this grid's end
  if (warp == 0) {
    find_start(p, &m->start);
  } else if (tid == 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m->q_full[i], C::kProdThreads);
      mbar_init(&m->q_empty[i], 1);
      mbar_init(&m->p_ready[i], 32 * C::kSoftWarps);
      mbar_init(&m->o_full[i], 1);
      mbar_init(&m->o_free[i], 128);
      mbar_init(&m->u_full[i], 1);
    }
    mbar_init(&m->l_full, 32 * C::kWgs);
    mbar_init(&m->l_free, 128);
    mbar_init(&m->drain, 1);
    for (int i = 0; i < C::kK; ++i) {
      mbar_init(&m->k_full[i], C::kProdThreads + 1);  // and the thread that writes k_last
      mbar_init(&m->k_done[i], 1);
    }
    for (int i = 0; i < C::kV; ++i) {
      mbar_init(&m->v_full[i], C::kProdThreads);
      mbar_init(&m->v_done[i], 1);
    }
    m->abort = 0;
    mbar_fence_init();
  } else if (warp == C::kMmaWarp) {
    tmem_alloc(&m->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Start s = m->start;
  const uint32_t tmem = m->tmem_base;
  if (blockIdx.x == 0 && tid == 0) p.status[1] = s.tokens;
  // Registers move between whole warpgroups, inside the roles' branches: the
  // compiler gives all code behind a change the smallest share that reaches it.
  static_assert(C::kProdWarp % 4 == 0 && (C::kMmaWarp + 1) % 4 == 0, "whole warpgroups");
  if (warp < C::kSoftWarps) {
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
    if (s.blocks > 0) softmax<D, N, kFp8>(p, s, m, tmem, smem_u32(sP));
  } else if (warp < C::kProdWarp) {
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kEpiRegs));
    if (s.blocks > 0) epilogue<D, N, kFp8>(p, s, m, tmem, tid - 32 * C::kSoftWarps);
  } else {
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kProdRegs));
    if (s.blocks > 0 && warp < C::kMmaWarp) {
      const int ptid = tid - 32 * C::kProdWarp;
      if constexpr (kFp8) produce_fp8<D, N>(p, s, m, smem_u32(sQ), smem_u32(sKV), ptid);
      else produce<D, N>(p, s, m, smem_u32(sQ), smem_u32(sKV), ptid);
    } else if (s.blocks > 0 && (tid & 31) == 0) {
      issue<D, N, kFp8>(p, s, m, tmem, smem_u32(sQ), smem_u32(sP), smem_u32(sKV));
      // MMAs issued before a wait gave up end before the CTA does
      umma_commit(&m->drain);
      mbar_wait_bounded(&m->drain, 0, nullptr, nullptr);
    }
  }
  __syncwarp();
  cp_async_wait_all();  // nothing of this CTA's shared memory is still being written
  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  grid_dep_wait();  // the combine after this grid also finds the one before it ended
}

// The states of a launch, as the combine reads them.
struct States {
  const int4* info;
  const float2* slot_ml;
  const float* slot_acc;
  const float2* row_ml;
  const float* row_acc;
  int32_t n;  // columns of a slot
};

struct CombineParams {
  States own, shared;  // shared.info == nullptr: no shared prefix
  __nv_bfloat16* out;
  const int* status;
  int32_t Hq;
  int64_t rows;
  float o_scale;
};

template <int D>
struct Merged {
  float m = -INFINITY, l = 0.f, acc[D / 32];
};

// A row's pieces w0, w0 + step, ... in one launch's states, 32 of them at a time.
template <int D>
SGL_DEV void merge(const States& st, int64_t row, const int4& at, int w0, int step, Merged<D>* r) {
  constexpr int E = D / 32, kBatch = 4;
  const int lane = threadIdx.x & 31;
  const int pieces = at.y - at.x + 1;
  const float2* whole_ml = pieces == 1 ? st.row_ml + row : nullptr;
  auto entry = [&](int i) -> int64_t { return (int64_t)(i == 0 ? 2 * at.x + 1 : 2 * (at.x + i)) * st.n + at.z; };
  for (int i0 = w0; i0 < pieces; i0 += 32 * step) {
    const int mine = i0 + lane * step;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (mine < pieces) ml = whole_ml ? *whole_ml : st.slot_ml[entry(mine)];
    if (!(ml.y > 0.f)) ml.x = -INFINITY;
    float top = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float now = fmaxf(r->m, top);
    if (now == -INFINITY) continue;  // no keys so far
    const float keep = ex2(r->m - now), w = ex2(ml.x - now);
    float sum = ml.y * w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    r->m = now;
    r->l = r->l * keep + sum;
#pragma unroll
    for (int e = 0; e < E; ++e) r->acc[e] *= keep;
    const int count = min(32, (pieces - i0 + step - 1) / step);
    for (int i = 0; i < count; i += kBatch) {
      float a[kBatch][E];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const float* p = (whole_ml ? st.row_acc + row * D : st.slot_acc + entry(i0 + (i + j) * step) * D) + lane;
#pragma unroll
        for (int e = 0; e < E; ++e) a[j][e] = i + j < count ? p[32 * e] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const float f = __shfl_sync(0xffffffffu, w, (i + j) & 31);
#pragma unroll
        for (int e = 0; e < E; ++e) r->acc[e] = fmaf(i + j < count ? f : 0.f, a[j][e], r->acc[e]);
      }
    }
  }
}

// Whether an entry of info names slots of its launch.  Where a wait gave up, rows' entries
// are what the workspace held before.
SGL_DEV bool named(const int4& at, int n) {
  return at.x >= 0 && at.x <= at.y && at.y < kMaxCtas && at.z >= 0 && at.z < n;
}

// A warp a (token, query head); kSplit: a block, whose warps share its pieces, for
// calls of few rows (one request of 16,384 tokens, 19 pieces a row: 29.9 -> 24.6 us).
template <int D, bool kSplit>
__global__ void __launch_bounds__(128) verify_combine_kernel(const CombineParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = kSplit ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + warp;
  grid_dep_wait();
  if (row >= p.rows || row >= (int64_t)p.status[1] * p.Hq) return;
  const int4 at = p.own.info[row];
  const int4 at_shared = p.shared.info != nullptr ? p.shared.info[row] : make_int4(0, 0, 0, 0);
  if (!named(at, p.own.n) || (p.shared.info != nullptr && !named(at_shared, p.shared.n))) return;
  if (at.x == at.y && p.own.row_ml == nullptr) return;  // written by the CTA that had its unit whole
  Merged<D> r;
#pragma unroll
  for (int e = 0; e < E; ++e) r.acc[e] = 0.f;
  const int w0 = kSplit ? warp : 0, step = kSplit ? 4 : 1;
  merge<D>(p.own, row, at, w0, step, &r);
  if (p.shared.info != nullptr) merge<D>(p.shared, row, at_shared, w0, step, &r);
  if constexpr (kSplit) {
    __shared__ float2 ml[4];
    __shared__ float acc[4][D];
    if (lane == 0) ml[warp] = make_float2(r.m, r.l);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[warp][lane + 32 * e] = r.acc[e];
    __syncthreads();
    float top = ml[0].x;
#pragma unroll
    for (int w = 1; w < 4; ++w) top = fmaxf(top, ml[w].x);
    float sum = 0.f, f[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) f[w] = ex2(ml[w].x - top), sum += f[w] * ml[w].y;
    const float inv = p.o_scale / sum;
    if (threadIdx.x < D) {
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) o = fmaf(f[w], acc[w][threadIdx.x], o);
      p.out[row * D + threadIdx.x] = __float2bfloat16_rn(o * inv);
    }
  } else {
    const float inv = p.o_scale / r.l;
#pragma unroll
    for (int e = 0; e < E; ++e) p.out[row * D + lane + 32 * e] = __float2bfloat16_rn(r.acc[e] * inv);
  }
}

template <int D>
cudaError_t launch_combine(const CombineParams& cp, cudaStream_t stream) {
  // up to 16 blocks an SM a row each
  if (cp.rows <= (int64_t)num_sms() * 16)
    return launch_dependent(verify_combine_kernel<D, true>, dim3((unsigned)cp.rows), dim3(128), 0, stream, cp);
  return launch_dependent(verify_combine_kernel<D, false>, dim3((unsigned)((cp.rows + 3) / 4)), dim3(128), 0, stream, cp);
}

// ----------------------------------------------------------------- host

// Columns of a tile for so many query rows a KV head.  (128 over an e4m3 pool left
// the softmax and the producers too few registers.)
int columns_for(int64_t rows, bool kv_fp8) {
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 || kv_fp8 ? 64 : 128;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace: 256 bytes (status, token count), then per launch the rows' info and
// the slots; with a shared prefix whole units leave row states too.
struct Layout {
  size_t bytes = 256;
  size_t at(size_t n) {
    const size_t o = bytes;
    bytes += round256(n);
    return o;
  }
};

struct Buffers {
  size_t info, slot_ml, slot_acc, row_ml, row_acc;
  Buffers(Layout* l, int64_t rows, int n, int D, bool with_rows) {
    info = l->at((size_t)rows * sizeof(int4));
    slot_ml = l->at((size_t)2 * kMaxCtas * n * sizeof(float2));
    slot_acc = l->at((size_t)2 * kMaxCtas * n * D * sizeof(float));
    row_ml = with_rows ? l->at((size_t)rows * sizeof(float2)) : 0;
    row_acc = with_rows ? l->at((size_t)rows * D * sizeof(float)) : 0;
  }
  void bind(char* base, Params* p) const {
    p->info = reinterpret_cast<int4*>(base + info);
    p->slot_ml = reinterpret_cast<float2*>(base + slot_ml);
    p->slot_acc = reinterpret_cast<float*>(base + slot_acc);
    p->row_ml = row_ml ? reinterpret_cast<float2*>(base + row_ml) : nullptr;
    p->row_acc = row_acc ? reinterpret_cast<float*>(base + row_acc) : nullptr;
  }
};

template <int D, int N, bool kFp8>
sgl_status launch_one(const Params& prm, bool dependent, cudaStream_t stream) {
  using C = Cfg<D, N, kFp8>;
  auto kern = verify_kernel<D, N, kFp8>;
  if (kernel_blocks_per_sm<verify_kernel<D, N, kFp8>>(C::kSmem, C::kThreads) < 0) return SGL_ERR_CUDA;
  if (C::kSplitRegs && !kernel_regs_at_least<verify_kernel<D, N, kFp8>>(C::kLaunchRegs)) return SGL_ERR_UNSUPPORTED;
  const int ctas = num_sms() < kMaxCtas ? num_sms() : kMaxCtas;
  if (dependent) {
    if (launch_dependent(kern, dim3(ctas), dim3(C::kThreads), C::kSmem, stream, prm) != cudaSuccess)
      return SGL_ERR_CUDA;
  } else {
    kern<<<ctas, C::kThreads, C::kSmem, stream>>>(prm);
  }
  return cudaGetLastError() == cudaSuccess ? SGL_OK : SGL_ERR_CUDA;
}

template <int D, bool kFp8>
sgl_status launch_n(const Params& prm, int n, bool dependent, cudaStream_t stream) {
  if (n == 16) return launch_one<D, 16, kFp8>(prm, dependent, stream);
  if (n == 32) return launch_one<D, 32, kFp8>(prm, dependent, stream);
  if constexpr (!kFp8) {
    if (n == 128) return launch_one<D, 128, kFp8>(prm, dependent, stream);
  }
  return launch_one<D, 64, kFp8>(prm, dependent, stream);
}

sgl_status launch_pass(const Params& prm, const VerifyArgs& a, int n, bool dependent, cudaStream_t stream) {
  if (a.head_dim == 128)
    return a.kv_fp8 ? launch_n<128, true>(prm, n, dependent, stream) : launch_n<128, false>(prm, n, dependent, stream);
  return a.kv_fp8 ? launch_n<64, true>(prm, n, dependent, stream) : launch_n<64, false>(prm, n, dependent, stream);
}

States states_of(const Params& p, int n) {
  return States{p.info, p.slot_ml, p.slot_acc, p.row_ml, p.row_acc, n};
}

}  // namespace
}  // namespace vfy

using namespace vfy;

size_t verify_workspace_bytes(int32_t total, int32_t max_draft, int32_t shared_len, int32_t Hq, int32_t Hkv, int32_t D) {
  Layout l;
  if (total <= 0 || max_draft <= 0 || Hkv <= 0 || Hq < Hkv) return l.bytes;
  const int g = Hq / Hkv;
  const int64_t rows = (int64_t)total * Hq;
  // (sized as over a bf16 pool: one size for both)
  Buffers own(&l, rows, columns_for((int64_t)max_draft * g, false), D, shared_len > 0);
  if (shared_len > 0) Buffers shared(&l, rows, columns_for((int64_t)total * g, false), D, true);
  return l.bytes;
}

sgl_status launch_verify(const VerifyArgs& a, cudaStream_t stream) {
  const int g = a.num_q_heads / a.num_kv_heads;
  Params prm = {};
  prm.q = static_cast<const __nv_bfloat16*>(a.q);
  prm.pool_k = a.pool_k;
  prm.pool_v = a.pool_v;
  prm.rtt = a.req_to_token;
  prm.rtt_stride = a.rtt_stride;
  prm.req_pool_idx = a.req_pool_idx;
  prm.prefix_lens = a.prefix_lens;
  prm.draft_lens = a.draft_lens;
  prm.parents = a.parents;
  prm.out = static_cast<__nv_bfloat16*>(a.out);
  prm.Hq = a.num_q_heads;
  prm.Hkv = a.num_kv_heads;
  prm.g = g;
  prm.batch = a.batch;
  prm.total = a.total_draft;
  prm.max_draft = a.max_draft;
  prm.max_prefix = a.max_prefix;
  prm.shared = a.shared_len;
  prm.scale_log2 = a.sm_scale * 1.4426950408889634f * (a.kv_fp8 ? a.k_scale : 1.f);
  prm.o_scale = a.kv_fp8 ? a.v_scale : 1.f;
  prm.status = static_cast<int*>(a.workspace);
  prm.wait_ns = device_wait_limit_ns();
  const int64_t rows = (int64_t)a.total_draft * a.num_q_heads;
  const int n = columns_for((int64_t)a.max_draft * g, a.kv_fp8), ns = columns_for((int64_t)a.total_draft * g, a.kv_fp8);
  const bool shared = a.shared_len > 0;
  Layout l;
  char* base = static_cast<char*>(a.workspace);
  Buffers(&l, rows, n, a.head_dim, shared).bind(base, &prm);
  prm.cols = n;
  CombineParams cp = {};
  cp.own = states_of(prm, n);
  if (shared) {
    Params sp = prm;
    Buffers(&l, rows, ns, a.head_dim, true).bind(base, &sp);
    sp.shared_pass = true;
    sp.cols = ns;
    cp.shared = states_of(sp, ns);
    const sgl_status st = launch_pass(sp, a, ns, false, stream);
    if (st != SGL_OK) return st;
  }
  const sgl_status st = launch_pass(prm, a, n, shared, stream);
  if (st != SGL_OK) return st;
  cp.out = prm.out;
  cp.status = prm.status;
  cp.Hq = prm.Hq;
  cp.rows = rows;
  cp.o_scale = prm.o_scale;
  const cudaError_t e = a.head_dim == 128 ? launch_combine<128>(cp, stream) : launch_combine<64>(cp, stream);
  return e == cudaSuccess ? SGL_OK : SGL_ERR_CUDA;
}

}  // namespace sgl
