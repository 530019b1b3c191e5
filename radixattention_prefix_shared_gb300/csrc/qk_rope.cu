// Head norms, rotary positions and the KV store in one pass.
//
// For every token t and head row x of D values: r = 1 / sqrt(mean(x^2) + eps)
// (1 without a norm), y_d = x_d r w_d, then the pairs (a, b) of the first
// rot_dim values -- (i, i + rot_dim / 2) or, interleaved, (2i, 2i + 1) -- turn
// by the angle positions[axis(i), t] * inv_freq[i]:
//   a' = a cos - b sin,   b' = b cos + a sin.
// Q rows go to q_out, K rows to pool_k[slots[t]], V rows unchanged to
// pool_v[slots[t]] (e4m3 pools: value / scale as a code).  All of it is fp32
// from the bf16 inputs to the one rounding of what is stored.
//
// A lane holds both values of its pairs, so a row needs no exchange but its
// norm's sum: with the products of weights and cosines or sines in registers
// (they depend on the token and the lane, not on the head) it costs four
// multiply-adds a pair and the scaling by r, on packed pairs of floats.
//
// The angle is kept exact modulo a turn: inv_freq / 2 pi as a 64-bit fixed
// point fraction of a turn (turn_fraction), multiplied by the position in
// wrapping 64-bit integers.  For frequencies up to 1 the fraction is good to
// 2^-64 turns, the angle at position 2^31 to 2^-33; a float32 product would be
// off by a twentieth of a radian at 2^20 already.  (In float64 the fraction
// took each warp some 20 instructions of a pipe that needs 16 cycles each.)
//
// Bound by HBM in long prefills: 16,384 tokens of 16 query and 8 KV heads of
// 128: 46.4 us, 5.8 TB/s (0.85 of the measured copy rate); 8,191 tokens of 32
// and 8 into an e4m3 pool, without norms, 32.5 us, 5.7 TB/s.  64 tokens take 3.2 us.
#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.h"

namespace sgl {

namespace {

// Measured (before rows whose squares overflow were looked for), 16,384 tokens
// (and 8,191 into an e4m3 pool): 3 warps x 6 blocks 45.4 us (32.6), 2 x 9 46.1
// (32.5), 1 x 18 46.1 (32.8), 4 x 4 47.3 (35.4), 8 x 2 47.4
// (35.9), 4 x 5 51.8 (37.0; 13,000 tokens 38.2 with 3 x 6, 40.0 with 4 x 4, and
// 4,500 16.6 with either: the rounds' ends differ, 18 warps an SM are as good
// as any).  Batches of 2, 6, 8 at 8 x 2 blocks: 58.5, 49.5, 52.4 against 47.6.
// K and V rows in one batch, half each: 47.4 (33.6), though 9.6 us instead of
// 10.7 with 4 KV heads of 64, whose batches of one section are mostly empty.
constexpr int kRopeWarps = 3;
constexpr int kRopeBatch = 4;   // row groups a warp loads at a time
constexpr int kRopeBlocks = 6;  // resident blocks an SM

struct RopeParams {
  const __nv_bfloat16* src[3];  // q, k, v
  int64_t stride[3];
  const __nv_bfloat16* weight[2];  // q, k (null: no norm)
  float eps;
  const int32_t* positions;
  int32_t n_axes;
  const float* inv_freq;
  const int32_t* freq_axis;
  int32_t rot_dim, interleaved;
  const int32_t* slots;
  int32_t n;
  __nv_bfloat16* q_out;
  uint8_t* pool[2];  // k, v
  int64_t pool_size;
  int32_t heads[2];  // query, KV
  float scale[2];    // k, v
  float rcp[2];      // 1 / scale, or 0 (quotient)
};

// (not .nc: q_out may be q)
SGL_DEV uint4 ld_row16(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
SGL_DEV uint2 ld_row8(const __nv_bfloat16* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
// 4 bf16 -> two packed pairs of floats
SGL_DEV void unpack4(uint32_t a, uint32_t b, float2 (&f)[2]) {
  f[0] = make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
  f[1] = make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u));
}
SGL_DEV float2 fmul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
SGL_DEV float2 dup(float x) { return make_float2(x, x); }

// y / s in IEEE float32.  With rcp the rounded 1 / s, q = y rcp is off by a few
// units in the last place, y - q s is exact in a fused multiply-add, and q plus
// that times rcp is the rounded quotient (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990).  It takes s and rcp
// far from the ends of the range (rcp = 0: they are not, and the quotient is
// divided out) and a q that does not overflow; from 1024 on the code saturates
// whatever q's last bits.  The divisions took 4 of 37 us on 8,191 tokens of 32
// query and 8 KV heads.
SGL_DEV float quotient(float y, float s, float rcp) {
  if (rcp == 0.f) return __fdiv_rn(y, s);
  const float q = y * rcp;
  const float d = fmaf(fmaf(-q, s, y), rcp, q);
  return copysignf(fabsf(q) < 1024.f ? d : q, y);  // (d loses the sign of a zero)
}
SGL_DEV uint32_t e4m3x4(const float2 (&y)[2], float s, float rcp) {
  const float2 a = make_float2(quotient(y[0].x, s, rcp), quotient(y[0].y, s, rcp));
  const float2 b = make_float2(quotient(y[1].x, s, rcp), quotient(y[1].y, s, rcp));
  return (uint32_t)__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
         ((uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16);
}

// f / 2 pi modulo 1, in units of 2^-64: f = m 2^e with m an integer of 24
// bits, and m times the first 64 bits of 1 / 2 pi, 2^66 / 2 pi, shifted to the
// place of 2^-64.
SGL_DEV uint64_t turn_fraction(float f) {
  constexpr uint64_t kInv2Pi = 0xa2f9836e4e441529ull;  // 2^66 / 2 pi
  const uint32_t bits = __float_as_uint(f);
  const int ex = (bits >> 23) & 0xff;
  const uint64_t m = (bits & 0x7fffffu) | (ex > 0 ? 0x800000u : 0u);
  const int sh = max(ex, 1) - 150 - 2;
  const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  uint64_t t;
  if (sh >= 0)
    t = sh < 64 ? lo << sh : 0;
  else if (sh > -64)
    t = (lo >> -sh) | (hi << (64 + sh));
  else
    t = sh > -128 ? hi >> (-sh - 64) : 0;
  return (bits >> 31) ? 0 - t : t;
}

// Sum over the D / 8 lanes of a row of the squares of its 8 values.
template <int D>
SGL_DEV float row_squares(const float2 (&y0)[2], const float2 (&y1)[2]) {
  const float2 q = ffma2(y1[1], y1[1], ffma2(y1[0], y1[0], ffma2(y0[1], y0[1], fmul2(y0[0], y0[0]))));
  float s = q.x + q.y;
#pragma unroll
  for (int o = 1; o < D / 8; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// What turns a lane's values y: y' = y C + other S, other being the pair's other
// value; the head weights w are in it (null: none).
template <bool kInterleaved>
struct Turn {
  float2 C0[2], C1[2], S0[2], S1[2];
  bool rotated;
  SGL_DEV Turn(const __nv_bfloat16* w, const float2* pairs, bool turned, int o0, int o1) : rotated(turned) {
    float2 w0[2] = {dup(1.f), dup(1.f)}, w1[2] = {dup(1.f), dup(1.f)};
    if (w != nullptr) {
      const uint2 a = *reinterpret_cast<const uint2*>(w + o0), c = *reinterpret_cast<const uint2*>(w + o1);
      unpack4(a.x, a.y, w0);
      unpack4(c.x, c.y, w1);
    }
    float2 v[4] = {make_float2(1.f, 0.f), make_float2(1.f, 0.f), make_float2(1.f, 0.f), make_float2(1.f, 0.f)};
    if (rotated) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = pairs[e];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (kInterleaved) {  // pair = the two floats of a packed pair
        C0[j] = fmul2(w0[j], dup(v[j].x));
        S0[j] = make_float2(-w0[j].y * v[j].y, w0[j].x * v[j].y);
        C1[j] = fmul2(w1[j], dup(v[2 + j].x));
        S1[j] = make_float2(-w1[j].y * v[2 + j].y, w1[j].x * v[2 + j].y);
      } else {  // pair = the same place of the two runs
        const float2 c = make_float2(v[2 * j].x, v[2 * j + 1].x), sn = make_float2(v[2 * j].y, v[2 * j + 1].y);
        C0[j] = fmul2(w0[j], c);
        C1[j] = fmul2(w1[j], c);
        S1[j] = fmul2(w0[j], sn);
        S0[j] = fmul2(w1[j], make_float2(-sn.x, -sn.y));
      }
    }
  }
  // the values turned, times r
  SGL_DEV void operator()(const float2 (&y0)[2], const float2 (&y1)[2], float r, float2 (&z0)[2], float2 (&z1)[2]) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      z0[j] = fmul2(y0[j], C0[j]);
      z1[j] = fmul2(y1[j], C1[j]);
      if (rotated) {  // (not + 0 * other: rows that do not turn keep their infinities)
        z0[j] = ffma2(kInterleaved ? make_float2(y0[j].y, y0[j].x) : y1[j], S0[j], z0[j]);
        z1[j] = ffma2(kInterleaved ? make_float2(y1[j].y, y1[j].x) : y0[j], S1[j], z1[j]);
      }
      z0[j] = fmul2(z0[j], dup(r));
      z1[j] = fmul2(z1[j], dup(r));
    }
  }
};

// A lane's finished values of row h of token tok (slot `at`): Q (sec 0) to
// q_out, K to its pool.
template <int D, bool kFp8, bool kInterleaved>
SGL_DEV void store_row(const RopeParams& p, int sec, int32_t tok, int64_t at, int h, int o0, int o1,
                       const float2 (&z0)[2], const float2 (&z1)[2]) {
  if (kFp8 && sec == 1) {
    uint8_t* dst = p.pool[0] + (at * p.heads[1] + h) * D;
    const uint32_t lo = e4m3x4(z0, p.scale[0], p.rcp[0]), hi = e4m3x4(z1, p.scale[0], p.rcp[0]);
    if constexpr (kInterleaved) {
      *reinterpret_cast<uint2*>(dst + o0) = make_uint2(lo, hi);
    } else {
      *reinterpret_cast<uint32_t*>(dst + o0) = lo;
      *reinterpret_cast<uint32_t*>(dst + o1) = hi;
    }
  } else {
    __nv_bfloat16* dst = sec == 0 ? p.q_out + ((int64_t)tok * p.heads[0] + h) * D
                                  : reinterpret_cast<__nv_bfloat16*>(p.pool[0]) + (at * p.heads[1] + h) * D;
    const uint2 lo = make_uint2(pack_bf16x2(z0[0].x, z0[0].y), pack_bf16x2(z0[1].x, z0[1].y));
    const uint2 hi = make_uint2(pack_bf16x2(z1[0].x, z1[0].y), pack_bf16x2(z1[1].x, z1[1].y));
    if constexpr (kInterleaved) {
      *reinterpret_cast<uint4*>(dst + o0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    } else {
      *reinterpret_cast<uint2*>(dst + o0) = lo;
      *reinterpret_cast<uint2*>(dst + o1) = hi;
    }
  }
}

// A row whose squares sum up to kFarSquares or more (an RMS from 2^57 on: none in
// practice, and past fp32 from 2^60 on) is left out; a warp that met one goes over
// its rows again at the end and finishes those from values at 2^-70 of their
// size, with eps at 2^-140 of its: r comes out at 2^70 of its size, and neither
// the squares (a bf16 is below 2^128, so D of them are below 2^123) nor a turned
// pair's sum overflow.  Leaving them out is a comparison a row: 16,384 tokens 47.9
// -> 48.3 us, 8,191 with norms into an e4m3 pool 39.8 -> 40.1 (a vote a row in
// the loop 48.4 and 41.1; a vote a batch and its rows again, 51 to 56 and 50 to
// 52).  Calls without norms (kNorm false) have no use for it: 33.4 us for 8,191
// tokens, 34.8 with it.
constexpr float kFarSquares = 0x1p121f, kFarScale = 0x1p-70f;

// A warp works on batches of kRopeBatch row groups, a group being the 32 / (D /
// 8) rows (heads of one token) that its lanes hold, 8 values each: lane i < rot
// / 8 of a row holds pairs 4 i .. 4 i + 3 (8 consecutive values when
// interleaved, else two runs of 4), the others 8 consecutive values that do
// not turn.
// kNorm: some rows have a weight.
// A token's batches are those of its Q rows, its K rows and its V rows in
// turn; block y takes an even share of them.  The next batch's rows, and the
// next token's slot and positions, are loaded before the current batch is
// worked on.
template <int D, bool kFp8, bool kInterleaved, bool kNorm>
__global__ void __launch_bounds__(kRopeWarps * 32, kRopeBlocks) qk_norm_rope_store_kernel(RopeParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kF = D / 64;
  __shared__ float2 s_turn[kRopeWarps][D / 2];  // (cos, sin) of the warp's token
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int li = lane % kLanes, sub = lane / kLanes;
  float2* turn = s_turn[warp];

  constexpr int kBatchRows = kRows * kRopeBatch;
  const int nq = (p.heads[0] + kBatchRows - 1) / kBatchRows, nk = (p.heads[1] + kBatchRows - 1) / kBatchRows;
  const int b0 = (nq + 2 * nk) * blockIdx.y / gridDim.y, b1 = (nq + 2 * nk) * (blockIdx.y + 1) / gridDim.y;
  const int nf = p.rot_dim / 2;
  const bool turns = b0 < nq + nk && nf > 0;  // this block has rows to turn

  // this lane's values: o0 .. o0 + 3 and o1 .. o1 + 3
  const bool rotated = 8 * li < p.rot_dim;
  const int o0 = rotated && !kInterleaved ? 4 * li : 8 * li;
  const int o1 = rotated && !kInterleaved ? 4 * li + nf : 8 * li + 4;

  int32_t t = blockIdx.x * kRopeWarps + warp;
  const int32_t stride = gridDim.x * kRopeWarps;
  if (t >= p.n) return;
  int b = b0;
  uint4 raw[kRopeBatch] = {};
  int32_t slot, pos[kF];
  auto section = [&](int bb) { return bb < nq ? 0 : (bb < nq + nk ? 1 : 2); };
  auto load_rows = [&](int32_t tt, int bb) {
    const int sec = section(bb);
    const int h0 = (bb - (sec == 0 ? 0 : (sec == 1 ? nq : nq + nk))) * kBatchRows + sub;
    const __nv_bfloat16* src = p.src[sec] + tt * p.stride[sec] + h0 * D;
    const int n_heads = p.heads[sec > 0];
    if (kInterleaved || sec == 2) {
      src += 8 * li;
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u)
        if (h0 + u * kRows < n_heads) raw[u] = ld_row16(src + u * kRows * D);
    } else {
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u)
        if (h0 + u * kRows < n_heads) {
          const uint2 lo = ld_row8(src + u * kRows * D + o0), hi = ld_row8(src + u * kRows * D + o1);
          raw[u] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
    }
  };
  const int32_t* fpos[kF];
  auto load_token = [&](int32_t tt) {
    slot = p.slots[tt];
    if (turns) {
#pragma unroll
      for (int i = 0; i < kF; ++i)
        if (lane + 32 * i < nf) pos[i] = fpos[i][tt];
    }
  };
  uint64_t freq[kF];
  auto fill_turns = [&] {  // of the token whose positions were loaded
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kF; ++i) {
      const int f = lane + 32 * i;
      if (f < nf) {
        const uint64_t a = (uint64_t)(int64_t)pos[i] * freq[i];
        float sn, cs;
        sincospif((float)(int32_t)(a >> 32) * 0x1p-31f, &sn, &cs);
        turn[f] = make_float2(cs, sn);
      }
    }
    __syncwarp();
  };
  load_rows(t, b);
#pragma unroll
  for (int i = 0; i < kF; ++i) {
    const int f = lane + 32 * i;
    freq[i] = 0;
    fpos[i] = p.positions;
    pos[i] = 0;
    if (turns && f < nf) {
      freq[i] = turn_fraction(p.inv_freq[f]);
      if (p.freq_axis != nullptr) fpos[i] += (int64_t)min(max(p.freq_axis[f], 0), p.n_axes - 1) * p.n;
    }
  }
  load_token(t);
  bool fresh = true;  // the token's first batch here
  bool far = false;   // a row was left out

  while (true) {
    const int sec = section(b);
    const int h0 = (b - (sec == 0 ? 0 : (sec == 1 ? nq : nq + nk))) * kBatchRows + sub;
    const int n_heads = p.heads[sec > 0];
    const int64_t at = slot;
    const bool live = at >= 0 && at < p.pool_size;  // else a padding token
    const int32_t tok = t;
    uint4 cur[kRopeBatch];
#pragma unroll
    for (int u = 0; u < kRopeBatch; ++u) cur[u] = raw[u];
    if (fresh && turns) fill_turns();
    // on to the next batch
    fresh = ++b == b1;
    if (fresh) {
      b = b0;
      t += stride;
    }
    const bool more = t < p.n;
    if (more) {
      load_rows(t, b);
      if (fresh) load_token(t);
    }
    if (live) {
      if (sec < 2) {
        const __nv_bfloat16* w = kNorm ? p.weight[sec] : nullptr;
        const Turn<kInterleaved> turned(w, turn + 4 * li, rotated, o0, o1);
#pragma unroll
        for (int u = 0; u < kRopeBatch; ++u) {
          const int h = h0 + u * kRows;
          if (h - sub >= n_heads) break;
          float2 y0[2], y1[2], z0[2], z1[2];
          unpack4(cur[u].x, cur[u].y, y0);
          unpack4(cur[u].z, cur[u].w, y1);
          float r = 1.f;
          bool stored = h < n_heads;
          if (w != nullptr) {
            const float s = row_squares<D>(y0, y1);
            far = far || !(s < kFarSquares);
            stored = stored && s < kFarSquares;
            r = rsqrtf(s * (1.f / D) + p.eps);
          }
          turned(y0, y1, r, z0, z1);
          if (stored) store_row<D, kFp8, kInterleaved>(p, sec, tok, at, h, o0, o1, z0, z1);
        }
      } else {
#pragma unroll
        for (int u = 0; u < kRopeBatch; ++u) {
          const int h = h0 + u * kRows;
          if (h >= n_heads) break;
          if constexpr (kFp8) {
            float2 y0[2], y1[2];
            unpack4(cur[u].x, cur[u].y, y0);
            unpack4(cur[u].z, cur[u].w, y1);
            *reinterpret_cast<uint2*>(p.pool[1] + (at * p.heads[1] + h) * D + 8 * li) =
                make_uint2(e4m3x4(y0, p.scale[1], p.rcp[1]), e4m3x4(y1, p.scale[1], p.rcp[1]));
          } else {
            *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.pool[1]) + (at * p.heads[1] + h) * D +
                                      8 * li) = cur[u];
          }
        }
      }
    }
    if (!more) break;
  }
  if constexpr (kNorm) {
    if (!__any_sync(0xffffffffu, far)) return;
#pragma unroll 1
    for (t = blockIdx.x * kRopeWarps + warp; t < p.n; t += stride) {
      load_token(t);
      if (slot < 0 || slot >= p.pool_size) continue;
      if (turns) fill_turns();
#pragma unroll 1
      for (int bb = b0; bb < b1 && bb < nq + nk; ++bb) {
        const int sec = section(bb), n_heads = p.heads[sec];
        const __nv_bfloat16* w = p.weight[sec];
        if (w == nullptr) continue;
        const int h0 = (bb - (sec == 0 ? 0 : nq)) * kBatchRows + sub;
#pragma unroll 1
        for (int h = h0; h < h0 + kBatchRows && h - sub < n_heads; h += kRows) {
          float2 y0[2] = {}, y1[2] = {}, z0[2], z1[2];
          if (h < n_heads) {
            const __nv_bfloat16* src = p.src[sec] + t * p.stride[sec] + h * D;
            const uint2 lo = ld_row8(src + o0), hi = ld_row8(src + o1);
            unpack4(lo.x, lo.y, y0);
            unpack4(hi.x, hi.y, y1);
          }
          const bool mine = !(row_squares<D>(y0, y1) < kFarSquares);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            y0[j] = fmul2(y0[j], dup(kFarScale));
            y1[j] = fmul2(y1[j], dup(kFarScale));
          }
          const float r = rsqrtf(row_squares<D>(y0, y1) * (1.f / D) + p.eps * kFarScale * kFarScale);
          Turn<kInterleaved>(w, turn + 4 * li, rotated, o0, o1)(y0, y1, r, z0, z1);
          if (mine) store_row<D, kFp8, kInterleaved>(p, sec, t, slot, h, o0, o1, z0, z1);
        }
      }
    }
  }
}

template <int D, bool kFp8, bool kInterleaved, bool kNorm>
sgl_status run(const RopeParams& p, cudaStream_t stream) {
  constexpr int kThreads = kRopeWarps * 32, kBatchRows = 32 / (D / 8) * kRopeBatch;
  const int per_sm = kernel_blocks_per_sm<qk_norm_rope_store_kernel<D, kFp8, kInterleaved, kNorm>>(0, kThreads);
  if (per_sm < 0) return SGL_ERR_CUDA;
  // a token's batches are dealt to several blocks while there are fewer
  // tokens than the part has warps for (and no further: 10,000 tokens dealt to
  // three warps each, for a fuller last round, took 46.7 us instead of 33.2)
  const int batches = (p.heads[0] + kBatchRows - 1) / kBatchRows + 2 * ((p.heads[1] + kBatchRows - 1) / kBatchRows);
  const int64_t resident = (int64_t)num_sms() * per_sm;
  int64_t parts = (resident * kRopeWarps + p.n - 1) / p.n;
  if (parts > batches) parts = batches;
  int64_t blocks = ((int64_t)p.n + kRopeWarps - 1) / kRopeWarps;
  const int64_t cap = (resident + parts - 1) / parts;
  if (blocks > cap) blocks = cap;
  qk_norm_rope_store_kernel<D, kFp8, kInterleaved, kNorm>
      <<<dim3((unsigned)blocks, (unsigned)parts), kThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SGL_OK : SGL_ERR_CUDA;
}

template <int D, bool kFp8, bool kInterleaved>
sgl_status run_n(const RopeParams& p, cudaStream_t stream) {
  return p.weight[0] != nullptr || p.weight[1] != nullptr ? run<D, kFp8, kInterleaved, true>(p, stream)
                                                          : run<D, kFp8, kInterleaved, false>(p, stream);
}

template <int D>
sgl_status run_d(const RopeParams& p, bool kv_fp8, cudaStream_t stream) {
  if (kv_fp8) return p.interleaved ? run_n<D, true, true>(p, stream) : run_n<D, true, false>(p, stream);
  return p.interleaved ? run_n<D, false, true>(p, stream) : run_n<D, false, false>(p, stream);
}

}  // namespace

sgl_status launch_qk_norm_rope_store(const RopeArgs& a, cudaStream_t stream) {
  if (a.n == 0) return SGL_OK;
  RopeParams p = {};
  p.src[0] = static_cast<const __nv_bfloat16*>(a.q);
  p.src[1] = static_cast<const __nv_bfloat16*>(a.k);
  p.src[2] = static_cast<const __nv_bfloat16*>(a.v);
  p.stride[0] = a.q_stride;
  p.stride[1] = a.k_stride;
  p.stride[2] = a.v_stride;
  p.weight[0] = static_cast<const __nv_bfloat16*>(a.q_weight);
  p.weight[1] = static_cast<const __nv_bfloat16*>(a.k_weight);
  p.eps = a.eps;
  p.positions = a.positions;
  p.n_axes = a.n_axes;
  p.inv_freq = a.inv_freq;
  p.freq_axis = a.freq_axis;
  p.rot_dim = a.rot_dim;
  p.interleaved = a.interleaved;
  p.slots = a.slots;
  p.n = a.n;
  p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
  p.pool[0] = static_cast<uint8_t*>(a.pool_k);
  p.pool[1] = static_cast<uint8_t*>(a.pool_v);
  p.pool_size = a.pool_size;
  p.heads[0] = a.num_q_heads;
  p.heads[1] = a.num_kv_heads;
  p.scale[0] = a.k_scale;
  p.scale[1] = a.v_scale;
  for (int i = 0; i < 2; ++i) p.rcp[i] = p.scale[i] >= 0x1p-60f && p.scale[i] <= 0x1p60f ? 1.f / p.scale[i] : 0.f;
  if (a.head_dim == 128) return run_d<128>(p, a.kv_fp8, stream);
  if (a.head_dim == 64) return run_d<64>(p, a.kv_fp8, stream);
  return SGL_ERR_UNSUPPORTED;
}

}  // namespace sgl
