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
// Written out per value, y' = r (x A + x' B) with x' the pair's other value,
// A = w cos and B = -+ w' sin: A and B depend on the token and the lane only,
// so the rows of a token share them and a row costs two multiply-adds a value
// besides its norm.
//
// The angle is kept exact modulo a turn: inv_freq / 2 pi as a 64-bit fixed
// point fraction of a turn, multiplied by the position in wrapping 64-bit
// integers.  The frequency's rounding (2^-53 of it, once a warp) grows with
// the position to 2^-33 turns at position 2^20; a float32 product would be off
// by a twentieth of a radian there.
#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.h"

namespace sgl {

namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeBatch = 4;  // row groups a warp loads before it works on them

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
};

// (not .nc: q_out may be q)
SGL_DEV uint4 ld_row(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

SGL_DEV uint32_t e4m3x2(float a, float b, float scale) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(a, scale), __fdiv_rn(b, scale)), __NV_SATFINITE,
                                            __NV_E4M3);
}

// D / 8 lanes hold a row, 8 consecutive values each: a warp works on a group
// of 32 / (D / 8) rows (heads of one token) at a time.
template <int D, bool kFp8>
__global__ void __launch_bounds__(kRopeWarps * 32) qk_norm_rope_store_kernel(RopeParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  __shared__ float2 s_turn[kRopeWarps][D / 2];  // (cos, sin) of the warp's token
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int li = lane % kLanes, sub = lane / kLanes;
  float2* turn = s_turn[warp];

  // this lane's share of the frequencies, in turns a position
  const int nf = p.rot_dim / 2;
  uint64_t freq[D / 64];
  const int32_t* fpos[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const int f = lane + 32 * i;
    freq[i] = 0;
    fpos[i] = p.positions;
    if (f < nf) {
      const double t = (double)p.inv_freq[f] * 0.15915494309189533577;  // 1 / 2 pi
      freq[i] = (uint64_t)((t - floor(t)) * 18446744073709551616.0);
      if (p.freq_axis != nullptr) fpos[i] += (int64_t)min(max(p.freq_axis[f], 0), p.n_axes - 1) * p.n;
    }
  }
  // this lane's values 8 li .. 8 li + 7: the lane holding their partners, the
  // first frequency and the sign of the sine
  const bool rotated = 8 * li < p.rot_dim;
  const int half = p.rot_dim / 16;
  const bool low = li < half;
  const int plane = p.interleaved || !rotated ? li : (low ? li + half : li - half);

  // this part's row groups of the list q, k, v
  const int gq = (p.heads[0] + kRows - 1) / kRows, gk = (p.heads[1] + kRows - 1) / kRows;
  const int total = gq + 2 * gk, part = blockIdx.y, parts = gridDim.y;
  const int g0 = (int)((int64_t)total * part / parts), g1 = (int)((int64_t)total * (part + 1) / parts);

  for (int64_t t = (int64_t)blockIdx.x * kRopeWarps + warp; t < p.n; t += (int64_t)gridDim.x * kRopeWarps) {
    const int64_t slot = p.slots[t];
    if (slot < 0 || slot >= p.pool_size) continue;  // a padding token

    float c[8], s[8];
    if (g0 < gq + gk && nf > 0) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const int f = lane + 32 * i;
        if (f < nf) {
          const uint64_t a = (uint64_t)(int64_t)fpos[i][t] * freq[i];
          float sn, cs;
          sincospif((float)(int32_t)(a >> 32) * 0x1p-31f, &sn, &cs);
          turn[f] = make_float2(cs, sn);
        }
      }
      __syncwarp();
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float2 v = make_float2(1.f, 0.f);
      if (rotated) v = turn[p.interleaved ? 4 * li + e / 2 : (low ? 8 * li + e : 8 * (li - half) + e)];
      c[e] = v.x;
      s[e] = (p.interleaved ? (e & 1) == 0 : low) ? -v.y : v.y;
    }
    int first = 0;  // first group of the section
#pragma unroll
    for (int sec = 0; sec < 3; ++sec) {
      const int n_groups = sec == 0 ? gq : gk, n_heads = p.heads[sec > 0];
      const int a0 = max(g0 - first, 0), a1 = min(g1 - first, n_groups);
      first += n_groups;
      if (a0 >= a1) continue;
      float A[8], B[8];
      bool norm = false;
      if (sec < 2) {
        float w[8], wp[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = wp[e] = 1.f;
        norm = p.weight[sec & 1] != nullptr;
        if (norm) {
          bf16x8_to_f32(*reinterpret_cast<const uint4*>(p.weight[sec & 1] + 8 * li), w);
          bf16x8_to_f32(*reinterpret_cast<const uint4*>(p.weight[sec & 1] + 8 * plane), wp);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          A[e] = w[e] * c[e];
          B[e] = (p.interleaved ? w[e ^ 1] : wp[e]) * s[e];
        }
      }
      const __nv_bfloat16* src = p.src[sec] + t * p.stride[sec] + 8 * li;
      for (int g = a0; g < a1; g += kRopeBatch) {
        uint4 raw[kRopeBatch];
#pragma unroll
        for (int u = 0; u < kRopeBatch; ++u) {
          const int h = (g + u) * kRows + sub;
          raw[u] = make_uint4(0u, 0u, 0u, 0u);
          if (g + u < a1 && h < n_heads) raw[u] = ld_row(src + (int64_t)h * D);
        }
#pragma unroll
        for (int u = 0; u < kRopeBatch; ++u) {
          if (g + u >= a1) break;
          const int h = (g + u) * kRows + sub;
          uint4 out = raw[u];
          float y[8];
          if (sec < 2 || kFp8) bf16x8_to_f32(raw[u], y);
          if (sec < 2) {
            float r = 1.f;
            if (norm) {
              float q2 = 0.f;
#pragma unroll
              for (int e = 0; e < 8; ++e) q2 = fmaf(y[e], y[e], q2);
#pragma unroll
              for (int o = 1; o < kLanes; o <<= 1) q2 += __shfl_xor_sync(0xffffffffu, q2, o);
              r = rsqrtf(q2 * (1.f / D) + p.eps);
            }
            float x[8];
            if (p.interleaved) {
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = y[e ^ 1];
            } else {
              uint4 other;
              other.x = __shfl_sync(0xffffffffu, raw[u].x, sub * kLanes + plane);
              other.y = __shfl_sync(0xffffffffu, raw[u].y, sub * kLanes + plane);
              other.z = __shfl_sync(0xffffffffu, raw[u].z, sub * kLanes + plane);
              other.w = __shfl_sync(0xffffffffu, raw[u].w, sub * kLanes + plane);
              bf16x8_to_f32(other, x);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = r * fmaf(y[e], A[e], rotated ? x[e] * B[e] : 0.f);
          }
          if (h >= n_heads) continue;
          if (kFp8 && sec > 0) {
            const float sc = p.scale[sec - 1];
            const uint2 code = make_uint2(e4m3x2(y[0], y[1], sc) | (e4m3x2(y[2], y[3], sc) << 16),
                                          e4m3x2(y[4], y[5], sc) | (e4m3x2(y[6], y[7], sc) << 16));
            *reinterpret_cast<uint2*>(p.pool[sec - 1] + (slot * p.heads[1] + h) * D + 8 * li) = code;
          } else {
            if (sec < 2)
              out = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                               pack_bf16x2(y[6], y[7]));
            __nv_bfloat16* dst = sec == 0 ? p.q_out + (t * p.heads[0] + h) * D
                                          : reinterpret_cast<__nv_bfloat16*>(p.pool[sec - 1]) +
                                                (slot * p.heads[1] + h) * D;
            *reinterpret_cast<uint4*>(dst + 8 * li) = out;
          }
        }
      }
    }
  }
}

template <int D, bool kFp8>
sgl_status run(RopeParams p, cudaStream_t stream) {
  constexpr int kThreads = kRopeWarps * 32;
  const int per_sm = kernel_blocks_per_sm<qk_norm_rope_store_kernel<D, kFp8>>(0, kThreads);
  if (per_sm < 0) return SGL_ERR_CUDA;
  constexpr int kRows = 32 / (D / 8);
  const int groups = (p.heads[0] + kRows - 1) / kRows + 2 * ((p.heads[1] + kRows - 1) / kRows);
  // A token's row groups are dealt to several warps while there are fewer
  // tokens than the part has warps for; a warp keeps at least a batch of them
  // unless that still leaves warps idle.
  const int64_t warps = (int64_t)num_sms() * per_sm * kRopeWarps;
  const int batches = (groups + kRopeBatch - 1) / kRopeBatch;
  const int64_t most = (int64_t)p.n * batches < warps ? groups : batches;
  int64_t parts = (warps + p.n - 1) / p.n;
  if (parts > most) parts = most;
  const int64_t cap = ((int64_t)num_sms() * per_sm + parts - 1) / parts;
  int64_t blocks = ((int64_t)p.n + kRopeWarps - 1) / kRopeWarps;
  if (blocks > cap) blocks = cap;
  qk_norm_rope_store_kernel<D, kFp8><<<dim3((unsigned)blocks, (unsigned)parts), kThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SGL_OK : SGL_ERR_CUDA;
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
  if (a.head_dim == 128) return a.kv_fp8 ? run<128, true>(p, stream) : run<128, false>(p, stream);
  if (a.head_dim == 64) return a.kv_fp8 ? run<64, true>(p, stream) : run<64, false>(p, stream);
  return SGL_ERR_UNSUPPORTED;
}

}  // namespace sgl
