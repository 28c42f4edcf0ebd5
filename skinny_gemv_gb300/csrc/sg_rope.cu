// Per-head RMS norm of queries and keys and the position rotation, in one pass:
//
//   y = x * rsqrt(mean(x^2) + eps) * w                     (rows with a weight)
//   (y_a, y_b) -> (y_a c - y_b s, y_a s + y_b c)           over the first rot dims
//
// with (a, b) = (i, i + rot/2), or (2i, 2i + 1) for neighbouring dims, and
// c, s = cos, sin of the token's position from an fp32 table (far positions keep
// the angles the caller computed, in whatever precision).  fp32 throughout, one
// bf16 rounding.
//
// A row (head) of head_dim elements is held by LPR lanes, 16 elements each as two
// chunks of 8 (16-byte loads).  The lane's chunks are j and j + rot/16 while j <
// rot/16, so both members of a rotated pair (i, i + rot/2) are in one lane and no
// value crosses lanes; the remaining chunks pass through.  A lane takes R rows of one
// token, so that its cosines and sines are read once for R heads and R rows' loads
// are in flight together; R is 1 where the step is too small to fill the SMs.
//
// Bound by memory.  Measured: 4096 tokens x (32 + 8) heads x 128 with both norms, 86 MB,
// 18.3 us (4.7 TB/s; a plain copy of the same bytes takes 14.7, so a launch this short
// reaches 0.87 of the copy roof at best); 64 tokens 1.9 us, where it is the launch's latency.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sg_internal.h"
#include "sg_ptx.cuh"

namespace sg {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeRows = 2;            // R for large steps
// Warps from which R = 2 pays, R = 1 / R = 2 in us (40 heads of 128): 640 warps 1.9 / 2.2, 5120
// 3.2 / 3.7, 8190 5.5 / 4.6, 10240 6.6 / 6.9, 16380 9.4 / 8.7, 40960 20.5 / 18.3.
constexpr int64_t kRopeManyWarps = 8192;

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// LPR lanes (a power of two, head_dim <= 16 LPR) per row, R rows per lane.
template <int LPR, int R>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeParams p) {
  constexpr int kRowsPerWarp = 32 / LPR * R;
  const int lane = threadIdx.x % 32;
  const uint32_t item = blockIdx.x * (kRopeThreads / 32) + threadIdx.x / 32;  // a warp's rows of one token
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t t = item / static_cast<uint32_t>(p.items_per_token);
  if (t >= static_cast<uint32_t>(p.tokens)) return;
  const int heads_all = p.heads + p.kv_heads;
  const int row0 = static_cast<int>(item - t * static_cast<uint32_t>(p.items_per_token)) * kRowsPerWarp + lane / LPR;
  const int j = lane % LPR;
  const bool own = j < p.head_dim / 16;
  const int half = p.rot / 16;  // chunks per half of the rotated dims
  const int c0 = j < half ? j : 2 * half + 2 * (j - half);
  const int c1 = j < half ? j + half : c0 + 1;
  const int32_t pos = p.rot > 0 ? p.positions[t] : 0;  // (the rows' loads go out before it is needed)
  uint4 v0[R], v1[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int hh = row0 + i * (32 / LPR);
    v0[i] = v1[i] = make_uint4(0u, 0u, 0u, 0u);
    if (own && hh < heads_all) {
      const bool is_k = hh >= p.heads;
      const uint16_t* src =
          (is_k ? p.K + t * p.ldk : p.Q + t * p.ldq) + static_cast<int64_t>(is_k ? hh - p.heads : hh) * p.head_dim;
      v0[i] = *reinterpret_cast<const uint4*>(src + 8 * c0);
      v1[i] = *reinterpret_cast<const uint4*>(src + 8 * c1);
    }
  }
  if (p.rot > 0 && (pos < 0 || pos >= p.max_pos)) {
    if (lane == 0) record_error(p.err, kDevBadPosition, t);
    return;
  }
  // this lane's cosines and sines: dims 8 j .. 8 j + 7 of the half, or (neighbours) the
  // four pairs of each chunk
  float cs[8], sn[8];
  if (j < half) {
    const float* row = p.cos_sin + static_cast<int64_t>(pos) * p.rot;
    const int a0 = p.neighbours ? 4 * c0 : 8 * j, a1 = p.neighbours ? 4 * c1 : 8 * j + 4;
    *reinterpret_cast<float4*>(cs) = *reinterpret_cast<const float4*>(row + a0);
    *reinterpret_cast<float4*>(cs + 4) = *reinterpret_cast<const float4*>(row + a1);
    *reinterpret_cast<float4*>(sn) = *reinterpret_cast<const float4*>(row + p.rot / 2 + a0);
    *reinterpret_cast<float4*>(sn + 4) = *reinterpret_cast<const float4*>(row + p.rot / 2 + a1);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int hh = row0 + i * (32 / LPR);
    const bool is_k = hh >= p.heads;
    float x0[8], x1[8];
    unpack8(v0[i], x0);
    unpack8(v1[i], x1);
    const uint16_t* w = is_k ? p.wk : p.wq;
    if (p.wq != nullptr || p.wk != nullptr) {  // every lane of the warp
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += x0[e] * x0[e] + x1[e] * x1[e];
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      if (w != nullptr && own) {
        const float inv = rsqrtf(ss / p.head_dim + p.eps);
        float f0[8], f1[8];
        unpack8(*reinterpret_cast<const uint4*>(w + 8 * c0), f0);
        unpack8(*reinterpret_cast<const uint4*>(w + 8 * c1), f1);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x0[e] = x0[e] * inv * f0[e];
          x1[e] = x1[e] * inv * f1[e];
        }
      }
    }
    if (j < half) {
      if (!p.neighbours) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = x0[e], b = x1[e];
          x0[e] = a * cs[e] - b * sn[e];
          x1[e] = a * sn[e] + b * cs[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = x0[2 * e], b = x0[2 * e + 1], c = x1[2 * e], d = x1[2 * e + 1];
          x0[2 * e] = a * cs[e] - b * sn[e];
          x0[2 * e + 1] = a * sn[e] + b * cs[e];
          x1[2 * e] = c * cs[4 + e] - d * sn[4 + e];
          x1[2 * e + 1] = c * sn[4 + e] + d * cs[4 + e];
        }
      }
    }
    if (own && hh < heads_all) {
      uint16_t* dst =
          (is_k ? p.Ko + t * p.ldko : p.Qo + t * p.ldqo) + static_cast<int64_t>(is_k ? hh - p.heads : hh) * p.head_dim;
      *reinterpret_cast<uint4*>(dst + 8 * c0) = pack8(x0);
      *reinterpret_cast<uint4*>(dst + 8 * c1) = pack8(x1);
    }
  }
}

template <int LPR, int R>
cudaError_t launch_rows(RopeParams p, cudaStream_t stream) {
  constexpr int kRowsPerWarp = 32 / LPR * R;
  p.items_per_token = (p.heads + p.kv_heads + kRowsPerWarp - 1) / kRowsPerWarp;
  const int64_t items = static_cast<int64_t>(p.tokens) * p.items_per_token;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      pdl_config((items + kRopeThreads / 32 - 1) / (kRopeThreads / 32), kRopeThreads, 0, stream, attr);
  return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<LPR, R>, p);
}

// R rows per lane once the rows fill the device's warps several times over.
template <int LPR>
cudaError_t launch(const RopeParams& p, cudaStream_t stream) {
  const int64_t warps = static_cast<int64_t>(p.tokens) * (p.heads + p.kv_heads) * LPR / 32;
  return warps >= kRopeManyWarps ? launch_rows<LPR, kRopeRows>(p, stream) : launch_rows<LPR, 1>(p, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& p, cudaStream_t stream) {
  const int lanes = p.head_dim / 16;
  if (lanes <= 4) return launch<4>(p, stream);
  if (lanes <= 8) return launch<8>(p, stream);
  if (lanes <= 16) return launch<16>(p, stream);
  return launch<32>(p, stream);
}

}  // namespace sg
