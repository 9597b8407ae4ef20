// Index queries and keys of a step, ready to be scored (dsa_index_prepare,
// dsa_index_prepare_fp8): per head row x of width 128
//
//   rms:    y = x / sqrt(mean(x^2) + eps) * weight + bias
//   layer:  y = (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps) * weight + bias
//   rotation of the pair (a, b) number i of the first `rot` dimensions by the
//   angle position * inv_freq[i]:  (a cos - b sin, a sin + b cos)
//   out:    y in bf16, or E4M3 codes of y / scale with scale = max|y| / 448
//
// in one pass: 256 bytes read and 256 (or 132) written per row, so HBM bounds
// it.  A row is 16 lanes of 16 bytes; its statistics are four shuffles.  The
// angles of a token are shared by all its rows: one warp of the block forms
// them (turns = position * inv_freq / 2 pi in fp64, since fp32 has no digits
// left of the fraction of a turn at positions near 10^6; the fraction is then
// exact enough for fp32 sincospi) while the rows' loads are in flight.
// Statistics, rotation and scales are fp32; the store rounds once.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "dsa_ptx.cuh"
#include "dsa_serve.cuh"

namespace dsa {

namespace {

constexpr int kPrepThreads = 256;
constexpr int kPrepRows = kPrepThreads / 16;  // rows in flight per step
constexpr int kW = 128;                       // row width

__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o, 16);
  return v;
}
__device__ __forceinline__ float max16(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o, 16));
  return v;
}

struct RowOut {
  uint4 bf16;    // 8 values
  uint2 e4m3;    // 8 codes
  float scale;
};

// Norm and rotation of one row held as 8 values per lane (dimensions
// 8 l .. 8 l + 7 of lane l of 16).  All 32 lanes of the warp call it.
template <bool FP8>
__device__ __forceinline__ RowOut prepare_row(const uint4 raw, const PrepareParams& p, int norm, const float* weight,
                                              const float* bias, const float2* s_cs, int l) {
  float x[8];
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
  if (norm != kNormNone) {
    if (norm == kNormLayer) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += x[i];
      const float mean = sum16(s) * (1.f / kW);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] -= mean;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
    const float inv = rsqrtf(fmaf(sum16(s), 1.f / kW, p.eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= inv;
    if (weight) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(weight) + 2 * l);
      const float4 b = __ldg(reinterpret_cast<const float4*>(weight) + 2 * l + 1);
      x[0] *= a.x; x[1] *= a.y; x[2] *= a.z; x[3] *= a.w;
      x[4] *= b.x; x[5] *= b.y; x[6] *= b.z; x[7] *= b.w;
    }
    if (bias) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(bias) + 2 * l);
      const float4 b = __ldg(reinterpret_cast<const float4*>(bias) + 2 * l + 1);
      x[0] += a.x; x[1] += a.y; x[2] += a.z; x[3] += a.w;
      x[4] += b.x; x[5] += b.y; x[6] += b.z; x[7] += b.w;
    }
  }
  if (p.interleaved) {
    if (8 * l < p.rot) {  // rot is a multiple of 16: a lane rotates all of its values or none
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 cs = s_cs[4 * l + i];
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * cs.x - b * cs.y;
        x[2 * i + 1] = a * cs.y + b * cs.x;
      }
    }
  } else {
    // dimension i pairs with i + rot / 2: the partner lane is rot / 16 away
    const int off = p.rot >> 4;
    const bool first = l < off, second = !first && l < 2 * off;
    const int partner = first ? l + off : second ? l - off : l;
    const float sign = first ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(~0u, x[i], partner, 16);
      if (first || second) {
        const float2 cs = s_cs[(first ? 8 * l : 8 * partner) + i];
        x[i] = x[i] * cs.x + sign * o * cs.y;
      }
    }
  }
  RowOut r{};
  if constexpr (FP8) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    m = max16(m);
    // a row of zeros has scale 1; a scale is never subnormal, so that its
    // reciprocal is finite
    r.scale = m > 0.f ? fmaxf(__fdiv_rn(m, 448.f), 1.17549435e-38f) : 1.f;
    // value * (1 / scale) instead of value / scale: within two fp32 roundings
    // of the quotient, against E4M3's 2^-4
    const float inv = __frcp_rn(r.scale);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    r.e4m3 = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  } else {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      c[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    r.bf16 = make_uint4(c[0], c[1], c[2], c[3]);
  }
  return r;
}

template <bool FP8>
__device__ __forceinline__ void store_row(const RowOut& r, void* out, float* scale, int64_t row, int l) {
  if constexpr (FP8) {
    reinterpret_cast<uint2*>(static_cast<uint8_t*>(out) + row * kW)[l] = r.e4m3;
    if (l == 0) scale[row] = r.scale;
  } else {
    reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row * kW)[l] = r.bf16;
  }
}

// Work unit = one token and U * 16 of its query heads; the unit of a token's
// first heads also does its key.
template <bool FP8, int U>
__global__ void __launch_bounds__(kPrepThreads) index_prepare_kernel(const PrepareParams p) {
  __shared__ float2 s_cs[2][kW / 2];
  const int tid = threadIdx.x, l = tid & 15, hw = tid >> 4;
  const int chunks = (p.H + U * kPrepRows - 1) / (U * kPrepRows);
  const int64_t units = p.T * chunks;
  int buf = 0;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x, buf ^= 1) {
    const int64_t t = u / chunks;
    const int h0 = static_cast<int>(u - t * chunks) * U * kPrepRows;
    const int32_t pos = __ldg(p.position + t);
    if (pos < 0) continue;  // padding (uniform over the block): nothing is written
    uint4 raw[U], rawk = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * kPrepRows + hw;
      raw[i] = h < p.H ? reinterpret_cast<const uint4*>(p.q + (t * p.H + h) * kW)[l] : make_uint4(0u, 0u, 0u, 0u);
    }
    int64_t slot = -1;
    if (h0 == 0 && hw < 2) {  // the key row: the first warp (its upper half repeats the lower)
      slot = p.slot_map ? __ldg(p.slot_map + t) : t;
      rawk = __ldg(reinterpret_cast<const uint4*>(p.k + t * kW) + l);
    }
    if (tid >= kPrepThreads - 64 && tid - (kPrepThreads - 64) < p.rot / 2) {
      const int i = tid - (kPrepThreads - 64);
      const double turns = static_cast<double>(pos) * static_cast<double>(__ldg(p.inv_freq + i)) * 0.15915494309189535;
      float sn, cs;
      sincospif(2.f * static_cast<float>(turns - rint(turns)), &sn, &cs);
      s_cs[buf][i] = make_float2(cs, sn);
    }
    __syncthreads();  // one per unit: the other buffer's readers have passed the last one
    if (h0 == 0 && hw < 2) {
      const RowOut r = prepare_row<FP8>(rawk, p, p.k_norm, p.k_weight, p.k_bias, s_cs[buf], l);
      if (hw == 0 && slot >= 0) {
        if (slot < p.n_slots)
          store_row<FP8>(r, p.k_out, p.k_scale, slot, l);
        else if (l == 0 && p.status)
          atomicOr(p.status, kErrOverflow);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * kPrepRows + hw;
      if (h0 + i * kPrepRows + (hw & ~1) < p.H) {  // warp-uniform
        const RowOut r = prepare_row<FP8>(raw[i], p, p.q_norm, p.q_weight, p.q_bias, s_cs[buf], l);
        if (h < p.H) store_row<FP8>(r, p.q_out, p.q_scale, t * p.H + h, l);
      }
    }
  }
}

template <bool FP8, int U>
cudaError_t launch_u(const PrepareParams& p, int sms, cudaStream_t st) {
  const int64_t units = p.T * ((p.H + U * kPrepRows - 1) / (U * kPrepRows));
  const int grid = static_cast<int>(std::min<int64_t>(units, static_cast<int64_t>(sms) * 8));
  index_prepare_kernel<FP8, U><<<grid, kPrepThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_index_prepare(const PrepareParams& p, int sms, cudaStream_t st) {
  if (p.T <= 0) return cudaSuccess;
  const bool wide = p.T >= sms;
  if (p.fp8) return wide ? launch_u<true, 4>(p, sms, st) : launch_u<true, 1>(p, sms, st);
  return wide ? launch_u<false, 4>(p, sms, st) : launch_u<false, 1>(p, sms, st);
}

}  // namespace dsa
