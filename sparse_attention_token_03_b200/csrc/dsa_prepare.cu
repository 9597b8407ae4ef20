// Index queries and keys of a step, ready to be scored (dsa_index_prepare,
// dsa_index_prepare_fp8): per head row x of width 128
//
//   rms:    y = x / sqrt(mean(x^2) + eps) * weight + bias
//   layer:  y = (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps) * weight + bias
//   rotation of the pair (a, b) number i of the first `rot` dimensions by the
//   angle position * inv_freq[i]:  (a cos - b sin, a sin + b cos)
//   out:    y in bf16, or E4M3 codes of y / scale with scale = max|y| / 448
//
// in one pass: 256 bytes read and 256 (or 132) written per row.  A row is 8 lanes of two 8-value chunks, chosen so that both members of
// every rotated pair are in one lane (lane l < rot / 16 of the half-split form
// holds chunks l and l + rot / 16); statistics are three shuffles.  The angles
// of a token are shared by all its rows: a block forms those of its tokens
// (turns = position * inv_freq / 2 pi in fp64, since fp32 has no digits left
// of the fraction of a turn at positions near 10^6; the fraction is then exact
// enough for fp32 sincospi), and a lane keeps its angles and weights in
// registers over the rows: read per row, they and the partners' shuffles made
// the L1 pipe the bound (86%, 163 us for 16384 tokens of 64 heads; now 110 us,
// 4.9 TB/s).  What bounds it now is the issue of instructions: the schedulers are
// busy 63% of all cycles (67% with FP8, some 290 instructions a row of a warp's
// four), at 3 blocks of 80 registers an SM, while HBM is at 57% (38%).
// Statistics, rotation and scales are fp32; the store rounds once.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "dsa_ptx.cuh"
#include "dsa_serve.cuh"

namespace dsa {

namespace {

constexpr int kPrepThreads = 256;
constexpr int kPrepRows = kPrepThreads / 8;  // rows in flight per step
constexpr int kW = 128;                      // row width

// A norm's mean square plus eps below which its squares have lost digits, and
// above which their sum may be infinite; a NaN is neither.  (Such rows scaled
// first, out of the walk's way, cost ordinary ones 20%: 134 us for 110.)
constexpr float kNormLow = 7.8886091e-31f, kNormHigh = 1.3292280e36f;  // 2^-100, 2^120
__device__ __forceinline__ void non_finite(uint32_t* status, int64_t row) {
  if (row >= 0 && status) atomicOr(status, kErrNonFinite);
}
__device__ __forceinline__ float sum8(float v) {
#pragma unroll
  for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o, 8);
  return v;
}
__device__ __forceinline__ float max8(float v) {
#pragma unroll
  for (int o = 4; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(~0u, v, o, 8));
  return v;
}

// The two 8-value chunks of a row that lane l of 8 holds.
struct Chunks {
  int a, b;
};
__device__ __forceinline__ Chunks chunks_of(const PrepareParams& p, bool interleaved, int l) {
  const int half = p.rot >> 4;  // chunks of half the rotated dimensions
  if (interleaved || l >= half) return {2 * l, 2 * l + 1};  // past the pairs: 2 half + 2 (l - half)
  return {l, l + half};
}

// Norm of a kind of rows: its weights for a lane's values, and where the bias is.
struct NormLane {
  int norm;
  float w[16];
  const float4* bias;
};
__device__ __forceinline__ void load_norm(NormLane& n, int norm, const float* weight, const float* bias, Chunks c) {
  n.norm = norm;
  n.bias = reinterpret_cast<const float4*>(bias);
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const float4 w = weight ? __ldg(reinterpret_cast<const float4*>(weight) + 2 * (h < 2 ? c.a : c.b) + (h & 1))
                            : make_float4(1.f, 1.f, 1.f, 1.f);
    n.w[4 * h] = w.x, n.w[4 * h + 1] = w.y, n.w[4 * h + 2] = w.z, n.w[4 * h + 3] = w.w;
  }
}

struct RawRow {
  uint4 a, b;
};
__device__ __forceinline__ RawRow load_row(const uint16_t* rows, int64_t row, Chunks c) {
  const uint4* src = reinterpret_cast<const uint4*>(rows + row * kW);
  return {__ldg(src + c.a), __ldg(src + c.b)};
}

// Norm, rotation (rotate: this lane holds pairs, cs their angles) and store of
// one row; nothing is stored for row < 0.  A stored row with a NaN or an
// infinity is reported.  All 32 lanes of the warp call it.
template <bool FP8, bool INTER>
__device__ __forceinline__ void finish_row(const RawRow& raw, const NormLane& n, float eps, bool rotate,
                                           const float2 (&cs)[8], Chunks c, void* out, float* scale, int64_t row, int l,
                                           uint32_t* status) {
  float x[16];
  const uint32_t u[8] = {raw.a.x, raw.a.y, raw.a.z, raw.a.w, raw.b.x, raw.b.y, raw.b.z, raw.b.w};
  if (!FP8 && n.norm == kNormNone) {
    uint32_t top = 0;  // the largest magnitudes' bits, two values a word
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __vmaxu2(top, u[i] & 0x7FFF7FFFu);
    if ((top & 0xFFFFu) >= 0x7F80u || top >= 0x7F800000u) non_finite(status, row);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
  if (n.norm != kNormNone) {
    if (n.norm == kNormLayer) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) s += x[i];
      const float mean = sum8(s) * (1.f / kW);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] -= mean;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s = fmaf(x[i], x[i], s);
    const float v = fmaf(sum8(s), 1.f / kW, eps);
    if (!(v >= kNormLow && v < kNormHigh)) non_finite(status, row);
    const float inv = rsqrtf(v);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = x[i] * inv * n.w[i];
    if (n.bias) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float4 b = __ldg(n.bias + 2 * (h < 2 ? c.a : c.b) + (h & 1));
        x[4 * h] += b.x, x[4 * h + 1] += b.y, x[4 * h + 2] += b.z, x[4 * h + 3] += b.w;
      }
    }
  }
  if (rotate) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float &a = INTER ? x[2 * i] : x[i], &b = INTER ? x[2 * i + 1] : x[i + 8];
      const float r = a * cs[i].x - b * cs[i].y;
      b = a * cs[i].y + b * cs[i].x;
      a = r;
    }
  }
  if constexpr (FP8) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max_nan(m, fabsf(x[i]));
    m = max8(m);
    if (!(m < INFINITY)) non_finite(status, row);
    // a row of zeros has scale 1; a scale is never subnormal, so that its
    // reciprocal is finite
    const float sc = m > 0.f ? fmaxf(__fdiv_rn(m, 448.f), 1.17549435e-38f) : 1.f;
    // value * (1 / scale) instead of value / scale: within two fp32 roundings
    // of the quotient, against E4M3's 2^-4
    const float inv = __frcp_rn(sc);
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo =
          __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * inv, x[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi =
          __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * inv, x[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
      v[i] = lo | (hi << 16);
    }
    if (row >= 0) {
      uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(out) + row * kW);
      dst[c.a] = make_uint2(v[0], v[1]);
      dst[c.b] = make_uint2(v[2], v[3]);
      if (l == 0) scale[row] = sc;
    }
  } else {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      v[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if (row >= 0) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row * kW);
      dst[c.a] = make_uint4(v[0], v[1], v[2], v[3]);
      dst[c.b] = make_uint4(v[4], v[5], v[6], v[7]);
    }
  }
}

// A block takes G consecutive tokens, or with G = 1 also just 32 of a token's
// heads (blockIdx.y): it forms the tokens' angles with all threads, then each
// group of 8 lanes walks the rows on its own, the next row in flight.
template <bool FP8, bool INTER, int G>
__global__ void __launch_bounds__(kPrepThreads, G > 1 ? 3 : 1) index_prepare_kernel(const PrepareParams p) {
  __shared__ float2 s_cs[G][kW / 2];
  __shared__ int s_pos[G];
  const int tid = threadIdx.x, l = tid & 7, hw = tid >> 3;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * G;
  const int h_lo = G > 1 ? 0 : blockIdx.y * kPrepRows, h_hi = G > 1 ? p.H : min(h_lo + kPrepRows, p.H);
  const Chunks c = chunks_of(p, INTER, l);
  const bool rotate = l < (p.rot >> 4);
  // units of this block: 32 heads of a token
  const int per = G > 1 ? (p.H + kPrepRows - 1) / kPrepRows : 1;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(G), p.T - t0));
  RawRow next, rawk{};
  auto load = [&](int g, int h0) { next = load_row(p.q, (t0 + g) * p.H + min(h0 + hw, p.H - 1), c); };
  load(0, h_lo);
  const bool key = h_lo == 0 && (hw & ~3) < tokens;  // key row of token hw
  int64_t slot = -1;
  if (key) {
    const int64_t t = t0 + min(hw, tokens - 1);
    if (hw < tokens) slot = p.slot_map ? __ldg(p.slot_map + t) : t;
    rawk = load_row(p.k, t, c);
  }
  for (int i = tid; i < tokens * (kW / 2); i += kPrepThreads) {
    const int g = i / (kW / 2), k = i % (kW / 2);
    const int pos = __ldg(p.position + t0 + g);
    if (k == 0) s_pos[g] = pos;
    if (k < p.rot / 2) {
      const double turns = static_cast<double>(pos) * static_cast<double>(__ldg(p.inv_freq + k)) * 0.15915494309189535;
      float sn, cs;
      sincospif(2.f * static_cast<float>(turns - rint(turns)), &sn, &cs);
      s_cs[g][k] = make_float2(cs, sn);
    }
  }
  NormLane n;
  __syncthreads();
  float2 cs[8];
  auto angles = [&](int g) {
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = s_cs[g][rotate ? 8 * l + i : 0];
  };
  if (key) {
    const int g = min(hw, tokens - 1);
    load_norm(n, p.k_norm, p.k_weight, p.k_bias, c);
    angles(g);
    if (s_pos[g] < 0) slot = -1;  // padding
    if (slot >= p.n_slots) {
      if (l == 0 && p.status) atomicOr(p.status, kErrOverflow);
      slot = -1;
    }
    finish_row<FP8, INTER>(rawk, n, p.eps, rotate, cs, c, p.k_out, p.k_scale, slot, l, p.status);
  }
  load_norm(n, p.q_norm, p.q_weight, p.q_bias, c);
#pragma unroll 1
  for (int u = 0, g = 0, h0 = h_lo; u < tokens * per; ++u) {
    const RawRow now = next;
    int g1 = g, h1 = h0 + kPrepRows;  // the next unit
    if (h1 >= h_hi) {
      h1 = h_lo;
      ++g1;
    }
    if (u + 1 < tokens * per) load(g1, h1);
    if (h0 == h_lo) angles(g);
    const int h = h0 + hw;
    if (s_pos[g] >= 0 && h0 + (hw & ~3) < h_hi)  // else padding, or no such heads; the same in all lanes of the warp
      finish_row<FP8, INTER>(now, n, p.eps, rotate, cs, c, p.q_out, p.q_scale, h < h_hi ? (t0 + g) * p.H + h : -1, l,
                             p.status);
    g = g1;
    h0 = h1;
  }
}

template <bool FP8, bool INTER, int G>
cudaError_t launch_groups(const PrepareParams& p, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((p.T + G - 1) / G), G > 1 ? 1 : (p.H + kPrepRows - 1) / kPrepRows);
  index_prepare_kernel<FP8, INTER, G><<<grid, kPrepThreads, 0, st>>>(p);
  return cudaGetLastError();
}

// Tokens of a block: more share the weights' loads and the block's start, fewer
// fill the GPU sooner.  With 64 heads, 300 tokens take 6.8 / 6.1 / 7.3 / 11.6 us
// in groups of 1 / 2 / 4 / 8, 1000 tokens 16.3 / 12.0 / 9.7 / 12.1, 2000 tokens
// - / 17.6 / 17.0 / 16.2.
template <bool FP8, bool INTER>
cudaError_t launch_prepare(const PrepareParams& p, int sms, cudaStream_t st) {
  const int64_t per_sm = p.T / std::max(sms, 1);
  if (per_sm >= 8) return launch_groups<FP8, INTER, 8>(p, st);
  if (per_sm >= 5) return launch_groups<FP8, INTER, 4>(p, st);
  if (per_sm >= 2) return launch_groups<FP8, INTER, 2>(p, st);
  return launch_groups<FP8, INTER, 1>(p, st);
}

}  // namespace

cudaError_t launch_index_prepare(const PrepareParams& p, int sms, cudaStream_t st) {
  if (p.T <= 0) return cudaSuccess;
  if (p.fp8) return p.interleaved ? launch_prepare<true, true>(p, sms, st) : launch_prepare<true, false>(p, sms, st);
  return p.interleaved ? launch_prepare<false, true>(p, sms, st) : launch_prepare<false, false>(p, sms, st);
}

}  // namespace dsa
