// Rows of the 4-bit latent cache, written and read by slot (dsa_kv4_write,
// dsa_kv4_read).  Per block of 16 latent dimensions
//
//   scale = E4M3(max|x| / 6)         (nearest, ties to even, at most 448)
//   code  = E2M1(x / scale)          (nearest, ties to even, at most 6; 0 where scale is 0)
//   value = code * scale             (6 significant bits: exact in bf16 and fp16)
//
// with both quotients in fp32, so the stored bytes are a function of the
// input alone.  A NaN makes its block's scale NaN, so the block reads back as
// NaN; infinities saturate.  One warp per token, one lane per block: 1152 bytes
// against 416 per token.  Bound by the launch for a decode step's rows and by
// latency for a chunk: a row's slot is loaded before the row is asked for (16383
// rows: 11 us written and 10 us read where their bytes take 4 each; warps wait
// for loads, HBM is at 20% and 9%).
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "dsa_ptx.cuh"
#include "dsa_serve.cuh"

namespace dsa {

namespace {

constexpr int kKvThreads = 256;

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// Cache entry of row t, or null for padding (slot < 0) and, with the status
// bit set, for a slot outside the pool.
__device__ __forceinline__ uint8_t* entry_of(const Kv4Params& p, int64_t t, int lane) {
  const int32_t slot = __ldg(p.slot_map + t);
  if (slot < 0) return nullptr;
  if (slot >= p.n_slots) {
    if (lane == 0 && p.status) atomicOr(p.status, kErrOverflow);
    return nullptr;
  }
  return p.kv + static_cast<int64_t>(slot) * kKvEntry;
}

__global__ void __launch_bounds__(kKvThreads) kv4_write_kernel(const Kv4Params p) {
  const int lane = threadIdx.x & 31;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kKvThreads / 32);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kKvThreads / 32) + (threadIdx.x >> 5); t < p.T; t += stride) {
    uint8_t* e = entry_of(p, t, lane);
    if (!e) continue;
    const uint4* src = reinterpret_cast<const uint4*>(p.latent + t * kKvLat) + 2 * lane;
    const uint4 a = __ldg(src), b = __ldg(src + 1);
    const uint32_t rope = __ldg(reinterpret_cast<const uint32_t*>(p.rope + t * kKvRope) + lane);
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float x[16], m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      m = max_nan(m, max_nan(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
    }
    if (p.status && !(m < INFINITY)) atomicOr(p.status, kErrNonFinite);
    const uint8_t sc = __nv_cvt_float_to_fp8(__fdiv_rn(m, 6.f), __NV_SATFINITE, __NV_E4M3);
    const float sv = e4m3_value(sc);
    uint32_t code[2] = {0u, 0u};
    if (sv > 0.f) {  // not where it is 0 or NaN
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t c = __nv_cvt_float2_to_fp4x2(make_float2(__fdiv_rn(x[2 * i], sv), __fdiv_rn(x[2 * i + 1], sv)),
                                                    __NV_E2M1, cudaRoundNearest);
        code[i >> 2] |= c << (8 * (i & 3));
      }
    }
    reinterpret_cast<uint2*>(e)[lane] = make_uint2(code[0], code[1]);
    e[kKvScaleOff + lane] = sc;
    reinterpret_cast<uint32_t*>(e + kKvRopeOff)[lane] = rope;
  }
}

__global__ void __launch_bounds__(kKvThreads) kv4_read_kernel(const Kv4Params p) {
  const int lane = threadIdx.x & 31;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kKvThreads / 32);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kKvThreads / 32) + (threadIdx.x >> 5); t < p.T; t += stride) {
    const uint8_t* e = entry_of(p, t, lane);
    if (!e) continue;
    const uint2 code = reinterpret_cast<const uint2*>(e)[lane];
    const float sv = e4m3_value(e[kKvScaleOff + lane]);
    const uint32_t rope = reinterpret_cast<const uint32_t*>(e + kKvRopeOff)[lane];
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c = ((i < 4 ? code.x : code.y) >> (8 * (i & 3))) & 0xFFu;
      const float2 f = __half22float2(__half2(__nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(c), __NV_E2M1)));
      // the products have 6 significant bits: their upper 16 bits are their bf16
      v[i] = (__float_as_uint(f.x * sv) >> 16) | (__float_as_uint(f.y * sv) & 0xFFFF0000u);
    }
    uint4* dst = reinterpret_cast<uint4*>(p.latent_out + t * kKvLat) + 2 * lane;
    dst[0] = make_uint4(v[0], v[1], v[2], v[3]);
    dst[1] = make_uint4(v[4], v[5], v[6], v[7]);
    reinterpret_cast<uint32_t*>(p.rope_out + t * kKvRope)[lane] = rope;
  }
}

int kv4_grid(int64_t T, int sms) {
  const int64_t blocks = (T + kKvThreads / 32 - 1) / (kKvThreads / 32);
  return static_cast<int>(std::min<int64_t>(blocks, static_cast<int64_t>(sms) * 8));
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4Params& p, int sms, cudaStream_t st) {
  if (p.T <= 0) return cudaSuccess;
  kv4_write_kernel<<<kv4_grid(p.T, sms), kKvThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4Params& p, int sms, cudaStream_t st) {
  if (p.T <= 0) return cudaSuccess;
  kv4_read_kernel<<<kv4_grid(p.T, sms), kKvThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace dsa
