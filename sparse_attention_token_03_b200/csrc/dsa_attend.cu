// Attention of all query heads over the selected keys of a 4-bit latent cache
// (dsa_attend_kv4): for row t, head h and the entries j of the row's list
//
//   z(t,h,j) = scale * (q(t,h) . [latent_j, rotary_j])
//   out(t,h) = sum_j softmax_j(z) latent_j,   lse(t,h) = log sum_j exp z
//
// One block per (row, 8 heads), one warp per head: 32 keys at a time are
// decoded to fp32 in shared memory; a lane scores one key, then holds 16
// output dimensions; running maximum and sum in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "dsa_ptx.cuh"
#include "dsa_serve.cuh"

namespace dsa {

namespace {

constexpr int kAttThreads = 256;
constexpr int kAttHeads = kAttThreads / 32;
constexpr int kAttKeys = 32;
constexpr int kAttPitch = kKvQ + 1;

// Pool row of list entry `pos` of sequence `seq`, or -1 (nothing listed, or a
// position or page outside its range, which sets the status bit).
__device__ __forceinline__ int64_t slot_of(const AttendParams& p, int seq, int pos) {
  if (pos < 0) return -1;
  const int blk = pos / p.page_size;
  if (blk < p.max_blocks) {
    const int page = __ldg(p.block_table + static_cast<int64_t>(seq) * p.max_blocks + blk);
    if (page >= 0 && page < p.n_pages) return static_cast<int64_t>(page) * p.page_size + (pos - blk * p.page_size);
  }
  if (p.status) atomicOr(p.status, kErrOverflow);
  return -1;
}

__global__ void __launch_bounds__(kAttThreads) attend_kv4_kernel(const AttendParams p) {
  extern __shared__ float smem[];
  float* s_k = smem;                              // [kAttKeys][kAttPitch]
  float* s_q = s_k + kAttKeys * kAttPitch;        // [kAttHeads][kKvQ]
  __shared__ int64_t s_slot[kAttKeys];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hb = (p.H + kAttHeads - 1) / kAttHeads;
  const int64_t t = blockIdx.x / hb;
  const int h = static_cast<int>(blockIdx.x % hb) * kAttHeads + warp;
  const int seq = p.row_seq ? __ldg(p.row_seq + t) : static_cast<int>(t);
  if (seq < 0) return;
  if (seq >= p.B) {
    if (tid == 0 && p.status) atomicOr(p.status, kErrOverflow);
    return;
  }
  const bool live = h < p.H;
  for (int d = lane; d < kKvQ; d += 32)
    s_q[warp * kKvQ + d] = live ? __uint_as_float(static_cast<uint32_t>(p.q[(t * p.H + h) * kKvQ + d]) << 16) : 0.f;
  float m = -INFINITY, sum = 0.f, acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int j0 = 0; j0 < p.n; j0 += kAttKeys) {
    __syncthreads();
    if (tid < kAttKeys) s_slot[tid] = j0 + tid < p.n ? slot_of(p, seq, __ldg(p.idx + t * p.n + j0 + tid)) : -1;
    __syncthreads();
    for (int c = tid; c < kAttKeys * 32; c += kAttThreads) {  // one block of 16 dimensions
      const int key = c >> 5, blk = c & 31;
      const int64_t s = s_slot[key];
      float* dst = s_k + key * kAttPitch + 16 * blk;
      float* rdst = s_k + key * kAttPitch + kKvLat + 2 * blk;
      if (s < 0) {
        for (int i = 0; i < 16; ++i) dst[i] = 0.f;
        rdst[0] = rdst[1] = 0.f;
        continue;
      }
      const uint8_t* e = p.kv + s * kKvEntry;
      const uint2 code = reinterpret_cast<const uint2*>(e)[blk];
      const float sv = __half2float(__half(__nv_cvt_fp8_to_halfraw(e[kKvScaleOff + blk], __NV_E4M3)));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t by = ((i < 4 ? code.x : code.y) >> (8 * (i & 3))) & 0xFFu;
        const float2 f =
            __half22float2(__half2(__nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(by), __NV_E2M1)));
        dst[2 * i] = f.x * sv;
        dst[2 * i + 1] = f.y * sv;
      }
      const uint32_t r = reinterpret_cast<const uint32_t*>(e + kKvRopeOff)[blk];
      rdst[0] = __uint_as_float(r << 16);
      rdst[1] = __uint_as_float(r & 0xFFFF0000u);
    }
    __syncthreads();
    const bool valid = s_slot[lane] >= 0;
    float z = 0.f;
    for (int d = 0; d < kKvQ; ++d) z = fmaf(s_q[warp * kKvQ + d], s_k[lane * kAttPitch + d], z);
    z = valid ? z * p.scale : -INFINITY;
    float mx = z;
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
    const float mn = fmaxf(m, mx);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float f = __expf(m - ref), e = valid ? __expf(z - ref) : 0.f;
    m = mn;
    float es = e;
#pragma unroll
    for (int o = 16; o; o >>= 1) es += __shfl_xor_sync(~0u, es, o);
    sum = sum * f + es;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] *= f;
    for (int k = 0; k < kAttKeys; ++k) {
      const float w = __shfl_sync(~0u, e, k);
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = fmaf(w, s_k[k * kAttPitch + i * 32 + lane], acc[i]);
    }
  }
  if (!live) return;
  const float inv = sum > 0.f ? 1.f / sum : (sum == sum ? 0.f : sum);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const __nv_bfloat16 b = __float2bfloat16_rn(acc[i] * inv);
    p.out[(t * p.H + h) * kKvLat + i * 32 + lane] = *reinterpret_cast<const uint16_t*>(&b);
  }
  if (p.lse && lane == 0) p.lse[t * p.H + h] = m + logf(sum);
}

}  // namespace

cudaError_t launch_attend_kv4(const AttendParams& p, int sms, cudaStream_t st) {
  (void)sms;
  constexpr int bytes = (kAttKeys * kAttPitch + kAttHeads * kKvQ) * 4;
  cudaError_t e = cudaFuncSetAttribute(attend_kv4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const int64_t grid = p.T * ((p.H + kAttHeads - 1) / kAttHeads);
  attend_kv4_kernel<<<static_cast<unsigned>(grid), kAttThreads, bytes, st>>>(p);
  return cudaGetLastError();
}

}  // namespace dsa
