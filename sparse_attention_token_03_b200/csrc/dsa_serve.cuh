// Parameters and launchers of the serving operators around the index Top-k:
// request layout (dsa_tables.cu), index preparation (dsa_prepare.cu), the
// 4-bit latent cache (dsa_kv4.cu) and attention over the selected keys
// (dsa_attend.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "dsa_ptx.cuh"

namespace dsa {

// One cached token of the 4-bit latent cache, 416 bytes: 512 E2M1 codes (two
// per byte, the even dimension in the low nibble), 32 E4M3 scales (one per 16
// dimensions), 64 rotary values in bf16.  416 = 13 x 32, so an entry of a
// 32-byte aligned pool is a whole number of DRAM sectors.
constexpr int kKvLat = 512;
constexpr int kKvRope = 64;
constexpr int kKvBlock = 16;
constexpr int kKvScaleOff = kKvLat / 2;
constexpr int kKvRopeOff = kKvScaleOff + kKvLat / kKvBlock;
constexpr int kKvEntry = kKvRopeOff + 2 * kKvRope;
constexpr int kKvQ = kKvLat + kKvRope;  // query row: latent part, then rotary part
static_assert(kKvEntry == 416, "cache entry layout");

// Row statistics of the index preparation (include/dsa_index.h, DSA_NORM_*).
enum : int { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };

// Division of a position (below 2^31) by the page size as a product: with s =
// ceil(log2 d) and mul = ceil(2^(31 + s) / d) the product's error n (mul d -
// 2^(31 + s)) / (d 2^(31 + s)) is below 1 / d, so the quotient is exact.
struct PageDiv {
  uint32_t mul, shift;
  __host__ __device__ int operator()(int n) const {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul >> shift);
  }
};
inline PageDiv page_div(int d) {
  uint32_t s = 0;
  while ((int64_t(1) << s) < d) ++s;
  return {static_cast<uint32_t>(((uint64_t(1) << (31 + s)) + d - 1) / d), 31 + s};
}

// The larger of two magnitudes, NaN where either is (fmaxf drops it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

struct TablesParams {
  const int32_t* cached_len;  // [B]
  const int32_t* new_len;     // [B]
  int B;
  int32_t* block_table;       // [B][max_blocks]
  int max_blocks;
  const int32_t* free_pages;  // [n_free]
  int64_t n_free;
  const int32_t* free_begin;  // [1]
  int64_t n_pages;
  int page_size;
  int T_cap;
  int32_t* slot_map;          // [T_cap]
  int32_t* position;          // [T_cap]
  int32_t* row_seq;           // [T_cap]
  int32_t* row_start;         // [B + 1]
  int32_t* seq_len;           // [B]
  int32_t* free_end;          // [1]
  uint32_t* status;           // may be null
};
cudaError_t launch_block_tables(const TablesParams& p, int sms, cudaStream_t st);

struct PrepareParams {
  const uint16_t* q;        // [T][H][128] bf16
  const uint16_t* k;        // [T][128] bf16
  const int32_t* position;  // [T]
  const float* inv_freq;    // [rot / 2]
  int rot;
  int interleaved;
  int64_t T;
  int H;
  int q_norm, k_norm;
  const float *q_weight, *q_bias, *k_weight, *k_bias;  // [128] or null
  float eps;
  const int32_t* slot_map;  // [T] or null (row t to slot t)
  int64_t n_slots;
  void* q_out;              // [T][H][128] bf16 or E4M3
  float* q_scale;           // [T][H] (E4M3 only)
  void* k_out;              // [n_slots][128]
  float* k_scale;           // [n_slots] (E4M3 only)
  uint32_t* status;         // may be null
  bool fp8;
};
cudaError_t launch_index_prepare(const PrepareParams& p, int sms, cudaStream_t st);

struct Kv4Params {
  const uint16_t* latent;   // [T][512] bf16 (write)
  const uint16_t* rope;     // [T][64] bf16 (write)
  uint16_t* latent_out;     // [T][512] bf16 (read)
  uint16_t* rope_out;       // [T][64] bf16 (read)
  uint8_t* kv;              // [n_slots][416]
  const int32_t* slot_map;  // [T]
  int64_t T;
  int64_t n_slots;
  uint32_t* status;         // may be null
};
cudaError_t launch_kv4_write(const Kv4Params& p, int sms, cudaStream_t st);
cudaError_t launch_kv4_read(const Kv4Params& p, int sms, cudaStream_t st);

struct AttendParams {
  const uint16_t* q;           // [T][H][576] bf16
  const uint8_t* kv;           // [n_pages][page_size][416]
  int64_t n_pages;
  int page_size;
  const int32_t* block_table;  // [B][max_blocks]
  int B;
  int max_blocks;
  const int32_t* row_seq;      // [T] or null (row t reads sequence t)
  const int32_t* idx;          // [T][n]
  int64_t T;
  int H;
  int n;
  float scale;
  uint16_t* out;               // [T][H][512] bf16
  float* lse;                  // [T][H] or null
  uint32_t* status;            // may be null
  // limit of a wait, and the tiles that a block's list warp hands out before it
  // stops as if it had died (no limit but in tests: dsa_test_inject_wait_timeout)
  uint64_t wait_ns = kWaitTimeoutNs;
  int hold_tiles = INT32_MAX;
};
size_t attend_workspace_bytes(int64_t T, int H, int n, int sms);
cudaError_t launch_attend_kv4(const AttendParams& p, void* workspace, int sms, cudaStream_t st);
// More than 64 heads (launch_attend_kv4 and attend_workspace_bytes choose).
size_t attend_pair_workspace_bytes(int64_t T, int H, int n, int sms);
cudaError_t launch_attend_kv4_pair(const AttendParams& p, void* workspace, int sms, cudaStream_t st);

}  // namespace dsa
