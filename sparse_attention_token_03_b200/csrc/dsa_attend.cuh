// Device parts shared by the attention kernels over the 4-bit latent cache
// (dsa_attend.cu, dsa_attend_pair.cu): operand descriptors, decoding, query
// staging and the list walk.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dsa_ptx.cuh"
#include "dsa_serve.cuh"

namespace dsa {

constexpr int kAttHeader = 256, kAttCounter = 128;  // bytes: start of a workspace, cleared by a launch: status word, row counter
// log2 of the largest weight over the reference's before the reference moves, and
// of the factor that all weights carry: fp16 holds weights from 2^-24 to below
// 2^16, so a weight is 0 only below 2^-32 of the reference's.
constexpr float kRise = 8.f, kLift = 7.f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

// Status bits of a call: into its workspace's word, which the launch clears, and
// into the caller's.
__device__ __forceinline__ void report(const AttendParams& p, uint32_t* word, uint32_t bits) {
  atomicOr(word, bits);
  if (p.status) atomicOr(p.status, bits);
}

// Looks at a barrier that warps of the partner block or an MMA over both blocks
// arrive on (arrive_cluster, commit_pair_if): the acquiring fence has cluster
// scope, restricted to shared memory, the only memory that the blocks of a pair
// share (an unrestricted one would order the loads of cache entries too).
__device__ __forceinline__ void acquire_cluster() {
  asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_test_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  acquire_cluster();
  return ok != 0;
}

// mbar_wait in fewer instructions (the roles of these kernels wait at some
// thirty places, and their loops share one instruction cache: the clock is
// read and the abort flag looked at after every 256 tries; a wait that gives up
// sets the flag, which the kernel reports at its end).  kPair: acquires at cluster
// scope.
template <bool kPair = false>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t n = 1; !(kPair ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)); ++n) {
    if (n & 255u) continue;
    const uint64_t now = globaltimer();
    if (t0 == 0) t0 = now;
    if (*abort_flag) return false;
    if (now - t0 > limit_ns) {
      *abort_flag = 1;
      return false;
    }
  }
  if constexpr (kPair) acquire_cluster();
  return true;
}

// tcgen05.mma and tcgen05.commit by one lane (`leader`, from elect_one) under a
// predicate instead of a branch, so that the warp stays converged (elect_one has
// the measured difference).
template <int kGroup>
__device__ __forceinline__ void mma_if(uint32_t leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (kGroup == 1)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(leader)
      : "memory");
}
// The same on this barrier of both blocks of a pair.
__device__ __forceinline__ void commit_pair_if(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(bar),
      "r"(leader)
      : "memory");
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits until bit `which` of `ready` is set, bit j telling that lane j's
// barrier (if `has`) has passed its phase.  A look at a barrier takes some 300
// cycles while the tensor core reads shared memory, so a warp that needs
// several in turn looks at all of them at once and only again for those that
// were not ready.  The vote tells the other lanes that a phase is complete, but
// orders no memory: __syncwarp hands them what the looking lane acquired.
template <bool kPair = false>
__device__ __forceinline__ bool wait_any(uint32_t& ready, int which, bool has, uint32_t bar, uint32_t parity,
                                         volatile int* abort_flag, uint64_t limit_ns) {
  if (!((ready >> which) & 1u)) {
    ready = __ballot_sync(~0u, has && (kPair ? mbar_test_cluster(bar, parity) : mbar_test(bar, parity)));
    __syncwarp();
    if (!((ready >> which) & 1u)) {
      // the blocking look: polling would take the shared memory's time
      const bool ok = wait_bar<kPair>(__shfl_sync(~0u, bar, which), __shfl_sync(~0u, parity, which), abort_flag, limit_ns);
      if (!__all_sync(~0u, ok)) return false;
      ready |= 1u << which;
    }
  }
  return true;
}

__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t addr, uint32_t mn_stride) {
  // M- or N-major operand: rows of 64 consecutive M (N) elements, 8 K rows per
  // 1024-byte atom; mn_stride between 64-element groups, 1024 between K groups
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((mn_stride >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// Instruction descriptors (kind::f16, fp32 accumulation): operand format 0 =
// fp16, 1 = bf16; bits 15 and 16 mark M- and N-major operands.
constexpr uint32_t idesc_att(int M, int N, uint32_t fmt, uint32_t m_major, uint32_t n_major) {
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (m_major << 15) | (n_major << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Eight E2M1 codes of a word to four fp16 pairs, times the block's scale pair.
__device__ __forceinline__ void decode8(uint32_t w, __half2 s, uint32_t (&o)[4]) {
  uint32_t v[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&v[i]), s);
    o[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

__device__ __forceinline__ void ldg256(uint32_t (&r)[8], const void* p) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "l"(p));
}

__device__ __forceinline__ void stg256(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Pool rows of four list entries of a sequence (its block table `table`), or -1
// where nothing is listed or the position or page is outside its range, which
// sets `bad`.  The four table loads are in flight together.
__device__ __forceinline__ void slots_of(const AttendParams& p, PageDiv div, const int32_t* table, const int (&pos)[4], int (&slot)[4],
                                         bool& bad) {
  int blk[4], page[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    blk[k] = div(max(pos[k], 0));
    page[k] = __ldg(table + min(blk[k], p.max_blocks - 1));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool in = blk[k] < p.max_blocks && page[k] >= 0 && page[k] < p.n_pages;
    bad |= pos[k] >= 0 && !in;
    slot[k] = pos[k] >= 0 && in ? page[k] * p.page_size + (pos[k] - blk[k] * p.page_size) : -1;
  }
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A query row as its warp's lanes hold it: 72 16-byte chunks, 64 latent and 8
// rotary; zeros for a head past the last.
constexpr int kQChunks = kKvQ / 8;
__device__ __forceinline__ void load_query_row(uint4 (&v)[3], const AttendParams& p, int64_t t, int h, bool live, int lane) {
  const uint4* src = reinterpret_cast<const uint4*>(p.q + (t * p.H + h) * kKvQ);
#pragma unroll
  for (int i = 0; i < 3; ++i)
    v[i] = live && lane + 32 * i < kQChunks ? __ldg(src + lane + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
}

// Row r of the staged queries: latent parts to fp16 and rotary parts to bf16,
// both times the power of two that puts the row's largest magnitude in [2^14,
// 2^15); s_c[r] takes the factor of its scores in log2 units.  Column blocks
// 2 s and 2 s + 1 (of q_block bytes) hold hand-over part s: the 32 dimensions
// of quarter p of it are the latent dimensions 256 hi + 64 p + 32 lo .. + 31
// with s = part_of(hi, lo); block 8 holds the rotary ones.  Few instructions
// rather than fast ones: this runs once a row, from a cold instruction cache.
// R rows at once, since one row is a chain of dependent instructions.
template <int R, typename PartOf>
__device__ __forceinline__ void store_query_rows(const uint4 (&v)[R][3], float scale, uint8_t* smem, uint32_t q_block,
                                                 const int (&r)[R], float* s_c, int lane, PartOf part_of) {
  uint32_t m[R];  // largest magnitude as bf16 bits (two lanes of 16)
  float up[R];
#pragma unroll
  for (int w = 0; w < R; ++w) {
    m[w] = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      m[w] = __vmaxu2(m[w], __vmaxu2(v[w][i].x & 0x7FFF7FFFu, v[w][i].y & 0x7FFF7FFFu));
      m[w] = __vmaxu2(m[w], __vmaxu2(v[w][i].z & 0x7FFF7FFFu, v[w][i].w & 0x7FFF7FFFu));
    }
  }
#pragma unroll
  for (int w = 0; w < R; ++w) {
    m[w] = __reduce_max_sync(~0u, max(m[w] & 0xFFFFu, m[w] >> 16));
    const int e = min(141 - static_cast<int>(m[w] >> 7), 126);  // biased exponent field -> shift
    up[w] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    // the power of two first: a large scale on a small row may pass fp32 times log2 e
    if (lane == 0) s_c[r[w]] = scale * __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * kLog2e;
  }
  uint4 now[R], next[R], last[R];
#pragma unroll
  for (int w = 0; w < R; ++w) now[w] = v[w][0], next[w] = v[w][1], last[w] = v[w][2];
#pragma unroll 1
  for (int c = lane; c < kQChunks; c += 32) {
    const bool rotary = c >= kKvLat / 8;
    const int p = (c >> 3) & 3;
    const int blk = rotary ? 8 : 2 * part_of(c >> 5, (c >> 2) & 1) + (p >> 1);
    const int at = rotary ? c & 7 : 4 * (p & 1) + (c & 3);
#pragma unroll
    for (int w = 0; w < R; ++w) {
      uint32_t u[4] = {now[w].x, now[w].y, now[w].z, now[w].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = __uint_as_float(u[k] << 16) * up[w], b = __uint_as_float(u[k] & 0xFFFF0000u) * up[w];
        const __half2 h = __floats2half2_rn(a, b);
        const __nv_bfloat162 f = __floats2bfloat162_rn(a, b);
        u[k] = rotary ? *reinterpret_cast<const uint32_t*>(&f) : *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(smem + blk * q_block + r[w] * 128 + ((at ^ (r[w] & 7)) << 4)) =
          make_uint4(u[0], u[1], u[2], u[3]);
      now[w] = next[w];
      next[w] = last[w];
    }
  }
}
template <typename PartOf>
__device__ __forceinline__ void store_query_row(const uint4 (&v)[3], float scale, uint8_t* smem, uint32_t q_block, int r,
                                                float* s_c, int lane, PartOf part_of) {
  const uint4 one[1][3] = {{v[0], v[1], v[2]}};
  const int rows[1] = {r};
  store_query_rows<1>(one, scale, smem, q_block, rows, s_c, lane, part_of);
}

}  // namespace dsa
