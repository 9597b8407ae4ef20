// Attention over the selected keys of a 4-bit latent cache for more than 64
// heads (dsa_attend.cu has the formulas and the kernel for up to 64): clusters
// of two blocks work on one row, 128 of its heads and a range of its list, in
// tiles of 128 keys, with MMAs over both blocks (cta_group::2),
//
//   S [128 heads x 128 keys]  = Q [128 x 576] K^T     (M = 128, N = 128, 36 K steps)
//   O [128 heads x 512]      += P [128 x 128] V       (M = 128, N = 256, 2 x 8 K steps)
//
// Block c holds the queries of heads 64 c .. 64 c + 63, K of the tile's keys
// 64 c .. 64 c + 63 (all dimensions) and V of all 128 keys (latent dimensions
// 256 c .. 256 c + 255), and gets the scores and outputs of its heads: TMEM
// lanes 0-63 the first half of a product's columns, lanes 64-127 the second.
//
// Why pairs: shared memory's 128-byte wavefronts bound these kernels.  64 heads
// of a block on their own move some 3000 for 64 keys; here 128 keys of 128
// heads move 3800 per block (operands of the MMAs 1920, decoding 1088, P 128,
// the rest slots, queries and conflicts) for twice the products, in 5470
// cycles (70% of one a cycle) against 36 x 53 + 16 x 65 = 2950 of MMAs.  2048
// rows of 128 heads and 2048 entries: 1.49 ms among other calls, 786 TFLOP/s;
// 1.32 ms in a burst of five (64-head blocks: 2.14).
//
//   warps 0-3    softmax and output; a thread has one head and half of the keys
//                (output dimensions), so maxima and sums need no shuffles
//   warps 4-11   decode K, eight keys a warp, handed over in four parts of 128
//                dimensions; warps 12-19 decode V, 16 keys a warp, handed over
//                in four parts of 32 keys
//   warps 20-23  stage half of the queries of the next row (the V warps the
//                other half)
//   warp 24      issues the MMAs of S, warp 26 those of O (in the cluster's
//                first block)
//   warp 25      packs the pool rows of the list's entries into tiles
//
// K and V are single buffers that are never idle for long: S of a tile and O
// of the one before run as their operands become ready, K is refilled during O
// and V during S.  The grid is persistent: a cluster takes every n-th row, and
// the next row's queries, keys and scores proceed while the last one's output
// is formed and stored.  What of that boundary still shows is the staging of the
// queries behind the row's last score (some 7000 cycles a row).
//
// Numbers as in dsa_attend.cu: latents exact in fp16, queries fp16 after an
// exact power of two, P fp16 relative to a reference that the weights pass by
// 2^8 at most and times 2^7, scores, sums and outputs fp32.
#include <algorithm>

#include "dsa_attend.cuh"

namespace dsa {

namespace {

constexpr int kTile = 128, kHalf = 64;            // keys of a tile; keys of K and heads of one block
constexpr uint32_t kBlk = kHalf * 128;            // a 64-column block of K, Q or P
constexpr uint32_t kVBlk = kTile * 128;           // a 64-column block of V
constexpr int kNBlk = kKvQ / 64;
constexpr int kK = 4, kV = 12, kQ = 20, kMma = 24, kList = 25, kMmaO = 26;  // first warps of the roles, softmax from 0
constexpr int kPairThreads = 28 * 32;
constexpr int kPairRing = 4;                      // tiles that the list warp may be ahead
// registers per thread: 72 at launch, then shared out by warpgroup
constexpr uint32_t kSoftRegs = 96, kKRegs = 72, kVRegs = 72, kQRegs = 64, kIssueRegs = 56;
static_assert(kSoftRegs * 128 + kKRegs * 256 + kVRegs * 256 + kQRegs * 128 + kIssueRegs * 128 <= 72 * kPairThreads,
              "register pool");

constexpr uint32_t kOffQ = 0, kOffK = kNBlk * kBlk, kOffV = 2 * kNBlk * kBlk, kOffP = kOffV + 4 * kVBlk;
constexpr uint32_t kOffRing = kOffP + 2 * kBlk;                  // pool rows of the next tiles' keys
constexpr uint32_t kOffMeta = kOffRing + kPairRing * kTile * 4;  // keys and flags of the next tiles
constexpr uint32_t kOffC = kOffMeta + kPairRing * 4;             // per head: factor of a score in log2 units
constexpr uint32_t kOffBars = kOffC + kHalf * 4;
// barriers: K full, K empty, V full, V empty [4 parts each], listed, taken
// [ring], scores [2], scores read [2], then P full, output done, Q full, Q empty, factors full,
// factors empty, drain [2]
constexpr int kBarKF = 0, kBarKE = 4, kBarVF = 8, kBarVE = 12, kBarListed = 16, kBarTaken = kBarListed + kPairRing,
              kBarS = kBarTaken + kPairRing, kBarSE = kBarS + 2, kBarP = kBarSE + 2, kBarO = kBarP + 1, kBarQF = kBarO + 1, kBarQE = kBarQF + 1,
              kBarCF = kBarQE + 1, kBarCE = kBarCF + 1, kBarDrain = kBarCE + 1, kBars = kBarDrain + 2;
constexpr uint32_t kOffMisc = kOffBars + 8 * kBars;
constexpr uint32_t kPairSmem = kOffMisc + 16;
static_assert(kOffBars % 8 == 0 && kPairSmem <= 227u * 1024u, "shared memory layout");

// Tile flags next to its number of keys.
constexpr int kFirst = 1 << 16, kLast = 1 << 17, kStop = 1 << 18;

struct PairGrid {
  int head_blocks, splits, tiles;  // tiles: of a whole list
  uint32_t items;                  // T * head_blocks * splits, below 2^31
  float* part_o;                   // [items][128][512]
  float2* part_ml;                 // [items][128]
  uint32_t* err;                   // the workspace's status word
  PageDiv div;
  bool out32;                      // out is 32-byte aligned
};

// A cluster's next item with a row to work on: item k and what it stands for.
struct PairItem {
  uint32_t k;
  int64_t t;
  int hb, split, seq;
};
__device__ __forceinline__ bool next_item(PairItem& it, const AttendParams& p, const PairGrid& g, bool tell) {
  for (; it.k < g.items; it.k += gridDim.x >> 1) {
    const uint32_t row = it.k / static_cast<uint32_t>(g.splits);
    it.split = static_cast<int>(it.k - row * g.splits);
    it.t = row / static_cast<uint32_t>(g.head_blocks);
    it.hb = static_cast<int>(row - static_cast<uint32_t>(it.t) * g.head_blocks);
    it.seq = p.row_seq ? __ldg(p.row_seq + it.t) : static_cast<int>(it.t);
    if (it.seq >= 0 && it.seq < p.B) return true;
    if (it.seq >= p.B && tell) report(p, g.err, kErrOverflow);  // else padding
  }
  return false;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The same barrier in the cluster's first block.
__device__ __forceinline__ uint32_t in_first(uint32_t bar) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(bar));
  return r;
}
// Arrives on a barrier of the cluster's first block.  What the warp wrote to
// its own block's shared memory is released at cluster scope, since the first
// block's MMAs read it; the fence is restricted to shared memory.  (With waits
// to match, a burst of 2048 rows of 128 heads takes 1.32 to 1.35 ms; 1.24 without
// the fences, which the PTX memory model does not allow, 1.60 to 1.96 with
// unrestricted ones.)
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_bar) {
  asm volatile(
      "fence.release.sync_restrict::shared::cta.cluster;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
      : "memory");
}
// Barrier over the two softmax warps of the same heads, with a predicate.
__device__ __forceinline__ bool heads_bar_or(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred.aligned q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}

// 128 latent dimensions of a key, two runs of 64: codes and scales.
struct RawLatent {
  uint32_t code[16];
  uint64_t scale;
};
// Runs number a and b of the entry's eight.
__device__ __forceinline__ void load_latent(RawLatent& r, const uint8_t* entry, int a, int b) {
  uint32_t x[8], y[8];
  ldg256(x, entry + a * 32);
  ldg256(y, entry + b * 32);
  const uint32_t lo = __ldg(reinterpret_cast<const uint32_t*>(entry + kKvScaleOff) + a);
  const uint32_t hi = __ldg(reinterpret_cast<const uint32_t*>(entry + kKvScaleOff) + b);
  r.scale = static_cast<uint64_t>(hi) << 32 | lo;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r.code[i] = x[i];
    r.code[8 + i] = y[i];
  }
}
__device__ __forceinline__ void zero_latent(RawLatent& r) {
#pragma unroll
  for (int i = 0; i < 16; ++i) r.code[i] = 0u;
  r.scale = 0u;
}
// Quarter p of hand-over part s of K holds latent dimensions 256 (s / 2) + 64 p
// + 32 (s % 2) .. + 31, so that the four lanes of a key load 128 contiguous
// bytes at a time.
__device__ __forceinline__ constexpr int part_of(int hi, int lo) { return 2 * hi + lo; }

// Decodes the next 32 dimensions to four chunks of 16 bytes, chunk k at dst +
// ((k ^ swz) << 4), and moves the rest down (a loop over all 128 keeps the
// code small, which counts here: the roles' loops together pass the size of
// the instruction cache).
__device__ __forceinline__ void decode_step(RawLatent& r, uint32_t dst, uint32_t swz) {
  const __half2 sc =
      __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(r.scale & 0xFFFFu), __NV_E4M3));
  const __half2 lo = __low2half2(sc), hi = __high2half2(sc);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t o[4];
    decode8(r.code[k], k < 2 ? lo : hi, o);
    sts128(dst + ((k ^ swz) << 4), o[0], o[1], o[2], o[3]);
  }
  r.scale >>= 16;
#pragma unroll
  for (int k = 0; k < 12; ++k) r.code[k] = r.code[k + 4];
}

__global__ void __launch_bounds__(kPairThreads, 1) attend_kv4_pair_kernel(const AttendParams p, const PairGrid g) {
  extern __shared__ __align__(1024) uint8_t pair_smem[];
  uint8_t* smem = pair_smem;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + kOffQ, sK = sbase + kOffK, sV = sbase + kOffV, sP = sbase + kOffP;
  volatile int* s_ring = reinterpret_cast<volatile int*>(smem + kOffRing);
  volatile int* s_meta = reinterpret_cast<volatile int*>(smem + kOffMeta);
  float* s_c = reinterpret_cast<float*>(smem + kOffC);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 8);
  auto bar = [&](int i) { return sbase + kOffBars + 8 * i; };
  constexpr uint32_t kTmemO = 0, kTmemS = 256;  // O: 2 x 128 columns, S: 2 x 64

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(kBarKF + i), 16);
      mbar_init(bar(kBarKE + i), 1);
      mbar_init(bar(kBarVF + i), 4);
      mbar_init(bar(kBarVE + i), 1);
    }
    for (int i = 0; i < kPairRing; ++i) {
      mbar_init(bar(kBarListed + i), 1);
      mbar_init(bar(kBarTaken + i), rank == 0 ? 22 : 20);  // K, V and softmax warps, the MMA warps
    }
    mbar_init(bar(kBarS), 1);
    mbar_init(bar(kBarS + 1), 1);
    mbar_init(bar(kBarSE), 8);
    mbar_init(bar(kBarSE + 1), 8);
    mbar_init(bar(kBarP), 8);
    mbar_init(bar(kBarO), 1);
    mbar_init(bar(kBarQF), 24);  // Q and V warps
    mbar_init(bar(kBarQE), 1);
    mbar_init(bar(kBarCF), 12);
    mbar_init(bar(kBarCE), 4);
    mbar_init(bar(kBarDrain), 1);
    mbar_init(bar(kBarDrain + 1), 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();

  PairItem it{blockIdx.x >> 1, 0, 0, 0, 0};
  auto wait = [&](int b, uint32_t parity) { return __all_sync(~0u, wait_bar<true>(bar(b), parity & 1u, s_abort, p.wait_ns)); };
  // on a barrier that only this block's warps arrive on
  auto wait_own = [&](int b, uint32_t parity) { return __all_sync(~0u, wait_bar(bar(b), parity & 1u, s_abort, p.wait_ns)); };
  // a tile's entry in the ring, for a warp that reads it
  auto listed = [&](int i) { return wait_own(kBarListed + i % kPairRing, static_cast<uint32_t>(i / kPairRing)); };
  auto taken = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarTaken + i % kPairRing));
  };

  // Queries of rows r0 .. r0 + rows - 1 of this block for its item number n (the
  // first item's are staged below), and the word that they are there.
  auto stage = [&](const PairItem& item, int n, int r0, int rows) {
    if (n > 0) {
      const int h0 = item.hb * 2 * kHalf + rank * kHalf;
      // all rows on their way to L2 during the wait, two at a time from there
      const char* src = reinterpret_cast<const char*>(p.q + (item.t * p.H + h0 + r0) * kKvQ);
      for (int b = lane * 128; b < min(rows, p.H - h0 - r0) * 2 * kKvQ; b += 32 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(src + b));
      auto live = [&](int r) { return h0 + r < p.H; };
      uint4 v[2][3];
      load_query_row(v[0], p, item.t, h0 + r0, live(r0), lane);
      load_query_row(v[1], p, item.t, h0 + r0 + 1, live(r0 + 1), lane);
      if (!wait(kBarQE, n + 1) || !wait_own(kBarCE, n + 1)) return false;
#pragma unroll 1
      for (int r = r0;;) {
        const int two[2] = {r, r + 1};
        store_query_rows<2>(v, p.scale, smem + kOffQ, kBlk, two, s_c, lane, part_of);
        r += 2;
        if (r >= r0 + rows) break;
        load_query_row(v[0], p, item.t, h0 + r, live(r), lane);
        load_query_row(v[1], p, item.t, h0 + r + 1, live(r + 1), lane);
      }
      fence_proxy_async_smem();
    }
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(bar(kBarCF));
      arrive_cluster(in_first(bar(kBarQF)));
    }
    return true;
  };

  // the first row's queries by all warps but the issuing ones and the list's
  if (warp < kMma) {
    PairItem first = it;
    if (next_item(first, p, g, false)) {
      const int h0 = first.hb * 2 * kHalf + rank * kHalf;
#pragma unroll 1
      for (int r = warp; r < kHalf; r += kMma) {
        uint4 v[3];
        load_query_row(v, p, first.t, h0 + r, h0 + r < p.H, lane);
        store_query_row(v, p.scale, smem + kOffQ, kBlk, r, s_c, lane, part_of);
      }
      fence_proxy_async_smem();
    }
    named_bar_sync(3, kMma * 32);
  }

  if (warp >= kMma) {
    regs_dec<kIssueRegs>();
    if (warp == kList) {
      // ------------------------------------------------------------- list
      int tile = 0, keys = 0;  // the open tile, and how many keys it has
      bool ok = true, bad = false, first = true;
      auto publish = [&](int flags) {  // the open tile
        if (lane == 0) s_meta[tile % kPairRing] = keys | flags;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarListed + tile % kPairRing));
      };
      auto turn = [&](int flags) {  // publishes the open tile and opens the next one
        publish(flags);
        ++tile;
        keys = 0;
        ok = wait_own(kBarTaken + tile % kPairRing, static_cast<uint32_t>(tile / kPairRing) + 1u) && tile < p.hold_tiles;
      };
      int j0 = 0, j_hi = 0;  // the item's entries that are left
      const int32_t *table = nullptr, *list = nullptr;
      int pos[4];
      auto fetch = [&] {
#pragma unroll
        for (int k = 0; k < 4; ++k) pos[k] = j0 + 32 * k + lane < j_hi ? __ldg(list + j0 + 32 * k + lane) : -1;
        j0 += 128;
      };
      while (ok && next_item(it, p, g, rank == 0 && lane == 0)) {
        table = p.block_table + static_cast<int64_t>(it.seq) * p.max_blocks;
        list = p.idx + it.t * p.n;
        // below 2^23 tiles and 2^8 splits
        j0 = static_cast<int>(static_cast<uint32_t>(g.tiles) * it.split / static_cast<uint32_t>(g.splits)) * kTile;
        j_hi = min(p.n, static_cast<int>(static_cast<uint32_t>(g.tiles) * (it.split + 1) / static_cast<uint32_t>(g.splits)) * kTile);
        first = true;
        fetch();
#pragma unroll 1
        for (int left = (j_hi - j0 + 255) >> 7; left > 0 && ok; --left) {  // steps of 128 entries
          int slot[4];
          slots_of(p, g.div, table, pos, slot, bad);
          fetch();
#pragma unroll 1
          for (int k = 0; k < 4 && ok; ++k) {
            int mine = slot[0];
            slot[0] = slot[1];
            slot[1] = slot[2];
            slot[2] = slot[3];
            const uint32_t m = __ballot_sync(~0u, mine >= 0);
            int at = keys + __popc(m & lanemask_lt());
            if (mine >= 0 && at < kTile) s_ring[tile % kPairRing * kTile + at] = mine;
            keys += __popc(m);
            if (keys > kTile) {  // the rest starts the next tile, so this one is not the last
              const int rest = keys - kTile;
              keys = kTile;
              turn(first ? kFirst : 0);
              first = false;
              if (mine >= 0 && at >= kTile) s_ring[tile % kPairRing * kTile + at - kTile] = mine;
              keys = rest;
            }
          }
        }
        it.k += gridDim.x >> 1;
        if (ok) turn(kLast | (first ? kFirst : 0));  // without keys where nothing is listed
      }
      if (ok && tile + 1 < p.hold_tiles) publish(kStop);
      if (__any_sync(~0u, bad) && rank == 0 && lane == 0) report(p, g.err, kErrOverflow);
    } else if (warp == kMma && rank == 0) {
      // -------------------------------------------------- MMAs of the scores
      constexpr uint32_t tmem = 0;  // all 512 columns are allocated
      constexpr uint32_t kIdS = idesc_att(128, 128, 0, 0, 0), kIdR = idesc_att(128, 128, 1, 0, 0);
      const uint64_t dQ = smem_desc_sw128(sQ), dK = smem_desc_sw128(sK);
      const uint32_t leader = elect_one();
      bool ok = true;
      int n_items = 0;
      for (int i = 0;; ++i) {
        if (!listed(i)) break;
        const int meta = s_meta[i % kPairRing];
        taken(i);
        if (meta & kStop) break;
        if ((meta & kFirst) && !wait(kBarQF, n_items++)) break;
        if (!wait(kBarSE + (i & 1), static_cast<uint32_t>(i >> 1) + 1u)) break;  // scores of tile i - 2 are read
        const uint32_t d = tmem + kTmemS + 64 * (i & 1);
        uint32_t ready = 0;  // of the four parts
#pragma unroll 1
        for (int s = 0; s < 4; ++s) {
          if (!((ready >> s) & 1u)) {
            if (!(ok = wait_any<true>(ready, s, lane < 4, bar(kBarKF + (lane & 3)), i & 1, s_abort, p.wait_ns))) break;
            tc_fence_after();
          }
          const uint64_t q0 = dQ + (2 * s * kBlk >> 4), k0 = dK + (2 * s * kBlk >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t o = ((k >> 2) * kBlk + 32 * (k & 3)) >> 4;
            mma_if<2>(leader, d, q0 + o, k0 + o, kIdS, s > 0 || k > 0);
          }
          if (s == 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_if<2>(leader, d, dQ + ((8 * kBlk + 32 * k) >> 4), dK + ((8 * kBlk + 32 * k) >> 4), kIdR, 1);
          }
          commit_pair_if(leader, bar(kBarKE + s));
          if (s == 3) {
            commit_pair_if(leader, bar(kBarS + (i & 1)));
            if (meta & kLast) commit_pair_if(leader, bar(kBarQE));
          }
        }
        if (!ok) break;
      }
      // nothing may be in flight when the tensor memory is freed (also after a wait that gave up)
      commit_pair_if(leader, bar(kBarDrain));
      int unused = 0;
      if (!wait_bar<true>(bar(kBarDrain), 0, &unused, p.wait_ns)) *s_abort = 1;
      __syncwarp();
    } else if (warp == kMmaO && rank == 0) {
      // ------------------------------------------------- MMAs of the outputs
      constexpr uint32_t tmem = 0;  // all 512 columns are allocated
      constexpr uint32_t kIdO = idesc_att(128, 256, 0, 0, 1);
      const uint64_t dP = smem_desc_sw128(sP), dV = desc_mn_sw128(sV, kVBlk);
      const uint32_t leader = elect_one();
      bool ok = true;
      for (int i = 0;; ++i) {
        if (!listed(i)) break;
        const int meta = s_meta[i % kPairRing];
        taken(i);
        if (meta & kStop) break;
        // lane by lane: the four parts of V, the weights
        const uint32_t mine = bar(lane == 4 ? kBarP : kBarVF + (lane & 3));
        uint32_t ready = 0;
        if (!wait_any<true>(ready, 4, lane < 5, mine, i & 1, s_abort, p.wait_ns)) break;
        tc_fence_after();
#pragma unroll 1
        for (int u = 0; u < 4; ++u) {
          if (!((ready >> u) & 1u)) {
            if (!(ok = wait_any<true>(ready, u, lane < 5, mine, i & 1, s_abort, p.wait_ns))) break;
            tc_fence_after();
          }
          const uint64_t a0 = dP + (((u >> 1) * kBlk + 64 * (u & 1)) >> 4), b0 = dV + (2 * u * 2048 >> 4);
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              mma_if<2>(leader, tmem + kTmemO + 128 * j, a0 + 2 * kk, b0 + ((kk * 2048 + 2 * j * kVBlk) >> 4), kIdO,
                        !((meta & kFirst) && u == 0 && kk == 0));
          }
          commit_pair_if(leader, bar(kBarVE + u));
          if (u == 3) commit_pair_if(leader, bar(kBarO));
        }
        if (!ok) break;
      }
      commit_pair_if(leader, bar(kBarDrain + 1));
      int unused = 0;
      if (!wait_bar<true>(bar(kBarDrain + 1), 0, &unused, p.wait_ns)) *s_abort = 1;
      __syncwarp();
    }
  } else if (warp >= kQ) {
    // ----------------------------------------------------------- queries
    regs_dec<kQRegs>();
    bool ok = true;
    for (int n = 0; ok && next_item(it, p, g, false); it.k += gridDim.x >> 1, ++n) ok = stage(it, n, 8 * (warp - kQ), 8);
  } else if (warp >= kV) {
    // ----------------------------------------------------------------- V
    const int lw = warp - kV, key = lw * 16 + (lane & 15), half = lane >> 4, u = lw >> 1;
    const uint32_t row = sV + half * kVBlk + key * 128, sw = static_cast<uint32_t>(key & 7);
    const uint32_t full = in_first(bar(kBarVF + u));
    RawLatent raw;
    int meta = 0, n = 0;
    bool ok = next_item(it, p, g, false) && stage(it, n, 32 + 4 * lw, 4);
    for (int i = -1; ok; ++i) {  // loads of tile i + 1, then tile i to shared memory
      if (!listed(i + 1)) break;
      RawLatent next;
      const int m = s_meta[(i + 1) % kPairRing];
      if (key < (m & 0xFFFF))
        load_latent(next, p.kv + static_cast<int64_t>(s_ring[(i + 1) % kPairRing * kTile + key]) * kKvEntry, 4 * rank + half,
                    4 * rank + 2 + half);
      else
        zero_latent(next);
      taken(i + 1);
      if (i >= 0) {
        if (!wait(kBarVE + u, i + 1)) break;
#pragma unroll 1
        for (int s = 0; s < 4; ++s) decode_step(raw, row + (s & 2) * kVBlk + ((((4 * s) ^ sw) & 4) << 4), sw & 3);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive_cluster(full);
        if (meta & kLast) {  // half of the next row's queries: V has the time, K has not
          it.k += gridDim.x >> 1;
          if (next_item(it, p, g, false)) ok = stage(it, ++n, 32 + 4 * lw, 4);
        }
      }
      if (m & kStop) break;
      raw = next;
      meta = m;
    }
  } else if (warp >= kK) {
    // ----------------------------------------------------------------- K
    const int lw = warp - kK, key = lw * 8 + (lane & 7), part = lane >> 3;
    const uint32_t row = sK + (part >> 1) * kBlk + key * 128, sw = static_cast<uint32_t>(key & 7);
    const uint32_t full = in_first(bar(kBarKF));
    RawLatent raw;
    uint32_t rope[8];
    bool ok = true;
    for (int i = -1; ok; ++i) {  // loads of tile i + 1, then tile i to shared memory
      if (!listed(i + 1)) break;
      RawLatent next;
      uint32_t next_rope[8];
      const int m = s_meta[(i + 1) % kPairRing];
      if (rank * kHalf + key < (m & 0xFFFF)) {
        const uint8_t* e =
            p.kv + static_cast<int64_t>(s_ring[(i + 1) % kPairRing * kTile + rank * kHalf + key]) * kKvEntry;
        load_latent(next, e, part, 4 + part);
        ldg256(next_rope, e + kKvRopeOff + part * 32);
      } else {
        zero_latent(next);
#pragma unroll
        for (int x = 0; x < 8; ++x) next_rope[x] = 0u;
      }
      taken(i + 1);
      if (i >= 0) {
        uint32_t ready = 0;  // of the four parts
#pragma unroll 1
        for (int s = 0; s < 4; ++s) {
          if (!(ok = wait_any<true>(ready, s, lane < 4, bar(kBarKE + (lane & 3)), (i + 1) & 1, s_abort, p.wait_ns))) break;
          if (s == 0) {
            const uint32_t dst = sK + 8 * kBlk + key * 128;
            sts128(dst + (((2 * part) ^ sw) << 4), rope[0], rope[1], rope[2], rope[3]);
            sts128(dst + (((2 * part + 1) ^ sw) << 4), rope[4], rope[5], rope[6], rope[7]);
          }
          decode_step(raw, row + 2 * s * kBlk + ((((4 * part) ^ sw) & 4) << 4), sw & 3);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) arrive_cluster(full + 8 * s);
        }
      }
      if (m & kStop) break;
      raw = next;
#pragma unroll
      for (int x = 0; x < 8; ++x) rope[x] = next_rope[x];
    }
  } else {
    // ----------------------------------------------------------- softmax
    regs_inc<kSoftRegs>();
    const uint32_t tmem = static_cast<uint32_t>(warp * 32) << 16;
    const int row = tid & (kHalf - 1), part = tid >> 6;  // head; half of the keys and of the dimensions
    const int bar_id = 1 + (warp & 1);
    const uint32_t full = in_first(bar(kBarP)), read = in_first(bar(kBarSE));
    const uint32_t p_row = sP + part * kBlk + row * 128, sw = static_cast<uint32_t>(row & 7);
    // a word of this thread's and its partner's rows of P, while P is not in use
    volatile float* mine = reinterpret_cast<volatile float*>(smem + kOffP + part * kBlk + row * 128);
    volatile float* other = reinterpret_cast<volatile float*>(smem + kOffP + (part ^ 1) * kBlk + row * 128);
    bool ok = true;
    int i = 0;
    for (int n = 0; ok && next_item(it, p, g, false); it.k += gridDim.x >> 1, ++n) {
      bool some = false;  // the row (its part) has keys
      float c = 0.f, m = 0.f, l = 0.f;  // factor to log2 units, kLift less the reference (from the first tile on), sum
      for (bool first = true, last = false; !last; first = false, ++i) {
        int n_keys = 0;
        if (listed(i)) {
          const int meta = s_meta[i % kPairRing];
          last = meta & kLast;
          some |= (meta & 0xFFFF) > 0;
          n_keys = (meta & 0xFFFF) - part * kHalf;  // of this thread's half
          taken(i);
        } else {
          ok = false;
        }
        ok = wait(kBarS + (i & 1), static_cast<uint32_t>(i >> 1)) && ok;
        if (first) {
          ok = wait_own(kBarCF, n) && ok;
          c = s_c[row];
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarCE));
        }
        tc_fence_after();
        const uint32_t ts = tmem + kTmemS + 64 * (i & 1);
        // 32 scores, relative to the reference, plus kLift, -inf behind the last key
        float x[32];
        auto scores = [&](int q) {
          tmem_ld32(ts + 32 * q, reinterpret_cast<uint32_t(&)[32]>(x));
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const float2 a = __ffma2_rn(make_float2(x[k], x[k + 1]), make_float2(c, c), make_float2(m, m));
            x[k] = a.x;
            x[k + 1] = a.y;
          }
          if (n_keys < kHalf) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (32 * q + k >= n_keys) x[k] = -INFINITY;
          }
        };
        float mx = -INFINITY;
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          scores(q);
#pragma unroll
          for (int k = 0; k < 32; k += 2) mx = fmaxf(mx, fmaxf(x[k], x[k + 1]));
        }
        // the same decision in both warps of these heads; a wait that gave up goes this way too
        if (heads_bar_or(bar_id, !ok || first || mx > kRise + kLift)) {
          if (!first) ok = wait(kBarO, i - 1) && ok;
          if (heads_bar_or(bar_id, !ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
          *mine = mx - m;
          named_bar_sync(bar_id, 64);
          float top = fmaxf(mx - m, *other);
          if (!first) top = fmaxf(top, kLift - m);
          if (top == -INFINITY) top = 0.f;  // no keys so far
          const float to = kLift - top, f = first ? 1.f : ex2(to - m);
          m = to;
          l *= f;
          named_bar_sync(bar_id, 64);
          if (!first) {
#pragma unroll 1
            for (int q = 0; q < 256; q += 16) {
              uint32_t o[16];
              tmem_ld16(tmem + kTmemO + q, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st16(tmem + kTmemO + q, o);
            }
            tmem_wait_st();
          }
        } else {
          // P of the last tile has to be consumed before it is overwritten
          ok = wait(kBarO, i - 1) && ok;
        }
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          scores(q);
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const float2 a = make_float2(ex2(x[k]), ex2(x[k + 1]));
            sum = __fadd2_rn(sum, a);
            const __half2 h = __floats2half2_rn(a.x, a.y);
            w[k >> 1] = *reinterpret_cast<const uint32_t*>(&h);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            sts128(p_row + (((4 * q + k) ^ sw) << 4), w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        }
        l += sum.x + sum.y;
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive_cluster(full);
          arrive_cluster(read + 8 * (i & 1));
        }
      }
      // ---------------------------------------------------------- output
      ok = ok && wait(kBarO, i - 1);
      if (heads_bar_or(bar_id, !ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      *mine = l;
      named_bar_sync(bar_id, 64);
      l += *other;
      named_bar_sync(bar_id, 64);
      const int h = it.hb * 2 * kHalf + rank * kHalf + row;
      const int64_t part_row = static_cast<int64_t>(it.k) * 2 * kHalf + rank * kHalf + row;
      const float f = g.splits > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;
      if (part == 0 && h < p.H) {
        // NaN or infinite scores; with finite ones the reference's own weight counts
        if (!(l < INFINITY) || (l == 0.f && some)) report(p, g.err, kErrNonFinite);
        if (g.splits > 1)
          g.part_ml[part_row] = make_float2(l == 0.f ? -INFINITY : -m, l);
        else if (p.lse)
          p.lse[it.t * p.H + h] = l == 0.f ? -INFINITY : (log2f(l) - m) * kLn2;
      }
#pragma unroll 1
      for (int q = 0; q < 8; ++q) {  // 32 dimensions
        uint32_t o[32];
        tmem_ld32(tmem + kTmemO + 32 * q, o);
        tmem_wait_ld();
        const int dim = 256 * part + 32 * q;
        if (h >= p.H) {
          // no such head
        } else if (g.splits > 1) {
          float* dst = g.part_o + part_row * kKvLat + dim;
#pragma unroll
          for (int k = 0; k < 4; ++k) stg256(dst + 8 * k, o + 8 * k);
        } else {
          uint32_t b[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const __nv_bfloat162 y =
                __floats2bfloat162_rn(__uint_as_float(o[2 * k]) * f, __uint_as_float(o[2 * k + 1]) * f);
            b[k] = *reinterpret_cast<const uint32_t*>(&y);
          }
          uint16_t* dst = p.out + (it.t * p.H + h) * kKvLat + dim;
          if (g.out32) {  // whole sectors
            stg256(dst, b);
            stg256(dst + 16, b + 8);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              reinterpret_cast<uint4*>(dst)[k] = make_uint4(b[4 * k], b[4 * k + 1], b[4 * k + 2], b[4 * k + 3]);
          }
        }
        __syncwarp();
      }
      tc_fence_before();
    }
  }
  // a block's memory and barriers are in use until its partner is done too
  __syncwarp();
  cluster_sync();
  if (tid == 0 && *s_abort) report(p, g.err, kErrTimeout);
  if (warp == kMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(*s_tmem) : "memory");
  }
}

// Joins the splits of one (row, head): out = sum_s 2^(m_s - m) O_s / sum_s
// 2^(m_s - m) l_s.
__global__ void __launch_bounds__(128) attend_pair_join_kernel(const AttendParams p, const PairGrid g) {
  const int64_t t = blockIdx.x / p.H;
  const int h = static_cast<int>(blockIdx.x % p.H);
  const int seq = p.row_seq ? __ldg(p.row_seq + t) : static_cast<int>(t);
  if (seq < 0 || seq >= p.B) return;
  const int64_t row0 = (t * g.head_blocks + h / kTile) * g.splits * kTile + h % kTile;
  float m = -INFINITY;
  for (int s = 0; s < g.splits; ++s) m = fmaxf(m, g.part_ml[row0 + s * kTile].x);
  const float ref = m == -INFINITY ? 0.f : m;
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < g.splits; ++s) {
    const float2 ml = g.part_ml[row0 + s * kTile];
    const float w = ex2(ml.x - ref);
    const float4 o = reinterpret_cast<const float4*>(g.part_o + (row0 + s * kTile) * kKvLat)[threadIdx.x];
    sum = fmaf(w, ml.y, sum);
    acc.x = fmaf(w, o.x, acc.x);
    acc.y = fmaf(w, o.y, acc.y);
    acc.z = fmaf(w, o.z, acc.z);
    acc.w = fmaf(w, o.w, acc.w);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  reinterpret_cast<uint2*>(p.out + (t * p.H + h) * kKvLat)[threadIdx.x] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  if (p.lse && threadIdx.x == 0) p.lse[t * p.H + h] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * kLn2;
}

struct PairPlan {
  int head_blocks, splits, tiles;
  int64_t items;
  size_t off_o, bytes;
};

PairPlan plan_pair(int64_t T, int H, int n, int sms) {
  PairPlan P{};
  P.head_blocks = (H + 2 * kHalf - 1) / (2 * kHalf);
  P.tiles = (n + kTile - 1) / kTile;
  const int64_t rows = T * P.head_blocks, clusters = std::max(sms / 2, 1);
  P.splits = rows >= clusters || rows == 0 ? 1 : static_cast<int>(std::min<int64_t>(clusters / rows, P.tiles));
  P.items = rows * P.splits;
  P.bytes = kAttHeader;
  if (P.splits > 1) {
    const size_t part_rows = static_cast<size_t>(P.items) * 2 * kHalf;
    P.off_o = (kAttHeader + part_rows * sizeof(float2) + 255) / 256 * 256;
    P.bytes = P.off_o + part_rows * kKvLat * sizeof(float);
  }
  return P;
}

}  // namespace

size_t attend_pair_workspace_bytes(int64_t T, int H, int n, int sms) { return plan_pair(T, H, n, sms).bytes; }

cudaError_t launch_attend_kv4_pair(const AttendParams& p, void* workspace, int sms, cudaStream_t st) {
  const PairPlan P = plan_pair(p.T, p.H, p.n, sms);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PairGrid g{P.head_blocks, P.splits, P.tiles, static_cast<uint32_t>(P.items), reinterpret_cast<float*>(ws + P.off_o),
             reinterpret_cast<float2*>(ws + kAttHeader), reinterpret_cast<uint32_t*>(ws),
             page_div(p.page_size), reinterpret_cast<uintptr_t>(p.out) % 32 == 0};
  cudaError_t e = cudaFuncSetAttribute(attend_kv4_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
  if (e != cudaSuccess) return e;
  if ((e = cudaMemsetAsync(g.err, 0, kAttHeader, st)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<int64_t>(P.items, std::max(sms / 2, 1))));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attend_kv4_pair_kernel, p, g);
  if (e != cudaSuccess || P.splits == 1) return e;
  attend_pair_join_kernel<<<static_cast<unsigned>(p.T * p.H), 128, 0, st>>>(p, g);
  return cudaGetLastError();
}

}  // namespace dsa
