// Attention of all query heads over the selected keys of a 4-bit latent cache
// (dsa_attend_kv4): for row t, head h and the entries j of the row's list
//
//   z(t,h,j) = scale * (q(t,h) . [latent_j, rotary_j])
//   out(t,h) = sum_j softmax_j(z) latent_j,   lse(t,h) = log sum_j exp z
//
// A block works on one row, all its heads (up to 64) and a range of its list, in
// tiles of 64 keys (dsa_attend_pair.cu has the kernel for more heads).  Both
// products have the keys' or the latent dimensions as the MMA's rows and the
// heads as its columns,
//
//   S^T [64 keys x heads]  = K [64 x 576] Q^T         (M = 64,  36 K steps)
//   O^T [512 x heads]     += V^T [512 x 64] P^T       (M = 128, 4 x 4 K steps)
//
// so that O^T of 64 heads takes 256 of the 512 TMEM columns (heads as rows
// would fill all of them with O alone) and few heads cost their columns, in
// blocks of 16, 32 or 64.  K and V are the same decoded tile: 64-dimension column
// blocks of [64 keys][128 bytes] with the 128-byte swizzle, read K-major for
// S and M-major for O.
//
//   warps 0-3     softmax: S^T from TMEM, exp2, P^T to shared memory; at the
//                 end of a row O^T from TMEM to the output
//   warps 4-19    gather and decode: eight lanes per key load its 416 bytes one
//                 tile ahead into registers, E2M1 -> fp16 times the block scale
//                 (exact), and store the swizzled tile, two tile buffers; they
//                 also stage the queries of the next row
//   warps 20, 23  issue the MMAs of S, one for each tile buffer
//   warp 22       issues the MMAs of O
//   warp 21       reads the list and the block table and packs the pool rows of
//                 the entries that name a key into tiles, so that gaps and
//                 short lists cost no tiles
//
// A tile buffer is handed over in four parts of 128 dimensions, both ways:
// O^T's product over a part frees it, so the next tile's decoding and scores
// follow part by part.  The gathering warps are two groups of eight; each
// lane decodes 64 consecutive dimensions of its key, 32 for each of its
// group's two parts (dim_of gives the order; staged queries and output rows
// follow it).
//
// The grid is persistent: a block takes rows as it gets free, and the next
// row's lists, queries, keys and scores proceed while the last one's output is
// formed and stored (a block per row: 85 us where this takes 70, 501 rows of 16
// heads and 512 entries).
//
// What bounds it: with 64 heads the 128-byte wavefronts of shared memory, some
// 3000 a tile (operands of the MMAs 1920, decoding 576, the rest P, slots and
// conflicts: 74% of one a cycle) in some 4100 cycles against 1970 cycles of MMAs;
// with few heads the way round a tile buffer (decode, S, softmax, O: some 6000
// cycles for two tiles in flight).  999 rows of 64 heads and 2048 entries: 469 us
// among other calls, 607 TFLOP/s (492 us in a burst of five: power); 148 rows of
// 16 heads: 63 us.
//
// Numbers: the latents are exact in fp16 (code x scale has 6 significant
// bits, 2^-10 .. 2688).  Queries go to fp16 too, each row scaled by the power
// of two that puts its largest magnitude in [2^14, 2^15): bf16's 8 bits fit,
// and only values below 2^-28 of that maximum round, to 2^-39 of it.  The
// rotary parts multiply as bf16 (same power of two, exact).  P is fp16, 2^-11
// relative (bf16's 2^-8 would double the output's error).  exp2 is taken
// relative to a reference per head, the maximum of the first tile, that moves
// to the running maximum when a weight passes the reference's by 2^8, so O^T in
// TMEM is rescaled only then, which ordinary score distributions never need.
// All weights carry a factor of 2^7, so that they fill fp16's range: at most
// 2^15, and each off by at most 2^-32 of the reference's below its normal range.
// The sums take the unrounded weights.  Scores, sums and O^T are fp32.
//
// Few rows: the list is split over blocks, each writes its fp32 O and (m, l),
// and a second kernel joins them.
#include <algorithm>

#include "dsa_attend.cuh"

namespace dsa {

namespace {

constexpr int kKt = 64;                          // keys per tile
constexpr int kBlocks = kKvQ / 64;               // 64-dimension column blocks: 8 latent, 1 rotary
constexpr int kParts = kKvLat / 128;             // hand-over parts of a tile buffer
constexpr uint32_t kBlockBytes = kKt * 128;      // one column block
constexpr uint32_t kTileBytes = kBlocks * kBlockBytes;
constexpr int kSoftWarps = 4, kLoadWarps = 16;   // loaders: two groups of 8 warps, 8 keys a warp
constexpr int kMmaWarp = kSoftWarps + kLoadWarps, kListWarp = kMmaWarp + 1, kMmaOWarp = kMmaWarp + 2,
              kMmaOddWarp = kMmaWarp + 3;
constexpr int kAttThreads = (kMmaWarp + 4) * 32;
constexpr int kWorkThreads = (kSoftWarps + kLoadWarps) * 32;
// registers per thread: 80 at launch, then shared out by warpgroup
constexpr uint32_t kSoftRegs = 136, kLoadRegs = 72, kIssueRegs = 56;
static_assert(kSoftRegs * 128 + kLoadRegs * 512 + kIssueRegs * 128 <= 80 * kAttThreads, "register pool");
constexpr int kRing = 4;                         // tiles of slots that the list warp may be ahead
// Tile word: keys, flags, and the number of the block's row modulo 256.
constexpr int kLast = 1 << 16, kStop = 1 << 17, kRowShift = 20;
constexpr int kSoftThreads = kSoftWarps * 32;
template <int NH>
struct AttSmem {
  static constexpr int q_bufs = NH <= 32 ? 2 : 1;        // rows of queries that fit next to the tile buffers
  static constexpr uint32_t q_block = NH * 128, q_bytes = kBlocks * q_block;
  static constexpr uint32_t off_k = (q_bufs * q_bytes + 1023) / 1024 * 1024;
  static constexpr uint32_t off_p = off_k + 2 * kTileBytes;
  static constexpr uint32_t off_c = off_p + kKt * 128;   // [2 rows] per head: factor of a score in log2 units
  static constexpr uint32_t off_f = off_c + 2 * NH * 4;  // per head: rescaling factor, then 1 / sum
  static constexpr uint32_t off_m = off_f + NH * 4;      // per head: reference less kLift, for the statistics
  static constexpr uint32_t off_ring = off_m + NH * 4;   // pool rows of the next tiles' keys
  static constexpr uint32_t off_count = off_ring + kRing * kKt * 4;  // words of the ring tiles, then of the buffers
  static constexpr uint32_t off_bars = off_count + 2 * (kRing + 2) * 4;  // and their items
  // part full and empty [2 buffers][4], ring full and empty, scores [2], scores read [2], queries full [2],
  // queries free [2], factors free [2], weights, output, drain [3]
  static constexpr uint32_t n_bars = 4 * kParts + 2 * kRing + 10 + 5;
  static constexpr uint32_t off_misc = off_bars + 8 * n_bars;
  static constexpr uint32_t bytes = off_misc + 16;
  static_assert(off_bars % 8 == 0, "mbarrier alignment");
};
static_assert(AttSmem<64>::bytes <= 227u * 1024u && AttSmem<32>::bytes <= 227u * 1024u, "shared memory budget");

// An item is one row and list range.
struct AttGrid {
  int splits, tiles;               // tiles: of a whole list
  uint32_t items;                  // T * splits, below 2^31
  uint32_t* next;                  // null (one item a block) or a counter at 0 of the items behind the blocks' first
                                   // ones that are taken
  float4* part_o;                  // [T][splits] blocks of NH x 512 in the order of part_index
  float2* part_ml;                 // [T][splits][NH]
  uint32_t* err;                   // the workspace's status word
  PageDiv div;
};

// 16 lanes x NH columns of fp32: thread i holds rows i / 4 (values 4j, 4j + 1)
// and i / 4 + 8 (4j + 2, 4j + 3) at columns 8j + 2 (i % 4) and the next.
__device__ __forceinline__ void tmem_ld_tile(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_tile(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_tile(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// Barrier over the softmax warps that also combines a predicate.
__device__ __forceinline__ bool soft_bar_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred.aligned q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "n"(kSoftThreads)
      : "memory");
  return r != 0;
}

// Four 8 x 8 matrices of 16-bit fragments: lane 8 i + r gives the address of
// row r of matrix i.
__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
// A key's raw bytes as one of its eight lanes (two groups of four) holds them:
// 64 codes, their four scales and 8 rotary values.
struct RawKey {
  uint32_t code[8];
  uint32_t scale;
  uint4 rope;
};

__device__ __forceinline__ void load_raw(RawKey& r, const uint8_t* kv, int slot, bool live, int part, int group) {
  if (live) {
    const uint8_t* e = kv + static_cast<int64_t>(slot) * kKvEntry;
    ldg256(r.code, e + group * 128 + part * 32);
    r.scale = __ldg(reinterpret_cast<const uint32_t*>(e + kKvScaleOff + group * 16 + part * 4));
    r.rope = __ldg(reinterpret_cast<const uint4*>(e + kKvRopeOff + (2 * part + group) * 16));
  } else {
    // behind the last key: zeros, so that no bit pattern of the pool meets a zero weight
#pragma unroll
    for (int i = 0; i < 8; ++i) r.code[i] = 0u;
    r.scale = 0u;
    r.rope = make_uint4(0u, 0u, 0u, 0u);
  }
}

// Quarter p of hand-over part s of a tile holds latent dimensions 256 (s % 2)
// + 64 p + 32 (s / 2) .. + 31: a group's four lanes of a key load 128
// contiguous bytes of codes and decode 32 dimensions of each of its parts.
__device__ __forceinline__ constexpr int part_of(int hi, int lo) { return hi + 2 * lo; }
__device__ __forceinline__ constexpr int dim_of(int s, int p) { return 256 * (s & 1) + 64 * p + 32 * (s >> 1); }

// Query rows r0, r0 + step, ... to shared memory as the MMA reads them (see the
// file's comment), two rows in flight.
template <int NH>
__device__ __forceinline__ void stage_queries(const AttendParams& p, int64_t t, uint8_t* q_buf, float* s_c, int r0,
                                              int step, int lane) {
  auto live = [&](int r) { return r < NH && r < p.H; };
  uint4 v[2][3];
  load_query_row(v[0], p, t, r0, live(r0), lane);
  load_query_row(v[1], p, t, r0 + step, live(r0 + step), lane);
#pragma unroll 1
  for (int r = r0; r < NH; r += step) {
    uint4 now[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      now[k] = v[0][k];
      v[0][k] = v[1][k];
    }
    load_query_row(v[1], p, t, r + 2 * step, live(r + 2 * step), lane);
    store_query_row(now, p.scale, q_buf, AttSmem<NH>::q_block, r, s_c, lane, part_of);
  }
}

// The same rows for a whole number of pairs, two at once.
template <int NH>
__device__ __forceinline__ void stage_query_pairs(const AttendParams& p, int64_t t, uint8_t* q_buf, float* s_c,
                                                  int r0, int step, int lane) {
  auto live = [&](int r) { return r < p.H; };
#pragma unroll 1
  for (int r = r0; r < NH; r += 2 * step) {
    uint4 v[2][3];
    load_query_row(v[0], p, t, r, live(r), lane);
    load_query_row(v[1], p, t, r + step, live(r + step), lane);
    const int two[2] = {r, r + step};
    store_query_rows<2>(v, p.scale, q_buf, AttSmem<NH>::q_block, two, s_c, lane, part_of);
  }
}

// What item k stands for; false for padding and a sequence that does not exist.
struct AttItem {
  int64_t t;
  int split, seq;
};
__device__ __forceinline__ bool item_of(AttItem& it, uint32_t k, const AttendParams& p, const AttGrid& g) {
  const uint32_t row = k / static_cast<uint32_t>(g.splits);
  it.split = static_cast<int>(k - row * g.splits);
  it.t = row;
  it.seq = p.row_seq ? __ldg(p.row_seq + it.t) : static_cast<int>(it.t);
  return it.seq >= 0 && it.seq < p.B;
}

// Float4 of a partial output block: 16 rows (dimensions) x NH columns (heads)
// of part s, warp quarter p and half, column group j of 8 heads: a lane's
// float4 holds rows lane / 4 and lane / 4 + 8 at heads 8 j + 2 (lane % 4) and
// the next.
template <int NH>
__device__ __forceinline__ int64_t part_index(int64_t item, int s, int p, int half, int j, int lane) {
  return ((((item * kParts + s) * 4 + p) * 2 + half) * (NH / 8) + j) * 32 + lane;
}

template <int NH>
__global__ void __launch_bounds__(kAttThreads, 1) attend_kv4_kernel(const AttendParams p, const AttGrid g) {
  using L = AttSmem<NH>;
  constexpr uint32_t kTmemO = 0, kTmemS = kParts * NH;  // columns
  // all of the tensor memory, so that it begins at column 0 (a constant for the
  // MMAs); shared memory keeps a second block off the SM anyway
  constexpr uint32_t kTmemCols = 512;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sK = sbase + L::off_k, sP = sbase + L::off_p;
  float* s_c = reinterpret_cast<float*>(smem + L::off_c);
  float* s_f = reinterpret_cast<float*>(smem + L::off_f);
  float* s_m = reinterpret_cast<float*>(smem + L::off_m);
  volatile int* s_ring = reinterpret_cast<volatile int*>(smem + L::off_ring);
  volatile int* s_ring_n = reinterpret_cast<volatile int*>(smem + L::off_count);
  volatile int* s_n = s_ring_n + kRing;
  volatile int *s_ring_k = s_n + 2, *s_k = s_ring_k + kRing;
  const uint32_t bars = sbase + L::off_bars;
  auto bar_full = [&](int b, int s) { return bars + 8 * (b * kParts + s); };
  auto bar_empty = [&](int b, int s) { return bars + 8 * (2 * kParts + b * kParts + s); };
  auto bar_listed = [&](int r) { return bars + 8 * (4 * kParts + r); };
  auto bar_taken = [&](int r) { return bars + 8 * (4 * kParts + kRing + r); };
  auto bar_s = [&](int b) { return bars + 8 * (4 * kParts + 2 * kRing + b); };
  auto bar_read = [&](int b) { return bar_s(2 + b); };
  auto bar_q = [&](int q) { return bar_s(4 + q); };
  auto bar_q_free = [&](int q) { return bar_s(6 + q); };
  auto bar_c_free = [&](int n) { return bar_s(8 + (n & 1)); };
  const uint32_t bar_p = bar_s(10), bar_o = bar_p + 8, bar_drain = bar_p + 16;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L::off_misc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + L::off_misc + 8);
  constexpr uint32_t tmem = 0;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto wait = [&](uint32_t bar, int parity) {
    return __all_sync(~0u, wait_bar(bar, static_cast<uint32_t>(parity) & 1u, s_abort, p.wait_ns));
  };

  if (tid == 0) {
    for (int i = 0; i < 2 * kParts; ++i) {
      mbar_init(bars + 8 * i, kLoadWarps / 2);
      mbar_init(bars + 8 * (2 * kParts + i), 1);
    }
    for (int r = 0; r < kRing; ++r) {
      mbar_init(bar_listed(r), 1);
      mbar_init(bar_taken(r), kLoadWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_s(i), 1);
      mbar_init(bar_read(i), kSoftWarps);
      mbar_init(bar_q(i), kLoadWarps);
      mbar_init(bar_q_free(i), kSoftWarps);
      mbar_init(bar_c_free(i), kSoftWarps);
    }
    mbar_init(bar_p, kSoftWarps);
    mbar_init(bar_o, 1);
    for (int i = 0; i < 3; ++i) mbar_init(bar_drain + 8 * i, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(s_tmem), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  AttItem it;
  const bool first_ok = item_of(it, blockIdx.x, p, g);
  // the queries of the block's first item by all warps but the issuing ones and the list's
  if (warp < kMmaWarp) {
    if (first_ok) {
      stage_queries<NH>(p, it.t, smem, s_c, warp, kMmaWarp, lane);
      fence_proxy_async_smem();
    }
    named_bar_sync(2, kWorkThreads);
  }

  // each warpgroup's share of the registers, set on its own path (behind a join
  // of the paths the compiler would hold all of them to the smallest)
  if (warp >= kMmaWarp) {
    regs_dec<kIssueRegs>();
    if (warp == kListWarp) {
      // --------------------------------------------------------------- list
      // Packs the pool rows of the entries that name a key into tiles, ahead of
      // the gathering warps; a row without any gets one tile of no keys.
      int tile = 0, keys = 0;  // the open tile, and how many keys it has
      bool ok = true, bad = false;
      uint32_t k = blockIdx.x;
      auto publish = [&](int flags) {  // the open tile
        if (lane == 0) {
          s_ring_n[tile % kRing] = keys | flags;
          s_ring_k[tile % kRing] = static_cast<int>(k);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_listed(tile % kRing));
      };
      auto turn = [&](int flags) {  // publishes the open tile and opens the next one
        publish(flags);
        ++tile;
        keys = 0;
        ok = wait(bar_taken(tile % kRing), tile / kRing + 1) && tile < p.hold_tiles;
      };
      int j0 = 0, j_hi = 0, pos[4];  // the item's entries that are left
      const int32_t* list = nullptr;
      auto fetch = [&] {
#pragma unroll
        for (int k = 0; k < 4; ++k) pos[k] = j0 + 32 * k + lane < j_hi ? __ldg(list + j0 + 32 * k + lane) : -1;
        j0 += 128;
      };
      auto advance = [&] {
        if (g.next) {
          if (lane == 0) k = gridDim.x + atomicAdd(g.next, 1u);
          k = __shfl_sync(~0u, k, 0);
        } else {
          k = g.items;
        }
      };
      for (int n = 0; ok && k < g.items; advance()) {
        if (!item_of(it, k, p, g)) {
          bad |= it.seq >= p.B;  // else padding
          continue;
        }
        const int32_t* table = p.block_table + static_cast<int64_t>(it.seq) * p.max_blocks;
        const int row = (n & 255) << kRowShift;
        list = p.idx + it.t * p.n;
        j0 = static_cast<int>(static_cast<int64_t>(g.tiles) * it.split / g.splits) * kKt;
        j_hi = static_cast<int>(
            min(static_cast<int64_t>(p.n), static_cast<int64_t>(g.tiles) * (it.split + 1) / g.splits * kKt));
        const int steps = (j_hi - j0 + 127) >> 7;  // of 128 entries
        fetch();
#pragma unroll 1
        for (int left = steps; left > 0 && ok; --left) {
          int slot[4];
          slots_of(p, g.div, table, pos, slot, bad);
          fetch();
#pragma unroll 1
          for (int q = 0; q < 4 && ok; ++q) {
            const int mine = slot[0];
            slot[0] = slot[1];
            slot[1] = slot[2];
            slot[2] = slot[3];
            const uint32_t m = __ballot_sync(~0u, mine >= 0);
            const int at = keys + __popc(m & lanemask_lt());
            if (mine >= 0 && at < kKt) s_ring[tile % kRing * kKt + at] = mine;
            keys += __popc(m);
            if (keys > kKt) {  // the rest starts the next tile, so this one is not the last
              const int rest = keys - kKt;
              keys = kKt;
              turn(row);
              if (mine >= 0 && at >= kKt) s_ring[tile % kRing * kKt + at - kKt] = mine;
              keys = rest;
            }
          }
        }
        if (ok) turn(row | kLast);
        ++n;
      }
      if (ok && tile + 1 < p.hold_tiles) publish(kStop);
      if (__any_sync(~0u, bad) && lane == 0) report(p, g.err, kErrOverflow);
    } else if (warp == kMmaWarp || warp == kMmaOddWarp) {
      // -------------------------------------------------- MMAs of the scores
      // One warp for each tile buffer: 36 MMAs take a warp longer to issue than
      // the tensor core to run when the heads are few.
      constexpr uint32_t kIdS = idesc_att(64, NH, 0, 0, 0), kIdR = idesc_att(64, NH, 1, 0, 0);
      const int b = warp == kMmaWarp ? 0 : 1;
      const uint64_t dK = smem_desc_sw128(sK + b * kTileBytes);
      const uint32_t leader = elect_one(), d = tmem + kTmemS + b * NH;
      bool ok = true;
      for (int k = 0; ok; ++k) {  // tile 2 k + b
        // lane by lane: the tile's four parts, and that the scores of the buffer's last tile are read
        const uint32_t mine = lane == 4 ? bar_read(b) : bar_full(b, lane & 3);
        const uint32_t par = static_cast<uint32_t>(lane == 4 ? k + 1 : k) & 1u;
        uint32_t ready = 0;
        if (!(ok = wait_any(ready, 0, lane < 5, mine, par, s_abort, p.wait_ns))) break;
        const int word = s_n[b];
        if (word & kStop) break;
        const int n = word >> kRowShift, q = L::q_bufs == 2 ? n & 1 : 0;
        if (!(ok = wait(bar_q(q), L::q_bufs == 2 ? n >> 1 : n))) break;
        if (!(ok = wait_any(ready, 4, lane < 5, mine, par, s_abort, p.wait_ns))) break;
        tc_fence_after();
        const uint64_t dQ = smem_desc_sw128(sbase + q * L::q_bytes);
#pragma unroll 1
        for (int s = 0; s < kParts; ++s) {
          if (!((ready >> s) & 1u)) {
            if (!(ok = wait_any(ready, s, lane < 5, mine, par, s_abort, p.wait_ns))) break;
            tc_fence_after();
          }
          const uint64_t k0 = dK + (2 * s * kBlockBytes >> 4), q0 = dQ + (2 * s * L::q_block >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_if<1>(leader, d, k0 + (((kk >> 2) * kBlockBytes + 32 * (kk & 3)) >> 4),
                      q0 + (((kk >> 2) * L::q_block + 32 * (kk & 3)) >> 4), kIdS, s > 0 || kk > 0);
          if (s == 1) {  // each group brings half of the rotary block with its first part
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_if<1>(leader, d, dK + ((8 * kBlockBytes + 32 * kk) >> 4), dQ + ((8 * L::q_block + 32 * kk) >> 4), kIdR, 1);
          }
          if (s == kParts - 1) commit_if(leader, bar_s(b));
        }
      }
      // nothing may be in flight when the tensor memory is freed (also after a wait that gave up)
      const uint32_t drain = bar_drain + (b ? 16 : 0);
      commit_if(leader, drain);
      int unused = 0;
      if (!wait_bar(drain, 0, &unused, p.wait_ns)) *s_abort = 1;
      __syncwarp();
    } else if (warp == kMmaOWarp) {
      // ------------------------------------------------- MMAs of the outputs
      constexpr uint32_t kIdO = idesc_att(128, NH, 0, 1, 1);
      const uint64_t dV = desc_mn_sw128(sK, kBlockBytes), dP = desc_mn_sw128(sP, kBlockBytes);
      const uint32_t leader = elect_one();
      bool first = true;
      for (int i = 0;; ++i) {  // O^T (+)= V^T P^T of tile i
        const int b = i & 1;
        if (!wait(bar_full(b, 0), i >> 1)) break;
        const int word = s_n[b];
        if ((word & kStop) || !wait(bar_p, i)) break;
        tc_fence_after();
#pragma unroll 1
        for (int s = 0; s < kParts; ++s) {
          const uint64_t v = dV + ((b * kTileBytes + 2 * s * kBlockBytes) >> 4);
#pragma unroll
          for (int k = 0; k < kKt / 16; ++k)
            mma_if<1>(leader, tmem + kTmemO + s * NH, v + (k * 2048 >> 4), dP + (k * 2048 >> 4), kIdO, !first || k > 0);
          commit_if(leader, bar_empty(b, s));
        }
        commit_if(leader, bar_o);
        first = word & kLast;
      }
      commit_if(leader, bar_drain + 8);
      int unused = 0;
      if (!wait_bar(bar_drain + 8, 0, &unused, p.wait_ns)) *s_abort = 1;
      __syncwarp();
    }
  } else if (warp >= kSoftWarps) {
    regs_dec<kLoadRegs>();
    // ------------------------------------------------------------- gather
    const int lw = (warp - kSoftWarps) & 7, group = (warp - kSoftWarps) >> 3;
    const int key = lw * 8 + (lane & 7), part = lane >> 3;
    const uint32_t row = static_cast<uint32_t>(key) * 128, sw = static_cast<uint32_t>(key & 7);
    bool ok = true;
    int n = -1;  // rows staged, less one
    if (first_ok) {
      n = 0;
      if (lane == 0) mbar_arrive(bar_q(0));
    }
    RawKey raw;
    int word = 0, item = 0, stops = 0;
    for (int i = -1; ok; ++i) {  // loads of tile i + 1, then tile i to shared memory
      RawKey next;
      int next_word = kStop, next_item = 0;
      if (!(word & kStop)) {
        const int k = (i + 1) % kRing;
        if (!wait(bar_listed(k), (i + 1) / kRing)) break;
        next_word = s_ring_n[k];
        next_item = s_ring_k[k];
        load_raw(next, p.kv, s_ring[k * kKt + key], key < (next_word & 0xFFFF), part, group);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_taken(k));
      }
      if (i >= 0) {
        const int b = i & 1;
        const uint32_t tile = sK + b * kTileBytes + row;
#pragma unroll 1
        for (int u = 0; u < kParts / 2; ++u) {
          const int s = 2 * u + group;
          if (!(ok = wait(bar_empty(b, s), (i >> 1) + 1))) break;
          if (u == 0) {
            if (warp == kSoftWarps && lane == 0) {
              s_n[b] = word;
              s_k[b] = item;
            }
            sts128(tile + 8 * kBlockBytes + (((2 * part + group) ^ sw) << 4), raw.rope.x, raw.rope.y, raw.rope.z, raw.rope.w);
          }
          const __half2 sc =
              __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(raw.scale & 0xFFFFu), __NV_E4M3));
          const __half2 lo = __low2half2(sc), hi = __high2half2(sc);
          const uint32_t dst = tile + (2 * s + (part >> 1)) * kBlockBytes;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t o[4];
            decode8(raw.code[k], k < 2 ? lo : hi, o);
            sts128(dst + (((4 * (part & 1) + k) ^ sw) << 4), o[0], o[1], o[2], o[3]);
            raw.code[k] = raw.code[k + 4];
          }
          raw.scale >>= 16;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_full(b, s));
          if (word & kStop) break;  // part 0 alone carries it
        }
        if ((word & kStop) && ++stops == 2) break;  // told to both buffers' readers
      }
      // the queries of a row whose first tile is next
      if (ok && (i < 0 ? !first_ok : (word & kLast) != 0) && !(next_word & kStop)) {
        item_of(it, static_cast<uint32_t>(next_item), p, g);
        ++n;
        const int q = L::q_bufs == 2 ? n & 1 : 0;
        // on their way to L2 during the wait
        const char* src = reinterpret_cast<const char*>(p.q + it.t * p.H * kKvQ);
        const int bytes = p.H * 2 * kKvQ;
        for (int at = (tid - kSoftThreads) * 128; at < bytes; at += kLoadWarps * 32 * 128)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(src + at));
        ok = wait(bar_q_free(q), (L::q_bufs == 2 ? n >> 1 : n) + 1) && wait(bar_c_free(n), (n >> 1) + 1);
        if (!ok) break;
        if constexpr (NH >= 2 * kLoadWarps)
          stage_query_pairs<NH>(p, it.t, smem + q * L::q_bytes, s_c + (n & 1) * NH, warp - kSoftWarps, kLoadWarps, lane);
        else
          stage_queries<NH>(p, it.t, smem + q * L::q_bytes, s_c + (n & 1) * NH, warp - kSoftWarps, kLoadWarps, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_q(q));
      }
      item = next_item;
      raw = next;
      word = next_word;
    }
  } else {
    regs_inc<kSoftRegs>();
    // ------------------------------------------------------------ softmax
    // Threads hold pairs of columns (heads): pair j is columns 8 j + 2 (lane %
    // 4) and the next, at keys (rows) r0 and r0 + 8 of the warp's 16.
    constexpr int C = NH / 8;
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    const int r0 = lane >> 2;
    const uint32_t p0 = sP + (warp * 16 + (lane & 15)) * 128;  // this lane's row in the 8 x 8 stores
    float* exch = reinterpret_cast<float*>(smem + L::off_p);  // [4 warps][NH], while P is not in use
    bool ok = true;
    int i = 0;
    for (int n = 0;; ++n) {
      // the next row's first tile, or the end; the same decision in all four warps
      ok = wait(bar_full(i & 1, 0), i >> 1) && ok;
      if (soft_bar_or(!ok || (s_n[i & 1] & kStop))) break;
      const uint32_t item = static_cast<uint32_t>(s_k[i & 1]);
      item_of(it, item, p, g);
      bool some = false;  // the row (its part) has keys
      float2 c[C], m[C], l[C];  // factor to log2 units, kLift less the reference (from the first tile on), sum
      for (bool first = true, last = false; !last; first = false, ++i) {
        const int b = i & 1;
        ok = wait(bar_s(b), i >> 1) && ok;
        const int word = s_n[b], n_keys = word & 0xFFFF;
        last = ok && (word & kLast);
        if (first) {
          some = n_keys > 0;
#pragma unroll
          for (int j = 0; j < C; ++j) {
            c[j] = *reinterpret_cast<const float2*>(s_c + (n & 1) * NH + 8 * j + 2 * (lane & 3));
            m[j] = make_float2(0.f, 0.f);
            l[j] = make_float2(0.f, 0.f);
          }
        }
        __syncwarp();
        if (lane == 0 && first) mbar_arrive(bar_c_free(n));
        if (lane == 0 && last) mbar_arrive(bar_q_free(L::q_bufs == 2 ? n & 1 : 0));  // all scores of the row are there
        float x[NH / 2];
        bool moved = false;
        tc_fence_after();
#pragma unroll 1
        for (int pass = 0;; ++pass) {
          // x <- score - reference + kLift, -inf behind the last key; mx: the largest
          float mx = -INFINITY;
          tmem_ld_tile(tmem + kTmemS + b * NH + lane_base, reinterpret_cast<uint32_t(&)[NH / 2]>(x));
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < C; ++j) {
            const float2 a = __ffma2_rn(make_float2(x[4 * j], x[4 * j + 1]), c[j], m[j]);
            const float2 d = __ffma2_rn(make_float2(x[4 * j + 2], x[4 * j + 3]), c[j], m[j]);
            x[4 * j] = a.x;
            x[4 * j + 1] = a.y;
            x[4 * j + 2] = d.x;
            x[4 * j + 3] = d.y;
          }
          if (n_keys < kKt) {
            const bool v0 = warp * 16 + r0 < n_keys, v1 = warp * 16 + 8 + r0 < n_keys;
#pragma unroll
            for (int k = 0; k < NH / 2; ++k)
              if (!(k & 2 ? v1 : v0)) x[k] = -INFINITY;
          }
#pragma unroll
          for (int k = 0; k < NH / 2; k += 2) mx = fmaxf(mx, fmaxf(x[k], x[k + 1]));
          if (pass > 0) break;
          // the same decision in all four warps; a row's first tile and a wait that gave up go this way too
          moved = soft_bar_or(!ok || first || mx > kRise + kLift);
          if (!moved) break;
          if (!first) ok = wait(bar_o, i - 1) && ok;
          if (soft_bar_or(!ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < C; ++j) {
            float2 t = make_float2(fmaxf(x[4 * j], x[4 * j + 2]) - m[j].x, fmaxf(x[4 * j + 1], x[4 * j + 3]) - m[j].y);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              t.x = fmaxf(t.x, __shfl_xor_sync(~0u, t.x, o));
              t.y = fmaxf(t.y, __shfl_xor_sync(~0u, t.y, o));
            }
            if (lane < 4) *reinterpret_cast<float2*>(exch + warp * NH + 8 * j + 2 * lane) = t;
          }
          named_bar_sync(1, kSoftThreads);
#pragma unroll
          for (int j = 0; j < C; ++j) {
            const int col = 8 * j + 2 * (lane & 3);
            float2 top = first ? make_float2(-INFINITY, -INFINITY) : make_float2(kLift - m[j].x, kLift - m[j].y);
#pragma unroll
            for (int w = 0; w < kSoftWarps; ++w) {
              const float2 e = *reinterpret_cast<const float2*>(exch + w * NH + col);
              top.x = fmaxf(top.x, e.x);
              top.y = fmaxf(top.y, e.y);
            }
            if (top.x == -INFINITY) top.x = 0.f;  // no keys
            if (top.y == -INFINITY) top.y = 0.f;
            const float2 to = make_float2(kLift - top.x, kLift - top.y);
            const float2 f = first ? make_float2(1.f, 1.f) : make_float2(ex2(to.x - m[j].x), ex2(to.y - m[j].y));
            m[j] = to;
            l[j].x *= f.x;
            l[j].y *= f.y;
            if (warp == 0 && lane < 4) *reinterpret_cast<float2*>(s_f + col) = f;
          }
          named_bar_sync(1, kSoftThreads);
          if (!first) {
#pragma unroll 1
            for (int q = 0; q < kParts * NH; q += 16) {
              uint32_t o[16];
              tmem_ld16(tmem + kTmemO + lane_base + q, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * s_f[q % NH + k]);
              tmem_st16(tmem + kTmemO + lane_base + q, o);
            }
            tmem_wait_st();
          }
        }
        if (moved && !ok) break;  // decided by all four warps
        uint32_t w[NH / 4];
#pragma unroll
        for (int j = 0; j < C; ++j) {
          const float2 a = make_float2(ex2(x[4 * j]), ex2(x[4 * j + 1])), d = make_float2(ex2(x[4 * j + 2]), ex2(x[4 * j + 3]));
          l[j] = __fadd2_rn(l[j], __fadd2_rn(a, d));
          const __half2 ha = __floats2half2_rn(a.x, a.y), hd = __floats2half2_rn(d.x, d.y);
          w[2 * j] = *reinterpret_cast<const uint32_t*>(&ha);
          w[2 * j + 1] = *reinterpret_cast<const uint32_t*>(&hd);
        }
        // P of the last tile is consumed (checked above when the reference moved, at the end of the last row)
        if (!moved) ok = wait(bar_o, i - 1) && ok;
#pragma unroll
        for (int j = 0; j < C; j += 2)
          stmatrix4(p0 + (((j + (lane >> 4)) ^ (lane & 7)) << 4), w[2 * j], w[2 * j + 1], w[2 * j + 2], w[2 * j + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar_p);
          mbar_arrive(bar_read(b));
        }
      }
      // ----------------------------------------------------------- output
      ok = ok && wait(bar_o, i - 1);
      if (soft_bar_or(!ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < C; ++j) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          l[j].x += __shfl_xor_sync(~0u, l[j].x, o);
          l[j].y += __shfl_xor_sync(~0u, l[j].y, o);
        }
        if (lane < 4) {
          *reinterpret_cast<float2*>(exch + warp * NH + 8 * j + 2 * lane) = l[j];
          if (warp == 0) *reinterpret_cast<float2*>(s_m + 8 * j + 2 * lane) = make_float2(-m[j].x, -m[j].y);
        }
      }
      named_bar_sync(1, kSoftThreads);
      if (tid < NH) {  // a head per thread
        const float sum = (exch[tid] + exch[NH + tid]) + (exch[2 * NH + tid] + exch[3 * NH + tid]);
        // NaN or infinite scores; with finite ones the reference's own weight counts
        if ((!(sum < INFINITY) || (sum == 0.f && some)) && tid < p.H) report(p, g.err, kErrNonFinite);
        if (g.splits > 1) {
          g.part_ml[static_cast<int64_t>(item) * NH + tid] = make_float2(sum == 0.f ? -INFINITY : s_m[tid], sum);
        } else {
          s_f[tid] = sum == 0.f ? 0.f : 1.f / sum;
          if (p.lse && tid < p.H)
            p.lse[it.t * p.H + tid] = sum == 0.f ? -INFINITY : (s_m[tid] + log2f(sum)) * kLn2;
        }
      }
      named_bar_sync(1, kSoftThreads);
      if (g.splits > 1) {
#pragma unroll 1
        for (int sh = 0; sh < 2 * kParts; ++sh) {  // part and half
          uint32_t o[NH / 2];
          tmem_ld_tile(tmem + kTmemO + (sh >> 1) * NH + lane_base + (static_cast<uint32_t>((sh & 1) * 16) << 16), o);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < NH / 8; ++j)
            g.part_o[part_index<NH>(item, sh >> 1, warp, sh & 1, j, lane)] =
                make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]), __uint_as_float(o[4 * j + 2]),
                            __uint_as_float(o[4 * j + 3]));
        }
      } else {
#pragma unroll 1
        for (int q = 0; q < kParts * NH; q += 16) {  // 16 heads of a part
          const int s = q / NH, h = q % NH;
          uint32_t o[16];
          tmem_ld16(tmem + kTmemO + lane_base + q, o);
          tmem_wait_ld();
          const int dim = (dim_of(s, warp) + lane) & ~1;
          uint16_t* dst = p.out + (it.t * p.H + h + (lane & 1)) * kKvLat + dim;
          // lanes pair up: the even one stores two dimensions of a head, the odd one of the next head
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const float2 f = *reinterpret_cast<const float2*>(s_f + h + k);
            const float a = __uint_as_float(o[k]) * f.x, d = __uint_as_float(o[k + 1]) * f.y;
            const float other = __shfl_xor_sync(~0u, lane & 1 ? a : d, 1);
            const __nv_bfloat162 v = lane & 1 ? __floats2bfloat162_rn(other, d) : __floats2bfloat162_rn(a, other);
            if (h + k + (lane & 1) < p.H) *reinterpret_cast<__nv_bfloat162*>(dst + k * kKvLat) = v;
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      named_bar_sync(1, kSoftThreads);  // s_f and P are free again
    }
  }
  __syncthreads();
  if (tid == 0 && *s_abort) report(p, g.err, kErrTimeout);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(*s_tmem, kTmemCols);
  }
}

// Joins the splits of eight heads of a row and one part of their dimensions:
// out = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s.
template <int NH>
__global__ void __launch_bounds__(256) attend_join_kernel(const AttendParams p, const AttGrid g) {
  __shared__ __align__(16) uint16_t s_o[8][128 + 8];
  const int s = blockIdx.x % kParts, j = blockIdx.x / kParts % (NH / 8);
  const int64_t t = blockIdx.x / (kParts * (NH / 8));
  const int seq = p.row_seq ? __ldg(p.row_seq + t) : static_cast<int>(t);
  const int h0 = 8 * j;
  if (seq < 0 || seq >= p.B || h0 >= p.H) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pq = warp & 3, half = warp >> 2;
  const int64_t item0 = t * g.splits;
  const float4* ml = reinterpret_cast<const float4*>(g.part_ml + item0 * NH + 8 * j + 2 * (lane & 3));  // two heads
  constexpr int kMl = NH / 2;                                 // float4 between splits
  constexpr int64_t kO = int64_t(NH) * kKvLat / 4;
  const float4* po = g.part_o + part_index<NH>(item0, s, pq, half, j, lane);
  float2 ref = make_float2(-INFINITY, -INFINITY);
#pragma unroll 8
  for (int k = 0; k < g.splits; ++k) {
    const float4 v = ml[static_cast<int64_t>(k) * kMl];
    ref.x = fmaxf(ref.x, v.x);
    ref.y = fmaxf(ref.y, v.z);
  }
  const float2 base = make_float2(ref.x == -INFINITY ? 0.f : ref.x, ref.y == -INFINITY ? 0.f : ref.y);
  float2 sum = make_float2(0.f, 0.f);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int k = 0; k < g.splits; ++k) {
    const float4 v = ml[static_cast<int64_t>(k) * kMl], o = po[k * kO];
    const float a = ex2(v.x - base.x), b = ex2(v.z - base.y);
    sum.x = fmaf(a, v.y, sum.x);
    sum.y = fmaf(b, v.w, sum.y);
    acc.x = fmaf(a, o.x, acc.x);
    acc.y = fmaf(b, o.y, acc.y);
    acc.z = fmaf(a, o.z, acc.z);
    acc.w = fmaf(b, o.w, acc.w);
  }
  const float fa = sum.x == 0.f ? 0.f : 1.f / sum.x, fb = sum.y == 0.f ? 0.f : 1.f / sum.y;
  const int r = 32 * pq + 16 * half + (lane >> 2), col = 2 * (lane & 3);
  s_o[col][r] = __bfloat16_as_ushort(__float2bfloat16_rn(acc.x * fa));
  s_o[col + 1][r] = __bfloat16_as_ushort(__float2bfloat16_rn(acc.y * fb));
  s_o[col][r + 8] = __bfloat16_as_ushort(__float2bfloat16_rn(acc.z * fa));
  s_o[col + 1][r + 8] = __bfloat16_as_ushort(__float2bfloat16_rn(acc.w * fb));
  if (p.lse && s == 0 && warp == 0 && lane < 4) {
    if (h0 + col < p.H)
      p.lse[t * p.H + h0 + col] = sum.x == 0.f ? -INFINITY : (base.x + log2f(sum.x)) * kLn2;
    if (h0 + col + 1 < p.H)
      p.lse[t * p.H + h0 + col + 1] = sum.y == 0.f ? -INFINITY : (base.y + log2f(sum.y)) * kLn2;
  }
  __syncthreads();
  if (threadIdx.x < 128 && h0 + (threadIdx.x >> 4) < p.H) {  // 16 bytes: 8 dimensions of a head
    const int h = threadIdx.x >> 4, c = threadIdx.x & 15;
    *reinterpret_cast<uint4*>(p.out + (t * p.H + h0 + h) * kKvLat + dim_of(s, c >> 2) + 8 * (c & 3)) =
        *reinterpret_cast<const uint4*>(&s_o[h][8 * c]);
  }
}

struct AttPlan {
  int NH, splits, tiles;
  size_t off_ml, off_o, bytes;
};

AttPlan plan_attend(int64_t T, int H, int n, int sms) {
  AttPlan P{};
  P.NH = H <= 16 ? 16 : H <= 32 ? 32 : 64;
  P.tiles = (n + kKt - 1) / kKt;
  // fewer rows than SMs: parts of at least two tiles (one row of 64 heads and 2048 entries: 21.6 us in 16 parts,
  // 25 us in 32 of one tile, whose partial outputs cost more than their tile)
  P.splits = T >= sms || T == 0 ? 1 : static_cast<int>(std::min<int64_t>(sms / T, (P.tiles + 1) / 2));
  P.off_ml = kAttHeader;
  P.off_o = P.off_ml;
  P.bytes = kAttHeader;
  if (P.splits > 1) {
    const size_t rows = static_cast<size_t>(T) * P.splits * P.NH;
    P.off_o = (P.off_ml + rows * sizeof(float2) + 255) / 256 * 256;
    P.bytes = P.off_o + rows * kKvLat * sizeof(float);
  }
  return P;
}

template <int NH>
cudaError_t launch_nh(const AttendParams& p, const AttGrid& g, int sms, cudaStream_t st) {
  constexpr int bytes = AttSmem<NH>::bytes;
  cudaError_t e = cudaFuncSetAttribute(attend_kv4_kernel<NH>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  if ((e = cudaMemsetAsync(g.err, 0, kAttHeader, st)) != cudaSuccess) return e;  // status word and counter
  attend_kv4_kernel<NH><<<std::min(g.items, static_cast<uint32_t>(std::max(sms, 1))), kAttThreads, bytes, st>>>(p, g);
  e = cudaGetLastError();
  if (e != cudaSuccess || g.splits == 1) return e;
  attend_join_kernel<NH><<<static_cast<unsigned>(p.T * kParts * (NH / 8)), 256, 0, st>>>(p, g);
  return cudaGetLastError();
}

}  // namespace

size_t attend_workspace_bytes(int64_t T, int H, int n, int sms) {
  return H > 64 ? attend_pair_workspace_bytes(T, H, n, sms) : plan_attend(T, H, n, sms).bytes;
}

cudaError_t launch_attend_kv4(const AttendParams& p, void* workspace, int sms, cudaStream_t st) {
  if (p.H > 64) return launch_attend_kv4_pair(p, workspace, sms, st);
  const AttPlan P = plan_attend(p.T, p.H, p.n, sms);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  AttGrid g{P.splits, P.tiles, static_cast<uint32_t>(p.T * P.splits), nullptr,
            reinterpret_cast<float4*>(ws + P.off_o),
            reinterpret_cast<float2*>(ws + P.off_ml), reinterpret_cast<uint32_t*>(ws), page_div(p.page_size)};
  // lists of unequal lengths: blocks take rows as they get free (501 rows of 16 heads and up to 1023 entries: 81 us,
  // 88 us in turn)
  if (g.items > static_cast<uint32_t>(sms)) g.next = reinterpret_cast<uint32_t*>(ws + kAttCounter);
  return P.NH == 16 ? launch_nh<16>(p, g, sms, st) : P.NH == 32 ? launch_nh<32>(p, g, sms, st) : launch_nh<64>(p, g, sms, st);
}

}  // namespace dsa
