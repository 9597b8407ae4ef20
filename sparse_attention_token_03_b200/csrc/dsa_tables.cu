// Request layout of one serving step (dsa_block_tables): from the cached and
// new lengths of B requests, the pages that the new tokens need, and for each
// new token (row) its cache slot, position and request.
//
//   R_b = sum of new_len before b          first row of request b
//   P_b = sum of ceil(seq/ps) - ceil(cached/ps) before b
//   row t of b:  position = cached_b + t - R_b
//                slot     = page(b, position / ps) * ps + position % ps
//   page(b, i) = block_table[b][i] for the blocks that b already has, else
//                free_pages[begin + P_b + i - ceil(cached_b / ps)]
//
// The work is a few bytes per row and request, so the launch and the chain of
// dependent loads bound it: one launch does all.  Every block repeats the
// prefix sums over the requests (one bucket of consecutive requests per thread;
// 8 bytes a request from L2) instead of waiting for another block or launch,
// then finds the owners of its rows by bisection in shared memory.  Up to 4096
// requests the sums of every request are kept there, and a row's only global
// load is its page (4096 requests, 131072 rows: 10 us); above that the sums
// of every bucket, and the row's bucket is walked (14 us for the same).
#include <algorithm>

#include "dsa_ptx.cuh"
#include "dsa_serve.cuh"

namespace dsa {

namespace {

constexpr int kTabThreadsMax = 1024;

struct Lens {
  int cached, fresh, old_blocks, need;  // need: new pages
};

// Lengths of one request; false when they are out of range.
__device__ __forceinline__ bool load_lens(const TablesParams& p, int b, Lens& L) {
  L.cached = __ldg(p.cached_len + b);
  L.fresh = __ldg(p.new_len + b);
  L.old_blocks = L.need = 0;
  if (L.cached < 0 || L.fresh < 0 ||
      static_cast<int64_t>(L.cached) + L.fresh > static_cast<int64_t>(p.max_blocks) * p.page_size)
    return false;
  // max_blocks * page_size < 2^31, so the rounded-up sums stay in range as unsigned
  const uint32_t ps = static_cast<uint32_t>(p.page_size);
  L.old_blocks = static_cast<int>((static_cast<uint32_t>(L.cached) + ps - 1) / ps);
  L.need = static_cast<int>((static_cast<uint32_t>(L.cached + L.fresh) + ps - 1) / ps) - L.old_blocks;
  return true;
}

// Largest i in [0, n) with pre[i] <= x (pre ascending, pre[0] <= x).
__device__ __forceinline__ int bucket_of(const int* pre, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTabThreadsMax) block_tables_kernel(const TablesParams p) {
  __shared__ int s_rows[kTabThreadsMax], s_pages[kTabThreadsMax];  // first row / page of each bucket
  __shared__ int64_t s_wr[32], s_wp[32];
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + nt - 1) / nt;  // requests per bucket
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);

  int64_t rows = 0, pages = 0;
  bool ok = true;
  for (int b = b0; b < b1; ++b) {
    Lens L;
    ok &= load_lens(p, b, L);
    rows += L.fresh;
    pages += L.need;
  }
  int64_t ir = rows, ip = pages;  // inclusive sums over the warp, then the block
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t r = __shfl_up_sync(~0u, ir, o), g = __shfl_up_sync(~0u, ip, o);
    if (lane >= o) {
      ir += r;
      ip += g;
    }
  }
  if (lane == 31) {
    s_wr[warp] = ir;
    s_wp[warp] = ip;
  }
  ok = __syncthreads_and(ok);
  int64_t total_rows = 0, total_pages = 0;
  for (int w = 0; w < nt / 32; ++w) {
    if (w < warp) {
      ir += s_wr[w];
      ip += s_wp[w];
    }
    total_rows += s_wr[w];
    total_pages += s_wp[w];
  }
  const int begin = __ldg(p.free_begin);
  // all or nothing: one request out of range, too many rows or too few pages
  // leave every request without new rows (sums of bad lengths are not used)
  ok = ok && total_rows <= p.T_cap && begin >= 0 && total_pages <= p.n_free - begin;
  if (!ok) {
    rows = pages = ir = ip = total_rows = total_pages = 0;
    if (blockIdx.x == 0 && tid == 0 && p.status) atomicOr(p.status, kErrOverflow);
  }
  s_rows[tid] = static_cast<int>(ir - rows);
  s_pages[tid] = static_cast<int>(ip - pages);
  __syncthreads();

  // per request: buckets are shared out over the blocks
  if (tid % gridDim.x == blockIdx.x) {
    int r = static_cast<int>(ir - rows);
    for (int b = b0; b < b1; ++b) {
      const int cached = __ldg(p.cached_len + b), fresh = ok ? __ldg(p.new_len + b) : 0;
      p.row_start[b] = r;
      p.seq_len[b] = cached + fresh;
      r += fresh;
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.row_start[p.B] = static_cast<int>(total_rows);
    p.free_end[0] = begin + static_cast<int>(total_pages);
  }

  const int gtid = blockIdx.x * nt + tid, gstride = gridDim.x * nt;
  bool bad_page = false;
  for (int t = gtid; t < p.T_cap; t += gstride) {
    int slot = -1, pos = -1, owner = -1;
    if (t < total_rows) {
      const int bk = bucket_of(s_rows, nt, t);
      int b = bk * per, r = s_rows[bk], g = s_pages[bk];
      Lens L;
      load_lens(p, b, L);
      while (t - r >= L.fresh) {  // ends: the bucket holds row t
        r += L.fresh;
        g += L.need;
        load_lens(p, ++b, L);
      }
      owner = b;
      pos = L.cached + (t - r);
      const int blk = pos / p.page_size;
      const int page = blk < L.old_blocks ? p.block_table[static_cast<int64_t>(b) * p.max_blocks + blk]
                                          : __ldg(p.free_pages + begin + g + (blk - L.old_blocks));
      if (page >= 0 && page < p.n_pages)
        slot = page * p.page_size + (pos - blk * p.page_size);
      else
        bad_page = true;
    }
    p.slot_map[t] = slot;
    p.position[t] = pos;
    p.row_seq[t] = owner;
  }
  // new entries of the block tables (no row above reads one)
  for (int j = gtid; j < total_pages; j += gstride) {
    const int bk = bucket_of(s_pages, nt, j);
    int b = bk * per, g = s_pages[bk];
    Lens L;
    load_lens(p, b, L);
    while (j - g >= L.need) {
      g += L.need;
      load_lens(p, ++b, L);
    }
    p.block_table[static_cast<int64_t>(b) * p.max_blocks + L.old_blocks + (j - g)] = __ldg(p.free_pages + begin + j);
  }
  if (bad_page && p.status) atomicOr(p.status, kErrOverflow);
}

constexpr int kTabKept = 4096, kTabBucket = 4;  // requests whose sums are kept; of one thread

// block_tables_kernel with the sums of every request in shared memory.
__global__ void __launch_bounds__(kTabThreadsMax) block_tables_kept_kernel(const TablesParams p, const PageDiv div) {
  extern __shared__ int s_sums[];  // [B + 1] first row, [B + 1] first page, [B] cached length
  __shared__ int64_t s_wr[32], s_wp[32];
  int *s_row = s_sums, *s_page = s_row + p.B + 1, *s_cached = s_page + p.B + 1;
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + nt - 1) / nt, b0 = tid * per;  // per <= kTabBucket
  const int64_t room = static_cast<int64_t>(p.max_blocks) * p.page_size;
  const int begin = __ldg(p.free_begin);
  auto blocks_of = [&](int n) { return n > 0 ? div(n - 1) + 1 : 0; };

  int cached[kTabBucket], fresh[kTabBucket], need[kTabBucket];
#pragma unroll
  for (int i = 0; i < kTabBucket; ++i) {
    const bool in = i < per && b0 + i < p.B;
    cached[i] = in ? __ldg(p.cached_len + b0 + i) : 0;
    fresh[i] = in ? __ldg(p.new_len + b0 + i) : 0;
  }
  int64_t rows = 0, pages = 0;
  bool ok = true;
#pragma unroll
  for (int i = 0; i < kTabBucket; ++i) {
    const bool good = cached[i] >= 0 && fresh[i] >= 0 && static_cast<int64_t>(cached[i]) + fresh[i] <= room;
    ok &= good;
    need[i] = good ? blocks_of(cached[i] + fresh[i]) - blocks_of(cached[i]) : 0;
    rows += fresh[i];
    pages += need[i];
  }
  int64_t ir = rows, ip = pages;  // inclusive sums over the warp, then the block
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t r = __shfl_up_sync(~0u, ir, o), g = __shfl_up_sync(~0u, ip, o);
    if (lane >= o) {
      ir += r;
      ip += g;
    }
  }
  if (lane == 31) {
    s_wr[warp] = ir;
    s_wp[warp] = ip;
  }
  ok = __syncthreads_and(ok);
  int64_t total_rows = 0, total_pages = 0;
  for (int w = 0; w < nt / 32; ++w) {
    if (w < warp) {
      ir += s_wr[w];
      ip += s_wp[w];
    }
    total_rows += s_wr[w];
    total_pages += s_wp[w];
  }
  // all or nothing, as above
  ok = ok && total_rows <= p.T_cap && begin >= 0 && total_pages <= p.n_free - begin;
  if (!ok) {
    total_rows = total_pages = 0;
    if (blockIdx.x == 0 && tid == 0 && p.status) atomicOr(p.status, kErrOverflow);
  }
  int r = ok ? static_cast<int>(ir - rows) : 0, g = ok ? static_cast<int>(ip - pages) : 0;
#pragma unroll
  for (int i = 0; i < kTabBucket; ++i) {
    if (i < per && b0 + i < p.B) {
      s_row[b0 + i] = r;
      s_page[b0 + i] = g;
      s_cached[b0 + i] = cached[i];
      if (ok) {
        r += fresh[i];
        g += need[i];
      }
    }
  }
  if (tid == 0) {
    s_row[p.B] = static_cast<int>(total_rows);
    s_page[p.B] = static_cast<int>(total_pages);
  }
  __syncthreads();

  const int gtid = blockIdx.x * nt + tid, gstride = gridDim.x * nt;
  bool bad_page = false;
  for (int t = gtid; t < p.T_cap; t += gstride) {
    int slot = -1, pos = -1, owner = -1;
    if (t < total_rows) {
      owner = bucket_of(s_row, p.B, t);  // the last request that starts at or before t
      pos = s_cached[owner] + (t - s_row[owner]);
      const int blk = div(pos), old = blocks_of(s_cached[owner]);
      const int page = blk < old ? p.block_table[static_cast<int64_t>(owner) * p.max_blocks + blk]
                                 : __ldg(p.free_pages + begin + s_page[owner] + (blk - old));
      if (page >= 0 && page < p.n_pages)
        slot = page * p.page_size + (pos - blk * p.page_size);
      else
        bad_page = true;
    }
    p.slot_map[t] = slot;
    p.position[t] = pos;
    p.row_seq[t] = owner;
  }
  // new entries of the block tables (no row above reads one)
  for (int j = gtid; j < total_pages; j += gstride) {
    const int b = bucket_of(s_page, p.B, j);
    p.block_table[static_cast<int64_t>(b) * p.max_blocks + blocks_of(s_cached[b]) + (j - s_page[b])] =
        __ldg(p.free_pages + begin + j);
  }
  for (int b = gtid; b <= p.B; b += gstride) {
    p.row_start[b] = s_row[b];
    if (b < p.B) p.seq_len[b] = s_cached[b] + (s_row[b + 1] - s_row[b]);
  }
  if (gtid == 0) p.free_end[0] = begin + static_cast<int>(total_pages);
  if (bad_page && p.status) atomicOr(p.status, kErrOverflow);
}

}  // namespace

cudaError_t launch_block_tables(const TablesParams& p, int sms, cudaStream_t st) {
  // one thread per request up to the block's limit
  const int threads = p.B <= 256 ? 256 : kTabThreadsMax;
  if (p.B <= kTabKept) {
    const int grid = std::clamp((p.T_cap + threads - 1) / threads, 1, std::max(sms, 1));
    const int bytes = (3 * p.B + 2) * static_cast<int>(sizeof(int));
    if (bytes > 40 * 1024) {
      cudaError_t e =
          cudaFuncSetAttribute(block_tables_kept_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * kTabKept * 4 + 8);
      if (e != cudaSuccess) return e;
    }
    block_tables_kept_kernel<<<grid, threads, bytes, st>>>(p, page_div(p.page_size));
    return cudaGetLastError();
  }
  const int grid = std::clamp((p.T_cap + 2 * threads - 1) / (2 * threads), 1, std::max(sms, 1));  // two rows per thread
  block_tables_kernel<<<grid, threads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace dsa
