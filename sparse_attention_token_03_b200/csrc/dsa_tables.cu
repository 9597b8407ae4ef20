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
// The work is a few bytes per row and request, so the launch bounds it: one
// launch does all.  Every block repeats the prefix sums over the requests
// (one bucket of consecutive requests per thread; 8 bytes a request from L2)
// instead of waiting for another block or launch, then finds the owners of
// its rows by bisection over the bucket sums in shared memory.
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

}  // namespace

cudaError_t launch_block_tables(const TablesParams& p, cudaStream_t st) {
  // one thread per request up to the block's limit; two rows per thread
  const int threads = p.B <= 256 ? 256 : kTabThreadsMax;
  const int grid = std::clamp((p.T_cap + 2 * threads - 1) / (2 * threads), 1, 148);
  block_tables_kernel<<<grid, threads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace dsa
