// Block tables and slot maps of a step over a paged cache, from the requests' lengths.
//
// One launch: every CTA scans all requests' new tokens and needed pages itself (at most
// 4096 of them, read from L2) and then writes its own run of tokens, so no CTA waits for
// another. A new page's table entry is written by the thread of the first token in it; the
// page number itself comes from the free list, never from the table entry that another CTA
// may be writing. Bound by launch and latency, 8 bytes being written per token: 256 requests of
// 204000 new tokens 8.0 us a call, one token 6.9.
#include <algorithm>

#include "common.cuh"
#include "ptx.cuh"

namespace bsa {

int check_paged_cache(const bsa_paged_cache& c) {
  if (c.dtype != BSA_BF16 && c.dtype != BSA_F16) return fail(BSA_ERR_UNSUPPORTED, "cache dtype %d", c.dtype);
  if (c.D != 64 && c.D != 128) return fail(BSA_ERR_UNSUPPORTED, "head dim %d not in {64,128}", c.D);
  if (c.page < 16 || c.page > 256 || (c.page & (c.page - 1)))
    return fail(BSA_ERR_UNSUPPORTED, "page of %d tokens, not 16, 32, 64, 128 or 256", c.page);
  if (c.n_pages <= 0 || c.Hkv <= 0) return fail(BSA_ERR_INVALID_ARG, "empty cache");
  if (static_cast<int64_t>(c.n_pages) * c.page > INT32_MAX)
    return fail(BSA_ERR_UNSUPPORTED, "cache of 2^31 tokens or more");
  if (!c.k || !c.v) return fail(BSA_ERR_INVALID_ARG, "cache pointer is null");
  const int64_t s[6] = {c.k_page_stride, c.k_head_stride, c.k_row_stride,
                        c.v_page_stride, c.v_head_stride, c.v_row_stride};
  for (int64_t x : s)
    if (x % 8 || x < 0 || x >= (int64_t(1) << 38))
      return fail(BSA_ERR_INVALID_ARG, "cache strides must be multiples of 16 bytes, below 2^39");
  if (reinterpret_cast<uintptr_t>(c.k) % 16 || reinterpret_cast<uintptr_t>(c.v) % 16)
    return fail(BSA_ERR_INVALID_ARG, "cache pointers must be 16-byte aligned");
  return BSA_OK;
}

namespace {

constexpr int kTablesThreads = 256;
constexpr int kTablesMaxR = 4096;
constexpr int kTablesPerThread = 4;
constexpr int kTablesSite = 130;

struct TablesArgs {
  const int32_t *ctx, *new_lens;
  int R;
  int32_t* table;
  int width;
  int64_t table_stride;
  const int32_t* free_pages;
  int n_free, T, page_shift, n_pages;
  int32_t *slots, *positions, *cu, *taken;
};

__global__ void __launch_bounds__(kTablesThreads) block_tables_kernel(const TablesArgs a) {
  __shared__ int32_t s_cu[kTablesMaxR + 1];  // first new token of each request
  __shared__ int32_t s_off[kTablesMaxR];     // first free-list entry of each request
  __shared__ int64_t s_warp[2][kTablesThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int page = 1 << a.page_shift;
  int64_t base_tok = 0, base_page = 0;
  for (int r0 = 0; r0 < a.R; r0 += kTablesThreads) {
    const int r = r0 + tid;
    int64_t n = 0, need = 0;
    if (r < a.R) {
      const int c0 = a.ctx[r], n0 = a.new_lens[r];
      if ((c0 < 0 || n0 < 0) && blockIdx.x == 0) report_device_error(kStatusBadLabel, kTablesSite);
      const int64_t c = max(c0, 0);
      n = max(n0, 0);
      need = ((c + n + page - 1) >> a.page_shift) - ((c + page - 1) >> a.page_shift);
    }
    int64_t it = n, ip = need;  // inclusive sums over the threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, it, o), z = __shfl_up_sync(0xffffffffu, ip, o);
      if (lane >= o) {
        it += y;
        ip += z;
      }
    }
    if (lane == 31) {
      s_warp[0][warp] = it;
      s_warp[1][warp] = ip;
    }
    __syncthreads();
    int64_t bt = base_tok, bp = base_page;
#pragma unroll
    for (int w = 0; w < kTablesThreads / 32; ++w) {
      if (w < warp) {
        bt += s_warp[0][w];
        bp += s_warp[1][w];
      }
      base_tok += s_warp[0][w];
      base_page += s_warp[1][w];
    }
    if (r < a.R) {
      // starts past the packed length, or past the free list, are capped there
      s_cu[r] = static_cast<int32_t>(min(bt + it - n, static_cast<int64_t>(a.T)));
      s_off[r] = static_cast<int32_t>(min(bp + ip - need, static_cast<int64_t>(INT32_MAX)));
    }
    __syncthreads();
  }
  if (tid == 0) s_cu[a.R] = static_cast<int32_t>(min(base_tok, static_cast<int64_t>(a.T)));
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int r = tid; r <= a.R; r += kTablesThreads) a.cu[r] = s_cu[r];
    if (tid == 0) {
      *a.taken = static_cast<int32_t>(min(base_page, static_cast<int64_t>(INT32_MAX)));
      if (base_tok > a.T) report_device_error(kStatusBadLabel, kTablesSite + 1);
    }
  }
  const int total = s_cu[a.R];
  const int t0 = (blockIdx.x * kTablesThreads + tid) * kTablesPerThread;
  if (t0 >= a.T) return;
  int lo = 0;
  if (t0 < total) {  // last request that starts at or before t0
    int hi = a.R - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_cu[mid] <= t0) lo = mid;
      else hi = mid - 1;
    }
  }
  int slot[kTablesPerThread], pos[kTablesPerThread];
  int r = lo;
  int ctx = a.R > 0 ? max(a.ctx[r], 0) : 0;
#pragma unroll
  for (int i = 0; i < kTablesPerThread; ++i) {
    const int t = t0 + i;
    slot[i] = pos[i] = -1;
    if (t >= total || t >= a.T) continue;
    while (r + 1 < a.R && s_cu[r + 1] <= t) {  // requests without new tokens are passed over
      ++r;
      ctx = max(a.ctx[r], 0);
    }
    const int64_t p = static_cast<int64_t>(ctx) + (t - s_cu[r]);
    if (p > INT32_MAX) {
      report_device_error(kStatusBadLabel, kTablesSite + 2);
      continue;
    }
    pos[i] = static_cast<int>(p);
    const int64_t j = p >> a.page_shift, have = (static_cast<int64_t>(ctx) + page - 1) >> a.page_shift;
    if (j >= a.width) {
      report_device_error(kStatusBadLabel, kTablesSite + 3);
      continue;
    }
    int32_t* entry = a.table + r * a.table_stride + j;
    int id = -1;
    if (j < have) {
      id = *entry;
      if (id < 0 || id >= a.n_pages) {
        report_device_error(kStatusBadLabel, kTablesSite + 4);
        id = -1;
      }
    } else {
      const int64_t f = s_off[r] + (j - have);
      if (f < a.n_free) {
        id = a.free_pages[f];
        if (id < 0 || id >= a.n_pages) {
          report_device_error(kStatusBadLabel, kTablesSite + 5);
          id = -1;
        }
      }
      if ((p & (page - 1)) == 0) *entry = id;
    }
    if (id >= 0) slot[i] = (id << a.page_shift) + static_cast<int>(p & (page - 1));
  }
  if (t0 + kTablesPerThread <= a.T && reinterpret_cast<uintptr_t>(a.slots) % 16 == 0 &&
      reinterpret_cast<uintptr_t>(a.positions) % 16 == 0) {
    *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
  } else {
#pragma unroll
    for (int i = 0; i < kTablesPerThread; ++i)
      if (t0 + i < a.T) {
        a.slots[t0 + i] = slot[i];
        a.positions[t0 + i] = pos[i];
      }
  }
}

}  // namespace
}  // namespace bsa

extern "C" int bsa_paged_block_tables(const int32_t* context_lens, const int32_t* new_lens, int R,
                                      int32_t* block_table, int width, int64_t table_stride,
                                      const int32_t* free_pages, int n_free, int T, int page,
                                      int n_pages, int32_t* slots, int32_t* positions,
                                      int32_t* cu_new, int32_t* taken, void* stream) {
  using namespace bsa;
  if (R < 0 || T < 0 || width < 0 || n_free < 0 || n_pages < 0)
    return fail(BSA_ERR_INVALID_ARG, "negative size");
  if (R > kTablesMaxR) return fail(BSA_ERR_UNSUPPORTED, "%d requests, at most %d", R, kTablesMaxR);
  if (page < 16 || page > 256 || (page & (page - 1)))
    return fail(BSA_ERR_UNSUPPORTED, "page of %d tokens, not 16, 32, 64, 128 or 256", page);
  if (static_cast<int64_t>(n_pages) * page > INT32_MAX)
    return fail(BSA_ERR_UNSUPPORTED, "cache of 2^31 tokens or more");
  if (T > INT32_MAX - kTablesThreads * kTablesPerThread) return fail(BSA_ERR_UNSUPPORTED, "T too large");
  if (table_stride < width && R > 1) return fail(BSA_ERR_INVALID_ARG, "table_stride < width");
  if (!cu_new || !taken || (R > 0 && (!context_lens || !new_lens)) ||
      (R > 0 && width > 0 && !block_table) || (n_free > 0 && !free_pages) ||
      (T > 0 && (!slots || !positions)))
    return fail(BSA_ERR_INVALID_ARG, "null pointer");
  TablesArgs a{context_lens, new_lens, R, block_table, width, table_stride, free_pages, n_free, T,
               __builtin_ctz(page), n_pages, slots, positions, cu_new, taken};
  const int per = kTablesThreads * kTablesPerThread;
  block_tables_kernel<<<std::max(1, ceil_div(T, per)), kTablesThreads, 0, as_stream(stream)>>>(a);
  count_launch();
  return check_cuda(cudaGetLastError(), "block_tables_kernel");
}
