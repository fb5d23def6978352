// Attention of every request's new tokens over its paged cache, block-sparse at page
// granularity. The rows of one (request, KV head) are its tokens times the G query heads of
// the KV head (row = token * G + head), so a key is read once for all heads that share it.
// Two kernels split the requests by that row count:
//
//   paged_token_kernel  at most kTokenRows rows (a step of single or few tokens). Bound by the
//       cache's bytes: keys and values go from global memory straight into the registers
//       that the matrix instruction takes, 16 keys at a time, with no shared memory on the
//       way. The (request, head, 64-key chunk) space is cut into equal contiguous spans, one
//       per CTA, so ragged lengths balance; a (request, head) that crosses a span border
//       leaves partial results that token_combine_kernel joins. 64 requests of 11000 keys on
//       average (24 / 8 heads of 128): 448 us, the cache's bytes at the measured copy rate; one
//       request of 32761 keys: 32 us, floor 20 us, the rest is the way from the lengths over the
//       pages to the first keys, and the join. Spans are cut by the requests' lengths alone, so
//       masked pages count as work: the 64 requests with two pages of five kept at random take 230
//       us in single calls, floor 179.
//   paged_tile_kernel   more rows. tcgen05: two 128-row tiles per CTA over 128-key chunks
//       gathered page by page with TMA, logits and weights in TMEM, two softmax threads per
//       row. Long requests are split over CTAs and tile_combine_kernel joins the parts. 1560
//       rows of 40 heads over 32760 keys: 970 us in single calls (1080 TFLOP/s, 0.65 of the
//       burst peak), 1.13 ms in calls without a pause, where the power limit lowers the
//       clocks. Of a chunk's 3400 cycles the tensor core works 2600 and the exponentials take
//       2050 of the special-function units; the rest is what passes between the two.
//
// Sums of a softmax are kept in fp32, in base-2 units: relative to a running maximum in the token
// kernel, to a fixed reference in the tile kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "ptx_paged.cuh"

namespace bsa {

namespace {

constexpr int kTokenRows = 16;      // rows per (request, KV head) of the token kernel
constexpr int kPagedMaxR = 4096;    // requests of one call
constexpr int kPagedSite = 140;

struct PagedArgs {
  const void* q;
  int64_t qh, qt;
  const void *kc, *vc;
  int64_t kp, kh, kr, vp, vh, vr;
  int n_pages, page_shift, Hkv, G, T, R;
  const int32_t* table;
  int width;
  int64_t table_stride;
  const int32_t *cu, *ctx;
  const uint8_t* mask;
  int64_t mr, mg;
  float scale_log2;
  int causal;
  void* out;
  int64_t oh, ot;
  int max_new;   // host bound of new tokens per request
  int min_rows;  // requests of at most this many rows belong to the token kernel
  float* part;
  int tile_ctas;   // tile kernel: CTAs per KV head (a bound: those past the last one end at once)
  int can_split;   // tile kernel: 0 when no request is long enough to be split
  int heads_first; // tile kernel: neighbouring CTAs take one job of all KV heads
  int workers;     // token kernel: CTAs
  int tok_rows;    // token kernel: rows of a request that its instance holds (8 or 16)
  int one_each;    // token kernel: one CTA per (request, KV head), nothing to join
};

// A request's lengths, made safe against any device contents: token range inside [0, T),
// context inside the table's reach.
struct Request {
  int t0, n;    // first token, tokens
  int ctx, len; // cached tokens before, keys in all
};

__device__ __forceinline__ Request load_request(const PagedArgs& a, int r) {
  Request q;
  const int t0 = a.cu[r], t1 = a.cu[r + 1];
  q.t0 = min(max(t0, 0), a.T);
  q.n = max(min(t1, a.T) - q.t0, 0);
  const int64_t reach = static_cast<int64_t>(a.width) << a.page_shift;
  const int64_t c = max(a.ctx[r], 0);
  q.ctx = static_cast<int>(min(c, reach));
  q.len = static_cast<int>(min(c + q.n, reach));
  return q;
}

__device__ __forceinline__ void check_request(const PagedArgs& a, int r) {
  const int64_t reach = static_cast<int64_t>(a.width) << a.page_shift;
  const int t0 = a.cu[r], t1 = a.cu[r + 1], c = a.ctx[r];
  const bool ok = t0 >= 0 && t1 >= t0 && t1 <= a.T && c >= 0 && t1 - t0 <= a.max_new &&
                  (t1 == t0 || static_cast<int64_t>(c) + (t1 - t0) <= reach);
  if (!ok) report_device_error(kStatusBadLabel, kPagedSite);
}

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  } else {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
}

// ================================================================ token kernel
// Two warps to a CTA and six CTAs per SM (by registers): at every border between two (request,
// head)s a CTA's warps wait for new queries, pages and keys, so more and smaller CTAs pass fewer
// borders each. 64 requests of 333 keys on average: 37 us, with four warps 41, with one 35;
// one request of 301 keys: 12, 10 and 14.
constexpr int kTokWarps = 2;
constexpr int kTokThreads = 32 * kTokWarps;
constexpr int kTokChunk = 64;     // keys of a work unit: two 16-key blocks per warp

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
      : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
      : "l"(p));
  return r;
}

template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}

// Weight of a partial result (maximum m, sum l) under the joint maximum: 0 for one that saw no key,
// NaN for one whose logits were all NaN (which no maximum shows).
__device__ __forceinline__ float part_weight(float m, float l, float joint) {
  return m == -INFINITY ? l : ex2(m - joint);
}

// Chunks of 64 keys of request r that the token kernel takes (0 for one of the tile kernel's).
__device__ __forceinline__ int token_chunks(const PagedArgs& a, const Request& q) {
  if (q.n <= 0 || q.n * static_cast<int64_t>(a.G) > a.tok_rows) return 0;
  return (q.len + kTokChunk - 1) / kTokChunk;
}

// The unit space: request-major, then KV head, then chunk; CTA w takes [w*span, (w+1)*span).
__device__ __forceinline__ int64_t token_span(int64_t units, int workers) {
  const int64_t s = (units + workers - 1) / workers;
  return s < 1 ? 1 : s;
}

// Partial results: two slots per CTA (0: a (request, head) that began before its span, 1: one
// that goes on behind it), each O (kTokenRows x D) unnormalised, then (max, sum) pairs.
__device__ __forceinline__ float* token_slot(const PagedArgs& a, int w, int slot, int D) {
  return a.part + (static_cast<size_t>(w) * 2 + slot) * kTokenRows * (D + 2);
}

// One warp's share of a (request, head): S^T = K Q^T with 16 keys as the M side and 8 rows
// as the N side, then O^T = V^T P^T. A lane (g = lane / 4, c = lane % 4) holds 16-byte pieces
// of keys g and g + 8 for the first product (the order of D inside a product is free, so a
// piece serves two K-steps), and of keys 2c, 2c+1, 2c+8, 2c+9 for the second, whose pairs of
// neighbouring keys are interleaved with byte permutes; the weights reach their second
// product's lane with one 8x8 transposition.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kTokThreads) paged_token_kernel(const PagedArgs a) {
  constexpr int KC = D / 32;  // 16-byte pieces of a key per lane (first product)
  constexpr int VC = D / 64;  // 16-byte pieces of a value row per lane (second product)
  constexpr int MT = D / 16;  // 16-wide slices of D in the second product
  extern __shared__ int32_t s_units[];  // prefix of units per KV head: R + 1 entries
  __shared__ float s_o[kTokWarps][8 * NT][D + 4];
  __shared__ float s_m[kTokWarps][8 * NT], s_l[kTokWarps][8 * NT];
  __shared__ int s_warp[kTokWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;

  int64_t u_begin, u_end;
  if (a.one_each) {
    if (tid == 0) check_request(a, blockIdx.x / a.Hkv);
    u_begin = 0;
    u_end = 1;
  } else {
    int base = 0;
    for (int r0 = 0; r0 < a.R; r0 += kTokThreads) {
      const int r = r0 + tid;
      int n = 0;
      if (r < a.R) {
        if (blockIdx.x == 0) check_request(a, r);
        n = token_chunks(a, load_request(a, r));
      }
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) s_warp[warp] = incl;
      __syncthreads();
      int b = base;
#pragma unroll
      for (int w = 0; w < kTokWarps; ++w) {
        if (w < warp) b += s_warp[w];
        base += s_warp[w];
      }
      if (r < a.R) s_units[r] = b + incl - n;
      __syncthreads();
    }
    if (tid == 0) s_units[a.R] = base;
    __syncthreads();
    const int64_t units = static_cast<int64_t>(base) * a.Hkv;
    const int64_t span = token_span(units, a.workers);
    u_begin = span * blockIdx.x;
    u_end = min(units, u_begin + span);
  }

  launch_dependents();
  for (int64_t u = u_begin; u < u_end;) {
    // the (request, head) of unit u and the chunks of it that lie in this span
    int r, h, ch0, ch1, nch;
    if (a.one_each) {
      r = blockIdx.x / a.Hkv;
      h = blockIdx.x % a.Hkv;
      ch0 = 0;
      ch1 = nch = token_chunks(a, load_request(a, r));
      u = u_end;
      if (nch == 0) break;
    } else {
      int lo = 0, hi = a.R - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (static_cast<int64_t>(s_units[mid]) * a.Hkv <= u) lo = mid;
        else hi = mid - 1;
      }
      r = lo;
      nch = s_units[r + 1] - s_units[r];
      const int64_t in = u - static_cast<int64_t>(s_units[r]) * a.Hkv;
      h = static_cast<int>(in / nch);
      ch0 = static_cast<int>(in % nch);
      ch1 = static_cast<int>(min(static_cast<int64_t>(nch), ch0 + (u_end - u)));
      u += ch1 - ch0;
    }
    const Request q = load_request(a, r);
    const int rows = q.n * a.G;

    // Q: row 8 nt + g of the group, pieces of 8 values at 32 j + 8 c
    uint4 qf[NT][KC];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = 8 * nt + g;
#pragma unroll
      for (int j = 0; j < KC; ++j) qf[nt][j] = make_uint4(0, 0, 0, 0);
      if (row < rows) {
        const T* p = static_cast<const T*>(a.q) + (static_cast<int64_t>(h) * a.G + row % a.G) * a.qh +
                     static_cast<int64_t>(q.t0 + row / a.G) * a.qt;
#pragma unroll
        for (int j = 0; j < KC; ++j) qf[nt][j] = ldg_stream(p + 32 * j + 8 * c);
      }
    }
    // last key that the lane's two softmax rows (2c, 2c + 1 of each 8) see
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 8 * nt + 2 * c + i;
        lim[nt][i] = row < rows ? min(a.causal ? q.ctx + row / a.G : q.len - 1, q.len - 1) : -1;
      }
    const int lim_all = a.causal ? min(q.ctx, q.len - 1) : q.len - 1;  // keys every row sees

    float m[NT][2], l[NT][2], o[MT][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][nt][i] = 0.f;
    }

    const T* kbase = static_cast<const T*>(a.kc) + h * a.kh;
    const T* vbase = static_cast<const T*>(a.vc) + h * a.vh;
    const int32_t* trow = a.table + r * a.table_stride;
    const uint8_t* mrow = a.mask ? a.mask + r * a.mr + h * a.mg : nullptr;
    const int blk_end = min(ch1 * (kTokChunk / 16), (q.len + 15) >> 4);
    const int bpp_shift = a.page_shift - 4;  // 16-key blocks per page
    // page of a block, -1 where there is nothing to read
    auto page_of = [&](int blk) -> int {
      if (blk >= blk_end) return -1;
      const int pg = blk >> bpp_shift;
      if (mrow && !mrow[pg]) return -1;
      const int id = trow[pg];
      if (id < 0 || id >= a.n_pages) {
        if (lane == 0) report_device_error(kStatusBadLabel, kPagedSite + 1);
        return -1;
      }
      return id;
    };
    uint4 kf[2][KC], vf[4][VC];
    auto load_k = [&](int id, int blk) {
      const int row0 = (blk << 4) & ((1 << a.page_shift) - 1);
      const T* p = kbase + static_cast<int64_t>(id) * a.kp + static_cast<int64_t>(row0) * a.kr + 8 * c;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool in = (blk << 4) + g + 8 * i < q.len;
#pragma unroll
        for (int j = 0; j < KC; ++j)
          kf[i][j] = in ? ldg_stream(p + (g + 8 * i) * a.kr + 32 * j) : make_uint4(0, 0, 0, 0);
      }
    };
    auto load_v = [&](int id, int blk) {
      const int row0 = (blk << 4) & ((1 << a.page_shift) - 1);
      const T* p = vbase + static_cast<int64_t>(id) * a.vp + static_cast<int64_t>(row0) * a.vr + 8 * g;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = 2 * c + (i & 1) + 8 * (i >> 1);
        const bool in = (blk << 4) + key < q.len;  // rows behind the last key count as zeros
#pragma unroll
        for (int j = 0; j < VC; ++j)
          vf[i][j] = in ? ldg_stream(p + key * a.vr + 64 * j) : make_uint4(0, 0, 0, 0);
      }
    };

    int blk = ch0 * (kTokChunk / 16) + warp;
    int id = page_of(blk), id_next = page_of(blk + kTokWarps);
    if (id >= 0) {
      load_k(id, blk);
      load_v(id, blk);
    }
#pragma unroll 1
    for (; blk < blk_end; blk += kTokWarps) {
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
        if (id >= 0) {
#pragma unroll
          for (int j = 0; j < KC; ++j) {
            mma_16816<T>(s[nt], kf[0][j].x, kf[1][j].x, kf[0][j].y, kf[1][j].y, qf[nt][j].x, qf[nt][j].y);
            mma_16816<T>(s[nt], kf[0][j].z, kf[1][j].z, kf[0][j].w, kf[1][j].w, qf[nt][j].z, qf[nt][j].w);
          }
        }
      }
      // the next block's keys are on their way during this block's softmax
      if (id_next >= 0) load_k(id_next, blk + kTokWarps);
      const int id_after = page_of(blk + 2 * kTokWarps);
      if (id >= 0) {
        const int key = (blk << 4) + g;
        const bool edge = (blk << 4) + 15 > lim_all;
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = s[nt][i] * a.scale_log2;
            if (edge && key + 8 * (i >> 1) > lim[nt][i & 1]) x[i] = -INFINITY;
          }
          float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
          }
          // The running maximum moves only when it is passed by more than 8 (weights stay
          // below 2^8), so the accumulators are rarely rescaled.
          const bool need = mx0 > m[nt][0] + 8.f || mx1 > m[nt][1] + 8.f;
          if (__any_sync(0xffffffffu, need)) {
            const float n0 = fmaxf(m[nt][0], mx0), n1 = fmaxf(m[nt][1], mx1);
            const float f0 = n0 == -INFINITY ? 1.f : ex2(m[nt][0] - n0);
            const float f1 = n1 == -INFINITY ? 1.f : ex2(m[nt][1] - n1);
            m[nt][0] = n0;
            m[nt][1] = n1;
            l[nt][0] *= f0;
            l[nt][1] *= f1;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              o[t][nt][0] *= f0;
              o[t][nt][1] *= f1;
              o[t][nt][2] *= f0;
              o[t][nt][3] *= f1;
            }
          }
          const float b0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
          const float b1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
          const float p0 = ex2(x[0] - b0), p1 = ex2(x[1] - b1), p2 = ex2(x[2] - b0), p3 = ex2(x[3] - b1);
          l[nt][0] += p0 + p2;
          l[nt][1] += p1 + p3;
          pb[nt][0] = transpose8x8(pack_pair<T>(p0, p1));
          pb[nt][1] = transpose8x8(pack_pair<T>(p2, p3));
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const int j = t / 4, w = t % 4;
          const uint32_t k0 = word_of(vf[0][j], w), k1 = word_of(vf[1][j], w);
          const uint32_t k8 = word_of(vf[2][j], w), k9 = word_of(vf[3][j], w);
          const uint32_t a0 = __byte_perm(k0, k1, 0x5410), a1 = __byte_perm(k0, k1, 0x7632);
          const uint32_t a2 = __byte_perm(k8, k9, 0x5410), a3 = __byte_perm(k8, k9, 0x7632);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_16816<T>(o[t][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
        }
      }
      if (id_next >= 0) load_v(id_next, blk + kTokWarps);
      id = id_next;
      id_next = id_after;
    }

    // the warps' results of this (request, head) joined through shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], d);
        if (g == 0) {
          s_m[warp][8 * nt + 2 * c + i] = m[nt][i];
          s_l[warp][8 * nt + 2 * c + i] = l[nt][i];
        }
      }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int d = (t / 4) * 64 + 8 * g + 2 * (t % 4);
          *reinterpret_cast<float2*>(&s_o[warp][8 * nt + 2 * c + i][d]) =
              make_float2(o[t][nt][i], o[t][nt][i + 2]);
        }
    __syncthreads();
    const bool whole = ch0 == 0 && ch1 == nch;
    float* slot = whole ? nullptr : token_slot(a, blockIdx.x, ch0 == 0 ? 1 : 0, D);
    for (int e = tid; e < rows * (D / 2); e += kTokThreads) {
      const int row = e / (D / 2), d = 2 * (e % (D / 2));
      float mt = -INFINITY;
#pragma unroll
      for (int w = 0; w < kTokWarps; ++w) mt = fmaxf(mt, s_m[w][row]);
      float lt = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
      for (int w = 0; w < kTokWarps; ++w) {
        const float f = part_weight(s_m[w][row], s_l[w][row], mt);
        lt = fmaf(s_l[w][row], f, lt);
        if (f != 0.f) {
          o0 = fmaf(s_o[w][row][d], f, o0);
          o1 = fmaf(s_o[w][row][d + 1], f, o1);
        }
      }
      if (whole) {
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
        T* po = static_cast<T*>(a.out) + (static_cast<int64_t>(h) * a.G + row % a.G) * a.oh +
                static_cast<int64_t>(q.t0 + row / a.G) * a.ot + d;
        *reinterpret_cast<uint32_t*>(po) = pack_pair<T>(o0 * inv, o1 * inv);
      } else {
        *reinterpret_cast<float2*>(slot + row * D + d) = make_float2(o0, o1);
        if (d == 0)
          *reinterpret_cast<float2*>(slot + kTokenRows * D + 2 * row) = make_float2(mt, lt);
      }
    }
    __syncthreads();
  }
}

// Joins the partial results of one row of a (request, KV head): grid (requests * heads, rows).
// The warps take the CTAs that shared the work in turn, their results are joined in order
// through shared memory. (One warp per row walking over all of them took 31 us for the 52
// CTAs of a 32761-key row, longer than the attention itself.)
constexpr int kCombWarps = 8;
template <typename T, int D>
__global__ void __launch_bounds__(32 * kCombWarps) token_combine_kernel(const PagedArgs a) {
  __shared__ int s_sum[2][kCombWarps];
  __shared__ float s_acc[kCombWarps][D];
  __shared__ float2 s_ml[kCombWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv, row = blockIdx.y;
  launch_dependents();
  // the lengths are inputs of the call, so the place of the row is found before the wait
  int before = 0, all = 0;
  for (int i = tid; i < a.R; i += 32 * kCombWarps) {
    const int n = token_chunks(a, load_request(a, i));
    all += n;
    if (i < r) before += n;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  all = __reduce_add_sync(0xffffffffu, all);
  if (lane == 0) {
    s_sum[0][warp] = before;
    s_sum[1][warp] = all;
  }
  __syncthreads();
  before = all = 0;
#pragma unroll
  for (int w = 0; w < kCombWarps; ++w) {
    before += s_sum[0][w];
    all += s_sum[1][w];
  }
  const Request q = load_request(a, r);
  const int nch = token_chunks(a, q);
  wait_for_primary();  // before any return: a dependent that has ended stands for its primary
  if (nch == 0 || row >= q.n * a.G) return;
  const int64_t span = token_span(static_cast<int64_t>(all) * a.Hkv, a.workers);
  const int64_t u0 = static_cast<int64_t>(before) * a.Hkv + static_cast<int64_t>(h) * nch;
  const int w0 = static_cast<int>(u0 / span), w1 = static_cast<int>((u0 + nch - 1) / span);
  if (w0 == w1) return;  // one CTA had all of it and wrote the result
  constexpr int kAhead = 8;  // parts on their way to a warp
  float mt = -INFINITY, lt = 0.f, acc[D / 32] = {};
  for (int w = w0 + warp; w <= w1; w += kAhead * kCombWarps) {
    float2 ml[kAhead], v[kAhead][D / 64];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int wi = w + i * kCombWarps;
      ml[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < D / 64; ++e) v[i][e] = make_float2(0.f, 0.f);
      if (wi <= w1) {
        const float* s = token_slot(a, wi, wi == w0 ? 1 : 0, D);
        ml[i] = *reinterpret_cast<const float2*>(s + kTokenRows * D + 2 * row);
#pragma unroll
        for (int e = 0; e < D / 64; ++e) v[i][e] = *reinterpret_cast<const float2*>(s + row * D + 64 * e + 2 * lane);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (ml[i].x == -INFINITY && ml[i].y == 0.f) continue;  // saw no key of this row
      const float mn = fmaxf(mt, ml[i].x), f0 = ex2(mt - mn), f1 = ex2(ml[i].x - mn);
      lt = lt * f0 + ml[i].y * f1;
#pragma unroll
      for (int e = 0; e < D / 64; ++e) {
        acc[2 * e] = acc[2 * e] * f0 + v[i][e].x * f1;
        acc[2 * e + 1] = acc[2 * e + 1] * f0 + v[i][e].y * f1;
      }
      mt = mn;
    }
  }
  if (lane == 0) s_ml[warp] = make_float2(mt, lt);
#pragma unroll
  for (int e = 0; e < D / 64; ++e)
    *reinterpret_cast<float2*>(&s_acc[warp][64 * e + 2 * lane]) = make_float2(acc[2 * e], acc[2 * e + 1]);
  __syncthreads();
  if (tid < D / 2) {
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kCombWarps; ++w) m = fmaxf(m, s_ml[w].x);
    float l = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int w = 0; w < kCombWarps; ++w) {
      const float f = part_weight(s_ml[w].x, s_ml[w].y, m);
      l = fmaf(s_ml[w].y, f, l);
      o0 = fmaf(s_acc[w][2 * tid], f, o0);
      o1 = fmaf(s_acc[w][2 * tid + 1], f, o1);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* po = static_cast<T*>(a.out) + (static_cast<int64_t>(h) * a.G + row % a.G) * a.oh +
            static_cast<int64_t>(q.t0 + row / a.G) * a.ot;
    *reinterpret_cast<uint32_t*>(po + 2 * tid) = pack_pair<T>(o0 * inv, o1 * inv);
  }
}

// ================================================================ tile kernel
constexpr int kTileRows = 256;   // rows of a CTA: two 128-row tiles
constexpr int kTileStages = 5;   // K/V stages of 128 rows
constexpr int kTileInfo = 4;     // chunk records in flight
constexpr int kTileThreads = 640;  // 16 softmax warps, two MMA warps, one TMA warp, one that waits for it
// Registers: the launch gives every thread 96 (65536 / 640, in steps of 8); the softmax
// warpgroups take 104 each, the last one keeps 64: 512 * 104 + 128 * 64 = 640 * 96.
constexpr int kSoftmaxRegs = 104, kOtherRegs = 64;

// A chunk's record: the key position of each of its eight 16-key granules (kAbsent where the
// chunk holds none), the rows of it that hold keys, and the last position in it (kAbsent when
// a granule is absent or a row of it lies behind the last key). rows == 0 ends the list.
constexpr int kAbsent = 0x3fffffff;
struct TileInfo {
  int pos[8];
  int rows, last;
};

template <int D>
struct TileCfg {
  static constexpr int TILE = 128 * D * 2;  // one operand tile
  static constexpr int NATOM = D / 64;      // 128-byte column slices
  static constexpr int MISC = 512 + 2 * 2 * 128 * 4;  // barriers and records, row maxima
  static constexpr int SMEM = (2 + kTileStages) * TILE + MISC;  // 231936 bytes at D = 128
  // one CTA per SM: it takes all 512 TMEM columns
  static constexpr int SMEM_LAUNCH = SMEM > 120 * 1024 ? SMEM : 120 * 1024;
};

enum {
  TB_KV_FULL = 0,
  TB_KV_EMPTY = TB_KV_FULL + kTileStages,
  TB_INFO = TB_KV_EMPTY + kTileStages,
  TB_Q = TB_INFO + kTileInfo,
  TB_S,             // four: logits of the keys 0..63 and 64..127 of a chunk ready, by tile
  TB_P = TB_S + 4,  // four: their weights written
  TB_X = TB_P + 4,  // eight: first maxima exchanged between a tile's halves, by 32 rows
  TB_TAIL = TB_X + 8,      // value rows without a key in the last chunk are zeros
  TB_DRAIN = TB_TAIL + 1,  // two
  TB_COUNT = TB_DRAIN + 2
};

// How the tile kernel's work is cut. A request's rows make tile pairs of 256 rows, and a pair's
// keys are split over CTAs so that none has many more than `quantum` chunks of 128 keys. With
// `share` the chunks of one SM if the whole call's were spread evenly: half the share where it is
// long (32 chunks, some 60 us), so that long requests are split among short ones and the last
// CTA ends little after the others; the share itself where it is short; and at least
// kTileMinChunks, since a CTA costs about as much as 4 chunks to start and end. A quantum below
// kTileLongShare, which a share of up to 63 chunks gives, then grows in calls of up to 32 requests
// until one wave does it all or nothing is split any more. With many more pairs than SMs none is
// split. Chunks are counted by the requests' lengths alone: a page mask, and the keys that a causal
// tile does not see, are not taken off. All of it follows from the lengths, which live on the GPU, so
// each CTA works it out.
constexpr int kTileSms = 148;
constexpr int kTileJobs = 2 * kTileSms;  // the quantum is never below the work over this
constexpr int kTileLongShare = 32;
constexpr int kTileMinChunks = 8;

struct TileJob {
  int r, tile, split, splits;
  int slot;  // of the partial results, when splits > 1: slot + split
};

__device__ __forceinline__ int tile_pairs(const PagedArgs& a, const Request& q) {
  const int64_t rows = static_cast<int64_t>(q.n) * a.G;
  return rows > a.min_rows ? static_cast<int>((rows + kTileRows - 1) / kTileRows) : 0;
}
__device__ __forceinline__ int tile_chunks(const Request& q) { return (q.len + 127) >> 7; }

__device__ __forceinline__ int64_t tile_quantum(const PagedArgs& a, int64_t work) {
  const int64_t all = work * a.Hkv, share = (all + kTileSms - 1) / kTileSms;
  if (share >= kTileLongShare) return (all + kTileJobs - 1) / kTileJobs;
  return share < kTileMinChunks ? kTileMinChunks : share;
}
// Up to a quarter more than the quantum is not split.
__device__ __forceinline__ int tile_splits(int chunks, int64_t quantum) {
  return 4 * static_cast<int64_t>(chunks) <= 5 * quantum ? 1 : static_cast<int>((chunks + quantum - 1) / quantum);
}

// CTA u's job of a KV head (by one warp, 32 requests at a time); with kJoin, the u-th pair that
// is split. False where there is none. Causal tiles near the end of a request see the most keys,
// so the last jobs go to the first CTAs. With heads first the CTAs without a job come last, except
// in calls of more than 32 requests, where counting the jobs would read the lengths once more.
template <bool kJoin>
__device__ __forceinline__ bool find_tile(const PagedArgs& a, int u, int lane, TileJob* job) {
  int pairs = 0, chunks = 0;  // of the lane's request of a round
  auto look = [&](int r0) {
    pairs = chunks = 0;
    if (r0 + lane < a.R) {
      const Request q = load_request(a, r0 + lane);
      pairs = tile_pairs(a, q);
      chunks = tile_chunks(q);
    }
  };
  look(0);
  int64_t quantum = INT32_MAX;
  if (a.can_split) {
    int64_t work = static_cast<int64_t>(pairs) * chunks;
    if (a.R > 32) {
      for (int r0 = 32; r0 < a.R; r0 += 32) {
        look(r0);
        work += static_cast<int64_t>(pairs) * chunks;
      }
      look(0);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) work += __shfl_xor_sync(0xffffffffu, work, o);
    quantum = tile_quantum(a, work);
    // Rounding up makes more jobs than the share allows for; where one wave is to do it all, the
    // quantum grows until it does (40 pairs of 68 chunks: 120 jobs of 23 chunks, 64 us; as 160 jobs
    // of 17 chunks, in two waves, 75), or until nothing is left to split (43 pairs of 2 to 68 chunks,
    // share 36: 372 jobs at a quantum of 18, 228 at 46, then 172 whole ones).
    if (a.R <= 32 && quantum < kTileLongShare) {
      for (int i = 0; i < 4; ++i) {
        const int jobs = __reduce_add_sync(0xffffffffu, pairs * tile_splits(chunks, quantum)) * a.Hkv;
        if (jobs <= kTileSms || __all_sync(0xffffffffu, pairs == 0 || tile_splits(chunks, quantum) == 1)) break;
        quantum = (quantum * jobs + kTileSms - 1) / kTileSms;
      }
    }
  }
  if (!kJoin) {
    const int jobs = a.heads_first && a.R <= 32 ? __reduce_add_sync(0xffffffffu, pairs * tile_splits(chunks, quantum)) : a.tile_ctas;
    u = jobs - 1 - u;
    if (u < 0) return false;
  }
  int base = 0, slots = 0;
  for (int r0 = 0; r0 < a.R; r0 += 32) {
    if (r0 > 0) look(r0);
    const int ns = tile_splits(chunks, quantum);
    const int n = kJoin ? (ns > 1 ? pairs : 0) : pairs * ns;  // this lane's jobs
    const int p = ns > 1 ? pairs * ns : 0;                    // and partial results
    int incl = n, pincl = p;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o), z = __shfl_up_sync(0xffffffffu, pincl, o);
      if (lane >= o) {
        incl += y;
        pincl += z;
      }
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + incl > u);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int k = u - base - __shfl_sync(0xffffffffu, incl - n, src);
      job->r = r0 + src;
      job->splits = __shfl_sync(0xffffffffu, ns, src);
      job->tile = kJoin ? k : k / job->splits;
      job->split = kJoin ? 0 : k % job->splits;
      job->slot = slots + __shfl_sync(0xffffffffu, pincl - p, src) + job->tile * job->splits;
      return true;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
    slots += __shfl_sync(0xffffffffu, pincl, 31);
  }
  return false;
}

// A pair is split only if it has more chunks than the quantum, which is at least the work over
// kTileJobs: the pairs that are split have at most 2 kTileJobs parts between them, over all heads.
constexpr int kTileSlots = 2 * kTileJobs;

__device__ __forceinline__ size_t tile_part_row(const PagedArgs& a, int slot, int h, int row) {
  return (static_cast<size_t>(slot) * a.Hkv + h) * kTileRows + row;
}
__device__ __forceinline__ float* tile_part_ml(const PagedArgs& a, int D) {
  return a.part + static_cast<size_t>(kTileSlots) * kTileRows * D;
}

// A softmax warp's chunks in an exact pass of the tile kernel: as its loop, 32 keys at a time, with
// the reference and the largest logit taken before the scale. A function of its own, so that the
// loop keeps its registers (inlined it cost that loop 1.6 %).
struct ExactPass {
  uint32_t bar0, tS;
  const TileInfo* info;
  volatile int* abort_flag;
  int t, hb, lim, lim_tile;
  float base, scale_log2;
};
template <typename T>
__device__ __noinline__ bool exact_pass(const ExactPass& e, float* largest, float* sum, int* chunks) {
  auto wait_all = [&](int bar, uint32_t parity, int site) -> bool {
    return __all_sync(0xffffffffu, mbar_wait_poll(e.bar0 + 8u * bar, parity, e.abort_flag, site));
  };
  float seen = -INFINITY, l = 0.f;
  int nch = 0;
#pragma unroll 1
  for (int j = 0;; ++j) {
    if (!wait_all(TB_INFO + j % kTileInfo, (j / kTileInfo) & 1, kPagedSite + 30)) return false;
    const TileInfo* ti = e.info + j % kTileInfo;
    if (ti->rows == 0) break;
    const bool edge = ti->last > e.lim_tile, has = ti->rows > 64 * e.hb;
    ++nch;
    if (!has) break;  // (the last chunk)
    if (!wait_all(TB_S + 2 * e.t + e.hb, j & 1, kPagedSite + 31)) return false;
    tc_fence_after();
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      float v[32];
      tmem_ld32(e.tS + 32 * i, v);
      tmem_wait_ld();
      uint32_t w[16];
      const int vis0 = edge ? e.lim - ti->pos[4 * e.hb + 2 * i] : 16;  // last visible column of a granule
      const int vis1 = edge ? e.lim - ti->pos[4 * e.hb + 2 * i + 1] : 16;
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (c % 16 > (c < 16 ? vis0 : vis1)) v[c] = -INFINITY;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        seen = max3(seen, v[2 * c], v[2 * c + 1]);
        const float x0 = ex2((v[2 * c] - e.base) * e.scale_log2), x1 = ex2((v[2 * c + 1] - e.base) * e.scale_log2);
        l += x0 + x1;
        w[c] = pack_pair<T>(x0, x1);
      }
      tmem_st16(e.tS + 16 * i, w);
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(e.bar0 + 8u * (TB_P + 2 * e.t + e.hb));
  }
  *largest = seen;
  *sum = l;
  *chunks = nch;
  return true;
}

template <typename T, int D>
__global__ void __launch_bounds__(kTileThreads, 1)
    paged_tile_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const PagedArgs a) {
  using Cfg = TileCfg<D>;
  constexpr bool kF16 = std::is_same<T, __half>::value;
  extern __shared__ __align__(1024) uint8_t tile_smem[];  // swizzled tiles start on 1 KB
  uint8_t* smem = tile_smem;
  const uint32_t sQ = smem_u32(smem), sKV = sQ + 2 * Cfg::TILE;
  uint8_t* misc = smem + (2 + kTileStages) * Cfg::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(misc);
  TileInfo* info = reinterpret_cast<TileInfo*>(misc + 8 * TB_COUNT);
  int* ids = reinterpret_cast<int*>(info + kTileInfo);  // 8: page ids of the chunk being loaded
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ids + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* never = reinterpret_cast<int*>(tmem_slot + 2);
  int* more = reinterpret_cast<int*>(tmem_slot + 3);  // passes behind the first
  TileJob* where = reinterpret_cast<TileJob*>(tmem_slot + 4);  // r < 0: none
  static_assert(8 * TB_COUNT + kTileInfo * sizeof(TileInfo) + 8 * 4 + 4 * 4 + sizeof(TileJob) <= 512, "MISC");
  volatile float* s_max = reinterpret_cast<volatile float*>(misc + 512);  // (tile, half, row)
  const uint32_t bar0 = smem_u32(bars);
#define TBAR(i) (bar0 + 8u * static_cast<uint32_t>(i))

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = a.heads_first ? blockIdx.x : blockIdx.y;
  auto init_barriers = [&](bool both) {
    for (int i = 0; i < TB_COUNT; ++i) {
      uint32_t n = 1;
      if (i == TB_Q) n = 16;                       // softmax warps
      if (i >= TB_KV_EMPTY && i < TB_KV_EMPTY + kTileStages) n = both ? 2 : 1;  // MMA warps
      if (i >= TB_P && i < TB_P + 4) n = (i - TB_P) & 1 ? 4u : 5u;  // warps of a half; low: the stage warp too
      if (i >= TB_X && i < TB_X + 8) n = 2;        // warps of 32 rows
      mbar_init(TBAR(i), n);
    }
    fence_mbarrier_init();
  };

  if (warp == 0) {
    TileJob job{};
    const bool found = find_tile<false>(a, a.heads_first ? blockIdx.y : blockIdx.x, lane, &job);
    if (lane == 0) {
      if (!found) job.r = -1;
      *where = job;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0)
      for (int i = lane; i < a.R; i += 32) check_request(a, i);
  } else if (warp == 1) {
    if (lane == 0) {
      *abort_flag = 0;
      *never = 0;
      *more = 0;
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
    }
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int r = where->r;
  launch_dependents();
  if (r < 0) {  // no such job: the same for the whole CTA
    if (warp == 2) tmem_dealloc(tmem, 512);
    wait_for_primary();
    return;
  }
  const Request q = load_request(a, r);
  const int row0 = where->tile * kTileRows, split = where->split, splits = where->splits;
  const int rows = min(kTileRows, q.n * a.G - row0);  // > 0
  const bool two = rows > 128;
  if (tid == 0) init_barriers(two);
  __syncthreads();
  // keys that the CTA's last row sees, and this split's share of them in 128-key steps
  const int last_tok = (row0 + rows - 1) / a.G;
  const int key_end = a.causal ? min(q.len, q.ctx + last_tok + 1) : q.len;
  const int steps = (key_end + 127) >> 7;
  const int key_lo = static_cast<int>(static_cast<int64_t>(steps) * split / splits) << 7;
  const int key_hi = min(key_end, static_cast<int>(static_cast<int64_t>(steps) * (split + 1) / splits) << 7);
  // a warp waits as one: what follows a wait is warp-wide
  auto wait_all = [&](uint32_t bar, uint32_t parity, int site) -> bool {
    return __all_sync(0xffffffffu, mbar_wait_poll(bar, parity, abort_flag, site));
  };
  // Softmax: two threads per row, one for each half of a chunk's 128 keys (two warpgroups per
  // tile, four softmax warps on each scheduler, so that one's arithmetic runs under another's
  // exponentials). A row's weights are relative to the largest logit of the first chunk, fixed
  // for good: nothing of a chunk waits for its maximum, and the output is never rescaled. That
  // is safe while no later logit is more than kExcess above it (base-2 units; the weights stay in
  // the type's range, and sums and outputs far inside fp32's). Each thread keeps the largest
  // logit that it saw; if some row went past the limit (fp16: 9.7 nats above its first 128 keys), the
  // whole CTA does its work once more, relative to the rows' largest logits of all, which cannot fail
  // below kExact (1560 rows of 40 heads over 15600 keys, fp16: 460 us, and 880 with such a row in
  // every CTA). A logit or reference of that size and more, of either sign, is rounded by a quarter of
  // a unit and more when it is scaled (past 2^28 by as much as the weights' range), and a difference
  // that large keeps little or nothing of a smaller logit. Such a CTA does two more passes, one for the
  // rows' largest logits before the scale, one that subtracts them before it scales.
  constexpr float kExcess = kF16 ? 14.f : 60.f;
  constexpr float kExact = 4194304.f;
  const int t = (warp >> 3) & 1, hb = (warp >> 2) & 1, rr = tid & 127;
  const int row = row0 + 128 * t + rr;
  const bool live = warp < 16 && 128 * t + rr < rows;
  const int tok = row / a.G, hq = h * a.G + row % a.G;
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t tO = tmem + 256 + 128 * t + (D / 2) * hb + lanes;  // this half's output columns
  // Rows of a warp move whole, UN lanes of 16 bytes to a row: with a lane per row every access
  // touched 32 lines, 4000 cycles of Q and 8000 of partial results for a CTA.
  constexpr int UN = D / 8;
  const int u = lane % UN;
  auto other_row = [&](const void* p, int r) {
    return reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(p), r));
  };
  float m_row = -INFINITY, l_run = 0.f;
  int nch = 0;
  bool ok_all = true;
  // The end of a pass, for every thread of the CTA: true when it was the last one (the first pass
  // says how many more there are).
  auto last_pass = [&](int pass) -> bool {
    tc_fence_before();
    named_bar_sync(1, kTileThreads);
    tc_fence_after();
    return pass == *reinterpret_cast<volatile int*>(more);
  };
  if (warp >= 16) {
    // registers go from the last warpgroup to the softmax warpgroups
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
#pragma unroll 1
    for (int pass = 0;; ++pass) {
      if (warp == 17) {
        // ------------------------------------------------ TMA warp: gathers chunks page by page
        // A load takes lu = min(page, 128) rows; chunk = 128 / lu loads of kept pages, in order.
        const int lu_shift = min(a.page_shift, 7), lu = 1 << lu_shift, per_chunk = 128 >> lu_shift;
        const int32_t* trow = a.table + r * a.table_stride;
        const uint8_t* mrow = a.mask ? a.mask + r * a.mr + h * a.mg : nullptr;
        const int end = (key_hi + lu - 1) >> lu_shift;
        // Lane i looks at load base + i of the request (its page, -1 where it is masked or behind the
        // end); the next 32 are looked up while these are used.
        auto look = [&](int base) -> int {
          const int i = base + lane;
          if (i >= end) return -1;
          const int pg = static_cast<int>((static_cast<int64_t>(i) << lu_shift) >> a.page_shift);
          const int id = trow[pg];
          if (mrow && !mrow[pg]) return -1;
          if (id < 0 || id >= a.n_pages) {
            report_device_error(kStatusBadLabel, kPagedSite + 1);
            return -1;
          }
          return id;
        };
        int base = key_lo >> lu_shift;
        int id = look(base), id_next = look(base + 32);
        unsigned left = __ballot_sync(0xffffffffu, id >= 0);
        uint32_t loads = 0;   // stages filled so far
        int tail_rows = 128;  // rows that hold keys in the last chunk (all in those before it)
        bool ok = true;
        for (int j = 0; ok; ++j) {
          // (the record is free: the stage of the last chunk's keys was last used by the values of
          // chunk j - 4, whose product waited for the softmax of that chunk)
          TileInfo* ti = info + j % kTileInfo;
          int filled = 0, last_i = -1;
          while (filled < per_chunk && base < end) {
            const int rank = filled + __popc(left & ((1u << lane) - 1u));
            const bool take = ((left >> lane) & 1u) && rank < per_chunk;
            if (take) {
              ids[rank] = id;
              for (int gk = 0; gk < lu / 16; ++gk) ti->pos[rank * (lu / 16) + gk] = ((base + lane) << lu_shift) + 16 * gk;
            }
            const unsigned taken = __ballot_sync(0xffffffffu, take);
            filled += __popc(taken);
            if (taken) last_i = base + 31 - __clz(taken);
            left &= ~taken;
            if (left == 0) {
              base += 32;
              id = id_next;
              id_next = look(base + 32);
              left = __ballot_sync(0xffffffffu, id >= 0);
            }
          }
          const int granules = filled * (lu / 16);
          if (lane < 8 && lane >= granules) ti->pos[lane] = kAbsent;
          // rows that hold keys: all of the loads but what lies behind the last key that a row of
          // the CTA sees
          int valid = filled * lu;
          if (filled) valid -= max(0, ((last_i + 1) << lu_shift) - key_end);
          if (lane == 0) {
            ti->rows = valid;
            ti->last = valid == 128 ? (last_i << lu_shift) + lu - 1 : kAbsent;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(TBAR(TB_INFO + j % kTileInfo));
          if (filled == 0) break;
          tail_rows = valid;
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t stage = loads % kTileStages;
            if (loads >= kTileStages) {
              ok = __all_sync(0xffffffffu, mbar_wait_poll(TBAR(TB_KV_EMPTY + stage), ((loads / kTileStages) - 1) & 1,
                                                     abort_flag, kPagedSite + 11));
              if (!ok) break;
            }
            if (lane == 0) mbar_arrive_expect_tx(TBAR(TB_KV_FULL + stage), filled * lu * D * 2);
            __syncwarp();
            if (lane < filled) {
              const int i_row = a.page_shift > 7 ? ti->pos[0] & ((1 << a.page_shift) - 1) : 0;
#pragma unroll
              for (int cc = 0; cc < Cfg::NATOM; ++cc)
                tma_load_4d(sKV + stage * Cfg::TILE + cc * 16384 + lane * lu * 128, kv ? &tmV : &tmK,
                            TBAR(TB_KV_FULL + stage), cc * 64, i_row, h, ids[lane]);
            }
            __syncwarp();
            ++loads;
          }
        }
        // value rows without a key in the last chunk: zeros (what lies there may be anything, and
        // 0 * NaN is NaN)
        if (ok && tail_rows < 128) {
          const uint32_t stage = (loads - 1) % kTileStages;
          ok = wait_all(TBAR(TB_KV_FULL + stage), ((loads - 1) / kTileStages) & 1, kPagedSite + 13);
          if (ok) {
            for (int i = tail_rows * 8 + lane; i < 128 * 8; i += 32)
#pragma unroll
              for (int cc = 0; cc < Cfg::NATOM; ++cc)
                *reinterpret_cast<uint4*>(smem + (2 + stage) * Cfg::TILE + cc * 16384 + i * 16) =
                    make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(TBAR(TB_TAIL));
          }
        }
        __syncwarp();
        if (lane == 0) ids[0] = static_cast<int>(loads);  // (no page is looked up any more)
        // every copy has landed before the CTA may end
        for (uint32_t i = loads > kTileStages ? loads - kTileStages : 0; i < loads; ++i)
          mbar_wait_poll(TBAR(TB_KV_FULL + i % kTileStages), (i / kTileStages) & 1, never, kPagedSite + 12);
      } else if (warp == 16 || (warp == 18 && two)) {
        // ------------------------------------------------ MMA warps, one per tile
        // The two halves of a chunk's keys are pipelines of their own: logits (and over them, their
        // weights) in TMEM columns 128 t + 64 half, the output of both in columns 256 + 128 t. A
        // half's next logits go where its weights were, QK(j + 1, half) right behind PV(j, half).
        // So four pipelines (two tiles, two halves) keep the tensor core and the exponentials busy
        // between them. A warp per tile, because a warp that has committed stands still until its
        // products are done; the whole warp runs on uniform values, so that descriptors live in
        // uniform registers (a lone thread took 75 cycles to issue a product that takes 64).
        const int t = warp == 18 ? 1 : 0;
        auto commit = [&](uint32_t bar) {
          if (elect_one()) tc_commit(bar);
          __syncwarp();
        };
        constexpr uint32_t kIdQK = make_idesc16(kF16, 128, 64, false, false);
        constexpr uint32_t kIdPV = make_idesc16(kF16, 128, D, false, true);
        const uint64_t dQ = smem_desc(sQ + t * Cfg::TILE, 16, 1024);
        const uint64_t dKV = smem_desc(sKV, 16, 1024);
        const uint64_t dV = smem_desc(sKV, 16384, 1024);
        const uint32_t tS = tmem + 128 * t, tO = tmem + 256 + 128 * t;
        auto issue_qk = [&](int half, uint32_t stage) {
          const uint64_t kd = dKV + static_cast<uint64_t>((stage * Cfg::TILE + half * 64 * 128) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = static_cast<uint64_t>(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
              mma_ss<false>(tS + 64 * half, dQ + off, kd + off, kIdQK, kk > 0 ? 1u : 0u);
            }
          }
          __syncwarp();
        };
        auto issue_pv = [&](int half, uint32_t stage, bool first) {
          const uint64_t vd = dV + static_cast<uint64_t>((stage * Cfg::TILE + half * 4 * 2048) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4)
              mma_ts<false>(tO, tS + 64 * half + k4 * 8, vd + static_cast<uint64_t>((k4 * 2048) >> 4), kIdPV,
                            (!first || k4 > 0) ? 1u : 0u);
          }
          __syncwarp();
        };
        uint32_t vst = 1, kst = 2;  // stages of V(j) and K(j + 1)
        bool ok = pass > 0 || wait_all(TBAR(TB_Q), 0, kPagedSite + 20);
        ok = ok && wait_all(TBAR(TB_INFO), 0, kPagedSite + 21);
        int rows_j = ok ? info[0].rows : 0;
        if (ok && rows_j > 0 && (ok = wait_all(TBAR(TB_KV_FULL), 0, kPagedSite + 22))) {
          tc_fence_after();
          issue_qk(0, 0);
          commit(TBAR(TB_S + 2 * t));
          if (rows_j > 64) {
            issue_qk(1, 0);
            commit(TBAR(TB_S + 2 * t + 1));
          }
          commit(TBAR(TB_KV_EMPTY));
        }
        for (int j = 0; ok && rows_j > 0; ++j) {
          // low half: its weights, V(j) and K(j + 1) are there
          if (!(ok = wait_all(TBAR(TB_P + 2 * t), j & 1, kPagedSite + 25))) break;
          tc_fence_after();
          issue_pv(0, vst, j == 0);
          const int next_rows = info[(j + 1) % kTileInfo].rows;
          if (next_rows > 0) {
            issue_qk(0, kst);
            commit(TBAR(TB_S + 2 * t));
          }
          if (rows_j <= 64) {  // (the last chunk)
            commit(TBAR(TB_KV_EMPTY + vst));
            break;
          }
          // high half
          if (!(ok = wait_all(TBAR(TB_P + 2 * t + 1), j & 1, kPagedSite + 28))) break;
          tc_fence_after();
          issue_pv(1, vst, false);
          if (next_rows > 64) {
            issue_qk(1, kst);
            commit(TBAR(TB_S + 2 * t + 1));
          }
          commit(TBAR(TB_KV_EMPTY + vst));
          if (next_rows > 0) commit(TBAR(TB_KV_EMPTY + kst));
          rows_j = next_rows;
          vst = vst + 2 >= kTileStages ? vst + 2 - kTileStages : vst + 2;
          kst = kst + 2 >= kTileStages ? kst + 2 - kTileStages : kst + 2;
        }
        // every product has completed before the CTA may end
        commit(TBAR(TB_DRAIN + t));
        mbar_wait_poll(TBAR(TB_DRAIN + t), 0, never, kPagedSite + 27);
      } else if (warp == 19) {
        // ------------------------------------------------ stage warp
        // A wait costs a warp 250 to 350 cycles here even when there is nothing to wait for, and the
        // MMA warps' instructions are what a chunk's time consists of; so this warp waits for
        // V(j), the next record and K(j + 1) in their place, and its arrival is one of those that
        // complete the low half's weights.
        uint32_t vst = 1, vph = 0, kst = 2, kph = 0;
        bool ok = wait_all(TBAR(TB_INFO), 0, kPagedSite + 36);
        int rows_j = ok ? info[0].rows : 0;
        for (int j = 0; ok && rows_j > 0; ++j) {
          if (!(ok = wait_all(TBAR(TB_KV_FULL + vst), vph, kPagedSite + 23))) break;
          if (rows_j < 128 && !(ok = wait_all(TBAR(TB_TAIL), 0, kPagedSite + 35))) break;
          if (!(ok = wait_all(TBAR(TB_INFO + (j + 1) % kTileInfo), ((j + 1) / kTileInfo) & 1, kPagedSite + 24))) break;
          rows_j = info[(j + 1) % kTileInfo].rows;
          if (rows_j > 0 && !(ok = wait_all(TBAR(TB_KV_FULL + kst), kph, kPagedSite + 26))) break;
          if (j > 0) {  // one arrival in each phase
            ok = wait_all(TBAR(TB_P), (j - 1) & 1, kPagedSite + 37);
            if (ok && two) ok = wait_all(TBAR(TB_P + 2), (j - 1) & 1, kPagedSite + 37);
            if (!ok) break;
          }
          if (lane == 0) {
            mbar_arrive(TBAR(TB_P));
            if (two) mbar_arrive(TBAR(TB_P + 2));
          }
          __syncwarp();
          vst += 2;
          if (vst >= kTileStages) { vst -= kTileStages; vph ^= 1u; }
          kst += 2;
          if (kst >= kTileStages) { kst -= kTileStages; kph ^= 1u; }
        }
      }
      if (last_pass(pass)) break;
      if (tid == 512) {
        // every stage's last release has arrived, before its barrier starts anew
        const int loads = ids[0];
        for (int s = 0; s < kTileStages && s < loads; ++s)
          mbar_wait_poll(TBAR(TB_KV_EMPTY + s), ((loads - s - 1) / kTileStages) & 1, abort_flag, kPagedSite + 14);
        for (int i = 0; i < TB_COUNT; ++i) mbar_inval(TBAR(i));
        init_barriers(two);
      }
      named_bar_sync(1, kTileThreads);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
#pragma unroll 1
    for (int pass = 0;; ++pass) {
      // ------------------------------------------------ softmax
      const uint32_t tS = tmem + 128 * t + 64 * hb + lanes;  // this half's logits and weights
      const uint32_t xbar = TBAR(TB_X + 4 * t + (warp & 3));
      volatile float* xmine = s_max + (t * 2 + hb) * 128 + rr;
      const volatile float* xother = s_max + (t * 2 + (hb ^ 1)) * 128 + rr;
      if (pass == 0) {
        // half of this warp's rows of Q into the swizzled tile (16-byte piece u of row r at u ^ (r & 7))
        const T* src = static_cast<const T*>(a.q) + hq * a.qh + static_cast<int64_t>(q.t0 + tok) * a.qt;
        uint4 v[UN / 2];
#pragma unroll
        for (int i = 0; i < UN / 2; ++i) {
          const int r = hb * 16 + i * (32 / UN) + lane / UN;
          const uint8_t* p = other_row(src, r) + 16 * u;
          v[i] = 128 * t + (warp & 3) * 32 + r < rows ? ldg_stream(p) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < UN / 2; ++i) {
          const int r = (warp & 3) * 32 + hb * 16 + i * (32 / UN) + lane / UN;
          *reinterpret_cast<uint4*>(smem + t * Cfg::TILE + (u >> 3) * 16384 + r * 128 + (((u & 7) ^ (r & 7)) << 4)) = v[i];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(TBAR(TB_Q));
      }
      const int lim = live ? (a.causal ? min(q.len - 1, q.ctx + tok) : q.len - 1) : -1;
      // the smallest reach of the tile's rows (its first row's): chunks up to it need no mask
      const int lim_tile = a.causal ? min(q.len - 1, q.ctx + (row0 + 128 * t) / a.G) : q.len - 1;
      float seen = -INFINITY;  // largest logit (times the scale, base 2)
      bool ok = t == 0 || two;
      const bool exact = pass > 0 && *reinterpret_cast<volatile int*>(more) == 2;
      l_run = 0.f;
      nch = 0;
#pragma unroll 1
      for (int j = 0; ok && !exact; ++j) {
        if (!(ok = wait_all(TBAR(TB_INFO + j % kTileInfo), (j / kTileInfo) & 1, kPagedSite + 30))) break;
        const TileInfo* ti = info + j % kTileInfo;
        if (ti->rows == 0) break;
        const bool edge = ti->last > lim_tile, has = ti->rows > 64 * hb;
        ++nch;
        float v[2][32];
        if (has) {
          if (!(ok = wait_all(TBAR(TB_S + 2 * t + hb), j & 1, kPagedSite + 31))) break;
          tc_fence_after();
          tmem_ld32(tS, v[0]);
          tmem_ld32(tS + 32, v[1]);
          tmem_wait_ld();
          if (edge) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int vis = lim - ti->pos[4 * hb + i];  // last visible column of the granule
#pragma unroll
              for (int c = 0; c < 16; ++c)
                if (c > vis) v[i >> 1][(i & 1) * 16 + c] = -INFINITY;
            }
          }
        }
        if (j == 0 && pass == 0) {  // the reference, of both halves
          *xmine = has ? max64(v[0], v[1]) * a.scale_log2 : -INFINITY;
          __syncwarp();
          if (lane == 0) mbar_arrive(xbar);
          if (!(ok = wait_all(xbar, 0, kPagedSite + 33))) break;
          m_row = fmaxf(*xmine, *xother);
        }
        if (!has) break;  // (the last chunk)
        const float neg = m_row == -INFINITY ? 0.f : -m_row;
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f, q0 = -INFINITY, q1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float x0, x1;
            fma2(x0, x1, v[i][2 * c], v[i][2 * c + 1], a.scale_log2, a.scale_log2, neg, neg);
            if (c & 1) q1 = max3(q1, x0, x1);
            else q0 = max3(q0, x0, x1);
            x0 = ex2(x0);
            x1 = ex2(x1);
            if (c & 1) add2(s2, s3, s2, s3, x0, x1);
            else add2(s0, s1, s0, s1, x0, x1);
            w[c] = pack_pair<T>(x0, x1);
          }
          tmem_st16(tS + 16 * i, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(TBAR(TB_P + 2 * t + hb));
        l_run += (s0 + s1) + (s2 + s3);
        seen = max3(seen, q0, q1);  // relative to the row's reference
      }
      if (exact && ok) {
        const ExactPass e{bar0, tS, info, abort_flag, t, hb, lim, lim_tile,
                          pass == 1 || m_row == -INFINITY ? 0.f : m_row, a.scale_log2};
        ok = exact_pass<T>(e, &seen, &l_run, &nch);
        if (pass == 2) m_row *= a.scale_log2;
      }
      ok_all = ok || !(t == 0 || two);
      if (pass == 0 && live) {
        // A row that the reference is too low for: its largest logit of all goes to both halves.
        // So it does where the first chunk gave no reference (all its logits -infinity).
        const bool low = seen > kExcess || (m_row == -INFINITY && seen > -INFINITY);
        const float size = fabsf(m_row == -INFINITY ? seen : m_row);
        const bool large = (size >= kExact && size < INFINITY) || seen >= kExact;
        if (low || large) atomicMax(more, large ? 2 : 1);
      }
      if (last_pass(pass)) break;
      // The words that held the halves' first maxima serve again only here: every thread of the CTA
      // has passed the barrier, so both halves have taken their references from them.
      *xmine = seen;
      named_bar_sync(2, 512);  // the softmax warps
      const float most = fmaxf(seen, *xother);
      if (exact) m_row = most;
      else m_row = m_row > -INFINITY ? m_row + fmaxf(most, 0.f) : most;
      named_bar_sync(1, kTileThreads);
    }
    // (every product and copy has ended) the sums of a row's halves, through the first stage
    volatile float* sums = reinterpret_cast<volatile float*>(smem + 2 * Cfg::TILE);
    sums[(t * 2 + hb) * 128 + rr] = l_run;
    named_bar_sync(2, 512);
    if (ok_all && (t == 0 || two)) {
      l_run = sums[t * 256 + rr] + sums[t * 256 + 128 + rr];
      // Out through the tile's Q, which no product reads any more: each lane's half row in pieces of
      // 16 bytes (piece x of row r at x ^ r), then row by row. A warp has 32 rows of D bytes.
      constexpr int UH = D / 16;  // pieces of a row
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
      uint8_t* stage = smem + t * Cfg::TILE + (warp & 7) * (Cfg::TILE / 8);
      const int uh = lane % UH;
      auto put = [&](int piece, const uint4& x) {
        *reinterpret_cast<uint4*>(stage + lane * D + ((piece ^ (lane & (UH - 1))) << 4)) = x;
      };
      auto drain = [&](void* row_ptr) {
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < UH; ++i) {
          const int r = i * (32 / UH) + lane / UH;
          uint8_t* p = other_row(row_ptr, r);
          const uint4 x = *reinterpret_cast<const uint4*>(stage + r * D + ((uh ^ (r & (UH - 1))) << 4));
          if (128 * t + (warp & 3) * 32 + r < rows) *reinterpret_cast<uint4*>(p + 16 * uh) = x;
        }
        __syncwarp();
      };
      auto take = [&](int col, float(&o)[16]) {
        if (nch > 0) {
          tmem_ld16(tO + col, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int c = 0; c < 16; ++c) o[c] = 0.f;
        }
      };
      if (splits > 1) {  // unnormalised fp32, D bytes of a row at a time
        const size_t prow = tile_part_row(a, where->slot + split, h, 128 * t + rr);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int p = 0; p < D / 64; ++p) {
            float o[16];
            take(half * (D / 4) + p * 16, o);
#pragma unroll
            for (int c = 0; c < 4; ++c) put(4 * p + c, *reinterpret_cast<uint4*>(o + 4 * c));
          }
          drain(a.part + prow * D + hb * (D / 2) + half * (D / 4));
        }
        if (live && hb == 0) *reinterpret_cast<float2*>(tile_part_ml(a, D) + prow * 2) = make_float2(m_row, l_run);
      } else {
#pragma unroll
        for (int p = 0; p < D / 32; ++p) {
          float o[16];
          take(p * 16, o);
          uint32_t w[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) w[c] = l_run == 0.f ? 0u : pack_pair<T>(o[2 * c] * inv, o[2 * c + 1] * inv);
          put(2 * p, make_uint4(w[0], w[1], w[2], w[3]));
          put(2 * p + 1, make_uint4(w[4], w[5], w[6], w[7]));
        }
        drain(static_cast<T*>(a.out) + hq * a.oh + static_cast<int64_t>(q.t0 + tok) * a.ot + hb * (D / 2));
      }
    }
  }
#undef TBAR
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // what follows on the stream waits for this kernel alone: it ends after the one before it
  wait_for_primary();
}

// Joins the parts of the pairs that are split: grid (pairs * heads, row groups), four rows (of
// 128 values; eight of 64) per warp at a time, four parts of each on their way at once.
constexpr int kJoinThreads = 256;
template <int D>
constexpr int tile_join_rows() { return kJoinThreads / 32 * 4 * (128 / D); }  // rows of a CTA
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) tile_combine_kernel(const PagedArgs a) {
  constexpr int L = D / 4;  // lanes of a row
  constexpr int kRows = 4;  // rows of a lane group
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x % a.Hkv, l = lane % L;
  TileJob job{};
  const bool found = find_tile<true>(a, blockIdx.x / a.Hkv, lane, &job);
  wait_for_primary();  // before any return: a dependent that has ended stands for its primary
  if (!found) return;
  const Request q = load_request(a, job.r);
  const int rows = min(kTileRows, q.n * a.G - job.tile * kTileRows);
  const float* ml = tile_part_ml(a, D);
  const int rr0 = (blockIdx.y * (kJoinThreads / 32) + warp) * kRows * (32 / L) + lane / L;
  float m[kRows], sum[kRows];
  float4 acc[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    m[i] = -INFINITY;
    sum[i] = 0.f;
    acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll 4
  for (int s = 0; s < job.splits; ++s) {
    float2 x[kRows];
    float4 o[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int rr = rr0 + i * (32 / L);
      x[i] = make_float2(-INFINITY, 0.f);
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (rr < rows) {
        const size_t prow = tile_part_row(a, job.slot + s, h, rr);
        x[i] = *reinterpret_cast<const float2*>(ml + 2 * prow);
        o[i] = *reinterpret_cast<const float4*>(a.part + prow * D + 4 * l);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (x[i].x == -INFINITY && x[i].y == 0.f) continue;  // a part that saw no key of this row
      const float mn = fmaxf(m[i], x[i].x), f0 = ex2(m[i] - mn), f1 = ex2(x[i].x - mn);
      sum[i] = sum[i] * f0 + x[i].y * f1;
      acc[i].x = acc[i].x * f0 + o[i].x * f1;
      acc[i].y = acc[i].y * f0 + o[i].y * f1;
      acc[i].z = acc[i].z * f0 + o[i].z * f1;
      acc[i].w = acc[i].w * f0 + o[i].w * f1;
      m[i] = mn;
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int rr = rr0 + i * (32 / L);
    if (rr >= rows) continue;
    const float inv = sum[i] == 0.f ? 0.f : 1.f / sum[i];
    const int row = job.tile * kTileRows + rr;
    T* po = static_cast<T*>(a.out) + (static_cast<int64_t>(h) * a.G + row % a.G) * a.oh +
            static_cast<int64_t>(q.t0 + row / a.G) * a.ot;
    *reinterpret_cast<uint2*>(po + 4 * l) =
        make_uint2(pack_pair<T>(acc[i].x * inv, acc[i].y * inv), pack_pair<T>(acc[i].z * inv, acc[i].w * inv));
  }
}

// A block table without columns: no key is left for any token, so their rows get 0 (grid: tokens),
// and every request that has tokens is recorded, as one that passes its table.
constexpr int kNoKeysThreads = 128;
__global__ void __launch_bounds__(kNoKeysThreads) paged_no_keys_kernel(const PagedArgs a, int D) {
  if (blockIdx.x == 0)
    for (int r = threadIdx.x; r < a.R; r += kNoKeysThreads) check_request(a, r);
  const int t = blockIdx.x, pieces = D / 8;  // of 16 bytes
  if (t < a.cu[0] || t >= a.cu[a.R]) return;
  for (int e = threadIdx.x; e < a.Hkv * a.G * pieces; e += kNoKeysThreads)
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + static_cast<int64_t>(e / pieces) * a.oh +
                              static_cast<int64_t>(t) * a.ot + 8 * (e % pieces)) = make_uint4(0, 0, 0, 0);
}

// ================================================================ host side
struct PagedPlan {
  bool token, tile;  // which kernels run
  int min_rows;      // rows up to which a request is the token kernel's
  int workers, one_each;
  int tile_ctas, can_split, join_pairs, heads_first;
  size_t bytes;
  size_t tile_off;
};

constexpr int kTokCtas = 148 * 6;

// With heads first the longest jobs of all heads start first and the CTAs without a job are the
// grid's last; with a head after the other, the CTAs at work share a head's keys. The first is
// faster while all the keys and values fit L2: 7 chunks of up to 600 rows x 16 heads of 64 with two
// pages of five kept, over up to 12000 keys (92 MB): 92 us and 100; 16000 keys (120 MB): 100 and 96;
// 1560 rows of 40 heads over 32760 keys: 1047 and 980.
constexpr int64_t kHeadsFirstBytes = int64_t(96) << 20;

PagedPlan paged_plan(int R, int T, int Hq, int Hkv, int D, int max_new, int width, int page) {
  PagedPlan p{};
  const int G = Hq / Hkv;
  const int64_t most = static_cast<int64_t>(std::min(max_new, T)) * G;
  p.token = most <= kTokenRows || R > 1;
  p.tile = most > kTokenRows;
  p.min_rows = p.token ? kTokenRows : 0;
  const int64_t keys = static_cast<int64_t>(width) * page;
  p.one_each = keys <= kTokChunk;  // nothing to share out
  p.workers = p.one_each ? R * Hkv : kTokCtas;
  size_t b = 0;
  if (p.token && !p.one_each)
    b = align_up(static_cast<size_t>(p.workers) * 2 * kTokenRows * (D + 2) * sizeof(float), 256);
  p.tile_off = b;
  if (p.tile) {
    // a request's pairs: at most its rows / 256, rounded up; splitting adds at most the work over
    // the quantum, which is at least the work over kTileJobs
    const int64_t pairs = static_cast<int64_t>(T) * G / kTileRows + std::min(R, T);
    p.can_split = keys > kTileMinChunks * 128;
    p.tile_ctas = static_cast<int>(pairs + (p.can_split ? ceil_div(kTileJobs, Hkv) : 0));
    p.heads_first = keys * R * Hkv * D * 4 <= kHeadsFirstBytes && p.tile_ctas < 65536;  // (grid.y)
    p.join_pairs = static_cast<int>(std::min<int64_t>(pairs, ceil_div(kTileJobs, Hkv)));
    if (p.can_split) b += align_up(static_cast<size_t>(kTileSlots) * kTileRows * (D + 2) * sizeof(float), 256);
  }
  p.bytes = std::max<size_t>(b, 256);
  return p;
}

int check_paged_sizes(const bsa_paged_cache& c, int R, int T, int Hq, int max_new, int width) {
  const int st = check_paged_cache(c);
  if (st != BSA_OK) return st;
  if (R < 0 || T < 0 || Hq <= 0 || max_new < 0 || width < 0) return fail(BSA_ERR_INVALID_ARG, "bad size");
  if (Hq % c.Hkv) return fail(BSA_ERR_INVALID_ARG, "Hq (%d) not a multiple of Hkv (%d)", Hq, c.Hkv);
  if (R > kPagedMaxR) return fail(BSA_ERR_UNSUPPORTED, "%d requests, at most %d", R, kPagedMaxR);
  if (c.Hkv > 4096 || Hq > 16384) return fail(BSA_ERR_UNSUPPORTED, "too many heads");
  if (static_cast<int64_t>(T) * Hq > INT32_MAX / 2) return fail(BSA_ERR_UNSUPPORTED, "T*Hq exceeds 2^30");
  if (static_cast<int64_t>(width) * c.page > (1 << 28))
    return fail(BSA_ERR_UNSUPPORTED, "a request of more than 2^28 keys");
  if (static_cast<int64_t>(width) * c.page * R > (int64_t(1) << 36))
    return fail(BSA_ERR_UNSUPPORTED, "block table of more than 2^36 keys");
  return BSA_OK;
}

template <typename T, int D>
int launch_paged(PagedArgs a, const PagedPlan& p, const bsa_paged_cache& c, char* ws, cudaStream_t st) {
  if (p.token) {
    PagedArgs t = a;
    t.part = reinterpret_cast<float*>(ws);
    t.workers = p.workers;
    t.one_each = p.one_each;
    const int smem = p.one_each ? 0 : (a.R + 1) * static_cast<int>(sizeof(int32_t));
    const int64_t most = static_cast<int64_t>(std::min(a.max_new, a.T)) * a.G;
    t.tok_rows = most <= 8 ? 8 : kTokenRows;
    auto kern = most <= 8 ? paged_token_kernel<T, D, 1> : paged_token_kernel<T, D, 2>;
    // At most 16.4 KB beside 17.2 KB of static shared memory: no opt-in (which is the function's, not
    // the call's: one of this call's size would lower the limit under a call of another thread).
    constexpr int kStatic = kTokWarps * 16 * (D + 6) * 4 + 4 * kTokWarps;
    static_assert((kPagedMaxR + 1) * 4 + kStatic <= 48 * 1024, "shared memory of the token kernel");
    kern<<<p.workers, kTokThreads, smem, st>>>(t);
    count_launch();
    int e = check_cuda(cudaGetLastError(), "paged_token_kernel");
    if (e != BSA_OK) return e;
    if (!p.one_each) {
      e = check_cuda(launch_dependent(token_combine_kernel<T, D>,
                                      dim3(a.R * a.Hkv, static_cast<unsigned>(std::min<int64_t>(most, kTokenRows))),
                                      dim3(32 * kCombWarps), 0, st, t), "token_combine_kernel");
      if (e != BSA_OK) return e;
      count_launch();
    }
  }
  if (p.tile) {
    PagedArgs t = a;
    t.part = reinterpret_cast<float*>(ws + p.tile_off);
    t.min_rows = p.min_rows;
    t.tile_ctas = p.tile_ctas;
    t.can_split = p.can_split;
    t.heads_first = p.heads_first;
    CUtensorMap mk, mv;
    const CUtensorMapDataType dt = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(c.page),
                              static_cast<uint64_t>(c.Hkv), static_cast<uint64_t>(c.n_pages)};
    const uint32_t box[4] = {64, static_cast<uint32_t>(std::min(c.page, 128)), 1, 1};
    const uint64_t ks[3] = {static_cast<uint64_t>(c.k_row_stride) * 2, static_cast<uint64_t>(c.k_head_stride) * 2,
                            static_cast<uint64_t>(c.k_page_stride) * 2};
    const uint64_t vs[3] = {static_cast<uint64_t>(c.v_row_stride) * 2, static_cast<uint64_t>(c.v_head_stride) * 2,
                            static_cast<uint64_t>(c.v_page_stride) * 2};
    int e = make_tmap_4d(&mk, c.k, dt, 2, dims, ks, box);
    if (e == BSA_OK) e = make_tmap_4d(&mv, c.v, dt, 2, dims, vs, box);
    if (e != BSA_OK) return e;
    auto kern = paged_tile_kernel<T, D>;
    e = check_cuda(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        TileCfg<D>::SMEM_LAUNCH), "cudaFuncSetAttribute(paged_tile_kernel)");
    if (e != BSA_OK) return e;
    const dim3 grid(p.heads_first ? a.Hkv : p.tile_ctas, p.heads_first ? p.tile_ctas : a.Hkv);
    // After the token kernel's join it starts at once: it shares neither rows nor workspace with it.
    if (p.token) {
      e = check_cuda(launch_dependent(kern, grid, dim3(kTileThreads), TileCfg<D>::SMEM_LAUNCH, st, mk, mv, t),
                     "paged_tile_kernel");
    } else {
      kern<<<grid, kTileThreads, TileCfg<D>::SMEM_LAUNCH, st>>>(mk, mv, t);
      e = check_cuda(cudaGetLastError(), "paged_tile_kernel");
    }
    if (e != BSA_OK) return e;
    count_launch();
    if (p.can_split) {
      e = check_cuda(launch_dependent(tile_combine_kernel<T, D>,
                                      dim3(p.join_pairs * a.Hkv, kTileRows / tile_join_rows<D>()),
                                      dim3(kJoinThreads), 0, st, t), "tile_combine_kernel");
      if (e != BSA_OK) return e;
      count_launch();
    }
  }
  return BSA_OK;
}

}  // namespace
}  // namespace bsa

extern "C" {

size_t bsa_paged_attention_workspace_bytes(bsa_paged_cache cache, int R, int T, int Hq, int max_new,
                                           int width) {
  if (bsa::check_paged_sizes(cache, R, T, Hq, max_new, width) != BSA_OK) return 0;
  return bsa::paged_plan(R, T, Hq, cache.Hkv, cache.D, max_new, width, cache.page).bytes;
}

int bsa_paged_chunk_attention(bsa_heads q, bsa_paged_cache cache, const int32_t* block_table,
                              int width, int64_t table_stride, const int32_t* cu_new,
                              const int32_t* context_lens, int R, int T, int Hq, int max_new,
                              const uint8_t* page_mask, int64_t mask_r_stride,
                              int64_t mask_g_stride, float scale, int causal, bsa_heads out,
                              void* workspace, size_t workspace_bytes, void* stream) {
  using namespace bsa;
  int st = check_paged_sizes(cache, R, T, Hq, max_new, width);
  if (st != BSA_OK) return st;
  if (R == 0 || T == 0 || max_new == 0) return BSA_OK;
  if ((width > 0 && !block_table) || !cu_new || !context_lens || !q.ptr || !out.ptr)
    return fail(BSA_ERR_INVALID_ARG, "null pointer");
  if (reinterpret_cast<uintptr_t>(q.ptr) % 16 || reinterpret_cast<uintptr_t>(out.ptr) % 16 ||
      q.stride_h % 8 || q.stride_s % 8 || out.stride_h % 8 || out.stride_s % 8)
    return fail(BSA_ERR_INVALID_ARG, "q or out: pointer or strides not multiples of 16 bytes");
  if (table_stride < 0 || mask_r_stride < 0 || mask_g_stride < 0)
    return fail(BSA_ERR_INVALID_ARG, "negative stride");
  const PagedPlan p = paged_plan(R, T, Hq, cache.Hkv, cache.D, max_new, width, cache.page);
  if (!workspace || workspace_bytes < p.bytes)
    return fail(BSA_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, p.bytes);
  if (reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(BSA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  PagedArgs a{};
  a.q = q.ptr;
  a.qh = q.stride_h;
  a.qt = q.stride_s;
  a.kc = cache.k;
  a.vc = cache.v;
  a.kp = cache.k_page_stride;
  a.kh = cache.k_head_stride;
  a.kr = cache.k_row_stride;
  a.vp = cache.v_page_stride;
  a.vh = cache.v_head_stride;
  a.vr = cache.v_row_stride;
  a.n_pages = cache.n_pages;
  a.page_shift = __builtin_ctz(cache.page);
  a.Hkv = cache.Hkv;
  a.G = Hq / cache.Hkv;
  a.T = T;
  a.R = R;
  a.table = block_table;
  a.width = width;
  a.table_stride = table_stride;
  a.cu = cu_new;
  a.ctx = context_lens;
  a.mask = page_mask;
  a.mr = mask_r_stride;
  a.mg = mask_g_stride;
  a.scale_log2 = (scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(cache.D))) * 1.4426950408889634f;
  a.causal = causal ? 1 : 0;
  a.out = out.ptr;
  a.oh = out.stride_h;
  a.ot = out.stride_s;
  a.max_new = max_new;
  char* ws = static_cast<char*>(workspace);
  cudaStream_t cs = as_stream(stream);
  if (width == 0) {
    paged_no_keys_kernel<<<T, kNoKeysThreads, 0, cs>>>(a, cache.D);
    count_launch();
    return check_cuda(cudaGetLastError(), "paged_no_keys_kernel");
  }
  if (cache.dtype == BSA_F16)
    return cache.D == 64 ? launch_paged<__half, 64>(a, p, cache, ws, cs)
                         : launch_paged<__half, 128>(a, p, cache, ws, cs);
  return cache.D == 64 ? launch_paged<__nv_bfloat16, 64>(a, p, cache, ws, cs)
                       : launch_paged<__nv_bfloat16, 128>(a, p, cache, ws, cs);
}

}  // extern "C"
