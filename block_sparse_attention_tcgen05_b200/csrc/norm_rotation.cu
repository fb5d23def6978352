// Per-head RMS norms of queries and keys with the position rotation in the same pass, its
// backward pass, and the same pass with the keys and values scattered into a paged cache.
//
// A row of D values is held by D/8 lanes, eight values each, so a warp holds 2 (D = 128) or
// 4 (D = 64) rows and the sum of squares is a butterfly over 16 or 8 lanes. The lane's eight
// values are the four pairs 4l .. 4l+3 of the rotation in both conventions: eight neighbours
// (pairs of neighbours), or four values of each half (pairs half a row apart), so no value
// moves between lanes and each lane reads four cosines and four sines. A lane group keeps
// its token and walks over heads, kUnroll rows at a time: the cosines, sines and both
// weights are read once per token and group.
//
// Everything is fp32 between the load and the one rounding of the store. The pass is bound
// by HBM: each input row is read once, each output row written once. 32760 tokens of 40 + 40
// heads of 128 in bf16, out of a fused projection: 225 us, 92 % of the copy rate (loading rows
// only when they are used, every head's pointer worked out anew: 326 us). The backward pass reads
// a row more: 146 us for 32768 tokens of 24 + 8 heads in single calls, 86 %; 156 in calls without
// a pause.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "ptx_paged.cuh"

namespace bsa {

namespace {

constexpr int kNormThreads = 256;

template <typename T>
struct Vec8;  // eight values of a lane: 16 bytes of a 16-bit type, 32 of fp32

__device__ __forceinline__ uint4 ld16(const void* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ uint2 ld8(const void* p) { return *reinterpret_cast<const uint2*>(p); }

template <typename T>
__device__ __forceinline__ void unpack2(uint32_t u, float& a, float& b) {
  if constexpr (sizeof(T) == 2) {
    if constexpr (std::is_same<T, __half>::value) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
      a = f.x;
      b = f.y;
    } else {
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
      a = f.x;
      b = f.y;
    }
  }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  } else {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
}

// The raw bits of a lane's eight values (kept unconverted while several rows are in flight).
template <typename T>
struct Raw {
  uint32_t w[2 * sizeof(T)];
};

// Lane l of a row: values 8l .. 8l+7 (interleaved pairs) or 4l .. 4l+3 and D/2 + 4l ..
template <typename T, int D, bool INTER>
__device__ __forceinline__ Raw<T> load_row(const T* row, int l) {
  Raw<T> r;
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
      const uint4 u = ld16(row + 8 * l + 4 * i);
      r.w[4 * i] = u.x;
      r.w[4 * i + 1] = u.y;
      r.w[4 * i + 2] = u.z;
      r.w[4 * i + 3] = u.w;
    }
  } else if constexpr (sizeof(T) == 2) {
    const uint2 a = ld8(row + 4 * l), b = ld8(row + D / 2 + 4 * l);
    r.w[0] = a.x;
    r.w[1] = a.y;
    r.w[2] = b.x;
    r.w[3] = b.y;
  } else {
    const uint4 a = ld16(row + 4 * l), b = ld16(row + D / 2 + 4 * l);
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
  }
  return r;
}

// Raw bits to pairs: a[i], b[i] are the two members of pair 4l + i.
template <typename T, bool INTER>
__device__ __forceinline__ void to_pairs(const Raw<T>& r, float (&a)[4], float (&b)[4]) {
  float f[8];
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2<T>(r.w[i], f[2 * i], f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r.w[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = INTER ? f[2 * i] : f[i];
    b[i] = INTER ? f[2 * i + 1] : f[4 + i];
  }
}

template <typename T, int D, bool INTER>
__device__ __forceinline__ void store_row(T* row, int l, const float (&a)[4], const float (&b)[4]) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[INTER ? 2 * i : i] = a[i];
    f[INTER ? 2 * i + 1 : 4 + i] = b[i];
  }
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
    if constexpr (INTER) {
      *reinterpret_cast<uint4*>(row + 8 * l) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<uint2*>(row + 4 * l) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(row + D / 2 + 4 * l) = make_uint2(w[2], w[3]);
    }
  } else {
    T* p = INTER ? row + 8 * l : row + 4 * l;
    T* q = INTER ? row + 8 * l + 4 : row + D / 2 + 4 * l;
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(q) = make_float4(f[4], f[5], f[6], f[7]);
  }
}

template <typename T, int D, bool INTER>
__device__ __forceinline__ void load_weight(const void* w, int f32, int l, float (&a)[4],
                                            float (&b)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int da = INTER ? 8 * l + 2 * i : 4 * l + i;
    const int db = INTER ? da + 1 : D / 2 + 4 * l + i;
    if (f32) {
      a[i] = static_cast<const float*>(w)[da];
      b[i] = static_cast<const float*>(w)[db];
    } else {
      a[i] = static_cast<float>(static_cast<const T*>(w)[da]);
      b[i] = static_cast<float>(static_cast<const T*>(w)[db]);
    }
  }
}

// Sum over the D/8 lanes of a row (every lane gets it).
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

struct HeadsIn {
  const void* p;
  int64_t sb, sh, ss;
};
struct HeadsOut {
  void* p;
  int64_t sb, sh, ss;
};

// The heads of a call are cut into runs, each inside one section (queries, keys, and the
// values of the paged form); grid (token groups, runs).
struct NormArgs {
  HeadsIn x[3];
  HeadsOut y[3];      // of a paged section: sb = page stride, sh = head stride, ss = row stride
  int heads[3];       // 0 values without a cache
  int first_run[3];   // first run of the keys and of the values in [1], [2]
  int per_run;
  int B, S;
  const void* w[2];
  int w_f32;
  const float *cos, *sin;
  int n_pos;
  const int32_t* positions;
  int64_t pos_b;
  float eps;
  const int32_t* slots;  // paged form: destination of the keys and values
  int page_shift, n_slots;
};

// -1 = skip silently, -2 = skip and report
__device__ __forceinline__ int checked_position(const int32_t* positions, int64_t pos_b, int b,
                                                int s, int n_pos) {
  const int p = positions ? positions[b * pos_b + s] : s;
  if (p >= 0 && p < n_pos) return p;
  return p == -1 ? -1 : -2;
}

constexpr int kNormSite = 120;

template <int D>
__device__ __forceinline__ void load_angles(const float* cos, const float* sin, int pos, int l,
                                            float (&c)[4], float (&s)[4]) {
  const float4 c4 = *reinterpret_cast<const float4*>(cos + static_cast<int64_t>(pos) * (D / 2) + 4 * l);
  const float4 s4 = *reinterpret_cast<const float4*>(sin + static_cast<int64_t>(pos) * (D / 2) + 4 * l);
  c[0] = c4.x; c[1] = c4.y; c[2] = c4.z; c[3] = c4.w;
  s[0] = s4.x; s[1] = s4.y; s[2] = s4.z; s[3] = s4.w;
}

template <typename T, int D, bool INTER, bool PAGED>
__global__ void __launch_bounds__(kNormThreads) norm_rotation_kernel(const NormArgs a) {
  constexpr int L = D / 8;
  constexpr int kUnroll = sizeof(T) == 2 ? 4 : 2;
  const int l = threadIdx.x % L;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * (kNormThreads / L) + threadIdx.x / L;
  const int64_t ntok = static_cast<int64_t>(a.B) * a.S;
  const bool in = tok < ntok;
  const int b = in ? static_cast<int>(tok / a.S) : 0, s = in ? static_cast<int>(tok % a.S) : 0;
  const int run = blockIdx.y;
  const int sec = PAGED && run >= a.first_run[2] ? 2 : (run >= a.first_run[1] ? 1 : 0);
  const int h_begin = (run - (sec ? a.first_run[sec] : 0)) * a.per_run;
  const int h_end = min(a.heads[sec], h_begin + a.per_run);
  const T* src = static_cast<const T*>(a.x[sec].p) + b * a.x[sec].sb + s * a.x[sec].ss;
  const int64_t xsh = a.x[sec].sh, ysh = a.y[sec].sh;

  Raw<T> cur[kUnroll], nxt[kUnroll];
  // rows of a token behind the last one, or of a head behind the run's, are not read
  auto load = [&](Raw<T>(&r)[kUnroll], int h0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (in && h0 + u < h_end) r[u] = load_row<T, D, INTER>(src + (h0 + u) * xsh, l);
      else r[u] = Raw<T>{};
    }
  };
  load(cur, h_begin);

  int pos = in ? checked_position(a.positions, a.pos_b, b, s, a.n_pos) : -1;
  if (pos == -2 && l == 0) report_device_error(kStatusBadLabel, kNormSite);
  bool put = pos >= 0;
  if (pos < 0) pos = 0;
  T* dst = static_cast<T*>(a.y[sec].p);
  if (PAGED && sec > 0) {
    const int slot = put ? a.slots[s] : -1;
    const bool fits = slot >= 0 && slot < a.n_slots;
    if (put && !fits && slot != -1 && l == 0) report_device_error(kStatusBadLabel, kNormSite + 1);
    put = put && fits;
    if (put)
      dst += static_cast<int64_t>(slot >> a.page_shift) * a.y[sec].sb +
             static_cast<int64_t>(slot & ((1 << a.page_shift) - 1)) * a.y[sec].ss;
  } else {
    dst += b * a.y[sec].sb + s * a.y[sec].ss;
  }
  if (PAGED && sec == 2) {  // values are copied (the conversion there and back is exact)
#pragma unroll 1
    for (int h0 = h_begin; h0 < h_end; h0 += kUnroll) {
      load(nxt, h0 + kUnroll);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float x[4], y[4];
        to_pairs<T, INTER>(cur[u], x, y);
        if (put && h0 + u < h_end) store_row<T, D, INTER>(dst + (h0 + u) * ysh, l, x, y);
        cur[u] = nxt[u];
      }
    }
    return;
  }
  float c[4] = {}, sn[4] = {}, wa[4], wb[4];
  if (put) load_angles<D>(a.cos, a.sin, pos, l, c, sn);
  load_weight<T, D, INTER>(a.w[sec], a.w_f32, l, wa, wb);
#pragma unroll 1
  for (int h0 = h_begin; h0 < h_end; h0 += kUnroll) {
    load(nxt, h0 + kUnroll);  // on their way while these rows are worked on
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float x[4], y[4];
      to_pairs<T, INTER>(cur[u], x, y);
      cur[u] = nxt[u];
      float p0 = 0.f, p1 = 0.f;
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        fma2(p0, p1, x[i], x[i + 1], x[i], x[i + 1], p0, p1);
        fma2(p0, p1, y[i], y[i + 1], y[i], y[i + 1], p0, p1);
      }
      const float r = rsqrtf(row_sum<D>(p0 + p1) * (1.f / D) + a.eps);
      float o0[4], o1[4];
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        float ya0, ya1, yb0, yb1, u0, u1;
        mul2(u0, u1, wa[i], wa[i + 1], r, r);
        mul2(ya0, ya1, x[i], x[i + 1], u0, u1);
        mul2(u0, u1, wb[i], wb[i + 1], r, r);
        mul2(yb0, yb1, y[i], y[i + 1], u0, u1);
        mul2(u0, u1, yb0, yb1, -sn[i], -sn[i + 1]);
        fma2(o0[i], o0[i + 1], ya0, ya1, c[i], c[i + 1], u0, u1);
        mul2(u0, u1, yb0, yb1, c[i], c[i + 1]);
        fma2(o1[i], o1[i + 1], ya0, ya1, sn[i], sn[i + 1], u0, u1);
      }
      if (put && h0 + u < h_end) store_row<T, D, INTER>(dst + (h0 + u) * ysh, l, o0, o1);
    }
  }
}

struct NormBackArgs {
  HeadsIn x[2], dy[2];  // queries, keys
  HeadsOut dx[2];
  int heads[2];
  int ctas[2];      // CTAs of each side: queries first in the grid
  int per_run;      // heads that one lane group walks over
  int B, S;
  const void* w[2];
  int w_f32;
  const float *cos, *sin;
  int n_pos;
  const int32_t* positions;
  int64_t pos_b;
  float eps;
  float* part;  // (CTAs, D) weight-gradient sums
};

// Asynchronous copy of a lane's eight values to its own shared-memory slot (zeros when !ok).
template <typename T, int D, bool INTER>
__device__ __forceinline__ void async_row(uint32_t dst, const T* row, int l, bool ok) {
  if constexpr (!INTER && sizeof(T) == 2) {
    const int n = ok ? 8 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(row + 4 * l), "r"(n) : "memory");
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst + 8), "l"(row + D / 2 + 4 * l), "r"(n)
                 : "memory");
  } else {
    const int n = ok ? 16 : 0;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * kNormThreads * 16),
                   "l"(INTER ? row + 8 * l + 4 * i : row + (i ? D / 2 : 0) + 4 * l), "r"(n)
                   : "memory");
  }
}

template <typename T>
__device__ __forceinline__ Raw<T> read_slot(const uint8_t* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
    const uint4 u = ld16(p + i * kNormThreads * 16);
    r.w[4 * i] = u.x;
    r.w[4 * i + 1] = u.y;
    r.w[4 * i + 2] = u.z;
    r.w[4 * i + 3] = u.w;
  }
  return r;
}

// Rows of a step and steps on their way: 64 KB in flight for a CTA, two CTAs per SM. Measured on
// 32768 tokens of 24 + 8 heads of 128 in bf16 (floor 125 us), the weight sums included: two
// steps of four rows 144 us; four of two 146; three of two with three CTAs per SM, whose 80
// registers leave less room between loads and use, 153.
template <typename T>
constexpr int norm_back_unroll() { return sizeof(T) == 2 ? 4 : 2; }
constexpr int kBackAhead = 2;

template <typename T>
constexpr int norm_back_smem() {
  return kBackAhead * norm_back_unroll<T>() * 2 * 8 * static_cast<int>(sizeof(T)) * kNormThreads;
}

// A CTA belongs to one side and takes that side's units (token group, run of heads) in a fixed
// stride, so its share of the weight sums, and the order inside it, depend on the sizes alone.
// The rows of kBackAhead steps are on their way to shared memory, across units, while one step
// is worked on: each lane copies what it will read itself, so nothing synchronises, and the
// bytes in flight cost no registers (holding one step ahead in registers ran at 71 % of the
// HBM rate, with two CTAs of 120 registers per SM).
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kNormThreads, 2) norm_rotation_back_kernel(const NormBackArgs a) {
  constexpr int L = D / 8, kGroups = kNormThreads / L;
  constexpr int kUnroll = norm_back_unroll<T>(), kRow = 8 * sizeof(T) * kNormThreads, kStep = 2 * kUnroll * kRow;
  extern __shared__ __align__(16) uint8_t ring[];
  const int l = threadIdx.x % L, grp = threadIdx.x / L;
  const int side = blockIdx.x >= a.ctas[0] ? 1 : 0;
  const int ntok = a.B * a.S;
  const int tgroups = ntok / kGroups + (ntok % kGroups ? 1 : 0);
  const int heads = a.heads[side];
  const int units = tgroups * ((heads + a.per_run - 1) / a.per_run);
  const int u0 = blockIdx.x - (side ? a.ctas[0] : 0);
  const uint32_t slot0 = smem_u32(ring) + threadIdx.x * 16;
  float dwa[4] = {}, dwb[4] = {}, wa[4], wb[4];
  load_weight<T, D, INTER>(a.w[side], a.w_f32, l, wa, wb);

  // the token and heads of a unit: runs change slowest, so that the CTAs work on neighbouring
  // tokens of the same heads
  auto open = [&](int u, int& b, int& s, int& h0, int& h1) -> bool {
    const unsigned tok = static_cast<unsigned>(u % tgroups) * kGroups + grp;
    h0 = u / tgroups * a.per_run;
    h1 = min(heads, h0 + a.per_run);
    const bool in = tok < static_cast<unsigned>(ntok);
    b = in ? static_cast<int>(tok / a.S) : 0;
    s = in ? static_cast<int>(tok % a.S) : 0;
    return in;
  };
  int fu = u0;   // the unit being fetched, its next head and rows
  int fh = 0, fh1 = 0, fstage = 0;
  bool fin = false;
  const T *fx = nullptr, *fg = nullptr;
  auto fetch = [&]() {
    if (fu < units) {
      if (fh >= fh1) {
        int b, s;
        fin = open(fu, b, s, fh, fh1);
        fx = static_cast<const T*>(a.x[side].p) + b * a.x[side].sb + s * a.x[side].ss;
        fg = static_cast<const T*>(a.dy[side].p) + b * a.dy[side].sb + s * a.dy[side].ss;
      }
      const uint32_t d = slot0 + fstage * kStep;
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const bool ok = fin && fh + j < fh1;
        const int h = fh + j < fh1 ? fh + j : 0;  // a copy of no bytes still names a valid row
        async_row<T, D, INTER>(d + 2 * j * kRow, fx + h * a.x[side].sh, l, ok);
        async_row<T, D, INTER>(d + (2 * j + 1) * kRow, fg + h * a.dy[side].sh, l, ok);
      }
      fh += kUnroll;
      if (fh >= fh1) fu += a.ctas[side];
      fstage = fstage + 1 == kBackAhead ? 0 : fstage + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kBackAhead; ++i) fetch();

  int stage = 0;
#pragma unroll 1
  for (int u = u0; u < units; u += a.ctas[side]) {
    int b, s, h_begin, h_end;
    const bool in = open(u, b, s, h_begin, h_end);
    const int pos = in ? checked_position(a.positions, a.pos_b, b, s, a.n_pos) : -1;
    if (pos == -2 && l == 0) report_device_error(kStatusBadLabel, kNormSite + 2);
    const bool live = pos >= 0;
    float c[4] = {}, sn[4] = {};
    if (live) load_angles<D>(a.cos, a.sin, pos, l, c, sn);
    T* drow = static_cast<T*>(a.dx[side].p) + b * a.dx[side].sb + s * a.dx[side].ss;
#pragma unroll 1
    for (int h0 = h_begin; h0 < h_end; h0 += kUnroll) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kBackAhead - 1) : "memory");
      Raw<T> rx[kUnroll], rg[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        rx[j] = read_slot<T>(ring + threadIdx.x * 16 + stage * kStep + 2 * j * kRow);
        rg[j] = read_slot<T>(ring + threadIdx.x * 16 + stage * kStep + (2 * j + 1) * kRow);
      }
      fetch();  // into the slots just read
      stage = stage + 1 == kBackAhead ? 0 : stage + 1;
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        float xa[4], xb[4], ga[4], gb[4], za[4], zb[4];
        to_pairs<T, INTER>(rx[j], xa, xb);
        to_pairs<T, INTER>(rg[j], ga, gb);
        if (!live) {  // a skipped row: zero gradients, nothing in the sums
#pragma unroll
          for (int i = 0; i < 4; ++i) xa[i] = xb[i] = ga[i] = gb[i] = 0.f;
        }
        // pairs of fp32 operations (f32x2): the pass is close to issue-bound
        float p0 = 0.f, p1 = 0.f, d0 = 0.f, d1 = 0.f, ta[4], tb[4];
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          float u0, u1;
          mul2(u0, u1, gb[i], gb[i + 1], sn[i], sn[i + 1]);
          fma2(za[i], za[i + 1], ga[i], ga[i + 1], c[i], c[i + 1], u0, u1);
          mul2(u0, u1, ga[i], ga[i + 1], -sn[i], -sn[i + 1]);
          fma2(zb[i], zb[i + 1], gb[i], gb[i + 1], c[i], c[i + 1], u0, u1);
          fma2(p0, p1, xa[i], xa[i + 1], xa[i], xa[i + 1], p0, p1);
          fma2(p0, p1, xb[i], xb[i + 1], xb[i], xb[i + 1], p0, p1);
          mul2(ta[i], ta[i + 1], za[i], za[i + 1], xa[i], xa[i + 1]);
          mul2(tb[i], tb[i + 1], zb[i], zb[i + 1], xb[i], xb[i + 1]);
          fma2(d0, d1, ta[i], ta[i + 1], wa[i], wa[i + 1], d0, d1);
          fma2(d0, d1, tb[i], tb[i + 1], wb[i], wb[i + 1], d0, d1);
        }
        const float ss = row_sum<D>(p0 + p1), dot = row_sum<D>(d0 + d1);
        // (a row behind the run's last head is zeros, whose root without an eps is infinite)
        const float r = live && h0 + j < h_end ? rsqrtf(ss * (1.f / D) + a.eps) : 0.f;
        const float nk = -(r * r * dot * (1.f / D)) * r;
        float oa[4], ob[4];
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          float u0, u1;
          fma2(dwa[i], dwa[i + 1], ta[i], ta[i + 1], r, r, dwa[i], dwa[i + 1]);
          fma2(dwb[i], dwb[i + 1], tb[i], tb[i + 1], r, r, dwb[i], dwb[i + 1]);
          mul2(u0, u1, wa[i], wa[i + 1], r, r);
          mul2(oa[i], oa[i + 1], za[i], za[i + 1], u0, u1);
          fma2(oa[i], oa[i + 1], xa[i], xa[i + 1], nk, nk, oa[i], oa[i + 1]);
          mul2(u0, u1, wb[i], wb[i + 1], r, r);
          mul2(ob[i], ob[i + 1], zb[i], zb[i + 1], u0, u1);
          fma2(ob[i], ob[i + 1], xb[i], xb[i + 1], nk, nk, ob[i], ob[i + 1]);
        }
        if (in && h0 + j < h_end) store_row<T, D, INTER>(drow + (h0 + j) * a.dx[side].sh, l, oa, ob);
      }
    }
  }
  launch_dependents();
  // the lane groups' sums, added in group order
  __shared__ float red[kGroups][D];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int da = INTER ? 8 * l + 2 * i : 4 * l + i;
    const int db = INTER ? da + 1 : D / 2 + 4 * l + i;
    red[grp][da] = dwa[i];
    red[grp][db] = dwb[i];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float t = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) t += red[g][threadIdx.x];
    a.part[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] = t;
  }
}

// Sum of the CTAs' shares; grid (D / 32, sides): warp w adds the side's shares w, w + 32, ...
// and the warps' sums are added in order, in fp64 (hundreds of shares with cancelling signs).
__global__ void __launch_bounds__(1024) norm_weight_sum_kernel(const float* __restrict__ part, int nq,
                                                               int nk, int D, float* __restrict__ dqw,
                                                               float* __restrict__ dkw) {
  __shared__ double red[32][33];
  wait_for_primary();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, side = blockIdx.y;
  const int col = blockIdx.x * 32 + lane;
  const float* p = part + (side ? static_cast<size_t>(nq) * D : 0) + col;
  const int n = side ? nk : nq;
  double t = 0.0;
#pragma unroll 4
  for (int i = w; i < n; i += 32) t += static_cast<double>(p[static_cast<size_t>(i) * D]);
  red[w][lane] = t;
  __syncthreads();
  if (w == 0) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][lane];
    (side ? dkw : dqw)[col] = static_cast<float>(s);
  }
}

constexpr int kNormBackCtas = 148 * 2;  // resident at once
constexpr int kNormBackRun = 8;          // heads of a unit at most: units much smaller than a CTA's share

int norm_elem_bytes(int dtype) { return dtype == BSA_F32 ? 4 : 2; }

int check_heads(const bsa_heads& h, int dtype, const char* name) {
  if (!h.ptr) return fail(BSA_ERR_INVALID_ARG, "%s is null", name);
  const int unit = 16 / norm_elem_bytes(dtype);
  if (reinterpret_cast<uintptr_t>(h.ptr) % 16 || h.stride_b % unit || h.stride_h % unit ||
      h.stride_s % unit)
    return fail(BSA_ERR_INVALID_ARG, "%s: pointer or strides not multiples of 16 bytes", name);
  return BSA_OK;
}

int check_norm_common(const bsa_shape& s, const void* qw, const void* kw, const float* cos,
                      const float* sin, int n_pos, float eps) {
  if (s.dtype != BSA_BF16 && s.dtype != BSA_F16 && s.dtype != BSA_F32)
    return fail(BSA_ERR_UNSUPPORTED, "dtype %d", s.dtype);
  if (s.D != 64 && s.D != 128) return fail(BSA_ERR_UNSUPPORTED, "head dim %d not in {64,128}", s.D);
  if (s.B < 0 || s.Sq < 0 || s.Hq <= 0 || s.Hkv <= 0 || s.Sq != s.Sk)
    return fail(BSA_ERR_INVALID_ARG, "bad shape");
  if (s.Hq > 16384 || s.Hkv > 16384) return fail(BSA_ERR_UNSUPPORTED, "more than 16384 heads");
  if (static_cast<int64_t>(s.B) * s.Sq > INT32_MAX)
    return fail(BSA_ERR_UNSUPPORTED, "B*S exceeds 2^31 - 1");
  if (static_cast<int64_t>(s.B) * s.Sq * std::max(s.Hq, s.Hkv) > (int64_t(1) << 36))
    return fail(BSA_ERR_UNSUPPORTED, "more than 2^36 rows");
  if (!(eps >= 0.f)) return fail(BSA_ERR_INVALID_ARG, "eps < 0");
  if (n_pos < 0) return fail(BSA_ERR_INVALID_ARG, "n_pos < 0");
  if (!qw || !kw || (n_pos > 0 && (!cos || !sin))) return fail(BSA_ERR_INVALID_ARG, "null pointer");
  if (reinterpret_cast<uintptr_t>(cos) % 16 || reinterpret_cast<uintptr_t>(sin) % 16)
    return fail(BSA_ERR_INVALID_ARG, "cos and sin must be 16-byte aligned");
  return BSA_OK;
}

HeadsIn in_of(const bsa_heads& h) { return {h.ptr, h.stride_b, h.stride_h, h.stride_s}; }
HeadsOut out_of(const bsa_heads& h) { return {h.ptr, h.stride_b, h.stride_h, h.stride_s}; }

// Heads of a run: a lane group walks over all heads of its token's section when the tokens
// alone fill the GPU several times over, and over fewer, in whole steps of 4, when not.
int heads_per_run(int64_t token_groups, int heads) {
  // CTAs to aim at. 1560 tokens into the cache: 13.3 us with 3, 4 or 6 per SM, 15.4 with 8;
  // 4000 tokens of 80 heads: 44, 44, 36.9 and 37.9.
  constexpr int64_t kWant = 148 * 6;
  const int64_t runs = std::min<int64_t>((heads + 3) / 4, std::max<int64_t>(1, kWant / std::max<int64_t>(token_groups, 1)));
  return static_cast<int>(((heads + runs - 1) / runs + 3) / 4 * 4);
}

template <typename T, int D, bool PAGED>
void launch_norm_t(const NormArgs& a, dim3 grid, int interleaved, cudaStream_t st) {
  if (interleaved) norm_rotation_kernel<T, D, true, PAGED><<<grid, kNormThreads, 0, st>>>(a);
  else norm_rotation_kernel<T, D, false, PAGED><<<grid, kNormThreads, 0, st>>>(a);
}

template <bool PAGED>
int launch_norm(NormArgs& a, int dtype, int D, int interleaved, cudaStream_t st) {
  const int64_t ntok = static_cast<int64_t>(a.B) * a.S;
  const int per_cta = kNormThreads / (D / 8);
  const int64_t tg = (ntok + per_cta - 1) / per_cta;
  a.per_run = heads_per_run(tg, a.heads[0] + a.heads[1] + a.heads[2]);
  a.first_run[1] = ceil_div(a.heads[0], a.per_run);
  a.first_run[2] = a.first_run[1] + ceil_div(a.heads[1], a.per_run);
  const dim3 grid(static_cast<unsigned>(tg), a.first_run[2] + ceil_div(a.heads[2], a.per_run));
#define BSA_NORM(T)                                                              \
  (D == 64 ? launch_norm_t<T, 64, PAGED>(a, grid, interleaved, st)               \
           : launch_norm_t<T, 128, PAGED>(a, grid, interleaved, st))
  if (dtype == BSA_BF16) BSA_NORM(__nv_bfloat16);
  else if (dtype == BSA_F16) BSA_NORM(__half);
  else if constexpr (!PAGED) BSA_NORM(float);
#undef BSA_NORM
  count_launch();
  return check_cuda(cudaGetLastError(), "norm_rotation_kernel");
}

template <typename T, int D>
int launch_norm_back(const NormBackArgs& a, int ctas, int interleaved, cudaStream_t st) {
  auto kern = interleaved ? norm_rotation_back_kernel<T, D, true> : norm_rotation_back_kernel<T, D, false>;
  constexpr int smem = norm_back_smem<T>();
  // the static part, 8 KB, counts too
  const int e = check_cuda(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                           "cudaFuncSetAttribute(norm_rotation_back_kernel)");
  if (e != BSA_OK) return e;
  kern<<<ctas, kNormThreads, smem, st>>>(a);
  count_launch();
  return check_cuda(cudaGetLastError(), "norm_rotation_back_kernel");
}

// CTAs of the backward pass, by side in proportion to the heads: each leaves one share of its
// side's weight sums.
void norm_back_plan(const bsa_shape& s, int* per_run, int (&ctas)[2]) {
  const int per_cta = kNormThreads / (s.D / 8);
  const int64_t tg = (static_cast<int64_t>(s.B) * s.Sq + per_cta - 1) / per_cta;
  *per_run = std::min(kNormBackRun, heads_per_run(tg, s.Hq + s.Hkv));
  const int h[2] = {s.Hq, s.Hkv};
  for (int i = 0; i < 2; ++i) {
    const int64_t units = std::max<int64_t>(1, tg * ceil_div(h[i], *per_run));
    const int64_t share = std::max<int64_t>(1, static_cast<int64_t>(kNormBackCtas) * h[i] / (s.Hq + s.Hkv));
    ctas[i] = static_cast<int>(std::min(units, share));
  }
}

}  // namespace

}  // namespace bsa

extern "C" {

int bsa_qk_norm_rotation(bsa_heads q, bsa_heads k, bsa_shape shape, const void* q_weight,
                         const void* k_weight, int weight_f32, const float* cos, const float* sin,
                         int n_pos, const int32_t* positions, int64_t pos_b_stride, float eps,
                         int interleaved, bsa_heads q_out, bsa_heads k_out, void* stream) {
  using namespace bsa;
  int st = check_norm_common(shape, q_weight, k_weight, cos, sin, n_pos, eps);
  if (st != BSA_OK) return st;
  if (static_cast<int64_t>(shape.B) * shape.Sq == 0) return BSA_OK;
  if ((st = check_heads(q, shape.dtype, "q")) || (st = check_heads(k, shape.dtype, "k")) ||
      (st = check_heads(q_out, shape.dtype, "q_out")) || (st = check_heads(k_out, shape.dtype, "k_out")))
    return st;
  if (!positions && shape.Sq > n_pos)
    return fail(BSA_ERR_INVALID_ARG, "%d tokens, %d positions in the table", shape.Sq, n_pos);
  NormArgs a{};
  a.x[0] = in_of(q);
  a.x[1] = in_of(k);
  a.y[0] = out_of(q_out);
  a.y[1] = out_of(k_out);
  a.B = shape.B;
  a.S = shape.Sq;
  a.heads[0] = shape.Hq;
  a.heads[1] = shape.Hkv;
  a.w[0] = q_weight;
  a.w[1] = k_weight;
  a.w_f32 = weight_f32;
  a.cos = cos;
  a.sin = sin;
  a.n_pos = n_pos;
  a.positions = positions;
  a.pos_b = pos_b_stride;
  a.eps = eps;
  return launch_norm<false>(a, shape.dtype, shape.D, interleaved, as_stream(stream));
}

size_t bsa_qk_norm_rotation_workspace_bytes(bsa_shape shape) {
  if ((shape.D != 64 && shape.D != 128) || shape.B < 0 || shape.Sq < 0 || shape.Hq <= 0 ||
      shape.Hkv <= 0 || shape.Hq > 16384 || shape.Hkv > 16384)
    return 0;
  int per_run, ctas[2];
  bsa::norm_back_plan(shape, &per_run, ctas);
  return bsa::align_up(static_cast<size_t>(ctas[0] + ctas[1]) * shape.D * sizeof(float), 256);
}

int bsa_qk_norm_rotation_backward(bsa_heads dq_out, bsa_heads dk_out, bsa_heads q, bsa_heads k,
                                  bsa_shape shape, const void* q_weight, const void* k_weight,
                                  int weight_f32, const float* cos, const float* sin, int n_pos,
                                  const int32_t* positions, int64_t pos_b_stride, float eps,
                                  int interleaved, bsa_heads dq, bsa_heads dk, float* dq_weight,
                                  float* dk_weight, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  using namespace bsa;
  int st = check_norm_common(shape, q_weight, k_weight, cos, sin, n_pos, eps);
  if (st != BSA_OK) return st;
  if (!dq_weight || !dk_weight) return fail(BSA_ERR_INVALID_ARG, "null weight gradient");
  const bool none = static_cast<int64_t>(shape.B) * shape.Sq == 0;
  if (!none) {
    if ((st = check_heads(dq_out, shape.dtype, "dq_out")) || (st = check_heads(dk_out, shape.dtype, "dk_out")) ||
        (st = check_heads(q, shape.dtype, "q")) || (st = check_heads(k, shape.dtype, "k")) ||
        (st = check_heads(dq, shape.dtype, "dq")) || (st = check_heads(dk, shape.dtype, "dk")))
      return st;
    if (!positions && shape.Sq > n_pos)
      return fail(BSA_ERR_INVALID_ARG, "%d tokens, %d positions in the table", shape.Sq, n_pos);
  }
  if (!workspace || workspace_bytes < bsa_qk_norm_rotation_workspace_bytes(shape))
    return fail(BSA_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes,
                bsa_qk_norm_rotation_workspace_bytes(shape));
  if (reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(BSA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  NormBackArgs a{};
  a.x[0] = in_of(q);
  a.x[1] = in_of(k);
  a.dy[0] = in_of(dq_out);
  a.dy[1] = in_of(dk_out);
  a.dx[0] = out_of(dq);
  a.dx[1] = out_of(dk);
  a.B = shape.B;
  a.S = shape.Sq;
  a.heads[0] = shape.Hq;
  a.heads[1] = shape.Hkv;
  a.w[0] = q_weight;
  a.w[1] = k_weight;
  a.w_f32 = weight_f32;
  a.cos = cos;
  a.sin = sin;
  a.n_pos = n_pos;
  a.positions = positions;
  a.pos_b = pos_b_stride;
  a.eps = eps;
  a.part = static_cast<float*>(workspace);
  if (!none) norm_back_plan(shape, &a.per_run, a.ctas);
  const int ctas = a.ctas[0] + a.ctas[1];
  cudaStream_t cs = as_stream(stream);
  if (!none) {
#define BSA_NORM_BACK(T)                                                       \
  (shape.D == 64 ? launch_norm_back<T, 64>(a, ctas, interleaved, cs)            \
                 : launch_norm_back<T, 128>(a, ctas, interleaved, cs))
    if (shape.dtype == BSA_BF16) st = BSA_NORM_BACK(__nv_bfloat16);
    else if (shape.dtype == BSA_F16) st = BSA_NORM_BACK(__half);
    else st = BSA_NORM_BACK(float);
#undef BSA_NORM_BACK
    if (st != BSA_OK) return st;
  }
  count_launch();
  return check_cuda(launch_dependent(norm_weight_sum_kernel, dim3(shape.D / 32, 2), dim3(1024), 0, cs, a.part,
                                     a.ctas[0], a.ctas[1], shape.D, dq_weight, dk_weight),
                    "norm_weight_sum_kernel");
}

int bsa_paged_qk_norm_append(bsa_heads q, bsa_heads k, bsa_heads v, int T, int Hq,
                             const void* q_weight, const void* k_weight, int weight_f32,
                             const float* cos, const float* sin, int n_pos,
                             const int32_t* positions, const int32_t* slots, float eps,
                             int interleaved, bsa_heads q_out, bsa_paged_cache cache,
                             void* stream) {
  using namespace bsa;
  int st = check_paged_cache(cache);
  if (st != BSA_OK) return st;
  const bsa_shape shape{1, Hq, cache.Hkv, T, T, cache.D, cache.dtype};
  if ((st = check_norm_common(shape, q_weight, k_weight, cos, sin, n_pos, eps)) != BSA_OK) return st;
  if (T == 0) return BSA_OK;
  if (!positions || !slots) return fail(BSA_ERR_INVALID_ARG, "positions or slots is null");
  q.stride_b = k.stride_b = v.stride_b = q_out.stride_b = 0;
  if ((st = check_heads(q, cache.dtype, "q")) || (st = check_heads(k, cache.dtype, "k")) ||
      (st = check_heads(v, cache.dtype, "v")) || (st = check_heads(q_out, cache.dtype, "q_out")))
    return st;
  NormArgs a{};
  a.x[0] = in_of(q);
  a.x[1] = in_of(k);
  a.x[2] = in_of(v);
  a.y[0] = out_of(q_out);
  a.y[1] = {cache.k, cache.k_page_stride, cache.k_head_stride, cache.k_row_stride};
  a.y[2] = {cache.v, cache.v_page_stride, cache.v_head_stride, cache.v_row_stride};
  a.B = 1;
  a.S = T;
  a.heads[0] = Hq;
  a.heads[1] = a.heads[2] = cache.Hkv;
  a.w[0] = q_weight;
  a.w[1] = k_weight;
  a.w_f32 = weight_f32;
  a.cos = cos;
  a.sin = sin;
  a.n_pos = n_pos;
  a.positions = positions;
  a.eps = eps;
  a.slots = slots;
  a.page_shift = __builtin_ctz(cache.page);
  a.n_slots = cache.n_pages * cache.page;
  return launch_norm<true>(a, cache.dtype, cache.D, interleaved, as_stream(stream));
}

}  // extern "C"
