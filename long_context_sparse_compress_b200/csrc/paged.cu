// Raw tokens in an 8-bit paged cache: the plan of a serving step, the store of
// new rows, the float32 form of the attention and the join of split items.
// The tensor-core forms of the attention are in paged_mma.cu; the schedule that
// all forms walk is in paged.cuh.
//
// Plain attention over raw tokens stands beside the compressed layers: "How
// DeepSeek V4 Handles 1M Token Context" (docs.bswen.com) puts the crossover of
// the compressed form at about 8K tokens.
#include <type_traits>

#include "kernels.cuh"
#include "launches.h"
#include "paged.cuh"

namespace lcsc {
namespace {

// ------------------------------------------------------------------- plan
// need_b = ceil((c_b + n_b) / P) - ceil(c_b / P) pages for each request; the
// exclusive prefix sum of need places a request's pages in the stack, that of
// n its rows.  One CTA makes the prefix sums over the requests (8 bytes read
// and 16 written per request); the rows are filled in by the same CTA when
// they are few, else by a grid of their own (see kFillHere).

constexpr int kPlanThreads = 1024;
// Rows up to which the planning CTA fills in the rows itself.
constexpr int64_t kFillHere = 4096;

struct PlanRow {
  bool ended, fits;
  int64_t n, have, need;
};

__device__ __forceinline__ PlanRow plan_row(const PagePlanLaunch& a, int b) {
  PlanRow r;
  const int64_t c = a.cached[b], n = a.n_new[b];
  r.ended = n < 0;
  r.n = n < 0 ? 0 : n;
  r.have = c > 0 ? (c + a.page - 1) >> a.page_log2 : 0;
  r.fits = !r.ended && c >= 0 && c + n <= a.max_blocks * a.page;
  r.need = r.fits ? ((c + n + a.page - 1) >> a.page_log2) - r.have : 0;
  return r;
}

// Inclusive sums over the CTA of two values, added to the carried ones.
__device__ __forceinline__ void plan_scan2(int64_t& x, int64_t& y, int64_t (*tot)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += u, y += v;
  }
  __syncthreads();
  if (lane == 31) tot[warp][0] = x, tot[warp][1] = y;
  __syncthreads();
  if (warp == 0) {
    int64_t u = tot[lane][0], v = tot[lane][1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t p = __shfl_up_sync(0xffffffffu, u, o), q = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) u += p, v += q;
    }
    tot[lane][0] = u, tot[lane][1] = v;
  }
  __syncthreads();
  if (warp > 0) x += tot[warp - 1][0], y += tot[warp - 1][1];
}

// Slot and position of row t, and the table's entry where the row is the
// first of a page.
__device__ __forceinline__ void plan_fill(const PagePlanLaunch& a, int64_t t) {
  int lo = 0, hi = a.B;  // the last request whose first row is <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.q_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  int32_t slot = -1, pos = -1;
  if (t < a.q_start[lo + 1] && a.ctx_len[lo] > 0) {
    const int32_t c = a.cached[lo];
    pos = (int32_t)(t - a.q_start[lo]) + c;
    const int64_t col = pos >> a.page_log2, have = ((int64_t)c + a.page - 1) >> a.page_log2;
    int32_t* entry = a.table + (int64_t)lo * a.max_blocks + col;
    int32_t page;
    if (col < have) {
      page = *entry;
    } else {
      page = a.free_pages[a.scratch[0] - 1 - (a.scratch[2 + lo] + col - have)];
      if ((pos & (a.page - 1)) == 0) *entry = page;
    }
    if (page < 0 || page >= a.n_pages) {
      if (a.status) atomicOr(a.status, LCSC_DEV_BAD_INDEX);
    } else {
      slot = (int32_t)((page << a.page_log2) + (pos & (a.page - 1)));
    }
  }
  a.slots[t] = slot;
  if (a.positions) a.positions[t] = pos;
}

// The pages among the table entries of a warp's ended requests (`give` of the
// lane's) onto the stack from place `at` of each on; returns the lane's count.
// With copy false they are only counted.
__device__ __noinline__ int64_t plan_return(const PagePlanLaunch& a, int b_warp, int64_t give, int64_t at, bool copy) {
  const int lane = threadIdx.x & 31;
  int64_t mine = 0;
  for (unsigned todo = __ballot_sync(0xffffffffu, give > 0); todo; todo &= todo - 1) {
    const int src = __ffs(todo) - 1;
    const int64_t n = __shfl_sync(0xffffffffu, give, src), first = __shfl_sync(0xffffffffu, at, src);
    const int32_t* row = a.table + (int64_t)(b_warp + src) * a.max_blocks;
    int64_t to = first;
    for (int64_t i0 = 0; i0 < n; i0 += 32) {
      const int32_t page = i0 + lane < n ? row[i0 + lane] : -1;
      const unsigned there = __ballot_sync(0xffffffffu, page >= 0);
      const int64_t place = to + __popc(there & ((1u << lane) - 1));
      if (copy && page >= 0 && place < a.n_pages) a.free_pages[place] = page;
      to += __popc(there);
    }
    if (lane == src) mine = to - first;
  }
  return mine;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const __grid_constant__ PagePlanLaunch a, bool fill) {
  grid_dep_wait();
  __shared__ int64_t tot[32][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t height = a.n_free[0];
  height = height < 0 ? 0 : height > a.n_pages ? a.n_pages : height;
  int bits = 0;
  // the ended requests' pages onto the stack
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int64_t give = 0, zero = 0;
    if (b < a.B) {
      const PlanRow r = plan_row(a, b);
      if (r.ended) {
        give = r.have;
        if (give > a.max_blocks) give = a.max_blocks, bits |= LCSC_DEV_BAD_LENGTH;
      }
    }
    if (!__syncthreads_or(give > 0)) continue;
    const int64_t mine = give, below = height;
    plan_scan2(give, zero, tot);
    const int64_t at = height + give - mine;
    height += tot[31][0];
    // a warp at a time copies the pages of its 32 requests
    int holes = 0;
    for (unsigned todo = __ballot_sync(0xffffffffu, mine > 0); todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const int64_t n = __shfl_sync(0xffffffffu, mine, src), to = __shfl_sync(0xffffffffu, at, src);
      const int32_t* row = a.table + (int64_t)(b0 + warp * 32 + src) * a.max_blocks;
      for (int64_t i0 = lane; i0 < n; i0 += 256) {  // eight loads in flight
        int32_t pg[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          pg[k] = i0 + 32 * k < n ? row[i0 + 32 * k] : 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i0 + 32 * k < n && to + i0 + 32 * k < a.n_pages) a.free_pages[to + i0 + 32 * k] = pg[k];
#pragma unroll
        for (int k = 0; k < 8; ++k) holes |= pg[k];
      }
    }
    if (__syncthreads_or(holes < 0)) {  // once more without the entries that are none (to count first always: 18.6 -> 32.3 us)
      const int64_t real = plan_return(a, b0 + warp * 32, mine, 0, false);
      int64_t upto = real;
      plan_scan2(upto, zero, tot);
      height = below + tot[31][0];
      plan_return(a, b0 + warp * 32, mine, below + upto - real, true);
      __syncthreads();
    }
  }
  if (height > a.n_pages) height = a.n_pages, bits |= LCSC_DEV_BAD_INDEX;
  // pages and rows, in request order
  int64_t pages0 = 0, rows0 = 0, taken = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    PlanRow r = {};
    int64_t c = 0;
    if (b < a.B) {
      r = plan_row(a, b);
      c = a.cached[b];
    }
    int64_t rows = r.n, zero = 0;
    plan_scan2(rows, zero, tot);
    const int64_t q_end = rows0 + rows;
    rows0 += tot[31][0];
    const bool fits = r.fits && q_end <= a.n_tokens;
    const int64_t need = fits ? r.need : 0;
    int64_t upto = need, got = 0;
    plan_scan2(upto, got, tot);
    upto += pages0;
    pages0 += tot[31][0];
    const bool part = fits && (need == 0 || upto <= height);
    if (b < a.B) {
      if (!r.ended && !fits) bits |= LCSC_DEV_BAD_LENGTH;
      if (fits && !part) bits |= LCSC_DEV_NO_PAGES;
      a.ctx_len[b] = part ? (int32_t)(c + r.n) : 0;
      const int64_t q0 = q_end - r.n;
      a.q_start[b] = (int32_t)(q0 < a.n_tokens ? q0 : a.n_tokens);
      if (b == a.B - 1) a.q_start[a.B] = (int32_t)(q_end < a.n_tokens ? q_end : a.n_tokens);
      a.scratch[2 + b] = upto - need;
      if (part) taken += need;
    }
  }
  int64_t zero = 0;
  plan_scan2(taken, zero, tot);
  if (tid == 0) {
    a.scratch[0] = height;
    a.n_free_out[0] = (int32_t)(height - tot[31][0]);
  }
  if (bits && a.status) atomicOr(a.status, bits);
  if (!fill) return;
  __syncthreads();
  for (int64_t t = tid; t < a.n_tokens; t += kPlanThreads) plan_fill(a, t);
}

__global__ void __launch_bounds__(256) page_fill_kernel(PagePlanLaunch a) {
  grid_dep_wait();
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < a.n_tokens; t += (int64_t)gridDim.x * 256)
    plan_fill(a, t);
}

// ------------------------------------------------------------------ store
// A run is the adjacent tokens of one page in rising slot order: the unit of
// work, as a page's scale needs the largest magnitude of all of them.  One CTA
// looks at TILE tokens, finds the runs that begin there and stores them for one
// KV head of K or of V.  A run of up to kWarpRun rows is a warp's own (decode
// steps: one row each); a longer one (prompts: whole pages) is cut into 16-byte
// chunks that the CTA's threads share, IT for each, so that they are all in
// flight at once and wait in IT x 4 registers for the maximum.  Every row is
// read once and written once.

constexpr int kStoreWarps = 8;
constexpr int kWarpRun = 8;
constexpr int kMaxPage = 128;

// The least power of two s with amax <= 448 s, not below 2^-100, as an exponent.
__device__ __forceinline__ int scale_exp(float amax) {
  // amax = m 2^e, m in [1, 2): 448 = 1.75 * 2^8
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127;
  const int s = e - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return s < -100 ? -100 : s;  // subnormal and zero amax: e = -127
}
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// Lane's VPL values of a row; values that are not finite become 0 (and are reported).
template <int VPL>
__device__ __forceinline__ bool store_load(const void* x, int64_t at, int dtype, float (&v)[VPL]) {
  if (dtype == LCSC_DT_BF16) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(x) + at;
    uint32_t w[VPL / 2];
    if constexpr (VPL == 4) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x, w[1] = u.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
#pragma unroll
    for (int i = 0; i < VPL / 2; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float* p = reinterpret_cast<const float*>(x) + at;
    if constexpr (VPL == 4) {
      const float4 u = *reinterpret_cast<const float4*>(p);
      v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    } else {
      const float2 u = *reinterpret_cast<const float2*>(p);
      v[0] = u.x, v[1] = u.y;
    }
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if (!(fabsf(v[i]) <= 3.402823466e38f)) v[i] = 0.f, bad = true;
  }
  return bad;
}

template <int VPL>
__device__ __forceinline__ float store_amax(const float (&v)[VPL]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) a = fmaxf(a, fabsf(v[i]));
  return a;
}

template <int VPL>
__device__ __forceinline__ void store_codes(uint8_t* dst, const float (&v)[VPL], float inv) {
  if constexpr (VPL == 4) {
    const uint32_t lo = e4m3x2_code(v[0] * inv, v[1] * inv), hi = e4m3x2_code(v[2] * inv, v[3] * inv);
    *reinterpret_cast<uint32_t*>(dst) = lo | (hi << 16);
  } else {
    *reinterpret_cast<uint16_t*>(dst) = e4m3x2_code(v[0] * inv, v[1] * inv);
  }
}

// The first `bytes` codes of a page's head, times r (a power of two < 1).
__device__ __forceinline__ void rescale_codes(uint8_t* p, int bytes, float r, int from, int step) {
  for (int i = from * 4; i < bytes; i += step * 4) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p + i);
    const float2 a = e4m3x2_val((uint16_t)w), b = e4m3x2_val((uint16_t)(w >> 16));
    *reinterpret_cast<uint32_t*>(p + i) =
        e4m3x2_code(a.x * r, a.y * r) | ((uint32_t)e4m3x2_code(b.x * r, b.y * r) << 16);
  }
}

// Values of a 16-byte chunk: eight of bf16 or four of float32.
template <bool F32>
__device__ __forceinline__ void chunk_values(const uint4& u, float (&v)[F32 ? 4 : 8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) {
      v[i] = __uint_as_float(w[i]);
    } else {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// Its largest magnitude, as float32 bits.
template <bool F32>
__device__ __forceinline__ uint32_t chunk_amax(const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = F32 ? max(m, w[i] & 0x7fffffffu) : __vmaxu2(m, w[i] & 0x7fff7fffu);
  return F32 ? m : max(m << 16, m & 0xffff0000u);
}

// Zero in the place of the values that are not finite.
template <bool F32>
__device__ __forceinline__ void chunk_finite(uint4& u) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (F32) {
      if ((w[i] & 0x7fffffffu) >= 0x7f800000u) w[i] = 0;
    } else {
      if ((w[i] & 0x7fffu) >= 0x7f80u) w[i] &= 0xffff0000u;
      if ((w[i] & 0x7fff0000u) >= 0x7f800000u) w[i] &= 0xffffu;
    }
  }
  u = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int VPL, int TILE, bool F32, int IT>
__global__ void __launch_bounds__(kStoreWarps * 32) paged_store_kernel(PagedStoreLaunch a) {
  grid_dep_wait();
  constexpr int D = VPL * 32, kDt = F32 ? LCSC_DT_F32 : LCSC_DT_BF16;
  constexpr int VPC = F32 ? 4 : 8, CPR = D / VPC;  // values of a chunk, chunks of a row
  constexpr int kLook = TILE + kMaxPage;  // a run that begins in the tile ends within these
  static_assert(kLook <= kStoreWarps * 32, "one thread per slot looked at");
  __shared__ int32_t slot_s[kLook];
  __shared__ uint32_t goes_on[kStoreWarps];  // bit: the row goes on its neighbour's run
  __shared__ uint32_t starts[kStoreWarps];   // bit: the row begins a run
  __shared__ int red[kStoreWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t0 = (int64_t)blockIdx.x * TILE;
  const int h = blockIdx.y, z = blockIdx.z;
  int bits = 0;
  {
    const int64_t t = t0 + tid;
    int32_t s = -1, before = -1;
    bool gap = false;
    if (tid < kLook && t < a.n_tokens) {
      s = a.slots[t];
      if (t > 0) before = a.slots[t - 1];
      // behind skipped rows it is the last one before them that may have the page
      gap = s >= 0 && t > 0 && before < 0;
      if (gap)
        for (int64_t u = t - 2; u >= 0 && u > t - kMaxPage && before < 0; --u) before = a.slots[u];
    }
    if (tid < kLook) slot_s[tid] = s;
    const bool same = s >= 0 && before >= 0 && (s >> a.page_log2) == (before >> a.page_log2);
    const bool on = same && !gap && s == before + 1;
    bool start = s >= 0 && !on && tid < TILE;
    // out of order within a page, or past the pool
    if (start && (same || (s >> a.page_log2) >= a.n_pages)) start = false, bits |= LCSC_DEV_BAD_INDEX;
    const uint32_t m_on = __ballot_sync(0xffffffffu, on), m_st = __ballot_sync(0xffffffffu, start);
    if (lane == 0) goes_on[warp] = m_on, starts[warp] = m_st;
  }
  __syncthreads();
  auto run_of = [&](int i) {  // rows of the run that begins at i
    int n = 1;
    while (i + n < kLook) {
      const int at = i + n;
      const uint32_t stop = ~goes_on[at >> 5] >> (at & 31);
      const int len = 32 - (at & 31);
      const int on = stop ? min(__ffs(stop) - 1, len) : len;
      n += on;
      if (on < len) break;
    }
    return n;
  };
  uint8_t* codes = z == 0 ? a.codes[0] : a.codes[1];
  float* scales = z == 0 ? a.scale[0] : a.scale[1];
  const void* x = z == 0 ? a.x[0] : a.x[1];
  const int64_t stride = z == 0 ? a.stride[0] : a.stride[1];
  const int64_t x0 = t0 * stride + h * D + lane * VPL;
  bool bad = false;
  // short runs, a warp each; the longer ones are left for the whole CTA
  int turn = 0;
  bool any_long = false;
#pragma unroll 1
  for (int wd = 0; wd < (TILE + 31) / 32; ++wd) {
#pragma unroll 1
    for (uint32_t m = starts[wd]; m; m &= m - 1) {
      const int i = wd * 32 + __ffs(m) - 1;
      const int n = run_of(i);
      if (n > kWarpRun) {
        any_long = true;
        continue;
      }
      if ((turn++ % kStoreWarps) != warp) continue;
      const int32_t s = slot_s[i];
      const int first = s & (a.page - 1);
      const int64_t ph = (int64_t)(s >> a.page_log2) * a.Hkv + h;
      const float old = first > 0 ? scales[ph] : 0.f;
      float v[kWarpRun][VPL], amax = 0.f;
#pragma unroll
      for (int r = 0; r < kWarpRun; ++r) {
        if (r < n) {
          bad |= store_load<VPL>(x, x0 + (i + r) * stride, kDt, v[r]);
          amax = fmaxf(amax, store_amax<VPL>(v[r]));
        }
      }
      const float want = exp2i(scale_exp(warp_max(amax)));
      const float sc = fmaxf(want, old), inv = 1.f / sc;
      uint8_t* page = codes + (ph * a.page) * D;
      if (first > 0 && sc > old) rescale_codes(page, first * D, old * inv, lane, 32);
#pragma unroll
      for (int r = 0; r < kWarpRun; ++r)
        if (r < n) store_codes<VPL>(page + (int64_t)(first + r) * D + lane * VPL, v[r], inv);
      if (lane == 0 && sc != old) scales[ph] = sc;
    }
  }
  // long runs, the whole CTA
  if (any_long) {
#pragma unroll 1
    for (int wd = 0; wd < (TILE + 31) / 32; ++wd) {
#pragma unroll 1
      for (uint32_t m = starts[wd]; m; m &= m - 1) {
        const int i = wd * 32 + __ffs(m) - 1;
        const int n = run_of(i);
        if (n <= kWarpRun) continue;
        const int32_t s = slot_s[i];
        const int first = s & (a.page - 1);
        const int64_t ph = (int64_t)(s >> a.page_log2) * a.Hkv + h;
        const float old = first > 0 ? scales[ph] : 0.f;
        const uint8_t* src = reinterpret_cast<const uint8_t*>(x) + ((t0 + i) * stride + h * D) * (F32 ? 4 : 2);
        uint4 u[IT];
        uint32_t amax = 0;  // float32 bits of the largest magnitude, which order as the numbers do
#pragma unroll
        for (int k = 0; k < IT; ++k) {
          const int c = tid + k * kStoreWarps * 32, row = c / CPR;
          u[k] = make_uint4(0, 0, 0, 0);
          if (row < n) u[k] = *reinterpret_cast<const uint4*>(src + row * stride * (F32 ? 4 : 2) + (c % CPR) * 16);
        }
#pragma unroll
        for (int k = 0; k < IT; ++k) amax = max(amax, chunk_amax<F32>(u[k]));
        // some value is not finite; with the barrier before this run's maxima
        if (__syncthreads_or(amax >= 0x7f800000u)) {
          bad |= amax >= 0x7f800000u;
          amax = 0;
#pragma unroll
          for (int k = 0; k < IT; ++k) {
            chunk_finite<F32>(u[k]);
            amax = max(amax, chunk_amax<F32>(u[k]));
          }
        }
        amax = __reduce_max_sync(0xffffffffu, amax);
        if (lane == 0) red[warp] = (int)amax;
        __syncthreads();
        int top = red[0];
#pragma unroll
        for (int w = 1; w < kStoreWarps; ++w) top = max(top, red[w]);
        const float want = exp2i(scale_exp(__int_as_float(top)));
        const float sc = fmaxf(want, old), inv = 1.f / sc;
        uint8_t* page = codes + (ph * a.page) * D;
        if (first > 0 && sc > old) rescale_codes(page, first * D, old * inv, tid, kStoreWarps * 32);
#pragma unroll
        for (int k = 0; k < IT; ++k) {
          const int c = tid + k * kStoreWarps * 32, row = c / CPR;
          if (row >= n) continue;
          float v[VPC];
          chunk_values<F32>(u[k], v);
          uint32_t code[VPC / 4];
#pragma unroll
          for (int q = 0; q < VPC / 4; ++q)
            code[q] = e4m3x2_code(v[4 * q] * inv, v[4 * q + 1] * inv) |
                      ((uint32_t)e4m3x2_code(v[4 * q + 2] * inv, v[4 * q + 3] * inv) << 16);
          uint8_t* dst = page + (int64_t)(first + row) * D + (c % CPR) * VPC;
          if constexpr (F32) *reinterpret_cast<uint32_t*>(dst) = code[0];
          else *reinterpret_cast<uint2*>(dst) = make_uint2(code[0], code[VPC / 4 - 1]);
        }
        if (tid == 0 && sc != old) scales[ph] = sc;
      }
    }
  }
  if (bad) bits |= LCSC_DEV_RANGE;
  if (bits && a.status) atomicOr(a.status, bits);
}

// ---------------------------------------------- attention, float32 queries
// Everything in float32 on the CUDA cores: 8 query rows against tiles of 64
// keys.  Scores: two threads per key, each the dot products of four rows;
// softmax: a warp for two rows; P V: a thread per dim (for D = 64 two, each
// half of the keys).  Codes come by cp.async, two tiles in flight, rows
// swizzled by 16-byte chunks so that 32 threads reading one chunk of 32
// rows touch all banks.

constexpr int kFmaRows = 8, kFmaKeys = 64, kFmaThreads = 128;

template <int D>
__global__ void __launch_bounds__(kFmaThreads) paged_fma_kernel(const __grid_constant__ PagedLaunch a) {
  grid_dep_wait();
  constexpr int M = kFmaRows, TK = kFmaKeys;
  constexpr int CH = D / 16;               // 16-byte chunks of a row
  constexpr int PARTS = kFmaThreads / D;   // key parts of P V
  __shared__ __align__(16) uint8_t kv_s[2][2][TK * D];  // stage, K / V
  __shared__ float sc_s[2][2][TK];                      // scales; K's is -1 where there is no key
  __shared__ __align__(16) float q_s[M][D];
  __shared__ float s_s[M][TK + 1];
  __shared__ __align__(16) float p_s[TK][M];
  __shared__ float al_s[M], m_s[M], l_s[M];
  __shared__ float o_s[PARTS > 1 ? D : 1][M];
  __shared__ int lo_s[M], hi_s[M], pos_s[M];
  __shared__ PagedScratch scan_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  PagedShare share;
  const PagedStart st = paged_start<M, TK>(a, &share, &scan_s);
  PagedWalk<M, TK> w(a, st, share);
  bool first = true;
  const float c2 = a.sm_scale * kPagedLog2e, cap2 = a.cap * kPagedLog2e;
  const bool bent = a.cap > 0.f || a.slopes;
  const float factor = bent ? 1.f : c2;  // from what s_s holds to base-2 units
  while (w.next()) {
    if (tid == 0 && first) w.write_meta(false);
    first = false;
    const int rows = w.rows(), r0 = w.p_mt * M;
    int item_lo, item_hi, x;
    paged_span(a, w.p_s, paged_prefix(a, w.p_b), paged_div(a, r0), &item_lo, &x);
    paged_span(a, w.p_s, paged_prefix(a, w.p_b), paged_div(a, r0 + rows - 1), &x, &item_hi);
    if ((a.docs || a.doc_ends) && w.p_s.L > 0) {  // pages outside every row's document are not looked at
      const int2 d = paged_docs(a, w.p_s, paged_div(a, r0), paged_div(a, r0 + rows - 1));
      item_lo = max(item_lo, d.x);
      item_hi = min(item_hi, d.y);
    }
    const int32_t* table = a.table + (int64_t)w.p_b * a.max_blocks;
    __syncthreads();  // the last piece is done with shared memory
    if (tid < M) {
      int lo = 0, hi = 0, pos = 0;
      if (tid < rows) {
        const int i = paged_div(a, r0 + tid);
        paged_row(a, w.p_s, paged_prefix(a, w.p_b), i, &lo, &hi);
        pos = w.p_s.L - w.p_s.n + i;
      }
      lo_s[tid] = lo, hi_s[tid] = hi, pos_s[tid] = pos;
      m_s[tid] = -INFINITY, l_s[tid] = 0.f;
    }
    for (int i = tid; i < M * D; i += kFmaThreads) {
      const int r = i / D, d = i % D;
      float v = 0.f;
      if (r < rows) {
        const int row = r0 + r, tok = paged_div(a, row);
        v = load_elem(a.q, (w.p_s.q0 + tok) * a.q_stride + (int64_t)(w.p_h * a.G + row - tok * a.G) * D + d, a.q_dtype);
      }
      q_s[r][d] = v;
    }
    auto page_of = [&](int key) -> int64_t {  // (page, head) index of a key's page, or -1 (no row sees the key)
      if (key >= item_hi || key < item_lo) return -1;
      const int32_t pg = table[key >> a.page_log2];
      if (pg < 0 || pg >= a.n_pages) {
        if (a.status) atomicOr(a.status, LCSC_DEV_BAD_INDEX);
        return -1;
      }
      return (int64_t)pg * a.Hkv + w.p_h;
    };
    auto load = [&](int t, int stage) {
      for (int u = tid; u < TK * CH; u += kFmaThreads) {
        const int r = u / CH, c = u % CH;
        const int key = t * TK + r;
        const int64_t ph = page_of(key);
        const int64_t off = ph < 0 ? 0 : (ph * a.page + (key & (a.page - 1))) * D + c * 16;
        const uint32_t dst = (uint32_t)(r * D + ((c ^ (r & (CH - 1))) * 16));
        const int n = ph < 0 ? 0 : 16;
        const uint32_t dk = (uint32_t)__cvta_generic_to_shared(&kv_s[stage][0][dst]);
        const uint32_t dv = (uint32_t)__cvta_generic_to_shared(&kv_s[stage][1][dst]);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dk), "l"(a.k + off), "r"(n) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dv), "l"(a.v + off), "r"(n) : "memory");
      }
      if (tid < TK) {
        const int64_t ph = page_of(t * TK + tid);
        sc_s[stage][0][tid] = ph < 0 ? -1.f : a.k_scale[ph];
        sc_s[stage][1][tid] = ph < 0 ? 0.f : a.v_scale[ph];
      }
    };
    load(w.p_t0, 0);
    asm volatile("cp.async.commit_group;" ::: "memory");
    float o[M];
#pragma unroll
    for (int r = 0; r < M; ++r) o[r] = 0.f;
    for (int t = w.p_t0; t < w.p_t1; ++t) {
      const int stage = (t - w.p_t0) & 1;
      if (t + 1 < w.p_t1) load(t + 1, stage ^ 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      {  // scores
        const int key = tid % TK, g = (tid / TK) * 4;
        float acc[4] = {};  // sums of the sums of 16 dims: a chain of all would round more
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const uint4 u = *reinterpret_cast<const uint4*>(&kv_s[stage][0][key * D + ((c ^ (key & (CH - 1))) * 16)]);
          const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
          float part[4][2] = {};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 k0 = e4m3x2_val((uint16_t)wd[i]), k1 = e4m3x2_val((uint16_t)(wd[i] >> 16));
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float4 q = *reinterpret_cast<const float4*>(&q_s[g + r][c * 16 + i * 4]);
              part[r][0] = fmaf(q.x, k0.x, fmaf(q.y, k0.y, part[r][0]));
              part[r][1] = fmaf(q.z, k1.x, fmaf(q.w, k1.y, part[r][1]));
            }
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[r] += part[r][0] + part[r][1];
        }
        // scores; where nothing bends them they stay without their constant
        // factor, which the exponential's argument takes in one rounding
        const float ks = sc_s[stage][0][key];
        const int j = t * TK + key;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float s = acc[r] * ks;
          if (bent) s *= c2;
          if (a.cap > 0.f) s = paged_cap(s, cap2);
          if (a.slopes && g + r < rows)
            s -= a.slopes[w.p_h * a.G + r0 + g + r - paged_div(a, r0 + g + r) * a.G] * (float)abs(pos_s[g + r] - j) * kPagedLog2e;
          s_s[g + r][key] = (ks >= 0.f && j >= lo_s[g + r] && j < hi_s[g + r]) ? s : -INFINITY;
        }
      }
      __syncthreads();
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {  // softmax of rows 2 warp, 2 warp + 1
        const int r = warp * 2 + rr;
        const float s0 = s_s[r][lane], s1 = s_s[r][lane + 32];
        const float m_old = m_s[r], m_new = fmaxf(m_old, warp_max(fmaxf(s0, s1)) * factor);
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        // (from 2^20 on a score is rounded as the maximum was: less its unrounded
        // self, it could pass the exponential's range)
        const bool big = fabsf(m_new) >= 0x1p20f;
        const float p0 = paged_ex2(big ? __fadd_rn(__fmul_rn(s0, factor), -ref) : fmaf(s0, factor, -ref));
        const float p1 = paged_ex2(big ? __fadd_rn(__fmul_rn(s1, factor), -ref) : fmaf(s1, factor, -ref));
        const float sum = warp_sum(p0 + p1);
        p_s[lane][r] = p0 * sc_s[stage][1][lane];
        p_s[lane + 32][r] = p1 * sc_s[stage][1][lane + 32];
        __syncwarp();
        if (lane == 0) {
          const float al = paged_ex2(m_old - ref);  // 0 before the first key
          al_s[r] = al;
          m_s[r] = m_new;
          l_s[r] = l_s[r] * al + sum;
        }
      }
      __syncthreads();
      {  // O = O alpha + P V
        const int d = tid % D, part = tid / D;
#pragma unroll
        for (int r = 0; r < M; ++r) o[r] *= al_s[r];
#pragma unroll 8
        for (int j = part * (TK / PARTS); j < (part + 1) * (TK / PARTS); ++j) {
          const float v = e4m3_val(kv_s[stage][1][j * D + (((d >> 4) ^ (j & (CH - 1))) * 16) + (d & 15)]);
          const float4 pa = *reinterpret_cast<const float4*>(&p_s[j][0]);
          const float4 pb = *reinterpret_cast<const float4*>(&p_s[j][4]);
          o[0] = fmaf(pa.x, v, o[0]), o[1] = fmaf(pa.y, v, o[1]), o[2] = fmaf(pa.z, v, o[2]), o[3] = fmaf(pa.w, v, o[3]);
          o[4] = fmaf(pb.x, v, o[4]), o[5] = fmaf(pb.y, v, o[5]), o[6] = fmaf(pb.z, v, o[6]), o[7] = fmaf(pb.w, v, o[7]);
        }
      }
      __syncthreads();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if constexpr (PARTS > 1) {
      if (tid >= D) {
#pragma unroll
        for (int r = 0; r < M; ++r) o_s[tid - D][r] = o[r];
      }
      __syncthreads();
      if (tid < D) {
#pragma unroll
        for (int r = 0; r < M; ++r) o[r] += o_s[tid][r];
      }
    }
    if (tid < D) {
      if (w.whole()) {
#pragma unroll
        for (int r = 0; r < M; ++r)
          if (r < rows) paged_write<D>(a, w.p_s, w.p_h, r0 + r, tid, o[r], m_s[r], l_s[r]);
      } else {
        const int64_t at = w.slot() * M;
#pragma unroll
        for (int r = 0; r < M; ++r) {
          a.part_o[(at + r) * D + tid] = o[r];
          if (tid == 0) a.part_ml[(at + r) * 2] = m_s[r], a.part_ml[(at + r) * 2 + 1] = l_s[r];
        }
      }
    }
  }
  if (first && tid == 0) w.write_meta(true);
}

// ---------------------------------------------------------- split items
// Joins the pieces of an item: O = sum_i 2^(m_i - m) O_i and the same for the
// sums.  The CTAs of the item's second piece do it.  A row is a warp's, or,
// where an item has few rows (and then often many pieces: one per CTA of the
// GPU for one long request), that of 2, 4 or 8 warps that share its pieces and
// join theirs in shared memory; which, follows from the item alone, so that the
// order of every sum is fixed.  A lane per piece for the maxima and sums, then 4
// (D = 64: 2) dims per lane over the pieces, four in flight.
constexpr int kCombineWarps = 8, kCombineY = 32;

template <int D>
__global__ void __launch_bounds__(kCombineWarps * 32) paged_combine_kernel(PagedLaunch a, int M) {
  grid_dep_wait();
  constexpr int VPL = D / 32;
  __shared__ float2 ml_s[kCombineWarps];
  __shared__ float o_s[kCombineWarps][D];
  const int c = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int32_t* m = a.meta + 8 * (int64_t)c;
  const int b = m[0], h = m[1], mt = m[2], c0 = m[3], c1 = m[4];
  if (b < 0 || c != c0 + 1) return;  // the same for the whole CTA
  const PagedSeq s = paged_seq(a, b);
  const int rows = min(M, s.n * a.G - mt * M);
  int per_cta = 1;  // rows of a CTA
  while (per_cta < kCombineWarps && per_cta * (int)gridDim.y < rows) per_cta *= 2;
  const int share = kCombineWarps / per_cta, sub = warp % share, r = blockIdx.y * per_cta + warp / share;
  float top = -INFINITY, l = 0.f, o[VPL] = {};
  if (r < rows) {
    // the place of the row in piece i (the first is its CTA's last)
    auto place = [&](int i) { return (2 * (int64_t)i + (i == c0 ? 1 : 0)) * M + r; };
    for (int i0 = c0 + sub; i0 <= c1; i0 += 32 * share) {  // 32 of this warp's pieces at a time
      const int mine = i0 + lane * share;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (mine <= c1) ml = *reinterpret_cast<const float2*>(a.part_ml + place(mine) * 2);
      const float high = fmaxf(top, warp_max(ml.x)), ref = high == -INFINITY ? 0.f : high;
      const float old = paged_ex2(top - ref), f = paged_ex2(ml.x - ref);
      top = high;
      l = fmaf(l, old, warp_sum(ml.y * f));
#pragma unroll
      for (int k = 0; k < VPL; ++k) o[k] *= old;
      const int n = min(32, ((c1 - i0) >> (31 - __clz(share))) + 1);  // share: a power of two
#pragma unroll 1
      for (int i = 0; i < n; i += 4) {  // four in flight, the last one again where there are fewer
        float v[4][VPL], fi[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int piece = min(i + q, n - 1);
          fi[q] = __shfl_sync(0xffffffffu, f, piece);
          const float* p = a.part_o + place(i0 + piece * share) * D + lane * VPL;
          if constexpr (VPL == 4) {
            const float4 u = *reinterpret_cast<const float4*>(p);
            v[q][0] = u.x, v[q][1] = u.y, v[q][2] = u.z, v[q][3] = u.w;
          } else {
            const float2 u = *reinterpret_cast<const float2*>(p);
            v[q][0] = u.x, v[q][1] = u.y;
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int k = 0; k < VPL; ++k) o[k] = i + q < n ? fmaf(fi[q], v[q][k], o[k]) : o[k];
      }
    }
  }
  if (share > 1) {
    if (lane == 0) ml_s[warp] = make_float2(top, l);
#pragma unroll
    for (int k = 0; k < VPL; ++k) o_s[warp][lane * VPL + k] = o[k];
    __syncthreads();
    if (sub != 0) return;
    float high = top;
    for (int i = 1; i < share; ++i) high = fmaxf(high, ml_s[warp + i].x);
    const float ref = high == -INFINITY ? 0.f : high, own = paged_ex2(top - ref);
    l *= own;
#pragma unroll
    for (int k = 0; k < VPL; ++k) o[k] *= own;
    for (int i = 1; i < share; ++i) {
      const float2 ml = ml_s[warp + i];
      const float f = paged_ex2(ml.x - ref);
      l = fmaf(ml.y, f, l);
#pragma unroll
      for (int k = 0; k < VPL; ++k) o[k] = fmaf(o_s[warp + i][lane * VPL + k], f, o[k]);
    }
    top = high;
  }
  if (r >= rows) return;
  int64_t at;
  const float f = paged_close(a, s, h, mt * M + r, top, l, lane == 0, &at);
#pragma unroll
  for (int k = 0; k < VPL; ++k) o[k] = f == 0.f ? 0.f : o[k] * f;
  at = at * D + lane * VPL;
#pragma unroll
  for (int k = 0; k < VPL; k += 2) {
    if (a.q_dtype == LCSC_DT_BF16)
      *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.out) + at + k) =
          (uint32_t)bf16_code(o[k]) | ((uint32_t)bf16_code(o[k + 1]) << 16);
    else
      *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out) + at + k) = make_float2(o[k], o[k + 1]);
  }
}

template <int D>
cudaError_t launch_fma(const PagedLaunch& a, cudaStream_t stream) {
  return launch_pdl(paged_fma_kernel<D>, dim3(a.ctas), dim3(kFmaThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanLaunch& a, cudaStream_t stream) {
  const bool here = a.n_tokens <= kFillHere;
  cudaError_t e = launch_pdl(page_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a, here);
  if (e != cudaSuccess || here) return e;
  const int64_t blocks = (a.n_tokens + 255) / 256, most = 8 * (int64_t)sm_count();
  return launch_pdl(page_fill_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, stream, a);
}

cudaError_t launch_paged_store(const PagedStoreLaunch& a, cudaStream_t stream) {
  // Tokens per CTA: 8 while that fills the GPU (a decode step's runs are one
  // row each, and one warp takes one), else 64, so that fewer CTAs look at rows
  // that others store.
  auto go = [&](auto kern, int tile) {
    return launch_pdl(kern, dim3((unsigned)((a.n_tokens + tile - 1) / tile), a.Hkv, 2), dim3(kStoreWarps * 32), 0, stream, a);
  };
  const int chunks = a.page * a.D * (a.x_dtype == LCSC_DT_F32 ? 4 : 2) / 16 / (kStoreWarps * 32);  // a thread's, of a page
  auto tile = [&](auto vpl, auto f32, auto it) {
    constexpr int V = decltype(vpl)::value, I = decltype(it)::value;
    constexpr bool F = decltype(f32)::value;
    return a.n_tokens <= 1024 ? go(paged_store_kernel<V, 8, F, I>, 8) : go(paged_store_kernel<V, 64, F, I>, 64);
  };
  auto depth = [&](auto vpl, auto f32) {
    return chunks <= 1   ? tile(vpl, f32, std::integral_constant<int, 1>())
           : chunks <= 4 ? tile(vpl, f32, std::integral_constant<int, 4>())
                         : tile(vpl, f32, std::integral_constant<int, 16>());
  };
  auto dtype = [&](auto vpl) {
    return a.x_dtype == LCSC_DT_F32 ? depth(vpl, std::true_type()) : depth(vpl, std::false_type());
  };
  return a.D == 128 ? dtype(std::integral_constant<int, 4>()) : dtype(std::integral_constant<int, 2>());
}

PagedForm paged_form(int q_dtype, int D, int G, int64_t max_new) {
  if (q_dtype == LCSC_DT_BF16) return paged_mma_form(D, G, max_new);
  return {0, kFmaRows, 4 * sm_count()};
}

cudaError_t launch_paged_attn(const PagedLaunch& a, const PagedForm& f, cudaStream_t stream) {
  cudaError_t e = f.kind ? launch_paged_mma(a, f, stream)
                  : a.D == 128 ? launch_fma<128>(a, stream) : launch_fma<64>(a, stream);
  if (e != cudaSuccess || a.ctas == 1) return e;
  const dim3 grid(a.ctas, f.rows / 4 < kCombineY ? f.rows / 4 : kCombineY), block(kCombineWarps * 32);
  return a.D == 128 ? launch_pdl(paged_combine_kernel<128>, grid, block, 0, stream, a, f.rows)
                    : launch_pdl(paged_combine_kernel<64>, grid, block, 0, stream, a, f.rows);
}

}  // namespace lcsc
