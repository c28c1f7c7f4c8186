// The paged 8-bit cache's attention: the launch's arguments, the rows and keys
// of a request, and the schedule that every form of the kernel walks.
//
// An item is (request, KV head, block of M query rows), a query row being one
// (new token, head of the group) pair, row = token * G + head in group.  An
// item's keys are cut into tiles of TK; a unit is one tile of one item.  All
// units of a call, in the order (request, head, row block, tile), are shared
// out evenly over the CTAs, CTA c taking the units [U c / C, U (c + 1) / C):
// lengths differ by orders of magnitude between the requests of a batch and are
// known on the device only, so an even split of tiles is the one that keeps
// every SM busy without the host knowing them.  A CTA's share is a run of
// pieces; a piece that covers its item whole writes the output, the others
// (at most two of a CTA: the one that ends an item begun by an earlier CTA, and
// the one that begins an item that goes on) leave (O, max, sum) in the
// workspace, which therefore does not grow with the lengths, and
// paged_combine_kernel joins them in CTA order.
#pragma once

#include "common.cuh"

namespace lcsc {

struct PagedLaunch {
  const void* q;
  int64_t q_stride;  // values from one token's row to the next
  int q_dtype;
  int Hq, Hkv, G, D;
  uint32_t g_mul;    // x / G = x * g_mul >> g_shift for 0 <= x < 2^31 (paged_divisor)
  int g_shift;
  int page, page_log2;
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int64_t n_pages;
  int B;
  int64_t n_tokens, max_blocks;
  const int32_t* q_start;
  const int32_t* ctx_len;
  const int32_t* table;
  const float* slopes;
  const float* sink;
  const int32_t* prefix;
  const int32_t* docs;
  const int32_t* doc_ends;
  float sm_scale, cap;
  int window;
  void* out;
  float* lse;
  int32_t* status;
  // workspace: of CTA c the unfinished pieces 2c (ends an item begun before)
  // and 2c + 1 (begins an item that goes on), and what its piece 2c belongs to
  float* part_o;   // [2 * ctas][rows per item][D], not normalised
  float* part_ml;  // [2 * ctas][rows per item][2]: max (base-2 units), sum
  int32_t* meta;   // [ctas][8]
  int ctas;
  // many rows: the earliest document start and the latest document end in a block
  // of rows (paged_block), or null
  int2* block_docs;  // [n_tokens * G / 256 + B]
};

struct PagedStoreLaunch {
  uint8_t* codes[2];  // K, V
  float* scale[2];
  const void* x[2];
  int64_t stride[2];
  int x_dtype, Hkv, D, page, page_log2;
  int64_t n_pages, n_tokens;
  const int32_t* slots;
  int32_t* status;
};

struct PagePlanLaunch {
  int page, page_log2, B;
  int64_t n_tokens, max_blocks, n_pages;
  const int32_t *cached, *n_new;
  int32_t *table, *free_pages;
  const int32_t* n_free;
  int32_t *n_free_out, *ctx_len, *q_start, *slots, *positions;
  int64_t* scratch;  // [2 + B]: stack height after the returns, unused, pages taken by earlier requests
  int32_t* status;
};

cudaError_t launch_page_plan(const PagePlanLaunch& a, cudaStream_t stream);
cudaError_t launch_paged_store(const PagedStoreLaunch& a, cudaStream_t stream);

// The form of the attention kernel that serves a call (from the host's
// arguments alone), its rows per item and the CTAs it launches.
struct PagedForm {
  int kind;  // 0: float32 on the CUDA cores, 1: few rows on the tensor cores, 2: many
  int rows;
  int ctas;
};
PagedForm paged_form(int q_dtype, int D, int G, int64_t max_new);
cudaError_t launch_paged_attn(const PagedLaunch& a, const PagedForm& f, cudaStream_t stream);
// The tensor-core forms (paged_mma.cu).
PagedForm paged_mma_form(int D, int G, int64_t max_new);
cudaError_t launch_paged_mma(const PagedLaunch& a, const PagedForm& f, cudaStream_t stream);

// Multiplier and shift of a division by d >= 1: with 2^(l-1) < d <= 2^l,
// m = floor(2^(31+l) / d) + 1 = (2^(31+l) + e) / d, 0 < e <= d <= 2^l, so that
// x m / 2^(31+l) = x / d + x e / (d 2^(31+l)) and the excess is below 1 / d for
// x < 2^31.  m < 2^32 for d > 1; d = 1 takes m = 2^31, shift 31.
inline void paged_divisor(int d, uint32_t* mul, int* shift) {
  int l = 0;
  while ((1 << l) < d) ++l;
  *shift = 31 + l;
  *mul = d == (1 << l) ? 1u << 31 : (uint32_t)(((uint64_t)1 << (31 + l)) / d + 1);
}

// A table ends this many positions before 2^31: the kernels compute positions in
// 32 bits, some of them behind the last tile (each says how far).
constexpr int kPagedAhead = 4096;

#ifdef __CUDACC__

__device__ __forceinline__ int paged_div(const PagedLaunch& a, int x) {
  return (int)(((uint64_t)(uint32_t)x * a.g_mul) >> a.g_shift);
}

constexpr float kPagedLog2e = 1.4426950408889634f;
constexpr float kPagedLn2 = 0.6931471805599453f;

// 2^x on the MUFU unit.
__device__ __forceinline__ float paged_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr int kPagedManyRows = 256;  // rows of a block of the many-rows kernel

struct PagedSeq {
  int64_t q0;  // first row
  int b;       // the request
  int n;       // rows' tokens (0: nothing to write)
  int L;       // length; 0: its rows get zeros
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedLaunch& a, int b) {
  PagedSeq s;
  const int32_t q0 = a.q_start[b], q1 = a.q_start[b + 1];
  int32_t L = a.ctx_len[b];
  const bool rows_ok = q0 >= 0 && q1 >= q0 && q1 <= a.n_tokens;
  const int n = rows_ok ? q1 - q0 : 0;
  const bool len_ok = L == 0 || (L >= n && L <= a.max_blocks * a.page);
  s.q0 = q0;
  s.b = b;
  s.n = n;
  s.L = len_ok ? L : 0;
  if ((!rows_ok || !len_ok) && a.status) atomicOr(a.status, LCSC_DEV_BAD_LENGTH);
  return s;
}

// Visible positions [lo, hi) of token i of a request, its document apart
// (paged_row has that too).
__device__ __forceinline__ void paged_span(const PagedLaunch& a, const PagedSeq& s, int prefix, int i, int* lo,
                                           int* hi) {
  if (s.L == 0) {
    *lo = *hi = 0;
    return;
  }
  const int p = s.L - s.n + i;
  *hi = min(s.L, max(p + 1, prefix));
  *lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
}

__device__ __forceinline__ void paged_row(const PagedLaunch& a, const PagedSeq& s, int prefix, int i, int* lo, int* hi) {
  paged_span(a, s, prefix, i, lo, hi);
  if (a.docs) *lo = max(*lo, a.docs[s.q0 + i]);
  if (a.doc_ends) *hi = min(*hi, max(0, a.doc_ends[s.q0 + i]));  // (differences from it stay in 32 bits)
}

// The earliest document start and the latest document end of the tokens i0 .. i1
// (a whole warp computes them; out of line: every role of a kernel asks for them,
// and five draft tokens without documents took 173 us with it in line, 167 so).
static __device__ __noinline__ int2 paged_docs(const PagedLaunch& a, const PagedSeq& s, int i0, int i1) {
  int first = 0, last = INT_MAX;
  if (a.docs) {
    first = INT_MAX;
    for (int i = i0 + (threadIdx.x & 31); i <= i1; i += 32) first = min(first, a.docs[s.q0 + i]);
    first = __reduce_min_sync(0xffffffffu, first);
  }
  if (a.doc_ends) {
    last = 0;
    for (int i = i0 + (threadIdx.x & 31); i <= i1; i += 32) last = max(last, a.doc_ends[s.q0 + i]);
    last = __reduce_max_sync(0xffffffffu, last);
  }
  return make_int2(first, last);
}

__device__ __forceinline__ int paged_prefix(const PagedLaunch& a, int b) { return a.prefix ? a.prefix[b] : 0; }

// Number of a request's block mt among all: the requests' rows follow one
// another, and floor(x) + ceil(y) - 1 <= floor(x + y) keeps their blocks apart.
__device__ __forceinline__ int64_t paged_block(const PagedLaunch& a, const PagedSeq& s, int mt) {
  return s.q0 * a.G / kPagedManyRows + s.b + mt;
}

// Tiles [t0, t1) of keys that the row block mt of M rows may see; at least one.
template <int M, int TK>
__device__ __forceinline__ void paged_tiles(const PagedLaunch& a, const PagedSeq& s, int prefix, int mt, int* t0,
                                            int* t1) {
  const int rows = s.n * a.G;
  int lo, hi, x;
  paged_span(a, s, prefix, paged_div(a, mt * M), &lo, &x);
  paged_span(a, s, prefix, paged_div(a, min(rows, (mt + 1) * M) - 1), &x, &hi);
  if constexpr (M == kPagedManyRows) {
    // An item's units are the tiles that its documents leave (packed documents
    // under a prefix, 5 requests of 11 to 3001 tokens: 14% less time).
    if (a.block_docs && s.L > 0) {
      const int2 d = a.block_docs[paged_block(a, s, mt)];
      lo = min(max(lo, d.x), hi - 1);
      hi = max(min(hi, d.y), lo + 1);
    }
  }
  *t0 = lo / TK;
  *t1 = max(*t0 + 1, (hi + TK - 1) / TK);
}

template <int M, int TK>
__device__ __forceinline__ int paged_tile_count(const PagedLaunch& a, const PagedSeq& s, int prefix, int mt) {
  if ((int64_t)mt * M >= (int64_t)s.n * a.G) return 0;
  int t0, t1;
  paged_tiles<M, TK>(a, s, prefix, mt, &t0, &t1);
  return t1 - t0;
}

__device__ __forceinline__ int64_t paged_warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Quotient of two numbers that fit 32 bits nearly always (a 64-bit division is a
// long piece of code, and code that runs once is paid for in instruction fetches).
__device__ __forceinline__ int64_t paged_quot(int64_t x, int64_t y) {
  if (((x | y) >> 32) == 0) return (int64_t)((uint32_t)x / (uint32_t)y);
  return x / y;
}

// Units of a head of request b, one request per lane (a.B: none): those of few
// row blocks by their lane, the others by the warp together.
template <int M, int TK>
__device__ __forceinline__ int64_t paged_units(const PagedLaunch& a, int b) {
  PagedSeq s = {0, 0, 0, 0};
  if (b < a.B) s = paged_seq(a, b);
  const int prefix = b < a.B ? paged_prefix(a, b) : 0;
  const bool few = (int64_t)s.n * a.G <= 4 * M;
  int64_t u = 0;
  if (few) {
#pragma unroll 1
    for (int mt = 0; mt < 4; ++mt) u += paged_tile_count<M, TK>(a, s, prefix, mt);
  }
#pragma unroll 1
  for (unsigned todo = __ballot_sync(0xffffffffu, !few); todo; todo &= todo - 1) {
    const int src = __ffs(todo) - 1, bs = __shfl_sync(0xffffffffu, b, src);
    const PagedSeq t = paged_seq(a, bs);
    const int pre = paged_prefix(a, bs);
    int64_t sum = 0;
#pragma unroll 1
    for (int mt = threadIdx.x & 31; (int64_t)mt * M < (int64_t)t.n * a.G; mt += 32)
      sum += paged_tile_count<M, TK>(a, t, pre, mt);
    sum = paged_warp_sum(sum);
    if ((int)(threadIdx.x & 31) == src) u = sum;
  }
  return u;
}

// The units' shares of the CTAs that have work: the first total % ctas have one more.
struct PagedShare {
  int64_t total, each;  // units of the call, units of a CTA (the fewer)
  int ctas, more;       // CTAs with work, CTAs with one unit more
  __device__ __forceinline__ int64_t begin(int c) const { return c * each + min(c, more); }
  __device__ __forceinline__ int owner(int64_t u) const {
    const int64_t high = (each + 1) * more;
    return u < high ? (int)paged_quot(u, each + 1) : more + (int)paged_quot(u - high, each);
  }
};

// Where a CTA's share begins: found once by the whole CTA.
struct PagedStart {
  int b, h, mt, t;  // b = -1: no share
};
struct PagedScratch {
  int64_t scan[33];         // sums of the warps; [32]: of the CTA
  int64_t first, per_head;  // units before the found request, and of one of its heads
  PagedStart st;
};

// Every thread of the CTA calls it.
template <int M, int TK>
__device__ __forceinline__ PagedStart paged_start(const PagedLaunch& a, PagedShare* share, PagedScratch* x) {
  const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = nthr >> 5;
  if (tid == 0) x->st.b = -1;
  int64_t u0 = 0, u = 0;
  // first for the sum over all requests, then for the one the share begins in
#pragma unroll 1
  for (int find = 0; find < 2; ++find) {
    int64_t base = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += nthr) {
      const int b = b0 + tid;
      if (!find || a.B > nthr) u = paged_units<M, TK>(a, b < a.B ? b : a.B);
      int64_t upto = u * a.Hkv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      __syncthreads();
      if (lane == 31) x->scan[warp] = upto;
      __syncthreads();
      int64_t all = 0;
#pragma unroll 1
      for (int i = 0; i < warps; ++i) {
        const int64_t y = x->scan[i];
        if (i < warp) upto += y;
        all += y;
      }
      upto += base;
      if (find && upto - u * a.Hkv <= u0 && u0 < upto) {  // one thread at most
        x->st.b = b;
        x->first = upto - u * a.Hkv;
        x->per_head = u;
      }
      base += all;
      if (find && base > u0) break;  // the same for the whole CTA
    }
    if (!find) {
      // At least two tiles for a CTA of few rows (decode of 16 requests with a
      // window of 128: 19.7 against 23.4 us with one, 28.1 with three), one of
      // many rows (a prompt of 400 tokens: 42.6 against 55.6 us with two).
      constexpr int kLeast = M > 64 ? 1 : 2;
      share->total = base;
      share->ctas = (int)min((int64_t)gridDim.x, (base + kLeast - 1) / kLeast);
      if ((int)blockIdx.x >= share->ctas) break;  // the same for the whole CTA
      share->each = paged_quot(base, share->ctas);
      share->more = (int)(base - share->each * share->ctas);
      u0 = share->begin(blockIdx.x);
    }
  }
  __syncthreads();
  if (warp == 0 && x->st.b >= 0) {  // the head, row block and tile
    const int b = x->st.b;
    const PagedSeq s = paged_seq(a, b);
    const int prefix = paged_prefix(a, b);
    int64_t off = u0 - x->first;
    const int h = (int)paged_quot(off, x->per_head);
    off -= h * x->per_head;
#pragma unroll 1
    for (int m0 = 0;; m0 += 32) {
      const int c = paged_tile_count<M, TK>(a, s, prefix, m0 + lane);
      int64_t upto = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const bool here = upto - c <= off && off < upto;
      if (here) {
        int t0, t1;
        paged_tiles<M, TK>(a, s, prefix, m0 + lane, &t0, &t1);
        x->st.h = h;
        x->st.mt = m0 + lane;
        x->st.t = t0 + (int)(off - (upto - c));
      }
      if (__any_sync(0xffffffffu, here)) break;
      off -= __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  __syncthreads();
  return x->st;
}

// The pieces of a CTA's share, one after another.  Every thread that walks
// them computes the same ones.
template <int M, int TK>
struct PagedWalk {
  const PagedLaunch& a;
  PagedShare share;
  int64_t left;  // units still to come
  int64_t unit;  // of the call: the next one
  int b, h, mt, t;
  PagedSeq s;
  int prefix;
  // the piece
  int p_b, p_h, p_mt, p_t0, p_t1;
  PagedSeq p_s;
  bool p_head, p_tail;  // it begins / ends its item
  int64_t p_item0, p_item1;  // units of the call of its item

  __device__ __forceinline__ PagedWalk(const PagedLaunch& a_, const PagedStart& st, const PagedShare& sh)
      : a(a_), share(sh), left(0), b(st.b), h(st.h), mt(st.mt), t(st.t) {
    if (b < 0) return;
    unit = share.begin(blockIdx.x);
    left = share.begin(blockIdx.x + 1) - unit;
    s = paged_seq(a, b);
    prefix = paged_prefix(a, b);
  }

  // Not inlined, so that the walk lies in local memory between pieces and its
  // state takes no registers from the tile loops.
  __device__ __noinline__ bool next() {
    if (left <= 0) return false;
    int t0, t1;
    paged_tiles<M, TK>(a, s, prefix, mt, &t0, &t1);
    p_b = b;
    p_h = h;
    p_mt = mt;
    p_s = s;
    p_t0 = t;
    p_t1 = (int)min((int64_t)t1, t + left);
    p_head = t == t0;
    p_tail = p_t1 == t1;
    p_item0 = unit - (t - t0);
    p_item1 = p_item0 + (t1 - t0);
    left -= p_t1 - t;
    unit += p_t1 - t;
    t = p_t1;
    if (p_tail && left > 0) {
      if ((mt + 1) * M < s.n * a.G) {
        ++mt;
      } else {
        mt = 0;
        if (++h == a.Hkv) {
          h = 0;
          do {
            s = paged_seq(a, ++b);
          } while (s.n == 0);
          prefix = paged_prefix(a, b);
        }
      }
      paged_tiles<M, TK>(a, s, prefix, mt, &t, &t1);
    }
    return true;
  }

  __device__ __forceinline__ bool whole() const { return p_head && p_tail; }
  // Where an unfinished piece goes.
  __device__ __forceinline__ int64_t slot() const { return 2 * (int64_t)blockIdx.x + (p_head ? 1 : 0); }
  __device__ __forceinline__ int rows() const { return min(M, p_s.n * a.G - p_mt * M); }

  // What the CTA's piece 2c belongs to, for paged_combine_kernel (one thread,
  // once the CTA's first piece is known; none: no such piece).
  __device__ __forceinline__ void write_meta(bool none) const {
    int32_t* m = a.meta + 8 * (int64_t)blockIdx.x;
    if (none || p_head) {
      m[0] = -1;
      return;
    }
    m[0] = p_b;
    m[1] = p_h;
    m[2] = p_mt;
    m[3] = share.owner(p_item0);
    m[4] = share.owner(p_item1 - 1);
  }
};

// tanh(y) / y on [-1, 1] as a polynomial in y^2, fitted to equal relative error
// (1.7e-7 in float32).
__device__ __forceinline__ constexpr float paged_tanh(int k) {
  constexpr float c[7] = {0.99999994f,   -0.333328396f,  0.13325204f,  -0.0534570217f,
                          0.0202899612f, -0.00620336272f, 0.00104101724f};
  return c[k];
}

// c tanh(x / c) by 1 - 2 / (e^(2x/c) + 1): off by about 1e-7 c.
__device__ __forceinline__ float paged_cap_far(float x, float c) {
  const float e = paged_ex2(x * (2.f * kPagedLog2e / c));
  return c - __fdividef(2.f * c, e + 1.f);
}

// c tanh(x / c): x times the polynomial while |x| <= c.
__device__ __forceinline__ float paged_cap(float x, float c) {
  const float y = x * (1.f / c), z = y * y;
  float p = paged_tanh(6);
#pragma unroll
  for (int k = 5; k >= 0; --k) p = fmaf(p, z, paged_tanh(k));
  return fabsf(y) <= 1.f ? x * p : paged_cap_far(x, c);
}

// What a finished row's sum O of the weights' products is multiplied by, from
// their max (base-2 units) and sum; the row's place in out and lse, which is
// written by the one thread that says so.  row = token * G + head in group.
__device__ __forceinline__ float paged_close(const PagedLaunch& a, const PagedSeq& s, int h, int row, float top,
                                             float l, bool write_lse, int64_t* at) {
  const int i = paged_div(a, row), head = h * a.G + row - i * a.G;
  *at = (s.q0 + i) * a.Hq + head;
  float f = 1.f, top_e = top * kPagedLn2;
  if (a.sink && s.L > 0) {
    const float sink = a.sink[head];
    float sg = sink * kPagedLog2e;  // finite where the sink is: the type's largest numbers pass it here
    if (fabsf(sg) > 3.402823466e38f && sink != -INFINITY) sg = copysignf(3.402823466e38f, sg);
    const float m = fmaxf(top, sg);
    if (m != -INFINITY) {
      f = paged_ex2(top - m);  // top -inf: 0
      l = fmaf(l, f, paged_ex2(sg - m));
      if (sg >= top) top_e = sink;
    }
  }
  if (write_lse && a.lse) a.lse[*at] = l == 0.f ? -INFINITY : fmaf(log2f(l), kPagedLn2, top_e);
  return l == 0.f ? 0.f : f / l;  // a sum that is no number stays one
}

template <int D>
__device__ __forceinline__ void paged_write(const PagedLaunch& a, const PagedSeq& s, int h, int row, int d, float o,
                                            float top, float l) {
  int64_t at;
  const float f = paged_close(a, s, h, row, top, l, d == 0, &at), r = f == 0.f ? 0.f : o * f;
  if (a.q_dtype == LCSC_DT_BF16) reinterpret_cast<uint16_t*>(a.out)[at * D + d] = bf16_code(r);
  else reinterpret_cast<float*>(a.out)[at * D + d] = r;
}

#endif

}  // namespace lcsc
