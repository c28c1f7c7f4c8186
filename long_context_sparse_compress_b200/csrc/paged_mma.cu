// Attention over the paged 8-bit cache on the 5th-generation tensor cores, for
// BF16 queries.  The schedule (items, units, pieces) is paged.cuh's.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kernels.cuh"
#include "launches.h"
#include "paged.cuh"
#include "sm100.cuh"

namespace lcsc {

using namespace sm100;

namespace {

// 32 lanes x N consecutive 32-bit columns of this warp's sub-partition.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld_32(taddr, r); }

// Store counterpart of tmem_ld_32.
__device__ __forceinline__ void tmem_st_32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]));
}

// Waits for this thread's tcgen05.ld with the registers passed through, so
// that no use of them moves before the wait.
template <int N>
__device__ __forceinline__ void tmem_ld_done(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Byte offset of (row, byte) in a swizzled block of rows of W bytes (W = 64:
// 64-byte swizzle, W = 128: 128-byte swizzle).
template <int W>
__device__ __forceinline__ uint32_t swz(int row, int byte) {
  if constexpr (W == 128) return (uint32_t)(row * 128 + ((((byte >> 4) ^ (row & 7)) << 4) | (byte & 15)));
  else return (uint32_t)(row * 64 + ((((byte >> 4) ^ ((row >> 1) & 3)) << 4) | (byte & 15)));
}
template <int W>
constexpr Swizzle kSwOf = W == 128 ? kSw128 : kSw64;

// 16-byte store to shared memory (the pointers of a swizzled buffer lose their
// address space on the way, and a generic store costs more).
__device__ __forceinline__ void st_shared16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ void st_shared8(uint32_t at, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(x), "r"(y) : "memory");
}

// Two float32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(x), "l"(y), "l"(z));
  return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(x), "l"(y));
  return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(x), "l"(y));
  return v;
}

// 2^e, e clamped to the normal range.
__device__ __forceinline__ float pow2(int e) {
  e = e < -126 ? -126 : (e > 127 ? 127 : e);
  return __int_as_float((e + 127) << 23);
}

// x 2^e for |e| up to 252 by two factors: 2^e itself need not be a number, or a normal one.
__device__ __forceinline__ float times_pow2(float x, int e) { return x * pow2(e / 2) * pow2(e - e / 2); }

__device__ __forceinline__ float warp_redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// True for one thread of a converged warp.  The compiler knows a branch on it as
// one thread's, and keeps the operands of tcgen05 instructions inside in
// uniform registers; under `lane == 0` it moves each there, which made an MMA
// cost about 110 cycles to issue.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Barrier `id` over n threads; true for all of them if `ok` is true for all.
__device__ __forceinline__ bool named_and(int id, int n, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

// mbar_wait that sleeps between polls, 16 of them between two looks at the
// clock: a polling warp takes issue slots and instruction fetches from the
// softmax warps of its scheduler.
__device__ __forceinline__ bool wait_asleep(uint64_t* bar, uint32_t parity, uint32_t ns, int32_t* status,
                                            uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      __nanosleep(ns);
      if (mbar_try_wait(bar, parity)) return true;
    }
    if (global_timer_ns() - t0 > limit_ns) {
      if (status) atomicOr(status, LCSC_DEV_TIMEOUT);
      return false;
    }
  }
}

// Bounded wait of a whole warp; false for every lane if one gave up or the CTA
// has.  What comes behind the first look at the barrier is out of line (chunk of
// 4096 tokens: 1,059 us with it in line, 1,036 so).
struct Waits {
  int32_t* status;
  uint64_t limit_ns;
  volatile int* abort;
  uint32_t ns;  // of sleep between polls
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    if (__all_sync(0xffffffffu, !*abort && mbar_try_wait(bar, parity))) return true;
    return longer(bar, parity, ns, status, limit_ns, abort);
  }
  static __device__ __noinline__ bool longer(uint64_t* bar, uint32_t parity, uint32_t ns, int32_t* status,
                                             uint64_t limit_ns, volatile int* abort) {
    // (one vote, as lanes apart could read the flag before and after it is set)
    if (__any_sync(0xffffffffu, *abort)) return false;
    const bool ok = __all_sync(0xffffffffu, wait_asleep(bar, parity, ns, status, limit_ns));
    if (!ok && (threadIdx.x & 31) == 0) *abort = 1;
    return ok;
  }
};

// First and past the last position that any row of a piece sees (a whole warp
// computes it), and the tiles [t0, t1) of the piece that hold them, maybe none.
template <int M, int TK>
struct PieceKeys {
  int lo, hi, t0, t1;
  __device__ __forceinline__ PieceKeys(const PagedLaunch& a, const PagedWalk<M, TK>& w) {
    const int prefix = paged_prefix(a, w.p_b), r0 = w.p_mt * M, r1 = r0 + w.rows() - 1;
    const int i0 = paged_div(a, r0), i1 = paged_div(a, r1);
    int x;
    paged_span(a, w.p_s, prefix, i0, &lo, &x);
    paged_span(a, w.p_s, prefix, i1, &x, &hi);
    if ((a.docs || a.doc_ends) && w.p_s.L > 0) {
      const int2 d = paged_docs(a, w.p_s, i0, i1);
      lo = max(lo, d.x);
      hi = min(hi, d.y);
    }
    t1 = min(w.p_t1, (hi + TK - 1) / TK);
    t0 = lo < hi ? min(t1, max(w.p_t0, lo / TK)) : t1;
  }
};

// Loads under a condition whose results nothing looks at before they are used
// (a select behind the load would wait for it).
__device__ __forceinline__ int32_t ld_if(const int32_t* p, bool cond, int32_t other) {
  int32_t v;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.b32 %0, %3;\n\t@p ld.global.b32 %0, [%1];\n\t}"
               : "=&r"(v)
               : "l"(p), "r"((uint32_t)cond), "r"(other));
  return v;
}
__device__ __forceinline__ float ld_if(const float* p, bool cond, float other) {
  return __int_as_float(ld_if(reinterpret_cast<const int32_t*>(p), cond, __float_as_int(other)));
}
__device__ __forceinline__ uint4 ld_if(const uint8_t* p, bool cond) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
      "mov.b32 %3, 0;\n\t@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((uint32_t)cond));
  return v;
}

// Page lookups run ahead of their use: the table's entry is loaded a tile before
// the page's scale or codes are asked for, and nothing looks at a loaded value
// before the next tile, so that no load is waited for.
template <int M, int TK>
struct PageAhead {
  const PagedLaunch& a;
  const int32_t* table;
  int lo, hi, end, h;  // keys looked at, and the tile the piece ends before
  __device__ __forceinline__ PageAhead(const PagedLaunch& a_, const PagedWalk<M, TK>& w, const PieceKeys<M, TK>& k)
      : a(a_), table(a_.table + (int64_t)w.p_b * a_.max_blocks), lo(k.lo), hi(k.hi), end(k.t1), h(w.p_h) {}
  // Table entry of key j of tile t (-1: no page of this piece).
  __device__ __forceinline__ int32_t entry(int t, int j) const {
    return ld_if(table + (j >> a.page_log2), t < end && j < hi && (j | (a.page - 1)) >= lo, -1);
  }
  // Its (page, head), or -1.
  __device__ __forceinline__ int64_t place(int32_t e) const {
    return e >= 0 && e < a.n_pages ? (int64_t)e * a.Hkv + h : -1;
  }
};

// =============================================================== few rows
// Decode steps and draft tokens: up to 16 query rows per item.  The keys lie on
// the M side of both products, so that a tile of 128 keys is one full-height MMA
// however few the rows are, and K and V go from TMA straight into the tensor
// cores as they are stored:
//   S^T [128 keys][rows] = K Q^T      K: A operand, K-major
//   O^T [D dims][rows]   = V^T P^T    V: A operand, M-major (the same bytes)
// Q and P, which are not stored values, are sums of E4M3 terms: two of the BF16
// query (times a power of two per row that brings its largest value into
// [128, 256)), three of the weights (11 bits).  One accumulating MMA chain per
// term.  A softmax thread owns one key: maxima go over a warp with redux and
// over the warps through shared memory.  Each tile's weights are taken against
// the tile's own maxima, and its O is read back and added to the running one in
// registers (a thread per dim), which is where rescaling happens: rows x 1
// FMA per thread and tile instead of a read-modify-write of TMEM.
// V's page scales go into the weights: a key's E4M3 terms hold e^x times its
// page's scale, from 2^8 down to steps of 2^-9.  They are taken relative to the
// tile's largest scale, in one multiplication, where no scale of the tile is
// below a quarter of it, and else relative to the row's own largest product of
// weight and scale, for which the maxima are taken again with the scales'
// exponents added.  So a row's largest product is at least 2^6, and each is off by
// half a step of f16 (2^-11 of it) and of the third term (2^-12 of it, or 2^-10,
// which is 2^-16 of the largest), whatever scales the tile's other pages have.
//
// Bound: HBM (2 D bytes per key and KV head).  Per tile the tensor pipe reads
// 5 x 16 KB of operands (640 cycles of shared memory at D = 128 against 1,420
// cycles of HBM time); two CTAs per SM overlap one's softmax with the other's
// copies and products.  16 requests of 16K to 64K tokens, 64 heads on 8, D = 128:
// 217 us, 5.4 TB/s, 84% of the measured copy rate.

constexpr int kFewThreads = 192;  // warps 0-3 softmax, 4 copies, 5 MMA
constexpr int kQTerms = 2, kPTerms = 3;

template <int D, int NR>
struct FewCfg {
  static constexpr int TK = 128;
  static constexpr int N = 16;                       // MMA columns (a multiple of 16)
  static constexpr int PW = 64;                      // bytes of a key's weights: 3 terms of N
  static constexpr int kTile = TK * D;               // K or V bytes of a tile
  static constexpr int kStages = 3;
  static constexpr int kPerSm = 2;
  static constexpr int kCols = 64;                   // TMEM columns: S twice, O
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + kStages * kTile;
  static constexpr int OFF_Q = OFF_V + kStages * kTile;
  static constexpr int kQBytes = N * D;              // one term
  static constexpr int OFF_P = OFF_Q + kQTerms * kQBytes;
  static constexpr int OFF_BAR = OFF_P + TK * PW;
  static constexpr int kBars = 2 * kStages + 6;
  static constexpr int OFF_F4 = OFF_BAR + kBars * 8;  // float4 [NR]: tile max, alpha, beta of the sums
  static constexpr int OFF_F2 = OFF_F4 + NR * 16;     // float2 [NR]: alpha, beta of O
  static constexpr int OFF_ROW = OFF_F2 + NR * 8;     // int4 [NR]: lo, hi, position, slope (float)
  static constexpr int OFF_QS = OFF_ROW + NR * 16;    // float [NR]: 2^e of the query row
  static constexpr int OFF_RED = OFF_QS + NR * 4;     // float [4][NR]
  static constexpr int OFF_VEND = OFF_RED + 4 * NR * 4;  // int [8]: V scales of the tile's 16-key groups, as bits
  static constexpr int OFF_M = OFF_VEND + 32;         // float [NR]
  static constexpr int OFF_SCAN = OFF_M + NR * 4;     // PagedScratch
  static constexpr int OFF_TM = OFF_SCAN + (int)sizeof(PagedScratch);
  static constexpr int OFF_ABORT = OFF_TM + 4;
  static constexpr int SMEM = OFF_ABORT + 4 + 1024;
  static_assert(kBars % 2 == 0 && OFF_F4 % 16 == 0 && OFF_F2 % 8 == 0 && OFF_ROW % 16 == 0 && OFF_VEND % 16 == 0 && OFF_SCAN % 8 == 0, "alignment");
  static_assert(OFF_Q % 1024 == 0 && OFF_P % 1024 == 0 && kQBytes % 1024 == 0, "swizzle atoms");
  static_assert(kPerSm * (SMEM + 1024) <= 228 * 1024, "resident CTAs");
  static_assert(NR <= N && kPTerms * N <= PW && 3 * N <= kCols, "a key's weights, the accumulators");
};

// A key's weights as E4M3 terms: term i of row r at byte i N + r of the key's row.
template <int NR>
__device__ __forceinline__ void few_codes(const float (&p)[NR], uint32_t prow) {
  constexpr int N = 16, PW = 64;
  static_assert(FewCfg<128, NR>::N == N && FewCfg<128, NR>::PW == PW, "the weights' layout");
  uint32_t code[kPTerms][4] = {};
#pragma unroll
  for (int r = 0; r < NR; r += 2) {
    __half2 x = __floats2half2_rn(p[r], p[r + 1]);
#pragma unroll
    for (int term = 0; term < kPTerms; ++term) {
      const uint32_t c8 = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(x), __NV_SATFINITE, __NV_E4M3);
      code[term][r / 4] |= c8 << (8 * (r % 4));
      if (term + 1 < kPTerms) x = __hsub2(x, __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c8, __NV_E4M3)));
    }
  }
#pragma unroll
  for (int term = 0; term < kPTerms; ++term)
    st_shared16(prow + swz<PW>(threadIdx.x, term * N), code[term][0], code[term][1], code[term][2], code[term][3]);
}

// The weights of a tile whose V scales lie far apart, in the place of those
// that are there: scores with the exponent of the key's scale added, and weights
// relative to the row's largest of these (a thread per key; out of line, so that
// the loop's code stays together).
template <int NR>
__device__ __noinline__ void few_far(const float (&s)[NR], float vs, float m_run, float* red_s, float2* f2_s,
                                     uint32_t prow) {
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int e = max(__float_as_int(vs) >> 23, 1) - 127;
  const float vr = vs * pow2(-e) * 224.f;
  float mine = -INFINITY, p[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const float top = warp_redux_max(s[r] + (float)e);
    if (lane == r) mine = top;
  }
  if (lane < NR) red_s[warp * NR + lane] = mine;
  named_sync(1, 128);
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const float top = fmaxf(fmaxf(red_s[r], red_s[NR + r]), fmaxf(red_s[2 * NR + r], red_s[3 * NR + r]));
    p[r] = paged_ex2(s[r] + (float)e - (top == -INFINITY ? 0.f : top)) * vr;
    if (tid == r) f2_s[r].y = paged_ex2(top - (m_run == -INFINITY ? 0.f : m_run)) * (1.f / 224.f);
  }
  few_codes<NR>(p, prow);
  named_sync(1, 128);  // red_s is read
}

// CAP: scores are capped (the code for it, though not run, cost the plain kernel 6%).
template <int D, int NR, bool CAP>
__global__ void __launch_bounds__(kFewThreads, (FewCfg<D, NR>::kPerSm))
    paged_few_kernel(const __grid_constant__ PagedLaunch a, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const WaitTest test) {
  using C = FewCfg<D, NR>;
  constexpr int TK = C::TK, N = C::N, PW = C::PW, NS = C::kStages;
  grid_dep_wait();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);  // a stage's K and V have landed
  uint64_t* empty = full + NS;                                    // its P V is done
  uint64_t* s_full = empty + NS;                                  // [2]
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 1;
  uint64_t* q_full = o_full + 1;
  uint64_t* drain = q_full + 1;
  float4* f4_s = reinterpret_cast<float4*>(sm + C::OFF_F4);
  float2* f2_s = reinterpret_cast<float2*>(sm + C::OFF_F2);
  int4* row_s = reinterpret_cast<int4*>(sm + C::OFF_ROW);
  float* qs_s = reinterpret_cast<float*>(sm + C::OFF_QS);
  float* red_s = reinterpret_cast<float*>(sm + C::OFF_RED);
  int* vend_s = reinterpret_cast<int*>(sm + C::OFF_VEND);
  float* m_s = reinterpret_cast<float*>(sm + C::OFF_M);
  uint32_t* tm_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_TM);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + C::OFF_ABORT);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const Waits wait{a.status, test.limit_ns, abort, 40u};

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s_full[i], 1);
    mbar_init(p_full, 4);
    mbar_init(o_full, 1);
    mbar_init(q_full, 4);
    mbar_init(drain, 1);
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 5) tmem_alloc(tm_slot, C::kCols);
  PagedShare share;
  const PagedStart st = paged_start<NR, TK>(a, &share, reinterpret_cast<PagedScratch*>(sm + C::OFF_SCAN));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tm_slot, tmem_o = tmem + 2 * N;
  PagedWalk<NR, TK> w(a, st, share);
  int n = 0;  // tiles so far

  if (warp == 4) {
    // ------------------------------------------------------------- copies
    constexpr int kMaxPages = TK / 16;
    const int per = TK >> a.page_log2;  // pages of a tile
    const uint32_t page_bytes = (uint32_t)a.page * D;
    bool go = true, first = true;
    while (go && w.next()) {
      if (lane == 0 && first) w.write_meta(false);
      first = false;
      const PieceKeys<NR, TK> keys(a, w);
      const PageAhead<NR, TK> pages(a, w, keys);
      // lane i < per: the tile's page i
      static_assert(3 * TK <= kPagedAhead, "positions of two tiles behind the last");
      auto entry = [&](int t) { return pages.entry(lane < per ? t : INT_MAX, t * TK + (lane & (per - 1)) * a.page); };
      int32_t e1 = entry(keys.t0), e2 = entry(keys.t0 + 1);
      for (int t = keys.t0; t < keys.t1; ++t, ++n) {
        const int64_t ph = pages.place(e1);
        if (ph < 0 && lane < per && t * TK + lane * a.page < keys.hi && t * TK + (lane + 1) * a.page > keys.lo && a.status)
          atomicOr(a.status, LCSC_DEV_BAD_INDEX);
        e1 = e2;
        e2 = entry(t + 2);
        const int s = n % NS;
        if (n >= NS && !wait(&empty[s], (uint32_t)(n / NS - 1) & 1u)) {
          go = false;
          break;
        }
        const uint32_t some = __ballot_sync(0xffffffffu, ph >= 0);
        if (lane == 0) mbar_arrive_expect_tx(&full[s], 2 * page_bytes * __popc(some));
        __syncwarp();
        if (ph >= 0) {
          const int32_t row = (int32_t)(ph << a.page_log2);
          tma_load_2d(sm + C::OFF_K + s * C::kTile + lane * page_bytes, &map_k, 0, row, &full[s]);
          tma_load_2d(sm + C::OFF_V + s * C::kTile + lane * page_bytes, &map_v, 0, row, &full[s]);
        }
        __syncwarp();
      }
    }
    static_assert(kMaxPages <= 32, "a lane per page");
    if (lane == 0 && first) w.write_meta(true);
    __syncwarp();
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMA
    const uint32_t idesc_qk = idesc_dense(0, 0, 128, N);
    const uint32_t idesc_pv = idesc_dense(0, 0, D, N, true, true);
    const uint32_t qa = smem_u32(sm + C::OFF_Q), pa = smem_u32(sm + C::OFF_P);
    bool go = !test.stall || wait(drain, 0);  // a test of the failure path: nothing has committed to it yet
    bool pend = false;
    int pieces = 0;
    auto issue_pv = [&](int m) -> bool {
      if (!wait(p_full, (uint32_t)m & 1u)) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t va = smem_u32(sm + C::OFF_V + (m % NS) * C::kTile);
#pragma unroll
        for (int k = 0; k < TK / 32; ++k)
#pragma unroll
          for (int term = 0; term < kPTerms; ++term)
            mma_ss<1>(tmem_o, smem_desc(va + k * 32 * D, 16, 8 * D, kSwOf<D>),
                      smem_desc(pa + k * 32 * PW + term * N, 16, 8 * PW, kSwOf<PW>), idesc_pv, k > 0 || term > 0);
        tc_commit(o_full);
        tc_commit(&empty[m % NS]);
      }
      __syncwarp();
      return true;
    };
    while (go && w.next()) {
      const PieceKeys<NR, TK> keys(a, w);
      if (keys.t0 >= keys.t1) continue;
      // the softmax warps lay out this piece's queries after the last piece's end
      if (pend && !(go = issue_pv(n - 1))) break;
      pend = false;
      if (!(go = wait(q_full, (uint32_t)pieces & 1u))) break;
      ++pieces;
      for (int t = keys.t0; t < keys.t1; ++t) {
        const int s = n % NS;
        if (!(go = wait(&full[s], (uint32_t)(n / NS) & 1u))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t ka = smem_u32(sm + C::OFF_K + s * C::kTile);
#pragma unroll
          for (int term = 0; term < kQTerms; ++term)
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              mma_ss<1>(tmem + (n & 1) * N, smem_desc(ka + k * 32, 16, 8 * D, kSwOf<D>),
                        smem_desc(qa + term * C::kQBytes + k * 32, 16, 8 * D, kSwOf<D>), idesc_qk, k > 0 || term > 0);
          tc_commit(&s_full[n & 1]);
        }
        __syncwarp();
        if (pend && !(go = issue_pv(n - 1))) break;
        pend = true;
        ++n;
      }
    }
    if (go && pend) issue_pv(n - 1);
    if (lane == 0) {  // every MMA has completed before TMEM is freed
      tc_commit(drain);
      mbar_wait(drain, 0, a.status, kDrainLimitNs);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const float c2 = a.sm_scale * kPagedLog2e, cap2 = a.cap * kPagedLog2e;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const bool has_dim = D == 128 || lane < 16;
    const int dim = D == 128 ? tid : warp * 16 + (lane & 15);  // M = 64 accumulators lie in lanes 0-15
    bool ok = true;
    while (ok && w.next()) {
      const PieceKeys<NR, TK> keys(a, w);
      const int rows = w.rows(), r0 = w.p_mt * NR;
      const bool work = keys.t0 < keys.t1;
      named_sync(1, 128);  // the last piece is done with shared memory
      if (tid < NR) {
        int4 r = make_int4(0, 0, 0, 0);
        if (tid < rows) {
          const int i = paged_div(a, r0 + tid);
          paged_row(a, w.p_s, paged_prefix(a, w.p_b), i, &r.x, &r.y);
          r.z = w.p_s.L - w.p_s.n + i;
          if (a.slopes) r.w = __float_as_int(a.slopes[w.p_h * a.G + r0 + tid - i * a.G] * kPagedLog2e);
        }
        row_s[tid] = r;
      }
      if (work) {
        // the query's terms, a warp per row
        for (int r = warp; r < N; r += 4) {
          constexpr int VPL = D / 32;
          float v[VPL];
#pragma unroll
          for (int i = 0; i < VPL; ++i) v[i] = 0.f;
          if (r < rows) {
            const int row = r0 + r, tok = paged_div(a, row);
            const uint16_t* p = reinterpret_cast<const uint16_t*>(a.q) + (w.p_s.q0 + tok) * a.q_stride +
                                (int64_t)(w.p_h * a.G + row - tok * a.G) * D + lane * VPL;
            if constexpr (VPL == 4) {
              const uint2 u = *reinterpret_cast<const uint2*>(p);
              v[0] = bf16_val((uint16_t)u.x), v[1] = bf16_val((uint16_t)(u.x >> 16));
              v[2] = bf16_val((uint16_t)u.y), v[3] = bf16_val((uint16_t)(u.y >> 16));
            } else {
              const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
              v[0] = bf16_val((uint16_t)u), v[1] = bf16_val((uint16_t)(u >> 16));
            }
          }
          float amax = 0.f;
#pragma unroll
          for (int i = 0; i < VPL; ++i) amax = fmaxf(amax, fabsf(v[i]));
          amax = warp_max(amax);
          const int ex = amax > 0.f ? (int)(__float_as_uint(amax) >> 23) - 127 - 7 : 0;
          uint16_t hi[VPL / 2], lo[VPL / 2];
#pragma unroll
          for (int i = 0; i < VPL / 2; ++i) {
            const float x = times_pow2(v[2 * i], -ex), y = times_pow2(v[2 * i + 1], -ex);
            hi[i] = e4m3x2_code(x, y);
            const float2 h = e4m3x2_val(hi[i]);
            lo[i] = e4m3x2_code(x - h.x, y - h.y);
          }
          uint8_t* q = sm + C::OFF_Q + swz<D>(r, lane * VPL);
          if constexpr (VPL == 4) {
            *reinterpret_cast<uint32_t*>(q) = hi[0] | ((uint32_t)hi[1] << 16);
            *reinterpret_cast<uint32_t*>(q + C::kQBytes) = lo[0] | ((uint32_t)lo[1] << 16);
          } else {
            *reinterpret_cast<uint16_t*>(q) = hi[0];
            *reinterpret_cast<uint16_t*>(q + C::kQBytes) = lo[0];
          }
          // a query that is not finite gives scores that are not numbers
          if (lane == 0 && r < NR) qs_s[r] = amax <= 3.402823466e38f ? times_pow2(1.f, ex) : NAN;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      named_sync(1, 128);  // row_s and qs_s
      int lo_max = 0, hi_min = INT_MAX;
      for (int r = 0; r < rows; ++r) lo_max = max(lo_max, row_s[r].x), hi_min = min(hi_min, row_s[r].y);
      const bool one_span = lo_max <= keys.lo && hi_min >= keys.hi;

      float l[NR], o[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) l[r] = 0.f, o[r] = 0.f;
      float m_run = -INFINITY;  // thread r < NR: running max of row r
      // this thread's key of a tile: its page two tiles ahead, its scales one
      const PageAhead<NR, TK> pages(a, w, keys);
      const int64_t ph0 = pages.place(pages.entry(keys.t0, keys.t0 * TK + tid));
      int32_t e1 = pages.entry(keys.t0 + 1, (keys.t0 + 1) * TK + tid);
      float ks = ph0 < 0 ? -1.f : a.k_scale[ph0], vs = ph0 < 0 ? 0.f : a.v_scale[ph0];
      auto add_o = [&](int m) -> bool {  // O of tile m into the running one
        if (!wait(o_full, (uint32_t)m & 1u)) return false;
        tc_fence_after();
        uint32_t x[NR];
        tmem_ld(tmem_o + lane_base, x);
        tmem_ld_done(x);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float2 f = f2_s[r];
          o[r] = fmaf(o[r], f.x, __uint_as_float(x[r]) * f.y);
        }
        return true;
      };
      for (int t = keys.t0; t < keys.t1; ++t, ++n) {
        const int64_t ph1 = pages.place(e1);
        const float ks_next = ld_if(a.k_scale + ph1, ph1 >= 0, -1.f), vs_next = ld_if(a.v_scale + ph1, ph1 >= 0, 0.f);
        e1 = pages.entry(t + 2, (t + 2) * TK + tid);
        const int j = t * TK + tid;
        const bool there = ks >= 0.f && j >= keys.lo && j < keys.hi;  // copied, and seen by some row
        const float kf = ks * c2;
        if (lane % 16 == 0) vend_s[tid / 16] = ks >= 0.f ? __float_as_int(vs) : -1;  // 16 keys lie in one page
        float s[NR];
        ok = wait(&s_full[n & 1], (uint32_t)(n >> 1) & 1u);
        if (ok) {
          tc_fence_after();
          uint32_t x[NR];
          tmem_ld(tmem + (n & 1) * N + lane_base, x);
          tmem_ld_done(x);
          float mine = -INFINITY;
          const bool inside = one_span || (t * TK >= lo_max && (t + 1) * TK <= hi_min);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            float y = __uint_as_float(x[r]) * (kf * qs_s[r]);
            if constexpr (CAP) y = paged_cap(y, cap2);
            if (a.slopes) y -= __int_as_float(row_s[r].w) * (float)abs(row_s[r].z - j);
            bool see = there;
            if (!inside) see = see && j >= row_s[r].x && j < row_s[r].y;
            s[r] = see ? y : -INFINITY;
            const float top = warp_redux_max(s[r]);
            if (lane == r) mine = top;
          }
          if (lane < NR) red_s[warp * NR + lane] = mine;
        }
        if (!(ok = named_and(1, 128, ok))) break;
        // (bits of numbers that are not negative order as the numbers do; -1 is the
        // least signed and the largest unsigned one)
        const int4 va = *reinterpret_cast<const int4*>(vend_s), vb = *reinterpret_cast<const int4*>(vend_s + 4);
        const float vmax = __int_as_float(max(max(max(max(va.x, va.y), max(va.z, va.w)), max(max(vb.x, vb.y), max(vb.z, vb.w))), 0));
        const float vmin = __uint_as_float(min(min(min((uint32_t)va.x, (uint32_t)va.y), min((uint32_t)va.z, (uint32_t)va.w)),
                                               min(min((uint32_t)vb.x, (uint32_t)vb.y), min((uint32_t)vb.z, (uint32_t)vb.w))));
        float al = 0.f, be = 0.f, mt = -INFINITY;
        if (tid < NR) {
          mt = fmaxf(fmaxf(red_s[tid], red_s[NR + tid]), fmaxf(red_s[2 * NR + tid], red_s[3 * NR + tid]));
          const float m_new = fmaxf(m_run, mt), ref = m_new == -INFINITY ? 0.f : m_new;
          al = paged_ex2(m_run - ref);
          be = paged_ex2(mt - ref);
          m_run = m_new;
          f4_s[tid] = make_float4(mt == -INFINITY ? 0.f : mt, al, be, 0.f);
        }
        // the last tile's O before its factors give way to this tile's
        const bool o_in = t == keys.t0 || add_o(n - 1);
        if (!(ok = named_and(1, 128, o_in))) break;
        if (tid < NR) f2_s[tid] = make_float2(al, be * vmax * (1.f / 256.f));
        // weights in [0, 256], relative to the tile's maxima and largest V scale
        const float vr = there && vmax > 0.f ? __fdividef(vs, vmax) * 256.f : 0.f;
        const uint32_t prow = smem_u32(sm + C::OFF_P);
        float p[NR];
#pragma unroll
        for (int r = 0; r < NR; r += 2) {
          const float4 fa = f4_s[r], fb = f4_s[r + 1];
          const float pa = paged_ex2(s[r] - fa.x), pb = paged_ex2(s[r + 1] - fb.x);
          l[r] = fmaf(l[r], fa.y, pa * fa.z);
          l[r + 1] = fmaf(l[r + 1], fb.y, pb * fb.z);
          p[r] = pa * vr, p[r + 1] = pb * vr;
        }
        few_codes<NR>(p, prow);
        if (vmin < 0.25f * vmax) {  // (no page at all: vmin is no number)
          float sx[NR];
#pragma unroll
          for (int r = 0; r < NR; ++r) sx[r] = s[r];
          few_far<NR>(sx, there ? vs : 0.f, m_run, red_s, f2_s, prow);
        }
        if (!there) {  // no row sees the key: its V may hold anything, and 0 x NaN is NaN
          uint4* v = reinterpret_cast<uint4*>(sm + C::OFF_V + (n % NS) * C::kTile + tid * D);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) v[i] = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
        ks = ks_next, vs = vs_next;
      }
      if (ok && work) {
        named_sync(1, 128);  // f2_s of the last tile
        ok = add_o(n - 1);
      }
      float mine = 0.f;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float sum = warp_sum(l[r]);
        if (lane == r) mine = sum;
      }
      if (lane < NR) red_s[warp * NR + lane] = mine;
      if (tid < NR) m_s[tid] = m_run;
      if (!(ok = named_and(1, 128, ok))) break;
      if (w.whole()) {
        if (has_dim) {
#pragma unroll
          for (int r = 0; r < NR; ++r)
            if (r < rows)
              paged_write<D>(a, w.p_s, w.p_h, r0 + r, dim, o[r], m_s[r],
                             red_s[r] + red_s[NR + r] + red_s[2 * NR + r] + red_s[3 * NR + r]);
        }
      } else {
        const int64_t at = w.slot() * NR;
        if (has_dim) {
#pragma unroll
          for (int r = 0; r < NR; ++r)
            if (r < rows) a.part_o[(at + r) * D + dim] = o[r];
        }
        if (tid < rows) {
          a.part_ml[(at + tid) * 2] = m_s[tid];
          a.part_ml[(at + tid) * 2 + 1] = red_s[tid] + red_s[NR + tid] + red_s[2 * NR + tid] + red_s[3 * NR + tid];
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Where a role gave up, maybe after the last copy went out, nobody may have
  // waited for the copies in flight: they land before the CTA's memory is another's.
  if (warp == 4 && *abort)
    for (int i = n > NS ? n - NS : 0; i < n; ++i) mbar_wait(&full[i % NS], (uint32_t)(i / NS) & 1u, a.status, kDrainLimitNs);
  if (warp == 5) tmem_dealloc(tmem, C::kCols);
}

// ============================================================== many rows
// Prompts, and decode of many heads on one: blocks of 256 query rows, as two
// tiles of 128 that share K and V.
//   S [128 rows][128 keys] = Q K^T     Q: two E4M3 terms, K as stored (kind::f8f6f4)
//   O [128 rows][D dims]  += P V       P and V in f16 (kind::f16)
// A softmax warpgroup owns a tile and a thread one row of it: maxima and sums
// need no exchange.  O stays in TMEM; it is rescaled only when a row's maximum
// has grown by more than 2^6.  Weights are f16 numbers from 2^15 down to steps of
// 2^-24, the row's largest at least 2^9: 11 bits down to 2^-23 of it, and below
// that an error of 2^-34 of it at most.  V's codes become f16 numbers: four warps
// read them from global memory a tile ahead and write code * 2^7 * (page scale /
// largest page scale of the piece), which is exact for scales down to 2^-22 of
// the largest and loses only what lies below 2^-32 of the largest possible |V|.
// Two tiles keep the tensor cores busy with one while the other's weights are
// made; a block of up to 128 rows is one tile, which the two warpgroups share by
// taking its tiles of keys in turn and joining their O at the end (16 requests of
// 4K to 32K tokens, 32 rows each, D = 128: 208 us, 2.7 TB/s; a million tokens for
// 64 capped heads on one: 120 us, 2.2 TB/s; both of a CTA's chain from scores to
// weights).
//
// Bound: per 256 x 128 step the products take 2,048 cycles of the tensor pipe,
// as do the exponentials of the MUFU (32 K at 16 a cycle), and shared memory
// about 2,900 (operands 2,048, P 512, V 256, K 128).  Measured 5,400 (the tensor
// pipe is active 38% of the time, the MUFU 39%, issue slots 42%): one warpgroup's
// chain of waiting for its scores, their maxima, weights and the copies'
// bookkeeping (700, 800 and 2,200 of the cycles by clock probes).  Of 8.4 warps
// an issue, 3.5 wait for TMEM loads or a barrier's look, 1.6 for fixed latencies,
// 0.9 for shared memory or the MUFU and 0.3 for instructions.  Taking work out of
// the kernel shows that no unit holds it (no exponentials: -2%, one query term:
// -4%, no V conversion: -8%), while larger loop bodies cost 10 to 30% and twice
// the softmax warps 46%.  Chunk of 4096 tokens on 4096 cached, 64 heads on 8,
// D = 128: 1,010 us, 0.82 PFLOP/s, 50% of the measured bf16 rate.

constexpr int kManyThreads = 448;  // warps 0-7 softmax (two tiles), 8-11 V, 12 copies, 13 MMA
constexpr int kManyRows = kPagedManyRows;
// A row's weights are 2^(x - reference), the reference kDrop below the row's
// maximum when it is taken, and taken anew, with O rescaled, when a score has
// grown past it by more than kLazy (base-2 units): f16 weights of up to 2^15.
// (Chunk of 4096 tokens: 1,041 us with a drop of 9 or 7, 1,051 with 11, which
// rescales more.)
constexpr float kDrop = 9.f, kLazy = 15.f;
constexpr float kBig = 0x1p20f;  // scores whose rounding is no small part of that range; their reference is the maximum

template <int D>
struct ManyCfg {
  static constexpr int TK = 128;
  static constexpr int kQTerm = 128 * D;              // one term of a tile's queries
  static constexpr int kK = TK * D;
  static constexpr int kV = TK * D * 2;
  static constexpr int kP = 128 * TK * 2;
  static constexpr int OFF_Q = 0;                     // [2 tiles][2 terms]
  static constexpr int OFF_K = OFF_Q + 4 * kQTerm;    // [2]
  static constexpr int OFF_V = OFF_K + 2 * kK;        // [2]
  static constexpr int OFF_P = OFF_V + 2 * kV;        // [2 tiles]
  static constexpr int OFF_BAR = OFF_P + 2 * kP;
  static constexpr int kBars = 22;
  static constexpr int OFF_ML = OFF_BAR + (kBars + 1) / 2 * 16;  // float2 [128]: the second warpgroup's maxima and sums
  static constexpr int OFF_SCAN = OFF_ML + 128 * 8;  // PagedScratch
  static constexpr int OFF_VREF = OFF_SCAN + (int)sizeof(PagedScratch);    // int: largest V scale of the piece (bits)
  static constexpr int OFF_TM = OFF_VREF + 4;
  static constexpr int OFF_ABORT = OFF_TM + 4;
  static constexpr int SMEM = OFF_ABORT + 4 + 1024;
  static_assert(OFF_K % 1024 == 0 && OFF_V % 1024 == 0 && OFF_P % 1024 == 0 && OFF_SCAN % 8 == 0, "alignment");
  static_assert(SMEM <= 232448 - 64, "shared memory per block");
};

// One row's scores: factors, mask and bias of the thread's query row.
struct ManyRow {
  int lo, hi, pos;
  float rf, slope;  // 2^e of the query; bias per position in base-2 units
};

// Bits of the keys j .. j + 31 that the row sees; `there`: bit i for a page of the keys j + 16 i ..
__device__ __forceinline__ uint32_t many_seen(const ManyRow& r, int j, uint32_t there) {
  const int lo = min(max(r.lo - j, 0), 32), hi = min(max(r.hi - j, 0), 32);
  const uint32_t below_hi = (uint32_t)((1ull << hi) - 1), below_lo = (uint32_t)((1ull << lo) - 1);
  return below_hi & ~below_lo & ((there & 1u ? 0x0000ffffu : 0u) | (there & 2u ? 0xffff0000u : 0u));
}

// 32 scores capped: while all of the warp's are within the cap, by paged_cap's
// polynomial in packed operations (4.5 a score, against two of the 8-cycle MUFU
// operations of the exponential form that takes the rest).
__device__ __forceinline__ void many_cap(float (&v)[32], float cap) {
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) most = fmaxf(most, fabsf(v[i]));
  if (__all_sync(0xffffffffu, !(most > cap))) {
    const float inv = 1.f / cap;
    const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const uint64_t x = pack2(v[i], v[i + 1]), y = mul2(x, inv2), z = mul2(y, y);
      uint64_t p = pack2(paged_tanh(6), paged_tanh(6));
#pragma unroll
      for (int k = 5; k >= 0; --k) p = fma2(p, z, pack2(paged_tanh(k), paged_tanh(k)));
      unpack2(mul2(x, p), v[i], v[i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = paged_cap_far(v[i], cap);
  }
}

// 32 scores of the keys j .. j + 31, less the row's slope times their distance.
__device__ __forceinline__ void many_bias(float (&v)[32], const ManyRow& r, int j) {
  if (__all_sync(0xffffffffu, r.pos - j >= 31)) {
    const float first = -r.slope * (float)(r.pos - j);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = fmaf(r.slope, (float)i, v[i] + first);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] -= r.slope * (float)abs(r.pos - (j + i));
  }
}

// A row's largest score over the keys h0 .. h1 of a tile, in base-2 units; lanes of .. of + 7 of
// `ks` hold the factors of the tile's 16-key groups (below 0: not there).  Three forms:
//   kPlain:  every row of the warp sees every key, no cap, no bias: the largest
//            raw product of each page, times its factor
//   kMasked: no cap, no bias
//   kScores: everything
// The last two put the scores themselves in the products' place, so that the
// weights are made alike for all.  Rolled loops: what a softmax warp runs over
// and over has to stay in the instruction cache (rolled against unrolled
// fourfold, chunk of 4096 tokens: 1,220 against 1,470 us).
enum ManyForm { kPlain, kMasked, kScores };
template <ManyForm F>
__device__ __forceinline__ float many_top(const PagedLaunch& a, const ManyRow& r, float cap2, float ks, int of, int j0,
                                          bool inside, uint32_t s_addr, int h0, int h1) {
  float top = -INFINITY;
#pragma unroll 1
  for (int h = h0; h < h1; h += 32) {
    uint32_t x[32];
    tmem_ld(s_addr + h, x);
    const float k0 = __shfl_sync(0xffffffffu, ks, of + (h >> 4)), k1 = __shfl_sync(0xffffffffu, ks, of + (h >> 4) + 1);
    const float c0 = k0 * r.rf, c1 = k1 * r.rf;
    uint32_t seen = 0xffffffffu;
    if constexpr (F != kPlain) seen = many_seen(r, j0 + h, (k0 >= 0.f ? 1u : 0u) | (k1 >= 0.f ? 2u : 0u));
    tmem_ld_done(x);
    if constexpr (F != kPlain) {
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(x[i]) * (i < 16 ? c0 : c1);
      if constexpr (F == kScores) {
        if (a.cap > 0.f) {
          if (!inside) {  // what lies behind the last key has no say in the cap's form
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = seen >> i & 1u ? v[i] : 0.f;
          }
          many_cap(v, cap2);
        }
        if (a.slopes) many_bias(v, r, j0 + h);
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(v[i]);
      if (!inside) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = seen >> i & 1u ? x[i] : 0xff800000u;
      }
      tmem_st_32(s_addr + h, x);
    }
    float m0 = __uint_as_float(x[0]), m1 = __uint_as_float(x[16]);
#pragma unroll
    for (int i = 1; i < 16; ++i) {
      m0 = fmaxf(m0, __uint_as_float(x[i]));
      m1 = fmaxf(m1, __uint_as_float(x[16 + i]));
    }
    top = fmaxf(top, F == kPlain ? fmaxf(m0 * c0, m1 * c1) : fmaxf(m0, m1));
  }
  if constexpr (F != kPlain) tmem_st_wait();
  return top;
}

template <int D>
__device__ __forceinline__ void many_rescale(uint32_t o_addr, float alpha) {
#pragma unroll 1
  for (int d = 0; d < D; d += 32) {
    uint32_t o[32];
    tmem_ld(o_addr + d, o);
    tmem_ld_done(o);
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
    tmem_st_32(o_addr + d, o);
  }
  tmem_st_wait();
}

// The earliest document start and the latest end of every block of rows, a warp per block.
__global__ void __launch_bounds__(256) paged_docs_kernel(const PagedLaunch a) {
  grid_dep_wait();
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const PagedSeq s = paged_seq(a, b);
  for (int mt = blockIdx.y * 8 + threadIdx.x / 32; (int64_t)mt * kManyRows < (int64_t)s.n * a.G; mt += gridDim.y * 8) {
    const int i0 = paged_div(a, mt * kManyRows), i1 = paged_div(a, min(s.n * a.G, (mt + 1) * kManyRows) - 1);
    const int2 d = paged_docs(a, s, i0, i1);
    if (lane == 0) a.block_docs[paged_block(a, s, mt)] = d;
  }
}

// GEN: scores are capped or biased (both forms of the loop in one kernel cost
// the plain one 1%, the other 4%).
template <int D, bool GEN>
__global__ void __launch_bounds__(kManyThreads, 1)
    paged_many_kernel(const __grid_constant__ PagedLaunch a, const __grid_constant__ CUtensorMap map_k, const WaitTest test) {
  using C = ManyCfg<D>;
  constexpr int TK = C::TK, M = kManyRows;
  grid_dep_wait();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);  // [2]
  uint64_t* k_empty = k_full + 2;    // [2] every Q K^T on it is done
  uint64_t* v_full = k_full + 4;     // [2] V is there in f16
  uint64_t* v_empty = k_full + 6;    // [2] every P V on it is done
  uint64_t* s_full = k_full + 8;     // [2 tiles]
  uint64_t* p_full = k_full + 10;    // [2 tiles] P is written, S is read
  uint64_t* pv_done = k_full + 12;   // [2 tiles]
  uint64_t* q_full = k_full + 14;    // [2 tiles] the queries
  uint64_t* ref_full = k_full + 16;  // the piece's largest V scale
  uint64_t* piece_done = k_full + 17;
  uint64_t* drain = k_full + 18;
  uint64_t* ml_full = k_full + 19;   // the second warpgroup's part of a shared block of rows
  uint64_t* swap_full = k_full + 20;  // [2 warpgroups]
  float2* ml_s = reinterpret_cast<float2*>(sm + C::OFF_ML);
  volatile int* vref_s = reinterpret_cast<volatile int*>(sm + C::OFF_VREF);
  uint32_t* tm_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_TM);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + C::OFF_ABORT);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const Waits wait{a.status, test.limit_ns, abort, warp == 13 ? 20u : warp >= 8 ? 100u : 50u};

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1), mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 4), mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1), mbar_init(&p_full[i], 4), mbar_init(&pv_done[i], 1);
      mbar_init(&swap_full[i], 4), mbar_init(&q_full[i], 4);
    }
    mbar_init(ref_full, 4);
    mbar_init(piece_done, 8);
    mbar_init(drain, 1);
    mbar_init(ml_full, 4);
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 13) tmem_alloc(tm_slot, 512);
  PagedShare share;
  const PagedStart st = paged_start<M, TK>(a, &share, reinterpret_cast<PagedScratch*>(sm + C::OFF_SCAN));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tm_slot;  // S of tile 0, 1 (128 columns each), O of tile 0, 1
  PagedWalk<M, TK> w(a, st, share);
  int copied = 0;  // tiles of K asked for (the copies' warp)

  if (warp == 12) {
    // ------------------------------------------------------------- copies
    const int per = TK >> a.page_log2;
    const uint32_t page_bytes = (uint32_t)a.page * D;
    bool go = true, first = true;
    while (go && w.next()) {
      if (lane == 0 && first) w.write_meta(false);
      first = false;
      const PieceKeys<M, TK> keys(a, w);
      const PageAhead<M, TK> pages(a, w, keys);
      // lane i < per: the tile's page i
      static_assert(3 * TK <= kPagedAhead, "positions of two tiles behind the last");
      auto entry = [&](int t) { return pages.entry(lane < per ? t : INT_MAX, t * TK + (lane & (per - 1)) * a.page); };
      int32_t e1 = entry(keys.t0), e2 = entry(keys.t0 + 1);
      for (int t = keys.t0; t < keys.t1; ++t, ++copied) {
        const int64_t ph = pages.place(e1);
        if (ph < 0 && lane < per && t * TK + lane * a.page < keys.hi && t * TK + (lane + 1) * a.page > keys.lo && a.status)
          atomicOr(a.status, LCSC_DEV_BAD_INDEX);
        e1 = e2;
        e2 = entry(t + 2);
        const int s = copied & 1;
        if (copied >= 2 && !wait(&k_empty[s], (uint32_t)((copied >> 1) - 1) & 1u)) {
          go = false;
          break;
        }
        const uint32_t some = __ballot_sync(0xffffffffu, ph >= 0);
        if (lane == 0) mbar_arrive_expect_tx(&k_full[s], page_bytes * __popc(some));
        __syncwarp();
        if (ph >= 0)
          tma_load_2d(sm + C::OFF_K + s * C::kK + lane * page_bytes, &map_k, 0, (int32_t)(ph << a.page_log2), &k_full[s]);
        __syncwarp();
      }
    }
    if (lane == 0 && first) w.write_meta(true);
    __syncwarp();
  } else if (warp == 13) {
    // ---------------------------------------------------------------- MMA
    const uint32_t idesc_qk = idesc_dense(0, 0, 128, TK);
    const uint32_t idesc_pv = idesc_dense(0, 0, 128, D, false, true);
    const uint32_t qa = smem_u32(sm + C::OFF_Q);
    bool go = !test.stall || wait(drain, 0);  // a test of the failure path: nothing has committed to it yet
    int n = 0, pieces[2] = {0, 0}, cnt[2] = {0, 0};
    while (go && w.next()) {
      const PieceKeys<M, TK> keys(a, w);
      if (keys.t0 >= keys.t1) continue;
      const bool shared = w.rows() <= 128;  // both warpgroups on one tile of rows
      if (!(go = wait(&q_full[0], (uint32_t)pieces[0]++ & 1u))) break;
      if (!shared && !(go = wait(&q_full[1], (uint32_t)pieces[1]++ & 1u))) break;
      // Per warpgroup: Q K^T of its next tile of keys as soon as its scores are
      // read, then P V of its last one (the tile before, or, where the
      // warpgroups take the tiles in turn, the one before that).
      const int T = keys.t1 - keys.t0, last = shared ? 0 : 1, lag = shared ? 2 : 1;
      for (int i = 0; go && i < T + lag; ++i) {
        const int s = (n + i) & 1;
        if (i < T && !(go = wait(&k_full[s], (uint32_t)((n + i) >> 1) & 1u))) break;
        for (int e = 0; e <= last; ++e) {
          const int g = shared ? i & 1 : e;
          if (i >= lag && !(go = wait(&p_full[g], (uint32_t)(cnt[g] - 1) & 1u))) break;
          if (i < T) {
            tc_fence_after();
            if (elect_one()) {
              const uint32_t ka = smem_u32(sm + C::OFF_K + s * C::kK), qt = qa + 2 * e * C::kQTerm;
#pragma unroll
              for (int term = 0; term < kQTerms; ++term)
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
                  mma_ss<1>(tmem + g * 128, smem_desc(qt + term * C::kQTerm + k * 32, 16, 8 * D, kSwOf<D>),
                            smem_desc(ka + k * 32, 16, 8 * D, kSwOf<D>), idesc_qk, k > 0 || term > 0);
              tc_commit(&s_full[g]);
              if (e == last) tc_commit(&k_empty[s]);
            }
            __syncwarp();
          }
          if (i >= lag) {
            const int m = n + i - lag, b = m & 1;
            if (e == 0 && !(go = wait(&v_full[b], (uint32_t)(m >> 1) & 1u))) break;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t pa = smem_u32(sm + C::OFF_P + g * C::kP), va = smem_u32(sm + C::OFF_V + b * C::kV);
              const bool acc = i >= 2 * lag;  // not the warpgroup's first tile
#pragma unroll
              for (int k = 0; k < TK / 16; ++k)
                mma_ss<0>(tmem + 256 + g * 128, smem_desc(pa + (k / 4) * (128 * 128) + (k % 4) * 32, 16, 1024, kSw128),
                          smem_desc(va + k * 16 * 128, TK * 128, 1024, kSw128), idesc_pv, acc || k > 0);
              tc_commit(&pv_done[g]);
              if (e == last) tc_commit(&v_empty[b]);
            }
            __syncwarp();
          }
          if (i < T) ++cnt[g];
        }
      }
      n += T;
    }
    if (lane == 0) {
      tc_commit(drain);
      mbar_wait(drain, 0, a.status, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ V
    // Warp v has the keys 32 v .. 32 v + 31 of a tile; 8 (D = 64: 4) lanes
    // read a row's chunks of 16 codes.
    constexpr int LPR = D / 16, RPI = 32 / LPR, IT = 32 / RPI;  // lanes per row, rows per step, steps
    const int v = warp - 8, c = lane % LPR, rsub = lane / LPR;
    int n = 0, pieces = 0;
    bool ok = true;
    while (ok && w.next()) {
      const PieceKeys<M, TK> keys(a, w);
      if (keys.t0 >= keys.t1) {
        // nothing to do, but the piece counts
        ok = named_and(2, 128, true);
        if (pieces > 0) ok = named_and(2, 128, wait(piece_done, (uint32_t)(pieces - 1) & 1u));
        ++pieces;
        if (ok && lane == 0) mbar_arrive(ref_full);
        continue;
      }
      const PageAhead<M, TK> pages(a, w, keys);
      // the largest scale of the piece's pages, by page numbers: 128 pages on, a
      // position may pass 2^31
      int top = 0;
      const int last = (min(keys.hi, keys.t1 * TK) - 1) >> a.page_log2;
      for (int pg = (max(keys.t0 * TK, keys.lo) >> a.page_log2) + tid - 256; pg <= last; pg += 128) {
        const int64_t ph = pages.place(pages.entry(keys.t0, pg << a.page_log2));
        if (ph >= 0) top = max(top, __float_as_int(a.v_scale[ph]));
      }
      top = __reduce_max_sync(0xffffffffu, top);
      // the last piece's softmax has read its scale
      ok = pieces == 0 || wait(piece_done, (uint32_t)(pieces - 1) & 1u);
      ++pieces;
      if (tid == 256) *vref_s = 0;
      if (!(ok = named_and(2, 128, ok))) break;
      if (lane == 0) atomicMax(const_cast<int*>(vref_s), top);
      named_sync(2, 128);
      const float vref = __int_as_float(*vref_s);
      if (lane == 0) mbar_arrive(ref_full);
      // codes to f16 (exact) and times 2^7 scale / vref: at most 448 * 2^7
      const float inv = vref > 0.f ? __fdividef(1.f, vref) * 128.f : 0.f;
      // A warp's 32 keys of a tile in two halves of 16 (one page each): as soon as
      // one is converted and stored, the codes of the next tile's are asked for in
      // its registers, and the page of the one after that is looked up.
      constexpr int HI = IT / 2;
      uint4 raw[2][HI];
      float sc[2];  // the half's scale (0: not there)
      int j = keys.t0 * TK + v * 32;  // the tile's first key of the warp
      auto entry = [&](int key) { return pages.entry(key / TK, key); };
      int32_t e[2] = {entry(j), entry(j + 16)};
      auto fetch = [&](int half, int key) {
        const int64_t ph = pages.place(e[half]);
        sc[half] = ld_if(a.v_scale + ph, ph >= 0, 0.f);
        const int j0 = key + rsub;
        const uint32_t span = (uint32_t)(keys.hi - keys.lo);
        const uint8_t* src = a.v + (ph * a.page + (j0 & (a.page - 1))) * D + c * 16;
#pragma unroll
        for (int i = 0; i < HI; ++i)  // zeros for the keys that no row sees
          raw[half][i] = ld_if(src + i * RPI * D, ph >= 0 && (uint32_t)(j0 + i * RPI - keys.lo) < span);
      };
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        fetch(half, j + 16 * half);
        e[half] = entry(j + 16 * half + TK);
      }
      const int flip = (c / 4) & 1;
      const uint32_t to = smem_u32(sm + C::OFF_V) + (c / 4) * (TK * 128);  // the 64-dim atom
#pragma unroll 1
      for (int t = keys.t0; t < keys.t1; ++t) {
        const int b = n & 1;
        if (n >= 2 && !(ok = wait(&v_empty[b], (uint32_t)((n >> 1) - 1) & 1u))) break;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const __half2 f = __float2half2_rn(sc[half] * inv);
#pragma unroll
          for (int i = 0; i < HI; ++i) {
            const uint32_t wd[4] = {raw[half][i].x, raw[half][i].y, raw[half][i].z, raw[half][i].w};
            uint32_t h[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const __half2 x(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(wd[q / 2] >> (16 * (q & 1))), __NV_E4M3));
              const __half2 y = __hmul2(x, f);
              h[q] = *reinterpret_cast<const uint32_t*>(&y);
            }
            // 16 dims are two chunks of the atom; the lanes of the second atom
            // store theirs in the other order, so that a store covers all banks
            const int r = v * 32 + half * 16 + i * RPI + rsub, ch = (c % 4) * 2;
            const uint32_t at = to + b * C::kV;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const bool second = (q ^ flip) != 0;
              st_shared16(at + swz<128>(r, (ch + (q ^ flip)) * 16), second ? h[4] : h[0], second ? h[5] : h[1],
                          second ? h[6] : h[2], second ? h[7] : h[3]);
            }
          }
          fetch(half, j + 16 * half + TK);
          e[half] = entry(j + 16 * half + 2 * TK);
        }
        j += TK;
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[b]);
        ++n;
      }
      if (!(ok = named_and(2, 128, ok))) break;  // the four warps go on or stop together
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int g = warp / 4;  // the tile
    const int row_in = tid % 128;
    const float c2 = a.sm_scale * kPagedLog2e, cap2 = a.cap * kPagedLog2e;
    const uint32_t lane_base = (uint32_t)((warp % 4) * 32) << 16;
    const uint32_t s_addr = tmem + g * 128 + lane_base, o_addr = tmem + 256 + g * 128 + lane_base;
    bool ok = true;
    // float [128]: in P's rows from 64 on, which a split block has no use for and
    // no other warpgroup writes (whatever P V makes of them)
    float* swap_s = reinterpret_cast<float*>(sm + C::OFF_P + g * C::kP + 64 * 128);
    int cnt = 0, pieces = 0, merges = 0, swaps = 0;
    while (ok && w.next()) {
      const PieceKeys<M, TK> keys(a, w);
      const int rows = w.rows();
      // Up to 128 rows are one tile that both warpgroups work on, taking its
      // tiles of keys in turn, each with its own maxima, sums and O.
      const bool shared = rows <= 128;
      // Up to 64 rows lie in the tile twice, and a row's two threads take a half of
      // each tile's keys; they agree on its maximum, and the first has its O.  Half
      // the scores a thread where they are long work (capped or biased: a million
      // tokens for 64 heads on one 157 -> 131 us, five draft tokens of 8 heads 186 ->
      // 178); plain ones gain 1% with 32 rows and lose 2% on a prompt's chunk.
      const bool split = GEN && rows <= 64;
      const int side = split ? row_in / 64 : 0, t_row = split ? row_in % 64 : row_in;
      const int h0 = 64 * side, h1 = split ? h0 + 64 : 128;
      const int base = shared ? 0 : g * 128, r_in = base + t_row, row = w.p_mt * M + r_in;
      const bool mine = r_in < rows;
      auto swapped = [&](float x, float* y) {  // the other thread's x
        swap_s[row_in] = x;
        __syncwarp();
        if (lane == 0) mbar_arrive(&swap_full[g]);
        const bool there = wait(&swap_full[g], (uint32_t)swaps++ & 1u);
        *y = swap_s[row_in ^ 64];
        return there;
      };
      ManyRow r = {0, INT_MAX, 1 << 30, 0.f, 0.f};  // a row that is not there sees everything and bears no bias
      if (mine) {
        const int i = paged_div(a, row);
        paged_row(a, w.p_s, paged_prefix(a, w.p_b), i, &r.lo, &r.hi);
        r.pos = w.p_s.L - w.p_s.n + i;
        if (a.slopes) r.slope = a.slopes[w.p_h * a.G + row - i * a.G] * kPagedLog2e;
      }
      const bool work = keys.t0 < keys.t1;
      if (work) {
        // The tile's query terms: LPR lanes read a row together, 8 dims each (a
        // thread per row: 32 lines a load, five draft tokens 187 against 178 us).
        {
          constexpr int LPR = D / 8, RPI = 32 / LPR, IT = 32 / RPI;  // lanes per row, rows per step, steps
          const int c = lane % LPR, first = warp % 4 * 32 + lane / LPR;
          const uint32_t dst = smem_u32(sm + C::OFF_Q + 2 * g * C::kQTerm);
          uint32_t amax = 0;  // the thread's own row's largest magnitude in bf16 bits; from 0x7f80 on: not finite
#pragma unroll 1
          for (int i0 = 0; i0 < IT; i0 += 4) {
            uint4 u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int y = first + (i0 + i) * RPI, in = base + (split ? y % 64 : y), of = w.p_mt * M + in;
              const int tok = paged_div(a, of);
              u[i] = ld_if(reinterpret_cast<const uint8_t*>(a.q) +
                               2 * ((w.p_s.q0 + tok) * a.q_stride + (int64_t)(w.p_h * a.G + of - tok * a.G) * D + c * 8),
                           in < rows);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // two magnitudes, whose bits' order is the numbers'
              uint32_t top = __vmaxu2(__vmaxu2(u[i].x & 0x7fff7fffu, u[i].y & 0x7fff7fffu),
                                      __vmaxu2(u[i].z & 0x7fff7fffu, u[i].w & 0x7fff7fffu));
#pragma unroll
              for (int o = LPR / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
              top = max(top & 0xffffu, top >> 16);
              const uint32_t own = __shfl_sync(0xffffffffu, top, lane % RPI * LPR);
              if (lane / RPI == i0 + i) amax = own;
              if (shared && g == 1) continue;  // the first warpgroup lays them out
              const int up = top ? 134 - (int)(top >> 7) : 0;
              const uint32_t wd[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
              uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float y0 = times_pow2(__uint_as_float(wd[q] << 16), up),
                            y1 = times_pow2(__uint_as_float(wd[q] & 0xffff0000u), up);
                const uint16_t hc = e4m3x2_code(y0, y1);
                const float2 h = e4m3x2_val(hc);
                hi[q / 2] |= (uint32_t)hc << (16 * (q & 1));
                lo[q / 2] |= (uint32_t)e4m3x2_code(y0 - h.x, y1 - h.y) << (16 * (q & 1));
              }
              const uint32_t at = dst + swz<D>(first + (i0 + i) * RPI, c * 8);
              st_shared8(at, hi[0], hi[1]);
              st_shared8(at + C::kQTerm, lo[0], lo[1]);
            }
          }
          const int ex = amax ? (int)(amax >> 7) - 134 : 0;
          // a query that is not finite gives scores that are not numbers
          r.rf = amax < 0x7f80u ? times_pow2(1.f, ex) : NAN;
        }
        // The second warpgroup may be a piece ahead of the first where it has no
        // tile of keys, so it arrives for its own tile only.
        fence_async_smem();
        __syncwarp();
        if (lane == 0 && !(shared && g == 1)) mbar_arrive(&q_full[g]);
      }
      if (!(ok = wait(ref_full, (uint32_t)pieces & 1u))) break;
      ++pieces;
      const float vref = __int_as_float(*vref_s);
      float m_ref = -INFINITY, l = 0.f;
      // Lane i holds the K scale (times the softmax's) of the keys 16 (i % 8) .. of
      // the i / 8th of four tiles; the next four tiles' pages are looked up with these four's
      // scales, and their scales asked for a batch ahead.
      const PageAhead<M, TK> pages(a, w, keys);
      static_assert(12 * TK <= kPagedAhead, "positions of eleven tiles behind the last");
      auto entry = [&](int t) { return pages.entry(t + lane / 8, (t + lane / 8) * TK + (lane % 8) * 16); };
      if (work) {
        const int64_t ph0 = pages.place(entry(keys.t0));
        int32_t e1 = entry(keys.t0 + 4);
        float ks = -1.f, ks_next = ld_if(a.k_scale + ph0, ph0 >= 0, -1.f);
        const uint32_t prow = smem_u32(sm + C::OFF_P + g * C::kP);
        const int t_first = keys.t0 + (shared ? g : 0), t_step = shared ? 2 : 1;
        for (int t = t_first; t < keys.t1; t += t_step) {
          const int of4 = (t - keys.t0) & 3;
          if (of4 < t_step) {  // the first of four tiles, or of this warpgroup's two of them
            ks = ks_next * c2;
            const int64_t ph1 = pages.place(e1);
            ks_next = ld_if(a.k_scale + ph1, ph1 >= 0, -1.f);
            e1 = entry(t - of4 + 8);
          }
          const int j0 = t * TK;
          const bool inside = __all_sync(0xffffffffu, r.lo <= j0 && r.hi >= j0 + TK && (lane / 8 != of4 || ks >= 0.f));
          if (!(ok = wait(&s_full[g], (uint32_t)cnt & 1u))) break;
          tc_fence_after();
          bool plain = !GEN && inside;  // the products are the scores but for a factor
          float top;
          if constexpr (GEN) {
            top = many_top<kScores>(a, r, cap2, ks, 8 * of4, j0, inside, s_addr, h0, h1);
          } else {
            if (plain) {
              top = many_top<kPlain>(a, r, cap2, ks, 8 * of4, j0, inside, s_addr, h0, h1);
              // (scores from 2^20 on are rounded before the maximum is taken from
              // them: weights of unrounded ones could pass f16's range)
              plain = __all_sync(0xffffffffu, fabsf(top) < kBig);
            }
            if (!plain) top = many_top<kMasked>(a, r, cap2, ks, 8 * of4, j0, inside, s_addr, h0, h1);
          }
          if (split) {
            float other;
            if (!(ok = swapped(top, &other))) break;
            top = fmaxf(top, other);
          }
          const bool fresh = t == t_first;
          float alpha = 1.f;
          bool grown = false;
          if (top - m_ref > kLazy || (fresh && top > -INFINITY)) {
            const float ref = fabsf(top) < kBig ? top - kDrop : top;
            alpha = paged_ex2(m_ref - ref);  // before the first key: 0
            grown = !fresh;
            m_ref = ref;
            l *= alpha;
          }
          // P and O: the last tile's P V has read and added to them
          if (!fresh && !(ok = wait(&pv_done[g], (uint32_t)(cnt - 1) & 1u))) break;
          if (side == 0 && __any_sync(0xffffffffu, grown)) {
            tc_fence_after();
            many_rescale<D>(o_addr, alpha);
          }
          const float ref = m_ref == -INFINITY ? 0.f : m_ref;
          const uint64_t ref2 = pack2(-ref, -ref);
          uint64_t sum2 = pack2(0.f, 0.f);
#pragma unroll 1
          for (int h = h0; h < h1; h += 32) {
            uint32_t x[32], pk[16];
            tmem_ld(s_addr + h, x);
            const float k0 = __shfl_sync(0xffffffffu, ks, 8 * of4 + (h >> 4)),
                        k1 = __shfl_sync(0xffffffffu, ks, 8 * of4 + (h >> 4) + 1);
            const float c0 = plain ? k0 * r.rf : 1.f, c1 = plain ? k1 * r.rf : 1.f;
            const uint64_t c02 = pack2(c0, c0), c12 = pack2(c1, c1);
            tmem_ld_done(x);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float y0, y1;
              unpack2(fma2(pack2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), i < 16 ? c02 : c12, ref2), y0, y1);
              const float p0 = paged_ex2(y0), p1 = paged_ex2(y1);
              sum2 = add2(sum2, pack2(p0, p1));
              const __half2 hp = __floats2half2_rn(p0, p1);
              pk[i / 2] = *reinterpret_cast<const uint32_t*>(&hp);
            }
            const uint32_t at = prow + (h >> 6) * (128 * 128);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              st_shared16(at + swz<128>(t_row, (h & 32) * 2 + i * 16), pk[4 * i], pk[4 * i + 1], pk[4 * i + 2],
                          pk[4 * i + 3]);
          }
          float s0, s1;
          unpack2(sum2, s0, s1);
          l += s0 + s1;
          fence_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[g]);
          ++cnt;
        }
        if (ok && t_first < keys.t1) ok = wait(&pv_done[g], (uint32_t)(cnt - 1) & 1u);
        if (ok && split) {
          float other;
          ok = swapped(l, &other);
          l += other;
        }
        tc_fence_after();
      }
      if (!ok) break;
      float f_own = 1.f, f_other = 0.f;  // of O in this warpgroup's and the other's columns
      if (shared && work) {
        if (g == 1) {
          ml_s[row_in] = make_float2(m_ref, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ml_full);
        } else {
          if (!(ok = wait(ml_full, (uint32_t)merges & 1u))) break;
          tc_fence_after();
          const float2 o = ml_s[row_in];
          const float m = fmaxf(m_ref, o.x), ref = m == -INFINITY ? 0.f : m;
          f_own = paged_ex2(m_ref - ref);
          f_other = paged_ex2(o.x - ref);
          l = fmaf(l, f_own, o.y * f_other);
          m_ref = m;
        }
        ++merges;
      }
      // O (times 2^7 / vref), the row's maximum and sum
      if (!(shared && g == 1) && side == 0) {
        const float unit = vref * (1.f / 128.f);
        int64_t at = 0;
        const int64_t part = w.slot() * M + r_in;
        float f = unit;
        if (mine && w.whole()) {
          f *= paged_close(a, w.p_s, w.p_h, row, m_ref, l, true, &at);
        } else if (mine) {
          a.part_ml[part * 2] = m_ref;
          a.part_ml[part * 2 + 1] = l;
        }
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t o[32];
          if (work) {
            tmem_ld(o_addr + d, o);
            tmem_ld_done(o);
          }
          if (shared && keys.t0 + 1 < keys.t1) {  // the other warpgroup had keys
            uint32_t x[32];
            tmem_ld(o_addr + 128 + d, x);
            tmem_ld_done(x);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(fmaf(__uint_as_float(o[i]), f_own, __uint_as_float(x[i]) * f_other));
          }
          if (!mine) continue;
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(work && f != 0.f ? __uint_as_float(o[i]) * f : 0.f);
          if (w.whole()) {
            uint4* out = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + at * D + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t pk[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                pk[q] = (uint32_t)bf16_code(__uint_as_float(o[8 * i + 2 * q])) |
                        ((uint32_t)bf16_code(__uint_as_float(o[8 * i + 2 * q + 1])) << 16);
              out[i] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
          } else {
            uint4* out = reinterpret_cast<uint4*>(a.part_o + part * D + d);
#pragma unroll
            for (int i = 0; i < 8; ++i) out[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(piece_done);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // as in paged_few_kernel: copies in flight where a role gave up
  if (warp == 12 && *abort)
    for (int i = copied > 2 ? copied - 2 : 0; i < copied; ++i)
      mbar_wait(&k_full[i & 1], (uint32_t)(i >> 1) & 1u, a.status, kDrainLimitNs);
  if (warp == 13) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- host side

PFN_cuTensorMapEncodeTiled_v12000 tiled_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// The pool's codes as rows of D bytes; a box is `rows` of them (16-byte aligned
// base, D a multiple of 16, every copy from column 0).
bool map_pool(CUtensorMap* m, const PagedLaunch& a, const void* base, int rows) {
  auto fn = tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)a.D, (cuuint64_t)a.n_pages * a.Hkv * a.page};
  cuuint64_t strides[1] = {(cuuint64_t)a.D};
  cuuint32_t box[2] = {(cuuint32_t)a.D, (cuuint32_t)rows};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, a.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NR>
cudaError_t launch_few(const PagedLaunch& a, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
  using C = FewCfg<D, NR>;
  auto kern = a.cap > 0.f ? paged_few_kernel<D, NR, true> : paged_few_kernel<D, NR, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.ctas), dim3(kFewThreads), C::SMEM, stream, a, k, v, wait_test());
}

template <int D>
cudaError_t launch_many(const PagedLaunch& a, const CUtensorMap& k, cudaStream_t stream) {
  if (a.block_docs) {
    const int64_t y = (a.n_tokens * a.G / kManyRows + 8) / 8;
    const cudaError_t e = launch_pdl(paged_docs_kernel, dim3(a.B, (unsigned)(y < 64 ? y : 64)), dim3(256), 0, stream, a);
    if (e != cudaSuccess) return e;
  }
  auto kern = a.cap > 0.f || a.slopes ? paged_many_kernel<D, true> : paged_many_kernel<D, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ManyCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.ctas), dim3(kManyThreads), ManyCfg<D>::SMEM, stream, a, k, wait_test());
}

template <int D>
cudaError_t launch_mma(const PagedLaunch& a, const PagedForm& f, const CUtensorMap& k, const CUtensorMap& v,
                       cudaStream_t stream) {
  if (f.kind == 2) return launch_many<D>(a, k, stream);
  switch (f.rows) {
    case 8: return launch_few<D, 8>(a, k, v, stream);
    default: return launch_few<D, 16>(a, k, v, stream);
  }
}

}  // namespace

PagedForm paged_mma_form(int D, int G, int64_t max_new) {
  // Few rows: up to 16 per KV head and request.  From 17 on two warpgroups over
  // 128 rows are faster, however many of them are empty (16 requests of 4K to
  // 32K tokens, 8 KV heads, us: D = 128, 8 rows 110 against 201, 16 rows 146
  // against 205, 32 rows 307 with a few-rows kernel of that size against 208;
  // D = 64, 8 rows 99 against 165, 16 rows 143 against 166, 32 rows 291 against
  // 170).  One form serves the call: 32 decodes at 16K to 64K tokens beside a
  // chunk of 2048 take 2,138 us, in two calls 467 and 712.
  const int64_t rows = max_new > 16 ? 17 : max_new * G;
  if (rows > 16) return {2, kManyRows, sm_count()};
  return {1, rows <= 8 ? 8 : 16, 2 * sm_count()};
}

cudaError_t launch_paged_mma(const PagedLaunch& a, const PagedForm& f, cudaStream_t stream) {
  CUtensorMap k, v;
  if (!map_pool(&k, a, a.k, a.page) || !map_pool(&v, a, a.v, a.page)) return cudaErrorInvalidValue;
  return a.D == 128 ? launch_mma<128>(a, f, k, v, stream) : launch_mma<64>(a, f, k, v, stream);
}

}  // namespace lcsc
