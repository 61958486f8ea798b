// The choices over a paged cache and the moves that follow them: the best pages of each query
// group, the tokens that an eviction keeps, and the move of kept tokens to the front.
//
// Top k of a row of floats: the row's keys (floats mapped to unsigned integers of the same order)
// are counted in four buckets a thread that evenly divide the range still in question, the bucket
// holding the k-th largest becomes the next range, and so on; once that bucket holds at most
// kDirect keys they are ranked against each other directly, mostly after one round (four rounds
// at most for 32-bit keys).  One CTA per row, everything after the first read in shared memory
// where it fits.  The buckets divide the range in use (min .. max first), not fixed bits of the
// key: rows of similar values would otherwise fall into a few buckets, whose counters then
// serialise.  Ties at the k-th value go to the lowest index, and the output is in index order, so
// nothing depends on the order in which threads run.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "cache_ops.h"
#include "page_mma.cuh"
#include "ptx.cuh"

namespace bdlm {
namespace {

constexpr int kTok = 16;       // tokens per page
constexpr int kRowThreads = 512;   // threads of a CTA that works on a long row
constexpr int kDirect = 128;   // keys ranked directly, four lanes a key (in the counters' memory)

// Unsigned key with the floats' order; -0 and +0 are equal, NaN comes below every number.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 0;
  const uint32_t u = __float_as_uint(f + 0.0f);   // -0 -> +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float key_value(uint32_t key) {   // of order_key (not NaN)
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

struct BlockSum {   // sums and scans over the CTA; s: one word per warp
  int* s;
  __device__ __forceinline__ int exclusive(int v, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    __syncthreads();
    if (lane == 31) s[warp] = x;
    __syncthreads();
    const int w = lane < warps ? s[lane] : 0;
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
    const int all = __reduce_add_sync(0xffffffffu, w);
    *total = all;
    return before + x - v;
  }
};

// Minimum and maximum over the CTA (every thread gets both); s: 64 values.
template <typename T>
__device__ __forceinline__ void block_range(T& lo, T& hi, T* s) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  auto warp_range = [&]() {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const T a = __shfl_xor_sync(0xffffffffu, lo, off), b = __shfl_xor_sync(0xffffffffu, hi, off);
      lo = a < lo ? a : lo;
      hi = b > hi ? b : hi;
    }
  };
  warp_range();
  __syncthreads();
  if (lane == 0) {
    s[threadIdx.x >> 5] = lo;
    s[32 + (threadIdx.x >> 5)] = hi;
  }
  __syncthreads();
  lo = s[lane < warps ? lane : 0];
  hi = s[32 + (lane < warps ? lane : 0)];
  warp_range();
}

// The same by ranking `count` <= kDirect keys, listed in `few`, against each other (after a
// barrier).  Whole CTA.
template <typename K>
__device__ __forceinline__ K kth_of_few(int k, const K* few, int count, int* s_scan, K* s_pick,
                                        int* above) {
  for (int c = static_cast<int>(threadIdx.x) >> 2; (c & ~7) < count;   // whole warps
       c += static_cast<int>(blockDim.x) >> 2) {
    const K key = few[c < count ? c : 0];
    int more = 0, same = 0;
#pragma unroll 8
    for (int i = threadIdx.x & 3; i < count; i += 4) {
      const K other = few[i];
      more += other > key;
      same += other == key;
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      more += __shfl_xor_sync(0xffffffffu, more, off);
      same += __shfl_xor_sync(0xffffffffu, same, off);
    }
    if (c < count && more < k && more + same >= k) {   // equal keys write the same
      s_pick[0] = key;
      s_scan[33] = more;
    }
  }
  __syncthreads();
  const K kth = s_pick[0];
  *above = s_scan[33];
  __syncthreads();
  return kth;
}

// The k-th largest of the keys that `each` yields (each(f): calls f(key) for this thread's share,
// the same keys every time), 1 <= k <= their number, all within [lo, hi].  Returns it, and in
// *above how many are larger.  hist: four counters a thread.  Whole CTA of THREADS.
template <int THREADS, typename K, typename Each>
__device__ __forceinline__ K kth_largest(int k, K lo, K hi, Each&& each, int* hist, int* s_scan,
                                         K* s_pick, int* above) {
  constexpr int kBuckets = 4 * THREADS, kLog = THREADS == 512 ? 11 : THREADS == 256 ? 10 : 9;
  static_assert(kBuckets == 1 << kLog, "");
  int larger = 0;
  BlockSum sum{s_scan};
  K* few = reinterpret_cast<K*>(hist);
  while (lo < hi) {
    const K range = hi - lo;
    int bits = sizeof(K) == 8 ? 64 - __clzll(static_cast<long long>(range))
                              : 32 - __clz(static_cast<int>(range));
    const int shift = bits > kLog ? bits - kLog : 0;
    reinterpret_cast<int4*>(hist)[threadIdx.x] = make_int4(0, 0, 0, 0);
    __syncthreads();
    each([&](K key) {
      const K off = key - lo;   // (below lo: wraps past the range)
      if (off <= range) atomicAdd(&hist[static_cast<int>(off >> shift)], 1);
    });
    __syncthreads();
    // this thread's four buckets, counted from the top
    const int4 h4 = reinterpret_cast<const int4*>(hist)[THREADS - 1 - threadIdx.x];
    const int mine[4] = {h4.w, h4.z, h4.y, h4.x};
    int total;
    int before = larger + sum.exclusive(mine[0] + mine[1] + mine[2] + mine[3], &total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (before < k && before + mine[i] >= k) {
        s_pick[0] = static_cast<K>(kBuckets - 1 - (static_cast<int>(threadIdx.x) * 4 + i));
        s_scan[33] = before;
        s_scan[34] = mine[i];
        s_scan[35] = 0;
      }
      before += mine[i];
    }
    __syncthreads();
    const K from = lo + (s_pick[0] << shift), width = (static_cast<K>(1) << shift) - 1;
    larger = s_scan[33];
    const int count = s_scan[34];
    if (hi - from > width) hi = from + width;
    lo = from;
    if (count <= kDirect && lo < hi) {
      const K span = hi - lo;
      each([&](K key) {
        if (key - lo <= span) few[atomicAdd(&s_scan[35], 1)] = key;
      });
      __syncthreads();
      int more;
      lo = kth_of_few(k - larger, few, count, s_scan, s_pick, &more);
      larger += more;
      break;
    }
    __syncthreads();
  }
  __syncthreads();
  *above = larger;
  return lo;
}

// ------------------------------------------------------------------ page selection
constexpr int kSelThreads = kRowThreads;
constexpr int kSelOwnPages = 512;    // pages of lists that the kernel scores itself
constexpr int kSelFewThreads = 128, kSelFewRows = 64;   // the variant for many short lists
constexpr int kOwn = 8;              // keys of a thread in registers
constexpr int kSelKeys = 12288;      // rows held in shared memory (96 KB); longer ones are re-read
constexpr int kSelExact = 1024;      // near ties held in shared memory

// The 16 chunks of query n of a group (n < 256: its position n / G, head n % G; G <= 16, so the
// division is a product).
__device__ __forceinline__ const uint4* group_query(const SelectParams& p, int b, int s, int kvh,
                                                    int n) {
  const int i = (n * ((65536 + p.G - 1) / p.G)) >> 16;
  return reinterpret_cast<const uint4*>(p.q) +
         ((static_cast<size_t>(b) * p.L + s * p.group + i) * p.Hq + kvh * p.G + (n - i * p.G)) * 16;
}

constexpr int kExactRows = 16;   // query rows of a warp's turn

// Scores of one page for query rows row0 .. rows - 1 (at most 16) of one group, in float32 with 11
// roundings of partial sums.  Whole warp, 16 lanes a row, two rows at a time: lane l has that of row
// near_row(l), lanes l % 16 >= 8 have -inf.  (All 16 rows' queries in registers at once, their sums
// crossed over the lanes together, takes fewer instructions but more code, which is read anew by
// every launch: 58 us a call against 53, 16 x 8 lists of 1875-3750 pages.)
__device__ __forceinline__ int near_row(int l) { return 2 * (l & 15) + (l >> 4); }
__device__ __forceinline__ float float_scores(const SelectParams& p, int b, int s, int kvh, int id,
                                              int row0, int rows) {
  const int c16 = threadIdx.x & 15, half = (threadIdx.x >> 4) & 1;
  const uint4* page = reinterpret_cast<const uint4*>(p.bounds) +
                      (static_cast<size_t>(id) * p.Hkv + kvh) * 32 + c16;
  const uint4 lo = __ldg(page), hi = __ldg(page + 16);
  const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, h[4] = {hi.x, hi.y, hi.z, hi.w};
  float mine = -CUDART_INF_F;
#pragma unroll 4
  for (int x = 0; x < kExactRows / 2; ++x) {
    const uint4 v = __ldg(group_query(p, b, s, kvh, min(row0 + 2 * x + half, rows - 1)) + c16);
    const uint32_t q[4] = {v.x, v.y, v.z, v.w};
    float f = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float q0 = bf16_lo(q[k]), q1 = bf16_hi(q[k]);
      f = fmaf(q0, q0 > 0.f ? bf16_lo(h[k]) : bf16_lo(l[k]), f);
      f = fmaf(q1, q1 > 0.f ? bf16_hi(h[k]) : bf16_hi(l[k]), f);
    }
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) f += __shfl_xor_sync(0xffffffffu, f, off);
    mine = c16 == x ? f : mine;
  }
  return mine;
}
__device__ __forceinline__ float warp_most(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// a + b as s + e exactly (Knuth's TwoSum)
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float bb = __fadd_rn(s, -a);
  e = __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -bb)), __fadd_rn(b, -bb));
}

// The largest score of one page over the rows of one group whose float32 score (`mine`, of rows row0 ..)
// is at least `from`, to about 2^-45 of its terms, as an ordered 64-bit key (never 0 or 1; 0: no such
// row): the products of two bf16 are exact in float32, and are added with the rounding errors
// carried along.  Whole warp.
__device__ __forceinline__ unsigned long long exact_score(const SelectParams& p, int b, int s,
                                                          int kvh, int id, int row0, int rows,
                                                          float mine, float from) {
  const int lane = threadIdx.x & 31;
  const uint2* page = reinterpret_cast<const uint2*>(p.bounds) +
                      (static_cast<size_t>(id) * p.Hkv + kvh) * 64 + lane;
  unsigned long long best = 0;
  for (uint32_t near = __ballot_sync(0xffffffffu, mine >= from && (lane & 15) < kExactRows / 2); near;
       near &= near - 1) {
    const int n = min(row0 + near_row(__ffs(static_cast<int>(near)) - 1), rows - 1);
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(group_query(p, b, s, kvh, n)) + lane);
    const uint2 lo = __ldg(page), hi = __ldg(page + 32);
    const float lv[4] = {bf16_lo(lo.x), bf16_hi(lo.x), bf16_lo(lo.y), bf16_hi(lo.y)};
    const float hv[4] = {bf16_lo(hi.x), bf16_hi(hi.x), bf16_lo(hi.y), bf16_hi(hi.y)};
    const float qv[4] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
    float a = 0.f, e = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float r;
      two_sum(a, __fmul_rn(qv[k], qv[k] > 0.f ? hv[k] : lv[k]), a, r);
      e = __fadd_rn(e, r);
    }
#pragma unroll 1
    for (int off = 16; off > 0; off >>= 1) {
      const float a2 = __shfl_xor_sync(0xffffffffu, a, off);
      const float e2 = __shfl_xor_sync(0xffffffffu, e, off);
      float r;
      two_sum(a, a2, a, r);
      e = __fadd_rn(__fadd_rn(e, e2), r);
    }
    float top, rest;
    two_sum(a, e, top, rest);   // normalised: top decides, then rest
    const unsigned long long key =
        static_cast<unsigned long long>(order_key(top)) << 32 | order_key(rest);
    best = key > best ? key : best;
  }
  return best;
}

// One CTA per (sequence, query group, KV head).  The scores come from the tensor core in float32;
// where two of them lie closer than their rounding could explain, float32 does not say which is
// larger.  So with T the k-th largest and E a bound on a score's error, pages above T + 2E are
// in, pages below T - 2E are out, and the few between are scored again: in float32 with few
// roundings, whose bound is 1/45 of E and settles nearly all; where it does not, to about 45 bits.
//   E = 16 * 17 * 2^-23 max_n |q_n|_1 max |bound|: a score sums 128 products (and 128 zeros) in 16
//   MMAs of 16, each of which rounds or truncates at most 17 values by 2^-23 of the largest
//   partial sum, and no partial sum exceeds |q|_1 max|bound|.
// Bound by latency: a dozen barriers and half a dozen loads that depend on each other.  So what can
// be asked for early is, a thread keeps its first eight keys in registers, and the exact scores
// of one page are spread over warps.
// 512 threads and CTAS 1, with all the registers it wants, for no more lists than SMs (128 lists of
// 1875-3750 pages: a call of 52 us against 56 with two CTAs per SM); CTAS 2 for more lists (1024 of
// 125-375 pages: 70 against 83).  128 threads, six CTAs per SM, for more lists than that has places
// for, of pages that fit the registers (the same 1024 lists 54 against 70, 2048 lists 54 against 87,
// 512 lists 38 against 44; with 128 lists of 500-1000 pages it loses, 33 against 29) and of up to 64
// query rows, which near ties need warps for (512 lists of 256 rows: 105 against 85).
//
// NT > 0: the kernel scores its list's pages itself, for up to 8 NT query rows and kSelOwnPages pages,
// which saves the scores' launch and their way through memory (8 lists of 125 pages and 8 rows: 8.7 us
// a call against 11.2; 128 lists of 62-187 pages and 32 rows: 17 against 23; at 500 pages a list it
// is even).
template <int THREADS, int CTAS, int NT = 0>
__global__ void __launch_bounds__(THREADS, CTAS)
select_pages_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint32_t sm[];
  __shared__ __align__(16) int hist[4 * THREADS];
  __shared__ unsigned long long s_exact[kSelExact];
  __shared__ uint32_t s_fast[kSelExact];
  __shared__ int s_page[kSelExact];
  __shared__ int s_scan[36];
  __shared__ unsigned long long s_wide[64];
  __shared__ unsigned long long s_pick[1];
  __shared__ int s_cand;
  __shared__ float s_f[32];
  __shared__ __align__(16) uint8_t sQ[NT > 0 ? NT * 8 * kDirectPitch : 16];
  __shared__ float s_score[NT > 0 ? kSelOwnPages : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = THREADS / 32;
  const int list = blockIdx.x;
  const int kvh = list % p.Hkv, bs = list / p.Hkv;
  const int b = bs / p.groups, s = bs - b * p.groups;
  griddep_wait();
  griddep_launch_dependents();
  const int prefix = p.prefix_lens[b];
  int32_t* out = p.sel_table + static_cast<size_t>(list) * p.sel_cols;
  const bool bad = prefix < 0 || static_cast<long long>(prefix) + p.L >
                                     static_cast<long long>(p.max_pages) * kTok;
  const int n = bad ? 0 : prefix / kTok;
  const int k = n < p.n_select ? n : p.n_select;
  const int tail = bad ? 0 : (prefix % kTok + p.L + kTok - 1) / kTok;
  if (kvh == 0 && tid == 0) {
    p.sel_lens[bs] = bad ? -1 : k * kTok + prefix % kTok + p.L - p.group;
    if (bad && s == 0) atomicOr(p.err, BDLM_DEVERR_LENGTH);
  }
  const int32_t* pt = p.page_table + static_cast<size_t>(b) * p.max_pages;
  // the unfinished page and the block's pages follow the selected ones; unused columns hold -1
  const int c0 = k + tid;
  const int32_t last = c0 < k + tail ? pt[n + tid] : -1;
  auto finish = [&]() {
    if (c0 < p.sel_cols) out[c0] = last;
    for (int c = c0 + THREADS; c < p.sel_cols; c += THREADS) out[c] = -1;   // (tail <= 5)
  };
  if (n <= p.n_select || k == 0) {
    for (int c = tid; c < (NT > 0 ? n : k); c += THREADS) {
      const int id = pt[c];
      if (c < k) out[c] = id;
      if (NT > 0 && (id < 0 || id >= p.num_pages)) atomicOr(p.err, BDLM_DEVERR_PAGE);
    }
    finish();
    return;
  }

  // ---- keys, magnitudes and queries: all asked for before any is used
  const float* row = NT > 0 ? s_score : p.scores + static_cast<size_t>(list) * p.max_pages;
  float early[kOwn];
  if constexpr (NT == 0) {
#pragma unroll
    for (int x = 0; x < kOwn; ++x)
      early[x] = tid + x * THREADS < n ? __ldcg(row + tid + x * THREADS) : 0.f;
  }
  if (n <= kSelKeys)   // the page ids go to shared memory meanwhile
    for (int i = tid; i < n; i += THREADS)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(sm + i)), "l"(pt + i)
                   : "memory");
  float q1 = 0.f, am = 0.f;   // the group's largest |q|_1, the list's largest |bound|
  if constexpr (NT == 0) {
    const int values = (n + kKeyTile - 1) / kKeyTile * kAmaxPerTile;
    const float* a = p.amax + (static_cast<size_t>(b) * p.Hkv + kvh) * p.max_tiles * kAmaxPerTile;
    for (int i = tid; i < values; i += THREADS) am = fmaxf(am, __ldcg(a + i));
  } else {
    // each warp scores 16 pages at a time; its first pages' bounds and the queries are asked for
    // together
    const int g = lane >> 2, t = lane & 3, rows = p.group * p.G;
    bool live[2];
    uint4 a[8][2];
    auto load = [&](int first) {   // pages g and g + 8
      int id[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int page = first + r * 8 + g;
        id[r] = page < n ? __ldg(pt + page) : -1;
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        live[r] = id[r] >= 0 && id[r] < p.num_pages;
        if (!live[r] && first + r * 8 + g < n && t == 0) atomicOr(p.err, BDLM_DEVERR_PAGE);
        load_page(p.bounds, id[r], live[r], p.Hkv, kvh, t, r, a);
      }
    };
    load(warp * 16);
    for (int c = tid; c < NT * 8 * 16; c += THREADS) {
      const int r = c >> 4, cc = c & 15;
      stage_query(sQ, r, cc, r < rows ? __ldg(group_query(p, b, s, kvh, r) + cc) : make_uint4(0, 0, 0, 0));
    }
    __syncthreads();
    uint32_t top = 0;
    for (int first = warp * 16; first < n;) {
      float d[NT][4], best[2] = {-CUDART_INF_F, -CUDART_INF_F};
      page_products<NT>(a, sQ, g, t, d, top);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (nt * 8 + 2 * t + x < rows) {
            best[0] = fmaxf(best[0], d[nt][x]);
            best[1] = fmaxf(best[1], d[nt][2 + x]);
          }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
        best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
        const int page = first + r * 8 + g;
        if (t == 0 && page < n) s_score[page] = live[r] ? best[r] : -CUDART_INF_F;
      }
      first += kWarps * 16;
      if (first < n) load(first);
    }
    am = warp_magnitude(top);
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kOwn; ++x)
      early[x] = tid + x * THREADS < n ? s_score[tid + x * THREADS] : 0.f;
  }
  for (int r = tid >> 1; r < p.group * p.G; r += THREADS / 2) {   // a row for two threads
    const uint4* src = group_query(p, b, s, kvh, r) + (tid & 1) * 8;
    uint4 q[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) q[x] = __ldg(src + x);
    float v = 0.f;
#pragma unroll
    for (int x = 0; x < 8; ++x)
      v += (fabsf(bf16_lo(q[x].x)) + fabsf(bf16_hi(q[x].x))) + (fabsf(bf16_lo(q[x].y)) + fabsf(bf16_hi(q[x].y))) +
           ((fabsf(bf16_lo(q[x].z)) + fabsf(bf16_hi(q[x].z))) + (fabsf(bf16_lo(q[x].w)) + fabsf(bf16_hi(q[x].w))));
    q1 = fmaxf(q1, v);
  }
  q1 += __shfl_xor_sync(0xffffffffu, q1, 1);   // (each half row's largest: not less than the row's)
#pragma unroll
  for (int off = 16; off > 1; off >>= 1) q1 = fmaxf(q1, __shfl_xor_sync(0xffffffffu, q1, off));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, off));
  if (lane == 0) {
    s_f[warp] = q1;
    s_f[16 + warp] = am;
  }
  // shared memory: page ids, then keys past the registers' share (rows of up to kSelKeys; longer
  // ones are read again each time), then the page bitmap and a second one
  uint32_t own[kOwn];
  const bool held = n <= kSelKeys;
  int32_t* ids = reinterpret_cast<int32_t*>(sm);
  uint32_t* keys = sm + n;
  uint32_t* taken = sm + (held ? (n > kOwn * THREADS ? 2 * n : n) : 0);
  const int words = (n + 31) / 32;
  uint32_t* second = taken + words;
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll
  for (int x = 0; x < kOwn; ++x) {
    own[x] = order_key(early[x]);
    if (tid + x * THREADS >= n) continue;
    lo = min(lo, own[x]);
    hi = max(hi, own[x]);
  }
  for (int i = tid + kOwn * THREADS; i < n; i += THREADS) {
    const uint32_t key = order_key(__ldcg(row + i));
    if (held) keys[i] = key;
    lo = min(lo, key);
    hi = max(hi, key);
  }
  for (int i = tid; i < words; i += THREADS) taken[i] = 0;
  if (tid == 0) s_cand = 0;
  asm volatile("cp.async.wait_all;" ::: "memory");
  auto page_id = [&](int i) { return held ? ids[i] : __ldg(pt + i); };
  // f(i, key) for this thread's keys
  auto each_key = [&](auto&& f) {
#pragma unroll
    for (int x = 0; x < kOwn; ++x)
      if (tid + x * THREADS < n) f(tid + x * THREADS, own[x]);
    for (int i = tid + kOwn * THREADS; i < n; i += THREADS)
      f(i, held ? keys[i] : order_key(__ldcg(row + i)));
  };

  // ---- T, the k-th largest
  int above;
  uint32_t T;
  uint32_t* pick = reinterpret_cast<uint32_t*>(s_pick);
  if (n <= kDirect) {
    uint32_t* few = reinterpret_cast<uint32_t*>(hist);
    each_key([&](int i, uint32_t key) { few[i] = key; });
    __syncthreads();
    T = kth_of_few<uint32_t>(k, few, n, s_scan, pick, &above);
  } else {
    block_range(lo, hi, reinterpret_cast<uint32_t*>(s_wide));
    T = kth_largest<THREADS, uint32_t>(
        k, lo, hi, [&](auto&& f) { each_key([&](int, uint32_t key) { f(key); }); }, hist, s_scan,
        pick, &above);
  }

  // ---- the band around T
  q1 = s_f[lane & (kWarps - 1)];
  am = s_f[16 + (lane & (kWarps - 1))];
#pragma unroll
  for (int off = kWarps / 2; off > 0; off >>= 1) {
    q1 = fmaxf(q1, __shfl_xor_sync(0xffffffffu, q1, off));
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, off));
  }
  const float band = q1 * am * (2 * 16 * 17 * 0x1p-23f);   // 2E
  const float t = key_value(T);
  // (scores or bounds that are not finite, or whose sums may not be, have no error bound: their
  // float32 order stands)
  const bool refine = T != 0 && q1 * am <= 1e38f && fabsf(t) <= 3e38f;
  const uint32_t k_hi = refine ? order_key(__fadd_ru(t, band)) : T;
  const uint32_t k_lo = refine ? order_key(__fadd_rd(t, -band)) : T;
  auto take = [&](int i) { atomicOr(&taken[i >> 5], 1u << (i & 31)); };
  int sure = 0;
  each_key([&](int i, uint32_t key) {
    if (key > k_hi) {
      take(i);
      ++sure;
    } else if (key >= k_lo) {
      const int c = atomicAdd(&s_cand, 1);
      if (c < kSelExact) {
        s_page[c] = i;
        s_fast[c] = 0;
        s_exact[c] = 0;
      }
    }
  });
  BlockSum sum{s_scan};
  int n_sure;
  sum.exclusive(sure, &n_sure);
  const int m = s_cand;
  int need = k - n_sure;   // how many of the m candidates are in (>= 1)
  if (m == need) {
    each_key([&](int i, uint32_t key) {
      if (key >= k_lo && key <= k_hi) take(i);
    });
  } else {
    // Up to kSelExact candidates are listed in shared memory, and a warp takes 16 of their rows.  First
    // their float32 scores; candidates that these leave open then get the exact ones of the rows
    // that can hold their maximum.  More candidates (pages that are copies of each other) keep exact
    // scores in the workspace.
    const bool listed = m <= kSelExact;
    const int rows = p.group * p.G, parts = (rows + kExactRows - 1) / kExactRows;
    // 2 * 12 * 2^-24 max |q|_1 max |bound| as a part of `band`, and some for roundings here
    const float near = band * 0.0235f;
    if (refine && listed) {
      // (a turn for each warp at most: at once the exact ones)
      for (int pass = m * parts <= kWarps ? 1 : 0;; ++pass) {
        for (int x = warp; x < m * parts; x += kWarps) {
          const int c = x / parts, first = (x - c * parts) * kExactRows, i = s_page[c];
          const int id = i >= 0 ? page_id(i) : -1;
          if (id < 0 || id >= p.num_pages) continue;   // (a bad page: below every score)
          const float mine = float_scores(p, b, s, kvh, id, first, rows);
          const float most = warp_most(mine);
          if (pass == 0) {
            if (lane == 0) atomicMax(&s_fast[c], order_key(most));
          } else {
            // the candidate's largest, where the first pass found it (else 0, whose value is NaN)
            const float f = fmaxf(most, key_value(s_fast[c]));
            const unsigned long long e =
                exact_score(p, b, s, kvh, id, first, rows, mine, __fadd_rd(f, -near));
            if (lane == 0 && e != 0) atomicMax(&s_exact[c], e);
          }
        }
        __syncthreads();
        if (pass > 0) break;
        int in = 0, open = 0;   // candidates
        for (int c = tid; c < m; c += THREADS) {
          const float f = key_value(s_fast[c]);
          int ahead = 0, maybe = -1;   // (-1: itself)
          for (int j = 0; j < m; ++j) {
            const float d = key_value(s_fast[j]) - f;
            ahead += d > near;
            maybe += d >= -near;
          }
          const bool out = s_fast[c] == 0 || ahead >= need, sure = !out && maybe < need;
          if (sure) take(s_page[c]);
          if (sure || out) s_page[c] = -1;   // decided
          in += sure;
          open += !sure && !out;
        }
        int n_in, n_open;
        sum.exclusive(in + (open << 16), &n_in);   // (at most 1024 of each)
        n_open = n_in >> 16;
        n_in &= 0xFFFF;
        need = n_open > 0 ? need - n_in : 0;
        if (n_open == 0) break;
      }
    }
    if (need > 0) {
      unsigned long long* exact = p.exact + static_cast<size_t>(list) * p.max_pages;
      unsigned long long elo = ~0ull, ehi = 0;
      if (!listed && refine) {
        each_key([&](int i, uint32_t key) { exact[i] = key >= k_lo && key <= k_hi ? 1 : 0; });
        __syncthreads();
        for (int i = warp; i < n; i += kWarps) {
          if (__ldcg(exact + i) == 0) continue;
          const int id = page_id(i);
          unsigned long long e = 1;   // a bad page: below every score
          if (id >= 0 && id < p.num_pages) {
            float most = -CUDART_INF_F;
            for (int x = 0; x < 2 * parts; ++x) {   // every row's float32 score, then again
              const int first = (x < parts ? x : x - parts) * kExactRows;
              const float mine = float_scores(p, b, s, kvh, id, first, rows);
              if (x < parts) {
                most = fmaxf(most, warp_most(mine));
                continue;
              }
              const unsigned long long part =
                  exact_score(p, b, s, kvh, id, first, rows, mine, __fadd_rd(most, -near));
              e = part > e ? part : e;
            }
          }
          __syncwarp();
          if (lane == 0) exact[i] = e;
          elo = e < elo ? e : elo;
          ehi = e > ehi ? e : ehi;
        }
      }
      __syncthreads();
      int equal = need;   // how many of `second`, the candidates equal to the last one in, are in
      for (int i = tid; i < words; i += THREADS) second[i] = 0;
      if (!refine) {
        __syncthreads();
        each_key([&](int i, uint32_t key) {
          if (key == T) atomicOr(&second[i >> 5], 1u << (i & 31));
        });
      } else if (listed) {
        equal = 0;
        for (int c = tid; c < m; c += THREADS) {
          const unsigned long long e = s_exact[c];
          const int page = s_page[c];
          if (page < 0) continue;
          int rank = 0;   // candidates ahead of this one
          for (int j = 0; j < m; ++j)
            rank += s_exact[j] > e || (s_exact[j] == e && s_page[j] < page);
          if (rank < need) take(page);
        }
      } else {
        block_range(elo, ehi, s_wide);
        int larger;
        const unsigned long long TE = kth_largest<THREADS, unsigned long long>(
            need, elo, ehi,
            [&](auto&& f) {
              for (int i = tid; i < n; i += THREADS) {
                const unsigned long long e = __ldcg(exact + i);
                if (e != 0) f(e);
              }
            },
            hist, s_scan, s_pick, &larger);
        equal = need - larger;
        for (int i = tid; i < n; i += THREADS) {
          const unsigned long long e = __ldcg(exact + i);
          if (e > TE) take(i);
          if (e == TE) atomicOr(&second[i >> 5], 1u << (i & 31));
        }
      }
      __syncthreads();
      int base = 0;   // of equal ones the lowest positions
      for (int w0 = 0; w0 < words && equal > 0; w0 += THREADS) {
        const int w = w0 + tid;
        const uint32_t bits = w < words ? second[w] : 0;
        int total;
        int before = base + sum.exclusive(__popc(bits), &total);
        uint32_t keep = 0;
        for (uint32_t x = bits; x && before < equal; x &= x - 1, ++before) keep |= x & (0u - x);
        if (keep) taken[w] |= keep;
        base += total;
      }
    }
  }
  __syncthreads();

  // ---- the taken pages in position order: where each bitmap word's pages begin, then a thread a page
  int base = 0;
  for (int w0 = 0; w0 < words; w0 += THREADS) {
    const int w = w0 + tid;
    int total;
    const int at = base + sum.exclusive(w < words ? __popc(taken[w]) : 0, &total);
    if (w < words) second[w] = static_cast<uint32_t>(at);
    base += total;
  }
  __syncthreads();
#pragma unroll 4
  for (int i = tid; i < n; i += THREADS) {
    const uint32_t bits = taken[i >> 5], bit = 1u << (i & 31);
    if (bits & bit) out[second[i >> 5] + __popc(bits & (bit - 1))] = page_id(i);
  }
  finish();
}

// ------------------------------------------------------------------ eviction
constexpr int kEvictThreads = kRowThreads;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictMoveKeep = 512;   // tokens that a list's own CTA moves to other pages
constexpr int kEvictKeys = 22528;   // 88 KB of keys: two CTAs per SM; longer rows are re-read (L2)

// One CTA per (sequence, KV head): the k = keep - recent largest weights before the last `recent`
// tokens, then the kept positions in order: each warp counts what its stretch of the row keeps, a
// sum over the warps says where its stretch begins, and it walks the stretch again, writing, with
// no barrier in between.  Weights go to another array on the way; in place they move afterwards, a
// round of positions at a time, all reads before the round's barrier and all writes after it: a
// token never moves to a later position, so no round reads what an earlier one wrote.
// Bound by the latency of its passes over a few ten thousand keys in shared memory.
// Returns how many tokens the list keeps.
__device__ __forceinline__ int choose_tokens(const EvictParams& p, uint32_t* sm) {
  __shared__ __align__(16) int hist[4 * kEvictThreads];
  __shared__ int s_scan[36];
  __shared__ uint32_t s_range[64];
  __shared__ uint32_t s_pick[1];
  __shared__ int s_gt[kEvictWarps], s_eq[kEvictWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.Hkv, kvh = blockIdx.x - b * p.Hkv;
  const int n = p.lens[b];
  const size_t stride = static_cast<size_t>(p.max_pages) * kTok;
  int32_t* kept = p.kept + static_cast<size_t>(blockIdx.x) * p.keep;
  const bool bad = n < 0 || n > static_cast<long long>(stride);
  if (kvh == 0 && tid == 0) {
    p.new_lens[b] = bad ? 0 : min(n, p.keep);
    if (bad) atomicOr(p.err, BDLM_DEVERR_LENGTH);
  }
  for (int i = (bad ? 0 : min(n, p.keep)) + tid; i < p.keep; i += kEvictThreads) kept[i] = -1;
  if (bad) return 0;
  const float* w = p.weights + blockIdx.x * stride;
  float* to = p.to_weights + blockIdx.x * stride;
  const bool in_place = to == w;
  if (n <= p.keep) {
    for (int i = tid; i < n; i += kEvictThreads) {
      kept[i] = i;
      if (!in_place) to[i] = w[i];
    }
    return n;
  }
  const int cand = n - p.recent, k = p.keep - p.recent;   // k < cand
  const bool held = cand <= kEvictKeys;
  uint32_t T = 0;
  int above = 0;
  // Four weights, i a multiple of 4: rows are multiples of 16 tokens, so past `cand` they are the row's.
  const bool wide = (reinterpret_cast<uintptr_t>(w) & 15) == 0;
  auto load4 = [&](int i) {
    return wide ? __ldcg(reinterpret_cast<const float4*>(w + i))
                : make_float4(__ldcg(w + i), __ldcg(w + i + 1), __ldcg(w + i + 2), __ldcg(w + i + 3));
  };
  // f(keys of i .. i + 3, how many of them are before `end`)
  auto four = [&](int i, int end, auto&& f) {
    uint32_t key[4];
    if (held) {
      const uint4 v = *reinterpret_cast<const uint4*>(sm + i);
      key[0] = v.x, key[1] = v.y, key[2] = v.z, key[3] = v.w;
    } else {
      const float4 v = load4(i);
      key[0] = order_key(v.x), key[1] = order_key(v.y), key[2] = order_key(v.z), key[3] = order_key(v.w);
    }
    f(key, end - i);
  };
  if (k > 0) {
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    constexpr int kBatch = 4;   // loads in flight per thread, of 16 bytes where the row is aligned
    for (int i0 = tid * 4; i0 < cand; i0 += kBatch * 4 * kEvictThreads) {
      float4 f[kBatch];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const int i = i0 + x * 4 * kEvictThreads;
        if (i >= cand) break;
        f[x] = load4(i);
      }
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const int i = i0 + x * 4 * kEvictThreads;
        if (i >= cand) break;
        const uint32_t key[4] = {order_key(f[x].x), order_key(f[x].y), order_key(f[x].z),
                                 order_key(f[x].w)};
        if (held) *reinterpret_cast<uint4*>(sm + i) = make_uint4(key[0], key[1], key[2], key[3]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (i + c < cand) {
            lo = min(lo, key[c]);
            hi = max(hi, key[c]);
          }
      }
    }
    block_range(lo, hi, s_range);
    T = kth_largest<kEvictThreads, uint32_t>(
        k, lo, hi,
        [&](auto&& f) {
#pragma unroll 2
          for (int i = tid * 4; i < cand; i += 4 * kEvictThreads)
            four(i, cand, [&](const uint32_t (&key)[4], int left) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (c < left) f(key[c]);
            });
        },
        hist, s_scan, s_pick, &above);
  }
  const int ties = k - above;   // tokens of weight T that stay
  // the last `recent` tokens stay, in the last places
  for (int j = k + tid; j < p.keep; j += kEvictThreads) {
    const int i = n - p.keep + j;
    kept[j] = i;
    if (!in_place) to[j] = __ldcg(w + i);
  }
  if (k > 0) {
    // this warp's stretch: what it keeps for sure (g) and what equals T (e)
    const int stretch = ((cand + kEvictWarps - 1) / kEvictWarps + 127) & ~127;
    const int s0 = warp * stretch, s1 = min(cand, s0 + stretch);
    int g = 0, e = 0;
#pragma unroll 2
    for (int i = s0 + lane * 4; i < s1; i += 128)
      four(i, s1, [&](const uint32_t (&key)[4], int left) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          g += c < left && key[c] > T;
          e += c < left && key[c] == T;
        }
      });
    g = __reduce_add_sync(0xffffffffu, g);
    e = __reduce_add_sync(0xffffffffu, e);
    if (lane == 0) {
      s_gt[warp] = g;
      s_eq[warp] = e;
    }
    __syncthreads();
    g = e = 0;
    int all = 0;
    for (int x = 0; x < kEvictWarps; ++x) {
      if (x < warp) {
        g += s_gt[x];
        e += s_eq[x];
      }
      all += s_eq[x];
    }
    // mostly all tokens of weight T stay (there is one): then one comparison decides a token
    const bool whole = all == ties;
    int at = g + (whole ? e : min(e, ties));
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll 2
    for (int i0 = s0; i0 < s1; i0 += 128) {
      const int i = i0 + lane * 4;
      uint32_t key[4] = {0, 0, 0, 0}, in = 0;   // `in`: a bit per key
      if (i < s1)
        four(i, s1, [&](const uint32_t (&v)[4], int left) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            key[c] = v[c];
            in |= (c < left && v[c] >= T) << c;
          }
        });
      if (!whole) {   // of those equal to T the first `ties` of the row
        int rank = e;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t be = __ballot_sync(0xffffffffu, (in >> c & 1) && key[c] == T);
          rank += __popc(be & below);
          e += __popc(be);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if ((in >> c & 1) && key[c] == T && rank++ >= ties) in &= ~(1u << c);
      }
      int j = at;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t bits = __ballot_sync(0xffffffffu, in >> c & 1);
        j += __popc(bits & below);
        at += __popc(bits);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (!(in >> c & 1)) continue;
        kept[j] = i + c;
        // (a zero's sign and a NaN's bits are not in the key)
        if (!in_place)
          to[j] = key[c] == 0 || key[c] == 0x80000000u ? __ldcg(w + i + c) : key_value(key[c]);
        ++j;
      }
    }
  }
  if (!in_place) return p.keep;
  __syncthreads();
  constexpr int kRound = 4;
  for (int j0 = 0; j0 < p.keep; j0 += kRound * kEvictThreads) {
    float v[kRound];
#pragma unroll
    for (int x = 0; x < kRound; ++x) {
      const int j = j0 + x * kEvictThreads + tid;
      if (j < p.keep) v[x] = __ldcg(w + __ldcg(kept + j));
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kRound; ++x) {
      const int j = j0 + x * kEvictThreads + tid;
      if (j < p.keep) to[j] = v[x];
    }
  }
  return p.keep;
}

// ------------------------------------------------------------------ moving tokens
// Token base + idx[j] of a sequence (and KV head) becomes token base + j.  Rows of K and V are 256
// bytes per head.  HBM bound: each kept row is read and written once.
//
// To other pages the moves are independent: a warp takes 32 tokens of one (sequence, KV head),
// lanes 0-15 the K row and 16-31 the V row, eight tokens in flight.
//
// In place (idx increasing, so every token moves to its own slot or an earlier one) a slot may only
// be written once the tokens before have been read.  A CTA therefore owns a (sequence, KV head) and
// moves some tokens at a time: all loads, a barrier, all stores.  The next loads may overtake the
// stores: they read only slots behind those.  Tokens that stay are skipped.  (A warp to a
// 64-byte column slice, walking all tokens without barriers: 299 us against 219, 32 x 8 lists of
// 8192-16384 tokens to 4096; eight warps of eight tokens instead of sixteen of four: 227.)
constexpr int kMoveWarps = 8, kInPlaceWarps = 16;

__device__ __forceinline__ long long token_row(const CompactParams& p, const int32_t* table, int b,
                                               long long tok, int kvh) {
  if (tok < 0 || tok >= static_cast<long long>(p.max_pages) * kTok) {
    atomicOr(p.err, BDLM_DEVERR_LENGTH);
    return -1;
  }
  const int id = __ldg(table + static_cast<size_t>(b) * p.max_pages + tok / kTok);
  if (id < 0 || id >= p.num_pages) {
    atomicOr(p.err, BDLM_DEVERR_PAGE);
    return -1;
  }
  return (static_cast<long long>(id) * kTok + tok % kTok) * p.Hkv + kvh;
}

// Tokens t0 .. t1 - 1 of the 32 tokens `run` of the first `count` (a warp).
__device__ __forceinline__ void move_run(const CompactParams& p, int b, int kvh, int run, int count,
                                         int t0, int t1) {
  const int lane = threadIdx.x & 31;
  const int j = run * 32 + lane;
  const int base = p.base ? p.base[b] : 0;
  long long from = -1, to = -1;   // this lane's token
  if (j < count && base >= 0) {
    const int i = __ldcg(p.idx + (static_cast<size_t>(b) * p.heads + (p.heads > 1 ? kvh : 0)) * p.n_max + j);
    if (i < 0) {
      atomicOr(p.err, BDLM_DEVERR_ROW);
    } else {
      from = token_row(p, p.page_table, b, static_cast<long long>(base) + i, kvh);
      to = token_row(p, p.to_table, b, static_cast<long long>(base) + j, kvh);
      if (from < 0) to = -1;
    }
  } else if (base < 0 && lane == 0) {
    atomicOr(p.err, BDLM_DEVERR_LENGTH);
  }
  uint4* pool = reinterpret_cast<uint4*>(lane < 16 ? p.k_pages : p.v_pages) + (lane & 15);
  constexpr int kBatch = 8;
  for (; t0 < t1; t0 += kBatch) {
    uint4 v[kBatch];
    long long dst[kBatch];
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const long long f = __shfl_sync(0xffffffffu, from, t0 + x);
      dst[x] = __shfl_sync(0xffffffffu, to, t0 + x);
      if (dst[x] >= 0) v[x] = __ldcs(pool + f * 16);
    }
#pragma unroll
    for (int x = 0; x < kBatch; ++x)
      if (dst[x] >= 0) pool[dst[x] * 16] = v[x];
  }
}

__global__ void __launch_bounds__(kMoveWarps * 32)
move_tokens_kernel(const CompactParams p, int runs) {
  griddep_wait();
  griddep_launch_dependents();
  const long long unit = static_cast<long long>(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5);
  if (unit >= static_cast<long long>(p.B) * p.Hkv * runs) return;
  const int run = static_cast<int>(unit % runs);
  const int bh = static_cast<int>(unit / runs);
  const int b = bh / p.Hkv, count = min(p.counts[b], p.n_max);
  if (run * 32 < count) move_run(p, b, bh - b * p.Hkv, run, count, 0, 32);
}

// The first `count` tokens of one (sequence, KV head) in place (a CTA of WARPS).
template <int WARPS, int BATCH>
__device__ __forceinline__ void move_in_place(const CompactParams& p, int b, int kvh, int count) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int base = p.base ? p.base[b] : 0;
  if (base < 0) {
    if (threadIdx.x == 0) atomicOr(p.err, BDLM_DEVERR_LENGTH);
    return;
  }
  const int32_t* idx = p.idx + (static_cast<size_t>(b) * p.heads + (p.heads > 1 ? kvh : 0)) * p.n_max;
  uint4* pool = reinterpret_cast<uint4*>(lane < 16 ? p.k_pages : p.v_pages) + (lane & 15);
  long long from, to;   // lanes below BATCH: the warp's tokens of a round
  auto look_up = [&](int j0) {
    const int j = j0 + warp * BATCH + lane;
    from = to = -1;
    if (lane >= BATCH || j >= count) return;
    const int i = __ldcg(idx + j);
    if (i == j) return;   // stays where it is
    if (i < 0) {
      atomicOr(p.err, BDLM_DEVERR_ROW);
      return;
    }
    from = token_row(p, p.page_table, b, static_cast<long long>(base) + i, kvh);
    to = token_row(p, p.to_table, b, static_cast<long long>(base) + j, kvh);
    if (from < 0) to = -1;
  };
  look_up(0);
  for (int j0 = 0; j0 < count; j0 += WARPS * BATCH) {
    uint4 v[BATCH];
    long long dst[BATCH];
#pragma unroll
    for (int x = 0; x < BATCH; ++x) {
      const long long f = __shfl_sync(0xffffffffu, from, x);
      dst[x] = __shfl_sync(0xffffffffu, to, x);
      if (dst[x] >= 0) v[x] = __ldcg(pool + f * 16);
    }
    look_up(j0 + WARPS * BATCH);   // the next round's rows meanwhile
    __syncthreads();   // every row of the round is read before a slot is written
#pragma unroll
    for (int x = 0; x < BATCH; ++x)
      if (dst[x] >= 0) pool[dst[x] * 16] = v[x];
  }
}

__global__ void __launch_bounds__(kInPlaceWarps * 32, 2)
move_in_place_kernel(const CompactParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / p.Hkv;
  move_in_place<kInPlaceWarps, 4>(p, b, blockIdx.x - b * p.Hkv, min(p.counts[b], p.n_max));
}

// The choice; with MOVE, the list's tokens move in the same kernel: for no more lists than SMs, in place,
// where a move is one CTA's work in either kernel, or of at most kEvictMoveKeep tokens to other pages.
// 64 lists cut back by half, one kernel against two: in place to 256 tokens 9.5 us against 11.0, to 1024
// 23 against 27, to 4096 114 against 128; to other pages to 64 tokens 6.7 against 10.4, to 256 8.6 against
// 10.6, to 512 11.9 against 10.9, to 1024 20 against 15.
template <bool MOVE>
__global__ void __launch_bounds__(kEvictThreads, MOVE ? 1 : 2)
evict_kernel(const EvictParams p, const CompactParams m) {
  extern __shared__ __align__(16) uint32_t sm[];
  griddep_wait();
  griddep_launch_dependents();
  const int count = choose_tokens(p, sm);
  if constexpr (MOVE) {
    __syncthreads();   // the kept positions are written
    const int warp = threadIdx.x >> 5, b = blockIdx.x / p.Hkv, kvh = blockIdx.x - b * p.Hkv;
    if (m.to_table != m.page_table) {
      for (int u = warp; u * 16 < count; u += kEvictWarps) {   // half a run
        const int t0 = (u & 1) * 16;
        move_run(m, b, kvh, u >> 1, count, t0, t0 + 16);
      }
    } else {
      move_in_place<kEvictWarps, 8>(m, b, kvh, count);
    }
  }
}

template <typename F>
cudaError_t allow_smem(std::atomic<unsigned long long>& done, F* kernel, size_t bytes) {
  return once_per_device(done, [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(bytes));
  });
}

}  // namespace

bool select_scores_itself(int lists, int max_pages, int rows, int num_sms) {
  return lists <= num_sms && max_pages <= kSelOwnPages && rows <= 32;
}

cudaError_t launch_select_pages(const SelectParams& p, int num_sms, cudaStream_t stream) {
  const size_t words = (static_cast<size_t>(p.max_pages) + 31) / 32;
  const unsigned lists = static_cast<unsigned>(p.B) * p.groups * p.Hkv;
  if (p.max_pages <= kOwn * kSelFewThreads && lists > 2u * static_cast<unsigned>(num_sms) &&
      p.group * p.G <= kSelFewRows)
    return launch_pdl(select_pages_kernel<kSelFewThreads, 6>, dim3(lists), dim3(kSelFewThreads),
                      (p.max_pages + 2 * words) * 4, stream, p);
  const int rows = p.group * p.G;
  if (select_scores_itself(static_cast<int>(lists), p.max_pages, rows, num_sms))
    return launch_pdl(rows <= 8    ? select_pages_kernel<kSelThreads, 1, 1>
                      : rows <= 16 ? select_pages_kernel<kSelThreads, 1, 2>
                                   : select_pages_kernel<kSelThreads, 1, 4>,
                      dim3(lists), dim3(kSelThreads), (p.max_pages + 2 * words) * 4, stream, p);
  // page ids and keys (of rows that fit), then two bitmaps of the row's pages
  const size_t keys = 2 * static_cast<size_t>(p.max_pages <= kSelKeys ? p.max_pages : kSelKeys);
  constexpr size_t kMost = (2 * kSelKeys + 2 * (kSelectMaxPages / 32)) * 4;
  static std::atomic<unsigned long long> one_done{0}, two_done{0};
  const bool one = lists <= static_cast<unsigned>(num_sms);
  auto* kernel = one ? select_pages_kernel<kSelThreads, 1> : select_pages_kernel<kSelThreads, 2>;
  cudaError_t e = allow_smem(one ? one_done : two_done, kernel, kMost);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(lists), dim3(kSelThreads), (keys + 2 * words) * 4, stream, p);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream) {
  if (p.to_table == p.page_table)
    return launch_pdl(move_in_place_kernel, dim3(static_cast<unsigned>(p.B) * p.Hkv),
                      dim3(kInPlaceWarps * 32), 0, stream, p);
  const int runs = (p.n_max + 31) / 32;
  const long long units = static_cast<long long>(p.B) * p.Hkv * runs;
  return launch_pdl(move_tokens_kernel,
                    dim3(static_cast<unsigned>((units + kMoveWarps - 1) / kMoveWarps)),
                    dim3(kMoveWarps * 32), 0, stream, p, runs);
}

cudaError_t launch_evict(const EvictParams& p, const CompactParams& m, int num_sms,
                         cudaStream_t stream) {
  const long long tokens = static_cast<long long>(p.max_pages) * kTok;
  const size_t keys = tokens <= kEvictKeys ? tokens : kEvictKeys;
  const long long lists = static_cast<long long>(p.B) * p.Hkv;
  const bool in_place = m.to_table == m.page_table;
  const bool move = lists <= num_sms && (in_place || p.keep <= kEvictMoveKeep);
  static std::atomic<unsigned long long> one_done{0}, two_done{0};
  auto* kernel = move ? evict_kernel<true> : evict_kernel<false>;
  cudaError_t e = allow_smem(move ? one_done : two_done, kernel, kEvictKeys * 4);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3(static_cast<unsigned>(lists)), dim3(kEvictThreads), keys * 4, stream, p, m);
  return e != cudaSuccess || move ? e : launch_compact(m, stream);
}

}  // namespace bdlm
