// Page tables, slot maps and rotary positions of a step, for sm_103a.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "ptx.cuh"
#include "step_ops.h"

namespace bdlm {
namespace {

constexpr int kPage = 16;

// ------------------------------------------------------------------ page tables and slot maps
//
// Sequence b grows from old[b] to new[b] tokens and needs ceil(new / 16) - ceil(old / 16) pages, taken from
// the list of free pages in sequence order: running sums over the sequences say where each one's pages and
// tokens begin.  A sequence is served where the pages up to and with its own, and the tokens, suffice;
// behind the first that is not served only those that need nothing are.
//
// Bound: latency.  A table costs a dozen bytes a sequence and row, but sums over all sequences come before the first
// row.  One launch of one CTA while its threads have no more than four rows each (a step of 128 sequences: 5.6 us); above
// that a CTA plans and a second kernel places the rows (256 prompts, 2^20 rows: 10.2 us; the rows alone 8.4 MB).
constexpr int kScanThreads = 1024;

// Running sums of two values over the CTA's threads, `a` and `b` becoming those up to and with the thread's
// own; returns both totals.
__device__ __forceinline__ void scan2(long long& a, long long& b, long long (&s)[2][32], long long& ta, long long& tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, off), y = __shfl_up_sync(0xffffffffu, b, off);
    if (lane >= off) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    s[0][warp] = a;
    s[1][warp] = b;
  }
  __syncthreads();
  long long x = lane < warps ? s[0][lane] : 0, y = lane < warps ? s[1][lane] : 0;   // every warp for itself
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, x, off), v = __shfl_up_sync(0xffffffffu, y, off);
    if (lane >= off) {
      x += u;
      y += v;
    }
  }
  ta = __shfl_sync(0xffffffffu, x, 31);
  tb = __shfl_sync(0xffffffffu, y, 31);
  const long long pa = __shfl_sync(0xffffffffu, x, warp > 0 ? warp - 1 : 0), pb = __shfl_sync(0xffffffffu, y, warp > 0 ? warp - 1 : 0);
  if (warp > 0) {
    a += pa;
    b += pb;
  }
  __syncthreads();
}

// The sequence in [lo, hi) that packed row r lies in: first[lo] <= r < first[hi].
__device__ __forceinline__ int sequence_of(const int32_t* first, int lo, int hi, int r) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= r)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Row r of the packed tokens, of sequence b: its position and slot, and the table's entry where it opens a page.
__device__ __forceinline__ int2 place_row(const TableParams& p, int first, int2 plan, int b, int r) {
  const int at = plan.x + (r - first);
  const int col = at / kPage, held = (plan.x + kPage - 1) / kPage;
  int32_t* entry = p.page_table + static_cast<size_t>(b) * p.max_pages + col;
  int id;
  if (col < held) {
    id = *entry;
  } else {
    id = __ldg(p.free_pages + plan.y + (col - held));
    if (at % kPage == 0) *entry = id;
  }
  const bool bad = id < 0 || id >= p.num_pages;
  if (bad) atomicOr(p.err, BDLM_DEVERR_PAGE);
  return make_int2(at, bad ? -1 : id * kPage + at % kPage);
}

// WHOLE: the rows too, in one launch, the sequences' first rows and plans at hand in shared memory.
constexpr int kWholeSequences = 1024;
template <bool WHOLE>
__global__ void __launch_bounds__(kScanThreads) table_plan_kernel(const TableParams p) {
  __shared__ long long s[2][32];
  __shared__ unsigned long long s_rows, s_pages;
  __shared__ int32_t s_first[WHOLE ? kWholeSequences + 1 : 1];
  __shared__ int2 s_plan[WHOLE ? kWholeSequences : 1];
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x, threads = blockDim.x;
  if (t == 0) s_rows = s_pages = 0;
  int from = p.free_from != nullptr ? *p.free_from : 0;
  const bool from_ok = from >= 0 && from <= p.n_free;
  if (!from_ok) {
    if (t == 0) atomicOr(p.err, BDLM_DEVERR_ROW);
    from = p.n_free;   // nothing is left
  }
  const long long max_tok = static_cast<long long>(p.max_pages) * kPage;
  long long pages = 0, rows = 0;   // of the sequences before this round
  for (int b0 = 0; b0 < p.B; b0 += threads) {
    const int b = b0 + t;
    int was = 0, now = 0;
    if (b < p.B) {
      was = p.old_lens[b];
      now = p.new_lens[b];
      if (was < 0 || now < 0 || was > max_tok || now > max_tok) {
        atomicOr(p.err, BDLM_DEVERR_LENGTH);
        now = was;
      }
    }
    // (where every page request is served, as it mostly is, one pass over both sums does)
    const long long need = now > was ? (now + kPage - 1) / kPage - (was + kPage - 1) / kPage : 0;
    long long upto = need, row = now > was ? now - was : 0, tp, tr;
    scan2(upto, row, s, tp, tr);
    upto += pages;
    bool served = need == 0 || upto <= p.n_free - from;
    const long long n = served && now > was ? now - was : 0;
    if (pages + tp > p.n_free - from) {   // (the same for all threads)
      long long unused = 0;
      row = n;
      scan2(row, unused, s, tr, unused);
    }
    pages += tp;
    row += rows;
    rows += tr;
    if (row > p.max_tokens && n > 0) served = false;
    if (b < p.B) {
      const int2 plan = make_int2(was, static_cast<int>(served ? from + upto - need : 0));
      // (a row past the last one served is cut to it below)
      const int next = static_cast<int>(row > 0x7FFFFFFFll ? 0x7FFFFFFFll : row);
      p.lens_out[b] = served ? now : was;
      if constexpr (WHOLE) {
        s_plan[b] = plan;
        s_first[b + 1] = next;
      } else {
        p.plan[b] = plan;
        p.first[b + 1] = next;
      }
      if (served && n > 0) atomicMax(&s_rows, static_cast<unsigned long long>(row));
      if (served && need > 0) atomicMax(&s_pages, static_cast<unsigned long long>(upto));
    }
  }
  __syncthreads();
  // rows grow along the sequences, so the last one served has the total
  const int total = static_cast<int>(s_rows);
  for (int b = t; b < p.B; b += threads) {
    if constexpr (WHOLE) {
      if (s_first[b + 1] > total) s_first[b + 1] = total;
      p.first[b + 1] = s_first[b + 1];
    } else {
      if (p.first[b + 1] > total) p.first[b + 1] = total;
    }
  }
  if (t == 0) {
    p.first[0] = 0;
    if constexpr (WHOLE) s_first[0] = 0;
    if (p.free_next != nullptr) *p.free_next = from + static_cast<int>(s_pages);
  }
  if constexpr (WHOLE) {
    __syncthreads();
    for (int r = t; r < p.max_tokens; r += threads) {
      int2 at = make_int2(-1, -1);
      if (r < total) {
        const int b = sequence_of(s_first, 0, p.B, r);
        at = place_row(p, s_first[b], s_plan[b], b, r);
      }
      if (p.positions != nullptr) p.positions[r] = at.x;
      if (p.slots != nullptr) p.slots[r] = at.y;
    }
  }
}

// Many rows: a thread places four in a row.  A warp's 128 rows mostly are of one sequence or two, which the warp looks
// for together, so that few threads search on their own.
constexpr int kRowThreads = 256, kRowsEach = 4;
__global__ void __launch_bounds__(kRowThreads) table_rows_kernel(const TableParams p, int wide) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long r0 = (static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x) * kRowsEach;
  const int total = p.first[p.B];
  const long long warp0 = r0 - lane * kRowsEach;
  int lo = 0;
  if (warp0 < total) {
    int n = p.B;   // first[lo] <= warp0 < first[lo + n]
    while (n > 1) {
      const int step = (n + 31) / 32;
      const int c = __popc(__ballot_sync(0xffffffffu, lane * step < n && p.first[lo + (lane * step < n ? lane * step : 0)] <= warp0)) - 1;
      lo += c * step;
      n = min(step, n - c * step);
    }
  }
  if (r0 >= p.max_tokens) return;
  int pos[kRowsEach], slot[kRowsEach];
  int begin = -1, end = -1;   // rows of sequence lo
  int2 plan = make_int2(0, 0);
#pragma unroll
  for (int k = 0; k < kRowsEach; ++k) {
    const long long r = r0 + k;
    pos[k] = slot[k] = -1;
    if (r >= total) continue;
    if (r >= end) {
      if (end >= 0 || r >= p.first[lo + 1]) lo = sequence_of(p.first, lo, p.B, static_cast<int>(r));
      begin = p.first[lo];
      end = p.first[lo + 1];
      plan = p.plan[lo];
    }
    const int2 at = place_row(p, begin, plan, lo, static_cast<int>(r));
    pos[k] = at.x;
    slot[k] = at.y;
  }
  if (wide && r0 + kRowsEach <= p.max_tokens) {
    if (p.positions != nullptr) *reinterpret_cast<int4*>(p.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    if (p.slots != nullptr) *reinterpret_cast<int4*>(p.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    return;
  }
#pragma unroll
  for (int k = 0; k < kRowsEach; ++k) {
    if (r0 + k >= p.max_tokens) break;
    if (p.positions != nullptr) p.positions[r0 + k] = pos[k];
    if (p.slots != nullptr) p.slots[r0 + k] = slot[k];
  }
}

// ------------------------------------------------------------------ rotary positions
//
// Pair i of a head turns by pos * f_i.  The frequency is kept as a fraction of a turn in 64 bits (53 of them known), so
// the product with the position, modulo 2^64, loses nothing of the angle modulo a turn, however far the position:
// float32 loses it (position 500000 has steps of 0.03 radians there).  Its upper 32 bits then suffice for
// sine and cosine in float32, which takes 24 of them: 2^-26 of a turn.
//
// Bound: HBM, 256 bytes read and as many written a token and head: 8 prompts of 4096 tokens, 40 heads, in 94 us, 6.7
// TB/s (99 % of the copy rate); 105 us with one head under way a thread instead of three.  A block's queries and keys
// (128 x 4 tokens) are latency, 4.4 us.
constexpr int kRotaryThreads = 256;
constexpr int kRotaryRows = 4;    // tokens of a CTA: a thread computes the angle of one pair
constexpr int kRotaryBatch = 3;

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two 16-byte pieces of a head, turned or not: INTER: pieces c and c + 8, each of whole pairs.  Halves: piece c and the
// one half of the turned part further on; behind them, two that stay as they are.
template <bool INTER>
__device__ __forceinline__ int2 pieces(int c, int rot) {
  if constexpr (INTER) return make_int2(c, c + 8);
  const int half = rot / 16;
  return c < half ? make_int2(c, c + half) : make_int2(rot / 8 + 2 * (c - half), rot / 8 + 2 * (c - half) + 1);
}

template <bool INTER>
__device__ __forceinline__ void turn(uint4& u, uint4& v, int c, int rot, const float2* cs) {
  uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {v.x, v.y, v.z, v.w};
  if constexpr (INTER) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (c * 8 < rot) {
        const float2 s = cs[c * 4 + k];
        const float x = bf16_lo(a[k]), y = bf16_hi(a[k]);
        a[k] = pack2(x * s.x - y * s.y, x * s.y + y * s.x);
      }
      if ((c + 8) * 8 < rot) {
        const float2 s = cs[(c + 8) * 4 + k];
        const float x = bf16_lo(b[k]), y = bf16_hi(b[k]);
        b[k] = pack2(x * s.x - y * s.y, x * s.y + y * s.x);
      }
    }
  } else if (c < rot / 16) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 lo = cs[c * 8 + 2 * k], hi = cs[c * 8 + 2 * k + 1];
      const float a0 = bf16_lo(a[k]), a1 = bf16_hi(a[k]), b0 = bf16_lo(b[k]), b1 = bf16_hi(b[k]);
      a[k] = pack2(a0 * lo.x - b0 * lo.y, a1 * hi.x - b1 * hi.y);
      b[k] = pack2(a0 * lo.y + b0 * lo.x, a1 * hi.y + b1 * hi.x);
    }
  }
  u = make_uint4(a[0], a[1], a[2], a[3]);
  v = make_uint4(b[0], b[1], b[2], b[3]);
}

template <bool INTER>
__global__ void __launch_bounds__(kRotaryThreads)
rotary_kernel(const RotaryParams p, const __grid_constant__ bdlm_rotary_desc r) {
  __shared__ float2 s_cs[kRotaryRows][64];   // cosine and sine, times the amplitude
  __shared__ int s_live[kRotaryRows];
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x, rot = r.rot_dim, pairs = rot / 2;
  const long long row0 = static_cast<long long>(blockIdx.x) * kRotaryRows;
  {
    const int y = t >> 6, i = t & 63;
    const long long row = row0 + y;
    long long at = -1;
    if (row < p.rows) {
      if (p.positions != nullptr) {
        at = p.positions[row];
      } else {
        const int b = static_cast<int>(row / p.n), start = p.start[b];
        if (start >= 0) at = start + (row - static_cast<long long>(b) * p.n);
      }
    }
    if (i == 0) s_live[y] = at >= 0;
    if (at >= 0 && i < pairs) {
      const unsigned long long phase = static_cast<unsigned long long>(at) * r.turns[i];
      float sn, cs;
      sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f, &sn, &cs);   // 2^-31
      s_cs[y][i] = make_float2(cs * r.amplitude, (p.inverse ? -sn : sn) * r.amplitude);
    }
  }
  __syncthreads();
  // Heads of the CTA's rows, end to end, eight threads a head; kRotaryBatch of them are under way in a thread at once.
  const int heads = p.Hq + p.Hkv, c = t & 7;
  const int2 at = pieces<INTER>(c, rot);
  int y = 0, h = t >> 3;
  while (h >= heads && y < kRotaryRows) {
    h -= heads;
    ++y;
  }
  while (y < kRotaryRows) {
    uint4 u[kRotaryBatch], v[kRotaryBatch];
    uint4* dst[kRotaryBatch];
    int row[kRotaryBatch];
#pragma unroll
    for (int k = 0; k < kRotaryBatch; ++k) {
      dst[k] = nullptr;
      row[k] = y;
      if (y < kRotaryRows && s_live[y]) {
        const bool is_q = h < p.Hq;
        const int hh = is_q ? h : h - p.Hq;
        const long long g = row0 + y;
        const uint4* src = reinterpret_cast<const uint4*>((is_q ? p.q + g * p.q_stride : p.k + g * p.k_stride) + hh * 128);
        dst[k] = reinterpret_cast<uint4*>(is_q ? p.q_out + (g * p.Hq + hh) * 128 : p.k_out + (g * p.Hkv + hh) * 128);
        u[k] = src[at.x];
        v[k] = src[at.y];
      }
      h += kRotaryThreads / 8;
      while (h >= heads && y < kRotaryRows) {
        h -= heads;
        ++y;
      }
    }
#pragma unroll
    for (int k = 0; k < kRotaryBatch; ++k) {
      if (dst[k] == nullptr) continue;
      turn<INTER>(u[k], v[k], c, rot, s_cs[row[k]]);
      dst[k][at.x] = u[k];
      dst[k][at.y] = v[k];
    }
  }
}

}  // namespace

cudaError_t launch_build_tables(const TableParams& p, cudaStream_t stream) {
  // few rows: the CTA that plans them places them
  if (p.max_tokens <= 4 * kScanThreads && p.B <= kWholeSequences)
    return launch_pdl(table_plan_kernel<true>, dim3(1), dim3(kScanThreads), 0, stream, p);
  const int threads = p.B >= kScanThreads ? kScanThreads : (p.B + 31) / 32 * 32;
  const cudaError_t e = launch_pdl(table_plan_kernel<false>, dim3(1), dim3(threads), 0, stream, p);
  if (e != cudaSuccess || p.max_tokens == 0) return e;
  const int wide = ((reinterpret_cast<uintptr_t>(p.positions) | reinterpret_cast<uintptr_t>(p.slots)) & 15) == 0;
  const long long each = static_cast<long long>(kRowThreads) * kRowsEach;
  return launch_pdl(table_rows_kernel, dim3(static_cast<unsigned>((p.max_tokens + each - 1) / each)), dim3(kRowThreads), 0,
                    stream, p, wide);
}

cudaError_t launch_rotary(const RotaryParams& p, const bdlm_rotary_desc& r, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((p.rows + kRotaryRows - 1) / kRotaryRows);
  return launch_pdl(r.interleaved ? rotary_kernel<true> : rotary_kernel<false>, dim3(grid), dim3(kRotaryThreads), 0,
                    stream, p, r);
}

}  // namespace bdlm
