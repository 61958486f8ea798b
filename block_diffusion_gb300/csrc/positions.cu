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
constexpr int kScanThreads = 1024;

// Running sums of two values over the CTA's threads, `a` and `b` becoming those up to and with the thread's
// own; returns both totals.
__device__ __forceinline__ void scan2(long long& a, long long& b, long long (&s)[2][33], long long& ta, long long& tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
  if (warp == 0) {
    long long x = s[0][lane], y = s[1][lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, x, off), v = __shfl_up_sync(0xffffffffu, y, off);
      if (lane >= off) {
        x += u;
        y += v;
      }
    }
    s[0][lane] = x;
    s[1][lane] = y;
  }
  __syncthreads();
  if (warp > 0) {
    a += s[0][warp - 1];
    b += s[1][warp - 1];
  }
  ta = s[0][31];
  tb = s[1][31];
  __syncthreads();
}

// Row r of the packed tokens: its position and slot, and the table's entry where it opens a page.
__device__ __forceinline__ void place_row(const TableParams& p, const int32_t* first, int r, int total) {
  int at = -1, slot = -1;
  if (r < total) {
    int lo = 0, hi = p.B;   // first[lo] <= r < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= r)
        lo = mid;
      else
        hi = mid;
    }
    const int2 plan = p.plan[lo];
    at = plan.x + (r - first[lo]);
    const int col = at / kPage, held = (plan.x + kPage - 1) / kPage;
    int32_t* entry = p.page_table + static_cast<size_t>(lo) * p.max_pages + col;
    int id;
    if (col < held) {
      id = *entry;
    } else {
      id = __ldg(p.free_pages + plan.y + (col - held));
      if (at % kPage == 0) *entry = id;
    }
    if (id < 0 || id >= p.num_pages)
      atomicOr(p.err, BDLM_DEVERR_PAGE);
    else
      slot = id * kPage + at % kPage;
  }
  if (p.positions != nullptr) p.positions[r] = at;
  if (p.slots != nullptr) p.slots[r] = slot;
}

// WHOLE: the rows too (one launch for few of them).
template <bool WHOLE>
__global__ void __launch_bounds__(kScanThreads) table_plan_kernel(const TableParams p) {
  __shared__ long long s[2][33];
  __shared__ long long s_rows, s_pages;
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x;
  if (t == 0) s_rows = s_pages = 0;
  int from = p.free_from != nullptr ? *p.free_from : 0;
  const bool from_ok = from >= 0 && from <= p.n_free;
  if (!from_ok) {
    if (t == 0) atomicOr(p.err, BDLM_DEVERR_ROW);
    from = p.n_free;   // nothing is left
  }
  const long long max_tok = static_cast<long long>(p.max_pages) * kPage;
  long long pages = 0, rows = 0;   // of the sequences before this round
  for (int b0 = 0; b0 < p.B; b0 += kScanThreads) {
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
    const long long need = now > was ? (now + kPage - 1) / kPage - (was + kPage - 1) / kPage : 0;
    long long upto = need, unused = 0, tp, tr;
    scan2(upto, unused, s, tp, tr);
    upto += pages;
    pages += tp;
    bool served = need == 0 || upto <= p.n_free - from;
    const long long n = served && now > was ? now - was : 0;
    long long row = n, most = need;
    scan2(row, most, s, tr, tp);
    row += rows;
    rows += tr;
    if (row > p.max_tokens && n > 0) served = false;
    if (b < p.B) {
      p.lens_out[b] = served ? now : was;
      p.plan[b] = make_int2(was, static_cast<int>(served ? from + upto - need : 0));
      // (a row past the last one served is cut to it below)
      p.first[b + 1] = static_cast<int>(row > 0x7FFFFFFFll ? 0x7FFFFFFFll : row);
      if (served && n > 0)
        atomicMax(reinterpret_cast<unsigned long long*>(&s_rows), static_cast<unsigned long long>(row));
      if (served && need > 0)
        atomicMax(reinterpret_cast<unsigned long long*>(&s_pages), static_cast<unsigned long long>(upto));
    }
  }
  __syncthreads();
  // rows grow along the sequences, so the last one served has the total
  const int total = static_cast<int>(s_rows);
  for (int b = t; b < p.B; b += kScanThreads)
    if (p.first[b + 1] > total) p.first[b + 1] = total;
  if (t == 0) {
    p.first[0] = 0;
    if (p.free_next != nullptr) *p.free_next = static_cast<int>(from + s_pages);
  }
  if constexpr (WHOLE) {
    __syncthreads();
    for (int r = t; r < p.max_tokens; r += kScanThreads) place_row(p, p.first, r, total);
  }
}

constexpr int kRowThreads = 256;
__global__ void __launch_bounds__(kRowThreads) table_rows_kernel(const TableParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.x * kRowThreads + threadIdx.x;
  if (r < p.max_tokens) place_row(p, p.first, r, p.first[p.B]);
}

// ------------------------------------------------------------------ rotary positions
//
// Pair i of a head turns by pos * f_i.  The frequency is kept as a fraction of a turn in 64 bits, so the
// product with the position, modulo 2^64, is the angle modulo a turn exactly, however far the position:
// float32 loses it (position 500000 has steps of 0.03 radians there).  Its upper 32 bits then suffice for
// sine and cosine in float32.
constexpr int kRotaryThreads = 256;
constexpr int kRotaryRows = 4;   // tokens of a CTA: a thread computes the angle of one pair

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
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
        const int b = static_cast<int>(row / p.n);
        at = static_cast<long long>(p.start[b]) + (row - static_cast<long long>(b) * p.n);
        if (p.start[b] < 0) at = -1;
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
  const int heads = p.Hq + p.Hkv, c = t & 7;
  for (int y = 0; y < kRotaryRows; ++y) {
    if (!s_live[y]) continue;
    const long long row = row0 + y;
    for (int h = t >> 3; h < heads; h += kRotaryThreads / 8) {
      const bool is_q = h < p.Hq;
      const int hh = is_q ? h : h - p.Hq;
      const uint4* src = reinterpret_cast<const uint4*>((is_q ? p.q + row * p.q_stride : p.k + row * p.k_stride) + hh * 128);
      uint4* dst = reinterpret_cast<uint4*>(is_q ? p.q_out + (row * p.Hq + hh) * 128 : p.k_out + (row * p.Hkv + hh) * 128);
      if constexpr (INTER) {
        // eight values are four pairs
        uint4 v[2] = {src[c], src[c + 8]};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int d = (c + 8 * x) * 8;
          uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
          if (d < rot) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 cs = s_cs[y][d / 2 + k];
              const float a = bf16_lo(w[k]), b = bf16_hi(w[k]);
              w[k] = pack2(a * cs.x - b * cs.y, a * cs.y + b * cs.x);
            }
          }
          dst[c + 8 * x] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      } else {
        // chunk c and the one half of the turned part further on; behind that, what stays as it is
        const int half = rot / 16;
        const bool turn = c < half;
        const int c0 = turn ? c : rot / 8 + 2 * (c - half), c1 = turn ? c + half : c0 + 1;
        const uint4 u = src[c0], v = src[c1];
        uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {v.x, v.y, v.z, v.w};
        if (turn) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 lo = s_cs[y][c * 8 + 2 * k], hi = s_cs[y][c * 8 + 2 * k + 1];
            const float a0 = bf16_lo(a[k]), a1 = bf16_hi(a[k]), b0 = bf16_lo(b[k]), b1 = bf16_hi(b[k]);
            a[k] = pack2(a0 * lo.x - b0 * lo.y, a1 * hi.x - b1 * hi.y);
            b[k] = pack2(a0 * lo.y + b0 * lo.x, a1 * hi.y + b1 * hi.x);
          }
        }
        dst[c0] = make_uint4(a[0], a[1], a[2], a[3]);
        dst[c1] = make_uint4(b[0], b[1], b[2], b[3]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_build_tables(const TableParams& p, cudaStream_t stream) {
  // few rows: the CTA that plans them places them
  if (p.max_tokens <= 4 * kScanThreads)
    return launch_pdl(table_plan_kernel<true>, dim3(1), dim3(kScanThreads), 0, stream, p);
  const cudaError_t e = launch_pdl(table_plan_kernel<false>, dim3(1), dim3(kScanThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(table_rows_kernel, dim3((p.max_tokens + kRowThreads - 1) / kRowThreads), dim3(kRowThreads), 0, stream, p);
}

cudaError_t launch_rotary(const RotaryParams& p, const bdlm_rotary_desc& r, int num_sms, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((p.rows + kRotaryRows - 1) / kRotaryRows);
  return launch_pdl(r.interleaved ? rotary_kernel<true> : rotary_kernel<false>, dim3(grid), dim3(kRotaryThreads), 0,
                    stream, p, r);
}

}  // namespace bdlm
