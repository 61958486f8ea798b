// The 8-bit K/V cache, for sm_103a: writing tokens into it.
//
// K and V are held in pages of 16 tokens, [num_pages, Hkv, 16, 128] e4m3, so the block of 16 tokens of a
// head that shares a scale is 2 KB in one piece.  scales [num_pages, Hkv, 2] holds K's and V's: a value is
// its code times its scale.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "kernels.h"
#include "ptx_kv8.cuh"
#include "step_ops.h"

namespace bdlm {
namespace {

constexpr int kPage = 16;

// ------------------------------------------------------------------ write
//
// A warp writes one page of one head, of K or of V.  The scale is the least power of two 2^e, -40 <= e <= 40,
// that takes the largest magnitude of the page's tokens to 448 (the largest e4m3) or less: dividing by it
// is exact, so a value is rounded once, to e4m3's four bits, whatever the scale, and tokens that the page
// held before move to another scale without rounding anew (but for those that fall below its smallest
// step).  A finer scale would gain up to one bit of range below, not of precision.
//
// Bound: HBM, 512 bytes read and 256 written a token and head: 32 prompts of up to 4096 tokens, 8 heads, in 70 us, 5.9
// TB/s (87 % of the copy rate).  The whole page is in the warp's registers between its maximum and its codes, as bf16
// pairs: as 64 floats a lane fewer pages were under way (100 us).  A block's write (128 pages) is latency, 5.3 us.
constexpr int kWriteWarps = 8;
constexpr int kScaleExp = 40;

// Largest magnitude of the warp's bf16 pairs (a NaN counts as nothing).
__device__ __forceinline__ float most_of(uint32_t top) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(fmaxf(bf16_lo(top), bf16_hi(top))));
  return y;
}

__global__ void __launch_bounds__(kWriteWarps * 32, 4)
write_kv8_kernel(const WriteKv8Params p, int max_touched) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int hw = blockIdx.y * kWriteWarps + (threadIdx.x >> 5);   // head and which of K, V
  const int b = blockIdx.x / max_touched, j = blockIdx.x - b * max_touched;
  if (hw >= 2 * p.Hkv) return;
  const int h = hw >> 1, which = hw & 1;
  const int prefix = __ldg(p.prefix_lens + b);
  int n = p.n;
  long long row0 = static_cast<long long>(b) * p.n;
  if (p.first != nullptr) {
    row0 = __ldg(p.first + b);
    const long long end = __ldg(p.first + b + 1);
    if (row0 < 0 || end < row0 || end > p.n_rows || end - row0 > p.n) {
      if (lane == 0 && hw == 0 && j == 0) atomicOr(p.err, BDLM_DEVERR_ROW);
      return;
    }
    n = static_cast<int>(end - row0);
  }
  if (n == 0) return;
  if (prefix < 0 || static_cast<long long>(prefix) + n > static_cast<long long>(p.max_pages) * kPage) {
    if (lane == 0 && hw == 0 && j == 0) atomicOr(p.err, BDLM_DEVERR_LENGTH);
    return;
  }
  const int col = prefix / kPage + j;
  if (col > (prefix + n - 1) / kPage) return;
  const int page = __ldg(p.page_table + static_cast<size_t>(b) * p.max_pages + col);
  const int t0 = col * kPage;                         // the page's first token
  const int held = max(0, prefix - t0);               // tokens before the new ones: slots 0 .. held - 1
  const int live = min(kPage, prefix + n - t0);       // slots at and past live are left as they are
  const uint16_t* x = p.x[which] + ((row0 + (t0 - prefix)) * p.Hkv + h) * 128;   // of slot 0, a new one or not
  // lane l: 8 dims of slots 2i + l / 16
  const int dim = (lane & 15) * 8, odd = lane >> 4;
  uint4 w[8];   // asked for before the page is known to be there
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int slot = 2 * i + odd;
    w[i] = make_uint4(0, 0, 0, 0);
    if (slot >= held && slot < live) w[i] = __ldg(reinterpret_cast<const uint4*>(x + static_cast<long long>(slot) * p.Hkv * 128 + dim));
  }
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0 && hw == 0) atomicOr(p.err, BDLM_DEVERR_PAGE);
    return;
  }
  const size_t unit = static_cast<size_t>(page) * p.Hkv + h;
  uint8_t* codes = p.pages[which] + unit * (kPage * 128);
  float* scale = p.scales + unit * 2 + which;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t mag = u[k] & 0x7FFF7FFFu;
      const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&top), *reinterpret_cast<const __nv_bfloat162*>(&mag));
      top = *reinterpret_cast<const uint32_t*>(&m);
    }
  }
  float most = most_of(top), was = 0.f;
  // Tokens that the page held before (one page of a sequence at most): their codes, 16 slots' at once
  uint2 c[8];
  if (held > 0) {
    was = *scale;
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = make_uint2(0, 0);
      if (2 * i + odd < held) c[i] = *reinterpret_cast<const uint2*>(codes + (2 * i + odd) * 128 + dim);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t cc[4] = {c[i].x & 0xFFFFu, c[i].x >> 16, c[i].y & 0xFFFFu, c[i].y >> 16};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = from_e4m3x2(cc[k]);
        m = fmaxf(m, fmaxf(fabsf(f.x * was), fabsf(f.y * was)));
      }
    }
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(m));
    most = fmaxf(most, m);
  }
  const int e = min(max(e4m3_exponent(most), -kScaleExp), kScaleExp);
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int slot = 2 * i + odd;
    if (slot >= live) continue;
    uint32_t o[4];
    if (slot >= held) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = e4m3x2(bf16_lo(u[k]) * inv, bf16_hi(u[k]) * inv);
    } else {
      const uint32_t cc[4] = {c[i].x & 0xFFFFu, c[i].x >> 16, c[i].y & 0xFFFFu, c[i].y >> 16};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = from_e4m3x2(cc[k]);
        o[k] = e4m3x2(f.x * was * inv, f.y * was * inv);   // (the value in float32 first)
      }
    }
    *reinterpret_cast<uint2*>(codes + slot * 128 + dim) = make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
  }
  if (lane == 0) *scale = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

}  // namespace

cudaError_t launch_write_kv8(const WriteKv8Params& p, cudaStream_t stream) {
  const int touched = static_cast<int>((p.n + 2ll * kPage - 2) / kPage);   // pages that n tokens lie in at most
  const dim3 grid(static_cast<unsigned>(p.B) * touched, (2 * p.Hkv + kWriteWarps - 1) / kWriteWarps);
  return launch_pdl(write_kv8_kernel, grid, dim3(kWriteWarps * 32), 0, stream, p, touched);
}

}  // namespace bdlm
