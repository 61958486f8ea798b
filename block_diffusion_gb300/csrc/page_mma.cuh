// Page scores on m16n8k16: a warp scores 16 pages for NT * 8 query rows straight from global memory.
// A page's bounds are 256 values (lo, then hi) and a query row's q-, then q+.  The order of the 256
// values along K is free as long as both operands have the same, so a lane's 16-byte chunk of a page
// row (8 values) serves as its fragments of two MMAs, 16 loads a lane are in flight at once, and
// nothing is staged but q- and q+.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>

#include "ptx.cuh"

namespace bdlm {

constexpr int kDirectPitch = 512 + 64;   // bytes of a q row: 64 more, so that 8 lanes miss no bank

// 16 bytes that are read once
__device__ __forceinline__ uint4 ld_stream16(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// max(q, 0) and min(q, 0) of eight bf16 (the sign bit decides)
__device__ __forceinline__ void split_signs(const uint4& q, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  const uint32_t x[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t neg = ((x[k] >> 15) & 0x00010001u) * 0xFFFFu;   // 16 ones per negative
    hi[k] = x[k] & ~neg;
    lo[k] = x[k] & neg;
  }
}

// The larger of the magnitudes of eight bf16 and of a bf16 pair (a NaN stays).
__device__ __forceinline__ void most_magnitude(uint32_t& top, const uint4& v) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t mag = x[k] & 0x7FFF7FFFu;
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&top),
                                         *reinterpret_cast<const __nv_bfloat162*>(&mag));
    top = *reinterpret_cast<const uint32_t*>(&m);
  }
}
// Over the warp; a NaN counts as infinite.
__device__ __forceinline__ float warp_magnitude(uint32_t top) {
  const float a = bf16_lo(top), z = bf16_hi(top);
  float m = a <= CUDART_INF_F && z <= CUDART_INF_F ? fmaxf(a, z) : CUDART_INF_F;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  return m;
}

// Chunk cc of query row r into shared memory.
__device__ __forceinline__ void stage_query(uint8_t* sQ, int r, int cc, const uint4& q) {
  uint32_t hi[4], lo[4];
  split_signs(q, hi, lo);
  *reinterpret_cast<uint4*>(sQ + r * kDirectPitch + cc * 16) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  *reinterpret_cast<uint4*>(sQ + r * kDirectPitch + 256 + cc * 16) =
      make_uint4(hi[0], hi[1], hi[2], hi[3]);
}

// A page's bounds into a[..][r] (not ok: zeros), lane t of four: chunks 4j + t of lo (j < 4), then of hi.
__device__ __forceinline__ void load_page(const uint16_t* bounds, int id, bool ok, int Hkv, int kvh,
                                          int t, int r, uint4 (&a)[8][2]) {
  const uint4* src =
      reinterpret_cast<const uint4*>(bounds) + (static_cast<size_t>(ok ? id : 0) * Hkv + kvh) * 32 + t;
#pragma unroll
  for (int j = 0; j < 8; ++j) a[j][r] = ok ? ld_stream16(src + 4 * j) : make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Scores of pages g and g + 8 (lane 4g + t) for rows 8 nt + 2t + {0, 1}: d[nt] = {g: two rows, g + 8: two
// rows}; top: the pages' largest magnitude, as a bf16 pair.
template <int NT>
__device__ __forceinline__ void page_products(const uint4 (&a)[8][2], const uint8_t* sQ, int g, int t,
                                              float (&d)[NT][4], uint32_t& top) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) d[nt][0] = d[nt][1] = d[nt][2] = d[nt][3] = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint4 x = a[j][0], y = a[j][1];
    most_magnitude(top, x);
    most_magnitude(top, y);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint4 q = *reinterpret_cast<const uint4*>(sQ + (nt * 8 + g) * kDirectPitch + j * 64 + t * 16);
      mma_16816(d[nt], x.x, y.x, x.y, y.y, q.x, q.y);
      mma_16816(d[nt], x.z, y.z, x.w, y.w, q.z, q.w);
    }
  }
}

}  // namespace bdlm
