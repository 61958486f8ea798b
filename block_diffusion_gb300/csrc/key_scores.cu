// One value per key of a paged cache, reduced over the query rows that share its KV head, for
// sm_103a: the attention weight each cached token receives, and the score of each page.
//
//   attention weights   w[j] = decay * w[j] + sum_n exp(scale * q_n . K[j] - lse_n)
//   page scores         s[p] = max_n sum_d (q_nd > 0 ? q_nd * hi_p[d] : q_nd * lo_p[d])
//                            = max_n (q_n+ . hi_p + q_n- . lo_p),  q+ = max(q, 0), q- = min(q, 0)
//
// Both are X = A Q^T (A: 128 keys x 128 dims, or 128 pages x 256 bound values) followed by a
// reduction of each row of X, so one kernel does both, with the keys on the UMMA M side: a key
// is one tensor-memory lane, its reduction over the query rows (UMMA N, up to 256) runs along
// the lane's columns in one thread, and no value crosses lanes.
//
// What bounds it: A is read once from HBM (256 bytes per token and KV head, 512 per page) and 8
// bytes per key move besides, so HBM does up to about 200 query rows; beyond, the tensor core and
// the exponentials (one per key and row; an SM does about 32 a clock) are close to it.
//
// One persistent CTA per SM walks items (a list = sequence and KV head, and a run of tiles of 128
// keys) in a fixed stride that every warp derives for itself, so no warp hands out work:
//   warp 0     one lane issues tcgen05.mma (and allocates tensor memory)
//   warps 1-2  weights: TMA, Q of an item (a 64-dim x G x L box per half) and one 16-slot page box
//              per page and half, alternate tiles each (one warp's 16 boxes take about 1 us)
//   warps 4-11 reduction, two sets of four warps (one per lane quadrant) on alternate tiles
//   warps 12-19  page scores: a page's bounds are 512 bytes, too small for a box each (128 boxes
//              of one row per K atom), so eight warps gather them with cp.async, 16 lanes a row,
//              into the 128-byte swizzle, and build q+ and q- in shared memory
// Stages are 32 KB (128 keys x 128 values); a page tile takes two (hi, then lo).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "cache_ops.h"
#include "ptx.cuh"

namespace bdlm {
namespace {

constexpr int kKeys = 128;           // keys per tile (UMMA M)
constexpr int kPageTokens = 16;
constexpr int kStage = 32768;        // 128 keys x 128 bf16, two 64-wide K atoms
constexpr int kAtom = 16384;
constexpr int kLoaders = 8;          // page scores: gathering warps

// WIDE: up to 256 query rows; else up to 32 (more stages, two Q buffers).
template <bool PAGES, bool WIDE>
struct Cfg {
  static constexpr int kRowsMax = WIDE ? 256 : 32;
  static constexpr int kQBytes = kRowsMax * (PAGES ? 512 : 256);
  static constexpr int kQBufs = WIDE ? 1 : 2;
  static constexpr int kStages = WIDE ? (PAGES ? 3 : 4) : (PAGES ? 5 : 6);
  static constexpr int kDBufs = WIDE ? 2 : 4;                  // X tiles in tensor memory
  static constexpr int kTmemCols = WIDE ? 512 : 128;
  static constexpr int kThreads = PAGES ? 640 : 384;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kQBufs) * kQBytes + kStages * kStage;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;   // invalid: 16 bytes of zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct KeyItem {
  int b, kvh, split, tile0, tiles, n;   // n: keys of the list
};

// Item idx of the schedule: runs of one list lie `lists` apart, so a CTA's items are spread over
// the lists and the short last runs of long lists come last.  False for a run past the list's end.
template <bool PAGES>
__device__ __forceinline__ bool key_item(int idx, const KeyParams& p, KeyItem& it) {
  const int lists = p.B * p.Hkv;
  it.split = idx / lists;
  const int list = idx - it.split * lists;
  it.b = list / p.Hkv;
  it.kvh = list - it.b * p.Hkv;
  const int prefix = __ldg(p.prefix_lens + it.b);
  if (prefix < 0 || static_cast<long long>(prefix) + p.L >
                        static_cast<long long>(p.max_pages) * kPageTokens) {
    if (it.split == 0 && it.kvh == 0 && threadIdx.x == 0) atomicOr(p.err, BDLM_DEVERR_LENGTH);
    return false;
  }
  it.n = PAGES ? prefix / kPageTokens : prefix;
  it.tile0 = it.split * p.tiles_per_item;
  const int tiles = (it.n + kKeys - 1) / kKeys - it.tile0;
  it.tiles = tiles < p.tiles_per_item ? tiles : p.tiles_per_item;
  return it.tiles > 0;
}

template <bool PAGES, bool WIDE>
__global__ void __launch_bounds__(Cfg<PAGES, WIDE>::kThreads, 1)
key_reduce_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const KeyParams p) {
  using C = Cfg<PAGES, WIDE>;
  constexpr int kHalves = PAGES ? 2 : 1;   // stages per tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = base;
  uint8_t* sA = base + C::kQBufs * C::kQBytes;
  __shared__ uint64_t bar_full[C::kStages], bar_empty[C::kStages];
  __shared__ uint64_t bar_qfull[C::kQBufs], bar_qempty[C::kQBufs];
  __shared__ uint64_t bar_dfull[C::kDBufs], bar_dempty[C::kDBufs], bar_lse[2], bar_done;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ __align__(16) float s_lse[PAGES ? 1 : 2][PAGES ? 4 : C::kRowsMax];   // log2 units

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n16 = (p.rows + 15) & ~15;   // UMMA N
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bar_full[s], PAGES ? kLoaders : 1);
      mbar_init(&bar_empty[s], 1);
    }
    for (int b = 0; b < C::kQBufs; ++b) {
      mbar_init(&bar_qfull[b], PAGES ? kLoaders : 1);
      mbar_init(&bar_qempty[b], 1);
    }
    for (int b = 0; b < C::kDBufs; ++b) {
      mbar_init(&bar_dfull[b], 1);
      mbar_init(&bar_dempty[b], 4);   // the four warps of a set
    }
    mbar_init(&bar_lse[0], 8);
    mbar_init(&bar_lse[1], 8);
    mbar_init(&bar_done, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  if (!PAGES) {
    // zero the padding rows of Q once: TMA writes rows 0 .. rows - 1 only
    for (int a = 0; a < C::kQBufs * 2; ++a) {
      uint8_t* z = sQ + (a >> 1) * C::kQBytes + ((a & 1) * n16 + p.rows) * 128;
      for (int o = threadIdx.x * 16; o < (n16 - p.rows) * 128; o += C::kThreads * 16)
        *reinterpret_cast<uint4*>(z + o) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  const uint32_t tmem = tmem_base;

  if (!PAGES && (warp == 1 || warp == 2)) {
    // ------------------------------------------------------------ TMA: Q and K pages
    const uint64_t policy = l2_policy_evict_first();   // K is read once
    bool ok = true;
    int u = 0, item = 0;   // tiles and items so far
    KeyItem it;
    for (int idx = blockIdx.x; idx < p.total_items && ok; idx += gridDim.x) {
      if (!key_item<PAGES>(idx, p, it)) continue;
      if (warp == 1) {
        const int qb = item % C::kQBufs;
        if (lane == 0) {
          ok = mbar_wait(&bar_qempty[qb], ((item / C::kQBufs) & 1) ^ 1, &abort_flag);
          if (ok) {
            mbar_arrive_expect_tx(&bar_qfull[qb], static_cast<uint32_t>(p.rows) * 256u);
            for (int h = 0; h < 2; ++h)
              tma_load_3d(sQ + qb * C::kQBytes + h * n16 * 128, &tm_q, &bar_qfull[qb], h * 64,
                          it.kvh * p.G, it.b * p.L + p.l0);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      ++item;
      const int32_t* pt = p.page_table + static_cast<size_t>(it.b) * p.max_pages;
      for (int j = 0; j < it.tiles && ok; ++j, ++u) {
        if ((u & 1) != warp - 1) continue;
        const int st = u % C::kStages;
        const int page = (it.tile0 + j) * (kKeys / kPageTokens) + (lane & 7);
        int id = -1;
        if (lane < 16 && page * kPageTokens < it.n) {
          id = __ldg(pt + page);
          if (id < 0 || id >= p.num_pages) {
            id = -1;
            atomicOr(p.err, BDLM_DEVERR_PAGE);
          }
        }
        const uint32_t have = __ballot_sync(0xffffffffu, id >= 0);
        if (lane == 0) {
          ok = mbar_wait(&bar_empty[st], ((u / C::kStages) & 1) ^ 1, &abort_flag);
          if (ok) {
            if (have)
              mbar_arrive_expect_tx(&bar_full[st], static_cast<uint32_t>(__popc(have)) * 2048u);
            else
              mbar_arrive(&bar_full[st]);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        __syncwarp();
        if (ok && id >= 0)
          tma_load_4d_hint(sA + st * kStage + (lane >> 3) * kAtom + (lane & 7) * 2048, &tm_k,
                           &bar_full[st], (lane >> 3) * 64, it.kvh, 0, id, policy);
      }
    }
    griddep_launch_dependents();
    if (!ok) {
      // a wait gave up: let this warp's copies in flight land before the CTA's memory goes away
      int dummy = 0;
      if (lane == 0)
        for (int s = 0; s < C::kStages; ++s) {
          mbar_wait(&bar_full[s], 0, &dummy, 1000000ull);
          mbar_wait(&bar_full[s], 1, &dummy, 1000000ull);
        }
      __syncwarp();
    }
  } else if (PAGES && warp >= 12) {
    // ------------------------------------------------------------ gather: q+ / q-, page bounds
    const int t = threadIdx.x - 384;   // 0 .. 255
    const int c16 = t & 15;            // 16-byte chunk of a 256-byte half row
    const uint32_t a_base = smem_u32(sA);
    const uint32_t a_off = static_cast<uint32_t>((c16 >> 3) * kAtom);
    bool ok = true;
    int u = 0, item = 0;               // stages issued, items
    int done = 0;                      // stages handed to the MMA
    uint32_t top = 0;                  // largest |bound| seen in the item, as a bf16 pair
    // Hands over the oldest stage in flight: the thread's own chunks have landed
    // (cp.async.wait_group), so it looks at their magnitudes and signs the stage off.
    auto hand_over = [&]() {
      const int st = done % C::kStages;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = i * 16 + (t >> 4);
        const uint4 v = *reinterpret_cast<const uint4*>(
            sA + st * kStage + a_off + r * 128 + (((c16 & 7) ^ (r & 7)) << 4));
        const uint32_t w[4] = {v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu,
                               v.w & 0x7FFF7FFFu};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 m =
              __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&top),
                          *reinterpret_cast<const __nv_bfloat162*>(&w[k]));
          top = *reinterpret_cast<const uint32_t*>(&m);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_full[st]);
      ++done;
    };
    KeyItem it;
    for (int idx = blockIdx.x; idx < p.total_items && ok; idx += gridDim.x) {
      if (!key_item<PAGES>(idx, p, it)) continue;
      const int qb = item % C::kQBufs;
      if (!(ok = mbar_wait_warp(&bar_qempty[qb], ((item / C::kQBufs) & 1) ^ 1, &abort_flag))) break;
      // row n of the item: query l0 + n / G, head kvh * G + n % G; padding rows repeat row 0, so
      // they cannot raise a maximum
      for (int c = t; c < n16 * 16; c += kLoaders * 32) {
        const int r = c >> 4, n = r < p.rows ? r : 0, cc = c & 15;
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(
                                  p.q + ((static_cast<size_t>(it.b) * p.L + p.l0 + n / p.G) * p.Hq +
                                         it.kvh * p.G + n % p.G) * 128) + cc);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t neg = ((w[k] >> 15) & 0x00010001u) * 0xFFFFu;   // 16 ones per negative
          hi[k] = w[k] & ~neg;
          lo[k] = w[k] & neg;
        }
        uint8_t* d = sQ + qb * C::kQBytes + ((cc >> 3) * n16 + r) * 128 + (((cc & 7) ^ (r & 7)) << 4);
        *reinterpret_cast<uint4*>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(d + 2 * n16 * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_qfull[qb]);
      ++item;
      top = 0;
      const int32_t* pt = p.page_table + static_cast<size_t>(it.b) * p.max_pages;
      constexpr int kAhead = C::kStages - 1;   // stages in flight per thread
      const int u0 = u;
      for (int j = 0; j < it.tiles && ok; ++j) {
        int id[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int page = (it.tile0 + j) * kKeys + i * 16 + (t >> 4);
          id[i] = page < it.n ? __ldg(pt + page) : -1;
          if (page < it.n && (id[i] < 0 || id[i] >= p.num_pages)) {
            id[i] = -1;
            if (c16 == 0) atomicOr(p.err, BDLM_DEVERR_PAGE);
          }
        }
        for (int h = 0; h < 2; ++h, ++u) {   // hi (row 1 of a page's bounds), then lo (row 0)
          if (u - u0 >= kAhead) {
            cp_async_wait<kAhead - 1>();
            hand_over();
          }
          const int st = u % C::kStages;
          if (!(ok = mbar_wait_warp(&bar_empty[st], ((u / C::kStages) & 1) ^ 1, &abort_flag))) break;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = i * 16 + (t >> 4);
            const size_t row =
                (static_cast<size_t>(id[i] < 0 ? 0 : id[i]) * p.Hkv + it.kvh) * 2 + (1 - h);
            cp_async16(a_base + st * kStage + a_off + r * 128 + (((c16 & 7) ^ (r & 7)) << 4),
                       p.bounds + row * 128 + c16 * 8, id[i] >= 0);
          }
          cp_async_commit();
        }
      }
      if (!ok) break;
      cp_async_wait<0>();
      while (done < u) hand_over();
      // the run's largest |bound|, one value per warp: what bounds the scores' rounding error
      __nv_bfloat162 m2 = *reinterpret_cast<const __nv_bfloat162*>(&top);
      float m = fmaxf(__low2float(m2), __high2float(m2));
      if (!(__low2float(m2) <= CUDART_INF_F) || !(__high2float(m2) <= CUDART_INF_F)) m = CUDART_INF_F;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      if (lane == 0)
        p.amax[((static_cast<size_t>(it.b) * p.Hkv + it.kvh) * p.items_per_list + it.split) *
                   kLoaders + (warp - 12)] = m;
    }
    cp_async_wait<0>();
    griddep_launch_dependents();
  } else if (warp == 0) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(128, n16, false, false);
      const uint32_t q_addr = smem_u32(sQ), a_addr = smem_u32(sA);
      bool ok = true;
      int u = 0, s = 0, item = 0;   // tiles, stages, items so far
      KeyItem it;
      for (int idx = blockIdx.x; idx < p.total_items && ok; idx += gridDim.x) {
        if (!key_item<PAGES>(idx, p, it)) continue;
        const int qb = item % C::kQBufs;
        if (!(ok = mbar_wait(&bar_qfull[qb], (item / C::kQBufs) & 1, &abort_flag))) break;
        for (int j = 0; j < it.tiles && ok; ++j, ++u) {
          const int db = u % C::kDBufs;
          if (!(ok = mbar_wait(&bar_dempty[db], ((u / C::kDBufs) & 1) ^ 1, &abort_flag))) break;
          const uint32_t d = tmem + static_cast<uint32_t>(db * C::kRowsMax);
          for (int h = 0; h < kHalves; ++h, ++s) {
            const int st = s % C::kStages;
            if (!(ok = mbar_wait(&bar_full[st], (s / C::kStages) & 1, &abort_flag))) break;
            tc_fence_after();
            const uint32_t qa = q_addr + qb * C::kQBytes + h * 2 * n16 * 128;
            const uint32_t aa = a_addr + st * kStage;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_bf16(d, smem_desc(aa + (kk >> 2) * kAtom + (kk & 3) * 32, 16, 1024),
                        smem_desc(qa + (kk >> 2) * n16 * 128 + (kk & 3) * 32, 16, 1024), idesc,
                        h > 0 || kk > 0 ? 1u : 0u);
            umma_commit(&bar_empty[st]);
          }
          if (ok) umma_commit(&bar_dfull[db]);
        }
        if (ok) umma_commit(&bar_qempty[qb]);
        ++item;
      }
      umma_commit(&bar_done);
    }
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------ reduction over the query rows
    const int q4 = warp & 3, set = (warp - 4) >> 2;
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    bool ok = true;
    int u = 0, item = 0;
    KeyItem it;
    for (int idx = blockIdx.x; idx < p.total_items && ok; idx += gridDim.x) {
      if (!key_item<PAGES>(idx, p, it)) continue;
      const float* lse = s_lse[0];
      if constexpr (!PAGES) {
        // the eight warps fill one of two buffers and wait for each other: a warp that writes
        // buffer x has seen every warp start the item between, so all are done with the item
        // that used x before
        float* w = s_lse[item & 1];
        for (int n = threadIdx.x - 128; n < n16; n += 256)
          w[n] = n < p.rows
                     ? __ldg(p.lse + (static_cast<size_t>(it.b) * p.L + p.l0 + n / p.G) * p.Hq +
                             it.kvh * p.G + n % p.G) * 1.4426950408889634f
                     : CUDART_INF_F;   // padding rows: 2^-inf = 0
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_lse[item & 1]);
        if (!(ok = mbar_wait_warp(&bar_lse[item & 1], (item >> 1) & 1, &abort_flag))) break;
        lse = w;
      }
      ++item;
      for (int j = 0; j < it.tiles && ok; ++j, ++u) {
        if ((u & 1) != set) continue;
        const int key = (it.tile0 + j) * kKeys + q4 * 32 + lane;
        bool live = key < it.n;
        const size_t list = static_cast<size_t>(it.b) * p.Hkv + it.kvh;
        float* wp = nullptr;
        float w_old = 0.f;
        if (live) {
          const int page = PAGES ? key : key / kPageTokens;
          const int id = __ldg(p.page_table + static_cast<size_t>(it.b) * p.max_pages + page);
          live = id >= 0 && id < p.num_pages;
        }
        if constexpr (!PAGES) {
          wp = p.weights + list * (static_cast<size_t>(p.max_pages) * kPageTokens) + key;
          if (live) w_old = *wp;
        }
        const int db = u % C::kDBufs;
        if (!(ok = mbar_wait_warp(&bar_dfull[db], (u / C::kDBufs) & 1, &abort_flag))) break;
        tc_fence_after();
        const uint32_t td = tmem + lane_off + static_cast<uint32_t>(db * C::kRowsMax);
        if constexpr (!PAGES) {
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          for (int c = 0; c < n16; c += 16) {
            uint32_t r[16];
            tmem_ld16(td + c, r);
            tmem_wait_ld();
            tmem_regs_ready(r);
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
              const float4 l4 = *reinterpret_cast<const float4*>(lse + c + k);
              sum[0] += ex2(fmaf(__uint_as_float(r[k]), p.scale_log2, -l4.x));
              sum[1] += ex2(fmaf(__uint_as_float(r[k + 1]), p.scale_log2, -l4.y));
              sum[2] += ex2(fmaf(__uint_as_float(r[k + 2]), p.scale_log2, -l4.z));
              sum[3] += ex2(fmaf(__uint_as_float(r[k + 3]), p.scale_log2, -l4.w));
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_dempty[db]);
          if (live) *wp = fmaf(p.decay, w_old, (sum[0] + sum[1]) + (sum[2] + sum[3]));
        } else {
          // a group's columns are `width` consecutive query rows
          float m = -CUDART_INF_F;
          int left = p.width, g = 0;
          float* out = p.scores + (static_cast<size_t>(it.b) * p.groups + p.l0 / p.group) *
                                      p.Hkv * static_cast<size_t>(p.max_pages) +
                       static_cast<size_t>(it.kvh) * p.max_pages + key;
          for (int c = 0; c < n16; c += 16) {
            uint32_t r[16];
            tmem_ld16(td + c, r);
            tmem_wait_ld();
            tmem_regs_ready(r);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              m = fmaxf(m, __uint_as_float(r[k]));
              if (--left == 0) {
                if (key < it.n && c + k < p.rows)
                  out[static_cast<size_t>(g) * p.Hkv * p.max_pages] = live ? m : -CUDART_INF_F;
                m = -CUDART_INF_F;
                left = p.width;
                ++g;
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_dempty[db]);
        }
      }
    }
  }

  // ---- teardown: every MMA retired before tensor memory is released
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    int dummy = 0;
    if (lane == 0) mbar_wait(&bar_done, 0, &dummy);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (threadIdx.x == 0 && abort_flag) atomicOr(p.err, BDLM_DEVERR_TIMEOUT);
}

// Bounds of the full pages that hold tokens from .. to - 1: lo and hi over the 16 slots, per head
// dim.  A thread takes 8 dims of one page and head: 16 independent 16-byte loads, then packed
// bf16 minima and maxima (exact).  HBM bound: 4 KB read and 512 bytes written per page and head.
__global__ void __launch_bounds__(128)
page_bounds_kernel(const uint16_t* __restrict__ k_pages, const int32_t* __restrict__ page_table,
                   const int32_t* __restrict__ from, const int32_t* __restrict__ to, int Hkv,
                   int max_pages, int num_pages, int ctas, uint16_t* __restrict__ bounds, int* err) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / ctas, cta = blockIdx.x - b * ctas;
  const int t0 = from ? from[b] : 0, t1 = to[b];
  if (t0 < 0 || t1 < t0 || t1 > static_cast<long long>(max_pages) * kPageTokens) {
    if (cta == 0 && threadIdx.x == 0) atomicOr(err, BDLM_DEVERR_LENGTH);
    return;
  }
  const int first = t0 / kPageTokens;
  const long long total = static_cast<long long>(t1 / kPageTokens - first) * Hkv * 16;
  const int per = Hkv * 16;
  for (long long i = static_cast<long long>(cta) * 128 + threadIdx.x; i < total;
       i += static_cast<long long>(ctas) * 128) {
    const int page = static_cast<int>(i / per), c = static_cast<int>(i - static_cast<long long>(page) * per);
    const int id = __ldg(page_table + static_cast<size_t>(b) * max_pages + first + page);
    if (id < 0 || id >= num_pages) {
      atomicOr(err, BDLM_DEVERR_PAGE);
      continue;
    }
    // chunk c of a token row: head c / 16, dims 8 * (c % 16) ..
    const uint4* src = reinterpret_cast<const uint4*>(k_pages) + static_cast<size_t>(id) * kPageTokens * per + c;
    uint4 v[kPageTokens];
#pragma unroll
    for (int s = 0; s < kPageTokens; ++s) v[s] = __ldg(src + static_cast<size_t>(s) * per);
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      auto word = [&](int s) {
        const uint32_t w = k == 0 ? v[s].x : k == 1 ? v[s].y : k == 2 ? v[s].z : v[s].w;
        return *reinterpret_cast<const __nv_bfloat162*>(&w);
      };
      __nv_bfloat162 a = word(0), z = a;
#pragma unroll
      for (int s = 1; s < kPageTokens; ++s) {
        a = __hmin2(a, word(s));
        z = __hmax2(z, word(s));
      }
      lo[k] = *reinterpret_cast<const uint32_t*>(&a);
      hi[k] = *reinterpret_cast<const uint32_t*>(&z);
    }
    uint4* dst = reinterpret_cast<uint4*>(bounds) +
                 (static_cast<size_t>(id) * Hkv + c / 16) * 32 + c % 16;
    dst[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    dst[16] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
}

template <bool PAGES, bool WIDE>
cudaError_t launch_key_t(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const KeyParams& p,
                         int num_sms, cudaStream_t stream) {
  using C = Cfg<PAGES, WIDE>;
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(key_reduce_kernel<PAGES, WIDE>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(C::kSmem));
  });
  if (e != cudaSuccess) return e;
  const int grid = p.total_items < num_sms ? p.total_items : num_sms;
  return launch_pdl(key_reduce_kernel<PAGES, WIDE>, dim3(grid), dim3(C::kThreads), C::kSmem, stream,
                    tm_q, tm_k, p);
}

}  // namespace

KeyPlan plan_keys(int B, int Hkv, int max_keys, int rows, int num_sms) {
  KeyPlan pl;
  const long long tiles = (static_cast<long long>(max_keys) + kKeys - 1) / kKeys;
  const long long lists = static_cast<long long>(B) * Hkv;
  // Runs of up to 16 tiles (32 for wide rows, whose Q costs an item up to 64 KB), shorter while
  // the batch has fewer than four runs per SM: a run's Q load is then cheap beside an idle SM.
  long long per = rows > 32 ? 32 : 16;
  while (per > 1 && lists * ((tiles + per - 1) / per) < 4ll * num_sms) per >>= 1;
  pl.tiles_per_item = static_cast<int>(per);
  pl.items_per_list = static_cast<int>((tiles + per - 1) / per);
  pl.total_items = lists * pl.items_per_list;
  pl.amax_floats = static_cast<size_t>(pl.total_items) * kLoaders;
  return pl;
}

int key_rows_max() { return 256; }

cudaError_t launch_keys(bool pages, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                        const KeyParams& p, int num_sms, cudaStream_t stream) {
  // Up to 32 query rows: more stages and two Q buffers; more rows need their shared memory for Q.
  const bool wide = p.rows > 32;
  if (pages)
    return wide ? launch_key_t<true, true>(tm_q, tm_k, p, num_sms, stream)
                : launch_key_t<true, false>(tm_q, tm_k, p, num_sms, stream);
  return wide ? launch_key_t<false, true>(tm_q, tm_k, p, num_sms, stream)
              : launch_key_t<false, false>(tm_q, tm_k, p, num_sms, stream);
}

cudaError_t launch_page_bounds(const uint16_t* k_pages, const int32_t* page_table,
                               const int32_t* from, const int32_t* to, int B, int Hkv,
                               int max_pages, int num_pages, int num_sms, uint16_t* bounds,
                               int* err, cudaStream_t stream) {
  // about 16 CTAs of 128 threads per SM in all, and no more per sequence than its pages can use
  long long ctas = (16ll * num_sms + B - 1) / B;
  const long long most = (static_cast<long long>(max_pages) * Hkv * 16 + 127) / 128;
  if (ctas > most) ctas = most;
  return launch_pdl(page_bounds_kernel, dim3(static_cast<unsigned>(ctas * B)), dim3(128), 0, stream,
                    k_pages, page_table, from, to, Hkv, max_pages, num_pages,
                    static_cast<int>(ctas), bounds, err);
}

}  // namespace bdlm
