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
// (Page scores of up to 64 rows: a kernel of its own, below.)
//
// Persistent CTAs, one or two per SM, each take an equal, contiguous share of all tiles of 128 keys,
// laid end to end list by list (a list = sequence and KV head): equal bytes per CTA whatever the
// lengths, and Q changes only where a list ends.  Every warp walks the share by itself, so no warp
// hands out work:
//   warp 0       one lane issues tcgen05.mma (and allocates tensor memory)
//   warps 1-2    weights: one 16-slot page box per page and half by TMA, alternate tiles each (one
//                warp's 16 boxes take about 1 us)
//   warp 3       finds the CTA's share; weights: Q of a list by TMA (a 64-dim x G x L box per half)
//   warps 4-     reduction, two or four sets of four warps (one per lane quadrant) in turn
//   page scores  warps 1-2 and two more: a page's bounds are two rows of 256 bytes, so TMA gathers
//                them, four rows of 128 bytes an instruction (about 50 ns each to issue, so four
//                warps); Q by TMA as for weights, which the last eight warps split into q+ and q- as
//                a list begins (two buffers up to 128 query rows); they also take the largest
//                magnitude of each stage.  (Loads to registers are slow beside 227 KB of shared
//                memory, which leave L1 few lines for what is in flight: 58 us a launch, 128 lists
//                of 1250-2500 pages and 256 rows, against 40.)
// Stages are 32 KB (128 keys x 128 values); a page tile takes two (hi, then lo).  (Halves of them, a
// ring of six, were no faster: 97 us against 93, 512 lists of 125-375 pages.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "cache_ops.h"
#include "page_mma.cuh"
#include "ptx.cuh"

namespace bdlm {
namespace {

constexpr int kKeys = kKeyTile;      // keys per tile (UMMA M)
constexpr int kPageTokens = 16;
constexpr int kStage = 32768;        // 128 keys x 128 bf16, two 64-wide K atoms
constexpr int kAtom = 16384;
constexpr int kHelpers = kAmaxPerTile;   // page scores: warps that split Q into q+ and q-

// WIDE: up to 256 query rows; else up to 32, two CTAs per SM (113 us a call against 117 with one CTA
// of twice the stages, 128 x 8 lists of 512-4096 tokens).
template <bool PAGES, bool WIDE>
struct Cfg {
  static constexpr int kRowsMax = WIDE ? 256 : 32;
  static constexpr int kQBytes = kRowsMax * (PAGES ? 512 : 256);
  static constexpr int kCtas = WIDE ? 1 : 2;   // per SM
  static_assert(WIDE || !PAGES, "page scores of few rows take the direct kernel below");
  // Weights of more than 32 rows: two sets share a tile, half of its columns each.  (The MMA stays
  // one of N = all rows: in halves of 128 it reads A twice, 128 bytes of shared memory a clock, and
  // the MMAs alone then took 99 us of what are 78 us of copies.)
  static constexpr bool kSplit = WIDE && !PAGES;
  static constexpr int kStages = 3;            // (weights of more than 32 rows: four were no faster)
  static constexpr int kDBufs = WIDE ? 2 : 4;                  // X tiles in tensor memory
  static constexpr int kSets = kSplit ? 4 : 2;                 // reducing sets of four warps
  static constexpr int kTmemCols = WIDE ? 512 : 128;
  static constexpr int kThreads = 128 + kSets * 128 + (PAGES ? (kHelpers + 2) * 32 : 0);
  // Weights of more than 32 rows: -lse / scale enters X through the MMA, as three bf16 numbers a row
  // (24 bits) against keys of 1, so that the reduction reads no table from shared memory beside
  // the MMAs (95 us a pass against 100, 16 x 64 x 4 rows over 8192-16384 tokens): one K step of 32
  // bytes a row, without swizzle, and one of 1s for the keys.
  static constexpr int kLseBytes = kSplit ? kRowsMax * 32 : 0, kOneBytes = kSplit ? kKeys * 32 : 0;
  static constexpr size_t kSmem =
      1024 + static_cast<size_t>(kQBytes) + kLseBytes + kOneBytes + kStages * kStage;
};

// Four rows r[] of 64 bf16 from column x of a two-dimensional map, to 512 consecutive bytes.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, uint64_t* bar, int x,
                                            const int (&r)[4]) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
      "r"(smem_u32(bar))
      : "memory");
}

// One K step (16 bf16 a row) without swizzle: core matrices of 8 rows x 16 bytes, two along K, then the
// next 8 rows.
__device__ __forceinline__ uint32_t step_chunk(int r, int c) { return (r >> 3) * 256 + c * 128 + (r & 7) * 16; }
__device__ __forceinline__ uint64_t step_desc(uint32_t saddr) {
  return smem_desc(saddr, 128, 256) & ~(static_cast<uint64_t>(7) << 61);
}

__device__ __forceinline__ void sts16(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3])
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// A walk over a CTA's share of the tiles.
template <bool PAGES>
struct KeyWalk {
  const KeyParams& p;
  int b, kvh, tile, left;   // left: tiles to go, this one included
  int n, tiles;             // keys and tiles of the list
  bool fresh;               // first tile of the share or of its list
  __device__ __forceinline__ KeyWalk(const KeyParams& prm, const int (&share)[4])
      : p(prm), b(share[0]), kvh(share[1]), tile(share[2]), left(share[3]), fresh(true) {
    if (left > 0) list();
  }
  __device__ __forceinline__ void list() {
    n = list_keys(p, b);
    tiles = (n + kKeys - 1) / kKeys;
  }
  static __device__ __forceinline__ int list_keys(const KeyParams& p, int b) {
    const int prefix = __ldg(p.prefix_lens + b);
    if (prefix < 0 || static_cast<long long>(prefix) + p.L >
                          static_cast<long long>(p.max_pages) * kPageTokens)
      return 0;
    return PAGES ? prefix / kPageTokens : prefix;
  }
  __device__ __forceinline__ void next() {
    fresh = false;
    if (--left == 0 || ++tile < tiles) return;
    tile = 0;
    fresh = true;
    if (++kvh < p.Hkv) return;
    kvh = 0;
    do {
      ++b;
      list();
    } while (tiles == 0);   // left > 0: a list with tiles follows
  }
  __device__ __forceinline__ size_t row() const { return static_cast<size_t>(b) * p.Hkv + kvh; }
};

// This CTA's share of the tiles (whole warp): every CTA adds up all sequences' tiles and takes an
// equal part of the total; CTA 0 reports bad lengths.
template <bool PAGES>
__device__ __forceinline__ void key_share(const KeyParams& p, int (&share)[4]) {
  const int lane = threadIdx.x & 31;
  auto seq_tiles = [&](int b) {
    return b < p.B ? static_cast<long long>((KeyWalk<PAGES>::list_keys(p, b) + kKeys - 1) / kKeys) *
                         p.Hkv
                   : 0ll;
  };
  long long total = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    total += seq_tiles(b);
    if (blockIdx.x == 0 && b < p.B) {
      const int prefix = __ldg(p.prefix_lens + b);
      if (prefix < 0 || static_cast<long long>(prefix) + p.L >
                            static_cast<long long>(p.max_pages) * kPageTokens)
        atomicOr(p.err, BDLM_DEVERR_LENGTH);
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  const long long first = total * blockIdx.x / gridDim.x;
  const long long end = total * (blockIdx.x + 1ll) / gridDim.x;
  if (lane == 0) share[3] = 0;
  __syncwarp();
  if (end == first) return;
  long long before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const long long mine = seq_tiles(b0 + lane);
    long long x = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    x += before;   // tiles up to and with this sequence
    if (first >= x - mine && first < x) {
      const long long at = first - (x - mine), per = mine / p.Hkv;
      share[0] = b0 + lane;
      share[1] = static_cast<int>(at / per);
      share[2] = static_cast<int>(at % per);
      share[3] = static_cast<int>(end - first);
    }
    before = __shfl_sync(0xffffffffu, x, 31);
    if (first < before) break;
  }
}

template <bool PAGES, bool WIDE>
__global__ void __launch_bounds__(Cfg<PAGES, WIDE>::kThreads, Cfg<PAGES, WIDE>::kCtas)
key_reduce_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const KeyParams p) {
  using C = Cfg<PAGES, WIDE>;
  constexpr int kHalves = PAGES ? 2 : 1;   // stages per tile
  constexpr int kGather2 = 4 + C::kSets * 4;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = base;
  uint8_t* sL = base + C::kQBytes;
  uint8_t* sOne = sL + C::kLseBytes;
  uint8_t* sA = sOne + C::kOneBytes;
  __shared__ uint64_t bar_full[C::kStages], bar_empty[C::kStages];
  __shared__ uint64_t bar_qfull[2], bar_qempty[2], bar_qraw[2];   // (qraw: page scores, Q as loaded)
  __shared__ uint64_t bar_dfull[C::kDBufs], bar_dempty[C::kDBufs], bar_lse[2], bar_done;
  __shared__ uint64_t bar_part[C::kSplit ? 4 : 1][4];        // second halves' sums: by tile, quadrant
  __shared__ float s_part[C::kSplit ? 4 : 1][C::kSplit ? 128 : 1];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ bool s_have[C::kStages];   // page scores: the stage holds pages
  __shared__ int s_share[4];
  constexpr bool kTable = !PAGES && !C::kSplit;   // -lse in shared memory (log2 units)
  __shared__ __align__(16) float s_lse[kTable ? 2 : 1][kTable ? C::kRowsMax : 4];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n16 = (p.rows + 15) & ~15;   // columns of X
  const int nq = PAGES && n16 <= C::kRowsMax / 2 ? 2 : 1;   // buffers of Q
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      // (page scores: both warps that fill the stage arrive, so that it is not consumed, where none of
      // its pages is there to be loaded, before both have seen it empty)
      mbar_init(&bar_full[s], PAGES ? 2 : 1);
      mbar_init(&bar_empty[s], PAGES ? 1 + kHelpers : 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bar_qfull[b], PAGES ? kHelpers : C::kSplit ? 2 : 1);
      mbar_init(&bar_qempty[b], 1);
      mbar_init(&bar_qraw[b], 1);
    }
    for (int b = 0; b < C::kDBufs; ++b) {
      mbar_init(&bar_dfull[b], 1);
      mbar_init(&bar_dempty[b], C::kSplit ? 8 : 4);   // the warps that read a tile
    }
    mbar_init(&bar_lse[0], C::kSets * 4);
    mbar_init(&bar_lse[1], C::kSets * 4);
    if constexpr (C::kSplit)
      for (int i = 0; i < 16; ++i) mbar_init(&bar_part[i >> 2][i & 3], 1);
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
    for (int a = 0; a < 2; ++a) {
      uint8_t* z = sQ + (a * n16 + p.rows) * 128;
      for (int o = threadIdx.x * 16; o < (n16 - p.rows) * 128; o += C::kThreads * 16)
        *reinterpret_cast<uint4*>(z + o) = make_uint4(0, 0, 0, 0);
    }
    if constexpr (C::kSplit) {
      // the K step of -lse: each key's row is 1, 1, 1, 0 ...; what the queries' rows do not use is 0
      for (int c = threadIdx.x; c < (C::kRowsMax + kKeys) * 2; c += C::kThreads) {
        const int r = c >> 1;
        const bool ones = r >= C::kRowsMax && (c & 1) == 0;
        *reinterpret_cast<uint4*>(sL + step_chunk(r, c & 1)) =
            ones ? make_uint4(0x3F803F80u, 0x3F80u, 0, 0) : make_uint4(0, 0, 0, 0);
      }
    }
    fence_proxy_async_smem();
  }
  griddep_wait();
  if (warp == 3) key_share<PAGES>(p, s_share);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;

  if (!PAGES && (warp == 1 || warp == 2)) {
    // ------------------------------------------------------------ TMA: K pages
    const uint64_t policy = l2_policy_evict_first();   // K is read once
    bool ok = true;
    int u = 0;
    for (KeyWalk<PAGES> w(p, s_share); w.left > 0 && ok; w.next(), ++u) {
      if ((u & 1) != warp - 1) continue;
      const int st = u % C::kStages;
      const int page = w.tile * (kKeys / kPageTokens) + (lane & 7);
      int id = -1;
      if (lane < 16 && page * kPageTokens < w.n) {
        id = __ldg(p.page_table + static_cast<size_t>(w.b) * p.max_pages + page);
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
                         &bar_full[st], (lane >> 3) * 64, w.kvh, 0, id, policy);
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
  } else if (warp == 3) {
    // ------------------------------------------------------------ TMA: Q; and -lse / scale
    bool ok = true;
    int q = 0;
    const float unscale = -1.4426950408889634f / p.scale_log2;
    for (KeyWalk<PAGES> w(p, s_share); w.left > 0 && ok; w.next()) {
      if (!w.fresh) continue;
      if (!(ok = mbar_wait_warp(&bar_qempty[q % nq], ((q / nq) & 1) ^ 1, &abort_flag))) break;
      if (lane == 0) {
        uint64_t* const bar = PAGES ? &bar_qraw[q % nq] : &bar_qfull[0];
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(p.rows) * 256u);
        for (int h = 0; h < 2; ++h)
          tma_load_3d(sQ + (q % nq) * n16 * 512 + h * n16 * 128, &tm_q, bar, h * 64, w.kvh * p.G,
                      w.b * p.L + p.l0);
      }
      if constexpr (C::kSplit) {
#pragma unroll 4
        for (int n = lane; n < n16; n += 32) {
          float c = -CUDART_INF_F;   // padding rows: 2^-inf = 0
          if (n < p.rows)
            c = __ldg(p.lse + (static_cast<size_t>(w.b) * p.L + p.l0 + n / p.G) * p.Hq +
                      w.kvh * p.G + n % p.G) * unscale;
          const __nv_bfloat16 hi = __float2bfloat16_rn(c);
          // (past bf16's range, a query that is left out: infinite, with nothing to add to it)
          const float c1 = fabsf(__bfloat162float(hi)) < CUDART_INF_F ? c - __bfloat162float(hi) : 0.f;
          const __nv_bfloat16 mid = __float2bfloat16_rn(c1);
          const __nv_bfloat16 lo = __float2bfloat16_rn(c1 - __bfloat162float(mid));
          *reinterpret_cast<uint2*>(sL + step_chunk(n, 0)) =
              make_uint2(__bfloat16_as_ushort(hi) | static_cast<uint32_t>(__bfloat16_as_ushort(mid)) << 16,
                         __bfloat16_as_ushort(lo));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_qfull[0]);
      }
      ++q;
    }
    if (!ok && lane == 0) {
      int dummy = 0;
      for (int b = 0; b < nq; ++b) {
        uint64_t* const bar = PAGES ? &bar_qraw[b] : &bar_qfull[0];
        mbar_wait(bar, 0, &dummy, 1000000ull);
        mbar_wait(bar, 1, &dummy, 1000000ull);
      }
    }
    __syncwarp();
  } else if (PAGES && (warp == 1 || warp == 2 || warp == kGather2 || warp == kGather2 + 1)) {
    // ------------------------------------------------------------ TMA: page bounds
    // half 0: hi (row 1 of a page's bounds), half 1: lo (row 0); which 64 of the 128 values
    const int h = warp < kGather2 ? warp - 1 : warp - kGather2, atom = warp < kGather2 ? 0 : 1;
    bool ok = true;
    KeyWalk<PAGES> w(p, s_share);
    int id[4], n_left;   // pages 4 * lane .. + 3 of the walk's tile
    auto load_ids = [&]() {
      const int page = w.tile * kKeys + lane * 4;
      n_left = w.left > 0 ? w.n - page : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        id[i] = i < n_left ? __ldg(p.page_table + static_cast<size_t>(w.b) * p.max_pages + page + i) : -1;
    };
    load_ids();
    for (int u = 0; w.left > 0 && ok; ++u) {
      const int s = 2 * u + h, st = s % C::kStages;
      // rows of pages that are not there repeat one that is, so that every value counts
      int row[4], any = -1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool good = id[i] >= 0 && id[i] < p.num_pages;
        if (!good && i < n_left) atomicOr(p.err, BDLM_DEVERR_PAGE);
        row[i] = good ? (id[i] * p.Hkv + w.kvh) * 2 + 1 - h : -1;
        any = max(any, row[i]);
      }
      const uint32_t have = __ballot_sync(0xffffffffu, any >= 0);
      const int fill = __shfl_sync(0xffffffffu, any, have ? __ffs(static_cast<int>(have)) - 1 : 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) row[i] = row[i] >= 0 ? row[i] : fill;
      w.next();
      load_ids();   // they arrive while the stage is waited for
      if (lane == 0) {
        ok = mbar_wait(&bar_empty[st], ((s / C::kStages) & 1) ^ 1, &abort_flag);
        if (ok && atom == 0) s_have[st] = have != 0;
        if (ok && have)
          mbar_arrive_expect_tx(&bar_full[st], kAtom);   // this warp's half of the stage
        else if (ok)
          mbar_arrive(&bar_full[st]);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      __syncwarp();
      if (ok && have)
        tma_gather4(sA + st * kStage + atom * kAtom + lane * 512, &tm_k, &bar_full[st], atom * 64, row);
    }
    if (!ok) {
      // as above: the copies in flight land before the CTA's memory goes away
      int dummy = 0;
      if (lane == 0)
        for (int s = 0; s < C::kStages; ++s) {
          mbar_wait(&bar_full[s], 0, &dummy, 1000000ull);
          mbar_wait(&bar_full[s], 1, &dummy, 1000000ull);
        }
      __syncwarp();
    }
  } else if (PAGES && warp >= C::kThreads / 32 - kHelpers) {
    // ------------------------------------------------------------ q+ and q-; largest magnitudes
    const int t = threadIdx.x - (C::kThreads - kHelpers * 32);   // 0 .. 255
    bool ok = true;
    int s = 0, q = 0;   // stages and lists so far
    auto split_q = [&]() {   // in place: q+ where Q is, q- behind it
      if (!(ok = mbar_wait_warp(&bar_qraw[q % nq], (q / nq) & 1, &abort_flag))) return;
      const uint32_t at = smem_u32(sQ) + (q % nq) * n16 * 512;
#pragma unroll 4
      for (int c = t * 16; c < n16 * 256; c += kHelpers * 512) {
        const uint4 v = lds16(at + c);
        uint32_t hi[4], lo[4];
        split_signs(v, hi, lo);
        sts16(at + c, hi);
        sts16(at + n16 * 256 + c, lo);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_qfull[q % nq]);
      ++q;
    };
    for (KeyWalk<PAGES> w(p, s_share); w.left > 0 && ok; w.next()) {
      if (w.fresh) split_q();
      uint32_t top = 0;   // largest |bound| seen in the tile, as a bf16 pair
      for (int h = 0; h < kHalves && ok; ++h, ++s) {
        const int st = s % C::kStages;
        if (!(ok = mbar_wait_warp(&bar_full[st], (s / C::kStages) & 1, &abort_flag))) break;
        if (s_have[st]) {
          const uint32_t a = smem_u32(sA) + st * kStage + t * 16;
#pragma unroll
          for (int i = 0; i < kStage / 16 / (kHelpers * 32); ++i)
            most_magnitude(top, lds16(a + i * kHelpers * 512));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_empty[st]);
      }
      // the largest magnitude of the tile, one value per warp, is what bounds its scores' rounding
      // error
      const float m = warp_magnitude(top);
      if (lane == 0)
        p.amax[(w.row() * p.max_tiles + w.tile) * kHelpers + (warp - (C::kThreads / 32 - kHelpers))] = m;
    }
    griddep_launch_dependents();
  } else if (warp == 0) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(128, n16, false, false);
      const uint32_t q_addr = smem_u32(sQ), a_addr = smem_u32(sA);
      bool ok = true;
      int u = 0, s = 0, q = -1;   // tiles, stages, lists so far
      for (KeyWalk<PAGES> w(p, s_share); w.left > 0 && ok; ++u) {
        if (w.fresh) {
          ++q;
          if (!(ok = mbar_wait(&bar_qfull[q % nq], (q / nq) & 1, &abort_flag))) break;
        }
        const int db = u % C::kDBufs;
        if (!(ok = mbar_wait(&bar_dempty[db], ((u / C::kDBufs) & 1) ^ 1, &abort_flag))) break;
        const uint32_t d = tmem + static_cast<uint32_t>(db * C::kRowsMax);
        for (int h = 0; h < kHalves; ++h, ++s) {
          const int st = s % C::kStages;
          if (!(ok = mbar_wait(&bar_full[st], (s / C::kStages) & 1, &abort_flag))) break;
          tc_fence_after();
          const uint32_t qa = q_addr + ((q % nq) * 2 + h) * 2 * n16 * 128;
          const uint32_t aa = a_addr + st * kStage;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16(d, smem_desc(aa + (kk >> 2) * kAtom + (kk & 3) * 32, 16, 1024),
                      smem_desc(qa + (kk >> 2) * n16 * 128 + (kk & 3) * 32, 16, 1024), idesc,
                      h > 0 || kk > 0 ? 1u : 0u);
          umma_commit(&bar_empty[st]);
        }
        if (!ok) break;
        if constexpr (C::kSplit)   // - lse / scale last: the sum is small then, and rounded once
          umma_bf16(d, step_desc(smem_u32(sOne)), step_desc(smem_u32(sL)), idesc, 1u);
        umma_commit(&bar_dfull[db]);
        w.next();
        if (w.left == 0 || w.fresh) umma_commit(&bar_qempty[q % nq]);
      }
      umma_commit(&bar_done);
    }
  } else if (warp >= 4 && warp < 4 + C::kSets * 4) {
    // ------------------------------------------------------------ reduction over the query rows
    const int q4 = warp & 3, set = (warp - 4) >> 2;
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    bool ok = true;
    int u = 0, q = 0;
    const float* lse = s_lse[0];
    for (KeyWalk<PAGES> w(p, s_share); w.left > 0 && ok; w.next(), ++u) {
      if constexpr (kTable) {
        if (w.fresh) {
          // the warps fill one of two buffers and wait for each other: a warp that writes
          // buffer x has seen every warp start the list between, so all are done with the list
          // that used x before
          float* x = s_lse[q & 1];   // -lse, so that the exponent is one FMA
          for (int n = threadIdx.x - 128; n < n16; n += C::kSets * 128)
            x[n] = n < p.rows
                       ? __ldg(p.lse + (static_cast<size_t>(w.b) * p.L + p.l0 + n / p.G) * p.Hq +
                               w.kvh * p.G + n % p.G) * -1.4426950408889634f
                       : -CUDART_INF_F;   // padding rows: 2^-inf = 0
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_lse[q & 1]);
          if (!(ok = mbar_wait_warp(&bar_lse[q & 1], (q >> 1) & 1, &abort_flag))) break;
          lse = x;
          ++q;
        }
      }
      if ((u & 1) != (C::kSplit ? set >> 1 : set)) continue;
      const int half = C::kSplit ? set & 1 : 0;   // which columns of the tile
      const int key = w.tile * kKeys + q4 * 32 + lane;
      bool live = key < w.n;
      float* wp = nullptr;
      float w_old = 0.f;
      if (live) {
        const int page = PAGES ? key : key / kPageTokens;
        const int id = __ldg(p.page_table + static_cast<size_t>(w.b) * p.max_pages + page);
        live = id >= 0 && id < p.num_pages;
      }
      if constexpr (!PAGES) {
        wp = p.weights + w.row() * (static_cast<size_t>(p.max_pages) * kPageTokens) + key;
        if (live && half == 0 && p.decay != 0.f) w_old = __ldcg(wp);
      }
      const int db = u % C::kDBufs;
      const int split = C::kSplit ? ((n16 >> 1) + 15) & ~15 : 0;   // columns of the first half
      const int cols = !C::kSplit ? n16 : half == 0 ? split : n16 - split;
      if (!(ok = mbar_wait_warp(&bar_dfull[db], (u / C::kDBufs) & 1, &abort_flag))) break;
      tc_fence_after();
      const uint32_t td =
          tmem + lane_off + static_cast<uint32_t>(db * C::kRowsMax + half * split);
      // 16 columns at a time.  The other warps of the scheduler cover the load's latency: fetching
      // the next 16 meanwhile, or 32 at a time, was slower (109 and 127 us against 99, 16 x 64 x 4
      // rows over 8192-16384 tokens).
      auto columns = [&](auto&& each) {
#pragma unroll 2
        for (int c = 0; c < cols; c += 16) {
          uint32_t r[16];
          tmem_ld16(td + c, r);
          tmem_wait_ld();
          tmem_regs_ready(r);
          each(c, r);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_dempty[db]);
      };
      if constexpr (!PAGES) {
        // two columns per packed instruction
        const float2 cs2 = make_float2(p.scale_log2, p.scale_log2);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        columns([&](int c, const uint32_t (&x)[16]) {
#pragma unroll
          for (int k = 0; k < 16; k += 4) {
            float4 l4 = make_float4(0.f, 0.f, 0.f, 0.f);   // (X holds -lse already)
            if constexpr (kTable) l4 = *reinterpret_cast<const float4*>(lse + c + k);
            const float2 a = __ffma2_rn(
                make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), cs2,
                make_float2(l4.x, l4.y));
            const float2 z = __ffma2_rn(
                make_float2(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3])), cs2,
                make_float2(l4.z, l4.w));
            sum[0] = __fadd2_rn(sum[0], make_float2(ex2(a.x), ex2(a.y)));
            sum[1] = __fadd2_rn(sum[1], make_float2(ex2(z.x), ex2(z.y)));
          }
        });
        float total = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        if constexpr (C::kSplit) {
          // the second half's sum goes to the first half's warp.  Four buffers, by tile: the next
          // tile to use this one is the second after it of the same sets, and its MMA waited for
          // both halves' warps to have read the tile between, by when the first half's was done
          // with this one
          uint64_t* bar = &bar_part[u & 3][q4];
          float* part = s_part[u & 3] + q4 * 32 + lane;
          if (half == 1) {
            *part = total;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
            live = false;
          } else {
            if (!(ok = mbar_wait_warp(bar, (u >> 2) & 1, &abort_flag))) break;
            total += *part;
          }
        }
        if (live) *wp = fmaf(p.decay, w_old, total);
      } else {
        // a group's columns are `width` consecutive query rows: 16 columns at a time where they are
        // all of one group
        float m = -CUDART_INF_F;
        int to_go = p.width;
        float* out = p.scores + (static_cast<size_t>(w.b) * p.groups + p.l0 / p.group) * p.Hkv *
                                    static_cast<size_t>(p.max_pages) +
                     static_cast<size_t>(w.kvh) * p.max_pages + key;
        auto flush = [&](int c) {
          if (key < w.n && c < p.rows) *out = live ? m : -CUDART_INF_F;
          out += static_cast<size_t>(p.Hkv) * p.max_pages;
          m = -CUDART_INF_F;
          to_go = p.width;
        };
        columns([&](int c, const uint32_t (&x)[16]) {
          if (to_go >= 16) {
            float v[5];
#pragma unroll
            for (int k = 0; k < 5; ++k)
              v[k] = fmax3(__uint_as_float(x[3 * k]), __uint_as_float(x[3 * k + 1]),
                           __uint_as_float(x[3 * k + 2]));
            m = fmax3(m, __uint_as_float(x[15]), fmaxf(fmax3(v[0], v[1], v[2]), fmaxf(v[3], v[4])));
            to_go -= 16;
            if (to_go == 0) flush(c + 15);
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              m = fmaxf(m, __uint_as_float(x[k]));
              if (--to_go == 0) flush(c + k);
            }
          }
        });
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

// Page scores of up to 64 query rows.  A page's 512 bytes take 2 * 16 to 64 rows * 256 flops: HBM
// is the only bound, and staging pages in shared memory for tcgen05 (the kernel above) costs more
// than it saves (16 x 8 lists of 1875-3750 pages, 16 rows: 42 us against 35; lists of 1250-2500 pages,
// 64 rows: a whole selection of 72 us against 62).  So each warp scores 16 pages straight from global
// memory (page_mma.cuh).  A CTA takes 128 pages a round (8 warps), its share of the tiles as above,
// two CTAs per SM.
template <int NT>   // query rows in tiles of 8
__global__ void __launch_bounds__(256, 2)
page_scores_direct_kernel(const KeyParams p) {
  __shared__ __align__(16) uint8_t sQ[NT * 8 * kDirectPitch];
  __shared__ int s_share[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 0) key_share<true>(p, s_share);
  __syncthreads();
  int gid[NT][2];   // the groups of this lane's columns 8 nt + 2t, + 1 (padding: none)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int n = nt * 8 + 2 * t + k;
      gid[nt][k] = n < p.rows ? n / p.width : -1;
    }
  const int groups = p.rows / p.width;
  const size_t group_stride = static_cast<size_t>(p.Hkv) * p.max_pages;
  KeyWalk<true> w(p, s_share);
  auto load_ids = [&](int (&id)[2]) {   // pages g and g + 8 of this warp's 16
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int page = w.tile * kKeys + warp * 16 + r * 8 + g;
      id[r] = w.left > 0 && page < w.n
                  ? __ldg(p.page_table + static_cast<size_t>(w.b) * p.max_pages + page)
                  : -1;
    }
  };
  int id[2];
  load_ids(id);
  while (w.left > 0) {
    if (w.fresh) {
      __syncthreads();   // every warp is done with the list before
      for (int c = threadIdx.x; c < NT * 8 * 16; c += 256) {
        const int r = c >> 4, cc = c & 15;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < p.rows)
          v = __ldg(reinterpret_cast<const uint4*>(
                        p.q + ((static_cast<size_t>(w.b) * p.L + p.l0 + r / p.G) * p.Hq +
                               w.kvh * p.G + r % p.G) * 128) + cc);
        stage_query(sQ, r, cc, v);
      }
      __syncthreads();
    }
    const int first = w.tile * kKeys + warp * 16, n = w.n;
    const size_t row = w.row(), out_row = (static_cast<size_t>(w.b) * p.groups + p.l0 / p.group) *
                                              group_stride +
                                          static_cast<size_t>(w.kvh) * p.max_pages;
    float* amax = p.amax + (row * p.max_tiles + w.tile) * kHelpers + warp;
    const int kvh = w.kvh;
    uint4 a[8][2];
    bool live[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      live[r] = id[r] >= 0 && id[r] < p.num_pages;
      if (!live[r] && first + r * 8 + g < n && t == 0) atomicOr(p.err, BDLM_DEVERR_PAGE);
      load_page(p.bounds, id[r], live[r], p.Hkv, kvh, t, r, a);
    }
    w.next();
    load_ids(id);   // the next tile's ids arrive with this tile's pages
    float d[NT][4];
    uint32_t top = 0;
    page_products<NT>(a, sQ, g, t, d, top);
    const float m = warp_magnitude(top);   // of the 16 pages
    if (lane == 0) *amax = m;
    // each group's maximum over its columns, spread over the four lanes of a page
    for (int s = 0; s < groups; ++s) {
      float best[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (gid[nt][k] == s) {
            best[0] = fmaxf(best[0], d[nt][k]);
            best[1] = fmaxf(best[1], d[nt][2 + k]);
          }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
        best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
        const int page = first + r * 8 + g;
        if (t == (s & 3) && page < n)
          p.scores[out_row + s * group_stride + page] = live[r] ? best[r] : -CUDART_INF_F;
      }
    }
  }
}

// Bounds of the full pages that hold tokens from .. to - 1: lo and hi over the 16 slots, per head
// dim.  A thread takes 8 dims of one page and head: 16 independent 16-byte loads, then packed
// bf16 minima and maxima (exact).  HBM bound: 4 KB read and 512 bytes written per page and head.
// 32 prompts of 4096 tokens, 8 heads: 50 us a call, 6.0 TB/s.  Over and over on one prompt 44 us with
// eight CTAs per SM and loads that pass L1 by; 47 with sixteen CTAs per SM, 59 with four, 51 with
// sixteen and cached loads.
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
    for (int s = 0; s < kPageTokens; ++s) v[s] = ld_stream16(src + static_cast<size_t>(s) * per);
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
  const long long most = static_cast<long long>(p.B) * p.Hkv * p.max_tiles;
  const long long ctas = static_cast<long long>(num_sms) * C::kCtas;
  const int grid = static_cast<int>(most < ctas ? most : ctas);
  return launch_pdl(key_reduce_kernel<PAGES, WIDE>, dim3(grid), dim3(C::kThreads), C::kSmem, stream,
                    tm_q, tm_k, p);
}

}  // namespace

int key_rows_max() { return 256; }

cudaError_t launch_attention_weights(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                     const KeyParams& p, int num_sms, cudaStream_t stream) {
  // up to 32 query rows: two CTAs per SM, 32-column tiles in four tensor-memory buffers, -lse from a table
  // in shared memory; more rows: one CTA per SM, a tile's columns split between sets, -lse by MMA
  return p.rows > 32 ? launch_key_t<false, true>(tm_q, tm_k, p, num_sms, stream)
                     : launch_key_t<false, false>(tm_q, tm_k, p, num_sms, stream);
}

namespace {
template <int NT>
cudaError_t launch_direct_t(const KeyParams& p, int num_sms, cudaStream_t stream) {
  const long long most = static_cast<long long>(p.B) * p.Hkv * p.max_tiles;
  const int grid = static_cast<int>(most < 2ll * num_sms ? most : 2ll * num_sms);
  return launch_pdl(page_scores_direct_kernel<NT>, dim3(grid), dim3(256), 0, stream, p);
}
}  // namespace

cudaError_t launch_page_scores(const CUtensorMap& tm_q, const CUtensorMap& tm_bounds,
                               const KeyParams& p, int num_sms, cudaStream_t stream) {
  if (p.rows <= 8) return launch_direct_t<1>(p, num_sms, stream);
  if (p.rows <= 16) return launch_direct_t<2>(p, num_sms, stream);
  if (p.rows <= 32) return launch_direct_t<4>(p, num_sms, stream);
  if (p.rows <= kDirectRows) return launch_direct_t<8>(p, num_sms, stream);
  return launch_key_t<true, true>(tm_q, tm_bounds, p, num_sms, stream);
}

cudaError_t launch_page_bounds(const uint16_t* k_pages, const int32_t* page_table,
                               const int32_t* from, const int32_t* to, int B, int Hkv,
                               int max_pages, int num_pages, int num_sms, uint16_t* bounds,
                               int* err, cudaStream_t stream) {
  // about 8 CTAs of 128 threads per SM in all, and no more per sequence than its pages can use
  long long ctas = (8ll * num_sms + B - 1) / B;
  const long long most = (static_cast<long long>(max_pages) * Hkv * 16 + 127) / 128;
  if (ctas > most) ctas = most;
  return launch_pdl(page_bounds_kernel, dim3(static_cast<unsigned>(ctas * B)), dim3(128), 0, stream,
                    k_pages, page_table, from, to, Hkv, max_pages, num_pages,
                    static_cast<int>(ctas), bounds, err);
}

}  // namespace bdlm
