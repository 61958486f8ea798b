// Block attention over the 8-bit cache, for sm_103a.
//
//     out = sum_t p_t sV_t v_t / sum_t p_t,   p_t = 2^(c sK_t q . k_t - m),   c = sm_scale log2 e
// with codes k_t, v_t in e4m3 and the scales sK_t, sV_t of a token's page and head.
//
//  * The codes go from memory to the tensor cores as they are (tcgen05 kind::f8f6f4, which adds up in
//    float32), so nothing is widened on the way and a token costs 256 bytes of shared memory.  The
//    other operand has 8 bits as well: q and p are held as two e4m3 parts each, the value rounded to four
//    bits and what that leaves, rounded to four bits again.  A pair is off by 2^-8 of the value, as bf16
//    is, and by no less than half its smallest step, 2^-18 of the largest value of what shares its power of
//    two (a KV head's queries; a query's weights).  Both parts of an operand multiply the same codes into
//    the same sums: twice the products of one part, at twice bf16's rate.
//  * A page's scale of K is a factor of its scores.  Its scale of V goes into the weight: with
//        x_t = c sK_t q . k_t + log2 sV_t    and its maximum m,
//    w_t = 2^(x_t - m + 7) is what the second product takes (no sum ever meets a scale) and
//    sum w_t / sV_t is the divisor.  So w's parts keep their precision where it counts, whatever the
//    scales are from page to page.
//  * Work: the tiles of 128 tokens of all (sequence, KV head, row group) lists, end to end, are cut
//    into units of equal numbers of tiles, which CTAs take in turn.  A list that a unit's border cuts is
//    written in parts (O, m, l) that a second kernel joins in order.  So the work is even whatever the
//    lengths, and there are at most two parts a unit.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "kernels.h"
#include "ptx.cuh"
#include "step_ops.h"

namespace bdlm {
namespace {

constexpr int kPage = 16;
constexpr int kTile = 128;             // tokens of a tile (UMMA M)
constexpr int kTilePages = kTile / kPage;
constexpr int kStage = kTile * 128;    // bytes of a tile's K or V
constexpr int kRing = 4;               // chunk descriptors in flight
constexpr float kWeightExp = 7.0f;     // a query's largest weight is 2^7 ...
constexpr float kLazy = 1.5f;          // ... to 2^8.5: a running maximum moves only when it rises by more (e4m3 ends at 448)
constexpr float kScaleLog = 40.0f;     // scales count as 2^-40 .. 2^40

struct Params {
  const uint16_t* q;
  const float2* scales;
  const int32_t* page_table;
  const int32_t* prefix_lens;
  uint16_t* out;
  float* part;       // unit u's parts: 2u (of a list that began before it), 2u + 1 (of one that begins in it)
  int* err;
  int* work;         // [0] next unit, [1] CTAs finished
  const int* cum;    // [B + 1] tiles of the sequences before each (null: up to 32 sequences)
  int B, L, Hq, Hkv, G, max_pages, num_pages, lsub, row_groups, rows;
  float scale_log2;
};

// Some tiles of a list, as the warps pass them on.
struct Chunk {
  int b, kvh, rg;
  int t0, t_end;     // first token; end of the list's tokens (or past the chunk)
  int n_tiles;
  int first, last;   // of the tiles that this CTA sums up together
  int slot;          // part to write at the last chunk, -1: the output
  int end;
  float q_scale;     // q = (hi + lo) * q_scale, times c
};

__device__ __forceinline__ void mbar_wait_drain(uint64_t* bar, uint32_t parity) {
  int dummy = 0;
  mbar_wait(bar, parity, &dummy);
}

__device__ __forceinline__ int kv_tokens(const Params& p, int b, bool* ok) {
  const int prefix = __ldg(p.prefix_lens + b);
  const long long max_tok = static_cast<long long>(p.max_pages) * kPage;
  const long long n = static_cast<long long>(prefix < 0 ? 0 : prefix) + p.L;
  *ok = prefix >= 0 && n <= max_tok;
  return static_cast<int>(n < max_tok ? n : max_tok);
}

// Tiles of a unit: all of the work in `ctas` even shares, or in four rounds of them where a share is long
// enough that CTAs' different speeds count for more than a unit's start and end.
constexpr int kRounds = 4;
constexpr int kRoundTiles = 32;   // tiles of a share from which on there are kRounds rounds
__host__ __device__ __forceinline__ long long unit_tiles(long long total, int ctas) {
  const long long share = (total + ctas - 1) / ctas;
  if (share < kRoundTiles) return share < 1 ? 1 : share;
  return (total + static_cast<long long>(kRounds) * ctas - 1) / (static_cast<long long>(kRounds) * ctas);
}

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// a and b in two e4m3 parts: each the low half for a, the high one for b.
__device__ __forceinline__ void split_e4m3x2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = e4m3x2(a, b);
  const float2 h = from_e4m3x2(hi);
  lo = e4m3x2(a - h.x, b - h.y);
}

// The largest of a few bf16 pairs' magnitudes as a float (NaN aside).
__device__ __forceinline__ float magnitude(const uint4& w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) m = fmaxf(m, fmaxf(fabsf(bf16_lo(u[k])), fabsf(bf16_hi(u[k]))));
  return m;
}

// The power of two 2^e that takes a largest magnitude to 448 or less (and above 224 where it can).
__device__ __forceinline__ int q_exponent(float most) {
  const uint32_t bits = __float_as_uint(most);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, -110), 119);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Maximum over the warp in one instruction (redux.sync of float32, sm_100 family).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// The walk over a CTA's units, list by list, in chunks of up to CHUNK tiles (whole warp, uniform).
template <int CHUNK>
struct Walk {
  long long total, per, pos, end;   // in tiles; pos, end: what is left of the unit
  int unit, units;
  int b, kv_len, tiles, lists;      // the sequence at pos
  long long base;                   // tiles before it
  int kvh, rg, tile, seg_end, slot, seg_first;
  bool len_ok;
  bool counted;

  __device__ __forceinline__ void init(const Params& p, int lane, int& my_cum) {
    lists = p.Hkv * p.row_groups;
    long long sum;
    if (p.cum == nullptr) {
      bool ok;
      int n = lane < p.B ? (kv_tokens(p, lane, &ok) + kTile - 1) / kTile : 0;
      int incl = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
      }
      my_cum = incl - n;
      sum = __shfl_sync(0xffffffffu, incl, 31);
    } else {
      sum = __ldg(p.cum + p.B);
    }
    total = sum * lists;
    per = unit_tiles(total, gridDim.x);
    units = static_cast<int>((total + per - 1) / per);
    counted = units > static_cast<int>(gridDim.x);
    unit = -1;
    pos = end = 0;
    tile = seg_end = 0;
  }

  __device__ __forceinline__ void sequence(const Params& p) {
    kv_len = kv_tokens(p, b, &len_ok);
    tiles = (kv_len + kTile - 1) / kTile;
  }

  // Goes to the next unit; false: there is none.
  __device__ __forceinline__ bool take(const Params& p, int lane, int my_cum) {
    if (unit < 0) {
      unit = blockIdx.x;
    } else {
      if (!counted) return false;
      int u = 0;
      if (lane == 0) u = atomicAdd(p.work, 1);
      unit = static_cast<int>(gridDim.x) + __shfl_sync(0xffffffffu, u, 0);
    }
    if (unit >= units) return false;
    pos = unit * per;
    end = pos + per < total ? pos + per : total;
    const int x = static_cast<int>(pos / lists);   // cum[b] <= x < cum[b + 1]
    int before;
    if (p.cum == nullptr) {
      b = __popc(__ballot_sync(0xffffffffu, lane < p.B && my_cum <= x)) - 1;
      before = __shfl_sync(0xffffffffu, my_cum, b);
    } else {
      int lo = 0, n = p.B;
      while (n > 1) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const int c = __popc(__ballot_sync(0xffffffffu, lane * step < n && __ldg(p.cum + at) <= x)) - 1;
        lo += c * step;
        n = min(step, n - c * step);
      }
      b = lo;
      before = __ldg(p.cum + b);
    }
    base = static_cast<long long>(before) * lists;
    sequence(p);
    return true;
  }

  // The next chunk; false: no work is left.
  __device__ __forceinline__ bool next(const Params& p, int lane, int my_cum, Chunk& c) {
    seg_first = 0;
    if (tile == seg_end) {
      if (pos == end && !take(p, lane, my_cum)) return false;
      long long r = pos - base;
      if (r >= static_cast<long long>(tiles) * lists) {
        base += static_cast<long long>(tiles) * lists;
        r = 0;
        ++b;
        sequence(p);
      }
      const int list = static_cast<int>(r / tiles);
      rg = list % p.row_groups;
      kvh = list / p.row_groups;
      tile = static_cast<int>(r - static_cast<long long>(list) * tiles);
      const int n = static_cast<int>(min(static_cast<long long>(tiles - tile), end - pos));
      seg_end = tile + n;
      pos += n;
      slot = tile == 0 && seg_end == tiles ? -1 : 2 * unit + (tile == 0 ? 1 : 0);
      seg_first = 1;
      if (!len_ok && tile == 0 && list == 0 && lane == 0) atomicOr(p.err, BDLM_DEVERR_LENGTH);
    }
    c.b = b;
    c.kvh = kvh;
    c.rg = rg;
    c.t0 = tile * kTile;
    c.t_end = kv_len;
    c.n_tiles = min(CHUNK, seg_end - tile);
    tile += c.n_tiles;
    c.first = seg_first;
    c.last = tile == seg_end;
    c.slot = slot;
    c.end = 0;
    return true;
  }
};

constexpr int kPartRow = 130;   // floats of a row's part: O, m, l

// ------------------------------------------------------------------ up to 32 query rows per KV head
//
// Transposed: S^T = K Q^T with 128 tokens on M and the query rows on N, O^T += V^T W^T with the 128 head
// dims on M, so a few rows fill the tensor cores' tiles.  Warp 0 streams K and V (TMA, a box of 2 KB a
// page, into a ring of 16 KB stages) and turns the queries into their parts; one thread of warp 1 issues the
// MMAs; warps 2-5, a token (of S^T) or head dim (of O^T) a thread, do the softmax.  A chunk of tiles whose
// S^T fit tensor memory is taken at once: the maxima over all of it, then its weights tile by tile.  S^T
// is double-buffered and K of chunk u + 1 streams ahead of V of chunk u.
constexpr int kSoftmaxThreads = 128;

template <int N, int STAGES>
struct Few {
  static constexpr int kTmemCols = 256;   // two CTAs per SM
  static constexpr int kChunk = (kTmemCols - N) / (2 * N);
  static constexpr int kChunkPages = kChunk * kTilePages;
  static constexpr size_t kSmem = 1024 + N * 256 + static_cast<size_t>(STAGES) * kStage + 2 * N * 256;
};

template <int N, int STAGES>
__global__ void __launch_bounds__(64 + kSoftmaxThreads, 2)
few_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using F = Few<N, STAGES>;
  constexpr int kChunk = F::kChunk;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = base;                  // two parts x N rows x 128 bytes, 128-byte swizzle
  uint8_t* sKV = sQ + N * 256;
  uint8_t* sP = sKV + STAGES * kStage;   // two buffers of two parts x N rows x 128 bytes
  __shared__ uint64_t bar_qfull, bar_qempty, bar_full[STAGES], bar_empty[STAGES];
  __shared__ uint64_t bar_sfull[2], bar_sfree[2], bar_pfull[2], bar_pempty[2];
  __shared__ uint64_t bar_oready, bar_ofull[2], bar_done;
  __shared__ uint64_t bar_cfull[kRing], bar_cempty[kRing];
  __shared__ Chunk s_chunk[kRing];
  __shared__ float2 s_scale[kRing][F::kChunkPages];   // sK, log2 sV
  __shared__ int s_page[3][F::kChunkPages];           // page * Hkv + head
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ float s_m[N], s_alpha[N], s_l[N], s_red[4][N];
  __shared__ int s_need[2], s_pflag[2];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&bar_qfull, 1);
    mbar_init(&bar_qempty, 1);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&bar_full[s], 1);
      mbar_init(&bar_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_sfull[i], 1);
      mbar_init(&bar_sfree[i], kSoftmaxThreads);
      mbar_init(&bar_pfull[i], kSoftmaxThreads);
      mbar_init(&bar_pempty[i], 1);
      mbar_init(&bar_ofull[i], 1);
    }
    mbar_init(&bar_oready, kSoftmaxThreads);
    mbar_init(&bar_done, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bar_cfull[i], 1);
      mbar_init(&bar_cempty[i], 2);   // the MMA warp and a softmax thread
    }
    abort_flag = 0;
    s_need[0] = s_need[1] = 0;
    s_pflag[0] = s_pflag[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base, F::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  const uint32_t tmem = tmem_base;
  const uint32_t tO = tmem + static_cast<uint32_t>(2 * kChunk * N);

  if (warp == 0) {
    // =================================================================== producer
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const uint64_t policy = l2_policy_evict_first();
    const int absent = p.num_pages * p.Hkv;   // past the pool: a box there reads zeros
    int st = 0, my_cum = 0;
    uint32_t ph = 0;
    bool ok = true;
    Walk<kChunk> walk;
    walk.init(p, lane, my_cum);
    uint4 qr[N / 2];    // the queries of the chunk prepared last, where it is a first one
    int q_exp = 0, q_loads = 0;
    int seq = -1;       // chunks published

    // Publishes the next chunk with its scales, and its pages for the copies.
    auto prepare = [&](Chunk& c) -> bool {
      const bool have = walk.next(p, lane, my_cum, c);
      ++seq;
      const int rs = seq % kRing;
      float2 sc[(F::kChunkPages + 31) / 32];
      if (have) {
        int* page = s_page[seq % 3];
        const int at = c.t0 / kPage, n = min(c.n_tiles * kTilePages, (c.t_end - c.t0 + kPage - 1) / kPage);
        int bad = 0;
#pragma unroll
        for (int i = 0; i < (F::kChunkPages + 31) / 32; ++i) {
          const int q = i * 32 + lane;
          int id = q < n ? __ldg(p.page_table + static_cast<size_t>(c.b) * p.max_pages + at + q) : -1;
          if (id < 0 || id >= p.num_pages) {
            bad |= q < n;
            id = -1;
          }
          const int unit = id * p.Hkv + c.kvh;
          sc[i] = id >= 0 ? __ldg(p.scales + unit) : make_float2(0.f, 0.f);
          if (q < F::kChunkPages) page[q] = id >= 0 ? unit : absent;
        }
        if (c.first) {
          float most = 0.f;
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            const int n = 2 * i + (lane >> 4);
            const int pos = c.rg * p.lsub + n / p.G;
            qr[i] = make_uint4(0, 0, 0, 0);
            if (n < p.rows && pos < p.L)
              qr[i] = __ldg(reinterpret_cast<const uint4*>(
                  p.q + ((static_cast<size_t>(c.b) * p.L + pos) * p.Hq + c.kvh * p.G + n % p.G) * 128) + (lane & 15));
          }
#pragma unroll
          for (int i = 0; i < N / 2; ++i) most = fmaxf(most, magnitude(qr[i]));
          q_exp = q_exponent(warp_max(most));
        }
        c.q_scale = pow2(q_exp) * p.scale_log2;
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.err, BDLM_DEVERR_PAGE);
      }
      if (ok) ok = mbar_wait_warp(&bar_cempty[rs], ((seq / kRing) & 1) ^ 1, &abort_flag);
      if (have) {
#pragma unroll
        for (int i = 0; i < (F::kChunkPages + 31) / 32; ++i) {
          const int q = i * 32 + lane;
          // (NaN counts as the smallest)
          const float lim = exp2f(kScaleLog), k = fminf(fmaxf(sc[i].x, 1.f / lim), lim);
          if (q < F::kChunkPages) s_scale[rs][q] = make_float2(k, fminf(fmaxf(__log2f(fmaxf(sc[i].y, 1.f / lim)), -kScaleLog), kScaleLog));
        }
      }
      __syncwarp();
      if (lane == 0) {
        if (have) {
          s_chunk[rs] = c;
        } else {
          s_chunk[rs].end = 1;
        }
        mbar_arrive(&bar_cfull[rs]);
      }
      return have;
    };
    // The parts of the prepared queries into shared memory, once the MMAs on the last ones are done.
    auto load_q = [&]() {
      if (ok) ok = mbar_wait_warp(&bar_qempty, (q_loads & 1) ^ 1, &abort_flag);
      if (!ok) return;
      const float inv = pow2(-q_exp);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const int n = 2 * i + (lane >> 4);
        const uint32_t u[4] = {qr[i].x, qr[i].y, qr[i].z, qr[i].w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) split_e4m3x2(bf16_lo(u[k]) * inv, bf16_hi(u[k]) * inv, hi[k], lo[k]);
        const uint32_t at = n * 128 + ((((lane & 15) >> 1) ^ (n & 7)) << 4) + (lane & 1) * 8;
        *reinterpret_cast<uint2*>(sQ + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
        *reinterpret_cast<uint2*>(sQ + N * 128 + at) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_qfull);
      ++q_loads;
    };
    // Streams the K or V tiles of chunk number s.
    auto emit = [&](const Chunk& c, int s, const CUtensorMap* tm) {
      for (int j = 0; j < c.n_tiles && ok; ++j) {
        if (lane == 0) {
          ok = mbar_wait(&bar_empty[st], ph ^ 1, &abort_flag);
          if (ok) mbar_arrive_expect_tx(&bar_full[st], kStage);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (lane < kTilePages)
          tma_load_3d_hint(sKV + st * kStage + lane * 2048, tm, &bar_full[st], 0, 0, s_page[s % 3][j * kTilePages + lane], policy);
        if (++st == STAGES) {
          st = 0;
          ph ^= 1;
        }
      }
    };
    // K of the next chunk, then V of this one; the one after is prepared in between, while the ring is full.
    Chunk cur, nxt, after;
    bool have = prepare(cur);
    int cs = 0;   // number of cur
    bool have_next = false;
    if (have) {
      load_q();
      emit(cur, 0, &tm_k);
      have_next = prepare(nxt);
    }
    while (have && ok) {
      bool have_after = false;
      if (have_next) {
        if (nxt.first) load_q();
        emit(nxt, cs + 1, &tm_k);
        have_after = prepare(after);
      }
      emit(cur, cs, &tm_v);
      cur = nxt;
      nxt = after;
      have = have_next;
      have_next = have_after;
      ++cs;
    }
    if (lane == 0) {
      griddep_launch_dependents();
      if (walk.counted) {
        // the last CTA to finish taking work resets the counter for the next launch
        __threadfence();
        if (atomicAdd(p.work + 1, 1) == static_cast<int>(gridDim.x) - 1) {
          p.work[0] = 0;
          p.work[1] = 0;
        }
      }
      if (!ok)
        for (int s = 0; s < STAGES; ++s) mbar_wait_drain(&bar_full[s], ph ^ (s < st ? 0 : 1));
    }
  } else if (warp == 1) {
    // =================================================================== MMA issuer
    if (lane == 0) {
      constexpr uint32_t kIdescS = idesc_e4m3_f32(128, N, false, false);
      constexpr uint32_t kIdescO = idesc_e4m3_f32(128, N, true, false);
      const uint32_t q_addr = smem_u32(sQ), kv_addr = smem_u32(sKV), p_addr = smem_u32(sP);
      bool ok = true;
      int st = 0, pcount = 0, ocount = 0, q_used = 0;
      uint32_t ph = 0;
      auto do_s = [&](const Chunk& c, int u) {
        if (!(ok = mbar_wait(&bar_sfree[u & 1], ((u >> 1) & 1) ^ 1, &abort_flag))) return;
        if (c.first) {
          if (!(ok = mbar_wait(&bar_qfull, q_used & 1, &abort_flag))) return;
          ++q_used;
        }
        for (int j = 0; j < c.n_tiles; ++j) {
          if (!(ok = mbar_wait(&bar_full[st], ph, &abort_flag))) return;
          tc_fence_after();
          const uint32_t ka = kv_addr + st * kStage;
          const uint32_t tS = tmem + static_cast<uint32_t>(((u & 1) * kChunk + j) * N);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)   // 32 head dims of either part of q
            umma_e4m3(tS, smem_desc(ka + (kk & 3) * 32, 16, 1024),
                      smem_desc(q_addr + (kk >> 2) * (N * 128) + (kk & 3) * 32, 16, 1024), kIdescS, kk > 0 ? 1u : 0u);
          umma_commit(&bar_empty[st]);
          if (++st == STAGES) {
            st = 0;
            ph ^= 1;
          }
        }
        umma_commit(&bar_sfull[u & 1]);
        if (c.last) umma_commit(&bar_qempty);
      };
      auto do_pv = [&](const Chunk& c, int u) {
        for (int j = 0; j < c.n_tiles; ++j) {
          if (!(ok = mbar_wait(&bar_full[st], ph, &abort_flag))) return;
          const int valid = min(kTile, c.t_end - (c.t0 + j * kTile));
          uint8_t* stage = sKV + st * kStage;
          if (valid % kPage != 0) {
            // slots behind the last token may hold anything (NaN); absent pages were read as zeros
            uint4* z = reinterpret_cast<uint4*>(stage + valid * 128);
            for (int o = 0; o < (kPage - valid % kPage) * 8; ++o) z[o] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          }
          const int pb = pcount & 1;
          if (!(ok = mbar_wait(&bar_pfull[pb], (pcount >> 1) & 1, &abort_flag))) return;
          if (!c.first && j == 0 && s_pflag[pb]) {   // the softmax brings O to new maxima first
            if (!(ok = mbar_wait(&bar_oready, ocount & 1, &abort_flag))) return;
            ++ocount;
          }
          tc_fence_after();
          const uint32_t va = kv_addr + st * kStage, pa = p_addr + pb * (N * 256);
          const int steps = (valid + 31) / 32;
          for (int q = 0; q < steps; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              umma_e4m3(tO, smem_desc(va + q * 4096, kStage, 1024), smem_desc(pa + h * (N * 128) + q * 32, 16, 1024),
                        kIdescO, c.first && j == 0 && q == 0 && h == 0 ? 0u : 1u);
          umma_commit(&bar_pempty[pb]);
          ++pcount;
          umma_commit(&bar_empty[st]);
          if (++st == STAGES) {
            st = 0;
            ph ^= 1;
          }
        }
        umma_commit(&bar_ofull[u & 1]);
      };
      Chunk cur, nxt;
      ok = mbar_wait(&bar_cfull[0], 0, &abort_flag);
      cur = s_chunk[0];
      if (ok && !cur.end) {
        do_s(cur, 0);
        for (int u = 0; ok; ++u) {
          const int rs = (u + 1) % kRing;
          if (!(ok = mbar_wait(&bar_cfull[rs], ((u + 1) / kRing) & 1, &abort_flag))) break;
          nxt = s_chunk[rs];
          if (!nxt.end) do_s(nxt, u + 1);   // ahead of PV(u), so that the softmax can go on meanwhile
          if (ok) do_pv(cur, u);
          if (!ok) break;
          mbar_arrive(&bar_cempty[u % kRing]);
          if (nxt.end) break;
          cur = nxt;
        }
      }
      umma_commit(&bar_done);
    }
  } else {
    // =================================================================== softmax, epilogue
    const int q4 = warp & 3;
    const int x = (q4 << 5) | lane;   // tensor-memory lane: token of a tile, or head dim
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    float l[N];
    bool ok = true;
    int pcount = 0;
    for (int u = 0; ok; ++u) {
      const int rs = u % kRing;
      if (!(ok = mbar_wait_warp(&bar_cfull[rs], (u / kRing) & 1, &abort_flag))) break;
      const Chunk c = s_chunk[rs];
      if (c.end) break;
      if (c.first) {
#pragma unroll
        for (int n = 0; n < N; ++n) l[n] = 0.f;
        if (x < N) s_m[x] = -CUDART_INF_F;
      }
      const uint32_t tS = tmem + lane_off + static_cast<uint32_t>((u & 1) * kChunk * N);
      if (!(ok = mbar_wait_warp(&bar_sfull[u & 1], (u >> 1) & 1, &abort_flag))) break;
      tc_fence_after();
      // the exact maxima of x over the chunk
#pragma unroll
      for (int cg = 0; cg < N / 16; ++cg) {
        float mx[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) mx[k] = -CUDART_INF_F;
        for (int j = 0; j < c.n_tiles; ++j) {
          uint32_t r[16];
          tmem_ld16(tS + j * N + cg * 16, r);
          const float2 sc = s_scale[rs][j * kTilePages + (x >> 4)];
          const float a = sc.x * c.q_scale;
          tmem_wait_ld();
          tmem_regs_ready(r);
          if (c.t0 + j * kTile + x < c.t_end) {
#pragma unroll
            for (int k = 0; k < 16; ++k) mx[k] = fmaxf(mx[k], fmaf(__uint_as_float(r[k]), a, sc.y));
          }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) mx[k] = warp_max(mx[k]);
        if (lane == 0) {
#pragma unroll
          for (int k = 0; k < 16; ++k) s_red[q4][cg * 16 + k] = mx[k];
        }
      }
      named_barrier(1, kSoftmaxThreads);
      if (x == 0) s_need[(u + 1) & 1] = 0;   // every reader of that slot is past this barrier
      if (x < N) {
        const float mc = fmaxf(fmaxf(s_red[0][x], s_red[1][x]), fmaxf(s_red[2][x], s_red[3][x]));
        const float mo = s_m[x];
        float alpha = 1.f;
        if (mo == -CUDART_INF_F) {
          s_m[x] = mc;
        } else if (mc - mo > kLazy) {
          alpha = ex2(mo - mc);
          s_m[x] = mc;
          s_need[u & 1] = 1;
        }
        s_alpha[x] = alpha;
      }
      named_barrier(1, kSoftmaxThreads);
      const bool need = s_need[u & 1] != 0;
      if (!c.first && need) {
        // O^T and l to the new maxima
        if (!(ok = mbar_wait_warp(&bar_ofull[(u - 1) & 1], ((u - 1) >> 1) & 1, &abort_flag))) break;
        tc_fence_after();
#pragma unroll
        for (int cg = 0; cg < N / 16; ++cg) {
          uint32_t r[16];
          tmem_ld16(tO + lane_off + cg * 16, r);
          tmem_wait_ld();
          tmem_regs_ready(r);
#pragma unroll
          for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * s_alpha[cg * 16 + k]);
          tmem_st16(tO + lane_off + cg * 16, r);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar_oready);
#pragma unroll
        for (int n = 0; n < N; ++n) l[n] *= s_alpha[n];
      }
      // the weights, tile by tile, into shared memory
      {
        float mr[N];
#pragma unroll
        for (int n = 0; n < N; ++n) mr[n] = s_m[n] - kWeightExp;
        uint32_t r[N];
#pragma unroll
        for (int cg = 0; cg < N / 16; ++cg) tmem_ld16(tS + cg * 16, *reinterpret_cast<uint32_t(*)[16]>(r + cg * 16));
        for (int j = 0; j < c.n_tiles && ok; ++j) {
          const float2 sc = s_scale[rs][j * kTilePages + (x >> 4)];
          const float a = sc.x * c.q_scale, inv = ex2(-sc.y);
          const bool valid = c.t0 + j * kTile + x < c.t_end;
          tmem_wait_ld();
#pragma unroll
          for (int cg = 0; cg < N / 16; ++cg) tmem_regs_ready(*reinterpret_cast<uint32_t(*)[16]>(r + cg * 16));
          float w[N];
#pragma unroll
          for (int n = 0; n < N; ++n) {
            w[n] = valid ? ex2(fmaf(__uint_as_float(r[n]), a, sc.y - mr[n])) : 0.f;
            l[n] = fmaf(w[n], inv, l[n]);
          }
          if (j + 1 < c.n_tiles) {
#pragma unroll
            for (int cg = 0; cg < N / 16; ++cg)
              tmem_ld16(tS + (j + 1) * N + cg * 16, *reinterpret_cast<uint32_t(*)[16]>(r + cg * 16));
          }
          const int pb = pcount & 1;
          if (!(ok = mbar_wait_warp(&bar_pempty[pb], ((pcount >> 1) & 1) ^ 1, &abort_flag))) break;
          uint8_t* pbuf = sP + pb * (N * 256) + (x & 15);
#pragma unroll
          for (int n = 0; n < N; n += 2) {
            uint32_t hi, lo;
            split_e4m3x2(w[n], w[n + 1], hi, lo);
            const uint32_t a0 = n * 128 + (((x >> 4) ^ (n & 7)) << 4), a1 = (n + 1) * 128 + (((x >> 4) ^ ((n + 1) & 7)) << 4);
            pbuf[a0] = static_cast<uint8_t>(hi);
            pbuf[a1] = static_cast<uint8_t>(hi >> 8);
            pbuf[N * 128 + a0] = static_cast<uint8_t>(lo);
            pbuf[N * 128 + a1] = static_cast<uint8_t>(lo >> 8);
          }
          if (x == 0) s_pflag[pb] = j == 0 && need;
          fence_proxy_async_smem();
          tc_fence_before();
          mbar_arrive(&bar_pfull[pb]);
          ++pcount;
        }
        if (!ok) tmem_wait_ld();
      }
      if (!ok) break;
      tc_fence_before();
      mbar_arrive(&bar_sfree[u & 1]);
      if (c.last) {
        if (!(ok = mbar_wait_warp(&bar_ofull[u & 1], (u >> 1) & 1, &abort_flag))) break;
        tc_fence_after();
#pragma unroll
        for (int n = 0; n < N; ++n) {
          float v = l[n];
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
          if (lane == 0) s_red[q4][n] = v;
        }
        named_barrier(1, kSoftmaxThreads);
        if (x < N) s_l[x] = (s_red[0][x] + s_red[1][x]) + (s_red[2][x] + s_red[3][x]);
        named_barrier(1, kSoftmaxThreads);
        if (c.slot < 0) {
          int i = c.rg * p.lsub, g = 0;
          uint16_t* o = p.out + ((static_cast<size_t>(c.b) * p.L + i) * p.Hq + static_cast<size_t>(c.kvh) * p.G) * 128 + x;
          const size_t next = static_cast<size_t>(p.Hq - p.G) * 128;   // past the other KV heads
#pragma unroll
          for (int cg = 0; cg < N / 16; ++cg) {
            uint32_t r[16];
            tmem_ld16(tO + lane_off + cg * 16, r);
            tmem_wait_ld();
            tmem_regs_ready(r);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int n = cg * 16 + k;
              if (n < p.rows && i < p.L) *o = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(r[k]) / s_l[n]));
              o += 128;
              if (++g == p.G) {
                g = 0;
                ++i;
                o += next;
              }
            }
          }
        } else {
          float* mine = p.part + static_cast<size_t>(c.slot) * N * kPartRow;
          const uint64_t keep = l2_policy_evict_last();   // read back soon
#pragma unroll
          for (int cg = 0; cg < N / 16; ++cg) {
            uint32_t r[16];
            tmem_ld16(tO + lane_off + cg * 16, r);
            tmem_wait_ld();
            tmem_regs_ready(r);
#pragma unroll
            for (int k = 0; k < 16; ++k) st_global_hint(mine + (cg * 16 + k) * 128 + x, __uint_as_float(r[k]), keep);
          }
          if (x < N) {
            st_global_hint(mine + N * 128 + x, s_m[x], keep);
            st_global_hint(mine + N * 129 + x, s_l[x], keep);
          }
        }
        tc_fence_before();
      }
      // the chunk's descriptor and scales (and O^T) are done with
      named_barrier(1, kSoftmaxThreads);
      if (x == 0) mbar_arrive(&bar_cempty[rs]);
    }
  }

  // ---- all MMAs retired before tensor memory is released
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) mbar_wait_drain(&bar_done, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, F::kTmemCols);
  }
  if (threadIdx.x == 0 && abort_flag) atomicOr(p.err, BDLM_DEVERR_TIMEOUT);
}

// Tiles of the sequences before each, for more than 32 sequences.  One CTA.
constexpr int kCumThreads = 1024;
__global__ void __launch_bounds__(kCumThreads) cum_tiles_kernel(const Params p, int* __restrict__ cum) {
  __shared__ int s_warp[32];
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += kCumThreads) {
    const int b = b0 + t;
    bool ok;
    const int n = b < p.B ? (kv_tokens(p, b, &ok) + kTile - 1) / kTile : 0;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int w = lane < 32 ? s_warp[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += v;
    }
    const int upto = warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
    const int all = __shfl_sync(0xffffffffu, w, 31);
    if (b < p.B) cum[b] = before + upto + incl - n;
    before += all;
    __syncthreads();
  }
  if (t == 0) cum[p.B] = before;
}

// Joins the parts of the lists that units' borders cut:  out = sum_s e_s O_s / sum_s e_s l_s,  e_s = 2^(m_s - M).
// CTA (list, eight rows): a warp a row where the parts are few, else eight warps a row, a part of the parts each.
constexpr int kFewParts = 16;
__global__ void __launch_bounds__(256) join_kernel(const Params p, int n_rows, int ctas) {
  __shared__ float s_acc[8][128], s_den[8], s_top[8];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lists = p.Hkv * p.row_groups;
  const int b = blockIdx.x / lists, list = blockIdx.x - b * lists;
  long long sum = 0, before = 0;
  bool ok;
  if (p.cum != nullptr) {
    sum = __ldg(p.cum + p.B);
    before = __ldg(p.cum + b);
  } else {
    const int n = lane < p.B ? (kv_tokens(p, lane, &ok) + kTile - 1) / kTile : 0;
    sum = __reduce_add_sync(0xffffffffu, n);
    before = __reduce_add_sync(0xffffffffu, lane < b ? n : 0);
  }
  const int tiles = (kv_tokens(p, b, &ok) + kTile - 1) / kTile;
  const long long per = unit_tiles(sum * lists, ctas);
  const long long c0 = before * lists + static_cast<long long>(list) * tiles;
  const int u0 = static_cast<int>(c0 / per), u1 = static_cast<int>((c0 + tiles - 1) / per);
  if (u0 == u1) return;
  const int ns = u1 - u0 + 1;
  const int rg = list % p.row_groups, kvh = list / p.row_groups;
  const size_t unit = static_cast<size_t>(n_rows) * kPartRow;
  // part s of the list: the first in its unit's second slot, the others in their units' first
  auto part = [&](int s) { return p.part + static_cast<size_t>(2 * (u0 + s) + (s == 0 ? 1 : 0)) * unit; };
  auto write = [&](int n, const float4& acc) {
    const int i = rg * p.lsub + n / p.G;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y), hi = __floats2bfloat162_rn(acc.z, acc.w);
    *reinterpret_cast<uint2*>(p.out + ((static_cast<size_t>(b) * p.L + i) * p.Hq + static_cast<size_t>(kvh) * p.G + n % p.G) * 128 +
                              4 * lane) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  };
  // sums of parts s0, s0 + step, ... of row n, relative to their largest m
  auto gather = [&](int n, int s0, int step, float& M, float& den, float4& acc) {
    M = -CUDART_INF_F;
    den = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int at = s0; at < ns; at += 32 * step) {
      const int s = at + lane * step;
      float m = -CUDART_INF_F, l = 0.f;
      if (s < ns) {
        m = __ldcg(part(s) + n_rows * 128 + n);
        l = __ldcg(part(s) + n_rows * 129 + n);
      }
      const float mn = fmaxf(M, warp_max(m));
      const float e = s < ns ? ex2(m - mn) : 0.f, was = ex2(M - mn);
      float d = e * l;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
      den = den * was + d;
      acc = make_float4(acc.x * was, acc.y * was, acc.z * was, acc.w * was);
      M = mn;
      const int cnt = min(32, (ns - at + step - 1) / step);
#pragma unroll 4
      for (int j = 0; j < cnt; ++j) {
        const float w = __shfl_sync(0xffffffffu, e, j);
        const float4 o = __ldcg(reinterpret_cast<const float4*>(part(at + j * step) + n * 128) + lane);
        acc.x += w * o.x;
        acc.y += w * o.y;
        acc.z += w * o.z;
        acc.w += w * o.w;
      }
    }
  };
  const int n0 = blockIdx.y * 8;
  float M, den;
  float4 acc;
  if (ns <= kFewParts) {
    const int n = n0 + warp;
    if (n >= p.rows || rg * p.lsub + n / p.G >= p.L) return;
    gather(n, 0, 1, M, den, acc);
    const float inv = 1.f / den;
    write(n, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    return;
  }
  for (int r = 0; r < 8; ++r) {
    const int n = n0 + r;
    if (n >= p.rows || rg * p.lsub + n / p.G >= p.L) return;
    gather(n, warp, 8, M, den, acc);
    *reinterpret_cast<float4*>(&s_acc[warp][4 * lane]) = acc;
    if (lane == 0) {
      s_den[warp] = den;
      s_top[warp] = M;
    }
    __syncthreads();
    if (warp == r) {
      float top = s_top[0];
      for (int w = 1; w < 8; ++w) top = fmaxf(top, s_top[w]);
      float d = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < 8; ++w) {
        const float e = ex2(s_top[w] - top);
        const float4 o = *reinterpret_cast<const float4*>(&s_acc[w][4 * lane]);
        d += e * s_den[w];
        a.x += e * o.x;
        a.y += e * o.y;
        a.z += e * o.z;
        a.w += e * o.w;
      }
      const float inv = 1.f / d;
      write(n, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
    }
    __syncthreads();
  }
}

template <int N, int STAGES>
cudaError_t launch_few(const CUtensorMap& tk, const CUtensorMap& tv, const Params& p, int grid, cudaStream_t stream) {
  constexpr size_t smem = Few<N, STAGES>::kSmem;
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = once_per_device(attr_done, [] {
    const cudaError_t r = cudaFuncSetAttribute(few_rows_kernel<N, STAGES>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(few_rows_kernel<N, STAGES>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(few_rows_kernel<N, STAGES>, dim3(grid), dim3(64 + kSoftmaxThreads), smem, stream, tk, tv, p);
}

}  // namespace

Kv8AttnPlan plan_attention_kv8(int B, int L, int Hq, int Hkv, int max_pages, int num_sms) {
  Kv8AttnPlan pl;
  const int G = Hq / Hkv;
  pl.lsub = G * L <= 32 ? L : 32 / G;
  pl.row_groups = (L + pl.lsub - 1) / pl.lsub;
  pl.rows = G * pl.lsub;
  pl.n_rows = pl.rows <= 16 ? 16 : 32;
  const long long tiles = static_cast<long long>(B) * Hkv * pl.row_groups * ((max_pages + kTilePages - 1) / kTilePages);
  pl.grid = static_cast<int>(tiles < 2ll * num_sms ? tiles : 2ll * num_sms);
  const long long units = tiles < static_cast<long long>(kRounds) * pl.grid ? tiles : static_cast<long long>(kRounds) * pl.grid;
  // (a tile a list at most: no list is cut)
  pl.parts = max_pages <= kTilePages ? 0 : 2 * units;
  pl.part_bytes = static_cast<size_t>(pl.parts) * pl.n_rows * kPartRow * sizeof(float);
  pl.cum_offset = (pl.part_bytes + 255) / 256 * 256;
  pl.bytes = pl.cum_offset + (B > 32 ? (static_cast<size_t>(B) + 1) * sizeof(int) : 0);
  return pl;
}

cudaError_t launch_attention_kv8(const Kv8AttnParams& a, const Kv8AttnPlan& pl, const CUtensorMap& tk, const CUtensorMap& tv,
                                 void* data, int* work, cudaStream_t stream) {
  Params p;
  p.q = a.q;
  p.scales = reinterpret_cast<const float2*>(a.scales);
  p.page_table = a.page_table;
  p.prefix_lens = a.prefix_lens;
  p.out = a.out;
  p.part = static_cast<float*>(data);
  p.err = a.err;
  p.work = work;
  p.cum = nullptr;
  p.B = a.B;
  p.L = a.L;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.lsub = pl.lsub;
  p.row_groups = pl.row_groups;
  p.rows = pl.rows;
  p.scale_log2 = a.scale_log2;
  cudaError_t e;
  if (a.B > 32) {
    int* cum = reinterpret_cast<int*>(static_cast<char*>(data) + pl.cum_offset);
    e = launch_pdl(cum_tiles_kernel, dim3(1), dim3(kCumThreads), 0, stream, p, cum);
    if (e != cudaSuccess) return e;
    p.cum = cum;
  }
  e = pl.n_rows == 16 ? launch_few<16, 6>(tk, tv, p, pl.grid, stream) : launch_few<32, 5>(tk, tv, p, pl.grid, stream);
  if (e != cudaSuccess || pl.parts == 0) return e;
  const dim3 grid(static_cast<unsigned>(p.B) * p.Hkv * p.row_groups, (p.rows + 7) / 8);
  return launch_pdl(join_kernel, grid, dim3(256), 0, stream, p, pl.n_rows, pl.grid);
}

}  // namespace bdlm
