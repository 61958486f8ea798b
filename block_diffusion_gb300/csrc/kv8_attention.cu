// Block attention over the 8-bit cache, for sm_103a.
//
//     out = sum_t p_t sV_t v_t / sum_t p_t,   p_t = 2^(c sK_t q . k_t - m),   c = sm_scale log2 e
// with codes k_t, v_t in e4m3 and the scales sK_t, sV_t of a token's page and head.
//
//  * The codes go from memory to the tensor cores as they are (tcgen05 kind::f8f6f4, which adds up in
//    float32), so nothing is widened on the way and a token costs 256 bytes of shared memory.  The
//    other operand has 8 bits as well: q and p are held as two e4m3 parts each, the value rounded to four
//    bits and what that leaves, rounded to four bits again.  A pair is off by 2^-8 of the value, as bf16
//    is, and by no less than half its smallest step: of q 2^-17.8 of the row's largest value, of a weight 2^-23 of
//    the query's largest in its chunk of tokens.  A row of q has a power of two of its own, so none depends on another
//    (128 blocks of 8 took 143.5 us with one a list, 148.4 so).  The weights' second part is 2^5 times itself, with
//    sums apart, and every chunk's weights are taken to its own maximum: with one dominant token the others' are small,
//    many, and all needed (held next to the list's maximum, without the 2^5, 32768 tokens beside one of 90 % came out
//    two fifths too small).  Twice the products of one part, at twice bf16's rate.
//  * A page's scale of K is a factor of its scores.  Its scale of V goes into the weight: with
//        x_t = c sK_t q . k_t + log2 sV_t    and its maximum m,
//    w_t = 2^(x_t - m + 8) is what the second product takes (no sum ever meets a scale) and
//    sum w_t / sV_t is the divisor.  So w's parts keep their precision where it counts, whatever the
//    scales are from page to page.
//  * Work: the tiles of 128 tokens of all (sequence, KV head, row group) lists, end to end, are cut
//    into units of equal numbers of tiles, one a CTA.  A list that a unit's border cuts is written in parts
//    (O, m, l), at most two a unit, that are joined in order: by the CTA that writes the last of them, or by a
//    kernel behind (plan_attention_kv8).  So the work is even whatever the lengths.
//
// Bound: the codes, 256 bytes a token and KV head, come once from HBM.  Measured (a graph of calls):
//     64 blocks of 2 over 2000-8000 tokens, 4 rows a KV head .... 104 us, 6.3 TB/s (93 % of the copy rate)
//     128 blocks of 4 over 512-4096 tokens, 16 rows a KV head ... 108.5 us, 5.7 TB/s (83 %)
//     32 single tokens over 16384-32768 tokens, 8 rows .......... 123 us, 6.6 TB/s (97 %)
//     128 blocks of 8 over 512-4096 tokens, 32 rows ............. 148 us, 4.2 TB/s (61 %): lists' ends
//     16 blocks of 32 over 8192-16384 tokens, 128 rows .......... 123 us, 3.4 TB/s: the softmax's latency
//     16 blocks of 64 over 8192-16384 tokens, 256 rows .......... 197 us, 1.05 PFLOP/s (55 %): MMAs and softmax in turn
//     1024 single tokens over 100-1000 tokens, 4 rows ........... 197 us, 5.9 TB/s (88 %)
//     one block of 4 over 2000 tokens, 8 rows .................... 10.6 us, latency
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "attention_common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "ptx_kv8.cuh"
#include "step_ops.h"

namespace bdlm {
namespace {

constexpr int kTilePages = kTile / kPage;
constexpr int kStage = kTile * 128;    // bytes of a tile's K or V
constexpr int kRing = 4;               // chunk descriptors in flight
constexpr int kAllTiles = 0x7FFFFFFF;  // a chunk as long as its list
constexpr float kWeightExp = 8.0f;     // a query's largest weight of a chunk is 2^8 (e4m3 ends at 448) ...
constexpr float kReach = 24.0f;        // ... or less: sums in a far lower power of two than the list's largest would overflow
constexpr float kLowPart = 32.0f;      // the second part: of weights up to 2^8 the first leaves 2^3 at most
constexpr float kWeightExpMany = 7.0f; // the same where weights are float16: 2^7 ...
constexpr float kLazyMany = 8.0f;      // ... to 2^15: a running maximum moves only when it rises by more

struct Params {
  const uint16_t* q;
  const float2* scales;
  const int32_t* page_table;
  const int32_t* prefix_lens;
  uint16_t* out;
  float* part;       // unit u's parts: 2u (of a list that began before it), 2u + 1 (of one that begins in it)
  int* err;
  int* work;         // [0] CTAs finished, then parts written of the list that each unit's end cuts (join_here)
  const int* cum;    // [B + 1] tiles of the sequences before each (null: up to kFewSequences sequences)
  const float* q_scale;   // many rows: 2^e of each query
  int B, L, Hq, Hkv, G, max_pages, num_pages, lsub, row_groups, rows;
  int join_here;     // the CTA that writes a list's last part joins them
  float scale_log2;
};
constexpr int kFewSequences = 256;

// Some tiles of a list, as the warps pass them on.
struct Chunk {
  int b, kvh, rg;
  int t0, t_end;     // first token; end of the list's tokens (or past the chunk)
  int n_tiles;
  int first, last;   // of the tiles that this CTA sums up together
  int slot;          // part to write at the last chunk, -1: the output
  int u0, parts;     // the list's first unit and its parts (slot >= 0)
  int final;         // the CTA's last chunk
  int end;           // no chunk: the CTA has no work
};

__device__ __forceinline__ int kv_tokens(const Params& p, int b, bool* ok) {
  const int prefix = __ldg(p.prefix_lens + b);
  const long long max_tok = static_cast<long long>(p.max_pages) * kPage;
  const long long n = static_cast<long long>(prefix < 0 ? 0 : prefix) + p.L;
  *ok = prefix >= 0 && n <= max_tok;
  return static_cast<int>(n < max_tok ? n : max_tok);
}

// a / b of numbers of tiles, which 32 bits mostly hold (a division of 64 takes some 150 cycles).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

// mbar_wait_warp; FAR: with all that follows a first failed try out of line.  Its loops in every place that waits made the
// warps wait for instructions: 128 blocks of 8 over 512-4096 tokens 153 us against 145, 1024 sequences of 100-1000 tokens
// 221 against 206, 16 blocks of 32 over 8192-16384 124.5 against 122.  With 256 rows, whose softmax has no registers to
// spare for a call, in line: 16 blocks of 64 197 us against 200.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, int* abort) { return mbar_wait_warp(bar, parity, abort); }
template <bool FAR>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* abort) {
  if constexpr (!FAR) return mbar_wait_warp(bar, parity, abort);
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return wait_on(bar, parity, abort);
}

// Tiles of a unit, a CTA's even share of all.  (Shares of a quarter, taken in turn, were no faster: what they gain
// in evenness goes into four times the parts.)
__device__ __forceinline__ long long unit_tiles(long long total, int ctas) {
  const long long share = quotient(total + ctas - 1, ctas);
  return share < 1 ? 1 : share;
}

// Tiles of the sequences before each: in the lanes of a warp, or in memory.
struct Before {
  int own[kFewSequences / 32];   // lane l: before sequence 32 i + l
  int all;

  __device__ __forceinline__ void init(const Params& p, int lane) {
    if (p.cum != nullptr) {
      all = __ldg(p.cum + p.B);
      return;
    }
    bool ok;
#pragma unroll
    for (int i = 0; i < kFewSequences / 32; ++i) {
      const int b = i * 32 + lane;
      own[i] = b < p.B ? (kv_tokens(p, b, &ok) + kTile - 1) / kTile : 0;
    }
    all = 0;
#pragma unroll
    for (int i = 0; i < kFewSequences / 32; ++i) {
      if (i * 32 >= p.B) break;
      int incl = own[i];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
      }
      own[i] = all + incl - own[i];
      all += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  // The sequence that tile x lies in, and the tiles before it.
  __device__ __forceinline__ int find(const Params& p, int lane, int x, int& before) const {
    int b = 0;
    if (p.cum == nullptr) {
#pragma unroll
      for (int i = 0; i < kFewSequences / 32; ++i) {
        if (i * 32 >= p.B) break;
        const int c = __popc(__ballot_sync(0xffffffffu, i * 32 + lane < p.B && own[i] <= x));
        if (c > 0) {
          b = i * 32 + c - 1;
          before = __shfl_sync(0xffffffffu, own[i], c - 1);
        }
      }
    } else {
      int n = p.B;
      while (n > 1) {
        const int step = (n + 31) / 32;
        const int c = __popc(__ballot_sync(0xffffffffu, lane * step < n && __ldg(p.cum + b + (lane * step < n ? lane * step : 0)) <= x)) - 1;
        b += c * step;
        n = min(step, n - c * step);
      }
      before = __ldg(p.cum + b);
    }
    return b;
  }
};

// a and b in two e4m3 parts: each the low half for a, the high one for b.
__device__ __forceinline__ void split_e4m3x2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = e4m3x2(a, b);
  const float2 h = from_e4m3x2(hi);
  lo = e4m3x2(a - h.x, b - h.y);
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The larger of two bf16 pairs, half by half (a NaN counts as nothing beside a number) ...
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
// ... and the magnitudes of eight values, as far as that goes.
__device__ __forceinline__ uint32_t magnitude(const uint4& w) {
  constexpr uint32_t kNoSign = 0x7FFF7FFFu;
  return max_pair(max_pair(w.x & kNoSign, w.y & kNoSign), max_pair(w.z & kNoSign, w.w & kNoSign));
}

// The largest magnitude of R queries, 16 lanes a query: lane l has query l R / 16's.  (A shuffle for each two lanes and query
// that are still apart, 15 for 16 queries instead of 64.)
template <int R>
__device__ __forceinline__ float rows_max(uint32_t (&m)[R], int lane) {
  int left = R;
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) {
    const bool up = lane & off;
    if (left > 1) {
      left /= 2;
#pragma unroll
      for (int i = 0; i < R / 2; ++i) {
        if (i >= left) break;
        const uint32_t give = up ? m[i] : m[i + left], keep = up ? m[i + left] : m[i];
        m[i] = max_pair(keep, __shfl_xor_sync(0xffffffffu, give, off));
      }
    } else {
      m[0] = max_pair(m[0], __shfl_xor_sync(0xffffffffu, m[0], off));
    }
  }
  return fmaxf(bf16_lo(m[0]), bf16_hi(m[0]));
}

// The power of two 2^e that takes a largest magnitude to 448 or less (and above 224 where it can).
__device__ __forceinline__ int q_exponent(float most) { return min(max(e4m3_exponent(most), -110), 120); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
// What scores of queries over 2^e are multiplied by, beside a page's sK: 2^e c, or 2^-86 where that is less.  Times the
// least sK, 2^-40, it is a normal number then: a score of -inf (behind the last token) stays one, where 0 would make it
// NaN.  Scores below it are 0 to within 2^25 2^40 2^-86 = 2^-21 either way.
__device__ __forceinline__ float q_factor(float pow2_e, float scale_log2) { return fmaxf(pow2_e * scale_log2, 1.2924697071141057e-26f); }

// A page's sK and log2 sV, as the softmax takes them (NaN counts as the smallest).
__device__ __forceinline__ float2 page_scale(float2 s) {
  constexpr float kLeast = 9.094947017729282e-13f, kMost = 1099511627776.f;   // 2^-40, 2^40
  return make_float2(fminf(fmaxf(s.x, kLeast), kMost), __log2f(fminf(fmaxf(s.y, kLeast), kMost)));
}

// The walk over a CTA's unit, list by list, in chunks of up to CHUNK tiles (whole warp, uniform).
template <int CHUNK>
struct Walk {
  long long per, pos, end;          // in tiles; pos: of what comes after the list at hand
  int b, kv_len, tiles, lists;      // the sequence at pos
  long long base;                   // tiles before it
  int kvh, rg, tile, seg_end, slot, u0, parts;
  bool len_ok, fresh;

  __device__ __forceinline__ void init(const Params& p, int lane) {
    Before before;
    before.init(p, lane);
    lists = p.Hkv * p.row_groups;
    const long long total = static_cast<long long>(before.all) * lists;
    per = unit_tiles(total, gridDim.x);
    pos = blockIdx.x * per;
    end = pos + per < total ? pos + per : total;
    tile = seg_end = 0;
    if (pos >= end) {
      pos = end;
      return;
    }
    int n;
    b = before.find(p, lane, static_cast<int>(quotient(pos, lists)), n);   // before[b] <= pos / lists < before[b + 1]
    base = static_cast<long long>(n) * lists;
    sequence(p);
  }

  __device__ __forceinline__ void sequence(const Params& p) {
    kv_len = kv_tokens(p, b, &len_ok);
    tiles = (kv_len + kTile - 1) / kTile;
  }

  // The next chunk; false: no work is left.
  __device__ __forceinline__ bool next(const Params& p, int lane, Chunk& c) {
    fresh = tile == seg_end;
    if (fresh) {
      if (pos == end) return false;
      long long r = pos - base;
      if (r >= static_cast<long long>(tiles) * lists) {
        base += static_cast<long long>(tiles) * lists;
        r = 0;
        ++b;
        sequence(p);
      }
      const int list = static_cast<int>(quotient(r, tiles));
      rg = list % p.row_groups;
      kvh = list / p.row_groups;
      tile = static_cast<int>(r - static_cast<long long>(list) * tiles);
      const int n = static_cast<int>(min(static_cast<long long>(tiles - tile), end - pos));
      slot = -1;
      if (n < tiles) {
        const long long c0 = pos - tile;   // the list's first tile
        u0 = tile == 0 ? static_cast<int>(blockIdx.x) : static_cast<int>(quotient(c0, per));
        parts = static_cast<int>(quotient(c0 + tiles - 1, per)) - u0 + 1;
        slot = 2 * static_cast<int>(blockIdx.x) + (tile == 0 ? 1 : 0);
      }
      seg_end = tile + n;
      pos += n;
      if (!len_ok && tile == 0 && list == 0 && lane == 0) atomicOr(p.err, BDLM_DEVERR_LENGTH);
    }
    c.b = b;
    c.kvh = kvh;
    c.rg = rg;
    c.t0 = tile * kTile;
    c.t_end = kv_len;
    c.n_tiles = min(CHUNK, seg_end - tile);
    tile += c.n_tiles;
    c.first = fresh;
    c.last = tile == seg_end;
    c.slot = slot;
    c.u0 = u0;
    c.parts = parts;
    c.final = c.last && pos == end;
    c.end = 0;
    return true;
  }
};

// A chunk's pages (page * Hkv + head, or `absent`) and scales, asked for lane by lane.
template <int PAGES>
struct PageLoads {
  static constexpr int kEach = (PAGES + 31) / 32;
  int unit[kEach];
  float2 scale[kEach];

  static __device__ __forceinline__ int count(const Chunk& c) {
    return min(c.n_tiles * kTilePages, (c.t_end - c.t0 + kPage - 1) / kPage);
  }
  __device__ __forceinline__ void ask_pages(const Params& p, const Chunk& c, int lane) {
    const int at = c.t0 / kPage, n = count(c);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int q = i * 32 + lane;
      unit[i] = q < n ? __ldg(p.page_table + static_cast<size_t>(c.b) * p.max_pages + at + q) : -1;
    }
  }
  __device__ __forceinline__ void ask_scales(const Params& p, const Chunk& c, int lane) {
    const int n = count(c);
    int bad = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      int id = unit[i];
      if (id < 0 || id >= p.num_pages) {
        bad |= i * 32 + lane < n;
        id = -1;
      }
      unit[i] = id >= 0 ? id * p.Hkv + c.kvh : p.num_pages * p.Hkv;   // past the pool: a box there reads zeros
      scale[i] = id >= 0 ? __ldg(p.scales + unit[i]) : make_float2(0.f, 0.f);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.err, BDLM_DEVERR_PAGE);
  }
  __device__ __forceinline__ void give(int* units, float2* scales, int lane) const {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int q = i * 32 + lane;
      if (q < PAGES) {
        units[q] = unit[i];
        scales[q] = page_scale(scale[i]);
      }
    }
  }
};

constexpr int kPartRow = 130;   // floats of a row's part: O, m, l
constexpr int kFewParts = 8;    // parts a list, about

// ------------------------------------------------------------------ up to 32 query rows per KV head
//
// Transposed: S^T = K Q^T with 128 tokens on M and the query rows on N, O^T += V^T W^T with the 128 head
// dims on M, so a few rows fill the tensor cores' tiles.  One warp walks the work ahead of all others and looks up
// pages and scales.  Warp 0 streams K and V (TMA, a box of 2 KB a page, into a ring of 16 KB stages); warp 1 turns the
// queries into their parts and issues the first MMAs, the last warp the second; four warps for every 16 rows, a
// token (of S^T) or head dim (of O^T) a thread, do the softmax.  A chunk of tiles whose S^T fit tensor memory is
// taken at once: the maxima over all of it, then its weights tile by tile.  S^T is double-buffered and K of chunk
// u + 1 streams ahead of V of chunk u.
//
// Bound: HBM with up to 16 rows.  With 32, each list's end (the last weights, O^T out, the next queries) holds the one CTA
// of an SM up for about a tile's time: 32 blocks of 8 over 2000-16000 tokens run at 4.7 TB/s, 128 over 512-4096 at 4.2.

// N: rows of the first MMAs, NC: rows that the softmax computes.
template <int N, int NC, int STAGES>
struct Few {
  static constexpr int CW = NC < 16 ? NC : 16;
  static constexpr int kSets = NC / CW;         // of softmax warps: 16 rows each (8), of all tokens
  static constexpr int kSoft = 128 * kSets;     // their threads
  static constexpr int kThreads = 128 + kSoft;
  static constexpr int kWalkWarp = 2 + kSoft / 32, kSecondWarp = kWalkWarp + 1;
  // Two CTAs per SM with 16 rows.  With 32 one, twice as wide: two left chunks of three tiles, whose ends took as long as
  // they (128 blocks of 8 over 512-4096 tokens: 186 us against 170, before the MMAs had a warp each).
  static constexpr int kCtas = N == 16 ? 2 : 1;
  static constexpr int kTmemCols = 512 / kCtas;
  static constexpr int kWeights = 2 * NC;       // rows of the second MMAs: both parts of the weights
  static constexpr int kWeightBuf = kWeights * kTile;
  static constexpr int kChunk = (kTmemCols - kWeights) / (2 * N);
  static constexpr int kChunkPages = kChunk * kTilePages;
  static constexpr size_t kSmem = 1024 + N * 256 + static_cast<size_t>(STAGES) * kStage + 2 * kWeightBuf;
};

// w's float16 pair in two e4m3 parts, the second kLowPart times itself (exact in float16): each the low byte for the low
// one.
__device__ __forceinline__ void split_half2(uint32_t w, uint32_t& hi, uint32_t& lo) {
  const __half2 h = *reinterpret_cast<const __half2*>(&w);
  hi = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(h), __NV_SATFINITE, __NV_E4M3);
  const __half2_raw back = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(hi), __NV_E4M3);
  const __half2 rest = __hmul2(__hsub2(h, *reinterpret_cast<const __half2*>(&back)), __float2half2_rn(kLowPart));
  lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(rest), __NV_SATFINITE, __NV_E4M3);
}

// Joins the parts of chunk c's list, in their order whoever comes last:
//     out = sum_s e_s O_s / sum_s e_s l_s,   e_s = 2^(m_s - M),
// two parts at a time, M and the sums brought along.  128 threads, a head dim each.
// Rows c0 .. c0 + CW - 1, of which `live` are there, from `row` of the output on; s_*: those rows'.
template <int N, int CW>
__device__ __forceinline__ void join_parts(const Params& p, const Chunk& c, int x, int c0, size_t row, int g, int live, float* s_l,
                                           float* s_alpha, float* s_e0, float* s_e1, int barrier) {
  auto part = [&](int s) { return p.part + static_cast<size_t>(2 * (c.u0 + s) + (s == 0 ? 1 : 0)) * N * kPartRow; };
  float acc[CW];
#pragma unroll
  for (int n = 0; n < CW; ++n) acc[n] = 0.f;
  float M = -CUDART_INF_F, den = 0.f;   // threads x < CW: of row c0 + x
#pragma unroll 1
  for (int s0 = 0; s0 < c.parts; s0 += 2) {
    const bool two = s0 + 1 < c.parts;
    const float *a = part(s0), *b = part(two ? s0 + 1 : s0);
    float o0[CW], o1[CW];
#pragma unroll
    for (int n = 0; n < CW; ++n) {
      o0[n] = n < live ? __ldcg(a + (c0 + n) * 128 + x) : 0.f;
      o1[n] = n < live ? __ldcg(b + (c0 + n) * 128 + x) : 0.f;
    }
    if (x < CW) {
      const float m0 = __ldcg(a + N * 128 + c0 + x), l0 = __ldcg(a + N * 129 + c0 + x);
      const float m1 = two ? __ldcg(b + N * 128 + c0 + x) : -CUDART_INF_F, l1 = __ldcg(b + N * 129 + c0 + x);
      const float top = fmaxf(M, fmaxf(m0, m1));
      const float was = ex2(M - top), e0 = ex2(m0 - top), e1 = ex2(m1 - top);
      den = fmaf(den, was, fmaf(e0, l0, e1 * l1));
      M = top;
      s_alpha[x] = was;
      s_e0[x] = e0;
      s_e1[x] = e1;
    }
    named_barrier(barrier, 128);
#pragma unroll
    for (int n = 0; n < CW; ++n) acc[n] = fmaf(acc[n], s_alpha[n], fmaf(s_e0[n], o0[n], s_e1[n] * o1[n]));
    named_barrier(barrier, 128);
  }
  if (x < CW) s_l[x] = 1.f / den;
  named_barrier(barrier, 128);
#pragma unroll
  for (int n = 0; n < CW; ++n) {
    if (n >= live) break;
    p.out[row * 128 + x] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[n] * s_l[n]));
    ++row;
    if (++g == p.G) {
      g = 0;
      row += p.Hq - p.G;
    }
  }
}

template <int N, int NC, int STAGES>
__global__ void __launch_bounds__(Few<N, NC, STAGES>::kThreads, Few<N, NC, STAGES>::kCtas)
few_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using F = Few<N, NC, STAGES>;
  constexpr int CW = F::CW;
  constexpr int kChunk = F::kChunk;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = base;                  // two parts x N rows x 128 bytes, 128-byte swizzle
  uint8_t* sKV = sQ + N * 256;
  uint8_t* sP = sKV + STAGES * kStage;   // two buffers of kWeights / 16 x 128 tokens x 16 bytes: a byte of each row
  __shared__ uint64_t bar_qempty, bar_kfull[STAGES], bar_vfull[STAGES], bar_empty[STAGES];
  __shared__ uint64_t bar_sfull[2], bar_sfree[2], bar_pfull[2], bar_pempty[2];
  __shared__ uint64_t bar_ofull[2], bar_done;
  __shared__ uint64_t bar_cfull[kRing], bar_cempty[kRing];
  __shared__ Chunk s_chunk[kRing];
  __shared__ float2 s_scale[kRing][F::kChunkPages];   // sK, log2 sV
  __shared__ int s_page[kRing][F::kChunkPages];       // page * Hkv + head
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ __align__(16) float s_m[N], s_top[N], s_alpha[N], s_l[N], s_red[4][N];
  __shared__ int s_leave[F::kSets][2], s_join[F::kSets];
  __shared__ __align__(16) float s_qscale[4][N];   // of a list's rows, times c: lists in turn (the softmax is two behind at most)

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&bar_qempty, 1);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&bar_kfull[s], 1);   // (apart: a warp that skips the other's tiles would meet a parity of two fills ago)
      mbar_init(&bar_vfull[s], 1);
      mbar_init(&bar_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_sfull[i], 2);   // the MMAs, and the queries' scale
      mbar_init(&bar_sfree[i], F::kSoft);
      mbar_init(&bar_pfull[i], F::kSoft);
      mbar_init(&bar_pempty[i], 1);
      mbar_init(&bar_ofull[i], 1);
    }
    mbar_init(&bar_done, 2);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bar_cfull[i], 1);
      mbar_init(&bar_cempty[i], 2 + F::kSets);   // copies, second MMAs, softmax
    }
    abort_flag = 0;
    for (int s = 0; s < F::kSets; ++s) s_leave[s][0] = s_leave[s][1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base, F::kTmemCols);
    tmem_relinquish();
  }
  // The walk begins beside the set-up.  Its first two chunks are asked for together: once the copies of the first are
  // under way a look-up takes microseconds, and the copies would stand still for the second's.  From then on the walk is
  // chunks ahead.  The first MMAs' warp walks from list to list, for
  // the queries.
  Walk<kChunk> walk;
  Walk<kAllTiles> lists;
  Chunk c, d;
  PageLoads<F::kChunkPages> pages, ahead;
  uint4 qr[NC / 2];   // rows 2i and 2i + 1 of the queries, eight values a lane
  auto ask_q = [&](const Chunk& c) {
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) {
      const int n = 2 * i + (lane >> 4);
      const int pos = c.rg * p.lsub + n / p.G;
      qr[i] = make_uint4(0, 0, 0, 0);
      if (n < p.rows && pos < p.L)
        qr[i] = __ldg(reinterpret_cast<const uint4*>(
            p.q + ((static_cast<size_t>(c.b) * p.L + pos) * p.Hq + c.kvh * p.G + n % p.G) * 128) + (lane & 15));
    }
  };
  if (warp == F::kWalkWarp) {
    griddep_wait();
    walk.init(p, lane);
    c.final = 1;
    c.end = !walk.next(p, lane, c);
    if (!c.end) {
      pages.ask_pages(p, c, lane);
      if (!c.final) {
        walk.next(p, lane, d);
        ahead.ask_pages(p, d, lane);
      }
      pages.ask_scales(p, c, lane);
      if (!c.final) ahead.ask_scales(p, d, lane);
    }
  } else if (warp == 1) {
    griddep_wait();
    lists.init(p, lane);
    c.end = !lists.next(p, lane, c);
    if (!c.end) ask_q(c);
    for (int n = NC; n < N; ++n)   // rows that no query fills
      *reinterpret_cast<uint2*>(sQ + (lane >> 4) * (N * 128) + n * 128 + (lane & 15) * 8) = make_uint2(0, 0);
    if (!c.end) c.end = !lists.next(p, lane, c);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  const uint32_t tmem = tmem_base;
  const uint32_t tO = tmem + static_cast<uint32_t>(2 * kChunk * N);

  if (warp == 0) {
    // =================================================================== copies
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const uint64_t policy = l2_policy_evict_first();
    int st = 0;
    uint32_t ph = 0, kbits = 0, vbits = 0;   // parities of the stages' next fills with K, with V
    bool ok = true;
    auto emit = [&](int s, int n_tiles, const CUtensorMap* tm, uint64_t* full, uint32_t& bits) {   // of chunk number s
      for (int j = 0; j < n_tiles && ok; ++j) {
        if (!(ok = wait_warp<true>(&bar_empty[st], ph ^ 1, &abort_flag))) break;
        if (lane == 0) mbar_arrive_expect_tx(&full[st], kStage);
        bits ^= 1u << st;
        __syncwarp();
        if (lane < kTilePages)
          tma_load_3d_hint(sKV + st * kStage + lane * 2048, tm, &full[st], 0, 0, s_page[s % kRing][j * kTilePages + lane], policy);
        if (++st == STAGES) {
          st = 0;
          ph ^= 1;
        }
      }
    };
    // K of the next chunk, then V of this one
    if ((ok = wait_warp<true>(&bar_cfull[0], 0, &abort_flag)) && !s_chunk[0].end) {
      int n_tiles = s_chunk[0].n_tiles, final = s_chunk[0].final;
      emit(0, n_tiles, &tm_k, bar_kfull, kbits);
      for (int u = 0; ok; ++u) {
        int next = 0, next_final = 0;
        if (!final) {
          const int rs = (u + 1) % kRing;
          if (!(ok = wait_warp<true>(&bar_cfull[rs], ((u + 1) / kRing) & 1, &abort_flag))) break;
          next = s_chunk[rs].n_tiles;
          next_final = s_chunk[rs].final;
          emit(u + 1, next, &tm_k, bar_kfull, kbits);
        }
        emit(u, n_tiles, &tm_v, bar_vfull, vbits);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_cempty[u % kRing]);
        if (final) break;
        n_tiles = next;
        final = next_final;
      }
    }
    if (lane == 0) {
      griddep_launch_dependents();
      if (!ok)
        for (int s = 0; s < STAGES; ++s) {
          mbar_wait_drain(&bar_kfull[s], ((kbits >> s) & 1) ^ 1);
          mbar_wait_drain(&bar_vfull[s], ((vbits >> s) & 1) ^ 1);
        }
    }
  } else if (warp == 1) {
    // =================================================================== queries, first MMAs
    // One warp each for the first and the second MMAs: a warp that issued both was busy with it for most of the time (128
    // blocks of 8 over 512-4096 tokens: 158 us against 153), and stood still for one's operands where it could have issued
    // the other's.
    constexpr uint32_t kIdescS = idesc_format0_f32(128, N, false, false);
    const uint64_t q_desc = smem_desc(smem_u32(sQ), 16, 1024), k_desc = smem_desc(smem_u32(sKV), 16, 1024);
    bool ok = true;
    int st = 0, n_list = 0;
    uint32_t bits = 0;   // parities of the stages' next fills with K
    // The list's queries in their two parts, once the MMAs on the last one's are done; the next one's are asked for, the
    // walk a list ahead of that.
    auto next_q = [&]() {
      constexpr int R = NC / 2;   // rows of each half of the warp
      uint32_t most[R];
#pragma unroll
      for (int i = 0; i < R; ++i) most[i] = magnitude(qr[i]);
      const int e = q_exponent(rows_max(most, lane));
      if (!(ok = wait_warp<true>(&bar_qempty, (n_list & 1) ^ 1, &abort_flag))) return;
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) {
        const int n = 2 * i + (lane >> 4);
        const float inv = __shfl_sync(0xffffffffu, pow2(-e), (lane & 16) | i * (16 / R));
        const uint32_t u[4] = {qr[i].x, qr[i].y, qr[i].z, qr[i].w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) split_e4m3x2(bf16_lo(u[k]) * inv, bf16_hi(u[k]) * inv, hi[k], lo[k]);
        const uint32_t at = n * 128 + ((((lane & 15) >> 1) ^ (n & 7)) << 4) + (lane & 1) * 8;
        *reinterpret_cast<uint2*>(sQ + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
        *reinterpret_cast<uint2*>(sQ + N * 128 + at) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
      }
      if (lane % (16 / R) == 0) s_qscale[n_list & 3][(lane & 15) / (16 / R) * 2 + (lane >> 4)] = q_factor(pow2(e), p.scale_log2);
      fence_proxy_async_smem();
      __syncwarp();
      ++n_list;
      if (!c.end) {
        ask_q(c);
        c.end = !lists.next(p, lane, c);
      }
    };
    int skip = 0;   // V's tiles of the chunk before the last, between the copies of K
    for (int u = 0; ok; ++u) {
      const int rs = u % kRing;
      if (!(ok = wait_warp<true>(&bar_cfull[rs], (u / kRing) & 1, &abort_flag))) break;
      const int n_tiles = s_chunk[rs].n_tiles, first = s_chunk[rs].first, last = s_chunk[rs].last, final = s_chunk[rs].final;
      if (s_chunk[rs].end) break;
      if (first) next_q();
      if (!ok || !(ok = wait_warp<true>(&bar_sfree[u & 1], ((u >> 1) & 1) ^ 1, &abort_flag))) break;
      if (lane == 0) mbar_arrive(&bar_sfull[u & 1]);
      for (int j = 0; j < n_tiles; ++j) {
        if (!(ok = wait_warp<true>(&bar_kfull[st], (bits >> st) & 1, &abort_flag))) break;
        bits ^= 1u << st;
        tc_fence_after();
        const uint32_t tS = tmem + static_cast<uint32_t>(((u & 1) * kChunk + j) * N);
        const uint64_t kd = k_desc + static_cast<uint32_t>(st * (kStage >> 4));
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)   // 32 head dims of either part of q
            umma_e4m3(tS, kd + (kk & 3) * 2, q_desc + ((kk >> 2) * (N * 128) + (kk & 3) * 32) / 16, kIdescS, kk > 0 ? 1u : 0u);
          umma_commit(&bar_empty[st]);
          if (j == n_tiles - 1) {
            umma_commit(&bar_sfull[u & 1]);
            if (last) umma_commit(&bar_qempty);
          }
        }
        __syncwarp();
        if (++st == STAGES) st = 0;
      }
      if (!ok || final) break;
      st = (st + skip) % STAGES;
      skip = n_tiles;
    }
    if (elect_one()) umma_commit(&bar_done);
    __syncwarp();
  } else if (warp == F::kSecondWarp) {
    // =================================================================== second MMAs
    constexpr uint32_t kIdescO = idesc_format0_f32(128, F::kWeights, true, true);
    const uint64_t v_desc = smem_desc(smem_u32(sKV), kStage, 1024), p_desc = smem_desc_plain(smem_u32(sP), 128, kTile * 16);
    bool ok = wait_warp<true>(&bar_cfull[0], 0, &abort_flag);
    int st = 0, pcount = 0;
    uint32_t bits = 0;   // parities of the stages' next fills with V
    Chunk cur, nxt;
    if (ok) cur = s_chunk[0];
    if (ok && !cur.end) {
      st = cur.n_tiles % STAGES;   // behind K's tiles
      for (int u = 0; ok; ++u) {
        if (!cur.final) {
          const int rs = (u + 1) % kRing;
          if (!(ok = wait_warp<true>(&bar_cfull[rs], ((u + 1) / kRing) & 1, &abort_flag))) break;
          nxt = s_chunk[rs];
          st = (st + nxt.n_tiles) % STAGES;
        }
        for (int j = 0; j < cur.n_tiles; ++j) {
          if (!(ok = wait_warp<true>(&bar_vfull[st], (bits >> st) & 1, &abort_flag))) break;
          bits ^= 1u << st;
          const int valid = min(kTile, cur.t_end - (cur.t0 + j * kTile));
          if (valid % kPage != 0) {
            // slots behind the last token may hold anything (NaN); absent pages were read as zeros
            uint4* z = reinterpret_cast<uint4*>(sKV + st * kStage + valid * 128);
            for (int o = lane; o < (kPage - valid % kPage) * 8; o += 32) z[o] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
          const int pb = pcount & 1;
          if (!(ok = wait_warp<true>(&bar_pfull[pb], (pcount >> 1) & 1, &abort_flag))) break;
          tc_fence_after();
          const uint64_t vd = v_desc + static_cast<uint32_t>(st * (kStage >> 4));
          const uint64_t pd = p_desc + static_cast<uint32_t>(pb * (F::kWeightBuf >> 4));
          const int steps = (valid + 31) / 32;
          if (elect_one()) {
            // 32 tokens of both parts of w, each part into sums of its own: an MMA for either into the same sums, in a
            // loop of `steps`, took 450 cycles a tile where this takes 170 to 190
#pragma unroll
            for (int q = 0; q < kTile / 32; ++q)
              if (q < steps) umma_e4m3(tO, vd + q * 256, pd + q * 32, kIdescO, q == 0 && cur.first && j == 0 ? 0u : 1u);
            umma_commit(&bar_pempty[pb]);
            umma_commit(&bar_empty[st]);
            if (j == cur.n_tiles - 1) umma_commit(&bar_ofull[u & 1]);
          }
          __syncwarp();
          ++pcount;
          if (++st == STAGES) st = 0;
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(&bar_cempty[u % kRing]);
        if (cur.final) break;
        cur = nxt;
      }
    }
    if (elect_one()) umma_commit(&bar_done);
    __syncwarp();
  } else if (warp == F::kWalkWarp) {
    // =================================================================== the walk
    bool ok = true;
    int seq = 0;
    auto publish = [&](Chunk& c, const PageLoads<F::kChunkPages>& pages) {   // chunk number seq
      const int rs = seq % kRing;
      if (!(ok = wait_warp<true>(&bar_cempty[rs], ((seq / kRing) & 1) ^ 1, &abort_flag))) return;
      if (!c.end) pages.give(s_page[rs], s_scale[rs], lane);
      __syncwarp();
      if (lane == 0) {
        s_chunk[rs] = c;
        mbar_arrive(&bar_cfull[rs]);
      }
      ++seq;
    };
    publish(c, pages);
    if (!c.final && ok) {
      while (!d.final) {   // the next chunk's pages are asked for ahead of the wait for a place, its scales behind it
        walk.next(p, lane, c);
        pages.ask_pages(p, c, lane);
        publish(d, ahead);
        if (!ok) break;
        pages.ask_scales(p, c, lane);
        d = c;
        ahead = pages;
      }
      if (ok) publish(d, ahead);
    }
  } else {
    // =================================================================== softmax, epilogue
    // Set `set` of four warps computes rows c0 .. c0 + CW - 1 of every token; c0 and the sets' own barrier aside they
    // do the same.
    static_assert(CW * F::kSets == NC && (CW == 8 || CW == 16), "whole sets");
    const int q4 = warp & 3, set = (warp - 2) >> 2, c0 = set * CW, own = 1 + set;
    const int x = (q4 << 5) | lane;   // tensor-memory lane: token of a tile, or head dim
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t tOx = tO + lane_off + static_cast<uint32_t>(c0);
    float2 l[CW / 2];
    int pcount = 0, n_list = -1;
    // The set meets at named barriers, which have no limit of their own.  So no warp leaves alone: one whose wait gives up
    // goes on with what there is (the call fails, its results are void), and all leave where one has no chunk.
    for (int u = 0;; ++u) {
      const int rs = u % kRing;
      const bool got = wait_warp<true>(&bar_cfull[rs], (u / kRing) & 1, &abort_flag);
      Chunk c = s_chunk[rs];
      if (!got || c.end) {
        c.n_tiles = c.first = 0;
        s_leave[set][u & 1] = 1;
      }
      if (c.first) {
        ++n_list;
#pragma unroll
        for (int n = 0; n < CW / 2; ++n) l[n] = make_float2(0.f, 0.f);
      }
      const uint32_t tS = tmem + lane_off + static_cast<uint32_t>((u & 1) * kChunk * N + c0);
      if (c.n_tiles > 0) wait_warp<true>(&bar_sfull[u & 1], (u >> 1) & 1, &abort_flag);
      tc_fence_after();
      float2 q_scale[CW / 2];   // of two rows each
#pragma unroll
      for (int n = 0; n < CW / 2; ++n) q_scale[n] = reinterpret_cast<const float2*>(s_qscale[n_list & 3] + c0)[n];
      // the exact maxima of x over the chunk (behind the last token scores may be anything: -inf)
      const int last_tile = (c.t_end - c.t0 - 1) / kTile;
      const bool cut = c.t_end - c.t0 - last_tile * kTile <= x;   // this thread's token of it is past the end
      auto load = [&](int j, uint32_t (&r)[CW]) {
        if constexpr (CW == 8)
          tmem_ld8(tS + j * N, r);
        else
          tmem_ld16(tS + j * N, r);
      };
      auto ready = [&](int j, uint32_t (&r)[CW]) {
        tmem_wait_ld();
        tmem_regs_ready(r);
        if (j == last_tile && cut) {
#pragma unroll
          for (int n = 0; n < CW; ++n) r[n] = 0xFF800000u;
        }
      };
      {
        float mx[CW];
#pragma unroll
        for (int n = 0; n < CW; ++n) mx[n] = -CUDART_INF_F;
#pragma unroll 1
        for (int j = 0; j < c.n_tiles; ++j) {
          uint32_t r[CW];
          load(j, r);
          const float2 sc = s_scale[rs][j * kTilePages + (x >> 4)];
          ready(j, r);
#pragma unroll
          for (int n = 0; n < CW; n += 2) {
            const float2 a = __fmul2_rn(q_scale[n / 2], make_float2(sc.x, sc.x));
            const float2 y = __ffma2_rn(make_float2(__uint_as_float(r[n]), __uint_as_float(r[n + 1])), a, make_float2(sc.y, sc.y));
            mx[n] = fmaxf(mx[n], y.x);
            mx[n + 1] = fmaxf(mx[n + 1], y.y);
          }
        }
#pragma unroll
        for (int n = 0; n < CW; ++n) mx[n] = warp_max(mx[n]);
        if (lane == 0) {
#pragma unroll
          for (int n = 0; n < CW; n += 4)
            *reinterpret_cast<float4*>(&s_red[q4][c0 + n]) = make_float4(mx[n], mx[n + 1], mx[n + 2], mx[n + 3]);
        }
      }
      named_barrier(own, 128);
      if (x == 0) s_leave[set][(u + 1) & 1] = 0;   // every reader of that slot is past this barrier
      if (x < CW) {
        const int n = c0 + x;
        const float mc = fmaxf(fmaxf(s_red[0][n], s_red[1][n]), fmaxf(s_red[2][n], s_red[3][n]));
        const float top = c.first ? mc : fmaxf(mc, s_top[n]), m = fmaxf(mc, top - kReach);   // top: of the list so far
        s_alpha[n] = ex2(s_m[n] - m);   // (not used of a first chunk)
        s_top[n] = top;
        s_m[n] = m;
      }
      named_barrier(own, 128);
      if (s_leave[set][u & 1]) break;
      if (!c.first) {
        // these rows of O^T and l from the last chunk's power of two to this one's
        wait_warp<true>(&bar_ofull[(u - 1) & 1], ((u - 1) >> 1) & 1, &abort_flag);
        tc_fence_after();
#pragma unroll 1
        for (uint32_t col = 0; col < F::kWeights; col += NC < 16 ? 16 : N) {   // (eight rows: both parts at once)
          uint32_t r[16];
          tmem_ld16(tOx + col, r);
          tmem_wait_ld();
          tmem_regs_ready(r);
#pragma unroll
          for (int n = 0; n < 16; ++n) r[n] = __float_as_uint(__uint_as_float(r[n]) * s_alpha[c0 + n % CW]);
          tmem_st16(tOx + col, r);
        }
        tmem_wait_st();
        tc_fence_before();
#pragma unroll
        for (int n = 0; n < CW / 2; ++n) l[n] = __fmul2_rn(l[n], make_float2(s_alpha[c0 + 2 * n], s_alpha[c0 + 2 * n + 1]));
      }
      // The weights, tile by tile, into shared memory.  2^(c sK q . k - m + 8) is what l adds up; times sV it is w, whose
      // float16 (finer than both parts, and exact to subtract from) is split.  (PV of the chunk's first tile waits for the
      // weights, and so for O's new maxima.)
      {
        float2 mr[CW / 2];
#pragma unroll
        for (int n = 0; n < CW / 2; ++n) mr[n] = make_float2(kWeightExp - s_m[c0 + 2 * n], kWeightExp - s_m[c0 + 2 * n + 1]);
        uint32_t r[CW];
        load(0, r);
        for (int j = 0; j < c.n_tiles; ++j) {
          const float2 sc = s_scale[rs][j * kTilePages + (x >> 4)];
          const float sv = ex2(sc.y);
          ready(j, r);
          uint32_t w[CW / 2];   // float16 pairs
#pragma unroll
          for (int n = 0; n < CW / 2; ++n) {
            const float2 a = __fmul2_rn(q_scale[n], make_float2(sc.x, sc.x));
            const float2 y = __ffma2_rn(make_float2(__uint_as_float(r[2 * n]), __uint_as_float(r[2 * n + 1])), a, mr[n]);
            const float2 e = make_float2(ex2(y.x), ex2(y.y));
            l[n] = __fadd2_rn(l[n], e);
            const float2 z = __fmul2_rn(e, make_float2(sv, sv));
            w[n] = half2_bits(z.x, z.y);
          }
          if (j + 1 < c.n_tiles) load(j + 1, r);
          uint32_t hi[CW / 4], lo[CW / 4];
#pragma unroll
          for (int n = 0; n < CW / 4; ++n) {
            uint32_t h[2], o[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) split_half2(w[2 * n + k], h[k], o[k]);
            hi[n] = h[0] | h[1] << 16;
            lo[n] = o[0] | o[1] << 16;
          }
          const int pb = pcount & 1;
          wait_warp<true>(&bar_pempty[pb], ((pcount >> 1) & 1) ^ 1, &abort_flag);
          uint8_t* to = sP + pb * F::kWeightBuf + set * (kTile * 16) + x * 16;
          if constexpr (CW == 8) {
            *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
          } else {
            *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[CW / 4 - 2], hi[CW / 4 - 1]);
            *reinterpret_cast<uint4*>(to + N * kTile) = make_uint4(lo[0], lo[1], lo[CW / 4 - 2], lo[CW / 4 - 1]);
          }
          fence_proxy_async_smem();
          tc_fence_before();
          mbar_arrive(&bar_pfull[pb]);
          ++pcount;
        }
      }
      tc_fence_before();
      mbar_arrive(&bar_sfree[u & 1]);
      if (c.last) {
        // The code from here on is met once a list, each time from memory: loops, not their bodies in a row.
        wait_warp<true>(&bar_ofull[u & 1], (u >> 1) & 1, &abort_flag);
        tc_fence_after();
        // the rows' sums, through the set's own pieces of the weights' buffers (no MMA reads them now): four rows a piece
        auto sums = [&](int n) { return reinterpret_cast<float*>(sP) + ((n >> 2) * F::kSets + set) * (4 * kTile) + (n & 3) * kTile; };
#pragma unroll
        for (int n = 0; n < CW / 2; ++n) {
          sums(2 * n)[x] = l[n].x;
          sums(2 * n + 1)[x] = l[n].y;
        }
        named_barrier(own, 128);
        {
          constexpr int kEach = 128 / CW;   // threads of a row
          float v = 0.f;
#pragma unroll 4
          for (int i = x % kEach; i < kTile; i += kEach) v += sums(x / kEach)[i];
#pragma unroll
          for (int off = kEach / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
          if (x % kEach == 0) s_l[c0 + x / kEach] = c.slot < 0 ? 1.f / v : v;
        }
        named_barrier(own, 128);   // before the set's next weights
        const int first = c.rg * p.lsub + c0 / p.G;   // block position and head of row c0
        const int live = max(0, min(min(p.rows, (p.L - c.rg * p.lsub) * p.G) - c0, CW));   // rows of the set that there are
        const size_t row0 = (static_cast<size_t>(c.b) * p.L + first) * p.Hq + static_cast<size_t>(c.kvh) * p.G + c0 % p.G;
        float* mine = p.part + static_cast<size_t>(c.slot < 0 ? 0 : c.slot) * N * kPartRow + c0 * 128;
        const uint64_t keep = l2_policy_evict_last();   // read back soon
        int g = c0 % p.G;
        size_t row = row0;
#pragma unroll 1
        for (int n0 = 0; n0 < live; n0 += 4) {
          uint32_t r[4], r2[4];
          tmem_ld4(tOx + n0, r);
          tmem_ld4(tOx + NC + n0, r2);   // the lower part's
          tmem_wait_ld();
          tmem_regs_ready(r);
          tmem_regs_ready(r2);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (n0 + k >= live) break;
            const float o = fmaf(__uint_as_float(r2[k]), 1.f / kLowPart, __uint_as_float(r[k]));
            if (c.slot < 0)
              p.out[row * 128 + x] = __bfloat16_as_ushort(__float2bfloat16_rn(o * s_l[c0 + n0 + k]));
            else
              st_global_hint(mine + (n0 + k) * 128 + x, o, keep);
            ++row;
            if (++g == p.G) {
              g = 0;
              row += p.Hq - p.G;
            }
          }
        }
        if (c.slot >= 0) {
          float* ml = p.part + static_cast<size_t>(c.slot) * N * kPartRow + N * 128 + c0;
          if (x < CW) {
            st_global_hint(ml + x, s_m[c0 + x], keep);
            st_global_hint(ml + N + x, s_l[c0 + x], keep);
          }
          if (p.join_here) {
            __threadfence();
            named_barrier(own, 128);
            if (x == 0) s_join[set] = atomicAdd(p.work + 1 + c.u0 * F::kSets + set, 1) == c.parts - 1;
            named_barrier(own, 128);
            if (s_join[set]) {
              __threadfence();
              join_parts<N, CW>(p, c, x, c0, row0, c0 % p.G, live, s_l + c0, s_alpha + c0, s_red[0] + c0, s_red[1] + c0, own);
            }
          }
        }
        tc_fence_before();
      }
      // the chunk's descriptor and scales (and O^T) are done with
      named_barrier(own, 128);
      if (x == 0) mbar_arrive(&bar_cempty[rs]);
      if (c.final) break;
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
  if (p.join_here && warp == 0) {
    // the last CTA to end leaves the counters as it found them
    int last = 0;
    if (lane == 0) {
      __threadfence();
      last = atomicAdd(p.work, 1) == static_cast<int>(gridDim.x) - 1;
    }
    if (__shfl_sync(0xffffffffu, last, 0))
      for (int u = lane; u <= static_cast<int>(gridDim.x) * F::kSets; u += 32) p.work[u] = 0;
  }
  if (threadIdx.x == 0 && abort_flag) atomicOr(p.err, BDLM_DEVERR_TIMEOUT);
}

// ------------------------------------------------------------------ more query rows per KV head
//
// S = Q K^T and O += W V with 128 query rows on M, a row a tensor-memory lane, up to two groups of 128
// that share every tile.  Here two parts of w would cost the softmax more than all else it does (three
// instructions a weight), so V is widened instead, once for all rows: converter warps turn a tile's codes
// into float16 (exactly) in shared memory, w is one float16 (written over S, the A operand in tensor
// memory) and the second product is kind::f16.  The first takes K's codes as they are and Q's two parts,
// which a small kernel makes beforehand.  Softmax: two threads a row, 64 tokens each; a page's scales are
// the same for 16 of them, so the maximum is taken of raw scores page by page.
//
// Bound, with 256 rows: a group's softmax (about 2000 cycles a tile) and its MMAs (1000 alone, 1400 beside the
// converters' and copies' use of shared memory) follow one another, and the two groups' overlap only in part; without the
// exponentials it takes as long.  197 us for 16 blocks of 64 over 8192-16384 tokens, of which the joins take about 10 and
// the queries' parts 5; bf16's block attention takes 237 for twice the bytes.
template <int SUB>
struct Many {
  static constexpr int kRowsItem = 128 * SUB;
  static constexpr int kStagesK = SUB == 2 ? 3 : 4, kStagesV = SUB == 2 ? 2 : 3;
  static constexpr int kSoftmaxWarps = 8 * SUB;
  static constexpr int kConvWarps = SUB == 2 ? 2 : 4;
  static constexpr int kSoftmax0 = 2 + kConvWarps;      // first softmax warp
  static constexpr int kThreads = 32 * (kSoftmax0 + kSoftmaxWarps);
  static constexpr int kChunk = 8;                      // tiles of a descriptor
  static constexpr int kWide = 2 * kStage;              // a tile's V in float16
  static constexpr size_t kSmem = 1024 + kRowsItem * 256 + (kStagesK + kStagesV) * kStage + 2 * kWide;
};

__device__ __forceinline__ uint32_t widen2(uint32_t two_codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two_codes), __NV_E4M3);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float max16(const uint32_t* r) {
  float v[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(r[k]);
  const float a = fmax3(v[0], v[1], v[2]), b = fmax3(v[3], v[4], v[5]), c = fmax3(v[6], v[7], v[8]);
  const float d = fmax3(v[9], v[10], v[11]), e = fmax3(v[12], v[13], v[14]);
  return fmax3(fmax3(a, b, c), fmaxf(d, e), v[15]);
}

// store_rows_128b with a staging buffer of 512 bytes, 4 rows at a time: 128 bytes per lane (w) to dst, or nowhere.
__device__ __forceinline__ void store_rows(const uint32_t (&w)[32], void* dst, uint8_t* stage, int lane) {
  const unsigned long long dptr = reinterpret_cast<unsigned long long>(dst);
#pragma unroll
  for (int p4 = 0; p4 < 8; ++p4) {
    if ((lane >> 2) == p4) {
      const int r = lane & 3;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(stage + r * 128 + ((c ^ r) << 4)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    }
    __syncwarp();
    const int r = lane >> 3, c = lane & 7;
    const unsigned long long d = __shfl_sync(0xffffffffu, dptr, p4 * 4 + r);
    const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + ((c ^ r) << 4));
    if (d) reinterpret_cast<uint4*>(d)[c] = v;
    __syncwarp();
  }
}

template <int SUB>
__global__ void __launch_bounds__(Many<SUB>::kThreads, 1)
many_rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using F = Many<SUB>;
  constexpr int KS = F::kStagesK, VS = F::kStagesV, kRowsItem = F::kRowsItem, kChunk = F::kChunk;
  constexpr int kChunkPages = kChunk * kTilePages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = base;                       // two parts x kRowsItem rows x 128 bytes
  uint8_t* sK = sQ + kRowsItem * 256;
  uint8_t* sV = sK + KS * kStage;
  uint8_t* sW = sV + VS * kStage;       // two buffers of V in float16: two halves of 64 dims x 128 tokens
  __shared__ uint64_t bar_qfull, bar_qempty, bar_kfull[KS], bar_kempty[KS], bar_vfull[VS], bar_vempty[VS];
  __shared__ uint64_t bar_wfull[2], bar_wempty[2], bar_sfull[2], bar_pfull[2], bar_ofull[2], bar_done;
  __shared__ uint64_t bar_cfull[kRing], bar_cempty[kRing], bar_pair[4 * SUB][2], bar_pair_end[4 * SUB];
  __shared__ Chunk s_chunk[kRing];
  __shared__ float2 s_scale[kRing][kChunkPages];
  __shared__ int s_page[3][kChunkPages];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ __align__(16) uint8_t s_stage[F::kSoftmaxWarps][512];
  __shared__ float s_hmax[2][SUB][2][128], s_hsum[SUB][2][128];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&bar_qfull, 1);
    mbar_init(&bar_qempty, 1);
    for (int s = 0; s < KS; ++s) {
      mbar_init(&bar_kfull[s], 1);
      mbar_init(&bar_kempty[s], 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(&bar_vfull[s], 1);
      mbar_init(&bar_vempty[s], F::kConvWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_wfull[i], F::kConvWarps);
      mbar_init(&bar_wempty[i], 1);
      mbar_init(&bar_sfull[i], 1);
      mbar_init(&bar_pfull[i], 256);
      mbar_init(&bar_ofull[i], 1);
    }
    mbar_init(&bar_done, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bar_cfull[i], 1);
      mbar_init(&bar_cempty[i], 1 + F::kConvWarps + F::kSoftmaxWarps);
    }
    for (int i = 0; i < 4 * SUB; ++i) {
      mbar_init(&bar_pair[i][0], 64);
      mbar_init(&bar_pair[i][1], 64);
      mbar_init(&bar_pair_end[i], 64);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  // rows that no query fills read as zeros
  for (int o = threadIdx.x * 16; o < (kRowsItem - p.rows) * 128; o += F::kThreads * 16) {
    *reinterpret_cast<uint4*>(sQ + p.rows * 128 + o) = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(sQ + kRowsItem * 128 + p.rows * 128 + o) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const uint32_t tO = tmem + 256;   // S: two buffers, or one of each group

  if (warp == 0) {
    // =================================================================== producer
    // All but the queries' parts and their scale can be read before the kernel that makes them is done: its CTAs let this
    // one start after they waited for what wrote the rest.  All else here waits for the first chunk.
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const uint64_t policy = l2_policy_evict_first();
    int kst = 0, vst = 0, q_loads = 0, seq = -1;
    uint32_t kph = 0, vph = 0;
    bool ok = true;
    Walk<kChunk> walk;
    walk.init(p, lane);
    PageLoads<kChunkPages> pages;
    auto look_up = [&](Chunk& c) -> bool {
      const bool have = walk.next(p, lane, c);
      if (have) {
        pages.ask_pages(p, c, lane);
        pages.ask_scales(p, c, lane);
      }
      return have;
    };
    auto publish = [&](Chunk& c, bool have) {
      ++seq;
      const int rs = seq % kRing;
      if (!have) c.end = 1;
      if (ok) ok = wait_warp<SUB == 1>(&bar_cempty[rs], ((seq / kRing) & 1) ^ 1, &abort_flag);
      if (have) pages.give(s_page[seq % 3], s_scale[rs], lane);
      __syncwarp();
      if (lane == 0) {
        s_chunk[rs] = c;
        mbar_arrive(&bar_cfull[rs]);
      }
    };
    auto prepare = [&](Chunk& c) -> bool {
      const bool have = look_up(c);
      publish(c, have);
      return have;
    };
    auto load_q = [&](const Chunk& c) {
      if (lane == 0) {
        if (ok) ok = mbar_wait(&bar_qempty, (q_loads & 1) ^ 1, &abort_flag);
        if (ok) {
          mbar_arrive_expect_tx(&bar_qfull, 256u * static_cast<uint32_t>(p.rows));
          for (int h = 0; h < 2; ++h)
            tma_load_3d(sQ + h * kRowsItem * 128, &tm_q, &bar_qfull, h * 128, c.kvh * p.G, c.b * p.L + c.rg * p.lsub);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      ++q_loads;
    };
    auto copy = [&](const CUtensorMap* tm, uint8_t* ring, uint64_t* full, uint64_t* empty, int stages, int& st, uint32_t& ph, int page) {
      if (lane == 0) {
        ok = mbar_wait(&empty[st], ph ^ 1, &abort_flag);
        if (ok) mbar_arrive_expect_tx(&full[st], kStage);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) return;
      if (lane < kTilePages) tma_load_3d_hint(ring + st * kStage + lane * 2048, tm, &full[st], 0, 0, page, policy);
      if (++st == stages) {
        st = 0;
        ph ^= 1;
      }
    };
    Chunk cur, nxt;
    bool have = look_up(cur), have_next = false;
    int cs = 0;
    if (have) copy(&tm_k, sK, bar_kfull, bar_kempty, KS, kst, kph, pages.unit[0]);   // (lane l: page l)
    griddep_wait();
    publish(cur, have);
    if (have) {
      load_q(cur);
      have_next = prepare(nxt);
    }
    while (have && ok) {
      for (int j = 0; j < cur.n_tiles && ok; ++j) {
        // K of the next tile, then V of this one
        if (j + 1 < cur.n_tiles) {
          copy(&tm_k, sK, bar_kfull, bar_kempty, KS, kst, kph, s_page[cs % 3][(j + 1) * kTilePages + (lane & 7)]);
        } else if (have_next) {
          if (nxt.first) load_q(nxt);
          if (ok) copy(&tm_k, sK, bar_kfull, bar_kempty, KS, kst, kph, s_page[(cs + 1) % 3][lane & 7]);
        }
        if (ok) copy(&tm_v, sV, bar_vfull, bar_vempty, VS, vst, vph, s_page[cs % 3][j * kTilePages + (lane & 7)]);
      }
      cur = nxt;
      have = have_next;
      ++cs;
      if (have && ok) have_next = prepare(nxt);
    }
    if (lane == 0) {
      griddep_launch_dependents();
      if (!ok) {
        for (int s = 0; s < KS; ++s) mbar_wait_drain(&bar_kfull[s], kph ^ (s < kst ? 0 : 1));
        for (int s = 0; s < VS; ++s) mbar_wait_drain(&bar_vfull[s], vph ^ (s < vst ? 0 : 1));
        if (q_loads > 0) mbar_wait_drain(&bar_qfull, (q_loads - 1) & 1);
      }
    }
  } else if (warp == 1) {
    // =================================================================== MMA issuer
    {
      constexpr uint32_t kIdescS = idesc_format0_f32(128, 128, false, false);
      constexpr uint32_t kIdescO = idesc_format0_f32(128, 128, false, true);
      const uint64_t q_desc = smem_desc(smem_u32(sQ), 16, 1024), k_desc = smem_desc(smem_u32(sK), 16, 1024);
      const uint64_t w_desc = smem_desc(smem_u32(sW), kStage, 1024);
      bool ok = true;
      int kst = 0, q_used = 0;
      uint32_t kph = 0;
      // S of tile number u, of group x
      auto issue_s = [&](int u, int x) {
        const uint32_t tS = tmem + static_cast<uint32_t>((SUB == 2 ? x : u & 1) * 128);
        const uint64_t kd = k_desc + static_cast<uint32_t>(kst * (kStage >> 4)), qd = q_desc + static_cast<uint32_t>(x * 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_e4m3(tS, qd + ((kk >> 2) * (kRowsItem * 128) + (kk & 3) * 32) / 16, kd + (kk & 3) * 2, kIdescS, kk > 0 ? 1u : 0u);
          umma_commit(&bar_sfull[SUB == 2 ? x : u & 1]);
        }
        __syncwarp();
      };
      auto wait_k = [&](bool first) {
        if (first) {
          if (!(ok = wait_warp<SUB == 1>(&bar_qfull, q_used & 1, &abort_flag))) return;
          ++q_used;
        }
        if (!(ok = wait_warp<SUB == 1>(&bar_kfull[kst], kph, &abort_flag))) return;
        tc_fence_after();
      };
      auto free_k = [&](bool last) {
        if (elect_one()) {
          umma_commit(&bar_kempty[kst]);
          if (last) umma_commit(&bar_qempty);
        }
        __syncwarp();
        if (++kst == KS) {
          kst = 0;
          kph ^= 1;
        }
      };
      auto issue_pv = [&](int u, int x, bool first, int valid) {
        const uint64_t wd = w_desc + static_cast<uint32_t>((u & 1) * (F::kWide >> 4));
        const uint32_t tP = tmem + static_cast<uint32_t>((SUB == 2 ? x : u & 1) * 128);
        const int steps = (valid + 15) / 16;
        if (elect_one()) {
#pragma unroll
          for (int q = 0; q < kTile / 16; ++q)   // keys 64h .. 64h + 63 of w as columns 64h .. 64h + 31
            if (q < steps)
              umma_bf16_ts(tO + static_cast<uint32_t>(x * 128), tP + static_cast<uint32_t>((q >> 2) * 64 + (q & 3) * 8),
                           wd + q * 128, kIdescO, first && q == 0 ? 0u : 1u);
          if (x == SUB - 1) {
            umma_commit(&bar_wempty[u & 1]);
            umma_commit(&bar_ofull[u & 1]);
          }
        }
        __syncwarp();
      };
      auto wait_p = [&](int u, int x) {
        ok = SUB == 2 ? wait_warp<SUB == 1>(&bar_pfull[x], u & 1, &abort_flag)
                      : wait_warp<SUB == 1>(&bar_pfull[u & 1], (u >> 1) & 1, &abort_flag);
        tc_fence_after();
      };
      Chunk cur, nxt;
      ok = wait_warp<SUB == 1>(&bar_cfull[0], 0, &abort_flag);
      cur = s_chunk[0];
      if (ok && !cur.end) {
        wait_k(true);
        if (ok) {
          for (int x = 0; x < SUB; ++x) issue_s(0, x);
          free_k(cur.last && cur.n_tiles == 1);
        }
        int cs = 0;
        for (int u = 0, j = 0; ok; ++u) {
          bool has_next = true, next_first = false, next_last;
          const bool whole = j + 1 == cur.n_tiles;   // of its descriptor
          if (!whole) {
            next_last = cur.last && j + 2 == cur.n_tiles;
          } else {
            const int rs = (cs + 1) % kRing;
            if (!(ok = wait_warp<SUB == 1>(&bar_cfull[rs], ((cs + 1) / kRing) & 1, &abort_flag))) break;
            nxt = s_chunk[rs];
            has_next = !nxt.end;
            next_first = nxt.first;
            next_last = nxt.last && nxt.n_tiles == 1;
          }
          const bool first = cur.first && j == 0;
          const int valid = min(kTile, cur.t_end - (cur.t0 + j * kTile));
          if (SUB == 1) {
            if (has_next) {   // S(u + 1) ahead of PV(u): the softmax goes on meanwhile
              wait_k(next_first);
              if (!ok) break;
              issue_s(u + 1, 0);
              free_k(next_last);
            }
            if (!(ok = wait_warp<SUB == 1>(&bar_wfull[u & 1], (u >> 1) & 1, &abort_flag))) break;
            wait_p(u, 0);
            if (!ok) break;
            issue_pv(u, 0, first, valid);
          } else {
            // PV_0(u), S_0(u + 1), PV_1(u), S_1(u + 1): S_x(u + 1) overwrites the weights that PV_x(u) reads, and
            // the tensor pipe executes one thread's MMAs in order.  Where the next tile has other queries
            // both PVs come first.
            if (!(ok = wait_warp<SUB == 1>(&bar_wfull[u & 1], (u >> 1) & 1, &abort_flag))) break;
            const bool inter = has_next && !next_first;
            for (int x = 0; x < 2 && ok; ++x) {
              wait_p(u, x);
              if (!ok) break;
              issue_pv(u, x, first, valid);
              if (!inter) continue;
              if (x == 0) wait_k(false);
              if (ok) issue_s(u + 1, x);
            }
            if (!ok) break;
            if (has_next && !inter) {
              wait_k(true);
              if (!ok) break;
              issue_s(u + 1, 0);
              issue_s(u + 1, 1);
            }
            if (has_next) free_k(next_last);
          }
          if (whole) {
            if (lane == 0) mbar_arrive(&bar_cempty[cs % kRing]);
            if (!has_next) break;
            cur = nxt;
            j = 0;
            ++cs;
          } else {
            ++j;
          }
        }
      }
      if (elect_one()) umma_commit(&bar_done);
      __syncwarp();
    }
  } else if (warp < 2 + F::kConvWarps) {
    // =================================================================== converters
    // Lane l takes 16 dims (chunk l % 8) of tokens l / 8 + 4k: 16 bytes in, twice 16 out.  Lanes of the two
    // halves write their two pieces in opposite order, so eight lanes' stores meet no bank twice.
    const int w = warp - 2, c8 = lane & 7;
    bool ok = true;
    int vst = 0, u = 0;
    uint32_t vph = 0;
    for (int cs = 0; ok; ++cs) {
      const int rs = cs % kRing;
      if (!(ok = wait_warp<SUB == 1>(&bar_cfull[rs], (cs / kRing) & 1, &abort_flag))) break;
      const Chunk c = s_chunk[rs];
      if (c.end) break;
      for (int j = 0; j < c.n_tiles; ++j, ++u) {
        const int valid = min(kTile, c.t_end - (c.t0 + j * kTile));
        if (!(ok = wait_warp<SUB == 1>(&bar_wempty[u & 1], ((u >> 1) & 1) ^ 1, &abort_flag))) break;
        if (!(ok = wait_warp<SUB == 1>(&bar_vfull[vst], vph, &abort_flag))) break;
        const uint8_t* src = sV + vst * kStage;
        uint8_t* dst = sW + (u & 1) * F::kWide + (c8 >> 2) * kStage;
        constexpr int kEach = kTile / 4 / F::kConvWarps;   // tokens of a lane
#pragma unroll(SUB == 1 ? 2 : 1)
        for (int k0 = 0; k0 < kEach; k0 += 4) {
          uint4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int t = w * (kTile / F::kConvWarps) + (k0 + k) * 4 + (lane >> 3);
            v[k] = *reinterpret_cast<const uint4*>(src + t * 128 + ((c8 ^ (t & 7)) << 4));
            if (t >= valid) v[k] = make_uint4(0, 0, 0, 0);   // slots behind the last token may hold anything
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int t = w * (kTile / F::kConvWarps) + (k0 + k) * 4 + (lane >> 3);
            const uint4 a = make_uint4(widen2(v[k].x & 0xFFFFu), widen2(v[k].x >> 16), widen2(v[k].y & 0xFFFFu), widen2(v[k].y >> 16));
            const uint4 b = make_uint4(widen2(v[k].z & 0xFFFFu), widen2(v[k].z >> 16), widen2(v[k].w & 0xFFFFu), widen2(v[k].w >> 16));
            const int first = c8 >> 2, at = (c8 & 3) * 2;
            *reinterpret_cast<uint4*>(dst + t * 128 + (((at + first) ^ (t & 7)) << 4)) = first ? b : a;
            *reinterpret_cast<uint4*>(dst + t * 128 + (((at + 1 - first) ^ (t & 7)) << 4)) = first ? a : b;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar_vempty[vst]);
          mbar_arrive(&bar_wfull[u & 1]);
        }
        if (++vst == VS) {
          vst = 0;
          vph ^= 1;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_cempty[rs]);
    }
  } else if (warp >= F::kSoftmax0) {
    // =================================================================== softmax, epilogue
    const int x = (warp - F::kSoftmax0) >> 3;
    const int half = ((warp - F::kSoftmax0) >> 2) & 1;
    const int q4 = warp & 3;
    const int n = (q4 << 5) | lane;
    const int pq = x * 4 + q4;   // the two halves' exchange barriers
    const int r_item = x * 128 + n;
    const int r_off = r_item / p.G * p.Hq + r_item % p.G;   // from the group's first row of q and the output
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t col0 = static_cast<uint32_t>(half * 64);
    const uint32_t tOx = tO + lane_off + static_cast<uint32_t>(x * 128) + col0;
    bool ok = true;
    int u = 0, pair_ends = 0;
    float m_run = -CUDART_INF_F, l_run = 0.f;   // kWeightExpMany below a running maximum; this half's sum
    for (int cs = 0; ok; ++cs) {
      const int rs = cs % kRing;
      if (!(ok = wait_warp<SUB == 1>(&bar_cfull[rs], (cs / kRing) & 1, &abort_flag))) break;
      const Chunk& at = s_chunk[rs];   // (what every tile needs is read once; a copy of all would take registers)
      const int n_tiles = at.n_tiles, t0 = at.t0, t_end = at.t_end;
      if (at.end) break;
      if (at.first) {
        m_run = -CUDART_INF_F;
        l_run = 0.f;
      }
      const size_t row0 = (static_cast<size_t>(at.b) * p.L + at.rg * p.lsub) * p.Hq + static_cast<size_t>(at.kvh) * p.G;
      const bool live = r_item < min(p.rows, (p.L - at.rg * p.lsub) * p.G);
      const float q_scale = q_factor(__ldcg(p.q_scale + row0 + (live ? r_off : 0)), p.scale_log2);   // q = (hi + lo) * q_scale, times c
      for (int j = 0; j < n_tiles; ++j, ++u) {
        const uint32_t tSx = tmem + lane_off + static_cast<uint32_t>((SUB == 2 ? x : u & 1) * 128) + col0;
        ok = SUB == 2 ? wait_warp<SUB == 1>(&bar_sfull[x], u & 1, &abort_flag)
                      : wait_warp<SUB == 1>(&bar_sfull[u & 1], (u >> 1) & 1, &abort_flag);
        if (!ok) break;
        tc_fence_after();
        const int nvalid = min(kTile, t_end - (t0 + j * kTile)) - half * 64;   // of this half's columns
        const float2* scales = &s_scale[rs][j * kTilePages + half * 4];
        if (nvalid < 64) {   // scores behind the last token may be anything: -inf
#pragma unroll 1
          for (int col = max(nvalid, 0); col < 64; ++col) tmem_st1(tSx + col, 0xFF800000u);
          tmem_wait_st();
        }
        // (Code that runs once a list, or seldom, is in rolled loops here, and so are the converters' of 256 rows: with all
        // of it unrolled the warps waited for instructions twice as long as they issued them.  Unrolling these two halves
        // of a tile, which every tile meets, was worth 210 -> 203 us for 16 blocks of 64 over 8192-16384 tokens.)
        float mx = -CUDART_INF_F;
#pragma unroll
        for (int g2 = 0; g2 < 2; ++g2) {
          uint32_t r[32];
          tmem_ld16(tSx + g2 * 32, *reinterpret_cast<uint32_t(*)[16]>(r));
          tmem_ld16(tSx + g2 * 32 + 16, *reinterpret_cast<uint32_t(*)[16]>(r + 16));
          const float2 s0 = scales[2 * g2], s1 = scales[2 * g2 + 1];
          tmem_wait_ld();
          tmem_regs_ready(*reinterpret_cast<uint32_t(*)[16]>(r));
          tmem_regs_ready(*reinterpret_cast<uint32_t(*)[16]>(r + 16));
          mx = fmax3(mx, fmaf(max16(r), s0.x * q_scale, s0.y), fmaf(max16(r + 16), s1.x * q_scale, s1.y));
        }
        s_hmax[u & 1][x][half][n] = mx;
        mbar_arrive(&bar_pair[pq][u & 1]);
        if (!(ok = wait_warp<SUB == 1>(&bar_pair[pq][u & 1], (u >> 1) & 1, &abort_flag))) break;
        mx = fmaxf(s_hmax[u & 1][x][0][n], s_hmax[u & 1][x][1][n]);
        float alpha = 1.f;
        bool resc = false;
        mx -= kWeightExpMany;
        if (m_run == -CUDART_INF_F) {
          m_run = mx;
        } else if (mx - m_run > kLazyMany) {
          alpha = ex2(m_run - mx);
          m_run = mx;
          resc = true;
        }
        float sum = 0.f;
#pragma unroll
        for (int g2 = 0; g2 < 2; ++g2) {
          uint32_t r[32];
          tmem_ld16(tSx + g2 * 32, *reinterpret_cast<uint32_t(*)[16]>(r));
          tmem_ld16(tSx + g2 * 32 + 16, *reinterpret_cast<uint32_t(*)[16]>(r + 16));
          tmem_wait_ld();
          tmem_regs_ready(*reinterpret_cast<uint32_t(*)[16]>(r));
          tmem_regs_ready(*reinterpret_cast<uint32_t(*)[16]>(r + 16));
          uint32_t pk[16];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float2 s = scales[2 * g2 + g];
            const float a = s.x * q_scale, b = s.y - m_run;
            const float2 a2 = make_float2(a, a), b2 = make_float2(b, b);
            float2 t2 = make_float2(0.f, 0.f);   // (a tree's partial sums would be spilled)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int at = g * 16 + 2 * k;
              const float2 y = __ffma2_rn(make_float2(__uint_as_float(r[at]), __uint_as_float(r[at + 1])), a2, b2);
              const float2 e = make_float2(ex2(y.x), ex2(y.y));
              pk[g * 8 + k] = half2_bits(e.x, e.y);
              t2 = __fadd2_rn(t2, e);
            }
            sum = fmaf(t2.x + t2.y, ex2(-s.y), sum);
          }
          tmem_st16(tSx + g2 * 16, pk);   // tokens 64h + 32 g2 .. + 31 as 16 columns
        }
        l_run = fmaf(l_run, alpha, sum);
        if (__any_sync(0xffffffffu, resc)) {
          // this warp's half of its rows of O to the new maxima once the last tile's PV is done
          if (!(ok = wait_warp<SUB == 1>(&bar_ofull[(u - 1) & 1], ((u - 1) >> 1) & 1, &abort_flag))) break;
          tc_fence_after();
#pragma unroll 1
          for (int g = 0; g < 4; ++g) {
            uint32_t o[16];
            tmem_ld16(tOx + g * 16, o);
            tmem_wait_ld();
            tmem_regs_ready(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st16(tOx + g * 16, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar_pfull[SUB == 2 ? x : u & 1]);
        if (!at.last || j != n_tiles - 1) continue;
        // ---- this half of the row of O, divided by the row's sum or as a part
        if (!(ok = wait_warp<SUB == 1>(&bar_ofull[u & 1], (u >> 1) & 1, &abort_flag))) break;
        tc_fence_after();
        s_hsum[x][half][n] = l_run;
        mbar_arrive(&bar_pair_end[pq]);
        if (!(ok = wait_warp<SUB == 1>(&bar_pair_end[pq], pair_ends & 1, &abort_flag))) break;
        const float l_row = s_hsum[x][0][n] + s_hsum[x][1][n];
        ++pair_ends;
        uint8_t* stage = s_stage[warp - F::kSoftmax0];
        if (at.slot < 0) {
          const float inv = 1.f / l_row;
          uint32_t w[32];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint32_t o[16];
            tmem_ld16(tOx + g * 16, o);
            tmem_wait_ld();
            tmem_regs_ready(o);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
              w[8 * g + k] = *reinterpret_cast<const uint32_t*>(&h2);
            }
          }
          uint16_t* dst = p.out + (row0 + r_off) * 128 + col0;
          store_rows(w, live ? dst : nullptr, stage, lane);
        } else {
          float* mine = p.part + static_cast<size_t>(at.slot) * kRowsItem * kPartRow;
#pragma unroll
          for (int g2 = 0; g2 < 2; ++g2) {
            uint32_t o[32];
            tmem_ld16(tOx + g2 * 32, *reinterpret_cast<uint32_t(*)[16]>(o));
            tmem_ld16(tOx + g2 * 32 + 16, *reinterpret_cast<uint32_t(*)[16]>(o + 16));
            tmem_wait_ld();
            tmem_regs_ready(*reinterpret_cast<uint32_t(*)[16]>(o));
            tmem_regs_ready(*reinterpret_cast<uint32_t(*)[16]>(o + 16));
            store_rows(o, live ? mine + r_item * 128 + col0 + g2 * 32 : nullptr, stage, lane);
          }
          if (live && half == 0) {
            mine[kRowsItem * 128 + r_item] = m_run;
            mine[kRowsItem * 129 + r_item] = l_row;
          }
        }
        tc_fence_before();   // O is read: the next list's first PV (after its weights) may overwrite it
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_cempty[rs]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) mbar_wait_drain(&bar_done, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && abort_flag) atomicOr(p.err, BDLM_DEVERR_TIMEOUT);
}

// The queries as two e4m3 parts of 128 bytes side by side, with each one's power of two: 16 lanes a query, kSplitEach of
// them under way a thread.
constexpr int kSplitThreads = 256, kSplitEach = 4;
__global__ void __launch_bounds__(kSplitThreads) split_q_kernel(const Params p, uint8_t* __restrict__ q8, float* __restrict__ q_scale) {
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x;
  const long long rows = static_cast<long long>(p.B) * p.L * p.Hq;
  const long long row0 = static_cast<long long>(blockIdx.x) * (kSplitThreads / 16 * kSplitEach) + (t >> 4);
  uint4 v[kSplitEach];
#pragma unroll
  for (int i = 0; i < kSplitEach; ++i) {
    const long long row = row0 + i * (kSplitThreads / 16);
    v[i] = make_uint4(0, 0, 0, 0);
    if (row < rows) v[i] = __ldg(reinterpret_cast<const uint4*>(p.q + row * 128) + (t & 15));
  }
#pragma unroll
  for (int i = 0; i < kSplitEach; ++i) {
    const long long row = row0 + i * (kSplitThreads / 16);
    uint32_t most[1] = {magnitude(v[i])};
    const int e = q_exponent(rows_max(most, t & 31));
    if (row >= rows) continue;
    const float inv = pow2(-e);
    if ((t & 15) == 0) q_scale[row] = pow2(e);
    const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) split_e4m3x2(bf16_lo(u[k]) * inv, bf16_hi(u[k]) * inv, hi[k], lo[k]);
    *reinterpret_cast<uint2*>(q8 + row * 256 + (t & 15) * 8) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
    *reinterpret_cast<uint2*>(q8 + row * 256 + 128 + (t & 15) * 8) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
  }
}

// Tiles of the sequences before each, for more than kFewSequences.  One CTA.
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
    int w = s_warp[lane];
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
// What a CTA of either kernel needs of its list; false: nothing was cut.
struct JoinList {
  int b, kvh, rg, u0, parts;

  __device__ __forceinline__ bool find(const Params& p, int list, int ctas, int lane) {
    const int lists = p.Hkv * p.row_groups;
    b = list / lists;
    list -= b * lists;
    rg = list % p.row_groups;
    kvh = list / p.row_groups;
    bool ok;
    int sum, before;
    if (p.cum != nullptr) {
      sum = __ldg(p.cum + p.B);
      before = __ldg(p.cum + b);
    } else {
      sum = before = 0;
      for (int i = lane; i < p.B; i += 32) {
        const int n = (kv_tokens(p, i, &ok) + kTile - 1) / kTile;
        sum += n;
        if (i < b) before += n;
      }
      sum = __reduce_add_sync(0xffffffffu, sum);
      before = __reduce_add_sync(0xffffffffu, before);
    }
    const int tiles = (kv_tokens(p, b, &ok) + kTile - 1) / kTile;
    const long long per = unit_tiles(static_cast<long long>(sum) * lists, ctas);
    const long long c0 = static_cast<long long>(before) * lists + static_cast<long long>(list) * tiles;
    u0 = static_cast<int>(quotient(c0, per));
    parts = static_cast<int>(quotient(c0 + tiles - 1, per)) - u0 + 1;
    return parts > 1;
  }
  // part s: the first in its unit's second slot, the others in their units' first
  __device__ __forceinline__ const float* part(const Params& p, int s, int n_rows) const {
    return p.part + static_cast<size_t>(2 * (u0 + s) + (s == 0 ? 1 : 0)) * n_rows * kPartRow;
  }
  __device__ __forceinline__ uint16_t* row(const Params& p, int n) const {
    return p.out + ((static_cast<size_t>(b) * p.L + rg * p.lsub + n / p.G) * p.Hq + static_cast<size_t>(kvh) * p.G + n % p.G) * 128;
  }
};

// Many lists of few parts: CTA (list, 8 R rows), R rows a warp, whose loads are under way together, four head dims a
// lane.
template <int R>
__global__ void __launch_bounds__(256) join_few_kernel(const Params p, int n_rows, int ctas) {
  const int lane = threadIdx.x & 31, n0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * R;
  // The lengths can be read before the attention kernel is done: its CTAs let this one start after they waited for what
  // wrote them.
  JoinList j;
  const bool cut = j.find(p, blockIdx.x, ctas, lane);
  griddep_wait();
  griddep_launch_dependents();
  if (!cut) return;
  const int live = min(R, min(p.rows, (p.L - j.rg * p.lsub) * p.G) - n0);   // of the warp's rows
  if (live <= 0) return;
  float M[R], den[R];
  float4 acc[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    M[k] = -CUDART_INF_F;
    den[k] = 0.f;
    acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int at = 0; at < j.parts; at += 32) {
    const int s = at + lane;
    float e[R], l[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      e[k] = -CUDART_INF_F;
      l[k] = 0.f;
      if (s < j.parts && k < live) {
        e[k] = __ldcg(j.part(p, s, n_rows) + n_rows * 128 + n0 + k);
        l[k] = __ldcg(j.part(p, s, n_rows) + n_rows * 129 + n0 + k);
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (k >= live) break;
      const float top = fmaxf(M[k], warp_max(e[k])), was = ex2(M[k] - top);
      e[k] = s < j.parts ? ex2(e[k] - top) : 0.f;
      float d = e[k] * l[k];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
      den[k] = den[k] * was + d;
      acc[k] = make_float4(acc[k].x * was, acc[k].y * was, acc[k].z * was, acc[k].w * was);
      M[k] = top;
    }
    const int cnt = min(32, j.parts - at);
#pragma unroll(R == 1 ? 4 : 1)
    for (int i = 0; i < cnt; ++i) {
      const float4* from = reinterpret_cast<const float4*>(j.part(p, at + i, n_rows) + n0 * 128) + lane;
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const float w = __shfl_sync(0xffffffffu, e[k], i);
        const float4 o = k < live ? __ldcg(from + k * 32) : make_float4(0.f, 0.f, 0.f, 0.f);
        acc[k].x += w * o.x;
        acc[k].y += w * o.y;
        acc[k].z += w * o.z;
        acc[k].w += w * o.w;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (k >= live) break;
    const float inv = 1.f / den[k];
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[k].x * inv, acc[k].y * inv), hi = __floats2bfloat162_rn(acc[k].z * inv, acc[k].w * inv);
    reinterpret_cast<uint2*>(j.row(p, n0 + k))[lane] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

// Few lists of many parts: CTA (list, row), four groups of 128 threads, a head dim each, that take every fourth part.
constexpr int kJoinThreads = 512;
constexpr int kMaxCtas = 1024;   // parts of a list are at most the grid
__global__ void __launch_bounds__(kJoinThreads) join_many_kernel(const Params p, int n_rows, int ctas) {
  __shared__ float s_w[kMaxCtas], s_red[kJoinThreads / 32], s_acc[4][128];
  const int t = threadIdx.x, lane = t & 31, n = blockIdx.y;
  JoinList j;
  const bool cut = j.find(p, blockIdx.x, ctas, lane);   // (before the wait, as above)
  griddep_wait();
  griddep_launch_dependents();
  if (!cut || j.rg * p.lsub + n / p.G >= p.L) return;
  float m[kMaxCtas / kJoinThreads], l[kMaxCtas / kJoinThreads], M = -CUDART_INF_F;
#pragma unroll
  for (int i = 0; i < kMaxCtas / kJoinThreads; ++i) {
    const int s = i * kJoinThreads + t;
    m[i] = -CUDART_INF_F;
    l[i] = 0.f;
    if (s < j.parts) {
      m[i] = __ldcg(j.part(p, s, n_rows) + n_rows * 128 + n);
      l[i] = __ldcg(j.part(p, s, n_rows) + n_rows * 129 + n);
    }
    M = fmaxf(M, m[i]);
  }
  M = warp_max(M);
  if (lane == 0) s_red[t >> 5] = M;
  __syncthreads();
  M = warp_max(s_red[lane % (kJoinThreads / 32)]);
  float den = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxCtas / kJoinThreads; ++i) {
    const float e = ex2(m[i] - M);
    if (i * kJoinThreads + t < j.parts) s_w[i * kJoinThreads + t] = e;
    den = fmaf(e, l[i], den);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) den += __shfl_xor_sync(0xffffffffu, den, off);
  __syncthreads();
  if (lane == 0) s_red[t >> 5] = den;
  const int x = t & 127, g = t >> 7;
  float acc = 0.f;
#pragma unroll 8
  for (int s = g; s < j.parts; s += 4) acc = fmaf(s_w[s], __ldcg(j.part(p, s, n_rows) + n * 128 + x), acc);
  s_acc[g][x] = acc;
  __syncthreads();
  if (t >= 128) return;
  den = 0.f;
  for (int w = 0; w < kJoinThreads / 32; ++w) den += s_red[w];
  j.row(p, n)[x] = __bfloat16_as_ushort(__float2bfloat16_rn(((s_acc[0][x] + s_acc[1][x]) + (s_acc[2][x] + s_acc[3][x])) / den));
}

template <int N, int NC, int STAGES>
cudaError_t launch_few(const CUtensorMap& tk, const CUtensorMap& tv, const Params& p, int grid, cudaStream_t stream) {
  using F = Few<N, NC, STAGES>;
  constexpr size_t smem = F::kSmem;
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = once_per_device(attr_done, [] {
    const cudaError_t r = cudaFuncSetAttribute(few_rows_kernel<N, NC, STAGES>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(few_rows_kernel<N, NC, STAGES>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(few_rows_kernel<N, NC, STAGES>, dim3(grid), dim3(F::kThreads), smem, stream, tk, tv, p);
}

}  // namespace

Kv8AttnPlan plan_attention_kv8(int B, int L, int Hq, int Hkv, int max_pages, int num_sms) {
  Kv8AttnPlan pl;
  const int G = Hq / Hkv;
  // up to 256 rows a group; more of them read their keys once a group
  pl.lsub = G * L <= 256 ? L : 256 / G;
  pl.row_groups = (L + pl.lsub - 1) / pl.lsub;
  pl.rows = G * pl.lsub;
  // Rows that the MMAs take, the fewest that hold them: 16 rows (128 blocks of 4) in 107 us against 140 as 32, 32 (blocks of
  // 8) in 148 against 207 as 128.
  pl.n_rows = pl.rows <= 16 ? 16 : pl.rows <= 32 ? 32 : pl.rows <= 128 ? 128 : 256;
  const bool many = pl.n_rows >= 128;
  const long long lists = static_cast<long long>(B) * Hkv * pl.row_groups;
  const long long tiles = lists * ((max_pages + kTilePages - 1) / kTilePages);
  const long long ctas = pl.n_rows == 16 ? 2ll * num_sms : num_sms;
  pl.grid = static_cast<int>(tiles < ctas ? tiles : ctas < kMaxCtas ? ctas : kMaxCtas);
  // (a tile a list at most: no list is cut)
  pl.parts = max_pages <= kTilePages ? 0 : 2 * pl.grid;
  // Parts a list: about the CTAs over the lists.  With more lists than CTAs the CTA that writes a list's last part joins
  // them, beside its copies (128 blocks of 4 over 512-4096 tokens: 107 us, 110 with a kernel for it; 1024 single tokens over
  // 100-1000: 195 against 206); with fewer, whose parts are all written last, a kernel is faster (8 blocks of 4 over
  // 500-1500: 13.8 us against 16.7; one request of 6000: 14.1 against 19.4).  Few lists of many parts take a CTA a row (that
  // request: 16.7 us against 23 to 30 with few parts' kernel, before the rest was faster).
  pl.many_parts = lists * kFewParts < pl.grid;
  pl.join_here = pl.parts > 0 && !many && lists >= pl.grid;
  pl.work_bytes = pl.join_here ? (static_cast<size_t>(pl.grid) * (pl.n_rows / 16) + 1) * sizeof(int) : 0;
  pl.part_bytes = static_cast<size_t>(pl.parts) * pl.n_rows * kPartRow * sizeof(float);
  auto place = [](size_t& end, size_t bytes) {
    const size_t at = (end + 255) / 256 * 256;
    end = at + bytes;
    return at;
  };
  pl.bytes = pl.part_bytes;
  pl.cum_offset = place(pl.bytes, B > kFewSequences ? (static_cast<size_t>(B) + 1) * sizeof(int) : 0);
  pl.q_offset = place(pl.bytes, many ? static_cast<size_t>(B) * L * Hq * 256 : 0);
  pl.q_scale_offset = place(pl.bytes, many ? static_cast<size_t>(B) * L * Hq * sizeof(float) : 0);
  return pl;
}

template <int SUB>
cudaError_t launch_many(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const Params& p, int grid,
                        cudaStream_t stream) {
  constexpr size_t smem = Many<SUB>::kSmem;
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(many_rows_kernel<SUB>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(many_rows_kernel<SUB>, dim3(grid), dim3(Many<SUB>::kThreads), smem, stream, tq, tk, tv, p);
}

cudaError_t launch_attention_kv8(const Kv8AttnParams& a, const Kv8AttnPlan& pl, const CUtensorMap& tq, const CUtensorMap& tk,
                                 const CUtensorMap& tv, void* data, int* work, cudaStream_t stream) {
  char* at = static_cast<char*>(data);
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
  p.q_scale = reinterpret_cast<const float*>(at + pl.q_scale_offset);
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
  p.join_here = pl.join_here;
  p.scale_log2 = a.scale_log2;
  const unsigned lists = static_cast<unsigned>(p.B) * p.Hkv * p.row_groups;
  cudaError_t e;
  if (a.B > kFewSequences) {
    int* cum = reinterpret_cast<int*>(at + pl.cum_offset);
    e = launch_pdl(cum_tiles_kernel, dim3(1), dim3(kCumThreads), 0, stream, p, cum);
    if (e != cudaSuccess) return e;
    p.cum = cum;
  }
  if (pl.n_rows >= 128) {
    constexpr long long kRows = kSplitThreads / 16 * kSplitEach;
    const unsigned ctas = static_cast<unsigned>((static_cast<long long>(p.B) * p.L * p.Hq + kRows - 1) / kRows);
    e = launch_pdl(split_q_kernel, dim3(ctas), dim3(kSplitThreads), 0, stream, p, reinterpret_cast<uint8_t*>(at + pl.q_offset),
                   reinterpret_cast<float*>(at + pl.q_scale_offset));
    if (e != cudaSuccess) return e;
    e = pl.n_rows == 128 ? launch_many<1>(tq, tk, tv, p, pl.grid, stream) : launch_many<2>(tq, tk, tv, p, pl.grid, stream);
  } else {
    // Stages of 16 KB: two CTAs of four keep 128 KB an SM under way.  Six, all that fit, are slower where lists are long (32
    // single tokens over 16384-32768 tokens 128.5 us against 122.7, 32 blocks of 4 over 2000-16000 99.7 against 95.8) and the
    // same where they are short; three cost 2 to 4 %.  The one CTA of 32 rows takes twelve: 148.5 us for 128 blocks of 8
    // over 512-4096, 153.7 with eight, 126.4 against 127.4 on long lists.
    e = pl.n_rows == 32  ? launch_few<32, 32, 12>(tk, tv, p, pl.grid, stream)
        // (eight rows: half the softmax; 1024 single tokens over 100-1000 tokens 195 us against 269, one block 10.2 against 11.2)
        : pl.rows <= 8 ? launch_few<16, 8, 4>(tk, tv, p, pl.grid, stream)
                       : launch_few<16, 16, 4>(tk, tv, p, pl.grid, stream);
  }
  if (e != cudaSuccess || pl.parts == 0 || pl.join_here) return e;
  if (pl.many_parts) return launch_pdl(join_many_kernel, dim3(lists, p.rows), dim3(kJoinThreads), 0, stream, p, pl.n_rows, pl.grid);
  if (pl.n_rows >= 128) return launch_pdl(join_few_kernel<4>, dim3(lists, (p.rows + 31) / 32), dim3(256), 0, stream, p, pl.n_rows, pl.grid);
  return launch_pdl(join_few_kernel<1>, dim3(lists, (p.rows + 7) / 8), dim3(256), 0, stream, p, pl.n_rows, pl.grid);
}

}  // namespace bdlm
