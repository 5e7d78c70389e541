// Attention of new tokens over the 4-bit cache (bq_attn_kv4).
//
// A value of the cache is x = low + step * u with a code u in 0..15 for each
// group of dims, so for a query q and weights p
//   q . k[t]        = sum_g step[t, g] * (sum_{d in g} q[d] u[t, d]) + low[t, g] * (sum_{d in g} q[d])
//   sum_t p[t] v[t] = sum_t (p[t] step[t, g]) (u[t, d] - 7.5) + sum_t p[t] (low[t, g] + 7.5 step[t, g])
// and the tensor cores multiply the codes themselves: as fp16 subnormals they
// need one LOP3 per two codes and no arithmetic (kv4_device.cuh).
//
// The keys are the rows of the first product's A operand and the dims the
// rows of the second one's (ldmatrix transposes their bytes), so 8 query rows
// (the heads that share a kv head, times the query tokens) are its 8 columns
// and none of an MMA is idle at q_heads / kv_heads = 8.  Scores leave the
// first MMA with a key per lane row, where its step and low are applied, and
// movmatrix turns the weights into the second MMA's B operand.
//
// Two things keep the second sum exact where it cancels.  The weights p step are
// rounded to fp16, so the codes count from their middle: from 0, the weights'
// errors met values of 2.5 to 5 times the size, and the result was 2.4 to 5 times
// as far off.  (A power of two for each group carries weight * step into fp16's
// range; it follows the steps, 32 keys at a time.)  And codes are not negative, while the tensor cores truncate as
// they add: every second 16 keys enter as -(p step) (15 - u), which turns about
// the middle and costs nothing (a LOP3 takes the complement), so that the
// accumulators stay as small as the result instead of growing with the sum of
// the weights (128k keys: 7e-4 off without, 2e-4 being the rounding of the result).
// What turns them back, 7.5 sum_t +-(p step), is summed beside from the rounded weights.
//
// What bounds it.  One new token a sequence should be bound by reading the cache:
// 32 sequences of 32k keys (D 128, 8 kv heads, 4 query heads each, groups of 64:
// 739 MB) take 138 us, 5.4 TB/s, 79 % of a plain copy's rate.  What is left is
// instructions (about 600 for a warp's tile, 60 % of the issue slots over the
// whole launch), the first data 4.6 us after the launch, and blocks that end up to
// 16 us apart.  A short cache is bound by the fixed 10 us or
// so of scan, first data, straddled units and join (16 sequences of 4k keys 20.9 us,
// one of 128k 34.1), and the direct form by its latency (97 keys 3.7 us).  Many
// queries are bound by arithmetic: 2 x 256 tokens on 16k keys take 383 us
// (240 TFLOP/s of the formula's), the tensor pipe busy 42 % of the time at the
// two warps a scheduler that 255 registers allow.
//
// Work is split over warps by tiles of 32 keys.  A unit is one (sequence,
// kv head, block of query rows); the blocks of the grid take equal contiguous
// ranges of the tiles of all units, whatever the lengths are, and a unit that
// falls into several ranges is joined by a second kernel from (maximum, sum,
// accumulator) parts.  Short caches run one block per unit and no join.
#include <cuda_fp16.h>

#include "bq_device.cuh"
#include "decode_internal.h"
#include "kv4_device.cuh"

namespace bq {

namespace {

constexpr int AW = 4;             // warps of a block
constexpr int TILE = 32;          // keys of a warp's tile
// Up to here one block takes a whole unit, beyond it the grid shares the keys and a second kernel joins them.  Direct and
// split, with 8 kv heads of 128: 16 sequences of 300 keys 5.4 and 11.9 us, of 500 6.0 and 11.7, of 1000 8.8 and 14.2, of
// 1500 12.1 and 16.0; one sequence of 300 5.2 and 7.3, of 500 5.7 and 7.4, of 768 7.0 and 7.6, of 1000 8.6 and 7.7, of 2000
// 13.8 and 10.7.  The bound is the largest power of two at which no batch loses; larger batches would gain up to 1500.
constexpr int64_t DIRECT_LEN = 512;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float M_NONE = -1e30f;  // running maximum before any key
constexpr float VF_MOST = 1073741824.0f;   // 2**30: the smallest step, 2**-24, times it is 64

// A unit that has to be joined: its blocks, the first of them, whether that holds it in its second slot, and what the
// join needs of the sequence
struct Meta {
  int32_t parts;       // 0: nothing to join
  int32_t block, slot;
  int32_t head, row0, rows;
  int64_t first;
};

struct AttnParams {
  const __half* q;
  int64_t ld_q, T;
  const uint8_t* codes;
  const uint8_t* params;
  int64_t num_pages;
  int page_log2, heads, rep;      // rep = q_heads / kv_heads
  const int32_t* table;
  int64_t ld_table;
  const int32_t *lens, *cu_q;
  int64_t B;
  int64_t max_q, max_len, window;
  int qtiles;                     // blocks of query rows for max_q tokens
  float scale;
  __half* out;
  float* lse;
  float* parts;                   // [2 * grid][rows][D + 2]
  Meta* meta;                     // by unit [B][qtiles][heads], or by the block where a unit begins [grid]
  int by_unit;
  int* status;
};

// One sequence as the kernels see it: its query rows and range of keys.
struct Seq {
  int64_t first;       // first row of q
  int n;               // query tokens
  int len;             // keys
  int begin;           // first key any row sees, rounded down to 16
  int tiles;           // tiles of TILE keys from begin (at least 1 where n > 0)
  int qtiles;
};

__device__ __forceinline__ Seq load_seq(const AttnParams& a, int64_t b, int rows) {
  Seq s;
  s.first = b;
  int64_t n = 1;
  bool bad = false;
  if (a.cu_q) {
    s.first = a.cu_q[b];
    n = (int64_t)a.cu_q[b + 1] - s.first;
    if (n < 0 || s.first < 0 || s.first + n > a.T) {
      bad = true;
      n = 0;
    }
  }
  if (n > a.max_q) {
    bad = true;
    n = a.max_q;
  }
  int64_t len = a.lens[b];
  if (len < 0 || len > a.max_len) {
    bad = true;
    len = len < 0 ? 0 : a.max_len;
  }
  if (bad) record_error(a.status, BQ_ERR_INVALID_ARG);
  s.n = (int)n;
  s.len = (int)len;
  int64_t begin = 0;
  if (a.window > 0) {
    begin = len - n + 1 - a.window;
    begin = begin > 0 ? begin & ~15 : 0;
  }
  s.begin = (int)begin;
  const int64_t span = len - begin;
  s.tiles = n == 0 ? 0 : (span <= TILE ? 1 : (int)((span + TILE - 1) / TILE));
  s.qtiles = (int)((n * a.rep + rows - 1) / rows);
  return s;
}

__device__ __forceinline__ int64_t seq_cost(const AttnParams& a, const Seq& s) {
  return (int64_t)s.tiles * s.qtiles * a.heads;
}

// Blocks per SM, by the registers of the accumulators.  With D = 128 and 8 query rows, 3 blocks (168 registers a thread,
// nothing spilled) took 133 us for 739 MB of cache, 4 blocks (128 registers) 147 us, 2 blocks 138 us (before the second
// sum's signs, which cost 3 us).  With more query rows a thread spills some of its values (16 rows: 0.1 to 0.5 KB; 32 rows
// at 255 registers: 0.2 to 0.9).
constexpr int blocks_per_sm(int D, int nt) { return D < 256 && D * nt <= 256 ? 3 : 2; }

template <int D, int NG, int NT>
struct Cfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int R = D / 2;                     // bytes of a code row
  static constexpr int G = D / NG;
  static constexpr int KW = G / 32;                   // key words of a lane in a group
  static constexpr int MT = G / 16;                   // 16-dim tiles of a group
  static constexpr int PER = R / 16;                  // 16-byte pieces of a code row
  static constexpr int STAGES = 2;   // 3 or 4 stages a warp read 1-2 % slower
  static constexpr int CODE_B = TILE * R;             // bytes of a tile's keys (or values)
  static constexpr int PAR_B = TILE * 4 * NG;
  static constexpr int STAGE_B = 2 * CODE_B + 2 * PAR_B;
  static constexpr int RING_B = AW * STAGES * STAGE_B;
  static constexpr int JOIN_B = AW * ROWS * (D + 4) * 4;
  static constexpr int WORK_B = RING_B > JOIN_B ? RING_B : JOIN_B;
  // With 64 accumulators a lane or more its queries and constants live in shared memory, and with 128 of D = 256 a
  // tile is worked on 16 keys at a time, for the registers' sake.
  static constexpr bool WIDE = D * NT >= 256;
  static constexpr int HB = D == 256 && NT == 2 ? 1 : 2;
  static constexpr int QF_B = NT * NG * KW * 512;
  static constexpr int SMEM = WORK_B + (WIDE ? QF_B + ROWS * 4 * (NG + 3) : 0);
  static constexpr int BLOCKS = blocks_per_sm(D, NT);
};

// XOR of the address bits of token `tok`'s row of key codes, so that the key
// loads (tokens 2g or 2g + 1, 16 / NG bytes of each quad lane) touch every bank
// once, and of its row of value codes for ldmatrix (8 consecutive tokens, 16
// bytes each).  Rows are D / 2 bytes apart.
template <int D>
__device__ __forceinline__ constexpr int key_swizzle(int tok) {
  const int b1 = (tok >> 1) & 1, b2 = (tok >> 2) & 1, b3 = (tok >> 3) & 1;
  return (D == 64 ? 0 : b1 << 6) | (b2 << 5) | (b3 << 4);
}
template <int D>
__device__ __forceinline__ constexpr int value_swizzle(int tok) {
  if (D == 64) return ((tok >> 2) & 1) << 4;
  if (D == 128) return ((tok >> 1) & 3) << 4;
  return (tok & 7) << 4;
}

template <int BYTES>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (BYTES == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (BYTES == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// What a row's sum makes of its accumulator, and the log-sum: a row that has seen no key has the sum 0, any other at
// least 1 (its largest weight) or NaN, which stays NaN.
__device__ __forceinline__ float inverse(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }
__device__ __forceinline__ float log_sum(float top, float sum) {
  return sum == 0.0f ? -INFINITY : (top + log2f(sum)) * LN2;
}

// x / p of a power of two p.  The inverse by its exponent saves 0.7 us at 97 keys and 3 at 16 sequences of 4k with D = 256;
// with several tiles of query rows, whose registers are all taken, ptxas keeps it over the loop: 2 x 256 tokens on 16k
// keys 404 us, 382 with a division, 16 x 4 tokens on 4k with D = 256 70 and 63.
template <bool DIVIDE>
__device__ __forceinline__ float over_power(float x, float p) {
  if constexpr (DIVIDE) return x / p;
  else return x * pow2f(-ilog2f(p));
}

// The params of two consecutive tokens
template <int NG>
__device__ __forceinline__ void load_pair(const uint8_t* p, uint32_t (&w)[2][NG]) {
  if constexpr (NG == 4) {
    load_words<16>(p, w[0]);
    load_words<16>(p + 16, w[1]);
  } else {
    uint32_t v[2 * NG];
    load_words<8 * NG>(p, v);
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      w[0][i] = v[i];
      w[1][i] = v[NG + i];
    }
  }
}

template <int D, int NG, int NT, bool SPLIT>
__global__ void __launch_bounds__(AW * 32, Cfg<D, NG, NT>::BLOCKS) attn_kv4_kernel(const AttnParams a) {
  using C = Cfg<D, NG, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t scan[AW + 2];
  __shared__ Seq first_seq;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- which tiles are ours ----
  int64_t at, stop, base = 0;       // tiles [at, stop) of all units; base: the first tile of sequence b
  int64_t b = 0;
  Seq s;
  int64_t each = 0, extra = 0;      // every block has `each` tiles, the first `extra` of them one more
  if constexpr (SPLIT) {
    // total tiles, then the sequence that holds our first tile: each thread
    // sums the costs of a contiguous share of the sequences
    const int64_t per = (a.B + AW * 32 - 1) / (AW * 32);
    const int64_t b0 = min((int64_t)tid * per, a.B), b1 = min(b0 + per, a.B);
    int64_t mine = 0;
    for (int64_t i = b0; i < b1; ++i) {
      s = load_seq(a, i, C::ROWS);
      mine += seq_cost(a, s);
    }
    int64_t inc = mine, total = 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int64_t before = 0;
#pragma unroll
    for (int w = 0; w < AW; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    inc += before;
    if (total >> 32) {
      each = total / gridDim.x;
      extra = total % gridDim.x;
    } else {
      each = (uint32_t)total / gridDim.x;
      extra = (uint32_t)total % gridDim.x;
    }
    at = each * blockIdx.x + min((int64_t)blockIdx.x, extra);
    stop = at + each + (blockIdx.x < extra ? 1 : 0);
    if (tid == 0 && !a.by_unit) a.meta[blockIdx.x] = Meta{};
    if (at >= stop) return;
    if (at >= inc - mine && at < inc) {
      int64_t sum = inc - mine, i = b0;
      if (per > 1) {
        for (;; ++i) {
          s = load_seq(a, i, C::ROWS);
          if (at < sum + seq_cost(a, s)) break;
          sum += seq_cost(a, s);
        }
      }
      first_seq = s;
      scan[AW] = i;
      scan[AW + 1] = sum;
    }
    __syncthreads();
    b = scan[AW];
    base = scan[AW + 1];
    s = first_seq;
  } else {
    const int64_t per_b = (int64_t)a.qtiles * a.heads;
    b = blockIdx.x / per_b;
    const int unit = (int)(blockIdx.x - b * per_b);
    s = load_seq(a, b, C::ROWS);
    if (unit >= s.qtiles * a.heads) return;
    at = (int64_t)unit * s.tiles;
    stop = at + s.tiles;
  }
  const int64_t at0 = at;

  // Rows g and g + 8 of a first MMA are keys 2g and 2g + 1 of its 16, so that the
  // k columns 2t, 2t + 1 and 2t + 8, 2t + 9 of the second one are keys 4t, 4t + 2
  // and 4t + 1, 4t + 3: the bytes 0, 2 and 1, 3 that ldmatrix hands out.
  const uint32_t ring = smem_u32(smem) + warp * C::STAGES * C::STAGE_B;
  const int P = 1 << a.page_log2;
  constexpr int PR = 4 * NG;                           // bytes of a token's params
  const uint32_t page_codes = 2u * a.heads * P * C::R, page_params = 2u * a.heads * P * PR;
  const uint32_t v_codes = (uint32_t)a.heads * P * C::R;   // from a key row to its value row
  // this lane's share of a copy of 16 keys: piece `lane` (+ 32 i) of their codes, and a piece of their params
  const int cp_tok = lane / C::PER;
  const uint32_t cp_lin = cp_tok * C::R + (lane % C::PER) * 16;
  const int pp = lane & 15;                            // params piece; keys by the low lanes, values by the high ones
  const uint32_t pp_dst = 2 * C::CODE_B + (lane >= 16 ? C::PAR_B : 0) + pp * 16;
  const uint32_t pp_src = (lane >= 16 ? (uint32_t)a.heads * P * PR : 0u) + pp * 16;
  // this lane's loads: key words of tokens 2g and 2g + 1 (group 0), rows of the values' matrices
  const uint32_t k_at0 = ((2 * g) * C::R + t * (C::G / 8)) ^ key_swizzle<D>(2 * g);
  const uint32_t v_at = C::CODE_B + (((lane & 15) * C::R + (lane >> 4) * 16) ^ value_swizzle<D>(lane & 15));

  while (at < stop) {
    while (at >= base + seq_cost(a, s)) {              // the next sequence with work
      base += seq_cost(a, s);
      s = load_seq(a, ++b, C::ROWS);
    }
    const int unit = (at - base) >> 32 ? (int)((at - base) / s.tiles) : (int)((uint32_t)(at - base) / (uint32_t)s.tiles);
    const int64_t u0 = base + (int64_t)unit * s.tiles;
    const int first_tile = (int)(at - u0);
    const int last_tile = (int)min((int64_t)s.tiles, stop - u0);
    const bool whole = !SPLIT || (first_tile == 0 && last_tile == s.tiles);
    const int qt = unit / a.heads, head = unit - qt * a.heads;
    const int row0 = qt * C::ROWS, rows = min(C::ROWS, s.n * a.rep - row0);
    const int ntile = last_tile - first_tile;
    const int mytiles = ntile > warp ? (ntile - warp + AW - 1) / AW : 0;

    // keys past `end` are seen by no row of this block; rows see [lo, hi]
    const int end = min(s.len, s.len - s.n + (row0 + rows - 1) / a.rep + 1);
    const int all_end = s.len - s.n + row0 / a.rep + 1;                 // every row sees below this
    const int all_begin = a.window > 0 ? max((int64_t)0, (int64_t)end - a.window) : 0;   // ... and from here on
    const int first_seen = a.window > 0 ? (int)max((int64_t)0, (int64_t)all_end - a.window) : 0;
    const int key0 = s.begin + first_tile * TILE;

    // pages of this warp's next 16 tiles: lane holds the page of 16 keys
    const int32_t* trow = a.table + b * a.ld_table;
    auto load_page = [&](int k0) -> int {
      const int key = key0 + (warp + AW * (k0 + (lane >> 1))) * TILE + (lane & 1) * 16;
      int page = 0;
      if (key < end && k0 + (lane >> 1) < mytiles) {
        page = trow[key >> a.page_log2];
        if (page < 0 || page >= a.num_pages) {
          record_error(a.status, BQ_ERR_INVALID_ARG);
          page = 0;
        }
      }
      return page;
    };
    int pages = load_page(0), pages_next = load_page(16);
    // Where the range goes on with the next unit of this sequence, its first tiles are brought to L2 while this one is
    // worked on (2 x 256 tokens on 16k keys 382 us, 393 without; 16 sequences of 4k 21.3 and 21.4).
    int ahead = -1;
    const int ahead_key = s.begin + warp * TILE + (lane >> 4) * 16;
    if (SPLIT && last_tile == s.tiles && u0 + s.tiles < stop && unit + 1 < s.qtiles * a.heads && ahead_key < s.len)
      ahead = trow[ahead_key >> a.page_log2];

    // ---- copy tile k of this warp into its ring ----
    // (keys from `end` on are not copied: what the ring holds there is masked)
    const uint8_t* const unit_codes = a.codes + (int64_t)head * P * C::R + lane * 16;
    const uint8_t* const unit_params = a.params + (int64_t)head * P * PR + pp_src;
    uint32_t put = ring;                               // stage that the next copy fills
    auto issue = [&](int k) {
      if (k < mytiles) {
        if (k > 0 && (k & 15) == 0) {
          pages = pages_next;
          pages_next = load_page(k + 16);
        }
        const int key = key0 + (warp + AW * k) * TILE;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t page = __shfl_sync(0xffffffffu, pages, 2 * (k & 15) + h);
          if (key + 16 * h < end) {
            const uint32_t off = (key + 16 * h) & (P - 1);
            const uint8_t* kc = unit_codes + (uint64_t)page * page_codes + off * C::R;
            const uint8_t* vc = kc + v_codes;
#pragma unroll
            for (int i = 0; i < C::PER / 2; ++i) {
              constexpr int STEP = 32 / C::PER;        // tokens of one copy of the warp
              const uint32_t lin = cp_lin + (16 * h + i * STEP) * C::R;
              cp_async_16_u(put + (lin ^ key_swizzle<D>(cp_tok + i * STEP)), kc + i * 512);
              cp_async_16_u(put + C::CODE_B + (lin ^ value_swizzle<D>(cp_tok + i * STEP)), vc + i * 512);
            }
            if (pp < PR) cp_async_16_u(put + pp_dst + h * 16 * PR, unit_params + (uint64_t)page * page_params + off * PR);
          }
        }
      }
      cp_async_commit();
      put = put == ring + (C::STAGES - 1) * C::STAGE_B ? ring : put + C::STAGE_B;
    };
    // ---- query fragments: column g of n-tile nt is row row0 + 8 nt + g ----
    struct Query {
      uint4 f[NG][C::KW];          // (low codes' pair, pair; high codes' pair, pair) of a key word
      float c, sum[NG];            // factor of the products, scaled sums over the groups
    };
    auto fetch_query = [&](int nt, Query& q) {
      const int r = row0 + min(8 * nt + g, rows - 1);
      const int tok = r / a.rep, hr = r - tok * a.rep;
      const __half* qp = a.q + (s.first + tok) * a.ld_q + (int64_t)(head * a.rep + hr) * D;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr)
#pragma unroll
        for (int i = 0; i < C::KW; ++i)
          q.f[gr][i] = *reinterpret_cast<const uint4*>(qp + gr * C::G + t * (C::G / 4) + 8 * i);
    };
    auto finish_query = [&](Query& q) {
      float top = 0.0f;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        q.sum[gr] = 0.0f;
#pragma unroll
        for (int i = 0; i < C::KW; ++i) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(&q.f[gr][i]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack_h2(w[e]);
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            q.sum[gr] += f.x + f.y;
          }
        }
      }
      const float sc = a.scale * LOG2E;
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) q.sum[gr] += __shfl_xor_sync(0xffffffffu, q.sum[gr], o);
        q.sum[gr] *= sc;
      }
      // the row times a power of two that brings its largest value to [2**10, 2**11): exact, and the
      // columns that meet low codes can carry the factor 16 that low and high codes differ by
      const int e = top > 0.0f ? 10 - ilog2f(top) : 0;
      const float f1 = pow2f(e), f16 = f1 * 16.0f;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr)
#pragma unroll
        for (int i = 0; i < C::KW; ++i) {
          const uint4 v = q.f[gr][i];
          const float2 d01 = unpack_h2(v.x), d23 = unpack_h2(v.y), d45 = unpack_h2(v.z), d67 = unpack_h2(v.w);
          q.f[gr][i] = make_uint4(pack_h2(d01.x * f16, d45.x * f16), pack_h2(d23.x * f16, d67.x * f16),
                                  pack_h2(d01.y * f1, d45.y * f1), pack_h2(d23.y * f1, d67.y * f1));
        }
      q.c = sc * pow2f(20 - e);
    };
    // (the loads of the queries go out before the copies, which wait for their pages)
    Query q0;
    if (!C::WIDE || warp < NT) fetch_query(C::WIDE ? warp : 0, q0);
#pragma unroll
    for (int k = 0; k < C::STAGES - 1; ++k) issue(k);

    if (SPLIT && ahead >= 0 && ahead < a.num_pages) {
      constexpr int LINES = 16 * C::R / 128;
      const int64_t row = (int64_t)(head + 1 == a.heads ? 0 : head + 1) * P + (ahead_key & (P - 1));
      const uint8_t* const kc = a.codes + (uint64_t)ahead * page_codes + row * C::R;
#pragma unroll
      for (int i = lane & 15; i < 2 * LINES; i += 16)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(kc + (i % LINES) * 128 + (i >= LINES ? v_codes : 0u)));
      if ((lane & 15) < 2)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.params + (uint64_t)ahead * page_params + row * PR +
                                                      (lane & 1 ? (uint32_t)a.heads * P * PR : 0u)));
    }

    // last and first key that row r (of the unit's n-tiles) sees
    auto last_key = [&](int r) { return s.len - s.n + (row0 + min(r, rows - 1)) / a.rep; };
    auto first_key = [&](int hi) { return a.window > 0 ? (int)max((int64_t)0, (int64_t)hi + 1 - a.window) : 0; };
    constexpr int NR = C::WIDE ? 1 : NT;
    uint4 qr[NR][NG][C::KW];              // the same in registers ...
    P2 cfr[NR], qsr[NR][NG];              // ... with the constants of columns 2t, 2t + 1
    int2 hir[NR];
    uint4* const qsm = reinterpret_cast<uint4*>(smem + C::WORK_B);   // or in shared memory: [nt][group][word][lane],
    float* const csm = reinterpret_cast<float*>(smem + C::WORK_B + C::QF_B);   // [factor, sums, last, first][row]
    if constexpr (C::WIDE) {
      static_assert(NT <= AW, "a warp prepares one tile of queries");
      if (warp < NT) {
        const int nt = warp;
        finish_query(q0);
        const Query& q = q0;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
#pragma unroll
          for (int i = 0; i < C::KW; ++i) qsm[((nt * NG + gr) * C::KW + i) * 32 + lane] = q.f[gr][i];
          if (t == 0) csm[(1 + gr) * C::ROWS + 8 * nt + g] = q.sum[gr];
        }
        if (t == 0) {
          const int hi = last_key(8 * nt + g);
          csm[8 * nt + g] = q.c;
          csm[(1 + NG) * C::ROWS + 8 * nt + g] = __int_as_float(hi);
          csm[(2 + NG) * C::ROWS + 8 * nt + g] = __int_as_float(first_key(hi));
        }
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt > 0) fetch_query(nt, q0);
        finish_query(q0);
        const Query& q = q0;
        const int src = 8 * t;             // lane of row 2t
        cfr[nt] = p2(__shfl_sync(0xffffffffu, q.c, src), __shfl_sync(0xffffffffu, q.c, src + 4));
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          qsr[nt][gr] = p2(__shfl_sync(0xffffffffu, q.sum[gr], src), __shfl_sync(0xffffffffu, q.sum[gr], src + 4));
#pragma unroll
          for (int i = 0; i < C::KW; ++i) qr[nt][gr][i] = q.f[gr][i];
        }
        hir[nt] = make_int2(last_key(8 * nt + 2 * t), last_key(8 * nt + 2 * t + 1));
      }
    }
    auto query = [&](int nt, int gr, int i) -> uint4 {
      if constexpr (C::WIDE) return qsm[((nt * NG + gr) * C::KW + i) * 32 + lane];
      else return qr[nt][gr][i];
    };
    auto factor = [&](int nt) -> P2 {
      if constexpr (C::WIDE) return *reinterpret_cast<const P2*>(csm + 8 * nt + 2 * t);
      else return cfr[nt];
    };
    auto query_sum = [&](int nt, int gr) -> P2 {
      if constexpr (C::WIDE) return *reinterpret_cast<const P2*>(csm + (1 + gr) * C::ROWS + 8 * nt + 2 * t);
      else return qsr[nt][gr];
    };
    auto lasts = [&](int nt) -> int2 {
      if constexpr (C::WIDE) return *reinterpret_cast<const int2*>(csm + (1 + NG) * C::ROWS + 8 * nt + 2 * t);
      else return hir[nt];
    };
    auto firsts = [&](int nt) -> int2 {
      if constexpr (C::WIDE) return *reinterpret_cast<const int2*>(csm + (2 + NG) * C::ROWS + 8 * nt + 2 * t);
      else return make_int2(first_key(hir[nt].x), first_key(hir[nt].y));
    };

    float o[NT][NG][C::MT][4];
    P2 mid[NT][NG], m[NT], l[NT];         // columns 2t, 2t + 1; mid: what the codes' middles add, times vf
    P2 back[NR][NG];                      // - 7.5 times the signed weights (with many rows, for the registers' sake, in mid)
    float vf[NG];                         // powers of two that the steps of a group of the values carry into fp16
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) vf[gr] = VF_MOST;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = l[nt] = p2(0.0f, 0.0f);
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        mid[nt][gr] = p2(0.0f, 0.0f);
        if (!C::WIDE) back[nt % NR][gr] = p2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[nt][gr][i][j] = 0.0f;
      }
    }

    // Columns that have seen a key have a running maximum m; the others hold 0
    // there, and while there are any (`fresh`) every step renews the maxima.
    bool fresh = true;
    uint32_t seen = 0;
    uint32_t st = ring;
    constexpr int HB = C::HB;             // halves (16 keys) of a step
#pragma unroll 1
    for (int k = 0; k < mytiles; ++k) {
      cp_async_wait<C::STAGES - 2>();
      __syncwarp();
      issue(k + C::STAGES - 1);
#pragma unroll
      for (int h0 = 0; h0 < 2; h0 += HB) {
      const uint32_t sth = st + 16 * h0 * C::R;
      const uint8_t* sp = smem + (sth - smem_u32(smem));
      const uint8_t* pp16 = smem + (st - smem_u32(smem)) + 2 * C::CODE_B + (16 * h0 + 2 * g) * PR;
      const int key = key0 + (warp + AW * k) * TILE + 16 * h0;

      // ---- scores: base-2 logits less the running maximum ----
      P2 sv[HB][NT][2];                   // [half][n-tile][key 2g, 2g + 1]
      uint32_t vp[HB][2][NG];             // (step, low) of the values, keys 2g and 2g + 1 of each half
#pragma unroll
      for (int h = 0; h < HB; ++h) {
        uint32_t kp[2][NG];
        load_pair<NG>(pp16 + 16 * h * PR, kp);
        load_pair<NG>(pp16 + 16 * h * PR + C::PAR_B, vp[h]);
        P2 x[NT][2], y[NT][2];            // products by the steps; what the lows add, less the maximum
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 mm = f2(m[nt]);
          y[nt][0] = y[nt][1] = p2(-mm.x, -mm.y);
        }
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          float acc[NT][4];
          uint32_t w0[C::KW], w1[C::KW];
          const uint8_t* kw = sp + (k_at0 ^ (gr * (C::G / 2))) + 16 * h * C::R;
          load_words<C::G / 8>(kw, w0);
          // token 2g + 1: the next row, in the same 128-byte line (or the next line) with the same swizzle
          load_words<C::G / 8>(C::R == 64 ? sp + (k_at0 ^ (gr * (C::G / 2)) ^ 64) + 16 * h * C::R
                                          : (C::R == 32 ? sp + (k_at0 ^ (gr * (C::G / 2)) ^ 32) + 16 * h * C::R
                                                        : kw + C::R),
                               w1);
#pragma unroll
          for (int i = 0; i < C::KW; ++i) {
            const uint32_t x0 = w0[i] >> 8, x1 = w1[i] >> 8;
            const uint32_t l0 = w0[i] & CODE_LO, l1 = w1[i] & CODE_LO, l2 = x0 & CODE_LO, l3 = x1 & CODE_LO;
            const uint32_t h0 = w0[i] & CODE_HI, h1 = w1[i] & CODE_HI, h2 = x0 & CODE_HI, h3 = x1 & CODE_HI;
            uint4 qv[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              qv[nt] = query(nt, gr, i);
              if (i == 0) mma_f16_zero(acc[nt], l0, l1, l2, l3, qv[nt].x, qv[nt].y);
              else mma_f16(acc[nt], l0, l1, l2, l3, qv[nt].x, qv[nt].y);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt], h0, h1, h2, h3, qv[nt].z, qv[nt].w);
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float2 p = unpack_h2(kp[r][gr]);
            const P2 step = p2(p.x, p.x), low = p2(p.y, p.y);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const P2 d = p2(acc[nt][2 * r], acc[nt][2 * r + 1]);
              x[nt][r] = gr == 0 ? mul2(step, d) : fma2(step, d, x[nt][r]);
              y[nt][r] = fma2(low, query_sum(nt, gr), y[nt][r]);
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const P2 c = factor(nt);
#pragma unroll
          for (int r = 0; r < 2; ++r) sv[h][nt][r] = fma2(x[nt][r], c, y[nt][r]);
        }
      }
      // keys that some row does not see, and what lies past the last one
      if (key < all_begin || key + 16 * HB > all_end) {
#pragma unroll
        for (int h = 0; h < HB; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int tok = key + 16 * h + 2 * g + r;
            if (tok >= end || tok < first_seen) {
#pragma unroll
              for (int gr = 0; gr < NG; ++gr) vp[h][r][gr] = 0;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int2 hi = lasts(nt), lo = firsts(nt);
              float2 v = f2(sv[h][nt][r]);
              if (tok > hi.x || tok < lo.x) v.x = -INFINITY;
              if (tok > hi.y || tok < lo.y) v.y = -INFINITY;
              sv[h][nt][r] = p2(v.x, v.y);
            }
          }
      }

      // ---- running maximum, renewed only when a score passes it by 2**8 ----
      float2 top[NT];
      float step_top[NG], most = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        top[nt] = f2(sv[0][nt][0]);
#pragma unroll
        for (int i = 1; i < 2 * HB; ++i) {
          const float2 v = f2(sv[i / 2][nt][i & 1]);
          top[nt].x = fmaxf(top[nt].x, v.x);
          top[nt].y = fmaxf(top[nt].y, v.y);
        }
        most = fmaxf(most, fmaxf(top[nt].x, top[nt].y));
      }
      // The largest step of a group times its factor is kept in [1, 240] (a lane that sees it elsewhere asks for the
      // renewal below, which looks at all of them): a weight is below 2**8, so that weight * step * factor stays below
      // fp16's 65504, and for that step weights down to 2**-14 stay normal numbers.  With one factor for all groups,
      // only ever lowered, the smaller of two groups 2**27 apart was 37 times as far off as its bound.  A factor for each
      // that also rises costs 0.5 us of 137 on 32 sequences of 32k keys.
      bool renew = fresh || most > 8.0f;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        __half2 most_step = __float2half2_rn(0.0f);
#pragma unroll
        for (int h = 0; h < HB; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            most_step = __hmax2(most_step, __habs2(*reinterpret_cast<const __half2*>(&vp[h][r][gr])));
        step_top[gr] = __low2float(most_step);
        const float v = step_top[gr] * vf[gr];
        renew = renew || !(v >= 1.0f && v <= 240.0f);
      }
      if (__any_sync(0xffffffffu, renew)) {
        float fv[NG];
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          // (not negative, so that its bits compare as integers)
          const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(step_top[gr])));
          const bool keep = top * vf[gr] <= 240.0f && (top * vf[gr] >= 1.0f || vf[gr] == VF_MOST);
          const float nv = keep ? vf[gr] : (top > 0.0f ? pow2f(6 - ilog2f(top)) : VF_MOST);   // top to [2**6, 2**7)
          fv[gr] = over_power<C::WIDE && (NT > 1)>(nv, vf[gr]);
          vf[gr] = nv;
        }
        bool all = true;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float up[2], f[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float v = j ? top[nt].y : top[nt].x;
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, x));
            const uint32_t bit = 1u << (2 * nt + j);
            // a first maximum may lie below 0; later ones only rise
            up[j] = seen & bit ? fmaxf(v, 0.0f) : (v == -INFINITY ? 0.0f : v);
            if (v != -INFINITY) seen |= bit;
            all = all && (seen & bit);
            f[j] = ex2(fminf(-up[j], 0.0f));       // (nothing has been summed where up < 0)
          }
          const P2 ff = p2(f[0], f[1]), down = p2(-up[0], -up[1]);
          m[nt] = add2(m[nt], p2(up[0], up[1]));
          l[nt] = mul2(l[nt], ff);
#pragma unroll
          for (int h = 0; h < HB; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) sv[h][nt][r] = add2(sv[h][nt][r], down);
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            const P2 of = p2(f[0] * fv[gr], f[1] * fv[gr]);
            mid[nt][gr] = mul2(mid[nt][gr], of);
            if (!C::WIDE) back[nt % NR][gr] = mul2(back[nt % NR][gr], of);
#pragma unroll
            for (int i = 0; i < C::MT; ++i)
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                const float2 v = f2(mul2(p2(o[nt][gr][i][e], o[nt][gr][i][e + 1]), of));
                o[nt][gr][i][e] = v.x;
                o[nt][gr][i][e + 1] = v.y;
              }
          }
        }
        fresh = !__all_sync(0xffffffffu, all);
      }

      // ---- weights, their sums, and the second product ----
#pragma unroll
      for (int h = 0; h < HB; ++h) {
        const bool turned = (h0 + h) & 1;
        uint32_t pf[NT][NG][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          P2 vs[NG], vl[NG];
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            const float2 v = unpack_h2(vp[h][r][gr]);
            const float w = v.x * (turned ? -vf[gr] : vf[gr]), low = vf[gr] * fmaf(7.5f, v.x, v.y);
            vs[gr] = p2(w, w);
            vl[gr] = p2(low, low);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 e = f2(sv[h][nt][r]);
            const P2 w = p2(ex2(e.x), ex2(e.y));
            l[nt] = add2(l[nt], w);
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
              // the only rounding to 16 bits: weight times step, 2**-11 relative
              const float2 v = f2(mul2(w, vs[gr]));
              const uint32_t w16 = pack_h2(v.x, v.y);
              mid[nt][gr] = fma2(w, vl[gr], mid[nt][gr]);
              P2& to = C::WIDE ? mid[nt][gr] : back[nt % NR][gr];
              to = fma_h2(w16, 0xc780u, to);       // 0xc780: -7.5
              pf[nt][gr][r] = movmatrix_trans(w16);
            }
          }
        }
#pragma unroll
        for (int c = 0; c < C::PER; c += 2) {
          // 16-byte pieces c and c + 1 (32 dims each) of 16 tokens
          uint32_t w[4];
          ldmatrix_b8_trans_x2(sth + (v_at ^ (c * 16)) + 16 * h * C::R, w);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int gr = (c + x / 2) * 32 / C::G, i = ((c + x / 2) * 32 % C::G) / 16 + (x & 1);
            const uint32_t e = w[x] >> 8;
            const uint32_t a0 = (turned ? ~w[x] : w[x]) & CODE_LO, a1 = (turned ? ~w[x] : w[x]) & CODE_HI;
            const uint32_t a2 = (turned ? ~e : e) & CODE_LO, a3 = (turned ? ~e : e) & CODE_HI;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][gr][i], a0, a1, a2, a3, pf[nt][gr][0], pf[nt][gr][1]);
          }
        }
      }
      }
      st = st == ring + (C::STAGES - 1) * C::STAGE_B ? ring : st + C::STAGE_B;
    }

    // ---- join the warps: accumulators in plain units through shared memory ----
    cp_async_wait<0>();
    __syncthreads();                      // every warp is done with its ring
    float* const js = reinterpret_cast<float*>(smem);
    constexpr int JS = D + 4;             // floats of a row: D values, maximum, sum, padding
    float unit_v[NG];
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) unit_v[gr] = over_power<C::WIDE && (NT > 1)>(pow2f(24), vf[gr]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 mm = f2(m[nt]), ll = f2(l[nt]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float sum = j ? ll.y : ll.x, low[NG];
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          const float2 x = f2(C::WIDE ? mid[nt][gr] : add2(mid[nt][gr], back[nt % NR][gr]));
          low[gr] = over_power<C::WIDE && (NT > 1)>(j ? x.y : x.x, vf[gr]);
        }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          sum += __shfl_xor_sync(0xffffffffu, sum, x);
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) low[gr] += __shfl_xor_sync(0xffffffffu, low[gr], x);
        }
        float* row = js + (warp * C::ROWS + 8 * nt + 2 * t + j) * JS;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr)
#pragma unroll
          for (int i = 0; i < C::MT; ++i) {
            // tile i of a group: byte g of its i-th 8, dims 2g and 2g + 1
            const int d = gr * C::G + 16 * i + 2 * g;
            *reinterpret_cast<float2*>(row + d) = make_float2(fmaf(o[nt][gr][i][j], unit_v[gr], low[gr]),
                                                              fmaf(o[nt][gr][i][2 + j], unit_v[gr] * 0.0625f, low[gr]));
          }
        if (g == 0) {
          row[D] = sum == 0.0f ? M_NONE : (j ? mm.y : mm.x);
          row[D + 1] = sum;
        }
      }
    }
    __syncthreads();
    constexpr int LANES = D / 4;          // threads of a row, 4 dims each
    for (int r = tid / LANES; r < rows; r += AW * 32 / LANES) {
      const int d = (tid % LANES) * 4;
      float mt = M_NONE;
#pragma unroll
      for (int w = 0; w < AW; ++w) mt = fmaxf(mt, js[(w * C::ROWS + r) * JS + D]);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < AW; ++w) {
        const float* row = js + (w * C::ROWS + r) * JS;
        const float f = ex2(row[D] - mt);
        const float4 x = *reinterpret_cast<const float4*>(row + d);
        v.x = fmaf(f, x.x, v.x);
        v.y = fmaf(f, x.y, v.y);
        v.z = fmaf(f, x.z, v.z);
        v.w = fmaf(f, x.w, v.w);
        sum = fmaf(f, row[D + 1], sum);
      }
      if (whole) {
        const int tok = (row0 + r) / a.rep, hr = row0 + r - tok * a.rep;
        const int64_t orow = (s.first + tok) * (int64_t)(a.heads * a.rep) + head * a.rep + hr;
        const float inv = inverse(sum);
        uint2 h;
        h.x = pack_h2(v.x * inv, v.y * inv);
        h.y = pack_h2(v.z * inv, v.w * inv);
        *reinterpret_cast<uint2*>(a.out + orow * D + d) = h;
        if (a.lse && d == 0) a.lse[orow] = log_sum(mt, sum);
      } else {
        const int64_t slot = 2 * (int64_t)blockIdx.x + (at != at0 ? 1 : 0);
        float* part = a.parts + (slot * C::ROWS + r) * JS;
        *reinterpret_cast<float4*>(part + d) = v;
        if (d == 0) {
          part[D] = mt;
          part[D + 1] = sum;
        }
      }
    }
    if (SPLIT && first_tile == 0 && tid == 0 && (!whole || a.by_unit)) {
      Meta mm{};
      if (!whole) {
        // the unit goes on in the blocks whose ranges cover its last tile
        const int64_t last = u0 + s.tiles - 1, big = (each + 1) * extra;
        const int64_t owner = last < big ? last / (each + 1) : extra + (last - big) / each;
        mm.parts = (int32_t)(owner - blockIdx.x + 1);
        mm.block = (int32_t)blockIdx.x;
        mm.slot = at != at0 ? 1 : 0;
        mm.head = head;
        mm.row0 = row0;
        mm.rows = rows;
        mm.first = s.first;
      }
      a.meta[a.by_unit ? (b * a.qtiles + qt) * a.heads + head : (int64_t)blockIdx.x] = mm;
    }
    at = u0 + last_tile;
    __syncthreads();                      // the ring is written again
  }
}

// Joins a unit that fell into several blocks' ranges.  With gridDim.y = 1 a block takes all rows of a unit at a time, a
// thread four dims of a row; with one block a row (few units, so many parts each) the threads share the parts.
template <int D, int NT>
__global__ void __launch_bounds__(256) attn_kv4_join_kernel(const AttnParams a) {
  constexpr int ROWS = 8 * NT, JS = D + 4, LANES = D / 4, SUBS = 256 / LANES;
  __shared__ float2 sums[SUBS];
  __shared__ float4 acc[256];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (a.by_unit && a.cu_q) {
    // units that do not exist (a sequence with fewer query tokens) have no meta
    const int qt = blockIdx.x / a.heads % a.qtiles;
    if (qt >= load_seq(a, blockIdx.x / (a.heads * a.qtiles), ROWS).qtiles) return;
  }
  const Meta mm = a.meta[blockIdx.x];
  const int n = mm.parts, row0 = mm.row0, rows = mm.rows;
  if (n == 0) return;
  const int d = (threadIdx.x % LANES) * 4, sub = threadIdx.x / LANES;
  auto part = [&](int i, int r) { return a.parts + ((2 * (int64_t)(mm.block + i) + (i == 0 ? mm.slot : 0)) * ROWS + r) * JS; };
  auto store = [&](int r, float4 v, float sum, float mt) {
    const int tok = (row0 + r) / a.rep, hr = row0 + r - tok * a.rep;
    const int64_t orow = (mm.first + tok) * (int64_t)(a.heads * a.rep) + mm.head * a.rep + hr;
    const float inv = inverse(sum);
    uint2 h;
    h.x = pack_h2(v.x * inv, v.y * inv);
    h.y = pack_h2(v.z * inv, v.w * inv);
    *reinterpret_cast<uint2*>(a.out + orow * D + d) = h;
    if (a.lse && d == 0) a.lse[orow] = log_sum(mt, sum);
  };
  // Adds parts i, i + by, ... of row r below n to (v, sum), four loads at a time, and keeps their maximum in mt.
  auto add = [&](int i, int by, int r, float4& v, float& sum, float& mt) {
    for (; i < n; i += 4 * by) {
      float4 x[4];
      float2 ml[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float* p = part(min(i + u * by, n - 1), r);
        x[u] = *reinterpret_cast<const float4*>(p + d);
        ml[u] = *reinterpret_cast<const float2*>(p + D);
        if (i + u * by >= n) ml[u] = make_float2(M_NONE, 0.0f);
      }
      const float top = fmaxf(fmaxf(mt, fmaxf(ml[0].x, ml[1].x)), fmaxf(ml[2].x, ml[3].x));
      const float f0 = ex2(mt - top);
      mt = top;
      v = make_float4(v.x * f0, v.y * f0, v.z * f0, v.w * f0);
      sum *= f0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = i + u * by < n ? ex2(ml[u].x - top) : 0.0f;
        v.x = fmaf(f, x[u].x, v.x);
        v.y = fmaf(f, x[u].y, v.y);
        v.z = fmaf(f, x[u].z, v.z);
        v.w = fmaf(f, x[u].w, v.w);
        sum = fmaf(f, ml[u].y, sum);
      }
    }
  };
  if (gridDim.y == 1) {
    for (int r = sub; r < rows; r += SUBS) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float sum = 0.0f, mt = M_NONE;
      add(0, 1, r, v, sum, mt);
      store(r, v, sum, mt);
    }
    return;
  }
  const int r = blockIdx.y;
  if (r >= rows) return;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float sum = 0.0f, mt = M_NONE;
  add(sub, SUBS, r, v, sum, mt);
  acc[threadIdx.x] = v;
  if (d == 0) sums[sub] = make_float2(mt, sum);
  __syncthreads();
  if (sub == 0) {
    float top = mt;
    for (int i = 1; i < SUBS; ++i) top = fmaxf(top, sums[i].x);
    const float f0 = ex2(mt - top);
    v = make_float4(v.x * f0, v.y * f0, v.z * f0, v.w * f0);
    sum *= f0;
    for (int i = 1; i < SUBS; ++i) {
      const float4 x = acc[threadIdx.x + i * LANES];
      const float f = ex2(sums[i].x - top);
      v.x = fmaf(f, x.x, v.x);
      v.y = fmaf(f, x.y, v.y);
      v.z = fmaf(f, x.z, v.z);
      v.w = fmaf(f, x.w, v.w);
      sum = fmaf(f, sums[i].y, sum);
    }
    store(r, v, sum, top);
  }
}

// Query rows of a block, in tiles of 8: what the longest query needs, at most 32 (16 with D = 256).  A conversion of the
// cache's codes serves all of a block's rows.
inline int row_tiles(int64_t rep, int64_t max_q, int64_t D) {
  const int64_t rows = rep * max_q;
  return rows <= 8 ? 1 : (rows <= 16 || D == 256 ? 2 : 4);
}

// Whether the tiles of all units are dealt out to a grid of resident blocks
// (and joined), or one block takes each unit.
inline bool split(int64_t max_len) { return max_len > DIRECT_LEN; }

// Few units have many parts each: a block of the join takes one row of one, its threads a share of the parts.  That and a
// block for all rows, on sequences of 4k keys with 8 kv heads: one sequence (8 units) 11.7 and 22.5 us, two 11.3 and 16.8,
// four (32 units) 12.9 and 15.2, eight 18.1 and 18.4, sixteen (128 units) 24.3 and 25.7.  Beyond 32 units it would
// still gain 0.3 to 1.5 us (the records hold as many units as the grid has blocks): not taken so far.
constexpr int64_t FEW_UNITS = 32;

inline size_t meta_bytes(size_t grid) { return (grid * sizeof(Meta) + 15) / 16 * 16; }

inline int split_grid(int64_t D, int nt) { return sm_count() * blocks_per_sm((int)D, nt); }

// Programmatic dependent launch: a kernel's blocks come up while the one before it ends, and wait for it.
template <class K>
cudaError_t launch_after(K kern, dim3 grid, int threads, int smem, cudaStream_t stream, const AttnParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int D, int NG, int NT>
cudaError_t launch(const AttnParams& p, const AttnKv4Args& a, cudaStream_t stream) {
  using C = Cfg<D, NG, NT>;
  const int64_t units = a.B * p.qtiles * p.heads;
  if (!split(a.max_len)) {
    if (units > 0x7fffffffLL) return cudaErrorInvalidValue;
    auto kern = attn_kv4_kernel<D, NG, NT, false>;
    cudaError_t e = set_smem_once(kern, C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_after(kern, dim3((unsigned)units), AW * 32, C::SMEM, stream, p);
  }
  auto kern = attn_kv4_kernel<D, NG, NT, true>;
  cudaError_t e = set_smem_once(kern, C::SMEM);
  if (e != cudaSuccess) return e;
  const int grid = split_grid(D, NT);
  e = launch_after(kern, dim3((unsigned)grid), AW * 32, C::SMEM, stream, p);
  if (e != cudaSuccess) return e;
  return launch_after(attn_kv4_join_kernel<D, NT>, p.by_unit ? dim3((unsigned)units, C::ROWS) : dim3((unsigned)grid), 256, 0,
                      stream, p);
}

template <int D, int NG>
cudaError_t launch_nt(const AttnParams& p, const AttnKv4Args& a, cudaStream_t stream) {
  const int nt = row_tiles(p.rep, a.max_q, D);
  if (nt == 1) return launch<D, NG, 1>(p, a, stream);
  if constexpr (D < 256)
    if (nt == 4) return launch<D, NG, 4>(p, a, stream);
  return launch<D, NG, 2>(p, a, stream);
}

}  // namespace

size_t attn_kv4_workspace(int64_t B, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_q, int64_t max_len) {
  if (!split(max_len)) return 0;
  const int nt = row_tiles(q_heads / kv_heads, max_q, D);
  const size_t grid = (size_t)split_grid(D, nt);
  return meta_bytes(grid) + 2 * grid * 8 * nt * (D + 4) * sizeof(float);
}

cudaError_t launch_attn_kv4(const AttnKv4Args& a, cudaStream_t stream) {
  AttnParams p{};
  cudaError_t e = device_status_ptr(&p.status);
  if (e != cudaSuccess) return e;
  p.q = reinterpret_cast<const __half*>(a.q);
  p.ld_q = a.ld_q;
  p.T = a.T;
  p.codes = a.pool.codes;
  p.params = reinterpret_cast<const uint8_t*>(a.pool.params);
  if (a.max_len == 0) {   // nothing is read, but the (empty) copies name an address
    p.codes = reinterpret_cast<const uint8_t*>(a.q);
    p.params = p.codes;
  }
  p.num_pages = a.pool.num_pages;
  p.page_log2 = __builtin_ctz((unsigned)a.pool.page_size);
  p.heads = a.pool.heads;
  p.rep = a.q_heads / a.pool.heads;
  p.table = a.table;
  p.ld_table = a.ld_table;
  p.lens = a.lens;
  p.cu_q = a.cu_q;
  p.B = a.B;
  p.max_q = a.max_q;
  p.max_len = a.max_len;
  p.window = a.window;
  const int rows = 8 * row_tiles(p.rep, a.max_q, a.pool.D);
  p.qtiles = (int)((a.max_q * p.rep + rows - 1) / rows);
  p.scale = a.scale;
  p.out = reinterpret_cast<__half*>(a.out);
  p.lse = a.lse;
  if (split(a.max_len)) {
    const size_t grid = (size_t)split_grid(a.pool.D, rows / 8);
    p.meta = static_cast<Meta*>(a.workspace);
    p.by_unit = a.B * p.qtiles * p.heads <= FEW_UNITS;
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + meta_bytes(grid));
  }
  const int D = a.pool.D, ng = D / a.pool.group;
  if (D == 64) return ng == 1 ? launch_nt<64, 1>(p, a, stream) : launch_nt<64, 2>(p, a, stream);
  if (D == 128) {
    if (ng == 1) return launch_nt<128, 1>(p, a, stream);
    return ng == 2 ? launch_nt<128, 2>(p, a, stream) : launch_nt<128, 4>(p, a, stream);
  }
  return ng == 2 ? launch_nt<256, 2>(p, a, stream) : launch_nt<256, 4>(p, a, stream);
}

}  // namespace bq
