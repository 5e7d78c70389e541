// A token for each row of logits (bq_sample).
//
// A row's weights are w = 2**-y, y = (max - x) / (t ln 2).  Which token u falls
// on is a matter of sums over up to half a million of them, so they are held in
// fixed point, 2**-44 of the largest weight a unit, and summed as integers:
// exactly, in any order.  y is formed in two fp32 parts (max - x and its error,
// times 1 / (t ln 2) and its error) and split as k / 32 + r, |r| <= 1/64:
//   2**-y = 2**-(k / 32) * (1 + d),  d = 2**-r - 1 by its series in fp32,
// with 2**-(j / 32) from a table of 60 bits; d * 2**-(j / 32) is rounded to 2**-28.
// fp32 weights summed in fp32 would put the borders of 50000 about equal tokens
// off by some 1e-7 of the sum each: one choice in a hundred would be another.
//
// The kept tokens are those above a cut, a pair (key of a logit, index among
// equal ones); every filter makes one and the strictest counts.  The cut of
// the first k, or of a prefix of weight p, is found by counts: a pass counts
// the logits by 2048 steps of y, which bounds the weight above every step to
// within a step; the tokens that may be the last kept one, between two steps,
// are gathered and searched in shared memory.  Where there are too many of
// them (thousands of about equal logits) the same is done again by their keys.
//
// A cluster of 1 to 8 blocks takes a row: its sums, counts and gathered tokens are
// exchanged through distributed shared memory, and every block decides for
// itself, on the same numbers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bq_device.cuh"
#include "draft_internal.h"

namespace bq {

namespace {

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int FRAC = 44;                     // bits of a weight below the largest
constexpr float Y_MOST = FRAC + 2.0f;        // from here on a weight is 0
constexpr int BINS = 2048, EACH = BINS / THREADS;
constexpr int LIST = 2048;                   // gathered tokens
constexpr int MOST_BLOCKS = 8;

// Keys of fp32 values: unsigned integers of the same order.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// Kept: logits above `x`, and of those equal to it the indices up to `last`.  (NaN and, with x = -inf, -inf are not.)
struct Cut {
  float x;
  int last;
};
__device__ __forceinline__ bool kept(const Cut& c, float x, int index) {
  return x > c.x || (x == c.x && index <= c.last);
}
constexpr int NONE = -16;                    // below every index, also those before a row that starts off a boundary
__device__ __forceinline__ Cut strictest(const Cut& a, const Cut& b) {
  if (a.x != b.x) return a.x > b.x ? a : b;
  return a.last < b.last ? a : b;
}

// Entries of 2**-(j / 32): 60 bits after the point, and as fp32.
struct Table {
  uint64_t fixed[32];
  float value[32];
};

// What the weights of a row depend on
struct Scale {
  float top, c_hi, c_lo;     // largest logit, 1 / (t ln 2)
};

template <bool WIDE>   // WIDE: logits of 24 bits, whose differences need an error term
__device__ __forceinline__ uint64_t weight(float x, const Scale& s, const Table& t) {
  const float hi = __fsub_rn(s.top, x);
  const float p = __fmul_rn(hi, s.c_hi);
  if (!(p < Y_MOST)) return 0;
  float e = fmaf(hi, s.c_hi, -p);
  e = fmaf(hi, s.c_lo, e);
  if constexpr (WIDE) {
    const float b = __fsub_rn(s.top, hi);                       // what was taken away
    const float lo = __fadd_rn(__fsub_rn(s.top, __fadd_rn(b, hi)), __fsub_rn(b, x));
    e = fmaf(lo, s.c_hi, e);
  }
  constexpr float NEAREST = 393216.0f;                          // 1.5 * 2**18: its ulp is 1 / 32
  const float a = __fadd_rn(p, NEAREST);
  const int k = __float_as_int(a) - __float_as_int(NEAREST);
  const float r = -__fadd_rn(__fsub_rn(p, __fsub_rn(a, NEAREST)), e);
  // (r ln 2)**i / i!
  float d = fmaf(r, 0.0096181291f, 0.055504109f);
  d = fmaf(r, d, 0.24022651f);
  d = fmaf(r, d, 0.69314718f);
  d = __fmul_rn(r, d);
  const int j = k & 31, n = k >> 5;
  constexpr float WHOLE = 12582912.0f;                          // 1.5 * 2**23: its ulp is 1
  const float q = fmaf(__fmul_rn(d, t.value[j]), 268435456.0f, WHOLE);
  const int64_t m = (int64_t)t.fixed[j] + ((int64_t)(__float_as_int(q) - __float_as_int(WHOLE)) << 32);
  return (uint64_t)m >> (60 - FRAC + n);
}

// Shared memory of a block
struct Shared {
  Table table;
  uint64_t part[2][WARPS];         // a warp's share of a sum, two in turn
  uint64_t own[WARPS];             // the same within the block
  uint32_t hist[BINS];
  float list_x[LIST];              // gathered tokens: the block's own, then the row's behind them
  int32_t list_i[LIST];
  union {                          // (the masses of bins are done with before a list is)
    float all_x[LIST];
    uint32_t mass_lo[BINS];
  };
  union {
    int32_t all_i[LIST];
    uint32_t mass_hi[BINS];
  };
  int n;                           // of the block's own
  int found;
  uint64_t reached;
  uint32_t scan[WARPS];
  float scan_lo[WARPS], scan_hi[WARPS];
  int edge[2];
};

__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t a) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// floor(f * n) and ceil(f * n), exactly, for f in [0, 1]
__device__ uint64_t times(float f, uint64_t n, bool up) {
  const uint32_t b = __float_as_uint(f);
  const int e = b >> 23;
  const uint64_t m = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int s = 150 - (e ? e : 1);            // f = m 2**-s, s >= 23
  const uint64_t hi = __umul64hi(m, n), lo = m * n;
  if (s >= 128) return up && (hi | lo) ? 1 : 0;
  const uint64_t q = s >= 64 ? (s == 64 ? hi : hi >> (s - 64)) : (hi << (64 - s)) | (lo >> s);
  const bool rest = s >= 64 ? (lo || (s > 64 && (hi & ((1ull << (s - 64)) - 1)))) : (lo & ((1ull << s) - 1)) != 0;
  return q + (up && rest ? 1 : 0);
}

template <class T>
__device__ __forceinline__ float to_float(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same<T, __half>::value) return __half2float(v);
  else return __bfloat162float(v);
}

// A row, as its cluster's warps share it: consecutive steps of 16 bytes each, on 16-byte boundaries.
template <class T>
struct Row {
  static constexpr int E = 16 / sizeof(T);
  const T* x;              // the row
  const uint4* base;       // the boundary at or before it
  int V, shift;            // elements from there to the row
  int first, last;         // this warp's steps
  int lane;

  __device__ Row(const T* x_, int V_, int warp, int warps, int lane_) : x(x_), V(V_), lane(lane_) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x);
    base = reinterpret_cast<const uint4*>(a & ~uintptr_t(15));
    shift = (int)((a & 15) / sizeof(T));
    const int steps = (V + shift + E - 1) / E, per = (steps + warps - 1) / warps;
    first = min(warp * per, steps);
    last = min(first + per, steps);
  }
  // Elements of step s: index of the first, values (-inf where there is none)
  __device__ __forceinline__ int load(int s, float (&v)[E]) const {
    const int i = s * E - shift;
    if (i >= 0 && i + E <= V) {
      const uint4 w = __ldg(base + s);
      const T* t = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = to_float(t[e]);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = i + e >= 0 && i + e < V ? to_float(x[i + e]) : -INFINITY;
    }
    return i;
  }
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    for (int s = first + lane; s < last; s += 32) {
      float v[E];
      const int i = load(s, v);
#pragma unroll
      for (int e = 0; e < E; ++e) f(v[e], i + e);
    }
  }
};

template <class T>
struct Sampler {
  static constexpr bool WIDE = sizeof(T) == 4;
  // of the keys of 16-bit logits the lowest bits are all equal
  static constexpr int KEY_SHIFT = WIDE ? 0 : (std::is_same<T, __half>::value ? 13 : 16);
  Shared& sh;
  const Row<T>& row;
  const int tid, warp, lane, blocks, rank;
  int phase = 0;
  Scale s;
  float bins;               // steps of y
  Cut cut;                  // what is kept so far

  __device__ Sampler(Shared& sh_, const Row<T>& row_, int blocks_, int rank_)
      : sh(sh_), row(row_), tid(threadIdx.x), warp(threadIdx.x >> 5), lane(threadIdx.x & 31), blocks(blocks_), rank(rank_) {}

  __device__ __forceinline__ void sync() const {
    if (blocks == 1) __syncthreads();
    else cluster_sync_all();
  }
  __device__ __forceinline__ uint32_t remote(const void* p, int block) const { return mapa_shared(smem_u32(p), block); }

  __device__ __forceinline__ uint64_t w_of(float x) const { return weight<WIDE>(x, s, sh.table); }
  __device__ __forceinline__ float y_of(float x) const { return __fmul_rn(__fsub_rn(s.top, x), s.c_hi); }
  __device__ __forceinline__ int bin_of(float y) const {
    constexpr float WHOLE = 8388608.0f;
    return min(__float_as_int(fmaf(y, bins, WHOLE)) - __float_as_int(WHOLE), BINS - 1);
  }

  // Every warp's share of a sum, exchanged: f(share of warp i of the row) for this lane's i.  One barrier; the next
  // exchange may follow at once.
  template <class F>
  __device__ __forceinline__ void exchange(uint64_t mine, F f) {
    if (lane == 0) sh.part[phase][warp] = mine;
    sync();
    for (int i = lane; i < blocks * WARPS; i += 32) {
      const uint64_t* p = &sh.part[phase][i % WARPS];
      f(i, blocks == 1 ? *p : ld_cluster_u64(remote(p, i / WARPS)));
    }
    phase ^= 1;
  }
  __device__ uint64_t row_sum(uint64_t v) {
    uint64_t t = 0;
    exchange(warp_sum(v), [&](int, uint64_t w) { t += w; });
    return warp_sum(t);
  }
  // The sum over the block alone, for numbers that every block has.
  __device__ uint64_t block_sum(uint64_t v) {
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) sh.own[warp] = v;
    __syncthreads();
    return warp_sum(lane < WARPS ? sh.own[lane] : 0);
  }

  // The index of the m-th (from 1) token with logit x, or V
  __device__ int nth(float x, uint64_t m) {
    uint32_t n = 0;
    row.each([&](float v, int) { n += v == x; });
    n = __reduce_add_sync(0xffffffffu, n);
    uint64_t before = 0;
    exchange(n, [&](int i, uint64_t w) { before += i < rank * WARPS + warp ? w : 0; });
    before = warp_sum(before);
    int at = row.V;
    if (before < m && m <= before + n) {
      uint32_t left = (uint32_t)(m - before);
      for (int s0 = row.first; s0 < row.last; s0 += 32) {
        float v[Row<T>::E];
        int i = 0;
        uint32_t c = 0;
        if (s0 + lane < row.last) {
          i = row.load(s0 + lane, v);
#pragma unroll
          for (int e = 0; e < Row<T>::E; ++e) c += v[e] == x;
        }
        uint32_t inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t up = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += up;
        }
        const uint32_t step = __shfl_sync(0xffffffffu, inc, 31);
        if (left <= step) {
          if (c && left <= inc && left > inc - c) {
            uint32_t k = inc - c;
#pragma unroll
            for (int e = 0; e < Row<T>::E; ++e) {
              k += v[e] == x;
              if (v[e] == x && k == left) at = i + e;
            }
          }
          break;
        }
        left -= step;
      }
    }
    at = __reduce_min_sync(0xffffffffu, at);
    exchange((uint64_t)at, [&](int, uint64_t w) { at = min(at, (int)w); });
    return __reduce_min_sync(0xffffffffu, at);
  }

  // The first bin whose tokens, with those before it, may reach `need`, and the first with which they surely do (the last
  // bin where none does), by the cluster's counts; returns the tokens from the one to the other.  A token of bin b is
  // worth low(b) to high(b).
  template <class L, class H>
  __device__ uint32_t find(float need, L low, H high, int& b0, int& b1) {
    sync();
    uint32_t n[EACH], count = 0;
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const uint32_t* p = &sh.hist[tid * EACH + i];
      n[i] = 0;
      for (int b = 0; b < blocks; ++b) n[i] += blocks == 1 ? *p : ld_cluster_u32(remote(p, b));
      count += n[i];
      lo += (float)n[i] * low(tid * EACH + i);
      hi += (float)n[i] * high(tid * EACH + i);
    }
    if (tid == 0) sh.edge[0] = sh.edge[1] = BINS - 1;
    uint32_t ic = count;
    float il = lo, ih = hi;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t uc = __shfl_up_sync(0xffffffffu, ic, o);
      const float ul = __shfl_up_sync(0xffffffffu, il, o), uh = __shfl_up_sync(0xffffffffu, ih, o);
      if (lane >= o) {
        ic += uc;
        il += ul;
        ih += uh;
      }
    }
    if (lane == 31) {
      sh.scan[warp] = ic;
      sh.scan_lo[warp] = il;
      sh.scan_hi[warp] = ih;
    }
    __syncthreads();
    uint32_t bc = ic - count;
    float bl = il - lo, bh = ih - hi;
    for (int w = 0; w < warp; ++w) {
      bc += sh.scan[w];
      bl += sh.scan_lo[w];
      bh += sh.scan_hi[w];
    }
    // (sums of 2048 fp32 terms are off by less than 2**-12 of themselves)
    constexpr float LESS = 1.0f - 1.0f / 4096, MORE = 1.0f + 1.0f / 4096;
    float l = bl, h = bh;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      l += (float)n[i] * low(tid * EACH + i);
      h += (float)n[i] * high(tid * EACH + i);
      if (n[i] && h * MORE >= need) atomicMin(&sh.edge[0], tid * EACH + i);
      if (n[i] && l * LESS >= need) atomicMin(&sh.edge[1], tid * EACH + i);
    }
    __syncthreads();
    b0 = sh.edge[0];
    b1 = sh.edge[1];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      if (tid * EACH + i == b0) sh.scan[0] = bc;
      bc += n[i];
      if (tid * EACH + i == b1) sh.scan[1] = bc;
    }
    __syncthreads();
    return sh.scan[1] - sh.scan[0];
  }

  __device__ void clear() {
    sync();                                  // (the others are done with the last counts)
    for (int i = tid; i < BINS; i += THREADS) sh.hist[i] = sh.mass_lo[i] = sh.mass_hi[i] = 0;
    if (tid == 0) sh.n = 0;
    __syncthreads();
  }

  // The cut below which nothing is kept: the shortest prefix of what `cut` keeps that has `need` tokens (MASS false), or
  // a weight of `need` or more.  There are that many, and their counts by steps of y are in hist.
  template <bool MASS>
  __device__ Cut descend(uint64_t need) {
    int b0, b1;
    const float step = 1.0f / bins;          // (bins is 0 where all are equal: then there is one bin, of weight 1)
    auto bound = [&](float y) { return bins > 0.0f ? exp2f(FRAC - fmaxf(y, 0.0f) * step) : exp2f(FRAC); };
    uint32_t n = find((float)need, [&](int b) { return MASS ? bound(b + 0.51f) : 1.0f; },
                      [&](int b) { return MASS ? bound(b - 0.51f) : 1.0f; }, b0, b1);
    // what lies between the edges, and above them
    auto inside = [&](float x, int i, bool& over) {
      over = false;
      if (!kept(cut, x, i)) return false;
      const float y = y_of(x);
      if (!(y < Y_MOST)) return false;
      const int b = bin_of(y);
      over = b < b0;
      return b >= b0 && b <= b1;
    };
    if (n <= LIST) return search<MASS>(need, inside);
    uint64_t above = 0;
    uint32_t lowest = 0xffffffffu, highest = 0;
    row.each([&](float x, int i) {
      bool over;
      if (inside(x, i, over)) {
        const uint32_t k = key_of(x + 0.0f);
        lowest = min(lowest, k);
        highest = max(highest, k);
      }
      if (over) above += MASS ? w_of(x) : 1;
    });
    above = row_sum(above);
    lowest = __reduce_min_sync(0xffffffffu, lowest);
    highest = __reduce_max_sync(0xffffffffu, highest);
    exchange((uint64_t)lowest << 32 | (0xffffffffu - highest), [&](int, uint64_t w) {
      lowest = min(lowest, (uint32_t)(w >> 32));
      highest = max(highest, 0xffffffffu - (uint32_t)w);
    });
    uint32_t k0 = __reduce_min_sync(0xffffffffu, lowest), k1 = __reduce_max_sync(0xffffffffu, highest);
    // by keys: exact sums of 2048 ranges of them, of which one holds the last kept token; at most three times
    for (;;) {
      const int bits = 32 - __clz((k1 - k0) | 1), shift = bits > 11 ? bits - 11 : 0;
      clear();
      row.each([&](float x, int i) {
        if (!kept(cut, x, i)) return;
        const uint32_t k = key_of(x + 0.0f);
        if (k < k0 || k > k1) return;
        const int b = (k1 - k) >> shift;
        atomicAdd(&sh.hist[b], 1);
        if (MASS) {
          const uint64_t w = w_of(x);
          const uint32_t low = (uint32_t)w, was = atomicAdd(&sh.mass_lo[b], low);
          atomicAdd(&sh.mass_hi[b], (uint32_t)(w >> 32) + (was + low < was ? 1 : 0));
        }
      });
      const int b = find_exact<MASS>(need - above, above, n);
      const uint32_t top_key = k1 - ((uint32_t)b << shift);
      if (shift == 0) return equal<MASS>(value_of(top_key), need - above, n);
      const uint32_t width = (1u << shift) - 1;
      k0 = width < top_key - k0 ? top_key - width : k0;
      k1 = top_key;
      if (n <= LIST)
        return search<MASS>(need, [&](float x, int i, bool& over) {
          over = false;
          if (!kept(cut, x, i)) return false;
          const uint32_t k = key_of(x + 0.0f);
          over = k > k1;
          return k >= k0 && k <= k1;
        });
    }
  }

  // The bin whose tokens reach `need`, by exact sums; what lies above it is added to `above`, n is its number of tokens.
  template <bool MASS>
  __device__ int find_exact(uint64_t need, uint64_t& above, uint32_t& n) {
    sync();
    uint32_t count[EACH];
    uint64_t v[EACH], sum = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int b = tid * EACH + i;
      count[i] = 0;
      v[i] = 0;
      for (int j = 0; j < blocks; ++j) {
        count[i] += ld_cluster_u32(remote(&sh.hist[b], j));
        if (MASS)
          v[i] += (uint64_t)ld_cluster_u32(remote(&sh.mass_hi[b], j)) << 32 | ld_cluster_u32(remote(&sh.mass_lo[b], j));
      }
      if (!MASS) v[i] = count[i];
      sum += v[i];
    }
    uint64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    __syncthreads();
    if (lane == 31) sh.own[warp] = inc;
    __syncthreads();
    uint64_t before = inc - sum;
    for (int w = 0; w < warp; ++w) before += sh.own[w];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      if (before < need && need <= before + v[i]) {
        sh.edge[0] = tid * EACH + i;
        sh.scan[0] = count[i];
        sh.reached = before;
      }
      before += v[i];
    }
    __syncthreads();
    above += sh.reached;
    n = sh.scan[0];
    return sh.edge[0];
  }

  // Of n equal tokens the last kept one
  template <bool MASS>
  __device__ Cut equal(float x, uint64_t need, uint32_t n) {
    uint64_t m = need;
    if (MASS) {
      const uint64_t w = w_of(x);
      m = w ? (need + w - 1) / w : n;
    }
    // (a cut at this very logit keeps fewer of them already)
    return Cut{x, m >= n ? (cut.x == x ? cut.last : row.V) : nth(x, m)};
  }

  // The cut where its token is among at most LIST ones: `inside` tells which, and which others lie above them.
  template <bool MASS, class F>
  __device__ Cut search(uint64_t need, F inside) {
    uint64_t above = 0;
    row.each([&](float x, int i) {
      bool over;
      if (inside(x, i, over)) {
        const int at = atomicAdd(&sh.n, 1);
        if (at < LIST) {
          sh.list_x[at] = x + 0.0f;
          sh.list_i[at] = i;
        }
      }
      if (over) above += MASS ? w_of(x) : 1;
    });
    need -= row_sum(above);
    // every block takes the whole list
    sync();
    int n = 0;
    for (int b = 0; b < blocks; ++b) {
      const int have = blocks == 1 ? sh.n : (int)ld_cluster_u32(remote(&sh.n, b));
      for (int i = tid; i < have && n + i < LIST; i += THREADS) {
        sh.all_x[n + i] = blocks == 1 ? sh.list_x[i] : __uint_as_float(ld_cluster_u32(remote(&sh.list_x[i], b)));
        sh.all_i[n + i] = blocks == 1 ? sh.list_i[i] : (int)ld_cluster_u32(remote(&sh.list_i[i], b));
      }
      n = min(n + have, LIST);
    }
    __syncthreads();
    constexpr int PER = LIST / THREADS;
    uint32_t key[PER], lo = 0xffffffffu, hi = 0;
    uint64_t w[PER];
    int index[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = tid + j * THREADS;
      const float x = i < n ? sh.all_x[i] : -INFINITY;
      index[j] = i < n ? sh.all_i[i] : -1;
      key[j] = i < n ? key_of(x) >> KEY_SHIFT : 0;
      w[j] = i < n ? (MASS ? w_of(x) : 1) : 0;
      if (i < n) {
        lo = min(lo, key[j]);
        hi = max(hi, key[j]);
      }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) sh.own[warp] = (uint64_t)lo << 32 | hi;
    __syncthreads();
    {
      const uint64_t v = lane < WARPS ? sh.own[lane] : 0xffffffff00000000ull;
      lo = __reduce_min_sync(0xffffffffu, (uint32_t)(v >> 32));
      hi = __reduce_max_sync(0xffffffffu, (uint32_t)v);
    }
    // the lowest key with less than `need` above it
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2;
      uint64_t t = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) t += key[j] > mid ? w[j] : 0;
      if (block_sum(t) < need) hi = mid;
      else lo = mid + 1;
    }
    uint64_t t = 0, one = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      t += key[j] > lo ? w[j] : 0;
      one += index[j] >= 0 && key[j] == lo;
    }
    const uint64_t left = need - block_sum(t);
    const uint64_t ties = block_sum(one);
    // of its tokens the first m, by index
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (index[j] >= 0 && key[j] == lo) {
        sh.found = tid + j * THREADS;        // (any of them: they are equal)
      }
    __syncthreads();
    const float x = sh.all_x[sh.found];
    uint64_t m = left;
    if (MASS) {
      const uint64_t each = w_of(x);
      m = each ? (left + each - 1) / each : ties;
    }
    if (m >= ties) return Cut{x, cut.x == x ? cut.last : row.V};
    int i0 = 0, i1 = row.V - 1;
    while (i0 < i1) {
      const int mid = (i0 + i1) / 2;
      uint64_t c = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) c += index[j] >= 0 && key[j] == lo && index[j] <= mid;
      if (block_sum(c) >= m) i1 = mid;
      else i0 = mid + 1;
    }
    return Cut{x, i0};
  }
};

template <class T>
__global__ void __launch_bounds__(THREADS, 2) sample_kernel(const SampleArgs a, int blocks) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blocks == 1 ? 0 : (int)cluster_ctarank();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t r = blockIdx.x / blocks;
  const int V = (int)a.V;
  const Row<T> row(static_cast<const T*>(a.logits) + r * a.ld, V, rank * WARPS + warp, blocks * WARPS, lane);
  if (tid < 32) {
    const double v = exp2(-tid / 32.0);
    sh.table.fixed[tid] = (uint64_t)(v * 1152921504606846976.0);     // 2**60
    sh.table.value[tid] = (float)v;
  }
  for (int i = tid; i < BINS; i += THREADS) sh.hist[i] = 0;
  if (tid == 0) sh.n = 0;

  Sampler<T> p(sh, row, blocks, rank);
  // ---- the largest and the smallest logit ----
  float top = -INFINITY, least = INFINITY;
  row.each([&](float x, int) {
    top = fmaxf(top, x);
    least = fminf(least, x > -INFINITY ? x : INFINITY);
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
  }
  p.exchange((uint64_t)__float_as_uint(top) << 32 | __float_as_uint(least), [&](int, uint64_t w) {
    top = fmaxf(top, __uint_as_float((uint32_t)(w >> 32)));
    least = fminf(least, __uint_as_float((uint32_t)w));
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
  }
  top += 0.0f;                               // (-0 is 0)
  const float heat = a.temperature ? a.temperature[r] : 1.0f;
  if (top == -INFINITY || !(heat > 0.0f) || top == INFINITY) {
    // nothing to take, or the largest
    const int at = top == -INFINITY ? -1 : p.nth(top, 1);
    if (rank == 0 && tid == 0) {
      a.tokens[r] = at;
      if (a.logprob) a.logprob[r] = at < 0 ? -INFINITY : 0.0f;
    }
    p.sync();
    return;
  }
  const double c = fmin(1.4426950408889634 / (double)heat, 1e30);
  p.s.top = top;
  p.s.c_hi = (float)c;
  p.s.c_lo = (float)(c - (double)p.s.c_hi);
  p.cut = Cut{-INFINITY, NONE};
  const float range = fminf(p.y_of(least), Y_MOST);
  p.bins = range > 1e-30f ? (BINS - 1) / range : 0.0f;

  const int k = a.top_k ? a.top_k[r] : 0;
  if (k > 0 && k < V) {
    uint64_t n = 0;
    __syncthreads();
    row.each([&](float x, int) {
      const float y = p.y_of(x);
      if (y < Y_MOST) {
        atomicAdd(&sh.hist[p.bin_of(y)], 1);
        ++n;
      }
    });
    n = p.row_sum(n);
    if (n > (uint64_t)k) p.cut = p.template descend<false>(k);
    p.clear();
  }
  const float share = a.top_p ? a.top_p[r] : 1.0f;
  if (share <= 0.0f) {
    p.cut = Cut{top, p.nth(top, 1)};
  } else if (share < 1.0f) {
    uint64_t w = 0;
    __syncthreads();
    row.each([&](float x, int i) {
      if (!kept(p.cut, x, i)) return;
      const float y = p.y_of(x);
      if (!(y < Y_MOST)) return;
      atomicAdd(&sh.hist[p.bin_of(y)], 1);
      w += p.w_of(x);
    });
    w = p.row_sum(w);
    p.cut = strictest(p.cut, p.template descend<true>(times(share, w, true)));
  }
  const float m = a.min_p ? a.min_p[r] : 0.0f;
  if (m > 1.0f) {
    p.cut = strictest(p.cut, Cut{top, p.nth(top, 1)});
  } else if (m > 0.0f) {
    // w >= m where x >= max + t ln m
    const float x = __double2float_ru((double)top + (double)heat * log((double)m));
    p.cut = strictest(p.cut, Cut{fminf(x, top), x > -INFINITY ? V : NONE});
  }

  // ---- kept weights by warp, and the one that u falls on ----
  uint64_t mine = 0;
  row.each([&](float x, int i) {
    if (kept(p.cut, x, i)) mine += p.w_of(x);
  });
  mine = warp_sum(mine);
  uint64_t before = 0, total = 0;
  p.exchange(mine, [&](int i, uint64_t w) {
    before += i < rank * WARPS + warp ? w : 0;
    total += w;
  });
  before = warp_sum(before);
  total = warp_sum(total);
  const float u = a.u[r];
  uint64_t at = !(u > 0.0f) ? 0 : (u < 1.0f ? times(u, total, false) : total - 1);
  if (at >= before && at < before + mine) {
    at -= before;
    for (int s0 = row.first; s0 < row.last; s0 += 32) {
      constexpr int E = Row<T>::E;
      float v[E];
      int i = 0;
      uint64_t w = 0;
      if (s0 + lane < row.last) {
        i = row.load(s0 + lane, v);
#pragma unroll
        for (int e = 0; e < E; ++e) w += kept(p.cut, v[e], i + e) ? p.w_of(v[e]) : 0;
      }
      uint64_t sum = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      const uint64_t step = __shfl_sync(0xffffffffu, sum, 31);
      if (at < step) {
        if (at < sum && at >= sum - w) {
          uint64_t run = sum - w;
          bool done = false;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            run += kept(p.cut, v[e], i + e) ? p.w_of(v[e]) : 0;
            if (!done && at < run) {
              done = true;
              a.tokens[r] = i + e;
              if (a.logprob)
                a.logprob[r] = (float)(-((double)top - (double)v[e]) / (double)heat -
                                       log((double)total / (double)(1ull << FRAC)));
            }
          }
        }
        break;
      }
      at -= step;
    }
  }
  p.sync();                                  // (the others may still read this block's shared memory)
}

// Blocks that share a row: as many as keep the GPU busy (two blocks an SM), each with 4096 logits or more.
inline int row_blocks(int64_t R, int64_t V) {
  int blocks = 1;
  while (blocks < MOST_BLOCKS && R * blocks * 2 <= 2 * sm_count() && V >= blocks * 2 * 4096) blocks *= 2;
  return blocks;
}

template <class T>
cudaError_t launch(const SampleArgs& a, cudaStream_t stream) {
  const int blocks = row_blocks(a.R, a.V);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.R * blocks));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = blocks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, blocks);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t stream) {
  if (a.ltype == BQ_LOGITS_F32) return launch<float>(a, stream);
  return a.ltype == BQ_LOGITS_F16 ? launch<__half>(a, stream) : launch<__nv_bfloat16>(a, stream);
}

}  // namespace bq
