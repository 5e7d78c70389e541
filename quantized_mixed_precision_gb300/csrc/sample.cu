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
// equal ones); every filter makes one and the strictest counts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bq_device.cuh"
#include "draft_internal.h"

namespace bq {

namespace {

constexpr int THREADS = 1024, WARPS = THREADS / 32;
constexpr int FRAC = 44;                     // bits of a weight below the largest

// Keys of fp32 values: unsigned integers of the same order.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t KEY_LOWEST = 0x007fffffu;   // of -inf: never kept

// Kept: keys above `key`, and of that key the indices up to `last`.
struct Cut {
  uint32_t key;
  int last;
};
__device__ __forceinline__ bool kept(const Cut& c, uint32_t key, int index) {
  return key > c.key || (key == c.key && index <= c.last);
}
__device__ __forceinline__ Cut strictest(const Cut& a, const Cut& b) {
  if (a.key != b.key) return a.key > b.key ? a : b;
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
  if (!(p < FRAC + 2.0f)) return 0;
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

template <class T>
__device__ __forceinline__ float load_logit(const T* p) {
  float x;
  if constexpr (sizeof(T) == 4) x = *p;
  else if constexpr (std::is_same<T, __half>::value) x = __half2float(*p);
  else x = __bfloat162float(*p);
  return x == x ? x + 0.0f : -INFINITY;      // NaN is never taken; -0 is 0
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The sum over the block, for every thread.
__device__ uint64_t block_sum(uint64_t v, uint64_t* share) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) share[threadIdx.x >> 5] = v;
  __syncthreads();
  uint64_t s = 0;
  for (int w = 0; w < WARPS; ++w) s += share[w];
  return s;
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
__global__ void __launch_bounds__(THREADS) sample_kernel(const SampleArgs a) {
  __shared__ Table table;
  __shared__ uint64_t share[WARPS + 1];
  __shared__ uint32_t ends[WARPS];
  __shared__ int found;
  constexpr bool WIDE = sizeof(T) == 4;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.logits) + row * a.ld;
  const int V = (int)a.V;
  // a warp's share of the row: whole steps of 32
  const int each = (V + THREADS - 1) / THREADS * 32;
  const int lo = min(warp * each, V), hi = min(lo + each, V);
  if (tid < 32) {
    const double v = exp2(-tid / 32.0);
    table.fixed[tid] = (uint64_t)(v * 1152921504606846976.0);     // 2**60
    table.value[tid] = (float)v;
  }

  // ---- the largest logit ----
  uint32_t top = 0;
  for (int i = lo + lane; i < hi; i += 32) top = max(top, key_of(load_logit(x + i)));
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) ends[warp] = top;
  __syncthreads();
  top = 0;
  for (int w = 0; w < WARPS; ++w) top = max(top, ends[w]);

  float heat = a.temperature ? a.temperature[row] : 1.0f;
  const bool greedy = !(heat > 0.0f) || value_of(top) == INFINITY;
  if (top <= KEY_LOWEST) {                   // nothing to take
    if (tid == 0) {
      a.tokens[row] = -1;
      if (a.logprob) a.logprob[row] = -INFINITY;
    }
    return;
  }
  Scale s;
  s.top = value_of(top);
  const double c = fmin(1.4426950408889634 / (double)heat, 1e30);
  s.c_hi = (float)c;
  s.c_lo = (float)(c - (double)s.c_hi);

  // the number of keys above one, and the sum of their weights, of what a cut keeps
  auto count_above = [&](uint32_t key, const Cut& cut) {
    uint64_t n = 0;
    for (int i = lo + lane; i < hi; i += 32) {
      const uint32_t k = key_of(load_logit(x + i));
      n += k > key && kept(cut, k, i);
    }
    return block_sum(n, share);
  };
  auto weight_above = [&](uint32_t key, const Cut& cut) {
    uint64_t n = 0;
    for (int i = lo + lane; i < hi; i += 32) {
      const float v = load_logit(x + i);
      const uint32_t k = key_of(v);
      if (k > key && kept(cut, k, i)) n += weight<WIDE>(v, s, table);
    }
    return block_sum(n, share);
  };
  // the index of the m-th (from 1) token of a key, or V
  auto nth = [&](uint32_t key, uint64_t m) -> int {
    uint32_t n = 0;
    for (int i = lo + lane; i < hi; i += 32) n += key_of(load_logit(x + i)) == key;
    n = __reduce_add_sync(0xffffffffu, n);
    __syncthreads();
    if (lane == 0) ends[warp] = n;
    if (tid == 0) found = V;
    __syncthreads();
    uint64_t before = 0;
    for (int w = 0; w < warp; ++w) before += ends[w];
    if (before < m && m <= before + n) {
      for (int i = lo; i < hi; i += 32) {
        const bool is = i + lane < hi && key_of(load_logit(x + i + lane)) == key;
        const uint32_t vote = __ballot_sync(0xffffffffu, is);
        const int c = __popc(vote);
        if (before + c >= m) {
          if (is && __popc(vote & ((2u << lane) - 1)) == (int)(m - before)) found = i + lane;
          break;
        }
        before += c;
      }
    }
    __syncthreads();
    return found;
  };

  Cut cut{KEY_LOWEST, -1};
  if (greedy) {
    cut = Cut{top, nth(top, 1)};
  } else {
    const int k = a.top_k ? a.top_k[row] : 0;
    if (k > 0 && k < V && count_above(KEY_LOWEST, cut) > (uint64_t)k) {
      // the lowest key with fewer than k above it, and of its tokens what is left of k
      uint32_t from = KEY_LOWEST + 1, to = top;
      while (from < to) {
        const uint32_t mid = from + (to - from) / 2;
        if (count_above(mid, cut) < (uint64_t)k) to = mid;
        else from = mid + 1;
      }
      const uint64_t above = count_above(from, cut);
      cut = Cut{from, nth(from, k - above)};
    }
    const float p = a.top_p ? a.top_p[row] : 1.0f;
    Cut tail = cut;
    if (p <= 0.0f) {
      tail = Cut{top, nth(top, 1)};
    } else if (p < 1.0f) {
      const uint64_t need = times(p, weight_above(KEY_LOWEST, cut), true);
      uint32_t from = KEY_LOWEST + 1, to = top;
      while (from < to) {
        const uint32_t mid = from + (to - from) / 2;
        if (weight_above(mid, cut) < need) to = mid;
        else from = mid + 1;
      }
      const uint64_t above = weight_above(from, cut);
      const uint64_t w = weight<WIDE>(value_of(from), s, table);
      tail = Cut{from, w == 0 ? V : nth(from, (need - above + w - 1) / w)};
    }
    cut = strictest(cut, tail);
    const float m = a.min_p ? a.min_p[row] : 0.0f;
    if (m > 1.0f) {
      cut = Cut{top, nth(top, 1)};
    } else if (m > 0.0f) {
      // w >= m where x >= max + t ln m
      const float least = __double2float_ru((double)s.top + (double)heat * log((double)m));
      cut = strictest(cut, Cut{min(key_of(least + 0.0f), top), V});
    }
  }

  // ---- kept weights by warp, and the one that u falls on ----
  uint64_t mine = 0;
  for (int i = lo + lane; i < hi; i += 32) {
    const float v = load_logit(x + i);
    if (kept(cut, key_of(v), i)) mine += greedy ? 1 : weight<WIDE>(v, s, table);
  }
  mine = warp_sum(mine);
  __syncthreads();
  if (lane == 0) share[warp] = mine;
  __syncthreads();
  uint64_t before = 0, total = 0;
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += share[w];
    total += share[w];
  }
  const float u = a.u[row];
  uint64_t at = !(u > 0.0f) ? 0 : (u < 1.0f ? times(u, total, false) : total - 1);
  if (at < before || at >= before + mine) return;
  at -= before;
  for (int i = lo; i < hi; i += 32) {
    const float v = i + lane < hi ? load_logit(x + i + lane) : -INFINITY;
    uint64_t w = 0;
    if (kept(cut, key_of(v), i + lane)) w = greedy ? 1 : weight<WIDE>(v, s, table);
    uint64_t sum = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    const uint64_t step = __shfl_sync(0xffffffffu, sum, 31);
    if (at < step) {
      if (at < sum && at >= sum - w) {
        a.tokens[row] = i + lane;
        if (a.logprob)
          a.logprob[row] = greedy ? 0.0f
                                  : (float)(-((double)s.top - (double)v) / (double)heat -
                                            log((double)total / (double)(1ull << FRAC)));
      }
      break;
    }
    at -= step;
  }
}

template <class T>
cudaError_t launch(const SampleArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.R);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t stream) {
  if (a.ltype == BQ_LOGITS_F32) return launch<float>(a, stream);
  return a.ltype == BQ_LOGITS_F16 ? launch<__half>(a, stream) : launch<__nv_bfloat16>(a, stream);
}

}  // namespace bq
