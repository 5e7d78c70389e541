// Acceptance of a branch of drafted tokens (bq_kv4_accept).
//
// Every node's parent is the last bit before its own, so whether its token is
// the one chosen there needs no walk: one bit a node, gathered by ballots, and
// a node is confirmed when its bits are among those bits.  The confirmed node
// with most bits is a maximum over one word, and its bits, counted from
// below, are the path.
//
// The lines of a (layer, key or value, head) move within its rows of pages
// alone, each to a place not behind its own: a warp reads some of them in
// order, then writes them, so that what it overwrites has been read.
//
// What bounds it: latency (loads of the tree, of tokens, of targets at
// parents, of pages, of lines, one behind the other); the lines themselves are
// a few MB.  64 trees of 64 nodes in the caches of 32 layers take 11 us (0.8 TB/s of lines),
// 13 trees in 7 layers 7.5, which is the host's part of a call.
#include "bq_device.cuh"
#include "draft_internal.h"
#include "kv4_device.cuh"

namespace bq {

namespace {

constexpr int THREADS = 256;
constexpr int MAX_NODES = 1024;

struct Params {
  AcceptArgs a;
  int page_log2, groups;
  int64_t items, per;      // (layer, key or value, head) of all layers; of a block
  int* status;
};

__global__ void __launch_bounds__(THREADS) kv4_accept_kernel(const Params p) {
  __shared__ uint32_t ok[MAX_NODES / 32];       // nodes that are roots or have the token chosen at their parent
  __shared__ int best;
  __shared__ int32_t path[MAX_NODES], from[MAX_NODES], to[MAX_NODES];
  const AcceptArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t b = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int64_t first = b * a.each, n = a.each;
  if (a.cu_q) {
    first = a.cu_q[b];
    n = (int64_t)a.cu_q[b + 1] - first;
  }
  const int64_t len = a.lens[b];
  if (n < 0 || first < 0 || first + n > a.T || n > a.max_q || len < n || len > a.max_len) {
    if (tid == 0) record_error(p.status, BQ_ERR_INVALID_ARG);
    n = 0;
  }
  const int64_t base = len - n;
  if (tid == 0) best = -1;

  // bit words of node i, without the bits above its own
  auto bits = [&](int i, int w) -> uint64_t {
    const uint64_t v = __ldg(a.tree + (first + i) * a.words + w);
    return w < (i >> 6) ? v : (w > (i >> 6) ? 0 : v & (~0ull >> (63 - (i & 63))));
  };
  const int rounds = (int)((n + THREADS - 1) / THREADS);
  for (int r = 0; r < rounds; ++r) {
    const int i = r * THREADS + tid;
    bool good = false;
    if (i < n) {
      int parent = -1;
      for (int w = i >> 6; w >= 0 && parent < 0; --w) {
        uint64_t v = bits(i, w);
        if (w == (i >> 6)) v &= ~(1ull << (i & 63));
        if (v) parent = 64 * w + 63 - __clzll(v);
      }
      good = parent < 0 || a.tokens[first + i] == a.targets[first + parent];
    }
    const uint32_t vote = __ballot_sync(0xffffffffu, good);
    if (lane == 0) ok[i >> 5] = vote;
  }
  __syncthreads();
  for (int r = 0; r < rounds; ++r) {
    const int i = r * THREADS + tid;
    if (i >= n) break;
    int count = 0;
    bool good = true, own = false;
    for (int w = 0; w <= i >> 6; ++w) {
      const uint64_t v = bits(i, w);
      const uint64_t k = (uint64_t)ok[2 * w] | (uint64_t)ok[2 * w + 1] << 32;
      good = good && (v & ~k) == 0;
      count += __popcll(v);
      if (w == i >> 6) own = (v >> (i & 63)) & 1;
    }
    if (own && good) atomicMax(&best, count << 10 | (MAX_NODES - 1 - i));
  }
  __syncthreads();
  const int end = best < 0 ? -1 : MAX_NODES - 1 - (best & (MAX_NODES - 1)), count = best < 0 ? 0 : best >> 10;
  // the path, and its lines' places in the pool (-1: not moved)
  for (int i = tid; i <= end; i += THREADS) {
    const uint64_t v = bits(end, i >> 6);
    if (!((v >> (i & 63)) & 1)) continue;
    int k = __popcll(v & ((1ull << (i & 63)) - 1));
    for (int w = 0; w < i >> 6; ++w) k += __popcll(bits(end, w));
    path[k] = i;
    int32_t at[2] = {-1, -1};
    if (k != i && p.items > 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t pos = base + (e ? k : i);
        const int64_t page = a.table[b * a.ld_table + (pos >> p.page_log2)];
        if (page >= 0 && page < a.pool.num_pages)
          at[e] = (int32_t)((page << p.page_log2) + (pos & (a.pool.page_size - 1)));
        else
          record_error(p.status, BQ_ERR_INVALID_ARG);
      }
    }
    from[k] = at[1] < 0 ? -1 : at[0];
    to[k] = at[1];
  }
  __syncthreads();
  if (blockIdx.y == 0) {
    for (int64_t k = tid; k < a.max_q; k += THREADS) a.path[b * a.max_q + k] = k < count ? path[k] : -1;
    if (tid == 0) {
      a.accepted[b] = count;
      a.next[b] = end < 0 ? -1 : a.targets[first + end];
      a.new_lens[b] = (int32_t)(base + count);
    }
  }
  int start = 0;
  while (start < count && from[start] < 0) ++start;     // (a branch often begins with the first nodes)
  if (start == count) return;

  // ---- lines: 16-byte pieces of codes, then the params ----
  const int R = a.pool.D / 2, pieces = R / 16, units = pieces + 1, PR = 4 * p.groups;
  const int64_t page_rows = (int64_t)2 * a.pool.heads << p.page_log2;     // rows of a page
  const int64_t layer_rows = a.pool.num_pages * page_rows;
  const int64_t i0 = blockIdx.y * p.per, i1 = min(i0 + p.per, p.items);
  const int lines = 32 / units;                          // of a warp's step
  const int line = lane / units, unit = lane % units;
  for (int64_t item = i0 + warp; item < i1; item += THREADS / 32) {
    const int64_t layer = item / (2 * a.pool.heads), sub = item % (2 * a.pool.heads);
    for (int k0 = start; k0 < count; k0 += lines) {
      const int k = k0 + line;
      const bool live = line < lines && k < count && from[k] >= 0;
      uint4 v = make_uint4(0, 0, 0, 0);
      auto row = [&](int32_t slot) {
        return layer * layer_rows + (slot >> p.page_log2) * page_rows + (sub << p.page_log2) +
               (slot & (a.pool.page_size - 1));
      };
      if (live) {
        const int64_t r = row(from[k]);
        if (unit < pieces) {
          v = *reinterpret_cast<const uint4*>(a.pool.codes + r * R + unit * 16);
        } else {
          const uint32_t* s = reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(a.pool.params) + r * PR);
          v.x = s[0];
          if (p.groups > 1) v.y = s[1];
          if (p.groups > 2) {
            v.z = s[2];
            v.w = s[3];
          }
        }
      }
      __syncwarp();
      if (live) {
        const int64_t r = row(to[k]);
        if (unit < pieces) {
          *reinterpret_cast<uint4*>(a.pool.codes + r * R + unit * 16) = v;
        } else {
          uint32_t* d = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(a.pool.params) + r * PR);
          d[0] = v.x;
          if (p.groups > 1) d[1] = v.y;
          if (p.groups > 2) {
            d[2] = v.z;
            d[3] = v.w;
          }
        }
      }
      __syncwarp();
    }
  }
}

}  // namespace

cudaError_t launch_kv4_accept(const AcceptArgs& a, cudaStream_t stream) {
  Params p{};
  cudaError_t e = device_status_ptr(&p.status);
  if (e != cudaSuccess) return e;
  p.a = a;
  p.page_log2 = __builtin_ctz((unsigned)a.pool.page_size);
  p.groups = a.pool.D / a.pool.group;
  p.items = a.pool.num_pages > 0 ? a.layers * 2 * a.pool.heads : 0;
  // blocks of at least one item a warp, some 8 of them an SM
  const int64_t warps = THREADS / 32, most = (p.items + warps - 1) / warps;
  int64_t split = (8 * sm_count() + a.B - 1) / a.B;
  split = split < most ? split : most;
  if (split < 1) split = 1;
  if (split > 65535) split = 65535;
  p.per = (p.items + split - 1) / split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.B, (unsigned)split);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_accept_kernel, p);
}

}  // namespace bq
