// Stable sort of the backward pass's (key, entry) pairs, kv head by kv head:
// least significant digit first, digits of equal width of at most 8 bits
// (two passes up to L = 65535).  A pass counts each tile's digits
// (sort_count), scans every digit's counts over the tiles (sort_scan) and
// places the entries (sort_place), which first orders its tile in shared
// memory so that what it writes is runs of consecutive places: with entries
// written where they stood, 32 lanes hit 32 sectors and placing 6.5 M entries
// took 118 us where it took 49.  Lists of one tile or a few (up to kSmall
// entries) are sorted by one CTA each in shared memory, in one launch
// instead of six (8704 entries: 18 us instead of 40).
#include "../launch.cuh"
#include "backward.cuh"

namespace ca {
namespace bwd {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSteps = kTile / kThreads;  // entries per thread

constexpr int kSmallThreads = 1024;
constexpr int kSmallSteps = 16;
constexpr int kSmall = kSmallThreads * kSmallSteps;
constexpr int kSmallDigit = 9;  // bits of a digit at most
// two buffers of keys and 16-bit entry numbers, each warp's digit counts
constexpr size_t kSmallSmem =
    (size_t)kSmall * 12 +
    (size_t)(kSmallThreads / 32) * (1 << kSmallDigit) * 2;
static_assert(kSmall <= 65536, "places and entries fit 16 bits");
static_assert(kSmallSmem <= 232448 - 1024, "fits an SM");

__global__ void __launch_bounds__(kThreads)
sort_count(Args a, const uint32_t* key, int shift, uint32_t mask) {
  __shared__ uint32_t cnt[256];
  chain();
  const int64_t base = (int64_t)blockIdx.y * a.w.per_head;
  const int64_t e0 = (int64_t)blockIdx.x * kTile;
  const int n = (int)min((int64_t)kTile, a.w.per_head - e0);
  if (threadIdx.x < 256) cnt[threadIdx.x] = 0;
  uint32_t kv[kSteps];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int t = u * kThreads + threadIdx.x;
    kv[u] = t < n ? key[base + e0 + t] : 0u;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kSteps; ++u)
    if (u * kThreads + threadIdx.x < n)
      atomicAdd(&cnt[(kv[u] >> shift) & mask], 1u);
  __syncthreads();
  if (threadIdx.x < 256)
    a.hist[((size_t)blockIdx.y * 256 + threadIdx.x) * a.w.tiles + blockIdx.x] =
        cnt[threadIdx.x];
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t x, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(kAll, x, off);
    if (lane >= off) x += y;
  }
  return x;  // inclusive
}

// One warp per (kv head, digit): exclusive scan of its counts over the tiles.
__global__ void __launch_bounds__(256) sort_scan(Args a) {
  chain();
  const int lane = threadIdx.x & 31;
  const int dg = blockIdx.x * 8 + (threadIdx.x >> 5);
  const size_t at = (size_t)blockIdx.y * 256 + dg;
  uint32_t* h = a.hist + at * a.w.tiles;
  uint32_t sum = 0;
  for (int c0 = 0; c0 < a.w.tiles; c0 += 32) {
    const int c = c0 + lane;
    const uint32_t v = c < a.w.tiles ? h[c] : 0u;
    const uint32_t x = warp_scan(v, lane);
    if (c < a.w.tiles) h[c] = sum + x - v;
    sum += __shfl_sync(kAll, x, 31);
  }
  if (lane == 0) a.totals[at] = sum;
}

// Exclusive scan over the CTA's first 32 * W threads (the others pass 0).
template <int W>
__device__ __forceinline__ uint32_t cta_scan(uint32_t v, uint32_t* s_warp) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const uint32_t x = warp_scan(v, lane);
  if (lane == 31 && wid < W) s_warp[wid] = x;
  __syncthreads();
  uint32_t before = 0;
#pragma unroll
  for (int w = 0; w < W; ++w)
    if (w < wid) before += s_warp[w];
  __syncthreads();
  return before + x - v;
}

// The lanes of the warp with this lane's digit (one vote per digit bit; a
// vote takes a few cycles where match.any takes one round per value).
__device__ __forceinline__ uint32_t peers(uint32_t dg, int bits) {
  uint32_t same = kAll;
#pragma unroll
  for (int i = 0; i < kSmallDigit; ++i) {
    if (i < bits) {
      const uint32_t set = __ballot_sync(kAll, (dg >> i) & 1u);
      same &= ((dg >> i) & 1u) ? set : ~set;
    }
  }
  return same;
}

// The rank of this lane's entry among a warp's entries of its digit: equal
// digits of the step by lane, earlier steps by the running counts cnt.
// Entries behind the end (!in) are the last lanes.
__device__ __forceinline__ uint32_t rank_step(uint32_t dg, bool in, int bits,
                                              uint16_t* cnt) {
  const int lane = threadIdx.x & 31;
  const uint32_t same = peers(dg, bits) & __ballot_sync(kAll, in);
  const uint32_t lower = same & ((1u << lane) - 1u);
  uint32_t before = 0;
  if (in) before = cnt[dg];
  __syncwarp();
  if (in && lower == 0) cnt[dg] = (uint16_t)(before + __popc(same));
  __syncwarp();
  return before + __popc(lower);
}

// The same with the lanes of each digit collected in shared memory, seen[]
// (zero before and after), instead of by a vote per digit bit: 39 instead of
// 47 us for 6.5 M entries.
__device__ __forceinline__ uint32_t rank_seen(uint32_t dg, bool in,
                                              uint32_t* seen, uint16_t* cnt) {
  const int lane = threadIdx.x & 31;
  if (in) atomicOr(seen + dg, 1u << lane);
  __syncwarp();
  const uint32_t same = seen[dg];
  const uint32_t before = cnt[dg];
  const uint32_t lower = same & ((1u << lane) - 1u);
  __syncwarp();
  if (in && lower == 0) {
    cnt[dg] = (uint16_t)(before + __popc(same));
    seen[dg] = 0;
  }
  __syncwarp();
  return before + __popc(lower);
}

// Places a tile: the warps' runs are ranked, their counts chained, and the
// tile, ordered by digit in shared memory, goes out run by run.  Bound by
// shared memory (79% of its cycles), two fifths of that bank conflicts of
// scattered words; three CTAs per SM spill registers and take 44 us.
__global__ void __launch_bounds__(kThreads, 2)
sort_place(Args a, const uint32_t* key, const uint32_t* ent, uint32_t* key_out,
           uint32_t* ent_out, int shift, uint32_t mask) {
  __shared__ uint16_t cnt[kWarps][256];  // a tile has kTile <= 65535 entries
  __shared__ uint32_t s_key[kTile], s_ent[kTile];
  __shared__ uint32_t s_dst[256];  // global place of the tile's run, less its
                                   // local place
  __shared__ uint32_t s_warp[8];
  chain();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int64_t base = (int64_t)blockIdx.y * a.w.per_head;
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  const int n = (int)min((int64_t)kTile, a.w.per_head - t0);
  const int l0 = wid * (32 * kSteps);
  uint32_t kv[kSteps], ev[kSteps], rank[kSteps];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int l = l0 + u * 32 + lane;
    kv[u] = l < n ? key[base + t0 + l] : 0u;
    ev[u] = ent && l < n ? ent[base + t0 + l] : (uint32_t)(t0 + l);
  }
  const int dg = threadIdx.x;  // one digit per thread of the first 256
  const bool mine = dg < 256;
  const size_t at_dg = (size_t)blockIdx.y * 256 + (mine ? dg : 0);
  const uint32_t all = mine ? a.totals[at_dg] : 0u;
  const uint32_t prior = a.hist[at_dg * a.w.tiles + blockIdx.x];
  // the digits' lanes lie in s_key, which is not needed before they are done
  static_assert(kWarps * 256 <= kTile, "they fit");
  for (int c = threadIdx.x; c < kWarps * 256; c += kThreads) {
    (&cnt[0][0])[c] = 0;
    s_key[c] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kSteps; ++u)
    rank[u] = rank_seen((kv[u] >> shift) & mask, l0 + u * 32 + lane < n,
                        s_key + wid * 256, cnt[wid]);
  __syncthreads();
  {
    uint32_t total = 0;
    if (mine)
#pragma unroll
      for (int w = 0; w < kWarps; ++w) total += cnt[w][dg];
    const uint32_t local = cta_scan<8>(total, s_warp);
    const uint32_t first = cta_scan<8>(all, s_warp);
    if (mine) {
      s_dst[dg] = first + prior - local;
      uint32_t x = local;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const uint32_t c = cnt[w][dg];
        cnt[w][dg] = (uint16_t)x;
        x += c;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    if (l0 + u * 32 + lane < n) {
      const uint32_t at = cnt[wid][(kv[u] >> shift) & mask] + rank[u];
      if (in_bounds(at < kTile, a.status)) {
        s_key[at] = kv[u];
        s_ent[at] = ev[u];
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int l = u * kThreads + threadIdx.x;
    if (l < n) {
      const uint32_t kk = s_key[l];
      const uint32_t at = s_dst[(kk >> shift) & mask] + (uint32_t)l;
      if (in_bounds(at < a.w.per_head, a.status)) {
        key_out[base + at] = kk;
        ent_out[base + at] = s_ent[l];
      }
    }
  }
}

// All passes over one kv head's list, one CTA, the list in shared memory.
__global__ void __launch_bounds__(kSmallThreads)
sort_small(Args a, const uint32_t* key, uint32_t* key_out, uint32_t* ent_out,
           int passes, int digit) {
  constexpr int kW = kSmallThreads / 32, kDigits = 1 << kSmallDigit;
  extern __shared__ __align__(16) unsigned char g_smem[];
  __shared__ uint32_t s_warp[kDigits / 32];
  chain();
  uint32_t* s_key = reinterpret_cast<uint32_t*>(g_smem);  // [2][kSmall]
  uint16_t* s_ent = reinterpret_cast<uint16_t*>(s_key + 2 * kSmall);
  uint16_t(*cnt)[kDigits] =
      reinterpret_cast<uint16_t(*)[kDigits]>(s_ent + 2 * kSmall);
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int64_t base = (int64_t)blockIdx.x * a.w.per_head;
  const int n = (int)a.w.per_head;
  // a warp's run: as many steps as the list needs
  const int steps = (n + kSmallThreads - 1) / kSmallThreads;
  const int l0 = wid * 32 * steps;
  const uint32_t mask = (1u << digit) - 1u;
  for (int l = threadIdx.x; l < n; l += kSmallThreads) {
    s_key[l] = key[base + l];
    s_ent[l] = (uint16_t)l;
  }
  for (int p = 0; p < passes; ++p) {
    const int shift = p * digit;
    const uint32_t* from = s_key + (p & 1) * kSmall;
    const uint16_t* efrom = s_ent + (p & 1) * kSmall;
    uint32_t* to = s_key + (p & 1 ^ 1) * kSmall;
    uint16_t* eto = s_ent + (p & 1 ^ 1) * kSmall;
    for (int c = threadIdx.x; c < kW * kDigits / 2; c += kSmallThreads)
      reinterpret_cast<uint32_t*>(&cnt[0][0])[c] = 0;
    __syncthreads();
    uint16_t rank[kSmallSteps];
#pragma unroll
    for (int u = 0; u < kSmallSteps; ++u) {
      if (u >= steps) break;
      const int l = l0 + u * 32 + lane;
      rank[u] = (uint16_t)rank_step(l < n ? (from[l] >> shift) & mask : 0u,
                                    l < n, digit, cnt[wid]);
    }
    __syncthreads();
    // a digit's entries in each warp's run, chained over the warps
    const int dg = threadIdx.x;
    uint32_t c[kW], total = 0;
    if (dg < kDigits) {
#pragma unroll
      for (int w = 0; w < kW; ++w) c[w] = cnt[w][dg];
#pragma unroll
      for (int w = 0; w < kW; ++w) total += c[w];
    }
    uint32_t x = cta_scan<kDigits / 32>(total, s_warp);
    if (dg < kDigits) {
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        cnt[w][dg] = (uint16_t)x;
        x += c[w];
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kSmallSteps; ++u) {
      if (u >= steps) break;
      const int l = l0 + u * 32 + lane;
      if (l < n) {
        const uint32_t kv = from[l];
        const uint32_t at = cnt[wid][(kv >> shift) & mask] + (uint32_t)rank[u];
        if (in_bounds(at < (uint32_t)kSmall, a.status)) {
          to[at] = kv;
          eto[at] = efrom[l];
        }
      }
    }
    __syncthreads();
  }
  const int last = passes & 1;
  for (int l = threadIdx.x; l < n; l += kSmallThreads) {
    key_out[base + l] = s_key[last * kSmall + l];
    ent_out[base + l] = s_ent[last * kSmall + l];
  }
}

}  // namespace

cudaError_t sort_launch(const Args& a, int* last, cudaStream_t s) {
  const Work& w = a.w;
  if (w.per_head <= kSmall) {
    const cudaError_t e = ensure_smem(sort_small, kSmallSmem);
    if (e != cudaSuccess) return e;
    *last = 1;
    const int passes = (w.bits + kSmallDigit - 1) / kSmallDigit;
    return launch("sort_small", sort_small, dim3(w.segs), kSmallThreads,
                  kSmallSmem, s, a, a.key[0], a.key[1], a.ent[1], passes,
                  (w.bits + passes - 1) / passes);
  }
  const dim3 grid(w.tiles, w.segs);
  int from = 0;
  for (int p = 0; p < w.passes; ++p) {
    const int shift = p * w.digit;
    const uint32_t mask = (1u << w.digit) - 1u;
    const uint32_t* ent = p ? a.ent[from] : nullptr;
    cudaError_t e = launch("sort_count", sort_count, grid, kThreads, 0, s, a,
                           a.key[from], shift, mask);
    if (e == cudaSuccess)
      e = launch("sort_scan", sort_scan, dim3(32, w.segs), 256, 0, s, a);
    if (e == cudaSuccess)
      e = launch("sort_place", sort_place, grid, kThreads, 0, s, a,
                 a.key[from], ent, a.key[from ^ 1], a.ent[from ^ 1], shift,
                 mask);
    if (e != cudaSuccess) return e;
    from ^= 1;
  }
  *last = from;
  return cudaSuccess;
}

}  // namespace bwd
}  // namespace ca
