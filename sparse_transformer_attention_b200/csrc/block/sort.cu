// Stable sort of the backward pass's (key, entry) pairs, kv head by kv head:
// least significant digit first, digits of equal width of at most 8 bits
// (two passes up to L = 65535).  A pass counts each tile's digits
// (sort_count), scans every digit's counts over the tiles (sort_scan) and
// places the entries (sort_place), which first orders its tile in shared
// memory so that what it writes is runs of consecutive places: with entries
// written where they stood, 32 lanes hit 32 sectors and a pass of the 8K
// GPT-2-small case took 100 us.
#include "../launch.cuh"
#include "../profile.cuh"
#include "backward.cuh"

namespace ca {
namespace bwd {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSteps = kTile / kThreads;  // entries per thread

__global__ void __launch_bounds__(kThreads)
sort_count(Args a, const uint32_t* key, int shift, uint32_t mask) {
  __shared__ uint32_t cnt[256];
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
__global__ void __launch_bounds__(kThreads) sort_scan(Args a) {
  const int lane = threadIdx.x & 31;
  const int dg = blockIdx.x * kWarps + (threadIdx.x >> 5);
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

// Exclusive scan over the CTA's threads.
__device__ __forceinline__ uint32_t cta_scan(uint32_t v, uint32_t* s_warp) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const uint32_t x = warp_scan(v, lane);
  if (lane == 31) s_warp[wid] = x;
  __syncthreads();
  uint32_t before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < wid) before += s_warp[w];
  __syncthreads();
  return before + x - v;
}

// Places a tile.  Every warp ranks its run of the tile's entries in order
// (equal digits of a step by lane, earlier steps by a running count), the
// warps' counts are chained, and the tile, ordered by digit in shared
// memory, goes out run by run.
__global__ void __launch_bounds__(kThreads, 2)
sort_place(Args a, const uint32_t* key, const uint32_t* ent, uint32_t* key_out,
           uint32_t* ent_out, int shift, uint32_t mask) {
  __shared__ uint16_t cnt[kWarps][256];  // a tile has kTile <= 65535 entries
  __shared__ uint32_t s_key[kTile], s_ent[kTile];
  __shared__ uint32_t s_dst[256];  // global place of the tile's run, less its
                                   // local place
  __shared__ uint32_t s_warp[kWarps];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int64_t base = (int64_t)blockIdx.y * a.w.per_head;
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  const int n = (int)min((int64_t)kTile, a.w.per_head - t0);
  const int l0 = wid * (32 * kSteps);
  for (int c = threadIdx.x; c < kWarps * 256; c += kThreads)
    (&cnt[0][0])[c] = 0;
  uint32_t kv[kSteps], ev[kSteps], rank[kSteps];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int l = l0 + u * 32 + lane;
    kv[u] = l < n ? key[base + t0 + l] : 0u;
    ev[u] = ent && l < n ? ent[base + t0 + l] : (uint32_t)(t0 + l);
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const bool live = l0 + u * 32 + lane < n;
    // lanes behind the tile's end share a digit that no other lane has
    const uint32_t dg = live ? (kv[u] >> shift) & mask : 256u;
    const uint32_t same = __match_any_sync(kAll, dg);
    const uint32_t lower = same & ((1u << lane) - 1u);
    uint32_t before = 0;
    if (live) before = cnt[wid][dg];
    __syncwarp();
    if (live && lower == 0) cnt[wid][dg] = (uint16_t)(before + __popc(same));
    __syncwarp();
    rank[u] = before + __popc(lower);
  }
  __syncthreads();
  {
    const int dg = threadIdx.x;  // one digit per thread of the first 256
    const bool mine = dg < 256;
    const size_t at = (size_t)blockIdx.y * 256 + (mine ? dg : 0);
    uint32_t total = 0;
    if (mine)
#pragma unroll
      for (int w = 0; w < kWarps; ++w) total += cnt[w][dg];
    const uint32_t local = cta_scan(total, s_warp);
    const uint32_t first = cta_scan(mine ? a.totals[at] : 0u, s_warp);
    if (mine) {
      s_dst[dg] = first + a.hist[at * a.w.tiles + blockIdx.x] - local;
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

}  // namespace

cudaError_t sort_launch(const Args& a, int* last, cudaStream_t s) {
  const Work& w = a.w;
  const dim3 grid(w.tiles, w.segs);
  int from = 0;
  for (int p = 0; p < w.passes; ++p) {
    const int shift = p * w.digit;
    const uint32_t mask = (1u << w.digit) - 1u;
    prof_before(s, "sort_count");
    sort_count<<<grid, kThreads, 0, s>>>(a, a.key[from], shift, mask);
    prof_after(s);
    prof_before(s, "sort_scan");
    sort_scan<<<dim3(256 / kWarps, w.segs), kThreads, 0, s>>>(a);
    prof_after(s);
    prof_before(s, "sort_place");
    sort_place<<<grid, kThreads, 0, s>>>(a, a.key[from],
                                         p ? a.ent[from] : nullptr,
                                         a.key[from ^ 1], a.ent[from ^ 1],
                                         shift, mask);
    prof_after(s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    from ^= 1;
  }
  *last = from;
  return cudaSuccess;
}

}  // namespace bwd
}  // namespace ca
