// Backward pass of the Condensate prefill: gradients of the softmax over
// C_i = {0} U [i-W_i+1, i] U Top-k_i with respect to Q, K and V, the
// selected positions being constants ("Condensate Theorem" page 1 §2.1
// Definition 1, §5.2.2).  The probabilities are computed again from Q, K and
// the sets:
//
//   t_ij = q_i . k_j / sqrt(d)     p_ij = exp(t_ij) / sum_C_i exp(t)
//   dP_ij = dO_i . v_j             D_i = sum_j p_ij dP_ij
//   dS_ij = p_ij (dP_ij - D_i) / sqrt(d)
//   dQ_i = sum_j dS_ij k_j,  dK_j = sum_i dS_ij q_i,  dV_j = sum_i p_ij dO_i
//
// dQ follows the rows, dK and dV the columns.  A column's window rows are a
// band next to its diagonal; its other rows, those that list it in their
// Top-k (and, for key 0, as their anchor), lie anywhere.  So the row pass
// writes p and dS of each listed slot, the slots are sorted by key (stable,
// so a key's rows stay in ascending order), a pass over the sorted slots
// sums each key's listed part, and the column pass adds its window part.  No
// sum depends on timing: every order of addition is fixed by the inputs.
#include "../launch.cuh"
#include "../profile.cuh"
#include "block.cuh"

namespace ca {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------- workspace
// Entry e of a kv head: (q-head of its group, query row, slot), slot 0 the
// anchor (when it lies outside the window), slots 1..k the Top-k positions
// in the order of idx; unused slots hold key L, which sorts behind all keys.
constexpr int kTile = 4096;   // entries per CTA of the sort
constexpr int kRange = 128;   // sorted entries per warp of the listed pass

struct Work {
  int64_t rows;      // B * Hq * nq
  int64_t per_head;  // entries of one kv head: G * nq * (k + 1)
  int segs;          // B * Hkv
  int tiles;         // sort tiles per segment
  int ranges;        // listed-pass ranges per segment
  int bits, passes;  // key bits; sort passes
  size_t wmax, stats, pds, key[2], ent[2], hist, span, top, carry, total;
};

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

bool plan(Work& w, int B, int nq, int L, int Hq, int Hkv, int d, int k) {
  w.rows = (int64_t)B * Hq * nq;
  w.segs = B * Hkv;
  const int64_t per = (int64_t)(Hq / Hkv) * nq * (k + 1);
  if (per > 0x7FFFFF00ll || (int64_t)L >= 0x7FFFFF00ll ||
      (int64_t)B * Hkv > 65535)
    return false;
  w.per_head = per;
  w.tiles = (int)((per + kTile - 1) / kTile);
  w.ranges = (int)((per + kRange - 1) / kRange);
  w.bits = 1;
  while (((int64_t)1 << w.bits) <= L) ++w.bits;  // keys 0..L
  w.passes = (w.bits + 7) / 8;
  const size_t n = (size_t)w.segs * per;
  size_t at = kStatusBytes;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += round256(bytes);
    return a;
  };
  w.wmax = take((size_t)B * 4);
  w.stats = take((size_t)w.rows * 8);
  w.pds = take(n * 8);
  for (int i = 0; i < 2; ++i) {
    w.key[i] = take(n * 4);
    w.ent[i] = take(n * 4);
  }
  w.hist = take((size_t)w.segs * 256 * w.tiles * 4);
  w.span = take((size_t)w.segs * L * 8);
  w.top = take((size_t)w.segs * L * 2 * d * 4);
  w.carry = take((size_t)w.segs * w.ranges * 2 * d * 4);
  w.total = at;
  return true;
}

struct Args : BackwardArgs {
  Work w;
  int* wmax;       // [B] largest window of each batch row (W_i given)
  float2* stats;   // [B, Hq, nq] log2-domain log-sum-exp, D
  float2* pds;     // [entries] p, dS
  uint32_t* key[2];
  uint32_t* ent[2];
  uint32_t* hist;  // [segs, 256, tiles]
  int2* span;      // [segs, L] first and behind-last sorted entry of a key
  float* top;      // [segs, L, 2, d] listed part of dK and dV
  float* carry;    // [segs, ranges, 2, d] a range's share of the key that
                   // began in an earlier range
};

// The window of query row r of head h: [lo, i].
__device__ __forceinline__ int window_lo(const Args& a, int b, int h, int r,
                                         bool report, int* w) {
  *w = row_window(a.W_i, (int64_t)b * a.nq + r, a.W_h, h, a.W, a.L, a.status,
                  report);
  const int lo = a.p0 + r - *w + 1;
  return lo > 0 ? lo : 0;
}

// Top-k entries of a row's index list: |C_i| less the anchor and the window.
// A count that does not fit the window, k or C_max raises kErrCmax.
__device__ __forceinline__ int listed_count(const Args& a, int64_t row, int i,
                                            int lo, int w, bool report) {
  const int c = __ldg(a.idx_count + row);
  if (lo == 0) {
    if (c != i + 1 && report) raise_flag(a.status, kErrCmax);
    return 0;
  }
  int m = c - 1 - w;
  const int most = min(a.k, a.C_max - 1);
  if (m < 0 || m > most) {
    if (report) raise_flag(a.status, kErrCmax);
    m = m < 0 ? 0 : most;
  }
  return m;
}

__global__ void backward_window_max(Args a) {
  const int b = blockIdx.y;
  const int r = blockIdx.x * blockDim.x + threadIdx.x;
  int w = r < a.nq ? min(max(a.W_i[(int64_t)b * a.nq + r], 1), a.L) : 1;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    w = max(w, __shfl_xor_sync(kAll, w, off));
  if ((threadIdx.x & 31) == 0) atomicMax(a.wmax + b, w);
}

// ---------------------------------------------------------------- row pass
// One warp per query row; eight lanes per key, four keys at a time.  One
// sweep over the set with a running maximum m and, behind it, the sums
//   l = sum e,  E = sum e dP,  A = sum e dP k,  Bk = sum e k   (e = 2^(x-m))
// so that D = E / l and dQ = (A - D Bk) / l without a second reading.
template <typename T, typename TD, int D>
struct RowState {
  static constexpr int DL = D / 8;
  float m = -INFINITY, l = 0.f, E = 0.f, A[DL], Bk[DL];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < DL; ++e) A[e] = Bk[e] = 0.f;
  }
  __device__ __forceinline__ void scale(float f) {
    l *= f;
    E *= f;
#pragma unroll
    for (int e = 0; e < DL; ++e) {
      A[e] *= f;
      Bk[e] *= f;
    }
  }
  __device__ __forceinline__ void add(float x, float dp, const float* kf) {
    if (x > m) {
      scale(exp2f(m - x));
      m = x;
    }
    const float e = exp2f(x - m);
    l += e;
    E = fmaf(e, dp, E);
#pragma unroll
    for (int c = 0; c < DL; ++c) {
      A[c] = fmaf(e * dp, kf[c], A[c]);
      Bk[c] = fmaf(e, kf[c], Bk[c]);
    }
  }
};

constexpr int kRowWarps = 8;

template <typename T, typename TD, int D>
__global__ void __launch_bounds__(kRowWarps * 32) backward_rows(Args a) {
  constexpr int DL = D / 8;
  extern __shared__ __align__(16) unsigned char g_smem[];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int sub = lane & 7, grp = lane >> 3;
  float2* s_x = reinterpret_cast<float2*>(g_smem) + wid * (a.k + 1);
  const int64_t row = (int64_t)blockIdx.x * kRowWarps + wid;
  if (row >= a.w.rows) return;  // the whole warp; no barrier follows
  const int r = (int)(row % a.nq);
  const int bh = (int)(row / a.nq);
  const int b = bh / a.Hq, h = bh % a.Hq;
  const int seg = b * a.Hkv + h / (a.Hq / a.Hkv);
  const int i = a.p0 + r;
  const T* K = reinterpret_cast<const T*>(a.K) + (int64_t)seg * a.L * D + sub * DL;
  const T* V = reinterpret_cast<const T*>(a.V) + (int64_t)seg * a.L * D + sub * DL;
  float q[DL], g[DL];
  load_row<T, DL>(reinterpret_cast<const T*>(a.Q) + row * D + sub * DL, q);
  load_row<TD, DL>(reinterpret_cast<const TD*>(a.dO) + row * D + sub * DL, g);
  const float sl2 = kLog2e / sqrtf((float)D), sc = 1.f / sqrtf((float)D);
  int w;
  const int lo = window_lo(a, b, h, r, lane == 0, &w);
  const int m_top = listed_count(a, row, i, lo, w, lane == 0);
  const int ns = lo > 0 ? 1 + m_top : 0;  // used slots
  const int32_t* ix = a.idx + row * a.C_max;
  uint32_t* key = a.key[0] + row * (a.k + 1);

  RowState<T, TD, D> st;
  st.clear();
  // slots, then window keys, four at a time
  const int nw = i - lo + 1;
#pragma unroll 1
  for (int t0 = 0; t0 < ns + nw; t0 += 4) {
    const int t = t0 + grp;
    bool act = t < ns + nw;
    int j = 0;
    if (act) {
      if (t >= ns) {
        j = lo + t - ns;
      } else if (t > 0) {
        j = __ldg(ix + t);
        if (j < 1 || j > i - w) {  // not a candidate of this row
          if (sub == 0) raise_flag(a.status, kErrCmax);
          act = false;
          j = 0;
        }
      }
      if (t < ns && sub == 0) key[t] = act ? (uint32_t)j : (uint32_t)a.L;
    }
    float kf[DL], vf[DL];
    load_row<T, DL>(K + (int64_t)j * D, kf);
    load_row<T, DL>(V + (int64_t)j * D, vf);
    float x = 0.f, dp = 0.f;
#pragma unroll
    for (int c = 0; c < DL; ++c) {
      x = fmaf(q[c], kf[c], x);
      dp = fmaf(g[c], vf[c], dp);
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) {
      x += __shfl_xor_sync(kAll, x, off);
      dp += __shfl_xor_sync(kAll, dp, off);
    }
    x *= sl2;
    if (t < ns && sub == 0) s_x[t] = make_float2(act ? x : -INFINITY, dp);
    if (act) st.add(x, dp, kf);
  }
  // the four groups' states, merged
#pragma unroll
  for (int off = 8; off <= 16; off <<= 1) {
    const float mo = __shfl_xor_sync(kAll, st.m, off);
    const float mn = fmaxf(st.m, mo);
    st.scale(st.m == -INFINITY ? 0.f : exp2f(st.m - mn));
    st.m = mn;
    st.l += __shfl_xor_sync(kAll, st.l, off);
    st.E += __shfl_xor_sync(kAll, st.E, off);
#pragma unroll
    for (int c = 0; c < DL; ++c) {
      st.A[c] += __shfl_xor_sync(kAll, st.A[c], off);
      st.Bk[c] += __shfl_xor_sync(kAll, st.Bk[c], off);
    }
  }
  const float inv = 1.f / st.l, Di = st.E * inv;
  if (lane == 0) a.stats[row] = make_float2(st.m + log2f(st.l), Di);
  if (grp == 0) {
    float dq[DL];
#pragma unroll
    for (int c = 0; c < DL; ++c)
      dq[c] = (st.A[c] - Di * st.Bk[c]) * inv * sc;
    store_row<T, DL>(reinterpret_cast<T*>(a.dQ) + row * D + sub * DL, dq);
  }
  __syncwarp();
  for (int t = lane; t <= a.k; t += 32) {
    float2 o = make_float2(0.f, 0.f);
    if (t < ns) {
      const float2 xd = s_x[t];
      o.x = xd.x == -INFINITY ? 0.f : exp2f(xd.x - st.m) * inv;
      o.y = o.x * (xd.y - Di) * sc;
    } else {
      key[t] = (uint32_t)a.L;
    }
    a.pds[row * (a.k + 1) + t] = o;
  }
}

// -------------------------------------------------------------------- sort
// Stable least-significant-digit sort of each kv head's entries by key.
// A CTA counts (sort_count) or places (sort_place) a tile of kTile entries;
// counts are laid out digit-major so that one exclusive scan per kv head
// (sort_scan) gives each (digit, tile) its first place.
constexpr int kSortThreads = 256;

__global__ void __launch_bounds__(kSortThreads)
sort_count(Args a, const uint32_t* key, int shift) {
  __shared__ uint32_t cnt[256];
  const int64_t base = (int64_t)blockIdx.y * a.w.per_head;
  const int64_t e0 = (int64_t)blockIdx.x * kTile;
  const int n = (int)min((int64_t)kTile, a.w.per_head - e0);
  cnt[threadIdx.x] = 0;
  __syncthreads();
  for (int t = threadIdx.x; t < n; t += kSortThreads)
    atomicAdd(&cnt[(key[base + e0 + t] >> shift) & 255u], 1u);
  __syncthreads();
  a.hist[((size_t)blockIdx.y * 256 + threadIdx.x) * a.w.tiles + blockIdx.x] =
      cnt[threadIdx.x];
}

__global__ void __launch_bounds__(1024) sort_scan(Args a) {
  __shared__ uint32_t s_warp[32];
  __shared__ uint32_t s_carry;
  const int n = 256 * a.w.tiles;
  uint32_t* h = a.hist + (size_t)blockIdx.x * n;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  if (threadIdx.x == 0) s_carry = 0;
  __syncthreads();
  for (int c0 = 0; c0 < n; c0 += 1024) {
    const int c = c0 + threadIdx.x;
    const uint32_t v = c < n ? h[c] : 0u;
    uint32_t x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) s_warp[wid] = x;
    __syncthreads();
    if (wid == 0) {
      uint32_t y = s_warp[lane];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t z = __shfl_up_sync(kAll, y, off);
        if (lane >= off) y += z;
      }
      s_warp[lane] = y;
    }
    __syncthreads();
    const uint32_t before = s_carry + (wid ? s_warp[wid - 1] : 0u);
    if (c < n) h[c] = before + x - v;
    __syncthreads();
    if (threadIdx.x == 0) s_carry += s_warp[31];
    __syncthreads();
  }
}

// Places a tile: every warp ranks its run of the tile's entries in order
// (equal digits of a step by lane, earlier steps by a running count), then
// the warps' counts are chained and each entry goes to its place.
__global__ void __launch_bounds__(kSortThreads)
sort_place(Args a, const uint32_t* key, const uint32_t* ent, uint32_t* key_out,
           uint32_t* ent_out, int shift) {
  constexpr int kW = kSortThreads / 32;
  constexpr int kSteps = kTile / kSortThreads;  // steps of 32 per warp
  __shared__ uint32_t cnt[kW][256];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int64_t base = (int64_t)blockIdx.y * a.w.per_head;
  const int64_t e0 = (int64_t)blockIdx.x * kTile + wid * (32 * kSteps);
  for (int c = threadIdx.x; c < kW * 256; c += kSortThreads)
    (&cnt[0][0])[c] = 0;
  __syncthreads();
  uint32_t kv[kSteps], rank[kSteps];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int64_t e = e0 + u * 32 + lane;
    kv[u] = e < a.w.per_head ? key[base + e] : 0xFFFFFFFFu;
  }
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const bool live = e0 + u * 32 + lane < a.w.per_head;
    // dead lanes are a tail of the last steps: a digit of their own
    const uint32_t dg = live ? (kv[u] >> shift) & 255u : 256u;
    const uint32_t same = __match_any_sync(kAll, dg);
    const uint32_t lower = same & ((1u << lane) - 1u);
    uint32_t before = 0;
    if (live) before = cnt[wid][dg];
    __syncwarp();
    if (live && lower == 0) cnt[wid][dg] = before + __popc(same);
    __syncwarp();
    rank[u] = before + __popc(lower);
  }
  __syncthreads();
  {
    const int dg = threadIdx.x;  // kSortThreads = 256 digits
    uint32_t at =
        a.hist[((size_t)blockIdx.y * 256 + dg) * a.w.tiles + blockIdx.x];
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      const uint32_t c = cnt[w][dg];
      cnt[w][dg] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int64_t e = e0 + u * 32 + lane;
    if (e < a.w.per_head) {
      const uint32_t at = cnt[wid][(kv[u] >> shift) & 255u] + rank[u];
      if (in_bounds(at < a.w.per_head, a.status)) {
        key_out[base + at] = kv[u];
        ent_out[base + at] = ent ? ent[base + e] : (uint32_t)e;
      }
    }
  }
}

// ------------------------------------------------- listed part of dK and dV
// A warp sums kRange consecutive sorted entries, one key after the other, so
// that the work is even however many rows list a key.  A key's sum goes to
// `top` if it began in this range, else (the range's head) to `carry`.
template <typename T, typename TD, int D>
__global__ void __launch_bounds__(256) backward_listed(Args a,
                                                       const uint32_t* keys,
                                                       const uint32_t* ents) {
  constexpr int DL = D / 32;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int seg = blockIdx.y;
  const int range = blockIdx.x * 8 + wid;
  if (range >= a.w.ranges) return;
  const int64_t base = (int64_t)seg * a.w.per_head;
  const int64_t x0 = (int64_t)range * kRange;
  const int64_t x1 = min(x0 + kRange, a.w.per_head);
  const T* Q = reinterpret_cast<const T*>(a.Q) + lane * DL;
  const TD* dO = reinterpret_cast<const TD*>(a.dO) + lane * DL;
  const int64_t row0 = (int64_t)seg * (a.Hq / a.Hkv) * a.nq;
  const float2* pds = a.pds + base;
  const uint32_t L = (uint32_t)a.L;
  uint32_t cur = x0 > 0 ? keys[base + x0 - 1] : 0xFFFFFFFFu;
  bool head = x0 > 0;  // the sum so far belongs to a key begun earlier
  float dk[DL], dv[DL];
#pragma unroll
  for (int c = 0; c < DL; ++c) dk[c] = dv[c] = 0.f;
  auto flush = [&]() {
    float* o = nullptr;
    if (head)
      o = a.carry + ((int64_t)seg * a.w.ranges + range) * 2 * D;
    else if (cur < L)
      o = a.top + ((int64_t)seg * L + cur) * 2 * D;
    if (!o) return;
#pragma unroll
    for (int c = 0; c < DL; ++c) {
      o[lane * DL + c] = dk[c];
      o[D + lane * DL + c] = dv[c];
    }
  };
  for (int64_t x = x0; x < x1; ++x) {
    const uint32_t kj = keys[base + x];
    if (kj != cur) {
      if (x > x0 || head) flush();
      head = false;
      if (lane == 0) {
        if (x > 0 && cur < L) a.span[(int64_t)seg * L + cur].y = (int)x;
        if (kj < L) a.span[(int64_t)seg * L + kj].x = (int)x;
      }
      cur = kj;
#pragma unroll
      for (int c = 0; c < DL; ++c) dk[c] = dv[c] = 0.f;
    }
    if (kj >= L) break;  // unused slots: nothing follows
    const uint32_t e = ents[base + x];
    const float2 pd = pds[e];
    const int64_t row = row0 + e / (uint32_t)(a.k + 1);
    float q[DL], g[DL];
    load_f32<T, DL>(Q + row * D, q);
    load_f32<TD, DL>(dO + row * D, g);
#pragma unroll
    for (int c = 0; c < DL; ++c) {
      dk[c] = fmaf(pd.y, q[c], dk[c]);
      dv[c] = fmaf(pd.x, g[c], dv[c]);
    }
  }
  if (cur < L || head) flush();
  if (x1 == a.w.per_head && cur < L && lane == 0)
    a.span[(int64_t)seg * L + cur].y = (int)x1;
}

// ------------------------------------------------------------- column pass
// One warp per key: its window rows, eight lanes per row, four rows at a
// time, then the listed part.
template <typename T, typename TD, int D>
__global__ void __launch_bounds__(256) backward_columns(Args a) {
  constexpr int DL = D / 8;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int sub = lane & 7, grp = lane >> 3;
  const int64_t col = (int64_t)blockIdx.x * 8 + wid;
  if (col >= (int64_t)a.w.segs * a.L) return;
  const int j = (int)(col % a.L), seg = (int)(col / a.L);
  const int b = seg / a.Hkv, g = seg % a.Hkv, G = a.Hq / a.Hkv;
  const float sl2 = kLog2e / sqrtf((float)D), sc = 1.f / sqrtf((float)D);
  float kf[DL], vf[DL], dk[DL], dv[DL];
  load_row<T, DL>(reinterpret_cast<const T*>(a.K) + col * D + sub * DL, kf);
  load_row<T, DL>(reinterpret_cast<const T*>(a.V) + col * D + sub * DL, vf);
#pragma unroll
  for (int c = 0; c < DL; ++c) dk[c] = dv[c] = 0.f;
  for (int hh = 0; hh < G; ++hh) {
    const int h = g * G + hh;
    int wm = a.W_i ? a.wmax[b] : (a.W_h ? a.W_h[h] : a.W);
    wm = min(max(wm, 1), a.L);
    // rows whose position i has i - wm + 1 <= j <= i
    const int r0 = max(j - a.p0, 0);
    const int r1 = (int)min((int64_t)j + wm - 1 - a.p0, (int64_t)a.nq - 1);
    const int64_t rowbase = ((int64_t)b * a.Hq + h) * a.nq;
    for (int rr = r0; rr <= r1; rr += 4) {
      const int r = min(rr + grp, r1);
      int w;
      bool act = rr + grp <= r1 && window_lo(a, b, h, r, false, &w) <= j;
      float qf[DL], of[DL];
      load_row<T, DL>(reinterpret_cast<const T*>(a.Q) + (rowbase + r) * D + sub * DL, qf);
      load_row<TD, DL>(reinterpret_cast<const TD*>(a.dO) + (rowbase + r) * D + sub * DL, of);
      const float2 st = a.stats[rowbase + r];
      float x = 0.f, dp = 0.f;
#pragma unroll
      for (int c = 0; c < DL; ++c) {
        x = fmaf(qf[c], kf[c], x);
        dp = fmaf(of[c], vf[c], dp);
      }
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) {
        x += __shfl_xor_sync(kAll, x, off);
        dp += __shfl_xor_sync(kAll, dp, off);
      }
      const float p = act ? exp2f(x * sl2 - st.x) : 0.f;
      const float ds = p * (dp - st.y) * sc;
#pragma unroll
      for (int c = 0; c < DL; ++c) {
        dk[c] = fmaf(ds, qf[c], dk[c]);
        dv[c] = fmaf(p, of[c], dv[c]);
      }
    }
  }
#pragma unroll
  for (int off = 8; off <= 16; off <<= 1)
#pragma unroll
    for (int c = 0; c < DL; ++c) {
      dk[c] += __shfl_xor_sync(kAll, dk[c], off);
      dv[c] += __shfl_xor_sync(kAll, dv[c], off);
    }
  if (grp != 0) return;
  const int2 sp = a.span[col];
  if (sp.y > sp.x) {
    const float* t = a.top + col * 2 * D + sub * DL;
#pragma unroll
    for (int c = 0; c < DL; ++c) {
      dk[c] += t[c];
      dv[c] += t[D + c];
    }
    for (int r = sp.x / kRange + 1; r <= (sp.y - 1) / kRange; ++r) {
      const float* cr = a.carry + ((int64_t)seg * a.w.ranges + r) * 2 * D + sub * DL;
#pragma unroll
      for (int c = 0; c < DL; ++c) {
        dk[c] += cr[c];
        dv[c] += cr[D + c];
      }
    }
  }
  store_row<T, DL>(reinterpret_cast<T*>(a.dK) + col * D + sub * DL, dk);
  store_row<T, DL>(reinterpret_cast<T*>(a.dV) + col * D + sub * DL, dv);
}

// --------------------------------------------------------------- host side
template <typename F, typename... P>
cudaError_t run(const char* name, F* kern, dim3 grid, int threads, size_t smem,
                cudaStream_t s, P... p) {
  prof_before(s, name);
  kern<<<grid, threads, smem, s>>>(p...);
  prof_after(s);
  return cudaGetLastError();
}

template <typename T, typename TD, int D>
cudaError_t launch_as(Args a, cudaStream_t s) {
  const Work& w = a.w;
  cudaError_t e;
  if (a.W_i) {
    e = run("backward_window_max", backward_window_max,
            dim3((a.nq + 255) / 256, a.B), 256, 0, s, a);
    if (e != cudaSuccess) return e;
  }
  e = run("backward_rows", backward_rows<T, TD, D>,
          dim3((unsigned)((w.rows + kRowWarps - 1) / kRowWarps)),
          kRowWarps * 32, (size_t)kRowWarps * (a.k + 1) * 8, s, a);
  if (e != cudaSuccess) return e;
  int from = 0;
  for (int p = 0; p < w.passes; ++p) {
    const dim3 grid(w.tiles, w.segs);
    const uint32_t* ent = p ? a.ent[from] : nullptr;
    if ((e = run("sort_count", sort_count, grid, kSortThreads, 0, s, a,
                 (const uint32_t*)a.key[from], 8 * p)) != cudaSuccess ||
        (e = run("sort_scan", sort_scan, dim3(w.segs), 1024, 0, s, a)) !=
            cudaSuccess ||
        (e = run("sort_place", sort_place, grid, kSortThreads, 0, s, a,
                 (const uint32_t*)a.key[from], ent, a.key[from ^ 1],
                 a.ent[from ^ 1], 8 * p)) != cudaSuccess)
      return e;
    from ^= 1;
  }
  e = cudaMemsetAsync(a.span, 0, (size_t)w.segs * a.L * 8, s);
  if (e != cudaSuccess) return e;
  e = run("backward_listed", backward_listed<T, TD, D>,
          dim3((w.ranges + 7) / 8, w.segs), 256, 0, s, a,
          (const uint32_t*)a.key[from], (const uint32_t*)a.ent[from]);
  if (e != cudaSuccess) return e;
  return run("backward_columns", backward_columns<T, TD, D>,
             dim3((unsigned)(((int64_t)w.segs * a.L + 7) / 8)), 256, 0, s, a);
}

}  // namespace

size_t backward_workspace(bool, bool, int B, int nq, int L, int Hq, int Hkv,
                          int d, int k) {
  Work w;
  return plan(w, B, nq, L, Hq, Hkv, d, k) ? w.total : 0;
}

cudaError_t backward_launch(const BackwardArgs& in, bool bf16, int d, void* ws,
                            cudaStream_t s) {
  Args a;
  static_cast<BackwardArgs&>(a) = in;
  if (!plan(a.w, a.B, a.nq, a.L, a.Hq, a.Hkv, d, a.k))
    return cudaErrorNotSupported;
  char* p = (char*)ws;
  a.wmax = (int*)(p + a.w.wmax);
  a.stats = (float2*)(p + a.w.stats);
  a.pds = (float2*)(p + a.w.pds);
  for (int i = 0; i < 2; ++i) {
    a.key[i] = (uint32_t*)(p + a.w.key[i]);
    a.ent[i] = (uint32_t*)(p + a.w.ent[i]);
  }
  a.hist = (uint32_t*)(p + a.w.hist);
  a.span = (int2*)(p + a.w.span);
  a.top = (float*)(p + a.w.top);
  a.carry = (float*)(p + a.w.carry);
  // the status area and, behind it, the window maxima
  cudaError_t e = cudaMemsetAsync(ws, 0, a.w.stats, s);
  if (e != cudaSuccess) return e;
  using bf = __nv_bfloat16;
  if (bf16) {
    if (a.do_bf16)
      return d == 64 ? launch_as<bf, bf, 64>(a, s)
                     : launch_as<bf, bf, 128>(a, s);
    return d == 64 ? launch_as<bf, float, 64>(a, s)
                   : launch_as<bf, float, 128>(a, s);
  }
  if (a.do_bf16)
    return d == 64 ? launch_as<float, bf, 64>(a, s)
                   : launch_as<float, bf, 128>(a, s);
  return d == 64 ? launch_as<float, float, 64>(a, s)
                 : launch_as<float, float, 128>(a, s);
}

}  // namespace ca
