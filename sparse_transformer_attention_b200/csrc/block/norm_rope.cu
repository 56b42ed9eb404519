// Per-head norm of queries and keys, the position rotation, and the move
// from the projection's token-major rows to the [B, H, n, d] layout the
// attention reads, in one pass; and its backward pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * w          (rows with a norm weight)
//   (a, b) -> (a cos - b sin, b cos + a sin)    angle = position * inv_freq
//
// Both are bound by HBM: every row is read once and written once.  A warp
// owns one token (or some of its heads, when there are few tokens), so the
// angles of that token are computed once, one or two pairs per lane, handed
// round by shuffles and kept in registers for all its heads: no table is
// read and no shared memory used.  A lane holds 16 bytes of a row (4 or 8
// elements), a row is 8 to 32 lanes, and four row groups are in flight per
// lane.  Arithmetic is fp32 with one rounding at the store.
#include "../launch.cuh"
#include "block.cuh"

namespace ca {
namespace {

constexpr int kWarps = 8;  // per CTA
constexpr unsigned kAll = 0xFFFFFFFFu;

// cos and sin of position * inv_freq.  The product is taken in 64 bits and
// reduced to a fraction of a turn there (at position 2^20 an fp32 product
// would be off by up to 2^-4 rad); what is left, |x| <= pi, is an fp32
// argument in half turns.
__device__ __forceinline__ void angle(int pos, float inv_freq, float* c,
                                      float* s) {
  double turns = (double)pos * (double)inv_freq * 0.15915494309189533577;
  turns -= rint(turns);
  sincospif(2.f * (float)turns, s, c);
}

// The EPL = 16 / sizeof(T) elements per lane of a row and what rotates them.
template <typename T, int D>
struct Lanes {
  static constexpr int EPL = Elem<T>::kPer16B;
  static constexpr int LPR = D / EPL;   // lanes per row
  static constexpr int RW = 32 / LPR;   // rows per warp and step
  int sub;        // this lane's place in its row
  int src;        // lane that holds the partners (split pairs)
  bool turns;     // whether this lane's elements are rotated
  float c[EPL], s[EPL];  // cos; sin with the sign of the element's place

  __device__ __forceinline__ void init(const NormRopeArgs& a, int lane) {
    sub = lane % LPR;
    const int half = a.rot / 2 / EPL;  // lanes of a half row (split pairs)
    turns = sub * EPL < a.rot;
    src = lane;
    if (!a.interleaved && turns) src = sub < half ? lane + half : lane - half;
  }

  // The angles of one token, with sign +1 for the rotation and -1 for its
  // transpose.
  __device__ __forceinline__ void set_token(const NormRopeArgs& a, int pos,
                                            int lane, float sign) {
    constexpr int NP = D / 2 / 32;  // pairs per lane: 1 or 2
    const int pairs = a.rot / 2;
    float pc[NP], ps[NP];
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int p = lane + 32 * u;
      pc[u] = 1.f;
      ps[u] = 0.f;
      if (p < pairs) angle(pos, __ldg(a.inv_freq + p), &pc[u], &ps[u]);
    }
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      const int el = sub * EPL + e;
      int p = a.interleaved ? el / 2 : (el < pairs ? el : el - pairs);
      const bool first = a.interleaved ? (e & 1) == 0 : el < pairs;
      if (!turns) p = 0;
      float cc = __shfl_sync(kAll, pc[0], p & 31);
      float ss = __shfl_sync(kAll, ps[0], p & 31);
      if constexpr (NP == 2) {
        const float c1 = __shfl_sync(kAll, pc[1], p & 31);
        const float s1 = __shfl_sync(kAll, ps[1], p & 31);
        if (p >= 32) {
          cc = c1;
          ss = s1;
        }
      }
      c[e] = turns ? cc : 1.f;
      s[e] = turns ? (first ? -sign * ss : sign * ss) : 0.f;
    }
  }

  // The rotation of one row (every lane of the warp takes part).
  __device__ __forceinline__ void rotate(bool interleaved, float* v) const {
    float o[EPL];
    if (interleaved) {
#pragma unroll
      for (int e = 0; e < EPL; ++e) o[e] = v[e ^ 1];
    } else {
#pragma unroll
      for (int e = 0; e < EPL; ++e) o[e] = __shfl_sync(kAll, v[e], src);
    }
#pragma unroll
    for (int e = 0; e < EPL; ++e) v[e] = fmaf(v[e], c[e], o[e] * s[e]);
  }

  __device__ __forceinline__ static float row_sum(float x) {
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1)
      x += __shfl_xor_sync(kAll, x, off);
    return x;
  }

  __device__ __forceinline__ void weights(const void* w, int bf16,
                                          float* f) const {
#pragma unroll
    for (int e = 0; e < EPL; ++e)
      f[e] = bf16 ? __bfloat162float(
                        reinterpret_cast<const __nv_bfloat16*>(w)[sub * EPL + e])
                  : reinterpret_cast<const float*>(w)[sub * EPL + e];
  }
};

template <typename T>
__device__ __forceinline__ const uint4* row_at(const Rows& r, int b, int t,
                                               int h, int el) {
  return reinterpret_cast<const uint4*>(
      reinterpret_cast<const T*>(r.p) + b * r.sb + t * r.st + h * r.sh + el);
}
template <typename T>
__device__ __forceinline__ uint4* row_to(const Rows& r, int b, int t, int h,
                                         int el) {
  return reinterpret_cast<uint4*>(reinterpret_cast<T*>(r.p) + b * r.sb +
                                  t * r.st + h * r.sh + el);
}

// Heads [h0, h1) of one kind (0 q, 1 k, 2 v) of one token.
template <typename T, int D, int U>
__device__ __forceinline__ void forward_heads(const NormRopeArgs& a,
                                              const Lanes<T, D>& L, int kind,
                                              int b, int t, int h0, int h1,
                                              int lane) {
  using LN = Lanes<T, D>;
  constexpr int EPL = LN::EPL;
  const Rows x = a.x[kind], y = a.y[kind];
  const bool norm = kind < 2 && a.w[kind];
  float w[EPL];
  if (norm) L.weights(a.w[kind], a.w_bf16, w);
  const int el = L.sub * EPL;
#pragma unroll 1
  for (int h = h0 + lane / LN::LPR; h - lane / LN::LPR < h1;
       h += U * LN::RW) {
    uint4 in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      in[u] = make_uint4(0, 0, 0, 0);
      if (h + u * LN::RW < h1)
        in[u] = __ldg(row_at<T>(x, b, t, h + u * LN::RW, el));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int hu = h + u * LN::RW;
      if (hu - lane / LN::LPR >= h1) break;  // uniform over the warp
      uint4 out = in[u];
      if (kind < 2) {
        float v[EPL];
        Elem<T>::unpack(in[u], v);
        if (norm) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < EPL; ++e) ss = fmaf(v[e], v[e], ss);
          ss = LN::row_sum(ss);
          const float r = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
          for (int e = 0; e < EPL; ++e) v[e] *= r * w[e];
        }
        L.rotate(a.interleaved, v);
        out = pack16<T>(v);
      }
      if (hu < h1) *row_to<T>(y, b, t, hu, el) = out;
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) norm_rope(NormRopeArgs a) {
  chain();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int heads = a.Hq + 2 * a.Hkv;
  const int per = (heads + a.chunk - 1) / a.chunk;  // warps per token
  const int64_t token = unit / per;
  if (token >= (int64_t)a.B * a.n) return;  // the whole warp
  const int c0 = (int)(unit % per) * a.chunk;
  const int c1 = min(c0 + a.chunk, heads);
  const int b = (int)(token / a.n), t = (int)(token % a.n);
  Lanes<T, D> L;
  L.init(a, lane);
  if (c0 < a.Hq + a.Hkv)
    L.set_token(a, a.positions ? a.positions[token] : a.pos0 + t, lane, 1.f);
#pragma unroll 1
  for (int kind = 0; kind < 3; ++kind) {
    const int k0 = kind == 0 ? 0 : a.Hq + (kind - 1) * a.Hkv;
    const int nh = kind == 0 ? a.Hq : a.Hkv;
    const int h0 = max(c0 - k0, 0), h1 = min(c1 - k0, nh);
    if (h0 < h1 && a.y[kind].p)
      forward_heads<T, D, 4>(a, L, kind, b, t, h0, h1, lane);
  }
}

// dx of one head row, and its part of the weight's gradient:
//   g = R^T dy,  xh = x r,  dw += g xh,
//   dx = r (w g - xh mean(w g xh))
template <typename T, int D, int U>
__device__ __forceinline__ void backward_heads(const NormRopeArgs& a,
                                               const Lanes<T, D>& L, int kind,
                                               int b, int t, int h0, int h1,
                                               int lane, float* dw) {
  using LN = Lanes<T, D>;
  constexpr int EPL = LN::EPL;
  const Rows x = a.x[kind], y = a.y[kind], dx = a.dx[kind];
  const bool norm = kind < 2 && a.w[kind];
  float w[EPL];
  if (norm) L.weights(a.w[kind], a.w_bf16, w);
  const int el = L.sub * EPL;
#pragma unroll 1
  for (int h = h0 + lane / LN::LPR; h - lane / LN::LPR < h1;
       h += U * LN::RW) {
    uint4 in[U], xin[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      in[u] = make_uint4(0, 0, 0, 0);
      xin[u] = make_uint4(0, 0, 0, 0);
      if (h + u * LN::RW < h1) {
        in[u] = __ldg(row_at<T>(y, b, t, h + u * LN::RW, el));
        if (norm) xin[u] = __ldg(row_at<T>(x, b, t, h + u * LN::RW, el));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int hu = h + u * LN::RW;
      if (hu - lane / LN::LPR >= h1) break;  // uniform over the warp
      uint4 out = in[u];
      if (kind < 2) {
        float g[EPL];
        Elem<T>::unpack(in[u], g);
        L.rotate(a.interleaved, g);
        if (norm) {
          float v[EPL];
          Elem<T>::unpack(xin[u], v);
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int e = 0; e < EPL; ++e) {
            ss = fmaf(v[e], v[e], ss);
            dot = fmaf(g[e] * w[e], v[e], dot);
          }
          ss = LN::row_sum(ss);
          dot = LN::row_sum(dot);
          const float r = rsqrtf(ss * (1.f / D) + a.eps);
          const float m = dot * r * (1.f / D);  // mean(w g xh)
#pragma unroll
          for (int e = 0; e < EPL; ++e) {
            const float xh = v[e] * r;
            dw[e] = fmaf(g[e], xh, dw[e]);  // rows past h1 hold zeros
            g[e] = r * (g[e] * w[e] - xh * m);
          }
        }
        out = pack16<T>(g);
      }
      if (hu < h1) *row_to<T>(dx, b, t, hu, el) = out;
    }
  }
}

// A CTA's warps walk over the tokens with a stride; each lane sums the
// weight gradients of its elements over all rows it sees (q and k apart).
// At the end the sums meet in a fixed order: over the row groups of a warp,
// over the warps, and over the CTAs (norm_rope_weights), so a result does
// not depend on timing.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32)
norm_rope_backward(NormRopeArgs a) {
  using LN = Lanes<T, D>;
  constexpr int EPL = LN::EPL;
  __shared__ float s_dw[kWarps][2][D];
  chain();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int heads = a.Hq + 2 * a.Hkv;
  const int per = (heads + a.chunk - 1) / a.chunk;
  const int64_t units = (int64_t)a.B * a.n * per;
  float dw[2][EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) dw[0][e] = dw[1][e] = 0.f;
  LN L;
  L.init(a, lane);
#pragma unroll 1
  for (int64_t unit = (int64_t)blockIdx.x * kWarps + wid; unit < units;
       unit += (int64_t)gridDim.x * kWarps) {
    const int64_t token = unit / per;
    const int c0 = (int)(unit % per) * a.chunk;
    const int c1 = min(c0 + a.chunk, heads);
    const int b = (int)(token / a.n), t = (int)(token % a.n);
    if (c0 < a.Hq + a.Hkv)
      L.set_token(a, a.positions ? a.positions[token] : a.pos0 + t, lane,
                  -1.f);
    {
      const int h1 = min(c1, a.Hq);
      if (c0 < h1)
        backward_heads<T, D, 2>(a, L, 0, b, t, c0, h1, lane, dw[0]);
    }
    {
      const int h0 = max(c0 - a.Hq, 0), h1 = min(c1 - a.Hq, a.Hkv);
      if (h0 < h1 && a.dx[1].p)
        backward_heads<T, D, 2>(a, L, 1, b, t, h0, h1, lane, dw[1]);
    }
    {
      const int k0 = a.Hq + a.Hkv;
      const int h0 = max(c0 - k0, 0), h1 = min(c1 - k0, a.Hkv);
      if (h0 < h1 && a.dx[2].p)
        backward_heads<T, D, 4>(a, L, 2, b, t, h0, h1, lane, nullptr);
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int kd = 0; kd < 2; ++kd)
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      float x = dw[kd][e];
#pragma unroll
      for (int off = 16; off >= LN::LPR; off >>= 1)
        x += __shfl_xor_sync(kAll, x, off);
      if (lane < LN::LPR) s_dw[wid][kd][lane * EPL + e] = x;
    }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += kWarps * 32) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x += s_dw[w][c / D][c % D];
    a.partial[(size_t)blockIdx.x * 2 * D + c] = x;
  }
}

// The CTAs' partial weight gradients, summed: 32 columns per CTA, 32 threads
// per column.
template <int D>
__global__ void __launch_bounds__(1024)
norm_rope_weights(NormRopeArgs a, int ctas) {
  __shared__ float s[32][33];
  chain();
  const int col = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + col;
  float x = 0.f;
  for (int i = part; i < ctas; i += 32) x += a.partial[(size_t)i * 2 * D + c];
  s[part][col] = x;
  __syncthreads();
  x = s[col][part];  // column `part`, piece `col`
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(kAll, x, off);
  if (col == 0) {
    const int cc = blockIdx.x * 32 + part;
    void* dw = a.dw[cc / D];
    if (!dw) return;
    if (a.w_bf16)
      reinterpret_cast<__nv_bfloat16*>(dw)[cc % D] = __float2bfloat16_rn(x);
    else
      reinterpret_cast<float*>(dw)[cc % D] = x;
  }
}

// Heads per warp: a whole token while tokens alone give every SM sixteen
// warps, fewer heads (down to one step of the warp) below that, where the
// call is bound by latency.
template <typename T, int D>
int head_chunk(const NormRopeArgs& a) {
  constexpr int RW = Lanes<T, D>::RW;
  const int heads = a.Hq + 2 * a.Hkv;
  const int64_t tokens = (int64_t)a.B * a.n;
  const int64_t want = (int64_t)sm_count() * 16;
  int64_t chunk = (heads * tokens + want - 1) / want;
  chunk = (chunk + RW - 1) / RW * RW;
  return (int)(chunk < heads ? chunk : heads);
}

template <typename T, int D>
cudaError_t forward_as(NormRopeArgs a, cudaStream_t s) {
  a.chunk = head_chunk<T, D>(a);
  const int heads = a.Hq + 2 * a.Hkv;
  const int64_t units =
      (int64_t)a.B * a.n * ((heads + a.chunk - 1) / a.chunk);
  const int64_t ctas = (units + kWarps - 1) / kWarps;
  if (ctas > 0x7FFFFFFF) return cudaErrorNotSupported;
  return launch("norm_rope", norm_rope<T, D>, dim3((unsigned)ctas),
                kWarps * 32, 0, s, a);
}

template <typename T, int D>
cudaError_t backward_as(NormRopeArgs a, cudaStream_t s) {
  a.chunk = head_chunk<T, D>(a);
  const int heads = a.Hq + 2 * a.Hkv;
  const int64_t units =
      (int64_t)a.B * a.n * ((heads + a.chunk - 1) / a.chunk);
  int64_t ctas = (units + kWarps - 1) / kWarps;
  if (ctas > kNormRopeMaxCtas) ctas = kNormRopeMaxCtas;
  if (!a.w[0] && !a.w[1]) a.partial = nullptr;
  const cudaError_t e = launch("norm_rope_backward", norm_rope_backward<T, D>,
                               dim3((unsigned)ctas), kWarps * 32, 0, s, a);
  if (e != cudaSuccess || !a.partial) return e;
  return launch("norm_rope_weights", norm_rope_weights<D>, dim3(2 * D / 32),
                1024, 0, s, a, (int)ctas);
}

}  // namespace

cudaError_t norm_rope_launch(NormRopeArgs a, bool bf16, int d,
                             cudaStream_t s) {
  if (bf16)
    return d == 64 ? forward_as<__nv_bfloat16, 64>(a, s)
                   : forward_as<__nv_bfloat16, 128>(a, s);
  return d == 64 ? forward_as<float, 64>(a, s) : forward_as<float, 128>(a, s);
}

cudaError_t norm_rope_backward_launch(NormRopeArgs a, bool bf16, int d,
                                      cudaStream_t s) {
  if (bf16)
    return d == 64 ? backward_as<__nv_bfloat16, 64>(a, s)
                   : backward_as<__nv_bfloat16, 128>(a, s);
  return d == 64 ? backward_as<float, 64>(a, s)
                 : backward_as<float, 128>(a, s);
}

}  // namespace ca
