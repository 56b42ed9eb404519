// The prefill's backward pass for bf16 on matrix instructions.  All products
// run as m16n8k16 bf16 with fp32 sums.  Operands that are not inputs (p, dS,
// e dP) enter in two bf16 parts, hi + lo, so that they keep 16 bits: with one
// part the gradients' error would be half as large again as that of the
// rounding to bf16 at the end.
//
// The work per (row, key) pair is small and most pairs are gathered, so what
// bounds these kernels is reading rows from L2 and issuing instructions, not
// the tensor pipe; the layouts below keep both low.
#include "../launch.cuh"
#include "../profile.cuh"
#include "backward.cuh"

namespace ca {
namespace bwd {
namespace {

using bf = __nv_bfloat16;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1,
                                    uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
      "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 tile of 16-bit elements held one row per four
// lanes, two elements per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void* p) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"((uint32_t)__cvta_generic_to_shared(p))
      : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const void* p) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"((uint32_t)__cvta_generic_to_shared(p))
      : "memory");
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
// Two values as the hi and lo parts of a bf16 pair each.
__device__ __forceinline__ void split2(float x, float y, uint32_t* hi,
                                       uint32_t* lo) {
  *hi = pack2(x, y);
  *lo = pack2(x - bf16lo(*hi), y - bf16hi(*hi));
}

// ---------------------------------------------------------------- row pass
// A CTA owns 64 query rows of one head, a warp 16.  In order:
//   1. the window's and the anchor's scores and dP: running (max, sum e,
//      sum e dP) of each row;
//   2. row by row, the Top-k, 16 gathered K and V rows at a time: as A
//      operands they meet q and dO, half lines as rows of A against half
//      lines as columns of B.  The sums A = sum e dP k and Bk = sum e k take
//      the same K registers, transposed in place, against a B operand whose
//      columns are e dP and e in two parts each.  So a gathered row is read
//      once, and dQ's listed part (A - D Bk) / l follows when the row's sums
//      are complete;
//   3. the window and the anchor again, now with the final log-sum-exp and
//      D: dS, and dQ's window part.
// The window is 5 blocks of 16 x 16 per 16 rows at W = 64, so computing its
// scores twice costs less than keeping a second accumulator.  What a warp
// waits for is latency (a gathered row comes from L2): the index rows are
// read in one batch, and the next V and K rows are asked for as soon as the
// registers of the current ones are free.
constexpr int kRowWarps = 4;

template <int D, int NP>
struct RowSmem {
  static constexpr int CK = 64;         // keys staged at a time
  static constexpr int RS = D * 2 + 16; // padded row (bytes)
  // K and V of the window, or q and dO of the CTA's rows
  static constexpr size_t stage = (size_t)(NP + 1) * 64 * RS;
  __host__ __device__ static size_t per_warp(int kk) {
    return (size_t)16 * D * 4 + 4 * 16 * 4 + (size_t)kk * 8 +
           (size_t)16 * kk * 4;
  }
  static size_t bytes(int k) {
    return stage + kRowWarps * per_warp((k + 15) / 16 * 16);
  }
};

// 16 gathered K or V rows: load i holds keys 4 i + gr / 2, eight lanes on one
// 128-byte line (four wavefronts a load; rows spread over four lanes each
// took eight).
template <int D>
struct Gather {
  static constexpr int NL = D / 64;  // lines of a row
  uint32_t v[4][NL][4];
  __device__ __forceinline__ void load(const bf* base, const int (&j)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4* p =
          reinterpret_cast<const uint4*>(base + (int64_t)max(j[i], 0) * D);
#pragma unroll
      for (int c = 0; c < NL; ++c) {
        const uint4 t = __ldg(p + 8 * c);
        v[i][c][0] = t.x;
        v[i][c][1] = t.y;
        v[i][c][2] = t.z;
        v[i][c][3] = t.w;
      }
    }
  }
  // Products of all rows with a vector whose halves of each line stand in
  // the even and odd columns of B (w: this lane's 16 bytes of a line).  The
  // result for key 4 tq + gr / 2.
  __device__ __forceinline__ float dot(const uint4 (&w)[NL], int gr,
                                       int tq) const {
    float d[2][4];
    add_dot(w, d, true);
    return pick(d, gr, tq);
  }
  __device__ __forceinline__ void add_dot(const uint4 (&w)[NL],
                                          float (&d)[2][4], bool clear) const {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      if (clear) d[g][0] = d[g][1] = d[g][2] = d[g][3] = 0.f;
#pragma unroll
      for (int c = 0; c < NL; ++c) {
        mma(d[g], v[2 * g][c][0], v[2 * g + 1][c][0], v[2 * g][c][1],
            v[2 * g + 1][c][1], w[c].x, w[c].y);
        mma(d[g], v[2 * g][c][2], v[2 * g + 1][c][2], v[2 * g][c][3],
            v[2 * g + 1][c][3], w[c].z, w[c].w);
      }
    }
  }
  // Row gr (and gr + 8) of a product is key gr / 2 of a load, its first half
  // at even gr (even columns), its second at odd gr (odd columns).
  __device__ __forceinline__ static float pick(const float (&d)[2][4], int gr,
                                               int tq) {
    const bool odd = gr & 1;
    const float a0 = odd ? d[0][1] : d[0][0], a1 = odd ? d[0][3] : d[0][2];
    const float b0 = odd ? d[1][1] : d[1][0], b1 = odd ? d[1][3] : d[1][2];
    const float a = (tq & 1) ? a1 : a0, b = (tq & 1) ? b1 : b0;
    const float x = (tq & 2) ? b : a;
    return x + __shfl_xor_sync(kAll, x, 4);
  }
};

// The largest of the warp's values.
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

template <int D, int NP>
__global__ void __launch_bounds__(kRowWarps * 32, D == 64 ? 4 : 2)
backward_rows_mma(Args a, int ntile) {
  using SM = RowSmem<D, NP>;
  constexpr int RS = SM::RS, CK = SM::CK;
  constexpr int KS = D / 16;  // steps of a product over the head dimension
  constexpr int NT = D / 8;   // its 8-wide tiles
  extern __shared__ __align__(16) unsigned char g_smem[];
  __shared__ int s_kmin, s_any;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int gr = lane >> 2, tq = lane & 3;
  const int k = a.k, kk = (k + 15) / 16 * 16;
  const int nq = a.nq, L = a.L;
  const int bh = blockIdx.x / ntile;
  const int r0 = (blockIdx.x % ntile) * 64;
  const int b = bh / a.Hq, h = bh % a.Hq;
  const int seg = b * a.Hkv + h / (a.Hq / a.Hkv);
  const int i0 = r0 + wid * 16;  // the warp's first row
  const int64_t rowbase = (int64_t)bh * nq;
  const bf* Qg = reinterpret_cast<const bf*>(a.Q) + rowbase * D;
  const bf* Kg = reinterpret_cast<const bf*>(a.K) + (int64_t)seg * L * D;
  const bf* Vg = reinterpret_cast<const bf*>(a.V) + (int64_t)seg * L * D;
  unsigned char* sK = g_smem;
  unsigned char* sV = g_smem + (size_t)CK * RS;
  float* s_dq = reinterpret_cast<float*>(g_smem + SM::stage +
                                         (size_t)wid * SM::per_warp(kk));
  float* s_m = s_dq + 16 * D;  // running maximum, then the log-sum-exp
  float* s_l = s_m + 16;
  float* s_E = s_l + 16;       // sum e dP, then D
  int* s_top = reinterpret_cast<int*>(s_E + 16);  // Top-k entries of a row
  float2* s_xd = reinterpret_cast<float2*>(s_top + 16);  // one row's (x, dP)
  int* s_idx = reinterpret_cast<int*>(s_xd + kk);
  const float sl2 = kLog2e / sqrtf((float)D), sc = 1.f / sqrtf((float)D);
  constexpr int kPieces = D * 2 / 16;  // 16-byte pieces of a row

  // q and the planes of dO, rows r0 .. r0 + 63, where K and V are staged in
  // the other phases
  auto stage_rows = [&]() {
    for (int e = threadIdx.x; e < 64 * kPieces; e += kRowWarps * 32) {
      const int rr = e / kPieces, pc = e % kPieces;
      const int64_t at = (int64_t)min(r0 + rr, nq - 1) * D + pc * 8;
      unsigned char* dst = g_smem + rr * RS + pc * 16;
      cp_async16(dst, Qg + at);
#pragma unroll
      for (int p = 0; p < NP; ++p)
        cp_async16(dst + (size_t)(p + 1) * 64 * RS, a.g[p] + rowbase * D + at);
    }
  };
  stage_rows();
  if (threadIdx.x == 0) {
    s_kmin = 0x7FFFFFFF;
    s_any = 0;
  }

  // the windows and Top-k counts of the warp's rows, a row per lane, and the
  // Top-k positions: checked, kept, and written as the entries' sort keys
  const int nrow = min(16, nq - i0);  // 0 or less: no rows
  {
    const int rr = min(lane, max(nrow, 1) - 1);
    const int r = min(i0 + rr, nq - 1);
    const bool mine = lane < nrow;
    int w;
    const int lo = window_lo(a, b, h, r, mine, &w);
    const int m = listed_count(a, rowbase + r, a.p0 + r, lo, w, mine);
    if (mine) s_top[lane] = m;
    const int last = a.p0 + r - w;  // the last candidate
    uint32_t* key = a.key[0] + (rowbase + i0) * (k + 1);
    if (mine) key[(int64_t)lane * (k + 1)] = lo > 0 ? 0u : (uint32_t)L;
    const int32_t* ix = a.idx + (rowbase + i0) * a.C_max + 1;
#pragma unroll 1
    for (int t0 = 0; t0 < k; t0 += 32) {
      const int t = t0 + lane;
      int j[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const int mu = __shfl_sync(kAll, m, u);
        j[u] = u < nrow && t < mu ? __ldg(ix + (int64_t)u * a.C_max + t) : -1;
      }
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const int mu = __shfl_sync(kAll, m, u);
        const int lu = __shfl_sync(kAll, last, u);
        if (u < nrow && t < k) {
          int v = j[u];
          if (t < mu && (v < 1 || v > lu)) {  // not a candidate of this row
            raise_flag(a.status, kErrCmax);
            v = -1;
          }
          s_idx[u * kk + t] = v;
          key[(int64_t)u * (k + 1) + 1 + t] = v < 0 ? (uint32_t)L : (uint32_t)v;
        }
      }
    }
  }
  cp_async_wait_all();
  __syncthreads();

  // this lane's two rows of the warp's 16 in the window products
  const bool wlive = nrow > 0;
  const int ra = i0 + gr, rb = ra + 8;
  const bool va = ra < nq, vb = rb < nq;
  const int ca = min(ra, nq - 1), cb = min(rb, nq - 1);
  const int ia = a.p0 + ca, ib = a.p0 + cb;
  int wa, wb;
  const int loa = window_lo(a, b, h, ca, false, &wa);
  const int lob = window_lo(a, b, h, cb, false, &wb);
  int kmin = min(loa, lob);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    kmin = min(kmin, __shfl_xor_sync(kAll, kmin, off));
  const int kmax = a.p0 + min(i0 + 15, nq - 1);
  const bool anchors = __any_sync(kAll, (va && loa > 0) || (vb && lob > 0));
  if (wlive && lane == 0) {
    atomicMin(&s_kmin, kmin);
    if (anchors) s_any = 1;
  }
  // A operands of the window products: q and dO of the warp's rows
  uint32_t qa[KS][4], ga[NP][KS][4];
  auto fragments = [&]() {
    const unsigned char* at =
        g_smem + (wid * 16 + (lane & 15)) * RS + (lane >> 4) * 16;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      ldsm4(qa[ks], at + ks * 32);
#pragma unroll
      for (int p = 0; p < NP; ++p)
        ldsm4(ga[p][ks], at + (size_t)(p + 1) * 64 * RS + ks * 32);
    }
  };
  fragments();
  __syncthreads();
  const int cs0 = s_kmin & ~15;
  const int kmax_c = a.p0 + min(r0 + 63, nq - 1);
  const int nch = (kmax_c - cs0) / CK + 1;
  const int m0 = s_any ? -1 : 0;  // chunk -1: the anchor's 16 keys

  auto stage = [&](int m) {
    const int cs = m < 0 ? 0 : cs0 + m * CK;
    const int rows = m < 0 ? 16 : min(CK, kmax_c + 1 - cs);
    for (int e = threadIdx.x; e < ((rows + 15) & ~15) * kPieces;
         e += kRowWarps * 32) {
      const int rr = e / kPieces, pc = e % kPieces;
      const int j = min(cs + rr, L - 1);  // rows past the cache: any valid
      cp_async16(sK + rr * RS + pc * 16, Kg + (size_t)j * D + pc * 8);
      cp_async16(sV + rr * RS + pc * 16, Vg + (size_t)j * D + pc * 8);
    }
    cp_async_wait_all();
  };
  // scores (log2 units, masked to -inf) and dP of the 16 x 16 block of keys
  // kb.. (at place kl of the staged chunk), as two accumulators of 8 keys
  auto block = [&](int kb, int kl, bool anchor, float (&x)[2][4],
                   float (&dp)[2][4]) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) x[t][c] = dp[t][c] = 0.f;
    const int lr = kl + (lane & 7) + ((lane >> 4) << 3);
    const int lc = ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t f[4];
      ldsm4(f, sK + lr * RS + ks * 32 + lc);
      mma(x[0], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], f[0], f[1]);
      mma(x[1], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], f[2], f[3]);
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t f[4];
      ldsm4(f, sV + lr * RS + ks * 32 + lc);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        mma(dp[0], ga[p][ks][0], ga[p][ks][1], ga[p][ks][2], ga[p][ks][3],
            f[0], f[1]);
        mma(dp[1], ga[p][ks][0], ga[p][ks][1], ga[p][ks][2], ga[p][ks][3],
            f[2], f[3]);
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int j = kb + 8 * t + 2 * tq + (c & 1);
        const bool ok = c < 2
            ? va && (anchor ? j == 0 && loa > 0 : j >= loa && j <= ia)
            : vb && (anchor ? j == 0 && lob > 0 : j >= lob && j <= ib);
        x[t][c] = ok ? x[t][c] * sl2 : -INFINITY;
      }
  };

  // ---- 1: window and anchor, running sums
  {
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, E[2] = {0.f, 0.f};
#pragma unroll 1
    for (int ch = m0; ch < nch; ++ch) {
      stage(ch);
      __syncthreads();
      const int cs = ch < 0 ? 0 : cs0 + ch * CK;
      const int jlo = ch < 0 ? 0 : max(cs, kmin & ~15);
      const int jhi = ch < 0 ? (anchors ? 0 : -1) : min(cs + CK - 1, kmax);
#pragma unroll 1
      for (int kb = jlo; wlive && kb <= jhi; kb += 16) {
        float x[2][4], dp[2][4];
        block(kb, kb - cs, ch < 0, x, dp);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float mx = fmaxf(fmaxf(x[0][2 * u], x[0][2 * u + 1]),
                                 fmaxf(x[1][2 * u], x[1][2 * u + 1]));
          if (mx > m[u]) {
            const float f = exp2f(m[u] - mx);
            l[u] *= f;
            E[u] *= f;
            m[u] = mx;
          }
          if (m[u] == -INFINITY) continue;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float e = exp2f(x[t][2 * u + c] - m[u]);
              l[u] += e;
              E[u] = fmaf(e, dp[t][2 * u + c], E[u]);
            }
        }
      }
      __syncthreads();
    }
    stage_rows();  // for the Top-k and the last phase
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float mx = m[u];
      mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2));
      const float f = m[u] == -INFINITY ? 0.f : exp2f(m[u] - mx);
      float ll = l[u] * f, EE = E[u] * f;
      ll += __shfl_xor_sync(kAll, ll, 1);
      EE += __shfl_xor_sync(kAll, EE, 1);
      ll += __shfl_xor_sync(kAll, ll, 2);
      EE += __shfl_xor_sync(kAll, EE, 2);
      if (tq == 0) {
        s_m[gr + 8 * u] = mx;
        s_l[gr + 8 * u] = ll;
        s_E[gr + 8 * u] = EE;
      }
    }
    cp_async_wait_all();
    __syncthreads();
  }

  // ---- 2: the Top-k, row by row, 16 entries at a time
  {
    constexpr int NL = D / 64;
    const bf* Kl = Kg + 8 * (lane & 7);
    const bf* Vl = Vg + 8 * (lane & 7);
    const int half = gr & 1, kq = gr >> 1;
    Gather<D> kr, vr;
    int j[4];  // the entries in kr and vr (-1: none, row 0 is read)
    auto entries = [&](int rr, int g0) {
      const int mt = s_top[rr];
      const int* ix = s_idx + rr * kk + g0 + kq;
#pragma unroll
      for (int i = 0; i < 4; ++i) j[i] = g0 + 4 * i + kq < mt ? ix[4 * i] : -1;
    };
    if (wlive && s_top[0] > 0) {
      entries(0, 0);
      kr.load(Kl, j);
      vr.load(Vl, j);
    }
#pragma unroll 1
    for (int rr = 0; rr < nrow; ++rr) {
      const int64_t row = rowbase + i0 + rr;
      const int mt = s_top[rr];
      float m = s_m[rr], l0 = s_l[rr], E0 = s_E[rr];  // window and anchor
      // even columns: first halves of the lines, odd columns: second halves
      const unsigned char* qrow =
          g_smem + (wid * 16 + rr) * RS + 64 * half + 16 * tq;
      // sums: acc of the rows' dimensions, sum of the weights alone (columns
      // 0, 1: e dP, columns 2, 3: e)
      float acc[2 * NL][4], sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < 2 * NL; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[t][c] = 0.f;
      if (mt == 0 && rr + 1 < nrow && s_top[rr + 1] > 0) {
        entries(rr + 1, 0);  // nothing was read ahead
        kr.load(Kl, j);
        vr.load(Vl, j);
      }
#pragma unroll 1
      for (int g0 = 0; g0 < mt; g0 += 16) {
        // this lane's key of the softmax: 4 tq + gr / 2
        const int mine = g0 + 4 * tq + kq;
        const bool use = mine < mt && s_idx[rr * kk + mine] >= 0;
        // the next entries: of this row, or the first of the next one
        const bool same = g0 + 16 < mt;
        entries(same ? rr : min(rr + 1, nrow - 1), same ? g0 + 16 : 0);
        float d[2][4];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          uint4 w[NL];
#pragma unroll
          for (int c = 0; c < NL; ++c)
            w[c] = *reinterpret_cast<const uint4*>(
                qrow + (size_t)(p + 1) * 64 * RS + 128 * c);
          vr.add_dot(w, d, p == 0);
        }
        vr.load(Vl, j);
        const float dp = Gather<D>::pick(d, gr, tq);
        float x;
        {
          uint4 w[NL];
#pragma unroll
          for (int c = 0; c < NL; ++c)
            w[c] = *reinterpret_cast<const uint4*>(qrow + 128 * c);
          x = kr.dot(w, gr, tq);
        }
        x = use ? x * sl2 : -INFINITY;
        const float mx = warp_max(x);
        if (mx > m) {  // the same for the whole warp
          const float f = exp2f(m - mx);
          l0 *= f;
          E0 *= f;
#pragma unroll
          for (int c = 0; c < 4; ++c) sum[c] *= f;
#pragma unroll
          for (int t = 0; t < 2 * NL; ++t)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[t][c] *= f;
          m = mx;
        }
        const float e = exp2f(x - m);
        if (half == 0) s_xd[mine] = make_float2(x, dp);
        // B: columns 0-3 (4-7) weigh the rows' first (second) halves with
        // e dP (hi, lo) and e (hi, lo); its row pair (2 tq, 2 tq + 1) is the
        // two halves of key tq of a load
        const float w = half ? e : e * dp;
        const int src = 8 * tq + 4 * ((gr >> 1) & 1);
        uint32_t B[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = __shfl_sync(kAll, w, src + i);
          const uint32_t hi = pack2(v, 0.f);
          const uint32_t t = half ? pack2(v - bf16lo(hi), 0.f) : hi;
          B[i] = gr >= 4 ? t << 16 : t;
        }
        constexpr uint32_t kOnes = 0x3F803F80u;  // two bf16 ones
        mma(sum, kOnes, kOnes, kOnes, kOnes, B[0], B[1]);
        mma(sum, kOnes, kOnes, kOnes, kOnes, B[2], B[3]);
#pragma unroll
        for (int c = 0; c < NL; ++c)
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int t = 0; t < 2; ++t)
              mma(acc[2 * c + t], transpose8x8(kr.v[2 * g][c][2 * t]),
                  transpose8x8(kr.v[2 * g][c][2 * t + 1]),
                  transpose8x8(kr.v[2 * g + 1][c][2 * t]),
                  transpose8x8(kr.v[2 * g + 1][c][2 * t + 1]), B[2 * g],
                  B[2 * g + 1]);
        kr.load(Kl, j);
      }
      const float l = l0 + __shfl_sync(kAll, sum[0] + sum[1], 1);
      const float E = E0 + __shfl_sync(kAll, sum[0] + sum[1], 0);
      const float inv = 1.f / l, Di = E * inv, lse = m + log2f(l);
      if (lane == 0) {
        s_m[rr] = lse;
        s_E[rr] = Di;
        a.stats[row] = make_float2(lse, Di);
      }
      // lanes tq = 0 (2) hold A of the lines' first (second) halves, tq = 1
      // (3) Bk: dimensions 8 (gr / 2) + gr % 2 + {0, 2, 4, 6} of a half
#pragma unroll
      for (int t = 0; t < 2 * NL; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float v = acc[t][2 * u] + acc[t][2 * u + 1];
          const float o = __shfl_down_sync(kAll, v, 1);
          if ((tq & 1) == 0)
            s_dq[rr * D + 64 * (t >> 1) + 16 * tq + 8 * kq + half +
                 4 * (t & 1) + 2 * u] = (v - Di * o) * inv * sc;
        }
      __syncwarp();
      float2* pds = a.pds + row * (k + 1);
      for (int t = lane; t < k; t += 32) {
        float2 o = make_float2(0.f, 0.f);
        if (t < mt) {
          const float2 xd = s_xd[t];
          o.x = exp2f(xd.x - lse);  // 0 where the slot was refused
          o.y = o.x * (xd.y - Di) * sc;
        }
        pds[1 + t] = o;
      }
      __syncwarp();
    }
  }

  // ---- 3: dS of the window and the anchor
  {
    fragments();
    __syncthreads();
    float o[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[t][c] = 0.f;
    const float lse[2] = {s_m[gr], s_m[gr + 8]}, Di[2] = {s_E[gr], s_E[gr + 8]};
#pragma unroll 1
    for (int ch = m0; ch < nch; ++ch) {
      stage(ch);
      __syncthreads();
      const int cs = ch < 0 ? 0 : cs0 + ch * CK;
      const int jlo = ch < 0 ? 0 : max(cs, kmin & ~15);
      const int jhi = ch < 0 ? (anchors ? 0 : -1) : min(cs + CK - 1, kmax);
#pragma unroll 1
      for (int kb = jlo; wlive && kb <= jhi; kb += 16) {
        float x[2][4], dp[2][4];
        block(kb, kb - cs, ch < 0, x, dp);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float p = exp2f(x[t][c] - lse[c >> 1]);
            const float ds = p * (dp[t][c] - Di[c >> 1]) * sc;
            if (ch < 0 && t == 0 && (c & 1) == 0 && tq == 0 &&
                (c ? vb : va))  // the anchor's entry (zeros without one)
              a.pds[(rowbase + (c ? rb : ra)) * (k + 1)] = make_float2(p, ds);
            x[t][c] = ds;
          }
        uint32_t hi[4], lo[4];
        split2(x[0][0], x[0][1], &hi[0], &lo[0]);
        split2(x[0][2], x[0][3], &hi[1], &lo[1]);
        split2(x[1][0], x[1][1], &hi[2], &lo[2]);
        split2(x[1][2], x[1][3], &hi[3], &lo[3]);
        const unsigned char* kp = sK + (kb - cs + (lane & 15)) * RS +
                                  (lane >> 4) * 16;
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
          uint32_t f[4];
          ldsm4t(f, kp + t * 16);
          mma(o[t], hi[0], hi[1], hi[2], hi[3], f[0], f[1]);
          mma(o[t], lo[0], lo[1], lo[2], lo[3], f[0], f[1]);
          mma(o[t + 1], hi[0], hi[1], hi[2], hi[3], f[2], f[3]);
          mma(o[t + 1], lo[0], lo[1], lo[2], lo[3], f[2], f[3]);
        }
      }
      __syncthreads();
    }
    if (!wlive) return;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float* pa = s_dq + gr * D + 8 * t + 2 * tq;
      float* pb = pa + 8 * D;
      pa[0] += o[t][0];
      pa[1] += o[t][1];
      pb[0] += o[t][2];
      pb[1] += o[t][3];
    }
    __syncwarp();
    bf* dQ = reinterpret_cast<bf*>(a.dQ) + (rowbase + i0) * D;
    for (int e = lane; e < 16 * (D / 8); e += 32)
      if (e / (D / 8) < nrow)
        reinterpret_cast<uint4*>(dQ)[e] = pack16<bf>(s_dq + e * 8);
  }
}

// ------------------------------------------------------------- column pass
// A CTA owns 64 keys of one kv head, a warp 16: S^T and dP^T of 16 keys x 16
// rows at a time, then dV += P^T dO and dK += dS^T Q with P^T and dS^T in two
// parts straight from their accumulators.  Query rows are staged 64 at a
// time with their log-sum-exp, D and window start; the listed part is added
// at the end.
constexpr int kColWarps = 4;

template <int D, int NP>
struct ColSmem {
  static constexpr int RS = D * 2 + 16;
  static constexpr size_t tile = (size_t)64 * RS;
  static constexpr size_t bytes = (3 + NP) * tile + 64 * 12;
};

template <int D, int NP>
__global__ void __launch_bounds__(kColWarps * 32)
backward_columns_mma(Args a, int ntile) {
  using SM = ColSmem<D, NP>;
  constexpr int RS = SM::RS;
  constexpr int KS = D / 16, NT = D / 8;
  extern __shared__ __align__(16) unsigned char g_smem[];
  unsigned char* sK = g_smem;
  unsigned char* sV = sK + SM::tile;
  unsigned char* sQ = sV + SM::tile;
  unsigned char* sG = sQ + SM::tile;  // NP planes
  float* s_lse = reinterpret_cast<float*>(sG + NP * SM::tile);
  float* s_D = s_lse + 64;
  int* s_lo = reinterpret_cast<int*>(s_D + 64);
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int gr = lane >> 2, tq = lane & 3;
  const int L = a.L, nq = a.nq, G = a.Hq / a.Hkv;
  const int seg = blockIdx.x / ntile;
  const int j0 = (blockIdx.x % ntile) * 64;
  const int b = seg / a.Hkv, g = seg % a.Hkv;
  const int kw = j0 + wid * 16;  // the warp's first key
  const float sl2 = kLog2e / sqrtf((float)D), sc = 1.f / sqrtf((float)D);
  constexpr int kPieces = D * 2 / 16;
  auto stage = [&](unsigned char* dst, const bf* src, int first, int limit) {
    for (int e = threadIdx.x; e < 64 * kPieces; e += kColWarps * 32) {
      const int rr = e / kPieces, pc = e % kPieces;
      cp_async16(dst + rr * RS + pc * 16,
                 src + (int64_t)min(first + rr, limit - 1) * D + pc * 8);
    }
  };
  stage(sK, reinterpret_cast<const bf*>(a.K) + (int64_t)seg * L * D, j0, L);
  stage(sV, reinterpret_cast<const bf*>(a.V) + (int64_t)seg * L * D, j0, L);
  float dk[NT][4], dv[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int c = 0; c < 4; ++c) dk[t][c] = dv[t][c] = 0.f;
  const int jl = min(j0 + 63, L - 1);  // the CTA's last key
  const int chunks = (nq + kRowChunk - 1) / kRowChunk;
#pragma unroll 1
  for (int hh = 0; hh < G; ++hh) {
    const int h = g * G + hh;
    int wm = a.W_i ? a.wmax[b] : (a.W_h ? a.W_h[h] : a.W);
    wm = min(max(wm, 1), L);
    // rows whose position i has i - wm + 1 <= jl and i >= j0
    const int rmin = max(j0 - a.p0, 0);
    const int rmax = (int)min((int64_t)jl + wm - 1 - a.p0, (int64_t)nq - 1);
    const int64_t rowbase = ((int64_t)b * a.Hq + h) * nq;
#pragma unroll 1
    for (int rc = rmin / 64 * 64; rc <= rmax; rc += 64) {
      if (a.W_i && a.lows[b * chunks + rc / 64] > jl) continue;
      __syncthreads();  // the last chunk has been read
      stage(sQ, reinterpret_cast<const bf*>(a.Q) + rowbase * D, rc, nq);
#pragma unroll
      for (int p = 0; p < NP; ++p)
        stage(sG + p * SM::tile, a.g[p] + rowbase * D, rc, nq);
      if (threadIdx.x < 64) {
        const int r = rc + threadIdx.x;
        int w, lo = 0x7FFFFFFF;  // rows behind the last: no key
        float2 st = make_float2(0.f, 0.f);
        if (r < nq) {
          lo = window_lo(a, b, h, r, false, &w);
          st = a.stats[rowbase + r];
        }
        s_lo[threadIdx.x] = lo;
        s_lse[threadIdx.x] = st.x;
        s_D[threadIdx.x] = st.y;
      }
      cp_async_wait_all();
      __syncthreads();
#pragma unroll 1
      for (int rb = 0; rb < 64; rb += 16) {
        // does any of these 16 rows see any of the warp's 16 keys?
        const int rl = rb + (lane & 15);
        if (!__any_sync(kAll, a.p0 + rc + rl >= kw && s_lo[rl] <= kw + 15))
          continue;
        float x[2][4], dp[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) x[t][c] = dp[t][c] = 0.f;
        const int ar = wid * 16 + (lane & 15), ac = (lane >> 4) * 16;
        const int br = rb + (lane & 7) + ((lane >> 4) << 3);
        const int bc = ((lane >> 3) & 1) * 16;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t A[4], B[4];
          ldsm4(A, sK + ar * RS + ks * 32 + ac);
          ldsm4(B, sQ + br * RS + ks * 32 + bc);
          mma(x[0], A[0], A[1], A[2], A[3], B[0], B[1]);
          mma(x[1], A[0], A[1], A[2], A[3], B[2], B[3]);
          ldsm4(A, sV + ar * RS + ks * 32 + ac);
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            ldsm4(B, sG + p * SM::tile + br * RS + ks * 32 + bc);
            mma(dp[0], A[0], A[1], A[2], A[3], B[0], B[1]);
            mma(dp[1], A[0], A[1], A[2], A[3], B[2], B[3]);
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int rl2 = rb + 8 * t + 2 * tq + (c & 1);
            const int j = kw + gr + (c >= 2 ? 8 : 0);
            const bool ok = j <= a.p0 + rc + rl2 && j >= s_lo[rl2];
            const float p = ok ? exp2f(x[t][c] * sl2 - s_lse[rl2]) : 0.f;
            x[t][c] = p;
            dp[t][c] = p * (dp[t][c] - s_D[rl2]) * sc;
          }
        uint32_t ph[4], pl[4], dh[4], dl[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          split2(x[c >> 1][(c & 1) * 2], x[c >> 1][(c & 1) * 2 + 1], &ph[c],
                 &pl[c]);
          split2(dp[c >> 1][(c & 1) * 2], dp[c >> 1][(c & 1) * 2 + 1], &dh[c],
                 &dl[c]);
        }
        const int tr = (rb + (lane & 15)) * RS + (lane >> 4) * 16;
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
          uint32_t f[4];
          ldsm4t(f, sQ + tr + t * 16);
          mma(dk[t], dh[0], dh[1], dh[2], dh[3], f[0], f[1]);
          mma(dk[t], dl[0], dl[1], dl[2], dl[3], f[0], f[1]);
          mma(dk[t + 1], dh[0], dh[1], dh[2], dh[3], f[2], f[3]);
          mma(dk[t + 1], dl[0], dl[1], dl[2], dl[3], f[2], f[3]);
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            ldsm4t(f, sG + p * SM::tile + tr + t * 16);
            mma(dv[t], ph[0], ph[1], ph[2], ph[3], f[0], f[1]);
            mma(dv[t + 1], ph[0], ph[1], ph[2], ph[3], f[2], f[3]);
            if (p == 0) {  // lo x lo is below what two parts keep
              mma(dv[t], pl[0], pl[1], pl[2], pl[3], f[0], f[1]);
              mma(dv[t + 1], pl[0], pl[1], pl[2], pl[3], f[2], f[3]);
            }
          }
        }
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // K and V, if unused
  __syncthreads();
  // The listed part: a key's first range (`top`) and the later ranges'
  // shares (`carry`).  Up to kShort shares are added by the lanes that hold
  // the key; longer runs (the anchor's spans nq G / kRange ranges) first by
  // the whole CTA, in a fixed order.
  constexpr int kShort = 4;
  constexpr int kCols = 2 * D / 4, kParts = kColWarps * 32 / kCols;
  int2* s_span = reinterpret_cast<int2*>(sQ);
  float4* s_sum = reinterpret_cast<float4*>(sQ + 64 * 8);  // [parts][2 D]
  if (threadIdx.x < 64)
    s_span[threadIdx.x] = j0 + threadIdx.x < L
                              ? a.span[(int64_t)seg * L + j0 + threadIdx.x]
                              : make_int2(0, 0);
  __syncthreads();
#pragma unroll 1
  for (int kl = 0; kl < 64; ++kl) {
    const int2 sp = s_span[kl];
    const int f = sp.x / kRange, e = (sp.y - 1) / kRange;
    if (sp.y <= sp.x || e - f <= kShort) continue;  // the same for the CTA
    const int c4 = threadIdx.x % kCols, part = threadIdx.x / kCols;
    const float4* p = reinterpret_cast<const float4*>(
                          a.carry + (int64_t)seg * a.w.ranges * 2 * D) + c4;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int r = f + 1 + part; r <= e; r += kParts) {
      const float4 v = p[(int64_t)r * kCols];
      t.x += v.x;
      t.y += v.y;
      t.z += v.z;
      t.w += v.w;
    }
    s_sum[part * kCols + c4] = t;
    __syncthreads();
    if (kl >> 4 == wid && (kl & 7) == gr) {
      const float* q = reinterpret_cast<const float*>(s_sum) + 2 * tq;
      const int u = (kl >> 3) & 1;
#pragma unroll
      for (int part2 = 0; part2 < kParts; ++part2)
#pragma unroll
        for (int t2 = 0; t2 < NT; ++t2)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float k2 = q[part2 * 2 * D + 8 * t2 + c];
            const float v2 = q[part2 * 2 * D + D + 8 * t2 + c];
            dk[t2][c] += u ? 0.f : k2;
            dk[t2][2 + c] += u ? k2 : 0.f;
            dv[t2][c] += u ? 0.f : v2;
            dv[t2][2 + c] += u ? v2 : 0.f;
          }
    }
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int j = kw + gr + 8 * u;
    if (j >= L) continue;
    const int64_t col = (int64_t)seg * L + j;
    const int2 sp = s_span[wid * 16 + gr + 8 * u];
    if (sp.y > sp.x) {
      const int f = sp.x / kRange, e = (sp.y - 1) / kRange;
      const int r1 = e - f > kShort ? f : e;
      for (int r = f; r <= r1; ++r) {
        const float* p =
            (r == f ? a.top + col * 2 * D
                    : a.carry + ((int64_t)seg * a.w.ranges + r) * 2 * D) +
            2 * tq;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float2 k2 = *reinterpret_cast<const float2*>(p + 8 * t);
          const float2 v2 = *reinterpret_cast<const float2*>(p + D + 8 * t);
          dk[t][2 * u] += k2.x;
          dk[t][2 * u + 1] += k2.y;
          dv[t][2 * u] += v2.x;
          dv[t][2 * u + 1] += v2.y;
        }
      }
    }
    uint32_t* ok = reinterpret_cast<uint32_t*>(
        reinterpret_cast<bf*>(a.dK) + col * D + 2 * tq);
    uint32_t* ov = reinterpret_cast<uint32_t*>(
        reinterpret_cast<bf*>(a.dV) + col * D + 2 * tq);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      ok[4 * t] = pack2(dk[t][2 * u], dk[t][2 * u + 1]);
      ov[4 * t] = pack2(dv[t][2 * u], dv[t][2 * u + 1]);
    }
  }
}

// --------------------------------------------------------------- host side
template <int D, int NP>
cudaError_t rows_as(const Args& a, cudaStream_t s) {
  const int ntile = (a.nq + 63) / 64;
  const int64_t ctas = (int64_t)a.B * a.Hq * ntile;
  if (ctas > 0x7FFFFFFF) return cudaErrorNotSupported;
  const size_t smem = RowSmem<D, NP>::bytes(a.k);
  auto kern = backward_rows_mma<D, NP>;
  cudaError_t e = ensure_smem(kern, smem);
  if (e != cudaSuccess) return e;
  prof_before(s, "backward_rows");
  kern<<<(unsigned)ctas, kRowWarps * 32, smem, s>>>(a, ntile);
  prof_after(s);
  return cudaGetLastError();
}

template <int D, int NP>
cudaError_t columns_as(const Args& a, cudaStream_t s) {
  const int ntile = (a.L + 63) / 64;
  const int64_t ctas = (int64_t)a.w.segs * ntile;
  if (ctas > 0x7FFFFFFF) return cudaErrorNotSupported;
  auto kern = backward_columns_mma<D, NP>;
  cudaError_t e = ensure_smem(kern, ColSmem<D, NP>::bytes);
  if (e != cudaSuccess) return e;
  prof_before(s, "backward_columns");
  kern<<<(unsigned)ctas, kColWarps * 32, ColSmem<D, NP>::bytes, s>>>(a, ntile);
  prof_after(s);
  return cudaGetLastError();
}

}  // namespace

cudaError_t rows_mma_launch(const Args& a, int d, cudaStream_t s) {
  if (d == 64) return a.g[1] ? rows_as<64, 2>(a, s) : rows_as<64, 1>(a, s);
  return a.g[1] ? rows_as<128, 2>(a, s) : rows_as<128, 1>(a, s);
}

cudaError_t columns_mma_launch(const Args& a, int d, cudaStream_t s) {
  if (d == 64)
    return a.g[1] ? columns_as<64, 2>(a, s) : columns_as<64, 1>(a, s);
  return a.g[1] ? columns_as<128, 2>(a, s) : columns_as<128, 1>(a, s);
}

}  // namespace bwd
}  // namespace ca
