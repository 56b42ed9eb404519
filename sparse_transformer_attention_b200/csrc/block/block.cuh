// The operators around the attention (internal): per-head norm with the
// position rotation, its backward pass, and the prefill's backward pass.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../common.cuh"
#include "../profile.cuh"

namespace ca {

// Kernels of one call follow each other by programmatic dependent launch:
// the next one's CTAs are set up while the last CTAs of the one before run.
// Every kernel calls chain() before it touches memory; it returns when the
// kernels before are complete and their writes visible, so the order is that
// of plain launches.
__device__ __forceinline__ void chain() {
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;" ::
                   : "memory");
}

template <typename... P, typename... V>
cudaError_t launch(const char* name, void (*kern)(P...), dim3 grid,
                   int threads, size_t smem, cudaStream_t s, V... v) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  prof_before(s, name);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<P>(v)...);
  prof_after(s);
  return e;
}

// N consecutive elements as floats: a multiple of 16 bytes (16-byte aligned),
// or eight bytes of bf16.
template <typename T, int N>
__device__ __forceinline__ void load_row(const T* p, float* f) {
  constexpr int kPer = Elem<T>::kPer16B;
  if constexpr (N < kPer) {
    load_f32<T, N>(p, f);
  } else {
#pragma unroll
    for (int v = 0; v < N / kPer; ++v) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + v);
      Elem<T>::unpack(u, f + v * kPer);
    }
  }
}

// 16 bytes of T from floats, each rounded to nearest even once.
template <typename T>
__device__ __forceinline__ uint4 pack16(const float* f);
template <>
__device__ __forceinline__ uint4 pack16<float>(const float* f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]),
                    __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 pack16<__nv_bfloat16>(const float* f) {
  uint4 u;
  uint32_t* w = &u.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return u;
}
template <typename T, int N>
__device__ __forceinline__ void store_row(T* p, const float* f) {
  constexpr int kPer = Elem<T>::kPer16B;
#pragma unroll
  for (int v = 0; v < N / kPer; ++v)
    reinterpret_cast<uint4*>(p)[v] = pack16<T>(f + v * kPer);
}

// ------------------------------------------------------- norm and rotation

// Rows of d contiguous elements of a [B, n, heads] grid, strides in elements.
struct Rows {
  void* p;
  int64_t sb, st, sh;
};

struct NormRopeArgs {
  Rows x[3];   // q, k, v before the operator (backward: q, k)
  Rows y[3];   // Q, K, V behind it (backward: their gradients, read)
  Rows dx[3];  // backward: gradients of q, k, v, written
  int B, n, Hq, Hkv;
  const void* w[2];     // norm weights [d] of q and k, NULL = no norm
  int w_bf16;
  float eps;
  const float* inv_freq;  // [rot / 2]
  int rot;                // rotated leading elements of each row
  int interleaved;        // pairs (2c, 2c+1) instead of (c, c + rot/2)
  const int32_t* positions;  // [B, n] or NULL (pos0 + t)
  int pos0;
  float* partial;       // backward: [CTAs, 2, d] weight-gradient partials
  void* dw[2];          // backward: [d] weight gradients
};

// CTAs of the backward pass at most (they keep weight-gradient sums in
// registers over many tokens; one partial row pair each).
constexpr int kNormRopeMaxCtas = 592;
cudaError_t norm_rope_launch(NormRopeArgs a, bool bf16, int d,
                             cudaStream_t s);
cudaError_t norm_rope_backward_launch(NormRopeArgs a, bool bf16, int d,
                                      cudaStream_t s);

// ------------------------------------------------- the prefill's backward

struct BackwardArgs {
  const void* Q;   // [B, Hq, nq, d]
  const void* K;   // [B, Hkv, L, d]
  const void* V;
  const void* dO;  // [B, Hq, nq, d]
  int do_bf16;
  int B, nq, L, p0, Hq, Hkv, W, k;
  const int32_t* W_i;  // [B, nq] or NULL
  const int32_t* W_h;  // [Hq] or NULL
  const int32_t* idx;        // [B, Hq, nq, C_max]
  const int32_t* idx_count;  // [B, Hq, nq]
  int C_max;
  void* dQ;
  void* dK;
  void* dV;
  uint32_t* status;
};

// Bytes of workspace (the status area included); 0 if one kv head's list
// does not fit 31-bit entry numbers.
size_t backward_workspace(bool bf16, bool do_bf16, int B, int nq, int L,
                          int Hq, int Hkv, int d, int k);
cudaError_t backward_launch(const BackwardArgs& a, bool bf16, int d, void* ws,
                            cudaStream_t s);

}  // namespace ca
