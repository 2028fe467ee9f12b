// Dropout of a layer's output with the residual added in the same pass, and
// its gradient: elementwise over n elements,
//
//   out[i] = (residual[i] +) (keep(i) ? x[i] * 256 / (256 - thr) : 0)
//   dx[i]  = keep(i) ? dout[i] * 256 / (256 - thr) : 0
//
// keep(i) is byte i & 15 of Philox4x32-10 at counter (i >> 4 low word,
// i >> 4 high word, site, 2^32 - 1) under the 64-bit seed, kept when >= thr.
// Nothing is stored: the backward draws the same decisions.  The attention's
// counters hold a batch index (< 65536) in word 3, so a seed shared with it
// never repeats a counter.
//
// One thread owns the 16 elements of one Philox call (32 bytes of bf16, 64
// of fp32).  The pass is bound by HBM: 2 or 3 tensors cross it once, and the
// ~100 integer operations a call needs (6 per element) fit beside that.
#include "common.cuh"
#include "dropout.cuh"

namespace bb {
namespace {

constexpr int kGroup = 16;  // elements per Philox call

struct DropArgs {
  const void* x;
  const void* residual;  // or null
  void* out;
  uint64_t n;
  uint32_t thr4;  // byte threshold in each byte
  float scale;    // 1 / keep probability
  uint32_t site, k0, k1;
};

__device__ __forceinline__ void load16(const float* p, float (&v)[kGroup]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float4 f = reinterpret_cast<const float4*>(p)[c];
    v[4 * c] = f.x; v[4 * c + 1] = f.y; v[4 * c + 2] = f.z; v[4 * c + 3] = f.w;
  }
}

__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&v)[kGroup]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[c];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * c + 2 * j] = __uint_as_float(w[j] << 16);
      v[8 * c + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ void store16(float* p, const float (&v)[kGroup]) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    reinterpret_cast<float4*>(p)[c] =
        make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}

__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[kGroup]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(v[8 * c + 2 * j], v[8 * c + 2 * j + 1]);
    reinterpret_cast<uint4*>(p)[c] = *reinterpret_cast<const uint4*>(h);
  }
}

// x and out, or residual and out, may be the same buffer: a thread reads its
// elements before it writes them and no other thread touches them.
template <typename T, bool kResidual>
__global__ void __launch_bounds__(256) out_dropout_kernel(const DropArgs a) {
  const uint64_t g = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const uint64_t i0 = g * kGroup;
  if (i0 >= a.n) return;
  const T* x = static_cast<const T*>(a.x) + i0;
  const T* r = static_cast<const T*>(a.residual) + i0;
  T* out = static_cast<T*>(a.out) + i0;
  if (i0 + kGroup <= a.n) {
    float v[kGroup], w[kGroup];
    load16(x, v);
    if (kResidual) load16(r, w);
    const uint32_t keep =
        keep16(philox4x32_10(make_uint4((uint32_t)g, (uint32_t)(g >> 32), a.site, 0xFFFFFFFFu),
                             a.k0, a.k1),
               a.thr4);
#pragma unroll
    for (int e = 0; e < kGroup; ++e) {
      // Selected, not multiplied: a dropped infinity or NaN leaves no trace.
      const bool k = (keep >> e) & 1u;
      if (kResidual)
        v[e] = k ? fmaf(v[e], a.scale, w[e]) : w[e];
      else
        v[e] = k ? v[e] * a.scale : 0.f;
    }
    store16(out, v);
  } else {
    // The last, partial group.
    const uint32_t keep =
        keep16(philox4x32_10(make_uint4((uint32_t)g, (uint32_t)(g >> 32), a.site, 0xFFFFFFFFu),
                             a.k0, a.k1),
               a.thr4);
    const int m = (int)(a.n - i0);
    for (int e = 0; e < m; ++e) {
      const bool k = (keep >> e) & 1u;
      const float w = kResidual ? to_f(r[e]) : 0.f;
      out[e] = from_f<T>(k ? (kResidual ? fmaf(to_f(x[e]), a.scale, w) : to_f(x[e]) * a.scale) : w);
    }
  }
}

template <typename T>
cudaError_t launch(const DropArgs& a, cudaStream_t s) {
  const uint64_t groups = (a.n + kGroup - 1) / kGroup;
  const unsigned grid = (unsigned)((groups + 255) / 256);
  if (a.residual)
    out_dropout_kernel<T, true><<<grid, 256, 0, s>>>(a);
  else
    out_dropout_kernel<T, false><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

int run_dropout(uint64_t n, int dtype, float rate, uint64_t seed, uint32_t site, const void* x,
                const void* residual, void* out, void* stream) {
  uint32_t thr;
  float scale;
  if (!resolve_dropout(rate, &thr, &scale)) return BB_ERR_INVALID;
  if (dtype != BB_F32 && dtype != BB_BF16) return BB_ERR_INVALID;
  if (n == 0 || !x || !out) return BB_ERR_INVALID;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(out)) return BB_ERR_INVALID;
  // One grid dimension of 256-thread blocks.
  if (n > (1ull << 42)) return BB_ERR_UNSUPPORTED;
  DropArgs a{x, residual, out, n, thr * 0x01010101u, scale, site, (uint32_t)seed,
             (uint32_t)(seed >> 32)};
  const cudaError_t e = dtype == BB_F32 ? launch<float>(a, (cudaStream_t)stream)
                                        : launch<__nv_bfloat16>(a, (cudaStream_t)stream);
  return e == cudaSuccess ? BB_OK : BB_ERR_CUDA;
}

}  // namespace
}  // namespace bb

extern "C" {

int bb_dropout_fwd(uint64_t n, int dtype, float rate, uint64_t seed, uint32_t site, const void* x,
                   const void* residual, void* out, void* stream) {
  return bb::run_dropout(n, dtype, rate, seed, site, x, residual, out, stream);
}

int bb_dropout_bwd(uint64_t n, int dtype, float rate, uint64_t seed, uint32_t site,
                   const void* dout, void* dx, void* stream) {
  return bb::run_dropout(n, dtype, rate, seed, site, dout, nullptr, dx, stream);
}

}  // extern "C"
