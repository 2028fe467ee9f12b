// RMS norm of each head's queries and keys and the rotary position rotation,
// in one pass between the Q/K/V projection and the attention, and the
// gradient of both.  For a row x of 64 components at position p:
//
//   r = rsqrt(mean(x^2) + eps),  n = x r,  u = gamma n
//   y[a] = u[a] cos t_i - u[b] sin t_i,  y[b] = u[b] cos t_i + u[a] sin t_i
//
// for pair i = (a, b) of the first rot_dim components at angle
// t_i = p theta^(-2i / rot_dim); the other components pass as they are.
// Backward, from dy:
//
//   g = R^T dy,  dgamma = sum over rows of g n,  v = gamma g,
//   dx = r (v - n mean(v n))
//
// Eight lanes own a row (eight components each); a warp takes four
// consecutive tokens of one head, 512 (bf16) or 1024 (fp32) contiguous
// bytes.  cos, sin and gamma of a lane's components depend on the token and
// not on the head, so a lane computes them once, folds gamma into them and
// walks its heads.  A component's partner sits eight components or a
// multiple away (shuffle), beside it (interleaved pairs), or, for the other
// rot_dim, is read again from L1.
//
// Angles: theta^(-2i / rot_dim) / 2 pi, a fraction of a turn per position, is
// held as a 64-bit fixed-point number, so the product with the position
// wraps at whole turns exactly; its top 32 bits leave an angle error of
// 2^-24 half turns (the float conversion) at every 32-bit position.
#include <math.h>

#include "common.cuh"

namespace bb {
namespace {

constexpr int kQkThreads = 256;
constexpr int kTokensPerBlock = kQkThreads / 8;
// Where a lane's partner components come from.
enum PairMode { kShuffle = 0, kInterleaved = 1, kReload = 2 };

struct QkArgs {
  const void* in[2];        // q, k
  const void* dy[2];        // backward: gradients of the rotated q, k
  void* out[2];             // forward: rotated q, k; backward: dq, dk
  const float* gamma[2];    // [64] or null (ones)
  const int32_t* pos;       // [B][L] or null (the index in the sequence)
  float* part;              // backward: [blocks][64] sums for dgamma, q's blocks then k's
  int B, H, L;
  int hsplit;               // head ranges a tensor's heads are split into
  int rot, half;            // rotated components; half of it
  float eps;
  uint64_t turn[32];        // turns per position of pair i, 64-bit fixed point
};

template <typename T>
struct Row8;  // eight components of a row in registers
template <>
struct Row8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ Row8 shfl(int src) const {
    Row8 o;
    o.u.x = __shfl_sync(0xffffffffu, u.x, src);
    o.u.y = __shfl_sync(0xffffffffu, u.y, src);
    o.u.z = __shfl_sync(0xffffffffu, u.z, src);
    o.u.w = __shfl_sync(0xffffffffu, u.w, src);
    return o;
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8]) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
  }
};
template <>
struct Row8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ Row8 shfl(int src) const {
    Row8 o;
    o.a = make_float4(__shfl_sync(0xffffffffu, a.x, src), __shfl_sync(0xffffffffu, a.y, src),
                      __shfl_sync(0xffffffffu, a.z, src), __shfl_sync(0xffffffffu, a.w, src));
    o.b = make_float4(__shfl_sync(0xffffffffu, b.x, src), __shfl_sync(0xffffffffu, b.y, src),
                      __shfl_sync(0xffffffffu, b.z, src), __shfl_sync(0xffffffffu, b.w, src));
    return o;
  }
  static __device__ __forceinline__ void store(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// Sum over the eight lanes of a row (a fixed tree: every lane gets the same).
__device__ __forceinline__ float sum8(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x;
}

// Index of the partner of component j, or j itself when it is not rotated.
template <int kMode>
__device__ __forceinline__ int partner_of(const QkArgs& a, int j) {
  if (j >= a.rot) return j;
  if (kMode == kInterleaved) return j ^ 1;
  return j < a.half ? j + a.half : j - a.half;
}

// The partners' values of a lane's eight components, given its own.
template <typename T, int kMode>
__device__ __forceinline__ void partners(const QkArgs& a, const Row8<T>& own,
                                         const float (&v)[8], const T* row, int c0, int src,
                                         float (&p)[8]) {
  if (kMode == kShuffle) {
    own.shfl(src).get(p);
  } else if (kMode == kInterleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = v[e ^ 1];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = to_f(row[partner_of<kMode>(a, c0 + e)]);
  }
  // An unrotated component has no partner (its sine is 0, but 0 times an
  // infinity is not).
  if (a.rot < kHeadDim) {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = c0 + e < a.rot ? p[e] : 0.f;
  }
}

template <typename T, int kMode, bool kBwd>
__global__ void __launch_bounds__(kQkThreads) qk_rope_kernel(const __grid_constant__ QkArgs a) {
  __shared__ float red[kQkThreads / 32][64];
  const int lane = threadIdx.x & 31, sub = lane & 7, c0 = sub * 8;
  const int t = blockIdx.y / a.hsplit;         // 0: q, 1: k
  const int split = blockIdx.y % a.hsplit;
  const int h0 = (int)((long long)a.H * split / a.hsplit);
  const int h1 = (int)((long long)a.H * (split + 1) / a.hsplit);
  const long long tokens = (long long)a.B * a.L;
  // Lane that holds the partners (whole lanes swap when half is a multiple
  // of eight).
  const int hl = a.half >> 3;
  const int src = kMode != kShuffle || c0 >= a.rot ? lane : (sub < hl ? lane + hl : lane - hl);

  float gam[8], dg[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    gam[e] = a.gamma[t] ? __ldg(a.gamma[t] + c0 + e) : 1.f;
    dg[e] = 0.f;
  }

  for (long long tb = (long long)blockIdx.x * kTokensPerBlock; tb < tokens;
       tb += (long long)gridDim.x * kTokensPerBlock) {
    const long long token = tb + (threadIdx.x >> 3);
    // Lanes past the last token redo the last one and store nothing, so that
    // every lane reaches the shuffles.
    const bool live = token < tokens;
    const long long tok = live ? token : tokens - 1;
    const int b = (int)(tok / a.L), l = (int)(tok % a.L);
    const int pos = a.pos ? __ldg(a.pos + tok) : l;
    // Forward: y = r (x ca + partner sa), gamma folded in.  Backward:
    // g = dy ca - partner sa without gamma.
    float ca[8], sa[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = c0 + e;
      float c = 1.f, s = 0.f;
      if (j < a.rot) {
        const bool second = kMode == kInterleaved ? (j & 1) : j >= a.half;
        const int i = kMode == kInterleaved ? j >> 1 : (second ? j - a.half : j);
        const uint64_t turns = a.turn[i] * (uint64_t)(int64_t)pos;
        sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
        if (!second) s = -s;
      }
      if (kBwd) {
        ca[e] = c;
        sa[e] = s;
      } else {
        const int jp = partner_of<kMode>(a, j);
        ca[e] = gam[e] * c;
        sa[e] = (a.gamma[t] ? __ldg(a.gamma[t] + jp) : 1.f) * s;
      }
    }
    const size_t step = (size_t)a.L * kHeadDim;
    size_t off = (((size_t)b * a.H + h0) * a.L + l) * kHeadDim;
    const T* in = static_cast<const T*>(a.in[t]);
    T* out = static_cast<T*>(a.out[t]);
    if (!kBwd) {
#pragma unroll 4
      for (int h = h0; h < h1; ++h, off += step) {
        Row8<T> x;
        x.load(in + off + c0);
        float v[8], p[8], ss = 0.f;
        x.get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
        const float r = rsqrtf(fmaf(sum8(ss), 1.f / kHeadDim, a.eps));
        partners<T, kMode>(a, x, v, in + off, c0, src, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = r * fmaf(v[e], ca[e], p[e] * sa[e]);
        // out may be the input: with kReload other lanes read these
        // components, so the row is read whole before any of it is written.
        if (kMode == kReload) __syncwarp();
        if (live) Row8<T>::store(out + off + c0, v);
      }
    } else {
      const T* dy = static_cast<const T*>(a.dy[t]);
#pragma unroll 2
      for (int h = h0; h < h1; ++h, off += step) {
        Row8<T> x, d;
        x.load(in + off + c0);
        d.load(dy + off + c0);
        float v[8], g[8], p[8], ss = 0.f, vx = 0.f;
        x.get(v);
        d.get(g);
        partners<T, kMode>(a, d, g, dy + off, c0, src, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          g[e] = fmaf(g[e], ca[e], -p[e] * sa[e]);
          ss = fmaf(v[e], v[e], ss);
          vx = fmaf(g[e] * gam[e], v[e], vx);
        }
        const float r = rsqrtf(fmaf(sum8(ss), 1.f / kHeadDim, a.eps));
        const float m = sum8(vx) * r * r * (1.f / kHeadDim);  // mean(v n) r
        if (kMode == kReload) __syncwarp();
        if (live) {
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            dg[e] = fmaf(g[e] * r, v[e], dg[e]);
            o[e] = r * fmaf(-m, v[e], g[e] * gam[e]);
          }
          Row8<T>::store(out + off + c0, o);
        }
      }
    }
  }

  if (kBwd) {
    // The block's sum of g n per component, in a fixed order: over the
    // warp's four tokens, then over its warps.
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dg[e] += __shfl_xor_sync(0xffffffffu, dg[e], 8);
      dg[e] += __shfl_xor_sync(0xffffffffu, dg[e], 16);
    }
    if (lane < 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) red[threadIdx.x >> 5][c0 + e] = dg[e];
    }
    __syncthreads();
    if (threadIdx.x < 64) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kQkThreads / 32; ++w) s += red[w][threadIdx.x];
      a.part[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * 64 + threadIdx.x] = s;
    }
  }
}

// dgamma of q (block.y 0) and k (1): the blocks' partial sums, in order.
// Eight components per block, 32 partial rows at a time.
__global__ void __launch_bounds__(256)
    qk_dgamma_kernel(const float* part, int rows, float* dgq, float* dgk) {
  __shared__ float red[32][8];
  const int c = threadIdx.x & 7, g = threadIdx.x >> 3;
  const float* p = part + (size_t)blockIdx.y * rows * 64 + blockIdx.x * 8 + c;
  float s = 0.f;
  for (int i = g; i < rows; i += 32) s += p[(size_t)i * 64];
  red[g][c] = s;
  __syncthreads();
  if (g == 0) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += red[i][c];
    float* out = blockIdx.y ? dgk : dgq;
    if (out) out[blockIdx.x * 8 + c] = t;
  }
}

// Blocks along the tokens (the backward's partial rows per head range).  A
// block past the cap walks several token tiles.
int token_blocks(const bb_qk_desc& d, bool bwd) {
  const long long tiles = ((long long)d.B * d.L + kTokensPerBlock - 1) / kTokensPerBlock;
  const long long cap = bwd ? 1024 : 1 << 20;
  return (int)(tiles < cap ? tiles : cap);
}

// Head ranges per tensor: enough blocks to fill the GPU (eight 256-thread
// blocks on each of 148 SMs), at most one per head; longer walks share the
// angles.
int head_splits(const bb_qk_desc& d, bool bwd) {
  const int want = 148 * 8, have = 2 * token_blocks(d, bwd);
  int s = (want + have - 1) / have;
  return s < d.H ? s : d.H;
}

int check_desc(const bb_qk_desc* d) {
  if (!d) return BB_ERR_INVALID;
  if (d->B <= 0 || d->H <= 0 || d->L <= 0 || d->d <= 0) return BB_ERR_INVALID;
  if (d->dtype != BB_F32 && d->dtype != BB_BF16) return BB_ERR_INVALID;
  if (!(d->eps >= 0.f) || !isfinite(d->eps)) return BB_ERR_INVALID;
  if (d->rot_dim < 0 || d->rot_dim > d->d || d->rot_dim % 2 != 0) return BB_ERR_INVALID;
  if (d->interleaved != 0 && d->interleaved != 1) return BB_ERR_INVALID;
  if (d->rot_dim > 0 && !(d->theta >= 1.0 && isfinite(d->theta))) return BB_ERR_INVALID;
  if (d->d != kHeadDim || d->H > 32767) return BB_ERR_UNSUPPORTED;
  return BB_OK;
}

QkArgs make_args(const bb_qk_desc& d, bool bwd) {
  QkArgs a{};
  a.B = d.B;
  a.H = d.H;
  a.L = d.L;
  a.hsplit = head_splits(d, bwd);
  a.rot = d.rot_dim;
  a.half = d.rot_dim / 2;
  a.eps = d.eps;
  // Turns per position as a fraction of 2^64, in extended precision: at
  // most 1 / 2 pi, so it fits.
  const long double tau = 6.283185307179586476925286766559005768L;
  for (int i = 0; i < a.half; ++i)
    a.turn[i] = (uint64_t)(powl((long double)d.theta, -2.0L * i / d.rot_dim) / tau *
                           18446744073709551616.0L);
  return a;
}

template <typename T, bool kBwd>
cudaError_t launch_mode(const bb_qk_desc& d, const QkArgs& a, cudaStream_t s) {
  const dim3 grid(token_blocks(d, kBwd), 2 * a.hsplit);
  if (d.interleaved || a.rot == 0)
    qk_rope_kernel<T, kInterleaved, kBwd><<<grid, kQkThreads, 0, s>>>(a);
  else if (a.half % 8 == 0)
    qk_rope_kernel<T, kShuffle, kBwd><<<grid, kQkThreads, 0, s>>>(a);
  else
    qk_rope_kernel<T, kReload, kBwd><<<grid, kQkThreads, 0, s>>>(a);
  return cudaGetLastError();
}

size_t part_floats(const bb_qk_desc& d) {
  return (size_t)2 * head_splits(d, true) * token_blocks(d, true) * 64;
}

}  // namespace
}  // namespace bb

using namespace bb;

extern "C" {

int bb_qk_norm_rope_workspace_size(const bb_qk_desc* desc, size_t* bytes) {
  if (!bytes) return BB_ERR_INVALID;
  const int st = check_desc(desc);
  if (st != BB_OK) return st;
  *bytes = part_floats(*desc) * sizeof(float);
  return BB_OK;
}

int bb_qk_norm_rope_fwd(const bb_qk_desc* desc, const void* q, const void* k,
                        const float* gamma_q, const float* gamma_k, const int32_t* positions,
                        void* q_out, void* k_out, void* stream) {
  const int st = check_desc(desc);
  if (st != BB_OK) return st;
  if (!q || !k || !q_out || !k_out) return BB_ERR_INVALID;
  const void* ptrs[] = {q, k, gamma_q, gamma_k, positions, q_out, k_out};
  for (const void* p : ptrs)
    if (!aligned16(p)) return BB_ERR_INVALID;
  QkArgs a = make_args(*desc, false);
  a.in[0] = q;
  a.in[1] = k;
  a.out[0] = q_out;
  a.out[1] = k_out;
  a.gamma[0] = gamma_q;
  a.gamma[1] = gamma_k;
  a.pos = positions;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = desc->dtype == BB_F32 ? launch_mode<float, false>(*desc, a, s)
                                              : launch_mode<__nv_bfloat16, false>(*desc, a, s);
  return e == cudaSuccess ? BB_OK : BB_ERR_CUDA;
}

int bb_qk_norm_rope_bwd(const bb_qk_desc* desc, const void* q, const void* k,
                        const float* gamma_q, const float* gamma_k, const int32_t* positions,
                        const void* dq_out, const void* dk_out, void* dq, void* dk,
                        float* dgamma_q, float* dgamma_k, void* workspace,
                        size_t workspace_bytes, void* stream) {
  const int st = check_desc(desc);
  if (st != BB_OK) return st;
  if (!q || !k || !dq_out || !dk_out || !dq || !dk) return BB_ERR_INVALID;
  const void* ptrs[] = {q, k, gamma_q, gamma_k, positions, dq_out, dk_out, dq, dk,
                        dgamma_q, dgamma_k, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return BB_ERR_INVALID;
  if (!workspace || workspace_bytes < part_floats(*desc) * sizeof(float))
    return BB_ERR_WORKSPACE;
  QkArgs a = make_args(*desc, true);
  a.in[0] = q;
  a.in[1] = k;
  a.dy[0] = dq_out;
  a.dy[1] = dk_out;
  a.out[0] = dq;
  a.out[1] = dk;
  a.gamma[0] = gamma_q;
  a.gamma[1] = gamma_k;
  a.pos = positions;
  a.part = static_cast<float*>(workspace);
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = desc->dtype == BB_F32 ? launch_mode<float, true>(*desc, a, s)
                                        : launch_mode<__nv_bfloat16, true>(*desc, a, s);
  if (e != cudaSuccess) return BB_ERR_CUDA;
  if (dgamma_q || dgamma_k) {
    qk_dgamma_kernel<<<dim3(8, 2), 256, 0, s>>>(a.part, a.hsplit * token_blocks(*desc, true),
                                                dgamma_q, dgamma_k);
    if (cudaGetLastError() != cudaSuccess) return BB_ERR_CUDA;
  }
  return BB_OK;
}

}  // extern "C"
