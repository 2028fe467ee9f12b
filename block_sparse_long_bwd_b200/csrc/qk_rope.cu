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
// Eight lanes own a row, four pairs each (both components of a pair, so the
// rotation needs no other lane); a warp takes four consecutive tokens of one
// head, 512 (bf16) or 1024 (fp32) contiguous bytes.  cos, sin and gamma of a
// lane's pairs depend on the token and not on the head, so a lane computes
// them once, folds gamma into them and walks its heads.  The 32 - rot_dim / 2
// "pairs" behind the rotated ones are neighbouring components at angle 0.
//
// Angles: theta^(-2i / rot_dim) / 2 pi, a fraction of a turn per position, is
// held as a 64-bit fixed-point number, so the product with the position
// wraps at whole turns exactly; its top 32 bits leave an angle error of
// 2^-24 half turns (the float conversion) at every 32-bit position.
#include <math.h>

#include "common.cuh"
#include "sm100.cuh"

namespace bb {
namespace {

using namespace sm100;

constexpr int kQkThreads = 256;
constexpr int kTokensPerBlock = kQkThreads / 8;
// Where a lane finds its pairs' components.
enum PairMode {
  kHalves = 0,       // (i, i + half), half a multiple of 4: two runs of four
  kInterleaved = 1,  // (2i, 2i + 1): one run of eight
  kScattered = 2     // (i, i + half), any half: one by one
};

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

// Components of pair p of a row (kHalves, from the lane's first pair on: the
// runs of four keep their order within an unrotated lane).
template <int kMode>
__device__ __forceinline__ int comp_a(const QkArgs& a, int p) {
  if (kMode == kInterleaved) return 2 * p;
  if (p < a.half) return p;
  if (kMode == kHalves) return a.rot + 2 * ((p & ~3) - a.half) + (p & 3);
  return a.rot + 2 * (p - a.half);
}
template <int kMode>
__device__ __forceinline__ int comp_b(const QkArgs& a, int p) {
  if (kMode == kInterleaved) return 2 * p + 1;
  if (p < a.half) return p + a.half;
  return comp_a<kMode>(a, p) + (kMode == kHalves ? 4 : 1);
}

// Four pairs of a row in registers: a[e], b[e] the components of pair e.
struct Pairs {
  float2 a[2], b[2];
};

// A lane's part of a row as it lies in memory.
template <typename T, int kMode>
struct Raw;
template <int kMode>
struct Raw<__nv_bfloat16, kMode> {
  uint32_t w[4];
  static __device__ __forceinline__ float2 lohi(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ __forceinline__ void load(const QkArgs& q, const __nv_bfloat16* row, int p, int oa,
                                       int ob) {
    if (kMode == kHalves) {
      const uint2 x = *reinterpret_cast<const uint2*>(row + oa);
      const uint2 y = *reinterpret_cast<const uint2*>(row + ob);
      w[0] = x.x; w[1] = x.y; w[2] = y.x; w[3] = y.y;
    } else if (kMode == kInterleaved) {
      const uint4 x = *reinterpret_cast<const uint4*>(row + oa);
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else {
      const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = r[comp_a<kMode>(q, p + e)] | ((uint32_t)r[comp_b<kMode>(q, p + e)] << 16);
    }
  }
  __device__ __forceinline__ Pairs get() const {
    Pairs o;
    if (kMode == kHalves) {
      o.a[0] = lohi(w[0]); o.a[1] = lohi(w[1]);
      o.b[0] = lohi(w[2]); o.b[1] = lohi(w[3]);
    } else {
      const float2 x[4] = {lohi(w[0]), lohi(w[1]), lohi(w[2]), lohi(w[3])};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        o.a[i] = make_float2(x[2 * i].x, x[2 * i + 1].x);
        o.b[i] = make_float2(x[2 * i].y, x[2 * i + 1].y);
      }
    }
    return o;
  }
  static __device__ __forceinline__ void store(const QkArgs& q, __nv_bfloat16* row, int p, int oa,
                                               int ob, const Pairs& v) {
    if (kMode == kHalves) {
      *reinterpret_cast<uint2*>(row + oa) =
          make_uint2(pack(v.a[0].x, v.a[0].y), pack(v.a[1].x, v.a[1].y));
      *reinterpret_cast<uint2*>(row + ob) =
          make_uint2(pack(v.b[0].x, v.b[0].y), pack(v.b[1].x, v.b[1].y));
    } else if (kMode == kInterleaved) {
      *reinterpret_cast<uint4*>(row + oa) =
          make_uint4(pack(v.a[0].x, v.b[0].x), pack(v.a[0].y, v.b[0].y),
                     pack(v.a[1].x, v.b[1].x), pack(v.a[1].y, v.b[1].y));
    } else {
      const float x[4] = {v.a[0].x, v.a[0].y, v.a[1].x, v.a[1].y};
      const float y[4] = {v.b[0].x, v.b[0].y, v.b[1].x, v.b[1].y};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        row[comp_a<kMode>(q, p + e)] = __float2bfloat16_rn(x[e]);
        row[comp_b<kMode>(q, p + e)] = __float2bfloat16_rn(y[e]);
      }
    }
  }
};
template <int kMode>
struct Raw<float, kMode> {
  float4 x, y;
  __device__ __forceinline__ void load(const QkArgs& q, const float* row, int p, int oa, int ob) {
    if (kMode != kScattered) {
      x = *reinterpret_cast<const float4*>(row + oa);
      y = *reinterpret_cast<const float4*>(row + ob);
    } else {
      x = make_float4(row[comp_a<kMode>(q, p)], row[comp_a<kMode>(q, p + 1)],
                      row[comp_a<kMode>(q, p + 2)], row[comp_a<kMode>(q, p + 3)]);
      y = make_float4(row[comp_b<kMode>(q, p)], row[comp_b<kMode>(q, p + 1)],
                      row[comp_b<kMode>(q, p + 2)], row[comp_b<kMode>(q, p + 3)]);
    }
  }
  __device__ __forceinline__ Pairs get() const {
    Pairs o;
    if (kMode == kInterleaved) {
      o.a[0] = make_float2(x.x, x.z); o.a[1] = make_float2(y.x, y.z);
      o.b[0] = make_float2(x.y, x.w); o.b[1] = make_float2(y.y, y.w);
    } else {
      o.a[0] = make_float2(x.x, x.y); o.a[1] = make_float2(x.z, x.w);
      o.b[0] = make_float2(y.x, y.y); o.b[1] = make_float2(y.z, y.w);
    }
    return o;
  }
  static __device__ __forceinline__ void store(const QkArgs& q, float* row, int p, int oa, int ob,
                                               const Pairs& v) {
    if (kMode == kInterleaved) {
      *reinterpret_cast<float4*>(row + oa) =
          make_float4(v.a[0].x, v.b[0].x, v.a[0].y, v.b[0].y);
      *reinterpret_cast<float4*>(row + ob) =
          make_float4(v.a[1].x, v.b[1].x, v.a[1].y, v.b[1].y);
    } else if (kMode == kHalves) {
      *reinterpret_cast<float4*>(row + oa) = make_float4(v.a[0].x, v.a[0].y, v.a[1].x, v.a[1].y);
      *reinterpret_cast<float4*>(row + ob) = make_float4(v.b[0].x, v.b[0].y, v.b[1].x, v.b[1].y);
    } else {
      const float s[4] = {v.a[0].x, v.a[0].y, v.a[1].x, v.a[1].y};
      const float t[4] = {v.b[0].x, v.b[0].y, v.b[1].x, v.b[1].y};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        row[comp_a<kMode>(q, p + e)] = s[e];
        row[comp_b<kMode>(q, p + e)] = t[e];
      }
    }
  }
};

// Sum over the eight lanes of a row (a fixed tree: every lane gets the same).
__device__ __forceinline__ float sum8(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x;
}

__device__ __forceinline__ float2 neg2(float2 x) { return make_float2(-x.x, -x.y); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A lane reads its own components of a row before it writes them and no other
// lane touches them, so the outputs may be the inputs.
template <typename T, int kMode, bool kBwd>
__global__ void __launch_bounds__(kQkThreads, kBwd ? 3 : 4)
    qk_rope_kernel(const __grid_constant__ QkArgs a) {
  constexpr int kAhead = kBwd || sizeof(T) == 4 ? 2 : 4;
  __shared__ float red[kQkThreads / 32][64];
  const int lane = threadIdx.x & 31, p0 = (lane & 7) * 4;
  const int t = blockIdx.y / a.hsplit;         // 0: q, 1: k
  const int split = blockIdx.y % a.hsplit;
  const int h0 = (int)((long long)a.H * split / a.hsplit);
  const int h1 = (int)((long long)a.H * (split + 1) / a.hsplit);
  const long long tokens = (long long)a.B * a.L;
  const int oa = comp_a<kMode>(a, p0);
  const int ob = kMode == kInterleaved ? oa + 4 : comp_b<kMode>(a, p0);

  float2 ga[2], gb[2], dga[2], dgb[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    ga[i] = gb[i] = both(1.f);
    dga[i] = dgb[i] = both(0.f);
    if (a.gamma[t]) {
      const float* g = a.gamma[t];
      ga[i] = make_float2(__ldg(g + comp_a<kMode>(a, p0 + 2 * i)),
                          __ldg(g + comp_a<kMode>(a, p0 + 2 * i + 1)));
      gb[i] = make_float2(__ldg(g + comp_b<kMode>(a, p0 + 2 * i)),
                          __ldg(g + comp_b<kMode>(a, p0 + 2 * i + 1)));
    }
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
    float2 c[2], s[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float co = 1.f, si = 0.f;
      if (p0 + e < a.half) {
        const uint64_t turns = a.turn[p0 + e] * (uint64_t)(int64_t)pos;
        sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &si, &co);
      }
      (e & 1 ? c[e >> 1].y : c[e >> 1].x) = co;
      (e & 1 ? s[e >> 1].y : s[e >> 1].x) = si;
    }
    // Forward: y_a = r (x_a (ga c) - x_b (gb s)), y_b = r (x_b (gb c) + x_a (ga s)).
    float2 ca[2], sa[2], cb[2], sb[2];
    if (!kBwd) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ca[i] = mul2(ga[i], c[i]);
        sa[i] = mul2(ga[i], s[i]);
        cb[i] = mul2(gb[i], c[i]);
        sb[i] = neg2(mul2(gb[i], s[i]));
      }
    }
    const size_t step = (size_t)a.L * kHeadDim;
    size_t off = (((size_t)b * a.H + h0) * a.L + l) * kHeadDim;
    const T* in = static_cast<const T*>(a.in[t]);
    const T* dy = static_cast<const T*>(a.dy[t]);
    T* out = static_cast<T*>(a.out[t]);
    // A few heads' rows are loaded before the first is used: inputs and
    // outputs may alias, so the compiler cannot move the loads up.
    for (int h = h0; h < h1; h += kAhead, off += kAhead * step) {
      Raw<T, kMode> rx[kAhead], rd[kBwd ? kAhead : 1];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (h + u < h1) {
          rx[u].load(a, in + off + u * step, p0, oa, ob);
          if (kBwd) rd[kBwd ? u : 0].load(a, dy + off + u * step, p0, oa, ob);
        }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (h + u >= h1) break;
        const Pairs x = rx[u].get();
        Pairs y;
        float2 sq = mul2(x.a[0], x.a[0]);
        sq = fma2(x.a[1], x.a[1], sq);
        sq = fma2(x.b[0], x.b[0], sq);
        sq = fma2(x.b[1], x.b[1], sq);
        const float r = rsqrtf(fmaf(sum8(sq.x + sq.y), 1.f / kHeadDim, a.eps));
        if (!kBwd) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            y.a[i] = mul2(both(r), fma2(x.b[i], sb[i], mul2(x.a[i], ca[i])));
            y.b[i] = mul2(both(r), fma2(x.a[i], sa[i], mul2(x.b[i], cb[i])));
          }
        } else {
          const Pairs d = rd[kBwd ? u : 0].get();
          float2 va[2], vb[2], vx = both(0.f);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // g = R^T dy; v = gamma g
            const float2 g = fma2(d.b[i], s[i], mul2(d.a[i], c[i]));
            const float2 k = fma2(d.a[i], neg2(s[i]), mul2(d.b[i], c[i]));
            va[i] = mul2(g, ga[i]);
            vb[i] = mul2(k, gb[i]);
            vx = fma2(va[i], x.a[i], vx);
            vx = fma2(vb[i], x.b[i], vx);
            if (live) {
              dga[i] = fma2(g, mul2(both(r), x.a[i]), dga[i]);
              dgb[i] = fma2(k, mul2(both(r), x.b[i]), dgb[i]);
            }
          }
          const float m = -sum8(vx.x + vx.y) * r * r * (1.f / kHeadDim);  // -mean(v n) r
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            y.a[i] = mul2(both(r), fma2(both(m), x.a[i], va[i]));
            y.b[i] = mul2(both(r), fma2(both(m), x.b[i], vb[i]));
          }
        }
        if (live) Raw<T, kMode>::store(a, out + off + u * step, p0, oa, ob, y);
      }
    }
  }

  if (kBwd) {
    // The block's sum of g n per component, in a fixed order: over the
    // warp's four tokens, then over its warps.
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float x = e & 1 ? dga[e >> 1].y : dga[e >> 1].x;
      float y = e & 1 ? dgb[e >> 1].y : dgb[e >> 1].x;
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      y += __shfl_xor_sync(0xffffffffu, y, 8);
      y += __shfl_xor_sync(0xffffffffu, y, 16);
      if (lane < 8) {
        red[threadIdx.x >> 5][comp_a<kMode>(a, p0 + e)] = x;
        red[threadIdx.x >> 5][comp_b<kMode>(a, p0 + e)] = y;
      }
    }
    __syncthreads();
    if (threadIdx.x < 64) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kQkThreads / 32; ++w) sum += red[w][threadIdx.x];
      a.part[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * 64 + threadIdx.x] = sum;
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

// Head ranges per tensor: enough blocks to fill the GPU (four 256-thread
// blocks on each of 148 SMs), at most one per head; longer walks share the
// angles.
int head_splits(const bb_qk_desc& d, bool bwd) {
  const int want = 148 * 4, have = 2 * token_blocks(d, bwd);
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
  const long double q = a.half ? powl((long double)d.theta, -2.0L / d.rot_dim) : 0.0L;
  long double f = 18446744073709551616.0L / tau;
  for (int i = 0; i < a.half; ++i, f *= q) a.turn[i] = (uint64_t)f;
  return a;
}

template <typename T, bool kBwd>
cudaError_t launch_mode(const bb_qk_desc& d, const QkArgs& a, cudaStream_t s) {
  const dim3 grid(token_blocks(d, kBwd), 2 * a.hsplit);
  if (d.interleaved || a.rot == 0)
    qk_rope_kernel<T, kInterleaved, kBwd><<<grid, kQkThreads, 0, s>>>(a);
  else if (a.half % 4 == 0)
    qk_rope_kernel<T, kHalves, kBwd><<<grid, kQkThreads, 0, s>>>(a);
  else
    qk_rope_kernel<T, kScattered, kBwd><<<grid, kQkThreads, 0, s>>>(a);
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
