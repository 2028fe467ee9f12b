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
// rotation needs no other lane); a warp takes four consecutive tokens and
// walks the heads of q, then of k.  cos and sin of a lane's pairs depend on the
// token alone, so a lane computes them once for all its heads.  The
// 32 - rot_dim / 2 "pairs" behind the rotated ones are neighbouring components
// at angle 0.
//
// The pass is bound by HBM (2 or 3 tensors cross it), and what it needs for
// that is enough bytes in flight: each warp copies its rows a few heads ahead
// into shared memory (cp.async, 16 bytes a lane), without registers or
// barriers between warps.  Loading a few heads into registers instead took
// 28.0 and 85.6 us where this takes 24.9 and 59.4 (forward of 4 x 16 x 4096
// rows of q and k, gradients of 8 x 12 x 4096, bf16, replayed in a graph; as
// calls 25.9 and 62.5: 5.2 and 4.8 TB/s).  The
// issue slots of the forward are then 68 % busy, those of the gradients 59 %
// (unpacking, the rotation, two sums over the row); two heads at a time took
// the gradients from 65.8 us (and the fp32 ones of 12 x 5003 from 21.2 to 22.1).
//
// Angles: theta^(-2i / rot_dim) / 2 pi, a fraction of a turn per position, is
// held as a 64-bit fixed-point number, so the product with the position
// wraps at whole turns exactly.  Of its top 32 bits fp32 takes 24 as the
// argument of cos and sin; the rest turns them a little further, to first
// order (dq, dk of 12 x 5003 rows in fp32: 6.8e-8 off as the formula in fp32
// is, 7.2e-8 without; the time is the same).
#include <math.h>

#include "layer.cuh"

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
  float* part;              // backward: [2][blocks][64] sums for dgamma of q and k
  int B, H, L;
  int splits;               // ranges the 2 H heads of q and k are split into
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

// A warp's four rows in shared memory, 16-byte chunks permuted so that the
// lanes' reads meet no bank twice: bf16 (eight chunks a row, lanes read 8 bytes)
// swaps the row's halves in odd rows, fp32 (sixteen) its neighbours in the
// upper half.
template <typename T>
struct Tile {
  static constexpr int kRow = kHeadDim * sizeof(T);
  static constexpr int kBytes = 4 * kRow;
  static __device__ __forceinline__ int chunk(int row, int c) {
    return sizeof(T) == 2 ? c ^ ((row & 1) << 2) : c ^ (c >> 3);
  }
  // Byte offset, and address, of component j of row `row`.
  static __device__ __forceinline__ int off(int row, int j) {
    const int byte = j * sizeof(T);
    return row * kRow + chunk(row, byte >> 4) * 16 + (byte & 15);
  }
  static __device__ __forceinline__ const T* at(const uint8_t* tile, int row, int j) {
    return reinterpret_cast<const T*>(tile + off(row, j));
  }
};

// A lane's four pairs of its row: from the tile (sa, sb: where its runs lie
// there), and to global memory (oa, ob: their first components).
template <int kMode>
__device__ __forceinline__ Pairs load_pairs(const QkArgs& q, const uint8_t* tile, int row, int p,
                                            int sa, int sb, const __nv_bfloat16*) {
  using R = Tile<__nv_bfloat16>;
  auto lohi = [](uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
  };
  Pairs o;
  if (kMode == kHalves) {
    const uint2 x = *reinterpret_cast<const uint2*>(tile + sa);
    const uint2 y = *reinterpret_cast<const uint2*>(tile + sb);
    o.a[0] = lohi(x.x); o.a[1] = lohi(x.y);
    o.b[0] = lohi(y.x); o.b[1] = lohi(y.y);
  } else if (kMode == kInterleaved) {
    const uint4 u = *reinterpret_cast<const uint4*>(tile + sa);
    const float2 x[4] = {lohi(u.x), lohi(u.y), lohi(u.z), lohi(u.w)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o.a[i] = make_float2(x[2 * i].x, x[2 * i + 1].x);
      o.b[i] = make_float2(x[2 * i].y, x[2 * i + 1].y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o.a[i] = make_float2(to_f(*R::at(tile, row, comp_a<kMode>(q, p + 2 * i))),
                           to_f(*R::at(tile, row, comp_a<kMode>(q, p + 2 * i + 1))));
      o.b[i] = make_float2(to_f(*R::at(tile, row, comp_b<kMode>(q, p + 2 * i))),
                           to_f(*R::at(tile, row, comp_b<kMode>(q, p + 2 * i + 1))));
    }
  }
  return o;
}
template <int kMode>
__device__ __forceinline__ Pairs load_pairs(const QkArgs& q, const uint8_t* tile, int row, int p,
                                            int sa, int sb, const float*) {
  using R = Tile<float>;
  Pairs o;
  if (kMode == kScattered) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o.a[i] = make_float2(*R::at(tile, row, comp_a<kMode>(q, p + 2 * i)),
                           *R::at(tile, row, comp_a<kMode>(q, p + 2 * i + 1)));
      o.b[i] = make_float2(*R::at(tile, row, comp_b<kMode>(q, p + 2 * i)),
                           *R::at(tile, row, comp_b<kMode>(q, p + 2 * i + 1)));
    }
    return o;
  }
  const float4 x = *reinterpret_cast<const float4*>(tile + sa);
  const float4 y = *reinterpret_cast<const float4*>(tile + sb);
  if (kMode == kInterleaved) {
    o.a[0] = make_float2(x.x, x.z); o.a[1] = make_float2(y.x, y.z);
    o.b[0] = make_float2(x.y, x.w); o.b[1] = make_float2(y.y, y.w);
  } else {
    o.a[0] = make_float2(x.x, x.y); o.a[1] = make_float2(x.z, x.w);
    o.b[0] = make_float2(y.x, y.y); o.b[1] = make_float2(y.z, y.w);
  }
  return o;
}
template <int kMode>
__device__ __forceinline__ void store_pairs(const QkArgs& q, __nv_bfloat16* row, int p, int oa,
                                            int ob, const Pairs& v) {
  auto pack = [](float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  };
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
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = e & 1 ? v.a[e >> 1].y : v.a[e >> 1].x;
      const float y = e & 1 ? v.b[e >> 1].y : v.b[e >> 1].x;
      row[comp_a<kMode>(q, p + e)] = __float2bfloat16_rn(x);
      row[comp_b<kMode>(q, p + e)] = __float2bfloat16_rn(y);
    }
  }
}
template <int kMode>
__device__ __forceinline__ void store_pairs(const QkArgs& q, float* row, int p, int oa, int ob,
                                            const Pairs& v) {
  if (kMode == kInterleaved) {
    *reinterpret_cast<float4*>(row + oa) = make_float4(v.a[0].x, v.b[0].x, v.a[0].y, v.b[0].y);
    *reinterpret_cast<float4*>(row + ob) = make_float4(v.a[1].x, v.b[1].x, v.a[1].y, v.b[1].y);
  } else if (kMode == kHalves) {
    *reinterpret_cast<float4*>(row + oa) = make_float4(v.a[0].x, v.a[0].y, v.a[1].x, v.a[1].y);
    *reinterpret_cast<float4*>(row + ob) = make_float4(v.b[0].x, v.b[0].y, v.b[1].x, v.b[1].y);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      row[comp_a<kMode>(q, p + e)] = e & 1 ? v.a[e >> 1].y : v.a[e >> 1].x;
      row[comp_b<kMode>(q, p + e)] = e & 1 ? v.b[e >> 1].y : v.b[e >> 1].x;
    }
  }
}

// Sum over the eight lanes of a row (a fixed tree: every lane gets the same).
__device__ __forceinline__ float sum8(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x;
}

__device__ __forceinline__ float2 neg2(float2 x) { return make_float2(-x.x, -x.y); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A warp works on two heads at a time (their waits and bookkeeping are
// shared): slots of two heads, and the bytes of shared memory a warp needs.
template <typename T, bool kBwd>
struct Ring {
  static constexpr int kDepth = sizeof(T) == 2 ? (kBwd ? 3 : 4) : 2;
  static constexpr int kItem = Tile<T>::kBytes * (kBwd ? 2 : 1);
  static constexpr int kSlot = 2 * kItem;
  static constexpr int kBytes = kDepth * kSlot;
};

// A warp has read a row whole before it writes any of it, and no other warp
// touches it, so the outputs may be the inputs.
template <typename T, int kMode, bool kBwd>
__global__ void __launch_bounds__(kQkThreads, kBwd ? 2 : 3)
    qk_rope_kernel(const __grid_constant__ QkArgs a) {
  using R = Ring<T, kBwd>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[kBwd ? 2 : 1][kQkThreads / 32][64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = lane >> 3, sub = lane & 7, p0 = sub * 4;
  uint8_t* ring = smem + warp * R::kBytes;
  const int i0 = (int)(2ll * a.H * blockIdx.y / a.splits);
  const int i1 = (int)(2ll * a.H * (blockIdx.y + 1) / a.splits);
  const long long tokens = (long long)a.B * a.L;
  const int oa = comp_a<kMode>(a, p0);
  const int ob = kMode == kInterleaved ? oa + 4 : comp_b<kMode>(a, p0);
  // Where the lane's copies and runs lie in a tile.
  constexpr int kRun = 16 / sizeof(T);  // components of a 16-byte chunk
  const int cp0 = Tile<T>::off(row, sub * kRun);
  const int cp1 = sizeof(T) == 4 ? Tile<T>::off(row, (sub + 8) * kRun) : 0;
  const int sh_a = Tile<T>::off(row, oa), sh_b = Tile<T>::off(row, ob);
  if (kBwd) {
    for (int i = threadIdx.x; i < 2 * (kQkThreads / 32) * 64; i += kQkThreads)
      (&red[0][0][0])[i] = 0.f;
    __syncthreads();
  }

  grid_launch_dependents();
  grid_wait();

  for (long long tb = (long long)blockIdx.x * kTokensPerBlock; tb < tokens;
       tb += (long long)gridDim.x * kTokensPerBlock) {
    const long long token = tb + warp * 4 + row;
    if (tb + warp * 4 >= tokens) continue;  // none of this warp's four
    // Lanes past the last token redo the last one and store nothing, so that
    // every lane reaches the shuffles.
    const bool live = token < tokens;
    const long long tok = live ? token : tokens - 1;
    const int b = (int)(tok / a.L), l = (int)(tok % a.L);
    const size_t step = (size_t)a.L * kHeadDim;
    const size_t base = ((size_t)b * a.H * a.L + l) * kHeadDim;  // head 0
    // Copies the next two items (heads of q, after q's last one of k) into the
    // next slot.
    int fi = i0, fe = i0 < a.H ? min(i1, a.H) : i1, fs = 0;
    const size_t first = base + (size_t)(i0 < a.H ? i0 : i0 - a.H) * step + sub * kRun;
    const T* fx = static_cast<const T*>(a.in[i0 >= a.H]) + first;
    const T* fd = static_cast<const T*>(a.dy[i0 >= a.H]) + first;
    auto fetch = [&]() {
      if (fi < i1) {
        uint8_t* slot = ring + fs;
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (u == 0 || fi + 1 < fe) {
            cp_async16(slot + u * R::kItem + cp0, fx + u * step);
            if (sizeof(T) == 4) cp_async16(slot + u * R::kItem + cp1, fx + u * step + 8 * kRun);
            if (kBwd) {
              uint8_t* dst = slot + u * R::kItem + Tile<T>::kBytes;
              cp_async16(dst + cp0, fd + u * step);
              if (sizeof(T) == 4) cp_async16(dst + cp1, fd + u * step + 8 * kRun);
            }
          }
        fs = fs == R::kBytes - R::kSlot ? 0 : fs + R::kSlot;
        fi += 2;
        fx += 2 * step;
        if (kBwd) fd += 2 * step;
        if (fi >= fe && fe < i1) {  // on to k
          fi = a.H;
          fe = i1;
          fx = static_cast<const T*>(a.in[1]) + base + sub * kRun;
          if (kBwd) fd = static_cast<const T*>(a.dy[1]) + base + sub * kRun;
        }
      }
      cp_async_commit();
    };
    __syncwarp();  // the last tile's slots are read
#pragma unroll
    for (int i = 0; i < R::kDepth - 1; ++i) fetch();

    const int pos = a.pos ? a.pos[tok] : l;
    float2 c[2], s[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float co = 1.f, si = 0.f;
      if (p0 + e < a.half) {
        const uint64_t turns = a.turn[p0 + e] * (uint64_t)(int64_t)pos;
        const int t = (int)(turns >> 32);
        const float f = (float)t;
        float s0, c0;
        sincospif(f * 0x1p-31f, &s0, &c0);
        // What the conversion rounded off, d radians: at most pi 2^-25.
        const float d = (float)(t - (int)f) * 1.46291808e-9f;
        co = fmaf(-s0, d, c0);
        si = fmaf(c0, d, s0);
      }
      (e & 1 ? c[e >> 1].y : c[e >> 1].x) = co;
      (e & 1 ? s[e >> 1].y : s[e >> 1].x) = si;
    }
    int rs = 0;  // slot of the item being worked on
    for (int t = i0 >= a.H, i = i0; i < i1; t = 1) {
      float2 ga[2], gb[2], dga[2], dgb[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ga[e] = gb[e] = both(1.f);
        dga[e] = dgb[e] = both(0.f);
        if (a.gamma[t]) {
          const float* g = a.gamma[t];
          ga[e] = make_float2(g[comp_a<kMode>(a, p0 + 2 * e)],
                              g[comp_a<kMode>(a, p0 + 2 * e + 1)]);
          gb[e] = make_float2(g[comp_b<kMode>(a, p0 + 2 * e)],
                              g[comp_b<kMode>(a, p0 + 2 * e + 1)]);
        }
      }
      // Forward: y_a = r (x_a (ga c) - x_b (gb s)), y_b = r (x_b (gb c) + x_a (ga s)).
      float2 ca[2], sa[2], cb[2], sb[2];
      if (!kBwd) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          ca[e] = mul2(ga[e], c[e]);
          sa[e] = mul2(ga[e], s[e]);
          cb[e] = mul2(gb[e], c[e]);
          sb[e] = neg2(mul2(gb[e], s[e]));
        }
      }
      const int end = t ? i1 : min(i1, a.H);
      T* out = static_cast<T*>(a.out[t]) + base + (size_t)(t ? i - a.H : i) * step;
      for (; i < end; i += 2, out += 2 * step) {
        fetch();
        cp_async_wait<R::kDepth - 1>();
        __syncwarp();
        const uint8_t* slot = ring + rs;
        rs = rs == R::kBytes - R::kSlot ? 0 : rs + R::kSlot;
        const bool two = i + 1 < end;  // (else the second one's work is discarded)
        Pairs x[2], d[2];
        float ss[2], vs[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint8_t* it = slot + (u && two ? R::kItem : 0);
          x[u] = load_pairs<kMode>(a, it, row, p0, sh_a, sh_b, (const T*)nullptr);
          if (kBwd)
            d[u] = load_pairs<kMode>(a, it + Tile<T>::kBytes, row, p0, sh_a, sh_b,
                                     (const T*)nullptr);
        }
        __syncwarp();  // the slot is read
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float2 sq = mul2(x[u].a[0], x[u].a[0]);
          sq = fma2(x[u].a[1], x[u].a[1], sq);
          sq = fma2(x[u].b[0], x[u].b[0], sq);
          sq = fma2(x[u].b[1], x[u].b[1], sq);
          ss[u] = sq.x + sq.y;
          if (kBwd) {
            // d becomes g = R^T dy; v = gamma g
            float2 vx = both(0.f);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 g = fma2(d[u].b[e], s[e], mul2(d[u].a[e], c[e]));
              const float2 k = fma2(d[u].a[e], neg2(s[e]), mul2(d[u].b[e], c[e]));
              vx = fma2(mul2(g, ga[e]), x[u].a[e], vx);
              vx = fma2(mul2(k, gb[e]), x[u].b[e], vx);
              d[u].a[e] = g;
              d[u].b[e] = k;
            }
            vs[u] = vx.x + vx.y;
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          ss[u] = sum8(ss[u]);
          if (kBwd) vs[u] = sum8(vs[u]);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (u && !two) break;
          const float r = rsqrtf(fmaf(ss[u], 1.f / kHeadDim, a.eps));
          Pairs y;
          if (!kBwd) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              y.a[e] = mul2(both(r), fma2(x[u].b[e], sb[e], mul2(x[u].a[e], ca[e])));
              y.b[e] = mul2(both(r), fma2(x[u].a[e], sa[e], mul2(x[u].b[e], cb[e])));
            }
          } else {
            const float m = -vs[u] * r * r * (1.f / kHeadDim);  // -mean(v n) r
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (live) {
                dga[e] = fma2(d[u].a[e], mul2(both(r), x[u].a[e]), dga[e]);
                dgb[e] = fma2(d[u].b[e], mul2(both(r), x[u].b[e]), dgb[e]);
              }
              y.a[e] = mul2(both(r), fma2(both(m), x[u].a[e], mul2(d[u].a[e], ga[e])));
              y.b[e] = mul2(both(r), fma2(both(m), x[u].b[e], mul2(d[u].b[e], gb[e])));
            }
          }
          if (live) store_pairs<kMode>(a, out + u * step, p0, oa, ob, y);
        }
      }
      i = end;  // (an odd range of q leaves i one past it, on k's second head)
      if (kBwd) {
        // The warp's sums of g n over its four tokens, added to those of its
        // earlier tokens.
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = e & 1 ? dga[e >> 1].y : dga[e >> 1].x;
          float y = e & 1 ? dgb[e >> 1].y : dgb[e >> 1].x;
          x += __shfl_xor_sync(0xffffffffu, x, 8);
          x += __shfl_xor_sync(0xffffffffu, x, 16);
          y += __shfl_xor_sync(0xffffffffu, y, 8);
          y += __shfl_xor_sync(0xffffffffu, y, 16);
          if (lane < 8) {
            red[t][warp][comp_a<kMode>(a, p0 + e)] += x;
            red[t][warp][comp_b<kMode>(a, p0 + e)] += y;
          }
        }
      }
    }
    cp_async_wait<0>();
  }

  if (kBwd) {
    // The block's sums, over its warps in order.
    __syncthreads();
    if (threadIdx.x < 128) {
      const int t = threadIdx.x >> 6, j = threadIdx.x & 63;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kQkThreads / 32; ++w) sum += red[t][w][j];
      const size_t blocks = (size_t)gridDim.x * gridDim.y;
      a.part[(t * blocks + (size_t)blockIdx.y * gridDim.x + blockIdx.x) * 64 + j] = sum;
    }
  }
}

// A sum and what its additions rounded off (Knuth's two-sum): as exact as 48
// bits, and without 64-bit additions, which took the gradients of 8 x 12 x 4096
// rows from 59.3 to 62.9 us.
struct Sum {
  float s = 0.f, e = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float t = s + x, y = t - s;
    e += (s - (t - y)) + (x - y);
    s = t;
  }
};

// dgamma of q (blocks 0-7) and k: the blocks' partial sums, up to 1024, in
// order.  (By plain fp32 additions dgamma of 12 x 5003 rows was off by 1.8e-7
// and 1.4e-7; the partial sums alone leave 1.2e-7 and 0.9e-7.)  Eight components
// per block, 32 partial rows at a time.
__global__ void __launch_bounds__(256)
    qk_dgamma_kernel(const float* part, int rows, float* dgq, float* dgk) {
  __shared__ float2 red[32][8];
  const int c = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int t = blockIdx.x >> 3, j = (blockIdx.x & 7) * 8 + c;
  const float* p = part + (size_t)t * rows * 64 + j;
  Sum s;
  grid_launch_dependents();
  grid_wait();
#pragma unroll 4
  for (int i = g; i < rows; i += 32) s.add(p[(size_t)i * 64]);
  red[g][c] = make_float2(s.s, s.e);
  __syncthreads();
  if (g == 0) {
    Sum sum;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      sum.add(red[i][c].x);
      sum.e += red[i][c].y;
    }
    float* out = t ? dgk : dgq;
    // (Nothing is rounded off an infinity: there e is not a number.)
    if (out) out[j] = sum.e == sum.e ? sum.s + sum.e : sum.s;
  }
}

// Blocks along the tokens.  The backward's write a partial sum each: past the
// cap a block walks several token tiles.
int token_blocks(const bb_qk_desc& d, bool bwd) {
  const long long tiles = ((long long)d.B * d.L + kTokensPerBlock - 1) / kTokensPerBlock;
  const long long cap = bwd ? 1024 : 1 << 20;
  return (int)(tiles < cap ? tiles : cap);
}

// Ranges the 2 H heads are split into: about four blocks for each of 148 SMs,
// at most one per head; longer walks share the angles and keep more rows in
// flight.  (Three are resident at a time in the forward and two in the
// backward, so few tokens run in two or three rounds, the last one part full:
// the gradients of 12 x 5003 fp32 rows are 628 blocks on 296 places.)
int head_splits(const bb_qk_desc& d, bool bwd) {
  const int want = 148 * 4, have = token_blocks(d, bwd);
  int s = (want + have - 1) / have;
  return s < 2 * d.H ? s : 2 * d.H;
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
  a.splits = head_splits(d, bwd);
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

template <typename T, int kMode, bool kBwd>
cudaError_t launch_as(const bb_qk_desc& d, const QkArgs& a, cudaStream_t s) {
  constexpr int smem = kQkThreads / 32 * Ring<T, kBwd>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(qk_rope_kernel<T, kMode, kBwd>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_chained(qk_rope_kernel<T, kMode, kBwd>, dim3(token_blocks(d, kBwd), a.splits),
                        kQkThreads, smem, false, s, a);
}

template <typename T, bool kBwd>
cudaError_t launch_mode(const bb_qk_desc& d, const QkArgs& a, cudaStream_t s) {
  if (d.interleaved || a.rot == 0) return launch_as<T, kInterleaved, kBwd>(d, a, s);
  if (a.half % 4 == 0) return launch_as<T, kHalves, kBwd>(d, a, s);
  return launch_as<T, kScattered, kBwd>(d, a, s);
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
    if (launch_chained(qk_dgamma_kernel, 16, 256, 0, false, s, (const float*)a.part,
                       a.splits * token_blocks(*desc, true), dgamma_q, dgamma_k) != cudaSuccess)
      return BB_ERR_CUDA;
  }
  return BB_OK;
}

}  // extern "C"
