// Softmax cross entropy of the vocabulary projection, and its gradients,
// with the logits never in memory as a whole:
//
//   z[n][v] = <h_n, w_v> + bias[v],  lse_n = log sum_v exp z[n][v]
//   loss_n  = lse_n - z[n][label_n]
//   dz[n][v] = dloss_n (exp(z[n][v] - lse_n) - [v = label_n])
//   dh = dz W,  dW = dz^T h,  dbias = sum_n dz
//
// Rows whose label is outside [0, V) have no loss: their loss and dh are 0
// and they are neither multiplied nor read into any result.  The first
// launch (rows_kernel) packs the rows that have one, in order; when every
// row has one, h is used where it lies.
//
// Forward: one GEMM over (row tile, vocabulary tile); the epilogue keeps, per
// row of a tile, the maximum and the sum of exponentials of its 256 logits
// and the label's logit, and a small launch merges the tiles' pairs in a
// fixed order.  Logits live in tensor memory and registers only.
//
// Backward: the vocabulary goes by in pieces whose dz (bf16) fits a fixed
// workspace.  Per piece, one GEMM launch computes the logits again and
// writes dz, and one GEMM launch forms the piece's rows of dW (complete) and
// its part of dh, added to an fp32 sum.  A last launch rounds dh and sums
// dbias.  Without the stored logits this is 6 R D V operations (R rows with
// a label) beside the forward's 2 R D V.
//
// dz is held in bf16, the type of the tensor-core operands it multiplies;
// dloss enters it relative to the largest |dloss| and that factor is applied
// in fp32 at the end, so for equal dloss a dz near -1 (a label of low
// probability) is exact and no rounding is shared by all rows.
#include "common.cuh"
#include "sm100.cuh"

namespace bb {
namespace {

using namespace sm100;

// A tile of the GEMMs is 256 x 256: a pair of CTAs (cta_group::2), 128 rows of
// A and 128 columns of B in each one's shared memory, 128 x 256 accumulators
// in each one's tensor memory, two of them, so that a tile's epilogue runs
// under the next tile's MMAs.
constexpr int kBM = 128;                            // rows of a CTA
constexpr int kTM = 2 * kBM, kTN = 256, kBK = 64;   // tile of a pair, K step
constexpr int kStages = 5;
constexpr uint32_t kBox = 64 * 64 * 2;              // one 64 x 64 bf16 box: 8 KB
constexpr uint32_t kOpTile = 128 * kBK * 2;         // a CTA's part of A or B: 16 KB
constexpr uint32_t kStageBytes = 2 * kOpTile;       // 32 KB
constexpr int kEpiWarps = 8;                        // two per TMEM lane quarter
constexpr uint32_t kStageOut = kEpiWarps * 4096;    // a 32 x 128 B block per warp
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kTmemCols = 512;                 // two 128 x 256 fp32 accumulators
constexpr int kHalf = kTN / 2;                      // columns of an epilogue warp
constexpr size_t kPieceBytes = 256u << 20;          // dz of one vocabulary piece

enum Mode { kLse = 0, kDz = 1, kGrad = 2 };

// What rows_kernel finds out on the device, at the workspace's start.
struct Info {
  int status;
  int pad[15];
  int rows;      // rows with a label
  int direct;    // 1: every row has one, h is read where it lies
  float dlref;   // largest |dloss| of those rows (1 when that is 0 or not finite)
};

struct CeArgs {
  int N, D, V;
  int Np;            // N rounded up to a tile's rows
  int Vp;            // columns of a piece (a multiple of 256)
  int v0, vn;        // this piece: first column, columns
  int splits;        // parts the piece's columns are cut into for dh
  int add;           // dh partials: 1 adds to what earlier pieces wrote
  Info* info;
  const float* bias;   // [V] or null
  const int* lab;      // packed rows: label,
  const float* rlse;   //   lse,
  const float* dls;    //   dloss / dlref
  float2* part;        // [vocabulary half tiles][Np] (max, sum of exponentials)
  float* zl;           // [N] logit of the label
  float* dbp;          // [Np / 128][Vp] column sums of dz, or null
  float* dbias;        // [V], with dbp
};

struct Bars {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], red;
};

// One output tile.
struct Job {
  int dw;           // kGrad: 1 = a tile of dW, 0 = of dh
  int m0, n0;       // first row and column of the tile
  int k0, ksteps;   // first K index, 64-wide K steps
  int nblk;         // 64-column blocks of B in each CTA: the tile has 128 nblk columns
  int row0;         // first row in the output
};

template <int kMode>
struct Work {
  int tiles, mt, dn, wm, th, hks, wks, dh_first;
  __device__ __forceinline__ Work(const CeArgs& a, int rows) {
    mt = (rows + kTM - 1) / kTM;
    if (kMode != kGrad) {
      tiles = mt * ((a.vn + kTN - 1) / kTN);
      return;
    }
    dn = (a.D + kTN - 1) / kTN;
    wm = (a.vn + kTM - 1) / kTM;
    hks = (a.vn + kBK - 1) / kBK;
    wks = (rows + kBK - 1) / kBK;
    th = mt * dn * a.splits;
    tiles = th + wm * dn;
    // Long tiles first.
    dh_first = hks / a.splits >= wks;
  }
  __device__ __forceinline__ Job job(const CeArgs& a, int t) const {
    Job j;
    j.nblk = 2;
    if (kMode != kGrad) {
      // Row tiles run fastest: the rows stay in L2 while W streams by once.
      j.dw = 0;
      j.m0 = (t % mt) * kTM;
      j.n0 = (t / mt) * kTN;
      j.k0 = 0;
      j.ksteps = (a.D + kBK - 1) / kBK;
      j.row0 = j.m0;
      return j;
    }
    j.dw = dh_first ? t >= th : t < wm * dn;
    int u = t;
    if (dh_first && j.dw) u -= th;
    if (!dh_first && !j.dw) u -= wm * dn;
    j.n0 = (u % dn) * kTN;
    if (a.D - j.n0 <= 128) j.nblk = 1;
    u /= dn;
    if (j.dw) {
      j.m0 = u * kTM;
      j.k0 = 0;
      j.ksteps = wks;
      j.row0 = a.v0 + j.m0;
    } else {
      const int s = u / mt;
      j.m0 = (u % mt) * kTM;
      j.k0 = (int)((long long)hks * s / a.splits);
      j.ksteps = (int)((long long)hks * (s + 1) / a.splits) - j.k0;
      j.row0 = s * a.Np + j.m0;
    }
    return j;
  }
};

// Sum over the 32 lanes of each of 32 columns held one row per lane; lane l
// returns column l.  Each step halves the columns a lane carries.
__device__ __forceinline__ float column_sums(float (&x)[32], int lane) {
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int e = 0; e < s; ++e) {
      const float give = up ? x[e] : x[e + s];
      const float keep = up ? x[e + s] : x[e];
      x[e] = keep + __shfl_xor_sync(0xffffffffu, give, s);
    }
  }
  return x[0];
}

// 32 logits of one row: the accumulator's columns plus bias.  Columns past V
// get `fill`.
__device__ __forceinline__ void logits32(const CeArgs& a, uint32_t taddr, int c0, float fill,
                                         float (&z)[32]) {
  uint32_t v[32];
  __syncwarp();
  tmem_ld32(taddr, v);
  tmem_ld_wait();
#pragma unroll
  for (int e = 0; e < 32; ++e) z[e] = __uint_as_float(v[e]);
  if (c0 + 32 <= a.V) {
    if (a.bias) {
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 b = __ldg(reinterpret_cast<const float4*>(a.bias + c0 + e));
        z[e] += b.x; z[e + 1] += b.y; z[e + 2] += b.z; z[e + 3] += b.w;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      z[e] = c0 + e < a.V ? z[e] + (a.bias ? __ldg(a.bias + c0 + e) : 0.f) : fill;
  }
}

template <int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    ce_gemm_kernel(const __grid_constant__ CeArgs a, const __grid_constant__ CUtensorMap tmH,
                   const __grid_constant__ CUtensorMap tmHp,
                   const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ CUtensorMap tmDz,
                   const __grid_constant__ CUtensorMap tmDw,
                   const __grid_constant__ CUtensorMap tmDh) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile int abort_flag;
  __shared__ float red[2][4][kTN];  // kDz: column sums of each warp's 32 rows
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* stages = base;                              // [kStages][A | B]
  uint8_t* stage_out = base + kStages * kStageBytes;   // [8 warps][32][128 B]
  int* status = &a.info->status;
  const int rows = a.info->rows;
  const CUtensorMap* mapH = a.info->direct ? &tmH : &tmHp;
  const Work<kMode> work(a, rows);

  // Barriers of the pair: `full` and `acc_empty` are used in rank 0 only (it
  // issues the MMAs); both CTAs' loads and epilogue warps signal them there.
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.acc_full[s], 1);
      mbar_init(&bars.acc_empty[s], 2 * kEpiWarps);
    }
    mbar_init(&bars.red, kEpiWarps);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&tmem_base_sh, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;

  if (warp == 0) {
    // ---------------- TMA loads (one thread of each CTA) ----------------
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int t = pair; t < work.tiles && ok; t += pairs) {
        const Job j = work.job(a, t);
        const int m0 = j.m0 + rank * kBM, n0 = j.n0 + rank * 64 * j.nblk;
        for (int ks = 0; ks < j.ksteps; ++ks, ++it) {
          const uint32_t st = it % kStages;
          if (!mbar_wait(&bars.empty[st], ((it / kStages) & 1) ^ 1, &abort_flag, status)) {
            ok = false;
            break;
          }
          uint8_t* pa = stages + st * kStageBytes;
          uint8_t* pb = pa + kOpTile;
          const uint32_t bar = map_rank(&bars.full[st], 0);
          if (rank == 0) mbar_expect_tx(&bars.full[st], 2 * (kOpTile + j.nblk * kBox));
          const int k = (j.k0 + ks) * kBK;
          if (kMode != kGrad) {
            tma_load_2d_pair(pa, mapH, bar, k, m0);
            tma_load_2d_pair(pb, &tmW, bar, k, a.v0 + n0);
          } else {
            // dW: A = dz^T (columns of dz along M), B = h; dh: A = dz, B = W.
            for (int i = 0; i < 2; ++i)
              tma_load_2d_pair(pa + i * kBox, &tmDz, bar, j.dw ? m0 + 64 * i : k,
                               j.dw ? k : m0 + 64 * i);
            for (int i = 0; i < j.nblk; ++i)
              tma_load_2d_pair(pb + i * kBox, j.dw ? mapH : &tmW, bar, n0 + 64 * i,
                               j.dw ? k : a.v0 + k);
          }
        }
      }
      // The last stages' releases reach this CTA before it may leave.
      for (int i = 0; i < kStages && ok; ++i, ++it)
        ok = mbar_wait(&bars.empty[it % kStages], ((it / kStages) & 1) ^ 1, &abort_flag, status);
      if (abort_flag && rank == 0) {
        // Let issued copies (both CTAs') land before shared memory goes away;
        // rank 1 waits at the cluster barrier meanwhile.
        for (uint32_t s = 0; s < (uint32_t)kStages; ++s)
          if (it >= s + 1) {
            const uint32_t last = it - 1 - ((it - 1 - s) % kStages);
            const uint64_t t0 = globaltimer();
            while (!mbar_try_wait(&bars.full[s], (last / kStages) & 1) &&
                   globaltimer() - t0 < 100000000ull) {
            }
          }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issue (one thread of rank 0) ----------------
    uint32_t it = 0, tc = 0;
    bool ok = rank == 0;
    for (int t = pair; t < work.tiles && ok; t += pairs, ++tc) {
      const Job j = work.job(a, t);
      const int acc = tc & 1;
      if (!mbar_wait(&bars.acc_empty[acc], ((tc >> 1) & 1) ^ 1, &abort_flag, status)) break;
      tc_fence_after();
      // K-major tiles step 32 bytes per 16 of K; MN-major ones 16 rows of 128.
      const uint32_t a_mn = kMode == kGrad && j.dw, b_mn = kMode == kGrad;
      const uint32_t idesc = idesc_bf16(kTM, 128 * j.nblk, a_mn, b_mn);
      const uint32_t astep = a_mn ? 2048 : 32, bstep = b_mn ? 2048 : 32;
      const uint32_t albo = a_mn ? kBox : 16, blbo = b_mn ? kBox : 16;
      for (int ks = 0; ks < j.ksteps; ++ks, ++it) {
        const uint32_t st = it % kStages;
        if (!mbar_wait(&bars.full[st], (it / kStages) & 1, &abort_flag, status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t aaddr = smem_u32(stages + st * kStageBytes);
          const uint32_t baddr = aaddr + kOpTile;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss_pair(tmem + acc * kTN, sdesc_sw128(aaddr + kk * astep, albo),
                        sdesc_sw128(baddr + kk * bstep, blbo), idesc,
                        (ks > 0 || kk > 0) ? 1u : 0u);
          mma_commit_pair(&bars.empty[st]);
        }
        __syncwarp();
      }
      if (ok && lane == 0) mma_commit_pair(&bars.acc_full[acc]);
      __syncwarp();
    }
  } else {
    // ------- epilogue (warps 2-9: 32 rows and half of the columns each) -------
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    uint8_t* stage = stage_out + (warp - 2) * 4096;
    uint8_t* rowp = stage + lane * 128;
    const int swz = lane & 7;
    const float dlref = kMode == kGrad ? a.info->dlref : 1.f;
    const uint32_t acc_empty = map_rank(&bars.acc_empty[0], 0);
    uint32_t tc = 0;
    for (int t = pair; t < work.tiles; t += pairs, ++tc) {
      const Job j = work.job(a, t);
      const int acc = tc & 1;
      if (!mbar_wait(&bars.acc_full[acc], (tc >> 1) & 1, &abort_flag, status)) break;
      tc_fence_after();
      const uint32_t tz = tmem + acc * kTN + lane_off;
      const int r0 = rank * kBM + quarter * 32;  // this warp's first row in the tile
      const int row = j.m0 + r0 + lane;          // packed row (kLse, kDz)
      const int cbeg = half * kHalf;
      if (kMode == kLse) {
        const int lab = row < rows ? __ldg(a.lab + row) : -1;
        float m = -INFINITY, s = 0.f;
#pragma unroll 1
        for (int c = cbeg; c < cbeg + kHalf; c += 32) {
          const int c0 = j.n0 + c;
          if (c0 >= a.V) break;
          float z[32];
          logits32(a, tz + c, c0, -INFINITY, z);
          if ((unsigned)(lab - c0) < 32u) {
            float zl = z[0];
#pragma unroll
            for (int e = 1; e < 32; ++e) zl = lab - c0 == e ? z[e] : zl;
            a.zl[row] = zl;
          }
          float cm = m;
#pragma unroll
          for (int e = 0; e < 32; e += 2) cm = fmax3(cm, z[e], z[e + 1]);
          // A row of -inf so far keeps a finite reference.  Differences are
          // taken before the scaling to base 2, so logits near the type's
          // lowest value do not overflow.
          const float ref = cm == -INFINITY ? 0.f : cm;
          float2 sum = make_float2(s * ex2((m - ref) * kLog2e), 0.f);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 d = mul2(sub2(make_float2(z[e], z[e + 1]), make_float2(ref, ref)),
                                  make_float2(kLog2e, kLog2e));
            sum = add2(sum, make_float2(ex2(d.x), ex2(d.y)));
          }
          s = sum.x + sum.y;
          m = cm;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty + 8 * acc);
        a.part[(size_t)((j.n0 + cbeg) / kHalf) * a.Np + row] = make_float2(m, s);
        continue;
      }
      if (kMode == kDz) {
        const bool live = row < rows;
        const int lab = live ? __ldg(a.lab + row) - a.v0 : -1;
        const float lse = live ? __ldg(a.rlse + row) : 0.f;
        const float dl = live ? __ldg(a.dls + row) : 0.f;
#pragma unroll 1
        for (int c = cbeg; c < cbeg + kHalf; c += 32) {
          const int c0 = j.n0 + c;  // column in the piece
          float z[32];
          logits32(a, tz + c, a.v0 + c0, 0.f, z);
          const int last = a.V - a.v0 - c0;  // columns of this block inside V
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 d = mul2(sub2(make_float2(z[e], z[e + 1]), make_float2(lse, lse)),
                                  make_float2(kLog2e, kLog2e));
            z[e] = dl * (ex2(d.x) - (lab - c0 == e ? 1.f : 0.f));
            z[e + 1] = dl * (ex2(d.y) - (lab - c0 == e + 1 ? 1.f : 0.f));
          }
          // Rows past the last and columns past V: exact zeros, whatever the
          // accumulator held.
          if (!live || last < 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e) z[e] = live && e < last ? z[e] : 0.f;
          }
          if ((c & 32) == 0) {
            // The previous block's store has read the staging area.
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
          }
#pragma unroll
          for (int ch = 0; ch < 4; ++ch)
            *reinterpret_cast<uint4*>(rowp + (((((c >> 5) & 1) * 4 + ch) ^ swz) << 4)) =
                make_uint4(pack_bf16(z[8 * ch], z[8 * ch + 1]),
                           pack_bf16(z[8 * ch + 2], z[8 * ch + 3]),
                           pack_bf16(z[8 * ch + 4], z[8 * ch + 5]),
                           pack_bf16(z[8 * ch + 6], z[8 * ch + 7]));
          if (c & 32) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmDz, stage, j.n0 + c - 32, j.m0 + r0);
              bulk_commit_group();
            }
          }
          if (a.dbp) red[acc][quarter][c + lane] = column_sums(z, lane);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty + 8 * acc);
        if (a.dbp) {
          // Column sums of the CTA's 128 rows: the four quarters' sums in order.
          if (lane == 0) mbar_arrive_release(&bars.red);
          if (!mbar_wait(&bars.red, tc & 1, &abort_flag, status)) break;
          const int c = (warp - 2) * 32 + lane;
          a.dbp[(size_t)(j.m0 / kBM + rank) * a.Vp + j.n0 + c] =
              red[acc][0][c] + red[acc][1][c] + red[acc][2][c] + red[acc][3][c];
        }
        continue;
      }
      // kGrad.  The first column tile of dW also sums dbias of its words,
      // over the blocks of 128 rows in order.
      if (j.dw && j.n0 == 0 && a.dbp && half == 0) {
        const int v = j.m0 + r0 + lane;
        const int blocks = (rows + kBM - 1) / kBM;
        float s = 0.f;
        for (int m = 0; m < blocks; ++m) s += a.dbp[(size_t)m * a.Vp + v];
        if (a.v0 + v < a.V) a.dbias[a.v0 + v] = s * dlref;
      }
      // A tile without K steps (no rows) is zero.
      const float f = j.ksteps > 0 ? 1.f : 0.f;
#pragma unroll 1
      for (int cb = half * j.nblk; cb < (half + 1) * j.nblk; ++cb) {
        uint32_t v0[32], v1[32];
        tmem_ld32(tz + cb * 64, v0);
        tmem_ld32(tz + cb * 64 + 32, v1);
        tmem_ld_wait();
        const int y = j.row0 + r0, x = j.n0 + cb * 64;
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
        if (j.dw) {
#pragma unroll
          for (int ch = 0; ch < 8; ++ch) {
            const uint32_t* src = ch < 4 ? v0 + 8 * ch : v1 + 8 * (ch - 4);
            float g[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              g[e] = f != 0.f ? dlref * __uint_as_float(src[e]) : 0.f;
            *reinterpret_cast<uint4*>(rowp + ((ch ^ swz) << 4)) =
                make_uint4(pack_bf16(g[0], g[1]), pack_bf16(g[2], g[3]), pack_bf16(g[4], g[5]),
                           pack_bf16(g[6], g[7]));
          }
          fence_proxy_async_smem();
          __syncwarp();
          // Boxes that start past the tensor's end have nothing to write.
          if (lane == 0 && y < a.V && x < a.D) {
            tma_store_2d(&tmDw, stage, x, y);
            bulk_commit_group();
          }
        } else {
          // fp32: two boxes of 32 columns, one after the other.
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t* v = i ? v1 : v0;
            if (i) {
              if (lane == 0) bulk_wait_read_all();
              __syncwarp();
            }
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)
              *reinterpret_cast<uint4*>(rowp + ((ch ^ swz) << 4)) =
                  make_uint4(v[4 * ch], v[4 * ch + 1], v[4 * ch + 2], v[4 * ch + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && x + 32 * i < a.D) {
              if (a.add)
                tma_reduce_add_2d(&tmDh, stage, x + 32 * i, y);
              else
                tma_store_2d(&tmDh, stage, x + 32 * i, y);
              bulk_commit_group();
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc_empty + 8 * acc);
    }
    if (kMode != kLse && lane == 0) bulk_wait_all();  // output stores complete
  }

  // Neither CTA leaves while the other may still signal its barriers.
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// ---- packing the rows that have a label ------------------------------------

struct RowsArgs {
  int N, D, V;
  const int32_t* labels;
  const uint16_t* h;
  const float* lse;     // backward
  const float* dloss;   // backward
  float *loss, *lse_out;  // forward: zeroed where there is no label
  Info* info;
  int *idx, *pos, *lab;
  float *rlse, *dls;
  uint16_t* hp;         // packed rows of h
};

constexpr int kRowsPerBlock = 256;

// Block b packs rows 256 b .. 256 b + 255.  Each block reads all labels (and
// dloss) to find how many rows with a label lie before its own, so one
// launch does; labels are a few KB to a few hundred and come from L2.
template <bool kBwd>
__global__ void __launch_bounds__(kRowsPerBlock) rows_kernel(const RowsArgs a) {
  __shared__ int cnt[3][8];
  __shared__ float mx[8];
  __shared__ int dst[kRowsPerBlock];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int base = blockIdx.x * kRowsPerBlock;
  int total = 0, before = 0, bad = 0;
  float big = 0.f;
  for (int i = tid; i < a.N; i += kRowsPerBlock) {
    const int l = __ldg(a.labels + i);
    if (l >= 0 && l < a.V) {
      ++total;
      before += i < base;
      if (kBwd) big = fmaxf(big, fabsf(__ldg(a.dloss + i)));
    }
    bad |= l >= a.V;
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, s);
    before += __shfl_xor_sync(0xffffffffu, before, s);
    bad |= __shfl_xor_sync(0xffffffffu, bad, s);
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, s));
  }
  if (lane == 0) {
    cnt[0][warp] = total;
    cnt[1][warp] = before;
    cnt[2][warp] = bad;
    mx[warp] = big;
  }
  __syncthreads();
  total = before = bad = 0;
  big = 0.f;
  for (int w = 0; w < 8; ++w) {
    total += cnt[0][w];
    before += cnt[1][w];
    bad |= cnt[2][w];
    big = fmaxf(big, mx[w]);
  }
  const float dlref = big > 0.f && big < INFINITY ? big : 1.f;
  __syncthreads();
  const int n = base + tid;
  const int l = n < a.N ? __ldg(a.labels + n) : -1;
  const bool live = l >= 0 && l < a.V;
  const unsigned m = __ballot_sync(0xffffffffu, live);
  if (lane == 0) cnt[0][warp] = __popc(m);
  __syncthreads();
  int p = before + __popc(m & ((1u << lane) - 1));
  for (int w = 0; w < warp; ++w) p += cnt[0][w];
  dst[tid] = live ? p : -1;
  if (live) {
    a.idx[p] = n;
    a.lab[p] = l;
    if (kBwd) {
      a.rlse[p] = __ldg(a.lse + n);
      a.dls[p] = __ldg(a.dloss + n) / dlref;
    }
  }
  if (n < a.N) {
    if (kBwd) {
      a.pos[n] = live ? p : -1;
    } else if (!live) {
      a.loss[n] = 0.f;
      a.lse_out[n] = 0.f;
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.info->status = bad ? BB_ERR_BAD_LABEL : BB_OK;
    a.info->rows = total;
    a.info->direct = total == a.N;
    a.info->dlref = dlref;
  }
  if (total == a.N) return;
  __syncthreads();
  const int chunks = a.D / 8;  // 16-byte pieces of a row
  for (int r = warp; r < kRowsPerBlock; r += 8) {
    if (dst[r] < 0) continue;
    const uint4* src = reinterpret_cast<const uint4*>(a.h + (size_t)(base + r) * a.D);
    uint4* out = reinterpret_cast<uint4*>(a.hp + (size_t)dst[r] * a.D);
    for (int c = lane; c < chunks; c += 32) out[c] = __ldg(src + c);
  }
  // The rest of the last 64 packed rows, which dW's last K step reads, is
  // zero (times the zeros of dz).
  if (blockIdx.x == 0) {
    const int end = (total + kBK - 1) / kBK * kBK;
    uint4* out = reinterpret_cast<uint4*>(a.hp);
    for (size_t c = (size_t)total * chunks + tid; c < (size_t)end * chunks; c += kRowsPerBlock)
      out[c] = make_uint4(0, 0, 0, 0);
  }
}

// Forward: merges the vocabulary half tiles' (max, sum) of 32 rows in a fixed
// order: eight warps take every eighth tile, then their eight pairs.
__global__ void __launch_bounds__(256)
    lse_merge_kernel(const Info* info, const float2* part, int vt, int Np, const float* zl,
                     const int* idx, float* loss, float* lse) {
  __shared__ float2 sh[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * 32 + lane;
  const int rows = info->rows;
  if ((int)blockIdx.x * 32 >= rows) return;
  float m = -INFINITY, s = 0.f;
  for (int i = warp; i < vt; i += 8) {
    const float2 p = part[(size_t)i * Np + row];
    const float mm = fmaxf(m, p.x);
    const float ref = mm == -INFINITY ? 0.f : mm;
    s = s * ex2((m - ref) * kLog2e) + p.y * ex2((p.x - ref) * kLog2e);
    m = mm;
  }
  sh[warp][lane] = make_float2(m, s);
  __syncthreads();
  if (warp == 0 && row < rows) {
    m = -INFINITY;
    for (int w = 0; w < 8; ++w) m = fmaxf(m, sh[w][lane].x);
    const float ref = m == -INFINITY ? 0.f : m;
    s = 0.f;
    for (int w = 0; w < 8; ++w) s += sh[w][lane].y * ex2((sh[w][lane].x - ref) * kLog2e);
    const float l = ref + logf(s);
    const int n = idx[row];
    lse[n] = l;
    loss[n] = l - zl[row];
  }
}

// Backward's end: dh rows rounded from the fp32 sums (0 where there is no
// label), eight columns per thread.
__global__ void __launch_bounds__(256)
    dh_round_kernel(const Info* info, int N, int D, int Np, int splits, const int* pos,
                    const float* acc, uint16_t* dh) {
  const int chunks = D / 8;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  const size_t n = i / chunks;
  if (n >= (size_t)N) return;
  const int c = (int)(i % chunks) * 8;
  const int p = pos[n];
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (p >= 0) {
    const float dlref = info->dlref;
    for (int s = 0; s < splits; ++s) {
      const float4* src = reinterpret_cast<const float4*>(acc + ((size_t)s * Np + p) * D + c);
      const float4 x = src[0], y = src[1];
      v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
      v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= dlref;
  }
  *reinterpret_cast<uint4*>(dh + n * D + c) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                 pack_bf16(v[6], v[7]));
}

// ---- host -------------------------------------------------------------------

struct Plan {
  int Np, pieces, Vp, splits, vt;
  size_t idx, pos, lab, rlse, dls, hp, part, zl, dz, dh, dbp, total;  // byte offsets
};

size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }

int make_plan(int N, int D, int V, int pass, Plan* p) {
  if (N <= 0 || D <= 0 || V <= 0 || (pass != 0 && pass != 1)) return BB_ERR_INVALID;
  if (D % 8 != 0 || D < 64 || D > 65536 || N > (1 << 24) || V > (1 << 24))
    return BB_ERR_UNSUPPORTED;
  p->Np = (int)up(N, kTM);
  p->vt = (V + kTN - 1) / kTN;
  if ((long long)(p->Np / kTM) * p->vt >= (1ll << 31)) return BB_ERR_UNSUPPORTED;
  // Pieces of equal size whose dz fits kPieceBytes (512 columns at least).
  size_t cols = kPieceBytes / 2 / p->Np / kTN * kTN;
  cols = cols < 512 ? 512 : cols;
  p->pieces = (int)((V + cols - 1) / cols);
  p->Vp = (int)up((V + p->pieces - 1) / p->pieces, kTN);
  p->pieces = (V + p->Vp - 1) / p->Vp;
  // dh has few tiles of a long K when there are few rows: cut K so that a
  // tile takes no more than half of a pair's share of the launch.
  const long long dn = (D + kTN - 1) / kTN, mt = p->Np / kTM;
  const long long hks = p->Vp / kBK, wks = (N + kBK - 1) / kBK;
  const long long share = (mt * dn * hks + (long long)(p->Vp / kTM) * dn * wks) / (2 * 74);
  const long long len = share < 8 ? 8 : share;
  long long s = (hks + len - 1) / len;
  p->splits = (int)(s < 1 ? 1 : s > 64 ? 64 : s);
  size_t off = 256;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = up(off + bytes, 256);
    return o;
  };
  p->idx = take((size_t)N * 4);
  p->lab = take((size_t)N * 4);
  p->hp = take((size_t)p->Np * D * 2);
  if (pass == 0) {
    p->part = take((size_t)2 * p->vt * p->Np * 8);
    p->zl = take((size_t)N * 4);
  } else {
    p->pos = take((size_t)N * 4);
    p->rlse = take((size_t)N * 4);
    p->dls = take((size_t)N * 4);
    p->dz = take((size_t)p->Np * p->Vp * 2);
    p->dh = take((size_t)p->splits * p->Np * D * 4);
    p->dbp = take((size_t)(p->Np / kBM) * p->Vp * 4);
  }
  p->total = off;
  return BB_OK;
}

template <int kMode>
cudaError_t launch_gemm(const CeArgs& a, int tiles, int sms, const CUtensorMap& h,
                        const CUtensorMap& hp, const CUtensorMap& w, const CUtensorMap& dz,
                        const CUtensorMap& dw, const CUtensorMap& dh, cudaStream_t s) {
  const size_t smem = 1024 + kStages * kStageBytes + kStageOut;
  cudaError_t e = cudaFuncSetAttribute(ce_gemm_kernel<kMode>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * (tiles < sms / 2 ? tiles : sms / 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ce_gemm_kernel<kMode>, a, h, hp, w, dz, dw, dh);
}

int sm_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

}  // namespace
}  // namespace bb

using namespace bb;

extern "C" {

int bb_linear_ce_workspace_size(int N, int hidden, int V, int pass, size_t* bytes) {
  if (!bytes) return BB_ERR_INVALID;
  Plan p{};
  const int st = make_plan(N, hidden, V, pass, &p);
  if (st == BB_OK) *bytes = p.total;
  return st;
}

int bb_linear_ce_fwd(int N, int hidden, int V, const void* h, const void* w, const float* bias,
                     const int32_t* labels, float* loss, float* lse, void* workspace,
                     size_t workspace_bytes, void* stream) {
  Plan p{};
  const int st = make_plan(N, hidden, V, 0, &p);
  if (st != BB_OK) return st;
  if (!h || !w || !labels || !loss || !lse) return BB_ERR_INVALID;
  const void* ptrs[] = {h, w, bias, labels, loss, lse, workspace};
  for (const void* x : ptrs)
    if (!aligned16(x)) return BB_ERR_INVALID;
  if (!workspace || workspace_bytes < p.total) return BB_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  cudaStream_t s = (cudaStream_t)stream;
  CUtensorMap tmH, tmHp, tmW;
  if (!encode_bf16_2d(&tmH, h, hidden, N, hidden, 64, kBM) ||
      !encode_bf16_2d(&tmHp, ws + p.hp, hidden, p.Np, hidden, 64, kBM) ||
      !encode_bf16_2d(&tmW, w, hidden, V, hidden, 64, 128))
    return BB_ERR_CUDA;
  RowsArgs r{};
  r.N = N;
  r.D = hidden;
  r.V = V;
  r.labels = labels;
  r.h = static_cast<const uint16_t*>(h);
  r.loss = loss;
  r.lse_out = lse;
  r.info = reinterpret_cast<Info*>(ws);
  r.idx = reinterpret_cast<int*>(ws + p.idx);
  r.lab = reinterpret_cast<int*>(ws + p.lab);
  r.hp = reinterpret_cast<uint16_t*>(ws + p.hp);
  rows_kernel<false><<<(N + kRowsPerBlock - 1) / kRowsPerBlock, kRowsPerBlock, 0, s>>>(r);
  if (cudaGetLastError() != cudaSuccess) return BB_ERR_CUDA;
  CeArgs a{};
  a.N = N;
  a.D = hidden;
  a.V = V;
  a.Np = p.Np;
  a.vn = V;
  a.info = r.info;
  a.bias = bias;
  a.lab = r.lab;
  a.part = reinterpret_cast<float2*>(ws + p.part);
  a.zl = reinterpret_cast<float*>(ws + p.zl);
  if (launch_gemm<kLse>(a, p.Np / kTM * p.vt, sm_count(), tmH, tmHp, tmW, tmW, tmW, tmW, s) !=
      cudaSuccess)
    return BB_ERR_CUDA;
  lse_merge_kernel<<<(N + 31) / 32, 256, 0, s>>>(a.info, a.part, (V + kHalf - 1) / kHalf, p.Np, a.zl, r.idx, loss,
                                                 lse);
  return cudaGetLastError() == cudaSuccess ? BB_OK : BB_ERR_CUDA;
}

int bb_linear_ce_bwd(int N, int hidden, int V, const void* h, const void* w, const float* bias,
                     const int32_t* labels, const float* lse, const float* dloss, void* dh,
                     void* dw, float* dbias, void* workspace, size_t workspace_bytes,
                     void* stream) {
  Plan p{};
  const int st = make_plan(N, hidden, V, 1, &p);
  if (st != BB_OK) return st;
  if (!h || !w || !labels || !lse || !dloss || !dh || !dw) return BB_ERR_INVALID;
  const void* ptrs[] = {h, w, bias, labels, lse, dloss, dh, dw, dbias, workspace};
  for (const void* x : ptrs)
    if (!aligned16(x)) return BB_ERR_INVALID;
  if (!workspace || workspace_bytes < p.total) return BB_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  cudaStream_t s = (cudaStream_t)stream;
  CUtensorMap tmH, tmHp, tmW, tmH64, tmHp64, tmW64, tmDz32, tmDz64, tmDw, tmDh;
  if (!encode_bf16_2d(&tmH, h, hidden, N, hidden, 64, kBM) ||
      !encode_bf16_2d(&tmHp, ws + p.hp, hidden, p.Np, hidden, 64, kBM) ||
      !encode_bf16_2d(&tmW, w, hidden, V, hidden, 64, 128) ||
      !encode_bf16_2d(&tmH64, h, hidden, N, hidden, 64, 64) ||
      !encode_bf16_2d(&tmHp64, ws + p.hp, hidden, p.Np, hidden, 64, 64) ||
      !encode_bf16_2d(&tmW64, w, hidden, V, hidden, 64, 64) ||
      !encode_bf16_2d(&tmDz32, ws + p.dz, p.Vp, p.Np, p.Vp, 64, 32) ||
      !encode_bf16_2d(&tmDz64, ws + p.dz, p.Vp, p.Np, p.Vp, 64, 64) ||
      !encode_bf16_2d(&tmDw, dw, hidden, V, hidden, 64, 32) ||
      !encode_f32_2d(&tmDh, ws + p.dh, hidden, (uint64_t)p.splits * p.Np, hidden, 32, 32))
    return BB_ERR_CUDA;
  RowsArgs r{};
  r.N = N;
  r.D = hidden;
  r.V = V;
  r.labels = labels;
  r.h = static_cast<const uint16_t*>(h);
  r.lse = lse;
  r.dloss = dloss;
  r.info = reinterpret_cast<Info*>(ws);
  r.idx = reinterpret_cast<int*>(ws + p.idx);
  r.pos = reinterpret_cast<int*>(ws + p.pos);
  r.lab = reinterpret_cast<int*>(ws + p.lab);
  r.rlse = reinterpret_cast<float*>(ws + p.rlse);
  r.dls = reinterpret_cast<float*>(ws + p.dls);
  r.hp = reinterpret_cast<uint16_t*>(ws + p.hp);
  rows_kernel<true><<<(N + kRowsPerBlock - 1) / kRowsPerBlock, kRowsPerBlock, 0, s>>>(r);
  if (cudaGetLastError() != cudaSuccess) return BB_ERR_CUDA;
  CeArgs a{};
  a.N = N;
  a.D = hidden;
  a.V = V;
  a.Np = p.Np;
  a.Vp = p.Vp;
  a.splits = p.splits;
  a.info = r.info;
  a.bias = bias;
  a.lab = r.lab;
  a.rlse = r.rlse;
  a.dls = r.dls;
  a.dbp = dbias ? reinterpret_cast<float*>(ws + p.dbp) : nullptr;
  a.dbias = dbias;
  const int sms = sm_count(), mt = p.Np / kTM, dn = (hidden + kTN - 1) / kTN;
  for (int i = 0; i < p.pieces; ++i) {
    a.v0 = i * p.Vp;
    a.vn = V - a.v0 < p.Vp ? V - a.v0 : p.Vp;
    a.add = i > 0;
    const int nt = (a.vn + kTN - 1) / kTN, wm = (a.vn + kTM - 1) / kTM;
    if (launch_gemm<kDz>(a, mt * nt, sms, tmH, tmHp, tmW, tmDz32, tmW, tmW, s) != cudaSuccess ||
        launch_gemm<kGrad>(a, mt * dn * p.splits + wm * dn, sms, tmH64, tmHp64, tmW64, tmDz64,
                           tmDw, tmDh, s) != cudaSuccess)
      return BB_ERR_CUDA;
  }
  dh_round_kernel<<<(unsigned)(((size_t)N * (hidden / 8) + 255) / 256), 256, 0, s>>>(
      a.info, N, hidden, p.Np, p.splits, r.pos, reinterpret_cast<float*>(ws + p.dh),
      static_cast<uint16_t*>(dh));
  return cudaGetLastError() == cudaSuccess ? BB_OK : BB_ERR_CUDA;
}

}  // extern "C"
