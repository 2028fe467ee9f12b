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
// launch (rows_kernel) packs the rows that have one, in order, and sums their
// labels' logits in fp32; when every row has one, h is used where it lies.
//
// Forward: one GEMM over (row tile, vocabulary tile); the epilogue keeps, per
// row, the maximum and the sum of exponentials of its columns of the tile, and
// a small launch merges these pairs in a fixed order.  Logits live in tensor
// memory and registers only.  Where the pairs would not fit a fixed workspace
// (from N V = 2^32 on) the vocabulary goes by in pieces, each merged into one
// running pair per row.
//
// Backward: the vocabulary goes by in pieces whose dz (bf16) fits a fixed
// workspace.  Per piece, one GEMM launch computes the logits again and
// writes dz, and one GEMM launch forms the piece's rows of dW (complete) and
// its part of dh, added to an fp32 sum (one addition per element and launch,
// so the order is fixed); dbias comes from column sums of dz taken before its
// rounding.  A last launch rounds dh.  Without the stored logits this is
// 6 R D V operations (R rows with a label) beside the forward's 2 R D V.
//
// What bounds it, measured on a B200.  Many rows: the tensor cores, and over
// longer runs the power limit (clocks settle near 1.3 GHz): the forward of
// 8192 x 1024 x 50021 takes 599 us back to back (1400 TFLOP/s; one cuBLAS
// product of that size, which also writes its logits, 714), its gradients 2190
// (1150 TFLOP/s over three products).  Few rows: 13 rows of 768 x 30011 take 20 us
// a call (46 MB; 7 at a copy's rate), 13.6 of them in the products, whose 235
// tiles are two rounds on 148 CTAs; the gradients of 77 rows of 776 x 30011 56
// (94 MB; 14.5), 19 in the dz kernel and 33 in that of dW and dh, which read W
// and write dW one after the other.
//
// dz lies in panels of 64 columns, [Vp / 64][Np][64], so that every box that is
// stored or loaded is one piece of memory.  It is held in bf16, the type of the
// tensor-core operands it multiplies; dloss enters it relative to the largest
// |dloss| and that factor is applied in fp32 at the end.
//
// A row of dz has one large entry, its label's, and rounding that one is
// rounding whole rows of dh and dW (errors of 0.22 % at 70 and 512 rows where
// rounding the results gives 0.17; the other entries' roundings average out
// in either product).  So what bf16 leaves of it (`rest`, one fp32 per row) is
// added back: rest x w[label] to the row of dh when that is rounded, rest x
// h[row] to the label's row of dW, for words with at most kFix rows (more
// average out too).  The rows of each word are listed under the first dz
// launch.  Few rows make dW's tiles short and all epilogue: there the fp32
// sums of a word that is a label go to memory and the last launch adds to them
// and rounds (in the epilogue, waiting for the rows of h, 129 and 256 rows took
// 58.4 and 60.5 us where this takes 53.5 and 56.2); many rows hide the wait
// under the products.  It costs 1.6 us of 54 at 77 rows, 2 at 129 and 256, 3.5 of
// 75.5 at 512, 2.5 of 123 at 1024, below 1 % from 4096 on.
//
// Up to 64 rows the other entries do not average out either (errors of 0.38 %).
// There dz is held in two parts, the second being what rounding left of the
// first, as further rows (from `low` on, 32 or 64): dW's K runs over both with
// h packed twice, and dh's rows are summed in pairs.  A tile has room for 128
// rows, so the gradients of 1 and of 64 rows take 47.7 and 51.3 us where bf16
// alone took 44.3 and 46.1.
#include "ce_runs.h"
#include "layer.cuh"

namespace bb {
namespace {

using namespace sm100;

constexpr int kSms = 148;                      // a B200's
constexpr int kBM = 128, kBK = 64;             // rows of a CTA's tile, K step
constexpr uint32_t kBox = 64 * 64 * 2;         // one 64 x 64 bf16 box: 8 KB
constexpr uint32_t kATile = kBM * kBK * 2;     // 16 KB
constexpr int kResA = 5;                       // A stages beside a resident B (below)
constexpr size_t kPieceBytes = 256u << 20;     // dz, or (max, sum) pairs, of one vocabulary piece
constexpr int kFix = 4;                        // most rows of a word whose entries are exact
constexpr int kSideRows = 1024;  // up to these rows the last launch adds what bf16 left to dW,
                                // above the epilogue (256 rows 56 and 60.5 us, 1024 128 and 129)

enum Mode { kLse = 0, kDz = 1, kGrad = 2 };

// Tile shapes.  Pairs of CTAs (cta_group::2) form 256 x 256 tiles: 128 rows of
// A and 128 columns of B in each CTA's shared memory.  Up to 128 rows a pair's
// second half would be empty, and the vocabulary's weights bound the launch:
// single CTAs take 128 x 128 logits (enough tiles to keep every SM loading)
// and 128 x 256 gradients.  There a dW tile's B, up to 128 rows of 256 columns
// of h, is the same for every tile of those columns: it stays in shared
// memory while the CTA walks down the words, and the freed stages hold A's.
// Two accumulators, so that a tile's epilogue runs under the next one's MMAs.
template <int kMode, bool kPair>
struct Cfg {
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kTM = kBM * kCtas;
  static constexpr int kTN = kPair || kMode == kGrad ? 256 : 128;
  static constexpr int kEpi = 8;                           // epilogue warps
  static constexpr int kCols = kTN / (kEpi / 4);           // columns of one (logits)
  // Staging blocks of one.  A pair's gradient tiles are long: a sixth stage
  // gives more than a second block (1-2 % at 256 to 1024 rows).
  static constexpr int kSlots = kMode == kLse ? 0 : kMode == kGrad && !kPair ? 2 : 1;
  static constexpr uint32_t kBTile = kTN / kCtas * kBK * 2;
  static constexpr uint32_t kStage = kATile + kBTile;
  static constexpr int kStages =
      kPair ? (kMode == kGrad ? 6 : 5) : kMode == kLse ? 6 : kMode == kDz ? 5 : 3;
  static constexpr uint32_t kOut = kEpi * kSlots * 4096;   // 32 x 128 B staging blocks
  static constexpr uint32_t kSmem = 1024 + kStages * kStage + kOut;
  static constexpr int kThreads = 64 + 32 * kEpi;
  static constexpr uint32_t kTmem = 2 * kTN;               // columns: two accumulators
};

// Cost of a gradient tile in K steps: a short one takes as long as its
// epilogue, measured as four.
__host__ __device__ constexpr int tile_cost(int ksteps) { return ksteps < 4 ? 4 : ksteps; }

// What rows_kernel finds out on the device, at the workspace's start.
struct Info {
  int status;
  int pad[15];
  int rows;      // rows with a label
  int direct;    // 1: every row has one, h is read where it lies
  int low;       // backward, dz in two parts: first row of the second; else 0
  float dlref;   // largest |dloss| of those rows (1 when that is 0 or not finite)
};

struct CeArgs {
  int N, D, V;
  int Np;            // N rounded up to a tile's rows
  int Vp;            // columns of a piece (a multiple of 256)
  int v0, vn;        // this piece: first column, columns
  int splits;        // parts the piece's columns are cut into for dh
  int a_bytes;       // logits: bytes of h's box per K step (its rows, at most kBM)
  int add;           // dh partials: 1 adds to what earlier pieces wrote
  Info* info;
  const float* bias;   // [V] or null
  const int* lab;      // packed rows: label,
  const float* rlse;   //   lse,
  const float* dls;    //   dloss / dlref,
  const float* zl;     //   logit of the label (rows_kernel)
  float2* part;        // [Plan::runs][Np] (max, sum of exponentials)
  uint16_t* dz;        // [Vp / 64][Np][64]
  // Where dz is in one part (see the top):
  float* rest;         // packed rows: what bf16 leaves of the label's dz
  unsigned* word_bits; // [V / 32]: the words that are labels,
  int *word_n, *word_rows;  // [V], [kFix][V]: and the packed rows that have them
  float* side;         // [N][D], by the first row of a word's list: its sums of dW; or null
  const uint16_t *h, *hp;   // rows of h as they lie, and packed (without side)
  float* dbp;          // [Np / 128][Vp] column sums of dz, or null
  float* dbias;        // [V], with dbp
  int dw_start[kSms + 1];  // kGrad of single CTAs: first tile of dW of each
};

struct Bars {
  uint64_t full[6], empty[6], acc_full[2], acc_empty[2], red;
  uint64_t a_full[kResA], a_empty[kResA], b_full;  // dW of a single CTA
};

// One output tile.
struct Job {
  int dw;           // kGrad: 1 = a tile of dW, 0 = of dh
  int m0, n0;       // first row and column of the tile
  int k0, ksteps;   // first K index, 64-wide K steps
  int nblk;         // 64-column blocks of B in each CTA
  int row0;         // first row in the output
};

// A launch's tiles and the share of each worker (a pair or a single CTA).
//
// Logits: every worker takes every `stride`-th tile.  Gradients: tiles of two
// costs, dh's (K: the piece's columns, cut into `splits`) and dW's (K: the
// rows).  The dearer kind is dealt out first; workers that got one fewer of
// it take `lead` more of the cheaper kind before that is dealt out to all, so
// the workers end within about one cheap tile of each other.  Single CTAs take
// their tiles of dh, then a run of dW's tiles, ordered by columns first so that
// h's part is loaded once or twice; the host cuts the runs (dw_runs).
template <int kMode, bool kPair>
struct Work {
  using C = Cfg<kMode, kPair>;
  int w, stride;                  // this worker, workers
  int tiles, mt, dn, hks, wks;
  int dw_first, na, nb, more, lead;  // kinds in order; workers with one more of the first
  int wm, dw0, dw1;                  // single CTAs: row tiles of dW; this one's run
  __device__ __forceinline__ Work(const CeArgs& a, int rows, int worker, int workers)
      : w(worker), stride(workers) {
    mt = (rows + C::kTM - 1) / C::kTM;
    if (kMode != kGrad) {
      tiles = mt * ((a.vn + C::kTN - 1) / C::kTN);
      return;
    }
    dn = (a.D + C::kTN - 1) / C::kTN;
    hks = (a.vn + kBK - 1) / kBK;
    wks = (rows + kBK - 1) / kBK;
    const int nh = mt * dn * a.splits, nw = (a.vn + C::kTM - 1) / C::kTM * dn;
    const int ch = tile_cost(hks / a.splits), cw = tile_cost(wks);
    if (!kPair) {
      dw_first = 0;
      na = nh;
      wm = nw / dn;
      more = nh % stride;
      dw0 = a.dw_start[w];
      dw1 = a.dw_start[w + 1];
      return;
    }
    dw_first = cw > ch;
    na = dw_first ? nw : nh;
    nb = dw_first ? nh : nw;
    more = na % stride;
    const int ca = dw_first ? cw : ch, cb = dw_first ? ch : cw, fewer = stride - more;
    lead = more ? (ca + cb / 2) / cb : 0;
    if (lead > nb / fewer) lead = nb / fewer;
  }
  // The i-th tile of this worker, or -1 after its last.
  __device__ __forceinline__ int tile(int i) const {
    if (kMode != kGrad) {
      const int t = w + i * stride;
      return t < tiles ? t : -1;
    }
    const int mine = na / stride + (w < more);
    if (i < mine) return i * stride + w;
    i -= mine;
    if (!kPair) return dw0 + i < dw1 ? na + dw0 + i : -1;
    int u;
    if (w >= more) {
      if (i < lead) return na + i * (stride - more) + (w - more);
      i -= lead;
    }
    u = lead * (stride - more) + i * stride + w;
    return u < nb ? na + u : -1;
  }
  __device__ __forceinline__ Job job(const CeArgs& a, int t) const {
    Job j;
    j.nblk = C::kTN / C::kCtas / 64;
    if (kMode != kGrad) {
      // Row tiles run fastest: the rows stay in L2 while W streams by once.
      j.dw = 0;
      j.m0 = (t % mt) * C::kTM;
      j.n0 = (t / mt) * C::kTN;
      j.k0 = 0;
      j.ksteps = (a.D + kBK - 1) / kBK;
      j.row0 = j.m0;
      return j;
    }
    j.dw = dw_first ? t < na : t >= na;
    int u = t < na ? t : t - na;
    if (!kPair && j.dw) u = u % wm * dn + u / wm;  // columns first
    j.n0 = (u % dn) * C::kTN;
    const int left = (a.D - j.n0 + 64 * C::kCtas - 1) / (64 * C::kCtas);
    j.nblk = left < j.nblk ? left : j.nblk;
    u /= dn;
    if (j.dw) {
      j.m0 = u * C::kTM;
      j.k0 = 0;
      j.ksteps = wks;
      j.row0 = a.v0 + j.m0;
    } else {
      const int s = u / mt;
      j.m0 = (u % mt) * C::kTM;
      j.k0 = (int)((long long)hks * s / a.splits);
      j.ksteps = (int)((long long)hks * (s + 1) / a.splits) - j.k0;
      j.row0 = s * a.Np + j.m0;
    }
    return j;
  }
};

// Sum over the 32 lanes of each of 32 columns held one row per lane; lane l
// returns column l.  Each step halves the columns a lane carries.
__device__ __forceinline__ float column_sums(const float2 (&z)[16], int lane) {
  float x[32];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    x[2 * e] = z[e].x;
    x[2 * e + 1] = z[e].y;
  }
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

// 32 logits of a row from its accumulator columns and their bias (in shared
// memory, the same for every lane).
__device__ __forceinline__ void add_bias(const uint32_t (&v)[32], const float* bias,
                                         float2 (&z)[16]) {
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const float4 b = *reinterpret_cast<const float4*>(bias + e);
    z[e / 2] = add2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])),
                    make_float2(b.x, b.y));
    z[e / 2 + 1] = add2(make_float2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])),
                        make_float2(b.z, b.w));
  }
}

// Element i of a row's 32 values, where 0 <= i < 32, becomes x.
__device__ __forceinline__ void put(float2 (&z)[16], int i, float x) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    z[e].x = i == 2 * e ? x : z[e].x;
    z[e].y = i == 2 * e + 1 ? x : z[e].y;
  }
}

// What bf16 leaves of x (of an infinity nothing).
__device__ __forceinline__ float bf16_rest(float x) {
  const float k = __uint_as_float(pack_bf16(0.f, x) & 0xFFFF0000u);
  return x == k ? 0.f : x - k;
}

// Appends packed rows to their labels' lists, a row per lane.  rows_kernel has
// cleared the bits, and the counts of the words that are labels (the other
// words' counts and lists are whatever the workspace held).
__device__ __forceinline__ void append_rows(const CeArgs& a, int row, int rows) {
  const int v = row < rows ? a.lab[row] : -1, lane = threadIdx.x & 31;
  const unsigned same = __match_any_sync(0xffffffffu, v);
  const int leader = __ffs(same) - 1;
  int at = 0;
  if (v >= 0 && lane == leader) {
    atomicOr(a.word_bits + v / 32, 1u << (v & 31));
    at = atomicAdd(a.word_n + v, __popc(same));
  }
  at = __shfl_sync(0xffffffffu, at, leader) + __popc(same & ((1u << lane) - 1));
  if (v >= 0 && at < kFix) a.word_rows[(size_t)at * a.V + v] = row;
}

// The n <= kFix rows of word v's list in order (the appends were not).
__device__ __forceinline__ void word_rows(const int* lists, int V, int v, int n,
                                          int (&p)[kFix]) {
#pragma unroll
  for (int k = 0; k < kFix; ++k) p[k] = k < n ? lists[(size_t)k * V + v] : 0x7FFFFFFF;
#pragma unroll
  for (int i = 1; i < kFix; ++i)
#pragma unroll
    for (int k = kFix - 1; k >= i; --k) {
      const int lo = min(p[k - 1], p[k]), hi = max(p[k - 1], p[k]);
      p[k - 1] = lo;
      p[k] = hi;
    }
}

// v += r times eight bf16 values; v as floats or as their bits.
__device__ __forceinline__ void fma_to(float& v, float r, float x) { v = fmaf(r, x, v); }
__device__ __forceinline__ void fma_to(uint32_t& v, float r, float x) {
  v = __float_as_uint(fmaf(r, x, __uint_as_float(v)));
}
template <typename T>
__device__ __forceinline__ void fma8(float r, const uint4& x, T* v) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    fma_to(v[2 * i], r, __uint_as_float(u[i] << 16));
    fma_to(v[2 * i + 1], r, __uint_as_float(u[i] & 0xFFFF0000u));
  }
}

template <int kMode, bool kPair>
__global__ void __launch_bounds__(Cfg<kMode, kPair>::kThreads, 1)
    ce_gemm_kernel(const __grid_constant__ CeArgs a, const __grid_constant__ CUtensorMap tmH,
                   const __grid_constant__ CUtensorMap tmHp,
                   const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ CUtensorMap tmDz,
                   const __grid_constant__ CUtensorMap tmDw,
                   const __grid_constant__ CUtensorMap tmDh) {
  using C = Cfg<kMode, kPair>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile int abort_flag;
  __shared__ float red[2][4][kMode == kDz ? C::kTN : 1];  // column sums of 32 rows
  __shared__ __align__(16) float bias_sh[kMode == kGrad ? 1 : C::kEpi][C::kCols];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_rank() : 0;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* stages = base;                                 // [kStages][A | B]
  uint8_t* stage_out = base + C::kStages * C::kStage;     // [warps][slots][32][128 B]
  int* status = &a.info->status;

  // Barriers of a pair: `full` and `acc_empty` are used in rank 0 only (it
  // issues the MMAs); both CTAs' loads and epilogue warps signal them there.
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.acc_full[s], 1);
      mbar_init(&bars.acc_empty[s], C::kCtas * C::kEpi);
    }
    mbar_init(&bars.red, C::kEpi);
    for (int s = 0; s < kResA; ++s) {
      mbar_init(&bars.a_full[s], 1);
      mbar_init(&bars.a_empty[s], 1);
    }
    mbar_init(&bars.b_full, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    if (kPair) {
      tmem_alloc_pair(&tmem_base_sh, C::kTmem);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&tmem_base_sh, C::kTmem);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  grid_launch_dependents();
  grid_wait();
  const int low = kMode == kLse ? 0 : a.info->low;
  const int rows = kMode == kGrad && low ? 2 * low : a.info->rows;
  const CUtensorMap* mapH = a.info->direct && !(kMode == kGrad && low) ? &tmH : &tmHp;
  const Work<kMode, kPair> work(a, rows, blockIdx.x / C::kCtas, gridDim.x / C::kCtas);

  if (warp == 0) {
    // ---------------- TMA loads ----------------
    {
      uint32_t it = 0, ia = 0;  // loads of the ring; of A beside a resident B
      int n_res = -1;           // columns of the resident B
      // dh of up to 64 rows: the lower half of A reaches no row that is used.
      const int a_boxes = !kPair && rows <= 64 ? 1 : 2;
      bool ok = true;
      auto load = [&](const uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
        tma_load_2d_warp(kPair, smem_u32(dst), map, kPair ? map_rank(bar, 0) : smem_u32(bar), x, y);
      };
      // Waits until the MMAs have released every stage loaded so far.
      auto drained = [&]() {
        bool done = true;
        for (uint32_t q = it > C::kStages ? it - C::kStages : 0; q < it && done; ++q)
          done = mbar_wait_warp(&bars.empty[q % C::kStages], (q / C::kStages) & 1, &abort_flag, status);
        for (uint32_t q = ia > kResA ? ia - kResA : 0; q < ia && done; ++q)
          done = mbar_wait_warp(&bars.a_empty[q % kResA], (q / kResA) & 1, &abort_flag, status);
        return done;
      };
      for (int i = 0, t; ok && (t = work.tile(i)) >= 0; ++i) {
        const Job j = work.job(a, t);
        if (!kPair && kMode == kGrad && j.dw) {
          if (n_res != j.n0 && j.ksteps > 0) {
            // Every MMA on what the stages and the old B hold is done.
            ok = drained();
            if (!ok) break;
            n_res = j.n0;
            mbar_expect_tx_warp(&bars.b_full, j.ksteps * j.nblk * kBox);
            for (int k = 0; k < j.ksteps; ++k)
              for (int b = 0; b < j.nblk; ++b)
                load(stages + (k * 4 + b) * kBox, mapH, &bars.b_full, j.n0 + 64 * b, k * kBK);
          }
          for (int k = 0; k < j.ksteps; ++k, ++ia) {
            const uint32_t st = ia % kResA;
            ok = mbar_wait_warp(&bars.a_empty[st], ((ia / kResA) & 1) ^ 1, &abort_flag, status);
            if (!ok) break;
            mbar_expect_tx_warp(&bars.a_full[st], kATile);
            for (int b = 0; b < 2; ++b)
              load(stages + 8 * kBox + st * kATile + b * kBox, &tmDz, &bars.a_full[st], 0,
                   (j.m0 / 64 + b) * a.Np + k * kBK);
          }
          continue;
        }
        // Single CTAs all read the same few rows of h: each tile begins at
        // another K step, or all would wait for the same lines of L2.
        const int k_first = !kPair && kMode != kGrad ? t % j.ksteps : 0;
        const int m0 = j.m0 + rank * kBM, n0 = j.n0 + rank * 64 * j.nblk;
        for (int ks = 0; ks < j.ksteps; ++ks, ++it) {
          const uint32_t st = it % C::kStages;
          if (!mbar_wait_warp(&bars.empty[st], ((it / C::kStages) & 1) ^ 1, &abort_flag, status)) {
            ok = false;
            break;
          }
          uint8_t* pa = stages + st * C::kStage;
          uint8_t* pb = pa + kATile;
          uint64_t* bar = &bars.full[st];
          if (rank == 0)
            mbar_expect_tx_warp(bar, C::kCtas * ((kMode == kGrad ? a_boxes * kBox : a.a_bytes) +
                                                 j.nblk * kBox));
          const int kr = k_first + ks;
          const int k = (j.k0 + (kr < j.ksteps ? kr : kr - j.ksteps)) * kBK;
          if (kMode != kGrad) {
            load(pa, mapH, bar, k, m0);
            load(pb, &tmW, bar, k, a.v0 + n0);
          } else {
            // dW: A = dz^T (columns of dz along M), B = h; dh: A = dz, B = W.
            // A 64 x 64 box of a panel of dz is 8 KB in one piece.
            for (int i = 0; i < a_boxes; ++i)
              load(pa + i * kBox, &tmDz, bar, 0,
                   j.dw ? (m0 / 64 + i) * a.Np + k : k / 64 * a.Np + m0 + 64 * i);
            for (int i = 0; i < j.nblk; ++i)
              load(pb + i * kBox, j.dw ? mapH : &tmW, bar, n0 + 64 * i, j.dw ? k : a.v0 + k);
          }
        }
      }
      // The last stages' releases reach this CTA before it may leave.
      if (ok) drained();
      if (abort_flag && rank == 0) {
        // Let issued copies (both CTAs') land before shared memory goes away;
        // rank 1 waits at the cluster barrier meanwhile.
        for (uint32_t s = 0; s < (uint32_t)C::kStages; ++s)
          if (it >= s + 1) {
            const uint32_t last = it - 1 - ((it - 1 - s) % C::kStages);
            const uint64_t t0 = globaltimer();
            while (!mbar_try_wait(&bars.full[s], (last / C::kStages) & 1) &&
                   globaltimer() - t0 < 100000000ull) {
            }
          }
        if (!kPair && kMode == kGrad) {
          const uint64_t t0 = globaltimer();
          for (uint32_t q = ia > kResA ? ia - kResA : 0; q < ia; ++q)
            while (!mbar_try_wait(&bars.a_full[q % kResA], (q / kResA) & 1) &&
                   globaltimer() - t0 < 100000000ull) {
            }
          // B's latest load: its phase is the number of columns taken so far,
          // which this wait does not know; it gives the copy time to land.
          while (n_res >= 0 && globaltimer() - t0 < 1000000ull) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issue (rank 0) ----------------
    uint32_t it = 0, tc = 0, ia = 0, ib = 0;
    int n_res = -1;
    bool ok = rank == 0;
    for (int t; ok && (t = work.tile(tc)) >= 0; ++tc) {
      const Job j = work.job(a, t);
      const int acc = tc & 1;
      if (!mbar_wait_warp(&bars.acc_empty[acc], ((tc >> 1) & 1) ^ 1, &abort_flag, status)) break;
      tc_fence_after();
      // K-major tiles step 32 bytes per 16 of K; MN-major ones 16 rows of 128.
      const uint32_t a_mn = kMode == kGrad && j.dw, b_mn = kMode == kGrad;
      const uint32_t idesc = idesc_bf16(C::kTM, 64 * C::kCtas * j.nblk, a_mn, b_mn);
      const uint32_t astep = a_mn ? 2048 : 32, bstep = b_mn ? 2048 : 32;
      const uint32_t albo = a_mn ? kBox : 16, blbo = b_mn ? kBox : 16;
      if (!kPair && kMode == kGrad && j.dw) {
        if (n_res != j.n0 && j.ksteps > 0) {
          ok = mbar_wait_warp(&bars.b_full, ib & 1, &abort_flag, status);
          if (!ok) break;
          n_res = j.n0;
          ++ib;
        }
        for (int k = 0; k < j.ksteps; ++k, ++ia) {
          const uint32_t st = ia % kResA;
          ok = mbar_wait_warp(&bars.a_full[st], (ia / kResA) & 1, &abort_flag, status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t aaddr = smem_u32(stages + 8 * kBox + st * kATile);
          const uint32_t baddr = smem_u32(stages + 4 * k * kBox);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss_warp(false, tmem + acc * C::kTN, sdesc_sw128(aaddr + kk * 2048, kBox),
                        sdesc_sw128(baddr + kk * 2048, kBox), idesc, (k > 0 || kk > 0) ? 1u : 0u);
          mma_commit_warp(false, &bars.a_empty[st]);
        }
        if (ok) mma_commit_warp(false, &bars.acc_full[acc]);
        continue;
      }
      for (int ks = 0; ks < j.ksteps; ++ks, ++it) {
        const uint32_t st = it % C::kStages;
        if (!mbar_wait_warp(&bars.full[st], (it / C::kStages) & 1, &abort_flag, status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t aaddr = smem_u32(stages + st * C::kStage);
        const uint32_t baddr = aaddr + kATile;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ss_warp(kPair, tmem + acc * C::kTN, sdesc_sw128(aaddr + kk * astep, albo),
                      sdesc_sw128(baddr + kk * bstep, blbo), idesc,
                      (ks > 0 || kk > 0) ? 1u : 0u);
        mma_commit_warp(kPair, &bars.empty[st]);
      }
      if (ok) mma_commit_warp(kPair, &bars.acc_full[acc]);
    }
  } else {
    // ------- epilogue (32 rows and, of eight warps, half of the columns each) -------
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    uint8_t* stage = stage_out + (warp - 2) * C::kSlots * 4096;
    uint8_t* rowp = stage + lane * 128;
    const int swz = lane & 7;
    const float dlref = kMode == kGrad ? a.info->dlref : 1.f;
    auto release = [&](int acc) {  // the accumulator is read
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kPair)
          mbar_arrive_cluster(map_rank(&bars.acc_empty[acc], 0));
        else
          mbar_arrive(&bars.acc_empty[acc]);
      }
    };
    const int hi_rows = low ? low : 2 * kBM;  // kDz: rows of dz, or of its first part
    int slot = 0;  // kGrad: staging slot of the latest store
    float m = -INFINITY, s = 0.f;  // kLse: maximum and sum of exponentials
    const int r0 = rank * kBM + quarter * 32;  // this warp's first row in a tile
    // This tile and, kGrad, the next two (a tile's place takes several
    // divisions: each is worked out once).
    struct Place {
      int t;
      Job j;
    } at[3];
    auto place = [&](Place& p, int i) {
      p.t = work.tile(i);
      if (p.t >= 0) p.j = work.job(a, p.t);
    };
    place(at[0], 0);
    if (kMode == kGrad) {
      place(at[1], 1);
      place(at[2], 2);
    }
    // kGrad, dz in one part: which of the warp's words of a tile are labels,
    // loaded two tiles ahead, and one tile ahead the first row of the lane's
    // word if it is one, so that nothing waits for them.
    const bool fix = kMode == kGrad && !low && rows > 0;
    auto word_bits = [&](const Place& p) {
      const int v = p.j.row0 + r0;
      return p.t >= 0 && p.j.dw && v < a.V ? a.word_bits[v / 32] : 0u;
    };
    auto list_head = [&](unsigned bits, const Place& p) {
      return (bits >> lane) & 1u ? a.word_rows[p.j.row0 + r0 + lane] : -1;
    };
    unsigned bits1 = 0;
    int head1 = -1;  // of the next tile
    if (fix) {
      head1 = list_head(word_bits(at[0]), at[0]);
      bits1 = word_bits(at[1]);
    }
    if (kMode == kDz && !low && !a.add)  // under the first tile's loads
      for (int i = (blockIdx.x * C::kEpi + warp - 2) * 32; i < rows;
           i += gridDim.x * C::kEpi * 32)
        append_rows(a, i + lane, rows);
    uint32_t tc = 0;
    auto advance = [&]() {
      ++tc;
      if (kMode == kGrad) {
        at[0] = at[1];
        at[1] = at[2];
        place(at[2], tc + 2);
      } else {
        place(at[0], tc);
      }
    };
    for (; at[0].t >= 0; advance()) {
      const Job j = at[0].j;
      const int acc = tc & 1;
      const int row = j.m0 + r0 + lane;          // packed row (logits)
      const bool live = row < rows;
      const int cbeg = half * C::kCols;
      int lab = -1;
      float zl = 0.f, lse = 0.f, dl = 0.f;
      if (kMode != kGrad) {
        // What the tile's epilogue reads besides the logits, under its MMAs.
        // Words past V are excluded.
        float b[C::kCols / 32];
#pragma unroll
        for (int i = 0; i < C::kCols / 32; ++i) {
          const int v = a.v0 + j.n0 + cbeg + 32 * i + lane;
          b[i] = v < a.V ? (a.bias ? a.bias[v] : 0.f) : -INFINITY;
        }
        if (live) {
          lab = a.lab[row];
          zl = a.zl[row];
          if (kMode == kDz) {
            lse = a.rlse[row];
            dl = a.dls[row];
          }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < C::kCols / 32; ++i) bias_sh[warp - 2][32 * i + lane] = b[i];
        __syncwarp();
      }
      int head = -1;  // kGrad: first row of the lane's word's list
      if (fix) {
        head = head1;
        head1 = list_head(bits1, at[1]);
        bits1 = word_bits(at[2]);
      }
      if (!mbar_wait_warp(&bars.acc_full[acc], (tc >> 1) & 1, &abort_flag, status)) break;
      tc_fence_after();
      const uint32_t tz = tmem + acc * C::kTN + lane_off;
      if (kMode != kGrad) {
        // Single CTAs see the same rows in every tile: one pair runs through.
        if (kPair) {
          m = -INFINITY;
          s = 0.f;
        }
        uint32_t v[32];
        __syncwarp();
        tmem_ld32(tz + cbeg, v);
#pragma unroll
        for (int c = 0; c < C::kCols; c += 32) {
          float2 z[16];
          tmem_ld_wait();
          add_bias(v, bias_sh[warp - 2] + c, z);
          if (c + 32 < C::kCols) tmem_ld32(tz + cbeg + c + 32, v);
          // The label's column of these 32.  Its logit is the one that
          // rows_kernel summed in fp32: the tensor core truncates its running
          // sum at every step, and the largest logits, mostly the labels',
          // show it first.
          const int hot = lab - a.v0 - j.n0 - cbeg - c;
          if (kMode == kLse) {
            if ((unsigned)hot < 32u) put(z, hot, zl);
            __syncwarp();
            float cm = m;
#pragma unroll
            for (int e = 0; e < 16; ++e) cm = fmax3(cm, z[e].x, z[e].y);
            // A row of -inf so far keeps a finite reference.  Differences are
            // taken before the scaling to base 2, so logits near the type's
            // lowest value do not overflow.
            const float ref = cm == -INFINITY ? 0.f : cm;
            float2 sum = make_float2(s * ex2((m - ref) * kLog2e), 0.f);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 d = mul2(sub2(z[e], make_float2(ref, ref)),
                                    make_float2(kLog2e, kLog2e));
              sum = add2(sum, make_float2(ex2(d.x), ex2(d.y)));
            }
            s = sum.x + sum.y;
            m = cm;
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 d = mul2(sub2(z[e], make_float2(lse, lse)),
                                    make_float2(kLog2e, kLog2e));
              z[e] = mul2(make_float2(ex2(d.x), ex2(d.y)), make_float2(dl, dl));
            }
            if ((unsigned)hot < 32u) {
              const float x = dl * (ex2((zl - lse) * kLog2e) - 1.f);
              put(z, hot, x);
              if (!low) a.rest[row] = bf16_rest(x);
            }
            // Rows past the last: exact zeros, whatever the accumulator held.
            if (!live) {
#pragma unroll
              for (int e = 0; e < 16; ++e) z[e] = make_float2(0.f, 0.f);
            }
            __syncwarp();
            // Staged and stored by TMA: 32-byte stores of a row per lane took the
            // gradients of 1024 rows 4 % longer, those of 8192 1.6 %.
            if ((c & 32) == 0) {
              // The previous block's store has read the staging block.
              if (lane == 0) bulk_wait_read_all();
              __syncwarp();
            }
#pragma unroll
            for (int ch = 0; ch < 4; ++ch)
              *reinterpret_cast<uint4*>(rowp + ((((c & 32) / 8 + ch) ^ swz) << 4)) =
                  make_uint4(pack_bf16(z[4 * ch].x, z[4 * ch].y),
                             pack_bf16(z[4 * ch + 1].x, z[4 * ch + 1].y),
                             pack_bf16(z[4 * ch + 2].x, z[4 * ch + 2].y),
                             pack_bf16(z[4 * ch + 3].x, z[4 * ch + 3].y));
            if (low > r0) {
              // What the rounding left (an infinity leaves nothing).
              uint32_t u[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const uint32_t k = pack_bf16(z[e].x, z[e].y);
                const float x = __uint_as_float(k << 16), y = __uint_as_float(k & 0xFFFF0000u);
                u[e] = pack_bf16(z[e].x == x ? 0.f : z[e].x - x, z[e].y == y ? 0.f : z[e].y - y);
              }
              uint4* out = reinterpret_cast<uint4*>(
                  a.dz + ((size_t)((j.n0 + cbeg + c) / 64) * a.Np + low + r0 + lane) * 64 + (c & 32));
#pragma unroll
              for (int e = 0; e < 4; ++e)
                out[e] = make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
            }
            // (The rows from `low` on are the second part's.)
            if ((c & 32) && r0 < hi_rows) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_2d(&tmDz, stage, 0, (j.n0 + cbeg + c) / 64 * a.Np + j.m0 + r0);
                bulk_commit_group();
              }
            }
            if (a.dbp) red[acc][quarter][cbeg + c + lane] = column_sums(z, lane);
          }
        }
        release(acc);
        if (kMode == kLse) {
          if (kPair)
            a.part[(size_t)((j.n0 + cbeg) / C::kCols) * a.Np + row] = make_float2(m, s);
          else if (work.tile(tc + 1) < 0)
            a.part[(size_t)(2 * work.w + half) * a.Np + row] = make_float2(m, s);
        } else if (a.dbp) {
          // Column sums of the CTA's 128 rows: the four quarters' sums in order.
          if (lane == 0) mbar_arrive_release(&bars.red);
          if (!mbar_wait_warp(&bars.red, tc & 1, &abort_flag, status)) break;
          for (int c = (warp - 2) * 32 + lane; c < C::kTN; c += 32 * C::kEpi)
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
      // The next staging slot, once the store that used it has read it.
      auto next_slot = [&]() {
        slot = C::kSlots - 1 - slot;
        if (lane == 0) {
          if (C::kSlots > 1)
            bulk_wait_read_but_one();
          else
            bulk_wait_read_all();
        }
        __syncwarp();
        return rowp + slot * 4096;
      };
#pragma unroll 1
      for (int cb = half; cb < C::kCtas * j.nblk; cb += 2) {
        uint32_t v0[32], v1[32];
        __syncwarp();
        tmem_ld32(tz + cb * 64, v0);
        tmem_ld32(tz + cb * 64 + 32, v1);
        tmem_ld_wait();
        if (j.ksteps == 0) {  // no rows at all: zero, whatever the accumulator holds
#pragma unroll
          for (int e = 0; e < 32; ++e) v0[e] = v1[e] = 0u;
        }
        const int y = j.row0 + r0, x = j.n0 + cb * 64;
        // Boxes that start past the tensor's end, and rows of dh behind the
        // last, have nothing to write.
        if (x >= a.D || (j.dw ? y >= a.V : j.m0 + r0 >= rows)) continue;
        if (j.dw) {
          if (head >= 0) {
            if (a.side) {
              float* side = a.side + (size_t)head * a.D + x;
#pragma unroll
              for (int ch = 0; ch < 16; ++ch)
                if (x + 4 * ch < a.D) {
                  const uint32_t* src = ch < 8 ? v0 + 4 * ch : v1 + 4 * (ch - 8);
                  *reinterpret_cast<uint4*>(side + 4 * ch) =
                      make_uint4(src[0], src[1], src[2], src[3]);
                }
            } else {
              const int n = a.word_n[y + lane];
              int p[kFix];
              if (n <= kFix) {
                word_rows(a.word_rows, a.V, y + lane, n, p);
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                  int row = p[0];
#pragma unroll
                  for (int k = 1; k < kFix; ++k) row = i == k ? p[k] : row;
                  const float r = a.rest[row];
                  const uint4* src = reinterpret_cast<const uint4*>(
                      (a.info->direct ? a.h : a.hp) + (size_t)row * a.D + x);
#pragma unroll
                  for (int ch = 0; ch < 8; ++ch)
                    if (x + 8 * ch < a.D)
                      fma8(r, src[ch], ch < 4 ? v0 + 8 * ch : v1 + 8 * (ch - 4));
                }
              }
            }
          }
          __syncwarp();
          uint8_t* out = next_slot();
#pragma unroll
          for (int ch = 0; ch < 8; ++ch) {
            const uint32_t* src = ch < 4 ? v0 + 8 * ch : v1 + 8 * (ch - 4);
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 g = mul2(make_float2(__uint_as_float(src[2 * e]),
                                                __uint_as_float(src[2 * e + 1])),
                                    make_float2(dlref, dlref));
              u[e] = pack_bf16(g.x, g.y);
            }
            *reinterpret_cast<uint4*>(out + ((ch ^ swz) << 4)) =
                make_uint4(u[0], u[1], u[2], u[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmDw, stage + slot * 4096, x, y);
            bulk_commit_group();
          }
        } else {
          // fp32: two boxes of 32 columns.
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (x + 32 * i >= a.D) break;
            const uint32_t* v = i ? v1 : v0;
            uint8_t* out = next_slot();
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)
              *reinterpret_cast<uint4*>(out + ((ch ^ swz) << 4)) =
                  make_uint4(v[4 * ch], v[4 * ch + 1], v[4 * ch + 2], v[4 * ch + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (a.add)
                tma_reduce_add_2d(&tmDh, stage + slot * 4096, x + 32 * i, y);
              else
                tma_store_2d(&tmDh, stage + slot * 4096, x + 32 * i, y);
              bulk_commit_group();
            }
          }
        }
      }
      release(acc);
    }
    if (kMode != kLse && lane == 0) bulk_wait_all();  // output stores complete
  }

  // Neither CTA leaves while the other may still signal its barriers.
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if (kPair)
      tmem_dealloc_pair(tmem, C::kTmem);
    else
      tmem_dealloc(tmem, C::kTmem);
  }
}

// ---- packing the rows that have a label ------------------------------------

struct RowsArgs {
  int N, D, V;
  int per_block;        // rows of a block
  const int32_t* labels;
  const uint16_t *h, *w;
  const float* bias;    // or null
  const float* lse;     // backward
  const float* dloss;   // backward
  float *loss, *lse_out;  // forward: zeroed where there is no label
  Info* info;
  int *idx, *pos, *lab, *word_n;
  unsigned* word_bits;
  float *rlse, *dls, *zl;
  uint16_t* hp;         // packed rows of h
};

constexpr int kRowsThreads = 256;
constexpr int kTwice = 64;  // the most rows whose dz is held in two parts: a tile's half
static_assert(2 * kTwice <= kBM, "both parts in one tile, and in Np rows");

__device__ __forceinline__ float dot8(const uint4& x, const uint4& y, float s) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16), s);
    s = fmaf(__uint_as_float(u[i] & 0xFFFF0000u), __uint_as_float(v[i] & 0xFFFF0000u), s);
  }
  return s;
}

// Block b takes per_block rows, 32 at a time: it packs those that have a label and
// computes their label's logit in fp32.  Each block reads all labels (and
// dloss) to find how many rows with a label lie before its own, so one
// launch does; labels are a few KB to a few hundred and come from L2.
template <bool kBwd>
__global__ void __launch_bounds__(kRowsThreads) rows_kernel(const RowsArgs a) {
  __shared__ int cnt[3][8];
  __shared__ float mx[8];
  __shared__ int dst[32], lab[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int base = blockIdx.x * a.per_block;
  grid_launch_dependents();
  grid_wait();
  int total = 0, before = 0, bad = 0;
  float big = 0.f;
  auto count = [&](int i, int l, float d) {
    const bool live = l >= 0 && l < a.V;
    total += live;
    before += live && i < base;
    bad |= l >= a.V;
    if (kBwd && live) big = fmaxf(big, fabsf(d));
  };
  const int4* labels4 = reinterpret_cast<const int4*>(a.labels);
  const float4* dloss4 = reinterpret_cast<const float4*>(a.dloss);
#pragma unroll 4
  for (int i = tid; i < a.N / 4; i += kRowsThreads) {
    const int4 l = labels4[i];
    const float4 d = kBwd ? dloss4[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    count(4 * i, l.x, d.x);
    count(4 * i + 1, l.y, d.y);
    count(4 * i + 2, l.z, d.z);
    count(4 * i + 3, l.w, d.w);
  }
  if (tid < (a.N & 3)) {
    const int i = (a.N & ~3) + tid;
    count(i, a.labels[i], kBwd ? a.dloss[i] : 0.f);
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
  const int low = kBwd && total <= kTwice ? (total + 31) / 32 * 32 : 0;
  if (blockIdx.x == 0 && tid == 0) {
    a.info->status = bad ? BB_ERR_BAD_LABEL : BB_OK;
    a.info->rows = total;
    a.info->direct = total == a.N;
    a.info->low = low;
    a.info->dlref = dlref;
  }
  const int chunks = a.D / 8;  // 16-byte pieces of a row
  const bool pack = low || total != a.N;
  for (int r0 = 0; r0 < a.per_block; r0 += 32) {
    if (warp == 0) {
      const int n = r0 + lane < a.per_block ? base + r0 + lane : a.N;
      const int l = n < a.N ? a.labels[n] : -1;
      const bool live = l >= 0 && l < a.V;
      const unsigned m = __ballot_sync(0xffffffffu, live);
      const int p = before + __popc(m & ((1u << lane) - 1));
      before += __popc(m);
      dst[lane] = live ? p : -1;
      lab[lane] = l;
      if (live) {
        a.idx[p] = n;
        a.lab[p] = l;
        if (kBwd) {
          a.rlse[p] = a.lse[n];
          a.dls[p] = a.dloss[n] / dlref;
          if (!low) a.word_n[l] = 0;
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
    }
    __syncthreads();
    for (int r = warp; r < 32; r += 8) {
      const int p = dst[r];
      if (p < 0) continue;
      const uint4* src = reinterpret_cast<const uint4*>(a.h + (size_t)(base + r0 + r) * a.D);
      const uint4* wl = reinterpret_cast<const uint4*>(a.w + (size_t)lab[r] * a.D);
      uint4* out = reinterpret_cast<uint4*>(a.hp + (size_t)p * a.D);
      float s = 0.f;
      for (int c0 = 0; c0 < chunks; c0 += 128) {
        uint4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + 32 * i + lane < chunks) {
            x[i] = src[c0 + 32 * i + lane];
            y[i] = wl[c0 + 32 * i + lane];
          }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + 32 * i + lane < chunks) {
            s = dot8(x[i], y[i], s);
            if (pack) out[c0 + 32 * i + lane] = x[i];
            if (low) out[(size_t)low * chunks + c0 + 32 * i + lane] = x[i];
          }
      }
#pragma unroll
      for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
      if (lane == 0) a.zl[p] = s + (a.bias ? a.bias[lab[r]] : 0.f);
    }
    __syncthreads();
  }
  if (kBwd && !low)
    for (int i = blockIdx.x * kRowsThreads + tid; i < (a.V + 31) / 32;
         i += gridDim.x * kRowsThreads)
      a.word_bits[i] = 0;
  // The packed rows behind the last (of either copy), up to the 64 of dW's last
  // K step, are zero (times the zeros of dz).
  if (pack) {
    const int end = low ? low : (total + kBK - 1) / kBK * kBK;
    uint4* out = reinterpret_cast<uint4*>(a.hp);
    for (size_t c = (size_t)total * chunks + blockIdx.x * kRowsThreads + tid;
         c < (size_t)end * chunks; c += (size_t)gridDim.x * kRowsThreads) {
      out[c] = make_uint4(0, 0, 0, 0);
      if (low) out[(size_t)low * chunks + c] = make_uint4(0, 0, 0, 0);
    }
  }
}

// Forward: merges the (max, sum) pairs of eight rows in a fixed order: 32
// groups take every 32nd pair, then one warp's lanes their 32 results and, past
// the first piece of the vocabulary, the pair of the pieces before; the last
// piece's launch writes the results, the others that pair.
struct MergeArgs {
  const Info* info;
  const float2* part;   // [runs][Np]
  float2* before;       // [Np]
  int runs, Np, first, last;
  const float* zl;
  const int* idx;
  float *loss, *lse;
};

__global__ void __launch_bounds__(256) lse_merge_kernel(const MergeArgs a) {
  __shared__ float2 sh[8][33];
  const int r = threadIdx.x & 7, g = threadIdx.x >> 3;
  grid_launch_dependents();
  grid_wait();
  const int rows = a.info->rows;
  if ((int)blockIdx.x * 8 >= rows) return;
  const int row = blockIdx.x * 8 + r;
  float m = -INFINITY, s = 0.f;
#pragma unroll 4
  for (int i = g; i < a.runs; i += 32) {
    const float2 p = a.part[(size_t)i * a.Np + row];
    const float mm = fmaxf(m, p.x);
    const float ref = mm == -INFINITY ? 0.f : mm;
    s = s * ex2((m - ref) * kLog2e) + p.y * ex2((p.x - ref) * kLog2e);
    m = mm;
  }
  sh[r][g] = make_float2(m, s);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int out = blockIdx.x * 8 + warp;
  if (out >= rows) return;
  const float2 p = sh[warp][lane], b = a.first ? make_float2(-INFINITY, 0.f) : a.before[out];
  m = fmaxf(p.x, b.x);
#pragma unroll
  for (int i = 16; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
  const float ref = m == -INFINITY ? 0.f : m;
  s = p.y * ex2((p.x - ref) * kLog2e);
#pragma unroll
  for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
  s += b.y * ex2((b.x - ref) * kLog2e);
  if (lane == 0) {
    if (a.last) {
      const float l = ref + logf(s);
      const int n = a.idx[out];
      a.lse[n] = l;
      a.loss[n] = l - a.zl[out];
    } else {
      a.before[out] = make_float2(m, s);
    }
  }
}

struct EndArgs {
  const Info* info;
  int N, D, V, Np, splits;
  int word_blocks;      // blocks that finish words of dW, in front of dh's
  const int *labels, *pos;
  const int* lab;       // packed rows: label,
  const float* rest;    //   what bf16 left of its dz
  const int *word_n, *word_rows;
  const float *acc, *side;
  const uint16_t *h, *hp, *w;
  uint16_t *dh, *dw;
};

__device__ __forceinline__ void store8(uint16_t* out, const float (&v)[8], float scale) {
  *reinterpret_cast<uint4*>(out) =
      make_uint4(pack_bf16(v[0] * scale, v[1] * scale), pack_bf16(v[2] * scale, v[3] * scale),
                 pack_bf16(v[4] * scale, v[5] * scale), pack_bf16(v[6] * scale, v[7] * scale));
}

// Eight columns of dW of the word whose list packed row p heads, where the
// list holds all its rows: the sums, and what bf16 left of each label's entry
// times the row's h, in order (the appends were not), rounded once.
__device__ __forceinline__ void finish_word(const EndArgs& a, int p, int c) {
  const uint16_t* h = (a.info->direct ? a.h : a.hp) + c;
  const int v = a.lab[p];
  const float4* src = reinterpret_cast<const float4*>(a.side + (size_t)p * a.D + c);
  const float4 x = src[0], y = src[1];
  // This row's own part, loaded beside the rest of what p leads to: most
  // often it is the only one.
  const float r = a.rest[p];
  const uint4 hr = *reinterpret_cast<const uint4*>(h + (size_t)p * a.D);
  const int n = a.word_n[v], first = a.word_rows[v];
  if (first != p || n > kFix) return;
  float s[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  if (n == 1) {
    fma8(r, hr, s);
  } else {
    int row[kFix];
    word_rows(a.word_rows, a.V, v, n, row);
#pragma unroll
    for (int k = 0; k < kFix; ++k)
      if (k < n)
        fma8(a.rest[row[k]], *reinterpret_cast<const uint4*>(h + (size_t)row[k] * a.D), s);
  }
  store8(a.dw + (size_t)v * a.D + c, s, a.info->dlref);
}

// Backward's end: dh rows rounded from the fp32 sums (0 where there is no
// label), of both parts of dz where it has two; where it has one, with what
// its rounding left of the label's entry times the label's weights.  A block
// takes 256 / kGroups pieces of eight columns; with several parts per sum,
// kGroups threads share a piece's parts and their sums are added in order.
template <int kGroups>
__global__ void __launch_bounds__(256) end_kernel(const EndArgs a) {
  constexpr int kPieces = 256 / kGroups;
  __shared__ float sh[kGroups > 1 ? kGroups : 1][kPieces][kGroups > 1 ? 9 : 1];
  const int chunks = a.D / 8;
  grid_launch_dependents();
  grid_wait();
  if ((int)blockIdx.x < a.word_blocks) {
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (!a.info->low && i / chunks < (size_t)a.info->rows)
      finish_word(a, (int)(i / chunks), (int)(i % chunks) * 8);
    return;
  }
  const int piece = threadIdx.x % kPieces, g = threadIdx.x / kPieces;
  const size_t i = (size_t)(blockIdx.x - a.word_blocks) * kPieces + piece;
  const size_t n = i / chunks;
  const bool live = n < (size_t)a.N;
  const int c = (int)(i % chunks) * 8;
  const int p = live ? a.pos[n] : -1, lab = live ? a.labels[n] : 0, low = a.info->low;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (p >= 0) {
    // The label's part goes to a group that has the fewest others.
    const bool label = !low && g == a.splits % kGroups;
#pragma unroll 4
    for (int s = g; s < a.splits; s += kGroups) {
      const float4* src = reinterpret_cast<const float4*>(a.acc + ((size_t)s * a.Np + p) * a.D + c);
      float4 x = src[0], y = src[1];
      if (low) {
        src = reinterpret_cast<const float4*>(a.acc + ((size_t)s * a.Np + low + p) * a.D + c);
        const float4 lx = src[0], ly = src[1];
        x.x += lx.x; x.y += lx.y; x.z += lx.z; x.w += lx.w;
        y.x += ly.x; y.y += ly.y; y.z += ly.z; y.w += ly.w;
      }
      v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
      v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
    }
    if (label)
      fma8(a.rest[p], *reinterpret_cast<const uint4*>(a.w + (size_t)lab * a.D + c), v);
  }
  if (kGroups > 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sh[g][piece][e] = v[e];
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int q = 1; q < kGroups; ++q)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += sh[q][piece][e];
  }
  if (!live) return;
  store8(a.dh + n * a.D + c, v, p >= 0 ? a.info->dlref : 0.f);
}

// ---- host -------------------------------------------------------------------

struct Plan {
  bool pair;
  int Np, a_rows, pieces, Vp, splits, runs;
  size_t idx, pos, lab, rlse, dls, zl, before, rest, word_bits, word_n, word_rows, side, hp, part,
      dz, dh, dbp, total;  // byte offsets
};

size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }

int make_plan(int N, int D, int V, int pass, Plan* p) {
  if (N <= 0 || D <= 0 || V <= 0 || (pass != 0 && pass != 1)) return BB_ERR_INVALID;
  if (D % 8 != 0 || D < 64 || D > 65536 || N > (1 << 20) || V > (1 << 24))
    return BB_ERR_UNSUPPORTED;
  p->pair = N > kBM;
  const int tm = p->pair ? 2 * kBM : kBM;
  p->Np = (int)up(N, tm);
  // Few rows load a lower box of h; what the MMA reads below it reaches only
  // accumulator rows that nothing uses.
  p->a_rows = N < kBM ? (int)up(N, 8) : kBM;
  // Pieces of equal size whose dz fits kPieceBytes (512 columns at least), or
  // whose pairs of (max, sum) do, one for 128 columns (single CTAs: two each,
  // however many columns).
  size_t fit = pass == 1 ? kPieceBytes / 2 / p->Np / 256 * 256
                         : (kPieceBytes / 8 / p->Np - 4) * 128 / 256 * 256;
  fit = fit < 512 ? 512 : fit;
  if (pass == 0 && !p->pair) fit = V;
  p->pieces = (int)((V + fit - 1) / fit);
  p->Vp = (int)up((V + p->pieces - 1) / p->pieces, 256);
  p->pieces = (V + p->Vp - 1) / p->Vp;
  p->runs = ((p->Vp < V ? p->Vp : V) + 127) / 128;
  if (!p->pair) p->runs = 2 * (p->runs > kSms ? kSms : p->runs);
  // dh has few tiles of a long K when there are few rows: cut K into the
  // fewest parts that keep a tile within a worker's share of the launch (each
  // part writes dh's rows once more, and the last launch reads them).
  const int workers = p->pair ? kSms / 2 : kSms;
  const long long dn = (D + 255) / 256, mt = p->Np / tm;
  const long long nw = (p->Vp + tm - 1) / tm * dn, cw = tile_cost((N + kBK - 1) / kBK);
  const int hks = p->Vp / kBK;
  for (const int s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
    if (s > 1 && hks / s < 4) break;
    const long long nh = mt * dn * s, ch = tile_cost((hks + s - 1) / s);
    p->splits = s;
    if ((nh + workers - 1) / workers * ch <= (nh * ch + nw * cw) / workers) break;
  }
  // The status word is at the workspace's start; the rest begins at the next
  // multiple of 256 bytes behind it (body()), so up to 512 bytes on.
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = up(off + bytes, 256);
    return o;
  };
  p->idx = take((size_t)N * 4);
  p->lab = take((size_t)N * 4);
  p->zl = take((size_t)N * 4);
  p->hp = take((size_t)p->Np * D * 2);
  if (pass == 0) {
    p->before = take((size_t)p->Np * 8);
    // Whole tiles write their runs, past V too.
    p->part = take(((size_t)p->runs + 4) * p->Np * 8);
  } else {
    p->pos = take((size_t)N * 4);
    p->rlse = take((size_t)N * 4);
    p->dls = take((size_t)N * 4);
    if (N > kTwice) {  // (dz is in two parts otherwise)
      p->rest = take((size_t)N * 4);
      p->word_bits = take((size_t)(V + 31) / 32 * 4);
      p->word_n = take((size_t)V * 4);
      p->word_rows = take((size_t)V * kFix * 4);
      if (N <= kSideRows) p->side = take((size_t)N * D * 4);
    }
    p->dz = take((size_t)p->Np * p->Vp * 2);
    p->dh = take((size_t)p->splits * p->Np * D * 4);
    p->dbp = take((size_t)(p->Np / kBM) * p->Vp * 4);
  }
  p->total = off + 512;
  return BB_OK;
}

char* body(void* workspace) {
  return reinterpret_cast<char*>(((uintptr_t)workspace + 511) & ~(uintptr_t)255);
}

template <int kMode, bool kPair>
cudaError_t launch_gemm_as(const CeArgs& a, long long tiles, int sms, const CUtensorMap& h,
                           const CUtensorMap& hp, const CUtensorMap& w, const CUtensorMap& dz,
                           const CUtensorMap& dw, const CUtensorMap& dh, cudaStream_t s) {
  using C = Cfg<kMode, kPair>;
  const cudaError_t e = cudaFuncSetAttribute(ce_gemm_kernel<kMode, kPair>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)C::kSmem);
  if (e != cudaSuccess) return e;
  const int workers = sms / C::kCtas;
  return launch_chained(ce_gemm_kernel<kMode, kPair>,
                        C::kCtas * (unsigned)(tiles < workers ? tiles : workers), C::kThreads,
                        C::kSmem, kPair, s, a, h, hp, w, dz, dw, dh);
}

// `a` by value: the launch's runs of dW are filled in.
template <int kMode>
cudaError_t launch_gemm(const Plan& p, CeArgs a, int sms, const CUtensorMap& h,
                        const CUtensorMap& hp, const CUtensorMap& w, const CUtensorMap& dz,
                        const CUtensorMap& dw, const CUtensorMap& dh, cudaStream_t s) {
  const int tm = p.pair ? 2 * kBM : kBM;
  const int tn = p.pair ? Cfg<kMode, true>::kTN : Cfg<kMode, false>::kTN;
  const long long mt = p.Np / tm, dn = (a.D + tn - 1) / tn, wm = (a.vn + tm - 1) / tm;
  const long long nh = mt * dn * p.splits;
  const long long tiles = kMode == kGrad ? nh + wm * dn : mt * ((a.vn + tn - 1) / tn);
  if (kMode == kGrad && !p.pair)
    // (Up to 128 rows are two K steps of dW at most: one cost.)
    dw_runs((int)wm, (int)dn, (a.D + 63) / 64, nh,
            tile_cost((a.vn + kBK - 1) / kBK / p.splits), tile_cost(kBM / kBK),
            (int)(tiles < sms ? tiles : sms), a.dw_start);
  return p.pair ? launch_gemm_as<kMode, true>(a, tiles, sms, h, hp, w, dz, dw, dh, s)
                : launch_gemm_as<kMode, false>(a, tiles, sms, h, hp, w, dz, dw, dh, s);
}

// Up to 1024 rows one for each of a block's warps; above, as many more as
// keep the blocks, which each read all labels, at 512.
int rows_per_block(int N) { return N <= 1024 ? 8 : 32 * ((N + 16383) / 16384); }

int sm_count() {
  int dev = 0, sms = kSms;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms < kSms ? sms : kSms;  // the plan sizes by a B200's
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
  char* ws = body(workspace);
  cudaStream_t s = (cudaStream_t)stream;
  CUtensorMap tmH, tmHp, tmW;
  if (!encode_bf16_2d(&tmH, h, hidden, N, hidden, 64, p.a_rows) ||
      !encode_bf16_2d(&tmHp, ws + p.hp, hidden, p.Np, hidden, 64, p.a_rows) ||
      !encode_bf16_2d(&tmW, w, hidden, V, hidden, 64, 128))
    return BB_ERR_CUDA;
  RowsArgs r{};
  r.N = N;
  r.per_block = rows_per_block(N);
  r.D = hidden;
  r.V = V;
  r.labels = labels;
  r.h = static_cast<const uint16_t*>(h);
  r.w = static_cast<const uint16_t*>(w);
  r.bias = bias;
  r.zl = reinterpret_cast<float*>(ws + p.zl);
  r.loss = loss;
  r.lse_out = lse;
  r.info = static_cast<Info*>(workspace);
  r.idx = reinterpret_cast<int*>(ws + p.idx);
  r.lab = reinterpret_cast<int*>(ws + p.lab);
  r.hp = reinterpret_cast<uint16_t*>(ws + p.hp);
  if (launch_chained(rows_kernel<false>, (N + r.per_block - 1) / r.per_block, kRowsThreads, 0,
                     false, s, r) != cudaSuccess)
    return BB_ERR_CUDA;
  CeArgs a{};
  a.N = N;
  a.D = hidden;
  a.V = V;
  a.Np = p.Np;
  a.a_bytes = p.a_rows * 2 * kBK;
  a.info = r.info;
  a.bias = bias;
  a.lab = r.lab;
  a.part = reinterpret_cast<float2*>(ws + p.part);
  a.zl = r.zl;
  const int sms = sm_count();
  MergeArgs m{};
  m.info = a.info;
  m.part = a.part;
  m.before = reinterpret_cast<float2*>(ws + p.before);
  m.Np = p.Np;
  m.zl = r.zl;
  m.idx = r.idx;
  m.loss = loss;
  m.lse = lse;
  for (int i = 0; i < p.pieces; ++i) {
    a.v0 = i * p.Vp;
    a.vn = V - a.v0 < p.Vp ? V - a.v0 : p.Vp;
    m.runs = p.pair ? (a.vn + 127) / 128 : p.runs < 2 * sms ? p.runs : 2 * sms;
    m.first = i == 0;
    m.last = i == p.pieces - 1;
    if (launch_gemm<kLse>(p, a, sms, tmH, tmHp, tmW, tmW, tmW, tmW, s) != cudaSuccess ||
        launch_chained(lse_merge_kernel, (N + 7) / 8, 256, 0, false, s, m) != cudaSuccess)
      return BB_ERR_CUDA;
  }
  return BB_OK;
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
  char* ws = body(workspace);
  cudaStream_t s = (cudaStream_t)stream;
  CUtensorMap tmH, tmHp, tmW, tmH64, tmHp64, tmW64, tmDz32, tmDz64, tmDw, tmDh;
  if (!encode_bf16_2d(&tmH, h, hidden, N, hidden, 64, p.a_rows) ||
      !encode_bf16_2d(&tmHp, ws + p.hp, hidden, p.Np, hidden, 64, p.a_rows) ||
      !encode_bf16_2d(&tmW, w, hidden, V, hidden, 64, 128) ||
      !encode_bf16_2d(&tmH64, h, hidden, N, hidden, 64, 64) ||
      !encode_bf16_2d(&tmHp64, ws + p.hp, hidden, p.Np, hidden, 64, 64) ||
      !encode_bf16_2d(&tmW64, w, hidden, V, hidden, 64, 64) ||
      !encode_bf16_2d(&tmDz32, ws + p.dz, 64, (uint64_t)p.Vp / 64 * p.Np, 64, 64, 32) ||
      !encode_bf16_2d(&tmDz64, ws + p.dz, 64, (uint64_t)p.Vp / 64 * p.Np, 64, 64, 64) ||
      !encode_bf16_2d(&tmDw, dw, hidden, V, hidden, 64, 32) ||
      !encode_f32_2d(&tmDh, ws + p.dh, hidden, (uint64_t)p.splits * p.Np, hidden, 32, 32))
    return BB_ERR_CUDA;
  RowsArgs r{};
  r.N = N;
  r.per_block = rows_per_block(N);
  r.D = hidden;
  r.V = V;
  r.labels = labels;
  r.h = static_cast<const uint16_t*>(h);
  r.w = static_cast<const uint16_t*>(w);
  r.bias = bias;
  r.zl = reinterpret_cast<float*>(ws + p.zl);
  r.lse = lse;
  r.dloss = dloss;
  r.info = static_cast<Info*>(workspace);
  r.idx = reinterpret_cast<int*>(ws + p.idx);
  r.pos = reinterpret_cast<int*>(ws + p.pos);
  r.lab = reinterpret_cast<int*>(ws + p.lab);
  r.rlse = reinterpret_cast<float*>(ws + p.rlse);
  r.dls = reinterpret_cast<float*>(ws + p.dls);
  r.hp = reinterpret_cast<uint16_t*>(ws + p.hp);
  r.word_n = reinterpret_cast<int*>(ws + p.word_n);
  r.word_bits = reinterpret_cast<unsigned*>(ws + p.word_bits);
  if (launch_chained(rows_kernel<true>, (N + r.per_block - 1) / r.per_block, kRowsThreads, 0,
                     false, s, r) != cudaSuccess)
    return BB_ERR_CUDA;
  CeArgs a{};
  a.N = N;
  a.D = hidden;
  a.V = V;
  a.Np = p.Np;
  a.Vp = p.Vp;
  a.splits = p.splits;
  a.a_bytes = p.a_rows * 2 * kBK;
  a.info = r.info;
  a.bias = bias;
  a.lab = r.lab;
  a.rlse = r.rlse;
  a.dls = r.dls;
  a.zl = r.zl;
  a.dz = reinterpret_cast<uint16_t*>(ws + p.dz);
  a.rest = reinterpret_cast<float*>(ws + p.rest);
  a.word_n = r.word_n;
  a.word_rows = reinterpret_cast<int*>(ws + p.word_rows);
  a.word_bits = r.word_bits;
  a.side = N <= kSideRows ? reinterpret_cast<float*>(ws + p.side) : nullptr;
  a.h = r.h;
  a.hp = r.hp;
  a.dbp = dbias ? reinterpret_cast<float*>(ws + p.dbp) : nullptr;
  a.dbias = dbias;
  const int sms = sm_count();
  for (int i = 0; i < p.pieces; ++i) {
    a.v0 = i * p.Vp;
    a.vn = V - a.v0 < p.Vp ? V - a.v0 : p.Vp;
    a.add = i > 0;
    if (launch_gemm<kDz>(p, a, sms, tmH, tmHp, tmW, tmDz32, tmW, tmW, s) != cudaSuccess ||
        launch_gemm<kGrad>(p, a, sms, tmH64, tmHp64, tmW64, tmDz64, tmDw, tmDh, s) != cudaSuccess)
      return BB_ERR_CUDA;
  }
  const size_t pieces = (size_t)N * (hidden / 8);
  const int groups = p.splits > 4 ? 8 : 1;
  EndArgs e{};
  e.info = a.info;
  e.N = N;
  e.D = hidden;
  e.V = V;
  e.Np = p.Np;
  e.splits = p.splits;
  e.word_blocks = N > kTwice && a.side ? (int)((pieces + 255) / 256) : 0;
  e.labels = labels;
  e.pos = r.pos;
  e.lab = r.lab;
  e.rest = a.rest;
  e.word_n = a.word_n;
  e.word_rows = a.word_rows;
  e.acc = reinterpret_cast<const float*>(ws + p.dh);
  e.side = a.side;
  e.h = r.h;
  e.hp = r.hp;
  e.w = r.w;
  e.dh = static_cast<uint16_t*>(dh);
  e.dw = static_cast<uint16_t*>(dw);
  if (launch_chained(groups > 1 ? end_kernel<8> : end_kernel<1>,
                     e.word_blocks + (unsigned)((pieces * groups + 255) / 256), 256, 0, false, s,
                     e) != cudaSuccess)
    return BB_ERR_CUDA;
  return BB_OK;
}

}  // extern "C"
