// Shared by the operators around the attention: argument checks, chained
// launches, and the inline-PTX wrappers that only they use (CTA pairs,
// instructions issued as uniform code, asynchronous copies).
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace bb {

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Dropout rate in [0, 1), rounded to 1/256: the byte threshold and 1 / keep
// probability.  False for a rate outside [0, 1) or one that rounds to 1
// (it would drop everything: infinite scale).
inline bool resolve_dropout(float rate, uint32_t* thr, float* scale) {
  if (!(rate >= 0.f && rate < 1.f)) return false;
  const int t = (int)((double)rate * 256.0 + 0.5);
  if (t > 255) return false;
  *thr = (uint32_t)t;
  *scale = (float)(256.0 / (256.0 - t));
  return true;
}

// encode_bf16_2d's fp32 counterpart (row stride a multiple of 4, box_inner = 32).
bool encode_f32_2d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows,
                   uint64_t row_stride, uint32_t box_inner, uint32_t box_rows);

// A launch whose kernel waits for the one in front on the device (grid_wait),
// so that its setup runs under that one's end; pair: in clusters of two.
template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                           bool pair, cudaStream_t s, Args... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = pair ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

namespace sm100 {

// ---- waits ------------------------------------------------------------------

// mbar_wait by a whole converged warp, with one answer for all its lanes
// (they may time out at different polls), so that they leave together.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity,
                                               volatile int* abort_flag, int* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status));
}

// ---- stores and copies --------------------------------------------------------

// 2-D tiled fp32 addition of one box from shared memory to global memory.
__device__ __forceinline__ void tma_reduce_add_2d(const CUtensorMap* map, const void* smem_src,
                                                  int x, int y) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], "
      "[%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(smem_src)), "r"(x), "r"(y)
      : "memory");
}
// The shared-memory sources of all committed bulk stores but the last group
// have been read.
__device__ __forceinline__ void bulk_wait_read_but_one() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}
// 16 bytes from global to shared memory without registers, in groups that are
// waited for in order.
__device__ __forceinline__ void cp_async16(void* smem_dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem_dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// All but the last `kLeft` groups of this thread have arrived.
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// 32 bytes from and to global memory, 32-byte aligned: one whole sector.
__device__ __forceinline__ void ld_global_32(const void* p, uint32_t (&v)[8]) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                 "=r"(v[6]), "=r"(v[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st_global_32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// ---- launches that begin before the one in front of them ends --------------

// Lets the next launch of the stream begin its setup.
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// Waits until the launches in front have completed and their writes are
// visible, to the async proxy (TMA) too.
__device__ __forceinline__ void grid_wait() {
  asm volatile("griddepcontrol.wait;\n\tfence.proxy.async;" ::: "memory");
}

// ---- CTA pairs (cta_group::2) ----------------------------------------------
//
// Two CTAs of a cluster share one MMA: each holds 128 of A's rows and half of
// B's columns in its own shared memory (at the same offsets) and receives its
// rows of D in its own tensor memory.  The CTA of rank 0 issues.

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// All threads of both CTAs; orders shared-memory writes before it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
// Address of `p` in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// Arrive on a barrier of the cluster by its mapped address.  Relaxed, as
// mbar_arrive is: it hands over tensor memory, ordered by the tcgen05 fences;
// a release would wait for the thread's global stores in flight.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr)
               : "memory");
}
// 2-D tiled load into this CTA's shared memory that signals a barrier of the
// pair, issued by a whole converged warp (its elected lane carries it out), and
// the barrier's expectation: as uniform code a load takes about half the
// clocks to issue that it takes in a branch of one lane.  `bar` is a mapped
// address in a pair, this CTA's own otherwise.
__device__ __forceinline__ void mbar_expect_tx_warp(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d_warp(bool pair, uint32_t smem_dst,
                                                 const CUtensorMap* map, uint32_t bar, int x,
                                                 int y) {
  if (pair)
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes."
        "cta_group::2 [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
// MMAs and commits issued by a whole converged warp, whose elected lane
// (always the same one) carries them out.  In a branch that one lane takes an
// MMA takes 80 clocks to issue; as uniform code 39 (128 x 16 x 16) to the 128
// that a 128 x 256 x 16 product runs.
__device__ __forceinline__ void mma_ss_warp(bool pair, uint32_t d_tmem, uint64_t a_desc,
                                            uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  if (pair)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive once on `bar` (in a pair: at the same offset in both CTAs) when every
// MMA the elected lane issued so far completes.
__device__ __forceinline__ void mma_commit_warp(bool pair, uint64_t* bar) {
  if (pair)
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster."
        "multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 "
        "[%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

}  // namespace sm100
}  // namespace bb
