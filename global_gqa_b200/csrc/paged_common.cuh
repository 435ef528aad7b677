// What the paged-cache kernels share.
//
// A paged cache of one layer is k_pages, v_pages [n_pages, Hkv, P, D] bf16: one
// (page, kv head) is P consecutive rows.  Logical page j of sequence b is
// block_table[b, j]; its token t sits in row t % P of logical page t / P.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "g3_internal.h"
#include "sm100_ptx.cuh"

namespace g3 {

// Lets the next kernel in the stream, when it was launched as a programmatic
// dependent, take its place on the SMs early; it still waits for this one's end.
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ int cluster_size() {
  int n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
// The cluster's barrier in two halves: what a thread wrote before its arrival is
// visible to those that have waited.  A block that only arrives may end.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The address of a shared variable in block `rank` of the cluster, and a store to one.
__device__ __forceinline__ uint32_t cluster_address(const void* p, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void cluster_store(uint32_t address, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(address), "r"(v) : "memory");
}

// griddep_wait(), with a token for reads that must not be moved in front of it.
__device__ __forceinline__ uint32_t griddep_wait_token() {
  uint32_t token;
  asm volatile("griddepcontrol.wait;\n\tmov.u32 %0, 0;" : "=r"(token)::"memory");
  return token;
}
// A 16-byte read of data that no one writes during the kernel: free to move, but not before the wait that gave the
// token (a compiler may take __ldg's address to be readable from the kernel's start).
__device__ __forceinline__ uint4 ldg_after(const void* p, uint32_t token) {
  uint4 v;
  asm("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p), "r"(token));
  return v;
}
// The same of data that the block reads once, in the order of the program.
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// The prefix sums below of n <= 32 * PER terms, by every warp for itself, all writing the same values: no barrier.
template <int PER, class F>
__device__ __forceinline__ void warp_prefix(int n, int* pref, F&& count) {
  const int lane = threadIdx.x & 31, first = PER * lane;
  int v[PER], sum = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) v[k] = first + k < n ? count(first + k) : 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) v[k] = sum += v[k];
  int inc = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += x;
  }
#pragma unroll
  for (int k = 0; k < PER; ++k)
    if (first + k < n) pref[first + k + 1] = inc - sum + v[k];
  if (lane == 0) pref[0] = 0;
  __syncwarp();
}

// Inclusive prefix sums of count(b), b < n, into pref[1 .. n], pref[0] = 0, by
// the whole block (a multiple of 32 threads; `warp_sums` holds one int per
// warp).  Every block of a grid repeats it: some microseconds at the largest n, for
// one launch less and no order between blocks.
template <class F>
__device__ __forceinline__ void block_prefix(int n, int* pref, int* warp_sums, F&& count) {
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5;
  if (n <= 32) return warp_prefix<1>(n, pref, count);
  if (n <= 128) return warp_prefix<4>(n, pref, count);  // 0.6 us less than below for 64 sequences
  // The terms first, in coalesced reads that do not wait for one another; then each thread sums a run of its own (of odd
  // length: the threads' runs begin in different banks).  8192 sequences: 12 us, 90 with the reads in the runs.
#pragma unroll 8
  for (int i = tid; i < n; i += threads) pref[i + 1] = count(i);
  __syncthreads();
  const int per = ((n + threads - 1) / threads) | 1;
  const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
  int sum = 0;
  for (int i = i0; i < i1; ++i) {
    sum += pref[i + 1];
    pref[i + 1] = sum;
  }
  int inc = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += v;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  const int before = inc - sum + __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[lane] : 0);
  for (int i = i0; i < i1; ++i) pref[i + 1] += before;
  if (tid == 0) pref[0] = 0;
  __syncthreads();
}

// The b with pref[b] * scale <= x < pref[b + 1] * scale; 0 <= x < pref[n] * scale < 2^30.
__device__ __forceinline__ int find_row(const int* pref, int n, int x, int scale) {
  int lo = 0, hi = n;  // pref[lo] * scale <= x < pref[hi] * scale
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid] * scale <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

}  // namespace g3
