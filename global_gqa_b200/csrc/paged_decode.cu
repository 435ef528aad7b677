// Attention of one new token per sequence over a paged KV cache.
//
//   paged_decode : the visible tokens of all (sequence, kv head) pairs, in units
//                  of 16, form one line that is cut into equal shares, one per
//                  block, whatever the lengths; a share that holds a whole pair
//                  writes its output, one that holds a part writes a partial
//                  softmax (max, sum, unnormalised output) in fp32.
//   paged_combine: merges the partials of the pairs that were cut, in the order
//                  of their blocks (the same result on every run).
//
// Visible: on a global layer all L cached tokens, on a local one the last W of
// them (Gemma 3 Technical Report, sections 1 and 2), or the tokens of the listed
// pages.
//
// HBM-bound: 4 D bytes per visible token and kv head, read once and shared by
// the group's G <= 8 query heads.  Both products run on mma.m16n8k16 with the
// heads as its 8 columns: S^T = K Q^T and O^T = V^T P^T.  K and V go straight
// from global memory into the A fragments: the order of the features inside
// q . k is free, so a lane's 16-byte pieces of a K row serve as they come (Q is
// laid out to match); for V a lane reads the same 8 features of four tokens and
// interleaves them in pairs.  No shared memory is touched in the loop.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "func_attr.cuh"
#include "g3_internal.h"
#include "paged_common.cuh"
#include "sm100_ptx.cuh"

namespace g3 {

constexpr int kPagedThreads = 128;
constexpr int kPagedWarps = kPagedThreads / 32;
constexpr int kUnit = 16;  // tokens of one warp step

__device__ __forceinline__ void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of 16-bit values held as an mma fragment.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint4 ldg_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t piece(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Number of units of one kv head of sequence b (0: nothing to attend to).
__device__ __forceinline__ int units_of(const PagedDecodeParams& p, int b, bool report) {
  const int L = p.seq_lens[b];
  if (L < 0 || L > ((long long)p.max_pages << p.page_shift)) {
    if (report) record_error(p.status, kErrInvalid, 340);
    return 0;
  }
  if (p.pages != nullptr) {
    const int np = (L + (1 << p.page_shift) - 1) >> p.page_shift;
    return min(np, p.n_select) << (p.page_shift - 4);
  }
  const int lo = p.kind == 0 ? max(0, L - p.window) : 0;
  return (L + kUnit - 1) / kUnit - lo / kUnit;
}
// How many blocks share the line of `total` units: none with less than one unit per warp.
__device__ __forceinline__ int active_blocks(long long total, int blocks) {
  return (int)max(1LL, min((long long)blocks, total / kPagedWarps));
}

template <int D>
__global__ void __launch_bounds__(kPagedThreads, D == 64 ? 6 : D == 128 ? 3 : 2) paged_decode_kernel(PagedDecodeParams p) {
  constexpr int KP = D / 32;  // 16-byte pieces of a K row per lane
  constexpr int VP = D / 64;  // 16-byte pieces of a V row per lane
  extern __shared__ int pref[];  // [B + 1] units of one head before each sequence
  __shared__ int warp_sums[kPagedWarps];
  __shared__ float s_m[kPagedWarps][8], s_l[kPagedWarps][8];
  __shared__ __align__(16) float s_o[kPagedWarps][8][D];
  griddep_wait();
  griddep_launch();
  block_prefix(p.B, pref, warp_sums, [&](int b) { return units_of(p, b, blockIdx.x == 0); });
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= p.B; b += kPagedThreads) p.pref[b] = pref[b];
  const long long total = (long long)pref[p.B] * p.Hkv;
  const int blocks = active_blocks(total, gridDim.x);
  if ((int)blockIdx.x >= blocks) return;
  const long long range0 = total * blockIdx.x / blocks, range1 = total * (blockIdx.x + 1) / blocks;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = lane >> 2, c = lane & 3;
  const int P = 1 << p.page_shift;

  for (long long g = range0; g < range1;) {
    const int b = find_row(pref, p.B, g, p.Hkv);
    const int n = pref[b + 1] - pref[b];
    const long long rel = g - (long long)pref[b] * p.Hkv;
    const int h = (int)(rel / n), i0 = (int)(rel % n);
    const int i1 = (int)min((long long)n, i0 + (range1 - g));
    const int L = p.seq_lens[b];
    const int lo = p.pages == nullptr && p.kind == 0 ? max(0, L - p.window) : 0;
    const int32_t* table = p.block_table + (size_t)b * p.max_pages;
    const int32_t* list = p.pages == nullptr ? nullptr : p.pages + ((size_t)b * p.Hkv + h) * p.n_select;

    // Q as the B fragments of S^T = K Q^T: column `row` is a head, features in the order of K's pieces.
    uint4 q[KP];
#pragma unroll
    for (int k = 0; k < KP; ++k)
      q[k] = row < p.G ? __ldg(reinterpret_cast<const uint4*>(p.q_hat + ((size_t)b * p.Hq + h * p.G + row) * D) + c + 4 * k)
                       : make_uint4(0u, 0u, 0u, 0u);

    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2c, 2c + 1; l: this lane's tokens only
    float o[VP][4][4];
#pragma unroll
    for (int j = 0; j < VP; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][t][e] = 0.f;

    // First token and cache row of unit i, or row -1 where its page is not to be read.
    auto locate = [&](int i, int& tok) -> long long {
      int j;
      if (list == nullptr) {
        tok = (lo / kUnit + i) * kUnit;
        j = tok >> p.page_shift;
      } else {
        const int e = i >> (p.page_shift - 4);
        j = list[e];
        // -1 pads a list.  Otherwise a page of the sequence, above the one before it.
        const bool ok = j >= 0 && ((long long)j << p.page_shift) < L && (e == 0 || list[e - 1] < j);
        if (!ok) {
          if (j != -1 && lane == 0) record_error(p.status, kErrInvalid, 342);
          tok = L;
          return -1;
        }
        tok = (j << p.page_shift) + (i & ((P >> 4) - 1)) * kUnit;
        if (tok >= L) return -1;
      }
      const int page = table[j];
      if (page < 0 || page >= p.n_pages) {
        if (lane == 0) record_error(p.status, kErrInvalid, 341);
        return -1;
      }
      return (((long long)page * p.Hkv + h) << p.page_shift) + (tok & (P - 1));
    };

    const uint4* kbase = reinterpret_cast<const uint4*>(p.k_pages);
    const uint4* vbase = reinterpret_cast<const uint4*>(p.v_pages);
    uint4 kx[2][KP];
    auto load_k = [&](long long r) {
      if (r >= 0) {
#pragma unroll
        for (int k = 0; k < KP; ++k) {
          kx[0][k] = ldg_stream(kbase + (r + row) * (D / 8) + c + 4 * k);
          kx[1][k] = ldg_stream(kbase + (r + row + 8) * (D / 8) + c + 4 * k);
        }
      }
    };

    int i = i0 + warp, tok = 0, tok_next = 0;
    long long r = -1, r_next = -1;
    if (i < i1) {
      r = locate(i, tok);
      load_k(r);
      if (i + kPagedWarps < i1) r_next = locate(i + kPagedWarps, tok_next);
    }
    for (; i < i1; i += kPagedWarps) {
      if (r >= 0) {
        // V: tokens 2c, 2c + 1, 2c + 8, 2c + 9; zero where not visible (the rows there may hold anything).
        uint4 vx[4][VP];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int vt = 2 * c + (t & 1) + (t >> 1) * 8;
          const bool seen = tok + vt >= lo && tok + vt < L;
#pragma unroll
          for (int j = 0; j < VP; ++j)
            vx[t][j] = seen ? ldg_stream(vbase + (r + vt) * (D / 8) + row + 8 * j) : make_uint4(0u, 0u, 0u, 0u);
        }
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KP; ++k) {
          mma_bf16(s, kx[0][k].x, kx[1][k].x, kx[0][k].y, kx[1][k].y, q[k].x, q[k].y);
          mma_bf16(s, kx[0][k].z, kx[1][k].z, kx[0][k].w, kx[1][k].w, q[k].z, q[k].w);
        }
        // K's registers are free: the next unit's K is on its way during the softmax and P V.
        load_k(r_next);
        const bool seen_a = tok + row >= lo && tok + row < L, seen_b = tok + row + 8 >= lo && tok + row + 8 < L;
        s[0] = seen_a ? s[0] * p.scale_log2 : -INFINITY;
        s[1] = seen_a ? s[1] * p.scale_log2 : -INFINITY;
        s[2] = seen_b ? s[2] * p.scale_log2 : -INFINITY;
        s[3] = seen_b ? s[3] * p.scale_log2 : -INFINITY;
        float n0 = fmaxf(s[0], s[2]), n1 = fmaxf(s[1], s[3]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, off));
          n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, off));
        }
        n0 = fmaxf(n0, m0);
        n1 = fmaxf(n1, m1);
        // With nothing above -inf so far every exponent is taken against 0 and gives 0.
        const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;
        if (__any_sync(0xffffffffu, n0 != m0 || n1 != m1)) {
          const float a0 = ex2_approx(m0 - b0), a1 = ex2_approx(m1 - b1);
          l0 *= a0;
          l1 *= a1;
#pragma unroll
          for (int j = 0; j < VP; ++j)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              o[j][t][0] *= a0;
              o[j][t][1] *= a1;
              o[j][t][2] *= a0;
              o[j][t][3] *= a1;
            }
          m0 = n0;
          m1 = n1;
        }
        const float p0 = ex2_approx(s[0] - b0), p1 = ex2_approx(s[1] - b1);
        const float p2 = ex2_approx(s[2] - b0), p3 = ex2_approx(s[3] - b1);
        l0 += p0 + p2;
        l1 += p1 + p3;
        // P in bf16 for the product with V, as in prefill: relative 2^-9 per weight, independent over the
        // tokens, beside the output's own rounding of 2^-9; the sum l keeps fp32.
        const uint32_t pb0 = transpose8(pack_bf16x2(p0, p1)), pb1 = transpose8(pack_bf16x2(p2, p3));
#pragma unroll
        for (int j = 0; j < VP; ++j)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t u0 = piece(vx[0][j], t), u1 = piece(vx[1][j], t), u2 = piece(vx[2][j], t), u3 = piece(vx[3][j], t);
            mma_bf16(o[j][t], __byte_perm(u0, u1, 0x5410), __byte_perm(u0, u1, 0x7632), __byte_perm(u2, u3, 0x5410),
                     __byte_perm(u2, u3, 0x7632), pb0, pb1);
          }
      } else {
        load_k(r_next);
      }
      r = r_next;
      tok = tok_next;
      r_next = i + 2 * kPagedWarps < i1 ? locate(i + 2 * kPagedWarps, tok_next) : -1;
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }

    // Merge the warps' parts.
    if (row == 0) {
      s_m[warp][2 * c] = m0;
      s_m[warp][2 * c + 1] = m1;
      s_l[warp][2 * c] = l0;
      s_l[warp][2 * c + 1] = l1;
    }
#pragma unroll
    for (int j = 0; j < VP; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int f = row * 8 + 64 * j + 2 * t;
        if (2 * c < p.G) *reinterpret_cast<float2*>(&s_o[warp][2 * c][f]) = make_float2(o[j][t][0], o[j][t][2]);
        if (2 * c + 1 < p.G) *reinterpret_cast<float2*>(&s_o[warp][2 * c + 1][f]) = make_float2(o[j][t][1], o[j][t][3]);
      }
    __syncthreads();
    const bool whole = i0 == 0 && i1 == n;
    const size_t slot = 2 * (size_t)blockIdx.x + (g == range0 ? 0 : 1);
    for (int idx = tid; idx < p.G * (D / 2); idx += kPagedThreads) {
      const int gh = idx / (D / 2), f = idx % (D / 2) * 2;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kPagedWarps; ++w) M = fmaxf(M, s_m[w][gh]);
      const float base = M == -INFINITY ? 0.f : M;
      float acc0 = 0.f, acc1 = 0.f, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kPagedWarps; ++w) {
        const float a = ex2_approx(s_m[w][gh] - base);
        const float2 v = *reinterpret_cast<const float2*>(&s_o[w][gh][f]);
        acc0 = fmaf(a, v.x, acc0);
        acc1 = fmaf(a, v.y, acc1);
        sum = fmaf(a, s_l[w][gh], sum);
      }
      const size_t oh = (size_t)b * p.Hq + h * p.G + gh;
      if (whole) {
        const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;  // nothing visible: a zero row
        *reinterpret_cast<uint32_t*>(p.out + oh * D + f) = pack_bf16x2(acc0 * inv, acc1 * inv);
        if (f == 0 && p.lse != nullptr) p.lse[oh] = sum > 0.f || sum != sum ? (M + log2f(sum)) * 0.6931471805599453f : -INFINITY;
      } else {
        *reinterpret_cast<float2*>(p.part_o + (slot * 8 + gh) * D + f) = make_float2(acc0, acc1);
        if (f == 0) *reinterpret_cast<float2*>(p.part_ml + (slot * 8 + gh) * 2) = make_float2(M, sum);
      }
    }
    __syncthreads();
    g += i1 - i0;
  }
}

// One block per (query head, sequence): groups of D / 4 threads take every
// n-th partial, 4 features per thread.
constexpr int kPagedCombineThreads = 256;

template <int D>
__global__ void __launch_bounds__(kPagedCombineThreads) paged_combine_kernel(PagedDecodeParams p) {
  constexpr int TPG = D / 4, NG = kPagedCombineThreads / TPG;
  __shared__ float s_m[NG], s_l[NG];
  __shared__ __align__(16) float s_o[NG][D];
  griddep_wait();
  griddep_launch();
  const int hq = blockIdx.x, b = blockIdx.y, h = hq / p.G, gh = hq % p.G;
  const int tid = threadIdx.x, grp = tid / TPG, f = tid % TPG * 4;
  const int n = p.pref[b + 1] - p.pref[b];
  const size_t oh = (size_t)b * p.Hq + hq;
  if (n == 0) {
    if (grp == 0) *reinterpret_cast<uint2*>(p.out + oh * D + f) = make_uint2(0u, 0u);
    if (tid == 0 && p.lse != nullptr) p.lse[oh] = -INFINITY;
    return;
  }
  const long long total = (long long)p.pref[p.B] * p.Hkv;
  const int blocks = active_blocks(total, p.n_blocks);
  const long long g0 = (long long)p.pref[b] * p.Hkv + (long long)h * n, g1 = g0 + n;
  // The block that holds unit x: the last w with total * w / blocks <= x.
  auto owner = [&](long long x) { return (int)(((x + 1) * blocks - 1) / total); };
  const int w0 = owner(g0), w1 = owner(g1 - 1);
  if (w0 == w1) return;  // written whole
  float M = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int w = w0 + grp; w <= w1; w += NG) {
    // A block's share starts inside the pair for all but the first, whose part may lie behind another's.
    const size_t slot = 2 * (size_t)w + (w == w0 && total * w / blocks != g0 ? 1 : 0);
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (slot * 8 + gh) * 2);
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + (slot * 8 + gh) * D + f);
    const float mn = fmaxf(M, ml.x), base = mn == -INFINITY ? 0.f : mn;
    const float a = ex2_approx(M - base), e = ex2_approx(ml.x - base);
    sum = sum * a + ml.y * e;
    acc[0] = acc[0] * a + v.x * e;
    acc[1] = acc[1] * a + v.y * e;
    acc[2] = acc[2] * a + v.z * e;
    acc[3] = acc[3] * a + v.w * e;
    M = mn;
  }
  if (f == 0) {
    s_m[grp] = M;
    s_l[grp] = sum;
  }
  *reinterpret_cast<float4*>(&s_o[grp][f]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  if (grp != 0) return;
  M = s_m[0];
#pragma unroll
  for (int k = 1; k < NG; ++k) M = fmaxf(M, s_m[k]);
  const float base = M == -INFINITY ? 0.f : M;
  sum = 0.f;
  acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    const float a = ex2_approx(s_m[k] - base);
    const float4 v = *reinterpret_cast<const float4*>(&s_o[k][f]);
    sum = fmaf(a, s_l[k], sum);
    acc[0] = fmaf(a, v.x, acc[0]);
    acc[1] = fmaf(a, v.y, acc[1]);
    acc[2] = fmaf(a, v.z, acc[2]);
    acc[3] = fmaf(a, v.w, acc[3]);
  }
  const bool any = sum > 0.f || sum != sum;
  const float inv = any ? 1.f / sum : 0.f;
  *reinterpret_cast<uint2*>(p.out + oh * D + f) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  if (f == 0 && p.lse != nullptr) p.lse[oh] = any ? (M + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

template <int D>
static cudaError_t launch_paged_d(const PagedDecodeParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ensure_dynamic_smem(paged_decode_kernel<D>, (kPagedMaxSeqs + 1) * (int)sizeof(int), done);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_decode_kernel<D>, dim3(p.n_blocks), dim3(kPagedThreads), (p.B + 1) * sizeof(int), st, p);
}

int paged_decode_blocks(int D) { return 148 * (D == 64 ? 6 : D == 128 ? 3 : 2); }

cudaError_t launch_paged_decode(const PagedDecodeParams& p, int D, cudaStream_t st) {
  switch (D) {
    case 64: return launch_paged_d<64>(p, st);
    case 128: return launch_paged_d<128>(p, st);
    case 256: return launch_paged_d<256>(p, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_paged_combine(const PagedDecodeParams& p, int D, cudaStream_t st) {
  const dim3 grid(p.Hq, p.B), block(kPagedCombineThreads);
  switch (D) {
    case 64: return launch_dependent(paged_combine_kernel<64>, grid, block, 0, st, p);
    case 128: return launch_dependent(paged_combine_kernel<128>, grid, block, 0, st, p);
    case 256: return launch_dependent(paged_combine_kernel<256>, grid, block, 0, st, p);
  }
  return cudaErrorInvalidValue;
}

}  // namespace g3
