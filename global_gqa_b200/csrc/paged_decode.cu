// Attention of one new token per sequence over a paged KV cache.
//
//   paged_decode : the visible tokens of all (sequence, kv head) pairs, in units
//                  of 16, form one line that is cut into equal shares, one per
//                  block, whatever the lengths; a share that holds a whole pair
//                  writes its output, one that holds a part writes a partial
//                  softmax (max, sum, unnormalised output) in fp32.  With many
//                  blocks per pair the blocks are dealt to the pairs instead, in
//                  proportion to their lengths, and none works on two of them.
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
__device__ __forceinline__ uint32_t piece(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// The bits of a bf16 number below x >= 0 (0 for 0) by at least 2^-16 of x's power of two and at most 2^-7 + 2^-16 of it:
// the rest, which the subtraction gives exactly, is positive wherever x is (above some 2^-110, where bf16 ends), and
// rounded to bf16 within 2^-16 of x.  Both parts of a weight are then positive, and an infinite V times them is that
// infinity; with x rounded to nearest the rest can be 0 or negative, which made a NaN of it.
__device__ __forceinline__ uint32_t high_part(float x) {
  return (uint32_t)__viaddmax_s32(__float_as_int(x), -0x80, 0) & 0xffff0000u;
}

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
// The line of `total` < 2^30 units cut into shares of q or q + 1 for `blocks`
// blocks: none with less than one unit per warp.
struct Shares {
  int blocks, q, r;  // the first r shares have q + 1 units
  __device__ Shares(int total, int most) {
    blocks = max(1, min(most, total / kPagedWarps));
    q = total / blocks;
    r = total - q * blocks;
  }
  __device__ int begin(int w) const { return w * q + min(w, r); }
  __device__ int owner(int x) const { return x < r * (q + 1) ? x / (q + 1) : r + (x - r * (q + 1)) / q; }
};

// Merges N partial softmaxes, `stride`s apart: max and sum at ml, 4 features' sums at o.
template <int N>
__device__ __forceinline__ void merge_groups(const float (*ml)[2], int ml_stride, const float* o, int o_stride, float& M, float& sum,
                                             float4& acc) {
  M = -INFINITY;
#pragma unroll
  for (int k = 0; k < N; ++k) M = fmaxf(M, ml[k * ml_stride][0]);
  const float base = M == -INFINITY ? 0.f : M;
  sum = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float a = ex2_approx(ml[k * ml_stride][0] - base);
    const float4 v = *reinterpret_cast<const float4*>(o + k * o_stride);
    sum = fmaf(a, ml[k * ml_stride][1], sum);
    acc.x = fmaf(a, v.x, acc.x);
    acc.y = fmaf(a, v.y, acc.y);
    acc.z = fmaf(a, v.z, acc.z);
    acc.w = fmaf(a, v.w, acc.w);
  }
}

// Four features of a finished row, and its lse at f = 0; nothing visible gives a zero row.
template <int D>
__device__ __forceinline__ void store_row(const PagedDecodeParams& p, size_t oh, int f, float M, float sum, const float4& acc) {
  const bool any = sum > 0.f || sum != sum;
  const float inv = any ? 1.f / sum : 0.f;
  *reinterpret_cast<uint2*>(p.out + oh * D + f) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (f == 0 && p.lse != nullptr) p.lse[oh] = any ? (M + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

// Bytes of shared memory for the queries.
constexpr int paged_shared_q(int D) { return D == 256 ? kPagedWarps * (D / 32) * 32 * 16 : 0; }

template <int D>
__global__ void __launch_bounds__(kPagedThreads, D == 64 ? 4 : D == 128 ? 3 : 2) paged_decode_kernel(PagedDecodeParams p) {
  constexpr int KP = D / 32;  // 16-byte pieces of a K row per lane
  constexpr int VP = D / 64;  // 16-byte pieces of a V row per lane
  // Queries (head dim 256), then [B + 1] units of one head before each sequence and, where blocks are dealt, [B + 1] blocks.
  extern __shared__ uint4 paged_smem[];
  int* const pref = reinterpret_cast<int*>(paged_smem) + paged_shared_q(D) / sizeof(int);
  __shared__ int warp_sums[kPagedWarps];
  __shared__ float s_ml[kPagedWarps][8][2];
  __shared__ __align__(16) float s_o[kPagedWarps][8][D];
  griddep_wait();
  block_prefix(p.B, pref, warp_sums, [&](int b) { return units_of(p, b, blockIdx.x == 0); });
  // Sequences that see nothing.
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (pref[b + 1] != pref[b]) continue;
    for (int i = threadIdx.x; i < p.Hq * (D / 4); i += kPagedThreads)
      store_row<D>(p, (size_t)b * p.Hq + i / (D / 4), i % (D / 4) * 4, -INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f));
    for (int h = threadIdx.x; p.deal && h < p.Hkv; h += kPagedThreads) p.cuts[b * p.Hkv + h] = make_int4(-1, 0, 0, 0);
  }
  const int total = pref[p.B] * p.Hkv;  // below 2^30: checked on the host for the widest table
  const Shares sh(total, gridDim.x);
  int range0 = 0, range1 = 0, dealt = 1, part = 0;  // units of this block; of its pair, where blocks are dealt
  int* deal = pref + p.B + 1;
  if (p.deal) {
    // Few pairs: each gets blocks of its own, one and its share of the rest, none with less than one unit per warp.
    // (Rounding in fp32 cannot raise the sum of the whole parts by one.)
    const float rate = total > 0 ? (float)((int)gridDim.x - p.B * p.Hkv) / (float)total : 0.f;
    block_prefix(p.B, deal, warp_sums, [&](int b) {
      const int n = pref[b + 1] - pref[b];
      return n == 0 ? 0 : p.Hkv * max(1, min(1 + (int)((float)n * rate), n / kPagedWarps));
    });
    if ((int)blockIdx.x < deal[p.B]) {
      const int b = find_row(deal, p.B, blockIdx.x, 1), n = pref[b + 1] - pref[b];
      dealt = (deal[b + 1] - deal[b]) / p.Hkv;
      const int k = blockIdx.x - deal[b], h = k / dealt, q = n / dealt, r = n - q * dealt;
      part = k - h * dealt;
      range0 = pref[b] * p.Hkv + h * n + part * q + min(part, r);
      range1 = range0 + q + (part < r ? 1 : 0);
    }
  } else if ((int)blockIdx.x < sh.blocks) {
    range0 = sh.begin(blockIdx.x);
    range1 = sh.begin(blockIdx.x + 1);
  }
  int4 cut = make_int4(-1, 0, 0, 0);  // the pair that this block begins and others end: pair, first and last block, first slot

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = lane >> 2, c = lane & 3;
  const int P = 1 << p.page_shift;

  // The pair that the block is in, the units [i0, i1) of it that are the block's.
  int b = 0, h = 0, n = 0, i0 = 0, i1 = 0, L = 0, lo = 0;
  const int32_t *table = nullptr, *list = nullptr;
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
  // Head dim 256 keeps Q in shared memory, each warp its own copy: the registers hold K, V and O.
  constexpr bool kSharedQ = paged_shared_q(D) != 0;
  uint4* const s_q = paged_smem + warp * KP * 32 + lane;
  uint4 q[kSharedQ ? 1 : KP];
  int i = 0, tok = 0, tok_next = 0;
  long long r = -1, r_next = -1;
  // Goes on to the next pair from unit g on that this warp has a part in, and enters it: its queries and the
  // warp's first keys are on their way.  A pair is worked on by all warps of the block together, unless it is a
  // small part of the block's share, or of one or two units: then by one of them, in turn, without a barrier (1024
  // pairs of up to 256 tokens: 188 us against 296; of one token: 6.9 against 11.6).
  int step = kPagedWarps, turn = 0;
  auto enter = [&](int g) {
    for (; g < range1; g += n) {
      while (g >= pref[b + 1] * p.Hkv) ++b;
      n = pref[b + 1] - pref[b];
      const int rel = g - pref[b] * p.Hkv;
      h = rel / n;
      i0 = rel - h * n;
      i1 = min(n, i0 + (range1 - g));
      step = i1 - i0 == n && n < range1 - range0 && n <= max((range1 - range0) / 16, 2) ? 1 : kPagedWarps;
      if (step == kPagedWarps || (turn++ & (kPagedWarps - 1)) == warp) break;
    }
    if (g >= range1) return g;
    L = p.seq_lens[b];
    lo = p.pages == nullptr && p.kind == 0 ? max(0, L - p.window) : 0;
    table = p.block_table + (size_t)b * p.max_pages;
    list = p.pages == nullptr ? nullptr : p.pages + ((size_t)b * p.Hkv + h) * p.n_select;
    i = i0 + (step == 1 ? 0 : warp);
    r = r_next = -1;
    if (i < i1) r = locate(i, tok);
    load_k(r);
    // Q as the B fragments of S^T = K Q^T: column `row` is a head, features in the order of K's pieces.
#pragma unroll
    for (int k = 0; k < KP; ++k) {
      uint4& to = kSharedQ ? s_q[k * 32] : q[kSharedQ ? 0 : k];
      to = row < p.G ? __ldg(reinterpret_cast<const uint4*>(p.q_hat + ((size_t)b * p.Hq + h * p.G + row) * D) + c + 4 * k)
                     : make_uint4(0u, 0u, 0u, 0u);
    }
    if (i + step < i1) r_next = locate(i + step, tok_next);
    return g;
  };

  if (range0 < range1) b = find_row(pref, p.B, range0, p.Hkv);
  for (int g = enter(range0); g < range1;) {
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2c, 2c + 1; l: this lane's tokens only
    float o[VP][4][4];
#pragma unroll
    for (int j = 0; j < VP; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][t][e] = 0.f;

    for (; i < i1; i += step) {
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
          const uint4 qk = kSharedQ ? s_q[k * 32] : q[kSharedQ ? 0 : k];  // written by this lane
          mma_bf16(s, kx[0][k].x, kx[1][k].x, kx[0][k].y, kx[1][k].y, qk.x, qk.y);
          mma_bf16(s, kx[0][k].z, kx[1][k].z, kx[0][k].w, kx[1][k].w, qk.z, qk.w);
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
        // P as the sum of two bf16 numbers, which leaves 2^-16 of each weight: P V then has fp32's precision up to the
        // output's rounding.  One bf16 number alone adds an error as large as that rounding, and saves nothing that
        // can be measured: the second product runs under the loads.
        const uint32_t h0 = high_part(p0), h1 = high_part(p1), h2 = high_part(p2), h3 = high_part(p3);
        const uint32_t pb0 = transpose8(__byte_perm(h0, h1, 0x7632)), pb1 = transpose8(__byte_perm(h2, h3, 0x7632));
        const uint32_t pl0 = transpose8(pack_bf16x2(p0 - __uint_as_float(h0), p1 - __uint_as_float(h1)));
        const uint32_t pl1 = transpose8(pack_bf16x2(p2 - __uint_as_float(h2), p3 - __uint_as_float(h3)));
#pragma unroll
        for (int j = 0; j < VP; ++j)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t u0 = piece(vx[0][j], t), u1 = piece(vx[1][j], t), u2 = piece(vx[2][j], t), u3 = piece(vx[3][j], t);
            const uint32_t v0 = __byte_perm(u0, u1, 0x5410), v1 = __byte_perm(u0, u1, 0x7632), v2 = __byte_perm(u2, u3, 0x5410),
                           v3 = __byte_perm(u2, u3, 0x7632);
            mma_bf16(o[j][t], v0, v1, v2, v3, pb0, pb1);
            mma_bf16(o[j][t], v0, v1, v2, v3, pl0, pl1);
          }
      } else {
        load_k(r_next);
      }
      r = r_next;
      tok = tok_next;
      r_next = i + 2 * step < i1 ? locate(i + 2 * step, tok_next) : -1;
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }

    // The pair's end: the first loads for the next one, then the merge of the warps' parts.
    const bool whole = i0 == 0 && i1 == n;
    const bool alone = step == 1;
    const int head0 = b * p.Hq + h * p.G, pair = b * p.Hkv + h, g0 = g - i0, g_pair = g0 + n, first = i0;
    g = enter(g + i1 - i0);
    if (row == 0) {
      *reinterpret_cast<float2*>(s_ml[warp][2 * c]) = make_float2(m0, l0);
      *reinterpret_cast<float2*>(s_ml[warp][2 * c + 1]) = make_float2(m1, l1);
    }
#pragma unroll
    for (int j = 0; j < VP; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int f = row * 8 + 64 * j + 2 * t;
        if (2 * c < p.G) *reinterpret_cast<float2*>(&s_o[warp][2 * c][f]) = make_float2(o[j][t][0], o[j][t][2]);
        if (2 * c + 1 < p.G) *reinterpret_cast<float2*>(&s_o[warp][2 * c + 1][f]) = make_float2(o[j][t][1], o[j][t][3]);
      }
    if (alone) {
      __syncwarp();
      for (int v = lane; v < p.G * (D / 4); v += 32) {
        const int gh = v / (D / 4), f = v % (D / 4) * 4;
        store_row<D>(p, (size_t)head0 + gh, f, s_ml[warp][gh][0], s_ml[warp][gh][1], *reinterpret_cast<const float4*>(&s_o[warp][gh][f]));
      }
      __syncwarp();
      continue;
    }
    __syncthreads();
    // A block's first part goes to its slot 0; one that begins behind another pair's end to slot 1.
    const int slot = 2 * blockIdx.x + (!p.deal && range0 < g0 ? 1 : 0);
    if (!whole && first == 0) cut = make_int4(pair, blockIdx.x, p.deal ? blockIdx.x + dealt - 1 : sh.owner(g_pair - 1), slot);
    if (p.deal && first == 0 && tid == 0) p.cuts[pair] = cut;
    for (int v = tid; v < p.G * (D / 4); v += kPagedThreads) {
      const int gh = v / (D / 4), f = v % (D / 4) * 4;
      float M, sum;
      float4 acc;
      merge_groups<kPagedWarps>(&s_ml[0][gh], 8, &s_o[0][gh][f], 8 * D, M, sum, acc);
      if (whole) {
        store_row<D>(p, (size_t)head0 + gh, f, M, sum, acc);
      } else {
        *reinterpret_cast<float4*>(p.part_o + ((size_t)slot * 8 + gh) * D + f) = acc;
        if (f == 0) *reinterpret_cast<float2*>(p.part_ml + ((size_t)slot * 8 + gh) * 2) = make_float2(M, sum);
      }
    }
    __syncthreads();
  }
  griddep_launch();  // only now: blocks that wait beside these cost them 2 % (1357 against 1328 us for 64 sequences of 4K-32K)
  if (!p.deal && tid == 0) p.cuts[blockIdx.x] = cut;
}

// The pairs that were cut.  With few parts (blocks in equal shares: nearly always
// two) one block merges a whole pair, one thread per 4 features; with many, groups
// of 16 threads take every NG-th part of 64 features of a head, and the blocks of
// grid.y the heads and features.
constexpr int kPagedCombineThreads = 256;

__device__ __forceinline__ void add_part(const PagedDecodeParams& p, int D, size_t at, int f, float& M, float& sum, float4& acc) {
  const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
  const float4 v = *reinterpret_cast<const float4*>(p.part_o + at * D + f);
  const float mn = fmaxf(M, ml.x), base = mn == -INFINITY ? 0.f : mn;
  const float a = ex2_approx(M - base), e = ex2_approx(ml.x - base);
  sum = sum * a + ml.y * e;
  acc.x = acc.x * a + v.x * e;
  acc.y = acc.y * a + v.y * e;
  acc.z = acc.z * a + v.z * e;
  acc.w = acc.w * a + v.w * e;
  M = mn;
}

template <int D>
__global__ void __launch_bounds__(kPagedCombineThreads) paged_combine_kernel(PagedDecodeParams p) {
  constexpr int NG = kPagedCombineThreads / 16;
  __shared__ float s_ml[NG][2];
  __shared__ __align__(16) float s_o[NG][64];
  griddep_wait();
  griddep_launch();
  const int4 cut = p.cuts[blockIdx.x];
  if (cut.x < 0) return;
  const int tid = threadIdx.x, parts = cut.z - cut.y + 1;
  auto slot = [&](int k) { return (size_t)(k == 0 ? cut.w : 2 * (cut.y + k)) * 8; };
  if (parts <= 4) {
    for (int v = blockIdx.y * kPagedCombineThreads + tid; v < p.G * (D / 4); v += gridDim.y * kPagedCombineThreads) {
      const int gh = v / (D / 4), f = v % (D / 4) * 4;
      float M = -INFINITY, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < parts) add_part(p, D, slot(k) + gh, f, M, sum, acc);
      store_row<D>(p, (size_t)cut.x * p.G + gh, f, M, sum, acc);
    }
    return;
  }
  const int grp = tid / 16, f = tid % 16 * 4;
  for (int y = blockIdx.y; y < p.G * (D / 64); y += gridDim.y) {
    const int gh = y / (D / 64), f0 = y % (D / 64) * 64;
    float M = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = grp; k < parts; k += NG) add_part(p, D, slot(k) + gh, f0 + f, M, sum, acc);
    if (f == 0) *reinterpret_cast<float2*>(s_ml[grp]) = make_float2(M, sum);
    *reinterpret_cast<float4*>(&s_o[grp][f]) = acc;
    __syncthreads();
    if (grp == 0) {
      merge_groups<NG>(s_ml, 1, &s_o[0][f], 64, M, sum, acc);
      store_row<D>(p, (size_t)cut.x * p.G + gh, f0 + f, M, sum, acc);
    }
    __syncthreads();
  }
}

template <int D>
static cudaError_t launch_paged_d(const PagedDecodeParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = ensure_dynamic_smem(paged_decode_kernel<D>, paged_shared_q(D) + 2 * (kPagedMaxSeqs + 1) * (int)sizeof(int), done);
  if (e != cudaSuccess) return e;
  const size_t smem = paged_shared_q(D) + (p.deal ? 2 : 1) * (p.B + 1) * sizeof(int);
  return launch_dependent(paged_decode_kernel<D>, dim3(p.n_blocks), dim3(kPagedThreads), smem, st, p);
}

int paged_decode_blocks(int D) { return 148 * (D == 64 ? 4 : D == 128 ? 3 : 2); }

cudaError_t launch_paged_decode(const PagedDecodeParams& p, int D, cudaStream_t st) {
  switch (D) {
    case 64: return launch_paged_d<64>(p, st);
    case 128: return launch_paged_d<128>(p, st);
    case 256: return launch_paged_d<256>(p, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_paged_combine(const PagedDecodeParams& p, int D, cudaStream_t st) {
  const dim3 grid(p.deal ? p.B * p.Hkv : p.n_blocks, p.deal ? p.G * (D / 64) : 1), block(kPagedCombineThreads);
  switch (D) {
    case 64: return launch_dependent(paged_combine_kernel<64>, grid, block, 0, st, p);
    case 128: return launch_dependent(paged_combine_kernel<128>, grid, block, 0, st, p);
    case 256: return launch_dependent(paged_combine_kernel<256>, grid, block, 0, st, p);
  }
  return cudaErrorInvalidValue;
}

}  // namespace g3
