// Paged KV cache: the page map, the append of new tokens, the pages' key bounds
// and the selection of pages by a score on those bounds.  (The attention over
// the pages is in paged_decode.cu.)
//
//   page_map      : block tables, slots and positions of a step's new tokens
//                   from the requests' lengths and a ring of free pages.
//   paged_append  : QK-RMSNorm + RoPE of packed tokens; keys and values go to
//                   their slots, queries to a packed buffer.
//   page_bounds   : feature-wise largest and smallest key of each page and kv
//                   head, in 8 bits.
//   page_select   : an upper bound of q . k over each page's keys, from the bounds,
//                   and the pages with the highest ones of each (sequence, kv head).
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

// ================================================================= page map
// Integer work of a few kilobytes: bound by launch and latency.  Every block
// scans all requests into shared memory (so blocks need no order among them)
// and then takes its share of the tokens and of the new table entries.
constexpr int kMapThreads = 1024;

// Sums of non-negative terms that stop at `cap`: associative, and 32 bits are
// enough for any lengths (cap < 2^31).
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b, uint32_t cap) { return min(a + b, cap); }

// The same of a warp's 32 terms.
__device__ __forceinline__ uint32_t warp_sum(uint32_t v, uint32_t cap) {
  const uint32_t lo = __reduce_add_sync(0xffffffffu, v & 0xffffu), hi = __reduce_add_sync(0xffffffffu, v >> 16);
  return (uint32_t)min(((unsigned long long)hi << 16) + lo, (unsigned long long)cap);
}

template <int ROWS, int THREADS>
__global__ void __launch_bounds__(THREADS) page_map_kernel(PageMapParams p) {
  extern __shared__ int map_smem[];
  uint32_t* ends = reinterpret_cast<uint32_t*>(map_smem);  // [B] rows up to and with request b (stops at max_tokens + 1)
  int* cum = map_smem + p.B;                               // [B] pages asked for up to and with request b
  int* olds = cum + p.B;                                   // [B] tokens cached before, -1 where request b is refused
  __shared__ uint32_t s_rows[32];
  __shared__ int s_need[32];
  __shared__ int s_taken;
  griddep_wait();  // and its dependents wait for its end: blocks beside these cost 2 of 9 us at 512000 rows
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int threads = THREADS, warps = THREADS / 32;
  const uint32_t cap = (uint32_t)p.max_tokens + 1u;
  const long long room = (long long)p.max_pages * p.page_size;
  int head = p.free_state[0], count = p.free_state[1];
  const bool ring_ok = head >= 0 && head < p.free_cap && count >= 0 && count <= p.free_cap;
  if (!ring_ok) {
    head = 0;
    count = 0;
  }
  if (tid == 0) s_taken = 0;

  // Rows first: whether a request fits the token buffer decides whether it asks for pages.
  uint32_t rows_before = 0;
  int need_before = 0;
  int next_old = 0, next_new = 0;
  if (tid < p.B) {
    next_old = p.old_lens[tid];
    next_new = p.new_lens[tid];
  }
  for (int b0 = 0; b0 < p.B; b0 += threads) {
    const int b = b0 + tid, old_len = next_old, new_len = next_new;
    next_old = next_new = 0;
    if (b + threads < p.B) {  // on their way during this turn's sums
      next_old = p.old_lens[b + threads];
      next_new = p.new_lens[b + threads];
    }
    uint32_t rows = min((uint32_t)max(new_len, 0), cap);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, rows, off);
      if (lane >= off) rows = sat_add(rows, v, cap);
    }
    if (lane == 31) s_rows[warp] = rows;
    __syncthreads();
    const uint32_t warp_rows = lane < warps ? s_rows[lane] : 0u;
    rows = sat_add(rows, sat_add(rows_before, warp_sum(lane < warp ? warp_rows : 0u, cap), cap), cap);
    rows_before = sat_add(rows_before, warp_sum(warp_rows, cap), cap);

    const bool valid = b < p.B && old_len >= 0 && new_len >= 0 && (long long)old_len + new_len <= room && rows < cap;
    const int have = valid ? (old_len + p.page_size - 1) >> p.page_shift : 0;
    const int need = valid ? (int)(((long long)old_len + new_len + p.page_size - 1) >> p.page_shift) - have : 0;
    int c = need;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, c, off);
      if (lane >= off) c += v;
    }
    if (lane == 31) s_need[warp] = c;
    __syncthreads();
    const int warp_need = lane < warps ? s_need[lane] : 0;
    c += need_before + __reduce_add_sync(0xffffffffu, lane < warp ? warp_need : 0);
    need_before += __reduce_add_sync(0xffffffffu, warp_need);
    if (b < p.B) {
      ends[b] = rows;
      cum[b] = c;
      const bool granted = valid && (need == 0 || c <= count);
      olds[b] = granted ? old_len : -1;
      if (granted && need > 0) atomicMax(&s_taken, c);
      if (blockIdx.x == 0) {
        p.seq_lens[b] = granted ? old_len + new_len : (old_len >= 0 && old_len <= room ? old_len : 0);
        p.cu_tokens[b + 1] = (int)min(rows, (uint32_t)p.max_tokens);
        if (b == 0) p.cu_tokens[0] = 0;
        if (!valid) record_error(p.status, kErrInvalid, 300);
        if (valid && !granted) record_error(p.status, kErrInvalid, 301);
      }
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.free_state_out[0] = (int)(((long long)head + s_taken) % p.free_cap);
    p.free_state_out[1] = count - s_taken;
    if (!ring_ok) record_error(p.status, kErrInvalid, 303);
  }

  // A granted request's fresh page i (0-based among its own) or -1.
  auto fresh_page = [&](int asked_before, int i) {
    const uint32_t at = (uint32_t)head + (uint32_t)(asked_before + i);  // both parts are below free_cap
    const int id = p.free_pages[at < (uint32_t)p.free_cap ? at : at - (uint32_t)p.free_cap];
    return id >= 0 && id < p.n_pages ? id : -1;
  };

  // New table entries: one warp per request.
  for (int b = blockIdx.x * warps + warp; b < p.B; b += gridDim.x * warps) {
    const int asked = b > 0 ? cum[b - 1] : 0, need = cum[b] - asked;
    if (need == 0 || olds[b] < 0) continue;
    const int have = (olds[b] + p.page_size - 1) >> p.page_shift;
    for (int i = lane; i < need; i += 32) {
      const int id = fresh_page(asked, i);
      p.block_table[(size_t)b * p.max_pages + have + i] = id;
      if (id < 0) record_error(p.status, kErrInvalid, 302);
    }
  }

  // Slot and position of every row of the token buffer: ROWS of them per thread and search.
  const uint32_t rows_end = ends[p.B - 1];
  for (int t0 = (blockIdx.x * threads + tid) * ROWS; t0 < p.max_tokens; t0 += gridDim.x * threads * ROWS) {
    int slot[ROWS], pos[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      slot[k] = -1;
      pos[k] = 0;
    }
    if ((uint32_t)t0 < rows_end) {
      int lo = -1, hi = p.B - 1;  // ends[lo] <= t0 < ends[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] <= (uint32_t)t0)
          lo = mid;
        else
          hi = mid;
      }
      int b = hi, last_b = -1, last_j = -1, page = -1;
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        const int t = t0 + k;
        if (t >= p.max_tokens || (uint32_t)t >= rows_end) break;
        while (ends[b] <= (uint32_t)t) ++b;
        const int old_len = olds[b];
        if (old_len < 0) continue;
        pos[k] = old_len + t - (b > 0 ? (int)ends[b - 1] : 0);
        const int j = pos[k] >> p.page_shift;
        if (b != last_b || j != last_j) {  // rows of one page follow one another: one look-up
          last_b = b;
          last_j = j;
          const int have = (old_len + p.page_size - 1) >> p.page_shift;
          page = j < have ? p.block_table[(size_t)b * p.max_pages + j] : fresh_page(b > 0 ? cum[b - 1] : 0, j - have);
          if (page < 0 || page >= p.n_pages) {
            if (j < have) record_error(p.status, kErrInvalid, 302);
            page = -1;
          }
        }
        if (page >= 0) slot[k] = (page << p.page_shift) + (pos[k] & (p.page_size - 1));
      }
    }
    if (ROWS == 4 && p.wide && t0 + 4 <= p.max_tokens) {
      *reinterpret_cast<int4*>(p.slots + t0) = make_int4(slot[0], slot[1 % ROWS], slot[2 % ROWS], slot[3 % ROWS]);
      *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1 % ROWS], pos[2 % ROWS], pos[3 % ROWS]);
    } else {
#pragma unroll
      for (int k = 0; k < ROWS; ++k)
        if (t0 + k < p.max_tokens) {
          p.slots[t0 + k] = slot[k];
          p.positions[t0 + k] = pos[k];
        }
    }
  }
}

template <int ROWS, int THREADS>
static cudaError_t launch_map(const PageMapParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = ensure_dynamic_smem(page_map_kernel<ROWS, THREADS>, 3 * kPagedMaxSeqs * (int)sizeof(int), done);
  if (e != cudaSuccess) return e;
  const int blocks = std::min(p.max_tokens / (THREADS * ROWS) + 1, 148 * kMapThreads / THREADS);
  return launch_dependent(page_map_kernel<ROWS, THREADS>, dim3(blocks), dim3(THREADS), 3 * p.B * sizeof(int), st, p);
}

// One row per thread keeps a step of single tokens short (64 requests: 4.0 us, 5.6 with four: their look-ups followed one
// another); four spare most searches and stores where one pass of the grid does not do (512000 rows: 6.5 against 7.7).
// Half the threads where one pass over the requests takes no more (64 requests: 3.3 us).
cudaError_t launch_page_map(const PageMapParams& p, cudaStream_t st) {
  if (p.max_tokens > 148 * kMapThreads) return launch_map<4, kMapThreads>(p, st);
  return p.B <= kMapThreads / 2 ? launch_map<1, kMapThreads / 2>(p, st) : launch_map<1, kMapThreads>(p, st);
}

// ============================================================= paged append
// The prefill prologue's arithmetic (norm x / sqrt(mean(x^2) + 1e-6) * gamma in
// fp32, angles in double, rotation in fp32, one rounding to bf16), one warp on a
// share of one token's rows; the keys go to their slots.  HBM-bound on prompts:
// (Hq + 2 Hkv) * D * 2 bytes read and as many written per token.
constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 2;

__device__ __forceinline__ void unpack8(const uint4 u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

//
// FEW: a warp has one share of one token (one turn of the loop), V's rows are rows of their own, and the first loads
// go out before anything else is read: a step's call is bound by the reads that wait for one another.  With many
// tokens the registers that this takes (80 for 64) cost more than it gives: 3.9 us against 3.7 for 256 tokens of
// 32/16 heads, D = 128, 10.5 against 8.5 for 1024; 64 tokens take 2.75 against 3.3.
template <int D, bool FEW>
__global__ void __launch_bounds__(kAppendThreads, FEW ? 3 : 4) paged_append_kernel(PagedAppendParams p) {
  constexpr int H2 = D / 2;
  constexpr int LPR = D / 16;    // lanes per row: each holds 8 features of each half
  constexpr int RPW = 32 / LPR;  // rows per warp step
  constexpr int FPL = (H2 + 31) / 32;
  __shared__ __align__(16) float gam[2 * D];  // q gain, then k gain
  __shared__ double inv_freq_s[H2];
  const int lane = threadIdx.x & 31;
  const int li = lane % LPR, sub = lane / LPR;
  const int d1 = li * 8;
  const int heads = p.Hq + p.Hkv;  // Hq = 0 without queries
  const int rows = FEW ? heads + p.Hkv : heads;
  // `share` of a token's rows: 2^warps_shift warps split them.
  const int warps_per_token = 1 << p.warps_shift;
  const long long items = (long long)p.T << p.warps_shift;
  const long long stride = (long long)gridDim.x * (kAppendThreads / 32);
  long long it = (long long)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  for (int i = threadIdx.x; i < H2; i += kAppendThreads) inv_freq_s[i] = p.inv_freq[i];
  const uint32_t token = griddep_wait_token();
  griddep_launch();
  uint4 xa[kAppendUnroll], xb[kAppendUnroll];
  auto load = [&](int t, int h0, bool keep) {
    const __nv_bfloat16* qrow = p.q + (size_t)t * p.Hq * D;
    const __nv_bfloat16* krow = p.k + (size_t)t * p.Hkv * D;
    const __nv_bfloat16* vrow = p.v + (size_t)t * p.Hkv * D;
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u) {
      const int h = h0 + u * RPW + sub;
      xa[u] = xb[u] = make_uint4(0u, 0u, 0u, 0u);
      if (h < rows && (h < p.Hq || keep)) {
        const __nv_bfloat16* src = h < p.Hq ? qrow + h * D : !FEW || h < heads ? krow + (h - p.Hq) * D : vrow + (h - heads) * D;
        xa[u] = ldg_after(src + d1, token);
        xb[u] = ldg_after(src + H2 + d1, token);
      }
    }
  };
  if (FEW && it < items) load((int)(it >> p.warps_shift), ((int)it & (warps_per_token - 1)) * RPW * kAppendUnroll, true);
  int slot = 0, position = 0;
  auto place = [&]() {
    slot = p.slots[it >> p.warps_shift];
    position = p.positions[it >> p.warps_shift];
  };
  if (FEW && it < items) place();
  for (int i = threadIdx.x; i < 2 * D; i += kAppendThreads)
    gam[i] = i >= D ? p.k_gamma[i - D] : p.Hq > 0 ? p.q_gamma[i] : 0.f;
  __syncthreads();

  for (; it < items; it += stride) {
    const int t = (int)(it >> p.warps_shift), share = (int)it & (warps_per_token - 1);
    if (!FEW) place();
    const bool keep = slot >= 0 && slot < p.n_slots;
    if (slot >= p.n_slots && lane == 0 && share == 0) record_error(p.status, kErrInvalid, 310);
    float cl[FPL], sl[FPL];
    const double pos = (double)position / p.interp;
#pragma unroll
    for (int i = 0; i < FPL; ++i) {
      const int f = FPL * lane + i;
      cl[i] = 1.f;
      sl[i] = 0.f;
      if (f < H2) {
        double sd, cd;
        sincos(pos * inv_freq_s[f], &sd, &cd);
        cl[i] = (float)cd;
        sl[i] = (float)sd;
      }
    }
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = __shfl_sync(0xffffffffu, cl[e % FPL], (d1 + e) / FPL);
      s[e] = __shfl_sync(0xffffffffu, sl[e % FPL], (d1 + e) / FPL);
    }
    // First row of the slot: rows of one (page, head) are P apart from the next head's.
    const size_t page = keep ? (size_t)(slot >> p.page_shift) : 0;
    const size_t crow0 = ((page * p.Hkv) << p.page_shift) + (keep ? slot & ((1 << p.page_shift) - 1) : 0);
    const int first = share * RPW * kAppendUnroll;
    for (int h0 = first; h0 < rows; h0 += warps_per_token * RPW * kAppendUnroll) {
      if (!FEW || h0 != first) load(t, h0, keep);
#pragma unroll
      for (int u = 0; u < kAppendUnroll; ++u) {
        float x[16];
        unpack8(xa[u], x);
        unpack8(xb[u], x + 8);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const int h = h0 + u * RPW + sub;
        if (h >= rows || (h >= p.Hq && !keep)) continue;
        if (FEW && h >= heads) {
          const size_t at = (crow0 + ((size_t)(h - heads) << p.page_shift)) * D;
          *reinterpret_cast<uint4*>(p.v_pages + at + d1) = xa[u];
          *reinterpret_cast<uint4*>(p.v_pages + at + H2 + d1) = xb[u];
          continue;
        }
        const bool is_q = h < p.Hq;
        const float rinv = rsqrtf(ss * (1.0f / D) + 1e-6f);
        const float* gs = gam + (is_q ? 0 : D);
        float g[16];
        *reinterpret_cast<float4*>(g) = *reinterpret_cast<const float4*>(gs + d1);
        *reinterpret_cast<float4*>(g + 4) = *reinterpret_cast<const float4*>(gs + d1 + 4);
        *reinterpret_cast<float4*>(g + 8) = *reinterpret_cast<const float4*>(gs + H2 + d1);
        *reinterpret_cast<float4*>(g + 12) = *reinterpret_cast<const float4*>(gs + H2 + d1 + 4);
        float o[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y1 = x[e] * rinv * g[e];
          const float y2 = x[8 + e] * rinv * g[8 + e];
          o[e] = y1 * c[e] - y2 * s[e];
          o[8 + e] = y1 * s[e] + y2 * c[e];
        }
        if (is_q) {
          __nv_bfloat16* dst = p.q_hat + ((size_t)t * p.Hq + h) * D;
          *reinterpret_cast<uint4*>(dst + d1) = pack8(o);
          *reinterpret_cast<uint4*>(dst + H2 + d1) = pack8(o + 8);
        } else {
          const int kh = h - p.Hq;
          const size_t at = (crow0 + ((size_t)kh << p.page_shift)) * D;
          *reinterpret_cast<uint4*>(p.k_pages + at + d1) = pack8(o);
          *reinterpret_cast<uint4*>(p.k_pages + at + H2 + d1) = pack8(o + 8);
          if (!FEW) {
            const __nv_bfloat16* vsrc = p.v + ((size_t)t * p.Hkv + kh) * D;
            *reinterpret_cast<uint4*>(p.v_pages + at + d1) = ldg_after(vsrc + d1, token);
            *reinterpret_cast<uint4*>(p.v_pages + at + H2 + d1) = ldg_after(vsrc + H2 + d1, token);
          }
        }
      }
    }
  }
}

cudaError_t launch_paged_append(PagedAppendParams p, int D, cudaStream_t st) {
  // A few tokens: split each one's rows over up to 8 warps, as long as each has a step of rows.
  const int rows_step = 32 / (D / 16) * kAppendUnroll;
  auto split = [&](int rows) {
    int shift = 0;
    while (shift < 3 && (rows_step << shift) < rows && ((long long)p.T << shift) < 148 * 16) ++shift;
    return shift;
  };
  p.warps_shift = split(p.Hq + 2 * p.Hkv);
  // FEW (see there) while one block per SM holds them.
  const bool few = (long long)p.T << p.warps_shift <= 148 * (kAppendThreads / 32);
  if (!few) p.warps_shift = split(p.Hq + p.Hkv);
  const long long blocks = (((long long)p.T << p.warps_shift) + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  const dim3 grid((unsigned)std::min<long long>(blocks, 148 * 8));
  switch (D) {
    case 64: return launch_dependent(few ? paged_append_kernel<64, true> : paged_append_kernel<64, false>, grid, dim3(kAppendThreads), 0, st, p);
    case 128: return launch_dependent(few ? paged_append_kernel<128, true> : paged_append_kernel<128, false>, grid, dim3(kAppendThreads), 0, st, p);
    case 256: return launch_dependent(few ? paged_append_kernel<256, true> : paged_append_kernel<256, false>, grid, dim3(kAppendThreads), 0, st, p);
  }
  return cudaErrorInvalidValue;
}

// ============================================================== page bounds
// HBM-bound: the rows of one (page, kv head) are read once, by one warp or, with
// few pages, by up to 8 that share them; a lane keeps the largest and smallest
// value of 8 features in packed bf16.  A page of no more rows than a warp has in
// flight goes to the D / 8 lanes of one row instead (OWN), so that a warp works
// on several pages: 36 us against 77 for 200K tokens of 8 kv heads, D = 64, pages
// of 16 (35 against 42 with pages of 32, 36 against 41 with D = 128); with pages
// of twice that size both take the same time.
constexpr int kBoundsThreads = 256;
constexpr int kBoundsUnroll = 8;  // 16-byte loads in flight per lane

// The largest e with amax * 2^e <= 127, kept within -50 .. 50 (so that products
// of two scaled sums stay finite in fp32), from the bits of a bf16 amax >= 0:
// amax = 2^x (1 + M / 128) gives e = 6 - x, one less when 64 + M / 2 > 127.
__device__ __forceinline__ int bound_exponent(uint32_t bf16_bits) {
  const int x = (int)((bf16_bits >> 7) & 0xff) - 127, m = bf16_bits & 0x7f;
  return max(-50, min(50, 6 - x - (m == 127 ? 1 : 0)));
}
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }  // |e| <= 126

template <int D, bool OWN>
__global__ void __launch_bounds__(kBoundsThreads, 4) page_bounds_kernel(PageBoundsParams p) {
  extern __shared__ int bounds_smem[];  // [B + 1] touched pages before each sequence
  __shared__ int warp_sums[kBoundsThreads / 32];
  __shared__ __nv_bfloat162 s_part[kBoundsThreads / 32][8][32];
  constexpr int LPT = D / 8;     // lanes per row
  constexpr int TPS = 32 / LPT;  // rows per warp-wide load
  griddep_wait();
  griddep_launch();
  const long long room = (long long)p.max_pages << p.page_shift;
  block_prefix(p.B, bounds_smem, warp_sums, [&](int b) {
    const int L = p.seq_lens[b], old = p.old_lens[b];
    if (L < 0 || L > room || old < 0) {
      if (blockIdx.x == 0) record_error(p.status, kErrInvalid, 320);
      return 0;
    }
    return old < L ? ((L + (1 << p.page_shift) - 1) >> p.page_shift) - (old >> p.page_shift) : 0;
  });
  const int units = bounds_smem[p.B] * p.Hkv;  // below 2^30: checked on the host for the widest table
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, li = lane % LPT, sub = lane / LPT;
  const int P = 1 << p.page_shift;
  constexpr int WARPS = kBoundsThreads / 32;
  int split = 1;  // warps that share a unit's rows
  while (!OWN && split < WARPS && units <= (int)gridDim.x * WARPS / (2 * split) && split * TPS * kBoundsUnroll < P) split *= 2;
  const int part = warp % split;
  constexpr int PER_WARP = OWN ? TPS : 1, ROW_STEP = OWN ? 1 : TPS;
  const int row0 = OWN ? 0 : sub;
  for (int u0 = blockIdx.x * (WARPS / split); u0 * PER_WARP < units; u0 += gridDim.x * (WARPS / split)) {
    const int u = OWN ? (u0 + warp) * TPS + sub : u0 + warp / split, pj = min(u, units - 1) / p.Hkv, h = u % p.Hkv;
    const int b = find_row(bounds_smem, p.B, pj, 1);
    const int j = (p.old_lens[b] >> p.page_shift) + pj - bounds_smem[b];
    const int page = p.block_table[(size_t)b * p.max_pages + j];
    const bool ok = u < units && page >= 0 && page < p.n_pages;
    if (u < units && !ok && li == 0) record_error(p.status, kErrInvalid, 321);
    const int rows = ok ? min(P, p.seq_lens[b] - (j << p.page_shift)) : 0;
    const uint4* base = reinterpret_cast<const uint4*>(p.k_pages + (((size_t)(ok ? page : 0) * p.Hkv + h) << p.page_shift) * D) + li;
    const __nv_bfloat162 ninf = __floats2bfloat162_rn(-INFINITY, -INFINITY), pinf = __floats2bfloat162_rn(INFINITY, INFINITY);
    __nv_bfloat162 mx[4], mn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mx[i] = ninf;
      mn[i] = pinf;
    }
    for (int r0 = part * ROW_STEP * kBoundsUnroll; r0 < rows; r0 += split * ROW_STEP * kBoundsUnroll) {
      uint4 x[kBoundsUnroll];
#pragma unroll
      for (int k = 0; k < kBoundsUnroll; ++k) {
        const int r = min(r0 + k * ROW_STEP + row0, rows - 1);  // a row read twice changes nothing
        x[k] = __ldg(base + (size_t)r * LPT);
      }
#pragma unroll
      for (int k = 0; k < kBoundsUnroll; ++k) {
        const __nv_bfloat162* v = reinterpret_cast<const __nv_bfloat162*>(&x[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // the _nan forms keep a NaN
          mx[i] = __hmax2_nan(mx[i], v[i]);
          mn[i] = __hmin2_nan(mn[i], v[i]);
        }
      }
    }
    if (!OWN) {
#pragma unroll
      for (int off = LPT; off < 32; off <<= 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mx[i] = __hmax2_nan(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], off));
          mn[i] = __hmin2_nan(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], off));
        }
      }
    }
    if (split > 1) {
      __syncthreads();  // the last unit's parts have been read
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s_part[warp][i][lane] = mx[i];
        s_part[warp][4 + i][lane] = mn[i];
      }
      __syncthreads();
      if (part == 0) {
        for (int w = 1; w < split; ++w)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mx[i] = __hmax2_nan(mx[i], s_part[warp + w][i][lane]);
            mn[i] = __hmin2_nan(mn[i], s_part[warp + w][4 + i][lane]);
          }
      }
    }
    if (part != 0) continue;
    // Bits of |x| of bf16 values order as integers; a NaN's are above infinity's.
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = *reinterpret_cast<uint32_t*>(&mx[i]) & 0x7fff7fffu, c = *reinterpret_cast<uint32_t*>(&mn[i]) & 0x7fff7fffu;
      amax = max(amax, max(max(a & 0xffffu, a >> 16), max(c & 0xffffu, c >> 16)));
    }
#pragma unroll
    for (int off = LPT / 2; off > 0; off >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    const int e = bound_exponent(amax);
    const float unit = exp2_int(e);
    uint32_t hi8[2] = {0, 0}, lo8[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 a = mx[i / 2], c = mn[i / 2];
      const float fa = __bfloat162float(i % 2 ? a.y : a.x), fc = __bfloat162float(i % 2 ? c.y : c.x);
      // Outward: the largest up, the smallest down (a product that underflows still counts as nonzero).
      float ua = ceilf(fa * unit), uc = floorf(fc * unit);
      if (fa > 0.f) ua = fmaxf(ua, 1.f);
      if (fc < 0.f) uc = fminf(uc, -1.f);
      ua = fa != fa ? 127.f : fminf(fmaxf(ua, -127.f), 127.f);
      uc = fc != fc ? -127.f : fminf(fmaxf(uc, -127.f), 127.f);
      hi8[i / 4] |= ((uint32_t)(int)ua & 0xffu) << (8 * (i % 4));
      lo8[i / 4] |= ((uint32_t)(int)uc & 0xffu) << (8 * (i % 4));
    }
    if (ok && (OWN || sub == 0)) {
      const size_t ph = (size_t)page * p.Hkv + h;
      uint2* dst = reinterpret_cast<uint2*>(p.bounds + ph * 2 * D);
      dst[li] = make_uint2(hi8[0], hi8[1]);
      dst[LPT + li] = make_uint2(lo8[0], lo8[1]);
      if (li == 0) p.exps[ph] = (int8_t)e;
    }
  }
}

cudaError_t launch_page_bounds(const PageBoundsParams& p, int D, cudaStream_t st) {
  const long long most = ((long long)p.B * p.max_pages * p.Hkv + kBoundsThreads / 32 - 1) / (kBoundsThreads / 32);
  const dim3 grid((unsigned)std::min<long long>(most, 148 * 4)), block(kBoundsThreads);
  const size_t smem = (p.B + 1) * sizeof(int);
  const bool own = (1 << p.page_shift) <= 256 / D * kBoundsUnroll;
  switch (D) {
    case 64: return launch_dependent(own ? page_bounds_kernel<64, true> : page_bounds_kernel<64, false>, grid, block, smem, st, p);
    case 128: return launch_dependent(own ? page_bounds_kernel<128, true> : page_bounds_kernel<128, false>, grid, block, smem, st, p);
    case 256: return launch_dependent(page_bounds_kernel<256, false>, grid, block, smem, st, p);
  }
  return cudaErrorInvalidValue;
}

// ============================================================== page select
// score(b, kv head, page) = max over the group's query heads of
//     2^-(eq + ek) * sum_d (q8_d >= 0 ? q8_d * max8_d : q8_d * min8_d),
// with q8 = the query's features rounded to 8 bits with a power-of-two exponent
// eq of its own.  As a product: [q8+, q8-] (2D features) with [max8, min8], whole
// numbers below 2^24 in any order, so the scores are exact and the selection does
// not depend on how they are summed.  HBM-bound: 2D + 1 bytes per (page, kv head).
//
// The warps of a block bring the group's queries to 8 bits, one head each, then
// score 16 pages at a time as mma.m16n8k32 of 8-bit whole numbers: rows are pages,
// columns the group's heads.  Each lane loads 16-byte pieces of two pages' bounds
// straight into its A fragments; the order of the features inside a product is
// free, so the pieces are used as they come and the query is laid out to match.
// (The same on fp16 numbers made from the bytes took half as long again, dp4a up
// to a tenth longer.)
//
// A cluster of blocks scores a pair (sequence, kv head) into the shared memory of
// its first block, which picks behind the cluster's barrier: the scores as ordered
// integers, the threshold by 11-bit digits below the highest bit in which they
// differ, then an ordered write.
__device__ __forceinline__ void mma_s8(int* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Ascending order of the floats (no NaN) as ascending unsigned integers; -0 counts as +0.
__device__ __forceinline__ uint32_t ordered_bits(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Pages of a sequence; 0 for a length out of range.
__device__ __forceinline__ int pages_of(const PageSelectParams& p, int b, bool report) {
  const int L = p.seq_lens[b];
  if (L < 0 || L > (long long)p.max_pages << p.page_shift) {
    if (report) record_error(p.status, kErrInvalid, 330);
    return 0;
  }
  return (L + (1 << p.page_shift) - 1) >> p.page_shift;
}

// One head of a group in 8 bits, held by the lanes of a warp: loaded, then laid out.
template <int D>
struct QueryHead {
  static constexpr int FPL = D / 32;
  static constexpr int ROW = 2 * D + 64;  // bytes from one head to the next: 16-byte reads without conflicts
  float x[FPL];
  __device__ void load(const PageSelectParams& p, int b, int h, int g, int lane) {
#pragma unroll
    for (int i = 0; i < FPL; ++i)
      x[i] = g < p.G ? __bfloat162float(p.q_hat[((size_t)b * p.Hq + h * p.G + g) * D + i * 32 + lane]) : 0.f;
  }
  // Positive parts, then negative parts, to q8's row g; the unit 2^-eq to unit[g].
  __device__ void store(int8_t* q8, float* unit, int g, int lane) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < FPL; ++i) {
      if (x[i] != x[i]) x[i] = 0.f;
      amax = max(amax, (__float_as_uint(x[i]) & 0x7fffffffu) >> 16);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    const int e = bound_exponent(amax);
    const float up = exp2_int(e);
#pragma unroll
    for (int i = 0; i < FPL; ++i) {
      const int v = (int)fminf(fmaxf(rintf(x[i] * up), -127.f), 127.f);
      q8[g * ROW + i * 32 + lane] = (int8_t)max(v, 0);
      q8[g * ROW + D + i * 32 + lane] = (int8_t)min(v, 0);
    }
    if (lane == 0) unit[g] = exp2_int(-e);
  }
};

// Scores pages j0 .. j0 + 15, then every `step`-th such run below `end`, of one pair
// with np pages, by one warp; put(page, key) receives each once.
template <int D, class Put>
__device__ __forceinline__ void score_pages(const PageSelectParams& p, const int32_t* table, int h, int np, int j0, int end, int step,
                                            const int8_t* q8, const float* unit, Put&& put) {
  constexpr int PIECES = 2 * D / 64;  // 16-byte pieces of a page's bounds per lane
  const int lane = threadIdx.x & 31, row = lane >> 2, c = lane & 3;
  const float unit0 = unit[2 * c], unit1 = unit[2 * c + 1];
  const bool has0 = 2 * c < p.G, has1 = 2 * c + 1 < p.G;
  int id0 = 0, id1 = 0;
  if (j0 < end) {
    id0 = table[min(j0 + row, np - 1)];
    id1 = table[min(j0 + row + 8, np - 1)];
  }
  for (; j0 < end; j0 += step) {
    // Physical pages of rows `row` and `row + 8` (past the last page it is repeated); a bad one scores -infinity.
    const bool bad0 = id0 < 0 || id0 >= p.n_pages, bad1 = id1 < 0 || id1 >= p.n_pages;
    if (bad0 || bad1) record_error(p.status, kErrInvalid, 331);
    const size_t ph0 = (size_t)(bad0 ? 0 : id0) * p.Hkv + h, ph1 = (size_t)(bad1 ? 0 : id1) * p.Hkv + h;
    const uint4* s0 = reinterpret_cast<const uint4*>(p.bounds + ph0 * 2 * D) + c;
    const uint4* s1 = reinterpret_cast<const uint4*>(p.bounds + ph1 * 2 * D) + c;
    uint4 a0[PIECES], a1[PIECES];
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
      a0[k] = __ldg(s0 + 4 * k);
      a1[k] = __ldg(s1 + 4 * k);
    }
    const int e0 = p.exps[ph0], e1 = p.exps[ph1];
    if (j0 + step < end) {
      id0 = table[min(j0 + step + row, np - 1)];
      id1 = table[min(j0 + step + row + 8, np - 1)];
    }
    int acc[2][4] = {};  // two chains
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
      const uint4 q = *reinterpret_cast<const uint4*>(&q8[row * QueryHead<D>::ROW + c * 16 + 64 * k]);
      mma_s8(acc[0], a0[k].x, a1[k].x, a0[k].y, a1[k].y, q.x, q.y);
      mma_s8(acc[1], a0[k].z, a1[k].z, a0[k].w, a1[k].w, q.z, q.w);
    }
    // Page row / row + 8, heads 2c and 2c + 1.
    const float lo0 = (float)(acc[0][0] + acc[1][0]) * unit0, lo1 = (float)(acc[0][1] + acc[1][1]) * unit1;
    const float hi0 = (float)(acc[0][2] + acc[1][2]) * unit0, hi1 = (float)(acc[0][3] + acc[1][3]) * unit1;
    float s_lo = fmaxf(has0 ? lo0 : -INFINITY, has1 ? lo1 : -INFINITY) * exp2_int(-e0);
    float s_hi = fmaxf(has0 ? hi0 : -INFINITY, has1 ? hi1 : -INFINITY) * exp2_int(-e1);
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      s_lo = fmaxf(s_lo, __shfl_xor_sync(0xffffffffu, s_lo, off));
      s_hi = fmaxf(s_hi, __shfl_xor_sync(0xffffffffu, s_hi, off));
    }
    if (c == 0) {
      if (j0 + row < np) put(j0 + row, ordered_bits(bad0 ? -INFINITY : s_lo));
      if (j0 + row + 8 < np) put(j0 + row + 8, ordered_bits(bad1 ? -INFINITY : s_hi));
    }
  }
}

constexpr int kPickBits = 11, kPickBins = 1 << kPickBits;
template <int THREADS>
struct PickSmem {
  __align__(16) uint32_t hist[kPickBins];  // highest digit first
  uint32_t sums[THREADS / 32], digit, left, count;
  uint32_t lo[THREADS / 32], hi[THREADS / 32];
  int gt[THREADS / 32], eq[THREADS / 32];
};

// The k highest of n keys (0 < k < n), equal ones by the lower index, in ascending
// order of the index, by the whole block.
template <int THREADS, class Key>
__device__ __forceinline__ void pick_pages(Key&& key, int n, int k, int32_t* out, PickSmem<THREADS>& sm) {
  constexpr int WARPS = THREADS / 32, PER = kPickBins / THREADS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t lo = 0xffffffffu, hi = 0;
#pragma unroll 4
  for (int i = tid; i < n; i += THREADS) {
    const uint32_t u = key(i);
    lo = min(lo, u);
    hi = max(hi, u);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    sm.lo[warp] = lo;
    sm.hi[warp] = hi;
  }
  // PER bins of the histogram from tid * PER on belong to this thread.
  uint32_t* mine = sm.hist + PER * tid;
#pragma unroll
  for (int i = 0; i < PER; ++i) mine[i] = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    lo = min(lo, sm.lo[w]);
    hi = max(hi, sm.hi[w]);
  }
  // (key - lo) >> shift of the k-th highest is `prefix`; `left` of the scores with that prefix are taken.
  uint32_t prefix = 0, left = k;
  int shift = 32 - __clz(hi - lo);
  while (shift > 0) {
    const int next = max(shift - kPickBits, 0), bits = shift - next;
#pragma unroll 4
    for (int i = tid; i < n; i += THREADS) {
      const uint32_t u = key(i) - lo;
      if (shift == 32 || (u >> shift) == prefix) atomicAdd(&sm.hist[kPickBins - 1 - ((u >> next) & ((1u << bits) - 1u))], 1u);
    }
    __syncthreads();
    uint32_t d[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      d[i] = mine[i];
      sum += d[i];
    }
    uint32_t before = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, before, off);
      if (lane >= off) before += v;
    }
    if (lane == 31) sm.sums[warp] = before;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine[i] = 0;  // for a finer digit
    __syncthreads();
    before -= sum;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) before += w < warp ? sm.sums[w] : 0u;
    if (before < left && before + sum >= left) {  // one thread: the digit at which the count from above reaches `left`
      uint32_t digit = 0, count = 0, taken = before;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (before < left) {
          digit = kPickBins - 1 - (tid * PER + i);
          count = d[i];
          taken = before;
        }
        before += d[i];
      }
      sm.digit = digit;
      sm.count = count;
      sm.left = left - taken;
    }
    __syncthreads();
    prefix = (shift == 32 ? 0u : prefix << bits) | sm.digit;
    left = sm.left;
    shift = next;
    if (sm.count == left) break;  // all of them are taken: no finer threshold is needed
  }
  const int per = ((n + WARPS - 1) / WARPS + 31) / 32 * 32, i0 = min(n, warp * per), i1 = min(n, i0 + per);
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint32_t u = (key(i) - lo) >> shift;
    gt += u > prefix;
    eq += u == prefix;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    sm.gt[warp] = gt;
    sm.eq[warp] = eq;
  }
  __syncthreads();
  int gt0 = 0, eq0 = 0;
  for (int w = 0; w < warp; ++w) {
    gt0 += sm.gt[w];
    eq0 += sm.eq[w];
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1;
    const uint32_t u = in ? (key(i + lane) - lo) >> shift : 0u;
    const bool is_gt = in && u > prefix, is_eq = in && u == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
    const int eq_rank = eq0 + __popc(be & below);
    const int at = gt0 + __popc(bg & below) + min(eq_rank, (int)left);
    if (is_gt || (is_eq && eq_rank < (int)left)) out[at] = i + lane;
    gt0 += __popc(bg);
    eq0 += __popc(be);
  }
}

// The newest page, and the picked ones before it.
template <int THREADS, class Key>
__device__ __forceinline__ void write_pages(Key&& key, int np, int n_select, int32_t* out, PickSmem<THREADS>& sm) {
  if (threadIdx.x == 0) out[n_select - 1] = np - 1;
  if (n_select > 1) pick_pages(key, np - 1, n_select - 1, out, sm);
}

// A sequence without a choice: all its pages.
template <int THREADS>
__device__ __forceinline__ void write_all(int np, int n_select, int32_t* out) {
  for (int i = threadIdx.x; i < n_select; i += THREADS) out[i] = i < np ? i : -1;
}

template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS, (D == 256 ? 512 : 1024) / THREADS) page_select_kernel(PageSelectParams p) {
  __shared__ __align__(16) int8_t q8[8 * QueryHead<D>::ROW];
  __shared__ float q_unit[8];
  __shared__ PickSmem<THREADS> pick;
  extern __shared__ uint32_t smem_keys[];  // the first block's: the scores as ordered integers
  constexpr int WARPS = THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ranks = cluster_size(), rank = blockIdx.x % ranks;
  const int turn = blockIdx.x / ranks / p.Hkv, h = blockIdx.x / ranks % p.Hkv;
  int b = turn;
  cluster_arrive_relaxed();  // waited for before the first store to the first block: it has to be running by then
  griddep_wait();
  griddep_launch();
  if (p.by_length) {
    // The `turn`-th longest sequence: the blocks that start last have the least to do.
    __shared__ int s_len[THREADS], s_b;
    const int t = threadIdx.x, mine = t < p.B ? p.seq_lens[t] : 0;
    s_len[t] = mine;
    __syncthreads();
    int before = 0;
    for (int j = 0; j < p.B; ++j) before += s_len[j] > mine || (s_len[j] == mine && j < t);
    if (t < p.B && before == turn) s_b = t;
    __syncthreads();
    b = s_b;
  }
  const int pair = b * p.Hkv + h;
  QueryHead<D> head;
  if (warp < 8) head.load(p, b, h, warp, lane);  // on its way while the length is read
  const int np = pages_of(p, b, rank == 0 && threadIdx.x == 0);
  int32_t* out = p.pages + (size_t)pair * p.n_select;
  if (np <= p.n_select) {  // the same for the whole cluster
    if (rank == 0) write_all<THREADS>(np, p.n_select, out);
    return;
  }
  if (warp < 8) head.store(q8, q_unit, warp, lane);
  __syncthreads();
  cluster_wait();
  const int32_t* table = p.block_table + (size_t)b * p.max_pages;
  uint32_t* keys = p.keys + (size_t)pair * p.max_pages;
  const bool in_smem = np <= p.keys_in_smem;
  const uint32_t first_keys = cluster_address(smem_keys, 0);
  score_pages<D>(p, table, h, np, (rank * WARPS + warp) * 16, np, ranks * WARPS * 16, q8, q_unit,
                 [&](int j, uint32_t key) {
                   if (in_smem)
                     cluster_store(first_keys + 4 * j, key);
                   else
                     keys[j] = key;
                 });
  cluster_arrive();  // releases the keys to the cluster
  if (rank != 0) return;
  cluster_wait();
  if (in_smem)
    write_pages([&](int i) { return smem_keys[i]; }, np, p.n_select, out, pick);
  else  // other blocks wrote them: read where they are written, in L2
    write_pages([&](int i) { return __ldcg(keys + i); }, np, p.n_select, out, pick);
}

template <int D, int THREADS>
static cudaError_t launch_select_d(PageSelectParams p, cudaStream_t st) {
  const long long pairs = (long long)p.B * p.Hkv;
  constexpr int WARPS = THREADS / 32;
  // Blocks per pair: up to 8, at least 16 pages for each of their warps, no more than find a place at once (2 per SM at
  // D = 256, else 4).  A second wave sets up and joins its clusters again: 200 pairs of D = 256 take 12.7 us in one wave
  // of single blocks against 18.3 with two blocks per pair for up to 512 pages, 34.7 against 34.9 for 2048, 250 pairs
  // 14.0 against 21.4 and 37.6 against 40.9; only around 160 pairs of 2048 pages is the second wave shorter (27.6
  // against 33.1).
  int ranks = 1;
  constexpr int kPlaces = 148 * (D == 256 ? 2 : 4);
  while (ranks < 8 && ranks * WARPS * 16 < p.max_pages && pairs * ranks * 2 <= kPlaces) ranks *= 2;
  // More blocks than find a place at once: the long sequences first (56 us against 61 for 1024 pairs of up to
  // 2048 pages), as far as a block can rank them with a thread each.
  p.by_length = pairs * ranks > kPlaces && p.B <= THREADS;
  // Room for the scores of the longest table, up to 32 KB: 8192 pages in a single sequence took 22 us so and 33 with
  // their scores in L2 (blocks of 256), while 32 KB for every call cost the short ones 0.4 us and the batch above 4.
  p.keys_in_smem = std::min(p.max_pages, kKeysInSmem);
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = p.keys_in_smem * sizeof(uint32_t);
  cfg.gridDim = dim3((unsigned)(pairs * ranks));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, page_select_kernel<D, THREADS>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_page_select(const PageSelectParams& p, int D, cudaStream_t st) {
  // Blocks of 512 threads where every cluster of 8 finds an SM for each of its blocks: the pick, by one block, takes half
  // the time.  One sequence with 16 kv heads of D = 128: 6.3 us against 6.7 at 1024 pages, 18-20 against 22 at 8192; with
  // one of D = 256 7.4 against 8.0 at 2048, 34 against 48 at 16384.  Two blocks per SM (32 pairs, 2048 pages): 11.2 against 9.2.
  const bool wide = (long long)p.B * p.Hkv * 8 <= 148 && p.max_pages >= 1024;
  switch (D) {
    case 64: return wide ? launch_select_d<64, 512>(p, st) : launch_select_d<64, 256>(p, st);
    case 128: return wide ? launch_select_d<128, 512>(p, st) : launch_select_d<128, 256>(p, st);
    case 256: return wide ? launch_select_d<256, 512>(p, st) : launch_select_d<256, 256>(p, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace g3
