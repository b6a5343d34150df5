// The paged K/V cache's writers: appending tokens to pages taken from the pool, forking
// (sharing, cutting and freeing) sequences, and compacting the pool.
//
// Free pages are bits in a map, and a call takes the lowest-numbered ones in the order of
// its sequences and their logical pages, so what a call does follows from lengths,
// table and counts alone and is the same every time.  A page that is not complete belongs to one
// sequence: a fork shares complete pages and copies a partial one, so appends never meet a
// shared page.
//
// Appends and compactions move bytes, at the memory's rate on large ones: four prompts of up to 32k tokens of 8
// heads of 128 channels 147 us for 973 MB (99% of the measured copy), 8100 of 16400 used pages of 32 KB moved 87 us
// for 537 MB (92%). What is small is a chain of latencies: single tokens of 32
// sequences 5.9 us, a reordering of 32 beams 9.0, of which the counts, the choice of the pages to copy and
// the second launch are about a third each, and 250 pages of 8 KB moved 6.7. (Times of the device alone, calls
// replayed from a graph.)
#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "paged.cuh"
#include "status.cuh"

namespace sls {

// Plans are made by one CTA, of 256 threads (1024 for more than 1024 sequences: a barrier of 32 warps
// costs several of 8) with up to four sequences each.
constexpr int kPlanThreads = 1024, kPlanFew = 256, kPlanMost = 4, kPlanPages = 1024;
static_assert(kPlanThreads * kPlanMost == kPagedMaxSeqs, "a plan holds every sequence");

// Exclusive scan of one int per thread over the CTA; `total` gets the sum.
template <int NT>
__device__ __forceinline__ int plan_scan(int v, int* tmp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // an earlier scan's reads of tmp
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    before += w < warp ? tmp[w] : 0;
    total += tmp[w];
  }
  return before + x - v;
}

template <int NT>
struct PlanShared {
  uint32_t word[NT];
  int base[NT], tmp[NT / 32];
};

// The `total` lowest-numbered free pages (there are as many): give(rank, page) for each.  TAKE: their
// bits are cleared.  All threads of the CTA call it.
template <int NT, bool TAKE, typename F>
__device__ __forceinline__ void find_pages(const Paged& c, int first, int total, PlanShared<NT>& sh, F give) {
  uint32_t* bits = paged_bits(c);
  const int words = paged_words(c.pages), tid = threadIdx.x, lane = tid & 31;
  int got = 0;
  for (int w0 = max(first, 0); got < total && w0 < words; w0 += NT) {
    const uint32_t word = w0 + tid < words ? bits[w0 + tid] : 0u;
    int sum;
    const int base = got + plan_scan<NT>(__popc(word), sh.tmp, sum);
    sh.word[tid] = word;
    sh.base[tid] = base;
    __syncthreads();
    for (int i = tid >> 5; i < NT && sh.base[i] < total; i += NT / 32) {
      const uint32_t x = sh.word[i];
      const int r = sh.base[i] + __popc(x & ((1u << lane) - 1u));
      if ((x >> lane & 1u) && r < total) give(r, (w0 + i) * 32 + lane);
    }
    if (TAKE && word && base < total) {
      uint32_t left = word;
      for (int k = base; k < total && left; ++k) left &= left - 1;
      bits[w0 + tid] = left;
      if (base + __popc(word) >= total) c.state[1] = w0 + tid;
    }
    got += sum;
    __syncthreads();
  }
  if (TAKE && tid == 0) c.state[0] -= total;
}

// Whether this CTA is the last of the grid's to get here: all others have read what they need of the
// cache's integers, and their writes before this are seen.  The count is zero again afterwards.
__device__ __forceinline__ bool last_to_arrive(const Paged& c, int ctas) {
  __shared__ int s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(c.state + 3, 1) == ctas - 1;
    if (s_last) c.state[3] = 0;
    __threadfence();
  }
  __syncthreads();
  return s_last != 0;
}

// ------------------------------------------------------------------- the state from the table

__global__ void __launch_bounds__(256)
paged_clear_kernel(const Paged c) {
  pdl_wait_then_release();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < c.pages) c.refs[i] = 0;
  if (i < kPagedHead) c.state[i] = 0;
}

// Counts every sequence's pages; entries past its length become -1.
__global__ void __launch_bounds__(256)
paged_count_kernel(const Paged c, int B, int Cap, int pshift) {
  pdl_wait_then_release();
  const int MP = Cap >> pshift;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)B * MP) return;
  const int b = (int)(i / MP), l = (int)(i % MP);
  const int n = clamp_len(c.ctx[b], Cap);
  if (l >= (n + (1 << pshift) - 1) >> pshift) {
    c.table[i] = -1;
  } else {
    const int p = c.table[i];
    if (paged_page(p, c.pages)) atomicAdd(c.refs + p, 1);
    else note_bad_pages(1);
  }
}

__global__ void __launch_bounds__(256)
paged_free_kernel(const Paged c) {
  pdl_wait_then_release();
  const int p = blockIdx.x * 256 + threadIdx.x;
  const uint32_t word = __ballot_sync(0xffffffffu, p < c.pages && c.refs[p] == 0);
  if ((threadIdx.x & 31) == 0 && p < c.pages) {
    paged_bits(c)[p >> 5] = word;
    atomicAdd(c.state, __popc(word));
  }
}

cudaError_t launch_paged_init(const Shape& s, const Paged& c, cudaStream_t st) {
  const int ctas = (c.pages + 255) / 256;
  const int64_t entries = (int64_t)s.B * (s.Cap >> s.pshift);
  cudaError_t e = launch_pdl(paged_clear_kernel, dim3(ctas), dim3(256), 0, st, c);
  if (e == cudaSuccess)
    e = launch_pdl(paged_count_kernel, dim3((unsigned)((entries + 255) / 256)), dim3(256), 0, st, c, s.B, s.Cap, s.pshift);
  if (e == cudaSuccess) e = launch_pdl(paged_free_kernel, dim3(ctas), dim3(256), 0, st, c);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ------------------------------------------------------------------- append

// Which sequences append, and how many pages that takes in all.  A sequence needs the pages between
// those it has and those its new length takes; it appends if its tokens fit its capacity and its and the
// earlier sequences' pages are there (or it needs none), and its partial page is its own.  Thread i has
// sequences [i per, (i + 1) per): start and n (0: it appends nothing), and the page of its partial one.
struct AppendPlan {
  int b0, b1, start[kPlanMost], n[kPlanMost], page[kPlanMost];
};
template <int NT>
__device__ __forceinline__ int append_plan(const Paged& c, const int32_t* new_len, int max_new, int B, int Cap, int pshift,
                                           bool count, AppendPlan& p, int* s_first, int* s_had, int* s_total, PlanShared<NT>& sh) {
  const int tid = threadIdx.x, P = 1 << pshift, MP = Cap >> pshift, free = c.state[0];
  const int per = (B + NT - 1) / NT;
  p.b0 = min(tid * per, B);
  p.b1 = min(p.b0 + per, B);
  int need[kPlanMost], sum = 0;
#pragma unroll
  for (int i = 0; i < kPlanMost; ++i) {
    const int b = p.b0 + i;
    p.start[i] = p.n[i] = need[i] = 0;
    p.page[i] = -1;
    if (b >= p.b1) continue;
    p.start[i] = clamp_len(c.ctx[b], Cap);
    p.n[i] = new_len ? min(max(new_len[b], 0), max_new) : max_new;
    if (p.n[i] > Cap - p.start[i]) p.n[i] = 0;
    if (p.n[i] && (p.start[i] & (P - 1))) {
      p.page[i] = c.table[(size_t)b * MP + (p.start[i] >> pshift)];
      if (!paged_page(p.page[i], c.pages) || c.refs[p.page[i]] != 1) {
        if (count) note_bad_pages(1);
        p.n[i] = 0;
      }
    }
    const int had = (p.start[i] + P - 1) >> pshift;
    if (p.n[i]) need[i] = (int)(((int64_t)p.start[i] + p.n[i] + P - 1) >> pshift) - had;
    s_had[b] = had;
    sum += need[i];
  }
  if (tid == 0) *s_total = 0;
  int all;
  int first = plan_scan<NT>(sum, sh.tmp, all), most = 0;
#pragma unroll
  for (int i = 0; i < kPlanMost; ++i) {
    const int b = p.b0 + i;
    if (b >= p.b1) continue;
    s_first[b] = first;
    first += need[i];
    if (need[i] && first <= free) most = first;
    else if (need[i]) p.n[i] = 0;
  }
  // the pages of the sequences that append are the first ones in order
  most = __reduce_max_sync(0xffffffffu, most);
  if ((tid & 31) == 0) atomicMax(s_total, most);
  __syncthreads();
  return *s_total;
}
// The sequence that takes the r-th page: the last one whose first page is r or before.
__device__ __forceinline__ int append_taker(const int* s_first, int B, int r) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_first[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The new lengths and the positions reported.
__device__ __forceinline__ void append_record(const Paged& c, const AppendPlan& p, int32_t* pos_out) {
#pragma unroll
  for (int i = 0; i < kPlanMost; ++i) {
    const int b = p.b0 + i;
    if (b >= p.b1) continue;
    if (p.n[i]) c.ctx[b] = p.start[i] + p.n[i];
    if (pos_out) pos_out[b] = p.n[i] ? p.start[i] : -1;
  }
}

template <int NT>
__global__ void __launch_bounds__(NT)
paged_plan_kernel(const Paged c, const int32_t* new_len, int max_new, int32_t* pos_out, int B, int Cap, int pshift) {
  __shared__ PlanShared<NT> sh;
  __shared__ int s_first[NT * kPlanMost], s_had[NT * kPlanMost], s_total;
  pdl_wait_then_release();
  const int MP = Cap >> pshift, first = c.state[1];
  AppendPlan p;
  const int total = append_plan<NT>(c, new_len, max_new, B, Cap, pshift, true, p, s_first, s_had, &s_total, sh);
#pragma unroll
  for (int i = 0; i < kPlanMost; ++i)
    if (p.b0 + i < p.b1) paged_spans(c)[p.b0 + i] = make_int2(p.start[i], p.n[i]);
  append_record(c, p, pos_out);
  if (total == 0) return;
  find_pages<NT, true>(c, first, total, sh, [&](int r, int page) {
    const int b = append_taker(s_first, B, r);
    c.table[(size_t)b * MP + s_had[b] + r - s_first[b]] = page;
    c.refs[page] = 1;
  });
}

template <typename T>
struct PagedLimits;
template <>
struct PagedLimits<bf16> {
  static __device__ __forceinline__ void fold(uint4& lo, uint4& hi, const uint4& a, const uint4& b) {
    __nv_bfloat162 *l = reinterpret_cast<__nv_bfloat162*>(&lo), *h = reinterpret_cast<__nv_bfloat162*>(&hi);
    const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162*>(&a), *y = reinterpret_cast<const __nv_bfloat162*>(&b);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      l[k] = __hmin2(l[k], x[k]);
      h[k] = __hmax2(h[k], y[k]);
    }
  }
};
template <>
struct PagedLimits<float> {
  static __device__ __forceinline__ void fold(uint4& lo, uint4& hi, const uint4& a, const uint4& b) {
    float *l = reinterpret_cast<float*>(&lo), *h = reinterpret_cast<float*>(&hi);
    const float *x = reinterpret_cast<const float*>(&a), *y = reinterpret_cast<const float*>(&b);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      l[k] = fminf(l[k], x[k]);
      h[k] = fmaxf(h[k], y[k]);
    }
  }
};

__device__ __forceinline__ uint4 shfl_vec(uint4 v, int lane) {
  return make_uint4(__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.y, lane),
                    __shfl_sync(0xffffffffu, v.z, lane), __shfl_sync(0xffffffffu, v.w, lane));
}

// The limits of one head's keys, rows [0, rows) of which NW warps have: a lane vector v of rows r0, r0 + 32 NW / V, ...
// (at least the first row is there).  Writes the page's; `merge`: with what is stored.
template <typename T, int NW>
__device__ __forceinline__ void write_limits(uint4 lo, uint4 hi, int rows, int r0, int v, int V, bool merge, uint4* kmin,
                                             uint4* kmax) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncwarp();
  // lanes without a row take those of the warp's first row (warps without one are left out)
  const int from = r0 < rows ? lane : v;
  lo = shfl_vec(lo, from);
  hi = shfl_vec(hi, from);
  for (int w = V; w < 32; w <<= 1) PagedLimits<T>::fold(lo, hi, shfl_vec(lo, lane ^ w), shfl_vec(hi, lane ^ w));
  if constexpr (NW > 1) {
    __shared__ uint4 s_lo[NW][32], s_hi[NW][32];
    if (lane < V) {
      s_lo[warp][lane] = lo;
      s_hi[warp][lane] = hi;
    }
    __syncthreads();
    if (warp == 0 && lane < V)
      for (int w = 1; w < NW && w * 32 / V < rows; ++w) PagedLimits<T>::fold(lo, hi, s_lo[w][lane], s_hi[w][lane]);
  }
  if (r0 == 0) {
    if (merge) PagedLimits<T>::fold(lo, hi, kmin[v], kmax[v]);
    kmin[v] = lo;
    kmax[v] = hi;
  }
}

constexpr int kWriteThreads = 128, kWriteUnroll = 4;
constexpr int kWriteWide = 512;  // vectors of a page's head from which a CTA writes it

// WPP warps (one, or the CTA's four) write the new tokens of one page and KV head: four 16-byte vectors of K and of V
// a lane in flight, the page's min/max by shuffles (and through shared memory).  Four prompts of 32k tokens of 8 heads,
// with min/max, a warp or a CTA each: 154 and 331 us on pages of 16 tokens at D = 128, 83 and 297 at D = 64; 152.6 and 149.8 on
// pages of 32 at D = 128, 155 and 151 on pages of 64 (floors 146 to 150, 75 at D = 64).  CTAs of eight warps: 153.5
// on pages of 64, 150 for 155 on pages of 256.
template <typename T, int WPP>
__global__ void __launch_bounds__(kWriteThreads)
paged_write_kernel(const Paged c, const PagedNew nw, int Hkv, int Cap, int D, int pshift) {
  constexpr int U = kWriteUnroll, E = Vec16<T>::N, NW = kWriteThreads / 32;
  static_assert(WPP == 1 || WPP == NW, "a page is a warp's or the CTA's, so that returns are uniform");
  pdl_wait_then_release();
  const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t unit = WPP == 1 ? blockIdx.x * NW + warp : blockIdx.x;
  const int h = unit % (uint32_t)Hkv;
  const int2 span = paged_spans(c)[b];
  const int64_t l = (span.x >> pshift) + (int64_t)(unit / (uint32_t)Hkv);
  if (span.y == 0 || l > (span.x + span.y - 1) >> pshift) return;
  const int page = c.table[(size_t)b * (Cap >> pshift) + l];
  if (!paged_page(page, c.pages)) return;
  const int P = 1 << pshift, t0 = max((int)l << pshift, span.x), rows = min(((int)l + 1) << pshift, span.x + span.y) - t0;
  // vectors of a token; the lane's, and its first row
  const int V = D / E, v = lane % V, r0 = ((WPP == 1 ? 0 : warp * 32) + lane) / V, step = 32 * WPP / V;
  const size_t at = (((size_t)page * Hkv + h) * P + (t0 & (P - 1))) * V + v;
  uint4 *kd = static_cast<uint4*>(c.k) + at, *vd = static_cast<uint4*>(c.v) + at;
  const T* ks = static_cast<const T*>(nw.k) + b * nw.kb + (int64_t)(t0 - span.x) * nw.kt + h * nw.kh + v * E;
  const T* vs = static_cast<const T*>(nw.v) + b * nw.vb + (int64_t)(t0 - span.x) * nw.vt + h * nw.vh + v * E;
  uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
  for (int r = r0; r < rows; r += step * U) {
    uint4 k[U], x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r + u * step < rows) {
        k[u] = ldg_stream(ks + (r + u * step) * nw.kt);
        x[u] = ldg_stream(vs + (r + u * step) * nw.vt);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r + u * step < rows) {
        kd[(r + u * step) * V] = k[u];
        vd[(r + u * step) * V] = x[u];
        if (c.kmin) {
          if (r == r0 && u == 0) lo = hi = k[u];
          else PagedLimits<T>::fold(lo, hi, k[u], k[u]);
        }
      }
  }
  if (!c.kmin) return;
  const size_t m = ((size_t)page * Hkv + h) * V;
  write_limits<T, WPP>(lo, hi, rows, r0, v, V, (t0 & (P - 1)) != 0, static_cast<uint4*>(c.kmin) + m,
                       static_cast<uint4*>(c.kmax) + m);
}

template <typename T>
static cudaError_t write_launch(const Shape& s, const Paged& c, const PagedNew& n, cudaStream_t st) {
  constexpr int NW = kWriteThreads / 32;
  const int most = std::min(n.max_new, s.Cap);  // more tokens fit no sequence
  const int64_t units = ((int64_t)(most - 1 + s.P - 1) / s.P + 1) * s.Hkv;  // pages and heads of a sequence
  if (s.P * (s.D / Vec16<T>::N) >= kWriteWide)
    return launch_pdl(paged_write_kernel<T, NW>, dim3((unsigned)units, s.B), dim3(kWriteThreads), 0, st, c, n, s.Hkv, s.Cap, s.D,
                      s.pshift);
  return launch_pdl(paged_write_kernel<T, 1>, dim3((unsigned)((units + NW - 1) / NW), s.B), dim3(kWriteThreads), 0, st, c, n,
                    s.Hkv, s.Cap, s.D, s.pshift);
}

// One token of every sequence in one launch: each CTA plans for itself and writes its share of the vectors, and the
// last one to have read what was records what changes (32 sequences: 7.0 us in two launches, 5.9 in this one, 8.7 in one
// launch of a cluster of eight CTAs of 1024 threads).
constexpr int kOnePerSm = 2;  // CTAs that plan, at most

template <typename T>
__global__ void __launch_bounds__(kPlanFew)
paged_append_one_kernel(const Paged c, const PagedNew nw, int32_t* pos_out, int Hkv, int B, int Cap, int D, int pshift) {
  constexpr int E = Vec16<T>::N, NT = kPlanFew;
  __shared__ PlanShared<NT> sh;
  __shared__ int s_first[NT * kPlanMost], s_had[NT * kPlanMost], s_slot[NT * kPlanMost], s_page[NT * kPlanMost], s_total;
  const int V = D / E, per = Hkv * V, all = B * per, tid = threadIdx.x, MP = Cap >> pshift, P = 1 << pshift;
  pdl_wait_then_release();
  const int first = c.state[1];
  // the thread's first vectors, in flight with the plan
  const int i0 = blockIdx.x * NT + tid;
  auto load = [&](const void* src, int64_t sb, int64_t sh2, int i) {
    return i < all ? ldg_stream(static_cast<const T*>(src) + i / per * sb + i % per / V * sh2 + i % V * E) : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 k = load(nw.k, nw.kb, nw.kh, i0), x = load(nw.v, nw.vb, nw.vh, i0);
  AppendPlan p;
  const int total = append_plan<NT>(c, nw.new_len, 1, B, Cap, pshift, blockIdx.x == 0, p, s_first, s_had, &s_total, sh);
#pragma unroll
  for (int i = 0; i < kPlanMost; ++i)
    if (p.b0 + i < p.b1) {
      s_page[p.b0 + i] = p.n[i] ? p.page[i] : -1;
      s_slot[p.b0 + i] = p.n[i] ? p.start[i] : -1;
    }
  __syncthreads();
  if (total)
    find_pages<NT, false>(c, first, total, sh, [&](int r, int page) { s_page[append_taker(s_first, B, r)] = page; });
  const bool last = last_to_arrive(c, gridDim.x);
  for (int i = i0; i < all; i += gridDim.x * NT) {
    if (i != i0) {
      k = load(nw.k, nw.kb, nw.kh, i);
      x = load(nw.v, nw.vb, nw.vh, i);
    }
    const int b = i / per, h = i % per / V, v = i % V, at = s_slot[b];
    if (at < 0 || !paged_page(s_page[b], c.pages)) continue;
    const size_t row = (size_t)s_page[b] * Hkv + h, to = (row * P + (at & (P - 1))) * V + v;
    static_cast<uint4*>(c.k)[to] = k;
    static_cast<uint4*>(c.v)[to] = x;
    if (c.kmin) {
      uint4 *kmin = static_cast<uint4*>(c.kmin) + row * V + v, *kmax = static_cast<uint4*>(c.kmax) + row * V + v, lo = k, hi = k;
      if (at & (P - 1)) PagedLimits<T>::fold(lo, hi, *kmin, *kmax);
      *kmin = lo;
      *kmax = hi;
    }
  }
  if (!last) return;
  append_record(c, p, pos_out);
#pragma unroll
  for (int i = 0; i < kPlanMost; ++i) {
    const int b = p.b0 + i;
    if (b >= p.b1 || !p.n[i] || p.page[i] >= 0 || !paged_page(s_page[b], c.pages)) continue;
    c.table[(size_t)b * MP + s_had[b]] = s_page[b];
    c.refs[s_page[b]] = 1;
  }
  if (total) find_pages<NT, true>(c, first, total, sh, [](int, int) {});
}

cudaError_t launch_paged_append(const Shape& s, const Paged& c, const PagedNew& n, int32_t* pos_out, cudaStream_t st) {
  cudaError_t e;
  const bool few = s.B <= kPlanFew * kPlanMost;
  const int64_t vecs = (int64_t)s.B * s.Hkv * s.D * (s.dtype == 0 ? 4 : 2) / 16;
  if (n.max_new == 1 && few && vecs <= (int64_t)kPlanFew * 4 * kOnePerSm * sm_count()) {
    const dim3 grid((unsigned)std::min<int64_t>((vecs + kPlanFew - 1) / kPlanFew, kOnePerSm * sm_count()));
    e = s.dtype == 0 ? launch_pdl(paged_append_one_kernel<float>, grid, dim3(kPlanFew), 0, st, c, n, pos_out, s.Hkv, s.B, s.Cap,
                                  s.D, s.pshift)
                     : launch_pdl(paged_append_one_kernel<bf16>, grid, dim3(kPlanFew), 0, st, c, n, pos_out, s.Hkv, s.B, s.Cap,
                                  s.D, s.pshift);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  // 1024 threads where there are many pages to give as well (16 prompts of one head of 64 channels that take 32768 pages:
  // 78 us with 256, 56 with 1024)
  const bool quick = few && (int64_t)s.B * (std::min(n.max_new, s.Cap) / s.P + 1) <= kPlanPages;
  e = quick ? launch_pdl(paged_plan_kernel<kPlanFew>, dim3(1), dim3(kPlanFew), 0, st, c, n.new_len, n.max_new, pos_out, s.B, s.Cap,
                         s.pshift)
            : launch_pdl(paged_plan_kernel<kPlanThreads>, dim3(1), dim3(kPlanThreads), 0, st, c, n.new_len, n.max_new, pos_out,
                         s.B, s.Cap, s.pshift);
  if (e == cudaSuccess && n.max_new > 0) e = s.dtype == 0 ? write_launch<float>(s, c, n, st) : write_launch<bf16>(s, c, n, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ------------------------------------------------------------------- fork

// What becomes of sequence b: row `parent` (-1: nothing) cut to `len` tokens.
struct ForkPlan {
  int parent, len, was;
  bool same, bad;
};
__device__ __forceinline__ ForkPlan fork_plan(const PagedFork& f, const int32_t* ctx, int b, int B, int Cap) {
  ForkPlan p;
  p.parent = f.parent[b];
  p.was = clamp_len(ctx[b], Cap);
  p.bad = p.parent < -1 || p.parent >= B;
  if (p.bad) p.parent = b;
  p.len = p.parent < 0 ? 0 : clamp_len(ctx[p.parent], Cap);
  if (f.keep && !p.bad) p.len = min(p.len, max(f.keep[b], 0));
  p.same = p.bad || (p.parent == b && p.len == p.was) || (p.len == 0 && p.was == 0);
  return p;
}

// Entry l of a changed sequence before and after: pages it lets go (or -1) and pages it takes over whole.
// Entries that stay are neither.
__device__ __forceinline__ void fork_entry(const Paged& c, const ForkPlan& p, int b, int l, int MP, int pshift, int& old,
                                           int& now) {
  const int P = 1 << pshift;
  old = l < (p.was + P - 1) >> pshift ? c.table[(size_t)b * MP + l] : -1;
  now = l < p.len >> pshift ? (p.parent == b ? old : c.table[(size_t)p.parent * MP + l]) : -1;
}

// Counts of pages as after the fork, but for the partial pages of changed sequences.
// Threads first, first + step, ... of sequence b.
__device__ __forceinline__ void fork_count(const Paged& c, const PagedFork& f, int b, int B, int Cap, int pshift, int first,
                                           int step) {
  const int MP = Cap >> pshift;
  const ForkPlan p = fork_plan(f, c.ctx, b, B, Cap);
  if (p.same) {
    if (p.bad && first == 0) note_bad_pages(1);
    return;
  }
  const int last = max((p.was + (1 << pshift) - 1) >> pshift, (p.len >> pshift) + 1);
  for (int l = first; l < min(last, MP); l += step) {
    int old, now;
    fork_entry(c, p, b, l, MP, pshift, old, now);
    if (old != now) {
      if (paged_page(old, c.pages)) atomicAdd(c.refs + old, -1);
      if (paged_page(now, c.pages)) atomicAdd(c.refs + now, 1);
    }
    // a partial last page: its source for now
    if (l == p.len >> pshift && (p.len & ((1 << pshift) - 1))) now = c.table[(size_t)p.parent * MP + l];
    f.rows[(size_t)b * MP + l] = now;
  }
}

// Who keeps, and who copies, a partial page; the pages for the copies; the new lengths.
template <int NT>
__device__ __forceinline__ void fork_choose(const Paged& c, const PagedFork& f, int B, int Cap, int pshift) {
  constexpr int MOST = kPlanMost;
  __shared__ PlanShared<NT> sh;
  __shared__ int s_copy[NT * MOST];
  const int tid = threadIdx.x, MP = Cap >> pshift, free = c.state[0], lowest = c.state[1];
  const int per = (B + NT - 1) / NT, b0 = min(tid * per, B), b1 = min(b0 + per, B);
  ForkPlan p[MOST];
  int src[MOST];
  bool held[MOST];
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    const int b = b0 + i;
    src[i] = -1;
    held[i] = false;
    if (b >= b1) continue;
    p[i] = fork_plan(f, c.ctx, b, B, Cap);
    if (!p[i].same && (p[i].len & ((1 << pshift) - 1))) {
      src[i] = f.rows[(size_t)b * MP + (p[i].len >> pshift)];
      if (!paged_page(src[i], c.pages)) {
        src[i] = -1;
        note_bad_pages(1);
      } else {
        held[i] = c.refs[src[i]] > 0;
      }
    }
  }
  __syncthreads();
  // a page that nobody holds whole: its lowest user keeps it, found by its number (below zero) in the page's count
  constexpr int kBelow = 1 << 30;
#pragma unroll
  for (int i = 0; i < MOST; ++i)
    if (src[i] >= 0 && !held[i]) atomicMin(c.refs + src[i], b0 + i - kBelow);
  __syncthreads();
  int copies = 0;
  bool copy[MOST];
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    copy[i] = src[i] >= 0 && (held[i] || __ldcg(c.refs + src[i]) != b0 + i - kBelow);
    copies += copy[i];
  }
  int total;
  int rank = plan_scan<NT>(copies, sh.tmp, total);
  const bool fail = total > free;
  if (tid == 0) {
    c.state[2] = fail;
    if (f.done) *f.done = !fail;
  }
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    const int b = b0 + i;
    if (b >= b1) continue;
    const int part = src[i] < 0 ? 0 : p[i].len & ((1 << pshift) - 1);
    f.copy[b] = make_int4(src[i], src[i], part, p[i].same ? -1 : p[i].was);
    if (p[i].same) continue;
    if (src[i] >= 0 && !copy[i]) c.refs[src[i]] = !fail;
    if (fail) continue;
    c.ctx[b] = p[i].len;
    if (copy[i]) s_copy[rank++] = b;
  }
  __syncthreads();
  if (fail || total == 0) return;
  find_pages<NT, true>(c, lowest, total, sh, [&](int r, int page) {
    const int b = s_copy[r];
    f.copy[b].y = page;
    f.rows[(size_t)b * MP + (c.ctx[b] >> pshift)] = page;
    c.refs[page] = 1;
  });
}

// New rows into the table, and pages that nobody holds any more freed.  Where the pool lacked pages:
// the counts as they were.
__device__ __forceinline__ void fork_commit(const Paged& c, const PagedFork& f, int b, int B, int Cap, int pshift, int first,
                                            int step) {
  const int MP = Cap >> pshift, P = 1 << pshift, was = f.copy[b].w;
  if (was < 0) return;
  if (c.state[2] != 0) {
    const ForkPlan p = fork_plan(f, c.ctx, b, B, Cap);
    const int last = max((p.was + P - 1) >> pshift, (p.len >> pshift) + 1);
    for (int l = first; l < min(last, MP); l += step) {
      int old, now;
      fork_entry(c, p, b, l, MP, pshift, old, now);
      if (old != now) {
        if (paged_page(old, c.pages)) atomicAdd(c.refs + old, 1);
        if (paged_page(now, c.pages)) atomicAdd(c.refs + now, -1);
      }
    }
    return;
  }
  const int had = (was + P - 1) >> pshift, has = (c.ctx[b] + P - 1) >> pshift;
  for (int l = first; l < max(had, has); l += step) {
    const int old = l < had ? c.table[(size_t)b * MP + l] : -1, now = l < has ? f.rows[(size_t)b * MP + l] : -1;
    if (old == now) continue;
    c.table[(size_t)b * MP + l] = now;
    if (paged_page(old, c.pages) && c.refs[old] == 0) {
      const uint32_t bit = 1u << (old & 31);
      if (!(atomicOr(paged_bits(c) + (old >> 5), bit) & bit)) {
        atomicAdd(c.state, 1);
        atomicMin(c.state + 1, old >> 5);
      }
    }
  }
}

// Head h of the partial page of sequence b copied, and summarised anew, by the CTA (a thread for all rows of a vector:
// 33 us for 32 beams on pages of 256 tokens, this 12).
constexpr int kForkThreads = 256;
template <typename T>
__device__ __forceinline__ void fork_copy(const Paged& c, const PagedFork& f, int b, int h, int Hkv, int D, int pshift) {
  constexpr int NW = kForkThreads / 32, U = 4;
  const int4 cp = f.copy[b];
  if (cp.w < 0 || cp.z == 0 || c.state[2] != 0) return;
  const bool copy = cp.x != cp.y;
  if (!copy && !c.kmin) return;
  const int V = D / Vec16<T>::N, v = threadIdx.x % V, r0 = threadIdx.x / V, step = kForkThreads / V;
  const size_t from = ((((size_t)cp.x * Hkv + h) << pshift) * V) + v, to = ((((size_t)cp.y * Hkv + h) << pshift) * V) + v;
  const uint4 *ks = static_cast<const uint4*>(c.k) + from, *vs = static_cast<const uint4*>(c.v) + from;
  uint4 *kd = static_cast<uint4*>(c.k) + to, *vd = static_cast<uint4*>(c.v) + to;
  uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
  for (int r = r0; r < cp.z; r += step * U) {
    uint4 k[U], x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r + u * step < cp.z) {
        k[u] = ks[(r + u * step) * V];
        if (copy) x[u] = vs[(r + u * step) * V];
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r + u * step < cp.z) {
        if (copy) {
          kd[(r + u * step) * V] = k[u];
          vd[(r + u * step) * V] = x[u];
        }
        if (r == r0 && u == 0) lo = hi = k[u];
        else PagedLimits<T>::fold(lo, hi, k[u], k[u]);
      }
  }
  if (!c.kmin) return;
  const size_t m = ((size_t)cp.y * Hkv + h) * V;
  write_limits<T, NW>(lo, hi, cp.z, r0, v, V, false, static_cast<uint4*>(c.kmin) + m, static_cast<uint4*>(c.kmax) + m);
}

// CTAs of a sequence in the steps over table rows: enough for a thread an entry, up to eight CTAs an SM in all
// (their arrivals are counted one by one).
static int fork_shares(int B, int pages, int nt) {
  return std::max(1, std::min((pages + nt - 1) / nt, 8 * sm_count() / B));
}

// The counts, and, by the last CTA, the choice (as a launch of its own: 0.6 us more).  All three steps in one
// launch of a cluster were slower: its eight CTAs took 14 us for 32 beams and 24 for 48 prompts' prefixes.
template <int NT>
__global__ void __launch_bounds__(NT)
fork_count_kernel(const Paged c, const PagedFork f, int B, int Cap, int pshift) {
  pdl_wait_then_release();
  fork_count(c, f, blockIdx.y, B, Cap, pshift, blockIdx.x * NT + threadIdx.x, gridDim.x * NT);
  if (last_to_arrive(c, gridDim.x * gridDim.y)) fork_choose<NT>(c, f, B, Cap, pshift);
}

template <typename T>
__global__ void __launch_bounds__(kForkThreads)
fork_commit_kernel(const Paged c, const PagedFork f, int Hkv, int B, int Cap, int D, int pshift, int chunks) {
  pdl_wait_then_release();
  const int b = blockIdx.y;
  if ((int)blockIdx.x < chunks) fork_commit(c, f, b, B, Cap, pshift, blockIdx.x * kForkThreads + threadIdx.x, chunks * kForkThreads);
  else fork_copy<T>(c, f, b, blockIdx.x - chunks, Hkv, D, pshift);
}

size_t paged_fork_workspace(const Shape& s) {
  return (size_t)s.B * sizeof(int4) + (size_t)s.B * (s.Cap >> s.pshift) * sizeof(int32_t);
}

cudaError_t launch_paged_fork(const Shape& s, const Paged& c, const int32_t* parent, const int32_t* keep, int32_t* done,
                              void* ws, cudaStream_t st) {
  PagedFork f = {parent, keep, done, static_cast<int4*>(ws), nullptr};
  f.rows = reinterpret_cast<int32_t*>(f.copy + s.B);
  const int MP = s.Cap >> s.pshift;
  cudaError_t e;
  const int nt = s.B <= kPlanFew * kPlanMost ? kPlanFew : kPlanThreads, shares = fork_shares(s.B, MP, nt);
  e = nt == kPlanFew ? launch_pdl(fork_count_kernel<kPlanFew>, dim3(shares, s.B), dim3(nt), 0, st, c, f, s.B, s.Cap, s.pshift)
                     : launch_pdl(fork_count_kernel<kPlanThreads>, dim3(shares, s.B), dim3(nt), 0, st, c, f, s.B, s.Cap, s.pshift);
  if (e == cudaSuccess) {
    const int chunks = fork_shares(s.B, MP, kForkThreads);
    const dim3 grid(chunks + s.Hkv, s.B);
    e = s.dtype == 0 ? launch_pdl(fork_commit_kernel<float>, grid, dim3(kForkThreads), 0, st, c, f, s.Hkv, s.B, s.Cap, s.D, s.pshift, chunks)
                     : launch_pdl(fork_commit_kernel<bf16>, grid, dim3(kForkThreads), 0, st, c, f, s.Hkv, s.B, s.Cap, s.D, s.pshift, chunks);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ------------------------------------------------------------------- compaction

// The i-th free page below U (the number of used pages) receives the i-th used one from U on:
// holes[i], movers[i], and rank[p] = i of a mover p.  A CTA takes `per` words of the bits and counts what lies
// before them: 64 words, or a 128th of the map where that is more (one CTA for 32768 pages takes 12 us).
constexpr int kCompactWords = 64, kCompactCtas = 128;

__global__ void __launch_bounds__(kPlanFew)
compact_plan_kernel(const Paged c, const PagedCompact m, int per) {
  constexpr int NT = kPlanFew;
  __shared__ PlanShared<NT> sh;
  pdl_wait_then_release();
  const uint32_t* bits = paged_bits(c);
  const int words = paged_words(c.pages), tid = threadIdx.x, lane = tid & 31, U = c.pages - c.state[0];
  const int w0 = blockIdx.x * per, w1 = min(w0 + per, words);
  int before = 0, below = 0, all, holes;
  // free pages before this CTA's words, and below page U
#pragma unroll 4
  for (int w = tid; w < min(max(w0, (U >> 5) + 1), words); w += NT) {
    const uint32_t x = bits[w];
    if (w < w0) before += __popc(x);
    if (w < U >> 5) below += __popc(x);
    else if (w == U >> 5) below += __popc(x & ((1u << (U & 31)) - 1u));
  }
  plan_scan<NT>(before, sh.tmp, all);
  before = all;
  plan_scan<NT>(below, sh.tmp, holes);
  if (blockIdx.x == 0 && tid == 0) *m.count = holes;
  for (int w = w0; w < w1; w += NT) {
    const uint32_t word = w + tid < w1 ? bits[w + tid] : 0u;
    const int base = before + plan_scan<NT>(__popc(word), sh.tmp, all);
    sh.word[tid] = word;
    sh.base[tid] = base;
    before += all;
    __syncthreads();
    for (int i = tid >> 5; i < min(NT, w1 - w); i += NT / 32) {
      const int p = (w + i) * 32 + lane;
      if (p >= c.pages) continue;
      const int f = sh.base[i] + __popc(sh.word[i] & ((1u << lane) - 1u));  // free pages below p
      const bool free = sh.word[i] >> lane & 1u;
      if (free) {
        if (p < U) m.holes[f] = p;
      } else if (p >= U) {
        const int r = p - U - (f - holes);
        m.movers[r] = p;
        m.rank[p] = r;
      }
      if (m.moved) m.moved[p] = free ? -1 : p;  // movers: below
    }
  }
}

constexpr int kMoveThreads = 256, kMoveUnroll = 4, kMovePerSm = 8;

// Copies the movers (a warp: 2 KB of a page's K and of its V, all loads in flight); the first eighth of the
// CTAs renames pages in the table and writes the bits anew before that, while the others copy.  Eight CTAs an SM: 90.4
// us for the pool above, 92 with two, 95 with four (through the read-only path; 87 with plain loads); 250 small pages 6.7 us, 8.1
// with the renaming at the end.
__global__ void __launch_bounds__(kMoveThreads)
compact_move_kernel(const Paged c, const PagedCompact m, int64_t page_vecs, int64_t meta_vecs, int B, int Cap, int pshift) {
  constexpr uint32_t NT = kMoveThreads, U = kMoveUnroll;
  pdl_wait_then_release();
  const int count = *m.count, used = c.pages - c.state[0], lane = threadIdx.x & 31;
  const uint32_t renamers = (gridDim.x + 7) / 8;
  if (blockIdx.x < renamers) {
    const int64_t tid = (int64_t)blockIdx.x * NT + threadIdx.x, all = (int64_t)renamers * NT;
    if (meta_vecs)
      for (int64_t x = tid; x < count * meta_vecs; x += all) {
        const int64_t i = x / meta_vecs, at = x % meta_vecs, from = m.movers[i] * meta_vecs + at, to = m.holes[i] * meta_vecs + at;
        static_cast<uint4*>(c.kmin)[to] = static_cast<const uint4*>(c.kmin)[from];
        static_cast<uint4*>(c.kmax)[to] = static_cast<const uint4*>(c.kmax)[from];
      }
    for (int64_t x = tid; x < count; x += all) {
      const int from = m.movers[x], to = m.holes[x];
      c.refs[to] = c.refs[from];
      c.refs[from] = 0;
      if (m.moved) m.moved[from] = to;
    }
    const int MP = Cap >> pshift;
    for (int64_t x = tid; x < (int64_t)B * MP; x += all) {
      const int p = c.table[x];
      if (p >= used && p < c.pages) {
        const int r = m.rank[p];
        if ((unsigned)r < (unsigned)count) c.table[x] = m.holes[r];
      }
    }
    for (int64_t w = tid; w < paged_words(c.pages); w += all) {
      uint32_t x = (w + 1) * 32 <= used ? 0u : w * 32 >= used ? 0xffffffffu : 0xffffffffu << (used & 31);
      if (w == c.pages >> 5) x &= (1u << (c.pages & 31)) - 1u;
      paged_bits(c)[w] = x;
    }
    if (tid == 0) c.state[1] = min(used >> 5, paged_words(c.pages) - 1);
  }
  // a page is whole units: 16 tokens of 64 channels in 2 bytes are one; the pool has less than 2^31 rows, so
  // fewer units
  const uint32_t parts = (uint32_t)(page_vecs / (32 * U)), units = (uint32_t)count * parts, warps = gridDim.x * (NT / 32);
  for (uint32_t x = blockIdx.x * (NT / 32) + (threadIdx.x >> 5); x < units; x += warps) {
    const uint32_t i = x / parts;
    const int64_t at = (int64_t)(x % parts) * 32 * U + lane, from = m.movers[i] * page_vecs + at, to = m.holes[i] * page_vecs + at;
    uint4 k[U], v[U];
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
      k[u] = ldg_stream(static_cast<const uint4*>(c.k) + from + 32 * u);
      v[u] = ldg_stream(static_cast<const uint4*>(c.v) + from + 32 * u);
    }
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
      static_cast<uint4*>(c.k)[to + 32 * u] = k[u];
      static_cast<uint4*>(c.v)[to + 32 * u] = v[u];
    }
  }
}

size_t paged_compact_workspace(const Paged& c) { return 16 + 3 * (size_t)((c.pages + 3) & ~3) * sizeof(int32_t); }

cudaError_t launch_paged_compact(const Shape& s, const Paged& c, int32_t* moved, void* ws, cudaStream_t st) {
  const size_t n = (size_t)((c.pages + 3) & ~3);
  PagedCompact m = {};
  m.count = static_cast<int32_t*>(ws);
  m.holes = m.count + 4;
  m.movers = m.holes + n;
  m.rank = m.movers + n;
  m.moved = moved;
  const int size = s.dtype == 0 ? 4 : 2;
  const int64_t meta_vecs = (int64_t)s.Hkv * s.D * size / 16, page_vecs = meta_vecs * s.P;
  const int words = paged_words(c.pages), per = std::max(kCompactWords, (words + kCompactCtas - 1) / kCompactCtas);
  cudaError_t e = launch_pdl(compact_plan_kernel, dim3((words + per - 1) / per), dim3(kPlanFew), 0, st, c, m, per);
  if (e == cudaSuccess)
    e = launch_pdl(compact_move_kernel, dim3(sm_count() * kMovePerSm), dim3(kMoveThreads), 0, st, c, m, page_vecs,
                   c.kmin ? meta_vecs : 0, s.B, s.Cap, s.pshift);
  return e != cudaSuccess ? e : cudaGetLastError();
}

DeviceStatus take_status_paged_cache() { return take_status_here(); }

}  // namespace sls
