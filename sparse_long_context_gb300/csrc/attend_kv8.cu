// Decode attention over the 8-bit cache: split-K online softmax, a CTA per
// (row, slice of its token groups), then the merge of a row's slices.
#include <algorithm>

#include "attend_common.cuh"
#include "kv8.cuh"
#include "launch.h"

namespace sls {

struct Kv8Attend {
  Kv8 c;
  const bf16* q;
  const int32_t *page_idx, *count, *ctx_len;
  int idx_stride, k_fixed, S, Hq, Hkv, G, Cap, P, pshift;
  float qscale;  // softmax scale * log2(e)
  const float* sink;
  bf16* out;
  float* lse;
  float *po, *pm, *pl;  // [B, Hq, S] partials
  float2* grp;          // [rows, Cap/16, G] weight sums of 16-token groups and the max they are relative to, or null
  float2* fin;          // [B, Hq] final max (base 2) and 1 / sum, or null
  const float* mass_in;
  float* mass_out;
};

// Number of 16-token groups of a row (list entries of P >= 16 tokens each, or
// the whole context).
__device__ __forceinline__ int kv8_groups(const Kv8Attend& a, int row, int N) {
  if (!a.page_idx) return (N + 15) >> 4;
  const int cnt = a.count ? a.count[row] : a.k_fixed;
  return min(max(cnt, 0), a.idx_stride) << (a.pshift - 4);
}

template <int D, int FMT>
__global__ void __launch_bounds__(256)
kv8_attend_kernel(const Kv8Attend a) {
  pdl_wait_then_release();
  constexpr int E = D / 32;
  const int row = blockIdx.x / a.S, split = blockIdx.x % a.S, b = row / a.Hkv, h = row % a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int N = clamp_len(a.ctx_len[b], a.Cap);
  const int ng = kv8_groups(a, row, N), per = (ng + a.S - 1) / a.S;
  const int g0 = min(split * per, ng), g1 = min(g0 + per, ng);
  const int32_t* list = a.page_idx ? a.page_idx + (size_t)row * a.idx_stride : nullptr;
  if (list && warp == 0) {
    unsigned bad = 0;
    for (int e = (g0 >> (a.pshift - 4)) + lane; e < (g1 + (a.P >> 4) - 1) >> (a.pshift - 4); e += 32)
      bad += ((e << (a.pshift - 4)) >= g0) && bad_page_id(list[e], a.Cap >> a.pshift) ? 1u : 0u;
    note_bad_pages(bad);
  }
  float q[8][E], o[8][E], m[8], l[8];
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    m[g] = kNegInf;
    l[g] = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      o[g][i] = 0.f;
      q[g][i] = g < a.G ? to_f32(a.q[((size_t)b * a.Hq + h * a.G + g) * D + lane * E + i]) * a.qscale : 0.f;
    }
  }
  const int newest = N >> a.c.bshift;
  for (int gi = g0 + warp; gi < g1; gi += 8) {
    int base = gi << 4;
    if (list) {
      const int pg = list[base >> a.pshift];
      if ((unsigned)pg >= (unsigned)(a.Cap >> a.pshift)) continue;
      base = (pg << a.pshift) + (base & (a.P - 1));
    }
    const int lim = min(16, N - base);
    if (lim <= 0) continue;
    const int blk = base >> a.c.bshift;
    const bool stored = blk < newest;
    const size_t sc = (size_t)row * (a.Cap >> a.c.bshift) + blk;
    const float ks = stored ? a.c.ks[sc] : 1.f, vs = stored ? a.c.vs[sc] : 1.f;
    float gsum[8], gmax[8];
#pragma unroll
    for (int g = 0; g < 8; ++g) { gsum[g] = 0.f; gmax[g] = kNegInf; }
    for (int t = 0; t < lim; ++t) {
      const int pos = base + t;
      float k[E], v[E];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (stored) {
          const size_t at = ((size_t)row * a.Cap + pos) * D + lane * E + i;
          k[i] = kv8_value<FMT>(a.c.kc[at]) * ks;
          v[i] = kv8_value<FMT>(a.c.vc[at]) * vs;
        } else {
          const size_t at = ((size_t)row * a.c.block + (pos & (a.c.block - 1))) * D + lane * E + i;
          k[i] = to_f32(static_cast<const bf16*>(a.c.kt)[at]);
          v[i] = to_f32(static_cast<const bf16*>(a.c.vt)[at]);
        }
      }
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        if (g >= a.G) break;
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) x = fmaf(q[g][i], k[i], x);
        x = warp_sum(x);
        const float mn = fmaxf(m[g], x);
        const float al = mn == kNegInf ? 1.f : exp2f(m[g] - mn), p = x == kNegInf ? 0.f : exp2f(x - mn);
        m[g] = mn;
        l[g] = l[g] * al + p;
        gsum[g] = gsum[g] * al + p;
        gmax[g] = mn;
#pragma unroll
        for (int i = 0; i < E; ++i) o[g][i] = fmaf(o[g][i], al, p * v[i]);
      }
    }
    if (a.grp && stored && lane == 0)
      for (int g = 0; g < a.G; ++g)
        a.grp[((size_t)row * (a.Cap >> 4) + (base >> 4)) * a.G + g] = make_float2(gsum[g], gmax[g]);
  }
  __shared__ float sm[8][8], sl[8][8], so[8][8][D];
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    if (lane == 0) { sm[warp][g] = m[g]; sl[warp][g] = l[g]; }
#pragma unroll
    for (int i = 0; i < E; ++i) so[warp][g][lane * E + i] = o[g][i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.G * D; i += 256) {
    const int g = i / D, d = i % D;
    float M = kNegInf, L = 0.f, O = 0.f;
    for (int w = 0; w < 8; ++w) M = fmaxf(M, sm[w][g]);
    for (int w = 0; w < 8; ++w) {
      const float f = sm[w][g] == kNegInf ? 0.f : exp2f(sm[w][g] - M);
      L = fmaf(sl[w][g], f, L);
      O = fmaf(so[w][g][d], f, O);
    }
    const size_t at = ((size_t)b * a.Hq + h * a.G + g) * a.S + split;
    a.po[at * D + d] = O;
    if (d == 0) { a.pm[at] = M; a.pl[at] = L; }
  }
}

template <int D>
__global__ void __launch_bounds__(D)
kv8_combine_kernel(const Kv8Attend a) {
  pdl_wait_then_release();
  const int hq = blockIdx.x, d = threadIdx.x;  // b * Hq + head
  const float sk = a.sink ? a.sink[hq % a.Hq] * kLog2e : kNegInf;
  float M = sk, L = 0.f, O = 0.f;
  for (int s = 0; s < a.S; ++s) M = fmaxf(M, a.pm[(size_t)hq * a.S + s]);
  for (int s = 0; s < a.S; ++s) {
    const size_t at = (size_t)hq * a.S + s;
    const float f = a.pm[at] == kNegInf ? 0.f : exp2f(a.pm[at] - M);
    L = fmaf(a.pl[at], f, L);
    O = fmaf(a.po[at * D + d], f, O);
  }
  if (a.sink && M != kNegInf) L += exp2f(sk - M);
  a.out[(size_t)hq * D + d] = __float2bfloat16_rn(L == 0.f ? 0.f : O / L);
  if (d == 0) {
    if (a.lse) a.lse[hq] = L == 0.f ? kNegInf : M * kLn2 + logf(L);
    if (a.fin) a.fin[hq] = make_float2(M, L == 0.f ? 0.f : 1.f / L);
  }
}

__global__ void __launch_bounds__(128)
kv8_mass_kernel(const Kv8Attend a, int per_row) {
  pdl_wait_then_release();
  const int row = blockIdx.x / per_row, blk = (blockIdx.x % per_row) * 128 + threadIdx.x;
  const int b = row / a.Hkv, h = row % a.Hkv;
  if (blk >= clamp_len(a.ctx_len[b], a.Cap) >> a.c.bshift) return;
  float sum = 0.f;
  const int gpb = a.c.block >> 4;
  for (int g = 0; g < a.G; ++g) {
    const float2 f = a.fin[(size_t)b * a.Hq + h * a.G + g];
    for (int i = 0; i < gpb; ++i) {
      const float2 x = a.grp[((size_t)row * (a.Cap >> 4) + blk * gpb + i) * a.G + g];
      if (x.y != kNegInf) sum += x.x * exp2f(x.y - f.x) * f.y;
    }
  }
  const size_t at = (size_t)row * (a.Cap >> a.c.bshift) + blk;
  a.mass_out[at] = (a.mass_in ? a.mass_in[at] : 0.f) + sum;
}

bool kv8_attend_supported(const Shape& s) {
  return s.dtype == 1 && s.B * (long long)s.Hkv <= 4096 && (long long)s.B * s.Hkv * s.Cap < (1ll << 31);
}

static size_t a256(size_t v) { return (v + 255) & ~(size_t)255; }
static int kv8_splits(const Shape& s) {
  return std::max(1, std::min((s.Cap + 511) / 512, 4 * sm_count() / (s.B * s.Hkv) + 1));
}

size_t kv8_attend_workspace(const Shape& s, const Kv8&, bool with_mass) {
  const size_t parts = (size_t)s.B * s.Hq * kv8_splits(s);
  return a256(parts * s.D * 4) + 2 * a256(parts * 4) +
         (with_mass ? a256((size_t)s.B * s.Hkv * (s.Cap / 16 + 1) * s.G * 8) + a256((size_t)s.B * s.Hq * 8) : 0);
}

template <int D>
static cudaError_t kv8_launch(const Kv8Attend& a, int rows, cudaStream_t st) {
  cudaError_t e = a.c.format == kKv8Int8
                      ? launch_pdl(kv8_attend_kernel<D, kKv8Int8>, dim3(rows * a.S), dim3(256), 0, st, a)
                      : launch_pdl(kv8_attend_kernel<D, kKv8E4m3>, dim3(rows * a.S), dim3(256), 0, st, a);
  if (e == cudaSuccess) e = launch_pdl(kv8_combine_kernel<D>, dim3(rows * a.G), dim3(D), 0, st, a);
  if (e == cudaSuccess && a.mass_out) {
    const int per_row = ((a.Cap >> a.c.bshift) + 127) / 128;
    e = launch_pdl(kv8_mass_kernel, dim3((unsigned)rows * per_row), dim3(128), 0, st, a, per_row);
  }
  return e;
}

cudaError_t launch_kv8_attend(const Shape& s, const Kv8& c, const void* q, const int32_t* page_idx, int idx_stride,
                              const int32_t* count, int k_fixed, const int32_t* ctx_len, const float* sink,
                              void* out, float* lse, const float* mass_in, float* mass_out, void* ws,
                              cudaStream_t st) {
  Kv8Attend a = {};
  a.c = c;
  a.q = static_cast<const bf16*>(q);
  a.page_idx = page_idx;
  a.count = count;
  a.ctx_len = ctx_len;
  a.idx_stride = idx_stride;
  a.k_fixed = k_fixed;
  a.S = kv8_splits(s);
  a.Hq = s.Hq; a.Hkv = s.Hkv; a.G = s.G; a.Cap = s.Cap; a.P = s.P; a.pshift = s.pshift;
  a.qscale = s.scale * kLog2e;
  a.sink = sink;
  a.out = static_cast<bf16*>(out);
  a.lse = lse;
  const size_t parts = (size_t)s.B * s.Hq * a.S;
  char* w = static_cast<char*>(ws);
  a.po = reinterpret_cast<float*>(w);
  w += a256(parts * s.D * 4);
  a.pm = reinterpret_cast<float*>(w);
  w += a256(parts * 4);
  a.pl = reinterpret_cast<float*>(w);
  w += a256(parts * 4);
  if (mass_out) {
    a.grp = reinterpret_cast<float2*>(w);
    w += a256((size_t)s.B * s.Hkv * (s.Cap / 16 + 1) * s.G * 8);
    a.fin = reinterpret_cast<float2*>(w);
    a.mass_in = mass_in;
    a.mass_out = mass_out;
  }
  const int rows = s.B * s.Hkv;
  cudaError_t e = s.D == 64 ? kv8_launch<64>(a, rows, st) : kv8_launch<128>(a, rows, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

DeviceStatus take_status_attend_kv8() { return take_status_here(); }

}  // namespace sls
