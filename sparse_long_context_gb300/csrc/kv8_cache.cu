// The 8-bit cache's writers: appending tokens (quantising the blocks they
// complete) and evicting blocks by accumulated attention weight.
#include "common.cuh"
#include "kv8.cuh"
#include "launch.h"

namespace sls {

// Start position and token count of sequence b in an append (count 0 when
// they do not all fit).
struct AppendSpan {
  int start, n;
};
__device__ __forceinline__ AppendSpan append_span(const Kv8New& nw, const int32_t* ctx_len, int b, int Cap) {
  AppendSpan s;
  s.start = clamp_len(ctx_len[b], Cap);
  s.n = nw.new_len ? min(max(nw.new_len[b], 0), nw.max_new) : nw.max_new;
  if (s.n > Cap - s.start) s.n = 0;
  return s;
}

// One CTA per (sequence, KV head, K or V, block touched): the
// block's tokens, the earlier ones from the tail buffer and the new ones from
// the caller, are read twice (largest magnitude, then the codes).  The CTA of
// a sequence's first block also writes its newest, partial block to the
// tail, after its own reads of it.
template <int FMT>
__global__ void __launch_bounds__(256)
kv8_append_kernel(const Kv8 c, const Kv8New nw, float* mass, const int32_t* ctx_len, int Hkv, int Cap, int D,
                  int units) {
  pdl_wait_then_release();
  const int u = blockIdx.x % units, x = blockIdx.x / units;
  const int isv = x & 1, h = (x >> 1) % Hkv, b = (x >> 1) / Hkv;
  const AppendSpan sp = append_span(nw, ctx_len, b, Cap);
  if (sp.n == 0) return;
  const int first = sp.start >> c.bshift, last = (sp.start + sp.n) >> c.bshift;  // `last`: the newest, partial block
  const int j = first + u;
  const int row = b * Hkv + h;
  const bf16* src = static_cast<const bf16*>(isv ? nw.v : nw.k) + b * (isv ? nw.vb : nw.kb) + h * (isv ? nw.vh : nw.kh);
  const int64_t st = isv ? nw.vt : nw.kt;
  bf16* tail = static_cast<bf16*>(isv ? c.vt : c.kt) + (size_t)row * c.block * D;
  const int cpr = D / 8, nvec = c.block * cpr;  // 16-byte vectors of a block
  if (j < last) {
    auto vec = [&](int i) {
      const int t = i / cpr, ch = (i % cpr) * 8, pos = (j << c.bshift) + t;
      const bf16* p = pos < sp.start ? tail + (size_t)t * D + ch : src + (pos - sp.start) * st + ch;
      return *reinterpret_cast<const uint4*>(p);
    };
    __shared__ uint32_t s_max[8];
    uint32_t mx = 0;  // magnitudes as bit patterns: NaN above infinity above the numbers
    for (int i = threadIdx.x; i < nvec; i += 256) {
      const uint4 v = vec(i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) mx = max(mx, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = mx;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) mx = max(mx, s_max[k]);
    const float amax = __uint_as_float(mx << 16);
    const bool finite = mx < 0x7f80u;
    const size_t blk = (size_t)row * (Cap >> c.bshift) + j;
    uint8_t* codes = (isv ? c.vc : c.kc) + blk * c.block * D;
    for (int i = threadIdx.x; i < nvec; i += 256) {
      float x[8];
      unpack_vec(vec(i), x);
      uint32_t w[2] = {0u, 0u};
      if (finite && mx)
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k >> 2] |= kv8_code<FMT>(x[k], amax) << (8 * (k & 3));
      *reinterpret_cast<uint2*>(codes + (size_t)i * 8) = make_uint2(w[0], w[1]);
    }
    if (threadIdx.x == 0) {
      (isv ? c.vs : c.ks)[blk] = finite ? __fdiv_rn(amax, kv8_top<FMT>()) : __int_as_float(0x7fffffff);
      if (mass && !isv) mass[blk] = 0.f;
    }
  }
  if (u == 0) {
    __syncthreads();  // the block just quantised has read the tail
    const int t0 = last == first ? sp.start - (first << c.bshift) : 0;
    const int t1 = (sp.start + sp.n) - (last << c.bshift);
    for (int i = threadIdx.x + t0 * cpr; i < t1 * cpr; i += 256) {
      const int t = i / cpr, ch = (i % cpr) * 8, pos = (last << c.bshift) + t;
      *reinterpret_cast<uint4*>(tail + (size_t)t * D + ch) =
          *reinterpret_cast<const uint4*>(src + (pos - sp.start) * st + ch);
    }
  }
}

// Page min/max of the new keys: one CTA per (page touched, KV head, sequence).
__global__ void __launch_bounds__(128)
kv8_pagemeta_kernel(const Kv8New nw, bf16* kmin, bf16* kmax, const int32_t* ctx_len, int Hkv, int Cap, int D,
                    int pshift, int units) {
  pdl_wait_then_release();
  const int x = blockIdx.x / units, h = x % Hkv, b = x / Hkv;
  const AppendSpan sp = append_span(nw, ctx_len, b, Cap);
  const int pg = (sp.start >> pshift) + blockIdx.x % units;
  if (sp.n == 0 || pg > (sp.start + sp.n - 1) >> pshift) return;
  const int d = threadIdx.x;
  if (d >= D) return;
  const bf16* src = static_cast<const bf16*>(nw.k) + b * nw.kb + h * nw.kh + d;
  const int p0 = max(pg << pshift, sp.start), p1 = min((pg + 1) << pshift, sp.start + sp.n);
  const size_t at = ((size_t)(b * Hkv + h) * (Cap >> pshift) + pg) * D + d;
  const bool going = (pg << pshift) < sp.start;
  float lo = going ? to_f32(kmin[at]) : to_f32(src[(p0 - sp.start) * nw.kt]);
  float hi = going ? to_f32(kmax[at]) : lo;
  for (int p = p0; p < p1; ++p) {
    const float x = to_f32(src[(p - sp.start) * nw.kt]);
    lo = fminf(lo, x);
    hi = fmaxf(hi, x);
  }
  kmin[at] = __float2bfloat16_rn(lo);
  kmax[at] = __float2bfloat16_rn(hi);
}

__global__ void kv8_advance_kernel(const Kv8New nw, const int32_t* ctx_len, int32_t* ctx_out, int32_t* pos_out, int B,
                                   int Cap) {
  pdl_wait_then_release();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= B) return;
  const AppendSpan sp = append_span(nw, ctx_len, b, Cap);
  ctx_out[b] = sp.start + sp.n;
  if (pos_out) pos_out[b] = sp.n ? sp.start : -1;
}

cudaError_t launch_kv8_append(const Shape& s, const Kv8& c, const Kv8New& n, void* kmin, void* kmax, float* mass,
                              const int32_t* ctx_len, int32_t* ctx_out, int32_t* pos_out, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (n.max_new > 0) {
    const int units = (n.max_new >> c.bshift) + 2, pages = (n.max_new >> s.pshift) + 2;
    const dim3 grid((unsigned)units * 2 * s.Hkv * s.B);
    e = c.format == kKv8Int8 ? launch_pdl(kv8_append_kernel<kKv8Int8>, grid, dim3(256), 0, st, c, n, mass, ctx_len,
                                          s.Hkv, s.Cap, s.D, units)
                             : launch_pdl(kv8_append_kernel<kKv8E4m3>, grid, dim3(256), 0, st, c, n, mass, ctx_len,
                                          s.Hkv, s.Cap, s.D, units);
    if (e == cudaSuccess && kmin)
      e = launch_pdl(kv8_pagemeta_kernel, dim3((unsigned)pages * s.Hkv * s.B), dim3(128), 0, st, n,
                     static_cast<bf16*>(kmin), static_cast<bf16*>(kmax), ctx_len, s.Hkv, s.Cap, s.D, s.pshift, pages);
  }
  if (e == cudaSuccess)
    e = launch_pdl(kv8_advance_kernel, dim3((s.B + 127) / 128), dim3(128), 0, st, n, ctx_len, ctx_out, pos_out, s.B,
                   s.Cap);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ---------------------------------------------------------------- eviction

// The blocks row `row` keeps, one CTA per row: a forced block's key is the
// largest, another's is its mass (order-preserving bits); the keep-th largest
// key T comes from four 8-bit radix passes, keys above T are kept, and keys
// equal to T from the lowest block up until the list is full.
__global__ void __launch_bounds__(256)
kv8_choose_kernel(const Kv8Evict e, int Hkv) {
  pdl_wait_then_release();
  const int row = blockIdx.x, bsh = e.src.bshift;
  const int nb = clamp_len(e.ctx_len[row / Hkv], e.cap) >> bsh;
  int32_t* kept = e.kept + (size_t)row * e.keep;
  const float* mass = e.mass + (size_t)row * (e.cap >> bsh);
  if (nb <= e.keep) {
    for (int i = threadIdx.x; i < e.keep; i += 256) kept[i] = i < nb ? i : -1;
    return;
  }
  auto key = [&](int i) -> uint32_t {
    if (i < e.n_sink || i >= nb - e.n_recent) return 0xffffffffu;
    const float m = mass[i] + 0.f;  // -0 counts as 0
    return m != m ? 0xfffffffeu : min(float_key(m), 0xfffffffdu);
  };
  __shared__ int s_hist[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left, s_warp[8], s_warp_eq[8], s_base, s_base_eq;
  if (threadIdx.x == 0) { s_prefix = 0; s_left = e.keep; }
  for (int shift = 24; shift >= 0; shift -= 8) {
    s_hist[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix, mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int i = threadIdx.x; i < nb; i += 256) {
      const uint32_t k = key(i);
      if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int left = s_left, d = 255;
      while (d > 0 && s_hist[d] < left) left -= s_hist[d--];
      s_left = left;
      s_prefix = prefix | ((uint32_t)d << shift);
    }
    __syncthreads();
  }
  const uint32_t T = s_prefix;
  const int take_eq = s_left;  // keys equal to T that are kept
  if (threadIdx.x == 0) { s_base = 0; s_base_eq = 0; }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i0 = 0; i0 < nb; i0 += 256) {
    const int i = i0 + threadIdx.x;
    const uint32_t k = i < nb ? key(i) : 0u;
    const bool eq = i < nb && k == T, gt = i < nb && k > T;
    const uint32_t beq = __ballot_sync(0xffffffffu, eq), bgt = __ballot_sync(0xffffffffu, gt);
    if (lane == 0) { s_warp_eq[warp] = __popc(beq); s_warp[warp] = __popc(bgt); }
    __syncthreads();
    int before = s_base, before_eq = s_base_eq;
    for (int w = 0; w < warp; ++w) { before += s_warp[w]; before_eq += s_warp_eq[w]; }
    const uint32_t lt = (1u << lane) - 1u;
    before += __popc(bgt & lt);
    before_eq += __popc(beq & lt);
    if (gt || (eq && before_eq < take_eq)) kept[before + min(before_eq, take_eq)] = i;
    __syncthreads();
    if (threadIdx.x == 0)
      for (int w = 0; w < 8; ++w) { s_base += s_warp[w]; s_base_eq += s_warp_eq[w]; }
    __syncthreads();
  }
}

// Moves 16-byte columns [col0, col0 + cols) of one row's kept items of
// `bytes` bytes each: item i of the destination is item kept[i] of the
// source.  The CTA goes up the items and reads a round of them before it writes
// any, so that in place nothing is overwritten before it has been read: item i
// goes to i <= kept[i], and what later rounds read lies above what this one
// writes.
__device__ __forceinline__ void move_column(const uint8_t* src, uint8_t* dst, const int32_t* kept, int n, int bytes,
                                            int col0, int cols) {
  constexpr int U = 4;
  const int total = n * cols;
  for (int i0 = 0; i0 < total; i0 += 256 * U) {
    uint4 v[U];
    bool go[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 256 + threadIdx.x;
      const int it = i / cols, cl = col0 + i % cols;
      go[u] = i < total && (src != dst || kept[it] != it);
      if (go[u]) v[u] = *reinterpret_cast<const uint4*>(src + (size_t)kept[it] * bytes + (size_t)cl * 16);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 256 + threadIdx.x;
      const int it = i / cols, cl = col0 + i % cols;
      if (go[u]) *reinterpret_cast<uint4*>(dst + (size_t)it * bytes + (size_t)cl * 16) = v[u];
    }
    __syncthreads();
  }
}

// Part x < 2 * slices of a row: a slice of the columns of K's or V's blocks;
// then one CTA for the scales, sums, tails and the length, and one each for
// kmin and kmax.
__global__ void __launch_bounds__(256)
kv8_move_kernel(const Kv8Evict e, int Hkv, int D, int P, int slices, int parts) {
  pdl_wait_then_release();
  const int row = blockIdx.x / parts, b = row / Hkv, block = e.src.block, bsh = e.src.bshift;
  const int N = clamp_len(e.ctx_len[b], e.cap);
  const int nb = N >> bsh, n = min(nb, e.keep), rest = N & (block - 1);
  const int nsrc = e.cap >> bsh, ndst = e.dcap >> bsh;
  const int32_t* kept = e.kept + (size_t)row * e.keep;
  const int x = blockIdx.x % parts;
  if (x < 2 * slices) {
    const size_t bytes = (size_t)block * D;
    const int cols = (int)(bytes / 16) / slices, col0 = (x >> 1) * cols;
    const uint8_t* s = ((x & 1) ? e.src.vc : e.src.kc) + (size_t)row * nsrc * bytes;
    uint8_t* d = ((x & 1) ? e.dst.vc : e.dst.kc) + (size_t)row * ndst * bytes;
    move_column(s, d, kept, n, (int)bytes, col0, cols);
  } else if (x == 2 * slices) {
    for (int i0 = 0; i0 < n; i0 += 256) {
      const int i = i0 + threadIdx.x;
      float a = 0.f, v = 0.f, m = 0.f;
      if (i < n) {
        const size_t at = (size_t)row * nsrc + kept[i];
        a = e.src.ks[at];
        v = e.src.vs[at];
        m = e.mass[at];
      }
      __syncthreads();
      if (i < n) {
        const size_t at = (size_t)row * ndst + i;
        e.dst.ks[at] = a;
        e.dst.vs[at] = v;
        if (e.mass_out) e.mass_out[at] = m;
      }
    }
    if (!e.in_place) {
      const size_t t0 = (size_t)row * block * D;
      for (int i = threadIdx.x; i < rest * D / 8; i += 256) {
        reinterpret_cast<uint4*>(static_cast<bf16*>(e.dst.kt) + t0)[i] =
            reinterpret_cast<const uint4*>(static_cast<const bf16*>(e.src.kt) + t0)[i];
        reinterpret_cast<uint4*>(static_cast<bf16*>(e.dst.vt) + t0)[i] =
            reinterpret_cast<const uint4*>(static_cast<const bf16*>(e.src.vt) + t0)[i];
      }
    }
  } else {
    const bool mx = x == 2 * slices + 2;
    const int ppb = block / P;
    const int item = ppb * D * 2;  // bytes of a block's page summaries
    const uint8_t* s = static_cast<const uint8_t*>(mx ? e.kmax : e.kmin) + (size_t)row * nsrc * item;
    uint8_t* d = static_cast<uint8_t*>(mx ? e.kmax_out : e.kmin_out) + (size_t)row * ndst * item;
    move_column(s, d, kept, n, item, 0, item / 16);
    // the pages of the newest, partial block
    const int vecs = (rest + P - 1) / P * D * 2 / 16;
    if (s + (size_t)nb * item != d + (size_t)n * item)
      for (int i = threadIdx.x; i < vecs; i += 256)
        reinterpret_cast<uint4*>(d + (size_t)n * item)[i] = reinterpret_cast<const uint4*>(s + (size_t)nb * item)[i];
  }
}

__global__ void kv8_evicted_len_kernel(const Kv8Evict e, int B) {
  pdl_wait_then_release();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= B) return;
  const int N = clamp_len(e.ctx_len[b], e.cap);
  e.ctx_out[b] = min(N >> e.src.bshift, e.keep) * e.src.block + (N & (e.src.block - 1));
}

cudaError_t launch_kv8_evict(const Shape& s, const Kv8Evict& e, cudaStream_t st) {
  const int rows = s.B * s.Hkv;
  cudaError_t r = launch_pdl(kv8_choose_kernel, dim3(rows), dim3(256), 0, st, e, s.Hkv);
  if (r != cudaSuccess) return r;
  const int slices = 4, parts = 2 * slices + (e.kmin ? 3 : 1);
  r = launch_pdl(kv8_move_kernel, dim3((unsigned)rows * parts), dim3(256), 0, st, e, s.Hkv, s.D, s.P, slices, parts);
  if (r != cudaSuccess) return r;
  r = launch_pdl(kv8_evicted_len_kernel, dim3((s.B + 127) / 128), dim3(128), 0, st, e, s.B);
  return r != cudaSuccess ? r : cudaGetLastError();
}

}  // namespace sls
