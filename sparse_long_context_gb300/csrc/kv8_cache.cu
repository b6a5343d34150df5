// The 8-bit cache's writers: appending tokens (quantising the blocks they
// complete) and evicting blocks by accumulated attention weight.
//
// Both are bound by memory on prompts: four prompts of up to 32k tokens, 8 heads of
// 128 channels, with page min/max: 122 us for 813 MB (98% of the measured copy); 8 x 4
// rows cut from 32k tokens to 16k: 49 us for 269 MB, of which the copies take 41 (97%)
// and the choice before them the rest; in place, in two launches, 52 us for the 267 MB of the
// blocks that move.  Single tokens and small caches are latency: 3.8 us for 32 sequences'
// tokens, 5.3 us for a small eviction, 7.9 in place.  (Times of the device alone, calls
// replayed from a graph, with lengths written to other memory; written in place they cost
// a prompt's append 0.5 us and an eviction 1.1 us more, a launch of its own.)
#include <algorithm>

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

// Page min/max of the new keys of one KV head: pages [p0, p1) of the row, by the
// CTA's NT threads, a thread per page and 16-byte chunk of channels.  `src` is the
// first new token.  A page that held tokens before is merged with what is stored.
template <int NT>
__device__ __forceinline__ void append_pagemeta(const bf16* src, int64_t st, bf16* kmin, bf16* kmax, size_t row, int Cap,
                                                int D, int pshift, const AppendSpan& sp, int p0, int p1) {
  const int cpr = D / 8;
  for (int i = threadIdx.x; i < (p1 - p0) * cpr; i += NT) {
    const int pg = p0 + i / cpr, ch = (i % cpr) * 8;
    const int t0 = max(pg << pshift, sp.start) - sp.start, t1 = min((pg + 1) << pshift, sp.start + sp.n) - sp.start;
    const size_t at = (row * (Cap >> pshift) + pg) * D + ch;
    uint4 lo, hi;
    if ((pg << pshift) < sp.start) {
      lo = *reinterpret_cast<const uint4*>(kmin + at);
      hi = *reinterpret_cast<const uint4*>(kmax + at);
    } else {
      lo = hi = *reinterpret_cast<const uint4*>(src + t0 * st + ch);
    }
    __nv_bfloat162* l2 = reinterpret_cast<__nv_bfloat162*>(&lo);
    __nv_bfloat162* h2 = reinterpret_cast<__nv_bfloat162*>(&hi);
#pragma unroll 8
    for (int t = t0; t < t1; ++t) {
      const uint4 x = *reinterpret_cast<const uint4*>(src + t * st + ch);
      const __nv_bfloat162* x2 = reinterpret_cast<const __nv_bfloat162*>(&x);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        l2[k] = __hmin2(l2[k], x2[k]);
        h2[k] = __hmax2(h2[k], x2[k]);
      }
    }
    *reinterpret_cast<uint4*>(kmin + at) = lo;
    *reinterpret_cast<uint4*>(kmax + at) = hi;
  }
}

// Codes of eight bf16 values by the IEEE division, one after the other: for blocks
// of subnormals, out of line so that the others' code stays short.
template <int FMT>
__device__ __noinline__ uint2 kv8_codes8_exact(uint4 raw, float amax) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll 1
  for (int k = 0; k < 8; ++k) {
    const uint32_t h = (k < 4 ? (k < 2 ? raw.x : raw.y) : (k < 6 ? raw.z : raw.w)) >> (16 * (k & 1)) << 16;
    const uint32_t c = kv8_code<FMT>(__uint_as_float(h), amax) << (8 * (k & 3));
    if (k < 4) w[0] |= c;
    else w[1] |= c;
  }
  return make_uint2(w[0], w[1]);
}

// Codes of eight bf16 values from products with rcp = top / amax; a division per
// value is three times the work, and a chunk's append is then bound by issue.  The
// product is within 2^-23 (relative) of the quotient top x / amax of numbers of at
// most 8 significant bits, which is either exactly on a tie between two codes or at
// least 2^-16 (int8; e4m3 2^-13) away from one: the tie (2n + 1) a 2^k = 2 top x has
// factors of at most 16 bits.  Rounded to 18 mantissa bits (within 2^-19), a product
// next to a tie becomes the tie itself, whose rounding to even then is that of exact
// arithmetic, and no other product crosses one.
template <int FMT>
__device__ __forceinline__ uint2 kv8_codes8(const uint4& raw, float rcp) {
  float y[8];
  unpack_vec(raw, y);
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] = __uint_as_float((__float_as_uint(y[k] * rcp) + 16u) & ~31u);
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if constexpr (FMT == kKv8Int8) {
      uint32_t c[4];  // 1.5 * 2^23 brings the nearest integer into the low bits
#pragma unroll
      for (int u = 0; u < 4; ++u) c[u] = __float_as_uint(y[4 * k + u] + 12582912.f);
      w[k] = __byte_perm(__byte_perm(c[0], c[1], 0x0040u), __byte_perm(c[2], c[3], 0x0040u), 0x5410u);
    } else {
      const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * k], y[4 * k + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * k + 2], y[4 * k + 3]), __NV_SATFINITE, __NV_E4M3);
      w[k] = a | b << 16;
    }
  }
  return make_uint2(w[0], w[1]);
}

// Largest magnitude of a vector's bf16 values as two bit patterns (NaN above
// infinity above the numbers).
__device__ __forceinline__ uint32_t abs_max2(const uint4& v) {
  const uint32_t m = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
}

// Quantises a block whose vectors the CTA's threads hold, VPT each: vector v of
// thread i is token v NT / (D / 8) + i / (D / 8).  Writes codes and scale.
template <int FMT, int VPT, int NT>
__device__ __forceinline__ void quantise_held(const uint4 (&x)[VPT], uint8_t* codes, float* scale, uint32_t* s_max) {
  uint32_t m2 = 0;
#pragma unroll
  for (int v = 0; v < VPT; ++v) m2 = __vmaxu2(m2, abs_max2(x[v]));
  uint32_t mx = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NT / 32; ++k) mx = max(mx, s_max[k]);
  const float amax = __uint_as_float(mx << 16);
  const bool finite = mx < 0x7f80u;
  const float rcp = __fdiv_rn(kv8_top<FMT>(), amax);
  const bool fast = rcp < 1e38f;  // a block of subnormals overflows the reciprocal
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    uint2 w = make_uint2(0u, 0u);
    if (finite && mx) w = fast ? kv8_codes8<FMT>(x[v], rcp) : kv8_codes8_exact<FMT>(x[v], amax);
    *reinterpret_cast<uint2*>(codes + ((size_t)v * NT + threadIdx.x) * 8) = w;
  }
  if (threadIdx.x == 0) *scale = finite ? __fdiv_rn(amax, kv8_top<FMT>()) : __int_as_float(0x7fffffff);
}

struct AppendOut {
  bf16 *kmin, *kmax;  // or null
  float* mass;        // or null
  const int32_t* ctx_len;
  int32_t *ctx_out, *pos_out;
  int Hkv, Cap, pshift;
  int advance;  // this kernel writes ctx_out and pos_out
};

// Prompts and chunks: one CTA per (sequence, block touched, KV head, K or V), the
// heads of a block next to each other (they share DRAM pages of the projection).
// A complete block's vectors are read once, all loads in flight together, the
// earlier tokens from the tail buffer; the CTA of a sequence's first block also
// writes its newest, partial block to the tail, after its own reads of it.
template <int FMT, int D, int VPT, int NT>
__global__ void __launch_bounds__(NT)
kv8_append_kernel(const Kv8 c, const Kv8New nw, const AppendOut o, int units) {
  pdl_wait_then_release();
  constexpr int CPR = D / 8;
  __shared__ uint32_t s_max[NT / 32];
  const int heads = 2 * o.Hkv;
  const int hv = blockIdx.x % heads, h = hv >> 1, isv = hv & 1, u = (blockIdx.x / heads) % units,
            b = blockIdx.x / heads / units;
  const AppendSpan sp = append_span(nw, o.ctx_len, b, o.Cap);
  if (o.advance && u == 0 && hv == 0 && threadIdx.x == 0) {
    o.ctx_out[b] = sp.start + sp.n;
    if (o.pos_out) o.pos_out[b] = sp.n ? sp.start : -1;
  }
  if (sp.n == 0) return;
  const int first = sp.start >> c.bshift, last = (sp.start + sp.n) >> c.bshift;  // `last`: the newest, partial block
  const int j = first + u;
  const size_t row = (size_t)b * o.Hkv + h;
  const bf16* src = static_cast<const bf16*>(isv ? nw.v : nw.k) + b * (isv ? nw.vb : nw.kb) + h * (isv ? nw.vh : nw.kh);
  const int64_t st = isv ? nw.vt : nw.kt;
  bf16* tail = static_cast<bf16*>(isv ? c.vt : c.kt) + row * c.block * D;
  const int ch = ((int)threadIdx.x % CPR) * 8;
  if (j < last) {
    uint4 x[VPT];
    const int from = (j << c.bshift) - sp.start;  // the block's first token, counted from the first new one
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int t = v * (NT / CPR) + (int)threadIdx.x / CPR;
      x[v] = *reinterpret_cast<const uint4*>(from + t < 0 ? tail + (size_t)t * D + ch : src + (from + t) * st + ch);
    }
    const size_t blk = row * (o.Cap >> c.bshift) + j;
    quantise_held<FMT, VPT, NT>(x, (isv ? c.vc : c.kc) + blk * c.block * D, (isv ? c.vs : c.ks) + blk, s_max);
    if (o.mass && !isv && threadIdx.x == 0) o.mass[blk] = 0.f;
  }
  if (o.kmin && !isv && j <= last) {
    // the pages that begin in this block, and for the first block the one before: the new tokens
    // are in the cache from the reads above
    const int pages = (sp.start + sp.n - 1) >> o.pshift;  // the last page
    const int p0 = u == 0 ? sp.start >> o.pshift : ((j << c.bshift) + (1 << o.pshift) - 1) >> o.pshift;
    const int p1 = min(((j + 1) << c.bshift) + (1 << o.pshift) - 1, INT32_MAX) >> o.pshift;
    append_pagemeta<NT>(src, st, o.kmin, o.kmax, row, o.Cap, D, o.pshift, sp, p0, min(p1, pages + 1));
  }
  if (u == 0) {
    __syncthreads();  // the block just quantised has read the tail
    const int t0 = last == first ? sp.start - (first << c.bshift) : 0;
    const int t1 = (sp.start + sp.n) - (last << c.bshift);
    const int from = (last << c.bshift) - sp.start;
#pragma unroll 4
    for (int t = t0 + (int)threadIdx.x / CPR; t < t1; t += NT / CPR)
      *reinterpret_cast<uint4*>(tail + (size_t)t * D + ch) = *reinterpret_cast<const uint4*>(src + (from + t) * st + ch);
  }
}

// Single tokens: a cluster per sequence, its CTAs taking the KV heads in turn, so
// that ctx_len may be advanced in place (rank 0 writes it when every CTA has read
// it).  Half of a CTA's threads take K, half V.  Only a token that completes its
// block reads the tail and quantises it.
template <int FMT, int D>
__global__ void __launch_bounds__(256)
kv8_append_one_kernel(const Kv8 c, const Kv8New nw, const AppendOut o, int cluster) {
  constexpr int CPR = D / 8, NT = 128;
  __shared__ uint32_t s_max[2][NT / 32];
  pdl_wait_then_release();
  const int b = blockIdx.x / cluster, rank = blockIdx.x % cluster;
  const int isv = threadIdx.x / NT, tid = threadIdx.x % NT, ch = (tid % CPR) * 8;
  auto source = [&](int h) {
    return static_cast<const bf16*>(isv ? nw.v : nw.k) + b * (isv ? nw.vb : nw.kb) + h * (isv ? nw.vh : nw.kh);
  };
  // the lane's channels of the first head's new token, in flight with the lengths
  uint4 token = *reinterpret_cast<const uint4*>(source(rank) + ch);
  const AppendSpan sp = append_span(nw, o.ctx_len, b, o.Cap);
  if (cluster > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // ctx_len has been read
  const int blk = sp.start >> c.bshift, slot = sp.start & (c.block - 1);
  const bool done = slot == c.block - 1;
  if (sp.n) {
    for (int h = rank; h < o.Hkv; h += cluster) {
      const size_t row = (size_t)b * o.Hkv + h;
      if (h != rank) token = *reinterpret_cast<const uint4*>(source(h) + ch);
      bf16* tail = static_cast<bf16*>(isv ? c.vt : c.kt) + row * c.block * D;
      if (!done) {
        if (tid < CPR) *reinterpret_cast<uint4*>(tail + (size_t)slot * D + ch) = token;
      } else {
        const size_t at = row * (o.Cap >> c.bshift) + blk;
        uint8_t* codes = (isv ? c.vc : c.kc) + at * c.block * D;
        auto vec = [&](int t) { return t < slot ? *reinterpret_cast<const uint4*>(tail + (size_t)t * D + ch) : token; };
        uint32_t m2 = 0;
#pragma unroll 8
        for (int t = tid / CPR; t < c.block; t += NT / CPR) m2 = __vmaxu2(m2, abs_max2(vec(t)));
        uint32_t mx = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
        __syncthreads();  // the head before has been read
        if ((tid & 31) == 0) s_max[isv][tid >> 5] = mx;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NT / 32; ++k) mx = max(mx, s_max[isv][k]);
        const float amax = __uint_as_float(mx << 16);
        const bool finite = mx < 0x7f80u;
        const float rcp = __fdiv_rn(kv8_top<FMT>(), amax);
        const bool fast = rcp < 1e38f;  // a block of subnormals overflows the reciprocal
#pragma unroll 8
        for (int t = tid / CPR; t < c.block; t += NT / CPR) {
          uint2 w = make_uint2(0u, 0u);
          if (finite && mx) w = fast ? kv8_codes8<FMT>(vec(t), rcp) : kv8_codes8_exact<FMT>(vec(t), amax);
          *reinterpret_cast<uint2*>(codes + (size_t)t * D + ch) = w;
        }
        if (tid == 0) {
          (isv ? c.vs : c.ks)[at] = finite ? __fdiv_rn(amax, kv8_top<FMT>()) : __int_as_float(0x7fffffff);
          if (o.mass && !isv) o.mass[at] = 0.f;
        }
      }
      // page min/max by the last warp of K's threads
      if (o.kmin && !isv && tid >= NT - CPR) {
        const size_t at = (row * (o.Cap >> o.pshift) + (sp.start >> o.pshift)) * D + ch;
        const uint4 x = token;
        uint4 lo = x, hi = x;
        if (sp.start & ((1 << o.pshift) - 1)) {
          lo = *reinterpret_cast<const uint4*>(o.kmin + at);
          hi = *reinterpret_cast<const uint4*>(o.kmax + at);
          const __nv_bfloat162* x2 = reinterpret_cast<const __nv_bfloat162*>(&x);
          __nv_bfloat162 *l2 = reinterpret_cast<__nv_bfloat162*>(&lo), *h2 = reinterpret_cast<__nv_bfloat162*>(&hi);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            l2[k] = __hmin2(l2[k], x2[k]);
            h2[k] = __hmax2(h2[k], x2[k]);
          }
        }
        *reinterpret_cast<uint4*>(o.kmin + at) = lo;
        *reinterpret_cast<uint4*>(o.kmax + at) = hi;
      }
    }
  }
  if (cluster > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  else __syncthreads();
  if (rank == 0 && threadIdx.x == 0) {
    o.ctx_out[b] = sp.start + sp.n;
    if (o.pos_out) o.pos_out[b] = sp.n ? sp.start : -1;
  }
}

__global__ void kv8_advance_kernel(const Kv8New nw, const AppendOut o, int B) {
  pdl_wait_then_release();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= B) return;
  const AppendSpan sp = append_span(nw, o.ctx_len, b, o.Cap);
  o.ctx_out[b] = sp.start + sp.n;
  if (o.pos_out) o.pos_out[b] = sp.n ? sp.start : -1;
}

template <int FMT, int D, int BLOCK>
static cudaError_t append_chunk(const Kv8& c, const Kv8New& n, const AppendOut& o, int units, int B, cudaStream_t st) {
  // a block's 16-byte vectors, at most eight a thread
  constexpr int NV = BLOCK * D / 8, NT = NV / 8 > 128 ? NV / 8 : 128, VPT = NV / NT;
  return launch_pdl(kv8_append_kernel<FMT, D, VPT, NT>, dim3((unsigned)units * 2 * o.Hkv * B), dim3(NT), 0, st, c, n, o,
                    units);
}

template <int FMT, int D>
static cudaError_t append_launch(const Kv8& c, const Kv8New& n, const AppendOut& o, int B, cudaStream_t st) {
  if (n.max_new == 1) {
    const int cl = std::min(o.Hkv, 8);
    return launch_pdl_cluster(kv8_append_one_kernel<FMT, D>, dim3((unsigned)B * cl), dim3(256), 0, cl, st, c, n, o, cl);
  }
  const int units = (n.max_new >> c.bshift) + 2;
  switch (c.block) {
    case 16: return append_chunk<FMT, D, 16>(c, n, o, units, B, st);
    case 32: return append_chunk<FMT, D, 32>(c, n, o, units, B, st);
    case 64: return append_chunk<FMT, D, 64>(c, n, o, units, B, st);
    case 128: return append_chunk<FMT, D, 128>(c, n, o, units, B, st);
    default: return append_chunk<FMT, D, 256>(c, n, o, units, B, st);
  }
}

cudaError_t launch_kv8_append(const Shape& s, const Kv8& c, const Kv8New& n, void* kmin, void* kmax, float* mass,
                              const int32_t* ctx_len, int32_t* ctx_out, int32_t* pos_out, cudaStream_t st) {
  AppendOut o = {static_cast<bf16*>(kmin), static_cast<bf16*>(kmax), mass, ctx_len, ctx_out, pos_out, s.Hkv, s.Cap,
                 s.pshift, 0};
  // The lengths may be written by the CTAs that still read them only where they
  // are other memory; in place a launch of its own follows a chunk's.
  auto apart = [&](const int32_t* p) {
    const uintptr_t x = (uintptr_t)p, y = (uintptr_t)ctx_len, n4 = (uintptr_t)s.B * 4;
    return !p || x + n4 <= y || y + n4 <= x;
  };
  o.advance = apart(ctx_out) && apart(pos_out);
  cudaError_t e = cudaSuccess;
  if (n.max_new > 0) {
    if (c.format == kKv8Int8)
      e = s.D == 64 ? append_launch<kKv8Int8, 64>(c, n, o, s.B, st) : append_launch<kKv8Int8, 128>(c, n, o, s.B, st);
    else
      e = s.D == 64 ? append_launch<kKv8E4m3, 64>(c, n, o, s.B, st) : append_launch<kKv8E4m3, 128>(c, n, o, s.B, st);
  }
  if (e == cudaSuccess && (n.max_new == 0 || (n.max_new > 1 && !o.advance)))
    e = launch_pdl(kv8_advance_kernel, dim3((s.B + 127) / 128), dim3(128), 0, st, n, o, s.B);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ---------------------------------------------------------------- eviction

constexpr int kChooseThreads = 256;
constexpr int kChooseStaged = 4096;  // keys of a row kept in shared memory; longer rows read them again

// Exclusive scan of one int per thread over the CTA.
template <int NT>
__device__ __forceinline__ int cta_scan(int v, int* tmp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    before += w < warp ? tmp[w] : 0;
    total += tmp[w];
  }
  __syncthreads();
  return before + x - v;
}

// The blocks a row with nb > keep complete blocks keeps: a forced block's key is the
// largest, another's is its mass (order-preserving bits).  The keep-th largest key T
// comes from four 8-bit radix passes over the keys in shared memory (the bins are
// summed by a scan over the threads, a bin each); keys above T are kept, and keys equal
// to T from the lowest block up until the list is full.  emit(place, block) is called
// for every kept block, places ascending.  Bound by the latency of its barriers: 4 us.
struct ChooseSmem {
  uint32_t key[kChooseStaged];
  int hist[256], tmp[kChooseThreads / 32], bin, above;
};
template <typename Emit>
__device__ __forceinline__ void choose_blocks(const Kv8Evict& e, const float* mass, int nb, ChooseSmem& sh, Emit emit) {
  constexpr int NT = kChooseThreads;
  const int tid = threadIdx.x;
  auto key_of = [&](int i) -> uint32_t {
    if (i < e.n_sink || i >= nb - e.n_recent) return 0xffffffffu;
    const float m = mass[i] + 0.f;  // -0 counts as 0
    return m != m ? 0xfffffffeu : min(float_key(m), 0xfffffffdu);
  };
  const int staged = min(nb, kChooseStaged);
#pragma unroll 4
  for (int i = tid; i < staged; i += NT) sh.key[i] = key_of(i);
  auto key = [&](int i) { return i < kChooseStaged ? sh.key[i] : key_of(i); };
  uint32_t prefix = 0;
  int left = e.keep;
  for (int shift = 24; shift >= 0; shift -= 8) {
    sh.hist[tid] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int i = tid; i < nb; i += NT) {
      const uint32_t k = key(i);
      if ((k & mask) == prefix) atomicAdd(&sh.hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    // thread i holds bin 255 - i; the bin in which the count from the top reaches `left`
    const int n = sh.hist[255 - tid];
    int total;
    const int above = cta_scan<NT>(n, sh.tmp, total);
    if (above < left && above + n >= left) {
      sh.bin = 255 - tid;
      sh.above = above;
    }
    __syncthreads();
    left -= sh.above;
    prefix |= (uint32_t)sh.bin << shift;
  }
  // ascending output: `left` of the keys equal to T (= prefix) are kept
  int base = 0, base_eq = 0;
  for (int i0 = 0; i0 < nb; i0 += NT) {
    const int i = i0 + tid;
    const uint32_t k = i < nb ? key(i) : 0u;
    const bool eq = i < nb && k == prefix, gt = i < nb && k > prefix;
    int total;
    const int at = cta_scan<NT>((int)gt | (int)eq << 16, sh.tmp, total);  // at most NT of each: no carry
    const int g = base + (at & 0xffff), q = base_eq + (at >> 16);
    if (gt || (eq && q < left)) emit(g + min(q, left), i);
    base += total & 0xffff;
    base_eq += total >> 16;
  }
}

__device__ __forceinline__ void evicted_len(const Kv8Evict& e, int b, int N) {
  e.ctx_out[b] = min(N >> e.src.bshift, e.keep) * e.src.block + (N & (e.src.block - 1));
}

// The list alone, before blocks move in place: one CTA per row.
__global__ void __launch_bounds__(kChooseThreads)
kv8_choose_kernel(const Kv8Evict e, int Hkv, int write_len) {
  __shared__ ChooseSmem sh;
  pdl_wait_then_release();
  const int row = blockIdx.x, tid = threadIdx.x;
  const int N = clamp_len(e.ctx_len[row / Hkv], e.cap), nb = N >> e.src.bshift;
  int32_t* kept = e.kept + (size_t)row * e.keep;
  if (write_len && row % Hkv == 0 && tid == 0) evicted_len(e, row / Hkv, N);
  if (nb <= e.keep) {
    for (int i = tid; i < e.keep; i += kChooseThreads) kept[i] = i < nb ? i : -1;
    return;
  }
  choose_blocks(e, e.mass + (size_t)row * (e.cap >> e.src.bshift), nb, sh, [&](int at, int i) { kept[at] = i; });
}

// Into another cache, choice and copies in one launch: every CTA of a row makes the
// row's choice for itself (4 us side by side, against a launch between the two) and
// copies the items [i0, i0 + per) of the list; the row's first CTA writes the list and
// the length, and copies the tails.  Eight loads of a thread are in flight together.
constexpr int kEvictSlice = 2048;  // list entries a CTA keeps
constexpr int kEvictPerSm = 2;     // CTAs per SM of the launch (3 to 8: up to 10% slower on prompts, 50% on small caches)
__global__ void __launch_bounds__(kChooseThreads)
kv8_evict_copy_kernel(const Kv8Evict e, int Hkv, int D, int P, int per, int parts, int write_len) {
  constexpr int NT = kChooseThreads, U = 4;
  __shared__ ChooseSmem sh;
  __shared__ int s_kept[kEvictSlice];
  pdl_wait_then_release();
  const int row = blockIdx.x / parts, part = blockIdx.x % parts, block = e.src.block, bsh = e.src.bshift;
  const int tid = threadIdx.x;
  const int N = clamp_len(e.ctx_len[row / Hkv], e.cap);
  const int nb = N >> bsh, n = min(nb, e.keep), rest = N & (block - 1);
  const size_t srow = (size_t)row * (e.cap >> bsh), drow = (size_t)row * (e.dcap >> bsh);
  const int i0 = part * per, i1 = min(n, i0 + per);
  int32_t* kept = e.kept + (size_t)row * e.keep;
  if (part == 0) {
    if (write_len && row % Hkv == 0 && tid == 0) evicted_len(e, row / Hkv, N);
    const size_t t0 = (size_t)row * block * D / 8;
#pragma unroll 2
    for (int i = tid; i < rest * D / 8; i += NT) {
      const uint4 a = static_cast<const uint4*>(e.src.kt)[t0 + i], b = static_cast<const uint4*>(e.src.vt)[t0 + i];
      static_cast<uint4*>(e.dst.kt)[t0 + i] = a;
      static_cast<uint4*>(e.dst.vt)[t0 + i] = b;
    }
    if (nb <= e.keep)
      for (int i = tid; i < e.keep; i += NT) kept[i] = i < nb ? i : -1;
  }
  if (nb <= e.keep) {
    for (int i = i0 + tid; i < i1; i += NT) s_kept[i - i0] = i;
  } else {
    choose_blocks(e, e.mass + srow, nb, sh, [&](int at, int i) {
      if (at >= i0 && at < i1) s_kept[at - i0] = i;
      if (part == 0) kept[at] = i;
    });
  }
  __syncthreads();
  for (int i = i0 + tid; i < i1; i += NT) {
    const size_t from = srow + s_kept[i - i0], to = drow + i;
    const float a = e.src.ks[from], b = e.src.vs[from], m = e.mass_out ? e.mass[from] : 0.f;
    e.dst.ks[to] = a;
    e.dst.vs[to] = b;
    if (e.mass_out) e.mass_out[to] = m;
  }
  const int vecs = block * D / 16, vsh = __ffs(vecs) - 1;  // 16-byte vectors of a block's codes, a power of two
  for (int x0 = 0; x0 < (i1 - i0) << vsh; x0 += NT * U) {
    uint4 k[U], v[U];
    size_t to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int w = x0 + u * NT + tid;
      if (w < (i1 - i0) << vsh) {
        const int it = w >> vsh, c = w & (vecs - 1);
        const size_t from = (srow + s_kept[it]) * vecs + c;
        to[u] = (drow + i0 + it) * vecs + c;
        k[u] = ldg_stream(reinterpret_cast<const uint4*>(e.src.kc) + from);
        v[u] = ldg_stream(reinterpret_cast<const uint4*>(e.src.vc) + from);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (x0 + u * NT + tid < (i1 - i0) << vsh) {
        reinterpret_cast<uint4*>(e.dst.kc)[to[u]] = k[u];
        reinterpret_cast<uint4*>(e.dst.vc)[to[u]] = v[u];
      }
  }
  if (e.kmin) {
    const int item = block / P * D / 8, ish = __ffs(item) - 1;  // 16-byte vectors of a block's page summaries
    const uint4 *smin = static_cast<const uint4*>(e.kmin) + srow * item, *smax = static_cast<const uint4*>(e.kmax) + srow * item;
    uint4 *dmin = static_cast<uint4*>(e.kmin_out) + drow * item, *dmax = static_cast<uint4*>(e.kmax_out) + drow * item;
#pragma unroll 4
    for (int w = tid; w < (i1 - i0) << ish; w += NT) {
      const int it = w >> ish, c = w & (item - 1);
      const size_t from = (size_t)s_kept[it] * item + c, to = (size_t)(i0 + it) * item + c;
      const uint4 a = smin[from], b = smax[from];
      dmin[to] = a;
      dmax[to] = b;
    }
    if (part == 0)  // the pages of the newest, partial block
      for (int w = tid; w < (rest + P - 1) / P * D / 8; w += NT) {
        const uint4 a = smin[(size_t)nb * item + w], b = smax[(size_t)nb * item + w];
        dmin[(size_t)n * item + w] = a;
        dmax[(size_t)n * item + w] = b;
      }
  }
}

// In place: moves 16-byte columns [col0, col0 + cols) of one row's kept items of
// `bytes` bytes each: item i becomes item kept[i].  The CTA goes up the items and
// reads a round of them before it writes any, so that nothing is overwritten before
// it has been read: item i goes to i <= kept[i], and what later rounds read lies
// above what this one writes.
constexpr int kMoveThreads = 512;
__device__ __forceinline__ void move_column(uint8_t* base, const int32_t* kept, int n, int bytes, int col0, int cols) {
  constexpr int U = 8, NT = kMoveThreads;
  const int sh = __ffs(cols) - 1;  // a power of two, as blocks, pages and D are
  const long long total = (long long)n << sh;
  for (long long i0 = 0; i0 < total; i0 += NT * U) {
    uint4 v[U];
    int from[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long i = i0 + u * NT + threadIdx.x;
      const int it = (int)(i >> sh), col = col0 + (int)(i & (cols - 1));
      from[u] = i < total ? kept[it] : -1;
      if (from[u] == it) from[u] = -1;  // in its place already
      if (from[u] >= 0) v[u] = *reinterpret_cast<const uint4*>(base + (size_t)from[u] * bytes + col * 16);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long i = i0 + u * NT + threadIdx.x;
      const int it = (int)(i >> sh), col = col0 + (int)(i & (cols - 1));
      if (from[u] >= 0) *reinterpret_cast<uint4*>(base + (size_t)it * bytes + col * 16) = v[u];
    }
    __syncthreads();
  }
}

// Part x < 2 slices of a row: a slice of the columns of K's or V's blocks; then
// one CTA for the scales and sums, and one each for kmin and kmax.
__global__ void __launch_bounds__(kMoveThreads)
kv8_move_kernel(const Kv8Evict e, int Hkv, int D, int P, int slices, int parts) {
  pdl_wait_then_release();
  const int row = blockIdx.x / parts, x = blockIdx.x % parts, block = e.src.block, bsh = e.src.bshift;
  const int N = clamp_len(e.ctx_len[row / Hkv], e.cap);
  const int nb = N >> bsh, rest = N & (block - 1);
  if (nb <= e.keep) return;  // nothing moves
  const int n = e.keep;
  const size_t row0 = (size_t)row * (e.cap >> bsh);
  const int32_t* kept = e.kept + (size_t)row * e.keep;
  if (x < 2 * slices) {
    const int bytes = block * D, cols = bytes / 16 / slices;
    move_column(((x & 1) ? e.src.vc : e.src.kc) + row0 * bytes, kept, n, bytes, (x >> 1) * cols, cols);
  } else if (x == 2 * slices) {
    float* const mass = e.mass_out;  // the caller's sums, which the choice has read
    for (int i0 = 0; i0 < n; i0 += kMoveThreads) {
      const int i = i0 + threadIdx.x;
      float a = 0.f, v = 0.f, m = 0.f;
      if (i < n) {
        const size_t at = row0 + kept[i];
        a = e.src.ks[at];
        v = e.src.vs[at];
        m = mass[at];
      }
      __syncthreads();
      if (i < n) {
        e.src.ks[row0 + i] = a;
        e.src.vs[row0 + i] = v;
        mass[row0 + i] = m;
      }
      __syncthreads();
    }
  } else {
    const int item = block / P * D * 2;  // bytes of a block's page summaries
    uint8_t* m = static_cast<uint8_t*>(x == 2 * slices + 1 ? e.kmin_out : e.kmax_out) + row0 * item;
    move_column(m, kept, n, item, 0, item / 16);
    // the pages of the newest, partial block (nb > n: no overlap)
    for (int i = threadIdx.x; i < (rest + P - 1) / P * D * 2 / 16; i += kMoveThreads)
      reinterpret_cast<uint4*>(m + (size_t)n * item)[i] = reinterpret_cast<const uint4*>(m + (size_t)nb * item)[i];
  }
}

__global__ void kv8_evicted_len_kernel(const Kv8Evict e, int B) {
  pdl_wait_then_release();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= B) return;
  evicted_len(e, b, clamp_len(e.ctx_len[b], e.cap));
}

cudaError_t launch_kv8_evict(const Shape& s, const Kv8Evict& e, cudaStream_t st) {
  const int rows = s.B * s.Hkv;
  // the lengths are written with the choice where they are other memory than
  // the ones that are read, else last
  const uintptr_t x = (uintptr_t)e.ctx_out, y = (uintptr_t)e.ctx_len, n4 = (uintptr_t)s.B * 4;
  const bool apart = x + n4 <= y || y + n4 <= x;
  cudaError_t r;
  if (e.in_place) {
    r = launch_pdl(kv8_choose_kernel, dim3(rows), dim3(kChooseThreads), 0, st, e, s.Hkv, (int)apart);
    if (r != cudaSuccess) return r;
    // enough CTAs for the GPU, each at least 64 bytes wide
    const int bytes = e.src.block * s.D;
    int slices = 1;
    while (rows * 2 * slices < 2 * sm_count() && bytes / 16 / (2 * slices) >= 4) slices *= 2;
    const int parts = 2 * slices + (e.kmin ? 3 : 1);
    r = launch_pdl(kv8_move_kernel, dim3((unsigned)rows * parts), dim3(kMoveThreads), 0, st, e, s.Hkv, s.D, s.P, slices,
                   parts);
  } else {
    // one wave of CTAs, each with a slice of the list that fits its shared memory
    const long long want = std::max(1, kEvictPerSm * sm_count() / rows);
    const int per = (int)std::min<long long>(kEvictSlice, (e.keep + want - 1) / want), parts = (e.keep + per - 1) / per;
    r = launch_pdl(kv8_evict_copy_kernel, dim3((unsigned)rows * parts), dim3(kChooseThreads), 0, st, e, s.Hkv, s.D, s.P,
                   per, parts, (int)apart);
  }
  if (r == cudaSuccess && !apart)
    r = launch_pdl(kv8_evicted_len_kernel, dim3((s.B + 127) / 128), dim3(128), 0, st, e, s.B);
  return r != cudaSuccess ? r : cudaGetLastError();
}

}  // namespace sls
