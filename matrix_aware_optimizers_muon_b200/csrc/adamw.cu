// Kernels of the AdamW step over many tensors, of the 8-bit moments and of
// gradient clipping.  All are bound by HBM traffic.
//
// A warp takes one 256-element block of a tensor, the unit that shares a scale
// of the 8-bit moments; a lane holds 8 of its elements in registers.  On the
// wide path (full block, aligned pointers) those are 8 neighbours, else
// elements 32 apart, so that narrow accesses of a warp stay contiguous.
//
// The moments are formed in fp32 with a fixed order of roundings,
//   m' = rn(rn(b1 m) + rn((1 - b1) g)),  v' = rn(rn(b2 v) + rn((1 - b2) rn(g g))),
// without fused multiply-adds: the 8-bit codes are taken of these values, and
// with 16-bit gradients b1 m + (1 - b1) g is so often a tie of two codes that
// only a stated order makes the codes reproducible.
#include "adamw.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "profile.h"
#include "ptx.cuh"
#include "runtime.h"

namespace mo {

namespace {

constexpr int PER = AW_BLOCK / 32;     // elements of a lane

// A warp's block of a tensor.
struct Block {
  size_t off;        // first element
  int left;          // elements of the block inside the tensor (1..256)
  bool wide;
  int lane;
  __device__ __forceinline__ int at(int j) const { return wide ? lane * PER + j : lane + 32 * j; }
  __device__ __forceinline__ bool has(int j) const { return wide || lane + 32 * j < left; }
};

__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
__device__ __forceinline__ float widen(float x) { return x; }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half narrow<__half>(float x) { return __float2half_rn(x); }

template <typename T>
struct alignas(sizeof(T) * PER) Pack {
  T x[PER];
};

template <typename T>
__device__ __forceinline__ void load_as(float (&x)[PER], const void* p, const Block& b) {
  const T* q = static_cast<const T*>(p) + b.off;
  if (b.wide) {
    const Pack<T> v = *reinterpret_cast<const Pack<T>*>(q + b.lane * PER);
#pragma unroll
    for (int j = 0; j < PER; ++j) x[j] = widen(v.x[j]);
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j) x[j] = b.has(j) ? widen(q[b.at(j)]) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void store_as(const float (&x)[PER], void* p, const Block& b) {
  T* q = static_cast<T*>(p) + b.off;
  if (b.wide) {
    Pack<T> v;
#pragma unroll
    for (int j = 0; j < PER; ++j) v.x[j] = narrow<T>(x[j]);
    *reinterpret_cast<Pack<T>*>(q + b.lane * PER) = v;
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (b.has(j)) q[b.at(j)] = narrow<T>(x[j]);
  }
}

__device__ __forceinline__ void load(float (&x)[PER], const void* p, AwType t, const Block& b) {
  if (t == AW_F32) load_as<float>(x, p, b);
  else if (t == AW_BF16) load_as<__nv_bfloat16>(x, p, b);
  else load_as<__half>(x, p, b);
}

__device__ __forceinline__ void store(const float (&x)[PER], void* p, AwType t, const Block& b) {
  if (t == AW_F32) store_as<float>(x, p, b);
  else if (t == AW_BF16) store_as<__nv_bfloat16>(x, p, b);
  else store_as<__half>(x, p, b);
}

__device__ __forceinline__ void load_codes(unsigned char (&c)[PER], const void* p, const Block& b) {
  const unsigned char* q = static_cast<const unsigned char*>(p) + b.off;
  if (b.wide) {
    const Pack<unsigned char> v = *reinterpret_cast<const Pack<unsigned char>*>(q + b.lane * PER);
#pragma unroll
    for (int j = 0; j < PER; ++j) c[j] = v.x[j];
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j) c[j] = b.has(j) ? q[b.at(j)] : 0;
  }
}

__device__ __forceinline__ void store_codes(const unsigned char (&c)[PER], void* p, const Block& b) {
  unsigned char* q = static_cast<unsigned char*>(p) + b.off;
  if (b.wide) {
    Pack<unsigned char> v;
#pragma unroll
    for (int j = 0; j < PER; ++j) v.x[j] = c[j];
    *reinterpret_cast<Pack<unsigned char>*>(q + b.lane * PER) = v;
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (b.has(j)) q[b.at(j)] = c[j];
  }
}

// Tensor of chunk c (the last one whose first chunk is at most c).
__device__ __forceinline__ int find(const AwTable& tab, unsigned c) {
  int lo = 0, hi = tab.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first[mid] <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ bool block_of(Block& b, const AwTensor& t, unsigned chunk) {
  b.off = (size_t)chunk * AW_CHUNK + (threadIdx.x >> 5) * AW_BLOCK;
  if ((long long)b.off >= t.numel) return false;
  const long long left = t.numel - (long long)b.off;
  b.left = left < AW_BLOCK ? (int)left : AW_BLOCK;
  b.wide = t.vec && b.left == AW_BLOCK;
  b.lane = threadIdx.x & 31;
  return true;
}

// ---------------------------------------------------------------- noise
// Bits for stochastic rounding: a function of (seed, step, place in the
// list, element), the same whatever the launch looks like.  A tensor's two
// 32-bit keys come from a 64-bit mix of the first three; each pair of
// neighbours takes two 32-bit words, 16 bits of each for an element: the
// first for its second moment, the second for a bf16 weight.
struct Keys {
  unsigned k1, k2;
};

__device__ __forceinline__ Keys keys_of(unsigned long long seed, long long step, unsigned index) {
  unsigned long long z = seed + (unsigned long long)step * 0x9E3779B97F4A7C15ull + index * 0xBB67AE8584CAA73Bull;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    z ^= z >> 32;
    z *= 0x6A09E667F3BCC909ull;
  }
  z ^= z >> 32;
  return {(unsigned)z, (unsigned)(z >> 32)};
}

__device__ __forceinline__ unsigned first_word(unsigned long long pair, Keys k) {
  unsigned x = (unsigned)pair ^ k.k1;
  x *= 0x9E3779B9u;
  x ^= x >> 16;
  x = x * 0x6A09E667u + k.k2 + (unsigned)(pair >> 32);
  x ^= x >> 15;
  x *= 0x9E3779B9u;
  return x ^ (x >> 16);
}

__device__ __forceinline__ unsigned second_word(unsigned first, Keys k) {
  const unsigned y = (first ^ k.k1) * 0x6A09E667u + k.k2;
  return y ^ (y >> 16);
}

// ---------------------------------------------------------------- 8-bit moments
// A block of 256 elements shares one scale 2^(s - 127) for each moment, a
// power of two taken from the exponent field E of its largest magnitude, so
// that scaling is exact and a code of an unchanged block stays what it is.
//   m: e4m3, s = max(1, E - 7), nearest-even.
//   v: exponent and mantissa of a float with 5 and 3 bits and no sign,
//      s = max(1, E - 15).  Its range 2^33 is about the square of e4m3's 2^17,
//      as v is of m.  Nearest-even, or stochastic: (1 - b2) (g^2 - v) is far
//      below half a step for the usual b2, and the nearest code would stay
//      where it is.  v > 0 never gets code 0, which would leave eps alone in
//      the denominator; code 255 stands for a value that is not finite.
__device__ __forceinline__ unsigned magnitude(float x) {
  const unsigned u = __float_as_uint(x) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}

// 2^(s - 127) of a scale byte; 2^-127 is subnormal
__device__ __forceinline__ float scale_of(unsigned s) { return __uint_as_float(s ? s << 23 : 0x00400000u); }

__device__ __forceinline__ float first_moment(unsigned char c, float scale) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3);
  return __half2float(__half(h)) * scale;
}

__device__ __forceinline__ float second_moment(unsigned char c, float scale) {
  const float v = __uint_as_float((unsigned)c << 20) * 0x1p112f * scale;
  return c == 255 ? __uint_as_float(0x7fffffffu) : v;
}

// The block's scale bytes, from the warp's largest magnitudes.
__device__ __forceinline__ unsigned scale_byte(const float (&x)[PER], int drop) {
  unsigned big = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) big = max(big, magnitude(x[j]));
  big = __reduce_max_sync(0xffffffffu, big);
  return (unsigned)max(1, (int)(big >> 23) - drop);
}

__device__ __forceinline__ unsigned char first_code(float m, float inv) {
  const float y = m * inv;
  // an infinity has no e4m3 code: y + 0 y makes it a NaN and leaves the rest
  return (unsigned char)__nv_cvt_float_to_fp8(fmaf(y, 0.f, y), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ unsigned char second_code(float v, float inv, int stochastic, unsigned bits) {
  const unsigned u = __float_as_uint(v * inv * 0x1p-112f);
  const unsigned r = u + (stochastic ? bits * 16u + 8u : 0x7ffffu + ((u >> 20) & 1u));
  const unsigned c = v > 0.f ? max(1u, r >> 20) : 0u;
  return (unsigned char)(fabsf(v) < __uint_as_float(0x7f800000u) ? c : 255u);
}

__device__ __forceinline__ void load_moments(float (&m)[PER], float (&v)[PER], const AwTensor& t, const Block& b) {
  unsigned char mc[PER], vc[PER];
  load_codes(mc, t.M, b);
  load_codes(vc, t.V, b);
  const size_t k = b.off / AW_BLOCK;
  const float ms = scale_of(t.MS[k]), vs = scale_of(t.VS[k]);
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    m[j] = first_moment(mc[j], ms);
    v[j] = second_moment(vc[j], vs);
  }
}

__device__ __forceinline__ void store_moments(const float (&m)[PER], const float (&v)[PER], const AwTensor& t,
                                              const Block& b, int stochastic, Keys k) {
  const unsigned ms = scale_byte(m, 7), vs = scale_byte(v, 15);
  const float mi = __uint_as_float((254u - ms) << 23), vi = __uint_as_float((254u - vs) << 23);
  unsigned char mc[PER], vc[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const unsigned long long e = b.off + b.at(j);
    unsigned bits = 0;
    if (stochastic) bits = (first_word(e >> 1, k) >> (16 * (e & 1))) & 0xffffu;
    mc[j] = first_code(m[j], mi);
    vc[j] = second_code(v[j], vi, stochastic, bits);
  }
  store_codes(mc, t.M, b);
  store_codes(vc, t.V, b);
  if (b.lane == 0) {
    const size_t at = b.off / AW_BLOCK;
    t.MS[at] = (unsigned char)ms;
    t.VS[at] = (unsigned char)vs;
  }
}

// ---------------------------------------------------------------- the step
struct Rates {
  float rate, decay, root;
};

__device__ __forceinline__ Rates rates_of(const AwHyper& h, const AwTensor& t) {
  float lr = h.lr, rate = h.rate, root = h.root;
  if (h.lr_dev != nullptr || h.step_dev != nullptr) {
    lr = h.lr_dev ? *h.lr_dev : h.lr;
    rate = lr;
    root = 1.f;
    if (h.bias) {
      // 1 - b^t = -expm1(t log b): fp32 keeps it to 2 ulp for every t
      const float n = (float)(h.step_dev ? *h.step_dev : h.step);
      rate = lr / -expm1f(n * h.log_b1);
      root = rsqrtf(-expm1f(n * h.log_b2));
    }
  }
  return {rate * t.lr_scale, fmaf(-lr * t.lr_scale, t.wd, 1.f), root};
}

__device__ __forceinline__ void update(float (&w)[PER], float (&m)[PER], float (&v)[PER], const float (&g)[PER],
                                       const AwHyper& h, const Rates& r) {
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    m[j] = __fadd_rn(__fmul_rn(h.b1, m[j]), __fmul_rn(h.c1, g[j]));
    v[j] = __fadd_rn(__fmul_rn(h.b2, v[j]), __fmul_rn(h.c2, __fmul_rn(g[j], g[j])));
    const float den = fmaf(sqrtf(v[j]), r.root, h.eps);
    w[j] = fmaf(r.decay, w[j], -(r.rate * m[j]) / den);
  }
}

// bf16 weights without an fp32 master: to the neighbour above with the
// probability of the distance, so that updates below half a step are not lost
__device__ __forceinline__ void round_weights(float (&w)[PER], const Block& b, Keys k) {
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const unsigned long long e = b.off + b.at(j);
    const unsigned bits = (second_word(first_word(e >> 1, k), k) >> (16 * (e & 1))) & 0xffffu;
    const unsigned u = __float_as_uint(w[j]);
    if ((u & 0x7fffffffu) < 0x7f800000u) w[j] = __uint_as_float((u + bits) & 0xffff0000u);
  }
}

template <bool EIGHT>
__global__ void __launch_bounds__(AW_THREADS) adamw_kernel(const __grid_constant__ AwTable tab,
                                                           const __grid_constant__ AwHyper h) {
  pdl_wait();
  pdl_trigger();
  if (h.skip != nullptr && *h.skip != 0) return;
  const float gs = h.gscale ? *h.gscale : 1.f;
  for (unsigned c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const int i = find(tab, c);
    const AwTensor& t = tab.t[i];
    Block b;
    if (!block_of(b, t, c - tab.first[i])) continue;
    float w[PER], g[PER], m[PER], v[PER];
    load(g, t.G, t.gt, b);
    load(w, t.W, t.wt, b);
    if (EIGHT) {
      load_moments(m, v, t, b);
    } else {
      load_as<float>(m, t.M, b);
      load_as<float>(v, t.V, b);
    }
    if (h.gscale != nullptr) {
#pragma unroll
      for (int j = 0; j < PER; ++j) g[j] *= gs;
    }
    update(w, m, v, g, h, rates_of(h, t));
    Keys k = {0, 0};
    if (h.stochastic) k = keys_of(h.seed, h.step_dev ? *h.step_dev : h.step, t.index);
    if (EIGHT) {
      store_moments(m, v, t, b, h.stochastic, k);
    } else {
      store_as<float>(m, t.M, b);
      store_as<float>(v, t.V, b);
    }
    if (t.ct != AW_NONE) store(w, t.C, t.ct, b);
    if (h.stochastic && t.wt == AW_BF16) round_weights(w, b, k);
    store(w, t.W, t.wt, b);
  }
}

__global__ void __launch_bounds__(AW_THREADS) pack_kernel(const __grid_constant__ AwTable tab,
                                                          const __grid_constant__ AwHyper h) {
  pdl_wait();
  pdl_trigger();
  for (unsigned c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const int i = find(tab, c);
    const AwTensor& t = tab.t[i];
    Block b;
    if (!block_of(b, t, c - tab.first[i])) continue;
    float m[PER], v[PER];
    load(m, t.G, t.gt, b);
    load(v, t.C, t.gt, b);
    Keys k = {0, 0};
    if (h.stochastic) k = keys_of(h.seed, h.step_dev ? *h.step_dev : h.step, t.index);
    store_moments(m, v, t, b, h.stochastic, k);
  }
}

__global__ void __launch_bounds__(AW_THREADS) unpack_kernel(const __grid_constant__ AwTable tab) {
  pdl_wait();
  pdl_trigger();
  for (unsigned c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const int i = find(tab, c);
    const AwTensor& t = tab.t[i];
    Block b;
    if (!block_of(b, t, c - tab.first[i])) continue;
    float m[PER], v[PER];
    load_moments(m, v, t, b);
    store(m, t.W, t.wt, b);
    store(v, t.C, t.wt, b);
  }
}

// ---------------------------------------------------------------- clipping
// norm    sum of squares: 8 at a time in fp32, then fp64; one partial sum per
//         CTA, in an order that the grid alone fixes
// finish  the partial sums in a fixed order, the norm and the factor
// scale   out = factor * G
__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sum over the CTA, in thread 0.
__device__ __forceinline__ double cta_sum(double x) {
  __shared__ double red[AW_THREADS / 32];
  x = warp_sum(x);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int k = 0; k < AW_THREADS / 32; ++k) s += red[k];
  }
  return s;
}

__global__ void __launch_bounds__(AW_THREADS) norm_kernel(const __grid_constant__ AwTable tab, double* partial) {
  pdl_wait();
  pdl_trigger();
  double sum = 0.0;
  for (unsigned c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const int i = find(tab, c);
    const AwTensor& t = tab.t[i];
    Block b;
    if (!block_of(b, t, c - tab.first[i])) continue;
    float g[PER];
    load(g, t.G, t.gt, b);
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) s = fmaf(g[j], g[j], s);
    sum += (double)s;
  }
  const double s = cta_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ void __launch_bounds__(AW_THREADS) finish_kernel(const __grid_constant__ ClipArgs a) {
  pdl_wait();
  pdl_trigger();
  double sum = 0.0;
  for (int i = threadIdx.x; i < a.parts; i += AW_THREADS) sum += a.partial[i];
  const double s = cta_sum(sum);
  if (threadIdx.x != 0) return;
  const float scale = a.scale ? *a.scale : 1.f;
  const float norm = (float)(fabs((double)scale) * sqrt(s));
  const float f = a.max_norm / (norm + 1e-6f);
  // a norm that is not a number gives such a factor (1 only where f >= 1)
  *a.norm = norm;
  *a.factor = scale * (f >= 1.f ? 1.f : f);
  if (a.nonfinite) *a.nonfinite = isfinite(norm) ? 0 : 1;
}

__global__ void __launch_bounds__(AW_THREADS) scale_kernel(const __grid_constant__ AwTable tab, const float* factor) {
  pdl_wait();
  pdl_trigger();
  const float f = *factor;
  for (unsigned c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const int i = find(tab, c);
    const AwTensor& t = tab.t[i];
    Block b;
    if (!block_of(b, t, c - tab.first[i])) continue;
    float g[PER];
    load(g, t.G, t.gt, b);
#pragma unroll
    for (int j = 0; j < PER; ++j) g[j] *= f;
    store(g, t.C, t.ct, b);
  }
}

// CTAs of a launch: as many as fit on the card, at most one per chunk.
unsigned grid_of(unsigned chunks, int per_sm) {
  const unsigned most = (unsigned)(device_sm_count() * per_sm);
  return chunks < most ? chunks : most;
}

constexpr int CTAS_PER_SM = 4;

}  // namespace

cudaError_t launch_adamw(const AwTable& t, const AwHyper& h, cudaStream_t s) {
  ProfScope prof(PK_ADAMW, s);
  return launch_pdl(adamw_kernel<false>, dim3(grid_of(t.chunks, CTAS_PER_SM)), dim3(AW_THREADS), 0, s, false, t, h);
}

cudaError_t launch_adamw8(const AwTable& t, const AwHyper& h, cudaStream_t s) {
  ProfScope prof(PK_ADAMW, s);
  return launch_pdl(adamw_kernel<true>, dim3(grid_of(t.chunks, CTAS_PER_SM)), dim3(AW_THREADS), 0, s, false, t, h);
}

cudaError_t launch_pack(const AwTable& t, const AwHyper& h, cudaStream_t s) {
  ProfScope prof(PK_MOMENTS, s);
  return launch_pdl(pack_kernel, dim3(grid_of(t.chunks, CTAS_PER_SM)), dim3(AW_THREADS), 0, s, false, t, h);
}

cudaError_t launch_unpack(const AwTable& t, cudaStream_t s) {
  ProfScope prof(PK_MOMENTS, s);
  return launch_pdl(unpack_kernel, dim3(grid_of(t.chunks, CTAS_PER_SM)), dim3(AW_THREADS), 0, s, false, t);
}

int clip_norm_ctas(unsigned chunks, int most) {
  const unsigned g = grid_of(chunks, CTAS_PER_SM);
  return (int)(g < (unsigned)most ? g : (unsigned)most);
}

cudaError_t launch_clip_norm(const AwTable& t, double* partial, int ctas, cudaStream_t s) {
  ProfScope prof(PK_CLIP, s);
  return launch_pdl(norm_kernel, dim3(ctas), dim3(AW_THREADS), 0, s, false, t, partial);
}

cudaError_t launch_clip_finish(const ClipArgs& a, cudaStream_t s) {
  ProfScope prof(PK_CLIP, s);
  return launch_pdl(finish_kernel, dim3(1), dim3(AW_THREADS), 0, s, false, a);
}

cudaError_t launch_clip_scale(const AwTable& t, const float* factor, cudaStream_t s) {
  ProfScope prof(PK_CLIP, s);
  return launch_pdl(scale_kernel, dim3(grid_of(t.chunks, CTAS_PER_SM)), dim3(AW_THREADS), 0, s, false, t, factor);
}

}  // namespace mo
