// Kernels of the AdamW step over many tensors, of the 8-bit moments and of
// gradient clipping.
//
// A CTA is one warp and works on one 256-element block of a tensor at a time, the
// unit that shares a scale of the 8-bit moments: the scale then needs one warp
// reduction and no shared memory, and a lane holds 8 of the elements in
// registers.  Those are 8 neighbours, read in one access of 32, 16 or 8 bytes;
// misaligned tensors take the aligned words around them (shifted), and blocks at
// a tensor's ends elements 32 apart (narrow), which a warp still reads in a row.
//
// What bounds them, and what they reach (218 M elements, one dense layer; 6.54 TB/s
// is the card's measured copy rate):
//   fp32 moments, fp32 W, bf16 G and copy   28 B an element   901 us   104 % of it
//   8-bit moments, bf16 W and G, noise      10 B              432 us    77 %
//       the same, first moment to nearest                     402 us    83 %
//   8-bit moments, fp32 W, bf16 G, noise    14 B              463 us   101 %
//   unpack to bf16                           6 B              197 us   102 %
//   pack from fp32, noise                   10 B              313 us   107 %
//   norm of bf16 G                           2 B               67 us    99 %
//   clip bf16 into fp32, G read twice        8 B              275 us    97 %
// All are bound by HBM but the 8-bit step of bf16 weights, which needs 67
// instructions an element (57 with the first moment to nearest) and keeps the
// schedulers 88 % busy.
//
// The moments are formed in fp32 with a fixed order of roundings,
//   m' = rn(rn(b1 m) + rn((1 - b1) g)),  v' = rn(rn(b2 v) + rn((1 - b2) rn(g g))),
// without fused multiply-adds: the 8-bit codes are taken of these values, and
// with 16-bit gradients b1 m + (1 - b1) g is so often a tie of two codes that
// only a stated order makes the codes reproducible.  (Packed fp32x2 instructions
// are not used for them: ptxas 12.9 joins mul.rn.f32x2 and add.rn.f32x2 into one
// rounding, and with separate sums the step was as fast as without.)
#include "adamw.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>
#include <utility>

#include "profile.h"
#include "ptx.cuh"
#include "runtime.h"

namespace mo {

namespace {

constexpr int PER = AW_BLOCK / 32;     // elements of a lane
// CTAs (warps) of a step on one SM, the same number for each of its four
// schedulers (with one warp more than the others, a scheduler finishes last: 21
// were as slow as 24 would be).  fp32 moments: 20 at 96 registers, 8 bits and
// shifted: 28 at 72 (50 M bf16 elements: 99 us; 24: 102, 32: 105).  At these limits
// ptxas spills 8 to 36 bytes of the fp32 step with bf16 weights or fp32
// gradients, 8 of some shifted 8-bit ones and none of the aligned 8-bit step.
constexpr int STEP32_CTAS = 20;
constexpr int STEP8_CTAS = 28;

// A lane's place in a block: wide lanes (1) and shifted ones (2) hold 8
// neighbours, narrow ones (0) elements 32 apart.
template <int WIDE>
struct Place {
  unsigned long long first;   // the lane's first element
  int left;                   // narrow: elements of the tensor from there on
  __device__ __forceinline__ bool has(int j) const { return WIDE || 32 * j < left; }
};

// Conditions that hold for few blocks: their code goes out of the way.
__device__ __forceinline__ bool rare(bool x) { return __builtin_expect(x, 0); }

__device__ __forceinline__ void scale_all(float (&x)[PER], float f) {
#pragma unroll
  for (int j = 0; j < PER; ++j) x[j] *= f;
}

// ---------------------------------------------------------------- loads and stores
using Code = unsigned char;            // of an 8-bit moment

// A lane's 8 elements of a tensor as they are stored, 16-bit ones two and codes
// four to a word.
template <typename T>
struct Raw {
  static constexpr int WORDS = PER * sizeof(T) / 4;
  unsigned w[WORDS];
  uint4 behind;                // shifted: the 16 bytes behind
};

__device__ __forceinline__ unsigned bits_of(float x) { return __float_as_uint(x); }
__device__ __forceinline__ unsigned bits_of(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }
__device__ __forceinline__ unsigned bits_of(unsigned char x) { return x; }
__device__ __forceinline__ unsigned bits_of(__half x) { return __half_as_ushort(x); }

// One access of 32 or 16 bytes (two of 16 for fp32 would each touch half of
// every 32-byte sector), `AT` bytes behind p.
template <int AT>
__device__ __forceinline__ void load_words(unsigned (&w)[8], const void* p) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8 + %9];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p), "n"(AT)
               : "memory");
}
template <int AT>
__device__ __forceinline__ void load_words(unsigned (&w)[4], const void* p) {
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4 + %5];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "l"(p), "n"(AT)
               : "memory");
}
template <int AT>
__device__ __forceinline__ void load_words(unsigned (&w)[2], const void* p) {
  asm volatile("ld.global.v2.b32 {%0, %1}, [%2 + %3];" : "=r"(w[0]), "=r"(w[1]) : "l"(p), "n"(AT) : "memory");
}
__device__ __forceinline__ void store_words(const unsigned (&w)[8], void* p) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void store_words(const unsigned (&w)[4], void* p) {
  asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}
__device__ __forceinline__ void store_words(const unsigned (&w)[2], void* p) {
  asm volatile("st.global.v2.b32 [%0], {%1, %2};" ::"l"(p), "r"(w[0]), "r"(w[1]) : "memory");
}

// Asks the block behind p's into L2.
template <typename T>
__device__ __forceinline__ void ask_next(const T* p) {
  asm volatile("prefetch.global.L2 [%0 + %1];" ::"l"(p), "n"(AW_BLOCK * (int)sizeof(T)));
}

// Shifted accesses: 8 neighbours of a lane at an address that is aligned to its
// elements alone.  A lane reads the 16-byte words that its elements begin in and
// the one behind, which L1 holds for the next lane; it writes the words that
// begin before its elements' end, with what the lane before has of them.  The
// words at the two ends of a block hold elements of its neighbours too, so those
// are written by elements.  What is read before a tensor's first element is in
// the same 16 bytes and so in the same allocation; behind its last one that need
// not be, so a block goes this way only where 8 elements of the tensor follow it.  54 M elements at odd offsets:
// 8-bit step and unpacking 199 us, element by element 307, aligned 155; clipping
// 78, 100 and 68.
template <int BY>
__device__ __forceinline__ void shift_words(unsigned (&w)[8], const unsigned (&c)[12]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = c[k + BY];
}

template <int BY>
__device__ __forceinline__ void shift_words(unsigned (&w)[4], const unsigned (&c)[8], unsigned bits) {
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(c[k + BY], c[k + BY + 1], bits);
}

// The aligned words around a lane's elements ...
template <int WORDS>
__device__ __forceinline__ void load_around(unsigned (&w)[WORDS], uint4& behind, const void* p) {
  const unsigned d = (unsigned)(reinterpret_cast<uintptr_t>(p) & 15u);
  const uint4* a = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - d);
#pragma unroll
  for (int k = 0; k < WORDS / 4; ++k) {
    const uint4 x = a[k];
    w[4 * k] = x.x;
    w[4 * k + 1] = x.y;
    w[4 * k + 2] = x.z;
    w[4 * k + 3] = x.w;
  }
  behind = make_uint4(0, 0, 0, 0);
  if (d != 0) behind = a[WORDS / 4];
}

// ... and the elements out of them.
__device__ __forceinline__ void settle(unsigned (&w)[8], const uint4& z, const void* p) {
  const unsigned d = (unsigned)(reinterpret_cast<uintptr_t>(p) & 15u);
  const unsigned c[12] = {w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7], z.x, z.y, z.z, z.w};
  switch (d >> 2) {
    case 0: shift_words<0>(w, c); break;
    case 1: shift_words<1>(w, c); break;
    case 2: shift_words<2>(w, c); break;
    default: shift_words<3>(w, c); break;
  }
}

__device__ __forceinline__ void settle(unsigned (&w)[4], const uint4& z, const void* p) {
  const unsigned d = (unsigned)(reinterpret_cast<uintptr_t>(p) & 15u);
  const unsigned c[8] = {w[0], w[1], w[2], w[3], z.x, z.y, z.z, z.w};
  const unsigned bits = (d & 2u) * 8u;
  switch (d >> 2) {
    case 0: shift_words<0>(w, c, bits); break;
    case 1: shift_words<1>(w, c, bits); break;
    case 2: shift_words<2>(w, c, bits); break;
    default: shift_words<3>(w, c, bits); break;
  }
}

// A fetched lane's elements in order: nothing to do unless they came shifted.
template <int WIDE, typename T>
__device__ __forceinline__ Raw<T> settled(const Raw<T>& r, const T* p) {
  Raw<T> s = r;
  if constexpr (WIDE == 2 && sizeof(T) > 1) settle(s.w, s.behind, p);
  return s;
}

__device__ __forceinline__ unsigned up(unsigned x) { return __shfl_up_sync(0xffffffffu, x, 1); }

template <int BY>
__device__ __forceinline__ void put_shifted(const unsigned (&w)[8], const unsigned (&before)[8], unsigned* p) {
  unsigned o[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) o[k] = k < BY ? before[8 - BY + k] : w[k - BY];
  uint4* a = reinterpret_cast<uint4*>(p - BY);
  if (threadIdx.x != 0 || BY == 0) {
    a[0] = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4 - BY; ++k) p[k] = w[k];
  }
  a[1] = make_uint4(o[4], o[5], o[6], o[7]);
  if (threadIdx.x == 31) {
#pragma unroll
    for (int k = 8 - BY; k < 8; ++k) p[k] = w[k];
  }
}

__device__ __forceinline__ void store_shifted(const unsigned (&w)[8], void* to) {
  unsigned* p = static_cast<unsigned*>(to);
  unsigned before[8] = {};
#pragma unroll
  for (int k = 5; k < 8; ++k) before[k] = up(w[k]);
  switch ((reinterpret_cast<uintptr_t>(p) >> 2) & 3u) {
    case 0: put_shifted<0>(w, before, p); break;
    case 1: put_shifted<1>(w, before, p); break;
    case 2: put_shifted<2>(w, before, p); break;
    default: put_shifted<3>(w, before, p); break;
  }
}

template <int BY>
__device__ __forceinline__ void shift_up(unsigned (&o)[4], const unsigned (&c)[8], bool odd) {
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = odd ? __funnelshift_l(c[3 + k - BY], c[4 + k - BY], 16) : c[4 + k - BY];
}

__device__ __forceinline__ void store_shifted(const unsigned (&w)[4], void* to) {
  unsigned short* p = static_cast<unsigned short*>(to);
  const int by = (int)(reinterpret_cast<uintptr_t>(p) >> 1) & 7;       // elements
  const unsigned c[8] = {up(w[0]), up(w[1]), up(w[2]), up(w[3]), w[0], w[1], w[2], w[3]};
  unsigned o[4];
  switch (by >> 1) {
    case 0: shift_up<0>(o, c, by & 1); break;
    case 1: shift_up<1>(o, c, by & 1); break;
    case 2: shift_up<2>(o, c, by & 1); break;
    default: shift_up<3>(o, c, by & 1); break;
  }
  if (threadIdx.x != 0 || by == 0) *reinterpret_cast<uint4*>(p - by) = make_uint4(o[0], o[1], o[2], o[3]);
  if (by != 0 && (threadIdx.x == 0 || threadIdx.x == 31)) {
    // the first lane's elements in the word that the block begins in, the last lane's in the one behind
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if ((j < PER - by) == (threadIdx.x == 0)) p[j] = (unsigned short)(w[j / 2] >> (16 * (j % 2)));
  }
}

// p is the lane's first element; a wide lane may read AT blocks further on.
template <int WIDE, int AT = 0, typename T>
__device__ __forceinline__ void fetch(Raw<T>& r, const T* p, const Place<WIDE>& b) {
  if constexpr (WIDE == 2 && sizeof(T) > 1) {
    load_around(r.w, r.behind, p + AT * AW_BLOCK);
  } else if constexpr (WIDE > 0) {
    load_words<AT * AW_BLOCK * (int)sizeof(T)>(r.w, p);
  } else {
    constexpr int IN = 4 / sizeof(T);                  // elements of a word
#pragma unroll
    for (int k = 0; k < Raw<T>::WORDS; ++k) {
      r.w[k] = 0;
#pragma unroll
      for (int j = IN * k; j < IN * (k + 1); ++j)
        if (b.has(j)) r.w[k] |= bits_of(p[32 * j]) << (8 * sizeof(T) * (j % IN));
    }
  }
}

template <int WIDE, typename T>
__device__ __forceinline__ void put(const Raw<T>& r, T* p, const Place<WIDE>& b) {
  if constexpr (WIDE == 2 && sizeof(T) > 1) {
    store_shifted(r.w, p);
  } else if constexpr (WIDE > 0) {
    store_words(r.w, p);
  } else {
    constexpr int IN = 4 / sizeof(T);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (!b.has(j)) continue;
      const unsigned x = r.w[j / IN] >> (8 * sizeof(T) * (j % IN));
      if (IN == 1) reinterpret_cast<unsigned*>(p)[32 * j] = x;
      else if (IN == 2) reinterpret_cast<unsigned short*>(p)[32 * j] = (unsigned short)x;
      else reinterpret_cast<unsigned char*>(p)[32 * j] = (unsigned char)x;
    }
  }
}

__device__ __forceinline__ void widen_all(float (&x)[PER], const Raw<float>& r) {
#pragma unroll
  for (int j = 0; j < PER; ++j) x[j] = __uint_as_float(r.w[j]);
}
__device__ __forceinline__ void widen_all(float (&x)[PER], const Raw<__nv_bfloat16>& r) {
#pragma unroll
  for (int q = 0; q < PER / 2; ++q) {
    x[2 * q] = __uint_as_float(r.w[q] << 16);
    x[2 * q + 1] = __uint_as_float(r.w[q] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen_all(float (&x)[PER], const Raw<__half>& r) {
#pragma unroll
  for (int q = 0; q < PER / 2; ++q) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[q]));
    x[2 * q] = f.x;
    x[2 * q + 1] = f.y;
  }
}

__device__ __forceinline__ void narrow_all(Raw<float>& r, const float (&x)[PER]) {
#pragma unroll
  for (int j = 0; j < PER; ++j) r.w[j] = __float_as_uint(x[j]);
}
__device__ __forceinline__ void narrow_all(Raw<__nv_bfloat16>& r, const float (&x)[PER]) {
#pragma unroll
  for (int q = 0; q < PER / 2; ++q) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * q], x[2 * q + 1]);
    r.w[q] = *reinterpret_cast<const unsigned*>(&h);
  }
}
__device__ __forceinline__ void narrow_all(Raw<__half>& r, const float (&x)[PER]) {
#pragma unroll
  for (int q = 0; q < PER / 2; ++q) {
    const __half2 h = __floats2half2_rn(x[2 * q], x[2 * q + 1]);
    r.w[q] = *reinterpret_cast<const unsigned*>(&h);
  }
}

template <int WIDE, typename T>
__device__ __forceinline__ void store(const float (&x)[PER], T* p, const Place<WIDE>& b) {
  Raw<T> r;
  narrow_all(r, x);
  put(r, p, b);
}

// ---------------------------------------------------------------- the list
// Tensor that holds run `run` of the list, none before tensor i.
template <int N>
__device__ __forceinline__ int find(const AwTableOf<N>& tab, unsigned run, int i) {
  if (i + 1 == tab.n || run < tab.t[i + 1].first) return i;
  int lo = i + 1, hi = tab.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.t[mid].first <= run) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <int WIDE, typename Op, int... K>
__device__ __forceinline__ void fetch_all(const Op& op, typename Op::Load (&in)[sizeof...(K)], unsigned at,
                                          std::integer_sequence<int, K...>) {
  (op.template fetch<K, WIDE>(in[K], at), ...);
}

// The first `end` blocks of a run, by what an Op asks for:
//   BATCH n > 0   n blocks are fetched and then worked on
//   BATCH 0       a block is fetched while the one before is worked on, in two
//                 buffers and two copies of the body so that nothing moves between
//                 them (shifted accesses need too many registers for that: as 1)
//   AHEAD         the next block is asked into L2: fewer registers and a shorter
//                 body than with two buffers
template <int WIDE, typename Op>
__device__ __forceinline__ void work_blocks(Op& op, unsigned long long first, int end) {
  unsigned at = threadIdx.x * PER;
  int r = 0;
  const auto work = [&](const typename Op::Load& in) {
    op.work(in, Place<WIDE>{first + at, 0}, at, r);
    at += AW_BLOCK;
    ++r;
  };
  constexpr int BATCH = Op::BATCH == 0 && WIDE == 2 ? 1 : Op::BATCH;
  if constexpr (BATCH > 0) {
    while (BATCH > 1 && r + BATCH <= end) {
      typename Op::Load in[BATCH];
      fetch_all<WIDE>(op, in, at, std::make_integer_sequence<int, BATCH>());
#pragma unroll
      for (int k = 0; k < BATCH; ++k) work(in[k]);
    }
    while (r < end) {
      typename Op::Load in;
      op.template fetch<0, WIDE>(in, at);
      if constexpr (Op::AHEAD)
        if (r + 1 < end) op.ask(at);
      work(in);
    }
  } else if (r < end) {
    typename Op::Load even, odd;
    op.template fetch<0, WIDE>(even, at);
    while (true) {
      if (r + 1 < end) op.template fetch<1, WIDE>(odd, at);
      work(even);
      if (r == end) break;
      if (r + 1 < end) op.template fetch<1, WIDE>(even, at);
      work(odd);
      if (r == end) break;
    }
  }
}

// A CTA is one warp.  It takes every gridDim-th run of tab.run blocks of a
// tensor.
//   Op::start(tensor, first element, blocks)   a run begins
//   Op::fetch<AT>(Load&, at)                   reads a whole block, AT blocks behind the lane's offset `at`
//   Op::work(Load, Place, at, r)               works on block r of the run
//   Op::narrow(tensor, Place, at, r)           reads and works on a partial block r, or one that has no other way
//   Op::finish(blocks)                         the run ends
// With VEC all tensors are aligned; without, their blocks are read shifted
// where that is possible (t.vec), and narrow at their ends.
template <bool VEC, int N, typename Op>
__device__ __forceinline__ void walk(const AwTableOf<N>& tab, Op& op) {
  const unsigned lane = threadIdx.x;
  int i = 0;
  for (unsigned turn = blockIdx.x; turn < tab.runs; turn += gridDim.x) {
    const unsigned run = Op::BACKWARDS ? tab.runs - 1 - turn : turn;
    i = find(tab, run, Op::BACKWARDS ? 0 : i);
    const AwTensor& t = tab.t[i];
    const long long block = (long long)(run - t.first) * tab.run;
    const unsigned long long first = (unsigned long long)block * AW_BLOCK;
    const int blocks = (int)min((long long)tab.run, (t.numel + AW_BLOCK - 1) / AW_BLOCK - block);
    // the whole blocks (VEC), or those with 8 elements behind them
    int whole = 0;
    if (VEC) whole = (int)min((long long)blocks, t.numel / AW_BLOCK - block);
    else if (t.vec) whole = (int)max(0ll, min((long long)blocks, (t.numel - 8) / AW_BLOCK - block));
    op.start(t, first, blocks);
    work_blocks<VEC ? 1 : 2>(op, first, whole);
    for (int r = whole; r < blocks; ++r) {
      const unsigned at = (unsigned)r * AW_BLOCK + lane;
      const long long left = t.numel - (long long)(first + at);
      op.narrow(t, Place<0>{first + at, left < AW_BLOCK ? (int)left : AW_BLOCK}, at, r);
    }
    op.finish(blocks);
  }
}

// ---------------------------------------------------------------- noise
// Bits for stochastic rounding: a function of (seed, step, place in the
// list, element), the same whatever the launch looks like.  A tensor's two
// 32-bit keys come from a 64-bit mix of the first three; each pair of
// neighbours takes three 32-bit words, 16 bits of each for an element: the
// first for its second moment, the second for a bf16 weight, the third for its
// first moment.
struct Keys {
  unsigned k1, k2;
};

__device__ __forceinline__ Keys keys_of(const AwHyper& h, unsigned index) {
  const unsigned long long step = (unsigned long long)(h.step_dev ? *h.step_dev : h.step);
  unsigned long long z = h.seed + step * 0x9E3779B97F4A7C15ull + index * 0xBB67AE8584CAA73Bull;
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
  x = x * 0x6A09E667u + (k.k2 + (unsigned)(pair >> 32));
  x ^= x >> 15;
  x *= 0x9E3779B9u;
  return x ^ (x >> 16);
}

__device__ __forceinline__ unsigned second_word(unsigned first, Keys k) {
  const unsigned y = (first ^ k.k1) * 0x6A09E667u + k.k2;
  return y ^ (y >> 16);
}

__device__ __forceinline__ unsigned third_word(unsigned first, Keys k) {
  const unsigned z = (first ^ k.k2) * 0x9E3779B9u + k.k1;
  return z ^ (z >> 16);
}

// The first words that a lane's elements need: wide lanes hold whole pairs,
// narrow ones an element of each.
template <int WIDE>
struct Noise {
  unsigned w[WIDE ? PER / 2 : PER];
  __device__ __forceinline__ void draw(const Place<WIDE>& b, Keys k) {
    const unsigned long long base = b.first >> 1;
#pragma unroll
    for (int q = 0; q < (WIDE ? PER / 2 : PER); ++q) w[q] = first_word(base + (WIDE ? q : 16 * q), k);
  }
  __device__ __forceinline__ Noise second(Keys k) const {
    Noise n;
#pragma unroll
    for (int q = 0; q < (WIDE ? PER / 2 : PER); ++q) n.w[q] = second_word(w[q], k);
    return n;
  }
  __device__ __forceinline__ Noise third(Keys k) const {
    Noise n;
#pragma unroll
    for (int q = 0; q < (WIDE ? PER / 2 : PER); ++q) n.w[q] = third_word(w[q], k);
    return n;
  }
  // Element j's 16 bits; and those with a half behind them in bits 7 to 23.  By
  // shifts and masks: made by byte permutations and packed by pack_tops they gave every v
  // of pack_kernel the code 1 (nvcc 12.9; why was not found).  The tests hold
  // the codes of this form to those of the definition, bit for bit.
  __device__ __forceinline__ unsigned bits16(int j) const {
    return (WIDE ? j : threadIdx.x) % 2 ? w[WIDE ? j / 2 : j] >> 16 : w[WIDE ? j / 2 : j] & 0xffffu;
  }
  __device__ __forceinline__ unsigned bits24(int j) const {
    const unsigned x = w[WIDE ? j / 2 : j];
    return (((WIDE ? j : threadIdx.x) % 2 ? x >> 8 : x << 8) & 0xffff00u) | 0x80u;
  }
};

// ---------------------------------------------------------------- 8-bit moments
// A block of 256 elements shares one scale 2^(s - 127) for each moment, a
// power of two taken from the exponent field E of its largest magnitude, so
// that scaling is exact and a code of an unchanged block stays what it is.
//   m: e4m3, s = max(1, E - 7).  Nearest-even, or stochastic (FIRST): a code step
//      is 6 to 12 % of m, and a step moves m by (1 - b1) (g - m).  Without a
//      gradient and with b1 = 0.95 the nearest code of 9 and 10 eighths is again 9
//      and 10: m stays for ever, v goes on sinking and the weights run away.
//   v: exponent and mantissa of a float with 5 and 3 bits and no sign,
//      s = max(1, E - 15).  Its range 2^33 is about the square of e4m3's 2^17,
//      as v is of m.  Nearest-even, or stochastic: (1 - b2) (g^2 - v) is far
//      below half a step for the usual b2, and the nearest code would stay
//      where it is.  v > 0 never gets code 0, which would leave eps alone in
//      the denominator; code 255 stands for a value that is not finite.
// An fp32 value times 2^(127 - s) 2^-112 has v's code in bits 20 to 27, its
// subnormals included, and what is rounded off below them; times
// 2^(127 - s) 2^-120 it has m's in bits 20 to 26, below its sign.  Noise is added
// there (16 bits and a half behind them), which is unbiased to 2^-17 of a code step.
// m's noise costs the step of 50 M elements 7 us with bf16 weights (106; v's alone
// 99, none 87) and nothing with fp32 ones (114), where HBM is the bound.
constexpr unsigned INF_BITS = 0x7f800000u;
constexpr unsigned HIGH_BITS = 0x4e000000u;   // 2^29: below, v's scale is at most 2^14
constexpr unsigned FIRST_HIGH_BITS = 0x46000000u;   // 2^13: below, m's scale is at most 2^5

// 2^(s - 127) of a scale byte; 2^-127 is subnormal
__device__ __forceinline__ float scale_of(unsigned s) { return __uint_as_float(s ? s << 23 : 0x00400000u); }
// Whether one of four codes of v is 248 or above.
__device__ __forceinline__ bool has_high(unsigned w) {
  const unsigned t = ~w & 0xf8f8f8f8u;
  return ((t - 0x01010101u) & ~t & 0x80808080u) != 0;
}

// Moments of a lane's codes, to be scaled.
__device__ __forceinline__ void decode(float (&m)[PER], float (&v)[PER], const Raw<Code>& mc, const Raw<Code>& vc) {
#pragma unroll
  for (int q = 0; q < PER / 2; ++q) {
    const unsigned pair = q % 2 ? mc.w[q / 2] >> 16 : mc.w[q / 2] & 0xffffu;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)pair, __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    m[2 * q] = f.x;
    m[2 * q + 1] = f.y;
  }
  // v's codes below 248 are the upper bits of an fp16 number without its sign
#pragma unroll
  for (int q = 0; q < PER / 2; ++q) {
    const unsigned w = vc.w[q / 2];
    const unsigned h = (q % 2 ? __byte_perm(w, 0, 0x4342) : __byte_perm(w, 0, 0x4140)) << 7;
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * q] = f.x;
    v[2 * q + 1] = f.y;
  }
  if (rare(has_high(vc.w[0]) || has_high(vc.w[1]))) {
    // 248 is 2^16, which a block's largest value may round up to; 255 is a NaN
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const unsigned c = (vc.w[j / 4] >> (8 * (j % 4))) & 0xffu;
      v[j] = c == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(c << 20) * 0x1p112f;
    }
  }
}

// The scale bytes of a run, m's below v's, block r's in lane r: they are read
// and written once for a run.  A byte at a time, reads of a 32-byte sector that
// waits for other bytes made the step 1.5 times as long (218 M bf16 elements:
// 975 us, and 615 without the stores).
struct Scales {
  unsigned all;
  __device__ __forceinline__ void load(const Code* ms, const Code* vs, int blocks) {
    all = 0;
    if ((int)threadIdx.x < blocks) all = ms[threadIdx.x] | (unsigned)vs[threadIdx.x] << 8;
  }
  __device__ __forceinline__ unsigned of(int r) const { return __shfl_sync(0xffffffffu, all, r); }
  __device__ __forceinline__ void set(int r, unsigned ms, unsigned vs) {
    if ((int)threadIdx.x == r) all = ms | vs << 8;
  }
  __device__ __forceinline__ void store(Code* ms, Code* vs, int blocks) const {
    if ((int)threadIdx.x < blocks) {
      ms[threadIdx.x] = (Code)all;
      vs[threadIdx.x] = (Code)(all >> 8);
    }
  }
};

__device__ __forceinline__ unsigned pack_tops(unsigned a, unsigned b, unsigned c, unsigned d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// Codes of v in bits 24 to 31 of r; vi is 2^(127 - s) 2^-112 of what v is in.  A
// subnormal product is cut off, which the noise does not see (see first_codes).  To
// nearest it must not be rounded before the code is: codes up to 8, which are the
// whole numbers of steps of 2^(s - 127) 2^-17, are formed again by a conversion.
template <bool STOCHASTIC, int WIDE>
__device__ __forceinline__ void second_codes(unsigned (&r)[PER], const float (&v)[PER], float vi, const Noise<WIDE>& n) {
  unsigned least = 0xffffffffu;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const unsigned u = __float_as_uint(__fmul_rz(v[j], vi));
    r[j] = STOCHASTIC ? u * 16u + n.bits24(j) : (u + 0x7ffffu + ((u >> 20) & 1u)) * 16u;
    least = min(least, r[j]);
  }
  if (rare(least < (STOCHASTIC ? 1u << 24 : 9u << 24))) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (!STOCHASTIC && r[j] < (9u << 24)) r[j] = __float2uint_rn(v[j] * (vi * 0x1p112f) * 0x1p17f) << 24;
      if (v[j] > 0.f && r[j] < (1u << 24)) r[j] = 1u << 24;
    }
  }
}

// Stochastic codes of m in bits 24 to 31 of r; mi is 2^(127 - s) 2^-120 of what m
// is in.  What falls below the last bit of a subnormal product is cut off: the noise is a
// whole number of these bits, so that it decides nothing.
template <int WIDE>
__device__ __forceinline__ void first_codes(unsigned (&r)[PER], const float (&m)[PER], float mi, const Noise<WIDE>& n) {
  unsigned any = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const unsigned u = __float_as_uint(__fmul_rz(m[j], mi));
    any |= u;
    r[j] = (u * 16u + n.bits24(j)) | (u & 0x80000000u);
  }
  if (rare((any & 0x78000000u) != 0)) {                // numbers stay below 2^-112 here
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (!(fabsf(m[j]) < __uint_as_float(INF_BITS))) r[j] = 127u << 24;
  }
}

// FIRST: both moments by noise; else m to nearest and v as `stochastic` says.
template <bool FIRST, int WIDE>
__device__ __forceinline__ void store_moments(float (&m)[PER], float (&v)[PER], Code* mp, Code* vp, Scales& scales, int r,
                                              const Place<WIDE>& b, bool stochastic, const Noise<WIDE>& n, Keys k) {
  float bm = 0.f;
  unsigned bv = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    bm = fmaxf(bm, fabsf(m[j]));                       // leaves NaN out
    bv = max(bv, __float_as_uint(v[j]));               // infinite, NaN and negative values come out largest
  }
  unsigned um = __reduce_max_sync(0xffffffffu, __float_as_uint(bm));
  unsigned uv = __reduce_max_sync(0xffffffffu, bv);
  unsigned odd = 0;                                    // elements whose v has code 255
  unsigned ms, vs;
  float mi, vi;       // 2^(127 - s) 2^-120 (FIRST) and 2^(127 - s) 2^-112, normal numbers below FIRST_HIGH_BITS and HIGH_BITS
  if (!rare(um >= (FIRST ? FIRST_HIGH_BITS : INF_BITS) || uv >= HIGH_BITS)) {
    ms = max(1, (int)(um >> 23) - 7);
    mi = __uint_as_float(((FIRST ? 134u : 254u) - ms) << 23);
    vs = max(1, (int)(uv >> 23) - 15);
    vi = __uint_as_float((142u - vs) << 23);
  } else {
    // the scale is that of the finite values; an infinite m has no code and becomes a NaN
    um = uv = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const unsigned a = __float_as_uint(fabsf(m[j])), c = __float_as_uint(fabsf(v[j]));
      if (a < INF_BITS) um = max(um, a); else m[j] = __uint_as_float(0x7fffffffu);
      if (c < INF_BITS) uv = max(uv, c); else odd |= 1u << j;
      if (c >= INF_BITS || v[j] < 0.f) v[j] = 0.f;
    }
    um = __reduce_max_sync(0xffffffffu, um);
    uv = __reduce_max_sync(0xffffffffu, uv);
    ms = max(1, (int)(um >> 23) - 7);
    vs = max(1, (int)(uv >> 23) - 15);
    // scaled in two steps: what the first cuts off below 2^-126 is far below any code, but it stays above 0
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (v[j] > 0.f) v[j] = fmaxf(v[j] * __uint_as_float((254u - vs) << 23), 0x1p-149f);
    vi = 0x1p-112f;
    mi = __uint_as_float((254u - ms) << 23);
    if constexpr (FIRST) {
      scale_all(m, mi);
      mi = 0x1p-120f;
    }
  }
  unsigned mw[PER / 4], vr[PER];                       // four codes of m to a word
  if constexpr (FIRST) {
    unsigned mr[PER];
    first_codes(mr, m, mi, n.third(k));
#pragma unroll
    for (int q = 0; q < PER / 4; ++q) mw[q] = pack_tops(mr[4 * q], mr[4 * q + 1], mr[4 * q + 2], mr[4 * q + 3]);
  } else {
    scale_all(m, mi);
    const auto pair = [&](int j) {
      return (unsigned)__nv_cvt_float2_to_fp8x2(make_float2(m[j], m[j + 1]), __NV_SATFINITE, __NV_E4M3);
    };
#pragma unroll
    for (int q = 0; q < PER / 4; ++q) mw[q] = __byte_perm(pair(4 * q), pair(4 * q + 2), 0x5410);
  }
  if (FIRST || stochastic) second_codes<true>(vr, v, vi, n);
  else second_codes<false>(vr, v, vi, n);
  if (rare(odd != 0)) {
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (odd & (1u << j)) vr[j] = 255u << 24;
  }
  put(Raw<Code>{{mw[0], mw[1]}, {}}, mp, b);
  put(Raw<Code>{{pack_tops(vr[0], vr[1], vr[2], vr[3]), pack_tops(vr[4], vr[5], vr[6], vr[7])}, {}}, vp, b);
  scales.set(r, ms, vs);
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

// sqrt and reciprocal of the special-function unit (2^-23 relative each): the
// update they scale is a small part of the weight.  The
// forms that take subnormal numbers as zeros need two instructions, the others
// ten; they change a denominator by less than 2^-63 root, which is below 2^-26 of
// an eps of 2^-37 root or more, and have no reciprocal for denominators above
// 2^126, which sqrt(v) root (2^64 2^27 at most) does not reach.
template <bool TINY>
__device__ __forceinline__ float sqrt_fast(float x) {
  float r;
  if (TINY) asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  else asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
template <bool TINY>
__device__ __forceinline__ float reciprocal_fast(float x) {
  float r;
  if (TINY) asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  else asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <bool TINY>
__device__ __forceinline__ void new_weights(float (&w)[PER], const float (&m)[PER], const float (&v)[PER], const Rates& r,
                                            float eps) {
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const float den = fmaf(sqrt_fast<TINY>(v[j]), r.root, eps);
    w[j] = fmaf(r.decay, w[j], -(r.rate * m[j]) * reciprocal_fast<TINY>(den));
  }
}

// m and v come in units of the scales ms and vs, powers of two that the
// constants take up exactly (fp32 moments: 1).
__device__ __forceinline__ void update(float (&w)[PER], float (&m)[PER], float (&v)[PER], const float (&g)[PER],
                                       const AwHyper& h, const Rates& r, float ms, float vs) {
  const float b1 = h.b1 * ms, b2 = h.b2 * vs;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    m[j] = __fadd_rn(__fmul_rn(b1, m[j]), __fmul_rn(h.c1, g[j]));
    v[j] = __fadd_rn(__fmul_rn(b2, v[j]), __fmul_rn(h.c2, __fmul_rn(g[j], g[j])));
  }
  if (rare(!(h.eps >= 0x1p-37f * r.root && h.eps <= 0x1p100f))) new_weights<true>(w, m, v, r, h.eps);
  else new_weights<false>(w, m, v, r, h.eps);
}

// bf16 weights without an fp32 master: to the neighbour above with the
// probability of the distance, so that updates below half a step are not lost
template <int WIDE>
__device__ __forceinline__ void round_weights(Raw<__nv_bfloat16>& out, const float (&w)[PER], const Noise<WIDE>& n) {
  float zero = 0.f;                                    // NaN when a weight is not finite
#pragma unroll
  for (int j = 0; j < PER; ++j) zero = fmaf(w[j], 0.f, zero);
  unsigned u[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) u[j] = __float_as_uint(w[j]) + n.bits16(j);
  if (rare(zero != 0.f)) {                                   // the sum may have made a number of a NaN
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (!(fabsf(w[j]) < __uint_as_float(INF_BITS))) u[j] = __float_as_uint(w[j]);
  }
#pragma unroll
  for (int q = 0; q < PER / 2; ++q) out.w[q] = __byte_perm(u[2 * q], u[2 * q + 1], 0x7632);
}

template <bool EIGHT, typename WT, typename GT>
struct StepLoad {
  using Moment = typename std::conditional<EIGHT, Code, float>::type;
  Raw<WT> w;
  Raw<GT> g;
  Raw<Moment> m, v;
};

// What a tensor's elements share in a step.
struct Shared {
  Rates r;
  Keys k;
  AwType ct;
  __device__ __forceinline__ void start(const AwHyper& h, const AwTensor& t) {
    r = rates_of(h, t);
    if (h.stochastic) k = keys_of(h, t.index);
    ct = t.ct;
  }
};

__device__ __forceinline__ void moments_of(float (&m)[PER], float (&v)[PER], const Raw<float>& mr, const Raw<float>& vr, float&,
                                           float&, unsigned, unsigned) {
  widen_all(m, mr);
  widen_all(v, vr);
}
__device__ __forceinline__ void moments_of(float (&m)[PER], float (&v)[PER], const Raw<Code>& mc, const Raw<Code>& vc, float& ms,
                                           float& vs, unsigned scales, unsigned least) {
  decode(m, v, mc, vc);
  const unsigned msb = scales & 0xffu, vsb = scales >> 8;
  ms = scale_of(msb);
  vs = scale_of(vsb);
  if (rare(min(msb, vsb) < least)) {
    // b1 ms or b2 vs may be subnormal and not exact: scale the moments themselves
    scale_all(m, ms);
    scale_all(v, vs);
    ms = vs = 1.f;
  }
}

template <bool EIGHT, bool FIRST, typename WT, typename GT>
struct StepOp {
  static constexpr int BATCH = EIGHT ? 1 : 0;
  static constexpr bool AHEAD = EIGHT;
  static constexpr bool BACKWARDS = true;        // clip_grads's norm has read the last gradients last: 620 -> 616 us
  using Load = StepLoad<EIGHT, WT, GT>;
  using Moment = typename Load::Moment;
  const AwHyper& h;
  float gs;
  // the run's buffers: pointers that are the same in all threads; lanes add their 32-bit offset
  WT* w;
  const GT* g;
  Moment* m;
  Moment* v;
  Code* ms;
  Code* vs;
  unsigned short* c;           // the copy's 16-bit elements
  Shared s;
  Scales scales;

  __device__ __forceinline__ StepOp(const AwHyper& hyper, float scale) : h(hyper), gs(scale) {}
  __device__ __forceinline__ void point(const AwTensor& t, unsigned long long first) {
    w = static_cast<WT*>(t.W) + first;
    g = static_cast<const GT*>(t.G) + first;
    m = static_cast<Moment*>(t.M) + first;
    v = static_cast<Moment*>(t.V) + first;
    c = static_cast<unsigned short*>(t.C) + first;
  }
  __device__ __forceinline__ void start(const AwTensor& t, unsigned long long first, int blocks) {
    point(t, first);
    s.start(h, t);
    if (EIGHT) {
      ms = t.MS + first / AW_BLOCK;
      vs = t.VS + first / AW_BLOCK;
      scales.load(ms, vs, blocks);
    }
  }
  template <int AT, int WIDE = 1>
  __device__ __forceinline__ void fetch(Load& in, unsigned at, const Place<WIDE>& b = {}) const {
    mo::fetch<WIDE, AT>(in.g, g + at, b);
    mo::fetch<WIDE, AT>(in.w, w + at, b);
    mo::fetch<WIDE, AT>(in.m, m + at, b);
    mo::fetch<WIDE, AT>(in.v, v + at, b);
  }
  __device__ __forceinline__ void ask(unsigned at) const {
    ask_next(g + at);
    ask_next(w + at);
    ask_next(m + at);
    ask_next(v + at);
  }
  template <int WIDE>
  __device__ __forceinline__ void work(const Load& in, const Place<WIDE>& b, unsigned at, int r) {
    float w1[PER], g1[PER], m1[PER], v1[PER];
    widen_all(g1, settled<WIDE>(in.g, g + at));
    widen_all(w1, settled<WIDE>(in.w, w + at));
    if (h.gscale != nullptr) scale_all(g1, gs);
    float sm = 1.f, sv = 1.f;
    moments_of(m1, v1, settled<WIDE>(in.m, m + at), settled<WIDE>(in.v, v + at), sm, sv, EIGHT ? scales.of(r) : 0, h.least_scale);
    update(w1, m1, v1, g1, h, s.r, sm, sv);
    constexpr bool LOW = sizeof(WT) == 2;
    Noise<WIDE> n;
    const bool noisy = FIRST || h.stochastic;
    if ((EIGHT || LOW) && noisy) n.draw(b, s.k);
    if constexpr (EIGHT) {
      store_moments<FIRST>(m1, v1, m + at, v + at, scales, r, b, noisy, n, s.k);
    } else {
      store(m1, m + at, b);
      store(v1, v + at, b);
    }
    if (!LOW && s.ct == AW_BF16) store(w1, reinterpret_cast<__nv_bfloat16*>(c) + at, b);
    if (!LOW && s.ct == AW_F16) store(w1, reinterpret_cast<__half*>(c) + at, b);
    if constexpr (LOW) {
      Raw<WT> out;
      if (noisy) round_weights(out, w1, n.second(s.k));
      else narrow_all(out, w1);
      put(out, w + at, b);
    } else {
      store(w1, w + at, b);
    }
  }
  __device__ __forceinline__ void work_narrow(const Place<0>& b, unsigned at, int r) {
    Load in;
    fetch<0, 0>(in, at, b);
    work(in, b, at, r);
  }
  __device__ __forceinline__ void narrow(const AwTensor& t, const Place<0>& b, unsigned at, int r);
  __device__ __forceinline__ void finish(int blocks) const {
    if (EIGHT) scales.store(ms, vs, blocks);
  }
};

// A narrow block, apart from the registers of the main path; returns the run's
// scales.
template <bool EIGHT, bool FIRST, typename WT, typename GT>
__device__ __noinline__ unsigned step_tail(const AwTensor& t, const AwHyper& h, float gs, Shared s, unsigned long long first,
                                           int left, unsigned scales, int r) {
  StepOp<EIGHT, FIRST, WT, GT> op(h, gs);
  op.point(t, first - threadIdx.x);
  op.s = s;
  op.scales.all = scales;
  op.work_narrow(Place<0>{first, left}, threadIdx.x, r);
  return op.scales.all;
}

template <bool EIGHT, bool FIRST, typename WT, typename GT>
__device__ __forceinline__ void StepOp<EIGHT, FIRST, WT, GT>::narrow(const AwTensor& t, const Place<0>& b, unsigned, int r) {
  scales.all = step_tail<EIGHT, FIRST, WT, GT>(t, h, gs, s, b.first, b.left, EIGHT ? scales.all : 0, r);
}

template <bool EIGHT, bool FIRST, typename WT, typename GT, bool VEC, int N>
__global__ void __launch_bounds__(AW_THREADS, VEC && !EIGHT ? STEP32_CTAS : STEP8_CTAS)
    adamw_kernel(const __grid_constant__ AwTableOf<N> tab, const __grid_constant__ AwHyper h) {
  pdl_wait();
  pdl_trigger();
  if (h.skip != nullptr && *h.skip != 0) return;
  StepOp<EIGHT, FIRST, WT, GT> op(h, h.gscale ? *h.gscale : 1.f);
  walk<VEC>(tab, op);
}

// ---------------------------------------------------------------- pack and unpack
template <bool FIRST, typename T>
struct PackOp {
  static constexpr bool AHEAD = false;
  static constexpr int BATCH = 2;                // 50 M elements: 78 us; with 1 82, with two buffers 85
  static constexpr bool BACKWARDS = false;
  struct Load {
    Raw<T> m, v;
  };
  const AwHyper& h;
  const T* m;
  const T* v;
  Code* m8;
  Code* v8;
  Code* ms;
  Code* vs;
  Keys k;
  Scales scales;
  __device__ __forceinline__ explicit PackOp(const AwHyper& hyper) : h(hyper) {}
  __device__ __forceinline__ void start(const AwTensor& t, unsigned long long first, int) {
    m = static_cast<const T*>(t.G) + first;
    v = static_cast<const T*>(t.C) + first;
    m8 = static_cast<Code*>(t.M) + first;
    v8 = static_cast<Code*>(t.V) + first;
    ms = t.MS + first / AW_BLOCK;
    vs = t.VS + first / AW_BLOCK;
    if (h.stochastic) k = keys_of(h, t.index);
    scales.all = 0;
  }
  template <int AT, int WIDE = 1>
  __device__ __forceinline__ void fetch(Load& in, unsigned at, const Place<WIDE>& b = {}) const {
    mo::fetch<WIDE, AT>(in.m, m + at, b);
    mo::fetch<WIDE, AT>(in.v, v + at, b);
  }
  template <int WIDE>
  __device__ __forceinline__ void work(const Load& in, const Place<WIDE>& b, unsigned at, int r) {
    float x[PER], y[PER];
    widen_all(x, settled<WIDE>(in.m, m + at));
    widen_all(y, settled<WIDE>(in.v, v + at));
    Noise<WIDE> n;
    const bool noisy = FIRST || h.stochastic;
    if (noisy) n.draw(b, k);
    store_moments<FIRST>(x, y, m8 + at, v8 + at, scales, r, b, noisy, n, k);
  }
  __device__ __forceinline__ void narrow(const AwTensor&, const Place<0>& b, unsigned at, int r) {
    Load in;
    fetch<0, 0>(in, at, b);
    work(in, b, at, r);
  }
  __device__ __forceinline__ void finish(int blocks) const { scales.store(ms, vs, blocks); }
};

template <bool FIRST, typename T, bool VEC, int N>
__global__ void __launch_bounds__(AW_THREADS) pack_kernel(const __grid_constant__ AwTableOf<N> tab,
                                                          const __grid_constant__ AwHyper h) {
  pdl_wait();
  pdl_trigger();
  PackOp<FIRST, T> op(h);
  walk<VEC>(tab, op);
}

template <typename T>
struct UnpackOp {
  static constexpr bool AHEAD = false;
  static constexpr int BATCH = 4;                // 50 M elements: 49 us; with 8 52, with two buffers 62
  static constexpr bool BACKWARDS = false;
  struct Load {
    Raw<Code> m, v;
  };
  const Code* m8;
  const Code* v8;
  T* m;
  T* v;
  Scales scales;
  __device__ __forceinline__ void start(const AwTensor& t, unsigned long long first, int blocks) {
    m8 = static_cast<const Code*>(t.M) + first;
    v8 = static_cast<const Code*>(t.V) + first;
    m = static_cast<T*>(t.W) + first;
    v = static_cast<T*>(t.C) + first;
    scales.load(t.MS + first / AW_BLOCK, t.VS + first / AW_BLOCK, blocks);
  }
  template <int AT, int WIDE = 1>
  __device__ __forceinline__ void fetch(Load& in, unsigned at, const Place<WIDE>& b = {}) const {
    mo::fetch<WIDE, AT>(in.m, m8 + at, b);
    mo::fetch<WIDE, AT>(in.v, v8 + at, b);
  }
  template <int WIDE>
  __device__ __forceinline__ void work(const Load& in, const Place<WIDE>& b, unsigned at, int r) const {
    float x[PER], y[PER];
    decode(x, y, in.m, in.v);
    const unsigned sc = scales.of(r);
    const float sm = scale_of(sc & 0xffu), sv = scale_of(sc >> 8);
    scale_all(x, sm);
    scale_all(y, sv);
    store(x, m + at, b);
    store(y, v + at, b);
  }
  __device__ __forceinline__ void narrow(const AwTensor&, const Place<0>& b, unsigned at, int r) const {
    Load in;
    fetch<0, 0>(in, at, b);
    work(in, b, at, r);
  }
  __device__ __forceinline__ void finish(int) const {}
};

template <typename T, bool VEC, int N>
__global__ void __launch_bounds__(AW_THREADS) unpack_kernel(const __grid_constant__ AwTableOf<N> tab) {
  pdl_wait();
  pdl_trigger();
  UnpackOp<T> op;
  walk<VEC>(tab, op);
}

// ---------------------------------------------------------------- clipping
// norm    sum of squares: 8 at a time in fp32 (in fp64 where fp32 does not hold
//         them), then fp64; one partial sum per CTA, in an order that the grid alone fixes
// finish  the partial sums in a fixed order, the norm and the factor
// scale   out = factor * G, the last runs first: L2 still holds them.  With few
//         partial sums every CTA sums them itself and `finish` is left out.
__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A lane's squares of a run, 64 at most, lose less than 2^-143 below fp32's
// smallest numbers: under 2^-43 of a sum from here on.
constexpr double LEAST_SQUARES = 0x1p-100;

__device__ __forceinline__ float wide(float x) { return x; }
__device__ __forceinline__ float wide(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float wide(__half x) { return __half2float(x); }

// A lane's part of a run's sum of squares in fp64.
template <typename T>
__device__ __noinline__ double squares64(const T* g, int elements) {
  double s = 0.0;
  for (int i = threadIdx.x; i < elements; i += 32) {
    const double x = wide(g[i]);
    s += x * x;
  }
  return s;
}

template <typename T>
struct NormOp {
  static constexpr bool AHEAD = false;
  static constexpr int BATCH = 4;                // with the scaling pass, 50 M elements: 67 us; with 1 76, with 8 69
  static constexpr bool BACKWARDS = false;
  using Load = Raw<T>;
  double sum = 0.0, run;
  const T* g;
  long long left;                                // elements of the tensor from the run on
  unsigned any;                                  // bits of the lane's elements: not all zeros, as unseen rows are
  __device__ __forceinline__ void start(const AwTensor& t, unsigned long long first, int) {
    g = static_cast<const T*>(t.G) + first;
    left = t.numel - (long long)first;
    run = 0.0;
    any = 0;
  }
  template <int AT, int WIDE = 1>
  __device__ __forceinline__ void fetch(Load& in, unsigned at, const Place<WIDE>& b = {}) const { mo::fetch<WIDE, AT>(in, g + at, b); }
  template <int WIDE>
  __device__ __forceinline__ void work(const Load& in, const Place<WIDE>&, unsigned at, int) {
    float x[PER], s = 0.f;
    const Load raw = settled<WIDE>(in, g + at);
    widen_all(x, raw);
#pragma unroll
    for (int j = 0; j < PER; ++j) s = fmaf(x[j], x[j], s);
#pragma unroll
    for (int k = 0; k < Load::WORDS; ++k) any |= raw.w[k];
    run += (double)s;
  }
  __device__ __forceinline__ void narrow(const AwTensor&, const Place<0>& b, unsigned at, int r) {
    Load in;
    fetch<0, 0>(in, at, b);
    work(in, b, at, r);
  }
  // A run whose squares fp32 does not hold is read again.
  __device__ __forceinline__ void finish(int blocks) {
    const unsigned some = any & (sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu);
    const bool odd = !(run < (double)__uint_as_float(INF_BITS)) || (run < LEAST_SQUARES && some != 0);
    if (rare(__any_sync(0xffffffffu, odd))) run = squares64(g, (int)min((long long)blocks * AW_BLOCK, left));
    sum += run;
  }
};

template <typename T, bool VEC, int N>
__global__ void __launch_bounds__(AW_THREADS) norm_kernel(const __grid_constant__ AwTableOf<N> tab, double* partial) {
  pdl_wait();
  pdl_trigger();
  NormOp<T> op;
  walk<VEC>(tab, op);
  const double s = warp_sum(op.sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// The factor from the sum of all squares, rounded to fp32 once; the caller with
// `write` stores the results.
__device__ __forceinline__ float factor_of(const ClipArgs& a, double squares, bool write) {
  const float scale = a.scale ? *a.scale : 1.f;
  const double exact = fabs((double)scale) * sqrt(squares);
  const float norm = (float)exact;
  // a norm that fp32 does not hold counts as infinite here too
  const double f = (double)a.max_norm / ((isfinite(norm) ? exact : (double)norm) + 1e-6);
  // a norm that is not a number gives such a factor (1 only where f >= 1)
  const float factor = (float)((double)scale * (f >= 1.0 ? 1.0 : f));
  if (write) {
    *a.norm = norm;
    *a.factor = factor;
    if (a.nonfinite) *a.nonfinite = isfinite(norm) ? 0 : 1;
  }
  return factor;
}

// The sum of at most FEW_PARTS partial sums, the same in every lane of a warp.
__device__ __forceinline__ double sum_few(const ClipArgs& a) {
  double sum = 0.0;
  for (int i = threadIdx.x % 32; i < a.parts; i += 32) sum += a.partial[i];
  return warp_sum(sum);
}

__global__ void __launch_bounds__(FINISH_THREADS) finish_kernel(const __grid_constant__ ClipArgs a) {
  __shared__ double red[FINISH_THREADS / 32];
  pdl_wait();
  pdl_trigger();
  double s = 0.0;
  if (a.parts <= FEW_PARTS) {
    s = sum_few(a);
  } else {
    double sum = 0.0;
    for (int i = threadIdx.x; i < a.parts; i += FINISH_THREADS) sum += a.partial[i];
    sum = warp_sum(sum);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = sum;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < FINISH_THREADS / 32; ++k) s += red[k];
  }
  if (threadIdx.x == 0) factor_of(a, s, true);
}

template <typename T, typename OUT>
struct ScaleOp {
  static constexpr bool AHEAD = false;
  static constexpr int BATCH = 4;
  static constexpr bool BACKWARDS = true;
  using Load = Raw<T>;
  float f;
  const T* g;
  OUT* out;
  __device__ __forceinline__ void start(const AwTensor& t, unsigned long long first, int) {
    g = static_cast<const T*>(t.G) + first;
    out = static_cast<OUT*>(t.C) + first;
  }
  template <int AT, int WIDE = 1>
  __device__ __forceinline__ void fetch(Load& in, unsigned at, const Place<WIDE>& b = {}) const { mo::fetch<WIDE, AT>(in, g + at, b); }
  template <int WIDE>
  __device__ __forceinline__ void work(const Load& in, const Place<WIDE>& b, unsigned at, int) const {
    float x[PER];
    widen_all(x, settled<WIDE>(in, g + at));
    scale_all(x, f);
    store(x, out + at, b);
  }
  __device__ __forceinline__ void narrow(const AwTensor&, const Place<0>& b, unsigned at, int r) const {
    Load in;
    fetch<0, 0>(in, at, b);
    work(in, b, at, r);
  }
  __device__ __forceinline__ void finish(int) const {}
};

template <typename T, typename OUT, bool VEC, int N>
__global__ void __launch_bounds__(AW_THREADS) scale_kernel(const __grid_constant__ AwTableOf<N> tab,
                                                           const __grid_constant__ ClipArgs a) {
  pdl_wait();
  pdl_trigger();
  ScaleOp<T, OUT> op;
  op.f = a.finish_here ? factor_of(a, sum_few(a), blockIdx.x == 0 && threadIdx.x == 0) : *a.factor;
  walk<VEC>(tab, op);
}

// Calls f with a null pointer of the element type t.
template <typename F>
cudaError_t with_type(AwType t, F f) {
  if (t == AW_F32) return f(static_cast<float*>(nullptr));
  if (t == AW_BF16) return f(static_cast<__nv_bfloat16*>(nullptr));
  return f(static_cast<__half*>(nullptr));
}
template <typename F>
cudaError_t with_wide_type(AwType t, F f) {
  return t == AW_F32 ? f(static_cast<float*>(nullptr)) : f(static_cast<__nv_bfloat16*>(nullptr));
}
template <typename P>
using Pointee = typename std::remove_pointer<P>::type;

// Launches one of four forms of a kernel: for aligned tensors or others, with a
// short or a full table (its first AW_SHORT tensors are all that the short form
// reads; 31 KB of parameters cost a launch 1.5 us more than 8).  The further
// argument is passed by its address, like the table, and copied once.
template <typename Arg>
cudaError_t launch_list(const void* (&forms)[2][2], int kind, const AwTable& t, unsigned grid, const Arg& arg, cudaStream_t s) {
  ProfScope prof(kind, s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(AW_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_off() ? 0 : 1;
  void* args[] = {const_cast<AwTable*>(&t), const_cast<Arg*>(&arg)};
  return cudaLaunchKernelExC(&cfg, forms[t.t[0].vec == 2][t.n > AW_SHORT], args);
}
#define MO_FORMS(KERNEL, ...)                                                                                       \
  {{(const void*)KERNEL<__VA_ARGS__, false, AW_SHORT>, (const void*)KERNEL<__VA_ARGS__, false, AW_MAX>},            \
   {(const void*)KERNEL<__VA_ARGS__, true, AW_SHORT>, (const void*)KERNEL<__VA_ARGS__, true, AW_MAX>}}

template <bool EIGHT, bool FIRST>
cudaError_t launch_step(const AwTable& t, const AwHyper& h, cudaStream_t s) {
  return with_wide_type(t.t[0].wt, [&](auto* w) {
    return with_type(t.t[0].gt, [&](auto* g) {
      using W = Pointee<decltype(w)>;
      using G = Pointee<decltype(g)>;
      const void* forms[2][2] = MO_FORMS(adamw_kernel, EIGHT, FIRST, W, G);
      return launch_list(forms, PK_ADAMW, t, t.runs, h, s);
    });
  });
}

}  // namespace

// A CTA for each run: the hardware hands runs out as CTAs end, which balances
// better than a fixed share for each of as many CTAs as fit (218 M elements:
// fp32 step 1000 -> 905 us, 8-bit step 473 -> 454).  Long runs share the search
// for their tensor, its rates and, with 8 bits, the sectors of the scales;
// short ones spread a short list over the card (of 16 they win 2 % of the 8-bit
// step at 218 M elements and lose 1 to 15 % below 80 M):
//   65 tensors of 4096 (1040 blocks)       runs of 1: 3.3 us    8: 7.7
//   300 odd ones, 8 bits (19 k blocks)     2: 40    4: 38       8: 48
//   218 M elements, 8 bits, unpacking      1: 1759  4: 685      8: 622
//   218 M elements, fp32                   1: 906   2: 903      8: 951
int run_of(long long blocks, int most, int warps, int sms) {
  int run = 1;
  while (run < most && blocks >= (long long)warps * run * sms) run *= 2;
  return run;
}

cudaError_t launch_adamw(const AwTable& t, const AwHyper& h, cudaStream_t s) { return launch_step<false, false>(t, h, s); }
cudaError_t launch_adamw8(const AwTable& t, const AwHyper& h, cudaStream_t s) {
  return h.first ? launch_step<true, true>(t, h, s) : launch_step<true, false>(t, h, s);
}

template <bool FIRST>
cudaError_t launch_pack_of(const AwTable& t, const AwHyper& h, cudaStream_t s) {
  return with_wide_type(t.t[0].gt, [&](auto* m) {
    const void* forms[2][2] = MO_FORMS(pack_kernel, FIRST, Pointee<decltype(m)>);
    return launch_list(forms, PK_MOMENTS, t, t.runs, h, s);
  });
}
cudaError_t launch_pack(const AwTable& t, const AwHyper& h, cudaStream_t s) {
  return h.first ? launch_pack_of<true>(t, h, s) : launch_pack_of<false>(t, h, s);
}

cudaError_t launch_unpack(const AwTable& t, cudaStream_t s) {
  return with_wide_type(t.t[0].wt, [&](auto* m) {
    const void* forms[2][2] = MO_FORMS(unpack_kernel, Pointee<decltype(m)>);
    return launch_list(forms, PK_MOMENTS, t, t.runs, 0, s);
  });
}

int clip_norm_ctas(const AwTable& t, int most) {
  return t.runs < (unsigned)most ? (int)t.runs : most;
}

cudaError_t launch_clip_norm(const AwTable& t, double* partial, int ctas, cudaStream_t s) {
  return with_type(t.t[0].gt, [&](auto* g) {
    const void* forms[2][2] = MO_FORMS(norm_kernel, Pointee<decltype(g)>);
    return launch_list(forms, PK_CLIP, t, (unsigned)ctas, partial, s);
  });
}

cudaError_t launch_clip_finish(const ClipArgs& a, cudaStream_t s) {
  ProfScope prof(PK_CLIP, s);
  return launch_pdl(finish_kernel, dim3(1), dim3(a.parts <= FEW_PARTS ? 32 : FINISH_THREADS), 0, s, false, a);
}

cudaError_t launch_clip_scale(const AwTable& t, const ClipArgs& a, cudaStream_t s) {
  return with_type(t.t[0].gt, [&](auto* g) {
    return with_type(t.t[0].ct, [&](auto* o) {
      using G = Pointee<decltype(g)>;
      using O = Pointee<decltype(o)>;
      const void* forms[2][2] = MO_FORMS(scale_kernel, G, O);
      return launch_list(forms, PK_CLIP, t, t.runs, a, s);
    });
  });
}

}  // namespace mo
