// grads.cu -- rank sum of many gradient tensors, their global norm, clipping.
//
//   G_t   = scale * sum_r g_{r,t}             (fp32, rank order)
//   norm  = sqrt(sum over all tensors of G^2)
//   out_t = rne_T(G_t) * min(1, max_norm / (norm + 1e-6)), rounded to T again
//
// Two passes: the first reads the W ranks, stores G in the tensors' own type
// and sums G^2 of the unrounded values; the second scales the stored values
// and does nothing when the norm is within the limit.  Keeping G in its type
// between the passes costs a clipped value one more rounding of half a step
// (what calling a reduce and then a clip would give) and keeps the second
// pass at one read and one write of the tensors.  Only where that rounding would
// lose the value is it not kept: an fp16 sum past 65504 is stored as infinity,
// and the second pass adds the ranks again for the vectors that hold one.  Where
// the output replaces an fp16 input, which is gone by then, the first pass
// stores nothing and the second adds the ranks of the whole tensor.  With one
// rank the first pass of car_grads_reduce_clip only reads: the second reads the
// input again, so that a clipped step moves 3 tensors' bytes instead of 4 (and
// rounds once), and one in place that needs no clipping moves 1.
//
// Where every value has to be rounded once (car_grads_reduce_clip_once), the
// second pass adds the ranks' 16-bit tensors again, if there is anything to
// clip: 64 M bf16 values, W = 4, clipped 182 us against 131, W = 8 329 against
// 218.  Both passes then read without the hints below, since what L2 keeps of
// the ranks is of use too (with them 192 and 355 us), and what they cost where
// nothing is clipped falls away (W = 4 94 against 101 us).
//
// Work is cut into chunks of one tensor each, all of about the same length; a
// wave of CTAs takes them in order, the second pass in the opposite order, the
// last written first: what the first pass left in L2 (129 MB) is read from
// there, and written over before it goes to HBM.  Where the outputs are not
// much larger than L2 the ranks' values are read with an evict-first hint, so
// that they do not push them out (W = 4, 134 MB: the second pass 42 -> 34 us);
// where they are, that only costs (W = 8, 400 MB: the first pass 531 -> 572).
// The second pass writes with that hint for all but short lists: its own
// output must not push out what it has yet to read (W = 1, 152 MB: 75.9 ->
// 73.5 us; W = 8, 400 MB: 711 -> 687).
//
// A chunk's descriptor holds its pointers.  The plan never changes, so the
// first descriptor, and a prefetch of the first 8 KB per rank into L2, come
// before the PDL wait (W = 4, 8 MB: 11.0 -> 9.3 us).  Squares are summed in
// fp32 over a thread's part of one chunk (kGradChunkVecs / kGradThreads = 8
// vectors, 64 values) and over its warp (in 64 bits near fp32's largest value),
// and in 64 bits from there on.  The CTAs' partials are added the same in any
// order, so the same call gives the same bits: by the last CTA to arrive where
// the caller wants the sum, and by every CTA of the second pass where that
// follows (car_grads_reduce_clip): the fence, the arrival and the partials'
// loads leave the tail of the first pass (W = 2, 0.2 MB, clipped 6.3 -> 4.0 us;
// W = 4, 8 MB 13.7 -> 11.2).
// Roofline: HBM, (W + 1) * 16 bytes per vector: 516 to 522 us for W = 8, 400 MB
// (1.02 of the copy peak).
#include <stdint.h>

#include "car_device.cuh"
#include "car_launch.h"

namespace car {
namespace {

template <int DT>
struct Scalar;
template <>
struct Scalar<kBF16> {
  using T = __nv_bfloat16;
  __device__ __forceinline__ static float up(T v) { return __bfloat162float(v); }
  __device__ __forceinline__ static T down(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Scalar<kFP16> {
  using T = __half;
  __device__ __forceinline__ static float up(T v) { return __half2float(v); }
  __device__ __forceinline__ static T down(float v) { return __float2half_rn(v); }
};
template <>
struct Scalar<kFP32> {
  using T = float;
  __device__ __forceinline__ static float up(T v) { return v; }
  __device__ __forceinline__ static T down(float v) { return v; }
};

// 64-bit floating point is scarce on this part (a warp's addition takes some
// tens of cycles of the one unit of an SM): a warp adds one such term per
// chunk, eight warps' sums are three additions of one warp, the partials' sum
// is integer arithmetic, and the square root and the quotient are fp32.  With
// every thread taking root and quotient in 64 bits a clip that had nothing to
// do took 12 us.
// Over the warp in fp32, or in 64 bits where that could overflow.
__device__ __forceinline__ double warp_sum(float v) {
  if (__any_sync(0xFFFFFFFFu, v >= 0x1p+122f)) {
    double d = v;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
    return d;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
// Sum over the block of a value that lane 0 of each warp holds; in thread 0.
__device__ __forceinline__ double block_sum(double v, double* s_warp) {
  constexpr int N = kGradThreads / 32;
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = s_warp[threadIdx.x % N];
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  }
  return v;
}

// Sum of n <= kMaxGradCtas values >= 0 by the whole block, in every thread:
// mantissa * 2^exponent, or not finite.  The mantissas (53 bits) are shifted
// to the largest exponent and added as integers: at most 2^11 of them, each
// cut by less than one unit of the last place of the largest, so that the sum
// is within 2^-41 of the exact one, and in any order the same.
struct Total {
  uint64_t mantissa;  // not finite: 0 for infinity, else NaN
  int exponent;
  bool finite;
};
struct TotalShared {
  uint32_t top[kGradThreads / 32], part[3][kGradThreads / 32];
};
__device__ __forceinline__ Total sum_values(const double* __restrict__ v, int n, TotalShared& s) {
  constexpr int K = kMaxGradCtas / kGradThreads, N = kGradThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t b[K];
  uint32_t top = 0u;  // exponent field; above 2047 for what is negative
#pragma unroll
  for (int k = 0; k < K; k++) {
    const int i = threadIdx.x + k * kGradThreads;
    b[k] = i < n ? (uint64_t)__double_as_longlong(__ldcg(v + i)) : 0u;
    if (b[k] << 1 == 0u) b[k] = 0u;  // -0
    top = max(top, (uint32_t)(b[k] >> 52));
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (lane == 0) s.top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < N; w++) top = max(top, s.top[w]);
  const bool finite = top < 2047u;
  uint64_t sum = 0u;
#pragma unroll
  for (int k = 0; k < K; k++) {
    const uint32_t e = (uint32_t)(b[k] >> 52);
    const uint64_t fraction = b[k] & ((1ull << 52) - 1u);
    const uint64_t m = e > 0u ? fraction | (1ull << 52) : fraction << 1;  // m * 2^(e - 1075)
    if (finite) {
      sum += top - e < 64u ? m >> (top - e) : 0u;
    } else if (e > 2047u || (e == 2047u && fraction != 0u)) {
      sum = 1u;  // a NaN, or the root of what is negative
    }
  }
  const uint32_t p0 = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)sum & 0xFFFFFFu);
  const uint32_t p1 = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)(sum >> 24) & 0xFFFFFFu);
  const uint32_t p2 = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)(sum >> 48));
  if (lane == 0) {
    s.part[0][warp] = p0;
    s.part[1][warp] = p1;
    s.part[2][warp] = p2;
  }
  __syncthreads();
  uint32_t t0 = 0u, t1 = 0u, t2 = 0u;
#pragma unroll
  for (int w = 0; w < N; w++) {
    t0 += s.part[0][w];
    t1 += s.part[1][w];
    t2 += s.part[2][w];
  }
  return Total{(uint64_t)t0 + ((uint64_t)t1 << 24) + ((uint64_t)t2 << 48), (int)top - 1075, finite};
}
__device__ __forceinline__ double to_double(const Total& t) {
  if (!t.finite) return t.mantissa ? nan("") : (double)INFINITY;
  return scalbn((double)t.mantissa, t.exponent);
}
// Its square root in fp32.
__device__ __forceinline__ float root(const Total& t) {
  if (!t.finite) return t.mantissa ? nanf("") : INFINITY;
  const int odd = t.exponent & 1;
  return scalbnf(sqrtf(__fmul_rn((float)t.mantissa, odd ? 2.f : 1.f)), (t.exponent - odd) / 2);
}

// L2 priority of values that are read once: first to be evicted, or as any.
__device__ __forceinline__ uint64_t read_policy(bool evict_first) {
  uint64_t first, normal;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
  return evict_first ? first : normal;
}
// A pass that stores may store over an input, or over what the first pass
// stored: its loads are ordinary ones.  (As loads of constant data they
// measure the same but for W = 4, 8 MB, 9.02 against 9.25 us.)
template <bool READ_ONLY>
__device__ __forceinline__ uint4 ld_hint(const void* p, uint64_t policy) {
  uint4 v;
  if constexpr (READ_ONLY)
    asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy));
  else
    asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy));
  return v;
}
__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void st_hint(void* p, uint4 v, uint64_t policy) {
  asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1,%2,%3,%4}, %5;" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w),
               "l"(policy)
               : "memory");
}

// Parts of a chunk: `head` elements up to a 16-byte boundary, whole vectors,
// and a tail; or, where the pointers share no boundary, all of it as a tail.
struct Span {
  int head, vecs, tail;
};
template <int DT>
__device__ __forceinline__ Span span_of(const GradChunk& c) {
  constexpr int E = Pack<DT>::kN;
  if (c.head < 0) return Span{0, 0, c.count};
  const int head = min((int)c.head, c.count);
  const int vecs = (c.count - head) / E;
  return Span{head, vecs, c.count - head - vecs * E};
}

// Vectors per thread per iteration: 4 to 16 loads in flight per thread (4, 8,
// 6, 8, then W).  Every rank count has its instance, compiled for as many CTAs
// per SM as its registers allow without spills.  One that takes the count at
// run time, a rank's four vectors at a time, is slower: W = 12, 32 M bf16 values
// 187 against 130 us, W = 9 146 / 103, W = 5 70.5 / 68.2; 0.24 M, W = 12 7.7 /
// 5.0, W = 5 5.5 / 4.1.
template <int W>
constexpr int kGradVectors = W >= 5 ? 1 : W >= 3 ? 2 : 4;

// CTAs per SM that the instances for W ranks are compiled for.  (The clip's
// kSums instances for 2, 8, 10 and 11 spill 12 to 40 bytes.)
template <int W>
constexpr int kGradMinCtas = W > 11 ? 2 : W > 8 ? 3 : 4;

// The clipped value of a sum whose stored form is `stored`: the sum itself
// counts where that is infinite, since a factor below 1 may bring it back.
__device__ __forceinline__ float clip_half(float stored, float sum, float coef) {
  return __fmul_rn(isinf(stored) ? sum : stored, coef);
}

// What a pass does with a chunk's sums G.
enum class SumUse {
  kSquare,  // adds their squares
  kStore,   // and stores them
  kClip,    // stores G * coef
  kClipRounded  // the same, of G as kStore would have left it
};

// Squares of the unrounded sums.  kept: what is stored is all that the caller
// will have of a sum, so one that fp16 stores as infinity (from 65520 on, half
// a step past its largest value) adds infinity.
template <int DT, int W, SumUse USE>
__device__ __forceinline__ float sum_chunk(const GradChunk& c, const void* const* __restrict__ in, float scale,
                                           uint64_t policy, bool kept, float coef = 1.f) {
  constexpr bool STORE = USE != SumUse::kSquare, CLIP = USE == SumUse::kClip || USE == SumUse::kClipRounded;
  using S = Scalar<DT>;
  using T = typename S::T;
  constexpr int E = Pack<DT>::kN;
  constexpr int U = kGradVectors<W>;
  const Span sp = span_of<DT>(c);
  const uint8_t* x[W];  // the whole vectors
#pragma unroll
  for (int r = 0; r < W; r++) x[r] = static_cast<const uint8_t*>(in[r]) + sp.head * sizeof(T);
  T* out = static_cast<T*>(c.out);
  uint8_t* to = reinterpret_cast<uint8_t*>(out + sp.head);
  constexpr bool LOSES = DT == kFP16 && USE == SumUse::kStore;
  float ss = 0.f, top = 0.f;
#pragma unroll 1
  for (int v0 = threadIdx.x; v0 < sp.vecs; v0 += kGradThreads * U) {
    // past the chunk's end the last vector is loaded again, and dropped below
    uint32_t at[U];
    float acc[U][E];
    uint4 raw[U][W];
#pragma unroll
    for (int u = 0; u < U; u++) {
      at[u] = (uint32_t)min(v0 + u * kGradThreads, sp.vecs - 1) * 16u;
#pragma unroll
      for (int r = 0; r < W; r++) raw[u][r] = ld_hint<!STORE>(x[r] + at[u], policy);
    }
#pragma unroll
    for (int u = 0; u < U; u++) rank_sum<DT, W>(raw[u], W, acc[u]);
#pragma unroll
    for (int u = 0; u < U; u++) {
      if (v0 + u * kGradThreads < sp.vecs) {
#pragma unroll
        for (int e = 0; e < E; e++) {
          acc[u][e] = __fmul_rn(acc[u][e], scale);
          if constexpr (USE == SumUse::kClip) acc[u][e] = __fmul_rn(acc[u][e], coef);
          if constexpr (!CLIP) ss = fmaf(acc[u][e], acc[u][e], ss);
          if constexpr (LOSES) top = fmaxf(top, fabsf(acc[u][e]));
        }
        if constexpr (USE == SumUse::kClipRounded) {
          float f[E];
          Pack<DT>::widen(Pack<DT>::narrow(acc[u]), f);
#pragma unroll
          for (int e = 0; e < E; e++) acc[u][e] = clip_half(f[e], acc[u][e], coef);
        }
        if constexpr (STORE) st16(to + at[u], Pack<DT>::narrow(acc[u]));
      }
    }
  }
  // the ragged ends
#pragma unroll 1
  for (int i = threadIdx.x; i < sp.head + sp.tail; i += kGradThreads) {
    const int at = i < sp.head ? i : i + sp.vecs * E;
    float acc = S::up(static_cast<const T*>(in[0])[at]);
    for (int r = 1; r < W; r++) acc = __fadd_rn(acc, S::up(static_cast<const T*>(in[r])[at]));
    acc = __fmul_rn(acc, scale);
    if constexpr (USE == SumUse::kClip) acc = __fmul_rn(acc, coef);
    if constexpr (USE == SumUse::kClipRounded) acc = clip_half(S::up(S::down(acc)), acc, coef);
    if constexpr (!CLIP) ss = fmaf(acc, acc, ss);
    if constexpr (LOSES) top = fmaxf(top, fabsf(acc));
    if constexpr (STORE) out[at] = S::down(acc);
  }
  if (LOSES && kept && top >= 65520.f) ss += INFINITY;  // (a NaN stays one)
  return ss;
}

// G of one element, as sum_chunk forms it.
template <int DT>
__device__ __forceinline__ float sum_element(const void* const* __restrict__ in, int n, int at, float scale) {
  using S = Scalar<DT>;
  using T = typename S::T;
  float acc = S::up(static_cast<const T*>(in[0])[at]);
  for (int r = 1; r < n; r++) acc = __fadd_rn(acc, S::up(static_cast<const T*>(in[r])[at]));
  return __fmul_rn(acc, scale);
}

// The same for the vector at byte offset `at` of every rank.
template <int DT>
__device__ __forceinline__ void sum_vector(const void* const* __restrict__ in, int n, uint32_t at, float scale,
                                           float (&acc)[Pack<DT>::kN]) {
  constexpr int E = Pack<DT>::kN;
#pragma unroll 1
  for (int r = 0; r < n; r++) {
    float f[E];
    Pack<DT>::widen(ld_once(static_cast<const uint8_t*>(in[r]) + at), f);
#pragma unroll
    for (int e = 0; e < E; e++) acc[e] = r == 0 ? f[e] : __fadd_rn(acc[e], f[e]);
  }
#pragma unroll
  for (int e = 0; e < E; e++) acc[e] = __fmul_rn(acc[e], scale);
}

__device__ __forceinline__ bool in_place(const GradChunk& c, const void* const* __restrict__ in, int n) {
  bool hit = false;
  for (int r = 0; r < n; r++) hit = hit || in[r] == c.out;
  return hit;
}

// Whether one of eight fp16 values is infinite.
__device__ __forceinline__ bool any_infinite(uint4 v) {
  auto top = [](uint32_t w) { return __habs2(*reinterpret_cast<const __half2*>(&w)); };
  const __half2 m = __hmax2(__hmax2(top(v.x), top(v.y)), __hmax2(top(v.z), top(v.w)));
  const uint32_t b = *reinterpret_cast<const uint32_t*>(&m);
  return (b & 0xFFFFu) == 0x7C00u || (b >> 16) == 0x7C00u;
}

// What clipping needs to add fp16 sums again (AGAIN): they were formed from
// these inputs with this scale.
struct SumSource {
  const void* const* in;
  int n;
  float scale;
};

// Whole vectors of out = (from * scale) * coef; from may be out itself.  AGAIN:
// from holds sums, and those that are infinite in fp16 are added again.
template <int DT, int U, bool AGAIN>
__device__ __forceinline__ void clip_vectors(uint4* to, const uint4* from, int vecs, float scale, float coef, uint64_t policy,
                                             const SumSource& src, int head) {
  constexpr int E = Pack<DT>::kN;
#pragma unroll 1
  for (int v0 = threadIdx.x; v0 < vecs; v0 += kGradThreads * U) {
    uint4 raw[U];
    uint32_t lost = 0u;
#pragma unroll
    for (int u = 0; u < U; u++) raw[u] = ld_once(from + min(v0 + u * kGradThreads, vecs - 1));
#pragma unroll
    for (int u = 0; u < U; u++) {
      if (v0 + u * kGradThreads < vecs) {
        float f[E];
        Pack<DT>::widen(raw[u], f);
#pragma unroll
        for (int e = 0; e < E; e++) f[e] = __fmul_rn(__fmul_rn(f[e], scale), coef);
        st_hint(to + v0 + u * kGradThreads, Pack<DT>::narrow(f), policy);
        if constexpr (AGAIN) lost |= any_infinite(raw[u]) ? 1u << u : 0u;
      }
    }
    if constexpr (AGAIN) {
#pragma unroll 1
      for (; lost; lost &= lost - 1u) {
        const int v = v0 + (__ffs((int)lost) - 1) * kGradThreads;
        float sum[E], f[E];
        sum_vector<DT>(src.in, src.n, ((uint32_t)head + (uint32_t)v * E) * (uint32_t)sizeof(__half), src.scale, sum);
        Pack<DT>::widen(Pack<DT>::narrow(sum), f);  // as they were stored
#pragma unroll
        for (int e = 0; e < E; e++) f[e] = clip_half(f[e], sum[e], coef);
        st_hint(to + v, Pack<DT>::narrow(f), policy);
      }
    }
  }
}

// One chunk of it, from being out itself or rank 0's input.  Eight loads in
// flight per thread against four: W = 4, 8 MB 11.2 -> 10.7 us, W = 8, 400 MB
// 680 -> 672; chunks of one vector per thread have no use for them.
template <int DT, bool AGAIN = false>
__device__ __forceinline__ void clip_chunk(const GradChunk& c, const void* from, float scale, float coef, uint64_t policy,
                                           const SumSource& src = SumSource{}) {
  using S = Scalar<DT>;
  using T = typename S::T;
  constexpr int E = Pack<DT>::kN;
  const Span sp = span_of<DT>(c);
  T* out = static_cast<T*>(c.out);
  const T* x = static_cast<const T*>(from);
  uint4* to = reinterpret_cast<uint4*>(out + sp.head);
  const uint4* body = reinterpret_cast<const uint4*>(x + sp.head);
  if (sp.vecs <= kGradThreads)
    clip_vectors<DT, 1, AGAIN>(to, body, sp.vecs, scale, coef, policy, src, sp.head);
  else
    clip_vectors<DT, AGAIN ? 4 : 8, AGAIN>(to, body, sp.vecs, scale, coef, policy, src, sp.head);
#pragma unroll 1
  for (int i = threadIdx.x; i < sp.head + sp.tail; i += kGradThreads) {
    const int at = i < sp.head ? i : i + sp.vecs * E;
    float f = __fmul_rn(S::up(x[at]), scale);
    if (AGAIN && isinf(f)) f = sum_element<DT>(src.in, src.n, at, src.scale);
    out[at] = S::down(__fmul_rn(f, coef));
  }
}

// Chunk i's descriptor: GradChunk, then the W input pointers.
__device__ __forceinline__ const GradChunk* chunk_at(const GradList& l, int stride, int i) {
  return reinterpret_cast<const GradChunk*>(l.chunks + (int64_t)i * stride);
}
__device__ __forceinline__ const void* const* inputs_of(const GradChunk* c) {
  return reinterpret_cast<const void* const*>(c + 1);
}

// Asks L2 for the first vectors (8 KB at most) of one of a chunk's buffers.
__device__ __forceinline__ void prefetch_chunk(const GradChunk& c, const void* from) {
  const uintptr_t size = (uintptr_t)c.count * (c.dtype == kFP32 ? 4u : 2u);
  const uintptr_t lo = (reinterpret_cast<uintptr_t>(from) + 15u) & ~(uintptr_t)15u;
  const uintptr_t hi = (reinterpret_cast<uintptr_t>(from) + size) & ~(uintptr_t)15u;
  if (hi > lo) prefetch_l2(reinterpret_cast<const void*>(lo), hi - lo < 8192u ? (uint32_t)(hi - lo) : 8192u);
}

template <int W, bool STORE>
__global__ void __launch_bounds__(kGradThreads, kGradMinCtas<W>)
    grads_reduce_kernel(const GradPlan p, const float scale, double* __restrict__ sumsq, const bool once) {
  __shared__ double s_warp[kGradThreads / 32];
  __shared__ TotalShared s_total;
  __shared__ bool s_last;
  const uint64_t policy = read_policy(STORE && p.evict_first && !once);
  const bool kept = sumsq != nullptr;  // else the second pass follows
  const int first = blockIdx.x, last = p.reduce.n, stride = (int)sizeof(GradChunk) + 8 * W;
  const GradChunk* d = chunk_at(p.reduce, stride, first);
  GradChunk c = {};
  if (first < last) {
    c = *d;
    if (threadIdx.x < W) prefetch_chunk(c, inputs_of(d)[threadIdx.x]);
  }
  pdl_wait_and_release();
  constexpr SumUse USE = STORE ? SumUse::kStore : SumUse::kSquare;
  double total = 0.0;
  for (int i = first; i < last; i += gridDim.x) {
    const void* const* in = inputs_of(d);
    const GradChunk cur = c;
    if (i + (int)gridDim.x < last) {  // the next descriptor while this chunk is summed
      d = chunk_at(p.reduce, stride, i + (int)gridDim.x);
      c = *d;
    }
    float ss;
    switch (cur.dtype) {
      case kBF16:
        if (STORE && W != 1 && once && in_place(cur, in, W))  // left to the second pass
          ss = sum_chunk<kBF16, W, SumUse::kSquare>(cur, in, scale, policy, kept);
        else
          ss = sum_chunk<kBF16, W, USE>(cur, in, scale, policy, kept);
        break;
      case kFP16:
        if (STORE && W != 1 && !kept && in_place(cur, in, W))  // so is this one
          ss = sum_chunk<kFP16, W, SumUse::kSquare>(cur, in, scale, policy, kept);
        else
          ss = sum_chunk<kFP16, W, USE>(cur, in, scale, policy, kept);
        break;
      default: ss = sum_chunk<kFP32, W, USE>(cur, in, scale, policy, kept); break;
    }
    const double chunk = warp_sum(ss);
    if ((threadIdx.x & 31) == 0) total += chunk;
  }
  total = block_sum(total, s_warp);
  if (!sumsq) {  // the second pass adds the partials
    if (threadIdx.x == 0) p.partial[blockIdx.x] = total;
    return;
  }
  if (threadIdx.x == 0) {
    p.partial[blockIdx.x] = total;
    __threadfence();
    s_last = atomicAdd(p.arrived, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (s_last) {
    __threadfence();
    const Total t = sum_values(p.partial, gridDim.x, s_total);
    if (threadIdx.x == 0) {
      *sumsq = to_double(t);
      *p.arrived = 0u;  // for the next call, which waits for this grid
    }
  }
}

// FROM: where the values come from (car_launch.h); W: the ranks for kSums and kOnce.
template <GradSource FROM, int W>
__global__ void __launch_bounds__(kGradThreads, kGradMinCtas<W>)
    grads_clip_kernel(const GradPlan p, const double* __restrict__ sums, const int n_sums, const float scale,
                      const float max_norm, float* __restrict__ norm_out) {
  constexpr bool FROM_INPUT = FROM == GradSource::kInput;
  __shared__ TotalShared s_total;
  const uint64_t policy = read_policy(FROM != GradSource::kOnce && p.pass_on);
  const int stride = (int)sizeof(GradChunk) + 8 * p.W;
  const GradList& list = FROM == GradSource::kOnce ? p.reduce : p.clip;  // (it reads what the reduce does)
  int i = list.n - 1 - (int)blockIdx.x;
  GradChunk c = {};
  const GradChunk* d = nullptr;
  const void* from = nullptr;
  if (i >= 0) {
    d = chunk_at(list, stride, i);
    c = *d;
    from = FROM_INPUT ? inputs_of(d)[0] : c.out;
  }
  // Released before the wait: where there is nothing to clip, the next
  // kernel's prologue runs in the tail of the first pass.  It waits for this
  // grid, and is only launched once every CTA here is resident.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float norm = root(sum_values(sums, n_sums, s_total));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  const float ratio = __fdiv_rn(max_norm, norm + 1e-6f);
  // within the limit, or no limit (false for a NaN norm, which then reaches every value)
  const bool whole = ratio >= 1.f || isinf(max_norm);
  const bool unsummed = FROM == GradSource::kOnce ? p.narrow_in_place : FROM == GradSource::kSums && p.half_in_place;
  if (whole && !FROM_INPUT && !unsummed) return;
  const float coef = whole ? 1.f : ratio;
  for (; i >= 0; i -= (int)gridDim.x) {
    const GradChunk cur = c;
    const void* const* in = inputs_of(d);
    const void* x = from;
    if (i >= (int)gridDim.x) {
      d = chunk_at(list, stride, i - (int)gridDim.x);
      c = *d;
      from = FROM_INPUT ? inputs_of(d)[0] : c.out;
    }
    if (FROM_INPUT && x == cur.out && whole && scale == 1.f) continue;  // already there
    if (FROM == GradSource::kSums && cur.dtype == kFP16) {
      if (unsummed && in_place(cur, in, W))
        sum_chunk<kFP16, W, SumUse::kClipRounded>(cur, in, scale, policy, false, coef);
      else if (!whole)
        clip_chunk<kFP16, true>(cur, x, 1.f, coef, policy, SumSource{in, W, scale});
      continue;
    }
    if (FROM == GradSource::kOnce && cur.dtype != kFP32) {
      if (whole && !in_place(cur, in, W)) continue;
      if (cur.dtype == kBF16)
        sum_chunk<kBF16, W, SumUse::kClip>(cur, in, scale, policy, false, coef);
      else
        sum_chunk<kFP16, W, SumUse::kClip>(cur, in, scale, policy, false, coef);
      continue;
    }
    if (!FROM_INPUT && whole) continue;
    const float once = FROM_INPUT ? scale : 1.f;  // what out holds is scaled
    if (FROM == GradSource::kOnce) {
      clip_chunk<kFP32>(cur, x, once, coef, policy);
      continue;
    }
    switch (cur.dtype) {
      case kBF16: clip_chunk<kBF16>(cur, x, once, coef, policy); break;
      case kFP16: clip_chunk<kFP16>(cur, x, once, coef, policy); break;
      default: clip_chunk<kFP32>(cur, x, once, coef, policy); break;
    }
  }
}

using ClipFn = void (*)(const GradPlan, const double*, const int, const float, const float, float*);
template <GradSource FROM>
ClipFn pick_clip_ranks(int W) {
  switch (W) {
    case 2: return grads_clip_kernel<FROM, 2>;
    case 3: return grads_clip_kernel<FROM, 3>;
    case 4: return grads_clip_kernel<FROM, 4>;
    case 5: return grads_clip_kernel<FROM, 5>;
    case 6: return grads_clip_kernel<FROM, 6>;
    case 7: return grads_clip_kernel<FROM, 7>;
    case 8: return grads_clip_kernel<FROM, 8>;
    case 9: return grads_clip_kernel<FROM, 9>;
    case 10: return grads_clip_kernel<FROM, 10>;
    case 11: return grads_clip_kernel<FROM, 11>;
    case 12: return grads_clip_kernel<FROM, 12>;
    case 13: return grads_clip_kernel<FROM, 13>;
    case 14: return grads_clip_kernel<FROM, 14>;
    case 15: return grads_clip_kernel<FROM, 15>;
    case 16: return grads_clip_kernel<FROM, 16>;
    default: return nullptr;
  }
}
ClipFn pick_clip(int W, GradSource from) {
  switch (from) {
    case GradSource::kOutput: return grads_clip_kernel<GradSource::kOutput, 1>;
    case GradSource::kSums: return pick_clip_ranks<GradSource::kSums>(W);
    case GradSource::kOnce: return pick_clip_ranks<GradSource::kOnce>(W);
    default: return grads_clip_kernel<GradSource::kInput, 1>;
  }
}

using GradsFn = void (*)(const GradPlan, const float, double*, const bool);
GradsFn pick_grads(int W, bool store) {
  if (!store) return W == 1 ? grads_reduce_kernel<1, false> : nullptr;
  switch (W) {
    case 1: return grads_reduce_kernel<1, true>;
    case 2: return grads_reduce_kernel<2, true>;
    case 3: return grads_reduce_kernel<3, true>;
    case 4: return grads_reduce_kernel<4, true>;
    case 5: return grads_reduce_kernel<5, true>;
    case 6: return grads_reduce_kernel<6, true>;
    case 7: return grads_reduce_kernel<7, true>;
    case 8: return grads_reduce_kernel<8, true>;
    case 9: return grads_reduce_kernel<9, true>;
    case 10: return grads_reduce_kernel<10, true>;
    case 11: return grads_reduce_kernel<11, true>;
    case 12: return grads_reduce_kernel<12, true>;
    case 13: return grads_reduce_kernel<13, true>;
    case 14: return grads_reduce_kernel<14, true>;
    case 15: return grads_reduce_kernel<15, true>;
    case 16: return grads_reduce_kernel<16, true>;
    default: return nullptr;
  }
}

}  // namespace

cudaError_t grads_occupancy(int W, bool store, int* reduce_per_sm) {
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(
      reduce_per_sm, reinterpret_cast<const void*>(pick_grads(W, store)), kGradThreads, 0);
}

cudaError_t grads_clip_occupancy(int W, GradSource from, int* per_sm) {
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(per_sm, reinterpret_cast<const void*>(pick_clip(W, from)), kGradThreads, 0);
}

cudaError_t launch_grads_reduce(const GradPlan& plan, float scale, bool store, double* sumsq, bool once, int grid,
                                cudaStream_t s) {
  GradsFn fn = pick_grads(plan.W, store);
  if (!fn) return cudaErrorInvalidValue;
  return launch_pdl(fn, (unsigned)grid, kGradThreads, 0, s, 1, plan, scale, sumsq, once);
}

cudaError_t launch_grads_clip(const GradPlan& plan, const double* sums, int n_sums, float scale, GradSource from,
                              float max_norm, float* norm_out, int grid, cudaStream_t s) {
  ClipFn fn = pick_clip(plan.W, from);
  if (!fn) return cudaErrorInvalidValue;
  return launch_pdl(fn, (unsigned)grid, kGradThreads, 0, s, 1, plan, sums, n_sums, scale, max_norm, norm_out);
}

}  // namespace car
