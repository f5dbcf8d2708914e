// branch_backward.cu -- backward of a block's branch (branch_rows.cu), for few
// rows, and the sums of the column gradients' partials for either backward
// kernel.
//
// Forward: a = sum_r x_r, u1 = a * q, q = rsqrt(mean(a^2) + norm_eps), h =
// residual_scale * residual + drop(u1 w1 gate), u = h * r, r = rsqrt(mean(h^2) +
// eps), out = u * w.  With g the rank sum of out's gradient and dres what
// arrives at residual_out:
//   dh = r * (g w - u * mean(g w u)) + dres;   dresidual = residual_scale * dh
//   dz = drop(dh);   t = dz * u1;   v = dz * gate * w1
//   dx = q * (v - u1 * mean(v u1))
//   dw = sum_m g u;   dw1 = sum_m gate t;   dgate = sum of t over its rows, * w1
// (without a norm: u1 = a, w1 = 1, dx = v).  The first exchange carries three
// sums (h^2, g w h, a^2), the second one (v u1); every input is read once and
// stays in registers between them.
//
// Column sums.  A CTA (or cluster) takes one contiguous span of rows, so a gate
// row that several spans share is cut at their ends only: t is summed in
// registers over a gate row's rows and leaves as the finished dgate where all of
// them lie in the span, else as one of two partials of the span (its first gate
// row, its last).  dw1 then needs gate * t once per gate row.  The CTAs'
// partials go to the caller's workspace and branch_sums_kernel adds them in a
// fixed order (no float atomics: the same call gives the same bits).
// Roofline: HBM, (W + 5) * 16 bytes per vector with norm and skip gradient, 2
// more for a gate of each row's own, and the partials (L2).  With a row for each CTA
// the partials are more than the data: 16 bytes per element in fp32, written and
// read again, where one rank in bf16 moves 12 (W = 1, M = 152, N = 8192 with norms:
// 11.9 us, floor 2.2, of which the second kernel is 5.8 by itself; W = 4 12.7, floor
// 3.3).  512 threads leave a thread 128 registers: the instances of the 16-bit types
// with a norm spill 36 to 60 bytes for two and four ranks (bf16 one, too), 180 to 240
// for sixteen and for rank counts without an instance of their own.
#include <algorithm>

#include "branch.cuh"

namespace car {
namespace {

struct BranchBackwardParams {
  RankPtrs dy;
  const uint4* h;
  const uint4* dres;         // may be null
  const uint4* ar;           // may be null
  const uint4* weight;
  const uint4* norm_weight;
  const uint4* gate;         // may be null
  uint4* dx;
  uint4* dresidual;          // may be null
  uint4* dgate_own;          // [M, N], or null
  float* dgate;              // [M / gate_span, N], or null
  float* part_w;             // [groups, N], or dweight with one group; may be null
  float* part_w1;            // the same for dnorm_weight
  float* part_gate;          // [groups, 2, N]: gate rows that a span's ends cut
  unsigned int* err;
  DropParams drop;
  float residual_scale;
  float eps, norm_eps;
  float cols;
  int64_t rows;
  uint32_t gate_span;        // rows that share a gate row; 1 for a gate of each row's own
  bool shared;               // t is summed by gate row (dgate, or dw1 behind a shared gate)
  int vec_per_row;
  int chunk;
  int cluster;
  int nranks;
  unsigned long long wait_ns;
  unsigned long long delay_ns;
  int64_t delay_row;
  int delay_cta;
};

// This CTA's piece of `row` into L2, one bulk prefetch per slice.
__device__ __forceinline__ void prefetch_row(const BranchBackwardParams& p, int n, int64_t row, int64_t end, int col0) {
  const int nvec = min(p.chunk, p.vec_per_row - col0);
  const int t = threadIdx.x;
  if (row >= end || nvec <= 0 || t > n + 3) return;
  const int64_t off = row * (int64_t)p.vec_per_row + col0;
  const uint4* src;
  if (t < n) src = static_cast<const uint4*>(p.dy.p[t]) + off;
  else if (t == n) src = p.h + off;
  else if (t == n + 1) src = p.dres ? p.dres + off : nullptr;
  else if (t == n + 2) src = p.ar ? p.ar + off : nullptr;
  else src = p.gate ? p.gate + (int64_t)((uint32_t)row / p.gate_span) * p.vec_per_row + col0 : nullptr;
  if (src) prefetch_l2(src, (uint32_t)nvec * 16u);
}

template <int E>
__device__ __forceinline__ void store_floats(float* to, const float2 (&f)[E / 2]) {
#pragma unroll
  for (int e = 0; e < E / 2; e += 2) *reinterpret_cast<float4*>(to + 2 * e) = make_float4(f[e].x, f[e].y, f[e + 1].x, f[e + 1].y);
}

template <int DT, int W, bool NORM>
__global__ void __launch_bounds__(kBranchThreads) reduce_branch_rmsnorm_backward_kernel(const BranchBackwardParams p) {
  constexpr int E = Pack<DT>::kN;
  constexpr int R = W > 0 ? W : kMaxRanks;
  const int n = W > 0 ? W : p.nranks;
  __shared__ __align__(16) RowSums s_sums;
  const int C = p.cluster;
  const int crank = C > 1 ? (int)cluster_rank() : 0;
  const int groups = gridDim.x / C, group = blockIdx.x / C;
  const int64_t first = span_start(p.rows, groups, group), end = span_start(p.rows, groups, group + 1);
  const int col0 = crank * p.chunk;
  const ClusterWait peers{crank, p.wait_ns, p.err};
  uint32_t x = 0;
  bool peers_ready = C == 1;
  if (C > 1) {
    if (threadIdx.x == 0) row_sums_init(s_sums, C);
    __syncthreads();
    cluster_arrive();
  }
  prefetch_row(p, n, first, end, col0);
  pdl_wait_and_release();
  const DropState state = drop_state(p.drop);
  const int v = threadIdx.x;
  const bool ok = v < p.chunk && col0 + v < p.vec_per_row;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint4 wv = ok ? __ldg(p.weight + col0 + v) : zero;
  const uint4 w1v = NORM && ok ? __ldg(p.norm_weight + col0 + v) : zero;
  const int64_t col = (int64_t)(col0 + v) * E, N = (int64_t)p.vec_per_row * E;
  float2 dw[E / 2], dw1[E / 2], tsum[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; e++) dw[e] = dw1[e] = tsum[e] = make_float2(0.f, 0.f);

  // rows [from, to) of gate row b are in tsum
  auto flush = [&](uint32_t b, int64_t from, int64_t to) {
    const int64_t lo = (int64_t)b * p.gate_span;
    const bool whole = from == lo && to == lo + p.gate_span;
    float2 w[E / 2], gf[E / 2];
    widen2<DT>(w1v, w);
    widen2<DT>(__ldg(p.gate + (int64_t)b * p.vec_per_row + col0 + v), gf);
    if (p.dgate) {
      float2 o[E / 2];
#pragma unroll
      for (int e = 0; e < E / 2; e++) o[e] = NORM && whole ? mul2(tsum[e], w[e]) : tsum[e];
      store_floats<E>(whole ? p.dgate + b * N + col : p.part_gate + (2 * (int64_t)group + (from == first ? 0 : 1)) * N + col, o);
    }
#pragma unroll
    for (int e = 0; e < E / 2; e++) {
      dw1[e] = fma2(gf[e], tsum[e], dw1[e]);
      tsum[e] = make_float2(0.f, 0.f);
    }
  };
  uint32_t b = p.gate ? (uint32_t)first / p.gate_span : 0;
  int64_t from = first, next = p.gate ? (int64_t)(b + 1) * p.gate_span : p.rows;

  for (int64_t row = first; row < end; row++) {
    const int64_t at = row * (int64_t)p.vec_per_row + col0 + v;
    prefetch_row(p, n, row + 1, end, col0);
    if (row == next) {
      if (p.shared && ok) flush(b, from, row);
      from = row;
      b++;
      next += p.gate_span;
    }
    uint4 raw[R], hv = zero, dv = zero, av = zero, gv = zero;
    if (ok) {
#pragma unroll
      for (int r = 0; r < R; r++)
        if (r < n) raw[r] = ld_stream(static_cast<const uint4*>(p.dy.p[r]) + at);
      hv = ld_stream(p.h + at);
      if (p.dres) dv = ld_stream(p.dres + at);
      if (p.ar) av = ld_stream(p.ar + at);
      if (p.gate) gv = __ldg(p.gate + (int64_t)b * p.vec_per_row + col0 + v);
    }
    uint32_t bits[E / 2];
    if (p.drop.active) drop_bits<E>(state, at, bits);
    float2 g[E / 2];
    float s[NORM ? 3 : 2] = {};
    if (ok) {
      float acc[E];
      rank_sum<DT, R>(raw, n, acc);
      float2 hf[E / 2], wf[E / 2], af[E / 2];
      widen2<DT>(hv, hf);
      widen2<DT>(wv, wf);
      widen2<DT>(av, af);
      float2 hh = make_float2(0.f, 0.f), gwh = hh, aa = hh;
#pragma unroll
      for (int e = 0; e < E / 2; e++) {
        g[e] = make_float2(acc[2 * e], acc[2 * e + 1]);
        hh = fma2(hf[e], hf[e], hh);
        gwh = fma2(mul2(g[e], wf[e]), hf[e], gwh);
        if constexpr (NORM) aa = fma2(af[e], af[e], aa);
      }
      s[0] = hh.x + hh.y;
      s[1] = gwh.x + gwh.y;
      if constexpr (NORM) s[2] = aa.x + aa.y;
    }
    if (!peers_ready) {
      cluster_wait();
      peers_ready = true;
    }
    // test hook: this whole CTA reaches the row's first exchange late
    if (C > 1 && crank == p.delay_cta && row == p.delay_row) spin_ns(p.delay_ns);
    row_sums(s_sums, s, x++, C, peers);
    const float r = rsqrtf(__fdiv_rn(s[0], p.cols) + p.eps);
    const float2 m = both(-__fdiv_rn(__fmul_rn(s[1], r), p.cols));
    const float2 q = NORM ? both(rsqrtf(__fdiv_rn(s[NORM ? 2 : 0], p.cols) + p.norm_eps)) : both(1.f);
    float2 vu = make_float2(0.f, 0.f), u1[E / 2];
    if (ok) {
      float2 hf[E / 2], wf[E / 2], f[E / 2];
      widen2<DT>(hv, hf);
      widen2<DT>(wv, wf);
      widen2<DT>(dv, f);
#pragma unroll
      for (int e = 0; e < E / 2; e++) {
        const float2 u = mul2(hf[e], both(r));
        dw[e] = fma2(g[e], u, dw[e]);
        g[e] = fma2(both(r), fma2(u, m, mul2(g[e], wf[e])), f[e]);  // dh
        hf[e] = mul2(g[e], both(p.residual_scale));
      }
      if (p.dresidual) st16(p.dresidual + at, narrow2<DT>(hf));
      if (p.drop.active) {
#pragma unroll
        for (int e = 0; e < E / 2; e++) g[e] = drop2(p.drop, bits[e], g[e]);
      }
      widen2<DT>(av, u1);
      widen2<DT>(w1v, wf);
      widen2<DT>(gv, f);
#pragma unroll
      for (int e = 0; e < E / 2; e++) {  // g: dz
        if constexpr (NORM) u1[e] = mul2(u1[e], q);
        const float2 t = mul2(g[e], u1[e]);
        if (p.shared) tsum[e] = add2(tsum[e], t);
        if (p.gate) g[e] = mul2(g[e], f[e]);
        hf[e] = NORM ? mul2(t, wf[e]) : t;  // dgate
        if constexpr (NORM) {
          if (!p.shared) dw1[e] = fma2(g[e], u1[e], dw1[e]);
          g[e] = mul2(g[e], wf[e]);  // v
          vu = fma2(g[e], u1[e], vu);
        }
      }
      if (p.dgate_own) st16(p.dgate_own + at, narrow2<DT>(hf));
    }
    if constexpr (NORM) {
      float t[1] = {vu.x + vu.y};
      row_sums(s_sums, t, x++, C, peers);
      const float2 mean = both(-__fdiv_rn(t[0], p.cols));
#pragma unroll
      for (int e = 0; e < E / 2; e++) g[e] = mul2(q, fma2(u1[e], mean, g[e]));
    }
    if (ok) st16(p.dx + at, narrow2<DT>(g));
  }
  if (ok) {
    if (p.shared && from < end) flush(b, from, end);
    if (p.part_w) store_floats<E>(p.part_w + group * N + col, dw);
    if (p.part_w1) store_floats<E>(p.part_w1 + group * N + col, dw1);
  }
  if (!peers_ready) cluster_wait();
}

// Sums of partials, in a fixed order: block row 0 adds part_w over the groups, 1
// part_w1, and 2 + i the partials of a gate row, which lie in the spans of the
// groups that its rows touch: in the second partial of the first of them if the
// gate row begins inside that span, else in the first.  (Which groups: found on
// the host; the divisions took 50 us here for a gate row of 152.)  A block's threads
// take 8 float4 columns and 32 parts of the sum, their loads in flight in
// batches, and those are added in order: the partials were just written and
// come from L2, so the kernel is bound by one L2 latency and its launch.  Where no
// gate row has more than 32 partials a block takes 32 columns of one and 8 parts:
// there are fewer blocks, which else do not fit at once (W = 1, M = 1216, N = 16384
// bf16 with norms, 38 gate rows of 4 partials: the whole backward 90.9 us with 8
// columns, 74.7 with 32; four of 20 partials 71.6 and 70.0; 16 of 10 at M = 16384, N =
// 4096 149.0 and 146.0).
struct BranchSums {
  const float4* part_w;
  const float4* part_w1;
  const float4* part_gate;
  float4* dweight;
  float4* dnorm_weight;
  float4* dgate;
  const void* norm_weight;  // of `dtype`; null: the gate's partials are final
  int dtype;
  int groups;
  int vecs;                 // float4 in a row
  bool add, add_gate;       // to what the launch before this one left
  int gate_blocks;          // blocks that sum a gate row, 0: as many as the others
  struct Cut {
    uint32_t row;         // of the gate
    uint16_t first, count;  // groups
    bool inside;          // begins inside the first one's span
  } cut[kMaxBranchGroups];
};
static_assert(sizeof(BranchSums) <= 4096, "kernel parameters");

__device__ __forceinline__ float weight_at(const void* w, int dtype, int64_t i) {
  if (dtype == kFP32) return static_cast<const float*>(w)[i];
  if (dtype == kBF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
  return __half2float(static_cast<const __half*>(w)[i]);
}

// Block `block` of a job: float4 columns VECS * block .. of out.
template <int VECS, int BATCH>
__device__ __forceinline__ void sum_partials(float4 (&s)[256], const float4* from, const float4* head, int64_t stride, int count,
                                             int block, int vecs, float4* out, bool add, const void* scale, int dtype) {
  constexpr int PARTS = 256 / VECS;
  const int col = threadIdx.x % VECS, part = threadIdx.x / VECS;
  const int v = block * VECS + col;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (v < vecs) {
    for (int k0 = part; k0 < count; k0 += BATCH * PARTS) {
      float4 x[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; i++) {
        const int k = k0 + i * PARTS;
        x[i] = k < count ? __ldcg((k == 0 ? from : head + k * stride) + v) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < BATCH; i++) {
        a.x += x[i].x;
        a.y += x[i].y;
        a.z += x[i].z;
        a.w += x[i].w;
      }
    }
  }
  s[threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.x < 4 * VECS) {
    const float* c = reinterpret_cast<const float*>(s) + threadIdx.x;
    float sum[PARTS];
#pragma unroll
    for (int k = 0; k < PARTS; k++) sum[k] = c[k * 4 * VECS];
#pragma unroll
    for (int n = PARTS / 2; n > 0; n /= 2) {  // in pairs: five roundings instead of 31
#pragma unroll
      for (int k = 0; k < n; k++) sum[k] += sum[k + n];
    }
    const int64_t i = (int64_t)block * 4 * VECS + threadIdx.x;
    if (i < 4 * (int64_t)vecs) {
      float* to = reinterpret_cast<float*>(out) + i;
      const float v = scale ? sum[0] * weight_at(scale, dtype, i) : sum[0];
      *to = add ? *to + v : v;
    }
  }
}

__global__ void __launch_bounds__(256) branch_sums_kernel(const __grid_constant__ BranchSums p) {
  __shared__ float4 s[256];
  // blocks of the two weights, then those of the gate rows
  const int across = (p.vecs + 7) / 8, per_cut = p.gate_blocks ? p.gate_blocks : across;
  int job = 0, block = (int)blockIdx.x;
  if (block >= across) {
    job = 1;
    block -= across;
  }
  if (job == 1 && block >= across) {
    block -= across;
    job = 2 + block / per_cut;
    block -= (job - 2) * per_cut;
  }
  const float4 *from, *head;  // entry 0, entry k > 0 at head + k * stride
  float4* out;
  int count;
  int64_t stride = p.vecs;
  const void* scale = nullptr;
  if (job < 2) {
    from = head = job == 0 ? p.part_w : p.part_w1;
    out = job == 0 ? p.dweight : p.dnorm_weight;
    count = p.groups;
  } else {
    const BranchSums::Cut& c = p.cut[job - 2];
    count = c.count;
    stride = 2 * (int64_t)p.vecs;
    head = p.part_gate + c.first * stride;
    from = head + (c.inside ? p.vecs : 0);
    out = p.dgate + (int64_t)c.row * p.vecs;
    scale = p.norm_weight;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!out) return;
  if (job >= 2 && p.gate_blocks)
    sum_partials<32, 2>(s, from, head, stride, count, block, p.vecs, out, p.add_gate, scale, p.dtype);
  else
    sum_partials<8, 5>(s, from, head, stride, count, block, p.vecs, out, job < 2 ? p.add : p.add_gate, scale, p.dtype);
}

using BackwardFn = void (*)(const BranchBackwardParams);

template <int DT, bool NORM>
BackwardFn pick_ranks(int W) {
  switch (W) {
    case 1: return reduce_branch_rmsnorm_backward_kernel<DT, 1, NORM>;
    case 2: return reduce_branch_rmsnorm_backward_kernel<DT, 2, NORM>;
    case 4: return reduce_branch_rmsnorm_backward_kernel<DT, 4, NORM>;
    case 8: return reduce_branch_rmsnorm_backward_kernel<DT, 8, NORM>;
    case 16: return reduce_branch_rmsnorm_backward_kernel<DT, 16, NORM>;
    default: return reduce_branch_rmsnorm_backward_kernel<DT, 0, NORM>;
  }
}
BackwardFn pick(int dtype, int W, bool norm) {
  switch (dtype) {
    case kBF16: return norm ? pick_ranks<kBF16, true>(W) : pick_ranks<kBF16, false>(W);
    case kFP16: return norm ? pick_ranks<kFP16, true>(W) : pick_ranks<kFP16, false>(W);
    default: return norm ? pick_ranks<kFP32, true>(W) : pick_ranks<kFP32, false>(W);
  }
}

}  // namespace

// As branch_resident_groups, and at most kMaxBranchGroups.
cudaError_t branch_backward_resident_groups(int dtype, int W, const FusedShape& sh, int num_sms, int* groups) {
  int least = kMaxBranchGroups;
  for (int norm = 0; norm < 2; norm++) {
    const void* f = reinterpret_cast<const void*>(pick(dtype, W, norm != 0));
    int got = 0;
    cudaError_t e;
    if (sh.cluster == 1) {
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&got, f, sh.threads, 0);
      got *= num_sms;
    } else {
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = (unsigned)sh.cluster;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)sh.cluster, 1, 1);
      cfg.blockDim = dim3((unsigned)sh.threads, 1, 1);
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&got, f, &cfg);
    }
    if (e != cudaSuccess) return e;
    least = std::min(least, got);
  }
  *groups = least;
  return cudaSuccess;
}

cudaError_t launch_branch_backward(int dtype, int W, const RankPtrs& dy, const BranchArgs& br, const BranchGradArgs& g,
                                   const void* weight, float eps, unsigned int* err, int64_t rows, int64_t cols,
                                   int vec_per_row, const FusedShape& sh, const WaitHook& hook, cudaStream_t s) {
  BranchBackwardParams p;
  p.dy = dy;
  p.h = static_cast<const uint4*>(g.h);
  p.dres = static_cast<const uint4*>(g.dres);
  p.ar = static_cast<const uint4*>(g.ar);
  p.weight = static_cast<const uint4*>(weight);
  p.norm_weight = static_cast<const uint4*>(br.norm_weight);
  p.gate = static_cast<const uint4*>(br.gate);
  p.dx = static_cast<uint4*>(g.dx);
  p.dresidual = static_cast<uint4*>(g.dresidual);
  const bool own = br.gate && br.gate_span == 0, one = sh.groups == 1;
  p.dgate_own = own ? static_cast<uint4*>(g.dgate) : nullptr;
  p.dgate = own ? nullptr : static_cast<float*>(g.dgate);
  const size_t plane = (size_t)sh.groups * (size_t)cols;
  p.part_w = g.dweight ? (one ? g.dweight : g.workspace) : nullptr;
  p.part_w1 = g.dnorm_weight ? (one ? g.dnorm_weight : g.workspace + plane) : nullptr;
  p.part_gate = one ? nullptr : g.workspace + 2 * plane;
  p.err = err;
  p.drop = br.drop;
  p.residual_scale = br.residual_scale;
  p.eps = eps;
  p.norm_eps = br.norm_eps;
  p.cols = (float)cols;
  p.rows = rows;
  p.gate_span = (uint32_t)std::max<int64_t>(br.gate_span, 1);
  p.shared = br.gate && !own && (g.dgate || g.dnorm_weight);
  p.vec_per_row = vec_per_row;
  p.chunk = (vec_per_row + sh.cluster - 1) / sh.cluster;
  p.cluster = sh.cluster;
  p.nranks = W;
  p.wait_ns = hook.wait_ns;
  p.delay_ns = hook.delay_ns;
  p.delay_row = hook.delay_row;
  p.delay_cta = hook.delay_cta;
  cudaError_t e = launch_pdl(pick(dtype, W, br.norm_weight != nullptr), (unsigned)(sh.groups * sh.cluster), (unsigned)sh.threads,
                             0, s, (unsigned)sh.cluster, p);
  return e == cudaSuccess ? launch_branch_sums(br, g, dtype, sh.groups, rows, cols, false, false, s) : e;
}

cudaError_t launch_branch_sums(const BranchArgs& br, const BranchGradArgs& g, int dtype, int groups, int64_t rows,
                               int64_t cols, bool add, bool add_gate, cudaStream_t s) {
  const bool gates = br.gate && br.gate_span > 0 && g.dgate;
  if (groups == 1 || (!g.dweight && !g.dnorm_weight && !gates)) return cudaSuccess;
  BranchSums p;
  const size_t plane = (size_t)groups * (size_t)cols;
  p.part_w = reinterpret_cast<const float4*>(g.workspace);
  p.part_w1 = reinterpret_cast<const float4*>(g.workspace + plane);
  p.part_gate = reinterpret_cast<const float4*>(g.workspace + 2 * plane);
  p.dweight = reinterpret_cast<float4*>(g.dweight);
  p.dnorm_weight = reinterpret_cast<float4*>(g.dnorm_weight);
  p.dgate = static_cast<float4*>(gates ? g.dgate : nullptr);
  p.norm_weight = br.norm_weight;
  p.dtype = dtype;
  p.groups = groups;
  p.add = add;
  p.add_gate = add_gate;
  p.vecs = (int)(cols / 4);
  // gate rows that an inner border of the spans cuts, each once
  int cuts = 0, most = 0;  // and the partials of any of them
  if (gates) {
    int64_t start = 0;  // of span c - 1
    for (int c = 1; c < groups; c++) {
      const int64_t at = span_start(rows, groups, c), b = at / br.gate_span;
      if (at % br.gate_span != 0) {
        if (cuts > 0 && p.cut[cuts - 1].row == b)
          p.cut[cuts - 1].count++;
        else
          p.cut[cuts++] = {(uint32_t)b, (uint16_t)(c - 1), 2, start < b * br.gate_span};
      }
      start = at;
    }
  }
  for (int c = 0; c < cuts; c++) most = std::max<int>(most, p.cut[c].count);
  const int across = (p.vecs + 7) / 8;
  p.gate_blocks = most <= 32 ? (p.vecs + 31) / 32 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * across + cuts * (p.gate_blocks ? p.gate_blocks : across)), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, branch_sums_kernel, p);
}

}  // namespace car
