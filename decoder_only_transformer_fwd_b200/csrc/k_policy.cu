// Clipped policy loss with a KL term, forward and backward, from the logits.
//
// Per token with target y, from the row z of softcapped logits ("The
// Mathematics of Karpathy's nanochat", §Cross-Entropy Loss: log p = z_y -
// logsumexp z), the log-probabilities lo and lr that an old and a reference
// policy gave it, and the advantage A:
//   lp = z_y - logsumexp(z),  x = lp - lo,  r = e^x
//   L  = -min(r A, clip(r, 1 - cl, 1 + ch) A) + beta (e^d - d - 1),  d = lr - lp
//   dL/dlp = (-r A unless the clipped branch is the smaller) + beta (1 - e^d)
//   dL/dz_v = dL/dlp ([v = y] - e^{z_v - logsumexp z})
// weighted by w_t and summed.  The clipped branch is the smaller one when
// A > 0 and x > log(1 + ch), or A < 0 and x < log(1 - cl); lp and both borders
// are held in fp64, since a token on the wrong side of a border changes its
// whole gradient row.
//
// HBM bound: the logits in once, the gradient out once (2 V elements per
// token).  Three forms, by a row's bytes:
//   k_policy_warp  rows up to 8 KB: a warp takes a row at a time;
//   k_policy_rows  rows up to 20 KB (fp32) or 40 KB (bf16): a CTA takes a row at a
//     time.  Both make one pass with a running maximum and sum, then a second one
//     that reads the row again (from L2, where the first left it) and writes the
//     gradient.  Many rows per SM cover each other's latencies.
//   k_policy_ring  longer rows: bulk copies bring a row into a shared-memory
//     ring, both passes read it there, and the next row's copies run meanwhile.
#include <cfloat>

#include "nc_internal.cuh"
#include "ptx.cuh"

namespace nc {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp_diff(float z, float m) {
  // the difference first: its rounding does not grow with |m|
  return ptx::ex2((z - m) * kLog2e);
}

// 16 bytes of a row
template <typename T> struct Quad;
template <> struct Quad<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void ld(const float* p, float (&f)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  }
  static __device__ __forceinline__ void st(float* p, const float (&f)[4]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
  }
};
template <> struct Quad<bf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void ld(const bf16* p, float (&f)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void st(bf16* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&v);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  }
};

// elements of `p`'s row before its first 16-byte boundary
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int V) {
  const int h = (int)(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T));
  return h < V ? h : V;
}

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The KL term e^d - d - 1 and its slope e^d - 1, neither with cancellation: the
// term's series where its terms fall fast (|d| <= 1/2: the first one left out is
// 2^-28 of the sum), else from expm1, which is then the slope (a term of 2^30
// would swallow its -1).
__device__ __forceinline__ float exp_excess(float d, float* slope) {
  if (fabsf(d) > 0.5f) {
    *slope = expm1f(d);
    return *slope - d;
  }
  float s = 1.0f / 3628800;
  s = fmaf(s, d, 1.0f / 362880);
  s = fmaf(s, d, 1.0f / 40320);
  s = fmaf(s, d, 1.0f / 5040);
  s = fmaf(s, d, 1.0f / 720);
  s = fmaf(s, d, 1.0f / 120);
  s = fmaf(s, d, 1.0f / 24);
  s = fmaf(s, d, 1.0f / 6);
  s = fmaf(s, d, 0.5f);
  s = s * d * d;
  *slope = s + d;
  return s;
}

// log of a sum S >= 1 in fp64, from a table in shared memory (Tang's method:
// "Table-driven implementation of the logarithm function", 1990): S = 2^k m,
// c = 1 + i/128 next to m in [1, 2), log S = k log 2 + log c + log(1 + r) with
// r = m / c - 1, |r| <= 2^-8, and six terms of the series (the next one is
// below 2^-58); S = 1 gives 0.  The library's log takes 0.4 us on the critical
// path of a row.
constexpr int kLogTable = 129;
__device__ __forceinline__ void fill_log_table(double2* tab, int tid, int threads) {
  for (int i = tid; i < kLogTable; i += threads) {
    const double inv = 1.0 / (1.0 + i / 128.0);
    tab[i] = make_double2(inv, -log(inv));
  }
}
__device__ __forceinline__ double log_sum(double S, const double2* tab) {
  const int hi = __double2hiint(S), k = (hi >> 20) - 1023;
  if ((unsigned)k > 1000u) return log(S);  // 0, infinity, NaN
  const double m = __hiloint2double((hi & 0xfffff) | 0x3ff00000, __double2loint(S));
  const double2 c = tab[((hi & 0xfffff) + 0x1000) >> 13];
  const double r = fma(m, c.x, -1.0), r2 = r * r;
  const double p = fma(r2, fma(r2, fma(r, -1.0 / 6, 0.2), fma(r, -0.25, 1.0 / 3)), fma(r, -0.5, 1.0));
  return fma((double)k, 0.6931471805599453, c.y) + r * p;
}

// what a token's row leaves: dL/dz_v = coef e^{z_v - top} + gz [v = y]
struct Row {
  float coef, gz;
};
struct RowStats {  // the last three weighted
  double lp, loss, kl, clipped;
};

// The part of a row's terms that its gradient waits for, from its maximum m and
// sum S of e^{z - m}; w: the token's weight.  One thread per row runs this while
// the others wait: fp64 only where the result needs it (lp and the comparison
// with the borders).
//
// e^x with x > kFar may pass fp32's range although the weighted term does not:
// r and kl (and the slope) then hold e^{x/2}, by which the weight is multiplied
// twice.  The KL term's -1 and -d are below a rounding there.  (The terms in fp64
// instead: 0.5 to 2.5% more time for rows up to 48 KB.)
constexpr float kFar = 80.f;
struct Terms {
  double lp, A, w;
  float r, kl;
  bool cut, far_r, far_kl;
  __device__ __forceinline__ Row begin(const PolicyArgs& a, float zy, float m, double S, const double2* tab, float adv,
                                       float old, float ref, double weight) {
    lp = ((double)zy - (double)m) - log_sum(S, tab);
    w = weight;
    A = (double)adv;
    const double x = a.old_logp != nullptr ? lp - (double)old : 0.0;
    cut = (A > 0.0 && x > a.log_high) || (A < 0.0 && x < a.log_low);
    // with the branch decided, fp32 does: the exponents are differences
    const float xf = (float)x;
    far_r = xf > kFar;
    r = expf(far_r ? 0.5f * xf : xf);
    // a term of weight 0 has no part in the gradient, however large it is (0 x inf)
    const float gain = cut || adv == 0.f ? 0.f : -r * adv;
    float cost = 0.f, rise = 0.f;
    kl = 0.f, far_kl = false;
    if (a.ref_logp != nullptr) {
      const float d = (float)((double)ref - lp);
      far_kl = d > kFar;
      kl = exp_excess(far_kl ? 0.5f * d : d, &rise);
      if (a.kl_beta > 0.f) cost = a.kl_beta * rise;
    }
    const float wf = (float)w;
    Row t;
    t.gz = wf * (gain - cost);
    if (far_r || far_kl) t.gz = wf * gain * (far_r && gain != 0.f ? r : 1.f) - wf * cost * (far_kl && cost != 0.f ? rise : 1.f);
    t.coef = -t.gz * (1.0f / (float)S);
    return t;
  }
  __device__ __forceinline__ RowStats finish(const PolicyArgs& a) const {
    RowStats t;
    t.lp = lp;
    const double ratio = (double)r * (far_r ? (double)r : 1.0), excess = (double)kl * (far_kl ? (double)kl : 1.0);
    const double gain = A == 0.0 ? (lp != lp ? lp : 0.0) : (cut ? (A > 0.0 ? a.ratio_high : a.ratio_low) : ratio) * A;
    t.loss = w * ((a.kl_beta > 0.f ? (double)a.kl_beta * excess : 0.0) - gain);
    t.kl = w * excess;
    t.clipped = cut ? w : 0.0;
    return t;
  }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// e^{f - top} of a pair, in packed fp32 (the special-function unit's rate of 16
// a clock bounds both passes, so the rest is kept short)
__device__ __forceinline__ float2 exp_pair(float2 f, float2 neg_top) {
  const float2 x = __fmul2_rn(__fadd2_rn(f, neg_top), make_float2(kLog2e, kLog2e));
  return make_float2(ptx::ex2(x.x), ptx::ex2(x.y));
}

struct Online {
  float m = -FLT_MAX, s = 0.f;
  __device__ __forceinline__ void add1(float f) {
    const float t = fmaxf(m, f);
    s = s * exp_diff(m, t) + exp_diff(f, t);
    m = t;
  }
  // K words of N elements, with one step of the maximum
  template <int K, int N>
  __device__ __forceinline__ void add_all(const float (&f)[K][N]) {
    float t[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      t[j] = fmaxf(f[j][0], f[j][1]);
#pragma unroll
      for (int i = 2; i < N; i += 2) t[j] = max3(t[j], f[j][i], f[j][i + 1]);
    }
    float top = m;
#pragma unroll
    for (int j = 0; j < K; ++j) top = fmaxf(top, t[j]);
    const float2 nt = make_float2(-top, -top);
    float2 e[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      e[j] = exp_pair(make_float2(f[j][0], f[j][1]), nt);
#pragma unroll
      for (int i = 2; i < N; i += 2) e[j] = __fadd2_rn(e[j], exp_pair(make_float2(f[j][i], f[j][i + 1]), nt));
    }
    s *= exp_diff(m, top);
#pragma unroll
    for (int j = 0; j < K; ++j) s += e[j].x + e[j].y;
    m = top;
  }
};

// a token's weight, from the count of tokens (norm 0) or of sequences and the
// tokens of its own (norm 1)
__device__ __forceinline__ double weight_of(const PolicyArgs& a, int count, int tokens) {
  return a.norm == 0 ? 1.0 / count : 1.0 / ((double)count * tokens);
}

__device__ __forceinline__ bool valid(int y, int V) { return (unsigned)y < (unsigned)V; }

// tokens (norm 0) or sequences (norm 1) with a target, by the block's threads
// first .. first + threads - 1; this thread's share of the sum
__device__ __forceinline__ int count_share(const PolicyArgs& a, int tid, int threads) {
  int n = 0;
  if (a.norm == 0) {
    const int M = a.B * a.T;
    const int head = min(M, (int)((16 - (reinterpret_cast<uintptr_t>(a.targets) & 15)) & 15) / 4), quads = (M - head) / 4;
    const int4* q = reinterpret_cast<const int4*>(a.targets + head);
#pragma unroll 4
    for (int i = tid; i < quads; i += threads) {
      const int4 v = q[i];
      n += valid(v.x, a.V) + valid(v.y, a.V) + valid(v.z, a.V) + valid(v.w, a.V);
    }
    if (tid < head) n += valid(a.targets[tid], a.V);
    if (head + 4 * quads + tid < M && tid < 4) n += valid(a.targets[head + 4 * quads + tid], a.V);
  } else {
    const int lane = tid & 31;
    for (int b = tid >> 5; b < a.B; b += threads >> 5) {
      bool any = false;
      for (int t0 = 0; t0 < a.T && !any; t0 += 32)
        any = __any_sync(0xffffffffu, t0 + lane < a.T && valid(a.targets[(size_t)b * a.T + t0 + lane], a.V));
      n += lane == 0 && any;
    }
  }
  return n;
}

// 16 bytes of the gradient, from element v0 of the row on
template <typename T>
__device__ __forceinline__ void grad_quad(float (&f)[Quad<T>::N], int v0, int y, const Row& t, float top) {
  const float2 nt = make_float2(-top, -top), c = make_float2(t.coef, t.coef);
#pragma unroll
  for (int e = 0; e < Quad<T>::N; e += 2) {
    const float2 g = __fmul2_rn(exp_pair(make_float2(f[e], f[e + 1]), nt), c);
    f[e] = g.x;
    f[e + 1] = g.y;
  }
  if ((unsigned)(y - v0) < (unsigned)Quad<T>::N) {
#pragma unroll
    for (int e = 0; e < Quad<T>::N; ++e) f[e] += v0 + e == y ? t.gz : 0.f;
  }
}

// A row without a target: zeros.
template <typename T>
__device__ __forceinline__ void zero_row(T* dz, int V, int tid, int threads) {
  const int head = head_of(dz, V), nq = (V - head) / Quad<T>::N, tail = head + nq * Quad<T>::N;
  if (tid < head) Act<T>::st(dz + tid, 0.f);
  if (tail + tid < V) Act<T>::st(dz + tail + tid, 0.f);
  float f[Quad<T>::N] = {};
  for (int i = tid; i < nq; i += threads) Quad<T>::st(dz + head + (size_t)i * Quad<T>::N, f);
}

// the second pass over a row: threads tid, tid + threads, ...
template <typename T>
__device__ __forceinline__ void write_grad(const T* z, T* dz, int V, int y, const Row& t, float top, int tid, int threads) {
  // the gradient's own 16-byte boundaries; the logits at the same element
  // offsets when both rows start alike, else one element at a time
  const int head = head_of(dz, V);
  const bool alike = ((reinterpret_cast<uintptr_t>(dz) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
  const int nq = (V - head) / Quad<T>::N, tail = head + nq * Quad<T>::N;
  auto one = [&](int v) { Act<T>::st(dz + v, t.coef * exp_diff(Act<T>::ld(z + v), top) + (v == y ? t.gz : 0.f)); };
  if (tid < head) one(tid);
  if (tail + tid < V) one(tail + tid);
#pragma unroll 4
  for (int i = tid; i < nq; i += threads) {
    const int v0 = head + i * Quad<T>::N;
    float f[Quad<T>::N];
    if (alike) {
      Quad<T>::ld(z + v0, f);
    } else {
#pragma unroll
      for (int e = 0; e < Quad<T>::N; ++e) f[e] = Act<T>::ld(z + v0 + e);
    }
    grad_quad<T>(f, v0, y, t, top);
    Quad<T>::st(dz + v0, f);
  }
}

// the first pass: this thread's running maximum and sum
template <typename T>
__device__ __forceinline__ Online row_sum(const T* z, int V, int tid, int threads) {
  const int head = head_of(z, V), nq = (V - head) / Quad<T>::N, tail = head + nq * Quad<T>::N;
  Online o;
  if (tid < head) o.add1(Act<T>::ld(z + tid));
  if (tail + tid < V) o.add1(Act<T>::ld(z + tail + tid));
#pragma unroll 4
  for (int i = tid; i < nq; i += threads) {
    float f[1][Quad<T>::N];
    Quad<T>::ld(z + head + (size_t)i * Quad<T>::N, f[0]);
    o.add_all(f);
  }
  return o;
}

// Short rows: a warp takes `per` consecutive rows (of one sequence, mostly, so
// that its tokens are counted once), one after the other.
constexpr int kWarpRows = 8, kWarpCtas = 4;  // rows at a time per CTA, CTAs per SM
template <typename T>
__global__ void __launch_bounds__(32 * kWarpRows, kWarpCtas) k_policy_warp(const PolicyArgs a, double* part, int per) {
  __shared__ double s_sum[kWarpRows][3];
  __shared__ int s_count;
  __shared__ double2 s_log[kLogTable];
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  fill_log_table(s_log, tid, 32 * kWarpRows);
  if (tid == 0) s_count = 0;
  pdl_wait();
  __syncthreads();
  const int share = __reduce_add_sync(0xffffffffu, count_share(a, tid, 32 * kWarpRows));
  if (lane == 0 && share != 0) atomicAdd(&s_count, share);
  __syncthreads();
  const int count = s_count, M = a.B * a.T, V = a.V;
  const double w_all = count > 0 ? 1.0 / count : 0.0;
  double part_of = 1.0, sums[3] = {0.0, 0.0, 0.0};
  const long long first = ((long long)blockIdx.x * kWarpRows + warp) * per;
  const int last = (int)min(first + per, (long long)M);
  int last_b = -1;
  for (int row = (int)min(first, (long long)M); row < last; ++row) {
    const T* z = static_cast<const T*>(a.logits) + (size_t)row * a.ldl;
    T* dz = a.dlogits != nullptr ? static_cast<T*>(a.dlogits) + (size_t)row * a.lddl : nullptr;
    const int y = a.targets[row];
    if (!valid(y, V)) {
      if (lane == 0) {
        a.out_logp[row] = 0.f;
        if (y != -1) atomicOr(a.status, kStatusData);
      }
      if (dz != nullptr) zero_row(dz, V, lane, 32);
      continue;
    }
    const float zy = Act<T>::ld(z + y), adv = a.advantages[a.adv_per_token ? row : row / a.T];
    const float old = a.old_logp != nullptr ? a.old_logp[row] : 0.f, ref = a.ref_logp != nullptr ? a.ref_logp[row] : 0.f;
    if (a.norm == 1 && row / a.T != last_b) {
      last_b = row / a.T;
      int mine = 0;
#pragma unroll 4
      for (int t = lane; t < a.T; t += 32) mine += valid(a.targets[(size_t)last_b * a.T + t], V);
      part_of = 1.0 / __reduce_add_sync(0xffffffffu, mine);
    }
    const Online o = row_sum(z, V, lane, 32);
    const float top = warp_max(o.m);
    const double S = warp_sum_d((double)(o.s * exp_diff(o.m, top)));
    // all lanes work the terms out alike
    Terms terms;
    const Row t = terms.begin(a, zy, top, S, s_log, adv, old, ref, w_all * part_of);
    if (dz != nullptr) write_grad(z, dz, V, y, t, top, lane, 32);
    if (lane == 0) {
      const RowStats st = terms.finish(a);
      a.out_logp[row] = (float)st.lp;
      sums[0] += st.loss;
      sums[1] += st.kl;
      sums[2] += st.clipped;
    }
  }
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i) s_sum[warp][i] = sums[i];
  }
  __syncthreads();
  if (tid < 3) {
    double v = 0.0;
    for (int i = 0; i < kWarpRows; ++i) v += s_sum[i][tid];
    part[3 * blockIdx.x + tid] = v;
  }
}

constexpr int kRowThreads = 1280;  // per SM
template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kRowThreads / kThreads) k_policy_rows(const PolicyArgs a, double* part) {
  __shared__ float s_m[kThreads / 32];
  __shared__ double s_s[kThreads / 32];
  __shared__ Row s_row;
  __shared__ float s_top;
  __shared__ int s_count;
  __shared__ double2 s_log[kLogTable];
  pdl_launch_dependents();
  fill_log_table(s_log, threadIdx.x, kThreads);
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int M = a.B * a.T, V = a.V;
  if (tid == 0) s_count = 0;
  __syncthreads();
  const int share = __reduce_add_sync(0xffffffffu, count_share(a, tid, kThreads));
  if (lane == 0 && share != 0) atomicAdd(&s_count, share);
  __syncthreads();
  const int count = s_count;
  double sum_loss = 0.0, sum_kl = 0.0, sum_clip = 0.0;  // thread 0's
  for (int row = blockIdx.x; row < M; row += gridDim.x) {
    const T* z = static_cast<const T*>(a.logits) + (size_t)row * a.ldl;
    T* dz = a.dlogits != nullptr ? static_cast<T*>(a.dlogits) + (size_t)row * a.lddl : nullptr;
    const int y = a.targets[row];
    if (!valid(y, V)) {  // no target, or a bad one: recorded, and the token counts as padding
      if (tid == 0) {
        a.out_logp[row] = 0.f;
        if (y != -1) atomicOr(a.status, kStatusData);
      }
      if (dz != nullptr) zero_row(dz, V, tid, kThreads);
      continue;
    }
    int tokens = count;
    if (a.norm == 1) {
      const int32_t* tg = a.targets + (size_t)(row / a.T) * a.T;
      tokens = 0;
      for (int t0 = 0; t0 < a.T; t0 += kThreads) tokens += __syncthreads_count(t0 + tid < a.T && valid(tg[t0 + tid], V));
    }
    const Online o = row_sum(z, V, tid, kThreads);
    const float wm = warp_max(o.m);
    const double ws = warp_sum_d((double)(o.s * exp_diff(o.m, wm)));
    if (lane == 0) {
      s_m[warp] = wm;
      s_s[warp] = ws;
    }
    __syncthreads();
    if (warp == 0) {
      const bool mine = lane < kThreads / 32;
      const float m0 = mine ? s_m[lane] : -FLT_MAX, m = warp_max(m0);
      const double S = warp_sum_d(mine ? s_s[lane] * (double)exp_diff(m0, m) : 0.0);
      if (lane == 0) {
        Terms terms;
        s_row = terms.begin(a, Act<T>::ld(z + y), m, S, s_log, a.advantages[a.adv_per_token ? row : row / a.T],
                            a.old_logp != nullptr ? a.old_logp[row] : 0.f, a.ref_logp != nullptr ? a.ref_logp[row] : 0.f,
                            weight_of(a, count, tokens));
        s_top = m;
        const RowStats t = terms.finish(a);
        a.out_logp[row] = (float)t.lp;
        sum_loss += t.loss;
        sum_kl += t.kl;
        sum_clip += t.clipped;
      }
    }
    __syncthreads();
    if (dz != nullptr) {
      const Row t = s_row;
      write_grad(z, dz, V, y, t, s_top, tid, kThreads);
    }
    __syncthreads();  // the next row reuses the scratch
  }
  if (tid == 0) {
    part[3 * blockIdx.x] = sum_loss;
    part[3 * blockIdx.x + 1] = sum_kl;
    part[3 * blockIdx.x + 2] = sum_clip;
  }
}

// Long rows.  All warps but the last work, the last one copies: a row's 16-byte words (up to 15
// bytes at either end are read directly) in chunks of 16 KB, chunk n of the
// CTA's sequence in slot n % NS.  Pass 1 leaves the row's last NS chunks where
// they are; pass 2 takes those first and frees them, and then the ones before,
// which were freed at once and are copied again (from L2).  CTA c takes the c-th
// row with a target, the (c + gridDim.x)-th and so on, which the copying warp
// finds by counting, so that padding leaves all CTAs the same work; between them
// the others write the zeros of rows without a target.
constexpr int kChunk = 16384, kMeta = 16;
template <int CPS> struct Ring {
  static constexpr int NS = CPS == 1 ? 13 : CPS == 2 ? 6 : 3;             // slots
  static constexpr int WORK = CPS == 1 ? 512 : CPS == 2 ? 256 : 128;      // working threads
  static constexpr int SMEM = NS * kChunk + 1024;
};

template <typename T, int CPS>
__global__ void __launch_bounds__(Ring<CPS>::WORK + 32, CPS) k_policy_ring(const PolicyArgs a, double* part) {
  constexpr int kWork = Ring<CPS>::WORK, kWarps = kWork / 32, NS = Ring<CPS>::NS, N = Quad<T>::N, kVec = kChunk / 16, kWords = kVec / kWork;
  static_assert(NS <= kMeta, "a row has a chunk at least, so the copies run less than kMeta rows ahead");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  __shared__ uint64_t bars[2 * NS + 2];
  __shared__ Row s_row[2];
  __shared__ float s_top[2];
  // of the CTA's k-th row, at k % kMeta: the row (-1: there is none) and its
  // target, there with its first chunk; norm 1: 1 / its sequence's tokens
  __shared__ int s_at[kMeta], s_y[kMeta];
  __shared__ double s_part[kMeta];
  __shared__ double2 s_log[kLogTable];
  __shared__ float s_m[2][kWarps];
  __shared__ double s_s[2][kWarps];
  __shared__ int s_count;
  __shared__ volatile int abort_flag;
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto full = [&](int n) { return bar0 + 8u * (n % NS); };
  auto empty = [&](int n) { return bar0 + 8u * (NS + n % NS); };
  const uint32_t red = bar0 + 8u * (2 * NS), ready = bar0 + 8u * (2 * NS + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int M = a.B * a.T, V = a.V;
  pdl_launch_dependents();
  fill_log_table(s_log, tid, kWork + 32);
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), kWarps);
    }
    ptx::mbar_init(red, kWarps);
    ptx::mbar_init(ready, 1);
    s_count = 0;
    abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  __syncthreads();
  pdl_wait();
  const bool grad = a.dlogits != nullptr;
  if (warp == kWarps) {
    int n = 0, last_b = -1, k = 0;
    double part_of = 1.0;
    bool ok = true;
    auto take = [&](int row, int y) {
      const T* z = static_cast<const T*>(a.logits) + (size_t)row * a.ldl;
      const int head = head_of(z, V), nq = (V - head) / N, C = (nq + kVec - 1) / kVec;
      const int again = grad && C > NS ? C - NS : 0;
      auto copy = [&](int i) {  // the row's i-th chunk in the order of use; lane 0
        const int c = i < C ? i : i - C;
        const uint32_t bytes = (uint32_t)min(kVec, nq - c * kVec) * 16u;
        if (abort_flag || !ptx::mbar_wait(empty(n), ((uint32_t)(n / NS) & 1u) ^ 1u, a.status)) return false;
        if (i == 0) {
          s_at[k % kMeta] = row;
          s_y[k % kMeta] = y;
        }
        ptx::mbar_arrive_expect_tx(full(n), bytes);
        ptx::bulk_load(ptx::smem_u32(ring + (n % NS) * kChunk), z + head + (size_t)c * kVec * N, bytes, full(n));
        ++n;
        return true;
      };
      // the sequence's share per token is there with the row's last chunk
      if (lane == 0 && C > 1) ok = copy(0);
      if (a.norm == 1 && row / a.T != last_b) {
        last_b = row / a.T;
        int mine = 0;
#pragma unroll 4
        for (int t = lane; t < a.T; t += 32) mine += valid(a.targets[(size_t)last_b * a.T + t], V);
        part_of = 1.0 / __reduce_add_sync(0xffffffffu, mine);
      }
      if (lane == 0) {
        s_part[k % kMeta] = part_of;
        for (int i = C > 1; ok && i < C + again; ++i) ok = copy(i);
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      ++k;
    };
    // 128 targets at a time, the next ones on their way
    constexpr int kScan = 4;
    int y[kScan], y_next[kScan], before = 0, rank = blockIdx.x;
    auto load = [&](int base) {
#pragma unroll
      for (int i = 0; i < kScan; ++i) y_next[i] = base + 32 * i + lane < M ? a.targets[base + 32 * i + lane] : -1;
    };
    load(0);
    for (int base = 0; ok && base < M; base += 32 * kScan) {
#pragma unroll
      for (int i = 0; i < kScan; ++i) y[i] = y_next[i];
      if (base < M - 32 * kScan) load(base + 32 * kScan);
#pragma unroll
      for (int i = 0; i < kScan; ++i) {
        const unsigned has = __ballot_sync(0xffffffffu, valid(y[i], V));
        const int mine = before + __popc(has & ((1u << lane) - 1u));
        while (ok && rank < before + __popc(has)) {
          const int src = __ffs((int)__ballot_sync(0xffffffffu, ((has >> lane) & 1u) != 0u && mine == rank)) - 1;
          take(base + 32 * i + src, __shfl_sync(0xffffffffu, y[i], src));
          rank += gridDim.x;
        }
        before += __popc(has);
      }
    }
    if (lane == 0 && ok) {  // no more rows
      ok = !abort_flag && ptx::mbar_wait(empty(n), ((uint32_t)(n / NS) & 1u) ^ 1u, a.status);
      if (ok) {
        s_at[k % kMeta] = -1;
        ptx::mbar_arrive(full(n));
        ++n;
      }
    }
    if (lane == 0) {
      if (!ok) abort_flag = 1;
      // every copy issued here has landed before the CTA may exit
      for (int i = max(0, n - NS); i < n; ++i) ptx::mbar_wait(full(i), (uint32_t)(i / NS) & 1u, a.status);
    }
  } else {
    const int share = __reduce_add_sync(0xffffffffu, count_share(a, tid, kWork));
    if (lane == 0) {
      if (share != 0) atomicAdd(&s_count, share);
      ptx::mbar_arrive(red);
    }
    bool ok = ptx::mbar_wait(red, 0, a.status);
    const int count = *(volatile int*)&s_count;
    double sum_loss = 0.0, sum_kl = 0.0, sum_clip = 0.0;
    int n = 0, k = 0;  // chunks and rows done
    const double w_all = count > 0 ? 1.0 / count : 0.0;
    auto wait_full = [&](int i) -> bool { return !abort_flag && ptx::mbar_wait(full(i), (uint32_t)(i / NS) & 1u, a.status); };
    // the zeros of rows without a target: the CTA's next row to look at
    int look = blockIdx.x, y_look = look < M ? a.targets[look] : -1;
    auto look_at_one = [&] {
      const int row = look, y = y_look;
      look += gridDim.x;
      y_look = look < M ? a.targets[look] : -1;
      if (valid(y, V)) return;
      if (tid == 0) {
        a.out_logp[row] = 0.f;
        if (y != -1) atomicOr(a.status, kStatusData);  // a bad target: recorded, and the token counts as padding
      }
      if (grad) zero_row(static_cast<T*>(a.dlogits) + (size_t)row * a.lddl, V, tid, kWork);
    };
    while (ok) {
      if (!wait_full(n)) {
        ok = false;
        break;
      }
      const int row = s_at[k % kMeta], y = s_y[k % kMeta];
      if (row < 0) break;
      const T* z = static_cast<const T*>(a.logits) + (size_t)row * a.ldl;
      T* dz = static_cast<T*>(a.dlogits) + (size_t)row * a.lddl;
      T zy = T(0.f);
      float adv = 0.f, old = 0.f, ref = 0.f;
      if (tid == 0) {  // on their way while the row is summed
        zy = z[y];
        adv = a.advantages[a.adv_per_token ? row : row / a.T];
        if (a.old_logp != nullptr) old = a.old_logp[row];
        if (a.ref_logp != nullptr) ref = a.ref_logp[row];
      }
      const int head = head_of(z, V), nq = (V - head) / N, tail = head + nq * N, C = (nq + kVec - 1) / kVec;
      const int again = grad && C > NS ? C - NS : 0;
      // the element at either end that this thread has, if any
      const int edge = tid < head ? tid : (tid >= 32 && tail + tid - 32 < V ? tail + tid - 32 : -1);
      Online o;
      float ze = 0.f;
      if (edge >= 0) {
        ze = Act<T>::ld(z + edge);
        o.add1(ze);
      }
      auto release = [&](int i) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(empty(i));
      };
      for (int c = 0; c < C; ++c) {
        if (!wait_full(n + c)) {
          ok = false;
          break;
        }
        const T* src = reinterpret_cast<const T*>(ring + ((n + c) % NS) * kChunk);
        if ((c + 1) * kVec <= nq) {  // one maximum for all of the thread's words
          float f[kWords][N];
#pragma unroll
          for (int j = 0; j < kWords; ++j) Quad<T>::ld(src + (tid + j * kWork) * N, f[j]);
          o.add_all(f);
        } else {
#pragma unroll
          for (int j = 0; j < kWords; ++j) {
            const int i = tid + j * kWork;
            if (c * kVec + i < nq) {
              float f[1][N];
              Quad<T>::ld(src + i * N, f[0]);
              o.add_all(f);
            }
          }
        }
        if (c < again || !grad) release(n + c);
      }
      if (!ok) break;
      const float wm = warp_max(o.m);
      const double ws = warp_sum_d((double)(o.s * exp_diff(o.m, wm)));
      if (lane == 0) {
        s_m[k & 1][warp] = wm;
        s_s[k & 1][warp] = ws;
        ptx::mbar_arrive(red);
      }
      // warp 0 joins the warps' sums and works out the row's terms
      if (warp == 0) {
        if (abort_flag || !ptx::mbar_wait(red, (uint32_t)(k + 1) & 1u, a.status)) {
          ok = false;
          break;
        }
        const float m0 = s_m[k & 1][lane % kWarps];  // every kWarps lanes hold the same
        float m = m0;
#pragma unroll
        for (int x = kWarps / 2; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        double S = s_s[k & 1][lane % kWarps] * (double)exp_diff(m0, m);
#pragma unroll
        for (int x = kWarps / 2; x > 0; x >>= 1) S += __shfl_xor_sync(0xffffffffu, S, x);
        if (lane == 0) {
          Terms terms;
          s_row[k & 1] = terms.begin(a, (float)zy, m, S, s_log, adv, old, ref, a.norm == 0 ? w_all : w_all * s_part[k % kMeta]);
          s_top[k & 1] = m;
          ptx::mbar_arrive(ready);
          const RowStats t = terms.finish(a);
          a.out_logp[row] = (float)t.lp;
          sum_loss += t.loss;
          sum_kl += t.kl;
          sum_clip += t.clipped;
        }
      }
      if (abort_flag || !ptx::mbar_wait(ready, (uint32_t)k & 1u, a.status)) {
        ok = false;
        break;
      }
      const Row t = s_row[k & 1];
      const float top = s_top[k & 1];
      if (grad) {
        const bool alike = ((reinterpret_cast<uintptr_t>(dz) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
        for (int i = again; i < C + again; ++i) {
          const int c = i < C ? i : i - C;  // chunks again .. C - 1, then 0 .. again - 1
          if (i >= C && !wait_full(n + i)) {
            ok = false;
            break;
          }
          const T* src = reinterpret_cast<const T*>(ring + ((n + i) % NS) * kChunk);
#pragma unroll
          for (int j = 0; j < kWords; ++j) {
            const int q = c * kVec + tid + j * kWork, v0 = head + q * N;
            if (q < nq) {
              float f[N];
              Quad<T>::ld(src + (tid + j * kWork) * N, f);
              grad_quad<T>(f, v0, y, t, top);
              if (alike) {
                Quad<T>::st(dz + v0, f);
              } else {
#pragma unroll
                for (int e = 0; e < N; ++e) Act<T>::st(dz + v0 + e, f[e]);
              }
            }
          }
          release(n + i);
        }
        if (edge >= 0) Act<T>::st(dz + edge, t.coef * exp_diff(ze, top) + (edge == y ? t.gz : 0.f));
      }
      n += C + again;
      ++k;
      if (look < M) look_at_one();
    }
    while (ok && look < M) look_at_one();
    if (!ok) abort_flag = 1;
    if (tid == 0) {
      part[3 * blockIdx.x] = sum_loss;
      part[3 * blockIdx.x + 1] = sum_kl;
      part[3 * blockIdx.x + 2] = sum_clip;
    }
  }
}

// the CTAs' sums in a fixed order, one warp per statistic, eight loads in flight
__global__ void __launch_bounds__(96) k_policy_stats(const double* part, int n, float* out) {
  pdl_launch_dependents();
  pdl_wait();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double s = 0.0;
  for (int i0 = lane; i0 < n; i0 += 256) {
    double v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = i0 + 32 * k < n ? part[3 * (i0 + 32 * k) + w] : 0.0;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += v[k];
  }
  s = warp_sum_d(s);
  if (lane == 0) out[w] = (float)s;
}

}  // namespace

template <typename T, int THREADS>
static int run_rows(const PolicyArgs& a, double* part, int num_sms, cudaStream_t st) {
  const int M = a.B * a.T;
  int grid = num_sms * (kRowThreads / THREADS) < kPolicyMaxCtas ? num_sms * (kRowThreads / THREADS) : kPolicyMaxCtas;
  if (grid > M) grid = M;
  launch_pdl(k_policy_rows<T, THREADS>, dim3(grid), dim3(THREADS), 0, st, 1, a, part);
  return grid;
}

template <typename T>
static int run_warp(const PolicyArgs& a, double* part, int num_sms, cudaStream_t st) {
  const int M = a.B * a.T;
  int grid = num_sms * kWarpCtas < kPolicyMaxCtas ? num_sms * kWarpCtas : kPolicyMaxCtas;
  const int per = (M + grid * kWarpRows - 1) / (grid * kWarpRows);
  grid = (M + per * kWarpRows - 1) / (per * kWarpRows);
  launch_pdl(k_policy_warp<T>, dim3(grid), dim3(32 * kWarpRows), 0, st, 1, a, part, per);
  return grid;
}

template <typename T, int CPS>
static int run_ring(const PolicyArgs& a, double* part, int num_sms, cudaStream_t st) {
  const int M = a.B * a.T, grid = num_sms * CPS < M ? num_sms * CPS : M;
  if (!smem_optin(k_policy_ring<T, CPS>, Ring<CPS>::SMEM)) return 0;
  launch_pdl(k_policy_ring<T, CPS>, dim3(grid), dim3(Ring<CPS>::WORK + 32), Ring<CPS>::SMEM, st, 1, a, part);
  return grid;
}

template <typename T>
static int run(const PolicyArgs& a, double* part, int num_sms, cudaStream_t st) {
  const size_t bytes = (size_t)a.V * sizeof(T);
  const int M = a.B * a.T;
  // Up to a row per SM, more threads have it sooner (64 rows of 32768 fp32 words:
  // 9.9 us with 512, 12.3 with 256; 100 rows of 20000 bf16 words 7.9 with 512,
  // 11.3 with 128).
  // Beyond, measured in us with gradient, three quarters of the rows with a target:
  //   fp32, 16384 rows: 2048 words 56 with a warp per row, 60 with a CTA of 128
  //   threads; 2500 words 82 against 73; 5000 words 122 against 125 with the ring;
  //   8192 rows: 6500 words 90 against 74; 9000 words 103 with four CTAs per SM on
  //   the ring, 116 with two; 12000 words 125 against 131; 20000 words 196 with two.
  //   bf16: 16384 rows of 5000 words 80 with a CTA of 128 threads, 99 with a warp;
  //   8192 rows: 17000 words 125 against 141 with the ring; 24000 words 194 against 163.
  const bool few = M <= num_sms;
  if (bytes <= 8192) return run_warp<T>(a, part, num_sms, st);
  if (bytes <= (sizeof(T) == 4 ? 20480 : 40960))
    return few ? run_rows<T, 512>(a, part, num_sms, st) : run_rows<T, 128>(a, part, num_sms, st);
  if (few) return run_ring<T, 1>(a, part, num_sms, st);
  if constexpr (sizeof(T) == 4) {
    if (bytes <= 49152) return run_ring<T, 4>(a, part, num_sms, st);
  }
  // two CTAs per SM overlap one row's sums with the other's writes, unless much
  // of a row does not fit half the memory and is copied twice (fp32, 8192 rows:
  // 32768 words 324 against 364 with one CTA, 40000 words 403 against 420; 4096
  // rows of 60000 words 359 against 308)
  return bytes <= 184320 ? run_ring<T, 2>(a, part, num_sms, st) : run_ring<T, 1>(a, part, num_sms, st);
}

bool launch_policy_loss(const PolicyArgs& a, int act_bf16, double* part, int num_sms, cudaStream_t st) {
  int grid;
  {
    LaunchScope scope_(KK_POLICY_LOSS, st);
    grid = act_bf16 ? run<bf16>(a, part, num_sms, st) : run<float>(a, part, num_sms, st);
  }
  if (grid == 0) return false;
  LaunchScope scope_(KK_POLICY_LOSS, st);
  launch_pdl(k_policy_stats, dim3(1), dim3(96), 0, st, 1, part, grid, a.out_stats);
  return true;
}

}  // namespace nc
