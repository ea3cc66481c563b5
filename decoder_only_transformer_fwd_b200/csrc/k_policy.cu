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
// token).  A CTA takes a row at a time: one pass with a running maximum and
// sum, then a second pass that reads the row again (from L2, where the first
// pass left it) and writes the gradient.
#include <cfloat>

#include "nc_internal.cuh"
#include "ptx.cuh"

namespace nc {

namespace {

constexpr int kThreads = 512;
constexpr int kCtasPerSm = 2;
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

struct Scratch {
  float m[kThreads / 32];
  double s[kThreads / 32];
  float coef, gz, top;  // of the row: -gz / S, gz = w dL/dlp, max
};

struct Online {
  float m = -FLT_MAX, s = 0.f;
  template <int N>
  __device__ __forceinline__ void add(const float (&f)[N]) {
    float t = m;
#pragma unroll
    for (int i = 0; i < N; ++i) t = fmaxf(t, f[i]);
    float e = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) e += exp_diff(f[i], t);
    s = s * exp_diff(m, t) + e;
    m = t;
  }
};

__device__ __forceinline__ bool valid(int y, int V) { return (unsigned)y < (unsigned)V; }

template <typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) k_policy_loss(const PolicyArgs a, double* part) {
  __shared__ Scratch sh;
  __shared__ int s_count;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int M = a.B * a.T;
  // tokens (norm 0) or sequences (norm 1) with a target, counted by every CTA
  if (tid == 0) s_count = 0;
  __syncthreads();
  {
    int n = 0;
    if (a.norm == 0) {
      for (int i = tid; i < M; i += kThreads) n += valid(a.targets[i], a.V);
    } else {
      for (int b = warp; b < a.B; b += kThreads / 32) {
        bool any = false;
        for (int t0 = 0; t0 < a.T && !any; t0 += 32)
          any = __any_sync(0xffffffffu, t0 + lane < a.T && valid(a.targets[(size_t)b * a.T + t0 + lane], a.V));
        n += lane == 0 && any;
      }
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0 && n != 0) atomicAdd(&s_count, n);
  }
  __syncthreads();
  const int count = s_count;
  double sum_loss = 0.0, sum_kl = 0.0, sum_clip = 0.0;  // thread 0's
  for (int row = blockIdx.x; row < M; row += gridDim.x) {
    const T* z = static_cast<const T*>(a.logits) + (size_t)row * a.ldl;
    T* dz = a.dlogits != nullptr ? static_cast<T*>(a.dlogits) + (size_t)row * a.lddl : nullptr;
    const int V = a.V;
    int y = a.targets[row];
    if (y != -1 && !valid(y, V)) {  // recorded, and the token counts as padding
      if (tid == 0) atomicOr(a.status, kStatusData);
      y = -1;
    }
    float gz = 0.f, coef = 0.f, top = 0.f;
    if (y >= 0) {
      int tokens = count;
      if (a.norm == 1) {
        const int32_t* tg = a.targets + (size_t)(row / a.T) * a.T;
        tokens = 0;
        for (int t0 = 0; t0 < a.T; t0 += kThreads) tokens += __syncthreads_count(t0 + tid < a.T && valid(tg[t0 + tid], a.V));
      }
      const int head = head_of(z, V);
      const int nq = (V - head) / Quad<T>::N;
      Online o;
      if (tid < head) {
        const float f[1] = {Act<T>::ld(z + tid)};
        o.add(f);
      }
#pragma unroll 4
      for (int i = tid; i < nq; i += kThreads) {
        float f[Quad<T>::N];
        Quad<T>::ld(z + head + (size_t)i * Quad<T>::N, f);
        o.add(f);
      }
      const int tail = head + nq * Quad<T>::N;
      if (tail + tid < V) {
        const float f[1] = {Act<T>::ld(z + tail + tid)};
        o.add(f);
      }
      const float wm = warp_max(o.m);
      const double ws = warp_sum_d((double)(o.s * exp_diff(o.m, wm)));
      if (lane == 0) {
        sh.m[warp] = wm;
        sh.s[warp] = ws;
      }
      __syncthreads();
      if (warp == 0) {
        const bool mine = lane < kThreads / 32;
        const float m0 = mine ? sh.m[lane] : -FLT_MAX, m = warp_max(m0);
        const double S = warp_sum_d(mine ? sh.s[lane] * (double)exp_diff(m0, m) : 0.0);
        if (lane == 0) {
          const double lp = (double)Act<T>::ld(z + y) - (double)m - log(S);
          const double w = a.norm == 0 ? 1.0 / count : 1.0 / ((double)count * tokens);
          const double A = (double)a.advantages[a.adv_per_token ? row : row / a.T];
          const double x = a.old_logp != nullptr ? lp - (double)a.old_logp[row] : 0.0;
          const bool over = A > 0.0 && x > a.log_high, under = A < 0.0 && x < a.log_low;
          const double r = exp(x);
          double loss = -(over ? a.ratio_high : (under ? a.ratio_low : r)) * A;
          double slope = over || under ? 0.0 : -r * A;
          double kl = 0.0;
          if (a.ref_logp != nullptr) {
            const double d = (double)a.ref_logp[row] - lp, em = expm1(d);
            kl = em - d;
            loss += (double)a.kl_beta * kl;
            slope -= (double)a.kl_beta * em;
          }
          a.out_logp[row] = (float)lp;
          sum_loss += w * loss;
          sum_kl += w * kl;
          sum_clip += over || under ? w : 0.0;
          sh.gz = (float)(w * slope);
          sh.coef = (float)(-(w * slope) / S);
          sh.top = m;
        }
      }
      __syncthreads();
      gz = sh.gz, coef = sh.coef, top = sh.top;
    } else if (tid == 0) {
      a.out_logp[row] = 0.f;
    }
    if (dz != nullptr) {
      // the gradient's own 16-byte boundaries; the logits at the same element
      // offsets when both rows start alike, else one element at a time
      const int head = head_of(dz, V);
      const bool alike = ((reinterpret_cast<uintptr_t>(dz) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
      const int nq = (V - head) / Quad<T>::N, tail = head + nq * Quad<T>::N;
      auto one = [&](int v) { Act<T>::st(dz + v, y < 0 ? 0.f : coef * exp_diff(Act<T>::ld(z + v), top) + (v == y ? gz : 0.f)); };
      if (tid < head) one(tid);
      if (tail + tid < V) one(tail + tid);
#pragma unroll 4
      for (int i = tid; i < nq; i += kThreads) {
        const int v0 = head + i * Quad<T>::N;
        float f[Quad<T>::N];
        if (y >= 0) {
          if (alike) {
            Quad<T>::ld(z + v0, f);
          } else {
#pragma unroll
            for (int e = 0; e < Quad<T>::N; ++e) f[e] = Act<T>::ld(z + v0 + e);
          }
#pragma unroll
          for (int e = 0; e < Quad<T>::N; ++e) f[e] = coef * exp_diff(f[e], top) + (v0 + e == y ? gz : 0.f);
        } else {
#pragma unroll
          for (int e = 0; e < Quad<T>::N; ++e) f[e] = 0.f;
        }
        Quad<T>::st(dz + v0, f);
      }
    }
    __syncthreads();  // the next row reuses the scratch
  }
  if (tid == 0) {
    part[3 * blockIdx.x] = sum_loss;
    part[3 * blockIdx.x + 1] = sum_kl;
    part[3 * blockIdx.x + 2] = sum_clip;
  }
}

// the CTAs' sums in a fixed order, one warp per statistic
__global__ void __launch_bounds__(96) k_policy_stats(const double* part, int n, float* out) {
  pdl_launch_dependents();
  pdl_wait();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double s = 0.0;
  for (int i = lane; i < n; i += 32) s += part[3 * i + w];
  s = warp_sum_d(s);
  if (lane == 0) out[w] = (float)s;
}

}  // namespace

void launch_policy_loss(const PolicyArgs& a, int act_bf16, double* part, int num_sms, cudaStream_t st) {
  const int M = a.B * a.T;
  int grid = num_sms * kCtasPerSm < kPolicyMaxCtas ? num_sms * kCtasPerSm : kPolicyMaxCtas;
  if (grid > M) grid = M;
  {
    LaunchScope scope_(KK_POLICY_LOSS, st);
    launch_pdl(act_bf16 ? k_policy_loss<bf16> : k_policy_loss<float>, dim3(grid), dim3(kThreads), 0, st, 1, a, part);
  }
  LaunchScope scope_(KK_POLICY_LOSS, st);
  launch_pdl(k_policy_stats, dim3(1), dim3(96), 0, st, 1, part, grid, a.out_stats);
}

}  // namespace nc
