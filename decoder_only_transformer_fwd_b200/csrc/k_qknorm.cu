// QK-norm with RoPE at given positions, written to a dense output or into cache
// rows, and its gradient.
//
// "The Mathematics of Karpathy's nanochat", §QK-Norm with Sharpening, §Rotary
// Position Embeddings: with R(t) the half-split rotation (u1 cos + u2 sin,
// -u1 sin + u2 cos) by t theta_i, theta_i = base^(-2i/D) (`reverse`: by the
// negated angles, as many other half-split models turn),
//   y = alpha R x / rho,   rho = sqrt(mean(x^2) + eps)
// (the rotation keeps the norm, so rho is taken from x).  Its gradient, with
// b = R^T dy,
//   dx = (alpha / rho) (b - x (x . b) / (D rho^2)).
//
// Both passes only move data: (H + 2 H_kv) D elements per token in and out
// (forward), 2 (H + H_kv) D in and (H + H_kv) D out (backward).
#include "nc_internal.cuh"

namespace nc {

namespace {

constexpr int kD = 128, kHalf = 64;
constexpr int kThreads = 256, kMaxTok = 8;

struct RopeFreq {
  // theta_i / 2 pi as a fraction of 2^64: position * turns mod 2^64 is the
  // phase in turns, exact in integers for every 31-bit position
  unsigned long long turns[kHalf];
};

struct Vec {  // one lane's part of a head vector: dims [8 j, 8 j + 8) and [64 + 8 j, 64 + 8 j + 8)
  float a[8], b[8];
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<uint32_t*>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T> struct Raw;  // the untouched 16-byte words of a Vec
template <> struct Raw<bf16> {
  uint4 w[2];
  __device__ __forceinline__ void load(const bf16* p, int j) {
    w[0] = *reinterpret_cast<const uint4*>(p + 8 * j);
    w[1] = *reinterpret_cast<const uint4*>(p + kHalf + 8 * j);
  }
  __device__ __forceinline__ void store(bf16* p, int j) const {
    *reinterpret_cast<uint4*>(p + 8 * j) = w[0];
    *reinterpret_cast<uint4*>(p + kHalf + 8 * j) = w[1];
  }
  __device__ __forceinline__ Vec get() const {
    Vec v;
    unpack8(w[0], v.a);
    unpack8(w[1], v.b);
    return v;
  }
  __device__ __forceinline__ void set(const Vec& v) {
    w[0] = pack8(v.a);
    w[1] = pack8(v.b);
  }
};
template <> struct Raw<float> {
  float4 w[4];
  __device__ __forceinline__ void load(const float* p, int j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(p + (i >> 1) * kHalf + 8 * j + 4 * (i & 1));
  }
  __device__ __forceinline__ void store(float* p, int j) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(p + (i >> 1) * kHalf + 8 * j + 4 * (i & 1)) = w[i];
  }
  __device__ __forceinline__ Vec get() const {
    Vec v;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v.a[4 * i] = w[i].x, v.a[4 * i + 1] = w[i].y, v.a[4 * i + 2] = w[i].z, v.a[4 * i + 3] = w[i].w;
      v.b[4 * i] = w[2 + i].x, v.b[4 * i + 1] = w[2 + i].y, v.b[4 * i + 2] = w[2 + i].z, v.b[4 * i + 3] = w[2 + i].w;
    }
    return v;
  }
  __device__ __forceinline__ void set(const Vec& v) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i] = make_float4(v.a[4 * i], v.a[4 * i + 1], v.a[4 * i + 2], v.a[4 * i + 3]);
      w[2 + i] = make_float4(v.b[4 * i], v.b[4 * i + 1], v.b[4 * i + 2], v.b[4 * i + 3]);
    }
  }
};

// sum over the eight lanes that share a head vector
__device__ __forceinline__ float sum8(float v, unsigned mask) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
  return v;
}

// cos and sin of a position's 64 angles into shared memory, one angle per
// thread: the upper 32 bits of position * turns are the phase in turns to
// 2^-32, a signed fraction in [-1/2, 1/2)
__device__ __forceinline__ void fill_angles(const RopeFreq& f, const int32_t* positions, int reverse, int n0, int ntok,
                                            float* cs, int* status) {
  for (int i = threadIdx.x; i < ntok * kHalf; i += kThreads) {
    int pos = positions[n0 + i / kHalf];
    if (pos < 0) {
      if (i % kHalf == 0) atomicOr(status, kStatusData);
      pos = 0;
    }
    const unsigned long long ph = (unsigned long long)(unsigned)pos * f.turns[i % kHalf];
    const float turn = (float)(int)(unsigned)(ph >> 32) * 2.3283064365386963e-10f;  // 2^-32
    float s, c;
    sincospif(reverse ? -2.0f * turn : 2.0f * turn, &s, &c);
    cs[(i / kHalf) * 2 * kHalf + i % kHalf] = c;
    cs[(i / kHalf) * 2 * kHalf + kHalf + i % kHalf] = s;
  }
}

// A lane's cos and sin, read again for every vector: kept in registers they
// would cost a CTA per SM, and with it the loads in flight that HBM needs.
__device__ __forceinline__ void load_angles(uint32_t p, float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(c[i]), "=f"(c[i + 1]), "=f"(c[i + 2]), "=f"(c[i + 3]) : "r"(p + 4 * i));
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(s[i]), "=f"(s[i + 1]), "=f"(s[i + 2]), "=f"(s[i + 3]) : "r"(p + 4 * (kHalf + i)));
  }
}

template <typename T>
struct FwdArgs {
  const T *q, *k, *v;
  T *qo, *ko, *vo;
  long long ldq, ldk, ldv, ldqo, ldko, ldvo;  // row strides, elements
  const int32_t *positions, *slots;
  int N, H, Hkv, reverse, tok;  // tok: tokens per CTA
  long long out_rows;
  float alpha, eps;
  int* status;
  RopeFreq f;
};

// A CTA takes `tok` tokens; its 32 eight-lane groups share them out evenly,
// and a group walks every (32 / tok)-th head vector of its token, the next two
// vectors' loads under the current one's arithmetic (and the first two's under
// the angles').  With one vector's loads ahead HBM waits: 8192 tokens, 12 + 12
// heads, bf16, 29.1 us against 26.7.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_qk_norm_rope(const __grid_constant__ FwdArgs<T> a) {
  __shared__ __align__(16) float cs[kMaxTok * 2 * kHalf];
  pdl_launch_dependents();
  pdl_wait();
  const int n0 = blockIdx.x * a.tok;
  const int ntok = min(a.tok, a.N - n0);
  const int group = threadIdx.x >> 3, j = threadIdx.x & 7;
  const int per = 32 / a.tok;  // groups per token
  const int tl = group / per;
  const bool live = tl < ntok;
  const int n = n0 + tl;
  const int kept = (a.v != nullptr ? 2 : 1) * a.Hkv;
  auto source = [&](int h) -> const T* {
    const int hk = h - a.H, hv = hk - a.Hkv;
    return hk < 0 ? a.q + n * a.ldq + h * kD : (hv < 0 ? a.k + n * a.ldk + hk * kD : a.v + n * a.ldv + hv * kD);
  };
  int h = group % per;
  Raw<T> ahead[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (live && h + i * per < a.H + kept) ahead[i].load(source(h + i * per), j);
  long long slot = live ? (a.slots != nullptr ? (long long)a.slots[n] : (long long)n) : 0;
  fill_angles(a.f, a.positions, a.reverse, n0, ntok, cs, a.status);
  __syncthreads();
  if (!live) return;
  const unsigned mask = 0xffu << ((threadIdx.x & 31) & ~7);
  if (slot < -1 || slot >= a.out_rows) {  // -1: a token that is not kept
    if (h == 0 && j == 0) atomicOr(a.status, kStatusData);
    slot = -1;
  }
  const uint32_t my_cs = static_cast<uint32_t>(__cvta_generic_to_shared(cs + tl * 2 * kHalf + 8 * j));
  const int heads = a.H + (slot >= 0 ? kept : 0);
  auto take = [&](int h, Raw<T>& next) {
    const int hk = h - a.H, hv = hk - a.Hkv;
    Raw<T> raw = next;
    if (h + 2 * per < heads) next.load(source(h + 2 * per), j);
    T* dst = hk < 0 ? a.qo + n * a.ldqo + h * kD
                    : (hv < 0 ? a.ko + slot * a.ldko + hk * kD : a.vo + slot * a.ldvo + hv * kD);
    if (hv < 0) {
      Vec x = raw.get();
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += x.a[i] * x.a[i] + x.b[i] * x.b[i];
      ss = sum8(ss, mask);
      const float r = a.alpha * rsqrtf(ss * (1.0f / kD) + a.eps);
      float c[8], s[8];
      load_angles(my_cs, c, s);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = x.a[i], w = x.b[i];
        x.a[i] = r * (u * c[i] + w * s[i]);
        x.b[i] = r * (w * c[i] - u * s[i]);
      }
      raw.set(x);
    }
    raw.store(dst, j);
  };
  while (h < heads) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (h >= heads) break;
      take(h, ahead[i]);
      h += per;
    }
  }
}

template <typename T>
struct BwdArgs {
  const T *q, *k, *gq, *gk;
  T *dq, *dk;
  long long ldq, ldk, ldgq, ldgk, lddq, lddk;
  const int32_t* positions;
  int N, H, Hkv, reverse, tok;
  float alpha, eps;
  int* status;
  RopeFreq f;
};

// MINB: CTAs per SM that the registers are kept to.
template <typename T, int MINB>
__global__ void __launch_bounds__(kThreads, MINB) k_qk_norm_rope_bwd(const __grid_constant__ BwdArgs<T> a) {
  __shared__ __align__(16) float cs[kMaxTok * 2 * kHalf];
  pdl_launch_dependents();
  pdl_wait();
  const int n0 = blockIdx.x * a.tok;
  const int ntok = min(a.tok, a.N - n0);
  const int group = threadIdx.x >> 3, j = threadIdx.x & 7;
  const int per = 32 / a.tok;
  const int tl = group / per;
  const bool live = tl < ntok;
  const int n = n0 + tl, heads = a.H + a.Hkv;
  int h = group % per;
  Raw<T> nx, ng;
  auto load = [&](int h) {
    const int hk = h - a.H;
    nx.load(hk < 0 ? a.q + n * a.ldq + h * kD : a.k + n * a.ldk + hk * kD, j);
    ng.load(hk < 0 ? a.gq + n * a.ldgq + h * kD : a.gk + n * a.ldgk + hk * kD, j);
  };
  if (live && h < heads) load(h);
  fill_angles(a.f, a.positions, a.reverse, n0, ntok, cs, a.status);
  __syncthreads();
  if (!live) return;
  const unsigned mask = 0xffu << ((threadIdx.x & 31) & ~7);
  const uint32_t my_cs = static_cast<uint32_t>(__cvta_generic_to_shared(cs + tl * 2 * kHalf + 8 * j));
  for (; h < heads; h += per) {
    const int hk = h - a.H;
    const Vec x = nx.get();
    Vec g = ng.get();
    if (h + per < heads) load(h + per);
    float c[8], s[8];
    load_angles(my_cs, c, s);
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = g.a[i], w = g.b[i];
      g.a[i] = u * c[i] - w * s[i];
      g.b[i] = w * c[i] + u * s[i];
      ss += x.a[i] * x.a[i] + x.b[i] * x.b[i];
      dot += x.a[i] * g.a[i] + x.b[i] * g.b[i];
    }
    ss = sum8(ss, mask);
    dot = sum8(dot, mask);
    const float inv = rsqrtf(ss * (1.0f / kD) + a.eps);
    const float r = a.alpha * inv, t = dot * (1.0f / kD) * inv * inv;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g.a[i] = r * (g.a[i] - x.a[i] * t);
      g.b[i] = r * (g.b[i] - x.b[i] * t);
    }
    Raw<T> out;
    out.set(g);
    out.store(hk < 0 ? a.dq + n * a.lddq + h * kD : a.dk + n * a.lddk + hk * kD, j);
  }
}

// base^(-2i/D) / (2 pi) as fractions of 2^64, by repeated multiplication in
// long double (64 factors: relative error below 2^-57).  A thread keeps those of
// the last base (a model has one); working them out takes 1 us of the host's time.
void rope_freq(float base, RopeFreq* f) {
  static thread_local float last = 0.f;
  static thread_local RopeFreq kept;
  if (base != last) {
    const long double ratio = expl(-logl((long double)base) / kHalf);
    long double t = 0.15915494309189533576888376337251436203L;  // 1 / (2 pi)
    for (int i = 0; i < kHalf; ++i, t *= ratio) kept.turns[i] = (unsigned long long)(t * 18446744073709551616.0L);
    last = base;
  }
  *f = kept;
}

// Tokens per CTA: as many as leave a CTA for each SM and a third more, and a
// group at most eight vectors.  Measured, bf16, 12 + 12 heads: forward of 300
// tokens 3.4 us with 1 token (4.2 with 4), of 1000 tokens 6.6 us with 4 (8.2
// with 1, 9.5 with 8); backward of 3000 tokens 10.0 us with 8 (11.0 with 4).
int tokens_per_cta(int N, int heads, int num_sms) {
  int tok = kMaxTok;
  while (tok > 1 && (heads * tok > 32 * 8 || (long long)3 * ((N + tok - 1) / tok) < (long long)4 * num_sms)) tok /= 2;
  return tok;
}

}  // namespace

template <typename T>
static void run_fwd(const QkNormArgs& p, int num_sms, cudaStream_t st) {
  FwdArgs<T> a;
  a.q = static_cast<const T*>(p.q), a.k = static_cast<const T*>(p.k), a.v = static_cast<const T*>(p.v);
  a.qo = static_cast<T*>(p.q_out), a.ko = static_cast<T*>(p.k_out), a.vo = static_cast<T*>(p.v_out);
  a.ldq = p.ldq, a.ldk = p.ldk, a.ldv = p.ldv, a.ldqo = p.ldqo, a.ldko = p.ldko, a.ldvo = p.ldvo;
  a.positions = p.positions, a.slots = p.slots;
  a.N = p.N, a.H = p.H, a.Hkv = p.Hkv, a.reverse = p.reverse, a.tok = tokens_per_cta(p.N, p.H + (p.v != nullptr ? 2 : 1) * p.Hkv, num_sms);
  a.out_rows = p.out_rows, a.alpha = p.alpha, a.eps = p.eps, a.status = p.status;
  rope_freq(p.rope_base, &a.f);
  LaunchScope scope_(KK_QK_NORM_ROPE, st);
  launch_pdl(k_qk_norm_rope<T>, dim3((p.N + a.tok - 1) / a.tok), dim3(kThreads), 0, st, 1, a);
}

void launch_qk_norm_rope(const QkNormArgs& p, int act_bf16, int num_sms, cudaStream_t st) {
  if (act_bf16)
    run_fwd<bf16>(p, num_sms, st);
  else
    run_fwd<float>(p, num_sms, st);
}

template <typename T>
static void run_bwd(const QkNormArgs& p, int num_sms, cudaStream_t st) {
  BwdArgs<T> a;
  a.q = static_cast<const T*>(p.q), a.k = static_cast<const T*>(p.k);
  a.gq = static_cast<const T*>(p.dq_hat), a.gk = static_cast<const T*>(p.dk_hat);
  a.dq = static_cast<T*>(p.q_out), a.dk = static_cast<T*>(p.k_out);
  a.ldq = p.ldq, a.ldk = p.ldk, a.ldgq = p.ldgq, a.ldgk = p.ldgk, a.lddq = p.ldqo, a.lddk = p.ldko;
  a.positions = p.positions;
  a.N = p.N, a.H = p.H, a.Hkv = p.Hkv, a.reverse = p.reverse, a.tok = tokens_per_cta(p.N, p.H + p.Hkv, num_sms);
  a.alpha = p.alpha, a.eps = p.eps, a.status = p.status;
  rope_freq(p.rope_base, &a.f);
  LaunchScope scope_(KK_QK_NORM_ROPE, st);
  const int grid = (p.N + a.tok - 1) / a.tok;
  // bf16 moves 32 bytes per thread and load, so a long batch wants the fourth CTA
  // on an SM (8192 tokens, 12 + 12 heads: 25.5 us against 28.2); with fewer CTAs
  // than that the freer schedule is faster (3000 tokens: 9.8 us against 12.2)
  auto kernel = k_qk_norm_rope_bwd<T, 3>;
  if constexpr (sizeof(T) == 2) {
    if (grid >= 4 * num_sms) kernel = k_qk_norm_rope_bwd<T, 4>;
  }
  launch_pdl(kernel, dim3(grid), dim3(kThreads), 0, st, 1, a);
}

void launch_qk_norm_rope_bwd(const QkNormArgs& p, int act_bf16, int num_sms, cudaStream_t st) {
  if (act_bf16)
    run_bwd<bf16>(p, num_sms, st);
  else
    run_bwd<float>(p, num_sms, st);
}

}  // namespace nc
