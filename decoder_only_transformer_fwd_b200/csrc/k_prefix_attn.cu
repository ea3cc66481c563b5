// Attention of a batch whose rows share a long prefix (tcgen05, head dim 128,
// bf16 q/k/v, fp32 scores, statistics and accumulation).
//
// Row b of group g = b / (B / G) holds the keys of its group's prefix
// (positions 0 .. P_g - 1) followed by S_b keys of its own; query i of its Tq
// has position P_g + S_b - Tq + i and sees key j iff j <= position and
// position - j < window ("The Mathematics of Karpathy's nanochat", §Scaled
// Dot-Product Attention with Sliding Window):
//   o = sum_j softmax_j(scale q . k_j) v_j.
//
// The prefix keys of a group are read once for all its rows: the queries of
// all rows (and of all query heads of one key head) form the 128-row tiles of
// one matrix product, so a long prefix costs its bytes once instead of once
// per row.  What bounds it: reading the caches from HBM, as long as a key
// head has fewer than about 250 query rows per group.
//
// Work is cut into units, one CTA each:
//   prefix unit: (group, key head, range of 64-key tiles, 128-row query tile),
//   suffix unit: (row, key head, range of 64-key tiles, query tile).
// Every unit leaves its rows' normalised output (fp32) and log-sum-exp in the
// workspace; k_prefix_combine joins a row's parts with weights
// exp(lse_part - lse).  A row for which a unit has no visible key gets
// lse = -inf there.  With one part in all, the unit writes the output itself.
//
// A CTA: warps 0..3 softmax (one row per thread = TMEM lane; warps without a
// row sit out), warp 4 TMA, warp 5 MMA.  64-key K and V tiles stream through
// a ring of 16 KB slots in the order K0 K1 V0 K2 V1 ...; S is double-buffered
// in TMEM, so Q K_{t+1}^T runs during tile t's exponentials, and P_t (bf16)
// overwrites the first half of S_t.  Two CTAs share an SM: one's set-up and
// drain overlap the other's stream.  Every wait is bounded.
#include "nc_internal.cuh"
#include "ptx.cuh"

namespace nc {

bool make_tmap_4d(CUtensorMap* map, const void* ptr, const uint64_t (&dims)[4], const uint64_t (&strides_bytes)[3],
                  const uint32_t (&box)[4]);

namespace {

using ptx::ex2;

constexpr int kD = 128, kRows = 128, kKeys = 64;
constexpr int Q_BOX = kRows * 128;         // 16 KB: 128 rows x 64 columns of Q
constexpr int KV_BOX = kKeys * 128;        // 8 KB: 64 keys x 64 columns
constexpr int SLOT_BYTES = 2 * KV_BOX;     // 16 KB
constexpr int SLOTS = 4;
constexpr int OFF_SLOT = 2 * Q_BOX;
constexpr int OFF_BAR = OFF_SLOT + SLOTS * SLOT_BYTES;
constexpr int SMEM_BYTES = OFF_BAR + 256 + 1024;
constexpr int kThreads = 192, kWarpTma = 4, kWarpMma = 5;
constexpr uint32_t TMEM_COLS = 256;        // S0 64 | S1 64 | O 128
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kLn2 = 0.6931471805599453f;

struct Unit {
  int suffix;      // 0: prefix keys, 1: a row's own keys
  int seq, hk;     // group or row, key head
  int split;
  int tok0, ntok;  // query tokens of the tile (token = row of the batch * Tq + i)
};

__device__ __forceinline__ Unit decode_unit(const PrefixAttnArgs& a, int u) {
  Unit w;
  w.suffix = u >= a.units_p;
  if (w.suffix) u -= a.units_p;
  const int tiles = w.suffix ? a.tiles_s : a.tiles_p, splits = w.suffix ? a.splits_s : a.splits_p;
  const int tt = u % tiles;
  u /= tiles;
  w.split = u % splits;
  u /= splits;
  w.hk = u % a.Hkv;
  w.seq = u / a.Hkv;
  const int tokens = (w.suffix ? 1 : a.rows_per_group) * a.Tq, box = w.suffix ? a.box_s : a.box_p;
  w.tok0 = w.seq * tokens + tt * box;
  w.ntok = min(box, tokens - tt * box);
  return w;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

__global__ void __launch_bounds__(kThreads, 2)
    k_prefix_attn(const __grid_constant__ CUtensorMap tmQp, const __grid_constant__ CUtensorMap tmQs,
                  const __grid_constant__ CUtensorMap tmKp, const __grid_constant__ CUtensorMap tmVp,
                  const __grid_constant__ CUtensorMap tmKs, const __grid_constant__ CUtensorMap tmVs,
                  const PrefixAttnArgs a) {
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  enum { B_Q = 0, B_F = 1, B_E = B_F + SLOTS, B_S = B_E + SLOTS, B_P = B_S + 2, B_O = B_P + 2, B_FIN, B_DONE, NB };
  static_assert(NB * 8 + 8 + 32 <= 256, "barrier area");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NB);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_range = reinterpret_cast<int*>(tmem_slot + 2);  // lo of warps 0..3, hi of warps 0..3
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8u * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Unit w = decode_unit(a, blockIdx.x);
  const int R = a.H / a.Hkv;
  const int nrows = w.ntok * R, nwarps = (nrows + 31) / 32;

  if (threadIdx.x == 0) {
    ptx::mbar_init(bar(B_Q), 1);
    for (int s = 0; s < SLOTS; ++s) {
      ptx::mbar_init(bar(B_F + s), 1);
      ptx::mbar_init(bar(B_E + s), 1);
    }
    for (int g = 0; g < 2; ++g) {
      ptx::mbar_init(bar(B_S + g), 1);
      ptx::mbar_init(bar(B_P + g), nwarps);
    }
    ptx::mbar_init(bar(B_O), 1);
    ptx::mbar_init(bar(B_FIN), 1);
    ptx::mbar_init(bar(B_DONE), 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  pdl_wait();  // lengths, q and the caches may come from the previous kernel

  // Visible keys of each row among the unit's keys: [lo, hi), counted from the
  // first key of the prefix or of the row's own keys.
  int lo = 0, hi = 0;
  const int token = w.tok0 + (int)threadIdx.x / R;
  if (warp < 4) {
    if ((int)threadIdx.x < nrows) {
      const int b = token / a.Tq, g = b / a.rows_per_group;
      int P = a.prefix_lens != nullptr ? a.prefix_lens[g] : 0, S = a.suffix_lens != nullptr ? a.suffix_lens[b] : 0;
      if (P < 0 || P > a.P_max || S < 0 || S > a.S_max) {
        atomicOr(a.status, kStatusData);
        P = min(max(P, 0), a.P_max);
        S = min(max(S, 0), a.S_max);
      }
      const int pos = P + S - a.Tq + token % a.Tq;
      const int base = w.suffix ? P : 0;
      lo = max(0, pos - a.window + 1 - base);
      hi = min(w.suffix ? S : P, pos + 1 - base);
      if (lo >= hi) lo = hi = 0;
    }
    const int l = __reduce_min_sync(0xffffffffu, lo < hi ? lo : 0x7fffffff);
    const int h = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      s_range[warp] = l;
      s_range[4 + warp] = h;
    }
  }
  __syncthreads();
  const int ulo = min(min(s_range[0], s_range[1]), min(s_range[2], s_range[3]));
  const int uhi = max(max(s_range[4], s_range[5]), max(s_range[6], s_range[7]));
  int nt = 0, t0 = 0;
  if (ulo < uhi) {
    const int first = ulo / kKeys, tiles = (uhi + kKeys - 1) / kKeys - first;
    const int splits = w.suffix ? a.splits_s : a.splits_p;
    const int chunk = max(a.min_tiles, (tiles + splits - 1) / splits);
    t0 = first + w.split * chunk;
    nt = min(chunk, tiles - w.split * chunk);
  }
  const int part = w.suffix ? a.splits_p + w.split : w.split;
  const bool direct = a.splits_p + a.splits_s == 1;
  const long long total_rows = (long long)a.B * a.Tq * a.H;
  // row of the outputs: token-major, then head
  const long long orow = (long long)token * a.H + w.hk * R + (int)threadIdx.x % R;
  if (nt <= 0) {
    if ((int)threadIdx.x < nrows) {
      if (direct) {
        uint4* d = reinterpret_cast<uint4*>(a.out + orow * kD);
        for (int i = 0; i < kD / 8; ++i) d[i] = make_uint4(0u, 0u, 0u, 0u);
        if (a.out_lse != nullptr) a.out_lse[orow] = -INFINITY;
      } else {
        a.part_lse[(long long)part * total_rows + orow] = -INFINITY;
      }
    }
    return;
  }
  if (warp == kWarpMma) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), TMEM_COLS);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto sSlot = [&](int s) { return ptx::smem_u32(smem + OFF_SLOT + s * SLOT_BYTES); };
  const uint32_t sQ = ptx::smem_u32(smem);
  // place in the ring's sequence of K_t and V_t
  auto seq_k = [](int t) { return t == 0 ? 0 : 2 * t - 1; };
  auto seq_v = [&](int t) { return t + 1 < nt ? 2 * t + 2 : 2 * nt - 1; };

  if (warp == kWarpTma) {
    if (ptx::elect_one()) {
      const void* tq = w.suffix ? (const void*)&tmQs : (const void*)&tmQp;
      const void* tk = w.suffix ? (const void*)&tmKs : (const void*)&tmKp;
      const void* tv = w.suffix ? (const void*)&tmVs : (const void*)&tmVp;
      const int box_tok = w.suffix ? a.box_s : a.box_p;
      ptx::mbar_arrive_expect_tx(bar(B_Q), (uint32_t)(2 * box_tok * R * 128));
      ptx::tma_load_4d(sQ, tq, bar(B_Q), 0, w.hk * R, w.tok0, 0);
      ptx::tma_load_4d(sQ + Q_BOX, tq, bar(B_Q), 64, w.hk * R, w.tok0, 0);
      bool ok = true;
      int issued = 0;
      for (int sc = 0; sc < 2 * nt; ++sc) {
        // K0 K1 V0 K2 V1 ... K_{nt-1} V_{nt-2} V_{nt-1}
        const bool is_k = sc == 0 || (sc % 2 == 1 && sc < 2 * nt - 1);
        const int t = sc == 0 ? 0 : (is_k ? (sc + 1) / 2 : (sc == 2 * nt - 1 ? nt - 1 : sc / 2 - 1));
        const int s = sc % SLOTS;
        const uint32_t ph = (uint32_t)(sc / SLOTS) & 1u;
        if (*abort_flag || !ptx::mbar_wait(bar(B_E + s), ph ^ 1, a.status)) {
          ok = false;
          break;
        }
        ptx::mbar_arrive_expect_tx(bar(B_F + s), SLOT_BYTES);
        const int key = (t0 + t) * kKeys;
        ptx::tma_load_4d(sSlot(s), is_k ? tk : tv, bar(B_F + s), 0, w.hk, key, w.seq);
        ptx::tma_load_4d(sSlot(s) + KV_BOX, is_k ? tk : tv, bar(B_F + s), 64, w.hk, key, w.seq);
        ++issued;
      }
      if (!ok) *abort_flag = 1;
      // every copy issued here has landed before the CTA may exit
      ptx::mbar_wait(bar(B_Q), 0, a.status);
      for (int sc = max(0, issued - SLOTS); sc < issued; ++sc)
        ptx::mbar_wait(bar(B_F + sc % SLOTS), (uint32_t)(sc / SLOTS) & 1u, a.status);
    }
  } else if (warp == kWarpMma) {
    if (ptx::elect_one()) {
      constexpr uint32_t idesc_qk = ptx::idesc_bf16(kRows, kKeys, 0, 0);
      constexpr uint32_t idesc_pv = ptx::idesc_bf16(kRows, kD, 0, 1);  // V is MN-major
      const uint64_t dq = ptx::desc_kmajor_sw128(sQ);
      const uint64_t dk0 = ptx::desc_kmajor_sw128(sSlot(0)), dv0 = ptx::desc_mnmajor_sw128(sSlot(0), KV_BOX);
      auto full = [&](int sc) -> bool {
        return !*abort_flag && ptx::mbar_wait(bar(B_F + sc % SLOTS), (uint32_t)(sc / SLOTS) & 1u, a.status);
      };
      auto qk = [&](int t) -> bool {
        const int sc = seq_k(t);
        if (!full(sc)) return false;
        ptx::tc_fence_after();
        const uint64_t dk = dk0 + (uint64_t)((sc % SLOTS) * (SLOT_BYTES >> 4));
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk)
          ptx::mma_bf16_ss(tmem + (uint32_t)((t & 1) * kKeys), dq + (uint64_t)((kk >> 2) * (Q_BOX >> 4) + (kk & 3) * 2),
                           dk + (uint64_t)((kk >> 2) * (KV_BOX >> 4) + (kk & 3) * 2), idesc_qk, kk > 0 ? 1u : 0u);
        ptx::mma_commit(bar(B_S + (t & 1)));
        ptx::mma_commit(bar(B_E + sc % SLOTS));
        return true;
      };
      bool ok = ptx::mbar_wait(bar(B_Q), 0, a.status) && qk(0);
      for (int t = 0; ok && t < nt; ++t) {
        // S_{t+1} goes where P_{t-1} was, whose product was issued before
        if (t + 1 < nt && !qk(t + 1)) {
          ok = false;
          break;
        }
        const int sc = seq_v(t);
        if (!full(sc) || *abort_flag || !ptx::mbar_wait(bar(B_P + (t & 1)), (uint32_t)(t >> 1) & 1u, a.status)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint64_t dv = dv0 + (uint64_t)((sc % SLOTS) * (SLOT_BYTES >> 4));
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          ptx::mma_bf16_ts(tmem + 128u, tmem + (uint32_t)((t & 1) * kKeys + kk * 8), dv + (uint64_t)(kk * (2048 >> 4)),
                           idesc_pv, (t > 0 || kk > 0) ? 1u : 0u);
        ptx::mma_commit(bar(B_E + sc % SLOTS));
        // the softmax waits for B_O only where S_t shows that phase t - 2 is over;
        // the last product has a barrier of its own
        ptx::mma_commit(bar(t + 1 < nt ? B_O : B_FIN));
      }
      if (!ok) *abort_flag = 1;
      ptx::mma_commit(bar(B_DONE));
      ptx::mbar_wait(bar(B_DONE), 0, a.status);
    }
  } else if (warp < nwarps) {
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const uint32_t tO = tmem + 128u + lane_off;
    const float c = a.scale_log2;
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int t = 0; t < nt; ++t) {
      const uint32_t tS = tmem + (uint32_t)((t & 1) * kKeys) + lane_off;
      const int k0 = (t0 + t) * kKeys;
      const int clo = lo - k0, chi = hi - k0;  // visible columns [clo, chi)
      if (*abort_flag || !ptx::mbar_wait(bar(B_S + (t & 1)), (uint32_t)(t >> 1) & 1u, a.status)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      float x[kKeys];
      {
        uint32_t u0[32], u1[32];
        ptx::tmem_ld32(tS, u0);
        ptx::tmem_ld32(tS + 32, u1);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          x[i] = __uint_as_float(u0[i]);
          x[32 + i] = __uint_as_float(u1[i]);
        }
      }
      if (!__all_sync(0xffffffffu, clo <= 0 && chi >= kKeys)) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i) x[i] = (i >= clo && i < chi) ? x[i] : -INFINITY;
      }
      float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int i = 4; i < kKeys; i += 4)
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], x[i + k]);
      const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      // the running max moves only when it grows by more than 2^8
      const bool rescale = (tmax - m_run) * c > kRescaleThreshold;
      const float m_new = rescale ? tmax : m_run;
      const float mc = m_new == -INFINITY ? 0.f : m_new * c;
      uint32_t pk[32];
      float2 sm[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float2 e = __ffma2_rn(make_float2(x[2 * i], x[2 * i + 1]), c2, mc2);
        const float2 p = make_float2(ex2(e.x), ex2(e.y));
        sm[i & 1] = __fadd2_rn(sm[i & 1], p);
        pk[i] = pack_bf16(p.x, p.y);
      }
      ptx::tmem_st32(tS, pk);
      const float alpha = rescale ? ex2(m_run * c - mc) : 1.f;  // 0 when m_run == -inf
      if (rescale) {
        l_run *= alpha;
        m_run = m_new;
      }
      const float2 s2 = __fadd2_rn(sm[0], sm[1]);
      l_run += s2.x + s2.y;
      // P V of tile t - 1 must have landed before O is rescaled
      if (t > 0 && __any_sync(0xffffffffu, rescale)) {
        if (!ptx::mbar_wait(bar(B_O), (uint32_t)(t - 1) & 1u, a.status)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
#pragma unroll 1
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t u[32];
          ptx::tmem_ld32(tO + (uint32_t)(cc * 32), u);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * alpha);
          ptx::tmem_st32(tO + (uint32_t)(cc * 32), u);
        }
      }
      // V rows that no row of the unit sees (behind the end, before the
      // window) may hold anything: they become zeros, since 0 x NaN is not 0
      if (k0 < ulo || k0 + kKeys > uhi) {
        const int sc = seq_v(t), s = sc % SLOTS;
        if (!ptx::mbar_wait(bar(B_F + s), (uint32_t)(sc / SLOTS) & 1u, a.status)) {
          ok = false;
          break;
        }
        for (int i = threadIdx.x; i < kKeys * 16; i += 32 * nwarps) {
          const int key = k0 + i / 16;
          if (key < ulo || key >= uhi)
            *reinterpret_cast<uint4*>(smem + OFF_SLOT + s * SLOT_BYTES + ((i & 8) ? KV_BOX : 0) + (i / 16) * 128 + (i & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        ptx::fence_proxy_async_smem();
      }
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(B_P + (t & 1)));
    }
    if (ok && ptx::mbar_wait(bar(B_FIN), 0, a.status)) {
      ptx::tc_fence_after();
      const bool live = (int)threadIdx.x < nrows;
      const float inv = l_run > 0.f ? 1.0f / l_run : 0.f;
      const float lse = l_run > 0.f ? (m_run * c + log2f(l_run)) * kLn2 : -INFINITY;
      const long long prow = (long long)part * total_rows + orow;
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        uint32_t u[32];
        ptx::tmem_ld32(tO + (uint32_t)(cc * 32), u);
        ptx::tmem_ld_wait();
        if (!live) continue;
        // a row whose keys are all masked in this unit: its accumulator holds
        // nothing of its own
        if (inv == 0.f) {
#pragma unroll
          for (int i = 0; i < 32; ++i) u[i] = 0u;
        }
        if (direct) {
          uint4* d = reinterpret_cast<uint4*>(a.out + orow * kD) + 4 * cc;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = pack_bf16(__uint_as_float(u[8 * q + 2 * e]) * inv, __uint_as_float(u[8 * q + 2 * e + 1]) * inv);
            d[q] = make_uint4(v[0], v[1], v[2], v[3]);
          }
        } else {
          float* d = a.part_o + prow * kD + 32 * cc;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(__uint_as_float(u[8 * q + e]) * inv);
            ptx::st_global_v8(d + 8 * q, v);
          }
        }
      }
      if (live) {
        if (!direct)
          a.part_lse[prow] = lse;
        else if (a.out_lse != nullptr)
          a.out_lse[orow] = lse;
      }
      ptx::tc_fence_before();
    } else {
      *abort_flag = 1;
    }
  }
  __syncthreads();
  if (warp == kWarpMma) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Joins the parts of a row: one warp per row, four columns per lane.
__global__ void __launch_bounds__(128) k_prefix_combine(const PrefixAttnArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const long long rows = (long long)a.B * a.Tq * a.H;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  const int parts = a.splits_p + a.splits_s;
  float m = -INFINITY;
  for (int p = lane; p < parts; p += 32) m = fmaxf(m, a.part_lse[p * rows + row]);
  m = warp_max(m);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  if (m != -INFINITY) {
    for (int p0 = 0; p0 < parts; p0 += 32) {
      const float l = p0 + lane < parts ? a.part_lse[(p0 + lane) * rows + row] : -INFINITY;
      const float wt = ex2((l - m) * 1.4426950408889634f);
      unsigned live = __ballot_sync(0xffffffffu, l != -INFINITY);
      while (live != 0u) {
        const int i = __ffs((int)live) - 1;
        live &= live - 1;
        const float wi = __shfl_sync(0xffffffffu, wt, i);
        const float4 o = *reinterpret_cast<const float4*>(a.part_o + ((p0 + i) * rows + row) * kD + 4 * lane);
        acc.x += wi * o.x, acc.y += wi * o.y, acc.z += wi * o.z, acc.w += wi * o.w;
        sum += wi;
      }
    }
    const float inv = 1.0f / sum;
    acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
  }
  *reinterpret_cast<uint2*>(a.out + row * kD + 4 * lane) = make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
  if (lane == 0 && a.out_lse != nullptr) a.out_lse[row] = m == -INFINITY ? m : m + logf(sum);
}

int ceil_div(long long a, long long b) {
  const long long c = (a + b - 1) / b;
  return c < 0x7fffffffLL ? (int)c : 0x7fffffff;
}

// q [tokens, H, 128] with row stride ldq: box of R heads x box_tok tokens x 64 columns
bool q_map(CUtensorMap* m, const void* q, long long ldq, int tokens, int H, int R, int box_tok) {
  const uint64_t dims[4] = {kD, (uint64_t)H, (uint64_t)tokens, 1};
  const uint64_t strides[3] = {kD * 2, (uint64_t)ldq * 2, (uint64_t)ldq * 2 * (uint64_t)tokens};
  const uint32_t box[4] = {64, (uint32_t)R, (uint32_t)box_tok, 1};
  return make_tmap_4d(m, q, dims, strides, box);
}

// a cache [seqs, len, Hkv, 128] with strides ld (keys) and ls (sequences)
bool kv_map(CUtensorMap* m, const void* p, long long ld, long long ls, int seqs, int len, int Hkv) {
  const uint64_t dims[4] = {kD, (uint64_t)Hkv, (uint64_t)len, (uint64_t)seqs};
  const uint64_t strides[3] = {kD * 2, (uint64_t)ld * 2, (uint64_t)(seqs > 1 ? ls : ld * len) * 2};
  const uint32_t box[4] = {64, 1, kKeys, 1};
  return make_tmap_4d(m, p, dims, strides, box);
}

}  // namespace

// How the work is cut, from the sizes alone (the lengths stay on the device).
// Units of about `target` equal shares of all key tiles keep two CTAs on each
// of 148 SMs busy for several rounds; a split is never shorter than min_tiles.
bool prefix_attn_plan(PrefixAttnArgs* a) {
  const int R = a->H / a->Hkv;
  a->rows_per_group = a->B / a->G;
  const int fit = kRows / R;  // tokens whose query rows fit a tile
  const int tok_p = a->rows_per_group * a->Tq;
  a->box_p = fit < tok_p ? fit : tok_p;
  a->box_s = fit < a->Tq ? fit : a->Tq;
  a->tiles_p = ceil_div(tok_p, a->box_p);
  a->tiles_s = ceil_div(a->Tq, a->box_s);
  // rows of a group differ in position by at most S_max, so a window limits the prefix keys that any of them sees
  const long long see_p = a->window < a->P_max ? (long long)a->window + a->S_max + a->Tq : a->P_max;
  const int kt_p = ceil_div(see_p < a->P_max ? see_p : a->P_max, kKeys) + (a->window < a->P_max ? 1 : 0);
  const long long see_s = (long long)a->window + a->Tq;
  const int kt_s = ceil_div(see_s < a->S_max ? see_s : a->S_max, kKeys) + (see_s < a->S_max ? 1 : 0);
  const long long base_p = a->P_max > 0 ? (long long)a->G * a->Hkv * a->tiles_p : 0;
  const long long base_s = a->S_max > 0 ? (long long)a->B * a->Hkv * a->tiles_s : 0;
  const long long work = base_p * kt_p + base_s * kt_s;
  const int target = 4 * 296;
  int chunk = ceil_div(work, target);
  a->min_tiles = chunk < 2 ? 1 : 2;
  if (chunk < 1) chunk = 1;
  a->splits_p = base_p > 0 ? ceil_div(kt_p, chunk) : 0;
  a->splits_s = base_s > 0 ? ceil_div(kt_s, chunk) : 0;
  if (a->splits_p > kPrefixMaxSplits) a->splits_p = kPrefixMaxSplits;
  if (a->splits_s > kPrefixMaxSplits) a->splits_s = kPrefixMaxSplits;
  const long long up = base_p * a->splits_p, us = base_s * a->splits_s;
  if (up + us > 0x7fffffffLL) return false;
  a->units_p = (int)up;
  a->units = (int)(up + us);
  return true;
}

bool launch_prefix_attn(const PrefixAttnArgs& a, const void* q, long long ldq, const void* kp, const void* vp,
                        long long ldp, long long lsp, const void* ks, const void* vs, long long lds, long long lss,
                        cudaStream_t st) {
  CUtensorMap m[6];
  const int tokens = a.B * a.Tq, R = a.H / a.Hkv;
  if (!q_map(&m[0], q, ldq, tokens, a.H, R, a.box_p) || !q_map(&m[1], q, ldq, tokens, a.H, R, a.box_s)) return false;
  for (int i = 0; i < 4; ++i) m[2 + i] = m[0];  // a side without keys has no units
  if (a.P_max > 0 && (!kv_map(&m[2], kp, ldp, lsp, a.G, a.P_max, a.Hkv) || !kv_map(&m[3], vp, ldp, lsp, a.G, a.P_max, a.Hkv)))
    return false;
  if (a.S_max > 0 && (!kv_map(&m[4], ks, lds, lss, a.B, a.S_max, a.Hkv) || !kv_map(&m[5], vs, lds, lss, a.B, a.S_max, a.Hkv)))
    return false;
  if (!smem_optin(k_prefix_attn, SMEM_BYTES)) return false;
  {
    LaunchScope scope_(KK_PREFIX_ATTN, st);
    if (launch_pdl(k_prefix_attn, dim3(a.units), dim3(kThreads), SMEM_BYTES, st, 1, m[0], m[1], m[2], m[3], m[4], m[5], a) !=
        cudaSuccess)
      return false;
  }
  if (a.splits_p + a.splits_s == 1) return true;
  const long long rows = (long long)tokens * a.H;
  LaunchScope scope_(KK_PREFIX_ATTN, st);
  return launch_pdl(k_prefix_combine, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, st, 1, a) == cudaSuccess;
}

}  // namespace nc
