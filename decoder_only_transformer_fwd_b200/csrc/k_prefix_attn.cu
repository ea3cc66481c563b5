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
// per row.  What bounds it (one B200): under a long prefix HBM (64 rows, 12
// heads, 32768 shared and up to 1024 own keys: 69 us, 5.5 TB/s); for few keys the
// latency of two kernels, tables, one tile and the join (10.9 us); in between a
// tile's softmax chain, 0.6 us per SM, which a row's own keys pay in full for the
// one or few queries that they have (16 rows, 2048 + 512 keys, window 1024: 16.3
// us, its bytes take 3.9).
//
// The work of a key head is a sequence of units, prefix units (group, 128-row
// query tile) and then suffix units (row, query tile), each a run of 64-key
// tiles.  Neighbouring CTAs take neighbouring heads (or, with many heads, bands
// of heads), and the CTAs of a band cut its sequence of tiles into equal shares,
// as the lengths in memory give them: a long unit is spread over many CTAs, a
// CTA takes many short ones, all finish together, and the heads' keys of one
// token, which lie side by side in memory, are read at the same time (68.8 us in
// the first case above, 69.4 with the heads one after the other).
// What a CTA does of a unit is a piece; it leaves its rows' normalised output
// (fp32) and log-sum-exp in the workspace, at slot (unit + CTA of the band),
// which no two pieces share.  k_prefix_combine joins a row's pieces with weights
// exp(lse_piece - lse).
//
// A CTA: warps 0..3 softmax (one row per thread = TMEM lane), warp 4 cuts the
// pieces and issues the copies (TMA), warp 5 MMA.  Warp 4 runs ahead: the next
// pieces' keys stream while the last piece's rows are written.  64-key K and V
// tiles go through a ring of 16 KB slots in the order K0 K1 V0 K2 V1 ...; S is
// double-buffered in TMEM, so Q K_{t+1}^T runs during tile t's exponentials,
// and P_t (bf16) overwrites the first half of S_t.  Two CTAs share an SM.
// Every wait is bounded.
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
constexpr int kPieces = 4;                 // depth of the ring of pieces
constexpr int kMaxBins = 512;              // entries of either side's table of starts
constexpr int OFF_SLOT = 2 * Q_BOX;
constexpr int OFF_BAR = OFF_SLOT + SLOTS * SLOT_BYTES;
constexpr int OFF_PIECE = OFF_BAR + 256;
constexpr int OFF_START = OFF_PIECE + kPieces * 64;
constexpr int OFF_SEEN = OFF_START + (2 * kMaxBins + 2) * 4;
constexpr int SMEM_BYTES = OFF_SEEN + kMaxBins * 8 + 1024;
static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs per SM");
constexpr int kThreads = 192, kWarpTma = 4, kWarpMma = 5;
constexpr uint32_t TMEM_COLS = 256;        // S0 64 | S1 64 | O 128
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kLn2 = 0.6931471805599453f;
// The workspace may start at any 16-byte boundary; rows of pieces are stored 32
// bytes at a time, so the areas in it start at the next multiple of this.
constexpr size_t kWsAlign = 256;

struct Piece {
  int suffix, seq, hk;  // side, group or row, key head
  int tok0, ntok;       // query tokens (token = row * Tq + i)
  int lo, hi;           // keys that some row of the unit's sequence sees, from the side's first key
  int t0, nt;           // key tiles; nt == 0: no more pieces
  int slot;
};
static_assert(sizeof(Piece) <= 64, "piece area");

struct Seq {  // a group's prefix or a row's own keys
  int P, S;
  int lo, hi;  // keys that some query sees
};

__device__ __forceinline__ int clamp_len(int n, int most) { return min(max(n, 0), most); }

// shortest own length of a group's rows from r0 on, every `step`-th
__device__ __forceinline__ int least_suffix(const PrefixAttnArgs& a, int g, int r0, int step) {
  if (a.S_max == 0) return 0;
  int least = a.S_max;
  for (int r = r0; r < a.rows_per_group; r += step)
    least = min(least, clamp_len(a.suffix_lens[g * a.rows_per_group + r], a.S_max));
  return least;
}

// Keys [lo, hi) of group g's prefix that a query of one of its rows sees; a
// window makes lo depend on the shortest row.
__device__ __forceinline__ Seq prefix_seq(const PrefixAttnArgs& a, int g, int least) {
  Seq s;
  s.P = s.hi = clamp_len(a.prefix_lens[g], a.P_max);
  s.S = 0;
  s.lo = min(s.P, max(0, s.P + least - a.Tq - a.window + 1));
  return s;
}
__device__ __forceinline__ bool windowed(const PrefixAttnArgs& a) { return a.window < a.P_max + a.S_max; }
__device__ __forceinline__ Seq prefix_seq(const PrefixAttnArgs& a, int g) {
  return prefix_seq(a, g, windowed(a) ? least_suffix(a, g, 0, 1) : 0);
}

__device__ __forceinline__ Seq suffix_seq(const PrefixAttnArgs& a, int b) {
  Seq s;
  s.P = a.P_max > 0 ? clamp_len(a.prefix_lens[b / a.rows_per_group], a.P_max) : 0;
  s.S = s.hi = clamp_len(a.suffix_lens[b], a.S_max);
  s.lo = min(s.S, max(0, s.S - a.Tq - a.window + 1));
  return s;
}

// first key and number of key tiles of a sequence's query tile tt (prefix:
// every tile has the same; suffix: keys behind the tile's last query are not
// its own)
__device__ __forceinline__ int unit_tiles(const PrefixAttnArgs& a, const Seq& s, int suffix, int tt, int* t0) {
  int lo = s.lo, hi = s.hi;
  if (suffix) {
    const int first = s.S - a.Tq + tt * a.box_s, last = s.S - a.Tq + min(a.Tq, (tt + 1) * a.box_s) - 1;
    lo = max(lo, first - a.window + 1);
    hi = min(hi, last + 1);
  }
  *t0 = lo / kKeys;
  return lo < hi ? (hi + kKeys - 1) / kKeys - *t0 : 0;
}

__device__ __forceinline__ int unit_cost(const PrefixAttnArgs& a, int suffix, int tiles) {
  return tiles > 0 ? tiles + (suffix ? a.fixed_s : a.fixed_p) : 0;
}

// cost of all query tiles of a row, for one key head
__device__ __forceinline__ int suffix_cost(const PrefixAttnArgs& a, const Seq& s) {
  int c = 0, t0;
  for (int tt = 0; tt < a.tiles_s; ++tt) c += unit_cost(a, 1, unit_tiles(a, s, 1, tt, &t0));
  return c;
}

// Fills the tables: start[i], the cost before each bin of groups, then of rows
// (the last entry is the total), and lo[g], hi[g] of each group's prefix where a
// bin is one group.  All threads of the CTA.
__device__ void fill_tables(const PrefixAttnArgs& a, int* start, int2* seen, int warp, int lane) {
  for (int i = warp; i < a.bins_p; i += kThreads / 32) {
    int c = 0, t0;
    for (int g = i * a.bin_p; g < min(a.G, (i + 1) * a.bin_p); ++g) {
      const int least = windowed(a) ? __reduce_min_sync(0xffffffffu, least_suffix(a, g, lane, 32)) : 0;
      const Seq s = prefix_seq(a, g, least);
      c += a.band * a.tiles_p * unit_cost(a, 0, unit_tiles(a, s, 0, 0, &t0));
      if (lane == 0 && a.bin_p == 1) seen[g] = make_int2(s.lo, s.hi);
    }
    if (lane == 0) start[i] = c;
  }
  // rows from the last thread down: few rows are not behind warp 0's groups
  for (int i = kThreads - 1 - threadIdx.x; i < a.bins_s; i += kThreads) {
    int c = 0;
    for (int b = i * a.bin_s; b < min(a.B, (i + 1) * a.bin_s); ++b) c += a.band * suffix_cost(a, suffix_seq(a, b));
    start[a.bins_p + i] = c;
  }
  __syncthreads();
  if (warp == 0) {
    const int n = a.bins_p + a.bins_s, per = (n + 31) / 32, i0 = min(n, lane * per), i1 = min(n, i0 + per);
    int sum = 0;
    for (int i = i0; i < i1; ++i) sum += start[i];
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += v;
    }
    const int total = __shfl_sync(0xffffffffu, before, 31);
    before -= sum;
    for (int i = i0; i < i1; ++i) {
      const int v = start[i];
      start[i] = before;
      before += v;
    }
    if (lane == 0) start[n] = total;
  }
  __syncthreads();
}

__device__ __forceinline__ Seq group_seq(const PrefixAttnArgs& a, const int2* seen, int g) {
  if (a.bin_p > 1) return prefix_seq(a, g);
  Seq s;
  s.P = s.hi = seen[g].y;
  s.S = 0;
  s.lo = seen[g].x;
  return s;
}

// share of a band's total cost that a CTA takes
__device__ __forceinline__ int share_of(const PrefixAttnArgs& a, int total) {
  return max((total + a.per_band - 1) / a.per_band, max(a.fixed_p, a.fixed_s) + 1);
}

// Slot of what CTA `cta` of band b does of the band's unit u.
__device__ __forceinline__ int slot_of(const PrefixAttnArgs& a, int suffix, int b, int u, int cta) {
  return b * ((suffix ? a.B * a.tiles_s : a.G * a.tiles_p) * a.band + a.per_band) + u + cta;
}

// The piece that holds cost position v, as far as `end`; *next: the position
// behind it.  All lanes of a warp.  A piece may have no tile (it holds only a unit's fixed cost).
// Lengths that change while the kernel runs give wrong pieces, but every loop
// ends and every index stays in range.
__device__ Piece piece_at(const PrefixAttnArgs& a, const int* start, const int2* seen, int band, int cta, int v, int end,
                          int lane, int* next) {
  // the last bin that starts at or before v: the warp looks at 32 places at once
  const int bins = a.bins_p + a.bins_s, step = (bins + 31) / 32;
  int lo = step * (__popc(__ballot_sync(0xffffffffu, lane * step < bins && start[lane * step] <= v)) - 1);
  if (step > 1) {
    const int i = lo + lane;
    lo += __popc(__ballot_sync(0xffffffffu, lane < step && i < bins && start[i] <= v)) - 1;
  }
  Piece p;
  p.suffix = lo >= a.bins_p;
  int at = v - start[lo], t0 = 0, tiles = 0, tt = 0;
  Seq s;
  if (!p.suffix) {
    for (p.seq = lo * a.bin_p;; ++p.seq) {
      s = group_seq(a, seen, p.seq);
      tiles = unit_tiles(a, s, 0, 0, &t0);
      const int all = a.band * a.tiles_p * unit_cost(a, 0, tiles);
      if (at < all || p.seq + 1 >= a.G) break;
      at -= all;
    }
    const int u = min(at / max(unit_cost(a, 0, tiles), 1), a.band * a.tiles_p - 1);
    at -= u * unit_cost(a, 0, tiles);
    p.hk = u / a.tiles_p;
    tt = u % a.tiles_p;
  } else {
    int one;
    for (p.seq = (lo - a.bins_p) * a.bin_s;; ++p.seq) {
      s = suffix_seq(a, p.seq);
      one = suffix_cost(a, s);
      if (at < a.band * one || p.seq + 1 >= a.B) break;
      at -= a.band * one;
    }
    p.hk = min(at / max(one, 1), a.band - 1);
    at -= p.hk * one;
    for (tt = 0;; ++tt) {
      tiles = unit_tiles(a, s, 1, tt, &t0);
      if (at < unit_cost(a, 1, tiles) || tt + 1 >= a.tiles_s) break;
      at -= unit_cost(a, 1, tiles);
    }
  }
  const int fixed = p.suffix ? a.fixed_s : a.fixed_p, unit_end = v - at + unit_cost(a, p.suffix, tiles);
  *next = max(v + 1, min(end, unit_end));
  const int first = max(0, at - fixed), last = *next - (v - at) - fixed;
  p.t0 = t0 + first;
  p.nt = min(max(0, last - first), max(0, tiles - first));
  p.lo = s.lo;
  p.hi = s.hi;
  const int tokens = (p.suffix ? 1 : a.rows_per_group) * a.Tq, box = p.suffix ? a.box_s : a.box_p;
  p.tok0 = p.seq * tokens + tt * box;
  p.ntok = min(box, tokens - tt * box);
  p.slot = slot_of(a, p.suffix, band, (p.seq * a.band + p.hk) * (p.suffix ? a.tiles_s : a.tiles_p) + tt, cta);
  p.hk += band * a.band;
  return p;
}

// Where the pieces of unit u of a side lie, for k_prefix_combine: first slot and
// number of CTAs that hold one of its tiles.  Units are numbered by sequence, key
// head, query tile.
__device__ int2 unit_pieces(const PrefixAttnArgs& a, const int* start, const int2* seen, int share, int suffix, int u) {
  const int tiles_q = suffix ? a.tiles_s : a.tiles_p, bin = suffix ? a.bin_s : a.bin_p;
  const int tt = u % tiles_q, hk = u / tiles_q % a.Hkv, seq = u / tiles_q / a.Hkv, i0 = seq / bin * bin;
  const int b = hk / a.band, hb = hk % a.band;  // band, head within it
  int at = start[(suffix ? a.bins_p : 0) + seq / bin] + (suffix ? a.fixed_s : a.fixed_p), t0, tiles;
  if (!suffix) {
    for (int i = i0; i < seq; ++i) at += a.band * a.tiles_p * unit_cost(a, 0, unit_tiles(a, group_seq(a, seen, i), 0, 0, &t0));
    tiles = unit_tiles(a, group_seq(a, seen, seq), 0, 0, &t0);
    at += (hb * a.tiles_p + tt) * unit_cost(a, 0, tiles);
  } else {
    for (int i = i0; i < seq; ++i) at += a.band * suffix_cost(a, suffix_seq(a, i));
    const Seq s = suffix_seq(a, seq);
    at += hb * suffix_cost(a, s);
    for (int i = 0; i < tt; ++i) at += unit_cost(a, 1, unit_tiles(a, s, 1, i, &t0));
    tiles = unit_tiles(a, s, 1, tt, &t0);
  }
  if (tiles == 0) return make_int2(0, 0);
  return make_int2(slot_of(a, suffix, b, (seq * a.band + hb) * tiles_q + tt, at / share),
                   (at + tiles - 1) / share - at / share + 1);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  enum {
    B_QF = 0, B_QE, B_F, B_E = B_F + SLOTS, B_S = B_E + SLOTS, B_P = B_S + 2, B_O = B_P + 2, B_FIN, B_OE, B_DF,
    B_DE = B_DF + kPieces, B_DONE = B_DE + kPieces, NB
  };
  static_assert(NB * 8 + 8 <= 256, "barrier area");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NB);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto piece_mem = [&](int i) { return reinterpret_cast<Piece*>(smem + OFF_PIECE + (i % kPieces) * 64); };
  int* start = reinterpret_cast<int*>(smem + OFF_START);
  int2* seen = reinterpret_cast<int2*>(smem + OFF_SEEN);
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8u * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int band = blockIdx.x % a.bands, cta = blockIdx.x / a.bands;  // band of heads, CTA of the band

  if (threadIdx.x == 0) {
    ptx::mbar_init(bar(B_QF), 1);
    ptx::mbar_init(bar(B_QE), 1);
    for (int s = 0; s < SLOTS; ++s) {
      ptx::mbar_init(bar(B_F + s), 1);
      ptx::mbar_init(bar(B_E + s), 1);
    }
    for (int g = 0; g < 2; ++g) {
      ptx::mbar_init(bar(B_S + g), 1);
      ptx::mbar_init(bar(B_P + g), 4);
    }
    ptx::mbar_init(bar(B_O), 1);
    ptx::mbar_init(bar(B_FIN), 1);
    ptx::mbar_init(bar(B_OE), 4);
    for (int i = 0; i < kPieces; ++i) {
      ptx::mbar_init(bar(B_DF + i), 1);
      ptx::mbar_init(bar(B_DE + i), 5);  // four softmax warps and the MMA thread
    }
    ptx::mbar_init(bar(B_DONE), 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == kWarpTma && lane < 6)
    ptx::prefetch_tmap(lane == 0 ? &tmQp : lane == 1 ? &tmQs : lane == 2 ? &tmKp : lane == 3 ? &tmVp : lane == 4 ? &tmKs : &tmVs);
  pdl_wait();  // lengths, q and the caches may come from the previous kernel
  // Tensor memory before anything else: the second CTA of an SM starts only when
  // the first has given up its allocation permit (measured: 2.6 us after it with
  // the allocation behind the tables, 0.6 us with it ahead of them).  It comes
  // after the wait, and the next kernel may start only after it: a CTA that holds
  // tensor memory never waits for a kernel that may still need some.
  if (warp == kWarpMma) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), TMEM_COLS);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
    pdl_launch_dependents();
  }
  fill_tables(a, start, seen, warp, lane);
  const int bins = a.bins_p + a.bins_s, total = start[bins];
  const int share = share_of(a, total);
  const long long v_begin = (long long)cta * share;
  const bool works = v_begin < total;
  const int v0 = (int)min(v_begin, (long long)total), v1 = (int)min(v_begin + share, (long long)total);
  ptx::tc_fence_after();  // the allocation, before the barriers of fill_tables
  const uint32_t tmem = *tmem_slot;
  if (warp < 4) {  // while the first copies are on their way
    const int units_p = a.P_max > 0 ? a.G * a.Hkv * a.tiles_p : 0, units_s = a.S_max > 0 ? a.B * a.Hkv * a.tiles_s : 0;
    for (int u = blockIdx.x * 128 + threadIdx.x; u < units_p + units_s; u += a.ctas * 128)
      a.pieces[u] = unit_pieces(a, start, seen, share, u >= units_p, u >= units_p ? u - units_p : u);
  }
  if (blockIdx.x + 1 == gridDim.x && warp < 4) {  // lengths out of range are reported once
    bool bad = false;
    if (a.P_max > 0)
      for (int g = threadIdx.x; g < a.G; g += 128) bad |= (unsigned)a.prefix_lens[g] > (unsigned)a.P_max;
    if (a.S_max > 0)
      for (int b = threadIdx.x; b < a.B; b += 128) bad |= (unsigned)a.suffix_lens[b] > (unsigned)a.S_max;
    if (bad) atomicOr(a.status, kStatusData);
  }
  if (!works) {
    if (warp == kWarpMma) ptx::tmem_dealloc(tmem, TMEM_COLS);
    return;
  }
  auto sSlot = [&](int s) { return ptx::smem_u32(smem + OFF_SLOT + s * SLOT_BYTES); };
  const uint32_t sQ = ptx::smem_u32(smem);
  const int R = a.H / a.Hkv;
  // place of a piece's K_t and V_t in its sequence of 2 nt tiles
  auto seq_k = [](int t) { return t == 0 ? 0 : 2 * t - 1; };
  auto seq_v = [](int t, int nt) { return t + 1 < nt ? 2 * t + 2 : 2 * nt - 1; };
  // the n-th piece; false on a timeout
  auto piece_wait = [&](int n, Piece* p) -> bool {
    if (*abort_flag || !ptx::mbar_wait(bar(B_DF + n % kPieces), (uint32_t)(n / kPieces) & 1u, a.status)) return false;
    *p = *piece_mem(n);
    return true;
  };

  if (warp == kWarpTma) {
    bool ok = true;
    int sc0 = 0, n = 0;           // tiles issued by earlier pieces, pieces
    int sc_done = 0, q_done = 0;  // lane 0: copies issued
    int v = v0;
    while (ok) {
      Piece p;
      p.nt = 0;
      while (v < v1 && p.nt == 0) {
        int next;
        p = piece_at(a, start, seen, band, cta, v, v1, lane, &next);
        v = next;
      }
      if (lane == 0) {
        ok = !*abort_flag && ptx::mbar_wait(bar(B_DE + n % kPieces), ((uint32_t)(n / kPieces) & 1u) ^ 1u, a.status);
        if (ok) {
          *piece_mem(n) = p;
          ptx::mbar_arrive(bar(B_DF + n % kPieces));
          const void* tq = p.suffix ? (const void*)&tmQs : (const void*)&tmQp;
          const void* tk = p.suffix ? (const void*)&tmKs : (const void*)&tmKp;
          const void* tv = p.suffix ? (const void*)&tmVs : (const void*)&tmVp;
          for (int i = 0; ok && i < 2 * p.nt; ++i) {
            // K0 K1 V0 K2 V1 ... K_{nt-1} V_{nt-2} V_{nt-1}
            const bool is_k = i == 0 || (i % 2 == 1 && i < 2 * p.nt - 1);
            const int t = i == 0 ? 0 : (is_k ? (i + 1) / 2 : (i == 2 * p.nt - 1 ? p.nt - 1 : i / 2 - 1));
            const int s = (sc0 + i) % SLOTS;
            if (*abort_flag || !ptx::mbar_wait(bar(B_E + s), ((uint32_t)((sc0 + i) / SLOTS) & 1u) ^ 1u, a.status)) {
              ok = false;
              break;
            }
            ptx::mbar_arrive_expect_tx(bar(B_F + s), SLOT_BYTES);
            const int key = (p.t0 + t) * kKeys;
            ptx::tma_load_4d(sSlot(s), is_k ? tk : tv, bar(B_F + s), 0, p.hk, key, p.seq);
            ptx::tma_load_4d(sSlot(s) + KV_BOX, is_k ? tk : tv, bar(B_F + s), 64, p.hk, key, p.seq);
            ++sc_done;
            if (i == 0) {
              // the first keys do not need the query buffer, which the last
              // piece's products may still be reading
              if (*abort_flag || !ptx::mbar_wait(bar(B_QE), ((uint32_t)n & 1u) ^ 1u, a.status)) {
                ok = false;
                break;
              }
              ptx::mbar_arrive_expect_tx(bar(B_QF), (uint32_t)(2 * (p.suffix ? a.box_s : a.box_p) * R * 128));
              ptx::tma_load_4d(sQ, tq, bar(B_QF), 0, p.hk * R, p.tok0, 0);
              ptx::tma_load_4d(sQ + Q_BOX, tq, bar(B_QF), 64, p.hk * R, p.tok0, 0);
              ++q_done;
            }
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      sc0 += 2 * p.nt;
      ++n;
      if (p.nt == 0) break;
    }
    if (lane == 0) {
      if (!ok) *abort_flag = 1;
      // every copy issued here has landed before the CTA may exit
      if (q_done > 0) ptx::mbar_wait(bar(B_QF), (uint32_t)(q_done - 1) & 1u, a.status);
      for (int sc = max(0, sc_done - SLOTS); sc < sc_done; ++sc)
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
      bool ok = true;
      int sc0 = 0, j0 = 0;  // ring tiles and key tiles of earlier pieces
      for (int n = 0;; ++n) {
        Piece p;
        if (!piece_wait(n, &p)) {
          ok = false;
          break;
        }
        ptx::mbar_arrive(bar(B_DE + n % kPieces));
        if (p.nt == 0) break;
        auto qk = [&](int t) -> bool {
          const int sc = sc0 + seq_k(t), j = j0 + t;
          if (!full(sc)) return false;
          ptx::tc_fence_after();
          const uint64_t dk = dk0 + (uint64_t)((sc % SLOTS) * (SLOT_BYTES >> 4));
#pragma unroll
          for (int kk = 0; kk < kD / 16; ++kk)
            ptx::mma_bf16_ss(tmem + (uint32_t)((j & 1) * kKeys), dq + (uint64_t)((kk >> 2) * (Q_BOX >> 4) + (kk & 3) * 2),
                             dk + (uint64_t)((kk >> 2) * (KV_BOX >> 4) + (kk & 3) * 2), idesc_qk, kk > 0 ? 1u : 0u);
          ptx::mma_commit(bar(B_S + (j & 1)));
          ptx::mma_commit(bar(B_E + sc % SLOTS));
          if (t + 1 == p.nt) ptx::mma_commit(bar(B_QE));
          return true;
        };
        ok = ptx::mbar_wait(bar(B_QF), (uint32_t)n & 1u, a.status) && qk(0);
        for (int t = 0; ok && t < p.nt; ++t) {
          // S_{t+1} goes where P_{t-1} was, whose product was issued before
          if (t + 1 < p.nt && !qk(t + 1)) {
            ok = false;
            break;
          }
          const int sc = sc0 + seq_v(t, p.nt), j = j0 + t;
          if (!full(sc) || *abort_flag || !ptx::mbar_wait(bar(B_P + (j & 1)), (uint32_t)(j >> 1) & 1u, a.status)) {
            ok = false;
            break;
          }
          // the last piece's rows have been read out of O
          if (t == 0 && n > 0 && !ptx::mbar_wait(bar(B_OE), (uint32_t)(n - 1) & 1u, a.status)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint64_t dv = dv0 + (uint64_t)((sc % SLOTS) * (SLOT_BYTES >> 4));
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            ptx::mma_bf16_ts(tmem + 128u, tmem + (uint32_t)((j & 1) * kKeys + kk * 8), dv + (uint64_t)(kk * (2048 >> 4)),
                             idesc_pv, (t > 0 || kk > 0) ? 1u : 0u);
          ptx::mma_commit(bar(B_E + sc % SLOTS));
          ptx::mma_commit(bar(B_O));
          if (t + 1 == p.nt) ptx::mma_commit(bar(B_FIN));
        }
        if (!ok) break;
        sc0 += 2 * p.nt;
        j0 += p.nt;
      }
      if (!ok) *abort_flag = 1;
      ptx::mma_commit(bar(B_DONE));
      ptx::mbar_wait(bar(B_DONE), 0, a.status);
    }
  } else {
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const uint32_t tO = tmem + 128u + lane_off;
    const float c = a.scale_log2;
    bool ok = true;
    int sc0 = 0, j0 = 0;
    const int my_tok = (int)threadIdx.x / R;
    Piece p, p_next;
    int lo_next, hi_next;
    // takes the n-th piece, and the keys [lo, hi) that this thread's row sees of
    // it, from the side's first key (a thread without a row masks nothing: no one
    // reads its weights)
    auto look = [&](int n) -> bool {
      if (!piece_wait(n, &p_next)) return false;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(B_DE + n % kPieces));
      lo_next = 0, hi_next = 0x7fffffff;
      if ((int)threadIdx.x < p_next.ntok * R && p_next.nt > 0) {
        const int token = p_next.tok0 + my_tok, b = token / a.Tq;
        const int P = a.P_max > 0 ? clamp_len(a.prefix_lens[b / a.rows_per_group], a.P_max) : 0;
        const int S = a.S_max > 0 ? clamp_len(a.suffix_lens[b], a.S_max) : 0;
        const int pos = P + S - a.Tq + token % a.Tq, base = p_next.suffix ? P : 0;
        lo_next = max(0, pos - a.window + 1 - base);
        hi_next = min(p_next.suffix ? S : P, pos + 1 - base);
        if (lo_next >= hi_next) lo_next = hi_next = 0;
      }
      return true;
    };
    p.nt = p.ntok = 0;
    int lo = 0, hi = 0;
    // The first turn only takes piece 0: every part of the loop stands in the code
    // once, since a CTA fetches it cold (a second copy of `look` or of the zeros
    // below costs 0.2 us of a short call each).
    for (int n = -1;; ++n) {
      const int nrows = p.ntok * R;
      const bool live = (int)threadIdx.x < nrows, warp_live = warp * 32 < nrows;
      float m_run = -INFINITY, l_run = 0.f;
      for (int t = 0; t < p.nt; ++t) {
        const int j = j0 + t;
        const uint32_t tS = tmem + (uint32_t)((j & 1) * kKeys) + lane_off;
        const int k0 = (p.t0 + t) * kKeys;
        if (*abort_flag || !ptx::mbar_wait(bar(B_S + (j & 1)), (uint32_t)(j >> 1) & 1u, a.status)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        if (warp_live) {
          const int clo = lo - k0, chi = hi - k0;  // visible columns [clo, chi)
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
          float mx[4] = {fmaxf(x[0], x[1]), fmaxf(x[2], x[3]), fmaxf(x[4], x[5]), fmaxf(x[6], x[7])};
#pragma unroll
          for (int i = 8; i < kKeys; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], x[i + 2 * k], x[i + 2 * k + 1]);
          const float tmax = max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
          // the running max moves only when it grows by more than 2^8
          const bool rescale = live && (tmax - m_run) * c > kRescaleThreshold;
          const float m_new = rescale ? tmax : m_run;
          const float mc = m_new == -INFINITY ? 0.f : m_new * c;
          float2 sm[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {  // the first half is stored under the second's exponentials
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 e = __ffma2_rn(make_float2(x[32 * hf + 2 * i], x[32 * hf + 2 * i + 1]), c2, mc2);
              const float2 q = make_float2(ex2(e.x), ex2(e.y));
              sm[i & 1] = __fadd2_rn(sm[i & 1], q);
              // V is bf16, and the product takes operands of one type; the sum keeps
              // the fp32 weights.  Error of the output against fp64, relative in the
              // mean: 0.0022, of which its own rounding to bf16 is 0.0016.
              pk[i] = pack_bf16(q.x, q.y);
            }
            ptx::tmem_st16(tS + (uint32_t)(16 * hf), pk);
          }
          const float alpha = rescale ? ex2(m_run * c - mc) : 1.f;  // 0 when m_run == -inf
          if (rescale) {
            l_run *= alpha;
            m_run = m_new;
          }
          const float2 s2 = __fadd2_rn(sm[0], sm[1]);
          l_run += s2.x + s2.y;
          // P V of tile t - 1 must have landed before O is rescaled (S_t shows
          // that the one before it has)
          if (t > 0 && __any_sync(0xffffffffu, rescale)) {
            if (!ptx::mbar_wait(bar(B_O), (uint32_t)(j - 1) & 1u, a.status)) {
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
        }
        // V rows that no query of the sequence sees (behind the end, before
        // the window) may hold anything: they become zeros, since 0 x NaN is not 0
        if (k0 < p.lo || k0 + kKeys > p.hi) {
          const int sc = sc0 + seq_v(t, p.nt), s = sc % SLOTS;
          if (!ptx::mbar_wait(bar(B_F + s), (uint32_t)(sc / SLOTS) & 1u, a.status)) {
            ok = false;
            break;
          }
          for (int i = threadIdx.x; i < kKeys * 16; i += 128) {
            const int key = k0 + i / 16;
            if (key < p.lo || key >= p.hi)
              *reinterpret_cast<uint4*>(smem + OFF_SLOT + s * SLOT_BYTES + ((i & 8) ? KV_BOX : 0) + (i / 16) * 128 +
                                        (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          ptx::fence_proxy_async_smem();
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(B_P + (j & 1)));
      }
      // the next piece, while the last product runs
      if (!ok || !look(n + 1) || (n >= 0 && !ptx::mbar_wait(bar(B_FIN), (uint32_t)n & 1u, a.status))) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      if (warp_live) {
        const float inv = l_run == 0.f ? 0.f : 1.0f / l_run;
        const long long prow = (long long)p.slot * ((p.suffix ? a.box_s : a.box_p) * R) + threadIdx.x;
        float* dst = (p.suffix ? a.part_os : a.part_op) + prow * kD;
#pragma unroll 1
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t u[32];
          ptx::tmem_ld32(tO + (uint32_t)(cc * 32), u);
          ptx::tmem_ld_wait();
          if (live && inv != 0.f) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(__uint_as_float(u[8 * q + e]) * inv);
              ptx::st_global_v8(dst + 32 * cc + 8 * q, w);
            }
          }
        }
        // a row that sees none of the piece's keys has weight 0 and no output there
        if (live)
          (p.suffix ? a.part_ls : a.part_lp)[prow] = inv != 0.f ? (m_run * c + log2f(l_run)) * kLn2 : -INFINITY;
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (n >= 0 && lane == 0) ptx::mbar_arrive(bar(B_OE));
      sc0 += 2 * p.nt;
      j0 += p.nt;
      if (p_next.nt == 0) break;
      p = p_next, lo = lo_next, hi = hi_next;
    }
    if (!ok) *abort_flag = 1;
  }
  __syncthreads();
  if (warp == kWarpMma) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Joins a row's pieces: WPR warps per row, four columns per lane; warp w takes
// every WPR-th piece and the warps' sums are joined in shared memory.
template <int WPR>
__global__ void __launch_bounds__(WPR > 4 ? 32 * WPR : 128) k_prefix_combine(const PrefixAttnArgs a) {
  __shared__ float4 s_acc[WPR > 1 ? WPR : 1][32];
  __shared__ float s_m[WPR], s_sum[WPR];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w0 = WPR > 1 ? warp : 0;
  const long long row = WPR > 1 ? (long long)blockIdx.x : (long long)blockIdx.x * 4 + warp;  // token-major, then head
  if (row >= (long long)a.B * a.Tq * a.H) return;
  const int R = a.H / a.Hkv, token = (int)(row / a.H), h = (int)(row % a.H), hk = h / R;
  // the row's unit on either side, and its row in the unit's tile
  int2 in_p = make_int2(0, 0), in_s = make_int2(0, 0);
  int rp = 0, rs = 0;
  if (a.P_max > 0) {
    const int per = a.rows_per_group * a.Tq, g = token / per, it = token % per;
    in_p = a.pieces[(g * a.Hkv + hk) * a.tiles_p + it / a.box_p];
    rp = it % a.box_p * R + h % R;
  }
  if (a.S_max > 0) {
    const int b = token / a.Tq, it = token % a.Tq;
    in_s = a.pieces[(a.P_max > 0 ? a.G * a.Hkv * a.tiles_p : 0) + (b * a.Hkv + hk) * a.tiles_s + it / a.box_s];
    rs = it % a.box_s * R + h % R;
  }
  const int parts = in_p.y + in_s.y;
  float m = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = w0; p0 < parts; p0 += 32 * WPR) {
    // lane i holds piece p0 + WPR i: its weight, and where its output row is
    const int p = p0 + WPR * lane, n = min(32, (parts - p0 + WPR - 1) / WPR);
    const bool side = p >= in_p.y;
    const long long r = side ? (long long)(in_s.x + min(p, parts - 1) - in_p.y) * (a.box_s * R) + rs
                             : (long long)(in_p.x + p) * (a.box_p * R) + rp;
    const float* lse = (side ? a.part_ls : a.part_lp) + r;
    const unsigned long long o = reinterpret_cast<unsigned long long>((side ? a.part_os : a.part_op) + r * kD);
    // four rows in flight, beside the weights; a piece of weight 0 may have left
    // no row (whatever is there is read and not used)
    float4 x[4];
    auto load = [&](int i0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned long long oi = __shfl_sync(0xffffffffu, o, min(i0 + i, n - 1));
        x[i] = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(oi) + 4 * lane);
      }
    };
    const float l = p < parts ? *lse : -INFINITY;
    load(0);
    const float m_new = fmaxf(m, warp_max(l));
    // (a maximum skips NaN, so a row of nothing else is told apart from an empty one)
    if (m_new == -INFINITY && !__any_sync(0xffffffffu, l != l)) continue;
    const float w = ex2((l - m_new) * 1.4426950408889634f), old = ex2((m - m_new) * 1.4426950408889634f);
    m = m_new;
    sum = sum * old + warp_sum(w);
    acc.x *= old, acc.y *= old, acc.z *= old, acc.w *= old;
    for (int i0 = 0; i0 < n; i0 += 4) {
      if (i0 > 0) load(i0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float wi = i0 + i < n ? __shfl_sync(0xffffffffu, w, i0 + i) : 0.f;
        if (wi != 0.f) acc.x += wi * x[i].x, acc.y += wi * x[i].y, acc.z += wi * x[i].z, acc.w += wi * x[i].w;
      }
    }
  }
  if (WPR > 1) {
    s_acc[warp][lane] = acc;
    if (lane == 0) s_m[warp] = m, s_sum[warp] = sum;
    __syncthreads();
    if (warp > 0) return;
    float top = s_m[0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) top = fmaxf(top, s_m[i]);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) {
      const float w = s_sum[i] == 0.f ? 0.f : ex2((s_m[i] - top) * 1.4426950408889634f);
      const float4 x = s_acc[i][lane];
      acc.x += w * x.x, acc.y += w * x.y, acc.z += w * x.z, acc.w += w * x.w;
      sum += w * s_sum[i];
    }
    m = top;
  }
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  *reinterpret_cast<uint2*>(a.out + row * kD + 4 * lane) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (lane == 0 && a.out_lse != nullptr) a.out_lse[row] = sum == 0.f ? m : m + logf(sum);
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// What a unit of so many query rows costs besides its tiles (query load, set-up,
// rows out), in tiles of about 1 us: 2, 3 or 4.  Against 2 for every unit: 3 x 20
// rows x 5 queries (126 and 15 rows) over 5000 + 333 keys 27.7 us for 28.8, 4 x
// 32 rows (128 and 4) over 2000 + 500 40.1 for 41.2.  Against 3 and 4: 64 rows over
// 4096 + 1024 keys (64 and 1) 43.2 for 44.6, 4 rows over 512 + 64 10.5 for 10.9.
int unit_fixed(int rows) { return 2 + (rows > 8) + (rows > 64); }

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

// The sizes that do not depend on the lengths, and the workspace's bytes; false
// where a count does not fit an int.
bool prefix_attn_plan(PrefixAttnArgs* a, size_t* bytes) {
  const int R = a->H / a->Hkv;
  a->rows_per_group = a->B / a->G;
  // Bands of heads: as narrow as leaves at most 5% of the CTAs without work
  // (12 heads: 12 bands of 24 CTAs; 100 heads: 25 bands of 11), or the best.
  int used = 0;
  for (int band = 1; band <= a->Hkv; ++band) {
    if (a->Hkv % band != 0 || a->Hkv / band > kPrefixCtas) continue;
    const int bands = a->Hkv / band, per = kPrefixCtas / bands;
    if (bands * per > used) {
      used = bands * per;
      a->band = band, a->bands = bands, a->per_band = per;
    }
    if (20 * used >= 19 * kPrefixCtas) break;
  }
  a->ctas = a->bands * a->per_band;
  const int fit = kRows / R;  // tokens whose query rows fit a tile
  const long long tok_p = (long long)a->rows_per_group * a->Tq;
  a->box_p = (int)(fit < tok_p ? fit : tok_p);
  a->box_s = fit < a->Tq ? fit : a->Tq;
  a->tiles_p = (int)ceil_div(tok_p, a->box_p);
  a->tiles_s = (int)ceil_div(a->Tq, a->box_s);
  a->bin_p = (int)ceil_div(a->G, kMaxBins);
  a->bin_s = (int)ceil_div(a->B, kMaxBins);
  a->bins_p = a->P_max > 0 ? (int)ceil_div(a->G, a->bin_p) : 0;
  a->bins_s = a->S_max > 0 ? (int)ceil_div(a->B, a->bin_s) : 0;
  const long long units_p = a->P_max > 0 ? (long long)a->G * a->Hkv * a->tiles_p : 0;
  const long long units_s = a->S_max > 0 ? (long long)a->B * a->Hkv * a->tiles_s : 0;
  // the cost of everything and its product with the CTAs' number fit an int
  const long long most = 0x7fffffffLL / 2;
  if (units_p > most || units_s > most) return false;
  const long long kt_p = ceil_div(a->P_max, kKeys), kt_s = ceil_div(a->S_max, kKeys);
  a->fixed_p = unit_fixed(a->box_p * R);
  a->fixed_s = unit_fixed(a->box_s * R);
  const long long cost = units_p * (kt_p + a->fixed_p) + units_s * (kt_s + a->fixed_s);
  if (cost > most) return false;
  // About how many pieces a row has with full caches: an estimate for the choice of
  // the join alone, which takes any number.  Shorter lengths make the shares smaller
  // and may cut a row more often than this, or less.
  const long long least = (a->fixed_p > a->fixed_s ? a->fixed_p : a->fixed_s) + 1;
  const long long share = ceil_div(cost, a->ctas) > least ? ceil_div(cost, a->ctas) : least;
  a->most_pieces = (int)(kt_p / share + kt_s / share + 2);
  auto align = [](size_t b) { return (b + kWsAlign - 1) & ~(kWsAlign - 1); };
  const size_t rows_p = units_p > 0 ? (size_t)(units_p + a->ctas) * (a->box_p * R) : 0;  // a slot per unit and CTA
  const size_t rows_s = units_s > 0 ? (size_t)(units_s + a->ctas) * (a->box_s * R) : 0;
  a->off_os = rows_p * kD * 4;
  a->off_lp = a->off_os + rows_s * kD * 4;
  a->off_ls = a->off_lp + align(rows_p * 4);
  a->off_pieces = a->off_ls + align(rows_s * 4);
  *bytes = a->off_pieces + align((size_t)(units_p + units_s) * 8) + kWsAlign - 16;
  return true;
}

bool launch_prefix_attn(const PrefixAttnArgs& args, const void* q, long long ldq, const void* kp, const void* vp,
                        long long ldp, long long lsp, const void* ks, const void* vs, long long lds, long long lss,
                        void* workspace, cudaStream_t st) {
  PrefixAttnArgs a = args;
  char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(workspace) + kWsAlign - 1) & ~uintptr_t(kWsAlign - 1));
  a.part_op = reinterpret_cast<float*>(ws);
  a.part_os = reinterpret_cast<float*>(ws + a.off_os);
  a.part_lp = reinterpret_cast<float*>(ws + a.off_lp);
  a.part_ls = reinterpret_cast<float*>(ws + a.off_ls);
  a.pieces = reinterpret_cast<int2*>(ws + a.off_pieces);
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
    if (launch_pdl(k_prefix_attn, dim3(a.ctas), dim3(kThreads), SMEM_BYTES, st, 1, m[0], m[1], m[2], m[3], m[4], m[5], a) !=
        cudaSuccess)
      return false;
  }
  const long long rows = (long long)tokens * a.H;
  LaunchScope scope_(KK_PREFIX_ATTN, st);
  // A row's pieces are joined by one warp, by four where rows are few or should have
  // many pieces and 148 SMs hold all rows' CTAs at once, by sixteen where both.
  // Measured in us for the whole call, (rows, pieces estimated), one against four
  // warps: (192, 5) 16.2, 15.5; (384, 7) 19.0, 18.5; (512, 6) 13.7, 14.4; (1152, 4)
  // 31.9, 33.2; (768, 9) 69.6, 69.1; (768, 12) 18.4, 18.7; (1280, 20) 29.4, 28.1;
  // (2048, 6) 27.0, 27.7; (3600, 9) 27.8, 32.1.
  // Four against sixteen: (12, 171) 16.1, 13.6; (48, 4) 10.7, 11.4.
  // Where lengths are far from the caches' the estimate may choose wrongly: 768 rows
  // over 512 + 64 keys in caches of 32768 + 1024 take four, 18.6 for 17.4; 500 rows
  // of which one has 12800 keys and the others none take one, 18.2 for 15.0.
  if (rows <= 148 && a.most_pieces > 32) return launch_pdl(k_prefix_combine<16>, dim3((unsigned)rows), dim3(512), 0, st, 1, a) == cudaSuccess;
  if (rows <= 3 * 148 || (a.most_pieces > 8 && rows <= 16 * 148)) return launch_pdl(k_prefix_combine<4>, dim3((unsigned)rows), dim3(128), 0, st, 1, a) == cudaSuccess;
  return launch_pdl(k_prefix_combine<1>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, st, 1, a) == cudaSuccess;
}

}  // namespace nc
