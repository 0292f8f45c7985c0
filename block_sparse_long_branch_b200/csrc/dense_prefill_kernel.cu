// dense_prefill_kernel.cu -- causal attention of new tokens over all of their keys.
//
//   out[t][h] = sum_{s <= p(t)} softmax_s(scale * <q[t][h], k[s][g]>) v[s][g]
//
// for packed prompts (keys and values beside the queries) and for chunks of new
// tokens over a paged cache; head h belongs to group g = h / (H/G).
//
// One work unit is 2 x 128 rows (a row = one head of one token: the H/G heads of
// group g of TT = floor(128 / (H/G)) consecutive tokens, twice) against a range of
// 128-key tiles.  Packing a group's heads into the rows means a key tile is loaded
// once for all of them, and a few tokens fill a tile.  One pass over the keys with
// the running maximum and sum of the softmax:
//   S = Q K_j^T          tcgen05.mma M=128 N=128 K=d       (TMEM, fp32)
//   m' = max(m, rowmax)  l = l 2^(m-m') + sum P,  P = 2^(scale log2e S - m')
//   O = O 2^(m-m') + P V_j   tcgen05.mma M=128 N=d K=128, P (bf16) from TMEM
// The factor 2^(m-m') is applied only where the maximum grew by more than 2^8
// since the last time: with any stale m the quotient O/l is the same, and P
// stays below 2^8, far inside fp32 and bf16.
//
// Precision: S, m, l and O are fp32.  P is rounded to bf16, since V is bf16 in
// the caller's cache and the two operands of one MMA share a type; each weight is
// then off by at most 2^-8 of itself, beside the 2^-8 of the bf16 output.
//
// Rows that a mask hides.  A hidden key has P = 0 exactly, but 0 * NaN = NaN on the
// tensor cores, so in the tiles that some row of the unit does not see whole
// (the last ones) V is first cleaned: rows past the sequence's end are zeroed,
// and infinities or NaNs are replaced by zero and added back, by the epilogue,
// to those rows that do see their key.
//
// Warp roles (384 threads, one CTA per SM, persistent over the units):
//   WG0, WG1  softmax of row tile 0 / 1, one thread per row; the rescaling of
//             O; the cleaning of V; the final O / l;
//   WG2       warp 8 loads Q and K, warp 11 V (TMA; with pages of 16 tokens a
//             tile of 128 keys is 16 copies), warp 9 issues S, warp 10 issues PV.
// TMEM (512 columns): one S buffer for both row tiles (0-127), P0, P1 (64 columns
// each) and O0, O1.  A softmax thread copies its row of S into registers at once,
// so the S buffer is free again for the other tile, whose next S is ready when its
// warpgroup comes for it.  With an S of its own per tile and P over it, a tile's
// next S had to wait for its product: 1400 of 3350 cycles per 128 keys.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "early.cuh"
#include "kernels.h"
#include "ring.h"
#include "sm100.cuh"
#include "tmap.h"

namespace msa {
namespace {

constexpr int kThreads = 384;
constexpr int kLoadWarp = 8, kSWarp = 9, kPVWarp = 10, kLoadVWarp = 11;
constexpr uint32_t kRegSoftmax = 208, kRegOther = 88;
constexpr int kLaunchRegs = 168;  // 2*128*208 + 128*88 = 384*168
constexpr int kRows = 128, kKeys = 128;
constexpr uint32_t kColS = 0, kColP = 128, kColO = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.f;  // log2 of the growth of the maximum left unapplied
constexpr int kFlagSlots = 8;
constexpr int kTurns = 8;
constexpr int kUnitTurns = 4;
constexpr int kDirectUnits = 160;  // as many as CTAs
constexpr int kBoxRows = 128;  // of a TMA copy, at most (smaller boxes gained nothing)

template <int D>
struct PrefillCfg {
  static constexpr int kChunks = D / 64;           // 128-byte column chunks
  static constexpr int kTileBytes = kRows * D * 2;  // Q, K and V tiles alike
  // Rings of K and of V tiles, each filled and emptied in its own order: what
  // 224 KiB hold beside the two Q tiles.  A tile takes some 2000 cycles to come
  // from L2.
  static constexpr int kKSlots = D == 128 ? 3 : 5, kVSlots = D == 128 ? 2 : 5;
  static constexpr int kOffK = 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kKSlots * kTileBytes;
  static constexpr int kSmem = kOffV + kVSlots * kTileBytes + 1024;
};

struct PrefillArgs {
  int32_t H, G, HG, TT;
  float scale_log2;
  const DenseUnit* units;  // device plan: the units (each for all groups) and their number
  const int32_t* n_units;
  int32_t* next_unit;      // units taken beyond the first of every CTA
  // paged keys and values; page_size 0: packed rows
  const int32_t* block_table;
  int32_t table_stride, page_size, num_pages;
  int32_t box_rows;     // of a TMA copy of keys or values
  int64_t page_stride;  // elements
  const __nv_bfloat16* v;
  __nv_bfloat16* out;
  float* part_o;     // [slot][256][D]
  float2* part_ml;   // [slot][256] (log2-domain maximum, sum)
  // Whether out and part_o are 32-byte aligned; callers promise 16.  Stores of 16 bytes
  // throughout cost 6 % of a small prompt (one of 4K, 4 heads: 30.8 -> 32.6 us), 1 % of
  // packed ones.
  bool out32, part32;
  int32_t clear_err;
  uint32_t* err;
};

// The units of a small batch whose lengths the host knows travel as a kernel
// parameter: no planning kernel in front (prefill of 128 tokens, replayed: 13.0 -> 9.3 us).
constexpr int kHostUnits = 128;
enum PlanMode { kPlanned, kHost, kDirect };
struct HostUnits {
  int32_t n;
  DenseUnit u[kHostUnits];
};
struct HostSplits {
  int32_t n;
  DenseSplit s[kHostUnits / 2];
};
struct NoUnits {};
// Paged batches of few units: every CTA works out its own from the lengths on the
// device (direct_plan), with no planning kernel in front.
struct DirectArgs {
  const int64_t* cu;
  const int32_t* seq_lens;
  int32_t B, T, table_rows, can_split;
  int32_t max_units;  // as many as T tokens of B sequences make
};
template <int MODE>
using ModeArgs = std::conditional_t<MODE == kHost, HostUnits,
                                    std::conditional_t<MODE == kDirect, DirectArgs, NoUnits>>;

struct Unit {
  DenseUnit d;
  int g;
  int nt;       // key tiles of the unit
  int c0, c1;   // of these, taken by row tile 0 / 1
  // A unit of one row tile is taken by both softmax warpgroups: "tile" i holds
  // the same rows and takes every other key tile, from i on.
  bool dual;
};

struct DirectUnit {
  DenseUnit d;  // slot: of this group
  int g;        // -1: none
};
// Where a CTA is in the line of all units (see direct_plan): unit `off` of sequence
// `seq` and group `g`, which begins at `start`.
struct LineState {
  long long start;
  int share;  // 0: no line
  int seq, off, g;
};

// Unit x of the line of all units (groups innermost, longest first).
template <int MODE>
__device__ __forceinline__ void read_unit(const PrefillArgs& a, const ModeArgs<MODE>& hu,
                                          const DirectUnit* own, unsigned x, Unit& u) {
  if constexpr (MODE == kDirect) {
    const volatile int* p = reinterpret_cast<const volatile int*>(own);
    u.d.tok0 = p[0], u.d.ntok = p[1], u.d.pos0 = p[2], u.d.seq = p[3];
    u.d.kv0 = p[4], u.d.kv1 = p[5], u.d.slot = p[6], u.d.row0 = p[7];
    u.g = p[8];
  } else {
    const unsigned i = x / (unsigned)a.G;
    u.g = (int)(x - i * (unsigned)a.G);
    if constexpr (MODE == kHost) {
      u.d = hu.u[i];
    } else {
      const int4* p = reinterpret_cast<const int4*>(a.units + i);
      const int4 x0 = __ldcg(p), x1 = __ldcg(p + 1);
      u.d.tok0 = x0.x, u.d.ntok = x0.y, u.d.pos0 = x0.z, u.d.seq = x0.w;
      u.d.kv0 = x1.x, u.d.kv1 = x1.y, u.d.slot = x1.z, u.d.row0 = x1.w;
    }
    if (u.d.slot >= 0) u.d.slot += u.g;
  }
  u.nt = u.d.kv1 - u.d.kv0;
  u.dual = u.d.ntok <= a.TT;
  if (u.dual) {
    u.c0 = (u.nt + 1) / 2;
    u.c1 = u.nt / 2;
    return;
  }
  const int last0 = u.d.pos0 + min(u.d.ntok, a.TT) - 1;  // last position of row tile 0
  u.c0 = max(0, min(u.d.kv1, last0 / kKeys + 1) - u.d.kv0);
  u.c1 = u.d.ntok > a.TT ? u.nt : 0;
}

// first key tile of the unit that some row does not see whole
__device__ __forceinline__ int first_partial(const Unit& u) { return (u.d.pos0 + 1) / kKeys; }

// V element (key s of the unit's sequence) straight from memory; the rare path of the epilogue
__device__ __forceinline__ const __nv_bfloat16* v_row(const PrefillArgs& a, const Unit& u, int s,
                                                      int D) {
  if (a.page_size == 0)
    return a.v + (((int64_t)u.d.row0 + s) * a.G + u.g) * D;
  const int pg = __ldg(a.block_table + (int64_t)u.d.seq * a.table_stride + s / a.page_size);
  if (pg < 0 || pg >= a.num_pages) return nullptr;
  return a.v + (int64_t)pg * a.page_stride + ((int64_t)(s % a.page_size) * a.G + u.g) * D;
}

constexpr int kMinPart = 4;  // key tiles worth a part: its overhead is about three

// First key tile of part k of `parts` of a unit of nt key tiles.  The last part has
// two tiles at least, so that row tile 0, which may end a key tile before row tile
// 1, has keys in every part.
__host__ __device__ __forceinline__ int part_begin(int k, int parts, int len, int nt) {
  if (k >= parts) return nt;
  return k > 0 && k * len > nt - 2 ? nt - 2 : k * len;
}

constexpr int kPartCost = 3;  // a unit's or a part's cost beside its key tiles, in key tiles
constexpr int kJoinCost = 7;  // partial results stored, read and joined, likewise: units of 27
                              // key tiles split to take 26 took 86 us instead of 66

// new tokens [lo, lo+n) of sequence b, the first at position pos; n = 0: none, or invalid
__device__ __forceinline__ void direct_seq(const DirectArgs& p, int b, uint32_t* err, int64_t& lo,
                                           int& n, int& pos) {
  lo = __ldg(p.cu + b);
  const int64_t hi = __ldg(p.cu + b + 1);
  const int64_t first = __ldg(p.cu), last = __ldg(p.cu + p.B);
  const int L = __ldg(p.seq_lens + b);
  n = (int)(hi - lo);
  pos = L - n;
  if (lo < 0 || lo < first || hi < lo || hi > p.T || hi > last ||
      (n > 0 && (pos < 0 || L > p.table_rows))) {
    record_error(err, kDevBadIndex);
    n = 0;
  }
}
// key tiles of the unit `off` of a sequence, and its weight: a unit of one row tile
// is taken by both softmax warpgroups, half as long
__device__ __forceinline__ int direct_tiles(int n, int pos, int off, int TT, int& w) {
  const int nt = (pos + min(n, off + 2 * TT) - 1) / kKeys + 1;
  w = n - off <= TT ? (nt + 1) / 2 : nt;
  return nt;
}

// The plan of units that fit the GPU at once, by one warp, up to 32 sequences: either
//  * as dense_plan_kernel does, all in parts of at most `part`, by weight, one a CTA; or
//  * the units of all groups as one line, cut into equal shares, one a CTA, which
//    leaves no CTA idle (100 units of one length do not make 148 parts): where that
//    shortens the longest CTA's work by an eighth.  It costs the units of a group
//    their common pace through the keys, which then come from memory several times.
//    Parts -> line, whole calls: 112 units over 0.1K to 50K (16 heads in one group)
//    353 -> 220 us, 52 over 30K (32 heads in 4) 238 -> 222, 88 (64 in 8) 426 -> 397;
//    104 (64 in 8) lose a little, 454 -> 471, and over 10K keys 164 -> 175.  More
//    units than CTAs lost about a third, their keys read eleven times from memory.
struct PlanUnit {
  int seq, off;  // sequence, first of its new tokens
  int nt, w;     // key tiles, weight
  int pre;       // the weights, each with kPartCost, of the units before
};
struct DirectPlan {
  int64_t lo;  // lane b: sequence b
  int n, pos;
  int total;   // units, in `u`
  int part;
  int share;   // of the line; 0: parts
  PlanUnit* u;
};
__device__ __forceinline__ void direct_plan(const DirectArgs& p, int G, int TT, int ctas,
                                            uint32_t* err, PlanUnit* tab, DirectPlan& d) {
  const int lane = lane_id(), U = 2 * TT;
  d.u = tab;
  d.lo = 0, d.n = 0, d.pos = 0;
  if (lane < p.B) direct_seq(p, lane, err, d.lo, d.n, d.pos);
  const int units = (d.n + U - 1) / U;
  int incl = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  // offsets that overlap could make more units than the host counted
  d.total = min(__shfl_sync(0xffffffffu, incl, 31), p.max_units);
  int longest = 0, line = 0;
#pragma unroll 1  // code that runs once: its size is its time
  for (int k = 0; k < d.total; k += 32) {
    const int x = k + lane;
    int s = 0;
#pragma unroll 1
    for (int b = 0; b < p.B; ++b) s += __shfl_sync(0xffffffffu, incl, b) <= x;
    s = min(s, 31);
    PlanUnit u;
    u.seq = s;
    u.off = (x - (__shfl_sync(0xffffffffu, incl, s) - __shfl_sync(0xffffffffu, units, s))) * U;
    const int len = __shfl_sync(0xffffffffu, d.n, s), p0 = __shfl_sync(0xffffffffu, d.pos, s);
    int c = 0;
    if (x < d.total) {
      u.nt = direct_tiles(len, p0, u.off, TT, u.w);
      longest = max(longest, u.w);
      c = u.w + kPartCost;
    }
    int y = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    u.pre = line + y - c;
    line += __shfl_sync(0xffffffffu, y, 31);
    if (x < d.total) tab[x] = u;
  }
  __syncwarp();
  longest = __reduce_max_sync(0xffffffffu, longest);
  d.part = 1 << 30;
  d.share = 0;
  if (!p.can_split) return;
  const int sum = line - kPartCost * d.total;
  // the least that makes no more parts than CTAs (their number falls with it): mostly
  // near the even share, so in growing steps from there, then by halves
  int c0 = max(kMinPart, (sum * G + ctas - 1) / ctas), c1 = longest, step = 1;
#pragma unroll 1
  while (c0 < c1) {
    const int c = step > 0 && step < c1 - c0 ? c0 + step - 1 : (c0 + c1) / 2;
    int m = 0;
#pragma unroll 1
    for (int x = lane; x < d.total; x += 32) m += ((unsigned)tab[x].w + c - 1) / (unsigned)c;
    if (__reduce_add_sync(0xffffffffu, m) * G <= ctas)
      c1 = c, step = 0;
    else
      c0 = c + 1, step *= 2;
  }
  if (c1 + kJoinCost < longest) d.part = c1;
  const int share = max((line * G + ctas - 1) / ctas, kMinPart + kPartCost);
  const int parted = d.part < longest ? d.part + kJoinCost : longest;
  if ((share + kJoinCost) * 8ll < parted * 7ll) d.share = share;
}
// The units of the plan in parts: `f` is called by one lane for each with its first
// packed row, tokens, first position, sequence, key tiles, key tiles per part, parts,
// and the parts of the units before it.
template <typename F>
__device__ __forceinline__ void direct_parts(const DirectPlan& d, int TT, F&& f) {
  const int lane = lane_id(), U = 2 * TT;
  int pre = 0;
#pragma unroll 1
  for (int k = 0; k < d.total; k += 32) {
    const bool mine = k + lane < d.total;
    PlanUnit u = {};
    int parts = 0, len = 1;
    if (mine) {
      u = d.u[k + lane];
      const int q = u.w > d.part ? (u.w + d.part - 1) / d.part : 1;
      len = (u.nt + q - 1) / q;
      parts = (u.nt + len - 1) / len;
    }
    int x = parts;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int64_t a = __shfl_sync(0xffffffffu, (long long)d.lo, u.seq);
    const int p0 = __shfl_sync(0xffffffffu, d.pos, u.seq), ln = __shfl_sync(0xffffffffu, d.n, u.seq);
    if (mine) f(a + u.off, min(U, ln - u.off), p0 + u.off, u.seq, u.nt, len, parts, pre + x - parts);
    pre += __shfl_sync(0xffffffffu, x, 31);
  }
}
// First key tile behind line offset x of a unit that takes `len` of the line: what
// would be a crumb of less than three tiles goes with the rest (the last part has
// two tiles at least: see part_begin).
__device__ __forceinline__ int line_cut(long long x, int len, int nt) {
  if (x <= 0) return 0;
  if (x >= len) return nt;
  const long long y = x * nt;
  const int t = (int)((y >> 32) == 0 ? (unsigned)y / (unsigned)len : y / len);
  return t < 3 ? 0 : t > nt - 3 ? nt : t;
}
// The next part of this CTA's share of the line; g = -1: none.  A whole warp.  Partial
// results: slot 2c of CTA c holds the unit that began in an earlier share, 2c + 1 the
// one that goes on in a later.
__device__ __forceinline__ void line_next(const DirectArgs& p, int G, int TT,
                                          volatile LineState& st, DirectUnit& out) {
  const int share = st.share;
  const long long lo = (long long)blockIdx.x * share, hi = lo + share;
  int s = st.seq, off = st.off, g = st.g;
  long long start = st.start;
  int64_t a = 0;
  int n = 0, pos = 0;
  out.g = -1;
  if (s < p.B) direct_seq(p, s, nullptr, a, n, pos);
  while (s < p.B && start < hi && out.g < 0) {
    if (off >= n) {
      off = 0;
      if (++s < p.B) direct_seq(p, s, nullptr, a, n, pos);
      continue;
    }
    int w;
    const int nt = direct_tiles(n, pos, off, TT, w), len = w + kPartCost;
    const int kv0 = line_cut(lo - start, len, nt), kv1 = line_cut(hi - start, len, nt);
    if (kv0 < kv1) {
      out.d = DenseUnit{(int)a + off, min(2 * TT, n - off), pos + off, s, kv0, kv1, -1, 0};
      if (kv0 > 0)
        out.d.slot = 2 * blockIdx.x;
      else if (kv1 < nt)
        out.d.slot = 2 * blockIdx.x + 1;
      out.g = g;
    }
    start += len;
    if (++g == G) g = 0, off += 2 * TT;
  }
  __syncwarp();
  if (lane_id() == 0) {
    st.start = start;
    st.seq = s, st.off = off, st.g = g;
  }
  __syncwarp();
}

template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    dense_prefill_kernel(const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const PrefillArgs a,
                         const __grid_constant__ ModeArgs<MODE> hu) {
  using Cfg = PrefillCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + Cfg::kOffK;
  uint8_t* sV = smem + Cfg::kOffV;
  constexpr uint32_t KS = Cfg::kKSlots, VS = Cfg::kVSlots;
  __shared__ uint64_t bar_q_full[2], bar_q_empty[2];
  // A wait for a phase's parity is right only while the phase before it is known
  // to be complete.  So every barrier is waited on by one warp (or warpgroup) use
  // by use, or (bar_spec, bar_clean) in turns that the steps around them order.
  __shared__ uint64_t bar_k_full[KS], bar_k_empty[KS], bar_v_empty[VS];
  // V tiles that every row sees whole, in turn; and the others, "special" ones:
  // loaded, and cleaned
  __shared__ uint64_t bar_v_full[VS], bar_spec[VS], bar_clean[kTurns];
  __shared__ uint64_t bar_s_full[2], bar_s_empty, bar_p_full[2], bar_pv_done[2];
  __shared__ uint64_t bar_drain[2];
  __shared__ uint64_t bar_half_done, bar_half_read;  // dual units: tile 1's result, and its reading
  __shared__ float half_m[kRows], half_l[kRows];
  __shared__ DirectUnit own_s[MODE == kDirect ? kUnitTurns : 1];
  __shared__ LineState line_s;
  // the CTA's units after its first: handed out by warp 8
  __shared__ uint64_t bar_u_full[kUnitTurns], bar_u_empty[kUnitTurns];
  __shared__ unsigned unit_s[kUnitTurns];
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;
  __shared__ int odd_v[kFlagSlots];  // an infinity or NaN was taken out of the unit's V

  const int warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    abort_s = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_q_full[i], 1);
      mbar_init(&bar_q_empty[i], 1);
      mbar_init(&bar_s_full[i], 1);
      mbar_init(&bar_p_full[i], 128);
      mbar_init(&bar_pv_done[i], 1);
    }
    for (uint32_t i = 0; i < KS; ++i) {
      mbar_init(&bar_k_full[i], 1);
      mbar_init(&bar_k_empty[i], 1);
    }
    for (uint32_t i = 0; i < VS; ++i) {
      mbar_init(&bar_v_full[i], 1);
      mbar_init(&bar_spec[i], 1);
      mbar_init(&bar_v_empty[i], 1);
    }
    for (int i = 0; i < kTurns; ++i) mbar_init(&bar_clean[i], 128);
    for (int i = 0; i < kUnitTurns; ++i) {
      mbar_init(&bar_u_full[i], 1);
      mbar_init(&bar_u_empty[i], kThreads / 32 - 1);
    }
    mbar_init(&bar_s_empty, 128);
    mbar_init(&bar_drain[0], 1);
    mbar_init(&bar_drain[1], 1);
    mbar_init(&bar_half_done, 128);
    mbar_init(&bar_half_read, 128);
    for (int i = 0; i < kFlagSlots; ++i) odd_v[i] = 0;
    fence_mbar_init();
    // nothing else clears it without a plan, and no wait runs out before this
    if (MODE == kHost && blockIdx.x == 0 && a.clear_err) *a.err = 0;
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
    own_s[0].g = -1;
    line_s.share = 0;
    line_s.seq = 1 << 30;  // of a share behind the line's end
    line_s.off = line_s.g = 0;
    line_s.start = 0;
  }
  if constexpr (MODE == kDirect) {
    if (warp == 1) {
      __syncwarp();
      // the units in what will be a Q tile
      PlanUnit* tab = reinterpret_cast<PlanUnit*>(sQ);
      static_assert(kDirectUnits * sizeof(PlanUnit) <= Cfg::kTileBytes, "the plan's units");
      DirectPlan d;
      direct_plan(hu, a.G, a.TT, gridDim.x, a.err, tab, d);
      if (d.share == 0) {
        const int i = blockIdx.x / a.G;
        direct_parts(d, a.TT, [&](int64_t tok0, int ntok, int pos0, int seq, int nt, int len,
                                  int parts, int pre) {
          if (i < pre || i >= pre + parts) return;
          const int k = i - pre, g = blockIdx.x - i * a.G;
          own_s[0].d = DenseUnit{(int)tok0, ntok, pos0, seq, part_begin(k, parts, len, nt),
                                 part_begin(k + 1, parts, len, nt), parts > 1 ? i * a.G + g : -1, 0};
          own_s[0].g = g;
        });
      } else {
        // the unit that holds this share's first position
        const long long lo = (long long)blockIdx.x * d.share;
#pragma unroll 1
        for (int x = lane; x < d.total; x += 32) {
          const int len = tab[x].w + kPartCost;
          const long long from = (long long)tab[x].pre * a.G;
          if (lo < from || lo >= from + (long long)len * a.G) continue;
          line_s.seq = tab[x].seq;
          line_s.off = tab[x].off;
          line_s.g = (int)((unsigned)(lo - from) / (unsigned)len);
          line_s.start = from + (long long)line_s.g * len;
        }
        if (lane == 0) line_s.share = d.share;
      }
      fence_async_smem();  // the Q tile's memory goes to TMA
    }
  }
  if (warp == 0) {
    tmem_alloc(&tmem_base_s, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  volatile int* abort_flag = &abort_s;
  pdl_launch_dependents();
  int total;
  if constexpr (MODE == kHost) {
    total = hu.n * a.G;
  } else if constexpr (MODE == kDirect) {
    total = 0;  // see next_unit
  } else {
    pdl_wait();  // for the units
    total = __ldcg(a.n_units) * a.G;
  }

  // The warp's r-th unit; false after the last.  A CTA starts with its own number
  // and takes the next one of the line whenever it has loaded a unit: longest
  // first, so the CTAs end nearly together whatever the lengths (chunks of four
  // caches of 1K to 30K: 943 -> 866 us against a fixed order).
  // With kDirect warp 8 hands out the CTA's own unit, or the parts of its share.
  auto next_unit = [&](int r, Unit& u) {
    constexpr bool kOwn = MODE == kDirect;
    unsigned x = blockIdx.x;
    const DirectUnit* own = own_s;
    const int q = kOwn ? r : r - 1;
    const int turn = q % kUnitTurns;
    if (kOwn || r > 0) {
      if (!kOwn && total <= (int)gridDim.x) return false;
      const uint32_t phase = (q / kUnitTurns) & 1;
      if (warp == kLoadWarp) {
        if (!__all_sync(0xffffffffu, mbar_wait(&bar_u_empty[turn], phase ^ 1, abort_flag, a.err,
                                               kDevTimeoutConsumer)))
          return false;
        if constexpr (kOwn) {
          if (line_s.share > 0) {
            DirectUnit next;
            line_next(hu, a.G, a.TT, line_s, next);
            if (lane == 0) own_s[turn] = next;
          } else if (r > 0 && lane == 0) {
            own_s[turn].g = -1;
          }
          if (lane == 0) mbar_arrive(&bar_u_full[turn]);
          __syncwarp();
        } else {
          if (lane == 0) {
            x = atomicAdd(a.next_unit, 1) + gridDim.x;
            unit_s[turn] = x;
            mbar_arrive(&bar_u_full[turn]);
          }
          x = __shfl_sync(0xffffffffu, x, 0);
        }
      } else {
        if (!__all_sync(0xffffffffu, mbar_wait(&bar_u_full[turn], phase, abort_flag, a.err,
                                               kDevTimeoutLoad)))
          return false;
        if constexpr (!kOwn) x = *reinterpret_cast<volatile unsigned*>(&unit_s[turn]);
      }
      if constexpr (kOwn) own = own_s + turn;
    }
    const bool any = kOwn || x < (unsigned)total;
    if (any) read_unit<MODE>(a, hu, own, x, u);
    if (kOwn || r > 0) {  // read: the turn is free again
      __syncwarp();
      if (warp != kLoadWarp && lane == 0) mbar_arrive(&bar_u_empty[turn]);
    }
    return any && (!kOwn || u.g >= 0);
  };

  if (warp >= 8) {
    regs_decrease<kRegOther>();
    if (warp == kLoadWarp || warp == kLoadVWarp) {
      // ---------------- TMA loads: Q and K, or V ----------------
      const bool is_v = warp == kLoadVWarp;
      const CUtensorMap* map = is_v ? &map_v : &map_k;
      const uint32_t slots = is_v ? VS : KS;
      uint64_t* empty = is_v ? bar_v_empty : bar_k_empty;
      uint8_t* ring = is_v ? sV : sK;
      uint32_t slot = 0, phase = 0;       // of the next tile
      uint32_t regular = 0, special = 0;  // V tiles of both kinds so far
      uint32_t qn[2] = {0, 0};      // Q tiles loaded so far
      bool ok = true;
      const int box_rows = a.box_rows, boxes = kKeys / box_rows;  // a lane per box of a tile
      auto load_q = [&](const Unit& u, int i) {
        if (!ok || is_v || (i == 0 ? u.c0 : u.c1) == 0) return;
        ok = __all_sync(0xffffffffu, mbar_wait(&bar_q_empty[i], (qn[i] & 1) ^ 1, abort_flag, a.err,
                                               kDevTimeoutMma));
        if (ok && elect_one()) {
          mbar_arrive_expect_tx(&bar_q_full[i], (uint32_t)(a.TT * a.HG * D * 2));
#pragma unroll
          for (int c = 0; c < Cfg::kChunks; ++c)
            tma_load_4d(sQ + i * Cfg::kTileBytes + c * kRows * 128, &map_q, &bar_q_full[i], 0,
                        u.g * a.HG, c, u.d.tok0 + (u.dual ? 0 : i * a.TT));
        }
        __syncwarp();
        if (ok) ++qn[i];
      };
      for (int r = 0; ok; ++r) {
        Unit u;
        if (!next_unit(r, u)) break;
        const int keys_end = u.d.pos0 + u.d.ntok;
        const int part0 = first_partial(u) - u.d.kv0;
        // lane i: page of box i of a key tile (0: none, or packed rows)
        auto page_of = [&](int j) {
          const int key = (u.d.kv0 + j) * kKeys + lane * box_rows;
          if (a.page_size == 0 || lane >= boxes || key >= keys_end || j >= u.nt) return 0;
          return __ldg(a.block_table + (int64_t)u.d.seq * a.table_stride + key / a.page_size);
        };
        int page_next = page_of(0);
        for (int j = 0; j < u.nt && ok; ++j) {
          const int key0 = (u.d.kv0 + j) * kKeys;
          int page = page_next;
          page_next = page_of(j + 1);  // its latency behind this tile's waits
          // boxes past the sequence's end are not read
          const int left = (keys_end - key0 + box_rows - 1) / box_rows;
          const int nbox = left < boxes ? left : boxes;
          int32_t row = u.d.row0 + key0 + lane * box_rows;
          if (a.page_size != 0) {
            row = (key0 + lane * box_rows) % a.page_size;
            if (lane < nbox && (page < 0 || page >= a.num_pages)) {
              record_error(a.err, kDevBadIndex);
              page = a.num_pages;  // outside the tensor: reads zeros
            }
          }
          if (j == 0) load_q(u, 0);
          if (!ok) break;
          uint64_t* full;
          if (!is_v)
            full = &bar_k_full[slot];
          else if (j < part0)
            full = &bar_v_full[regular++ % VS];
          else
            full = &bar_spec[special++ % VS];
          ok = __all_sync(0xffffffffu,
                          mbar_wait(&empty[slot], phase ^ 1, abort_flag, a.err, kDevTimeoutMma));
          if (!ok) {
            if (is_v) --(j < part0 ? regular : special);  // not issued
            break;
          }
          if (elect_one()) mbar_arrive_expect_tx(full, (uint32_t)(nbox * box_rows * D * 2));
          __syncwarp();
          // One copy after the other with operands known to be the same in the
          // whole warp; a lane each, they are issued in a loop over the lanes.
          uint8_t* dst = ring + slot * Cfg::kTileBytes;
          for (int b = 0; b < nbox; ++b, dst += box_rows * 128) {
            const int row_b = __shfl_sync(0xffffffffu, row, b);
            const int page_b = __shfl_sync(0xffffffffu, page, b);
            if (elect_one()) {
#pragma unroll
              for (int c = 0; c < Cfg::kChunks; ++c)
                tma_load_5d(dst + c * kKeys * 128, map, full, 0, row_b, c, u.g, page_b);
            }
          }
          __syncwarp();
          if (++slot == slots) slot = 0, phase ^= 1;
          if (j == 0) load_q(u, 1);
        }
      }
      if (lane == 0 && *abort_flag) {
        // The copies in flight must land before the CTA's shared memory goes.  (Where
        // the flag comes up after this, a wait of 2 s has run out behind them.)
        volatile int no_abort = 0;
        for (int i = 0; i < 2; ++i)
          if (qn[i]) mbar_wait(&bar_q_full[i], (qn[i] - 1) & 1, &no_abort, nullptr, 0);
#pragma unroll 1
        for (uint32_t i = 0; i < slots; ++i) {
          if (is_v) {
            // the i-th from the end of both kinds, see ring_parity
            const uint32_t r = regular + VS - 1 - i, s = special + VS - 1 - i;
            if (r >= VS) mbar_wait(&bar_v_full[r % VS], ring_parity(r, VS), &no_abort, nullptr, 0);
            if (s >= VS) mbar_wait(&bar_spec[s % VS], ring_parity(s, VS), &no_abort, nullptr, 0);
          } else {
            mbar_wait(&bar_k_full[i], ring_last_parity(i, slot, phase), &no_abort, nullptr, 0);
          }
        }
      }
    } else if (warp == kSWarp || warp == kPVWarp) {
      // ---------------- MMA issuers ----------------
      // The whole warp walks the units, so that the operands of the MMAs are
      // warp-uniform (uniform registers); one lane issues.  With the walk in
      // one lane alone a batch of eight MMAs took 870 cycles to issue.
      constexpr uint32_t kTile16 = Cfg::kTileBytes / 16;  // descriptor units
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t code) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.err, code));
        return ok;
      };
      if (warp == kSWarp) {
        // S = Q_i K^T of both row tiles in turn, into the one S buffer as soon as
        // the softmax has copied the S before into its registers
        constexpr uint32_t idesc_s = idesc_bf16(kRows, kKeys, false, false);
        const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t k_desc = smem_desc_sw128(smem_u32(sK), 16, 1024);
        uint32_t qn[2] = {0, 0}, sn = 0;
        uint32_t slot = 0, phase = 0;  // of the K tile
        for (int r = 0; ok; ++r) {
          Unit u;
          if (!next_unit(r, u)) break;
          // broadcasts: known to be the same in every lane
          const int cnt[2] = {__shfl_sync(0xffffffffu, u.c0, 0), __shfl_sync(0xffffffffu, u.c1, 0)};
          const bool dual = __shfl_sync(0xffffffffu, (int)u.dual, 0) != 0;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (ok && cnt[i] > 0) wait(&bar_q_full[i], qn[i]++ & 1, kDevTimeoutLoad);
          const int most = max(cnt[0], cnt[1]);
          for (int j = 0; j < most && ok; ++j) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!ok || j >= cnt[i]) continue;
              if (dual || i == (j < cnt[0] ? 0 : 1)) {
                if (!wait(&bar_k_full[slot], phase, kDevTimeoutLoad)) break;
              }
              if (!wait(&bar_s_empty, (sn & 1) ^ 1, kDevTimeoutConsumer)) break;
              ++sn;
              tc_fence_after();
              if (elect_one()) {
                const uint64_t qd = q_desc + (uint32_t)i * kTile16, kd = k_desc + slot * kTile16;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint32_t off = ((kk >> 2) * kRows * 128 + (kk & 3) * 32) / 16;
                  umma_bf16(tmem + kColS, qd + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
                }
                umma_commit(&bar_s_full[i]);
                if (j == cnt[i] - 1) umma_commit(&bar_q_empty[i]);
              }
              __syncwarp();
              if (dual || i == (j < cnt[1] ? 1 : 0)) {  // the tile's last use
                if (elect_one()) umma_commit(&bar_k_empty[slot]);
                __syncwarp();
                if (++slot == KS) slot = 0, phase ^= 1;
              }
            }
          }
        }
      } else {
        // O_i += P_i V once P_i is there
        constexpr uint32_t idesc_o = idesc_bf16(kRows, D, false, true);
        const uint64_t v_desc = smem_desc_sw128(smem_u32(sV), kKeys * 128, 1024);
        uint32_t pn[2] = {0, 0}, regular = 0, special = 0;
        uint32_t slot = 0;  // of the V tile
        for (int r = 0; ok; ++r) {
          Unit u;
          if (!next_unit(r, u)) break;
          const int cnt[2] = {__shfl_sync(0xffffffffu, u.c0, 0), __shfl_sync(0xffffffffu, u.c1, 0)};
          const int part0 = __shfl_sync(0xffffffffu, first_partial(u) - u.d.kv0, 0);
          const bool dual = __shfl_sync(0xffffffffu, (int)u.dual, 0) != 0;
          const int most = max(cnt[0], cnt[1]);
          for (int j = 0; j < most && ok; ++j) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!ok || j >= cnt[i]) continue;
              if (dual || i == (j < cnt[0] ? 0 : 1)) {
                // V as loaded, or cleaned where some row does not see the whole tile
                if ((dual ? 2 * j + i : j) < part0) {
                  const uint32_t n = regular++;
                  if (!wait(&bar_v_full[n % VS], (n / VS) & 1, kDevTimeoutLoad)) break;
                } else {
                  const uint32_t n = special++;
                  if (!wait(&bar_clean[n % kTurns], (n / kTurns) & 1, kDevTimeoutConsumer)) break;
                }
              }
              if (!wait(&bar_p_full[i], pn[i] & 1, kDevTimeoutConsumer)) break;
              ++pn[i];
              tc_fence_after();
              if (elect_one()) {
                const uint64_t vd = v_desc + slot * kTile16;
#pragma unroll
                for (int kk = 0; kk < kKeys / 16; ++kk)  // keys 16kk .. 16kk+15: 8 columns of P
                  umma_f16_ts(tmem + kColO + i * 128, tmem + kColP + i * 64 + kk * 8,
                              vd + (uint32_t)(kk * 16 * 128 / 16), idesc_o,
                              (j > 0 || kk > 0) ? 1u : 0u);
                umma_commit(&bar_pv_done[i]);
              }
              __syncwarp();
              if (dual || i == (j < cnt[1] ? 1 : 0)) {  // the tile's last use
                if (elect_one()) umma_commit(&bar_v_empty[slot]);
                __syncwarp();
                if (++slot == VS) slot = 0;
              }
            }
          }
        }
      }
      // every product and commit must be done before TMEM and shared memory go
      if (elect_one()) {
        volatile int no_abort = 0;
        uint64_t* drain = &bar_drain[warp - kSWarp];
        umma_commit(drain);
        mbar_wait(drain, 0, &no_abort, a.err, kDevTimeoutMma);
      }
    }
  } else {
    regs_increase<kRegSoftmax>();
    // ---------------- softmax of row tile i; epilogue ----------------
    const int i = warp >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const int tt = row / a.HG;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_addr = lane_addr + kColS;
    const uint32_t p_addr = lane_addr + kColP + i * 64;
    const uint32_t o_addr = lane_addr + kColO + i * 128;
    const uint64_t k2 = f2_pack(a.scale_log2, a.scale_log2);
    uint32_t sn = 0, pvn = 0, halves = 0;
    int n = 0;
    uint32_t base = 0;     // V tiles of the units before
    uint32_t cleaned = 0;  // special ones of them
    int prev_nt = 0, prev_special = 0;
    bool ok = true;
    // Takes infinities and NaNs, and rows past the sequence's end, out of V tile
    // j of a unit.
    auto clean = [&](const Unit& u, int j, uint32_t n, int flag_slot) {  // n: special ones before
      const uint32_t slot = (base + j) % VS;
      if (!mbar_wait(&bar_spec[n % VS], (n / VS) & 1, abort_flag, a.err, kDevTimeoutLoad))
        return false;
      const int key0 = (u.d.kv0 + j) * kKeys, keys_end = u.d.pos0 + u.d.ntok;
      // 16-byte pieces, 8 per 128-byte line, lines chunk-major; where a piece
      // lies within its line does not matter
      uint4* tile = reinterpret_cast<uint4*>(sV + slot * Cfg::kTileBytes);
      bool odd = false;
#pragma unroll 4
      for (int q = (int)threadIdx.x & 127; q < Cfg::kTileBytes / 16; q += 128) {
        uint4 v = tile[q];
        uint32_t* e = &v.x;
        uint32_t bad = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) bad |= ((e[k] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
        const int key = key0 + ((q >> 3) & (kKeys - 1));
        if (key >= keys_end) {
          tile[q] = make_uint4(0, 0, 0, 0);
        } else if (bad != 0 && key > u.d.pos0) {  // some row does not see it
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if ((e[k] & 0x7F80u) == 0x7F80u) e[k] &= 0xFFFF0000u;
            if ((e[k] & 0x7F800000u) == 0x7F800000u) e[k] &= 0x0000FFFFu;
          }
          tile[q] = v;
          odd = true;
        }
      }
      if (odd) odd_v[flag_slot] = 1;
      fence_async_smem();
      return true;
    };
    for (int r = 0; ok; ++r) {
      Unit u;
      if (!next_unit(r, u)) break;
      base += prev_nt;
      cleaned += prev_special;
      const int part0 = first_partial(u) - u.d.kv0;
      prev_nt = u.nt;
      prev_special = max(0, u.nt - max(part0, 0));
      const int flag_slot = n % kFlagSlots;
      // of the unit after next: nobody sets or reads it any more or yet
      if (threadIdx.x == 0) odd_v[(n + 2) % kFlagSlots] = 0;
      ++n;
      const int cnt = i == 0 ? u.c0 : u.c1;
      const int tok = (u.dual ? 0 : i * a.TT) + tt;  // token of this row within the unit
      const bool valid = tt < a.TT && tok < u.d.ntok;
      const int pos = u.d.pos0 + tok;
      float m = -INFINITY, l = 0.f;  // m: of the raw scores
      for (int j = 0; j < cnt; ++j) {
        const int jt = u.dual ? 2 * j + i : j;  // key tile of the unit, and of the sequence
        const int kt = u.d.kv0 + jt;
        // While S is on its way: clean V, where some row does not see all of it.
        // One warpgroup does, the first that takes the tile.
        if (jt >= part0 && (i == 0 || u.dual || jt >= u.c0)) {
          const uint32_t n = cleaned + jt - max(part0, 0);
          ok = clean(u, jt, n, flag_slot);
          if (!ok) break;
          mbar_arrive(&bar_clean[n % kTurns]);
        }
        const int lim = valid ? pos - kt * kKeys : kKeys;
        ok = mbar_wait(&bar_s_full[i], sn & 1, abort_flag, a.err, kDevTimeoutMma);
        if (!ok) break;
        ++sn;
        tc_fence_after();
        uint32_t s[kKeys];
        tmem_ld_32x32b_x32_at<0>(s_addr, s);
        tmem_ld_32x32b_x32_at<32>(s_addr + 32, s);
        tmem_ld_32x32b_x32_at<64>(s_addr + 64, s);
        tmem_ld_32x32b_x32_at<96>(s_addr + 96, s);
        tmem_wait();
        reg_fence(s);
        tc_fence_before();
        mbar_arrive(&bar_s_empty);  // the next S may be computed
        if (__any_sync(0xffffffffu, lim < kKeys - 1)) {
#pragma unroll
          for (int c = 0; c < kKeys; ++c)
            if (c > lim) s[c] = 0xFF800000u;  // -inf
        }
        float mx;
        {
          float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
          for (int c = 0; c < kKeys; c += 8) {
            m0 = max3f(m0, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
            m1 = max3f(m1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
            m2 = max3f(m2, __uint_as_float(s[c + 4]), __uint_as_float(s[c + 5]));
            m3 = max3f(m3, __uint_as_float(s[c + 6]), __uint_as_float(s[c + 7]));
          }
          mx = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
        }
        // the maximum grew by more than 2^kGrow: take it over, and rescale l and O
        const bool grow = (mx - m) * a.scale_log2 > kGrow;
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? fast_exp2((m - mx) * a.scale_log2) : 1.f;
          if (grow) m = mx;
          l *= f;
          if (j > 0) {
            ok = mbar_wait(&bar_pv_done[i], (pvn - 1) & 1, abort_flag, a.err, kDevTimeoutMma);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(o_addr + c, o);
              tmem_wait();
              reg_fence(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st_32x32b_x16(o_addr + c, o);
            }
            tmem_wait_st();
          }
        }
        const float ms = m > -INFINITY ? m * a.scale_log2 : 0.f;
        const uint64_t nm2 = f2_pack(-ms, -ms);
        uint64_t acc_a = f2_pack(0.f, 0.f), acc_b = acc_a;
        // P in place of the S it comes from: word c of the row's 64 in s[c]
#pragma unroll
        for (int c = 0; c < kKeys / 2; ++c) {
          float p0, p1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), k2, nm2),
                    p0, p1);
          p0 = fast_exp2(p0), p1 = fast_exp2(p1);
          s[c] = pack_bf16x2(p0, p1);
          if (c & 1)
            acc_b = f2_add(acc_b, f2_pack(p0, p1));
          else
            acc_a = f2_add(acc_a, f2_pack(p0, p1));
        }
        // the product of the tile before has read its P by now
        if (j > 0) {
          ok = mbar_wait(&bar_pv_done[i], (pvn - 1) & 1, abort_flag, a.err, kDevTimeoutMma);
          if (!ok) break;
          tc_fence_after();
        }
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) tmem_st_32x32b_x16(p_addr + 16 * q4, s + 16 * q4);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar_p_full[i]);
        ++pvn;
        float la0, la1, lb0, lb1;
        f2_unpack(acc_a, la0, la1);
        f2_unpack(acc_b, lb0, lb1);
        l += (la0 + la1) + (lb0 + lb1);
      }
      if (!ok) break;
      if (cnt > 0) {
        ok = mbar_wait(&bar_pv_done[i], (pvn - 1) & 1, abort_flag, a.err, kDevTimeoutMma);
        if (!ok) break;
        tc_fence_after();
      }
      if (u.dual) {
        if (i == 1) {
          // hand the maximum and sum to the other warpgroup's thread of this row,
          // which reads O from TMEM itself
          half_m[row] = m;
          half_l[row] = l;
          tc_fence_before();
          mbar_arrive(&bar_half_done);
          ok = mbar_wait(&bar_half_read, halves & 1, abort_flag, a.err, kDevTimeoutConsumer);
          ++halves;
          if (!ok) break;
          continue;
        }
        ok = mbar_wait(&bar_half_done, halves & 1, abort_flag, a.err, kDevTimeoutConsumer);
        ++halves;
        if (!ok) break;
        tc_fence_after();
        const float m1 = half_m[row], l1 = half_l[row];
        const float mn = fmaxf(m, m1), mu = mn > -INFINITY ? mn : 0.f;
        const float w0 = fast_exp2((m - mu) * a.scale_log2);
        const float w1 = fast_exp2((m1 - mu) * a.scale_log2);
        m = mn;
        l = l * w0 + l1 * w1;
        if (u.c1 > 0) {  // O_0 = w0 O_0 + w1 O_1, in place
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16], o2[16];
            tmem_ld_32x32b_x16(o_addr + c, o);
            tmem_ld_32x32b_x16(o_addr + 128 + c, o2);
            tmem_wait();
            reg_fence(o);
            reg_fence(o2);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * w0 + __uint_as_float(o2[e]) * w1);
            tmem_st_32x32b_x16(o_addr + c, o);
          }
          tmem_wait_st();
        }
      }
      // 32 columns of O
      auto load_o = [&](int c, float (&f)[32]) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(o_addr + c, o);
        tmem_wait();
        reg_fence(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]);
      };
      const bool odd = *reinterpret_cast<volatile int*>(&odd_v[flag_slot]) != 0;
      // infinities and NaNs taken out of V, back into the rows that see their keys
      auto add_odd = [&](int c, float (&f)[32]) {
        const int lo = max(u.d.pos0 + 1, u.d.kv0 * kKeys);
        const int hi = min(pos, u.d.kv1 * kKeys - 1);
        for (int s = lo; s <= hi; ++s) {
          const __nv_bfloat16* vr = v_row(a, u, s, D);
          if (!vr) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float v = __bfloat162float(vr[c + e]);
            if (!(fabsf(v) <= 3.4e38f)) f[e] += v;
          }
        }
      };
      if (u.d.slot >= 0) {
        // one part of a split unit: O unnormalised, with its maximum (log2 domain) and sum
        const int64_t prow = (int64_t)u.d.slot * 2 * kRows + i * kRows + row;
        float* dst = a.part_o + prow * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float f[32];
          if (cnt > 0) {
            load_o(c, f);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = 0.f;
          }
          if (!valid) continue;
          if (odd) add_odd(c, f);
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            st_global_32(dst + c + e, reinterpret_cast<const uint32_t*>(f + e), a.part32);
        }
        if (valid) a.part_ml[prow] = make_float2(m * a.scale_log2, l);
      } else if (cnt > 0) {
        const float inv = 1.f / l;
        __nv_bfloat16* dst =
            a.out + (((int64_t)u.d.tok0 + tok) * a.H + u.g * a.HG + (row - tt * a.HG)) * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float f[32];
          load_o(c, f);
          if (!valid) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] *= inv;
          if (odd) add_odd(c, f);
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
          st_global_32(dst + c, w, a.out32);  // whole sectors: no staging for coalesced stores
          st_global_32(dst + c + 16, w + 8, a.out32);
        }
      }
      tc_fence_before();
      if (u.dual) mbar_arrive(&bar_half_read);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// The units of a batch.  One CTA: counts the units and their key tiles and decides
// whether they are split along the keys.  Units that fit the GPU at once are split
// so that their parts still do, into the shortest parts that allows; the rest are
// placed longest first, by a counting sort over their number of key tiles (buckets
// of an eighth of an octave), and split where one alone would outlast an even share.
// Clears the call's error word.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;  // at most
constexpr int kBuckets = 256;

__device__ __forceinline__ int bucket_of(int tiles) {  // longer first; tiles >= 1
  const int e = 31 - __clz(tiles);
  const int f = e >= 3 ? (tiles >> (e - 3)) & 7 : (tiles << (3 - e)) & 7;
  return kBuckets - 1 - (e * 8 + f);
}

struct PlanArgs {
  const int64_t* cu;          // device offsets of the new tokens, or null: `off`
  const int32_t* seq_lens;    // device, null: whole prompts
  int32_t B, T, G, TT, table_rows;  // table_rows: keys a row of the block table holds
  int32_t ctas;               // CTAs to keep busy
  int32_t can_split;          // room for partial results
  int32_t max_units, clear_err;
  DenseUnit* units;
  DenseSplit* splits;
  int32_t* counts;            // [0] units, [1] split units, [2] units handed out
  uint32_t* err;
};

// tokens [a, a+n) of sequence b, the first one at position p; n = 0 when empty or invalid
__device__ __forceinline__ void plan_seq(const PlanArgs& p, const DenseOffsets& off, int b,
                                         int64_t& a, int& n, int& pos) {
  const int64_t lo = p.cu ? __ldg(p.cu + b) : off.cu[b];
  const int64_t hi = p.cu ? __ldg(p.cu + b + 1) : off.cu[b + 1];
  const int64_t first = p.cu ? __ldg(p.cu) : 0, last = p.cu ? __ldg(p.cu + p.B) : p.T;
  const int L = p.seq_lens ? __ldg(p.seq_lens + b) : 0;
  a = lo;
  n = 0;
  pos = 0;
  if (lo < 0 || lo < first || hi < lo || hi > p.T || hi > last) {
    record_error(p.err, kDevBadIndex);
    return;
  }
  if (p.seq_lens && hi > lo) {
    if (L < hi - lo || L > p.table_rows) {
      record_error(p.err, kDevBadIndex);
      return;
    }
    pos = L - (int)(hi - lo);
  }
  n = (int)(hi - lo);
}

__global__ void __launch_bounds__(kPlanThreads)
    dense_plan_kernel(const __grid_constant__ DenseOffsets off, const PlanArgs p) {
  __shared__ int hist[kBuckets];
  __shared__ unsigned long long sum_s;
  __shared__ int longest_s, n_units_s, n_split_s, n_slot_s, part_s;
  pdl_launch_dependents();
  const int tid = threadIdx.x, warps = blockDim.x / 32;
  if (tid == 0) {
    if (p.clear_err) *p.err = 0;
    sum_s = 0, longest_s = 0, n_units_s = 0, n_split_s = 0, n_slot_s = 0, part_s = 1 << 30;
  }
  for (int i = tid; i < kBuckets; i += blockDim.x) hist[i] = 0;
  __syncthreads();
  const int U = 2 * p.TT;  // tokens per unit
  // a warp per sequence, a lane per unit of it
  auto for_units = [&](auto&& f) {
    for (int b = warp_id(); b < p.B; b += warps) {
      int64_t a;
      int n, pos;
      plan_seq(p, off, b, a, n, pos);
      for (int i = lane_id() * U; i < n; i += 32 * U)
        f(b, a, i, min(U, n - i), pos + i, (pos + min(n, i + U) - 1) / kKeys + 1);
    }
  };
  // ---- how much work there is ----
  {
    unsigned long long tiles = 0;
    int longest = 0, n = 0;
    for_units([&](int, int64_t, int, int ntok, int, int nt) {
      const int w = ntok <= p.TT ? (nt + 1) / 2 : nt;  // see weight below
      tiles += w;
      longest = max(longest, w);
      ++n;
    });
    atomicAdd(&sum_s, tiles);
    atomicMax(&longest_s, longest);
    atomicAdd(&n_units_s, n);
  }
  __syncthreads();
  const bool one_wave = (long long)n_units_s * p.G <= p.ctas;
  // kept far from 2^31, whatever the lengths
  const int share = (int)min((sum_s * p.G + p.ctas - 1) / p.ctas, 1ull << 29);
  // a unit of one row tile is taken by both softmax warpgroups: half as long
  auto weight = [&](int ntok, int nt) { return ntok <= p.TT ? (nt + 1) / 2 : nt; };
  int part = 1 << 30;  // longest part, by weight
  if (!p.can_split) {
  } else if (one_wave) {
    // the shortest parts that leave at most one per CTA: a warp per candidate
    for (int base = max(kMinPart, share); base < longest_s; base += warps) {
      const int c = base + (int)warp_id();
      long long n = 0;
      for (int b = 0; b < p.B; ++b) {
        int64_t a;
        int len, pos;
        plan_seq(p, off, b, a, len, pos);
        for (int i = (int)lane_id() * U; i < len; i += 32 * U) {
          const int w = weight(min(U, len - i), (pos + min(len, i + U) - 1) / kKeys + 1);
          n += (w + c - 1) / c;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      if (lane_id() == 0 && n * p.G <= p.ctas) atomicMin(&part_s, c);
      __syncthreads();
      const int found = part_s;
      __syncthreads();
      if (found < 1 << 30) break;
    }
    if (part_s + kJoinCost < longest_s) part = part_s;
  } else if (longest_s > share + share / 4) {
    part = max(share, kMinPart);
  }
  // parts of a unit, and the key tiles of each
  auto parts_of = [&](int ntok, int nt, int& len) {
    const int w = weight(ntok, nt);
    const int k = w > part ? (w + part - 1) / part : 1;
    len = (nt + k - 1) / k;
    return (nt + len - 1) / len;
  };
  if (!one_wave) {
    for_units([&](int, int64_t, int, int ntok, int, int nt) {
      int len;
      const int parts = parts_of(ntok, nt, len);
      for (int k = 0; k < parts; ++k)
        atomicAdd(&hist[bucket_of(part_begin(k + 1, parts, len, nt) - part_begin(k, parts, len, nt))], 1);
    });
    __syncthreads();
    if (tid < 32) {  // exclusive prefix over the buckets
      int run = 0;
      for (int i = 0; i < kBuckets; i += 32) {
        const int v = hist[i + tid];
        int x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (tid >= o) x += y;
        }
        hist[i + tid] = run + x - v;
        run += __shfl_sync(0xffffffffu, x, 31);
      }
      if (tid == 0) n_units_s = run;
    }
    __syncthreads();
  }
  for_units([&](int b, int64_t a, int i, int ntok, int pos0, int nt) {
    int len;
    const int parts = parts_of(ntok, nt, len);
    int slot = -1;
    if (parts > 1) {
      slot = atomicAdd(&n_slot_s, parts * p.G);
      const int x = atomicAdd(&n_split_s, 1);
      *reinterpret_cast<int4*>(p.splits + x) = make_int4((int)a + i, ntok, slot, parts);
    }
    for (int k = 0; k < parts; ++k) {
      const int kv0 = part_begin(k, parts, len, nt), kv1 = part_begin(k + 1, parts, len, nt);
      const int x = one_wave ? atomicAdd(&hist[0], 1) : atomicAdd(&hist[bucket_of(kv1 - kv0)], 1);
      if (x < p.max_units) {
        int4* dst = reinterpret_cast<int4*>(p.units + x);
        dst[0] = make_int4((int)a + i, ntok, pos0, b);
        dst[1] = make_int4(kv0, kv1, slot < 0 ? -1 : slot + k * p.G,
                           p.seq_lens ? 0 : (int)a);
      }
    }
  });
  __syncthreads();
  if (tid == 0) {
    p.counts[0] = min(one_wave ? hist[0] : n_units_s, p.max_units);
    p.counts[1] = n_split_s;
    p.counts[2] = 0;
  }
}

// out = sum_z 2^(m_z - M) O_z / sum_z 2^(m_z - M) l_z over the partials z of every
// split unit; a warp per row, D/32 columns a lane.
struct Join {
  int tok0, ntok, g, parts;
  int slot0, slot1, step;  // slots of parts 0, 1, 1 + step, ..
};
constexpr int kJoins = 160;  // one per CTA at most: each begins in one of its own; a multiple of 32

template <int D, int MODE>
__global__ void __launch_bounds__(256)
    dense_combine_kernel(const __grid_constant__ std::conditional_t<
                             MODE == kHost, HostSplits,
                             std::conditional_t<MODE == kDirect, DirectArgs, NoUnits>> hs,
                         const DenseSplit* splits, const int32_t* counts, const float* part_o,
                         const float2* part_ml, int H, int G, int TT, int ctas,
                         __nv_bfloat16* out) {
  const int HG = H / G;
  int n;
  // kDirect: by the CTA whose part is the first, and these CTAs in order (every block
  // makes the table for itself, so its order must not depend on timing)
  __shared__ Join table[MODE == kDirect ? kJoins : 1];
  __shared__ int list[MODE == kDirect ? kJoins : 1];
  if constexpr (MODE == kDirect) {
    __shared__ PlanUnit unit_s[kDirectUnits];
    __shared__ int2 seq_s[32];  // first packed row, tokens
    __shared__ int n_s, share_s, total_s;
    for (int i = threadIdx.x; i < kJoins; i += blockDim.x) table[i].parts = 0;
    __syncthreads();
    if (warp_id() == 0) {
      DirectPlan d;
      direct_plan(hs, G, TT, ctas, nullptr, unit_s, d);
      seq_s[lane_id()] = make_int2((int)d.lo, d.n);
      if (lane_id() == 0) share_s = d.share, total_s = d.total;
      if (d.share == 0) {
        direct_parts(d, TT, [&](int64_t tok0, int ntok, int, int, int, int, int parts, int pre) {
          if (parts <= 1) return;
          for (int g = 0, c = pre * G; g < G && c < kJoins; ++g, ++c)
            table[c] = Join{(int)tok0, ntok, g, parts, c, c + G, G};
        });
      }
    }
    __syncthreads();
    if (share_s > 0) {  // which units the shares' ends cut
      for (int x = threadIdx.x; x < total_s * G; x += blockDim.x) {
        const PlanUnit u = unit_s[x / G];
        const int g = x % G, len = u.w + kPartCost;
        const long long start = (long long)u.pre * G + (long long)g * len;
        int z = (int)(start / share_s);
        int first = -1, cuts = 0;
        for (;; ++z) {
          const int t = line_cut((long long)(z + 1) * share_s - start, len, u.nt);
          if (t >= u.nt) break;
          if (t == 0) continue;
          if (cuts == 0) first = z;
          ++cuts;
        }
        if (cuts > 0 && first < kJoins)
          table[first] = Join{seq_s[u.seq].x + u.off, min(2 * TT, seq_s[u.seq].y - u.off), g,
                              cuts + 1, 2 * first + 1, 2 * (first + 1), 2};
      }
      __syncthreads();
    }
    if (warp_id() == 0) {
      int k = 0;
      for (int c = lane_id(); c < kJoins; c += 32) {
        const unsigned m = __ballot_sync(0xffffffffu, table[c].parts > 0);
        if (table[c].parts > 0) list[k + __popc(m & ((1u << lane_id()) - 1))] = c;
        k += __popc(m);
      }
      if (lane_id() == 0) n_s = k;
    }
    __syncthreads();
    n = n_s;
    pdl_wait();
  } else if constexpr (MODE == kHost) {
    pdl_wait();
    n = hs.n;
  } else {
    pdl_wait();
    n = __ldcg(counts + 1);
  }
  const int per_tile = TT * HG, per_unit = 2 * per_tile;  // rows
  const int joins = MODE == kDirect ? n : n * G;
  const unsigned rows = (unsigned)joins * per_unit;  // at most CTAs * 256
  const int lane = lane_id();
  constexpr int C = D / 32;
  for (unsigned x = blockIdx.x * 8 + warp_id(); x < rows; x += gridDim.x * 8) {
    const unsigned y = x / per_unit;
    const int urow = (int)(x - y * per_unit);
    Join jn;
    if constexpr (MODE == kDirect) {
      jn = table[list[y]];
    } else {
      const int g = (int)(y % G);
      int4 sp;
      if constexpr (MODE == kHost) {
        const DenseSplit* d = hs.s + y / G;
        sp = make_int4(d->tok0, d->ntok, d->slot, d->parts);
      } else {
        sp = __ldcg(reinterpret_cast<const int4*>(splits + y / G));
      }
      jn = Join{sp.x, sp.y, g, sp.w, sp.z + g, sp.z + G + g, G};
    }
    const int tok = urow / HG, hh = urow - tok * HG;
    if (tok >= jn.ntok) continue;
    const int prow = tok >= TT ? kRows + urow - per_tile : urow;  // row of the partial
    const int np = jn.parts;
    auto at = [&](int z) {  // row of partial z
      return (int64_t)(z == 0 ? jn.slot0 : jn.slot1 + (z - 1) * jn.step) * 2 * kRows + prow;
    };
    float M = -INFINITY, L = 0.f, acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
    for (int z0 = 0; z0 < np; z0 += 32) {
      // lane z: partial z's maximum and sum
      float2 ml = make_float2(-INFINITY, 0.f);
      if (z0 + lane < np) ml = __ldcg(part_ml + at(z0 + lane));
      float mx = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(M, mx), mu = mn > -INFINITY ? mn : 0.f;
      const float f0 = fast_exp2(M - mu);
      const float w = fast_exp2(ml.x - mu);
      float ls = w * ml.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
      L = L * f0 + ls;
      M = mn;
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] *= f0;
      const int m = min(32, np - z0);
      // 8 rows' loads in flight at a time
      for (int z1 = 0; z1 < m; z1 += 8) {
        float v[8][C];
#pragma unroll
        for (int z = 0; z < 8; ++z) {
          const float* src = part_o + at(z0 + min(z1 + z, m - 1)) * D + lane * C;
          if constexpr (C == 4) {
            const float4 y = __ldcg(reinterpret_cast<const float4*>(src));
            v[z][0] = y.x, v[z][1] = y.y, v[z][2] = y.z, v[z][3] = y.w;
          } else {
            const float2 y = __ldcg(reinterpret_cast<const float2*>(src));
            v[z][0] = y.x, v[z][1] = y.y;
          }
        }
#pragma unroll
        for (int z = 0; z < 8; ++z) {
          const float f = __shfl_sync(0xffffffffu, w, z1 + z);
          if (z1 + z < m) {
#pragma unroll
            for (int c = 0; c < C; ++c) acc[c] += f * v[z][c];
          }
        }
      }
    }
    const float inv = 1.f / L;
    __nv_bfloat16* o = out + (((int64_t)jn.tok0 + tok) * H + jn.g * HG + hh) * D + lane * C;
    if constexpr (C == 4) {
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                pack_bf16x2(acc[2] * inv, acc[3] * inv));
    } else {
      *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    }
  }
}

// The plan of a batch with host offsets, by the rules of dense_plan_kernel; false
// when it has more units than travel as a parameter.
bool host_plan(const DensePrefillLaunch& p, int TT, HostUnits& hu, HostSplits& hs) {
  const int U = 2 * TT;
  int n = 0, longest = 0;
  int64_t sum = 0;
  int w[kHostUnits];
  auto tiles = [&](int len, int i) { return ((i + U < len ? i + U : len) - 1) / kKeys + 1; };
  auto weight = [&](int len, int i) {
    const int nt = tiles(len, i);
    return len - i <= TT ? (nt + 1) / 2 : nt;
  };
  if (p.T / U > kHostUnits) return false;
  for (int b = 0; b < p.B; ++b) {
    const int len = (int)(p.offsets->cu[b + 1] - p.offsets->cu[b]);
    for (int i = 0; i < len; i += U) {
      if (n == kHostUnits) return false;
      w[n] = weight(len, i);
      sum += w[n];
      longest = w[n] > longest ? w[n] : longest;
      ++n;
    }
  }
  const int ctas = p.grid;
  const bool one_wave = (int64_t)n * p.G <= ctas;
  const int share = (int)((sum * p.G + ctas - 1) / ctas);
  int part = 1 << 30;
  if (p.max_slots > 0) {
    if (one_wave) {
      for (int c = share > kMinPart ? share : kMinPart; c < longest; ++c) {
        int64_t m = 0;
        for (int i = 0; i < n; ++i) m += (w[i] + c - 1) / c;
        if (m * p.G <= ctas) {
          if (c + kJoinCost < longest) part = c;
          break;
        }
      }
    } else if (longest > share + share / 4) {
      part = share > kMinPart ? share : kMinPart;
    }
  }
  hu.n = hs.n = 0;
  int slots = 0;
  for (int b = 0; b < p.B; ++b) {
    const int a = (int)p.offsets->cu[b], len = (int)p.offsets->cu[b + 1] - a;
    for (int i = 0; i < len; i += U) {
      const int nt = tiles(len, i), wt = weight(len, i);
      int k = wt > part ? (wt + part - 1) / part : 1;
      const int plen = (nt + k - 1) / k;
      k = (nt + plen - 1) / plen;
      const int ntok = len - i < U ? len - i : U;
      if (hu.n + k > kHostUnits || (k > 1 && hs.n == kHostUnits / 2)) return false;
      if (k > 1) hs.s[hs.n++] = DenseSplit{a + i, ntok, slots, k};
      for (int x = 0; x < k; ++x) {
        hu.u[hu.n++] = DenseUnit{a + i, ntok, i, b, part_begin(x, k, plen, nt),
                                 part_begin(x + 1, k, plen, nt),
                                 k > 1 ? slots + x * p.G : -1, a};
      }
      if (k > 1) slots += k * p.G;
    }
  }
  if (!one_wave)
    std::stable_sort(hu.u, hu.u + hu.n, [](const DenseUnit& x, const DenseUnit& y) {
      return x.kv1 - x.kv0 > y.kv1 - y.kv0;
    });
  return true;
}

// the register split needs exactly the launch budget it was written for
template <typename K>
cudaError_t prepare(K kern, int smem) {
  static_assert(2 * 128 * kRegSoftmax + 128 * kRegOther == (uint32_t)kThreads * kLaunchRegs,
                "register split must add up to the launch budget");
  cudaFuncAttributes attr;
  const cudaError_t e = cudaFuncGetAttributes(&attr, kern);
  if (e != cudaSuccess) return e;
  if (attr.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

template <int D>
cudaError_t launch_impl(const DensePrefillLaunch& p, cudaStream_t s, int* launches) {
  using Cfg = PrefillCfg<D>;
  const int HG = p.H / p.G;
  const int TT = dense_tile_tokens(p.H, p.G);
  CUtensorMap mq, mk, mv;
  const uint64_t GD = (uint64_t)p.G * D, HD = (uint64_t)p.H * D;
  const bool paged = p.cache.page_size > 0;
  const int rows_box = paged && p.cache.page_size < kBoxRows ? p.cache.page_size : kBoxRows;
  {
    const uint64_t dims[4] = {64, (uint64_t)p.H, D / 64, (uint64_t)p.T};
    const uint64_t str[3] = {D, 64, HD};
    const uint32_t box[4] = {64, (uint32_t)HG, 1, (uint32_t)TT};
    if (!make_tmap_bf16_nd(&mq, p.q, 4, dims, str, box)) return cudaErrorInvalidValue;
  }
  {
    const uint64_t dims[5] = {64, paged ? (uint64_t)p.cache.page_size : (uint64_t)p.T, D / 64,
                              (uint64_t)p.G, paged ? (uint64_t)p.cache.num_pages : 1};
    const uint64_t str[4] = {GD, 64, D, paged ? (uint64_t)p.cache.page_stride : GD};
    const uint32_t box[5] = {64, (uint32_t)rows_box, 1, 1, 1};
    if (!make_tmap_bf16_nd(&mk, paged ? p.cache.k : p.k, 5, dims, str, box) ||
        !make_tmap_bf16_nd(&mv, paged ? p.cache.v : p.v, 5, dims, str, box))
      return cudaErrorInvalidValue;
  }
  PrefillArgs a;
  a.H = p.H;
  a.G = p.G;
  a.HG = HG;
  a.TT = TT;
  a.scale_log2 = p.scale * kLog2e;
  a.units = p.units;
  a.n_units = p.counts;
  a.next_unit = p.counts + 2;
  a.block_table = p.cache.block_table;
  a.table_stride = p.cache.table_stride;
  a.page_size = p.cache.page_size;
  a.num_pages = (int32_t)p.cache.num_pages;
  a.page_stride = p.cache.page_stride;
  a.box_rows = rows_box;
  a.v = static_cast<const __nv_bfloat16*>(paged ? p.cache.v : p.v);
  a.out = static_cast<__nv_bfloat16*>(p.out);
  a.part_o = p.part_o;
  a.part_ml = p.part_ml;
  // every row of either is a multiple of 32 bytes behind its base
  a.out32 = reinterpret_cast<uintptr_t>(p.out) % 32 == 0;
  a.part32 = reinterpret_cast<uintptr_t>(p.part_o) % 32 == 0;
  a.clear_err = p.clear_err;
  a.err = p.err;
  // a warp per row of the split units, as far as there can be rows (those of
  // tokens that a unit lacks included)
  const int64_t rows = min64(p.T * p.H + (int64_t)p.B * p.G * 2 * kRows, (int64_t)p.grid * 2 * kRows);
  const int combine_grid = (int)min64((rows + 7) / 8, (int64_t)p.grid * 16);
  // every block plans for itself: no more than are resident
  const int direct_grid = (int)min64(combine_grid, (int64_t)p.grid * 3);

  HostUnits hu;
  HostSplits hs;
  cudaError_t e;
  if (!p.cu && host_plan(p, TT, hu, hs)) {
    auto kern = dense_prefill_kernel<D, kHost>;
    if ((e = prepare(kern, Cfg::kSmem)) != cudaSuccess) return e;
    const int grid = (int)min64((int64_t)hu.n * p.G, p.grid);
    if ((int64_t)hu.n * p.G > grid) {  // more units than CTAs: handed out one by one
      if ((e = cudaMemsetAsync(p.counts + 2, 0, sizeof(int32_t), s)) != cudaSuccess) return e;
    }
    kern<<<grid, kThreads, Cfg::kSmem, s>>>(mq, mk, mv, a, hu);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ++*launches;
    if (hs.n > 0) {
      e = launch_early(dense_combine_kernel<D, kHost>, combine_grid, 256, 0, s, hs,
                       (const DenseSplit*)nullptr, (const int32_t*)nullptr, (const float*)p.part_o,
                       (const float2*)p.part_ml, p.H, p.G, TT, p.grid, a.out);
      if (e != cudaSuccess) return e;
      ++*launches;
    }
    return cudaSuccess;
  }

  const int table_rows = paged ? (int)min64((int64_t)p.cache.table_stride * p.cache.page_size,
                                            (int64_t)1 << 30)
                               : 0;
  const int64_t most = p.T / (2 * TT) + p.B;  // units, of one group
  if (p.cu && p.B <= 32 && most * p.G <= min64(p.grid, kDirectUnits)) {
    if ((e = cudaMemsetAsync(p.err, 0, sizeof(uint32_t), s)) != cudaSuccess) return e;
    DirectArgs da;
    da.cu = p.cu;
    da.seq_lens = p.seq_lens;
    da.B = p.B;
    da.T = (int32_t)p.T;
    da.table_rows = table_rows;
    da.can_split = p.max_slots > 0;
    da.max_units = (int32_t)most;
    auto kern = dense_prefill_kernel<D, kDirect>;
    if ((e = prepare(kern, Cfg::kSmem)) != cudaSuccess) return e;
    kern<<<p.grid, kThreads, Cfg::kSmem, s>>>(mq, mk, mv, a, da);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ++*launches;
    if (p.max_slots > 0) {
      e = launch_early(dense_combine_kernel<D, kDirect>, direct_grid, 256, 0, s, da,
                       (const DenseSplit*)nullptr, (const int32_t*)nullptr, (const float*)p.part_o,
                       (const float2*)p.part_ml, p.H, p.G, TT, p.grid, a.out);
      if (e != cudaSuccess) return e;
      ++*launches;
    }
    return cudaSuccess;
  }

  PlanArgs pl;
  pl.cu = p.cu;
  pl.seq_lens = p.seq_lens;
  pl.B = p.B;
  pl.T = (int32_t)p.T;
  pl.G = p.G;
  pl.TT = TT;
  pl.table_rows = table_rows;
  pl.ctas = p.grid;
  pl.can_split = p.max_slots > 0;
  pl.max_units = p.max_units;
  pl.units = p.units;
  pl.splits = p.splits;
  pl.counts = p.counts;
  pl.clear_err = p.clear_err;
  pl.err = p.err;
  // few units: a small block, whose barriers and launch are quicker
  const int plan_threads = p.T / (2 * TT) + p.B <= 256 ? 256 : kPlanThreads;
  dense_plan_kernel<<<1, plan_threads, 0, s>>>(*p.offsets, pl);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  ++*launches;
  auto kern = dense_prefill_kernel<D, kPlanned>;
  if ((e = prepare(kern, Cfg::kSmem)) != cudaSuccess) return e;
  e = launch_early(kern, p.grid, kThreads, Cfg::kSmem, s, mq, mk, mv, a, NoUnits{});
  if (e != cudaSuccess) return e;
  ++*launches;
  if (p.max_slots > 0) {
    e = launch_early(dense_combine_kernel<D, kPlanned>, combine_grid, 256, 0, s, NoUnits{},
                     (const DenseSplit*)p.splits, (const int32_t*)p.counts, (const float*)p.part_o,
                     (const float2*)p.part_ml, p.H, p.G, TT, p.grid, a.out);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaSuccess;
}

}  // namespace

int dense_tile_tokens(int H, int G) { return kRows / (H / G); }

cudaError_t launch_dense_prefill(const DensePrefillLaunch& p, cudaStream_t s, int* launches) {
  return p.d == 128 ? launch_impl<128>(p, s, launches) : launch_impl<64>(p, s, launches);
}

}  // namespace msa
