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
// then off by at most 2^-9 of itself, beside the 2^-9 of the bf16 output.
//
// Rows that a mask hides.  A hidden key has P = 0 exactly, but 0 * NaN = NaN on the
// tensor cores, so in the tiles that some row of the unit does not see whole
// (the last ones) V is first cleaned: rows past the sequence's end are zeroed,
// and infinities or NaNs are replaced by zero and added back, by the epilogue,
// to those rows that do see their key.
//
// Warp roles (384 threads, one CTA per SM, persistent over the units):
//   WG0, WG1  softmax of row tile 0 / 1, one thread per row; the rescaling of
//             O; the final O / l;
//   WG2       warp 8 TMA loads, warp 9 MMA issuer (one thread), warps 10, 11
//             cleaning of V.
// TMEM (512 columns): S0, S1 (fp32; each P overwrites the first half of its S)
// and O0, O1.  While one tile's exponentials are computed the tensor cores work
// on the other tile.
#include "kernels.h"
#include "sm100.cuh"
#include "tmap.h"

namespace msa {
namespace {

constexpr int kThreads = 384;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kCleanWarp0 = 10;
constexpr int kCleanThreads = 64;
constexpr uint32_t kRegSoftmax = 208, kRegOther = 88;
constexpr int kLaunchRegs = 168;  // 2*128*208 + 128*88 = 384*168
constexpr int kRows = 128, kKeys = 128;
constexpr uint32_t kColS = 0, kColO = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.f;  // log2 of the growth of the maximum left unapplied
constexpr int kFlagSlots = 4;

template <int D>
struct PrefillCfg {
  static constexpr int kChunks = D / 64;           // 128-byte column chunks
  static constexpr int kTileBytes = kRows * D * 2;  // Q, K and V tiles alike
  // one ring for K and V tiles in the order of their use (K0 V0 K1 V1 ...): what
  // 224 KiB hold beside the two Q tiles.  A tile takes some 2000 cycles to come
  // from L2; with two K and two V tiles the MMAs waited for it.
  static constexpr int kSlots = D == 128 ? 5 : 10;
  // P handed over in two parts (96 and 32 keys): 680 against 644 TFLOP/s at d = 64
  // (8K prompt, 64 heads), nothing gained at d = 128 (1161 against 1176)
  static constexpr bool kSplitP = D == 64;
  static constexpr int kOffRing = 2 * kTileBytes;
  static constexpr int kSmem = kOffRing + kSlots * kTileBytes + 1024;
};

// position in the ring: slot and the parity of its use
template <int N>
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) slot = 0, phase ^= 1;
  }
};

struct PrefillArgs {
  int32_t H, G, HG, TT;
  float scale, scale_log2;
  const DenseUnit* units;
  const int32_t* n_units;  // tile pairs (each for all groups)
  // paged keys and values; page_size 0: packed rows
  const int32_t* block_table;
  int32_t table_stride, page_size, num_pages;
  int64_t page_stride;  // elements
  const __nv_bfloat16* v;
  __nv_bfloat16* out;
  float* part_o;     // [slot][256][D]
  float2* part_ml;   // [slot][256] (log2-domain maximum, sum)
  uint32_t* err;
};

struct Unit {
  DenseUnit d;
  int g;
  int c0, c1;   // key tiles of row tile 0 / 1
  int nt;       // key tiles of the unit
};

// The r-th unit of this CTA: units come longest first, and every other round
// runs through the CTAs backwards, so that no CTA always gets the longer ones.
__device__ __forceinline__ bool get_unit(const PrefillArgs& a, int total, int r, Unit& u) {
  const int c = (r & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x;
  const int64_t x = (int64_t)r * gridDim.x + c;
  if (x >= total) return false;
  const int i = (int)(x / a.G);
  u.g = (int)(x - (int64_t)i * a.G);
  const int4* p = reinterpret_cast<const int4*>(a.units + i);
  const int4 x0 = __ldg(p), x1 = __ldg(p + 1);
  u.d.tok0 = x0.x, u.d.ntok = x0.y, u.d.pos0 = x0.z, u.d.seq = x0.w;
  u.d.kv0 = x1.x, u.d.kv1 = x1.y, u.d.slot = x1.z, u.d.row0 = x1.w;
  u.nt = u.d.kv1 - u.d.kv0;
  const int last0 = u.d.pos0 + min(u.d.ntok, a.TT) - 1;  // last position of row tile 0
  u.c0 = max(0, min(u.d.kv1, last0 / kKeys + 1) - u.d.kv0);
  u.c1 = u.d.ntok > a.TT ? u.nt : 0;
  return true;
}
__device__ __forceinline__ int n_rounds(int total) {
  return (total + (int)gridDim.x - 1) / (int)gridDim.x;
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

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    dense_prefill_kernel(const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const PrefillArgs a) {
  using Cfg = PrefillCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sR = smem + Cfg::kOffRing;
  __shared__ uint64_t bar_q_full[2], bar_q_empty[2];
  __shared__ uint64_t bar_full[Cfg::kSlots], bar_empty[Cfg::kSlots];
  __shared__ uint64_t bar_clean[2];  // V tiles cleaned, in turn
  __shared__ uint64_t bar_s_full[2], bar_p_most[2], bar_p_full[2], bar_pv_done[2], bar_drain;
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;
  __shared__ int odd_v[kFlagSlots];  // an infinity or NaN was taken out of the unit's V

  const int warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    abort_s = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_q_full[i], 1);
      mbar_init(&bar_q_empty[i], 1);
      mbar_init(&bar_clean[i], kCleanThreads);
      mbar_init(&bar_s_full[i], 1);
      mbar_init(&bar_p_most[i], 128);
      mbar_init(&bar_p_full[i], 128);
      mbar_init(&bar_pv_done[i], 1);
    }
    for (int i = 0; i < Cfg::kSlots; ++i) {
      mbar_init(&bar_full[i], 1);
      mbar_init(&bar_empty[i], 1);
    }
    mbar_init(&bar_drain, 1);
    for (int i = 0; i < kFlagSlots; ++i) odd_v[i] = 0;
    fence_mbar_init();
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
  const int total = __ldg(a.n_units) * a.G;
  const int rounds = n_rounds(total);

  if (warp >= 8) {
    regs_decrease<kRegOther>();
    if (warp == kLoadWarp) {
      // ---------------- TMA loads ----------------
      if (lane == 0) {
        tma_prefetch_desc(&map_q);
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
      }
      Ring<Cfg::kSlots> ring;
      uint32_t loads = 0;         // copies into the ring so far
      uint32_t qn[2] = {0, 0};    // Q tiles loaded so far
      bool ok = true;
      const int boxes = a.page_size == 0 ? 1 : (a.page_size >= kKeys ? 1 : kKeys / a.page_size);
      const int box_rows = kKeys / boxes;
      auto load_q = [&](const Unit& u, int i) {
        if (!ok || (i == 0 ? u.c0 : u.c1) == 0) return;
        if (lane == 0) {
          ok = mbar_wait(&bar_q_empty[i], (qn[i] & 1) ^ 1, abort_flag, a.err, kDevTimeoutMma);
          if (ok) {
            mbar_arrive_expect_tx(&bar_q_full[i], (uint32_t)(a.TT * a.HG * D * 2));
#pragma unroll
            for (int c = 0; c < Cfg::kChunks; ++c)
              tma_load_4d(sQ + i * Cfg::kTileBytes + c * kRows * 128, &map_q, &bar_q_full[i], 0,
                          u.g * a.HG, c, u.d.tok0 + i * a.TT);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (ok) ++qn[i];
      };
      // the next tile into the ring: one box per page, a lane each; pages past
      // the sequence's end are not read
      auto load_kv = [&](const CUtensorMap* map, int g, int32_t row, int32_t page, int nbox) {
        if (!ok) return;
        uint64_t* full = &bar_full[ring.slot];
        if (lane == 0) {
          ok = mbar_wait(&bar_empty[ring.slot], ring.phase ^ 1, abort_flag, a.err, kDevTimeoutMma);
          if (ok) mbar_arrive_expect_tx(full, (uint32_t)(nbox * box_rows * D * 2));
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) return;
        if (lane < nbox) {
          uint8_t* dst = sR + ring.slot * Cfg::kTileBytes + lane * box_rows * 128;
#pragma unroll
          for (int c = 0; c < Cfg::kChunks; ++c)
            tma_load_5d(dst + c * kKeys * 128, map, full, 0, row, c, g, page);
        }
        __syncwarp();
        ++loads;
        ring.next();
      };
      for (int r = 0; r < rounds && ok; ++r) {
        Unit u;
        if (!get_unit(a, total, r, u)) continue;
        const int keys_end = u.d.pos0 + u.d.ntok;
        for (int j = 0; j < u.nt && ok; ++j) {
          const int key0 = (u.d.kv0 + j) * kKeys;
          int32_t row, page = 0;
          int nbox = 1;
          if (a.page_size == 0) {
            row = u.d.row0 + key0;
          } else {
            const int left = (keys_end - key0 + box_rows - 1) / box_rows;
            nbox = left < boxes ? left : boxes;
            const int key = key0 + lane * box_rows;
            row = key % a.page_size;
            if (lane < nbox) {
              page = __ldg(a.block_table + (int64_t)u.d.seq * a.table_stride + key / a.page_size);
              if (page < 0 || page >= a.num_pages) {
                record_error(a.err, kDevBadIndex);
                page = a.num_pages;  // outside the tensor: reads zeros
              }
            }
          }
          if (j == 0) load_q(u, 0);
          load_kv(&map_k, u.g, row, page, nbox);
          if (j == 0) load_q(u, 1);
          load_kv(&map_v, u.g, row, page, nbox);
        }
      }
      if (lane == 0 && *abort_flag) {
        // the copies in flight must land before the CTA's shared memory goes
        volatile int no_abort = 0;
        for (int i = 0; i < 2; ++i)
          if (qn[i]) mbar_wait(&bar_q_full[i], (qn[i] - 1) & 1, &no_abort, nullptr, 0);
        for (uint32_t x = loads > Cfg::kSlots ? loads - Cfg::kSlots : 0; x < loads; ++x)
          mbar_wait(&bar_full[x % Cfg::kSlots], (x / Cfg::kSlots) & 1, &no_abort, nullptr, 0);
      }
    } else if (warp == kMmaWarp) {
      // ---------------- MMA issuer ----------------
      // The whole warp walks the units, so that the operands of the MMAs are
      // warp-uniform (uniform registers); one lane issues.  With the walk in
      // one lane alone a batch of eight MMAs took 870 cycles to issue.
      constexpr uint32_t idesc_s = idesc_bf16(kRows, kKeys, false, false);
      constexpr uint32_t idesc_o = idesc_bf16(kRows, D, false, true);
      constexpr uint32_t kTile16 = Cfg::kTileBytes / 16;  // descriptor units
      const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t k_desc = smem_desc_sw128(smem_u32(sR), 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(smem_u32(sR), kKeys * 128, 1024);
      uint32_t qn[2] = {0, 0}, pn[2] = {0, 0}, cleaned = 0;
      Ring<Cfg::kSlots> ring;
      bool ok = true;
      auto issue_s = [&](int i, uint32_t slot, bool last) {
        if (elect_one()) {
          const uint64_t qd = q_desc + (uint32_t)i * kTile16, kd = k_desc + slot * kTile16;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * kRows * 128 + (kk & 3) * 32) / 16;
            umma_bf16(tmem + kColS + i * 128, qd + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
          }
          umma_commit(&bar_s_full[i]);
          if (last) umma_commit(&bar_q_empty[i]);
        }
        __syncwarp();
      };
      auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t code) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.err, code));
        return ok;
      };
      for (int r = 0; r < rounds && ok; ++r) {
        Unit u;
        if (!get_unit(a, total, r, u)) continue;
        // broadcasts: known to be the same in every lane
        const int nt = __shfl_sync(0xffffffffu, u.nt, 0);
        const int cnt[2] = {__shfl_sync(0xffffffffu, u.c0, 0), __shfl_sync(0xffffffffu, u.c1, 0)};
        const int part0 = __shfl_sync(0xffffffffu, first_partial(u) - u.d.kv0, 0);
        if (!wait(&bar_full[ring.slot], ring.phase, kDevTimeoutLoad)) break;
        uint32_t k_slot = ring.slot;
        ring.next();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (cnt[i] == 0) continue;
          if (!wait(&bar_q_full[i], qn[i] & 1, kDevTimeoutLoad)) break;
          ++qn[i];
          tc_fence_after();
          issue_s(i, k_slot, cnt[i] == 1);
        }
        if (!ok) break;
        if (elect_one()) umma_commit(&bar_empty[k_slot]);
        __syncwarp();
        for (int j = 0; j < nt; ++j) {
          const uint32_t v_slot = ring.slot;
          // V as loaded, or cleaned where some row does not see the whole tile
          if (j >= part0) {
            if (!wait(&bar_clean[cleaned & 1], (cleaned >> 1) & 1, kDevTimeoutConsumer)) break;
            ++cleaned;
          } else {
            if (!wait(&bar_full[v_slot], ring.phase, kDevTimeoutLoad)) break;
          }
          ring.next();
          if (j + 1 < nt) {
            if (!wait(&bar_full[ring.slot], ring.phase, kDevTimeoutLoad)) break;
            k_slot = ring.slot;
            ring.next();
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (j >= cnt[i]) continue;
            const uint64_t vd = v_desc + v_slot * kTile16;
            auto issue_pv = [&](int kk) {  // keys 16kk .. 16kk+15
              umma_f16_ts(tmem + kColO + i * 128, tmem + kColS + i * 128 + kk * 8,
                          vd + (uint32_t)(kk * 16 * 128 / 16), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
            };
            if (Cfg::kSplitP) {
              if (!wait(&bar_p_most[i], pn[i] & 1, kDevTimeoutConsumer)) break;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 6; ++kk) issue_pv(kk);
              }
              __syncwarp();
            }
            if (!wait(&bar_p_full[i], pn[i] & 1, kDevTimeoutConsumer)) break;
            ++pn[i];
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = Cfg::kSplitP ? 6 : 0; kk < 8; ++kk) issue_pv(kk);
              umma_commit(&bar_pv_done[i]);
            }
            __syncwarp();
            if (j + 1 < cnt[i]) issue_s(i, k_slot, j + 2 == cnt[i]);
          }
          if (!ok) break;
          if (elect_one()) {
            umma_commit(&bar_empty[v_slot]);
            if (j + 1 < nt) umma_commit(&bar_empty[k_slot]);
          }
          __syncwarp();
        }
      }
      // after an abort every product issued must be done before TMEM and shared
      // memory go; the drain barrier is used for nothing else
      if (*abort_flag && elect_one()) {
        volatile int no_abort = 0;
        umma_commit(&bar_drain);
        mbar_wait(&bar_drain, 0, &no_abort, nullptr, 0);
      }
    } else {
      // ---------------- cleaning of V ----------------
      const int x = (int)threadIdx.x - kCleanWarp0 * 32;
      Ring<Cfg::kSlots> ring;
      int n = 0;
      uint32_t cleaned = 0;
      bool ok = true;
      for (int r = 0; r < rounds && ok; ++r) {
        Unit u;
        if (!get_unit(a, total, r, u)) continue;
        const int part0 = first_partial(u) - u.d.kv0;
        const int keys_end = u.d.pos0 + u.d.ntok;
        if (x == 0) odd_v[n % kFlagSlots] = 0;
        for (int j = 0; j < u.nt && ok; ++j) {
          ring.next();  // past the K tile
          const uint32_t slot = ring.slot;
          ok = mbar_wait(&bar_full[slot], ring.phase, abort_flag, a.err, kDevTimeoutLoad);
          ring.next();
          if (!ok || j < part0) continue;
          const int key0 = (u.d.kv0 + j) * kKeys;
          uint8_t* base = sR + slot * Cfg::kTileBytes;
          bool odd = false;
          // 16-byte pieces, 8 per 128-byte line, lines chunk-major; where a
          // piece lies within its line does not matter
          for (int p = x; p < Cfg::kTileBytes / 16; p += kCleanThreads) {
            const int line = p >> 3;
            const int key = key0 + (line & (kKeys - 1));
            if (key <= u.d.pos0) continue;  // every row sees it
            uint4* w = reinterpret_cast<uint4*>(base) + p;
            if (key >= keys_end) {
              *w = make_uint4(0, 0, 0, 0);
              continue;
            }
            uint4 v = *w;
            uint32_t* e = &v.x;
            bool bad = false;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              bad |= (((e[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u) != 0;
            if (bad) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if ((e[i] & 0x7F80u) == 0x7F80u) e[i] &= 0xFFFF0000u;
                if ((e[i] & 0x7F800000u) == 0x7F800000u) e[i] &= 0x0000FFFFu;
              }
              *w = v;
              odd = true;
            }
          }
          if (odd) odd_v[n % kFlagSlots] = 1;
          fence_async_smem();
          mbar_arrive(&bar_clean[cleaned++ & 1]);
        }
        ++n;
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
    const uint32_t s_addr = lane_addr + kColS + i * 128;
    const uint32_t o_addr = lane_addr + kColO + i * 128;
    const uint64_t k2 = f2_pack(a.scale_log2, a.scale_log2);
    uint32_t sn = 0, pvn = 0;
    int n = 0;
    bool ok = true;
    for (int r = 0; r < rounds && ok; ++r) {
      Unit u;
      if (!get_unit(a, total, r, u)) continue;
      const int flag_slot = n++ % kFlagSlots;
      const int cnt = i == 0 ? u.c0 : u.c1;
      const int tok = i * a.TT + tt;  // token of this row within the unit
      const bool valid = tt < a.TT && tok < u.d.ntok;
      const int pos = u.d.pos0 + tok;
      float m = -INFINITY, l = 0.f;  // m: of the raw scores
      for (int j = 0; j < cnt; ++j) {
        const int lim = valid ? pos - (u.d.kv0 + j) * kKeys : kKeys;
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
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          uint32_t w[16];
#pragma unroll
          for (int x2 = 0; x2 < 16; ++x2) {
            const int col = 32 * q4 + 2 * x2;
            const uint64_t x = f2_fma(f2_pack(__uint_as_float(s[col]), __uint_as_float(s[col + 1])),
                                      k2, nm2);
            float p0, p1;
            f2_unpack(x, p0, p1);
            p0 = fast_exp2(p0), p1 = fast_exp2(p1);
            w[x2] = pack_bf16x2(p0, p1);
            if (x2 & 1)
              acc_b = f2_add(acc_b, f2_pack(p0, p1));
            else
              acc_a = f2_add(acc_a, f2_pack(p0, p1));
          }
          tmem_st_32x32b_x16(s_addr + 16 * q4, w);
          if (Cfg::kSplitP && q4 == 2) {  // the product with the first 96 keys' values may start
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bar_p_most[i]);
          }
        }
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
      const bool odd = cnt > 0 && *reinterpret_cast<volatile int*>(&odd_v[flag_slot]) != 0;
      const int64_t slot = u.d.slot >= 0 ? (int64_t)u.d.slot + u.g : -1;
      const int prow = i * kRows + row;  // row of the unit
      if (slot >= 0) {
        // one part of a split unit: O unnormalised, with its maximum (log2 domain) and sum
        float* dst = a.part_o + (slot * 2 * kRows + prow) * D;
        const int k_lo = max(u.d.pos0 + 1, u.d.kv0 * kKeys);
        const int k_hi = min(pos, u.d.kv1 * kKeys - 1);
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t o[16];
          if (cnt > 0) {
            tmem_ld_32x32b_x16(o_addr + c, o);
            tmem_wait();
            reg_fence(o);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0;
          }
          if (odd && valid) {
            for (int s = k_lo; s <= k_hi; ++s) {
              const __nv_bfloat16* vr = v_row(a, u, s, D);
              if (!vr) continue;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float v = __bfloat162float(vr[c + e]);
                if (!(fabsf(v) <= 3.4e38f)) o[e] = __float_as_uint(__uint_as_float(o[e]) + v);
              }
            }
          }
          if (valid) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<uint4*>(dst + c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        if (valid) a.part_ml[slot * 2 * kRows + prow] = make_float2(m * a.scale_log2, l);
        tc_fence_before();
        continue;
      }
      const float inv = 1.f / l;
      __nv_bfloat16* dst =
          a.out + (((int64_t)u.d.tok0 + tok) * a.H + u.g * a.HG + (row - tt * a.HG)) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(o_addr + c, o);
        tmem_wait();
        reg_fence(o);
        if (!valid) continue;
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * inv;
        if (odd) {
          for (int s = u.d.pos0 + 1; s <= pos; ++s) {
            const __nv_bfloat16* vr = v_row(a, u, s, D);
            if (!vr) continue;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float v = __bfloat162float(vr[c + e]);
              if (!(fabsf(v) <= 3.4e38f)) f[e] += v;
            }
          }
        }
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
        // a row's 32-byte sectors whole: no staging for coalesced stores
        st_global_32(dst + c, w);
        st_global_32(dst + c + 16, w + 8);
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// The units of a batch, longest first.  One CTA: counts the units and their key
// tiles, decides whether units are split along the keys, and places every unit
// (or part) by a counting sort over its number of key tiles (buckets of an
// eighth of an octave).
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
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
  int32_t split_ctas;         // CTAs to keep busy; 0: never split
  int32_t max_slots, max_units;
  DenseUnit* units;
  DenseSplit* splits;
  int32_t* counts;            // [0] units, [1] split units
  uint32_t* err;
};

// tokens [a, a+n) of sequence b, the first one at position p; n = 0 when empty or invalid
__device__ __forceinline__ void plan_seq(const PlanArgs& p, const DenseOffsets& off, int b,
                                         int64_t& a, int& n, int& pos) {
  const int64_t lo = p.cu ? __ldg(p.cu + b) : off.cu[b];
  const int64_t hi = p.cu ? __ldg(p.cu + b + 1) : off.cu[b + 1];
  a = lo;
  n = 0;
  pos = 0;
  if (lo < 0 || hi < lo || hi > p.T) {
    record_error(p.err, kDevBadIndex);
    return;
  }
  if (p.seq_lens && hi > lo) {
    const int L = __ldg(p.seq_lens + b);
    if (L < hi - lo || L > p.table_rows) {
      record_error(p.err, kDevBadIndex);
      return;
    }
    pos = L - (int)(hi - lo);
  }
  n = (int)(hi - lo);
}

__device__ __forceinline__ unsigned long long block_sum64(unsigned long long v,
                                                          unsigned long long* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane_id() == 0) red[warp_id()] = v;
  __syncthreads();
  unsigned long long s = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) s += red[w];
  __syncthreads();
  return s;
}

__global__ void __launch_bounds__(kPlanThreads)
    dense_plan_kernel(const __grid_constant__ DenseOffsets off, const PlanArgs p) {
  __shared__ int hist[kBuckets];
  __shared__ unsigned long long red[kPlanThreads / 32];
  __shared__ int longest_s, n_split_s, n_slot_s;
  const int tid = threadIdx.x;
  if (tid == 0) longest_s = 0, n_split_s = 0, n_slot_s = 0;
  for (int i = tid; i < kBuckets; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  const int U = 2 * p.TT;  // tokens per unit
  // ---- how much work there is ----
  // A warp per sequence, a lane per unit of it.
  unsigned long long tiles = 0;
  int longest = 0;
  for (int b = warp_id(); b < p.B; b += kPlanThreads / 32) {
    int64_t a;
    int n, pos;
    plan_seq(p, off, b, a, n, pos);
    for (int i = lane_id() * U; i < n; i += 32 * U) {
      const int nt = (pos + min(n, i + U) - 1) / kKeys + 1;
      tiles += nt;
      longest = max(longest, nt);
    }
  }
  atomicMax(&longest_s, longest);
  const unsigned long long sum = block_sum64(tiles, red) * p.G;
  // ---- split the longest units when they would outlast an even share ----
  int part = 1 << 30;
  if (p.split_ctas > 0) {
    const int share = (int)((sum + p.split_ctas - 1) / p.split_ctas);
    if (longest_s > share + share / 4) part = max(share, 4);
  }
  auto for_units = [&](auto&& f) {
    for (int b = warp_id(); b < p.B; b += kPlanThreads / 32) {
      int64_t a;
      int n, pos;
      plan_seq(p, off, b, a, n, pos);
      for (int i = lane_id() * U; i < n; i += 32 * U) {
        const int nt = (pos + min(n, i + U) - 1) / kKeys + 1;
        const int parts = (nt + part - 1) / part;
        f(b, a, i, n, pos, nt, parts);
      }
    }
  };
  for_units([&](int, int64_t, int, int, int, int nt, int parts) {
    const int len = (nt + parts - 1) / parts;
    for (int k = 0; k < parts; ++k) {
      const int c = min(len, nt - k * len);
      if (c > 0) atomicAdd(&hist[bucket_of(c)], 1);
    }
  });
  __syncthreads();
  if (tid < 32) {  // exclusive prefix over the buckets
    int run = 0;
    for (int i = 0; i < kBuckets; i += 32) {
      int v = hist[i + tid], x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (tid >= o) x += y;
      }
      hist[i + tid] = run + x - v;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (tid == 0) p.counts[0] = min(run, p.max_units);
  }
  __syncthreads();
  for_units([&](int b, int64_t a, int i, int n, int pos, int nt, int parts) {
    const int len = (nt + parts - 1) / parts;
    parts = (nt + len - 1) / len;
    DenseUnit d;
    d.tok0 = (int)a + i;
    d.ntok = min(U, n - i);
    d.pos0 = pos + i;
    d.seq = b;
    d.slot = -1;
    d.row0 = p.seq_lens ? 0 : (int)a;
    int slot = -1;
    if (parts > 1) {
      slot = atomicAdd(&n_slot_s, parts * p.G);
      const int x = atomicAdd(&n_split_s, 1);
      DenseSplit sp;
      sp.tok0 = d.tok0, sp.ntok = d.ntok, sp.slot = slot, sp.parts = parts;
      p.splits[x] = sp;
    }
    for (int k = 0; k < parts; ++k) {
      d.kv0 = k * len;
      d.kv1 = min(nt, (k + 1) * len);
      d.slot = slot < 0 ? -1 : slot + k * p.G;
      const int x = atomicAdd(&hist[bucket_of(d.kv1 - d.kv0)], 1);
      if (x < p.max_units) {
        int4* dst = reinterpret_cast<int4*>(p.units + x);
        dst[0] = make_int4(d.tok0, d.ntok, d.pos0, d.seq);
        dst[1] = make_int4(d.kv0, d.kv1, d.slot, d.row0);
      }
    }
  });
  __syncthreads();
  if (tid == 0) p.counts[1] = n_split_s;
}

// out = sum_z 2^(m_z - M) O_z / sum_z 2^(m_z - M) l_z over the parts z of every
// split unit; a warp per row, D/32 columns a lane.
template <int D>
__global__ void __launch_bounds__(256)
    dense_combine_kernel(const DenseSplit* splits, const int32_t* counts, const float* part_o,
                         const float2* part_ml, int H, int G, int TT, __nv_bfloat16* out) {
  const int HG = H / G;
  const int n = __ldg(counts + 1);
  const int64_t rows = (int64_t)n * G * 2 * kRows;
  const int lane = lane_id();
  constexpr int C = D / 32;
  for (int64_t x = (int64_t)blockIdx.x * 8 + warp_id(); x < rows; x += (int64_t)gridDim.x * 8) {
    const int prow = (int)(x % (2 * kRows));
    const int64_t y = x / (2 * kRows);
    const int g = (int)(y % G);
    const int4 sp = __ldg(reinterpret_cast<const int4*>(splits + y / G));
    const int tile = prow / kRows, row = prow % kRows;
    const int tt = row / HG, tok = tile * TT + tt;
    if (tt >= TT || tok >= sp.y) continue;
    // lane z reads part z's maximum and sum
    float M = -INFINITY;
    for (int z = lane; z < sp.w; z += 32)
      M = fmaxf(M, part_ml[((int64_t)sp.z + (int64_t)z * G + g) * 2 * kRows + prow].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (!(M > -INFINITY)) M = 0.f;
    float L = 0.f, acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
#pragma unroll 4
    for (int z = 0; z < sp.w; ++z) {
      const int64_t pr = ((int64_t)sp.z + (int64_t)z * G + g) * 2 * kRows + prow;
      const float2 ml = __ldg(part_ml + pr);
      const float w = fast_exp2(ml.x - M);
      L += w * ml.y;
      const float* src = part_o + pr * D + lane * C;
      if constexpr (C == 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(src));
        acc[0] += w * v.x, acc[1] += w * v.y, acc[2] += w * v.z, acc[3] += w * v.w;
      } else {
        const float2 v = __ldg(reinterpret_cast<const float2*>(src));
        acc[0] += w * v.x, acc[1] += w * v.y;
      }
    }
    const float inv = 1.f / L;
    __nv_bfloat16* o = out + (((int64_t)sp.x + tok) * H + g * HG + (row - tt * HG)) * D + lane * C;
    if constexpr (C == 4) {
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                pack_bf16x2(acc[2] * inv, acc[3] * inv));
    } else {
      *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    }
  }
}

template <int D>
cudaError_t launch_impl(const DensePrefillLaunch& p, cudaStream_t s, int* launches) {
  using Cfg = PrefillCfg<D>;
  const int HG = p.H / p.G;
  const int TT = dense_tile_tokens(p.H, p.G);
  CUtensorMap mq, mk, mv;
  const uint64_t GD = (uint64_t)p.G * D, HD = (uint64_t)p.H * D;
  const bool paged = p.cache.page_size > 0;
  const int rows_box = paged && p.cache.page_size < kKeys ? p.cache.page_size : kKeys;
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
  PlanArgs pl;
  pl.cu = p.cu;
  pl.seq_lens = p.seq_lens;
  pl.B = p.B;
  pl.T = (int32_t)p.T;
  pl.G = p.G;
  pl.TT = TT;
  pl.table_rows = paged ? (int32_t)min64((int64_t)p.cache.table_stride * p.cache.page_size,
                                         (int64_t)1 << 30)
                        : 0;
  pl.split_ctas = p.max_slots > 0 ? p.grid : 0;
  pl.max_slots = p.max_slots;
  pl.max_units = p.max_units;
  pl.units = p.units;
  pl.splits = p.splits;
  pl.counts = p.counts;
  pl.err = p.err;
  dense_plan_kernel<<<1, kPlanThreads, 0, s>>>(*p.offsets, pl);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ++*launches;

  PrefillArgs a;
  a.H = p.H;
  a.G = p.G;
  a.HG = HG;
  a.TT = TT;
  a.scale = p.scale;
  a.scale_log2 = p.scale * kLog2e;
  a.units = p.units;
  a.n_units = p.counts;
  a.block_table = p.cache.block_table;
  a.table_stride = p.cache.table_stride;
  a.page_size = p.cache.page_size;
  a.num_pages = (int32_t)p.cache.num_pages;
  a.page_stride = p.cache.page_stride;
  a.v = static_cast<const __nv_bfloat16*>(paged ? p.cache.v : p.v);
  a.out = static_cast<__nv_bfloat16*>(p.out);
  a.part_o = p.part_o;
  a.part_ml = p.part_ml;
  a.err = p.err;
  auto kern = dense_prefill_kernel<D>;
  // the register split needs exactly the launch budget it was written for
  cudaFuncAttributes attr;
  e = cudaFuncGetAttributes(&attr, kern);
  if (e != cudaSuccess) return e;
  static_assert(2 * 128 * kRegSoftmax + 128 * kRegOther == (uint32_t)kThreads * kLaunchRegs,
                "register split must add up to the launch budget");
  if (attr.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<p.grid, kThreads, Cfg::kSmem, s>>>(mq, mk, mv, a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ++*launches;
  if (p.max_slots > 0) {
    dense_combine_kernel<D><<<p.grid * 4, 256, 0, s>>>(p.splits, p.counts, p.part_o, p.part_ml,
                                                       p.H, p.G, TT, a.out);
    e = cudaGetLastError();
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
