// dense_decode_kernel.cu -- attention of one new token per sequence over its
// paged cache:  out[b][h] = sum_{s < L_b} softmax_s(scale <q[b][h], k[s][g]>) v[s][g].
//
// Memory bound: 4 d bytes of K and V per (key, group) against 4 d (H/G) operations.
// The keys of all sequences are one line of 16-key steps (32 at d = 64), cut into
// equal shares, one per CTA; what lies in several shares is joined from partial
// results by whoever finishes last, always in the order of the shares, so results
// do not depend on timing.
//
// The eight warps of a CTA take gw groups x 8/gw neighbouring steps at a time.
// Where there is work enough gw is 8: the warps read whole rows of the cache
// between them, and none waits for another.  A short line is cut finer with gw
// down to 1, eight steps of one group at a time.  Each warp has a ring of its own
// in shared memory that it fills by TMA (a copy of K and one of V per step, never
// across a page), and keeps the running maximum, sum and output of its steps in
// registers:
//   S = Q K^T  mma.m16n8k16: the 16 rows are the group's heads (8 heads: rows 8-15
//              are zero; 16 heads: all used)
//   O += P V   P in two bf16 parts, hi = p cut to 8 bits and lo = bf16(p - hi), so
//              the product sees p to 2^-16 of itself: 8 heads put lo into rows 8-15 of the
//              same MMA, 16 heads take a second one.
// S, the maximum, the sum and O are fp32.
//
// A key past the sequence's end has P = 0, and its V row (memory that may hold
// anything) is zeroed in shared memory first, since 0 * NaN = NaN.
#include "early.cuh"
#include "kernels.h"
#include "sm100.cuh"
#include "tmap.h"

namespace msa {
namespace {

constexpr int kWarps = kDenseDecodeWarps;
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;

// ROWS: head rows of an item (8 or 16)
template <int D, int ROWS>
struct DecodeCfg {
  // keys per step: 8 KiB of K and V either way.  At d = 64 steps of 16 keys leave a
  // warp waiting on its own chain of instructions (52 requests of 1 to 16K tokens, 32
  // heads in 8 groups: 98 us, with steps of 32 keys 77)
  static constexpr int kStep = D == 128 ? 16 : 32;
  static constexpr int kHalf = kStep * D * 2;  // K or V of one step
  static constexpr int kStageBytes = 2 * kHalf;
  static constexpr int kJoin = kWarps * ROWS * D * 4;  // the warps' outputs of an item
  // what 224 KiB hold beside the join buffer: 3 stages of 8 KiB a warp for 8 heads of 128
  static constexpr int kStages = (224 * 1024 - kJoin) / (kWarps * kStageBytes);
  static_assert(kWarps * kStages <= kThreads, "one thread per barrier");
  static constexpr int kSmem = kWarps * kStages * kStageBytes + kJoin + 1024;
  static constexpr int kPart = ROWS * (D + 2);  // floats of a partial
};

struct Args {
  const __nv_bfloat16* q;
  const int32_t* seq_lens;
  const int32_t* block_table;
  int32_t table_stride, page_size, num_pages;
  int32_t B, H, G, HG, HC;  // HC: items per group (HG heads in chunks of ROWS)
  float scale_log2;
  __nv_bfloat16* out;
  int32_t* tickets;
  float* part;
  uint32_t* err;
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// valid length of sequence b: 0 for an empty or an impossible one
__device__ __forceinline__ int seq_len(const Args& a, int b) {
  const int L = __ldg(a.seq_lens + b);
  if (L < 0 || (int64_t)L > (int64_t)a.table_stride * a.page_size) {
    record_error_early(a.err, kDevBadIndex);
    return 0;
  }
  return L;
}
template <int STEP>
__device__ __forceinline__ int n_steps(int L) {
  return (L + STEP - 1) / STEP;
}

// quotients of the line, mostly far below 2^32 (a 64-bit division is ten times slower)
__device__ __forceinline__ long long div_down(long long x, long long y) {
  return ((x | y) >> 32) == 0 ? (long long)((unsigned)x / (unsigned)y) : x / y;
}
__device__ __forceinline__ long long div_up(long long x, long long y) {
  return div_down(x + y - 1, y);
}

// A position in the line: step `st` of bundle `bd` (gw neighbouring items) of sequence b.
struct Cursor {
  int b, bd;
  int L, n;        // length and steps of sequence b
  int st;          // step within the bundle
  int steps;       // steps of this part, from st on
  long long left;  // line positions from this part's first to the end of the share
};

template <int D, int ROWS>
__global__ void __launch_bounds__(kThreads, 1)
    dense_decode_kernel(const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const Args a) {
  using Cfg = DecodeCfg<D, ROWS>;
  constexpr int kStep = Cfg::kStep;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float* join = reinterpret_cast<float*>(smem + kWarps * Cfg::kStages * Cfg::kStageBytes);
  __shared__ uint64_t bar_full[kWarps][Cfg::kStages];
  __shared__ float jm[kWarps][ROWS], jl[kWarps][ROWS], jf[kWarps][ROWS];
  __shared__ long long red[kWarps];
  __shared__ long long start_off;
  __shared__ int start_b, start_len;
  __shared__ int abort_s, last_s[kWarps];
  const int tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  const int items = a.G * a.HC;
  if (tid < kWarps * Cfg::kStages) {
    mbar_init(&bar_full[0][0] + tid, 1);
    fence_mbar_init();
  }
  if (tid == 0) {
    abort_s = 0;
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  // ---- the number of steps of all sequences ----
  // Sum over the block and this thread's exclusive prefix; up to 32 sequences
  // every warp does it for itself.
  const bool few = a.B <= 32;
  auto prefix = [&](long long n, long long& before) {
    long long x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    before = x - n;
    if (few) return __shfl_sync(0xffffffffu, x, 31);
    __syncthreads();
    if (lane == 31) red[warp] = x;
    __syncthreads();
    long long sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += red[w];
      sum += red[w];
    }
    return sum;
  };
  const int me = few ? lane : tid;  // the sequence of this thread, of 256 (32) at a time
  long long total = 0, seqs = 0, before = 0;
  int len = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + me;
    len = b < a.B ? seq_len(a, b) : 0;
    // steps below 2^40, sequences above it: one sum for both
    const long long sum = prefix((long long)n_steps<kStep>(len) + (len > 0 ? 1ll << 40 : 0), before);
    total += sum & ((1ll << 40) - 1);
    seqs += sum >> 40;
  }
  // empty sequences: zeros
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (seq_len(a, b) > 0) continue;
    uint4* o = reinterpret_cast<uint4*>(a.out + (int64_t)b * a.H * D);
    for (int x = tid; x < a.H * D / 8; x += kThreads) o[x] = make_uint4(0, 0, 0, 0);
  }
  // ---- groups at a time, and the line ----
  // gw: as many groups as divide the items evenly, while a share keeps 16 steps
  // and a bundle spans 16 shares at most on average: its parts are joined by one
  // CTA (8 groups, all eight at a time or fewer: one sequence of 1M 749 -> 644 us, of
  // 30K 86 -> 35).  Where both are met it decides little: 16 of 256K and one of 1M take
  // 3.06 to 3.35 ms with eight, from one GPU to another, and 3.14 to 3.17 with one to four.
  int gw = (items & 7) == 0 ? 8 : (items & 3) == 0 ? 4 : (items & 1) == 0 ? 2 : 1;
  while (gw > 1 && (total * items < 16ll * gw * gridDim.x || seqs * items * 16 < (long long)gw * gridDim.x))
    gw >>= 1;
  const int kw = kWarps / gw, bundles = items / gw;
  const int gi = warp % gw, ki = warp / gw;  // this warp's group of the bundle, and its steps' offset
  // A part costs about as much as 4 steps of each warp beside its steps (its
  // queries' latency, the join, the output): so much longer is its bundle in the
  // line.  Few bundles are padded to whole shares instead, so that no share holds
  // the ends of two, which would take it twice the time.
  const long long n_bundles = seqs * bundles;
  const bool padded = n_bundles * 8 <= gridDim.x;
  const int cost = padded ? 0 : 4 * kw;
  const long long line = total * bundles + cost * n_bundles;
  const long long ctas = padded ? gridDim.x - n_bundles : gridDim.x;
  long long share = div_up(line, ctas);
  if (share < kw) share = kw;
  auto length = [&](int n) -> long long {  // of a bundle of n steps in the line
    if (n == 0) return 0;
    return padded ? div_up(n, share) * share : (long long)n + cost;
  };
  const long long lo = share * blockIdx.x, hi = lo + share;
  // ---- the sequence that holds position lo ----
  {
    long long base = 0;
    bool found = false;
    for (int b0 = 0; b0 < a.B && base <= lo; b0 += kThreads) {
      const int b = b0 + me;
      if (a.B > kThreads) len = b < a.B ? seq_len(a, b) : 0;
      const long long mine = length(n_steps<kStep>(len)) * bundles;
      const long long sum = prefix(mine, before);
      before += base;
      found = lo >= before && lo < before + mine;
      if (found && tid == me) start_b = b, start_len = len, start_off = lo - before;
      base += sum;
    }
    if (lo >= base) {  // the line ends before this share: the same for all threads
      pdl_wait();
      return;
    }
  }
  __syncthreads();

  // the part at line offset `off` of the cursor's bundle
  auto set_part = [&](Cursor& c, long long off) {
    const long long end = off + c.left;  // where the share ends
    const long long s0 = off - cost, s1 = end - cost;
    c.st = (int)(s0 < 0 ? 0 : s0);
    const long long e = s1 < c.n ? s1 : c.n;
    c.steps = e > c.st ? (int)(e - c.st) : 0;
  };
  auto next_part = [&](Cursor& c, long long used) {  // `used` line positions on: the next bundle
    c.left -= used;
    if (c.left <= 0) return;
    if (++c.bd == bundles) {
      c.bd = 0;
      do {
        if (++c.b >= a.B) {
          c.left = 0;
          return;
        }
        c.L = seq_len(a, c.b);
      } while (c.L == 0);
      c.n = n_steps<kStep>(c.L);
    }
    set_part(c, 0);
  };
  // line positions from the part's first to its bundle's end
  long long cur_rest;
  Cursor cur;
  {
    cur.b = start_b;
    cur.L = start_len;
    cur.n = n_steps<kStep>(cur.L);
    const long long len1 = length(cur.n);
    cur.bd = (int)div_down(start_off, len1);
    const long long off = start_off - cur.bd * len1;
    cur.left = hi - lo;
    set_part(cur, off);
    cur_rest = len1 - off;
  }

  // ---- this warp's loads: its steps of every part, in order ----
  uint8_t* ring = smem + warp * Cfg::kStages * Cfg::kStageBytes;
  Cursor ld = cur;  // part of the next load
  long long ld_rest = cur_rest;
  int ld_k = 0;     // this warp's number of the next step in its part
  uint32_t issued = 0, used = 0;
  // a step lies in one page, or (32 keys in pages of 16) in two
  const int box_rows = a.page_size < kStep ? a.page_size : kStep;
  const int boxes = kStep / box_rows;
  const int ahead = 32 / boxes;  // steps whose page ids one load of the warp brings
  int pages = 0;                 // lane i: page of box i % boxes of step i / boxes of those
  auto load = [&]() {
    while (ld.left > 0 && ki + ld_k * kw >= ld.steps) {
      next_part(ld, ld_rest);
      if (ld.left > 0) ld_rest = length(ld.n);
      ld_k = 0;
    }
    if (ld.left <= 0) return;
    if (ld_k % ahead == 0) {
      const int st = ki + (ld_k + lane / boxes) * kw;
      const int key = (ld.st + st) * kStep + lane % boxes * box_rows;
      pages = 0;
      if (st < ld.steps && key < ld.L)
        pages = __ldg(a.block_table + (int64_t)ld.b * a.table_stride + key / a.page_size);
    }
    const uint32_t s = issued % Cfg::kStages;
    const int key0 = (ld.st + ki + ld_k * kw) * kStep;
    const int n = min(boxes, (ld.L - key0 + box_rows - 1) / box_rows);
    // copies with operands known to be the same in the whole warp (see elect_one)
    const int g = (ld.bd * gw + gi) / a.HC;
    uint64_t* bar = &bar_full[warp][s];
    uint8_t* dst = ring + s * Cfg::kStageBytes;
    if (elect_one()) mbar_arrive_expect_tx(bar, n * box_rows * D * 4);
    for (int b = 0; b < n; ++b, dst += box_rows * 128) {
      int pg = __shfl_sync(0xffffffffu, pages, ld_k % ahead * boxes + b);
      if (pg < 0 || pg >= a.num_pages) {
        record_error_early(a.err, kDevBadIndex);
        pg = a.num_pages;  // outside the tensor: reads zeros
      }
      const int row = (key0 + b * box_rows) % a.page_size;
      if (elect_one()) {
        tma_load_5d(dst, &map_k, bar, 0, row, 0, g, pg);
        tma_load_5d(dst + Cfg::kHalf, &map_v, bar, 0, row, 0, g, pg);
      }
    }
    __syncwarp();
    ++issued;
    ++ld_k;
  };
#pragma unroll 1
  for (int s = 0; s < Cfg::kStages; ++s) load();
  pdl_wait();  // for the cleared error word and tickets

  constexpr int NT = kStep / 8;
  const int gq = lane >> 2, tq = lane & 3;
  const uint32_t ring_u = smem_u32(ring);
  // lane addresses within a step: K rows (lane & 7), 16-byte column lane >> 3;
  // V rows lane & 15, column lane >> 4
  const int k_r = lane & 7, k_c = lane >> 3;
  const int v_r = (lane & 7) + ((lane >> 3) & 1) * 8, v_c = lane >> 4;

  while (cur.left > 0) {
    const int item = cur.bd * gw + gi;
    const int g = item / a.HC, h0 = item % a.HC * ROWS;
    const int nh = min(ROWS, a.HG - h0);
    // Q fragments: rows gq and gq + 8
    uint32_t qa[D / 16][ROWS / 4];
    {
      const __nv_bfloat16* qb = a.q + ((int64_t)cur.b * a.H + g * a.HG + h0) * D + 2 * tq;
#pragma unroll
      for (int rr = 0; rr < ROWS / 8; ++rr) {
        const int h = rr * 8 + gq;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(qb + (int64_t)h * D);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qa[kk][rr] = h < nh ? __ldg(src + kk * 8) : 0u;
          qa[kk][ROWS / 8 + rr] = h < nh ? __ldg(src + kk * 8 + 4) : 0u;
        }
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[ROWS / 8], l[ROWS / 8];
#pragma unroll
    for (int rr = 0; rr < ROWS / 8; ++rr) m[rr] = -INFINITY, l[rr] = 0.f;

    for (int st = ki; st < cur.steps; st += kw) {
      const uint32_t sg = used % Cfg::kStages;
      if (!mbar_wait(&bar_full[warp][sg], (used / Cfg::kStages) & 1, &abort_s, a.err,
                     kDevTimeoutLoad))
        break;
      const uint32_t kb = ring_u + sg * Cfg::kStageBytes, vb = kb + Cfg::kHalf;
      const int valid = cur.L - (cur.st + st) * kStep;  // keys of this step that exist
      if (valid < kStep) {
        // 128-byte lines, chunk-major; a line is one row's 64 columns
        uint4* vz = reinterpret_cast<uint4*>(ring + sg * Cfg::kStageBytes + Cfg::kHalf);
        for (int x = lane; x < Cfg::kHalf / 16; x += 32)
          if (((x >> 3) & (kStep - 1)) >= valid) vz[x] = make_uint4(0, 0, 0, 0);
        fence_async_smem();
        __syncwarp();
      }
      // ---- S: tiles of 8 keys; even and odd k-steps in sums of their own ----
      float s[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float s2[4] = {0.f, 0.f, 0.f, 0.f};
        s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
        for (int kp = 0; kp < D / 32; ++kp) {  // 32 dimensions: two k-steps
          uint32_t b[4];
          const int col = kp * 4 + k_c;
          ldsm_x4(b, kb + (col >> 3) * (kStep * 128) + sw128_offset(t * 8 + k_r, col & 7));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int kk = 2 * kp + x;
            if (ROWS == 8)
              mma_16816(x ? s2 : s[t], qa[kk][0], 0u, qa[kk][1], 0u, b[2 * x], b[2 * x + 1]);
            else
              mma_16816(x ? s2 : s[t], qa[kk][0], qa[kk][1 % (ROWS / 4)], qa[kk][2 % (ROWS / 4)],
                        qa[kk][3 % (ROWS / 4)], b[2 * x], b[2 * x + 1]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] += s2[e];
      }
      // ---- running maximum, P, sum ----
      float f[ROWS / 8];
      float p[ROWS / 8][2 * NT];
      bool grew = false;
#pragma unroll
      for (int rr = 0; rr < ROWS / 8; ++rr) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = s[t][2 * rr + e] * a.scale_log2;
            p[rr][2 * t + e] = t * 8 + 2 * tq + e < valid ? x : -INFINITY;
          }
        float mx = p[rr][0];
#pragma unroll
        for (int e = 1; e < 2 * NT; ++e) mx = fmaxf(mx, p[rr][e]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[rr], mx);
        const float mu = mn > -INFINITY ? mn : 0.f;
        f[rr] = fast_exp2(m[rr] - mu);
        grew |= mn > m[rr];
        m[rr] = mn;
#pragma unroll
        for (int e = 0; e < 2 * NT; ++e) p[rr][e] = fast_exp2(p[rr][e] - mu);
        float ls = p[rr][0];
#pragma unroll
        for (int e = 1; e < 2 * NT; ++e) ls += p[rr][e];
        l[rr] = l[rr] * f[rr] + ls;
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= f[0], o[i][1] *= f[0];
          o[i][2] *= f[ROWS / 8 - 1], o[i][3] *= f[ROWS / 8 - 1];
        }
      }
      // ---- O += P V, P = hi + lo ----
      uint32_t hi2[ROWS / 8][NT], lo2[ROWS / 8][NT];
#pragma unroll
      for (int rr = 0; rr < ROWS / 8; ++rr)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          // hi cut, not rounded, and the last bit of p set: lo > 0 wherever p > 0, so
          // that an infinity in V stays one (with lo < 0, inf - inf, and with lo = 0,
          // 0 * inf, are NaN)
          const uint32_t p0 = __float_as_uint(p[rr][2 * t]) | 1u;
          const uint32_t p1 = __float_as_uint(p[rr][2 * t + 1]) | 1u;
          hi2[rr][t] = __byte_perm(p0, p1, 0x7632);
          lo2[rr][t] = pack_bf16x2(__uint_as_float(p0) - __uint_as_float(p0 & 0xFFFF0000u),
                                   __uint_as_float(p1) - __uint_as_float(p1 & 0xFFFF0000u));
        }
#pragma unroll
      for (int kt = 0; kt < NT / 2; ++kt)  // 16 keys
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {  // 16 dimensions
          uint32_t b[4];
          const int col = 2 * i + v_c;
          ldsm_x4_t(b, vb + (col >> 3) * (kStep * 128) + sw128_offset(kt * 16 + v_r, col & 7));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (ROWS == 8) {
              mma_16816(o[2 * i + x], hi2[0][2 * kt], lo2[0][2 * kt], hi2[0][2 * kt + 1],
                        lo2[0][2 * kt + 1], b[2 * x], b[2 * x + 1]);
            } else {
              constexpr int R1 = ROWS / 8 - 1;
              mma_16816(o[2 * i + x], hi2[0][2 * kt], hi2[R1][2 * kt], hi2[0][2 * kt + 1],
                        hi2[R1][2 * kt + 1], b[2 * x], b[2 * x + 1]);
              mma_16816(o[2 * i + x], lo2[0][2 * kt], lo2[R1][2 * kt], lo2[0][2 * kt + 1],
                        lo2[R1][2 * kt + 1], b[2 * x], b[2 * x + 1]);
            }
          }
        }
      ++used;
      __syncwarp();  // every lane has read the stage
      load();
    }

    // ---- join the warps of a group; none to join when each has its own ----
    // (warps gi, gi + gw, ...; the buffers are a warp's own)
    auto sync = [&]() {
      if (kw == 1)
        __syncwarp();
      else
        __syncthreads();
    };
    if (ROWS == 8) {
      // lo products are in rows 8-15 of the same head
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] += o[i][2], o[i][1] += o[i][3];
    }
#pragma unroll
    for (int rr = 0; rr < ROWS / 8; ++rr) {
      l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 1);
      l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 2);
      const int h = rr * 8 + gq;
      if (tq == 0) jm[warp][h] = m[rr], jl[warp][h] = l[rr];
      float* dst = join + (warp * ROWS + h) * D + 2 * tq;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(dst + i * 8) = make_float2(o[i][2 * rr], o[i][2 * rr + 1]);
    }
    sync();
    const int tg = ki * 32 + lane, n_tg = kw * 32;  // thread of the group's warps
    const bool whole = cur.steps == cur.n;
    // slot 0: the bundle began in an earlier share; 1: it begins in this one
    float* part = a.part + (((int64_t)blockIdx.x * 2 + (cur.st > 0 ? 0 : 1)) * kWarps + gi) * Cfg::kPart;
    __nv_bfloat16* orow = a.out + ((int64_t)cur.b * a.H + g * a.HG + h0) * D;
    if (cur.steps > 0) {
      for (int x = tg; x < nh * (D / 4); x += n_tg) {
        const int h = x / (D / 4), c = x % (D / 4);
        float M = -INFINITY;
        for (int w = gi; w < kWarps; w += gw) M = fmaxf(M, jm[w][h]);
        const float Mu = M > -INFINITY ? M : 0.f;
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = gi; w < kWarps; w += gw) {
          const float f = fast_exp2(jm[w][h] - Mu);
          const float4 y = *reinterpret_cast<const float4*>(join + (w * ROWS + h) * D + 4 * c);
          L += f * jl[w][h];
          acc.x += f * y.x, acc.y += f * y.y, acc.z += f * y.z, acc.w += f * y.w;
        }
        if (whole) {
          const float inv = 1.f / L;
          *reinterpret_cast<uint2*>(orow + (int64_t)h * D + 4 * c) = make_uint2(
              pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        } else {
          *reinterpret_cast<float4*>(part + h * D + 4 * c) = acc;
          if (c == 0) *reinterpret_cast<float2*>(part + ROWS * D + 2 * h) = make_float2(M, L);
        }
      }
      if (!whole) {
        // the shares that hold steps of this bundle
        const long long at = hi - cur.left;                 // the part's line position
        const long long first = at + cur_rest - length(cur.n) + cost;  // of step 0
        const int c_first = (int)div_down(first, share);
        const int c_last = (int)div_down(first + cur.n - 1, share);
        __threadfence();
        sync();
        if (tg == 0)
          last_s[gi] =
              atomicAdd(a.tickets + (int64_t)cur.b * items + item, 1) == c_last - c_first;
        sync();
        if (last_s[gi]) {
          __threadfence();
          // only this group's warps are here
          auto group_sync = [&]() {
            if (kw == 1)
              __syncwarp();
            else
              named_barrier(1 + gi, n_tg);
          };
          // Parts in chunks of D/2.  Their maxima and sums go to shared memory in one
          // round trip and become weights there; then 16 loads of O in flight a thread.
          constexpr int kChunk = D / 2, kItems = ROWS * D / 128;
          float2(*wl)[ROWS] = reinterpret_cast<float2(*)[ROWS]>(join + gi * ROWS * D);
          static_assert(kChunk * ROWS * sizeof(float2) <= ROWS * D * 4, "a warp's join buffer");
          auto at_part = [&](int z) {
            return a.part + (((int64_t)z * 2 + (z == c_first ? 1 : 0)) * kWarps + gi) * Cfg::kPart;
          };
          float4 acc[kItems];
#pragma unroll
          for (int i = 0; i < kItems; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int z0 = c_first; z0 <= c_last; z0 += kChunk) {
            const int nz = min(kChunk, c_last - z0 + 1);
            if (z0 > c_first) group_sync();  // the chunk before has been used
            for (int x = tg; x < nz * ROWS; x += n_tg)
              if (x % ROWS < nh)
                wl[x / ROWS][x % ROWS] = __ldcg(reinterpret_cast<const float2*>(
                    at_part(z0 + x / ROWS) + ROWS * D + 2 * (x % ROWS)));
            group_sync();
            if (ki == 0) {
              // lanes h, h + ROWS, ..: head h
              const int h = lane % ROWS;
              const float m0 = z0 > c_first ? jm[gi][h] : -INFINITY;
              const float l0 = z0 > c_first ? jl[gi][h] : 0.f;
              float mx = m0;
              if (h < nh)
                for (int z = lane / ROWS; z < nz; z += 32 / ROWS) mx = fmaxf(mx, wl[z][h].x);
#pragma unroll
              for (int o = ROWS; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              const float mu = mx > -INFINITY ? mx : 0.f;
              float ls = 0.f;
              if (h < nh)
                for (int z = lane / ROWS; z < nz; z += 32 / ROWS) {
                  const float w = fast_exp2(wl[z][h].x - mu);
                  ls += w * wl[z][h].y;
                  wl[z][h].x = w;
                }
#pragma unroll
              for (int o = ROWS; o < 32; o <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
              const float f = fast_exp2(m0 - mu);
              __syncwarp();
              if (lane < ROWS) jm[gi][h] = mx, jl[gi][h] = l0 * f + ls, jf[gi][h] = f;
            }
            group_sync();
#pragma unroll
            for (int i0 = 0; i0 < kItems; i0 += 4) {
              if (tg + i0 * n_tg >= nh * (D / 4)) break;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float f = jf[gi][min(tg + (i0 + i) * n_tg, nh * (D / 4) - 1) / (D / 4)];
                acc[i0 + i].x *= f, acc[i0 + i].y *= f, acc[i0 + i].z *= f, acc[i0 + i].w *= f;
              }
              for (int z = 0; z < nz; z += 4) {
                float4 y[4][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float* pz = at_part(z0 + min(z + e, nz - 1));
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const int x = min(tg + (i0 + i) * n_tg, nh * (D / 4) - 1);
                    y[e][i] = __ldcg(reinterpret_cast<const float4*>(pz + 4 * x));
                  }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if (z + e >= nz) continue;
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const int x = min(tg + (i0 + i) * n_tg, nh * (D / 4) - 1);
                    const float f = wl[z + e][x / (D / 4)].x;
                    float4& v = acc[i0 + i];
                    v.x += f * y[e][i].x, v.y += f * y[e][i].y;
                    v.z += f * y[e][i].z, v.w += f * y[e][i].w;
                  }
                }
              }
            }
          }
#pragma unroll
          for (int i = 0; i < kItems; ++i) {
            const int x = tg + i * n_tg;
            if (x >= nh * (D / 4)) continue;
            const int h = x / (D / 4), c = x % (D / 4);
            const float inv = 1.f / jl[gi][h];
            *reinterpret_cast<uint2*>(orow + (int64_t)h * D + 4 * c) = make_uint2(
                pack_bf16x2(acc[i].x * inv, acc[i].y * inv), pack_bf16x2(acc[i].z * inv, acc[i].w * inv));
          }
        }
      }
    }
    sync();  // the buffers are reused by the next part
    next_part(cur, cur_rest);
    if (cur.left > 0) cur_rest = length(cur.n);
  }
  if (abort_s) {
    // copies in flight must land before the CTA's shared memory goes
    int no_abort = 0;
    for (uint32_t x = used; x < issued; ++x)
      mbar_wait(&bar_full[warp][x % Cfg::kStages], (x / Cfg::kStages) & 1, &no_abort, nullptr, 0);
  }
}

template <int D, int ROWS>
cudaError_t launch_impl(const DenseDecodeLaunch& p, cudaStream_t s) {
  using Cfg = DecodeCfg<D, ROWS>;
  CUtensorMap mk, mv;
  const uint64_t GD = (uint64_t)p.G * D;
  const uint64_t dims[5] = {64, (uint64_t)p.cache.page_size, D / 64, (uint64_t)p.G,
                            (uint64_t)p.cache.num_pages};
  const uint64_t str[4] = {GD, 64, D, (uint64_t)p.cache.page_stride};
  const uint32_t box_rows = p.cache.page_size < Cfg::kStep ? p.cache.page_size : Cfg::kStep;
  const uint32_t box[5] = {64, box_rows, D / 64, 1, 1};
  if (!make_tmap_bf16_nd(&mk, p.cache.k, 5, dims, str, box) ||
      !make_tmap_bf16_nd(&mv, p.cache.v, 5, dims, str, box))
    return cudaErrorInvalidValue;
  Args a;
  a.q = static_cast<const __nv_bfloat16*>(p.q);
  a.seq_lens = p.seq_lens;
  a.block_table = p.cache.block_table;
  a.table_stride = p.cache.table_stride;
  a.page_size = p.cache.page_size;
  a.num_pages = (int32_t)p.cache.num_pages;
  a.B = p.B;
  a.H = p.H;
  a.G = p.G;
  a.HG = p.H / p.G;
  a.HC = dense_decode_chunks(p.H, p.G) / p.G;
  a.scale_log2 = p.scale * kLog2e;
  a.out = static_cast<__nv_bfloat16*>(p.out);
  a.tickets = p.tickets;
  a.part = p.part;
  a.err = p.err;
  auto kern = dense_decode_kernel<D, ROWS>;
  cudaError_t e = launch_clear(p.err, p.clear_words, s);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
  if (e != cudaSuccess) return e;
  return launch_early(kern, p.grid, kThreads, Cfg::kSmem, s, mk, mv, a);
}

}  // namespace

int dense_decode_chunks(int H, int G) {
  const int HG = H / G;
  return G * (HG <= 8 ? 1 : (HG + 15) / 16);
}

size_t dense_decode_partial_floats(int H, int G, int d) {
  return (size_t)(H / G <= 8 ? 8 : 16) * (d + 2);
}

cudaError_t launch_dense_decode(const DenseDecodeLaunch& p, cudaStream_t s) {
  const bool small = p.H / p.G <= 8;
  if (p.d == 128) return small ? launch_impl<128, 8>(p, s) : launch_impl<128, 16>(p, s);
  return small ? launch_impl<64, 8>(p, s) : launch_impl<64, 16>(p, s);
}

}  // namespace msa
