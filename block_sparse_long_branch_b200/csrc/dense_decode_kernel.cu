// dense_decode_kernel.cu -- attention of one new token per sequence over its
// paged cache:  out[b][h] = sum_{s < L_b} softmax_s(scale <q[b][h], k[s][g]>) v[s][g].
//
// Memory bound: 4 d bytes of K and V per (key, group) against 4 d (H/G) operations.
// The keys of all (sequence, group) items are one line of 16-key steps, cut into
// equal shares, one per CTA; an item that lies in several shares is joined from
// their partial results by the CTA that finishes last, always in the order of
// the shares, so results do not depend on timing.
//
// In a CTA eight warps take an item's steps in turn.  Each warp has a ring of its
// own in shared memory that its lane 0 fills by TMA (one copy of 16 rows of K and
// one of V per step, never across a page), so the warps do not wait for one another
// until an item ends.  A warp keeps the running maximum, sum and output of its
// steps in registers:
//   S = Q K^T  mma.m16n8k16: the 16 rows are the group's heads (8 heads: rows 8-15
//              are zero; 16 heads: all used)
//   O += P V   P in two bf16 parts, hi = bf16(p) and lo = bf16(p - hi), so the
//              product sees p to 16 bits: 8 heads put lo into rows 8-15 of the
//              same MMA, 16 heads take a second one.
// S, the maximum, the sum and O are fp32.
//
// A key past the sequence's end has P = 0, and its V row (memory that may hold
// anything) is zeroed in shared memory first, since 0 * NaN = NaN.
#include "kernels.h"
#include "sm100.cuh"
#include "tmap.h"

namespace msa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 16;  // keys per step
constexpr float kLog2e = 1.4426950408889634f;

// ROWS: head rows of an item (8 or 16)
template <int D, int ROWS>
struct DecodeCfg {
  static constexpr int kHalf = kStep * D * 2;  // K or V of one step
  static constexpr int kStageBytes = 2 * kHalf;
  static constexpr int kJoin = kWarps * ROWS * D * 4;  // the warps' outputs of an item
  // what 224 KiB hold beside the join buffer: 3 stages of 8 KiB a warp for 8 heads of 128
  static constexpr int kStages = (224 * 1024 - kJoin) / (kWarps * kStageBytes);
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
    record_error(a.err, kDevBadIndex);
    return 0;
  }
  return L;
}
__device__ __forceinline__ int n_steps(int L) { return (L + kStep - 1) / kStep; }

// A position in the line of all steps: step `st` of item `item` of sequence b.
struct Cursor {
  int b, item;     // item in [0, G*HC)
  int L, n;        // length and steps of sequence b
  int st;          // step within the item
  int64_t left;    // steps from here to the end of the share
};

template <int D, int ROWS>
__global__ void __launch_bounds__(kThreads, 1)
    dense_decode_kernel(const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const Args a) {
  using Cfg = DecodeCfg<D, ROWS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float* join = reinterpret_cast<float*>(smem + kWarps * Cfg::kStages * Cfg::kStageBytes);
  __shared__ uint64_t bar_full[kWarps][Cfg::kStages];
  __shared__ float jm[kWarps][ROWS], jl[kWarps][ROWS];
  __shared__ long long red[kWarps];
  __shared__ long long scan_base;
  __shared__ int start_b;
  __shared__ long long start_off;
  __shared__ int abort_s, last_s;
  const int tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  const int items = a.G * a.HC;
  if (tid == 0) {
    abort_s = 0;
    for (int w = 0; w < kWarps; ++w)
      for (int s = 0; s < Cfg::kStages; ++s) mbar_init(&bar_full[w][s], 1);
    fence_mbar_init();
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  // ---- the total number of steps, and this CTA's share ----
  long long mine = 0;
  for (int b = tid; b < a.B; b += kThreads) mine += n_steps(seq_len(a, b));
  long long v = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) red[warp] = v;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += red[w];
  total *= items;
  // a share is at least one step per warp, so that a short line is not spread thin
  long long share = (total + gridDim.x - 1) / gridDim.x;
  if (share < kWarps) share = kWarps;
  const long long lo = share * blockIdx.x;
  const long long hi = lo + share < total ? lo + share : total;
  // empty sequences: zero rows
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (seq_len(a, b) == 0) {
      uint4* o = reinterpret_cast<uint4*>(a.out + (int64_t)b * a.H * D);
      for (int x = tid; x < a.H * D / 8; x += kThreads) o[x] = make_uint4(0, 0, 0, 0);
    }
  }
  if (lo >= hi) return;
  // ---- the sequence that holds step lo ----
  if (tid == 0) scan_base = 0;
  __syncthreads();
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    const long long n = b < a.B ? (long long)n_steps(seq_len(a, b)) * items : 0;
    long long x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    const long long base0 = scan_base;
    long long base = base0;
    for (int w = 0; w < warp; ++w) base += red[w];
    const long long first = base + x - n;
    if (lo >= first && lo < first + n) {
      start_b = b;
      start_off = lo - first;
    }
    long long sum = 0;
    for (int w = 0; w < kWarps; ++w) sum += red[w];
    __syncthreads();
    if (tid == 0) scan_base = base0 + sum;
    __syncthreads();
    if (base0 + sum > lo) break;
  }

  auto next_item = [&](Cursor& c) {
    if (++c.item < items) return;
    c.item = 0;
    do {
      ++c.b;
      c.L = c.b < a.B ? seq_len(a, c.b) : 1;
    } while (c.L == 0);
    c.n = n_steps(c.L);
  };
  Cursor cur;  // of the part being computed: its first step
  cur.b = start_b;
  cur.L = seq_len(a, cur.b);
  cur.n = n_steps(cur.L);
  cur.item = (int)(start_off / cur.n);
  cur.st = (int)(start_off % cur.n);
  cur.left = hi - lo;

  // ---- this warp's loads: its steps of every part, in order ----
  uint8_t* ring = smem + warp * Cfg::kStages * Cfg::kStageBytes;
  Cursor ld = cur;      // part that the next load belongs to
  int ld_st = cur.st + warp;
  uint32_t issued = 0, used = 0;
  int page_next = 0;    // page id of the next load
  auto part_end = [&](const Cursor& c) {
    return (int)(c.left < (long long)(c.n - c.st) ? c.st + c.left : c.n);
  };
  // move `ld` to the part that holds this warp's next step; false at the end
  auto settle = [&]() {
    while (ld.left > 0) {
      const int e = part_end(ld);
      if (ld_st < e) {
        page_next = __ldg(a.block_table + (int64_t)ld.b * a.table_stride +
                          ld_st * kStep / a.page_size);
        return true;
      }
      ld.left -= e - ld.st;
      if (ld.left > 0) {
        next_item(ld);
        ld.st = 0;
        ld_st = warp;
      }
    }
    return false;
  };
  bool more = settle();
  auto load = [&]() {
    if (!more) return;
    const uint32_t s = issued % Cfg::kStages;
    if (lane == 0) {
      int pg = page_next;
      if (pg < 0 || pg >= a.num_pages) {
        record_error(a.err, kDevBadIndex);
        pg = a.num_pages;  // outside the tensor: reads zeros
      }
      const int row = ld_st * kStep % a.page_size;
      uint8_t* dst = ring + s * Cfg::kStageBytes;
      mbar_arrive_expect_tx(&bar_full[warp][s], Cfg::kStageBytes);
      tma_load_5d(dst, &map_k, &bar_full[warp][s], 0, row, 0, ld.item / a.HC, pg);
      tma_load_5d(dst + Cfg::kHalf, &map_v, &bar_full[warp][s], 0, row, 0, ld.item / a.HC, pg);
    }
    ++issued;
    ld_st += kWarps;
    more = settle();
  };
#pragma unroll 1
  for (int s = 0; s < Cfg::kStages; ++s) load();

  const int gq = lane >> 2, tq = lane & 3;
  const uint32_t ring_u = smem_u32(ring);
  // lane addresses within a step: K rows (lane & 7), 16-byte column lane >> 3;
  // V rows lane & 15, column lane >> 4
  const int k_r = lane & 7, k_c = lane >> 3;
  const int v_r = (lane & 7) + ((lane >> 3) & 1) * 8, v_c = lane >> 4;

  while (cur.left > 0) {
    const int end = part_end(cur);
    const int g = cur.item / a.HC, h0 = (cur.item % a.HC) * ROWS;
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

    for (int st = cur.st + warp; st < end; st += kWarps) {
      const uint32_t sg = used % Cfg::kStages;
      if (!mbar_wait(&bar_full[warp][sg], (used / Cfg::kStages) & 1, &abort_s, a.err,
                     kDevTimeoutLoad))
        break;
      const uint32_t kb = ring_u + sg * Cfg::kStageBytes, vb = kb + Cfg::kHalf;
      const int valid = cur.L - st * kStep;  // keys of this step that exist
      if (valid < kStep) {
        // 128-byte lines, chunk-major; a line is one row's 64 columns
        uint4* vz = reinterpret_cast<uint4*>(ring + sg * Cfg::kStageBytes + Cfg::kHalf);
        for (int x = lane; x < Cfg::kHalf / 16; x += 32)
          if (((x >> 3) & (kStep - 1)) >= valid) vz[x] = make_uint4(0, 0, 0, 0);
        fence_async_smem();
        __syncwarp();
      }
      // ---- S: two tiles of 8 keys ----
      float s[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
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
              mma_16816(s[t], qa[kk][0], 0u, qa[kk][1], 0u, b[2 * x], b[2 * x + 1]);
            else
              mma_16816(s[t], qa[kk][0], qa[kk][1 % (ROWS / 4)], qa[kk][2 % (ROWS / 4)],
                        qa[kk][3 % (ROWS / 4)], b[2 * x], b[2 * x + 1]);
          }
        }
      }
      // ---- running maximum, P, sum ----
      float f[ROWS / 8];
      float p[ROWS / 8][4];
      bool grew = false;
#pragma unroll
      for (int rr = 0; rr < ROWS / 8; ++rr) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = s[t][2 * rr + e] * a.scale_log2;
            p[rr][2 * t + e] = t * 8 + 2 * tq + e < valid ? x : -INFINITY;
          }
        float mx = fmaxf(fmaxf(p[rr][0], p[rr][1]), fmaxf(p[rr][2], p[rr][3]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[rr], mx);
        const float mu = mn > -INFINITY ? mn : 0.f;
        f[rr] = fast_exp2(m[rr] - mu);
        grew |= mn > m[rr];
        m[rr] = mn;
#pragma unroll
        for (int e = 0; e < 4; ++e) p[rr][e] = fast_exp2(p[rr][e] - mu);
        l[rr] = l[rr] * f[rr] + ((p[rr][0] + p[rr][1]) + (p[rr][2] + p[rr][3]));
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= f[0], o[i][1] *= f[0];
          o[i][2] *= f[ROWS / 8 - 1], o[i][3] *= f[ROWS / 8 - 1];
        }
      }
      // ---- O += P V, P = hi + lo ----
      uint32_t hi2[ROWS / 8][2], lo2[ROWS / 8][2];
#pragma unroll
      for (int rr = 0; rr < ROWS / 8; ++rr)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t w = pack_bf16x2(p[rr][2 * t], p[rr][2 * t + 1]);
          hi2[rr][t] = w;
          lo2[rr][t] = pack_bf16x2(p[rr][2 * t] - __uint_as_float(w << 16),
                                   p[rr][2 * t + 1] - __uint_as_float(w & 0xFFFF0000u));
        }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {  // 16 dimensions
        uint32_t b[4];
        const int col = 2 * i + v_c;
        ldsm_x4_t(b, vb + (col >> 3) * (kStep * 128) + sw128_offset(v_r, col & 7));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (ROWS == 8) {
            mma_16816(o[2 * i + x], hi2[0][0], lo2[0][0], hi2[0][1], lo2[0][1], b[2 * x],
                      b[2 * x + 1]);
          } else {
            constexpr int R1 = ROWS / 8 - 1;
            mma_16816(o[2 * i + x], hi2[0][0], hi2[R1][0], hi2[0][1], hi2[R1][1], b[2 * x],
                      b[2 * x + 1]);
            mma_16816(o[2 * i + x], lo2[0][0], lo2[R1][0], lo2[0][1], lo2[R1][1], b[2 * x],
                      b[2 * x + 1]);
          }
        }
      }
      ++used;
      __syncwarp();  // every lane has read the stage
      load();
    }

    // ---- join the warps ----
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
      float* dst = join + ((int64_t)warp * ROWS + h) * D + 2 * tq;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(dst + i * 8) = make_float2(o[i][2 * rr], o[i][2 * rr + 1]);
    }
    __syncthreads();
    const bool whole = cur.st == 0 && end == cur.n;
    // slot 0: the item began in an earlier share; 1: it begins in this one
    float* part = a.part + ((int64_t)blockIdx.x * 2 + (cur.st > 0 ? 0 : 1)) * Cfg::kPart;
    __nv_bfloat16* orow = a.out + ((int64_t)cur.b * a.H + g * a.HG + h0) * D;
    for (int x = tid; x < nh * (D / 4); x += kThreads) {
      const int h = x / (D / 4), c = x % (D / 4);
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, jm[w][h]);
      const float Mu = M > -INFINITY ? M : 0.f;
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = fast_exp2(jm[w][h] - Mu);
        const float4 y = *reinterpret_cast<const float4*>(join + ((int64_t)w * ROWS + h) * D + 4 * c);
        L += f * jl[w][h];
        acc.x += f * y.x, acc.y += f * y.y, acc.z += f * y.z, acc.w += f * y.w;
      }
      if (whole) {
        const float inv = 1.f / L;
        *reinterpret_cast<uint2*>(orow + (int64_t)h * D + 4 * c) = make_uint2(
            pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      } else {
        *reinterpret_cast<float4*>(part + h * D + 4 * c) = acc;
        if (c == 0) part[ROWS * D + 2 * h] = M, part[ROWS * D + 2 * h + 1] = L;
      }
    }
    if (!whole) {
      // shares that hold parts of this item
      const long long at = hi - cur.left;  // line position of this part
      const long long first = at - cur.st, last = first + cur.n - 1;
      const int c_first = (int)(first / share), c_last = (int)(last / share);
      __threadfence();
      __syncthreads();
      if (tid == 0)
        last_s = atomicAdd(a.tickets + (int64_t)cur.b * items + cur.item, 1) == c_last - c_first;
      __syncthreads();
      if (last_s) {
        __threadfence();
        for (int x = tid; x < nh * (D / 4); x += kThreads) {
          const int h = x / (D / 4), c = x % (D / 4);
          auto at_part = [&](int z) {
            return a.part + ((int64_t)z * 2 + (z == c_first ? 1 : 0)) * Cfg::kPart;
          };
          float M = -INFINITY;
#pragma unroll 4
          for (int z = c_first; z <= c_last; ++z)
            M = fmaxf(M, __ldcg(at_part(z) + ROWS * D + 2 * h));
          const float Mu = M > -INFINITY ? M : 0.f;
          float L = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int z = c_first; z <= c_last; ++z) {
            const float* pz = at_part(z);
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(pz + ROWS * D + 2 * h));
            const float4 y = __ldcg(reinterpret_cast<const float4*>(pz + h * D + 4 * c));
            const float f = fast_exp2(ml.x - Mu);
            L += f * ml.y;
            acc.x += f * y.x, acc.y += f * y.y, acc.z += f * y.z, acc.w += f * y.w;
          }
          const float inv = 1.f / L;
          *reinterpret_cast<uint2*>(orow + (int64_t)h * D + 4 * c) = make_uint2(
              pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        }
      }
    }
    __syncthreads();  // join, jm, jl are reused by the next part
    cur.left -= end - cur.st;
    if (cur.left > 0) {
      next_item(cur);
      cur.st = 0;
    }
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
  const uint32_t box[5] = {64, kStep, D / 64, 1, 1};
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
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<p.grid, kThreads, Cfg::kSmem, s>>>(mk, mv, a);
  return cudaGetLastError();
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
