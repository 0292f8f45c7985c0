// rope_append_kernel.cu -- rotation of the new tokens' queries and keys by their
// positions, and the append of keys and values to a paged cache.
//
//   a_j = p * w_j (p the token's position, w_j = inv_freq[j], j < rot/2)
//   (x, y) -> (x cos a_j - y sin a_j, y cos a_j + x sin a_j)
// for the pairs (x_j, x_{j + rot/2}), or (x_2j, x_{2j+1}) when interleaved; the
// dimensions from rot on are copied.  The angle is formed and reduced to a
// fraction of a turn in fp64 (p * w_j reaches 10^6 radians, where fp32 would be
// off by 0.06); sine and cosine of the fraction, the rotation and nothing else
// are fp32, rounded once to bf16.
//
// Memory bound: every element is read and written once.  A thread owns the same
// 16 dimensions of a head (two 16-byte pieces that hold 8 whole pairs in either
// layout) in every head it visits, so a token's 8 sines and cosines are read
// from shared memory once per thread, not once per head; a token's angles are
// computed once per CTA.
#include "kernels.h"
#include "sm100.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;

// Largest b with cu[b] <= t, for t in [cu[0], cu[B]); a whole warp, 32 samples a step.
__device__ __forceinline__ int find_seq(const int64_t* __restrict__ cu, int B, int64_t t) {
  int lo = 0, n = B;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + (int)lane_id() * step;
    const bool le = i < lo + n && __ldg(cu + i) <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int k = m ? 31 - __clz(m) : 0;
    const int rest = n - k * step;
    lo += k * step;
    n = rest < step ? rest : step;
  }
  return lo;
}

struct Args {
  PagedCache cache;
  const uint8_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // bytes
  const float* inv_freq;
  int32_t rot;
  const int64_t* cu;
  const int32_t* seq_lens;
  int32_t B, H, G;
  int64_t T;
  uint8_t* q_out;
  uint32_t* err;
};

// D: head size; IL: adjacent pairs; TOK: tokens per CTA.
template <int D, bool IL, int TOK>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const Args a) {
  constexpr int kItems = D / 16;               // 16-dimension items of a head
  constexpr int kHeadLanes = kThreads / kItems;  // heads visited at once
  __shared__ float2 cs[TOK][D / 2];  // (cos, sin)
  __shared__ int64_t kv_off[TOK];    // element offset of the token's row in the cache, -1: none
  __shared__ int64_t pos_s[TOK];     // -1: not a token of any sequence
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * TOK;
  for (int i = warp_id(); i < TOK; i += kThreads / 32) {
    const int64_t t = t0 + i;
    int64_t pos = -1, off = -1;
    if (t < a.T && t >= __ldg(a.cu) && t < __ldg(a.cu + a.B)) {
      const int b = find_seq(a.cu, a.B, t);
      const int64_t end = __ldg(a.cu + b + 1);
      pos = (int64_t)__ldg(a.seq_lens + b) - (end - t);
      // a sequence with fewer keys than new tokens, offsets that are not
      // ascending, or a row past the block table
      if (t < __ldg(a.cu + b) || t >= end ||
          pos < t - __ldg(a.cu + b) ||
          pos >= (int64_t)a.cache.table_stride * a.cache.page_size) {
        if (lane_id() == 0) record_error(a.err, kDevBadIndex);
        pos = -1;
      } else {
        const int pg = __ldg(a.cache.block_table + (int64_t)b * a.cache.table_stride +
                             pos / a.cache.page_size);
        if (pg < 0 || pg >= a.cache.num_pages) {
          if (lane_id() == 0) record_error(a.err, kDevBadIndex);
        } else {
          off = (int64_t)pg * a.cache.page_stride +
                (pos % a.cache.page_size) * (int64_t)a.G * D;
        }
      }
    }
    if (lane_id() == 0) pos_s[i] = pos, kv_off[i] = off;
  }
  __syncthreads();
  const int nf = a.rot / 2;
  for (int x = tid; x < TOK * nf; x += kThreads) {
    const int i = x / nf, j = x - i * nf;
    const int64_t pos = pos_s[i];
    if (pos < 0) continue;
    constexpr double kInvPi = 0.31830988618379067154;  // 1 / pi
    double h = (double)pos * (double)__ldg(a.inv_freq + j) * kInvPi;  // half turns
    h -= 2.0 * rint(h * 0.5);
    float s, c;
    sincospif((float)h, &s, &c);
    cs[i][j] = make_float2(c, s);
  }
  __syncthreads();

  const int item = tid % kItems, hl = tid / kItems;
  const bool rotated = item * 16 < a.rot;
  // the two 16-byte pieces of the item
  int c0, c1;
  if (IL || !rotated) {
    c0 = item * 2;
    c1 = c0 + 1;
  } else {
    c0 = item;
    c1 = item + a.rot / 16;
  }
  const int heads = (a.q ? a.H : 0) + a.G;  // rotated heads; the values follow
#pragma unroll 1
  for (int i = 0; i < TOK; ++i) {
    if (pos_s[i] < 0) continue;
    const int64_t t = t0 + i;
    float cc[8], ss[8];
    if (rotated) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float4 w = *reinterpret_cast<const float4*>(&cs[i][item * 8 + e]);
        cc[e] = w.x, ss[e] = w.y, cc[e + 1] = w.z, ss[e + 1] = w.w;
      }
    }
    const int64_t off = kv_off[i];
    const uint8_t* qrow = a.q + t * a.q_stride;
    const uint8_t* krow = a.k + t * a.k_stride;
    const uint8_t* vrow = a.v + t * a.v_stride;
    const int nq = heads - a.G;
    const int end = off >= 0 ? heads + a.G : nq;  // a token without a row in the cache: q only
#pragma unroll 3
    for (int h = hl; h < end; h += kHeadLanes) {
      const uint8_t* src;
      uint8_t* dst;
      if (h < nq) {
        src = qrow + (int64_t)h * D * 2;
        dst = a.q_out + (t * a.H + h) * (int64_t)D * 2;
      } else if (h < heads) {
        src = krow + (int64_t)(h - nq) * D * 2;
        dst = static_cast<uint8_t*>(a.cache.k) + (off + (int64_t)(h - nq) * D) * 2;
      } else {
        src = vrow + (int64_t)(h - heads) * D * 2;
        dst = static_cast<uint8_t*>(a.cache.v) + (off + (int64_t)(h - heads) * D) * 2;
      }
      uint4 x = *reinterpret_cast<const uint4*>(src + c0 * 16);
      uint4 y = *reinterpret_cast<const uint4*>(src + c1 * 16);
      if (rotated && h < heads) {
        uint32_t *xw = &x.x, *yw = &y.x;
        if (IL) {
          // a word holds one pair
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t& w = e < 4 ? xw[e] : yw[e - 4];
            const float p = __uint_as_float(w << 16), q = __uint_as_float(w & 0xFFFF0000u);
            w = pack_bf16x2(p * cc[e] - q * ss[e], q * cc[e] + p * ss[e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p0 = __uint_as_float(xw[e] << 16);
            const float p1 = __uint_as_float(xw[e] & 0xFFFF0000u);
            const float q0 = __uint_as_float(yw[e] << 16);
            const float q1 = __uint_as_float(yw[e] & 0xFFFF0000u);
            const float c_0 = cc[2 * e], s_0 = ss[2 * e], c_1 = cc[2 * e + 1], s_1 = ss[2 * e + 1];
            xw[e] = pack_bf16x2(p0 * c_0 - q0 * s_0, p1 * c_1 - q1 * s_1);
            yw[e] = pack_bf16x2(q0 * c_0 + p0 * s_0, q1 * c_1 + p1 * s_1);
          }
        }
      }
      *reinterpret_cast<uint4*>(dst + c0 * 16) = x;
      *reinterpret_cast<uint4*>(dst + c1 * 16) = y;
    }
  }
}

template <int D, bool IL>
cudaError_t launch_d(const RopeAppendLaunch& p, const Args& a, cudaStream_t s) {
  // one token per CTA while that leaves CTAs idle, four otherwise
  constexpr int kTok = 4;
  if (p.T <= (int64_t)p.num_sms * 8) {
    rope_append_kernel<D, IL, 1><<<(unsigned)p.T, kThreads, 0, s>>>(a);
  } else {
    rope_append_kernel<D, IL, kTok><<<(unsigned)((p.T + kTok - 1) / kTok), kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendLaunch& p, cudaStream_t s) {
  Args a;
  a.cache = p.cache;
  a.q = static_cast<const uint8_t*>(p.q);
  a.k = static_cast<const uint8_t*>(p.k);
  a.v = static_cast<const uint8_t*>(p.v);
  a.q_stride = p.q_stride * 2;
  a.k_stride = p.k_stride * 2;
  a.v_stride = p.v_stride * 2;
  a.inv_freq = p.inv_freq;
  a.rot = p.rot;
  a.cu = p.cu;
  a.seq_lens = p.seq_lens;
  a.B = p.B;
  a.H = p.H;
  a.G = p.G;
  a.T = p.T;
  a.q_out = static_cast<uint8_t*>(p.q_out);
  a.err = p.err;
  if (p.d == 128) return p.interleaved ? launch_d<128, true>(p, a, s) : launch_d<128, false>(p, a, s);
  return p.interleaved ? launch_d<64, true>(p, a, s) : launch_d<64, false>(p, a, s);
}

}  // namespace msa
