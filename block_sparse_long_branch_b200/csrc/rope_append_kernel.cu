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
// Memory bound: every element is read and written once.  A CTA takes a few tokens:
// their rows in the cache and their sines and cosines first, then 16 dimensions of
// a head per thread and turn (two 16-byte pieces that hold 8 whole pairs in either
// layout).  A 32K prompt of 64 + 2 x 8 heads of 128 takes 218 to 234 us from one GPU to
// another: 5.7 to 6.2 TB/s.
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
  bool checked;  // the last CTA checks the batch (check_batch), else the last ones its offsets
  int32_t checks;  // CTAs behind those of the tokens
};

// Whether a sequence of offsets [lo, hi) and length L takes part: the offsets ascend and
// lie within those of the batch and the tokens given, and it has at least as many keys
// as new tokens and no more than its row of the block table holds.
__device__ __forceinline__ bool seq_ok(const Args& a, int64_t lo, int64_t hi, int64_t L,
                                       int64_t first, int64_t last) {
  return lo >= 0 && lo >= first && hi >= lo && hi <= last && hi <= a.T &&
         (hi == lo || (L >= hi - lo && L <= (int64_t)a.cache.table_stride * a.cache.page_size));
}

// Where token t's row is: its position (-1: of no sequence, or of an invalid one)
// and the element offset in the cache (-1: none).  A whole warp.
__device__ __forceinline__ void locate(const Args& a, int64_t t, int row_elems, int64_t& pos,
                                       int64_t& off) {
  pos = off = -1;
  if (t >= a.T) return;
  const int lane = lane_id();
  int b = -1;
  int64_t end = 0;
  int L = 0;
  if (a.B < 32) {  // all offsets and lengths in one round trip
    const int64_t c = lane <= a.B ? __ldg(a.cu + lane) : 0;
    const int l = lane < a.B ? __ldg(a.seq_lens + lane) : 0;
    const int64_t c1 = __shfl_down_sync(0xffffffffu, c, 1);
    const int64_t first = __shfl_sync(0xffffffffu, c, 0), last = __shfl_sync(0xffffffffu, c, a.B);
    const unsigned m = __ballot_sync(
        0xffffffffu, lane < a.B && c <= t && t < c1 && seq_ok(a, c, c1, l, first, last));
    if (m == 0) return;
    b = 31 - __clz(m);
    end = __shfl_sync(0xffffffffu, c1, b);
    L = __shfl_sync(0xffffffffu, l, b);
  } else {
    const int64_t first = __ldg(a.cu), last = __ldg(a.cu + a.B);
    if (t < first || t >= last) return;
    const int s = find_seq(a.cu, a.B, t);
    const int64_t lo = __ldg(a.cu + s);
    end = __ldg(a.cu + s + 1);
    L = __ldg(a.seq_lens + s);
    if (lo <= t && t < end && seq_ok(a, lo, end, L, first, last)) {
      b = s;
    } else {
      // an invalid sequence; where offsets descend another may hold the token
      for (int b0 = 0; b0 < a.B && b < 0; b0 += 32) {
        const int i = b0 + lane;
        const int64_t c = i < a.B ? __ldg(a.cu + i) : 0, c1 = i < a.B ? __ldg(a.cu + i + 1) : 0;
        const int l = i < a.B ? __ldg(a.seq_lens + i) : 0;
        const unsigned m =
            __ballot_sync(0xffffffffu, c <= t && t < c1 && seq_ok(a, c, c1, l, first, last));
        if (m == 0) continue;
        const int k = __ffs(m) - 1;
        b = b0 + k;
        end = __shfl_sync(0xffffffffu, c1, k);
        L = __shfl_sync(0xffffffffu, l, k);
      }
      if (b < 0) return;
    }
  }
  pos = (int64_t)L - (end - t);
  const int pg =
      __ldg(a.cache.block_table + (int64_t)b * a.cache.table_stride + pos / a.cache.page_size);
  if (pg < 0 || pg >= a.cache.num_pages) {
    if (lane == 0 && !a.checked) record_error(a.err, kDevBadIndex);
    return;
  }
  off = (int64_t)pg * a.cache.page_stride + (pos % a.cache.page_size) * (int64_t)row_elems;
}

// The offsets and lengths of 256 sequences of a larger batch, a thread each; bad page ids
// are recorded by the CTAs that meet them.
__device__ __forceinline__ void check_offsets(const Args& a, int64_t b) {
  if (b >= a.B) return;
  if (!seq_ok(a, __ldg(a.cu + b), __ldg(a.cu + b + 1), __ldg(a.seq_lens + b), __ldg(a.cu),
              __ldg(a.cu + a.B)))
    record_error(a.err, kDevBadIndex);
}

// The error word of a batch of up to kThreads sequences, written whole by one CTA that
// looks at every length and page id while the others work: no memset in front of the
// kernel (16 tokens, issued one by one: 14.8 -> 12.8 us; 4.3 of it the kernel's).  A
// thread per sequence; pages beyond a sequence's second by the warps.
__device__ __forceinline__ void check_batch(const Args& a) {
  __shared__ int long_s[kThreads], n_long;
  const int b = threadIdx.x, ps = a.cache.page_size;
  if (b == 0) n_long = 0;
  __syncthreads();
  auto bad_page = [&](int seq, int64_t p) {
    const int pg = __ldg(a.cache.block_table + (int64_t)seq * a.cache.table_stride + p);
    return pg < 0 || pg >= a.cache.num_pages;
  };
  bool bad = false;
  if (b < a.B) {
    const int64_t lo = __ldg(a.cu + b), hi = __ldg(a.cu + b + 1);
    const int64_t L = __ldg(a.seq_lens + b), first = L - (hi - lo);
    if (!seq_ok(a, lo, hi, L, __ldg(a.cu), __ldg(a.cu + a.B))) {
      bad = true;
    } else if (hi > lo) {
      const int64_t p0 = first / ps, p1 = (L - 1) / ps;
      bad = bad_page(b, p0) | bad_page(b, p0 < p1 ? p0 + 1 : p0);
      if (p0 + 1 < p1) long_s[atomicAdd(&n_long, 1)] = b;
    }
  }
  __syncthreads();
  for (int i = warp_id(); i < n_long; i += kThreads / 32) {
    const int s = long_s[i];
    const int64_t L = __ldg(a.seq_lens + s), first = L - (__ldg(a.cu + s + 1) - __ldg(a.cu + s));
    for (int64_t p = first / ps + 2 + lane_id(); p <= (L - 1) / ps; p += 32) bad |= bad_page(s, p);
  }
  const bool any = __syncthreads_or(bad);
  if (b == 0) *a.err = any ? kDevBadIndex : 0;
}

constexpr int kMaxTok = 16;

// D: head size; IL: adjacent pairs; tok: tokens per CTA.
template <int D, bool IL>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const Args a, const int tok) {
  constexpr int kItems = D / 16;     // 16-dimension items of a head
  __shared__ alignas(16) float2 cs[kMaxTok][D / 2];  // (cos, sin), read two at a time
  __shared__ int64_t off_s[kMaxTok], pos_s[kMaxTok];
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * tok;
  if (t0 >= a.T) {
    if (a.checked)
      check_batch(a);
    else
      check_offsets(a, (int64_t)(blockIdx.x - (gridDim.x - a.checks)) * kThreads + tid);
    return;
  }
  for (int i = warp_id(); i < tok; i += kThreads / 32) {
    int64_t pos, off;
    locate(a, t0 + i, a.G * D, pos, off);
    if (lane_id() == 0) pos_s[i] = pos, off_s[i] = off;
  }
  __syncthreads();
  const int nf = a.rot / 2;
  for (int x = tid; x < tok * nf; x += kThreads) {
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

  const int nq = a.q ? a.H : 0, nr = nq + a.G, heads = nr + a.G;  // queries, keys; then values
  const int per_tok = heads * kItems, total = tok * per_tok;
#pragma unroll 4
  for (int x = tid; x < total; x += kThreads) {
    const int i = x / per_tok, y = x - i * per_tok;
    const int h = y / kItems, item = y % kItems;
    const int64_t t = t0 + i, off = off_s[i];
    if (pos_s[i] < 0 || (h >= nq && off < 0)) continue;
    const bool rotated = h < nr && item * 16 < a.rot;
    // the two 16-byte pieces of the item
    int c0 = item * 2, c1 = item * 2 + 1;
    if (!IL && item * 16 < a.rot) c0 = item, c1 = item + a.rot / 16;
    const uint8_t* src;
    uint8_t* dst;
    if (h < nq) {
      src = a.q + t * a.q_stride + h * (D * 2);
      dst = a.q_out + (t * a.H + h) * (int64_t)(D * 2);
    } else if (h < nr) {
      src = a.k + t * a.k_stride + (h - nq) * (D * 2);
      dst = static_cast<uint8_t*>(a.cache.k) + (off + (h - nq) * D) * 2;
    } else {
      src = a.v + t * a.v_stride + (h - nr) * (D * 2);
      dst = static_cast<uint8_t*>(a.cache.v) + (off + (h - nr) * D) * 2;
    }
    uint4 u = *reinterpret_cast<const uint4*>(src + c0 * 16);
    uint4 w = *reinterpret_cast<const uint4*>(src + c1 * 16);
    if (rotated) {
      uint32_t *uw = &u.x, *ww = &w.x;
      const float4* tr = reinterpret_cast<const float4*>(&cs[i][item * 8]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 r = tr[e];  // cos, sin of pairs 2e and 2e + 1
        if (IL) {
          // a word holds one pair
          uint32_t& w0 = e < 2 ? uw[2 * e] : ww[2 * e - 4];
          uint32_t& w1 = e < 2 ? uw[2 * e + 1] : ww[2 * e - 3];
          const float p0 = __uint_as_float(w0 << 16), q0 = __uint_as_float(w0 & 0xFFFF0000u);
          const float p1 = __uint_as_float(w1 << 16), q1 = __uint_as_float(w1 & 0xFFFF0000u);
          w0 = pack_bf16x2(p0 * r.x - q0 * r.y, q0 * r.x + p0 * r.y);
          w1 = pack_bf16x2(p1 * r.z - q1 * r.w, q1 * r.z + p1 * r.w);
        } else {
          const float p0 = __uint_as_float(uw[e] << 16), p1 = __uint_as_float(uw[e] & 0xFFFF0000u);
          const float q0 = __uint_as_float(ww[e] << 16), q1 = __uint_as_float(ww[e] & 0xFFFF0000u);
          uw[e] = pack_bf16x2(p0 * r.x - q0 * r.y, p1 * r.z - q1 * r.w);
          ww[e] = pack_bf16x2(q0 * r.x + p0 * r.y, q1 * r.z + p1 * r.w);
        }
      }
    }
    *reinterpret_cast<uint4*>(dst + c0 * 16) = u;
    *reinterpret_cast<uint4*>(dst + c1 * 16) = w;
  }
}

template <int D, bool IL>
cudaError_t launch_d(const RopeAppendLaunch& p, const Args& a, cudaStream_t s) {
  // Items per CTA: ten a thread where that still makes eight CTAs per SM, which
  // spreads a token's sequence search and angles over more bytes; else two or
  // three, for more CTAs at once.
  const int64_t per_tok = (int64_t)((p.q ? p.H : 0) + 2 * p.G) * (D / 16);
  const int64_t want = p.T * per_tok >= (int64_t)p.num_sms * 8 * 10 * kThreads ? 10 * kThreads
                                                                              : 5 * kThreads / 2;
  int tok = 1;
  while (tok < kMaxTok && 2 * tok * per_tok <= want) tok *= 2;
  const unsigned ctas = (unsigned)((p.T + tok - 1) / tok) + a.checks;
  if (!a.checked) {
    const cudaError_t e = cudaMemsetAsync(p.err, 0, sizeof(uint32_t), s);
    if (e != cudaSuccess) return e;
  }
  rope_append_kernel<D, IL><<<ctas, kThreads, 0, s>>>(a, tok);
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
  a.checked = p.B <= kThreads;
  a.checks = (p.B + kThreads - 1) / kThreads;
  if (p.d == 128) return p.interleaved ? launch_d<128, true>(p, a, s) : launch_d<128, false>(p, a, s);
  return p.interleaved ? launch_d<64, true>(p, a, s) : launch_d<64, false>(p, a, s);
}

}  // namespace msa
