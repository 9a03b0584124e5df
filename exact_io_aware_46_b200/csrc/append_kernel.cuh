// append_kernel.cuh -- appending new tokens' keys and values to a paged cache,
// with the rotary position rotation applied on the way.
//
// Token t of sequence b goes to cache row r = k_lens[b] - n_b + i (n_b new
// tokens, t the i-th of them), which is also its position.  A head row of d
// elements consists of `maps` parts (one, or the two halves of a differential
// head), and the first `rope` elements of each part are rotated in pairs:
//   y_a = x_a cos(r, p) - x_b sin(r, p),   y_b = x_b cos(r, p) + x_a sin(r, p),
// with (a, b) = (p, p + rope / 2), or (2p, 2p + 1) when interleaved.  The cosines
// and sines come from the caller's fp32 tables, so any frequency scaling is the
// caller's; products and sums are fp32, rounded once to bf16.  V is copied.
//
// HBM-bound: each element is read once and written once.  A head row is D / 16
// units of two 16-byte chunks, chosen so that neighbouring lanes hold neighbouring
// chunks (64 to 128 bytes a run) in either pairing: a rotated unit of the split
// pairing is the two chunks that rotate into each other, rope / 2 apart.  A thread
// keeps its unit while it walks the token's head rows, so its 16 fp32 cosines and
// sines are read once per token instead of once per row (twice the row's own bytes).
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "launch_cache.cuh"
#include "sm100.cuh"

namespace attn_append_impl {

struct Params {
  const __nv_bfloat16 *Q, *K, *V;  // [T][heads][d] with the token strides below; Q may be nullptr
  long long q_stride, k_stride, v_stride;  // elements between tokens
  __nv_bfloat16* Q_out;                    // [T][Hq][d]
  __nv_bfloat16 *Kp, *Vp;                  // [n_pages][Hkv][page][d]
  const int* block_table;                  // [B][max_blocks]
  const int* cu;                           // [B + 1], or nullptr: token t is sequence t
  const int* k_lens;                       // [B], rows after the append
  const float *cos_t, *sin_t;              // [n_pos][rope / 2]
  int* status;
  int B, T, Hq, Hkv, max_blocks, page_log2, n_pages, n_pos, rope, maps, interleaved;
  int q_rows;      // Hq, or 0 without Q
  int rows_per_y;  // head rows (Q, then K, then V) of a token that one block walks
};

// Small blocks: a block's index loads are a chain (offsets, length, block table), which others
// cover.  Measured on B200 (40,897 packed tokens, Hq = Hkv = 16, d = 128, interleaved, 1.0 GB):
// 256 threads 213 us, 128 172 us, 64 167 us (6.0 TB/s; a copy of as many bytes 156 us).
constexpr int NTHREADS = 64;
constexpr int BAD_KLEN = 1, BAD_PAGE = 4;  // device status bits

// The sequence that token t belongs to: the number of sequences ending at or
// before t (B when t lies behind the last one).  One warp, 32 offsets a step.
__device__ __forceinline__ int find_sequence(const int* cu, int B, int t) {
  int lo = 0, n = B;  // the answer is in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lo + (static_cast<int>(sm100::lane_id()) + 1) * step;  // ends of the strides
    const bool before = i <= lo + n && __ldg(cu + i) <= t;
    const int k = __popc(__ballot_sync(0xffffffffu, before));
    const int rest = lo + n;
    lo += k * step;
    n = min(step - 1, rest - lo);
  }
  return lo;
}

// Sixteen bytes that nothing else will read; not the read-only path, since Q may be
// rotated in place.
__device__ __forceinline__ uint4 load_once(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int D>
__global__ void __launch_bounds__(NTHREADS) append_kernel(const Params p) {
  sm100::grid_launch_dependents();  // launches overlap; nothing is read or written before the wait
  sm100::grid_wait();
  constexpr int UPR = D / 16;               // units per head row
  constexpr int LANES = NTHREADS / UPR;     // head rows a block handles at a time
  const int t = blockIdx.x;
  const int u = threadIdx.x % UPR;
  const int row_end = min((static_cast<int>(blockIdx.y) + 1) * p.rows_per_y, p.q_rows + 2 * p.Hkv);
  int row = blockIdx.y * p.rows_per_y + threadIdx.x / UPR;

  // this thread's unit: its two chunks, of its part's pc chunks (rc of them rotated)
  const int part = D / p.maps, pc = part / 8, rc = p.rope / 8;
  const int m = u / (pc / 2), w = u % (pc / 2);
  int ca, cb;         // chunks within the part
  bool rot_a, rot_b;  // rotated
  if (p.interleaved || w >= rc / 2) {
    // pairs lie within a chunk, or nothing is rotated: chunks half the range apart
    const int lo = p.interleaved ? 0 : rc, half = (pc - lo) / 2;
    ca = lo + w - (p.interleaved ? 0 : rc / 2);
    cb = ca + half;
    rot_a = ca < rc;
    rot_b = cb < rc;
  } else {
    ca = w;
    cb = w + rc / 2;
    rot_a = rot_b = true;
  }
  const int a_off = m * part + 8 * ca, b_off = m * part + 8 * cb;

  auto source = [&](int r) -> const __nv_bfloat16* {
    if (r < p.q_rows) return p.Q + t * p.q_stride + static_cast<long long>(r) * D;
    r -= p.q_rows;
    if (r < p.Hkv) return p.K + t * p.k_stride + static_cast<long long>(r) * D;
    return p.V + t * p.v_stride + static_cast<long long>(r - p.Hkv) * D;
  };
  // the first row's data is requested before the chain of index loads
  uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
  if (row < row_end) {
    const __nv_bfloat16* s = source(row);
    a = load_once(s + a_off);
    b = load_once(s + b_off);
  }

  // sequence, cache row and page of the token (uniform over the block)
  int seq = t, first = t, n_new = 1;
  bool ok = true;
  if (p.cu) {
    seq = find_sequence(p.cu, p.B, t);
    if (seq >= p.B) ok = false;  // behind the last sequence: nothing is written
    if (ok) {
      first = __ldg(p.cu + seq);
      const int end = __ldg(p.cu + seq + 1);
      n_new = end - first;
      ok = first >= 0 && first <= t && t < end && end <= p.T;
    }
  }
  const long long cap = static_cast<long long>(p.max_blocks) << p.page_log2;
  int r = 0, pg = 0;
  if (ok) {
    const int kl = __ldg(p.k_lens + seq);
    r = kl - n_new + (t - first);
    ok = kl >= n_new && kl <= cap && (p.rope == 0 || r < p.n_pos);
    if (!ok && threadIdx.x == 0) atomicOr(p.status, BAD_KLEN);
  }
  if (ok) {
    pg = __ldg(p.block_table + static_cast<size_t>(seq) * p.max_blocks + (r >> p.page_log2));
    ok = pg >= 0 && pg < p.n_pages;
    if (!ok && threadIdx.x == 0) atomicOr(p.status, BAD_PAGE);
  }
  if (ok) {
    // four angles of each chunk's pairs (interleaved), or the eight that both share
    float c[8], s[8];
    if (rot_a || rot_b) {
      const size_t row_at = static_cast<size_t>(r) * (p.rope / 2);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int first4 = p.interleaved ? 4 * (v ? cb : ca) : 8 * ca + 4 * v;
        float4 cv = make_float4(1.f, 1.f, 1.f, 1.f), sv = make_float4(0.f, 0.f, 0.f, 0.f);
        if (v ? rot_b : rot_a) {
          cv = __ldg(reinterpret_cast<const float4*>(p.cos_t + row_at + first4));
          sv = __ldg(reinterpret_cast<const float4*>(p.sin_t + row_at + first4));
        }
        c[4 * v] = cv.x; c[4 * v + 1] = cv.y; c[4 * v + 2] = cv.z; c[4 * v + 3] = cv.w;
        s[4 * v] = sv.x; s[4 * v + 1] = sv.y; s[4 * v + 2] = sv.z; s[4 * v + 3] = sv.w;
      }
    }
    const int in_page = r & ((1 << p.page_log2) - 1);
    while (row < row_end) {
      __nv_bfloat16* dst;
      bool turn_a = rot_a, turn_b = rot_b;
      if (row < p.q_rows) {
        dst = p.Q_out + (static_cast<size_t>(t) * p.Hq + row) * D;
      } else {
        int h = row - p.q_rows;
        const bool is_v = h >= p.Hkv;
        if (is_v) h -= p.Hkv;
        turn_a = rot_a && !is_v;
        turn_b = rot_b && !is_v;
        dst = (is_v ? p.Vp : p.Kp) +
              (((static_cast<size_t>(pg) * p.Hkv + h) << p.page_log2) + in_page) * D;
      }
      const int next = row + LANES;
      uint4 na = a, nb = b;
      if (next < row_end) {  // the next row's data before this row's arithmetic
        const __nv_bfloat16* sp = source(next);
        na = load_once(sp + a_off);
        nb = load_once(sp + b_off);
      }
      if (turn_a || turn_b) {
        uint32_t* av = reinterpret_cast<uint32_t*>(&a);
        uint32_t* bv = reinterpret_cast<uint32_t*>(&b);
        auto lo = [](uint32_t x) { return __uint_as_float(x << 16); };
        auto hi = [](uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); };
        if (p.interleaved) {  // a word is one pair
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float xa = lo(av[e]), ya = hi(av[e]), xb = lo(bv[e]), yb = hi(bv[e]);
            if (turn_a) av[e] = sm100::pack_bf16x2(xa * c[e] - ya * s[e], ya * c[e] + xa * s[e]);
            if (turn_b)
              bv[e] = sm100::pack_bf16x2(xb * c[4 + e] - yb * s[4 + e],
                                         yb * c[4 + e] + xb * s[4 + e]);
          }
        } else {  // element e of the first chunk pairs with element e of the second
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x0 = lo(av[e]), x1 = hi(av[e]), y0 = lo(bv[e]), y1 = hi(bv[e]);
            av[e] = sm100::pack_bf16x2(x0 * c[2 * e] - y0 * s[2 * e],
                                       x1 * c[2 * e + 1] - y1 * s[2 * e + 1]);
            bv[e] = sm100::pack_bf16x2(y0 * c[2 * e] + x0 * s[2 * e],
                                       y1 * c[2 * e + 1] + x1 * s[2 * e + 1]);
          }
        }
      }
      *reinterpret_cast<uint4*>(dst + a_off) = a;
      *reinterpret_cast<uint4*>(dst + b_off) = b;
      a = na;
      b = nb;
      row = next;
    }
  }
  // the offsets as a whole, once, and the lengths of sequences without new tokens: one that
  // breaks the rules may own no token
  if (p.cu && blockIdx.x == 0 && blockIdx.y == 0) {
    bool bad = threadIdx.x == 0 && __ldg(p.cu) != 0;
    for (int i = threadIdx.x; i < p.B; i += NTHREADS) {
      const int c0 = __ldg(p.cu + i), c1 = __ldg(p.cu + i + 1);
      bad |= c0 < 0 || c1 < c0 || c1 > p.T;
      if (c0 == c1) {
        const int kl = __ldg(p.k_lens + i);
        bad |= kl < 0 || kl > cap;
      }
    }
    if (bad) atomicOr(p.status, BAD_KLEN);
  }
}

// Small launches spread a token's head rows over blocks, one row per thread, for
// latency; large ones give a block the whole token, so its angles are read once.
inline int rows_per_block(int T, int rows, int lanes, int sms) {
  const long long spread = static_cast<long long>(T) * ((rows + lanes - 1) / lanes);
  return spread <= 4LL * sms ? lanes : rows;
}

template <int D>
cudaError_t launch_d(Params p, int sms, cudaStream_t s) {
  constexpr int LANES = NTHREADS / (D / 16);
  const int rows = p.q_rows + 2 * p.Hkv;
  p.rows_per_y = rows_per_block(p.T, rows, LANES, sms);
  const dim3 grid(p.T, (rows + p.rows_per_y - 1) / p.rows_per_y);
  return attn_host::launch_overlapped(append_kernel<D>, grid, dim3(NTHREADS), 0, s, p);
}

inline cudaError_t launch(const Params& p, int d, int sms, cudaStream_t s) {
  return d == 128 ? launch_d<128>(p, sms, s) : launch_d<64>(p, sms, s);
}

}  // namespace attn_append_impl
