// diff_bwd_kernel.cuh -- backward of differential attention by recomputation.
//
// Head rows hold the halves of two maps, Q = [q_1 q_2], K = [k_1 k_2], over one V:
//   P_m = exp(scale q_m k_m^T - LSE_m),  O = P_1 V - lam P_2 V,  O_2 = P_2 V.
// With dP = dO V^T (shared by both maps) and D_m = dO . O_m (so D_2 = dO . O_2 and
// D_1 = dO . O + lam D_2) the calculus of the definition gives
//   dV = (P_1 - lam P_2)^T dO,   dS_1 = P_1 o (dP - D_1),  dS_2 = -lam P_2 o (dP - D_2),
//   dq_m = scale dS_m k_m,  dk_m = scale dS_m^T q_m,  dlam = - sum P_2 o dP.
//
// One pass forms both maps from one read of Q, dO, K and V: five GEMMs' worth of
// MMA work per tile, as for one map of the full width, with one dP and one dV
// product instead of two.  Launches, work items (128 keys of one batch and
// key/value head) and their order are those of bwd_kernel.cuh; a 128-row query tile
// is worked as two halves of 64 rows in turn, with keys on the 128 TMEM lanes (a
// half's columns are query rows):
//   S_1^T, S_2^T = K_m Q_m^T   (SS, half the K steps each, one after the other in
//                               the half's 64 columns: S_1 is read out before S_2
//                               is issued)
//   dP^T = V dO^T              (SS, 64 columns)
//   dV  += W^T dO              (TS, W = P_1 - lam P_2 in bf16 over the dP columns)
//   dK_m += dS_m^T Q_m         (N = 64, dS_m staged in shared memory; dS_1 is also put beside
//                               W over the dP columns, so that dK_1 reads it there: TS)
//   dQ_m^T = K_m^T dS_m^T      (SS, M = 64, lanes = head dimension, over the dP columns:
//                               map 1 in lanes 0-15 of each 32, map 2 in lanes 16-31)
// dV (d columns) and dK (64 per map) stay in TMEM for the item: 512 columns in all.
// At d = 64 the maps are 32 columns wide but the dK and dQ products still run over the whole
// 64-column panel, and the half that belongs to the other map is not read: 14 d FLOP are
// executed where 10 d are needed.  dQ's M has no smaller value; dK at N = 32 is not tried.
//
// Warps 0-7 and 8-15 work half 0 and half 1, half a tile apart: one group's scalar
// work (a key row per thread, two warps per row) runs while the tensor core works
// for the other.  Per half and tile a group forms P_1, adds the tile before's dQ^T
// into the fp32 accumulator, and then forms P_2, W and both dS sixteen columns at a
// time, dP at hand, so that 96 registers hold nearly all of it (ptxas: 72 bytes of spill stores
// and 164 of loads a thread at d = 128, 60 and 176 at d = 64).  dQ^T goes out by 4-byte reductions
// that cover 128 contiguous bytes (the accumulator's columns are ordered as the lanes
// are).  Those additions happen at L2, at a rate that no way of sending them changed
// (64 KB per tile and SM in 2.1 us: reductions of 4 bytes a lane 4628 GB/s, bulk
// reduce-adds 4593, tensor reduce-adds 4312; 16 bytes a lane with a row per lane 2484),
// so the way that needs no shared memory was taken.  Warp 16 feeds K, V and Q by TMA,
// warps 18 and 19 a half's statistics and dO each, warp 17 issues the MMAs.
//
// Measured on B200 (causal B2 H16 L8192 d128, calls timed alone; one after another the kernel
// draws the card's power limit and takes a sixth longer): dQ staged in the dS buffers and one tile
// at a time 2715 us; dQ by reductions 2392; halves in turn 2031; fewer waits and no
// divisions 1869; P_2 and dS in one go 1672; dK_1 by TS 1637; set-up overlapped with the
// kernel before 1601; P_1 kept as scaled fp16 1638 (for its precision).  What bounds it now is
// not established.  A 128-row tile takes ~6300 cycles.  Counted in cycles of shared memory its
// products' operands take 3250 (416 KB), the copies in 512, dS 512 and the statistics' reads
// (a wavefront a value and warp) 2048, as many in all; but without those reads (timing only) it
// ran 1.6 % faster, so they do not simply add up.  The tensor pipe is 51 % active and 68 % busy
// on its issue side, the special-function unit 35 %, issue 43 %.
//
// dlam needs more of P_2 than bf16 gives: its terms P_2 dP have both signs, and
// the roundings of P_2 (2^-9 relative on average) do not shrink with the sum.
// The sums take P_2 in fp32, as it comes from the exponential.  Sums per (item, head,
// warp) go to the workspace and are added in a fixed order, in fp64, so dlam is the same
// from run to run.  It is rounded once, to bf16 like every gradient of this library (2^-8 of
// the sum at most): callers that accumulate over several calls add in a type of their own.
#pragma once

#include <cuda_fp16.h>

#include <climits>
#include <cmath>
#include <cstring>

#include "bwd_kernel.cuh"

namespace attn_diff_bwd_impl {

using attn_bwd_impl::BMQ;
using attn_bwd_impl::BN;
using attn_bwd_impl::get_item;
using attn_bwd_impl::Item;
using attn_bwd_impl::NI;
using attn_bwd_impl::PANEL;
using attn_bwd_impl::st_global_v8;
using attn_bwd_impl::tile_of;

constexpr int NSMX = 16;  // P/dS warps: 4 lane quarters x 4 quarters of the query rows
constexpr int W_LOAD = NSMX;
constexpr int W_MMA = NSMX + 1;
constexpr int W_HALF = NSMX + 2;  // two warps: each half's statistics and dO
constexpr int NTHREADS = 32 * (NSMX + 4);
constexpr int ITEM_READERS = NSMX + 3;
constexpr int NQS = 2;  // Q ring stages

template <int DH>
struct Cfg {
  static_assert(DH == 64 || DH == 128, "head dimension");
  static constexpr int PANELS = DH / 64;
  static constexpr int TILE = PANELS * PANEL;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = TILE;
  static constexpr int OFF_Q = 2 * TILE;             // NQS stages
  static constexpr int OFF_DO = OFF_Q + NQS * TILE;
  static constexpr int OFF_DS = OFF_DO + TILE;       // dS_1^T, dS_2^T: two panels of 64 rows each
  static constexpr int OFF_LD = OFF_DS + 4 * PANEL;  // [half] -lse2_1, -lse2_2, -D_1, lam D_2: [64]
  static constexpr int OFF_BAR = OFF_LD + 2048;
  static constexpr int SMEM_BYTES = OFF_BAR + 512;
  static_assert(SMEM_BYTES <= 232448, "dynamic shared memory limit");
  static constexpr uint32_t IDESC_DV = sm100::idesc_bf16_f32(128, DH, false, true);
};
constexpr int HQ = 64;             // query rows of a half tile, the unit of each warp group
constexpr int HROWS = HQ * 128;    // bytes of 64 rows of a swizzle panel
constexpr uint32_t IDESC_S = sm100::idesc_bf16_f32(128, HQ, false, false);
constexpr uint32_t IDESC_DK = sm100::idesc_bf16_f32(128, 64, false, true);
constexpr uint32_t IDESC_DQ = sm100::idesc_bf16_f32(64, HQ, true, true);

// Where column c of a dQ row lies in the accumulator's row: the order of the TMEM lanes of
// dQ^T, so that a warp's 32 lanes add into 128 contiguous bytes (d = 64: the natural order,
// a half-warp adds 64 bytes).
template <int DH>
__host__ __device__ constexpr int acc_pos(int c) {
  return DH == 128 ? 32 * ((c & 63) >> 4) + 16 * (c >> 6) + (c & 15) : c;
}

// TMEM columns
constexpr uint32_t S_COL = 0;     // S_m^T
constexpr uint32_t DP_COL = 128;  // dP^T; W^T and dS_1^T (8 of every 16 columns each); dQ^T of both maps
constexpr uint32_t DV_COL = 256;
constexpr uint32_t DK_COL = 384;  // dK_1, dK_2 (64 each)

// All exponentials are on the special-function unit: with polynomials for an eighth or a quarter
// of them the kernel ran 2 to 4 % slower (causal B2 H16 L8192 d128), as issue slots, not that
// unit, are short.

struct Params : attn_bwd_impl::Params {
  // [B*Hq][n_qt][2 halves][4][64]: -lse2_1, -lse2_2 (both plus P_SCALE_LOG2), -D_1, lam D_2
  const float* stats;
  const float* lam;    // [n_lam]
  int n_lam;
  float* lam_part;  // [B*Hkv][n_kv][n_split][G][NSMX] sums of P_2 dP
  int n_split;      // parts that an item's query tiles are shared out to
  float* kv_part;   // n_split > 1: [n_split][B*Hkv*Lk][dV, dK][d] fp32
};

// Part `part` of an item: its query tiles t0 ... t0 + T - 1.
struct Part {
  Item it;
  int part, t0, T;
};
__device__ __forceinline__ Part get_part(const Params& p, int w, bool* bad) {
  Part q;
  q.it = get_item(p, w / p.n_split, bad);
  q.part = w % p.n_split;
  q.t0 = static_cast<int>(static_cast<long long>(q.it.T) * q.part / p.n_split);
  q.T = static_cast<int>(static_cast<long long>(q.it.T) * (q.part + 1) / p.n_split) - q.t0;
  return q;
}

// Every probability is formed 2^14 times too large (in the statistics' exponent), and the
// outputs' factors take that back.  P_1 waits in 16 bits for dP: as fp16 its rounding is
// 2^-12 relative instead of bf16's 2^-9, which would be as large as that of dS itself, and the
// scale keeps that down to probabilities of 4e-9 (one of 1 becomes 16384, of 65504).
constexpr float P_SCALE_LOG2 = 14.f, P_UNSCALE = 1.f / 16384.f;

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) {
  __half2 h;
  memcpy(&h, &v, 4);
  return __half22float2(h);
}

// sm100::mbar_wait by shared address, its slow path out of line: inlined at every wait it cost
// registers that the softmax warps need (1907 against 1957 us).
__device__ __noinline__ bool mbar_wait_slow(uint32_t a, uint32_t parity, volatile int* abort,
                                            int* status, int site) {
  const long long t0 = clock64();
  for (uint32_t it = 0; it < 0x40000000u; ++it) {
    if (sm100::mbar_try_wait(a, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > ATTN_WAIT_CYCLES) break;
  }
  *abort = 1;
  sm100::record_timeout(status, site);
  return false;
}
__device__ __forceinline__ bool mbar_wait_at(uint32_t a, uint32_t parity, volatile int* abort,
                                             int* status, int site) {
  if (sm100::mbar_try_wait(a, parity)) return true;
  return mbar_wait_slow(a, parity, abort, status, site);
}

// Four words to shared memory, free to move among loads (no memory clobber: the statistics read
// around it lie elsewhere); later volatile statements, the proxy fence among them, stay behind.
__device__ __forceinline__ void st_shared_v4(uint32_t at, const uint32_t (&w)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]));
}

// ------------------------------------------------------------------ prep

// D_1, D_2, the log2-LSEs and a zeroed accumulator row of every (padded) query row: DH / 8
// lanes a row, sixteen bytes each of O, O2 and dO.  And zeroed scheduler counters, so that
// a call with query rows works on any workspace.
template <int DH>
__global__ void __launch_bounds__(256)
    prep_kernel(const __nv_bfloat16* O, const __nv_bfloat16* O2, const __nv_bfloat16* dO,
                const float* lse, const float* lam, int n_lam, float* dq_acc, float* stats,
                int* sched, long long rows, int Hq, int Lq, int Lqp) {
  constexpr int LPR = DH / 8;  // lanes per row
  sm100::grid_launch_dependents();
  sm100::grid_wait();
  if (blockIdx.x == 0 && threadIdx.x < 2) sched[threadIdx.x] = 0;
  const long long row = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / LPR;
  const int lane = threadIdx.x % LPR;
  if (row >= rows) return;  // whole rows, and rows is a multiple of 128: whole warps
  const long long bh = row / Lqp;
  const int r = static_cast<int>(row - bh * Lqp);
  float a1 = 0.f, a2 = 0.f;
  if (r < Lq) {
    const size_t off = (static_cast<size_t>(bh) * Lq + r) * DH + lane * 8;
    const uint4 o = __ldg(reinterpret_cast<const uint4*>(O + off));
    const uint4 o2 = __ldg(reinterpret_cast<const uint4*>(O2 + off));
    const uint4 g = __ldg(reinterpret_cast<const uint4*>(dO + off));
    const uint32_t ov[4] = {o.x, o.y, o.z, o.w}, o2v[4] = {o2.x, o2.y, o2.z, o2.w};
    const uint32_t gv[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float g0 = __uint_as_float(gv[e] << 16), g1 = __uint_as_float(gv[e] & 0xFFFF0000u);
      a1 += __uint_as_float(ov[e] << 16) * g0 + __uint_as_float(ov[e] & 0xFFFF0000u) * g1;
      a2 += __uint_as_float(o2v[e] << 16) * g0 + __uint_as_float(o2v[e] & 0xFFFF0000u) * g1;
    }
  }
#pragma unroll
  for (int o = LPR / 2; o >= 1; o >>= 1) {
    a1 += __shfl_xor_sync(0xffffffffu, a1, o);
    a2 += __shfl_xor_sync(0xffffffffu, a2, o);
  }
  float4* zrow = reinterpret_cast<float4*>(dq_acc + static_cast<size_t>(row) * DH);
  zrow[lane] = make_float4(0.f, 0.f, 0.f, 0.f);
  zrow[lane + LPR] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (lane < 4) {
    const int h = static_cast<int>(bh % Hq);
    const float l = __ldg(lam + (n_lam == 1 ? 0 : h));
    float v;
    if (lane < 2) {  // -inf where the row sees no key or lies past Lq: P is exactly 0
      v = r < Lq ? P_SCALE_LOG2 - lse[(static_cast<size_t>(bh) * 2 + lane) * Lq + r] *
                                      1.4426950408889634f
                 : -INFINITY;
      if (v == INFINITY) v = -INFINITY;
    } else {
      v = lane == 2 ? -(a1 + l * a2) : l * a2;
    }
    stats[(static_cast<size_t>(bh) * (Lqp / HQ) + r / HQ) * 256 + lane * HQ + r % HQ] = v;
  }
}

// dQ = bf16(scale * accumulator), eight elements a thread; the blocks behind those that
// convert add up dlam (one block per weight), each warp's sums in a fixed order, and the
// parts' dV and dK where an item was split.
template <int DH>
__global__ void __launch_bounds__(256)
    finish_kernel(const float* dq_acc, __nv_bfloat16* dQ, long long BH, int Lq, int Lqp,
                  float scale, long long conv_blocks, const float* lam_part, __nv_bfloat16* dlam,
                  int B, int Hq, int Hkv, int Lk, int n_lam, int n_split, const float* kv_part,
                  __nv_bfloat16* dK, __nv_bfloat16* dV) {
  // (no launch of the kernel behind from here: a next backward's preparation, resident early,
  // cost 1886 -> 1955 us a backward of causal B2 H16 L8192 d128, one after another)
  sm100::grid_wait();
  const int n_kv = (Lk + BN - 1) / BN;
  if (blockIdx.x >= conv_blocks + n_lam) {
    // dV and dK of the parts, added in their order: eight elements a thread
    const size_t rows = static_cast<size_t>(B) * Hkv * Lk;
    const size_t i = (static_cast<size_t>(blockIdx.x) - conv_blocks - n_lam) * 256 + threadIdx.x;
    if (i >= rows * (DH / 4)) return;
    const size_t row = i / (DH / 4);
    const int m = static_cast<int>(i / (DH / 8)) & 1, c8 = static_cast<int>(i % (DH / 8));
    float a[8] = {};
    for (int k = 0; k < n_split; ++k) {
      const float4* src = reinterpret_cast<const float4*>(
          kv_part + ((k * rows + row) * 2 + m) * DH + 8 * c8);
      const float4 u = src[0], v = src[1];
      a[0] += u.x; a[1] += u.y; a[2] += u.z; a[3] += u.w;
      a[4] += v.x; a[5] += v.y; a[6] += v.z; a[7] += v.w;
    }
    const float f = (m == 0 ? 1.f : scale) * P_UNSCALE;
    uint4 o;
    o.x = sm100::pack_bf16x2(a[0] * f, a[1] * f);
    o.y = sm100::pack_bf16x2(a[2] * f, a[3] * f);
    o.z = sm100::pack_bf16x2(a[4] * f, a[5] * f);
    o.w = sm100::pack_bf16x2(a[6] * f, a[7] * f);
    reinterpret_cast<uint4*>((m == 0 ? dV : dK) + row * DH)[c8] = o;
    return;
  }
  if (blockIdx.x < conv_blocks) {
    scale *= P_UNSCALE;
    const size_t i = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const size_t total = static_cast<size_t>(BH) * Lq * (DH / 8);
    if (i >= total) return;
    const size_t row = i / (DH / 8);
    const int c8 = static_cast<int>(i % (DH / 8));
    const size_t bh = row / Lq, r = row - bh * Lq;
    const float4* src =
        reinterpret_cast<const float4*>(dq_acc + (bh * Lqp + r) * DH + acc_pos<DH>(8 * c8));
    const float4 u = src[0], v = src[1];
    uint4 o;
    o.x = sm100::pack_bf16x2(u.x * scale, u.y * scale);
    o.y = sm100::pack_bf16x2(u.z * scale, u.w * scale);
    o.z = sm100::pack_bf16x2(v.x * scale, v.y * scale);
    o.w = sm100::pack_bf16x2(v.z * scale, v.w * scale);
    reinterpret_cast<uint4*>(dQ + row * DH)[c8] = o;
    return;
  }
  const int w = static_cast<int>(blockIdx.x - conv_blocks);
  const int G = Hq / Hkv;
  // partials [B][Hkv][n_kv][n_split][G][NSMX], read in vectors of four; n_lam == 1 adds all
  constexpr int V4 = NSMX / 4;
  const float4* part4 = reinterpret_cast<const float4*>(lam_part);
  const long long per_head = static_cast<long long>(n_kv) * n_split;
  const long long n = B * per_head * V4 * (n_lam == 1 ? Hq : 1);
  double acc = 0.;
#pragma unroll 4
  for (long long e = threadIdx.x; e < n; e += 256) {
    long long at = e;
    if (n_lam != 1) {
      const long long bn = e / V4;  // batch, key tile and part
      const long long part_at = ((bn / per_head) * Hkv + w / G) * per_head + bn % per_head;
      at = (part_at * G + w % G) * V4 + e % V4;
    }
    const float4 v = part4[at];
    acc += static_cast<double>(v.x) + v.y + v.z + v.w;
  }
  __shared__ double part[256];
  part[threadIdx.x] = acc;
  __syncthreads();
  for (int o = 128; o >= 1; o >>= 1) {
    if (threadIdx.x < o) part[threadIdx.x] += part[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0)
    dlam[w] = __float2bfloat16_rn(static_cast<float>(-part[0] * P_UNSCALE));
}

// ------------------------------------------------------------------ main

template <int DH>
__global__ void __launch_bounds__(NTHREADS, 1)
    main_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
                const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const Params p) {
  using C = Cfg<DH>;
  // the swizzle panels need 1024-byte alignment; at d = 128 there is no room to align by hand
  extern __shared__ __align__(1024) uint8_t smem_diff[];
  uint8_t* smem = smem_diff;
  const uint32_t sbase = sm100::smem_u32(smem);
  if (sbase & 1023) {  // never with this declaration; nothing could be computed
    if (threadIdx.x == 0) sm100::record_timeout(p.status, 40);
    return;
  }

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* kv_full = bars + 0;
  uint64_t* kv_empty = bars + 1;
  uint64_t* dkv_full = bars + 2;
  uint64_t* dkv_empty = bars + 3;
  uint64_t* drain = bars + 4;
  uint64_t* item_full = bars + 5;   // [NI]
  uint64_t* item_empty = bars + 9;  // [NI]
  // of each half tile's pipeline h
  auto half_bar = [&](int h, int i) -> uint64_t* { return bars + 13 + 13 * h + i; };
  auto q_full = [&](int h, uint32_t tile) { return half_bar(h, tile % NQS); };
  auto q_empty = [&](int h, uint32_t tile) { return half_bar(h, 2 + tile % NQS); };
  auto do_full = [&](int h) { return half_bar(h, 4); };
  auto do_empty = [&](int h) { return half_bar(h, 5); };
  auto s1_full = [&](int h) { return half_bar(h, 6); };  // S_1, and -lse2_1 has landed
  auto s1_read = [&](int h) { return half_bar(h, 7); };
  auto s2_read = [&](int h) { return half_bar(h, 8); };  // frees the -lse2_1 as well
  // dP and S_2, the dS buffer is free (the products of the dS before precede dP), and the
  // other three statistics have landed
  auto dp_full = [&](int h) { return half_bar(h, 9); };
  auto ds_full = [&](int h) { return half_bar(h, 10); };  // dS and W; frees those three
  auto dq_full = [&](int h) { return half_bar(h, 11); };
  auto dq_empty = [&](int h) { return half_bar(h, 12); };  // the dP columns: dQ has left
  int* item_ring = reinterpret_cast<int*>(bars + 39);  // [NI]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(item_ring + NI);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert(39 * 8 + NI * 4 + 8 <= 512, "barrier area");

  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    auto init = [](uint64_t* b, uint32_t n) { sm100::mbar_init(b, n); };
    init(kv_full, 1);
    init(kv_empty, 1);
    init(dkv_full, 1);
    init(dkv_empty, NSMX);
    init(drain, 1);
    for (int i = 0; i < NI; ++i) {
      init(&item_full[i], 1);
      init(&item_empty[i], ITEM_READERS);
    }
    for (int h = 0; h < 2; ++h) {
      for (uint32_t i = 0; i < NQS; ++i) {
        init(q_full(h, i), 1);
        init(q_empty(h, i), 1);
      }
      init(do_full(h), 1);
      init(do_empty(h), 1);
      init(s1_full(h), 2);  // the product's commit and the statistics' copy
      init(s1_read(h), NSMX / 2);
      init(s2_read(h), NSMX / 2);
      init(dp_full(h), 2);
      init(ds_full(h), NSMX / 2);
      init(dq_full(h), 1);
      init(dq_empty(h), NSMX / 2);
    }
    *abort_flag = 0;
    sm100::fence_barrier_init();
  }
  if (warp == W_LOAD && sm100::lane_id() == 0) {
    sm100::prefetch_tmap(&tmQ);
    sm100::prefetch_tmap(&tmdO);
    sm100::prefetch_tmap(&tmK);
    sm100::prefetch_tmap(&tmV);
  }
  if (warp == W_MMA) {
    sm100::tmem_alloc(tmem_slot, 512);
    sm100::tmem_relinquish();
  }
  // the set-up so far ran beside the preparation's end; its statistics and zeroes are used from here
  sm100::grid_wait();
  sm100::grid_launch_dependents();
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int off = p.Lk - p.Lq;  // bottom-right causal alignment
  auto wait = [&](uint64_t* b, uint32_t parity, int site) -> bool {
    return mbar_wait_at(sm100::smem_u32(b), parity, abort_flag, p.status, site);
  };
  auto next_item = [&](uint32_t k, int& w) -> bool {
    if (!wait(&item_full[k % NI], (k / NI) & 1, 41)) return false;
    w = *reinterpret_cast<volatile int*>(&item_ring[k % NI]);
    __syncwarp();
    if (sm100::lane_id() == 0) sm100::mbar_arrive(&item_empty[k % NI]);
    return true;
  };

  if (warp == W_LOAD) {
    // ------------------------------------------------------------ TMA producer
    // the items, K and V of each, and Q of each query tile (a two-stage ring per half)
    if (sm100::lane_id() == 0) {
      uint32_t tq = 0, ik = 0, kv_issued = 0, n_q[2] = {0, 0};
      bool ok = true;
      for (; ok; ++ik) {
        if (!(ok = wait(&item_empty[ik % NI], ((ik / NI) & 1) ^ 1, 42))) break;
        int w = (ik == 0) ? static_cast<int>(blockIdx.x)
                          : atomicAdd(p.sched, 1) + static_cast<int>(gridDim.x);
        if (w >= p.n_items) w = -1;
        *reinterpret_cast<volatile int*>(&item_ring[ik % NI]) = w;
        sm100::mbar_arrive(&item_full[ik % NI]);
        if (w < 0) break;
        const Part pt = get_part(p, w, nullptr);
        const Item& it = pt.it;
        if (!(ok = wait(kv_empty, (ik & 1) ^ 1, 43))) break;
        sm100::mbar_arrive_expect_tx(kv_full, 2 * C::TILE);
        ++kv_issued;
        const int kvh = it.b * p.Hkv + it.hkv;
        for (int c = 0; c < C::PANELS; ++c) {
          sm100::tma_load_3d(&tmK, kv_full, smem + C::OFF_K + c * PANEL, c * 64, it.n * BN, kvh);
          sm100::tma_load_3d(&tmV, kv_full, smem + C::OFF_V + c * PANEL, c * 64, it.n * BN, kvh);
        }
        const int nq = it.T > 0 ? it.T / p.G : 0;
        for (int t = pt.t0; t < pt.t0 + pt.T && ok; ++t, ++tq) {
          int g, i;
          tile_of(it, t, nq, g, i);
          for (int h = 0; h < 2; ++h) {
            if (!(ok = wait(q_empty(h, tq), ((tq / NQS) & 1) ^ 1, 44))) break;
            sm100::mbar_arrive_expect_tx(q_full(h, tq), C::TILE / 2);
            for (int c = 0; c < C::PANELS; ++c)
              sm100::tma_load_3d(&tmQ, q_full(h, tq),
                                 smem + C::OFF_Q + (tq % NQS) * C::TILE + c * PANEL + h * HROWS,
                                 c * 64, i * BMQ + h * HQ, it.b * p.Hq + it.hkv * p.G + g);
            ++n_q[h];
          }
        }
      }
      // the CTA must not exit while copies still land in its shared memory, which an
      // expired wait elsewhere could otherwise allow
      if (kv_issued > 0) sm100::mbar_wait_drain(kv_full, (kv_issued - 1) & 1);
      for (int h = 0; h < 2; ++h)
        for (uint32_t k = n_q[h] > NQS ? n_q[h] - NQS : 0; k < n_q[h]; ++k)
          sm100::mbar_wait_drain(q_full(h, k), (k / NQS) & 1);
    }
  } else if (warp >= W_HALF) {
    // ------------------------------------------------------------ a half's statistics and dO
    // each into a single buffer that the half's tile before has left by then
    const int h = warp - W_HALF;
    uint8_t* ld = smem + C::OFF_LD + h * 1024;
    uint32_t tq = 0, n_l = 0, n_do = 0, n_d = 0;
    bool ok = true;
    for (uint32_t ik = 0; ok; ++ik) {
      int w;
      if (!(ok = next_item(ik, w)) || w < 0) break;
      if (sm100::lane_id() == 0) {
        const Part pt = get_part(p, w, nullptr);
        const Item& it = pt.it;
        const int nq = it.T > 0 ? it.T / p.G : 0;
        for (int t = pt.t0; t < pt.t0 + pt.T && ok; ++t, ++tq) {
          int g, i;
          tile_of(it, t, nq, g, i);
          const int qh = it.b * p.Hq + it.hkv * p.G + g;
          const uint32_t par = (tq & 1) ^ 1;
          const float* st = p.stats + (static_cast<size_t>(qh) * p.n_qt + i) * 512 + h * 256;
          if (!(ok = wait(s2_read(h), par, 45))) break;
          sm100::mbar_arrive_expect_tx(s1_full(h), 256);
          attn_bwd_impl::bulk_g2s(ld, st, 256, s1_full(h));
          ++n_l;
          if (!(ok = wait(ds_full(h), par, 47))) break;
          sm100::mbar_arrive_expect_tx(dp_full(h), 768);
          attn_bwd_impl::bulk_g2s(ld + 256, st + 64, 768, dp_full(h));
          ++n_d;
          if (!(ok = wait(do_empty(h), par, 46))) break;
          sm100::mbar_arrive_expect_tx(do_full(h), C::TILE / 2);
          for (int c = 0; c < C::PANELS; ++c)
            sm100::tma_load_3d(&tmdO, do_full(h), smem + C::OFF_DO + c * PANEL + h * HROWS, c * 64,
                               i * BMQ + h * HQ, qh);
          ++n_do;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (sm100::lane_id() == 0) {
      if (n_l > 0) sm100::mbar_wait_drain(s1_full(h), (n_l - 1) & 1);
      if (n_do > 0) sm100::mbar_wait_drain(do_full(h), (n_do - 1) & 1);
      if (n_d > 0) sm100::mbar_wait_drain(dp_full(h), (n_d - 1) & 1);
    }
  } else if (warp == W_MMA) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = sm100::elect_one();
    uint32_t tq = 0, ik = 0;
    bool ok = true;
    const uint32_t kA = sbase + C::OFF_K, vA = sbase + C::OFF_V, doA = sbase + C::OFF_DO;
    auto qA = [&](uint32_t tile) { return sbase + C::OFF_Q + (tile % NQS) * C::TILE; };
    auto commit = [&](uint64_t* bar) {
      if (leader) sm100::tc_commit(bar);
      __syncwarp();
    };
    // S_m^T of half h: both operands K-major, map m's half of the columns (its own panel at
    // d = 128, 64 bytes into the rows at d = 64)
    constexpr uint32_t MHALF = DH == 128 ? PANEL : 64;
    auto issue_s = [&](uint32_t tile, int h, int m) {
      const uint64_t ad = sm100::sdesc_sw128(kA + m * MHALF, 16, 1024);
      const uint64_t bd = sm100::sdesc_sw128(qA(tile) + m * MHALF + h * HROWS, 16, 1024);
      if (leader) {
#pragma unroll
        for (int k = 0; k < DH / 32; ++k)
          sm100::mma_ss(tmem + S_COL + HQ * h, ad + 2 * k, bd + 2 * k, IDESC_S, k > 0);
      }
    };
    auto issue_dp = [&](int h) {  // dP^T = V dO^T
      const uint64_t ad = sm100::sdesc_sw128(vA, 16, 1024);
      const uint64_t bd = sm100::sdesc_sw128(doA + h * HROWS, 16, 1024);
      if (leader) {
#pragma unroll
        for (int k = 0; k < DH / 16; ++k) {
          const uint64_t o = static_cast<uint64_t>(((k >> 2) * PANEL + (k & 3) * 32) >> 4);
          sm100::mma_ss(tmem + DP_COL + HQ * h, ad + o, bd + o, IDESC_S, k > 0);
        }
      }
    };
    auto issue_dv = [&](int h, bool first) {  // W: sixteen rows are 8 of every 16 columns
      const uint64_t bd = sm100::sdesc_sw128(doA + h * HROWS, PANEL, 1024);
      if (leader) {
#pragma unroll
        for (int k = 0; k < HQ / 16; ++k)
          sm100::mma_ts(tmem + DV_COL, tmem + DP_COL + HQ * h + 16 * k,
                        bd + ((k * 2048) >> 4), C::IDESC_DV, (!first || k > 0) ? 1u : 0u);
      }
    };
    // dK_m += dS_m^T Q_m (K steps of 16 rows) and dQ_m^T = K_m^T dS_m^T (of 16 keys); at d = 64
    // both maps multiply the one 64-column panel
    constexpr uint32_t MPANEL = DH == 128 ? PANEL : 0;
    auto ds_at = [&](int h, int m) { return sbase + C::OFF_DS + (m * 2 + h) * PANEL; };
    auto issue_dk = [&](uint32_t tile, int h, int m, bool first) {
      const uint64_t ad = sm100::sdesc_sw128(ds_at(h, m), 16, 1024);
      const uint64_t bd = sm100::sdesc_sw128(qA(tile) + m * MPANEL + h * HROWS, PANEL, 1024);
      if (leader) {
#pragma unroll
        for (int k = 0; k < HQ / 16; ++k)
          sm100::mma_ss(tmem + DK_COL + 64 * m, ad + 2 * k, bd + ((k * 2048) >> 4), IDESC_DK,
                        (!first || k > 0) ? 1u : 0u);
      }
    };
    auto issue_dk1_ts = [&](uint32_t tile, int h, bool first) {  // dS_1 from the dP columns
      const uint64_t bd = sm100::sdesc_sw128(qA(tile) + h * HROWS, PANEL, 1024);
      if (leader) {
#pragma unroll
        for (int k = 0; k < HQ / 16; ++k)
          sm100::mma_ts(tmem + DK_COL, tmem + DP_COL + HQ * h + 16 * k + 8, bd + ((k * 2048) >> 4),
                        IDESC_DK, (!first || k > 0) ? 1u : 0u);
      }
    };
    auto issue_dq = [&](int h, int m) {
      const uint64_t bd = sm100::sdesc_sw128(ds_at(h, m), PANEL, 1024);
      const uint64_t ad = sm100::sdesc_sw128(kA + m * MPANEL, PANEL, 1024);
      if (leader) {
#pragma unroll
        for (int k = 0; k < BN / 16; ++k)
          sm100::mma_ss(tmem + DP_COL + HQ * h + (static_cast<uint32_t>(16 * m) << 16),
                        ad + ((k * 2048) >> 4), bd + ((k * 2048) >> 4), IDESC_DQ,
                        k > 0 ? 1u : 0u);
      }
    };
    // K and V rows at and past the sequence's end (kv_len < Lk) may hold anything:
    // cleared, so that their zero dS and P meet zeros
    auto clear_tail = [&](int from) {
      for (int e = from * 8 + sm100::lane_id(); e < BN * 8; e += 32)
        for (int c = 0; c < C::PANELS; ++c) {
          *reinterpret_cast<uint4*>(smem + C::OFF_K + c * PANEL + e * 16) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(smem + C::OFF_V + c * PANEL + e * 16) = make_uint4(0, 0, 0, 0);
        }
      sm100::fence_proxy_async_smem();
      __syncwarp();
    };
    for (; ok; ++ik) {
      int w;
      if (!(ok = next_item(ik, w)) || w < 0) break;
      const Part pt = get_part(p, w, nullptr);
      const Item& it = pt.it;
      const int T = pt.T;
      if (!(ok = wait(kv_full, ik & 1, 48))) break;
      sm100::tc_fence_after();
      if (T == 0) {
        if (!(ok = wait(dkv_empty, (ik & 1) ^ 1, 49))) break;
        commit(dkv_full);
        commit(kv_empty);
        continue;
      }
      if (it.kv_len < p.Lk && it.kv_len < (it.n + 1) * BN) clear_tail(it.kv_len - it.n * BN);
      // S_1 of a half's tile (its S columns are free: S_2 of the tile before has been read)
      auto first_s = [&](uint32_t tile, int h) -> bool {
        if (!wait(q_full(h, tile), (tile / NQS) & 1, 50)) return false;
        sm100::tc_fence_after();
        issue_s(tile, h, 0);
        commit(s1_full(h));
        return true;
      };
      // dV of W and then both dQ of dS, over the columns that W was in
      auto dv_dq = [&](int t, int h) -> bool {
        if (!wait(ds_full(h), (tq + t) & 1, 51)) return false;
        const bool first = t == 0 && h == 0;
        if (first && !wait(dkv_empty, (ik & 1) ^ 1, 56)) return false;
        sm100::tc_fence_after();
        issue_dv(h, first);
        commit(do_empty(h));
        issue_dk1_ts(tq + t, h, first);
        issue_dq(h, 0);
        issue_dq(h, 1);
        commit(dq_full(h));
        return true;
      };
      auto both_dk = [&](int t, int h) {
        const bool first = t == 0 && h == 0;
        issue_dk(tq + t, h, 1, first);
        commit(q_empty(h, tq + t));
      };
      auto second_s = [&](int t, int h) -> bool {
        if (!wait(s1_read(h), (tq + t) & 1, 52)) return false;
        sm100::tc_fence_after();
        issue_s(tq + t, h, 1);
        if (t > 0) both_dk(t - 1, h);
        return true;
      };
      auto first_dp = [&](int t, int h) -> bool {
        const uint32_t cur = tq + t;
        if (!wait(do_full(h), cur & 1, 53)) return false;
        if (!wait(dq_empty(h), (cur & 1) ^ 1, 54)) return false;
        sm100::tc_fence_after();
        issue_dp(h);
        commit(dp_full(h));
        return true;
      };
      auto next_s = [&](int t, int h) -> bool {
        if (t + 1 >= T) return true;
        return wait(s2_read(h), (tq + t) & 1, 55) && first_s(tq + t + 1, h);
      };
      // Issue order: half 1 runs half a tile behind half 0, so that one half's softmax warps
      // have the tensor core's results of theirs while it works for the other:
      //   dV_0 dQ_0(t-1) S2_0(t) dK_0(t-1) | S1_1(t) | dP_0(t) |
      //   dV_1 dQ_1(t-1) S2_1(t) dK_1(t-1) | S1_0(t+1) | dP_1(t)
      if (!(ok = first_s(tq, 0))) break;
      for (int t = 0; t < T && ok; ++t)
        ok = (t == 0 || dv_dq(t - 1, 0)) && second_s(t, 0) &&
             (t == 0 ? first_s(tq, 1) : next_s(t - 1, 1)) && first_dp(t, 0) &&
             (t == 0 || dv_dq(t - 1, 1)) && second_s(t, 1) && next_s(t, 0) && first_dp(t, 1);
      for (int h = 0; h < 2 && ok; ++h) {
        if (!(ok = dv_dq(T - 1, h))) break;
        both_dk(T - 1, h);
      }
      if (!ok) break;
      tq += T;
      commit(dkv_full);
      commit(kv_empty);
    }
    commit(drain);
    sm100::mbar_wait_drain(drain, 0);
  } else {
    // ------------------------------------------------------------ P, W and dS; dQ
    // Little state is kept across tiles (barriers as 32-bit addresses, one accumulator
    // pointer, the mask as one bound), since 96 registers have to hold 48 of probabilities.
    const int qd = warp & 3, cq = warp >> 2, lane = sm100::lane_id();
    const int h = cq >> 1;  // half tile of this warp's group
    const int kl_ = qd * 32 + lane;  // key row within the tile = TMEM lane
    const uint32_t s_addr = tmem + (static_cast<uint32_t>(qd * 32) << 16) + S_COL + 32 * cq;
    const uint32_t dp_addr = s_addr + (DP_COL - S_COL);
    const uint32_t hb = sm100::smem_u32(half_bar(h, 0));
    constexpr uint32_t S1_FULL = 6 * 8, S1_READ = 7 * 8, S2_READ = 8 * 8, DP_FULL = 9 * 8,
                       DS_FULL = 10 * 8, DQ_FULL = 11 * 8, DQ_EMPTY = 12 * 8;
    // this warp's 32 rows of the half's four statistics
    const float4* l1v =
        reinterpret_cast<const float4*>(smem + C::OFF_LD + h * 1024 + (cq & 1) * 128);
    const float4 *l2v = l1v + 16, *d1v = l1v + 32, *d2v = l1v + 48;
    // its 64 bytes of this key row's dS line
    const uint32_t line = sbase + C::OFF_DS + h * PANEL + kl_ * 128;
    // this lane's place in an accumulator row (d = 64: only the half of the lanes whose map owns
    // this quarter's columns)
    const bool acc_on = DH == 128 || (lane >> 4) == (qd >> 1);
    uint32_t cur = 0;  // query tiles done
    bool ok = true;
    auto wait_at = [&](uint32_t bar, uint32_t tile, int site) -> bool {
      return mbar_wait_at(hb + bar, tile & 1, abort_flag, p.status, site);
    };
    auto arrive_at = [&](uint32_t bar) {
      sm100::tc_fence_before();
      __syncwarp();
      if (sm100::lane_id() == 0)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(hb + bar) : "memory");
    };
    auto f2 = [](uint32_t a, uint32_t b) {
      return make_float2(__uint_as_float(a), __uint_as_float(b));
    };
    for (uint32_t ik = 0; ok; ++ik) {
      int w;
      if (!(ok = next_item(ik, w)) || w < 0) break;
      bool bad = false;
      const Part pt = get_part(p, w, &bad);
      const Item& it = pt.it;
      if (bad && threadIdx.x == 0) atomicOr(p.status, 1);
      const int kvh = it.b * p.Hkv + it.hkv;
      const int key = it.n * BN + kl_;
      // query row r0 + c (r0 the warp's first row of tile i) sees the key iff c >= cmin0 - 128 i
      // (causal), for every c or for none
      const int cmin0 = key >= it.kv_len ? INT_MAX : p.causal ? key - off - 32 * cq : INT_MIN / 2;
      const int cstep = p.causal ? BMQ : 0;
      // query head g of the group and query tile i, from the part's first on
      const int nq = it.T > 0 ? it.T / p.G : 1, i_end = it.i_lo + nq;
      int g = pt.t0 / nq, i = it.i_lo + pt.t0 % nq;
      float* lam_part =
          p.lam_part + ((static_cast<size_t>(kvh) * p.n_kv + it.n) * p.n_split + pt.part) * p.G * NSMX + warp;
      if (lane == 0)  // heads that this part does not visit
        for (int e = 0; e < p.G; ++e)
          if (pt.T == 0 || e < g || e > (pt.t0 + pt.T - 1) / nq) lam_part[e * NSMX] = 0.f;
      const float* lam = p.lam + (p.n_lam == 1 ? 0 : it.hkv * p.G);
      const int lam_step = p.n_lam == 1 ? 0 : 1;
      // where the next dQ goes
      float* acc = p.dq_acc + (DH == 128 ? 32 * qd + lane : 16 * qd + (lane & 15)) +
                   (static_cast<size_t>(it.b * p.Hq + it.hkv * p.G + g) * p.Lqp + i * BMQ + 32 * cq) * DH;
      // adds this warp's 32 rows of a tile's dQ^T (lanes = head dimension) into the accumulator
      auto drain_dq = [&](uint32_t tile) -> bool {
        if (!wait_at(DQ_FULL, tile, 65)) return false;
        sm100::tc_fence_after();
        uint32_t v[32];
        sm100::tmem_ld32(dp_addr, v);
        sm100::tmem_ld_wait();
        arrive_at(DQ_EMPTY);
        if (acc_on) {
#pragma unroll
          for (int c = 0; c < 32; ++c) attn_bwd_impl::red_add_f32(acc + c * DH, __uint_as_float(v[c]));
        }
        acc += BMQ * DH;
        return true;
      };
      const uint32_t cur0 = cur;
      for (int left = pt.T; left > 0 && ok; ++g) {  // a head's tiles of the part
        const int i_stop = min(i_end, i + left);
        left -= i_stop - i;
        const float nl = -__ldg(lam + g * lam_step);
        float2 lam_acc = make_float2(0.f, 0.f);
        for (; i < i_stop; ++i, ++cur) {
          const int cmin = cmin0 - i * cstep;
          const bool all_vis = __all_sync(0xffffffffu, cmin <= 0);
          const float2 sl2 = make_float2(p.scale_log2, p.scale_log2), nlam = make_float2(nl, nl);
          // ---- P_1, kept in fp16 (see P_SCALE)
          if (!(ok = wait_at(S1_FULL, cur, 59))) break;
          sm100::tc_fence_after();
          uint32_t p1[16];
          {
            uint32_t s[32];
            sm100::tmem_ld32(s_addr, s);
            sm100::tmem_ld_wait();
            arrive_at(S1_READ);
            if (!all_vis) {
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (c < cmin) s[c] = __float_as_uint(-INFINITY);
            }
#pragma unroll
            for (int c4 = 0; c4 < 8; ++c4) {
              const float4 nlse = l1v[c4];
              const float2 n2[2] = {make_float2(nlse.x, nlse.y), make_float2(nlse.z, nlse.w)};
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int cp = 2 * c4 + e;
                const float2 x = __ffma2_rn(f2(s[2 * cp], s[2 * cp + 1]), sl2, n2[e]);
                p1[cp] = pack_f16x2(sm100::ex2(x.x), sm100::ex2(x.y));
              }
            }
          }
          // ---- the previous tile's dQ
          if (cur != cur0 && !(ok = drain_dq(cur - 1))) break;
          if (cur != cur0 && i == it.i_lo)  // that was the last tile of the head before
            acc += static_cast<size_t>(p.Lqp - nq * BMQ) * DH;
          // ---- sixteen columns at a time: P_2, W = P_1 - lam P_2 (over the dP it goes with),
          // dS_1 = P_1 (dP - D_1), dS_2 = P_2 (-lam dP + lam D_2), row-contiguous per key,
          // 16-byte chunk q of line kl_ at q ^ (kl_ & 7)
          if (!(ok = wait_at(DP_FULL, cur, 62))) break;
          sm100::tc_fence_after();
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t s[16], dp[16], wv[16];  // wv: W, then dS_1, eight words each
            sm100::tmem_ld16(s_addr + 16 * k, s);
            sm100::tmem_ld16(dp_addr + 16 * k, dp);
            sm100::tmem_ld_wait();
            if (k == 1) arrive_at(S2_READ);
            if (!all_vis) {
#pragma unroll
              for (int c = 0; c < 16; ++c)
                if (16 * k + c < cmin) s[c] = __float_as_uint(-INFINITY);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {  // eight columns: one 16-byte chunk of each map
              uint32_t w1[4], w2[4];
#pragma unroll
              for (int c4 = 0; c4 < 2; ++c4) {
                const int cc = 4 * k + 2 * q + c4;  // columns 4 cc ... of the thread's 32
                const float4 nl4 = l2v[cc], n1 = d1v[cc], n2 = d2v[cc];
                const float2 nlse[2] = {make_float2(nl4.x, nl4.y), make_float2(nl4.z, nl4.w)};
                const float2 nd1[2] = {make_float2(n1.x, n1.y), make_float2(n1.z, n1.w)};
                const float2 ld2[2] = {make_float2(n2.x, n2.y), make_float2(n2.z, n2.w)};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int j = 8 * q + 4 * c4 + 2 * e;  // of the sixteen columns
                  const float2 pa = unpack_f16x2(p1[2 * cc + e]), gp = f2(dp[j], dp[j + 1]);
                  const float2 x = __ffma2_rn(f2(s[j], s[j + 1]), sl2, nlse[e]);
                  const float2 pb = make_float2(sm100::ex2(x.x), sm100::ex2(x.y));
                  const float2 wf = __ffma2_rn(pb, nlam, pa);
                  const float2 a = __fmul2_rn(pa, __fadd2_rn(gp, nd1[e]));
                  const float2 b = __fmul2_rn(pb, __ffma2_rn(gp, nlam, ld2[e]));
                  lam_acc = __ffma2_rn(pb, gp, lam_acc);
                  wv[4 * q + 2 * c4 + e] = sm100::pack_bf16x2(wf.x, wf.y);
                  w1[2 * c4 + e] = sm100::pack_bf16x2(a.x, a.y);
                  w2[2 * c4 + e] = sm100::pack_bf16x2(b.x, b.y);
                }
              }
              const uint32_t at = line + (((4 * (cq & 1) + 2 * k + q) ^ (kl_ & 7)) << 4);
#pragma unroll
              for (int e = 0; e < 4; ++e) wv[8 + 4 * q + e] = w1[e];
              st_shared_v4(at, w1);
              st_shared_v4(at + 2 * PANEL, w2);
            }
            sm100::tmem_st16(dp_addr + 16 * k, wv);
          }
          sm100::tmem_st_wait();
          sm100::fence_proxy_async_smem();
          arrive_at(DS_FULL);
        }
        if (!ok) break;
        float x = lam_acc.x + lam_acc.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) lam_part[g * NSMX] = x;
        i = it.i_lo;
      }
      if (!ok) break;
      if (pt.T > 0 && !(ok = drain_dq(cur - 1))) break;
      // ---------------- epilogue: dV, dK (x scale) of this key row, a quarter of the columns
      if (!(ok = wait(dkv_full, ik & 1, 64))) break;
      sm100::tc_fence_after();
      const bool live = key < p.Lk;
      const size_t orow = static_cast<size_t>(kvh) * p.Lk + (live ? key : 0);
      const bool wide =
          ((reinterpret_cast<uintptr_t>(p.dV) | reinterpret_cast<uintptr_t>(p.dK)) & 31) == 0;
      constexpr int DQ = DH / 4;
#pragma unroll 1
      for (int m = 0; m < 2; ++m) {
        __nv_bfloat16* dst = (m == 0 ? p.dV : p.dK) + orow * DH + DQ * cq;
        const float f = (m == 0 ? 1.f : p.scale) * P_UNSCALE;
        // dK: map 2's half starts 64 columns on (d = 64: its own columns of a full-width product)
        const uint32_t col = s_addr - S_COL - 32 * cq + DQ * cq +
                             (m == 0 ? DV_COL : DK_COL + (DH == 64 ? 64 * h : 0));
#pragma unroll 1
        for (int c = 0; c < DQ; c += 16) {
          uint32_t v[16], o[8];
          sm100::tmem_ld16(col + c, v);
          sm100::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            o[e] = pt.T > 0 ? sm100::pack_bf16x2(__uint_as_float(v[2 * e]) * f,
                                                 __uint_as_float(v[2 * e + 1]) * f)
                            : 0u;
          if (p.n_split > 1) {  // the parts' sums are added, scaled and rounded at the end
            if (live) {
              if (pt.T == 0)
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = 0u;
              float* part = p.kv_part +
                            ((static_cast<size_t>(pt.part) * p.B * p.Hkv * p.Lk + orow) * 2 + m) * DH +
                            DQ * cq + c;
              st_global_v8(part, v);
              st_global_v8(part + 8, v + 8);
            }
          } else if (live) {
            if (wide) {
              st_global_v8(dst + c, o);
            } else {
              uint4* d4 = reinterpret_cast<uint4*>(dst + c);
              d4[0] = make_uint4(o[0], o[1], o[2], o[3]);
              d4[1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
          }
        }
      }
      sm100::tc_fence_before();
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(dkv_empty);
    }
  }

  sm100::tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    sm100::tc_fence_after();
    sm100::tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0) {
    // the last CTA to finish re-arms the dynamic scheduler for the next launch
    __threadfence();
    if (atomicAdd(p.sched + 1, 1) == static_cast<int>(gridDim.x) - 1) {
      p.sched[0] = 0;
      p.sched[1] = 0;
      __threadfence();
    }
  }
}

// ------------------------------------------------------------------ host side

struct Args : attn_bwd_impl::Args {
  const __nv_bfloat16* O2;
  const float* lam;
  int n_lam;
  __nv_bfloat16* dlam;
};

// Parts that the items' query tiles are shared out to.  An item -- 128 keys of one key/value
// head -- walks the query tiles of every head of the group, so a few key/value heads, or
// the causal mask's unequal items, leave SMs idle behind the longest one.  In units of a
// tile, a part costs about one more (its K, V, first products and sums); the makespan
// is the larger of the mean load and the longest part, and the least estimate wins.
// The lengths are on the device, so a padded batch counts its empty tiles, too.
// Measured on B200 (1 part / 4 parts / this rule's parts, us a call, one after another): causal B1
// Hq32 Hkv1 L4096 d128 3212 / 870 / 470, causal B1 Hq16 Hkv2 L8192 d128 1656 / 923 / 988, B1 Hq8
// Hkv2 L2048 d128 215 / 84 / 81, B1 H4 L2048 d128 64 / 64 / 50, causal B3 Hq16 Hkv4 L1999 d64
// 197 / 207 / 218, and padded to 1999, 1600 and 1200 keys 197 / 201 / 202: there the rule splits
// where one part is as good or better.
inline int n_split(int B, int Hq, int Hkv, int Lq, int Lk, bool causal) {
  constexpr double SMS = 148.;  // of every B200; the workspace query takes no device
  const double items = static_cast<double>(B) * Hkv * ((Lk + BN - 1) / BN);
  const double longest = static_cast<double>(Hq / Hkv) * ((Lq + BMQ - 1) / BMQ);
  if (items <= 0. || longest <= 0.) return 1;
  const double mean = items * longest * (causal && Lq > BMQ ? 0.5 : 1.0) / SMS;
  int best = 1;
  double least = 0.;
  for (int s = 1; s <= 64 && s <= longest; ++s) {
    const double part = longest / s + 1.;
    double load = mean + items * s / SMS;
    if (!causal) load = ceil(items * s / SMS) * part;  // equal parts run in waves
    const double est = part > load ? part : load;
    if (s == 1 || est < 0.95 * least) {
      best = s;
      least = est;
    }
  }
  return best;
}

// fp32 accumulator, statistics, dlam partials and the parts' dV and dK
struct Scratch {
  size_t acc, stats, lam, kv, total;
};
inline Scratch scratch(int B, int Hq, int Hkv, int Lq, int Lk, int d, int split) {
  const size_t rows = static_cast<size_t>(B) * Hq * attn_bwd_impl::lq_pad(Lq);
  const size_t n_kv = (static_cast<size_t>(Lk) + BN - 1) / BN;
  Scratch s;
  s.acc = 0;
  s.stats = rows * d * 4;
  s.lam = s.stats + rows * 16;
  s.kv = s.lam + static_cast<size_t>(B) * Hq * n_kv * split * NSMX * 4;
  s.total = s.kv;
  if (split > 1) s.total += static_cast<size_t>(split) * B * Hkv * Lk * d * 8;
  s.total = (s.total + 255) & ~static_cast<size_t>(255);
  return s;
}
inline size_t scratch_bytes(int B, int Hq, int Hkv, int Lq, int Lk, int d) {  // for either mask
  const size_t a = scratch(B, Hq, Hkv, Lq, Lk, d, n_split(B, Hq, Hkv, Lq, Lk, false)).total;
  const size_t c = scratch(B, Hq, Hkv, Lq, Lk, d, n_split(B, Hq, Hkv, Lq, Lk, true)).total;
  return a > c ? a : c;
}

template <int DH>
attn_status_t launch_d(const Args& a, cudaStream_t s) {
  using C = Cfg<DH>;
  Params p{};
  p.n_split = n_split(a.B, a.Hq, a.Hkv, a.Lq, a.Lk, a.causal != 0);
  const Scratch sc = scratch(a.B, a.Hq, a.Hkv, a.Lq, a.Lk, DH, p.n_split);
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.Lq = a.Lq;
  p.Lk = a.Lk;
  p.Lqp = attn_bwd_impl::lq_pad(a.Lq);
  p.scale = a.scale;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.causal = a.causal;
  p.k_lens = a.k_lens;
  p.status = a.status;
  p.sched = a.status + 1;
  p.dK = a.dK;
  p.dV = a.dV;
  p.n_kv = (a.Lk + BN - 1) / BN;
  p.n_qt = p.Lqp / BMQ;
  p.n_items = a.B * a.Hkv * p.n_kv * p.n_split;
  p.dq_acc = reinterpret_cast<float*>(a.scratch + sc.acc);
  float* stats = reinterpret_cast<float*>(a.scratch + sc.stats);
  p.stats = stats;
  p.lam_part = reinterpret_cast<float*>(a.scratch + sc.lam);
  p.kv_part = reinterpret_cast<float*>(a.scratch + sc.kv);
  p.lam = a.lam;
  p.n_lam = a.n_lam;
  const long long BH = static_cast<long long>(a.B) * a.Hq;

  if (a.Lq > 0) {
    const long long rows = BH * p.Lqp;
    const dim3 grid(static_cast<unsigned>((rows * (DH / 8) + 255) / 256));
    if (attn_host::report(
            attn_host::launch_overlapped(prep_kernel<DH>, grid, dim3(256), 0, s, a.O, a.O2, a.dO,
                                         a.lse, a.lam, a.n_lam, p.dq_acc, stats, p.sched, rows, a.Hq,
                                         a.Lq, p.Lqp),
            "diff prep_kernel") != cudaSuccess)
      return ATTN_ERR_CUDA;
  }
  if (p.n_items > 0) {
    // Lq == 0: no query tile is loaded; the maps only need an address
    const void* q = a.Lq > 0 ? a.Q : a.K;
    const void* g = a.Lq > 0 ? a.dO : a.K;
    const long long kvh = static_cast<long long>(a.B) * a.Hkv;
    CUtensorMap tq, tdo, tk, tv;
    if (!attn_bwd_impl::make_tmap_rows(&tq, q, DH, a.Lq, BH, HQ) ||
        !attn_bwd_impl::make_tmap_rows(&tdo, g, DH, a.Lq, BH, HQ) ||
        !attn_bwd_impl::make_tmap_rows(&tk, a.K, DH, a.Lk, kvh, BN) ||
        !attn_bwd_impl::make_tmap_rows(&tv, a.V, DH, a.Lk, kvh, BN)) {
      attn_host::report(cudaErrorInvalidValue, "diff bwd tensor maps");
      return ATTN_ERR_CUDA;
    }
    if (attn_host::report(attn_host::set_smem(main_kernel<DH>, C::SMEM_BYTES),
                          "diff main_kernel shared-memory attribute") != cudaSuccess)
      return ATTN_ERR_CUDA;
    const int grid = p.n_items < a.sms ? p.n_items : a.sms;
    if (attn_host::report(attn_host::launch_overlapped(main_kernel<DH>, dim3(grid), dim3(NTHREADS),
                                                       C::SMEM_BYTES, s, tq, tdo, tk, tv, p),
                          "diff main_kernel") != cudaSuccess)
      return ATTN_ERR_CUDA;
  }
  const long long conv = (BH * a.Lq * (DH / 8) + 255) / 256;
  const long long kv =
      p.n_split > 1 ? (static_cast<long long>(a.B) * a.Hkv * a.Lk * (DH / 4) + 255) / 256 : 0;
  return attn_host::report(
             attn_host::launch_overlapped(
                 finish_kernel<DH>, dim3(static_cast<unsigned>(conv + a.n_lam + kv)), dim3(256), 0,
                 s, p.dq_acc, a.dQ, BH, a.Lq, p.Lqp, a.scale, conv, p.lam_part, a.dlam, a.B, a.Hq,
                 a.Hkv, a.Lk, a.n_lam, p.n_split, p.kv_part, a.dK, a.dV),
             "diff finish_kernel") == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

inline attn_status_t launch(const Args& a, cudaStream_t s) {
  return a.d == 128 ? launch_d<128>(a, s) : launch_d<64>(a, s);
}

}  // namespace attn_diff_bwd_impl
