// Gradients of causal attention over packed sequences with grouped heads, on tcgen05.
//
// With x = s q.k, p = exp(x - lse), D_r = do_r . o_r:
//   dv_j = sum_r p_rj do_r,   dp_rj = do_r . v_j,   ds_rj = p_rj (dp_rj - D_r),
//   dq_r = s sum_j ds_rj k_j,   dk_j = s sum_r ds_rj q_r.
//
// Two launches. The first writes (lse log2(e), D_r) of every row, in the packed
// order (key head, token, head of the group) in which tiles take rows. In the second,
// some CTAs give dK and dV, one per key block of 128, over the query tiles that see
// it (the group's query heads are rows of the same tile, so their sum is the
// product's own), and some give dQ, one per query tile, over its key blocks. Splitting dQ off costs two of seven products (S and dP are formed
// twice) and buys an exact order of summation, no atomics and no fp32 copy of dQ.
//
// dK and dV, per query tile i (rows = keys, columns = queries):
//   S^T = K Q_i^T, dP^T = V dO_i^T (operands in shared memory), P^T and dS^T as
//   bf16 back into the TMEM columns they came from, dV += P^T dO_i,
//   dK += dS^T Q_i (left operands from TMEM). S and dP of the next tile are issued
//   as soon as the product that reads their columns is, so tensor cores and
//   exponentials overlap. Sixteen warps share the elementwise work, a quarter of
//   the columns each (with eight, a tile's two elementwise phases took 3460 of its
//   4360 cycles).
// dQ, per key block i (rows = queries): S = Q K_i^T into one of two
//   buffers, dP = dO V_i^T, dS as bf16 over S, dQ += dS K_i.
//
// P and dS are rounded to bf16 for the products (the operand type); everything
// else is fp32. In blocks on the diagonal dS enters as two bf16 parts (16 bits
// together): rows that see few keys, whose gradients are the largest, have all of
// theirs there, and it is one product more for one block of a long row. (dQ and dK
// against 64 bits: 2.6e-3 to 2.3e-3 of the norm, of which the results' own
// rounding is 1.7e-3.) Masked pairs are selected to zero, and rows that lie behind a
// sequence are zeroed in shared memory where a product sums over them.
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "seq.cuh"
#include "sm100.cuh"
#include "tmap.h"

namespace vda {

namespace {

constexpr int kTile = 128;
constexpr int kThreads = 576;  // TMA warp, MMA warp, sixteen elementwise warps

template <int D>
struct CbCfg {
  static constexpr int kAtoms = D / 64;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kRing = D == 128 ? 5 : 8;  // tiles in flight
  static constexpr int kRingOff = 2 * kTileBytes;  // behind the CTA's own two tiles (K, V or Q, dO)
  static constexpr int kStatOff = kRingOff + kRing * kTileBytes;  // two stages of 128 (lse2, D)
  static constexpr int kBarOff = kStatOff + 2 * kTile * 8;
  static constexpr int kSmemBytes = kBarOff + 512;  // the array is declared 1024-byte aligned: no room to align it
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kIdescS = sm100::idesc_bf16_f32(128, 128, false, false);
  static constexpr uint32_t kIdescG = sm100::idesc_bf16_f32(128, D, false, true);
  static_assert(kSmemBytes <= 232448, "more shared memory than a CTA may use");
};

struct CbArgs {
  int N, Hkv, G, tpt;
  int Tq, Tk;
  const int *cu_q, *cu_k, *k_len;
  float sl, scale;
  const float2* stat;  // [Hkv][Tq][G] (lse log2(e), D)
  __nv_bfloat16 *dQ, *dK, *dV;
  uint32_t* status;
  uint32_t wait_ns;
};

__device__ __forceinline__ void key_range(const CbArgs& a, int i, int& lo, int& n) {
  int hi;
  seq::bounds(a.cu_k, i, a.Tk, lo, hi);
  n = hi - lo;
  if (a.k_len) n = min(n, max(__ldg(a.k_len + i), 0));
}

// Token and query head of a row; 32-bit division where the row allows it (a 64-bit one
// costs more than the row's loads).
__device__ __forceinline__ void split_row(long long row, int Hq, long long& tok, int& h) {
  if (row < (1LL << 31)) {
    const unsigned t = (unsigned)row / (unsigned)Hq;
    tok = t;
    h = (int)((unsigned)row - t * (unsigned)Hq);
  } else {
    tok = row / Hq;
    h = (int)(row % Hq);
  }
}

// D / 8 threads per row (token, query head), 16 bytes each; kPerThread rows in
// flight per thread.
template <int D>
__global__ void __launch_bounds__(256) attn_rowdot_kernel(const __nv_bfloat16* O, const __nv_bfloat16* dO,
                                                          long long o_row, const float* lse, float2* stat, int Tq,
                                                          int Hq, int G) {
  constexpr int kLanes = D / 8, kRows = 256 / kLanes, kPerThread = 4;
  seq::grid_trigger();
  const int part = threadIdx.x % kLanes;
  const long long rows = (long long)Tq * Hq;
  const long long row0 = (long long)blockIdx.x * (kRows * kPerThread) + threadIdx.x / kLanes;
  uint4 x[kPerThread], y[kPerThread];
  long long tok;
  int h;
#pragma unroll
  for (int u = 0; u < kPerThread; ++u) {
    const long long row = row0 + u * kRows;
    if (row < rows) {
      split_row(row, Hq, tok, h);
      const long long at = tok * o_row + h * D + part * 8;
      x[u] = __ldcs(reinterpret_cast<const uint4*>(O + at));
      y[u] = __ldg(reinterpret_cast<const uint4*>(dO + at));
    }
  }
#pragma unroll
  for (int u = 0; u < kPerThread; ++u) {
    const long long row = row0 + u * kRows;
    float s = 0.f;
    if (row < rows) {
      const uint32_t a[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, b[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s = fmaf(__uint_as_float(a[e] << 16), __uint_as_float(b[e] << 16), s);
        s = fmaf(__uint_as_float(a[e] & 0xffff0000u), __uint_as_float(b[e] & 0xffff0000u), s);
      }
    }
#pragma unroll
    for (int m = kLanes / 2; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (part == 0 && row < rows) {
      split_row(row, Hq, tok, h);
      stat[((long long)(h / G) * Tq + tok) * G + h % G] = make_float2(lse[row] * 1.4426950408889634f, s);
    }
  }
}

// Barriers and bookkeeping both kernels share.
template <int D>
struct CbBars {
  uint64_t *own, *rfull, *rempty, *sfull, *pfull, *dpfull, *dsfull, *stfull, *stempty, *done, *drain;
  uint32_t* tmem_slot;
  volatile int* abort_flag;
  int* scratch;
  __device__ __forceinline__ explicit CbBars(uint8_t* p) {
    own = reinterpret_cast<uint64_t*>(p);
    rfull = own + 1;
    rempty = rfull + CbCfg<D>::kRing;
    sfull = rempty + CbCfg<D>::kRing;
    pfull = sfull + 2;
    dpfull = pfull + 1;
    dsfull = dpfull + 1;
    stfull = dsfull + 1;
    stempty = stfull + 2;
    done = stempty + 2;
    drain = done + 1;
    tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    scratch = reinterpret_cast<int*>(tmem_slot + 4);
    static_assert((1 + 2 * CbCfg<D>::kRing + 11) * 8 + 16 + 160 <= 512, "barrier block overflows its allowance");
  }
  __device__ __forceinline__ void init() {
    using namespace sm100;
    mbar_init(own, 1);
    for (int i = 0; i < CbCfg<D>::kRing; ++i) {
      mbar_init(&rfull[i], 1);
      mbar_init(&rempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&stfull[i], 1);
      mbar_init(&stempty[i], 16);
    }
    mbar_init(pfull, 16);
    mbar_init(dpfull, 1);
    mbar_init(dsfull, 16);
    mbar_init(done, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
};

// ---------------------------------------------------------------- dK and dV
// TMEM: S^T | dP^T | dV | dK. Query column c of P^T (dS^T) lies, packed, at
// column (c % 32) / 2 + (c / 32) * 32 of S^T (dP^T), dS^T's second part 16 columns
// on: each quarter of the elementwise warps overwrites only columns that it has
// read itself.
template <int D>
__device__ __forceinline__ void attn_dkdv(const CUtensorMap* mQ, const CUtensorMap* mK, const CUtensorMap* mV,
                                          const CUtensorMap* mG, const CbArgs& a, int bid, uint8_t* smem) {
  using C = CbCfg<D>;
  using namespace sm100;
  constexpr uint32_t kS = 0, kDP = 128, kDV = 256, kDK = 256 + D;
  uint8_t* sK = smem;
  uint8_t* sV = smem + C::kTileBytes;
  uint8_t* sR = smem + C::kRingOff;
  float* stat = reinterpret_cast<float*>(smem + C::kStatOff);  // per stage -lse log2(e), then -D
  CbBars<D> b(smem + C::kBarOff);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp == 0 && lane == 0) {
    b.init();
    prefetch_tmap(mQ);
    prefetch_tmap(mK);
    prefetch_tmap(mV);
    prefetch_tmap(mG);
  }
  if (warp == 1) {
    tmem_alloc(b.tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  const int hk = bid % a.Hkv;
  int kb;
  const int sq = seq::find_item(
      bid / a.Hkv, a.N, b.scratch, reinterpret_cast<int*>(smem),
      [&](int i) {
        int lo, n;
        key_range(a, i, lo, n);
        return n;
      },
      [&](int n) { return (n + kTile - 1) / kTile; }, kb);
  seq::grid_wait();
  if (sq < 0) {
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(*b.tmem_slot, C::kTmemCols);
    return;
  }
  int q_lo, q_hi, k_lo, nk;
  seq::bounds(a.cu_q, sq, a.Tq, q_lo, q_hi);
  key_range(a, sq, k_lo, nk);
  const int nq = q_hi - q_lo;
  const int k0 = kb * kTile;
  const int shift = nk - nq;  // query r sees keys 0 .. shift + r
  const int tiles = (nq + a.tpt - 1) / a.tpt;
  // The first tile with a row that sees key k0.
  const int i0 = min(tiles, max(0, k0 - shift) / a.tpt);
  const int n_it = tiles - i0;
  const int rows = a.tpt * a.G;
  // Some row of the i-th tile does not see the whole key block.
  auto on_diagonal = [&](int i) { return shift + (i0 + i) * a.tpt < k0 + kTile - 1; };

  // Rows that no tile has (128 is not a multiple of G) are summed over too: zero.
  for (int r = rows + (int)threadIdx.x; r < kTile; r += kThreads)
    for (int t = 0; t < C::kRing; ++t) seq::zero_row(sR + t * C::kTileBytes, C::kAtoms, r, kTile);
  fence_proxy_async_smem();
  seq::set_up(warp == 0);
  tc_fence_after();
  const uint32_t tmem = *b.tmem_slot;
  int issued = 0;
  // After a wait gave up: let every issued copy land before the CTA's shared memory is released.
  auto land = [&](int n) {
    if (!*b.abort_flag) return;
    mbar_wait(b.own, 0, nullptr, a.status, a.wait_ns);
    for (int i = max(0, n - C::kRing); i < n; ++i)
      mbar_wait(&b.rfull[i % C::kRing], (i / C::kRing) & 1, nullptr, a.status, a.wait_ns);
  };
  auto wait1 = [&](uint64_t* bar, uint32_t n) -> bool {
    return seq::bar_wait(bar, n & 1, b.abort_flag, a.status, a.wait_ns);
  };
  auto warp_wait = [&](uint64_t* bar, uint32_t n) -> bool { return __all_sync(0xffffffffu, wait1(bar, n)); };

  if (warp == 0) {
    // ---------------- TMA producer, and the rows' (lse, D)
    if (n_it > 0) {
      if (seq::elect_one()) {
        mbar_arrive_expect_tx(b.own, 2 * C::kTileBytes);
#pragma unroll
        for (int at = 0; at < C::kAtoms; ++at) {
          tma_load_3d(sK + at * (kTile * 128), mK, b.own, at * 64, hk, k_lo + k0);
          tma_load_3d(sV + at * (kTile * 128), mV, b.own, at * 64, hk, k_lo + k0);
        }
      }
      bool ok = true;
      for (int i = 0; i < n_it && ok; ++i) {
        const int t0 = (i0 + i) * a.tpt;
        for (int u = 0; u < 2 && ok; ++u) {
          const int slot = issued % C::kRing;
          if (!(ok = warp_wait(&b.rempty[slot], issued / C::kRing + 1))) break;
          if (seq::elect_one()) {
            mbar_arrive_expect_tx(&b.rfull[slot], (uint32_t)rows * 128u * C::kAtoms);
#pragma unroll
            for (int at = 0; at < C::kAtoms; ++at)
              tma_load_3d(sR + slot * C::kTileBytes + at * (kTile * 128), u ? mG : mQ, &b.rfull[slot], at * 64,
                          hk * a.G, q_lo + t0);
          }
          ++issued;
        }
        if (!ok) break;
        if (!(ok = warp_wait(&b.stempty[i & 1], i / 2 + 1))) break;
        const float2* src = a.stat + ((long long)hk * a.Tq + q_lo + t0) * a.G;
        const int live = min(a.tpt, nq - t0) * a.G;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = u * 32 + lane;
          const float2 v = r < live ? src[r] : make_float2(INFINITY, 0.f);  // a row that is none weighs 0
          stat[(i & 1) * 2 * kTile + r] = -v.x;
          stat[(i & 1) * 2 * kTile + kTile + r] = -v.y;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.stfull[i & 1]);
      }
      land(issued);
    }
  } else if (warp == 1) {
    if (seq::elect_one()) {
      bool ok = n_it > 0 && wait1(b.own, 0);
      auto slot_of = [&](int i, int u) { return (2 * i + u) % C::kRing; };
      // S^T (u = 0: K Q^T) or dP^T (u = 1: V dO^T) of tile i.
      auto issue_sd = [&](int i, int u) -> bool {
        const int slot = slot_of(i, u);
        if (!wait1(&b.rfull[slot], (2 * i + u) / C::kRing)) return false;
        tc_fence_after();
        // The address field of a descriptor counts 16 bytes: steps are added to it.
        const uint64_t da = smem_desc_sw128(smem_u32(u ? sV : sK), 16, 1024);
        const uint64_t db = smem_desc_sw128(smem_u32(sR + slot * C::kTileBytes), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk / 4) * (kTile * 128) + (kk % 4) * 32) / 16;
          mma_f16(tmem + (u ? kDP : kS), da + off, db + off, C::kIdescS, kk > 0 ? 1u : 0u);
        }
        mma_commit(u ? b.dpfull : &b.sfull[0]);
        return true;
      };
      // dV += P^T dO (u = 0) or dK += dS^T Q (u = 1) of tile i.
      auto issue_g = [&](int i, int u) -> bool {
        if (!wait1(u ? b.dsfull : b.pfull, i)) return false;
        tc_fence_after();
        const uint64_t db = smem_desc_sw128(smem_u32(sR + slot_of(i, 1 - u) * C::kTileBytes), kTile * 128, 1024);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          mma_f16_ts(tmem + (u ? kDK : kDV), tmem + (u ? kDP : kS) + (kk / 2) * 32 + (kk % 2) * 8, db + kk * 128,
                     C::kIdescG, (i > 0 || kk > 0) ? 1u : 0u);
        if (u && on_diagonal(i)) {  // the second parts
#pragma unroll 1
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_f16_ts(tmem + kDK, tmem + kDP + 16 + (kk / 2) * 32 + (kk % 2) * 8, db + kk * 128, C::kIdescG, 1u);
        }
        return true;
      };
      ok = ok && issue_sd(0, 0) && issue_sd(0, 1);
      for (int i = 0; i < n_it && ok; ++i) {
        if (!(ok = issue_g(i, 0))) break;
        mma_commit(&b.rempty[slot_of(i, 1)]);  // dO: read by dP and dV
        if (i + 1 < n_it && !(ok = issue_sd(i + 1, 0))) break;
        if (!(ok = issue_g(i, 1))) break;
        mma_commit(&b.rempty[slot_of(i, 0)]);  // Q: read by S and dK
        if (i + 1 < n_it && !(ok = issue_sd(i + 1, 1))) break;
      }
      if (ok) mma_commit(b.done);
      mma_commit(b.drain);
    }
  } else {
    // ---------------- elementwise: key row per thread, 32 query columns
    const int part = (warp - 2) / 4;
    const int quad = warp % 4;
    const int r = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t sa = tmem + lane_off + kS + part * 32, da = tmem + lane_off + kDP + part * 32;
    const int key = k0 + r;
    const float2 sl2 = make_float2(a.sl, a.sl);
    bool ok = true;
    for (int i = 0; i < n_it; ++i) {
      const int t0 = (i0 + i) * a.tpt;
      const bool ragged = t0 + a.tpt > nq;
      // Every key of the block is seen by every row of the tile. (Where 128 is not a
      // multiple of G, the columns that are no rows are zero in Q and dO.)
      const bool diagonal = on_diagonal(i), full = !ragged && !diagonal;
      // Else this row's key is seen by columns first .. end - 1 (token >= key - shift).
      const int first = max(0, (key - shift - t0)) * a.G - part * 32;
      const int end = min(a.tpt, nq - t0) * a.G - part * 32;
      auto mask = [&](uint32_t (&w)[16]) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int c = 2 * k;
          w[k] = (c >= first && c < end ? w[k] & 0xffffu : 0u) |
                 (c + 1 >= first && c + 1 < end ? w[k] & 0xffff0000u : 0u);
        }
      };
      if (!(ok = warp_wait(&b.stfull[i & 1], i / 2))) break;
      if (!(ok = warp_wait(&b.sfull[0], i))) break;
      tc_fence_after();
      const float* st = stat + (i & 1) * 2 * kTile + part * 32;
      uint32_t v[32], w[16];
      float2 p[16];
      seq::tmem_ld32(sa, v);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        const float4 l = *reinterpret_cast<const float4*>(st + 2 * k);
        const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), sl2,
                                    make_float2(l.x, l.y));
        const float2 y = __ffma2_rn(make_float2(__uint_as_float(v[2 * k + 2]), __uint_as_float(v[2 * k + 3])), sl2,
                                    make_float2(l.z, l.w));
        p[k] = make_float2(seq::ex2_approx(x.x), seq::ex2_approx(x.y));
        p[k + 1] = make_float2(seq::ex2_approx(y.x), seq::ex2_approx(y.y));
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) w[k] = seq::pack_bf16(p[k].x, p[k].y);
      if (!full) mask(w);
      tmem_st16(sa, w);
      tmem_st_wait();
      if (ragged) {
        // Query rows behind the sequence: zero them in both tiles (Q by two of the quarters, dO by the others).
        const int gs = 2 * i + 1;
        if (!(ok = warp_wait(&b.rfull[gs % C::kRing], gs / C::kRing))) break;
        if (part < 2 && r >= (nq - t0) * a.G)
          seq::zero_row(sR + ((2 * i + part) % C::kRing) * C::kTileBytes, C::kAtoms, r, kTile);
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b.pfull);
      if (!(ok = warp_wait(b.dpfull, i))) break;
      tc_fence_after();
      seq::tmem_ld32(da, v);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        const float4 l = *reinterpret_cast<const float4*>(st + kTile + 2 * k);
        const float2 x = __fmul2_rn(
            p[k], __fadd2_rn(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), make_float2(l.x, l.y)));
        const float2 y = __fmul2_rn(p[k + 1], __fadd2_rn(make_float2(__uint_as_float(v[2 * k + 2]),
                                                                     __uint_as_float(v[2 * k + 3])),
                                                         make_float2(l.z, l.w)));
        if (diagonal) {
          p[k] = x;
          p[k + 1] = y;
        }
        w[k] = seq::pack_bf16(x.x, x.y);
        w[k + 1] = seq::pack_bf16(y.x, y.y);
      }
      if (!full) mask(w);
      tmem_st16(da, w);
      if (diagonal) {
#pragma unroll
        for (int k = 0; k < 16; ++k) w[k] = seq::pack_rest(p[k], w[k]);
        mask(w);
        tmem_st16(da + 16, w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&b.stempty[i & 1]);
        mbar_arrive(b.dsfull);
      }
    }
    // ---------------- epilogue: two quarters write dV, two dK, half the channels each
    if (ok && (n_it == 0 || warp_wait(b.done, 0))) {
      tc_fence_after();
      const bool live = key < nk;
      const bool is_k = part >= 2;
      const int col = part % 2 * (D / 2);
      const float f = is_k ? a.scale : 1.f;
      const long long at = ((long long)(k_lo + (live ? key : k0)) * a.Hkv + hk) * D + col;
      const uint32_t ga = tmem + lane_off + (is_k ? kDK : kDV) + col;
      uint32_t w[D / 4];
#pragma unroll
      for (int c4 = 0; c4 < D / 64; ++c4) {
        uint32_t v[32];
        seq::tmem_ld32(ga + c4 * 32, v);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; ++k)
          w[c4 * 16 + k] =
              n_it > 0 ? seq::pack_bf16(__uint_as_float(v[2 * k]) * f, __uint_as_float(v[2 * k + 1]) * f) : 0u;
      }
      // Through the CTA's own tiles, which every product has read.
      seq::store_rows<D / 2>(smem + (part * 4 + quad) * (32 * D), w, live ? (is_k ? a.dK : a.dV) + at : nullptr);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) mbar_wait(b.drain, 0, nullptr, a.status, a.wait_ns);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ---------------------------------------------------------------- dQ
// TMEM: S (two buffers) | dP | dQ. Ring tiles: K_i, V_i.
template <int D>
__device__ __forceinline__ void attn_dq(const CUtensorMap* mQ, const CUtensorMap* mK, const CUtensorMap* mV,
                                        const CUtensorMap* mG, const CbArgs& a, int bid, uint8_t* smem) {
  using C = CbCfg<D>;
  using namespace sm100;
  constexpr uint32_t kS = 0, kDP = 256, kDQ = 384;
  uint8_t* sQ = smem;
  uint8_t* sG = smem + C::kTileBytes;
  uint8_t* sR = smem + C::kRingOff;
  CbBars<D> b(smem + C::kBarOff);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp == 0 && lane == 0) {
    b.init();
    prefetch_tmap(mQ);
    prefetch_tmap(mK);
    prefetch_tmap(mV);
    prefetch_tmap(mG);
  }
  if (warp == 1) {
    tmem_alloc(b.tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  const int hk = bid % a.Hkv;
  int idx;
  const int sq = seq::find_item(
      bid / a.Hkv, a.N, b.scratch, reinterpret_cast<int*>(smem),
      [&](int i) {
        int lo, hi;
        seq::bounds(a.cu_q, i, a.Tq, lo, hi);
        return hi - lo;
      },
      [&](int n) { return (n + a.tpt - 1) / a.tpt; }, idx);
  seq::grid_wait();
  if (sq < 0) {
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(*b.tmem_slot, C::kTmemCols);
    return;
  }
  int q_lo, q_hi, k_lo, nk;
  seq::bounds(a.cu_q, sq, a.Tq, q_lo, q_hi);
  key_range(a, sq, k_lo, nk);
  const int nq = q_hi - q_lo;
  idx = (nq + a.tpt - 1) / a.tpt - 1 - idx;  // longest first
  const int t0 = idx * a.tpt;
  const int shift = nk - nq;
  const int last = min(t0 + a.tpt, nq) - 1;
  const int n_it = (min(nk, max(0, shift + last + 1)) + kTile - 1) / kTile;
  const int min_lim = shift + t0 + 1;  // keys the tile's first row sees
  const int rows = a.tpt * a.G;

  seq::set_up(warp == 0);
  tc_fence_after();
  const uint32_t tmem = *b.tmem_slot;
  int issued = 0;
  // After a wait gave up: let every issued copy land before the CTA's shared memory is released.
  auto land = [&](int n) {
    if (!*b.abort_flag) return;
    mbar_wait(b.own, 0, nullptr, a.status, a.wait_ns);
    for (int i = max(0, n - C::kRing); i < n; ++i)
      mbar_wait(&b.rfull[i % C::kRing], (i / C::kRing) & 1, nullptr, a.status, a.wait_ns);
  };
  auto wait1 = [&](uint64_t* bar, uint32_t n) -> bool {
    return seq::bar_wait(bar, n & 1, b.abort_flag, a.status, a.wait_ns);
  };
  auto warp_wait = [&](uint64_t* bar, uint32_t n) -> bool { return __all_sync(0xffffffffu, wait1(bar, n)); };

  if (warp == 0) {
    if (n_it > 0 && seq::elect_one()) {
      mbar_arrive_expect_tx(b.own, 2u * rows * 128u * C::kAtoms);
#pragma unroll
      for (int at = 0; at < C::kAtoms; ++at) {
        tma_load_3d(sQ + at * (kTile * 128), mQ, b.own, at * 64, hk * a.G, q_lo + t0);
        tma_load_3d(sG + at * (kTile * 128), mG, b.own, at * 64, hk * a.G, q_lo + t0);
      }
      bool ok = true;
      for (int i = 0; i < n_it && ok; ++i)
        for (int u = 0; u < 2 && ok; ++u) {
          const int slot = issued % C::kRing;
          if (!(ok = wait1(&b.rempty[slot], issued / C::kRing + 1))) break;
          mbar_arrive_expect_tx(&b.rfull[slot], C::kTileBytes);
#pragma unroll
          for (int at = 0; at < C::kAtoms; ++at)
            tma_load_3d(sR + slot * C::kTileBytes + at * (kTile * 128), u ? mV : mK, &b.rfull[slot], at * 64, hk,
                        k_lo + i * kTile);
          ++issued;
        }
      land(issued);
    }
  } else if (warp == 1) {
    if (seq::elect_one()) {
      bool ok = n_it > 0 && wait1(b.own, 0);
      auto slot_of = [&](int i, int u) { return (2 * i + u) % C::kRing; };
      // S = Q K^T (u = 0) or dP = dO V^T (u = 1) of block i.
      auto issue_sd = [&](int i, int u) -> bool {
        const int slot = slot_of(i, u);
        if (!wait1(&b.rfull[slot], (2 * i + u) / C::kRing)) return false;
        tc_fence_after();
        const uint64_t da = smem_desc_sw128(smem_u32(u ? sG : sQ), 16, 1024);
        const uint64_t db = smem_desc_sw128(smem_u32(sR + slot * C::kTileBytes), 16, 1024);
        const uint32_t d = tmem + (u ? kDP : kS + (i & 1) * 128);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk / 4) * (kTile * 128) + (kk % 4) * 32) / 16;
          mma_f16(d, da + off, db + off, C::kIdescS, kk > 0 ? 1u : 0u);
        }
        if (u) mma_commit(&b.rempty[slot]);
        mma_commit(u ? b.dpfull : &b.sfull[i & 1]);
        return true;
      };
      ok = ok && issue_sd(0, 0) && issue_sd(0, 1);
      for (int i = 0; i < n_it && ok; ++i) {
        // S of the next block goes where dS of block i - 1 was: that product is issued before.
        if (i + 1 < n_it && !(ok = issue_sd(i + 1, 0))) break;
        if (!(ok = wait1(b.dsfull, i))) break;  // dS written, dP read
        tc_fence_after();
        if (i + 1 < n_it && !(ok = issue_sd(i + 1, 1))) break;
        const int slot = slot_of(i, 0);
        const uint64_t db = smem_desc_sw128(smem_u32(sR + slot * C::kTileBytes), kTile * 128, 1024);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          mma_f16_ts(tmem + kDQ, tmem + kS + (i & 1) * 128 + (kk / 2) * 32 + (kk % 2) * 8, db + kk * 128, C::kIdescG,
                     (i > 0 || kk > 0) ? 1u : 0u);
        if ((i + 1) * kTile > min_lim) {  // on the diagonal: the second parts
#pragma unroll 1
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_f16_ts(tmem + kDQ, tmem + kS + (i & 1) * 128 + 16 + (kk / 2) * 32 + (kk % 2) * 8, db + kk * 128,
                       C::kIdescG, 1u);
        }
        mma_commit(&b.rempty[slot]);
      }
      if (ok) mma_commit(b.done);
      mma_commit(b.drain);
    }
  } else {
    // ---------------- elementwise: query row per thread, 32 key columns
    const int part = (warp - 2) / 4;
    const int quad = warp % 4;
    const int r = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const int tok = t0 + r / a.G;
    const bool live = r < rows && tok < nq;
    const int lim = min(nk, shift + tok + 1);
    const float2 st = live ? a.stat[((long long)hk * a.Tq + q_lo + t0) * a.G + r] : make_float2(0.f, 0.f);
    const float2 sl2 = make_float2(a.sl, a.sl), nl2 = make_float2(-st.x, -st.x), nd2 = make_float2(-st.y, -st.y);
    bool ok = true;
    for (int i = 0; i < n_it; ++i) {
      const int k0 = i * kTile;
      const uint32_t sa = tmem + lane_off + kS + (i & 1) * 128 + part * 32, da = tmem + lane_off + kDP + part * 32;
      if (!(ok = warp_wait(&b.sfull[i & 1], i / 2))) break;
      tc_fence_after();
      uint32_t v[32], w[16];
      float2 p[16];
      seq::tmem_ld32(sa, v);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), sl2, nl2);
        p[k] = make_float2(seq::ex2_approx(x.x), seq::ex2_approx(x.y));
      }
      if (!(ok = warp_wait(b.dpfull, i))) break;
      tc_fence_after();
      seq::tmem_ld32(da, v);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float2 x = __fmul2_rn(
            p[k], __fadd2_rn(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), nd2));
        p[k] = x;
        w[k] = seq::pack_bf16(x.x, x.y);
      }
      if (k0 + kTile > min_lim) {
        const int end = lim - k0 - part * 32;
        uint32_t rest[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const uint32_t seen = (2 * k < end ? 0xffffu : 0u) | (2 * k + 1 < end ? 0xffff0000u : 0u);
          rest[k] = seq::pack_rest(p[k], w[k]) & seen;
          w[k] &= seen;
        }
        tmem_st16(sa + 16, rest);
      }
      tmem_st16(sa, w);
      tmem_st_wait();
      if (k0 + kTile > nk) {
        // Key rows behind the sequence are summed over: zero them.
        if (part == 0 && k0 + r >= nk) seq::zero_row(sR + ((2 * i) % C::kRing) * C::kTileBytes, C::kAtoms, r, kTile);
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b.dsfull);
    }
    // ---------------- epilogue: a quarter of the channels each
    if (ok && (n_it == 0 || warp_wait(b.done, 0))) {
      tc_fence_after();
      constexpr int kCols = D / 4;
      const long long at = ((long long)(q_lo + (live ? tok : t0)) * (a.Hkv * a.G) + hk * a.G + r % a.G) * D;
      uint32_t w[kCols / 2];
#pragma unroll
      for (int c = 0; c < kCols / 16; ++c) {
        uint32_t v[16];
        tmem_ld16(tmem + lane_off + kDQ + part * kCols + c * 16, v);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          w[c * 8 + k] = n_it > 0 ? seq::pack_bf16(__uint_as_float(v[2 * k]) * a.scale,
                                                   __uint_as_float(v[2 * k + 1]) * a.scale)
                                  : 0u;
      }
      seq::store_rows<kCols>(smem + (part * 4 + quad) * (32 * kCols * 2), w, live ? a.dQ + at + part * kCols : nullptr);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) mbar_wait(b.drain, 0, nullptr, a.status, a.wait_ns);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Both in one launch: the blocks of dK and dV first, those of dQ fill the SMs as the
// last of them run out. (One CTA to an SM either way, so an SM runs one role's code.)
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_tc_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                       const __grid_constant__ CUtensorMap mV, const __grid_constant__ CUtensorMap mG, const CbArgs a,
                       const int k_items) {
  extern __shared__ __align__(1024) uint8_t smem_1024[];
  // (The waits for the rows' statistics stand before each one's first way out.)
  if ((int)blockIdx.x < k_items)
    attn_dkdv<D>(&mQ, &mK, &mV, &mG, a, blockIdx.x, smem_1024);
  else
    attn_dq<D>(&mQ, &mK, &mV, &mG, a, (int)blockIdx.x - k_items, smem_1024);
}

template <int D>
cudaError_t launch_d(const vda_attention_config& c, const void* Q, const void* K, const void* V, const void* O,
                     const void* dO, const float* lse, const int* cu_q, const int* cu_k, const int* k_len, void* dQ,
                     void* dK, void* dV, void* ws, uint32_t* status, cudaStream_t s) {
  using C = CbCfg<D>;
  CbArgs a{};
  a.N = c.N; a.Hkv = c.Hkv; a.G = c.Hq / c.Hkv; a.tpt = kTile / a.G; a.Tq = c.Tq; a.Tk = c.Tk;
  a.cu_q = cu_q; a.cu_k = cu_k; a.k_len = k_len;
  a.scale = c.scale;
  a.sl = c.scale * 1.4426950408889634f;
  a.stat = static_cast<const float2*>(ws);
  a.dQ = static_cast<__nv_bfloat16*>(dQ);
  a.dK = static_cast<__nv_bfloat16*>(dK);
  a.dV = static_cast<__nv_bfloat16*>(dV);
  a.status = status;
  a.wait_ns = 2000000000u;
  cudaError_t e;
  const long long k_items = ((long long)c.Tk / kTile + c.N) * c.Hkv;
  const long long q_items = ((long long)c.Tq / a.tpt + c.N) * c.Hkv;
  const long long rows = (long long)c.Tq * c.Hq;
  if (k_items + q_items >= (1LL << 31) || (rows + 7) / 8 >= (1LL << 31))
    return cudaErrorInvalidConfiguration;
  if ((e = set_max_dynamic_smem(reinterpret_cast<const void*>(attn_bwd_tc_kernel<D>), C::kSmemBytes)) != cudaSuccess)
    return e;
  // An empty side is described by the other: nothing is loaded from it.
  const void* qp = c.Tq ? Q : K;
  const void* gp = c.Tq ? dO : K;
  const void* kp = c.Tk ? K : Q;
  const void* vp = c.Tk ? V : Q;
  const int qh = c.Tq ? c.Hq : 1, kh = c.Tk ? c.Hkv : 1;
  uint64_t qdims[3] = {(uint64_t)D, (uint64_t)qh, (uint64_t)std::max(1, c.Tq)};
  uint64_t kdims[3] = {(uint64_t)D, (uint64_t)kh, (uint64_t)std::max(1, c.Tk)};
  uint64_t qstr[2] = {(uint64_t)D * 2, (uint64_t)c.q_row * 2}, gstr[2] = {(uint64_t)D * 2, (uint64_t)c.o_row * 2};
  uint64_t kstr[2] = {(uint64_t)D * 2, (uint64_t)c.k_row * 2}, vstr[2] = {(uint64_t)D * 2, (uint64_t)c.v_row * 2};
  uint32_t qbox[3] = {64, (uint32_t)a.G, (uint32_t)a.tpt}, kbox[3] = {64, 1, (uint32_t)kTile};
  CUtensorMap mQ, mK, mV, mG;
  if ((e = make_tmap_bf16(&mQ, qp, 3, qdims, qstr, qbox)) != cudaSuccess) return e;
  if ((e = make_tmap_bf16(&mG, gp, 3, qdims, gstr, qbox)) != cudaSuccess) return e;
  if ((e = make_tmap_bf16(&mK, kp, 3, kdims, kstr, kbox)) != cudaSuccess) return e;
  if ((e = make_tmap_bf16(&mV, vp, 3, kdims, vstr, kbox)) != cudaSuccess) return e;
  if (rows > 0) {
    const int per = 256 / (D / 8) * 4;
    attn_rowdot_kernel<D><<<(unsigned)((rows + per - 1) / per), 256, 0, s>>>(
        static_cast<const __nv_bfloat16*>(O), static_cast<const __nv_bfloat16*>(dO), c.o_row, lse,
        static_cast<float2*>(ws), c.Tq, c.Hq, a.G);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const long long kb = c.Tk > 0 ? k_items : 0, qb = c.Tq > 0 ? q_items : 0;
  if (rows > 0)
    return seq::launch_behind(attn_bwd_tc_kernel<D>, dim3((unsigned)(kb + qb)), kThreads, C::kSmemBytes, s, mQ, mK, mV,
                              mG, a, (int)kb);
  attn_bwd_tc_kernel<D><<<(unsigned)kb, kThreads, C::kSmemBytes, s>>>(mQ, mK, mV, mG, a, (int)kb);
  return cudaGetLastError();
}

}  // namespace

size_t causal_attention_backward_workspace(const vda_attention_config& c) {
  return (size_t)c.Tq * c.Hq * sizeof(float2);
}

cudaError_t launch_causal_attention_backward(const vda_attention_config& c, const void* Q, const void* K,
                                             const void* V, const void* O, const void* dO, const float* lse,
                                             const int* cu_q, const int* cu_k, const int* k_len, void* dQ, void* dK,
                                             void* dV, void* ws, uint32_t* status, cudaStream_t s) {
  return c.d == 128
             ? launch_d<128>(c, Q, K, V, O, dO, lse, cu_q, cu_k, k_len, dQ, dK, dV, ws, status, s)
             : launch_d<64>(c, Q, K, V, O, dO, lse, cu_q, cu_k, k_len, dQ, dK, dV, ws, status, s);
}

}  // namespace vda
