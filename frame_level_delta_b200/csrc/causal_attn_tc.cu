// Causal softmax attention over packed sequences with grouped heads, on tcgen05.
//
// For row r of sequence i (nq queries, nk keys; the last query stands at the
// last key) and query head h of key head h / G:
//   o_r = sum_{j <= nk - nq + r} p_rj v_j,  p_rj = exp(s q_r.k_j) / l_r
// and lse_r = log l_r. A row that sees no key gives 0 and -inf.
//
// Tiles. A tile is 128 rows: 128 / G tokens times the G query heads that share
// one key head, packed (token, head), so that a key block is read once for the
// whole group and a diagonal block wastes 128 / G tokens only. Rows are
// independent in every product, so rows that do not exist (G not dividing 128,
// tokens past the sequence) carry what lies there and are not stored.
//
// An SM works on two tiles at a time, so that the tensor cores have one's products
// while the other's exponentials run. Each tile has eight softmax warps (two threads to
// a row, half the keys each; with four a packed batch took 6% longer when the second four
// were added), its logits
// S and its accumulator O in TMEM (128 and D columns; the probabilities overwrite their
// logits as packed bf16). The two are streams of one CTA that share each key block
// (long prompts at d = 128, where the reads of K and V count), or two CTAs of one
// stream, so that one's start and end hide behind the other's blocks.
//
// Few rows on long keys (single new tokens) are bound by the bytes of K and V, and
// by how evenly sequences of different lengths fill the SMs: there a tile's key
// blocks are shared out over several CTAs, each of which leaves a partial (o
// normalised by its own l, its log-sum) that a second kernel joins.
//
// Per key block: S = Q K^T (M = 128, N = 128), m = running row maximum in the
// log2 domain, P = 2^(S s log2(e) - m) rounded to bf16 (the tensor cores' operand
// type; the row sum l is taken over the unrounded values, so a weight is off by
// half a bf16 step at most), O += P V. O is rescaled only where a row's maximum
// grew by more than 2^8.
//
// Masks select: a masked logit becomes -inf whatever it was, and value rows past
// a sequence's end are zeroed in shared memory before the product that reads
// them, so neither infinities nor NaN behind a sequence reach a result. What is not
// finite within a sequence is not hidden: a row that sees a logit of NaN or +inf (or
// nothing but -inf) gives NaN, as the softmax's definition does. (A value that is not
// finite also reaches the rows of its block that do not see it, as 0 x NaN.)
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "seq.cuh"
#include "sm100.cuh"
#include "tmap.h"

namespace vda {

namespace {

constexpr int kTile = 128;
constexpr int kMinSplitBlocks = 4;
// Times in this file are of calls behind one another in a captured graph, under lasting load
// (about 1.7 GHz; in short bursts the longer ones take 9 to 13% less), with
// inputs larger than L2.
//
// Rows of a tile in the split form where sequences have few, which makes room for a third block
// in flight. In us, with such tiles (with whole ones): 8 caches of 4096 slots, four tokens each,
// 32 / 8 heads 27 (30); 16 of up to 8192, eight tokens each, 32 / 8 heads, d = 64 48 (53); one
// token each: 16 of up to 8192, 8 / 1 heads, d = 64 19 (20); 48 of up to 8192, 32 / 8 heads 121
// (119), 8 / 8 heads 160 (157), at d = 64 101 (96).
constexpr int kFewRows = 32;
// CTAs per SM that the split form aims at. 48 ragged caches of up to 8192 slots, 32 / 8 heads
// (16; 32 of them): two 127 (45; 82) us, three 121 (45; 82), four 121 (47; 83), five 121
// (47; 84), eight 128 (53; 92).
constexpr int kSplitCtas = 4;
constexpr int kShortKeys = 2304;  // d = 128: mean keys below which a CTA has one stream
constexpr uint32_t kFma = 0x22;  // pairs of eight whose exponentials the FMA pipe takes

template <int D, int kStreams, bool kFew>
struct CaCfg {
  static constexpr int kThreads = 128 + 256 * kStreams;  // TMA warp, MMA warp, two idle ones, eight warps a stream
  static constexpr int kAtoms = D / 64;
  static constexpr int kTileBytes = kTile * D * 2;
  // Key and value blocks in flight, one ring.
  static constexpr int kRing = kFew ? (D == 64 ? 6 : 3) : kStreams == 2 || D == 64 ? 5 : 2;
  // A tile of few rows keeps kFewRows of Q only: the products take whatever lies behind
  // them for the other rows, which are none.
  static constexpr int kQAtom = (kFew ? kFewRows : kTile) * 128, kQBytes = kAtoms * kQAtom;
  static constexpr int kQOff = 0;
  static constexpr int kRingOff = kStreams * kQBytes;
  static constexpr int kBarOff = kRingOff + kRing * kTileBytes;
  static constexpr int kPairOff = kBarOff + 512;  // per stream, half and row: what a row's two threads exchange
  static constexpr int kSmemBytes = kPairOff + kStreams * 1024;  // the array is declared 1024-byte aligned
  static constexpr uint32_t kS = 0, kO = 128 * kStreams;  // stream s: + 128 s, + D s columns
  static constexpr uint32_t kTmemCols = kStreams == 2 ? 512 : 256;
  static constexpr uint32_t kIdescS = sm100::idesc_bf16_f32(128, 128, false, false);
  static constexpr uint32_t kIdescO = sm100::idesc_bf16_f32(128, D, false, true);
  // 227 KB to a CTA; 228 KB to an SM, 1 KB of it taken by each CTA.
  static_assert(kSmemBytes <= (kStreams == 2 ? 232448 : 115712), "more shared memory than a CTA may use");
  static_assert(kRingOff >= 8 * seq::kSorted, "the list's search works in the Q tiles");
};

struct CaArgs {
  int N, Hkv, G, tpt;  // tpt: tokens per tile, 128 / G
  int Tq, Tk;
  int nsplit;          // shares of the keys (split form)
  const int *cu_q, *cu_k, *k_len;
  float sl;            // scale * log2(e)
  __nv_bfloat16* O;
  long long o_row;
  float* lse;          // [Tq, Hq], nullable
  float* part_o;       // split form: [nsplit][Tq * Hq][D]
  float* part_l;       // split form: [nsplit][Tq * Hq], log2 domain
  uint32_t* status;
  uint32_t wait_ns;
};

// Keys of sequence i: first token and count (k_len, where given, is the filled
// part of the sequence's room).
__device__ __forceinline__ void key_range(const CaArgs& a, int i, int& lo, int& n) {
  int hi;
  seq::bounds(a.cu_k, i, a.Tk, lo, hi);
  n = hi - lo;
  if (a.k_len) n = min(n, max(__ldg(a.k_len + i), 0));
}

// How many of nsplit shares a tile of nb key blocks uses (a share of fewer than
// kMinSplitBlocks blocks costs more to start than it saves), and share z of them.
__device__ __forceinline__ int used_splits(int nb, int nsplit) {
  return max(1, min(nsplit, (nb + kMinSplitBlocks - 1) / kMinSplitBlocks));
}

template <int D, int kStreams, bool kSplit, bool kFew>
__global__ void __launch_bounds__((CaCfg<D, kStreams, kFew>::kThreads), 3 - kStreams)
    causal_attn_tc_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                          const __grid_constant__ CUtensorMap mV, const CaArgs a) {
  using C = CaCfg<D, kStreams, kFew>;
  using namespace sm100;
  extern __shared__ __align__(1024) uint8_t smem_1024[];
  uint8_t* smem = smem_1024;
  uint8_t* sQ = smem + C::kQOff;
  uint8_t* sR = smem + C::kRingOff;
  uint64_t* qfull = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* rfull = qfull + 1;
  uint64_t* rempty = rfull + C::kRing;
  uint64_t* sfull = rempty + C::kRing;  // [2] logits of stream s in TMEM
  uint64_t* pfull = sfull + 2;          // [2][2] weights of stream s in TMEM: first (second) 32 keys of each half
  uint64_t* pvdone = pfull + 4;         // [2] O of stream s accumulated
  uint64_t* drain = pvdone + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* scratch = reinterpret_cast<int*>(tmem_slot + 4);
  static_assert((1 + 2 * C::kRing + 9) * 8 + 16 + 160 <= 512, "barrier block overflows its allowance");

  if (kSplit) seq::grid_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp == 0 && lane == 0) {
    mbar_init(qfull, 1);
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(&rfull[i], 1);
      mbar_init(&rempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[2 * i], 8);
      mbar_init(&pfull[2 * i + 1], 8);
      mbar_init(&pvdone[i], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&mQ);
    prefetch_tmap(&mK);
    prefetch_tmap(&mV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  const int hk = blockIdx.x % a.Hkv;
  const int rest = blockIdx.x / a.Hkv;
  const int z = kSplit ? rest % a.nsplit : 0;
  const int per_item = kStreams * a.tpt;
  int idx, sq;
  auto tokens = [&](int i) {
    int lo, hi;
    seq::bounds(a.cu_q, i, a.Tq, lo, hi);
    return hi - lo;
  };
  auto tiles = [&](int n) { return (n + per_item - 1) / per_item; };
  if constexpr (kSplit) {
    // Few rows: a sequence's work goes by its keys.
    sq = seq::find_item(rest / a.nsplit, a.N, scratch, reinterpret_cast<int*>(sQ), tokens, tiles, idx, [&](int i) {
      int lo, n;
      key_range(a, i, lo, n);
      return n;
    });
  } else {
    sq = seq::find_item(rest, a.N, scratch, reinterpret_cast<int*>(sQ), tokens, tiles, idx);
  }
  auto leave = [&] {
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(*tmem_slot, C::kTmemCols);
  };
  if (sq < 0) {
    leave();
    return;
  }
  int q_lo, q_hi, k_lo, nk;
  seq::bounds(a.cu_q, sq, a.Tq, q_lo, q_hi);
  key_range(a, sq, k_lo, nk);
  const int nq = q_hi - q_lo;
  // Longest tiles first: a sequence's last rows see the most keys.
  idx = (nq + per_item - 1) / per_item - 1 - idx;
  // Per stream: first token within the sequence and key blocks seen.
  int t0[2], nb[2] = {0, 0};
#pragma unroll
  for (int s = 0; s < kStreams; ++s) {
    t0[s] = idx * per_item + s * a.tpt;
    const int last = min(t0[s] + a.tpt, nq) - 1;
    const int seen = t0[s] < nq ? min(nk, max(0, nk - nq + last + 1)) : 0;
    nb[s] = (seen + kTile - 1) / kTile;
  }
  int b_lo = 0;  // first key block of this CTA's share
  if (kSplit) {
    const int used = used_splits(nb[0], a.nsplit);
    if (z >= used) {
      leave();
      return;
    }
    b_lo = (int)((long long)nb[0] * z / used);
    nb[0] = (int)((long long)nb[0] * (z + 1) / used) - b_lo;
  }
  const int nb_all = max(nb[0], nb[1]);

  seq::set_up(kStreams == 1 && warp == 0);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // 640 (384) threads start with 96 (80) registers each; the first four warps give some
  // of theirs to the others (4 x 64 + 16 x 104 = 20 x 96; 4 x 48 + 8 x 96 = 12 x 80).
  if (warp < 4) {
    if constexpr (kStreams == 1)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) {
      // ---------------- TMA producer. Ring order is the order in which the MMA
      // warp takes blocks: K0, then V_t and the next K in turn.
      if (nb_all > 0 && seq::elect_one()) {
        const uint32_t q_bytes = (uint32_t)(a.tpt * a.G) * 128u;
        const int q_tiles = nb[1] > 0 ? 2 : 1;
        mbar_arrive_expect_tx(qfull, q_bytes * C::kAtoms * q_tiles);
        for (int s = 0; s < q_tiles; ++s)
#pragma unroll
          for (int at = 0; at < C::kAtoms; ++at)
            tma_load_3d(sQ + s * C::kQBytes + at * C::kQAtom, &mQ, qfull, at * 64, hk * a.G, q_lo + t0[s]);
        int issued = 0;  // ring copies
        auto load = [&](const CUtensorMap* m, int blk) -> bool {
          const int slot = issued % C::kRing;
          if (!seq::bar_wait(&rempty[slot], ((issued / C::kRing) & 1) ^ 1, abort_flag, a.status, a.wait_ns)) return false;
          mbar_arrive_expect_tx(&rfull[slot], C::kTileBytes);
#pragma unroll
          for (int at = 0; at < C::kAtoms; ++at)
            tma_load_3d(sR + slot * C::kTileBytes + at * (kTile * 128), m, &rfull[slot], at * 64, hk,
                        k_lo + (b_lo + blk) * kTile);
          ++issued;
          return true;
        };
        bool ok = load(&mK, 0);
        for (int t = 0; t < nb_all && ok; ++t) {
          ok = load(&mV, t);
          if (ok && t + 1 < nb_all) ok = load(&mK, t + 1);
        }
        if (*abort_flag) {
          // Let every issued copy land before the CTA's shared memory is released.
          mbar_wait(qfull, 0, nullptr, a.status, a.wait_ns);
          for (int i = max(0, issued - C::kRing); i < issued; ++i)
            mbar_wait(&rfull[i % C::kRing], (i / C::kRing) & 1, nullptr, a.status, a.wait_ns);
        }
      }
    } else if (warp == 1) {
      // ---------------- MMA issuer. Products of one thread run in issue order, so
      // the next S of a stream, issued after P V of the last, cannot overwrite the
      // probabilities that product reads.
      if (seq::elect_one()) {
        bool ok = nb_all == 0 || seq::bar_wait(qfull, 0, abort_flag, a.status, a.wait_ns);
        int taken = 0;  // ring position
        auto take = [&](int& slot) -> bool {
          slot = taken % C::kRing;
          const bool r = seq::bar_wait(&rfull[slot], (taken / C::kRing) & 1, abort_flag, a.status, a.wait_ns);
          ++taken;
          return r;
        };
        auto issue_s = [&](int s, int slot) {
          // The address field of a descriptor counts 16 bytes: steps are added to it.
          const uint64_t dq = smem_desc_sw128(smem_u32(sQ + s * C::kQBytes), 16, 1024);
          const uint64_t dk = smem_desc_sw128(smem_u32(sR + slot * C::kTileBytes), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk / 4) * (kTile * 128) + (kk % 4) * 32) / 16;
            const uint32_t q_off = ((kk / 4) * C::kQAtom + (kk % 4) * 32) / 16;
            mma_f16(tmem + C::kS + s * 128, dq + q_off, dk + off, C::kIdescS, kk > 0 ? 1u : 0u);
          }
          mma_commit(&sfull[s]);
        };
        auto issue_pv = [&](int s, int j, int slot) -> bool {
          const uint64_t dv = smem_desc_sw128(smem_u32(sR + slot * C::kTileBytes), kTile * 128, 1024);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (!seq::bar_wait(&pfull[2 * s + u], j & 1, abort_flag, a.status, a.wait_ns)) return false;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int half = k / 2, kk = half * 4 + u * 2 + k % 2;
              mma_f16_ts(tmem + C::kO + s * D, tmem + C::kS + s * 128 + half * 64 + (u * 2 + k % 2) * 8, dv + kk * 128,
                         C::kIdescO, (j > 0 || u + k > 0) ? 1u : 0u);
            }
          }
          mma_commit(&pvdone[s]);
          return true;
        };
        int slot = 0, vslot = 0;
        if (ok && nb_all > 0) {
          if ((ok = take(slot))) {
            for (int s = 0; s < kStreams; ++s)
              if (nb[s] > 0) issue_s(s, slot);
            mma_commit(&rempty[slot]);
          }
          for (int i = 0; i < nb_all && ok; ++i) {
            if (!(ok = take(vslot))) break;
            bool have = false;
            for (int s = 0; s < kStreams && ok; ++s) {
              if (i < nb[s] && !(ok = issue_pv(s, i, vslot))) break;
              if (s == kStreams - 1) mma_commit(&rempty[vslot]);
              if (i + 1 < nb[s]) {
                if (!have && !(ok = take(slot))) break;
                have = true;
                issue_s(s, slot);
              }
            }
            if (ok && have) mma_commit(&rempty[slot]);
          }
        }
        mma_commit(drain);
      }
    }
    __syncwarp();
  } else {
    if constexpr (kStreams == 1)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ---------------- softmax and epilogue: stream s, a row to two threads, half the
    // keys (channels) each
    const int s = (warp - 4) / 8, half = (warp - 4) / 4 % 2;
    const int quad = warp % 4;
    const int r = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const int my_nb = nb[s];
    const int tok = t0[s] + r / a.G;  // row's token within the sequence
    const int head = hk * a.G + r % a.G;
    const bool live = r < a.tpt * a.G && tok < nq;
    const int lim = min(nk, nk - nq + tok + 1);  // keys this row sees
    const int warp_lim = __shfl_sync(0xffffffffu, lim, 31);  // and any row of this warp
    const bool any_live = quad * 32 < min(a.tpt, nq - t0[s]) * a.G;  // some row of this warp exists
    const int min_lim = nk - nq + t0[s] + 1;                         // keys the tile's first row sees
    const uint32_t sa = tmem + lane_off + C::kS + s * 128 + half * 64;
    const uint32_t oa = tmem + lane_off + C::kO + s * D + half * (D / 2);
    volatile float* mine = reinterpret_cast<float*>(smem + C::kPairOff) + (s * 2 + half) * kTile + r;
    volatile float* other = reinterpret_cast<float*>(smem + C::kPairOff) + (s * 2 + 1 - half) * kTile + r;
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      const bool w = seq::bar_wait(bar, parity, abort_flag, a.status, a.wait_ns);
      return __all_sync(0xffffffffu, w);
    };
    // The two warps of 32 rows meet, and go on if no wait has given up. A warp that goes no
    // further arrives once more (fail), so that the other, which sees the flag behind the
    // barrier, never waits for it.
    const int pair = 1 + s * 4 + quad;
    auto meet = [&]() -> bool {
      asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
      return !__any_sync(0xffffffffu, *abort_flag != 0);
    };
    auto fail = [&] {
      ok = false;
      __syncwarp();
      asm volatile("bar.arrive %0, 64;" ::"r"(pair) : "memory");
    };
    for (int j = 0; j < my_nb; ++j) {
      const int k0 = (b_lo + j) * kTile;
      const int kh = k0 + half * 64;  // this thread's first key
      if (!warp_wait(&sfull[s], j & 1)) { fail(); break; }
      tc_fence_after();
      if (k0 + kTile > nk && half == 0) {
        // The keys end inside this block: zero the value rows behind them. The
        // block's ring position follows from the loading order; its copy must
        // have landed first.
        const int pos = 2 * j + 1;
        const int slot = pos % C::kRing;
        if (!warp_wait(&rfull[slot], (pos / C::kRing) & 1)) { fail(); break; }
        if (k0 + r >= nk) seq::zero_row(sR + slot * C::kTileBytes, C::kAtoms, r, kTile);
        fence_proxy_async_smem();
        __syncwarp();  // every lane's rows, before lane 0 signals the product that reads them
      }
      if (any_live) {
        const bool masked = k0 + kTile > min_lim;
        const int n = lim - kh;  // keys of this half that the row sees
        // Logits are read twice, for the maximum and for the weights: kept, they would
        // leave no registers to work with.
        float mb = -INFINITY;
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2) {
          uint32_t v[32];
          seq::tmem_ld32(sa + c2 * 32, v);
          tmem_ld_wait();
          if (masked) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (c2 * 32 + k >= n) v[k] = 0xff800000u;
          }
          float mx[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = __uint_as_float(v[q]);
#pragma unroll
          for (int k = 4; k < 32; ++k) mx[k & 3] = seq::max_nan(mx[k & 3], __uint_as_float(v[k]));
          mb = seq::max_nan(mb, seq::max_nan(seq::max_nan(mx[0], mx[1]), seq::max_nan(mx[2], mx[3])));
        }
        mb *= a.sl;
        // (The other thread has read the last block's: the product that this block's
        // logits came behind waited for its probabilities.)
        *mine = mb;
        if (!meet()) { fail(); break; }
        mb = seq::max_nan(mb, *other);
        // A NaN among a row's logits, or one beyond the range, makes its weights NaN, and
        // so its O and its sum: the maximum carries it, and stays NaN from here on.
        if (!(mb < INFINITY)) mb = NAN;
        const bool grow = live && j > 0 && !(mb <= m_run + 8.f);
        if (j == 0) m_run = mb;
        if (__any_sync(0xffffffffu, grow)) {
          if (!warp_wait(&pvdone[s], (j - 1) & 1)) { fail(); break; }
          tc_fence_after();
          const float f = grow ? seq::ex2_approx(m_run - mb) : 1.f;
#pragma unroll
          for (int c2 = 0; c2 < D / 64; ++c2) {
            uint32_t v[32];
            seq::tmem_ld32(oa + c2 * 32, v);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t w[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) w[k] = v[q * 16 + k];
              tmem_st16(oa + c2 * 32 + q * 16, w);
            }
          }
          if (grow) {
            l_run *= f;
            m_run = mb;
          }
        }
        // A row that has seen no key yet keeps m = -inf; its weights are 0.
        const float m_use = m_run == -INFINITY ? 0.f : m_run;
        const float2 sl2 = make_float2(a.sl, a.sl), nm2 = make_float2(-m_use, -m_use);
        float2 ls2[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) ls2[q] = make_float2(0.f, 0.f);
        // Two of eight pairs on the FMA pipe: the exponentials of two streams
        // would keep the special-function units as long as the products keep the
        // tensor cores (packed batch, and 8191 tokens: none so 125.7 and 551 us, one 124.2
        // and 550, two 124.5 and 548, three 126.1 and 554, four 126.5 and 566). Not in masked
        // blocks (its smallest value is not 0), where 32 keys that no row of the warp sees
        // are left out.
        auto weights = [&](auto plain) {
#pragma unroll
          for (int c2 = 0; c2 < 2; ++c2) {
            uint32_t w[16];
            if (plain.value || kh + c2 * 32 < warp_lim) {
              uint32_t v[32];
              seq::tmem_ld32(sa + c2 * 32, v);
              tmem_ld_wait();
              if (!plain.value) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (c2 * 32 + k >= n) v[k] = 0xff800000u;
              }
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float2 y = __ffma2_rn(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), sl2, nm2);
                const float2 p = plain.value && (kFma >> (k & 7) & 1)
                                     ? seq::ex2_fma(y)
                                     : make_float2(seq::ex2_approx(y.x), seq::ex2_approx(y.y));
                ls2[k & 3] = __fadd2_rn(ls2[k & 3], p);
                w[k] = seq::pack_bf16(p.x, p.y);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 16; ++k) w[k] = 0u;
            }
            tmem_st16(sa + c2 * 16, w);
            if (c2 == 0) {
              // The first 32 keys of this half: their product may start.
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&pfull[2 * s]);
            }
          }
        };
        if (masked)
          weights(std::false_type{});
        else
          weights(std::true_type{});
        l_run += ((ls2[0].x + ls2[0].y) + (ls2[1].x + ls2[1].y)) + ((ls2[2].x + ls2[2].y) + (ls2[3].x + ls2[3].y));
        tmem_st_wait();
      } else if (lane == 0) {
        mbar_arrive(&pfull[2 * s]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pfull[2 * s + 1]);
    }
    // ---------------- epilogue
    const bool have = my_nb > 0;
    if (ok && have && !warp_wait(&pvdone[s], (my_nb - 1) & 1)) fail();
    if (ok && have && any_live) {
      *mine = l_run;
      ok = meet();
      l_run = half ? *other + l_run : l_run + *other;
    }
    if (ok) {
      tc_fence_after();
      // No finite logit: the row sees no key, or -inf - (-inf) of those it sees is NaN.
      const bool none = m_run == -INFINITY, sees = lim > 0;
      const float inv = none ? 0.f : 1.f / l_run;
      const long long tok_g = (long long)q_lo + (live ? tok : 0);
      const long long rows = (long long)a.Tq * a.Hkv * a.G;
      const long long row = tok_g * a.Hkv * a.G + head;
      if (kSplit) {
        const long long at = (long long)z * rows + row;
        if (live && half == 0) a.part_l[at] = none ? -INFINITY : m_run + log2f(l_run);
        float4* dst = reinterpret_cast<float4*>(a.part_o + at * D + half * (D / 2));
        if (any_live && have) {
#pragma unroll
          for (int c2 = 0; c2 < D / 64; ++c2) {
            uint32_t v[32];
            seq::tmem_ld32(oa + c2 * 32, v);
            tmem_ld_wait();
            if (live) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                dst[c2 * 8 + k] = make_float4(__uint_as_float(v[4 * k]) * inv, __uint_as_float(v[4 * k + 1]) * inv,
                                              __uint_as_float(v[4 * k + 2]) * inv, __uint_as_float(v[4 * k + 3]) * inv);
            }
          }
        }
      } else {
        if (live && a.lse && half == 0)
          a.lse[row] = none ? (sees ? NAN : -INFINITY) : (m_run + log2f(l_run)) * 0.6931471805599453f;
        const uint32_t fill = sees ? 0x7fff7fffu : 0u;  // two bf16 NaN
        uint32_t w[D / 4];
#pragma unroll
        for (int c2 = 0; c2 < D / 64; ++c2) {
          uint32_t v[32];
          seq::tmem_ld32(oa + c2 * 32, v);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k)
            w[c2 * 16 + k] =
                none ? fill : seq::pack_bf16(__uint_as_float(v[2 * k]) * inv, __uint_as_float(v[2 * k + 1]) * inv);
        }
        // Through the stream's own Q tile, which its products have read. (Where it has
        // none, the tile's copy must have landed.)
        if (!have && nb_all > 0) warp_wait(qfull, 0);
        seq::store_rows<D / 2>(sQ + s * C::kTileBytes + (half * 4 + quad) * (32 * D), w,
                               live ? a.O + tok_g * a.o_row + (long long)head * D + half * (D / 2) : nullptr);
      }
    }
  }

  // ---------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) mbar_wait(drain, 0, nullptr, a.status, a.wait_ns);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the partials of the split form: one warp per row (token, query head).
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const CaArgs a) {
  const int Hq = a.Hkv * a.G;
  const long long rows = (long long)a.Tq * Hq;
  const long long row = (long long)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int tok = (int)(row / Hq), head = (int)(row % Hq);
  // Rows outside the sequences are left as they were.
  if (row >= rows || tok < __ldg(a.cu_q) || tok >= __ldg(a.cu_q + a.N)) {
    seq::grid_wait();
    return;
  }
  // The row's sequence: the last one that starts at or before it.
  int lo = 0, hi = a.N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (__ldg(a.cu_q + mid) <= tok) lo = mid;
    else hi = mid - 1;
  }
  int q_lo, q_hi, k_lo, nk;
  seq::bounds(a.cu_q, lo, a.Tq, q_lo, q_hi);
  key_range(a, lo, k_lo, nk);
  const int nq = q_hi - q_lo;
  const int last = min((tok - q_lo) / a.tpt * a.tpt + a.tpt, nq) - 1;
  const int nb = (min(nk, max(0, nk - nq + last + 1)) + kTile - 1) / kTile;
  const int n = used_splits(nb, a.nsplit);
  seq::grid_wait();
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = seq::max_nan(m, a.part_l[i * rows + row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = seq::max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  constexpr int kPer = D / 32;
  float acc[kPer], w_all = 0.f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
  const bool none = m == -INFINITY;
  if (!none) {
    for (int i = 0; i < n; ++i) {
      const float l = a.part_l[i * rows + row];
      if (l == -INFINITY) continue;  // a share without a finite logit has no weight (without keys, it has written no o)
      const float w = exp2f(l - m);
      w_all += w;
      const float* src = a.part_o + (i * rows + row) * D + lane * kPer;
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = fmaf(w, src[k], acc[k]);
    }
  }
  // As in the other kernel: 0 for a row that sees no key, NaN for one whose logits are all -inf.
  const bool sees = min(nk, nk - nq + tok - q_lo + 1) > 0;
  const float inv = none ? (sees ? NAN : 0.f) : 1.f / w_all;
  __nv_bfloat16* dst = a.O + (long long)tok * a.o_row + (long long)head * D + lane * kPer;
#pragma unroll
  for (int k = 0; k < kPer; k += 2)
    *reinterpret_cast<__nv_bfloat162*>(dst + k) = __floats2bfloat162_rn(acc[k] * inv, acc[k + 1] * inv);
  if (lane == 0 && a.lse) a.lse[row] = none ? (sees ? NAN : -INFINITY) : (m + log2f(w_all)) * 0.6931471805599453f;
}

// The form and the number of key shares for a call, by mean lengths (the lengths
// themselves are on the device).
//  - Few rows on long keys: one stream a CTA, the keys shared out, in enough shares
//    to give each SM several CTAs. Where a sequence has up to kFewRows rows on average,
//    tiles are that high, which leaves room for one more block in flight.
//  - d = 64, and short sequences at d = 128: one stream a CTA, two CTAs to an SM: one's
//    start and end hide behind the other's blocks.
//  - Else two streams a CTA, which halves the reads of K and V.
// Measured at d = 128, 24 / 8 heads, one stream (two): 16 x 256 tokens 34.6 (44.9) us,
// 16 x 512 75.6 (86.7), 8 x 1024 101 (102), 8 x 1536 188 (186), 6 x 2048 226 (224; in a short
// burst 197 and 205), 4 x 3000 298 (279), 2 x 4096 260 (240); at d = 64, 8 / 8 heads: 16 x 512
// 25.8 (28.1), 8 x 1536 57.2 (62.1), 2 x 4096 67.2 (68.1).
struct Plan {
  int streams;
  bool split;
  int nsplit;
  int tpt;
};
Plan plan_of(const vda_attention_config& c) {
  const int G = c.Hq / c.Hkv, tpt = kTile / G;
  const long long ctas = ((long long)c.Tq / (2 * tpt) + (c.N + 1) / 2) * c.Hkv;
  const long long keys = (long long)c.Tk / c.N;  // mean room per sequence
  const long long rows = (long long)c.Tq / c.N;
  const bool few = (long long)c.Tq <= (long long)c.N * tpt;  // about one tile per sequence
  Plan p{few || c.d == 64 || keys < kShortKeys ? 1 : 2, false, 1, tpt};
  if (keys >= 2 * kMinSplitBlocks * kTile && (few || (ctas < 148 && keys >= 4 * rows))) {
    p.streams = 1;
    p.split = true;
    if (G <= kFewRows && c.Tq <= (long long)c.N * (kFewRows / G)) p.tpt = kFewRows / G;
    const long long tiles = ((long long)c.Tq / p.tpt + c.N) * c.Hkv;
    const long long want = (148LL * kSplitCtas + tiles - 1) / tiles;
    const long long most = std::max(1LL, ((long long)c.Tk + kTile * kMinSplitBlocks - 1) / (kTile * kMinSplitBlocks));
    p.nsplit = (int)std::max(1LL, std::min({want, most, 64LL}));
  }
  return p;
}

template <int D>
cudaError_t launch_d(const vda_attention_config& c, const void* Q, const void* K, const void* V, const int* cu_q,
                     const int* cu_k, const int* k_len, void* O, float* lse, void* ws, uint32_t* status,
                     cudaStream_t s) {
  using C1 = CaCfg<D, 1, false>;
  using CF = CaCfg<D, 1, true>;
  const Plan p = plan_of(c);
  CaArgs a{};
  a.N = c.N; a.Hkv = c.Hkv; a.G = c.Hq / c.Hkv; a.tpt = p.tpt; a.Tq = c.Tq; a.Tk = c.Tk;
  a.nsplit = p.nsplit;
  a.cu_q = cu_q; a.cu_k = cu_k; a.k_len = k_len;
  a.sl = c.scale * 1.4426950408889634f;
  a.O = static_cast<__nv_bfloat16*>(O);
  a.o_row = c.o_row;
  a.lse = lse;
  const long long rows = (long long)c.Tq * c.Hq;
  if (p.split) {
    a.part_o = static_cast<float*>(ws);
    a.part_l = a.part_o + (long long)p.nsplit * rows * D;
  }
  a.status = status;
  a.wait_ns = 2000000000u;
  const int per_item = p.streams * a.tpt;
  // ceil(n / per_item) summed over the sequences is at most Tq / per_item + N.
  const long long items = (long long)c.Tq / per_item + c.N;
  const long long grid = items * c.Hkv * p.nsplit;
  if (grid >= (1LL << 31)) return cudaErrorInvalidConfiguration;
  const bool few = p.tpt < kTile / a.G;
  auto* fn = few       ? causal_attn_tc_kernel<D, 1, true, true>
             : p.split ? causal_attn_tc_kernel<D, 1, true, false>
                       : causal_attn_tc_kernel<D, 1, false, false>;
  int threads = C1::kThreads, smem = few ? CF::kSmemBytes : C1::kSmemBytes;
  if constexpr (D == 128) {
    using C2 = CaCfg<D, 2, false>;
    if (p.streams == 2) {
      fn = causal_attn_tc_kernel<D, 2, false, false>;
      threads = C2::kThreads;
      smem = C2::kSmemBytes;
    }
  }
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(fn), smem);
  if (e != cudaSuccess) return e;
  uint64_t qdims[3] = {(uint64_t)D, (uint64_t)c.Hq, (uint64_t)c.Tq};
  uint64_t qstr[2] = {(uint64_t)D * 2, (uint64_t)c.q_row * 2};
  uint32_t qbox[3] = {64, (uint32_t)a.G, (uint32_t)a.tpt};
  // Without keys nothing is loaded from K and V: their maps describe one row of Q.
  const bool none = c.Tk == 0;
  uint64_t kdims[3] = {(uint64_t)D, (uint64_t)c.Hkv, (uint64_t)(none ? 1 : c.Tk)};
  uint64_t kstr[2] = {(uint64_t)D * 2, (uint64_t)(none ? c.q_row : c.k_row) * 2};
  uint64_t vstr[2] = {(uint64_t)D * 2, (uint64_t)(none ? c.q_row : c.v_row) * 2};
  uint32_t kbox[3] = {64, 1, (uint32_t)kTile};
  CUtensorMap mQ, mK, mV;
  if ((e = make_tmap_bf16(&mQ, Q, 3, qdims, qstr, qbox)) != cudaSuccess) return e;
  if ((e = make_tmap_bf16(&mK, none ? Q : K, 3, kdims, kstr, kbox)) != cudaSuccess) return e;
  if ((e = make_tmap_bf16(&mV, none ? Q : V, 3, kdims, vstr, kbox)) != cudaSuccess) return e;
  fn<<<(unsigned)grid, threads, smem, s>>>(mQ, mK, mV, a);
  if (!p.split) return cudaGetLastError();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return seq::launch_behind(attn_join_kernel<D>, dim3((unsigned)((rows + 7) / 8)), 256, 0, s, a);
}

}  // namespace

size_t causal_attention_workspace(const vda_attention_config& c) {
  const Plan p = plan_of(c);
  if (!p.split) return 0;
  return (size_t)p.nsplit * c.Tq * c.Hq * (c.d + 1) * sizeof(float);
}

cudaError_t launch_causal_attention(const vda_attention_config& c, const void* Q, const void* K, const void* V,
                                    const int* cu_q, const int* cu_k, const int* k_len, void* O, float* lse, void* ws,
                                    uint32_t* status, cudaStream_t s) {
  return c.d == 128 ? launch_d<128>(c, Q, K, V, cu_q, cu_k, k_len, O, lse, ws, status, s)
                    : launch_d<64>(c, Q, K, V, cu_q, cu_k, k_len, O, lse, ws, status, s);
}

}  // namespace vda
