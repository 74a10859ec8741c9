// Linear attention whose state decays by a factor of each head, over packed
// sequences, on tcgen05: whole prompts, and the three passes of the backward.
//
//   S_t = a S_{t-1} + v_t k_t^T   (d_v x d_k, fp32),   o_t = s S_t q_t,   a = exp(log_decay[head]).
//
// In chunks of 128 tokens (n in the last), with X the state before the chunk,
//   o_i = s [ sum_{j <= i} a^(i-j) (q_i.k_j) v_j + a^(i+1) X q_i ],
//   X'  = a^n X + sum_j a^(n-1-j) v_j k_j^T.
//
// The gradients have the same form. With D_t = s do_t q_t^T + a D_{t+1}
// (D_T = s do_T q_T^T + dS):
//   dq_t = s S_t^T do_t   runs forward  with (q, k, v) := (do, v, k), state S0^T,
//   dk_t = D_t^T v_t      runs backward with (v, do, q), state dS^T,
//   dv_t = D_t k_t        runs backward with (k, q, do), state dS; its last state
// is dS0. A pass that runs backward carries R_t = a D_t (the state is decayed
// when it leaves a token, not when it enters the next), so with i counted from
// the sequence's end its factors are a^i on the state and a^(n-j) on the update.
// One kernel takes a list of such passes ("jobs"); the three of a backward run
// in one launch and share their tensors' reads through L2.
//
// One CTA takes one (sequence, head, job, segment) and walks the segment's
// chunks with X in registers. Per chunk: S1 = Q K^T; masked and weighted, P = bf16
// in TMEM; O = Q X^T, its rows times a^(i+1) in TMEM, then O += P V, with X rounded to
// bf16 in shared memory (outputs are bf16, so each of the two operand roundings adds
// what the output's own rounding is). (With the factor's inverse in P and the factor
// on the way out that pass can be saved, 0.6 of 21.1 us at 512 tokens, 2.4 of 117 at
// 11300; but the inverse is out of range where a head forgets fast, and held back it
// lets a share of the old state through that the head has forgotten.)
// W = V'^T K, where V' = a^(n-1-j) v_j enters
// as three bf16 parts (24 bits together), so that the state, which is fp32
// outside, keeps fp32 accuracy. W starts from zero in every chunk and is added to
// X in registers: the tensor cores' accumulation rounds toward zero, and over a
// long sequence that would pull the state down.
//
// V'^T is the left operand from TMEM: transposed loads of V's tile give a thread
// pairs of tokens of a channel, the words of that operand. (As a shared
// memory operand it cost 96 KB of stores a chunk and twice the tensor time: the
// products then read both operands at the rate of shared memory.)
//
// What bounds it: a chunk's four tiles (128 KB at d = 128) take about 2.9 us of
// one SM's share of the HBM rate; its products about 4500 cycles (QK and QX with
// both operands in shared memory 1100 each, PV 560, three parts of W 1700). No
// part may wait for another, so each has its own warps, joined by barriers:
//   warp 0 TMA loads; warp 1 issues QK, QX, PV; warp 2 issues W; warp 3 TMA stores;
//   warps 4-11 make P and the output rows (half the columns each four warps);
//   warps 12-19 hold the state (two threads to a row of X, half its columns each);
//   warps 20-27 make V'.
// V' is made in steps of 32 tokens, the two halves of warps 20-27 taking turns
// with a buffer each. Two chunks' tiles are in shared memory; an output tile is
// staged in the slot of the V tile it no longer needs and leaves by TMA.
// Where (sequences x heads) leave SMs idle, long sequences are cut into segments:
// a first launch forms every segment's own state from K and V alone, a small
// kernel joins them in order, and the main launch starts each segment from its
// state.
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "seq.cuh"
#include "sm100.cuh"
#include "tmap.h"

namespace vda {

namespace {

constexpr int kC = 128;  // tokens per chunk
constexpr int kThreads = 896;
constexpr int kMaxJobs = 3;

template <int D>
struct DaCfg {
  static constexpr int kAtoms = D / 64;
  static constexpr int kTileBytes = kC * D * 2;
  static constexpr int kStep = 32;           // tokens of V' per step
  static constexpr int kSteps = kC / kStep;  // steps per chunk
  static constexpr int kXOff = 6 * kTileBytes;
  static constexpr int kBarOff = kXOff + D * D * 2;
  static constexpr int kSmemBytes = kBarOff + 2048 + 1024;
  // TMEM columns: S1, O, W (where there is room two of D columns, see kWs); V' in 64
  // columns a buffer (three parts of 16).
  static constexpr uint32_t kS1 = 0, kO = 128, kW = 256, kVp = 384;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kIdescS = sm100::idesc_bf16_f32(128, 128, false, false);
  static constexpr uint32_t kIdescPV = sm100::idesc_bf16_f32(128, D, false, true);
  static constexpr uint32_t kIdescQX = sm100::idesc_bf16_f32(128, D, false, false);
  static_assert(kSmemBytes <= 232448, "more shared memory than a CTA may use");
};

struct DaMaps {
  CUtensorMap m[4];            // token tensors
  CUtensorMap out[kMaxJobs];   // the jobs' outputs
};

struct DaJob {
  int q, k, v;               // which map plays which part
  int reverse;
  int init_t;                // the initial state is read transposed
  float s_in, s_out, s_up;   // factors of P V (beside X Q), of the output and of the update
  const float* init;         // [N, H, d, d], nullable (zero)
  float* last;               // [N, H, d, d], nullable
  __nv_bfloat16* out;
  long long out_row;
};

struct DaArgs {
  int N, H, T, njobs;
  int seg;                  // chunks per segment
  int items;                // entries of seg_state: segments of the sequences that have several, at most
  const int* cu;
  const float* log_decay;   // [H]
  DaJob job[kMaxJobs];
  float* seg_state;         // [items][H][njobs][d * d]
  uint32_t* status;
  uint32_t wait_ns;
};

// a^e for the head's log2 decay g2 (finite, see head_decay).
__device__ __forceinline__ float power(float g2, int e) { return exp2f(g2 * (float)e); }

// log2 of the head's decay. From 2^-300 down a factor is 0 in fp32 whatever the
// exponent, and -inf would give NaN at distance 0.
__device__ __forceinline__ float head_decay(const DaArgs& a, int h) {
  const float g = __ldg(a.log_decay + h) * 1.4426950408889634f;
  return g < -300.f ? -300.f : g;
}

// Tokens [lo, hi) of the processing-order chunks [p0, p1) of a sequence of len tokens.
__device__ __forceinline__ void chunk_tokens(int len, int reverse, int p0, int p1, int& lo, int& hi) {
  const int nch = (len + kC - 1) / kC;
  lo = reverse ? (nch - p1) * kC : p0 * kC;
  hi = min(len, reverse ? (nch - p0) * kC : p1 * kC);
}

// Segments of sequence i, where it has several: a sequence of one has no entry in seg_state.
__device__ __forceinline__ int cut_segments(const DaArgs& a, int i, int seg_tokens) {
  int lo, hi;
  seq::bounds(a.cu, i, a.T, lo, hi);
  const int n = (hi - lo + seg_tokens - 1) / seg_tokens;
  return n > 1 ? n : 0;
}

// Those of the sequences before sequence sq: where its own begin in seg_state. Every
// thread of the block calls it; up to 32 sequences each warp counts by itself.
__device__ __forceinline__ int segments_before(const DaArgs& a, int sq, int* scratch) {
  const int seg_tokens = a.seg * kC;
  if (a.N <= 32) {
    const int lane = threadIdx.x % 32;
    return (int)__reduce_add_sync(0xffffffffu, lane < sq ? cut_segments(a, lane, seg_tokens) : 0);
  }
  if (threadIdx.x == 0) *scratch = 0;
  __syncthreads();
  int n = 0;
  for (int i = threadIdx.x; i < sq; i += blockDim.x) n += cut_segments(a, i, seg_tokens);
  if (n) atomicAdd(scratch, n);
  __syncthreads();
  return *scratch;
}

// x = hi + mid + lo, each a bf16 (the upper half of a word), exactly: 8 bits of
// the 24 each, cut off, not rounded. Returns the packed pairs of two values.
__device__ __forceinline__ void split3(float2 x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  const float2 neg = make_float2(-1.f, -1.f);
  hi = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
  x = __ffma2_rn(make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)), neg, x);
  mid = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
  x = __ffma2_rn(make_float2(__uint_as_float(mid << 16), __uint_as_float(mid & 0xffff0000u)), neg, x);
  lo = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
}

// Shared memory read where it stands: the weights do not change from chunk to
// chunk, and hoisted out of the loop they would not fit the registers.
__device__ __forceinline__ float shared_float(const float* p) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(sm100::smem_u32(p)));
  return v;
}
__device__ __forceinline__ float2 shared_float2(const float* p) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(sm100::smem_u32(p)));
  return v;
}
// A value the compiler may not carry over from an earlier pass of a loop: the
// issuing warps have few registers, and operands built from loop constants would
// be kept in spilled ones.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
  asm volatile("" : "+r"(v));
  return v;
}

template <int D, bool kStateOnly>
__global__ void __launch_bounds__(kThreads, 1) decay_attn_tc_kernel(const __grid_constant__ DaMaps maps,
                                                                    const __grid_constant__ DaArgs a) {
  using C = DaCfg<D>;
  using namespace sm100;
  // Groups of four warps that make V', each with a buffer and every kMakers-th
  // step. Where no output is made all four groups do, in the columns S1 and O leave.
  constexpr int kMakers = kStateOnly ? 4 : 2;
  constexpr uint32_t kVpCol = kStateOnly ? 0 : C::kVp;
  // Buffers of W: with two the next chunk's products need not wait until the state's
  // warps have read the last one's. Only with outputs at d = 128 all columns are taken.
  constexpr int kWs = kStateOnly || D == 64 ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  uint8_t* sX = smem + C::kXOff;
  uint64_t* rfull = reinterpret_cast<uint64_t*>(smem + C::kBarOff);  // [6], see slot_of
  uint64_t* rempty = rfull + 6;
  uint64_t* sfull = rempty + 6;
  uint64_t* pfull = sfull + 1;
  uint64_t* qxdone = pfull + 1;
  uint64_t* odone = qxdone + 1;
  uint64_t* oempty = odone + 1;
  uint64_t* vpfull = oempty + 1;  // [kMakers]
  uint64_t* vpempty = vpfull + kMakers;
  uint64_t* wfull = vpempty + kMakers;  // [kWs]
  uint64_t* wempty = wfull + kWs;
  uint64_t* xfull = wempty + kWs;
  uint64_t* ofull = xfull + 1;  // an output tile is staged
  uint64_t* drain = ofull + 1;  // both issuing warps
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* v_read = tmem_slot + 2;  // chunks whose V tile V' has been made from
  int* scratch = reinterpret_cast<int*>(tmem_slot + 4);
  float* pw = reinterpret_cast<float*>(scratch + 40);  // [32 + 64], see below
  float* wt = pw + 96;                                 // [256] weights of V' in a whole chunk, then zeros
  static_assert((21 + 2 * kMakers + 2 * kWs) * 8 + 16 + 160 + 4 * (96 + 256) + 16 <= 2048, "barrier block overflows its allowance");

  if (kStateOnly) seq::grid_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int jb = blockIdx.x % a.njobs;
  const int h = (blockIdx.x / a.njobs) % a.H;
  const int item = blockIdx.x / a.njobs / a.H;
  const DaJob& job = a.job[jb];
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < 6; ++i) {
      mbar_init(&rfull[i], 1);
      mbar_init(&rempty[i], 2);
    }
    *abort_flag = 0;
    fence_mbar_init();
    if (!kStateOnly) prefetch_tmap(&maps.m[job.q]);
    prefetch_tmap(&maps.m[job.k]);
    prefetch_tmap(&maps.m[job.v]);
  }
  if (warp == 1 && lane == 0) {
    mbar_init(sfull, 1);
    mbar_init(pfull, 8);
    mbar_init(qxdone, 1);
    mbar_init(odone, 1);
    mbar_init(oempty, 8);
    for (int i = 0; i < kMakers; ++i) {
      mbar_init(&vpfull[i], 4);
      mbar_init(&vpempty[i], 1);
    }
    for (int i = 0; i < kWs; ++i) {
      mbar_init(&wfull[i], 1);
      mbar_init(&wempty[i], 8);
    }
    mbar_init(xfull, 8);
    mbar_init(ofull, 8);
    mbar_init(drain, 2);
    *v_read = 0;
    fence_mbar_init();
  }
  const int seg_tokens = a.seg * kC;
  const float g2 = head_decay(a, h);
  int part;
  // An empty sequence still has a state. The launch that forms states leaves out a
  // sequence's last segment: nothing follows it.
  const int sq = seq::find_item(
      item, a.N, scratch, reinterpret_cast<int*>(smem),
      [&](int i) {
        int lo, hi;
        seq::bounds(a.cu, i, a.T, lo, hi);
        return hi - lo;
      },
      [&](int n) { return max(1, (n + seg_tokens - 1) / seg_tokens) - (kStateOnly ? 1 : 0); }, part);
  if (sq < 0) {
    if (!kStateOnly) seq::grid_wait();
    return;
  }
  int lo, hi;
  seq::bounds(a.cu, sq, a.T, lo, hi);
  const int len = hi - lo;
  const int nch_all = (len + kC - 1) / kC;
  const int nparts = max(1, (len + seg_tokens - 1) / seg_tokens);
  const int p0 = part * a.seg, nch = min(nch_all, p0 + a.seg) - p0;
  const int rev = job.reverse;
  const long long st_off = ((long long)sq * a.H + h) * (D * D);
  float* seg_state = nullptr;
  if (a.seg_state && nparts > 1) {
    const int at = segments_before(a, sq, scratch) + part;
    if (at < a.items) seg_state = a.seg_state + (((long long)at * a.H + h) * a.njobs + jb) * (D * D);
  }
  // First token (within the tensor) and token count of the c-th chunk in processing order.
  // A segment's own state is formed from its last chunk to its first, so that what the
  // main launch reads first is what L2 has seen last.
  auto chunk = [&](int c, int& tok, int& n) {
    if (kStateOnly) c = nch - 1 - c;
    const int cc = rev ? nch_all - 1 - (p0 + c) : p0 + c;
    tok = lo + cc * kC;
    n = min(kC, len - cc * kC);
  };
  // A slot is free after two arrivals: of Q, two commits behind QX; of K, QK's and
  // W's; of V, W's (V' has been read) and the output tile's.
  // The six slots hold two chunks' tiles, or, without Q, three chunks'.
  constexpr int kStages = kStateOnly ? 3 : 2;
  auto slot_of = [&](int c, int t) { return kStateOnly ? c % 3 * 2 + t - 1 : (c & 1) * 3 + t; };
  auto tile_of = [&](int c, int t) { return smem + slot_of(c, t) * C::kTileBytes; };

  // The weight of a pair is a power of the row's distance from the near edge of a
  // block of 32 columns times one of the column's distance from that edge; on the
  // diagonal, where the two would overflow apart, one power of their distance, 0
  // where the row does not see the column: entry 32 + column - row of the second
  // table. The factor of P V goes with it.
  if (warp == 2) {
    pw[lane] = job.s_in * power(g2, rev ? lane : 31 - lane);
    pw[32 + lane] = rev || lane == 0 ? 0.f : job.s_in * power(g2, 32 - lane);
    pw[64 + lane] = rev || lane == 0 ? job.s_in * power(g2, lane) : 0.f;
  }
  if (warp >= 4 && warp < 12) {
    const int j = threadIdx.x - 128;
    wt[j] = j >= kC ? 0.f : job.s_up * power(g2, rev ? j + 1 : kC - 1 - j);
  }
  if (warp == 3) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  seq::set_up(warp == 0);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int loaded = 0;  // chunks whose copies have been issued
  auto wait1 = [&](uint64_t* bar, uint32_t n) -> bool {  // n-th phase of the barrier, n = 0, 1, ...
    return seq::bar_wait(bar, n & 1, abort_flag, a.status, a.wait_ns);
  };
  auto warp_wait = [&](uint64_t* bar, uint32_t n) -> bool {
    return seq::warp_wait(bar, n & 1, abort_flag, a.status, a.wait_ns);
  };

  // One step of V' by a group of four warps: its 32 tokens, 32 value channels (TMEM
  // lanes) to each warp. `maker` is the group's number.
  const int quad = warp % 4;
  const int row = quad * 32 + lane;
  const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
  // Each thread's row of V's tile for the transposed loads: eight tokens by eight
  // channels to a matrix, matrices (token group 0, 1) x (channel group 2 b, 2 b + 1).
  // A thread then holds pairs of tokens of channel lane / 4: words of the operand,
  // and the lanes and columns of a 16 x 128-bit store.
  const uint32_t v_off = (row / 64) * (kC * 128) + ((lane / 16) * 8 + lane % 8) * 128;
  const uint32_t v_chunk = (((quad & 1) * 4 + (lane / 8) % 2) ^ (lane % 8)) * 16;
  auto make_step = [&](int maker, int g) -> bool {
    const int c = g / C::kSteps, q = g % C::kSteps;
    int tok, n;
    chunk(c, tok, n);
    if (!warp_wait(&rfull[slot_of(c, 2)], c / kStages)) return false;
    if (n < kC && q < kMakers) {
      // Key and value rows behind the sequence are zeroed (by every group: each
      // reads and signals steps of its own).
      if (!warp_wait(&rfull[slot_of(c, 1)], c / kStages)) return false;
      if (row >= n) {
        seq::zero_row(tile_of(c, 1), C::kAtoms, row, kC);
        seq::zero_row(tile_of(c, 2), C::kAtoms, row, kC);
      }
      fence_proxy_async_smem();
      __syncwarp();
      asm volatile("bar.sync %0, 128;" ::"r"(1 + maker) : "memory");
    }
    if (g >= kMakers && !warp_wait(&vpempty[maker], g / kMakers - 1)) return false;
    tc_fence_after();
    if (row < D) {
      // Forward, a token's weight goes by its distance from the chunk's end: in a
      // ragged chunk the table is read from further on.
      const float* w = wt + (rev ? 0 : kC - n) + q * C::kStep + (lane % 4) * 2;
      const uint8_t* src = tile_of(c, 2) + v_off + q * (C::kStep * 128);
      uint32_t dst = tmem + lane_off + kVpCol + maker * 64;
      uint32_t chunk_at = v_chunk;
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {  // channels 16 b .. 16 b + 15 of the warp's 32
        uint32_t out[3][8];
#pragma unroll
        for (int t2 = 0; t2 < 2; ++t2) {  // tokens 16 t2 .. 16 t2 + 15
          uint32_t in[4];
          seq::ldmatrix4_trans(in, src + t2 * 2048 + chunk_at);
#pragma unroll
          for (int m = 0; m < 4; ++m) {  // tokens 8 (m / 2) .., channels 8 (m % 2) ..
            const int o = t2 * 4 + m, j = t2 * 16 + (m / 2) * 8;
            split3(__fmul2_rn(make_float2(__uint_as_float(in[m] << 16), __uint_as_float(in[m] & 0xffff0000u)),
                              make_float2(w[j], w[j + 1])),
                   out[0][o], out[1][o], out[2][o]);
          }
        }
#pragma unroll
        for (int p3 = 0; p3 < 3; ++p3) seq::tmem_st_16x128b_x4(dst + p3 * 16, out[p3]);
        dst += 16u << 16;
        chunk_at ^= 32;  // two 16-byte chunks on
      }
      tmem_st_wait();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&vpfull[maker]);
    return true;
  };
  // A warp's steps, every kMakers-th. One whose wait gave up arrives at the group's
  // barrier (a ragged chunk is the walk's last or first, so a group meets there once),
  // so that the other three do not wait for it.
  auto make_steps = [&](int maker, int steps) {
    for (int g = maker; g < steps; g += kMakers)
      if (!make_step(maker, g)) {
        __syncwarp();
        asm volatile("bar.arrive %0, 128;" ::"r"(1 + maker) : "memory");
        break;
      }
  };

  // 896 threads start with 72 registers each; the loading, issuing and V' warps give
  // some of theirs to the others (40 + 2 x 80 + 2 x 96 + 2 x 56 = 504 = 7 x 72).
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      if (seq::elect_one()) {
        bool ok = true;
        for (int c = 0; c < nch && ok; ++c) {
          int tok, n;
          chunk(c, tok, n);
          for (int t = kStateOnly ? 1 : 0; t < 3; ++t) {
            const CUtensorMap* m = &maps.m[t == 0 ? job.q : t == 1 ? job.k : job.v];
            uint64_t* full = &rfull[slot_of(c, t)];
            if (!(ok = wait1(&rempty[slot_of(c, t)], c / kStages + 1))) break;
            mbar_arrive_expect_tx(full, C::kTileBytes);
#pragma unroll
            for (int at = 0; at < C::kAtoms; ++at)
              tma_load_3d(tile_of(c, t) + at * (kC * 128), m, full, at * 64, h, tok);
            loaded = c * 3 + t + 1;
          }
        }
        if (*abort_flag) {
          // Let every issued copy land before the CTA's shared memory is released.
          for (int i = max(0, loaded - 3 * kStages); i < loaded; ++i)
            if (!kStateOnly || i % 3 != 0)
              mbar_wait(&rfull[slot_of(i / 3, i % 3)], (i / 3 / kStages) & 1, nullptr, a.status, a.wait_ns);
        }
      }
    } else if (warp == 1) {
      if (seq::elect_one()) {
        bool ok = true;
        if (!kStateOnly) {
          for (int c = 0; c < nch; ++c) {
            // The address field of a descriptor counts 16 bytes: steps are added to it.
            const uint64_t dq = smem_desc_sw128(smem_u32(tile_of(c, 0)), 16, 1024);
            const uint64_t dk = smem_desc_sw128(smem_u32(tile_of(c, 1)), 16, 1024);
            const uint64_t dv = smem_desc_sw128(smem_u32(tile_of(c, 2)), kC * 128, 1024);
            const uint64_t dx = smem_desc_sw128(opaque(smem_u32(sX)), 16, 1024);
            const uint32_t tm = opaque(tmem);
            if (!(ok = wait1(&rfull[slot_of(c, 0)], c / kStages) && wait1(&rfull[slot_of(c, 1)], c / kStages))) break;
            tc_fence_after();
#pragma unroll 1
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk / 4) * (kC * 128) + (kk % 4) * 32;
              mma_f16(tm + C::kS1, dq + (off >> 4), dk + (off >> 4), C::kIdescS, kk > 0 ? 1u : 0u);
            }
            mma_commit(sfull);
            mma_commit(&rempty[slot_of(c, 1)]);
            if (!(ok = wait1(xfull, c))) break;
            if (c > 0 && !(ok = wait1(oempty, c - 1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk / 4) * (kC * 128) + (kk % 4) * 32;
              const uint32_t xoff = (kk / 4) * (D * 128) + (kk % 4) * 32;
              mma_f16(tm + C::kO, dq + (off >> 4), dx + (xoff >> 4), C::kIdescQX, kk > 0 ? 1u : 0u);
            }
            mma_commit(qxdone);
            mma_commit(&rempty[slot_of(c, 0)]);
            mma_commit(&rempty[slot_of(c, 0)]);
            if (!(ok = wait1(pfull, c) && wait1(&rfull[slot_of(c, 2)], c / kStages))) break;
            tc_fence_after();
#pragma unroll 1
            for (int kk = 0; kk < kC / 16; ++kk)
              mma_f16_ts(tm + C::kO, tm + C::kS1 + (kk / 4) * 64 + (kk % 4) * 8, dv + kk * 128, C::kIdescPV, 1u);
            mma_commit(odone);
          }
        }
        mma_commit(drain);
      }
    } else if (warp == 2) {
      if (seq::elect_one()) {
        bool ok = true;
        for (int c = 0; c < nch && ok; ++c) {
          const uint64_t dk = smem_desc_sw128(smem_u32(tile_of(c, 1)), kC * 128, 1024);
          const int wb = c % kWs;
          const uint32_t w_at = tmem + C::kW + wb * D;
          if (!(ok = wait1(&rfull[slot_of(c, 1)], c / kStages))) break;
#pragma unroll 1
          for (int q = 0; q < C::kSteps; ++q) {
            const int g = c * C::kSteps + q, maker = g % kMakers;
            if (!(ok = wait1(&vpfull[maker], g / kMakers))) break;
            if (q == 0 && c >= kWs && !(ok = wait1(&wempty[wb], c / kWs - 1))) break;
            tc_fence_after();
            const uint32_t av = tmem + kVpCol + maker * 64;
#pragma unroll 1
            for (int p3 = 0; p3 < 3; ++p3)
#pragma unroll
              for (int kk = 0; kk < C::kStep / 16; ++kk)
                mma_f16_ts(w_at, av + p3 * 16 + kk * 8, dk + (q * (C::kStep / 16) + kk) * 128, C::kIdescPV,
                           (q > 0 || p3 > 0 || kk > 0) ? 1u : 0u);
            mma_commit(&vpempty[maker]);
          }
          if (!ok) break;
          smem_release_u32(v_read, c + 1);
          mma_commit(&wfull[wb]);
          mma_commit(&rempty[slot_of(c, 1)]);
          mma_commit(&rempty[slot_of(c, 2)]);
          if (kStateOnly) {
            mma_commit(&rempty[slot_of(c, 1)]);
            mma_commit(&rempty[slot_of(c, 2)]);
          }
        }
        mma_commit(drain);
      }
    } else if (!kStateOnly) {
      if (seq::elect_one()) {
        // Whole tiles leave by TMA; of a ragged one the threads have stored the rows.
        for (int c = 0; c < nch; ++c) {
          int tok, n;
          chunk(c, tok, n);
          if (!wait1(ofull, c)) break;
          if (n == kC) {
#pragma unroll
            for (int at = 0; at < C::kAtoms; ++at)
              seq::tma_store_3d(&maps.out[jb], tile_of(c, 2) + at * (kC * 128), at * 64, h, tok);
            seq::bulk_commit();
            seq::bulk_wait_read0();
          }
          mbar_arrive(&rempty[slot_of(c, 2)]);
        }
      }
    }
    __syncwarp();
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 80;");
    // ---------------- P and the output rows: row i of the chunk per thread, half
    // the columns. The packed P of a half lies in the first columns of its own
    // logits, so no half overwrites what the other has yet to read.
    if (!kStateOnly) {
      const int half = (warp - 4) / 4;
      const int i = row;
      const uint32_t sa = tmem + lane_off + C::kS1 + half * 64;
      const uint32_t oa = tmem + lane_off + C::kO + half * (D / 2);
      bool ok = true;
      for (int c = 0; c < nch && ok; ++c) {
        int tok, n;
        chunk(c, tok, n);
        // The square root of the state's factor, a^(i+1) forward, a^(distance from the end)
        // backward: the factor alone may lie below fp32's range where its product does not.
        const float r = exp2f(0.5f * g2 * (float)(rev ? max(0, n - 1 - i) : i + 1));
        if (!(ok = warp_wait(sfull, c))) break;
        tc_fence_after();
        // Weight a^|i - j| of the pairs a row sees: j <= i forward, i <= j < n
        // backward. Of the four 32-column blocks this warp's own is the diagonal;
        // those before it (behind it) are seen whole, the others not at all.
#pragma unroll 1
        for (int b2 = 0; b2 < 2; ++b2) {
          const int c4 = half * 2 + b2, j0 = c4 * 32;
          uint32_t w[16];
          if (rev ? c4 < quad : c4 > quad) {
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = 0u;
          } else {
            uint32_t v[32];
            seq::tmem_ld32(sa + b2 * 32, v);
            tmem_ld_wait();
            if (c4 == quad) {
              const float* t = pw + 64 - lane;
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float wx = shared_float(t + 2 * k), wy = shared_float(t + 2 * k + 1);
                w[k] = seq::pack_bf16(wx != 0.f ? __uint_as_float(v[2 * k]) * wx : 0.f,
                                      wy != 0.f ? __uint_as_float(v[2 * k + 1]) * wy : 0.f);
              }
            } else {
              const float base = power(g2, rev ? j0 - i : i - j0 - 31);
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float2 x = __fmul2_rn(__fmul2_rn(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])),
                                                       make_float2(base, base)),
                                            shared_float2(pw + 2 * k));
                w[k] = seq::pack_bf16(x.x, x.y);
              }
            }
            if (n < j0 + 32) {  // columns behind the sequence
#pragma unroll
              for (int k = 0; k < 16; ++k) w[k] = j0 + 2 * k >= n ? 0u : j0 + 2 * k + 1 >= n ? w[k] & 0xffffu : w[k];
            }
          }
          tmem_st16(sa + b2 * 16, w);
        }
        // X's share by its factor, before P V is added.
        if (!(ok = warp_wait(qxdone, c))) break;
        tc_fence_after();
#pragma unroll 1
        for (int u = 0; u < D / 32; ++u) {
          uint32_t y[16];
          tmem_ld16(oa + u * 16, y);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * r * r);
          tmem_st16(oa + u * 16, y);
        }
        tmem_st_wait();
        uint8_t* vt = tile_of(c, 2);
        if (n < kC) {
          // Value rows behind the sequence are zeroed: 0 x NaN is NaN.
          if (!(ok = warp_wait(&rfull[slot_of(c, 2)], c / kStages))) break;
          if (i >= n) seq::zero_row(vt, C::kAtoms, i, kC);
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull);
        if (!(ok = warp_wait(odone, c))) break;
        tc_fence_after();
        // O into registers first: the next chunk's QX may then take its columns.
        const float f = job.s_out;
        uint32_t op[D / 64][16];
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
          uint32_t y[32];
          seq::tmem_ld32(oa + u * 32, y);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k)
            op[u][k] = seq::pack_bf16(__uint_as_float(y[2 * k]) * f, __uint_as_float(y[2 * k + 1]) * f);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(oempty);
        // A whole tile is staged where V was: P V is done with it, and V' when the
        // W warp has counted the chunk (that chain may be a chunk ahead of this
        // one, so it is a count and not a barrier's phase).
        if (n == kC && !(ok = __all_sync(0xffffffffu, smem_wait_geq(v_read, c + 1, abort_flag, a.status, a.wait_ns))))
          break;
        uint4* dst = reinterpret_cast<uint4*>(job.out + (long long)(tok + min(i, n - 1)) * job.out_row + h * D);
#pragma unroll
        for (int q8 = 0; q8 < D / 16; ++q8) {
          const uint32_t* o = &op[q8 / 4][q8 % 4 * 4];
          const uint4 o4 = make_uint4(o[0], o[1], o[2], o[3]);
          const int ch = half * (D / 16) + q8;
          if (n == kC) {
            *reinterpret_cast<uint4*>(vt + (ch / 8) * (kC * 128) + i * 128 + (((ch % 8) ^ (i & 7)) * 16)) = o4;
          } else if (i < n) {
            dst[ch] = o4;
          }
        }
        if (n == kC) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(ofull);
      }
    } else {
      make_steps((warp - 4) / 4, nch * C::kSteps);
    }
  } else if (warp < 20) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
    // ---------------- the state
    constexpr int kCols = D / 2;
    const int half = (warp - 12) / 4;
    const bool has_row = row < D;  // row of X
    float X[kCols];
    {
      const bool joined = !kStateOnly && nparts > 1;
      const float* src = kStateOnly ? nullptr : joined ? seg_state : job.init ? job.init + st_off : nullptr;
      const bool tr = !joined && job.init_t;
      if (!kStateOnly) seq::grid_wait();
#pragma unroll
      for (int k = 0; k < kCols; ++k) X[k] = 0.f;
      if (src && has_row) {
        if (tr) {
#pragma unroll
          for (int k = 0; k < kCols; ++k) X[k] = src[(half * kCols + k) * D + row];
        } else if constexpr (D == 128) {
          // Whole lines of the warp's 32 rows, then by way of shared memory (32 columns at
          // a time, in the part of the operand that this warp writes) to the rows' threads:
          // from those threads the loads took 4.5 us.
          uint8_t* st = sX + half * (D * 128) + quad * 4096;
          const float* at = src + (quad * 32 + lane / 8) * D + half * kCols + lane % 8 * 4;
          float4 in[2][8];
#pragma unroll
          for (int u = 0; u < 16; ++u) in[u / 8][u % 8] = *reinterpret_cast<const float4*>(at + u % 8 * 4 * D + u / 8 * 32);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = i * 4 + lane / 8;
              *reinterpret_cast<float4*>(st + r * 128 + ((lane ^ r) & 7) * 16) = in[u][i];
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float4 x = *reinterpret_cast<const float4*>(st + lane * 128 + ((lane ^ k) & 7) * 16);
              float* to = &X[u * 32 + k * 4];
              to[0] = x.x;
              to[1] = x.y;
              to[2] = x.z;
              to[3] = x.w;
            }
            __syncwarp();
          }
        } else {
#pragma unroll
          for (int k = 0; k < kCols; k += 4) {
            const float4 x = *reinterpret_cast<const float4*>(src + row * D + half * kCols + k);
            X[k] = x.x;
            X[k + 1] = x.y;
            X[k + 2] = x.z;
            X[k + 3] = x.w;
          }
        }
      }
    }
    // X as the bf16 K-major operand of Q X^T: row (value channel) x 64-column atoms.
    auto write_x = [&] {
      if (has_row) {
#pragma unroll
        for (int k8 = 0; k8 < kCols / 8; ++k8) {
          const int col = half * kCols + k8 * 8;
          uint8_t* p = sX + (col / 64) * (D * 128) + row * 128 + ((((col % 64) / 8) ^ (row & 7)) * 16);
          *reinterpret_cast<uint4*>(p) =
              make_uint4(seq::pack_bf16(X[k8 * 8], X[k8 * 8 + 1]), seq::pack_bf16(X[k8 * 8 + 2], X[k8 * 8 + 3]),
                         seq::pack_bf16(X[k8 * 8 + 4], X[k8 * 8 + 5]), seq::pack_bf16(X[k8 * 8 + 6], X[k8 * 8 + 7]));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(xfull);
    };
    // X' = a^n X + W of chunk c; from the last chunk to the first X' = X + a^(tokens behind) W.
    int seg_lo = 0, seg_hi = 0;
    if (kStateOnly) chunk_tokens(len, rev, p0, p0 + nch, seg_lo, seg_hi);
    auto take_w = [&](int c) -> bool {
      int tok, n;
      chunk(c, tok, n);
      const int wb = c % kWs;
      if (!warp_wait(&wfull[wb], c / kWs)) return false;
      tc_fence_after();
      const float f = power(g2, !kStateOnly ? n : rev ? tok - lo - seg_lo : seg_hi - (tok - lo + n));
#pragma unroll
      for (int k4 = 0; k4 < kCols / 16; ++k4) {
        uint32_t v[16];
        tmem_ld16(tmem + lane_off + C::kW + wb * D + half * kCols + k4 * 16, v);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          float* x = &X[k4 * 16 + k];
          const float2 w = make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
          const float2 was = make_float2(x[0], x[1]);
          const float2 y = __ffma2_rn(make_float2(f, f), kStateOnly ? w : was, kStateOnly ? was : w);
          x[0] = y.x;
          x[1] = y.y;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&wempty[wb]);
      return true;
    };
    bool ok = true;
    if (!kStateOnly && nch > 0) write_x();
    for (int c = 0; c < nch && ok; ++c) {
      if (!(ok = take_w(c))) break;
      if (!kStateOnly && c + 1 < nch) {
        if (!(ok = warp_wait(qxdone, c))) break;  // Q X^T of this chunk has read the old X
        write_x();
      }
    }
    float* last = kStateOnly ? seg_state : (part == nparts - 1 && job.last) ? job.last + st_off : nullptr;
    if (ok && last && has_row) {
      // Through shared memory, so that a warp's store takes whole lines (straight from
      // the rows' threads it took 3 us at d = 128): 32 rows of 16-byte pieces, swizzled
      // by the row, in the Q and K slots that the last chunk has not used. What used
      // them is done: W of the last chunk, which comes behind, has been read.
      constexpr int kPieces = kCols / 4, kRows = 32 / kPieces;
      uint8_t* st = smem + slot_of(nch, kStateOnly ? 1 : 0) * C::kTileBytes +
                    (half * (D / 32) + quad) * (32 * kCols * 4);
#pragma unroll
      for (int k = 0; k < kPieces; ++k)
        *reinterpret_cast<float4*>(st + lane * (kCols * 4) + ((k ^ (lane % kPieces)) * 16)) =
            make_float4(X[4 * k], X[4 * k + 1], X[4 * k + 2], X[4 * k + 3]);
      __syncwarp();
      const int piece = lane % kPieces;
#pragma unroll 4
      for (int r = lane / kPieces; r < 32; r += kRows)
        *reinterpret_cast<float4*>(last + (quad * 32 + r) * D + half * kCols + piece * 4) =
            *reinterpret_cast<const float4*>(st + r * (kCols * 4) + ((piece ^ (r % kPieces)) * 16));
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    // ---------------- V'
    make_steps(kMakers - 2 + (warp - 20) / 4, nch * C::kSteps);
  }

  // ---------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    if (lane == 0) mbar_wait(drain, 0, nullptr, a.status, a.wait_ns);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Turns each segment's own state into the state before it, in order, for the
// sequences that have several: block (sequence, head, job) x slices of the matrix.
template <int D>
__global__ void __launch_bounds__(256) decay_join_kernel(const __grid_constant__ DaArgs a) {
  constexpr int kBatch = 8;
  __shared__ int scratch;
  seq::grid_trigger();
  const int sq = blockIdx.y;
  const int jb = blockIdx.x % a.njobs, h = (blockIdx.x / a.njobs) % a.H;
  const int slice = blockIdx.x / a.njobs / a.H;
  const DaJob& job = a.job[jb];
  const int seg_tokens = a.seg * kC;
  int lo, hi;
  seq::bounds(a.cu, sq, a.T, lo, hi);
  const int len = hi - lo;
  const int nparts = max(1, (len + seg_tokens - 1) / seg_tokens);
  if (nparts == 1) {
    seq::grid_wait();
    return;
  }
  const int first_s = segments_before(a, sq, &scratch);
  // Sequences that overlap (a wrong prefix array) have more segments than there is room for.
  if (first_s + nparts > a.items) {
    seq::grid_wait();
    return;
  }
  const int e = (slice * 256 + threadIdx.x) * 4;
  const int r = e / D, c = e % D;
  const float g2 = head_decay(a, h);
  const float* init = job.init ? job.init + ((long long)sq * a.H + h) * (D * D) : nullptr;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (init) {
    if (job.init_t)
      x = make_float4(init[c * D + r], init[(c + 1) * D + r], init[(c + 2) * D + r], init[(c + 3) * D + r]);
    else
      x = *reinterpret_cast<const float4*>(init + e);
  }
  const int nch = (len + kC - 1) / kC;
  const long long stride = (long long)a.H * a.njobs * (D * D);
  seq::grid_wait();  // all that is read before is the caller's
  float* base = a.seg_state + (((long long)first_s * a.H + h) * a.njobs + jb) * (D * D) + e;
  for (int p0 = 0; p0 < nparts; p0 += kBatch) {  // the loads of a batch are in flight together
    float4 y[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (p0 + u + 1 < nparts) y[u] = *reinterpret_cast<const float4*>(base + (p0 + u) * stride);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int p = p0 + u;
      if (p >= nparts) break;
      *reinterpret_cast<float4*>(base + p * stride) = x;
      if (p + 1 == nparts) break;
      int t0, t1;
      chunk_tokens(len, job.reverse, p * a.seg, min(nch, (p + 1) * a.seg), t0, t1);
      const float f = power(g2, t1 - t0);
      x = make_float4(fmaf(f, x.x, y[u].x), fmaf(f, x.y, y[u].y), fmaf(f, x.z, y[u].z), fmaf(f, x.w, y[u].w));
    }
  }
}

// One token of every sequence: S <- a S + v k^T in place, o = s S q. Memory
// bound: the state is read and written once. A CTA of four warps takes kSlab rows of
// S (a value channel each), a lane D / 32 key channels of a row; two rows are in
// flight per warp. 32 rows to a CTA, or 8 (every row in flight at once) where CTAs
// are fewer than the SMs hold. Measured at 160 sequences of 24 heads, d = 128 (503 MB): 84.7 us, 5946
// GB/s; with four rows in flight 90.9, eight warps of four rows to a whole matrix
// 94.3, eight rows 101: many small CTAs mix reads and writes best.
template <int D, int kSlab>
__global__ void __launch_bounds__(128) decay_step_kernel(const vda_decay_config c, const __nv_bfloat16* Q,
                                                         const __nv_bfloat16* K, const __nv_bfloat16* V,
                                                         const float* log_decay, float* S, __nv_bfloat16* O) {
  constexpr int kPer = D / 32;
  constexpr int kRows = 2, slabs = D / kSlab;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int slab = blockIdx.x % slabs;
  const long long nh = blockIdx.x / slabs;
  const int h = (int)(nh % c.H);
  const long long n = nh / c.H;
  const float a = expf(__ldg(log_decay + h));
  float k[kPer], q[kPer];
#pragma unroll
  for (int e = 0; e < kPer; e += 2) {
    const float2 kf = __bfloat1622float2(
        *reinterpret_cast<const __nv_bfloat162*>(K + n * c.k_row + (long long)h * D + lane * kPer + e));
    const float2 qf = __bfloat1622float2(
        *reinterpret_cast<const __nv_bfloat162*>(Q + n * c.q_row + (long long)h * D + lane * kPer + e));
    k[e] = kf.x;
    k[e + 1] = kf.y;
    q[e] = qf.x;
    q[e + 1] = qf.y;
  }
  float* Sm = S + nh * (D * D);
  const __nv_bfloat16* Vr = V + n * c.v_row + (long long)h * D;
  __nv_bfloat16* Or = O + n * c.o_row + (long long)h * D;
#pragma unroll 1
  for (int r0 = slab * kSlab + warp * kRows; r0 < (slab + 1) * kSlab; r0 += 4 * kRows) {
    float x[kRows][kPer], o[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if constexpr (kPer == 4) {
        const float4 f = __ldcs(reinterpret_cast<const float4*>(Sm + (r0 + r) * D) + lane);
        x[r][0] = f.x; x[r][1] = f.y; x[r][2] = f.z; x[r][3] = f.w;
      } else {
        const float2 f = __ldcs(reinterpret_cast<const float2*>(Sm + (r0 + r) * D) + lane);
        x[r][0] = f.x; x[r][1] = f.y;
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float v = __bfloat162float(Vr[r0 + r]);
      o[r] = 0.f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        x[r][e] = fmaf(a, x[r][e], v * k[e]);
        o[r] = fmaf(x[r][e], q[e], o[r]);
      }
      if constexpr (kPer == 4)
        __stcs(reinterpret_cast<float4*>(Sm + (r0 + r) * D) + lane, make_float4(x[r][0], x[r][1], x[r][2], x[r][3]));
      else
        __stcs(reinterpret_cast<float2*>(Sm + (r0 + r) * D) + lane, make_float2(x[r][0], x[r][1]));
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1)
#pragma unroll
      for (int r = 0; r < kRows; ++r) o[r] += __shfl_xor_sync(0xffffffffu, o[r], m);
    if (lane < kRows) {
      float y = o[0];
#pragma unroll
      for (int r = 1; r < kRows; ++r) y = lane == r ? o[r] : y;
      Or[r0 + lane] = __float2bfloat16_rn(c.scale * y);
    }
  }
}

constexpr int kMinSegChunks = 4;
constexpr int kWholeChunks = 9;

// Chunks per segment: one SM's share of the whole work, so that a long sequence
// is cut into about as many CTAs as there are SMs, but not into less than
// kMinSegChunks (a segment reads its keys and values twice, and the launch that
// forms the segments' states costs its start). Up to kWholeChunks in all, nothing is
// cut: the two launches more cost what the shorter chain saves (one sequence of 24
// heads, d = 128, uncut, and in segments of 4: 6 chunks 27.5 and 32.6 us, 9 chunks 37.0
// and 33.3, 12 chunks 46.6 and 36.4; at d = 64 21.0 and 23.4, 28.8 and 26.1, 36.2 and
// 27.0: the two meet between 7 and 8).
int segment_chunks(const vda_decay_config& c, int njobs) {
  const long long chunks = ((long long)c.T + kC - 1) / kC;
  if (chunks <= kWholeChunks) return kWholeChunks;
  const long long share = ((chunks + c.N / 2) * c.H * njobs + 147) / 148;
  return (int)std::min<long long>(1 << 20, std::max<long long>(kMinSegChunks, share));
}
// Segments of all sequences, at most.
long long segment_items(const vda_decay_config& c, int seg) { return (long long)c.T / ((long long)seg * kC) + c.N; }
// Those of the sequences that have several: a sequence of x > 1 segments' tokens has
// ceil(x) <= 2 floor(x), and the floors together are at most the tensor's.
long long state_items(const vda_decay_config& c, int seg) {
  return std::min(segment_items(c, seg), 2 * ((long long)c.T / ((long long)seg * kC)));
}

template <int D>
cudaError_t launch_d(const vda_decay_config& c, DaArgs& a, const void* const ptr[4], const long long row[4], int nmaps,
                     void* ws, cudaStream_t s) {
  using C = DaCfg<D>;
  a.seg = segment_chunks(c, a.njobs);
  const bool whole = (long long)c.T <= (long long)a.seg * kC;  // no sequence can be longer than a segment
  const long long items = segment_items(c, a.seg);
  a.items = (int)state_items(c, a.seg);
  a.seg_state = whole ? nullptr : static_cast<float*>(ws);
  a.wait_ns = 2000000000u;
  const long long grid = items * c.H * a.njobs;
  if (grid >= (1LL << 31) || c.N > 65535) return cudaErrorInvalidConfiguration;
  DaMaps maps{};
  cudaError_t e;
  uint64_t dims[3] = {(uint64_t)D, (uint64_t)c.H, (uint64_t)std::max(1, c.T)};
  uint32_t box[3] = {64, 1, (uint32_t)kC};
  for (int i = 0; i < nmaps; ++i) {
    uint64_t str[2] = {(uint64_t)D * 2, (uint64_t)row[i] * 2};
    if ((e = make_tmap_bf16(&maps.m[i], ptr[i], 3, dims, str, box)) != cudaSuccess) return e;
  }
  for (int j = 0; j < a.njobs; ++j) {
    uint64_t str[2] = {(uint64_t)D * 2, (uint64_t)a.job[j].out_row * 2};
    if ((e = make_tmap_bf16(&maps.out[j], a.job[j].out, 3, dims, str, box)) != cudaSuccess) return e;
  }
  const void* main_fn = reinterpret_cast<const void*>(decay_attn_tc_kernel<D, false>);
  const void* state_fn = reinterpret_cast<const void*>(decay_attn_tc_kernel<D, true>);
  if ((e = set_max_dynamic_smem(main_fn, C::kSmemBytes)) != cudaSuccess) return e;
  if ((e = set_max_dynamic_smem(state_fn, C::kSmemBytes)) != cudaSuccess) return e;
  if (!whole) {
    // Segments that another one follows: at most T / (a segment's tokens) of them.
    const long long states = (long long)c.T / ((long long)a.seg * kC) * c.H * a.njobs;
    decay_attn_tc_kernel<D, true><<<(unsigned)states, kThreads, C::kSmemBytes, s>>>(maps, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const dim3 jg((unsigned)(c.H * a.njobs * (D * D / 1024)), (unsigned)c.N);
    if ((e = seq::launch_behind(decay_join_kernel<D>, jg, 256, 0, s, a)) != cudaSuccess) return e;
    return seq::launch_behind(decay_attn_tc_kernel<D, false>, dim3((unsigned)grid), kThreads, C::kSmemBytes, s, maps, a);
  }
  decay_attn_tc_kernel<D, false><<<(unsigned)grid, kThreads, C::kSmemBytes, s>>>(maps, a);
  return cudaGetLastError();
}

}  // namespace

size_t decay_attention_workspace(const vda_decay_config& c, bool backward) {
  const int njobs = backward ? 3 : 1;
  const int seg = segment_chunks(c, njobs);
  if ((long long)c.T <= (long long)seg * kC) return 0;
  return (size_t)state_items(c, seg) * c.H * njobs * c.d * c.d * sizeof(float);
}

cudaError_t launch_decay_attention(const vda_decay_config& c, const void* Q, const void* K, const void* V,
                                   const float* log_decay, const int* cu, const float* S0, void* O, float* S_last,
                                   void* ws, uint32_t* status, cudaStream_t s) {
  DaArgs a{};
  a.N = c.N; a.H = c.H; a.T = c.T; a.njobs = 1;
  a.cu = cu;
  a.log_decay = log_decay;
  a.status = status;
  a.job[0] = DaJob{0, 1, 2, 0, 0, 1.f, c.scale, 1.f, S0, S_last, static_cast<__nv_bfloat16*>(O), c.o_row};
  const void* ptr[4] = {Q, K, V, nullptr};
  const long long row[4] = {c.q_row, c.k_row, c.v_row, 0};
  return c.d == 128 ? launch_d<128>(c, a, ptr, row, 3, ws, s) : launch_d<64>(c, a, ptr, row, 3, ws, s);
}

cudaError_t launch_decay_attention_backward(const vda_decay_config& c, const void* Q, const void* K, const void* V,
                                            const void* dO, const float* log_decay, const int* cu, const float* S0,
                                            const float* dS, void* dQ, void* dK, void* dV, float* dS0, void* ws,
                                            uint32_t* status, cudaStream_t s) {
  DaArgs a{};
  a.N = c.N; a.H = c.H; a.T = c.T; a.njobs = 3;
  a.cu = cu;
  a.log_decay = log_decay;
  a.status = status;
  const long long g_row = (long long)c.H * c.d;  // gradients are packed without gaps
  // Maps: 0 Q, 1 K, 2 V, 3 dO.
  a.job[0] = DaJob{3, 2, 1, 0, 1, 1.f, c.scale, 1.f, S0, nullptr, static_cast<__nv_bfloat16*>(dQ), g_row};
  a.job[1] = DaJob{2, 3, 0, 1, 1, c.scale, 1.f, c.scale, dS, nullptr, static_cast<__nv_bfloat16*>(dK), g_row};
  a.job[2] = DaJob{1, 0, 3, 1, 0, c.scale, 1.f, c.scale, dS, dS0, static_cast<__nv_bfloat16*>(dV), g_row};
  const void* ptr[4] = {Q, K, V, dO};
  const long long row[4] = {c.q_row, c.k_row, c.v_row, c.o_row};
  return c.d == 128 ? launch_d<128>(c, a, ptr, row, 4, ws, s) : launch_d<64>(c, a, ptr, row, 4, ws, s);
}

cudaError_t launch_decay_step(const vda_decay_config& c, const void* Q, const void* K, const void* V,
                              const float* log_decay, float* S, void* O, cudaStream_t s) {
  // Measured with 24 heads, d = 128, 8 (32) rows to a CTA: one sequence 1.9 (3.2) us,
  // four 2.9 (3.6), eight 4.7 (4.6), 24 9.9 (9.0).
  const bool few = (long long)c.N * c.H * (c.d / 32) < 148 * 5;
  const int slab = few ? 8 : 32;
  const long long grid = (long long)c.N * c.H * (c.d / slab);
  if (grid >= (1LL << 31)) return cudaErrorInvalidConfiguration;
  const auto* q = static_cast<const __nv_bfloat16*>(Q);
  const auto* k = static_cast<const __nv_bfloat16*>(K);
  const auto* v = static_cast<const __nv_bfloat16*>(V);
  auto* o = static_cast<__nv_bfloat16*>(O);
  auto* fn = c.d == 128 ? (few ? decay_step_kernel<128, 8> : decay_step_kernel<128, 32>)
                        : (few ? decay_step_kernel<64, 8> : decay_step_kernel<64, 32>);
  fn<<<(unsigned)grid, 128, 0, s>>>(c, q, k, v, log_decay, S, o);
  return cudaGetLastError();
}

}  // namespace vda
