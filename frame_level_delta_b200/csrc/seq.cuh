// Packed sequences: what the kernels of the prompt path share. Sequence i of a
// packed tensor holds tokens cu[i] .. cu[i+1]-1. The prefix array is device data
// that the host never reads, so every bound taken from it is clamped to the
// tensor: a wrong array gives wrong rows, never an access out of range.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "sm100.cuh"

namespace vda {
namespace seq {

// [lo, hi) of sequence i, clamped to a tensor of T tokens.
__device__ __forceinline__ void bounds(const int* cu, int i, int T, int& lo, int& hi) {
  lo = min(max(__ldg(cu + i), 0), T);
  hi = min(max(__ldg(cu + i + 1), lo), T);
}

// Work item x of a list in which a sequence of size n has count(n) items (size(i):
// sequence i's tokens): returns the sequence and x's index within it, or -1 past the
// list's end. Up to kSorted sequences, the largest (by key(i), or by size) come first, so that no long one
// starts when the others are done; beyond, in their order. Every thread of the block
// calls it; `scratch` holds 40 ints, `big` 2 kSorted. Up to 32 sequences each warp
// finds the item by itself, so the warp that loads can start at once (a search by the
// block cost 2 us of a CTA's start, its code's first execution and four barriers); beyond,
// each pass takes blockDim.x sequences (one load and one scan). The caller
// synchronises the block.
constexpr int kSorted = 128;
struct BySize {};
template <typename Size, typename Count, typename Key = BySize>
__device__ __forceinline__ int find_item(int x, int N, int* scratch, int* big, Size size, Count count, int& idx,
                                         Key key = Key()) {
  constexpr bool by_size = std::is_same<Key, BySize>::value;
  auto key_of = [&](int i, int n) {
    if constexpr (by_size) return n;
    else return key(i);
  };
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = blockDim.x >> 5;
  if (N <= 32) {
    const int n_own = lane < N ? size(lane) : 0, c = lane < N ? count(n_own) : 0;
    const int own = lane < N ? key_of(lane, n_own) : 0;
    int lo = 0;  // items of the sequences before this lane's
#pragma unroll 4
    for (int j = 0; j < N; ++j) {
      const int s = __shfl_sync(0xffffffffu, own, j), n = __shfl_sync(0xffffffffu, c, j);
      lo += s > own || (s == own && j < lane) ? n : 0;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, lane < N && x >= lo && x - lo < c);
    if (hit == 0) return -1;
    const int sq = __ffs(hit) - 1;
    idx = x - __shfl_sync(0xffffffffu, lo, sq);
    return sq;
  }
  if (t == 0) scratch[33] = -1;
  const bool sorted = N <= kSorted;
  int own = 0;
  if (sorted) {
    if (t < N) big[t] = own = key_of(t, by_size ? size(t) : 0);
    __syncthreads();
    if (t < N) {
      int rank = 0;
      for (int j = 0; j < N; ++j) rank += big[j] > own || (big[j] == own && j < t);
      big[kSorted + rank] = t;
    }
    __syncthreads();
  }
  for (int base = 0; base < N; base += blockDim.x) {
    const int i = base + t;
    const int sq = sorted && i < N ? big[kSorted + i] : i;
    const int c = i < N ? count(by_size && sorted ? big[sq] : size(sq)) : 0;
    int inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    int off = 0, total = 0;
    for (int w = 0; w < warps; ++w) {
      const int n = scratch[w];
      if (w < warp) off += n;
      total += n;
    }
    const int hi = off + inc, lo = hi - c;
    if (x >= lo && x < hi) {
      scratch[33] = sq;
      scratch[34] = x - lo;
    }
    __syncthreads();
    if (scratch[33] >= 0) break;
    x -= total;
  }
  sm100::fence_proxy_async_smem();  // copies may land in `big` from here on
  __syncthreads();
  idx = scratch[34];
  return scratch[33];
}

// Of a call's launches, each after the first starts as the programmatic dependent of
// the one before it: its launch and set-up run under the other's end. The first
// starts in stream order, so what a call reads is complete for all of them. Every CTA
// of the others waits (grid_wait: until the launch before has ended and its writes are
// there) before it ends, or a later kernel of the stream could find an earlier launch
// still running.
__device__ __forceinline__ void grid_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P>
cudaError_t launch_behind(void (*fn)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s,
                          const P&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

// End of a CTA's set-up: every warp waits for it but the one that loads (`first`),
// whose copies need nothing that the others set up.
__device__ __forceinline__ void set_up(bool first) {
  if (first) {
    __syncwarp();
    asm volatile("bar.arrive 15, %0;" ::"r"(blockDim.x) : "memory");
  } else {
    asm volatile("bar.sync 15, %0;" ::"r"(blockDim.x) : "memory");
  }
}

// One lane of a converged warp, chosen by the hardware.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// Bounded wait for the phase with the given parity, with mbar_wait's rules, in few
// instructions: a kernel whose warps have different roles runs several loops at
// once, and their code has to fit the instruction caches together (with
// mbar_wait's longer loop and everything unrolled, the linear attention's working
// warps spent 8 to 10 cycles an instruction). The clock's lower word serves limits
// below 4 s. Every lane polls: with one lane polling for its warp, the backward's
// kernels took 6 to 19% longer.
__device__ __forceinline__ uint32_t globaltimer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status,
                                         uint32_t limit_ns) {
  const uint32_t t0 = globaltimer_lo();
  while (!sm100::mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    if (globaltimer_lo() - t0 > limit_ns) {
      *abort = 1;
      *reinterpret_cast<volatile uint32_t*>(status) = (uint32_t)VDA_ERR_TIMEOUT;
      return false;
    }
  }
  return true;
}
// The same by all lanes of a warp, which goes on only if all of them saw the phase.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status,
                                          uint32_t limit_ns) {
  return __all_sync(0xffffffffu, bar_wait(bar, parity, abort, status, limit_ns));
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The larger of two, NaN if one of them is (fmaxf gives the other).
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// 2^x for a pair on the FMA pipe, for -126 <= x (smaller arguments give 2^-126) and
// x < 127: x = n + r with n the nearest integer, taken from the low bits of
// x + 1.5 2^23, and 2^r by a polynomial of degree 4, the minimax fit of the
// relative error on [-1/2, 1/2] by the Remez exchange (2.6e-6).
__device__ __forceinline__ float2 ex2_fma(float2 x) {
  x = make_float2(fmaxf(x.x, -126.f), fmaxf(x.y, -126.f));
  const float magic = 12582912.f;
  const float2 t = __fadd2_rn(x, make_float2(magic, magic));
  const float2 r = __fadd2_rn(x, __ffma2_rn(t, make_float2(-1.f, -1.f), make_float2(magic, magic)));
  float2 p = make_float2(0.00957010190f, 0.00957010190f);
  p = __ffma2_rn(p, r, make_float2(0.05591786032f, 0.05591786032f));
  p = __ffma2_rn(p, r, make_float2(0.24024744828f, 0.24024744828f));
  p = __ffma2_rn(p, r, make_float2(0.69312181474f, 0.69312181474f));
  p = __ffma2_rn(p, r, make_float2(0.99999926145f, 0.99999926145f));
  return make_float2(__uint_as_float((__float_as_uint(t.x) << 23) + __float_as_uint(p.x)),
                     __uint_as_float((__float_as_uint(t.y) << 23) + __float_as_uint(p.y)));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return sm100::bf162_bits(__floats2bfloat162_rn(a, b));
}

// What a pair's packed bf16 values leave of it, packed.
__device__ __forceinline__ uint32_t pack_rest(float2 x, uint32_t w) {
  return pack_bf16(x.x - __uint_as_float(w << 16), x.y - __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// 16 lanes x 16 columns from the fragments of 8 x 8 matrices: word 2 i (2 i + 1) of
// a thread goes to lane thread / 4 (+ 8), column 4 i + thread % 4.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// Four 8 x 8 matrices of 16-bit values, transposed: lane l gives the address of row
// l % 8 of matrix l / 8 and receives values (2 (l % 4), 2 (l % 4) + 1) of column
// l / 4 of each.
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(sm100::smem_u32(p))
               : "memory");
}

// Stores a warp's 32 rows of kCols bf16 values, one row per lane (w: the lane's
// packed row; row: where it goes, null for a row that is none), through 32 x kCols
// values of shared memory that only this warp uses: the lanes of a store then write
// whole rows. (Row by row from the lanes that hold them, a store touches 32 lines;
// a tile's epilogue took 4500 cycles.)
template <int kCols>
__device__ __forceinline__ void store_rows(uint8_t* stage, const uint32_t (&w)[kCols / 2], __nv_bfloat16* row) {
  constexpr int kChunks = kCols / 8, kPer = 32 / kChunks;  // 16-byte chunks per row; rows per store
  const int lane = threadIdx.x & 31;
  auto at = [&](int r, int c) {
    // The 8 lanes of a phase hit 8 different 16-byte columns.
    const int x = kChunks >= 8 ? r & 7 : (r * kChunks / 8) & (kChunks - 1);
    return reinterpret_cast<uint4*>(stage + r * (kCols * 2) + ((c ^ x) * 16));
  };
#pragma unroll
  for (int c = 0; c < kChunks; ++c) *at(lane, c) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  __syncwarp();
  const int c = lane % kChunks;
#pragma unroll
  for (int it = 0; it < kChunks; ++it) {
    const int r = it * kPer + lane / kChunks;
    const unsigned long long p = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), r);
    const uint4 v = *at(r, c);
    if (p) *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p) + c * 8) = v;
  }
}

// 3-D tiled bulk tensor copy shared -> global (the issuing thread's bulk group),
// and the wait until the group's copies have read shared memory.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(sm100::smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read0() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// Zeroes token row `row` in each of `atoms` boxes of 64 channels (128-byte rows;
// whole rows, so the swizzle does not matter). For rows past a sequence's end:
// they hold another sequence's values or whatever lies behind the last one, and
// 0 x NaN is NaN.
__device__ __forceinline__ void zero_row(uint8_t* tile, int atoms, int row, int rows_per_atom) {
  for (int at = 0; at < atoms; ++at) {
    uint4* p = reinterpret_cast<uint4*>(tile + (size_t)at * rows_per_atom * 128 + row * 128);
#pragma unroll
    for (int c = 0; c < 8; ++c) p[c] = make_uint4(0, 0, 0, 0);
  }
}

}  // namespace seq

// One 32-bit status word per device, owned by the library: zero until a bounded
// device-side wait of a packed-sequence kernel gives up (then VDA_ERR_TIMEOUT),
// cleared by vda_sequence_poll. Returns the current device's address of it.
cudaError_t sequence_status(uint32_t** word);

}  // namespace vda
