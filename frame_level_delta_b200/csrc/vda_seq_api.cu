// Host side of the prompt path's calls (packed sequences): argument checks and
// the per-device status word. Every call only enqueues work.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <initializer_list>
#include <mutex>

#include "internal.h"
#include "seq.cuh"

namespace vda {

namespace {

// Word 0 is the status, word kTaken what the last poll took from it.
__device__ __align__(256) uint32_t g_sequence_status[64];
constexpr int kTaken = 32;

constexpr int kMaxDevices = 64;
std::atomic<void*> g_status_addr[kMaxDevices];
std::mutex g_status_mu;
std::mutex g_poll_mu;

// Reads the word and clears it in one step: what another stream's kernel reports
// meanwhile is either taken or left for the next poll.
__global__ void take_status_kernel(uint32_t* word) { word[kTaken] = atomicExch(word, 0u); }

}  // namespace

// The current device's address of the word, asked of the runtime once per device.
cudaError_t sequence_status(uint32_t** word) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  void* p = g_status_addr[dev].load(std::memory_order_acquire);
  if (p == nullptr) {
    std::lock_guard<std::mutex> lock(g_status_mu);
    p = g_status_addr[dev].load(std::memory_order_relaxed);
    if (p == nullptr) {
      if ((e = cudaGetSymbolAddress(&p, g_sequence_status)) != cudaSuccess) return e;
      g_status_addr[dev].store(p, std::memory_order_release);
    }
  }
  *word = static_cast<uint32_t*>(p);
  return cudaSuccess;
}

}  // namespace vda

using namespace vda;

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool any_null(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p) return true;
  return false;
}
bool all_aligned(std::initializer_list<const void*> ps, uintptr_t n) {
  for (const void* p : ps)
    if (p && !aligned(p, n)) return false;
  return true;
}
// Rows of `width` elements, `row` apart. 2^37 elements between rows is what a
// tensor map's stride field holds.
bool good_row(long long row, long long width) { return row >= width && row % 8 == 0 && row < (1LL << 37); }

vda_status check(const vda_attention_config* c) {
  if (!c || c->N < 1 || c->Hq < 1 || c->Hkv < 1 || c->Tq < 0 || c->Tk < 0) return VDA_ERR_INVALID_ARG;
  if (c->Hq % c->Hkv != 0) return VDA_ERR_INVALID_ARG;
  if (!(c->scale > 0.f) || !std::isfinite(c->scale)) return VDA_ERR_INVALID_ARG;
  if ((c->d != 64 && c->d != 128) || c->Hq / c->Hkv > 128) return VDA_ERR_UNSUPPORTED;
  const long long wq = (long long)c->Hq * c->d, wk = (long long)c->Hkv * c->d;
  if (!good_row(c->q_row, wq) || !good_row(c->o_row, wq) || !good_row(c->k_row, wk) || !good_row(c->v_row, wk))
    return VDA_ERR_INVALID_ARG;
  // The tile lists are 32-bit: N + Tq, Tk stay below 2^30.
  if (c->N >= (1 << 30) || c->Tq >= (1 << 30) || c->Tk >= (1 << 30)) return VDA_ERR_UNSUPPORTED;
  return VDA_OK;
}

vda_status check(const vda_decay_config* c) {
  if (!c || c->N < 1 || c->H < 1 || c->T < 0 || !std::isfinite(c->scale)) return VDA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return VDA_ERR_UNSUPPORTED;
  const long long w = (long long)c->H * c->d;
  if (!good_row(c->q_row, w) || !good_row(c->k_row, w) || !good_row(c->v_row, w) || !good_row(c->o_row, w))
    return VDA_ERR_INVALID_ARG;
  if (c->T >= (1 << 30)) return VDA_ERR_UNSUPPORTED;
  return VDA_OK;
}
// The prompt kernels run sequences on grid.y of one of their launches.
vda_status check_prompt(const vda_decay_config* c) {
  vda_status st = check(c);
  return st != VDA_OK ? st : c->N > 65535 ? VDA_ERR_UNSUPPORTED : VDA_OK;
}

vda_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return VDA_OK;
  if (!ws) return VDA_ERR_INVALID_ARG;
  if (!aligned(ws, 256)) return VDA_ERR_ALIGNMENT;
  return have < need ? VDA_ERR_WORKSPACE_TOO_SMALL : VDA_OK;
}

vda_status of(cudaError_t e) {
  return e == cudaSuccess ? VDA_OK : e == cudaErrorInvalidConfiguration ? VDA_ERR_UNSUPPORTED : VDA_ERR_CUDA;
}

// Rows of a tensor in memory: `count` of `width` bytes, `row` bytes apart.
struct Rows {
  const void* p;
  long long count, row, width;
};
Rows tokens(const void* p, long long count, long long row, long long width) { return {p, count, row * 2, width * 2}; }
Rows flat(const void* p, long long bytes) { return {p, 1, bytes, bytes}; }

// Whether two of them share a byte. Parts of one tensor (heads of a joint projection) lie
// between one another without sharing any.
bool overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || a.count < 1 || b.count < 1 || a.width < 1 || b.width < 1) return false;
  const unsigned long long pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
  auto end = [](unsigned long long p, const Rows& r) { return p + (unsigned long long)((r.count - 1) * r.row + r.width); };
  if (end(pa, a) <= pb || end(pb, b) <= pa) return false;
  if (a.count == 1 && b.count == 1) return true;
  if (a.row == b.row) {
    const long long at = (long long)(pb - pa) % a.row, off = at < 0 ? at + a.row : at;  // b's start within a's rows
    if (off >= a.width && a.row - off >= b.width) return false;
  }
  for (long long i = 0, j = 0; i < a.count && j < b.count;) {
    const unsigned long long x = pa + i * a.row, y = pb + j * b.row;
    if (x + a.width <= y) ++i;
    else if (y + b.width <= x) ++j;
    else return true;
  }
  return false;
}

// Outputs may not share memory with inputs or with one another.
bool outputs_overlap(std::initializer_list<Rows> outs, std::initializer_list<Rows> ins) {
  for (const Rows* o = outs.begin(); o != outs.end(); ++o) {
    for (const Rows& i : ins)
      if (overlap(*o, i)) return true;
    for (const Rows* p = o + 1; p != outs.end(); ++p)
      if (overlap(*o, *p)) return true;
  }
  return false;
}

// What becomes of states when there is no token at all: the state stays.
cudaError_t keep_state(const vda_decay_config& c, const float* from, float* to, cudaStream_t s) {
  if (!to || to == from) return cudaSuccess;
  const size_t bytes = (size_t)c.N * c.H * c.d * c.d * sizeof(float);
  return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(to, 0, bytes, s);
}

}  // namespace

extern "C" {

vda_status vda_causal_attention_workspace(const vda_attention_config* cfg, size_t* bytes) {
  if (!bytes) return VDA_ERR_INVALID_ARG;
  vda_status st = check(cfg);
  if (st == VDA_OK) *bytes = causal_attention_workspace(*cfg);
  return st;
}

vda_status vda_causal_attention(const vda_attention_config* cfg, const void* Q, const void* K, const void* V,
                                const int32_t* cu_q, const int32_t* cu_k, const int32_t* k_len, void* O, float* lse,
                                void* workspace, size_t workspace_bytes, void* stream) {
  vda_status st = check(cfg);
  if (st != VDA_OK) return st;
  if (any_null({cu_q, cu_k}) || (cfg->Tq > 0 && any_null({Q, O})) || (cfg->Tk > 0 && any_null({K, V})))
    return VDA_ERR_INVALID_ARG;
  if (!all_aligned({Q, K, V, O}, 16) || !all_aligned({cu_q, cu_k, k_len, lse}, 4)) return VDA_ERR_ALIGNMENT;
  if ((st = check_ws(workspace, workspace_bytes, causal_attention_workspace(*cfg))) != VDA_OK) return st;
  const long long wq = (long long)cfg->Hq * cfg->d, wk = (long long)cfg->Hkv * cfg->d;
  if (outputs_overlap({tokens(O, cfg->Tq, cfg->o_row, wq), flat(lse, 4LL * cfg->Tq * cfg->Hq)},
                      {tokens(Q, cfg->Tq, cfg->q_row, wq), tokens(K, cfg->Tk, cfg->k_row, wk),
                       tokens(V, cfg->Tk, cfg->v_row, wk)}))
    return VDA_ERR_INVALID_ARG;
  if (cfg->Tq == 0) return VDA_OK;
  uint32_t* status = nullptr;
  cudaError_t e = sequence_status(&status);
  if (e == cudaSuccess)
    e = launch_causal_attention(*cfg, Q, K, V, cu_q, cu_k, k_len, O, lse, workspace, status,
                                static_cast<cudaStream_t>(stream));
  return of(e);
}

vda_status vda_causal_attention_backward_workspace(const vda_attention_config* cfg, size_t* bytes) {
  if (!bytes) return VDA_ERR_INVALID_ARG;
  vda_status st = check(cfg);
  if (st == VDA_OK) *bytes = causal_attention_backward_workspace(*cfg);
  return st;
}

vda_status vda_causal_attention_backward(const vda_attention_config* cfg, const void* Q, const void* K,
                                         const void* V, const void* O, const void* dO, const float* lse,
                                         const int32_t* cu_q, const int32_t* cu_k, const int32_t* k_len, void* dQ,
                                         void* dK, void* dV, void* workspace, size_t workspace_bytes, void* stream) {
  vda_status st = check(cfg);
  if (st != VDA_OK) return st;
  if (any_null({cu_q, cu_k}) || (cfg->Tq > 0 && any_null({Q, O, dO, lse, dQ})) ||
      (cfg->Tk > 0 && any_null({K, V, dK, dV})))
    return VDA_ERR_INVALID_ARG;
  if (!all_aligned({Q, K, V, O, dO, dQ, dK, dV}, 16) || !all_aligned({cu_q, cu_k, k_len, lse}, 4))
    return VDA_ERR_ALIGNMENT;
  if ((st = check_ws(workspace, workspace_bytes, causal_attention_backward_workspace(*cfg))) != VDA_OK) return st;
  const long long wq = (long long)cfg->Hq * cfg->d, wk = (long long)cfg->Hkv * cfg->d;
  if (outputs_overlap({tokens(dQ, cfg->Tq, wq, wq), tokens(dK, cfg->Tk, wk, wk), tokens(dV, cfg->Tk, wk, wk)},
                      {tokens(Q, cfg->Tq, cfg->q_row, wq), tokens(K, cfg->Tk, cfg->k_row, wk),
                       tokens(V, cfg->Tk, cfg->v_row, wk), tokens(O, cfg->Tq, cfg->o_row, wq),
                       tokens(dO, cfg->Tq, cfg->o_row, wq), flat(lse, 4LL * cfg->Tq * cfg->Hq)}))
    return VDA_ERR_INVALID_ARG;
  if (cfg->Tq == 0 && cfg->Tk == 0) return VDA_OK;
  uint32_t* status = nullptr;
  cudaError_t e = sequence_status(&status);
  if (e == cudaSuccess)
    e = launch_causal_attention_backward(*cfg, Q, K, V, O, dO, lse, cu_q, cu_k, k_len, dQ, dK, dV, workspace, status,
                                         static_cast<cudaStream_t>(stream));
  return of(e);
}

vda_status vda_decay_attention_workspace(const vda_decay_config* cfg, size_t* bytes) {
  if (!bytes) return VDA_ERR_INVALID_ARG;
  vda_status st = check_prompt(cfg);
  if (st == VDA_OK) *bytes = decay_attention_workspace(*cfg, false);
  return st;
}

vda_status vda_decay_attention(const vda_decay_config* cfg, const void* Q, const void* K, const void* V,
                               const float* log_decay, const int32_t* cu, const float* S0, void* O, float* S,
                               void* workspace, size_t workspace_bytes, void* stream) {
  vda_status st = check_prompt(cfg);
  if (st != VDA_OK) return st;
  if (any_null({log_decay, cu}) || (cfg->T > 0 && any_null({Q, K, V, O}))) return VDA_ERR_INVALID_ARG;
  if (!all_aligned({Q, K, V, O, S0, S}, 16) || !all_aligned({log_decay, cu}, 4)) return VDA_ERR_ALIGNMENT;
  if ((st = check_ws(workspace, workspace_bytes, decay_attention_workspace(*cfg, false))) != VDA_OK) return st;
  const long long w = (long long)cfg->H * cfg->d, states = 4LL * cfg->N * w * cfg->d;
  if (outputs_overlap({tokens(O, cfg->T, cfg->o_row, w), flat(S, states)},
                      {tokens(Q, cfg->T, cfg->q_row, w), tokens(K, cfg->T, cfg->k_row, w),
                       tokens(V, cfg->T, cfg->v_row, w), flat(S == S0 ? nullptr : S0, states)}))
    return VDA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cfg->T == 0) return of(keep_state(*cfg, S0, S, s));
  uint32_t* status = nullptr;
  cudaError_t e = sequence_status(&status);
  if (e == cudaSuccess) e = launch_decay_attention(*cfg, Q, K, V, log_decay, cu, S0, O, S, workspace, status, s);
  return of(e);
}

vda_status vda_decay_attention_step(const vda_decay_config* cfg, const void* Q, const void* K, const void* V,
                                    const float* log_decay, float* S, void* O, void* stream) {
  vda_status st = check(cfg);
  if (st != VDA_OK) return st;
  if (cfg->T != cfg->N || any_null({Q, K, V, log_decay, S, O})) return VDA_ERR_INVALID_ARG;
  if (!all_aligned({Q, K, V, O, S}, 16) || !all_aligned({log_decay}, 4)) return VDA_ERR_ALIGNMENT;
  const long long w = (long long)cfg->H * cfg->d;
  if (outputs_overlap({tokens(O, cfg->T, cfg->o_row, w), flat(S, 4LL * cfg->N * w * cfg->d)},
                      {tokens(Q, cfg->T, cfg->q_row, w), tokens(K, cfg->T, cfg->k_row, w),
                       tokens(V, cfg->T, cfg->v_row, w)}))
    return VDA_ERR_INVALID_ARG;
  return of(launch_decay_step(*cfg, Q, K, V, log_decay, S, O, static_cast<cudaStream_t>(stream)));
}

vda_status vda_decay_attention_backward_workspace(const vda_decay_config* cfg, size_t* bytes) {
  if (!bytes) return VDA_ERR_INVALID_ARG;
  vda_status st = check_prompt(cfg);
  if (st == VDA_OK) *bytes = decay_attention_workspace(*cfg, true);
  return st;
}

vda_status vda_decay_attention_backward(const vda_decay_config* cfg, const void* Q, const void* K, const void* V,
                                        const void* dO, const float* log_decay, const int32_t* cu, const float* S0,
                                        const float* dS, void* dQ, void* dK, void* dV, float* dS0, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  vda_status st = check_prompt(cfg);
  if (st != VDA_OK) return st;
  if (any_null({log_decay, cu}) || (cfg->T > 0 && any_null({Q, K, V, dO, dQ, dK, dV}))) return VDA_ERR_INVALID_ARG;
  if (!all_aligned({Q, K, V, dO, dQ, dK, dV, S0, dS, dS0}, 16) || !all_aligned({log_decay, cu}, 4))
    return VDA_ERR_ALIGNMENT;
  if ((st = check_ws(workspace, workspace_bytes, decay_attention_workspace(*cfg, true))) != VDA_OK) return st;
  const long long w = (long long)cfg->H * cfg->d, states = 4LL * cfg->N * w * cfg->d;
  if (outputs_overlap({tokens(dQ, cfg->T, w, w), tokens(dK, cfg->T, w, w), tokens(dV, cfg->T, w, w), flat(dS0, states)},
                      {tokens(Q, cfg->T, cfg->q_row, w), tokens(K, cfg->T, cfg->k_row, w),
                       tokens(V, cfg->T, cfg->v_row, w), tokens(dO, cfg->T, cfg->o_row, w), flat(S0, states),
                       flat(dS, states)}))
    return VDA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cfg->T == 0) return of(keep_state(*cfg, dS, dS0, s));
  uint32_t* status = nullptr;
  cudaError_t e = sequence_status(&status);
  if (e == cudaSuccess)
    e = launch_decay_attention_backward(*cfg, Q, K, V, dO, log_decay, cu, S0, dS, dQ, dK, dV, dS0, workspace, status,
                                        s);
  return of(e);
}

vda_status vda_selftest_sequence_wait(uint64_t spins, void* stream) {
  uint32_t* word = nullptr;
  cudaError_t e = sequence_status(&word);
  if (e == cudaSuccess) e = launch_selftest_wait(word, spins, static_cast<cudaStream_t>(stream));
  return of(e);
}

vda_status vda_sequence_poll(void* stream) {
  uint32_t* word = nullptr;
  if (sequence_status(&word) != cudaSuccess) return VDA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return VDA_ERR_CUDA;
  // One poll at a time: kTaken is one word. The stream's work is done, so the wait below is short.
  std::lock_guard<std::mutex> lock(g_poll_mu);
  uint32_t v = 0;
  take_status_kernel<<<1, 1, 0, s>>>(word);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpyAsync(&v, word + kTaken, sizeof(v), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return VDA_ERR_CUDA;
  return v == 0 ? VDA_OK : VDA_ERR_TIMEOUT;
}

}  // extern "C"
