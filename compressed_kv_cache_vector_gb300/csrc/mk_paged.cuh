// Declarations shared by the paged cache's kernels and their host side.
#pragma once

#include <cuda.h>
#include <cuda_fp8.h>

#include "mk_internal.cuh"

namespace mk {

// One layer of the pools and what every paged kernel needs besides.
struct PagedLayer {
  uint8_t* k;                   // [n_pages][n_kv][P][128] bf16 or e4m3
  uint8_t* v;
  float* k_scale;               // [n_pages][n_kv] (e4m3)
  float* v_scale;
  int32_t* err;                 // [0] status, [1] call that set it, [2] detail, [3] sequence, [4] aux
  uint32_t call;                // number of this call of the handle
  int32_t n_pages, n_kv, G, P, p_log2, e4m3;
};

// Device error codes of the paged calls (detail word), after DevErr's.
enum PagedErr : int32_t {
  ERR_PAGED_BATCH = 16,     // cu_new not ascending or past n_tokens, more new tokens than max_new, a length out of range
  ERR_PAGED_PAGE = 17,      // a page id outside [0, n_pages)
  ERR_PAGED_POSITION = 18,  // a rotary position outside [0, n_pos)
  ERR_PAGED_WAIT = 19,      // a copy or a matrix instruction did not complete within the wait bound (MK_ETIMEOUT)
};

constexpr uint32_t kPagedClosed = 0xffffffffu;  // in place of the call's number: no call's
constexpr int kPagedMaxCtas = 160;  // CTAs of a persistent attention kernel (GB300: 152 SMs)

// Tensor maps of the pools, 128-byte swizzle, dimensions {128 channels,
// kv head x page slot, layer x page}; a box is one 128-byte run of channels
// (all of them in e4m3, half in bf16) by 16 or 32 tokens.
struct PagedMaps {
  CUtensorMap k, v;
};
// The workspace's parts that the attention kernels use.
struct PagedScratch {
  float* part_acc;
  float* part_ml;
  int32_t* counters;          // [max_seqs][n_kv], zero between calls
  int32_t* prefill_counters;  // [kPagedMaxCtas], zero between calls
  float* prefill_part;        // paged_prefill_part_floats()
};
int64_t paged_prefill_part_floats();

#ifdef __CUDACC__
__device__ __forceinline__ void paged_error(const PagedLayer& L, int32_t detail, int32_t seq, int32_t aux,
                                            int32_t status = (int32_t)MK_EDEVICE) {
  const unsigned long long word = (unsigned long long)L.call << 32 | (uint32_t)status;
  if (atomicCAS(reinterpret_cast<unsigned long long*>(L.err), 0ull, word) == 0) {
    L.err[2] = detail;
    L.err[3] = seq;
    L.err[4] = aux;
  }
}
// Whether the error word keeps this call from working.  An error that the same
// call has set does not: its CTAs do not all start at once, and those behind
// the one that met a bad page have good ones to do (after a wait that ran out
// nothing is left to do).  A call that is kept from working closes the error
// word, so that a replay of the call that set it is kept from working too.
__device__ __forceinline__ bool paged_stopped(const PagedLayer& L) {
  const unsigned long long word = *reinterpret_cast<volatile unsigned long long*>(L.err);
  if (word == 0 || ((uint32_t)(word >> 32) == L.call && (uint32_t)word != (uint32_t)MK_ETIMEOUT)) return false;
  *reinterpret_cast<volatile uint32_t*>(&L.err[1]) = kPagedClosed;
  return true;
}

// Bounded wait for the phase with the given parity, as mbar_wait, with the
// limit (about 20 ms) counted in clocks: reading the global timer between two
// tries costs several hundred cycles of every wait that does not end at once.
__device__ __forceinline__ bool paged_wait(uint64_t* bar, unsigned parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > 40000000ll) return false;
  return true;
}
// The same for a full warp: if any lane gave up, all report failure.
__device__ __forceinline__ bool paged_wait_warp(uint64_t* bar, unsigned parity) {
  return __all_sync(FULL, paged_wait(bar, parity)) != 0;
}

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two e4m3 codes (low 16 bits) as two halves.
__device__ __forceinline__ uint32_t e4m3_h2(uint32_t two) {
  uint32_t r;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(r) : "r"(two));
  return r;
}
// Two numbers rounded to fp16 (F16) or bf16, the first in the low half.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (F16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Sequence i of a batch: its first row, new tokens and length.  ok is false
// (and the error word set by the callers) when they contradict the batch.
struct PagedSeq {
  int row0, n_new, len;
  bool ok;
};
__device__ __forceinline__ PagedSeq paged_seq(const mk_paged_batch& b, int P, int i, bool new_in_len) {
  PagedSeq s;
  s.row0 = b.cu_new ? b.cu_new[i] : i;
  s.n_new = (b.cu_new ? b.cu_new[i + 1] : i + 1) - s.row0;
  s.len = b.kv_len[i];
  s.ok = s.row0 >= 0 && s.n_new >= 0 && s.n_new <= b.max_new && (int64_t)s.row0 + s.n_new <= b.n_tokens && s.len >= 0 &&
         s.len <= (int64_t)b.table_stride * P && (!new_in_len || s.len >= s.n_new);
  return s;
}
#endif

cudaError_t launch_paged_append(const PagedLayer& L, const mk_paged_batch& b, const mk_rope& rope, const uint16_t* k,
                                int64_t k_stride, const uint16_t* v, int64_t v_stride, const uint16_t* q,
                                int64_t q_stride, uint16_t* q_out, int64_t q_out_stride, cudaStream_t s);
cudaError_t launch_paged_decode(const PagedLayer& L, const PagedMaps& maps, const PagedScratch& w, int layer,
                                const mk_paged_batch& b, bool several, bool causal, const uint16_t* q, int64_t q_stride,
                                float scale, uint16_t* out, int64_t out_stride, float* lse, cudaStream_t s);
cudaError_t launch_paged_prefill(const PagedLayer& L, const PagedScratch& w, const mk_paged_batch& b, bool causal,
                                 const uint16_t* q, int64_t q_stride, float scale, uint16_t* out, int64_t out_stride,
                                 float* lse, cudaStream_t s);

}  // namespace mk
