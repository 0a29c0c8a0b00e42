// Attention mass over the paged cache: what softmax weights each held token
// got, summed over query tokens and over the query heads of its kv head.
#include <algorithm>

#include "mk_paged.cuh"

namespace mk {

namespace {

// ---- a decode step's weights, from the logits that the attention left ----
// A thread a token: the group's weights 2^(z - lse2) summed and added.  HBM
// (mostly L2, where the logits still are): 4 G bytes read, 8 for the mass.
constexpr int kFoldThreads = 256;

__global__ void __launch_bounds__(kFoldThreads)
    k_mass_fold(PagedLayer L, mk_paged_batch b, const float* logits, const float* lse2, float* mass, int32_t first) {
  __shared__ int64_t s_end[MK_MAX_CALL_SEQS];  // tiles up to and with a sequence
  __shared__ int64_t s_wsum[kFoldThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_kv = L.n_kv, G = L.G;
  pdl_wait();
  pdl_trigger();
  if (__syncthreads_or(tid == 0 && paged_stopped(L))) return;
  int64_t total = 0;
  static_assert(kFoldThreads >= MK_MAX_CALL_SEQS, "one thread a sequence");
  {
    int64_t x = 0;
    if (tid < b.n_seqs) {
      const PagedSeq s = paged_seq(b, L.P, tid, false);
      if (s.ok && s.n_new == 1 && s.len > first) x = (int64_t)((s.len - first + kFoldThreads - 1) / kFoldThreads) * n_kv;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(FULL, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_wsum[warp] = x;
    __syncthreads();
    for (int w = 0; w < kFoldThreads / 32; ++w) {
      if (w < warp) x += s_wsum[w];
      total += s_wsum[w];
    }
    s_end[tid] = x;
    __syncthreads();
  }
  for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
    int seq = 0, hi = b.n_seqs - 1;
    while (seq < hi) {
      const int mid = (seq + hi) >> 1;
      if (s_end[mid] > tile) hi = mid; else seq = mid + 1;
    }
    const int64_t in = tile - (seq ? s_end[seq - 1] : 0);
    const int len = b.kv_len[seq], head = (int)(in % n_kv);
    const int64_t t = first + in / n_kv * kFoldThreads + tid;
    if (t >= len) continue;
    const int page = b.page_table[(int64_t)seq * b.table_stride + (t >> L.p_log2)];
    if (page < 0 || page >= L.n_pages) continue;  // recorded by the attention
    const int64_t unit = (int64_t)page * n_kv + head;
    const int slot = (int)t & (L.P - 1);
    float* to = mass + unit * L.P + slot;
    const float* z = logits + unit * G * L.P + slot;
    const float* ls = lse2 + ((int64_t)seq * n_kv + head) * G;
    float sum = 0.0f;
    for (int g = 0; g < G; ++g) sum += ex2(z[g * L.P] - ls[g]);
    *to = t == len - 1 ? sum : *to + sum;
  }
}

// ---- a prompt's weights ----
constexpr int kMassThreads = 256;

// A warp a key: lanes hold four channels each.
__global__ void __launch_bounds__(kMassThreads)
    k_prefill_mass(PagedLayer L, mk_paged_batch b, int32_t causal, const uint16_t* q, int64_t q_stride, float scale,
                   const float* lse, float* mass, int32_t first, int32_t add) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_kv = L.n_kv, G = L.G;
  pdl_wait();
  if (__syncthreads_or(tid == 0 && paged_stopped(L))) return;
  const int head = (int)(blockIdx.x % n_kv), seq = (int)(blockIdx.x / n_kv);
  const PagedSeq s = paged_seq(b, L.P, seq, false);
  if (!s.ok) {
    if (tid == 0) paged_error(L, ERR_PAGED_BATCH, seq, s.len);
    return;
  }
  if (s.n_new == 0) return;
  const int64_t step = (int64_t)gridDim.y * (kMassThreads / 32);
  for (int64_t t = first + (int64_t)blockIdx.y * (kMassThreads / 32) + warp; t < s.len; t += step) {
    const int page = b.page_table[(int64_t)seq * b.table_stride + (t >> L.p_log2)];
    if (page < 0 || page >= L.n_pages) {
      if (lane == 0) paged_error(L, ERR_PAGED_PAGE, seq, page);
      continue;
    }
    const int64_t unit = (int64_t)page * n_kv + head, row = unit * L.P + (t & (L.P - 1));
    float k[4];
    if (L.e4m3) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(L.k + row * D)[lane];
      const float sc = L.k_scale[unit];
      for (int e = 0; e < 2; ++e) {
        const uint32_t h = e4m3_h2(w >> (16 * e));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        k[2 * e] = f.x * sc;
        k[2 * e + 1] = f.y * sc;
      }
    } else {
      const uint2 w = reinterpret_cast<const uint2*>(L.k + row * D * 2)[lane];
      k[0] = bf2f(w.x & 0xffff);
      k[1] = bf2f(w.x >> 16);
      k[2] = bf2f(w.y & 0xffff);
      k[3] = bf2f(w.y >> 16);
    }
    // Query j sees the first len - n_new + j + 1 keys.
    const int64_t j0 = causal ? std::max<int64_t>(0, t - (s.len - s.n_new)) : 0;
    float sum = 0.0f;
    for (int64_t r = j0 * G; r < (int64_t)s.n_new * G; ++r) {
      const int64_t tok = s.row0 + r / G;
      const int h = head * G + (int)(r % G);
      const uint2 w = reinterpret_cast<const uint2*>(q + tok * q_stride + h * D)[lane];
      float z = bf2f(w.x & 0xffff) * k[0] + bf2f(w.x >> 16) * k[1] + bf2f(w.y & 0xffff) * k[2] + bf2f(w.y >> 16) * k[3];
      z = warp_sum(z);
      const float ls = lse[tok * n_kv * G + h];
      if (ls != -INFINITY) sum += ex2(z * scale - ls * kLog2e);
    }
    if (lane == 0) mass[row] = add && (!causal || t < s.len - s.n_new) ? mass[row] + sum : sum;
  }
}

}  // namespace

cudaError_t launch_paged_mass_fold(const PagedLayer& L, const PagedScratch& w, const mk_paged_batch& b,
                                   const float* logits, float* mass, int32_t first, cudaStream_t s) {
  int occ = 0, sms = 0;
  const cudaError_t e = kernel_smem_attr((const void*)k_mass_fold, 0, kFoldThreads, &occ, &sms);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_mass_fold, dim3((unsigned)((sms > 0 ? sms : 128) * occ)), dim3(kFoldThreads), 0, s, 0, L, b, logits,
                    (const float*)w.lse2, mass, first);
}

cudaError_t launch_paged_prefill_mass(const PagedLayer& L, const PagedScratch& w, const mk_paged_batch& b, bool causal,
                                      const uint16_t* q, int64_t q_stride, float scale, const float* lse, float* mass,
                                      int32_t first, bool add, cudaStream_t s) {
  (void)w;
  return launch_pdl(k_prefill_mass, dim3((unsigned)(b.n_seqs * L.n_kv), 256), dim3(kMassThreads), 0, s, 0, L, b,
                    (int32_t)causal, q, q_stride, scale * kLog2e, lse, mass, first, (int32_t)add);
}

}  // namespace mk
