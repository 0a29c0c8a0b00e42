// Host side of the paged cache (include/mosaickv.h): configuration and
// argument checks, the workspace layout, and the launches.  No device memory
// is allocated here, and no call throws: nothing in it allocates but the
// handle itself (nothrow).
#include <cmath>
#include <new>

#include "mk_paged.cuh"

struct mk_paged {
  mk_paged_config cfg;
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  char* ws;
  int64_t ws_clear;   // leading bytes of the workspace that must start at zero
  int64_t pool_layer, scale_layer;
  mk::PagedMaps dec;        // boxes of the decode kernel
  mk::PagedScratch scratch;
  uint32_t call;            // calls so far, kPagedClosed left out
  int device;
};

namespace {

constexpr int64_t kAlign = 256;
inline int64_t align_up(int64_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

mk_status check(const mk_paged_config* c) {
  if (!c || c->head_dim != MK_HEAD_DIM) return MK_EINVAL;
  if (c->n_kv_heads < 1 || c->n_q_heads < 1 || c->n_q_heads % c->n_kv_heads) return MK_EINVAL;
  const int G = c->n_q_heads / c->n_kv_heads;
  if (G != 1 && G != 2 && G != 4 && G != 8) return MK_EINVAL;
  if (c->n_kv_heads > 1024 || c->n_layers < 1 || c->n_pages < 1) return MK_EINVAL;
  if (c->max_seqs < 1 || c->max_seqs > MK_MAX_CALL_SEQS) return MK_EINVAL;
  if (c->page != 16 && c->page != 32 && c->page != 64) return MK_EINVAL;
  if (c->kv_type != MK_KV_BF16 && c->kv_type != MK_KV_E4M3) return MK_EINVAL;
  if ((int64_t)c->n_layers * c->n_pages > 0x7fffffff) return MK_EINVAL;  // a copy's coordinate
  return MK_OK;
}
inline int64_t elem(const mk_paged_config* c) { return c->kv_type == MK_KV_E4M3 ? 1 : 2; }
inline int64_t pool_layer_bytes(const mk_paged_config* c) {
  return (int64_t)c->n_pages * c->n_kv_heads * c->page * MK_HEAD_DIM * elem(c);
}
inline int64_t scale_layer_count(const mk_paged_config* c) {
  return c->kv_type == MK_KV_E4M3 ? (int64_t)c->n_pages * c->n_kv_heads : 0;
}
// Workspace: [error word][counters, zero between calls][split-token parts].
inline int64_t clear_bytes(const mk_paged_config* c) {
  return align_up(kAlign + ((int64_t)c->max_seqs * c->n_kv_heads + mk::kPagedMaxCtas) * 4);
}
// Rows of a unit of the decode kernel: at most 16 (several tokens a sequence).
inline int64_t part_acc_bytes(const mk_paged_config*) {
  return align_up((int64_t)2 * mk::kPagedMaxCtas * 16 * MK_HEAD_DIM * 4);
}
inline int64_t part_ml_bytes(const mk_paged_config*) {
  return align_up((int64_t)2 * mk::kPagedMaxCtas * 16 * 2 * 4);
}

inline int64_t prefill_part_bytes() { return align_up(mk::paged_prefill_part_floats() * 4); }

// Rows (query token, query head) of a kv head up to which several query tokens
// go to the decode kernel, which reads the pages at its rate, and not to row
// tiles of 256, which would be nearly empty: 16 sequences of 2K-16K with 4
// tokens (16 rows) 79 us against 141, e4m3, and 94 against 127, bf16; at 20
// rows it would take two readings, 142 us against 141.
constexpr int kFewRows = 16;

// The driver's tensor-map encoder, looked up through the runtime (the library
// links no driver stub).
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encoder() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess)
    return nullptr;
  return reinterpret_cast<EncodeFn>(fn);
}
bool pool_map(EncodeFn enc, const mk_paged_config* c, void* pool, int rows, CUtensorMap* m) {
  const int64_t es = elem(c), row = MK_HEAD_DIM * es;
  const cuuint64_t dim[3] = {MK_HEAD_DIM, (cuuint64_t)c->n_kv_heads * c->page, (cuuint64_t)c->n_layers * c->n_pages};
  const cuuint64_t stride[2] = {(cuuint64_t)row, (cuuint64_t)(row * c->n_kv_heads * c->page)};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / es), (cuuint32_t)rows, 1}, one[3] = {1, 1, 1};
  return enc(m, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, pool, dim, stride, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Makes the handle's device current for the call and restores the caller's.
struct DeviceGuard {
  int before = -1;
  bool ok = false, changed = false;
  explicit DeviceGuard(int want) {
    if (cudaGetDevice(&before) != cudaSuccess) return;
    if (before != want) {
      if (cudaSetDevice(want) != cudaSuccess) return;
      changed = true;
    }
    ok = true;
  }
  ~DeviceGuard() {
    if (changed) (void)cudaSetDevice(before);
  }
};

mk::PagedLayer layer_of(mk_paged* h, int layer) {
  mk::PagedLayer L{};
  L.k = h->k + layer * h->pool_layer;
  L.v = h->v + layer * h->pool_layer;
  L.k_scale = h->k_scale ? h->k_scale + layer * h->scale_layer : nullptr;
  L.v_scale = h->v_scale ? h->v_scale + layer * h->scale_layer : nullptr;
  L.err = reinterpret_cast<int32_t*>(h->ws);
  h->call = (h->call + 1) & 0x7fffffffu;
  L.call = h->call;
  L.n_pages = h->cfg.n_pages;
  L.n_kv = h->cfg.n_kv_heads;
  L.G = h->cfg.n_q_heads / h->cfg.n_kv_heads;
  L.P = h->cfg.page;
  L.p_log2 = L.P == 16 ? 4 : L.P == 32 ? 5 : 6;
  L.e4m3 = h->cfg.kv_type == MK_KV_E4M3;
  return L;
}

// An array of 4-byte words, or none.
bool words_ok(const void* p) { return ((uintptr_t)p & 3) == 0; }

// Arguments every call has.
mk_status check_call(const mk_paged* h, int32_t layer, const mk_paged_batch* b) {
  if (!h || !b) return MK_EINVAL;
  if (layer < 0 || layer >= h->cfg.n_layers) return MK_EINVAL;
  if (b->n_seqs < 0 || b->n_seqs > h->cfg.max_seqs || b->n_tokens < 0 || b->max_new < 1) return MK_EINVAL;
  if (b->n_seqs == 0 || b->n_tokens == 0) return MK_OK;  // nothing to do, nothing read
  if (!b->kv_len || !b->page_table || b->table_stride < 1) return MK_EINVAL;
  if (!words_ok(b->kv_len) || !words_ok(b->page_table) || !words_ok(b->cu_new)) return MK_EINVAL;
  if ((int64_t)b->table_stride * h->cfg.page > 0x7fffff00) return MK_EINVAL;  // token numbers and a step past them
  if (!b->cu_new && (b->max_new != 1 || b->n_tokens < b->n_seqs)) return MK_EINVAL;
  return MK_OK;
}
bool rows_ok(const void* p, int64_t stride, int64_t heads) {
  return p && ((uintptr_t)p & 15) == 0 && stride >= heads * MK_HEAD_DIM && stride % 8 == 0;
}

mk_status check_attn(const mk_paged* h, int32_t layer, const mk_paged_batch* b, const void* q, int64_t q_stride,
                     float scale, const void* out, int64_t out_stride, const float* lse) {
  mk_status st = check_call(h, layer, b);
  if (st != MK_OK) return st;
  if (!std::isfinite(scale)) return MK_EINVAL;
  if (b->n_seqs == 0 || b->n_tokens == 0) return MK_OK;
  if (!rows_ok(q, q_stride, h->cfg.n_q_heads) || !rows_ok(out, out_stride, h->cfg.n_q_heads)) return MK_EINVAL;
  if (!words_ok(lse)) return MK_EINVAL;
  return MK_OK;
}

}  // namespace

extern "C" {

mk_status mk_paged_sizes(const mk_paged_config* cfg, size_t* pool_bytes, size_t* scale_bytes, size_t* workspace_bytes) {
  mk_status st = check(cfg);
  if (st != MK_OK) return st;
  if (pool_bytes) *pool_bytes = (size_t)(pool_layer_bytes(cfg) * cfg->n_layers);
  if (scale_bytes) *scale_bytes = (size_t)(scale_layer_count(cfg) * cfg->n_layers * 4);
  if (workspace_bytes) *workspace_bytes = (size_t)(clear_bytes(cfg) + part_acc_bytes(cfg) + part_ml_bytes(cfg) + prefill_part_bytes());
  return MK_OK;
}

mk_status mk_paged_create(const mk_paged_config* cfg, void* k_pool, void* v_pool, float* k_scale, float* v_scale,
                          void* workspace, size_t workspace_bytes, mk_paged** out) {
  mk_status st = check(cfg);
  if (st != MK_OK) return st;
  if (!k_pool || !v_pool || !workspace || !out) return MK_EINVAL;
  if (((uintptr_t)k_pool | (uintptr_t)v_pool | (uintptr_t)workspace) % kAlign) return MK_EINVAL;
  const bool e4m3 = cfg->kv_type == MK_KV_E4M3;
  if (e4m3 != (k_scale != nullptr) || e4m3 != (v_scale != nullptr)) return MK_EINVAL;
  if (!words_ok(k_scale) || !words_ok(v_scale)) return MK_EINVAL;
  size_t need = 0;
  (void)mk_paged_sizes(cfg, nullptr, nullptr, &need);
  if (workspace_bytes < need) return MK_ENOMEM;
  mk_paged* h = new (std::nothrow) mk_paged();
  if (!h) return MK_ENOMEM;
  h->cfg = *cfg;
  h->k = static_cast<uint8_t*>(k_pool);
  h->v = static_cast<uint8_t*>(v_pool);
  h->k_scale = k_scale;
  h->v_scale = v_scale;
  h->ws = static_cast<char*>(workspace);
  h->ws_clear = clear_bytes(cfg);
  h->pool_layer = pool_layer_bytes(cfg);
  h->scale_layer = scale_layer_count(cfg);
  h->scratch.counters = reinterpret_cast<int32_t*>(h->ws + kAlign);
  h->scratch.prefill_counters = h->scratch.counters + (int64_t)cfg->max_seqs * cfg->n_kv_heads;
  h->scratch.part_acc = reinterpret_cast<float*>(h->ws + h->ws_clear);
  h->scratch.part_ml = reinterpret_cast<float*>(h->ws + h->ws_clear + part_acc_bytes(cfg));
  h->scratch.prefill_part = reinterpret_cast<float*>(h->ws + h->ws_clear + part_acc_bytes(cfg) + part_ml_bytes(cfg));
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) {
    const EncodeFn enc = encoder();
    const int rows = e4m3 && cfg->page >= 32 ? 32 : 16;
    if (!enc || !pool_map(enc, cfg, k_pool, rows, &h->dec.k) || !pool_map(enc, cfg, v_pool, rows, &h->dec.v))
      e = cudaErrorInvalidValue;
  }
  // Whatever is queued may still write this memory: its last user's work ends first.
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemset(workspace, 0, (size_t)h->ws_clear);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    delete h;
    return MK_ECUDA;
  }
  *out = h;
  return MK_OK;
}

mk_status mk_paged_destroy(mk_paged* h) {
  delete h;
  return MK_OK;
}

mk_status mk_paged_append(mk_paged* h, int32_t layer, const mk_paged_batch* batch, const mk_rope* rope, const void* k,
                          int64_t k_stride, const void* v, int64_t v_stride, const void* q, int64_t q_stride,
                          void* q_out, int64_t q_out_stride, mk_stream stream) {
  mk_status st = check_call(h, layer, batch);
  if (st != MK_OK) return st;
  mk_rope r{};
  if (rope) r = *rope;
  if (r.rot_dim < 0 || r.rot_dim > MK_HEAD_DIM || r.rot_dim % 16) return MK_EINVAL;
  if (r.rot_dim && (!r.cos_sin || ((uintptr_t)r.cos_sin & 15) || r.n_pos < 1 || !words_ok(r.positions)))
    return MK_EINVAL;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return MK_OK;
  if (!rows_ok(k, k_stride, h->cfg.n_kv_heads) || !rows_ok(v, v_stride, h->cfg.n_kv_heads)) return MK_EINVAL;
  if ((q == nullptr) != (q_out == nullptr)) return MK_EINVAL;
  if (q && (!rows_ok(q, q_stride, h->cfg.n_q_heads) || !rows_ok(q_out, q_out_stride, h->cfg.n_q_heads)))
    return MK_EINVAL;
  DeviceGuard dev(h->device);
  if (!dev.ok) return MK_ECUDA;
  const cudaError_t e = mk::launch_paged_append(
      layer_of(h, layer), *batch, r, static_cast<const uint16_t*>(k), k_stride, static_cast<const uint16_t*>(v), v_stride,
      static_cast<const uint16_t*>(q), q_stride, static_cast<uint16_t*>(q_out), q_out_stride, (cudaStream_t)stream);
  return e == cudaSuccess ? MK_OK : MK_ECUDA;
}

mk_status mk_paged_decode_attn(mk_paged* h, int32_t layer, const mk_paged_batch* batch, const void* q, int64_t q_stride,
                               float scale, void* out, int64_t out_stride, float* lse, mk_stream stream) {
  mk_status st = check_attn(h, layer, batch, q, q_stride, scale, out, out_stride, lse);
  if (st != MK_OK) return st;
  if (batch->max_new != 1) return MK_EINVAL;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return MK_OK;
  DeviceGuard dev(h->device);
  if (!dev.ok) return MK_ECUDA;
  const cudaError_t e =
      mk::launch_paged_decode(layer_of(h, layer), h->dec, h->scratch, layer, *batch, false, false,
                              static_cast<const uint16_t*>(q), q_stride, scale, static_cast<uint16_t*>(out), out_stride,
                              lse, (cudaStream_t)stream);
  return e == cudaSuccess ? MK_OK : MK_ECUDA;
}

mk_status mk_paged_prefill_attn(mk_paged* h, int32_t layer, const mk_paged_batch* batch, int32_t causal, const void* q,
                                int64_t q_stride, float scale, void* out, int64_t out_stride, float* lse,
                                mk_stream stream) {
  mk_status st = check_attn(h, layer, batch, q, q_stride, scale, out, out_stride, lse);
  if (st != MK_OK) return st;
  if (causal != 0 && causal != 1) return MK_EINVAL;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return MK_OK;
  DeviceGuard dev(h->device);
  if (!dev.ok) return MK_ECUDA;
  const uint16_t* qq = static_cast<const uint16_t*>(q);
  uint16_t* oo = static_cast<uint16_t*>(out);
  const bool few = (int64_t)batch->max_new * (h->cfg.n_q_heads / h->cfg.n_kv_heads) <= kFewRows;
  const cudaError_t e = few ? mk::launch_paged_decode(layer_of(h, layer), h->dec, h->scratch, layer, *batch, true,
                                                      causal != 0, qq, q_stride, scale, oo, out_stride, lse,
                                                      (cudaStream_t)stream)
                            : mk::launch_paged_prefill(layer_of(h, layer), h->scratch, *batch, causal != 0, qq, q_stride,
                                                       scale, oo, out_stride, lse, (cudaStream_t)stream);
  return e == cudaSuccess ? MK_OK : MK_ECUDA;
}

mk_status mk_paged_poll_error(mk_paged* h, int32_t* detail) {
  if (!h) return MK_EINVAL;
  DeviceGuard dev(h->device);
  int32_t w[4] = {0, 0, 0, 0};  // status, call, detail, sequence
  cudaError_t e = dev.ok ? cudaDeviceSynchronize() : cudaErrorInvalidDevice;
  if (e == cudaSuccess) e = cudaMemcpy(w, h->ws, sizeof(w), cudaMemcpyDeviceToHost);
  // Closed, as paged_stopped does it: a replay of the call does no work either.
  if (e == cudaSuccess && w[0] != 0) {
    e = cudaMemset(h->ws + 4, 0xff, 4);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
  }
  if (e != cudaSuccess) return MK_ECUDA;
  if (detail) *detail = w[2];
  return w[0] == 0 ? MK_OK : (mk_status)w[0];
}

mk_status mk_paged_clear_error(mk_paged* h) {
  if (!h) return MK_EINVAL;
  DeviceGuard dev(h->device);
  cudaError_t e = dev.ok ? cudaDeviceSynchronize() : cudaErrorInvalidDevice;
  if (e == cudaSuccess) e = cudaMemset(h->ws, 0, (size_t)h->ws_clear);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  return e == cudaSuccess ? MK_OK : MK_ECUDA;
}

}  // extern "C"
