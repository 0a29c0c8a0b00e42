// Host side of the paged cache (include/mosaickv.h): configuration and
// argument checks, the workspace layout, and the launches.  No device memory
// is allocated here, and no call throws: nothing in it allocates but the
// handle itself (nothrow).
#include <algorithm>
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
  mk::PagedEvictScratch evict;
  uint32_t call;            // calls so far, kPagedClosed left out
  int device;
};

namespace mk {

TensorMapEncoder tensor_map_encoder() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess)
    return nullptr;
  return reinterpret_cast<TensorMapEncoder>(fn);
}

}  // namespace mk

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
// Attention mass: one word per slot of a layer's pool; the logits of a decode
// step: one per slot and query head of its kv head.
inline int64_t mass_layer_count(const mk_paged_config* c) { return (int64_t)c->n_pages * c->n_kv_heads * c->page; }
inline int64_t logits_bytes(const mk_paged_config* c) { return (int64_t)c->n_pages * c->n_q_heads * c->page * 4; }
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

inline int64_t shared_bytes() { return align_up(sizeof(mk::PagedShared)); }
inline int64_t row_part_bytes(const mk_paged_config* c) {
  return align_up((int64_t)c->max_seqs * c->n_q_heads * mk::kPagedRowPart * 4);
}
inline int64_t own_bytes(const mk_paged_config* c) { return align_up((int64_t)c->max_seqs * c->n_kv_heads * 8); }
inline int64_t lse2_bytes(const mk_paged_config* c) { return align_up((int64_t)c->max_seqs * c->n_q_heads * 4); }
// Eviction: the counter (a line of its own) and the plan, then two words per page and head.
inline int64_t plan_bytes(const mk_paged_config* c) { return align_up(kAlign + (int64_t)c->max_seqs * 8); }
inline int64_t group_words_bytes(const mk_paged_config* c) { return align_up((int64_t)c->n_pages * c->n_kv_heads * 4); }
// Shared prefixes, a step's mass and eviction take the same bytes: a handle's
// calls are ordered, and nothing of one is left for the next.
inline int64_t turns_bytes(const mk_paged_config* c) {
  return std::max(std::max(shared_bytes() + 2 * row_part_bytes(c) + own_bytes(c), lse2_bytes(c)), plan_bytes(c) + 2 * group_words_bytes(c));
}
inline int64_t prefill_part_bytes() { return align_up(mk::paged_prefill_part_floats() * 4); }

// Rows (query token, query head) of a kv head up to which several query tokens
// go to the decode kernel, which reads the pages at its rate, and not to row
// tiles of 256, which would be nearly empty: 16 sequences of 2K-16K with 4
// tokens (16 rows) 79 us against 141, e4m3, and 94 against 127, bf16; at 20
// rows it would take two readings, 142 us against 141.
constexpr int kFewRows = 16;

bool pool_map(mk::TensorMapEncoder enc, const mk_paged_config* c, void* pool, int rows, CUtensorMap* m) {
  const int64_t es = elem(c), row = MK_HEAD_DIM * es;
  const cuuint64_t dim[3] = {MK_HEAD_DIM, (cuuint64_t)c->n_kv_heads * c->page, (cuuint64_t)c->n_layers * c->n_pages};
  const cuuint64_t stride[2] = {(cuuint64_t)row, (cuuint64_t)(row * c->n_kv_heads * c->page)};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / es), (cuuint32_t)rows, 1}, one[3] = {1, 1, 1};
  return enc(m, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, pool, dim, stride, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Bytes of keys and values of a decode step up to which its sequences read what
// they share each by themselves (the groups are checked all the same): one
// kernel fewer to wait for, and no parts to join.  32 query heads over 8, us a
// call of many in a row (and with cold caches), sharing against not with the
// check (2 to 4 us): 24 sequences on 2K 35.9 (49.8) and 33.7 (41.6), 111 MiB; 16
// on 4K 41.1 (57) and 36.3 (43.7), 138 MiB; 32 on 2K 36.7 (50) and 39.7 (46), 148
// MiB; 64 on 1K 38.0 (52) and 46.3 (54), 168 MiB; in bf16 8 on 4K 32.9 (44) and
// 26.5 (35.5), 138 MiB, 32 on 1K 29 (38) and 29 (38), 168 MiB.
constexpr int64_t kSmallShared = 144 << 20;

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
  if (workspace_bytes)
    *workspace_bytes =
        (size_t)(clear_bytes(cfg) + part_acc_bytes(cfg) + part_ml_bytes(cfg) + prefill_part_bytes() + turns_bytes(cfg));
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
  char* at = h->ws + h->ws_clear;
  auto take = [&](int64_t bytes) {
    char* p = at;
    at += bytes;
    return p;
  };
  h->scratch.part_acc = reinterpret_cast<float*>(take(part_acc_bytes(cfg)));
  h->scratch.part_ml = reinterpret_cast<float*>(take(part_ml_bytes(cfg)));
  h->scratch.prefill_part = reinterpret_cast<float*>(take(prefill_part_bytes()));
  h->scratch.mass_part = h->scratch.prefill_part;  // calls of a handle are ordered
  char* const turns = at;
  h->scratch.shared = reinterpret_cast<mk::PagedShared*>(take(shared_bytes()));
  h->scratch.row_part = reinterpret_cast<float*>(take(row_part_bytes(cfg)));
  h->scratch.own_row = reinterpret_cast<float*>(take(row_part_bytes(cfg)));
  h->scratch.own = reinterpret_cast<int32_t*>(take(own_bytes(cfg)));
  h->scratch.lse2 = reinterpret_cast<float*>(turns);
  at = turns;
  char* plan = take(plan_bytes(cfg));
  h->evict.ticket = reinterpret_cast<int32_t*>(plan);
  h->evict.plan = reinterpret_cast<int32_t*>(plan + kAlign);
  h->evict.rank0 = reinterpret_cast<int32_t*>(take(group_words_bytes(cfg)));
  h->evict.flag = reinterpret_cast<int32_t*>(take(group_words_bytes(cfg)));
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) {
    const mk::TensorMapEncoder enc = mk::tensor_map_encoder();
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

mk_status mk_paged_prefix_attn(mk_paged* h, int32_t layer, const mk_paged_batch* batch, const mk_paged_prefix* prefix,
                               const void* q, int64_t q_stride, float scale, void* out, int64_t out_stride, float* lse,
                               mk_stream stream) {
  mk_status st = check_attn(h, layer, batch, q, q_stride, scale, out, out_stride, lse);
  if (st != MK_OK) return st;
  if (batch->max_new != 1 || !prefix || prefix->n_groups < 0 || prefix->n_groups > batch->n_seqs) return MK_EINVAL;
  if (prefix->n_groups && (!prefix->cu_group || !prefix->prefix_len)) return MK_EINVAL;
  if (!words_ok(prefix->cu_group) || !words_ok(prefix->prefix_len)) return MK_EINVAL;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return MK_OK;
  DeviceGuard dev(h->device);
  if (!dev.ok) return MK_ECUDA;
  const mk::PagedLayer L = layer_of(h, layer);
  const uint16_t* qq = static_cast<const uint16_t*>(q);
  uint16_t* oo = static_cast<uint16_t*>(out);
  // What the batch could read at most, everything for every sequence.
  const int64_t most = (int64_t)batch->n_seqs * batch->table_stride * h->cfg.page * h->cfg.n_kv_heads * 2 * MK_HEAD_DIM * elem(&h->cfg);
  const bool small = most <= kSmallShared;
  cudaError_t e = cudaSuccess;
  if (prefix->n_groups > 0)
    e = mk::launch_paged_prefix(L, h->dec, h->scratch, layer, *batch, *prefix, qq, q_stride, scale, small, (cudaStream_t)stream);
  if (e == cudaSuccess && (small || prefix->n_groups == 0)) {
    e = mk::launch_paged_decode(L, h->dec, h->scratch, layer, *batch, false, false, qq, q_stride, scale, oo, out_stride, lse,
                                (cudaStream_t)stream);
  } else {
    if (e == cudaSuccess)
      e = mk::launch_paged_decode_own(L, h->dec, h->scratch, layer, *batch, qq, q_stride, scale, (cudaStream_t)stream);
    if (e == cudaSuccess)
      e = mk::launch_paged_join(L, h->scratch, *batch, oo, out_stride, lse, (cudaStream_t)stream);
  }
  return e == cudaSuccess ? MK_OK : MK_ECUDA;
}

mk_status mk_paged_mass_sizes(const mk_paged_config* cfg, size_t* mass_bytes, size_t* scratch_bytes) {
  mk_status st = check(cfg);
  if (st != MK_OK) return st;
  if (mass_bytes) *mass_bytes = (size_t)(mass_layer_count(cfg) * cfg->n_layers * 4);
  if (scratch_bytes) *scratch_bytes = (size_t)logits_bytes(cfg);
  return MK_OK;
}

mk_status mk_paged_decode_attn_mass(mk_paged* h, int32_t layer, const mk_paged_batch* batch, const void* q,
                                    int64_t q_stride, float scale, void* out, int64_t out_stride, float* lse,
                                    float* mass, int32_t first, void* scratch, size_t scratch_bytes, mk_stream stream) {
  mk_status st = check_attn(h, layer, batch, q, q_stride, scale, out, out_stride, lse);
  if (st != MK_OK) return st;
  if (batch->max_new != 1 || !mass || !words_ok(mass) || first < 0) return MK_EINVAL;
  if (!scratch || ((uintptr_t)scratch & 15)) return MK_EINVAL;
  if (scratch_bytes < (size_t)logits_bytes(&h->cfg)) return MK_ENOMEM;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return MK_OK;
  DeviceGuard dev(h->device);
  if (!dev.ok) return MK_ECUDA;
  const mk::PagedLayer L = layer_of(h, layer);
  float* logits = static_cast<float*>(scratch);
  cudaError_t e = mk::launch_paged_decode_mass(L, h->dec, h->scratch, layer, *batch, static_cast<const uint16_t*>(q),
                                               q_stride, scale, static_cast<uint16_t*>(out), out_stride, lse, logits,
                                               (cudaStream_t)stream);
  if (e == cudaSuccess)
    e = mk::launch_paged_mass_fold(L, h->scratch, *batch, logits, mass + layer * mass_layer_count(&h->cfg), first,
                                   (cudaStream_t)stream);
  return e == cudaSuccess ? MK_OK : MK_ECUDA;
}

mk_status mk_paged_prefill_mass(mk_paged* h, int32_t layer, const mk_paged_batch* batch, int32_t causal, const void* q,
                                int64_t q_stride, float scale, const float* lse, float* mass, int32_t first,
                                int32_t add, mk_stream stream) {
  mk_status st = check_call(h, layer, batch);
  if (st != MK_OK) return st;
  if (!std::isfinite(scale) || (causal != 0 && causal != 1) || (add != 0 && add != 1) || first < 0) return MK_EINVAL;
  if (!mass || !words_ok(mass)) return MK_EINVAL;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return MK_OK;
  if (!rows_ok(q, q_stride, h->cfg.n_q_heads) || !lse || !words_ok(lse)) return MK_EINVAL;
  DeviceGuard dev(h->device);
  if (!dev.ok) return MK_ECUDA;
  const cudaError_t e = mk::launch_paged_prefill_mass(
      layer_of(h, layer), h->dec, h->scratch, layer, *batch, causal != 0, static_cast<const uint16_t*>(q), q_stride, scale, lse,
      mass + layer * mass_layer_count(&h->cfg), first, add != 0, (cudaStream_t)stream);
  return e == cudaSuccess ? MK_OK : MK_ECUDA;
}

mk_status mk_paged_evict(mk_paged* h, int32_t layer, const mk_paged_batch* batch, float* mass, const int32_t* keep,
                         int32_t first, int32_t recent, int32_t* kept, int32_t kept_stride, int32_t* new_len,
                         mk_stream stream) {
  if (!h || !batch) return MK_EINVAL;
  if (layer < 0 || layer >= h->cfg.n_layers || batch->n_seqs < 0 || batch->n_seqs > h->cfg.max_seqs) return MK_EINVAL;
  if (first < 0 || recent < 0 || kept_stride < 0) return MK_EINVAL;
  if (batch->n_seqs == 0) return MK_OK;
  if (!batch->kv_len || !batch->page_table || batch->table_stride < 1) return MK_EINVAL;
  if ((int64_t)batch->table_stride * h->cfg.page > 0x7fffff00) return MK_EINVAL;
  if (!mass || !keep || !new_len || (kept_stride > 0 && !kept)) return MK_EINVAL;
  if (!words_ok(batch->kv_len) || !words_ok(batch->page_table) || !words_ok(mass) || !words_ok(keep) ||
      !words_ok(kept) || !words_ok(new_len) || new_len == batch->kv_len)
    return MK_EINVAL;
  DeviceGuard dev(h->device);
  if (!dev.ok) return MK_ECUDA;
  const cudaError_t e =
      mk::launch_paged_evict(layer_of(h, layer), h->evict, *batch, mass + layer * mass_layer_count(&h->cfg), keep, first,
                             recent, kept, kept_stride, new_len, (cudaStream_t)stream);
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
