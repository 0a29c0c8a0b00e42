// Attention over the paged cache, the plain way: one warp per (query row,
// query head) walks its keys one at a time with a running maximum and sum.
#include "mk_paged.cuh"

namespace mk {

namespace {

struct SimpleArgs {
  mk_paged_batch b;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t q_stride, out_stride;
  float scale;
  int32_t causal;
};

template <bool E4M3>
__global__ void __launch_bounds__(128) k_paged_attn_simple(PagedLayer L, SimpleArgs a) {
  const int lane = threadIdx.x & 31;
  const int n_q = L.n_kv * L.G;
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  if (paged_has_error(L) || r >= (int64_t)a.b.n_tokens * n_q) return;
  const int t = (int)(r / n_q), h = (int)(r % n_q), kvh = h / L.G;
  int seq = -1;
  PagedSeq s{};
  for (int i = 0; i < a.b.n_seqs; ++i) {
    const PagedSeq x = paged_seq(a.b, L.P, i, false);
    if (!x.ok) {
      paged_error(L, ERR_PAGED_BATCH, i, x.len);
      return;
    }
    if (t >= x.row0 && t < x.row0 + x.n_new) {
      seq = i;
      s = x;
    }
  }
  if (seq < 0) return;
  const int sees = min(s.len, a.causal ? s.len - s.n_new + (t - s.row0) + 1 : s.len);
  float q[4], o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0.0f, rest = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) q[e] = bf2f(a.q[(int64_t)t * a.q_stride + h * D + lane * 4 + e]) * a.scale;
  for (int p = 0; p < sees; ++p) {
    const int page = a.b.page_table[(int64_t)seq * a.b.table_stride + (p >> L.p_log2)];
    if (page < 0 || page >= L.n_pages) {
      paged_error(L, ERR_PAGED_PAGE, seq, page);
      return;
    }
    const int64_t unit = (int64_t)page * L.n_kv + kvh;
    const int64_t at = (unit * L.P + (p & (L.P - 1))) * D + lane * 4;
    float k[4], v[4];
    if (E4M3) {
      const float ks = L.k_scale[unit], vs = L.v_scale[unit];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        k[e] = ks * __half2float(__half(__nv_cvt_fp8_to_halfraw(L.k[at + e], __NV_E4M3)));
        v[e] = vs * __half2float(__half(__nv_cvt_fp8_to_halfraw(L.v[at + e], __NV_E4M3)));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        k[e] = bf2f(reinterpret_cast<const uint16_t*>(L.k)[at + e]);
        v[e] = bf2f(reinterpret_cast<const uint16_t*>(L.v)[at + e]);
      }
    }
    const float z = warp_sum(q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3]);
    const float mn = fmaxf(m, z), c = __expf(m - mn), w = __expf(z - mn);
    const float add = __fsub_rn(w, rest * c), sum = __fadd_rn(l * c, add);  // compensated: the keys are added one by one
    rest = __fsub_rn(__fsub_rn(sum, l * c), add);
    l = sum;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = o[e] * c + w * v[e];
    m = mn;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    a.out[(int64_t)t * a.out_stride + h * D + lane * 4 + e] =
        __bfloat16_as_ushort(__float2bfloat16_rn(sees > 0 ? o[e] / l : 0.0f));
  if (a.lse && lane == 0) a.lse[(int64_t)t * n_q + h] = sees > 0 ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_paged_attn_simple(const PagedLayer& L, const mk_paged_batch& b, bool causal, const uint16_t* q,
                                     int64_t q_stride, float scale, uint16_t* out, int64_t out_stride, float* lse,
                                     cudaStream_t s) {
  SimpleArgs a{b, q, out, lse, q_stride, out_stride, scale, causal ? 1 : 0};
  const int64_t rows = (int64_t)b.n_tokens * L.n_kv * L.G;
  const dim3 grid((unsigned)((rows + 3) / 4)), block(128);
  return L.e4m3 ? launch_pdl(k_paged_attn_simple<true>, grid, block, 0, s, 0, L, a)
                : launch_pdl(k_paged_attn_simple<false>, grid, block, 0, s, 0, L, a);
}

}  // namespace mk
