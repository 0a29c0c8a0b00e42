// Appending keys and values to the paged cache, rotated on the way.
//
// Mathematics.  A token at position p of its sequence has its key's (and
// query's) first R channels turned in R / 2 planes by the angles of p:
// (x1, x2) -> (x1 c - x2 s, x2 c + x1 s), products and sum rounded in fp32.
// A bf16 pool stores the result rounded once.  An e4m3 pool holds code =
// rn(y / s) under one scale s per (page, kv head), the smallest power of two
// with amax <= 448 s over the page's tokens (at least 2^-64).  A power of two
// costs an e4m3 code no precision, only up to one binade of its 18, and makes
// raising a page's scale exact: the codes held before are multiplied by
// s_old / s_new, which rounds only those that become subnormal.
//
// Work split: a page of one kv head of one tensor per CTA, 16 threads a row (8
// channels each), so that the page's maximum is a reduction inside the CTA and
// a row's rotation partner is in the same 16 lanes.  The values stay in
// registers between the maximum and the rounding: one pass.  A thread has at
// most four rows of a page (pages of 64 tokens take 256 threads), which keeps
// enough CTAs on an SM for the loads in flight that HBM wants.  Queries: 16
// threads a (token, few heads), the angles loaded once for all of its heads
// (they are four times a head's data).
//
// What bounds it: HBM for prompts, the launch and three dependent loads (batch,
// page id, row) for single tokens.  32K tokens with 32 query heads into e4m3
// pages of 64: 162 us, 4.7 TB/s of the 755 MB it has to move (69% of the copy
// rate; 128 threads and eight rows a thread: 408 us, with four CTAs an SM); 64
// single tokens 6.7 us a call (4.1 in a graph of calls).
#include "mk_paged.cuh"

namespace mk {

namespace {

template <int P>
struct Shape {
  static constexpr int threads = P == 64 ? 256 : 128;
};

struct AppendArgs {
  mk_paged_batch b;
  mk_rope rope;
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  int64_t k_stride, v_stride, q_stride, q_out_stride;
  int32_t n_units;  // page slots x kv heads x 2
  int32_t q_heads;  // query heads of a (token, heads) item
};

// The angles that chunk j (8 channels) of a row at position `pos` needs.
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void load_angles(const mk_rope& r, int pos, int j, Angles& g) {
  const int half = r.rot_dim >> 1, c0 = j * 8;
  if (c0 >= r.rot_dim) return;
  const float* row = r.cos_sin + (int64_t)pos * r.rot_dim;
  if (r.interleaved) {
    *reinterpret_cast<float4*>(g.c) = *reinterpret_cast<const float4*>(row + c0 / 2);
    *reinterpret_cast<float4*>(g.s) = *reinterpret_cast<const float4*>(row + half + c0 / 2);
    return;
  }
  const int i = c0 >= half ? c0 - half : c0;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    *reinterpret_cast<float4*>(g.c + 4 * v) = *reinterpret_cast<const float4*>(row + i + 4 * v);
    *reinterpret_cast<float4*>(g.s + 4 * v) = *reinterpret_cast<const float4*>(row + half + i + 4 * v);
  }
}
// Eight channels (16-lane group: chunk j of the row) turned by the row's
// angles; every lane of the group must call.
__device__ __forceinline__ void rotate8(const mk_rope& r, const Angles& g, int j, int lane, const uint4 raw, float (&y)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[2 * e] = __uint_as_float(w[e] << 16);
    y[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
  if (r.rot_dim == 0) return;
  const int half = r.rot_dim >> 1, c0 = j * 8;
  if (r.interleaved) {
    if (c0 < r.rot_dim) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = y[2 * e], b = y[2 * e + 1];
        y[2 * e] = __fsub_rn(__fmul_rn(a, g.c[e]), __fmul_rn(b, g.s[e]));
        y[2 * e + 1] = __fadd_rn(__fmul_rn(b, g.c[e]), __fmul_rn(a, g.s[e]));
      }
    }
    return;
  }
  // Half split: the partner chunk is half / 8 lanes away in the same group.
  const bool second = c0 >= half;
  const int partner = (lane & 16) | ((second ? j - half / 8 : j + half / 8) & 15);
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = __shfl_sync(FULL, w[e], partner);
  if (c0 < r.rot_dim) {
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const float other = (n & 1) ? __uint_as_float(o[n >> 1] & 0xffff0000u) : __uint_as_float(o[n >> 1] << 16);
      const float p = __fmul_rn(y[n], g.c[n]), t = __fmul_rn(other, g.s[n]);
      y[n] = second ? __fadd_rn(p, t) : __fsub_rn(p, t);
    }
  }
}

__device__ __forceinline__ uint4 pack_bf16(const float (&y)[8]) {
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    o[e] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(y[2 * e])) |
           ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(y[2 * e + 1])) << 16);
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void unpack_e4m3(uint2 c, float (&y)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = e < 2 ? c.x : c.y;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (e & 1))), __NV_E4M3);
    y[2 * e] = __half2float(__half(__half_raw{h.x}));
    y[2 * e + 1] = __half2float(__half(__half_raw{h.y}));
  }
}
__device__ __forceinline__ int clamp_position(const PagedLayer& L, const mk_rope& r, int pos, int seq) {
  if (r.rot_dim && (pos < 0 || pos >= r.n_pos)) {
    paged_error(L, ERR_PAGED_POSITION, seq, pos);
    return 0;
  }
  return pos;
}

template <int P, bool E4M3>
__global__ void __launch_bounds__(Shape<P>::threads) k_paged_append(PagedLayer L, AppendArgs a) {
  constexpr int kThreads = Shape<P>::threads;
  __shared__ int s_wsum[kThreads / 32], s_seq, s_idx;
  __shared__ float s_max[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, j = tid & 15, rr = tid >> 4;
  // No early trigger, since q_out may be the query of mk_block_select, whose
  // prologue reads it before its own wait: behind a kernel that triggers early
  // it could start before this one's stores.  Without a trigger it starts when
  // this one's CTAs have ended, as behind any other producer of a query; that
  // their stores are seen before the wait is what the older kernels rest on,
  // not something that the launch order promises.
  pdl_wait();
  if (__syncthreads_or(tid == 0 && paged_stopped(L))) return;  // one thread's reading for the CTA

  if ((int)blockIdx.x >= a.n_units) {  // a query CTA: 16 threads a (token, q_heads heads)
    const int n_q = L.n_kv * L.G, groups = (n_q + a.q_heads - 1) / a.q_heads;
    const int64_t at = (int64_t)((int)blockIdx.x - a.n_units) * (kThreads / 16) + rr;
    const int t = (int)(at / groups), h0 = (int)(at - (int64_t)t * groups) * a.q_heads;
    int lo = 0, pos = 0;
    bool in = t < a.b.n_tokens;
    if (in) {
      if (a.b.cu_new) {
        int hi = a.b.n_seqs - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (a.b.cu_new[mid] <= t) lo = mid; else hi = mid - 1;
        }
      } else {
        lo = min(t, a.b.n_seqs - 1);
      }
      const PagedSeq s = paged_seq(a.b, P, lo, true);
      in = s.ok && t >= s.row0 && t < s.row0 + s.n_new;  // rows behind the last sequence stay as they were
      if (in) pos = clamp_position(L, a.rope, a.rope.positions ? a.rope.positions[t] : s.len - s.n_new + (t - s.row0), lo);
    }
    Angles g;
    if (in) load_angles(a.rope, pos, j, g);
    const uint16_t* from = a.q + (int64_t)t * a.q_stride + h0 * D + j * 8;
    uint16_t* to = a.q_out + (int64_t)t * a.q_out_stride + h0 * D + j * 8;
    for (int i0 = 0; i0 < a.q_heads; i0 += 4) {
      uint4 raw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        raw[i] = make_uint4(0, 0, 0, 0);
        if (in && i0 + i < a.q_heads && h0 + i0 + i < n_q) raw[i] = *reinterpret_cast<const uint4*>(from + (i0 + i) * D);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float y[8];
        rotate8(a.rope, g, j, lane, raw[i], y);
        if (in && i0 + i < a.q_heads && h0 + i0 + i < n_q) *reinterpret_cast<uint4*>(to + (i0 + i) * D) = pack_bf16(y);
      }
    }
    return;
  }

  const int is_v = (int)blockIdx.x & 1;
  const int head = ((int)blockIdx.x >> 1) % L.n_kv;
  const int slot = ((int)blockIdx.x >> 1) / L.n_kv;
  int seq, idx;  // the sequence and which of its touched pages
  if (a.b.max_new == 1) {
    seq = slot;
    idx = 0;
  } else {  // the slot-th touched page over all sequences
    if (tid == 0) s_seq = -1;
    int base = 0;
    for (int i0 = 0; i0 < a.b.n_seqs; i0 += kThreads) {
      const int i = i0 + tid;
      int cnt = 0;
      if (i < a.b.n_seqs) {
        const PagedSeq s = paged_seq(a.b, P, i, true);
        if (!s.ok) paged_error(L, ERR_PAGED_BATCH, i, s.len);
        if (s.ok && s.n_new > 0) cnt = (s.len - 1) / P - (s.len - s.n_new) / P + 1;
      }
      const int ex = warp_excl_scan(cnt, lane);
      if (lane == 31) s_wsum[warp] = ex + cnt;
      __syncthreads();
      int off = base;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) off += s_wsum[w];
        base += s_wsum[w];
      }
      if (slot >= off + ex && slot < off + ex + cnt) {
        s_seq = i;
        s_idx = slot - off - ex;
      }
      __syncthreads();
      if (base > slot) break;
    }
    seq = s_seq;
    idx = s_idx;
    if (seq < 0) return;
  }
  const PagedSeq sq = paged_seq(a.b, P, seq, true);
  if (!sq.ok) {
    if (tid == 0) paged_error(L, ERR_PAGED_BATCH, seq, sq.len);
    return;
  }
  if (sq.n_new == 0) return;
  const int start = sq.len - sq.n_new;
  const int pg = start / P + idx;
  const int s0 = max(start - pg * P, 0), s1 = min(sq.len - pg * P, P);  // new tokens' slots of this page
  const int page = a.b.page_table[(int64_t)seq * a.b.table_stride + pg];
  if (page < 0 || page >= L.n_pages) {
    if (tid == 0) paged_error(L, ERR_PAGED_PAGE, seq, page);
    return;
  }
  const int64_t unit = (int64_t)page * L.n_kv + head;
  const uint16_t* src = is_v ? a.v : a.k;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  mk_rope rope = a.rope;
  if (is_v) rope.rot_dim = 0;
  constexpr int NP = P / (kThreads / 16);  // rows of a thread
  float y[NP][8];
  float amax = 0.0f;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int sl = p * (kThreads / 16) + rr;
    const bool in = sl >= s0 && sl < s1;
    const int64_t t = sq.row0 + (int64_t)pg * P + sl - start;
    int pos = 0;
    if (in && !is_v) pos = clamp_position(L, rope, rope.positions ? rope.positions[t] : pg * P + sl, seq);
    const uint4 raw = in ? *reinterpret_cast<const uint4*>(src + t * stride + head * D + j * 8) : make_uint4(0, 0, 0, 0);
    Angles g;
    if (in && !is_v) load_angles(rope, pos, j, g);
    rotate8(rope, g, j, lane, raw, y[p]);
    if (E4M3) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float m = fabsf(y[p][e]);
        if (m <= 3.402823466e38f) amax = fmaxf(amax, m);  // infinities and NaN do not set the scale
      }
    } else if (in) {
      *reinterpret_cast<uint4*>((is_v ? L.v : L.k) + ((unit * P + sl) * D + j * 8) * 2) = pack_bf16(y[p]);
    }
  }
  if (!E4M3) return;
  amax = warp_max(amax);
  if (lane == 0) s_max[warp] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
  float scale = scale_of(amax);
  uint8_t* dst = (is_v ? L.v : L.k) + unit * P * D;
  float* sc = (is_v ? L.v_scale : L.k_scale) + unit;
  if (s0 > 0) {  // tokens of earlier calls in this page
    const float was = *sc;
    scale = fmaxf(scale, was);
    if (scale > was) {
      const float ratio = __fdiv_rn(was, scale);
      for (int sl = rr; sl < s0; sl += kThreads / 16) {
        uint2* c = reinterpret_cast<uint2*>(dst + sl * D + j * 8);
        float h[8];
        unpack_e4m3(*c, h);
        *c = pack_e4m3(h, ratio);
      }
    }
  }
  const float inv = __frcp_rn(scale);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int sl = p * (kThreads / 16) + rr;
    if (sl >= s0 && sl < s1) *reinterpret_cast<uint2*>(dst + sl * D + j * 8) = pack_e4m3(y[p], inv);
  }
  __syncthreads();  // every thread has read the page's earlier scale
  if (tid == 0) *sc = scale;
}

}  // namespace

cudaError_t launch_paged_append(const PagedLayer& L, const mk_paged_batch& b, const mk_rope& rope, const uint16_t* k,
                                int64_t k_stride, const uint16_t* v, int64_t v_stride, const uint16_t* q,
                                int64_t q_stride, uint16_t* q_out, int64_t q_out_stride, cudaStream_t s) {
  // Touched pages: at most 2 + (n - 2) / P of a sequence with n >= 2 new
  // tokens, 1 of one with a single one.
  int64_t slots = b.max_new == 1 ? b.n_seqs : (int64_t)b.n_tokens / L.P + 2 * (int64_t)b.n_seqs;
  if (slots > b.n_tokens && b.max_new != 1) slots = b.n_tokens;
  const int64_t units = slots * L.n_kv * 2;
  // Heads of a query item: few rows want many items (latency), many rows want
  // the angles' loads spread over more heads: 64 tokens x 32 heads 1 head,
  // thousands of tokens 8.
  const int64_t rows = (int64_t)b.n_tokens * L.n_kv * L.G;
  const int q_heads = rows >= 32768 ? 8 : rows >= 8192 ? 4 : 1;
  const int threads = L.P == 64 ? Shape<64>::threads : Shape<16>::threads;
  const int64_t items = (int64_t)b.n_tokens * ((L.n_kv * L.G + q_heads - 1) / q_heads);
  const int64_t qb = q ? (items + threads / 16 - 1) / (threads / 16) : 0;
  if (units + qb == 0) return cudaSuccess;
  if (units + qb > 0x7fffffff) return cudaErrorInvalidValue;
  AppendArgs a{b, rope, k, v, q, q_out, k_stride, v_stride, q_stride, q_out_stride, (int32_t)units, q_heads};
  const dim3 grid((unsigned)(units + qb)), block(threads);
#define MK_LAUNCH_APPEND(PP)                                                                \
  return L.e4m3 ? launch_pdl(k_paged_append<PP, true>, grid, block, 0, s, 0, L, a)          \
                : launch_pdl(k_paged_append<PP, false>, grid, block, 0, s, 0, L, a)
  if (L.P == 16) MK_LAUNCH_APPEND(16);
  if (L.P == 32) MK_LAUNCH_APPEND(32);
  MK_LAUNCH_APPEND(64);
#undef MK_LAUNCH_APPEND
}

}  // namespace mk
