// Attention of single tokens over the paged cache (bf16, or e4m3 with a scale
// per page and head).
//
// Mathematics.  With z_t = scale q.k_t, out = sum_t e^(z_t) v_t / sum_t e^(z_t),
// kept as a running maximum, sum and accumulator in fp32, base 2.  In e4m3,
// k_t = a_p K_t and v_t = b_p V_t with one a_p, b_p per page: a_p multiplies
// the logit, and b_p is added to it as log2 b_p, so that the weight that
// multiplies the codes is 2^(z_t + log2 b_p - m); the sum of the plain weights
// takes it back with 1 / b_p.  The maximum m is over z_t + log2 b_p: the
// weights that reach the value product are relative to the largest
// contribution, and with scales up to 2^80 apart none that matters to the sum
// falls below the smallest exponent (2^-126).
//
// What bounds it: HBM, each page is read once for all query heads that share
// it (4 flops a byte and head).  The layout therefore follows the loads:
//  * Work split on the device, from the lengths: the tokens of all (sequence,
//    kv head) units are cut into chunks (32 tokens in e4m3, 16 in bf16: 8 KB of
//    keys and values), and every CTA takes an equal run of the flat list of
//    chunks, so a batch of uneven lengths and a single long context load the
//    SMs alike and no length is needed on the host.
//  * Each warp has its own ring of stages, filled by tensor copies with a
//    128-byte swizzle (no barrier between warps while a unit lasts); page ids
//    are read one chunk ahead of the copy that needs them.
//  * e4m3 codes become fp16 (exact) and q, scaled by a power of two per head
//    so that it fits, fp16 too; products on mma.sync m16n8k16.  Few rows: the
//    tensor cores idle either way, and this form needs no shared-memory
//    round trip for the weights.  S = Q K^T puts a head's weights in the lanes
//    that hold them as the B operand of O^T = V^T P.  V's transpose is taken
//    in registers: a lane loads 16 channels of 4 tokens and pairs bytes of two
//    tokens, one permute and two conversions for four elements.
//  * The weights are rounded to fp16 after a factor 2^14 (smallest step
//    2^-38 of the largest weight: a long flat tail under one dominant token
//    is not lost); for bf16 values they are two bf16 parts (16 bits).
//  * A unit that lies in several CTAs is joined by the last of them to arrive
//    (counter, no waiting), in the order of the parts: the same result in
//    every run.
// Measured (GB300, 32 query heads over 8): 1M tokens e4m3 330 us (6.5 TB/s,
// 96% of the copy rate), 128K 56 us (4.7 TB/s: about 15 us are launch, ramp and
// joining), 4K 12 us, 64 ragged sequences 206 us (5.3 TB/s), 4 x 32K bf16 93 us
// (5.8 TB/s).  Reads its algorithmic bytes once (268.9 MB of DRAM reads at 128K).
#include "mk_paged.cuh"

namespace mk {

namespace {

constexpr int kStageBytes = 8192;

struct DecodeArgs {
  mk_paged_batch b;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t q_stride, out_stride;
  float scale;          // times log2 e
  int32_t layer_page0;  // first page of the layer in the maps
  int32_t causal;       // several tokens a sequence: token j sees the first len - n_new + j + 1 keys
  float* part_acc;      // [2 grid][rows][128]
  float* part_ml;       // [2 grid][rows][2]
  int32_t* counters;    // [max_seqs][n_kv]
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void tma3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// A place in the flat list of chunks: chunk ch of (sequence seq, kv head).
struct Cursor {
  int seq, head, ch;
};

// C = 1: one token a sequence, a unit's rows are the head's G query heads.
// C = 2: a few tokens a sequence (verification), a unit's rows are up to 16
// (token, query head) rows: they fill the rows of the A operand that one token
// leaves empty.
template <bool E4M3, int NW, int NS, int C>
struct DecodeSmem {
  static constexpr int CH = E4M3 ? 32 : 16;  // tokens of a chunk
  static constexpr int ring = NW * NS * kStageBytes;
  static int rows(int G) { return C == 1 ? G : 16; }
  static int bytes(int G) { return 1024 + ring + NW * rows(G) * D * 4; }
};

template <bool E4M3, int NW, int NS, int C>
__global__ void __launch_bounds__(NW * 32, 1)
    k_paged_decode(PagedLayer L, DecodeArgs a, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
  constexpr int CH = DecodeSmem<E4M3, NW, NS, C>::CH, NT = CH / 8, NTHR = NW * 32;
  constexpr float kShift = E4M3 ? 14.0f : 0.0f;  // weights times 2^kShift before their rounding
  extern __shared__ unsigned char dyn[];
  __shared__ int64_t s_pre[MK_MAX_CALL_SEQS + 1];
  __shared__ int s_len[MK_MAX_CALL_SEQS], s_row[MK_MAX_CALL_SEQS], s_new[C == 1 ? 1 : MK_MAX_CALL_SEQS];
  __shared__ int64_t s_wsum[NW];
  __shared__ __align__(8) uint64_t s_bar[NW][NS];
  __shared__ __align__(16) float s_sc[NW][NS][4];  // k scale of box 0, 1; v scale of box 0, 1
  __shared__ float s_ml[NW][8 * C][2];
  __shared__ float s_M[8 * C], s_L[8 * C];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  unsigned char* ring = dyn + ((1024 - (smem_u32(dyn) & 1023)) & 1023);
  float* s_acc = reinterpret_cast<float*>(ring + DecodeSmem<E4M3, NW, NS, C>::ring);
  const int n_kv = L.n_kv, G = L.G, n_seqs = a.b.n_seqs, R = C == 1 ? G : 16;

  if (lane == 0)
    for (int i = 0; i < NS; ++i) mbar_init(&s_bar[warp][i], E4M3 ? 5 : 1);
  mbar_init_fence();
  pdl_wait();
  pdl_trigger();
  if (__syncthreads_or(tid == 0 && paged_stopped(L))) return;  // one thread's reading for the CTA

  int units = 0;  // (sequence, kv head) pairs with keys
  for (int i0 = 0; i0 < n_seqs; i0 += NTHR) {
    const int i = i0 + tid;
    bool keys = false;
    if (i < n_seqs) {
      const PagedSeq s = paged_seq(a.b, L.P, i, false);
      if (!s.ok) paged_error(L, ERR_PAGED_BATCH, i, s.len);
      const bool live = s.ok && (C == 1 ? s.n_new == 1 : s.n_new > 0);  // C = 2: n_new <= max_new <= 16 / G
      s_len[i] = live ? s.len : 0;
      s_row[i] = live ? s.row0 : -1;
      if (C > 1) s_new[i] = live ? s.n_new : 0;
      keys = live && s.len > 0;
    }
    units += __syncthreads_count(keys) * n_kv;
  }
  // The list of chunks: exclusive prefix over the sequences, each unit rounded
  // up to a multiple of `pad` places.
  auto n_chunks = [&](int seq) { return (s_len[seq] + CH - 1) / CH; };
  auto places = [&](int seq, int pad) { return (n_chunks(seq) + pad - 1) / pad * pad; };
  auto list = [&](int pad) {
    int64_t base = 0;
    for (int i0 = 0; i0 < n_seqs; i0 += NTHR) {
      const int i = i0 + tid;
      const int64_t mine = i < n_seqs ? (int64_t)places(i, pad) * n_kv : 0;
      int64_t x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) s_wsum[warp] = x;
      __syncthreads();
      int64_t off = base;
      for (int w = 0; w < NW; ++w) {
        if (w < warp) off += s_wsum[w];
        base += s_wsum[w];
      }
      if (i < n_seqs) s_pre[i] = off + x - mine;
      __syncthreads();
    }
    if (tid == 0) s_pre[n_seqs] = base;
    __syncthreads();
    return base;
  };
  int64_t total = list(1);

  // Rows of empty sequences.
  for (int i = blockIdx.x; i < n_seqs; i += gridDim.x)
    if (s_row[i] >= 0 && s_len[i] == 0) {
      for (int t = 0; t < (C == 1 ? 1 : s_new[i]); ++t) {
        for (int e = tid; e < n_kv * G * D / 8; e += NTHR)
          *reinterpret_cast<uint4*>(a.out + (int64_t)(s_row[i] + t) * a.out_stride + e * 8) = make_uint4(0, 0, 0, 0);
        if (a.lse)
          for (int e = tid; e < n_kv * G; e += NTHR) a.lse[(int64_t)(s_row[i] + t) * n_kv * G + e] = -INFINITY;
      }
    }

  int64_t per = (total + gridDim.x - 1) / gridDim.x;
  // A run that ends one unit and begins another joins twice, 5 us a time: where
  // runs are short (up to kAligned chunks) and the CTAs suffice, every unit
  // begins a run of its own (4K tokens in a graph of calls: 15.0 us without,
  // 11.5 with).
  constexpr int kAligned = 64, kShortest = 4;
  int pad = 1;
  if (total > 0 && units < (int)gridDim.x) {
    const int spare = (int)gridDim.x - units;
    int64_t p = (total + spare - 1) / spare;  // sum of ceil(n / p) <= total / p + units <= CTAs
    if (p < kShortest) p = kShortest;
    if (p <= kAligned) {
      per = pad = (int)p;
      total = list(pad);
    }
  }
  const int64_t c0 = (int64_t)blockIdx.x * per;
  if (c0 >= total) return;

  Cursor first;
  {
    int lo = 0, hi = n_seqs - 1;
    while (lo < hi) {  // the last sequence whose prefix is <= c0 and that has chunks
      const int mid = (lo + hi + 1) >> 1;
      if (s_pre[mid] <= c0) lo = mid; else hi = mid - 1;
    }
    const int64_t rem = c0 - s_pre[lo];
    const int n = places(lo, pad);
    first.seq = lo;
    first.head = (int)(rem / n);
    first.ch = (int)(rem - (int64_t)first.head * n);
  }
  // The CTA's chunks, from `first` on: of one unit only where units are padded.
  const int n_flat = pad > 1 ? min(pad, n_chunks(first.seq) - first.ch) : (int)(c0 + per < total ? per : total - c0);
  auto advance = [&](Cursor& k, int by) {
    k.ch += by;
    while (k.seq < n_seqs) {
      const int n = n_chunks(k.seq);
      if (k.ch < n) break;
      k.ch -= n;
      if (n == 0 || ++k.head == n_kv) {
        k.head = 0;
        ++k.seq;
      }
    }
  };

  // ---- the warp's copies ----
  const int box = E4M3 ? (L.P < 32 ? L.P : 32) : 16;  // tokens of one copy
  const int n_box = CH / box;
  Cursor ic = first;
  int issued = warp;  // flat index of the next chunk to copy
  advance(ic, warp);
  int pid = 0;
  auto fetch_pid = [&]() {
    if (issued < n_flat && lane < n_box) {
      const int p = (ic.ch * CH + lane * box) >> L.p_log2;
      if (ic.ch * CH + lane * box < s_len[ic.seq]) pid = a.b.page_table[(int64_t)ic.seq * a.b.table_stride + p];
    }
  };
  auto issue = [&](int stage) {
    if (issued >= n_flat) return;
    const int valid = s_len[ic.seq] - ic.ch * CH;  // tokens from the chunk's start
    if (lane < n_box && lane * box < valid && (pid < 0 || pid >= L.n_pages)) {
      paged_error(L, ERR_PAGED_PAGE, ic.seq, pid);
      pid = 0;
    }
    const int boxes = valid >= CH ? n_box : (valid + box - 1) / box;
    unsigned char* st = ring + (warp * NS + stage) * kStageBytes;
    uint64_t* bar = &s_bar[warp][stage];
    fence_proxy_async();  // this warp's earlier accesses to the stage come before the copies
    const int p0 = __shfl_sync(FULL, pid, 0), p1 = __shfl_sync(FULL, pid, 1);
    if (lane == 0) {
      mbar_expect_tx(bar, boxes * box * (E4M3 ? 2 * D : 4 * D));
      const int y = ic.head * L.P + ((ic.ch * CH) & (L.P - 1));
      for (int i = 0; i < boxes; ++i) {
        const int z = a.layer_page0 + (i ? p1 : p0);
        if (E4M3) {
          tma3(smem_u32(st) + i * box * D, &kmap, 0, y, z, bar);
          tma3(smem_u32(st) + 4096 + i * box * D, &vmap, 0, y, z, bar);
        } else {
          tma3(smem_u32(st), &kmap, 0, y, z, bar);
          tma3(smem_u32(st) + 2048, &kmap, 64, y, z, bar);
          tma3(smem_u32(st) + 4096, &vmap, 0, y, z, bar);
          tma3(smem_u32(st) + 6144, &vmap, 64, y, z, bar);
        }
      }
    }
    if (E4M3 && lane < 4) {
      float* to = &s_sc[warp][stage][lane];
      const int i = lane & 1;
      if (i < boxes) {
        const float* from = (lane < 2 ? L.k_scale : L.v_scale) + (int64_t)(i ? p1 : p0) * n_kv + ic.head;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from) : "memory");
      } else {
        *to = 1.0f;
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
    }
    issued += NW;
    if (issued < n_flat) advance(ic, NW);
    fetch_pid();
  };

  fetch_pid();
#pragma unroll
  for (int i = 0; i < NS; ++i) issue(i);
  __syncwarp();

  // ---- the units ----
  const uint32_t kRow = (uint32_t)(lane & 7) * 128u, kXor = (uint32_t)(lane & 7);
  int flat = warp, fs = 0, stage = 0;  // the warp's next chunk; the unit's first flat index; ring place
  unsigned phase = 0;
  bool dead = false;
  Cursor u = first;
  while (fs < n_flat) {
    const int len = s_len[u.seq], nch = n_chunks(u.seq);
    const int fe = min(n_flat, fs + nch - u.ch);  // the unit's chunks of this CTA: flat [fs, fe)
    const int row = s_row[u.seq], n_new = C == 1 ? 1 : s_new[u.seq];
    // Row x of the unit: its token, query head and whether there is one.
    auto tok_of = [&](int x) { return C == 1 ? 0 : x / G; };
    auto head_of = [&](int x) { return u.head * G + (C == 1 ? x : x % G); };
    auto live_row = [&](int x) { return C == 1 ? x < G : tok_of(x) < n_new; };

    // The unit's queries as A fragments: rows g and (C = 2) g + 8.  e4m3: fp16
    // after a power of two per row, in the channel order that the codes' pairs have.
    uint32_t qa[C][8], qb[C][8];
    float zf[C];
    int see[C];  // keys that the row sees
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int x = g + 8 * i;
      const bool on = live_row(x);
      const uint16_t* qp = a.q + (int64_t)(row + (on ? tok_of(x) : 0)) * a.q_stride + (on ? head_of(x) : 0) * D;
      zf[i] = a.scale;
      see[i] = C > 1 && a.causal && on ? max(0, min(len, len - n_new + tok_of(x) + 1)) : len;
      if (E4M3) {
        uint2 w[8];
        float top = 0.0f;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          w[s] = on ? *reinterpret_cast<const uint2*>(qp + 16 * s + 4 * c) : make_uint2(0, 0);
          top = fmaxf(top, fmaxf(fmaxf(fabsf(bf2f(w[s].x & 0xffff)), fabsf(bf2f(w[s].x >> 16))),
                                 fmaxf(fabsf(bf2f(w[s].y & 0xffff)), fabsf(bf2f(w[s].y >> 16)))));
        }
        top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
        top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
        int e = (int)(__float_as_uint(top) >> 23) - 127;
        e = max(-100, min(e, 120));
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        zf[i] *= __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          qa[i][s] = pack2<true>(bf2f(w[s].x & 0xffff) * down, bf2f(w[s].x >> 16) * down);
          qb[i][s] = pack2<true>(bf2f(w[s].y & 0xffff) * down, bf2f(w[s].y >> 16) * down);
        }
      } else {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          qa[i][s] = on ? *reinterpret_cast<const uint32_t*>(qp + 16 * s + 2 * c) : 0u;
          qb[i][s] = on ? *reinterpret_cast<const uint32_t*>(qp + 16 * s + 8 + 2 * c) : 0u;
        }
      }
    }
    // The first row sees the least: from there on chunks are masked by row.
    const int see_all = C > 1 && a.causal ? max(0, min(len, len - n_new + tok_of(0) + 1)) : len;
    float m[C], l[C];
    float o[C][8][4];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.0f;
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][n][e] = 0.0f;
    }

    for (; flat < fe; flat += NW) {
      const int tok0 = (u.ch + flat - fs) * CH;
      const int valid = min(CH, len - tok0);
      unsigned char* st = ring + (warp * NS + stage) * kStageBytes;
      // After a wait that ran out nothing more is copied; what is in flight is
      // still waited for (with the same limit) before the kernel ends.
      if (flat < issued && !paged_wait_warp(&s_bar[warp][stage], phase)) {
        dead = true;
        if (lane == 0) paged_error(L, ERR_PAGED_WAIT, u.seq, flat, (int32_t)MK_ETIMEOUT);
      }
      if (!dead) {
        const uint32_t kb = smem_u32(st), vb = kb + 4096;
        if (valid < CH) {  // slots past the length hold anything: their values must not reach 0 * value
          for (int r = valid + (lane >> 3); r < CH; r += 4) {
            const uint32_t at = vb + r * 128 + (lane & 7) * 16;
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0) : "memory");
            if (!E4M3) asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at + 2048), "r"(0) : "memory");
          }
          __syncwarp();
        }
        // logits: rows g and g + 8, columns = tokens 8 nt + 2 c (+ 1)
        float z[C][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          if (E4M3) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t r[4];
              ldsm4(r, kb + nt * 1024 + kRow + (((uint32_t)(4 * h + (lane >> 3)) ^ kXor) << 4));
#pragma unroll
              for (int s = 0; s < 4; ++s)
                mma16<true>(acc, qa[0][4 * h + s], C > 1 ? qa[C - 1][4 * h + s] : 0u, qb[0][4 * h + s],
                            C > 1 ? qb[C - 1][4 * h + s] : 0u, e4m3_h2(r[s]), e4m3_h2(r[s] >> 16));
            }
          } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint32_t r[4];
              ldsm4(r, kb + (h >> 1) * 2048 + nt * 1024 + kRow + (((uint32_t)(4 * (h & 1) + (lane >> 3)) ^ kXor) << 4));
#pragma unroll
              for (int s = 0; s < 2; ++s)
                mma16<false>(acc, qa[0][2 * h + s], C > 1 ? qa[C - 1][2 * h + s] : 0u, qb[0][2 * h + s],
                             C > 1 ? qb[C - 1][2 * h + s] : 0u, r[2 * s], r[2 * s + 1]);
            }
          }
#pragma unroll
          for (int i = 0; i < C; ++i) {
            z[i][nt][0] = acc[2 * i];
            z[i][nt][1] = acc[2 * i + 1];
          }
        }
        float inv[2] = {1.0f, 1.0f};
        float4 sc = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
        float b0 = 0.0f, b1 = 0.0f;
        const bool two = box < 32;
        if (E4M3) {
          sc = *reinterpret_cast<const float4*>(&s_sc[warp][stage][0]);
          const float v1 = two ? sc.w : sc.z;
          b0 = __log2f(sc.z);
          b1 = __log2f(v1);
          inv[0] = __frcp_rn(sc.z);
          inv[1] = __frcp_rn(v1);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
          if (E4M3) {
            const float k0 = zf[i] * sc.x, k1 = two ? zf[i] * sc.y : k0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) z[i][nt][e] = fmaf(z[i][nt][e], nt < 2 ? k0 : k1, nt < 2 ? b0 : b1);
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) z[i][nt][e] *= zf[i];
          }
          if (tok0 + CH > see_all) {
            const int lim = see[i] - tok0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (8 * nt + 2 * c + e >= lim) z[i][nt][e] = -INFINITY;
          }
          float mx = z[i][0][0];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mx = fmaxf(mx, fmaxf(z[i][nt][0], z[i][nt][1]));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
          if (__any_sync(FULL, mx > m[i])) {
            const float mn = fmaxf(m[i], mx);
            const float cr = m[i] == -INFINITY ? 0.0f : ex2(m[i] - mn);
            m[i] = mn;
            l[i] *= cr;
            const float c0f = __shfl_sync(FULL, cr, 8 * c), c1f = __shfl_sync(FULL, cr, 8 * c + 4);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              o[i][n][0] *= c0f;
              o[i][n][1] *= c1f;
              o[i][n][2] *= c0f;
              o[i][n][3] *= c1f;
            }
          }
          const float ms = (m[i] == -INFINITY ? 0.0f : m[i]) - kShift;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            z[i][nt][0] = ex2(z[i][nt][0] - ms);
            z[i][nt][1] = ex2(z[i][nt][1] - ms);
            l[i] = E4M3 ? fmaf(z[i][nt][0] + z[i][nt][1], inv[nt >> 1], l[i]) : l[i] + (z[i][nt][0] + z[i][nt][1]);
          }
        }
        // values: rows = channels, columns = the unit's rows, eight at a time
        if (E4M3) {
#pragma unroll
          for (int t = 0; t < CH / 16; ++t) {
            uint32_t p0[C], p1[C];
#pragma unroll
            for (int i = 0; i < C; ++i) {
              p0[i] = pack2<true>(z[i][2 * t][0], z[i][2 * t][1]);
              p1[i] = pack2<true>(z[i][2 * t + 1][0], z[i][2 * t + 1][1]);
            }
            const uint32_t r0 = vb + (16 * t + 2 * c) * 128;
            const uint32_t x0 = ((uint32_t)g ^ (uint32_t)(2 * c)) << 4, x1 = ((uint32_t)g ^ (uint32_t)(2 * c + 1)) << 4;
            const uint4 w0 = lds128(r0 + x0), w1 = lds128(r0 + 128 + x1), w2 = lds128(r0 + 1024 + x0),
                        w3 = lds128(r0 + 1152 + x1);
            const uint32_t a0[4] = {w0.x, w0.y, w0.z, w0.w}, a1[4] = {w1.x, w1.y, w1.z, w1.w},
                           a2[4] = {w2.x, w2.y, w2.z, w2.w}, a3[4] = {w3.x, w3.y, w3.z, w3.w};
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const uint32_t x = __byte_perm(a0[n >> 1], a1[n >> 1], n & 1 ? 0x7362 : 0x5140);
              const uint32_t y = __byte_perm(a2[n >> 1], a3[n >> 1], n & 1 ? 0x7362 : 0x5140);
              const uint32_t v0 = e4m3_h2(x), v1 = e4m3_h2(x >> 16), v2 = e4m3_h2(y), v3 = e4m3_h2(y >> 16);
#pragma unroll
              for (int i = 0; i < C; ++i) mma16<true>(o[i][n], v0, v1, v2, v3, p0[i], p1[i]);
            }
          }
        } else {
          uint32_t p0[C], p1[C], q0[C], q1[C];
#pragma unroll
          for (int i = 0; i < C; ++i) {
            p0[i] = pack2<false>(z[i][0][0], z[i][0][1]);
            p1[i] = pack2<false>(z[i][1][0], z[i][1][1]);
            q0[i] = pack2<false>(z[i][0][0] - bf2f(p0[i] & 0xffff), z[i][0][1] - bf2f(p0[i] >> 16));
            q1[i] = pack2<false>(z[i][1][0] - bf2f(p1[i] & 0xffff), z[i][1][1] - bf2f(p1[i] >> 16));
          }
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            uint32_t r[4];
            const int tr = ((lane >> 4) & 1) * 8 + (lane & 7), ck = 2 * n + ((lane >> 3) & 1);
            ldsm4_t(r, vb + (ck >> 3) * 2048 + tr * 128 + (((uint32_t)(ck & 7) ^ kXor) << 4));
#pragma unroll
            for (int i = 0; i < C; ++i) {
              mma16<false>(o[i][n], r[0], r[1], r[2], r[3], p0[i], p1[i]);
              mma16<false>(o[i][n], r[0], r[1], r[2], r[3], q0[i], q1[i]);
            }
          }
        }
      }
      __syncwarp();
      if (!dead) issue(stage);
      if (++stage == NS) {
        stage = 0;
        phase ^= 1u;
      }
    }

    // ---- join the warps ----
#pragma unroll
    for (int i = 0; i < C; ++i) {
      l[i] += __shfl_xor_sync(FULL, l[i], 1);
      l[i] += __shfl_xor_sync(FULL, l[i], 2);
      if (c == 0) {
        s_ml[warp][8 * i + g][0] = m[i];
        s_ml[warp][8 * i + g][1] = l[i];
      }
    }
    __syncthreads();
    if (tid < 8 * C) {
      float M = -INFINITY, S = 0.0f;
      for (int w = 0; w < NW; ++w) M = fmaxf(M, s_ml[w][tid][0]);
      // A part whose maximum is -infinity has no weights, or only NaN: its sum, 0 or NaN, counts as it is.
      for (int w = 0; w < NW; ++w) S += s_ml[w][tid][1] * (s_ml[w][tid][0] == -INFINITY ? 1.0f : ex2(s_ml[w][tid][0] - M));
      s_M[tid] = M;
      s_L[tid] = S;
    }
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 8 * i + 2 * c + e;
        if (h < R) {
          float M = -INFINITY;
          for (int w = 0; w < NW; ++w) M = fmaxf(M, s_ml[w][h][0]);
          const float f = s_ml[warp][h][0] == -INFINITY ? 0.0f : ex2(s_ml[warp][h][0] - M);
          float* to = s_acc + (warp * R + h) * D;
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            if (E4M3) {
              *reinterpret_cast<float2*>(to + 16 * g + 2 * n) = make_float2(o[i][n][e] * f, o[i][n][2 + e] * f);
            } else {
              to[16 * n + g] = o[i][n][e] * f;
              to[16 * n + 8 + g] = o[i][n][2 + e] * f;
            }
          }
        }
      }
    __syncthreads();
    // Row x of the result (where it has one): its output, and its lse.
    auto put = [&](int e, float x, float y) {
      const int r = e >> 6;
      if (!live_row(r)) return;
      const float f = s_L[r] > 0.0f || s_L[r] != s_L[r] ? 1.0f / s_L[r] : 0.0f;
      *reinterpret_cast<uint32_t*>(a.out + (int64_t)(row + tok_of(r)) * a.out_stride + head_of(r) * D + 2 * (e & 63)) =
          pack2<false>(x * f, y * f);
    };
    auto put_lse = [&](int r) {
      if (!a.lse || !live_row(r)) return;
      a.lse[(int64_t)(row + tok_of(r)) * n_kv * G + head_of(r)] =
          s_L[r] > 0.0f || s_L[r] != s_L[r] ? (log2f(s_L[r]) + (s_M[r] - kShift)) * 0.6931471805599453f : -INFINITY;
    };
    const bool whole = u.ch == 0 && fe - fs == nch;
    const int64_t part = 2 * (int64_t)blockIdx.x + (u.ch == 0 ? 1 : 0);
    for (int e = tid; e < R * D / 2; e += NTHR) {
      float x = 0.0f, y = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(s_acc + w * R * D + 2 * e);
        x += v.x;
        y += v.y;
      }
      if (whole)
        put(e, x, y);
      else
        *reinterpret_cast<float2*>(a.part_acc + part * R * D + 2 * e) = make_float2(x, y);
    }
    if (tid < R) {
      if (whole) {
        put_lse(tid);
      } else {
        a.part_ml[(part * R + tid) * 2] = s_M[tid];
        a.part_ml[(part * R + tid) * 2 + 1] = s_L[tid];
      }
    }
    if (!whole) {
      // CTAs that hold a part of this unit: b_lo .. b_hi; the last to arrive joins them.
      const int64_t u0 = s_pre[u.seq] + (int64_t)u.head * places(u.seq, pad);
      const int b_lo = (int)(u0 / per), b_hi = (int)((u0 + nch - 1) / per), parts = b_hi - b_lo + 1;
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        int32_t* ctr = a.counters + (int64_t)u.seq * n_kv + u.head;
        const int old = atomicAdd(ctr, 1);
        s_last = old == parts - 1;
        if (s_last) *ctr = 0;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        auto slot = [&](int i) { return 2 * (int64_t)(b_lo + i) + (i == 0 ? 1 : 0); };
        for (int h = warp; h < R; h += NW) {  // a warp per row: the joined maximum and sum
          float M = -INFINITY, S = 0.0f;
          for (int i = lane; i < parts; i += 32) M = fmaxf(M, __ldcg(a.part_ml + (slot(i) * R + h) * 2));
          M = warp_max(M);
          for (int i = lane; i < parts; i += 32) {
            const float mi = __ldcg(a.part_ml + (slot(i) * R + h) * 2);
            S += __ldcg(a.part_ml + (slot(i) * R + h) * 2 + 1) * (mi == -INFINITY ? 1.0f : ex2(mi - M));
          }
          S = warp_sum(S);
          if (lane == 0) {
            s_M[h] = M;
            s_L[h] = S;
          }
        }
        __syncthreads();
        for (int e = tid; e < R * D / 2; e += NTHR) {
          const int h = e >> 6;
          const float M = s_M[h];
          float x = 0.0f, y = 0.0f;
#pragma unroll 8
          for (int i = 0; i < parts; ++i) {
            const float mi = __ldcg(a.part_ml + (slot(i) * R + h) * 2);
            const float f = mi == -INFINITY ? 0.0f : ex2(mi - M);
            const float2 v = __ldcg(reinterpret_cast<const float2*>(a.part_acc + slot(i) * R * D + 2 * e));
            x = fmaf(v.x, f, x);
            y = fmaf(v.y, f, y);
          }
          put(e, x, y);
        }
        if (tid < R) put_lse(tid);
      }
    }
    __syncthreads();  // s_ml, s_acc, s_M, s_L are free again
    fs = fe;
    u.ch = 0;
    if (++u.head == n_kv) {
      u.head = 0;
      ++u.seq;
    }
    while (u.seq < n_seqs && n_chunks(u.seq) == 0) ++u.seq;
  }
}

template <bool E4M3, int NW, int NS, int C = 1>
cudaError_t launch(const PagedLayer& L, const PagedMaps& maps, DecodeArgs a, cudaStream_t s) {
  const int bytes = DecodeSmem<E4M3, NW, NS, C>::bytes(L.G);
  int sms = 0;
  const cudaError_t e = kernel_smem_attr((const void*)k_paged_decode<E4M3, NW, NS, C>, bytes, NW * 32, nullptr, &sms);
  if (e != cudaSuccess) return e;
  const int grid = sms > 0 && sms <= kPagedMaxCtas ? sms : 128;
  return launch_pdl(k_paged_decode<E4M3, NW, NS, C>, dim3(grid), dim3(NW * 32), (size_t)bytes, s, 0, L, a, maps.k, maps.v);
}

}  // namespace

cudaError_t launch_paged_decode(const PagedLayer& L, const PagedMaps& maps, const PagedScratch& w, int layer,
                                const mk_paged_batch& b, bool several, bool causal, const uint16_t* q, int64_t q_stride,
                                float scale, uint16_t* out, int64_t out_stride, float* lse, cudaStream_t s) {
  DecodeArgs a{b, q, out, lse, q_stride, out_stride, scale * kLog2e, layer * L.n_pages, causal ? 1 : 0,
               w.part_acc, w.part_ml, w.counters};
  // 16 rows: 64 accumulators more a lane, eight warps of 255 registers.
  if (several) return L.e4m3 ? launch<true, 8, 2, 2>(L, maps, a, s) : launch<false, 8, 2, 2>(L, maps, a, s);
  // 12 warps of two 8 KB stages: the conversion of a chunk takes a warp about
  // 3 000 clocks, so eight were bound by it (64 ragged sequences 228 us, 12
  // warps 203); 16 with one stage wait for their copies (221).  Eight heads'
  // joining buffer (10 x 4 KB) leaves room for ten: the same batch with 64 query
  // heads 250 us, 344 in bf16 (32 heads: 206, 334).
  if (L.G == 8) return L.e4m3 ? launch<true, 10, 2>(L, maps, a, s) : launch<false, 10, 2>(L, maps, a, s);
  return L.e4m3 ? launch<true, 12, 2>(L, maps, a, s) : launch<false, 12, 2>(L, maps, a, s);
}

}  // namespace mk
