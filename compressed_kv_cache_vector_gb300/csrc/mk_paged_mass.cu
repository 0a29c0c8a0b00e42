// Attention mass over the paged cache: what softmax weights each held token
// got, summed over query tokens and over the query heads of its kv head.
#include <type_traits>

#include "mk_paged_tc.cuh"

namespace mk {

namespace {

// ---- a decode step's weights, from the logits that the attention left ----
// A thread a token: the group's weights 2^(z - lse2) summed and added.  HBM
// (mostly L2, where the logits still are): 4 G bytes read, 8 for the mass.
// 48 sequences of mixed lengths, 8 kv heads: 19 us behind 134 of attention (the
// call 155; with one token a thread 161); 3 sequences of 100K tokens 19 behind 207.
constexpr int kFoldThreads = 256, kFoldTokens = 4;  // tokens of a thread, for the loads in flight
constexpr int kFoldTile = kFoldThreads * kFoldTokens;

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
      if (s.ok && s.n_new == 1 && s.len > first) x = (int64_t)((s.len - first + kFoldTile - 1) / kFoldTile) * n_kv;
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
    const int64_t t0 = first + in / n_kv * kFoldTile + tid;
    const float* ls = lse2 + ((int64_t)seq * n_kv + head) * G;
    int64_t unit[kFoldTokens];
#pragma unroll
    for (int e = 0; e < kFoldTokens; ++e) {
      const int64_t t = t0 + e * kFoldThreads;
      const int page = t < len ? b.page_table[(int64_t)seq * b.table_stride + (t >> L.p_log2)] : -1;
      unit[e] = page < 0 || page >= L.n_pages ? -1 : (int64_t)page * n_kv + head;  // a bad one is recorded by the attention
    }
    float sum[kFoldTokens], old[kFoldTokens];
#pragma unroll
    for (int e = 0; e < kFoldTokens; ++e) {
      const int64_t t = t0 + e * kFoldThreads;
      sum[e] = old[e] = 0.0f;
      if (unit[e] >= 0 && t < len - 1) old[e] = mass[unit[e] * L.P + (t & (L.P - 1))];
    }
    for (int g = 0; g < G; ++g) {
      const float s = ls[g];
#pragma unroll
      for (int e = 0; e < kFoldTokens; ++e)
        if (unit[e] >= 0) sum[e] += ex2(logits[(unit[e] * G + g) * L.P + ((t0 + e * kFoldThreads) & (L.P - 1))] - s);
    }
#pragma unroll
    for (int e = 0; e < kFoldTokens; ++e)
      if (unit[e] >= 0) mass[unit[e] * L.P + ((t0 + e * kFoldThreads) & (L.P - 1))] = old[e] + sum[e];
  }
}

// ---- a prompt's weights ----
// Products on the 5th-generation tensor cores with the keys as rows: S^T = K
// Q^T, 128 keys by 128 rows (query token, query head).  A thread then has one
// key: its sum over the rows needs no exchange, a causal mask is a first
// column, and its page's scale one factor.  A weight is 2^(S k + n) with the
// key's factor k and the row's n = -lse log2 e from shared memory.
// What bounds it: the summing warps' instructions, the exponentials (32 a clock
// and SM: 62 us of a 6000-token prompt with 32 query heads) with the reading of
// logits and rows' numbers beside them: 154 us where the products take 76.
constexpr int kMassKeys = 256;   // keys of an item: two tiles of 128
constexpr int kMassRows = 128;   // rows of a step
constexpr int kMassTile = 128 * D * 2;
constexpr int kMassThreads = 448;  // 8 warps sum, 4 load keys, 1 loads queries, 1 issues
constexpr int kMassItemCost = 1;   // an item's begin and end take as long as this many steps
constexpr int kMassMinRun = 4;
constexpr int kMassSmem = 1024 + 6 * kMassTile;
constexpr int kMeta = 8;           // items whose pages are kept

struct MassArgs {
  mk_paged_batch b;
  const uint16_t* q;
  int64_t q_stride;
  const float* lse;
  float* mass;
  float scale;  // times log2 e
  int32_t causal, first, add, layer_page0;
  float* part;        // [2 kPagedMaxCtas][kMassKeys]
  int32_t* counters;  // [kPagedMaxCtas]
};

// A place in the list of items: 256 keys of a (sequence, kv head), and where
// it begins in the CTA's run (negative: in an earlier CTA's).
struct MassCursor {
  int seq, head, kt, rel;
};

// The list of items, and a CTA's run of it.
struct MassList {
  int64_t pre[MK_MAX_CALL_SEQS + 1];  // cost of the sequences before each
  int row0[MK_MAX_CALL_SEQS], n_new[MK_MAX_CALL_SEQS], len[MK_MAX_CALL_SEQS];
  MassCursor start;
  int64_t f0, per;
  int span, patience;
  int G, n_kv, n_seqs, kt0, causal;

  __device__ int tiles_of(int seq) const { return (int)(((int64_t)n_new[seq] * G + kMassRows - 1) / kMassRows); }
  __device__ int ends_of(int seq) const { return (len[seq] + kMassKeys - 1) / kMassKeys; }
  __device__ int skip_of(int seq, int kt) const {  // row tiles before the first that sees the item's first key
    const int64_t t = (int64_t)kt * kMassKeys - (len[seq] - n_new[seq]);
    return causal && t > 0 ? (int)(t * G / kMassRows) : 0;
  }
  __device__ int cost_of(int seq, int kt) const { return tiles_of(seq) - skip_of(seq, kt) + kMassItemCost; }
  __device__ void next(MassCursor& k) const {
    k.rel += cost_of(k.seq, k.kt);
    if (++k.kt < ends_of(k.seq)) return;
    k.kt = kt0;
    if (++k.head < n_kv) return;
    k.head = 0;
    do ++k.seq;
    while (k.seq < n_seqs && ends_of(k.seq) <= kt0);
  }
  // The item's steps in this run are the row tiles [j0, j1) behind the skipped ones.
  __device__ int steps(const MassCursor& k, int& j0, int& j1) const {
    const int n = cost_of(k.seq, k.kt) - kMassItemCost;
    j0 = max(0, -k.rel);
    j1 = min(n, span - k.rel);
    return n;
  }
};

// What the two groups of four summing warps (each with 64 columns of a step)
// share.  They take the items' ends in turn: one leaves its sums here, the
// other adds them to its own.  Four items' room: a group is at most two steps
// behind the other, since the logits' buffers want both.
struct MassSums {
  uint64_t full[4], met[2];
  float other[4][2][128];
  int last[2];
};
struct MassShared {
  MassList list;
  uint64_t q_full[2], q_free[2], s_full[2], s_free[2], k_full[2], k_free[2], done;
  // -lse log2 e of a step's rows, -infinity where there is none.  A sum gives its
  // logits back before it has read the last of these, hence more than four.
  __align__(16) float nlse[8][kMassRows];
  int page[kMeta][kMassKeys / 16];         // pages of an item's keys, -1: none
  float ks[kMeta][kMassKeys / 16];         // their scales (e4m3)
  MassSums sums;
  uint32_t tmem;
  volatile int dead;
};

// Forms the list (an item's steps are the row tiles that see its first key; it
// is as long as these and kMassItemCost) and the CTA's run: the list is cut
// into equal runs, one a CTA.  False where nothing is left for this CTA.
__device__ bool mass_list(const PagedLayer& L, const MassArgs& a, MassList& m) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_seqs = a.b.n_seqs, n_kv = L.n_kv, warps = blockDim.x / 32;
  if (tid == 0) {
    m.G = L.G;
    m.n_kv = n_kv;
    m.n_seqs = n_seqs;
    m.kt0 = a.first / kMassKeys;
    m.causal = a.causal;
  }
  __syncthreads();
  const int kt0 = m.kt0;
  for (int i = warp; i < n_seqs; i += warps) {
    PagedSeq s = paged_seq(a.b, L.P, i, false);
    if (!s.ok) {
      if (lane == 0) paged_error(L, ERR_PAGED_BATCH, i, s.len);
      s.n_new = 0;
    }
    if (s.n_new == 0) s.len = 0;
    if (lane == 0) {
      m.row0[i] = s.row0;
      m.n_new[i] = s.n_new;
      m.len[i] = s.len;
    }
    __syncwarp();
    int64_t x = 0;
    for (int kt = kt0 + lane, n = m.ends_of(i); kt < n; kt += 32) x += m.cost_of(i, kt);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
    if (lane == 0) m.pre[i] = x * n_kv;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t at = 0;
    for (int i0 = 0; i0 < n_seqs; i0 += 32) {
      const int i = i0 + lane;
      const int64_t mine = i < n_seqs ? m.pre[i] : 0;
      int64_t x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x += y;
      }
      if (i < n_seqs) m.pre[i] = at + x - mine;
      at += __shfl_sync(FULL, x, 31);
    }
    if (lane == 0) m.pre[n_seqs] = at;
  }
  __syncthreads();
  const int64_t total = m.pre[n_seqs];
  int64_t per = (total + gridDim.x - 1) / gridDim.x;
  if (per < kMassMinRun) per = kMassMinRun;
  const int64_t f0 = (int64_t)blockIdx.x * per;
  if (f0 >= total) return false;
  if (warp == 0) {
    int lo = 0, hi = n_seqs - 1;
    while (lo < hi) {  // the last sequence that begins at or before f0
      const int mid = (lo + hi + 1) >> 1;
      if (m.pre[mid] <= f0) lo = mid; else hi = mid - 1;
    }
    const int64_t one = (m.pre[lo + 1] - m.pre[lo]) / n_kv;  // a kv head's items
    const int head = (int)((f0 - m.pre[lo]) / one);
    int64_t at = m.pre[lo] + head * one;
    for (int k0 = kt0, n = m.ends_of(lo); k0 < n; k0 += 32) {
      const int kt = k0 + lane;
      const int64_t cost = kt < n ? m.cost_of(lo, kt) : 0;
      int64_t x = cost;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x += y;
      }
      const unsigned past = __ballot_sync(FULL, at + x > f0);
      if (past) {
        if (lane == __ffs(past) - 1) m.start = MassCursor{lo, head, kt, (int)(at + x - cost - f0)};
        break;
      }
      at += __shfl_sync(FULL, x, 31);
    }
    if (lane == 0) {
      m.f0 = f0;
      m.per = per;
      m.span = (int)(total - f0 < per ? total - f0 : per);
      m.patience = 100 + m.span / 1024;
    }
  }
  __syncthreads();
  return true;
}

// One step of a warp: 64 of its 128 columns (from `col` on) for two keys a
// thread, whose factors are k[0] and k[1]: a row's numbers, read from shared
// memory for all lanes at once (as many cycles as columns), serve both.
// kCut: columns before c[e], which key e is not seen by, and from `cols` on
// count nothing.  ZE: a row has a factor of its own.  free() is called when all
// logits have been read.
template <bool kCut, bool ZE, typename Free>
__device__ __forceinline__ void mass_step(uint32_t taddr, int col, const float* nl, const float* ze, const float (&k)[2], const int (&c)[2],
                                          int cols, uint64_t (&add)[2][2], Free free) {
  const uint64_t k2[2] = {pair(k[0], k[0]), pair(k[1], k[1])};
  uint32_t v[2][2][16];
#pragma unroll
  for (int e = 0; e < 2; ++e) tmem_ld16_async(taddr + e * 256, v[0][e]);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    tmem_ld_wait16(v[g & 1][0]);
    tmem_ld_wait16(v[g & 1][1]);
    if (g < 3) {
#pragma unroll
      for (int e = 0; e < 2; ++e) tmem_ld16_async(taddr + e * 256 + 16 * (g + 1), v[(g + 1) & 1][e]);
    } else {
      free();
    }
    if (kCut && col + 16 * g >= cols) continue;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 n4 = *reinterpret_cast<const float4*>(&nl[col + 16 * g + i]);
      float4 z4;
      if (ZE) z4 = *reinterpret_cast<const float4*>(&ze[col + 16 * g + i]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t(&z)[16] = v[g & 1][e];
        const uint64_t f0 = ZE ? mul2(pair(z4.x, z4.y), k2[e]) : k2[e], f1 = ZE ? mul2(pair(z4.z, z4.w), k2[e]) : k2[e];
        float x[4];
        unpair(fma2(pair(__uint_as_float(z[i]), __uint_as_float(z[i + 1])), f0, pair(n4.x, n4.y)), x[0], x[1]);
        unpair(fma2(pair(__uint_as_float(z[i + 2]), __uint_as_float(z[i + 3])), f1, pair(n4.z, n4.w)), x[2], x[3]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          x[u] = ex2(x[u]);
          if (kCut && (col + 16 * g + i + u < c[e] || col + 16 * g + i + u >= cols)) x[u] = 0.0f;
        }
        add[e][0] = add2(add[e][0], pair(x[0], x[1]));
        add[e][1] = add2(add[e][1], pair(x[2], x[3]));
      }
    }
  }
}

// Two keys' sums (key and key + 128 of the item) over the item's steps [j0, j1)
// of n: into the mass, or a part where several CTAs have steps of the item: the
// last to come adds the parts, in their order.  128 threads.
template <typename Meet>
__device__ __forceinline__ bool mass_leave(const PagedLayer& L, const MassArgs& a, const MassList& list, const MassCursor& k, int j0,
                                           int j1, int n, const int* pages, int key, const float (&sum)[2], int* last, Meet meet) {
  const int len = list.len[k.seq], n_new = list.n_new[k.seq];
  auto put = [&](int e, float x) {
    const int at = e * 128 + key, t = k.kt * kMassKeys + at, page = pages[at >> 4];
    if (page < 0 || t < a.first || t >= len) return;
    float* to = a.mass + ((int64_t)page * L.n_kv + k.head) * L.P + (t & (L.P - 1));
    *to = a.add && (!a.causal || t < len - n_new) ? *to + x : x;
  };
  if (j0 == 0 && j1 == n) {
    put(0, sum[0]);
    put(1, sum[1]);
    return true;
  }
  const int64_t place = list.f0 + k.rel;
  const int b_lo = (int)(place / list.per), parts = (int)((place + n - 1) / list.per) - b_lo + 1;
  auto slot = [&](int i) { return a.part + (2 * (int64_t)(b_lo + i) + (i == 0 ? 1 : 0)) * kMassKeys + key; };
  float* const mine = slot((int)blockIdx.x - b_lo);
  mine[0] = sum[0];
  mine[128] = sum[1];
  __threadfence();
  if (!meet()) return false;
  if (key == 0) {
    int32_t* ctr = &a.counters[b_lo];  // one item at most begins in b_lo and ends after it
    const int old = atomicAdd(ctr, 1);
    *last = old == parts - 1;
    if (*last) *ctr = 0;
  }
  if (!meet()) return false;
  if (*last) {
    __threadfence();
    float x = 0.0f, y = 0.0f;
    for (int i = 0; i < parts; ++i) {
      x += __ldcg(slot(i));
      y += __ldcg(slot(i) + 128);
    }
    put(0, x);
    put(1, y);
  }
  return meet();  // *last is free again
}

__device__ __forceinline__ void mass_sums_init(MassSums& m) {
  for (int i = 0; i < 4; ++i) mbar_init(&m.full[i], 4);
  for (int i = 0; i < 2; ++i) mbar_init(&m.met[i], 4);
}

// The keys of two items and two tiles of queries are held: the next item's keys
// are there early.  One item and four tiles: 161 against 153 us (6000 tokens),
// 78 against 76 (five ragged chunks).
template <bool E4M3>
__global__ void __launch_bounds__(kMassThreads, 1)
    k_prefill_mass(PagedLayer L, MassArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ unsigned char dyn[];
  __shared__ MassShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
  constexpr int NK = 2, NQ = 2;  // items' keys, tiles of queries
  const uint32_t sk = base, sq = base + 2 * NK * kMassTile;
  const int G = L.G, g_log2 = __ffs(G) - 1, n_kv = L.n_kv;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_free[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_free[i], 8);
      mbar_init(&sh.k_full[i], E4M3 ? 4 : 1);
      mbar_init(&sh.k_free[i], 1);
    }
    mass_sums_init(sh.sums);
    mbar_init(&sh.done, 1);
    sh.dead = 0;
  }
  mbar_init_fence();
  pdl_wait();
  pdl_trigger();
  if (__syncthreads_or(tid == 0 && paged_stopped(L))) return;

  if (!mass_list(L, a, sh.list)) return;
  const MassList& list = sh.list;
  if (warp == 13) tmem_alloc(&sh.tmem, 512);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tmem = sh.tmem;

  auto slow = [&](uint64_t* bar, unsigned parity, int times) {
    for (int i = 0; i < times; ++i) {
      if (sh.dead) return false;
      if (paged_wait(bar, parity)) return true;
    }
    sh.dead = 1 + warp;
    return false;
  };
  auto wait = [&](uint64_t* bar, unsigned parity) { return mbar_try_wait(bar, parity) || slow(bar, parity, 1); };
  // For a wait that an item's steps can lie between.
  auto wait_long = [&](uint64_t* bar, unsigned parity) { return mbar_try_wait(bar, parity) || slow(bar, parity, list.patience); };
  if (warp == 13) {
    // ---- issues the products ----
    if (elect_one()) {
      unsigned c = 0, ic = 0;
      bool ok = true;
      const uint64_t dk = sw128_desc(sk, 16), dq = sw128_desc(sq, 16);
      int j0, j1;
      for (MassCursor k = list.start; ok && k.rel < list.span; list.next(k)) {
        list.steps(k, j0, j1);
        if (j0 >= j1) continue;
        ok = wait(&sh.k_full[ic % NK], (ic / NK) & 1);
        for (int j = j0; ok && j < j1; ++j, ++c) {
          ok = wait(&sh.q_full[c % NQ], (c / NQ) & 1);
          ok = ok && (c < 2 || wait(&sh.s_free[c & 1], ((c >> 1) - 1) & 1));
          if (!ok) break;
          tmem_fence_after_sync();
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint64_t da = dk + (uint64_t)((((ic % NK) * 2 + w) * kMassTile) >> 4), db = dq + (uint64_t)(((c % NQ) * kMassTile) >> 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t o = ((i >> 2) * (kMassTile / 2) + (i & 3) * 32) >> 4;
              umma_ss(tmem + w * 256 + (c & 1) * 128, da + o, db + o, idesc(1, 0), i > 0);
            }
          }
          umma_commit(&sh.s_full[c & 1]);
          umma_commit(&sh.q_free[c % NQ]);
        }
        if (ok) umma_commit(&sh.k_free[ic % NK]);
        ++ic;
      }
      umma_commit(&sh.done);
    }
    // Nothing is in flight when the tensor memory is freed.
    __syncwarp();
    (void)paged_wait_warp(&sh.done, 0);
  } else if (warp == 12) {
    // ---- loads queries and the rows' sums ----
    unsigned c = 0;
    bool ok = true;
    int j0, j1;
    const int n_q = n_kv * G;
    for (MassCursor k = list.start; ok && k.rel < list.span; list.next(k)) {
      list.steps(k, j0, j1);
      const int row0 = list.row0[k.seq];
      const int64_t rows = (int64_t)list.n_new[k.seq] * G;
      const int skip = list.skip_of(k.seq, k.kt);
      for (int j = j0; ok && j < j1; ++j, ++c) {
        const int64_t r0 = (int64_t)(skip + j) * kMassRows;
        float n[4];
        bool none = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t r = r0 + lane * 4 + e;
          const float ls = r < rows ? a.lse[(row0 + (r >> g_log2)) * n_q + k.head * G + (int)(r & (G - 1))] : -INFINITY;
          n[e] = ls == -INFINITY ? -INFINITY : -ls * kLog2e;
          none |= r < rows && ls == -INFINITY;
        }
        none = __any_sync(FULL, none);
        ok = c < NQ || __all_sync(FULL, wait(&sh.q_free[c % NQ], (c / NQ - 1) & 1));
        if (!ok) break;
        *reinterpret_cast<float4*>(&sh.nlse[c & 7][lane * 4]) = make_float4(n[0], n[1], n[2], n[3]);
        __syncwarp();
        const uint32_t to = sq + (c % NQ) * kMassTile;
        if (none) {  // a row without a sum, whatever its query holds: the step's queries by hand, without it
#pragma unroll 8
          for (int i = lane; i < kMassRows * 16; i += 32) {
            const int x = i >> 4, ck = i & 15;
            const int64_t tok = row0 + ((r0 + x) >> g_log2);
            const int h = k.head * G + (x & (G - 1));
            uint4 v = make_uint4(0, 0, 0, 0);
            float ls = -INFINITY;
            if (r0 + x < rows) {
              v = *reinterpret_cast<const uint4*>(a.q + tok * a.q_stride + h * D + ck * 8);
              ls = a.lse[tok * n_q + h];
            }
            if (ls == -INFINITY) v = make_uint4(0, 0, 0, 0);
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to + (ck >> 3) * (kMassTile / 2) + x * 128 + (((ck & 7) ^ (x & 7)) << 4)),
                         "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                         : "memory");
          }
          fence_proxy_async();
          mbar_arrive_warp(&sh.q_full[c % NQ], lane);
        } else if (lane == 0) {
          mbar_expect_tx(&sh.q_full[c % NQ], kMassTile);
          const int tok = row0 + (int)(r0 >> g_log2);
          tma3(to, &qmap, 0, k.head * G, tok, &sh.q_full[c % NQ]);
          tma3(to + kMassTile / 2, &qmap, 64, k.head * G, tok, &sh.q_full[c % NQ]);
        }
      }
    }
    // No copy is in flight when the kernel ends, also after a wait that ran out.
    for (unsigned i = c < NQ ? 0 : c - NQ; i < c; ++i) (void)paged_wait_warp(&sh.q_full[i % NQ], (i / NQ) & 1);
  } else if (warp >= 8) {
    // ---- keys into shared memory ----
    const int lt = tid - 256;
    unsigned ic = 0;
    bool ok = true;
    int j0, j1;
    auto page_at = [&](const MassCursor& k) {  // lane g < 16: the page of the item's 16-key group g, -1 where there is none
      const int tok = k.kt * kMassKeys + lane * 16;
      int p = -1;
      if (lane < 16 && tok < list.len[k.seq]) {
        p = a.b.page_table[(int64_t)k.seq * a.b.table_stride + (tok >> L.p_log2)];
        if (p < 0 || p >= L.n_pages) {
          paged_error(L, ERR_PAGED_PAGE, k.seq, p);
          p = -1;
        }
      }
      return p;
    };
    if (E4M3) {
      // 16 codes ck of rows r + 16 i, as the attention of several query tokens loads them.
      const int ck = (lane & 3) | (lane >> 1 & 4), r = (lane >> 2 & 1) | (lane >> 3 & 2) | (warp & 3) << 2;
      const uint32_t put = (ck >> 2) * (kMassTile / 2) + r * 128 + ((((2 * ck) & 7) ^ (r & 7)) << 4);
      const int64_t page_stride = (int64_t)n_kv * L.P * D;
      for (MassCursor k = list.start; ok && k.rel < list.span; list.next(k)) {
        list.steps(k, j0, j1);
        if (j0 >= j1) continue;
        const int pg = page_at(k);
        uint4 x[16];
        const uint8_t* from = L.k + (int64_t)k.head * L.P * D + ck * 16;
        const int slot = k.kt * kMassKeys + r;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int p = __shfl_sync(FULL, pg, i);
          x[i] = make_uint4(0, 0, 0, 0);
          if (p >= 0) x[i] = *reinterpret_cast<const uint4*>(from + p * page_stride + ((slot + 16 * i) & (L.P - 1)) * D);
        }
        float ks = 1.0f;
        if (lt < 16 && pg >= 0) ks = L.k_scale[(int64_t)pg * n_kv + k.head];
        ok = ic < NK || __all_sync(FULL, wait_long(&sh.k_free[ic % NK], (ic / NK - 1) & 1));
        if (!ok) break;
        if (lt < 16) {
          sh.page[ic % kMeta][lt] = pg;
          sh.ks[ic % kMeta][lt] = ks;
        }
        const uint32_t to = sk + (ic % NK) * 2 * kMassTile + put;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {  // exact: e4m3 has 4 significant bits
            const uint32_t h = e4m3_h2(w[e >> 1] >> (16 * (e & 1)));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            o[e] = pack2<false>(f.x, f.y);
          }
          const uint32_t at = to + (i >> 3) * kMassTile + (i & 7) * 2048;
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]) : "memory");
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at ^ 16), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]) : "memory");
        }
        fence_proxy_async();
        mbar_arrive_warp(&sh.k_full[ic % NK], lane);
        ++ic;
      }
    } else if (warp == 8) {
      for (MassCursor k = list.start; ok && k.rel < list.span; list.next(k)) {
        list.steps(k, j0, j1);
        if (j0 >= j1) continue;
        const int pg = page_at(k);
        ok = ic < NK || __all_sync(FULL, wait_long(&sh.k_free[ic % NK], (ic / NK - 1) & 1));
        if (!ok) break;
        if (lane < 16) sh.page[ic % kMeta][lane] = pg;
        const unsigned groups = __ballot_sync(FULL, pg >= 0);
        __syncwarp();
        if (lane == 0) mbar_expect_tx(&sh.k_full[ic % NK], __popc(groups) * 16 * D * 2);
        __syncwarp();
        if (pg >= 0) {
          const uint32_t to = sk + ((ic % NK) * 2 + (lane >> 3)) * kMassTile + (lane & 7) * 2048;
          const int y = k.head * L.P + ((k.kt * kMassKeys + lane * 16) & (L.P - 1)), z = a.layer_page0 + pg;
          tma3(to, &kmap, 0, y, z, &sh.k_full[ic % NK]);
          tma3(to + kMassTile / 2, &kmap, 64, y, z, &sh.k_full[ic % NK]);
        }
        ++ic;
      }
      for (unsigned i = ic < NK ? 0 : ic - NK; i < ic; ++i) (void)paged_wait_warp(&sh.k_full[i % NK], (i / NK) & 1);
    }
  } else {
    // ---- sums: two keys a thread, half of the columns ----
    int j0, j1;
    const int w = warp >> 2, key = tid & 127;
    const uint32_t ts = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + w * 64;
    unsigned c = 0, ic = 0, meets = 0;
    bool ok = true;
    auto meet = [&]() {  // the four warps of this half
      mbar_arrive_warp(&sh.sums.met[w], lane);
      const unsigned parity = meets++ & 1;
      return __all_sync(FULL, wait(&sh.sums.met[w], parity)) != 0;
    };
    for (MassCursor k = list.start; ok && k.rel < list.span; list.next(k)) {
      const int n = list.steps(k, j0, j1);
      if (j0 >= j1) continue;
      const int len = list.len[k.seq], n_new = list.n_new[k.seq], t = k.kt * kMassKeys + key, skip = list.skip_of(k.seq, k.kt);
      // Rows left of the sequence from the step's first one on, and the first of them that sees each key.
      int64_t left = (int64_t)n_new * G - (int64_t)(skip + j0) * kMassRows, from[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        from[e] = (a.causal ? max((int64_t)0, (int64_t)t + 128 * e - (len - n_new)) * G : 0) - (int64_t)(skip + j0) * kMassRows;
      float sum[2] = {0.0f, 0.0f}, low[2] = {0.0f, 0.0f};
      for (int j = j0; j < j1; ++j, ++c, left -= kMassRows, from[0] -= kMassRows, from[1] -= kMassRows) {
        ok = __all_sync(FULL, wait(&sh.s_full[c & 1], (c >> 1) & 1));
        if (!ok) break;
        tmem_fence_after_sync();
        const float kf[2] = {E4M3 ? a.scale * sh.ks[ic % kMeta][key >> 4] : a.scale, E4M3 ? a.scale * sh.ks[ic % kMeta][8 + (key >> 4)] : a.scale};
        const int cols = (int)min(left, (int64_t)kMassRows);
        const int c0[2] = {(int)min(max(from[0], (int64_t)0), (int64_t)kMassRows), (int)min(max(from[1], (int64_t)0), (int64_t)kMassRows)};
        uint64_t add[2][2] = {{0, 0}, {0, 0}};
        auto free = [&]() {
          tmem_fence_before_sync();
          mbar_arrive_warp(&sh.s_free[c & 1], lane);
        };
        if (cols < kMassRows || __any_sync(FULL, c0[1] > 0))
          mass_step<true, false>(ts + (c & 1) * 128, w * 64, sh.nlse[c & 7], nullptr, kf, c0, cols, add, free);
        else
          mass_step<false, false>(ts + (c & 1) * 128, w * 64, sh.nlse[c & 7], nullptr, kf, c0, cols, add, free);
        // Steps are added with the rounding's rest carried along: a key's rows may be millions.
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x[4];
          unpair(add[e][0], x[0], x[1]);
          unpair(add[e][1], x[2], x[3]);
          const float y = ((x[0] + x[1]) + (x[2] + x[3])) - low[e], s = sum[e] + y;
          low[e] = (s - sum[e]) - y;
          sum[e] = s;
        }
      }
      if (!ok) break;
      float(&other)[2][128] = sh.sums.other[ic & 3];
      if ((ic & 1) != (unsigned)w) {
        other[0][key] = sum[0];
        other[1][key] = sum[1];
        mbar_arrive_warp(&sh.sums.full[ic & 3], lane);
      } else {
        ok = __all_sync(FULL, wait(&sh.sums.full[ic & 3], (ic >> 2) & 1));
        if (!ok) break;
        // The first half of the columns first: the order does not depend on who adds.
        const float x[2] = {w ? other[0][key] + sum[0] : sum[0] + other[0][key], w ? other[1][key] + sum[1] : sum[1] + other[1][key]};
        ok = mass_leave(L, a, list, k, j0, j1, n, sh.page[ic % kMeta], key, x, &sh.sums.last[w], meet);
      }
      ++ic;
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 13) tmem_dealloc(tmem, 512);
  if (tid == 0 && sh.dead) paged_error(L, ERR_PAGED_WAIT, (int32_t)blockIdx.x, sh.dead - 1, (int32_t)MK_ETIMEOUT);
}

// ---- the weights of a few queries: up to 256 rows a kv head ----
// A window of a prompt's last queries, or drafted tokens, against long
// contexts: every key is read for a step or two, so HBM bounds it.  The
// queries of a (sequence, kv head) stay in shared memory, and keys go by in a
// ring of copies.  e4m3 keys are multiplied as they are, a query row being the
// sum of three e5m2 numbers each after a power of two (exact but for channels
// below 2^-23 of the row's largest, off by at most 2^-31 of it): no conversion
// of keys that are used once.  32 queries of 6 sequences of 5K to 40K tokens 56 us
// (17 at the copy's rate): copies, and a step's chain of latencies; with two
// parts, which lost channels below 2^-13, and a ring of four tiles 53.
constexpr int kWindowRows = 256;

// TILES: row tiles of a sequence, at most.  With one, the next (sequence, kv
// head)'s queries are loaded while this one's are in use.
template <bool E4M3, int TILES>
struct WindowShared {
  MassList list;
  static constexpr int NU = 2 / TILES, NK = E4M3 ? 3 : 2;
  uint64_t q_full[NU], q_free[NU], s_full[2], s_free[2], k_full[NK], k_free[NK], done;
  __align__(16) float nlse[2][kMassRows], ze[2][kMassRows];  // by row tile of a unit, or by unit
  int page[kMeta][kMassKeys / 16];
  float ks[kMeta][kMassKeys / 16];
  MassSums sums;
  uint32_t tmem;
  volatile int dead;
};

template <bool E4M3, int TILES>
__global__ void __launch_bounds__(kMassThreads, 1)
    k_window_mass(PagedLayer L, MassArgs a, const __grid_constant__ CUtensorMap kmap) {
  using Sh = WindowShared<E4M3, TILES>;
  constexpr int NU = Sh::NU, NK = Sh::NK, kItem = E4M3 ? kMassTile : 2 * kMassTile, kSide = kMassTile / 2;
  constexpr int kQTile = E4M3 ? 3 * kSide : kMassTile;  // queries of a row tile: three 8-bit parts, or two halves of the channels
  static_assert(1024 + 2 * kQTile + NK * kItem <= kMassSmem, "shared memory");
  extern __shared__ unsigned char dyn[];
  __shared__ Sh sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
  const uint32_t sq = base, sk = base + 2 * kQTile;
  const int G = L.G, g_log2 = __ffs(G) - 1, n_kv = L.n_kv;

  if (tid == 0) {
    for (int i = 0; i < NU; ++i) {
      mbar_init(&sh.q_full[i], 4);
      mbar_init(&sh.q_free[i], 9);  // the products' end and the eight summing warps
    }
    for (int i = 0; i < NK; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_free[i], 8);
    }
    mass_sums_init(sh.sums);
    mbar_init(&sh.done, 1);
    sh.dead = 0;
  }
  mbar_init_fence();
  pdl_wait();
  pdl_trigger();
  if (__syncthreads_or(tid == 0 && paged_stopped(L))) return;
  if (!mass_list(L, a, sh.list)) return;
  const MassList& list = sh.list;
  if (warp == 13) tmem_alloc(&sh.tmem, 512);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tmem = sh.tmem;

  auto slow = [&](uint64_t* bar, unsigned parity, int times) {
    for (int i = 0; i < times; ++i) {
      if (sh.dead) return false;
      if (paged_wait(bar, parity)) return true;
    }
    sh.dead = 1 + warp;
    return false;
  };
  auto wait = [&](uint64_t* bar, unsigned parity) { return mbar_try_wait(bar, parity) || slow(bar, parity, 1); };
  // For a wait that a unit's items can lie between.
  auto wait_long = [&](uint64_t* bar, unsigned parity) { return mbar_try_wait(bar, parity) || slow(bar, parity, list.patience); };
  // Every role goes through the same items; `u` counts the units (sequence, kv
  // head), -1 before the first.
  auto enters = [](const MassCursor& k, int& seq, int& head) {
    const bool is = k.seq != seq || k.head != head;
    seq = k.seq;
    head = k.head;
    return is;
  };
  int j0, j1, seq = -1, head = -1, u = -1;

  if (warp == 13) {
    // ---- issues the products ----
    if (elect_one()) {
      unsigned c = 0, ic = 0;
      bool ok = true;
      for (MassCursor k = list.start; ok && k.rel < list.span; list.next(k)) {
        list.steps(k, j0, j1);
        if (j0 >= j1) continue;
        if (enters(k, seq, head)) {
          if (u >= 0) umma_commit(&sh.q_free[u % NU]);
          ++u;
          ok = wait(&sh.q_full[u % NU], (u / NU) & 1);
        }
        const int skip = list.skip_of(k.seq, k.kt);
        ok = ok && wait(&sh.k_full[ic % NK], (ic / NK) & 1);
        const uint64_t dk = sw128_desc(sk + (ic % NK) * kItem, 16);
        for (int j = j0; ok && j < j1; ++j, ++c) {
          const uint64_t dq = sw128_desc(sq + (TILES == 2 ? skip + j : u % NU) * kQTile, 16);
          ok = c < 2 || wait(&sh.s_free[c & 1], ((c >> 1) - 1) & 1);
          if (!ok) break;
          tmem_fence_after_sync();
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t d = tmem + w * 256 + (c & 1) * 128;
            const uint64_t da = dk + (uint64_t)((w * (kItem / 2)) >> 4);
            if (E4M3) {
#pragma unroll
              for (int i = 0; i < 12; ++i) umma8(d, da + (i & 3) * 2, dq + (i >> 2) * (kSide >> 4) + (i & 3) * 2, idesc8(0, 1), i > 0);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint32_t o = ((i >> 2) * kSide + (i & 3) * 32) >> 4;
                umma_ss(d, da + o, dq + o, idesc(1, 0), i > 0);
              }
            }
          }
          umma_commit(&sh.s_full[c & 1]);
        }
        if (ok) umma_commit(&sh.k_free[ic % NK]);
        ++ic;
      }
      umma_commit(&sh.done);
    }
    // Nothing is in flight when the tensor memory is freed.
    __syncwarp();
    (void)paged_wait_warp(&sh.done, 0);
  } else if (warp == 12) {
    // ---- keys: copies, their pages and scales a step ahead ----
    unsigned ic = 0;
    bool ok = true;
    const int box = !E4M3 || L.P < 32 ? 16 : 32, boxes = kMassKeys / box;
    // Lane g < 16: the page and scale of the item's 16-key group g; -1 where there is none.
    int pg = -1;
    float ks = 1.0f;
    auto fetch = [&](const MassCursor& k) {
      const int tok = k.kt * kMassKeys + lane * 16;
      pg = -1;
      ks = 1.0f;
      if (k.rel < list.span && lane < 16 && tok < list.len[k.seq]) {
        pg = a.b.page_table[(int64_t)k.seq * a.b.table_stride + (tok >> L.p_log2)];
        if (pg < 0 || pg >= L.n_pages) {
          paged_error(L, ERR_PAGED_PAGE, k.seq, pg);
          pg = -1;
        }
        if (E4M3 && pg >= 0) ks = L.k_scale[(int64_t)pg * n_kv + k.head];
      }
    };
    MassCursor k = list.start;
    auto skip_empty = [&]() {  // to the next item with steps in this run
      for (; k.rel < list.span; list.next(k)) {
        list.steps(k, j0, j1);
        if (j0 < j1) return;
      }
    };
    skip_empty();
    fetch(k);
    while (ok && k.rel < list.span) {
      ok = ic < NK || __all_sync(FULL, wait_long(&sh.k_free[ic % NK], (ic / NK - 1) & 1));
      if (!ok) break;
      if (lane < 16) {
        sh.page[ic % kMeta][lane] = pg;
        sh.ks[ic % kMeta][lane] = ks;
      }
      // Lane b < boxes copies `box` keys.
      const int first = __shfl_sync(FULL, pg, (lane * box / 16) & 15);
      const bool in = lane < boxes && first >= 0;
      const unsigned n = __popc(__ballot_sync(FULL, in));
      uint64_t* bar = &sh.k_full[ic % NK];
      if (lane == 0) mbar_expect_tx(bar, n * box * D * (E4M3 ? 1 : 2));
      __syncwarp();
      if (in) {
        const int key = lane * box, y = k.head * L.P + ((k.kt * kMassKeys + key) & (L.P - 1)), z = a.layer_page0 + first;
        const uint32_t to = sk + (ic % NK) * kItem + (key >> 7) * (kItem / 2) + (key & 127) * 128;
        tma3(to, &kmap, 0, y, z, bar);
        if (!E4M3) tma3(to + kSide, &kmap, 64, y, z, bar);
      }
      ++ic;
      list.next(k);
      skip_empty();
      fetch(k);
    }
    for (unsigned i = ic < NK ? 0 : ic - NK; i < ic; ++i) (void)paged_wait_warp(&sh.k_full[i % NK], (i / NK) & 1);
  } else if (warp >= 8) {
    // ---- queries of a unit, 16 lanes a row ----
    const int ck = lane & 15, n_q = n_kv * G;
    bool ok = true;
    for (MassCursor k = list.start; ok && k.rel < list.span; list.next(k)) {
      list.steps(k, j0, j1);
      if (j0 >= j1 || !enters(k, seq, head)) continue;
      ++u;
      ok = u < NU || __all_sync(FULL, wait_long(&sh.q_free[u % NU], (u / NU - 1) & 1));
      if (!ok) break;
      const int64_t row0 = list.row0[k.seq];
      const int rows = list.n_new[k.seq] * G, tiles = list.tiles_of(k.seq);
      for (int t = 0; t < tiles; ++t) {
        const int at = TILES == 2 ? t : u % NU;
        const uint32_t to = sq + at * kQTile;
#pragma unroll 1
        for (int i0 = 0; i0 < 16; i0 += 8) {  // eight rows' loads in flight
          uint4 v[8];
          float ls[8];
          auto row_of = [&](int i) { return (i0 + i) * 8 + (warp & 3) * 2 + (lane >> 4); };
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int x = t * kMassRows + row_of(i);
            const int64_t tok = row0 + (x >> g_log2);
            const int h = k.head * G + (x & (G - 1));
            v[i] = make_uint4(0, 0, 0, 0);
            ls[i] = -INFINITY;
            if (x < rows) {
              v[i] = *reinterpret_cast<const uint4*>(a.q + tok * a.q_stride + h * D + ck * 8);
              if (ck == 0) ls[i] = a.lse[tok * n_q + h];
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = row_of(i);
            ls[i] = __shfl_sync(FULL, ls[i], lane & 16);
            if (ls[i] == -INFINITY) v[i] = make_uint4(0, 0, 0, 0);  // a row without a sum, whatever it holds
            if (E4M3) {
              uint32_t part[3][2];
              const float scale = split8(v[i], lane, part);
              const uint32_t o = to + r * 128 + (((ck >> 1) ^ (r & 7)) << 4) + (ck & 1) * 8;
#pragma unroll
              for (int p = 0; p < 3; ++p)
                asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(o + p * kSide), "r"(part[p][0]), "r"(part[p][1]) : "memory");
              if (ck == 0) sh.ze[at][r] = scale;
            } else {
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to + (ck >> 3) * kSide + r * 128 + (((ck & 7) ^ (r & 7)) << 4)),
                           "r"(v[i].x), "r"(v[i].y), "r"(v[i].z), "r"(v[i].w)
                           : "memory");
            }
            if (ck == 0) sh.nlse[at][r] = ls[i] == -INFINITY ? -INFINITY : -ls[i] * kLog2e;
          }
        }
      }
      fence_proxy_async();
      mbar_arrive_warp(&sh.q_full[u % NU], lane);
    }
  } else {
    // ---- sums: two keys a thread, half of the columns ----
    const int w = warp >> 2, key = tid & 127;
    const uint32_t ts = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + w * 64;
    unsigned c = 0, ic = 0, meets = 0;
    bool ok = true;
    auto meet = [&]() {  // the four warps of this half
      mbar_arrive_warp(&sh.sums.met[w], lane);
      const unsigned parity = meets++ & 1;
      return __all_sync(FULL, wait(&sh.sums.met[w], parity)) != 0;
    };
    for (MassCursor k = list.start; ok && k.rel < list.span; list.next(k)) {
      const int n = list.steps(k, j0, j1);
      if (j0 >= j1) continue;
      if (enters(k, seq, head)) {
        if (u >= 0) mbar_arrive_warp(&sh.q_free[u % NU], lane);
        ++u;
      }
      const int len = list.len[k.seq], n_new = list.n_new[k.seq], t = k.kt * kMassKeys + key, skip = list.skip_of(k.seq, k.kt);
      // Rows left of the sequence from the step's first one on, and the first of them that sees each key.
      int64_t left = (int64_t)n_new * G - (int64_t)(skip + j0) * kMassRows, from[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        from[e] = (a.causal ? max((int64_t)0, (int64_t)t + 128 * e - (len - n_new)) * G : 0) - (int64_t)(skip + j0) * kMassRows;
      float sum[2] = {0.0f, 0.0f}, low[2] = {0.0f, 0.0f};
      for (int j = j0; j < j1; ++j, ++c, left -= kMassRows, from[0] -= kMassRows, from[1] -= kMassRows) {
        ok = __all_sync(FULL, wait(&sh.s_full[c & 1], (c >> 1) & 1));
        if (!ok) break;
        tmem_fence_after_sync();
        const float kf[2] = {E4M3 ? a.scale * sh.ks[ic % kMeta][key >> 4] : a.scale, E4M3 ? a.scale * sh.ks[ic % kMeta][8 + (key >> 4)] : a.scale};
        const int cols = (int)min(left, (int64_t)kMassRows);
        const int c0[2] = {(int)min(max(from[0], (int64_t)0), (int64_t)kMassRows), (int)min(max(from[1], (int64_t)0), (int64_t)kMassRows)};
        uint64_t add[2][2] = {{0, 0}, {0, 0}};
        auto free = [&]() {
          tmem_fence_before_sync();
          mbar_arrive_warp(&sh.s_free[c & 1], lane);
        };
        if (cols < kMassRows || __any_sync(FULL, c0[1] > 0))
          mass_step<true, E4M3>(ts + (c & 1) * 128, w * 64, sh.nlse[TILES == 2 ? skip + j : u % NU], sh.ze[TILES == 2 ? skip + j : u % NU], kf, c0, cols, add, free);
        else
          mass_step<false, E4M3>(ts + (c & 1) * 128, w * 64, sh.nlse[TILES == 2 ? skip + j : u % NU], sh.ze[TILES == 2 ? skip + j : u % NU], kf, c0, cols, add, free);
        // Steps are added with the rounding's rest carried along: a key's rows may be millions.
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x[4];
          unpair(add[e][0], x[0], x[1]);
          unpair(add[e][1], x[2], x[3]);
          const float y = ((x[0] + x[1]) + (x[2] + x[3])) - low[e], s = sum[e] + y;
          low[e] = (s - sum[e]) - y;
          sum[e] = s;
        }
      }
      if (!ok) break;
      float(&other)[2][128] = sh.sums.other[ic & 3];
      if ((ic & 1) != (unsigned)w) {
        other[0][key] = sum[0];
        other[1][key] = sum[1];
        mbar_arrive_warp(&sh.sums.full[ic & 3], lane);
      } else {
        ok = __all_sync(FULL, wait(&sh.sums.full[ic & 3], (ic >> 2) & 1));
        if (!ok) break;
        // The first half of the columns first: the order does not depend on who adds.
        const float x[2] = {w ? other[0][key] + sum[0] : sum[0] + other[0][key], w ? other[1][key] + sum[1] : sum[1] + other[1][key]};
        ok = mass_leave(L, a, list, k, j0, j1, n, sh.page[ic % kMeta], key, x, &sh.sums.last[w], meet);
      }
      ++ic;
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 13) tmem_dealloc(tmem, 512);
  if (tid == 0 && sh.dead) paged_error(L, ERR_PAGED_WAIT, (int32_t)blockIdx.x, sh.dead - 1, (int32_t)MK_ETIMEOUT);
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

cudaError_t launch_paged_prefill_mass(const PagedLayer& L, const PagedMaps& maps, const PagedScratch& w, int layer,
                                      const mk_paged_batch& b, bool causal, const uint16_t* q, int64_t q_stride,
                                      float scale, const float* lse, float* mass, int32_t first, bool add,
                                      cudaStream_t s) {
  const MassArgs a{b, q, q_stride, lse, mass, scale * kLog2e, causal ? 1 : 0, first, add ? 1 : 0, layer * L.n_pages, w.mass_part, w.prefill_counters};
  const int64_t rows = (int64_t)b.max_new * L.G;
  if (rows <= kWindowRows) {
    const bool two = rows > kMassRows;
    auto fn = L.e4m3 ? (two ? k_window_mass<true, 2> : k_window_mass<true, 1>) : (two ? k_window_mass<false, 2> : k_window_mass<false, 1>);
    int sms = 0;
    const cudaError_t e = kernel_smem_attr((const void*)fn, kMassSmem, kMassThreads, nullptr, &sms);
    if (e != cudaSuccess) return e;
    const int grid = sms > 0 && sms <= kPagedMaxCtas ? sms : 128;
    return launch_pdl(fn, dim3(grid), dim3(kMassThreads), (size_t)kMassSmem, s, 0, L, a, maps.k);
  }
  auto fn = L.e4m3 ? k_prefill_mass<true> : k_prefill_mass<false>;
  int sms = 0;
  const cudaError_t e = kernel_smem_attr((const void*)fn, kMassSmem, kMassThreads, nullptr, &sms);
  if (e != cudaSuccess) return e;
  const int grid = sms > 0 && sms <= kPagedMaxCtas ? sms : 128;
  // Queries as {channels, heads, tokens}; a box is 64 channels of the 128 rows
  // (token, head of the group) of a step.
  const TensorMapEncoder enc = tensor_map_encoder();
  CUtensorMap qmap;
  const cuuint64_t dim[3] = {(cuuint64_t)D, (cuuint64_t)L.n_kv * L.G, (cuuint64_t)b.n_tokens};
  const cuuint64_t stride[2] = {(cuuint64_t)D * 2, (cuuint64_t)q_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)L.G, (cuuint32_t)(kMassRows / L.G)}, one[3] = {1, 1, 1};
  if (!enc || enc(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(q), dim, stride, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return launch_pdl(fn, dim3(grid), dim3(kMassThreads), (size_t)kMassSmem, s, 0,
                    L, a, maps.k, qmap);
}

}  // namespace mk
