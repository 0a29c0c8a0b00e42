// Eviction from the paged cache by attention mass: every kv head of a sequence
// keeps its first, its last and its heaviest tokens, moved to the front.
//
// Selection.  The k heaviest of the n tokens between are those above the k-th
// largest mass, and of those equal to it the lowest numbers.  The k-th largest
// is found digit by digit (11, 11 and 10 bits of an order-preserving key) from
// histograms in shared memory; a cluster of CTAs takes a (sequence, kv head),
// each a slice of its tokens, whose keys stay in shared memory between the
// passes (up to kCache of them; a longer slice is read again, from L2).  The
// kept tokens' numbers are then written in order: a warp has a run of the
// slice, counts it, learns what lies before it, and writes.
//
// Move.  In place: kept token number r goes from its slot s(r) >= r to slot r.
// An item is 64 slots of a (sequence, kv head): its CTA reads the rows that go
// there into registers, then says so, then waits until whoever takes tokens out
// of these 64 slots has read them, and writes.  Tokens from 64 neighbouring
// slots go to at most two items, both no later than this one, and items are
// handed out in order by a counter, so whoever is waited for has begun and
// reads without waiting: every wait ends.
//
// What bounds it: HBM for many sequences (24 in bf16 47 to 51 us from box to box,
// its bytes 49 at the rate of a plain copy, some of them from L2), chains of dependent steps for one (64K tokens in e4m3
// 44 us, its bytes 10).  About half of these is the selection: loads 7 us, three
// passes of histogram and cluster barriers 3-4 each, the writing of the numbers
// 4.  An item of the move waits for a ticket, its tokens' numbers, their pages,
// the rows and whoever reads here, 9 us in all; everything that depends on
// nothing is asked for together (one lookup after the other 52 and 56 us).  The
// next ticket drawn an item ahead is slower (58 against 52): items that others
// wait for begin later.
#include <cooperative_groups.h>

#include <algorithm>
#include <utility>

#include "mk_paged.cuh"

namespace cg = cooperative_groups;

namespace mk {

namespace {

constexpr int kSelThreads = 512;
constexpr int kCache = 22 * 1024;  // keys of a slice that stay in shared memory: two CTAs an SM
constexpr int kBins = 2048;
constexpr int kGroup = 64;         // slots of a move item
constexpr int kMoveThreads = 256;

struct EvictArgs {
  mk_paged_batch b;
  float* mass;           // the layer's
  const int32_t* keep;
  int32_t* kept;
  int32_t* new_len;
  int32_t first, recent, kept_stride;
  int32_t* ticket;       // items handed out
  int2* plan;            // [max_seqs] length and tokens kept; x < 0: nothing to move
  int32_t* rank0;        // [n_pages][n_kv], at a group's first page: kept tokens before the group
  // [n_pages][n_kv]: an item's rows are read, at the page of the last slot that
  // it fills.  Of an item that moves anything this page is written, so no other
  // sequence has it; the first one may be of a shared prefix.
  int32_t* flag;
};

// Larger key: larger mass.  -0 is 0; NaN is the least.
__device__ __forceinline__ uint32_t mass_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int page_of(const PagedLayer& L, const mk_paged_batch& b, int seq, int tok) {
  const int p = b.page_table[(int64_t)seq * b.table_stride + (tok >> L.p_log2)];
  if (p >= 0 && p < L.n_pages) return p;
  paged_error(L, ERR_PAGED_PAGE, seq, p);
  return -1;
}

template <int CL>
__global__ void __launch_bounds__(kSelThreads, 2) k_evict_select(PagedLayer L, EvictArgs a) {
  extern __shared__ uint32_t cache[];  // [kCache]
  __shared__ uint32_t hist[kBins], sums[CL > 1 ? kBins : 1];
  __shared__ int s_warp[kSelThreads / 32][2], s_tot[2], s_pick[2], s_scan[kSelThreads / 32];
  constexpr int kWarps = kSelThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CL > 1 ? (int)(blockIdx.x % CL) : 0;
  const int unit = (int)(blockIdx.x / CL), seq = unit / L.n_kv, head = unit % L.n_kv;
  pdl_wait();
  pdl_trigger();
  // Every CTA of a cluster sees the same word (no kernel of the handle runs
  // beside this one), unless one of this call sets it: that one does not stop.
  if (__syncthreads_or(tid == 0 && paged_stopped(L))) return;
  if (blockIdx.x == 0 && tid == 0) *a.ticket = 0;

  const int len = a.b.kv_len[seq], keep = a.keep[seq];
  const bool len_ok = len >= 0 && len <= (int64_t)a.b.table_stride * L.P;
  const bool cut = len_ok && keep >= 0 && len > keep;
  const bool ok = len_ok && keep >= 0 && min(len, keep) <= a.kept_stride && (!cut || keep - a.first >= a.recent);
  if (head == 0 && rank == 0 && tid == 0) {
    if (!ok) paged_error(L, ERR_PAGED_BATCH, seq, len_ok ? keep : len);
    a.new_len[seq] = ok ? min(len, keep) : len;
    a.plan[seq] = make_int2(ok && cut ? len : -1, keep);
  }
  if (!ok) return;
  int32_t* kept = a.kept + ((int64_t)seq * L.n_kv + head) * a.kept_stride;
  // Token numbers are below 2^31 - 256; a step past them need not be.
  if (!cut) {
    for (int64_t t = rank * kSelThreads + tid; t < len; t += CL * kSelThreads) kept[t] = (int)t;
    return;
  }
  for (int64_t t = (rank * kSelThreads + tid) * kGroup; t < keep; t += CL * kSelThreads * kGroup) {
    const int p = page_of(L, a.b, seq, (int)min(t + kGroup, (int64_t)keep) - 1);
    if (p >= 0) a.flag[(int64_t)p * L.n_kv + head] = 0;
  }
  // Tokens lo .. hi - 1 are chosen from, k of them stay; this CTA has t0 .. t1 - 1.
  const int lo = a.first, hi = len - a.recent, k = keep - a.first - a.recent;
  const int per = (hi - lo + CL - 1) / CL;
  const int t0 = lo + min(hi - lo, rank * per), t1 = lo + (int)min((int64_t)(hi - lo), (int64_t)(rank + 1) * per), n = t1 - t0;
  auto load_key = [&](int i) {
    const int t = t0 + i, p = page_of(L, a.b, seq, t);
    return p < 0 ? 0u : mass_key(a.mass[((int64_t)p * L.n_kv + head) * L.P + (t & (L.P - 1))]);
  };
  auto key_of = [&](int i) { return i < kCache ? cache[i] : load_key(i); };
  const int held = min(n, kCache);
  const int32_t* const table = a.b.page_table + (int64_t)seq * a.b.table_stride;
  for (int i0 = tid; i0 < held; i0 += 8 * kSelThreads) {  // eight tokens at a time: the loads' latency
    int page[8];
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = i0 + e * kSelThreads;
      page[e] = i < held ? table[(t0 + i) >> L.p_log2] : 0;
    }
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int t = t0 + i0 + e * kSelThreads;
      const bool there = page[e] >= 0 && page[e] < L.n_pages;
      bad |= !there;
      w[e] = there && i0 + e * kSelThreads < held ? a.mass[((int64_t)page[e] * L.n_kv + head) * L.P + (t & (L.P - 1))] : __int_as_float(0x7fffffff);
    }
    if (bad)
      for (int e = 0; e < 8; ++e)
        if (i0 + e * kSelThreads < held) (void)page_of(L, a.b, seq, t0 + i0 + e * kSelThreads);  // records it
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = i0 + e * kSelThreads;
      if (i < held) cache[i] = mass_key(w[e]);
    }
  }

  // The k-th largest key, digit by digit: those above `prefix` are kept, of
  // the ones that begin with it `left`.
  uint32_t prefix = 0;
  int left = k, shift = 21;
  if (k > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass == 2 ? 10 : 11, bins = 1 << bits;
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      auto count = [&](uint32_t key) {
        if (pass == 0 || (key ^ prefix) >> (shift + bits) == 0) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1u);
      };
#pragma unroll 8
      for (int i = tid; i < held; i += kSelThreads) count(cache[i]);
      for (int i = tid + (held - tid + kSelThreads - 1) / kSelThreads * kSelThreads; held < n && i < n; i += kSelThreads) count(load_key(i));
      if (CL == 1) __syncthreads();
      if (CL > 1) {
        // Each CTA adds up a share of the bins and hands the sums to all.
        auto cluster = cg::this_cluster();
        cluster.sync();
        constexpr int kShare = kBins / CL;
        for (int i = tid; i < kShare; i += kSelThreads) {
          const int bin = rank * kShare + i;
          uint32_t x = 0;
#pragma unroll
          for (int r = 0; r < CL; ++r) x += *cluster.map_shared_rank(&hist[bin], r);
#pragma unroll
          for (int r = 0; r < CL; ++r) *cluster.map_shared_rank(&sums[bin], r) = x;
        }
        cluster.sync();
      }
      // From the top down, four bins a thread: b = bins - 1 - 4 tid - i.
      int c[4], mine = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int bin = bins - 1 - 4 * tid - i;
        c[i] = bin >= 0 ? (int)(CL > 1 ? sums[bin] : hist[bin]) : 0;
        mine += c[i];
      }
      const int ex = warp_excl_scan(mine, lane);
      if (lane == 31) s_scan[warp] = ex + mine;
      __syncthreads();
      int before = ex;
      for (int w = 0; w < warp; ++w) before += s_scan[w];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (before < left && left <= before + c[i]) {
          s_pick[0] = bins - 1 - 4 * tid - i;
          s_pick[1] = left - before;
        }
        before += c[i];
      }
      __syncthreads();
      prefix |= (uint32_t)s_pick[0] << shift;
      left = s_pick[1];
      shift -= pass == 0 ? 11 : 10;
      __syncthreads();
    }
  } else {
    __syncthreads();
  }
  // k = 0: nothing is above the largest key, and none of its equals stays.
  const uint32_t bar = k > 0 ? prefix : 0xffffffffu;

  // Kept tokens in order: warp w has run [w0, w1) of the slice.
  const int run = ((n + kWarps - 1) / kWarps + 31) & ~31, w0 = min(n, warp * run), w1 = min(n, w0 + run);
  int above = 0, equal = 0;
  {
    const int w2 = min(w1, held);
    auto count = [&](uint32_t key) {
      above += key > bar;
      equal += key == bar;
    };
#pragma unroll 4
    for (int i = w0 + lane; i < w2; i += 32) count(cache[i]);
    for (int i = max(w0, w2) + lane; i < w1; i += 32) count(load_key(i));
  }
  above = __reduce_add_sync(FULL, above);
  equal = __reduce_add_sync(FULL, equal);
  if (lane == 0) {
    s_warp[warp][0] = above;
    s_warp[warp][1] = equal;
  }
  __syncthreads();
  if (warp < 2) {
    const int x = __reduce_add_sync(FULL, lane < kWarps ? s_warp[lane][warp] : 0);
    if (lane == 0) s_tot[warp] = x;
  }
  __syncthreads();
  int a0 = 0, e0 = 0;  // above and equal before this warp's run
  cg::cluster_group::arrival_token read;
  if (CL > 1) {
    cg::this_cluster().sync();
    if (lane < rank) {
      a0 = *cg::this_cluster().map_shared_rank(&s_tot[0], lane);
      e0 = *cg::this_cluster().map_shared_rank(&s_tot[1], lane);
    }
    a0 = __reduce_add_sync(FULL, a0);
    e0 = __reduce_add_sync(FULL, e0);
    read = cg::this_cluster().barrier_arrive();
  }
  for (int w = 0; w < warp; ++w) {
    a0 += s_warp[w][0];
    e0 += s_warp[w][1];
  }
  const int stay_eq = k > 0 ? left : 0;
  int at = lo + a0 + min(e0, stay_eq);
  // What lies before each group of slots: 32 groups at a time, a lane each, for
  // their pages' latency.
  int n_groups = 0, group_tok = 0, group_rank = 0;
  auto leave = [&]() {
    if (lane < n_groups && group_tok < keep) {
      const int p = page_of(L, a.b, seq, group_tok);
      if (p >= 0) a.rank0[(int64_t)p * L.n_kv + head] = group_rank;
    }
    n_groups = 0;
  };
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < w1 ? key_of(i) : 0u;
    const unsigned eq = __ballot_sync(FULL, i < w1 && key == bar), below = (1u << lane) - 1u;
    const bool in = i < w1 && (key > bar || (key == bar && e0 + __popc(eq & below) < stay_eq));
    const unsigned ins = __ballot_sync(FULL, in);
    const int r = at + __popc(ins & below), t = t0 + i;
    if (in) kept[r] = t;
    const int x = -(t0 + i0) & (kGroup - 1);  // the lane with a group's first token
    if (x < 32 && i0 + x < w1) {
      const int v = __shfl_sync(FULL, r, x);
      if (lane == n_groups) {
        group_tok = t0 + i0 + x;
        group_rank = v;
      }
      if (++n_groups == 32) leave();
    }
    at += __popc(ins);
    e0 += __popc(eq);
  }
  leave();
  // The tokens that are kept anyway.
  for (int64_t t = rank * kSelThreads + tid; t < lo; t += CL * kSelThreads) kept[t] = (int)t;
  for (int64_t i = rank * kSelThreads + tid; i < a.recent; i += CL * kSelThreads) kept[lo + k + i] = (int)(hi + i);
  if (CL > 1) cg::this_cluster().barrier_wait(std::move(read));  // no CTA ends before its shared memory has been read
}

// Eight e4m3 codes as floats times s (a power of two or any scale).
__device__ __forceinline__ void codes_to(uint32_t lo, uint32_t hi, float s, float (&y)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t h = e4m3_h2((e < 2 ? lo : hi) >> (16 * (e & 1)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    y[2 * e] = f.x * s;
    y[2 * e + 1] = f.y * s;
  }
}

template <bool E4M3>
__global__ void __launch_bounds__(kMoveThreads, 4) k_evict_move(PagedLayer L, EvictArgs a) {
  constexpr int kChunks = E4M3 ? 8 : 16;                       // 16 bytes of a row
  constexpr int kRowsPass = kMoveThreads / kChunks, kPass = kGroup / kRowsPass;
  __shared__ int64_t s_end[MK_MAX_CALL_SEQS];                  // items up to and with a sequence
  __shared__ int64_t s_wsum[kMoveThreads / 32];
  __shared__ int64_t s_at[kGroup];                             // where a row comes from
  __shared__ int s_tok[kGroup], s_page[kGroup / 16], s_item;   // and its token, the pages that rows go to
  __shared__ float s_scale[2][kGroup], s_max[2][kGroup / 4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_kv = L.n_kv, n_seqs = a.b.n_seqs;
  pdl_wait();
  pdl_trigger();
  if (__syncthreads_or(tid == 0 && paged_stopped(L))) return;
  int64_t total = 0;
  {
    const int2 p = tid < n_seqs ? a.plan[tid] : make_int2(-1, 0);
    const int64_t mine = p.x < 0 ? 0 : (int64_t)((p.y + kGroup - 1) / kGroup) * n_kv;
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(FULL, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_wsum[warp] = x;
    __syncthreads();
    for (int w = 0; w < kMoveThreads / 32; ++w) {
      if (w < warp) x += s_wsum[w];
      total += s_wsum[w];
    }
    s_end[tid] = x;
  }
  static_assert(kMoveThreads >= MK_MAX_CALL_SEQS, "one thread a sequence");
  for (;;) {
    __syncthreads();  // the previous item's shared memory is free
    if (tid == 0) {
      const int mine = atomicAdd(a.ticket, 1);
      const int32_t status = *reinterpret_cast<volatile int32_t*>(L.err);
      s_item = status == (int32_t)MK_ETIMEOUT ? 0x7fffffff : mine;  // after a wait that ran out nothing is left to do
    }
    __syncthreads();
    const int64_t item = s_item;
    if (item >= total) return;
    int seq = 0, hi = n_seqs - 1;
    while (seq < hi) {
      const int mid = (seq + hi) >> 1;
      if (s_end[mid] > item) hi = mid; else seq = mid + 1;
    }
    const int2 plan = a.plan[seq];
    const int len = plan.x, keep = plan.y;
    const int64_t in = item - (seq ? s_end[seq - 1] : 0);
    const int j = (int)(in / n_kv), head = (int)(in % n_kv);
    const int r0 = j * kGroup, cnt = min(kGroup, keep - r0);
    const int32_t* kept = a.kept + ((int64_t)seq * n_kv + head) * a.kept_stride;
    if (tid < cnt) s_tok[tid] = kept[r0 + tid];
    if (tid >= kMoveThreads - kGroup / 16) {
      const int i = tid - (kMoveThreads - kGroup / 16), slot = r0 + i * L.P;
      if (i * L.P < cnt) s_page[i] = a.b.page_table[(int64_t)seq * a.b.table_stride + (slot >> L.p_log2)];
    }
    __syncthreads();
    if (s_tok[cnt - 1] == r0 + cnt - 1) continue;  // all stay: nothing else reads or writes here
    // ---- read ----
    auto held_at = [&](int x) {  // the row of slot x of the group: its page and place, or -1
      const int t = s_tok[x];
      const int p = t >= 0 && t < len ? page_of(L, a.b, seq, t) : -1;
      return p < 0 ? (int64_t)-1 : ((int64_t)p * n_kv + head) * L.P + (t & (L.P - 1));
    };
    auto page_to = [&](int x) {  // the page of the group that row x goes to, or -1
      const int p = s_page[x >> L.p_log2];
      if (p >= 0 && p < L.n_pages) return p;
      paged_error(L, ERR_PAGED_PAGE, seq, p);
      return -1;
    };
    if (tid < kGroup) s_at[tid] = tid < cnt ? held_at(tid) : -1;
    __syncthreads();
    float w = 0.0f, scale[2] = {1.0f, 1.0f};
    if (tid < cnt) {
      const int64_t at = s_at[tid];
      w = at < 0 ? 0.0f : a.mass[at];
      if (E4M3 && at >= 0) {
        scale[0] = L.k_scale[at >> L.p_log2];
        scale[1] = L.v_scale[at >> L.p_log2];
      }
    }
    uint4 x[2][kPass];
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
      const int row = i * kRowsPass + tid / kChunks;
      const int64_t at = s_at[row];
#pragma unroll
      for (int t = 0; t < 2; ++t)
        x[t][i] = at < 0 ? make_uint4(0, 0, 0, 0)
                         : *reinterpret_cast<const uint4*>((t ? L.v : L.k) + at * (D * (E4M3 ? 1 : 2)) + (tid % kChunks) * 16);
    }
    if (E4M3 && tid < cnt) {
      s_scale[0][tid] = scale[0];
      s_scale[1][tid] = scale[1];
    }
    const int my_page = page_to(cnt - 1);
    const int64_t here = (int64_t)my_page * n_kv + head;
    const int32_t* from = nullptr;  // the flag of an item that reads here
    int g = 0;
    if (warp == 0) {
      // Ranks of the kept tokens that come from slots r0 .. r0 + 63.
      auto rank_of = [&](int t) {  // kept tokens before token t (a group's first); -1: its page is bad, nothing is waited for
        if (t <= a.first) return t;
        if (t >= len) return keep;
        if (t >= len - a.recent) return keep - (len - t);
        const int p = page_of(L, a.b, seq, t);
        return p < 0 ? -1 : a.rank0[(int64_t)p * n_kv + head];
      };
      const int b0 = rank_of(r0);
      int b1 = r0 + kGroup < keep ? rank_of(r0 + kGroup) : min(keep, b0 + kGroup);
      b1 = min(b1, b0 + kGroup);
      g = b0 / kGroup + lane;  // at most two items, none later than this one
      if (lane < 2 && b0 >= 0 && b1 > b0 && g <= (b1 - 1) / kGroup && g < j) {
        const int p = page_of(L, a.b, seq, g * kGroup + kGroup - 1);  // an earlier item is full
        if (p >= 0) from = a.flag + (int64_t)p * n_kv + head;
      }
    }
    // ---- say so, and wait for those who read here ----
    __threadfence();
    __syncthreads();
    if (tid == 0 && my_page >= 0) {
      asm volatile("st.release.gpu.global.s32 [%0], 1;" ::"l"(a.flag + here) : "memory");
    }
    bool late = false;
    if (from) {
      const long long t0 = clock64();
      int32_t done = 0;
      do {
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(done) : "l"(from) : "memory");
      } while (!done && clock64() - t0 < 400000000ll);
      late = !done;
      if (late) paged_error(L, ERR_PAGED_WAIT, seq, g, (int32_t)MK_ETIMEOUT);
    }
    if (E4M3) {  // largest value of every four rows
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < kPass; ++i) {
          const int row = i * kRowsPass + tid / kChunks;
          // The largest code, as fp16 (exact; NaN counts as nothing), times the scale.
          __half2 most = __float2half2_rn(0.0f);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t w = e < 2 ? x[t][i].x : e < 4 ? x[t][i].y : e < 6 ? x[t][i].z : x[t][i].w;
            const uint32_t h = e4m3_h2(w >> (16 * (e & 1)));
            most = __hmax2(most, __habs2(*reinterpret_cast<const __half2*>(&h)));
          }
          const float2 m = __half22float2(most);
          const float top = warp_max(fminf(fmaxf(m.x, m.y) * (row < cnt ? s_scale[t][row] : 0.0f), 3.402823466e38f));
          if (lane == 0) s_max[t][(i * kRowsPass) / 4 + warp] = top;
        }
    }
    if (__syncthreads_or(late)) return;  // whoever reads here may not have read yet: its rows stay
    // ---- write ----
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
      const int row = i * kRowsPass + tid / kChunks;
      const int p0 = row & ~(L.P - 1), last = min(cnt, p0 + L.P) - 1;  // the row's page in the group
      if (row >= cnt || s_tok[last] == r0 + last) continue;            // a page whose tokens all stay
      const int page = page_to(row);
      if (page < 0) continue;
      const int64_t at = ((int64_t)page * n_kv + head) * L.P + (row & (L.P - 1));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint4 o = x[t][i];
        if (E4M3) {
          float top = 0.0f;
          for (int g = p0 >> 2; g < (p0 + L.P) >> 2; ++g) top = fmaxf(top, s_max[t][g]);
          const float scale = scale_of(top), s = s_scale[t][row];
          if (s != scale) {  // the codes of the same scale stay
            const float inv = __frcp_rn(scale);
            float y[8];
            codes_to(o.x, o.y, s, y);
            uint2 c = pack_e4m3(y, inv);
            o.x = c.x;
            o.y = c.y;
            codes_to(o.z, o.w, s, y);
            c = pack_e4m3(y, inv);
            o.z = c.x;
            o.w = c.y;
          }
          if (row == p0 && tid % kChunks == 0) (t ? L.v_scale : L.k_scale)[at >> L.p_log2] = scale;
        }
        *reinterpret_cast<uint4*>((t ? L.v : L.k) + at * (D * (E4M3 ? 1 : 2)) + (tid % kChunks) * 16) = o;
      }
    }
    if (tid < cnt) {
      const int last = min(cnt, (tid & ~(L.P - 1)) + L.P) - 1;
      const int page = s_tok[last] != r0 + last ? page_to(tid) : -1;
      if (page >= 0) a.mass[((int64_t)page * n_kv + head) * L.P + (tid & (L.P - 1))] = w;
    }
  }
}

template <int CL>
cudaError_t launch_select(const PagedLayer& L, const EvictArgs& a, cudaStream_t s) {
  const cudaError_t e = kernel_smem_attr((const void*)k_evict_select<CL>, kCache * 4, kSelThreads, nullptr, nullptr);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_evict_select<CL>, dim3((unsigned)(a.b.n_seqs * L.n_kv * CL)), dim3(kSelThreads), kCache * 4, s,
                    CL > 1 ? CL : 0, L, a);
}

}  // namespace

cudaError_t launch_paged_evict(const PagedLayer& L, const PagedEvictScratch& w, const mk_paged_batch& b, float* mass,
                               const int32_t* keep, int32_t first, int32_t recent, int32_t* kept, int32_t kept_stride,
                               int32_t* new_len, cudaStream_t s) {
  const EvictArgs a{b, mass, keep, kept, new_len, first, recent, kept_stride, w.ticket, reinterpret_cast<int2*>(w.plan), w.rank0, w.flag};
  const int64_t units = (int64_t)b.n_seqs * L.n_kv;
  // CTAs of a (sequence, kv head): as many as fill the GPU (two an SM), where
  // a sequence may be long enough to be worth cutting.
  const int64_t longest = (int64_t)b.table_stride * L.P;
  const int64_t want = longest <= 2048 ? 1 : longest <= 8192 ? 4 : 8;
  int occ = 0, sms = 0;
  const void* fn = L.e4m3 ? (const void*)k_evict_move<true> : (const void*)k_evict_move<false>;
  cudaError_t e = kernel_smem_attr(fn, 0, kMoveThreads, &occ, &sms);
  if (e != cudaSuccess) return e;
  const int64_t room = 2 * (int64_t)(sms > 0 ? sms : 128);
  if (want >= 8 && units * 8 <= room)
    e = launch_select<8>(L, a, s);
  else if (want >= 4 && units * 4 <= room)
    e = launch_select<4>(L, a, s);
  else if (want >= 2 && units * 2 <= room)
    e = launch_select<2>(L, a, s);
  else
    e = launch_select<1>(L, a, s);
  if (e != cudaSuccess) return e;
  int64_t grid = (int64_t)(sms > 0 ? sms : 128) * (occ > 0 ? occ : 1);
  const int64_t items = units * ((std::min<int64_t>(kept_stride, longest) + kGroup - 1) / kGroup);
  if (items == 0) return cudaSuccess;
  if (grid > items) grid = items;
  return launch_pdl(L.e4m3 ? k_evict_move<true> : k_evict_move<false>, dim3((unsigned)grid), dim3(kMoveThreads), 0, s, 0, L, a);
}

}  // namespace mk
