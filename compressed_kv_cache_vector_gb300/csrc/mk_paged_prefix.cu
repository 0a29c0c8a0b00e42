// Attention of a batch's query rows over the pages that a group of its
// sequences shares: the shared part of mk_paged_prefix_attn.  Its results are
// parts (reference, sum and weighted values of each row), which k_paged_join
// below joins with those over the sequences' own tokens (kOwn in
// mk_paged_decode.cu).
//
// Mathematics as in mk_paged_decode.cu; every row of a group sees all keys.  A
// weight is 2^(z - r) with r the row's reference, its maximum less kShift; while
// new logits stay within 2^kLazy of it the reference is kept, and the weights
// are formed in one reading of the logits, from which the largest exponent tells
// whether they fit.  Where not, the maximum is raised and they are formed anew.
//
// What bounds it: HBM up to about a hundred rows of a kv head (every page is
// read once for 128 rows), the tensor cores and shared memory's rate beyond.
// 128 rows are one accumulator, so there is one row tile and not two in turn
// (mk_paged_prefill.cu): two groups of four warps take the steps of 128 keys in
// turn instead, each with logits, weights and an accumulator of its own in
// tensor memory, so that one group's products run while the other forms its
// weights; their halves are joined when the cell ends.  A thread has one row:
// its maximum and sum need no exchange.  One CTA per SM:
//  * warps 0-3 and 4-7: softmax of the even and the odd steps;
//  * warps 8-11 (e4m3): value codes to fp16, exact, two tiles;
//  * warp 12 issues the products, warp 13 the copies.
//  * e4m3 keys are multiplied as they are: a query row, after a power of two, is
//    the sum of three e5m2 numbers each, exact but for channels below 2^-23 of
//    the row's largest, which are off by at most 2^-31 of it.  That spares the
//    keys' conversion, which shared memory's rate would pay for (16 KB read and
//    32 KB written a step).
//  * Work split on the device: all (group, 128 rows, kv head) cells' steps of
//    128 keys in a row, cut into equal runs, one a CTA.
//  * Weights are rounded once: to fp16 (e4m3), or to one bf16 number.  Two bf16
//    parts, as the decode kernel has them, would double the value products and
//    want 64 registers more while a step's weights wait for their maximum; one
//    part puts 32 sequences on 64K at 0.0020 of 64 bits where the output's own
//    rounding is 0.0017, as in the attention of several query tokens.
//  * fp16 weights have room for 2^15: 2^7 for the reference and 2^8 for logits
//    that pass it.  2^11 and 2^4 keep more of far tails, but raise the maximum
//    so much more often that 192 sequences on 32K took 207 us in place of 171.
// With queries of two 8-bit parts, not three: keys as rows of the logits (a
// thread a key, weights through shared memory) was the first form, 135 us for
// the shared part of 192 sequences of 32 query heads on 32K tokens of 8 kv heads
// in e4m3, bound by shared memory, against 117; both groups at a half of every
// step 171 us for the whole call against 165 (96 sequences in 7 groups, with
// short cells, 97 against 100).  The third part costs 5 us of the 171 and 3 of
// the 104 that these take now.
//
// The whole call in three kernels (shared, own, joined; alone, cold): 192
// sequences on 32K 122, 39 and 13 us; 32 on 64K in bf16 62, 12 and 22, its shared
// pages (269 MB, 40 us at the measured 6.79 TB/s) read once.
#include "mk_paged_tc.cuh"

namespace mk {

namespace {

constexpr int kRows = 128;                // rows of a cell
constexpr int kKeys = 128;                // keys of a step
constexpr int kTile = kKeys * D * 2;      // 32 KB: a 16-bit tile
constexpr int kHalf = kTile / 2;          // its channels 0-63, then 64-127
constexpr int kThreads = 512;
constexpr int kCellCost = 3;              // a cell's queries and result take as long as this many steps
constexpr int kMinRun = 2;                // shortest run of a CTA, in steps
// Tiles on their way: of keys and of values (e4m3: codes, 16 KB each, besides
// the two tiles of values in fp16).
template <bool E4M3>
struct Ring {
  static constexpr int tile = E4M3 ? kTile / 2 : kTile, keys = E4M3 ? 3 : 2, values = 3;
  static constexpr int queries = E4M3 ? 3 * kHalf : kTile;  // e4m3: three 8-bit parts
  static constexpr int smem = 1024 + queries + (keys + values) * tile + (E4M3 ? 2 * kTile : 0);
};
// Registers of a thread of each four warps; the launch gives 128 each.
template <bool E4M3>
struct Regs {
  static constexpr int softmax = 176, load = 96, issue = 64;
  static_assert(2 * softmax + load + issue == 4 * 128, "register shares");
};

struct PrefixArgs {
  mk_paged_batch b;
  mk_paged_prefix p;
  const uint16_t* q;
  int64_t q_stride;
  float scale;       // |scale| log2 e
  uint32_t q_sign;   // 0x80008000 when the scale is negative
  int32_t layer_page0, check_only;
  float* part;       // [2 kPagedMaxCtas][128] row parts
  float* row_part;   // [n_seqs][n_kv G] row parts
  PagedShared* shared;
};

// One cell of a group in a CTA's run, and a place in the list of cells.
struct Cursor {
  int group, block, head, rel;
};

struct Shared {
  int64_t pre[MK_MAX_CALL_SEQS + 1];  // cost of the groups before each
  int first[MK_MAX_CALL_SEQS], last[MK_MAX_CALL_SEQS], len[MK_MAX_CALL_SEQS], table_row[MK_MAX_CALL_SEQS];
  Cursor start;
  int64_t f0, per;
  int span, bad;
  uint64_t q_full, s_full[2], p_full[2], o_full, met, done;
  uint64_t k_full[3], k_free[3], v_full[3], v_free[3];  // the copies' rings
  uint64_t c_full[2], c_free[2];                        // e4m3: values in fp16
  float ml[2][kRows][2];                                // the two groups' maxima and sums
  // e4m3, per 16 keys of a step, ring of 8 steps: {k scale, log2 v scale}, 1 / v scale
  __align__(16) float2 kb[8][8];
  __align__(16) float inv[8][8];
  uint32_t tmem;
  volatile int dead;
};

// A place in a ring of N tiles and the parity of its phase.
template <int N>
struct Place {
  unsigned slot = 0, phase = 0;
  __device__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

template <bool E4M3>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_prefix(PagedLayer L, PrefixArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  constexpr float kShift = E4M3 ? 7.0f : 0.0f;  // weights times 2^kShift before their rounding
  constexpr float kLazy = 8.0f;                 // how far logits may pass the running maximum
  constexpr int NK = Ring<E4M3>::keys, NV = Ring<E4M3>::values, kSlot = Ring<E4M3>::tile;
  extern __shared__ unsigned char dyn[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
  const uint32_t sq = base, sk = base + Ring<E4M3>::queries, sv = sk + NK * kSlot, sc = sv + NV * kSlot;
  const int G = L.G, g_log2 = __ffs(G) - 1, n_kv = L.n_kv, n_groups = a.p.n_groups, members = kRows / G;

  if (tid == 0) {
    mbar_init(&sh.q_full, E4M3 ? 12 : 8);
    mbar_init(&sh.o_full, 1);
    mbar_init(&sh.met, 8);
    mbar_init(&sh.done, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.c_full[i], 4);
      mbar_init(&sh.c_free[i], 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_free[i], 1);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.v_free[i], E4M3 ? 4 : 1);
    }
    sh.dead = 0;
    sh.bad = 0;
  }
  mbar_init_fence();
  pdl_wait();
  pdl_trigger();
  if (__syncthreads_or(tid == 0 && paged_stopped(L))) return;

  // ---- what each group shares, and the CTA's run of the list of cells ----
  for (int g = tid; g < n_groups; g += kThreads) {
    const int lo = a.p.cu_group[g], hi = a.p.cu_group[g + 1];
    if (lo < 0 || hi < lo || hi > a.b.n_seqs || a.p.prefix_len[g] < 0) {
      paged_error(L, ERR_PAGED_BATCH, g, a.p.prefix_len[g]);
      sh.bad = 1;
    }
  }
  __syncthreads();
  if (a.check_only) return;
  const int groups = sh.bad ? 0 : n_groups;  // nothing is shared when the list is wrong
  auto blocks_of = [&](int g) { return (sh.last[g] - sh.first[g] + members - 1) / members; };
  auto steps_of = [&](int g) { return (sh.len[g] + kKeys - 1) / kKeys; };
  auto cost_of = [&](int g) { return steps_of(g) + kCellCost; };
  for (int g = warp; g < groups; g += kThreads / 32) {
    const int lo = a.p.cu_group[g], hi = a.p.cu_group[g + 1];
    int len = 0x7fffffff, row = 0x7fffffff, held = 0;
    for (int i = lo + lane; i < hi; i += 32) {
      const PagedSeq s = paged_seq(a.b, L.P, i, false);
      if (s.ok && s.n_new == 1 && s.len > 0) {
        len = min(len, s.len);
        row = min(row, i);
        ++held;
      }
    }
    len = __reduce_min_sync(FULL, len);
    row = __reduce_min_sync(FULL, row);
    held = __reduce_add_sync(FULL, held);
    len = held < 2 ? 0 : min(len, a.p.prefix_len[g]) & ~(L.P - 1);
    if (lane == 0) {
      sh.first[g] = lo;
      sh.last[g] = hi;
      sh.len[g] = len;
      sh.table_row[g] = row;
      sh.pre[g] = len ? (int64_t)blocks_of(g) * n_kv * cost_of(g) : 0;
    }
  }
  __syncthreads();
  if (warp == 0) {
    int64_t at = 0;
    for (int g0 = 0; g0 < groups; g0 += 32) {
      const int g = g0 + lane;
      const int64_t mine = g < groups ? sh.pre[g] : 0;
      int64_t x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x += y;
      }
      if (g < groups) sh.pre[g] = at + x - mine;
      at += __shfl_sync(FULL, x, 31);
    }
    if (lane == 0) sh.pre[groups] = at;
  }
  __syncthreads();
  const int64_t total = sh.pre[groups];
  int64_t per = (total + gridDim.x - 1) / gridDim.x;
  if (per < kMinRun) per = kMinRun;
  if (blockIdx.x == 0) {  // for the kernel that joins the parts
    if (tid == 0) a.shared->per = per;
    for (int i = tid; i < a.b.n_seqs; i += kThreads) {
      PagedShared::Seq s{0, 0, 0, 0, 0};
      for (int g = 0; g < groups; ++g)
        if (i >= sh.first[g] && i < sh.last[g] && sh.len[g] > 0) {
          const int at = i - sh.first[g];
          s.place = sh.pre[g] + (int64_t)(at / members) * n_kv * cost_of(g);
          s.len = sh.len[g];
          s.row = at % members * G;
          s.steps = steps_of(g);
          s.cost = cost_of(g);
        }
      a.shared->seq[i] = s;
    }
  }
  const int64_t f0 = (int64_t)blockIdx.x * per;
  if (f0 >= total) return;
  if (tid == 0) {
    int lo = 0, hi = groups - 1;
    while (lo < hi) {  // the last group that begins at or before f0
      const int mid = (lo + hi + 1) >> 1;
      if (sh.pre[mid] <= f0) lo = mid; else hi = mid - 1;
    }
    const int64_t in = f0 - sh.pre[lo];
    const int cost = cost_of(lo), cell = (int)(in / cost);
    sh.start = Cursor{lo, cell / n_kv, cell % n_kv, -(int)(in - (int64_t)cell * cost)};
    sh.f0 = f0;
    sh.per = per;
    sh.span = (int)(total - f0 < per ? total - f0 : per);
  }
  __syncthreads();
  if (warp == 12) tmem_alloc(&sh.tmem, 512);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tmem = sh.tmem;

  auto wait = [&](uint64_t* bar, unsigned parity) {
    if (mbar_try_wait(bar, parity)) return true;
    if (!sh.dead && paged_wait(bar, parity)) return true;
    if (!sh.dead) sh.dead = 1 + warp;
    return false;
  };
  auto next = [&](Cursor& k) {
    k.rel += cost_of(k.group);
    if (++k.head < n_kv) return;
    k.head = 0;
    if (++k.block < blocks_of(k.group)) return;
    k.block = 0;
    do ++k.group;
    while (k.group < groups && sh.len[k.group] == 0);
  };
  // The cell's steps in this run.
  auto steps = [&](const Cursor& k, int& j0, int& j1) {
    j0 = max(0, -k.rel);
    j1 = min(steps_of(k.group), sh.span - k.rel);
    return j0 < j1;
  };
  auto rows_of = [&](const Cursor& k) { return min(members, sh.last[k.group] - sh.first[k.group] - k.block * members) * G; };
  int j0, j1;

  if (warp >= 12) {
    fewer_registers<Regs<E4M3>::issue>();
    if (warp == 12) {
      // ---- issues the products: a step's logits before the values of the one before it ----
      if (elect_one()) {
        unsigned c = 0, ic = 0;  // steps and cells so far
        bool ok = true;
        Place<NK> kp;
        Place<NV> vp;
        unsigned ph = 0;  // bit w: phase of p_full[w]
        const uint64_t dq = sw128_desc(sq, 16);
        for (Cursor k = sh.start; ok && k.rel < sh.span; next(k)) {
          if (!steps(k, j0, j1)) continue;
          const int len = sh.len[k.group];
          ok = wait(&sh.q_full, ic++ & 1);
          for (int j = j0 - 1; ok && j < j1; ++j) {
            if (j + 1 < j1) {
              const unsigned w = (j < j0 ? c : c + 1) & 1;
              ok = wait(&sh.k_full[kp.slot], kp.phase);
              if (!ok) break;
              tmem_fence_after_sync();
              const uint64_t d = sw128_desc(sk + kp.slot * kSlot, 16);
              if (E4M3) {
#pragma unroll
                for (int i = 0; i < 12; ++i)
                  umma8(tmem + w * 128, dq + (i >> 2) * (kHalf >> 4) + (i & 3) * 2, d + (i & 3) * 2, idesc8(1, 0), i > 0);
              } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const uint32_t o = ((i >> 2) * kHalf + (i & 3) * 32) >> 4;
                  umma_ss(tmem + w * 128, dq + o, d + o, idesc(1, 0), i > 0);
                }
              }
              umma_commit(&sh.s_full[w]);
              umma_commit(&sh.k_free[kp.slot]);
              kp.next();
            }
            if (j < j0) continue;
            const unsigned w = c & 1;
            ok = (E4M3 ? wait(&sh.c_full[w], (c >> 1) & 1) : wait(&sh.v_full[vp.slot], vp.phase)) && wait(&sh.p_full[w], (ph >> w) & 1);
            if (!ok) break;
            tmem_fence_after_sync();
            const uint64_t d = sw128_desc(E4M3 ? sc + w * kTile : sv + vp.slot * kSlot, kHalf);
            const int blocks = (len - j * kKeys) / 16;  // whole pages: 16 keys each, none hidden
            const uint32_t o = tmem + 256 + w * 128, p = tmem + w * 128;
            const int more = j >= j0 + 2;  // the group has an accumulator
            if (blocks >= 8) {
#pragma unroll
              for (int i = 0; i < 8; ++i) umma_ts(o, p + i * 8, d + i * (2048 >> 4), idesc(!E4M3, 1), more || i > 0);
            } else {
#pragma unroll 1
              for (int i = 0; i < blocks; ++i) umma_ts(o, p + i * 8, d + i * (2048 >> 4), idesc(!E4M3, 1), more || i > 0);
            }
            ph ^= 1u << w;
            umma_commit(E4M3 ? &sh.c_free[w] : &sh.v_free[vp.slot]);
            vp.next();
            ++c;
            if (j == j1 - 1) umma_commit(&sh.o_full);
          }
        }
        umma_commit(&sh.done);
      }
      // Nothing is in flight when the tensor memory is freed.
      __syncwarp();
      (void)paged_wait_warp(&sh.done, 0);
    } else if (warp == 13) {
      // ---- issues the copies, in the order of the products ----
      Place<NK> kp;
      Place<NV> vp;
      unsigned nk = 0, nv = 0;
      bool ok = true;
      const int box = !E4M3 || L.P < 32 ? 16 : 32, lanes = kKeys / box;
      for (Cursor k = sh.start; ok && k.rel < sh.span; next(k)) {
        if (!steps(k, j0, j1)) continue;
        const int len = sh.len[k.group];
        const int32_t* table = a.b.page_table + (int64_t)sh.table_row[k.group] * a.b.table_stride;
        auto fetch = [&](int j) {
          const int tok = j * kKeys + lane * box;
          return lane < lanes && j < j1 && tok < len ? table[tok >> L.p_log2] : -1;
        };
        auto copy = [&](const CUtensorMap* map, int j, int pg, uint64_t* full, uint64_t* free, bool first, unsigned phase, uint32_t to) {
          ok = ok && (first || __all_sync(FULL, wait(free, phase ^ 1u)));
          if (!ok) return;
          const bool in = lane < lanes && j * kKeys + lane * box < len;
          const int boxes = __popc(__ballot_sync(FULL, in));
          if (lane == 0) mbar_expect_tx(full, boxes * box * D * (E4M3 ? 1 : 2));
          __syncwarp();
          if (in) {
            const int y = k.head * L.P + ((j * kKeys + lane * box) & (L.P - 1)), z = a.layer_page0 + pg;
            tma3(to + lane * box * 128, map, 0, y, z, full);
            if (!E4M3) tma3(to + kHalf + lane * box * 128, map, 64, y, z, full);
          }
        };
        auto checked = [&](int j, int pg) {
          if (lane < lanes && j < j1 && j * kKeys + lane * box < len && (pg < 0 || pg >= L.n_pages)) {
            paged_error(L, ERR_PAGED_PAGE, sh.table_row[k.group], pg);
            return 0;
          }
          return pg;
        };
        int pg = 0, pg_next = checked(j0, fetch(j0)), pg_after = fetch(j0 + 1);  // of steps j, j + 1, j + 2
        for (int j = j0 - 1; ok && j < j1; ++j) {
          if (j + 1 < j1) {
            copy(&kmap, j + 1, pg_next, &sh.k_full[kp.slot], &sh.k_free[kp.slot], nk < NK, kp.phase, sk + kp.slot * kSlot);
            if (ok) kp.next(), ++nk;
          }
          if (j >= j0) {
            copy(&vmap, j, pg, &sh.v_full[vp.slot], &sh.v_free[vp.slot], nv < NV, vp.phase, sv + vp.slot * kSlot);
            if (ok) vp.next(), ++nv;
          }
          pg = pg_next;
          pg_next = checked(j + 2, pg_after);
          pg_after = fetch(j + 3);
        }
      }
      // No copy is in flight when the kernel ends, also after a wait that ran out.
      for (unsigned i = 0; i < NK && i < nk; ++i) {
        const unsigned at = nk - 1 - i;
        (void)paged_wait_warp(&sh.k_full[at % NK], (at / NK) & 1);
      }
      for (unsigned i = 0; i < NV && i < nv; ++i) {
        const unsigned at = nv - 1 - i;
        (void)paged_wait_warp(&sh.v_full[at % NV], (at / NV) & 1);
      }
    }
  } else if (warp >= 8) {
    fewer_registers<Regs<E4M3>::load>();
    if (E4M3) {
      // ---- values to 16 bits ----
      // 16 codes ck of rows r + 16 i: eight neighbouring lanes are four chunks
      // of one half by two rows of different parity, whose stores meet in no bank.
      const int ck = (lane & 3) | (lane >> 1 & 4), r = (lane >> 2 & 1) | (lane >> 3 & 2) | (warp & 3) << 2, lt = tid - 256;
      const uint32_t put = (ck >> 2) * kHalf + r * 128 + ((((2 * ck) & 7) ^ (r & 7)) << 4);
      const uint32_t get = r * 128 + ((ck ^ (r & 7)) << 4);
      unsigned c = 0, ic = 0;
      bool ok = true;
      Place<NV> vp;
      for (Cursor k = sh.start; ok && k.rel < sh.span; next(k)) {
        if (!steps(k, j0, j1)) continue;
        const int len = sh.len[k.group];
        const int32_t* table = a.b.page_table + (int64_t)sh.table_row[k.group] * a.b.table_stride;
        // Threads < 8: the scales of 16 keys of a step.
        float ks = 1.0f, vs = 1.0f;
        auto fetch = [&](int j) {
          const int tok = j * kKeys + lt * 16;
          ks = vs = 1.0f;
          if (lt < 8 && j < j1 && tok < len) {
            const int p = table[tok >> L.p_log2];
            if (p >= 0 && p < L.n_pages) {
              ks = L.k_scale[(int64_t)p * n_kv + k.head];
              vs = L.v_scale[(int64_t)p * n_kv + k.head];
            }
          }
        };
        auto leave = [&](unsigned step) {  // for the softmax of a step, before its logits can be there
          if (lt < 8) {
            sh.kb[step & 7][lt] = make_float2(ks, __log2f(vs));
            sh.inv[step & 7][lt] = __frcp_rn(vs);
          }
        };
        fetch(j0);
        leave(c);
        fetch(j0 + 1);
        leave(c + 1);
        fetch(j0 + 2);
        // The first two steps' scales are there: the products may begin, once
        // those of the cell before have (its phase is complete).
        ok = ic == 0 || __all_sync(FULL, wait(&sh.q_full, (ic - 1) & 1));
        if (!ok) break;
        ++ic;
        mbar_arrive_warp(&sh.q_full, lane);
        for (int j = j0; ok && j < j1; ++j, ++c) {
          ok = __all_sync(FULL, wait(&sh.v_full[vp.slot], vp.phase)) &&
               (c < 2 || __all_sync(FULL, wait(&sh.c_free[c & 1], ((c >> 1) - 1) & 1)));
          if (!ok) break;
          const uint32_t from = sv + vp.slot * kSlot + get, to = sc + (c & 1) * kTile + put;
          uint4 x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(x[i].x), "=r"(x[i].y), "=r"(x[i].z), "=r"(x[i].w)
                         : "r"(from + i * 2048));
          leave(c + 2);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int e = 0; e < 2; ++e)
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"((to + i * 2048) ^ (e * 16)), "r"(e4m3_h2(w[2 * e])),
                           "r"(e4m3_h2(w[2 * e] >> 16)), "r"(e4m3_h2(w[2 * e + 1])), "r"(e4m3_h2(w[2 * e + 1] >> 16))
                           : "memory");
          }
          fence_proxy_async();
          mbar_arrive_warp(&sh.v_free[vp.slot], lane);
          if (lane == 0) mbar_arrive(&sh.c_full[c & 1]);
          vp.next();
          fetch(j + 3);
        }
      }
    }
  } else {
    // ---- softmax: one row a thread, every other step ----
    more_registers<Regs<E4M3>::softmax>();
    const int w = warp >> 2, wrow = (warp & 3) * 32, row = wrow + lane;
    const uint32_t trow = tmem + ((uint32_t)wrow << 16);
    const uint32_t ts = trow + w * 128, to = trow + 256 + w * 128;
    bool ok = true;
    unsigned c = 0, ic = 0, ph = 0;  // steps and cells so far; bit 0: phase of s_full, bit 1: of met
    // What the weights' exponents are taken from: rounded up, so that no weight
    // passes 2^(kShift + kLazy) however large the logits.
    auto less = [](float x) { return __fsub_ru(x, kShift); };
    auto meet = [&]() {  // the eight softmax warps
      mbar_arrive_warp(&sh.met, lane);
      ph ^= 2u;
      return __all_sync(FULL, wait(&sh.met, (~ph >> 1) & 1)) != 0;
    };
    for (Cursor k = sh.start; ok && k.rel < sh.span; next(k)) {
      if (!steps(k, j0, j1)) continue;
      const int rows = rows_of(k), len = sh.len[k.group], seq0 = sh.first[k.group] + k.block * members;
      const bool live = wrow < rows;  // this warp has rows
      float zf = fmaxf(a.scale, kTiny);
      // ---- the cell's queries: 16 lanes a row, eight warps ----
      {
        const int ck = lane & 15;
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const int x = 2 * i + (lane >> 4), r = (warp & 3) * 32 + w * 16 + x;  // this warp writes 16 of the rows
          uint4 q = make_uint4(0, 0, 0, 0);
          if (r < rows) {
            const PagedSeq s = paged_seq(a.b, L.P, seq0 + (r >> g_log2), false);
            if (s.ok && s.n_new == 1 && s.len > 0)
              q = *reinterpret_cast<const uint4*>(a.q + (int64_t)s.row0 * a.q_stride + (k.head * G + (r & (G - 1))) * D + ck * 8);
          }
          const uint32_t h[4] = {q.x ^ a.q_sign, q.y ^ a.q_sign, q.z ^ a.q_sign, q.w ^ a.q_sign};
          if (E4M3) {
            uint32_t part[3][2];
            const float scale = split8(make_uint4(h[0], h[1], h[2], h[3]), lane, part);
            const uint32_t at = sq + r * 128 + (((ck >> 1) ^ (r & 7)) << 4) + (ck & 1) * 8;
#pragma unroll
            for (int p = 0; p < 3; ++p)
              asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(at + p * kHalf), "r"(part[p][0]), "r"(part[p][1]) : "memory");
            if (ck == 0) sh.ml[0][r][0] = scale;
          } else {
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(sq + (ck >> 3) * kHalf + r * 128 + (((ck & 7) ^ (r & 7)) << 4)),
                         "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                         : "memory");
          }
        }
        fence_proxy_async();
        mbar_arrive_warp(&sh.q_full, lane);
        if (E4M3) {
          if (!(ok = meet())) break;
          zf *= sh.ml[0][row][0];
          if (!(ok = meet())) break;  // sh.ml is free again
        }
      }
      float m = -INFINITY, l = 0.0f;
      bool begun = false;
      const unsigned c_end = c + (unsigned)(j1 - j0);
      for (int j = j0 + (int)((c ^ (unsigned)w) & 1u); j < j1; j += 2) {
        const unsigned step = c + (unsigned)(j - j0);
        ok = __all_sync(FULL, wait(&sh.s_full[w], ph & 1));
        ph ^= 1u;
        if (!ok) break;
        tmem_fence_after_sync();
        if (live) {
          const int lim = len - j * kKeys;  // columns from here on are hidden
          const bool cut = lim < kKeys;
          // The scales, all at once: read one by one, each would be waited for.
          float kk[E4M3 ? 8 : 1], kb[E4M3 ? 8 : 1], inv[E4M3 ? 8 : 1];
          if (E4M3) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float4 x = *reinterpret_cast<const float4*>(&sh.kb[step & 7][i]);
              kk[i] = fmaxf(zf * x.x, kTiny);
              kb[i] = x.y;
              kk[i + 1] = fmaxf(zf * x.z, kTiny);
              kb[i + 1] = x.w;
            }
#pragma unroll
            for (int i = 0; i < 8; i += 4) *reinterpret_cast<float4*>(&inv[i]) = *reinterpret_cast<const float4*>(&sh.inv[step & 7][i]);
          }
          uint32_t v[32];
          auto logits = [&](int h) {  // columns 32 h ..
            tmem_ld32_async(ts + h * 32, v);
            tmem_ld_wait(v);
            if (cut) {
              asm volatile("");  // a branch, not 32 selections in every step
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i >= lim - 32 * h) v[i] = 0xff800000u;
            }
          };
          // Weights under the maximum so far, in one reading of the logits: the
          // largest exponent tells whether all fit.  Where not, and in a row's
          // first step, the maximum is raised first.  The weights replace the
          // logits, so they stay in registers until they are right.
          float sum;
          uint32_t p[64];
          bool raise = !begun;
          for (;;) {
            if (__any_sync(FULL, raise)) {
              float mx = -INFINITY;
#pragma unroll 1
              for (int h = 0; h < 4; ++h) {
                logits(h);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                  const uint32_t* z = &v[16 * s];
                  float x = max3(z[0], z[1], z[2]);
                  float y = max3(z[3], z[4], z[5]);
                  x = max3(__float_as_uint(x), z[6], z[7]);
                  y = max3(__float_as_uint(y), z[8], z[9]);
                  x = max3(__float_as_uint(x), z[10], z[11]);
                  y = max3(__float_as_uint(y), z[12], z[13]);
                  x = fmaxf(max3(__float_as_uint(x), z[14], z[15]), y);
                  if (E4M3) {
                    const float2 b = sh.kb[step & 7][2 * h + s];
                    x = fmaf(x, fmaxf(zf * b.x, kTiny), b.y);
                  } else {
                    x *= zf;
                  }
                  mx = fmaxf(mx, x);
                }
              }
              const float mn = raise ? fmaxf(m, mx) : m;
              const float f = m == -INFINITY ? 1.0f : ex2(less(m) - less(mn));  // no weights yet: nothing to bring along
              l *= f;
              m = mn;
              if (begun) {
#pragma unroll 2
                for (int h = 0; h < 8; ++h) {
                  uint32_t x[16];
                  tmem_ld16(to + h * 16, x);
#pragma unroll
                  for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                  tmem_st16(to + h * 16, x);
                }
              }
            }
            // A row whose logits were all -infinity so far: any other is above.
            const float ms = m == -INFINITY ? -1e30f : less(m);
            const uint64_t m2 = pair(-ms, -ms);
            float top0 = -INFINITY, top1 = -INFINITY;
            sum = 0.0f;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              logits(h);
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                const float kf = E4M3 ? kk[2 * h + s] : zf, bb = E4M3 ? kb[2 * h + s] : 0.0f;
                const uint64_t k2 = pair(kf, kf), b2 = pair(bb, bb);
                uint64_t add = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const uint32_t* z = &v[16 * s + 2 * i];
                  float x, y;
                  // The logit is rounded before the maximum is taken off, as it was in the maximum:
                  // one fused step would leave the largest of huge logits above it.
                  unpair(add2(fma2(pair(__uint_as_float(z[0]), __uint_as_float(z[1])), k2, b2), m2), x, y);
                  (i & 1 ? top1 : top0) = max3(__float_as_uint(i & 1 ? top1 : top0), __float_as_uint(x), __float_as_uint(y));
                  x = ex2(x);
                  y = ex2(y);
                  add = add2(add, pair(x, y));
                  p[16 * h + 8 * s + i] = pack2<E4M3>(x, y);
                }
                float x, y;
                unpair(add, x, y);
                sum = E4M3 ? fmaf(x + y, inv[2 * h + s], sum) : sum + (x + y);
              }
            }
            raise = fmaxf(top0, top1) > kShift + kLazy;
            if (!__any_sync(FULL, raise)) break;  // so after a maximum was raised
          }
          l += sum;
#pragma unroll
          for (int h = 0; h < 4; ++h) tmem_st16(ts + h * 16, *reinterpret_cast<const uint32_t(*)[16]>(&p[16 * h]));
          tmem_wait_st();
          tmem_fence_before_sync();
          mbar_arrive_warp(&sh.p_full[w], lane);
        } else {  // no rows here: the weights may be anything
          mbar_arrive_warp(&sh.p_full[w], lane);
        }
        begun = true;
      }
      if (!ok) break;
      c = c_end;
      ok = __all_sync(FULL, wait(&sh.o_full, ic++ & 1));
      if (!ok) break;
      tmem_fence_after_sync();
      // ---- the rows' results, a part: the two groups' joined, half of the channels each ----
      sh.ml[w][row][0] = m;
      sh.ml[w][row][1] = l;
      if (!(ok = meet())) break;
      if (live) {
        const float m0 = sh.ml[0][row][0], m1 = sh.ml[1][row][0], M = fmaxf(m0, m1);
        // The references that the weights were formed with; a group without steps has none.
        const float r0 = less(m0), r1 = less(m1), R = less(M);
        const bool has0 = j1 - j0 > 1 || ((c_end - 1) & 1) == 0, has1 = j1 - j0 > 1 || ((c_end - 1) & 1) == 1;
        const float f0 = r0 == -INFINITY ? 0.0f : ex2(r0 - R), f1 = r1 == -INFINITY ? 0.0f : ex2(r1 - R);
        const bool whole = j1 - j0 == steps_of(k.group);
        float* const part = whole ? a.row_part + ((int64_t)seq0 * n_kv + k.head) * G * kPagedRowPart
                                  : a.part + (2 * (int64_t)blockIdx.x + (j0 == 0 ? 1 : 0)) * kPagedPrefixPart;
        auto row_at = [&](int r) {
          return part + (int64_t)(whole ? (r >> g_log2) * (n_kv * G) + (r & (G - 1)) : r) * kPagedRowPart;
        };
        if (w == 0 && row < rows) {
          float* const at = row_at(row);
          // A sum of NaN, or of a group whose every logit was one, counts as it is.
          const float s0 = sh.ml[0][row][1], s1 = sh.ml[1][row][1];
          at[D] = R;
          at[D + 1] = s0 * (r0 == -INFINITY ? 1.0f : f0) + s1 * (r1 == -INFINITY ? 1.0f : f1);
        }
        // 32 channels at a time, through the warp's 4 KB of the query tile: rows
        // leave 128 bytes at a time.
        const uint32_t stage = sq + warp * 4096;
#pragma unroll 1
        for (int b = 2 * w; b < 2 * w + 2; ++b) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t x[16], y[16];
            tmem_ld16(trow + 256 + b * 32 + h * 16, x);
            tmem_ld16(trow + 384 + b * 32 + h * 16, y);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              x[i] = __float_as_uint((has0 ? __uint_as_float(x[i]) * f0 : 0.0f) + (has1 ? __uint_as_float(y[i]) * f1 : 0.0f));
#pragma unroll
            for (int i = 0; i < 4; ++i)
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(stage + lane * 128 + (((4 * h + i) ^ (lane & 7)) << 4)), "r"(x[4 * i]),
                           "r"(x[4 * i + 1]), "r"(x[4 * i + 2]), "r"(x[4 * i + 3])
                           : "memory");
          }
          __syncwarp();
#pragma unroll 4
          for (int i = 0; i < 8; ++i) {
            const int x = 4 * i + (lane >> 3);
            uint4 o;
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
                         : "r"(stage + x * 128 + (((lane & 7) ^ (x & 7)) << 4)));
            if (wrow + x < rows) *reinterpret_cast<uint4*>(row_at(wrow + x) + b * 32 + (lane & 7) * 4) = o;
          }
          __syncwarp();
        }
      }
      tmem_fence_before_sync();
      ok = meet();  // sh.ml and the accumulators are free again
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 12) tmem_dealloc(tmem, 512);
  if (tid == 0 && sh.dead) paged_error(L, ERR_PAGED_WAIT, (int32_t)blockIdx.x, sh.dead - 1, (int32_t)MK_ETIMEOUT);
}

// ---- joins a row's parts: over shared tokens and over its sequence's own ----
// A warp a row, four channels a lane.
constexpr int kJoinWarps = 4;

struct JoinArgs {
  mk_paged_batch b;
  const PagedShared* shared;
  const float *part, *row_part, *own_part, *own_row;
  const int2* own;
  uint16_t* out;
  float* lse;
  int64_t out_stride;
};

__global__ void __launch_bounds__(kJoinWarps * 32) k_paged_join(PagedLayer L, JoinArgs a) {
  const int lane = threadIdx.x & 31, G = L.G, n_q = L.n_kv * G;
  const int64_t at = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  const int seq = (int)(at / n_q), h = (int)(at % n_q), head = h / G, r = h % G;
  pdl_wait();
  pdl_trigger();
  if (seq >= a.b.n_seqs) return;
  // Everything that depends on nothing is asked for at once: the kernel is a
  // chain of such waits.
  const bool stopped = paged_stopped(L);
  const PagedSeq s = paged_seq(a.b, L.P, seq, false);
  const PagedShared::Seq c = a.shared->seq[seq];
  const int64_t per = a.shared->per;
  const int2 own = a.own[seq * L.n_kv + head];
  if (stopped || !s.ok || s.n_new != 1) return;
  const float *sp = nullptr, *op = nullptr;  // the first part of each kind
  int64_t s_rest = 0, o_rest = 0;            // from it to the second, and the distance of the others
  int ns = 0, no = 0;
  const int64_t s_slot = 2 * (int64_t)kPagedPrefixPart, o_slot = 2 * (int64_t)G * kPagedRowPart;
  int off = 0;
  if (s.len > 0) {
    off = c.len;
    if (off > 0) {
      const int64_t place = c.place + (int64_t)head * c.cost, b_lo = place / per;
      ns = (int)((place + c.steps - 1) / per - b_lo) + 1;
      sp = ns == 1 ? a.row_part + ((int64_t)seq * n_q + h) * kPagedRowPart
                   : a.part + (2 * b_lo + 1) * kPagedPrefixPart + (int64_t)(c.row + r) * kPagedRowPart;
      s_rest = kPagedPrefixPart;
    }
    if (s.len > off) {
      no = own.y;
      op = no == 1 ? a.own_row + ((int64_t)seq * n_q + h) * kPagedRowPart
                   : a.own_part + ((2 * (int64_t)own.x + 1) * G + r) * kPagedRowPart;
      o_rest = (int64_t)G * kPagedRowPart;
    }
  }
  // A run that begins an item has its odd slot, one that goes on with it the even one.
  auto part = [&](int i) {
    if (i < ns) return i == 0 ? sp : sp - s_rest + i * s_slot;
    i -= ns;
    return i == 0 ? op : op - o_rest + i * o_slot;
  };
  const int n = ns + no;
  float M = -INFINITY, S = 0.0f;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, __ldcg(part(i) + D));
  M = warp_max(M);
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i0 = 0; i0 < n; i0 += 32) {
    float mine = 0.0f;
    if (i0 + lane < n) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(part(i0 + lane) + D));
      // A part whose reference is -infinity has no weights, or only NaN: its sum, 0 or NaN, counts as it is.
      mine = ml.x == -INFINITY ? 0.0f : ex2(ml.x - M);
      S += ml.y * (ml.x == -INFINITY ? 1.0f : mine);
    }
    const int m = min(32, n - i0);
#pragma unroll 8
    for (int i = 0; i < m; ++i) {
      const float f = __shfl_sync(FULL, mine, i);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(part(i0 + i)) + lane);
      o.x = fmaf(v.x, f, o.x);
      o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z);
      o.w = fmaf(v.w, f, o.w);
    }
  }
  S = warp_sum(S);
  const bool any = S > 0.0f || S != S;
  const float f = any ? 1.0f / S : 0.0f;
  const uint2 w = make_uint2(pack2<false>(o.x * f, o.y * f), pack2<false>(o.z * f, o.w * f));
  *reinterpret_cast<uint2*>(a.out + (int64_t)s.row0 * a.out_stride + h * D + lane * 4) = w;
  if (a.lse && lane == 0) a.lse[(int64_t)s.row0 * n_q + h] = any ? (log2f(S) + M) * kLn2 : -INFINITY;
}

}  // namespace

cudaError_t launch_paged_join(const PagedLayer& L, const PagedScratch& w, const mk_paged_batch& b, uint16_t* out,
                              int64_t out_stride, float* lse, cudaStream_t s) {
  const JoinArgs a{b, w.shared, w.prefill_part, w.row_part, paged_own_parts(w), w.own_row, reinterpret_cast<const int2*>(w.own),
                   out, lse, out_stride};
  const int64_t rows = (int64_t)b.n_seqs * L.n_kv * L.G;
  return launch_pdl(k_paged_join, dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps)), dim3(kJoinWarps * 32), 0, s, 0, L, a);
}

cudaError_t launch_paged_prefix(const PagedLayer& L, const PagedMaps& maps, const PagedScratch& w, int layer,
                                const mk_paged_batch& b, const mk_paged_prefix& p, const uint16_t* q, int64_t q_stride,
                                float scale, bool check_only, cudaStream_t s) {
  static_assert(kRows * kPagedRowPart == kPagedPrefixPart, "a part's size");
  const void* fn = L.e4m3 ? (const void*)k_paged_prefix<true> : (const void*)k_paged_prefix<false>;
  int sms = 0;
  const int smem = L.e4m3 ? Ring<true>::smem : Ring<false>::smem;
  const cudaError_t e = kernel_smem_attr(fn, smem, kThreads, nullptr, &sms);
  if (e != cudaSuccess) return e;
  const int grid = sms > 0 && sms <= kPagedMaxCtas ? sms : 128;
  const PrefixArgs a{b, p, q, q_stride, (scale < 0.0f ? -scale : scale) * kLog2e, scale < 0.0f ? 0x80008000u : 0u,
                     layer * L.n_pages, check_only ? 1 : 0, w.prefill_part, w.row_part, w.shared};
  return launch_pdl(L.e4m3 ? k_paged_prefix<true> : k_paged_prefix<false>, dim3(check_only ? 1 : grid), dim3(kThreads), (size_t)smem, s, 0, L, a,
                    maps.k, maps.v);
}

}  // namespace mk
