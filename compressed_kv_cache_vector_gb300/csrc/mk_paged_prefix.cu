// Attention of a batch's query rows over the pages that a group of its
// sequences shares: the shared part of mk_paged_prefix_attn.  Its results are
// parts (maximum, sum and weighted values of each row), which the attention of
// the sequences' own tokens joins with its own (mk_paged_decode.cu).
//
// Mathematics as in mk_paged_decode.cu; every row of a group sees all keys.
//
// What bounds it: HBM up to about a hundred rows of a kv head (every page is
// read once for 128 rows), the tensor cores and the exponentials beyond.  The
// rows of a decode step are few and ragged, so the keys take the 128 rows of a
// product and the query rows its columns: S^T = K Q^T and O^T = V^T P with 64
// or 128 columns, no row of the tensor cores empty however few the queries.  A
// thread has one key of a step and one half of the columns:
//  * a row's running maximum is needed only as a bound.  A step first looks
//    whether any logit passes its row's by 2^4 (fp16 weights) or 2^8 (bf16):
//    one comparison a logit and one vote of four warps.  Only then are maxima
//    formed over the threads and the accumulator rescaled.
//  * a row's sum stays in the threads, one number a key and row, until the end.
//  * the weights go to shared memory as the B operand, as they come.
// One CTA per SM:
//  * warps 0-3 and 4-7: softmax of the first and the second half of the columns;
//  * warps 8-11 (e4m3): codes to bf16 (keys) and fp16 (values), both exact;
//  * warp 12 issues the products, warp 13 the copies (a ring of four tiles).
//  * Work split on the device: all (group, 128 rows, kv head) cells' steps of
//    128 keys in a row, cut into equal runs, one a CTA.
#include "mk_paged_tc.cuh"

namespace mk {

namespace {

constexpr int kRows = 128;                // rows of a cell
constexpr int kKeys = 128;                // keys of a step
constexpr int kTile = kKeys * D * 2;      // 32 KB: a 16-bit tile
constexpr int kHalf = kTile / 2;          // its channels 0-63, then 64-127
constexpr int kRaw = kKeys * D;           // 16 KB: a tile of codes
constexpr int kThreads = 512;
constexpr int kCellCost = 3;              // a cell's queries and result take as long as this many steps
constexpr int kMinRun = 2;                // shortest run of a CTA, in steps
constexpr int kSmem = 1024 + 6 * kTile;   // queries, weights, keys and values
// Registers of a thread of each four warps; the launch gives 128 each.
constexpr int kSoftmaxRegs = 168, kLoadRegs = 112, kIssueRegs = 64;
static_assert(2 * kSoftmaxRegs + kLoadRegs + kIssueRegs == 4 * 128, "register shares");
constexpr float kNone = 1e30f;            // stands for a bound that no logit has set yet

struct PrefixArgs {
  mk_paged_batch b;
  mk_paged_prefix p;
  const uint16_t* q;
  int64_t q_stride;
  float scale;       // |scale| log2 e
  uint32_t q_sign;   // 0x80008000 when the scale is negative
  int32_t layer_page0;
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
  uint64_t q_full, s_full[2], s_free[2], p_full[2], pv_done[2], done;
  uint64_t kv_full[4], kv_free[4];          // the ring of copies
  uint64_t k_full, k_free, v_full, v_free;  // e4m3: the tiles formed from it
  uint64_t met[2];
  __align__(16) float nm[kRows];            // shift - bound of each row
  float m[kRows], f[kRows], top[2][4][kRows / 2];
  int vote[2][2][4];
  // e4m3, per 16 keys of a step, ring of 4 steps: {k scale, log2 v scale}, 1 / v scale
  __align__(16) float2 kb[4][8];
  float inv[4][8];
  uint32_t tmem;
  volatile int dead;
};

// D (128 x N, fp32) of A and B of one 16-bit type, each along its rows' own
// direction where the flag is set.
__device__ __forceinline__ uint32_t idesc_of(int bf16, int a_mn, int b_mn, int n) {
  return (1u << 4) | ((uint32_t)bf16 << 7) | ((uint32_t)bf16 << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15])::"memory");
}
// Over the 32 lanes and 16 columns each: lane c < 16 (and 16 + c) gets the
// result of column c.
template <typename Op>
__device__ __forceinline__ float across16(float (&x)[16], int lane, Op op) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = up ? x[i] : x[i + o], keep = up ? x[i + o] : x[i];
      x[i] = op(keep, __shfl_xor_sync(FULL, give, o));
    }
  }
  return op(x[0], __shfl_xor_sync(FULL, x[0], 16));
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_prefix(PagedLayer L, PrefixArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  constexpr float kShift = E4M3 ? 10.0f : 0.0f;  // weights times 2^kShift before their rounding
  constexpr float kLazy = E4M3 ? 4.0f : 8.0f;    // how far logits may pass a row's bound
  extern __shared__ unsigned char dyn[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
  // bf16: a ring of four tiles (K, V, K, V).  e4m3: four tiles of codes, one of keys, one of values.
  const uint32_t sq = base, sp = base + kTile, ring = base + 2 * kTile, sk = ring + 4 * kRaw, sv = sk + kTile;
  constexpr int kSlot = E4M3 ? kRaw : kTile;
  const int G = L.G, g_log2 = __ffs(G) - 1, n_kv = L.n_kv, n_groups = a.p.n_groups, members = kRows / G;

  if (tid == 0) {
    mbar_init(&sh.q_full, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_free[i], 8);
      mbar_init(&sh.p_full[i], 8);
      mbar_init(&sh.pv_done[i], 1);
      mbar_init(&sh.met[i], 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh.kv_full[i], 1);
      mbar_init(&sh.kv_free[i], E4M3 ? 4 : 1);
    }
    mbar_init(&sh.k_full, 4);
    mbar_init(&sh.v_full, 4);
    mbar_init(&sh.k_free, 1);
    mbar_init(&sh.v_free, 1);
    mbar_init(&sh.done, 1);
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
    fewer_registers<kIssueRegs>();
    if (warp == 12) {
      // ---- issues the products ----
      if (elect_one()) {
        unsigned c = 0, ic = 0;
        bool ok = true;
        const uint64_t dq = sw128_desc(sq, 16);
        for (Cursor k = sh.start; ok && k.rel < sh.span; next(k)) {
          if (!steps(k, j0, j1)) continue;
          const int n = rows_of(k) <= 64 ? 64 : 128, len = sh.len[k.group];
          const uint32_t id_s = idesc_of(1, 0, 0, n), id_o = idesc_of(!E4M3, 1, 1, n);
          ok = wait(&sh.q_full, ic++ & 1);
          for (int j = j0 - 1; ok && j < j1; ++j) {
            if (j + 1 < j1) {  // the next step's logits
              const unsigned s = j < j0 ? c : c + 1, slot = (2 * s) & 3;
              ok = wait(E4M3 ? &sh.k_full : &sh.kv_full[slot], E4M3 ? s & 1 : (s >> 1) & 1) &&
                   (s < 2 || wait(&sh.s_free[s & 1], ((s >> 1) - 1) & 1));
              if (!ok) break;
              tmem_fence_after_sync();
              const uint64_t d = sw128_desc(E4M3 ? sk : ring + slot * kSlot, 16);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint32_t o = ((i >> 2) * kHalf + (i & 3) * 32) >> 4;
                umma_ss(tmem + (s & 1) * 128, d + o, dq + o, id_s, i > 0);
              }
              umma_commit(&sh.s_full[s & 1]);
              umma_commit(E4M3 ? &sh.k_free : &sh.kv_free[slot]);
            }
            if (j < j0) continue;
            const unsigned slot = (2 * c + 1) & 3;
            ok = wait(E4M3 ? &sh.v_full : &sh.kv_full[slot], E4M3 ? c & 1 : (c >> 1) & 1) && wait(&sh.p_full[c & 1], (c >> 1) & 1);
            if (!ok) break;
            tmem_fence_after_sync();
            const uint64_t dv = sw128_desc(E4M3 ? sv : ring + slot * kSlot, kHalf);
            const uint64_t dp = sw128_desc(sp + (n == 64 ? (c & 1) * kHalf : 0), kHalf);
            const int blocks = min(8, (len - j * kKeys) / 16);  // whole pages: 16 keys each, none hidden
#pragma unroll 1
            for (int i = 0; i < blocks; ++i)
              umma_ss(tmem + 256, dv + i * (2048 >> 4), dp + i * (2048 >> 4), id_o, j > j0 || i > 0);
            umma_commit(&sh.pv_done[c & 1]);
            umma_commit(E4M3 ? &sh.v_free : &sh.kv_free[slot]);
            ++c;
          }
        }
        umma_commit(&sh.done);
      }
      // Nothing is in flight when the tensor memory is freed.
      __syncwarp();
      (void)paged_wait_warp(&sh.done, 0);
    } else if (warp == 13) {
      // ---- issues the copies: keys, then values of each step ----
      unsigned c = 0;  // tiles so far
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
        int pg_next = fetch(j0);
        for (int j = j0; ok && j < j1; ++j) {
          int pg = pg_next;
          pg_next = fetch(j + 1);
          const bool in = lane < lanes && j * kKeys + lane * box < len;
          if (in && (pg < 0 || pg >= L.n_pages)) {
            paged_error(L, ERR_PAGED_PAGE, sh.table_row[k.group], pg);
            pg = 0;
          }
          const int boxes = __popc(__ballot_sync(FULL, in));
          const int y = k.head * L.P + ((j * kKeys + lane * box) & (L.P - 1)), z = a.layer_page0 + pg;
#pragma unroll
          for (int t = 0; t < 2; ++t, ++c) {
            ok = ok && (c < 4 || __all_sync(FULL, wait(&sh.kv_free[c & 3], ((c >> 2) - 1) & 1)));
            if (!ok) break;
            uint64_t* bar = &sh.kv_full[c & 3];
            if (lane == 0) mbar_expect_tx(bar, boxes * box * D * (E4M3 ? 1 : 2));
            __syncwarp();
            if (in) {
              const uint32_t to = ring + (c & 3) * kSlot + lane * box * 128;
              const CUtensorMap* map = t ? &vmap : &kmap;
              tma3(to, map, 0, y, z, bar);
              if (!E4M3) tma3(to + kHalf, map, 64, y, z, bar);
            }
          }
        }
      }
      // No copy is in flight when the kernel ends, also after a wait that ran out.
      for (unsigned i = c < 4 ? 0 : c - 4; i < c; ++i) (void)paged_wait_warp(&sh.kv_full[i & 3], (i >> 2) & 1);
    }
  } else if (warp >= 8) {
    fewer_registers<kLoadRegs>();
    if (E4M3) {
      // ---- codes to 16 bits ----
      // 16 codes ck of rows r + 16 i: eight neighbouring lanes are four chunks
      // of one half by two rows of different parity, whose stores meet in no bank.
      const int ck = (lane & 3) | (lane >> 1 & 4), r = (lane >> 2 & 1) | (lane >> 3 & 2) | (warp & 3) << 2, lt = tid - 256;
      const uint32_t put = (ck >> 2) * kHalf + r * 128 + ((((2 * ck) & 7) ^ (r & 7)) << 4);
      const uint32_t get = r * 128 + ((ck ^ (r & 7)) << 4);
      unsigned c = 0;
      bool ok = true;
      for (Cursor k = sh.start; ok && k.rel < sh.span; next(k)) {
        if (!steps(k, j0, j1)) continue;
        const int len = sh.len[k.group];
        const int32_t* table = a.b.page_table + (int64_t)sh.table_row[k.group] * a.b.table_stride;
        // Threads < 8: the scales of 16 keys of a step, fetched a step ahead.
        float ks = 1.0f, vs = 1.0f;
        auto scales = [&](int j) {
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
        scales(j0);
        for (int j = j0; ok && j < j1; ++j, ++c) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const unsigned tile = 2 * c + t, slot = tile & 3;
            ok = ok && __all_sync(FULL, wait(&sh.kv_full[slot], (tile >> 2) & 1)) &&
                 (c == 0 || __all_sync(FULL, wait(t ? &sh.v_free : &sh.k_free, (c - 1) & 1)));
            if (!ok) break;
            const uint32_t from = ring + slot * kSlot + get, to = (t ? sv : sk) + put;
            uint4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                           : "=r"(x[i].x), "=r"(x[i].y), "=r"(x[i].z), "=r"(x[i].w)
                           : "r"(from + i * 2048));
            if (t == 0 && lt < 8) {
              sh.kb[c & 3][lt] = make_float2(ks, __log2f(vs));
              sh.inv[c & 3][lt] = __frcp_rn(vs);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
              uint32_t o[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                o[e] = e4m3_h2(w[e >> 1] >> (16 * (e & 1)));
                if (t == 0) {
                  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&o[e]));
                  o[e] = pack2<false>(f.x, f.y);
                }
              }
              const uint32_t at = to + i * 2048;
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]) : "memory");
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at ^ 16), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]) : "memory");
            }
            fence_proxy_async();
            mbar_arrive_warp(&sh.kv_free[slot], lane);
            if (lane == 0) mbar_arrive(t ? &sh.v_full : &sh.k_full);
            if (t == 0) scales(j + 1);
          }
        }
      }
    }
  } else {
    // ---- softmax: one key a thread, half of the columns ----
    more_registers<kSoftmaxRegs>();
    const int w = warp >> 2, key = tid & 127;
    const uint32_t tlane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    unsigned c = 0, meets = 0;
    bool ok = true;
    auto meet = [&]() {  // the four warps of this half
      mbar_arrive_warp(&sh.met[w], lane);
      const unsigned parity = meets++ & 1;
      return __all_sync(FULL, wait(&sh.met[w], parity)) != 0;
    };
    for (Cursor k = sh.start; ok && k.rel < sh.span; next(k)) {
      if (!steps(k, j0, j1)) continue;
      const int rows = rows_of(k), len = sh.len[k.group];
      // Columns of each half, in groups of 16.
      const int ng = rows <= 32 ? 1 : rows <= 64 ? 2 : 4, cw = ng * 16, col0 = w * cw;
      const bool two = rows <= 64;  // two buffers of weights
      // ---- the cell's queries: 16 lanes a row ----
      {
        const int ck = tid & 15, seq0 = sh.first[k.group] + k.block * members;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = 16 * i + (tid >> 4);
          uint4 x = make_uint4(0, 0, 0, 0);
          if (row < rows) {
            const PagedSeq s = paged_seq(a.b, L.P, seq0 + (row >> g_log2), false);
            if (s.ok && s.n_new == 1 && s.len > 0)
              x = *reinterpret_cast<const uint4*>(a.q + (int64_t)s.row0 * a.q_stride + (k.head * G + (row & (G - 1))) * D + ck * 8);
          }
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(sq + (ck >> 3) * kHalf + row * 128 + (((ck & 7) ^ (row & 7)) << 4)),
                       "r"(x.x ^ a.q_sign), "r"(x.y ^ a.q_sign), "r"(x.z ^ a.q_sign), "r"(x.w ^ a.q_sign)
                       : "memory");
        }
        if (key < cw) {
          sh.m[col0 + key] = -INFINITY;
          sh.nm[col0 + key] = kNone;
        }
        fence_proxy_async();
        mbar_arrive_warp(&sh.q_full, lane);
        ok = meet();  // the rows' bounds are set
      }
      uint64_t l[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) l[i] = 0;
      for (int j = j0; ok && j < j1; ++j, ++c) {
        const bool cut = len - j * kKeys < kKeys, in = j * kKeys + key < len;
        ok = __all_sync(FULL, wait(&sh.s_full[c & 1], (c >> 1) & 1));
        if (!ok) break;
        tmem_fence_after_sync();
        const uint32_t ts = tlane + (c & 1) * 128 + col0;
        float kf = fmaxf(a.scale, kTiny), lv = 0.0f, inv = 1.0f;
        if (E4M3) {
          const float2 kb = sh.kb[c & 3][key >> 4];
          kf = fmaxf(a.scale * kb.x, kTiny);
          lv = kb.y;
          inv = sh.inv[c & 3][key >> 4];
        }
        const uint64_t k2 = pair(kf, kf), lv2 = pair(lv, lv), inv2 = pair(inv, inv);
        uint32_t v[2][16];
        auto load = [&](int h) {  // columns 16 h .. are in v[h & 1], the next are asked for
          tmem_ld_wait16(v[h & 1]);
          if (h + 1 < ng) tmem_ld16_async(ts + (h + 1) * 16, v[(h + 1) & 1]);
          if (cut) {
            asm volatile("");  // a branch, not 16 selections in every step
            if (!in) {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[h & 1][i] = 0xff800000u;
            }
          }
        };
        auto pair_at = [&](int h, int i) {
          return pair(__uint_as_float(v[h & 1][i]), __uint_as_float(v[h & 1][i + 1]));
        };
        // Does a logit pass its row's bound?  The logit is rounded before the
        // bound is taken off, here as in the maximum and the weights: one
        // fused step would leave the largest of huge logits above its bound.
        float top = -INFINITY;
        tmem_ld16_async(ts, v[0]);
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (h < ng) {
            load(h);
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 nm = *reinterpret_cast<const float4*>(&sh.nm[col0 + 16 * h + i]);
              float x, y;
              unpair(add2(fma2(pair_at(h, i), k2, lv2), pair(nm.x, nm.y)), x, y);
              top = fmaxf(top, fmaxf(x, y));
              unpair(add2(fma2(pair_at(h, i + 2), k2, lv2), pair(nm.z, nm.w)), x, y);
              top = fmaxf(top, fmaxf(x, y));
            }
          }
        const bool over = __any_sync(FULL, top > kShift + kLazy);
        int* vote = sh.vote[w][meets & 1];
        if (lane == 0) vote[warp & 3] = over;
        if (!(ok = meet())) break;
        if (vote[0] | vote[1] | vote[2] | vote[3]) {
          // ---- the rows' maxima over the step's keys; bounds, sums and accumulator follow ----
          tmem_ld16_async(ts, v[0]);
#pragma unroll
          for (int h = 0; h < 4; ++h)
            if (h < ng) {
              load(h);
              float x[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] = fmaf(__uint_as_float(v[h & 1][i]), kf, lv);
              const float y = across16(x, lane, [](float p, float q) { return fmaxf(p, q); });
              if (lane < 16) sh.top[w][warp & 3][16 * h + lane] = y;
            }
          if (!(ok = meet())) break;
          if (key < cw) {
            const float mx = fmaxf(fmaxf(sh.top[w][0][key], sh.top[w][1][key]), fmaxf(sh.top[w][2][key], sh.top[w][3][key]));
            const float m = sh.m[col0 + key];
            const bool raise = mx > m + kLazy || (m == -INFINITY && mx != -INFINITY);
            sh.f[col0 + key] = !raise ? 1.0f : m == -INFINITY ? 0.0f : ex2(m - mx);
            if (raise) {
              sh.m[col0 + key] = mx;
              sh.nm[col0 + key] = __fsub_rd(kShift, mx);  // never above it, however large
            }
          }
          if (!(ok = meet())) break;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (2 * i < cw) {
              float x, y;
              unpair(l[i], x, y);
              l[i] = pair(x * sh.f[col0 + 2 * i], y * sh.f[col0 + 2 * i + 1]);
            }
          if (j > j0) {
            ok = __all_sync(FULL, wait(&sh.pv_done[(c - 1) & 1], ((c - 1) >> 1) & 1));
            if (!ok) break;
            tmem_fence_after_sync();
#pragma unroll 1
            for (int h = 0; h < ng; ++h) {
              uint32_t o[16];
              tmem_ld16(tlane + 256 + col0 + h * 16, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * sh.f[col0 + h * 16 + i]);
              tmem_st16(tlane + 256 + col0 + h * 16, o);
            }
            tmem_wait_st();
          }
        }
        // ---- the weights ----
        const unsigned back = two ? 2 : 1;  // the step whose weights were in this buffer
        if (c >= back) ok = __all_sync(FULL, wait(&sh.pv_done[(c - back) & 1], ((c - back) >> 1) & 1));
        if (!ok) break;
        const uint32_t to = sp + (two ? (c & 1) * kHalf : 0) + key * 128;
        tmem_ld16_async(ts, v[0]);
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (h < ng) {
            load(h);
            if (h == ng - 1) {  // all of S is in registers
              tmem_fence_before_sync();
              mbar_arrive_warp(&sh.s_free[c & 1], lane);
            }
            uint32_t p[8];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 nm = *reinterpret_cast<const float4*>(&sh.nm[col0 + 16 * h + i]);
              float x[4];
              unpair(add2(fma2(pair_at(h, i), k2, lv2), pair(nm.x, nm.y)), x[0], x[1]);
              unpair(add2(fma2(pair_at(h, i + 2), k2, lv2), pair(nm.z, nm.w)), x[2], x[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = ex2(x[e]);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint64_t& s = l[8 * h + i / 2 + e];
                s = E4M3 ? fma2(pair(x[2 * e], x[2 * e + 1]), inv2, s) : add2(s, pair(x[2 * e], x[2 * e + 1]));
                p[i / 2 + e] = pack2<E4M3>(x[2 * e], x[2 * e + 1]);
              }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int chunk = (col0 + 16 * h) / 8 + e;  // 8 columns
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to + (chunk >> 3) * kHalf + (((chunk & 7) ^ (key & 7)) << 4)),
                           "r"(p[4 * e]), "r"(p[4 * e + 1]), "r"(p[4 * e + 2]), "r"(p[4 * e + 3])
                           : "memory");
            }
          }
        tmem_fence_before_sync();
        fence_proxy_async();
        mbar_arrive_warp(&sh.p_full[c & 1], lane);
      }
      if (!ok) break;
      // ---- the rows' results: a part ----
      const bool whole = j1 - j0 == steps_of(k.group);
      const int seq0 = sh.first[k.group] + k.block * members;
      auto row_at = [&](int r) {
        return whole ? a.row_part + ((int64_t)(seq0 + (r >> g_log2)) * n_kv * G + k.head * G + (r & (G - 1))) * kPagedRowPart
                     : a.part + (2 * (int64_t)blockIdx.x + (j0 == 0 ? 1 : 0)) * kPagedPrefixPart + r * kPagedRowPart;
      };
#pragma unroll
      for (int h = 0; h < 4; ++h)
        if (h < ng) {
          float x[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) unpair(l[8 * h + i], x[2 * i], x[2 * i + 1]);
          const float y = across16(x, lane, [](float p, float q) { return p + q; });
          if (lane < 16) sh.top[w][warp & 3][16 * h + lane] = y;
        }
      if (!(ok = meet())) break;
      if (key < cw && col0 + key < rows) {
        float* ml = row_at(col0 + key) + D;
        ml[0] = sh.m[col0 + key] == -INFINITY ? -INFINITY : -sh.nm[col0 + key];
        ml[1] = (sh.top[w][0][key] + sh.top[w][1][key]) + (sh.top[w][2][key] + sh.top[w][3][key]);
      }
      ok = __all_sync(FULL, wait(&sh.pv_done[(c - 1) & 1], ((c - 1) >> 1) & 1));
      if (!ok) break;
      tmem_fence_after_sync();
#pragma unroll 1
      for (int h = 0; h < ng; ++h) {
        uint32_t o[16];
        tmem_ld16(tlane + 256 + col0 + h * 16, o);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (col0 + h * 16 + i < rows) row_at(col0 + h * 16 + i)[key] = __uint_as_float(o[i]);
      }
      tmem_fence_before_sync();
      ok = meet();  // the bounds and sums may be set anew
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 12) tmem_dealloc(tmem, 512);
  if (tid == 0 && sh.dead) paged_error(L, ERR_PAGED_WAIT, (int32_t)blockIdx.x, sh.dead - 1, (int32_t)MK_ETIMEOUT);
}

}  // namespace

cudaError_t launch_paged_prefix(const PagedLayer& L, const PagedMaps& maps, const PagedScratch& w, int layer,
                                const mk_paged_batch& b, const mk_paged_prefix& p, const uint16_t* q, int64_t q_stride,
                                float scale, cudaStream_t s) {
  static_assert(kRows * kPagedRowPart == kPagedPrefixPart, "a part's size");
  const void* fn = L.e4m3 ? (const void*)k_paged_prefix<true> : (const void*)k_paged_prefix<false>;
  int sms = 0;
  const cudaError_t e = kernel_smem_attr(fn, kSmem, kThreads, nullptr, &sms);
  if (e != cudaSuccess) return e;
  const int grid = sms > 0 && sms <= kPagedMaxCtas ? sms : 128;
  const PrefixArgs a{b, p, q, q_stride, (scale < 0.0f ? -scale : scale) * kLog2e, scale < 0.0f ? 0x80008000u : 0u,
                     layer * L.n_pages, w.prefill_part, w.row_part, w.shared};
  return launch_pdl(L.e4m3 ? k_paged_prefix<true> : k_paged_prefix<false>, dim3(grid), dim3(kThreads), (size_t)kSmem, s, 0, L, a,
                    maps.k, maps.v);
}

}  // namespace mk
