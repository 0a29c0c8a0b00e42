// Attention of several query tokens per sequence over the paged cache: prompt
// chunks, verification of drafted tokens, cross attention.
//
// Mathematics as in mk_paged_decode.cu; one row per (query token, query head
// of the kv head's group), so the heads of a group share every key and value
// tile.  A tile of 256 rows is two accumulators of 128 rows.
//
// What bounds it: the tensor cores (4 x 128 flops a pair) and, at the same
// order, the exponentials.  Hence the 5th-generation tensor cores with every
// accumulator in tensor memory, and two row tiles in turn: while one tile's
// weights are formed, the products of the other run.  One CTA per SM:
//  * warps 0-3 and 4-7: the softmax of row tile 0 and 1, one row a thread;
//  * warps 8-11: keys and values into shared memory (e4m3 codes to fp16 on the
//    way, exact; rows past the length as zeros), two stages each;
//  * warps 12 and 14: issue the products, one of them for each row tile.
//    S = Q K^T into tensor memory; the weights replace S there in 16 bits and
//    are the A operand of O += P V.  A tile's products are issued by one lane
//    in order, so that the completion of its S is also that of its previous
//    value product.  Warp 13 lists the work items.
//  * The running maximum is raised only when a row's logits pass it by 2^4
//    (fp16 weights) or 2^8 (bf16): only then is the accumulator rescaled.
//    e4m3: weights in fp16 after a factor 2^10 (at most 2^14, smallest step
//    2^-34 of the maximum's); bf16: weights in bf16, off by up to 2^-8 each.
//    Their sum is of the unrounded ones.  Two bf16 parts, as the decode kernel
//    has them, bring the relative error of ragged chunks against 64 bits from
//    0.0022 to 0.0017 (the output's own rounding) and cost half of the value
//    products again: 8K prompt bf16 512 -> 674 us, ragged chunks 108 -> 129,
//    1K tokens behind 64K 904 -> 1195.
//  * Work split on the device, from the lengths: all row tiles' steps of 128
//    keys in a row, cut into equal runs, one a CTA, so that uneven batches,
//    causal masks and a few rows against a long context load the SMs alike.  A
//    row tile that lies in several runs is joined by the last CTA of it to
//    arrive, in the order of the parts.
// Measured (GB300, 32 query heads over 8): an 8K prompt e4m3 615 us, 895
// TFLOP/s of the visible pairs (47% of cuBLAS's burst), bf16 512; six ragged
// chunks bf16 108 us, 600 TFLOP/s; 16 x 5 tokens against 2K-16K 140 us; cross
// attention of 8 x 40-300 queries 45 us.  Equal runs cost whole prompts some
// 4% (592 us e4m3 in whole items) and halve the few-row cases.  A step of 128 keys for both tiles takes 2.2-2.4
// us where its products alone would take 1.1: the tensor cores are busy 38% of
// the time, XU 19%.  The rest is the latency of the chain products -> logits
// read -> maximum -> exponentials -> weights written -> products, with one
// warp of a role on each scheduler: an empty copy of the loop takes 1.5 us a
// step.  Code size matters as much as instruction counts here: variants with
// the products unrolled to constants were slower (714 us).
#include "mk_paged.cuh"

namespace mk {

namespace {

constexpr int kRows = 256;                 // rows of a work item: two tiles of 128
constexpr int kKeys = 128;                 // keys of a step
constexpr int kTile = kKeys * D * 2;       // 32 KB: a 16-bit tile
constexpr int kHalf = kTile / 2;           // its channels 0-63, then 64-127
constexpr int kThreads = 512;              // 8 softmax warps, 4 loading, 2 issuing, 1 listing (and 1 without work)
// Registers of a thread of each group of four warps; the launch gives 128 each
// (512 x 128 = 65,536), and the shares add up to that.
template <bool E4M3>
struct Regs {
  static constexpr int softmax = E4M3 ? 160 : 168, load = E4M3 ? 128 : 112, issue = 64;
  static_assert(2 * softmax + load + issue == 4 * 128, "register shares");
};
constexpr int kItemCost = 3;               // an item's queries and result take as long as this many steps
constexpr int kItems = 4;                  // items that the list may run ahead of the slowest group
constexpr int kMinRun = 4;                 // shortest run of a CTA, in steps
constexpr int kSmem = 1024 + 2 * kTile + 4 * kTile;
// Logit factors are at least this, so that a hidden key's -infinity stays one
// (a row of zeros or a scale of 0 would make it NaN).
constexpr float kTiny = 1.17549435e-38f;
constexpr float kLn2 = 0.6931471805599453f;

struct PrefillArgs {
  mk_paged_batch b;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t q_stride, out_stride;
  float scale;        // |scale| log2 e
  uint32_t q_sign;    // 0x80008000 when the scale is negative
  int32_t causal;
  float* part;        // [2 x kPagedMaxCtas][128 / 4][kRows] float4, then [..][2][kRows]: see part_of
  int32_t* counters;  // [kPagedMaxCtas]
};

// Descriptor of a 128-byte-swizzled operand: rows of 128 bytes, groups of 8
// rows 1024 bytes apart.  Along the rows' direction (K-major: Q, K) `lbo` has
// no use; for an operand whose rows run along the products' K (V), it is the
// distance between its two 64-channel halves.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr, uint32_t lbo) {
  uint64_t d = (uint64_t)((addr >> 4) & 0x3fffu);
  d |= (uint64_t)((lbo >> 4) & 0x3fffu) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// D (128 x 128, fp32): fp16 (0) or bf16 (1) operands; B along N when b_mn.
__host__ __device__ constexpr uint32_t idesc(int bf16, int b_mn) {
  return (1u << 4) | ((uint32_t)bf16 << 7) | ((uint32_t)bf16 << 10) | ((uint32_t)b_mn << 16) | ((uint32_t)(128 >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, int acc) {
  umma_bf16(d, a, b, id, acc);  // kind::f16; the descriptor names the type
}
// A from tensor memory.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, int acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}
// Values loaded by earlier tmem_ld32_async may be used after this: they pass
// through it so that no use is moved before the wait.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                 "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                 "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])::"memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};\n" ::"r"(
          v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
      : "memory");
}
// Two fp32 operations at once.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// One lane of a converged warp (the tensor-core instructions take their
// operands from uniform registers: a branch that only the lane's number
// decides would make each of them a loop over the lanes).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float max3(uint32_t a, uint32_t b, uint32_t c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return r;
}
template <int R>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// One arrival for a warp whose lanes have all done their part (and fenced it):
// 32 arrivals at one barrier are 32 operations in a row on its word.
__device__ __forceinline__ void mbar_arrive_warp(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void cp_async16_z(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// One work item of a CTA: a row tile of one (sequence, kv head) against its
// keys [j0, j1) x 128 (of n steps in all).
struct Item {
  int seq, head, q0, row0, n_new, len, n, j0, j1;
  int b_lo, parts;  // the CTAs b_lo .. b_lo + parts - 1 have a part of it
  int end;          // 1: no item, the list is at its end
};
// A place in the list of all items: its sequence, row tile (the last queries
// first: with a causal mask they see the most keys), head, and where it begins
// in the CTA's run (negative: in an earlier CTA's).
struct Cursor {
  int seq, tile, head, rel;
};

struct Shared {
  int64_t pre[MK_MAX_CALL_SEQS + 1];   // cost of the sequences before each
  int row0[MK_MAX_CALL_SEQS], n_new[MK_MAX_CALL_SEQS], len[MK_MAX_CALL_SEQS];
  Cursor start;
  int64_t f0, per;                     // the CTA's run: its begin and the length of all runs
  int span;                            // its length
  int patience;                        // limits of a wait that may span several items, in limits of a single one
  Item ring[kItems];                   // items on their way to the groups of warps
  uint64_t item_full[kItems], item_free[kItems], met, done;
  uint64_t q_full[2], s_full[2], p_half[2], p_full[2], o_full[2], k_full[2], k_free[2], v_full[2], v_free[2];
  // e4m3, per 16 keys of a step, ring of 4 steps: {k scale, log2 v scale}, 1 / v scale
  __align__(16) float2 kb[4][8];
  float inv[4][8];
  uint32_t tmem;
  int last;
  volatile int dead;  // 0, or 1 + the warp whose wait ran out: recorded when the kernel ends
};

// The rest of a wait that has not ended at once, up to `times` times its limit.
__device__ __forceinline__ bool wait_slow(uint64_t* bar, unsigned parity, int times, volatile int* dead) {
  for (int i = 0; i < times; ++i) {
    if (*dead) return false;
    if (paged_wait(bar, parity)) return true;
  }
  *dead = 1 + (int)(threadIdx.x >> 5);
  return false;
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) k_paged_prefill(PagedLayer L, PrefillArgs a) {
  constexpr float kShift = E4M3 ? 10.0f : 0.0f;   // weights times 2^kShift before their rounding
  constexpr float kLazy = E4M3 ? 4.0f : 8.0f;     // how far logits may pass the running maximum
  extern __shared__ unsigned char dyn[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
  const uint32_t sq = base, sk = base + 2 * kTile, sv = base + 4 * kTile;
  const int G = L.G, n_kv = L.n_kv, n_seqs = a.b.n_seqs;
  const int q_tile = kRows / G;                    // query tokens of a work item

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 4);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_half[i], 4);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.o_full[i], 1);
      mbar_init(&sh.k_full[i], 4);
      mbar_init(&sh.k_free[i], 2);
      mbar_init(&sh.v_full[i], 4);
      mbar_init(&sh.v_free[i], 2);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&sh.item_full[i], 1);
      mbar_init(&sh.item_free[i], 14);  // one arrival of each softmax, loading and issuing warp
    }
    mbar_init(&sh.met, 8);
    mbar_init(&sh.done, 2);
    sh.dead = 0;
  }
  mbar_init_fence();
  pdl_wait();
  pdl_trigger();
  if (__syncthreads_or(tid == 0 && paged_stopped(L))) return;

  // ---- the CTA's run of the list of work items ----
  // All items in a row, each as long as its steps and kItemCost (its queries
  // and its result), are cut into equal runs, one a CTA: an item may lie in
  // several.  Its step j is at its place plus j.
  auto tiles_of = [&](int seq) { return (sh.n_new[seq] + q_tile - 1) / q_tile; };
  auto steps_of = [&](int seq, int tile) {  // 128-key steps that the tile's last query needs
    const int n_new = sh.n_new[seq], len = sh.len[seq];
    const int q1 = min((tiles_of(seq) - tile) * q_tile, n_new);
    const int see = a.causal ? max(0, min(len, len - n_new + q1)) : len;
    return (see + kKeys - 1) / kKeys;
  };
  for (int i = warp; i < n_seqs; i += kThreads / 32) {
    PagedSeq s = paged_seq(a.b, L.P, i, false);
    if (!s.ok) {
      if (lane == 0) paged_error(L, ERR_PAGED_BATCH, i, s.len);
      s.n_new = 0;
    }
    if (lane == 0) {
      sh.row0[i] = s.row0;
      sh.n_new[i] = s.n_new;
      sh.len[i] = s.len;
    }
    __syncwarp();
    int64_t x = 0;
    for (int t = lane, nt = tiles_of(i); t < nt; t += 32) x += max(steps_of(i, t), 1) + kItemCost;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
    if (lane == 0) sh.pre[i] = x * n_kv;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t base = 0;
    for (int i0 = 0; i0 < n_seqs; i0 += 32) {
      const int i = i0 + lane;
      const int64_t mine = i < n_seqs ? sh.pre[i] : 0;
      int64_t x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x += y;
      }
      if (i < n_seqs) sh.pre[i] = base + x - mine;
      base += __shfl_sync(FULL, x, 31);
    }
    if (lane == 0) sh.pre[n_seqs] = base;
  }
  __syncthreads();
  const int64_t total = sh.pre[n_seqs];
  int64_t per = (total + gridDim.x - 1) / gridDim.x;
  if (per < kMinRun) per = kMinRun;
  const int64_t f0 = (int64_t)blockIdx.x * per;
  if (f0 >= total) return;
  if (tid == 0) {
    sh.f0 = f0;
    sh.per = per;
    sh.span = (int)(total - f0 < per ? total - f0 : per);
    // 1024 steps take 2 to 3 ms, a limit is about 20.
    sh.patience = 100 + sh.span / 1024;
  }
  if (warp == 0) {
    int lo = 0, hi = n_seqs - 1;
    while (lo < hi) {  // the last sequence that begins at or before f0 (one without queries begins where the next does)
      const int mid = (lo + hi + 1) >> 1;
      if (sh.pre[mid] <= f0) lo = mid; else hi = mid - 1;
    }
    int64_t at = sh.pre[lo];
    for (int t0 = 0, nt = tiles_of(lo); t0 < nt; t0 += 32) {
      const int t = t0 + lane;
      const int cost = t < nt ? max(steps_of(lo, t), 1) + kItemCost : 0;
      int64_t x = (int64_t)cost * n_kv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x += y;
      }
      const unsigned past = __ballot_sync(FULL, at + x > f0);
      if (past) {
        if (lane == __ffs(past) - 1) {
          const int64_t begin = at + x - (int64_t)cost * n_kv;
          const int head = (int)((f0 - begin) / cost);
          sh.start = Cursor{lo, t, head, (int)(begin + (int64_t)head * cost - f0)};
        }
        break;
      }
      at += __shfl_sync(FULL, x, 31);
    }
  }
  __syncthreads();
  if (warp == 12) tmem_alloc(&sh.tmem, 512);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tmem = sh.tmem;

  auto wait = [&](uint64_t* bar, unsigned parity) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, 1, &sh.dead);
  };
  // A wait that steps of the run can lie between, as many as it has: for an
  // item, for a slot of the list, and wherever row tile 1's softmax, which has
  // no part in items of one row tile and runs up to kItems of them ahead, meets
  // the others again (a single sequence of 1M keys has 8192 steps an item).
  auto wait_long = [&](uint64_t* bar, unsigned parity) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, sh.patience, &sh.dead);
  };
  // The next item of the list for a group of warps; nullptr at its end.
  auto take = [&](unsigned c) -> const Item* {
    if (!__all_sync(FULL, wait_long(&sh.item_full[c % kItems], (c / kItems) & 1))) return nullptr;
    const Item* it = &sh.ring[c % kItems];
    return it->end ? nullptr : it;
  };
  auto give_back = [&](unsigned c) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.item_free[c % kItems]);
  };

  if (warp >= 12) {
    fewer_registers<Regs<E4M3>::issue>();
    if (warp == 13 && lane == 0) {
      // ---- lists the items ----
      Cursor k = sh.start;
      unsigned c = 0;
      auto put = [&](const Item& it) {
        if (c >= kItems && !wait_long(&sh.item_free[c % kItems], (c / kItems - 1) & 1)) return false;
        sh.ring[c % kItems] = it;
        mbar_arrive(&sh.item_full[c % kItems]);
        ++c;
        return true;
      };
      Item it;
      it.end = 0;
      bool ok = true;
      while (ok && k.rel < sh.span) {
        it.n = steps_of(k.seq, k.tile);
        it.j0 = max(0, -k.rel);
        it.j1 = min(it.n, sh.span - k.rel);
        if (it.n == 0 ? k.rel >= 0 : it.j0 < it.j1) {
          it.seq = k.seq;
          it.head = k.head;
          it.row0 = sh.row0[k.seq];
          it.n_new = sh.n_new[k.seq];
          it.len = sh.len[k.seq];
          it.q0 = (tiles_of(k.seq) - 1 - k.tile) * q_tile;
          const int64_t place = sh.f0 + k.rel;
          it.b_lo = (int)(place / sh.per);
          it.parts = it.n == 0 ? 1 : (int)((place + it.n - 1) / sh.per) - it.b_lo + 1;
          ok = put(it);
        }
        k.rel += max(it.n, 1) + kItemCost;
        if (++k.head == n_kv) {
          k.head = 0;
          if (++k.tile == tiles_of(k.seq)) {
            k.tile = 0;
            do ++k.seq;
            while (k.seq < n_seqs && sh.n_new[k.seq] == 0);
          }
        }
      }
      it.end = 1;
      if (ok) put(it);
    }
    // ---- issue the products: warp 12 those of row tile 0, warp 14 of tile 1 ----
    // One elected lane does it all: between two products every instruction
    // counts, as they run one after the other.
    if (warp == 12 || warp == 14) {
      const int t = warp == 14;
      if (elect_one()) {
        unsigned c = 0, qc = 0, pc = 0;  // steps so far; phases of q_full and of p_half, p_full
        bool ok = true;
        const uint64_t dq = sw128_desc(sq + t * kTile, 16), dk = sw128_desc(sk, 16), dv = sw128_desc(sv, kHalf);
        for (unsigned ic = 0; ok; ++ic) {
          if (!wait_long(&sh.item_full[ic % kItems], (ic / kItems) & 1)) break;
          const Item* it = &sh.ring[ic % kItems];
          if (it->end) break;
          const int n = it->j1 - it->j0;
          const bool alone = min(it->n_new - it->q0, q_tile) * G <= 128;  // the item has no rows in tile 1
          mbar_arrive(&sh.item_free[ic % kItems]);
          if (n == 0) continue;
          if (t == 1 && alone) {  // no products here: the stages are passed on, step by step
            for (int j = 0; j < n && ok; ++j, ++c) {
              ok = wait(&sh.k_full[c & 1], (c >> 1) & 1);
              if (ok) mbar_arrive(&sh.k_free[c & 1]);
              ok = ok && wait(&sh.v_full[c & 1], (c >> 1) & 1);
              if (ok) mbar_arrive(&sh.v_free[c & 1]);
            }
            continue;
          }
          ok = wait(&sh.q_full[t], qc++ & 1);
          for (int j = -1; j < n && ok; ++j) {
            if (j >= 0) {
              // The value product, 64 keys at a time as their weights come.
              const uint64_t d = dv + (uint64_t)((c & 1) * (kTile >> 4));
              ok = wait(&sh.v_full[c & 1], (c >> 1) & 1) && wait(&sh.p_half[t], pc & 1);
              if (!ok) break;
              tmem_fence_after_sync();
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_ts(tmem + 256 + t * 128, tmem + t * 128 + k * 8, d + k * (2048 >> 4), idesc(!E4M3, 1), j > 0 || k > 0);
              ok = wait(&sh.p_full[t], pc++ & 1);
              if (!ok) break;
              tmem_fence_after_sync();
#pragma unroll
              for (int k = 4; k < 8; ++k)
                umma_ts(tmem + 256 + t * 128, tmem + t * 128 + k * 8, d + k * (2048 >> 4), idesc(!E4M3, 1), 1);
              umma_commit(&sh.v_free[c & 1]);
              ++c;
              if (j == n - 1) {
                umma_commit(&sh.o_full[t]);
                break;
              }
            }
            ok = wait(&sh.k_full[c & 1], (c >> 1) & 1);
            if (!ok) break;
            tmem_fence_after_sync();
            const uint64_t d = dk + (uint64_t)((c & 1) * (kTile >> 4));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t o = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
              umma_ss(tmem + t * 128, dq + o, d + o, idesc(!E4M3, 0), k > 0);
            }
            umma_commit(&sh.s_full[t]);
            umma_commit(&sh.k_free[c & 1]);
          }
        }
        umma_commit(&sh.done);
      }
      // Nothing is in flight when the tensor memory is freed, also after a
      // wait that ran out.
      __syncwarp();
      (void)paged_wait_warp(&sh.done, 0);
    }
  } else if (warp >= 8) {
    // ---- keys and values into shared memory ----
    fewer_registers<Regs<E4M3>::load>();
    const int lt = tid - 256;
    unsigned c = 0;  // steps so far
    bool ok = true;
    const Item* item;
    for (unsigned ic = 0; ok && (item = take(ic)); ++ic) {
      const Item it = *item;
      give_back(ic);
      const int32_t* table = a.b.page_table + (int64_t)it.seq * a.b.table_stride;
      // Lane g < 8 of each warp: the page of 16-key group g of step j, read two
      // steps ahead of its use; a bad id is recorded and page 0 read.
      auto fetch = [&](int j) {
        const int tok = j * kKeys + lane * 16;
        return lane < 8 && j < it.j1 && tok < it.len ? table[tok >> L.p_log2] : 0;
      };
      auto checked = [&](int p) {
        if (p >= 0 && p < L.n_pages) return p;
        paged_error(L, ERR_PAGED_PAGE, it.seq, p);
        return 0;
      };
      int pg = checked(fetch(it.j0)), pg_next = fetch(it.j0 + 1);
      if (E4M3) {
        // 16 codes ck of rows r + 16 i.  Eight neighbouring lanes are four
        // chunks of one half by two rows of different parity: their 16-byte
        // stores meet in no bank.
        const int ck = (lane & 3) | (lane >> 1 & 4), r = (lane >> 2 & 1) | (lane >> 3 & 2) | (warp & 3) << 2;
        const uint32_t put = (ck >> 2) * kHalf + r * 128 + ((((2 * ck) & 7) ^ (r & 7)) << 4);
        const int64_t page_stride = (int64_t)n_kv * L.P * D;
        const int64_t at = (int64_t)it.head * L.P * D + ck * 16;
        uint4 kr[8], vr[8];
        auto load = [&](int j, const uint8_t* pool, uint4 (&x)[8]) {
          const uint8_t* from = pool + at;
          const int left = it.len - j * kKeys - r;  // row 16 i + r is held where 16 i < left
          const int slot = (j * kKeys + r) & (L.P - 1), mask = L.P - 1;
          if (__all_sync(FULL, left > 112)) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              x[i] = *reinterpret_cast<const uint4*>(from + __shfl_sync(FULL, pg, i) * page_stride + ((slot + 16 * i) & mask) * D);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int64_t p = __shfl_sync(FULL, pg, i);
              x[i] = make_uint4(0, 0, 0, 0);
              if (16 * i < left) x[i] = *reinterpret_cast<const uint4*>(from + p * page_stride + ((slot + 16 * i) & mask) * D);
            }
          }
        };
        auto store = [&](uint32_t to, const uint4 (&x)[8]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            const uint32_t a0 = to + put + i * 2048;
#pragma unroll
            for (int k = 0; k < 2; ++k)
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a0 ^ (k * 16)), "r"(e4m3_h2(w[2 * k])),
                           "r"(e4m3_h2(w[2 * k] >> 16)), "r"(e4m3_h2(w[2 * k + 1])), "r"(e4m3_h2(w[2 * k + 1] >> 16))
                           : "memory");
          }
        };
        float ks = 1.0f, vs = 1.0f;  // lanes < 8 of the first warp: the groups' scales of the step that pg belongs to
        auto scales = [&](int j) {
          ks = vs = 1.0f;
          if (lt < 8 && j < it.j1 && j * kKeys + lt * 16 < it.len) {
            ks = L.k_scale[(int64_t)pg * n_kv + it.head];
            vs = L.v_scale[(int64_t)pg * n_kv + it.head];
          }
        };
        if (it.j0 < it.j1) {
          load(it.j0, L.k, kr);
          scales(it.j0);
        }
        for (int j = it.j0; j < it.j1; ++j, ++c) {
          load(j, L.v, vr);
          const float ks0 = ks, vs0 = vs;
          pg = checked(pg_next);
          pg_next = fetch(j + 2);
          scales(j + 1);
          ok = c < 2 || __all_sync(FULL, wait(&sh.k_free[c & 1], ((c >> 1) - 1) & 1));
          if (!ok) break;
          if (lt < 8) {
            sh.kb[c & 3][lt] = make_float2(ks0, __log2f(vs0));
            sh.inv[c & 3][lt] = __frcp_rn(vs0);
          }
          store(sk + (c & 1) * kTile, kr);
          fence_proxy_async();
          mbar_arrive_warp(&sh.k_full[c & 1], lane);
          if (j + 1 < it.j1) load(j + 1, L.k, kr);
          ok = c < 2 || __all_sync(FULL, wait(&sh.v_free[c & 1], ((c >> 1) - 1) & 1));
          if (!ok) break;
          store(sv + (c & 1) * kTile, vr);
          fence_proxy_async();
          mbar_arrive_warp(&sh.v_full[c & 1], lane);
        }
      } else {
        const int ck = lt & 15, r = lt >> 4;  // 8 channels ck of rows r + 8 i
        const uint32_t put = (ck >> 3) * kHalf + r * 128 + (((ck & 7) ^ r) << 4);
        const int64_t page_stride = (int64_t)n_kv * L.P * D * 2;
        const int64_t at = ((int64_t)it.head * L.P * D + ck * 8) * 2;
        auto load = [&](int j, const uint8_t* pool, uint32_t to) {
          const uint8_t* from = pool + at;
          const int left = it.len - j * kKeys - r;  // row 8 i + r is held where 8 i < left
          const int slot = (j * kKeys + r) & (L.P - 1), mask = L.P - 1;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int64_t p = __shfl_sync(FULL, pg, i >> 1);
            cp_async16_z(to + put + i * 1024, from + p * page_stride + ((slot + 8 * i) & mask) * (D * 2), 8 * i < left);
          }
          cp_async_commit();
        };
        uint64_t* pending = nullptr;
        auto signal = [&](bool last) {
          if (!pending) return;
          if (last)
            asm volatile("cp.async.wait_group 0;\n" ::: "memory");
          else
            asm volatile("cp.async.wait_group 1;\n" ::: "memory");
          fence_proxy_async();
          mbar_arrive_warp(pending, lane);
        };
        for (int j = it.j0; j < it.j1; ++j, ++c) {
          ok = c < 2 || __all_sync(FULL, wait(&sh.k_free[c & 1], ((c >> 1) - 1) & 1));
          if (!ok) break;
          load(j, L.k, sk + (c & 1) * kTile);
          signal(false);
          pending = &sh.k_full[c & 1];
          ok = c < 2 || __all_sync(FULL, wait(&sh.v_free[c & 1], ((c >> 1) - 1) & 1));
          if (!ok) break;
          load(j, L.v, sv + (c & 1) * kTile);
          signal(false);
          pending = &sh.v_full[c & 1];
          pg = checked(pg_next);
          pg_next = fetch(j + 2);
        }
        if (ok) signal(true);
        asm volatile("cp.async.wait_group 0;\n" ::: "memory");
      }
    }
  } else {
    // ---- softmax: one row a thread ----
    more_registers<Regs<E4M3>::softmax>();
    const int t = warp >> 2;
    const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t ts = trow + t * 128, to = trow + 256 + t * 128;
    bool ok = true;
    // One register: phases of s_full (bit 0), o_full (1) and met (2); place in
    // the scales' ring (bits 4, 5); items so far (from bit 8).
    unsigned st = 0;
    auto step_ring = [&](unsigned by) { st = (st & ~0x30u) | ((st + (by << 4)) & 0x30u); };
    // The eight softmax warps meet (an mbarrier: with the limit that every wait has).
    auto meet = [&]() {
      mbar_arrive_warp(&sh.met, lane);
      st ^= 4u;
      return __all_sync(FULL, wait_long(&sh.met, (~st >> 2) & 1)) != 0;
    };
    // Row x of the warp's 32, from its item.
    struct Place {
      int tok, head;
      bool live;
      int64_t out_row;
    };
    const int g_log2 = __ffs(G) - 1, wrow = t * 128 + (warp & 3) * 32;
    auto place_of = [&](const Item& it, int x) {
      Place y;
      y.tok = it.q0 + ((wrow + x) >> g_log2);
      y.head = it.head * G + ((wrow + x) & (G - 1));
      y.live = y.tok < it.n_new;
      y.out_row = (int64_t)it.row0 + y.tok;
      return y;
    };
    auto see_of = [&](const Item& it, const Place& y) {  // keys that the row sees
      return !y.live ? 0 : a.causal ? max(0, min(it.len, it.len - it.n_new + y.tok + 1)) : it.len;
    };
    // 16 bytes (8 channels) of row x of the warp in the query tile, where its
    // results are staged too once its products are done: rows move to and from
    // global memory 256 bytes at a time.
    auto stage_at = [&](int x, int chunk) {
      const int y = (warp & 3) * 32 + x;
      return sq + t * kTile + (chunk >> 3) * kHalf + y * 128 + (((chunk & 7) ^ (y & 7)) << 4);
    };
    auto stage_out = [&](int chunk, uint32_t h0, uint32_t h1, uint32_t h2, uint32_t h3) {
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(stage_at(lane, chunk)), "r"(h0), "r"(h1), "r"(h2), "r"(h3)
                   : "memory");
    };
    auto write_out = [&](const Item& it) {
      __syncwarp();
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const int x = 2 * i + (lane >> 4);
        const Place y = place_of(it, x);
        uint4 w;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(stage_at(x, lane & 15)));
        if (y.live) *reinterpret_cast<uint4*>(a.out + y.out_row * a.out_stride + y.head * D + (lane & 15) * 8) = w;
      }
      __syncwarp();
    };
    const Item* it;
    for (; (it = take(st >> 8)); st += 0x100u) {
      // The item is formed anew after the steps: in them, the registers are
      // for the row's logits.
      int n, lim0, nt;
      float m = -INFINITY, l = 0.0f, zf = fmaxf(a.scale, kTiny);
      {
        n = it->j1 - it->j0;
        nt = min(it->n_new - it->q0, q_tile) * G > 128 ? 2 : 1;
        lim0 = see_of(*it, place_of(*it, lane)) - it->j0 * kKeys;
        if (t < nt && n > 0 && ok) {
          // The warp's 32 queries into the operand tile: 16 lanes a row.
          // Loops kept short here and at the result: this code runs once an
          // item, and what it does not fetch anew each time it runs faster.
#pragma unroll 1
          for (int i0 = 0; i0 < 16; i0 += 8) {
            uint4 w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const Place y = place_of(*it, 2 * (i0 + i) + (lane >> 4));
              w[i] = make_uint4(0, 0, 0, 0);
              if (y.live) w[i] = *reinterpret_cast<const uint4*>(a.q + y.out_row * a.q_stride + y.head * D + (lane & 15) * 8);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t h[4] = {w[i].x ^ a.q_sign, w[i].y ^ a.q_sign, w[i].z ^ a.q_sign, w[i].w ^ a.q_sign};
              if (E4M3) {  // fp16, after a power of two that brings the row into its range
                float top = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  top = fmaxf(top, fmaxf(fabsf(__uint_as_float(h[k] << 16)), fabsf(__uint_as_float(h[k] & 0xffff0000u))));
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
                int ex = (int)(__float_as_uint(top) >> 23) - 127;
                ex = max(-100, min(ex, 120));
                const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  h[k] = pack2<true>(__uint_as_float(h[k] << 16) * down, __uint_as_float(h[k] & 0xffff0000u) * down);
                const int own = __shfl_sync(FULL, ex, (lane & 1) << 4);  // row 2 i + (lane & 1)
                if (lane >> 1 == i0 + i) zf *= __uint_as_float((uint32_t)(127 + own) << 23);
              }
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(stage_at(2 * (i0 + i) + (lane >> 4), lane & 15)),
                           "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                           : "memory");
            }
          }
          fence_proxy_async();
          mbar_arrive_warp(&sh.q_full[t], lane);
        }
      }
      if (t < nt && n > 0 && ok) {
        for (int j = 0; j < n; ++j, step_ring(1)) {
          ok = __all_sync(FULL, mbar_try_wait(&sh.s_full[t], st & 1) ||
                                    wait_slow(&sh.s_full[t], st & 1, j == 0 ? sh.patience : 1, &sh.dead));
          st ^= 1u;
          if (!ok) break;
          tmem_fence_after_sync();
          const int lim = lim0 - j * kKeys;  // columns from here on are hidden
          const bool cut = __any_sync(FULL, lim < kKeys);
          // The logits are read twice from tensor memory, 32 columns at a time,
          // the next ones on their way: holding all 128 in registers spilled.
          uint32_t v[2][32];
          auto arrive = [&](int h, int hh) {  // columns 32 h .. are in v[hh], the next are asked for
            tmem_ld_wait(v[hh]);
            if (h < 3) tmem_ld32_async(ts + (h + 1) * 32, v[hh ^ 1]);
            if (cut) {
              asm volatile("");  // a branch, not 32 selections in every step
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i >= lim - 32 * h) v[hh][i] = 0xff800000u;
            }
          };
          tmem_ld32_async(ts, v[0]);
          float mx = -INFINITY;
#pragma unroll 1
          for (int h0 = 0; h0 < 4; h0 += 2)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int h = h0 + hh;
            arrive(h, hh);
#pragma unroll
            for (int s = 0; s < 2; ++s) {  // 16 keys: one scale
              const uint32_t* z = &v[hh][16 * s];
              float x = max3(z[0], z[1], z[2]);
              float y = max3(z[3], z[4], z[5]);
              x = max3(__float_as_uint(x), z[6], z[7]);
              y = max3(__float_as_uint(y), z[8], z[9]);
              x = max3(__float_as_uint(x), z[10], z[11]);
              y = max3(__float_as_uint(y), z[12], z[13]);
              x = fmaxf(max3(__float_as_uint(x), z[14], z[15]), y);
              if (E4M3) {
                const float2 kb = sh.kb[(st >> 4) & 3][2 * h + s];
                x = fmaf(x, fmaxf(zf * kb.x, kTiny), kb.y);
              }
              mx = fmaxf(mx, x);
            }
          }
          tmem_ld32_async(ts, v[0]);
          if (!E4M3) mx *= zf;
          const bool raise = mx > m + kLazy || (m == -INFINITY && mx != -INFINITY);
          if (__any_sync(FULL, raise)) {
            const float mn = raise ? mx : m;
            const float f = m == -INFINITY ? 0.0f : ex2(m - mn);  // rows that stay: 2^0
            l *= f;
            m = mn;
            if (j > 0) {
#pragma unroll 2
              for (int h = 0; h < 8; ++h) {
                uint32_t w[16];
                tmem_ld16(to + h * 16, w);
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
                tmem_st16(to + h * 16, w);
              }
            }
          }
          const float ms = (m == -INFINITY ? 0.0f : m) - kShift;
#pragma unroll 1
          for (int h0 = 0; h0 < 4; h0 += 2) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int h = h0 + hh;
            arrive(h, hh);
            uint32_t p[16];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              float k = zf, bb = -ms;
              if (E4M3) {
                const float2 kb = sh.kb[(st >> 4) & 3][2 * h + s];
                k = fmaxf(zf * kb.x, kTiny);
                bb = kb.y - ms;
              }
              const uint64_t k2 = pair(k, k), b2 = pair(bb, bb);
              uint64_t add = 0;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint32_t* z = &v[hh][16 * s + 2 * i];
                float x, y;
                unpair(fma2(pair(__uint_as_float(z[0]), __uint_as_float(z[1])), k2, b2), x, y);
                x = ex2(x);
                y = ex2(y);
                add = add2(add, pair(x, y));
                p[8 * s + i] = pack2<E4M3>(x, y);
              }
              float x, y;
              unpair(add, x, y);
              l = E4M3 ? fmaf(x + y, sh.inv[(st >> 4) & 3][2 * h + s], l) : l + (x + y);
            }
            tmem_st16(ts + h * 16, p);
          }
          // Half of the weights are enough to begin the value product.
          tmem_wait_st();
          tmem_fence_before_sync();
          mbar_arrive_warp(h0 == 0 ? &sh.p_half[t] : &sh.p_full[t], lane);
          }
        }
        if (ok) {
          ok = __all_sync(FULL, wait(&sh.o_full[t], (st >> 1) & 1));
          st ^= 2u;
          tmem_fence_after_sync();
        }
      } else {
        step_ring((unsigned)n);
      }
      // ---- the row's result ----
      asm volatile("" ::: "memory");  // formed anew, as above
      const Item item = *it;
      give_back(st >> 8);
      const Place x = place_of(item, lane);
      const int row = wrow + lane, see = see_of(item, x), parts = item.parts, b_lo = item.b_lo;
      if (parts == 1) {
        if (t < nt && ok) {
          const float f = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll 1
          for (int h = 0; h < 4; ++h) {
            uint32_t v[32];
            if (n > 0) {
              tmem_ld32_async(to + h * 32, v);
              tmem_ld_wait(v);
            }
            if (n == 0 || see == 0) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pack2<false>(__uint_as_float(v[8 * i + 2 * k]) * f, __uint_as_float(v[8 * i + 2 * k + 1]) * f);
              stage_out(4 * h + i, w[0], w[1], w[2], w[3]);
            }
          }
          write_out(item);
          if (x.live && a.lse)
            a.lse[x.out_row * (n_kv * G) + x.head] = see > 0 ? (log2f(l) + (m - kShift)) * kLn2 : -INFINITY;
          tmem_fence_before_sync();
        }
        continue;
      }
      // A part of a split row tile: [32 column groups][256 rows] float4, then
      // the rows' maxima and sums.
      constexpr int64_t kPartFloats = (int64_t)kRows * (D + 2);
      auto part_of = [&](int64_t slot) { return a.part + slot * kPartFloats; };
      // A CTA can hold the beginning of one item and the rest of another.
      const int64_t mine = 2 * (int64_t)blockIdx.x + (item.j0 == 0 ? 1 : 0);
      auto slot = [&](int i) { return 2 * (int64_t)(b_lo + i) + (i == 0 ? 1 : 0); };
      if (t < nt) {
        float4* op = reinterpret_cast<float4*>(part_of(mine));
        float* ml = part_of(mine) + (int64_t)kRows * D;
        ml[row] = m;
        ml[kRows + row] = l;
#pragma unroll 1
        for (int h = 0; h < 4; ++h) {
          uint32_t v[32];
          if (n > 0 && ok) {
            tmem_ld32_async(to + h * 32, v);
            tmem_ld_wait(v);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            op[(8 * h + i) * kRows + row] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                                        __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
        }
        tmem_fence_before_sync();
      }
      __threadfence();
      if (!meet()) break;
      if (tid == 0) {
        const int old = atomicAdd(&a.counters[b_lo], 1);  // one item at most begins in b_lo and ends after it
        sh.last = old == parts - 1;
        if (sh.last) a.counters[b_lo] = 0;
      }
      if (!meet()) break;
      if (sh.last) {
        __threadfence();
        if (t < nt) {
          float M = -INFINITY, S = 0.0f;
          for (int i = 0; i < parts; ++i) M = fmaxf(M, __ldcg(part_of(slot(i)) + (int64_t)kRows * D + row));
          for (int i = 0; i < parts; ++i) {
            const float mi = __ldcg(part_of(slot(i)) + (int64_t)kRows * D + row);
            // A part without a maximum has the sum 0, or NaN where its logits were.
            S = fmaf(__ldcg(part_of(slot(i)) + (int64_t)kRows * (D + 1) + row), mi == -INFINITY ? 1.0f : ex2(mi - M), S);
          }
          const float f = S > 0.0f || S != S ? 1.0f / S : 0.0f;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {  // 64 columns at a time: 16 loads in flight
            float4 o[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int i = 0; i < parts; ++i) {
              const float mi = __ldcg(part_of(slot(i)) + (int64_t)kRows * D + row);
              const float w = mi == -INFINITY ? 0.0f : ex2(mi - M);
              const float4* op = reinterpret_cast<const float4*>(part_of(slot(i))) + 16 * h * kRows + row;
              float4 u[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) u[k] = __ldcg(op + k * kRows);
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                o[k].x = fmaf(u[k].x, w, o[k].x);
                o[k].y = fmaf(u[k].y, w, o[k].y);
                o[k].z = fmaf(u[k].z, w, o[k].z);
                o[k].w = fmaf(u[k].w, w, o[k].w);
              }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
              stage_out(8 * h + k, pack2<false>(o[2 * k].x * f, o[2 * k].y * f), pack2<false>(o[2 * k].z * f, o[2 * k].w * f),
                        pack2<false>(o[2 * k + 1].x * f, o[2 * k + 1].y * f),
                        pack2<false>(o[2 * k + 1].z * f, o[2 * k + 1].w * f));
          }
          write_out(item);
          if (x.live && a.lse)
            a.lse[x.out_row * (n_kv * G) + x.head] = see > 0 ? (log2f(S) + (M - kShift)) * kLn2 : -INFINITY;
        }
      }
      if (!meet()) break;  // sh.last is free again
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 12) tmem_dealloc(tmem, 512);
  if (tid == 0 && sh.dead) paged_error(L, ERR_PAGED_WAIT, (int32_t)blockIdx.x, sh.dead - 1, (int32_t)MK_ETIMEOUT);
}

}  // namespace

int64_t paged_prefill_part_floats() { return (int64_t)2 * kPagedMaxCtas * kRows * (D + 2); }

cudaError_t launch_paged_prefill(const PagedLayer& L, const PagedScratch& w, const mk_paged_batch& b, bool causal,
                                 const uint16_t* q, int64_t q_stride, float scale, uint16_t* out, int64_t out_stride,
                                 float* lse, cudaStream_t s) {
  const void* fn = L.e4m3 ? (const void*)k_paged_prefill<true> : (const void*)k_paged_prefill<false>;
  int sms = 0;
  const cudaError_t e = kernel_smem_attr(fn, kSmem, kThreads, nullptr, &sms);
  if (e != cudaSuccess) return e;
  const int grid = sms > 0 && sms <= kPagedMaxCtas ? sms : 128;
  const PrefillArgs a{b,   q,      out,
                      lse, q_stride, out_stride,
                      (scale < 0.0f ? -scale : scale) * kLog2e,
                      scale < 0.0f ? 0x80008000u : 0u, causal ? 1 : 0, w.prefill_part, w.prefill_counters};
  return L.e4m3 ? launch_pdl(k_paged_prefill<true>, dim3(grid), dim3(kThreads), (size_t)kSmem, s, 0, L, a)
                : launch_pdl(k_paged_prefill<false>, dim3(grid), dim3(kThreads), (size_t)kSmem, s, 0, L, a);
}

}  // namespace mk
