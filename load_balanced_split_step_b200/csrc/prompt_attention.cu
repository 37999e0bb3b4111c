// Attention of whole prompts on the 5th-generation tensor cores: packed sequences, grouped heads,
// causal, K and V packed or in the pages of the cache.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = 2^(c (s_ij - m_i)),   s_ij = q_i . k_j,   c = sm_scale log2 e
// over the keys j that query i sees, in one pass over the keys with a running reference m_i.
//
// A unit of work is 256 query rows of one kv head: the group's G heads of 256 / G consecutive tokens of one
// sequence, as two tiles A and B of 128 rows (row = G * token + head), so that a K or V block is
// loaded once for all heads that share it. Per block of 128 keys each tile X takes two products,
//   S[128 x 128]  = Q_X . K^T      (tensor memory)
//   O_X[128 x D] += P_X . V        (P_X read from tensor memory)
// with S, P_A, P_B, O_A, O_B filling the 512 columns of tensor memory. Four warps run the softmax of a tile, a
// thread per row, so that maxima and sums cross no threads; they hold the block's scores in registers.
// The tiles alternate half a period apart, so that one S buffer serves both: S_B is computed while the
// softmax of A works on the S_A it has read, and the next S_A while that of B works; neither waits for
// a product. (With an S buffer per tile, P had to lie over S, and each S waited for the product that read that
// P: 3700 cycles per pair of blocks, of which the softmax waited 1550. Now 2750, of which it waits 100.)
//
// m_i moves only when a block's maximum exceeds it by more than 8 (log2 units): p stays below 2^8, sums
// and O are fp32, and the rescaling of O in tensor memory becomes rare. P is rounded to bf16 for its
// product (relative error 2^-8 per weight at most, which the output's own bf16 rounding matches); the sum l_i is
// taken over the unrounded values.
//
// Persistent CTAs (one per SM) take units longest first from a counter: units are put in 64 buckets by the number
// of keys they reach, in a table that every CTA builds from cu_seqlens at the start. (Where there is a CTA for every
// unit they are dealt as they come, without the table: a prompt of 200 tokens takes 11.3 us instead of 12.5. Where there
// is one for every tile (or two, if units may be cut), a unit is one tile, which does not wait for another's scores:
// 10.3 us; 1024 tokens of 8/8 heads 17.8 instead of 20.4.)
// Where a bucket's units are longer than a CTA's share of all blocks (few heads, or a few new tokens on a long
// cache), they are cut into parts of about that share; parts leave (m, l, O) in the caller's scratch, and a second
// kernel, launched behind this one, joins them (a last part that joined the others by itself took 40 us for 18 parts
// of a tile: one SM reads too little at a time). 16 new tokens of 64/8 heads on 30000 keys: 285 us uncut, 40 us so.
// The rule of the cuts, and what each of its numbers is for, by the times of 22 shapes without it: a part has 6
// blocks at least (9: half of the shapes 8 to 30% slower; 2 and 4 are as fast, and 10 to 20% faster for up to 200 queries on
// 1600 keys); a unit up to 1.3 times the share stays whole (16 x 1 on 4000 keys of 32/8 heads 54 us, 66 without); cutting
// has to save 5 blocks (1700 tokens of 16/8 heads 34 us, 38; but 2518 of 4/2 30.5, 27.9); where it makes up to a third
// more parts than CTAs, the parts are made longer (900 on 2400 keys of 16/2 heads 38 us, 43).
// The producer warp looks the units up, ahead of the others, and loads Q and a ring of K and V blocks by TMA
// (swizzled planes of 64 elements). The next unit's Q has to wait for its place, and comes as far as L2 meanwhile
// (its arrival after that took 3000 cycles, now 1400).
//
// Bound by the tensor cores, and in long prompts by power: 8192 tokens of 64/8 heads of 128 take 840 us cold
// (1.31 PFLOP/s of the triangle's products) and 955 us in a row (1000 W, 1.4 GHz), where a large library product
// falls to 1.37 PFLOP/s. Short prompts are bound by the softmax warps' own chain (scores, exponentials, epilogue: 7300
// cycles per unit of one block): 64 prompts of 128 tokens take 92 us, twice what their bytes would.
//
// Roles (384 threads): warps 0-3 softmax of A, 4-7 of B (also the epilogues), warp 8 issues the products with
// K, warp 10 those with V, warp 9 looks up units and loads, warp 11 checks V. A softmax thread holds the 128
// scores of its row, so the softmax warpgroups take registers from the third (208 + 208 + 88 = 3 x the 168 of the
// launch). Every wait is bounded and ends in HPC_DEV_TIMEOUT: by 2 s and 64 us for each key that a sequence can have,
// since rows that are done one by one (values that are not finite) keep the other roles waiting. The 32 rows of a warp
// took 6 to 21 us for each key (packed, and pages of 16 with every CTA at it), so that 2 s alone passed at 96000 keys.
// (Waits that look whether such rows advance kept to 2 s, and cost 2 to 12% of every call.)
#include <cmath>

#include "umma_bf16.cuh"

namespace hpc {
namespace {

constexpr int kPaThreads = 384;
constexpr int kPaSoftRegs = 208, kPaOtherRegs = 88;
constexpr int kPaScoreWarp = 8, kPaLoadWarp = 9, kPaValueWarp = 10, kPaCheckWarp = 11;
constexpr int kPaRows = 128;            // query rows per tile
constexpr int kPaKeys = 128;            // keys per block
constexpr int kPaPlane = 128 * 128;     // 128 rows of 64 bf16: one swizzled plane
constexpr int kPaBuckets = 64;
constexpr int kPaTileRing = 3;          // units looked up ahead
constexpr uint32_t kPaCols = 512;       // S 0, P_A 128, P_B 192, O_A 256, O_B 384
constexpr float kPaMove = 8.f;
constexpr int kPaSplit = 2;               // P is handed over in two parts: after 64 keys, and whole
constexpr int kPaStages64 = 8, kPaStages128 = 5;
constexpr int kPaMinPart = 6;           // blocks: joining costs more than shorter parts save
constexpr int kPaMinSave = 5;           // blocks that cutting has to save
constexpr int kPaMaxParts = 32;
constexpr int kPaCuts = 512;            // cut units that the scratch can describe, ahead of the slots
constexpr uint64_t kPaRowsNs = 64000;   // 32 rows one by one, for each key: three times the slowest seen

template <int D>
struct PaLayout {
  static constexpr int kPlanes = D / 64;
  static constexpr int kStages = D == 128 ? kPaStages128 : kPaStages64;
  static constexpr int kTile = kPlanes * kPaPlane;  // a Q tile, a K block or a V block
  static constexpr int kOffRing = 2 * kTile;
  static constexpr int kBytes = kOffRing + kStages * kTile + 1024;  // + alignment slack
};

// One unit of work, or a part of it, as the producer publishes it.
struct PaUnit {
  int32_t valid;
  int32_t q0, q_end;  // row of q of the first token; end of the sequence
  int32_t kv0;        // packed: row of key 0; paged: the request
  int32_t keys;       // keys of the sequence
  int32_t vis;        // keys that the unit's first token sees, one more for each token after it
  int32_t blocks[2];  // key blocks of tile A and B in this part
  int32_t kvh;
  int32_t from;       // first block of the part
  int32_t part;       // which part
  int32_t parts[2];   // parts that hold blocks of tile A and B
  int32_t slot;       // the part's place in the scratch; those of one unit are Hkv apart
  int32_t pad[2];
};

// A cut unit, as the joining kernel finds it at the head of the scratch.
struct PaCut {
  int32_t q0, q_end, kvh, slot, parts[2], pad[2];
};
constexpr size_t kPaCutBytes = kPaCuts * sizeof(PaCut);

struct PaArgs {
  const int32_t* cu_q;
  const int32_t* cu_k;      // packed
  const int32_t* table;     // paged
  const int32_t* seq_lens;  // paged
  const __nv_bfloat16 *q, *k, *v;  // packed rows, or pages; for pa_row
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
  uint32_t* work;  // units taken, units cut; zero at the start
  PaCut* cuts;
  float* partial;  // [slots][2 tiles][m 128, l 128, O (D / 4) x 128 x 4]
  int64_t tokens, kv_tokens, max_pages;
  uint64_t limit_ns;  // of a wait
  float scale_log2, scale;
  int32_t batch, Hq, Hkv, group, causal, P, num_pages, nhd, slots;
  int32_t unsorted;  // a CTA for every unit: they are dealt as they come
  int32_t single;    // so few that a unit is one tile: A, and no B
};

struct PaBars {
  uint64_t kv_full[8], kv_empty[8];
  uint64_t q_full, q_free;
  uint64_t s_full[2], s_read[2], p_full[2][2], pv_done[2];
  uint64_t unit_full[kPaTileRing], unit_free[kPaTileRing];
  uint64_t checked[kPaTileRing];  // per slot: the check may be a unit ahead of the epilogues
  uint64_t drained[2];
};

struct PaShared {
  PaBars bars;
  PaUnit unit[kPaTileRing];
  int32_t found[kPaTileRing];  // the unit's partly visible blocks hold a value that is not finite
  int32_t base[kPaBuckets];   // parts of token tiles in the buckets above
  int32_t count[kPaBuckets];  // and in this one
  int32_t parts[kPaBuckets];  // per tile of the bucket
  unsigned long long blocks;  // of all token tiles, about
  int32_t hist[kPaBuckets + 1], rem[kPaBuckets + 1];
  int32_t span;               // extent of the cost axis
  int32_t tiles;              // parts of all token tiles
  int32_t bad;
  uint32_t tmem;
};

// A sequence's tokens and keys; false when the lengths do not hold together.
__device__ __forceinline__ bool pa_sequence(const PaArgs& a, bool paged, int32_t s, int32_t& q0, int32_t& q1, int32_t& k0,
                                            int32_t& keys) {
  q0 = a.cu_q[s];
  q1 = a.cu_q[s + 1];
  bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.tokens;
  if (paged) {
    k0 = s;
    keys = a.seq_lens[s];
    ok = ok && keys >= q1 - q0 && static_cast<int64_t>(keys) <= a.max_pages * a.P;
  } else {
    k0 = a.cu_k[s];
    const int32_t k1 = a.cu_k[s + 1];
    keys = k1 - k0;
    ok = ok && k0 >= 0 && k1 >= k0 && k1 <= a.kv_tokens;
  }
  if (!ok) q0 = q1 = keys = 0;
  return ok;
}

// The sequence's units on the cost axis [lo, hi): a unit of 2^shift tokens costs the units' worth of keys it reaches.
__device__ __forceinline__ void pa_span(const PaArgs& a, int32_t q0, int32_t q1, int32_t keys, int shift, int32_t& lo,
                                        int32_t& hi) {
  const int32_t n = q1 - q0, before = a.causal ? (keys > n ? keys - n : 0) : keys;
  lo = before >> shift;
  hi = lo + ((n + (1 << shift) - 1) >> shift);
}

// One step of a transposition over lanes: the upper lane's `a` and the lower lane's `b` change places.
__device__ __forceinline__ void swap_pieces(uint4& a, uint4& b, bool upper, int mask) {
  uint4 s = upper ? a : b;
  s.x = __shfl_xor_sync(0xffffffffu, s.x, mask);
  s.y = __shfl_xor_sync(0xffffffffu, s.y, mask);
  s.z = __shfl_xor_sync(0xffffffffu, s.z, mask);
  s.w = __shfl_xor_sync(0xffffffffu, s.w, mask);
  if (upper) a = s;
  else b = s;
}

// One row by one warp from global memory, without a product over keys that it does not see. For units whose
// partly visible blocks of V hold infinities or NaN: there the tensor cores' 0 * v would reach rows that do not
// see v. Such a prompt is broken; this keeps it from changing the tokens before the break. Keys [from, vis);
// to the output, or as part of a unit to row `r` of its slot.
template <int D, bool kPaged>
__device__ __noinline__ void pa_row(const PaArgs& a, const PaUnit& x, int32_t token, int32_t head_in, int32_t from,
                                    int32_t vis, float* slot, int32_t r) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const int32_t head = x.kvh * a.group + head_in;
  const __nv_bfloat16* q = a.q + token * a.q_token + head * a.q_head;
  float qf[kPer], o[kPer] = {};
#pragma unroll
  for (int e = 0; e < kPer; ++e) qf[e] = __bfloat162float(q[lane + 32 * e]);
  float m = -INFINITY, l = 0.f;
  constexpr int kBatch = 8;  // keys loaded together: one at a time waits for memory at every key
  for (int32_t j0 = from; j0 < vis; j0 += kBatch) {
    float s[kBatch], vf[kBatch][kPer];
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const int32_t j = j0 + n < vis ? j0 + n : vis - 1;
      const __nv_bfloat16 *k, *v;
      if (kPaged) {
        int32_t page = a.table[static_cast<int64_t>(x.kv0) * a.max_pages + j / a.P];
        if (page < 0 || page >= a.num_pages) page = 0;
        const int64_t at = a.nhd ? (static_cast<int64_t>(page) * a.P + j % a.P) * a.Hkv + x.kvh
                                 : (static_cast<int64_t>(page) * a.Hkv + x.kvh) * a.P + j % a.P;
        k = a.k + at * D;
        v = a.v + at * D;
      } else {
        k = a.k + (x.kv0 + static_cast<int64_t>(j)) * a.k_token + x.kvh * a.k_head;
        v = a.v + (x.kv0 + static_cast<int64_t>(j)) * a.v_token + x.kvh * a.v_head;
      }
      s[n] = 0.f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        s[n] = fmaf(qf[e], __bfloat162float(k[lane + 32 * e]), s[n]);
        vf[n][e] = __bfloat162float(v[lane + 32 * e]);
      }
    }
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) s[n] += __shfl_xor_sync(0xffffffffu, s[n], w);
    }
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      if (j0 + n >= vis || s[n] == -INFINITY) continue;  // no weight
      if (s[n] > m) {
        const float shrink = m == -INFINITY ? 0.f : ex2((m - s[n]) * a.scale_log2);
        l *= shrink;
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = m == -INFINITY ? o[e] : o[e] * shrink;
        m = s[n];
      }
      const float p = ex2((s[n] - m) * a.scale_log2);
      l += p;
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[e] = fmaf(p, vf[n][e], o[e]);
    }
  }
  if (slot) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int d = lane + 32 * e;
      slot[2 * kPaRows + ((d >> 2) * kPaRows + r) * 4 + (d & 3)] = o[e];
    }
    if (lane == 0) {
      slot[r] = m;
      slot[kPaRows + r] = l;
    }
    return;
  }
  const bool some = l > 0.f || l != l;
  const int64_t at = static_cast<int64_t>(token) * a.Hq + head;
#pragma unroll
  for (int e = 0; e < kPer; ++e) a.out[at * D + lane + 32 * e] = __float2bfloat16_rn(some ? o[e] / l : 0.f);
  if (a.lse && lane == 0) a.lse[at] = some ? m * a.scale + logf(l) : -INFINITY;
}

template <int D, bool kPaged>
__global__ void __launch_bounds__(kPaThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PaArgs a) {
  using L = PaLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ PaShared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + L::kOffRing;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group_shift = 31 - __clz(a.group), unit_shift = 8 - group_shift - a.single;  // 1, 2, 4 or 8 heads
  const int32_t tokens_per_unit = 1 << unit_shift, tokens_per_tile = kPaRows >> group_shift;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar(sh.bars.kv_full[s]), 1);
      mbar_init(bar(sh.bars.kv_empty[s]), 2);  // the products, and the check of V
    }
    mbar_init(bar(sh.bars.q_full), 1);
    mbar_init(bar(sh.bars.q_free), 1);
    for (int x = 0; x < 2; ++x) mbar_init(bar(sh.bars.drained[x]), 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(sh.bars.s_full[x]), 1);
      mbar_init(bar(sh.bars.s_read[x]), 4);
      for (int h = 0; h < 2; ++h) mbar_init(bar(sh.bars.p_full[x][h]), 4);
      mbar_init(bar(sh.bars.pv_done[x]), 1);
    }
    for (int t = 0; t < kPaTileRing; ++t) {
      mbar_init(bar(sh.bars.unit_full[t]), 1);
      mbar_init(bar(sh.bars.checked[t]), 1);
      mbar_init(bar(sh.bars.unit_free[t]), 11);  // 8 softmax warps, the two that issue, the check
    }
    fence_barrier_init();
    sh.span = 0;
    sh.blocks = 0;
    sh.bad = 0;
  }
  for (int i = threadIdx.x; i <= kPaBuckets; i += kPaThreads) sh.hist[i] = sh.rem[i] = 0;
  if (warp == kPaScoreWarp) tmem_alloc(smem_u32(&sh.tmem), kPaCols);
  if (warp == kPaLoadWarp && lane == 0) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait();
  pdl_launch_dependents();

  // ---- the table of units: buckets of 2^bucket units of the cost axis, 64 at most
  int bucket = 0;
  uint32_t units = 0;
  if (!a.unsorted) {
    int32_t lo0 = 0, hi0 = 0;  // the thread's first sequence
    {
      int32_t span = 0, bad = 0;
      int64_t rows = 0;  // keys that the units reach
      for (int32_t s = threadIdx.x; s < a.batch; s += kPaThreads) {
        int32_t q0, q1, k0, keys, lo, hi;
        bad |= !pa_sequence(a, kPaged, s, q0, q1, k0, keys);
        pa_span(a, q0, q1, keys, unit_shift, lo, hi);
        if (hi > span) span = hi;
        rows += ((static_cast<int64_t>(hi) * (hi + 1) - static_cast<int64_t>(lo) * (lo + 1)) / 2) << unit_shift;
        if (s == static_cast<int32_t>(threadIdx.x)) lo0 = lo, hi0 = hi;
      }
      if (span > 0) atomicMax(&sh.span, span);
      if (rows > 0 && a.slots > 0) atomicAdd(&sh.blocks, static_cast<unsigned long long>(rows / kPaKeys + 1));
      if (bad) sh.bad = 1;
      __syncthreads();
      if (threadIdx.x == 0 && sh.bad && blockIdx.x == 0) atomicOr(a.status, HPC_DEV_BAD_SEQLEN);
    }
    const int32_t per_bucket = (sh.span + kPaBuckets - 1) / kPaBuckets;
    bucket = per_bucket > 1 ? 32 - __clz(per_bucket - 1) : 0;
    for (int32_t s = threadIdx.x; s < a.batch; s += kPaThreads) {
      int32_t lo = lo0, hi = hi0;
      if (s >= kPaThreads) {
        int32_t q0, q1, k0, keys;
        pa_sequence(a, kPaged, s, q0, q1, k0, keys);
        pa_span(a, q0, q1, keys, unit_shift, lo, hi);
      }
      if (hi > lo) {
        const int32_t mask = (1 << bucket) - 1;
        atomicAdd(&sh.hist[hi >> bucket], 1);
        atomicAdd(&sh.rem[hi >> bucket], hi & mask);
        atomicAdd(&sh.hist[lo >> bucket], -1);
        atomicAdd(&sh.rem[lo >> bucket], -(lo & mask));
      }
    }
    __syncthreads();
    if (warp == 0) {
      // longest first: lane l holds the buckets 63 - 2 l and 62 - 2 l
      const int b0 = kPaBuckets - 1 - 2 * lane, b1 = b0 - 1;
      auto scan = [&](int32_t v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int32_t y = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += y;
        }
        return v;
      };
      const int32_t h0 = sh.hist[b0], h1 = sh.hist[b1];
      const int32_t above = sh.hist[kPaBuckets] + scan(h0 + h1) - h0 - h1;  // sequences that end past bucket b0
      const int32_t c0 = (above << bucket) + sh.rem[b0], c1 = ((above + h0) << bucket) + sh.rem[b1];
      int32_t p0 = 1, p1 = 1;
      if (a.slots > 0) {
        // Parts per unit: about a CTA's share of all blocks each, as long as the scratch has a place for them. The
        // buckets that are cut come first, so that a part's number is its place.
        const float share = static_cast<float>(sh.blocks) * a.Hkv / gridDim.x;  // the same in every CTA
        int32_t length = share > kPaMinPart ? static_cast<int32_t>(fminf(ceilf(share), 1e9f)) : kPaMinPart;
        auto cut = [&](int b) -> int32_t {
          const int64_t most = (((static_cast<int64_t>(b + 1) << bucket) + 1) << unit_shift) / kPaKeys + 1,
                        least = ((static_cast<int64_t>(b) << bucket) << unit_shift) / kPaKeys;
          // a unit a little over the share is better left whole; a bucket of short ones beside a long one too
          if (10 * most <= 13ll * length || most < length + kPaMinSave || 2 * least < length) return 1;
          const float n = ceilf(static_cast<float>(most) / static_cast<float>(length));
          return n < kPaMaxParts ? static_cast<int32_t>(n) : kPaMaxParts;
        };
        const int32_t room = a.slots / a.Hkv;
        int32_t end = 0;
        for (int again = 0; again < 2; ++again) {
          p0 = cut(b0), p1 = cut(b1);
          end = scan(c0 * p0 + c1 * p1);
          // a few parts more than CTAs would take a second turn: rather longer parts
          const int64_t all = static_cast<int64_t>(__shfl_sync(0xffffffffu, end, 31)) * a.Hkv;
          if (all <= gridDim.x || 20 * all > 27ll * gridDim.x) break;
          length = static_cast<int32_t>((static_cast<int64_t>(length) * all + gridDim.x - 1) / gridDim.x);
        }
        if (end - c1 * p1 > room) p0 = 1;
        if (end > room) p1 = 1;
      }
      const int32_t n0 = c0 * p0, n1 = c1 * p1, upto = scan(n0 + n1);
      sh.parts[b0] = p0;
      sh.parts[b1] = p1;
      sh.count[b0] = n0;
      sh.count[b1] = n1;
      sh.base[b0] = upto - n0 - n1;
      sh.base[b1] = upto - n1;
      if (lane == 31) sh.tiles = upto;
    }
    __syncthreads();
    units = static_cast<uint32_t>(sh.tiles) * a.Hkv;  // fewer than rows of q
  } else if (blockIdx.x == 0) {
    for (int32_t s = threadIdx.x; s < a.batch; s += kPaThreads) {
      int32_t q0, q1, k0, keys;
      if (!pa_sequence(a, kPaged, s, q0, q1, k0, keys)) atomicOr(a.status, HPC_DEV_BAD_SEQLEN);
    }
  }
  bool ok = true;
  uint32_t err = 0;
  auto wait = [&](uint64_t& b, uint32_t parity) -> bool {
    if (ok && !mbar_wait(smem_u32(&b), parity, a.limit_ns)) {
      ok = false;
      err = HPC_DEV_TIMEOUT;
    }
    return ok;
  };

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPaSoftRegs));
    // ------------------------------------------------------------------ softmax, tile t of every unit
    const int t = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t p_at = lanes + 128 + 64 * t, o_at = lanes + 256 + 128 * t;
    const int32_t tok = t * tokens_per_tile + (row >> group_shift);
    const int32_t tok_low = t * tokens_per_tile + ((row & ~31) >> group_shift);  // of the warp
    const float c = a.scale_log2;
    uint32_t done = 0;  // blocks of this tile so far
    uint32_t fill = 0;  // ring stages of the units before
    for (int32_t n_unit = 0;; ++n_unit) {
      const int slot = n_unit % kPaTileRing;
      wait(sh.bars.unit_full[slot], (n_unit / kPaTileRing) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const PaUnit x = sh.unit[slot];
      if (!x.valid) break;
      const int nb = t == 0 ? x.blocks[0] : x.blocks[1];
      const int nb_unit = x.blocks[0] > x.blocks[1] ? x.blocks[0] : x.blocks[1];
      // keys this row sees; fewest of the warp's rows
      const int32_t vis = a.causal ? min(x.vis + tok, x.keys) : x.keys;
      const int32_t vis_low = a.causal ? min(x.vis + tok_low, x.keys) : x.keys;
      float m = -INFINITY, l = 0.f;
      for (int j = x.from; j < x.from + nb && ok; ++j) {
        wait(sh.bars.s_full[t], done & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        float v[128];
        umma::ld128(lanes, v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.bars.s_read[t]));  // S is free for the other tile
        if ((j + 1) * kPaKeys > vis_low) {
          const int32_t lim = vis - j * kPaKeys, low = vis_low - j * kPaKeys;
          // groups of 32 keys that the whole warp sees stay as they are
#pragma unroll
          for (int h = 0; h < kPaKeys / 32; ++h) {
            if (32 * (h + 1) > low) {
#pragma unroll
              for (int i = 32 * h; i < 32 * (h + 1); ++i) v[i] = i < lim ? v[i] : -INFINITY;
            }
          }
        }
        float x0 = v[0], x1 = v[1], x2 = v[2], x3 = v[3];
#pragma unroll
        for (int i = 4; i < 128; i += 8) {
          x0 = fmaxf(fmaxf(x0, v[i]), v[i + 1]);
          x1 = fmaxf(fmaxf(x1, v[i + 2]), v[i + 3]);
          if (i + 4 < 128) {
            x2 = fmaxf(fmaxf(x2, v[i + 4]), v[i + 5]);
            x3 = fmaxf(fmaxf(x3, v[i + 6]), v[i + 7]);
          }
        }
        const float mx = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3));
        // the reference: set by the first block with a key, then moved only past the margin
        bool move = false;
        float shrink = 1.f;
        if (mx > m) {
          if (m == -INFINITY) {
            m = mx;
          } else if ((mx - m) * c > kPaMove) {
            shrink = ex2((m - mx) * c);
            m = mx;
            l *= shrink;
            move = true;
          }
        }
        // the product of the block before: it reads the P that is written next, and O is complete without it
        if (done > 0) {
          wait(sh.bars.pv_done[t], (done - 1) & 1);
          tc_fence_after();
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            float o[32];
            umma::ld32(o_at + c0, o);
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(o[i] * shrink);
            umma::st32(o_at + c0, w);
          }
        }
        const float mc = m == -INFINITY ? 0.f : m * c;
        const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
        if ((j + 1) * kPaKeys > x.keys && (t == 0 || j >= x.from + x.blocks[0])) {
          // Rows of V past the last key hold another sequence's values or what the memory held: zero, so that
          // 0 * v stays 0. The fill is the only one that its parity can mean: the stage's fill before was read
          // by products that this block's S follows.
          const uint32_t f = fill + 2 * (j - x.from) + 1;
          wait(sh.bars.kv_full[f % L::kStages], (f / L::kStages) & 1);
          ok = __all_sync(0xffffffffu, ok);
          uint8_t* vt = ring + (f % L::kStages) * L::kTile;
          const int32_t first = x.keys - j * kPaKeys;
          for (int i = threadIdx.x & 127; i < (kPaKeys - first) * 8; i += 128)
            for (int pl = 0; pl < L::kPlanes; ++pl)
              *reinterpret_cast<uint4*>(vt + pl * kPaPlane + first * 128 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_shared();
        }
        float2 sum[4] = {};
#pragma unroll
        for (int h = 0; h < kPaKeys / 32; ++h) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 e = fma2(make_float2(v[32 * h + 2 * i], v[32 * h + 2 * i + 1]), c2, mc2);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            sum[i & 3] = add2(sum[i & 3], e);
            w[i] = pack_bf16x2(e.x, e.y);
          }
          umma::st16(p_at + 16 * h, w);
          if (h == kPaSplit - 1 || h == kPaKeys / 32 - 1) {  // a part of P is complete
            umma::st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(sh.bars.p_full[t][h == kPaSplit - 1 ? 0 : 1]));
          }
        }
        const float2 s2 = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += s2.x + s2.y;
        ++done;
      }
      fill += 2 * nb_unit;
      // ---- epilogue
      if (nb > 0) {
        wait(sh.bars.pv_done[t], (done - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
      }
      wait(sh.bars.checked[slot], (n_unit / kPaTileRing) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const bool found = sh.found[slot] != 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh.bars.unit_free[slot]));
      const int parts = t == 0 ? x.parts[0] : x.parts[1];
      if (nb == 0 && (x.part > 0 || parts > 0)) {  // another part has this tile's keys
        tc_fence_before();
        continue;
      }
      const bool live = x.q0 + tok < x.q_end;
      float* slot_at = parts > 1 ? a.partial + (static_cast<int64_t>(x.slot) * 2 + t) * (kPaRows * (D + 2)) : nullptr;
      if (found) {
        // 0 * v is not 0 for some v that a row does not see: the rows of this tile one by one
        for (int i = 0; i < 32; ++i) {
          const int32_t rk = (row & ~31) + i, tk = t * tokens_per_tile + (rk >> group_shift);
          const int32_t seen = min(min(x.vis + tk, x.keys), parts > 1 ? (x.from + nb) * kPaKeys : x.keys);
          if (x.q0 + tk < x.q_end) pa_row<D, kPaged>(a, x, x.q0 + tk, rk & (a.group - 1), x.from * kPaKeys, seen, slot_at, rk);
        }
        if (parts <= 1) {
          tc_fence_before();
          continue;
        }
      }
      if (parts > 1) {
        // ---- a part: its state to the scratch, row by row of the tile side by side
        if (!found) {
          if (live) {
            slot_at[row] = m;
            slot_at[kPaRows + row] = l;
          }
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            float o[32];
            umma::ld32(o_at + c0, o);
            float4* at = reinterpret_cast<float4*>(slot_at + 2 * kPaRows) + (c0 / 4) * kPaRows + row;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (live) at[i * kPaRows] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        tc_fence_before();
        continue;
      }
      // ---- the whole unit; a NaN stays one; a row without keys is zero (O then holds anything).
      // A thread holds a row of O. Four lanes exchange 16-byte pieces of their rows, so that each stores 64
      // bytes of a row with its neighbours: whole sectors (16 bytes of every row at a time took 3800 cycles).
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      __nv_bfloat16* dst[4];
      bool there[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int32_t rk = (row & ~3) + k, tk = x.q0 + t * tokens_per_tile + (rk >> group_shift);
        there[k] = tk < x.q_end;
        dst[k] = a.out + (static_cast<int64_t>(tk) * a.Hq + x.kvh * a.group + (rk & (a.group - 1))) * D + 8 * (lane & 3);
      }
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        float o[32];
        umma::ld32(o_at + c0, o);
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = nb > 0 ? o[i] * inv : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]), pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                            pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
        swap_pieces(w[0], w[1], lane & 1, 1);
        swap_pieces(w[2], w[3], lane & 1, 1);
        swap_pieces(w[0], w[2], lane & 2, 2);
        swap_pieces(w[1], w[3], lane & 2, 2);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (there[k]) *reinterpret_cast<uint4*>(dst[k] + c0) = w[k];
      }
      if (a.lse && live)
        a.lse[static_cast<int64_t>(x.q0 + tok) * a.Hq + x.kvh * a.group + (row & (a.group - 1))] =
            l > 0.f || l != l ? m * a.scale + logf(l) : -INFINITY;
      tc_fence_before();
    }
    if (err && lane == 0) atomicOr(a.status, err);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPaOtherRegs));
    if (warp == kPaLoadWarp) {
      // ------------------------------------------------------------------ units and loads
      uint32_t fill = 0;  // ring fills so far
      int32_t n_unit = 0, n_q = 0;
      // Where the last lookup ended: this CTA's units come in order, so that within a bucket the next one
      // goes on from there (a batch of thousands of sequences is gone through once for each bucket).
      int32_t last_b = -1, last_s0 = 0, last_sum = 0;
      uint32_t dealt = blockIdx.x;
      for (bool begun = false;; begun = true) {
        uint32_t u = blockIdx.x;
        if (a.unsorted) {
          u = dealt;
          dealt += gridDim.x;  // none is left, unless the lengths overlap
        } else if (begun) {
          if (lane == 0) u = gridDim.x + atomicAdd(a.work, 1u);
          u = __shfl_sync(0xffffffffu, u, 0);
        }
        PaUnit x = {};
        if (a.unsorted || u < units) {
          const int32_t tile = static_cast<int32_t>(u / static_cast<uint32_t>(a.Hkv));
          x.kvh = static_cast<int32_t>(u) - tile * a.Hkv;
          int32_t rank = tile, parts = 1, bucket_lo = 0, bucket_hi = INT32_MAX;
          if (!a.unsorted) {
            // bucket: the one with base <= tile < base + count
            uint32_t m0 = __ballot_sync(0xffffffffu, tile >= sh.base[lane] && tile < sh.base[lane] + sh.count[lane]);
            uint32_t m1 = __ballot_sync(0xffffffffu, tile >= sh.base[lane + 32] && tile < sh.base[lane + 32] + sh.count[lane + 32]);
            const int b = m0 ? __ffs(m0) - 1 : 32 + __ffs(m1) - 1;
            parts = sh.parts[b];
            rank -= sh.base[b];
            if (parts > 1) {
              x.part = rank % parts;
              rank /= parts;
              x.slot = static_cast<int32_t>(u);
            }
            bucket_lo = b << bucket;
            bucket_hi = (b + 1) << bucket;
            if (b != last_b) last_b = b, last_s0 = last_sum = 0;
          }
          rank -= last_sum;
          // sequence: prefix of the tiles that each has in the bucket
          for (int32_t s0 = last_s0; s0 < a.batch; s0 += 32) {
            const int32_t s = s0 + lane;
            int32_t q0 = 0, q1 = 0, k0 = 0, keys = 0, lo = 0, hi = 0, from = 0, n = 0;
            if (s < a.batch) {
              pa_sequence(a, kPaged, s, q0, q1, k0, keys);
              pa_span(a, q0, q1, keys, unit_shift, lo, hi);
              from = max(lo, bucket_lo);
              const int32_t to = min(hi, bucket_hi);
              n = to > from ? to - from : 0;
            }
            int32_t inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int32_t y = __shfl_up_sync(0xffffffffu, inc, o);
              if (lane >= o) inc += y;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, rank < inc);
            if (hit) {
              x.valid = 1;
              const int w = __ffs(hit) - 1;
              const int32_t i = __shfl_sync(0xffffffffu, from - lo + rank - (inc - n), w);
              q0 = __shfl_sync(0xffffffffu, q0, w);
              q1 = __shfl_sync(0xffffffffu, q1, w);
              keys = __shfl_sync(0xffffffffu, keys, w);
              x.kv0 = __shfl_sync(0xffffffffu, k0, w);
              x.q0 = q0 + i * tokens_per_unit;
              x.q_end = q1;
              x.keys = keys;
              x.vis = a.causal ? keys - (q1 - q0) + i * tokens_per_unit + 1 : keys;
              for (int t = 0; t < 2; ++t) {
                // the last token of the tile that exists sees the most
                const int32_t first = x.q0 + t * tokens_per_tile;
                const int32_t last = first + tokens_per_tile < q1 ? first + tokens_per_tile : q1;
                int32_t seen = a.causal ? x.vis + (last - 1 - x.q0) : keys;
                if (seen > keys) seen = keys;
                x.blocks[t] = first < q1 && seen > 0 ? (seen + kPaKeys - 1) / kPaKeys : 0;
              }
              if (a.single) x.blocks[1] = 0;
              // the part's blocks
              int32_t length = x.blocks[0] > x.blocks[1] ? x.blocks[0] : x.blocks[1];
              if (parts > 1) {
                length = (length + parts - 1) / parts;
                if (length < kPaMinPart) length = kPaMinPart;
              }
              x.from = x.part * length;
              for (int t = 0; t < 2; ++t) {
                const int32_t have = x.blocks[t], left = have - x.from;
                x.parts[t] = parts > 1 ? (have + length - 1) / length : (have > 0 ? 1 : 0);
                x.blocks[t] = left < 0 ? 0 : (left < length ? left : length);
              }
              if (a.single) x.parts[1] = 1;  // the tile is another unit's
              break;
            }
            const int32_t sum = __shfl_sync(0xffffffffu, inc, 31);
            rank -= sum;
            last_sum += sum;
            last_s0 = s0 + 32;
          }
        }
        if (x.valid && x.part > 0 && x.blocks[0] == 0 && x.blocks[1] == 0) continue;  // fewer parts than the bucket's
        const int slot = n_unit % kPaTileRing;
        if (n_unit >= kPaTileRing) wait(sh.bars.unit_free[slot], ((n_unit / kPaTileRing) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) x.valid = 0;
        if (lane == 0) {
          if (x.valid && x.part == 0 && (x.parts[0] > 1 || x.parts[1] > 1))
            a.cuts[atomicAdd(a.work + 1, 1u)] = {x.q0, x.q_end, x.kvh, x.slot, {x.parts[0], x.parts[1]}, {}};
          sh.unit[slot] = x;
          mbar_arrive(bar(sh.bars.unit_full[slot]));
        }
        ++n_unit;
        if (!x.valid) break;
        const int nb = x.blocks[0] > x.blocks[1] ? x.blocks[0] : x.blocks[1];
        if (nb == 0) continue;  // no keys: the epilogue writes zeros
        // Q, once the products of the unit before have read theirs; until then it comes as far as L2
        if (n_q > 0 && lane < 2 * L::kPlanes)
          tma_prefetch_4d(&tm_q, 64 * (lane / 2), x.kvh * a.group, x.q0 + (lane & 1) * tokens_per_tile, 0);
        if (n_q > 0) wait(sh.bars.q_free, (n_q - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++n_q;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(sh.bars.q_full), a.single ? L::kTile : 2 * L::kTile);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int pl = 0; pl < L::kPlanes; ++pl)
              if (t == 0 || !a.single)
                tma_load_4d(smem_u32(smem) + t * L::kTile + pl * kPaPlane, &tm_q, bar(sh.bars.q_full), 64 * pl,
                            x.kvh * a.group, x.q0 + t * tokens_per_tile, 0);
        }
        // K_0, V_0, K_1, V_1, ...
        if (!kPaged) {
          if (lane == 0) {
            for (int f = 0; f < 2 * nb && ok; ++f, ++fill) {
              const int st = fill % L::kStages;
              if (fill >= L::kStages && !wait(sh.bars.kv_empty[st], (fill / L::kStages - 1) & 1)) break;
              mbar_arrive_expect_tx(bar(sh.bars.kv_full[st]), L::kTile);
              for (int pl = 0; pl < L::kPlanes; ++pl)
                tma_load_4d(smem_u32(ring) + st * L::kTile + pl * kPaPlane, (f & 1) ? &tm_v : &tm_k,
                            bar(sh.bars.kv_full[st]), 64 * pl, x.kvh, x.kv0 + (x.from + (f >> 1)) * kPaKeys, 0);
            }
          }
        } else {
          // 32 page ids at a time; pages of one block never straddle two batches of ids
          const int per_block = kPaKeys / a.P;
          const int32_t* row = a.table + static_cast<int64_t>(x.kv0) * a.max_pages + x.from * per_block;
          const int32_t live = (x.keys + a.P - 1) / a.P - x.from * per_block;  // pages that hold keys, from the part on
          for (int32_t p0 = 0; p0 < nb * per_block && ok; p0 += 32) {
            int32_t id = 0;
            if (p0 + lane < live && p0 + lane < nb * per_block) {
              id = row[p0 + lane];
              if (id < 0 || id >= a.num_pages) {
                id = 0;
                err |= HPC_DEV_BAD_PAGE;  // a stand-in; the request's output is unspecified
              }
            }
            const int blocks = (nb * per_block - p0 < 32 ? nb * per_block - p0 : 32) / per_block;
            for (int f = 0; f < 2 * blocks && ok; ++f, ++fill) {
              const int st = fill % L::kStages;
              if (fill >= L::kStages) wait(sh.bars.kv_empty[st], (fill / L::kStages - 1) & 1);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              const int first = (f >> 1) * per_block;
              const int n = live - p0 - first < per_block ? live - p0 - first : per_block;
              if (lane == 0) mbar_arrive_expect_tx(bar(sh.bars.kv_full[st]), n * L::kPlanes * a.P * 128);
              __syncwarp();
              if (lane >= first && lane < first + n) {
                const uint32_t dst = smem_u32(ring) + st * L::kTile + (lane - first) * a.P * 128;
                for (int pl = 0; pl < L::kPlanes; ++pl)
                  tma_load_4d(dst + pl * kPaPlane, (f & 1) ? &tm_v : &tm_k, bar(sh.bars.kv_full[st]), 64 * pl,
                              a.nhd ? x.kvh : 0, a.nhd ? 0 : x.kvh, id);
              }
            }
          }
        }
        fill = __shfl_sync(0xffffffffu, fill, 0);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      // every load has to land before the CTA may exit
      if (lane == 0) {
        if (n_q > 0 && !mbar_wait(bar(sh.bars.q_full), (n_q - 1) & 1)) err |= HPC_DEV_TIMEOUT;
        for (uint32_t f = fill > L::kStages ? fill - L::kStages : 0; f < fill; ++f)
          if (!mbar_wait(bar(sh.bars.kv_full[f % L::kStages]), (f / L::kStages) & 1)) err |= HPC_DEV_TIMEOUT;
      }
      if (err) atomicOr(a.status, err);
      __syncwarp();
    } else if (warp == kPaCheckWarp) {
      // ------------------------------------------------------------------ values that are not finite
      // In a block that some row of the unit sees only in part, a weight of 0 does not remove an infinity or
      // a NaN: such blocks of V are looked through while the others work, and a unit with a find is done row by row.
      int stage = 0;
      uint32_t phase = 0;
      for (int32_t n_unit = 0;; ++n_unit) {
        const int slot = n_unit % kPaTileRing;
        wait(sh.bars.unit_full[slot], (n_unit / kPaTileRing) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int32_t valid = sh.unit[slot].valid, keys = sh.unit[slot].keys;
        const int32_t from = sh.unit[slot].from;
        const int32_t whole = a.causal ? sh.unit[slot].vis : keys;  // keys that every row of the unit sees
        const int nb = max(sh.unit[slot].blocks[0], sh.unit[slot].blocks[1]);
        if (!valid) break;
        bool found = false;
        for (int f = 0; f < 2 * nb && ok; ++f) {
          wait(sh.bars.kv_full[stage], phase);
          ok = __all_sync(0xffffffffu, ok);
          const int32_t first = (from + (f >> 1)) * kPaKeys;
          if (ok && (f & 1) && whole < keys && first + kPaKeys > whole) {
            const int32_t rows = keys - first < kPaKeys ? keys - first : kPaKeys;  // those past it are zeroed
            // 0 * v added up is 0 for finite v, and a NaN from the first one that is not
            __nv_bfloat162 sum[4] = {};
            const __nv_bfloat162 zero = {};
            for (int pl = 0; pl < L::kPlanes; ++pl) {
              const uint8_t* vt = ring + stage * L::kTile + pl * kPaPlane;
#pragma unroll 8
              for (int i = lane; i < rows * 8; i += 32) {
                const uint4 w = *reinterpret_cast<const uint4*>(vt + i * 16);
                sum[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.x), zero, sum[0]);
                sum[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.y), zero, sum[1]);
                sum[2] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.z), zero, sum[2]);
                sum[3] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.w), zero, sum[3]);
              }
            }
            const float2 all = __bfloat1622float2(__hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3])));
            found |= !(all.x == 0.f) || !(all.y == 0.f);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(sh.bars.kv_empty[stage]));
          if (++stage == L::kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        found = __any_sync(0xffffffffu, found);
        if (lane == 0) {
          sh.found[slot] = found;
          mbar_arrive(bar(sh.bars.checked[slot]));
          mbar_arrive(bar(sh.bars.unit_free[slot]));
        }
      }
      if (err && lane == 0) atomicOr(a.status, err);
    } else if (warp == kPaScoreWarp || warp == kPaValueWarp) {
      // ------------------------------------------------------------------ products (whole warp, lane 0 issues)
      // One warp issues S = Q . K^T, another O += P . V. Issuing blocks for about as long as the product runs, so
      // that with one warp for both every wait in between would leave the tensor cores idle.
      const bool scores = warp == kPaScoreWarp;
      constexpr uint32_t kIdS = umma::idesc(128, 128, false), kIdO = umma::idesc(128, D, true);
      constexpr uint32_t kStep = L::kTile >> 4;  // a ring stage, in descriptor units
      const uint32_t lead = lane == 0;
      const uint64_t q_desc = umma_desc(smem_u32(smem), 16, 1024, 2);
      const uint64_t ring_desc = umma_desc(smem_u32(ring), scores ? 16 : kPaPlane, 1024, 2);
      int stage = scores ? 0 : 1;  // ring position of K_j (V_j): stage and phase
      uint32_t phase = 0;
      auto wait_all = [&](uint64_t& b, uint32_t parity) -> bool {
        ok = __all_sync(0xffffffffu, ok && mbar_wait(smem_u32(&b), parity, a.limit_ns));
        if (!ok) err = HPC_DEV_TIMEOUT;
        return ok;
      };
      uint32_t done[2] = {0, 0};  // products of tile A, B issued so far: phases of the tile's barriers
      int prev = -1;              // the tile of the last S
      int32_t n_q = 0;
      for (int32_t n_unit = 0;; ++n_unit) {
        const int slot = n_unit % kPaTileRing;
        if (!wait_all(sh.bars.unit_full[slot], (n_unit / kPaTileRing) & 1)) break;
        // the same for every lane; the exchange tells the compiler so
        const int32_t valid = __shfl_sync(0xffffffffu, sh.unit[slot].valid, 0);
        const int nb0 = __shfl_sync(0xffffffffu, sh.unit[slot].blocks[0], 0);
        const int nb1 = __shfl_sync(0xffffffffu, sh.unit[slot].blocks[1], 0);
        if (lane == 0) mbar_arrive(bar(sh.bars.unit_free[slot]));
        __syncwarp();
        if (!valid) break;
        const int nb = nb0 > nb1 ? nb0 : nb1;
        if (nb == 0) continue;
        if (scores) {
          if (!wait_all(sh.bars.q_full, n_q & 1)) break;
          ++n_q;
        }
        for (int j = 0; j < nb && ok; ++j) {
          if (!wait_all(sh.bars.kv_full[stage], phase)) break;
          const uint64_t at = ring_desc + static_cast<uint32_t>(stage) * kStep;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (j >= (t == 0 ? nb0 : nb1)) continue;
            if (scores) {
              // once the softmax that the last S was for has read it
              if (prev >= 0) wait_all(sh.bars.s_read[prev], ((prev == 0 ? done[0] : done[1]) - 1) & 1);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * kPaPlane + 32 * (kk & 3)) >> 4;
                umma::mma_ss(tmem, q_desc + t * kStep + off, at + off, kIdS, kk > 0, lead);
              }
              umma::commit(bar(sh.bars.s_full[t]), lead);
              prev = t;
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) {  // the parts of P as they come
                wait_all(sh.bars.p_full[t][h], done[t] & 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kPaKeys / 16; ++kk)
                  if ((kk < 2 * kPaSplit) == (h == 0))
                    umma::mma_ts(tmem + 256 + 128 * t, tmem + 128 + 64 * t + 8 * kk, at + 128 * kk, kIdO,
                                 (j > 0 || kk > 0) ? 1u : 0u, lead);
              }
              umma::commit(bar(sh.bars.pv_done[t]), lead);
            }
            ++done[t];
          }
          umma::commit(bar(sh.bars.kv_empty[stage]), lead);
          if (scores && j == nb - 1) umma::commit(bar(sh.bars.q_free), lead);  // the last read of Q
          stage += 2;
          if (stage >= L::kStages) {
            stage -= L::kStages;
            phase ^= 1;
          }
        }
      }
      // the products in flight read shared and tensor memory
      umma::commit(bar(sh.bars.drained[scores]), lead);
      if (!mbar_wait(bar(sh.bars.drained[scores]), 0)) err |= HPC_DEV_TIMEOUT;
      if (err && lane == 0) atomicOr(a.status, err);
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kPaScoreWarp) {
    tc_fence_after();
    tmem_free(tmem, kPaCols);
  }
}

// Joins the parts of cut units by log-sum-exp: M = max m_i, w_i = 2^(c (m_i - M)), out = sum w_i O_i / sum w_i l_i.
// A block takes four columns of a tile, a thread per row, so that the parts are read side by side and the whole
// GPU reads them. Parts are added in order: the same result every time. With 4 CTAs for each SM a call of 900 queries on 2400
// keys of 16/2 heads takes 46 us, with 8 of them 38, with 16 36; where nothing is cut 16 take 1 us more.
constexpr int kPaJoin = 8;      // parts loaded together
constexpr int kPaJoinCtas = 8;  // per SM: all that fit
template <int D>
__global__ void __launch_bounds__(kPaRows) prompt_join_kernel(const PaArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t cuts = a.work[1];
  const int row = threadIdx.x, tokens_per_tile = kPaRows / a.group;
  constexpr int64_t kTileFloats = kPaRows * (D + 2);
  for (uint32_t u = blockIdx.x; u < cuts * (2 * (D / 4)); u += gridDim.x) {
    const int c4 = u % (D / 4), t = u / (D / 4) % 2;
    const PaCut x = a.cuts[u / (2 * (D / 4))];
    const int parts = x.parts[t], token = x.q0 + t * tokens_per_tile + row / a.group;
    if (parts <= 1 || token >= x.q_end) continue;
    const float* first = a.partial + (static_cast<int64_t>(x.slot) * 2 + t) * kTileFloats;
    const int64_t apart = static_cast<int64_t>(a.Hkv) * 2 * kTileFloats;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < parts; i0 += kPaJoin) {
      float mi[kPaJoin], li[kPaJoin];
      float4 v[kPaJoin];
#pragma unroll
      for (int i = 0; i < kPaJoin; ++i) {
        const bool have = i0 + i < parts;
        const float* at = first + (have ? i0 + i : i0) * apart;
        mi[i] = have ? at[row] : -INFINITY;
        li[i] = have ? at[kPaRows + row] : 0.f;
        v[i] = reinterpret_cast<const float4*>(at + 2 * kPaRows)[c4 * kPaRows + row];
      }
      float top = m;
#pragma unroll
      for (int i = 0; i < kPaJoin; ++i) top = fmaxf(top, mi[i]);
      const float shrink = m == -INFINITY ? 0.f : ex2((m - top) * a.scale_log2);
      m = top;
      l = l == 0.f ? 0.f : l * shrink;
      o = make_float4(o.x * shrink, o.y * shrink, o.z * shrink, o.w * shrink);
#pragma unroll
      for (int i = 0; i < kPaJoin; ++i) {
        // a part without keys has no weight (its O may be anything), but a NaN of its sum stays
        const float w = mi[i] == -INFINITY ? 0.f : ex2((mi[i] - m) * a.scale_log2);
        l += li[i] != li[i] ? li[i] : li[i] * w;
        if (w != 0.f) o = make_float4(fmaf(w, v[i].x, o.x), fmaf(w, v[i].y, o.y), fmaf(w, v[i].z, o.z), fmaf(w, v[i].w, o.w));
      }
    }
    const bool some = l > 0.f || l != l;
    const float inv = some ? 1.f / l : 0.f;
    const int64_t at = static_cast<int64_t>(token) * a.Hq + x.kvh * a.group + row % a.group;
    *reinterpret_cast<uint2*>(a.out + at * D + 4 * c4) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (a.lse && c4 == 0) a.lse[at] = some ? m * a.scale + logf(l) : -INFINITY;
  }
}

// ---------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 pa_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
}

// A map of 128-byte swizzled boxes [box3][box2][box1][64 elements].
int pa_map(CUtensorMap* map, const void* base, const uint64_t (&dims)[4], const uint64_t (&strides)[3],
           const uint32_t (&box)[4]) {
  auto fn = pa_encode();
  if (!fn) return fail(HPC_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const uint32_t ones[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
                        reinterpret_cast<const cuuint64_t*>(dims), reinterpret_cast<const cuuint64_t*>(strides),
                        reinterpret_cast<const cuuint32_t*>(box), reinterpret_cast<const cuuint32_t*>(ones),
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(HPC_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return HPC_OK;
}

// [tokens][heads][D] with the given strides (elements), in boxes of `box_heads` x `box_tokens`.
int pa_packed_map(CUtensorMap* map, const void* base, int64_t tokens, int32_t heads, int32_t D, int64_t token_stride,
                  int64_t head_stride, uint32_t box_heads, uint32_t box_tokens) {
  const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(heads), static_cast<uint64_t>(tokens), 1};
  const uint64_t strides[3] = {static_cast<uint64_t>(head_stride) * 2, static_cast<uint64_t>(token_stride) * 2,
                               static_cast<uint64_t>(token_stride) * 2 * static_cast<uint64_t>(tokens)};
  const uint32_t box[4] = {64, box_heads, box_tokens, 1};
  return pa_map(map, base, dims, strides, box);
}

template <int D, bool kPaged>
int pa_launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, PaArgs a, cudaStream_t stream) {
  using L = PaLayout<D>;
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  auto kern = prompt_attention_kernel<D, kPaged>;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
    if (e != cudaSuccess) return launched(e, "cudaFuncSetAttribute(prompt_attention_kernel)");
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  const int sms = device_sm_count() > 0 ? device_sm_count() : 148;
  // units of one or two tiles: at most one part-filled per sequence and kv head
  auto units = [&](int64_t rows) { return (a.tokens / (rows / a.group) + (a.batch < a.tokens ? a.batch : a.tokens)) * a.Hkv; };
  a.single = units(kPaRows) <= (a.slots > 0 ? sms / 2 : sms);
  const int64_t most = units(a.single ? kPaRows : 2 * kPaRows);
  a.unsorted = a.slots == 0 && most <= sms;
  const int grid = a.slots > 0 ? sms : static_cast<int>(most < sms ? most : sms);
  const cudaError_t e = launch_pdl(kern, dim3(grid), dim3(kPaThreads), static_cast<size_t>(L::kBytes), stream, q, k, v, a);
  const int rc = launched(e, "prompt_attention_kernel");
  if (rc != HPC_OK || a.slots == 0) return rc;
  const cudaError_t j = launch_pdl(prompt_join_kernel<D>, dim3(kPaJoinCtas * sms), dim3(kPaRows), 0, stream, a);
  return launched(j, "prompt_join_kernel");
}

size_t pa_slot_bytes(int32_t head_dim) { return static_cast<size_t>(2) * kPaRows * (head_dim + 2) * sizeof(float); }

// Two parts for every SM: units are cut into a share of the blocks each.
size_t pa_most_slots() {
  const size_t n = 2 * static_cast<size_t>(device_sm_count() > 0 ? device_sm_count() : 148);
  return n < kPaCuts ? n : kPaCuts;
}

// What both entry points check of the queries and the shape; fills the common arguments.
int pa_common(const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t tokens, const int32_t* cu_seqlens,
              int32_t batch, int32_t num_heads, int32_t kv_heads, int32_t head_dim, float sm_scale, void* out,
              float* lse, uint32_t* work, void* partial, size_t partial_bytes, int64_t max_keys, uint32_t* status,
              PaArgs& a) {
  if (tokens < 0 || tokens > INT32_MAX - 1024) return fail(HPC_ERR_ARG, "tokens out of range");
  if (!cu_seqlens || !status || !work || (tokens > 0 && (!q || !out)) || (partial_bytes > 0 && !partial))
    return fail(HPC_ERR_ARG, "null pointer argument");
  if (batch < 1 || num_heads < 1 || kv_heads < 1) return fail(HPC_ERR_ARG, "sizes must be >= 1");
  if (num_heads % kv_heads) return fail(HPC_ERR_SHAPE, "num_heads %% kv_heads != 0");
  const int32_t g = num_heads / kv_heads;
  if (g != 1 && g != 2 && g != 4 && g != 8) return fail(HPC_ERR_SHAPE, "num_heads / kv_heads must be 1, 2, 4 or 8");
  if (head_dim != 64 && head_dim != 128) return fail(HPC_ERR_SHAPE, "head_dim must be 64 or 128");
  if (!(sm_scale > 0.f) || !std::isfinite(sm_scale)) return fail(HPC_ERR_ARG, "sm_scale must be positive and finite");
  a.cu_q = cu_seqlens;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.status = status;
  a.work = work;
  if (!aligned16(partial)) return fail(HPC_ERR_ALIGN, "partial must be 16-byte aligned");
  // units are cut only where some sequence can be long enough
  if (max_keys > HPC_PROMPT_SPLIT_KEYS && partial_bytes > kPaCutBytes) {
    const size_t room = (partial_bytes - kPaCutBytes) / pa_slot_bytes(head_dim);
    a.slots = static_cast<int32_t>(room < pa_most_slots() ? room : pa_most_slots());
    a.cuts = static_cast<PaCut*>(partial);
    a.partial = reinterpret_cast<float*>(static_cast<char*>(partial) + kPaCutBytes);
  }
  a.limit_ns = kWaitLimitNs + (max_keys > 0 ? static_cast<uint64_t>(max_keys) * kPaRowsNs : 0);
  a.tokens = tokens;
  a.scale = sm_scale;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.batch = batch;
  a.Hq = num_heads;
  a.Hkv = kv_heads;
  a.group = g;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  if (tokens == 0) return HPC_OK;
  if (!aligned16(q) || !aligned16(out)) return fail(HPC_ERR_ALIGN, "q and out must be 16-byte aligned");
  if (q_token_stride % 8 || q_head_stride % 8 || q_token_stride < 0 || q_head_stride < 0)
    return fail(HPC_ERR_ALIGN, "strides must be multiples of 8 elements");
  return HPC_OK;
}

int pa_query_map(CUtensorMap* map, const PaArgs& a, int32_t head_dim) {
  return pa_packed_map(map, a.q, a.tokens, a.Hq, head_dim, a.q_token, a.q_head, a.group, kPaRows / a.group);
}

}  // namespace
}  // namespace hpc

using namespace hpc;

extern "C" size_t hpc_prompt_attention_partial_bytes(int32_t head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  return kPaCutBytes + pa_most_slots() * pa_slot_bytes(head_dim);
}

extern "C" int hpc_prompt_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                                    int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                                    int64_t v_head_stride, int64_t tokens, int64_t kv_tokens, const int32_t* cu_seqlens,
                                    const int32_t* cu_seqlens_k, int32_t batch, int32_t num_heads, int32_t kv_heads,
                                    int32_t head_dim, int32_t causal, float sm_scale, void* out, float* lse,
                                    uint32_t* work, void* partial, size_t partial_bytes, uint32_t* status, void* stream) {
  PaArgs a = {};
  CUtensorMap mq, mk, mv;
  int rc = pa_common(q, q_token_stride, q_head_stride, tokens, cu_seqlens, batch, num_heads, kv_heads, head_dim, sm_scale,
                     out, lse, work, partial, partial_bytes, kv_tokens, status, a);
  if (rc != HPC_OK) return rc;
  if (kv_tokens < 0 || kv_tokens > INT32_MAX - 1024) return fail(HPC_ERR_ARG, "kv_tokens out of range");
  if (!cu_seqlens_k && kv_tokens != tokens)
    return fail(HPC_ERR_ARG, "without cu_seqlens_k the keys are the tokens (kv_tokens == tokens)");
  if (kv_tokens > 0 && (!k || !v)) return fail(HPC_ERR_ARG, "null pointer argument");
  if (tokens == 0) return HPC_OK;
  if (!aligned16(k) || !aligned16(v)) return fail(HPC_ERR_ALIGN, "k and v must be 16-byte aligned");
  if ((k_token_stride | k_head_stride | v_token_stride | v_head_stride) % 8 || k_token_stride < 0 || k_head_stride < 0 ||
      v_token_stride < 0 || v_head_stride < 0)
    return fail(HPC_ERR_ALIGN, "strides must be multiples of 8 elements");
  a.cu_k = cu_seqlens_k ? cu_seqlens_k : cu_seqlens;
  a.kv_tokens = kv_tokens;
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.k_token = k_token_stride;
  a.k_head = k_head_stride;
  a.v_token = v_token_stride;
  a.v_head = v_head_stride;
  a.causal = causal != 0;
  if ((rc = pa_query_map(&mq, a, head_dim)) != HPC_OK) return rc;
  if (kv_tokens > 0) {
    if ((rc = pa_packed_map(&mk, k, kv_tokens, kv_heads, head_dim, k_token_stride, k_head_stride, 1, kPaKeys)) != HPC_OK)
      return rc;
    if ((rc = pa_packed_map(&mv, v, kv_tokens, kv_heads, head_dim, v_token_stride, v_head_stride, 1, kPaKeys)) != HPC_OK)
      return rc;
  } else {
    mk = mv = mq;  // never loaded from: no sequence has keys
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return head_dim == 128 ? pa_launch<128, false>(mq, mk, mv, a, st) : pa_launch<64, false>(mq, mk, mv, a, st);
}

extern "C" int hpc_prompt_attention_paged(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                          const void* k_pages, const void* v_pages, hpc_dtype kv_dtype,
                                          hpc_kv_layout kv_layout, int32_t num_pages, int32_t page_size,
                                          const int32_t* block_table, int32_t max_pages_per_req,
                                          const int32_t* seq_lens, int64_t tokens, const int32_t* cu_seqlens,
                                          int32_t batch, int32_t num_heads, int32_t kv_heads, int32_t head_dim,
                                          float sm_scale, void* out, float* lse, uint32_t* work, void* partial,
                                          size_t partial_bytes, uint32_t* status, void* stream) {
  PaArgs a = {};
  CUtensorMap mq, mk, mv;
  int rc = pa_common(q, q_token_stride, q_head_stride, tokens, cu_seqlens, batch, num_heads, kv_heads, head_dim, sm_scale,
                     out, lse, work, partial, partial_bytes, static_cast<int64_t>(max_pages_per_req) * page_size, status,
                     a);
  if (rc != HPC_OK) return rc;
  if (!k_pages || !v_pages || !block_table || !seq_lens) return fail(HPC_ERR_ARG, "null pointer argument");
  if (kv_dtype != HPC_BF16) return fail(HPC_ERR_DTYPE, "the paged prompt attention reads BF16 caches");
  if (kv_layout != HPC_HND && kv_layout != HPC_NHD) return fail(HPC_ERR_ARG, "kv_layout must be HND or NHD");
  if (num_pages < 1 || max_pages_per_req < 1) return fail(HPC_ERR_ARG, "sizes must be >= 1");
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return fail(HPC_ERR_SHAPE, "page_size must be 16, 32, 64 or 128");
  if (static_cast<int64_t>(max_pages_per_req) * page_size > INT32_MAX - 1024)
    return fail(HPC_ERR_SHAPE, "max_pages_per_req x page_size out of range");
  if (!aligned16(k_pages) || !aligned16(v_pages)) return fail(HPC_ERR_ALIGN, "caches must be 16-byte aligned");
  if (tokens == 0) return HPC_OK;
  a.k = static_cast<const __nv_bfloat16*>(k_pages);
  a.v = static_cast<const __nv_bfloat16*>(v_pages);
  a.table = block_table;
  a.seq_lens = seq_lens;
  a.max_pages = max_pages_per_req;
  a.P = page_size;
  a.num_pages = num_pages;
  a.nhd = kv_layout == HPC_NHD;
  a.causal = 1;
  const uint64_t D = head_dim, H = kv_heads, P = page_size;
  const uint64_t dims[4] = {D, a.nhd ? H : P, a.nhd ? P : H, static_cast<uint64_t>(num_pages)};
  const uint64_t strides[3] = {D * 2, D * 2 * dims[1], D * 2 * H * P};
  const uint32_t box[4] = {64, a.nhd ? 1u : static_cast<uint32_t>(P), a.nhd ? static_cast<uint32_t>(P) : 1u, 1};
  if ((rc = pa_query_map(&mq, a, head_dim)) != HPC_OK) return rc;
  if ((rc = pa_map(&mk, k_pages, dims, strides, box)) != HPC_OK) return rc;
  if ((rc = pa_map(&mv, v_pages, dims, strides, box)) != HPC_OK) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return head_dim == 128 ? pa_launch<128, true>(mq, mk, mv, a, st) : pa_launch<64, true>(mq, mk, mv, a, st);
}
