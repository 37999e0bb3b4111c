// Upkeep of a paged KV cache on the device: resize (grow and free), fork, compact, and the copy of
// the pages that those list.
//
// The state is a block table int32 [rows][max_pages], the lengths, and one reference count per
// page (0 = free); there is no free list to keep in step. The pages taken are always the lowest
// free ones, in request order, so a result depends on the inputs alone and not on which thread
// came first (the counts change by integer atomics, whose order does not matter).
//
// Each planner is one launch of one cluster of 8 CTAs x 1024 threads. Its phases need a barrier over
// all of the state (every release before the free pages are counted, every count before a page is
// handed out); a cluster barrier costs a few hundred ns where another launch costs microseconds,
// and the tables of a serving batch (64 K entries, 64 K pages) are a few hundred KB, which eight SMs
// stream in a few microseconds. Free pages are found by a scan of the counts: each of the 256 warps
// owns a contiguous run of pages, counts its free ones by ballot, and the warps' counts are prefixed
// through distributed shared memory.
//
// The data is moved by pages_copy_kernel, for any number of caches (the K and V of every layer
// share the table), from the list a planner leaves on the device. A destination was free and a
// source is live, so no page is both.
//
// The planners are bound by latency (about eight dependent accesses and three to four barriers) and, in large pools, by
// what eight SMs copy, about half each: a resize of 256 requests in a pool of 40000 pages takes 11.5 us, of 4 requests
// in one of 512 5.7 us; forks 13.7 and 7.2 us. Each warp reads its run of counts once and keeps it as bits; lengths and
// entries that later phases want are loaded under the copy of the counts; divisions are 32-bit (12.9 and 6.6 us without
// the three).
#include "hpc_common.cuh"

namespace hpc {
namespace {

constexpr int kPgCtas = 8;        // one portable cluster
constexpr int kPgThreads = 1024;  // per CTA
constexpr int kPgWarps = kPgThreads / 32;
constexpr int kPgAllWarps = kPgCtas * kPgWarps;
constexpr int kPgHeld = 8;
constexpr int kPgMaxRows = 8192;  // rows whose needs fit in shared memory (12 bytes each at most)

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// All threads of the cluster; orders their global and shared memory accesses. Not the .aligned forms: the
// threads of a warp may come here from different branches.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Store to the same shared variable of CTA `rank` of the cluster.
__device__ __forceinline__ void st_remote(uint32_t saddr, uint32_t rank, int32_t v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Arrays that other CTAs of the cluster change: read past L1, and not moved over a barrier.
__device__ __forceinline__ int32_t ld_shared_state(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ int2 ld_shared_state(const int2* p) {
  int2 v;
  asm volatile("ld.global.cg.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}


// In place, the kN arrays s[k][0 .. n) -> exclusive prefix sums; their totals (whole block).
template <int kN>
__device__ __forceinline__ void block_prefix(int32_t* const (&s)[kN], int32_t n, int32_t (&red)[2][kPgWarps],
                                             int32_t (&total)[kN]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < kN; ++k) total[k] = 0;
  for (int32_t i0 = 0; i0 < n; i0 += kPgThreads) {
    const int32_t i = i0 + static_cast<int32_t>(threadIdx.x);
    int32_t v[kN], x[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k) x[k] = v[k] = i < n ? s[k][i] : 0;  // the thread's own entry
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int32_t y = __shfl_up_sync(0xffffffffu, x[k], o);
        if (lane >= o) x[k] += y;
      }
    }
    if (i0 > 0) __syncthreads();  // the sums before are read
    if (lane == 31) {
#pragma unroll
      for (int k = 0; k < kN; ++k) red[k][warp] = x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int32_t w = red[k][lane];
      if (i < n) s[k][i] = total[k] + x[k] - v[k];
      const int32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
      if (i < n) s[k][i] += before;
      total[k] += __reduce_add_sync(0xffffffffu, w);
    }
  }
  __syncthreads();
}

// Largest i with s[i] <= k, for an ascending prefix s[0 .. n) with s[0] = 0.
__device__ __forceinline__ int32_t prefix_find(const int32_t* s, int32_t n, int32_t k) {
  int32_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (s[mid] <= k) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct PgShared {
  int32_t red[2][kPgWarps];
  int32_t a[kPgCtas];  // per CTA of the cluster
  int32_t wa[kPgWarps];
};

// The run of pages [begin, end) of a warp: the pool in 256 contiguous runs.
__device__ __forceinline__ void warp_run(int32_t num_pages, int32_t gw, int32_t& begin, int32_t& end) {
  const int64_t per = (((static_cast<int64_t>(num_pages) + kPgAllWarps - 1) / kPgAllWarps) + 31) & ~int64_t(31);
  const int64_t b = per * gw, e = b + per;
  begin = static_cast<int32_t>(b < num_pages ? b : num_pages);
  end = static_cast<int32_t>(e < num_pages ? e : num_pages);
}

__device__ __forceinline__ uint32_t low_bits(int32_t n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }

// Which of the 32 pages from p0 on are in use (whole warp; none at or past the end of the run).
__device__ __forceinline__ uint32_t used_pages(const int32_t* ref, int32_t p0, int32_t end) {
  const int32_t p = p0 + (threadIdx.x & 31);
  return __ballot_sync(0xffffffffu, p < end && ld_shared_state(ref + p) != 0);
}

// A warp's run of pages as bits, read once for counting and for handing out: kPgHeld groups of 32 in registers (all
// of a pool of 65536), the rest from memory again. `pick` turns the bits of a group into those that are asked for.
struct PgRun {
  const int32_t* ref;
  int32_t begin, end;
  uint32_t used[kPgHeld];

  __device__ __forceinline__ PgRun(const int32_t* r, int32_t num_pages, int32_t gw) : ref(r) {
    warp_run(num_pages, gw, begin, end);
    int32_t c[kPgHeld];
#pragma unroll
    for (int g = 0; g < kPgHeld; ++g) {
      const int32_t p = begin + 32 * g + static_cast<int32_t>(threadIdx.x & 31);
      c[g] = p < end ? ld_shared_state(ref + p) : 0;
    }
#pragma unroll
    for (int g = 0; g < kPgHeld; ++g) used[g] = __ballot_sync(0xffffffffu, c[g] != 0);
  }
  __device__ __forceinline__ uint32_t valid(int32_t p0) const { return low_bits(end - p0); }

  template <typename F>
  __device__ __forceinline__ int32_t count(F pick) const {
    int32_t n = 0;
#pragma unroll
    for (int g = 0; g < kPgHeld; ++g) n += __popc(pick(used[g], begin + 32 * g));
    for (int32_t p0 = begin + 32 * kPgHeld; p0 < end; p0 += 32) n += __popc(pick(used_pages(ref, p0, end), p0));
    return n;
  }
  // visit(page, rank) for the pages that are picked, ranks ascending from `rank`, until `limit`.
  template <typename F, typename V>
  __device__ __forceinline__ void visit(int32_t rank, int32_t limit, F pick, V visit) const {
    const int lane = threadIdx.x & 31;
    auto group = [&](uint32_t m, int32_t p0) {
      const int32_t k = rank + __popc(m & ((1u << lane) - 1u));
      if ((m >> lane & 1u) && k < limit) visit(p0 + lane, k);
      rank += __popc(m);
    };
#pragma unroll 1
    for (int g = 0; g < kPgHeld && rank < limit; ++g) {
      uint32_t m = used[0];
#pragma unroll
      for (int i = 1; i < kPgHeld; ++i) m = g == i ? used[i] : m;
      if (begin + 32 * g < end) group(pick(m, begin + 32 * g), begin + 32 * g);
    }
    for (int32_t p0 = begin + 32 * kPgHeld; p0 < end && rank < limit; p0 += 32)
      group(pick(used_pages(ref, p0, end), p0), p0);
  }
};

// Per-warp counts -> this warp's exclusive prefix over the cluster and the total. Every thread of
// the cluster calls it, after a first cluster_sync (a CTA's shared memory may be written only once it
// runs); cta[] is the array of the CTAs' sums and warps[] the CTA's warps' counts.
__device__ void cluster_prefix(int32_t count, int32_t* cta, int32_t* warps, int32_t& before, int32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_rank();
  if (lane == 0) warps[warp] = count;
  __syncthreads();
  const int32_t mine = __reduce_add_sync(0xffffffffu, warps[lane]);
  if (threadIdx.x < kPgCtas) st_remote(smem_u32(cta + rank), threadIdx.x, mine);
  cluster_sync();
  before = total = 0;
  for (int c = 0; c < kPgCtas; ++c) {
    total += cta[c];
    if (c < static_cast<int>(rank)) before += cta[c];
  }
  before += __reduce_add_sync(0xffffffffu, lane < warp ? warps[lane] : 0);
}

__device__ __forceinline__ void copy_counts(const int32_t* in, int32_t* out, int32_t n, int32_t gtid) {
  if (in == out) return;
  constexpr int kAll = kPgCtas * kPgThreads;
  if (((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0) {
    const int32_t n4 = n >> 2;
#pragma unroll 4
    for (int32_t i = gtid; i < n4; i += kAll)
      reinterpret_cast<int4*>(out)[i] = reinterpret_cast<const int4*>(in)[i];
    for (int32_t i = 4 * n4 + gtid; i < n; i += kAll) out[i] = in[i];
  } else {
    for (int32_t i = gtid; i < n; i += kAll) out[i] = in[i];
  }
}

struct PgArgs {
  const int32_t* table_in;
  int32_t* table_out;
  const int32_t* lens;      // lengths of the rows of table_in
  const int32_t* want;      // resize: new lengths; fork: parents
  int32_t* lens_out;        // fork
  const int32_t* ref_in;
  int32_t* ref_out;
  int32_t* page_map;        // compact
  int2* moves;              // (source page, destination page)
  int32_t* n_moves;
  uint32_t* status;
  int32_t rows_in, rows_out, max_pages, num_pages, page_size, max_len;
};

// Lengths and page_size fit in 31 bits together (max_len = max_pages * page_size): 32-bit divisions.
__device__ __forceinline__ bool len_ok(const PgArgs& a, int32_t n) { return n >= 0 && n <= a.max_len; }
__device__ __forceinline__ int32_t held(const PgArgs& a, int32_t n) {
  return static_cast<int32_t>((static_cast<uint32_t>(n) + static_cast<uint32_t>(a.page_size) - 1u) / static_cast<uint32_t>(a.page_size));
}
__device__ __forceinline__ int32_t column(const PgArgs& a, int32_t n) {  // of token n
  return static_cast<int32_t>(static_cast<uint32_t>(n) / static_cast<uint32_t>(a.page_size));
}
__device__ __forceinline__ bool part_filled(const PgArgs& a, int32_t n) { return column(a, n) * a.page_size != n; }

// ---- resize -----------------------------------------------------------------------------
// Row r goes from lens[r] to want[r] tokens. Pages past the new length are released (count - 1); a row
// that grows takes pages for its new columns. A row that grows inside a part-filled page which
// others still hold (count > 1 after the releases) first moves to a copy of it.
__global__ void __cluster_dims__(kPgCtas, 1, 1) __launch_bounds__(kPgThreads, 1) pages_resize_kernel(const PgArgs a) {
  extern __shared__ int32_t s_dyn[];
  __shared__ PgShared sh;
  int32_t* s_need = s_dyn;               // [rows] -> exclusive prefix
  int32_t* s_cow = s_dyn + a.rows_out;   // [rows] 0 / 1 -> exclusive prefix
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int32_t gtid = static_cast<int32_t>(rank) * kPgThreads + static_cast<int32_t>(threadIdx.x);
  const int32_t gw = gtid >> 5;
  const int32_t M = a.max_pages, rows = a.rows_out;
  pdl_wait();
  pdl_launch_dependents();

  // Lengths and entries that later phases want, of this warp's and this thread's first rows: loaded under the copy.
  const int32_t t = static_cast<int32_t>(threadIdx.x);
  const int32_t row_old = gw < rows ? a.lens[gw] : 0, row_new = gw < rows ? a.want[gw] : 0;
  const int32_t own_old = t < rows ? a.lens[t] : 0, own_new = t < rows ? a.want[t] : 0;
  auto lengths = [&](int32_t r, int32_t& o, int32_t& n) {  // of a row of the warp
    o = r == gw ? row_old : a.lens[r];
    n = r == gw ? row_new : a.want[r];
    return len_ok(a, o) && len_ok(a, n);
  };
  copy_counts(a.ref_in, a.ref_out, a.num_pages, gtid);
  // the first 32 entries that the warp's first row releases
  const bool row_shrinks = gw < rows && len_ok(a, row_old) && len_ok(a, row_new) && row_new < row_old;
  const int32_t row_from = row_shrinks ? held(a, row_new) + lane : 0;
  const int32_t row_entry = row_shrinks && row_from < held(a, row_old) ? a.table_in[static_cast<int64_t>(gw) * M + row_from] : 0;
  // the part-filled page that the thread's first row grows in
  const bool own_grows = t < rows && len_ok(a, own_old) && len_ok(a, own_new) && own_new > own_old;
  const int32_t own_page = own_grows && part_filled(a, own_old) ? a.table_in[static_cast<int64_t>(t) * M + column(a, own_old)] : 0;

  // The entries that stay, and -1 past them; the new ones are written below by whoever holds the page. A new
  // table is written now, under the latencies of the first phases, and an old one once nothing can fail.
  auto keep_entries = [&]() {
    for (int32_t r = gw; r < rows; r += kPgAllWarps) {
      int32_t o, n;
      const bool ok = lengths(r, o, n);
      const int32_t from = ok ? held(a, o) : M, to = ok ? held(a, n) : M;
      const int32_t keep = from < to ? from : to;
      const int32_t* in = a.table_in + static_cast<int64_t>(r) * M;
      int32_t* out = a.table_out + static_cast<int64_t>(r) * M;
      if (in != out) {
#pragma unroll 8
        for (int32_t j = lane; j < keep; j += 32) out[j] = in[j];
      }
#pragma unroll 4
      for (int32_t j = to + lane; j < M; j += 32) out[j] = -1;
    }
  };
  if (a.table_in != a.table_out) keep_entries();
  cluster_sync();
  // releases; `sign` +1 takes them back
  auto release = [&](int32_t sign) {
    for (int32_t r = gw; r < rows; r += kPgAllWarps) {
      int32_t o, n;
      if (!lengths(r, o, n)) {
        if (lane == 0) atomicOr(a.status, HPC_DEV_BAD_SEQLEN);
        continue;
      }
      for (int32_t j = held(a, n) + lane; j < held(a, o); j += 32) {
        const int32_t p = r == gw && j == row_from ? row_entry : a.table_in[static_cast<int64_t>(r) * M + j];
        if (p >= 0 && p < a.num_pages) atomicAdd(a.ref_out + p, sign);
        else atomicOr(a.status, HPC_DEV_BAD_PAGE);
      }
    }
  };
  release(-1);
  cluster_sync();
  const PgRun run(a.ref_out, a.num_pages, gw);
  // what every row needs, in every CTA
  for (int32_t r = t; r < rows; r += kPgThreads) {
    const int32_t o = r == t ? own_old : a.lens[r], n = r == t ? own_new : a.want[r];
    int32_t need = 0, cow = 0;
    if (len_ok(a, o) && len_ok(a, n) && n > o) {
      need = held(a, n) - held(a, o);
      if (part_filled(a, o)) {
        const int32_t p = r == t ? own_page : a.table_in[static_cast<int64_t>(r) * M + column(a, o)];
        if (p < 0 || p >= a.num_pages) atomicOr(a.status, HPC_DEV_BAD_PAGE);
        else if (ld_shared_state(a.ref_out + p) > 1) cow = 1;
      }
    }
    s_need[r] = need + cow;
    s_cow[r] = cow;
  }
  int32_t totals[2];
  block_prefix<2>({s_need, s_cow}, rows, sh.red, totals);
  const int32_t total = totals[0], copies = totals[1];
  int32_t before, free_pages;
  auto is_free = [&](uint32_t used, int32_t p0) { return ~used & run.valid(p0); };
  cluster_prefix(run.count(is_free), sh.a, sh.wa, before, free_pages);
  const bool fits = total <= free_pages;
  if (gtid == 0) *a.n_moves = fits ? copies : 0;
  if (!fits) {
    // too few pages: the call changes nothing
    if (gtid == 0) atomicOr(a.status, HPC_DEV_CAPACITY);
    release(1);
    if (a.table_in != a.table_out)
      for (int64_t i = gtid; i < static_cast<int64_t>(rows) * M; i += kPgCtas * kPgThreads) a.table_out[i] = a.table_in[i];
    return;
  }
  if (a.table_in == a.table_out) keep_entries();
  run.visit(before, total, is_free, [&](int32_t p, int32_t k) {
    const int32_t r = prefix_find(s_need, rows, k);
    const int32_t o = a.lens[r];
    const bool cow = (r + 1 < rows ? s_cow[r + 1] : copies) != s_cow[r];
    const int32_t nth = k - s_need[r];
    const bool copy = cow && nth == 0;
    const int32_t j = copy ? column(a, o) : held(a, o) + nth - (cow ? 1 : 0);
    const int64_t i = static_cast<int64_t>(r) * M + j;
    if (copy) a.moves[s_cow[r]] = make_int2(a.table_in[i], p);  // the entry itself is this thread's
    a.table_out[i] = p;
    a.ref_out[p] = 1;
  });
  // The sources lose their sharer only once every warp has passed its free pages: a count that falls
  // to zero here must not be taken in this call (its data is still to be copied).
  if (copies > 0) {  // the same in every CTA
    cluster_sync();
    for (int32_t i = gtid; i < copies; i += kPgCtas * kPgThreads) {
      const int2 mv = ld_shared_state(a.moves + i);
      atomicAdd(a.ref_out + mv.x, -1);
    }
  }
}

// ---- fork -------------------------------------------------------------------------------
// New row r is old row want[r] (-1: empty). A page that several rows come to hold is shared, except
// a part-filled last page: the first child keeps it and every other takes a copy. Rows that no
// child names are released with it.
__global__ void __cluster_dims__(kPgCtas, 1, 1) __launch_bounds__(kPgThreads, 1) pages_fork_kernel(const PgArgs a) {
  extern __shared__ int32_t s_dyn[];
  __shared__ PgShared sh;
  int32_t* s_need = s_dyn;                  // [rows_out] -> exclusive prefix
  int32_t* s_kids = s_dyn + a.rows_out;     // [rows_in]
  int32_t* s_first = s_kids + a.rows_in;    // [rows_in] first child
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int32_t gtid = static_cast<int32_t>(rank) * kPgThreads + static_cast<int32_t>(threadIdx.x);
  const int32_t gw = gtid >> 5;
  const int32_t M = a.max_pages, rows = a.rows_out;
  pdl_wait();
  pdl_launch_dependents();

  // Parents and lengths of this thread's and this warp's first rows: loaded under the copy.
  const int32_t t = static_cast<int32_t>(threadIdx.x);
  const int32_t own_f = t < rows ? a.want[t] : -1, row_f = gw < rows ? a.want[gw] : -1;
  const int32_t src_len = gw < a.rows_in ? a.lens[gw] : 0;
  copy_counts(a.ref_in, a.ref_out, a.num_pages, gtid);
  const int32_t own_len = own_f >= 0 && own_f < a.rows_in ? a.lens[own_f] : 0;
  const int32_t row_len = row_f >= 0 && row_f < a.rows_in ? a.lens[row_f] : 0;
  for (int32_t s = threadIdx.x; s < a.rows_in; s += kPgThreads) {
    s_kids[s] = 0;
    s_first[s] = rows;
  }
  __syncthreads();
  for (int32_t r = threadIdx.x; r < rows; r += kPgThreads) {
    const int32_t f = r == t ? own_f : a.want[r];
    if (f >= 0 && f < a.rows_in) {
      atomicAdd(s_kids + f, 1);
      atomicMin(s_first + f, r);
    } else if (f != -1 && rank == 0) {
      atomicOr(a.status, HPC_DEV_BAD_INDEX);
    }
  }
  __syncthreads();
  // length of new row r (0 for an empty row or a parent with an invalid length)
  auto length = [&](int32_t r, int32_t& f) -> int32_t {
    f = a.want[r];
    if (f < 0 || f >= a.rows_in) return 0;
    const int32_t n = a.lens[f];
    return len_ok(a, n) ? n : 0;
  };
  for (int32_t r = threadIdx.x; r < rows; r += kPgThreads) {
    int32_t f = own_f;
    const int32_t n = r == t ? (len_ok(a, own_len) ? own_len : 0) : length(r, f);
    s_need[r] = part_filled(a, n) && s_first[f] != r ? 1 : 0;
  }
  int32_t totals[1];
  block_prefix<1>({s_need}, rows, sh.red, totals);
  const int32_t total = totals[0];
  // The rows, but for the pages that are copied: those are written below by whoever holds the new page.
  auto write_rows = [&](bool filled) {
    for (int32_t r = gw; r < rows; r += kPgAllWarps) {
      int32_t f = row_f;
      const int32_t n = !filled ? 0 : (r == gw ? (len_ok(a, row_len) ? row_len : 0) : length(r, f));
      if (lane == 0) a.lens_out[r] = n;
      const int32_t np = held(a, n);
      const bool fresh = (r + 1 < rows ? s_need[r + 1] : total) != s_need[r];
      const int32_t* in = a.table_in + static_cast<int64_t>(f < 0 ? 0 : f) * M;
      int32_t* out = a.table_out + static_cast<int64_t>(r) * M;
#pragma unroll 8
      for (int32_t j = lane; j < np - (fresh ? 1 : 0); j += 32) out[j] = in[j];
#pragma unroll 4
      for (int32_t j = np + lane; j < M; j += 32) out[j] = -1;
    }
  };
  write_rows(true);
  cluster_sync();  // the counts are copied
  // One change of count per held entry of an old row: its children less itself. Of a part-filled last
  // page one child keeps the reference and the others leave.
  auto recount = [&](int32_t sign) {
    for (int32_t s = gw; s < a.rows_in; s += kPgAllWarps) {
      const int32_t n = s == gw ? src_len : a.lens[s];
      if (!len_ok(a, n)) {
        if (lane == 0) atomicOr(a.status, HPC_DEV_BAD_SEQLEN);
        continue;
      }
      const int32_t kids = s_kids[s], np = held(a, n);
      for (int32_t j = lane; j < np; j += 32) {
        const int32_t p = a.table_in[static_cast<int64_t>(s) * M + j];
        const bool part = j == np - 1 && part_filled(a, n);
        const int32_t d = part ? (kids > 0 ? 0 : -1) : kids - 1;
        if (p < 0 || p >= a.num_pages) atomicOr(a.status, HPC_DEV_BAD_PAGE);
        else if (d != 0) atomicAdd(a.ref_out + p, sign * d);
      }
    }
  };
  recount(1);
  cluster_sync();
  const PgRun run(a.ref_out, a.num_pages, gw);
  int32_t before, free_pages;
  auto is_free = [&](uint32_t used, int32_t p0) { return ~used & run.valid(p0); };
  cluster_prefix(run.count(is_free), sh.a, sh.wa, before, free_pages);
  const bool fits = total <= free_pages;
  if (gtid == 0) {
    *a.n_moves = fits ? total : 0;
    if (!fits) atomicOr(a.status, HPC_DEV_CAPACITY);
  }
  if (!fits) {
    recount(-1);  // too few pages: the counts as they were, and empty rows
    write_rows(false);
    return;
  }
  run.visit(before, total, is_free, [&](int32_t p, int32_t k) {
    const int32_t r = prefix_find(s_need, rows, k);
    int32_t f;
    const int32_t n = length(r, f);
    const int32_t j = column(a, n);
    a.moves[k] = make_int2(a.table_in[static_cast<int64_t>(f) * M + j], p);
    a.table_out[static_cast<int64_t>(r) * M + j] = p;
    a.ref_out[p] = 1;
  });
}

// ---- compact ----------------------------------------------------------------------------
// With n pages in use, the i-th used page at or past n goes to the i-th free page below n.
__global__ void __cluster_dims__(kPgCtas, 1, 1) __launch_bounds__(kPgThreads, 1) pages_compact_kernel(const PgArgs a) {
  __shared__ PgShared sh;
  __shared__ int32_t s_c[kPgCtas], s_w[kPgWarps];
  const uint32_t rank = cluster_rank();
  const int32_t gtid = static_cast<int32_t>(rank) * kPgThreads + static_cast<int32_t>(threadIdx.x);
  const int32_t gw = gtid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  int32_t used_before, n, src0, srcs;
  const PgRun run(a.ref_in, a.num_pages, gw);
  cluster_sync();
  cluster_prefix(run.count([](uint32_t used, int32_t) { return used; }), s_c, s_w, used_before, n);
  auto is_src = [&](uint32_t used, int32_t p0) { return used & ~low_bits(n - p0); };
  auto is_dst = [&](uint32_t used, int32_t p0) { return ~used & low_bits(n - p0) & run.valid(p0); };
  cluster_prefix(run.count(is_src), sh.a, sh.wa, src0, srcs);
  // There are as many destinations: the used pages below n and the sources make up n. A run that has some starts
  // below n, behind begin - used_before free pages.
  run.visit(src0, srcs, is_src, [&](int32_t p, int32_t k) { a.moves[k].x = p; });
  run.visit(run.begin - used_before, srcs, is_dst, [&](int32_t p, int32_t k) { a.moves[k].y = p; });
#pragma unroll 4
  for (int32_t p = run.begin + (threadIdx.x & 31); p < run.end; p += 32) {
    const int32_t c = a.ref_in[p];
    if (a.ref_in != a.ref_out) a.ref_out[p] = c;
    a.page_map[p] = c != 0 ? p : -1;
  }
  if (gtid == 0) *a.n_moves = srcs;
  cluster_sync();
  for (int32_t k = gtid; k < srcs; k += kPgCtas * kPgThreads) {
    const int2 mv = ld_shared_state(a.moves + k);
    a.page_map[mv.x] = mv.y;
    a.ref_out[mv.y] = ld_shared_state(a.ref_out + mv.x);
    a.ref_out[mv.x] = 0;
  }
  cluster_sync();
  const int64_t entries = static_cast<int64_t>(a.rows_in) * a.max_pages;
#pragma unroll 4
  for (int64_t i = gtid; i < entries; i += kPgCtas * kPgThreads) {
    const int32_t p = a.table_in[i];
    if (p >= a.num_pages) atomicOr(a.status, HPC_DEV_BAD_PAGE);
    a.table_out[i] = p >= 0 && p < a.num_pages ? ld_shared_state(a.page_map + p) : -1;
  }
}

// ---- copy -------------------------------------------------------------------------------
constexpr int kPgCopyThreads = 256;
constexpr int kPgCopyVecs = 8;  // 16-byte loads in flight per thread
constexpr int kPgCopyCtas = 8;  // per SM
constexpr int kPgCopyChunk = kPgCopyThreads * kPgCopyVecs;
constexpr int kPgMaxCaches = 256;  // pointers in one launch's parameters

struct PgCaches {
  uint4* base[kPgMaxCaches];
};

// Work is (move, cache, 32 KB chunk of the page), dealt over the grid in that order. Of the 8 CTAs for each SM five fit at
// a time; the others even the work out. 268 MB read and written in 88 us (with four loads a thread, all CTAs resident, 96;
// with 32 CTAs for each SM 85, but a call that finds nothing to copy takes 6.3 instead of 3.1).
__global__ void __launch_bounds__(kPgCopyThreads)
    pages_copy_kernel(const __grid_constant__ PgCaches caches, int32_t n_caches, int64_t page_vecs, int32_t num_pages,
                      const int2* moves, const int32_t* n_moves, int32_t capacity, uint32_t* status) {
  pdl_wait();
  pdl_launch_dependents();
  int32_t n = *n_moves;
  if (n < 0 || n > capacity) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(status, HPC_DEV_CAPACITY);
    n = n < 0 ? 0 : capacity;
  }
  const int64_t chunks = (page_vecs + kPgCopyChunk - 1) / kPgCopyChunk;
  const int64_t per_move = chunks * n_caches;
  for (int64_t w = blockIdx.x; w < per_move * n; w += gridDim.x) {
    const int64_t m = w / per_move, rest = w - m * per_move;
    const int64_t cache = rest / chunks, chunk = rest - cache * chunks;
    const int2 mv = moves[m];
    if (mv.x < 0 || mv.x >= num_pages || mv.y < 0 || mv.y >= num_pages) {
      if (rest == 0 && threadIdx.x == 0) atomicOr(status, HPC_DEV_BAD_PAGE);
      continue;
    }
    const uint4* src = caches.base[cache] + mv.x * page_vecs;
    uint4* dst = caches.base[cache] + mv.y * page_vecs;
    const int64_t i0 = chunk * kPgCopyChunk + threadIdx.x;
    uint4 v[kPgCopyVecs];
#pragma unroll
    for (int k = 0; k < kPgCopyVecs; ++k)
      if (i0 + k * kPgCopyThreads < page_vecs) v[k] = src[i0 + k * kPgCopyThreads];
#pragma unroll
    for (int k = 0; k < kPgCopyVecs; ++k)
      if (i0 + k * kPgCopyThreads < page_vecs) dst[i0 + k * kPgCopyThreads] = v[k];
  }
}

int check_common(const int32_t* table_in, const int32_t* table_out, const int32_t* ref_in, const int32_t* ref_out,
                 int32_t rows_in, int32_t rows_out, int32_t max_pages, int32_t num_pages, const int32_t* moves,
                 const int32_t* n_moves, const uint32_t* status) {
  if (!table_in || !table_out || !ref_in || !ref_out || !moves || !n_moves || !status)
    return fail(HPC_ERR_ARG, "null pointer argument");
  if (rows_in < 1 || rows_out < 1 || max_pages < 1 || num_pages < 1) return fail(HPC_ERR_ARG, "sizes must be >= 1");
  if (reinterpret_cast<uintptr_t>(moves) & 7u) return fail(HPC_ERR_ALIGN, "moves must be 8-byte aligned");
  return HPC_OK;
}

int check_rows(int32_t rows, int32_t max_pages, int32_t page_size) {
  // the pages that all rows need together are counted in 32 bits
  if (static_cast<int64_t>(rows) * max_pages > INT32_MAX) return fail(HPC_ERR_SHAPE, "rows x max_pages_per_req exceeds INT32_MAX");
  if (rows > kPgMaxRows) return fail(HPC_ERR_SHAPE, "more than %d rows", kPgMaxRows);
  if (page_size < 1) return fail(HPC_ERR_ARG, "page_size must be >= 1");
  if (static_cast<int64_t>(max_pages) * page_size > INT32_MAX)
    return fail(HPC_ERR_SHAPE, "max_pages_per_req x page_size exceeds INT32_MAX");
  return HPC_OK;
}

int launch_planner(void (*kernel)(PgArgs), const char* name, const PgArgs& args, size_t smem, void* stream) {
  // Without the attribute a block has 48 KB, the kernel's own variables (below 1 KB) among them.
  if (smem + 1024 > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return launched(e, name);
  }
  const cudaError_t e = launch_pdl(kernel, dim3(kPgCtas), dim3(kPgThreads), smem, static_cast<cudaStream_t>(stream), args);
  return launched(e, name);
}

}  // namespace
}  // namespace hpc

using namespace hpc;

extern "C" int hpc_pages_resize(const int32_t* table_in, int32_t* table_out, int32_t batch, int32_t max_pages_per_req,
                                int32_t page_size, const int32_t* old_lens, const int32_t* new_lens,
                                const int32_t* ref_in, int32_t* ref_out, int32_t num_pages, int32_t* moves,
                                int32_t move_capacity, int32_t* n_moves, uint32_t* status, void* stream) {
  int rc = check_common(table_in, table_out, ref_in, ref_out, batch, batch, max_pages_per_req, num_pages, moves,
                        n_moves, status);
  if (rc != HPC_OK) return rc;
  if (!old_lens || !new_lens) return fail(HPC_ERR_ARG, "null pointer argument");
  if ((rc = check_rows(batch, max_pages_per_req, page_size)) != HPC_OK) return rc;
  if (move_capacity < batch) return fail(HPC_ERR_CAPACITY, "moves must hold batch (%d) pairs", batch);
  PgArgs a = {};
  a.table_in = table_in;
  a.table_out = table_out;
  a.lens = old_lens;
  a.want = new_lens;
  a.ref_in = ref_in;
  a.ref_out = ref_out;
  a.moves = reinterpret_cast<int2*>(moves);
  a.n_moves = n_moves;
  a.status = status;
  a.rows_in = a.rows_out = batch;
  a.max_pages = max_pages_per_req;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.max_len = max_pages_per_req * page_size;
  return launch_planner(pages_resize_kernel, "pages_resize_kernel", a, static_cast<size_t>(batch) * 8, stream);
}

extern "C" int hpc_pages_fork(const int32_t* table_in, const int32_t* lens_in, int32_t rows_in, const int32_t* parents,
                              int32_t* table_out, int32_t* lens_out, int32_t rows_out, int32_t max_pages_per_req,
                              int32_t page_size, const int32_t* ref_in, int32_t* ref_out, int32_t num_pages,
                              int32_t* moves, int32_t move_capacity, int32_t* n_moves, uint32_t* status, void* stream) {
  int rc = check_common(table_in, table_out, ref_in, ref_out, rows_in, rows_out, max_pages_per_req, num_pages, moves,
                        n_moves, status);
  if (rc != HPC_OK) return rc;
  if (!lens_in || !lens_out || !parents) return fail(HPC_ERR_ARG, "null pointer argument");
  if ((rc = check_rows(rows_in > rows_out ? rows_in : rows_out, max_pages_per_req, page_size)) != HPC_OK) return rc;
  if (table_in == table_out || lens_in == lens_out)
    return fail(HPC_ERR_ARG, "the forked table and lengths need buffers of their own");
  if (move_capacity < rows_out) return fail(HPC_ERR_CAPACITY, "moves must hold rows_out (%d) pairs", rows_out);
  PgArgs a = {};
  a.table_in = table_in;
  a.table_out = table_out;
  a.lens = lens_in;
  a.want = parents;
  a.lens_out = lens_out;
  a.ref_in = ref_in;
  a.ref_out = ref_out;
  a.moves = reinterpret_cast<int2*>(moves);
  a.n_moves = n_moves;
  a.status = status;
  a.rows_in = rows_in;
  a.rows_out = rows_out;
  a.max_pages = max_pages_per_req;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.max_len = max_pages_per_req * page_size;
  return launch_planner(pages_fork_kernel, "pages_fork_kernel", a,
                        (static_cast<size_t>(rows_out) + 2 * static_cast<size_t>(rows_in)) * 4, stream);
}

extern "C" int hpc_pages_compact(const int32_t* table_in, int32_t* table_out, int32_t batch, int32_t max_pages_per_req,
                                 const int32_t* ref_in, int32_t* ref_out, int32_t num_pages, int32_t* page_map,
                                 int32_t* moves, int32_t move_capacity, int32_t* n_moves, uint32_t* status,
                                 void* stream) {
  const int rc = check_common(table_in, table_out, ref_in, ref_out, batch, batch, max_pages_per_req, num_pages, moves,
                              n_moves, status);
  if (rc != HPC_OK) return rc;
  if (!page_map) return fail(HPC_ERR_ARG, "null pointer argument");
  if (move_capacity < num_pages / 2)
    return fail(HPC_ERR_CAPACITY, "moves must hold num_pages / 2 (%d) pairs", num_pages / 2);
  PgArgs a = {};
  a.table_in = table_in;
  a.table_out = table_out;
  a.ref_in = ref_in;
  a.ref_out = ref_out;
  a.page_map = page_map;
  a.moves = reinterpret_cast<int2*>(moves);
  a.n_moves = n_moves;
  a.status = status;
  a.rows_in = a.rows_out = batch;
  a.max_pages = max_pages_per_req;
  a.num_pages = num_pages;
  return launch_planner(pages_compact_kernel, "pages_compact_kernel", a, 0, stream);
}

extern "C" int hpc_pages_copy(void* const* caches, int32_t n_caches, int64_t page_bytes, int32_t num_pages,
                              const int32_t* moves, int32_t move_capacity, const int32_t* n_moves, uint32_t* status,
                              void* stream) {
  if (!caches || !moves || !n_moves || !status) return fail(HPC_ERR_ARG, "null pointer argument");
  if (n_caches < 0 || page_bytes < 1 || num_pages < 1 || move_capacity < 0)
    return fail(HPC_ERR_ARG, "sizes out of range");
  if (page_bytes % 16) return fail(HPC_ERR_SHAPE, "page_bytes must be a multiple of 16");
  if (reinterpret_cast<uintptr_t>(moves) & 7u) return fail(HPC_ERR_ALIGN, "moves must be 8-byte aligned");
  for (int32_t i = 0; i < n_caches; ++i) {
    if (!caches[i]) return fail(HPC_ERR_ARG, "null pointer argument");
    if (!aligned16(caches[i])) return fail(HPC_ERR_ALIGN, "caches must be 16-byte aligned");
  }
  if (n_caches == 0 || move_capacity == 0) return HPC_OK;
  const int64_t page_vecs = page_bytes / 16;
  const int64_t chunks = (page_vecs + kPgCopyChunk - 1) / kPgCopyChunk;
  const int sms = device_sm_count();
  const int64_t cap = static_cast<int64_t>(sms > 0 ? sms : 148) * kPgCopyCtas;
  for (int32_t c0 = 0; c0 < n_caches; c0 += kPgMaxCaches) {
    PgCaches list = {};
    const int32_t nc = n_caches - c0 < kPgMaxCaches ? n_caches - c0 : kPgMaxCaches;
    for (int32_t i = 0; i < nc; ++i) list.base[i] = static_cast<uint4*>(caches[c0 + i]);
    const int64_t most = chunks * nc * move_capacity;  // the count itself is on the device
    const cudaError_t e = launch_pdl(pages_copy_kernel, dim3(static_cast<unsigned>(most < cap ? most : cap)),
                                     dim3(kPgCopyThreads), 0, static_cast<cudaStream_t>(stream), list, nc, page_vecs,
                                     num_pages, reinterpret_cast<const int2*>(moves), n_moves, move_capacity, status);
    const int rc = launched(e, "pages_copy_kernel");
    if (rc != HPC_OK) return rc;
  }
  return HPC_OK;
}
