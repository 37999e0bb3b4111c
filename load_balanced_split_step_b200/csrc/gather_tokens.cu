// The cached tokens of a batch as packed bf16 rows: request r's K and V, in order, at rows cu[r] .. cu[r + 1] - 1 of two
// [tokens][kv_heads][head_dim] arrays, with cu the prefix sums of the lengths. What reads packed rows only (prompt attention
// over E4M3 caches, whose scales are applied here, or over pages of any size) reads them behind it.
//
// Bound by memory: every value is read once and written once. Every CTA takes an equal run of output rows, whatever
// the lengths are, and sums the lengths up for itself, a few hundred ns for a batch, instead of a launch. Writes are
// contiguous, reads are rows of head_dim. 58992 tokens of 8 heads of 128 in pages of 64: bf16 90 us, 5.4 TB/s of reads and
// writes; E4M3 70 us, 5.2 TB/s. Two or four pieces per thread in flight with fewer CTAs are no faster (89, 90 and 71, 70 us);
// whole 16-byte loads of E4M3, which leave gaps between a warp's stores, take 79 us.
#include <type_traits>

#include "hpc_common.cuh"

namespace hpc {
namespace {

constexpr int kGtThreads = 256;
constexpr int kGtWarps = kGtThreads / 32;

constexpr int kGtCtas = 8;         // per SM: all that fit; latency is hidden by threads
constexpr int kGtMaxBatch = 8192;  // prefix sums in shared memory

struct GtArgs {
  const void *k_pages, *v_pages;
  const float *k_scale, *v_scale;
  const int32_t *table, *seq_lens;
  const int32_t* cu_q;  // or null: no queries to count
  __nv_bfloat16 *k, *v;
  int32_t* cu;
  uint32_t* status;
  int64_t max_pages;
  int32_t batch, H, num_pages, P, nhd, capacity;
};

// Sums stop at INT32_MAX instead of wrapping.
__device__ __forceinline__ int32_t gt_add(int32_t a, int32_t b) {
  const uint32_t s = static_cast<uint32_t>(a) + static_cast<uint32_t>(b);
  return static_cast<int32_t>(s < 0x7fffffffu ? s : 0x7fffffffu);
}

// 8 cached values -> 16 bytes of bf16. E4M3 codes times the scale are rounded to bf16, as a bf16 cache's values were.
__device__ __forceinline__ uint4 gt_row(const uint4& x, float) { return x; }
__device__ __forceinline__ uint4 gt_row(const uint2& x, float scale) {
  float f[4], g[4];
  e4m3x4_to_f32x4(x.x, f);
  e4m3x4_to_f32x4(x.y, g);
  return make_uint4(pack_bf16x2(f[0] * scale, f[1] * scale), pack_bf16x2(f[2] * scale, f[3] * scale),
                    pack_bf16x2(g[0] * scale, g[1] * scale), pack_bf16x2(g[2] * scale, g[3] * scale));
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kGtThreads, kGtCtas) gather_tokens_kernel(const GtArgs a) {
  using Piece = std::conditional_t<kFp8, uint2, uint4>;  // 8 values
  constexpr int kPieces = D / 8;
  extern __shared__ int32_t s_cu[];               // [batch + 1]
  __shared__ int32_t s_sum[kGtWarps], s_total, s_bad;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) s_total = s_bad = 0;

  // ---- prefix sums; requests from the first that does not fit on are left out
  int32_t base = 0;
  for (int32_t r0 = 0; r0 < a.batch; r0 += kGtThreads) {
    const int32_t r = r0 + static_cast<int32_t>(threadIdx.x);
    int32_t n = r < a.batch ? a.seq_lens[r] : 0;
    bool bad = n < 0 || static_cast<int64_t>(n) > a.max_pages * a.P;
    if (a.cu_q && r < a.batch) bad |= static_cast<int64_t>(a.cu_q[r + 1]) - a.cu_q[r] > n;
    if (bad) n = 0;
    int32_t x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = gt_add(x, y);
    }
    __syncthreads();  // the sums before are read; s_bad is set
    if (lane == 31) s_sum[warp] = x;
    if (bad) s_bad = 1;
    __syncthreads();
    int32_t before = base;
    for (int w = 0; w < kGtWarps; ++w) {
      if (w < warp) before = gt_add(before, s_sum[w]);
      base = gt_add(base, s_sum[w]);
    }
    x = gt_add(before, x);
    if (r < a.batch) {
      s_cu[r + 1] = x;
      if (x <= a.capacity) atomicMax(&s_total, x);
    }
  }
  if (threadIdx.x == 0) s_cu[0] = 0;
  __syncthreads();
  const int32_t total = s_total;
  for (int32_t r = threadIdx.x; r <= a.batch; r += kGtThreads) {
    const int32_t x = s_cu[r] <= total ? s_cu[r] : total;
    s_cu[r] = x;
    if (blockIdx.x == 0) a.cu[r] = x;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && (s_bad || base > total))
    atomicOr(a.status, (s_bad ? HPC_DEV_BAD_SEQLEN : 0u) | (base > total ? HPC_DEV_CAPACITY : 0u));
  __syncthreads();

  // ---- the rows: an equal run of tokens for every CTA
  const uint32_t H = a.H, P = a.P;
  const int32_t i0 = static_cast<int32_t>(static_cast<int64_t>(total) * blockIdx.x / gridDim.x);
  const int32_t i1 = static_cast<int32_t>(static_cast<int64_t>(total) * (blockIdx.x + 1) / gridDim.x);
  int32_t r = 0, hi = a.batch;  // the last r with cu[r] <= i0; it only grows
  while (hi - r > 1) {
    const int32_t mid = (r + hi) >> 1;
    if (s_cu[mid] <= i0) r = mid;
    else hi = mid;
  }
  const uint32_t pieces = static_cast<uint32_t>(i1 - i0) * H * kPieces;  // of arrays that fit into memory
  for (uint32_t e = threadIdx.x; e < pieces; e += kGtThreads) {
    const uint32_t row = e / kPieces, piece = e % kPieces, tok = row / H, h = row - tok * H;
    const int32_t i = i0 + static_cast<int32_t>(tok);
    while (i >= s_cu[r + 1]) ++r;
    const uint32_t pos = i - s_cu[r], col = pos / P, slot = pos - col * P;
    const int32_t page = a.table[r * a.max_pages + col];
    const bool ok = page >= 0 && page < a.num_pages;
    if (!ok && piece == 0 && h == 0) atomicOr(a.status, HPC_DEV_BAD_PAGE);
    const int64_t at = (a.nhd ? (static_cast<int64_t>(page) * P + slot) * H + h
                              : (static_cast<int64_t>(page) * H + h) * P + slot) * kPieces + piece;
    Piece k = {}, v = {};
    if (ok) {
      k = static_cast<const Piece*>(a.k_pages)[at];
      v = static_cast<const Piece*>(a.v_pages)[at];
    }
    const int64_t to = (static_cast<int64_t>(i) * H + h) * kPieces + piece;
    reinterpret_cast<uint4*>(a.k)[to] = gt_row(k, kFp8 ? a.k_scale[h] : 1.f);
    reinterpret_cast<uint4*>(a.v)[to] = gt_row(v, kFp8 ? a.v_scale[h] : 1.f);
  }
}

int gather(const void* k_pages, const void* v_pages, hpc_dtype kv_dtype, hpc_kv_layout kv_layout, const float* k_scale,
           const float* v_scale, int32_t num_pages, int32_t page_size, const int32_t* block_table,
           int32_t max_pages_per_req, const int32_t* seq_lens, const int32_t* cu_queries, int32_t batch, int32_t kv_heads,
           int32_t head_dim, int64_t kv_tokens, void* k_out, void* v_out, int32_t* cu_seqlens, uint32_t* status,
           void* stream) {
  if (kv_tokens < 0 || kv_tokens > INT32_MAX - 1024) return fail(HPC_ERR_ARG, "kv_tokens out of range");
  if (!k_pages || !v_pages || !block_table || !seq_lens || !cu_seqlens || !status || (kv_tokens > 0 && (!k_out || !v_out)))
    return fail(HPC_ERR_ARG, "null pointer argument");
  if (kv_dtype != HPC_BF16 && kv_dtype != HPC_E4M3) return fail(HPC_ERR_DTYPE, "kv_dtype must be BF16 or E4M3");
  if (kv_layout != HPC_HND && kv_layout != HPC_NHD) return fail(HPC_ERR_ARG, "kv_layout must be HND or NHD");
  const bool fp8 = kv_dtype == HPC_E4M3;
  if (fp8 && (!k_scale || !v_scale)) return fail(HPC_ERR_ARG, "E4M3 cache needs k_scale and v_scale");
  if (batch < 1 || kv_heads < 1 || num_pages < 1 || page_size < 1 || max_pages_per_req < 1)
    return fail(HPC_ERR_ARG, "sizes must be >= 1");
  if (head_dim != 64 && head_dim != 128) return fail(HPC_ERR_SHAPE, "head_dim must be 64 or 128");
  if (batch > kGtMaxBatch) return fail(HPC_ERR_SHAPE, "more than %d requests", kGtMaxBatch);
  if (kv_heads > 65536) return fail(HPC_ERR_SHAPE, "more than 65536 kv heads");
  if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_out) || !aligned16(v_out))
    return fail(HPC_ERR_ALIGN, "the caches, k_out and v_out must be 16-byte aligned");
  GtArgs a = {};
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.table = block_table;
  a.seq_lens = seq_lens;
  a.cu_q = cu_queries;
  a.k = static_cast<__nv_bfloat16*>(k_out);
  a.v = static_cast<__nv_bfloat16*>(v_out);
  a.cu = cu_seqlens;
  a.status = status;
  a.max_pages = max_pages_per_req;
  a.batch = batch;
  a.H = kv_heads;
  a.num_pages = num_pages;
  a.P = page_size;
  a.nhd = kv_layout == HPC_NHD;
  a.capacity = static_cast<int32_t>(kv_tokens);
  // as many CTAs as stay, with a few pieces for every thread
  const int64_t pieces = kv_tokens * kv_heads * (head_dim / 8), each = 2 * kGtThreads;
  const int64_t most = static_cast<int64_t>(kGtCtas) * (device_sm_count() > 0 ? device_sm_count() : 148);
  const int64_t want = (pieces + each - 1) / each, blocks = want < 1 ? 1 : (want < most ? want : most);
  auto kern = head_dim == 128 ? (fp8 ? gather_tokens_kernel<128, true> : gather_tokens_kernel<128, false>)
                              : (fp8 ? gather_tokens_kernel<64, true> : gather_tokens_kernel<64, false>);
  const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kGtThreads),
                                   (static_cast<size_t>(batch) + 1) * 4, static_cast<cudaStream_t>(stream), a);
  return launched(e, "gather_tokens_kernel");
}

}  // namespace
}  // namespace hpc

using namespace hpc;

extern "C" int hpc_gather_tokens(const void* k_pages, const void* v_pages, hpc_dtype kv_dtype, hpc_kv_layout kv_layout,
                                 const float* k_scale, const float* v_scale, int32_t num_pages, int32_t page_size,
                                 const int32_t* block_table, int32_t max_pages_per_req, const int32_t* seq_lens,
                                 int32_t batch, int32_t kv_heads, int32_t head_dim, int64_t kv_tokens, void* k_out,
                                 void* v_out, int32_t* cu_seqlens, uint32_t* status, void* stream) {
  return gather(k_pages, v_pages, kv_dtype, kv_layout, k_scale, v_scale, num_pages, page_size, block_table,
                max_pages_per_req, seq_lens, nullptr, batch, kv_heads, head_dim, kv_tokens, k_out, v_out, cu_seqlens,
                status, stream);
}

extern "C" int hpc_gather_prompt_tokens(const void* k_pages, const void* v_pages, hpc_dtype kv_dtype,
                                        hpc_kv_layout kv_layout, const float* k_scale, const float* v_scale,
                                        int32_t num_pages, int32_t page_size, const int32_t* block_table,
                                        int32_t max_pages_per_req, const int32_t* seq_lens, const int32_t* cu_queries,
                                        int32_t batch, int32_t kv_heads, int32_t head_dim, int64_t kv_tokens, void* k_out,
                                        void* v_out, int32_t* cu_seqlens, uint32_t* status, void* stream) {
  if (!cu_queries) return fail(HPC_ERR_ARG, "null pointer argument");
  return gather(k_pages, v_pages, kv_dtype, kv_layout, k_scale, v_scale, num_pages, page_size, block_table,
                max_pages_per_req, seq_lens, cu_queries, batch, kv_heads, head_dim, kv_tokens, k_out, v_out, cu_seqlens,
                status, stream);
}
