// Verification of drafted tokens against the target's probabilities (speculative decoding), from
// given random numbers.
//
// With p_t the target's and q_t the draft's distribution at step t, drafted token x_t is kept when
// u_t q_t(x_t) < p_t(x_t). At the first token that is not, one is drawn from the rest
// max(p_t - q_t, 0) instead; when all are kept, one is drawn from p_T. The draw inverts the cumulative
// sum: the lowest i with sum_{j <= i} w_j > u sum_j w_j. The result is distributed as the target's own
// samples. Everything is compared and summed in fp64 (u q is exact there, and so is p - q for most
// pairs of floats), so that the choice next to a border does not hang on the order of a sum.
//
// One cluster of up to 8 CTAs per request. Each CTA decides the kept tokens on its own (a few words), so
// that only the one row that is drawn from is read: 2 V values at a rejection, V otherwise, each once
// from HBM. A warp owns a contiguous run of the vocabulary and sums it; the sums meet in distributed
// shared memory; the CTA whose run holds the crossing reads it again (from L2) to find it.
//
// A call is about 5 us of latencies (launch, the drafts' words, two passes; one request of 32000 takes no more) and the row
// streams. 64 requests, vocabulary 131071, fp32: 11.9 us where every draft is kept and one row read, 18.6 where every one is
// rejected and two are (the second at 4.8 TB/s), 16.4 mixed: the requests with two rows set the time, with as many CTAs
// each as those with one. (25 us with every value tested in fp64, 39 us with one warp searching the run; the
// conversions to fp64 are under 4 us of it.) bf16 takes 14.5: half of the bytes in as many loads. A one-hot draft that is
// rejected has every value tested, for the one that is left out: 23.6.
#include <type_traits>

#include "hpc_common.cuh"

namespace hpc {
namespace {

constexpr int kVfThreads = 512;
constexpr int kVfWarps = kVfThreads / 32;
constexpr int kVfMaxCtas = 8;  // portable cluster
constexpr int kVfMaxDrafts = 256;
constexpr int kVfBatch = 8;   // entries per lane loaded together
constexpr int kVfRows = 4;    // rows of 32 entries looked at together in the end

// Plain loads: an __ldg of a bf16 is an asm statement that the compiler may move ahead of the test
// that guards it.
__device__ __forceinline__ float vf_load(const float* p) { return *p; }
__device__ __forceinline__ float vf_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// A probability: what is not a positive finite number counts as zero.
__device__ __forceinline__ double vf_prob(float x) { return x > 0.f && x <= 3.402823466e38f ? static_cast<double>(x) : 0.0; }

__device__ __forceinline__ double vf_warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Inclusive prefix over the lanes.
__device__ __forceinline__ double vf_scan(double v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// The part (of n <= 32, in order) in which the running sum passes the target, or the last with any mass;
// `from` is the sum before the parts and becomes the sum before the chosen one. Whole warp, mass somewhere.
// Sums of parts can round differently from the part's own sums, so that "passes" may find no entry inside; the
// last with mass is then the entry up to that rounding. A target that nothing passes (u >= 1, NaN) ends
// there too.
__device__ __forceinline__ int vf_choose(const double* sums, int n, double target, double& from) {
  const int lane = threadIdx.x & 31;
  const double s = lane < n ? sums[lane] : 0.0, inc = vf_scan(s);
  const uint32_t over = __ballot_sync(0xffffffffu, s > 0.0 && from + inc > target);
  const uint32_t mass = __ballot_sync(0xffffffffu, s > 0.0);
  const int sel = over ? __ffs(over) - 1 : 31 - __clz(mass);
  const double before = __shfl_sync(0xffffffffu, inc, sel > 0 ? sel - 1 : 0);
  from += sel > 0 ? before : 0.0;
  return sel;
}

struct VfArgs {
  const int32_t* drafts;
  const void* p;
  const void* q;
  int64_t p_stride, q_stride;  // elements between rows (r, t)
  const float* u;
  const int32_t* draft_lens;
  const int32_t* seq_lens;
  int32_t* tokens;
  int32_t* accepted;
  int32_t* new_lens;
  uint32_t* status;
  int32_t T, V;
};

template <typename S>
__global__ void __launch_bounds__(kVfThreads, 2) verify_kernel(const VfArgs a, int32_t ctas) {
  __shared__ int32_t s_lost[kVfMaxDrafts / 32];
  __shared__ double s_sub[kVfWarps];
  __shared__ double s_warp[kVfWarps];
  __shared__ double s_cta[3][kVfMaxCtas];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t r = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  const int32_t T = a.T, V = a.V;
  // Shared memory of another CTA may be written only once that CTA runs: it says so here, and is
  // waited for before the first such store.
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  pdl_wait();
  pdl_launch_dependents();

  // The kept tokens, a thread per draft; its words are loaded side by side with the count.
  const S* p_rows = static_cast<const S*>(a.p) + static_cast<int64_t>(r) * (T + 1) * a.p_stride;
  const S* q_rows = a.q ? static_cast<const S*>(a.q) + static_cast<int64_t>(r) * T * a.q_stride : nullptr;
  const float* u_row = a.u + static_cast<int64_t>(r) * (T + 1);
  const double u = static_cast<double>(u_row[T]);
  int32_t n = a.draft_lens ? a.draft_lens[r] : T;
  if (warp < kVfMaxDrafts / 32) {
    const int32_t t = threadIdx.x;
    bool keep = true;
    if (t < T) {
      const int32_t x = a.drafts[static_cast<int64_t>(r) * T + t];
      const float ut = u_row[t];
      if (x < 0 || x >= V) {
        if (rank == 0 && t < n) atomicOr(a.status, HPC_DEV_BAD_INDEX);
        keep = false;
      } else {
        const double px = vf_prob(vf_load(p_rows + t * a.p_stride + x));
        const double qx = q_rows ? vf_prob(vf_load(q_rows + t * a.q_stride + x)) : 1.0;
        keep = static_cast<double>(ut) * qx < px;
      }
    }
    const uint32_t lost = __ballot_sync(0xffffffffu, !keep);
    if (lane == 0) s_lost[warp] = lost ? 32 * warp + __ffs(lost) - 1 : T;
  }
  if (n < 0 || n > T) {
    if (rank == 0 && threadIdx.x == 0) atomicOr(a.status, HPC_DEV_BAD_SEQLEN);
    n = n < 0 ? 0 : T;
  }
  __syncthreads();
  int32_t at = n;  // tokens kept; the step that is drawn
#pragma unroll
  for (int w = 0; w < kVfMaxDrafts / 32; ++w) at = min(at, s_lost[w]);
  const bool cut = at < n;
  const S* p = p_rows + at * a.p_stride;
  bool rest = cut && q_rows;
  const S* q = rest ? q_rows + at * a.q_stride : p;  // a valid row either way
  int32_t gone = cut && !q_rows ? a.drafts[static_cast<int64_t>(r) * T + at] : -1;  // one-hot draft

  // this warp's run of the vocabulary
  const int64_t per = (((static_cast<int64_t>(V) + ctas * kVfWarps - 1) / (ctas * kVfWarps)) + 31) & ~int64_t(31);
  const int64_t b64 = per * (rank * kVfWarps + warp);
  const int32_t begin = static_cast<int32_t>(b64 < V ? b64 : V);
  const int32_t end = static_cast<int32_t>(b64 + per < V ? b64 + per : V);

  // The weights of entries i0 + 32 k + lane, k < kN, zero past `stop`; all loads before the first use.
  auto load = [&](auto count, int32_t i0, int32_t stop, double* w) {
    constexpr int kN = decltype(count)::value;
    float x[kN], y[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int32_t i = i0 + 32 * k + lane;
      x[k] = i < stop ? vf_load(p + i) : 0.f;
      y[k] = rest && i < stop ? vf_load(q + i) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const double d = vf_prob(x[k]) - vf_prob(y[k]);
      w[k] = d > 0.0 && i0 + 32 * k + lane != gone ? d : 0.0;
    }
  };
  // Sum of the weights of [from, stop) (whole warp). Conversions to fp64 and the instructions around them bound
  // this as much as memory does, so whole batches go without tests: fmaxf makes NaN and negative values 0, and
  // an infinity shows in the sum (of q: in the maximum). Then (`careful`) every value is tested.
  bool careful = false;
  auto sum_run = [&](int32_t from, int32_t stop) {
    double sum = 0.0;
    int32_t i = from;
    if (!careful && gone < 0) {
      if (rest) {
        float top = 0.f;
        for (; i + 32 * kVfBatch <= stop; i += 32 * kVfBatch) {
          float x[kVfBatch], y[kVfBatch];
#pragma unroll
          for (int k = 0; k < kVfBatch; ++k) {
            x[k] = vf_load(p + i + lane + 32 * k);
            y[k] = vf_load(q + i + lane + 32 * k);
          }
#pragma unroll
          for (int k = 0; k < kVfBatch; ++k) {
            const float a = fmaxf(x[k], 0.f), b = fmaxf(y[k], 0.f);
            const double d = static_cast<double>(a) - static_cast<double>(b);
            if (a > b) sum += d;
            top = fmaxf(top, b);
          }
        }
        if (top > 3.402823466e38f) sum = top;
      } else {
        for (; i + 32 * kVfBatch <= stop; i += 32 * kVfBatch) {
          float x[kVfBatch];
#pragma unroll
          for (int k = 0; k < kVfBatch; ++k) x[k] = vf_load(p + i + lane + 32 * k);
#pragma unroll
          for (int k = 0; k < kVfBatch; ++k) sum += static_cast<double>(fmaxf(x[k], 0.f));
        }
      }
    }
    for (; i < stop; i += 32 * kVfRows) {
      double w[kVfRows];
      load(std::integral_constant<int, kVfRows>{}, i, stop, w);
#pragma unroll
      for (int k = 0; k < kVfRows; ++k) sum += w[k];
    }
    return vf_warp_sum(sum);
  };
  double total = 0.0;
  int used = 0;  // the round whose sums hold
  for (int round = 0; round < 3; ++round) {
    const double sum = sum_run(begin, end);
    if (lane == 0) s_warp[warp] = sum;
    __syncthreads();
    if (round == 0) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (static_cast<int32_t>(threadIdx.x) < ctas) {
      double mine = 0.0;
      for (int w = 0; w < kVfWarps; ++w) mine += s_warp[w];
      uint32_t dst;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(smem_u32(&s_cta[round][rank])), "r"(threadIdx.x));
      asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(dst), "d"(mine) : "memory");
    }
    // not the .aligned forms: nothing holds a warp together after the branch above
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    used = round;
    total = __shfl_sync(0xffffffffu, vf_scan(lane < ctas ? s_cta[round][lane] : 0.0), ctas - 1);
    const bool finite = total <= 1.7976931348623157e308;  // the same in every CTA, as all that follows
    if (finite && (total > 0.0 || (!rest && gone < 0))) break;
    __syncthreads();
    if (!finite) {
      careful = true;
    } else {
      // The rest has no mass (the target gives nothing outside the draft's share): the target's own row.
      rest = false;
      gone = -1;
    }
  }

  int32_t* tokens = a.tokens + static_cast<int64_t>(r) * (T + 1);
  if (rank == 0) {
    for (int32_t t = threadIdx.x; t <= T; t += kVfThreads)
      if (t < at) tokens[t] = a.drafts[static_cast<int64_t>(r) * T + t];
      else if (t > at || !(total > 0.0)) tokens[t] = -1;
    if (threadIdx.x == 0) {
      a.accepted[r] = at;
      if (a.new_lens) a.new_lens[r] = a.seq_lens[r] - n + at;
      if (!(total > 0.0)) atomicOr(a.status, HPC_DEV_BAD_PROBS);
    }
  }
  if (!(total > 0.0)) return;

  // The CTA, then the warp's run, then the part of the run, then the entry at which the running sum passes
  const double target = u * total;
  double base = 0.0;
  if (vf_choose(s_cta[used], ctas, target, base) != rank) return;
  // All warps take a part of the chosen run, and the one whose part holds the crossing looks at it 32
  // entries at a time. (One warp alone spent 4 to 10 us here.)
  const int64_t run0 = per * (rank * kVfWarps + vf_choose(s_warp, kVfWarps, target, base));
  const int64_t run1 = run0 + per < V ? run0 + per : V, part = ((per + kVfWarps - 1) / kVfWarps + 31) & ~int64_t(31);
  auto edge = [&](int w) { return static_cast<int32_t>(run0 + part * w < run1 ? run0 + part * w : run1); };
  {
    const double sum = sum_run(edge(warp), edge(warp + 1));
    if (lane == 0) s_sub[warp] = sum;
  }
  __syncthreads();
  const int sel = vf_choose(s_sub, kVfWarps, target, base);
  if (warp != sel) return;
  int32_t found = -1, final_mass = -1;
  for (int32_t i0 = edge(sel); i0 < edge(sel + 1) && found < 0; i0 += 32 * kVfRows) {
    double rows[kVfRows];
    load(std::integral_constant<int, kVfRows>{}, i0, edge(sel + 1), rows);
#pragma unroll
    for (int k = 0; k < kVfRows; ++k) {
      const double w = rows[k];
      const double c = vf_scan(w);
      const uint32_t mass = __ballot_sync(0xffffffffu, w > 0.0);
      const uint32_t over = __ballot_sync(0xffffffffu, w > 0.0 && base + c > target);
      if (over && found < 0) found = i0 + 32 * k + __ffs(over) - 1;
      if (mass) final_mass = i0 + 32 * k + 31 - __clz(mass);
      base += __shfl_sync(0xffffffffu, c, 31);
    }
  }
  if (lane == 0) tokens[at] = found >= 0 ? found : final_mass;
}

template <typename S>
cudaError_t launch_verify(const VfArgs& a, int32_t batch, int32_t ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(batch) * ctas);
  cfg.blockDim = dim3(kVfThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<S>, a, ctas);
}

}  // namespace
}  // namespace hpc

using namespace hpc;

extern "C" int hpc_verify_drafts(const int32_t* draft_tokens, const void* target_probs, int64_t target_stride,
                                 const void* draft_probs, int64_t draft_stride, hpc_dtype prob_dtype,
                                 const float* uniforms, const int32_t* draft_lens, const int32_t* seq_lens,
                                 int32_t batch, int32_t max_drafts, int32_t vocab, int32_t* out_tokens,
                                 int32_t* accepted, int32_t* new_lens, uint32_t* status, void* stream) {
  if (!target_probs || !uniforms || !out_tokens || !accepted || !status || (max_drafts > 0 && !draft_tokens))
    return fail(HPC_ERR_ARG, "null pointer argument");
  if (new_lens && !seq_lens) return fail(HPC_ERR_ARG, "new_lens needs seq_lens");
  if (prob_dtype != HPC_FP32 && prob_dtype != HPC_BF16) return fail(HPC_ERR_DTYPE, "probabilities must be FP32 or BF16");
  if (batch < 1 || max_drafts < 0 || vocab < 1) return fail(HPC_ERR_ARG, "sizes out of range");
  if (vocab > INT32_MAX - 4096) return fail(HPC_ERR_SHAPE, "vocab too large");
  if (max_drafts > kVfMaxDrafts) return fail(HPC_ERR_SHAPE, "max_drafts above %d", kVfMaxDrafts);
  if (batch > INT32_MAX / kVfMaxCtas) return fail(HPC_ERR_SHAPE, "batch too large");
  if (target_stride < vocab || (draft_probs && draft_stride < vocab))
    return fail(HPC_ERR_ARG, "a row stride is smaller than the vocabulary");
  VfArgs a = {};
  a.drafts = draft_tokens;
  a.p = target_probs;
  a.q = max_drafts > 0 ? draft_probs : nullptr;
  a.p_stride = target_stride;
  a.q_stride = draft_stride;
  a.u = uniforms;
  a.draft_lens = draft_lens;
  a.seq_lens = seq_lens;
  a.tokens = out_tokens;
  a.accepted = accepted;
  a.new_lens = new_lens;
  a.status = status;
  a.T = max_drafts;
  a.V = vocab;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // As many CTAs per request (a power of two, at most 8) as are on the GPU at once, two per SM: those of a
  // second wave would start only when the first has streamed its rows.
  const int64_t room = 2 * static_cast<int64_t>(device_sm_count() > 0 ? device_sm_count() : 148);
  int32_t ctas = kVfMaxCtas;
  while (ctas > 1 && static_cast<int64_t>(batch) * ctas > room) ctas /= 2;
  const cudaError_t e = prob_dtype == HPC_FP32 ? launch_verify<float>(a, batch, ctas, st)
                                               : launch_verify<__nv_bfloat16>(a, batch, ctas, st);
  return launched(e, "verify_kernel");
}
