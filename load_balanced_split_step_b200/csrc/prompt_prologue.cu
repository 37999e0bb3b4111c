// Prompt prologue: QK-RMSNorm + RoPE on every token of a packed batch of prompts, and the write of
// their K and V into the cache pages. The decode prologue (prologue.cu) for many tokens per request.
//
// y = x w / sqrt(mean x^2 + eps), then the NeoX rotation of the pairs (i, i + D/2) by pos theta^(-2i/D);
// angles in fp64, because pos reaches 1e5. Token i of request r sits at position
// seq_lens[r] - (cu[r+1] - cu[r]) + (i - cu[r]): the new tokens are the last of the request.
//
// Bound by memory: every head of a token is read once and written once or twice. A head is spread over
// D/16 lanes: a lane holds 8 consecutive elements of each half, so that loads and stores are 16 bytes
// wide, the rotation needs no exchange, and the mean square is reduced over D/16 lanes. A warp
// therefore takes 512/D heads of one token at a time, two such groups in work and the next two on their way. It
// computes its token's D/2 angles itself (one or two per lane) and never meets another warp; norm weights and
// rotation are folded into four factors per pair, once per token, and applied two floats at a time. Warps take equal
// runs of groups, parts of tokens too (whole tokens left a seventh of the warps idle at 8192 tokens).
//
// 8192 tokens of 64/8 heads of 128 into an E4M3 cache: 61 us, 5.5 TB/s of reads and writes (76 us with whole tokens, single
// floats and a division per element); 5 or 6 CTAs per SM spill and take 73 and 81. 100 tokens of 8/2 heads of 64: 3.0 us.
#include <cmath>
#include <type_traits>

#include "f32x2.cuh"
#include "hpc_common.cuh"

namespace hpc {
namespace {

constexpr int kPpThreads = 128;
constexpr int kPpWarps = kPpThreads / 32;
constexpr int kPpCtas = 4;  // per SM: 128 registers a thread, two groups of heads in work and two on their way

struct PpArgs {
  const __nv_bfloat16* qkv;
  const int32_t* cu;
  const int32_t* seq_lens;
  const float* q_w;
  const float* k_w;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;
  void* k_pages;
  void* v_pages;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  uint32_t* status;
  int64_t tokens, max_pages;
  double log2_theta;
  float eps;
  int32_t batch, Hq, Hkv, num_pages, P, nhd, fp8;
};

// The request that token i belongs to: the last r with cu[r] <= i (whole warp, 32 probes a step).
// cu[0] is 0 or less than i for every token it is asked about.
__device__ __forceinline__ int32_t find_request(const int32_t* cu, int32_t batch, int64_t i) {
  const int lane = threadIdx.x & 31;
  int32_t lo = 0, n = batch;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int32_t step = (n + 31) >> 5;
    const int32_t at = lo + lane * step;
    const bool le = lane * step < n && cu[at] <= i;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int32_t k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// 8 elements as 4 pairs.
__device__ __forceinline__ void unpack8(uint4 v, float2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
}

__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                    pack_bf16x2(f[3].x, f[3].y));
}

// x / sc as E4M3, by the reciprocal and one step of the remainder (Markstein's correction: q + r (x - q sc), which
// leaves the rounded quotient but for rare last bits, far below an E4M3 step): a division for every element took 5 of 65
// us. The bound keeps a quotient that overflows from turning into NaN; it saturates.
__device__ __forceinline__ uint2 pack8_e4m3(const float2 (&f)[4], float sc, float r) {
  const float top = 1.2676506e30f;  // 2^100
  const float2 r2 = make_float2(r, r), sc2 = make_float2(-sc, -sc);
  float2 q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float2 p = mul2(f[k], r2);
    p = make_float2(fminf(fmaxf(p.x, -top), top), fminf(fmaxf(p.y, -top), top));
    q[k] = fma2(fma2(p, sc2, f[k]), r2, p);
    q[k] = make_float2(copysignf(q[k].x, p.x), copysignf(q[k].y, p.y));  // -0 stays one
  }
  return make_uint2(f32x4_to_e4m3x4(q[0].x, q[0].y, q[1].x, q[1].y), f32x4_to_e4m3x4(q[2].x, q[2].y, q[3].x, q[3].y));
}

// Between 2^-100 and 2^100 the reciprocal is a normal number, and so is the remainder of every quotient that is not 0 as
// an E4M3 code; under other scales (0, subnormal ones, whose reciprocal overflows, infinities, NaN) the codes are written over
// with those of a division. (Choosing before writing took 1.4 us of 61, this takes 0.3.)
__device__ __forceinline__ bool usual_scale(float sc) { return fabsf(sc) >= 7.888609e-31f && fabsf(sc) <= 1.2676506e30f; }
__device__ __forceinline__ uint2 pack8_quotient(const float2 (&f)[4], float sc) {
  return make_uint2(f32x4_to_e4m3x4(f[0].x / sc, f[0].y / sc, f[1].x / sc, f[1].y / sc),
                    f32x4_to_e4m3x4(f[2].x / sc, f[2].y / sc, f[3].x / sc, f[3].y / sc));
}

__device__ __forceinline__ void load8(const float* p, float2 (&f)[4]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w), f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
}

template <int D>
__global__ void __launch_bounds__(kPpThreads, kPpCtas) prompt_prologue_kernel(const PpArgs a) {
  constexpr int kLanes = D / 16;       // lanes per head
  constexpr int kHeads = 32 / kLanes;  // heads per warp at a time
  constexpr int kAngles = D / 64;      // angles per lane
  __shared__ __align__(16) float s_cos[kPpWarps][D / 2];
  __shared__ __align__(16) float s_sin[kPpWarps][D / 2];
  __shared__ __align__(16) float s_w[2][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % kLanes, in_group = lane / kLanes;
  const int heads = a.Hq + 2 * a.Hkv;
  double freq[kAngles];
#pragma unroll
  for (int k = 0; k < kAngles; ++k) freq[k] = exp2(-2.0 * (lane + 32 * k) / D * a.log2_theta);
  pdl_wait();
  pdl_launch_dependents();
  for (int k = threadIdx.x; k < D; k += kPpThreads) {
    s_w[0][k] = a.q_w[k];
    s_w[1][k] = a.k_w[k];
  }
  __syncthreads();
  const int32_t first = a.cu[0], past = a.cu[a.batch];
  // A unit is a group of heads of a token. Each warp takes as many consecutive ones, whole tokens and parts of them, so that
  // all warps end together and a request is looked up once for a run of its tokens.
  const int groups_q = (a.Hq + kHeads - 1) / kHeads, groups_kv = (a.Hkv + kHeads - 1) / kHeads;
  const int groups = groups_q + 2 * groups_kv;
  const int64_t units = a.tokens * groups, warps = static_cast<int64_t>(gridDim.x) * kPpWarps;
  int64_t per = (units + warps - 1) / warps;
  if (per > 1) per += per & 1;  // two groups are in work at a time
  const int64_t u0 = (static_cast<int64_t>(blockIdx.x) * kPpWarps + warp) * per;
  const int64_t u1 = u0 + per < units ? u0 + per : units;
  int64_t i = u0 / groups;
  int g0 = static_cast<int>(u0 - i * groups);
  int64_t b = 0, e = 0, L = 0;
  int32_t r = 0;
  for (int64_t u = u0; u < u1; ++i, g0 = 0) {
    const int g1 = u1 - u < groups - g0 ? g0 + static_cast<int>(u1 - u) : groups;
    u += g1 - g0;
    if (i < first || i >= past) continue;  // no request's token: left as it is
    if (i < b || i >= e) {
      r = find_request(a.cu, a.batch, i);
      b = a.cu[r];
      e = a.cu[r + 1];
      L = a.seq_lens[r];
    }
    // what the lengths say has to hold together before anything is addressed by them
    const bool ok = b <= i && i < e && L >= e - b && L <= a.max_pages * a.P;
    const int64_t pos = ok ? L - (e - i) : 0;
    const int32_t page = ok ? a.table[r * a.max_pages + pos / a.P] : -1;
    const bool page_ok = ok && page >= 0 && page < a.num_pages;
    if (g0 == 0 && lane == 0 && !page_ok) atomicOr(a.status, ok ? HPC_DEV_BAD_PAGE : HPC_DEV_BAD_SEQLEN);
    const int tok = static_cast<int>(pos % a.P);
    const __nv_bfloat16* src = a.qkv + i * heads * D + 8 * sub;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kAngles; ++k) {
      double sn, cs;
      sincos(static_cast<double>(pos) * freq[k], &sn, &cs);
      s_cos[warp][lane + 32 * k] = static_cast<float>(cs);
      s_sin[warp][lane + 32 * k] = static_cast<float>(sn);
    }
    __syncwarp();
    // the groups [lo, hi) of one kind: q (0), k (1), v (2)
    auto run = [&](auto kind_c, int lo, int hi) {
      constexpr int kind = decltype(kind_c)::value;
      const int n = kind == 0 ? a.Hq : a.Hkv;                          // heads of the kind
      const int h0 = kind == 0 ? 0 : (kind == 1 ? a.Hq : a.Hq + a.Hkv);  // the first one's place
      // y1 = inv (w1 cos x1 - w2 sin x2), y2 = inv (w2 cos x2 + w1 sin x1)
      float2 w1c[4], w2s[4], w2c[4], w1s[4];  // w2s with its sign
      if (kind < 2) {
        float2 c[4], s[4], v1[4], v2[4];
        load8(s_cos[warp] + 8 * sub, c);
        load8(s_sin[warp] + 8 * sub, s);
        load8(s_w[kind & 1] + 8 * sub, v1);
        load8(s_w[kind & 1] + D / 2 + 8 * sub, v2);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w1c[k] = mul2(v1[k], c[k]), w2c[k] = mul2(v2[k], c[k]), w1s[k] = mul2(v1[k], s[k]);
          w2s[k] = mul2(v2[k], make_float2(-s[k].x, -s[k].y));
        }
      }
      uint4 in[2][2], next[2][2];
      auto load = [&](int g, uint4 (&v)[2][2]) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int h = (g + z) * kHeads + in_group;
          v[z][0] = v[z][1] = make_uint4(0u, 0u, 0u, 0u);
          if (g + z < hi && h < n) {
            const __nv_bfloat16* at = src + static_cast<int64_t>(h0 + h) * D;
            v[z][0] = *reinterpret_cast<const uint4*>(at);
            v[z][1] = *reinterpret_cast<const uint4*>(at + D / 2);
          }
        }
      };
      load(lo, in);
      for (int g = lo; g < hi; g += 2) {
        load(g + 2, next);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int h = (g + z) * kHeads + in_group;
          const bool live = g + z < hi && h < n;
          float2 x[4], y[4];
          unpack8(in[z][0], x);
          unpack8(in[z][1], y);
          if (kind < 2) {
            float2 s2 = make_float2(0.f, 0.f), t2 = s2;
#pragma unroll
            for (int k = 0; k < 4; ++k) s2 = fma2(x[k], x[k], s2), t2 = fma2(y[k], y[k], t2);
            float ss = (s2.x + s2.y) + (t2.x + t2.y);
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float inv = rsqrtf(ss * (1.f / D) + a.eps);  // 2 ulp, far below a bf16 step
            const float2 inv2 = make_float2(inv, inv);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 p = mul2(x[k], inv2), q = mul2(y[k], inv2);
              x[k] = fma2(p, w1c[k], mul2(q, w2s[k]));
              y[k] = fma2(q, w2c[k], mul2(p, w1s[k]));
            }
          }
          if (live && (kind == 0 || (kind == 1 && a.k_out))) {
            __nv_bfloat16* dst = (kind == 0 ? a.q_out + (i * a.Hq + h) * D : a.k_out + (i * a.Hkv + h) * D) + 8 * sub;
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(dst) = ok ? pack8(x) : zero;
            *reinterpret_cast<uint4*>(dst + D / 2) = ok ? pack8(y) : zero;
          }
          if (kind > 0 && live && page_ok) {
            const int64_t base = (a.nhd ? (static_cast<int64_t>(page) * a.P + tok) * a.Hkv + h
                                        : (static_cast<int64_t>(page) * a.Hkv + h) * a.P + tok) * D + 8 * sub;
            void* pages = kind == 1 ? a.k_pages : a.v_pages;
            if (a.fp8) {
              const float sc = (kind == 1 ? a.k_scale : a.v_scale)[h];
              uint8_t* dst = static_cast<uint8_t*>(pages) + base;
              const float r = 1.f / sc;
              *reinterpret_cast<uint2*>(dst) = pack8_e4m3(x, sc, r);
              *reinterpret_cast<uint2*>(dst + D / 2) = pack8_e4m3(y, sc, r);
              if (!usual_scale(sc)) {
                *reinterpret_cast<uint2*>(dst) = pack8_quotient(x, sc);
                *reinterpret_cast<uint2*>(dst + D / 2) = pack8_quotient(y, sc);
              }
            } else {
              __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(pages) + base;
              *reinterpret_cast<uint4*>(dst) = kind == 2 ? in[z][0] : pack8(x);
              *reinterpret_cast<uint4*>(dst + D / 2) = kind == 2 ? in[z][1] : pack8(y);
            }
          }
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) in[z][0] = next[z][0], in[z][1] = next[z][1];
      }
    };
    auto clip = [&](int lo, int n, int& x, int& y) {  // the part's share of the groups [lo, lo + n)
      x = g0 > lo ? g0 - lo : 0;
      y = g1 < lo + n ? g1 - lo : n;
    };
    int x, y;
    clip(0, groups_q, x, y);
    if (x < y) run(std::integral_constant<int, 0>{}, x, y);
    clip(groups_q, groups_kv, x, y);
    if (x < y) run(std::integral_constant<int, 1>{}, x, y);
    clip(groups_q + groups_kv, groups_kv, x, y);
    if (x < y) run(std::integral_constant<int, 2>{}, x, y);
  }
}

}  // namespace
}  // namespace hpc

using namespace hpc;

extern "C" int hpc_prompt_prologue(const void* qkv, int64_t tokens, const int32_t* cu_seqlens, int32_t batch,
                                   const float* q_norm_w, const float* k_norm_w, float eps, float rope_theta,
                                   void* q_out, void* k_out, void* k_pages, void* v_pages, hpc_dtype kv_dtype,
                                   hpc_kv_layout kv_layout, const float* k_scale, const float* v_scale,
                                   int32_t num_pages, int32_t page_size, const int32_t* block_table,
                                   int32_t max_pages_per_req, const int32_t* seq_lens, int32_t num_heads,
                                   int32_t kv_heads, int32_t head_dim, uint32_t* status, void* stream) {
  if (tokens < 0) return fail(HPC_ERR_ARG, "tokens must be >= 0");
  if (tokens > INT32_MAX) return fail(HPC_ERR_SHAPE, "more tokens than int32 counts");
  if (!cu_seqlens || !q_norm_w || !k_norm_w || !k_pages || !v_pages || !block_table || !seq_lens || !status ||
      (tokens > 0 && (!qkv || !q_out)))
    return fail(HPC_ERR_ARG, "null pointer argument");
  if (kv_dtype != HPC_BF16 && kv_dtype != HPC_E4M3) return fail(HPC_ERR_DTYPE, "kv_dtype must be BF16 or E4M3");
  if (kv_layout != HPC_HND && kv_layout != HPC_NHD) return fail(HPC_ERR_ARG, "kv_layout must be HND or NHD");
  const bool fp8 = kv_dtype == HPC_E4M3;
  if (fp8 && (!k_scale || !v_scale)) return fail(HPC_ERR_ARG, "E4M3 cache needs k_scale and v_scale");
  if (batch < 1 || num_heads < 1 || kv_heads < 1 || num_pages < 1 || page_size < 1 || max_pages_per_req < 1)
    return fail(HPC_ERR_ARG, "sizes must be >= 1");
  if (num_heads % kv_heads) return fail(HPC_ERR_SHAPE, "num_heads %% kv_heads != 0");
  if (head_dim != 64 && head_dim != 128) return fail(HPC_ERR_SHAPE, "head_dim must be 64 or 128");
  if (!(rope_theta > 0.f) || !(eps >= 0.f)) return fail(HPC_ERR_ARG, "rope_theta must be > 0 and eps >= 0");
  if (!aligned16(qkv) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(k_pages) || !aligned16(v_pages))
    return fail(HPC_ERR_ALIGN, "qkv, q_out, k_out and the caches must be 16-byte aligned");
  if (tokens == 0) return HPC_OK;
  PpArgs a = {};
  a.qkv = static_cast<const __nv_bfloat16*>(qkv);
  a.cu = cu_seqlens;
  a.seq_lens = seq_lens;
  a.q_w = q_norm_w;
  a.k_w = k_norm_w;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.table = block_table;
  a.status = status;
  a.tokens = tokens;
  a.max_pages = max_pages_per_req;
  a.log2_theta = std::log2(static_cast<double>(rope_theta));
  a.eps = eps;
  a.batch = batch;
  a.Hq = num_heads;
  a.Hkv = kv_heads;
  a.num_pages = num_pages;
  a.P = page_size;
  a.nhd = kv_layout == HPC_NHD;
  a.fp8 = fp8;
  const int sms = device_sm_count() > 0 ? device_sm_count() : 148;
  const int per_group = 512 / head_dim;  // heads a warp takes at a time
  const int groups = (num_heads + per_group - 1) / per_group + 2 * ((kv_heads + per_group - 1) / per_group);
  int64_t blocks = (tokens * groups + kPpWarps - 1) / kPpWarps;
  const int64_t cap = static_cast<int64_t>(sms) * kPpCtas;
  if (blocks > cap) blocks = cap;
  auto kern = head_dim == 128 ? prompt_prologue_kernel<128> : prompt_prologue_kernel<64>;
  const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kPpThreads), 0,
                                   static_cast<cudaStream_t>(stream), a);
  return launched(e, "prompt_prologue_kernel");
}
