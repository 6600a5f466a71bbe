// paged_decode.cu -- attention of one decode query per head over paged caches.
//
// FastKV (gist.science 2502.01068) sections 1 and 2.B: decoding is bound by
// reading the retained entries; StructKV (gist.science 2604.06746) section
// 2.A: attention accumulated per token.  With entry j of KV head g in page
// table[j / page], and query head h of the group:
//     s_j = scale * q_h . k_j,  out_h = sum_j exp(s_j - lse_h) v_j,  weights_j += sum_h exp(s_j - lse_h).
#include <algorithm>

#include <cuda_bf16.h>

#include "paged.cuh"
#include "tc.cuh"

namespace kvc {
namespace {

constexpr int kPdThreads = 256;
constexpr int kPdWarps = kPdThreads / 32;
constexpr int kPdMaxG = 16;
constexpr double kLog2e = 1.4426950408889634;
constexpr double kLn2 = 0.6931471805599453;

struct PdArgs {
  Paged c;
  const uint16_t* q;
  int64_t q_sb, q_sh;
  int H, G;
  float c2;  // scale * log2(e)
  int64_t max_len;
  int accumulate;
  float* out;     // [B][H][d]
  float* lse;     // [B][H] or nullptr
  float* logits;  // [B][H][max_len], log2 domain (accumulate)
  int32_t* err;
};

// CTA (KV head, sequence); entry j belongs to warp j % 8, its lanes hold D/32
// dimensions each, with one online softmax per head and warp.
template <int D>
__global__ void __launch_bounds__(kPdThreads) paged_decode_kernel(const PdArgs a) {
  constexpr int kDL = D / 32;
  extern __shared__ float sm[];  // [warps][G]: max, sum; [warps][G][D]: output rows
  __shared__ int bad;
  pdl_wait();
  const Paged& c = a.c;
  const int g = blockIdx.x, b = blockIdx.y, G = a.G;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t n = c.seq_lens[b];
  if (tid == 0) bad = n < 0 || n > a.max_len;
  __syncthreads();
  if (!bad)
    for (int64_t s = (int64_t)tid * c.page; s < n; s += (int64_t)kPdThreads * c.page)
      if (c.page_of(b, s) < 0) bad = 1;
  __syncthreads();
  const int64_t len = bad ? 0 : n;
  if (bad && tid == 0) set_dev_err(a.err, KVC_DEV_ERR_PAGES);
  float* sm_m = sm;
  float* sm_l = sm + kPdWarps * G;
  float* sm_o = sm + 2 * kPdWarps * G;
  for (int hl = 0; hl < G; ++hl) {
    const int h = g * G + hl;
    float q[kDL], o[kDL], m = -INFINITY, l = 0.f;
    for (int e = 0; e < kDL; ++e) {
      q[e] = __uint_as_float((uint32_t)a.q[(int64_t)b * a.q_sb + (int64_t)h * a.q_sh + lane * kDL + e] << 16);
      o[e] = 0.f;
    }
    for (int64_t j = warp; j < len; j += kPdWarps) {
      const int64_t row = c.row(c.page_of(b, j), g, j) + lane * kDL;
      float s = 0.f;
      for (int e = 0; e < kDL; ++e) s += q[e] * __uint_as_float((uint32_t)c.k[row + e] << 16);
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= a.c2;
      if (a.accumulate && lane == 0) a.logits[((int64_t)b * a.H + h) * a.max_len + j] = s;
      const float mn = fmaxf(m, s);
      const float al = m == -INFINITY ? 0.f : exp2f(m - mn), p = exp2f(s - mn);
      l = l * al + p;
      for (int e = 0; e < kDL; ++e) o[e] = o[e] * al + p * __uint_as_float((uint32_t)c.v[row + e] << 16);
      m = mn;
    }
    if (lane == 0) {
      sm_m[warp * G + hl] = m;
      sm_l[warp * G + hl] = l;
    }
    for (int e = 0; e < kDL; ++e) sm_o[(warp * G + hl) * D + lane * kDL + e] = o[e];
  }
  __syncthreads();
  for (int i = tid; i < G * D; i += kPdThreads) {
    const int hl = i / D, e = i % D;
    float M = -INFINITY, L = 0.f, O = 0.f;
    for (int w = 0; w < kPdWarps; ++w) M = fmaxf(M, sm_m[w * G + hl]);
    for (int w = 0; w < kPdWarps; ++w) {
      const float mw = sm_m[w * G + hl], f = mw == -INFINITY ? 0.f : exp2f(mw - M);
      L += f * sm_l[w * G + hl];
      O += f * sm_o[(w * G + hl) * D + e];
    }
    const int64_t bh = (int64_t)b * a.H + g * G + hl;
    a.out[bh * D + e] = len > 0 ? O / L : 0.f;
    if (e == 0) {
      const float z = len > 0 ? M + log2f(L) : -INFINITY;
      if (a.lse) a.lse[bh] = (float)((double)z * kLn2);
    }
  }
  if (!a.accumulate) return;
  __syncthreads();
  for (int64_t j = tid; j < len; j += kPdThreads) {
    float w = 0.f;
    for (int hl = 0; hl < G; ++hl) {
      const float* sl = a.logits + ((int64_t)b * a.H + g * G + hl) * a.max_len;
      float M = -INFINITY, L = 0.f;
      for (int x = 0; x < kPdWarps; ++x) M = fmaxf(M, sm_m[x * G + hl]);
      for (int x = 0; x < kPdWarps; ++x)
        if (sm_m[x * G + hl] != -INFINITY) L += exp2f(sm_m[x * G + hl] - M) * sm_l[x * G + hl];
      w += exp2f(sl[j] - M) / L;
    }
    c.weights[c.entry(c.page_of(b, j), g, j)] += w;
  }
}

kvc_status check_paged_decode(const Paged& c, int32_t H, int64_t max_len) {
  KVC_CHECK_ARG(H >= 1 && H % c.Hkv == 0, "num_heads must be a positive multiple of num_kv_heads");
  if (H / c.Hkv > kPdMaxG) return fail(KVC_ERR_UNSUPPORTED, "at most 16 query heads per KV head");
  KVC_CHECK_ARG(max_len >= 1 && max_len <= c.room(), "need 1 <= max_len <= max_pages * page_size");
  return KVC_OK;
}

size_t paged_decode_ws_bytes(const Paged& c, int32_t H, int64_t max_len, int32_t accumulate) {
  return kWsAlign + (accumulate ? round_up((size_t)c.batch * H * (size_t)max_len * 4, kWsAlign) : 0);
}

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" kvc_status kvc_paged_decode_workspace_size(const kvc_paged_cache* c, int32_t num_heads, int64_t max_len,
                                                      int32_t accumulate, size_t* bytes) {
  clear_error();
  Paged p;
  kvc_status s = check_paged(c, &p);
  if (s == KVC_OK) s = check_paged_decode(p, num_heads, max_len);
  if (s != KVC_OK) return s;
  KVC_CHECK_ARG(bytes != nullptr, "bytes must be non-NULL");
  *bytes = paged_decode_ws_bytes(p, num_heads, max_len, accumulate);
  return KVC_OK;
}

extern "C" kvc_status kvc_paged_decode_attention(const kvc_paged_cache* c, const uint16_t* q, int64_t q_stride_b,
                                                 int64_t q_stride_h, int32_t num_heads, float scale, int64_t max_len,
                                                 int32_t accumulate, float* out, float* lse, void* ws,
                                                 size_t ws_bytes, int32_t* dev_err, void* stream) {
  clear_error();
  PdArgs a{};
  kvc_status s = check_paged(c, &a.c);
  if (s == KVC_OK) s = check_paged_pointers(a.c);
  if (s == KVC_OK) s = check_paged_decode(a.c, num_heads, max_len);
  if (s != KVC_OK) return s;
  KVC_CHECK_ARG(q && out && aligned(q, 16) && aligned(out, 16), "q and out must be non-NULL and 16-byte aligned");
  KVC_CHECK_ARG(q_stride_b >= 0 && q_stride_h >= 0 && q_stride_b % 8 == 0 && q_stride_h % 8 == 0,
                "strides of q must be multiples of 8 elements");
  KVC_CHECK_ARG(scale > 0.f && scale < 1e30f, "scale must be positive and finite");
  KVC_CHECK_ARG(!accumulate || a.c.weights, "accumulating needs the cache's weights");
  if (!ws || ws_bytes < paged_decode_ws_bytes(a.c, num_heads, max_len, accumulate) || !aligned(ws, kWsAlign))
    return fail(KVC_ERR_WORKSPACE, "paged decode workspace missing, too small or not 256-B aligned");
  a.q = q;
  a.q_sb = q_stride_b;
  a.q_sh = q_stride_h;
  a.H = num_heads;
  a.G = num_heads / a.c.Hkv;
  a.c2 = (float)((double)scale * kLog2e);
  a.max_len = max_len;
  a.accumulate = accumulate != 0;
  a.out = out;
  a.lse = lse;
  a.logits = reinterpret_cast<float*>(static_cast<char*>(ws) + kWsAlign);
  a.err = dev_err;
  const int d = a.c.d;
  const size_t smem = (size_t)kPdWarps * a.G * (d + 2) * 4;
  const Launch l(dim3((unsigned)a.c.Hkv, (unsigned)a.c.batch), dim3(kPdThreads), smem, (cudaStream_t)stream);
  static ContextCache cache;
  s = once_per_context(cache, [] {
    KVC_CUDA_TRY(cudaFuncSetAttribute(paged_decode_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      kPdWarps * kPdMaxG * 130 * 4));
    KVC_CUDA_TRY(cudaFuncSetAttribute(paged_decode_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      kPdWarps * kPdMaxG * 130 * 4));
    return KVC_OK;
  });
  if (s != KVC_OK) return s;
  KVC_CUDA_TRY(d == 128 ? l.run(paged_decode_kernel<128>, a) : l.run(paged_decode_kernel<64>, a));
  count_launch();
  return KVC_OK;
}
