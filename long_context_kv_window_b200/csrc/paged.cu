// paged.cu -- the paged cache's writes: appending tokens, and eviction by
// accumulated attention weight.
//
// FastKV (gist.science 2502.01068) sections 2.A and 2.B: a budget of entries
// per KV head, the most recent tokens always kept; every decoding step reads
// the retained entries and adds one.  StructKV (gist.science 2604.06746)
// section 2.A: attention accumulated per token ranks the tokens.
#include <algorithm>

#include "paged.cuh"

namespace kvc {
namespace {

// ------------------------------------------------------------------- append
// A copy: per kept entry 2 d bf16 values of k and of v in, the same out, and
// (weight, position).  CTA (run of kAppRows entries, sequence); its items are
// 16-byte pieces in the order (piece, head, entry) -- the order in memory of
// the packed source -- and a thread requests kAppUnroll of them before its
// first store.  Lengths move on once every CTA has read them: the last CTA of
// the grid (a ticket counter, returned to zero) adds the new entries.
constexpr int kAppThreads = 256;
constexpr int kAppRows = 16;
constexpr int kAppUnroll = 4;

struct AppArgs {
  Paged c;
  const uint16_t* k;
  const uint16_t* v;
  int64_t sn, sh, total, max_seqlen;
  const int32_t* cu;   // nullptr: one token per sequence
  const int32_t* idx;  // [B][Hkv][kk] or nullptr
  int64_t kk;
  const float* scores;  // [Hkv][total] or nullptr
  uint32_t* ticket;
  int32_t* err;
};

// Sequence b's tokens [start, start + len), entries kept and first slot; an
// error bit where nothing of it is to be appended (kept = 0 then).
struct AppSeq {
  int64_t start, len, kept, slot;
  int32_t bad;
};
__device__ AppSeq app_seq(const AppArgs& a, int b) {
  AppSeq s{b, 1, 1, a.c.seq_lens[b], 0};
  if (a.cu) {
    s.start = a.cu[b];
    s.len = (int64_t)a.cu[b + 1] - s.start;
    if (s.start < 0 || s.len < 0 || s.start + s.len > a.total || s.len > a.max_seqlen) s.bad = KVC_DEV_ERR_SEQLENS;
  }
  s.kept = a.idx ? (s.len < a.kk ? s.len : a.kk) : s.len;
  if (!s.bad && (s.slot < 0 || s.slot + s.kept > a.c.room())) s.bad = KVC_DEV_ERR_PAGES;
  if (s.bad) s.len = s.kept = 0;
  return s;
}

__global__ void __launch_bounds__(kAppThreads) append_kernel(const AppArgs a) {
  __shared__ int last;
  pdl_wait();
  const int b = blockIdx.y;
  const Paged& c = a.c;
  const AppSeq q = app_seq(a, b);
  const int64_t r0 = (int64_t)blockIdx.x * kAppRows;
  const int rows = (int)(q.kept - r0 < kAppRows ? q.kept - r0 : kAppRows);  // <= 0 past the entries
  const int np = c.d / 8;                                                 // 16-byte pieces per row
  const int per_row = np * c.Hkv, items = rows * per_row;
  const int64_t npos = c.next_pos ? c.next_pos[b] : 0;
  for (int i0 = threadIdx.x; i0 < items; i0 += kAppThreads * kAppUnroll) {
    uint4 kv[kAppUnroll], vv[kAppUnroll];
    int64_t dst[kAppUnroll];
#pragma unroll
    for (int u = 0; u < kAppUnroll; ++u) {
      const int i = i0 + u * kAppThreads;
      dst[u] = -1;
      if (i >= items) continue;
      const int r = i / per_row, g = (i % per_row) / np, piece = i % np;
      const int64_t slot = q.slot + r0 + r;
      int64_t t = r0 + r;  // local token
      if (a.idx) {
        t = a.idx[((int64_t)b * c.Hkv + g) * a.kk + r0 + r];
        if (t < 0 || t >= q.len) t = -1;
      }
      const int p = c.page_of(b, slot);
      if (p < 0) {
        set_dev_err(a.err, KVC_DEV_ERR_PAGES);
        continue;
      }
      kv[u] = vv[u] = make_uint4(0u, 0u, 0u, 0u);
      if (t >= 0) {
        const int64_t src = (q.start + t) * a.sn + (int64_t)g * a.sh + piece * 8;
        kv[u] = __ldcs(reinterpret_cast<const uint4*>(a.k + src));
        vv[u] = __ldcs(reinterpret_cast<const uint4*>(a.v + src));
      } else {
        set_dev_err(a.err, KVC_DEV_ERR_INDEX);
      }
      dst[u] = c.row(p, g, slot) + piece * 8;
      if (piece == 0) {
        const int64_t e = c.entry(p, g, slot);
        if (c.pos) c.pos[e] = t >= 0 ? (int32_t)(npos + t) : -1;
        if (c.weights) c.weights[e] = a.scores && t >= 0 ? a.scores[(int64_t)g * a.total + q.start + t] : 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < kAppUnroll; ++u)
      if (dst[u] >= 0) {
        *reinterpret_cast<uint4*>(c.k + dst[u]) = kv[u];
        *reinterpret_cast<uint4*>(c.v + dst[u]) = vv[u];
      }
  }
  __syncthreads();  // every thread has read the lengths
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == gridDim.x * gridDim.y - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int s = threadIdx.x; s < c.batch; s += kAppThreads) {
    const AppSeq n = app_seq(a, s);
    if (n.bad) set_dev_err(a.err, n.bad);
    c.seq_lens[s] += (int32_t)n.kept;
    if (c.next_pos) c.next_pos[s] += (int32_t)n.len;
  }
  if (threadIdx.x == 0) *a.ticket = 0u;
}

// -------------------------------------------------------------------- evict
// CTA (KV head, sequence).  Keys are the order-preserving uint32 image of the
// weights (recent entries the largest key, NaN 0); a radix select finds the
// key T of the budget-th largest; one pass in slot order ranks the keys equal
// to T and lists the slots given up below the budget and the kept slots above
// it; their rows are then moved pairwise.  Sources lie at or above the budget
// and destinations below it, so the moves need no order among themselves.
constexpr int kEvThreads = 1024;
constexpr uint32_t kRecentKey = 0xFFFFFFFFu;

struct EvArgs {
  Paged c;
  int64_t max_len, budget, recent;
  int64_t max_move;
  uint32_t* tickets;  // [batch]
  uint32_t* keys;     // [batch*Hkv][max_len]
  int32_t* moves;     // [batch*Hkv][2][max_move]: slots given up, kept slots above the budget
  int32_t* err;
};

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (!(w == w)) return 0u;                       // NaN: below -inf
  const uint32_t u = __float_as_uint(w + 0.f);    // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of `v` over the CTA's threads, and the total.
__device__ __forceinline__ int block_prefix(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const int before = warp == 0 ? 0 : warp_sums[warp - 1];
  *total = warp_sums[31];
  __syncthreads();
  return before + x - v;
}

__global__ void __launch_bounds__(kEvThreads) evict_kernel(const EvArgs a) {
  __shared__ uint32_t hist[2048];
  __shared__ int warp_sums[32];
  __shared__ int bad, sh_bin, sh_left;
  pdl_wait();
  const Paged& c = a.c;
  const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int64_t n = c.seq_lens[b];
  if (tid == 0) bad = n < 0 || n > a.max_len;
  __syncthreads();
  if (!bad)
    for (int64_t s = (int64_t)tid * c.page; s < n; s += (int64_t)kEvThreads * c.page)
      if (c.page_of(b, s) < 0) bad = 1;
  __syncthreads();
  if (bad) {
    if (tid == 0) set_dev_err(a.err, KVC_DEV_ERR_PAGES);
  } else if (n > a.budget) {
    const int64_t limit = a.recent > 0 ? (int64_t)c.next_pos[b] - a.recent : 0;
    uint32_t* keys = a.keys + ((int64_t)b * c.Hkv + g) * a.max_len;
    for (int64_t s = tid; s < n; s += kEvThreads) {
      const int64_t e = c.entry(c.page_of(b, s), g, s);
      keys[s] = a.recent > 0 && c.pos[e] >= limit ? kRecentKey : weight_key(c.weights[e]);
    }
    // the budget-th largest key, 11 + 11 + 10 bits from the top
    uint32_t prefix = 0, mask = 0;
    int left = (int)a.budget;  // kept keys that match the prefix so far
    for (int level = 0; level < 3; ++level) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bins = level == 2 ? 1024 : 2048;
      for (int i = tid; i < 2048; i += kEvThreads) hist[i] = 0u;
      __syncthreads();
      for (int64_t s = tid; s < n; s += kEvThreads) {
        const uint32_t key = keys[s];
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1u);
      }
      __syncthreads();
      // thread t holds two bins from the top: 2t and 2t + 1 counted from the largest
      const int h0 = 2 * tid < bins ? (int)hist[bins - 1 - 2 * tid] : 0;
      const int h1 = 2 * tid + 1 < bins ? (int)hist[bins - 2 - 2 * tid] : 0;
      int total;
      const int above = block_prefix(h0 + h1, warp_sums, &total);
      if (above < left && left <= above + h0) {
        sh_bin = bins - 1 - 2 * tid;
        sh_left = left - above;
      } else if (above + h0 < left && left <= above + h0 + h1) {
        sh_bin = bins - 2 - 2 * tid;
        sh_left = left - above - h0;
      }
      __syncthreads();
      prefix |= (uint32_t)sh_bin << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      left = sh_left;
      __syncthreads();
    }
    const uint32_t T = prefix;  // `left` of the keys equal to T are kept, the lowest slots
    int32_t* give = a.moves + ((int64_t)b * c.Hkv + g) * 2 * a.max_move;
    int32_t* take = give + a.max_move;
    int eq_seen = 0, n_give = 0, n_take = 0;
    for (int64_t s0 = 0; s0 < n; s0 += kEvThreads) {
      const int64_t s = s0 + tid;
      const uint32_t key = s < n ? keys[s] : 0u;
      const int eq = s < n && key == T;
      int total;
      const int rank = eq_seen + block_prefix(eq, warp_sums, &total);
      eq_seen += total;
      const bool kept = s < n && (key > T || (eq && rank < left));
      const int gv = s < n && s < a.budget && !kept, tk = s >= a.budget && kept;
      const int both = block_prefix(gv | (tk << 16), warp_sums, &total);
      if (gv) give[n_give + (both & 0xFFFF)] = (int32_t)s;
      if (tk) take[n_take + (both >> 16)] = (int32_t)s;
      n_give += total & 0xFFFF;
      n_take += total >> 16;
    }
    __syncthreads();
    const int np = c.d / 8;
    for (int i = tid; i < n_take * np; i += kEvThreads) {
      const int m = i / np, piece = i % np;
      const int64_t from = take[m], to = give[m];
      const int pf = c.page_of(b, from), pt = c.page_of(b, to);
      const int64_t src = c.row(pf, g, from) + piece * 8, dst = c.row(pt, g, to) + piece * 8;
      *reinterpret_cast<uint4*>(c.k + dst) = *reinterpret_cast<const uint4*>(c.k + src);
      *reinterpret_cast<uint4*>(c.v + dst) = *reinterpret_cast<const uint4*>(c.v + src);
      if (piece == 0) {
        const int64_t ef = c.entry(pf, g, from), et = c.entry(pt, g, to);
        c.weights[et] = c.weights[ef];
        if (c.pos) c.pos[et] = c.pos[ef];
      }
    }
  }
  // the length of the sequence moves once all its heads have read it
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(&a.tickets[b], 1u) == (uint32_t)c.Hkv - 1) {
      if (!bad && n > a.budget) c.seq_lens[b] = (int32_t)a.budget;
      a.tickets[b] = 0u;
    }
  }
}

int64_t evict_max_move(int64_t max_len, int64_t budget) {
  return std::max<int64_t>(0, std::min(budget, max_len - budget));
}

kvc_status check_evict(const Paged& c, int64_t max_len, int64_t budget) {
  KVC_CHECK_ARG(max_len >= 1 && max_len <= c.room(), "need 1 <= max_len <= max_pages * page_size");
  KVC_CHECK_ARG(budget >= 1 && budget < (int64_t(1) << 31), "need 1 <= budget < 2^31");
  return KVC_OK;
}

size_t evict_ws_bytes(const Paged& c, int64_t max_len, int64_t budget) {
  const size_t bg = (size_t)c.batch * c.Hkv;
  return round_up((size_t)c.batch * 4, kWsAlign) + round_up(bg * (size_t)max_len * 4, kWsAlign) +
         round_up(bg * 2 * (size_t)std::max<int64_t>(1, evict_max_move(max_len, budget)) * 4, kWsAlign);
}

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" kvc_status kvc_paged_append_workspace_size(const kvc_paged_cache* c, size_t* bytes) {
  clear_error();
  Paged p;
  const kvc_status s = check_paged(c, &p);
  if (s != KVC_OK) return s;
  KVC_CHECK_ARG(bytes != nullptr, "bytes must be non-NULL");
  *bytes = kWsAlign;
  return KVC_OK;
}

extern "C" kvc_status kvc_paged_append(const kvc_paged_cache* c, const uint16_t* k, const uint16_t* v,
                                       int64_t stride_n, int64_t stride_h, const int32_t* cu_seqlens, int64_t total,
                                       int64_t max_seqlen, const int32_t* idx, int64_t kk, const float* scores,
                                       void* ws, size_t ws_bytes, int32_t* dev_err, void* stream) {
  clear_error();
  AppArgs a{};
  kvc_status s = check_paged(c, &a.c);
  if (s == KVC_OK) s = check_paged_pointers(a.c);
  if (s != KVC_OK) return s;
  KVC_CHECK_ARG(k && v && aligned(k, 16) && aligned(v, 16), "k and v must be non-NULL and 16-byte aligned");
  KVC_CHECK_ARG(stride_n >= 0 && stride_h >= 0 && stride_n % 8 == 0 && stride_h % 8 == 0,
                "strides must be multiples of 8 elements");
  KVC_CHECK_ARG(total >= 0 && total < (int64_t(1) << 31), "need 0 <= total < 2^31");
  KVC_CHECK_ARG(cu_seqlens ? max_seqlen >= 0 && max_seqlen < (int64_t(1) << 31) : total == a.c.batch && max_seqlen == 1,
                "without cu_seqlens every sequence brings one token (total == batch, max_seqlen == 1)");
  KVC_CHECK_ARG(!idx || kk >= 0, "need kk >= 0");
  if (!ws || ws_bytes < kWsAlign || !aligned(ws, kWsAlign))
    return fail(KVC_ERR_WORKSPACE, "append workspace missing, too small or not 256-B aligned");
  a.k = k;
  a.v = v;
  a.sn = stride_n;
  a.sh = stride_h;
  a.total = total;
  a.max_seqlen = max_seqlen;
  a.cu = cu_seqlens;
  a.idx = idx;
  a.kk = kk;
  a.scores = scores;
  a.ticket = static_cast<uint32_t*>(ws);
  a.err = dev_err;
  const int64_t most = idx ? std::min(kk, max_seqlen) : max_seqlen;
  const unsigned runs = (unsigned)std::max<int64_t>(1, (most + kAppRows - 1) / kAppRows);
  const Launch l(dim3(runs, (unsigned)a.c.batch), dim3(kAppThreads), 0, (cudaStream_t)stream);
  KVC_CUDA_TRY(l.run(append_kernel, a));
  count_launch();
  return KVC_OK;
}

extern "C" kvc_status kvc_paged_evict_workspace_size(const kvc_paged_cache* c, int64_t max_len, int64_t budget,
                                                     size_t* bytes) {
  clear_error();
  Paged p;
  kvc_status s = check_paged(c, &p);
  if (s == KVC_OK) s = check_evict(p, max_len, budget);
  if (s != KVC_OK) return s;
  KVC_CHECK_ARG(bytes != nullptr, "bytes must be non-NULL");
  *bytes = evict_ws_bytes(p, max_len, budget);
  return KVC_OK;
}

extern "C" kvc_status kvc_paged_evict(const kvc_paged_cache* c, int64_t max_len, int64_t budget, int64_t recent,
                                      void* ws, size_t ws_bytes, int32_t* dev_err, void* stream) {
  clear_error();
  EvArgs a{};
  kvc_status s = check_paged(c, &a.c);
  if (s == KVC_OK) s = check_paged_pointers(a.c);
  if (s == KVC_OK) s = check_evict(a.c, max_len, budget);
  if (s != KVC_OK) return s;
  KVC_CHECK_ARG(recent >= 0 && recent <= budget, "need 0 <= recent <= budget");
  KVC_CHECK_ARG(a.c.weights, "eviction ranks by the cache's weights: they must be non-NULL");
  KVC_CHECK_ARG(recent == 0 || a.c.pos, "keeping recent entries needs pos and next_pos");
  if (!ws || ws_bytes < evict_ws_bytes(a.c, max_len, budget) || !aligned(ws, kWsAlign))
    return fail(KVC_ERR_WORKSPACE, "evict workspace missing, too small or not 256-B aligned");
  const size_t bg = (size_t)a.c.batch * a.c.Hkv;
  a.max_len = max_len;
  a.budget = budget;
  a.recent = recent;
  a.max_move = std::max<int64_t>(1, evict_max_move(max_len, budget));
  WsCursor wc{static_cast<char*>(ws), ws_bytes};
  a.tickets = wc.take<uint32_t>((size_t)a.c.batch);
  a.keys = wc.take<uint32_t>(bg * (size_t)max_len);
  a.moves = wc.take<int32_t>(bg * 2 * (size_t)a.max_move);
  if (!wc.ok) return fail(KVC_ERR_WORKSPACE, "evict workspace too small");
  a.err = dev_err;
  const Launch l(dim3((unsigned)a.c.Hkv, (unsigned)a.c.batch), dim3(kEvThreads), 0, (cudaStream_t)stream);
  KVC_CUDA_TRY(l.run(evict_kernel, a));
  count_launch();
  return KVC_OK;
}
