// paged.cu -- the paged cache's writes: appending tokens, and eviction by
// accumulated attention weight.
//
// FastKV (gist.science 2502.01068) sections 2.A and 2.B: a budget of entries
// per KV head, the most recent tokens always kept; every decoding step reads
// the retained entries and adds one.  StructKV (gist.science 2604.06746)
// section 2.A: attention accumulated per token ranks the tokens.
#include <cooperative_groups.h>

#include <algorithm>

#include "paged.cuh"

namespace cg = cooperative_groups;

namespace kvc {
namespace {

// ------------------------------------------------------------------- append
// A copy: per kept entry and KV head d bf16 values of k and of v in, the same
// out, and (weight, position).  A warp takes kRowItems (entry, head) items: one
// lane each finds its token, half the lanes (or a quarter, d = 64) request an
// item's k row and as many its v row, all items before the first store, and
// the lanes of the items find the places meanwhile.  Items go head by head
// within an entry where the tokens lie so (a whole prompt), entry by entry
// within a head where a list selects them (the list and the pages then run
// on).  Lengths move on once every CTA has read them: the last CTA of the grid (a ticket counter,
// returned to zero) adds the new entries.  8 x 8 x 1024 selected rows (67 MB
// in all) take 19.6 us cold, 3.4 TB/s in and out together (DRAM reads 1.9 TB/s
// at 44 % of the warps).  What bounds it is the chain of lengths, list, rows and
// stores that each of 1024 CTAs goes through once, four at a time on an SM: 1.7
// waves with nothing of the next rows under way.  One token for each of 64 sequences is four dependent round trips, 5 us.
constexpr int kAppThreads = 256;

// A warp copies up to kRowItems items, lane i < kRowItems holding item i's
// place in the source (elements; -1: a zero row) and, once found(), in the
// destination (-1: nothing is written).
constexpr int kRowItems = 8;
template <int D, class F>
__device__ __forceinline__ void copy_rows(const uint16_t* ks, const uint16_t* vs, uint16_t* kd, uint16_t* vd, int64_t src,
                                          F&& found) {
  constexpr int kPieces = D / 8;             // 16-byte pieces per row
  constexpr int kAtOnce = 32 / (2 * kPieces);  // items per instruction
  const int lane = threadIdx.x & 31, sub = lane / (2 * kPieces), piece = lane % kPieces * 8;
  const bool value = (lane / kPieces) & 1;
  const uint16_t* from = value ? vs : ks;
  uint16_t* to = value ? vd : kd;
  uint4 x[kRowItems / kAtOnce];
#pragma unroll
  for (int u = 0; u < kRowItems / kAtOnce; ++u) {
    const int64_t s = __shfl_sync(0xffffffffu, src, u * kAtOnce + sub);
    x[u] = s >= 0 ? __ldcs(reinterpret_cast<const uint4*>(from + s + piece)) : make_uint4(0u, 0u, 0u, 0u);
  }
  const int64_t dst = found();  // while the rows are on their way
#pragma unroll
  for (int u = 0; u < kRowItems / kAtOnce; ++u) {
    const int64_t d = __shfl_sync(0xffffffffu, dst, u * kAtOnce + sub);
    if (d >= 0) *reinterpret_cast<uint4*>(to + d + piece) = x[u];
  }
}

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

constexpr int kAppSpan = kAppThreads / 32 * kRowItems;
template <int D>
__global__ void __launch_bounds__(kAppThreads) append_kernel(const AppArgs a) {
  __shared__ int last;
  pdl_wait();
  const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Paged& c = a.c;
  const AppSeq q = app_seq(a, b);
  const unsigned kept = (unsigned)q.kept, heads = (unsigned)c.Hkv, items = kept * heads;  // below 2^31
  const unsigned i0 = blockIdx.x * kAppSpan + warp * kRowItems;
  if (i0 < items) {
    int64_t src = -1, t = -1, r = 0;  // t: local token
    int g = 0;
    const bool mine = lane < kRowItems && i0 + lane < items;
    if (mine) {
      const unsigned i = i0 + lane, by = a.idx ? kept : heads, hi = i / by, lo = i - hi * by;
      r = a.idx ? lo : hi;
      g = (int)(a.idx ? hi : lo);
      t = a.idx ? a.idx[((int64_t)b * c.Hkv + g) * a.kk + r] : r;
      if (t < 0 || t >= q.len) t = -1;
      if (t >= 0) src = (q.start + t) * a.sn + (int64_t)g * a.sh;
    }
    copy_rows<D>(a.k, a.v, c.k, c.v, src, [&]() -> int64_t {
      if (!mine) return -1;
      const int64_t slot = q.slot + r;
      const int p = c.page_of(b, slot);
      if (t < 0) set_dev_err(a.err, KVC_DEV_ERR_INDEX);
      if (p < 0) {
        set_dev_err(a.err, KVC_DEV_ERR_PAGES);
        return -1;
      }
      const int64_t e = c.entry(p, g, slot);
      if (c.pos) c.pos[e] = t >= 0 ? (int32_t)(c.next_pos[b] + t) : -1;
      if (c.weights) c.weights[e] = a.scores && t >= 0 ? a.scores[(int64_t)g * a.total + q.start + t] : 0.f;
      return c.row(p, g, slot);
    });
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
// A pair (KV head, sequence) is a CTA, or a cluster of up to 8 where the pairs
// are few and long, each with a run of the slots.  Keys are the
// order-preserving uint32 image of the weights (recent entries the largest key,
// NaN 0), kept in shared memory where they fit.  One entry too many -- every
// decoding step -- needs the lowest ranked entry only, one reduction.
// Otherwise the budget-th largest key T is found by histograms of 2048 equal
// bins over the range of the keys, then over the bin that holds it, until the
// bin is one key or is kept whole (weights span few exponents, so bins over
// their range part them better than fixed
// digits do).  Warps then own runs of slots: counted with ballots, prefixed
// once over the warps, listed with ballots: the slots given up below the
// budget and the kept slots above it, both ascending.
// The rows are moved pairwise; sources lie at or above the budget and
// destinations below it, so the moves need no order among themselves.  Few
// moves are made by the CTA itself, many by a second kernel over all SMs.
// What bounds it are dependent round trips (table, weights, barriers), not
// bytes: 64 x 8 pairs of 1025 entries, one out, 10.9 us cold; 4 x 8 pairs,
// 32768 -> 2048, 30.7 us for the lists and 15.9 for 61440 moved rows.
constexpr uint32_t kRecentKey = 0xFFFFFFFFu;
constexpr int kEvBins = 2048;
constexpr int64_t kEvSmemKeys = 48 * 1024;  // keys of a CTA held in shared memory (192 KB)
constexpr int64_t kEvInline = 64;           // moves a pair's CTA makes itself: one per warp and item of 256 threads
constexpr int64_t kEvSmall = 4096;          // up to here a pair is a CTA of 256 threads, else of 1024
constexpr int kMvThreads = 256;
constexpr int kMvSpan = kMvThreads / 32 * kRowItems;  // moves per CTA of the second kernel

struct EvArgs {
  Paged c;
  int64_t max_len, budget, recent;
  int64_t max_move;
  uint32_t* tickets;  // [batch]
  int32_t* moves;     // [batch*Hkv]: moves of the pair
  int32_t* lists;     // [batch*Hkv][2][max_move]: slots given up, kept slots above the budget
  uint32_t* keys;     // [batch*Hkv][max_len], or nullptr: shared memory
  int in_place;       // the pair's first CTA makes the moves itself
  int cluster;        // CTAs per pair
  int resident;       // the grid runs at once
  int32_t* err;
};

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (!(w == w)) return 0u;                       // NaN: below -inf
  const uint32_t u = __float_as_uint(w + 0.f);    // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Moves [i0, i0 + kRowItems) of a pair's n, by one warp.
template <int D>
__device__ __forceinline__ void move_rows(const Paged& c, int b, int g, const int32_t* give, const int32_t* take, int i0,
                                          int n) {
  const int lane = threadIdx.x & 31;
  const bool mine = lane < kRowItems && i0 + lane < n;
  int64_t from = 0, src = -1;
  int pf = 0;
  if (mine) {
    from = take[i0 + lane];
    pf = c.page_of(b, from);
    src = c.row(pf, g, from);
  }
  copy_rows<D>(c.k, c.v, c.k, c.v, src, [&]() -> int64_t {
    if (!mine) return -1;
    const int64_t to = give[i0 + lane], ef = c.entry(pf, g, from);
    const int pt = c.page_of(b, to);
    const int64_t et = c.entry(pt, g, to);
    c.weights[et] = c.weights[ef];
    if (c.pos) c.pos[et] = c.pos[ef];
    return c.row(pt, g, to);
  });
}

// What the CTAs of a pair tell one another, each field written once.
struct EvShare {
  uint32_t lo, hi;      // smallest key; largest key that is not recent
  int low_slot, fresh;  // lowest ranked slot; recent entries
  int bad;              // a page id outside the pool
  int eq, give, take;   // keys equal to T; slots given up; kept slots above the budget
};

template <int kThreads>
__global__ void __launch_bounds__(kThreads) evict_kernel(const EvArgs a) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kPer = kEvBins / kThreads;  // bins per thread
  extern __shared__ uint32_t sm_keys[];
  __shared__ uint32_t hist[2][kEvBins];
  __shared__ uint32_t red[3][kWarps];
  __shared__ int cnt[2][kWarps];
  __shared__ EvShare sh;
  __shared__ int sh_bin, sh_left, sh_in;
  pdl_wait();
  if (a.resident) pdl_trigger();  // the kernel of the moves may be brought in
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = a.cluster, me = (int)blockIdx.x % cs;
  auto sync_pair = [&] {  // the CTAs of a pair
    if (cs > 1) cluster.sync(); else __syncthreads();
  };
  const Paged& c = a.c;
  const int g = (int)blockIdx.x / cs, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = c.seq_lens[b], budget = (int)std::min<int64_t>(a.budget, 0x7FFFFFFF);
  const int64_t pair = (int64_t)b * c.Hkv + g;
  int32_t* give = a.lists + pair * 2 * a.max_move;
  int32_t* take = give + a.max_move;
  bool bad = n < 0 || n > a.max_len;
  int n_moves = 0;
  if (!bad && n > budget) {  // the same for every CTA of the pair
    // ---- the keys of this CTA's slots [s0, s1), and the lowest ranked entry
    // (lowest key, then highest slot)
    const int seg = ((n + cs - 1) / cs + 31) / 32 * 32, s0 = min(n, me * seg), s1 = min(n, s0 + seg);
    uint32_t* keys = (a.keys ? a.keys + pair * a.max_len + s0 : sm_keys) - s0;  // indexed by slot
    const int64_t limit = a.recent > 0 ? (int64_t)c.next_pos[b] - a.recent : 0;
    // One entry too many: the only slot above the budget is the one that moves,
    // if any does, so its row is on its way while the keys are looked at.
    const bool one = n - budget == 1;
    const int np = c.d / 8;
    uint4 held = make_uint4(0u, 0u, 0u, 0u);
    float held_w = 0.f;
    int held_pos = 0;
    if (one && me == 0 && tid < 2 * np) {
      const int p = c.page_of(b, budget);
      if (p >= 0) {
        held = *reinterpret_cast<const uint4*>((tid < np ? c.k : c.v) + c.row(p, g, budget) + tid % np * 8);
        if (tid == 0) {
          const int64_t e = c.entry(p, g, budget);
          held_w = c.weights[e];
          if (c.pos) held_pos = c.pos[e];
        }
      }
    }
    uint32_t lo = kRecentKey, hi = 0u;
    int low_slot = -1, fresh = 0, gone = 0;
#pragma unroll 4
    for (int s = s0 + tid; s < s1; s += kThreads) {
      const int p = c.page_of(b, s);
      uint32_t key = 0u;
      if (p < 0) {
        gone = 1;
      } else {
        const int64_t e = c.entry(p, g, s);
        key = weight_key(c.weights[e]);
        if (a.recent > 0 && c.pos[e] >= limit) key = kRecentKey;
      }
      if (!one) keys[s] = key;
      if (key <= lo) {
        lo = key;
        low_slot = s;
      }
      if (key == kRecentKey) ++fresh; else hi = max(hi, key);
    }
    {
      const uint32_t lo_w = __reduce_min_sync(0xffffffffu, lo);
      const int slot_w = __reduce_max_sync(0xffffffffu, lo == lo_w ? low_slot : -1);
      const uint32_t hi_w = __reduce_max_sync(0xffffffffu, hi);
      const int fresh_w = __reduce_add_sync(0xffffffffu, fresh);
      const int gone_w = __any_sync(0xffffffffu, gone);
      if (lane == 0) {
        red[0][warp] = lo_w;
        red[1][warp] = (uint32_t)slot_w;
        red[2][warp] = hi_w;
        cnt[0][warp] = fresh_w;
        cnt[1][warp] = gone_w;
      }
    }
    __syncthreads();
    if (warp == 0) {
      const bool in = lane < kWarps;
      const uint32_t lo_w = in ? red[0][lane] : kRecentKey, lo_c = __reduce_min_sync(0xffffffffu, lo_w);
      const int slot_c = __reduce_max_sync(0xffffffffu, in && lo_w == lo_c ? (int)red[1][lane] : -1);
      const uint32_t hi_c = __reduce_max_sync(0xffffffffu, in ? red[2][lane] : 0u);
      const int fresh_c = __reduce_add_sync(0xffffffffu, in ? cnt[0][lane] : 0);
      const int bad_c = __any_sync(0xffffffffu, in && cnt[1][lane]);
      if (lane == 0) sh = EvShare{lo_c, hi_c, slot_c, fresh_c, bad_c, 0, 0, 0};
    }
    sync_pair();
    lo = kRecentKey;
    hi = 0u;
    low_slot = -1;
    fresh = 0;
    for (int r = 0; r < cs; ++r) {
      const EvShare& x = *cluster.map_shared_rank(&sh, r);
      if (x.lo < lo || (x.lo == lo && x.low_slot > low_slot)) low_slot = x.low_slot;
      lo = min(lo, x.lo);
      hi = max(hi, x.hi);
      fresh += x.fresh;
      bad |= x.bad != 0;
    }
    if (!bad && one) {
      if (low_slot < budget && me == 0 && tid < 2 * np) {
        const int p = c.page_of(b, low_slot);
        *reinterpret_cast<uint4*>((tid < np ? c.k : c.v) + c.row(p, g, low_slot) + tid % np * 8) = held;
        if (tid == 0) {
          const int64_t e = c.entry(p, g, low_slot);
          c.weights[e] = held_w;
          if (c.pos) c.pos[e] = held_pos;
        }
      }
    } else if (!bad) {
      // ---- T: `left` of the keys equal to T are kept, the lowest slots
      uint32_t T = kRecentKey;
      int left = budget;
      if (fresh < budget) {
        left = budget - fresh;
        for (int level = 0;; ++level) {
          T = lo;
          if (lo == hi) break;
          // two histograms in turn: the other CTAs have read this one's last
          // use before they passed the last level's barrier
          uint32_t* h_me = hist[level & 1];
          const int bits = 32 - __clz(hi - lo), sft = bits > 11 ? bits - 11 : 0;
          for (int i = tid; i < kEvBins; i += kThreads) h_me[i] = 0u;
          __syncthreads();
#pragma unroll 4
          for (int s = s0 + tid; s < s1; s += kThreads) {
            const uint32_t key = keys[s];
            if (key >= lo && key <= hi) atomicAdd(&h_me[(key - lo) >> sft], 1u);
          }
          sync_pair();
          int h[kPer], sum = 0;  // this thread's bins over all CTAs, from the largest down
#pragma unroll
          for (int u = 0; u < kPer; ++u) h[u] = 0;
          for (int r = 0; r < cs; ++r) {
            const uint32_t* hr = cluster.map_shared_rank(h_me, r);
#pragma unroll
            for (int u = 0; u < kPer; ++u) h[u] += (int)hr[kEvBins - 1 - kPer * tid - u];
          }
#pragma unroll
          for (int u = 0; u < kPer; ++u) sum += h[u];
          int inc = sum;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
          }
          if (lane == 31) cnt[0][warp] = inc;
          __syncthreads();
          int above = inc - sum;
          for (int w = 0; w < warp; ++w) above += cnt[0][w];
#pragma unroll
          for (int u = 0; u < kPer; ++u) {
            if (above < left && left <= above + h[u]) {
              sh_bin = kEvBins - 1 - kPer * tid - u;
              sh_left = left - above;
              sh_in = h[u];
            }
            above += h[u];
          }
          __syncthreads();
          left = sh_left;
          lo += (uint32_t)sh_bin << sft;
          hi = min(hi, lo + ((1u << sft) - 1u));
          T = lo;
          const bool whole = sh_in == left;
          __syncthreads();
          if (whole) {  // every key of the bin is kept
            left = n;
            break;
          }
          if (sft == 0) break;
        }
      }
      // ---- ranks and lists; a warp owns a run of the CTA's slots
      const int run = (s1 - s0 + kThreads - 1) / kThreads * 32, w0 = min(s1, s0 + warp * run), w1 = min(s1, w0 + run);
      int eq_before = 0;  // keys equal to T before this warp's slots (not needed where all are kept)
      if (left < n) {
        int eq = 0, eq_all = 0;
        for (int s = w0 + lane; s < w1; s += 32) eq += keys[s] == T;
        eq = __reduce_add_sync(0xffffffffu, eq);
        if (lane == 0) cnt[0][warp] = eq;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) eq_before += cnt[0][w];
          eq_all += cnt[0][w];
        }
        if (tid == 0) sh.eq = eq_all;
        sync_pair();
        for (int r = 0; r < me; ++r) eq_before += cluster.map_shared_rank(&sh, r)->eq;
      }
      int at[2] = {0, 0};  // slots given up and slots taken before this warp's
      for (int phase = 0; phase < 2; ++phase) {
        int rank = eq_before, n_give = at[0], n_take = at[1];
        const unsigned below = (1u << lane) - 1u;
        for (int sw = w0; sw < w1; sw += 32) {
          const int s = sw + lane;
          const bool in = s < w1;
          const uint32_t key = in ? keys[s] : 0u;
          const unsigned eqs = __ballot_sync(0xffffffffu, in && key == T);
          const bool kept = in && (key > T || (key == T && rank + __popc(eqs & below) < left));
          const unsigned gv = __ballot_sync(0xffffffffu, in && s < budget && !kept);
          const unsigned tk = __ballot_sync(0xffffffffu, s >= budget && kept);
          if (phase == 1) {
            if ((gv >> lane) & 1) give[n_give + __popc(gv & below)] = s;
            if ((tk >> lane) & 1) take[n_take + __popc(tk & below)] = s;
          }
          rank += __popc(eqs);
          n_give += __popc(gv);
          n_take += __popc(tk);
        }
        if (phase == 0) {
          if (lane == 0) {
            cnt[0][warp] = n_give;
            cnt[1][warp] = n_take;
          }
          __syncthreads();
          int all[2] = {0, 0};
          for (int w = 0; w < kWarps; ++w)
            for (int k = 0; k < 2; ++k) {
              if (w < warp) at[k] += cnt[k][w];
              all[k] += cnt[k][w];
            }
          if (tid == 0) {
            sh.give = all[0];
            sh.take = all[1];
          }
          sync_pair();
          for (int r = 0; r < cs; ++r) {
            const EvShare& x = *cluster.map_shared_rank(&sh, r);
            if (r < me) {
              at[0] += x.give;
              at[1] += x.take;
            }
            n_moves += x.take;
          }
        }
      }
    }
    sync_pair();  // the lists are written, and nobody reads another CTA's memory any more
    if (a.in_place && me == 0 && warp * kRowItems < n_moves) {
      if (c.d == 128)
        move_rows<128>(c, b, g, give, take, warp * kRowItems, n_moves);
      else
        move_rows<64>(c, b, g, give, take, warp * kRowItems, n_moves);
    }
  } else {
    sync_pair();  // every CTA of the pair has read the length
  }
  if (me == 0 && tid == 0) {
    if (bad) set_dev_err(a.err, KVC_DEV_ERR_PAGES);
    a.moves[pair] = n_moves;
    // the length of the sequence moves once all its heads have read it
    __threadfence();
    if (atomicAdd(&a.tickets[b], 1u) == (uint32_t)c.Hkv - 1) {
      if (!bad && n > budget) c.seq_lens[b] = budget;
      a.tickets[b] = 0u;
    }
  }
}

// CTA (span of moves, KV head, sequence), a warp per kRowItems of them.
template <int D>
__global__ void __launch_bounds__(kMvThreads) evict_move_kernel(const EvArgs a) {
  pdl_wait();
  const int g = blockIdx.y, b = blockIdx.z;
  const int64_t pair = (int64_t)b * a.c.Hkv + g;
  const int n = a.moves[pair];
  const int32_t* give = a.lists + pair * 2 * a.max_move;
  const int i0 = ((int)blockIdx.x * (kMvThreads / 32) + (threadIdx.x >> 5)) * kRowItems;
  if (i0 < n) move_rows<D>(a.c, b, g, give, give + a.max_move, i0, n);
}

int64_t evict_max_move(int64_t max_len, int64_t budget) {
  return std::max<int64_t>(0, std::min(budget, max_len - budget));
}

kvc_status check_evict(const Paged& c, int64_t max_len, int64_t budget) {
  KVC_CHECK_ARG(max_len >= 1 && max_len <= c.room(), "need 1 <= max_len <= max_pages * page_size");
  KVC_CHECK_ARG(budget >= 1 && budget < (int64_t(1) << 31), "need 1 <= budget < 2^31");
  return KVC_OK;
}

// CTAs per pair: as many as the SMs hold at once (one of 1024 threads each),
// with at least kEvSmall slots each.  32 pairs of 32768 entries cut to 2048,
// replayed from a graph, what restores the cache between the calls included
// (called eagerly 60 to 63 us with four): 72.4 us with one CTA per
// pair, 56.9 with two, 52.4 with four, 110.9 with eight (two waves).
int evict_cluster(const Paged& c, int64_t max_len) {
  const int64_t pairs = (int64_t)c.batch * c.Hkv;
  int cs = 1;
  while (cs < 8 && pairs * cs * 2 <= num_sms() && max_len >= kEvSmall * cs * 2) cs *= 2;
  return cs;
}
int64_t evict_segment(int64_t max_len, int cs) { return ((max_len + cs - 1) / cs + 31) / 32 * 32; }

// The workspace: counters first.  One per sequence is used, but what follows
// starts behind one per pair: that much is zero before and after every call on
// a paged cache, so that one workspace can serve them all.
bool carve_evict(const Paged& c, int64_t max_len, int64_t budget, WsCursor* w, EvArgs* a) {
  const size_t bg = (size_t)c.batch * c.Hkv;
  a->max_move = std::max<int64_t>(1, evict_max_move(max_len, budget));
  a->tickets = w->take<uint32_t>(bg);
  a->moves = w->take<int32_t>(bg);
  a->lists = w->take<int32_t>(bg * 2 * (size_t)a->max_move);
  a->cluster = evict_cluster(c, max_len);
  a->resident = (int64_t)bg * a->cluster <= num_sms();
  a->keys = evict_segment(max_len, a->cluster) > kEvSmemKeys ? w->take<uint32_t>(bg * (size_t)max_len) : nullptr;
  return w->ok;
}

template <int kThreads>
kvc_status launch_evict(const EvArgs& a, cudaStream_t st) {
  static ContextCache cache;
  const kvc_status s = once_per_context(cache, [] {
    KVC_CUDA_TRY(cudaFuncSetAttribute(evict_kernel<kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)kEvSmemKeys * 4));
    return KVC_OK;
  });
  if (s != KVC_OK) return s;
  const size_t smem = a.keys ? 0 : (size_t)evict_segment(a.max_len, a.cluster) * 4;
  Launch l(dim3((unsigned)(a.c.Hkv * a.cluster), (unsigned)a.c.batch), dim3(kThreads), smem, st);
  if (a.cluster > 1) l.cluster_x((unsigned)a.cluster);
  KVC_CUDA_TRY(l.run(evict_kernel<kThreads>, a));
  count_launch();
  return KVC_OK;
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
  if (total == 0 && cu_seqlens) return KVC_OK;  // no token to write
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
  const int64_t most = (idx ? std::min(kk, max_seqlen) : max_seqlen) * a.c.Hkv;
  KVC_CHECK_ARG(most < (int64_t(1) << 31), "a sequence's new entries times num_kv_heads must be below 2^31");
  // no sequence brings more than all tokens; the ticket counts the CTAs in 32 bits
  const int64_t spans = std::max<int64_t>(1, (std::min(most, total * a.c.Hkv) + kAppSpan - 1) / kAppSpan);
  KVC_CHECK_ARG(spans * a.c.batch < (int64_t(1) << 32),
                "batch times a sequence's new entries times num_kv_heads must be below 2^38");
  const Launch l(dim3((unsigned)spans, (unsigned)a.c.batch), dim3(kAppThreads), 0, (cudaStream_t)stream);
  KVC_CUDA_TRY(a.c.d == 128 ? l.run(append_kernel<128>, a) : l.run(append_kernel<64>, a));
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
  WsCursor w{nullptr, ~size_t(0)};
  EvArgs a{};
  carve_evict(p, max_len, budget, &w, &a);
  *bytes = w.off;
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
  if (!ws || !aligned(ws, kWsAlign)) return fail(KVC_ERR_WORKSPACE, "evict workspace missing or not 256-B aligned");
  WsCursor w{static_cast<char*>(ws), ws_bytes};
  if (!carve_evict(a.c, max_len, budget, &w, &a)) return fail(KVC_ERR_WORKSPACE, "evict workspace too small");
  a.max_len = max_len;
  a.budget = budget;
  a.recent = recent;
  a.in_place = a.max_move <= kEvInline;
  a.err = dev_err;
  const cudaStream_t st = (cudaStream_t)stream;
  s = max_len <= kEvSmall ? launch_evict<256>(a, st) : launch_evict<1024>(a, st);
  if (s != KVC_OK || a.in_place) return s;
  const Launch l(dim3((unsigned)((a.max_move + kMvSpan - 1) / kMvSpan), (unsigned)a.c.Hkv, (unsigned)a.c.batch),
                 dim3(kMvThreads), 0, st);
  KVC_CUDA_TRY(a.c.d == 128 ? l.run(evict_move_kernel<128>, a) : l.run(evict_move_kernel<64>, a));
  count_launch();
  return KVC_OK;
}
