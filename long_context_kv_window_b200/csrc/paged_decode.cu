// paged_decode.cu -- attention of one decode query per head over paged caches.
//
// FastKV (gist.science 2502.01068) sections 1 and 2.B: decoding is bound by
// reading the retained entries; StructKV (gist.science 2604.06746) section
// 2.A: attention accumulated per token.  With entry j of KV head g in page
// table[j / page], and query head h of the group:
//     s_j = scale * q_h . k_j,  out_h = sum_j exp(s_j - lse_h) v_j,  weights_j += sum_h exp(s_j - lse_h).
//
// A stream from HBM (4 d bytes per entry, 4 G d operations on them).  The
// entries of all (sequence, KV head) pairs form one row of 64-entry tiles,
// which is cut into equal runs, one per CTA, whatever the sequences' lengths:
// a ragged batch loads every SM alike.  A run covers pieces of one or more
// pairs; a pair that lies in one run is finished there, the others leave
// (max, sum, output) per run and the last of their CTAs joins them in run
// order (a ticket counter per pair, returned to zero).
// A piece that met a page id outside the pool or an entry that did not arrive
// has no result; nor has its pair, which adds no weights.
//
// Every warp streams its own 16 entries of each tile (one page holds them)
// through a ring of its own -- TMA boxes, 128-byte swizzle, requested by the
// warp itself -- and shares nothing with the other warps until a pair ends,
// so no barrier joins them in the loop.  Both contractions are mma.sync: the
// logits S[head][entry] (M = 16 heads, the group's and zero rows) come out in
// the layout in which the second one takes P, so P stays in registers, which
// the tcgen05 form cannot do; at 4 d bytes per entry the legacy tensor rate is
// many times what the stream needs.  P enters as three bf16 terms, its 24 bits
// (two, good to 2^-17, left the output 2.3e-6 off, three 5e-7, for 1 to
// 6 % of the time); up to 8 heads per group the first two ride in one MMA, in rows 0..7
// and 8..15.  Row maxima are references that move only when a logit
// passes them by more than 8 log2 units (a warp vote; p <= 2^8 otherwise).
//
// Measured: 1 x 131072 entries, 40/8 heads, d = 128: 90.9 us, 5.9 TB/s (91 % of
// the measured copy bandwidth; of the time 3.6 us are the first tiles' queue and
// about 4 the joins); 524288 entries 6.8 TB/s; 8 x 13107 entries with weights
// 88 us (10 of them the weights).  DRAM bounds it.
//
// With `accumulate` the logits go to the workspace (4 G bytes per entry, which
// stay in L2 for most sizes) and a second kernel adds exp(s - lse) to the
// weights once the log-sum-exp is known.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include <cuda_bf16.h>

#include "paged.cuh"
#include "tc.cuh"

namespace kvc {
namespace {

constexpr int kPdWarps = 4;
constexpr int kPdThreads = 32 * kPdWarps;
constexpr int kPdUnit = 16;                  // entries a warp takes at a time
constexpr int kPdTile = kPdUnit * kPdWarps;  // entries of a tile
constexpr int kPdMaxG = 16;
constexpr int kPdCtasPerSm = 2;
constexpr int kPdMaxBatch = 1024;
// What a pair costs beside its tiles, in tiles: reading q, joining the warps,
// writing the result.  A ragged batch of 64 (1..8192 entries, 32/8 heads, half
// of them within one tile, weights included) takes 104.5 us with 0, 76.4 with
// 1, 60.4 with 2, 57.6 with 4, 61.1 with 6; equal lengths do not care.
constexpr int kPdPairCost = 4;
constexpr float kPdSlack = 8.f;
constexpr double kLog2e = 1.4426950408889634;
constexpr double kLn2 = 0.6931471805599453;

struct PdArgs {
  Paged c;
  const uint16_t* q;
  int64_t q_sb, q_sh;
  int H, G;
  float c2;  // scale * log2(e)
  int64_t max_len, ld;  // ld: max_len rounded up to whole units
  float* out;     // [B][H][d]
  float* lse;     // [B][H] or nullptr
  float* z;       // [B][H]: log-sum-exp in log2 units, +inf (which none is): no result (accumulate; else nullptr)
  float* logits;  // [B][H][ld], log2 units (accumulate)
  uint32_t* tickets;  // [B*Hkv]: runs of the pair done
  float* part_ml;     // [2 * runs][G][2]: max, sum (sum -1: the piece has no result)
  float* part_o;      // [2 * runs][G][d]
  int32_t* err;
};

// D: head_dim; G16: more than 8 heads per group.
template <int D, bool G16>
struct PdSmem {
  static constexpr int kRows = G16 ? 16 : 8;
  static constexpr int kBox = kPdUnit * 128;            // 16 entries x 64 columns (2 KB)
  static constexpr int kMat = (D / 64) * kBox;          // 16 entries of k or v
  static constexpr int kStage = 2 * kMat;
  // Two stages keep 128 KB per SM on their way (d = 128), which streams as
  // fast as 192 KB and queues less: with three the first tile took 4.9 us
  // instead of 3.6, the slowest CTA ended 12 us after the median instead of 3
  // (128K entries, 40/8 heads: 99.0 us with three, 93.8 with two).
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kRing = kPdWarps * kStages * kStage;
  static constexpr int kRow = D + 4;                           // floats per row: output, max, sum
  static constexpr int kMerge = kPdWarps * kRows * kRow * 4;  // every warp's rows
  static constexpr size_t kBytes = 1024 + (size_t)kRing + kMerge + (kPdMaxBatch + 1) * 4 + 512;
  static_assert(kPdCtasPerSm * (kBytes + 1024) <= 233472, "CTAs per SM");
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(tc::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// (x, y) as bf16 pairs hi + lo + lo2: the 24 bits of a float, 8 each
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t& hi, uint32_t& lo, uint32_t& lo2) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  const float2 f = __bfloat1622float2(h);
  x -= f.x;
  y -= f.y;
  const __nv_bfloat162 l = __floats2bfloat162_rn(x, y);
  const float2 e = __bfloat1622float2(l);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
  lo2 = pack_bf16(x - e.x, y - e.y);
}

// Tiles of a sequence of n entries, per KV head.
__device__ __forceinline__ int pd_tiles(int n, int64_t max_len) {
  return n > 0 && n <= max_len ? (n + kPdTile - 1) / kPdTile : 0;
}
// The runs: a pair of nu tiles is kPdPairCost + nu places of one row (what it
// costs to begin and end a pair, then its tiles); run i holds the places
// [total * i / runs, total * (i + 1) / runs).
struct Runs {
  int64_t total;
  int runs;
  __device__ __forceinline__ int64_t start(int i) const { return total * i / runs; }
  // the run that holds place x
  __device__ __forceinline__ int of(int64_t x) const { return (int)(((x + 1) * runs + total - 1) / total) - 1; }
};

// A pair's places inside a run.
struct Piece {
  int b, g;
  int len, nu;   // entries and tiles of the pair
  int t0, t1;    // tiles of the piece (none if t1 <= t0)
  int64_t pair;  // the pair's first tile, as a place
  int64_t next;  // the place behind the piece
};

template <int D, bool G16>
__global__ void __launch_bounds__(kPdThreads, kPdCtasPerSm)
paged_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const PdArgs a) {
  using L = PdSmem<D, G16>;
  constexpr int kRows = L::kRows, kKS = D / 16, kNT = D / 8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* merge = reinterpret_cast<float*>(sm + L::kRing);                       // [warps][kRows][kRow]
  int* first = reinterpret_cast<int*>(sm + L::kRing + L::kMerge);              // [B + 1]: places before sequence b (per head)
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kRing + L::kMerge + (kPdMaxBatch + 2) / 2 * 8);  // [warps][stages]
  int* flags = reinterpret_cast<int*>(full + kPdWarps * L::kStages);           // abort, last, warp totals, warps' bad flags
  volatile int* abort_flag = flags;
  const Paged& c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.G, B = c.batch, Hkv = c.Hkv;

  if (tid == 0) {
    for (int i = 0; i < kPdWarps * L::kStages; ++i) tc::mbar_init(&full[i], 1);
    flags[0] = 0;
    tc::fence_mbar_init();
    tc::prefetch_tmap(&kmap);
    tc::prefetch_tmap(&vmap);
  }
  pdl_wait();  // the cache and q may come from the previous kernels of the stream
  pdl_trigger();  // this grid is resident at once: the next kernel may be brought in as its CTAs leave
  // ---- places before each sequence
  {
    const int per = (B + kPdThreads - 1) / kPdThreads, b0 = tid * per;
    int mine = 0;
    for (int u = 0; u < per; ++u) {
      const int b = b0 + u;
      if (b >= B) break;
      const int nu = pd_tiles(c.seq_lens[b], a.max_len);
      mine += nu > 0 ? nu + kPdPairCost : 0;
    }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) flags[2 + warp] = inc;
    __syncthreads();
    int at = inc - mine;
    for (int w = 0; w < warp; ++w) at += flags[2 + w];
    for (int u = 0; u < per; ++u) {
      const int b = b0 + u;
      if (b >= B) break;
      first[b] = at;
      const int nu = pd_tiles(c.seq_lens[b], a.max_len);
      at += nu > 0 ? nu + kPdPairCost : 0;
      if (b == B - 1) first[B] = at;
    }
    __syncthreads();
  }
  // ---- sequences without entries (or with a length that cannot be), dealt out over the CTAs
  for (int b = blockIdx.x; b < B; b += gridDim.x) {
    if (first[b + 1] != first[b]) continue;
    if (tid == 0 && c.seq_lens[b] != 0) set_dev_err(a.err, KVC_DEV_ERR_PAGES);
    for (int i = tid; i < a.H * D; i += kPdThreads) a.out[(int64_t)b * a.H * D + i] = 0.f;
    for (int h = tid; h < a.H; h += kPdThreads) {
      if (a.lse) a.lse[(int64_t)b * a.H + h] = -INFINITY;
      if (a.z) a.z[(int64_t)b * a.H + h] = -INFINITY;
    }
  }
  Runs rs;
  rs.total = (int64_t)first[B] * Hkv;
  rs.runs = (int)std::min<int64_t>(gridDim.x, rs.total);
  const int run = blockIdx.x;
  if (run >= rs.runs) return;
  const int64_t x0 = rs.start(run), x1 = rs.start(run + 1);

  // the piece of the run [x0, x1) that starts at place x
  auto piece_at = [&](int64_t x) {
    Piece p;
    int lo = 0, hi = B - 1;  // the last sequence whose places begin at or before x
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)first[mid] * Hkv <= x) lo = mid; else hi = mid - 1;
    }
    const int places = first[lo + 1] - first[lo];
    const int64_t r = x - (int64_t)first[lo] * Hkv;
    const int at = (int)(r % places);
    p.b = lo;
    p.g = (int)(r / places);
    p.nu = places - kPdPairCost;
    p.pair = x - at + kPdPairCost;
    p.next = std::min<int64_t>(x1, x - at + places);
    p.t0 = max(0, at - kPdPairCost);
    p.t1 = (int)(p.next - p.pair);
    p.len = c.seq_lens[lo];
    return p;
  };

  // ---- producer state of this warp: the next unit to request
  uint8_t* ring = sm + (size_t)warp * L::kStages * L::kStage;
  const uint32_t ring_u32 = tc::smem_u32(ring);
  uint64_t* bar = full + warp * L::kStages;
  Piece pp = piece_at(x0);
  int pt = pp.t0;        // next tile of the piece
  int page_base = -32;   // tile of lane 0's page id
  int page_id = 0;
  unsigned issued = 0;   // units requested
  uint32_t bad_units = 0;  // bit s: the unit in stage s had a page id outside the pool
  auto request = [&]() {  // requests this warp's next unit, if the run has one; warp-uniform
    for (;;) {
      if (pt >= pp.t1) {
        if (pp.next >= x1) return;
        pp = piece_at(pp.next);
        pt = pp.t0;
        page_base = -32;
      }
      if (pt * kPdTile + warp * kPdUnit < pp.len) break;
      ++pt;  // the last tile of a pair: no entry for this warp
    }
    if (pt >= page_base + 32 || page_base < 0) {  // page ids of the next 32 tiles
      page_base = pt;
      const int64_t s = (int64_t)(pt + lane) * kPdTile + warp * kPdUnit;
      page_id = pt + lane < pp.t1 && s < pp.len ? c.page_of(pp.b, s) : 0;
    }
    const int p = __shfl_sync(0xffffffffu, page_id, pt - page_base);
    const int s = (int)(issued % L::kStages);
    bad_units = p < 0 ? bad_units | 1u << s : bad_units & ~(1u << s);
    if (lane == 0) {
      tc::mbar_arrive_expect_tx(&bar[s], (uint32_t)L::kStage);
      const int slot = (pt * kPdTile + warp * kPdUnit) & (c.page - 1), at = p < 0 ? c.num_pages : p;  // past the pool: zeros
      const uint32_t dst = ring_u32 + (uint32_t)(s * L::kStage);
#pragma unroll
      for (int cb = 0; cb < D / 64; ++cb) {
        tma_load_4d(dst + cb * L::kBox, &kmap, &bar[s], cb * 64, slot, pp.g, at);
        tma_load_4d(dst + L::kMat + cb * L::kBox, &vmap, &bar[s], cb * 64, slot, pp.g, at);
      }
    }
    ++issued;
    ++pt;
  };
  for (int i = 0; i < L::kStages; ++i) request();

  // ---- the run, piece by piece
  const int row = lane >> 2, col = 2 * (lane & 3);  // accumulator rows row, row + 8 and columns col, col + 1
  // ldmatrix rows: K 8 entries x 4 pieces of 8 columns; V two blocks of 8 entries x two of 8 columns
  const int k_row = lane & 7, k_piece = lane >> 3;
  const int v_row = lane & 15, v_piece = lane >> 4;
  unsigned taken = 0;
  bool lost = false;  // a wait of this warp gave up: from then on its stages are not the units it is at
  for (int64_t x = x0; x < x1;) {
    const Piece p = piece_at(x);
    x = p.next;
    if (p.t1 <= p.t0) continue;  // the cost of a pair whose tiles are the next run's
    const int64_t qb = (int64_t)p.b * a.q_sb + (int64_t)p.g * G * a.q_sh;
    uint32_t qa[kKS][2], qc[G16 ? kKS : 1][2];  // Q rows row (and row + 8) as MMA A operand
#pragma unroll
    for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = ks * 16 + 8 * u + col;
        qa[ks][u] = row < G ? *reinterpret_cast<const uint32_t*>(a.q + qb + (int64_t)row * a.q_sh + k) : 0u;
        if constexpr (G16)
          qc[ks][u] = row + 8 < G ? *reinterpret_cast<const uint32_t*>(a.q + qb + (int64_t)(row + 8) * a.q_sh + k) : 0u;
      }
    float o[kNT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    int marks = 0;  // why the piece has no result; 1: a page id outside the pool, 2: a unit that did not land
    for (int t = p.t0; t < p.t1; ++t) {
      const int s0 = t * kPdTile + warp * kPdUnit;  // first entry of the unit
      if (s0 >= p.len) break;
      const int st = (int)(taken % L::kStages);
      // the warp goes on or gives up as one
      lost = lost || !__all_sync(0xffffffffu, tc::mbar_wait(&bar[st], (taken / L::kStages) & 1, abort_flag));
      if (lost) {
        marks |= 2;
        break;
      }
      const uint32_t kt = ring_u32 + (uint32_t)(st * L::kStage), vt = kt + L::kMat;
      marks |= (bad_units >> st) & 1;
      const int left = p.len - s0;  // valid entries of the unit, if below 16
      if (left < kPdUnit) {  // what lies behind the entries must not meet p = 0 as infinity or NaN
        for (int i = lane; i < (kPdUnit - left) * (D / 8); i += 32) {
          const int r = left + i / (D / 8), pc = i % (D / 8);
          *reinterpret_cast<uint4*>(ring + st * L::kStage + L::kMat + (pc >> 3) * L::kBox + r * 128 + (pc & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        tc::fence_proxy_async_smem();  // before the stage's next copy
        __syncwarp();
      }
      // logits of 16 entries: two 8-entry column blocks
      float sc[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
#pragma unroll
        for (int k4 = 0; k4 < D / 32; ++k4) {
          const int r = 8 * n + k_row, pc = 4 * k4 + k_piece;  // 16-byte piece of the row
          uint32_t b[4];
          ldsm4(b, kt + (uint32_t)((pc >> 3) * L::kBox + r * 128 + (((pc & 7) ^ (r & 7)) << 4)));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int ks = 2 * k4 + u;
            if constexpr (G16)
              mma_16816(sc[n], qa[ks][0], qc[ks][0], qa[ks][1], qc[ks][1], b[2 * u], b[2 * u + 1]);
            else
              mma_16816(sc[n], qa[ks][0], 0u, qa[ks][1], 0u, b[2 * u], b[2 * u + 1]);
          }
        }
      }
      constexpr int kHalf = G16 ? 2 : 1;  // accumulator row halves in use
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2 * kHalf; ++e) {
          const bool valid = 8 * n + col + (e & 1) < left;
          sc[n][e] = valid ? sc[n][e] : -INFINITY;
          mx[e >> 1] = fmaxf(mx[e >> 1], sc[n][e]);
        }
      mx[0] *= a.c2;
      mx[1] *= a.c2;
      if (a.logits) {
#pragma unroll
        for (int hf = 0; hf < kHalf; ++hf)
          if (row + 8 * hf < G) {
            float* dst = a.logits + ((int64_t)p.b * a.H + p.g * G + row + 8 * hf) * a.ld + s0 + col;
            *reinterpret_cast<float2*>(dst) = make_float2(sc[0][2 * hf] * a.c2, sc[0][2 * hf + 1] * a.c2);
            *reinterpret_cast<float2*>(dst + 8) = make_float2(sc[1][2 * hf] * a.c2, sc[1][2 * hf + 1] * a.c2);
          }
      }
      bool move = mx[0] > m[0] + kPdSlack || (m[0] == -INFINITY && mx[0] > -INFINITY);
      if constexpr (G16) move |= mx[1] > m[1] + kPdSlack || (m[1] == -INFINITY && mx[1] > -INFINITY);
      if (__any_sync(0xffffffffu, move)) {
        float al[2] = {1.f, 1.f};
#pragma unroll
        for (int hf = 0; hf < kHalf; ++hf) {
          float v = mx[hf];
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
          if (v > m[hf]) {
            al[hf] = m[hf] == -INFINITY ? 0.f : tc::ex2_approx(m[hf] - v);
            m[hf] = v;
          }
          l[hf] *= al[hf];
        }
        if constexpr (!G16) al[1] = al[0];  // rows 8..15 hold the second terms of the same heads
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][e] *= al[e >> 1];
      }
      uint32_t hi[2][2], lo[2][2], lo2[2][2];  // [column block][row half]
#pragma unroll
      for (int hf = 0; hf < kHalf; ++hf) {
        const float ref = m[hf] == -INFINITY ? 0.f : m[hf];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = tc::ex2_approx(fmaf(sc[n][2 * hf], a.c2, -ref));
          const float p1 = tc::ex2_approx(fmaf(sc[n][2 * hf + 1], a.c2, -ref));
          l[hf] += p0 + p1;
          split_bf16(p0, p1, hi[n][hf], lo[n][hf], lo2[n][hf]);
        }
      }
#pragma unroll
      for (int d16 = 0; d16 < D / 16; ++d16) {
        const int pc = 2 * d16 + v_piece;
        uint32_t b[4];
        ldsm4_t(b, vt + (uint32_t)((pc >> 3) * L::kBox + v_row * 128 + (((pc & 7) ^ (v_row & 7)) << 4)));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // a product of its own, added with rounding: the tensor core's
          // accumulation truncates, which over thousands of units would show
          float y[4] = {0.f, 0.f, 0.f, 0.f};
          if constexpr (G16) {
            mma_16816(y, hi[0][0], hi[0][1], hi[1][0], hi[1][1], b[2 * u], b[2 * u + 1]);
            mma_16816(y, lo[0][0], lo[0][1], lo[1][0], lo[1][1], b[2 * u], b[2 * u + 1]);
            mma_16816(y, lo2[0][0], lo2[0][1], lo2[1][0], lo2[1][1], b[2 * u], b[2 * u + 1]);
          } else {
            mma_16816(y, hi[0][0], lo[0][0], hi[1][0], lo[1][0], b[2 * u], b[2 * u + 1]);
            mma_16816(y, lo2[0][0], 0u, lo2[1][0], 0u, b[2 * u], b[2 * u + 1]);
          }
          float(&on)[4] = o[2 * d16 + u];
          const float2 s01 = tc::add2(make_float2(on[0], on[1]), make_float2(y[0], y[1]));
          const float2 s23 = tc::add2(make_float2(on[2], on[3]), make_float2(y[2], y[3]));
          on[0] = s01.x;
          on[1] = s01.y;
          on[2] = s23.x;
          on[3] = s23.y;
        }
      }
      __syncwarp();  // every lane has read the stage
      ++taken;
      request();
    }
    // ---- join the four warps (the lanes of a quad hold the columns of a row)
    if constexpr (!G16) {
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        o[n][0] += o[n][2];
        o[n][1] += o[n][3];
      }
    }
    constexpr int kHalf = G16 ? 2 : 1;
    __syncthreads();  // the rows of the piece before are read
#pragma unroll
    for (int hf = 0; hf < kHalf; ++hf) {
      l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 1);
      l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 2);
      float* r = merge + (warp * kRows + row + 8 * hf) * L::kRow;
#pragma unroll
      for (int n = 0; n < kNT; ++n) *reinterpret_cast<float2*>(r + 8 * n + col) = make_float2(o[n][2 * hf], o[n][2 * hf + 1]);
      if ((lane & 3) == 0) {
        r[D] = m[hf];
        r[D + 1] = l[hf];
      }
    }
    if (lane == 0) flags[6 + warp] = marks;
    __syncthreads();
    const bool whole = p.t0 == 0 && p.t1 == p.nu;
    const int64_t h0 = (int64_t)p.b * a.H + p.g * G;  // first head of the pair
    // The four rows of a head as one: its result, or (slot >= 0) a piece's
    // (max, sum, output).  A thread per four columns.
    auto combine = [&](int64_t slot, bool none) {
      bool odd = false;
      for (int i = tid; i < G * (D / 4); i += kPdThreads) {
        const int h = i / (D / 4), c4 = i % (D / 4);
        const float* r0 = merge + h * L::kRow;
        float mw[kPdWarps], M = -INFINITY, Ls = 0.f;
#pragma unroll
        for (int w = 0; w < kPdWarps; ++w) {
          mw[w] = r0[w * kRows * L::kRow + D];
          M = fmaxf(M, mw[w]);
        }
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kPdWarps; ++w) {
          const float* r = r0 + w * kRows * L::kRow;
          const float f = mw[w] == -INFINITY ? 0.f : tc::ex2_approx(mw[w] - M);
          const float4 x = *reinterpret_cast<const float4*>(r + 4 * c4);
          Ls += f * r[D + 1];
          y.x += f * x.x;
          y.y += f * x.y;
          y.z += f * x.z;
          y.w += f * x.w;
        }
        if (slot >= 0) {
          *reinterpret_cast<float4*>(a.part_o + (slot * G + h) * D + 4 * c4) = y;
          if (c4 == 0) *reinterpret_cast<float2*>(a.part_ml + (slot * G + h) * 2) = make_float2(M, none ? -1.f : Ls);
          continue;
        }
        const float inv = 1.f / Ls;
        *reinterpret_cast<float4*>(a.out + (h0 + h) * D + 4 * c4) =
            none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
        const float any = (y.x + y.y) + (y.z + y.w);
        odd |= !none && Ls > 0.f && Ls < INFINITY && !(any - any == 0.f);
        if (c4 == 0) {
          const float z = none ? -INFINITY : M + log2f(Ls);
          if (a.lse) a.lse[h0 + h] = (float)((double)z * kLn2);
          if (a.z) a.z[h0 + h] = none ? INFINITY : z;
        }
      }
      if (slot >= 0 || !__syncthreads_or(odd)) return;
      // Sound probabilities and an output that is not finite: entries hold
      // infinities or NaN in v, and a bf16 term of p that is 0 makes NaN of an
      // infinity.  The columns that hold them get what sum_j p_j v_j is.
      int* kinds = reinterpret_cast<int*>(merge);  // per column, 1: +inf, 2: -inf, 4: NaN among the entries
      for (int i = tid; i < D; i += kPdThreads) kinds[i] = 0;
      __syncthreads();
      for (int j = tid; j < p.len; j += kPdThreads) {
        const uint16_t* vr = c.v + c.row(c.page_of(p.b, j), p.g, j);
        for (int e = 0; e < D; ++e) {
          const uint32_t v = vr[e];
          if ((v & 0x7F80u) == 0x7F80u) atomicOr(&kinds[e], (v & 0x7Fu) ? 4 : (v & 0x8000u) ? 2 : 1);
        }
      }
      __syncthreads();
      for (int i = tid; i < G * D; i += kPdThreads) {
        const int kind = kinds[i % D];
        if (kind) a.out[h0 * D + i] = kind == 1 ? INFINITY : kind == 2 ? -INFINITY : __int_as_float(0x7FFFFFFF);
      }
      __syncthreads();
    };
    marks = flags[6] | flags[7] | flags[8] | flags[9];
    if ((marks & 1) && tid == 0) set_dev_err(a.err, KVC_DEV_ERR_PAGES);
    combine(whole ? -1 : 2 * run + (p.t0 == 0 ? 1 : 0), marks != 0);
    if (whole) continue;
    // ---- the last run of the pair joins the pieces
    const int c0 = rs.of(p.pair), c1 = rs.of(p.pair + p.nu - 1);
    __syncthreads();
    uint32_t* ticket = a.tickets + (int64_t)p.b * Hkv + p.g;
    if (tid == 0) {
      __threadfence();
      const bool last = atomicAdd(ticket, 1u) == (uint32_t)(c1 - c0);
      if (last) *ticket = 0u;
      flags[1] = last;
    }
    __syncthreads();
    if (!flags[1]) continue;
    __threadfence();
    // Piece i is slot 1 of run c0 or slot 0 of run c0 + i.  The warps share out
    // the pieces, kIn of them requested at once and a head's while the head
    // before is worked off; every warp's (max, sum, output) of a head then
    // goes into the rows in shared memory.
    const int np = c1 - c0 + 1;
    constexpr int kIn = 5, kDL = D / 32;
    using Vec = typename std::conditional<D == 128, float4, float2>::type;
    bool none = false;
    float2 ml[2][kIn];
    Vec y[2][kIn];
    auto fetch = [&](float2(&mlb)[kIn], Vec(&yb)[kIn], int h, int i0) {
#pragma unroll
      for (int j = 0; j < kIn; ++j) {
        const int i = i0 + warp + kPdWarps * j;
        mlb[j] = make_float2(-INFINITY, 0.f);
        yb[j] = Vec{};
        if (i < np) {
          const int64_t at = (int64_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * G + h;
          mlb[j] = __ldcg(reinterpret_cast<const float2*>(a.part_ml + at * 2));
          yb[j] = __ldcg(reinterpret_cast<const Vec*>(a.part_o + at * D) + lane);
        }
      }
    };
    const int batches = (np + kPdWarps * kIn - 1) / (kPdWarps * kIn), steps = G * batches;
    float M = -INFINITY, Ls = 0.f, acc[kDL];
    auto step = [&](float2(&mlb)[kIn], Vec(&yb)[kIn], int st) {
      if (st % batches == 0) {
        M = -INFINITY;
        Ls = 0.f;
#pragma unroll
        for (int e = 0; e < kDL; ++e) acc[e] = 0.f;
      }
      float mx = M;
#pragma unroll
      for (int j = 0; j < kIn; ++j) mx = fmaxf(mx, mlb[j].x);
      const float f0 = M == -INFINITY ? 0.f : tc::ex2_approx(M - mx);
      M = mx;
      Ls *= f0;
#pragma unroll
      for (int e = 0; e < kDL; ++e) acc[e] *= f0;
#pragma unroll
      for (int j = 0; j < kIn; ++j) {
        const float f = mlb[j].x == -INFINITY ? 0.f : tc::ex2_approx(mlb[j].x - M);
        none |= mlb[j].y == -1.f;
        Ls += f * mlb[j].y;
        const float* v = reinterpret_cast<const float*>(&yb[j]);
#pragma unroll
        for (int e = 0; e < kDL; ++e) acc[e] += f * v[e];
      }
      if (st % batches == batches - 1) {
        float* r = merge + (warp * kRows + st / batches) * L::kRow;
        Vec out{};
#pragma unroll
        for (int e = 0; e < kDL; ++e) reinterpret_cast<float*>(&out)[e] = acc[e];
        *reinterpret_cast<Vec*>(r + lane * kDL) = out;
        if (lane == 0) {
          r[D] = M;
          r[D + 1] = Ls;
        }
      }
    };
    fetch(ml[0], y[0], 0, 0);
    for (int st = 0; st < steps; st += 2) {
      if (st + 1 < steps) fetch(ml[1], y[1], (st + 1) / batches, (st + 1) % batches * kPdWarps * kIn);
      step(ml[0], y[0], st);
      if (st + 2 < steps) fetch(ml[0], y[0], (st + 2) / batches, (st + 2) % batches * kPdWarps * kIn);
      if (st + 1 < steps) step(ml[1], y[1], st + 1);
    }
    if (lane == 0) flags[6 + warp] = none;
    __syncthreads();
    combine(-1, flags[6] | flags[7] | flags[8] | flags[9]);
  }
  if (*abort_flag) {  // a copy never landed: nothing of the stages may be in flight when the CTA leaves
    for (unsigned i = issued > (unsigned)L::kStages ? issued - L::kStages : 0; i < issued; ++i)
      if (lane == 0) tc::mbar_drain(&bar[i % L::kStages], (i / L::kStages) & 1);
    if (lane == 0) set_dev_err(a.err, KVC_DEV_ERR_TIMEOUT);
  }
}

// weights[j] += sum_h 2^(s_hj - z_h), heads in order: a thread per four
// entries, 1024 entries of a pair at a time; the CTAs go over the 1024s of all
// pairs in turn, so short sequences of a ragged batch leave none idle.  What
// comes before pdl_wait reads only what the decode kernel read too.
constexpr int kWtThreads = 256;
constexpr int kWtSpan = 4 * kWtThreads;
constexpr int kWtCtasPerSm = 6;
__global__ void __launch_bounds__(kWtThreads, kWtCtasPerSm) paged_weights_kernel(const PdArgs a) {
  __shared__ int spans[kPdMaxBatch + 1];  // [b]: spans of the sequences before b (per head)
  __shared__ int warp_sum[kWtThreads / 32];
  const Paged& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = c.batch;
  const int per = (B + kWtThreads - 1) / kWtThreads;
  auto of = [&](int b) {
    const int n = c.seq_lens[b];
    return n > 0 && n <= a.max_len ? (n + kWtSpan - 1) / kWtSpan : 0;
  };
  int mine = 0;
  for (int u = 0; u < per; ++u)
    if (tid * per + u < B) mine += of(tid * per + u);
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int at = inc - mine;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
  for (int u = 0; u < per; ++u) {
    const int b = tid * per + u;
    if (b >= B) break;
    spans[b] = at;
    at += of(b);
    if (b == B - 1) spans[B] = at;
  }
  __syncthreads();
  pdl_wait();
  const int64_t total = (int64_t)spans[B] * c.Hkv;
  for (int64_t x = blockIdx.x; x < total; x += gridDim.x) {
    int lo = 0, hi = B - 1;  // the last sequence whose spans begin at or before x
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)spans[mid] * c.Hkv <= x) lo = mid; else hi = mid - 1;
    }
    const int b = lo, mine_n = spans[b + 1] - spans[b];
    const int r = (int)(x - (int64_t)spans[b] * c.Hkv), g = r / mine_n;
    const int n = c.seq_lens[b];
    const int64_t s = (int64_t)(r % mine_n) * kWtSpan + 4 * tid;
    if (s >= n) continue;
    const int64_t h0 = (int64_t)b * a.H + (int64_t)g * a.G;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    bool read = true;
#pragma unroll 4
    for (int h = 0; h < a.G; ++h) {
      const float z = a.z[h0 + h];
      const float4 y = *reinterpret_cast<const float4*>(a.logits + (h0 + h) * a.ld + s);
      read &= z != INFINITY;  // otherwise the pair's entries could not be read, or not all of them
      w[0] += tc::ex2_approx(y.x - z);
      w[1] += tc::ex2_approx(y.y - z);
      w[2] += tc::ex2_approx(y.z - z);
      w[3] += tc::ex2_approx(y.w - z);
    }
    if (!read) continue;
    float* dst = c.weights + c.entry(c.page_of(b, s), g, s);
    if (s + 4 <= n) {
      float4 old = *reinterpret_cast<float4*>(dst);
      *reinterpret_cast<float4*>(dst) = make_float4(old.x + w[0], old.y + w[1], old.z + w[2], old.w + w[3]);
    } else {
      for (int e = 0; e < 4; ++e)
        if (s + e < n) dst[e] += w[e];
    }
  }
}

kvc_status check_paged_decode(const Paged& c, int32_t H, int64_t max_len) {
  KVC_CHECK_ARG(H >= 1 && H % c.Hkv == 0, "num_heads must be a positive multiple of num_kv_heads");
  if (H / c.Hkv > kPdMaxG) return fail(KVC_ERR_UNSUPPORTED, "at most 16 query heads per KV head");
  KVC_CHECK_ARG(max_len >= 1 && max_len <= c.room(), "need 1 <= max_len <= max_pages * page_size");
  // the kernels count the places of all sequences, and the spans of all pairs, in 32 bits
  KVC_CHECK_ARG((int64_t)c.batch * ((max_len + kPdTile - 1) / kPdTile + kPdPairCost) < (int64_t(1) << 31) &&
                    (int64_t)c.batch * c.Hkv * ((max_len + kWtSpan - 1) / kWtSpan) < (int64_t(1) << 31),
                "batch * max_len must be below 2^36, and batch * num_kv_heads * max_len below 2^40");
  return KVC_OK;
}

int64_t round_unit(int64_t n) { return (n + kPdUnit - 1) / kPdUnit * kPdUnit; }

// CTAs of a call: two per SM, never more than there can be tiles.
int paged_runs(const Paged& c, int64_t max_len) {
  const int64_t tiles = (int64_t)c.batch * c.Hkv * ((max_len + kPdTile - 1) / kPdTile);
  return (int)std::min<int64_t>((int64_t)kPdCtasPerSm * num_sms(), tiles);
}

// The workspace: counters first (their place depends on the cache alone).
bool carve(const Paged& c, int H, int64_t max_len, bool accumulate, WsCursor* w, PdArgs* a) {
  const size_t slots = 2 * (size_t)kPdCtasPerSm * num_sms() * (H / c.Hkv);
  a->tickets = w->take<uint32_t>((size_t)c.batch * c.Hkv);
  a->part_ml = w->take<float>(slots * 2);
  a->part_o = w->take<float>(slots * c.d);
  if (accumulate) {
    a->z = w->take<float>((size_t)c.batch * H);
    a->logits = w->take<float>((size_t)c.batch * H * (size_t)round_unit(max_len));
  }
  return w->ok;
}

template <int D, bool G16>
kvc_status launch_paged_decode(int runs, cudaStream_t st, const CUtensorMap (&maps)[2], const PdArgs& a) {
  static ContextCache cache;
  const kvc_status s = once_per_context(cache, [] {
    KVC_CUDA_TRY(cudaFuncSetAttribute(paged_decode_kernel<D, G16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)PdSmem<D, G16>::kBytes));
    return KVC_OK;
  });
  if (s != KVC_OK) return s;
  const Launch l(dim3((unsigned)runs), dim3(kPdThreads), PdSmem<D, G16>::kBytes, st);
  KVC_CUDA_TRY(l.run(paged_decode_kernel<D, G16>, maps[0], maps[1], a));
  count_launch();
  return KVC_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" kvc_status kvc_paged_decode_workspace_size(const kvc_paged_cache* c, int32_t num_heads, int64_t max_len,
                                                      int32_t accumulate, size_t* bytes) {
  clear_error();
  PdArgs a{};
  kvc_status s = check_paged(c, &a.c);
  if (s == KVC_OK) s = check_paged_decode(a.c, num_heads, max_len);
  if (s != KVC_OK) return s;
  KVC_CHECK_ARG(bytes != nullptr, "bytes must be non-NULL");
  WsCursor w{nullptr, ~size_t(0)};
  carve(a.c, num_heads, max_len, accumulate != 0, &w, &a);
  *bytes = w.off;
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
  KVC_CHECK_ARG(!accumulate || (a.c.weights && aligned(a.c.weights, 16)),
                "accumulating needs the cache's weights, 16-byte aligned");
  if (!ws || !aligned(ws, kWsAlign)) return fail(KVC_ERR_WORKSPACE, "paged decode workspace missing or not 256-B aligned");
  WsCursor w{static_cast<char*>(ws), ws_bytes};
  if (!carve(a.c, num_heads, max_len, accumulate != 0, &w, &a))
    return fail(KVC_ERR_WORKSPACE, "paged decode workspace too small");
  if (!encode_fn()) return fail(KVC_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  a.q = q;
  a.q_sb = q_stride_b;
  a.q_sh = q_stride_h;
  a.H = num_heads;
  a.G = num_heads / a.c.Hkv;
  a.c2 = (float)((double)scale * kLog2e);
  a.max_len = max_len;
  a.ld = round_unit(max_len);
  a.out = out;
  a.lse = lse;
  a.err = dev_err;
  // 4-D maps [page][KV head][slot][d], boxes of 64 columns x 16 slots
  CUtensorMap maps[2];
  const uint16_t* srcs[2] = {a.c.k, a.c.v};
  const int d = a.c.d;
  for (int i = 0; i < 2; ++i) {
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)a.c.page, (cuuint64_t)a.c.Hkv, (cuuint64_t)a.c.num_pages};
    cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)a.c.page * d * 2, (cuuint64_t)a.c.page_stride * 2};
    cuuint32_t box[4] = {64u, (cuuint32_t)kPdUnit, 1u, 1u};
    cuuint32_t es[4] = {1u, 1u, 1u, 1u};
    if (encode_fn()(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(srcs[i]), dims, strides, box,
                    es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return fail(KVC_ERR_CUDA, "cuTensorMapEncodeTiled failed for the pages");
  }
  const int runs = paged_runs(a.c, max_len);
  const cudaStream_t st = (cudaStream_t)stream;
  if (d == 128)
    s = a.G > 8 ? launch_paged_decode<128, true>(runs, st, maps, a) : launch_paged_decode<128, false>(runs, st, maps, a);
  else
    s = a.G > 8 ? launch_paged_decode<64, true>(runs, st, maps, a) : launch_paged_decode<64, false>(runs, st, maps, a);
  if (s != KVC_OK || !accumulate) return s;
  const int64_t spans = (int64_t)a.c.batch * a.c.Hkv * ((max_len + kWtSpan - 1) / kWtSpan);
  const Launch l(dim3((unsigned)std::min<int64_t>(spans, (int64_t)kWtCtasPerSm * num_sms())), dim3(kWtThreads), 0, st);
  KVC_CUDA_TRY(l.run(paged_weights_kernel, a));
  count_launch();
  return KVC_OK;
}
