// prefill_varlen.cu -- causal attention of packed sequences with every row's
// log-sum-exp, on tcgen05 with the probabilities kept in TMEM.
//
// FastKV (gist.science 2502.01068) section 1 (full attention over the prompt
// at prefill) and 2.A (the window rows' normalisers); FastKV abstract:
// grouped-query heads.  Query i of a sequence sees the keys j <= i + lk - lq.
//
// The rows of an MMA tile are (token, head of the group) pairs: 128 / G
// tokens times the G query heads of KV head g, so that a chunk of few tokens
// still fills the tensor core and every K/V tile serves the whole group.  A
// CTA holds two such tiles (2 * (128 / G) consecutive tokens) and walks the
// key tiles of 128 up to its last row's limit:
//   S_i = Q_i . K_t^T    M = 128 rows, N = 128 keys, K = d, fp32 in TMEM;
//   P_i = 2^(S_i c - m)  two threads per row, c = scale * log2 e, m the row's
//                        reference; P_i goes back into TMEM as bf16 over S_i,
//                        the A operand of
//   O_i += P_i . V_t     M = 128, N = d, K = 128 keys, fp32 in TMEM.
// The tensor core's shared-memory reads decide this layout: a 128^3 MMA with
// both operands in shared memory reads 64 KB in the 512 cycles it computes,
// all that an SM's shared memory delivers, so P in shared memory (written,
// then read back) would bound the kernel at two thirds of the MMA rate.
//
// P enters as one bf16 term, as in the single-sequence call: at most 2^-8 of
// itself off, so the output by at most 2^-8 of the mean of |v|, as much as its
// own rounding to bf16.  A second term would be a third MMA per key tile.  The
// sums and the log-sum-exp take the fp32 values.
//
// The reference m is the row's max over its first key tile.  bf16 has the range
// of fp32 and its precision does not depend on the size of p, so m need not
// follow the max: later tiles take no max.  Where a row's sum over 64 keys
// passes 2^60 -- logits 41 above all of the first 128 keys -- the block is
// computed again: a pass over the logits finds the rows' maxima, and the pass
// after it uses those for the rows that need them.  (So it is where a row's
// first 128 logits are all -inf.)
//
// P overwrites the logits it came from (the TMEM has room for a second buffer
// only with 80-key tiles, where the narrower MMAs cost more than the overlap
// gives: 32K tokens 8.4 ms against 7.9), so logits, softmax and output of an
// MMA tile follow one another, and while one tile is at the tensor core the
// other is at its softmax.  Two threads per row halve the time the softmax
// takes.
//
// A CTA goes on to blocks of CTAs of the grid that have not started
// (clusterlaunchcontrol): the next block is found, and its Q and first key
// tiles land, while the softmax warps store the output of the one before.
// What a block costs beside its key tiles went from 9.7 to 6.2 us (about 3.5
// tiles: the first tile's way through, the last one's, the stores), of a
// batch of 512 from 14 to 7.
//
// Measured (32/8 heads, d = 128): 32K tokens 6.9 ms in bursts (1.27 PFLOP/s, 75 %
// of the measured burst rate of a library GEMM), 7.8 to 7.9 ms for seconds on end
// (1.12 PFLOP/s, 80 % of the sustained rate; the board's power bounds it: SM clock
// 1.55 GHz); 8 prompts of 1K to 8K 1.55 to 1.64 ms; 512 prompts of 64 tokens 240 us.
// A key tile takes 3400 cycles of 2048 that its MMAs need: per MMA tile the
// softmax 1700 (1450 of them the exponentials, 1024 at the MUFU's rate) and MMAs
// with their hand-overs 1700.  Tried: a part of the exponentials on the
// FMA pipe as polynomials (1/8: 3 %, 1/2: 10 % slower: more instructions, more
// power); 64-key logits in four chains (19 % slower: N = 64 MMAs take 450 cycles
// where N = 128 ones take 512); half-signals of P; polling instead of suspended
// waits (2 to 4 % slower).
//
// Few rows over many keys: the keys of a block are shared among CTAs, whose
// (log-sum-exp, output) a second kernel joins.
//
// Keys a row does not see are masked before the max.  A masked value row still
// meets p = 0 in the MMA, and 0 * inf = NaN; so the value tiles in which some
// row of the block masks a key are looked over first, infinities and NaN in
// them are set to 0, and the rows that do see such a value add it at the end.
//
// Warps: 0 TMA producer, 1 and 2 MMA issuers of tiles 0 and 1 (1: TMEM), 3 the
// next block and the value check, 4..11 and 12..19 the softmax of tiles 0 and 1.  Every wait is
// bounded; on a timeout the CTA records KVC_DEV_ERR_TIMEOUT, lets its copies
// and MMAs land, frees TMEM and exits.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include <cuda_bf16.h>

#include "common.cuh"
#include "tc.cuh"

namespace kvc {
namespace {

constexpr int kVT = 128;          // rows per MMA tile, keys per key tile
constexpr int kVBlock = 640;      // 20 warps
constexpr int kVMaxClean = 4;     // key tiles of a block in which some row masks a key: at most 3
constexpr float kVMost = 0x1p60f;  // a row's sum over 64 keys past which its reference is too far below its max
constexpr double kLn2 = 0.6931471805599453;
constexpr double kLog2e = 1.4426950408889634;

struct VarArgs {
  const uint16_t* v;     // for the rows that see a non-finite value
  int64_t v_sn, v_sh;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int64_t total_q, total_k, max_q, max_k;
  int batch, H, Hkv, G;
  int nt;                // tokens per tile: 128 / G
  float c;               // scale * log2(e)
  int splits;            // CTAs that share the keys of a block
  int64_t part_rows;     // splits > 1: rows of the partial results, min(total_q, batch * max_q)
  float* part_z;         // [splits][part_rows][H] log-sum-exp of the split, log2 units
  float* part_o;         // [splits][part_rows][H][D] its output
  uint16_t* out;         // [total_q][H][D] or nullptr
  float* lse;            // [total_q][H] or nullptr
  int32_t* err;
};

// The partial results hold the rows of q as they lie there, or, where q has
// room for many more rows than the sequences can have, max_q rows for each.
__device__ __forceinline__ bool parts_by_sequence(const VarArgs& a) { return a.part_rows < a.total_q; }

constexpr int kVBarBytes = 2048;

template <int D>
struct VarSmem {
  static constexpr int kBlk = kVT * 128;         // 128 rows x 128 B: one 64-column block (16 KB)
  static constexpr int kTile = (D / 64) * kBlk;  // a 128 x D bf16 tile
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kRing = 2 * kTile;        // Q: two tiles, then the K/V ring
  static constexpr int kBarOff = kRing + kStages * kTile;
  static constexpr size_t kBytes = 1024 + (size_t)kBarOff + kVBarBytes;
  static_assert(kBytes <= 232448, "shared memory of one CTA");
};

// A block of queries as a CTA computes it, found while the block before runs.
struct VarBlk {
  int seq;             // -1: no more blocks
  int g, split;        // KV head, split
  int q0, k0, lq, lk;  // first query and key of the sequence, and its lengths
  int i0;              // first query of the block in the sequence
  int nt, t_mask, kf;  // key tiles; first of them in which some row masks a key; first key of the first
  int dirty, redo;     // a checked tile holds infinities or NaN; some row passed its reference by too much
  int stop[3];         // by pass: a wait of some thread gave up
};

struct VarBars {
  uint64_t qfull[2], full[8], empty[8];
  uint64_t s_full[2], p_full[2], o_done[2], turn[2];
  uint64_t vland[kVMaxClean], clean[kVMaxClean];  // value tiles to be checked, in turn: landed, checked
  uint64_t stored;   // the output rows of a block have left the ring
  uint64_t claimed;  // the next CTA of the grid was asked for
  uint64_t mma_done;
  uint4 claim;
  uint32_t tmem_base;
  int abort;
  int land[8];  // by stage: the checked tile that was requested into it, or -1
  VarBlk blk[3];
  float swap[2][kVT];  // [tile][row]: what the two threads of a row tell each other
};

// Takes over a CTA of the grid that has not started, if there is one: its index
// lands in *claim with 16 bytes on `bar`.
__device__ __forceinline__ void claim_cta(uint4* claim, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   tc::smem_u32(claim)),
               "r"(tc::smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ int claimed_cta(const uint4* claim) {  // its blockIdx.x, or -1
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(tc::smem_u32(claim))
      : "memory");
  return got ? (int)x : -1;
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem]^T, A bf16 (two K values per 32-bit column).
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// MN-major operand descriptor, 128-byte swizzle: 64 MN-consecutive elements
// per 128-byte row, K rows at 128 B; `lbo` bytes between 64-element MN
// blocks, 1024 B between 8-row K groups.
__device__ __forceinline__ uint64_t desc_mn(uint32_t smem_addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// Blocks of sequence b (0 if it is empty or malformed; *bad then says which).
__device__ __forceinline__ int seq_blocks(const VarArgs& a, int b, bool* bad) {
  const int64_t q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
  *bad = q0 < 0 || q1 < q0 || q1 > a.total_q || k0 < 0 || k1 < k0 || k1 > a.total_k || q1 - q0 > a.max_q ||
         k1 - k0 > a.max_k;
  return *bad ? 0 : (int)(((uint32_t)(q1 - q0) + 2u * a.nt - 1u) / (2u * a.nt));
}

template <int D>
__global__ void __launch_bounds__(kVBlock, 1)
prefill_varlen_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const VarArgs a) {
  using L = VarSmem<D>;
  constexpr int kCB = D / 64;        // 64-column blocks of a tile
  constexpr uint32_t kO = 256;       // first O column; S at 0 and 128
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  VarBars* bars = reinterpret_cast<VarBars*>(sm + L::kBarOff);
  static_assert(sizeof(VarBars) <= kVBarBytes, "barrier block");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      tc::mbar_init(&bars->full[s], 1);
      tc::mbar_init(&bars->empty[s], 2);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars->qfull[i], 1);
      tc::mbar_init(&bars->s_full[i], 1);
      tc::mbar_init(&bars->p_full[i], 8);
      tc::mbar_init(&bars->o_done[i], 1);
      tc::mbar_init(&bars->turn[i], 1);
    }
    for (int i = 0; i < kVMaxClean; ++i) {
      tc::mbar_init(&bars->vland[i], 1);
      tc::mbar_init(&bars->clean[i], 1);
    }
    tc::mbar_init(&bars->stored, 16);
    tc::mbar_init(&bars->claimed, 1);
    tc::mbar_init(&bars->mma_done, 2);
    bars->abort = 0;
    tc::fence_mbar_init();
    tc::prefetch_tmap(&qmap);
    tc::prefetch_tmap(&kmap);
    tc::prefetch_tmap(&vmap);
  }
  if (warp == 1) {
    tc::tmem_alloc(&bars->tmem_base, 512);
    tc::tmem_relinquish();
  }
  // rows past the tokens of a tile (128 % G of them) are zero
  for (int i = tid; i < 2 * kCB * 8 * (kVT - a.nt * a.G); i += kVBlock) {
    const int blk = i / (8 * (kVT - a.nt * a.G)), j = i % (8 * (kVT - a.nt * a.G));
    *reinterpret_cast<uint4*>(sm + blk * L::kBlk + a.nt * a.G * 128 + j * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  tc::fence_proxy_async_smem();
  pdl_wait();  // the inputs may come from the previous kernel of the stream
  // The block of CTA `item` of the grid, by a warp: the splits of a block side by
  // side, then its heads, then the blocks, the last (longest) of a sequence
  // first; up to 32 sequences the longest first, more in order.  Four chunks of
  // 512 queries over 8K to 32K keys: 1010 us in order, 836 us sorted (in turn, at
  // that step; 850 to 890 us since).
  // It looks at 32 sequences, one per lane, and keeps them for the next search.
  int cur_b = 0, cur_before = 0, cur_blocks = 0;  // the first of them, blocks before it, their blocks
  int c_nb = 0, c_before = 0, c_q0 = 0, c_k0 = 0, c_lq = 0, c_lk = 0;  // the lane's: blocks, blocks of them before it
  auto read_sequences = [&]() {
    const int b = cur_b + lane;
    c_nb = 0;
    if (b < a.batch) {
      bool bad;
      c_nb = seq_blocks(a, b, &bad);
      c_q0 = a.cu_q[b];
      c_k0 = a.cu_k[b];
      c_lq = a.cu_q[b + 1] - c_q0;
      c_lk = a.cu_k[b + 1] - c_k0;
    }
    if (a.batch <= 32) {
      const int keys = c_nb > 0 ? c_lk : -1;
      c_before = 0;
#pragma unroll 8
      for (int j = 0; j < a.batch; ++j) {
        const int kj = __shfl_sync(0xffffffffu, keys, j), nj = __shfl_sync(0xffffffffu, c_nb, j);
        if (kj > keys || (kj == keys && j < lane)) c_before += nj;
      }
    } else {
      int inc = c_nb;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      c_before = inc - c_nb;
    }
    cur_blocks = __reduce_add_sync(0xffffffffu, c_nb);
  };
  auto find = [&](int item, VarBlk* out) {
    const unsigned at = (unsigned)item / (unsigned)a.splits;
    const int block = (int)(at / (unsigned)a.Hkv);
    if (item >= 0) {
      if (block < cur_before) {
        cur_b = cur_before = 0;
        read_sequences();
      }
      while (block >= cur_before + cur_blocks && cur_b + 32 < a.batch) {
        cur_before += cur_blocks;
        cur_b += 32;
        read_sequences();
      }
    }
    const int left = block - cur_before;
    const unsigned hit = __ballot_sync(0xffffffffu, item >= 0 && left >= c_before && left < c_before + c_nb);
    const bool mine = hit ? lane == __ffs(hit) - 1 : lane == 0;  // the lane that has the sequence
    if (mine) {
      VarBlk b{};
      b.seq = hit ? cur_b + lane : -1;
      if (hit) {
        b.split = item % a.splits;
        b.g = (int)(at % (unsigned)a.Hkv);
        b.q0 = c_q0;
        b.k0 = c_k0;
        b.lq = c_lq;
        b.lk = c_lk;
        b.i0 = (c_nb - 1 - (left - c_before)) * 2 * a.nt;
        const int lim = std::min(b.lq - b.i0, 2 * a.nt) - 1 + b.i0 + b.lk - b.lq;  // the last row sees keys up to here
        int t0 = 0;
        b.nt = lim >= 0 ? lim / kVT + 1 : 0;
        if (a.splits > 1) {
          t0 = (int)((int64_t)b.nt * b.split / a.splits);
          b.nt = (int)((int64_t)b.nt * (b.split + 1) / a.splits) - t0;
        }
        b.t_mask = std::max(0, std::max(0, b.i0 + b.lk - b.lq + 1) / kVT - t0);
        b.kf = t0 * kVT;
      }
      *out = b;
    }
    __syncwarp();
  };
  if (warp == 3) {
    read_sequences();
    find((int)blockIdx.x, &bars->blk[0]);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort_flag = &bars->abort;
  // The CTA goes from block to block.  Ring and barriers go on counting
  // from block to block, and from pass to pass of a block: pass 0 computes; if
  // a row passed its reference by too much, pass 1 finds every row's max and
  // pass 2 computes with that of the rows that did.
  int n3 = 0;         // the block's number, modulo 3
  int ring0 = 0;      // K and V tiles of the blocks and passes before
  int checks = 0;     // of them the checked ones
  int tiles = 0;      // logits tiles of the blocks and passes before
  bool quit = bars->blk[0].seq < 0;
  // ends a pass; whether the block needs another.  What every thread decides
  // by is written before the barrier and not after it.
  auto again = [&](int pass, int nt, int nc) {
    VarBlk* b = &bars->blk[n3];
    if (*abort_flag) *(volatile int*)&b->stop[pass] = 1;
    tc::named_bar_sync(15, kVBlock);
    ring0 += pass == 1 ? nt : 2 * nt;
    tiles += nt;
    if (pass != 1) checks += nc;
    if (*(volatile int*)&b->stop[pass]) {
      quit = true;
      return false;
    }
    return pass == 0 ? *(volatile int*)&b->redo != 0 : pass == 1;
  };
  auto next_block = [&]() {
    n3 = n3 == 2 ? 0 : n3 + 1;
    if (!quit) quit = *(volatile int*)&bars->blk[n3].seq < 0;
  };
  int issued = 0;           // producer: K and V tiles requested
  int q_loads[2] = {0, 0};  // and Q tiles

  // registers: 640 x 96 at launch; the softmax warps take over what the others do not need
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) {
      // ---- producer: Q of tile 0, K(0), Q of tile 1, then V(0), K(1), V(1), ... (pass 1: K alone)
      for (int n = 0; !quit; ++n, next_block()) {
        const VarBlk b = bars->blk[n3];
        const int nc = std::max(0, b.nt - b.t_mask), first = issued;
        auto load_q = [&](int i) {
          tc::mbar_arrive_expect_tx(&bars->qfull[i], (uint32_t)(kCB * a.nt * a.G * 128));
          for (int cb = 0; cb < kCB; ++cb)
            tc::tma_load_3d(sm + i * L::kTile + cb * L::kBlk, &qmap, &bars->qfull[i], cb * 64, b.g * a.G,
                            b.q0 + b.i0 + i * a.nt);
          ++q_loads[i];
        };
        if (lane == 0 && b.nt > 0) load_q(0);
        for (int pass = 0; pass == 0 || again(pass - 1, b.nt, nc); ++pass) {
          const int count = lane != 0 ? 0 : pass == 1 ? b.nt : 2 * b.nt;
          for (int j = 0; j < count; ++j, ++issued) {
            const int s = issued % L::kStages;
            if (issued >= L::kStages && !tc::mbar_wait(&bars->empty[s], ((issued / L::kStages) - 1) & 1, abort_flag))
              break;
            // the two stages before the block's first hold output rows of the block before
            if (n > 0 && issued == first + L::kStages - 2 && !tc::mbar_wait(&bars->stored, (n - 1) & 1, abort_flag))
              break;
            // a value tile to be checked lands on a barrier of its own, which its
            // readers can wait for without following the ring's phases
            const int t = pass == 1 ? j : j >> 1;
            const bool value = pass != 1 && (j & 1), checked = value && t >= b.t_mask;
            const int c = checks + t - b.t_mask;
            uint64_t* land = checked ? &bars->vland[c % kVMaxClean] : &bars->full[s];
            bars->land[s] = checked ? c : -1;
            if (checked) tc::mbar_arrive(&bars->full[s]);
            tc::mbar_arrive_expect_tx(land, (uint32_t)L::kTile);
            for (int cb = 0; cb < kCB; ++cb)
              tc::tma_load_3d(sm + L::kRing + s * L::kTile + cb * L::kBlk, value ? &vmap : &kmap, land, cb * 64, b.g,
                              b.k0 + b.kf + t * kVT);
            if (issued == first) load_q(1);
          }
          __syncwarp();
        }
      }
    } else if (warp < 3) {
      // ---- MMA issuers, one per MMA tile: S of key tile 0, then for every key
      // tile the output and the next logits, which overwrite the P just used with
      // no wait between the two.  That relies on the tensor core running the MMAs
      // of one issuing thread one after another, in order; PTX promises the order
      // only for MMAs of the same accumulator and shape, which these are not.  No
      // comparison, of any length, has shown otherwise; a commit of P . V and a
      // wait for it would do without, and takes 6 to 9 % (32K tokens 8.4 ms, 8
      // prompts of 1K to 8K 1.66 ms, four chunks 0.95 ms, in turn with 7.8, 1.57, 0.87).
      // The tensor core queues hardly ahead, so what a warp spends on waits and
      // commits would leave it idle; the other tile's MMAs fill that.  They
      // take turns, the next one invited two MMAs early: mixed, both tiles'
      // MMAs would end late and both softmaxes run while the tensor core waits.
      // Stages are released by the softmax warps, which learn from S(t) that
      // everything before it is done: a commit costs the pipe about 100 cycles.
      const int i = warp - 1;
      const uint32_t id_s = tc::idesc_bf16_f32(128, 128);
      const uint32_t id_o = tc::idesc_bf16_f32(128, D) | (1u << 16);  // B (V) MN-major
      const uint64_t q_desc = tc::desc_k_sw128(tc::smem_u32(sm + i * L::kTile));
      const uint64_t k_desc = tc::desc_k_sw128(tc::smem_u32(sm + L::kRing));
      const uint64_t v_desc = desc_mn(tc::smem_u32(sm + L::kRing), (uint32_t)L::kBlk);
      const uint32_t s_tmem = tmem + (uint32_t)(128 * i), o_tmem = tmem + kO + (uint32_t)(D * i);
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) tc::mma_commit(bar);
      };
      int turns = 0;  // groups issued
      auto my_turn = [&]() { return (i == 0 && turns == 0) || tc::mbar_wait(&bars->turn[i], (turns - (i == 0)) & 1, abort_flag); };
      auto your_turn = [&]() {
        ++turns;
        if (elect_one()) tc::mbar_arrive(&bars->turn[i ^ 1]);
      };
      auto logits = [&](int s) {  // S from the K tile in stage s
        const uint64_t kd = k_desc + (uint64_t)((uint32_t)(s * L::kTile) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (uint32_t)((ks >> 2) * L::kBlk + (ks & 3) * 32) >> 4;
          if (ks == D / 16 - 2) your_turn();
          if (elect_one()) tc::mma_bf16(s_tmem, q_desc + off, kd + off, id_s, ks != 0);
        }
        commit(&bars->s_full[i]);
      };
      auto wait_full = [&](int j) { return tc::mbar_wait(&bars->full[j % L::kStages], (j / L::kStages) & 1, abort_flag); };
      for (int qn = 0; !quit; next_block()) {
        const int nt = bars->blk[n3].nt, t_mask = bars->blk[n3].t_mask, nc = std::max(0, nt - t_mask);
        for (int pass = 0; pass == 0 || again(pass - 1, nt, nc); ++pass) {
          if (nt == 0) continue;
          const int base = ring0;
          const bool maxes = pass == 1;
          bool ok = (pass > 0 || tc::mbar_wait(&bars->qfull[i], qn++ & 1, abort_flag)) && wait_full(base) && my_turn();
          if (ok) {
            tc::tc_fence_after();
            logits(base % L::kStages);
          }
          for (int t = 0; ok && t < nt; ++t) {
            const int vj = base + 2 * t + 1, vs = vj % L::kStages;               // V(t)
            const int kj = maxes ? base + t + 1 : vj + 1, ks_ = kj % L::kStages;  // K(t + 1)
            if (!maxes) {
              ok = wait_full(vj);
              const int c = checks + t - t_mask;
              if (ok && t >= t_mask) ok = tc::mbar_wait(&bars->clean[c % kVMaxClean], (c / kVMaxClean) & 1, abort_flag);
            }
            if (ok && t + 1 < nt) ok = wait_full(kj);
            if (ok) ok = tc::mbar_wait(&bars->p_full[i], (tiles + t) & 1, abort_flag);
            if (ok) ok = my_turn();
            if (!ok) break;
            tc::tc_fence_after();
            if (!maxes) {
              const uint64_t vd = v_desc + (uint64_t)((uint32_t)(vs * L::kTile) >> 4);
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)  // 16 keys: 8 columns of P (64 keys over each half of S), 16 value rows of 128 B
                if (elect_one())
                  mma_bf16_ts(o_tmem, s_tmem + (uint32_t)(64 * (ks >> 2) + 8 * (ks & 3)),
                              vd + (uint64_t)((uint32_t)(ks * 16 * 128) >> 4), id_o, (t > 0 || ks > 0) ? 1u : 0u);
            }
            if (t + 1 < nt) {
              logits(ks_);
            } else {
              your_turn();
              if (!maxes) commit(&bars->o_done[i]);
            }
          }
        }
      }
      commit(&bars->mma_done);  // every MMA issued above has completed before TMEM is freed
      tc::mbar_drain(&bars->mma_done, 0);
    } else {
      // ---- value check: the tiles in which some row masks a key; and the next block
      constexpr int kVec = L::kTile / 16;
      auto look = [&]() {
        for (int b = lane; b < a.batch; b += 32) {
          bool bad;
          seq_blocks(a, b, &bad);
          if (bad) set_dev_err(a.err, KVC_DEV_ERR_SEQLENS);
        }
      };
      int claims = 0;
      bool scan = blockIdx.x == 0;  // by whoever computes item 0: every sequence is looked at, for the error word
      for (; !quit; next_block()) {
        const int nt = bars->blk[n3].nt, t_mask = bars->blk[n3].t_mask, nc = std::max(0, nt - t_mask);
        bool first = false;
        auto find_next = [&]() {
          const bool got = tc::mbar_wait(&bars->claimed, claims++ & 1, abort_flag);
          const int item = __shfl_sync(0xffffffffu, got ? claimed_cta(&bars->claim) : -1, 0);
          find(item, &bars->blk[n3 == 2 ? 0 : n3 + 1]);
          first = item == 0;
        };
        for (int pass = 0; pass == 0 || again(pass - 1, nt, nc); ++pass) {
          if (pass == 1) continue;
          if (pass == 0) {
            // The next block is claimed when the first of the tiles to be checked,
            // the last ones of a block, has landed: early enough, and not so early
            // that a CTA with a long block takes one from those that end sooner.
            if (nc > 0) tc::mbar_wait(&bars->vland[checks % kVMaxClean], (checks / kVMaxClean) & 1, abort_flag);
            __syncwarp();
            if (lane == 0) {
              tc::fence_proxy_async_smem();  // the last answer is read
              tc::mbar_arrive_expect_tx(&bars->claimed, 16u);
              claim_cta(&bars->claim, &bars->claimed);
            }
            __syncwarp();
          }
          for (int t = t_mask; t < nt; ++t) {
            const int s = (ring0 + 2 * t + 1) % L::kStages, c = checks + t - t_mask;
            if (!tc::mbar_wait(&bars->vland[c % kVMaxClean], (c / kVMaxClean) & 1, abort_flag)) break;
            uint4* tile = reinterpret_cast<uint4*>(sm + L::kRing + s * L::kTile);
            uint32_t top = 0;  // the largest magnitude, per 16-bit half
#pragma unroll 8
            for (int i = lane; i < kVec; i += 32) {
              const uint4 w = tile[i];
              top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                           __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
            }
            if ((top & 0xFFFFu) >= 0x7F80u || (top >> 16) >= 0x7F80u) {
              bars->blk[n3].dirty = 1;
              for (int i = lane; i < kVec; i += 32) {
                uint32_t* w = reinterpret_cast<uint32_t*>(tile + i);
                for (int u = 0; u < 4; ++u) {
                  uint32_t x = w[u];
                  if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
                  if ((x & 0x7F800000u) == 0x7F800000u) x &= 0x0000FFFFu;
                  w[u] = x;
                }
              }
              tc::fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars->clean[c % kVMaxClean]);
          }
          if (pass == 0) find_next();
        }
        if (scan) look();
        scan = first;
      }
      if (scan) look();
      if (lane == 0 && claims > 0) tc::mbar_drain(&bars->claimed, (claims - 1) & 1);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ---- softmax of one MMA tile, two threads per row: 64 keys of a key tile
    // each, P over the first half of the logits they came from
    const int i = (warp - 4) >> 3, hf = ((warp - 4) >> 2) & 1, wq = warp & 3;
    const int r = 32 * wq + lane;
    const int ti = i * a.nt + r / a.G;  // token of this row in the block
    const uint32_t lane_base = tmem + ((uint32_t)(32 * wq) << 16);
    const uint32_t s_col = lane_base + (uint32_t)(128 * i + 64 * hf), o_col = lane_base + kO + (uint32_t)(D * i + (D / 2) * hf);
    const int pair_bar = 1 + 4 * i + wq;  // named barrier of the two warps that share these rows
    // f(x of half 0, x of half 1) for both threads of the row
    volatile float* swap = &bars->swap[i][r];
    auto both = [&](float mine_x, auto f) {
      if (hf) *swap = mine_x;
      tc::named_bar_sync(pair_bar, 64);
      if (!hf) *swap = mine_x = f(mine_x, *swap);
      tc::named_bar_sync(pair_bar, 64);
      return hf ? *swap : mine_x;
    };
    auto larger = [](float x0, float x1) { return fmaxf(x0, x1); };
    uint32_t x[64];
    auto row_max = [&]() {  // of this thread's logits, in log2 units
      float mx[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) mx[e] = __uint_as_float(x[e]);
#pragma unroll
      for (int e = 4; e < 64; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(x[e]));
      return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.c;
    };
    const bool releases = wq == 0 && hf == 0 && lane == 0;  // tells the producer for this tile
    for (int outs = 0; !quit; next_block()) {
      const VarBlk* b = &bars->blk[n3];
      const int nt = b->nt, t_mask = b->t_mask;
      auto mine = [&]() { return r < a.nt * a.G && ti < b->lq - b->i0; };
      // the last key the row sees, counted from the first one of this thread
      const int limit = std::min(ti, b->lq - b->i0 - 1) + b->i0 + b->lk - b->lq - b->kf - 64 * hf;
      float m_ref = -INFINITY, top = -INFINITY;
      bool past = false;  // the row needs its maximum as reference
      double l = 0.0;  // this thread's half of the row sum
      bool ok = true;
      for (int pass = 0; pass == 0 || again(pass - 1, nt, 0); ++pass) {
        const int base = ring0;
        l = 0.0;
        for (int t = 0; t < nt; ++t) {
          if (!tc::mbar_wait(&bars->s_full[i], (tiles + t) & 1, abort_flag)) ok = false;
          if (releases && ok) {  // S(t) is there: K(t) and, before it, V(t - 1) are read
            if (pass == 1) {
              tc::mbar_arrive(&bars->empty[(base + t) % L::kStages]);
            } else {
              tc::mbar_arrive(&bars->empty[(base + 2 * t) % L::kStages]);
              if (t > 0) tc::mbar_arrive(&bars->empty[(base + 2 * t - 1) % L::kStages]);
            }
          }
          __syncwarp();
          tc::tc_fence_after();
          KVC_TMEM_LD64(s_col, x);
          KVC_TMEM_WAIT_LD64(x);
          if (t >= t_mask) {
            const int lim = limit - t * kVT;  // the last visible column
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (e > lim) x[e] = __float_as_uint(-INFINITY);
          }
          if (pass == 1) {
            top = fmaxf(top, row_max());
          } else {
            if (pass == 0 && t == 0) {  // the first tile sets the references, if it has a logit above -inf
              m_ref = both(row_max(), larger);
              past = m_ref == -INFINITY && limit >= kVT - 64 * hf;
            }
            // a row that has seen no key yet has only x = -inf: p = 2^-inf = 0
            const float ref = m_ref == -INFINITY ? 0.f : m_ref;
            const float2 c2 = make_float2(a.c, a.c), nm2 = make_float2(-ref, -ref);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int u = 0; u < 32; ++u) {
              const float2 y = tc::fma2(make_float2(__uint_as_float(x[2 * u]), __uint_as_float(x[2 * u + 1])), c2, nm2);
              const float2 p = make_float2(tc::ex2_approx(y.x), tc::ex2_approx(y.y));
              sum[u & 1] = tc::add2(sum[u & 1], p);
              const __nv_bfloat162 hp = __floats2bfloat162_rn(p.x, p.y);
              x[u] = *reinterpret_cast<const uint32_t*>(&hp);
            }
            tmem_st32(s_col, *reinterpret_cast<const uint32_t(*)[32]>(x));
            const float2 s2 = tc::add2(sum[0], sum[1]);
            const float s = s2.x + s2.y;
            past |= s > kVMost;
            l += (double)s;
            tmem_wait_st();
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0 && ok) tc::mbar_arrive(&bars->p_full[i]);
        }
        if (pass == 1) {
          // the other rows keep theirs, and their results to the last bit
          top = both(top, larger);
          if (both(past ? 1.f : 0.f, larger) > 0.f) m_ref = top;
        } else {
          if (nt > 0 && !tc::mbar_wait(&bars->o_done[i], outs++ & 1, abort_flag)) ok = false;
          if (nt > 0 && releases && ok) tc::mbar_arrive(&bars->empty[(base + 2 * nt - 1) % L::kStages]);
          if (pass == 0 && past && mine()) bars->blk[n3].redo = 1;
        }
      }
      // ---- the output rows and log-sum-exp; the halves store a half of the columns each
      if (quit) break;
      __syncwarp();
      int ln = lane;  // the lane, from which nothing can be computed ahead of the loop over the blocks
      asm volatile("" : "+r"(ln));
      const int q0 = b->q0, k0 = b->k0, i0 = b->i0, g = b->g, h = g * a.G + r % a.G;
      const bool own = mine();
      const int64_t row = (int64_t)(q0 + i0) + ti;  // the row of out and lse
      const int64_t part = b->split * a.part_rows + (parts_by_sequence(a) ? b->seq * a.max_q + i0 + ti : row);
      const float sum_row = both((float)l, [](float x0, float x1) { return x0 + x1; });
      {
        tc::tc_fence_after();
        const bool seen = limit >= -64 * hf && nt > 0;  // no key of this CTA otherwise
        const float inv = seen ? 1.f / sum_row : 0.f;
        const bool dirty = *(volatile int*)&b->dirty != 0;
        // this warp's rows, in one of the ring's two stages that are requested last: pieces of 16 bytes, swizzled
        constexpr int kCols = D / 2, kPitch = kCols * 2;  // columns of this thread
        uint8_t* stage = sm + L::kRing + (ring0 + L::kStages - 2 + i) % L::kStages * L::kTile + ((warp - 4) & 7) * 32 * kPitch;
        auto piece_of = [](int row_, int piece_) {
          return row_ * kPitch + ((piece_ ^ (D == 128 ? row_ & 7 : row_ >> 1 & 3)) << 4);
        };
#pragma unroll 1
        for (int c0 = 0; c0 < kCols; c0 += 32) {
          uint32_t o[32];
          if (nt > 0) {
            KVC_TMEM_LD32(o_col + (uint32_t)c0, o);
            KVC_TMEM_WAIT_LD32(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (!a.out && !a.part_o) continue;
          float f[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] = seen ? __uint_as_float(o[e]) * inv : 0.f;
          const int col = kCols * hf + c0;
          if (dirty && own)  // non-finite values of the checked tiles, where this row sees them
            for (int kf = b->kf, j = kf + t_mask * kVT; j <= limit + kf + 64 * hf && j < kf + nt * kVT; ++j) {
              const uint16_t* vr = a.v + (int64_t)(k0 + j) * a.v_sn + (int64_t)g * a.v_sh + col;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const uint32_t bits = vr[e];
                if ((bits & 0x7F80u) == 0x7F80u) f[e] += __uint_as_float(bits << 16);
              }
            }
          if (a.part_o) {
            float4* po = reinterpret_cast<float4*>(a.part_o + (part * a.H + h) * D + col);
            if (own)
#pragma unroll
              for (int u = 0; u < 8; ++u) po[u] = make_float4(f[4 * u], f[4 * u + 1], f[4 * u + 2], f[4 * u + 3]);
            continue;
          }
#pragma unroll
          for (int v8 = 0; v8 < 4; ++v8) {
            uint32_t w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const __nv_bfloat162 hp = __floats2bfloat162_rn(f[8 * v8 + 2 * u], f[8 * v8 + 2 * u + 1]);
              w[u] = *reinterpret_cast<const uint32_t*>(&hp);
            }
            *reinterpret_cast<uint4*>(stage + piece_of(ln, c0 / 8 + v8)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if (a.out && !a.part_o) {
          // through the ring, so that a store covers whole lines of a
          // few rows instead of 16 bytes of 32
          __syncwarp();
          constexpr int kPer = kCols / 8, kAt = 32 / kPer;  // lns per row, rows per store
          const int rel = own ? ti * a.H + h : -1, piece = ln % kPer;
          uint16_t* base = a.out + (int64_t)(q0 + i0) * a.H * D + kCols * hf + piece * 8;
#pragma unroll
          for (int k = 0; k < 32 / kAt; ++k) {
            const int src = kAt * k + ln / kPer;
            const int at = __shfl_sync(0xffffffffu, rel, src);
            const uint4 y = *reinterpret_cast<const uint4*>(stage + piece_of(src, piece));
            if (at >= 0) *reinterpret_cast<uint4*>(base + (int64_t)at * D) = y;
          }
        }
        if (own && hf == 0) {
          // m_ref + log2(sum), the logarithm from the sum's mantissa and exponent
          int e2;
          const float f2 = frexpf(sum_row, &e2);
          const double z = (double)m_ref + ((double)e2 + (double)log2f(f2));
          if (a.part_z)
            a.part_z[part * a.H + h] = seen ? (float)z : -INFINITY;
          else if (a.lse)
            a.lse[row * a.H + h] = seen ? (float)(z * kLn2) : -INFINITY;
        }
        tc::tc_fence_before();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->stored);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (*abort_flag && tid == 0) {
    set_dev_err(a.err, KVC_DEV_ERR_TIMEOUT);
    for (int i = 0; i < 2; ++i)
      if (q_loads[i] > 0) tc::mbar_drain(&bars->qfull[i], (q_loads[i] - 1) & 1);
    for (int j = std::max(0, issued - L::kStages); j < issued; ++j) {
      const int s = j % L::kStages, c = bars->land[s];
      if (c >= 0)
        tc::mbar_drain(&bars->vland[c % kVMaxClean], (c / kVMaxClean) & 1);
      else
        tc::mbar_drain(&bars->full[s], (j / L::kStages) & 1);
    }
  }
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Joins the splits of a row, one warp per (row of the partial results, head):
// out = sum_s 2^(z_s - Z) o_s, Z = log2 sum_s 2^z_s; rows of no (sound) sequence are left as they are.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) prefill_join_kernel(const VarArgs a) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int ph = (int)blockIdx.x * (kJoinThreads / 32) + (int)(threadIdx.x >> 5);  // partial row * H + head
  const int n = (int)a.part_rows * a.H;  // times the splits below 2^17
  if (ph >= n) return;
  const int part = ph / a.H;
  int row = part;  // of q
  int keys = -1;       // the keys that the row sees; -1: a row of no (sound) sequence
  auto look = [&](int b) {
    bool bad;
    seq_blocks(a, b, &bad);
    if (bad || row < a.cu_q[b] || row >= a.cu_q[b + 1]) return;
    keys = std::max(0, row + 1 - a.cu_q[b + 1] + (a.cu_k[b + 1] - a.cu_k[b]));
  };
  if (parts_by_sequence(a)) {
    const int most = (int)a.max_q, b = part / most;
    row = a.cu_q[b] + part % most;
    look(b);
  } else {
    for (int b = lane; b < a.batch; b += 32) look(b);
  }
  keys = __reduce_max_sync(0xffffffffu, keys);
  if (keys < 0) return;
  const int64_t rh = (int64_t)row * a.H + ph % a.H;  // of out and lse
  float Z = -INFINITY;
  for (int s = 0; s < a.splits; ++s) Z = fmaxf(Z, a.part_z[s * n + ph]);
  float acc[D / 32], sum = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
#pragma unroll 8
  for (int s = 0; s < a.splits; ++s) {
    const float z = a.part_z[s * n + ph];
    if (z == -INFINITY) continue;  // no key of the split, or all its logits are -inf
    const float w = tc::ex2_approx(z - Z);
    sum += w;
    const float* o = a.part_o + (s * n + ph) * D + lane * (D / 32);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] += w * o[e];
  }
  const bool seen = keys > 0;  // not told by Z: it is -inf as well where every logit is, or is NaN
  const float inv = seen ? 1.f / sum : 0.f;
  if (a.out) {
#pragma unroll
    for (int e = 0; e < D / 32; e += 2) {
      const __nv_bfloat162 hp = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
      *reinterpret_cast<__nv_bfloat162*>(a.out + rh * D + lane * (D / 32) + e) = hp;
    }
  }
  if (a.lse && lane == 0) a.lse[rh] = seen ? (float)(((double)Z + log2((double)sum)) * kLn2) : -INFINITY;
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

// 3-D map over a strided [n][heads][d] bf16 tensor: boxes of 64 columns x box_h heads x box_n rows.
kvc_status make_map(CUtensorMap* m, const uint16_t* base, int d, int heads, int64_t n, int64_t sn, int64_t sh, int box_h,
                    int box_n) {
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)n};
  cuuint64_t strides[2] = {(cuuint64_t)sh * 2, (cuuint64_t)sn * 2};
  cuuint32_t box[3] = {64u, (cuuint32_t)box_h, (cuuint32_t)box_n};
  cuuint32_t es[3] = {1u, 1u, 1u};
  if (heads == 1) strides[0] = (cuuint64_t)d * 2;  // a size-1 dimension still needs a legal stride
  if (n == 1) strides[1] = (cuuint64_t)d * 2;
  if (encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return fail(KVC_ERR_CUDA, "cuTensorMapEncodeTiled failed for the prefill operands");
  return KVC_OK;
}

kvc_status check_varlen(int32_t H, int32_t Hkv, int32_t d, int32_t batch, int64_t total_q, int64_t max_q,
                        int64_t max_k) {
  if (d != 64 && d != 128) return fail(KVC_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  KVC_CHECK_ARG(H >= 1 && Hkv >= 1 && H % Hkv == 0, "num_heads must be a positive multiple of num_kv_heads");
  if (H / Hkv > kVT) return fail(KVC_ERR_UNSUPPORTED, "at most 128 query heads per KV head");
  KVC_CHECK_ARG(batch >= 1 && batch <= 1024, "batch must be in 1..1024");
  KVC_CHECK_ARG(total_q >= 0 && total_q < (int64_t(1) << 31), "need 0 <= total_q < 2^31");
  KVC_CHECK_ARG(max_q >= 0 && max_k >= 0 && max_q < (int64_t(1) << 31) && max_k < (int64_t(1) << 31),
                "need 0 <= max_seqlen < 2^31");
  return KVC_OK;
}

template <int D>
kvc_status launch_varlen(dim3 grid, cudaStream_t st, const CUtensorMap (&maps)[3], const VarArgs& a) {
  static ContextCache cache;
  const kvc_status s = once_per_context(cache, [] {
    KVC_CUDA_TRY(cudaFuncSetAttribute(prefill_varlen_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)VarSmem<D>::kBytes));
    return KVC_OK;
  });
  if (s != KVC_OK) return s;
  const Launch l(grid, dim3(kVBlock), VarSmem<D>::kBytes, st);
  KVC_CUDA_TRY(l.run(prefill_varlen_kernel<D>, maps[0], maps[1], maps[2], a));
  count_launch();
  if (a.splits == 1) return KVC_OK;
  const int64_t warps = a.part_rows * a.H, per = kJoinThreads / 32;
  const Launch j(dim3((unsigned)((warps + per - 1) / per)), dim3(kJoinThreads), 0, st);
  KVC_CUDA_TRY(j.run(prefill_join_kernel<D>, a));
  count_launch();
  return KVC_OK;
}

// Blocks of all sequences: at most one that is not full per sequence.
int64_t varlen_blocks(int nt, int batch, int64_t total_q, int64_t max_q) {
  const int64_t per = 2 * nt;
  return std::min(total_q / per + batch, (int64_t)batch * ((max_q + per - 1) / per));
}

// CTAs that share the keys of a block.  Few rows over many keys (a window's
// or a small chunk's queries) leave most SMs without a CTA; the splits are
// chosen by the time of all waves, in key tiles, with kSplitCost for what a CTA
// and the joining cost beside its tiles.  At most three CTAs per SM come of it,
// which bounds the workspace: their blocks hold at most 256 (row, head) pairs
// each, whatever room q has behind the sequences.
constexpr int64_t kSplitCost = 6;
int varlen_splits(int64_t items, int64_t max_k) {
  const int64_t sms = num_sms(), tiles = (max_k + kVT - 1) / kVT;
  auto cost = [&](int64_t n) {
    return (items * n + sms - 1) / sms * ((tiles + n - 1) / n + kSplitCost) + (n > 1 ? kSplitCost : 0);
  };
  int64_t best = 1;
  for (int64_t n = 2; n <= 64 && n <= tiles && items * n <= 3 * sms; ++n)
    if (cost(n) < cost(best)) best = n;
  return (int)best;
}

bool carve_varlen(int H, int Hkv, int d, int batch, int64_t total_q, int64_t max_q, int64_t max_k, WsCursor* w, VarArgs* a) {
  a->splits = varlen_splits(varlen_blocks(kVT / (H / Hkv), batch, total_q, max_q) * Hkv, max_k);
  if (a->splits == 1) return true;
  a->part_rows = std::min(total_q, batch * max_q);
  const size_t rows = (size_t)a->splits * (size_t)a->part_rows * H;
  a->part_z = w->take<float>(rows);
  a->part_o = w->take<float>(rows * d);
  return w->ok;
}

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" kvc_status kvc_prefill_varlen_workspace_size(int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                                        int32_t batch, int64_t total_q, int64_t max_seqlen_q,
                                                        int64_t max_seqlen_k, size_t* bytes) {
  clear_error();
  const kvc_status s = check_varlen(num_heads, num_kv_heads, head_dim, batch, total_q, max_seqlen_q, max_seqlen_k);
  if (s != KVC_OK) return s;
  KVC_CHECK_ARG(bytes != nullptr, "bytes must be non-NULL");
  WsCursor w{nullptr, ~size_t(0)};
  VarArgs a{};
  carve_varlen(num_heads, num_kv_heads, head_dim, batch, total_q, max_seqlen_q, max_seqlen_k, &w, &a);
  *bytes = w.off;
  return KVC_OK;
}

extern "C" kvc_status kvc_prefill_attention_varlen(
    const uint16_t* q, int64_t q_stride_n, int64_t q_stride_h, const uint16_t* k, int64_t k_stride_n,
    int64_t k_stride_h, const uint16_t* v, int64_t v_stride_n, int64_t v_stride_h, const int32_t* cu_seqlens_q,
    const int32_t* cu_seqlens_k, int32_t batch, int64_t total_q, int64_t total_k, int64_t max_seqlen_q,
    int64_t max_seqlen_k, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, float scale, uint16_t* out,
    float* lse, void* ws, size_t ws_bytes, int32_t* dev_err, void* stream) {
  clear_error();
  kvc_status s = check_varlen(num_heads, num_kv_heads, head_dim, batch, total_q, max_seqlen_q, max_seqlen_k);
  if (s != KVC_OK) return s;
  if (total_q == 0) return KVC_OK;  // no row to write
  KVC_CHECK_ARG(total_k >= 0 && total_k < (int64_t(1) << 31), "need 0 <= total_k < 2^31");
  if (total_k == 0) k = v = q;  // no key to read: the maps only need an address
  KVC_CHECK_ARG(q && k && v && cu_seqlens_q && cu_seqlens_k, "q, k, v and the cu_seqlens must be non-NULL");
  KVC_CHECK_ARG(scale > 0.f && scale < 1e30f, "scale must be positive and finite");
  KVC_CHECK_ARG(aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && (!out || aligned(out, 16)),
                "q, k, v and out must be 16-byte aligned");
  for (const int64_t st : {q_stride_n, q_stride_h, k_stride_n, k_stride_h, v_stride_n, v_stride_h})
    KVC_CHECK_ARG(st >= head_dim && st % 8 == 0 && st < (int64_t(1) << 36),
                  "strides must be multiples of 8 elements, at least head_dim");
  VarArgs a{};
  a.v = v;
  a.v_sn = v_stride_n;
  a.v_sh = v_stride_h;
  a.cu_q = cu_seqlens_q;
  a.cu_k = cu_seqlens_k;
  a.total_q = total_q;
  a.total_k = total_k;
  a.max_q = max_seqlen_q;
  a.max_k = max_seqlen_k;
  a.batch = batch;
  a.H = num_heads;
  a.Hkv = num_kv_heads;
  a.G = num_heads / num_kv_heads;
  a.nt = kVT / a.G;
  a.c = (float)((double)scale * kLog2e);
  a.out = out;
  a.lse = lse;
  a.err = dev_err;
  // with max_seqlen_q 0 there is no block, but a sequence that has queries all the same is to be reported
  const int64_t blocks = std::max<int64_t>(1, varlen_blocks(a.nt, batch, total_q, max_seqlen_q));
  KVC_CHECK_ARG(blocks * num_kv_heads < (int64_t(1) << 31), "too many query blocks for one call");
  WsCursor w{static_cast<char*>(ws), ws_bytes};
  if (!carve_varlen(num_heads, num_kv_heads, head_dim, batch, total_q, max_seqlen_q, max_seqlen_k, &w, &a) ||
      (a.splits > 1 && (!ws || !aligned(ws, kWsAlign))))
    return fail(KVC_ERR_WORKSPACE, "prefill workspace missing, too small or not 256-B aligned");
  if (!encode_fn()) return fail(KVC_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  CUtensorMap maps[3];
  s = make_map(&maps[0], q, head_dim, num_heads, total_q, q_stride_n, q_stride_h, a.G, a.nt);
  if (s == KVC_OK) s = make_map(&maps[1], k, head_dim, num_kv_heads, std::max<int64_t>(1, total_k), k_stride_n, k_stride_h, 1, kVT);
  if (s == KVC_OK) s = make_map(&maps[2], v, head_dim, num_kv_heads, std::max<int64_t>(1, total_k), v_stride_n, v_stride_h, 1, kVT);
  if (s != KVC_OK) return s;
  const dim3 grid((unsigned)(blocks * num_kv_heads * a.splits));
  const cudaStream_t st = (cudaStream_t)stream;
  return head_dim == 128 ? launch_varlen<128>(grid, st, maps, a) : launch_varlen<64>(grid, st, maps, a);
}
