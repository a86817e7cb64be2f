// Weight gradient from an 8-bit activation checkpoint:  dw[i][j] (+)= alpha sum_m dy[m][i] x[m][j],  x = code * step.
//
// A matrix product with the tokens m as its long axis: 2 m n k operations on m (2 n + k) bytes, so it belongs on the tensor
// cores (tcgen05).  Decoding x to memory first would write and read 2 m k bytes more and hold a full bf16 copy; here the
// codes are decoded on the way into shared memory, by warps that do nothing else.
//
// Two CTAs (a cluster) work on one 256 x 256 tile of dw with tcgen05.mma.cta_group::2: each holds 128 of the tile's rows
// (dy columns) and decodes 128 of its columns; the pair shares both halves of x, so a step of 64 tokens costs each SM 16 KB of dy
// and 16 KB of decoded x in shared memory against 512 cycles of matrix work.  One-CTA tiles would decode twice as much.
// Both operands have the token as their row in memory, that is, the contraction is the slow axis ("MN-major" operands):
// a slab of 64 columns x 64 tokens lies as 64 rows of 128 bytes, 128-byte swizzled, which is how TMA writes dy's slabs and
// how the decoding warps write theirs.
//
// Warps of a CTA: 0 loads dy by TMA; 1 (of the first CTA) issues the MMAs; 2 passes complete stages on; 4-11 take the
// accumulators out of TMEM; 12-19 decode.  The decoders load their codes straight from global memory into registers, three
// steps ahead: through shared memory they would take a quarter more of its bandwidth.
//
// Sums: the tensor cores cut the sums that they accumulate in TMEM rather than round them, so the error of a long sum grows with
// its length (5.7e-6 of the result's norm after 8192 tokens, where fp32 rounded at every step gives 5.4e-7).  So every
// 512 tokens start a new accumulator, and the finished one is added, rounded, to sums that eight warps hold in registers
// (128 a thread: setmaxnreg gives them what the other warps do without).  TMEM holds two accumulators, so the MMAs go on.
//
// Decoding: with b = code bits, 0x4300 | (b & 0x7f) is the bf16 128 + (b & 0x7f), and 0x4300 | (b & 0x80) is 128, or 256 for a
// negative code; their difference is the code, exactly, and times a power of two it stays exact: five instructions for two
// values, no conversion instruction.
//
// Few tiles and many tokens: the tokens are split into slices, each slice's product goes to the workspace in fp32, and a
// second kernel adds the slices in order.
//
// Waits are bounded.  One that runs out makes the CTA stop and fill its tiles with NaN, which the step's check of the
// gradients turns into a skipped step.
#include <cuda.h>

#include "op_common.cuh"

namespace dp {
namespace {

constexpr int BM = 256, BN = 256, BK = 64;       // dw rows, dw columns, tokens of a step (of a CTA pair)
constexpr int STAGES = 6;
constexpr int SLAB = 64 * 128;                   // 64 tokens x 64 bf16
constexpr int A_BYTES = 2 * SLAB, B_BYTES = 2 * SLAB, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int STAGING = 32 * 33 * 4;             // a warp's 32 x 32 block of the result
constexpr int CHUNK = 8;                         // steps of one accumulator
constexpr int EPI0 = 4, EPI_WARPS = 8, DEC0 = 12, DEC_WARPS = 8;
constexpr int THREADS = (DEC0 + DEC_WARPS) * 32;
constexpr int AHEAD = 3;                         // steps of codes in registers; divides STAGES
// Registers a thread: 96 at launch (640 threads); control warps give up 48, decoders 40, summing warps take 64: 48 + 2 * 160
// + 2 * 56 = 5 * 96.
constexpr int REGS_CONTROL = 48, REGS_SUM = 160, REGS_DECODE = 56;
constexpr int BARS = 8 * (4 * STAGES + 7);
constexpr int SMEM = STAGES * STAGE_BYTES + EPI_WARPS * STAGING + 1024 + BARS;
constexpr int MAX_SLICES = 32;

struct WgradParams {
  const uint16_t* dy;
  const int8_t* codes;
  const uint8_t* scales;
  void* dw;
  float* part;      // slices' products, or NULL for one slice
  int64_t rows, n, k, lddy, pitch;
  int64_t tiles_k, tiles, items, steps;  // steps: of 64 tokens, of one slice
  float alpha;
  int dtype, accumulate;
  uint64_t timeout_ns;
};

// ---------------------------------------------------------------------------------------------- PTX building blocks

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Bounded wait; one that runs out, or that finds the CTA stopping, returns false and leaves the CTA stopping.
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint64_t timeout_ns, volatile int* stop) {
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*stop) return false;
    if (globaltimer_ns() - t0 > timeout_ns) {
      *stop = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, uint64_t timeout_ns, volatile int* stop) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, timeout_ns, stop);
}
// Arrives at the barrier of the same shared-memory offset in CTA `rank` of the cluster.
__device__ __forceinline__ void arrive_at(uint32_t bar, uint32_t rank) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar), "r"(rank)
      : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Shared-memory descriptor of an MN-major operand with 128-byte swizzle: slabs of 64 columns SLAB bytes apart (leading
// offset), groups of eight tokens 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(SLAB >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: bf16 x bf16 -> fp32, both operands MN-major, M = 256, N = 256.
constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) | ((BN / 8) << 17) | ((BM / 16) << 24);

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(IDESC), "r"(add)
      : "memory");
}
// Arrives at `bar` in both CTAs once all MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
}
// 32 bytes of codes, 32-byte aligned.
__device__ __forceinline__ void load_codes(const int8_t* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}

// Two bf16 values of two codes already spread over bytes 0 and 2: lo7 = 0x43 mm 0x43 mm, sign = 0x43 ss 0x43 ss.
__device__ __forceinline__ uint32_t decode2(uint32_t lo7, uint32_t sign, __nv_bfloat162 step) {
  const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162*>(&lo7);
  const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&sign);
  const __nv_bfloat162 r = __hmul2(__hsub2(a, b), step);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint2 decode4(uint32_t w, __nv_bfloat162 step) {
  const uint32_t lo = w & 0x7f7f7f7fu, hi = w & 0x80808080u;
  return make_uint2(decode2(__byte_perm(lo, 0x43434343u, 0x4140), __byte_perm(hi, 0x43434343u, 0x4140), step),
                    decode2(__byte_perm(lo, 0x43434343u, 0x4342), __byte_perm(hi, 0x43434343u, 0x4342), step));
}

// The tile, slice and first token of an item; items of one slice run through the tiles with dw's columns fastest, so
// that CTAs that run together share dy's columns and the codes in L2.
struct Item {
  int64_t row0, col0, slice, token0;
  int steps;
};
__device__ __forceinline__ Item item_at(const WgradParams& P, int64_t item) {
  Item it;
  it.slice = item / P.tiles;
  const int64_t tile = item - it.slice * P.tiles;
  const int64_t tr = tile / P.tiles_k;
  it.row0 = tr * BM;
  it.col0 = (tile - tr * P.tiles_k) * BN;
  it.token0 = it.slice * P.steps * BK;
  const int64_t left = (P.rows - it.token0 + BK - 1) / BK;
  it.steps = (int)(left < P.steps ? left : P.steps);
  return it;
}

// One element of the result of an item.
__device__ __forceinline__ void put_result(const WgradParams& P, int64_t slice, int64_t row, int64_t col, float v) {
  if (P.part) P.part[(slice * P.n + row) * P.k + col] = v;
  else grad_put(P.dw, row * P.k + col, P.dtype, P.accumulate, v);
}

// Up to 32 rows of one column of a warp's block to memory.  Adding in fp32 is left to the L2: each element gets one
// addition a call, so nothing depends on an order, and nobody waits for the old value.  bf16 has to be added in fp32 and
// rounded once, so its old values are read, 8 rows in flight.
__device__ __forceinline__ void store_block(const WgradParams& P, int64_t slice, int64_t row0, int64_t col, const float* block,
                                            int rows) {
  if (!P.part && P.dtype == DP_BF16) {
    bf16_t* dst = static_cast<bf16_t*>(P.dw) + row0 * P.k + col;
    for (int r0 = 0; r0 < rows; r0 += 8) {
      float old[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) old[r] = P.accumulate && r0 + r < rows ? bf16_to_f32(dst[r * P.k]) : 0.0f;
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r0 + r < rows) dst[r * P.k] = bf16_rn(__fadd_rn(old[r], block[(r0 + r) * 33]));
      dst += 8 * P.k;
    }
    return;
  }
  float* dst = (P.part ? P.part + slice * P.n * P.k : static_cast<float*>(P.dw)) + row0 * P.k + col;
  const bool add = !P.part && P.accumulate;
#pragma unroll 4
  for (int r = 0; r < rows; ++r) {
    const float v = block[r * 33];
    if (add) asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(dst), "f"(v) : "memory");
    else *dst = v;
    dst += P.k;
  }
}

template <bool TMA>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    wgrad8_kernel(const __grid_constant__ WgradParams P, const __grid_constant__ CUtensorMap map_dy) {
  extern __shared__ char smem_raw[];
  const uint32_t smem0 = smem_u32(smem_raw);
  const uint32_t tiles = (smem0 + 1023) & ~1023u;  // the swizzle pattern repeats every 1024 bytes
  char* smem = smem_raw + (tiles - smem0);
  char* after = smem + STAGES * STAGE_BYTES;
  float* staging = reinterpret_cast<float*>(after);
  uint64_t* bars = reinterpret_cast<uint64_t*>(after + EPI_WARPS * STAGING);
  const uint32_t bar0 = smem_u32(bars);
  auto a_full = [&](int s) { return bar0 + 8 * s; };
  auto full = [&](int s) { return bar0 + 8 * (STAGES + s); };
  auto empty = [&](int s) { return bar0 + 8 * (2 * STAGES + s); };
  auto acc_full = [&](int b) { return bar0 + 8 * (3 * STAGES + b); };
  auto acc_empty = [&](int b) { return bar0 + 8 * (3 * STAGES + 2 + b); };
  auto decoded = [&](int s) { return bar0 + 8 * (3 * STAGES + 4 + s); };
  const uint32_t drained = bar0 + 8 * (4 * STAGES + 4);
  volatile int* stop = reinterpret_cast<int*>(bars + 4 * STAGES + 5);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 4 * STAGES + 6);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(a_full(s), 1);
      mbar_init(decoded(s), DEC_WARPS);
      mbar_init(full(s), 2);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 2 * EPI_WARPS);
    }
    mbar_init(drained, 1);
    *stop = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);

  if (warp < EPI0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_CONTROL));
  if (warp == 0) {
    // ---------------------------------------------------------------- dy by TMA: two slabs of 64 columns a step
    if (TMA && lane == 0) {
      int s = 0, phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (int64_t item = pair; ok && item < P.items; item += pairs) {
        const Item it = item_at(P, item);
        const int x = (int)(it.row0 + rank * 128);
        for (int i = 0; ok && i < it.steps; ++i) {
          ok = wait_bar(empty(s), phase ^ 1, P.timeout_ns, stop);
          if (!ok) break;
          const uint32_t a = tiles + s * STAGE_BYTES;
          const int y = (int)(it.token0 + (int64_t)i * BK);
          mbar_arrive_expect_tx(a_full(s), A_BYTES);
          tma_load(a, &map_dy, x, y, a_full(s));
          tma_load(a + SLAB, &map_dy, x + 64, y, a_full(s));
          ++issued;
          if (++s == STAGES) s = 0, phase ^= 1;
        }
      }
      if (!ok) {  // the copies still in flight land before the CTA may end
        volatile int none = 0;
        for (int64_t q = issued > STAGES ? issued - STAGES : 0; q < issued; ++q)
          wait_bar(a_full((int)(q % STAGES)), (uint32_t)(q / STAGES) & 1, P.timeout_ns, &none);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- the pair's MMAs
    if (rank == 0 && lane == 0) {
      int s = 0, phase = 0, b = 0, bphase = 0;
      bool ok = true;
      for (int64_t item = pair; ok && item < P.items; item += pairs) {
        const Item it = item_at(P, item);
        for (int i = 0; i < it.steps; ++i) {
          const bool fresh = i % CHUNK == 0;
          ok = (!fresh || wait_bar(acc_empty(b), bphase ^ 1, P.timeout_ns, stop)) && wait_bar(full(s), phase, P.timeout_ns, stop);
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t a = tiles + s * STAGE_BYTES;
#pragma unroll
          for (int q = 0; q < BK / 16; ++q)  // 16 tokens: two groups of eight, 2048 bytes on
            mma_pair(tmem + b * BN, operand_desc(a + q * 2048), operand_desc(a + A_BYTES + q * 2048), !fresh || q != 0);
          commit_pair(empty(s));
          if (++s == STAGES) s = 0, phase ^= 1;
          if (i % CHUNK == CHUNK - 1 || i == it.steps - 1) {
            commit_pair(acc_full(b));
            if (++b == 2) b = 0, bphase ^= 1;
          }
        }
      }
      if (!ok) {  // MMAs in flight end before the CTA may end
        volatile int none = 0;
        commit_pair(drained);
        wait_bar(drained, 0, P.timeout_ns, &none);
      }
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- stages complete in this CTA -> the pair's MMAs
    // This warp orders the decoders' writes before the tensor cores' reads and tells the first CTA.  The decoders do not
    // do so themselves: the fence and the cluster-wide release would wait for the codes that they have in flight.
    if (lane == 0) {
      int s = 0, phase = 0;
      bool ok = true;
      for (int64_t item = pair; ok && item < P.items; item += pairs) {
        const int steps = item_at(P, item).steps;
        for (int i = 0; ok && i < steps; ++i) {
          ok = (!TMA || wait_bar(a_full(s), phase, P.timeout_ns, stop)) && wait_bar(decoded(s), phase, P.timeout_ns, stop);
          if (!ok) break;
          fence_proxy_async_smem();
          arrive_at(full(s), 0);
          if (++s == STAGES) s = 0, phase ^= 1;
        }
      }
    }
  } else if (warp >= EPI0 && warp < DEC0) {
    // ---------------------------------------------------------------- sums, and the result to memory
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SUM));
    const int quad = warp & 3;               // TMEM lanes 32 quad .. + 31: a warp may read no others
    const int half = (warp - EPI0) >> 2;     // columns 128 half .. + 127
    float* mine = staging + (warp - EPI0) * (32 * 33);
    const uint32_t from = tmem + ((uint32_t)quad << 21) + half * 128;
    int b = 0, bphase = 0;
    bool ok = true;
    for (int64_t item = pair; ok && item < P.items; item += pairs) {
      float sum[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) sum[i] = 0.0f;
      for (int left = item_at(P, item).steps; left > 0; left -= CHUNK) {
        ok = wait_bar(acc_full(b), bphase, P.timeout_ns, stop);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
        for (int c = 0; c < 128; c += 16) {
          uint32_t v[16];
          tmem_load16(from + b * BN + c, v);
#pragma unroll
          for (int q = 0; q < 16; ++q) sum[c + q] = __fadd_rn(sum[c + q], __uint_as_float(v[q]));
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive_at(acc_empty(b), 0);
        if (++b == 2) b = 0, bphase ^= 1;
      }
      if (!ok) break;
      const Item it = item_at(P, item);
      const int64_t row0 = it.row0 + rank * 128 + quad * 32;
      const int rows = (int)(row0 >= P.n ? 0 : P.n - row0 < 32 ? P.n - row0 : 32);
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        __syncwarp();  // the previous block has been read
#pragma unroll
        for (int i = 0; i < 32; ++i) mine[lane * 33 + i] = sum[c + i] * P.alpha;
        __syncwarp();
        // Row by row: 32 lanes, 32 consecutive columns.
        const int64_t col = it.col0 + half * 128 + c + lane;
        if (col < P.k) store_block(P, it.slice, row0, col, mine + lane, rows);
      }
    }
  } else if (warp >= DEC0) {
    // ---------------------------------------------------------------- codes to bf16 tiles
    // A thread decodes one group of 32 codes of one token a step; a warp 8 tokens x 4 groups.  Eight neighbours, whose
    // 16-byte stores go together, hold 4 tokens x 2 groups of one slab: the swizzle puts these into 8 different places.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_DECODE));
    const int t = threadIdx.x - DEC0 * 32;
    const int token = (t >> 5) * 8 + ((t >> 4) & 1) * 4 + ((t >> 1) & 3), q = ((t >> 3) & 1) * 2 + (t & 1);
    uint32_t c[AHEAD][8];
    uint32_t E[AHEAD];
    // The loading side runs AHEAD steps before the decoding side.  Where a token or a group is beyond the end, the step 0
    // makes zeros of whatever codes the registers hold.
    int64_t litem = pair;
    int lsteps = 0, lvalid = 0;      // steps of the item, and of them this thread's, still to load
    const int8_t* code_at = nullptr;
    const uint8_t* scale_at = nullptr;
    const int64_t code_step = BK * P.pitch, scale_step = BK * (P.pitch / DP_CKPT8_GROUP);
    auto load = [&](uint32_t (&w)[8], uint32_t& e) {
      if (lsteps == 0) {
        if (litem >= P.items) return;
        const Item it = item_at(P, litem);
        litem += pairs;
        lsteps = it.steps;
        const int64_t m = it.token0 + token, col = it.col0 + rank * 128 + q * 32;
        const int64_t valid = col < P.pitch && m < P.rows ? (P.rows - m + BK - 1) / BK : 0;
        lvalid = (int)(valid < lsteps ? valid : lsteps);
        code_at = P.codes + m * P.pitch + col;
        scale_at = P.scales + m * (P.pitch / DP_CKPT8_GROUP) + col / DP_CKPT8_GROUP;
      }
      e = 0;
      if (lvalid > 0) {
        load_codes(code_at, w);
        e = __ldg(scale_at);
      }
      code_at += code_step;
      scale_at += scale_step;
      --lvalid;
      --lsteps;
    };
    int64_t total = 0;
    for (int64_t item = pair; item < P.items; item += pairs) total += item_at(P, item).steps;
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) c[u][i] = 0;
      E[u] = 0;
      load(c[u], E[u]);
    }
    // The thread's four 16-byte pieces: slab q / 2, row `token`, piece p at place p ^ (token mod 8).
    char* line = smem + A_BYTES + (q >> 1) * SLAB + token * 128;
    const uint32_t first = ((uint32_t)(q & 1) * 4 ^ (uint32_t)(token & 7)) << 4;
    int64_t citem = pair;            // (without TMA) the item and step whose dy is copied
    int ci = 0;
    uint32_t phase = 1;
    bool ok = true;
    for (int64_t done = 0; ok && done < total; done += STAGES, phase ^= 1) {
#pragma unroll
      for (int s = 0; s < STAGES; ++s) {
        if (done + s >= total) break;
        const int u = s % AHEAD;
        // A step byte is a bf16's exponent.  255, an infinity, makes NaNs of the zero codes of such a group.
        const uint32_t sb = __byte_perm(E[u] << 7, 0, 0x1010);
        const __nv_bfloat162 step = *reinterpret_cast<const __nv_bfloat162*>(&sb);
        ok = wait_bar(empty(s), phase, P.timeout_ns, stop);
        if (!ok) break;
        char* to = line + s * STAGE_BYTES;
#pragma unroll
        for (uint32_t p = 0; p < 4; ++p) {
          const uint2 lo = decode4(c[u][2 * p], step), hi = decode4(c[u][2 * p + 1], step);
          *reinterpret_cast<uint4*>(to + (first ^ (p << 4))) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
        load(c[u], E[u]);
        if (!TMA) {
          // dy's rows are not 16-byte aligned: the decoders copy its tile too, one element at a time.
          const Item it = item_at(P, citem);
          const int64_t m0 = it.token0 + (int64_t)ci * BK, n0 = it.row0 + rank * 128;
          char* stage = smem + s * STAGE_BYTES;
#pragma unroll 4
          for (int e = t; e < BK * 128; e += DEC_WARPS * 32) {
            const int tok = e >> 7, col = e & 127;
            uint16_t v = 0;
            if (m0 + tok < P.rows && n0 + col < P.n) v = P.dy[(m0 + tok) * P.lddy + n0 + col];
            *reinterpret_cast<uint16_t*>(stage + (col >> 6) * SLAB + tok * 128 + ((((col & 63) >> 3) ^ (tok & 7)) << 4) +
                                         (col & 7) * 2) = v;
          }
          if (++ci == it.steps) ci = 0, citem += pairs;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(decoded(s));
      }
    }
  }

  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  if (*stop) {
    for (int64_t item = pair; item < P.items; item += pairs) {
      const Item it = item_at(P, item);
      for (int e = threadIdx.x; e < 128 * BN; e += THREADS) {
        const int64_t row = it.row0 + rank * 128 + e / BN, col = it.col0 + e % BN;
        if (row < P.n && col < P.k) put_result(P, it.slice, row, col, __uint_as_float(0x7fc00000u));
      }
    }
  }
}

// dw (+)= the slices' products in order.
__global__ void __launch_bounds__(256) wgrad8_join_kernel(const float* part, void* dw, int64_t size, int slices, int dtype,
                                                          int accumulate) {
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < size; i += step) {
    float v = 0.0f;
#pragma unroll 4
    for (int s = 0; s < slices; ++s) v += part[s * size + i];
    grad_put(dw, i, dtype, accumulate, v);
  }
}

// ---------------------------------------------------------------------------------------------------- host side

struct Split {
  int64_t tiles_k, tiles, slices, steps;
};
// Slices of the tokens: enough items for all CTA pairs, at least 4 steps (256 tokens) each, so that a slice's fp32 product
// costs less than what it saves.
Split split_of(int64_t rows, int64_t n, int64_t k) {
  Split s;
  s.tiles_k = (k + BN - 1) / BN;
  s.tiles = (n + BM - 1) / BM * s.tiles_k;
  const int64_t all = (rows + BK - 1) / BK, pairs = 76;
  s.slices = pairs / s.tiles;
  if (s.slices > all / 4) s.slices = all / 4;
  if (s.slices > MAX_SLICES) s.slices = MAX_SLICES;
  if (s.slices < 1) s.slices = 1;
  s.steps = all ? (all + s.slices - 1) / s.slices : 0;
  if (all) s.slices = (all + s.steps - 1) / s.steps;
  return s;
}

dp_status_t check_product(int64_t rows, int64_t n, int64_t k) {
  if (rows < 0 || rows > INT32_MAX - BK) return op_fail(DP_ERR_INVALID_ARG, "rows = %lld not in 0..2^31-65", (long long)rows);
  if (n < 1 || n > (1 << 28)) return op_fail(DP_ERR_INVALID_ARG, "n = %lld not in 1..2^28", (long long)n);
  if (k < 1 || k > (1 << 28)) return op_fail(DP_ERR_INVALID_ARG, "k = %lld not in 1..2^28", (long long)k);
  return DP_OK;
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static EncodeTiled f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeTiled)p;
  }();
  return f;
}

}  // namespace
}  // namespace dp

using namespace dp;

extern "C" {

size_t dp_wgrad8_workspace_size(int64_t rows, int64_t n, int64_t k) {
  if (check_product(rows, n, k) != DP_OK) return 0;
  const Split s = split_of(rows, n, k);
  return s.slices > 1 ? (size_t)s.slices * (size_t)n * (size_t)k * 4 : 0;
}

dp_status_t dp_wgrad8(void* dw, const uint16_t* dy, const int8_t* codes, const uint8_t* scales, int64_t rows, int64_t n,
                      int64_t k, int64_t lddy, float alpha, int32_t accumulate, int32_t dtype, void* ws,
                      dp_stream_t stream_) {
  DP_TRY(check_product(rows, n, k));
  DP_TRY(check_dtype(dtype, "dtype"));
  if (accumulate != 0 && accumulate != 1) return op_fail(DP_ERR_INVALID_ARG, "accumulate = %d is neither 0 nor 1", accumulate);
  if (!(alpha > -1e30f && alpha < 1e30f)) return op_fail(DP_ERR_INVALID_ARG, "alpha must be finite");
  if (lddy < n || lddy > (int64_t(1) << 32)) return op_fail(DP_ERR_INVALID_ARG, "lddy = %lld is below n (or far too large)", (long long)lddy);
  DP_TRY(check_dev(dw, elem_size(dtype), true, "dw"));
  DP_TRY(check_dev(dy, 2, rows > 0, "dy"));
  if (rows > 0 && (!codes || !scales)) return op_fail(DP_ERR_INVALID_ARG, "codes or scales are NULL");
  if (!is_aligned(codes, 32)) return op_fail(DP_ERR_ALIGNMENT, "codes are not 32-byte aligned");
  const Split s = split_of(rows, n, k);
  DP_TRY(check_dev(ws, 256, s.slices > 1, "ws"));
  const cudaStream_t stream = (cudaStream_t)stream_;
  NvtxRange range("weight gradient");
  if (rows == 0) {
    if (accumulate) return DP_OK;
    const cudaError_t e = cudaMemsetAsync(dw, 0, (size_t)(n * k) * elem_size(dtype), stream);
    return e == cudaSuccess ? DP_OK : op_fail(DP_ERR_CUDA, "weight gradient fill: %s", cudaGetErrorString(e));
  }
  WgradParams P = {};
  P.dy = dy;
  P.codes = codes;
  P.scales = scales;
  P.dw = dw;
  P.part = s.slices > 1 ? static_cast<float*>(ws) : nullptr;
  P.rows = rows;
  P.n = n;
  P.k = k;
  P.lddy = lddy;
  P.pitch = dp_ckpt8_pitch(k);
  P.tiles_k = s.tiles_k;
  P.tiles = s.tiles;
  P.items = s.tiles * s.slices;
  P.steps = s.steps;
  P.alpha = alpha;
  P.dtype = dtype;
  P.accumulate = accumulate;
  P.timeout_ns = dp_get_wait_timeout_ns();
  // TMA wants 16-byte aligned rows; other rows are copied by the decoding warps.
  const bool tma = is_aligned(dy, 16) && lddy % 8 == 0;
  CUtensorMap map = {};
  if (tma) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return op_fail(DP_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[2] = {(cuuint64_t)n, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)lddy * 2};
    const cuuint32_t box[2] = {64, BK}, one[2] = {1, 1};
    const CUresult r = encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(dy), dims, strides, box, one,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return op_fail(DP_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", (int)r);
  }
  auto kernel = tma ? wgrad8_kernel<true> : wgrad8_kernel<false>;
  const cudaError_t attr = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (attr != cudaSuccess) return op_fail(DP_ERR_CUDA, "weight gradient: %s", cudaGetErrorString(attr));
  const int64_t pairs = sm_count() / 2;
  kernel<<<(unsigned)(2 * (P.items < pairs ? P.items : pairs)), THREADS, SMEM, stream>>>(P, map);
  if (!P.part) return op_launched("weight gradient launch", 1);
  const int64_t size = n * k, ctas = (size + 1023) / 1024, most = (int64_t)sm_count() * 8;
  wgrad8_join_kernel<<<(unsigned)(ctas < most ? ctas : most), 256, 0, stream>>>(P.part, dw, size, (int)s.slices, dtype,
                                                                               accumulate);
  return op_launched("weight gradient launch", 2);
}

}  // extern "C"
