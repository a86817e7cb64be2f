// The norms around a block, fused with its gate and residual scale, and their gradient.
//
//   r = a x + b g N_post(y),   z = N_pre(r),   N(v) = (v - mean) rstd w + c
//
// Apart, these are two norms, a product and a scaled sum: x, y, r and the post norm's output go through memory several
// times.  Here a row stays in registers from y to z: x and y are read once, r and z written once (four row passes
// forward; six backward: dr, dz, r, y in, dx, dy out).  What bounds both is memory.
//
// A row is held by a group of threads, eight consecutive elements each, NV such pieces a thread.  A group is one warp for short rows, else the whole CTA; CTAs are
// persistent, so parameters are read once per CTA and held in registers, and the next rows are on their way to shared memory
// while a row is summed (three rows ahead at 4096 columns: 96 KB in flight an SM).  Mean and variance are taken in two passes over the registers: no cancellation.
//
// Gradient, with yh, rh the rows before weights and biases, D = dr + N_pre'(dz) and q = g D for a gate per token, else D:
//   v  = w_pre dz:      D  = dr + rstd_pre (v - rh mean(v rh) - mean(v))          (RMS: without mean(v))
//   v' = b g w_post D:  dy = rstd_post (v' - yh mean(v' yh) - mean(v')),   dx = a D
//   P1 = sum dz rh, P0 = sum dz, S1 = sum q yh, S0 = sum q   over the rows, for each column
//   dw_pre = P1, db_pre = P0, dw_post = b g S1, db_post = b g S0, dgate = b (w_post S1 + c_post S0) for a gate per
//   channel; for one per token, dgate = b (sum over the row of D (w_post yh + c_post)).
// So all five parameter gradients come from four column sums (two for RMS norms without biases), kept in registers over
// the rows of a CTA, left in the workspace as one partial row a CTA, and added in CTA order by a second kernel.
#include <math.h>

#include <initializer_list>

#include "op_common.cuh"

namespace dp {
namespace {

constexpr int NORM_THREADS = 512;   // most threads of a group
constexpr int MAX_PARTS = 1024;     // most CTAs (partial rows) of the gradient
constexpr int FIN_COLS = 16, FIN_ROWS = 64;
constexpr int MAX_SLOTS = 4;

struct NormParams {
  void *r, *z, *dx, *dy, *dgate_token;
  const void *x, *y, *dr, *dz;
  const void *w_post, *b_post, *gate, *w_pre, *b_pre;
  float2 *post_stats, *pre_stats;
  float* part;
  int64_t rows;
  int dim, group, per_cta, slots;  // threads of a row, rows of a CTA at a time, rows in flight
  int layer, post, pre, gate_mode, pdt, accumulate, bias;
  float eps, a, b;
};

// The element numbers of a thread: k-th of eight of piece j.
__device__ __forceinline__ int col_of(int tid, int group, int j, int k) { return (tid + j * group) * 8 + k; }
// A row's pieces in a thread's registers.  Rows whose pieces are 16-byte words (VEC) pass through shared memory, P.slots - 1 rows
// ahead.  A slot is an image of the row, and a warp copies just the part that its own threads read: no barrier wider than
// the warp is needed.
template <typename T, int VEC, int NV>
struct RowRegs {
  static constexpr int WORDS = sizeof(T) / 2;  // 16-byte words of eight elements
  Raw8<T> w[NV];
  static __device__ __forceinline__ int bytes(int group) { return NV * group * 16 * WORDS; }
  static __device__ __forceinline__ void fetch(char* slot, const T* row, int tid, int group, int dim) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int q = 0; q < WORDS; ++q) {  // neighbours copy neighbouring words
        const int at = (j * group + (tid & ~31)) * 16 * WORDS + q * 512 + (tid & 31) * 16;
        if (at < dim * (int)sizeof(T))
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(slot + at)),
                       "l"(reinterpret_cast<const char*>(row) + at)
                       : "memory");
      }
    }
  }
  // From the slot, or (not VEC) from the row itself, in [lo, hi); what lies beyond dim is zero.
  __device__ __forceinline__ void load(const char* slot, const T* lo, int64_t at, const T* hi, int tid, int group, int dim) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (VEC) {
        if (col_of(tid, group, j, 0) < dim) {
          uint4* to = reinterpret_cast<uint4*>(&w[j]);
#pragma unroll
          for (int q = 0; q < WORDS; ++q) to[q] = *reinterpret_cast<const uint4*>(slot + ((j * group + tid) * WORDS + q) * 16);
        } else {
          w[j].pack(v);
        }
      } else {
        const int c = col_of(tid, group, j, 0);
        w[j] = load_any8(lo + at + c, there8(c, dim), lo, hi);
      }
    }
  }
};
__device__ __forceinline__ void fetched() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until all but the last `rows` fetched rows are there.
__device__ __forceinline__ void fetch_wait(int rows) {
  if (rows == 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (rows == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (rows == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
}

template <typename T, int VEC, int NV>
__device__ __forceinline__ void store_row2(T* row, int tid, int group, int dim, const f2_t (&v)[NV][4]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = col_of(tid, group, j, 0);
    Raw8<T> o;
    o.pack2(v[j]);
    if (!VEC) store_any8(row + c, there8(c, dim), o);
    else if (c < dim) store_raw8(row + c, o);
  }
}

template <int VEC, int NV>
__device__ __forceinline__ void load_param(const void* p, int dtype, float none, int tid, int group, int dim,
                                           float (&v)[NV][8]) {
  if (VEC && p && ((uintptr_t)p & 15) == 0) {  // whole pieces as 16-byte words
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = col_of(tid, group, j, 0);
      if (c >= dim) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] = 0.0f;
      } else if (dtype == DP_BF16) {
        load_raw8(static_cast<const bf16_t*>(p) + c).unpack(v[j]);
      } else {
        load_raw8(static_cast<const float*>(p) + c).unpack(v[j]);
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = col_of(tid, group, j, k);
      v[j][k] = c < dim ? param_at(p, c, dtype, none) : 0.0f;
    }
}

// Sums of N values over a group of threads; every thread gets them.  A CTA-wide group alternates between two halves of
// `buf` (zero beyond the group's warps), so one barrier a call is enough: a half is written again only after the barrier
// of the call in between.  The warps' sums are read as broadcast words, which takes less than another five shuffles.
typedef float GroupBuf[2][3][16];
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int warps, GroupBuf& buf, int& half) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (warps == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[half][i][warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float4* p = reinterpret_cast<const float4*>(buf[half][i]);
    const float4 a = p[0], b = p[1], c = p[2], d = p[3];
    v[i] = (((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w))) + (((c.x + c.y) + (c.z + c.w)) + ((d.x + d.y) + (d.z + d.w)));
  }
  half ^= 1;
}
__device__ __forceinline__ void clear(GroupBuf& buf) {
  for (int i = threadIdx.x; i < 96; i += blockDim.x) (&buf[0][0][0])[i] = 0.0f;
  __syncthreads();
}

// Mean (0 for RMS) and 1 / sqrt(var + eps) of a row held in registers, which is centred on the way.  Pieces beyond dim hold
// zeros, before and after.
template <int VEC, int NV, bool LAYER>
__device__ __forceinline__ float2 row_stats(f2_t (&v)[NV][4], float eps, float inv, int tid, int group, int dim, GroupBuf& buf,
                                            int& half) {
  float s[1], mean = 0.0f;
  f2_t sum = f2_both(0.0f);
  if (LAYER) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) sum = f2_add(sum, v[j][k]);
    s[0] = f2_sum(sum);
    group_sum<1>(s, group >> 5, buf, half);
    mean = s[0] * inv;
    const f2_t less = f2_both(-mean);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (VEC) {
          if (col_of(tid, group, j, 0) < dim) v[j][k] = f2_add(v[j][k], less);
        } else {
          float a, b;
          f2_unpack(v[j][k], a, b);
          v[j][k] = f2_pack(col_of(tid, group, j, 2 * k) < dim ? a - mean : 0.0f,
                            col_of(tid, group, j, 2 * k + 1) < dim ? b - mean : 0.0f);
        }
      }
    sum = f2_both(0.0f);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) sum = f2_fma(v[j][k], v[j][k], sum);
  s[0] = f2_sum(sum);
  group_sum<1>(s, group >> 5, buf, half);
  return make_float2(mean, 1.0f / sqrtf(fmaf(s[0], inv, eps)));
}

// Which row a group of threads starts with, and the step between its rows.
__device__ __forceinline__ int64_t first_row(const NormParams& P, int& tid) {
  if (P.per_cta == 1) {
    tid = threadIdx.x;
    return blockIdx.x;
  }
  tid = threadIdx.x & 31;
  return (int64_t)blockIdx.x * P.per_cta + (threadIdx.x >> 5);
}

// LAYER: rows are centred.  BIAS: some norm has a bias.
template <typename TS, typename TB, int VEC, int NV, bool LAYER, bool BIAS>
__global__ void __launch_bounds__(NORM_THREADS, NV == 1 && !BIAS ? 2 : 1) norm_kernel(const __grid_constant__ NormParams P) {
  extern __shared__ char slots[];
  __shared__ __align__(16) GroupBuf buf;
  clear(buf);
  typedef RowRegs<TS, VEC, NV> RowS;
  typedef RowRegs<TB, VEC, NV> RowB;
  int half = 0, tid;
  const int64_t row0 = first_row(P, tid), step = (int64_t)gridDim.x * P.per_cta;
  const int group = P.group, dim = P.dim;
  const int at_x = RowB::bytes(group), slot_bytes = at_x + RowS::bytes(group);
  char* mine = slots + (P.per_cta == 1 ? 0 : (threadIdx.x >> 5) * P.slots * slot_bytes);
  auto fetch = [&](int64_t row, int slot) {
    if (VEC) __syncwarp();  // the slot's last row has been read
    if (VEC && row < P.rows) {
      char* to = mine + slot * slot_bytes;
      if (P.y) RowB::fetch(to, static_cast<const TB*>(P.y) + row * dim, tid, group, dim);
      RowS::fetch(to + at_x, static_cast<const TS*>(P.x) + row * dim, tid, group, dim);
    }
    if (VEC) fetched();
  };
  for (int s = 0; s + 1 < P.slots; ++s) fetch(row0 + s * step, s);
  int slot = 0;
  const bool token = P.gate_mode == DP_GATE_TOKEN;
  f2_t A[NV][4], B[NV][4], wp[NV][4], bp[NV][4];  // b g w_post, b g b_post, w_pre, b_pre
  {
    float g[NV][8], w[NV][8];
    auto pairs = [&](f2_t (&to)[NV][4], bool scaled) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          to[j][k] = scaled ? f2_pack(w[j][2 * k] * g[j][2 * k], w[j][2 * k + 1] * g[j][2 * k + 1]) : f2_pack(w[j][2 * k], w[j][2 * k + 1]);
    };
    load_param<VEC, NV>(P.gate_mode == DP_GATE_CHANNEL ? P.gate : nullptr, P.pdt, 1.0f, tid, group, dim, g);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) g[j][k] *= P.b;
    load_param<VEC, NV>(P.w_post, P.pdt, 1.0f, tid, group, dim, w);
    pairs(A, true);
    load_param<VEC, NV>(P.w_pre, P.pdt, 1.0f, tid, group, dim, w);
    pairs(wp, false);
    if (BIAS) {
      load_param<VEC, NV>(P.b_post, P.pdt, 0.0f, tid, group, dim, w);
      pairs(B, true);
      load_param<VEC, NV>(P.b_pre, P.pdt, 0.0f, tid, group, dim, w);
      pairs(bp, false);
    }
  }
  const float inv = 1.0f / (float)dim;
  uint32_t next_gate = P.pdt == DP_BF16 ? 0x3f80u : 0x3f800000u;  // as it lies in memory: a conversion would wait for it
  auto scalars = [&](int64_t row) {
    if (token && row < P.rows)
      next_gate = P.pdt == DP_BF16 ? __ldg(static_cast<const uint16_t*>(P.gate) + row) : __ldg(static_cast<const uint32_t*>(P.gate) + row);
  };
  scalars(row0);

  for (int64_t row = row0; row < P.rows; row += step) {
    fetch(row + (P.slots - 1) * step, slot == 0 ? P.slots - 1 : slot - 1);
    const float gt = __uint_as_float(P.pdt == DP_BF16 ? next_gate << 16 : next_gate);
    scalars(row + step);
    if (VEC) fetch_wait(P.slots - 1);
    const char* here = mine + slot * slot_bytes;
    if (++slot == P.slots) slot = 0;
    f2_t r[NV][4];
    {
      RowS xr;
      xr.load(here + at_x, static_cast<const TS*>(P.x), row * dim, static_cast<const TS*>(P.x) + P.rows * dim, tid, group, dim);
#pragma unroll
      for (int j = 0; j < NV; ++j) xr.w[j].unpack2(r[j]);
    }
    if (P.y) {
      RowB yr;
      yr.load(here, static_cast<const TB*>(P.y), row * dim, static_cast<const TB*>(P.y) + P.rows * dim, tid, group, dim);
      f2_t v[NV][4];
#pragma unroll
      for (int j = 0; j < NV; ++j) yr.w[j].unpack2(v[j]);
      float2 st = make_float2(0.0f, 1.0f);
      if (P.post) {
        st = row_stats<VEC, NV, LAYER>(v, P.eps, inv, tid, group, dim, buf, half);
        if (P.post_stats && tid == 0) P.post_stats[row] = st;
      }
      const f2_t a = f2_both(P.a), rstd = f2_both(st.y), gate = f2_both(gt);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f2_t ax = f2_mul(a, r[j][k]), n = f2_mul(v[j][k], A[j][k]);
          r[j][k] = f2_fma(BIAS ? f2_fma(n, rstd, B[j][k]) : f2_mul(n, rstd), gate, ax);
        }
      store_row2<TS, VEC, NV>(static_cast<TS*>(P.r) + row * dim, tid, group, dim, r);
    }
    if (P.pre) {
      const float2 st = row_stats<VEC, NV, LAYER>(r, P.eps, inv, tid, group, dim, buf, half);
      if (P.pre_stats && tid == 0) P.pre_stats[row] = st;
      const f2_t rstd = f2_both(st.y);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f2_t n = f2_mul(r[j][k], wp[j][k]);
          r[j][k] = BIAS ? f2_fma(n, rstd, bp[j][k]) : f2_mul(n, rstd);
        }
      store_row2<TB, VEC, NV>(static_cast<TB*>(P.z) + row * dim, tid, group, dim, r);
    }
  }
}

// LAYER: rows are centred.  SUM0: some gradient needs S0 or P0 (a bias is there).  The workspace holds, for each group of
// threads, S1 and P1 and (SUM0) S0 and P0, dim floats each.
template <typename TS, typename TB, int VEC, int NV, bool LAYER, bool SUM0>
__global__ void __launch_bounds__(NORM_THREADS) norm_grad_kernel(const __grid_constant__ NormParams P) {
  extern __shared__ char slots[];
  __shared__ __align__(16) GroupBuf buf;
  clear(buf);
  typedef RowRegs<TS, VEC, NV> RowS;
  typedef RowRegs<TB, VEC, NV> RowB;
  int half = 0, tid;
  const int64_t row0 = first_row(P, tid), step = (int64_t)gridDim.x * P.per_cta;
  const int group = P.group, dim = P.dim;
  const int at_dz = RowB::bytes(group), at_r = 2 * at_dz, at_dr = at_r + RowS::bytes(group);
  const int slot_bytes = at_dr + RowS::bytes(group);
  char* mine = slots + (P.per_cta == 1 ? 0 : (threadIdx.x >> 5) * P.slots * slot_bytes);
  auto fetch = [&](int64_t row, int slot) {
    if (VEC) __syncwarp();  // the slot's last row has been read
    if (VEC && row < P.rows) {
      char* to = mine + slot * slot_bytes;
      if (P.y) RowB::fetch(to, static_cast<const TB*>(P.y) + row * dim, tid, group, dim);
      if (P.pre) {
        RowB::fetch(to + at_dz, static_cast<const TB*>(P.dz) + row * dim, tid, group, dim);
        RowS::fetch(to + at_r, static_cast<const TS*>(P.x) + row * dim, tid, group, dim);
      }
      if (P.dr) RowS::fetch(to + at_dr, static_cast<const TS*>(P.dr) + row * dim, tid, group, dim);
    }
    if (VEC) fetched();
  };
  grid_go();
  for (int s = 0; s + 1 < P.slots; ++s) fetch(row0 + s * step, s);
  int slot = 0;
  // For the gradient of a gate per token: the post norm's bias, read for every row.
  float* bias = reinterpret_cast<float*>(slots + (VEC ? P.per_cta * P.slots * slot_bytes : 0));
  if (P.bias) {
    for (int c = threadIdx.x; c < dim; c += blockDim.x) bias[c] = param_at(P.b_post, c, P.pdt, 0.0f);
    __syncthreads();
  }
  const bool has_y = P.y != nullptr, token = P.gate_mode == DP_GATE_TOKEN;
  f2_t A[NV][4], wp[NV][4];  // b g w_post, w_pre
  f2_t S1[NV][4], P1[NV][4], S0[NV][4], P0[NV][4];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) A[j][k] = wp[j][k] = S1[j][k] = P1[j][k] = S0[j][k] = P0[j][k] = f2_both(0.0f);
  {
    float v[NV][8];
    if (has_y) {
      load_param<VEC, NV>(P.w_post, P.pdt, 1.0f, tid, group, dim, v);
      float g[NV][8];
      load_param<VEC, NV>(P.gate_mode == DP_GATE_CHANNEL ? P.gate : nullptr, P.pdt, 1.0f, tid, group, dim, g);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[j][k] *= P.b * g[j][k];
          if (k & 1) A[j][k >> 1] = f2_pack(v[j][k - 1], v[j][k]);
        }
    }
    if (P.pre) {
      load_param<VEC, NV>(P.w_pre, P.pdt, 1.0f, tid, group, dim, v);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) wp[j][k] = f2_pack(v[j][2 * k], v[j][2 * k + 1]);
    }
  }
  const float inv = 1.0f / (float)dim;
  // The next row's statistics are loaded a row ahead, like its elements.
  float2 next_pre = make_float2(0.0f, 1.0f), next_post = make_float2(0.0f, 1.0f);
  uint32_t next_gate = P.pdt == DP_BF16 ? 0x3f80u : 0x3f800000u;  // as it lies in memory: a conversion would wait for it
  auto scalars = [&](int64_t row) {
    if (row >= P.rows) return;
    if (P.pre) next_pre = P.pre_stats[row];
    if (P.post) next_post = P.post_stats[row];
    if (token) next_gate = P.pdt == DP_BF16 ? __ldg(static_cast<const uint16_t*>(P.gate) + row) : __ldg(static_cast<const uint32_t*>(P.gate) + row);
  };
  scalars(row0);

  for (int64_t row = row0; row < P.rows; row += step) {
    fetch(row + (P.slots - 1) * step, slot == 0 ? P.slots - 1 : slot - 1);
    const float2 pre = next_pre, post = next_post;
    const float gt = __uint_as_float(P.pdt == DP_BF16 ? next_gate << 16 : next_gate);
    scalars(row + step);
    if (VEC) fetch_wait(P.slots - 1);
    const char* here = mine + slot * slot_bytes;
    if (++slot == P.slots) slot = 0;
    f2_t D[NV][4];
    RowB yr;
    if (has_y && !VEC) yr.load(here, static_cast<const TB*>(P.y), row * dim, static_cast<const TB*>(P.y) + P.rows * dim, tid, group, dim);
    if (P.dr) {
      RowS w;
      w.load(here + at_dr, static_cast<const TS*>(P.dr), row * dim, static_cast<const TS*>(P.dr) + P.rows * dim, tid, group, dim);
#pragma unroll
      for (int j = 0; j < NV; ++j) w.w[j].unpack2(D[j]);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) D[j][k] = f2_both(0.0f);
    }
    if (P.pre) {
      RowB zr;
      RowS rr;
      zr.load(here + at_dz, static_cast<const TB*>(P.dz), row * dim, static_cast<const TB*>(P.dz) + P.rows * dim, tid, group, dim);
      rr.load(here + at_r, static_cast<const TS*>(P.x), row * dim, static_cast<const TS*>(P.x) + P.rows * dim, tid, group, dim);
      const f2_t less = f2_both(-pre.x), rstd = f2_both(pre.y);
      f2_t v[NV][4], h[NV][4], s1 = f2_both(0.0f), s0 = f2_both(0.0f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        zr.w[j].unpack2(v[j]);
        rr.w[j].unpack2(h[j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (LAYER) h[j][k] = f2_add(h[j][k], less);
          h[j][k] = f2_mul(h[j][k], rstd);
          P1[j][k] = f2_fma(v[j][k], h[j][k], P1[j][k]);
          if (SUM0) P0[j][k] = f2_add(P0[j][k], v[j][k]);
          v[j][k] = f2_mul(v[j][k], wp[j][k]);  // zero beyond dim
          s1 = f2_fma(v[j][k], h[j][k], s1);
          if (LAYER) s0 = f2_add(s0, v[j][k]);
        }
      }
      float s[LAYER ? 2 : 1] = {f2_sum(s1)};
      if (LAYER) s[LAYER ? 1 : 0] = f2_sum(s0);
      group_sum<LAYER ? 2 : 1>(s, group >> 5, buf, half);
      const f2_t c1 = f2_both(-s[0] * inv), c0 = f2_both(LAYER ? -s[LAYER ? 1 : 0] * inv : 0.0f);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f2_t x = f2_fma(h[j][k], c1, v[j][k]);
          if (LAYER) x = f2_add(x, c0);
          D[j][k] = f2_fma(x, rstd, D[j][k]);
        }
    }
    if (has_y) {
      if (VEC) yr.load(here, static_cast<const TB*>(P.y), row * dim, static_cast<const TB*>(P.y) + P.rows * dim, tid, group, dim);
      const f2_t less = f2_both(-post.x), rstd = f2_both(post.y), gate = f2_both(gt);
      f2_t v[NV][4], h[NV][4], s1 = f2_both(0.0f), s0 = f2_both(0.0f);
      float s2 = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        yr.w[j].unpack2(h[j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (LAYER) h[j][k] = f2_add(h[j][k], less);
          h[j][k] = f2_mul(h[j][k], rstd);
          const f2_t q = f2_mul(gate, D[j][k]);
          v[j][k] = f2_mul(A[j][k], D[j][k]);
          S1[j][k] = f2_fma(q, h[j][k], S1[j][k]);
          if (SUM0) S0[j][k] = f2_add(S0[j][k], q);
          s1 = f2_fma(v[j][k], h[j][k], s1);
          if (LAYER) s0 = f2_add(s0, v[j][k]);
        }
      }
      if (P.bias) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int c = col_of(tid, group, j, k);
            float d[2];
            f2_unpack(D[j][k >> 1], d[0], d[1]);
            if (c < dim) s2 = fmaf(d[k & 1], bias[c], s2);
          }
      }
      float c1 = f2_sum(s1), c0 = LAYER ? f2_sum(s0) : 0.0f;
      if (token) {
        float s[3] = {c1, c0, s2};
        group_sum<3>(s, group >> 5, buf, half);
        c1 = s[0];
        c0 = s[1];
        if (P.dgate_token && tid == 0) grad_put(P.dgate_token, row, P.pdt, P.accumulate, fmaf(P.b, s[2], s[0]));
      } else if (P.post) {
        float s[LAYER ? 2 : 1] = {c1};
        if (LAYER) s[LAYER ? 1 : 0] = c0;
        group_sum<LAYER ? 2 : 1>(s, group >> 5, buf, half);
        c1 = s[0];
        if (LAYER) c0 = s[LAYER ? 1 : 0];
      }
      const f2_t m1 = f2_both(P.post ? -c1 * inv : 0.0f), m0 = f2_both(P.post ? -c0 * inv : 0.0f), f = f2_both(gt * post.y);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f2_t x = f2_fma(h[j][k], m1, v[j][k]);
          if (LAYER) x = f2_add(x, m0);
          h[j][k] = f2_mul(x, f);
        }
      store_row2<TB, VEC, NV>(static_cast<TB*>(P.dy) + row * dim, tid, group, dim, h);
    }
    const f2_t a = f2_both(P.a);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) D[j][k] = f2_mul(D[j][k], a);
    store_row2<TS, VEC, NV>(static_cast<TS*>(P.dx) + row * dim, tid, group, dim, D);
  }
  // One partial row a group of threads.
  const int64_t part = (int64_t)blockIdx.x * P.per_cta + (P.per_cta == 1 ? 0 : threadIdx.x >> 5);
  auto leave = [&](int which, const f2_t (&sum)[NV][4]) {
    float* p = P.part + (part * (SUM0 ? 4 : 2) + which) * dim;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = col_of(tid, group, j, k);
        float x[2];
        f2_unpack(sum[j][k >> 1], x[0], x[1]);
        if (c < dim) p[c] = x[k & 1];
      }
  };
  leave(0, S1);
  leave(1, P1);
  if (SUM0) {
    leave(2, S0);
    leave(3, P0);
  }
}

struct FinishParams {
  const float* part;
  int64_t parts;
  int dim, sum0, gate_mode, pdt, accumulate;
  const void *w_post, *b_post, *gate;
  void *dw_post, *db_post, *dgate, *dw_pre, *db_pre;
  float b;
};

// Adds the partial rows of 16 columns: 64 threads a column take the parts in turn, then a warp adds the 64 in a fixed order.
__global__ void __launch_bounds__(FIN_COLS* FIN_ROWS) norm_finish_kernel(const __grid_constant__ FinishParams P) {
  __shared__ float sums[4 * FIN_COLS][FIN_ROWS + 1];
  __shared__ float done[4 * FIN_COLS];
  grid_wait();
  const int c0 = blockIdx.x * FIN_COLS + threadIdx.x;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c0 < P.dim) {
#pragma unroll 5
    for (int64_t i = threadIdx.y; i < P.parts; i += FIN_ROWS) {
      const float* p = P.part + i * (P.sum0 ? 4 : 2) * P.dim + c0;
      s[0] += p[0];
      s[1] += p[P.dim];
      if (P.sum0) {
        s[2] += p[2 * (int64_t)P.dim];
        s[3] += p[3 * (int64_t)P.dim];
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) sums[q * FIN_COLS + threadIdx.x][threadIdx.y] = s[q];
  __syncthreads();
  const int t = threadIdx.y * FIN_COLS + threadIdx.x, lane = t & 31;
  for (int i = t >> 5; i < 4 * FIN_COLS; i += FIN_COLS * FIN_ROWS / 32) {
    float v = sums[i][lane] + sums[i][lane + 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) done[i] = v;
  }
  __syncthreads();
  const int c = blockIdx.x * FIN_COLS + t;
  if (t >= FIN_COLS || c >= P.dim) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) s[q] = done[q * FIN_COLS + t];
  const float g = P.b * (P.gate_mode == DP_GATE_CHANNEL ? param_at(P.gate, c, P.pdt, 1.0f) : 1.0f);
  if (P.dw_post) grad_put(P.dw_post, c, P.pdt, P.accumulate, g * s[0]);
  if (P.db_post) grad_put(P.db_post, c, P.pdt, P.accumulate, g * s[2]);
  if (P.dgate)
    grad_put(P.dgate, c, P.pdt, P.accumulate,
             P.b * fmaf(param_at(P.w_post, c, P.pdt, 1.0f), s[0], param_at(P.b_post, c, P.pdt, 0.0f) * s[2]));
  if (P.dw_pre) grad_put(P.dw_pre, c, P.pdt, P.accumulate, s[1]);
  if (P.db_pre) grad_put(P.db_pre, c, P.pdt, P.accumulate, s[3]);
}

// ---------------------------------------------------------------------------------------------------- host side

// Pieces of eight a thread holds: one up to 4096 columns, so that a row has as many threads as it can use.
int pieces_of(int dim) { return dim <= NORM_THREADS * 8 ? 1 : dim <= NORM_THREADS * 16 ? 2 : 4; }

struct Shape {
  int nv, group, per_cta, threads;
};
Shape shape_of(int dim) {
  Shape s;
  s.nv = pieces_of(dim);
  s.group = (dim + s.nv * 8 * 32 - 1) / (s.nv * 8 * 32) * 32;
  s.per_cta = s.group == 32 ? 4 : 1;
  s.threads = s.group * s.per_cta;
  return s;
}

// Rows in flight, and with that the shared memory, of a kernel whose CTAs take `set` bytes a row: four where all CTAs that the
// registers allow an SM still fit, fewer for long rows.  A kernel's last answer is kept: asking takes longer than a launch.
struct Plan1 {
  int device = -1, threads = 0, slots = 1, ctas = 0;  // ctas: one wave
  int64_t set = -1, more = -1;
};
template <typename K>
void plan_of(K kernel, int threads, int64_t set, int64_t more, Plan1& c) {
  int device = 0;
  cudaGetDevice(&device);
  if (c.device == device && c.threads == threads && c.set == set && c.more == more) return;
  c.slots = 1;
  int per_sm = 1;
  if (set > 0) {
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, 0);
    const int64_t room = 220 * 1024;
    if (per_sm < 1) per_sm = 1;
    while (per_sm > 1 && per_sm * (set * 2 + more) > room) --per_sm;
    const int64_t n = (room / per_sm - more) / set;
    c.slots = (int)(n < 1 ? 1 : n > MAX_SLOTS ? MAX_SLOTS : n);
  }
  const size_t smem = (size_t)(c.slots * set + more);
  cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  c.ctas = occupancy_grid(kernel, threads, smem, INT32_MAX);
  c.device = device;
  c.threads = threads;
  c.set = set;
  c.more = more;
}
template <typename K>
int launch_rows(K kernel, Plan1& c, const Shape& s, NormParams& P, int64_t set, int64_t more, int most, cudaStream_t stream) {
  plan_of(kernel, s.threads, set, more, c);
  P.slots = c.slots;
  const int64_t want = (P.rows + s.per_cta - 1) / s.per_cta;
  int64_t grid = want < c.ctas ? want : c.ctas;
  if (grid > most) grid = most;
  kernel<<<(unsigned)grid, s.threads, (size_t)(c.slots * set + more), stream>>>(P);
  return (int)grid;
}

template <typename TS, typename TB, int VEC, int NV>
void run_forward(NormParams P, const Shape& s, cudaStream_t stream) {
  static thread_local Plan1 plan[4];
  const bool bias = P.b_post || P.b_pre;
  auto k = P.layer ? (bias ? norm_kernel<TS, TB, VEC, NV, true, true> : norm_kernel<TS, TB, VEC, NV, true, false>)
                   : (bias ? norm_kernel<TS, TB, VEC, NV, false, true> : norm_kernel<TS, TB, VEC, NV, false, false>);
  launch_rows(k, plan[2 * P.layer + bias], s, P, VEC ? (int64_t)s.threads * NV * 8 * (sizeof(TS) + sizeof(TB)) : 0, 0, INT32_MAX, stream);
}
template <typename TS, typename TB, int VEC, int NV>
int run_grad(NormParams P, const Shape& s, bool sum0, cudaStream_t stream) {
  static thread_local Plan1 plan[3];
  const int which = P.layer ? 2 : sum0 ? 1 : 0;
  auto k = P.layer ? norm_grad_kernel<TS, TB, VEC, NV, true, true>
           : sum0  ? norm_grad_kernel<TS, TB, VEC, NV, false, true>
                   : norm_grad_kernel<TS, TB, VEC, NV, false, false>;
  return s.per_cta * launch_rows(k, plan[which], s, P, VEC ? (int64_t)s.threads * NV * 8 * 2 * (sizeof(TS) + sizeof(TB)) : 0,
                                 P.bias ? P.dim * 4 : 0, MAX_PARTS / s.per_cta, stream);
}

// f(stream type, block type, VEC, NV) for the sizes and types of one call.
template <typename F>
auto dispatch(const dp_block_norm_t& p, bool vec, int nv, F&& f) {
#define DP_NV(TS, TB, V) \
  (nv == 1 ? f.template operator()<TS, TB, V, 1>() : nv == 2 ? f.template operator()<TS, TB, V, 2>() \
                                                             : f.template operator()<TS, TB, V, 4>())
#define DP_VEC(TS, TB) (vec ? DP_NV(TS, TB, 1) : DP_NV(TS, TB, 0))
  if (p.stream_dtype == DP_BF16) return DP_VEC(bf16_t, bf16_t);
  if (p.block_dtype == DP_BF16) return DP_VEC(float, bf16_t);
  return DP_VEC(float, float);
#undef DP_VEC
#undef DP_NV
}

struct Forward {
  const NormParams& P;
  const Shape& s;
  cudaStream_t stream;
  template <typename TS, typename TB, int VEC, int NV>
  int operator()() const {
    run_forward<TS, TB, VEC, NV>(P, s, stream);
    return 0;
  }
};
struct Gradient {
  const NormParams& P;
  const Shape& s;
  bool sum0;
  cudaStream_t stream;
  template <typename TS, typename TB, int VEC, int NV>
  int operator()() const {
    return run_grad<TS, TB, VEC, NV>(P, s, sum0, stream);
  }
};

dp_status_t check_norm(const dp_block_norm_t* p, bool has_y, bool gate) {
  if (!p) return op_fail(DP_ERR_INVALID_ARG, "p is NULL");
  if (p->rows < 0 || p->rows > INT32_MAX) return op_fail(DP_ERR_INVALID_ARG, "rows = %lld not in 0..2^31-1", (long long)p->rows);
  if (p->dim < 1 || p->dim > DP_MAX_NORM_DIM) return op_fail(DP_ERR_INVALID_ARG, "dim = %d not in 1..%d", p->dim, DP_MAX_NORM_DIM);
  if (p->kind != DP_NORM_RMS && p->kind != DP_NORM_LAYER) return op_fail(DP_ERR_INVALID_ARG, "kind = %d unknown", p->kind);
  if (p->norms & ~(DP_NORM_POST | DP_NORM_PRE)) return op_fail(DP_ERR_INVALID_ARG, "norms = %d unknown", p->norms);
  if (p->gate_mode < DP_GATE_NONE || p->gate_mode > DP_GATE_TOKEN) return op_fail(DP_ERR_INVALID_ARG, "gate_mode = %d unknown", p->gate_mode);
  DP_TRY(check_dtype(p->stream_dtype, "stream_dtype"));
  DP_TRY(check_dtype(p->block_dtype, "block_dtype"));
  DP_TRY(check_dtype(p->param_dtype, "param_dtype"));
  if (p->stream_dtype == DP_BF16 && p->block_dtype == DP_F32)
    return op_fail(DP_ERR_INVALID_ARG, "fp32 block tensors need an fp32 stream");
  if (p->accumulate != 0 && p->accumulate != 1) return op_fail(DP_ERR_INVALID_ARG, "accumulate = %d is neither 0 nor 1", p->accumulate);
  if (!(p->eps > 0.0f) || !(p->eps < 1e30f)) return op_fail(DP_ERR_INVALID_ARG, "eps must be finite and > 0");
  if (!(fabsf(p->res_scale) < 1e30f) || !(fabsf(p->branch_scale) < 1e30f))
    return op_fail(DP_ERR_INVALID_ARG, "res_scale and branch_scale must be finite");
  if (p->rows == 0) return DP_OK;  // empty tensors have no address: nothing says which of them are there
  if ((p->gate_mode != DP_GATE_NONE) != gate)
    return op_fail(DP_ERR_INVALID_ARG, "gate and gate_mode disagree");
  if (!has_y && (p->norms & DP_NORM_POST || gate || p->res_scale != 1.0f))
    return op_fail(DP_ERR_INVALID_ARG, "without y there is no post norm, no gate and res_scale is 1");
  if (!has_y && !(p->norms & DP_NORM_PRE)) return op_fail(DP_ERR_INVALID_ARG, "neither a block output nor a norm before the next block");
  return DP_OK;
}

NormParams base_params(const dp_block_norm_t& p, const Shape& s) {
  NormParams P = {};
  P.rows = p.rows;
  P.dim = p.dim;
  P.group = s.group;
  P.per_cta = s.per_cta;
  P.layer = p.kind == DP_NORM_LAYER;
  P.post = (p.norms & DP_NORM_POST) != 0;
  P.pre = (p.norms & DP_NORM_PRE) != 0;
  P.gate_mode = p.gate_mode;
  P.pdt = p.param_dtype;
  P.accumulate = p.accumulate;
  P.eps = p.eps;
  P.a = p.res_scale;
  P.b = p.branch_scale;
  return P;
}

// Whether one row of a CTA fits its shared memory (`pairs` rows of the stream and of the block).
bool slots_fit(const dp_block_norm_t& p, const Shape& s, int pairs) {
  return (int64_t)s.threads * s.nv * 8 * pairs * (elem_size(p.stream_dtype) + elem_size(p.block_dtype)) + 4 * p.dim <= 220 * 1024;
}

bool all16(std::initializer_list<const void*> ps) {
  for (const void* q : ps)
    if (!is_aligned(q, 16)) return false;
  return true;
}

}  // namespace
}  // namespace dp

using namespace dp;

extern "C" {

dp_status_t dp_block_norm(const dp_block_norm_t* p, void* r, void* z, const void* x, const void* y,
                          const void* w_post, const void* b_post, const void* gate, const void* w_pre,
                          const void* b_pre, float* post_stats, float* pre_stats, dp_stream_t stream) {
  DP_TRY(check_norm(p, y != nullptr, gate != nullptr));
  const bool some = p->rows > 0, pre = (p->norms & DP_NORM_PRE) != 0;
  const int es = elem_size(p->stream_dtype), eb = elem_size(p->block_dtype), ep = elem_size(p->param_dtype);
  DP_TRY(check_dev(x, es, some, "x"));
  DP_TRY(check_dev(y, eb, false, "y"));
  DP_TRY(check_dev(r, es, some && y, "r"));
  DP_TRY(check_dev(z, eb, some && pre, "z"));
  if (some && !y && r) return op_fail(DP_ERR_INVALID_ARG, "r must be NULL without y");
  if (some && !pre && z) return op_fail(DP_ERR_INVALID_ARG, "z must be NULL without DP_NORM_PRE");
  DP_TRY(check_dev(w_post, ep, false, "w_post"));
  DP_TRY(check_dev(b_post, ep, false, "b_post"));
  DP_TRY(check_dev(gate, ep, false, "gate"));
  DP_TRY(check_dev(w_pre, ep, false, "w_pre"));
  DP_TRY(check_dev(b_pre, ep, false, "b_pre"));
  DP_TRY(check_dev(post_stats, 8, false, "post_stats"));
  DP_TRY(check_dev(pre_stats, 8, false, "pre_stats"));
  if (!some) return DP_OK;
  const Shape s = shape_of(p->dim);
  NormParams P = base_params(*p, s);
  P.r = r;
  P.z = z;
  P.x = x;
  P.y = y;
  // Without the post norm its weight and bias are not used: N_post(y) = y.
  P.w_post = P.post ? w_post : nullptr;
  P.b_post = P.post ? b_post : nullptr;
  P.gate = gate;
  P.w_pre = w_pre;
  P.b_pre = b_pre;
  P.post_stats = reinterpret_cast<float2*>(post_stats);
  P.pre_stats = reinterpret_cast<float2*>(pre_stats);
  NvtxRange range("block norm");
  dispatch(*p, p->dim % 8 == 0 && slots_fit(*p, s, 1) && all16({x, y, r, z}), s.nv, Forward{P, s, (cudaStream_t)stream});
  return op_launched("block norm launch", 1);
}

size_t dp_block_norm_workspace_size(int64_t rows, int64_t dim) {
  if (rows < 0 || rows > INT32_MAX || dim < 1 || dim > DP_MAX_NORM_DIM) {
    op_fail(DP_ERR_INVALID_ARG, "rows = %lld or dim = %lld out of range", (long long)rows, (long long)dim);
    return 0;
  }
  const int64_t parts = rows + 3 < MAX_PARTS ? rows + 3 : MAX_PARTS;
  return (size_t)(parts * 4 * dim * 4 + 255) / 256 * 256;
}

dp_status_t dp_block_norm_grad(const dp_block_norm_t* p, void* dx, void* dy, const void* dr, const void* dz,
                               const void* r, const void* y, const void* w_post, const void* b_post, const void* gate,
                               const void* w_pre, const float* post_stats, const float* pre_stats, void* dw_post,
                               void* db_post, void* dgate, void* dw_pre, void* db_pre, void* ws, dp_stream_t stream_) {
  DP_TRY(check_norm(p, y != nullptr, gate != nullptr));
  const bool some = p->rows > 0, pre = (p->norms & DP_NORM_PRE) != 0, post = (p->norms & DP_NORM_POST) != 0;
  const int es = elem_size(p->stream_dtype), eb = elem_size(p->block_dtype), ep = elem_size(p->param_dtype);
  DP_TRY(check_dev(dx, es, some, "dx"));
  DP_TRY(check_dev(dy, eb, some && y, "dy"));
  DP_TRY(check_dev(dr, es, false, "dr"));
  DP_TRY(check_dev(dz, eb, some && pre, "dz"));
  DP_TRY(check_dev(r, es, some && pre, "r"));
  DP_TRY(check_dev(y, eb, false, "y"));
  if (some && !y && dy) return op_fail(DP_ERR_INVALID_ARG, "dy must be NULL without y");
  DP_TRY(check_dev(w_post, ep, false, "w_post"));
  DP_TRY(check_dev(b_post, ep, false, "b_post"));
  DP_TRY(check_dev(gate, ep, false, "gate"));
  DP_TRY(check_dev(w_pre, ep, false, "w_pre"));
  DP_TRY(check_dev(post_stats, 8, some && post, "post_stats"));
  DP_TRY(check_dev(pre_stats, 8, some && pre, "pre_stats"));
  DP_TRY(check_dev(dw_post, ep, false, "dw_post"));
  DP_TRY(check_dev(db_post, ep, false, "db_post"));
  DP_TRY(check_dev(dgate, ep, false, "dgate"));
  DP_TRY(check_dev(dw_pre, ep, false, "dw_pre"));
  DP_TRY(check_dev(db_pre, ep, false, "db_pre"));
  if (!post && (dw_post || db_post)) return op_fail(DP_ERR_INVALID_ARG, "dw_post and db_post need DP_NORM_POST");
  if (!pre && (dw_pre || db_pre)) return op_fail(DP_ERR_INVALID_ARG, "dw_pre and db_pre need DP_NORM_PRE");
  if (p->gate_mode == DP_GATE_NONE && dgate) return op_fail(DP_ERR_INVALID_ARG, "dgate needs a gate");
  DP_TRY(check_dev(ws, 256, some, "ws"));
  const cudaStream_t stream = (cudaStream_t)stream_;
  NvtxRange range("block norm gradient");
  int64_t parts = 0;
  int launches = 0;
  // S0 and P0 are summed for the biases' gradients, and for a channel gate's where the post norm has a bias.
  const bool sum0 = p->kind == DP_NORM_LAYER || db_post || db_pre || (dgate && post && b_post);
  if (some) {
    const Shape s = shape_of(p->dim);
    NormParams P = base_params(*p, s);
    P.dx = dx;
    P.dy = dy;
    P.dr = dr;
    P.dz = dz;
    P.x = r;
    P.y = y;
    P.w_post = post ? w_post : nullptr;
    P.b_post = post ? b_post : nullptr;
    P.gate = gate;
    P.w_pre = w_pre;
    P.post_stats = reinterpret_cast<float2*>(const_cast<float*>(post_stats));
    P.pre_stats = reinterpret_cast<float2*>(const_cast<float*>(pre_stats));
    P.dgate_token = p->gate_mode == DP_GATE_TOKEN ? dgate : nullptr;
    P.part = static_cast<float*>(ws);
    P.bias = P.dgate_token && P.b_post;
    parts = dispatch(*p, p->dim % 8 == 0 && slots_fit(*p, s, 2) && all16({dx, dy, dr, dz, r, y}), s.nv, Gradient{P, s, sum0, stream});
    ++launches;
  }
  FinishParams F = {};
  F.part = static_cast<const float*>(ws);
  F.parts = parts;
  F.dim = p->dim;
  F.sum0 = sum0;
  F.gate_mode = p->gate_mode;
  F.pdt = p->param_dtype;
  F.accumulate = p->accumulate;
  F.w_post = post ? w_post : nullptr;
  F.b_post = post ? b_post : nullptr;
  F.gate = gate;
  F.dw_post = dw_post;
  F.db_post = db_post;
  F.dgate = p->gate_mode == DP_GATE_CHANNEL ? dgate : nullptr;
  F.dw_pre = dw_pre;
  F.db_pre = db_pre;
  F.b = p->branch_scale;
  if (F.dw_post || F.db_post || F.dgate || F.dw_pre || F.db_pre) {
    const cudaError_t e = launch_after(norm_finish_kernel, (p->dim + FIN_COLS - 1) / FIN_COLS, dim3(FIN_COLS, FIN_ROWS), stream, F);
    if (e != cudaSuccess) return op_fail(DP_ERR_CUDA, "block norm gradient launch: %s", cudaGetErrorString(e));
    ++launches;
  }
  return launches ? op_launched("block norm gradient launch", launches) : DP_OK;
}

}  // extern "C"
