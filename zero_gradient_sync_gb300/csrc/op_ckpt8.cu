// Activation checkpoints in 8 bits, and the gated activation whose forward writes them and whose gradient reads them.
//
// A group of 32 values of a row is kept as int8 codes and one byte E: value = code 2^(E - 127).  The step is the least
// power of two with max|x| <= 127 step, so codes use the range 64..127 of their magnitude: the rounding error is at most
// max|x| / 128.  A power of two costs up to one bit against the step max|x| / 127, and buys that scaling and decoding are
// exact: code * step has 7 significant bits, so a bf16 product sees just what the checkpoint holds.
//
// Everything here is elementwise and bounded by memory: for a gated activation the forward reads 4 bytes and writes
// 2 + 2 (1 + 1/32) an element, the gradient reads 2 + 2 (1 + 1/32) and writes 6 -- against 6 read and 6 written from
// bf16 copies, and the saved bytes are the point: a third of the memory between the passes is gone.  A thread takes eight
// consecutive elements (16 bytes of bf16, 8 of codes); four neighbours make a group and find its maximum by two shuffles.
#include "op_common.cuh"

namespace dp {
namespace {

constexpr int THREADS = 256;
constexpr int GROUP = DP_CKPT8_GROUP;

// The byte E of a group whose largest magnitude is `top` (an infinity or a NaN there gives 255).
__device__ __forceinline__ uint32_t step_byte(float top) {
  // top = f 2^e with f in [1, 2): 127 2^k >= top needs k = e - 6 where f <= 127/64, else e - 5.  As integers: E = k +
  // 127 = exponent field - 6, plus one where the fraction is above 63/64.  Below 2^-120 the step stays at 2^-126.
  const uint32_t bits = __float_as_uint(top) & 0x7fffffffu;
  if (bits >= 0x7f800000u) return 255u;
  const int e = (int)(bits >> 23) - 6 + ((bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return (uint32_t)(e < 1 ? 1 : e);
}
__device__ __forceinline__ float step_of(uint32_t E) { return E == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(E << 23); }
// 1 / step: exact, and normal for E <= 253 (no group has more than 249).
__device__ __forceinline__ float inv_step_of(uint32_t E) { return __uint_as_float((254u - E) << 23); }

// Codes of eight values, the group's byte known.
__device__ __forceinline__ uint2 codes_of(const float (&v)[8], uint32_t E) {
  if (E == 255u) return make_uint2(0u, 0u);
  const float s = inv_step_of(E);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k >> 2] |= ((uint32_t)__float2int_rn(v[k] * s) & 0xffu) << (8 * (k & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void values_of(uint2 c, uint32_t E, float (&v)[8]) {
  const float s = step_of(E);
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = (float)(int8_t)(((k < 4 ? c.x : c.y) >> (8 * (k & 3))) & 0xffu) * s;
}

// Largest magnitude of the group that this thread and its three neighbours hold.  fmaxf drops a NaN, so one is carried
// as an infinity.
__device__ __forceinline__ float group_top(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = fmaxf(m, nonfinite(v[k]) ? __uint_as_float(0x7f800000u) : fabsf(v[k]));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// Where a thread's eight elements lie.  Elements are numbered through the padded rows, so a group never leaves a warp's
// aligned quad of threads; a CTA finds its first row by one 64-bit division.
struct Place {
  int64_t row;
  int col;
  bool on;
};
struct Walk {
  int64_t rows;
  int pieces;  // eights of a padded row
  int dim;
};
__device__ __forceinline__ Place place_of(const Walk& W) {
  const int64_t first = (int64_t)blockIdx.x * THREADS;
  const int64_t row0 = first / W.pieces;
  const uint32_t rest = (uint32_t)(first - row0 * W.pieces) + threadIdx.x;
  const uint32_t down = rest / (uint32_t)W.pieces;
  Place p;
  p.row = row0 + down;
  p.col = (int)(rest - down * (uint32_t)W.pieces) * 8;
  p.on = p.row < W.rows;
  return p;
}

template <typename T>
__device__ __forceinline__ void load_piece(const T* base, int64_t ld, const Place& p, int dim, int vec, float (&v)[8]) {
  const T* q = base + p.row * ld + p.col;
  if (p.on && vec && p.col < dim) {  // vec: dim is a multiple of 8
    const Raw8<T> w = load_raw8(q);
    w.unpack(v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = p.on && p.col + k < dim ? Elem<T>::get(q[k]) : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ void store_piece(T* base, int64_t ld, const Place& p, int dim, int vec, const float (&v)[8]) {
  T* q = base + p.row * ld + p.col;
  if (!p.on) return;
  if (vec) {
    if (p.col >= dim) return;
    Raw8<T> o;
    o.pack(v);
    store_raw8(q, o);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (p.col + k < dim) q[k] = Elem<T>::put(v[k]);
  }
}
struct Ckpt {
  int8_t* codes;
  uint8_t* scales;
};
__device__ __forceinline__ void put_ckpt(const Ckpt& c, const Place& p, int pitch, const float (&v)[8]) {
  const uint32_t E = step_byte(group_top(v));
  if (!p.on) return;
  *reinterpret_cast<uint2*>(c.codes + p.row * pitch + p.col) = codes_of(v, E);
  if ((p.col & (GROUP - 1)) == 0) c.scales[p.row * (pitch / GROUP) + p.col / GROUP] = (uint8_t)E;
}
__device__ __forceinline__ void get_ckpt(const Ckpt& c, const Place& p, int pitch, float (&v)[8]) {
  uint2 w = make_uint2(0u, 0u);
  uint32_t E = 1u;
  if (p.on) {
    w = __ldcs(reinterpret_cast<const uint2*>(c.codes + p.row * pitch + p.col));
    E = c.scales[p.row * (pitch / GROUP) + p.col / GROUP];
  }
  values_of(w, E, v);
}

template <typename T>
__global__ void __launch_bounds__(THREADS) encode_kernel(Ckpt c, const T* x, int64_t ldx, Walk W, int vec) {
  const Place p = place_of(W);
  float v[8];
  load_piece(x, ldx, p, W.dim, vec, v);
  put_ckpt(c, p, W.pieces * 8, v);
}
template <typename T>
__global__ void __launch_bounds__(THREADS) decode_kernel(T* x, int64_t ldx, Ckpt c, Walk W, int vec) {
  const Place p = place_of(W);
  float v[8];
  get_ckpt(c, p, W.pieces * 8, v);
  store_piece(x, ldx, p, W.dim, vec, v);
}

// f(g) and f'(g), with s the logistic function.  SiLU: f = g s(g), f' = s (1 + g (1 - s)).  GELU's tanh form is
// f = g s(2y), y = c (g + 0.044715 g^3), c = sqrt(2 / pi), since (1 + tanh y) / 2 = s(2y); f' = s + 2 f (1 - s) c (1 +
// 0.134145 g^2).  With t = e^-|v| and q = 1 / (1 + t), s(v) and 1 - s(v) are q and t q, or the reverse: neither cancels,
// and t runs out of range only where it is below fp32.  g^2 stops at 10^4, where t has long been 0, so that no product of
// infinity and zero appears.
__device__ __forceinline__ void logistic(float v, float& s, float& rest) {
  const float t = __expf(-fabsf(v));
  const float q = __fdividef(1.0f, 1.0f + t), tq = t * q;
  s = v < 0.0f ? tq : q;
  rest = v < 0.0f ? q : tq;
}
template <int ACT>
__device__ __forceinline__ void act_of(float g, float& f, float& df) {
  float s, rest;
  if (ACT == DP_ACT_SILU) {
    logistic(g, s, rest);
    f = g * s;
    df = s * fmaf(g, rest, 1.0f);
  } else {
    const float c = 0.7978845608028654f;
    const float g2 = fminf(g * g, 1e4f);
    logistic(2.0f * c * g * fmaf(0.044715f, g2, 1.0f), s, rest);
    f = g * s;
    df = fmaf(f * rest, 2.0f * c * fmaf(0.134145f, g2, 1.0f), s);
  }
}

template <int ACT, bool GATED>
__global__ void __launch_bounds__(THREADS) act_kernel(bf16_t* h, const bf16_t* g, const bf16_t* u, Ckpt g8, Ckpt u8,
                                                      int64_t ld, int64_t ldh, Walk W, int vec) {
  const Place p = place_of(W);
  float gv[8], uv[8], f, df;
  load_piece(g, ld, p, W.dim, vec, gv);
  if (GATED) load_piece(u, ld, p, W.dim, vec, uv);
  put_ckpt(g8, p, W.pieces * 8, gv);
  if (GATED) put_ckpt(u8, p, W.pieces * 8, uv);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    act_of<ACT>(gv[k], f, df);
    gv[k] = GATED ? f * uv[k] : f;
  }
  store_piece(h, ldh, p, W.dim, vec, gv);
}

template <int ACT, bool GATED>
__global__ void __launch_bounds__(THREADS) act_grad_kernel(bf16_t* dg, bf16_t* du, bf16_t* h, const bf16_t* dh, Ckpt g8,
                                                           Ckpt u8, int64_t ld, int64_t ldh, Walk W, int vec) {
  const Place p = place_of(W);
  float dv[8], gv[8], uv[8], hv[8];
  load_piece(dh, ldh, p, W.dim, vec, dv);
  get_ckpt(g8, p, W.pieces * 8, gv);
  if (GATED) get_ckpt(u8, p, W.pieces * 8, uv);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float f, df;
    act_of<ACT>(gv[k], f, df);
    hv[k] = GATED ? f * uv[k] : f;
    gv[k] = (GATED ? dv[k] * uv[k] : dv[k]) * df;
    dv[k] *= f;
  }
  store_piece(dg, ld, p, W.dim, vec, gv);
  if (GATED) store_piece(du, ld, p, W.dim, vec, dv);
  if (h) store_piece(h, ldh, p, W.dim, vec, hv);
}

// ---------------------------------------------------------------------------------------------------- host side

dp_status_t check_rows(int64_t rows, int64_t dim) {
  if (rows < 0) return op_fail(DP_ERR_INVALID_ARG, "rows < 0");
  if (dim < 1 || dim > (1 << 28)) return op_fail(DP_ERR_INVALID_ARG, "dim = %lld not in 1..2^28", (long long)dim);
  const int64_t pieces = dp_ckpt8_pitch(dim) / 8;
  if (rows > (int64_t(INT32_MAX) * THREADS) / pieces) return op_fail(DP_ERR_INVALID_ARG, "rows x dim is too large");
  return DP_OK;
}
dp_status_t check_ld(int64_t ld, int64_t dim, const char* name) {
  if (ld < dim || ld > (int64_t(1) << 40)) return op_fail(DP_ERR_INVALID_ARG, "%s = %lld is below the row's %lld elements (or far too large)", name, (long long)ld, (long long)dim);
  return DP_OK;
}
dp_status_t check_ckpt(const int8_t* codes, const uint8_t* scales, bool needed, const char* name) {
  if ((!codes || !scales) && needed) return op_fail(DP_ERR_INVALID_ARG, "%s: codes or scales are NULL", name);
  if (!is_aligned(codes, 32)) return op_fail(DP_ERR_ALIGNMENT, "%s: codes are not 32-byte aligned", name);
  return DP_OK;
}
Walk walk_of(int64_t rows, int64_t dim) { return Walk{rows, (int)(dp_ckpt8_pitch(dim) / 8), (int)dim}; }
unsigned grid_of(const Walk& W) { return (unsigned)((W.rows * W.pieces + THREADS - 1) / THREADS); }
bool rows16(const void* p, int64_t ld, int size) { return is_aligned(p, 16) && ld * size % 16 == 0; }

}  // namespace
}  // namespace dp

using namespace dp;

extern "C" {

int64_t dp_ckpt8_pitch(int64_t dim) { return dim < 1 ? -1 : (dim + GROUP - 1) / GROUP * GROUP; }

dp_status_t dp_ckpt8_encode(int8_t* codes, uint8_t* scales, const void* x, int64_t rows, int64_t dim, int64_t ldx,
                            int32_t dtype, dp_stream_t stream) {
  DP_TRY(check_rows(rows, dim));
  DP_TRY(check_ld(ldx, dim, "ldx"));
  DP_TRY(check_dtype(dtype, "dtype"));
  const int e = elem_size(dtype);
  DP_TRY(check_dev(x, e, rows > 0, "x"));
  DP_TRY(check_ckpt(codes, scales, rows > 0, "checkpoint"));
  if (rows == 0) return DP_OK;
  const Walk W = walk_of(rows, dim);
  const int vec = dim % 8 == 0 && rows16(x, ldx, e);
  NvtxRange range("checkpoint encode");
  if (dtype == DP_BF16)
    encode_kernel<<<grid_of(W), THREADS, 0, (cudaStream_t)stream>>>(Ckpt{codes, scales}, (const bf16_t*)x, ldx, W, vec);
  else
    encode_kernel<<<grid_of(W), THREADS, 0, (cudaStream_t)stream>>>(Ckpt{codes, scales}, (const float*)x, ldx, W, vec);
  return op_launched("checkpoint encode launch", 1);
}

dp_status_t dp_ckpt8_decode(void* x, const int8_t* codes, const uint8_t* scales, int64_t rows, int64_t dim, int64_t ldx,
                            int32_t dtype, dp_stream_t stream) {
  DP_TRY(check_rows(rows, dim));
  DP_TRY(check_ld(ldx, dim, "ldx"));
  DP_TRY(check_dtype(dtype, "dtype"));
  const int e = elem_size(dtype);
  DP_TRY(check_dev(x, e, rows > 0, "x"));
  DP_TRY(check_ckpt(codes, scales, rows > 0, "checkpoint"));
  if (rows == 0) return DP_OK;
  const Walk W = walk_of(rows, dim);
  const Ckpt c{const_cast<int8_t*>(codes), const_cast<uint8_t*>(scales)};
  const int vec = dim % 8 == 0 && rows16(x, ldx, e);
  NvtxRange range("checkpoint decode");
  if (dtype == DP_BF16)
    decode_kernel<<<grid_of(W), THREADS, 0, (cudaStream_t)stream>>>((bf16_t*)x, ldx, c, W, vec);
  else
    decode_kernel<<<grid_of(W), THREADS, 0, (cudaStream_t)stream>>>((float*)x, ldx, c, W, vec);
  return op_launched("checkpoint decode launch", 1);
}

dp_status_t dp_act_ckpt8(uint16_t* h, const uint16_t* g, const uint16_t* u, int8_t* g8, uint8_t* g8_scales, int8_t* u8,
                         uint8_t* u8_scales, int64_t rows, int64_t dim, int64_t ld, int64_t ldh, int32_t act,
                         dp_stream_t stream) {
  DP_TRY(check_rows(rows, dim));
  DP_TRY(check_ld(ld, dim, "ld"));
  DP_TRY(check_ld(ldh, dim, "ldh"));
  if (act != DP_ACT_SILU && act != DP_ACT_GELU) return op_fail(DP_ERR_INVALID_ARG, "act = %d unknown", act);
  DP_TRY(check_dev(h, 2, rows > 0, "h"));
  DP_TRY(check_dev(g, 2, rows > 0, "g"));
  DP_TRY(check_dev(u, 2, false, "u"));
  DP_TRY(check_ckpt(g8, g8_scales, rows > 0, "g8"));
  DP_TRY(check_ckpt(u8, u8_scales, u != nullptr, "u8"));
  if (!u && (u8 || u8_scales)) return op_fail(DP_ERR_INVALID_ARG, "u8 must be NULL without u");
  if (rows == 0) return DP_OK;
  const Walk W = walk_of(rows, dim);
  const int vec = dim % 8 == 0 && rows16(g, ld, 2) && rows16(u, ld, 2) && rows16(h, ldh, 2);
  const Ckpt a{g8, g8_scales}, b{u8, u8_scales};
  auto k = act == DP_ACT_SILU ? (u ? act_kernel<DP_ACT_SILU, true> : act_kernel<DP_ACT_SILU, false>)
                              : (u ? act_kernel<DP_ACT_GELU, true> : act_kernel<DP_ACT_GELU, false>);
  NvtxRange range("activation with checkpoint");
  k<<<grid_of(W), THREADS, 0, (cudaStream_t)stream>>>(h, g, u, a, b, ld, ldh, W, vec);
  return op_launched("activation launch", 1);
}

dp_status_t dp_act_ckpt8_grad(uint16_t* dg, uint16_t* du, uint16_t* h, const uint16_t* dh, const int8_t* g8,
                              const uint8_t* g8_scales, const int8_t* u8, const uint8_t* u8_scales, int64_t rows,
                              int64_t dim, int64_t ld, int64_t ldh, int32_t act, dp_stream_t stream) {
  DP_TRY(check_rows(rows, dim));
  DP_TRY(check_ld(ld, dim, "ld"));
  DP_TRY(check_ld(ldh, dim, "ldh"));
  if (act != DP_ACT_SILU && act != DP_ACT_GELU) return op_fail(DP_ERR_INVALID_ARG, "act = %d unknown", act);
  DP_TRY(check_dev(dg, 2, rows > 0, "dg"));
  DP_TRY(check_dev(du, 2, rows > 0 && u8, "du"));
  DP_TRY(check_dev(h, 2, false, "h"));
  DP_TRY(check_dev(dh, 2, rows > 0, "dh"));
  DP_TRY(check_ckpt(g8, g8_scales, rows > 0, "g8"));
  DP_TRY(check_ckpt(u8, u8_scales, u8 || u8_scales, "u8"));
  if (!u8 && du) return op_fail(DP_ERR_INVALID_ARG, "du needs the checkpoint of u");
  if (rows == 0) return DP_OK;
  const Walk W = walk_of(rows, dim);
  const int vec = dim % 8 == 0 && rows16(dg, ld, 2) && rows16(du, ld, 2) && rows16(h, ldh, 2) && rows16(dh, ldh, 2);
  const Ckpt a{const_cast<int8_t*>(g8), const_cast<uint8_t*>(g8_scales)};
  const Ckpt b{const_cast<int8_t*>(u8), const_cast<uint8_t*>(u8_scales)};
  auto k = act == DP_ACT_SILU ? (u8 ? act_grad_kernel<DP_ACT_SILU, true> : act_grad_kernel<DP_ACT_SILU, false>)
                              : (u8 ? act_grad_kernel<DP_ACT_GELU, true> : act_grad_kernel<DP_ACT_GELU, false>);
  NvtxRange range("activation gradient");
  k<<<grid_of(W), THREADS, 0, (cudaStream_t)stream>>>(dg, du, h, dh, a, b, ld, ldh, W, vec);
  return op_launched("activation gradient launch", 1);
}

}  // extern "C"
