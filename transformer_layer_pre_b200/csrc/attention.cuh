// attention.cuh — what the kernels of the attention entry points
// (tl_attention_forward, tl_attention_backward) share: the launch arguments
// and the layout of the prepared workspace.
//
// Per sequence b and head h (c = scale, T the bias table):
//   x_ij = log2(e) (c q_i.k_j + T[bucket(j - i), h] + mask_bj)
//   P_ij = 2^(x_ij - lse2_i), lse2_i = log2 sum_j 2^x_ij
// Everything added to q_i.k_j is prepared in log2 units by one launch
// (attn_prep_kernel) into the workspace:
//   maskx  [B or 1][Sp]      log2(e) * mask, -inf for a removed key and past the sequence end
//   flags  [B or 1][Sp / 64] of each 64 keys: 0 all of maskx is 0, 1 mixed, 2 every key removed
//   vec    [heads][dirs][4][len] the bias along the diagonals, see bias_at
//   bid    [len]             the bucket of each of those diagonals
//   stats  [B * heads][Sp / 64][2][64] backward, per 64 queries: -lse2 (-inf for an empty row and past
//          the end), then -D = -(dO.O); for 16-bit storage log2(kAttnPUp) - lse2 and -D / kAttnPUp
//   smax   [B * heads][nmax] backward, float16: of each attn_prep_rows(d) tokens the largest |dO| of a row
//          with a key and the largest |V| of a key that is not removed (ds_factor)
//   dpart  backward: partial sums of the bias table's gradient, zeroed
// with Sp = the sequence length rounded up to 128.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace tlp {

constexpr float kAttnLog2e = 1.4426950408889634f;
constexpr float kAttnLn2 = 0.6931471805599453f;
constexpr float kAttnMasked = -1e30f;      // a mask value at or below this removes the key
constexpr int kAttnMaxBuckets = 256;
constexpr int kAttnFlagKeys = 64;
constexpr float kAttnPUp = 256.0f;         // 16-bit storage, backward: the factor that P is held at (attention_tc.cu)

// Tokens of a block of attn_prep_kernel's row part: 256 / G groups of G lanes
// (16 bytes each), prep_rows(G) rows to a group.
constexpr int kPrepThreads = 256;
__host__ __device__ constexpr int prep_rows(int G) { return G == 4 ? 2 : 4; }
inline int attn_prep_rows(int d) { return d * 2 <= 128 ? 128 : 64; }   // 16-bit storage

// float16 storage: dS is held at a power of two chosen per sequence and head,
// so that gradients of any size (a loss scale, or none) keep its precision:
// float16 loses bits below 2^-14 and ends at 65504.  |dS_ij| <= P_ij (|dO_i.v_j|
// + |D_i|) <= 2 M, M := d max|dO| max|V|, and the factor is the power of two F
// with 2^13 < M F <= 2^14: no overflow (2^15 with room for rounding), and an
// entry is off by at most 2^-25 / F < 2^-38 M where it is subnormal.  F enters
// with dP and D and leaves where dQ, dK and the table's gradient are written
// out; all of it is exact.  m: max|dO| and max|V|.
__device__ __forceinline__ float ds_factor(__half2 m, int d) {
  const float M = __low2float(m) * __high2float(m) * (float)d;
  if (M == 0.0f || isinf(M)) return 1.0f;
  // 2^e <= M < 2^(e + 1), M from 2^-45 to 2^39
  const int e = (__float_as_int(M) >> 23) - 127;
  return __int_as_float((127 + 13 - e) << 23);
}
// The larger magnitudes, lane by lane (NaN left out).
__device__ __forceinline__ __half2 max_abs(__half2 m, uint32_t x) {
  return __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&x)));
}
__device__ __forceinline__ __half2 max_abs(__half2 m, const uint4& x) {
  return max_abs(max_abs(max_abs(max_abs(m, x.x), x.y), x.z), x.w);
}
// The largest of both lanes of a, and of b.
__device__ __forceinline__ __half2 fold_max(__half2 a, __half2 b) {
  return __hmax2(__lows2half2(a, b), __highs2half2(a, b));
}
__device__ __forceinline__ __half2 warp_max2(__half2 m) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = __hmax2(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
// lse in log2 units, for P = 2^(x - lse2).  Both come through some six roundings
// of their own size; where those are worth more than a factor (|lse2| above
// 2^21: finite masks over a whole row, -1e8 and the like), P is not known, and
// lse2 is raised by eight of them, so that P stays below 1 instead of passing
// the storage type's end.
__device__ __forceinline__ float lse_log2(float lse) {
  const float x = lse * kAttnLog2e, slack = fabsf(x) * (1.0f / (1 << 20));
  return slack > 2.0f ? x + slack : x;
}
// 1 / x of a power of two.
__device__ __forceinline__ float inv_pow2(float x) { return __int_as_float((254 << 23) - __float_as_int(x)); }

// A (batch, token, head, dim) tensor: element strides, dim contiguous.
struct AttnView {
  void* p;
  long long sb, st, sh;
};

struct AttnOp {
  int B, S, Sp, nh, d;
  float scale;               // c
  float c2;                  // c * log2(e)
  AttnView q, k, v, o, dout, dq, dk, dv;
  float* lse;                // (B, nh, S)
  // prepared inputs
  const float* mask;         // (B, S) or null
  const void* table;         // (buckets, nh) or null
  int buckets;
  float* maskx;
  int* flags;
  int mask_seqs;             // B, or 1 without a mask (every sequence reads row 0)
  float* vec;                // null without a table
  int vec_len, vec_off;      // floats per copy; offset of diagonal 0
  int sat;                   // |j - i| >= sat: the bias no longer depends on the distance
  uint8_t* bid;
  float* stats;
  __half2* smax;             // null but for float16
  int nmax;
  // bias table gradient: partial sums [B * nh][ditems][buckets], null when not wanted
  float* dpart;
  int ditems;                // partial rows per (b, h)
  float* dtable;             // (buckets, nh)
  int daccumulate;
  // bucket u holds the diagonals j - i in [lo[u], lo[u] + n[u]) (n = 0: none)
  int lo[kAttnMaxBuckets], n[kAttnMaxBuckets];
};

// The bias of diagonal x = j - i (direction 0) or x = i - j (direction 1), in
// log2 units: copy s of a direction holds the diagonal x at index
// x + vec_off - s - 1, so a run that starts at any x begins 16-byte aligned in
// one of the four copies.
__device__ __forceinline__ const float* bias_copy(const AttnOp& a, int h, int dir, int s) {
  return a.vec + ((size_t)(h * 2 + dir) * 4 + s) * a.vec_len;
}

// Whether the backward takes a sequence and head as one tile of keys and queries.
bool attn_one_tile(int dt, int seq, int head_dim);

void attn_prep_run(int dt, const AttnOp& a, bool backward, cudaStream_t s);
void attn_table_grad_run(const AttnOp& a, cudaStream_t s);
// float32 storage
void attention_f32_fwd_run(const AttnOp& a, cudaStream_t s);
void attention_f32_bwd_run(const AttnOp& a, cudaStream_t s);
// 16-bit storage; false when a tensor could not be described to the TMA unit
bool attention_tc_fwd_run(int dt, const AttnOp& a, cudaStream_t s);
bool attention_tc_bwd_run(int dt, const AttnOp& a, cudaStream_t s);

}  // namespace tlp
