// attention_simt.cu — attention with a relative position bias, forward and
// backward, in IEEE float32 products and sums (SIMT): the path of float32
// storage, whose outputs are held to float32 rounding.
//
// Tiles of 64 rows x 64 columns, 256 threads, a 4 x 4 block of scores per
// thread.  Operands lie transposed in shared memory ([dim][64 + 4]), so both
// kinds of product read float4: S = A B^T walks the dims (two float4 per 16
// FMAs), acc += P B walks the columns of P four at a time.
//
// The backward has two kinds of items, each with its rows stationary and its
// columns moving, and no sum shared between blocks (bitwise reproducible):
//   key rows    S^T = K Q^T, dP^T = V dO^T;  dV += P^T dO, dK += dS^T Q
//   query rows  S   = Q K^T, dP   = dO V^T;  dQ += dS K, and the bias
//               gradient: dS summed along its diagonals, then by bucket.
//
// Bound: FP32 FMAs and the shared-memory reads that feed them (two float4 per 16
// FMAs), and too few blocks for the SMs at small batches: 6 to 12 TFLOP/s; B1 h4
// d64 S1024 forward 103 us with 64 blocks on 148 SMs.
#include <math.h>

#include "attention.cuh"
#include "kernels.h"
#include "profile.h"

namespace tlp {
namespace {

constexpr int kT = 64;          // rows and columns of a tile
constexpr int kLd = kT + 4;     // padded row of the transposed operands
constexpr int kThr = 256;

__device__ __forceinline__ const float* row_ptr(const AttnView& v, int b, int h, int i) {
  return static_cast<const float*>(v.p) + (size_t)b * v.sb + (size_t)h * v.sh + (size_t)i * v.st;
}

// Rows r0 .. r0 + 63 of one head, transposed into t[dim][kLd]; zeros past the
// sequence and past the head dim.
template <int D>
__device__ __forceinline__ void load_t(float* t, const AttnView& v, int b, int h, int r0, int S, int d) {
  for (int x = threadIdx.x; x < kT * (D / 4); x += kThr) {
    const int r = x % kT, c = (x / kT) * 4;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    if (r0 + r < S && c < d) {
      const float4 x = *reinterpret_cast<const float4*>(row_ptr(v, b, h, r0 + r) + c);
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) t[(c + k) * kLd + r] = w[k];
  }
}

// s[i][j] = sum_c A[c][4 ty + i] B[c][4 tx + j]
template <int D>
__device__ __forceinline__ void scores(const float* A, const float* B, int ty, int tx, float (&s)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
#pragma unroll 8
  for (int c = 0; c < D; ++c) {
    const float4 x = *reinterpret_cast<const float4*>(A + c * kLd + 4 * ty);
    const float4 y = *reinterpret_cast<const float4*>(B + c * kLd + 4 * tx);
    const float xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = fmaf(xa[i], ya[j], s[i][j]);
  }
}

// acc[i][m] += sum_t P[4 ty + i][t] B[tx + 16 m][t]
template <int D>
__device__ __forceinline__ void product(const float* P, const float* B, int ty, int tx, float (&acc)[4][D / 16]) {
#pragma unroll 4
  for (int t = 0; t < kT; t += 4) {
    float4 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(P + (4 * ty + i) * kLd + t);
#pragma unroll
    for (int m = 0; m < D / 16; ++m) {
      const float4 y = *reinterpret_cast<const float4*>(B + (tx + 16 * m) * kLd + t);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i][m] = fmaf(p[i].x, y.x, acc[i][m]);
        acc[i][m] = fmaf(p[i].y, y.y, acc[i][m]);
        acc[i][m] = fmaf(p[i].z, y.z, acc[i][m]);
        acc[i][m] = fmaf(p[i].w, y.w, acc[i][m]);
      }
    }
  }
}

template <int D>
__device__ __forceinline__ void store_rows(const AttnView& v, int b, int h, int r0, int S, int d, int ty, int tx,
                                           const float (&acc)[4][D / 16], const float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 4 * ty + i;
    if (r >= S) continue;
    float* p = const_cast<float*>(row_ptr(v, b, h, r));
#pragma unroll
    for (int m = 0; m < D / 16; ++m)
      if (tx + 16 * m < d) p[tx + 16 * m] = acc[i][m] * f[i];
  }
}

// The bias of diagonal x (key minus query), log2 units.
__device__ __forceinline__ float bias_at(const AttnOp& a, const float* vec, int x) {
  x = max(-a.sat, min(a.sat, x));
  return vec[x + a.vec_off - 1];
}

template <int D>
__global__ void __launch_bounds__(kThr) attn_fwd_kernel(const __grid_constant__ AttnOp a) {
  extern __shared__ __align__(16) float sm[];
  float* sQ = sm;
  float* sK = sQ + D * kLd;
  float* sV = sK + D * kLd;
  float* sP = sV + D * kLd;
  pdl_wait();
  pdl_launch_dependents();
  const int nq = (a.S + kT - 1) / kT;
  const int it = blockIdx.x, bh = it / nq, q0 = (it - bh * nq) * kT, b = bh / a.nh, h = bh - b * a.nh;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int mb = a.mask_seqs == 1 ? 0 : b;
  const float* vec = a.vec ? bias_copy(a, h, 0, 0) : nullptr;
  load_t<D>(sQ, a.q, b, h, q0, a.S, a.d);
  float o[4][D / 16] = {};
  float m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = -INFINITY, l[i] = 0.0f;
  for (int k0 = 0; k0 < a.S; k0 += kT) {
    if (a.flags[mb * (a.Sp / kAttnFlagKeys) + k0 / kAttnFlagKeys] == 2) continue;
    __syncthreads();
    load_t<D>(sK, a.k, b, h, k0, a.S, a.d);
    load_t<D>(sV, a.v, b, h, k0, a.S, a.d);
    __syncthreads();
    float s[4][4];
    scores<D>(sQ, sK, ty, tx, s);
    const float4 mk = *reinterpret_cast<const float4*>(a.maskx + (size_t)mb * a.Sp + k0 + 4 * tx);
    const float mm[4] = {mk.x, mk.y, mk.z, mk.w};
    float corr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float bias = vec ? bias_at(a, vec, k0 + 4 * tx + j - q0 - 4 * ty - i) : 0.0f;
        // a removed key is left out whatever its score is
        s[i][j] = mm[j] == -INFINITY ? -INFINITY : fmaf(s[i][j], a.c2, bias + mm[j]);
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      const float mnew = fmaxf(m[i], top);
      const float sub = mnew == -INFINITY ? 0.0f : mnew;
      corr[i] = exp2f(m[i] - sub);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = exp2f(s[i][j] - sub);
        sum += s[i][j];
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[i] = l[i] * corr[i] + sum;
      m[i] = mnew;
      *reinterpret_cast<float4*>(sP + (4 * ty + i) * kLd + 4 * tx) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[i][c] *= corr[i];
    }
    __syncwarp();   // a warp reads only the P rows that it wrote
    product<D>(sP, sV, ty, tx, o);
  }
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = l[i] > 0.0f ? 1.0f / l[i] : (l[i] == 0.0f ? 0.0f : l[i]);   // NaN stays NaN
    const int r = q0 + 4 * ty + i;
    if (tx == 0 && r < a.S) a.lse[(size_t)bh * a.S + r] = l[i] == 0.0f ? INFINITY : (m[i] + log2f(l[i])) * kAttnLn2;
  }
  store_rows<D>(a.o, b, h, q0, a.S, a.d, ty, tx, o, f);
}

template <int D>
__global__ void __launch_bounds__(kThr) attn_bwd_kernel(const __grid_constant__ AttnOp a) {
  extern __shared__ __align__(16) float sm[];
  float* sA1 = sm;                 // stationary rows: K, V or Q, dO
  float* sA2 = sA1 + D * kLd;
  float* sB1 = sA2 + D * kLd;      // moving columns: Q, dO or K, V
  float* sB2 = sB1 + D * kLd;
  float* sP = sB2 + D * kLd;
  float* sD = sP + kT * kLd;
  float* sBins = sD + kT * kLd;    // [buckets] (query rows)
  pdl_wait();
  pdl_launch_dependents();
  const int nt = (a.S + kT - 1) / kT, items = a.B * a.nh * nt;
  const bool keys = (int)blockIdx.x < items;
  const int it = keys ? blockIdx.x : blockIdx.x - items;
  const int bh = it / nt, ri = it - bh * nt, r0 = ri * kT, b = bh / a.nh, h = bh - b * a.nh;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int mb = a.mask_seqs == 1 ? 0 : b;
  const float* vec = a.vec ? bias_copy(a, h, 0, 0) : nullptr;
  const float* mask = a.maskx + (size_t)mb * a.Sp;
  const int* flags = a.flags + mb * (a.Sp / kAttnFlagKeys);
  const float* nlse = a.stats + (size_t)bh * 2 * a.Sp;
  const float* nd = nlse + 64;
  float acc1[4][D / 16] = {}, acc2[4][D / 16] = {};
  const bool grad = !keys && a.dpart;
  if (grad)
    for (int u = threadIdx.x; u < a.buckets; u += kThr) sBins[u] = 0.0f;
  load_t<D>(sA1, keys ? a.k : a.q, b, h, r0, a.S, a.d);
  load_t<D>(sA2, keys ? a.v : a.dout, b, h, r0, a.S, a.d);
  const bool none = keys && flags[r0 / kAttnFlagKeys] == 2;   // dK = dV = 0
  for (int c0 = 0; c0 < a.S && !none; c0 += kT) {
    if (!keys && flags[c0 / kAttnFlagKeys] == 2) continue;
    __syncthreads();
    load_t<D>(sB1, keys ? a.q : a.k, b, h, c0, a.S, a.d);
    load_t<D>(sB2, keys ? a.dout : a.v, b, h, c0, a.S, a.d);
    __syncthreads();
    float s[4][4], dp[4][4];
    scores<D>(sA1, sB1, ty, tx, s);
    scores<D>(sA2, sB2, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = r0 + 4 * ty + i, col = c0 + 4 * tx + j;
        const int qi = keys ? col : row, kj = keys ? row : col;   // both below Sp
        const float bias = vec ? bias_at(a, vec, kj - qi) : 0.0f;
        const int st = (qi >> 6) * 128 + (qi & 63);
        const float mk = mask[kj], nl = nlse[st];
        // a removed key, an empty row: p = 0
        const float p = mk == -INFINITY || nl == -INFINITY ? 0.0f : exp2f(fmaf(s[i][j], a.c2, bias + mk) + nl);
        s[i][j] = p;
        dp[i][j] = p == 0.0f ? 0.0f : p * (dp[i][j] + nd[st]);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      *reinterpret_cast<float4*>(sP + (4 * ty + i) * kLd + 4 * tx) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
      *reinterpret_cast<float4*>(sD + (4 * ty + i) * kLd + 4 * tx) =
          make_float4(dp[i][0], dp[i][1], dp[i][2], dp[i][3]);
    }
    __syncwarp();
    if (keys) product<D>(sP, sB2, ty, tx, acc2);   // dV
    product<D>(sD, sB1, ty, tx, acc1);             // dK or dQ
    if (grad) {
      // diagonals of the tile into sP (free in this mode), then by bucket
      __syncthreads();
      const int x = (int)threadIdx.x - (kT - 1);   // column minus row
      if (threadIdx.x < 2 * kT - 1) {
        float t = 0.0f;
        for (int i = max(0, -x); i < min(kT, kT - x); ++i) t += sD[i * kLd + i + x];
        sP[threadIdx.x] = t;
      }
      __syncthreads();
      for (int u = threadIdx.x; u < a.buckets; u += kThr) {
        const int x0 = c0 - r0 - (kT - 1);         // diagonal of sP[0]
        const int from = max(a.lo[u] - x0, 0);
        const int to = (int)min((long long)a.lo[u] + a.n[u] - x0, (long long)(2 * kT - 1));
        float t = 0.0f;
        for (int y = from; y < to; ++y) t += sP[y];
        sBins[u] += t;
      }
    }
  }
  const float one[4] = {1.f, 1.f, 1.f, 1.f}, sc[4] = {a.scale, a.scale, a.scale, a.scale};
  store_rows<D>(keys ? a.dk : a.dq, b, h, r0, a.S, a.d, ty, tx, acc1, sc);
  if (keys) store_rows<D>(a.dv, b, h, r0, a.S, a.d, ty, tx, acc2, one);
  if (grad) {
    __syncthreads();
    for (int u = threadIdx.x; u < a.buckets; u += kThr)
      a.dpart[((size_t)bh * a.ditems + ri) * a.buckets + u] = sBins[u];
  }
}

template <int D>
void fwd(const AttnOp& a, cudaStream_t s) {
  constexpr int smem = (3 * D + kT) * kLd * 4;
  static std::atomic<uint64_t> ready{0};
  allow_smem(attn_fwd_kernel<D>, smem, ready);
  launch_pdl(attn_fwd_kernel<D>, a.B * a.nh * ((a.S + kT - 1) / kT), kThr, smem, s, a);
  count_launch();
}
template <int D>
void bwd(const AttnOp& a, cudaStream_t s) {
  constexpr int smem = (4 * D + 2 * kT) * kLd * 4 + kAttnMaxBuckets * 4;
  static std::atomic<uint64_t> ready{0};
  allow_smem(attn_bwd_kernel<D>, smem, ready);
  launch_pdl(attn_bwd_kernel<D>, 2 * a.B * a.nh * ((a.S + kT - 1) / kT), kThr, smem, s, a);
  count_launch();
}

}  // namespace

void attention_f32_fwd_run(const AttnOp& a, cudaStream_t s) {
  if (a.d <= 16) fwd<16>(a, s);
  else if (a.d <= 32) fwd<32>(a, s);
  else if (a.d <= 64) fwd<64>(a, s);
  else fwd<128>(a, s);
}

void attention_f32_bwd_run(const AttnOp& a, cudaStream_t s) {
  if (a.d <= 16) bwd<16>(a, s);
  else if (a.d <= 32) bwd<32>(a, s);
  else if (a.d <= 64) bwd<64>(a, s);
  else bwd<128>(a, s);
}

}  // namespace tlp
