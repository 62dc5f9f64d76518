// attention.cu — the attention entry points: argument checks, the workspace,
// the launch that prepares it, and the sum of the bias table's gradient.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/tlp.h"
#include "attention.cuh"
#include "kernels.h"
#include "overlap.h"
#include "profile.h"

namespace tlp {
namespace {

// One launch fills the workspace (layout at the top of attention.cuh).
// Blocks [0, nmask): 256 keys each of maskx and flags.  Then nvec blocks: 256
// diagonals of one head each, written to every copy.  Then (backward) nzero
// blocks that clear dpart, and blocks of prep_rows(G) * 256 / G tokens of one
// sequence and head for stats (and, float16, smax), G lanes per row reading 16
// bytes each.
// Bound: launch latency (3 us) in the forward and where the backward forms D
// itself; else the latency of a group's loads: O and dO of B16 h16 d64 S512, 33.6
// MB, 15 us (2.2 TB/s), with V of float16, 50.3 MB, 18 us.  Eight rows in flight
// per group made a whole backward 6 % slower.
template <typename T, int G>
__global__ void __launch_bounds__(kPrepThreads) attn_prep_kernel(const __grid_constant__ AttnOp a, int nmask, int nvec, int nzero) {
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  int blk = blockIdx.x;
  if (blk < nmask) {
    __shared__ int any[kPrepThreads / kAttnFlagKeys], zero[kPrepThreads / kAttnFlagKeys];
    const int per = (a.Sp + kPrepThreads - 1) / kPrepThreads;
    const int b = blk / per, j = (blk - b * per) * kPrepThreads + tid;
    const int g = tid / kAttnFlagKeys;
    if (tid < kPrepThreads / kAttnFlagKeys) any[tid] = 0, zero[tid] = 1;
    __syncthreads();
    if (j < a.Sp) {
      float v = -INFINITY;
      if (j < a.S) {
        const float m = a.mask ? a.mask[(size_t)b * a.S + j] : 0.0f;
        v = m <= kAttnMasked ? -INFINITY : m * kAttnLog2e;
      }
      a.maskx[(size_t)b * a.Sp + j] = v;
      if (v != -INFINITY) any[g] = 1;
      if (v != 0.0f) zero[g] = 0;
    }
    __syncthreads();
    if (j < a.Sp && tid % kAttnFlagKeys == 0)
      a.flags[b * (a.Sp / kAttnFlagKeys) + j / kAttnFlagKeys] = zero[g] ? 0 : (any[g] ? 1 : 2);
    return;
  }
  blk -= nmask;
  if (blk < nvec) {
    const int per = (a.vec_len + kPrepThreads - 1) / kPrepThreads;
    const int h = blk / per, X = (blk - h * per) * kPrepThreads + tid;
    if (X >= a.vec_len) return;
    const int x = max(-a.sat, min(a.sat, X - a.vec_off));   // key minus query
    // the last bucket of the side that begins at or before the distance
    const int half = a.buckets / 2, dist = abs(x);
    int u = 0;
    for (int end = half - 1; u < end;) {
      const int mid = (u + end + 1) >> 1;
      if (a.lo[half + mid] <= dist) u = mid;
      else end = mid - 1;
    }
    if (x > 0) u += half;
    const float v = to_f(static_cast<const T*>(a.table)[(size_t)u * a.nh + h]) * kAttnLog2e;
    if (h == 0) a.bid[X] = (uint8_t)u;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      float* base = a.vec + ((size_t)h * 8 + s) * a.vec_len;
      if (X - s - 1 >= 0) base[X - s - 1] = v;
      // direction 1: diagonal -x
      const int Y = 2 * a.vec_off - X - s - 1;
      if (Y >= 0 && Y < a.vec_len) base[(size_t)4 * a.vec_len + Y] = v;
    }
    return;
  }
  blk -= nvec;
  if (blk < nzero) {
    const long long total = (long long)a.B * a.nh * a.ditems * a.buckets;
    for (long long i = (long long)blk * kPrepThreads + tid; i < total; i += (long long)nzero * kPrepThreads) a.dpart[i] = 0.0f;
    return;
  }
  blk -= nzero;
  constexpr bool kMax = std::is_same<T, half_t>::value;
  constexpr int kEl = 16 / sizeof(T), kRows = prep_rows(G), kStep = kPrepThreads / G;
  const int lane = tid % G;
  // neighbouring blocks take the heads of the same tokens, which lie side by side in (B, S, heads, d) memory
  const int per = a.Sp / (kRows * kStep), bc = blk / a.nh, h = blk - bc * a.nh, b = bc / per, chunk = bc - b * per;
  const int bh = b * a.nh + h;
  const int i0 = chunk * kRows * kStep + tid / G;
  float t[kRows];                                       // dO.O
  __half2 mdo[kRows], mv[kRows];                        // largest |dO| and |V|, of even and odd dims
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int i = i0 + k * kStep;
    t[k] = 0.0f;
    mdo[k] = mv[k] = __float2half2_rn(0.0f);
    if (i < a.S)
      for (int c = lane * kEl; c < a.d; c += G * kEl) {
        auto at = [&](const AttnView& v) {
          return *reinterpret_cast<const uint4*>(static_cast<const T*>(v.p) + (size_t)b * v.sb + (size_t)i * v.st +
                                                 (size_t)h * v.sh + c);
        };
        const uint4 x = at(a.o), y = at(a.dout), z = kMax ? at(a.v) : make_uint4(0u, 0u, 0u, 0u);
        const T *xe = reinterpret_cast<const T*>(&x), *ye = reinterpret_cast<const T*>(&y);
#pragma unroll
        for (int e = 0; e < kEl; ++e) t[k] = fmaf(to_f(xe[e]), to_f(ye[e]), t[k]);
        if (kMax) {
          mdo[k] = max_abs(mdo[k], y);
          mv[k] = max_abs(mv[k], z);
        }
      }
  }
  __half2 most = __float2half2_rn(0.0f);                // of dO, of V
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
#pragma unroll
    for (int w = G / 2; w > 0; w >>= 1) t[k] += __shfl_xor_sync(0xffffffffu, t[k], w);
    const int i = i0 + k * kStep;
    float lse = INFINITY;
    if ((lane == 0 || kMax) && i < a.S) lse = a.lse[(size_t)bh * a.S + i];
    if (lane == 0) {
      float* st = a.stats + (size_t)bh * 2 * a.Sp;
      const int x = (i >> 6) * 128 + (i & 63);
      constexpr float up = sizeof(T) == 2 ? kAttnPUp : 1.0f, up2 = sizeof(T) == 2 ? 8.0f : 0.0f;   // and its log2
      static_assert(kAttnPUp == 256.0f, "up2 is its logarithm");
      st[x] = up2 - lse_log2(lse);
      st[x + 64] = i < a.S ? -t[k] * (1.0f / up) : 0.0f;
    }
    if (kMax && i < a.S) {
      if (lse == INFINITY) mdo[k] = __float2half2_rn(0.0f);
      if (a.mask && a.mask[(size_t)b * a.S + i] <= kAttnMasked) mv[k] = __float2half2_rn(0.0f);
      most = __hmax2(most, fold_max(mdo[k], mv[k]));
    }
  }
  if (kMax) {
    __shared__ __half2 red[kPrepThreads / 32];
    most = warp_max2(most);
    if ((tid & 31) == 0) red[tid >> 5] = most;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int w = 1; w < kPrepThreads / 32; ++w) most = __hmax2(most, red[w]);
      a.smax[(size_t)bh * a.nmax + chunk] = most;
    }
  }
}

// dtable[u, h] (+)= sum over sequences and items of dpart, in a fixed order
// and in float64: a block per head and 32 buckets, a lane per bucket (whole
// lines of dpart), the rows dealt to the warps.  Bound: latency; 4 us for 64 rows per
// head of 16 heads and 32 buckets, 6 for 512.
constexpr int kTableWarps = 32;
__global__ void __launch_bounds__(32 * kTableWarps) attn_table_grad_kernel(const __grid_constant__ AttnOp a) {
  __shared__ double red[kTableWarps][33];
  pdl_wait();
  pdl_launch_dependents();
  const int h = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, u = blockIdx.y * 32 + lane;
  const unsigned rows = (unsigned)a.B * a.ditems, per = a.ditems;   // below 2^30
  double t = 0.0;
  if (u < a.buckets) {
#pragma unroll 8
    for (unsigned r = warp; r < rows; r += kTableWarps) {
      const unsigned b = r / per;
      t += (double)a.dpart[((size_t)(b * a.nh + h) * per + (r - b * per)) * a.buckets + u];
    }
  }
  red[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && u < a.buckets) {
    t = 0.0;
#pragma unroll
    for (int w = 0; w < kTableWarps; ++w) t += red[w][lane];
    float* d = a.dtable + (size_t)u * a.nh + h;
    *d = (float)(a.daccumulate ? (double)*d + t : t);
  }
}

template <typename T, int G>
void prep(const AttnOp& a, bool backward, cudaStream_t s) {
  const int nmask = a.mask_seqs * ((a.Sp + kPrepThreads - 1) / kPrepThreads);
  const int nvec = a.vec ? a.nh * ((a.vec_len + kPrepThreads - 1) / kPrepThreads) : 0;
  const int nzero = backward && a.dpart ? 64 : 0;
  const int nrow = backward ? a.B * a.nh * (a.Sp / (prep_rows(G) * kPrepThreads / G)) : 0;
  launch_pdl(attn_prep_kernel<T, G>, nmask + nvec + nzero + nrow, kPrepThreads, 0, s, a, nmask, nvec, nzero);
  count_launch();
}

template <typename T>
void prep_t(const AttnOp& a, bool backward, cudaStream_t s) {
  // lanes per row of the D = rowsum(dO O) part: 16 bytes each
  const int vecs = a.d * (int)sizeof(T) / 16;
  if (vecs <= 4) prep<T, 4>(a, backward, s);
  else if (vecs <= 8) prep<T, 8>(a, backward, s);
  else prep<T, 16>(a, backward, s);
}

// Bucket of a key n >= 0 positions behind the query (half = buckets of a side).
int side_bucket(long long n, int half, int max_distance) {
  const int first = half / 2;
  if (n < first) return (int)n;
  const double f = std::log((double)n / first) / std::log((double)max_distance / first) * (half - first) + 1e-9;
  return first + (int)std::min((double)(half - first - 1), std::floor(f));
}

// The diagonals of every bucket, and the distance from which on the last one holds.
void bucket_ranges(AttnOp& a, int max_distance) {
  const int half = a.buckets / 2, first = half / 2;
  constexpr int kFar = 1 << 30;
  int from[kAttnMaxBuckets / 2 + 1];   // smallest distance of each bucket of a side
  for (int u = 0; u < half; ++u) {
    if (u <= first) {
      from[u] = u;
      continue;
    }
    long long n = (long long)std::ceil(first * std::pow((double)max_distance / first, (double)(u - first) / (half - first)));
    n = std::max<long long>(n, first);
    while (n > first && side_bucket(n - 1, half, max_distance) >= u) --n;
    while (side_bucket(n, half, max_distance) < u) ++n;
    from[u] = (int)n;
  }
  from[half] = kFar;
  for (int u = 0; u < half; ++u) {
    // keys at or behind the query: diagonals -(from[u+1] - 1) .. -from[u]
    a.n[u] = std::max(0, from[u + 1] - from[u]);
    a.lo[u] = -(from[u + 1] - 1);
    // keys ahead: the same distances, without 0
    const int f = std::max(1, from[u]);
    a.n[half + u] = std::max(0, from[u + 1] - f);
    a.lo[half + u] = f;
  }
  a.sat = std::max(1, from[half - 1]);
}

bool view_ok(const tl_heads* v, int dt, int B, int S, int nh, int d) {
  if (!v || !v->data) return false;
  const int64_t per = dt == DT_F32 ? 4 : 8;   // elements in 16 bytes
  if (reinterpret_cast<uintptr_t>(v->data) & 15) return false;
  const int64_t st[3] = {v->batch, v->token, v->head};
  const int n[3] = {B, S, nh};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (st[i] < d || st[i] % per != 0 || st[i] >= (1ll << 36))) return false;
  return true;
}

// Whether no two entries of an output share memory: sorted by stride, every
// dimension steps over the whole of the ones inside it.
bool disjoint(const tl_heads* v, int B, int S, int nh, int d) {
  struct { int64_t stride; int n; } x[3] = {{v->batch, B}, {v->token, S}, {v->head, nh}};
  std::sort(x, x + 3, [](const auto& l, const auto& r) { return l.stride < r.stride; });
  int64_t span = d;
  for (const auto& e : x) {
    if (e.n == 1) continue;
    if (e.stride < span) return false;
    span += e.stride * (e.n - 1);
  }
  return true;
}

// Strides of dimensions of one entry mean nothing and may hold anything.
AttnView view(const tl_heads* v, int B, int S, int nh, int d) {
  AttnView w;
  w.p = v->data;
  w.sb = B > 1 ? v->batch : (d + 7) / 8 * 8;
  w.st = S > 1 ? v->token : (d + 7) / 8 * 8;
  w.sh = nh > 1 ? v->head : (d + 7) / 8 * 8;
  return w;
}

size_t take(size_t& off, size_t bytes) {
  const size_t at = off;
  off += (bytes + 255) & ~(size_t)255;
  return at;
}

// Checks what does not depend on the tensors and lays out the workspace
// (base null: measures).
tl_status plan(const tl_attention* c, bool backward, char* base, AttnOp& a, size_t& bytes) {
  memset(&a, 0, sizeof(a));
  if (!c || c->dtype < TL_F32 || c->dtype > TL_BF16) return TL_EINVAL;
  if (c->batch <= 0 || c->seq <= 0 || c->heads <= 0) return TL_EINVAL;
  if (c->head_dim <= 0 || c->head_dim > 128 || c->head_dim % 8 != 0) return TL_EINVAL;
  if (!(c->scale >= 0.0f) || isinf(c->scale)) return TL_EINVAL;
  if (reinterpret_cast<uintptr_t>(c->mask) & 3) return TL_EINVAL;
  if (c->bias_table) {
    if (c->buckets < 4 || c->buckets > kAttnMaxBuckets || c->buckets % 2 != 0) return TL_EINVAL;
    if (c->max_distance <= c->buckets / 4 || c->max_distance > (1 << 20)) return TL_EINVAL;
    if (reinterpret_cast<uintptr_t>(c->bias_table) & (dtype_size(c->dtype) - 1)) return TL_EINVAL;
  }
  if (c->seq > (1 << 20) || (long long)c->batch * c->heads * ((c->seq + 127) / 128 * 128) > (1ll << 30))
    return TL_EUNSUPPORTED;
  a.B = c->batch; a.S = c->seq; a.nh = c->heads; a.d = c->head_dim;
  a.Sp = (a.S + 127) / 128 * 128;
  a.scale = c->scale > 0.0f ? c->scale : (float)(1.0 / std::sqrt((double)a.d));
  a.c2 = a.scale * kAttnLog2e;
  a.mask = c->mask;
  a.mask_seqs = c->mask ? a.B : 1;
  size_t off = 0;
  a.maskx = (float*)(base + take(off, (size_t)a.mask_seqs * a.Sp * 4));
  a.flags = (int*)(base + take(off, (size_t)a.mask_seqs * (a.Sp / kAttnFlagKeys) * 4));
  if (c->bias_table) {
    a.table = c->bias_table;
    a.buckets = c->buckets;
    bucket_ranges(a, c->max_distance);
    // no diagonal beyond the sequence is read: windows of 256 diagonals start
    // up to 128 before and end up to 256 after the last one that matters
    const int reach = std::min(a.sat, a.Sp);
    a.vec_off = (reach + 127) / 128 * 128 + 384;
    a.vec_len = 2 * a.vec_off + 128;
    a.sat = reach;
    a.vec = (float*)(base + take(off, (size_t)a.nh * 8 * a.vec_len * 4));
    a.bid = (uint8_t*)(base + take(off, a.vec_len));
  }
  if (backward) {
    const bool one = attn_one_tile(c->dtype, a.S, a.d);
    if (!one) a.stats = (float*)(base + take(off, (size_t)a.B * a.nh * 2 * a.Sp * 4));
    if (!one && c->dtype == TL_F16) {
      a.nmax = a.Sp / attn_prep_rows(a.d);
      a.smax = (__half2*)(base + take(off, (size_t)a.B * a.nh * a.nmax * sizeof(__half2)));
    }
    if (c->bias_table) {
      // one row per item of 64 queries (float32), per softmax warp of one of 128, or per (sequence, head)
      a.ditems = c->dtype == TL_F32 ? (a.S + 63) / 64 : one ? 1 : a.Sp / 128 * 8;
      a.dpart = (float*)(base + take(off, (size_t)a.B * a.nh * a.ditems * a.buckets * 4));
    }
  }
  bytes = off;
  return TL_OK;
}

// Whether every output (the first `outs`) is apart from every other tensor.
bool apart(const ByteRows* x, int outs, int n) {
  for (int i = 0; i < outs; ++i)
    for (int j = i + 1; j < n; ++j)
      if (overlap(x[i], x[j])) return false;
  return true;
}
ByteRows rows_of(const tl_heads* v, const tl_attention* c) {
  return ByteRows(v->data, v->batch, c->batch, v->token, c->seq, v->head, c->heads, c->head_dim, (int)dtype_size(c->dtype));
}
// The dense ones; an absent one is empty.
ByteRows lse_rows(const float* lse, const tl_attention* c) { return ByteRows(lse, (int64_t)c->batch * c->heads * c->seq * 4); }
ByteRows mask_rows(const tl_attention* c) { return ByteRows(c->mask, c->mask ? (int64_t)c->batch * c->seq * 4 : 0); }
ByteRows table_rows(const void* t, const tl_attention* c, size_t es) {
  return ByteRows(t, t ? (int64_t)c->buckets * c->heads * (int64_t)es : 0);
}

}  // namespace

bool attn_one_tile(int dt, int seq, int head_dim) { return dt != DT_F32 && seq <= 128 && head_dim <= 64; }

void attn_prep_run(int dt, const AttnOp& a, bool backward, cudaStream_t s) {
  if (dt == DT_F32) prep_t<float>(a, backward, s);
  else if (dt == DT_F16) prep_t<half_t>(a, backward, s);
  else prep_t<bf16_t>(a, backward, s);
}

void attn_table_grad_run(const AttnOp& a, cudaStream_t s) {
  launch_pdl(attn_table_grad_kernel, dim3(a.nh, (a.buckets + 31) / 32), 32 * kTableWarps, 0, s, a);
  count_launch();
}

}  // namespace tlp

using namespace tlp;

extern "C" {

size_t tl_attention_workspace_bytes(const tl_attention* c, int backward) {
  AttnOp a;
  size_t bytes = 0;
  return plan(c, backward != 0, nullptr, a, bytes) == TL_OK ? bytes : 0;
}

tl_status tl_attention_forward(const tl_attention* c, const tl_heads* q, const tl_heads* k, const tl_heads* v,
                               const tl_heads* o, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  AttnOp a;
  size_t need = 0;
  const tl_status st = plan(c, false, (char*)workspace, a, need);
  if (st != TL_OK) return st;
  const tl_heads* all[4] = {q, k, v, o};
  for (const tl_heads* t : all)
    if (!view_ok(t, c->dtype, a.B, a.S, a.nh, a.d)) return TL_EINVAL;
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3)) return TL_EINVAL;
  if (!disjoint(o, a.B, a.S, a.nh, a.d)) return TL_EINVAL;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < need) return TL_EINVAL;
  const ByteRows parts[8] = {rows_of(o, c), lse_rows(lse, c), ByteRows(workspace, (int64_t)need), rows_of(q, c),
                             rows_of(k, c), rows_of(v, c), mask_rows(c), table_rows(c->bias_table, c, dtype_size(c->dtype))};
  if (!apart(parts, 3, 8)) return TL_EINVAL;
  if (cudaGetLastError() != cudaSuccess) return TL_ECUDA;
  a.q = view(q, a.B, a.S, a.nh, a.d);
  a.k = view(k, a.B, a.S, a.nh, a.d);
  a.v = view(v, a.B, a.S, a.nh, a.d);
  a.o = view(o, a.B, a.S, a.nh, a.d);
  a.lse = lse;
  cudaStream_t s = (cudaStream_t)stream;
  ProfScope p_(PC_ATTN_FWD, s);
  attn_prep_run(c->dtype, a, false, s);
  bool ok = true;
  if (c->dtype == TL_F32) attention_f32_fwd_run(a, s);
  else ok = attention_tc_fwd_run(c->dtype, a, s);
  return ok && cudaGetLastError() == cudaSuccess ? TL_OK : TL_ECUDA;
}

tl_status tl_attention_backward(const tl_attention* c, const tl_heads* q, const tl_heads* k, const tl_heads* v,
                                const tl_heads* o, const tl_heads* dout, const float* lse, const tl_heads* dq,
                                const tl_heads* dk, const tl_heads* dv, float* dtable, int accumulate, void* workspace,
                                size_t workspace_bytes, void* stream) {
  AttnOp a;
  size_t need = 0;
  const tl_status st = plan(c, true, (char*)workspace, a, need);
  if (st != TL_OK) return st;
  const tl_heads* all[8] = {q, k, v, o, dout, dq, dk, dv};
  for (const tl_heads* t : all)
    if (!view_ok(t, c->dtype, a.B, a.S, a.nh, a.d)) return TL_EINVAL;
  for (int i = 5; i < 8; ++i)
    if (!disjoint(all[i], a.B, a.S, a.nh, a.d)) return TL_EINVAL;
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3)) return TL_EINVAL;
  if (dtable && (!c->bias_table || (reinterpret_cast<uintptr_t>(dtable) & 3))) return TL_EINVAL;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < need) return TL_EINVAL;
  const ByteRows parts[13] = {rows_of(dq, c), rows_of(dk, c), rows_of(dv, c), table_rows(dtable, c, 4),
                              ByteRows(workspace, (int64_t)need), rows_of(q, c), rows_of(k, c), rows_of(v, c), rows_of(o, c),
                              rows_of(dout, c), lse_rows(lse, c), mask_rows(c),
                              table_rows(c->bias_table, c, dtype_size(c->dtype))};
  if (!apart(parts, 5, 13)) return TL_EINVAL;
  if (cudaGetLastError() != cudaSuccess) return TL_ECUDA;
  a.q = view(q, a.B, a.S, a.nh, a.d);
  a.k = view(k, a.B, a.S, a.nh, a.d);
  a.v = view(v, a.B, a.S, a.nh, a.d);
  a.o = view(o, a.B, a.S, a.nh, a.d);
  a.dout = view(dout, a.B, a.S, a.nh, a.d);
  a.dq = view(dq, a.B, a.S, a.nh, a.d);
  a.dk = view(dk, a.B, a.S, a.nh, a.d);
  a.dv = view(dv, a.B, a.S, a.nh, a.d);
  a.lse = const_cast<float*>(lse);
  a.dtable = dtable;
  a.daccumulate = accumulate ? 1 : 0;
  if (!dtable) a.dpart = nullptr;
  cudaStream_t s = (cudaStream_t)stream;
  ProfScope p_(PC_ATTN_BWD, s);
  // one tile per sequence and head: its kernel forms D itself and writes every row of dpart
  attn_prep_run(c->dtype, a, !attn_one_tile(c->dtype, a.S, a.d), s);
  bool ok = true;
  if (c->dtype == TL_F32) attention_f32_bwd_run(a, s);
  else ok = attention_tc_bwd_run(c->dtype, a, s);
  if (dtable) attn_table_grad_run(a, s);
  return ok && cudaGetLastError() == cudaSuccess ? TL_OK : TL_ECUDA;
}

}  // extern "C"
