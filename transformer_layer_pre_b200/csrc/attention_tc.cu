// attention_tc.cu — attention with a relative position bias on the tensor
// cores (tcgen05), 16-bit storage, any head dim up to 128 that is a multiple
// of 8.  The math, and the prepared inputs, are at the top of attention.cuh.
//
// Head dims below a kernel's D (64 or 128) are padded by the TMA unit: the
// box is D wide, columns past the head dim read as 0 and are not written.
// Rows past the sequence likewise, so ragged ends need no code but the mask.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "attention.cuh"
#include "kernels.h"
#include "profile.h"
#include "sm100.cuh"

namespace tlp {

using namespace sm100;

namespace {

// error word of these kernels' bounded waits (layout in sm100.cuh)
__device__ __align__(16) int g_attention_err[4];

constexpr int kRegion = 16384;    // [128 rows][64] 16-bit, 128-byte swizzle

__device__ __forceinline__ float ex2f(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// x[0..1] = x[0..1] * m + w, in one packed instruction
__device__ __forceinline__ void fma_to(float* x, float m, float2 w) {
  const float2 y = __ffma2_rn(make_float2(x[0], x[1]), f2(m), w);
  x[0] = y.x;
  x[1] = y.y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<half_t>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<bf16_t>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 32 TMEM columns, no wait (the caller waits once for several).
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32f(uint32_t taddr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
      "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
      "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]),
      "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]),
      "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]),
      "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]),
      "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
      "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
      : "memory");
}
// 8 TMEM columns times f, in place (few registers: the caller holds a tile).
__device__ __forceinline__ void tmem_scale8(uint32_t taddr, float f) {
  float v[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "r"(taddr));
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= f;
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Descriptors.  K-major: rows x D, K step kk of 16 columns, `region` bytes
// between 64-column groups.  MN-major: K runs along the rows, 16 per step.
__device__ __forceinline__ uint64_t desc_k(uint32_t base, int kk, int region) {
  return smem_desc_sw128(base + (kk >> 2) * region + (kk & 3) * 32, 16, 1024);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t base, int kk, int region) {
  return smem_desc_sw128(base + kk * 2048, region, 1024);
}

// Waits until the last of `issued` loads into each slot of a ring has landed
// (the wind-down after a wait that gave up).
template <int R>
__device__ __forceinline__ void drain(uint64_t* full, uint32_t issued) {
  for (uint32_t i = 0; i < R; ++i)
    if (issued > i) mbar_wait(&full[i], ((issued - 1 - i) / R) & 1, nullptr, 0);
}

// What a consumer has to know of one tile, left in shared memory by the
// producer warp.
struct alignas(16) TileInfo {
  int tile;        // column tile, -1: the item has none
  int bits;
  float bias;      // the one bias of a tile beyond the last bucket's border (0 without a table)
  int item;        // running number of the item in this block
};
enum { kLast = 1, kNear = 2, kMixed = 4, kFirst = 8, kKeys = 16, kAhead = 32, kEnd = 64 };

// Walks the column tiles of an item that hold a key which is not removed;
// every lane of the warp calls it.  PER flags of 64 keys per tile.
template <int PER>
struct LiveTiles {
  const int* flags;
  int n, lane, group;
  uint32_t live, mixed;
  __device__ LiveTiles(const int* f, int n_, int lane_) : flags(f), n(n_), lane(lane_), group(-1), live(0), mixed(0) {}
  __device__ void load(int g) {
    group = g;
    const int t = g * 32 + lane;
    int f0 = 2, f1 = 2;
    if (t < n) {
      f0 = flags[t * PER];
      f1 = flags[t * PER + PER - 1];
    }
    live = __ballot_sync(0xffffffffu, f0 != 2 || f1 != 2);
    mixed = __ballot_sync(0xffffffffu, f0 != 0 || f1 != 0);
  }
  // the first one at or after j (n: none); mix: whether its mask has to be read
  __device__ int next(int j, bool& mix) {
    while (j < n) {
      if ((j >> 5) != group) load(j >> 5);
      const uint32_t m = live >> (j & 31);
      if (m) {
        j += __ffs(m) - 1;
        mix = (mixed >> (j & 31)) & 1u;
        return j;
      }
      j = (j | 31) + 1;
    }
    return n;
  }
};

// ============================================================================ forward
// Blocks of six warps, four on an SM (D = 64; two for D = 128), each walking
// items (sequence, head, 128 queries) over tiles of 64 (128) keys: while one
// block's softmax fills the special-function units, the others' products and
// loads are under way.  Warps 0-3: softmax, one query row (TMEM lane) per
// thread; 4: TMA; 5: MMA.  TMEM: S, P over S once it is read, O.
//
// Online softmax with a lazy reference: P = 2^(x - ref), ref the row maximum
// when O was last rescaled; O and the row sum are rescaled only once the
// maximum has grown by more than 2^8, so P stays below 256 and most tiles
// skip it.  P is rounded to the storage type (at most half a step, relative)
// for its product with V; the row sum takes the unrounded P.
//
// The bias is one number for a tile beyond the last bucket's border; else the
// tile's 255 diagonals are staged as four copies shifted by one float each, so
// that every row reads its run of 128 in aligned float4 without bank
// conflicts.
template <int D>
struct Fwd {
  static constexpr int kTK = D == 64 ? 64 : 128;                    // keys per tile
  static constexpr int kBlocks = D == 64 ? 4 : 2;                   // per SM
  static constexpr int kCols = D == 64 ? 128 : 256;                 // TMEM columns: S with P over it, O
  static constexpr uint32_t kO = kTK;
  static constexpr int kQBytes = D / 64 * kRegion;
  static constexpr int kKvRegion = kTK * 128;
  static constexpr int kKvBytes = D / 64 * kKvRegion;
  static constexpr int kKv = D == 64 ? 2 : 1;
  static constexpr int kAux = 2;
  static constexpr int kRun = kTK + 128;                            // diagonals of a tile, rounded up
  static constexpr int kWin = kRun + 8;                             // floats of a window copy, 8 banks apart
  static constexpr int kAuxBytes = 4 * kWin * 4 + kTK * 4 + 16;
  static constexpr int kSmem = kQBytes + 2 * kKv * kKvBytes + kAux * kAuxBytes + 208;
};
static_assert(4 * (Fwd<64>::kSmem + 1024) <= 228 * 1024 && 2 * (Fwd<128>::kSmem + 1024) <= 228 * 1024,
              "the blocks of an SM do not fit its shared memory");
constexpr int kFwdThreads = 192;
constexpr float kRescale = 8.0f;

template <typename T, int D>
__global__ void __launch_bounds__(kFwdThreads, Fwd<D>::kBlocks)
    attention_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                         const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to,
                         const __grid_constant__ AttnOp a) {
  using C = Fwd<D>;
  // the only shared memory of the kernel: its start is 1024-byte aligned
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sQ = smem_raw;
  uint8_t* sK = sQ + C::kQBytes;
  uint8_t* sV = sK + C::kKv * C::kKvBytes;
  uint8_t* sAux = sV + C::kKv * C::kKvBytes;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sAux + C::kAux * C::kAuxBytes);
  uint64_t *q_full = bar, *q_empty = q_full + 1, *k_full = q_empty + 1, *k_empty = k_full + C::kKv,
           *v_full = k_empty + C::kKv, *v_empty = v_full + C::kKv, *aux_full = v_empty + C::kKv,
           *aux_empty = aux_full + C::kAux, *s_full = aux_empty + C::kAux, *p_full = s_full + 1, *pv_done = p_full + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(pv_done + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* err = g_attention_err;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < C::kKv; ++i) {
      mbar_init(&k_full[i], 1), mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1), mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < C::kAux; ++i) mbar_init(&aux_full[i], 1), mbar_init(&aux_empty[i], 5);
    mbar_init(s_full, 1);
    mbar_init(p_full, 4);
    mbar_init(pv_done, 1);
    fence_barrier_init();
  }
  if (warp == 5) tmem_alloc(tslot, C::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  pdl_wait();
  pdl_launch_dependents();

  const int nq = (a.S + 127) / 128, nk = (a.S + C::kTK - 1) / C::kTK;
  const int nitems = a.B * a.nh * nq;
  auto info_of = [&](uint32_t g) -> TileInfo* {
    return reinterpret_cast<TileInfo*>(sAux + (g % C::kAux) * C::kAuxBytes + 4 * C::kWin * 4 + C::kTK * 4);
  };

  if (warp == 4) {
    // ---- producer
    uint32_t g = 0, kc = 0;      // entries and loaded tiles so far
    uint32_t nq_issued = 0, nk_issued = 0, nv_issued = 0, g_issued = 0;
    int n = 0;
    bool ok = true;
    for (int it = blockIdx.x; it < nitems && ok; it += gridDim.x, ++n) {
      const int bh = it / nq, i = it - bh * nq, b = bh / a.nh, h = bh - b * a.nh;
      const int mb = a.mask_seqs == 1 ? 0 : b;
      const float* vec = a.vec ? bias_copy(a, h, 0, 0) : nullptr;
      const float behind = vec ? vec[a.vec_off - a.sat] : 0.0f, ahead = vec ? vec[a.vec_off + a.sat] : 0.0f;
      if (lane == 0) {
        ok = mbar_wait(q_empty, (n & 1) ^ 1, err, 201);
        if (ok) {
          ++nq_issued;
          mbar_arrive_expect_tx(q_full, C::kQBytes);
          for (int c = 0; c < D / 64; ++c) tma_load_4d(sQ + c * kRegion, &tq, q_full, c * 64, i * 128, h, b);
        }
      }
      LiveTiles<C::kTK / kAttnFlagKeys> tiles(a.flags + mb * (a.Sp / kAttnFlagKeys), nk, lane);
      bool mix = false;
      int j = tiles.next(0, mix);
      const bool none = j == nk;
      bool first = true;
      do {
        bool nmix = false;
        const int jn = none ? nk : tiles.next(j + 1, nmix);
        if (lane == 0 && ok) {
          const int as = g % C::kAux;
          TileInfo t;
          t.tile = none ? -1 : j;
          t.item = n;
          t.bits = (jn == nk ? kLast : 0) | (first ? kFirst : 0);
          t.bias = 0.0f;
          const int x0 = j * C::kTK - i * 128;   // diagonal of the tile's corner
          bool near = false;
          if (!none) {
            if (mix) t.bits |= kMixed;
            if (vec) {
              if (x0 - 127 >= a.sat) t.bias = ahead;
              else if (x0 + C::kTK - 1 <= -a.sat) t.bias = behind;
              else near = true;
            }
            const int ks = kc % C::kKv;
            if ((ok = mbar_wait(&k_empty[ks], ((kc / C::kKv) & 1) ^ 1, err, 202))) {
              ++nk_issued;
              mbar_arrive_expect_tx(&k_full[ks], C::kKvBytes);
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(sK + ks * C::kKvBytes + c * C::kKvRegion, &tk, &k_full[ks], c * 64, j * C::kTK, h, b);
            }
          }
          if (near) t.bits |= kNear;
          if (ok && (ok = mbar_wait(&aux_empty[as], ((g / C::kAux) & 1) ^ 1, err, 203))) {
            uint8_t* ax = sAux + as * C::kAuxBytes;
            *info_of(g) = t;
            const bool mk = !none && mix;
            ++g_issued;
            mbar_arrive_expect_tx(&aux_full[as], (near ? 4 * C::kRun * 4 : 0) + (mk ? C::kTK * 4 : 0));
            if (near)
              for (int s = 0; s < 4; ++s)
                bulk_load_1d(ax + s * C::kWin * 4, bias_copy(a, h, 0, s) + x0 - 128 + a.vec_off, C::kRun * 4,
                             &aux_full[as]);
            if (mk) bulk_load_1d(ax + 4 * C::kWin * 4, a.maskx + (size_t)mb * a.Sp + j * C::kTK, C::kTK * 4, &aux_full[as]);
          }
          if (ok && !none) {
            const int ks = kc % C::kKv;
            if ((ok = mbar_wait(&v_empty[ks], ((kc / C::kKv) & 1) ^ 1, err, 204))) {
              ++nv_issued;
              mbar_arrive_expect_tx(&v_full[ks], C::kKvBytes);
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(sV + ks * C::kKvBytes + c * C::kKvRegion, &tv, &v_full[ks], c * 64, j * C::kTK, h, b);
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        first = false;
        ++g;
        if (!none) ++kc;
        j = jn;
        mix = nmix;
      } while (ok && j < nk);
    }
    if (!ok && lane == 0) {
      // a wait gave up: what was issued lands before the block exits
      drain<1>(q_full, nq_issued);
      drain<C::kKv>(k_full, nk_issued);
      drain<C::kKv>(v_full, nv_issued);
      drain<C::kAux>(aux_full, g_issued);
    }
  } else if (warp == 5) {
    if (lane == 0) {
      const bool bf = std::is_same<T, bf16_t>::value;
      const uint32_t id_s = idesc_f16(128, C::kTK, bf, false, false);
      const uint32_t id_o = idesc_f16(128, D, bf, false, true);
      // descriptors of slot 0; a K step, a 64-column region and a slot are
      // offsets of the address field (16-byte units)
      const uint64_t dq = desc_k(smem_u32(sQ), 0, kRegion), dk = desc_k(smem_u32(sK), 0, C::kKvRegion),
                     dv = desc_mn(smem_u32(sV), 0, C::kKvRegion);
      uint32_t g = 0, kc = 0;
      int n = 0;
      bool ok = true;
      TileInfo t;
      auto next_info = [&](uint32_t e) -> bool {
        const int as = e % C::kAux;
        if (!mbar_wait(&aux_full[as], (e / C::kAux) & 1, err, 213)) return false;
        t = *info_of(e);
        mbar_arrive(&aux_empty[as]);
        return t.tile < 0 || mbar_wait(&k_full[kc % C::kKv], (kc / C::kKv) & 1, err, 216);
      };
      for (int it = blockIdx.x; it < nitems && ok; it += gridDim.x, ++n) {
        if (!(ok = next_info(g)) || !(ok = mbar_wait(q_full, n & 1, err, 214))) break;
        for (;; ++g) {
          const bool last = t.bits & kLast, first = t.bits & kFirst;
          if (t.tile < 0) {
            // nothing to multiply: the phases go on
            mbar_arrive(s_full);
            if (!(ok = mbar_wait(p_full, g & 1, err, 211))) break;
            mbar_arrive(pv_done);
            break;
          }
          const int ks = kc % C::kKv;
          const uint32_t kp = (kc / C::kKv) & 1;
          ++kc;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_f16(tmem, dq + (kk >> 2) * (kRegion >> 4) + (kk & 3) * 2,
                    dk + ks * (C::kKvBytes >> 4) + (kk >> 2) * (C::kKvRegion >> 4) + (kk & 3) * 2, id_s, kk > 0);
          mma_commit(s_full);
          mma_commit(&k_empty[ks]);
          // what the next tile needs, ahead of the wait for P (an item's first
          // tile waits for the rows of the item before)
          if (!last && !(ok = next_info(g + 1))) break;
          if (!(ok = mbar_wait(&v_full[ks], kp, err, 212))) break;
          // P lies over S, so its product comes before the next Q K^T
          if (!(ok = mbar_wait(p_full, g & 1, err, 211))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < C::kTK / 16; ++kk)
            mma_f16_ts(tmem + C::kO, tmem + kk * 8, dv + ks * (C::kKvBytes >> 4) + kk * 128, id_o,
                       (!first || kk > 0) ? 1u : 0u);
          if (last) mma_commit(pv_done);
          mma_commit(&v_empty[ks]);
          if (last) break;
        }
        ++g;
      }
    }
  } else {
    // ---- softmax
    const int r = threadIdx.x;
    const uint32_t lo = (uint32_t)(warp * 32) << 16;
    const float c2 = a.c2;
    uint32_t g = 0;
    int n = 0;
    bool ok = true;
    for (int it = blockIdx.x; it < nitems && ok; it += gridDim.x, ++n) {
      const int bh = it / nq, i = it - bh * nq, b = bh / a.nh, h = bh - b * a.nh;
      float ref = -INFINITY, l = 0.0f;
      bool last = false;
      for (; !last; ++g) {
        const int as = g % C::kAux;
        if (!(ok = mbar_wait_warp(&aux_full[as], (g / C::kAux) & 1, err, 221))) break;
        const TileInfo t = *info_of(g);
        last = t.bits & kLast;
        if (!(ok = mbar_wait_warp(s_full, g & 1, err, 222))) break;
        if (t.tile < 0) {
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&aux_empty[as]);
            mbar_arrive(p_full);
          }
          continue;
        }
        tc_fence_after();
        // first pass: the row maximum.  Where the bias or the mask varies along
        // the row, the finished scores go back to TMEM, so that the second pass
        // reads no shared memory.
        float mul = c2, add = t.bias, m0 = -INFINITY, m1 = -INFINITY;
        const uint8_t* ax = sAux + as * C::kAuxBytes;
        if (t.bits & (kNear | kMixed)) {
          // row r's run of diagonals starts at 128 - r of the window
          const int start = 128 - r;
          const float* wnd = reinterpret_cast<const float*>(ax) + (start & 3) * C::kWin + (start & ~3);
          const float* mrow = reinterpret_cast<const float*>(ax + 4 * C::kWin * 4);
          const bool near = t.bits & kNear, mixed = t.bits & kMixed;
          mul = 1.0f;
          add = 0.0f;
#pragma unroll 1
          for (int c = 0; c < C::kTK / 32; ++c) {
            float x[32];
            tmem_ld32_nowait(tmem + lo + c * 32, x);
            tmem_ld_wait();
            if (near) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 w = *reinterpret_cast<const float4*>(wnd + c * 32 + e);
                fma_to(x + e, c2, make_float2(w.x, w.y));
                fma_to(x + e + 2, c2, make_float2(w.z, w.w));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 2) fma_to(x + e, c2, f2(t.bias));
            }
            if (mixed) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 w = *reinterpret_cast<const float4*>(mrow + c * 32 + e);
                fma_to(x + e, 1.0f, make_float2(w.x, w.y));
                fma_to(x + e + 2, 1.0f, make_float2(w.z, w.w));
              }
            }
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              m0 = max3(m0, x[e], x[e + 1]);
              m1 = max3(m1, x[e + 2], x[e + 3]);
            }
            tmem_st32f(tmem + lo + c * 32, x);
          }
          tmem_store_wait();
        } else {
#pragma unroll 1
          for (int c = 0; c < C::kTK / 32; ++c) {
            float x[32];
            tmem_ld32_nowait(tmem + lo + c * 32, x);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              m0 = max3(m0, x[e], x[e + 1]);
              m1 = max3(m1, x[e + 2], x[e + 3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&aux_empty[as]);
        const float top = fmaf(fmaxf(m0, m1), mul, add);
        // O holds the products of every tile before: they were issued ahead of this Q K^T
        const float mnew = fmaxf(ref, top);
        if (t.bits & kFirst) {
          ref = mnew;
        } else if (__any_sync(0xffffffffu, mnew > ref + kRescale)) {
          const float f = mnew > ref + kRescale ? ex2f(ref - mnew) : 1.0f;
          if (f != 1.0f) ref = mnew;
          l *= f;
#pragma unroll 1
          for (int c = 0; c < D; c += 8) tmem_scale8(tmem + lo + C::kO + c, f);
        }
        const float sub = add - (ref == -INFINITY ? 0.0f : ref);
        float2 sum0 = f2(0.0f), sum1 = f2(0.0f);
#pragma unroll 1
        for (int c = 0; c < C::kTK / 32; ++c) {
          float x[32];
          tmem_ld32_nowait(tmem + lo + c * 32, x);
          tmem_ld_wait();
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = __ffma2_rn(make_float2(x[2 * e], x[2 * e + 1]), f2(mul), f2(sub));
            const float2 p = make_float2(ex2f(y.x), ex2f(y.y));
            if (e & 1) sum1 = __fadd2_rn(sum1, p);
            else sum0 = __fadd2_rn(sum0, p);
            w[e] = pack2<T>(p.x, p.y);
          }
          // over S columns that this thread has read
          tmem_st16u(tmem + lo + c * 16, w);
        }
        sum0 = __fadd2_rn(sum0, sum1);
        l += sum0.x + sum0.y;
        tmem_store_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      if (!ok) break;
      // ---- the item's rows: O / l through the Q tile (no product reads it any more)
      if (!(ok = mbar_wait_warp(pv_done, n & 1, err, 225))) break;
      tc_fence_after();
      uint8_t* stage = sQ;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        tmem_ld32_nowait(tmem + lo + C::kO + c * 32, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // an empty row may never have had a product
            const float y0 = l == 0.0f ? 0.0f : o[e * 8 + 2 * k] * inv;
            const float y1 = l == 0.0f ? 0.0f : o[e * 8 + 2 * k + 1] * inv;
            w[k] = pack2<T>(y0, y1);
          }
          const int ch = c * 4 + e;   // 16-byte chunk of the row
          *reinterpret_cast<uint4*>(stage + (ch >> 3) * kRegion + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      tc_fence_before();
      const int row = i * 128 + r;
      if (row < a.S) a.lse[(size_t)bh * a.S + row] = l == 0.0f ? INFINITY : (ref + log2f(l)) * kAttnLn2;
      fence_proxy_async_smem();
      named_barrier(1, 128);
      if (threadIdx.x == 0) {
        for (int c = 0; c < D / 64; ++c) tma_store_4d(&to, stage + c * kRegion, c * 64, i * 128, h, b);
        bulk_commit();
        bulk_wait_read<0>();
        mbar_arrive(q_empty);
      }
    }
    if (threadIdx.x == 0) bulk_wait_all();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, C::kCols);
}

// ------------------------------------------------------------------ host side
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// (dim, token, head, batch) map in boxes of 64 dims x `rows` tokens.
bool encode(CUtensorMap* m, const AttnView& v, const AttnOp& a, bool bf16, int rows) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)a.d, (cuuint64_t)a.S, (cuuint64_t)a.nh, (cuuint64_t)a.B};
  const cuuint64_t strides[3] = {(cuuint64_t)v.st * 2, (cuuint64_t)v.sh * 2, (cuuint64_t)v.sb * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, v.p, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
  int dev = 0, n = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

template <typename T, int D>
bool fwd(const AttnOp& a, cudaStream_t s) {
  const bool bf = std::is_same<T, bf16_t>::value;
  CUtensorMap mq, mk, mv, mo;
  if (!encode(&mq, a.q, a, bf, 128) || !encode(&mk, a.k, a, bf, Fwd<D>::kTK) ||
      !encode(&mv, a.v, a, bf, Fwd<D>::kTK) || !encode(&mo, a.o, a, bf, 128))
    return false;
  cudaFuncSetAttribute(attention_fwd_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Fwd<D>::kSmem);
  const int items = a.B * a.nh * ((a.S + 127) / 128);
  launch_pdl(attention_fwd_kernel<T, D>, std::min(items, Fwd<D>::kBlocks * sm_count()), kFwdThreads, Fwd<D>::kSmem, s, mq, mk, mv, mo, a);
  count_launch();
  return true;
}

}  // namespace

bool attention_tc_fwd_run(int dt, const AttnOp& a, cudaStream_t s) {
  if (dt == DT_F16) return a.d <= 64 ? fwd<half_t, 64>(a, s) : fwd<half_t, 128>(a, s);
  return a.d <= 64 ? fwd<bf16_t, 64>(a, s) : fwd<bf16_t, 128>(a, s);
}

int attention_tc_take_error() {
  int v = 0;
  cudaMemcpyFromSymbol(&v, g_attention_err, sizeof(int));
  if (v) {
    const int z = 0;
    cudaMemcpyToSymbol(g_attention_err, &z, sizeof(int));
  }
  return v;
}

void attention_tc_set_wait_limit(uint64_t ns) { cudaMemcpyToSymbol(g_attention_err, &ns, sizeof(ns), 2 * sizeof(int)); }

}  // namespace tlp
