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

// The same for probabilities, which scores so large that float32 rounds them by
// whole units (from 2^23) may bring above float16's end: kept finite.
template <typename T> __device__ __forceinline__ uint32_t pack_p(float lo, float hi) { return pack2<T>(lo, hi); }
template <> __device__ __forceinline__ uint32_t pack_p<half_t>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Bounded wait on an mbarrier that pauses between its polls: polls go through
// the shared memory that the products read their operands from (a tight loop
// of polls in every waiting warp made the backward 14 % slower).
template <int NS>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, int* err, int code) {
  if (mbar_try_wait(bar, parity)) return true;
  if (NS > 0) {
#pragma unroll 1
    for (int i = 0; i < 256; ++i) {
      __nanosleep(NS);
      if (mbar_try_wait(bar, parity)) return true;
    }
  }
  return mbar_wait(bar, parity, err, code);
}
// The same by a whole warp, whose lanes go on together.
template <int NS>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* err, int code) {
  return __all_sync(0xffffffffu, wait_bar<NS>(bar, parity, err, code)) != 0;
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
// when O was last rescaled, less 7; O and the row sum are rescaled only once the
// maximum has grown by more than 2^8, so P stays below 2^15 and most tiles skip
// it.  P is rounded to the storage type (at most half a step, relative) for its
// product with V; the row sum takes the unrounded P.  The 7: float16's subnormals,
// whose rounding is absolute, begin at 2^-21 of the row's maximum instead of
// 2^-14, and what 2^20 small probabilities lose there is at most 2^-12 of the
// largest |V|.  O / l does not see it, and lse takes ref as it was used.
//
// The bias is one number for a tile beyond the last bucket's border; else the
// tile's 255 diagonals are staged as four copies shifted by one float each, so
// that every row reads its run of 128 in aligned float4 without bank
// conflicts.
//
// Bound: the special-function unit (16 exponentials per clock and SM against
// 128 x 64 of them per tile) and the latency of a tile's chain product -> maximum
// -> exponentials -> product.  B4 h16 d64 S2048: 128 us a call (L2 warm; 138 cold),
// 537 TFLOP/s (0.32 of the measured GEMM rate), exponentials 52 % of their unit's
// rate, tensor pipe 26 %; h8 d128: 94 us, 731 TFLOP/s; B64 h16 S128, 67.6 MB: 21
// us cold, 3.2 TB/s.
// Per 128 x 64 tile, when first built: two blocks of 128-key tiles on an SM took
// 168 us, four of 64 keys 146; windows read straight from global memory 159.
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
constexpr float kRescale = 8.0f, kFwdUp = 7.0f;   // log2

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
    mbar_init(s_full, 2);
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
      const float behind = vec ? vec[a.vec_off - a.sat - 1] : 0.0f, ahead = vec ? vec[a.vec_off + a.sat - 1] : 0.0f;
      if (lane == 0) {
        ok = wait_bar<0>(q_empty, (n & 1) ^ 1, err, 201);
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
            if ((ok = wait_bar<0>(&k_empty[ks], ((kc / C::kKv) & 1) ^ 1, err, 202))) {
              ++nk_issued;
              mbar_arrive_expect_tx(&k_full[ks], C::kKvBytes);
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(sK + ks * C::kKvBytes + c * C::kKvRegion, &tk, &k_full[ks], c * 64, j * C::kTK, h, b);
            }
          }
          if (near) t.bits |= kNear;
          if (ok && (ok = wait_bar<0>(&aux_empty[as], ((g / C::kAux) & 1) ^ 1, err, 203))) {
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
            if ((ok = wait_bar<0>(&v_empty[ks], ((kc / C::kKv) & 1) ^ 1, err, 204))) {
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
        if (!wait_bar<0>(&aux_full[as], (e / C::kAux) & 1, err, 213)) return false;
        t = *info_of(e);
        mbar_arrive(&aux_empty[as]);
        return t.tile < 0 || wait_bar<0>(&k_full[kc % C::kKv], (kc / C::kKv) & 1, err, 216);
      };
      for (int it = blockIdx.x; it < nitems && ok; it += gridDim.x, ++n) {
        if (!(ok = next_info(g)) || !(ok = wait_bar<0>(q_full, n & 1, err, 214))) break;
        for (;; ++g) {
          const bool last = t.bits & kLast, first = t.bits & kFirst;
          if (t.tile < 0) {
            // nothing to multiply: the phases go on
            mbar_arrive(s_full);
            mbar_arrive(s_full);
            if (!(ok = wait_bar<0>(p_full, g & 1, err, 211))) break;
            mbar_arrive(pv_done);
            break;
          }
          const int ks = kc % C::kKv;
          const uint32_t kp = (kc / C::kKv) & 1;
          // S goes over the P that the last product read, and products with
          // different accumulators may overtake one another
          if (kc > 0 && !(ok = wait_bar<0>(&v_empty[(kc - 1) % C::kKv], ((kc - 1) / C::kKv) & 1, err, 217))) break;
          ++kc;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_f16(tmem, dq + (kk >> 2) * (kRegion >> 4) + (kk & 3) * 2,
                    dk + ks * (C::kKvBytes >> 4) + (kk >> 2) * (C::kKvRegion >> 4) + (kk & 3) * 2, id_s, kk > 0);
          mma_commit(s_full);
          mbar_arrive(s_full);   // orders what this thread waited for; the commit, the products
          mma_commit(&k_empty[ks]);
          // what the next tile needs, ahead of the wait for P (an item's first
          // tile waits for the rows of the item before)
          if (!last && !(ok = next_info(g + 1))) break;
          if (!(ok = wait_bar<0>(&v_full[ks], kp, err, 212))) break;
          // P lies over S, so its product comes before the next Q K^T
          if (!(ok = wait_bar<0>(p_full, g & 1, err, 211))) break;
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
        // S is there, and with it the description and the vectors, which its
        // issuing thread waited for
        if (!(ok = wait_warp<0>(s_full, g & 1, err, 222))) break;
        const TileInfo t = *info_of(g);
        last = t.bits & kLast;
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
          // row r's run of diagonals starts at 128 - r of the window (copy s is
          // shifted by s + 1)
          const int start = 127 - r;
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
        if (t.bits & kFirst) {
          ref = top - kFwdUp;
        } else if (__any_sync(0xffffffffu, top - ref > kFwdUp + kRescale)) {
          const float next = top - kFwdUp;
          const float f = top - ref > kFwdUp + kRescale ? ex2f(ref - next) : 1.0f;
          if (f != 1.0f) ref = next;
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
            w[e] = pack_p<T>(p.x, p.y);
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
      // ---- the item's rows: O / l through the Q tile (no product reads it any more)
      if (ok && (ok = wait_warp<0>(pv_done, n & 1, err, 225))) {
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
      }
      // each warp times its own waits: all four go on, or none does
      if (!(ok = named_barrier_all(1, 128, ok))) break;
      if (threadIdx.x == 0) {
        for (int c = 0; c < D / 64; ++c) tma_store_4d(&to, sQ + c * kRegion, c * 64, i * 128, h, b);
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

// ============================================================================ backward
// One block per SM walks items of 128 stationary rows against moving tiles of
// 64 columns.  Key items (all of them first): rows K and V, columns Q and dO,
//   S^T = K Q^T, dP^T = V dO^T;  dV += P^T dO, dK += dS^T Q
// query items: rows Q and dO, columns K and V,
//   S = Q K^T, dP = dO V^T;  dQ += dS K, and dS summed into the bias gradient.
// S and dP are formed twice (7 products instead of 5), and in return no sum
// is shared between blocks: no atomics, every gradient bitwise reproducible.
//
// Warps 0-3 and 4-7 take the moving tiles in turn (one row, that is one TMEM
// lane, per thread), so one tile's exponentials run while the other's
// products do; 8-11 write the finished rows out; 12: TMA; 13 issues S and dP,
// 14 the sums (one thread for both spent its time in waits of the one that the
// other did not need).  P and dS
// (rounded to the storage type, at most half a step) overwrite S and dP in
// TMEM and are the A operands of the second pair of products from there, so
// they never touch shared memory.  P is held kAttnPUp times too large: the
// probabilities of a long row (1/S each) then stay clear of float16's
// subnormals, whose rounding is absolute, up to S = 2^22.  The factor comes with
// -lse2, leaves dS through the product dP / kAttnPUp - D / kAttnPUp, and dV as it
// is written out; all of it is exact.  dS, which has the size of a gradient, is
// held at a factor of its own for float16 (ds_factor in attention.cuh).
// TMEM: three (head dim 128: two) buffers of S and dP, 64 columns each, then the
// two sums.
//
// Bound: the chain of a tile (operands, product, exponentials, product) through
// the barriers between its warps: tensor pipe 33 %, exponentials 38 %, issue
// slots 41 % busy.  A call (L2 warm), B4 h16 d64 S2048: 368 us, 467 TFLOP/s of the
// 5 products that the formulas have (654 of the 7 formed); h8 d128: 287 us, 599
// TFLOP/s; B16 h16 S512: 148 us.
constexpr int kRun = 192, kWin = 200;           // diagonals of a 128 x 64 tile, floats of a window copy
constexpr int kVecs = 4 * kWin * 4;             // column vectors after the four copies
constexpr int kChain = 40;                      // floats of a diagonal chain
constexpr int kChains = 8;                      // of a tile's 64 columns, 8 each
template <int D, bool LONG>
struct Bwd {
  static constexpr int kSt = D / 64 * kRegion;                      // a stationary tile
  static constexpr int kMvRegion = 64 * 128;
  static constexpr int kMv = D / 64 * kMvRegion;                    // a moving tile
  static_assert(D == 128 || !LONG, "head dim 128 alone has two forms");
  static constexpr int kSlots = LONG ? 1 : 2;                       // stationary pairs
  static constexpr int kNs = D == 64 || LONG ? 4 : 2;               // moving pairs
  static constexpr int kBuf = D == 64 ? 3 : 2;                      // S, dP buffers
  // Barriers of finished scores.  Two groups take the tiles in turn, and a wait
  // for a parity cannot tell the phase before the last one done from its own: a
  // barrier belongs to one group, which then waits for each of its phases.
  static constexpr int kFull = kBuf % 2 ? 2 * kBuf : kBuf;
  static constexpr uint32_t kSums = kBuf * 128;                     // their first TMEM column
  static constexpr int kAuxBytes = kVecs + 512 + 16;                // window, two column vectors, description
  static constexpr int kStAux = 2 * 128 * 4 + 16;                   // row vectors, empty flag, dS factor
  static constexpr int kSmem = kSlots * 2 * kSt + 2 * kNs * kMv + kNs * kAuxBytes + kSlots * kStAux +
                               8 * kAttnMaxBuckets * 4 + 8 * kChains * kChain * 4 + 400;
  static constexpr int kBars = 2 * kSlots + 2 * kNs + kFull + 2 * kBuf + 2;
  static_assert(kFull % 2 == 0, "a barrier of finished scores serves both softmax groups");
  static_assert(kBars * 8 + 4 <= 400, "the barriers do not fit their shared memory");
  static_assert(kSums + 2 * D <= 512, "the sums do not fit the tensor memory");
  static_assert(kSmem <= 227 * 1024, "the backward's shared memory exceeds a block's maximum");
};
// Head dim 128, LONG from this length on: one stationary pair and four moving
// ones instead of two and two (shared memory holds six), which a short item does
// not repay.  B8 h8, us, float16: S 192 30.0 against 28.1, 384 52.1 and 51.4, 512
// 75.8 and 76.3; bfloat16: S 1024 183 and 201, 1536 361 and 419.
// At head dims up to 64 two buffers of scores and two sets of sums, so that the
// next item starts while one is written out, lost to three buffers from S 129 on
// (B16 h16 S129 45.2 against 46.8 us, S512 151 and 157; B8 h16 S1536 436 and 488).
constexpr int kLongSeq = 512;
constexpr int kBwdThreads = 480;
constexpr int kPauseLoad = 50, kPauseSoft = 20, kPauseStore = 200;   // ns between polls

// Whether dS is held at a factor of its own (float16; bfloat16 has float32's range).
template <typename T> constexpr bool kHoldsDs = std::is_same<T, half_t>::value;

// Sums the diagonals of a warp's 32 rows x 32 columns (v: this lane's row), as
// four chains of 8 columns whose steps are independent of one another.  Diagonal
// t - lane moves up one lane per column, so a chain's running sums are shifted
// along; the one that leaves at lane 31 is done and goes to out[t], the 32 left
// at the end to out[8 ..], in order of the diagonal: out[y] is diagonal y - 31.
__device__ __forceinline__ void diagonal_chains(const float (&v)[32], float* out, int lane) {
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int t = 0; t < 8; ++t) {
#pragma unroll
    for (int c = 0; c < 4; ++c) s[c] += v[8 * c + t];
    if (t < 7) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (lane == 31) out[c * kChain + t] = s[c];
        s[c] = __shfl_up_sync(0xffffffffu, s[c], 1);
        if (lane == 0) s[c] = 0.0f;
      }
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) out[c * kChain + 38 - lane] = s[c];
}

// One warp's 32 rows x 64 columns of dS, from its chains into its bins: each of
// the 95 diagonals is the sum of the chains that cross it; those of one bucket
// are neighbours and are summed by a segmented scan.  bid: the bucket of
// diagonal 0 of the block (its column 0, its row 0); DIR: 1 where the columns
// are keys, -1 where they are queries.
template <int DIR>
__device__ __forceinline__ void bin_diagonals(const float* chains, const uint8_t* bid, float* bins, int lane) {
  float s[3];
  int u[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int y = lane + 32 * k;            // diagonal y - 31
    u[k] = y < 95 ? bid[DIR * (y - 31)] : 256;
    s[k] = 0.0f;
#pragma unroll
    for (int c = 0; c < kChains; ++c) {
      const int z = y - 8 * c;
      if (z >= 0 && z < 39) s[k] += chains[c * kChain + z];
    }
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const float s2 = __shfl_up_sync(0xffffffffu, s[k], o);
      const int u2 = __shfl_up_sync(0xffffffffu, u[k], o);
      if (lane >= o && u2 == u[k]) s[k] += s2;
    }
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int next = __shfl_down_sync(0xffffffffu, u[k], 1);
    if (u[k] < 256 && (lane == 31 || next != u[k])) bins[u[k]] += s[k];
    __syncwarp();
  }
}

// A tile's scores and dP, 64 columns of this thread's row, into P and dS.
// ax: the tile's staged vectors; row: what this row adds (log2 units, bias of
// a far tile included).  With F the factor that dS is held at (ds_factor; none
// for bfloat16): nd_row: -D F / kAttnPUp of a query row, up: F / kAttnPUp there,
// F for keys, whose column vector -D / kAttnPUp does not hold it (P times F took
// 287 us where the vector times F, with more values alive, took 306: B4 h8 d128
// S2048).
template <typename T, bool KEYS, bool NEAR, bool MIX>
__device__ __forceinline__ void bwd_tile(uint32_t tS, const uint8_t* ax, int win, const float* vecA, const float* vecB,
                                         float c2, float row, float nd_row, float up, int r, bool grad, float& far_sum,
                                         float* chains, int lane) {
  const int start = 127 - r;   // the row's run of diagonals; copy s is shifted by s + 1
  const float* wnd = reinterpret_cast<const float*>(ax) + (start & 3) * win + (start & ~3);
  float2 fs = f2(0.0f);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float s[32], dp[32];
    tmem_ld32_nowait(tS + c * 32, s);
    tmem_ld32_nowait(tS + 64 + c * 32, dp);
    tmem_ld_wait();
    uint32_t wp[16], wd[16];
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      float2 add0 = f2(row), add1 = f2(row), nd0 = f2(nd_row), nd1 = f2(nd_row);
      if (KEYS || MIX) {
        const float4 w = *reinterpret_cast<const float4*>(vecA + c * 32 + e);
        add0 = __fadd2_rn(add0, make_float2(w.x, w.y));
        add1 = __fadd2_rn(add1, make_float2(w.z, w.w));
      }
      if (KEYS) {
        const float4 w = *reinterpret_cast<const float4*>(vecB + c * 32 + e);
        nd0 = make_float2(w.x, w.y);
        nd1 = make_float2(w.z, w.w);
      }
      if (NEAR) {
        const float4 w = *reinterpret_cast<const float4*>(wnd + c * 32 + e);
        add0 = __fadd2_rn(add0, make_float2(w.x, w.y));
        add1 = __fadd2_rn(add1, make_float2(w.z, w.w));
      }
      const float2 x0 = __ffma2_rn(make_float2(s[e], s[e + 1]), f2(c2), add0);
      const float2 x1 = __ffma2_rn(make_float2(s[e + 2], s[e + 3]), f2(c2), add1);
      const float2 p0 = make_float2(ex2f(x0.x), ex2f(x0.y)), p1 = make_float2(ex2f(x1.x), ex2f(x1.y));
      float2 g0 = p0, g1 = p1;
      if (KEYS && kHoldsDs<T>) g0 = __fmul2_rn(p0, f2(up)), g1 = __fmul2_rn(p1, f2(up));
      const float m = KEYS || !kHoldsDs<T> ? 1.0f / kAttnPUp : up;
      const float2 d0 = __fmul2_rn(g0, __ffma2_rn(make_float2(dp[e], dp[e + 1]), f2(m), nd0));
      const float2 d1 = __fmul2_rn(g1, __ffma2_rn(make_float2(dp[e + 2], dp[e + 3]), f2(m), nd1));
      if (KEYS) {
        wp[e / 2] = pack2<T>(p0.x, p0.y);
        wp[e / 2 + 1] = pack2<T>(p1.x, p1.y);
      }
      wd[e / 2] = pack2<T>(d0.x, d0.y);
      wd[e / 2 + 1] = pack2<T>(d1.x, d1.y);
      if (!KEYS) {
        if (NEAR) {
          dp[e] = d0.x, dp[e + 1] = d0.y, dp[e + 2] = d1.x, dp[e + 3] = d1.y;
        } else {
          fs = __fadd2_rn(fs, __fadd2_rn(d0, d1));
        }
      }
    }
    // over S and dP columns that this thread has read
    if (KEYS) tmem_st16u(tS + c * 16, wp);
    tmem_st16u(tS + 64 + c * 16, wd);
    if (!KEYS && NEAR && grad) diagonal_chains(dp, chains + 4 * c * kChain, lane);
  }
  far_sum += fs.x + fs.y;
}

template <typename T, int D, bool LONG>
__global__ void __launch_bounds__(kBwdThreads, 1)
    attention_bwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                         const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                         const __grid_constant__ CUtensorMap tq2, const __grid_constant__ CUtensorMap tk2,
                         const __grid_constant__ CUtensorMap tv2, const __grid_constant__ CUtensorMap tdo2,
                         const __grid_constant__ CUtensorMap tdq, const __grid_constant__ CUtensorMap tdk,
                         const __grid_constant__ CUtensorMap tdv, const __grid_constant__ AttnOp a) {
  using C = Bwd<D, LONG>;
  // the only shared memory of the kernel: its start is 1024-byte aligned
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sSt = smem_raw;                                  // [kSlots] x (A1, A2)
  uint8_t* sMv = sSt + C::kSlots * 2 * C::kSt;                          // [kNs] x (B1, B2)
  uint8_t* sAux = sMv + 2 * C::kNs * C::kMv;                // [kNs]
  uint8_t* sStAux = sAux + C::kNs * C::kAuxBytes;           // [2]
  float* sBins = reinterpret_cast<float*>(sStAux + C::kSlots * C::kStAux);
  float* sChains = sBins + 8 * kAttnMaxBuckets;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sChains + 8 * kChains * kChain);
  uint64_t *st_full = bar, *st_empty = st_full + C::kSlots, *mv_full = st_empty + C::kSlots,
           *mv_empty = mv_full + C::kNs, *s_full = mv_empty + C::kNs, *p_full = s_full + C::kFull, *s_free = p_full + C::kBuf,
           *acc_full = s_free + C::kBuf, *acc_free = acc_full + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(acc_free + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* err = g_attention_err;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) mbar_init(&st_full[i], 1), mbar_init(&st_empty[i], 1);
    for (int i = 0; i < C::kFull; ++i) mbar_init(&s_full[i], 2);
    for (int i = 0; i < C::kBuf; ++i) mbar_init(&p_full[i], 4), mbar_init(&s_free[i], 1);
    for (int i = 0; i < C::kNs; ++i) mbar_init(&mv_full[i], 1), mbar_init(&mv_empty[i], 1);
    mbar_init(acc_full, 1), mbar_init(acc_free, 4);
    fence_barrier_init();
  }
  if (warp == 13) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  pdl_wait();
  pdl_launch_dependents();

  const int nr = (a.S + 127) / 128, nm = (a.S + 63) / 64;
  const int items = a.B * a.nh * nr;
  auto info_of = [&](uint32_t g) -> TileInfo* {
    return reinterpret_cast<TileInfo*>(sAux + (g % C::kNs) * C::kAuxBytes + kVecs + 512);
  };
  auto row_vec = [&](int n) { return reinterpret_cast<float*>(sStAux + (n % C::kSlots) * C::kStAux); };
  auto none_flag = [&](int n) { return reinterpret_cast<int*>(sStAux + (n % C::kSlots) * C::kStAux + 1024); };
  auto factor = [&](int n) { return reinterpret_cast<float*>(sStAux + (n % C::kSlots) * C::kStAux + 1028); };

  if (warp == 12) {
    // ---- producer
    uint32_t g = 0, st_issued = 0;
    int n = 0;
    bool ok = true;
    // the first of an item's magnitudes, read one item ahead
    auto first_max = [&](int it) {
      const int bh = (it < items ? it : it - items) / nr;
      return it < 2 * items && lane < a.nmax ? a.smax[(size_t)bh * a.nmax + lane] : __float2half2_rn(0.0f);
    };
    __half2 most = kHoldsDs<T> ? first_max(blockIdx.x) : __float2half2_rn(0.0f);
    for (int it = blockIdx.x; it < 2 * items && ok; it += gridDim.x, ++n) {
      const bool keys = it < items;
      const int x = keys ? it : it - items, bh = x / nr, ri = x - bh * nr, b = bh / a.nh, h = bh - b * a.nh;
      const int mb = a.mask_seqs == 1 ? 0 : b;
      const int* flags = a.flags + mb * (a.Sp / kAttnFlagKeys);
      const float* vec = a.vec ? bias_copy(a, h, 0, 0) : nullptr;
      const float behind = vec ? vec[a.vec_off - a.sat - 1] : 0.0f, ahead = vec ? vec[a.vec_off + a.sat - 1] : 0.0f;
      const float* stats = a.stats + (size_t)bh * 2 * a.Sp;
      LiveTiles<1> tiles(flags, nm, lane);
      bool mix = false;
      int j = keys ? (flags[2 * ri] == 2 && flags[2 * ri + 1] == 2 ? nm : 0) : tiles.next(0, mix);
      const bool none = j == nm;
      const int slot = n % C::kSlots;
      float F = 1.0f;
      if (kHoldsDs<T>) {
        __half2 m = most;
        for (int c = 32 + lane; c < a.nmax; c += 32) m = __hmax2(m, a.smax[(size_t)bh * a.nmax + c]);
        F = ds_factor(warp_max2(m), a.d);
        most = first_max(it + gridDim.x);
      }
      if (lane == 0 && (ok = wait_bar<kPauseLoad>(&st_empty[slot], ((n / C::kSlots) & 1) ^ 1, err, 301))) {
        *none_flag(n) = none;
        *factor(n) = F;
        ++st_issued;
        mbar_arrive_expect_tx(&st_full[slot], 2 * C::kSt + (keys ? 512 : 1024));
        uint8_t* st = sSt + slot * 2 * C::kSt;
        for (int c = 0; c < D / 64; ++c) {
          tma_load_4d(st + c * kRegion, keys ? &tk2 : &tq2, &st_full[slot], c * 64, ri * 128, h, b);
          tma_load_4d(st + C::kSt + c * kRegion, keys ? &tv2 : &tdo2, &st_full[slot], c * 64, ri * 128, h, b);
        }
        if (keys) bulk_load_1d(row_vec(n), a.maskx + (size_t)mb * a.Sp + ri * 128, 512, &st_full[slot]);
        else bulk_load_1d(row_vec(n), stats + ri * 256, 1024, &st_full[slot]);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      bool first = true;
      do {
        bool nmix = false;
        const int jn = none ? nm : (keys ? j + 1 : tiles.next(j + 1, nmix));
        const int ms = g % C::kNs;
        TileInfo t;
        t.tile = none ? -1 : j;
        t.item = n;
        t.bits = (jn == nm ? kLast : 0) | (first ? kFirst : 0) | (keys ? kKeys : 0);
        t.bias = 0.0f;
        // diagonal of the tile's corner, column minus row
        const int x0 = j * 64 - ri * 128;
        if (!none) {
          if (vec) {
            // key minus query: the columns are the keys, or the rows are
            const int lo = keys ? -(x0 + 63) : x0 - 127, hi = keys ? 127 - x0 : x0 + 63;
            if (lo >= a.sat) t.bias = ahead, t.bits |= kAhead;
            else if (hi <= -a.sat) t.bias = behind;
            else t.bits |= kNear;
          }
          if (mix && !keys) t.bits |= kMixed;
        }
        const bool near = t.bits & kNear, mk = near && !keys || (t.bits & kMixed);
        if (lane == 0 && ok && (ok = wait_bar<kPauseLoad>(&mv_empty[ms], ((g / C::kNs) & 1) ^ 1, err, 303))) {
          *info_of(g) = t;
          mbar_arrive_expect_tx(&mv_full[ms], none ? 0 : 2 * C::kMv + (keys ? 512 : 0) + (mk ? 256 : 0) +
                                                             (near ? 4 * kRun * 4 : 0));
          if (!none) {
            uint8_t* ax = sAux + ms * C::kAuxBytes;
            uint8_t* mv = sMv + ms * 2 * C::kMv;
            for (int c = 0; c < D / 64; ++c) {
              tma_load_4d(mv + c * C::kMvRegion, keys ? &tq : &tk, &mv_full[ms], c * 64, j * 64, h, b);
              tma_load_4d(mv + C::kMv + c * C::kMvRegion, keys ? &tdo : &tv, &mv_full[ms], c * 64, j * 64, h, b);
            }
            if (keys) bulk_load_1d(ax + kVecs, stats + j * 128, 512, &mv_full[ms]);
            if (mk) bulk_load_1d(ax + kVecs, a.maskx + (size_t)mb * a.Sp + j * 64, 256, &mv_full[ms]);
            if (near)
              for (int k = 0; k < 4; ++k)
                bulk_load_1d(ax + k * kWin * 4, bias_copy(a, h, keys ? 1 : 0, k) + x0 - 128 + a.vec_off, kRun * 4,
                             &mv_full[ms]);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        first = false;
        ++g;
        j = jn;
        mix = nmix;
      } while (j < nm);
    }
    // the end, for either softmax group
    for (int e = 0; e < 2 && ok && lane == 0; ++e, ++g) {
      if (!(ok = wait_bar<kPauseLoad>(&mv_empty[g % C::kNs], ((g / C::kNs) & 1) ^ 1, err, 304))) break;
      *info_of(g) = TileInfo{-1, kEnd, 0.0f, -1};
      mbar_arrive(&mv_full[g % C::kNs]);
    }
    if (!ok && lane == 0) {
      drain<C::kSlots>(st_full, st_issued);
      drain<C::kNs>(mv_full, g);
    }
  } else if (warp == 13) {
    // ---- S and dP of each tile, as soon as its operands and a buffer are there
    if (lane == 0) {
      const uint32_t id = idesc_f16(128, 64, std::is_same<T, bf16_t>::value, false, false);
      const uint64_t dst = desc_k(smem_u32(sSt), 0, kRegion), dmv = desc_k(smem_u32(sMv), 0, C::kMvRegion);
      for (uint32_t g = 0, ends = 0; ends < 2; ++g) {
        const int ms = g % C::kNs, w = g % C::kBuf;
        uint64_t* sf = &s_full[g % C::kFull];
        if (!wait_bar<0>(&mv_full[ms], (g / C::kNs) & 1, err, 313)) break;
        const TileInfo t = *info_of(g);
        const int slot = t.item % C::kSlots;
        if ((t.bits & kFirst) && !wait_bar<0>(&st_full[slot], (t.item / C::kSlots) & 1, err, 314)) break;
        // the buffer's last tile has been multiplied out of it
        if (!wait_bar<0>(&s_free[w], ((g / C::kBuf) & 1) ^ 1, err, 316)) break;
        if (t.tile < 0) {
          if (t.bits & kEnd) ++ends;
          mbar_arrive(sf);
          mbar_arrive(sf);
          continue;
        }
        tc_fence_after();
        const uint64_t a1 = dst + slot * (2 * C::kSt >> 4), a2 = a1 + (C::kSt >> 4);
        const uint64_t b1 = dmv + ms * (2 * C::kMv >> 4), b2 = b1 + (C::kMv >> 4);
        const uint32_t tS = tmem + w * 128;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_f16(tS, a1 + (kk >> 2) * (kRegion >> 4) + (kk & 3) * 2, b1 + (kk >> 2) * (C::kMvRegion >> 4) + (kk & 3) * 2,
                  id, kk > 0);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_f16(tS + 64, a2 + (kk >> 2) * (kRegion >> 4) + (kk & 3) * 2,
                  b2 + (kk >> 2) * (C::kMvRegion >> 4) + (kk & 3) * 2, id, kk > 0);
        mma_commit(sf);
        mbar_arrive(sf);   // orders what this thread waited for; the commit, the products
      }
    }
  } else if (warp == 14) {
    // ---- the sums, as soon as a tile's P and dS are there
    if (lane == 0) {
      const uint32_t id = idesc_f16(128, D, std::is_same<T, bf16_t>::value, false, true);
      const uint64_t dmn = desc_mn(smem_u32(sMv), 0, C::kMvRegion);
      for (uint32_t g = 0, ends = 0; ends < 2; ++g) {
        const int ms = g % C::kNs, w = g % C::kBuf;
        if (!wait_bar<0>(&p_full[w], (g / C::kBuf) & 1, err, 311)) break;
        const TileInfo t = *info_of(g);
        if ((t.bits & kFirst) && !wait_bar<0>(acc_free, (t.item & 1) ^ 1, err, 312)) break;
        if (t.tile < 0) {
          mbar_arrive(&mv_empty[ms]);
          mbar_arrive(&s_free[w]);
          if (t.bits & kEnd) ++ends;
          else mbar_arrive(acc_full);
          continue;
        }
        tc_fence_after();
        const uint32_t acc1 = tmem + C::kSums, acc2 = acc1 + D, tS = tmem + w * 128;
        const uint64_t b1 = dmn + ms * (2 * C::kMv >> 4), b2 = b1 + (C::kMv >> 4);
        const uint32_t more = t.bits & kFirst ? 0u : 1u;
        if (t.bits & kKeys) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_f16_ts(acc2, tS + kk * 8, b2 + kk * 128, id, more | (kk > 0));
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_f16_ts(acc1, tS + 64 + kk * 8, b1 + kk * 128, id, more | (kk > 0));
        mma_commit(&s_free[w]);
        mma_commit(&mv_empty[ms]);
        if (t.bits & kLast) mma_commit(acc_full);
      }
    }
  } else if (warp >= 8) {
    // ---- finished rows: TMEM -> scale -> the item's own stationary tiles (no
    // product reads them any more) -> TMA store
    const int r = threadIdx.x - 256;
    const uint32_t lo = (uint32_t)((warp & 3) * 32) << 16;
    bool ok = true;
    int n = 0;
    for (int it = blockIdx.x; it < 2 * items && ok; it += gridDim.x, ++n) {
      const bool keys = it < items;
      const int x = keys ? it : it - items, bh = x / nr, ri = x - bh * nr, b = bh / a.nh, h = bh - b * a.nh;
      const int slot = n % C::kSlots;
      uint8_t* st = sSt + slot * 2 * C::kSt;
      ok = wait_warp<kPauseStore>(&st_full[slot], (n / C::kSlots) & 1, err, 321);
      const bool none = ok && *none_flag(n) != 0;
      const float F = kHoldsDs<T> && ok ? *factor(n) : 1.0f;
      if (ok && (ok = wait_warp<kPauseStore>(acc_full, n & 1, err, 322))) {
        tc_fence_after();
#pragma unroll 1
        for (int q = 0; q < (keys ? 2 : 1); ++q) {
          const float f = q == 0 ? a.scale * inv_pow2(F) : 1.0f / kAttnPUp;
          uint8_t* out = st + q * C::kSt;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float v[32];
            tmem_ld32_nowait(tmem + lo + C::kSums + q * D + c * 32, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = none ? 0u : pack2<T>(v[e * 8 + 2 * k] * f, v[e * 8 + 2 * k + 1] * f);
              const int ch = c * 4 + e;
              *reinterpret_cast<uint4*>(out + (ch >> 3) * kRegion + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_free);
        fence_proxy_async_smem();
      }
      // each warp times its own waits: all four go on, or none does
      if (!(ok = named_barrier_all(1, 128, ok))) break;
      if (r == 0) {
        for (int c = 0; c < D / 64; ++c) {
          tma_store_4d(keys ? &tdk : &tdq, st + c * kRegion, c * 64, ri * 128, h, b);
          if (keys) tma_store_4d(&tdv, st + C::kSt + c * kRegion, c * 64, ri * 128, h, b);
        }
        bulk_commit();
        bulk_wait_read<0>();
        mbar_arrive(&st_empty[slot]);
      }
    }
    if (r == 0) bulk_wait_all();
    __syncwarp();
  } else {
    // ---- softmax groups
    const int wg = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lo = (uint32_t)((warp & 3) * 32) << 16;
    const float c2 = a.c2;
    float* bins = sBins + warp * kAttnMaxBuckets;
    float* chains = sChains + warp * kChains * kChain;
    const bool want = a.dpart != nullptr;
    if (want)
      for (int u = lane; u < a.buckets; u += 32) bins[u] = 0.0f;
    __syncwarp();
    int cur = -1, row0 = 0;
    size_t part = 0;               // this warp's row of dpart for the current item
    bool grad = false, any_far = false;
    float add = 0.0f, nd = 0.0f, far_behind = 0.0f, far_ahead = 0.0f;
    float up = 1.0f / kAttnPUp;
    // the item's bias gradient: this warp's share
    auto flush = [&]() {
      if (any_far) {
        const float fb = warp_sum(far_behind), fa = warp_sum(far_ahead);
        if (lane == 0) {
          bins[a.buckets / 2 - 1] += fb;
          bins[a.buckets - 1] += fa;
        }
        __syncwarp();
        far_behind = far_ahead = 0.0f;
        any_far = false;
      }
      for (int u = lane; u < a.buckets; u += 32) {
        a.dpart[part + u] = kHoldsDs<T> ? bins[u] * inv_pow2(up * kAttnPUp) : bins[u];
        bins[u] = 0.0f;
      }
      __syncwarp();
    };
    for (uint32_t g = wg;; g += 2) {
      const int buf = g % C::kBuf;
      // S is there, and with it everything that its issuing thread waited for:
      // the description, the vectors, the item's row vectors (each wait costs
      // 150 clocks even when there is nothing to wait for)
      if (!wait_warp<kPauseSoft>(&s_full[g % C::kFull], (g / C::kFull) & 1, err, 333)) break;
      const TileInfo t = *info_of(g);
      if (t.bits & kEnd) {
        if (lane == 0) mbar_arrive(&p_full[buf]);
        break;
      }
      const bool keys = t.bits & kKeys;
      if (t.item != cur) {
        if (grad) flush();
        cur = t.item;
        const float* rv = row_vec(cur);
        add = rv[keys ? r : (r >> 6) * 128 + (r & 63)];
        nd = keys ? 0.0f : rv[(r >> 6) * 128 + 64 + (r & 63)];
        if (kHoldsDs<T>) {
          const float F = *factor(cur);
          up = keys ? F : F * (1.0f / kAttnPUp);
          nd *= F;
        }
        grad = want && !keys;
        const int x = (int)(blockIdx.x + (unsigned)cur * gridDim.x) - (keys ? 0 : items);
        const int bh = x / nr, ri = x - bh * nr;
        row0 = ri * 128 + (warp & 3) * 32;
        part = ((size_t)bh * a.ditems + ri * 8 + warp) * a.buckets;
      }
      if (t.tile >= 0) {
        tc_fence_after();
        const uint32_t tS = tmem + buf * 128 + lo;
        const uint8_t* ax = sAux + (g % C::kNs) * C::kAuxBytes;
        const float* va = reinterpret_cast<const float*>(ax + kVecs);
        const float* vb = reinterpret_cast<const float*>(ax + kVecs + 256);
        const float row = add + t.bias;
        float far = 0.0f;
        if (keys) {
          if (t.bits & kNear) bwd_tile<T, true, true, false>(tS, ax, kWin, va, vb, c2, row, nd, up, r, false, far, chains, lane);
          else bwd_tile<T, true, false, false>(tS, ax, kWin, va, vb, c2, row, nd, up, r, false, far, chains, lane);
        } else if (t.bits & kNear) {
          bwd_tile<T, false, true, true>(tS, ax, kWin, va, vb, c2, row, nd, up, r, grad, far, chains, lane);
        } else if (t.bits & kMixed) {
          bwd_tile<T, false, false, true>(tS, ax, kWin, va, vb, c2, row, nd, up, r, grad, far, chains, lane);
        } else {
          bwd_tile<T, false, false, false>(tS, ax, kWin, va, vb, c2, row, nd, up, r, grad, far, chains, lane);
        }
        if (!(t.bits & kNear)) {
          any_far = true;
          if (t.bits & kAhead) far_ahead += far;
          else far_behind += far;
        }
        tmem_store_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[buf]);
      if (grad && (t.bits & kNear)) bin_diagonals<1>(chains, a.bid + a.vec_off + t.tile * 64 - row0, bins, lane);
    }
    if (grad) flush();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------- backward, one tile per sequence and head
// Sequences up to 128 at head dims up to 64: one block takes a whole (sequence,
// head), rows = keys, so S and dP are formed once (5 products instead of 7):
//   S^T = K Q^T, dP^T = V dO^T;  dV = P^T dO, dK = dS^T Q, dQ = dS K
// D = dO.O is formed here too, from tiles that the products need (dO) or that
// make room later (O): nothing of size (tokens, hidden) is read twice.
// Two blocks of 8 warps share an SM, and one block's softmax runs while the
// other loads, multiplies or writes.  A warp has 32 keys and one half of the
// queries.  Head dim 128 would leave room for one block only and takes the
// kernel above.
//
// Bound: the latency of a pair's load, two rounds of products and write, which two
// blocks on an SM do not hide (HBM at 27 % of its peak): B64 h16 S128, 134.7 MB,
// 43 us, 3.1 TB/s; loads and stores alone 26 us.  The kernel above took 57 us
// there, and 14 more for D in the prepared workspace.  One block walking several pairs (the
// next V and O loaded ahead, prefetched to L2, or dQ written straight to its rows
// so that Q, K and dO load ahead too) came to the same or 2 us more.
//
// TMEM columns: S 0..127, dP 128..255.  P (16-bit) goes to 0..31 (queries
// 0..63) and 96..127 (the others), which leaves 32..95 for dV; dS goes to
// shared memory, over the tiles of O and V, where one copy serves as the A
// operand of dK (its rows) and of dQ (its columns), and dP makes room for
// dK (128..191) and dQ (192..255).  The results leave through dO, Q and K.
struct One {
  static constexpr int kThreads = 256;
  static constexpr int kWin = 264;                // floats of a window copy: 256 diagonals, 8 banks apart
  static constexpr int kChainFloats = 8 * kChains * kChain;
  static constexpr int kSmem = 5 * kRegion + 4 * kWin * 4 + 2 * 128 * 4 + 8 * kAttnMaxBuckets * 4 + kChainFloats * 4 + 32 + 48;
};
static_assert(2 * (One::kSmem + 1024) <= 228 * 1024, "two blocks do not fit an SM's shared memory");

template <typename T, bool BIAS>
__global__ void __launch_bounds__(One::kThreads, 2)
    attention_bwd_one_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                             const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to,
                             const __grid_constant__ CUtensorMap tdo, const __grid_constant__ CUtensorMap tdq,
                             const __grid_constant__ CUtensorMap tdk, const __grid_constant__ CUtensorMap tdv,
                             const __grid_constant__ AttnOp a) {
  // the only shared memory of the kernel: its start is 1024-byte aligned
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *sQ = smem_raw, *sK = sQ + kRegion, *sDo = sK + kRegion, *sO = sDo + kRegion, *sV = sO + kRegion;
  uint8_t* sDs = sO;                                                  // [2] x [128 keys][64 queries]
  float* sWin = reinterpret_cast<float*>(sV + kRegion);
  float* vecA = sWin + 4 * One::kWin;                                 // log2(kAttnPUp) - lse2 of every query
  float* vecB = vecA + 128;                                           // -D / kAttnPUp
  float* sBins = vecB + 128;
  float* sChains = sBins + 8 * kAttnMaxBuckets;
  __half2* sMax = reinterpret_cast<__half2*>(sChains + One::kChainFloats);  // per warp, largest |dO| and |V|
  uint64_t* bar = reinterpret_cast<uint64_t*>(sMax + 8);
  uint64_t *qk_full = bar, *vd_full = bar + 1, *o_full = bar + 2, *s_done = bar + 3, *sums_done = bar + 4;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 5);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = warp >> 2, r = (warp & 3) * 32 + lane;             // this thread's queries and key
  int* err = g_attention_err;
  if (tid == 0) {
    for (int i = 0; i < 5; ++i) mbar_init(&bar[i], 1);
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(tslot, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  pdl_wait();
  pdl_launch_dependents();

  const int bh = blockIdx.x, b = bh / a.nh, h = bh - b * a.nh;
  const int mb = a.mask_seqs == 1 ? 0 : b;
  const bool none = a.flags[mb * 2] == 2 && a.flags[mb * 2 + 1] == 2;   // no key left: every gradient is 0
  const bool grad = BIAS && a.dpart != nullptr;
  float* bins = sBins + warp * kAttnMaxBuckets;
  float* chains = sChains + warp * kChains * kChain;
  if (grad) {
    for (int u = lane; u < a.buckets; u += 32) bins[u] = 0.0f;
    __syncwarp();
  }
  auto bin = [&] { bin_diagonals<-1>(chains, a.bid + a.vec_off - half * 64 + (warp & 3) * 32, bins, lane); };
  bool ok = true;
  float F = 1.0f;                                                     // what dS is held at
  if (!none) {
    if (tid == 0) {
      mbar_arrive_expect_tx(qk_full, 2 * kRegion);
      tma_load_4d(sQ, &tq, qk_full, 0, 0, h, b);
      tma_load_4d(sK, &tk, qk_full, 0, 0, h, b);
      mbar_arrive_expect_tx(vd_full, 2 * kRegion);
      tma_load_4d(sDo, &tdo, vd_full, 0, 0, h, b);
      tma_load_4d(sV, &tv, vd_full, 0, 0, h, b);
      mbar_arrive_expect_tx(o_full, kRegion + (BIAS ? 4 * 256 * 4 : 0));
      tma_load_4d(sO, &to, o_full, 0, 0, h, b);
      if (BIAS)
        for (int k = 0; k < 4; ++k)
          bulk_load_1d(sWin + k * One::kWin, bias_copy(a, h, 1, k) + a.vec_off - 128, 256 * 4, o_full);
    }
    const int row = tid >> 1, part = tid & 1;                           // D: two threads to a query
    const float lse = part && row < a.S ? a.lse[(size_t)bh * a.S + row] : 0.0f;
    const float mask = a.maskx[(size_t)mb * a.Sp + r];
    const bool gone = kHoldsDs<T> && a.maskx[(size_t)mb * a.Sp + row] == -INFINITY;
    if (tid == 0) {
      const uint32_t id = idesc_f16(128, 128, std::is_same<T, bf16_t>::value, false, false);
      const uint64_t dq = desc_k(smem_u32(sQ), 0, kRegion), dk = desc_k(smem_u32(sK), 0, kRegion),
                     dv = desc_k(smem_u32(sV), 0, kRegion), dd = desc_k(smem_u32(sDo), 0, kRegion);
      ok = wait_bar<0>(qk_full, 0, err, 401);
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) mma_f16(tmem, dk + kk * 2, dq + kk * 2, id, kk > 0);
      ok = wait_bar<0>(vd_full, 0, err, 402) && ok;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) mma_f16(tmem + 128, dv + kk * 2, dd + kk * 2, id, kk > 0);
      mma_commit(s_done);
    }
    __syncwarp();
    ok = wait_warp<kPauseSoft>(vd_full, 0, err, 403) && ok;
    ok = wait_warp<kPauseSoft>(o_full, 0, err, 404) && ok;
    float d = 0.0f;
    __half2 mdo = __float2half2_rn(0.0f), mv = mdo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = row * 128 + (((part * 4 + j) ^ (row & 7)) << 4);
      const uint4 x = *reinterpret_cast<const uint4*>(sO + at), y = *reinterpret_cast<const uint4*>(sDo + at);
      const T *xe = reinterpret_cast<const T*>(&x), *ye = reinterpret_cast<const T*>(&y);
#pragma unroll
      for (int e = 0; e < 8; ++e) d = fmaf(to_f(xe[e]), to_f(ye[e]), d);
      if (kHoldsDs<T>) {
        mdo = max_abs(mdo, y);
        mv = max_abs(mv, *reinterpret_cast<const uint4*>(sV + at));
      }
    }
    d += __shfl_xor_sync(0xffffffffu, d, 1);
    if (part) vecA[row] = row < a.S ? 8.0f - lse_log2(lse) : -INFINITY;
    else vecB[row] = -d * (1.0f / kAttnPUp);
    if (kHoldsDs<T>) {
      // a sequence with a key has no empty row; rows past the end were read as 0
      if (gone) mv = __float2half2_rn(0.0f);
      const __half2 m = warp_max2(fold_max(mdo, mv));
      if (lane == 0) sMax[warp] = m;
    }
    __syncthreads();
    if (kHoldsDs<T>) {
      __half2 m = sMax[0];
#pragma unroll
      for (int w = 1; w < 8; ++w) m = __hmax2(m, sMax[w]);
      F = ds_factor(m, a.d);
    }
    const float up = F * (1.0f / kAttnPUp);
    ok = wait_warp<kPauseSoft>(s_done, 0, err, 405) && ok;
    tc_fence_after();

    // ---- P and dS of this thread's key and 64 queries, 32 at a time; the upper
    // half goes downwards, so that P lands on columns already read
    const uint32_t lo = (uint32_t)((warp & 3) * 32) << 16;
    const int start = 127 - r;   // the row's run of diagonals; copy s is shifted by s + 1
    const float* wnd = sWin + (start & 3) * One::kWin + (start & ~3) + half * 64;
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      const int c = half ? 1 - k : k, q0 = half * 64 + c * 32;
      float s[32], dp[32];
      tmem_ld32_nowait(tmem + lo + q0, s);
      tmem_ld32_nowait(tmem + lo + 128 + q0, dp);
      tmem_ld_wait();
      uint32_t wp[16], wd[16];
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 l = *reinterpret_cast<const float4*>(vecA + q0 + e), n = *reinterpret_cast<const float4*>(vecB + q0 + e);
        float2 add0 = __fadd2_rn(f2(mask), make_float2(l.x, l.y)), add1 = __fadd2_rn(f2(mask), make_float2(l.z, l.w));
        if (BIAS) {
          const float4 w = *reinterpret_cast<const float4*>(wnd + c * 32 + e);
          add0 = __fadd2_rn(add0, make_float2(w.x, w.y));
          add1 = __fadd2_rn(add1, make_float2(w.z, w.w));
        }
        const float2 x0 = __ffma2_rn(make_float2(s[e], s[e + 1]), f2(a.c2), add0);
        const float2 x1 = __ffma2_rn(make_float2(s[e + 2], s[e + 3]), f2(a.c2), add1);
        const float2 p0 = make_float2(ex2f(x0.x), ex2f(x0.y)), p1 = make_float2(ex2f(x1.x), ex2f(x1.y));
        float2 nd0 = make_float2(n.x, n.y), nd1 = make_float2(n.z, n.w);
        if (kHoldsDs<T>) nd0 = __fmul2_rn(nd0, f2(F)), nd1 = __fmul2_rn(nd1, f2(F));
        const float2 d0 = __fmul2_rn(p0, __ffma2_rn(make_float2(dp[e], dp[e + 1]), f2(up), nd0));
        const float2 d1 = __fmul2_rn(p1, __ffma2_rn(make_float2(dp[e + 2], dp[e + 3]), f2(up), nd1));
        wp[e / 2] = pack2<T>(p0.x, p0.y);
        wp[e / 2 + 1] = pack2<T>(p1.x, p1.y);
        wd[e / 2] = pack2<T>(d0.x, d0.y);
        wd[e / 2 + 1] = pack2<T>(d1.x, d1.y);
        dp[e] = d0.x, dp[e + 1] = d0.y, dp[e + 2] = d1.x, dp[e + 3] = d1.y;
      }
      tmem_st16u(tmem + lo + half * 96 + c * 16, wp);
      uint8_t* ds = sDs + half * kRegion + r * 128;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(ds + (((c * 4 + j) ^ (r & 7)) << 4)) =
            make_uint4(wd[4 * j], wd[4 * j + 1], wd[4 * j + 2], wd[4 * j + 3]);
      if (BIAS && grad) diagonal_chains(dp, chains + 4 * c * kChain, lane);
    }
    tmem_store_wait();
    tc_fence_before();
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      constexpr bool bf = std::is_same<T, bf16_t>::value;
      const uint32_t id = idesc_f16(128, 64, bf, false, true), id_q = idesc_f16(128, 64, bf, true, true);
      const uint64_t dq = desc_mn(smem_u32(sQ), 0, kRegion), dk = desc_mn(smem_u32(sK), 0, kRegion),
                     dd = desc_mn(smem_u32(sDo), 0, kRegion);
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_f16_ts(tmem + 32, tmem + (kk >> 2) * 96 + (kk & 3) * 8, dd + kk * 128, id, kk > 0);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_f16(tmem + 128, desc_k(smem_u32(sDs), kk, kRegion), dq + kk * 128, id, kk > 0);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_f16(tmem + 192, desc_mn(smem_u32(sDs), kk, kRegion), dk + kk * 128, id_q, kk > 0);
      mma_commit(sums_done);
    }
    __syncwarp();
    // warp 0, whose thread issues the products, does so behind the stores
    if (grad && warp > 0) bin();
    ok = wait_warp<kPauseSoft>(sums_done, 0, err, 406) && ok;
    tc_fence_after();
  }
  // ---- dV by the lower warps, dK by the upper ones, half of dQ each
#pragma unroll 1
  for (int k = 0; k < 3; ++k) {
    const uint32_t col = k == 2 ? 192 + half * 32 : (half ? 128 : 32) + k * 32;
    uint8_t* out = k == 2 ? sK : (half ? sQ : sDo);
    const int c = k == 2 ? half : k;
    const float f = k == 2 || half ? a.scale * inv_pow2(F) : 1.0f / kAttnPUp;
    float v[32];
    tmem_ld32_nowait(tmem + ((uint32_t)((warp & 3) * 32) << 16) + col, v);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = none ? 0u : pack2<T>(v[e * 8 + 2 * j] * f, v[e * 8 + 2 * j + 1] * f);
      *reinterpret_cast<uint4*>(out + r * 128 + (((c * 4 + e) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  tc_fence_before();
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0 && ok) {
    tma_store_4d(&tdv, sDo, 0, 0, h, b);
    tma_store_4d(&tdk, sQ, 0, 0, h, b);
    tma_store_4d(&tdq, sK, 0, 0, h, b);
    bulk_commit();
  }
  __syncwarp();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 256);
  if (grad) {
    if (warp == 0 && !none) bin();
    __syncthreads();
    for (int u = tid; u < a.buckets; u += One::kThreads) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) t += sBins[w * kAttnMaxBuckets + u];
      a.dpart[(size_t)bh * a.buckets + u] = t * inv_pow2(F);
    }
  }
  if (tid == 0) {
    bulk_wait_all();
    // a wait gave up: what was issued lands before the block exits
    for (int i = 0; i < 3 && !ok; ++i) mbar_wait(&bar[i], 0, nullptr, 0);
  }
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

template <typename T, int D>
bool fwd(const AttnOp& a, cudaStream_t s) {
  const bool bf = std::is_same<T, bf16_t>::value;
  CUtensorMap mq, mk, mv, mo;
  if (!encode(&mq, a.q, a, bf, 128) || !encode(&mk, a.k, a, bf, Fwd<D>::kTK) ||
      !encode(&mv, a.v, a, bf, Fwd<D>::kTK) || !encode(&mo, a.o, a, bf, 128))
    return false;
  static std::atomic<uint64_t> ready{0};
  allow_smem(attention_fwd_kernel<T, D>, Fwd<D>::kSmem, ready);
  const int items = a.B * a.nh * ((a.S + 127) / 128);
  launch_pdl(attention_fwd_kernel<T, D>, std::min(items, Fwd<D>::kBlocks * sm_count()), kFwdThreads, Fwd<D>::kSmem, s, mq, mk, mv, mo, a);
  count_launch();
  return true;
}

template <typename T, int D, bool LONG>
bool bwd(const AttnOp& a, cudaStream_t s) {
  const bool bf = std::is_same<T, bf16_t>::value;
  CUtensorMap mq, mk, mv, mdo, mq2, mk2, mv2, mdo2, mdq, mdk, mdv;   // in boxes of 64 and of 128 tokens
  if (!encode(&mq, a.q, a, bf, 64) || !encode(&mk, a.k, a, bf, 64) || !encode(&mv, a.v, a, bf, 64) ||
      !encode(&mdo, a.dout, a, bf, 64) || !encode(&mq2, a.q, a, bf, 128) || !encode(&mk2, a.k, a, bf, 128) ||
      !encode(&mv2, a.v, a, bf, 128) || !encode(&mdo2, a.dout, a, bf, 128) || !encode(&mdq, a.dq, a, bf, 128) || !encode(&mdk, a.dk, a, bf, 128) ||
      !encode(&mdv, a.dv, a, bf, 128))
    return false;
  static std::atomic<uint64_t> ready{0};
  allow_smem(attention_bwd_kernel<T, D, LONG>, Bwd<D, LONG>::kSmem, ready);
  const int items = a.B * a.nh * ((a.S + 127) / 128);
  launch_pdl(attention_bwd_kernel<T, D, LONG>, std::min(2 * items, sm_count()), kBwdThreads, Bwd<D, LONG>::kSmem, s, mq, mk, mv, mdo,
             mq2, mk2, mv2, mdo2, mdq, mdk, mdv, a);
  count_launch();
  return true;
}

template <typename T, bool BIAS>
bool bwd_one(const AttnOp& a, cudaStream_t s) {
  const bool bf = std::is_same<T, bf16_t>::value;
  CUtensorMap mq, mk, mv, mo, mdo, mdq, mdk, mdv;
  if (!encode(&mq, a.q, a, bf, 128) || !encode(&mk, a.k, a, bf, 128) || !encode(&mv, a.v, a, bf, 128) ||
      !encode(&mo, a.o, a, bf, 128) || !encode(&mdo, a.dout, a, bf, 128) || !encode(&mdq, a.dq, a, bf, 128) ||
      !encode(&mdk, a.dk, a, bf, 128) || !encode(&mdv, a.dv, a, bf, 128))
    return false;
  static std::atomic<uint64_t> ready{0};
  allow_smem(attention_bwd_one_kernel<T, BIAS>, One::kSmem, ready);
  launch_pdl(attention_bwd_one_kernel<T, BIAS>, a.B * a.nh, One::kThreads, One::kSmem, s, mq, mk, mv, mo, mdo, mdq, mdk, mdv, a);
  count_launch();
  return true;
}

}  // namespace

bool attention_tc_fwd_run(int dt, const AttnOp& a, cudaStream_t s) {
  if (dt == DT_F16) return a.d <= 64 ? fwd<half_t, 64>(a, s) : fwd<half_t, 128>(a, s);
  return a.d <= 64 ? fwd<bf16_t, 64>(a, s) : fwd<bf16_t, 128>(a, s);
}

bool attention_tc_bwd_run(int dt, const AttnOp& a, cudaStream_t s) {
  const bool h = dt == DT_F16;
  if (attn_one_tile(dt, a.S, a.d)) {
    if (a.vec) return h ? bwd_one<half_t, true>(a, s) : bwd_one<bf16_t, true>(a, s);
    return h ? bwd_one<half_t, false>(a, s) : bwd_one<bf16_t, false>(a, s);
  }
  if (a.d <= 64) return h ? bwd<half_t, 64, false>(a, s) : bwd<bf16_t, 64, false>(a, s);
  if (a.S >= kLongSeq) return h ? bwd<half_t, 128, true>(a, s) : bwd<bf16_t, 128, true>(a, s);
  return h ? bwd<half_t, 128, false>(a, s) : bwd<bf16_t, 128, false>(a, s);
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
