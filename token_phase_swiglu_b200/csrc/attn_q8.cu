// Attention of one token a sequence over an int8 KV cache (fmlp_attn_decode_q8):
//     o_h = softmax(scale q_h . K_g[0..L-1]) V_g[0..L-1],  g = h / G,
// where row j of K and V stands for int8 codes times an f32 scale (ks_j, vs_j).
//
// The codes go to the tensor cores as they are (tcgen05 kind::i8, exact 32-bit
// integer sums), so no thread ever unpacks a cache byte:
//     S^T[j, h] = K_j . Q_h      A = 128 rows of K, as stored (row-major)
//     O^T[d, h] = V^T[d, .] W_h  A = V transposed by the operand descriptor
// The few queries are the narrow operand.  A query value, over a power of two near its
// head's largest, is split into four int8 digits and a softmax weight, over its unit's
// largest, into three, as many columns a head, joined in f32 after the product: queries
// to 2^-30 of the largest (a bf16 value whose exponent is up to 22 lower exactly, so that
// an outlier does not coarsen the rest: three digits, the same width for up to 8 heads a KV
// head, would hold 2^-22), weights to 2^-24.
// With the scales,
//     s_j = (S^T joined) * power * ks_j * scale * log2 e,
//     weight of V's codes: 2^(s_j + log2 vs_j - M), M the unit's largest exponent,
// so a unit's product is exact against its own largest weight whatever the other
// units hold; units are then joined in f32 (accumulators in registers, one thread
// per column d of V), and l = sum 2^(s_j - m) runs beside it, per thread and row.
//
// Bound by HBM: 2 (D + 4) bytes a row and KV head, read once for its G heads.
// Roles of a CTA (one per SM, 11 warps): warp 8 streams units of 128 rows of K and V
// (TMA, 128-byte swizzle; columns past D and rows past n_max read zeros) and their
// scales (cp.async) into a ring, warp 9 issues the products, warp 10 splits the
// queries of the next segment, and two groups of four warps take the units in turn,
// one row (then one column of V) per thread; the group reads its unit's O only after
// the next unit's S, so neither waits for the tensor cores.  The units of all
// (sequence, KV head) regions are split evenly over the CTAs; a region cut by a
// border leaves f32 pieces in the workspace, merged in order by the last CTA.
//
// Measured on a B200: 16 sequences of up to 16k rows, 32 query heads over 8 KV heads of
// 128, 66-68 us (5.1 TB/s of cache, 78% of the measured copy rate); one sequence of 4096
// rows, 32 heads of 96, 15 us, where launch, lengths, first tiles and merge take most.
// At D = 64 a unit moves half the bytes through the same chain of waits: 8 sequences of up
// to 8k rows, 32 heads each with its KV head, 52 us (3.4 TB/s) against 59.6 us (5.8) of 128.
#include "common.cuh"
#include "internal.h"
#include "plan.cuh"
#include "ring.cuh"
#include "tcgen05.cuh"
#include "tmap.h"

#include <math_constants.h>

#include <algorithm>
#include <mutex>
#include <set>

namespace fmlp {
namespace {

constexpr int kU = 128;                 // rows of a unit
constexpr int kQ8Threads = 352;
constexpr int kQ8Producer = 8, kQ8Mma = 9, kQ8Split = 10;  // warps
constexpr int kQ8MaxSlots = 6;
constexpr int kQ8TileBytes = kU * 128;
constexpr int kQ8SlotBytes = 2 * kQ8TileBytes + 1024;  // K, V, then both rows of scales
constexpr int kQ8Header = 1024;
constexpr int kQ8MaxCtas = 256;
// A region costs its units and, to start and to finish, about as much as this many
// more; the shares of the CTAs are counted in both.  4 against 2 and 8: 8 sequences of up to
// 8k rows, 8 KV heads of 128 with 4 heads each 28.3 us (29.4, 28.4), 32 with one 59.6 (59.6,
// 61.0), of 64 with 4 heads 25.9 (26.9, 25.9), with one 52.2 (52.3, 54.0), with 16 34.8
// (40.6, 34.3).
constexpr int kRegionCost = 4;

struct Q8Params {
  CUtensorMap k_map, v_map;  // int8 [B H_kv][n_max][D], box 1 x 128 x 128
  const __nv_bfloat16* q;    // [B x H x D]
  const float *k_s, *v_s;    // [B x H_kv x n_max]
  const int32_t* kv_len;
  float* out;                // [B x H x D]
  float* partials;           // two slots a CTA: [G][3 + D]: m, l, reference of acc, acc
  uint32_t* counters;        // [kQ8MaxCtas] (zero between calls)
  Control ctl;
  int64_t B, n_max;
  int H, H_kv, G;
  float scale_log2;
  int slots;
};

// Columns of the score products (4 digits a head) and of those with V (3).
__host__ __device__ constexpr int q8_q_cols(int GP) { return (4 * GP + 15) / 16 * 16; }
__host__ __device__ constexpr int q8_w_cols(int GP) { return (3 * GP + 15) / 16 * 16; }

template <int GP>
struct Q8Shared {
  uint64_t full[kQ8MaxSlots], empty[kQ8MaxSlots];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], mma_done;
  uint32_t tmem;
  int abort, issued, last;
  UnitPlan<kQ8Threads> plan;
};
// After the header: the split queries and weights (swizzled operand tiles) and
// what the groups exchange.
template <int GP>
struct Q8Tiles {
  uint8_t q[2][q8_q_cols(GP) * 128];  // of the current segment and the next one
  uint8_t w[2][q8_w_cols(GP) * 128];  // of the two groups' units
  float acc[GP * kU];               // group 1's, joined by group 0
  float q_scale[2][GP];
  float top[2][2][4][GP];           // largest exponents: group, unit parity, warp
  float wm[8][GP], wl[8][GP];       // softmax maxima and sums of the warps
  float ref[GP];                    // group 1's reference
};

__device__ __forceinline__ uint32_t idesc_i8(int N) {  // int8 x int8 -> int32, M = 128
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kU >> 4) << 24);
}
constexpr uint32_t kTransposeA = 1u << 15;
template <bool kAccumulate>
__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " setp.ne.b32 p, %5, 0;\n"
      " tcgen05.mma.cta_group::1.kind::i8 [%0], a, b, %4, p;\n}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "n"(kSw128DescHi), "r"(idesc), "n"((int)kAccumulate));
}
__device__ __forceinline__ void tma_load_rows(void* dst, const void* tmap, int y, int z, uint64_t* bar,
                                              uint64_t policy) {
  tma_load_3d(dst, tmap, 0, y, z, bar, policy);
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(in ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Largest of a warp's values (NaN passed over).
__device__ __forceinline__ float warp_top(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// Byte of (row n, column c) in an operand tile of 128-byte rows, 128-byte swizzle.
__device__ __forceinline__ int tile_byte(int n, int c) {
  return n * 128 + (((c >> 4) ^ (n & 7)) << 4) + (c & 15);
}
// The four digits of an integer |x| <= 2^30 into rows n .. n + 3 of column c, lowest first,
// each within [-128, 127]: with 128 added to the lower three, they are the bytes of a sum.
__device__ __forceinline__ void split4(uint8_t* tile, int n, int c, int x) {
  const uint32_t d = ((uint32_t)x + 0x00808080u) ^ 0x00808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i) tile[tile_byte(n + i, c)] = (uint8_t)(d >> (8 * i));
}
// Their sums joined, in units of the highest digit.
__device__ __forceinline__ float join4(const uint32_t* s) {
  constexpr float kStep = 0x1p-8f;
  return fmaf(fmaf(fmaf((float)(int)s[0], kStep, (float)(int)s[1]), kStep, (float)(int)s[2]), kStep, (float)(int)s[3]);
}
// The three digits of y in [-127, 127] into rows n, n + 1, n + 2 of column c: y0 = rint(y),
// then what is left, times the base, twice.  Base 254 is the largest whose digits stay
// within +-127.  Adding 1.5 * 2^23 rounds to an integer whose two's complement is in the
// low bits.
constexpr float kBase = 254.f;
__device__ __forceinline__ void split3(uint8_t* tile, int n, int c, float y) {
  constexpr float kMagic = 12582912.f;
  const float b0 = y + kMagic, r1 = (y - (b0 - kMagic)) * kBase;
  const float b1 = r1 + kMagic, r2 = (r1 - (b1 - kMagic)) * kBase;
  const float b2 = r2 + kMagic;
  tile[tile_byte(n, c)] = (uint8_t)__float_as_uint(b0);
  tile[tile_byte(n + 1, c)] = (uint8_t)__float_as_uint(b1);
  tile[tile_byte(n + 2, c)] = (uint8_t)__float_as_uint(b2);
}
__device__ __forceinline__ float join3(const uint32_t* s) {
  return fmaf(fmaf((float)(int)s[2], 1.f / kBase, (float)(int)s[1]), 1.f / kBase, (float)(int)s[0]);
}
// 2^(a - b), with 2^(-inf - anything) = 0
__device__ __forceinline__ float ex2_diff(float a, float b) {
  return a == -CUDART_INF_F ? 0.f : ex2(a - b);
}
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N >= 32) tmem_ld<32>(addr, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
  if constexpr (N % 32) tmem_ld<16>(addr + N / 32 * 32, *reinterpret_cast<uint32_t(*)[16]>(&r[N / 32 * 32]));
  tmem_wait();
}

// A (sequence, KV head) region's units; an empty one still takes one (its zeros).
__device__ __forceinline__ int region_units(int len) { return max((len + kU - 1) / kU, 1); }

// Walks the segments (parts of regions) of a CTA's share.  Unit j of a region stands at
// cost kRegionCost + j behind its start, so a share may hold a region's start and none of
// its units: such segments are passed over.
struct Q8Walk {
  const Q8Params* p;
  int64_t u0, u1, region, b;  // the share; where the region starts, its sequence
  int g, len, units, j0, j1;
  __device__ __forceinline__ void load() {
    len = __ldg(p->kv_len + b);
    units = region_units(len);
  }
  __device__ __forceinline__ void cut() {
    j0 = (int)max(u0 - region - kRegionCost, (int64_t)0);
    j1 = (int)min(max(u1 - region - kRegionCost, (int64_t)0), (int64_t)units);
  }
  template <typename Plan>
  __device__ __forceinline__ bool start(const Q8Params& pp, const Plan& plan, int64_t begin, int64_t end) {
    p = &pp;
    u0 = begin;
    u1 = end;
    if (u0 >= u1) return false;
    b = plan.first_b;
    load();
    g = (int)((u0 - plan.first_prefix) / (units + kRegionCost));
    region = plan.first_prefix + (int64_t)g * (units + kRegionCost);
    cut();
    return j0 < j1 || next();
  }
  __device__ __forceinline__ bool next() {
    do {
      region += units + kRegionCost;
      if (region >= u1) return false;
      if (++g == p->H_kv) {
        g = 0;
        do {
          ++b;
          load();
        } while (len < 0 || len > p->n_max);  // more follow, so one is taken
      }
      cut();
    } while (j0 >= j1);
    return true;
  }
  __device__ __forceinline__ bool last() const { return region + units + kRegionCost >= u1; }
  __device__ __forceinline__ int count() const { return len ? j1 - j0 : 0; }  // units with rows
};

template <int D, int GP>
__global__ void __launch_bounds__(kQ8Threads, 1)
attn_decode_q8(const __grid_constant__ Q8Params p) {
  constexpr int NS = q8_q_cols(GP), NO = q8_w_cols(GP);  // columns of S and O
  constexpr uint32_t kTmemCols = GP <= 4 ? 64 : GP <= 8 ? 128 : 256;  // S, then O, of two groups
  static_assert(2 * (NS + NO) <= (int)kTmemCols, "tensor memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Q8Shared<GP>& sh = *reinterpret_cast<Q8Shared<GP>*>(smem);
  Q8Tiles<GP>& tl = *reinterpret_cast<Q8Tiles<GP>*>(smem + kQ8Header);
  uint8_t* ring = smem + kQ8Header + (sizeof(Q8Tiles<GP>) + 1023) / 1024 * 1024;
  static_assert(sizeof(Q8Shared<GP>) <= kQ8Header, "header");
  static_assert(NS % 8 == 0 && NO % 8 == 0, "operand tiles are whole swizzle atoms");

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.slots; ++i) {
      mbar_init(&sh.full[i], 1 + 32);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 32);
      mbar_init(&sh.q_empty[i], 1 + 8);  // the last product, and the groups' warps
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], kU);
      mbar_init(&sh.o_full[i], 1);
    }
    mbar_init(&sh.mma_done, 1);
    sh.abort = sh.issued = 0;
    sh.plan.total = 0;
    fence_barrier_init();
  }
  for (int i = threadIdx.x; i < (int)sizeof(tl.w) / 4; i += kQ8Threads)
    reinterpret_cast<uint32_t*>(&tl.w[0][0])[i] = 0;  // columns of no digit stay zero
  for (int i = threadIdx.x; i < (int)sizeof(tl.q) / 4; i += kQ8Threads)
    reinterpret_cast<uint32_t*>(&tl.q[0][0])[i] = 0;
  if (warp == kQ8Mma) tmem_alloc(&sh.tmem, kTmemCols);
  __syncthreads();
  grid_launch_dependents();
  grid_dependency_wait();  // every input may come from the previous kernel

  int64_t u0, u1;
  const int64_t ctas = plan_units(
      sh.plan, p.B,
      [&](int64_t b, bool first) -> int64_t {
        const int len = __ldg(p.kv_len + b);
        if (len < 0 || len > p.n_max) {  // refused: the sequence's outputs stay as they were
          if (first && blockIdx.x == 0) atomicOr(p.ctl.status, kStatusBadInput);
          return 0;
        }
        return (int64_t)p.H_kv * (region_units(len) + kRegionCost);
      },
      u0, u1);
  const int64_t total = sh.plan.total;
  const uint32_t tmem = sh.tmem;
  volatile int* abort = &sh.abort;
  const auto wait = [&](uint64_t* bar, int phase) {  // by a whole warp
    if (mbar_wait_warp(bar, (uint32_t)(phase & 1), p.ctl.wait_ns, abort)) return true;
    if (lane == 0) {
      sh.abort = 1;
      atomicOr(p.ctl.status, kStatusTimeout);
    }
    return false;
  };

  if (warp == kQ8Producer) {
    // ---------------- producer ----------------
    Q8Walk w;
    int k = 0;
    bool ok = true;
    const uint64_t pol = evict_first_policy();
    for (bool more = w.start(p, sh.plan, u0, u1); more && ok; more = w.next()) {
      const int64_t seg = w.b * p.H_kv + w.g;
      const int n = w.count();
      for (int i = 0; i < n; ++i, ++k) {
        const int slot = k % p.slots, row0 = (w.j0 + i) * kU;
        if (p.ctl.drop_last && i == n - 1 && w.last()) {  // testing
          ok = false;
          break;
        }
        if (k >= p.slots && !(ok = wait(&sh.empty[slot], k / p.slots - 1))) break;
        uint8_t* dst = ring + (size_t)slot * kQ8SlotBytes;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh.full[slot], 2 * kQ8TileBytes);  // boxes land whole
          tma_load_rows(dst, &p.k_map, row0, (int)seg, &sh.full[slot], pol);
          tma_load_rows(dst + kQ8TileBytes, &p.v_map, row0, (int)seg, &sh.full[slot], pol);
          sh.issued = k + 1;
        }
        float* sc = reinterpret_cast<float*>(dst + 2 * kQ8TileBytes);
        const int64_t s0 = seg * p.n_max + row0;
#pragma unroll
        for (int e = 0; e < kU; e += 32) {
          const bool in = row0 + e + lane < w.len;
          cp_async4(sc + e + lane, p.k_s + (in ? s0 + e + lane : 0), in);
          cp_async4(sc + kU + e + lane, p.v_s + (in ? s0 + e + lane : 0), in);
        }
        cp_async_arrive(&sh.full[slot]);
      }
    }
    __syncwarp();
  } else if (warp == kQ8Split) {
    // ---------------- queries of the segments, split into digits ----------------
    Q8Walk w;
    int s = 0;
    for (bool more = w.start(p, sh.plan, u0, u1); more; more = w.next()) {
      if (w.count() == 0) continue;
      const int buf = s & 1;
      float x[GP][D / 32];
#pragma unroll
      for (int h = 0; h < GP; ++h)
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          x[h][i] = h < p.G ? __bfloat162float(p.q[(w.b * p.H + (int64_t)w.g * p.G + h) * D + i * 32 + lane])
                            : 0.f;
      if (s >= 2 && !wait(&sh.q_empty[buf], s / 2 - 1)) break;
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        float top = 0.f, zero = 0.f;  // zero becomes NaN with a value that is not finite
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          top = fmaxf(top, fabsf(x[h][i]));
          zero = fmaf(x[h][i], 0.f, zero);
        }
        top = warp_top(top);
        const bool finite = __all_sync(0xffffffffu, zero == 0.f);
        // over a power of two, so that the largest lies in [2^29, 2^30); heads under 2^-98 are
        // all taken over 2^-127
        const uint32_t e = max((__float_as_uint(top) >> 23) & 255u, 29u);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          split4(tl.q[buf], 4 * h, i * 32 + lane, __float2int_rn(x[h][i] * __uint_as_float((283u - e) << 23)));
        // digits cannot say NaN: the scale does, and every score and sum of the head with it
        if (lane == 0) tl.q_scale[buf][h] = finite ? __uint_as_float((e - 5u) << 23) * p.scale_log2 : CUDART_NAN_F;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&sh.q_full[buf]);
      ++s;
    }
    __syncwarp();
  } else if (warp == kQ8Mma) {
    // ---------------- MMA issuer (one lane) ----------------
    if (elect_one()) {
      Q8Walk w;
      const uint32_t idesc_s = idesc_i8(NS), idesc_o = idesc_i8(NO) | kTransposeA;
      const uint32_t ring_lo = sw128_desc_lo(smem_u32(ring));
      const uint32_t q_lo[2] = {sw128_desc_lo(smem_u32(tl.q[0])), sw128_desc_lo(smem_u32(tl.q[1]))};
      const uint32_t w_lo[2] = {sw128_desc_lo(smem_u32(tl.w[0])), sw128_desc_lo(smem_u32(tl.w[1]))};
      const auto wait_one = [&](uint64_t* bar, int phase) {
        if (mbar_wait_bounded(bar, (uint32_t)(phase & 1), p.ctl.wait_ns, abort)) return true;
        sh.abort = 1;
        atomicOr(p.ctl.status, kStatusTimeout);
        return false;
      };
      int kq = 0, s = 0, i = 0;  // S products issued; segment and unit of the next one
      bool ok = true, more = w.start(p, sh.plan, u0, u1);
      while (more && w.count() == 0) more = w.next();
      const auto next_qk = [&]() {  // S^T of unit kq
        if (!more) return;
        if (i == 0 && !(ok = wait_one(&sh.q_full[s & 1], s / 2))) return;
        const int slot = kq % p.slots;
        if (!(ok = wait_one(&sh.full[slot], kq / p.slots))) return;
        tc_fence_after();
        const bool last = i + 1 == w.count();
        const uint32_t a = ring_lo + slot * (kQ8SlotBytes >> 4), b = q_lo[s & 1], d = tmem + (kq & 1) * NS;
        mma_i8<false>(d, a, b, idesc_s);
#pragma unroll
        for (int c = 1; c < D / 32; ++c) mma_i8<true>(d, a + c * 2, b + c * 2, idesc_s);
        mma_commit(&sh.s_full[kq & 1]);
        if (last) mma_commit(&sh.q_empty[s & 1]);
        ++kq;
        ++i;
        if (last) {
          ++s;
          i = 0;
          do more = w.next(); while (more && w.count() == 0);
        }
      };
      next_qk();
      if (ok) next_qk();
      for (int k = 0; ok && k < kq; ++k) {
        const int wg = k & 1, slot = k % p.slots;
        if (!(ok = wait_one(&sh.p_full[wg], k >> 1))) break;
        tc_fence_after();
        const uint32_t a = ring_lo + slot * (kQ8SlotBytes >> 4) + (kQ8TileBytes >> 4), b = w_lo[wg];
        const uint32_t d = tmem + 2 * NS + wg * NO;
        mma_i8<false>(d, a, b, idesc_o);
#pragma unroll
        for (int c = 1; c < kU / 32; ++c) mma_i8<true>(d, a + c * (4096 >> 4), b + c * 2, idesc_o);
        mma_commit(&sh.o_full[wg]);
        mma_commit(&sh.empty[slot]);
        next_qk();  // W of unit k is in, so its S has been read
      }
      if (sh.abort) {
        mma_commit(&sh.mma_done);
        mbar_wait_bounded(&sh.mma_done, 0, kDrainNs, nullptr);
      }
    }
    __syncwarp();
  } else {
    // ---------------- softmax groups ----------------
    const int wg = warp >> 2, r = threadIdx.x & (kU - 1);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // TMEM lanes 32 (warp % 4) ..
    Q8Walk w;
    int k = 0, s = 0;     // units and segments of the CTA so far
    int mine = 0;         // units of this group so far
    bool ok = true;
    for (bool more = w.start(p, sh.plan, u0, u1); more && ok; more = w.next()) {
      const int n = w.count();
      float m[GP], l[GP], ref[GP], acc[GP], top[GP], qs[GP];
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        m[h] = ref[h] = -CUDART_INF_F;
        l[h] = acc[h] = qs[h] = 0.f;
      }
      if (n) {
        ok = wait(&sh.q_full[s & 1], s / 2);
        if (ok) {
#pragma unroll
          for (int h = 0; h < GP; ++h) qs[h] = tl.q_scale[s & 1][h];
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.q_empty[s & 1]);
        }
        ++s;
      }
      bool pending = false;  // this group's last unit's O is still to be added
      const auto add_o = [&]() {
        ok = wait(&sh.o_full[wg], mine - 1);
        if (!ok) return;
        tc_fence_after();
        uint32_t o[NO];
        tmem_ld_cols<NO>(tmem + lanes + 2 * NS + wg * NO, o);
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          const float nref = fmaxf(ref[h], top[h]);
          acc[h] = acc[h] * ex2_diff(ref[h], nref) +
                   join3(o + 3 * h) * ex2_diff(top[h], nref);
          ref[h] = nref;
        }
      };
      for (int i = 0; i < n; ++i, ++k) {
        if ((k & 1) != wg) continue;
        const int slot = k % p.slots;
        if (ok) ok = wait(&sh.full[slot], k / p.slots) && wait(&sh.s_full[wg], mine);
        float sc[GP], exps[GP];
        if (ok) {
          tc_fence_after();
          const float* scales = reinterpret_cast<const float*>(ring + (size_t)slot * kQ8SlotBytes + 2 * kQ8TileBytes);
          const bool valid = (w.j0 + i) * kU + r < w.len;
          const float ks = scales[r], vs = scales[kU + r];
          const float lv = valid ? __log2f(vs) : -CUDART_INF_F;
          const float one = fmaf(vs, 0.f, 1.f);  // NaN for a scale of V that is not finite
          constexpr int kPart = NS < 32 ? NS : 32;  // columns read at a time
          uint32_t a[kPart];
#pragma unroll
          for (int h = 0; h < GP; ++h) {
            if (h % (kPart / 4) == 0) {
              __syncwarp();
              tmem_ld_cols<kPart>(tmem + lanes + wg * NS + 4 * h, a);
            }
            sc[h] = join4(a + 4 * h % kPart) * qs[h] * ks;
            if (valid) {  // running maximum and sum of this thread's rows
              const float d = sc[h] - m[h], e = ex2(-fabsf(d));
              l[h] = d > 0.f ? fmaf(l[h], e, one) : fmaf(e, one, l[h]);
              m[h] = fmaxf(m[h], sc[h]);
            }
            exps[h] = valid ? sc[h] + lv : -CUDART_INF_F;
            const float t = warp_top(exps[h]);
            if (lane == 0) tl.top[wg][mine & 1][warp & 3][h] = t;
          }
        }
        if (consumer_barrier_any<kU>(2 + wg, !ok)) {
          ok = false;
          break;
        }
        // a warp that gives up leaves at the next barrier, with its group
        if (pending) add_o();
        if (ok) {
#pragma unroll
          for (int h = 0; h < GP; ++h) {
            const float(*t)[GP] = tl.top[wg][mine & 1];
            top[h] = fmaxf(fmaxf(t[0][h], t[1][h]), fmaxf(t[2][h], t[3][h]));
            split3(tl.w[wg], 3 * h, r, 127.f * ex2_diff(exps[h], top[h]));
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          tc_fence_before();
          mbar_arrive(&sh.p_full[wg]);
        }
        ++mine;
        pending = true;
      }
      if (ok && pending) add_o();
      // ---- the segment's end: join the warps and the groups ----
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        const float wm = warp_top(m[h]);
        const float wl = warp_sum(l[h] * ex2_diff(m[h], wm));
        if (lane == 0) {
          tl.wm[warp][h] = wm;
          tl.wl[warp][h] = wl;
        }
        if (wg == 1) {
          tl.acc[h * kU + r] = acc[h];
          if (r == 0) tl.ref[h] = ref[h];
        }
      }
      if (consumer_barrier_any<2 * kU>(1, !ok)) break;
      const int64_t begin = w.region + kRegionCost;  // the CTAs of the region's first and last unit
      const int cf = share_of(begin, ctas, total), cl = share_of(begin + w.units - 1, ctas, total);
      float* out = p.out + (w.b * p.H + (int64_t)w.g * p.G) * D;
      const auto piece = [&](int c, int h) {
        return p.partials + ((size_t)(c == cf ? 2 * c + 1 : 2 * c) * p.G + h) * (3 + D);
      };
      if (wg == 0) {
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          if (h >= p.G) break;
          float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
          for (int x = 0; x < 8; ++x) M = fmaxf(M, tl.wm[x][h]);
#pragma unroll
          for (int x = 0; x < 8; ++x) L += tl.wl[x][h] * ex2_diff(tl.wm[x][h], M);
          const float R = fmaxf(ref[h], tl.ref[h]);
          const float A = acc[h] * ex2_diff(ref[h], R) + tl.acc[h * kU + r] * ex2_diff(tl.ref[h], R);
          if (cf == cl) {
            if (r < D) out[h * D + r] = L == 0.f ? 0.f : A * ex2_diff(R, M) / (127.f * L);
          } else {
            float* pc = piece((int)blockIdx.x, h);
            if (r < 3) pc[r] = r == 0 ? M : r == 1 ? L : R;
            if (r < D) pc[3 + r] = A;
          }
        }
      }
      if (cf != cl) {
        if (wg == 0) {
          __threadfence();
          named_barrier_sync(2, kU);
          if (r == 0) sh.last = atomicAdd(p.counters + cf, 1u) == (uint32_t)(cl - cf);
        }
        named_barrier_sync(1, 2 * kU);
        if (sh.last) {  // a warp per head; a lane per piece, then per column
          __threadfence();
          for (int h = warp; h < p.G; h += 8) {
            float M = -CUDART_INF_F, R = -CUDART_INF_F, L = 0.f, A[D / 32];
#pragma unroll
            for (int i = 0; i < D / 32; ++i) A[i] = 0.f;
            for (int c = cf + lane; c <= cl; c += 32) {
              M = fmaxf(M, __ldcg(piece(c, h)));
              R = fmaxf(R, __ldcg(piece(c, h) + 2));
            }
            M = warp_top(M);
            R = warp_top(R);
            for (int c0 = cf; c0 <= cl; c0 += 32) {
              float f = 0.f;
              if (c0 + lane <= cl) {
                const float* pc = piece(c0 + lane, h);
                L = fmaf(__ldcg(pc + 1), ex2_diff(__ldcg(pc), M), L);
                f = ex2_diff(__ldcg(pc + 2), R);
              }
              const int n = min(32, cl - c0 + 1);
#pragma unroll 4
              for (int k = 0; k < n; ++k) {
                const float* pc = piece(c0 + k, h) + 3 + lane;
                const float fk = __shfl_sync(0xffffffffu, f, k);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) A[i] = fmaf(__ldcg(pc + 32 * i), fk, A[i]);
              }
            }
            L = warp_sum(L);
            const float s = L == 0.f ? 0.f : ex2_diff(R, M) / (127.f * L);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) out[h * D + lane + 32 * i] = A[i] * s;
          }
          if (threadIdx.x == 0) atomicExch(p.counters + cf, 0u);
        }
      }
      if (consumer_barrier_any<2 * kU>(1, false)) break;  // what was exchanged is written again
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && sh.abort)  // copies in flight land in this CTA's memory
    for (int k = max(0, sh.issued - p.slots); k < sh.issued; ++k)
      mbar_wait_bounded(&sh.full[k % p.slots], (uint32_t)((k / p.slots) & 1), kDrainNs, nullptr);
  __syncthreads();
  if (warp == kQ8Mma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <int D, int GP>
cudaError_t launch_q8_t(Q8Params& p, const DeviceInfo& dev, cudaStream_t stream) {
  static std::mutex mu;
  static std::set<int> done;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done.count(dev.device)) {
      cudaError_t e = cudaFuncSetAttribute(attn_decode_q8<D, GP>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           dev.max_smem_optin);
      if (e != cudaSuccess) return e;
      done.insert(dev.device);
    }
  }
  const size_t fixed = 1024 + kQ8Header + (sizeof(Q8Tiles<GP>) + 1023) / 1024 * 1024;
  p.slots = (int)std::min<size_t>(kQ8MaxSlots, (dev.max_smem_optin - fixed) / kQ8SlotBytes);
  if (p.slots < 3) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  const int64_t most = p.B * p.H_kv * ((p.n_max + kU - 1) / kU);
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(std::min(dev.sm_count, kQ8MaxCtas), most));
  cfg.blockDim = dim3(kQ8Threads);
  cfg.dynamicSmemBytes = fixed + (size_t)p.slots * kQ8SlotBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, attn_decode_q8<D, GP>, p);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

template <int D>
cudaError_t launch_q8_d(Q8Params& p, const DeviceInfo& dev, cudaStream_t stream) {
  // compiled for the next power of two of heads (columns of the others are zero)
  if (p.G <= 1) return launch_q8_t<D, 1>(p, dev, stream);
  if (p.G <= 2) return launch_q8_t<D, 2>(p, dev, stream);
  if (p.G <= 4) return launch_q8_t<D, 4>(p, dev, stream);
  if (p.G <= 8) return launch_q8_t<D, 8>(p, dev, stream);
  return launch_q8_t<D, 16>(p, dev, stream);
}

}  // namespace

bool attn_q8_shape_ok(int H, int H_kv) { return H % H_kv == 0 && H / H_kv <= 16; }

AttnLayout attn_q8_layout(int H, int H_kv, int D) {
  AttnLayout z;
  static_assert(kQ8MaxCtas * sizeof(uint32_t) <= kPackedCounterBytes, "counters");
  z.counters = kPackedCounters;
  z.partials = z.counters + kPackedCounterBytes;
  z.total = z.partials + (size_t)2 * kQ8MaxCtas * (H / H_kv) * (3 + D) * sizeof(float);
  return z;
}

cudaError_t launch_attn_decode_q8(const void* q, const void* k_q, const float* k_s, const void* v_q,
                                  const float* v_s, const int32_t* kv_len, int64_t B, int H,
                                  int H_kv, int D, int64_t n_max, float scale, float* out,
                                  void* workspace, const DeviceInfo& dev, cudaStream_t stream) {
  const AttnLayout z = attn_q8_layout(H, H_kv, D);
  Q8Params p = {};
  p.q = (const __nv_bfloat16*)q;
  p.k_s = k_s;
  p.v_s = v_s;
  p.kv_len = kv_len;
  p.out = out;
  p.counters = (uint32_t*)((char*)workspace + z.counters);
  p.partials = (float*)((char*)workspace + z.partials);
  p.ctl.status = (uint32_t*)workspace;
  p.ctl.wait_ns = wait_timeout_ns();
  p.ctl.drop_last = fault_injection();
  p.B = B;
  p.n_max = n_max;
  p.H = H;
  p.H_kv = H_kv;
  p.G = H / H_kv;
  p.scale_log2 = scale * 1.44269504f;
  cudaError_t e = encode_tmap_rows_i8(&p.k_map, k_q, (uint64_t)D, (uint64_t)n_max, (uint64_t)(B * H_kv), kU);
  if (e == cudaSuccess)
    e = encode_tmap_rows_i8(&p.v_map, v_q, (uint64_t)D, (uint64_t)n_max, (uint64_t)(B * H_kv), kU);
  if (e != cudaSuccess) return e;
  switch (D) {
    case 64: return launch_q8_d<64>(p, dev, stream);
    case 96: return launch_q8_d<96>(p, dev, stream);
    case 128: return launch_q8_d<128>(p, dev, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fmlp
