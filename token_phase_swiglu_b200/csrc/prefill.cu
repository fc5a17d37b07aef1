// Causal attention of a packed batch over its KV cache (fmlp_attn_prefill).
//
// For token i of sequence b (n new tokens, L rows held with them), at position
// p = L - n + i, and query head h of KV head g = h / G:
//     o = softmax(scale q . K_g[0..p]) V_g[0..p]
// in one pass over the rows, 128 at a time, with a running reference m and sum l
// of every query row (base 2: scores carry scale * log2 e):
//     w = 2^(s - m),  l <- l + sum w,  O <- O + w V,  o = O / l at the end.
// m follows the running maximum lazily: l and O are rescaled only when a row's
// maximum has grown by more than 8 (a factor of 256), so that w stays below 2^8
// and the rescaling of O, in TMEM, is rare; o is exact for any reference.
//
// Rows of a tile.  The G query heads of a KV head share its rows, so a tile of
// the tensor cores' 128 rows holds TPT = floor(128 / G) tokens times G heads
// (row = token * G + head), and a work item, one (sequence, pair of tiles, KV
// head), 2 TPT tokens.  One K tile and one V tile then serve 256 query rows of
// a prompt, and a few tokens of a verify or decode batch still read the cache
// once for all their heads.
//
// Roles of a CTA (one per SM, 10 warps): warp 8 streams Q tiles and the ring of
// K and V tiles by TMA (128-byte swizzle, 64-column blocks; columns past D = 96
// and rows past n_max read zeros), warp 9 issues the tcgen05 products
//     S = Q K^T  (both operands in shared memory, f32 in TMEM)
//     O += W V   (W bf16 in TMEM over the S it came from, V as a
//                 column-major operand straight from its row-major tile)
// and warps 0-3 and 4-7 hold one query row per thread of the two tiles and turn S
// into W.  The two 64-row halves of a unit have their own S and barriers: while the
// products of one are under way (O += W V, then the next unit's S of that half), the
// softmax works on the other.  W is rounded to bf16 (half a step, 2^-8 relative at
// most): it must match V's type, and the output is bf16 as well.  l sums the
// unrounded w.
//
// Schedule.  The 128-row units of all items (one KV tile against one pair of
// query tiles) are split evenly and contiguously over the CTAs, a fixed cost for
// each item's start and end counted with them (a prompt of 8192 tokens took 962 us
// without it, 600 with), so a long cache read by few tokens is spread over the whole
// GPU and ragged prompts balance.
// An item cut by a CTA border leaves f32 pieces (m, l, O) in the workspace; the
// last CTA to finish merges them in order (nobody waits on another CTA).  Every
// CTA finds its first unit from the device-side lengths: the units of a
// sequence are a sum of rounded-up arithmetic terms, which has a closed form.
//
// Measured on a B200 (32 query heads over 8 KV heads of 128; back to back in a graph, and
// as one pass among others): a prompt of 8192 tokens 508-565 and 580 us (1080-950 TFLOP/s,
// under the power cap), of 2048 tokens 60 and 60 us (570 TFLOP/s), 4 tokens of 32 sequences
// over caches of 4k rows 107 and 121 us (5.0 and 4.5 TB/s).
// Prompts are bound by the products: scores of 64 rows at a time read shared memory
// at its limit (48 cycles for 32 of work), but with 128 rows at once, which leaves no
// room in TMEM for a second set, the softmax waits for them and the prompt of 8192
// tokens takes 614 us.  Short ones are bound by starting and finishing items.
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

constexpr int kTile = 128;                    // query rows of a tile, KV rows of a unit
constexpr int kPfThreads = 320;
constexpr int kPfProducer = 8, kPfMma = 9;    // warps
constexpr int kPfBlock = kTile * 128;         // bytes of 128 rows x 64 bf16 columns
constexpr int kPfMaxSlots = 8;
constexpr int kPfMaxCtas = 256;
constexpr int kPfHeader = 1024;
constexpr float kRescaleAbove = 8.f;
// An item costs its units and, to start (Q, the first K) and to finish (O), about as
// much as this many more; the shares of the CTAs are counted in both.  2 against 1 and 4:
// five prompts of up to 1500 tokens, 16 heads of 128 over 4 70.3 us (71.9, 73.4), over 16
// 81.5 (83.7, 82.4); of 64 54.1 (52.8, 58.2) and 56.9 (55.5, 60.1).
constexpr int kPfItemCost = 2;
// TMEM columns: S of the two tiles in halves of 64 (W over the first 32 of each), O of them
constexpr uint32_t kColS = 0, kColO = 256, kPfTmemCols = 512;

struct PrefillParams {
  CUtensorMap q_map;   // [T][H_kv][G][D], box TPT x 1 x G x 64
  CUtensorMap k_map;   // [B H_kv][n_max][D], box 1 x 128 x 64
  CUtensorMap v_map;
  CUtensorMap o_map;   // out, boxes as of q
  __nv_bfloat16* out;  // [T x H x D]
  const int32_t* cu;
  const int32_t* kv_len;
  float* partials;     // two slots a CTA, see piece()
  uint32_t* counters;  // [2 kPfMaxCtas] arrivals (zero between calls)
  Control ctl;
  int64_t B;
  int T, H, H_kv, G;
  int64_t n_max;
  float scale_log2;    // scale * log2(e)
  int slots;           // K/V tiles in the ring
  int piece_rows;      // rows of a tile that a piece holds
  int piece_tiles;     // 1 if no item has a second tile
};

struct PfBarriers {
  uint64_t q_full, q_empty;
  uint64_t kv_full[kPfMaxSlots], kv_empty[kPfMaxSlots];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2], o_full[2], mma_done;  // [tile][half]
  uint32_t tmem;
  int abort, q_issued, kv_issued;
  int last[2];
  int first_p;               // pair of this CTA's first unit
  UnitPlan<kPfThreads> plan;
};
static_assert(sizeof(PfBarriers) <= kPfHeader, "header");

// sum over k = 0 .. n-1 of floor((a k + b) / kTile), for a > 0 and b >= 0: what the terms
// a k + b add up to, less their remainders.  With g the largest power of two that divides
// both a and kTile, the remainders repeat every P = kTile / g terms, and a period meets each
// of b mod g, b mod g + g, ... once; the last, incomplete period (at most 63 terms, none or
// one for up to 4 heads a KV head) is gone through.
__device__ __forceinline__ int64_t tiles_below(int64_t n, int a, int64_t b) {
  const int g = min(a & -a, kTile), P = kTile / g, rest = (int)(n & (P - 1));
  int64_t left = (n - rest) / P * (P * (int)(b & (g - 1)) + kTile * (P - 1) / 2);
  int r = (int)(b & (kTile - 1));
#pragma unroll 1
  for (int k = 0; k < rest; ++k) {
    left += r;
    r = (r + a) & (kTile - 1);
  }
  return (a * (n * (n - 1) / 2) + b * n - left) / kTile;
}

// One sequence's place in the batch.
struct Sequence {
  int c0, n, len, pairs;  // first token, new tokens, rows held, pairs of tiles (0: nothing to do)
  bool bad;
};
__device__ __forceinline__ Sequence sequence(const PrefillParams& p, int64_t b, int TP) {
  Sequence s;
  s.c0 = __ldg(p.cu + b);
  const int c1 = __ldg(p.cu + b + 1);
  s.len = __ldg(p.kv_len + b);
  s.bad = s.c0 < 0 || c1 < s.c0 || c1 > p.T || s.len < 0 || s.len > p.n_max;
  s.n = s.bad ? 0 : c1 - s.c0;
  s.pairs = (s.n + TP - 1) / TP;
  return s;
}
// KV units that tokens up to `end` (exclusive) of a sequence see.
__device__ __forceinline__ int units_to(const Sequence& s, int end) {
  return (max(s.len - s.n + end, 0) + kTile - 1) / kTile;
}
// Units of pair i of a sequence; a pair of padding tokens still takes one (its zeros).
__device__ __forceinline__ int pair_units(const Sequence& s, int i, int TP) {
  return max(units_to(s, min((i + 1) * TP, s.n)), 1);
}
// Cost of the items of one KV head before pair i (all of them whole).  Called, not inlined:
// the roles that start with it stay smaller (nine ragged prompts of D = 64: 86.5 us inlined,
// 83.8 called).
__device__ __noinline__ int64_t cost_before(const Sequence& s, int i, int TP) {
  const int base = s.len - s.n;  // pair k ends at base + (k + 1) TP
  const int lead = base >= 0 ? 0 : min(i, -base / TP);  // pairs of padding only
  const int64_t fixed = (int64_t)i * kPfItemCost + lead;
  if (i == lead) return fixed;
  return fixed + tiles_below(i - lead, TP, (int64_t)base + (int64_t)(lead + 1) * TP + kTile - 1);
}
__device__ __forceinline__ int64_t sequence_cost(const Sequence& s, int TP, int H_kv) {
  if (s.pairs == 0) return 0;
  return H_kv * (cost_before(s, s.pairs - 1, TP) + pair_units(s, s.pairs - 1, TP) + kPfItemCost);
}

// Walks the segments (parts of items) of a CTA's share.  Unit j of an item stands at
// cost kPfItemCost + j behind the item's start, so a share may hold an item's start and
// none of its units: such segments are passed over.
struct Walk {
  const PrefillParams* p;
  int TP;
  int64_t u0, u1;      // the share
  int64_t item, b;     // where the item starts; its sequence,
  Sequence s;
  int pair, g, units;  // pair, KV head and units
  int j0, j1;          // this segment's units
  __device__ __forceinline__ void cut() {
    j0 = (int)max(u0 - item - kPfItemCost, (int64_t)0);
    j1 = (int)min(max(u1 - item - kPfItemCost, (int64_t)0), (int64_t)units);
  }
  __device__ __forceinline__ bool start(const PrefillParams& pp, const PfBarriers& sh, int TPT,
                                        int64_t begin, int64_t end) {
    p = &pp;
    TP = 2 * TPT;
    u0 = begin;
    u1 = end;
    if (u0 >= u1) return false;
    b = sh.plan.first_b;
    s = sequence(pp, b, TP);
    pair = sh.first_p;
    units = pair_units(s, pair, TP);
    const int64_t pair0 = sh.plan.first_prefix + pp.H_kv * cost_before(s, pair, TP);
    g = (int)((u0 - pair0) / (units + kPfItemCost));
    item = pair0 + (int64_t)g * (units + kPfItemCost);
    cut();
    return j0 < j1 || next();
  }
  __device__ __forceinline__ bool next() {
    do {
      item += units + kPfItemCost;
      if (item >= u1) return false;
      if (++g == p->H_kv) {
        g = 0;
        if (++pair == s.pairs) {
          pair = 0;
          do s = sequence(*p, ++b, TP); while (s.pairs == 0);  // more follow, so one has some
        }
        units = pair_units(s, pair, TP);
      }
      cut();
    } while (j0 >= j1);
    return true;
  }
  // Halves (64 rows) that tile t sees of unit j < end_unit(t).
  __device__ __forceinline__ int halves(int t, int j) const {
    const int rows = s.len - s.n + first_token(t) + tokens(t) - j * kTile;
    return rows > kTile / 2 ? 2 : 1;
  }
  __device__ __forceinline__ bool last() const { return item + units + kPfItemCost >= u1; }
  // Tile t's tokens and the end of its units within this segment.
  __device__ __forceinline__ int first_token(int t) const { return pair * TP + t * (TP / 2); }
  __device__ __forceinline__ int tokens(int t) const {
    return min(max(s.n - first_token(t), 0), TP / 2);
  }
  __device__ __forceinline__ int end_unit(int t) const {
    const int k = tokens(t);
    return k ? max(j0, min(j1, units_to(s, first_token(t) + k))) : j0;
  }
};

__device__ __forceinline__ void tma_load_kv(void* dst, const void* tmap, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_q(void* dst, const void* tmap, int x, int g, int t,
                                           uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(smem_u32(dst)), "l"(tmap), "r"(x), "r"(0), "r"(g), "r"(t), "r"(smem_u32(bar)) : "memory");
}

// V as the B operand: element (k = row, n = column) of row-major rows of 64 columns (128
// bytes, swizzled), groups of 8 rows 1024 bytes apart, blocks of 64 columns kPfBlock apart.
__device__ __forceinline__ uint32_t desc_v(uint32_t saddr) {
  return (saddr >> 4) | ((uint32_t)(kPfBlock >> 4) << 16);
}
constexpr uint32_t kTransposeB = 1u << 16;

// D (TMEM) = A B^T or += it: A and B in shared memory, or A as bf16 in TMEM.
template <bool kAccumulate>
__device__ __forceinline__ void pf_mma(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " setp.ne.b32 p, %5, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "n"(kSw128DescHi), "r"(idesc), "n"((int)kAccumulate));
}
__device__ __forceinline__ void pf_mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n mov.b64 b, {%2, %3};\n setp.ne.b32 p, %5, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "n"(kSw128DescHi), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void unpk2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// s[0..63] <- w = 2^(s sc + nref) as 32 bf16 pairs in s[0..31]; sum += w.  (A quarter of
// the exponentials as polynomials on the FMA pipes made an 8192-token prompt 4% slower:
// the exp2 unit is not what the kernel waits for.)
__device__ __forceinline__ void weights(uint32_t (&s)[64], uint64_t sc2, uint64_t nref2,
                                        uint64_t (&sum)[2]) {
#pragma unroll
  for (int i = 0; i < 64; i += 2) {
    float x, y;
    unpk2(ffma2(pk2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), sc2, nref2), x, y);
    x = ex2(x);
    y = ex2(y);
    sum[(i >> 1) & 1] = fadd2(sum[(i >> 1) & 1], pk2(x, y));
    s[i >> 1] = bf16x2(x, y);
  }
}

__device__ __forceinline__ void tma_store_out(const void* tmap, const void* src, int x, int g, int t) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
          tmap),
      "r"(x), "r"(0), "r"(g), "r"(t), "r"(smem_u32(src))
      : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_read_wait() {  // the source may be written again
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1)
attn_prefill(const __grid_constant__ PrefillParams p) {
  constexpr int kBlocks = (D + 63) / 64;             // 64-column blocks of a row
  constexpr int kTileBytes = kBlocks * kPfBlock;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  PfBarriers& sh = *reinterpret_cast<PfBarriers*>(smem);
  uint8_t* q_smem = smem + kPfHeader;
  uint8_t* o_smem = q_smem + 2 * kTileBytes;         // 64 columns of each tile's output
  uint8_t* kv_smem = o_smem + 2 * kPfBlock;

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int TPT = kTile / p.G, TP = 2 * TPT;

  if (threadIdx.x == 0) {
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    for (int i = 0; i < p.slots; ++i) {
      mbar_init(&sh.kv_full[i], 1);
      mbar_init(&sh.kv_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sh.s_full[t][h], 1);
        mbar_init(&sh.p_full[t][h], kTile);
      }
      mbar_init(&sh.pv_done[t], 1);
      mbar_init(&sh.o_full[t], 1);
    }
    mbar_init(&sh.mma_done, 1);
    sh.abort = sh.q_issued = sh.kv_issued = 0;
    sh.plan.total = 0;
    fence_barrier_init();
  }
  if (warp == kPfMma) tmem_alloc(&sh.tmem, kPfTmemCols);
  __syncthreads();
  grid_launch_dependents();
  grid_dependency_wait();  // every input may come from the previous kernel

  int64_t u0, u1;
  const int64_t ctas = plan_units(
      sh.plan, p.B,
      [&](int64_t b, bool first) {
        const Sequence s = sequence(p, b, TP);
        if (first && s.bad && blockIdx.x == 0) atomicOr(p.ctl.status, kStatusBadInput);
        return sequence_cost(s, TP, p.H_kv);
      },
      u0, u1);
  const int64_t total = sh.plan.total;
  if (u0 < u1) {
    if (warp == 0) {  // the pair: a 32-ary search over the closed form
      const Sequence s = sequence(p, sh.plan.first_b, TP);
      const int64_t local = u0 - sh.plan.first_prefix;
      int lo = 0, hi = s.pairs;
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const bool le = at < hi && p.H_kv * cost_before(s, at, TP) <= local;
        const int k = __popc(__ballot_sync(0xffffffffu, le));  // lane 0's holds: at least 1
        lo += (k - 1) * step;
        hi = min(hi, lo + step);
      }
      if (lane == 0) sh.first_p = lo;
    }
    __syncthreads();
  }
  const uint32_t tmem = sh.tmem;
  volatile int* abort = &sh.abort;
  const uint64_t wait_ns = p.ctl.wait_ns;

  if (warp == kPfProducer) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      Walk w;
      int nq = 0, nkv = 0;  // Q loads, K/V tiles issued
      bool ok = true;
      for (bool more = w.start(p, sh, TPT, u0, u1); more && ok; more = w.next()) {
        const int jend = max(w.end_unit(0), w.end_unit(1));
        if (jend == w.j0) continue;
        if (nq > 0 && !mbar_wait_bounded(&sh.q_empty, (uint32_t)((nq - 1) & 1), wait_ns, abort)) {
          sh.abort = 1;
          atomicOr(p.ctl.status, kStatusTimeout);
          ok = false;
          break;
        }
        const int tiles = w.tokens(1) ? 2 : 1;
        mbar_arrive_expect_tx(&sh.q_full, (uint32_t)(tiles * kBlocks * TPT * p.G * 128));
        for (int t = 0; t < tiles; ++t)
          for (int z = 0; z < kBlocks; ++z)
            tma_load_q(q_smem + t * kTileBytes + z * kPfBlock, &p.q_map, z * 64, w.g,
                       w.s.c0 + w.first_token(t), &sh.q_full);
        sh.q_issued = ++nq;
        const int seg = (int)(w.b * p.H_kv + w.g);
        for (int j = w.j0; j < jend && ok; ++j) {
          for (int kv = 0; kv < 2; ++kv) {
            const int slot = nkv % p.slots;
            if (p.ctl.drop_last && kv && j == jend - 1 && w.last()) {
              ok = false;  // testing: withhold the last tile
              break;
            }
            if (nkv >= p.slots &&
                !mbar_wait_bounded(&sh.kv_empty[slot], (uint32_t)((nkv / p.slots - 1) & 1), wait_ns,
                                   abort)) {
              sh.abort = 1;
              atomicOr(p.ctl.status, kStatusTimeout);
              ok = false;
              break;
            }
            uint8_t* dst = kv_smem + slot * kTileBytes;
            mbar_arrive_expect_tx(&sh.kv_full[slot], kTileBytes);
            for (int z = 0; z < kBlocks; ++z)
              tma_load_kv(dst + z * kPfBlock, kv ? &p.v_map : &p.k_map, z * 64, j * kTile, seg,
                          &sh.kv_full[slot]);
            sh.kv_issued = ++nkv;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == kPfMma) {
    // ---------------- MMA issuer ----------------
    if (elect_one()) {
      Walk w;
      int nq = 0, nkv = 0;              // Q loads and K/V tiles consumed
      int np[2][2] = {{0, 0}, {0, 0}};  // W halves consumed
      bool ok = true;
      constexpr uint32_t kIdescS = idesc_bf16(kTile / 2), kIdescO = idesc_bf16(D) | kTransposeB;
      const uint32_t q_lo = sw128_desc_lo(smem_u32(q_smem)), kv_addr = smem_u32(kv_smem);
      const auto wait = [&](uint64_t* bar, int phase) {
        if (mbar_wait_bounded(bar, (uint32_t)(phase & 1), wait_ns, abort)) return true;
        sh.abort = 1;
        atomicOr(p.ctl.status, kStatusTimeout);
        return false;
      };
      const auto qk = [&](int t, int h, int slot) {  // half h of S_t = Q_t K^T
        const uint32_t a = q_lo + t * (kTileBytes >> 4);
        const uint32_t b = sw128_desc_lo(kv_addr + slot * kTileBytes + h * (kPfBlock / 2));
        const uint32_t d = tmem + kColS + t * kTile + h * 64;
        pf_mma<false>(d, a, b, kIdescS);
#pragma unroll
        for (int k = 1; k < D / 16; ++k) {
          const uint32_t off = ((k / 4) * kPfBlock + (k % 4) * 32) >> 4;
          pf_mma<true>(d, a + off, b + off, kIdescS);
        }
        mma_commit(&sh.s_full[t][h]);
      };
      for (bool more = w.start(p, sh, TPT, u0, u1); more && ok; more = w.next()) {
        const int end[2] = {w.end_unit(0), w.end_unit(1)};
        const int jend = max(end[0], end[1]);
        if (jend == w.j0) continue;
        if (!wait(&sh.q_full, nq)) break;
        ++nq;
        // the tiles arrive K, V, K, V, ...
        int k_slot = nkv % p.slots;
        if (!wait(&sh.kv_full[k_slot], nkv / p.slots)) break;
        ++nkv;
        tc_fence_after();
        int have[2] = {end[0] > w.j0 ? w.halves(0, w.j0) : 0, end[1] > w.j0 ? w.halves(1, w.j0) : 0};
        for (int h = 0; h < 2; ++h)
          for (int t = 0; t < 2; ++t)
            if (h < have[t]) qk(t, h, k_slot);
        mma_commit(&sh.kv_empty[k_slot]);
        if (jend == w.j0 + 1) mma_commit(&sh.q_empty);  // Q has had its last product
        for (int j = w.j0; j < jend; ++j) {
          const int v_slot = nkv % p.slots;
          if (!(ok = wait(&sh.kv_full[v_slot], nkv / p.slots))) break;
          ++nkv;
          const bool more_k = j + 1 < jend;
          if (more_k) {
            k_slot = nkv % p.slots;
            if (!(ok = wait(&sh.kv_full[k_slot], nkv / p.slots))) break;
            ++nkv;
          }
          const int next[2] = {j + 1 < end[0] ? w.halves(0, j + 1) : 0, j + 1 < end[1] ? w.halves(1, j + 1) : 0};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (h >= have[t] || !ok) continue;
              if (!(ok = wait(&sh.p_full[t][h], np[t][h]))) continue;
              ++np[t][h];
              tc_fence_after();
              const uint32_t v = desc_v(kv_addr + v_slot * kTileBytes + h * (kPfBlock / 2));
              const uint32_t d = tmem + kColO + t * kTile;
              const uint32_t a = tmem + kColS + t * kTile + h * 64;
              pf_mma_ta(d, a, v, kIdescO, j > w.j0 || h > 0);
#pragma unroll
              for (int k = 1; k < 4; ++k)
                pf_mma_ta(d, a + k * 8, v + k * (2048 >> 4), kIdescO, 1);
              mma_commit(&sh.pv_done[t]);
              if (j + 1 >= end[t] && h + 1 >= have[t]) mma_commit(&sh.o_full[t]);
              if (h < next[t]) qk(t, h, k_slot);
            }
          }
          if (!ok) break;
          have[0] = next[0];
          have[1] = next[1];
          mma_commit(&sh.kv_empty[v_slot]);
          if (more_k) {
            mma_commit(&sh.kv_empty[k_slot]);
            if (j + 2 == jend) mma_commit(&sh.q_empty);
          }
        }
      }
      if (sh.abort) {  // MMAs in flight read shared memory and write TMEM
        mma_commit(&sh.mma_done);
        mbar_wait_bounded(&sh.mma_done, 0, kDrainNs, nullptr);
      }
    }
    __syncwarp();
  } else {
    // ---------------- softmax: thread = query row ----------------
    const int t = warp >> 2, r = threadIdx.x & (kTile - 1), wl = (warp & 3) * 32;
    const uint32_t lane_base = (uint32_t)wl << 16;
    const uint32_t s_addr = tmem + lane_base + kColS + t * kTile;
    const uint32_t o_addr = tmem + lane_base + kColO + t * kTile;
    const int tok_r = r / p.G, head_r = r % p.G;
    Walk w;
    int ns[2] = {0, 0};  // halves of S consumed
    int no = 0;          // finished O taken
    int nu = 0;          // units of the CTA before this segment
    const auto wait = [&](uint64_t* bar, int phase) {
      if (mbar_wait_warp(bar, (uint32_t)(phase & 1), wait_ns, abort)) return true;
      if (lane == 0) {
        sh.abort = 1;
        atomicOr(p.ctl.status, kStatusTimeout);
      }
      return false;
    };
    for (bool more = w.start(p, sh, TPT, u0, u1); more; more = w.next()) {
      const int ntok = w.tokens(t), unit0 = nu;
      nu += max(w.end_unit(0), w.end_unit(1)) - w.j0;
      if (ntok == 0) continue;
      const int jend = w.end_unit(t);
      const bool row_ok = tok_r < ntok && r < TPT * p.G;
      const bool warp_ok = wl < ntok * p.G;  // some row of the warp counts
      const int first = w.first_token(t);
      // rows past the tile's tokens follow the last one (their results go nowhere)
      const int rows = w.s.len - w.s.n + first + min(tok_r, ntok - 1) + 1;  // KV rows it sees
      float m = -CUDART_INF_F, l = 0.f;
      bool ok = true;
      for (int j = w.j0; j < jend && ok; ++j) {
        const int held = w.s.len - j * kTile;
        const int halves = w.halves(t, j);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h >= halves || !ok) continue;
          if (!(ok = wait(&sh.s_full[t][h], ns[h]))) continue;
          ++ns[h];
          if (h == 0 && held < kTile) {
            // V's rows past the sequence's end may hold anything, and 0 * NaN is NaN: zeroed
            // before this tile's products (tiles arrive K, V, K, V, ..., by unit).  Only now:
            // this unit's S says that all tiles before its K have arrived, so that the wait is
            // for this V.  Before, a group that had no part in some units could be so far
            // ahead that the barrier's last phase but one looked like the one waited for.
            const int n = 2 * (unit0 + j - w.j0) + 1, slot = n % p.slots;
            if (!(ok = wait(&sh.kv_full[slot], n / p.slots))) continue;
            uint4* v = reinterpret_cast<uint4*>(kv_smem + slot * kTileBytes);
            for (int z = 0; z < kBlocks; ++z)
              for (int i = held * 8 + r; i < kTile * 8; i += kTile)
                v[z * (kPfBlock / 16) + i] = make_uint4(0, 0, 0, 0);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          if (warp_ok) {
            tc_fence_after();
            uint32_t s[64];
            tmem_ld<32>(s_addr + h * 64, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
            tmem_ld<32>(s_addr + h * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
            tmem_wait();
            const int cols = rows - j * kTile - h * 64;
            if (__any_sync(0xffffffffu, cols < 64)) {
#pragma unroll
              for (int i = 0; i < 64; ++i)
                if (i >= cols) s[i] = 0xff800000u;  // -inf
            }
            float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
            for (int i = 0; i < 64; i += 8)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                mx[c] = max3(mx[c], __uint_as_float(s[i + 2 * c]), __uint_as_float(s[i + 2 * c + 1]));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
            if (j == w.j0 && h == 0) {
              m = top;
            } else if (__any_sync(0xffffffffu, row_ok && top > m + kRescaleAbove)) {
              // (rows of no token have no say: where 128 is not a multiple of G the last ones
              // meet whatever shared memory held, and a result would depend on it)
              // this S came after the product with W of two halves ago, so only the last
              // one's can be pending (the phase waited for is the barrier's or the one before)
              if (!(ok = wait(&sh.pv_done[t], ns[0] + ns[1] - 2))) continue;
              tc_fence_after();
              const float mnew = fmaxf(m, top);
              const float f = mnew == m ? 1.f : ex2(m - mnew);
              m = mnew;
              l *= f;
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld<32>(o_addr + c * 32, o);
                tmem_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st32(o_addr + c * 32, o);
              }
            }
            const float ref = m == -CUDART_INF_F ? 0.f : m;
            const uint64_t sc2 = pk2(p.scale_log2, p.scale_log2), ref2 = pk2(-ref, -ref);
            uint64_t sum[2] = {0ull, 0ull};
            weights(s, sc2, ref2, sum);
            tmem_st32(s_addr + h * 64, s);
            l += hsum2(fadd2(sum[0], sum[1]));
            tmem_st_wait();
            tc_fence_before();
          }
          mbar_arrive(&sh.p_full[t][h]);
        }
      }
      const bool any = jend > w.j0;
      if (ok && any) {
        ok = wait(&sh.o_full[t], no++);
      }
      if (consumer_barrier_any<kTile>(1 + t, !ok)) break;
      const int64_t begin = w.item + kPfItemCost;  // the CTAs of the item's first and last unit
      const int cf = share_of(begin, ctas, total), cl = share_of(begin + w.units - 1, ctas, total);
      __nv_bfloat16* out =
          p.out + (((int64_t)w.s.c0 + first + tok_r) * p.H + (int64_t)w.g * p.G + head_r) * D;
      // this tile's part of a slot: m, l, then O as float4 [D / 4][rows]
      const auto piece = [&](int c) {
        const int slot = c == cf ? 2 * c + 1 : 2 * c;
        return p.partials + ((size_t)slot * p.piece_tiles + t) * p.piece_rows * (2 + D);
      };
      const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
      const auto load_o = [&](int c, uint32_t (&o)[32]) {  // columns c .. c + 31, by whole warps
        __syncwarp();  // lanes without a row pass over the stores of the columns before
        if (any) {
          tmem_ld<32>(o_addr + c, o);
          tmem_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0;
        }
      };
      const auto pack8 = [&](const uint32_t* o) {
        return make_uint4(bf16x2(__uint_as_float(o[0]) * inv, __uint_as_float(o[1]) * inv),
                          bf16x2(__uint_as_float(o[2]) * inv, __uint_as_float(o[3]) * inv),
                          bf16x2(__uint_as_float(o[4]) * inv, __uint_as_float(o[5]) * inv),
                          bf16x2(__uint_as_float(o[6]) * inv, __uint_as_float(o[7]) * inv));
      };
      tc_fence_after();
      // The CTA that holds an item's start comes to it last of its own work, the others
      // first of theirs: if they have all arrived it joins their pieces to its O as it is.
      bool own = false;
      if (cf != cl && (int)blockIdx.x == cf) {
        if (r == 0) sh.last[t] = ld_acquire_gpu(p.counters + 2 * cf + t) == (uint32_t)(cl - cf);
        named_barrier_sync(1 + t, kTile);
        own = sh.last[t];
      }
      if (cf == cl && ntok == TPT) {
        // a whole tile: through shared memory, 64 columns at a time, and one TMA store
        // (a thread's own row in 16-byte stores would touch 32 lines an instruction)
        uint8_t* stage = o_smem + t * kPfBlock;
#pragma unroll
        for (int z = 0; z < kBlocks; ++z) {
          if (r == 0) tma_store_read_wait();  // of the stage's last contents
          named_barrier_sync(1 + t, kTile);
#pragma unroll
          for (int c = 0; c < 64 && z * 64 + c < D; c += 32) {
            uint32_t o[32];
            load_o(z * 64 + c, o);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(stage + r * 128 + (((c / 8 + i) ^ (r & 7)) << 4)) =
                  pack8(o + 8 * i);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          named_barrier_sync(1 + t, kTile);
          if (r == 0) tma_store_out(&p.o_map, stage, z * 64, w.g, w.s.c0 + first);
        }
      } else if (warp_ok && !own) {
        float* pc = piece((int)blockIdx.x);
        if (cf != cl && row_ok) {
          pc[r] = m;
          pc[p.piece_rows + r] = l;
        }
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          load_o(c, o);
          if (row_ok && cf == cl) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) *reinterpret_cast<uint4*>(out + c + i) = pack8(o + i);
          } else if (row_ok) {
            float4* dst = reinterpret_cast<float4*>(pc + 2 * p.piece_rows);
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              dst[(c + i) / 4 * p.piece_rows + r] =
                  make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]),
                              __uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
          }
        }
      }
      if (cf != cl) {
        if (!own) {
          __threadfence();
          named_barrier_sync(1 + t, kTile);
          if (r == 0) sh.last[t] = atomicAdd(p.counters + 2 * cf + t, 1u) == (uint32_t)(cl - cf);
          named_barrier_sync(1 + t, kTile);
        }
        if (sh.last[t]) {
          __threadfence();
          if (warp_ok) {
            const int c0 = own ? cf + 1 : cf;  // the pieces in the workspace, in their order
            const auto at = [&](int c, int i) { return __ldcg(piece(c) + i * p.piece_rows + r); };
            float M = own ? m : -CUDART_INF_F, L = 0.f;
            if (row_ok) {
#pragma unroll 4
              for (int c = c0; c <= cl; ++c) M = fmaxf(M, at(c, 0));
            }
            if (M == -CUDART_INF_F) M = 0.f;
            const float f0 = exp2f(m - M);
            if (own) L = fmaf(f0, l, 0.f);  // as a piece's
            if (row_ok) {
#pragma unroll 4
              for (int c = c0; c <= cl; ++c) L = fmaf(exp2f(at(c, 0) - M), at(c, 1), L);
            }
            const float inv = L > 0.f || L != L ? 1.0f / L : 0.f;
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 32) {  // 8 loads of each of two pieces in flight
              float acc[32];
              if (own) {
                uint32_t o[32];
                load_o(d0, o);
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[i] = fmaf(f0, __uint_as_float(o[i]), 0.f);
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[i] = 0.f;
              }
              if (row_ok) {
#pragma unroll 2
                for (int c = c0; c <= cl; ++c) {
                  const float* pc = piece(c);
                  const float4* src = reinterpret_cast<const float4*>(pc + 2 * p.piece_rows) + (size_t)(d0 / 4) * p.piece_rows + r;
                  float4 v[8];
#pragma unroll
                  for (int i = 0; i < 8; ++i) v[i] = __ldcg(src + i * p.piece_rows);
                  const float f = exp2f(at(c, 0) - M);
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    acc[4 * i] = fmaf(f, v[i].x, acc[4 * i]);
                    acc[4 * i + 1] = fmaf(f, v[i].y, acc[4 * i + 1]);
                    acc[4 * i + 2] = fmaf(f, v[i].z, acc[4 * i + 2]);
                    acc[4 * i + 3] = fmaf(f, v[i].w, acc[4 * i + 3]);
                  }
                }
#pragma unroll
                for (int i = 0; i < 32; i += 8)
                  *reinterpret_cast<uint4*>(out + d0 + i) =
                      make_uint4(bf16x2(acc[i] * inv, acc[i + 1] * inv), bf16x2(acc[i + 2] * inv, acc[i + 3] * inv),
                                 bf16x2(acc[i + 4] * inv, acc[i + 5] * inv), bf16x2(acc[i + 6] * inv, acc[i + 7] * inv));
              }
            }
          }
          if (r == 0) atomicExch(p.counters + 2 * cf + t, 0u);
        }
        named_barrier_sync(1 + t, kTile);  // sh.last is written again
      }
      tc_fence_before();
    }
    if (r == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncthreads();
  if (threadIdx.x == 0 && sh.abort) {  // copies in flight land in this CTA's memory
    for (int k = max(0, sh.kv_issued - p.slots); k < sh.kv_issued; ++k)
      mbar_wait_bounded(&sh.kv_full[k % p.slots], (uint32_t)((k / p.slots) & 1), kDrainNs, nullptr);
    if (sh.q_issued)
      mbar_wait_bounded(&sh.q_full, (uint32_t)((sh.q_issued - 1) & 1), kDrainNs, nullptr);
  }
  __syncthreads();
  if (warp == kPfMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kPfTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <int D>
cudaError_t launch_prefill_d(PrefillParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  constexpr int kTileBytes = (D + 63) / 64 * kPfBlock;
  static std::mutex mu;
  static std::set<int> done;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done.count(dev.device)) {
      cudaError_t e = cudaFuncSetAttribute(attn_prefill<D>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           dev.max_smem_optin);
      if (e != cudaSuccess) return e;
      done.insert(dev.device);
    }
  }
  const size_t fixed = 1024 + kPfHeader + 2 * kTileBytes + 2 * kPfBlock;  // alignment, barriers, Q, out
  p.slots = (int)std::min<size_t>(kPfMaxSlots, (dev.max_smem_optin - fixed) / kTileBytes);
  if (p.slots < 4) return cudaErrorInvalidValue;  // a V, the next K and one of each ahead
  cudaLaunchConfig_t cfg = {};
  // no more CTAs than there can be units
  const int TPT = kTile / p.G;
  const int64_t pairs = (p.T + 2 * TPT - 1) / (2 * TPT) + std::min<int64_t>(p.B, p.T);
  const int64_t most = pairs * p.H_kv * ((p.n_max + kTile - 1) / kTile);
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(std::min(dev.sm_count, kPfMaxCtas), most));
  cfg.blockDim = dim3(kPfThreads);
  cfg.dynamicSmemBytes = fixed + (size_t)p.slots * kTileBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, attn_prefill<D>, p);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

int piece_rows_of(int64_t T, int G) {
  return (int)std::min<int64_t>(kTile, (T * G + 31) / 32 * 32);
}
int piece_tiles_of(int64_t T, int G) { return T > kTile / G ? 2 : 1; }

}  // namespace

bool prefill_shape_ok(int H, int H_kv) { return H % H_kv == 0 && H / H_kv <= kTile; }

PrefillLayout prefill_layout(int64_t T, int H, int H_kv, int D) {
  PrefillLayout z;
  const int G = H / H_kv;
  static_assert(2 * kPfMaxCtas * sizeof(uint32_t) <= kPackedCounterBytes, "counters");
  z.counters = kPackedCounters;
  z.partials = z.counters + kPackedCounterBytes;
  z.total = z.partials + (size_t)2 * kPfMaxCtas * piece_tiles_of(T, G) * piece_rows_of(T, G) * (2 + D) * sizeof(float);
  return z;
}

cudaError_t launch_attn_prefill(const void* q, int64_t q_stride, const void* k_cache,
                                const void* v_cache, const int32_t* cu_seqlens,
                                const int32_t* kv_len, int64_t T, int64_t B, int H, int H_kv, int D,
                                int64_t n_max, float scale, void* out, void* workspace,
                                const DeviceInfo& dev, cudaStream_t stream) {
  const PrefillLayout z = prefill_layout(T, H, H_kv, D);
  PrefillParams p = {};
  p.out = (__nv_bfloat16*)out;
  p.cu = cu_seqlens;
  p.kv_len = kv_len;
  p.counters = (uint32_t*)((char*)workspace + z.counters);
  p.partials = (float*)((char*)workspace + z.partials);
  p.ctl.status = (uint32_t*)workspace;
  p.ctl.wait_ns = wait_timeout_ns();
  p.ctl.drop_last = fault_injection();
  p.B = B;
  p.T = (int)T;
  p.H = H;
  p.H_kv = H_kv;
  p.G = H / H_kv;
  p.n_max = n_max;
  p.scale_log2 = scale * 1.44269504f;
  p.piece_rows = piece_rows_of(T, p.G);
  p.piece_tiles = piece_tiles_of(T, p.G);
  const uint64_t q_dims[4] = {(uint64_t)D, (uint64_t)p.G, (uint64_t)H_kv, (uint64_t)T};
  const uint64_t q_strides[3] = {(uint64_t)D * 2, (uint64_t)p.G * D * 2, (uint64_t)q_stride * 2};
  const uint32_t q_box[4] = {64, (uint32_t)p.G, 1, (uint32_t)(kTile / p.G)};
  cudaError_t e = encode_tmap_bf16(&p.q_map, q, 4, q_dims, q_strides, q_box);
  const uint64_t o_strides[3] = {q_strides[0], q_strides[1], (uint64_t)H * D * 2};
  if (e == cudaSuccess) e = encode_tmap_bf16(&p.o_map, out, 4, q_dims, o_strides, q_box);
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)n_max, (uint64_t)(B * H_kv)};
  const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)n_max * D * 2};
  const uint32_t box[3] = {64, kTile, 1};
  if (e == cudaSuccess) e = encode_tmap_bf16(&p.k_map, k_cache, 3, dims, strides, box);
  if (e == cudaSuccess) e = encode_tmap_bf16(&p.v_map, v_cache, 3, dims, strides, box);
  if (e != cudaSuccess) return e;
  switch (D) {
    case 64: return launch_prefill_d<64>(p, dev, stream);
    case 96: return launch_prefill_d<96>(p, dev, stream);
    case 128: return launch_prefill_d<128>(p, dev, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fmlp
