// Filling and reading back the KV cache of a packed batch of new tokens.
//
// rope_append: for every token of every sequence, in one pass over its q, k
// and v rows (one row = one head of D values):
//   * q and k rows, optionally: x <- x / sqrt(mean x^2 + eps) * gamma, in f32;
//   * the first R of the D values of a q or k row are rotated in pairs by the
//     angles p f_i, with p the token's position and f_i the (scaled)
//     frequency of pair i.  The angles are formed in binary64 (at p = 10^6 an
//     f32 angle is off by 0.06 rad) and their cosines and sines rounded to f32
//     once; the rotation itself is f32;
//   * q is rounded to bf16 into q_out; k and v go to row p of their head's
//     cache region, as bf16 (v a bit copy), or as int8 codes with one f32
//     scale a row: s = fl32(max |x| / 127), code = rint(x / s), taken from the
//     f32 values, so a key is rounded once.
// Bound by HBM for prompts (each row read once and written once) and by the
// latency of one launch for decode steps.
//
// Split: a CTA takes one token (or, when there are few tokens, a slice of one
// token's rows), so the R/2 sines and cosines are computed once for all heads.
// A group of 4 (D = 64) or 8 (D = 96, 128) lanes takes a row; a lane owns two
// 16-byte pieces of it that hold whole pairs in either layout (pieces u and
// u + R/16 of rotate-half rows), so rotating needs no exchange between lanes,
// and the norm and the row maximum take two or three shuffles.
//
// kv_read_q8: rows [0, kv_len) of an int8 cache as bf16 (code times scale, in
// f32, rounded once).  HBM-bound; every CTA walks 128-row tiles of all
// (sequence, head) regions, lengths taken from the device.
//
// Measured on a B200: 8192 tokens of 32 + 8 + 8 heads of 128 with norms 37 us (5.4 TB/s,
// 83% of the measured copy rate); 4235 tokens of 32 + 32 + 32 heads of 96 into an int8
// cache of 9870 rows a head, read back, 80 us (4.0 TB/s); 8 tokens 2.8 us.
#include "common.cuh"
#include "internal.h"

#include <math_constants.h>

#include <algorithm>
#include <cmath>

namespace fmlp {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendBatch = 3;  // rows of a lane group on their way at once
constexpr int kReadThreads = 256;
constexpr int kReadRows = 128;  // rows of a tile of kv_read_q8

struct AppendParams {
  const __nv_bfloat16 *q, *k, *v;  // rows of a token start at multiples of the strides
  int64_t q_stride, k_stride, v_stride;
  const __nv_bfloat16 *q_gamma, *k_gamma;  // [D] or null
  float eps;
  const int32_t* cu;      // [B + 1]
  const int32_t* kv_len;  // [B]
  int64_t B;
  int H, H_kv, R, interleaved;
  int64_t n_max;
  __nv_bfloat16* q_out;              // [T x H x D]
  __nv_bfloat16 *k_cache, *v_cache;  // [B x H_kv x n_max x D] (bf16 cache)
  int8_t *k_q, *v_q;                 // the same of an int8 cache, with
  float *k_s, *v_s;                  // [B x H_kv x n_max] scales
  uint32_t* status;
  double freq[kMaxRopePairs], amplitude;
};

// Sequence b's lengths: new tokens [c0, c1) of the batch's T (the grid's first dimension),
// len rows held with them.
struct Lengths {
  int c0, c1, len;
  __device__ __forceinline__ Lengths(const AppendParams& p, int64_t b)
      : c0(__ldg(p.cu + b)), c1(__ldg(p.cu + b + 1)), len(__ldg(p.kv_len + b)) {}
  __device__ __forceinline__ bool ok(const AppendParams& p) const {
    return c0 >= 0 && c0 <= c1 && c1 <= (int)gridDim.x && len >= 0 && len <= p.n_max;
  }
};
// The first of the 32 N sequences from b0 on that may be processed and holds token t, by one
// warp with all their lengths in one round trip: -1 if none does, with the token's position
// in `pos` if one does.
template <int N>
__device__ __forceinline__ int64_t owner(const AppendParams& p, int64_t b0, int t, int lane, int& pos) {
  bool mine[N];
  int at[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t b = b0 + i * 32 + lane;
    const Lengths s(p, min(b, p.B - 1));
    mine[i] = b < p.B && s.ok(p) && s.c0 <= t && t < s.c1;
    at[i] = mine[i] ? s.len - (s.c1 - t) : -1;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t found = __ballot_sync(0xffffffffu, mine[i]);
    if (found) {
      pos = __shfl_sync(0xffffffffu, at[i], __ffs(found) - 1);
      return b0 + i * 32 + __ffs(found) - 1;
    }
  }
  return -1;
}
// The last b with cu[b] <= t, if cu does not decrease (some b if it does).  A 32-ary search
// by one warp.
__device__ __forceinline__ int64_t sequence_of(const int32_t* cu, int64_t B, int64_t t, int lane) {
  int64_t lo = 0, hi = B;
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 31) / 32;
    const int64_t at = lo + lane * step;
    const bool le = at < hi && __ldg(cu + at) <= t;
    const int n = max(1, __popc(__ballot_sync(0xffffffffu, le)));
    lo += (int64_t)(n - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

struct Chunk {
  float x[8];
};
__device__ __forceinline__ Chunk unpack(uint4 w) {
  Chunk c;
  c.x[0] = bf16lo(w.x); c.x[1] = bf16hi(w.x); c.x[2] = bf16lo(w.y); c.x[3] = bf16hi(w.y);
  c.x[4] = bf16lo(w.z); c.x[5] = bf16hi(w.z); c.x[6] = bf16lo(w.w); c.x[7] = bf16hi(w.w);
  return c;
}
__device__ __forceinline__ uint4 pack(const Chunk& c) {
  return make_uint4(bf16x2(c.x[0], c.x[1]), bf16x2(c.x[2], c.x[3]), bf16x2(c.x[4], c.x[5]),
                    bf16x2(c.x[6], c.x[7]));
}
// rint(x / s) of 8 values as bytes (|x / s| < 127.5), ties to even, with inv = fl32(1 / s):
// adding 1.5 * 2^23 to the exact product x inv rounds it to an integer whose two's complement
// is in the low bits.  That is rint(x / s) unless the quotient stands next to a half, which
// the remainder x - code s, exact in f32, says.  (Dividing each value by the scale made the
// kernel bound by its instructions; looking twice at the rare rest costs 2%.)
__device__ __forceinline__ uint2 codes(const Chunk& c, float s, float inv) {
  constexpr float kMagic = 12582912.f;
  const float half = s > 0.f ? 0.5f * s : CUDART_INF_F;  // none for rows of zeros (or NaN)
  uint32_t t[8];
  bool near_half = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float y = fmaf(c.x[j], inv, kMagic);
    t[j] = __float_as_uint(y);
    near_half |= fabsf(fmaf(kMagic - y, s, c.x[j])) >= half;
  }
  if (near_half) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float rest = fmaf(kMagic - __uint_as_float(t[j]), s, c.x[j]), a = fabsf(rest);
      if (a > half || (a == half && (t[j] & 1u))) t[j] += rest < 0.f ? -1 : 1;
    }
  }
  const auto join = [&](int i) {
    return __byte_perm(__byte_perm(t[i], t[i + 1], 0x0040), __byte_perm(t[i + 2], t[i + 3], 0x0040), 0x5410);
  };
  return make_uint2(join(0), join(4));
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Sequence and position of token t, by one warp: position -1 for a token that is passed
// over (in no sequence, padding, or of a refused sequence), kUnplaced if the search among
// more than 32 sequences does not find one that holds it.  Then it is in none, unless cu
// decreases somewhere; a token that some of cu's entries lie before and some behind is then
// looked for in all sequences (place_anywhere).
constexpr int kUnplaced = -2;
__device__ __forceinline__ int place(const AppendParams& p, int t, int lane, int64_t& b) {
  if (p.B <= 32) {
    int pos = -1;
    b = owner<1>(p, 0, t, lane, pos);
    return max(pos, -1);
  }
  b = sequence_of(p.cu, p.B, t, lane);
  const Lengths s(p, b);
  return s.ok(p) && s.c0 <= t && t < s.c1 ? max(s.len - (s.c1 - t), -1) : kUnplaced;
}
// Which sides of t the entries first, first + step, ... of cu lie on: bit 0 if some are behind
// it or at it, bit 1 if some are before it.  If all of them lie on one side, no sequence holds
// t (the tokens of a padded batch).
__device__ __forceinline__ int sides(const AppendParams& p, int t, int64_t first, int step) {
  int found = 0;
  for (int64_t i = first; i <= p.B; i += step) found |= __ldg(p.cu + i) <= t ? 1 : 2;
  return found;
}
// Sequence and position by asking all sequences, by one warp (64 at a time: 32 and 256 made
// the rest of the kernel slower, 39.4 and 38.3 us against 37.2 for 8192 tokens).
__device__ __forceinline__ int place_anywhere(const AppendParams& p, int t, int lane, int64_t& b) {
  int pos = -1;
  b = -1;
  for (int64_t b0 = 0; b0 < p.B && b < 0; b0 += 64) b = owner<2>(p, b0, t, lane, pos);
  return max(pos, -1);
}

template <int D, bool kQ8>
__global__ void __launch_bounds__(kAppendThreads, 8) rope_append(const __grid_constant__ AppendParams p) {
  constexpr int L = D == 64 ? 4 : 8;   // lanes per row
  constexpr int kUnits = D / 16;       // of them at work (6 of 8 for D = 96)
  constexpr int kGroups = kAppendThreads / L;
  __shared__ float cs[kMaxRopePairs], sn[kMaxRopePairs];
  __shared__ int64_t s_seq;
  __shared__ int s_pos, s_sides[kAppendThreads / 32];

  grid_launch_dependents();
  grid_dependency_wait();  // every input may come from the previous kernel

  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  // this lane's two 8-value pieces of a row
  const int u = tid % L, ru = p.R / 16;
  const bool works = u < kUnits, rotates = u < ru;
  const int c0 = p.interleaved || !rotates ? 2 * u : u;
  const int c1 = p.interleaved || !rotates ? 2 * u + 1 : u + ru;

  const int rows = p.H + 2 * p.H_kv;
  const int per = (rows + gridDim.y - 1) / gridDim.y;
  const int r0 = blockIdx.y * per, r1 = min(rows, r0 + per);
  int64_t b = 0;
  int pos = -1;
  for (int base = r0; base < r1; base += kAppendBatch * kGroups) {
    // the rows of a batch, asked for before anything else
    uint4 w0[kAppendBatch], w1[kAppendBatch];
#pragma unroll
    for (int i = 0; i < kAppendBatch; ++i) {
      const int r = base + i * kGroups + tid / L;
      const __nv_bfloat16* src =
          r < p.H ? p.q + t * p.q_stride + (int64_t)r * D
                  : r < p.H + p.H_kv ? p.k + t * p.k_stride + (int64_t)(r - p.H) * D
                                     : p.v + t * p.v_stride + (int64_t)(r - p.H - p.H_kv) * D;
      w0[i] = w1[i] = make_uint4(0, 0, 0, 0);
      if (works && r < r1) {
        w0[i] = *reinterpret_cast<const uint4*>(src + 8 * c0);
        w1[i] = *reinterpret_cast<const uint4*>(src + 8 * c1);
      }
    }
    if (base == r0) {  // meanwhile: the token's place, then its cosines and sines
      constexpr int kOthers = kAppendThreads - 32;
      const bool few = p.B < 4 * kOthers;  // cu's sides looked at beside the search, not after it
      if (tid < 32) {
        const int at = place(p, (int)t, tid, b);
        if (tid == 0) {
          s_seq = b;
          s_pos = at;
        }
      } else {
        if (few && p.B > 32) {
          const int both = __reduce_or_sync(0xffffffffu, sides(p, (int)t, tid - 32, kOthers));
          if (tid % 32 == 0) s_sides[tid / 32] = both;
        }
        if (blockIdx.y == 0) {  // lengths to be reported
          for (int64_t i = (int64_t)blockIdx.x * kOthers + tid - 32; i < p.B; i += (int64_t)gridDim.x * kOthers)
            if (!Lengths(p, i).ok(p)) atomicOr(p.status, kStatusBadInput);
        }
      }
      __syncthreads();
      if (s_pos == kUnplaced) {
        if (!few) {
          const int both = __reduce_or_sync(0xffffffffu, sides(p, (int)t, tid, kAppendThreads));
          if (tid % 32 == 0) s_sides[tid / 32] = both;
          __syncthreads();
        }
        if (((few ? 0 : s_sides[0]) | s_sides[1] | s_sides[2] | s_sides[3]) != 3) return;
        __syncthreads();  // every thread has seen s_pos before it is written again
        if (tid < 32) {
          const int at = place_anywhere(p, (int)t, tid, b);
          if (tid == 0) {
            s_seq = b;
            s_pos = at;
          }
        }
        __syncthreads();
      }
      pos = s_pos;
      if (pos < 0) return;
      b = s_seq;
      for (int i = tid; i < p.R / 2; i += kAppendThreads) {
        double s, c;
        sincos((double)pos * p.freq[i], &s, &c);
        cs[i] = (float)(c * p.amplitude);
        sn[i] = (float)(s * p.amplitude);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kAppendBatch; ++i) {
      if (base + i * kGroups >= r1) break;  // uniform: the shuffles below need every lane
      const int r = base + i * kGroups + tid / L;
      const bool live = works && r < r1;
      const bool is_q = r < p.H, is_v = r >= p.H + p.H_kv;
      const int g = is_q ? r : is_v ? r - p.H - p.H_kv : r - p.H;
      Chunk x0 = unpack(w0[i]), x1 = unpack(w1[i]);
      const __nv_bfloat16* gamma = is_q ? p.q_gamma : p.k_gamma;
      if (p.q_gamma || p.k_gamma) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x0.x[j], x0.x[j], fmaf(x1.x[j], x1.x[j], ss));
        ss = group_sum<L>(ss);
        if (live && !is_v && gamma) {
          const float rinv = 1.0f / sqrtf(ss / (float)D + p.eps);
          const Chunk g0 = unpack(ld_keep(gamma + 8 * c0)), g1 = unpack(ld_keep(gamma + 8 * c1));
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x0.x[j] *= rinv * g0.x[j];
            x1.x[j] *= rinv * g1.x[j];
          }
        }
      }
      if (rotates && !is_v) {
        if (p.interleaved) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float ca = cs[8 * u + j], sa = sn[8 * u + j];
            const float cb = cs[8 * u + 4 + j], sb = sn[8 * u + 4 + j];
            const float a0 = x0.x[2 * j], a1 = x0.x[2 * j + 1], b0 = x1.x[2 * j], b1 = x1.x[2 * j + 1];
            x0.x[2 * j] = a0 * ca - a1 * sa;
            x0.x[2 * j + 1] = a0 * sa + a1 * ca;
            x1.x[2 * j] = b0 * cb - b1 * sb;
            x1.x[2 * j + 1] = b0 * sb + b1 * cb;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float c = cs[8 * u + j], s = sn[8 * u + j], a0 = x0.x[j], a1 = x1.x[j];
            x0.x[j] = a0 * c - a1 * s;
            x1.x[j] = a0 * s + a1 * c;
          }
        }
      }
      float s = 0.f, inv = 0.f;
      if (kQ8) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max_nan(m, max_nan(fabsf(x0.x[j]), fabsf(x1.x[j])));
        s = __fdiv_rn(group_max<L>(m), 127.f);
        if (!(s < CUDART_INF_F))
          s = CUDART_NAN_F;  // codes cannot hold a NaN or an infinity: the scale says so
        else if (s < 0x1p-125f)
          s = 0.f;  // its reciprocal may overflow
        else
          inv = __frcp_rn(s);
      }
      if (!live) continue;
      const int64_t row = (b * p.H_kv + g) * p.n_max + pos;  // of the cache, for k and v
      if (is_q) {
        __nv_bfloat16* dst = p.q_out + (t * p.H + g) * D;
        *reinterpret_cast<uint4*>(dst + 8 * c0) = pack(x0);
        *reinterpret_cast<uint4*>(dst + 8 * c1) = pack(x1);
      } else if (kQ8) {
        int8_t* dst = (is_v ? p.v_q : p.k_q) + row * D;
        *reinterpret_cast<uint2*>(dst + 8 * c0) = codes(x0, s, inv);
        *reinterpret_cast<uint2*>(dst + 8 * c1) = codes(x1, s, inv);
        if (u == 0) (is_v ? p.v_s : p.k_s)[row] = s;
      } else {
        __nv_bfloat16* dst = (is_v ? p.v_cache : p.k_cache) + row * D;
        *reinterpret_cast<uint4*>(dst + 8 * c0) = is_v ? w0[i] : pack(x0);
        *reinterpret_cast<uint4*>(dst + 8 * c1) = is_v ? w1[i] : pack(x1);
      }
    }
  }
}

struct ReadParams {
  const int8_t *k_q, *v_q;
  const float *k_s, *v_s;
  const int32_t* kv_len;
  __nv_bfloat16 *k_out, *v_out;
  int64_t B, n_max;
  int H_kv;
  uint32_t* status;
};

template <int D>
__global__ void __launch_bounds__(kReadThreads) kv_read_q8(const __grid_constant__ ReadParams p) {
  constexpr int kPieces = kReadRows * (D / 16);  // 16-byte pieces of a tile of K (or V)
  constexpr int kPer = (kPieces + kReadThreads - 1) / kReadThreads;
  __shared__ int len[kReadThreads];
  grid_launch_dependents();
  grid_dependency_wait();

  int64_t w = blockIdx.x, base = 0;  // next tile of this CTA; tiles of the sequences before
  for (int64_t b0 = 0; b0 < p.B; b0 += kReadThreads) {
    __syncthreads();
    if (b0 + threadIdx.x < p.B) {
      int64_t n = __ldg(p.kv_len + b0 + threadIdx.x);
      if (n < 0 || n > p.n_max) {  // refused: the sequence's rows stay as they were
        if (blockIdx.x == 0) atomicOr(p.status, kStatusBadInput);
        n = 0;
      }
      len[threadIdx.x] = (int)n;
    }
    __syncthreads();
    const int nb = (int)min((int64_t)kReadThreads, p.B - b0);
    for (int i = 0; i < nb; ++i) {
      const int n = len[i], per_head = (n + kReadRows - 1) / kReadRows;
      const int64_t tiles = (int64_t)per_head * p.H_kv;
      for (; w < base + tiles; w += gridDim.x) {
        const uint32_t at = (uint32_t)(w - base);  // a cache of 2^32 tiles is past any memory
        const int64_t seg = (b0 + i) * p.H_kv + at / (uint32_t)per_head;
        const int row0 = (int)(at % (uint32_t)per_head) * kReadRows;
        const int64_t r0 = seg * p.n_max + row0;
        const int pieces = min(kReadRows, n - row0) * (D / 16);
        uint4 kw[kPer], vw[kPer];
        float ks[kPer], vs[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int e = threadIdx.x + j * kReadThreads;
          if (e >= pieces) continue;
          kw[j] = reinterpret_cast<const uint4*>(p.k_q + r0 * D)[e];
          vw[j] = reinterpret_cast<const uint4*>(p.v_q + r0 * D)[e];
          ks[j] = p.k_s[r0 + e / (D / 16)];
          vs[j] = p.v_s[r0 + e / (D / 16)];
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int e = threadIdx.x + j * kReadThreads;
          if (e >= pieces) continue;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint4 w4 = kv ? vw[j] : kw[j];
            const float s = kv ? vs[j] : ks[j];
            const uint32_t in[4] = {w4.x, w4.y, w4.z, w4.w};
            uint32_t o[8];
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
              // byte b + 128 as the low byte of 2^23, less 2^23 + 128: exact
              const uint32_t c = in[i4] ^ 0x80808080u;
              const float f0 = __uint_as_float(__byte_perm(c, 0x4B000000u, 0x7440)) - 8388736.f;
              const float f1 = __uint_as_float(__byte_perm(c, 0x4B000000u, 0x7441)) - 8388736.f;
              const float f2 = __uint_as_float(__byte_perm(c, 0x4B000000u, 0x7442)) - 8388736.f;
              const float f3 = __uint_as_float(__byte_perm(c, 0x4B000000u, 0x7443)) - 8388736.f;
              o[2 * i4] = bf16x2(f0 * s, f1 * s);
              o[2 * i4 + 1] = bf16x2(f2 * s, f3 * s);
            }
            uint4* dst = reinterpret_cast<uint4*>((kv ? p.v_out : p.k_out) + r0 * D) + 2 * e;
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
      }
      base += tiles;
    }
  }
}

template <typename Kernel, typename Params>
cudaError_t launch(Kernel kern, dim3 grid, int threads, const Params& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

template <int D>
cudaError_t launch_append_d(const AppendParams& p, bool q8, dim3 grid, cudaStream_t stream) {
  return q8 ? launch(rope_append<D, true>, grid, kAppendThreads, p, stream)
            : launch(rope_append<D, false>, grid, kAppendThreads, p, stream);
}

}  // namespace

// Frequencies of the R/2 pairs, scaled for long contexts (fmlp.h).
bool rope_frequencies(const fmlp_rope& r, int D, double* freq) {
  const int R = r.rotary_dim;
  if (R < 0 || R > D || R % 16 != 0) return false;
  if (R == 0) return true;
  if (!std::isfinite(r.theta) || !(r.theta > 0) || !std::isfinite(r.amplitude)) return false;
  if (r.scaling < FMLP_ROPE_PLAIN || r.scaling > FMLP_ROPE_YARN) return false;
  if (r.scaling != FMLP_ROPE_PLAIN && !(std::isfinite(r.factor) && r.factor > 0)) return false;
  if (r.scaling == FMLP_ROPE_BANDS || r.scaling == FMLP_ROPE_YARN) {
    if (!std::isfinite(r.low) || !std::isfinite(r.high) || !(r.low > 0) || !(r.high > r.low) ||
        r.original_ctx < 1)
      return false;
  }
  if (r.scaling == FMLP_ROPE_YARN && !(r.theta > 1)) return false;  // its log divides
  const double two_pi = 6.283185307179586476925;
  double lo = 0, hi = 0;
  if (r.scaling == FMLP_ROPE_YARN) {
    const auto pair_of = [&](double turns) {
      return R * std::log((double)r.original_ctx / (two_pi * turns)) / (2 * std::log(r.theta));
    };
    lo = std::max(std::floor(pair_of(r.high)), 0.0);
    hi = std::min(std::ceil(pair_of(r.low)), (double)(R - 1));
  }
  for (int i = 0; i < R / 2; ++i) {
    double f = std::pow(r.theta, -2.0 * i / R);
    double interpolated = 0;  // share of the frequency that is divided by the factor
    if (r.scaling == FMLP_ROPE_LINEAR) interpolated = 1;
    if (r.scaling == FMLP_ROPE_BANDS) {
      const double turns = (double)r.original_ctx * f / two_pi;  // over the original context
      interpolated = 1 - std::min(1.0, std::max(0.0, (turns - r.low) / (r.high - r.low)));
    }
    if (r.scaling == FMLP_ROPE_YARN)
      interpolated = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 1e-3)));
    freq[i] = r.scaling == FMLP_ROPE_PLAIN ? f : interpolated * (f / r.factor) + (1 - interpolated) * f;
  }
  return true;
}

cudaError_t launch_rope_append(const AppendArgs& a, const double* freq, const DeviceInfo& dev,
                               cudaStream_t stream) {
  AppendParams p = {};
  p.q = (const __nv_bfloat16*)a.q;
  p.k = (const __nv_bfloat16*)a.k;
  p.v = (const __nv_bfloat16*)a.v;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.q_gamma = (const __nv_bfloat16*)a.q_gamma;
  p.k_gamma = (const __nv_bfloat16*)a.k_gamma;
  p.eps = a.eps;
  p.cu = a.cu_seqlens;
  p.kv_len = a.kv_len;
  p.B = a.B;
  p.H = a.H;
  p.H_kv = a.H_kv;
  p.R = a.rope.rotary_dim;
  p.interleaved = a.rope.interleaved != 0;
  p.n_max = a.n_max;
  p.q_out = (__nv_bfloat16*)a.q_out;
  const bool q8 = a.k_s != nullptr;
  if (q8) {
    p.k_q = (int8_t*)a.k_cache;
    p.v_q = (int8_t*)a.v_cache;
    p.k_s = a.k_s;
    p.v_s = a.v_s;
  } else {
    p.k_cache = (__nv_bfloat16*)a.k_cache;
    p.v_cache = (__nv_bfloat16*)a.v_cache;
  }
  p.status = (uint32_t*)a.workspace;
  for (int i = 0; i < p.R / 2; ++i) p.freq[i] = freq[i];
  p.amplitude = a.rope.amplitude;
  // Few tokens: a token's rows are sliced over CTAs (whole passes of the row
  // groups) until the grid covers the SMs; the table is then computed per slice.
  const int groups = kAppendThreads / (a.D == 64 ? 4 : 8);
  const int passes = (a.H + 2 * a.H_kv + groups - 1) / groups;
  const int64_t slices = std::min<int64_t>(passes, std::max<int64_t>(1, dev.sm_count / a.T));
  const dim3 grid((unsigned)a.T, (unsigned)slices);
  switch (a.D) {
    case 64: return launch_append_d<64>(p, q8, grid, stream);
    case 96: return launch_append_d<96>(p, q8, grid, stream);
    case 128: return launch_append_d<128>(p, q8, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_kv_read_q8(const void* k_q, const float* k_s, const void* v_q, const float* v_s,
                              const int32_t* kv_len, int64_t B, int H_kv, int D, int64_t n_max,
                              void* k_cache, void* v_cache, void* workspace, const DeviceInfo& dev,
                              cudaStream_t stream) {
  ReadParams p = {};
  p.k_q = (const int8_t*)k_q;
  p.v_q = (const int8_t*)v_q;
  p.k_s = k_s;
  p.v_s = v_s;
  p.kv_len = kv_len;
  p.k_out = (__nv_bfloat16*)k_cache;
  p.v_out = (__nv_bfloat16*)v_cache;
  p.B = B;
  p.n_max = n_max;
  p.H_kv = H_kv;
  p.status = (uint32_t*)workspace;
  const int64_t most = B * H_kv * ((n_max + kReadRows - 1) / kReadRows);
  const dim3 grid((unsigned)std::min<int64_t>(most, (int64_t)dev.sm_count * 8));
  switch (D) {
    case 64: return launch(kv_read_q8<64>, grid, kReadThreads, p, stream);
    case 96: return launch(kv_read_q8<96>, grid, kReadThreads, p, stream);
    case 128: return launch(kv_read_q8<128>, grid, kReadThreads, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fmlp
