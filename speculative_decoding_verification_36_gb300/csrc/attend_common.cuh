// attend_common.cuh -- what the attention kernels share: which keys a row sees, how
// the work is cut into equal shares, and how the shares' results are joined.
//
// A segment is a (sequence, head of keys, tile of rows); its rows are the queries
// of the tile's tokens in the heads that share the keys, row = token * G + head.
// A segment's keys come in units of kKeys: first the codes, then the plain entries.
// All segments' units in a row are cut into as many equal shares as there are CTAs,
// whatever the sequences' lengths; where a segment falls into several shares, each
// leaves its sums (running maximum, sum, weighted values) in the workspace, and a
// second launch adds them in the order of the shares: no atomics, the same bits
// on every run.
#pragma once
#include "sv_common.cuh"
#include "sv_kernels.h"

#include <cuda_fp16.h>
#include <string.h>

namespace sv {

constexpr long long kAttendMaxKeys = (1LL << 31) - (1 << 16);  // positions and ends of units stay below 2^31

struct Sequence {
  int len, stored, n_new;  // entries before the step, of which codes; the step's tokens
  bool bad;
};

__device__ __forceinline__ Sequence attend_sequence(const KvAttendArgs& a, int b) {
  Sequence s;
  s.len = __ldg(a.lengths + b);
  s.stored = __ldg(a.stored + b);
  s.n_new = a.n_new ? __ldg(a.n_new + b) : a.T;
  const long long end = (long long)s.len + s.n_new;
  s.bad = s.len < 0 || s.n_new < 0 || s.n_new > a.T || end > (long long)a.max_pages * a.page_size || end > kAttendMaxKeys || s.stored < 0 ||
          s.stored > end || s.stored > (long long)a.max_code_pages * a.block ||
          fdiv(max(s.stored, 0), a.div_block) * a.block != s.stored;
  if (s.bad) s.len = s.stored = 0, s.n_new = a.T;
  return s;
}

// The keys [0, codes) and [stored, end) that a tile's rows may see.
struct Keys {
  int codes, stored, end;
};
template <int kRows>
__device__ __forceinline__ Keys attend_keys(const KvAttendArgs& a, const Sequence& s, int tile) {
  Keys k;
  const int t1 = min(s.n_new, fdiv((tile + 1) * kRows - 1, a.div_g) + 1);  // behind the tile's last token
  k.end = a.parents ? s.len + s.n_new : s.len + t1;
  k.codes = min(s.stored, k.end);
  k.stored = s.stored;
  return k;
}
// Units of a segment: none where the tile has no tokens, one (which reads nothing)
// for a bad sequence.
template <int kRows, int kKeys>
__device__ __forceinline__ int attend_units(const KvAttendArgs& a, const Sequence& s, int tile) {
  if (fdiv(tile * kRows, a.div_g) >= s.n_new) return 0;
  if (s.bad) return 1;
  const Keys k = attend_keys<kRows>(a, s, tile);
  return (k.codes + kKeys - 1) / kKeys + (k.end - k.codes + kKeys - 1) / kKeys;
}

// The share of one CTA, as a place among the segments and a number of units.
struct Share {
  long long all, from, left;  // units of the launch, those before the place, those of this share from there on
  int shares;                 // CTAs with a share
  int b, h, tile, u;          // the place: unit u of its segment
  Sequence s;
};

// All threads of the CTA, of which the first kThreads (a power of two) count.  s_scan:
// kThreads + 1 words of 8 bytes.
template <int kThreads, int kRows, int kKeys>
__device__ __forceinline__ Share attend_share(const KvAttendArgs& a, unsigned long long* s_scan) {
  __shared__ unsigned long long s_warp[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Share w;
  auto count = [&](int b) -> unsigned long long {
    if (b >= a.B) return 0;
    const Sequence s = attend_sequence(a, b);
    unsigned long long n = 0;
    for (int t = 0; t < a.tiles; ++t) n += attend_units<kRows, kKeys>(a, s, t);
    return n * a.Hkv;
  };
  // sums of a round of kThreads sequences: s_scan[i] before sequence i, s_scan[kThreads] of all
  auto scan = [&](int b0) {
    const bool counts = threadIdx.x < kThreads;
    const unsigned long long n = counts ? count(b0 + threadIdx.x) : 0;
    unsigned long long x = n;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    __syncthreads();
    if (counts && lane == 31) s_warp[warp] = x;
    __syncthreads();
    unsigned long long before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += s_warp[i];
      all += s_warp[i];
    }
    if (counts) s_scan[threadIdx.x] = before + x - n;
    if (threadIdx.x == 0) s_scan[kThreads] = all;
    __syncthreads();
  };
  w.all = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    scan(b0);
    w.all += s_scan[kThreads];
  }
  w.shares = (int)min((long long)gridDim.x, w.all);
  if ((int)blockIdx.x >= w.shares) {
    w.left = 0;
    return w;
  }
  w.from = (long long)((unsigned long long)blockIdx.x * w.all / w.shares);
  w.left = (long long)((unsigned long long)(blockIdx.x + 1) * w.all / w.shares) - w.from;
  unsigned long long before = 0;
  int b0 = 0;
  if (a.B > kThreads) {
    for (;; b0 += kThreads) {
      scan(b0);
      if (before + s_scan[kThreads] > (unsigned long long)w.from) break;
      before += s_scan[kThreads];
    }
  }
  int i = 0;  // the last sequence that begins at the place or before
#pragma unroll
  for (int d = kThreads / 2; d >= 1; d /= 2)
    if (before + s_scan[i + d] <= (unsigned long long)w.from) i += d;
  w.b = b0 + i;
  long long rest = w.from - (long long)(before + s_scan[i]);
  const long long head = (long long)((s_scan[i + 1] - s_scan[i]) / (unsigned)a.Hkv);  // units of each of its heads
  w.s = attend_sequence(a, w.b);
  w.h = (int)(rest / head);
  rest -= (long long)w.h * head;
  w.tile = 0;
  for (;;) {
    const int n = attend_units<kRows, kKeys>(a, w.s, w.tile);
    if (rest < n) break;
    rest -= n;
    ++w.tile;
  }
  w.u = (int)rest;
  return w;
}
// The next segment with units, once `done` of the place's have been taken.
template <int kRows, int kKeys>
__device__ __forceinline__ void attend_advance(const KvAttendArgs& a, Share& w, int done) {
  w.left -= done;
  w.from += done;
  w.u = 0;
  if (w.left <= 0) return;
  do {
    if (++w.tile == a.tiles) {
      w.tile = 0;
      if (++w.h == a.Hkv) {
        w.h = 0;
        w.s = attend_sequence(a, ++w.b);
      }
    }
  } while (attend_units<kRows, kKeys>(a, w.s, w.tile) == 0);
}
// The share that unit `u` falls into.
__device__ __forceinline__ int attend_share_of(const Share& w, long long u) {
  return (int)(((unsigned long long)(u + 1) * w.shares - 1) / (unsigned long long)w.all);
}

constexpr float kLow = -3.402823466e38f;  // a running maximum before any key
constexpr float kSlack = 4.f;  // p grows to 2^4 before the maximum moves (log2)
constexpr float kMostWeight = 32768.f;  // a weight grows to this before its unit moves

// Weights go into the second product in fp16, as p sv 2^-unit: p = 2^(x - m) of a score x under the
// running maximum m, sv the scale of the key's values.  2^unit follows the largest p sv of the row, which
// becomes 2^7 to 2^10: weights stay below 2^15 until the unit moves again, have 11 bits down to 2^-21
// of the largest and are off by 2^-32 of it below.  p below 2^-126 is 0.  (A unit of the largest sv
// alone, whatever its p, lost all weights beside one key with values 2^36 times theirs, though it
// counted for nothing.  2^9 to 2^12 has two bits more and moves more often: 31 tokens of 32
// sequences of 8192 170 us instead of 167, prompts 793 instead of 781.)
// Ancestors of a token as bits: token 0 is the root, token j + 1 node j.
__device__ __forceinline__ void attend_bits(const int* parents, int token, int words, uint32_t* bits) {
  for (int w = 0; w < words; ++w) bits[w] = 0;
  bits[0] = 1u;  // the root
  for (int node = token - 1; node >= 0; node = parents[node]) bits[(node + 1) >> 5] |= 1u << ((node + 1) & 31);
}

// The power of two that brings a magnitude (its bits) into [2^7, 2^8), and the one back.
__device__ __forceinline__ float scale_up(unsigned bits) {
  return __uint_as_float((261u - max(min(bits >> 23, 254u), 8u)) << 23);
}
__device__ __forceinline__ float scale_down(unsigned bits) {
  return __uint_as_float((max(min(bits >> 23, 254u), 8u) - 7u) << 23);
}

// 2^k, 0 below fp32's normal values, 2^127 above.
__device__ __forceinline__ float two_to(int k) { return __uint_as_float((unsigned)(max(min(k, 127), -127) + 127) << 23); }

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

// Codes to fp16.  int8: with its sign bit turned, a code is the low byte of an fp16
// between 1024 and 1279, and 1152 is taken off exactly.
template <bool kE4m3>
struct Code {
  // the four codes of a word as two pairs
  static __device__ __forceinline__ void word(uint32_t w, uint32_t& p0, uint32_t& p1) {
    if constexpr (kE4m3) {
      asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
          : "=r"(p0), "=r"(p1)
          : "r"(w));
    } else {
      const uint32_t x = w ^ 0x80808080u;
      p0 = less(__byte_perm(x, 0x64646464u, 0x4140));
      p1 = less(__byte_perm(x, 0x64646464u, 0x4342));
    }
  }
  static __device__ __forceinline__ uint32_t less(uint32_t h) {
    uint32_t y;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(h), "r"(0x64806480u));
    return y;
  }
};

__device__ __forceinline__ uint4 stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// Eight values in a row, rounded once.
template <class S>
__device__ __forceinline__ void attend_store8(S* to, const float (&f)[8]) {
  if constexpr (sizeof(S) == 4) {
    ((float4*)to)[0] = make_float4(f[0], f[1], f[2], f[3]);
    ((float4*)to)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    *(uint4*)to = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The unit of values that come together under the maximum `most`: no weighted unit, 2^(m - most + unit),
// is above it by more than a half.  (high: the largest m + unit, -infinity where there is none.)
__device__ __forceinline__ int attend_unit(float high, float most) { return (int)fminf(fmaxf(rintf(high - most), -126.f), 126.f); }
// The unit of weights under the maximum `most`, where the largest x + log_above(sv) is `high`.
__device__ __forceinline__ int attend_weight_unit(float high, float most) { return max(attend_unit(high, most) - 9, -126); }
// The exponent of the power of two above a scale; -infinity of one that is not finite: it makes its weights NaN whatever the unit.
__device__ __forceinline__ float log_above(float scale) {
  const unsigned bits = __float_as_uint(scale);
  return bits < 0x7f800000u ? (float)((int)(bits >> 23) - 126) : -INFINITY;
}

// What a share leaves of a tile: floats [rows][DP], then the rows' maxima, sums and units: the
// floats are in units of 2^unit, the sums are not.
__host__ __device__ constexpr int attend_slot(int rows, int DP) { return rows * DP + 3 * rows; }
__device__ __forceinline__ void attend_leave(float* part, int rows, int DP, int row, float m, float l, int unit) {
  part += rows * DP + row;
  part[0] = m, part[rows] = l, part[2 * rows] = __int_as_float(unit);
}

// What a share leaves for the joining: the last share of the segment that begins in it and goes
// on, and its rows.
__device__ __forceinline__ int attend_joint(int last, int rows) { return last | rows << 16; }

// All T rows of a sequence with a bad parent are NaN.  The rows below n_new[b] are the other kernel's, which
// meets the tree with them; padding is written here, and a tree without tokens is looked at here alone.
template <class S>
__device__ __forceinline__ void attend_padding(const KvAttendArgs& a) {
  const int N = a.T - 1;
  for (int b = blockIdx.y * gridDim.x + blockIdx.x; b < a.B; b += gridDim.x * gridDim.y) {
    const Sequence s = attend_sequence(a, b);
    if (s.n_new == a.T) continue;
    bool wrong = false;
    for (int j = threadIdx.x; j < N; j += blockDim.x) {
      const int p = __ldg(a.parents + (long long)b * N + j);
      wrong |= p < -1 || p >= j;
    }
    if (!__syncthreads_or(wrong)) continue;
    if (threadIdx.x == 0) atomicOr(a.status, kStatusBadData);
    const long long row = (long long)a.Hq * a.D, end = (a.T - s.n_new) * row;
    S* out = (S*)a.out + ((long long)b * a.T + s.n_new) * row;
    for (long long i = threadIdx.x; i < end; i += blockDim.x) out[i] = (S)0x7fffffffu;  // NaN in either type
  }
}

// Joins a segment that fell into several shares, in their order: CTAs x join the one that
// begins in share x and goes on.  A warp asks for the maxima, sums and values of 8 shares at once.  Either each warp
// has rows of its own or the four take a quarter of a row's shares each, whichever waits for
// memory less often (one token with 2048 entries in 32 shares: the call took 23 us where a
// warp had all of a row's shares, 17 so).
template <class S, int DP, int kRows>
__global__ void __launch_bounds__(128) attend_join_kernel(const __grid_constant__ KvAttendArgs a) {
  constexpr int kSlot = attend_slot(kRows, DP), kN = DP / 32;
  __shared__ float s_f[4][DP], s_m[4], s_l[4];
  __shared__ int s_unit[4];
  if (a.parents && a.n_new) attend_padding<S>(a);  // (beside the other kernel, which writes other rows)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 meta = a.meta[blockIdx.x];
  if (meta.x < 0) return;
  const int first = blockIdx.x, n = (meta.x & 0xffff) - first + 1, live = meta.x >> 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row0 = meta.w * kRows;
  auto slot = [&](int s) { return a.part + (2LL * (first + s) + (s == 0)) * kSlot; };
  float most, sum, f[kN];
  int unit;  // f is in units of 2^unit
  // the shares from `from` to `to` of row r
  auto take = [&](int r, int from, int to) {
    most = kLow, sum = 0.f, unit = 0;
#pragma unroll
    for (int k = 0; k < kN; ++k) f[k] = 0.f;
    for (int s = from; s < to; s += 8) {
      const int count = min(8, to - s);
      const float* p = slot(s + min(lane & 7, count - 1)) + kRows * DP + r;
      const float m = p[0], l = p[kRows];
      const int its = __float_as_int(p[2 * kRows]);
      float x[8][kN];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float* at = slot(s + min(e, count - 1)) + r * DP + kN * lane;
#pragma unroll
        for (int k = 0; k < kN; k += 2) *(float2*)&x[e][k] = *(const float2*)(at + k);
      }
      float top = fmaxf(m, most);
#pragma unroll
      for (int d = 4; d >= 1; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float by = ex2(m - top), old = ex2(most - top), part = l * by;
      float high = fmaxf(by > 0.f ? m + (float)its : -INFINITY, old > 0.f ? most + (float)unit : -INFINITY);
#pragma unroll
      for (int d = 4; d >= 1; d /= 2) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, d));
      const int to_unit = attend_unit(high, top);
      const float of = by * two_to(its - to_unit), old_of = old * two_to(unit - to_unit);
      most = top, unit = to_unit;
      sum *= old;
#pragma unroll
      for (int k = 0; k < kN; ++k) f[k] *= old_of;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= count) break;
        const float w = __shfl_sync(0xffffffffu, of, e);
        sum += __shfl_sync(0xffffffffu, part, e);
#pragma unroll
        for (int k = 0; k < kN; ++k) f[k] += x[e][k] * w;
      }
    }
  };
  auto put = [&](int r) {
    if (kN * lane >= a.D) return;
    const int half = unit / 2;
    const float by = sum == 0.f ? 0.f : 1.f / sum * two_to(half), rest = two_to(unit - half);
    const int token = fdiv(row0 + r, a.div_g);
    S* out = (S*)a.out + (((long long)meta.y * a.T + token) * a.Hq + (long long)meta.z * a.G + row0 + r - token * a.G) * a.D + kN * lane;
#pragma unroll
    for (int k = 0; k < kN; k += 2) {
      if constexpr (sizeof(S) == 4) {
        *(float2*)(out + k) = make_float2(f[k] * by * rest, f[k + 1] * by * rest);
      } else {
        uint32_t y;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(f[k + 1] * by * rest), "f"(f[k] * by * rest));
        *(uint32_t*)(out + k) = y;
      }
    }
  };
  const int alone = (live + 4 * gridDim.y - 1) / (4 * gridDim.y) * ((n + 7) / 8), together = (live + gridDim.y - 1) / gridDim.y * ((n + 31) / 32);
  if (alone <= together) {
    for (int r = blockIdx.y * 4 + warp; r < live; r += gridDim.y * 4) {
      take(r, 0, n);
      put(r);
    }
    return;
  }
  const int each = (n + 3) / 4;
  for (int r = blockIdx.y; r < live; r += gridDim.y) {
    take(r, min(n, warp * each), min(n, (warp + 1) * each));
    if (lane == 0) s_m[warp] = most, s_l[warp] = sum, s_unit[warp] = unit;
#pragma unroll
    for (int k = 0; k < kN; ++k) s_f[warp][32 * k + lane] = f[k];
    __syncthreads();
    if (warp == 0) {
      most = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
      sum = 0.f;
      float high = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if (ex2(s_m[w] - most) > 0.f) high = fmaxf(high, s_m[w] + (float)s_unit[w]);
      unit = attend_unit(high, most);
#pragma unroll
      for (int k = 0; k < kN; ++k) f[k] = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float by = ex2(s_m[w] - most), of = by * two_to(s_unit[w] - unit);
        sum += s_l[w] * by;
#pragma unroll
        for (int k = 0; k < kN; ++k) f[k] += s_f[w][32 * k + lane] * of;
      }
      put(r);
    }
    __syncthreads();
  }
}

template <class S, int DP, int kRows>
static cudaError_t launch_join(const KvAttendArgs& a, int grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3((unsigned)grid, 8);
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_join_kernel<S, DP, kRows>, a);
}

}  // namespace sv
