// attend_rows.cuh -- attention of a step's tokens to a cache whose older blocks are
// 8-bit codes: few rows a head of keys, by warps that feed mma.sync from registers.
//
//   out = softmax(scale q K^T) V over the keys that a token sees.
//
// Codes are exact in fp16, so q K^T and P V are fp16 products with fp32 sums: a code's
// scale multiplies the score or the weight, never the code.  Queries come as fp16
// times a power of two for each row (bf16 queries exactly, fp32 ones as a sum of two
// fp16 parts), weights as fp16 (fp32: two parts) times a power of two that follows the
// values' scales.  Plain entries become fp16 (two parts) times a power of two for each
// key.  The softmax runs in the log2 domain with one pass over the keys.
#pragma once
#include "attend_common.cuh"


namespace sv {

constexpr int kARThreads = 128;
constexpr int kARWarps = kARThreads / 32;
constexpr int kARKeys = 16 * kARWarps;  // keys of a unit: 16 to a warp

__device__ __forceinline__ void mma16816(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float2 floats_of(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
// What is left of two values behind their fp16 parts `w`.
__device__ __forceinline__ uint32_t rest_of(float lo, float hi, uint32_t w) {
  const float2 f = floats_of(w);
  return half2_of(lo - f.x, hi - f.y);
}

// A lane's place in the products (g = lane / 4, t = lane % 4).  The order in which a
// product runs over its inner index is free, so a lane's operands are bytes that lie
// together in memory and go from global memory to registers without a shuffle:
//   q K^T, chunk c of 64 values: the lane's 16 codes of key g at 64 c + 16 t feed
//     four steps of 16 (step 4 c + s: its codes 4 s .. 4 s + 3);
//   P V: the lane's DP / 8 codes of its keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9 at g DP / 8
//     are the columns n = g of the DP / 8 products, so that a row's sums of product j
//     are the values 2 t DP / 8 + j and (2 t + 1) DP / 8 + j: DP / 4 in a row.
template <class S, bool kE4m3, int DP, int MT>
struct Rows {
  static constexpr bool kTwo = sizeof(S) == 4;  // two fp16 parts
  static constexpr int kSteps = DP / 16, kChunks = DP / 64, NT = DP / 8, kParts = kTwo ? 2 : 1;
  static constexpr int kFrag = kSteps * 32;                  // uint4's of one row tile's queries
  // A warp's ring: 16 keys' codes, their values' and both scales a stage.
  static constexpr int kStages = DP < 256 ? 4 : kTwo ? 2 : 3, kStage = 2 * 16 * DP + 2 * 16 * 4;
  static_assert(MT * NT * 4 * 32 * 4 <= kARWarps * kStages * kStage, "the warps' sums go over the rings");
  // Where 16 bytes (unit u) of a row lie: both products' reads fall on all banks.
  static __device__ __forceinline__ int at(int row, int u) {
    const int turn = DP == 64 ? (row & 2) : ((row ^ (row >> 2)) & 1) << 2 | (row & 2);
    return row * DP + ((u ^ turn) << 4);
  }
  static constexpr size_t smem(int T, bool tree) {
    return (size_t)MT * kParts * kFrag * 16 + (size_t)kARWarps * kStages * kStage + 2 * kARWarps * 16 * MT * 4 + 16 * MT * 4 +
           (tree ? (size_t)T * 4 + (size_t)16 * MT * ((T + 31) / 32) * 4 : 0);
  }
};

// 16 bytes (zeros where !in) or 4 from global to shared memory, asynchronously.
__device__ __forceinline__ void copy16(void* to, const void* from, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(void* to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}

template <class S>
__device__ __forceinline__ float value_of(S x);
template <>
__device__ __forceinline__ float value_of<uint32_t>(uint32_t x) { return __uint_as_float(x); }
template <>
__device__ __forceinline__ float value_of<uint16_t>(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

// N values from memory (N * sizeof(S) a multiple of 16 bytes), in fp32.
template <class S, int N>
__device__ __forceinline__ void plain_values(const S* p, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N * (int)sizeof(S) / 16; ++i) {
    const uint4 v = ((const uint4*)p)[i];
    if constexpr (sizeof(S) == 4) {
      f[4 * i] = __uint_as_float(v.x), f[4 * i + 1] = __uint_as_float(v.y), f[4 * i + 2] = __uint_as_float(v.z),
                                  f[4 * i + 3] = __uint_as_float(v.w);
    } else {
      f[8 * i] = bf16_lo(v.x), f[8 * i + 1] = bf16_hi(v.x), f[8 * i + 2] = bf16_lo(v.y), f[8 * i + 3] = bf16_hi(v.y);
      f[8 * i + 4] = bf16_lo(v.z), f[8 * i + 5] = bf16_hi(v.z), f[8 * i + 6] = bf16_lo(v.w), f[8 * i + 7] = bf16_hi(v.w);
    }
  }
}
template <class S>
__device__ __forceinline__ void four_values(const S* p, float (&f)[4]) {
  if constexpr (sizeof(S) == 4) {
    const uint4 v = *(const uint4*)p;
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  } else {
    const uint2 v = *(const uint2*)p;
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
  }
}
template <int N>
__device__ __forceinline__ unsigned top_bits(const float (&f)[N]) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  return m;
}

template <class S, bool kE4m3, int DP, int MT, int kCtas>
__global__ void __launch_bounds__(kARThreads, kCtas) attend_rows_kernel(const __grid_constant__ KvAttendArgs a) {
  using R = Rows<S, kE4m3, DP, MT>;
  constexpr int NT = R::NT, kChunks = R::kChunks, kRows = 16 * MT;
  constexpr bool kTwo = R::kTwo;
  constexpr int VW = DP / 32;               // words of V's codes per key and lane
  extern __shared__ __align__(16) unsigned char s_attend[];
  uint4* s_q = (uint4*)s_attend;                                   // [MT][parts][steps][32]
  unsigned char* s_ring = (unsigned char*)(s_q + MT * R::kParts * R::kFrag);  // the warps' rings, then
  float* s_acc = (float*)s_ring;                                              // [MT][NT][4][32]
  float* s_m = (float*)(s_ring + kARWarps * R::kStages * R::kStage);          // [warps][rows], then sums
  float* s_l = s_m + kARWarps * kRows;
  float* s_qs = s_l + kARWarps * kRows;                            // [rows]
  int* s_par = (int*)(s_qs + kRows);                               // [T]
  uint32_t* s_bits = (uint32_t*)(s_par + a.T);                     // [rows][words]
  __shared__ unsigned long long s_scan[kARThreads + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int words = (a.T + 31) / 32;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  Share w = attend_share<kARThreads, kRows, kARKeys>(a, s_scan);
  int meta_last = -1, meta_b = 0, meta_h = 0, meta_tile = 0;
  int loaded_b = -1, loaded_tile = -1;
  bool bad = false;
  while (w.left > 0) {
    const int n = attend_units<kRows, kARKeys>(a, w.s, w.tile);
    const int u0 = w.u, u1 = (int)min((long long)n, u0 + w.left);
    const Keys keys = attend_keys<kRows>(a, w.s, w.tile);
    const int row0 = w.tile * kRows, rows = w.s.n_new * a.G;

    // ---- the tile's queries, and a tree's ancestors ----
    __syncthreads();
    if (a.parents && (w.b != loaded_b || w.tile != loaded_tile)) {
      const int N = a.T - 1;
      bool wrong = false;
      for (int j = threadIdx.x; j < N; j += kARThreads) {
        const int p = __ldg(a.parents + (long long)w.b * N + j);
        s_par[j] = p;
        wrong |= p < -1 || p >= j;
      }
      bad = __syncthreads_or(wrong);
      if (!bad)
        for (int r = threadIdx.x; r < kRows; r += kARThreads) {
          const int token = fdiv(row0 + r, a.div_g);
          if (token < a.T) attend_bits(s_par, token, words, s_bits + r * words);
        }
    }
    const bool lost = w.s.bad || (a.parents && bad);
    if (lost && threadIdx.x == 0) atomicOr(a.status, kStatusBadData);
    loaded_b = w.b, loaded_tile = w.tile;
    for (int r = warp; r < kRows; r += kARWarps) {
      const int token = fdiv(row0 + r, a.div_g);
      const bool live = row0 + r < rows && !lost;
      const S* q = (const S*)a.q + ((long long)w.b * a.T + token) * a.q_stride + ((long long)w.h * a.G + row0 + r - token * a.G) * a.D;
      float x[DP / 32];
      unsigned top = 0;
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) {
        const int d = lane + 32 * i;
        x[i] = live && d < a.D ? value_of<S>(q[d]) : 0.f;
        top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
      }
      top = __reduce_max_sync(0xffffffffu, top);
      const bool finite = top < 0x7f800000u;
      const float up = scale_up(top);
      if (lane == 0) s_qs[r] = lost || !finite ? __uint_as_float(0x7fffffffu) : scale_down(top) * a.scale;
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) {
        const int d = lane + 32 * i;
        // value d: chunk d / 64, lane t = d % 64 / 16, step d % 16 / 4, register pair by d % 4 / 2
        const int step = 4 * (d >> 6) + ((d & 15) >> 2), at = (r & 7) * 4 + ((d & 63) >> 4), reg = ((r >> 3) & 1) + 2 * ((d & 3) >> 1);
        const float y = finite ? x[i] * up : 0.f;
        const __half hi = __float2half_rn(y);
        __half* to = (__half*)(s_q + ((r >> 4) * R::kParts * R::kSteps + step) * 32 + at) + reg * 2 + (d & 1);
        *to = hi;
        if (kTwo) to[R::kFrag * 8] = __float2half_rn(y - __half2float(hi));
      }
    }
    __syncthreads();

    // ---- the lane's rows ----
    float qs[MT][2], m[MT][2], l[MT][2];
    int seen[MT][2];  // a chain's last key
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 16 * i + 8 * e + g;
        qs[i][e] = s_qs[r];
        m[i][e] = kLow;
        l[i][e] = 0.f;
        seen[i][e] = w.s.len + fdiv(row0 + r, a.div_g);
      }
    const int first_seen = w.s.len + fdiv(row0, a.div_g);
    float o[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
    unsigned ref[MT][2];  // exponent bits above every scale of V that the row has seen
#pragma unroll
    for (int i = 0; i < MT; ++i) ref[i][0] = ref[i][1] = 11u;

    auto visible = [&](int i, int e, int key, int end) {
      if (key >= end) return false;
      if (!a.parents) return key <= seen[i][e];
      const int at = key - w.s.len;
      return at < 0 || (lost ? false : ((s_bits[(16 * i + 8 * e + g) * words + (at >> 5)] >> (at & 31)) & 1u) != 0);
    };

    // Scores of 16 keys to weights; the lane's keys are base + 2 t + {0, 1, 8, 9}.
    // sk, sv: their scales.  wt: the weights as products' left sides.
    auto weights = [&](float (&c)[MT][2][4], const float (&sk)[4], const float (&sv)[4], int base, int end, bool masked,
                       uint4 (&wt)[MT][R::kParts]) {
      float x[MT][2][4];
      unsigned top[4], all = 11u;  // exponents above the keys' scales of V; a scale that is not finite makes its weights NaN whatever the reference
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        top[k] = __float_as_uint(sv[k]) < 0x7f800000u ? max((__float_as_uint(sv[k]) >> 23) + 1u, 11u) : 11u;
        all = max(all, top[k]);
      }
      bool grow = false;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          unsigned mine = masked ? 11u : all;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[i][e][k] = c[i][k >> 1][2 * e + (k & 1)] * sk[k] * qs[i][e];
            if (masked) {
              if (visible(i, e, base + 2 * t + (k & 1) + 8 * (k >> 1), end))
                mine = max(mine, top[k]);
              else
                x[i][e][k] = -INFINITY;
            }
            grow |= x[i][e][k] > m[i][e] + kSlack;
          }
          grow |= mine > ref[i][e];
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = fmaxf(fmaxf(x[i][e][0], x[i][e][1]), fmaxf(x[i][e][2], x[i][e][3]));
            unsigned to = ref[i][e];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (!masked || x[i][e][k] != -INFINITY) to = max(to, top[k]);
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
            y = fmaxf(y, m[i][e]);
            to = max(to, __shfl_xor_sync(0xffffffffu, to, 1));
            to = max(to, __shfl_xor_sync(0xffffffffu, to, 2));
            const float f = ex2(m[i][e] - y), both = f * ex2((float)((int)ref[i][e] - (int)to));
            m[i][e] = y;
            ref[i][e] = to;
            l[i][e] *= f;
#pragma unroll
            for (int j = 0; j < NT; ++j) o[i][j][2 * e] *= both, o[i][j][2 * e + 1] *= both;
          }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        float y[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // 2^11 over the reference: weights stay below 2^15 and keep fp16's full precision 2^25 below it
          const float over = __uint_as_float((265u - ref[i][e]) << 23);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float p = ex2(x[i][e][k] - m[i][e]);
            l[i][e] += p;
            y[e][k] = masked && x[i][e][k] == -INFINITY ? 0.f : p * (sv[k] * over);
          }
        }
        wt[i][0] = make_uint4(half2_of(y[0][0], y[0][1]), half2_of(y[1][0], y[1][1]), half2_of(y[0][2], y[0][3]), half2_of(y[1][2], y[1][3]));
        if constexpr (kTwo)
          wt[i][1] = make_uint4(rest_of(y[0][0], y[0][1], wt[i][0].x), rest_of(y[1][0], y[1][1], wt[i][0].y),
                                rest_of(y[0][2], y[0][3], wt[i][0].z), rest_of(y[1][2], y[1][3], wt[i][0].w));
      }
    };
    auto query = [&](int i, int part, int step) { return s_q[((i * R::kParts + part) * R::kSteps + step) * 32 + lane]; };

    // ---- codes ----
    const int n_codes = w.s.bad ? 0 : (keys.codes + kARKeys - 1) / kARKeys;
    const int uc = min(u1, n_codes);
    if (u0 < uc) {
      const int32_t* table = a.code_table + (long long)w.b * a.max_code_pages;
      const uint8_t* kc = a.k_codes + (long long)w.h * a.D;
      const uint8_t* vc = a.v_codes + (long long)w.h * a.D;
      const long long entry = (long long)a.Hkv * a.D;
      // lane x looks up key x % 16 of the warp's tile
      int page, within;
      auto look = [&](int u) {
        const int key = min(u * kARKeys + 16 * warp + (lane & 15), keys.codes - 1), block = fdiv(key, a.div_block);
        within = key - block * a.block;
        page = __ldg(table + block);
      };
      unsigned char* ring = s_ring + warp * R::kStages * R::kStage;
      // Keys, values and scales of the tile that was looked up go to a stage of the warp's ring.
      auto fetch = [&](int stage, bool some) {
        if (some) {
          const bool on = page >= 0 && page < a.code_pages;
          const int e = on ? page * a.block + within : 0;
          unsigned char* to = ring + stage * R::kStage;
          float* scales = (float*)(to + 2 * 16 * DP);
          if (on) {
            copy4(scales + lane, (lane < 16 ? a.k_scales : a.v_scales) + (long long)page * a.Hkv + w.h);
          } else {
            scales[lane] = __uint_as_float(0x7fffffffu);
            atomicOr(a.status, kStatusBadData);
          }
#pragma unroll
          for (int j = 0; j < DP / 32; ++j) {
            const int x = lane + 32 * j, row = x / (DP / 16), u = x % (DP / 16);
            const long long from = __shfl_sync(0xffffffffu, e, row) * entry + 16 * u;
            const bool in = 16 * u < a.D;  // (zeros behind the head)
            copy16(to + R::at(row, u), kc + (in ? from : 0), in);
            copy16(to + 16 * DP + R::at(row, u), vc + (in ? from : 0), in);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      constexpr int kAhead = R::kStages - 1;
      look(u0);
      for (int j = 0; j < kAhead; ++j) {
        fetch(j, u0 + j < uc);
        if (u0 + j + 1 < uc) look(u0 + j + 1);
      }
      int stage = 0;
      for (int u = u0; u < uc; ++u) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        __syncwarp();  // the tile is there, and all lanes are done with the last one
        fetch(stage ? stage - 1 : kAhead, u + kAhead < uc);
        if (u + kAhead + 1 < uc) look(u + kAhead + 1);
        const unsigned char* from = ring + stage * R::kStage;
        const float* scales = (const float*)(from + 2 * 16 * DP);
        if (++stage == R::kStages) stage = 0;
        float c[MT][2][4] = {};
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch) {
          const uint4 k0 = *(const uint4*)(from + R::at(g, 4 * ch + t)), k1 = *(const uint4*)(from + R::at(g + 8, 4 * ch + t));
          const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint32_t b0, b1, b2, b3;
            Code<kE4m3>::word(w0[s], b0, b1);
            Code<kE4m3>::word(w1[s], b2, b3);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int part = 0; part < R::kParts; ++part) {
                const uint4 q = query(i, part, 4 * ch + s);
                mma16816(c[i][0], q, b0, b1);
                mma16816(c[i][1], q, b2, b3);
              }
          }
        }
        float sk[4], sv[4];
        *(float2*)sk = *(const float2*)(scales + 2 * t), *(float2*)(sk + 2) = *(const float2*)(scales + 2 * t + 8);
        *(float2*)sv = *(const float2*)(scales + 16 + 2 * t), *(float2*)(sv + 2) = *(const float2*)(scales + 24 + 2 * t);
        const int base = u * kARKeys + 16 * warp;
        uint4 wt[MT][R::kParts];
        weights(c, sk, sv, base, keys.codes, base + 16 > keys.codes || (a.parents ? base + 16 > w.s.len : base + 15 > first_seen), wt);
        const unsigned char* values = from + 16 * DP;
        constexpr int kWords = VW < 4 ? VW : 4;  // of a place, 16 bytes at most at a time
#pragma unroll
        for (int x0 = 0; x0 < VW; x0 += kWords) {
          uint32_t v[4][kWords];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = 2 * t + (k & 1) + 8 * (k >> 1), byte = g * (DP / 8) + 4 * x0;
            if constexpr (kWords == 2) {
              const uint2 y = *(const uint2*)(values + R::at(row, byte >> 4) + (byte & 15));
              v[k][0] = y.x, v[k][1] = y.y;
            } else {
              const uint4 y = *(const uint4*)(values + R::at(row, byte >> 4));
              v[k][0] = y.x, v[k][1] = y.y, v[k][2] = y.z, v[k][3] = y.w;
            }
          }
#pragma unroll
          for (int x = 0; x < kWords; ++x) {
            // codes of one place in the head, of the keys 2 t and 2 t + 1, side by side
            const uint32_t lo0 = __byte_perm(v[0][x], v[1][x], 0x5140), hi0 = __byte_perm(v[0][x], v[1][x], 0x7362);
            const uint32_t lo1 = __byte_perm(v[2][x], v[3][x], 0x5140), hi1 = __byte_perm(v[2][x], v[3][x], 0x7362);
            uint32_t b0[4], b1[4];
            Code<kE4m3>::word(lo0, b0[0], b0[1]);
            Code<kE4m3>::word(hi0, b0[2], b0[3]);
            Code<kE4m3>::word(lo1, b1[0], b1[1]);
            Code<kE4m3>::word(hi1, b1[2], b1[3]);
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
              for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int part = 0; part < R::kParts; ++part) mma16816(o[i][4 * (x0 + x) + y], wt[i][part], b0[y], b1[y]);
          }
        }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }

    // ---- plain entries ----
    for (int u = max(u0, n_codes); u < u1 && !w.s.bad; ++u) {
      const int base = keys.stored + (u - n_codes) * kARKeys + 16 * warp;
      if (base >= keys.end) continue;
      const int key = min(base + (lane & 15), keys.end - 1), p = fdiv(key, a.div_page);
      const int page = __ldg(a.page_table + (long long)w.b * a.max_pages + p);
      const bool on = page >= 0 && page < a.pages;
      if (!on) atomicOr(a.status, kStatusBadData);
      const int e = on ? page * a.page_size + (key - p * a.page_size) : -1;
      const S* kc = (const S*)a.k_cache + (long long)w.h * a.D;
      const S* vc = (const S*)a.v_cache + (long long)w.h * a.D;
      const long long entry = (long long)a.Hkv * a.D;
      float c[MT][2][4] = {};
      float sk_own[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // key g + 8 k: its largest magnitude first, then its parts
        const int at = __shfl_sync(0xffffffffu, e, g + 8 * k);
        const S* from = kc + (long long)max(at, 0) * entry + 16 * t;
        unsigned top = 0;
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch)
          if (64 * ch + 16 * t < a.D) {
            float f[16];
            plain_values<S, 16>(from + 64 * ch, f);
            top = max(top, top_bits(f));
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const bool finite = top < 0x7f800000u;
        sk_own[k] = at < 0 || !finite ? __uint_as_float(0x7fffffffu) : scale_down(top);
        const float up = scale_up(top);
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch) {
          float f[16] = {};
          if (64 * ch + 16 * t < a.D && finite) plain_values<S, 16>(from + 64 * ch, f);
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const float y0 = f[4 * s] * up, y1 = f[4 * s + 1] * up, y2 = f[4 * s + 2] * up, y3 = f[4 * s + 3] * up;
            const uint32_t b0 = half2_of(y0, y1), b1 = half2_of(y2, y3);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int part = 0; part < R::kParts; ++part) mma16816(c[i][k], query(i, part, 4 * ch + s), b0, b1);
            if constexpr (kTwo) {
              const uint32_t r0 = rest_of(y0, y1, b0), r1 = rest_of(y2, y3, b1);
#pragma unroll
              for (int i = 0; i < MT; ++i) mma16816(c[i][k], query(i, 0, 4 * ch + s), r0, r1);
            }
          }
        }
      }
      // V: the lane's four keys
      float sk[4], sv[4], up[4];
      const S* from[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int x = 2 * t + (k & 1);
        sk[k] = __shfl_sync(0xffffffffu, sk_own[k >> 1], 4 * x);
        const int at = __shfl_sync(0xffffffffu, e, x + 8 * (k >> 1));
        from[k] = vc + (long long)max(at, 0) * entry + g * (DP / 8);
        unsigned top = 0;
#pragma unroll
        for (int i = 0; i < DP / 64; ++i)
          if (g * (DP / 8) + 8 * i < a.D) {
            float f[8];
            plain_values<S, 8>(from[k] + 8 * i, f);
            top = max(top, top_bits(f));
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 4));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const bool finite = top < 0x7f800000u;
        sv[k] = at < 0 || !finite ? __uint_as_float(0x7fffffffu) : scale_down(top);
        up[k] = finite ? scale_up(top) : 0.f;
      }
      uint4 wt[MT][R::kParts];
      weights(c, sk, sv, base, keys.end, true, wt);
#pragma unroll
      for (int x = 0; x < NT / 4; ++x) {  // four values at a time: registers are scarce
        float f[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f[k][0] = f[k][1] = f[k][2] = f[k][3] = 0.f;
          if (g * (DP / 8) + 4 * x < a.D && up[k] > 0.f) four_values<S>(from[k] + 4 * x, f[k]);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float y0 = f[0][y] * up[0], y1 = f[1][y] * up[1], y2 = f[2][y] * up[2], y3 = f[3][y] * up[3];
          const uint32_t b0 = half2_of(y0, y1), b1 = half2_of(y2, y3);
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int part = 0; part < R::kParts; ++part) mma16816(o[i][4 * x + y], wt[i][part], b0, b1);
          if constexpr (kTwo) {
            const uint32_t r0 = rest_of(y0, y1, b0), r1 = rest_of(y2, y3, b1);
#pragma unroll
            for (int i = 0; i < MT; ++i) mma16816(o[i][4 * x + y], wt[i][0], r0, r1);
          }
        }
        asm volatile("" ::: "memory");
      }
    }

    // ---- the warps' sums become one ----
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], 1);
        l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], 2);
        if (lost) l[i][e] = __uint_as_float(0x7fffffffu);
        if (t == 0) s_m[warp * kRows + 16 * i + 8 * e + g] = m[i][e], s_l[warp * kRows + 16 * i + 8 * e + g] = l[i][e];
      }
    __syncthreads();
    float factor[MT][2], back[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 16 * i + 8 * e + g;
        float most = s_m[r];
#pragma unroll
        for (int x = 1; x < kARWarps; ++x) most = fmaxf(most, s_m[x * kRows + r]);
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < kARWarps; ++x) sum += s_l[x * kRows + r] * ex2(s_m[x * kRows + r] - most);
        // 2^(ref - 138) in two steps: it may lie below fp32's normal values
        const int half = ((int)ref[i][e] - 138) / 2;
        factor[i][e] = ex2(m[i][e] - most) * __uint_as_float((unsigned)(127 + half) << 23);
        back[i][e] = __uint_as_float((unsigned)((int)ref[i][e] - 11 - half) << 23);
        m[i][e] = most;
        l[i][e] = sum;
      }
    for (int x = 0; x < kARWarps; ++x) {
      if (warp == x) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float* to = s_acc + ((i * NT + j) * 4 + e) * 32 + lane;
              const float y = o[i][j][e] * factor[i][e >> 1] * back[i][e >> 1];
              *to = x ? *to + y : y;
            }
      }
      __syncthreads();
    }

    // ---- out, or to the workspace ----
    const bool whole = u0 == 0 && u1 == n;
    float* part = a.part + (2LL * blockIdx.x + (u0 == 0)) * attend_slot(kRows, DP);
    // item: a row's half c and eight of its values in a row
    for (int x = warp; x < MT * 4 * (NT / 8); x += kARWarps) {
      const int oct = x % (NT / 8), c = x / (NT / 8) % 4, i = x / (NT / 8) / 4;
      const int r = 16 * i + 8 * (c >> 1) + g, d = (2 * t + (c & 1)) * NT + 8 * oct;
      if (row0 + r >= rows || d >= a.D) continue;
      float sum = 0.f, f[8];
#pragma unroll
      for (int y = 0; y < MT; ++y)
        if (i == y) sum = c >> 1 ? l[y][1] : l[y][0];
      const float by = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int y = 0; y < 8; ++y) f[y] = s_acc[((i * NT + 8 * oct + y) * 4 + c) * 32 + lane] * by;
      if (whole) {
        const int token = fdiv(row0 + r, a.div_g);
        attend_store8<S>((S*)a.out + (((long long)w.b * a.T + token) * a.Hq + (long long)w.h * a.G + row0 + r - token * a.G) * a.D + d, f);
      } else {
        attend_store8<uint32_t>((uint32_t*)part + r * DP + d, f);
      }
    }
    if (!whole) {
      if (warp == 0 && t == 0)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            part[kRows * DP + 16 * i + 8 * e + g] = m[i][e];
            part[kRows * DP + kRows + 16 * i + 8 * e + g] = l[i][e];
          }
      if (u0 == 0) {
        meta_last = attend_share_of(w, w.from + n - 1);
        meta_b = w.b, meta_h = w.h, meta_tile = w.tile;
      }
    }
    attend_advance<kRows, kARKeys>(a, w, u1 - u0);
  }
  if (threadIdx.x == 0) a.meta[blockIdx.x] = make_int4(meta_last, meta_b, meta_h, meta_tile);
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
// With `bytes`, only says how much workspace (a.part) the launch takes.
template <class S, bool kE4m3, int DP, int MT, int kCtas>
static cudaError_t launch_rows(KvAttendArgs a, int sms, size_t* bytes, cudaStream_t s) {
  using R = Rows<S, kE4m3, DP, MT>;
  constexpr int kRows = 16 * MT;
  auto kernel = attend_rows_kernel<S, kE4m3, DP, MT, kCtas>;
  a.tiles = (int)(((long long)a.T * a.G + kRows - 1) / kRows);
  const size_t smem = R::smem(a.T, a.parents != nullptr);
  // no more CTAs than units can be
  const long long keys = (long long)a.max_code_pages * a.block + (long long)a.max_pages * a.page_size;
  const double most = (double)a.B * a.Hkv * a.tiles * (double)(keys / kARKeys + 2);
  const int grid = (int)fmin((double)sms * kCtas, most);
  const size_t slots = ((size_t)grid * 2 * attend_slot(kRows, DP) * 4 + 255) / 256 * 256;
  if (bytes) {
    *bytes = slots + (size_t)grid * sizeof(int4);
    return cudaSuccess;
  }
  a.meta = (int4*)((char*)a.part + slots);
  if (smem > 47 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, kARThreads, smem, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_join<S, DP, kRows>(a, grid, s);
}

// CTAs of an SM by the registers that a thread needs and by the rings.
template <class S, bool kE4m3>
static cudaError_t launch_rows_of(const KvAttendArgs& a, int sms, size_t* bytes, cudaStream_t s) {
  if (a.D <= 64) return launch_rows<S, kE4m3, 64, 1, sizeof(S) == 2 ? 4 : 3>(a, sms, bytes, s);
  if (a.D <= 128) return launch_rows<S, kE4m3, 128, 1, sizeof(S) == 2 ? 3 : 2>(a, sms, bytes, s);
  return launch_rows<S, kE4m3, 256, 1, 2>(a, sms, bytes, s);
}

}  // namespace sv
