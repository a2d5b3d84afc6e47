// attend_rows.cuh -- attention of a step's tokens to a cache whose older blocks are
// 8-bit codes: few rows a head of keys, by warps with mma.sync.
//
//   out = softmax(scale q K^T) V over the keys that a token sees.
//
// A CTA takes tiles of 8 rows and units of 64 keys, a warp 16 keys of each: they come through
// its ring in shared memory by cp.async, and a warp's running maximum, sum and values stay in its
// registers; the four warps' are joined at the end of a segment.  With more rows the cache is
// read once for each tile of 8.
//
// Measured (GB300; the codes' bytes at 6.77 TB/s beside it): single tokens, 64 sequences of
// 4096 to 8192 entries, 32 heads to 8 of keys of 128, int8: 174 to 182 us (121); chains of 5 in
// fp32, 8 sequences of up to 4000, 8 heads of 80: 31 us (4.4).  In the first nothing is at its limit
// (issue slots 54 %, the integer pipe, which turns codes to fp16, 48 %, DRAM 59 % of its peak): 168 registers
// leave 12 warps an SM, and a warp's steps for 16 keys follow on one another.  The second is the chain
// of a CTA's few units, the prologue (lengths, shares, tables: about three trips to memory)
// and the joining launch.  From steps before: fragments
// from global memory to registers 212 us, with the ring 197, with the keys as the products'
// rows instead of the queries 169.
//
// Codes are exact in fp16, so q K^T and P V are fp16 products with fp32 sums: a code's
// scale multiplies the score or the weight, never the code.  Queries come as fp16
// times a power of two for each row (bf16 queries exactly, fp32 ones as a sum of two
// fp16 parts), weights as fp16 (fp32: two parts) times a power of two that follows the
// weighted scales of the values.  Plain entries become fp16 (two parts) times a power of two for each
// key.  In bf16 calls one part is enough: weights off by 2^-12 in the mean leave a result's error
// against 64 bits at that of its rounding to bf16 (0.0017 of it, as with weights in fp32).  The softmax runs in the log2 domain with one pass over the keys.
#pragma once
#include "attend_common.cuh"


namespace sv {

constexpr int kARThreads = 128;
constexpr int kARWarps = kARThreads / 32;
constexpr int kARRows = 8;              // of a tile
constexpr int kARKeys = 16 * kARWarps;  // keys of a unit: 16 to a warp
// Units whose products a warp adds up.  The products' sums drop bits, up to 2^-23 of the sum for each 16
// keys, always downwards: 2^-12 in as many units.  Longer runs are taken in pieces and added up in the workspace.
constexpr int kARPiece = 2048;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, const uint2& b) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}
// The products' own sums drop bits instead of rounding, which adds up over a long sequence: in fp32
// calls a product's sum starts at zero, its smaller parts first, and is added here.
__device__ __forceinline__ void add4(float (&c)[4], const float (&d)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] += d[i];
}
// An 8 x 8 matrix of 16-bit values (row lane / 4, columns 2 (lane % 4) and the next) turned over.
__device__ __forceinline__ uint32_t turned(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float2 floats_of(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
// What is left of two values behind their fp16 parts `w`.
__device__ __forceinline__ uint32_t rest_of(float lo, float hi, uint32_t w) {
  const float2 f = floats_of(w);
  return half2_of(lo - f.x, hi - f.y);
}

// The keys are the products' 16 rows and the queries their 8 columns (an mma.sync takes
// 8 clocks of an SM here, so half-empty sides cost as much as memory does):
//   S^T = K Q^T, O^T = V^T P^T, and P^T turns between them by movmatrix.
// A lane's place in the products (g = lane / 4, t = lane % 4).  The order in which a
// product runs over its inner index is free, so a lane's operands are bytes that lie
// together:
//   K, chunk c of 64 values: the lane's 16 codes of the keys g and g + 8 at 64 c + 16 t feed
//     four steps of 16 (step 4 c + s: its codes 4 s .. 4 s + 3);
//   V: the lane's DP / 8 codes of its keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9 at g DP / 8 are
//     the rows g and g + 8 of the DP / 16 products, so that a lane's sums of the query rows
//     2 t and 2 t + 1 are DP / 8 values in a row.
template <class S, int DP>
struct Rows {
  static constexpr bool kTwo = sizeof(S) == 4;  // two fp16 parts
  static constexpr int kSteps = DP / 16, kChunks = DP / 64, NT = DP / 16, kParts = kTwo ? 2 : 1;
  static constexpr int kFrag = kSteps * 32;  // uint2's of the queries
  // A warp's ring: 16 keys' codes, their values' and both scales a stage.
  static constexpr int kStages = DP == 256 ? 3 : 4, kStage = 2 * 16 * DP + 2 * 16 * 4;
  static_assert(NT * 4 * 32 * 4 <= kARWarps * kStages * kStage, "the warps' sums go over the rings");
  // Where 16 bytes (unit u) of a row lie: both products' reads fall on all banks.
  static __device__ __forceinline__ int at(int row, int u) {
    const int turn = DP == 64 ? (row & 2) : ((row ^ (row >> 2)) & 1) << 2 | (row & 2);
    return row * DP + ((u ^ turn) << 4);
  }
  static constexpr size_t smem(int T, bool tree) {
    return (size_t)kParts * kFrag * 8 + (size_t)kARWarps * kStages * kStage + 3 * kARWarps * kARRows * 4 + kARRows * 4 +
           (tree ? (size_t)T * 4 + (size_t)kARRows * ((T + 31) / 32) * 4 : 0);
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

// Four values in fp32.
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

template <class S, bool kE4m3, int DP, int kCtas>
__global__ void __launch_bounds__(kARThreads, kCtas) attend_rows_kernel(const __grid_constant__ KvAttendArgs a) {
  using R = Rows<S, DP>;
  constexpr int NT = R::NT, kChunks = R::kChunks, kRows = kARRows;
  constexpr bool kTwo = R::kTwo;
  constexpr int VW = DP / 32;  // words of V's codes per key and lane
  extern __shared__ __align__(16) unsigned char s_attend[];
  uint2* s_q = (uint2*)s_attend;                                      // [parts][steps][32]
  unsigned char* s_ring = (unsigned char*)(s_q + R::kParts * R::kFrag);  // the warps' rings, then
  float* s_acc = (float*)s_ring;                                      // [NT][4][32]
  float* s_m = (float*)(s_ring + kARWarps * R::kStages * R::kStage);  // [warps][rows], then sums and units
  float* s_l = s_m + kARWarps * kRows;
  int* s_unit = (int*)(s_l + kARWarps * kRows);
  float* s_qs = (float*)(s_unit + kARWarps * kRows);                  // [rows]
  int* s_par = (int*)(s_qs + kRows);                                  // [T]
  uint32_t* s_bits = (uint32_t*)(s_par + a.T);                        // [rows][words]
  __shared__ unsigned long long s_scan[kARThreads + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int words = (a.T + 31) / 32;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  Share w = attend_share<kARThreads, kRows, kARKeys>(a, s_scan);
  int meta_last = -1, meta_b = 0, meta_h = 0, meta_tile = 0;
  int loaded_b = -1, loaded_tile = -1;
  bool bad = false;
  int done = 0;  // of the share's units of the segment
  while (w.left > 0) {
    const int n = attend_units<kRows, kARKeys>(a, w.s, w.tile);
    const int last = (int)min((long long)n, w.u + w.left);
    const int u0 = w.u + done, u1 = min(last, u0 + kARPiece);
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
        // value d: chunk d / 64, lane t = d % 64 / 16, step d % 16 / 4, register d % 4 / 2
        const int step = 4 * (d >> 6) + ((d & 15) >> 2), at = r * 4 + ((d & 63) >> 4);
        const float y = finite ? x[i] * up : 0.f;
        const __half hi = __float2half_rn(y);
        __half* to = (__half*)(s_q + step * 32 + at) + (d & 3);
        *to = hi;
        if (kTwo) to[R::kFrag * 4] = __float2half_rn(y - __half2float(hi));
      }
    }
    __syncthreads();

    // ---- the lane's rows, 2 t and the next ----
    float qs[2], m[2], l[2];
    int seen[2];                // a chain's last key
    float high[2], over[2];     // the largest x + log_above(sv), and 2^-unit
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      qs[e] = s_qs[2 * t + e];
      m[e] = kLow;
      l[e] = 0.f;
      high[e] = kLow;
      over[e] = 1.f;
      seen[e] = w.s.len + fdiv(row0 + 2 * t + e, a.div_g);
    }
    const int first_seen = w.s.len + fdiv(row0, a.div_g);
    float o[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

    auto visible = [&](int e, int key, int end) {
      if (key >= end) return false;
      if (!a.parents) return key <= seen[e];
      const int at = key - w.s.len;
      return at < 0 || (lost ? false : ((s_bits[(2 * t + e) * words + (at >> 5)] >> (at & 31)) & 1u) != 0);
    };

    auto unit_of = [](float over) { return 127 - (int)(__float_as_uint(over) >> 23); };

    // Scores of the keys base + g and base + g + 8 (c[0], c[1] and c[2], c[3]) to weights.
    // sk, sv: the keys' scales.  wt: the weights as the products' right sides.
    auto weights = [&](const float (&c)[4], const float (&sk)[2], const float (&sv)[2], int base, int end, bool masked, uint2 (&wt)[R::kParts]) {
      float x[2][2];  // [row][key]
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          x[e][k] = c[2 * k + e] * (sk[k] * qs[e]);
          if (masked && !visible(e, base + g + 8 * k, end)) x[e][k] = -INFINITY;
        }
      }
      // Weights under the maximum and the unit as they are; where a row has outgrown them, they move
      // and the weights are taken again.
      float y[2][2], p[2][2];  // [key][row]
      for (bool again = false;; again = true) {
        bool grow = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            p[k][e] = ex2(x[e][k] - m[e]);
            y[k][e] = masked && x[e][k] == -INFINITY ? 0.f : p[k][e] * sv[k] * over[e];
            grow |= x[e][k] > m[e] + kSlack || y[k][e] > kMostWeight;
          }
        }
        if (again || !__any_sync(0xffffffffu, grow)) break;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float most = fmaxf(fmaxf(x[e][0], x[e][1]), m[e]);
          high[e] = fmaxf(high[e], fmaxf(x[e][0] + log_above(sv[0]), x[e][1] + log_above(sv[1])));
#pragma unroll
          for (int d = 4; d < 32; d *= 2) {
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
            high[e] = fmaxf(high[e], __shfl_xor_sync(0xffffffffu, high[e], d));
          }
          const int unit = attend_weight_unit(high[e], most);
          const float f = ex2(m[e] - most), both = f * two_to(unit_of(over[e]) - unit);
          m[e] = most;
          over[e] = two_to(-unit);
          l[e] *= f;
#pragma unroll
          for (int j = 0; j < NT; ++j) o[j][e] *= both, o[j][2 + e] *= both;
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) l[e] += p[0][e] + p[1][e];
      const uint32_t w0 = half2_of(y[0][0], y[0][1]), w1 = half2_of(y[1][0], y[1][1]);
      wt[0] = make_uint2(turned(w0), turned(w1));
      if constexpr (kTwo) wt[1] = make_uint2(turned(rest_of(y[0][0], y[0][1], w0)), turned(rest_of(y[1][0], y[1][1], w1)));
    };
    auto query = [&](int part, int step) { return s_q[(part * R::kSteps + step) * 32 + lane]; };

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
          const int e = on ? page * a.block + within : -1;
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
            const int of = __shfl_sync(0xffffffffu, e, row);
            const long long from = of * entry + 16 * u;
            // zeros behind the head, and for a page outside: a row that does not see it would get 0 * NaN
            const bool in = of >= 0 && 16 * u < a.D;
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
        float c[4] = {}, low[4] = {};
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch) {
          float part_of[4] = {};
          const uint4 k0 = *(const uint4*)(from + R::at(g, 4 * ch + t)), k1 = *(const uint4*)(from + R::at(g + 8, 4 * ch + t));
          const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint32_t b0, b1, b2, b3;
            Code<kE4m3>::word(w0[s], b0, b1);
            Code<kE4m3>::word(w1[s], b2, b3);
            if constexpr (kTwo) {
              mma16816(part_of, b0, b2, b1, b3, query(0, 4 * ch + s));
              mma16816(low, b0, b2, b1, b3, query(1, 4 * ch + s));
            } else {
              mma16816(c, b0, b2, b1, b3, query(0, 4 * ch + s));
            }
          }
          if constexpr (kTwo) add4(c, part_of);
        }
        if constexpr (kTwo) add4(c, low);
        const float sk[2] = {scales[g], scales[g + 8]}, sv[2] = {scales[16 + g], scales[24 + g]};
        const int base = u * kARKeys + 16 * warp;
        uint2 wt[R::kParts];
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
            for (int y = 0; y < 4; y += 2) {
              if constexpr (kTwo) {
                float part_of[4] = {};
                mma16816(part_of, b0[y], b0[y + 1], b1[y], b1[y + 1], wt[1]);
                mma16816(part_of, b0[y], b0[y + 1], b1[y], b1[y + 1], wt[0]);
                add4(o[2 * (x0 + x) + y / 2], part_of);
              } else {
                mma16816(o[2 * (x0 + x) + y / 2], b0[y], b0[y + 1], b1[y], b1[y + 1], wt[0]);
              }
            }
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
      // K: the keys g and g + 8; their largest magnitudes first, then their parts
      float c[4] = {}, low[4] = {}, sk[2], sv[2], up[2];
      const S* from[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int at = __shfl_sync(0xffffffffu, e, g + 8 * k);
        from[k] = kc + (long long)max(at, 0) * entry + 16 * t;
        unsigned top = 0;
#pragma unroll
        for (int x = 0; x < DP / 16; ++x)
          if (64 * (x / 4) + 16 * t < a.D) {
            float f[4];
            four_values<S>(from[k] + 64 * (x / 4) + 4 * (x & 3), f);
            top = max(top, top_bits(f));
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const bool finite = top < 0x7f800000u;
        sk[k] = at < 0 || !finite ? __uint_as_float(0x7fffffffu) : scale_down(top);
        up[k] = finite ? scale_up(top) : 0.f;
      }
#pragma unroll
      for (int x = 0; x < DP / 16; ++x) {
        float f[2][4] = {};
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (64 * (x / 4) + 16 * t < a.D && up[k] > 0.f) four_values<S>(from[k] + 64 * (x / 4) + 4 * (x & 3), f[k]);
        uint32_t p[4], r[4];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            p[k + 2 * y] = half2_of(f[k][2 * y] * up[k], f[k][2 * y + 1] * up[k]);
            if (kTwo) r[k + 2 * y] = rest_of(f[k][2 * y] * up[k], f[k][2 * y + 1] * up[k], p[k + 2 * y]);
          }
        if constexpr (kTwo) {
          float part_of[4] = {};
          mma16816(part_of, p[0], p[1], p[2], p[3], query(0, x));
          add4(c, part_of);
          mma16816(low, p[0], p[1], p[2], p[3], query(1, x));
          mma16816(low, r[0], r[1], r[2], r[3], query(0, x));
        } else {
          mma16816(c, p[0], p[1], p[2], p[3], query(0, x));
        }
      }
      if constexpr (kTwo) add4(c, low);
      // V: the scales of the keys 2 t, 2 t + 1, 2 t + 8 and 2 t + 9, then of g and g + 8
      float of[4], raise[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int at = __shfl_sync(0xffffffffu, e, 2 * t + (k & 1) + 8 * (k >> 1));
        from[k] = vc + (long long)max(at, 0) * entry + g * (DP / 8);
        unsigned top = 0;
#pragma unroll
        for (int x = 0; x < DP / 32; ++x)
          if (g * (DP / 8) + 4 * x < a.D) {
            float f[4];
            four_values<S>(from[k] + 4 * x, f);
            top = max(top, top_bits(f));
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 4));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const bool finite = top < 0x7f800000u;
        of[k] = at < 0 || !finite ? __uint_as_float(0x7fffffffu) : scale_down(top);
        raise[k] = finite ? scale_up(top) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float even = __shfl_sync(0xffffffffu, of[2 * k], g >> 1), odd = __shfl_sync(0xffffffffu, of[2 * k + 1], g >> 1);
        sv[k] = g & 1 ? odd : even;
      }
      uint2 wt[R::kParts];
      weights(c, sk, sv, base, keys.end, true, wt);
#pragma unroll
      for (int x = 0; x < DP / 32; ++x) {  // four values of a place at a time
        float f[4][4] = {};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (g * (DP / 8) + 4 * x < a.D && raise[k] > 0.f) four_values<S>(from[k] + 4 * x, f[k]);
#pragma unroll
        for (int y = 0; y < 4; y += 2) {
          uint32_t p[4], r[4];
#pragma unroll
          for (int d = 0; d < 2; ++d)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float y0 = f[2 * k][y + d] * raise[2 * k], y1 = f[2 * k + 1][y + d] * raise[2 * k + 1];
              p[d + 2 * k] = half2_of(y0, y1);
              if (kTwo) r[d + 2 * k] = rest_of(y0, y1, p[d + 2 * k]);
            }
          if constexpr (kTwo) {
            float part_of[4] = {};
            mma16816(part_of, p[0], p[1], p[2], p[3], wt[1]);
            mma16816(part_of, r[0], r[1], r[2], r[3], wt[0]);
            mma16816(part_of, p[0], p[1], p[2], p[3], wt[0]);
            add4(o[2 * x + y / 2], part_of);
          } else {
            mma16816(o[2 * x + y / 2], p[0], p[1], p[2], p[3], wt[0]);
          }
        }
        asm volatile("" ::: "memory");
      }
    }

    // ---- the warps' sums become one ----
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int d = 4; d < 32; d *= 2) l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
      if (lost) l[e] = __uint_as_float(0x7fffffffu);
      if (g == 0) {
        const int at = warp * kRows + 2 * t + e;
        s_m[at] = m[e], s_l[at] = l[e], s_unit[at] = unit_of(over[e]);
      }
    }
    __syncthreads();
    const bool more = done > 0;  // to sums that are in the workspace
    float* part = a.part + (2LL * blockIdx.x + (w.u == 0)) * attend_slot(kRows, DP);
    float factor[2], of[2];
    int unit[2];  // of the sums
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 2 * t + e;
      float most = s_m[r];
#pragma unroll
      for (int x = 1; x < kARWarps; ++x) most = fmaxf(most, s_m[x * kRows + r]);
      float sum = 0.f, top = -INFINITY, old = 0.f;
      int its = 0;
      if (more) {
        const float* there = part + kRows * DP + r;
        most = fmaxf(most, there[0]);
        old = ex2(there[0] - most), its = __float_as_int(there[2 * kRows]);
        sum = there[kRows] * old;
        if (old > 0.f) top = there[0] + (float)its;
      }
#pragma unroll
      for (int x = 0; x < kARWarps; ++x) {
        const float by = ex2(s_m[x * kRows + r] - most);
        sum += s_l[x * kRows + r] * by;
        if (by > 0.f) top = fmaxf(top, s_m[x * kRows + r] + (float)s_unit[x * kRows + r]);
      }
      unit[e] = attend_unit(top, most);
      factor[e] = ex2(m[e] - most) * two_to(unit_of(over[e]) - unit[e]);
      of[e] = old * two_to(its - unit[e]);
      m[e] = most;
      l[e] = sum;
    }
    for (int x = 0; x < kARWarps; ++x) {
      if (warp == x) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* to = s_acc + (j * 4 + e) * 32 + lane;
            const float y = o[j][e] * factor[e & 1];
            *to = x ? *to + y : y;
          }
      }
      __syncthreads();
    }

    // ---- out, or to the workspace ----
    const bool whole = w.u == 0 && u1 == n;
    // item: row 2 t + e of a lane, eight of its values in a row
    for (int x = warp; x < 2 * (NT / 4); x += kARWarps) {
      const int e = x & 1, oct = x >> 1, r = 2 * t + e, d = g * (DP / 8) + 8 * oct;
      if (row0 + r >= rows || d >= a.D) continue;
      // 2^unit in two steps: their product may lie outside fp32's normal values
      const int its = e ? unit[1] : unit[0], half = its / 2;
      const float by = !whole ? 1.f : l[0] == 0.f && !e || l[1] == 0.f && e ? 0.f : 1.f / (e ? l[1] : l[0]) * two_to(half);
      const float rest = whole ? two_to(its - half) : 1.f;
      float f[8];
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        f[y] = s_acc[((4 * oct + y / 2) * 4 + 2 * (y & 1) + e) * 32 + lane];
        if (more) f[y] += part[r * DP + d + y] * (e ? of[1] : of[0]);
        f[y] = f[y] * by * rest;
      }
      if (whole) {
        const int token = fdiv(row0 + r, a.div_g);
        attend_store8<S>((S*)a.out + (((long long)w.b * a.T + token) * a.Hq + (long long)w.h * a.G + row0 + r - token * a.G) * a.D + d, f);
      } else {
        attend_store8<uint32_t>((uint32_t*)part + r * DP + d, f);
      }
    }
    if (!whole) {
      if (warp == 0 && g == 0)
#pragma unroll
        for (int e = 0; e < 2; ++e) attend_leave(part, kRows, DP, 2 * t + e, m[e], l[e], unit[e]);
      if (w.u == 0 && last < n) {
        meta_last = attend_joint(attend_share_of(w, w.from + n - 1), min(kRows, rows - row0));
        meta_b = w.b, meta_h = w.h, meta_tile = w.tile;
      }
    }
    done += u1 - u0;
    if (u1 < last) continue;  // (the slot is read behind the next barrier)
    attend_advance<kRows, kARKeys>(a, w, done);
    done = 0;
  }
  if (threadIdx.x == 0) a.meta[blockIdx.x] = make_int4(meta_last, meta_b, meta_h, meta_tile);
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
// With `bytes`, only says how much workspace (a.part) the launch takes.
template <class S, bool kE4m3, int DP, int kCtas>
static cudaError_t launch_rows(KvAttendArgs a, int sms, size_t* bytes, cudaStream_t s) {
  using R = Rows<S, DP>;
  constexpr int kRows = kARRows;
  auto kernel = attend_rows_kernel<S, kE4m3, DP, kCtas>;
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
  // The attribute is the largest tree's, always: another host thread's call may set it between this one's and the launch.
  constexpr size_t most_smem = R::smem(kMaxTreeNodes + 1, true);
  if (most_smem > 47 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most_smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, kARThreads, smem, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_join<S, DP, kRows>(a, grid, s);
}

// CTAs of an SM by the registers that a thread needs without spilling (fp32 calls hold two
// parts of everything) and by the rings.
template <class S, bool kE4m3>
static cudaError_t launch_rows_of(const KvAttendArgs& a, int sms, size_t* bytes, cudaStream_t s) {
  if (a.D <= 64) return launch_rows<S, kE4m3, 64, sizeof(S) == 4 ? 4 : 5>(a, sms, bytes, s);
  if (a.D <= 128) return launch_rows<S, kE4m3, 128, sizeof(S) == 4 ? 2 : 3>(a, sms, bytes, s);
  return launch_rows<S, kE4m3, 256, 2>(a, sms, bytes, s);
}

}  // namespace sv
