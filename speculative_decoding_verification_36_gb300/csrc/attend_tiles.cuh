// attend_tiles.cuh -- attention of a step's tokens to a cache whose older blocks are
// 8-bit codes: many rows a head of keys, on the tensor cores of the SM (tcgen05).
//
// One CTA an SM takes tiles of 128 rows and units of 128 keys:
//   S = Q K^T      128 x 128 x D, both operands in shared memory as fp16
//   P = weights    fp16, over S's columns in tensor memory
//   O += P V       128 x D x 128, P from tensor memory, V from shared memory
// Eight warps bring keys and values: codes go from global memory to registers two
// units ahead, become fp16 (exactly) and are written to shared memory in the 128-byte
// swizzle; plain entries become fp16 times a power of two for each key.  Eight warps make weights of
// scores: a thread has one row and half of the unit's keys, so that rows need no
// shuffles and two threads agree on a row's maximum through shared memory.  One thread
// issues the products; S is double-buffered, so that the next scores are computed
// while the weights of the last ones are made.
//
// The scales never touch the codes: a key's scale multiplies its scores, a value's its
// weight.  With M = m + ref - 138 (m the running maximum in log2, ref exponent bits above every
// scale of V that the row has seen) a weight is 2^(x - M) sv, below 2^15, and the row's sum is
// that of 2^(x - M): the powers of two cancel in the quotient.
#pragma once
#include "attend_common.cuh"
#include "sv_bulk.cuh"

namespace sv {

constexpr int kATRows = 128, kATKeys = 128;
constexpr int kATSoft = 8, kATLoad = 8;                    // warps of each kind
constexpr int kATThreads = 32 * (kATSoft + kATLoad + 1);   // and one that issues
constexpr int kATRing = 4;                                 // units whose scales are held
constexpr unsigned kATLeastRef = 64;  // values below 2^-82 lose bits, which keeps a row's sum below 2^128

// Shared memory; each operand begins on a 1024-byte boundary, as the swizzle wants.
template <int DP>
struct Tiles {
  static constexpr int kTile = 128 * DP * 2;  // bytes of an operand
  static constexpr int kChunk = 128 * 128;    // 128 rows of 64 fp16
  static constexpr int kQ = 0, kK = kTile, kV = 3 * kTile, kRest = 5 * kTile;
  static constexpr int kSlot = 128 * DP + 2 * 128;  // floats that a share leaves
  struct Rest {
    float sk[kATRing][kATKeys], sv[kATRing][kATKeys];
    float qs[kATRows];
    float most[2][2][kATRows];     // [turn][half]
    unsigned top[2][2][kATRows];
    float sum[2][kATRows];
    uint32_t bits[kATRows][4];
    int parents[128];
    unsigned long long k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_ready[2], pv_done[2], q_full, drain;
    uint32_t tmem;
    int wrong;
    int meta[4];
  };
  static constexpr size_t smem = kRest + sizeof(Rest) + 1024;
};

// ---- tcgen05 ----
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(unsigned long long* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// D = A B (+ D), A in shared memory
__device__ __forceinline__ void tc_mma(uint32_t d, unsigned long long a, unsigned long long b, uint32_t kind, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
      : "memory");
}
// ... A in tensor memory
__device__ __forceinline__ void tc_mma_t(uint32_t d, uint32_t a, unsigned long long b, uint32_t kind, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
      : "memory");
}
#define SV_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define SV_W8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
// 32 columns of the warp's 32 lanes (a register a column)
__device__ __forceinline__ void tc_load32(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
      "%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : SV_R8(r, 0), SV_R8(r, 8), SV_R8(r, 16), SV_R8(r, 24)
      : "r"(at));
}
__device__ __forceinline__ void tc_load16(uint32_t at, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : SV_R8(r, 0), SV_R8(r, 8)
               : "r"(at));
}
__device__ __forceinline__ void tc_store16(uint32_t at, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::SV_W8(r, 0),
               SV_W8(r, 8), "r"(at)
               : "memory");
}
// The loads have come: the registers are operands, so that nothing uses them before.
#define SV_M8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
__device__ __forceinline__ void tc_loaded16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : SV_M8(r, 0), SV_M8(r, 8)::"memory");
}
__device__ __forceinline__ void tc_loaded64(uint32_t (&r)[64]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : SV_M8(r, 0), SV_M8(r, 8)::"memory");
  asm volatile("" : SV_M8(r, 16), SV_M8(r, 24));
  asm volatile("" : SV_M8(r, 32), SV_M8(r, 40));
  asm volatile("" : SV_M8(r, 48), SV_M8(r, 56));
}
__device__ __forceinline__ void tc_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// An operand of 128-byte rows in the 128-byte swizzle: groups of 8 rows 1024 bytes
// apart, columns past 64 values a chunk further on.
__device__ __forceinline__ unsigned long long tc_operand(uint32_t at, uint32_t chunk) {
  return (unsigned long long)((at & 0x3ffffu) >> 4) | (unsigned long long)(chunk >> 4) << 16 | (unsigned long long)(1024u >> 4) << 32 |
         1ull << 46 | 2ull << 61;
}
// fp16 operands, fp32 sums, M = 128; the right side's rows are the inner index where `by_rows`
__device__ __forceinline__ constexpr uint32_t tc_kind(int n, bool by_rows) {
  return 1u << 4 | (by_rows ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 | (128u / 16) << 24;
}

__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// Where 16 bytes (unit u of 8 in a 128-byte row) of a row lie.
__device__ __forceinline__ int swizzled(int row, int u) { return row * 128 + ((u ^ (row & 7)) << 4); }

template <bool kE4m3, int DP>
__global__ void __launch_bounds__(kATThreads, 1) attend_tiles_kernel(const __grid_constant__ KvAttendArgs a) {
  using L = Tiles<DP>;
  extern __shared__ unsigned char s_raw[];
  __shared__ unsigned long long s_scan[512 + 1];
  unsigned char* base = s_raw + ((1024u - (smem_addr(s_raw) & 1023u)) & 1023u);
  typename L::Rest& r = *(typename L::Rest*)(base + L::kRest);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned tries = mbar_tries(spin_limit());
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&r.k_full[i], kATLoad);
      mbar_init(&r.v_full[i], kATLoad);
      mbar_init(&r.k_empty[i], 1);
      mbar_init(&r.v_empty[i], 1);
      mbar_init(&r.s_full[i], 2);
      mbar_init(&r.pv_done[i], 1);
      mbar_init(&r.p_ready[i], kATSoft);
    }
    mbar_init(&r.q_full, kATSoft);
    mbar_init(&r.drain, 1);
    r.wrong = 0;
    r.meta[0] = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kATSoft + kATLoad) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&r.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  Share w = attend_share<512, kATRows, kATKeys>(a, s_scan);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *(volatile uint32_t*)&r.tmem;
  const uint32_t t_o = tmem + 256;  // S at 0 and 128, O at 256
  // Once a wait has run out the warp goes on without waiting and takes part in every
  // barrier that is left: no warp waits for one that is gone.
  bool dead = false;
  auto wait = [&](unsigned long long* bar, unsigned parity) {
    if (!dead && !warp_wait(bar, parity & 1, tries)) dead = true;
  };

  if (warp < kATSoft) {
    // =====================================================================
    // weights
    // =====================================================================
    const int half = warp >> 2, quarter = warp & 3, row = 32 * quarter + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    int i = 0, turn = 0;  // units so far; exchanges so far
    int loaded_b = -1, loaded_tile = -1;
    bool bad = false;
    auto both = [&]() { bar_sync(1 + quarter, 64); };  // the two warps of these rows
    while (w.left > 0) {
      const int n = attend_units<kATRows, kATKeys>(a, w.s, w.tile);
      const int u0 = w.u, u1 = (int)min((long long)n, u0 + w.left);
      const Keys keys = attend_keys<kATRows>(a, w.s, w.tile);
      const int row0 = w.tile * kATRows, rows = w.s.n_new * a.G;
      // ---- queries to shared memory: all scores of the last segment are there ----
      if (a.parents && (w.b != loaded_b || w.tile != loaded_tile)) {
        bar_sync(5, 32 * kATSoft);  // nobody reads the last tree
        if (threadIdx.x == 0) r.wrong = 0;
        bar_sync(5, 32 * kATSoft);
        const int N = a.T - 1;
        if ((int)threadIdx.x < N) {
          const int p = __ldg(a.parents + (long long)w.b * N + threadIdx.x);
          r.parents[threadIdx.x] = p;
          if (p < -1 || p >= (int)threadIdx.x) r.wrong = 1;
        }
        bar_sync(5, 32 * kATSoft);
        bad = r.wrong != 0;
        if (!bad && threadIdx.x < kATRows) {
          const int token = fdiv(row0 + threadIdx.x, a.div_g);
          if (token < a.T) attend_bits(r.parents, token, 4, r.bits[threadIdx.x]);
        }
      }
      loaded_b = w.b, loaded_tile = w.tile;
      const bool lost = w.s.bad || (a.parents && bad);
      if (lost && threadIdx.x == 0) atomicOr(a.status, kStatusBadData);
      {
        // a warp a row, a lane four values in a row; eight rows in flight
        const bool fast = ((uintptr_t)a.q & 7) == 0 && a.q_stride % 4 == 0;
        const int live = min(kATRows, rows - row0);
        for (int r0 = warp; r0 < live; r0 += 8 * kATSoft) {
          uint2 x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int q = r0 + k * kATSoft;
            x[k] = make_uint2(0, 0);
            if (q < live && 4 * lane < a.D && !lost) {
              const int token = fdiv(row0 + q, a.div_g);
              const uint16_t* p = (const uint16_t*)a.q + ((long long)w.b * a.T + token) * a.q_stride +
                                  ((long long)w.h * a.G + row0 + q - token * a.G) * a.D + 4 * lane;
              if (fast)
                x[k] = *(const uint2*)p;
              else
                x[k] = make_uint2(p[0] | (uint32_t)p[1] << 16, p[2] | (uint32_t)p[3] << 16);
            }
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int q = r0 + k * kATSoft;
            if (q >= live) break;
            unsigned top = max(max(x[k].x << 16 & 0x7fff0000u, x[k].x & 0x7fff0000u), max(x[k].y << 16 & 0x7fff0000u, x[k].y & 0x7fff0000u));
            top = __reduce_max_sync(0xffffffffu, top);
            const bool finite = top < 0x7f800000u;
            // the scale's sign goes with the query: what multiplies the scores is positive
            const float up = !finite ? 0.f : a.scale < 0.f ? -scale_up(top) : scale_up(top);
            if (lane == 0) r.qs[q] = lost || !finite ? __uint_as_float(0x7fffffffu) : scale_down(top) * fabsf(a.scale);
            if (4 * lane < a.D) {
              uint2 y = make_uint2(0, 0);
              if (finite)
                y = make_uint2(half2_of(bf16_lo(x[k].x) * up, bf16_hi(x[k].x) * up), half2_of(bf16_lo(x[k].y) * up, bf16_hi(x[k].y) * up));
              const int d = 4 * lane;
              *(uint2*)(base + L::kQ + (d >> 6) * L::kChunk + swizzled(q, (d & 63) >> 3) + (d & 4) * 2) = y;
            }
          }
        }
        fence_async();
        bar_sync(5, 32 * kATSoft);  // also: r.qs and the tree's bits
        if (lane == 0) mbar_arrive(&r.q_full);
      }
      const float qs = r.qs[row];
      const bool active = 32 * quarter < rows - row0;
      const int last_seen = w.s.len + fdiv(row0 + row, a.div_g), first_seen = w.s.len + fdiv(row0, a.div_g);
      float m = kLow, M = kLow, l = 0.f;
      unsigned ref = kATLeastRef;
      const int n_codes = w.s.bad ? 0 : (keys.codes + kATKeys - 1) / kATKeys;
      for (int u = u0; u < u1; ++u, ++i) {
        const int s = i & 1;
        wait(&r.s_full[s], i >> 1);
        tc_after();
        if (active && !w.s.bad) {
          const float* sk = r.sk[i & (kATRing - 1)] + 64 * half;
          const float* sv = r.sv[i & (kATRing - 1)] + 64 * half;
          const uint32_t t_s = tmem + 128 * s + 64 * half + lanes;
          uint32_t x[64];
          tc_load32(t_s, x);
          tc_load32(t_s + 32, x + 32);
          const bool codes = u < n_codes;
          const int first = (codes ? u * kATKeys : keys.stored + (u - n_codes) * kATKeys) + 64 * half;  // the thread's first key
          const int end = codes ? keys.codes : keys.end;
          const int unit = first - 64 * half;
          const bool masked = unit + kATKeys > end || (a.parents ? unit + kATKeys > w.s.len : unit + kATKeys - 1 > first_seen);
          const bool groups = codes && !masked && a.block % 16 == 0;  // 16 keys in a row share their scales
          float most = -INFINITY;
          unsigned top = kATLeastRef;
          tc_loaded64(x);
          if (groups) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              float y = __uint_as_float(x[16 * g]);
#pragma unroll
              for (int k = 1; k < 16; ++k) y = fmaxf(y, __uint_as_float(x[16 * g + k]));
              most = fmaxf(most, y * sk[16 * g]);
              const unsigned b = __float_as_uint(sv[16 * g]);
              if (b < 0x7f800000u) top = max(top, (b >> 23) + 1u);
            }
          } else {
            // the keys that the row sees, as bits
            uint32_t vis[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int f = first + 32 * k, behind = min(end - f, a.parents ? 32 : last_seen - f + 1);
              vis[k] = behind <= 0 ? 0u : behind >= 32 ? 0xffffffffu : (1u << behind) - 1u;
              if (a.parents) {
                const int at = f - w.s.len;  // the first key as a token of the step
                if (at > -32) {
                  const int word = at >> 5;  // -1 .. 3
                  const uint32_t lo = word < 0 ? 0xffffffffu : word < 4 ? r.bits[row][word] : 0u;
                  const uint32_t hi = word + 1 < 4 ? r.bits[row][word + 1] : 0u;
                  vis[k] &= __funnelshift_r(lo, hi, at & 31);
                }
              }
            }
#pragma unroll
            for (int k = 0; k < 64; ++k) {
              const bool see = (vis[k >> 5] >> (k & 31)) & 1u;
              const float y = __uint_as_float(x[k]) * sk[k];
              x[k] = __float_as_uint(see ? y : -INFINITY);
              most = fmaxf(most, __uint_as_float(x[k]));
              const unsigned b = __float_as_uint(sv[k]);
              if (see && b < 0x7f800000u) top = max(top, (b >> 23) + 1u);
            }
          }
          most *= qs;  // (a scale of 0: -inf becomes NaN, which no maximum takes)
          top = min(top, 254u);
          r.most[turn & 1][half][row] = most;
          r.top[turn & 1][half][row] = top;
          both();
          most = fmaxf(most, r.most[turn & 1][half ^ 1][row]);
          top = max(top, r.top[turn & 1][half ^ 1][row]);
          ++turn;
          if (__any_sync(0xffffffffu, most > m + kSlack || top > ref)) {
            m = fmaxf(m, most);
            ref = max(ref, top);
            const float M2 = m + ((float)ref - 138.f), f = ex2(M - M2);
            M = M2;
            l *= f;
            if (u > u0) {
              const int j = i - 1;
              wait(&r.pv_done[j & 1], j >> 1);
              tc_after();
#pragma unroll 1
              for (int c = 0; c < DP / 2; c += 16) {
                uint32_t o[16];
                const uint32_t at = t_o + lanes + half * (DP / 2) + c;
                tc_load16(at, o);
                tc_loaded16(o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tc_store16(at, o);
              }
            }
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t p[16];
            if (groups) {
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                const float by = sk[32 * c + 16 * g] * qs, v = sv[32 * c + 16 * g];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const float p0 = ex2(fmaf(__uint_as_float(x[32 * c + 16 * g + 2 * k]), by, -M));
                  const float p1 = ex2(fmaf(__uint_as_float(x[32 * c + 16 * g + 2 * k + 1]), by, -M));
                  l += p0 + p1;
                  p[8 * g + k] = half2_of(p0 * v, p1 * v);
                }
              }
            } else {
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float x0 = __uint_as_float(x[32 * c + 2 * k]), x1 = __uint_as_float(x[32 * c + 2 * k + 1]);
                // what is not seen has no part, whatever its scales are
                const float p0 = x0 == -INFINITY ? 0.f : ex2(fmaf(x0, qs, -M)), p1 = x1 == -INFINITY ? 0.f : ex2(fmaf(x1, qs, -M));
                l += p0 + p1;
                p[k] = half2_of(x0 == -INFINITY ? 0.f : p0 * sv[32 * c + 2 * k], x1 == -INFINITY ? 0.f : p1 * sv[32 * c + 2 * k + 1]);
              }
            }
            tc_store16(t_s + 16 * c, p);
          }
          tc_stored();
        }
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&r.p_ready[s]);
      }
      // ---- out, or to the workspace ----
      const int j = i - 1;
      wait(&r.pv_done[j & 1], j >> 1);
      tc_after();
      if (active) {
        if (lost) l = __uint_as_float(0x7fffffffu);
        both();
        r.sum[half][row] = l;
        both();
        l += r.sum[half ^ 1][row];
        const bool whole = u0 == 0 && u1 == n, mine = row0 + row < rows;
        const float by = l == 0.f ? 0.f : 1.f / l;
        const int token = fdiv(row0 + row, a.div_g);
        uint16_t* out = (uint16_t*)a.out + (((long long)w.b * a.T + token) * a.Hq + (long long)w.h * a.G + row0 + row - token * a.G) * a.D;
        float* part = a.part + (2LL * blockIdx.x + (u0 == 0)) * L::kSlot;
#pragma unroll 1
        for (int c = half * (DP / 2); c < (half + 1) * (DP / 2); c += 16) {
          uint32_t o[16];
          tc_load16(t_o + lanes + c, o);
          tc_loaded16(o);
          if (mine && c < a.D) {
            if (whole) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float f[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = lost ? l : __uint_as_float(o[8 * e + k]) * by;
                attend_store8<uint16_t>(out + c + 8 * e, f);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                ((uint4*)(part + row * DP + c))[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
          }
          __syncwarp();
        }
        if (!whole && half == 0 && mine) part[128 * DP + row] = M, part[128 * DP + 128 + row] = l;
      }
      tc_before();
      if (u0 == 0 && u1 < n && threadIdx.x == 0) {
        r.meta[0] = attend_share_of(w, w.from + n - 1);
        r.meta[1] = w.b, r.meta[2] = w.h, r.meta[3] = w.tile;
      }
      attend_advance<kATRows, kATKeys>(a, w, u1 - u0);
    }
  } else if (warp < kATSoft + kATLoad) {
    // =====================================================================
    // keys and values
    // =====================================================================
    constexpr int kPer = DP / 16, kAtOnce = 32 * kATLoad / kPer, kRounds = kATKeys / kAtOnce;  // lanes a key, keys at once
    const int x = threadIdx.x - 32 * kATSoft, part = x % kPer, mine = x / kPer;
    const bool on = 16 * part < a.D;
    const long long entry = (long long)a.Hkv * a.D;
    int i = 0;
    auto wait_empty = [&](unsigned long long* bar) {  // the operand of two units ago has been read
      if (i >= 2) wait(&bar[i & 1], (i >> 1) + 1);
    };
    auto full = [&](unsigned long long* bar) {
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[i & 1]);
    };
    while (w.left > 0) {
      const int n = attend_units<kATRows, kATKeys>(a, w.s, w.tile);
      const int u0 = w.u, u1 = (int)min((long long)n, u0 + w.left);
      const Keys keys = attend_keys<kATRows>(a, w.s, w.tile);
      const int n_codes = w.s.bad ? 0 : (keys.codes + kATKeys - 1) / kATKeys, uc = min(u1, n_codes);
      if (u0 < uc) {
        const int32_t* table = a.code_table + (long long)w.b * a.max_code_pages;
        const uint8_t* kc = a.k_codes + (long long)w.h * a.D + 16 * part;
        const uint8_t* vc = a.v_codes + (long long)w.h * a.D + 16 * part;
        uint4 k[2][kRounds], v[2][kRounds];
        float scale[2];  // lane `part` has one of the scales of its keys: K's of key part % kRounds, or V's
        int page[kRounds], at[2][kRounds];
        auto look = [&](int u) {
#pragma unroll
          for (int q = 0; q < kRounds; ++q) page[q] = __ldg(table + fdiv(min(u * kATKeys + mine + q * kAtOnce, keys.codes - 1), a.div_block));
        };
        auto place = [&](int u, int b) {  // of the unit that was looked up
          int p = page[0];
#pragma unroll
          for (int q = 0; q < kRounds; ++q) {
            const int key = min(u * kATKeys + mine + q * kAtOnce, keys.codes - 1), in = key - fdiv(key, a.div_block) * a.block;
            if (part % kRounds == q) p = page[q];
            at[b][q] = page[q] >= 0 && page[q] < a.code_pages ? page[q] * a.block + in : 0;
          }
          scale[b] = __uint_as_float(0x7fffffffu);
          if (part < 2 * kRounds) {
            if (p >= 0 && p < a.code_pages)
              scale[b] = __ldg((part < kRounds ? a.k_scales : a.v_scales) + (long long)p * a.Hkv + w.h);
            else
              atomicOr(a.status, kStatusBadData);
          }
        };
        auto load = [&](const uint8_t* from, const int (&e)[kRounds], uint4 (&to)[kRounds]) {
#pragma unroll
          for (int q = 0; q < kRounds; ++q) to[q] = on ? stream16(from + (long long)e[q] * entry) : make_uint4(0, 0, 0, 0);
        };
        auto put = [&](const uint4 (&from)[kRounds], unsigned char* to) {
          if (!on) return;
#pragma unroll
          for (int q = 0; q < kRounds; ++q) {
            const int key = mine + q * kAtOnce;
            uint4 y[2];
            Code<kE4m3>::word(from[q].x, y[0].x, y[0].y);
            Code<kE4m3>::word(from[q].y, y[0].z, y[0].w);
            Code<kE4m3>::word(from[q].z, y[1].x, y[1].y);
            Code<kE4m3>::word(from[q].w, y[1].z, y[1].w);
            // eight lanes write eight different units: those of the second chunk their upper one first
            unsigned char* c = to + (part >> 2) * L::kChunk;
            const int unit = 2 * (part & 3), up = part >> 2;
            *(uint4*)(c + swizzled(key, unit + up)) = up ? y[1] : y[0];
            *(uint4*)(c + swizzled(key, unit + 1 - up)) = up ? y[0] : y[1];
          }
        };
        look(u0);
        place(u0, 0);
        load(kc, at[0], k[0]);
        load(vc, at[0], v[0]);
        if (u0 + 1 < uc) {
          look(u0 + 1);
          place(u0 + 1, 1);
          load(kc, at[1], k[1]);
          load(vc, at[1], v[1]);
          if (u0 + 2 < uc) look(u0 + 2);
        }
        for (int u = u0; u < uc; u += 2) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            if (u + b >= uc) break;
            const bool more = u + b + 2 < uc;
            wait_empty(r.k_empty);
            put(k[b], base + L::kK + (i & 1) * L::kTile);
            if (part < 2 * kRounds)
              (part < kRounds ? r.sk : r.sv)[i & (kATRing - 1)][mine + (part % kRounds) * kAtOnce] = scale[b];
            if (more) {
              place(u + b + 2, b);
              load(kc, at[b], k[b]);
            }
            full(r.k_full);
            wait_empty(r.v_empty);
            put(v[b], base + L::kV + (i & 1) * L::kTile);
            if (more) load(vc, at[b], v[b]);
            if (u + b + 3 < uc) look(u + b + 3);
            full(r.v_full);
            ++i;
          }
        }
      }
      // plain entries: twice as many lanes a key, eight values each
      for (int u = max(u0, uc); u < u1; ++u) {
        constexpr int kPer2 = DP / 8, kAtOnce2 = 32 * kATLoad / kPer2, kRounds2 = kATKeys / kAtOnce2;
        const int part2 = x % kPer2, mine2 = x / kPer2;
        const bool on2 = 8 * part2 < a.D;
        int at[kRounds2];
        if (!w.s.bad) {
#pragma unroll
          for (int q = 0; q < kRounds2; ++q) {
            const int key = min(keys.stored + (u - n_codes) * kATKeys + mine2 + q * kAtOnce2, keys.end - 1), p = fdiv(key, a.div_page);
            const int page = __ldg(a.page_table + (long long)w.b * a.max_pages + p);
            const bool ok = page >= 0 && page < a.pages;
            if (!ok) atomicOr(a.status, kStatusBadData);
            at[q] = ok ? page * a.page_size + (key - p * a.page_size) : -1;
          }
        }
        auto fetch = [&](const void* cache, unsigned char* to, float* scales) {
          uint4 y[kRounds2];
#pragma unroll
          for (int q = 0; q < kRounds2; ++q)
            y[q] = on2 && at[q] >= 0 ? *(const uint4*)((const uint16_t*)cache + (long long)at[q] * entry + w.h * a.D + 8 * part2)
                                     : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int q = 0; q < kRounds2; ++q) {
            const unsigned lo = max(max(y[q].x & 0x7fffu, y[q].y & 0x7fffu), max(y[q].z & 0x7fffu, y[q].w & 0x7fffu));
            const unsigned hi = max(max(y[q].x & 0x7fff0000u, y[q].y & 0x7fff0000u), max(y[q].z & 0x7fff0000u, y[q].w & 0x7fff0000u));
            unsigned top = max(lo << 16, hi);
#pragma unroll
            for (int d = 1; d < kPer2; d *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
            const bool finite = top < 0x7f800000u;
            const float up = finite ? scale_up(top) : 0.f;
            if (part2 == 0) scales[mine2 + q * kAtOnce2] = at[q] >= 0 && finite ? scale_down(top) : __uint_as_float(0x7fffffffu);
            uint4 z = make_uint4(0, 0, 0, 0);
            if (finite)
              z = make_uint4(half2_of(bf16_lo(y[q].x) * up, bf16_hi(y[q].x) * up), half2_of(bf16_lo(y[q].y) * up, bf16_hi(y[q].y) * up),
                             half2_of(bf16_lo(y[q].z) * up, bf16_hi(y[q].z) * up), half2_of(bf16_lo(y[q].w) * up, bf16_hi(y[q].w) * up));
            if (on2) *(uint4*)(to + (part2 >> 3) * L::kChunk + swizzled(mine2 + q * kAtOnce2, part2 & 7)) = z;
          }
        };
        // the values' scales have to be there with the scores: both are fetched first
        wait_empty(r.k_empty);
        if (!w.s.bad) fetch(a.k_cache, base + L::kK + (i & 1) * L::kTile, r.sk[i & (kATRing - 1)]);
        wait_empty(r.v_empty);
        if (!w.s.bad) fetch(a.v_cache, base + L::kV + (i & 1) * L::kTile, r.sv[i & (kATRing - 1)]);
        full(r.k_full);
        full(r.v_full);
        ++i;
      }
      attend_advance<kATRows, kATKeys>(a, w, u1 - u0);
    }
  } else {
    // =====================================================================
    // products
    // =====================================================================
    const uint32_t s_q = smem_addr(base + L::kQ), s_k = smem_addr(base + L::kK), s_v = smem_addr(base + L::kV);
    const uint32_t kind_s = tc_kind(128, false), kind_o = tc_kind(a.D, true);
    int i = 0, segments = 0;
    bool open = false;  // unit i - 1 has no P V yet
    bool fresh = false; // ... and begins its segment
    auto pv = [&]() {   // of unit i - 1
      const int j = i - 1, s = j & 1;
      wait(&r.p_ready[s], j >> 1);
      wait(&r.v_full[s], j >> 1);
      tc_after();
      if (lane == 0 && !dead) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc_mma_t(t_o, tmem + 128 * s + 64 * (k >> 2) + 8 * (k & 3), tc_operand(s_v + s * L::kTile + k * 2048, L::kChunk), kind_o,
                   k > 0 || !fresh);
        tc_commit(&r.v_empty[s]);
        tc_commit(&r.pv_done[s]);
      }
      __syncwarp();
      open = false;
    };
    while (w.left > 0) {
      const int n = attend_units<kATRows, kATKeys>(a, w.s, w.tile);
      const int u0 = w.u, u1 = (int)min((long long)n, u0 + w.left);
      for (int u = u0; u < u1; ++u, ++i) {
        const int s = i & 1;
        if (u == u0) {  // the last segment's products come to their end, then its queries go
          if (open) pv();
          wait(&r.q_full, segments++);
        }
        // S's columns hold the weights of unit i - 2 until P V has read them
        wait(&r.k_full[s], i >> 1);
        if (i >= 2) wait(&r.pv_done[s], (i >> 1) + 1);
        tc_after();
        if (lane == 0 && !dead) {
          for (int k = 0; k < a.D / 16; ++k) {
            const uint32_t off = (k >> 2) * L::kChunk + (k & 3) * 32;
            tc_mma(tmem + 128 * s, tc_operand(s_q + off, 16), tc_operand(s_k + s * L::kTile + off, 16), kind_s, k > 0);
          }
          tc_commit(&r.k_empty[s]);
          tc_commit(&r.s_full[s]);
          mbar_arrive(&r.s_full[s]);  // with what k_full brought: the scales
        }
        __syncwarp();
        if (open) pv();
        open = true;
        fresh = u == u0;
      }
      attend_advance<kATRows, kATKeys>(a, w, u1 - u0);
    }
    if (open) pv();
    // nothing of the tensor cores is in flight when the tensor memory goes back
    if (lane == 0) tc_commit(&r.drain);
    __syncwarp();
    if (!warp_wait(&r.drain, 0, mbar_tries(kSpinLimit))) dead = true;
  }
  if (dead && lane == 0) atomicOr(a.status, kStatusTimeout);
  tc_before();
  __syncthreads();
  if (warp == kATSoft + kATLoad) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
  if (threadIdx.x == 0) a.meta[blockIdx.x] = make_int4(r.meta[0], r.meta[1], r.meta[2], r.meta[3]);
}

// Joins a segment that fell into several shares, in their order: a warp to a row.
template <int DP>
__global__ void __launch_bounds__(128) attend_tiles_join_kernel(const __grid_constant__ KvAttendArgs a) {
  constexpr int kSlot = Tiles<DP>::kSlot, kN = DP / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 meta = a.meta[blockIdx.x];
  const int first = blockIdx.x, last = meta.x;
  if (last < 0) return;
  const Sequence q = attend_sequence(a, meta.y);
  const int lane = threadIdx.x & 31, row0 = meta.w * kATRows, live = min(kATRows, q.n_new * a.G - row0);
  auto slot = [&](int s) { return a.part + (2LL * s + (s == first)) * kSlot; };
  for (int r = blockIdx.y * 4 + (threadIdx.x >> 5); r < live; r += gridDim.y * 4) {
    float most = kLow;
#pragma unroll 4
    for (int s = first; s <= last; ++s) most = fmaxf(most, slot(s)[128 * DP + r]);
    float sum = 0.f, f[kN] = {};
#pragma unroll 4
    for (int s = first; s <= last; ++s) {
      const float* p = slot(s);
      const float by = ex2(p[128 * DP + r] - most);
      sum += p[128 * DP + 128 + r] * by;
#pragma unroll
      for (int k = 0; k < kN; ++k) f[k] += p[r * DP + kN * lane + k] * by;
    }
    if (kN * lane >= a.D) continue;
    const float by = sum == 0.f ? 0.f : 1.f / sum;
    const int token = fdiv(row0 + r, a.div_g);
    uint16_t* out = (uint16_t*)a.out + (((long long)meta.y * a.T + token) * a.Hq + (long long)meta.z * a.G + row0 + r - token * a.G) * a.D +
                    kN * lane;
#pragma unroll
    for (int k = 0; k < kN; k += 2) {
      uint32_t y;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(f[k + 1] * by), "f"(f[k] * by));
      *(uint32_t*)(out + k) = y;
    }
  }
}

template <bool kE4m3, int DP>
static cudaError_t launch_tiles(KvAttendArgs a, int sms, size_t* bytes, cudaStream_t s) {
  using L = Tiles<DP>;
  a.tiles = (int)(((long long)a.T * a.G + kATRows - 1) / kATRows);
  const long long keys = (long long)a.max_code_pages * a.block + (long long)a.max_pages * a.page_size;
  const double most = (double)a.B * a.Hkv * a.tiles * (double)(keys / kATKeys + 2);
  const int grid = (int)fmin((double)sms, most);
  const size_t slots = ((size_t)grid * 2 * L::kSlot * 4 + 255) / 256 * 256;
  if (bytes) {
    *bytes = slots + (size_t)grid * sizeof(int4);
    return cudaSuccess;
  }
  a.meta = (int4*)((char*)a.part + slots);
  auto kernel = attend_tiles_kernel<kE4m3, DP>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kATThreads, L::smem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
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
  return cudaLaunchKernelEx(&cfg, attend_tiles_join_kernel<DP>, a);
}

}  // namespace sv
