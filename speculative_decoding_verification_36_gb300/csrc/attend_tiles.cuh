// attend_tiles.cuh -- attention of a step's tokens to a cache whose older blocks are
// 8-bit codes: many rows a head of keys, on the tensor cores of the SM (tcgen05).
//
// A CTA takes tiles of 128 rows and units of 64 keys:
//   S = Q K^T      128 x 64 x D, both operands in shared memory as fp16
//   P = weights    fp16, over S's columns in tensor memory
//   O += P V       128 x D x 64, P from tensor memory, V from shared memory
// Four warps bring keys and four values: codes go from global memory to registers two
// units ahead, become fp16 (exactly) and are written to shared memory in the 128-byte
// swizzle; plain entries become fp16 times a power of two for each key.  Three warps look the
// entries' places and scales up further ahead.  Four warps make weights of scores: a
// thread has one row, so that rows need no shuffles.  One thread issues the products; S
// is double-buffered, so that the next scores are computed while the weights of the
// last ones are made.  Two CTAs share an SM: what one waits for, the other uses.
//
// The scales never touch the codes: a key's scale multiplies its scores, a value's its
// weight.  With M = m + ref - 138 (m the running maximum in log2, ref exponent bits above every
// scale of V that the row has seen) a weight is 2^(x - M) sv, below 2^15, and the row's sum is
// that of 2^(x - M): the powers of two cancel in the quotient.
#pragma once
#include "attend_common.cuh"
#include "sv_bulk.cuh"

namespace sv {

constexpr int kATRows = 128, kATKeys = 64;
constexpr int kATSoft = 4, kATLoad = 4;                        // warps that make weights; that bring keys, and as many values
constexpr int kATThreads = 32 * (kATSoft + 2 * kATLoad + 4);   // and a group of one that issues and three that look up places
constexpr int kATCtas = 2;                                     // of an SM
// Registers of a thread: 64 at the launch, then by kind (512 * 64 = 128 * 96 + 256 * 56 + 128 * 48).
constexpr int kATSoftRegs = 96, kATLoadRegs = 56, kATIssueRegs = 48;
static_assert(kATCtas * kATThreads * 64 <= 65536 && 32 * kATSoft * kATSoftRegs + 64 * kATLoad * kATLoadRegs + 128 * kATIssueRegs <= kATThreads * 64,
              "registers");
constexpr int kATRing = 8;    // units whose places and scales are held
constexpr int kATLook = 3;    // warps that look them up, by turns: two trips to memory a unit
constexpr unsigned kATLeastRef = 64;  // values below 2^-82 lose bits, which keeps a row's sum below 2^128

// Shared memory; each operand begins on a 1024-byte boundary, as the swizzle wants.
template <int DP>
struct Tiles {
  static constexpr int kTile = kATKeys * DP * 2;    // bytes of a unit's keys or values
  static constexpr int kChunk = kATKeys * 128;      // its rows of 64 fp16
  static constexpr int kQChunk = kATRows * 128;     // the queries'
  static constexpr int kQ = 0, kK = kATRows * DP * 2, kV = kK + 2 * kTile, kRest = kV + 2 * kTile;
  static constexpr int kSlot = 128 * DP + 2 * 128;  // floats that a share leaves
  struct Rest {
    float sk[kATRing][kATKeys], sv[kATRing][kATKeys];
    int at[kATRing][kATKeys];      // a key's entry in its pool, -1: a page outside; the keys of a loading thread side by side
    float qs[kATRows];
    uint32_t bits[kATRows][4];
    int parents[128];
    unsigned long long at_full[kATRing], at_empty[kATRing], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_ready[2], pv_done[2], q_full, drain;
    uint32_t tmem;
    int wrong;
    int meta[4];
  };
  // Keys that eight loading warps take at once, and where a key's place is held.
  static constexpr int kAtOnce = 32 * kATLoad / (DP / 16);
  static __device__ __forceinline__ int place(int key) { return key % kAtOnce * (kATKeys / kAtOnce) + key / kAtOnce; }
  static constexpr size_t smem = kRest + sizeof(Rest) + 1024;
};

// ---- tcgen05 ----
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ bool tc_elect() {
  uint32_t is;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
  return is != 0;
}
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
__device__ __forceinline__ void tc_loaded32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : SV_M8(r, 0), SV_M8(r, 8)::"memory");
  asm volatile("" : SV_M8(r, 16), SV_M8(r, 24));
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
__global__ void __launch_bounds__(kATThreads, kATCtas) attend_tiles_kernel(const __grid_constant__ KvAttendArgs a) {
  using L = Tiles<DP>;
  extern __shared__ unsigned char s_raw[];
  __shared__ unsigned long long s_scan[512 + 1];
  unsigned char* base = s_raw + ((1024u - (smem_addr(s_raw) & 1023u)) & 1023u);
  typename L::Rest& r = *(typename L::Rest*)(base + L::kRest);
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const unsigned tries = mbar_tries(spin_limit());
  constexpr int kIssue = kATSoft + 2 * kATLoad;  // the warp that issues
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
    for (int i = 0; i < kATRing; ++i) {
      mbar_init(&r.at_full[i], 1);
      mbar_init(&r.at_empty[i], 1);
    }
    mbar_init(&r.q_full, kATSoft);
    mbar_init(&r.drain, 1);
    r.wrong = 0;
    r.meta[0] = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssue) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(smem_addr(&r.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  Share w = attend_share<512, kATRows, kATKeys>(a, s_scan);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *(volatile uint32_t*)&r.tmem;
  const uint32_t t_o = tmem + 128;  // S at 0 and 64, O at 128
  // Once a wait has run out the warp goes on without waiting and takes part in every
  // barrier that is left: no warp waits for one that is gone.
  bool dead = false;
  auto wait = [&](unsigned long long* bar, unsigned parity) {
    if (!dead && !warp_wait(bar, parity & 1, tries)) dead = true;
  };

  if (warp < kATSoft) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kATSoftRegs));
    // =====================================================================
    // weights
    // =====================================================================
    const int row = 32 * warp + lane;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    int i = 0;  // units so far
    int loaded_b = -1, loaded_tile = -1;
    bool bad = false;
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
              *(uint2*)(base + L::kQ + (d >> 6) * L::kQChunk + swizzled(q, (d & 63) >> 3) + (d & 4) * 2) = y;
            }
          }
        }
        fence_async();
        bar_sync(5, 32 * kATSoft);  // also: r.qs and the tree's bits
        if (lane == 0) mbar_arrive(&r.q_full);
      }
      const float qs = r.qs[row];
      const bool active = 32 * warp < rows - row0;
      const int last_seen = w.s.len + fdiv(row0 + row, a.div_g), first_seen = w.s.len + fdiv(row0, a.div_g);
      float m = kLow, M = kLow, l = 0.f;
      unsigned ref = kATLeastRef;
      const int n_codes = w.s.bad ? 0 : (keys.codes + kATKeys - 1) / kATKeys;
      for (int u = u0; u < u1; ++u, ++i) {
        const int s = i & 1;
        wait(&r.s_full[s], i >> 1);
        tc_after();
        if (active && !w.s.bad) {
          const float *sk = r.sk[i & (kATRing - 1)], *sv = r.sv[i & (kATRing - 1)];
          const uint32_t t_s = tmem + 64 * s + lanes;
          const bool codes = u < n_codes;
          if (!codes) wait(&r.v_full[s], i >> 1);  // the plain values' scales
          const int unit = codes ? u * kATKeys : keys.stored + (u - n_codes) * kATKeys, end = codes ? keys.codes : keys.end;
          const bool masked = unit + kATKeys > end || (a.parents ? unit + kATKeys > w.s.len : unit + kATKeys - 1 > first_seen);
          const bool groups = codes && !masked && a.block % 16 == 0;  // 16 keys in a row share their scales
          // of 32 keys, those that the row sees
          auto seen = [&](int c) {
            if (!masked) return 0xffffffffu;
            const int f = unit + 32 * c, behind = min(end - f, a.parents ? 32 : last_seen - f + 1);
            uint32_t vis = behind <= 0 ? 0u : behind >= 32 ? 0xffffffffu : (1u << behind) - 1u;
            if (a.parents) {
              const int at = f - w.s.len;  // the first key as a token of the step
              if (at > -32) {
                const int word = at >> 5;  // -1 .. 3
                const uint32_t lo = word < 0 ? 0xffffffffu : word < 4 ? r.bits[row][word] : 0u;
                const uint32_t hi = word + 1 < 4 ? r.bits[row][word + 1] : 0u;
                vis &= __funnelshift_r(lo, hi, at & 31);
              }
            }
            return vis;
          };
          // Twice over the row's 64 scores, 32 in registers at a time (those that came last
          // stay): the maximum, then the weights.
          uint32_t x[32];
          float most = -INFINITY;
          unsigned top = kATLeastRef;
          auto exponent = [&](float v) {
            const unsigned b = __float_as_uint(v);
            return b < 0x7f800000u ? (b >> 23) + 1u : 0u;  // one that is not finite makes its weights NaN whatever the reference
          };
#pragma unroll
          for (int c = 1; c >= 0; --c) {
            tc_load32(t_s + 32 * c, x);
            tc_loaded32(x);
            if (groups) {
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                float y = __uint_as_float(x[16 * g]);
#pragma unroll
                for (int k = 1; k < 16; ++k) y = fmaxf(y, __uint_as_float(x[16 * g + k]));
                most = fmaxf(most, y * sk[32 * c + 16 * g]);
                top = max(top, exponent(sv[32 * c + 16 * g]));
              }
            } else {
              const uint32_t vis = seen(c);
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const float4 y = *(const float4*)(sk + 32 * c + k), v = *(const float4*)(sv + 32 * c + k);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (vis >> (k + e) & 1u) {
                    most = fmaxf(most, __uint_as_float(x[k + e]) * (e == 0 ? y.x : e == 1 ? y.y : e == 2 ? y.z : y.w));
                    top = max(top, exponent(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w));
                  }
              }
            }
          }
          most *= qs;  // (a scale of 0: -inf becomes NaN, which no maximum takes)
          top = min(top, 254u);
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
              for (int c = 0; c < DP; c += 16) {
                uint32_t o[16];
                const uint32_t at = t_o + lanes + c;
                tc_load16(at, o);
                tc_loaded16(o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tc_store16(at, o);
              }
            }
          }
          f2_t sum = 0;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (c == 1) {
              tc_load32(t_s + 32, x);
              tc_loaded32(x);
            }
            uint32_t p[16];
            if (groups) {
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                const float by = sk[32 * c + 16 * g] * qs, v = sv[32 * c + 16 * g];
                const f2_t by2 = f2(by, by), v2 = f2(v, v), less = f2(-M, -M);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const f2_t y = f2fma(f2(__uint_as_float(x[16 * g + 2 * k]), __uint_as_float(x[16 * g + 2 * k + 1])), by2, less);
                  const f2_t e = f2(ex2(f2lo(y)), ex2(f2hi(y)));
                  sum = f2add(sum, e);
                  const f2_t z = f2mul(e, v2);
                  p[8 * g + k] = half2_of(f2lo(z), f2hi(z));
                }
              }
            } else {
              const uint32_t vis = seen(c);
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const float4 y = *(const float4*)(sk + 32 * c + k), v = *(const float4*)(sv + 32 * c + k);
                float z[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float by = (e == 0 ? y.x : e == 1 ? y.y : e == 2 ? y.z : y.w) * qs;
                  // what is not seen has no part, whatever its scales are
                  const bool see = vis >> (k + e) & 1u;
                  const float q = see ? ex2(fmaf(__uint_as_float(x[k + e]), by, -M)) : 0.f;
                  l += q;
                  z[e] = see ? q * (e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w) : 0.f;
                }
                p[k / 2] = half2_of(z[0], z[1]);
                p[k / 2 + 1] = half2_of(z[2], z[3]);
              }
            }
            tc_store16(t_s + 16 * c, p);
          }
          l += f2lo(sum) + f2hi(sum);
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
        const bool whole = u0 == 0 && u1 == n, mine = row0 + row < rows;
        const float by = l == 0.f ? 0.f : 1.f / l;
        const int token = fdiv(row0 + row, a.div_g);
        uint16_t* out = (uint16_t*)a.out + (((long long)w.b * a.T + token) * a.Hq + (long long)w.h * a.G + row0 + row - token * a.G) * a.D;
        float* part = a.part + (2LL * blockIdx.x + (u0 == 0)) * L::kSlot;
#pragma unroll 1
        for (int c = 0; c < DP; c += 16) {
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
        if (!whole && mine) part[128 * DP + row] = M, part[128 * DP + 128 + row] = l;
      }
      tc_before();
      if (u0 == 0 && u1 < n && threadIdx.x == 0) {
        r.meta[0] = attend_share_of(w, w.from + n - 1);
        r.meta[1] = w.b, r.meta[2] = w.h, r.meta[3] = w.tile;
      }
      attend_advance<kATRows, kATKeys>(a, w, u1 - u0);
    }
  } else if (warp < kIssue) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kATLoadRegs));
    // =====================================================================
    // keys and values
    // =====================================================================
    const bool values = warp >= kATSoft + kATLoad;
    const int wx = warp - (values ? kATSoft + kATLoad : kATSoft), x = 32 * wx + lane;
    // Eight lanes in a row write four units of two keys, which the swizzle puts on all
    // banks; a warp reads whole heads.
    constexpr int kPer = DP / 16, kAtOnce = L::kAtOnce, kRounds = kATKeys / kAtOnce;  // lanes a key, keys at once
    const int part = (lane & 3) | (kPer == 8 ? (lane >> 1) & 4 : 0);
    const int mine = wx * (32 / kPer) + (((lane >> 2) & 1) | (kPer == 8 ? (lane >> 3) & 2 : (lane >> 2) & 6));
    const bool on = 16 * part < a.D;
    const long long entry = (long long)a.Hkv * a.D;
    unsigned char* operand = base + (values ? L::kV : L::kK);
    unsigned long long *is_full = values ? r.v_full : r.k_full, *is_empty = values ? r.v_empty : r.k_empty;
    const int put0 = (part >> 2) * L::kChunk + swizzled(mine, 2 * (part & 3)), put1 = (part >> 2) * L::kChunk + swizzled(mine, 2 * (part & 3) + 1);
    int i = 0;
    auto wait_empty = [&]() {  // the operand of two units ago has been read
      if (i >= 2) wait(&is_empty[i & 1], (i >> 1) + 1);
    };
    auto full = [&]() {
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&is_full[i & 1]);
    };
    while (w.left > 0) {
      const int n = attend_units<kATRows, kATKeys>(a, w.s, w.tile);
      const int u0 = w.u, u1 = (int)min((long long)n, u0 + w.left);
      const Keys keys = attend_keys<kATRows>(a, w.s, w.tile);
      const int n_codes = w.s.bad ? 0 : (keys.codes + kATKeys - 1) / kATKeys, uc = min(u1, n_codes);
      if (u0 < uc) {
        const uint8_t* from = (values ? a.v_codes : a.k_codes) + (long long)w.h * a.D + 16 * part;
        uint4 c[2][kRounds];
        auto load = [&](int j, int b) {  // unit j of the CTA's
          wait(&r.at_full[j & (kATRing - 1)], j / kATRing);
          const int* p = &r.at[j & (kATRing - 1)][mine * kRounds];
          int at[kRounds];
          if constexpr (kRounds == 4) {
            const int4 v = *(const int4*)p;
            at[0] = v.x, at[1] = v.y, at[2] = v.z, at[3] = v.w;
          } else {
            const int2 v = *(const int2*)p;
            at[0] = v.x, at[1] = v.y;
          }
#pragma unroll
          for (int q = 0; q < kRounds; ++q) c[b][q] = on ? stream16(from + max(at[q], 0) * entry) : make_uint4(0, 0, 0, 0);
        };
        load(i, 0);
        if (u0 + 1 < uc) load(i + 1, 1);
        for (int u = u0; u < uc; u += 2) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            if (u + b >= uc) break;
            wait_empty();
            unsigned char* to = operand + (i & 1) * L::kTile;
            if (on) {
#pragma unroll
              for (int q = 0; q < kRounds; ++q) {
                uint4 z[2];
                Code<kE4m3>::word(c[b][q].x, z[0].x, z[0].y);
                Code<kE4m3>::word(c[b][q].y, z[0].z, z[0].w);
                Code<kE4m3>::word(c[b][q].z, z[1].x, z[1].y);
                Code<kE4m3>::word(c[b][q].w, z[1].z, z[1].w);
                *(uint4*)(to + put0 + q * kAtOnce * 128) = z[0];
                *(uint4*)(to + put1 + q * kAtOnce * 128) = z[1];
              }
            }
            full();
            if (u + b + 2 < uc) load(i + 2, b);
            ++i;
          }
        }
      }
      // plain entries: twice as many lanes a key, eight values each
      for (int u = max(u0, uc); u < u1; ++u) {
        constexpr int kPer2 = DP / 8, kAtOnce2 = 32 * kATLoad / kPer2, kRounds2 = kATKeys / kAtOnce2, kBatch = 4;
        const int part2 = x % kPer2, mine2 = x / kPer2;
        const bool on2 = 8 * part2 < a.D;
        wait_empty();
        if (!w.s.bad) {
          wait(&r.at_full[i & (kATRing - 1)], i / kATRing);
          const uint16_t* from = (const uint16_t*)(values ? a.v_cache : a.k_cache) + w.h * a.D + 8 * part2;
          unsigned char* to = operand + (i & 1) * L::kTile + (part2 >> 3) * L::kChunk;
          float* scales = (values ? r.sv : r.sk)[i & (kATRing - 1)];
#pragma unroll 1
          for (int q0 = 0; q0 < kRounds2; q0 += kBatch) {
            uint4 y[kBatch];
            bool ok[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
              const int row = mine2 + (q0 + q) * kAtOnce2, at = r.at[i & (kATRing - 1)][L::place(row)];
              ok[q] = at >= 0;
              y[q] = on2 && ok[q] ? *(const uint4*)(from + at * entry) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
              const int row = mine2 + (q0 + q) * kAtOnce2;
              const unsigned lo = max(max(y[q].x & 0x7fffu, y[q].y & 0x7fffu), max(y[q].z & 0x7fffu, y[q].w & 0x7fffu));
              const unsigned hi = max(max(y[q].x & 0x7fff0000u, y[q].y & 0x7fff0000u), max(y[q].z & 0x7fff0000u, y[q].w & 0x7fff0000u));
              unsigned top = max(lo << 16, hi);
#pragma unroll
              for (int d = 1; d < kPer2; d *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
              const bool finite = top < 0x7f800000u;
              const float up = finite ? scale_up(top) : 0.f;
              if (part2 == 0) scales[row] = ok[q] && finite ? scale_down(top) : __uint_as_float(0x7fffffffu);
              uint4 z = make_uint4(0, 0, 0, 0);
              if (finite)
                z = make_uint4(half2_of(bf16_lo(y[q].x) * up, bf16_hi(y[q].x) * up), half2_of(bf16_lo(y[q].y) * up, bf16_hi(y[q].y) * up),
                               half2_of(bf16_lo(y[q].z) * up, bf16_hi(y[q].z) * up), half2_of(bf16_lo(y[q].w) * up, bf16_hi(y[q].w) * up));
              if (on2) *(uint4*)(to + swizzled(row, part2 & 7)) = z;
            }
          }
        }
        full();
        ++i;
      }
      attend_advance<kATRows, kATKeys>(a, w, u1 - u0);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kATIssueRegs));
    if (warp == kIssue) {
      // ===================================================================
      // products
      // ===================================================================
      // The warp walks along together and its elected lane issues: what the products take is
      // then known to be the same in all lanes (an issue under `lane == 0` took 100 clocks,
      // 64 being the product's own time).
      const bool leader = tc_elect();
      const unsigned long long d_q = tc_operand(smem_addr(base + L::kQ), 16), d_k = tc_operand(smem_addr(base + L::kK), 16);
      const unsigned long long d_v = tc_operand(smem_addr(base + L::kV), L::kChunk);
      const uint32_t kind_s = tc_kind(kATKeys, false), kind_o = tc_kind(a.D, true);
      const int steps = a.D / 16;
      int i = 0, segments = 0;
      bool open = false;   // unit i - 1 has no P V yet
      bool fresh = false;  // ... and begins its segment
      auto pv = [&]() {    // of unit i - 1
        const int j = i - 1, s = j & 1;
        wait(&r.p_ready[s], j >> 1);
        wait(&r.v_full[s], j >> 1);
        tc_after();
        if (leader && !dead) {
          const unsigned long long d = d_v + s * (L::kTile >> 4);
          const bool add = !fresh;
#pragma unroll
          for (int k = 0; k < kATKeys / 16; ++k) tc_mma_t(t_o, tmem + 64 * s + 8 * k, d + k * (2048 >> 4), kind_o, k > 0 || add);
          tc_commit(&r.v_empty[s]);
          tc_commit(&r.pv_done[s]);
          tc_commit(&r.at_empty[j & (kATRing - 1)]);  // its places and scales have been used
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
          if (leader && !dead) {
            const unsigned long long d = d_k + s * (L::kTile >> 4);
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
              if (k < steps)
                tc_mma(tmem + 64 * s, d_q + (((k >> 2) * L::kQChunk + (k & 3) * 32) >> 4), d + (((k >> 2) * L::kChunk + (k & 3) * 32) >> 4), kind_s,
                       k > 0);
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
      if (leader) tc_commit(&r.drain);
      __syncwarp();
      if (!warp_wait(&r.drain, 0, mbar_tries(kSpinLimit))) dead = true;
    } else {
      // ===================================================================
      // places and scales: this warp's units
      // ===================================================================
      int i = 0, turn = warp - kIssue - 1;  // units so far; until this warp's next one
      while (w.left > 0) {
        const int n = attend_units<kATRows, kATKeys>(a, w.s, w.tile);
        const int u0 = w.u, u1 = (int)min((long long)n, u0 + w.left);
        const Keys keys = attend_keys<kATRows>(a, w.s, w.tile);
        const int n_codes = w.s.bad ? 0 : (keys.codes + kATKeys - 1) / kATKeys;
        for (int u = u0; u < u1; ++u, ++i) {
          if (turn-- != 0) continue;
          turn = kATLook - 1;
          const int slot = i & (kATRing - 1);
          const bool codes = u < n_codes;
          constexpr int kQ = kATKeys / 32;
          int at[kQ], page[kQ];
          if (!w.s.bad) {
#pragma unroll
            for (int q = 0; q < kQ; ++q) {  // (keys past the end stand for the last one: they are read and not seen)
              const int k = 32 * q + lane;
              const int key = codes ? min(u * kATKeys + k, keys.codes - 1) : min(keys.stored + (u - n_codes) * kATKeys + k, keys.end - 1);
              const int p = fdiv(key, codes ? a.div_block : a.div_page);
              at[q] = key - p * (codes ? a.block : a.page_size);
              page[q] = codes ? __ldg(a.code_table + (long long)w.b * a.max_code_pages + p) : __ldg(a.page_table + (long long)w.b * a.max_pages + p);
            }
          }
          if (i >= kATRing) wait(&r.at_empty[slot], i / kATRing + 1);
          if (!w.s.bad) {
            float sk[kQ], sv[kQ];
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
              const bool ok = page[q] >= 0 && page[q] < (codes ? a.code_pages : a.pages);
              if (!ok) atomicOr(a.status, kStatusBadData);
              at[q] = ok ? page[q] * (codes ? a.block : a.page_size) + at[q] : -1;
              sk[q] = sv[q] = __uint_as_float(0x7fffffffu);
              if (codes && ok) {
                sk[q] = __ldg(a.k_scales + (long long)page[q] * a.Hkv + w.h);
                sv[q] = __ldg(a.v_scales + (long long)page[q] * a.Hkv + w.h);
              }
            }
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
              const int k = 32 * q + lane;
              r.at[slot][L::place(k)] = at[q];
              if (codes) r.sk[slot][k] = sk[q], r.sv[slot][k] = sv[q];
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&r.at_full[slot]);
        }
        attend_advance<kATRows, kATKeys>(a, w, u1 - u0);
      }
    }
  }
  if (dead && lane == 0) atomicOr(a.status, kStatusTimeout);
  tc_before();
  __syncthreads();
  if (warp == kIssue) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem) : "memory");
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
  const int grid = (int)fmin((double)sms * kATCtas, most);
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
