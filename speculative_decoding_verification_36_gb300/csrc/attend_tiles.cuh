// attend_tiles.cuh -- attention of a step's tokens to a cache whose older blocks are
// 8-bit codes: many rows a head of keys, on the tensor cores of the SM (tcgen05).
//
// A CTA takes tiles of 128 rows and units of 64 keys:
//   S = Q K^T      128 x 64 x D, Q from tensor memory, K from shared memory, both fp16
//   P = weights    fp16, over S's columns in tensor memory (as attend_rows.cuh says, the rounding does
//                  not show in a bf16 result)
//   O += P V       128 x D x 64, P from tensor memory, V from shared memory
// Four warps bring keys and four values: codes go from global memory to registers a
// unit ahead (two ahead: chains 306 us instead of 266, prompts 1096 instead of 845; two warps for
// each: chains 253, prompts 915), become fp16 (exactly) and are written to shared memory
// in the 128-byte swizzle; plain entries become fp16 times a power of two for each key.  Three warps look the
// entries' places and scales up further ahead.  Four warps make weights of scores: a
// thread has one row, so that rows need no shuffles.  One thread issues the products.
// Two CTAs share an SM (heads of more than 128: one, which has all the tensor memory): while one
// waits for its weights, the other's products run.  They share shared memory's bandwidth: 512
// bytes a key and head of 128 written, 512 read.
//
// Measured (GB300, 32 heads to 8 of keys of 128; the floor by bytes, or by products at 1.95
// PFLOP/s, beside it): chains of 9, 64 sequences of 4096 to 8192 entries, int8: 266 us (123);
// trees of 31 tokens, 32 such sequences, e4m3: 171 us (65); 5 tokens, two sequences of 131072 to
// 262144, e4m3: 159 us (81); prompts of up to 2048 tokens behind 16384, int8: 846 us (298); three
// tokens with 8 heads to one of 256, 16 sequences of 5000 to 10000: 46 us (9.4).
// A unit takes a CTA 2000 to 3300 clocks.  800 to 1000 are its products (chains: the tensor pipe is busy
// in 35 % of the clocks).  Its weights took 1200 to 1600 when last counted (with two units ahead, and a
// reference by scales alone), 450 with nothing else on the SM: the two CTAs' 32
// warps issue in half of all clocks, so a warp waits for its turn at each step, and S, weights and
// P V follow on one another.  A segment cost a CTA 15 000 to 20 000 clocks at its ends, most of
// them for its queries.
// Steps before: units of 128 keys with one CTA an SM 440 us (chains), queries in shared
// memory 203 (trees), three stages or spilled registers slower (L1 is small beside this much
// shared memory); tiles of up to 64 rows taken twice or four times, each copy with its part of the keys:
// no faster (chains 380 of 380), the weights' own instructions are not what is waited for.
// A check for each unit in the loading warps costs a tenth.
//
// The scales never touch the codes: a key's scale multiplies its scores, a value's its
// weight.  With m the running maximum (log2) a weight is 2^(x - m) sv 2^-unit, below 2^15, where
// 2^unit follows the largest 2^(x - m) sv that the row has seen: a key with large values and
// little weight takes no bits from the others.  The row's sum is that of 2^(x - m) alone, so that no
// size of the values rescales it.
#pragma once
#include "attend_common.cuh"
#include "sv_bulk.cuh"

namespace sv {

constexpr int kATRows = 128, kATKeys = 64;
constexpr int kATSoft = 4, kATLoad = 4;                        // warps that make weights; that bring keys, and as many values
constexpr int kATThreads = 32 * (kATSoft + 2 * kATLoad + 4);   // and a group of one that issues and three that look up places
// Registers of a thread with two CTAs an SM: 64 at the launch, then by kind (512 * 64 = 128 * 88 + 256 * 56 + 128 * 56).
constexpr int kATSoftRegs = 88, kATLoadRegs = 56, kATIssueRegs = 56;
static_assert(2 * kATThreads * 64 <= 65536 && 32 * kATSoft * kATSoftRegs + 64 * kATLoad * kATLoadRegs + 128 * kATIssueRegs <= kATThreads * 64,
              "registers");
constexpr int kATStages = 2;  // units whose keys and values are in shared memory
constexpr int kATRing = 8;    // units whose places and scales are held
constexpr int kATCodes = 0, kATPlain = 1, kATNone = 2;  // kinds of units (log2 of a value's bytes); the last: a bad sequence's, or one without pages
// Units whose products are added up in tensor memory.  The products' sums drop bits, up to 2^-23 of the sum for each 16
// keys, always downwards: 2^-12 in as many units.  (Without an end to it 262144 keys in one CTA came out
// 0.1 to 0.2 % small.)  Longer runs are taken in pieces and added up in the workspace, in fp32.
constexpr int kATPiece = 512;
constexpr int kATLook = 3;    // warps that look them up, by turns: two trips to memory a unit

// A CTA's waits.  Once one has run out all warps go on without waiting and take part in every
// barrier that is left: no warp waits for one that is gone.
struct Waits {
  volatile unsigned tries;  // of a wait after its first look, 0 once one has run out
  volatile unsigned out;    // one has
};
__device__ __forceinline__ void bounded_wait(Waits& w, unsigned long long* bar, unsigned parity) {
  if (__all_sync(0xffffffffu, mbar_test(bar, parity & 1))) return;
  for (unsigned n = __reduce_min_sync(0xffffffffu, w.tries); n > 0; --n)
    if (__all_sync(0xffffffffu, mbar_try(bar, parity & 1))) return;
  w.tries = 0;
  w.out = 1;
}

// Shared memory; each operand begins on a 1024-byte boundary, as the swizzle wants.
template <int DP>
struct Tiles {
  static constexpr int kTile = kATKeys * DP * 2;    // bytes of a unit's keys or values
  static constexpr int kCtas = DP == 256 ? 1 : 2;   // of an SM
  // Columns of tensor memory: S and its weights from 0 on, the queries from 64 on, then O.
  static constexpr int kColumns = 512 / kCtas, kO = kColumns / 2;
  static constexpr int kChunk = kATKeys * 128;      // its rows of 64 fp16
  static constexpr int kK = 0, kV = kATStages * kTile, kRest = 2 * kATStages * kTile;
  struct Rest {
    float sk[kATRing][kATKeys], sv[kATRing][kATKeys], above[kATRing][kATKeys];  // above: log_above(sv)
    int kind[kATRing];
    // where a key's head lies in the pool of codes and in that of plain entries, in 16 bytes (0: a page
    // outside, or none yet); the keys of a loading thread side by side
    unsigned at[2][kATRing][kATKeys];
    unsigned outside[kATRing][kATKeys / 32];  // keys whose page is outside, as bits
    float top[kATRing];            // exponent bits above a unit's scales of V
    uint32_t bits[kATRows][4];
    int parents[128];
    unsigned long long at_full[kATRing], at_empty[kATRing], k_full[kATStages], k_empty[kATStages], v_full[kATStages],
        v_empty[kATStages], s_full, p_ready, pv_done, q_full, drain;
    uint32_t tmem;
    int wrong;
    Waits waits;
    int meta[4];
    int live;  // rows of the segment
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
// D = A B (+ D), A in tensor memory
__device__ __forceinline__ void tc_mma_t(uint32_t d, uint32_t a, unsigned long long b, uint32_t kind, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
      : "memory");
}
#define SV_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define SV_W8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
// 16 columns of the warp's 32 lanes (a register a column)
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
__device__ __forceinline__ void tc_store8(uint32_t at, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::SV_W8(r, 0), "r"(at) : "memory");
}
__device__ __forceinline__ void tc_store1(uint32_t at, uint32_t x) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%1], {%0};" ::"r"(x), "r"(at) : "memory");
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
__global__ void __launch_bounds__(kATThreads, DP == 256 ? 1 : 2) attend_tiles_kernel(const __grid_constant__ KvAttendArgs a) {
  using L = Tiles<DP>;
  extern __shared__ unsigned char s_raw[];
  __shared__ unsigned long long s_scan[512 + 1];
  unsigned char* base = s_raw + ((1024u - (smem_addr(s_raw) & 1023u)) & 1023u);
  typename L::Rest& r = *(typename L::Rest*)(base + L::kRest);
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  constexpr int kIssue = kATSoft + 2 * kATLoad;  // the warp that issues
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int i = 0; i < kATStages; ++i) {
      mbar_init(&r.k_full[i], kATLoad);
      mbar_init(&r.v_full[i], kATLoad);
      mbar_init(&r.k_empty[i], 1);
      mbar_init(&r.v_empty[i], 1);
    }
    mbar_init(&r.s_full, 2);
    mbar_init(&r.pv_done, 1);
    mbar_init(&r.p_ready, kATSoft);
    for (int i = 0; i < kATRing; ++i) {
      mbar_init(&r.at_full[i], 1);
      mbar_init(&r.at_empty[i], 1);
    }
    mbar_init(&r.q_full, kATSoft);
    mbar_init(&r.drain, 1);
    r.wrong = 0;
    r.waits.tries = mbar_tries(spin_limit());
    r.waits.out = 0;
    r.meta[0] = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssue) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&r.tmem)), "n"(L::kColumns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  for (int i = threadIdx.x; i < 2 * kATRing * kATKeys; i += kATThreads) (&r.at[0][0][0])[i] = 0;
  if (threadIdx.x < kATRing) r.kind[threadIdx.x] = kATNone;
  for (int i = threadIdx.x; i < kATStages * L::kTile / 16; i += kATThreads) ((uint4*)(base + L::kV))[i] = make_uint4(0, 0, 0, 0);
  fence_async();
  Share w = attend_share<512, kATRows, kATKeys>(a, s_scan);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *(volatile uint32_t*)&r.tmem;
  const uint32_t t_q = tmem + 64, t_o = tmem + L::kO;  // S, then its weights, at 0
  // After a wait that ran out, what the warps read may be another unit's, and the places in shared
  // memory are at any time ones inside their pools.
  auto wait = [&](unsigned long long* bar, unsigned parity) { bounded_wait(r.waits, bar, parity); };

  if (warp < kATSoft) {
    if constexpr (L::kCtas == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kATSoftRegs));
    // =====================================================================
    // weights
    // =====================================================================
    const int row = 32 * warp + lane;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    int i = 0;     // units so far
    int done = 0;  // of the share's units of the segment
    int loaded_b = -1, loaded_tile = -1;
    bool bad = false;
    while (w.left > 0) {
      const int n = attend_units<kATRows, kATKeys>(a, w.s, w.tile), last = (int)min((long long)n, w.u + w.left);
      const int u0 = w.u + done, u1 = min(last, u0 + kATPiece);
      const Keys keys = attend_keys<kATRows>(a, w.s, w.tile);
      const int row0 = w.tile * kATRows, rows = w.s.n_new * a.G;
      // ---- queries to shared memory: all scores of the last piece are there ----
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
          if (token < a.T) attend_bits(r.parents, token, 4, r.bits[threadIdx.x]);  // (its own row's)
        }
      }
      loaded_b = w.b, loaded_tile = w.tile;
      if (threadIdx.x == 0) r.live = min(kATRows, rows - row0);
      const bool lost = w.s.bad || (a.parents && bad);
      if (lost && threadIdx.x == 0) atomicOr(a.status, kStatusBadData);
      const bool active = 32 * warp < rows - row0, mine = row0 + row < rows;
      float qs = __uint_as_float(0x7fffffffu);
      if (active) {
        // A thread has its row, and lays it down in tensor memory: the products read it from there,
        // which leaves shared memory to the keys and values.
        const int token = fdiv(row0 + row, a.div_g);
        const uint16_t* q = (const uint16_t*)a.q + ((long long)w.b * a.T + token) * a.q_stride + ((long long)w.h * a.G + row0 + row - token * a.G) * a.D;
        const bool fast = ((uintptr_t)a.q & 15) == 0 && a.q_stride % 8 == 0, there = mine && !lost;
        auto eight = [&](int d) { return there && d < a.D ? __ldg((const uint4*)(q + d)) : make_uint4(0, 0, 0, 0); };
        // once from memory (the first trip brings the whole row to L2), then from tensor memory
        if (there)
          for (int d = 0; d < a.D; d += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + d));
        unsigned lo = 0, hi = 0;
        if (fast) {
#pragma unroll 2
          for (int d = 0; d < DP; d += 32) {
            uint4 x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = eight(d + 8 * e);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              lo = max(lo, max(max(x[e].x & 0x7fffu, x[e].y & 0x7fffu), max(x[e].z & 0x7fffu, x[e].w & 0x7fffu)));
              hi = max(hi, max(max(x[e].x & 0x7fff0000u, x[e].y & 0x7fff0000u), max(x[e].z & 0x7fff0000u, x[e].w & 0x7fff0000u)));
            }
            tc_store16(t_q + lanes + d / 2, (const uint32_t*)x);
          }
        } else {
#pragma unroll 1
          for (int d = 0; d < DP; d += 2) {
            const uint32_t x = there && d < a.D ? q[d] | (uint32_t)q[d + 1] << 16 : 0u;
            lo = max(lo, x & 0x7fffu), hi = max(hi, x & 0x7fff0000u);
            tc_store1(t_q + lanes + d / 2, x);
          }
        }
        tc_stored();
        const unsigned top = max(lo << 16, hi);
        const bool finite = top < 0x7f800000u;
        // the scale's sign goes with the query: what multiplies the scores is positive
        const float up = a.scale < 0.f ? -scale_up(top) : scale_up(top);
        if (!lost && finite) qs = scale_down(top) * fabsf(a.scale);
        auto two = [&](uint32_t v) { return finite ? half2_of(bf16_lo(v) * up, bf16_hi(v) * up) : 0u; };
#pragma unroll 1
        for (int d = 0; d < DP; d += 32) {
          uint32_t y[16];
          tc_load16(t_q + lanes + d / 2, y);
          tc_loaded16(y);
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = two(y[e]);
          tc_store16(t_q + lanes + d / 2, y);
        }
        tc_stored();
      }
      tc_before();
      bar_sync(5, 32 * kATSoft);  // no warp is more than a piece ahead
      if (lane == 0) mbar_arrive(&r.q_full);
      const int last_seen = w.s.len + fdiv(row0 + row, a.div_g), first_seen = w.s.len + fdiv(row0, a.div_g);
      float m = kLow, high = kLow, l = 0.f, over = 1.f;  // high: the largest x + log_above(sv)
      float room = 142.f;  // 15 + unit + 127: how far a score with its scale's exponent bits may be above the maximum, for weights below 2^15
      int unit = 0;        // over = 2^-unit
      const int n_codes = w.s.bad ? 0 : (keys.codes + kATKeys - 1) / kATKeys;
      // units of codes that every row sees whole and whose keys share their scales by 16
      const int u_groups = w.s.bad || a.block % 16 ? 0 : min(keys.codes, a.parents ? w.s.len : first_seen + 1) / kATKeys;
      // warps without rows stay away: the first arrives for them
      const unsigned arrivals = warp ? 1u : 1u + kATSoft - min(kATSoft, (rows - row0 + 31) / 32);
      if (!active) i += u1 - u0;
      for (int u = active ? u0 : u1; u < u1; ++u, ++i) {
        wait(&r.s_full, i);
        tc_after();
        if (!w.s.bad) {
          const int slot = i & (kATRing - 1);
          const float *sk = r.sk[slot], *sv = r.sv[slot], *above = r.above[slot];
          const uint32_t t_s = tmem + lanes;
          // the maximum and the unit move, and with them the sums: to scores up to `most` and weighted scales up to `weighted` (log2)
          auto move = [&](float most, float weighted) {
            const float m2 = fmaxf(m, most), by = ex2(m - m2);
            high = fmaxf(high, weighted);
            const int unit2 = attend_weight_unit(high, m2);
            const float f = by * two_to(unit - unit2);
            m = m2, unit = unit2, over = two_to(-unit), room = (float)(142 + unit);
            l *= by;
            if (u > u0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
              for (int c = 0; c < DP; c += 16) {  // (no product is under way: the scores came after the last one)
                uint32_t o[16];
                const uint32_t at = t_o + lanes + c;
                tc_load16(at, o);
                tc_loaded16(o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tc_store16(at, o);
              }
            }
          };
          bool grouped = u < u_groups;
          if (grouped) {
            const float top = r.top[slot];
            // Scores to weights under the maximum as it is; where one of the warp's rows may have
            // outgrown it, it moves and the scores, which are still there, are taken again.
            uint32_t p[32];
            f2_t sum0, sum1;
            for (bool again = false;; again = true) {
              uint32_t x[2][16];  // the next 16 come while these are taken
              tc_load16(t_s, x[0]);
              float most0 = -INFINITY, most1 = -INFINITY;  // of the exponents
              sum0 = sum1 = 0;
              const f2_t less = f2(-m, -m);
              tc_loaded16(x[0]);
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                if (g < 3) tc_load16(t_s + 16 * (g + 1), x[(g + 1) & 1]);
                const float b = sk[16 * g] * qs, v = sv[16 * g] * over;
                const f2_t by = f2(b, b), of = f2(v, v);
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                  const uint32_t(&z)[16] = x[g & 1];
                  const f2_t y0 = f2fma(f2(__uint_as_float(z[k]), __uint_as_float(z[k + 1])), by, less);
                  const f2_t y1 = f2fma(f2(__uint_as_float(z[k + 2]), __uint_as_float(z[k + 3])), by, less);
                  most0 = fmaxf(most0, fmaxf(f2lo(y0), f2hi(y0)));
                  most1 = fmaxf(most1, fmaxf(f2lo(y1), f2hi(y1)));
                  const f2_t e0 = f2(ex2(f2lo(y0)), ex2(f2hi(y0))), e1 = f2(ex2(f2lo(y1)), ex2(f2hi(y1)));
                  sum0 = f2add(sum0, e0);
                  sum1 = f2add(sum1, e1);
                  const f2_t z0 = f2mul(e0, of), z1 = f2mul(e1, of);
                  p[8 * g + k / 2] = half2_of(f2lo(z0), f2hi(z0));
                  p[8 * g + k / 2 + 1] = half2_of(f2lo(z1), f2hi(z1));
                }
                if (g < 3) tc_loaded16(x[(g + 1) & 1]);
              }
              // (rows past the last hold anything; a score that is infinite outgrows every maximum)
              const float lim = fminf(kSlack, room - top);  // where the largest score and the largest scale are one key's
              if (!__any_sync(0xffffffffu, mine && (fmaxf(most0, most1) > lim || lim < -96.f))) break;
              if (again) {
                grouped = !__any_sync(0xffffffffu, mine && lim < -96.f);  // sv over may not be finite
                break;
              }
              float most = -INFINITY, weighted = -INFINITY;
#pragma unroll 1
              for (int g = 0; g < 4; ++g) {
                uint32_t z[16];
                tc_load16(t_s + 16 * g, z);
                tc_loaded16(z);
                float y = __uint_as_float(z[0]);
#pragma unroll
                for (int k = 1; k < 16; ++k) y = fmaxf(y, __uint_as_float(z[k]));
                y *= sk[16 * g] * qs;  // (a maximum takes no NaN)
                most = fmaxf(most, y);
                weighted = fmaxf(weighted, y + above[16 * g]);
              }
              move(most, weighted);
            }
            if (grouped) {
              sum0 = f2add(sum0, sum1);
              l += f2lo(sum0) + f2hi(sum0);
              tc_store16(t_s, p);
              tc_store16(t_s + 16, p + 16);
            }
          }
          if (!grouped) {
            // A scale for each key, and keys that some rows do not see: twice over the scores, 16
            // at a time.  What is not seen has no part, whatever its scales are.
            const bool codes = u < n_codes;
            if (!codes) wait(&r.v_full[i % kATStages], i / kATStages);  // the plain values' scales
            const int unit = codes ? u * kATKeys : keys.stored + (u - n_codes) * kATKeys, end = codes ? keys.codes : keys.end;
            const bool masked = unit + kATKeys > end || (a.parents ? unit + kATKeys > w.s.len : unit + kATKeys - 1 > first_seen);
            // of 32 keys, those that the row sees
            auto seen = [&](int f) {
              if (!masked) return 0xffffffffu;
              const int behind = min(end - f, a.parents ? 32 : last_seen - f + 1);
              uint32_t vis = behind <= 0 ? 0u : behind >= 32 ? 0xffffffffu : (1u << behind) - 1u;
              const int at = f - w.s.len;  // the first key as a token of the step
              if (a.parents && at > -32) {
                const int word = at >> 5;  // -1 .. 3
                const uint32_t lo = word < 0 ? 0xffffffffu : word < 4 ? r.bits[row][word] : 0u;
                const uint32_t hi = word + 1 < 4 ? r.bits[row][word + 1] : 0u;
                vis &= __funnelshift_r(lo, hi, at & 31);
              }
              return vis;
            };
            const uint32_t vis0 = seen(unit), vis1 = seen(unit + 32);
            // the largest score, and the largest with its key's scale of V
            float most = -INFINITY, weighted = -INFINITY;
            const f2_t by = f2(qs, qs);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const uint32_t vis = (c < 2 ? vis0 : vis1) >> (16 * (c & 1)) & 0xffffu;
              if (!__any_sync(0xffffffffu, vis)) continue;
              uint32_t x[16];
              tc_load16(t_s + 16 * c, x);
              tc_loaded16(x);
#pragma unroll
              for (int k = 0; k < 16; k += 4) {
                const float4 y = *(const float4*)(sk + 16 * c + k), v = *(const float4*)(above + 16 * c + k);
                const f2_t y0 = f2mul(f2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), f2mul(f2(y.x, y.y), by));
                const f2_t y1 = f2mul(f2(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3])), f2mul(f2(y.z, y.w), by));
                const float z0 = vis >> k & 1u ? f2lo(y0) : -INFINITY, z1 = vis >> (k + 1) & 1u ? f2hi(y0) : -INFINITY,
                            z2 = vis >> (k + 2) & 1u ? f2lo(y1) : -INFINITY, z3 = vis >> (k + 3) & 1u ? f2hi(y1) : -INFINITY;
                most = fmaxf(most, fmaxf(fmaxf(z0, z1), fmaxf(z2, z3)));
                weighted = fmaxf(weighted, fmaxf(fmaxf(z0 + v.x, z1 + v.y), fmaxf(z2 + v.z, z3 + v.w)));
              }
            }
            if (__any_sync(0xffffffffu, mine && (most - m > kSlack || weighted - m > room - 127.f))) {
              move(most, weighted);
            }
            f2_t sum = 0;
            const f2_t less = f2(-m, -m), of = f2(over, over);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const uint32_t vis = (c < 2 ? vis0 : vis1) >> (16 * (c & 1)) & 0xffffu;
              uint32_t x[16], p[8] = {};
              if (!__any_sync(0xffffffffu, vis)) {
                tc_store8(t_s + 8 * c, p);
                continue;
              }
              tc_load16(t_s + 16 * c, x);
              tc_loaded16(x);
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                const float2 y = *(const float2*)(sk + 16 * c + k), v = *(const float2*)(sv + 16 * c + k);
                const f2_t t = f2fma(f2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), f2mul(f2(y.x, y.y), by), less);
                f2_t e = f2(ex2(f2lo(t)), ex2(f2hi(t))), z;
                if (masked) {
                  const bool s0 = vis >> k & 1u, s1 = vis >> (k + 1) & 1u;
                  e = f2(s0 ? f2lo(e) : 0.f, s1 ? f2hi(e) : 0.f);
                  z = f2mul(f2mul(e, f2(s0 ? v.x : 0.f, s1 ? v.y : 0.f)), of);
                } else {
                  z = f2mul(f2mul(e, f2(v.x, v.y)), of);
                }
                sum = f2add(sum, e);
                p[k / 2] = half2_of(f2lo(z), f2hi(z));
              }
              tc_store8(t_s + 8 * c, p);  // over scores that have been taken
            }
            l += f2lo(sum) + f2hi(sum);
          }
          tc_stored();
        }
        tc_before();
        __syncwarp();
        if (lane < arrivals) mbar_arrive(&r.p_ready);
      }
      // ---- out, or to the workspace ----
      if (active) {
        wait(&r.pv_done, i - 1);
        tc_after();
        if (lost) l = __uint_as_float(0x7fffffffu);
        const bool whole = w.u == 0 && u1 == n;
        float* part = a.part + (2LL * blockIdx.x + (w.u == 0)) * attend_slot(kATRows, DP);
        if (done > 0) {  // with the sums that are in the workspace
          const float* there = part + kATRows * DP + (mine ? row : 0);
          const float most = fmaxf(m, there[0]), f = ex2(m - most), old = ex2(there[0] - most);
          const int its = __float_as_int(there[2 * kATRows]);
          const int to = attend_unit(fmaxf(f > 0.f ? m + (float)unit : -INFINITY, old > 0.f ? there[0] + (float)its : -INFINITY), most);
          const float of = old * two_to(its - to), now = f * two_to(unit - to);
          l = l * f + there[kATRows] * old;
          m = most, unit = to;
#pragma unroll 1
          for (int c = 0; c < a.D; c += 16) {
            uint32_t o[16];
            tc_load16(t_o + lanes + c, o);
            tc_loaded16(o);
            const float* x = part + (mine ? row : 0) * DP + c;
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * now + x[e] * of);
            tc_store16(t_o + lanes + c, o);
          }
          tc_stored();
        }
        const int half = unit / 2;  // 2^unit in two steps: their product may lie outside fp32's normal values
        const float by = l == 0.f ? 0.f : 1.f / l * two_to(half), rest = two_to(unit - half);
        const int token = fdiv(row0 + row, a.div_g);
        uint16_t* out = (uint16_t*)a.out + (((long long)w.b * a.T + token) * a.Hq + (long long)w.h * a.G + row0 + row - token * a.G) * a.D;
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
                for (int k = 0; k < 8; ++k) f[k] = lost ? l : __uint_as_float(o[8 * e + k]) * by * rest;
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
        if (!whole && mine) attend_leave(part, kATRows, DP, row, m, l, unit);
      }
      tc_before();
      done += u1 - u0;
      if (u1 < last) continue;
      if (w.u == 0 && last < n && threadIdx.x == 0) {
        r.meta[0] = attend_joint(attend_share_of(w, w.from + n - 1), r.live);
        r.meta[1] = w.b, r.meta[2] = w.h, r.meta[3] = w.tile;
      }
      attend_advance<kATRows, kATKeys>(a, w, done);
      done = 0;
    }
  } else if (warp < kIssue) {
    if constexpr (L::kCtas == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kATLoadRegs));
    // =====================================================================
    // keys and values
    // =====================================================================
    const bool values = warp >= kATSoft + kATLoad;
    const int wx = warp - (values ? kATSoft + kATLoad : kATSoft);
    // Eight lanes in a row write four units of two keys, which the swizzle puts on all
    // banks; a warp reads whole heads.
    constexpr int kPer = DP / 16, kAtOnce = L::kAtOnce, kRounds = kATKeys / kAtOnce;  // lanes a key, keys at once
    const int part = (lane & 3) | (kPer == 4 ? 0 : (lane >> 1) & (kPer == 8 ? 4 : 12));
    const int mine = wx * (32 / kPer) + (((lane >> 2) & 1) | (kPer == 4 ? (lane >> 2) & 6 : kPer == 8 ? (lane >> 3) & 2 : 0));
    const bool on = 16 * part < a.D;
    unsigned char* operand = base + (values ? L::kV : L::kK);
    unsigned long long *is_full = values ? r.v_full : r.k_full, *is_empty = values ? r.v_empty : r.k_empty;
    const int put0 = (part >> 2) * L::kChunk + swizzled(mine, 2 * (part & 3)), put1 = (part >> 2) * L::kChunk + swizzled(mine, 2 * (part & 3) + 1);
    const int units = (int)w.left;
    uint4 c[kRounds];  // of the next unit: 16 codes of each key, or the first 8 of 16 plain values
    // (Registers are scarce here: a spilled one would come back from L2, for L1 is small beside
    // this much shared memory.)
    auto places = [&](int kind, int slot, unsigned (&at)[kRounds]) {
      const unsigned* p = &r.at[kind == kATPlain][slot][mine * kRounds];
      if constexpr (kRounds % 4 == 0) {
#pragma unroll
        for (int q = 0; q < kRounds; q += 4) {
          const uint4 v = *(const uint4*)(p + q);
          at[q] = v.x, at[q + 1] = v.y, at[q + 2] = v.z, at[q + 3] = v.w;
        }
      } else {
        const uint2 v = *(const uint2*)p;
        at[0] = v.x, at[1] = v.y;
      }
    };
    const unsigned part_of = on ? 16 * part : 0;  // (lanes past the head read its first values again)
    auto pool = [&](int kind) {
      return (kind == kATPlain ? (const char*)(values ? a.v_cache : a.k_cache) : (const char*)(values ? a.v_codes : a.k_codes)) + (part_of << kind);
    };
    auto load = [&](int j, uint4 (&to)[kRounds]) {
      const int slot = j & (kATRing - 1);
      wait(&r.at_full[slot], j / kATRing);
      const int kind = r.kind[slot];
      // one load whatever the kind: where two paths met, their values would have to be there
      const char* from = pool(kind == kATPlain ? kATPlain : kATCodes);
      unsigned at[kRounds];
      places(kind, slot, at);
#pragma unroll
      for (int q = 0; q < kRounds; ++q) to[q] = stream16(from + at[q] * 16ull);
    };
    if (units > 0) load(0, c);
    int stage = 0, lap = 0;
    for (int i = 0; i < units; ++i) {
      const int slot = i & (kATRing - 1);
      const int kind = r.kind[slot];
      unsigned char* to = operand + stage * L::kTile;
      if (lap) wait(&is_empty[stage], lap + 1);  // what lay there has been read
      if (kind == kATCodes) {
        if (on) {
#pragma unroll
          for (int q = 0; q < kRounds; ++q) {
            uint4 z[2];
            Code<kE4m3>::word(c[q].x, z[0].x, z[0].y);
            Code<kE4m3>::word(c[q].y, z[0].z, z[0].w);
            Code<kE4m3>::word(c[q].z, z[1].x, z[1].y);
            Code<kE4m3>::word(c[q].w, z[1].z, z[1].w);
            *(uint4*)(to + put0 + q * kAtOnce * 128) = z[0];
            *(uint4*)(to + put1 + q * kAtOnce * 128) = z[1];
          }
        }
      } else if (kind == kATPlain) {
        float* scales = (values ? r.sv : r.sk)[slot];
        const char* from = pool(kATPlain) + 16;
        unsigned at[kRounds];
        places(kATPlain, slot, at);
#pragma unroll
        for (int q = 0; q < kRounds; ++q) {
          // the other 8 values came into L2 with the first: they share a sector
          const int key = mine + q * kAtOnce;
          const bool in = !(r.outside[slot][key >> 5] >> (key & 31) & 1u);
          const uint4 other = stream16(from + at[q] * 16ull);
          const uint4 y = on && in ? c[q] : make_uint4(0, 0, 0, 0), z = on && in ? other : make_uint4(0, 0, 0, 0);
          const unsigned lo = max(max(max(y.x & 0x7fffu, y.y & 0x7fffu), max(y.z & 0x7fffu, y.w & 0x7fffu)),
                                  max(max(z.x & 0x7fffu, z.y & 0x7fffu), max(z.z & 0x7fffu, z.w & 0x7fffu)));
          const unsigned hi = max(max(max(y.x & 0x7fff0000u, y.y & 0x7fff0000u), max(y.z & 0x7fff0000u, y.w & 0x7fff0000u)),
                                  max(max(z.x & 0x7fff0000u, z.y & 0x7fff0000u), max(z.z & 0x7fff0000u, z.w & 0x7fff0000u)));
          unsigned top = max(lo << 16, hi);
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          if (kPer >= 8) top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
          if (kPer == 16) top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const bool finite = top < 0x7f800000u;
          const float down = in && finite ? scale_down(top) : __uint_as_float(0x7fffffffu);
          if (part == 0) {
            scales[key] = down;
            if (values) r.above[slot][key] = log_above(down);
          }
          if (values) {
            const unsigned above = __reduce_max_sync(0xffffffffu, in && finite ? (__float_as_uint(down) >> 23) + 1u : 0u);
            if (lane == 0) atomicMax((unsigned*)&r.top[slot], __float_as_uint((float)above));
          }
          const float up = finite ? scale_up(top) : 0.f;
          auto two = [&](uint32_t v) { return finite ? half2_of(bf16_lo(v) * up, bf16_hi(v) * up) : 0u; };
          if (on) {
            *(uint4*)(to + put0 + q * kAtOnce * 128) = make_uint4(two(y.x), two(y.y), two(y.z), two(y.w));
            *(uint4*)(to + put1 + q * kAtOnce * 128) = make_uint4(two(z.x), two(z.y), two(z.z), two(z.w));
          }
          if (q % 2) asm volatile("" ::: "memory");  // two keys at a time
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&is_full[stage]);
      if (++stage == kATStages) stage = 0, ++lap;
      if (i + 1 < units) load(i + 1, c);
    }
  } else {
    if constexpr (L::kCtas == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kATIssueRegs));
    if (warp == kIssue) {
      // ===================================================================
      // products
      // ===================================================================
      // The warp walks along together and its elected lane issues: what the products take is
      // then known to be the same in all lanes (an issue under `lane == 0` took 100 clocks,
      // 64 being the product's own time).
      const bool leader = tc_elect();
      const unsigned long long d_k = tc_operand(smem_addr(base + L::kK), 16), d_v = tc_operand(smem_addr(base + L::kV), L::kChunk);
      const uint32_t kind_s = tc_kind(kATKeys, false), kind_o = tc_kind(a.D, true);
      const int steps = a.D / 16;
      int i = 0, stage = 0, lap = 0, pieces = 0, done = 0;
      while (w.left > 0) {
        const int n = attend_units<kATRows, kATKeys>(a, w.s, w.tile), last = (int)min((long long)n, w.u + w.left);
        const int u0 = w.u + done, u1 = min(last, u0 + kATPiece);
        wait(&r.q_full, pieces++);
        for (int u = u0; u < u1; ++u, ++i) {
          wait(&r.k_full[stage], lap);
          if (i > 0) wait(&r.pv_done, i - 1);  // S's columns hold the weights of the last unit until P V has read them
          tc_after();
          if (leader) {
            const unsigned long long d = d_k + stage * (L::kTile >> 4);
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
              if (k < steps) tc_mma_t(tmem, t_q + 8 * k, d + (((k >> 2) * L::kChunk + (k & 3) * 32) >> 4), kind_s, k > 0);
            tc_commit(&r.k_empty[stage]);
            tc_commit(&r.s_full);
            mbar_arrive(&r.s_full);  // with what k_full brought: the scales
          }
          __syncwarp();
          wait(&r.v_full[stage], lap);
          wait(&r.p_ready, i);
          tc_after();
          if (leader) {
            const unsigned long long d = d_v + stage * (L::kTile >> 4);
            const bool add = u > u0;
#pragma unroll
            for (int k = 0; k < kATKeys / 16; ++k) tc_mma_t(t_o, tmem + 8 * k, d + k * (2048 >> 4), kind_o, k > 0 || add);
            tc_commit(&r.v_empty[stage]);
            tc_commit(&r.pv_done);
            tc_commit(&r.at_empty[i & (kATRing - 1)]);  // its places and scales have been used
          }
          __syncwarp();
          if (++stage == kATStages) stage = 0, ++lap;
        }
        done += u1 - u0;
        if (u1 < last) continue;
        attend_advance<kATRows, kATKeys>(a, w, done);
        done = 0;
      }
      // nothing of the tensor cores is in flight when the tensor memory goes back
      if (leader) tc_commit(&r.drain);
      __syncwarp();
      if (!warp_wait(&r.drain, 0, mbar_tries(kSpinLimit))) r.waits.out = 1;
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
            unsigned top = 0;
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
            for (int q = 0; q < kQ; ++q)
              if (__float_as_uint(sv[q]) < 0x7f800000u) top = max(top, (__float_as_uint(sv[q]) >> 23) + 1u);
            top = __reduce_max_sync(0xffffffffu, top);
            if (lane == 0) r.top[slot] = (float)top;
            // Codes of a page outside may be seen by some rows alone, and a product with a weight of 0 has to
            // be 0: another key of the unit stands for them or, if there is none, what lies in shared memory.
            const int some = __reduce_max_sync(0xffffffffu, max(at[0], at[kQ - 1]));
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
              const int k = 32 * q + lane;
              r.at[!codes][slot][L::place(k)] = some < 0 ? 0u : (unsigned)((((long long)(at[q] < 0 ? some : at[q]) * a.Hkv + w.h) * a.D >> 4) << (codes ? 0 : 1));
              const unsigned out = __ballot_sync(0xffffffffu, at[q] < 0);
              if (lane == 0) r.outside[slot][q] = out;
              if (codes) r.sk[slot][k] = sk[q], r.sv[slot][k] = sv[q], r.above[slot][k] = log_above(sv[q]);
            }
            if (lane == 0) r.kind[slot] = !codes ? kATPlain : some < 0 ? kATNone : kATCodes;
          }
          if (w.s.bad && lane == 0) r.kind[slot] = kATNone;
          __syncwarp();
          if (lane == 0) mbar_arrive(&r.at_full[slot]);
        }
        attend_advance<kATRows, kATKeys>(a, w, u1 - u0);
      }
    }
  }
  tc_before();
  __syncthreads();
  if (threadIdx.x == 0 && r.waits.out) atomicOr(a.status, kStatusTimeout);
  if (warp == kIssue) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(L::kColumns) : "memory");
  }
  if (threadIdx.x == 0) a.meta[blockIdx.x] = make_int4(r.meta[0], r.meta[1], r.meta[2], r.meta[3]);
}

template <bool kE4m3, int DP>
static cudaError_t launch_tiles(KvAttendArgs a, int sms, size_t* bytes, cudaStream_t s) {
  using L = Tiles<DP>;
  a.tiles = (int)(((long long)a.T * a.G + kATRows - 1) / kATRows);
  const long long keys = (long long)a.max_code_pages * a.block + (long long)a.max_pages * a.page_size;
  const double most = (double)a.B * a.Hkv * a.tiles * (double)(keys / kATKeys + 2);
  const int grid = (int)fmin((double)sms * L::kCtas, most);
  const size_t slots = ((size_t)grid * 2 * attend_slot(kATRows, DP) * 4 + 255) / 256 * 256;
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
  return launch_join<uint16_t, DP, kATRows>(a, grid, s);
}

}  // namespace sv
