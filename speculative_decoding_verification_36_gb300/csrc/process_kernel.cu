// process_kernel.cu -- what a user's settings do to the logits before a verify
// step reads them: penalties for repeated tokens, additive biases and grammar
// masks, for chains and for trees of drafts, and the token counts behind them.
//
// With c_r(v) the occurrences of v among the sequence's output tokens and the
// drafted tokens above row r (chain: x_0 .. x_{r-1}; tree: node r - 1 and its
// ancestors), seen_r(v) = v in the prompt or c_r(v) > 0:
//   z1 = seen_r(v) ? (z > 0 ? z / rho : z rho) : z
//   z2 = z1 - f c_r(v) - p [c_r(v) > 0] + sum of v's biases
//   z' = v allowed in row r ? z2 : -inf
// in fp32, rounded once to the logits' type.  A verify under these settings
// needs them per row: row r of a chain already counts the r drafts before it.
#include "sv_bulk.cuh"
#include "sv_common.cuh"
#include "sv_kernels.h"

#include <cooperative_groups.h>
#include <string.h>

namespace sv {

// ---------------------------------------------------------------------------
// token counts
// ---------------------------------------------------------------------------
// state row of a sequence: P = V rounded up to 32 counts (bits 0..30: output
// tokens, bit 31: in the prompt), then P / 32 words with one bit per non-zero
// count.  The bitmap is what lets the processing kernel skip the counts of
// the tokens that never occurred: V / 8 bytes instead of 4 V.
constexpr int kCountThreads = 256;

// A row's lengths; false for bad data.
__device__ __forceinline__ bool count_lengths(const CountArgs& a, int b, int& L, int& Lp) {
  const long long n = a.lengths ? a.lengths[b] : a.stride, np = a.prompt_lengths ? a.prompt_lengths[b] : 0;
  L = (int)n;
  Lp = (int)np;
  return n >= 0 && n <= a.stride && np >= 0 && np <= n;
}

// Adding to a state: one atomic for the count and one for the bitmap per
// token.  Meant for the few tokens of a step.
__global__ void __launch_bounds__(kCountThreads) count_kernel(const __grid_constant__ CountArgs a) {
  const int b = blockIdx.y;
  int L, Lp;
  if (!count_lengths(a, b, L, Lp)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, kStatusBadData);
    return;
  }
  int32_t* count = a.state + (long long)b * a.words;
  unsigned* bitmap = (unsigned*)(count + a.P);
  const int32_t* h = a.tokens + (long long)b * a.stride;
  for (long long i = (long long)blockIdx.x * kCountThreads + threadIdx.x; i < L; i += (long long)gridDim.x * kCountThreads) {
    const int t = __ldg(h + i);
    if (t < 0 || t >= a.V) continue;
    if (i < Lp)
      atomicOr((unsigned*)count + t, 0x80000000u);
    else
      atomicAdd(count + t, 1);
    atomicOr(bitmap + (t >> 5), 1u << (t & 31));
  }
}

// A state made anew: a CTA counts one range of the vocabulary of one sequence
// in shared memory, from the whole history (4 bytes a token, from L2 for every
// range but the first), and writes the range's counts and bitmap once.  The
// bound is the state's 4 1/8 bytes a token of the vocabulary: 40 us for B = 256,
// V = 152064 and histories of up to 8192 tokens (0.17 GB, 4.2 TB/s; a range is
// cleared, counted and written by turns, and the history read once per range).
// Zeroing the state and adding with atomics,
// which fetch and write a sector each, took 74 us.
// Few sequences with long histories: a cluster of CTAs shares a range, each
// counts a part of the history, and then each adds up a part of the range over
// the cluster's shared memory.  (One history of 131072 tokens, V = 128256: 9 us,
// and 26 us with one CTA per range.)
// kPacked: no history has over 32767 tokens, so that a count and the prompt's
// bit fit 16 bits, and a range of twice the tokens the same memory: half the
// readings of the history.
constexpr int kCountNewThreads = 512;
constexpr int kCountPackedMost = 32767;
template <bool kPacked>
__global__ void __launch_bounds__(kCountNewThreads) count_new_kernel(const __grid_constant__ CountArgs a) {
  extern __shared__ __align__(16) unsigned s_count[];
  namespace cg = cooperative_groups;
  const cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int unit = blockIdx.x / C;
  const int b = unit / a.ranges, c0 = (unit - b * a.ranges) * a.range;
  const int n = (int)min((long long)a.range, a.P - c0);  // a multiple of 32
  const int tid = threadIdx.x;
  int L, Lp;
  const bool ok = count_lengths(a, b, L, Lp);
  for (int i = tid; i < n / (kPacked ? 8 : 4); i += kCountNewThreads) ((uint4*)s_count)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (!ok && c0 == 0 && rank == 0 && tid == 0) atomicOr(a.status, kStatusBadData);
  __syncthreads();
  if (ok) {
    const int32_t* h = a.tokens + (long long)b * a.stride;
    const unsigned end = (unsigned)min(n, a.V - c0);
    // tokens [from, to) of the history: the prompt's set a bit, the others count.
    // A negative token's offset is above every range's end.
    const int step = C * kCountNewThreads, me = rank * kCountNewThreads + tid;
    auto scan = [&](int from, int to, auto&& put) {
      auto one = [&](int t) {
        const unsigned off = (unsigned)t - (unsigned)c0;
        if (off < end) put(kPacked ? s_count + (off >> 1) : s_count + off, kPacked ? 16 * (off & 1) : 0);
      };
      int q0 = from, q1 = from;  // whole 16-byte loads
      if (a.vec && to - from >= 8) {
        q0 = (from + 3) & ~3;
        q1 = to & ~3;
#pragma unroll 4
        for (int q = q0 + 4 * me; q < q1; q += 4 * step) {
          const int4 v = __ldg((const int4*)(h + q));
          one(v.x), one(v.y), one(v.z), one(v.w);
        }
        if (me < q0 - from) one(__ldg(h + from + me));
      }
      for (int i = q1 + me; i < to; i += step) one(__ldg(h + i));
    };
    scan(0, Lp, [](unsigned* p, int at) { atomicOr(p, (kPacked ? 0x8000u : 0x80000000u) << at); });
    scan(Lp, L, [](unsigned* p, int at) { atomicAdd(p, 1u << at); });
  }
  if (C > 1)
    cluster.sync();
  else
    __syncthreads();
  int32_t* row = a.state + (long long)b * a.words;
  // the CTA's part of the range, four tokens a lane, eight lanes a word of the bitmap
  const int lane = tid & 31, words = n / 32, per = (words + C - 1) / C;
  const int o0 = 32 * rank * per, o1 = min(n, o0 + 32 * per);
  for (int o = o0 + 128 * (tid >> 5); o < o1; o += 128 * (kCountNewThreads / 32)) {
    const int off = o + 4 * lane;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (off < o1) {
      if constexpr (kPacked) {
        const uint2 w = *(const uint2*)(s_count + off / 2);
        auto wide = [](unsigned x) { return (x & 0x7fffu) | (x & 0x8000u) << 16; };
        v = make_uint4(wide(w.x), wide(w.x >> 16), wide(w.y), wide(w.y >> 16));
      } else {
        v = *(const uint4*)(s_count + off);
      }
      if (!kPacked && C > 1) {
        uint4 sum = make_uint4(0u, 0u, 0u, 0u), top = sum;
        for (int r = 0; r < C; ++r) {
          const uint4 x = *cluster.map_shared_rank((const uint4*)(s_count + off), r);
          sum.x += x.x & 0x7fffffffu, sum.y += x.y & 0x7fffffffu, sum.z += x.z & 0x7fffffffu, sum.w += x.w & 0x7fffffffu;
          top.x |= x.x, top.y |= x.y, top.z |= x.z, top.w |= x.w;
        }
        v.x = sum.x | (top.x & 0x80000000u), v.y = sum.y | (top.y & 0x80000000u);
        v.z = sum.z | (top.z & 0x80000000u), v.w = sum.w | (top.w & 0x80000000u);
      }
      *(uint4*)(row + c0 + off) = v;
    }
    unsigned bits = ((v.x != 0u) | (v.y != 0u) << 1 | (v.z != 0u) << 2 | (v.w != 0u) << 3) << (4 * (lane & 7));
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) bits |= __shfl_xor_sync(0xffffffffu, bits, d);
    if ((lane & 7) == 0 && off < o1) ((unsigned*)row)[a.P + (c0 + off) / 32] = bits;
  }
  // the padding behind the bitmap
  if (c0 + n >= a.P && rank == 0 && tid < a.words - a.P - a.P / 32) row[a.P + a.P / 32 + tid] = 0;
  if (C > 1) cluster.sync();  // the others read this CTA's shared memory until here
}

constexpr int kCountRange = 16384;     // most counts of a range: 64 KB, three CTAs per SM (packed: twice as many)
constexpr int kCountMinRange = 1024;

cudaError_t count_configure() {
  const cudaError_t e =
      cudaFuncSetAttribute(count_new_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCountRange * 4);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(count_new_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCountRange * 4);
}

cudaError_t launch_count(const CountArgs& a, int sms, cudaStream_t s) {
  CountArgs c = a;
  if (a.reset) {
    // Ranges as large as they may be while every SM has its CTAs; where even
    // the largest leave SMs without one, a cluster to each range if there is
    // enough history to share out.
    int C = 1;
    while (C < 8 && (long long)a.B * ((a.P + kCountRange - 1) / kCountRange) * C < sms && a.stride >= 4096LL * C) C *= 2;
    const bool packed = C == 1 && a.stride <= kCountPackedMost;
    const int most = packed ? 2 * kCountRange : kCountRange;
    const long long want = ((long long)a.B * a.P * C + 2LL * sms - 1) / (2LL * sms);
    c.range = want > most ? most : (int)((want + 31) / 32 * 32);
    if (c.range < kCountMinRange) c.range = kCountMinRange;
    c.ranges = (int)((a.P + c.range - 1) / c.range);
    c.range = (int)(((a.P + c.ranges - 1) / c.ranges + 127) / 128 * 128);  // of equal lengths
    c.ranges = (int)((a.P + c.range - 1) / c.range);
    c.vec = ((uintptr_t)a.tokens & 15) == 0 && a.stride % 4 == 0;
    const long long per = (1LL << 27) / c.ranges;  // sequences of one launch
    for (long long b0 = 0; b0 < a.B; b0 += per) {
      c.B = (int)(a.B - b0 < per ? a.B - b0 : per);
      c.tokens = a.tokens + b0 * a.stride;
      c.lengths = a.lengths ? a.lengths + b0 : nullptr;
      c.prompt_lengths = a.prompt_lengths ? a.prompt_lengths + b0 : nullptr;
      c.state = a.state + b0 * a.words;
      cudaLaunchConfig_t cfg;
      memset(&cfg, 0, sizeof cfg);
      cfg.gridDim = dim3((unsigned)(c.B * c.ranges * C));
      cfg.blockDim = dim3(kCountNewThreads);
      cfg.dynamicSmemBytes = (size_t)c.range * (packed ? 2 : 4);
      cfg.stream = s;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = (unsigned)C;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      const cudaError_t e =
          packed ? cudaLaunchKernelEx(&cfg, count_new_kernel<true>, c) : cudaLaunchKernelEx(&cfg, count_new_kernel<false>, c);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  if (a.stride == 0 && !a.lengths && !a.prompt_lengths) return cudaSuccess;
  // (rows without entries: one CTA each, to judge their lengths)
  const int per_row = a.stride ? (int)((a.stride + kCountThreads - 1) / kCountThreads) : 1;
  const int x = per_row < 4 * sms ? per_row : 4 * sms;
  for (int b0 = 0; b0 < a.B; b0 += 65535) {  // the grid's y extent
    c.B = a.B - b0 < 65535 ? a.B - b0 : 65535;
    c.tokens = a.tokens + (long long)b0 * a.stride;
    c.lengths = a.lengths ? a.lengths + b0 : nullptr;
    c.prompt_lengths = a.prompt_lengths ? a.prompt_lengths + b0 : nullptr;
    c.state = a.state + (long long)b0 * a.words;
    count_kernel<<<dim3((unsigned)x, (unsigned)c.B), kCountThreads, 0, s>>>(c);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// ---------------------------------------------------------------------------
// logits
// ---------------------------------------------------------------------------
// A CTA takes one chunk of the vocabulary of one sequence and all rows of a
// row group; each of its warps has 512 of the chunk's tokens.  What the rows
// share is worked out once: few tokens are touched by the history, a bias or a
// draft (a few percent of the vocabulary under a long history), so each warp
// lists its own, with the additive term -f c - p [c > 0] + biases.  After the
// lists no barrier joins the warps until the next unit.
//
// Apart from its input (process_kernel): a warp's parts of kBatch rows at a time
// come to shared memory by bulk copies, with further batches behind them; the
// list is applied to them there, and they go out through registers, masked.
// The bound is one reading and one writing of the logits: 241 us for B = 256,
// R = 9, V = 152064 in bf16 with histories of up to 8192 tokens, 300 biases and
// a mask for every row (1.46 GB, 6.0 TB/s; without any of them 207 us, as fast
// as a plain copy).  What else was measured on that workload: the terms worked
// into every vector that holds a touched token, from a dense table, 333 us
// (nearly every warp-wide vector holds one); a copying pass and then single
// touched tokens read and written over it, 292 us (32 sectors a step).
// A small call is bound by its chain of two trips to memory, the barrier and
// the launch: 6.9 us for B = 1, R = 5, V = 32000.
//
// In place (process_mask_kernel, process_in_place_kernel): only the vectors that
// hold a forbidden token and the listed tokens are read and written, where they
// lie.  That is the caller's choice, by out == in, and gains where little is
// touched.  B = 256, R = 9, V = 152064 in bf16, us in place and apart: histories
// of up to 512 tokens 92 and 211, of up to 8192 tokens 178 and 223; with a mask
// for every row beside them, which makes a second pass over the same rows, 253
// and 221 (512 tokens), 300 and 241 (8192 tokens and 300 biases).  Masks alone,
// R = 5, V = 128256: 61 and 107.
constexpr int kProcThreads = 256;
constexpr int kProcWarps = kProcThreads / 32;
constexpr int kProcPiece = 512;                        // tokens of a warp
constexpr int kProcChunk = kProcPiece * kProcWarps;    // ... of a CTA
constexpr int kProcWords = kProcChunk / 32;            // ... in bitmap words
constexpr int kProcRows = 4;       // rows of an entry at once when in place
constexpr int kProcMaxDrafts = 1024;
constexpr int kProcDrafts = 256;   // drafts in a chunk that are listed; more are looked up in the input
constexpr int kProcMostRows = 12;  // rows of a group (in a tree, their paths are kept as bit sets)
static_assert(kProcPiece == 16 * 32, "a lane holds 16 of its warp's tokens");
static_assert(kProcWords <= kProcThreads, "a thread clears a word");
// list entries: offset in the chunk, then
constexpr unsigned kProcSeen = 1u << 12;     // in the history
constexpr unsigned kProcCounted = 1u << 13;  // c > 0 without the drafts
constexpr unsigned kProcDraft = 1u << 14;    // some draft carries it
constexpr unsigned kProcOffset = kProcSeen - 1u;
static_assert(kProcChunk <= (int)kProcSeen, "an offset leaves the flags free");

// What the CTA's threads gather for their unit's lists; two, by turns, so that
// the next unit's is cleared while this one's is in use.
struct ProcGather {
  unsigned bias[kProcWords];     // tokens with a bias
  unsigned draft[kProcWords];    // tokens that some draft carries
  unsigned drafts[kProcDrafts];  // drafts in the chunk: (offset << 16) | node
  int n_draft;
  int twice;  // a token with several biases
  int bad, pad;
};
struct ProcShared {
  float adj[kProcChunk];            // of the listed tokens, without the drafts
  unsigned short list[kProcChunk];  // each warp's in its own part
  int4 own[kProcThreads];           // per lane: offset and flags (-1: no terms), node (-1: none), lanes with the token, terms
  ProcGather gather[2];
};
__device__ __forceinline__ void proc_clear(ProcGather& g) {
  if (threadIdx.x < kProcWords) g.bias[threadIdx.x] = g.draft[threadIdx.x] = 0u;
  if (threadIdx.x == 0) g.n_draft = g.twice = g.bad = 0;
}
// tree: the nodes above each row of the group
struct ProcPaths {
  unsigned row[kProcMostRows][kProcMaxDrafts / 32];
};

struct Bf16Tag {};
template <class T>
struct ProcType;
template <>
struct ProcType<float> {
  using storage = uint32_t;
  static constexpr int kVec = 4, kBatch = 1, kBatches = 2;
  static constexpr uint32_t kNegInf = 0xff800000u, kNan = 0x7fc00000u;
  static __device__ __forceinline__ float widen(uint32_t w) { return __uint_as_float(w); }
  static __device__ __forceinline__ uint32_t round(float f) { return __float_as_uint(f); }
};
template <>
struct ProcType<Bf16Tag> {
  using storage = uint16_t;
  static constexpr int kVec = 8, kBatch = 2, kBatches = 2;
  static constexpr uint16_t kNegInf = 0xff80u, kNan = 0x7fc0u;
  static __device__ __forceinline__ float widen(uint16_t w) { return __uint_as_float((uint32_t)w << 16); }
  static __device__ __forceinline__ uint16_t round(float f) {
    uint16_t r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(f));
    return r;
  }
};

// A warp's rows in flight: a piece each, and its phase.
template <class T>
struct alignas(16) ProcStages {
  static constexpr int kStage = kProcPiece + ProcType<T>::kVec;
  typename ProcType<T>::storage row[ProcType<T>::kBatches][ProcType<T>::kBatch][kStage];
};
template <class T>
struct ProcCopyShared : ProcShared {
  ProcStages<T> stages[kProcWarps];
  unsigned long long full[kProcWarps][ProcType<T>::kBatches];
  uint4 claim[2];                // answers to the requests for further units
  unsigned long long claimed[2];
  int unit[2];                   // the unit of each round, by turns
  // then, for a tree, ProcPaths
};

// A vector with -inf where the element's bit is clear.
template <class T>
__device__ __forceinline__ uint4 proc_keep(uint4 x, unsigned bits) {
  if constexpr (sizeof(typename ProcType<T>::storage) == 4) {
    x.x = bits & 1u ? x.x : ProcType<T>::kNegInf;
    x.y = bits & 2u ? x.y : ProcType<T>::kNegInf;
    x.z = bits & 4u ? x.z : ProcType<T>::kNegInf;
    x.w = bits & 8u ? x.w : ProcType<T>::kNegInf;
  } else {
    constexpr uint32_t fill = ProcType<T>::kNegInf * 0x10001u;
    // four bits to the tops of four bytes, then each top over two bytes
    const uint32_t lo = (bits & 15u) * 0x10204080u, hi = (bits >> 4) * 0x10204080u;
    auto one = [](uint32_t w, uint32_t tops, unsigned which) {
      uint32_t keep;  // a selector digit of 8 and up spreads the byte's top bit
      asm("prmt.b32 %0, %1, 0, %2;" : "=r"(keep) : "r"(tops), "r"(which));
      return (w & keep) | (fill & ~keep);
    };
    x.x = one(x.x, lo, 0x9988u), x.y = one(x.y, lo, 0xbbaau), x.z = one(x.z, hi, 0x9988u), x.w = one(x.w, hi, 0xbbaau);
  }
  return x;
}

// Where a unit lies: a chunk of a sequence's vocabulary in a group of its rows.
struct ProcUnit {
  int b, base;        // sequence, first token of the chunk
  int r0, rows;       // first row, rows
  int start, n_tok;   // first token and tokens of this warp's piece
  long long row0;     // elements before the piece in row r0
};
// The order of the units: by sequence and row group, then by chunk; but the
// first chunks, where a tokenizer puts what is frequent and the lists are long,
// are dealt out evenly over the first half, so that none of them is still under
// way when the others end.  (B = 256, R = 9, V = 152064, everything on: 266 us
// without this, 241 with it.)
__device__ __forceinline__ ProcUnit proc_unit(const ProcessArgs& a, unsigned unit) {
  ProcUnit u;
  int pair = 0, chunk = 0, x = (int)unit;
  const int pairs = a.B * a.groups;
  if (a.chunks > 1) {
    const int turn = fdiv(x, a.div_turn);  // one first chunk, then turn_length - 1 others
    if (turn < pairs && x == turn * a.turn_length) {
      pair = turn;
    } else {
      x -= min(turn + 1, pairs);
      pair = fdiv(x, a.div_rest);
      chunk = 1 + x - pair * (a.chunks - 1);
    }
  } else {
    pair = x;
  }
  u.base = chunk * kProcChunk;
  u.b = fdiv(pair, a.div_groups);
  u.r0 = (pair - u.b * a.groups) * a.rows_per;
  u.rows = min(a.rows_per, a.R - u.r0);
  u.start = u.base + (int)(threadIdx.x >> 5) * kProcPiece;
  u.n_tok = max(0, min(kProcPiece, a.V - u.start));
  u.row0 = ((long long)u.b * a.R + u.r0) * a.V + u.start;
  return u;
}

// What the rows of a unit share, for one warp.
struct ProcShare {
  int n_list;
  float rep, inv, freq, pres;
  bool bad;
  ProcPaths* paths;
  // Up to 32 drafts in the chunk: their tokens are not in the list, but lane i
  // has draft i (ProcShared::own), and its token's terms where it is the lowest
  // lane that carries the token and the token is the warp's.
  bool few, here;  // ... so; some lane of the warp has terms
  const ProcGather* gather;
};

// What a unit's lists are made from, on its way into a thread's registers: the
// bitmap of the thread's 16 tokens, the penalties, and of the drafts and biases
// as many as fit (longer lists are read to the end later).
constexpr int kProcBiasRegs = 2;
constexpr int kProcCountRegs = 2;  // counts of the thread's tokens that occurred, the first of them
struct ProcAhead {
  unsigned mine;
  int count[kProcCountRegs];
  int draft, parent;
  int bias_t[kProcBiasRegs];
  float bias_v[kProcBiasRegs];
  float rep, freq, pres;
};
__device__ __forceinline__ ProcAhead proc_ahead(const ProcessArgs& a, const ProcUnit& u) {
  const int tid = threadIdx.x;
  ProcAhead h;
  h.mine = a.state && u.base + 16 * tid < a.P
               ? __ldg((const unsigned short*)(a.state + (long long)u.b * a.words + a.P) + (u.base >> 4) + tid)
               : 0u;
  // a state counted for a larger vocabulary may hold tokens that these rows do not have
  const int own = a.V - u.base - 16 * tid;
  if (own < 16) h.mine &= (1u << max(own, 0)) - 1u;
  const int N = a.drafts ? a.R - 1 : 0;
  h.draft = tid < N ? __ldg(a.drafts + (long long)u.b * N + tid) : -1;
  h.parent = a.parents && tid < N ? __ldg(a.parents + (long long)u.b * N + tid) : -1;
#pragma unroll
  for (int q = 0; q < kProcBiasRegs; ++q) {
    const int i = q * kProcThreads + tid;
    const long long at = (long long)u.b * a.n_bias + i;
    h.bias_t[q] = i < a.n_bias ? __ldg(a.bias_tokens + at) : -1;
    h.bias_v[q] = i < a.n_bias ? __ldg(a.bias_values + at) : 0.f;
  }
  h.rep = a.rep ? __ldg(a.rep + u.b) : 1.f;
  h.freq = a.freq ? __ldg(a.freq + u.b) : 0.f;
  h.pres = a.pres ? __ldg(a.pres + u.b) : 0.f;
  return h;
}
// ... and, once the bitmap is there, the counts.
__device__ __forceinline__ void proc_counts(const ProcessArgs& a, const ProcUnit& u, ProcAhead& h) {
  unsigned left = h.mine;
#pragma unroll
  for (int q = 0; q < kProcCountRegs; ++q) {
    h.count[q] = left ? __ldg(a.state + (long long)u.b * a.words + u.base + 16 * (int)threadIdx.x + __ffs(left) - 1) : 0;
    left &= left - 1;
  }
}

// Some token has several biases: each warp sums those of its own tokens, in the
// order given.
__device__ __forceinline__ void proc_twice(const ProcessArgs& a, float* adj, int b, int base, int n_tok) {
  const int lane = threadIdx.x & 31, lo = (int)(threadIdx.x >> 5) * kProcPiece;
  const long long first = (long long)b * a.n_bias;
  for (int i = lane; i < kProcPiece; i += 32) adj[lo + i] = 0.f;
  __syncwarp();
  for (int i0 = 0; i0 < a.n_bias; i0 += 32) {
    const int i = i0 + lane;
    const int t = i < a.n_bias ? __ldg(a.bias_tokens + first + i) - base - lo : -1;
    const bool own = t >= 0 && t < n_tok;
    const float v = own ? __ldg(a.bias_values + first + i) : 0.f;
    for (unsigned m = __ballot_sync(0xffffffffu, own); m; m &= m - 1) {
      const int l = __ffs(m) - 1;
      const int off = lo + __shfl_sync(0xffffffffu, t, l);
      const float x = __shfl_sync(0xffffffffu, v, l);
      if (lane == 0) adj[off] += x;
    }
  }
}

// The lists of a unit from what came ahead.  Every thread of the CTA takes part,
// behind a barrier that says that the lists before are done with and `g`, the
// unit's gathering, is empty; on return each warp may go on.  idle: the other
// gathering, which is emptied for the next unit.
__device__ __forceinline__ void proc_lists(const ProcessArgs& a, ProcShared& sh, ProcGather& g, ProcGather& idle,
                                           const ProcUnit& u, const ProcAhead& h, ProcShare& c) {
  const int tid = threadIdx.x, lane = tid & 31, lo = tid >> 5 << 9;  // the warp's first token in the chunk
  const int32_t* state = a.state + (long long)u.b * a.words;
  const int N = a.drafts ? a.R - 1 : 0;
  const int32_t* draft_row = a.drafts + (long long)u.b * N;
  const int32_t* parent_row = a.parents + (long long)u.b * N;
  const long long first = (long long)u.b * a.n_bias;
  const int left = min(kProcChunk, a.V - u.base);
  const unsigned mine = h.mine;
  c.rep = h.rep;
  c.freq = h.freq;
  c.pres = h.pres;
  c.inv = 1.f / c.rep;
  c.gather = &g;
  // drafts and biases may be any warp's; without them no barrier is needed
  const bool shared = N > 0 || a.n_bias > 0;
  if (shared) proc_clear(idle);
  auto put_draft = [&](int j, int t, int parent) {
    if (t >= 0 && t < left) {
      const int at = atomicAdd(&g.n_draft, 1);
      if (at < kProcDrafts) g.drafts[at] = ((unsigned)t << 16) | (unsigned)j;
      atomicOr(&g.draft[t >> 5], 1u << (t & 31));
    }
    if (parent < -1 || parent >= j) g.bad = 1;
  };
  if (tid < N) put_draft(tid, h.draft - u.base, h.parent);
#pragma unroll 1
  for (int j = kProcThreads + tid; j < N; j += kProcThreads)
    put_draft(j, __ldg(draft_row + j) - u.base, a.parents ? __ldg(parent_row + j) : -1);
  auto put_bias = [&](int t, float v) {
    if (t < 0 || t >= left) return;
    if (atomicOr(&g.bias[t >> 5], 1u << (t & 31)) >> (t & 31) & 1u)
      g.twice = 1;
    else
      sh.adj[t] = v;
  };
#pragma unroll
  for (int q = 0; q < kProcBiasRegs; ++q)
    if (q * kProcThreads + tid < a.n_bias) put_bias(h.bias_t[q] - u.base, h.bias_v[q]);
#pragma unroll 1
  for (int i = kProcBiasRegs * kProcThreads + tid; i < a.n_bias; i += kProcThreads)
    put_bias(__ldg(a.bias_tokens + first + i) - u.base, __ldg(a.bias_values + first + i));
  if (shared) __syncthreads();
  // a penalty that is no number, or a factor that it is not possible to divide by:
  // within these limits its reciprocal is a normal number too
  c.bad = (shared && g.bad) || !(c.rep >= 0x1p-126f && c.rep <= 0x1p126f) || !(fabsf(c.freq) < INFINITY) || !(fabsf(c.pres) < INFINITY);
  if (c.bad && tid == 0) atomicOr(a.status, kStatusBadData);

  const int n_draft = shared ? g.n_draft : 0;
  c.few = n_draft <= 32;
  const unsigned draft = shared ? (g.draft[tid >> 1] >> (16 * (tid & 1))) & 0xffffu : 0u;
  const unsigned bias = shared ? (g.bias[tid >> 1] >> (16 * (tid & 1))) & 0xffffu : 0u;
  unsigned touch = mine | bias;
  touch = c.few ? touch & ~draft : touch | draft;
  int at = __popc(touch);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, at, d);
    if (lane >= d) at += o;
  }
  c.n_list = __shfl_sync(0xffffffffu, at, 31);
  at += lo - __popc(touch);
  if (shared && g.twice) proc_twice(a, sh.adj, u.b, u.base, u.n_tok);
  __syncwarp();
  c.here = false;
  if (c.few && n_draft > 0) {
    const unsigned d = lane < n_draft ? g.drafts[lane] : 0xffffffffu;
    int off = lane < n_draft ? (int)(d >> 16) : -1 - lane;
    const unsigned same = __match_any_sync(0xffffffffu, off);
    const unsigned bits = __shfl_sync(0xffffffffu, mine, off >> 4 & 31);
    if (off < 0 || off >> 9 != tid >> 5 || lane != __ffs(same) - 1) off = -1;
    c.here = __any_sync(0xffffffffu, off >= 0);
    if (c.here) {
      const bool seen = off >= 0 && (bits >> (off & 15) & 1u);
      const int n = seen ? __ldg(state + u.base + off) & 0x7fffffff : 0;
      float add = off >= 0 && (g.bias[off >> 5] >> (off & 31) & 1u) ? sh.adj[off] : 0.f;
      if (n > 0) add += -c.freq * (float)n - c.pres;
      if (off >= 0) off |= (seen ? kProcSeen : 0u) | (n > 0 ? kProcCounted : 0u);
      sh.own[tid] = make_int4(off, lane < n_draft ? (int)(d & 0xffffu) : -1, (int)same, __float_as_int(add));
    }
  }
  // the entries and their terms
  auto put_entry = [&](int i, int n, float adj) {
    const int off = 16 * tid + i;
    if (n > 0) adj += -c.freq * (float)n - c.pres;
    sh.adj[off] = adj;
    sh.list[at++] = (unsigned short)(off | (mine >> i & 1u ? kProcSeen : 0u) | (n > 0 ? kProcCounted : 0u) |
                                     (draft >> i & 1u ? kProcDraft : 0u));
  };
  if (!__any_sync(0xffffffffu, __popc(mine) > kProcCountRegs)) {
    int rank = 0;
#pragma unroll 1
    for (unsigned all = mine | touch; all; all &= all - 1) {
      const int i = __ffs(all) - 1;
      int n = 0;
      if (mine >> i & 1u) {
        static_assert(kProcCountRegs == 2, "named one by one");
        n = (rank == 0 ? h.count[0] : h.count[1]) & 0x7fffffff;
        ++rank;
      }
      if (touch >> i & 1u) put_entry(i, n, bias >> i & 1u ? sh.adj[16 * tid + i] : 0.f);
    }
  } else {
    // more counts than came ahead: entries first, then their counts all at once
#pragma unroll 1
    for (unsigned all = touch; all; all &= all - 1) {
      const int i = __ffs(all) - 1;
      put_entry(i, 0, bias >> i & 1u ? sh.adj[16 * tid + i] : 0.f);
    }
    __syncwarp();
#pragma unroll 4
    for (int e = lane; e < c.n_list; e += 32) {
      const unsigned entry = sh.list[lo + e];
      const int off = entry & kProcOffset, n = entry & kProcSeen ? __ldg(state + u.base + off) & 0x7fffffff : 0;
      if (n > 0) {
        sh.adj[off] += -c.freq * (float)n - c.pres;
        sh.list[lo + e] = (unsigned short)(entry | kProcCounted);
      }
    }
  }
  if (a.parents && n_draft > 0) {
    // the nodes above each row of the group; a parent precedes its child
    const int W = (N + 31) >> 5;
    if (!c.bad)
#pragma unroll 1
      for (int r = u.r0 + tid; r < u.r0 + u.rows; r += kProcThreads) {
        unsigned* path = c.paths->row[r - u.r0];
#pragma unroll 1
        for (int w = 0; w < W; ++w) path[w] = 0u;
#pragma unroll 1
        for (int j = r - 1; j >= 0; j = __ldg(a.parents + (long long)u.b * N + j)) path[j >> 5] |= 1u << (j & 31);
      }
    __syncthreads();
  }
  __syncwarp();
}

// The occurrences of the chunk's token `off` among the drafts above row r.
__device__ __forceinline__ int proc_extra(const ProcessArgs& a, const ProcGather* g, const ProcPaths* paths, int b, int base,
                                       int r0, int off, int r) {
  int extra = 0;
  const unsigned* path = a.parents ? paths->row[r - r0] : nullptr;
  if (g->n_draft <= kProcDrafts) {
    for (int i = 0; i < g->n_draft; ++i) {
      const unsigned d = g->drafts[i];
      const int j = d & 0xffffu;
      extra += (int)(d >> 16) == off && (path ? (path[j >> 5] >> (j & 31) & 1u) : j < r);
    }
  } else {
    const int32_t* tok = a.drafts + (long long)b * (a.R - 1);
    for (int j = 0; j < r; ++j)  // the nodes above a row have lower indexes than it
      extra += __ldg(tok + j) == base + off && (!path || (path[j >> 5] >> (j & 31) & 1u));
  }
  return extra;
}

// What a listed token's logit z becomes: z up + add where z > 0, z down + add
// elsewhere.  -inf stays -inf, whatever is added: a masked vocabulary stays masked.
struct ProcTerm {
  float up, down, add;
  __device__ __forceinline__ float operator()(float z) const {
    return z == neg_inf() ? z : fmaf(z, z > 0.f ? up : down, add);
  }
};
__device__ __forceinline__ ProcTerm proc_term(const ProcShare& c, bool seen, float add) {
  return {seen ? c.inv : 1.f, seen ? c.rep : 1.f, add};
}
// ... of a token that some draft carries, in row r
__device__ __forceinline__ ProcTerm proc_draft_term(const ProcessArgs& a, const ProcUnit& u, const ProcShare& c,
                                                    unsigned entry, float add, int r) {
  const int extra = proc_extra(a, c.gather, c.paths, u.b, u.base, u.r0, entry & kProcOffset, r);
  if (extra) {
    add -= c.freq * (float)extra;
    if (!(entry & kProcCounted)) add -= c.pres;
  }
  return proc_term(c, (entry & kProcSeen) || extra, add);
}

// The terms that a lane has of its own (ProcShared::own) in row r.
__device__ __forceinline__ ProcTerm proc_own_term(const ProcessArgs& a, const ProcUnit& u, const ProcShare& c, int4 own, int r) {
  const int j = own.y;
  const bool on = j >= 0 && (a.parents ? (c.paths->row[r - u.r0][j >> 5] >> (j & 31) & 1u) : j < r);
  const int extra = __popc(__ballot_sync(0xffffffffu, on) & (unsigned)own.z);
  float add = __int_as_float(own.w);
  if (extra) {
    add -= c.freq * (float)extra;
    if (!(own.x & kProcCounted)) add -= c.pres;
  }
  return proc_term(c, (own.x & kProcSeen) || extra, add);
}

// kShifted: rows start off 16-byte boundaries (the vocabulary's size, or the
// buffers).  A row keeps its phase in shared memory: element t of the piece
// lies at phase + t.  The copies take the 16-byte vectors that hold the piece,
// the output is written in whole vectors and, at its ends, by single elements.
//
// The grid has a CTA for every unit, but those that start take over the ones
// that have not: a CTA goes from unit to unit, and each warp's ring of batches
// runs on across them, so that the rows of the next unit are under way while
// the lists of this one are made.  (One CTA per unit with the same passes: 343
// us for B = 256, R = 9, V = 152064 in bf16, everything on; equal shares for
// the CTAs of a persistent grid: 258 us, with SMs that are done early.)
template <class T, bool kShifted, bool kMask>
__global__ void __launch_bounds__(kProcThreads, 3) process_kernel(const __grid_constant__ ProcessArgs a) {
  using Ty = ProcType<T>;
  using S = typename Ty::storage;
  constexpr int VEC = Ty::kVec, RB = Ty::kBatch, NB = Ty::kBatches;
  constexpr int kVecs = kProcPiece / VEC / 32;  // vectors of a piece per lane
  constexpr unsigned kAll = (1u << VEC) - 1u;
  extern __shared__ __align__(16) unsigned char s_raw[];
  ProcCopyShared<T>& sh = *(ProcCopyShared<T>*)s_raw;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const S* in = (const S*)a.in;
  S* out = (S*)a.out;
  auto phase_of = [&](const ProcUnit& u, int i) { return kShifted ? (int)((u.row0 + (long long)i * a.V + a.phase) & (VEC - 1)) : 0; };
  const long long elements = (long long)a.B * a.R * a.V;
  auto stage = [&](int g, int j) { return sh.stages[warp].row[g % NB][j]; };

  if (lane == 0) {
    for (int k = 0; k < NB; ++k) mbar_init(&sh.full[warp][k], RB);
    if (warp == 0) {
      mbar_init(&sh.claimed[0], 1);
      mbar_init(&sh.claimed[1], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (warp == 0 && a.take_over) cta_request(&sh.claim[0], &sh.claimed[0]);
  }
  __syncwarp();

  ProcUnit u = proc_unit(a, blockIdx.x);
  int next = -1;  // the unit after it, once known

  // ---- the ring: the batches of a unit up to `most` set out, a lane with each row's copy ----
  long long load_row0 = u.row0;  // of the unit whose batch sets out next
  int load_rows = u.rows, load_tok = u.n_tok;
  bool load_ahead = false;  // ... which is the one after u
  int load_i = 0, load_g = 0;
  auto refill = [&](int most) {
    if (load_i >= load_rows) {
      if (load_ahead || next < 0) return;
      const ProcUnit v = proc_unit(a, (unsigned)next);
      load_row0 = v.row0, load_rows = v.rows, load_tok = v.n_tok;
      load_ahead = true;
      load_i = 0;
    }
    const int batches = min(most - load_g, (load_rows - load_i + RB - 1) / RB);
    if (lane < batches * RB) {
      // each of a batch's lanes arrives, with its row's bytes
      const int i = load_i + lane, s = (load_g + lane / RB) % NB;
      const long long row = load_row0 + (long long)i * a.V;
      int lo = 0, bytes = i < load_rows ? load_tok / VEC * 16 : 0, ph = 0;
      if constexpr (kShifted) {
        // the 16-byte vectors that hold the piece, but none past the input's ends
        ph = (int)((row + a.phase) & (VEC - 1));
        const int nv = (ph + load_tok + VEC - 1) / VEC;
        lo = row < ph;
        const int hi = row - ph + nv * VEC > elements;
        bytes = i < load_rows && load_tok > 0 ? max(nv - lo - hi, 0) * 16 : 0;
      }
      if (bytes) {
        mbar_arrive_tx(&sh.full[warp][s], (unsigned)bytes);
        bulk_load(sh.stages[warp].row[s][lane % RB] + lo * VEC, in + row - ph + lo * VEC, (unsigned)bytes, &sh.full[warp][s]);
      } else {
        mbar_arrive(&sh.full[warp][s]);
      }
    }
    load_i += batches * RB;
    load_g += batches;
  };
  refill(NB);

  // ---- masks of the next batch, one batch ahead ----
  // Lane w holds word w of the piece's mask, of the rows of a batch.
  auto mask_row = [&](const ProcUnit& u, int i) {
    return a.mask + ((long long)u.b * a.mask_rows + (a.mask_rows > 1 ? u.r0 + i : 0)) * a.W + (u.start >> 5);
  };
  auto allowed_at = [&](const ProcUnit& u, int i, int t) {
    return !kMask || (__ldg((const uint8_t*)mask_row(u, i) + (t >> 3)) >> (t & 7) & 1u);
  };
  unsigned next_word[RB];
  // A lane's element at the ends of a row's piece, in no whole vector of it: of
  // row lane / 16 of a batch, eight lanes those before the first vector, eight
  // those after the last.  From the boundary below the piece; -1 for none.
  const int edge_row = lane >> 4, edge_side = lane >> 3 & 1;
  auto edge_at = [&](const ProcUnit& u, int ph) {
    const int end = u.n_tok + ph, v1 = end / VEC;
    if (edge_side) return v1 * VEC + (lane & 7) < end && (v1 > 0 || ph == 0) ? v1 * VEC + (lane & 7) : -1;
    return (lane & 7) >= ph && ph > 0 && (lane & 7) < min(VEC, end) ? lane & 7 : -1;
  };
  auto look = [&](const ProcUnit& u, int batch) {
    if constexpr (kMask) {
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        const int i = batch * RB + j;
        next_word[j] = i < u.rows && 32 * lane < u.n_tok ? __ldg(mask_row(u, i) + lane) : 0xffffffffu;
      }
    }
  };

  look(u, 0);
  ProcAhead ahead = proc_ahead(a, u);
  proc_clear(sh.gather[0]);
  proc_counts(a, u, ahead);
  ProcShare c;
  c.paths = (ProcPaths*)(s_raw + sizeof(ProcCopyShared<T>));
  const unsigned short* list = sh.list + warp * kProcPiece;
  const unsigned tries = mbar_tries(spin_limit());
  constexpr unsigned kMostTries = mbar_tries(kSpinLimit);
  bool dead = false;
  int g = 0;
  for (unsigned round = 0;; ++round) {
    if (threadIdx.x == 0 && a.take_over) {
      // the unit after this one, asked for a round ago; and the one after that
      const unsigned k = round & 1;
      int answer = -1;
      bool came = mbar_test(&sh.claimed[k], (round >> 1) & 1);
#pragma unroll 1
      for (unsigned it = 0; !came && it < tries; ++it) came = mbar_try(&sh.claimed[k], (round >> 1) & 1);
      if (!came) {
        // out of time; but the answer has to have come before the CTA leaves
        atomicOr(a.status, kStatusTimeout);
#pragma unroll 1
        for (unsigned it = 0; !came && it < kMostTries; ++it) came = mbar_try(&sh.claimed[k], (round >> 1) & 1);
      }
      if (came) answer = cta_answer(&sh.claim[k]);
      sh.unit[k] = answer;
      if (answer >= 0) {
        fence_async();
        cta_request(&sh.claim[~round & 1], &sh.claimed[~round & 1]);
      }
    }
    __syncthreads();  // and every warp is done with the lists before
    if (a.take_over) next = sh.unit[round & 1];
    proc_lists(a, sh, sh.gather[round & 1], sh.gather[~round & 1], u, ahead, c);
    if (next >= 0) ahead = proc_ahead(a, proc_unit(a, (unsigned)next));
    for (int i0 = 0; i0 < u.rows; i0 += RB, ++g) {
      if (i0 + RB >= u.rows && next >= 0) proc_counts(a, proc_unit(a, (unsigned)next), ahead);
      const int n = min(RB, u.rows - i0);
      unsigned word[RB];
#pragma unroll
      for (int j = 0; j < RB; ++j) word[j] = kMask ? next_word[j] : 0xffffffffu;
      if (i0 + RB < u.rows)
        look(u, i0 / RB + 1);
      else if (next >= 0)
        look(proc_unit(a, (unsigned)next), 0);
      if (!dead && !warp_wait(&sh.full[warp][g % NB], (g / NB) & 1, tries)) {
        // a copy that never came: this warp hands out nothing more, and waits
        // for what is in flight, so that no copy outlives the CTA's memory
        if (lane == 0) atomicOr(a.status, kStatusTimeout);
#pragma unroll 1
        for (int q = g; q < load_g; ++q) warp_wait(&sh.full[warp][q % NB], (q / NB) & 1, kMostTries);
        dead = true;
      }
      if (dead) continue;
      int edge = -1, edge_ph = 0;
      if constexpr (kShifted) {
        if (edge_row < n) {
          edge_ph = phase_of(u, i0 + edge_row);
          edge = edge_at(u, edge_ph);
          // vectors that reach over the input's ends were not copied (a piece's
          // first vector may be the input's last)
          const long long from = u.row0 + (long long)(i0 + edge_row) * a.V - edge_ph + (edge & -VEC);
          if (edge >= 0 && (from < 0 || from + VEC > elements))
            stage(g, edge_row)[edge] = in[from + (edge & (VEC - 1))];
        }
        __syncwarp();
      }
      // the listed tokens, each for all rows of the batch
#pragma unroll 1
      for (int e = lane; e < c.n_list; e += 32) {
        const unsigned entry = list[e];
        const int off = entry & kProcOffset;
        const float add = sh.adj[off];
        S* x = stage(g, 0) + off - warp * kProcPiece;
        ProcTerm term = proc_term(c, entry & kProcSeen, add);
#pragma unroll
        for (int j = 0; j < RB; ++j)
          if (j < n) {
            if (entry & kProcDraft) term = proc_draft_term(a, u, c, entry, add, u.r0 + i0 + j);
            S* at = x + j * ProcStages<T>::kStage + phase_of(u, i0 + j);
            *at = Ty::round(term(Ty::widen(*at)));
          }
      }
      if (c.here && !c.bad) {
        const int4 own = sh.own[threadIdx.x];
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          const ProcTerm term = proc_own_term(a, u, c, own, u.r0 + i0 + j);
          if (own.x >= 0) {
            S* at = stage(g, j) + phase_of(u, i0 + j) + (own.x & kProcOffset) - warp * kProcPiece;
            *at = Ty::round(term(Ty::widen(*at)));
          }
        }
      }
      // the rows go out: shared -> registers, masked, -> global
      __syncwarp();
      if (c.bad) {
#pragma unroll 1
        for (int j = 0; j < n; ++j)
#pragma unroll 1
          for (int t = lane; t < u.n_tok; t += 32) out[u.row0 + (long long)(i0 + j) * a.V + t] = Ty::kNan;
      } else if (kShifted && a.split) {
        // the output's vectors lie at another phase: element by element
#pragma unroll 1
        for (int j = 0; j < n; ++j)
#pragma unroll 1
          for (int t = lane; t < u.n_tok; t += 32)
            out[u.row0 + (long long)(i0 + j) * a.V + t] =
                allowed_at(u, i0 + j, t) ? stage(g, j)[phase_of(u, i0 + j) + t] : Ty::kNegInf;
      } else {
#pragma unroll
        for (int j = 0; j < RB; ++j) {
          if (j >= n) break;
          const int ph = phase_of(u, i0 + j);
          unsigned& w = word[j];
          if constexpr (kShifted && kMask) {
            // the bits of the 16-byte lattice
            const unsigned below = __shfl_up_sync(0xffffffffu, w, 1);
            w = __funnelshift_l(lane ? below : 0xffffffffu, w, ph);
          }
          const uint4* x = (const uint4*)stage(g, j);
          S* to = out + u.row0 + (long long)(i0 + j) * a.V - ph;
          const int v0 = kShifted && ph ? 1 : 0, v1 = (u.n_tok + ph) / VEC;  // whole vectors of the piece
#pragma unroll
          for (int q = 0; q < kVecs; ++q) {
            const int v = 32 * q + lane;  // of the lattice
            const unsigned bits = kMask ? __shfl_sync(0xffffffffu, w, v * VEC >> 5) >> (v * VEC & 31) & kAll : kAll;
            if (v >= v0 && v < v1) {
              uint4 y = x[v];
              if (kMask && bits != kAll) y = proc_keep<T>(y, bits);
              *(uint4*)(to + v * VEC) = y;
            }
          }
        }
        if constexpr (kShifted) {
          bool on = true;
          if constexpr (kMask) {
#pragma unroll
            for (int j = 0; j < RB; ++j) {
              const unsigned w = __shfl_sync(0xffffffffu, word[j], max(edge, 0) >> 5);
              if (j == edge_row) on = w >> (edge & 31) & 1u;
            }
          }
          if (edge >= 0)
            out[u.row0 + (long long)(i0 + edge_row) * a.V - edge_ph + edge] = on ? stage(g, edge_row)[edge] : Ty::kNegInf;
        }
      }
      // the stages are free: the next batch goes there
      fence_async();
      __syncwarp();
      // (the next unit is known by then: its first batch sets out here at the latest)
      refill(g + 1 + NB);
    }
    if (next < 0) break;
    u = proc_unit(a, (unsigned)next);
    if (!load_ahead) {  // all of the unit before had set out
      load_row0 = u.row0, load_rows = u.rows, load_tok = u.n_tok;
      load_i = 0;
    }
    load_ahead = false;
    next = -1;
  }
}

// In place, the forbidden tokens: a warp takes 1024 tokens of one row, a lane
// their mask word; a vector that holds a forbidden token is read (unless all
// of it is forbidden) and written, no other is touched.  The bound is the
// traffic of the sectors that hold one (the other tokens of a vector are written
// as they were): 61 us for B = 256, R = 5, V = 128256
// in bf16 where a quarter of the rows is free and the others allow 0.2, 10 or
// 95 % (about 0.35 GB by that count; 104 us as a part of process_kernel).
constexpr int kMaskThreads = 128;
constexpr int kMaskPiece = 1024;
template <class T, bool kShifted>
__global__ void __launch_bounds__(kMaskThreads) process_mask_kernel(const __grid_constant__ ProcessArgs a) {
  using Ty = ProcType<T>;
  using S = typename Ty::storage;
  constexpr int VEC = Ty::kVec;
  constexpr int kVecs = kMaskPiece / VEC / 32;  // vectors of a piece per lane
  constexpr unsigned kAll = (1u << VEC) - 1u;
  const int lane = threadIdx.x & 31;
  const unsigned pieces = ((unsigned)a.V + kMaskPiece - 1) / kMaskPiece;
  const unsigned long long unit = (unsigned long long)blockIdx.x * (kMaskThreads / 32) + (threadIdx.x >> 5);
  const long long row = (long long)(unit / pieces);  // b R + r
  if (row >= (long long)a.B * a.R) return;
  const int start = (int)(unit - (unsigned long long)row * pieces) * kMaskPiece, n = min(kMaskPiece, a.V - start);
  const long long mrow = a.mask_rows > 1 ? row : row / a.R;
  const uint32_t* mask = a.mask + mrow * a.W + (start >> 5);
  unsigned w = 32 * lane < n ? __ldg(mask + lane) : 0xffffffffu;
  S* z = (S*)a.out + row * a.V + start;
  const int ph = kShifted ? (int)((row * a.V + start + a.phase) & (VEC - 1)) : 0;
  if (!__any_sync(0xffffffffu, w != 0xffffffffu)) return;
  if constexpr (kShifted) {
    // the elements before the first and after the last whole vector
    const int head = ph ? min(VEC - ph, n) : 0, tail = max(head, (n + ph) / VEC * VEC - ph);
    const int t = lane < 16 ? lane : tail + lane - 16;
    if ((lane < 16 ? t < head : t < n) && !(__ldg((const uint8_t*)mask + (t >> 3)) >> (t & 7) & 1u)) z[t] = Ty::kNegInf;
    // the bits of the 16-byte lattice
    const unsigned below = __shfl_up_sync(0xffffffffu, w, 1);
    w = __funnelshift_l(lane ? below : 0xffffffffu, w, ph);
  }
  const int v0 = ph ? 1 : 0, v1 = (n + ph) / VEC;
  uint4 x[kVecs];
  unsigned bits[kVecs];
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const int v = 32 * k + lane;
    bits[k] = __shfl_sync(0xffffffffu, w, v * VEC >> 5) >> (v * VEC & 31) & kAll;
    if (v < v0 || v >= v1) bits[k] = kAll;
    if (bits[k] != kAll && bits[k]) x[k] = *(const uint4*)(z - ph + v * VEC);
  }
#pragma unroll
  for (int k = 0; k < kVecs; ++k)
    if (bits[k] != kAll) *(uint4*)(z - ph + (32 * k + lane) * VEC) = proc_keep<T>(x[k], bits[k]);
}

// In place, the listed tokens (after the forbidden ones: what is not allowed is
// left alone).  A lane has an entry, for kProcRows rows at a time.  Each token
// costs the reading and writing of a sector, whatever else is in it: 178 us
// for B = 256, R = 9, V = 152064 in bf16 and histories of up to 8192 tokens
// (3 % of the tokens in 37 % of the sectors, 76 us by their bytes), 92 us with
// up to 512 tokens.
template <class T>
__global__ void __launch_bounds__(kProcThreads, 5) process_in_place_kernel(const __grid_constant__ ProcessArgs a) {
  using Ty = ProcType<T>;
  using S = typename Ty::storage;
  __shared__ __align__(16) ProcShared sh;
  __shared__ ProcPaths s_paths;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const ProcUnit u = proc_unit(a, blockIdx.x);
  ProcShare c;
  c.paths = &s_paths;
  {
    ProcAhead ahead = proc_ahead(a, u);
    proc_clear(sh.gather[0]);
    proc_counts(a, u, ahead);
    __syncthreads();
    proc_lists(a, sh, sh.gather[0], sh.gather[1], u, ahead, c);
  }
  S* z = (S*)a.out + u.row0;
  const int rows = u.n_tok > 0 ? u.rows : 0;
  if (c.bad) {
    for (int i = 0; i < rows; ++i)
      for (int t = lane; t < u.n_tok; t += 32) z[(long long)i * a.V + t] = Ty::kNan;
    return;
  }
  const uint32_t* mask0 =
      a.mask ? a.mask + ((long long)u.b * a.mask_rows + (a.mask_rows > 1 ? u.r0 : 0)) * a.W + (u.start >> 5) : nullptr;
  const int mask_step = a.mask_rows > 1 ? a.W : 0;
  auto allowed_at = [&](int i, int t) {
    return !mask0 || (__ldg((const uint8_t*)(mask0 + (long long)i * mask_step) + (t >> 3)) >> (t & 7) & 1u);
  };
  for (int e = lane; e < c.n_list; e += 32) {
    const unsigned entry = sh.list[warp * kProcPiece + e];
    const int t = (int)(entry & kProcOffset) - warp * kProcPiece;
    const float add = sh.adj[entry & kProcOffset];
    ProcTerm term = proc_term(c, entry & kProcSeen, add);
    for (int rb = 0; rb < rows; rb += kProcRows) {
      S* at = z + (long long)rb * a.V + t;
      unsigned on = 0;
      S v[kProcRows];
#pragma unroll
      for (int i = 0; i < kProcRows; ++i)
        if (rb + i < rows && allowed_at(rb + i, t)) {
          on |= 1u << i;
          v[i] = at[(long long)i * a.V];
        }
#pragma unroll
      for (int i = 0; i < kProcRows; ++i)
        if (on >> i & 1u) {
          if (entry & kProcDraft) term = proc_draft_term(a, u, c, entry, add, u.r0 + rb + i);
          at[(long long)i * a.V] = Ty::round(term(Ty::widen(v[i])));
        }
    }
  }
  if (c.here) {
    const int4 own = sh.own[threadIdx.x];
    const int t = (own.x & kProcOffset) - warp * kProcPiece;
    for (int i = 0; i < rows; ++i) {
      const ProcTerm term = proc_own_term(a, u, c, own, u.r0 + i);
      if (own.x >= 0 && allowed_at(i, t)) {
        S* at = z + (long long)i * a.V + t;
        *at = Ty::round(term(Ty::widen(*at)));
      }
    }
  }
}

int process_chunk() { return kProcChunk; }
int process_most_rows() { return kProcMostRows; }
int process_blocks_per_sm() { return 3; }

template <class T>
static int copy_smem(bool tree) { return (int)(sizeof(ProcCopyShared<T>) + (tree ? sizeof(ProcPaths) : 0)); }

template <class T>
static cudaError_t allow_smem() {
  cudaError_t e = cudaSuccess;
  auto one = [&](const void* f) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, copy_smem<T>(true));
  };
  one((const void*)process_kernel<T, false, false>);
  one((const void*)process_kernel<T, false, true>);
  one((const void*)process_kernel<T, true, false>);
  one((const void*)process_kernel<T, true, true>);
  return e;
}
cudaError_t process_configure() {
  cudaError_t e = count_configure();
  if (e == cudaSuccess) e = allow_smem<float>();
  if (e == cudaSuccess) e = allow_smem<Bf16Tag>();
  return e;
}

template <class T, bool kShifted, bool kMask>
static void launch_one(const ProcessArgs& a, int sms, cudaStream_t s) {
  const unsigned units = (unsigned)a.B * (unsigned)a.groups * (unsigned)a.chunks;
  if (a.in != a.out) {
    ProcessArgs k = a;
    k.take_over = units > (unsigned)(sms * process_blocks_per_sm());  // else all start at once
    process_kernel<T, kShifted, kMask><<<units, kProcThreads, copy_smem<T>(a.parents != nullptr), s>>>(k);
    return;
  }
  if (kMask) {
    const long long warps = (long long)a.B * a.R * ((a.V + kMaskPiece - 1) / kMaskPiece);
    process_mask_kernel<T, kShifted><<<(unsigned)((warps + kMaskThreads / 32 - 1) / (kMaskThreads / 32)), kMaskThreads, 0, s>>>(a);
  }
  if (a.state || a.drafts || a.n_bias || a.rep || a.freq || a.pres) process_in_place_kernel<T><<<units, kProcThreads, 0, s>>>(a);
}
template <class T>
static void launch_type(const ProcessArgs& a, bool shifted, int sms, cudaStream_t s) {
  if (shifted && a.mask)
    launch_one<T, true, true>(a, sms, s);
  else if (shifted)
    launch_one<T, true, false>(a, sms, s);
  else if (a.mask)
    launch_one<T, false, true>(a, sms, s);
  else
    launch_one<T, false, false>(a, sms, s);
}

cudaError_t launch_process(const ProcessArgs& a, bool bf16, int sms, cudaStream_t s) {
  const int esz = bf16 ? 2 : 4;
  const unsigned in_off = (unsigned)((uintptr_t)a.in & 15), out_off = (unsigned)((uintptr_t)a.out & 15);
  ProcessArgs k = a;
  k.turn_length = a.chunks > 3 ? a.chunks / 2 : 1;
  k.div_turn = make_fastdiv((uint32_t)k.turn_length);
  k.div_rest = make_fastdiv((uint32_t)(a.chunks > 1 ? a.chunks - 1 : 1));
  k.div_groups = make_fastdiv((uint32_t)a.groups);
  k.phase = (int)in_off / esz;
  k.split = in_off != out_off;
  const bool shifted = in_off || out_off || (long long)a.V * esz % 16;
  if (bf16)
    launch_type<Bf16Tag>(k, shifted, sms, s);
  else
    launch_type<float>(k, shifted, sms, s);
  return cudaGetLastError();
}

cudaError_t process_set_spin_limit(unsigned n) { return set_spin_limit_here(n); }

}  // namespace sv
