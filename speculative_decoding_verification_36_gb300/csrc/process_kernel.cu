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
#include "sv_common.cuh"
#include "sv_kernels.h"

namespace sv {

// ---------------------------------------------------------------------------
// token counts
// ---------------------------------------------------------------------------
// state row of a sequence: P = V rounded up to 32 counts (bits 0..30: output
// tokens, bit 31: in the prompt), then P / 32 words with one bit per non-zero
// count.  The bitmap is what lets the processing kernel skip the counts of
// the tokens that never occurred: V / 8 bytes instead of 4 V.
constexpr int kCountThreads = 256;

__global__ void __launch_bounds__(kCountThreads) count_kernel(const __grid_constant__ CountArgs a) {
  const int b = blockIdx.y;
  const long long L = a.lengths ? a.lengths[b] : a.stride;
  const long long Lp = a.prompt_lengths ? a.prompt_lengths[b] : 0;
  if (L < 0 || L > a.stride || Lp < 0 || Lp > L) {
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

cudaError_t launch_count(const CountArgs& a, int sms, cudaStream_t s) {
  if (a.reset) {
    const cudaError_t e = cudaMemsetAsync(a.state, 0, (size_t)a.B * a.words * sizeof(int32_t), s);
    if (e != cudaSuccess) return e;
  }
  if (a.stride == 0) return cudaSuccess;
  const int per_row = (int)((a.stride + kCountThreads - 1) / kCountThreads);
  const int x = per_row < 4 * sms ? per_row : 4 * sms;
  for (int b0 = 0; b0 < a.B; b0 += 65535) {  // the grid's y extent
    CountArgs c = a;
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
// row group, in two passes.  The dense one copies the rows through registers
// and puts -inf where the mask forbids; it needs nothing but the masks, so it
// runs while the history's counts come in.  The sparse one visits only the
// tokens that the history, a bias or a draft touches (a few percent of the
// vocabulary under a long history), which the CTA lists once for all its rows:
// it reads each one's logit again (from L2: the dense pass has just been
// there), and writes the result over the copy.  In place the dense pass reads
// and writes only vectors that hold a forbidden token.
constexpr int kProcThreads = 256;
constexpr int kProcWarps = kProcThreads / 32;
constexpr int kProcChunk = 4096;                     // tokens of a CTA's chunk
constexpr int kProcWords = kProcChunk / 32;          // ... in bitmap words
constexpr int kProcWarpToks = kProcChunk / kProcWarps;  // tokens of one warp's threads
constexpr int kProcBatch = 4;                        // vectors in flight per thread
constexpr int kProcItems = 4;                        // listed logits in flight per thread
constexpr int kProcMaxDrafts = 1024;
constexpr int kProcDrafts = 256;   // drafts in a chunk that are listed; more are looked up in the input
constexpr int kProcTreeRows = 32;  // rows of a group whose paths are kept as bit sets
static_assert(kProcChunk == 16 * kProcThreads, "16 tokens per thread");
// list entries: offset, then
constexpr unsigned kProcSeen = 1u << 12;     // in the history
constexpr unsigned kProcCounted = 1u << 13;  // c > 0 without the drafts
constexpr unsigned kProcDraft = 1u << 14;    // some draft carries it
constexpr unsigned kProcOffset = kProcSeen - 1u;
static_assert(kProcChunk <= (int)kProcSeen, "an offset leaves the flags free");

struct ProcShared {
  float adj[kProcChunk];             // listed tokens: -f c - p [c > 0] + biases, without the drafts
  unsigned short list[kProcChunk];   // in no particular order
  unsigned bias[kProcWords];         // tokens with a bias
  unsigned draft[kProcWords];        // tokens that some draft carries
  unsigned drafts[kProcDrafts];      // drafts in the chunk: (offset << 16) | node
  unsigned path[kProcTreeRows][kProcMaxDrafts / 32];  // tree: the nodes above each row of the group
  int n_list, n_draft;
  int twice;  // a token with several biases
  int bad;
};

struct Bf16Tag {};
template <class T>
struct ProcType;
template <>
struct ProcType<float> {
  using storage = uint32_t;
  static constexpr int kVec = 4;
  static constexpr uint32_t kNegInf = 0xff800000u, kNan = 0x7fc00000u;
  static __device__ __forceinline__ float widen(uint32_t w) { return __uint_as_float(w); }
  static __device__ __forceinline__ uint32_t round(float f) { return __float_as_uint(f); }
};
template <>
struct ProcType<Bf16Tag> {
  using storage = uint16_t;
  static constexpr int kVec = 8;
  static constexpr uint16_t kNegInf = 0xff80u, kNan = 0x7fc0u;
  static __device__ __forceinline__ float widen(uint16_t w) { return __uint_as_float((uint32_t)w << 16); }
  static __device__ __forceinline__ uint16_t round(float f) {
    uint16_t r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(f));
    return r;
  }
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
    auto one = [](uint32_t w, uint32_t b) {
      const uint32_t keep = (b & 1u) * 0xffffu + (b & 2u) * 0x7fff8000u;  // each bit widened to 16
      return (w & keep) | (fill & ~keep);
    };
    x.x = one(x.x, bits), x.y = one(x.y, bits >> 2), x.z = one(x.z, bits >> 4), x.w = one(x.w, bits >> 6);
  }
  return x;
}

// The occurrences of the chunk's token `off` among the drafts above row r.
__device__ __forceinline__ int proc_extra(const ProcessArgs& a, const ProcShared& sh, int b, int base, int off, int r,
                                          int r0) {
  int extra = 0;
  const unsigned* path = a.parents ? sh.path[r - r0] : nullptr;
  if (sh.n_draft <= kProcDrafts) {
    for (int i = 0; i < sh.n_draft; ++i) {
      const unsigned d = sh.drafts[i];
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

template <class T, bool kShifted, bool kInPlace>
__global__ void __launch_bounds__(kProcThreads) process_kernel(const __grid_constant__ ProcessArgs a) {
  using Ty = ProcType<T>;
  using S = typename Ty::storage;
  constexpr int VEC = Ty::kVec;
  constexpr unsigned kAll = (1u << VEC) - 1u;
  constexpr int kPer = kProcChunk / (kProcThreads * VEC);  // vectors per thread and row
  constexpr int RU = kProcBatch / kPer;                    // rows of a batch
  static_assert(kProcBatch % kPer == 0, "whole rows in flight");
  __shared__ __align__(16) ProcShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int unit = blockIdx.x;
  const int chunk = unit % a.chunks;
  unit /= a.chunks;
  const int group = unit % a.groups;
  const int b = unit / a.groups;
  const int base = chunk * kProcChunk;
  const int n_tok = min(kProcChunk, a.V - base);
  const int r0 = group * a.rows_per, r1 = min(a.R, r0 + a.rows_per);
  const int N = a.drafts ? a.R - 1 : 0;
  const S* in = (const S*)a.in;
  S* out = (S*)a.out;

  // ---- what the history, the drafts and the biases hold of the chunk ----
  const int32_t* state = a.state ? a.state + (long long)b * a.words : nullptr;
  unsigned mine = 0;  // the bitmap of the thread's 16 tokens
  if (state && base + 16 * tid < a.P) mine = __ldg((const unsigned short*)(state + a.P) + (base >> 4) + tid);
  if (tid < kProcWords) {
    sh.bias[tid] = 0u;
    sh.draft[tid] = 0u;
  }
  if (tid == 0) sh.n_list = sh.n_draft = sh.twice = sh.bad = 0;
  int count[16];  // all at once: one trip to memory
#pragma unroll
  for (int i = 0; i < 16; ++i) count[i] = mine >> i & 1u ? __ldg(state + base + 16 * tid + i) : 0;
  __syncthreads();
  for (int j = tid; j < N; j += kProcThreads) {
    const int t = __ldg(a.drafts + (long long)b * N + j) - base;
    if (t >= 0 && t < n_tok) {
      const int at = atomicAdd(&sh.n_draft, 1);
      if (at < kProcDrafts) sh.drafts[at] = ((unsigned)t << 16) | (unsigned)j;
      atomicOr(&sh.draft[t >> 5], 1u << (t & 31));
    }
    if (a.parents) {
      const int p = __ldg(a.parents + (long long)b * N + j);
      if (p < -1 || p >= j) sh.bad = 1;
    }
  }
  for (int i = tid; i < a.n_bias; i += kProcThreads) {
    const int t = __ldg(a.bias_tokens + (long long)b * a.n_bias + i) - base;
    if (t >= 0 && t < n_tok) {
      if (atomicOr(&sh.bias[t >> 5], 1u << (t & 31)) >> (t & 31) & 1u)
        sh.twice = 1;
      else
        sh.adj[t] = __ldg(a.bias_values + (long long)b * a.n_bias + i);
    }
  }

  // ---- dense pass: copy and mask ----
  auto row_at = [&](int r) { return ((long long)b * a.R + r) * a.V + base; };
  const uint32_t* mask0 = a.mask ? a.mask + (long long)b * a.mask_rows * a.W + (base >> 5) : nullptr;
  const int mask_step = a.mask_rows > 1 ? a.W : 0;
  const int mask_end = 4 * (a.W - (base >> 5));  // bytes of a mask row from the chunk on
  auto mask_row = [&](int r) { return (const uint8_t*)(mask0 + (long long)r * mask_step); };
  auto allowed_at = [&](int r, int t) { return !mask0 || (__ldg(mask_row(r) + (t >> 3)) >> (t & 7) & 1u); };
  // elements of a row's part of the chunk before its first 16-byte boundary
  auto head_of = [&](int r) {
    if constexpr (!kShifted) return 0;
    const int off = (int)((row_at(r) + a.phase) & (VEC - 1));
    return min(off ? VEC - off : 0, n_tok);
  };
  if (a.split) {
    // the output's vectors lie at another phase than the input's: single elements
    for (int r = r0; r < r1; ++r)
#pragma unroll 4
      for (int t = tid; t < n_tok; t += kProcThreads) {
        const S x = in[row_at(r) + t];
        out[row_at(r) + t] = allowed_at(r, t) ? x : Ty::kNegInf;
      }
  } else if (!kInPlace || mask0) {
    for (int rb = r0; rb < r1; rb += RU) {
      uint4 x[RU][kPer];
      unsigned allowed[RU][kPer];
      int at[RU][kPer];  // -1: no work here
#pragma unroll
      for (int i = 0; i < RU; ++i)
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
          const int r = rb + i, v = (p * kProcThreads + tid) * VEC + (r < r1 ? head_of(r) : 0);
          at[i][p] = r < r1 && v + VEC <= n_tok ? v : -1;
          allowed[i][p] = kAll;
          if (mask0 && at[i][p] >= 0) {
            const uint8_t* m = mask_row(r) + (v >> 3);
            unsigned w = __ldg(m);
            if (kShifted && (v & 7) > 8 - VEC) w |= (unsigned)__ldg(m + ((v >> 3) + 1 < mask_end ? 1 : 0)) << 8;
            allowed[i][p] = w >> (v & 7) & kAll;
          }
        }
#pragma unroll
      for (int i = 0; i < RU; ++i)
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
          if (kInPlace && allowed[i][p] == kAll) at[i][p] = -1;
          if (at[i][p] >= 0 && !(kInPlace && allowed[i][p] == 0u)) x[i][p] = *(const uint4*)(in + row_at(rb + i) + at[i][p]);
        }
#pragma unroll
      for (int i = 0; i < RU; ++i)
#pragma unroll
        for (int p = 0; p < kPer; ++p)
          if (at[i][p] >= 0) {
            if (allowed[i][p] != kAll) x[i][p] = proc_keep<T>(x[i][p], allowed[i][p]);
            *(uint4*)(out + row_at(rb + i) + at[i][p]) = x[i][p];
          }
    }
    if constexpr (kShifted) {
      // the elements before the first and after the last whole vector of each row
      for (int r = r0 + warp; r < r1; r += kProcWarps) {
        const int head = head_of(r), tail = head + (n_tok - head) / VEC * VEC;
        const int t = lane < 16 ? lane : tail + lane - 16;
        if (lane < 16 ? t >= head : t >= n_tok) continue;
        out[row_at(r) + t] = allowed_at(r, t) ? in[row_at(r) + t] : Ty::kNegInf;
      }
    }
  }

  // ---- the list ----
  const float rep = a.rep ? __ldg(a.rep + b) : 1.f;
  const float freq = a.freq ? __ldg(a.freq + b) : 0.f;
  const float pres = a.pres ? __ldg(a.pres + b) : 0.f;
  const float inv = 1.f / rep;
  // a penalty that is no number, or a factor that is not positive
  if (!(rep > 0.f && rep < INFINITY) || !(fabsf(freq) < INFINITY) || !(fabsf(pres) < INFINITY)) sh.bad = 1;
  __syncthreads();
  if (sh.bad) {
    if (tid == 0) atomicOr(a.status, kStatusBadData);
    for (int r = r0; r < r1; ++r)
      for (int t = tid; t < n_tok; t += kProcThreads) out[row_at(r) + t] = Ty::kNan;
    return;
  }
  if (sh.twice) {
    // some token has several biases: each warp sums those of its own tokens,
    // in the list's order
    const int lo = warp * kProcWarpToks;
    const long long first = (long long)b * a.n_bias;
    for (int i = lane; i < kProcWarpToks; i += 32) sh.adj[lo + i] = 0.f;
    __syncwarp();
    for (int i0 = 0; i0 < a.n_bias; i0 += 32) {
      const int i = i0 + lane;
      const int t = i < a.n_bias ? __ldg(a.bias_tokens + first + i) - base - lo : -1;
      const bool own = t >= 0 && t < kProcWarpToks && lo + t < n_tok;
      const float v = own ? __ldg(a.bias_values + first + i) : 0.f;
      for (unsigned m = __ballot_sync(0xffffffffu, own); m; m &= m - 1) {
        const int l = __ffs(m) - 1;
        const int off = lo + __shfl_sync(0xffffffffu, t, l);
        const float x = __shfl_sync(0xffffffffu, v, l);
        if (lane == 0) sh.adj[off] += x;
      }
    }
    __syncwarp();
  }
  {
    static_assert(kProcWarpToks == 16 * 32, "a warp's threads hold the warp's tokens");
    const unsigned bias = (sh.bias[tid >> 1] >> (16 * (tid & 1))) & 0xffffu;
    const unsigned draft = (sh.draft[tid >> 1] >> (16 * (tid & 1))) & 0xffffu;
    const unsigned touch = mine | bias | draft;
    if (touch) {
      int at = atomicAdd(&sh.n_list, __popc(touch));
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (touch >> i & 1u) {
          const int off = 16 * tid + i, n = count[i] & 0x7fffffff;
          float adj = bias >> i & 1u ? sh.adj[off] : 0.f;
          if (n > 0) adj += -freq * (float)n - pres;
          sh.adj[off] = adj;
          sh.list[at++] = (unsigned short)(off | (mine >> i & 1u ? kProcSeen : 0u) | (n > 0 ? kProcCounted : 0u) |
                                           (draft >> i & 1u ? kProcDraft : 0u));
        }
    }
  }
  if (a.parents && sh.n_draft > 0) {
    // the nodes above each row of the group; a parent precedes its child
    const int W = (N + 31) >> 5;
    for (int r = r0 + tid; r < r1; r += kProcThreads) {
      unsigned* path = sh.path[r - r0];
      for (int w = 0; w < W; ++w) path[w] = 0u;
      for (int j = r - 1; j >= 0; j = __ldg(a.parents + (long long)b * N + j)) path[j >> 5] |= 1u << (j & 31);
    }
  }
  __syncthreads();

  // ---- sparse pass: 32 entries of one row per step of a warp ----
  const int n_list = sh.n_list, blocks = (n_list + 31) >> 5, steps = blocks * (r1 - r0);
  for (int k0 = warp; k0 < steps; k0 += kProcItems * kProcWarps) {
    unsigned entry[kProcItems];
    int row[kProcItems];  // -1: nothing to do
    S z[kProcItems];
#pragma unroll
    for (int i = 0; i < kProcItems; ++i) {
      const int k = k0 + i * kProcWarps;
      const int r = (int)((unsigned)k / (unsigned)blocks), e = (k - r * blocks) * 32 + lane;
      row[i] = -1;
      if (k < steps && e < n_list) {
        entry[i] = sh.list[e];
        if (allowed_at(r0 + r, entry[i] & kProcOffset)) row[i] = r0 + r;
      }
    }
#pragma unroll
    for (int i = 0; i < kProcItems; ++i)
      if (row[i] >= 0) z[i] = in[row_at(row[i]) + (entry[i] & kProcOffset)];
#pragma unroll
    for (int i = 0; i < kProcItems; ++i)
      if (row[i] >= 0) {
        const int off = entry[i] & kProcOffset;
        float adj = sh.adj[off];
        bool seen = entry[i] & kProcSeen;
        if (entry[i] & kProcDraft) {
          const int extra = proc_extra(a, sh, b, base, off, row[i], r0);
          if (extra) {
            seen = true;
            adj -= freq * (float)extra;
            if (!(entry[i] & kProcCounted)) adj -= pres;
          }
        }
        const float x = Ty::widen(z[i]);
        out[row_at(row[i]) + off] = Ty::round((seen ? (x > 0.f ? x * inv : x * rep) : x) + adj);
      }
  }
}

int process_chunk() { return kProcChunk; }
int process_tree_rows() { return kProcTreeRows; }

template <class T>
static void launch_one(const ProcessArgs& a, bool shifted, unsigned grid, cudaStream_t s) {
  const bool in_place = a.in == a.out;
  if (shifted && in_place)
    process_kernel<T, true, true><<<grid, kProcThreads, 0, s>>>(a);
  else if (shifted)
    process_kernel<T, true, false><<<grid, kProcThreads, 0, s>>>(a);
  else if (in_place)
    process_kernel<T, false, true><<<grid, kProcThreads, 0, s>>>(a);
  else
    process_kernel<T, false, false><<<grid, kProcThreads, 0, s>>>(a);
}

cudaError_t launch_process(const ProcessArgs& a, bool bf16, cudaStream_t s) {
  const unsigned grid = (unsigned)((long long)a.B * a.groups * a.chunks);
  const int esz = bf16 ? 2 : 4;
  const unsigned in_off = (unsigned)((uintptr_t)a.in & 15), out_off = (unsigned)((uintptr_t)a.out & 15);
  ProcessArgs k = a;
  k.phase = (int)in_off / esz;
  k.split = in_off != out_off;
  const bool shifted = in_off || (long long)a.V * esz % 16;
  if (bf16)
    launch_one<Bf16Tag>(k, shifted, grid, s);
  else
    launch_one<float>(k, shifted, grid, s);
  return cudaGetLastError();
}

}  // namespace sv
