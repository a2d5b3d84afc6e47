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
// row group.  What the rows share is laid out once in shared memory: per token
// of the chunk the additive term of the history and the biases, and bitmaps of
// the tokens that something touches, that were seen, that occurred in the
// output and that a draft carries.  Then the chunk's logits stream through
// registers row by row; a vector that nothing touches is only masked.
constexpr int kProcThreads = 256;
constexpr int kProcWarps = kProcThreads / 32;
constexpr int kProcChunk = 4096;                     // tokens of a CTA's chunk
constexpr int kProcWords = kProcChunk / 32;          // ... in bitmap words
constexpr int kProcWarpToks = kProcChunk / kProcWarps;  // tokens whose biases one warp sums
constexpr int kProcMaxDrafts = 1024;
constexpr int kProcTreeRows = 32;  // rows of a group whose paths are kept as bit sets
static_assert(kProcThreads >= kProcWords, "one thread per bitmap word");
static_assert(kProcChunk % (2 * kProcThreads) == 0, "a half-word of the bitmap per thread");

struct ProcShared {
  float adj[kProcChunk];        // -f c - p [c > 0] + biases, without the drafts
  unsigned touch[kProcWords];   // history, draft or bias
  unsigned seen[kProcWords];    // history
  unsigned out[kProcWords];     // c > 0 without the drafts
  unsigned draft[kProcWords];   // some draft carries it
  unsigned list[kProcMaxDrafts];  // drafts in the chunk: (offset << 16) | node
  unsigned path[kProcTreeRows][kProcMaxDrafts / 32];  // tree: the nodes above each row of the group
  int n_list;
  int bad;
};

template <class T>
struct ProcType;
template <>
struct ProcType<float> {
  static constexpr int kVec = 4;
  using storage = uint32_t;
  static __device__ __forceinline__ float widen(uint32_t w) { return __uint_as_float(w); }
  static __device__ __forceinline__ uint32_t round(float f) { return __float_as_uint(f); }
  static constexpr uint32_t kNegInf = 0xff800000u, kNan = 0x7fc00000u;
};
struct Bf16Tag {};
template <>
struct ProcType<Bf16Tag> {
  static constexpr int kVec = 8;
  using storage = uint16_t;
  static __device__ __forceinline__ float widen(uint16_t w) { return __uint_as_float((uint32_t)w << 16); }
  static __device__ __forceinline__ uint16_t round(float f) {
    uint16_t r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(f));
    return r;
  }
  static constexpr uint16_t kNegInf = 0xff80u, kNan = 0x7fc0u;
};

template <class S, int VEC>
union ProcVec {
  S e[VEC];
  uint4 q;
};

// n bits (n a power of two <= 8) of a bitmap in shared memory from bit v on;
// v is a multiple of n
template <int N>
__device__ __forceinline__ unsigned bits_at(const unsigned* words, int v) {
  return (words[v >> 5] >> (v & 31)) & ((1u << N) - 1u);
}

template <class T, bool kVecPath, bool kInPlace>
__global__ void __launch_bounds__(kProcThreads) process_kernel(const __grid_constant__ ProcessArgs a) {
  using Ty = ProcType<T>;
  using S = typename Ty::storage;
  constexpr int VEC = kVecPath ? Ty::kVec : 1;
  constexpr int U = 4;  // vectors in flight per thread
  __shared__ ProcShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int unit = blockIdx.x;
  const int chunk = unit % a.chunks;
  unit /= a.chunks;
  const int group = unit % a.groups;
  const int b = unit / a.groups;
  const int base = chunk * kProcChunk;
  const int n_tok = min(kProcChunk, a.V - base);
  const int r0 = group * a.rows_per, r1 = min(a.R, r0 + a.rows_per);
  const float rep = a.rep ? __ldg(a.rep + b) : 1.f;
  const float freq = a.freq ? __ldg(a.freq + b) : 0.f;
  const float pres = a.pres ? __ldg(a.pres + b) : 0.f;
  const float inv = 1.f / rep;
  const int N = a.drafts ? a.R - 1 : 0;

  // ---- what the rows share ----
  const int32_t* state = a.state ? a.state + (long long)b * a.words : nullptr;
  if (tid == 0) {
    sh.n_list = 0;
    // a penalty that is no number, or a factor that is not positive
    sh.bad = !(rep > 0.f && rep < INFINITY) || !(fabsf(freq) < INFINITY) || !(fabsf(pres) < INFINITY);
  }
  if (tid < kProcWords) {
    const unsigned w = state && base + 32 * tid < a.P ? __ldg((const unsigned*)state + a.P + (base >> 5) + tid) : 0u;
    sh.touch[tid] = w;
    sh.seen[tid] = w;
    sh.draft[tid] = 0u;
    sh.out[tid] = 0u;
  }
  for (int i = tid; i < kProcChunk / 4; i += kProcThreads) ((float4*)sh.adj)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  {  // history: 16 tokens of the bitmap per thread
    unsigned w = (sh.seen[tid >> 1] >> (16 * (tid & 1))) & 0xffffu;
    unsigned counted = 0;
    while (w) {
      const int i = __ffs(w) - 1;
      w &= w - 1;
      const int off = 16 * tid + i;
      const int c = __ldg(state + base + off) & 0x7fffffff;
      if (c > 0) {
        sh.adj[off] = -freq * (float)c - pres;
        counted |= 1u << i;
      }
    }
    ((unsigned short*)sh.out)[tid] = (unsigned short)counted;
  }
  for (int j = tid; j < N; j += kProcThreads) {
    const int t = __ldg(a.drafts + (long long)b * N + j) - base;
    if (t >= 0 && t < n_tok) {
      sh.list[atomicAdd(&sh.n_list, 1)] = ((unsigned)t << 16) | (unsigned)j;
      atomicOr(&sh.draft[t >> 5], 1u << (t & 31));
      atomicOr(&sh.touch[t >> 5], 1u << (t & 31));
    }
    if (a.parents) {
      const int p = __ldg(a.parents + (long long)b * N + j);
      if (p < -1 || p >= j) sh.bad = 1;
    }
  }
  __syncthreads();
  if (a.n_bias > 0) {
    // each warp sums the biases of its own tokens, in the list's order
    const int lo = warp * kProcWarpToks;
    const long long at = (long long)b * a.n_bias;
    for (int i0 = 0; i0 < a.n_bias; i0 += 32) {
      const int i = i0 + lane;
      const int t = i < a.n_bias ? __ldg(a.bias_tokens + at + i) - base - lo : -1;
      const bool mine = t >= 0 && t < kProcWarpToks && lo + t < n_tok;
      const float v = mine ? __ldg(a.bias_values + at + i) : 0.f;
      for (unsigned m = __ballot_sync(0xffffffffu, mine); m; m &= m - 1) {
        const int l = __ffs(m) - 1;
        const int off = lo + __shfl_sync(0xffffffffu, t, l);
        const float x = __shfl_sync(0xffffffffu, v, l);
        if (lane == 0) {
          sh.adj[off] += x;
          sh.touch[off >> 5] |= 1u << (off & 31);
        }
      }
    }
  }
  const int n_list = sh.n_list;
  if (a.parents && n_list > 0 && !sh.bad) {
    // the nodes above each row of the group; a parent precedes its child
    const int W = (N + 31) >> 5;
    for (int r = r0 + tid; r < r1; r += kProcThreads) {
      unsigned* path = sh.path[r - r0];
      for (int w = 0; w < W; ++w) path[w] = 0u;
      for (int j = r - 1; j >= 0; j = __ldg(a.parents + (long long)b * N + j)) path[j >> 5] |= 1u << (j & 31);
    }
  }
  __syncthreads();
  const bool bad = sh.bad != 0;
  if (bad && tid == 0) atomicOr(a.status, kStatusBadData);

  // ---- the rows ----
  const S* in = (const S*)a.in;
  S* out = (S*)a.out;
  constexpr unsigned kAll = (1u << VEC) - 1u;
  for (int r = r0; r < r1; ++r) {
    const long long row = ((long long)b * a.R + r) * a.V + base;
    const uint8_t* mask =
        a.mask ? (const uint8_t*)(a.mask + ((long long)b * a.mask_rows + (a.mask_rows > 1 ? r : 0)) * a.W + (base >> 5))
               : nullptr;
    for (int v0 = tid * VEC; v0 < n_tok; v0 += U * kProcThreads * VEC) {
      ProcVec<S, VEC> x[U];
      unsigned allowed[U], touch[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * kProcThreads * VEC;
        allowed[u] = kAll;
        touch[u] = 0;
        if (v < n_tok) {
          if (mask) allowed[u] = ((unsigned)__ldg(mask + (v >> 3)) >> (v & 7)) & kAll;
          touch[u] = bits_at<VEC>(sh.touch, v);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * kProcThreads * VEC;
        if (v < n_tok && !(kInPlace && (allowed[u] == 0u || (allowed[u] == kAll && touch[u] == 0u)))) {
          if constexpr (kVecPath)
            x[u].q = *(const uint4*)(in + row + v);
          else
            x[u].e[0] = in[row + v];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * kProcThreads * VEC;
        if (v >= n_tok) continue;
        if (kInPlace && !bad && allowed[u] == kAll && touch[u] == 0u) continue;
        if (touch[u] & allowed[u]) {
          const unsigned seen = bits_at<VEC>(sh.seen, v), counted = bits_at<VEC>(sh.out, v);
          const unsigned draft = bits_at<VEC>(sh.draft, v);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            if (!(touch[u] >> e & 1u)) continue;
            float adj = sh.adj[v + e];
            bool hit = seen >> e & 1u;
            if (draft >> e & 1u) {
              int extra = 0;
              for (int i = 0; i < n_list; ++i) {
                const unsigned entry = sh.list[i];
                const int j = entry & 0xffffu;
                const bool on = a.parents ? (sh.path[r - r0][j >> 5] >> (j & 31) & 1u) : j < r;
                extra += (int)(entry >> 16) == v + e && on;
              }
              if (extra) {
                hit = true;
                adj -= freq * (float)extra;
                if (!(counted >> e & 1u)) adj -= pres;
              }
            }
            const float z = Ty::widen(x[u].e[e]);
            x[u].e[e] = Ty::round((hit ? (z > 0.f ? z * inv : z * rep) : z) + adj);
          }
        }
        if (allowed[u] != kAll) {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (!(allowed[u] >> e & 1u)) x[u].e[e] = Ty::kNegInf;
        }
        if (bad) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) x[u].e[e] = Ty::kNan;
        }
        if constexpr (kVecPath)
          *(uint4*)(out + row + v) = x[u].q;
        else
          out[row + v] = x[u].e[0];
      }
    }
  }
}

int process_chunk() { return kProcChunk; }
int process_tree_rows() { return kProcTreeRows; }

template <class T>
static void launch_one(const ProcessArgs& a, bool vec, unsigned grid, cudaStream_t s) {
  const bool in_place = a.in == a.out;
  if (vec && in_place)
    process_kernel<T, true, true><<<grid, kProcThreads, 0, s>>>(a);
  else if (vec)
    process_kernel<T, true, false><<<grid, kProcThreads, 0, s>>>(a);
  else if (in_place)
    process_kernel<T, false, true><<<grid, kProcThreads, 0, s>>>(a);
  else
    process_kernel<T, false, false><<<grid, kProcThreads, 0, s>>>(a);
}

cudaError_t launch_process(const ProcessArgs& a, bool bf16, bool vec, cudaStream_t s) {
  const unsigned grid = (unsigned)((long long)a.B * a.groups * a.chunks);
  if (bf16)
    launch_one<Bf16Tag>(a, vec, grid, s);
  else
    launch_one<float>(a, vec, grid, s);
  return cudaGetLastError();
}

}  // namespace sv
