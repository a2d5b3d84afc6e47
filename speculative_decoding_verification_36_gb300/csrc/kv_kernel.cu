// kv_kernel.cu -- the paged key/value cache around a verify step: the step's
// keys and values go in rotated to their positions, and after a tree verify
// the accepted path's entries move to consecutive slots.
//
// The target's forward pass of a verify step takes the last committed token
// (the root) and the drafts.  Token i of sequence b goes to slot
// lengths[b] + i; its position is lengths[b] + depth(i), where a chain's depth
// is i and a tree's is the node's level (0 for the root, token 0; node j is
// token j + 1).  Siblings therefore share a position and a rotation, and no
// entry has to be turned again when it moves.
//
// Rotation by theta = 2 pi frac(pos f): the frequencies come as 64-bit
// fractions of a turn, so pos * f modulo 2^64 is exactly the fraction of a
// turn left after the whole ones, for every position; its top 32 bits go to
// sincospi.  No table of angles is read and no far position loses digits.
#include "sv_common.cuh"
#include "sv_kernels.h"

namespace sv {

constexpr int kKvThreads = 256;
constexpr int kKvTokens = 4;  // tokens of a CTA

template <class S>
__device__ __forceinline__ float kv_widen(S w);
template <>
__device__ __forceinline__ float kv_widen<uint32_t>(uint32_t w) { return __uint_as_float(w); }
template <>
__device__ __forceinline__ float kv_widen<uint16_t>(uint16_t w) { return __uint_as_float((uint32_t)w << 16); }
template <class S>
__device__ __forceinline__ S kv_round(float f);
template <>
__device__ __forceinline__ uint32_t kv_round<uint32_t>(float f) { return __float_as_uint(f); }
template <>
__device__ __forceinline__ uint16_t kv_round<uint16_t>(float f) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(f));
  return r;
}

template <class S, int VEC>
struct alignas(sizeof(S) * VEC) KvVec {
  S e[VEC];
};

// One token's place, as a CTA works it out for its tokens.
struct KvToken {
  long long dst;  // element offset of its entry in the caches, -1: not written
  int state;      // 0: behind the sequence's new tokens, 1: valid, 2: bad sequence
};

// Shared memory: the tokens, then cos and sin [kKvTokens][rot / 2].
template <class S, int VEC>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const __grid_constant__ KvAppendArgs a) {
  extern __shared__ __align__(16) float2 s_cs[];
  __shared__ KvToken s_tok[kKvTokens];
  __shared__ unsigned long long s_pos[kKvTokens];
  using V = KvVec<S, VEC>;
  const int tid = threadIdx.x;
  const long long first = (long long)blockIdx.x * kKvTokens;
  const int n = (int)min((long long)kKvTokens, (long long)a.B * a.T - first);
  if (tid < n) {
    const long long g = first + tid;
    const int b = (int)(g / a.T), i = (int)(g - (long long)b * a.T);
    const long long len = __ldg(a.lengths + b);
    const int n_new = a.n_new ? __ldg(a.n_new + b) : a.T;
    KvToken t = {-1, 1};
    int depth = i;
    if (len < 0 || n_new < 0 || n_new > a.T || len + n_new > (long long)a.max_pages * a.page_size) t.state = 2;
    if (a.parents) {
      // every parent of the sequence has to precede its node
      const int32_t* par = a.parents + (long long)b * (a.T - 1);
      for (int j = 0; j < a.T - 1; ++j) {
        const int p = __ldg(par + j);
        if (p < -1 || p >= j) t.state = 2;
      }
      depth = 0;
      if (t.state != 2)
        for (int j = i - 1; j >= 0; j = __ldg(par + j)) ++depth;
    }
    if (t.state == 1 && i >= n_new) t.state = 0;
    if (t.state == 1) {
      const long long slot = len + i;
      const int page = __ldg(a.page_table + (long long)b * a.max_pages + slot / a.page_size);
      if (page < 0 || page >= a.pages)
        atomicOr(a.status, kStatusBadData);
      else
        t.dst = ((long long)page * a.page_size + slot % a.page_size) * a.Hkv * a.D;
    }
    if (t.state == 2) atomicOr(a.status, kStatusBadData);
    s_tok[tid] = t;
    s_pos[tid] = (unsigned long long)(len + depth);
  }
  __syncthreads();
  const int half = a.rot / 2;
  for (int x = tid; x < n * half; x += kKvThreads) {
    const int t = x / half, f = x - t * half;
    const unsigned long long turn = s_pos[t] * __ldg(a.turns + f);
    float s, c;
    // the fraction of a turn in [-1/2, 1/2); half turns in, radians / pi
    sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f, &s, &c);
    s_cs[x] = make_float2(c, s);
  }
  __syncthreads();

  // items of a token: per head of K and Q the rotated vectors (pairs of
  // vectors when the halves rotate against each other) and the plain ones,
  // per head of V the plain ones
  const int rot_items = a.interleaved ? a.rot / (VEC > 1 ? VEC : 2) : half / VEC;
  const int head_items = rot_items + (a.D - a.rot) / VEC;
  const int k_items = a.Hkv * head_items, q_items = a.Hq * head_items, v_items = a.Hkv * (a.D / VEC);
  const int items = k_items + q_items + v_items;
  for (int x = tid; x < n * items; x += kKvThreads) {
    const int t = x / items;
    int it = x - t * items;
    const KvToken tok = s_tok[t];
    if (tok.state == 0) continue;
    const long long g = first + t;
    if (it >= k_items + q_items) {
      it -= k_items + q_items;
      if (tok.dst >= 0) *(V*)((S*)a.v_cache + tok.dst + it * VEC) = *(const V*)((const S*)a.v + g * a.kv_stride + it * VEC);
      continue;
    }
    const bool is_q = it >= k_items;
    if (is_q) it -= k_items;
    const int head = it / head_items, j = it - head * head_items;
    const S* src = is_q ? (const S*)a.q + g * a.q_stride + head * a.D : (const S*)a.k + g * a.kv_stride + head * a.D;
    S* dst = is_q ? (S*)a.out_q + (g * a.Hq + head) * a.D : (S*)a.k_cache + tok.dst + head * a.D;
    if (!is_q && tok.dst < 0) continue;
    const bool nan = tok.state == 2;  // a bad sequence's queries
    const float2* cs = s_cs + t * half;
    if (j >= rot_items) {
      const int e = a.rot + (j - rot_items) * VEC;
      V v = *(const V*)(src + e);
      if (nan)
#pragma unroll
        for (int i = 0; i < VEC; ++i) v.e[i] = kv_round<S>(NAN);
      *(V*)(dst + e) = v;
    } else if (a.interleaved) {
      if constexpr (VEC > 1) {
        V v = *(const V*)(src + j * VEC);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
          const float2 w = cs[j * (VEC / 2) + i];
          const float p = kv_widen<S>(v.e[2 * i]), q = kv_widen<S>(v.e[2 * i + 1]);
          v.e[2 * i] = kv_round<S>(nan ? NAN : p * w.x - q * w.y);
          v.e[2 * i + 1] = kv_round<S>(nan ? NAN : p * w.y + q * w.x);
        }
        *(V*)(dst + j * VEC) = v;
      } else {
        const float2 w = cs[j];
        const float p = kv_widen<S>(src[2 * j]), q = kv_widen<S>(src[2 * j + 1]);
        dst[2 * j] = kv_round<S>(nan ? NAN : p * w.x - q * w.y);
        dst[2 * j + 1] = kv_round<S>(nan ? NAN : p * w.y + q * w.x);
      }
    } else {
      V lo = *(const V*)(src + j * VEC), hi = *(const V*)(src + half + j * VEC);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float2 w = cs[j * VEC + i];
        const float p = kv_widen<S>(lo.e[i]), q = kv_widen<S>(hi.e[i]);
        lo.e[i] = kv_round<S>(nan ? NAN : p * w.x - q * w.y);
        hi.e[i] = kv_round<S>(nan ? NAN : p * w.y + q * w.x);
      }
      *(V*)(dst + j * VEC) = lo;
      *(V*)(dst + half + j * VEC) = hi;
    }
  }
}

int kv_max_rot() { return 1024; }

cudaError_t launch_kv_append(const KvAppendArgs& a, bool bf16, bool vec, cudaStream_t s) {
  const unsigned grid = (unsigned)(((long long)a.B * a.T + kKvTokens - 1) / kKvTokens);
  const size_t smem = (size_t)kKvTokens * (a.rot / 2) * sizeof(float2);
  if (bf16 && vec)
    kv_append_kernel<uint16_t, 8><<<grid, kKvThreads, smem, s>>>(a);
  else if (bf16)
    kv_append_kernel<uint16_t, 1><<<grid, kKvThreads, smem, s>>>(a);
  else if (vec)
    kv_append_kernel<uint32_t, 4><<<grid, kKvThreads, smem, s>>>(a);
  else
    kv_append_kernel<uint32_t, 1><<<grid, kKvThreads, smem, s>>>(a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// commit
// ---------------------------------------------------------------------------
// One CTA per (sequence, layer, cache).  It finds the path's nodes level by
// level (a node is on level d when its parent is on level d - 1 and it carries
// the path's d-th token), takes the lowest node of the last level and its
// ancestors, and moves the entries: slot len + 1 + node_d to slot len + d.
// node_d >= d - 1, so moving in ascending order never overwrites an entry that
// is still to be read; each thread keeps that order for its own bytes.
constexpr int kCommitThreads = 256;
constexpr int kCommitBatch = 4;  // entries in flight per thread

template <class V>
__global__ void __launch_bounds__(kCommitThreads) kv_commit_kernel(const __grid_constant__ KvCommitArgs a) {
  __shared__ short s_level[kMaxTreeNodes];     // 1-based level, 0: not on the path
  __shared__ int s_node[kMaxTreeNodes];        // the path's nodes, by level
  __shared__ long long s_slot[2][kMaxTreeNodes];  // byte offsets: to, from
  __shared__ int s_last;
  const int tid = threadIdx.x;
  const int b = blockIdx.x;
  const int layer = blockIdx.y >> 1, which = blockIdx.y & 1;
  const int N = a.N;
  const int32_t* tok = a.tokens + (long long)b * N;
  const int32_t* par = a.parents + (long long)b * N;
  const int32_t* path = a.path + (long long)b * (N + 1);
  const int size = __ldg(a.path_len + b);
  const long long len = __ldg(a.lengths + b);
  const int n = size > 0 ? size - 1 : 0;
  const long long most = min((long long)a.max_pages * a.page_size, 2147483647LL);
  // every verdict below is the whole CTA's: the barriers stay uniform
  bool bad = size != -1 && (size < 1 || n > N || len < 0 || len + N + 1 > most);
  const bool go = size != -1 && !bad;
  if (go) {
    if (tid == 0) s_last = N;
    bool wrong = false;
    for (int j = tid; j < N; j += kCommitThreads) {
      s_level[j] = 0;
      const int p = __ldg(par + j);
      wrong |= p < -1 || p >= j;
    }
    bad = __syncthreads_or(wrong);
  }
  if (go && !bad) {
    for (int d = 1; d <= n; ++d) {
      const int want = __ldg(path + d - 1);
      for (int j = tid; j < N; j += kCommitThreads) {
        const int p = __ldg(par + j);
        if ((d == 1 ? p == -1 : p >= 0 && s_level[p] == d - 1) && __ldg(tok + j) == want) {
          s_level[j] = (short)d;
          if (d == n) atomicMin(&s_last, j);
        }
      }
      __syncthreads();
    }
    bad = n > 0 && s_last >= N;  // no path of the tree carries these tokens
  }
  if (go && !bad) {
    if (tid == 0 && n > 0)
      for (int j = s_last, d = n; d >= 1; --d, j = __ldg(par + j)) s_node[d - 1] = j;
    __syncthreads();
    bool wrong = false;
    for (int d = tid; d < n; d += kCommitThreads) {
      const long long to = len + 1 + d, from = len + 1 + s_node[d];
      const int32_t* table = a.page_table + (long long)b * a.max_pages;
      const int p0 = __ldg(table + to / a.page_size), p1 = __ldg(table + from / a.page_size);
      wrong |= p0 < 0 || p0 >= a.pages || p1 < 0 || p1 >= a.pages;
      s_slot[0][d] = ((long long)p0 * a.page_size + to % a.page_size) * a.entry_bytes;
      s_slot[1][d] = ((long long)p1 * a.page_size + from % a.page_size) * a.entry_bytes;
    }
    bad = __syncthreads_or(wrong);
  }
  if (blockIdx.y == 0) {
    for (int d = tid; d <= N; d += kCommitThreads) a.out_nodes[(long long)b * (N + 1) + d] = go && !bad && d < n ? s_node[d] : -1;
    if (tid == 0) {
      a.out_lengths[b] = (int)(go && !bad ? len + size : len);
      if (bad) atomicOr(a.status, kStatusBadData);
    }
  }
  if (!go || bad) return;
  char* cache = (char*)(which ? a.v_cache : a.k_cache) + (long long)layer * a.layer_bytes;
  const int vecs = a.entry_bytes / (int)sizeof(V);
  for (int x = tid; x < vecs; x += kCommitThreads) {
    for (int d0 = 0; d0 < n; d0 += kCommitBatch) {
      V v[kCommitBatch];
#pragma unroll
      for (int i = 0; i < kCommitBatch; ++i)
        if (d0 + i < n) v[i] = ((const V*)(cache + s_slot[1][d0 + i]))[x];
#pragma unroll
      for (int i = 0; i < kCommitBatch; ++i)
        if (d0 + i < n) ((V*)(cache + s_slot[0][d0 + i]))[x] = v[i];
    }
  }
}

cudaError_t launch_kv_commit(const KvCommitArgs& a, int vec_bytes, cudaStream_t s) {
  const dim3 grid((unsigned)a.B, (unsigned)(2 * a.layers));
  if (vec_bytes == 16)
    kv_commit_kernel<uint4><<<grid, kCommitThreads, 0, s>>>(a);
  else if (vec_bytes == 4)
    kv_commit_kernel<uint32_t><<<grid, kCommitThreads, 0, s>>>(a);
  else
    kv_commit_kernel<uint8_t><<<grid, kCommitThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace sv
