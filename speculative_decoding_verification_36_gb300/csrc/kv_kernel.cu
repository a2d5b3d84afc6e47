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

constexpr int kKvThreads = 128;
constexpr int kKvWarps = kKvThreads / 32;

// VEC values of a type (S: its bits) as they lie in memory, in whole words:
// 16 bytes, or a single value.
template <class S, int VEC>
struct KvVec;
template <>
struct KvVec<uint32_t, 4> {
  uint4 q;
  __device__ __forceinline__ void load(const uint32_t* p) { q = *(const uint4*)p; }
  __device__ __forceinline__ void store(uint32_t* p) const { *(uint4*)p = q; }
  __device__ __forceinline__ void get(float (&f)[4]) const {
    f[0] = __uint_as_float(q.x), f[1] = __uint_as_float(q.y), f[2] = __uint_as_float(q.z), f[3] = __uint_as_float(q.w);
  }
  __device__ __forceinline__ void set(const float (&f)[4]) {
    q = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct KvVec<uint16_t, 8> {
  uint4 q;
  __device__ __forceinline__ void load(const uint16_t* p) { q = *(const uint4*)p; }
  __device__ __forceinline__ void store(uint16_t* p) const { *(uint4*)p = q; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = bf16_lo(q.x), f[1] = bf16_hi(q.x), f[2] = bf16_lo(q.y), f[3] = bf16_hi(q.y);
    f[4] = bf16_lo(q.z), f[5] = bf16_hi(q.z), f[6] = bf16_lo(q.w), f[7] = bf16_hi(q.w);
  }
  static __device__ __forceinline__ uint32_t two(float lo, float hi) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    q = make_uint4(two(f[0], f[1]), two(f[2], f[3]), two(f[4], f[5]), two(f[6], f[7]));
  }
};
template <>
struct KvVec<uint32_t, 1> {
  uint32_t v;
  __device__ __forceinline__ void load(const uint32_t* p) { v = *p; }
  __device__ __forceinline__ void store(uint32_t* p) const { *p = v; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __uint_as_float(v); }
  __device__ __forceinline__ void set(const float (&f)[1]) { v = __float_as_uint(f[0]); }
};
template <>
struct KvVec<uint16_t, 1> {
  uint32_t v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *p; }
  __device__ __forceinline__ void store(uint16_t* p) const { *p = (uint16_t)v; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = bf16_lo(v); }
  __device__ __forceinline__ void set(const float (&f)[1]) { v = KvVec<uint16_t, 8>::two(f[0], 0.f); }
};

constexpr int kKvHeads = 2;  // rounds of heads in flight per warp
constexpr int kKvVals = 2;   // ... of V's vectors

// A warp takes a token, or one of `parts` shares of its heads where there are
// few tokens, and works by itself.  A lane keeps its place within the head from
// head to head, and with it its cosines and sines in registers (kRegs; heads
// of more vectors than a warp has lanes read them from shared memory).  A
// token's values are read once and written once; the reads of the first heads
// need only the token's index and set out before the two trips to memory that
// its slot takes.
//
// The bound is one reading and one writing of the values: 81 us for a padded
// batch of 8 x 4096 tokens, 63 % of them new, of 32 + 8 + 8 heads of 128 in bf16
// (0.51 GB, 6.3 TB/s); 4.1 us for one chain of 5.  More heads in flight per warp
// (3, 4) and more registers for them measured slower (81 to 94 us), as did
// CTAs of four tokens with a shared table of angles (84 us).
// Shared memory, per warp: cos and sin [rot / 2], then for a tree the parents [T - 1].
template <class S, int VEC, bool kInterleaved, bool kRegs>
__global__ void __launch_bounds__(kKvThreads, 8) kv_append_kernel(const __grid_constant__ KvAppendArgs a) {
  extern __shared__ __align__(16) unsigned char s_kv[];
  using V = KvVec<S, VEC>;
  constexpr int kFreqs = kInterleaved ? (VEC > 1 ? VEC / 2 : 1) : VEC;  // frequencies of an item
  constexpr int kPair = kInterleaved && VEC == 1 ? 1 : 0;              // interleaved single values go by two
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int half = a.rot / 2;
  const int N = a.parents ? a.T - 1 : 0;
  float2* cs = (float2*)(s_kv + (size_t)warp * a.warp_bytes);
  int* par = (int*)(cs + half);
  const long long unit = (long long)blockIdx.x * kKvWarps + warp;
  if (unit >= (long long)a.B * a.T * a.parts) return;
  const int g = (int)(unit / a.parts), part = (int)(unit - (long long)g * a.parts);
  const int b = fdiv(g, a.div_t), i = g - b * a.T;

  // its heads: K's, then Q's; items of a head: rotated vectors (pairs of
  // vectors where the halves rotate against each other)
  const int H = a.Hkv + a.Hq, h0 = (int)((long long)H * part / a.parts), h1 = (int)((long long)H * (part + 1) / a.parts);
  const int per = half / kFreqs;
  auto src_of = [&](int h) {
    return h < a.Hkv ? (const S*)a.k + (long long)g * a.kv_stride + h * a.D
                     : (const S*)a.q + (long long)g * a.q_stride + (h - a.Hkv) * a.D;
  };
  V lo[kKvHeads], hi[kKvHeads];
  auto load = [&](int x, int h, int j) {  // item j of head h
    const S* src = src_of(h) + j * (kInterleaved ? VEC + kPair : VEC);
    lo[x].load(src);
    if (!kInterleaved) hi[x].load(src + half);
    if (kPair) hi[x].load(src + 1);
  };
  // kRegs: lanes by place in the head, then by head
  const int at_once = kRegs ? 32 / max(per, 1) : 0;  // heads at once
  const int jr = kRegs ? lane % max(per, 1) : 0, hr = kRegs && lane < at_once * per ? lane / max(per, 1) : 1 << 28;
  const int all = a.Hkv * (a.D / VEC);  // V's vectors
  const int v0 = (int)((long long)all * part / a.parts), v1 = (int)((long long)all * (part + 1) / a.parts);
  const S* v_from = (const S*)a.v + (long long)g * a.kv_stride;
  V val[kKvVals];
  // its first values set out as soon as it is known that it is no padding
  auto first = [&]() {
    if constexpr (kRegs) {
#pragma unroll
      for (int x = 0; x < kKvHeads; ++x)
        if (h0 + hr + x * at_once < h1 && per) load(x, h0 + hr + x * at_once, jr);
    }
#pragma unroll
    for (int q = 0; q < kKvVals; ++q)
      if (v0 + lane + 32 * q < v1) val[q].load(v_from + (v0 + lane + 32 * q) * VEC);
  };
  if (!a.n_new) first();

  // ---- its place ----
  unsigned long long turn[2];  // the lane's first frequencies
#pragma unroll
  for (int q = 0; q < 2; ++q) turn[q] = lane + 32 * q < half ? __ldg(a.turns + lane + 32 * q) : 0ull;
  const int len = __ldg(a.lengths + b);
  const int n_new = a.n_new ? __ldg(a.n_new + b) : a.T;
  bool bad = len < 0 || n_new < 0 || n_new > a.T || (long long)len + n_new > (long long)a.max_pages * a.page_size;
  const unsigned slot = (unsigned)len + (unsigned)i, in_table = slot / (unsigned)a.page_size;
  const int page = !bad && i < n_new ? __ldg(a.page_table + (long long)b * a.max_pages + in_table) : -1;
  int depth = i;
  if (a.parents) {
    // every parent of the sequence has to precede its node
    for (int j = lane; j < N; j += 32) {
      const int p = __ldg(a.parents + (long long)b * N + j);
      par[j] = p;
      bad |= p < -1 || p >= j;
    }
    bad = __any_sync(0xffffffffu, bad);
    __syncwarp();
    depth = 0;
    if (!bad)
      for (int j = i - 1; j >= 0; j = par[j]) ++depth;
  }
  if (!bad && i >= n_new) return;  // behind the sequence's new tokens
  if (a.n_new) first();
  const unsigned long long pos = (unsigned long long)((long long)len + depth);
  for (int f = lane, q = 0; f < half; f += 32, ++q) {
    const unsigned long long angle = pos * (q == 0 ? turn[0] : q == 1 ? turn[1] : __ldg(a.turns + f));
    float s, c;
    // the fraction of a turn in [-1/2, 1/2): half turns in, radians / pi
    sincospif((float)(int)(angle >> 32) * 4.656612873077393e-10f, &s, &c);
    if (bad) s = c = NAN;  // a bad sequence's queries
    cs[f] = make_float2(c, s);
  }
  __syncwarp();
  const bool lost = bad || page < 0 || page >= a.pages;
  if (lost && lane == 0) atomicOr(a.status, kStatusBadData);
  // element offset of its entry in the caches, -1: not written
  const long long dst =
      lost ? -1 : ((long long)page * a.page_size + (slot - in_table * (unsigned)a.page_size)) * a.Hkv * a.D;
  if (dst >= 0) {
    S* v_to = (S*)a.v_cache + dst;
    for (int x = v0 + lane; x < v1; x += kKvVals * 32) {
      if (x != v0 + lane)
#pragma unroll
        for (int q = 0; q < kKvVals; ++q)
          if (x + 32 * q < v1) val[q].load(v_from + (x + 32 * q) * VEC);
#pragma unroll
      for (int q = 0; q < kKvVals; ++q)
        if (x + 32 * q < v1) val[q].store(v_to + (x + 32 * q) * VEC);
    }
  }

  auto dst_of = [&](int h) -> S* {
    if (h >= a.Hkv) return (S*)a.out_q + ((long long)g * a.Hq + h - a.Hkv) * a.D;
    return dst < 0 ? nullptr : (S*)a.k_cache + dst + h * a.D;
  };
  auto store = [&](int x, int h, int j, const float2 (&w)[kFreqs]) {
    S* to = dst_of(h);
    if (!to) return;
    to += j * (kInterleaved ? VEC + kPair : VEC);
    float p[VEC], q[VEC];
    lo[x].get(p);
    if constexpr (kInterleaved && VEC > 1) {
#pragma unroll
      for (int e = 0; e < VEC; e += 2) {
        q[e] = p[e] * w[e / 2].x - p[e + 1] * w[e / 2].y;
        q[e + 1] = p[e] * w[e / 2].y + p[e + 1] * w[e / 2].x;
      }
      lo[x].set(q);
      lo[x].store(to);
    } else {
      hi[x].get(q);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float r = p[e] * w[e].x - q[e] * w[e].y;
        q[e] = p[e] * w[e].y + q[e] * w[e].x;
        p[e] = r;
      }
      lo[x].set(p);
      hi[x].set(q);
      lo[x].store(to);
      hi[x].store(to + (kInterleaved ? 1 : half));
    }
  };
  if (per > 0) {
    if constexpr (kRegs) {
      float2 w[kFreqs];
#pragma unroll
      for (int e = 0; e < kFreqs; ++e) w[e] = cs[jr * kFreqs + e];
      for (int h = h0 + hr; h < h1; h += kKvHeads * at_once) {
        if (h != h0 + hr)
#pragma unroll
          for (int x = 0; x < kKvHeads; ++x)
            if (h + x * at_once < h1) load(x, h + x * at_once, jr);
#pragma unroll
        for (int x = 0; x < kKvHeads; ++x)
          if (h + x * at_once < h1) store(x, h + x * at_once, jr, w);
      }
    } else {
      for (int h = h0; h < h1; ++h)
        for (int j = lane; j < per; j += 32) {
          float2 w[kFreqs];
#pragma unroll
          for (int e = 0; e < kFreqs; ++e) w[e] = cs[j * kFreqs + e];
          load(0, h, j);
          store(0, h, j, w);
        }
    }
  }
  // what is not turned: the rest of the heads, and V
  const int rest = (a.D - a.rot) / VEC;
  for (int x = lane; x < rest * (h1 - h0); x += 32) {
    const int h = h0 + x / rest, e = a.rot + x % rest * VEC;
    S* to = dst_of(h);
    if (!to) continue;
    V v;
    v.load(src_of(h) + e);
    if (bad) {
      float f[VEC];
#pragma unroll
      for (int q = 0; q < VEC; ++q) f[q] = NAN;
      v.set(f);
    }
    v.store(to + e);
  }
}

int kv_max_rot() { return 1024; }

template <class S, int VEC, bool kInterleaved>
static void launch_append(const KvAppendArgs& a, cudaStream_t s) {
  KvAppendArgs k = a;
  const long long all = (long long)a.B * a.T;
  // few tokens: a token's heads go to several warps, until every SM has some
  k.parts = 1;
  while (k.parts < 8 && all * k.parts < 8LL * a.sms) k.parts *= 2;
  k.div_t = make_fastdiv((uint32_t)a.T);
  k.warp_bytes = (int)(((a.rot / 2) * sizeof(float2) + (a.parents ? (a.T - 1) * sizeof(int) : 0) + 15) / 16 * 16);
  const unsigned grid = (unsigned)((all * k.parts + kKvWarps - 1) / kKvWarps);
  const size_t smem = (size_t)kKvWarps * k.warp_bytes;
  const int per = a.rot / 2 / (kInterleaved ? (VEC > 1 ? VEC / 2 : 1) : VEC);
  if (per <= 32)
    kv_append_kernel<S, VEC, kInterleaved, true><<<grid, kKvThreads, smem, s>>>(k);
  else
    kv_append_kernel<S, VEC, kInterleaved, false><<<grid, kKvThreads, smem, s>>>(k);
}
template <class S, int VEC>
static void launch_append(const KvAppendArgs& a, cudaStream_t s) {
  if (a.interleaved)
    launch_append<S, VEC, true>(a, s);
  else
    launch_append<S, VEC, false>(a, s);
}

cudaError_t launch_kv_append(const KvAppendArgs& a, bool bf16, bool vec, cudaStream_t s) {
  if (bf16 && vec)
    launch_append<uint16_t, 8>(a, s);
  else if (bf16)
    launch_append<uint16_t, 1>(a, s);
  else if (vec)
    launch_append<uint32_t, 4>(a, s);
  else
    launch_append<uint32_t, 1>(a, s);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// commit
// ---------------------------------------------------------------------------
// Bound by its chain of trips to memory (lengths and tree, page table, entries):
// 9 us for 128 trees of 62 nodes and 4 layers of 2 KB entries.
// One CTA per (sequence, layer, cache).  Every thread takes nodes that carry the
// path's last token and follows them up, token by token; the lowest node whose
// way to the root spells the path is the path's last.  Then the entries move:
// slot len + 1 + node_d to slot len + d.  node_d >= d - 1, so moving in
// ascending order never overwrites an entry that is still to be read; each
// thread keeps that order for its own bytes.
constexpr int kCommitThreads = 128;
constexpr int kCommitBatch = 4;  // entries in flight per thread

template <class V>
__global__ void __launch_bounds__(kCommitThreads) kv_commit_kernel(const __grid_constant__ KvCommitArgs a) {
  extern __shared__ __align__(16) long long s_commit[];
  const int N = a.N;
  long long *s_to = s_commit, *s_from = s_to + N;  // the path's byte offsets, by level
  int *s_par = (int*)(s_from + N), *s_tok = s_par + N, *s_path = s_tok + N;
  int* s_node = s_path + N;  // the path's nodes, by level
  __shared__ int s_last;
  const int tid = threadIdx.x;
  const int b = blockIdx.x;
  const int layer = blockIdx.y >> 1, which = blockIdx.y & 1;
  const int size = __ldg(a.path_len + b);
  const long long len = __ldg(a.lengths + b);
  const int n = size > 0 ? size - 1 : 0;
  const long long most = min((long long)a.max_pages * a.page_size, 2147483647LL);
  bool wrong = false;
  for (int j = tid; j < N; j += kCommitThreads) {
    const int p = __ldg(a.parents + (long long)b * N + j);
    s_par[j] = p;
    s_tok[j] = __ldg(a.tokens + (long long)b * N + j);
    s_path[j] = __ldg(a.path + (long long)b * (N + 1) + j);
    wrong |= p < -1 || p >= j;
  }
  if (tid == 0) s_last = N;
  // every verdict below is the whole CTA's: the barriers stay uniform
  bool bad = __syncthreads_or(wrong) || size < 1 || n > N || len < 0 || len + N + 1 > most;
  const bool go = size != -1;  // a verify's bad sequence is left as it is
  if (go && !bad && n > 0) {
    for (int j = tid; j < N; j += kCommitThreads) {
      int at = j, d = n;
      while (d > 0 && at >= 0 && s_tok[at] == s_path[d - 1]) at = s_par[at], --d;
      if (d == 0 && at < 0) atomicMin(&s_last, j);
    }
    __syncthreads();
    bad = s_last >= N;  // no path of the tree carries these tokens
  }
  if (go && !bad) {
    if (tid == 0 && n > 0)
      for (int j = s_last, d = n; d >= 1; --d, j = s_par[j]) s_node[d - 1] = j;
    __syncthreads();
    wrong = false;
    for (int d = tid; d < n; d += kCommitThreads) {
      const long long to = len + 1 + d, from = len + 1 + s_node[d];
      const int32_t* table = a.page_table + (long long)b * a.max_pages;
      const int p0 = __ldg(table + to / a.page_size), p1 = __ldg(table + from / a.page_size);
      wrong |= p0 < 0 || p0 >= a.pages || p1 < 0 || p1 >= a.pages;
      s_to[d] = ((long long)p0 * a.page_size + to % a.page_size) * a.entry_bytes;
      s_from[d] = ((long long)p1 * a.page_size + from % a.page_size) * a.entry_bytes;
    }
    bad = __syncthreads_or(wrong);
  }
  if (blockIdx.y == 0) {
    for (int d = tid; d <= N; d += kCommitThreads) a.out_nodes[(long long)b * (N + 1) + d] = go && !bad && d < n ? s_node[d] : -1;
    if (tid == 0) {
      a.out_lengths[b] = (int)(go && !bad ? len + size : len);
      if (go && bad) atomicOr(a.status, kStatusBadData);
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
        if (d0 + i < n) v[i] = ((const V*)(cache + s_from[d0 + i]))[x];
#pragma unroll
      for (int i = 0; i < kCommitBatch; ++i)
        if (d0 + i < n) ((V*)(cache + s_to[d0 + i]))[x] = v[i];
    }
  }
}

cudaError_t launch_kv_commit(const KvCommitArgs& a, int vec_bytes, cudaStream_t s) {
  const dim3 grid((unsigned)a.B, (unsigned)(2 * a.layers));
  const size_t smem = (size_t)a.N * (2 * sizeof(long long) + 4 * sizeof(int));
  if (vec_bytes == 16)
    kv_commit_kernel<uint4><<<grid, kCommitThreads, smem, s>>>(a);
  else if (vec_bytes == 4)
    kv_commit_kernel<uint32_t><<<grid, kCommitThreads, smem, s>>>(a);
  else
    kv_commit_kernel<uint8_t><<<grid, kCommitThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace sv
