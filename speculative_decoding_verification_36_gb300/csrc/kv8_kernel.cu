// kv8_kernel.cu -- the paged key/value cache in 8 bits: whole blocks of committed
// tokens become codes with a scale for each block and head, and codes become
// plain entries again.
//
// A block is a page of the code pool.  Of the block x's values in one head, with
// top = max |x|, the scale is top / 127 (int8) or top / 448 (e4m3) and a code is
// x * (127 / top) or x * (448 / top), rounded to the nearest, ties to even.  A
// block is written once, from entries that no longer change: no code is ever
// rounded a second time, and drafts that a verify may reject never reach one.
//
// Both are bound by HBM where there is much.  Measured (GB300, the bytes at 6.77 TB/s beside it):
// 8 prompts of up to 8192 tokens, 8 heads of 128, bf16 to int8: quantised in 90 us (59), read
// back in 70 (59); 2 layers of 8 sequences of up to 16384 read back in 194 us (179); the few blocks
// of a commit, 64 sequences in 16 layers: 23 us for both calls (8.8), two launches and
// three trips to memory each.
#include "sv_common.cuh"
#include "sv_kernels.h"

namespace sv {

constexpr int kQThreads = 128;
constexpr int kQVecs = 8;        // vectors of 16 bytes that a thread keeps in registers
constexpr float kLeast = 7.888609052210118e-31f;  // 2^-100: a block below is all zeros (127 / top stays finite)

// Numbers of pieces of the sequences b0 .. b0 + kQThreads - 1, summed up: s_sum[i] is
// where sequence b0 + i begins.  All threads of the CTA.
__device__ __forceinline__ int sum_up(int n, int* s_sum, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = n;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kQThreads / 32; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  s_sum[threadIdx.x] = before + x - n;
  __syncthreads();
  return all;
}
// The sequence that piece `at` is of: the last one that begins at it or before.
__device__ __forceinline__ int sequence_of(int at, const int* s_sum) {
  int i = 0;
#pragma unroll
  for (int d = kQThreads / 2; d >= 1; d /= 2)
    if (s_sum[i + d] <= at) i += d;
  return i;
}

// The blocks of sequence b that are to be stored, 0 where its data are bad.
__device__ __forceinline__ int blocks_to_store(const Kv8Args& a, int b, int* first, int* stored, bool* bad) {
  const int from = __ldg(a.first + b), len = __ldg(a.last + b);
  const int whole = len > 0 ? fdiv(len, a.div_block) : 0;
  *bad = from < 0 || len < from || len > (long long)a.max_pages * a.page_size || whole > a.max_code_pages ||
         from != (from > 0 ? fdiv(from, a.div_block) * a.block : 0);
  *stored = from;
  *first = *bad ? 0 : fdiv(from, a.div_block);
  return *bad ? 0 : whole - *first;
}

template <class S>
struct Bits;  // the magnitudes in a vector, as integers: they order like the values, NaN above infinity
template <>
struct Bits<uint32_t> {
  static constexpr int n = 4;
  static __device__ __forceinline__ unsigned top(const uint4& v) {
    return max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
  }
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
};
template <>
struct Bits<uint16_t> {
  static constexpr int n = 8;
  static __device__ __forceinline__ unsigned top(const uint4& v) {
    const unsigned lo = max(max(v.x & 0x7fffu, v.y & 0x7fffu), max(v.z & 0x7fffu, v.w & 0x7fffu));
    const unsigned hi = max(max(v.x & 0x7fff0000u, v.y & 0x7fff0000u), max(v.z & 0x7fff0000u, v.w & 0x7fff0000u));
    return max(lo << 16, hi);
  }
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[8]) {
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
  }
};

template <bool kE4m3>
__device__ __forceinline__ uint32_t four_codes(float x0, float x1, float x2, float x3) {
  if constexpr (kE4m3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1), "f"(x0));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3), "f"(x2));
    return (uint32_t)lo | (uint32_t)hi << 16;
  } else {
    // next to 1.5 * 2^23 an fp32 holds whole numbers, to the nearest and ties to even, in its low bits
    auto whole = [](float x) { return __float_as_uint(__fadd_rn(x, 12582912.f)); };
    return __byte_perm(__byte_perm(whole(x0), whole(x1), 0x0040), __byte_perm(whole(x2), whole(x3), 0x0040), 0x5410);
  }
}

// One (block, head) of one cache by a warp (kThreads == 32) or by the CTA: its
// values are read once into registers (a block of more than 8 vectors a thread
// reads the rest a second time), the largest magnitude found, and the codes written.
template <class S, bool kE4m3, int kThreads>
__global__ void __launch_bounds__(kQThreads, 8) kv_quantize_kernel(const __grid_constant__ Kv8Args a) {
  __shared__ int s_sum[kQThreads], s_warp[kQThreads / 32];
  __shared__ unsigned s_top[2][kQThreads / 32];
  constexpr int kGroups = kQThreads / kThreads, kN = Bits<S>::n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int me = kThreads == 32 ? lane : (int)threadIdx.x;
  const int layer = blockIdx.y >> 1, which = blockIdx.y & 1;
  const int slot = blockIdx.x / a.Hkv, h = blockIdx.x - slot * a.Hkv, slots = gridDim.x / a.Hkv;
  const S* cache = (const S*)(which ? a.v_cache : a.k_cache) + layer * a.layer_stride;
  uint8_t* codes = (uint8_t*)(which ? a.v_codes : a.k_codes) + layer * a.code_stride;
  float* scales = (which ? a.v_scales : a.k_scales) + layer * a.scale_stride;
  const int per = a.D / kN, vecs = a.block * per;  // vectors of a token's head, and of the block's
  int turn = 0;
  for (int b0 = 0; b0 < a.B; b0 += kQThreads) {
    int first = 0, stored = 0, n = 0;
    bool bad = false;
    if (b0 + (int)threadIdx.x < a.B) n = blocks_to_store(a, b0 + threadIdx.x, &first, &stored, &bad);
    const int all = sum_up(n, s_sum, s_warp);
    for (int at = slot * kGroups + (kThreads == 32 ? warp : 0); at < all; at += slots * kGroups) {
      const int i = sequence_of(at, s_sum), b = b0 + i;
      const int block = fdiv(__ldg(a.first + b), a.div_block) + at - s_sum[i];
      const int code_page = __ldg(a.code_table + (long long)b * a.max_code_pages + block);
      auto entry = [&](int v) -> long long {  // vector v's values in the cache, -1: a page outside the pool
        const int tok = fdiv(v, a.div_per), s = block * a.block + tok, p = fdiv(s, a.div_page);
        const int page = __ldg(a.page_table + (long long)b * a.max_pages + p);
        if (page < 0 || page >= a.pages) return -1;
        return (((long long)page * a.page_size + (s - p * a.page_size)) * a.Hkv + h) * a.D + (v - tok * per) * kN;
      };
      long long where[kQVecs];
      uint4 x[kQVecs];
      unsigned top = code_page < 0 || code_page >= a.code_pages ? 0xffffffffu : 0u;  // all ones: not to be written
#pragma unroll
      for (int j = 0; j < kQVecs; ++j) where[j] = me + j * kThreads < vecs ? entry(me + j * kThreads) : -2;
#pragma unroll
      for (int j = 0; j < kQVecs; ++j) {
        x[j] = where[j] >= 0 ? *(const uint4*)(cache + where[j]) : make_uint4(0, 0, 0, 0);
        if (where[j] == -1) top = 0xffffffffu;
      }
#pragma unroll
      for (int j = 0; j < kQVecs; ++j) top = max(top, Bits<S>::top(x[j]));
      for (int v = me + kQVecs * kThreads; v < vecs; v += kThreads) {
        const long long e = entry(v);
        top = max(top, e < 0 ? 0xffffffffu : Bits<S>::top(*(const uint4*)(cache + e)));
      }
      top = __reduce_max_sync(0xffffffffu, top);
      if constexpr (kThreads > 32) {
        if (lane == 0) s_top[turn & 1][warp] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kQThreads / 32; ++w) top = max(top, s_top[turn & 1][w]);
        ++turn;  // the other half is free again once all have passed the next barrier
      }
      if (top == 0xffffffffu) continue;
      const bool finite = top < 0x7f800000u;
      const float most = __uint_as_float(top);
      constexpr float kTop = kE4m3 ? 448.f : 127.f;
      const bool some = finite && most >= kLeast;
      const float inv = some ? __fdiv_rn(kTop, most) : 0.f;
      if (me == 0)
        scales[(long long)code_page * a.Hkv + h] = !finite ? __uint_as_float(0x7fffffffu) : some ? __fmul_rn(most, 1.f / kTop) : 0.f;
      uint8_t* to = codes + ((long long)code_page * a.block * a.Hkv + h) * a.D;
      auto put = [&](int v, const uint4& q) {
        const int tok = fdiv(v, a.div_per);
        uint8_t* at_ = to + (long long)tok * a.Hkv * a.D + (v - tok * per) * kN;
        float f[kN];
        Bits<S>::get(q, f);
        uint32_t c[kN / 4];
#pragma unroll
        for (int e = 0; e < kN / 4; ++e)
          c[e] = some ? four_codes<kE4m3>(__fmul_rn(f[4 * e], inv), __fmul_rn(f[4 * e + 1], inv), __fmul_rn(f[4 * e + 2], inv),
                                          __fmul_rn(f[4 * e + 3], inv))
                      : 0u;
        if constexpr (kN == 8)
          *(uint2*)at_ = make_uint2(c[0], c[1]);
        else
          *(uint32_t*)at_ = c[0];
      };
#pragma unroll
      for (int j = 0; j < kQVecs; ++j)
        if (me + j * kThreads < vecs) put(me + j * kThreads, x[j]);
      for (int v = me + kQVecs * kThreads; v < vecs; v += kThreads) put(v, *(const uint4*)(cache + entry(v)));
    }
    // the answers: a warp of one head's and one cache's CTAs for each sequence, which
    // looks whether all its pages are of their pools
    if (h == 0 && blockIdx.y == 0) {
      for (int i = slot * (kQThreads / 32) + warp; i < min(kQThreads, a.B - b0); i += slots * (kQThreads / 32)) {
        const int b = b0 + i;
        n = blocks_to_store(a, b, &first, &stored, &bad);
        for (int x = lane; x < n; x += 32) {
          const int page = __ldg(a.code_table + (long long)b * a.max_code_pages + first + x);
          bad |= page < 0 || page >= a.code_pages;
        }
        if (n > 0) {
          const int p0 = fdiv(stored, a.div_page), p1 = fdiv((first + n) * a.block - 1, a.div_page);
          for (int p = p0 + lane; p <= p1; p += 32) {
            const int page = __ldg(a.page_table + (long long)b * a.max_pages + p);
            bad |= page < 0 || page >= a.pages;
          }
        }
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) {
          a.out_stored[b] = bad ? stored : (first + n) * a.block;
          if (bad) atomicOr(a.status, kStatusBadData);
        }
      }
    }
    __syncthreads();  // s_sum is written anew
  }
}

// Codes to plain entries: a warp takes a run of tokens of one sequence, so that its
// place is looked up once for the run, a lane 16 codes at a time.  Where there are no
// more runs than CTAs, a CTA takes one: 11 us instead of 21 for the few blocks of a commit
// in 16 layers; warps of their own are faster where there is much (196 us instead of 233 for
// 8 x 12288 tokens of 2 layers of 8 heads of 128 in bf16).
constexpr int kRun = 8;     // tokens
constexpr int kRFlight = 4; // vectors in flight per lane

__device__ __forceinline__ int runs_to_read(const Kv8Args& a, int b, bool* bad) {
  const int from = __ldg(a.first + b), to = __ldg(a.last + b);
  *bad = from < 0 || to < from || to > (long long)a.max_pages * a.page_size || to > (long long)a.max_code_pages * a.block;
  return *bad ? 0 : (int)(((long long)to - from + kRun - 1) / kRun);
}

template <class S, bool kE4m3>
__global__ void __launch_bounds__(kQThreads) kv_dequantize_kernel(const __grid_constant__ Kv8Args a) {
  __shared__ int s_sum[kQThreads], s_warp[kQThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int layer = blockIdx.y >> 1, which = blockIdx.y & 1;
  S* cache = (S*)(which ? a.v_cache : a.k_cache) + layer * a.layer_stride;
  const uint8_t* codes = (const uint8_t*)(which ? a.v_codes : a.k_codes) + layer * a.code_stride;
  const float* scales = (which ? a.v_scales : a.k_scales) + layer * a.scale_stride;
  const int entry = a.Hkv * a.D, per = entry / 16;
  for (int b0 = 0; b0 < a.B; b0 += kQThreads) {
    int n = 0;
    bool bad = false;
    if (b0 + (int)threadIdx.x < a.B) n = runs_to_read(a, b0 + threadIdx.x, &bad);
    if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.status, kStatusBadData);
    const int all = sum_up(n, s_sum, s_warp);
    const bool few = all <= (int)gridDim.x;
    const int me = few ? (int)threadIdx.x : lane, step = few ? kQThreads : 32;
    for (int at = few ? (int)blockIdx.x : (int)blockIdx.x * (kQThreads / 32) + warp; at < all; at += gridDim.x * (kQThreads / 32)) {
      const int i = sequence_of(at, s_sum), b = b0 + i;
      const int s0 = __ldg(a.first + b) + (at - s_sum[i]) * kRun, count = min(kRun, __ldg(a.last + b) - s0);
      // lane x of every warp looks up token x
      int code_page = -1, from = -1, to = -1;
      if (lane < count) {
        const int s = s0 + lane, c = fdiv(s, a.div_block), p = fdiv(s, a.div_page);
        code_page = __ldg(a.code_table + (long long)b * a.max_code_pages + c);
        const int page = __ldg(a.page_table + (long long)b * a.max_pages + p);
        if (code_page < 0 || code_page >= a.code_pages || page < 0 || page >= a.pages) {
          atomicOr(a.status, kStatusBadData);
        } else {
          from = code_page * a.block + (s - c * a.block);
          to = page * a.page_size + (s - p * a.page_size);
        }
      }
      const int total = count * per;
      for (int v0 = me; v0 - lane < total; v0 += step * kRFlight) {
        uint4 x[kRFlight];
        float scale[kRFlight];
        long long out[kRFlight];
#pragma unroll
        for (int q = 0; q < kRFlight; ++q) {
          const int v = v0 + step * q, tok = v < total ? fdiv(v, a.div_per) : 0, r = v - tok * per;
          const int f = __shfl_sync(0xffffffffu, from, tok), t = __shfl_sync(0xffffffffu, to, tok);
          const int cp = __shfl_sync(0xffffffffu, code_page, tok);
          out[q] = v < total && f >= 0 ? (long long)t * entry + r * 16 : -1;
          if (out[q] >= 0) {
            x[q] = __ldg((const uint4*)(codes + (long long)f * entry + r * 16));
            scale[q] = __ldg(scales + (long long)cp * a.Hkv + fdiv(r, a.div_head));
          }
        }
#pragma unroll
        for (int q = 0; q < kRFlight; ++q) {
          if (out[q] < 0) continue;
          const uint32_t w[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
          float f[16];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (kE4m3) {
              uint32_t lo, hi;
              asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
                  : "=r"(lo), "=r"(hi)
                  : "r"(w[e]));
              asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
                  : "=f"(f[4 * e]), "=f"(f[4 * e + 1])
                  : "r"(lo));
              asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
                  : "=f"(f[4 * e + 2]), "=f"(f[4 * e + 3])
                  : "r"(hi));
            } else {
#pragma unroll
              for (int y = 0; y < 4; ++y) f[4 * e + y] = (float)(int)(int8_t)(w[e] >> (8 * y));
            }
          }
          S* to_ = cache + out[q];
          if constexpr (sizeof(S) == 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              ((float4*)to_)[e] = make_float4(__fmul_rn(f[4 * e], scale[q]), __fmul_rn(f[4 * e + 1], scale[q]),
                                              __fmul_rn(f[4 * e + 2], scale[q]), __fmul_rn(f[4 * e + 3], scale[q]));
          } else {
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                  : "=r"(o[e])
                  : "f"(__fmul_rn(f[2 * e + 1], scale[q])), "f"(__fmul_rn(f[2 * e], scale[q])));
            ((uint4*)to_)[0] = make_uint4(o[0], o[1], o[2], o[3]);
            ((uint4*)to_)[1] = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
      }
    }
    __syncthreads();  // s_sum is written anew
  }
}

static void set_divisions(Kv8Args& a, int values) {
  a.div_block = make_fastdiv((uint32_t)a.block);
  a.div_page = make_fastdiv((uint32_t)a.page_size);
  a.div_per = make_fastdiv((uint32_t)values);
  a.div_head = make_fastdiv((uint32_t)(a.D / 16));
}
// CTAs of one cache of one layer: enough for every SM's threads, no more than pieces.
static unsigned ctas(const Kv8Args& a, long long pieces, int sms) {
  const long long want = (16LL * sms + 2 * a.layers - 1) / (2 * a.layers);
  return (unsigned)max(1LL, min(pieces, want));
}

cudaError_t launch_kv_quantize(const Kv8Args& args, bool bf16, bool e4m3, int sms, cudaStream_t s) {
  Kv8Args a = args;
  const int n = bf16 ? 8 : 4;
  set_divisions(a, a.D / n);
  const bool warps = (long long)a.block * a.D / n <= 32 * kQVecs;
  const long long blocks = (long long)a.B * a.max_code_pages, groups = warps ? kQThreads / 32 : 1;
  const unsigned slots = ctas(a, (blocks + groups - 1) / groups, (sms + a.Hkv - 1) / a.Hkv);
  const dim3 grid(slots * a.Hkv, 2 * a.layers);
#define SV_GO(S, E)                                                        \
  if (warps)                                                               \
    kv_quantize_kernel<S, E, 32><<<grid, kQThreads, 0, s>>>(a);            \
  else                                                                     \
    kv_quantize_kernel<S, E, kQThreads><<<grid, kQThreads, 0, s>>>(a)
  if (bf16 && e4m3) {
    SV_GO(uint16_t, true);
  } else if (bf16) {
    SV_GO(uint16_t, false);
  } else if (e4m3) {
    SV_GO(uint32_t, true);
  } else {
    SV_GO(uint32_t, false);
  }
#undef SV_GO
  return cudaGetLastError();
}

cudaError_t launch_kv_dequantize(const Kv8Args& args, bool bf16, bool e4m3, int sms, cudaStream_t s) {
  Kv8Args a = args;
  set_divisions(a, a.Hkv * a.D / 16);
  const long long most = min((long long)a.max_pages * a.page_size, (long long)a.max_code_pages * a.block);
  const dim3 grid(ctas(a, a.B * ((most + kRun - 1) / kRun), sms), 2 * a.layers);
  if (bf16 && e4m3)
    kv_dequantize_kernel<uint16_t, true><<<grid, kQThreads, 0, s>>>(a);
  else if (bf16)
    kv_dequantize_kernel<uint16_t, false><<<grid, kQThreads, 0, s>>>(a);
  else if (e4m3)
    kv_dequantize_kernel<uint32_t, true><<<grid, kQThreads, 0, s>>>(a);
  else
    kv_dequantize_kernel<uint32_t, false><<<grid, kQThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace sv
