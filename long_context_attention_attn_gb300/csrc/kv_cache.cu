// The paged 8-bit key / value cache: appending tokens and copying pages.
//
// Both are bound by HBM traffic (append: 2 bytes in and 1 out per value; copy:
// 1 in and 1 out), and by launch latency where a decoding step appends one
// token per sequence.
#include <cuda_bf16.h>

#include "internal.h"
#include "rotation.cuh"

namespace gb300 {

namespace {

struct AppendArgs {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  const int* table;
  const int* start;
  const int* lens;
  const int* tok_start;
  int64_t tokens, token_stride, row_tokens, page_stride, units;
  int num_pages, h_kv, page_size, max_pages, max_new, pages_per_seq;
};

// Two e4m3 codes of two fp32 values (round to nearest even, saturating; NaN
// stays NaN): lo in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The two fp32 values of two e4m3 codes (exact).
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)codes));
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h2));
  return f;
}

// max(m, |both|) over the values that are finite
__device__ __forceinline__ float amax_finite(float m, uint32_t w) {
  const float2 f = widen_bf16x2(w);
  const float a = fabsf(f.x), b = fabsf(f.y);
  if (a < INFINITY) m = fmaxf(m, a);
  if (b < INFINITY) m = fmaxf(m, b);
  return m;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Exponent k of the smallest power of two with amax <= 448 * 2^k (448 = 1.75 *
// 2^8, so the exponent less 8, and one more above a mantissa of 1.75), no less
// than -126.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(k, -126);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

constexpr int kChunksPerThread = 4;  // 16-value chunks a thread holds in registers

// How K is turned by its positions on the way.
enum { kAsIs, kHalf, kInterleaved };

// The values of a chunk of 16 (two vectors of 16 bytes), turned.
template <int kTurn>
__device__ __forceinline__ void turn_chunk(float (&x)[16], uint4 v0, uint4 v1, int pos, const uint64_t (&turns)[8],
                                           float amp, bool turning) {
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = widen_bf16x2(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
  if (!turning) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = cos_sin(pos, turns[i], amp);
    const int p = kTurn == kHalf ? i : 2 * i, q = kTurn == kHalf ? i + 8 : 2 * i + 1;
    const float y = x[p], z = x[q];
    x[p] = y * f.x - z * f.y;
    x[q] = z * f.x + y * f.y;
  }
}

// 16 codes of a chunk: 8 for each of its vectors.
__device__ __forceinline__ void codes_of(const float (&x)[16], float inv, uint32_t (&o)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    o[e] = to_e4m3x2(x[4 * e] * inv, x[4 * e + 1] * inv) | (to_e4m3x2(x[4 * e + 2] * inv, x[4 * e + 3] * inv) << 16);
}

// T threads take one unit: the new tokens of one sequence that fall on one
// page, for one head of K or of V.  They hold the unit's values in registers
// (T * 4 chunks of 16 values cover it), so every value is read once: the
// largest magnitude first, then the codes.  Neighbouring units are the heads
// of the same tokens, whose rows are neighbours in memory.
//
// With kTurn, K's chunks are the units of rotation.cuh, whose pairs are their own, and
// stay in registers turned (fp32: 16 more of them a chunk than bf16).  s_turns: the
// pairs' turns per position.
template <int T, int D, int kTurn>
__device__ __forceinline__ void append_unit(const AppendArgs& a, const Turning* t, const uint64_t* s_turns) {
  constexpr int kUnits = T < 128 ? 128 / T : 1;  // units per CTA
  constexpr int kRowChunks = D / 16;
  const int tid = threadIdx.x % T;
  const int64_t unit = (int64_t)blockIdx.x * kUnits + threadIdx.x / T;
  if (unit >= a.units) return;  // whole warps: T >= 32
  const int h = (int)(unit % a.h_kv);
  int64_t rest = unit / a.h_kv;
  const bool is_v = rest & 1;
  rest >>= 1;
  const int j = (int)(rest % a.pages_per_seq);
  const int64_t i = rest / a.pages_per_seq;
  const int start = a.start[i];
  int len = a.max_new;
  if (a.lens) len = min(max(a.lens[i], 0), a.max_new);
  const int64_t row0 = a.tok_start ? (int64_t)a.tok_start[i] : i * a.row_tokens;
  if (start < 0 || len == 0) return;
  const int entry = start / a.page_size + j;  // page table column
  if (entry >= a.max_pages) return;
  // the slots [lo, hi) of this page that get new tokens
  const int64_t page_first = (int64_t)entry * a.page_size;
  const int64_t end = (int64_t)start + len;
  // slot t takes token row at0 + t, of the rows that there are
  const int64_t at0 = row0 + (page_first - start);
  const int64_t lo64 = max(max((int64_t)start - page_first, (int64_t)0), -at0);
  const int64_t hi64 = min(min(end - page_first, (int64_t)a.page_size), a.tokens - at0);
  if (hi64 <= lo64) return;
  const int lo = (int)lo64, hi = (int)hi64;  // 0 <= lo < hi <= page_size
  const int pid = a.table[i * a.max_pages + entry];
  if (pid < 0 || pid >= a.num_pages) return;

  const __nv_bfloat16* x = (is_v ? a.v : a.k) + (int64_t)h * D;
  uint8_t* page = (is_v ? a.vc : a.kc) + pid * a.page_stride + (int64_t)h * a.page_size * D;
  float* scale = (is_v ? a.vs : a.ks) + (int64_t)pid * a.h_kv + h;
  const float old = lo > 0 ? *scale : 0.f;

  const int chunks = (hi - lo) * kRowChunks;
  const __nv_bfloat16* row = x + (at0 + lo + tid / kRowChunks) * a.token_stride;
  constexpr int kStep = T / kRowChunks;  // tokens between a thread's chunks (T % kRowChunks == 0)
  uint4 r[kChunksPerThread][2];
  float y[kTurn ? kChunksPerThread : 1][16];  // K turned
  const bool turn = kTurn && !is_v;
  int va = 0, vb = 0;  // the first values of the chunk's vectors
  float amax = 0.f;
  if (turn) {
    const HeadUnits<__nv_bfloat16, kTurn == kInterleaved> units(D, t->rot, true);
    const int u = tid % kRowChunks;
    va = units.at(u, 0, t->rot, t->offset);
    vb = units.at(u, 1, t->rot, t->offset);
#pragma unroll
    for (int c = 0; c < kChunksPerThread; ++c) {
      r[c][0] = r[c][1] = make_uint4(0u, 0u, 0u, 0u);
      if (c * T + tid < chunks) {
        r[c][0] = load_stream(row + (int64_t)c * kStep * a.token_stride + va);
        r[c][1] = load_stream(row + (int64_t)c * kStep * a.token_stride + vb);
      }
    }
    uint64_t turns[8];
    const bool turning = u < units.turning;
    if (turning) {
#pragma unroll
      for (int i = 0; i < 8; ++i) turns[i] = s_turns[8 * u + i];
    }
    const int pos = (int)(page_first + lo) + tid / kRowChunks;
#pragma unroll
    for (int c = 0; c < kChunksPerThread; ++c) {
      turn_chunk<kTurn>(y[kTurn ? c : 0], r[c][0], r[c][1], pos + c * kStep, turns, t->amp, turning);
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(y[kTurn ? c : 0][i]));  // (NaN counts as nothing)
    }
    if (!(amax < INFINITY)) {  // infinities: only what is finite counts
      amax = 0.f;
#pragma unroll
      for (int c = 0; c < kChunksPerThread; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float m = fabsf(y[kTurn ? c : 0][i]);
          if (m < INFINITY) amax = fmaxf(amax, m);
        }
    }
  } else {
    const uint4* src = reinterpret_cast<const uint4*>(row) + 2 * (tid % kRowChunks);
    const int64_t step = (int64_t)kStep * a.token_stride / 8;
#pragma unroll
    for (int u = 0; u < kChunksPerThread; ++u) {
      r[u][0] = r[u][1] = make_uint4(0u, 0u, 0u, 0u);
      if (u * T + tid < chunks) {
        r[u][0] = __ldcs(src + u * step);
        r[u][1] = __ldcs(src + u * step + 1);
      }
    }
    // magnitudes of bf16 order like their bits, two in a word
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < kChunksPerThread; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top = max_u16x2(top, r[u][e].x & 0x7fff7fffu);
        top = max_u16x2(top, r[u][e].y & 0x7fff7fffu);
        top = max_u16x2(top, r[u][e].z & 0x7fff7fffu);
        top = max_u16x2(top, r[u][e].w & 0x7fff7fffu);
      }
    amax = __uint_as_float(max(top << 16, top & 0xffff0000u));
    if (!(amax < INFINITY)) {  // infinities or NaN: only what is finite counts
      amax = 0.f;
#pragma unroll
      for (int u = 0; u < kChunksPerThread; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          amax = amax_finite(amax, r[u][e].x);
          amax = amax_finite(amax, r[u][e].y);
          amax = amax_finite(amax, r[u][e].z);
          amax = amax_finite(amax, r[u][e].w);
        }
    }
  }
  // non-negative floats order like their bits
  uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
  if constexpr (T > 32) {
    __shared__ uint32_t s_max[T / 32];
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x / 32] = bits;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < T / 32; ++w) bits = max(bits, s_max[w]);
  } else {
    __syncwarp();
  }
  const int k = scale_exponent(__uint_as_float(bits));
  const float need = pow2f(k);
  const bool grew = lo > 0 && need > old;
  const float now = lo > 0 && !grew ? old : need;
  const float inv = 1.f / now;  // exact: scales that this kernel writes are powers of two
  if (grew) {
    // the older tokens of the page, in the new scale
    const float ratio = old * inv;
    for (int c = tid; c < lo * kRowChunks; c += T) {
      uint4* p = reinterpret_cast<uint4*>(page) + c;
      const uint4 w = *p;
      const uint32_t in[4] = {w.x, w.y, w.z, w.w};
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f0 = from_e4m3x2(in[e]), f1 = from_e4m3x2(in[e] >> 16);
        o[e] = to_e4m3x2(f0.x * ratio, f0.y * ratio) | (to_e4m3x2(f1.x * ratio, f1.y * ratio) << 16);
      }
      *p = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  if (turn) {
    uint8_t* dst = page + (int64_t)(lo + tid / kRowChunks) * D;
#pragma unroll
    for (int c = 0; c < kChunksPerThread; ++c) {
      if (c * T + tid < chunks) {
        uint32_t o[4];
        codes_of(y[kTurn ? c : 0], inv, o);
        *reinterpret_cast<uint2*>(dst + c * kStep * D + va) = make_uint2(o[0], o[1]);
        *reinterpret_cast<uint2*>(dst + c * kStep * D + vb) = make_uint2(o[2], o[3]);
      }
    }
  } else {
    uint4* dst = reinterpret_cast<uint4*>(page) + lo * kRowChunks + tid;
#pragma unroll
    for (int u = 0; u < kChunksPerThread; ++u) {
      if (u * T + tid < chunks) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t w[4] = {r[u][e].x, r[u][e].y, r[u][e].z, r[u][e].w};
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float2 f0 = widen_bf16x2(w[2 * q]), f1 = widen_bf16x2(w[2 * q + 1]);
            o[2 * e + q] = to_e4m3x2(f0.x * inv, f0.y * inv) | (to_e4m3x2(f1.x * inv, f1.y * inv) << 16);
          }
        }
        dst[u * T] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  // every thread read the old scale before the barrier behind the maximum
  if (tid == 0) *scale = now;
}

template <int T, int D>
__global__ void __launch_bounds__(T < 128 ? 128 : T) kv_append_kernel(const AppendArgs a) {
  append_unit<T, D, kAsIs>(a, nullptr, nullptr);
}

// The new tokens' rows of q, by the CTAs behind those of the cache: a warp takes a
// run of a sequence's tokens, or some heads of one token where there are few.
struct TurnArgs {
  Turning turning;
  const __nv_bfloat16* q;
  __nv_bfloat16* q_out;
  int64_t q_stride, q_out_stride, q_items;
  int h_q, run, runs, chunks, heads_per_chunk;
  unsigned kv_ctas;
  bool copy;
};

template <int D, bool kPairs>
__device__ __forceinline__ void turn_q(const AppendArgs& a, const TurnArgs& t, float* tab) {
  const int64_t item = (int64_t)(blockIdx.x - t.kv_ctas) * (blockDim.x / 32) + threadIdx.x / 32;
  if (item >= t.q_items) return;
  const int64_t i = item / ((int64_t)t.runs * t.chunks);
  const int rest = (int)(item - i * t.runs * t.chunks);
  const int start = a.start[i];
  int len = a.max_new;
  if (a.lens) len = min(max(a.lens[i], 0), a.max_new);
  const int first = rest / t.chunks * t.run, end = min(first + t.run, len);
  if (start < 0 || first >= end) return;
  const int64_t row0 = a.tok_start ? (int64_t)a.tok_start[i] : i * a.row_tokens;
  const int h0 = rest % t.chunks * t.heads_per_chunk, h1 = min(h0 + t.heads_per_chunk, t.h_q);
  uint64_t turns[4];
  load_turns(t.turning, turns);
  for (int j = first; j < end; ++j) {
    const int64_t row = row0 + j;
    if (row < 0 || row >= a.tokens) continue;
    // (a position past 32 bits is none: it is past every page table too)
    turn_token<__nv_bfloat16, kPairs>(t.q + row * t.q_stride, t.q_out + row * t.q_out_stride, nullptr, nullptr, D,
                                      t.h_q, h0, h1, t.copy, t.turning, (int)((uint32_t)start + (uint32_t)j), turns,
                                      tab + threadIdx.x / 32 * kMaxRot);
  }
}

template <int T, int D, int kTurn>
__global__ void __launch_bounds__(T < 128 ? 128 : T)
    kv_append_rope_kernel(const AppendArgs a, const __grid_constant__ TurnArgs t) {
  constexpr int kWarps = (T < 128 ? 128 : T) / 32;
  __shared__ __align__(16) union {
    uint64_t turns[kMaxRot / 2];
    float tab[kWarps * kMaxRot];
  } sm;
  if (blockIdx.x >= t.kv_ctas) {
    turn_q<D, kTurn == kInterleaved>(a, t, sm.tab);
    return;
  }
  if (threadIdx.x < t.turning.rot / 2) sm.turns[threadIdx.x] = turns_of(t.turning.freqs[threadIdx.x]);
  __syncthreads();
  append_unit<T, D, kTurn>(a, &t.turning, sm.turns);
}

template <int T, int D>
cudaError_t launch_append_t(const AppendArgs& a, TurnArgs* t, bool interleaved, cudaStream_t st) {
  constexpr int per_cta = T < 128 ? 128 / T : 1, kThreads = T < 128 ? 128 : T;
  const int64_t ctas = (a.units + per_cta - 1) / per_cta;
  if (!t) {
    if (ctas > 0x7fffffffll) return cudaErrorNotSupported;
    kv_append_kernel<T, D><<<(unsigned)ctas, kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  const int64_t q_ctas = (t->q_items + kThreads / 32 - 1) / (kThreads / 32);
  if (ctas > 0x7fffffffll || q_ctas > 0x7fffffffll - ctas) return cudaErrorNotSupported;
  t->kv_ctas = (unsigned)ctas;
  if (interleaved)
    kv_append_rope_kernel<T, D, kInterleaved><<<(unsigned)(ctas + q_ctas), kThreads, 0, st>>>(a, *t);
  else
    kv_append_rope_kernel<T, D, kHalf><<<(unsigned)(ctas + q_ctas), kThreads, 0, st>>>(a, *t);
  return cudaGetLastError();
}

// Threads per unit: the fewest whose registers hold the largest unit (one warp
// for up to 128 / (D / 16) tokens).
template <int D>
cudaError_t launch_append_d(const AppendArgs& a, TurnArgs* t, bool interleaved, cudaStream_t st) {
  const int chunks = (a.max_new < a.page_size ? a.max_new : a.page_size) * (D / 16);
  if (chunks <= 32 * kChunksPerThread) return launch_append_t<32, D>(a, t, interleaved, st);
  if (chunks <= 128 * kChunksPerThread) return launch_append_t<128, D>(a, t, interleaved, st);
  if (chunks <= 256 * kChunksPerThread) return launch_append_t<256, D>(a, t, interleaved, st);
  return launch_append_t<512, D>(a, t, interleaved, st);
}

// ---------------------------------------------------------------- page copies
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 8;  // 16-byte vectors in flight per thread
constexpr int kCopyChunk = kCopyThreads * kCopyVecs;

// One CTA moves one run of 32 KB of a page of K or of V.
__global__ void __launch_bounds__(kCopyThreads)
    kv_copy_kernel(uint8_t* kc, uint8_t* vc, float* ks, float* vs, const int* __restrict__ src,
                   const int* __restrict__ dst, int64_t page_stride, int page_vecs, int h_kv,
                   int num_pages, int runs) {
  const int run = blockIdx.x % runs;
  const unsigned rest = blockIdx.x / runs;
  const bool is_v = rest & 1u;
  const int64_t i = rest >> 1;
  const int s = src[i], d = dst[i];
  if (s < 0 || s >= num_pages || d < 0 || d >= num_pages || s == d) return;
  uint8_t* base = is_v ? vc : kc;
  const uint4* from = reinterpret_cast<const uint4*>(base + s * page_stride);
  uint4* to = reinterpret_cast<uint4*>(base + d * page_stride);
  const int v0 = run * kCopyChunk + threadIdx.x;
  uint4 x[kCopyVecs];
#pragma unroll
  for (int u = 0; u < kCopyVecs; ++u)
    if (v0 + u * kCopyThreads < page_vecs) x[u] = __ldcs(from + v0 + u * kCopyThreads);
#pragma unroll
  for (int u = 0; u < kCopyVecs; ++u)
    if (v0 + u * kCopyThreads < page_vecs) __stcs(to + v0 + u * kCopyThreads, x[u]);
  if (run == 0) {
    float* sc = is_v ? vs : ks;
    for (int h = threadIdx.x; h < h_kv; h += kCopyThreads)
      sc[(int64_t)d * h_kv + h] = sc[(int64_t)s * h_kv + h];
  }
}

}  // namespace

static AppendArgs append_args(const attn_kv_append_params& p) {
  const attn_kv_cache& c = p.cache;
  AppendArgs a;
  a.k = static_cast<const __nv_bfloat16*>(p.k);
  a.v = static_cast<const __nv_bfloat16*>(p.v);
  a.kc = static_cast<uint8_t*>(c.k);
  a.vc = static_cast<uint8_t*>(c.v);
  a.ks = c.k_scale;
  a.vs = c.v_scale;
  a.table = p.page_table;
  a.start = p.start;
  a.lens = p.lens;
  a.tok_start = p.tok_start;
  a.tokens = p.tokens;
  a.token_stride = p.token_stride > 0 ? p.token_stride : c.h_kv * c.d;
  a.row_tokens = p.row_tokens;
  a.page_stride = c.page_stride > 0 ? c.page_stride : c.h_kv * c.page_size * c.d;
  a.num_pages = (int)c.num_pages;
  a.h_kv = (int)c.h_kv;
  a.page_size = (int)c.page_size;
  a.max_pages = (int)p.max_pages;
  a.max_new = (int)p.max_new;
  // most pages that max_new tokens in a row can touch
  int64_t pages = (p.max_new + c.page_size - 2) / c.page_size + 1;
  if (pages > p.max_pages) pages = p.max_pages;
  a.pages_per_seq = (int)pages;
  a.units = p.n * pages * 2 * c.h_kv;
  return a;
}

static cudaError_t launch_append(const AppendArgs& a, TurnArgs* t, int64_t d, bool interleaved, cudaStream_t st) {
  if (d == 64) return launch_append_d<64>(a, t, interleaved, st);
  if (d == 128) return launch_append_d<128>(a, t, interleaved, st);
  return launch_append_d<256>(a, t, interleaved, st);
}

cudaError_t launch_kv_append(const attn_kv_append_params& p, cudaStream_t st) {
  return launch_append(append_args(p), nullptr, p.cache.d, false, st);
}

cudaError_t launch_kv_append_rope(const attn_kv_append_rope_params& p, cudaStream_t st) {
  const int64_t d = p.append.cache.d;
  const AppendArgs a = append_args(p.append);
  const attn_rotation& r = p.rotation;
  TurnArgs t;
  t.turning = Turning{r.freqs, (int)r.rot, (int)r.offset, r.amplitude == 0.f ? 1.f : r.amplitude, false};
  t.q = static_cast<const __nv_bfloat16*>(p.q);
  t.q_out = static_cast<__nv_bfloat16*>(p.q_out);
  t.q_stride = p.q_stride > 0 ? p.q_stride : p.h_q * d;
  t.q_out_stride = p.q_out_stride > 0 ? p.q_out_stride : p.h_q * d;
  t.h_q = (int)p.h_q;
  t.copy = p.q != p.q_out;
  t.run = t.runs = t.chunks = t.heads_per_chunk = 1;
  t.q_items = 0;
  if (p.h_q > 0) {
    // a warp for each of a run of tokens, or for some of one token's heads
    const int64_t warps = (int64_t)sm_count() * 64, tokens = p.append.n * p.append.max_new;
    const int64_t run = tokens / warps;
    t.run = (int)(run < 1 ? 1 : run > 32 ? 32 : run);
    t.runs = (int)((p.append.max_new + t.run - 1) / t.run);
    const int per = 32 / (int)((t.copy ? d : r.rot) / 16);
    const int64_t most = (p.h_q + per - 1) / per;
    int64_t chunks = warps / 4 / tokens;
    chunks = chunks < 1 ? 1 : chunks > most ? most : chunks;
    t.heads_per_chunk = (int)((p.h_q + chunks - 1) / chunks);
    t.chunks = (int)((p.h_q + t.heads_per_chunk - 1) / t.heads_per_chunk);
    t.q_items = p.append.n * t.runs * t.chunks;
  }
  return launch_append(a, &t, d, r.interleaved != 0, st);
}

cudaError_t launch_kv_copy(const attn_kv_cache& c, const int* src, const int* dst, int64_t n,
                           cudaStream_t st) {
  const int64_t page_bytes = c.h_kv * c.page_size * c.d;
  const int64_t vecs = page_bytes / 16;
  const int64_t runs = (vecs + kCopyChunk - 1) / kCopyChunk;
  const int64_t ctas = n * 2 * runs;
  if (ctas > 0x7fffffffll || vecs > 0x7fffffffll - kCopyChunk) return cudaErrorNotSupported;
  kv_copy_kernel<<<(unsigned)ctas, kCopyThreads, 0, st>>>(
      static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v), c.k_scale, c.v_scale, src, dst,
      c.page_stride > 0 ? c.page_stride : page_bytes, (int)vecs, (int)c.h_kv, (int)c.num_pages,
      (int)runs);
  return cudaGetLastError();
}

}  // namespace gb300
