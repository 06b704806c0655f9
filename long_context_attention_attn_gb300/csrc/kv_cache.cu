// The paged 8-bit key / value cache: appending tokens and copying pages.
//
// Both are bound by HBM traffic (append: 2 bytes in and 1 out per value; copy:
// 1 in and 1 out), and by launch latency where a decoding step appends one
// token per sequence.
#include "kv_cache.cuh"

namespace gb300 {

namespace {

constexpr int kChunksPerThread = 4;  // 16-value chunks a thread holds in registers

// T threads take one unit: the new tokens of one sequence that fall on one
// page, for one head of K or of V.  They hold the unit's values in registers
// (T * 4 chunks of 16 values cover it), so every value is read once: the
// largest magnitude first, then the codes.  Neighbouring units are the heads
// of the same tokens, whose rows are neighbours in memory.
template <int T, int D>
__global__ void __launch_bounds__(T < 128 ? 128 : T) kv_append_kernel(const AppendArgs a) {
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
  const uint4* src = reinterpret_cast<const uint4*>(x + (at0 + lo + tid / kRowChunks) * a.token_stride) +
                     2 * (tid % kRowChunks);
  const int64_t step = (int64_t)(T / kRowChunks) * a.token_stride / 8;  // T % kRowChunks == 0
  uint4 r[kChunksPerThread][2];
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
  float amax = __uint_as_float(max(top << 16, top & 0xffff0000u));
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
  // every thread read the old scale before the barrier behind the maximum
  if (tid == 0) *scale = now;
}

template <int T, int D>
cudaError_t launch_append_t(const AppendArgs& a, cudaStream_t st) {
  constexpr int per_cta = T < 128 ? 128 / T : 1;
  const int64_t ctas = (a.units + per_cta - 1) / per_cta;
  if (ctas > 0x7fffffffll) return cudaErrorNotSupported;
  kv_append_kernel<T, D><<<(unsigned)ctas, T < 128 ? 128 : T, 0, st>>>(a);
  return cudaGetLastError();
}

// Threads per unit: the fewest whose registers hold the largest unit (one warp
// for up to 128 / (D / 16) tokens).
template <int D>
cudaError_t launch_append_d(const AppendArgs& a, cudaStream_t st) {
  const int chunks = (a.max_new < a.page_size ? a.max_new : a.page_size) * (D / 16);
  if (chunks <= 32 * kChunksPerThread) return launch_append_t<32, D>(a, st);
  if (chunks <= 128 * kChunksPerThread) return launch_append_t<128, D>(a, st);
  if (chunks <= 256 * kChunksPerThread) return launch_append_t<256, D>(a, st);
  return launch_append_t<512, D>(a, st);
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

cudaError_t launch_kv_append(const attn_kv_append_params& p, cudaStream_t st) {
  const AppendArgs a = append_args(p);
  if (p.cache.d == 64) return launch_append_d<64>(a, st);
  if (p.cache.d == 128) return launch_append_d<128>(a, st);
  return launch_append_d<256>(a, st);
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
