// Appending to the paged 8-bit cache with the position rotation applied on the way:
//
//   K: (x1, x2) -> amp (x1 cos t - x2 sin t, x2 cos t + x1 sin t), t = pos * f_i, in fp32,
//      then the code e4m3(x / scale), scale the page's power of two
//   V: e4m3(x / scale);   q of the same tokens turned, rounded to bf16
//
// Bound by HBM: 2 bytes in and 1 out per value of K and V, 2 and 2 of q; by launch
// latency where a decoding step appends one token per sequence.  One launch does it
// all: CTAs of the cache and CTAs of q, spread evenly among each other, since the
// former spend instructions on angles (8 pairs of cos and sin a chunk of 16 values) and
// the latter, which share a token's angles among its heads, next to none.  Two prompts of
// 32768 tokens (Hq 32, Hkv 8, d 128): 254 us, 5.8 TB/s; one token of 32 sequences 4.4 us.
#include "kv_cache.cuh"

namespace gb300 {

namespace {

struct TurnArgs {
  Turning turning;
  const __nv_bfloat16* q;
  __nv_bfloat16* q_out;
  int64_t q_stride, q_out_stride, q_items;
  int h_q, run, runs, chunks, heads_per_chunk;
  unsigned q_ctas;
  bool copy;
};

// The new tokens' rows of q: a warp takes a run of a sequence's tokens, or some heads
// of one token where there are few.
template <int D, bool kPairs>
__device__ __forceinline__ void turn_q(const AppendArgs& a, const TurnArgs& t, unsigned block, float* tab) {
  const int64_t item = (int64_t)block * (blockDim.x / 32) + threadIdx.x / 32;
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
    // (positions past 31 bits wrap: no page table goes there)
    turn_token<__nv_bfloat16, kPairs, 2, false>(t.q + row * t.q_stride, t.q_out + row * t.q_out_stride, nullptr, nullptr, D,
                                      t.h_q, h0, h1, t.copy, t.turning, (int)((uint32_t)start + (uint32_t)j), turns,
                                      tab + threadIdx.x / 32 * kMaxRot);
  }
}

// 8 codes of 8 values.
__device__ __forceinline__ uint2 codes_of(const float* x, float inv) {
  return make_uint2(to_e4m3x2(x[0] * inv, x[1] * inv) | (to_e4m3x2(x[2] * inv, x[3] * inv) << 16),
                    to_e4m3x2(x[4] * inv, x[5] * inv) | (to_e4m3x2(x[6] * inv, x[7] * inv) << 16));
}

// T threads take one unit: the new tokens of one sequence that fall on one page, for
// one head of K or of V, in chunks of 16 values (the units of rotation.cuh, whose pairs
// are their own; kC a thread).  They stay in registers, K's turned, between the largest
// magnitude and the codes, so every value is read once.
template <int T, int kC, int D, bool kPairs>
__device__ __forceinline__ void append_unit(const AppendArgs& a, const Turning& t, unsigned block,
                                            const uint64_t* s_turns) {
  constexpr int kUnits = T < 128 ? 128 / T : 1;  // units per CTA
  constexpr int kRowChunks = D / 16;
  const int tid = threadIdx.x % T;
  const int64_t unit = (int64_t)block * kUnits + threadIdx.x / T;
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

  uint8_t* page = (is_v ? a.vc : a.kc) + pid * a.page_stride + (int64_t)h * a.page_size * D;
  float* scale = (is_v ? a.vs : a.ks) + (int64_t)pid * a.h_kv + h;
  const float old = lo > 0 ? *scale : 0.f;

  const int chunks = (hi - lo) * kRowChunks;
  constexpr int kStep = T / kRowChunks;  // tokens between a thread's chunks (T % kRowChunks == 0)
  const HeadUnits<__nv_bfloat16, kPairs> units(D, t.rot, true);
  const int u = tid % kRowChunks, slot = lo + tid / kRowChunks;
  // the first values of the chunk's two vectors
  const int va = is_v ? 16 * u : units.at(u, 0, t.rot, t.offset), vb = is_v ? va + 8 : units.at(u, 1, t.rot, t.offset);
  const __nv_bfloat16* row = (is_v ? a.v : a.k) + (int64_t)h * D + (at0 + slot) * a.token_stride;
  uint4 r[kC][2];
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    r[c][0] = r[c][1] = make_uint4(0u, 0u, 0u, 0u);
    if (c * T + tid < chunks) {
      r[c][0] = __ldg(reinterpret_cast<const uint4*>(row + (int64_t)c * kStep * a.token_stride + va));
      r[c][1] = __ldg(reinterpret_cast<const uint4*>(row + (int64_t)c * kStep * a.token_stride + vb));
    }
  }
  float x[kC][16];
  float amax = 0.f;
  const bool turning = !is_v && u < units.turning;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const uint32_t w[8] = {r[c][0].x, r[c][0].y, r[c][0].z, r[c][0].w, r[c][1].x, r[c][1].y, r[c][1].z, r[c][1].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 f = widen_bf16x2(w[e]);
      x[c][2 * e] = f.x;
      x[c][2 * e + 1] = f.y;
    }
    if (turning) {
      const int pos = (int)page_first + slot + c * kStep;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 f = cos_sin(pos, s_turns[8 * u + e], t.amp);
        const int p = kPairs ? 2 * e : e, q = kPairs ? 2 * e + 1 : e + 8;
        const float y = x[c][p], z = x[c][q];
        x[c][p] = y * f.x - z * f.y;
        x[c][q] = z * f.x + y * f.y;
      }
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[c][e]));  // (NaN counts as nothing)
  }
  if (!(amax < INFINITY)) {  // infinities: only what is finite counts
    amax = 0.f;
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float m = fabsf(x[c][e]);
        if (m < INFINITY) amax = fmaxf(amax, m);
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
    __syncwarp();  // everybody has read the old scale
  }
  const float need = pow2f(scale_exponent(__uint_as_float(bits)));
  const bool grew = lo > 0 && need > old;
  const float now = lo > 0 && !grew ? old : need;
  const float inv = 1.f / now;  // exact: scales that these kernels write are powers of two
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
  uint8_t* dst = page + (int64_t)slot * D;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    if (c * T + tid < chunks) {
      *reinterpret_cast<uint2*>(dst + c * kStep * D + va) = codes_of(x[c], inv);
      *reinterpret_cast<uint2*>(dst + c * kStep * D + vb) = codes_of(x[c] + 8, inv);
    }
  }
  if (tid == 0) *scale = now;
}

// (two prompts of 32768 tokens: 276 us at 80 registers, 254 at 64)
template <int T>
constexpr int kMinCtas = T <= 128 ? 8 : T == 256 ? 4 : 1;

template <int T, int kC, int D, bool kPairs>
__global__ void __launch_bounds__(T < 128 ? 128 : T, kMinCtas<T>)
    kv_append_rope_kernel(const AppendArgs a, const __grid_constant__ TurnArgs t) {
  constexpr int kWarps = (T < 128 ? 128 : T) / 32;
  __shared__ __align__(16) union {
    uint64_t turns[kMaxRot / 2];
    float tab[kWarps * kMaxRot];
  } sm;
  // CTA b is one of q where the share of those before it passes a whole number
  const unsigned b = blockIdx.x, q_before = (unsigned)((uint64_t)b * t.q_ctas / gridDim.x);
  if ((uint64_t)(b + 1) * t.q_ctas / gridDim.x > q_before) {
    turn_q<D, kPairs>(a, t, q_before, sm.tab);
    return;
  }
  if (threadIdx.x < t.turning.rot / 2) sm.turns[threadIdx.x] = turns_of(t.turning.freqs[threadIdx.x]);
  __syncthreads();
  append_unit<T, kC, D, kPairs>(a, t.turning, b - q_before, sm.turns);
}

template <int T, int kC, int D>
cudaError_t launch_t(const AppendArgs& a, TurnArgs& t, bool interleaved, cudaStream_t st) {
  constexpr int per_cta = T < 128 ? 128 / T : 1, kThreads = T < 128 ? 128 : T;
  const int64_t kv_ctas = (a.units + per_cta - 1) / per_cta, q_ctas = (t.q_items + kThreads / 32 - 1) / (kThreads / 32);
  if (kv_ctas > 0x7fffffffll || q_ctas > 0x7fffffffll - kv_ctas) return cudaErrorNotSupported;
  t.q_ctas = (unsigned)q_ctas;
  const unsigned grid = (unsigned)(kv_ctas + q_ctas);
  if (interleaved)
    kv_append_rope_kernel<T, kC, D, true><<<grid, kThreads, 0, st>>>(a, t);
  else
    kv_append_rope_kernel<T, kC, D, false><<<grid, kThreads, 0, st>>>(a, t);
  return cudaGetLastError();
}

// Two chunks a thread (four, with their 16 values in fp32, took 161 registers: 323 us for two
// prompts of 32768 tokens where two took 277), four for units of more than 1024.
template <int D>
cudaError_t launch_d(const AppendArgs& a, TurnArgs& t, bool interleaved, cudaStream_t st) {
  const int chunks = (a.max_new < a.page_size ? a.max_new : a.page_size) * (D / 16);
  if (chunks <= 64) return launch_t<32, 2, D>(a, t, interleaved, st);
  if (chunks <= 256) return launch_t<128, 2, D>(a, t, interleaved, st);
  if (chunks <= 512) return launch_t<256, 2, D>(a, t, interleaved, st);
  if (chunks <= 1024) return launch_t<512, 2, D>(a, t, interleaved, st);
  return launch_t<512, 4, D>(a, t, interleaved, st);
}

}  // namespace

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
  if (d == 64) return launch_d<64>(a, t, r.interleaved != 0, st);
  if (d == 128) return launch_d<128>(a, t, r.interleaved != 0, st);
  return launch_d<256>(a, t, r.interleaved != 0, st);
}

}  // namespace gb300
