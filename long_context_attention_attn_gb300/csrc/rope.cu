// Position rotation of q and k rows, and of their gradients (the same by the negative
// angle: the transposed map).
//
//   y1 = amp (x1 cos t - x2 sin t),  y2 = amp (x2 cos t + x1 sin t),  t = pos * f_i
//
// Bound by HBM: every value is read and written once, with 3 flops.  A warp takes a
// token: its angles once, for all heads, then 32 lanes' worth of rows at a time stream
// through.  65536 tokens of 40 heads of 192 (64 turn): 297 us, 6.79 TB/s; 16384 tokens of 20
// heads of 128 29.6 us, 5.7 TB/s, in fp32 53.6 us, 6.3 TB/s; of 256, where a warp has one fp32 head
// at a time, 102 us, 6.6 TB/s.
#include "internal.h"
#include "rotation.cuh"

namespace gb300 {

namespace {

constexpr int kWarps = 4;

struct RopeArgs {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  const int* pos;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride, items;
  int h_q, h, d, chunks, heads_per_chunk;
  bool copy;
  Turning turning;
};

template <typename E, bool kInterleaved>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ __align__(16) float tab[kWarps][kMaxRot];
  const int warp = threadIdx.x / 32;
  uint64_t turns[4];
  load_turns(a.turning, turns);
  const int64_t step = (int64_t)gridDim.x * kWarps;
  for (int64_t item = (int64_t)blockIdx.x * kWarps + warp; item < a.items; item += step) {
    const int64_t token = item / a.chunks;
    const int h0 = (int)(item - token * a.chunks) * a.heads_per_chunk;
    turn_token<E, kInterleaved, 4, true>(static_cast<const E*>(a.q) + token * a.q_stride,
                                static_cast<E*>(a.q_out) + token * a.q_out_stride,
                                static_cast<const E*>(a.k) + token * a.k_stride,
                                static_cast<E*>(a.k_out) + token * a.k_out_stride, a.d, a.h_q, h0,
                                min(h0 + a.heads_per_chunk, a.h), a.copy, a.turning, a.pos[token], turns, tab[warp]);
  }
}

template <typename E>
cudaError_t launch(const RopeArgs& a, bool interleaved, cudaStream_t st) {
  const int64_t need = (a.items + kWarps - 1) / kWarps;
  // (65536 tokens of 40 heads of 192: 325 us with 12 CTAs per SM, 299 with 24, 299 with 64)
  const int64_t most = (int64_t)sm_count() * 24;
  const unsigned grid = (unsigned)(need < most ? need : most);
  if (interleaved)
    rope_kernel<E, true><<<grid, kWarps * 32, 0, st>>>(a);
  else
    rope_kernel<E, false><<<grid, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const attn_rope_params& p, cudaStream_t st) {
  RopeArgs a;
  a.q = p.q;
  a.k = p.k;
  a.q_out = p.q_out;
  a.k_out = p.k_out;
  a.pos = p.pos;
  a.q_stride = p.q_stride > 0 ? p.q_stride : p.h_q * p.d;
  a.k_stride = p.k_stride > 0 ? p.k_stride : p.h_k * p.d;
  a.q_out_stride = p.q_out_stride > 0 ? p.q_out_stride : p.h_q * p.d;
  a.k_out_stride = p.k_out_stride > 0 ? p.k_out_stride : p.h_k * p.d;
  a.h_q = (int)p.h_q;
  a.h = (int)(p.h_q + p.h_k);
  a.d = (int)p.d;
  a.copy = (p.h_q > 0 && p.q != p.q_out) || (p.h_k > 0 && p.k != p.k_out);
  const attn_rotation& r = p.rotation;
  a.turning = Turning{r.freqs, (int)r.rot, (int)r.offset, r.amplitude == 0.f ? 1.f : r.amplitude, p.inverse != 0};
  // Few tokens: several warps share a token's heads, down to one round of loads each.
  const int values = p.fp32 ? 8 : 16;  // of a unit
  const int per = 32 / (a.copy ? a.d / values : a.turning.rot / values);
  int64_t chunks = (int64_t)sm_count() * 16 / p.tokens;
  const int64_t most = (a.h + per - 1) / per;
  chunks = chunks < 1 ? 1 : chunks > most ? most : chunks;
  a.heads_per_chunk = (int)((a.h + chunks - 1) / chunks);
  a.chunks = (a.h + a.heads_per_chunk - 1) / a.heads_per_chunk;
  a.items = p.tokens * a.chunks;
  return p.fp32 ? launch<float>(a, r.interleaved != 0, st) : launch<__nv_bfloat16>(a, r.interleaved != 0, st);
}

}  // namespace gb300
