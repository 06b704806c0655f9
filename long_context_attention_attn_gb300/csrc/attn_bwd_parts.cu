// Parts of key tiles that hold kept tokens (backward; PartHeader in internal.h):
// the list of parts from the tile plan, and the fold of their dK / dV.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace gb300 {

namespace {

constexpr int kListThreads = 1024;

// One CTA.  A key tile sees at most window / 128 + 2 query tiles through the
// window; tiles above that and above 2 / max_parts of all work are cut into
// equal runs of their query-tile range.  A tile of w over the cap takes at most
// 2 w / cap parts, so max_parts is never exceeded.
__global__ void __launch_bounds__(kListThreads)
    key_parts_kernel(const int* __restrict__ weight, const int2* __restrict__ range, int n, int least,
                     KeyParts kp) {
  __shared__ unsigned long long warp_sum[32];
  __shared__ unsigned long long s_base;  // parts so far, tiles so far in the high word
  const int t = threadIdx.x, lane = t & 31, wid = t >> 5;
  unsigned long long sum = 0;
  for (int i = t; i < n; i += kListThreads) sum += weight[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) warp_sum[wid] = sum;
  if (t == 0) s_base = 0;
  __syncthreads();
  unsigned long long total = 0;
  for (int w = 0; w < kListThreads / 32; ++w) total += warp_sum[w];
  const unsigned long long share = (2 * total + kp.max_parts - 1) / kp.max_parts;
  const int cap = (int)(share > (unsigned long long)least ? share : least);
  for (int i0 = 0; i0 < n; i0 += kListThreads) {
    const int i = i0 + t;
    const int w = i < n ? weight[i] : 0;
    const int parts = w > cap ? (w + cap - 1) / cap : 0;
    const unsigned long long mine = parts ? ((1ull << 32) | (unsigned)parts) : 0ull;
    unsigned long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    __syncthreads();  // warp_sum is free
    if (lane == 31) warp_sum[wid] = incl;
    __syncthreads();
    unsigned long long base = s_base;
    for (int v = 0; v < wid; ++v) base += warp_sum[v];
    const unsigned long long before = base + incl - mine;
    if (parts) {
      const int first = (int)(uint32_t)before, tile = (int)(before >> 32);
      const int2 r = range[i];
      const int len = r.y - r.x + 1;
      kp.tiles[tile] = make_int4(i, first, parts, 0);
      for (int c = 0; c < parts; ++c)
        kp.parts[first + c] = make_int4(i, r.x + (int)((int64_t)len * c / parts),
                                        r.x + (int)((int64_t)len * (c + 1) / parts) - 1, 0);
    }
    __syncthreads();
    if (t == kListThreads - 1) s_base = base + incl;
    __syncthreads();
  }
  if (t == 0) *kp.header = PartHeader{cap, (int)(uint32_t)s_base, (int)(s_base >> 32), 0};
}

constexpr int kFoldRows = 8;  // key rows per CTA
constexpr int kFoldThreads = 256;

// dK / dV of a cut key tile: its parts' sums, in order.
__global__ void __launch_bounds__(kFoldThreads)
    fold_parts_kernel(const KeyParts kp, void* dk, void* dv, int64_t k_stride, int64_t v_stride, int nk,
                      int s_kv, int hkv, int d, int d_v, int accumulate) {
  if ((int)blockIdx.x >= kp.header->n_tiles) return;
  const int4 tile = kp.tiles[blockIdx.x];
  const int kvh = blockIdx.y;
  const int bi = tile.x / nk, kt = tile.x % nk;
  const int width = d + d_v, vecs = width / 4;
  const int64_t part_step = (int64_t)hkv * 128 * width;
  for (int u = threadIdx.x; u < kFoldRows * vecs; u += kFoldThreads) {
    const int row = blockIdx.z * kFoldRows + u / vecs, c = 4 * (u % vecs);
    const int key = kt * 128 + row;
    if (key >= s_kv) break;
    const float* src = kp.buf + (((int64_t)tile.y * hkv + kvh) * 128 + row) * width + c;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < tile.z; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(src + i * part_step);
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
    const bool is_v = c >= d;
    const int64_t at = ((int64_t)bi * s_kv + key) * (is_v ? v_stride : k_stride) +
                       (int64_t)kvh * (is_v ? d_v : d) + (is_v ? c - d : c);
    void* out = is_v ? dv : dk;
    if (accumulate) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
      const float4 x = *p;
      *p = make_float4(x.x + s.x, x.y + s.y, x.z + s.z, x.w + s.w);
    } else {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
          make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
    }
  }
}

}  // namespace

cudaError_t launch_key_parts(const attn_fwd_params& f, const PlanPtrs& pp, int64_t nk,
                             const KeyParts& kp, cudaStream_t st) {
  key_parts_kernel<<<1, kListThreads, 0, st>>>(pp.kv_weight, pp.kv_range, (int)(f.b * nk), (int)least_cut(f),
                                           kp);
  return cudaGetLastError();
}

cudaError_t launch_fold_parts(const attn_bwd_params& p, int64_t nk, const KeyParts& kp,
                              cudaStream_t st) {
  const attn_fwd_params& f = p.fwd;
  const int64_t dv = f.d_v > 0 ? f.d_v : f.d;
  const int64_t ks = f.kv_token_stride > 0 ? f.kv_token_stride : f.h_kv * f.d;
  const int64_t vs = f.kv_token_stride > 0 ? f.kv_token_stride : f.h_kv * dv;
  // a cut tile has two parts or more
  const dim3 grid((unsigned)((kp.max_parts + 1) / 2), (unsigned)f.h_kv, 128 / kFoldRows);
  fold_parts_kernel<<<grid, kFoldThreads, 0, st>>>(kp, p.dk, p.dv, ks, vs, (int)nk, (int)f.s_kv, (int)f.h_kv,
                                                   (int)f.d, (int)dv, p.accumulate_fp32 ? 1 : 0);
  return cudaGetLastError();
}

}  // namespace gb300
