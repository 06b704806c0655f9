// attn_decode: attention of a few query tokens per sequence over the paged 8-bit cache
// (the kernels: attn_decode_kernels.cuh).
#include "attn_decode_kernels.cuh"

namespace gb300 {

namespace {

template <typename F>
cudaError_t dispatch(const attn_decode_params& p, F&& f) {
  const int64_t rows = p.s_q * (p.h_q / p.cache.h_kv);
  if (p.cache.d == 64) return with_rows<64, kWhole>(p, 0, rows, f);
  if (p.cache.d == 128) return with_rows<128, kWhole>(p, 0, rows, f);
  return with_rows<256, kWhole>(p, 0, rows, f);
}

}  // namespace

cudaError_t decode_workspace(const attn_decode_params& p, size_t* bytes) {
  return dispatch(p, [&](auto k, const Shape& sh) {
    const size_t rows = (size_t)sh.runs * sh.row_tiles * decltype(k)::C::R;
    *bytes = sh.cluster ? 0 : align_up(2 * rows * (p.cache.d + 1) * 4, 256);
    return cudaSuccess;
  });
}

cudaError_t launch_attn_decode(const attn_decode_params& p, cudaStream_t st) {
  return launch_attn_decode(p, false, st);
}

cudaError_t launch_attn_decode(const attn_decode_params& p, bool withhold, cudaStream_t st) {
  DecodeArgs a = decode_args(p);
  a.withhold = withhold ? 1 : 0;
  return dispatch(p, [&](auto k, const Shape& sh) {
    const cudaError_t e = k.launch(a, sh, false, st);
    return e != cudaSuccess || sh.cluster ? e : k.fold(a, st);
  });
}

}  // namespace gb300
