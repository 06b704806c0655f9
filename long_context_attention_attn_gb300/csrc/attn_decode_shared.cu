// attn_decode_shared: attn_decode for groups of sequences whose first pages are the same,
// which are read once for all of a group.
//
//   keys [0, P) of a group:     one list whose items are (group, kv head, tile of rows),
//                               the rows being those of all members
//   keys [P, ..) of a sequence: attn_decode's list, counted from the first own key
//
// Both are lists of attn_decode_kernels.cuh, whose kernels leave finished partials (O, lse
// in base 2) in the workspace; the last kernel folds a row's, shared ones first, in
// their order, so results do not depend on timing:
//   lse = log2 sum 2^lse_i,  O = sum 2^(lse_i - lse) O_i
//
// The shared keys have members * s_q * g rows, 4 d flops each for 2 d bytes: from about
// 140 rows on they are bound by the products, below by reading the keys; the own
// keys by reading them (a group's rows would be 2 d bytes each without sharing).
#include "attn_decode_kernels.cuh"

namespace gb300 {

namespace {

// What one list's kernel leaves.
struct Part {
  const float* part_o;    // pieces of items that several CTAs took
  const float* part_lse;
  const float* whole_o;   // [n, s_q, h_q, D]: rows of items that one CTA took
  const float* whole_lse; // [n, h_q, s_q]
  int block, item_cost, tile, runs, row_tiles;
};

constexpr int kFoldMost = 32;  // pieces at a time

// Where a row's pieces lie.
struct RowPieces {
  int64_t c0, s0, run;  // first CTA's run, first block of the item
  int n, rt, in_tile;   // pieces, row tile, row in the tile
};

// A list with its runs, as its kernel cuts it.
struct List {
  DecodeArgs a;
  Part part;
  int64_t run;
};

template <int M>
__device__ __forceinline__ RowPieces pieces_of(const List& l, const Entry& e, int64_t entry_at, int kvh, int row) {
  RowPieces p;
  p.rt = row / l.part.tile;
  p.in_tile = row - p.rt * l.part.tile;
  const int64_t item = M == kShared ? (int64_t)kvh * e.tiles + p.rt : kvh;
  p.s0 = entry_at + item * e.span.weight + l.part.item_cost;
  p.run = l.run;
  p.c0 = p.s0 / l.run;
  p.n = e.span.count ? (int)((p.s0 + e.span.count - 1) / l.run - p.c0) + 1 : 0;
  if (M == kShared) p.rt = 0;  // (a CTA's run has all of its tiles)
  return p;
}

// Row of part_o / part_lse of piece i.
__device__ __forceinline__ int64_t piece_row(const Part& l, const RowPieces& p, int i) {
  // a piece that starts inside its item is the first of its CTA, one that ends inside it the last
  const int64_t slot = 2 * ((p.c0 + i) * l.row_tiles + p.rt) + ((p.c0 + i) * p.run <= p.s0 ? 1 : 0);
  return slot * l.tile + p.in_tile;
}

// One thread per four values of a row, the rows of an item over blockIdx.y.
template <int D>
__global__ void __launch_bounds__(kFoldThreads)
    decode_shared_fold_kernel(const DecodeArgs a, const Part shared, const Part own, int n_groups) {
  constexpr int kVec = D / 4, RP = kFoldThreads / kVec;
  __shared__ int64_t before_s[kThreads + 1], before_o[kThreads + 1];
  __shared__ RowPieces rows_s[RP], rows_o[RP];
  __shared__ float s_w[kFoldMost][RP];
  __shared__ float s_ref[RP], s_old[RP];
  __shared__ int s_most;
  List ls{a, shared, 0}, lo{a, own, 0};
  ls.a.n = n_groups;
  ls.a.runs = shared.runs;
  lo.a.runs = own.runs;
  const Placement ps = place<kShared>(ls.a, before_s, shared.block, shared.item_cost, shared.tile);
  const Placement po = place<kOwn>(lo.a, before_o, own.block, own.item_cost, own.tile);
  ls.run = run_length(ls.a, before_s[kThreads] * a.h_kv);
  lo.run = run_length(lo.a, before_o[kThreads] * a.h_kv);
  const int kvh = blockIdx.x % a.h_kv, seq = blockIdx.x / a.h_kv, r0 = blockIdx.y * RP;
  if (threadIdx.x == 0) s_most = 0;
  __syncthreads();
  if (threadIdx.x < RP) {
    // the sequence's group: the last one that starts at or before it
    int lo_g = 0, hi_g = n_groups;
    while (hi_g - lo_g > 1) {
      const int mid = (lo_g + hi_g) / 2;
      if (group_bound(a, mid) <= seq)
        lo_g = mid;
      else
        hi_g = mid;
    }
    const int row = r0 + threadIdx.x;
    RowPieces s, o;
    s.n = o.n = 0;
    if (row < a.rows) {
      const Entry eg = entry_of<kShared>(ls.a, lo_g, shared.block, shared.item_cost, shared.tile);
      const int in_group = seq - eg.first;
      if (in_group >= 0 && (in_group + 1) * a.rows <= eg.rows && a.lens[seq] - a.s_q + row / a.g >= 0) {
        const int t = lo_g / ps.per;
        int64_t at = before_s[t];
        for (int i = t * ps.per; i < lo_g; ++i) {
          const Entry e = entry_of<kShared>(ls.a, i, shared.block, shared.item_cost, shared.tile);
          at += (int64_t)e.span.weight * e.tiles;
        }
        s = pieces_of<kShared>(ls, eg, at * a.h_kv, kvh, in_group * a.rows + row);
      }
      const int t = seq / po.per;
      int64_t at = before_o[t];
      for (int i = t * po.per; i < seq; ++i)
        at += entry_of<kOwn>(lo.a, i, own.block, own.item_cost, own.tile).span.weight;
      o = pieces_of<kOwn>(lo, entry_of<kOwn>(lo.a, seq, own.block, own.item_cost, own.tile), at * a.h_kv, kvh, row);
    }
    rows_s[threadIdx.x] = s;
    rows_o[threadIdx.x] = o;
    atomicMax(&s_most, s.n + o.n);
    s_ref[threadIdx.x] = -INFINITY;
  }
  __syncthreads();
  const int most = s_most;
  // everything the two grids before this one wrote
  asm volatile("griddepcontrol.wait;" ::: "memory");

  struct Source {
    const float* o;
    const float* lse;
  };
  // piece i of the CTA's row r: its values and its lse
  auto source = [&](int r, int i) {
    const RowPieces& s = rows_s[r];
    const bool sh = i < s.n;
    const RowPieces& p = sh ? s : rows_o[r];
    const Part& l = sh ? shared : own;
    if (p.n == 1) {
      const int row = r0 + r, tok = row / a.g, head = kvh * a.g + row % a.g;
      return Source{l.whole_o + (((int64_t)seq * a.s_q + tok) * a.h_q + head) * D,
                    l.whole_lse + ((int64_t)seq * a.h_q + head) * a.s_q + tok};
    }
    const int64_t at = piece_row(l, p, sh ? i : i - s.n);
    return Source{l.part_o + at * D, l.part_lse + at};
  };
  const int r = threadIdx.x / kVec, d4 = threadIdx.x % kVec;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float z = 0.f;
  for (int b0 = 0; b0 < most; b0 += kFoldMost) {
    const int np = min(kFoldMost, most - b0);
    for (int u = threadIdx.x; u < np * RP; u += kFoldThreads) {
      const int i = u / RP, row = u % RP;
      s_w[i][row] = b0 + i < rows_s[row].n + rows_o[row].n ? *source(row, b0 + i).lse : -INFINITY;
    }
    __syncthreads();
    if (threadIdx.x < RP) {
      float top = s_ref[threadIdx.x];
      for (int i = 0; i < np; ++i) top = fmaxf(top, s_w[i][threadIdx.x]);
      s_old[threadIdx.x] = top == -INFINITY ? 0.f : ex2(s_ref[threadIdx.x] - top);
      s_ref[threadIdx.x] = top;
    }
    __syncthreads();
    const float top = s_ref[r], ref = top == -INFINITY ? 0.f : top, old = s_old[r];
    z *= old;
    acc.x *= old;
    acc.y *= old;
    acc.z *= old;
    acc.w *= old;
    const int mine = min(np, rows_s[r].n + rows_o[r].n - b0);
#pragma unroll 4
    for (int i = 0; i < mine; ++i) {
      const float f = ex2(s_w[i][r] - ref);
      const float4 v = reinterpret_cast<const float4*>(source(r, b0 + i).o)[d4];
      z += f;
      acc.x += v.x * f;
      acc.y += v.y * f;
      acc.z += v.z * f;
      acc.w += v.w * f;
    }
    __syncthreads();
  }
  const int row = r0 + r;
  if (row >= a.rows) return;
  const float inv = z == 0.f ? 0.f : 1.f / z;
  const int tok = row / a.g, head = kvh * a.g + row % a.g;
  const int64_t orow = ((int64_t)seq * a.s_q + tok) * a.h_q + head;
  const float4 o = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  if (a.out_fp32)
    reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * D)[d4] = o;
  else
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * D)[d4] =
        make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
  if (d4 == 0)
    a.lse[((int64_t)seq * a.h_q + head) * a.s_q + tok] = z == 0.f ? -INFINITY : (s_ref[r] + log2f(z)) * kLn2;
}

// f(kernel of the shared keys, its shape, kernel of the own keys, its shape)
template <int D, typename F>
cudaError_t with_both(const attn_decode_shared_params& p, F&& f) {
  const attn_decode_params& q = p.base;
  const int64_t rows = q.s_q * (q.h_q / q.cache.h_kv);
  return with_rows<D, kShared>(q, p.n_groups, p.max_group * rows, [&](auto ks, const Shape& ss) {
    return with_rows<D, kOwn>(q, 0, rows, [&](auto ko, const Shape& so) { return f(ks, ss, ko, so); });
  });
}

template <typename F>
cudaError_t dispatch(const attn_decode_shared_params& p, F&& f) {
  if (p.base.cache.d == 64) return with_both<64>(p, f);
  if (p.base.cache.d == 128) return with_both<128>(p, f);
  return with_both<256>(p, f);
}

// Floats of a list's partials, and of a problem's rows.
template <typename K>
size_t part_floats(const Shape& sh, int64_t d) {
  return align_up(2 * (size_t)sh.runs * sh.row_tiles * K::C::R * (d + 1), 64);
}
size_t row_floats(const attn_decode_params& p) { return align_up((size_t)p.n * p.s_q * p.h_q * (p.cache.d + 1), 64); }

template <typename K>
Part part_of(const DecodeArgs& a, const Shape& sh) {
  return Part{a.part_o, a.part_lse, static_cast<const float*>(a.out), a.lse, K::T::kBlock, K::T::kItemCost, K::C::R,
              sh.runs, sh.row_tiles};
}

}  // namespace

cudaError_t decode_shared_workspace(const attn_decode_shared_params& p, size_t* bytes) {
  if (p.max_group <= 1) return decode_workspace(p.base, bytes);
  return dispatch(p, [&](auto ks, const Shape& ss, auto ko, const Shape& so) {
    *bytes = 4 * (part_floats<decltype(ks)>(ss, p.base.cache.d) + part_floats<decltype(ko)>(so, p.base.cache.d) +
                  2 * row_floats(p.base));
    return cudaSuccess;
  });
}

cudaError_t launch_attn_decode_shared(const attn_decode_shared_params& p, bool withhold, cudaStream_t st) {
  const attn_decode_params& q = p.base;
  // (no group has two members: nothing is read twice)
  if (p.max_group <= 1) return launch_attn_decode(q, withhold, st);
  return dispatch(p, [&](auto ks, const Shape& ss, auto ko, const Shape& so) {
    using KS = decltype(ks);
    using KO = decltype(ko);
    constexpr int D = KS::kD;
    const DecodeArgs a = [&] {
      DecodeArgs x = decode_args(q);
      x.shared_pages = p.shared_pages;
      x.group_start = p.group_start;
      return x;
    }();
    const size_t row_values = (size_t)q.n * q.s_q * q.h_q * D;
    float* ws = static_cast<float*>(q.workspace);
    DecodeArgs s = a, o = a;
    s.n = (int)p.n_groups;
    s.withhold = withhold ? 1 : 0;
    s.part_o = ws;
    o.part_o = s.part_o + part_floats<KS>(ss, D);
    float* rows = o.part_o + part_floats<KO>(so, D);
    s.out = rows;
    s.lse = rows + row_values;
    o.out = rows + row_floats(q);
    o.lse = rows + row_floats(q) + row_values;
    s.out_fp32 = o.out_fp32 = 1;
    cudaError_t e = ks.launch(s, ss, false, st);
    if (e == cudaSuccess) e = ko.launch(o, so, true, st);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    constexpr int RP = kFoldThreads / (D / 4);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)(q.n * q.cache.h_kv), (unsigned)((a.rows + RP - 1) / RP));
    cfg.blockDim = dim3(kFoldThreads);
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, decode_shared_fold_kernel<D>, a, part_of<KS>(s, ss), part_of<KO>(o, so),
                              (int)p.n_groups);
  });
}

}  // namespace gb300
