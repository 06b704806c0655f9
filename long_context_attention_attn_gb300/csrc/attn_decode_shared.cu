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
// keys by reading them.  us (attn_decode's in brackets), Hkv 8, d 128, 60 to 200 own tokens: 64
// sequences behind 8192, Hq 32, 45 (112); 64 behind 16384 56 (209); 128 behind 32768, Hq 128,
// 320 (1024).  d 256, Hkv 8, Hq 64: 32 sequences behind 16384 77 (199).
#include "attn_decode_kernels.cuh"

namespace gb300 {

namespace {

#include "attn_decode_group.cuh"

// What one list's kernel leaves.
struct Part {
  const float* part_o;    // pieces of items that several CTAs took: slots of part_rows rows
  const float* part_lse;
  const float* whole_o;   // [copies][n, s_q, h_q, D]: rows of items that one CTA took
  const float* whole_lse; // [copies][n, h_q, s_q]
  int64_t copy_floats;    // between copies
  int block, item_cost, shortest, tile, part_rows, copies, runs, row_tiles;
};

// Where a row's partials lie.
struct RowPieces {
  int64_t c0, s0, run;  // first CTA's run, first block of the item
  int n, rt, in_tile;   // partials (copies of pieces), row tile, row in the tile
};

template <int M>
__device__ __forceinline__ RowPieces pieces_of(const Part& l, int64_t run, const Entry& e, int64_t entry_at, int kvh,
                                               int row) {
  RowPieces p;
  p.rt = row / l.tile;
  p.in_tile = row - p.rt * l.tile;
  const int64_t item = M == kShared ? (int64_t)kvh * e.tiles + p.rt : kvh;
  p.s0 = entry_at + item * e.span.weight + l.item_cost;
  p.run = run;
  p.c0 = p.s0 / run;
  p.n = e.span.count ? ((int)((p.s0 + e.span.count - 1) / run - p.c0) + 1) * l.copies : 0;
  if (M == kShared) p.rt = 0;  // (a CTA's run has all of its tiles)
  return p;
}

constexpr int kFoldMost = 64;  // partials at a time

// The rows of a sequence and kv head over blockIdx.y, a thread per four values; where a CTA
// has fewer rows than its threads hold, several threads share a row's partials.
template <int D>
__global__ void __launch_bounds__(kFoldThreads)
    decode_shared_fold_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ Part shared,
                              const __grid_constant__ Part own, int n_groups, int heads) {
  constexpr int kVec = D / 4, RP = kFoldThreads / kVec;
  __shared__ int64_t before_s[kThreads + 1], before_o[kThreads + 1];
  __shared__ RowPieces rows_s[RP], rows_o[RP];
  __shared__ const float* s_src[kFoldMost][RP];
  __shared__ float s_w[kFoldMost][RP];
  __shared__ float s_ref[RP], s_old[RP];
  __shared__ float4 s_acc[kFoldThreads];
  __shared__ float s_z[kFoldThreads / kVec];
  __shared__ int s_most;
  DecodeArgs as = a, ao = a;
  as.n = n_groups;
  as.runs = shared.runs;
  ao.runs = own.runs;
  const Placement ps = place<kShared>(as, before_s, shared.block, shared.item_cost, shared.tile);
  const Placement po = place<kOwn>(ao, before_o, own.block, own.item_cost, own.tile);
  const int parts = (a.h_kv + heads - 1) / heads;
  const int seq = blockIdx.x / parts, r0 = blockIdx.y * RP;
  const int kvh0 = blockIdx.x % parts * heads, kvh1 = min(kvh0 + heads, a.h_kv);
  const int rows = min(RP, a.rows - r0);
  // the sequence's group (the last one that starts at or before it), and where the lists have them
  __shared__ Entry s_eg, s_eo;
  __shared__ int64_t s_at[2];
  if (threadIdx.x == 0) {
    int g = 0, end = n_groups;
    while (end - g > 1) {
      const int mid = (g + end) / 2;
      if (group_bound(a, mid) <= seq)
        g = mid;
      else
        end = mid;
    }
    int64_t at = before_s[g / ps.per];
    for (int i = g / ps.per * ps.per; i < g; ++i) {
      const Entry e = entry_of<kShared>(as, i, shared.block, shared.item_cost, shared.tile);
      at += (int64_t)e.span.weight * e.tiles;
    }
    s_at[0] = at * a.h_kv;
    s_eg = entry_of<kShared>(as, g, shared.block, shared.item_cost, shared.tile);
  }
  if (threadIdx.x == 32) {
    int64_t at = before_o[seq / po.per];
    for (int i = seq / po.per * po.per; i < seq; ++i)
      at += entry_of<kOwn>(ao, i, own.block, own.item_cost, own.tile).span.weight;
    s_at[1] = at * a.h_kv;
    s_eo = entry_of<kOwn>(ao, seq, own.block, own.item_cost, own.tile);
  }
  const int64_t run_s = run_length(as, before_s[kThreads] * a.h_kv, shared.shortest);
  const int64_t run_o = run_length(ao, before_o[kThreads] * a.h_kv, own.shortest);
  const int len = max(a.lens[seq], 0);
  bool waited = false;
  for (int kvh = kvh0; kvh < kvh1; ++kvh) {
    __syncthreads();  // (the last head's partials have been read)
    if (threadIdx.x == 0) s_most = 0;
    __syncthreads();
    if (threadIdx.x < rows) {
      const int row = r0 + threadIdx.x, in_group = seq - s_eg.first;
      RowPieces s;
      s.n = 0;
      if (in_group >= 0 && (in_group + 1) * a.rows <= s_eg.rows && len - a.s_q + row / a.g >= 0)
        s = pieces_of<kShared>(shared, run_s, s_eg, s_at[0], kvh, in_group * a.rows + row);
      const RowPieces o = pieces_of<kOwn>(own, run_o, s_eo, s_at[1], kvh, row);
      rows_s[threadIdx.x] = s;
      rows_o[threadIdx.x] = o;
      atomicMax(&s_most, s.n + o.n);
      s_ref[threadIdx.x] = -INFINITY;
    }
    __syncthreads();
    const int most = s_most;
    // everything the two grids before this one wrote
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
    waited = true;

    // Partial i of the CTA's row r: its values; its lse.
    auto source = [&](int r, int i, const float*& lse) -> const float* {
      const bool sh = i < rows_s[r].n;
      const RowPieces& p = sh ? rows_s[r] : rows_o[r];
      const Part& l = sh ? shared : own;
      const int j = sh ? i : i - rows_s[r].n;
      const int piece = j / l.copies, copy = j - piece * l.copies;
      if (p.n == l.copies) {
        const int row = r0 + r, tok = row / a.g, head = kvh * a.g + row % a.g;
        lse = l.whole_lse + copy * l.copy_floats + ((int64_t)seq * a.h_q + head) * a.s_q + tok;
        return l.whole_o + copy * l.copy_floats + (((int64_t)seq * a.s_q + tok) * a.h_q + head) * D;
      }
      // a piece that starts inside its item is the first of its CTA, one that ends inside it the last
      const int64_t slot = 2 * ((p.c0 + piece) * l.row_tiles + p.rt) + ((p.c0 + piece) * p.run <= p.s0 ? 1 : 0);
      const int64_t at = slot * l.part_rows + copy * l.tile + p.in_tile;
      lse = l.part_lse + at;
      return l.part_o + at * D;
    };
    const int q = threadIdx.x / kVec, d4 = threadIdx.x % kVec;
    int held = 1;  // rows, as a power of two
    while (held < rows) held *= 2;
    const int ways = RP / held, r = q & (held - 1), way = q / held;
    const bool mine = r < rows;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float z = 0.f;
    for (int b0 = 0; b0 < most; b0 += kFoldMost) {
      const int np = min(kFoldMost, most - b0);
      for (int u = threadIdx.x; u < np * held; u += kFoldThreads) {
        const int i = u / held, row = u & (held - 1);
        float w = -INFINITY;
        const float* src = nullptr;
        if (row < rows && b0 + i < rows_s[row].n + rows_o[row].n) {
          const float* lse;
          src = source(row, b0 + i, lse);
          w = *lse;
        }
        s_w[i][row] = w;
        s_src[i][row] = src;
      }
      __syncthreads();
      if (threadIdx.x < rows) {
        float top = s_ref[threadIdx.x];
        for (int i = 0; i < np; ++i) top = fmaxf(top, s_w[i][threadIdx.x]);
        s_old[threadIdx.x] = top == -INFINITY ? 0.f : ex2(s_ref[threadIdx.x] - top);
        s_ref[threadIdx.x] = top;
      }
      __syncthreads();
      if (mine) {
        const float top = s_ref[r], ref = top == -INFINITY ? 0.f : top, old = s_old[r];
        z *= old;
        acc.x *= old;
        acc.y *= old;
        acc.z *= old;
        acc.w *= old;
        const int here = min(np, rows_s[r].n + rows_o[r].n - b0);
#pragma unroll 4
        for (int i = way; i < here; i += ways) {
          const float f = ex2(s_w[i][r] - ref);
          const float4 v = reinterpret_cast<const float4*>(s_src[i][r])[d4];
          z += f;
          acc.x += v.x * f;
          acc.y += v.y * f;
          acc.z += v.z * f;
          acc.w += v.w * f;
        }
      }
      __syncthreads();
    }
    if (ways > 1) {
      s_acc[threadIdx.x] = acc;
      if (d4 == 0) s_z[q] = z;
      __syncthreads();
      if (way > 0) continue;
      for (int w = 1; w < ways; ++w) {
        const float4 v = s_acc[(w * held + r) * kVec + d4];
        z += s_z[w * held + r];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
    }
    if (!mine) continue;
    const int row = r0 + r;
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
}

// From more rows than this on a group's keys take attn_decode_group.cuh.
template <int D>
constexpr int kGroupRows = D == 64 ? 32 : 64;

// f(kernel of the shared keys, its shape, kernel of the own keys, its shape)
template <int D, typename F>
cudaError_t with_both(const attn_decode_shared_params& p, F&& f) {
  const attn_decode_params& q = p.base;
  const int64_t rows = q.s_q * (q.h_q / q.cache.h_kv), most = p.max_group * rows;
  auto with_own = [&](auto ks, const Shape& ss) {
    return with_rows<D, kOwn>(q, 0, rows, [&](auto ko, const Shape& so) { return f(ks, ss, ko, so); });
  };
  if constexpr (D < 256) {
    // (us of the whole call, Hkv 8, 60 to 200 own tokens, by attn_decode_tensor.cuh / attn_decode_group.cuh:
    // d 64, 32768 keys, 40 rows 38.2 / 37.0, 64 rows 39.4 / 38.4, 96 rows 47.8 / 39.8, 128 rows 49.0 / 40.5;
    // d 128, 32768 keys, 40 rows 41.6 / 46.1, 64 rows 45.3 / 47.6, 80 rows 58.2 / 49.9, 128 rows 58.8 / 54.1;
    // 8192 keys, 40 rows 27.9 / 30.0, 64 rows 31.2 / 31.4, 96 rows 36.5 / 34.3, 128 rows 38.5 / 37.8)
    if (most > kGroupRows<D>) {
      auto use = [&](auto k) {
        Shape sh;
        const cudaError_t e = k.shape(q, p.n_groups, &sh);
        return e == cudaSuccess ? with_own(k, sh) : e;
      };
      return most > 128 ? use(GroupKernel<D, false>()) : use(GroupKernel<D, true>());
    }
  }
  return with_rows<D, kShared>(q, p.n_groups, most, with_own);
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
  return align_up(2 * (size_t)sh.runs * sh.row_tiles * K::kPartRows * (d + 1), 64);
}
size_t row_floats(const attn_decode_params& p) { return align_up((size_t)p.n * p.s_q * p.h_q * (p.cache.d + 1), 64); }

template <typename K>
Part part_of(const DecodeArgs& a, const Shape& sh) {
  return Part{a.part_o,        a.part_lse,       static_cast<const float*>(a.out),
              a.lse,           a.copy_floats,    K::T::kBlock,
              K::T::kItemCost, K::T::kMinRun,    K::C::R,
              K::kPartRows,    K::kCopies,       sh.runs,
              sh.row_tiles};
}

}  // namespace

// Whether attn_decode does it better: no group has two members, or the problem is so
// small (by the page table's width) that it takes a cluster of CTAs per item, one launch in
// place of three that wait for one another (and uses no scratch).  us of attn_decode and of
// the three, Hq 32, Hkv 8, d 128, own tokens 60 to 200, by clusters: 4 sequences behind 2048
// tokens 8.8 / 15.4, behind 8192 14.8 / 16.7; 16 behind 2048 14.8 / 25.6; by the list: 8 behind
// 8192 23.4 / 22.1, behind 16384 35.3 / 26.1; 32 behind 4096 37.7 / 32.0.
static cudaError_t plain_is_better(const attn_decode_shared_params& p, bool* plain, size_t* bytes) {
  const cudaError_t e = decode_workspace(p.base, bytes);
  *plain = p.max_group <= 1 || *bytes == 0;
  return e;
}

cudaError_t decode_shared_workspace(const attn_decode_shared_params& p, size_t* bytes) {
  bool plain = false;
  const cudaError_t e = plain_is_better(p, &plain, bytes);
  if (e != cudaSuccess || plain) return e;
  return dispatch(p, [&](auto ks, const Shape& ss, auto ko, const Shape& so) {
    using KS = decltype(ks);
    *bytes = 4 * (part_floats<decltype(ks)>(ss, p.base.cache.d) + part_floats<decltype(ko)>(so, p.base.cache.d) +
                  (KS::kCopies + 1) * row_floats(p.base));
    return cudaSuccess;
  });
}

cudaError_t launch_attn_decode_shared(const attn_decode_shared_params& p, bool withhold, cudaStream_t st) {
  const attn_decode_params& q = p.base;
  bool plain = false;
  size_t bytes = 0;
  const cudaError_t e = plain_is_better(p, &plain, &bytes);
  if (e != cudaSuccess) return e;
  if (plain) return launch_attn_decode(q, withhold, st);
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
    s.copy_floats = (int64_t)row_floats(q);
    rows += KS::kCopies * row_floats(q);
    o.out = rows;
    o.lse = rows + row_values;
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
    // kv heads of a CTA: as many as leave work for every SM several times over (where lists lie is
    // looked up once for them)
    const int64_t blocks = (a.rows + RP - 1) / RP;
    int64_t heads = q.n * q.cache.h_kv * blocks / ((int64_t)sm_count() * 3);
    heads = heads < 1 ? 1 : heads > q.cache.h_kv ? q.cache.h_kv : heads;
    cfg.gridDim = dim3((unsigned)(q.n * ((q.cache.h_kv + heads - 1) / heads)), (unsigned)blocks);
    cfg.blockDim = dim3(kFoldThreads);
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, decode_shared_fold_kernel<D>, a, part_of<KS>(s, ss), part_of<KO>(o, so),
                              (int)p.n_groups, (int)heads);
  });
}

}  // namespace gb300
