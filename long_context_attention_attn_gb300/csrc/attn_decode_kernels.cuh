// Attention of a few query tokens per sequence over the paged 8-bit cache.
//
//   O = softmax(scale * q K^T + M) V,  K = codes * k_scale, V = codes * v_scale
//
// Bound by reading the cache once (2 * d bytes per key and kv head); the GQA
// group's query heads and the query tokens share each key read as the rows of
// one small matrix product.
//
// An item is a sequence, a kv head and a tile of its rows.  Small problems give
// each item a cluster of CTAs that fold their results through shared memory, in
// one launch.  Others are cut by keys, not by sequence: the blocks of 32 (16)
// keys of all items form one list, and every CTA of a grid that fills the GPU
// once takes an equal run of it, so ragged batches and single long sequences
// load every SM alike.  A run that ends inside an item leaves a finished
// partial (O, lse) in the workspace, and the combine kernel folds an item's
// partials in their order (the result does not depend on timing).
//
// A CTA's four warps take the blocks of a piece in turn, each with a ring of
// its own in shared memory, filled by 16-byte asynchronous copies, so that no
// warp waits for another before the piece's end.  Both products run with the
// keys on the matrix unit's M side:
//   S^T[keys, rows] = K q^T,  O^T[d, rows] += V^T P^T   (m16n8k16, f16 in, fp32
// sums), so a group of 8 rows is one N tile and the 8-bit codes are widened to
// f16 (exactly) once for all rows.  q enters as f16 after a power-of-two scale
// of its row (all of its 8 bits down to 2^-31 of the row's largest value; below
// that off by 2^-39 of it at most), P as f16 relative to a running maximum (11
// bits).
// The sums over d and over keys do not care for order, so a thread takes its
// d's as 16 neighbouring bytes of a key (K) or of four keys (V) and byte
// permutes pair the keys: no transposing loads.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <type_traits>

#include "attn_decode.h"
#include "internal.h"
#include "ptx.cuh"

namespace gb300 {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLn2 = 0.69314718055994530942f;
// The running maximum is raised only when a value exceeds it by more than this
// (in powers of two), so P <= 256.
constexpr float kRescale = 8.f;
// P * v_scale is held 2^7 times larger (<= 2^15, f16 ends at 2^16): it keeps its 11
// bits down to 2^-21 of the largest, where one key has nearly all the weight and a
// zero code others decide the sum; below that it is off by 2^-32 of the largest.
constexpr float kShift = 7.f;

// What a list of keys holds: a sequence's whole context; what a sequence does not share
// with others; or what a group of sequences shares, whose rows are then those of all
// its members (attn_decode_shared).
enum { kWhole, kOwn, kShared };

struct DecodeArgs {
  const __nv_bfloat16* q;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  const int* table;
  const int* lens;
  void* out;
  float* lse;
  float* part_o;    // [2 * runs * row_tiles, R, D]
  float* part_lse;  // [2 * runs * row_tiles, R] (base 2)
  int64_t page_stride;
  int n, s_q, h_q, h_kv, g, rows, row_tiles, max_pages, page_shift, num_pages;
  int window, sink, out_fp32;
  int withhold;  // debug hook: copy nothing, so that every wait runs out (tensor memory only)
  int runs;     // of the list; row_tiles CTAs take each
  int cluster;  // CTAs per item (0: by the list)
  float scale_log2;
  // kOwn, kShared: pages that each sequence shares, and the groups (n of them: kShared)
  const int* shared_pages;
  const int* group_start;
  int n_seq;
  int64_t copy_floats;  // between out (and lse) of a row's partials (attn_decode_group.cuh)
};

// How a kernel is cut.  A block of K and V is 8 KB (4 KB at d = 64): 32 keys, 16
// at d = 256, whose accumulators leave no registers for two groups of 16.  Two
// or three ring slots a warp keep 64 to 190 KB of copies in flight on an SM;
// what counts more are warps to issue from, so the q fragments move to shared
// memory where that makes room for another CTA.  On GB300 (64 sequences of 200
// to 16384 tokens, Hkv 8, d 128): two CTAs per SM and three slots 179 us,
// three CTAs and two slots 173 us (1.09 GB).
template <int D, int NT>
struct Tune {
  // Shortest run: a shorter one would only add partials to fold.
  static constexpr int kMinRun = 16;
  static constexpr bool kTensor = false;
  static constexpr int kBlock = D == 256 ? 16 : 32;
  static constexpr int kStages = (D == 128 && NT <= 2) || (D == 256 && NT == 1) ? 2 : 3;
  static constexpr int kCtas = D == 64 ? (NT == 1 ? 4 : NT == 2 ? 3 : 2) : D * NT <= 256 ? 3 : 2;
  static constexpr bool kQRegs = D * NT <= 128 || D == 64;
  // What the start and the end of an item (q, the first copies' latency, the
  // fold of the warps) cost, in blocks: the runs are cut by blocks plus this.
  // Without it the CTAs with many short sequences end last: 243 us for the
  // batch above, 197 us with 16.
  static constexpr int kItemCost = D * NT >= 512 ? 32 : 16;
  // Most blocks per warp for which an item gets a cluster of its own (up to 8
  // CTAs, all items at once on the GPU, by the longest sequence that the page
  // table can hold).  That saves the list, the scratch and the second launch;
  // the list balances unlike lengths and uses the SMs that clusters leave.  One
  // sequence, Hkv 8 d 128, us by list / by cluster: Hq 32 at 512 tokens 8.7 /
  // 6.3, 4096 11.5 / 8.9, 16384 19.6 / 18.5, 32768 29.3 / 31.5; Hq 128 at 4096
  // 15.1 / 12.8, 8192 16.8 / 16.4, 16384 23.2 / 25.2.
  static constexpr int kClusterBlocks = (NT == 1 ? 16 : NT == 2 ? 8 : 0) * (D == 64 ? 2 : 1);
};
// The kernel of 64 or 128 rows per CTA (attn_decode_tensor.cuh), one CTA per SM.
template <int D>
struct TensorTune {
  static constexpr int kMinRun = 16;
  static constexpr bool kTensor = true;
  static constexpr int kBlock = 32;
  static constexpr int kStages = D == 64 ? 8 : 3;  // tiles of codes: of 128 keys (64 at d = 256)
  // (us of 48 sequences of 100 to 12000 tokens with 32 / 64: d 64 252 / 241, d 128
  // 326 / 313; d 256 with 16 / 32: 563 / 572)
  static constexpr int kItemCost = D == 256 ? 16 : 64;
  static constexpr int kClusterBlocks = 0;
};
template <int D>
struct Tune<D, 8> : TensorTune<D> {};
template <int D>
struct Tune<D, 16> : TensorTune<D> {};
// Most blocks per warp for which a CTA takes an item alone, however many items
// there are (twice that where all fit on the GPU at once): 64 sequences of up to
// 512 tokens (Hq 32 Hkv 8 d 128) 17.3 us by the list, 15.6 us so; of up to 2048
// 31.8 and 32.9.
constexpr int kAloneBlocks = 4;
constexpr int kMaxCluster = 8;  // CTAs per item, at most (a size every GPU takes)

// The blocks of keys that some query of a sequence of length `len` may see:
// first those of the kept tokens, then those from the window's start on.
struct Span {
  int hi;        // keys below this exist
  int lo;        // first key of the window of the first query
  int sink_hi;   // kept keys
  int nb_sink;   // blocks taken before the window's first
  int first;     // the window's first block
  int count;     // blocks
  int weight;    // what the item counts in the list: blocks and the cost of its start and end
  __device__ __forceinline__ int block(int t) const { return t < nb_sink ? t : first + t - nb_sink; }
};

// p0: the first query's position (0 where it is negative); cap: keys that the page
// table can hold.
__device__ __forceinline__ Span make_span(int len, int cap, int p0, int window, int sink, int block, int item_cost) {
  Span s;
  s.hi = min(max(len, 0), cap);
  s.lo = window < 0 ? 0 : max(p0 - window, 0);
  s.sink_hi = window < 0 ? 0 : min(sink, s.hi);
  const int last = (s.hi + block - 1) / block;
  s.first = min(s.lo / block, last);
  s.nb_sink = min((s.sink_hi + block - 1) / block, s.first);
  s.count = s.nb_sink + last - s.first;
  s.weight = s.count ? s.count + item_cost : 0;
  return s;
}

// An entry of the list: a sequence, or a group of them.
struct Entry {
  int len;    // kWhole, kOwn: the sequence's tokens (kOwn: behind the shared ones, whose count may exceed them)
  int skip;   // kOwn: shared pages, before the first key here
  int sink;   // kept tokens, from the first key here on
  int first;  // kShared: the first sequence
  int rows;   // rows of a kv head
  int tiles;  // kShared: row tiles, each an item of its own
  Span span;
};

__device__ __forceinline__ int pages_shared(const DecodeArgs& a, int seq) {
  return min(max(a.shared_pages[seq], 0), a.max_pages);
}

// (no array: one group of all sequences)
__device__ __forceinline__ int group_bound(const DecodeArgs& a, int i) {
  return a.group_start ? min(max(a.group_start[i], 0), a.n_seq) : i ? a.n_seq : 0;
}

// (block, item_cost, tile: of the kernel that goes through the list)
template <int M>
__device__ __forceinline__ Entry entry_of(const DecodeArgs& a, int i, int block, int item_cost, int tile) {
  Entry e;
  e.first = e.skip = 0;
  e.sink = a.sink;
  e.rows = a.rows;
  e.tiles = 1;
  if constexpr (M == kShared) {
    e.first = group_bound(a, i);
    const int members = max(group_bound(a, i + 1) - e.first, 0);
    e.rows = members * a.s_q * a.g;
    e.tiles = (e.rows + tile - 1) / tile;
    e.len = members ? pages_shared(a, e.first) << a.page_shift : 0;
    int p0 = 0;
    if (a.window >= 0 && e.len > 0) {  // the first position of any that sees a key
      p0 = 0x7fffffff;
#pragma unroll 8
      for (int m = 0; m < members; ++m) {
        const int len = a.lens[e.first + m];
        if (len > 0) p0 = min(p0, max(len - a.s_q, 0));
      }
    }
    e.span = make_span(e.len, a.max_pages << a.page_shift, p0, a.window, a.sink, block, item_cost);
  } else {
    e.len = a.lens[i];
    int cap = a.max_pages << a.page_shift;
    if constexpr (M == kOwn) {
      e.skip = pages_shared(a, i);
      const int tokens = e.skip << a.page_shift;
      e.len = max(e.len, 0) - tokens;
      e.sink = max(e.sink - tokens, 0);
      cap -= tokens;
    }
    e.span = make_span(e.len, cap, max(e.len - a.s_q, 0), a.window, e.sink, block, item_cost);
  }
  return e;
}
template <typename T, int M, int R>
__device__ __forceinline__ Entry entry_of(const DecodeArgs& a, int i) {
  return entry_of<M>(a, i, T::kBlock, T::kItemCost, R);
}

// Where the list of all blocks puts each sequence: thread t of the CTA sums
// the blocks of `per` neighbouring sequences; `before` is the sum ahead of
// them (shared memory, one entry per thread, then the total).
struct Placement {
  const int64_t* before;
  int per;
};

template <int M>
__device__ __forceinline__ Placement place(const DecodeArgs& a, int64_t* before, int block, int item_cost, int tile) {
  __shared__ int64_t warp_sum[kWarps];
  const int t = threadIdx.x, lane = t & 31, wid = t >> 5;
  const int per = (a.n + kThreads - 1) / kThreads;
  const bool mine = t < kThreads;  // (the combine kernel has more)
  int64_t sum = 0;
  for (int i = mine ? t * per : a.n; i < min((t + 1) * per, a.n); ++i) {
    const Entry e = entry_of<M>(a, i, block, item_cost, tile);
    sum += (int64_t)e.span.weight * e.tiles;
  }
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (mine && lane == 31) warp_sum[wid] = incl;
  __syncthreads();
  int64_t base = 0;
  for (int w = 0; w < min(wid, kWarps); ++w) base += warp_sum[w];
  if (mine) before[t] = base + incl - sum;
  if (t == kThreads - 1) before[kThreads] = base + incl;
  __syncthreads();
  return Placement{before, per};
}
template <typename T, int M, int R>
__device__ __forceinline__ Placement place(const DecodeArgs& a, int64_t* before) {
  return place<M>(a, before, T::kBlock, T::kItemCost, R);
}

// Weight per CTA: an equal share of the list, and no less than the shortest.
__device__ __forceinline__ int64_t run_length(const DecodeArgs& a, int64_t total, int shortest) {
  return max((total + a.runs - 1) / a.runs, (int64_t)shortest);
}

// ---------------------------------------------------------------- primitives
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(take ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(take ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// f16 pair of the two e4m3 codes in the low / high half of a word (exact)
__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Hardware base-2 logarithm (exact for powers of two, subnormal ones too); of 0 -inf.
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Transposes the 8 x 8 f16 matrix that the warp holds one row per four lanes.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Clusters: a barrier of all threads, and loads from another CTA's shared memory.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_address(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float load_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 load_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Key of matrix row r (0..7) inside its group of 8: rows 2i and 2i + 1 are keys
// i and i + 4, whose shared-memory chunks sit in different bank halves.
__device__ __forceinline__ int key_of_row(int r) { return (r >> 1) | ((r & 1) << 2); }

// Byte offset of 16-byte chunk c of key row `key` inside a block's K or V tile.
// D = 128: the chunk index is XORed with the row.  D = 256: the same within
// each 128-byte half.  D = 64: two rows share 128 bytes; the row's half and the
// 32-byte part are chosen so that both the K reads (four chunks of keys i and
// i + 4) and the V reads (one 8-byte piece of four keys i, i + 1, ..) meet all
// banks once.
template <int D>
__device__ __forceinline__ int tile_offset(int key, int c) {
  if constexpr (D == 64)
    return (key >> 1) * 128 + (((key ^ (key >> 2)) & 1) << 6) + ((c ^ (key & 2)) << 4);
  else
    return key * D + ((c & 8) << 4) + (((c ^ key) & 7) << 4);
}

// 0xff in the bytes of w that are the e4m3 NaN (0x7f or 0xff)
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((((w & 0x7f7f7f7fu) + 0x01010101u) >> 7) & 0x01010101u) * 0xffu;
}

// O^T += V^T P^T over one block: o[i][nt] are the d's of thread n8 (16 (or 8)
// neighbouring ones, two per i) against rows 8 nt + 2 t4 + {0, 1}.  kNoNan
// takes zeros for NaN codes; kOnlyNan turns o to NaN where a NaN code meets a
// key whose value in pb (0 or 1) says that the row sees it.
enum { kPlain, kNoNan, kOnlyNan };
template <int D, int NT, int MT, int kMode>
__device__ __forceinline__ void add_pv(float (&o)[D / 16][NT][4], const uint8_t* vt,
                                       const uint32_t (&pb)[MT][NT][2], int n8, int t4) {
  constexpr int kParts = D == 256 ? 2 : 1;  // 16-byte pieces of a key per thread
  constexpr int kWords = D == 64 ? 2 : 4;   // words per piece
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int hh = 0; hh < kParts; ++hh) {
      uint32_t w[4][kWords];  // keys t4, t4 + 4, t4 + 8, t4 + 12 of the group
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int key = mt * 16 + t4 + 4 * y;
        if constexpr (D == 64) {
          const uint2 x = *reinterpret_cast<const uint2*>(vt + tile_offset<D>(key, n8 >> 1) + (n8 & 1) * 8);
          w[y][0] = x.x;
          w[y][1] = x.y;
        } else {
          const uint4 x = *reinterpret_cast<const uint4*>(vt + tile_offset<D>(key, key_of_row(n8) + 8 * hh));
          w[y][0] = x.x;
          w[y][1] = x.y;
          w[y][2] = x.z;
          w[y][3] = x.w;
        }
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          if constexpr (kMode == kNoNan) w[y][j] &= ~nan_bytes(w[y][j]);
          if constexpr (kMode == kOnlyNan) w[y][j] = nan_bytes(w[y][j]) & 0x38383838u;  // e4m3 1.0
        }
      }
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        const uint32_t ab0 = __byte_perm(w[0][j], w[1][j], 0x5140), ab1 = __byte_perm(w[0][j], w[1][j], 0x7362);
        const uint32_t cd0 = __byte_perm(w[2][j], w[3][j], 0x5140), cd1 = __byte_perm(w[2][j], w[3][j], 0x7362);
        const uint32_t f0[4] = {widen_lo(ab0), widen_hi(ab0), widen_lo(cd0), widen_hi(cd0)};
        const uint32_t f1[4] = {widen_lo(ab1), widen_hi(ab1), widen_lo(cd1), widen_hi(cd1)};
        const int i = (hh * kWords + j) * 2;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (kMode == kOnlyNan) {
            float n0[4] = {0.f, 0.f, 0.f, 0.f}, n1[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816(n0, f0, pb[mt][nt][0], pb[mt][nt][1]);
            mma16816(n1, f1, pb[mt][nt][0], pb[mt][nt][1]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (n0[c] != 0.f) o[i][nt][c] = __int_as_float(0x7fffffff);
              if (n1[c] != 0.f) o[i + 1][nt][c] = __int_as_float(0x7fffffff);
            }
          } else {
            mma16816(o[i][nt], f0, pb[mt][nt][0], pb[mt][nt][1]);
            mma16816(o[i + 1][nt], f1, pb[mt][nt][0], pb[mt][nt][1]);
          }
        }
      }
    }
  }
}

// Whether a block's V tile holds the e4m3 NaN (0x7f or 0xff) anywhere.
template <int D, int kBlock>
__device__ __forceinline__ bool holds_nan(const uint8_t* vt, int lane) {
  bool nan = false;
#pragma unroll 2
  for (int u = lane; u < kBlock * D / 16; u += 32) {
    const uint4 x = reinterpret_cast<const uint4*>(vt)[u];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) nan |= nan_bytes(w[j]) != 0u;
  }
  return __any_sync(0xffffffffu, nan);
}

// Where the 512 bytes number u of a tile go, from the place of the lane's 16 in
// the first 512 (tile_offset of row lane / (D / 16)): the following rows only
// turn the XORed chunk bits.
template <int D>
__device__ __forceinline__ uint32_t copy_offset(uint32_t lane_off, int u) {
  const uint32_t turn = D == 64 ? 0 : D == 128 ? (u & 1) * 64 : (u & 3) * 32;
  return (lane_off ^ turn) + u * 512;
}

template <int D, int NT>
struct Cfg {
  static constexpr int R = NT * 8;                  // rows per tile
  static constexpr int kBlock = Tune<D, NT>::kBlock;
  static constexpr int kTile = kBlock * D;          // bytes of a K or V tile
  static constexpr int kStage = 2 * kTile;
  static constexpr int kStages = Tune<D, NT>::kStages;
  static constexpr int kKSteps = D / 16;
  static constexpr bool kQRegs = Tune<D, NT>::kQRegs;  // q fragments in registers
  static constexpr int q_off = kWarps * kStages * kStage;          // uint4 [NT * kKSteps / 2][32]
  static constexpr int meta_off = q_off + NT * kKSteps / 2 * 512;  // per warp and stage: 8 words
  static constexpr int row_off = meta_off + kWarps * kStages * 32; // row factors, positions
  static constexpr int bytes = row_off + 2 * R * 4;
  // the ring's room holds the four warps' results at the end of a piece
  static constexpr int kMergeRow = D + 4;
  // behind them, with a cluster per item, the CTA's own: [R][D], then [R]
  static constexpr int fin_off = kWarps * R * (kMergeRow + 3) * 4;
  static_assert(fin_off % 16 == 0 && fin_off + R * (D + 1) * 4 <= q_off, "merge buffer");
};

// One piece of work: blocks [t0, t1) of an item.
template <int M>
struct Piece {
  int seq, kvh, rt, t0, t1;
  Span span;
  int len;
  __device__ __forceinline__ void take(const Entry& e) {
    span = e.span;
    len = e.len;
  }
  __device__ __forceinline__ int rows(const DecodeArgs& a) const { return a.rows; }
  __device__ __forceinline__ int sink(const DecodeArgs& a) const { return a.sink; }
  // the page table's entry of the first key
  __device__ __forceinline__ const int* table(const DecodeArgs& a) const { return a.table + (int64_t)seq * a.max_pages; }
};
template <>
struct Piece<kOwn> : Piece<kWhole> {
  int sink_, skip;
  __device__ __forceinline__ void take(const Entry& e) {
    Piece<kWhole>::take(e);
    sink_ = e.sink;
    skip = e.skip;
  }
  __device__ __forceinline__ int sink(const DecodeArgs&) const { return sink_; }
  __device__ __forceinline__ const int* table(const DecodeArgs& a) const { return Piece<kWhole>::table(a) + skip; }
};
template <>
struct Piece<kShared> : Piece<kWhole> {
  int first, rows_;  // (len is not used: every row has its own)
  __device__ __forceinline__ void take(const Entry& e) {
    Piece<kWhole>::take(e);
    first = e.first;
    rows_ = e.rows;
  }
  __device__ __forceinline__ int rows(const DecodeArgs&) const { return rows_; }
  __device__ __forceinline__ const int* table(const DecodeArgs& a) const { return a.table + (int64_t)first * a.max_pages; }
};

// Where row `row` of a piece lies: its token and head, the row of q and out, the place of
// its lse.
template <int M>
struct RowPlace {
  int tok, head;
  int64_t orow, lse;
  int pos;  // of the query, counted from the list's first key
  template <typename P>
  __device__ __forceinline__ RowPlace(const DecodeArgs& a, const P& p, int row) {
    tok = row / a.g;
    head = p.kvh * a.g + (row - tok * a.g);
    int seq = p.seq, t = tok;
    if constexpr (M == kShared) {
      seq = p.first + tok / a.s_q;
      t = tok % a.s_q;
      pos = max(a.lens[seq], 0) - a.s_q + t;
    } else {
      pos = p.len - a.s_q + t;
    }
    orow = ((int64_t)seq * a.s_q + t) * a.h_q + head;
    lse = ((int64_t)seq * a.h_q + head) * a.s_q + t;
  }
};
// The largest magnitudes of bf16 pairs: they order like their bits, two in a word.
__device__ __forceinline__ uint32_t top_bf16x2(uint32_t top, uint32_t w) { return __vmaxu2(top, w & 0x7fff7fffu); }
// As the bits of a float (0x7f800000 and above: an infinity or NaN is among them).
__device__ __forceinline__ uint32_t top_of(uint32_t top) { return max(top << 16, top & 0xffff0000u); }
// What the scores of a row are multiplied by, whose q was divided by 2^ex.  A row with an infinity or
// NaN has no softmax (minus infinity for every score would pass for a row that sees no key): all
// of it is NaN.
__device__ __forceinline__ float row_factor(const DecodeArgs& a, int ex, bool finite) {
  return finite ? a.scale_log2 * __uint_as_float((uint32_t)(127 + ex) << 23) : __int_as_float(0x7fffffff);
}

// (the parts of a shared problem are folded in base 2)
template <int M>
__device__ __forceinline__ float lse_out(float lse2) {
  return M == kWhole ? lse2 * kLn2 : lse2;
}

// CL: one cluster per item, its CTAs taking equal shares of the item's blocks
// and folding their results through each other's shared memory (no list, no
// scratch, no second launch); else each CTA takes a run of the list.
template <int D, int NT, bool CL, int M>
__global__ void __launch_bounds__(kThreads, Tune<D, NT>::kCtas) attn_decode_kernel(const DecodeArgs a) {
  using C = Cfg<D, NT>;
  using T = Tune<D, NT>;
  constexpr int kBlock = T::kBlock, kItemCost = T::kItemCost;
  constexpr int MT = kBlock / 16;  // groups of 16 keys
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int n8 = lane >> 2, t4 = lane & 3;

  int64_t at = 0, end = 1;  // the run of the list; with CL a single turn
  int seq;
  int64_t seq_at = 0;  // where the sequence starts in the list
  if constexpr (CL) {
    seq = (int)(blockIdx.x / a.cluster) / (a.h_kv * a.row_tiles);
  } else {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int64_t before[kThreads + 1];
    const Placement pl = place<T, M, C::R>(a, before);
    const int64_t total = before[kThreads] * a.h_kv;
    const int64_t run = run_length(a, total, T::kMinRun);
    at = blockIdx.x / a.row_tiles * run;
    end = min(at + run, total);
    if (at >= end) {
      if (M == kOwn && blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
      return;
    }
    // the sequence of the run's first block
    int t = 0;
#pragma unroll
    for (int step = kThreads / 2; step > 0; step >>= 1)
      if (before[t + step] * a.h_kv <= at) t += step;
    // (entries behind the last sequence repeat the total, which is above `at`)
    seq = t * pl.per;
    seq_at = before[t] * a.h_kv;
    for (; seq < a.n - 1; ++seq) {
      const Entry e = entry_of<T, M, C::R>(a, seq);
      const int64_t c = (int64_t)e.span.weight * e.tiles * a.h_kv;
      if (at < seq_at + c) break;
      seq_at += c;
    }
  }

  uint8_t* ring = smem + warp * C::kStages * C::kStage;
  uint32_t* meta = reinterpret_cast<uint32_t*>(smem + C::meta_off) + warp * C::kStages * 8;
  uint4* s_q = reinterpret_cast<uint4*>(smem + C::q_off);
  float* s_fac = reinterpret_cast<float*>(smem + C::row_off);
  int* s_pos = reinterpret_cast<int*>(s_fac + C::R);
  const uint32_t ring_u = smem_u32(ring), meta_u = smem_u32(meta);
  const uint32_t lane_off = tile_offset<D>(lane / (D / 16), lane % (D / 16));

  while (at < end && seq < a.n) {
    Piece<M> p;
    p.seq = seq;
    const Entry entry = entry_of<T, M, C::R>(a, seq);
    p.take(entry);
    bool item_done = true;
    if constexpr (CL) {
      const int item = (int)(blockIdx.x / a.cluster) % (a.h_kv * a.row_tiles), rank = blockIdx.x % a.cluster;
      p.kvh = item / a.row_tiles;
      p.rt = item % a.row_tiles;
      p.t0 = (int)((int64_t)p.span.count * rank / a.cluster);
      p.t1 = (int)((int64_t)p.span.count * (rank + 1) / a.cluster);
      at = end;
    } else {
      if (p.span.count == 0) {
        ++seq;
        continue;
      }
      // the piece [w0, w1) of the item's weight: its first kItemCost hold no block
      const int64_t in_seq = at - seq_at;
      const int weight = p.span.weight;
      const int item = (int)(in_seq / weight);
      p.kvh = item;
      p.rt = blockIdx.x % a.row_tiles;
      const int w0 = (int)(in_seq - (int64_t)item * weight);
      const int w1 = (int)min((int64_t)weight, w0 + (end - at));
      p.t0 = max(w0 - kItemCost, 0);
      p.t1 = max(w1 - kItemCost, 0);
      at += w1 - w0;
      item_done = w1 == weight;
      if (item_done && item == a.h_kv * entry.tiles - 1) {
        seq_at += (int64_t)weight * a.h_kv * entry.tiles;
        ++seq;
      }
      if constexpr (M == kShared) {
        p.kvh = item / entry.tiles;
        p.rt = item % entry.tiles;
      }
      if (p.t1 == p.t0) continue;
    }

    // ---- the rows of q: their loads are in flight while the ring fills
    constexpr int kE = D / 32;               // values of a row per lane, neighbours
    constexpr int kRows = C::R / kWarps;     // rows per warp
    uint32_t qw[kRows][kE / 2];
    bool qin[kRows];
    int qpos[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = p.rt * C::R + warp + i * kWarps;
      const bool in = row < p.rows(a);
      const RowPlace<M> at_row(a, p, in ? row : 0);
      const uint32_t* src = reinterpret_cast<const uint32_t*>(a.q + at_row.orow * D + lane * kE);
      qin[i] = in;
      qpos[i] = in ? at_row.pos : -1;
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) qw[i][e] = in ? src[e] : 0u;
    }

    // ---- the asynchronous copies of one block into a ring slot
    const int* table = p.table(a);
    const int page_mask = (1 << a.page_shift) - 1;
    auto fetch = [&](int t, int slot) {
      if (t < p.t1) {
        const int key0 = p.span.block(t) * kBlock;
        // the block's two groups of 16 keys lie on one page each
        int pid[MT];
        bool ok[MT];
        pid[0] = table[key0 >> a.page_shift];
        if constexpr (MT == 2) pid[1] = pid[0];
        if (MT == 2 && a.page_shift == 4) pid[MT - 1] = key0 + 16 < p.span.hi ? table[(key0 >> 4) + 1] : -1;
#pragma unroll
        for (int u = 0; u < MT; ++u) {
          ok[u] = pid[u] >= 0 && pid[u] < a.num_pages;
          if (!ok[u]) pid[u] = 0;
        }
        // a group's rows are neighbours in memory, 32 lanes take 512 bytes at a time
        const uint32_t dst = ring_u + slot * C::kStage;
        constexpr int kPer = kBlock * D / 512;
        const uint8_t *kp[MT], *vp[MT];
#pragma unroll
        for (int u = 0; u < MT; ++u) {
          const int64_t src = (int64_t)pid[u] * a.page_stride +
                              (((int64_t)p.kvh << a.page_shift) + ((key0 + 16 * u) & page_mask)) * D + lane * 16;
          kp[u] = a.k + src;
          vp[u] = a.v + src;
        }
        const bool whole = ok[0] && ok[MT - 1] && key0 + kBlock <= p.span.hi &&
                           (key0 >= p.span.lo || key0 + kBlock <= p.span.sink_hi);
        if (whole) {
#pragma unroll
          for (int u = 0; u < kPer; ++u) {
            const uint32_t off = copy_offset<D>(lane_off, u);
            cp_async16(dst + off, kp[MT * u / kPer] + (u % (kPer / MT)) * 512);
            cp_async16(dst + C::kTile + off, vp[MT * u / kPer] + (u % (kPer / MT)) * 512);
          }
        } else {
          // zeros for what no query sees
#pragma unroll
          for (int u = 0; u < kPer; ++u) {
            const int key = key0 + u * (512 / D) + lane / (D / 16);
            const bool take = ok[MT * u / kPer] && key < p.span.hi && (key >= p.span.lo || key < p.span.sink_hi);
            const uint32_t off = copy_offset<D>(lane_off, u);
            cp_async16_or_zero(dst + off, kp[MT * u / kPer] + (u % (kPer / MT)) * 512, take);
            cp_async16_or_zero(dst + C::kTile + off, vp[MT * u / kPer] + (u % (kPer / MT)) * 512, take);
          }
        }
        // K and V scales of the two groups, and whether they have a page
        if (lane < 4 && (lane & 1) < MT) {
          const bool second = MT == 2 && (lane & 1);
          const float* sc = (lane < 2 ? a.k_scale : a.v_scale) + (int64_t)pid[second ? MT - 1 : 0] * a.h_kv + p.kvh;
          cp_async4(meta_u + slot * 32 + lane * 4, sc, second ? ok[MT - 1] : ok[0]);
        }
        if (lane == 0) meta[slot * 8 + 4] = (ok[0] ? 1u : 0u) | (ok[MT - 1] ? 2u : 0u);
      }
      cp_async_commit();
    };
    int t_load = p.t0 + warp;
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) {
      fetch(t_load, s);
      t_load += kWarps;
    }

    // ---- q of the item's rows as f16 fragments, row factors and positions
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = warp + i * kWarps;
      float x[kE];
      uint32_t top = 0u;
#pragma unroll
      for (int e = 0; e < kE; e += 2) {
        x[e] = __uint_as_float(qw[i][e / 2] << 16);
        x[e + 1] = __uint_as_float(qw[i][e / 2] & 0xffff0000u);
        top = top_bf16x2(top, qw[i][e / 2]);
      }
      const uint32_t bits = __reduce_max_sync(0xffffffffu, top_of(top));
      const bool finite = bits < 0x7f800000u;
      // the row's largest value goes to [2^14, 2^15)
      const int ex = finite && bits ? max((int)(bits >> 23) - 127, -100) - 14 : 0;
      const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
      // value e of the lane's is element (d & 3) of k step (d >> 6) * 4 + ((d & 15) >> 2)
      // of lane (r & 7) * 4 + ((d >> 4) & 3), in pairs
      uint32_t* sq = reinterpret_cast<uint32_t*>(s_q);
#pragma unroll
      for (int e = 0; e < kE; e += 2) {
        const int d = lane * kE + e;
        const int ks = (d >> 6) * 4 + ((d & 15) >> 2);
        const int ln = (r & 7) * 4 + ((d >> 4) & 3);
        sq[((((r >> 3) * C::kKSteps + ks) >> 1) * 32 + ln) * 4 + (ks & 1) * 2 + ((d & 3) >> 1)] =
            pack_f16(x[e] * inv, x[e + 1] * inv);
      }
      if (lane == 0) {
        s_fac[r] = qin[i] ? row_factor(a, ex, finite) : 0.f;
        s_pos[r] = qpos[i];
      }
    }
    __syncthreads();
    uint4 qf[C::kQRegs ? NT * C::kKSteps / 2 : 1];
    if constexpr (C::kQRegs) {
#pragma unroll
      for (int i = 0; i < NT * C::kKSteps / 2; ++i) qf[i] = s_q[i * 32 + lane];
    }

    // ---- running state: thread (n8, t4) holds rows 8 nt + 2 t4 + {0, 1}
    float o[D / 16][NT][4];
    // the references of P and of P * v_scale (base 2, negated; at first below every
    // score), and the sum of P
    float nm[NT][2], nmo[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][nt][c] = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        nm[nt][c] = nmo[nt][c] = FLT_MAX;
        l[nt][c] = 0.f;
      }
    }
    int p_first = p.len - a.s_q, p_last = p.len - 1;  // query positions
    if constexpr (M == kShared) {
      p_first = 0x7fffffff;
      p_last = -1;
#pragma unroll
      for (int r = lane; r < C::R; r += 32) {
        if (s_pos[r] >= 0) {  // (rows at negative positions see nothing: the fold leaves them out)
          p_first = min(p_first, s_pos[r]);
          p_last = max(p_last, s_pos[r]);
        }
      }
      p_first = __reduce_min_sync(0xffffffffu, p_first);
      p_last = __reduce_max_sync(0xffffffffu, p_last);
    }

    int slot = 0;
    for (int t = p.t0 + warp; t < p.t1; t += kWarps) {
      cp_async_wait<C::kStages - 2>();
      __syncwarp();
      {
        const int next = slot == 0 ? C::kStages - 1 : slot - 1;  // the slot read last time
        fetch(t_load, next);
        t_load += kWarps;
      }
      const uint8_t* kt = ring + slot * C::kStage;
      const uint8_t* vt = kt + C::kTile;
      const uint32_t* mw = meta + slot * 8;
      const uint32_t pages_ok = mw[4];
      const int key0 = p.span.block(t) * kBlock;

      // S^T = K q^T
      float s[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[mt][nt][c] = 0.f;
#pragma unroll
      for (int cc = 0; cc < D / 64; ++cc) {
        uint32_t w[MT][2][4];  // [mt][key group of 8][4 words of 4 codes]
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint4 x = *reinterpret_cast<const uint4*>(
                kt + tile_offset<D>(mt * 16 + hf * 8 + key_of_row(n8), t4 + 4 * cc));
            w[mt][hf][0] = x.x;
            w[mt][hf][1] = x.y;
            w[mt][hf][2] = x.z;
            w[mt][hf][3] = x.w;
          }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t af[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            af[mt][0] = widen_lo(w[mt][0][j]);
            af[mt][1] = widen_lo(w[mt][1][j]);
            af[mt][2] = widen_hi(w[mt][0][j]);
            af[mt][3] = widen_hi(w[mt][1][j]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int ks = cc * 4 + j;
            const int qi = (nt * C::kKSteps + ks) >> 1;
            uint4 f;
            if constexpr (C::kQRegs)
              f = qf[qi];
            else
              f = s_q[qi * 32 + lane];
            const uint32_t b0 = (ks & 1) ? f.z : f.x, b1 = (ks & 1) ? f.w : f.y;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma16816(s[mt][nt], af[mt], b0, b1);
          }
        }
      }

      // scores in base 2; s[mt][nt][c]: key 16 mt + 8 (c >> 1) + key_of_row(n8),
      // row 8 nt + 2 t4 + (c & 1)
      float ks_[MT], lvs[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        ks_[mt] = __uint_as_float(mw[mt]);
        lvs[mt] = lg2(__uint_as_float(mw[2 + mt]));
      }
      const bool all_seen = pages_ok == 3u && key0 + kBlock - 1 <= p_first &&
                            (a.window < 0 || p_last - key0 <= a.window || key0 + kBlock - 1 < p.sink(a));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 row = *reinterpret_cast<const float2*>(s_fac + 8 * nt + 2 * t4);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float f0, f1;
          mul_f32x2(f0, f1, row.x, row.y, ks_[mt], ks_[mt]);
          mul_f32x2(s[mt][nt][0], s[mt][nt][1], s[mt][nt][0], s[mt][nt][1], f0, f1);
          mul_f32x2(s[mt][nt][2], s[mt][nt][3], s[mt][nt][2], s[mt][nt][3], f0, f1);
        }
      }
      if (!all_seen) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int2 pq = *reinterpret_cast<const int2*>(s_pos + 8 * nt + 2 * t4);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int key = key0 + 16 * mt + 8 * (c >> 1) + key_of_row(n8);
              const int q = (c & 1) ? pq.y : pq.x;
              const bool see = ((pages_ok >> mt) & 1u) && key < p.span.hi && key <= q &&
                               (a.window < 0 || q - key <= a.window || key < p.sink(a));
              if (!see) s[mt][nt][c] = -INFINITY;
            }
        }
      }

      // raise the references where a score passed them by more than kRescale
      // (the largest score of this thread's keys, alone and with V's scale)
      auto largest = [&](int nt, float (&x)[2], float (&xo)[2]) {
        x[0] = x[1] = xo[0] = xo[1] = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float y0 = fmaxf(s[mt][nt][0], s[mt][nt][2]), y1 = fmaxf(s[mt][nt][1], s[mt][nt][3]);
          x[0] = fmaxf(x[0], y0);
          x[1] = fmaxf(x[1], y1);
          add_f32x2(y0, y1, y0, y1, lvs[mt], lvs[mt]);
          xo[0] = fmaxf(xo[0], y0);
          xo[1] = fmaxf(xo[1], y1);
        }
      };
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[2], xo[2];
        largest(nt, x, xo);
        add_f32x2(x[0], x[1], x[0], x[1], nm[nt][0], nm[nt][1]);
        add_f32x2(xo[0], xo[1], xo[0], xo[1], nmo[nt][0], nmo[nt][1]);
        raise |= fmaxf(x[0], xo[0]) > kRescale;
        raise |= fmaxf(x[1], xo[1]) > kRescale;
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float x[2], xo[2];
          largest(nt, x, xo);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
              x[c] = fmaxf(x[c], __shfl_xor_sync(0xffffffffu, x[c], off));
              xo[c] = fmaxf(xo[c], __shfl_xor_sync(0xffffffffu, xo[c], off));
            }
            if (x[c] + nm[nt][c] > 0.f) {
              l[nt][c] *= ex2(-nm[nt][c] - x[c]);
              nm[nt][c] = -x[c];
            }
            if (xo[c] + nmo[nt][c] > 0.f) {
              const float f = ex2(-nmo[nt][c] - xo[c]);
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                o[i][nt][c] *= f;
                o[i][nt][c + 2] *= f;
              }
              nmo[nt][c] = -xo[c];
            }
          }
        }
      }

      // P^T fragments: p = 2^(x - m) for the sum, p * 2^(lvs + m - mo + kShift) for O
      uint32_t pb[MT][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float b0, b1;  // m - mo + kShift
        fma_f32x2(b0, b1, nm[nt][0], nm[nt][1], -1.f, -1.f, nmo[nt][0], nmo[nt][1]);
        add_f32x2(b0, b1, b0, b1, kShift, kShift);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float u0, u1, e[4];
          add_f32x2(u0, u1, lvs[mt], lvs[mt], b0, b1);
          u0 = ex2(fminf(u0, 120.f));
          u1 = ex2(fminf(u1, 120.f));
#pragma unroll
          for (int c = 0; c < 4; c += 2) {
            add_f32x2(e[c], e[c + 1], s[mt][nt][c], s[mt][nt][c + 1], nm[nt][0], nm[nt][1]);
            e[c] = ex2(e[c]);
            e[c + 1] = ex2(e[c + 1]);
            add_f32x2(l[nt][0], l[nt][1], l[nt][0], l[nt][1], e[c], e[c + 1]);
            mul_f32x2(e[c], e[c + 1], e[c], e[c + 1], u0, u1);
          }
          pb[mt][nt][0] = transpose8x8(pack_f16(e[0], e[1]));
          pb[mt][nt][1] = transpose8x8(pack_f16(e[2], e[3]));
        }
      }

      // O^T += V^T P^T
      if ((a.s_q > 1 || M == kShared) && !all_seen && holds_nan<D, kBlock>(vt, lane)) {
        // NaN among keys that not every query sees (0 * NaN is NaN): the product
        // without them, then NaN where a query sees one
        uint32_t see[MT][NT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int2 pq = *reinterpret_cast<const int2*>(s_pos + 8 * nt + 2 * t4);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int key = key0 + 16 * mt + 8 * hf + key_of_row(n8);
              const bool s0 = key <= pq.x && (a.window < 0 || pq.x - key <= a.window || key < p.sink(a));
              const bool s1 = key <= pq.y && (a.window < 0 || pq.y - key <= a.window || key < p.sink(a));
              see[mt][nt][hf] = transpose8x8(pack_f16(s0 ? 1.f : 0.f, s1 ? 1.f : 0.f));
            }
          }
        add_pv<D, NT, MT, kNoNan>(o, vt, pb, n8, t4);
        add_pv<D, NT, MT, kOnlyNan>(o, vt, see, n8, t4);
      } else {
        add_pv<D, NT, MT, kPlain>(o, vt, pb, n8, t4);
      }
      slot = slot == C::kStages - 1 ? 0 : slot + 1;
    }
    cp_async_wait<0>();

    // ---- the four warps' results through shared memory (the ring is empty)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], off);
    __syncthreads();
    float* buf = reinterpret_cast<float*>(smem);                        // [warp][R][kMergeRow]
    float* st = buf + kWarps * C::R * C::kMergeRow;                     // [warp][R][3]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * nt + 2 * t4 + c;
        float* row = buf + (warp * C::R + r) * C::kMergeRow;
        if constexpr (D == 64) {
#pragma unroll
          for (int j = 0; j < 2; ++j)  // d = 8 n8 + 4 j ..
            *reinterpret_cast<float4*>(row + 8 * n8 + 4 * j) =
                make_float4(o[2 * j][nt][c], o[2 * j][nt][c + 2], o[2 * j + 1][nt][c], o[2 * j + 1][nt][c + 2]);
        } else {
#pragma unroll
          for (int j = 0; j < D / 32; ++j)  // d = 128 (j / 4) + 16 key_of_row(n8) + 4 (j % 4) ..
            *reinterpret_cast<float4*>(row + (j >> 2) * 128 + 16 * key_of_row(n8) + 4 * (j & 3)) =
                make_float4(o[2 * j][nt][c], o[2 * j][nt][c + 2], o[2 * j + 1][nt][c], o[2 * j + 1][nt][c + 2]);
        }
        if (n8 == 0) {
          float* x = st + (warp * C::R + r) * 3;
          x[0] = -nm[nt][c];
          x[1] = -nmo[nt][c] - kShift;
          x[2] = l[nt][c];
        }
      }
    __syncthreads();
    {
      const bool whole = p.t0 == 0 && item_done;
      // a piece that starts inside its item is the first of this CTA, one that
      // ends inside it the last: one slot each
      const int64_t part = 2 * (int64_t)blockIdx.x + (p.t0 == 0 ? 1 : 0);
      constexpr int kVec = D / 4;
      for (int u = threadIdx.x; u < C::R * kVec; u += kThreads) {
        const int r = u / kVec, d4 = u % kVec;
        const int row = p.rt * C::R + r;
        if (row >= p.rows(a)) break;
        float ref = -FLT_MAX;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) ref = fmaxf(ref, st[(w * C::R + r) * 3]);
        float z = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float* x = st + (w * C::R + r) * 3;
          z += x[2] * ex2(x[0] - ref);
          // (in two halves: for small V alone the factor is below fp32's normal numbers)
          const float f = ex2(0.5f * (x[1] - ref));
          const float4 v = *reinterpret_cast<const float4*>(buf + (w * C::R + r) * C::kMergeRow + 4 * d4);
          acc.x += v.x * f * f;
          acc.y += v.y * f * f;
          acc.z += v.z * f * f;
          acc.w += v.w * f * f;
        }
        const float inv = z == 0.f ? 0.f : 1.f / z;
        acc.x *= inv;
        acc.y *= inv;
        acc.z *= inv;
        acc.w *= inv;
        const float lse2 = z == 0.f ? -INFINITY : ref + log2f(z);
        if constexpr (CL) {
          *reinterpret_cast<float4*>(smem + C::fin_off + (r * D + 4 * d4) * 4) = acc;
          if (d4 == 0) reinterpret_cast<float*>(smem + C::fin_off + C::R * D * 4)[r] = lse2;
          continue;
        }
        if (whole) {
          const RowPlace<M> to(a, p, row);
          const int64_t orow = to.orow;
          if (M != kWhole || a.out_fp32)
            reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * D)[d4] = acc;
          else
            reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * D)[d4] =
                make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
          if (d4 == 0) a.lse[to.lse] = lse_out<M>(lse2);
        } else {
          reinterpret_cast<float4*>(a.part_o + (part * C::R + r) * D)[d4] = acc;
          if (d4 == 0) a.part_lse[part * C::R + r] = lse2;
        }
      }
    }
    if constexpr (CL) {
      // every CTA folds its share of the rows from all of the cluster
      cluster_barrier();
      const uint32_t fin = smem_u32(smem) + C::fin_off;
      constexpr int kVec = D / 4;
      for (int u = (int)(blockIdx.x % a.cluster) * kThreads + threadIdx.x; u < C::R * kVec;
           u += a.cluster * kThreads) {
        const int r = u / kVec, d4 = u % kVec;
        const int row = p.rt * C::R + r;
        if (row >= p.rows(a)) break;
        float lses[kMaxCluster], top = -INFINITY;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          lses[c] = c < a.cluster ? load_cluster(cluster_address(fin + (C::R * D + r) * 4, c)) : -INFINITY;
          top = fmaxf(top, lses[c]);
        }
        const float ref = top == -INFINITY ? 0.f : top;
        float z = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          if (c >= a.cluster) break;
          const float f = ex2(lses[c] - ref);
          const float4 v = load_cluster4(cluster_address(fin + (r * D + 4 * d4) * 4, c));
          z += f;
          acc.x += v.x * f;
          acc.y += v.y * f;
          acc.z += v.z * f;
          acc.w += v.w * f;
        }
        const float inv = z == 0.f ? 0.f : 1.f / z;
        const int tok = row / a.g, head = p.kvh * a.g + row % a.g;
        const int64_t orow = ((int64_t)p.seq * a.s_q + tok) * a.h_q + head;
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (a.out_fp32)
          reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * D)[d4] = acc;
        else
          reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * D)[d4] =
              make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
        if (d4 == 0)
          a.lse[((int64_t)p.seq * a.h_q + head) * a.s_q + tok] = z == 0.f ? -INFINITY : (ref + log2f(z)) * kLn2;
      }
      cluster_barrier();  // nobody leaves while its results are read
    } else {
      __syncthreads();  // the ring, q and the row values are free again
    }
  }
  // (this grid may begin before the one of the shared keys ends, but does not end before: its
  // first CTA stays, the others make room)
  if (M == kOwn && blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Folds the partials of an item that several CTAs shared, and writes the empty
// result of a sequence without keys: one thread per four values, the rows of an
// item over blockIdx.y.
constexpr int kFoldThreads = 2 * kThreads;
template <int D, int NT>
constexpr int kFoldRows = NT * 8 * (D / 4) < kFoldThreads ? NT * 8 : kFoldThreads / (D / 4);

template <int D, int NT>
__global__ void __launch_bounds__(kFoldThreads) attn_decode_combine_kernel(const DecodeArgs a) {
  using T = Tune<D, NT>;
  constexpr int R = NT * 8, RP = kFoldRows<D, NT>, kVec = D / 4;
  __shared__ int64_t before[kThreads + 1];
  const Placement pl = place<T, kWhole, R>(a, before);
  const int rt = blockIdx.x % a.row_tiles, kvh = blockIdx.x / a.row_tiles % a.h_kv;
  const int seq = blockIdx.x / (a.row_tiles * a.h_kv);
  const int64_t total = before[kThreads] * a.h_kv;
  const int64_t run = run_length(a, total, T::kMinRun);
  const int t = seq / pl.per;
  int64_t seq_at = before[t];
  for (int i = t * pl.per; i < seq; ++i) seq_at += entry_of<T, kWhole, R>(a, i).span.weight;
  const Span sp = entry_of<T, kWhole, R>(a, seq).span;
  const int count = sp.count;
  const int64_t s0 = seq_at * a.h_kv + (int64_t)kvh * sp.weight + T::kItemCost;  // the item's blocks: [s0, s0 + count)
  const int64_t c0 = count ? s0 / run : 0, c1 = count ? (s0 + count - 1) / run : 0;
  // every CTA waits, so that this grid never ends before the one it depends on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (count && c0 == c1) return;  // written whole
  // The weights of up to kMost pieces at a time through shared memory, then
  // their rows, several loads in flight; later batches of pieces rescale.
  constexpr int kMost = 32;
  __shared__ float s_w[kMost][RP];
  __shared__ float s_ref[RP], s_old[RP];
  const int r = threadIdx.x / kVec, d4 = threadIdx.x % kVec;  // this thread's row and values
  const int r0 = blockIdx.y * RP;                             // the CTA's first row
  const bool mine = r < RP;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float z = 0.f;
  if (threadIdx.x < RP) s_ref[threadIdx.x] = -INFINITY;
  __syncthreads();
  for (int64_t b0 = c0; count && b0 <= c1; b0 += kMost) {
    const int np = (int)min((int64_t)kMost, c1 - b0 + 1);
    // only the first piece can be a CTA's last one (it starts at the item's start)
    auto slot = [&](int i) { return 2 * ((b0 + i) * a.row_tiles + rt) + ((b0 + i) * run <= s0 ? 1 : 0); };
    for (int u = threadIdx.x; u < np * RP; u += kFoldThreads)
      s_w[u / RP][u % RP] = a.part_lse[slot(u / RP) * R + r0 + u % RP];
    __syncthreads();
    if (threadIdx.x < RP) {
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
#pragma unroll 8
      for (int i = 0; i < np; ++i) {
        const float f = ex2(s_w[i][r] - ref);
        const float4 v = reinterpret_cast<const float4*>(a.part_o + (slot(i) * R + r0 + r) * D)[d4];
        z += f;
        acc.x += v.x * f;
        acc.y += v.y * f;
        acc.z += v.z * f;
        acc.w += v.w * f;
      }
    }
    __syncthreads();
  }
  const int row = rt * R + r0 + r;
  if (!mine || row >= a.rows) return;
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

#include "attn_decode_tensor.cuh"

// How a problem is launched: a cluster of `cluster` CTAs per item, or (0) `runs`
// runs of the list.
struct Shape {
  int row_tiles, runs, cluster;
};

template <int D, int NT, int M>
struct Kernel {
  static constexpr int kD = D, kCopies = 1;  // partials of a row
  using T = Tune<D, NT>;
  using C = std::conditional_t<T::kTensor, TensorCfg<D, NT>, Cfg<D, NT>>;
  static constexpr int kPartRows = C::R;  // of a slot of partials
  // CTAs that fill the device once
  static cudaError_t resident(int* n) {
    static std::atomic<int> cache[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool cached = dev >= 0 && dev < kMaxDevices;
    *n = cached ? cache[dev].load(std::memory_order_acquire) : 0;
    if (*n > 0) return cudaSuccess;
    int per_sm = 1;
    if constexpr (T::kTensor) {
      e = cudaFuncSetAttribute(attn_decode_tensor_kernel<D, NT, M>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::bytes);
      if (e != cudaSuccess) return e;
    } else {
      e = cudaFuncSetAttribute(attn_decode_kernel<D, NT, false, M>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               C::bytes);
      if constexpr (T::kClusterBlocks > 0 && M == kWhole) {
        if (e == cudaSuccess)
          e = cudaFuncSetAttribute(attn_decode_kernel<D, NT, true, M>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   C::bytes);
      }
      if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, attn_decode_kernel<D, NT, false, M>, kThreads,
                                                          C::bytes);
      if (e != cudaSuccess) return e;
      if (per_sm < 1) return cudaErrorInvalidConfiguration;
    }
    *n = per_sm * sm_count();
    if (cached) cache[dev].store(*n, std::memory_order_release);
    return cudaSuccess;
  }
  // groups: with kShared, how many
  static cudaError_t shape(const attn_decode_params& p, int64_t groups, Shape* s) {
    const int64_t rows = p.s_q * (p.h_q / p.cache.h_kv);
    const int64_t row_tiles = M == kShared ? 1 : (rows + C::R - 1) / C::R;
    s->row_tiles = (int)row_tiles;
    int n = 0;
    const cudaError_t e = resident(&n);
    if (e != cudaSuccess) return e;
    // blocks of the longest sequence that the page table can hold, as far as the
    // window and the kept tokens reach (which may begin and end inside blocks); a group's
    // reach from its shortest member's window to the end of what is shared
    int64_t blocks = (p.max_pages * p.cache.page_size + T::kBlock - 1) / T::kBlock;
    if (M != kShared && p.window_left >= 0) {
      const int64_t seen = (p.window_left + p.s_q) / T::kBlock + 2 + (p.sink_tokens + T::kBlock - 1) / T::kBlock;
      if (seen < blocks) blocks = seen;
    }
    const int64_t items = p.n * p.cache.h_kv * row_tiles;
    s->cluster = 0;
    if constexpr (T::kClusterBlocks > 0 && M == kWhole) {
      for (int c = kMaxCluster; c > 1 && !s->cluster; c /= 2)
        if (items * c <= n && blocks <= (int64_t)c * kWarps * T::kClusterBlocks) s->cluster = c;
      if (!s->cluster && blocks <= kWarps * (items <= n ? 2 : 1) * kAloneBlocks) s->cluster = 1;
    }
    // no more than shortest runs
    const int64_t entries = M == kShared ? groups + p.n * rows / C::R : p.n;
    const int64_t most = ((blocks + T::kItemCost) * entries * p.cache.h_kv + T::kMinRun - 1) / T::kMinRun;
    const int64_t runs = n / row_tiles > 1 ? n / row_tiles : 1;
    s->runs = most < runs ? (int)most : (int)runs;
    return cudaSuccess;
  }
  // early: the grid may begin before the one before it in the stream has ended
  static cudaError_t launch(DecodeArgs& a, const Shape& sh, bool early, cudaStream_t st) {
    if (a.withhold && !T::kTensor) return cudaErrorNotSupported;
    a.row_tiles = sh.row_tiles;
    a.runs = sh.runs;
    a.cluster = sh.cluster;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.stream = st;
    cfg.attrs = at;
    cfg.dynamicSmemBytes = C::bytes;
    if constexpr (T::kClusterBlocks > 0 && M == kWhole) {
      if (sh.cluster) {
        cfg.gridDim = dim3((unsigned)((int64_t)a.n * a.h_kv * a.row_tiles * sh.cluster));
        cfg.blockDim = dim3(kThreads);
        cfg.numAttrs = 1;
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = sh.cluster;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        return cudaLaunchKernelEx(&cfg, attn_decode_kernel<D, NT, true, M>, a);
      }
    }
    cfg.gridDim = dim3((unsigned)(sh.runs * a.row_tiles));
    if (early) {
      cfg.numAttrs = 1;
      at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[0].val.programmaticStreamSerializationAllowed = 1;
    }
    a.part_lse = a.part_o + (int64_t)2 * sh.runs * a.row_tiles * C::R * D;
    if constexpr (T::kTensor) {
      CUtensorMap tm_k, tm_v;
      if (!encode_page_map(&tm_k, a.k, a.num_pages, a.h_kv, 1 << a.page_shift, D, a.page_stride) ||
          !encode_page_map(&tm_v, a.v, a.num_pages, a.h_kv, 1 << a.page_shift, D, a.page_stride))
        return cudaErrorInvalidValue;
      cfg.blockDim = dim3(C::kThreads);
      return cudaLaunchKernelEx(&cfg, attn_decode_tensor_kernel<D, NT, M>, a, tm_k, tm_v);
    } else {
      cfg.blockDim = dim3(kThreads);
      return cudaLaunchKernelEx(&cfg, attn_decode_kernel<D, NT, false, M>, a);
    }
  }
  // (of the whole contexts, where no cluster took an item alone)
  static cudaError_t fold(const DecodeArgs& a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)((int64_t)a.n * a.h_kv * a.row_tiles), C::R / kFoldRows<D, NT>);
    cfg.blockDim = dim3(kFoldThreads);
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, attn_decode_combine_kernel<D, NT>, a);
  }
};

// f(kernel, shape) with 8 or 16 rows per CTA.  Above 16 rows clusters stay with
// them (twice the CTAs: one sequence of 4096 tokens, Hkv 8 d 128, 64 rows 14.6 us),
// and where the list cuts the work a CTA widens each code for more rows: up to 32 rows
// 32 (at d = 256 the registers end at 16), above 64 or 128 on the tensor-memory path.
// 48 sequences of 100 to 12000 tokens, Hkv 8, us at 32 / 64 / 128 rows by the
// warp-level kernel and by the other: d 64 112 / 214 / 396 and 201 / 201 / 281; d 128
// 186 / 334 / 641 and 235 / 241 / 327; d 256 360 / 703 / 1390 and 402 / 442 / 474.
// (rows: of an item, at most)
template <int D, int M, typename F>
cudaError_t with_rows(const attn_decode_params& p, int64_t groups, int64_t rows, F&& f) {
  auto use = [&](auto k) {
    Shape sh;
    const cudaError_t e = k.shape(p, groups, &sh);
    return e == cudaSuccess ? f(k, sh) : e;
  };
  if (rows <= 8) return use(Kernel<D, 1, M>());
  if (rows > 16) {
    Shape sh;
    const cudaError_t e = Kernel<D, 2, M>::shape(p, groups, &sh);
    if (e != cudaSuccess) return e;
    if (!sh.cluster) {
      // (shared keys of more rows: attn_decode_group.cuh)
      if constexpr (M != kShared || D == 256)
        if (rows > 64) return use(Kernel<D, 16, M>());
      if constexpr (M != kShared || D >= 128)
        if (rows > 32) return use(Kernel<D, 8, M>());
      if constexpr (D < 256) return use(Kernel<D, 4, M>());
    }
  }
  return use(Kernel<D, 2, M>());
}

// The parameters of every list of a problem.
inline DecodeArgs decode_args(const attn_decode_params& p) {
  const attn_kv_cache& c = p.cache;
  DecodeArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(p.q);
  a.k = static_cast<const uint8_t*>(c.k);
  a.v = static_cast<const uint8_t*>(c.v);
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.table = p.page_table;
  a.lens = p.seqlens;
  a.out = p.out;
  a.lse = p.lse;
  a.part_o = static_cast<float*>(p.workspace);
  a.page_stride = c.page_stride > 0 ? c.page_stride : c.h_kv * c.page_size * c.d;
  a.n = a.n_seq = (int)p.n;
  a.s_q = (int)p.s_q;
  a.h_q = (int)p.h_q;
  a.h_kv = (int)c.h_kv;
  a.g = (int)(p.h_q / c.h_kv);
  a.rows = a.s_q * a.g;
  a.max_pages = (int)p.max_pages;
  a.page_shift = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
  a.num_pages = (int)c.num_pages;
  a.window = p.window_left;
  a.sink = (int)p.sink_tokens;
  a.out_fp32 = p.out_fp32 ? 1 : 0;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  return a;
}

}  // namespace

}  // namespace gb300
