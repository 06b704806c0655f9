// The shared keys of groups with more than 32 rows (64 at d 128), on the tensor-memory path,
// included by attn_decode_shared.cu.
//
//   S[rows, keys] = q K^T (8 bits in, q as three e5m2 values),  O[rows, d] += P V (f16 in), fp32 sums
//
// K's codes are multiplied as they lie in the cache, without widening: a bf16 value has 8
// bits, an e5m2 one 3 and a sign, so q, scaled by its row's power of two to at most 57344, is
// the sum of q0 = e5m2(q), q1 = e5m2(q - q0) and q2 = e5m2(q - q0 - q1): what a rounding leaves is
// at most 16 units (of the value's 8 bits) after the first, 1 after the second, 0 after the third.
// That is exact as long as the last of the 8 bits is no less than e5m2's least, 2^-16, which
// holds for values down to 2^-23 of the row's largest; those below are off by at most 2^-17,
// 2^-31 of the largest.  (Two e4m3 values take two products in place of three, but leave
// 2^-18 of the largest: with one value 1000 times the others, in a channel where the keys are
// zero, scores were off by up to 0.08.)  V is widened to f16, P is f16 as in attn_decode_tensor.cuh,
// whose references and factors these are.
//
// A CTA has two softmax groups of 128 threads (a thread per row) on 128-key tiles: with
// 256 rows each has its own rows and both take every tile; with up to 128 rows both have the
// same rows and take the tiles in turn, each with references, sums and an O of its own
// (two partials).  While one group's softmax runs, the tensor unit works for the other.
// Warps by role: 0-7 softmax, 8-11 widen V (a thread per key), 12 loads, 13 and 14 issue the
// products of a group each.
//
// Tensor memory holds, per group, S [128][128] and O [128][D].  A tile goes in halves of 64
// keys: P of a half lies over its S, and the S of the next tile's half is computed as soon
// as O has it, while the softmax works on the other half.
//
// Bound by latency: 2048 rows over 32768 keys, Hkv 8, d 128, in 286 us (970 TFLOP/s, 50 % of
// the measured rate), tensor pipe 52 % and issue 43 % of the time.  With two products for q (259 us, 42 %
// and 49 %) a half of 64 keys took a softmax warp some 2000 cycles for 280 instructions, two such
// warps to a scheduler, and from P to O to the next S of the same half were 1700 more, beside the
// other half's softmax; the third product lengthens that chain.
//
// Every wait ends as in attn_decode_tensor.cuh.
#pragma once

// A tile: every row sees all of it; all of its keys exist.
enum { kAllRows = 1, kAllKeys = 2 };

struct GroupTune {
  static constexpr int kBlock = 128;  // a tile
  // q's conversion, the first copies' latency and the last O, in tiles (us with 1 / 3 / 6: three
  // groups under a window 37.3 / 34.3 / 34.9; 16 sequences behind 60000 tokens, d 64, 57 / 55 / 51;
  // 64 behind 8192, own 100 to 2000, 73.6 / 71.6 / 71.3, own 60 to 200 47.8 / 44.5 / 44.9)
  static constexpr int kItemCost = 6;
  // Longer runs take fewer CTAs, beside which the own keys begin: that pays only where those
  // are many (us with 4 / 5 / 8: 64 sequences behind 2048 tokens, own 60 to 200, 35.5 / 35.7 / 42.0;
  // three groups under a window 34.9 / 36.5 / 42.2; 64 behind 8192, own 60 to 200, 44.9 / 39.6 /
  // 45.3, own 100 to 2000 71.3 / 70.9 / 59.6)
  static constexpr int kMinRun = 4;
};

template <int D, bool kTurns>
struct GroupCfg {
  static constexpr int R = kTurns ? 128 : 256;  // rows of a tile
  static constexpr int kCopies = kTurns ? 2 : 1;  // partials of a row
  static constexpr int kThreads = 32 * 15;
  static constexpr int kKeys = 128;
  static constexpr int kStages = D == 64 ? 4 : kTurns ? 3 : 2;  // tiles of K's codes
  // tiles of V's, which wait in registers and as f16 too (one in place of two: no slower)
  static constexpr int kStagesV = D == 128 && !kTurns ? 1 : kStages;
  static constexpr int kCodes = kKeys * D;      // of K (V)
  static constexpr int kBlock64 = kKeys * 128;  // 64 d's of V in f16
  static constexpr int kV16 = D / 64 * kBlock64;
  static constexpr int kParts = 3, kQ = R * D;  // of q; bytes of one
  static constexpr int k_off = kParts * kQ, v8_off = k_off + kStages * kCodes, v_off = v8_off + kStagesV * kCodes;
  static constexpr int nan_off = v_off + 2 * kV16;  // [D][R / 32] bits: rows that see a NaN of V
  static constexpr int bytes = nan_off + D * R / 8 + 1024;  // (and up to 1023 to align)
  // Scales and the like of a tile are kept until its softmax is done: the loader fills
  // tile i after S of tile i - kStages, which is issued after the softmax of the group's
  // tile before that.
  static constexpr int kMeta = 8;
  static_assert(kStages + 3 <= kMeta, "tiles under way");
  static constexpr uint32_t kCols = 512, kGroupCols = kKeys + D;
  static_assert(2 * kGroupCols <= kCols, "tensor memory");
  static_assert(bytes <= 232448 - 4096, "shared memory");
};

// Instruction descriptor: e5m2 A, e4m3 B (K-major both), fp32 D.
__host__ __device__ constexpr uint32_t idesc_codes_f32(int M, int N) {
  return (1u << 4) | (1u << 7) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// High word of the descriptor of K-major rows of D bytes, swizzled over D bytes (128 or 64).
template <int D>
constexpr uint32_t kSdescHiCodes = ((8u * D) >> 4) | (1u << 14) | ((D == 128 ? 2u : 4u) << 29);

// D[tmem] (+)= A[smem] * B[smem]^T, 32 values of 8 bits along K
template <int D>
__device__ __forceinline__ void mma_codes(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kSdescHiCodes<D>)
      : "memory");
}

// 8 consecutive fp32 values: a whole 32-byte sector.
__device__ __forceinline__ void store8(float* dst, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// The e5m2 codes of two values, which then are what the codes leave of them.
__device__ __forceinline__ uint32_t take_codes(float& x, float& y) {
  uint16_t c;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(c) : "f"(y), "f"(x));
  uint32_t f;
  asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(f) : "h"(c));
  const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&f));
  x -= back.x;
  y -= back.y;
  return c;
}

template <int D, bool kTurns>
__global__ void __launch_bounds__(GroupCfg<D, kTurns>::kThreads, 1)
    decode_group_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v) {
  using C = GroupCfg<D, kTurns>;
  using T = GroupTune;
  constexpr int R = C::R, kStages = C::kStages, kStagesV = C::kStagesV, kKeys = C::kKeys, kUsers = kTurns ? 1 : 2;
  extern __shared__ uint8_t smem_raw[];
  struct Bars {
    uint64_t k_full[kStages];    // a tile's codes of K are there
    uint64_t v_full8[kStagesV];  // and of V
    uint64_t k_free[kStages];    // its K has been multiplied (by every group that takes it)
    uint64_t v_free[kStagesV];   // its V has been read
    uint64_t v_full[2];          // V is there in f16
    uint64_t v_used[2];          // and has been multiplied
    uint64_t q_full, widened;    // of a piece: q in shared memory; all of V widened
    // of a group
    uint64_t meta_full[2];     // a tile's scales are there
    uint64_t s_full[2][2];     // half of S is
    uint64_t p_full[2][2];     // half of P is
    uint64_t o_done[2][2];     // O has it
    uint64_t drain[2];
  };
  __shared__ Bars bars;
  __shared__ TensorWalk<T, kShared, R> walk;
  __shared__ int64_t before[kThreads + 1];
  // of a tile's groups of 16 keys: scales, V's logarithms and inverses, and whether they
  // have a page; the least and the largest scale of V, its first key
  // and kAllRows, kAllKeys
  __shared__ __align__(16) float s_ks[C::kMeta][8], s_vs[C::kMeta][8], s_lv[C::kMeta][8], s_iv[C::kMeta][8];
  __shared__ uint8_t s_ok[C::kMeta][8];
  __shared__ float2 s_range[C::kMeta];
  __shared__ int2 s_tile[C::kMeta];
  __shared__ float s_fac[R];  // what the scores of q's rows are multiplied by
  __shared__ int s_any_nan;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.k_full[i], 8);
      mbar_init(&bars.k_free[i], kUsers);
    }
    for (int i = 0; i < kStagesV; ++i) {
      mbar_init(&bars.v_full8[i], 8);
      mbar_init(&bars.v_free[i], 4);  // (a warp each)
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.v_full[i], 4);
      mbar_init(&bars.v_used[i], kUsers);
      mbar_init(&bars.meta_full[i], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&bars.s_full[i][h], 1);
        mbar_init(&bars.p_full[i][h], 4);
        mbar_init(&bars.o_done[i][h], 1);
      }
      mbar_init(&bars.drain[i], 1);
    }
    mbar_init(&bars.q_full, R / 32);
    mbar_init(&bars.widened, 4);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 13) {
    tmem_alloc(&s_tmem, C::kCols);
    tmem_relinquish();
  }
  const Placement pl = place<T, kShared, R>(a, before);
  if (threadIdx.x == 0) walk.begin(a, pl);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const WaitCtx ctx{&s_abort, nullptr};
  const float bad = __int_as_float(0x7fffffff);
  uint32_t* s_nan = reinterpret_cast<uint32_t*>(smem + C::nan_off);

  uint32_t i0 = 0, n = 0;  // tiles and pieces before this piece
  uint32_t c0 = 0;         // tiles of this warp's group
  uint32_t k_loaded = 0, v_loaded = 0;  // tiles whose copies the loader began
  bool ok = true;
  while (true) {
    if (threadIdx.x == 0) {
      walk.more = walk.advance(a);
      s_any_nan = 0;
    }
    __syncthreads();
    if (!walk.more) break;
    const TensorPiece<kShared>& p = walk.piece;
    const int tiles = p.t1 - p.t0;
    // the group's tiles of this piece
    auto tiles_of = [&](int g) { return kTurns ? (tiles + 1 - g) / 2 : tiles; };

    if (warp == 12) {
      // ====================================================== loader
      // 4 tiles at a time, a lane per 16 keys: their pages are looked up two turns and
      // their scales one turn ahead
      constexpr int kTurn = 4;
      const int* table = p.table(a);
      const int page_mask = (1 << a.page_shift) - 1;
      // the positions of the rows here (those at negative ones see nothing: the fold leaves
      // them out)
      int p_first = 0x7fffffff, p_last = -1;
      {
        const int rows = a.s_q * a.g, end = p.first + (min(p.rows(a), p.rt * R + R) - 1) / rows;
        for (int m = p.first + p.rt * R / rows + lane; m <= end; m += 32) {
          const int len = a.lens[m];
          if (len > 0) p_first = min(p_first, max(len - a.s_q, 0));
          p_last = max(p_last, len - 1);
        }
        p_first = __reduce_min_sync(0xffffffffu, p_first);
        p_last = __reduce_max_sync(0xffffffffu, p_last);
      }
      auto key_of = [&](int t) { return p.span.block(t + (lane >> 3)) * kKeys + (lane & 7) * 16; };
      auto look_up = [&](int t) {
        return t + (lane >> 3) < p.t1 && key_of(t) < p.span.hi ? table[key_of(t) >> a.page_shift] : -1;
      };
      auto valid = [&](int pid) { return pid >= 0 && pid < a.num_pages; };
      auto scale_at = [&](int pid) { return (int64_t)(valid(pid) ? pid : 0) * a.h_kv + p.kvh; };
      int pid0 = look_up(p.t0), pid1 = look_up(p.t0 + kTurn);
      float ks = a.k_scale[scale_at(pid0)], vs = a.v_scale[scale_at(pid0)];
      uint32_t i = i0;
      for (int t = p.t0; t < p.t1 && ok && !a.withhold; t += kTurn) {
        const float ks1 = a.k_scale[scale_at(pid1)], vs1 = a.v_scale[scale_at(pid1)];
        const int pid2 = look_up(t + 2 * kTurn);
        const int key = key_of(t), key0 = key - (lane & 7) * 16;
        const bool take = valid(pid0);
        const bool whole = ((__ballot_sync(0xffffffffu, take) >> (lane & 24)) & 0xffu) == 0xffu;
        const bool keys = whole && key0 + kKeys <= p.span.hi;
        const bool all = keys && key0 + kKeys - 1 <= p_first &&
                         (a.window < 0 || p_last - key0 <= a.window || key0 + kKeys - 1 < a.sink);
        float2 range = make_float2(vs, vs);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          range.x = fminf(range.x, __shfl_xor_sync(0xffffffffu, range.x, o));
          range.y = fmaxf(range.y, __shfl_xor_sync(0xffffffffu, range.y, o));
        }
        for (int u = 0; u < kTurn && t + u < p.t1; ++u, ++i) {
          const int slot = i % kStages, slot_v = i % kStagesV, g = lane & 7, y = key & page_mask;
          if (i >= kStages) ok = wait_on(&bars.k_free[slot], (i / kStages - 1) & 1, ctx);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane >> 3 == u) {
            const int m = i % C::kMeta;
            s_ks[m][g] = take ? ks : 0.f;
            s_vs[m][g] = take ? vs : 0.f;
            s_lv[m][g] = take ? lg2(vs) : 0.f;
            s_iv[m][g] = take ? 1.f / vs : 0.f;
            s_ok[m][g] = take;
            if (g == 0) {
              s_tile[m] = make_int2(key0, (all ? kAllRows : 0) | (keys ? kAllKeys : 0));
              s_range[m] = range;
            }
            if (take) {
              mbar_arrive_expect_tx(&bars.k_full[slot], 16 * D);
              tma_load_4d(smem_u32(smem + C::k_off + slot * C::kCodes) + g * 16 * D, &tm_k, 0, y, p.kvh, pid0,
                          &bars.k_full[slot]);
            } else {
              mbar_arrive(&bars.k_full[slot]);
            }
          }
          k_loaded = i + 1;
          if (i >= kStagesV) ok = wait_on(&bars.v_free[slot_v], (i / kStagesV - 1) & 1, ctx);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane >> 3 == u) {
            if (take) {
              mbar_arrive_expect_tx(&bars.v_full8[slot_v], 16 * D);
              tma_load_4d(smem_u32(smem + C::v8_off + slot_v * C::kCodes) + g * 16 * D, &tm_v, 0, y, p.kvh, pid0,
                          &bars.v_full8[slot_v]);
            } else {
              mbar_arrive(&bars.v_full8[slot_v]);
            }
          }
          v_loaded = i + 1;
        }
        pid0 = pid1;
        pid1 = pid2;
        ks = ks1;
        vs = vs1;
      }
    } else if (warp >= 13) {
      // ====================================================== products of a group: one thread
      const int g = warp - 13;
      constexpr int kEvery = kTurns ? 2 : 1;
      constexpr uint32_t idesc_s = idesc_codes_f32(128, kKeys / 2), idesc_o = idesc_f16_f32(128, D, false, true);
      const int t0 = kTurns ? g : 0;
      if (lane > 0) {
        // (nothing to do)
      } else if (!kTurns && p.rt * R + g * 128 >= p.rows(a)) {
        // a group without rows: in step, since a stage is not filled again before both groups
        // have passed it
        for (int t = 0; t < tiles && ok; ++t) {
          const uint32_t i = i0 + t;
          ok = mbar_wait(&bars.k_full[i % kStages], (i / kStages) & 1, ctx);
          if (ok) ok = mbar_wait(&bars.v_full[i & 1], (i >> 1) & 1, ctx);
          if (!ok) break;
          mbar_arrive(&bars.k_free[i % kStages]);
          mbar_arrive(&bars.v_used[i & 1]);
        }
      } else if (ok && t0 < tiles) {
        const uint32_t t_s = tmem + g * C::kGroupCols, t_o = t_s + kKeys;
        const uint32_t q_lo = sdesc_lo(smem_u32(smem + (kTurns ? 0 : g) * 128 * D), 16);
        const uint32_t k_lo = sdesc_lo(smem_u32(smem + C::k_off), 16);
        const uint32_t v_lo = sdesc_lo(smem_u32(smem + C::v_off), C::kBlock64);
        ok = mbar_wait(&bars.q_full, n & 1, ctx);
        uint32_t c = c0;
        // t = t0 - kEvery: both halves of S of the first tile; then, half by half, O of tile t
        // and S of the tile after it, over P that O has just taken
        for (int t = t0 - kEvery; t < tiles && ok; t += kEvery) {
          const uint32_t i = i0 + t, i1 = i + kEvery;
          const int buf = i & 1, slot = i1 % kStages;
          const bool begun = t >= t0, more = t + kEvery < tiles;
          if (begun) ok = mbar_wait(&bars.v_full[buf], (i >> 1) & 1, ctx);
          const uint32_t v = v_lo + ((buf * C::kV16) >> 4), k = k_lo + ((slot * C::kCodes) >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (begun) {
              if (ok) ok = mbar_wait(&bars.p_full[g][h], (c - 1) & 1, ctx);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ts_lo(t_o, t_s + h * 64 + kk * 8, v + (((h * 4 + kk) * 2048) >> 4), idesc_o,
                          kk > 0 || h > 0 || t > t0 ? 1u : 0u);
              mma_commit(&bars.o_done[g][h]);
              if (h == 1) mma_commit(&bars.v_used[buf]);
            }
            if (more) {
              if (h == 0) ok = mbar_wait(&bars.k_full[slot], (i1 / kStages) & 1, ctx);
              if (ok && c > 0) ok = mbar_wait(&bars.o_done[g][h], (c - 1) & 1, ctx);
              if (!ok) break;
              tc_fence_after();
              if (h == 0) mbar_arrive(&bars.meta_full[g]);
#pragma unroll
              for (int kk = 0; kk < C::kParts * (D / 32); ++kk) {  // q0, q1, q2
                const int part = kk / (D / 32), at = kk % (D / 32) * 32;
                mma_codes<D>(t_s + h * 64, q_lo + ((part * C::kQ + at) >> 4), k + ((h * 64 * D + at) >> 4), idesc_s,
                             kk > 0 ? 1u : 0u);
              }
              mma_commit(&bars.s_full[g][h]);
              if (h == 1) mma_commit(&bars.k_free[slot]);
            }
          }
          ++c;
        }
      }
      __syncwarp();
    } else if (warp >= 8) {
      // ====================================================== V to f16
      const int k = threadIdx.x & 127;  // this thread's key of a tile
      for (int u = k; u < D * R / 32; u += 128) s_nan[u] = 0u;
      asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
      for (int t = 0; t < tiles; ++t) {
        const uint32_t i = i0 + t;
        const int slot = i % kStagesV, buf = i & 1, m = i % C::kMeta;
        if (ok) ok = wait_on(&bars.v_full8[slot], (i / kStagesV) & 1, ctx);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint8_t* base = smem + C::v8_off + slot * C::kCodes;
        uint32_t w[D / 4];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(base + code_offset<D>(k, c));
          w[4 * c] = x.x;
          w[4 * c + 1] = x.y;
          w[4 * c + 2] = x.z;
          w[4 * c + 3] = x.w;
        }
        const int2 tile = s_tile[m];
        if (!(tile.y & kAllRows)) {
          const int key = tile.x + k;
          const bool some = s_ok[m][k >> 4] && key < p.span.hi && (key >= p.span.lo || key < p.span.sink_hi);
          if (some) {
            // a NaN that not every row sees (0 * NaN is NaN) is left out of the product and
            // noted for those that do
            uint32_t any = 0u;
#pragma unroll
            for (int j = 0; j < D / 4; ++j) any |= nan_bytes(w[j]);
            if (any) {
              s_any_nan = 1;
              const int rows = min(p.rows(a) - p.rt * R, R);
#pragma unroll 1
              for (int r32 = 0; r32 < rows; r32 += 32) {
                uint32_t mask = 0u;
#pragma unroll 1
                for (int r = r32; r < min(rows, r32 + 32); ++r) {
                  const int q = RowPlace<kShared>(a, p, p.rt * R + r).pos;
                  if (key <= q && (a.window < 0 || q - key <= a.window || key < a.sink)) mask |= 1u << (r & 31);
                }
#pragma unroll 1
                for (int d = 0; d < D; ++d)
                  if ((base[code_offset<D>(k, d >> 4) + (d & 15)] & 0x7f) == 0x7f)
                    atomicOr(s_nan + d * (R / 32) + (r32 >> 5), mask);
              }
#pragma unroll
              for (int j = 0; j < D / 4; ++j) w[j] &= ~nan_bytes(w[j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < D / 4; ++j) w[j] = 0u;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.v_free[slot]);
        // the f16 tile that was there has been multiplied
        if (i >= 2) ok = wait_on(&bars.v_used[buf], ((i >> 1) - 1) & 1, ctx);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t* dst = smem + C::v_off + buf * C::kV16;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {  // 8 d's
          uint4 f;
          f.x = widen_lo(w[2 * c]);
          f.y = widen_hi(w[2 * c]);
          f.z = widen_lo(w[2 * c + 1]);
          f.w = widen_hi(w[2 * c + 1]);
          *reinterpret_cast<uint4*>(dst + (c >> 3) * C::kBlock64 + k * 128 + (((c ^ k) & 7) << 4)) = f;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.v_full[buf]);
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&bars.widened);
    } else {
      // ====================================================== softmax
      const int g = warp >> 2, wq = warp & 3, th = threadIdx.x & 127;
      const int r = kTurns ? th : threadIdx.x;  // this thread's row of the tile
      const int row = p.rt * R + r;
      const bool mine = row < p.rows(a), busy = row - lane < p.rows(a);  // (this warp has rows)
      const RowPlace<kShared> to(a, p, mine ? row : 0);
      const int pos = mine ? to.pos : -1;
      if (!kTurns || g == 0) {
        // ---- q's row (all of its loads at once) as three e5m2 values each, the largest value in
        // (28672, 57344]
        const uint4* src = reinterpret_cast<const uint4*>(a.q + to.orow * D);
        uint4 x[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) x[c] = mine ? src[c] : make_uint4(0u, 0u, 0u, 0u);
        uint32_t top = 0u;
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          top = top_bf16x2(top_bf16x2(top_bf16x2(top_bf16x2(top, x[c].x), x[c].y), x[c].z), x[c].w);
        const uint32_t bits = top_of(top);
        const bool finite = bits < 0x7f800000u;
        const int over = (bits & 0x7fffffu) > 0x600000u ? 1 : 0;
        const int ex = finite && bits ? max((int)(bits >> 23) - 127 + over, -100) - 15 : 0;
        const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
        s_fac[r] = mine ? row_factor(a, ex, finite) : 0.f;
        uint8_t* dst = smem + (kTurns ? 0 : g) * 128 * D;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {  // 16 values
          uint32_t part[C::kParts][8];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t w[4] = {x[2 * c + u].x, x[2 * c + u].y, x[2 * c + u].z, x[2 * c + u].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float y = __uint_as_float(w[j] << 16) * inv, z = __uint_as_float(w[j] & 0xffff0000u) * inv;
#pragma unroll
              for (int i = 0; i < C::kParts; ++i) part[i][4 * u + j] = take_codes(y, z);
            }
          }
#pragma unroll
          for (int i = 0; i < C::kParts; ++i)
            *reinterpret_cast<uint4*>(dst + i * C::kQ + code_offset<D>(th, c)) =
                make_uint4(part[i][0] | part[i][1] << 16, part[i][2] | part[i][3] << 16,
                           part[i][4] | part[i][5] << 16, part[i][6] | part[i][7] << 16);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&bars.q_full);
      }
      if (ok) ok = wait_on(&bars.q_full, n & 1, ctx);
      const float fac = s_fac[r];
      const uint32_t t_s = tmem + ((uint32_t)(wq * 32) << 16) + g * C::kGroupCols, t_o = t_s + kKeys;
      // the references of P and of P * v_scale (negated; at first below every score),
      // 2^(m - mo + kShift), the sum of P
      float nm = FLT_MAX, nmo = FLT_MAX, b = 1.f, l = 0.f;
      float shift = FLT_MAX, b_inv = 1.f;  // nmo + kShift, 1 / b
      const int count = busy || kTurns || p.rt * R + g * 128 < p.rows(a) ? tiles_of(g) : 0;
      uint32_t c = c0;
#pragma unroll 1
      for (int t = 0; t < count; ++t, ++c) {
        const uint32_t i = i0 + (kTurns ? 2 * t + g : t);
        const int m = i % C::kMeta;
        if (ok) ok = mbar_wait(&bars.meta_full[g], c & 1, ctx);
        __syncwarp();
        const int2 tile = s_tile[m];
        const bool all_seen = tile.y & kAllRows;
        // this row sees all of the tile, or nothing
        const bool full = tile.x + kKeys - 1 <= pos &&
                          (a.window < 0 || pos - tile.x <= a.window || tile.x + kKeys - 1 < a.sink);
        const bool none = tile.x > pos || (a.window >= 0 && pos - (tile.x + kKeys - 1) > a.window && tile.x >= a.sink);
        const bool quick = all_seen || ((tile.y & kAllKeys) && __all_sync(0xffffffffu, full || none));
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int col0 = h * 64;
          if (ok) ok = mbar_wait(&bars.s_full[g][h], c & 1, ctx);
          __syncwarp();
          tc_fence_after();
          if (busy) {
            // Where each row sees all keys or none and b * v_scale is far from fp32's ends (it is but for
            // pages of zeros and the like), P * v_scale comes straight from the exponential, and the
            // sum of P from the sums over 16 keys, which tell of values past f16's range too (and
            // of NaN, which may be out of sight).
            bool done = quick;
            if (done) {
              uint32_t pk[32];
              float sum = 0.f, most = 0.f;
              float2 e[32];
              tmem_ld32(t_s + col0, reinterpret_cast<uint32_t*>(e));
              tmem_ld32(t_s + col0 + 32, reinterpret_cast<uint32_t*>(e) + 32);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 4; ++x) {  // 16 keys
                const float f = fac * s_ks[m][4 * h + x], o = s_lv[m][4 * h + x] + (none ? -INFINITY : shift);
#pragma unroll
                for (int j = 8 * x; j < 8 * x + 8; ++j) e[j] = __ffma2_rn(e[j], make_float2(f, f), make_float2(o, o));
              }
#pragma unroll
              for (int j = 0; j < 32; ++j) e[j] = make_float2(ex2(e[j].x), ex2(e[j].y));
#pragma unroll
              for (int j = 0; j < 32; ++j) pk[j] = pack_f16(e[j].x, e[j].y);
#pragma unroll
              for (int w = 1; w < 8; w *= 2)
#pragma unroll
                for (int j = 0; j < 32; j += 2 * w) e[j] = __fadd2_rn(e[j], e[j + w]);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const float y = e[8 * x].x + e[8 * x].y;
                most = fmaxf(most, y);
                sum += y * (s_iv[m][4 * h + x] * b_inv);
              }
              const float2 range = s_range[m];
              done = __all_sync(0xffffffffu, most <= 32768.f && sum <= 16384.f && b * range.y < 0x1p60f &&
                                                 b * range.x > 0x1p-60f);
              if (done) {
                l += sum;
                tmem_st32(t_s + col0, pk);
              }
            }
            if (!done) {
              // keys of the tile that this row sees: up to j_last, from j_first on or below j_sink, on pages
              // that there are
              const int j_last = min(pos, p.span.hi - 1) - tile.x, j_first = a.window < 0 ? 0 : max(pos - tile.x, 0) - a.window,
                        j_sink = a.window < 0 ? 0 : a.sink - tile.x;
              auto sees = [&](int j) { return j <= j_last && (j >= j_first || j < j_sink); };
              // raise the references where a score passes them by more than kRescale, to the largest of
              // these keys
              float x = -INFINITY, xo = -INFINITY;
#pragma unroll 1
              for (int j0 = col0; j0 < col0 + 64; j0 += 16) {
                float e[16];
                tmem_ld16(t_s + j0, reinterpret_cast<uint32_t*>(e));
                tmem_wait_ld();
                const float f = fac * s_ks[m][j0 / 16], lv = lg2(s_vs[m][j0 / 16]);
                float y = -INFINITY;
#pragma unroll
                for (int j = 0; j < 16; ++j) y = fmaxf(y, sees(j0 + j) ? e[j] * f : -INFINITY);
                if (!s_ok[m][j0 / 16]) y = -INFINITY;
                x = fmaxf(x, y);
                xo = fmaxf(xo, y + lv);
              }
              if (__any_sync(0xffffffffu, x + nm > kRescale || xo + nmo > (b * s_range[m].y > FLT_MAX ? 0.f : kRescale))) {
                const float nm1 = x + nm > 0.f ? -x : nm;
                // (b stays a normal number: attn_decode_tensor.cuh)
                const float nmo1 = fminf(fmaxf(xo + nmo > 0.f ? -xo : nmo, nm1 - 130.f), nm1 + 119.f);
                const float fo = ex2(nmo1 - nmo);
                l *= ex2(nm1 - nm);
                nm = nm1;
                nmo = nmo1;
                b = ex2(nmo1 - nm1 + kShift);
                b_inv = ex2(nm1 - nmo1 - kShift);
                shift = nmo1 + kShift;
                if (t > 0 || h > 0) {
                  if (ok)
                    ok = h ? wait_on(&bars.o_done[g][0], c & 1, ctx) : wait_on(&bars.o_done[g][1], (c - 1) & 1, ctx);
                  __syncwarp();
                  tc_fence_after();
#pragma unroll 1
                  for (int cc = 0; cc < D; cc += 32) {
                    float o[32];
                    tmem_ld32(t_o + cc, reinterpret_cast<uint32_t*>(o));
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] *= fo;
                    tmem_st32(t_o + cc, reinterpret_cast<const uint32_t*>(o));
                  }
                }
              }
              // P 16 keys at a time, over scores that have been read
#pragma unroll 1
              for (int cc = 0; cc < 64; cc += 16) {
                float2 e[8];
                uint32_t pk[8];
                tmem_ld16(t_s + col0 + cc, reinterpret_cast<uint32_t*>(e));
                // (b * v_scale may pass fp32's range where keys are out of sight or of next to no weight: 0
                // * infinity is NaN, so P takes the largest finite value)
                const float f = fac * s_ks[m][(col0 + cc) / 16], v = fminf(b * s_vs[m][(col0 + cc) / 16], FLT_MAX);
                const bool here = s_ok[m][(col0 + cc) / 16];
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  e[j] = __ffma2_rn(e[j], make_float2(f, f), make_float2(nm, nm));
                  if (!here || !sees(col0 + cc + 2 * j)) e[j].x = -INFINITY;
                  if (!here || !sees(col0 + cc + 2 * j + 1)) e[j].y = -INFINITY;
                  e[j] = make_float2(ex2(e[j].x), ex2(e[j].y));
                  l += e[j].x + e[j].y;
                  e[j] = __fmul2_rn(e[j], make_float2(v, v));
                  pk[j] = pack_f16(e[j].x, e[j].y);
                }
                tmem_st8(t_s + col0 + cc / 2, pk);
              }
            }
            tmem_wait_st();
          }
          tc_fence_before();
          // (a lane that gave up has only its own row to spoil, and that one ends as NaN)
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(&bars.p_full[g][h]);
        }
      }
      if (count > 0) {
        if (ok) ok = wait_on(&bars.o_done[g][1], (c - 1) & 1, ctx);
        if (ok) ok = wait_on(&bars.widened, n & 1, ctx);
      }
      __syncwarp();
      tc_fence_after();

      // ---- the row's result; a piece that starts inside its item is the first of
      // this CTA, one that ends inside it the last: one slot each
      if (busy) {
        const int64_t part_row = (2 * (int64_t)blockIdx.x + (p.t0 == 0 ? 1 : 0)) * 256 + threadIdx.x;
        const int copy = kTurns ? g : 0;
        if (!ok) l = bad;
        // O times 2^(mo - m) / l, as w * w2 (for small V alone the product is below fp32's
        // normal numbers)
        const float w2 = ex2(0.5f * (-nmo + nm - kShift));
        const float w = (l == 0.f ? 0.f : 1.f / l) * w2;
        float* lse = p.whole ? a.lse + copy * a.copy_floats + to.lse : a.part_lse + part_row;
        float* dst = p.whole ? static_cast<float*>(a.out) + copy * a.copy_floats + to.orow * D : a.part_o + part_row * D;
        if (mine) *lse = l == 0.f ? -INFINITY : log2f(l) - nm;
        const bool nans = s_any_nan;
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
          float o[32];
          if (count > 0) {
            tmem_ld32(t_o + cc, reinterpret_cast<uint32_t*>(o));
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              mul_f32x2(o[j], o[j + 1], o[j], o[j + 1], w, w);
              mul_f32x2(o[j], o[j + 1], o[j], o[j + 1], w2, w2);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = ok ? 0.f : bad;
          }
          // (both partials of a row have the mark: NaN however little one of them weighs)
          if (nans) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if ((s_nan[(cc + j) * (R / 32) + (r >> 5)] >> lane) & 1u) o[j] = bad;
          }
          if (mine) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) store8(dst + cc + j, o + j);
          }
        }
      }
      tc_fence_before();
    }
    i0 += tiles;
    const int own_g = warp >= 13 ? warp - 13 : (warp >> 2) & 1;
    if (kTurns || p.rt * R + own_g * 128 < p.rows(a)) c0 += tiles_of(own_g);
    ++n;
    __syncthreads();
    tc_fence_after();
  }
  // copies and products have ended (so they have, unless a wait ran out somewhere)
  if (warp == 12 && lane == 0) {
    for (uint32_t j = k_loaded < kStages ? 0 : k_loaded - kStages; j < k_loaded; ++j)
      mbar_wait_drain(&bars.k_full[j % kStages], (j / kStages) & 1, nullptr);
    for (uint32_t j = v_loaded < kStagesV ? 0 : v_loaded - kStagesV; j < v_loaded; ++j)
      mbar_wait_drain(&bars.v_full8[j % kStagesV], (j / kStagesV) & 1, nullptr);
  }
  if (warp >= 13 && lane == 0) {
    mma_commit(&bars.drain[warp - 13]);
    mbar_wait_drain(&bars.drain[warp - 13], 0, nullptr);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

template <int D, bool kTurns>
struct GroupKernel {
  static constexpr int kD = D, kCopies = kTurns ? 2 : 1;
  using T = GroupTune;
  using C = GroupCfg<D, kTurns>;
  static constexpr int kPartRows = 256;  // of a slot
  static cudaError_t shape(const attn_decode_params& p, int64_t groups, Shape* s) {
    static std::atomic<int> done[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool cached = dev >= 0 && dev < kMaxDevices;
    if (!cached || !done[dev].load(std::memory_order_acquire)) {
      e = cudaFuncSetAttribute(decode_group_kernel<D, kTurns>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::bytes);
      if (e != cudaSuccess) return e;
      if (cached) done[dev].store(1, std::memory_order_release);
    }
    s->row_tiles = 1;
    s->cluster = 0;
    // no more than shortest runs
    const int64_t tiles = (p.max_pages * p.cache.page_size + T::kBlock - 1) / T::kBlock;
    const int64_t entries = groups + p.n * p.s_q * (p.h_q / p.cache.h_kv) / C::R;
    const int64_t most = ((tiles + T::kItemCost) * entries * p.cache.h_kv + T::kMinRun - 1) / T::kMinRun;
    const int sms = sm_count();
    s->runs = most < sms ? (int)most : sms;
    return cudaSuccess;
  }
  static cudaError_t launch(DecodeArgs& a, const Shape& sh, bool, cudaStream_t st) {
    a.row_tiles = 1;
    a.runs = sh.runs;
    a.cluster = 0;
    a.part_lse = a.part_o + (int64_t)2 * sh.runs * kPartRows * D;
    CUtensorMap tm_k, tm_v;
    if (!encode_page_map(&tm_k, a.k, a.num_pages, a.h_kv, 1 << a.page_shift, D, a.page_stride) ||
        !encode_page_map(&tm_v, a.v, a.num_pages, a.h_kv, 1 << a.page_shift, D, a.page_stride))
      return cudaErrorInvalidValue;
    decode_group_kernel<D, kTurns><<<sh.runs, C::kThreads, C::bytes, st>>>(a, tm_k, tm_v);
    return cudaGetLastError();
  }
};
