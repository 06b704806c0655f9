// The kernel for more rows than the warp-level one is good for (drafted tokens
// times a large group): 128 rows per CTA on the tensor-memory path, included by
// attn_decode.cu.
//
//   S[rows, keys] = q K^T,  O[rows, d] += P V   (f16 in, fp32 sums)
//
// One CTA per SM, its warps by role:
//   loader    copies the codes of 16 keys at a time (TMA, swizzled) into a ring
//   widening  a thread per key, one group of warps for K and one for V: the codes,
//             exactly, into f16 rows of 64 d's, in place (a slot has the room)
//   products  one thread: S in two buffers, O behind P
//   softmax   4 warps, a thread per row: q's row as f16 into tensor memory once a
//             piece; scores out of it, P (f16) back in their place
// The time is the softmax's: its 128 keys of a tile take a warp 2900 cycles (one warp
// per scheduler, so latencies count: the e^x 1090, the sums, factors and packing
// 1100, the maxima 440), where HBM would take 1410 at d = 128.  That does not depend
// on the rows.  Tried, 128 rows at d = 128 (305 us for 48 sequences of 100 to 12000
// tokens, Hkv 8): two softmax groups on tiles of 64 keys with an accumulator each 392;
// 216 registers for the softmax and a thread each for S and O 374; keys on the M side
// (a thread per key, P through shared memory, votes over threads) 495 with two CTAs
// per SM, 541 by roles.
#pragma once

// One piece of work: blocks [t0, t1) of an item; whole: all of it.
struct TensorPiece {
  int seq, kvh, rt, t0, t1, len;
  bool whole;
  Span span;
};

// A way through the CTA's run of the list, one per role, in shared memory: the
// role's leader goes on, sync is the role's barrier.
template <typename T>
struct TensorWalk {
  int64_t at, end;
  int64_t seq_at;  // where the sequence starts in the list
  int seq;
  bool more;
  TensorPiece piece;

  // (one thread, after place)
  __device__ __forceinline__ void begin(const DecodeArgs& a, const Placement& pl) {
    const int64_t total = pl.before[kThreads] * a.h_kv;
    const int64_t run = run_length(a, total);
    at = blockIdx.x / a.row_tiles * run;
    end = min(at + run, total);
    if (at >= end) return;
    // the sequence of the run's first block
    int t = 0;
#pragma unroll
    for (int step = kThreads / 2; step > 0; step >>= 1)
      if (pl.before[t + step] * a.h_kv <= at) t += step;
    // (entries behind the last sequence repeat the total, which is above `at`)
    seq = t * pl.per;
    seq_at = pl.before[t] * a.h_kv;
    for (; seq < a.n - 1; ++seq) {
      const int64_t c = (int64_t)span_of<T>(a, a.lens[seq]).weight * a.h_kv;
      if (at < seq_at + c) break;
      seq_at += c;
    }
  }
  // The next piece with a block, if there is one (false: the run is done).
  template <typename Sync>
  __device__ __forceinline__ bool next(const DecodeArgs& a, TensorPiece& p, bool leader, Sync&& sync) {
    sync();  // everybody has the last one
    if (leader) more = advance(a);
    sync();
    p = piece;
    return more;
  }

 private:
  __device__ __forceinline__ bool advance(const DecodeArgs& a) {
    while (at < end && seq < a.n) {
      TensorPiece p;
      p.seq = seq;
      p.len = a.lens[seq];
      p.span = span_of<T>(a, p.len);
      if (p.span.count == 0) {
        ++seq;
        continue;
      }
      // the piece [w0, w1) of the item's weight: its first kItemCost hold no block
      const int64_t in_seq = at - seq_at;
      const int weight = p.span.weight;
      p.kvh = (int)(in_seq / weight);
      p.rt = blockIdx.x % a.row_tiles;
      const int w0 = (int)(in_seq - (int64_t)p.kvh * weight);
      const int w1 = (int)min((int64_t)weight, w0 + (end - at));
      p.t0 = max(w0 - T::kItemCost, 0);
      p.t1 = max(w1 - T::kItemCost, 0);
      p.whole = p.t0 == 0 && w1 == weight;
      at += w1 - w0;
      if (w1 == weight && p.kvh == a.h_kv - 1) {
        seq_at += (int64_t)weight * a.h_kv;
        ++seq;
      }
      if (p.t1 > p.t0) {
        piece = p;
        return true;
      }
    }
    return false;
  }
};

// Instruction descriptor: f16 A and B, fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// mbar_wait, asleep once before the clock is read.
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, const WaitCtx& ctx) {
  if (mbar_try_wait_sleep(smem_u32(bar), parity, kSleepHintNs)) return true;
  if (*ctx.abort_flag) return false;
  return mbar_wait(bar, parity, ctx);
}

template <int D>
struct TensorCfg {
  using T = Tune<D, kTensorNT>;
  static constexpr int R = kTensorNT * 8;
  static constexpr int kThreads = 32 * 14;  // K 4, V 4, softmax 4, products, loader
  static constexpr int kKeys = D == 256 ? 64 : 128;  // per tile
  static constexpr int kBlocks = kKeys / 32;
  static constexpr int kStages = T::kStages;
  // A slot: K, then V, 64 d's after another, a key's 128 bytes after another's (4 KB
  // per block of keys).  The codes come into the first half of a block's room.
  static constexpr int kBlock64 = kKeys * 128;
  static constexpr int kHalf = D / 64 * kBlock64;
  static constexpr int kStage = 2 * kHalf;
  static constexpr int nan_off = kStages * kStage;  // of two pieces: [D][4] bits: rows that see a NaN of V
  static constexpr int bytes = nan_off + 2 * D * 16 + 1024;  // (and up to 1023 to align)
  // tensor memory: q [rows][D / 2], S [rows][kKeys] twice (later P in its first half), O [rows][D]
  static constexpr uint32_t col_s = D / 2, col_o = col_s + 2 * kKeys;
  static constexpr uint32_t kCols = 512;
  static_assert(R == 128, "rows");
  static_assert(col_o + D <= kCols, "tensor memory");
  static_assert(bytes <= 232448 - 4096, "shared memory");
};

// Where 16-byte piece c of key row `row` of a block's codes lies in its room (the
// copy's 64-byte or 128-byte swizzle).
template <int D>
__device__ __forceinline__ int code_offset(int row, int c) {
  if constexpr (D == 64)
    return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
  else
    return (c >> 3) * (D == 256 ? 64 * 128 : 128 * 128) + row * 128 + (((c ^ row) & 7) << 4);
}

template <int D>
__global__ void __launch_bounds__(TensorCfg<D>::kThreads, 1)
attn_decode_tensor_kernel(const DecodeArgs a, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v) {
  using C = TensorCfg<D>;
  using T = typename C::T;
  constexpr int R = C::R, kStages = C::kStages, NB = C::kBlocks, kKeys = C::kKeys;
  extern __shared__ uint8_t smem_raw[];
  struct Bars {
    uint64_t full[kStages];    // a tile's codes are there
    uint64_t k_full[kStages];  // its K is f16
    uint64_t v_full[kStages];  // its V is
    uint64_t free[kStages];    // the tile is done with
    uint64_t q_full;           // q is in tensor memory
    uint64_t s_full[2];        // S is there
    uint64_t p_full[2];        // P is in its place
    uint64_t o_done[2];        // O has it
    uint64_t widened[2], done[2];  // of a piece: V, everything
    uint64_t drain;
  };
  __shared__ Bars bars;
  __shared__ TensorWalk<T> walks[5];
  __shared__ int64_t before[kThreads + 1];
  // of a tile's groups of 16 keys: scales and whether they have a page; of its
  // blocks: the first key and whether every query sees all of them
  __shared__ float s_ks[kStages][2 * NB], s_vs[kStages][2 * NB];
  __shared__ uint8_t s_ok[kStages][2 * NB];
  __shared__ int2 s_block[kStages][NB];
  __shared__ int s_any_nan[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.full[i], 2 * NB);
      mbar_init(&bars.k_full[i], kKeys);
      mbar_init(&bars.v_full[i], kKeys);
      mbar_init(&bars.free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], 128);
      mbar_init(&bars.o_done[i], 1);
      mbar_init(&bars.widened[i], 128);
      mbar_init(&bars.done[i], 128);
    }
    mbar_init(&bars.q_full, 128);
    mbar_init(&bars.drain, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, C::kCols);
    tmem_relinquish();
  }
  const Placement pl = place<T>(a, before);
  // roles: 0 K, 1 V, 2 softmax, 3 products, 4 loader
  const int role = warp < 12 ? warp >> 2 : warp - 9;
  if (lane == 0 && (warp >= 12 || (warp & 3) == 0)) walks[role].begin(a, pl);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const WaitCtx ctx{&s_abort, nullptr};
  TensorWalk<T>& walk = walks[role];
  auto warp_sync = [] { __syncwarp(); };
  auto group_sync = [&] { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + role) : "memory"); };
  // of piece number n
  auto s_nan = [&](int n) { return reinterpret_cast<uint32_t*>(smem + C::nan_off) + (n & 1) * (D * 4); };

  TensorPiece p;
  if (role == 4) {
    // ======================================================== loader
    // lane g < 2 NB: 16 keys, half of block g / 2; pages are looked up two tiles and
    // scales one tile ahead
    uint32_t i = 0;  // tiles so far
    bool ok = true;
    while (walk.next(a, p, lane == 0, warp_sync)) {
      const int* table = a.table + (int64_t)p.seq * a.max_pages;
      const int page_mask = (1 << a.page_shift) - 1;
      const int p_first = p.len - a.s_q, p_last = p.len - 1;  // query positions
      auto key_of = [&](int t) { return p.span.block(t + (lane >> 1)) * 32 + (lane & 1) * 16; };
      auto in = [&](int t) { return lane < 2 * NB && t + (lane >> 1) < p.t1 && key_of(t) < p.span.hi; };
      auto look_up = [&](int t) { return in(t) ? table[key_of(t) >> a.page_shift] : -1; };
      auto valid = [&](int pid) { return pid >= 0 && pid < a.num_pages; };
      int pid0 = look_up(p.t0), pid1 = look_up(p.t0 + NB);
      int64_t at = (int64_t)(valid(pid0) ? pid0 : 0) * a.h_kv + p.kvh;
      float ks = a.k_scale[at], vs = a.v_scale[at];
      for (int t = p.t0; t < p.t1; t += NB, ++i) {
        const int slot = i % kStages;
        if (i >= kStages) ok = wait_on(&bars.free[slot], (i / kStages - 1) & 1, ctx);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const bool take = valid(pid0);
        const uint32_t taken = __ballot_sync(0xffffffffu, take);
        if (lane < 2 * NB) {
          const int key = key_of(t);
          s_ks[slot][lane] = take ? ks : 0.f;
          s_vs[slot][lane] = take ? vs : 0.f;
          s_ok[slot][lane] = take;
          if (!(lane & 1)) {
            const bool all = ((taken >> lane) & 3u) == 3u && key + 32 <= p.span.hi &&
                             (key >= p.span.lo || key + 32 <= p.span.sink_hi) && key + 31 <= p_first &&
                             (a.window < 0 || p_last - key <= a.window || key + 31 < a.sink);
            s_block[slot][lane >> 1] = make_int2(key, all);
          }
          if (take) {
            mbar_arrive_expect_tx(&bars.full[slot], 2 * 16 * D);
            const int y = key & page_mask;
            const uint32_t dst =
                smem_u32(smem + slot * C::kStage) + (lane >> 1) * 4096 + (lane & 1) * 16 * (D < 128 ? 64 : 128);
#pragma unroll
            for (int h = 0; h < (D + 127) / 128; ++h) {
              tma_load_4d(dst + h * C::kBlock64, &tm_k, h * 128, y, p.kvh, pid0, &bars.full[slot]);
              tma_load_4d(dst + C::kHalf + h * C::kBlock64, &tm_v, h * 128, y, p.kvh, pid0, &bars.full[slot]);
            }
          } else {
            mbar_arrive(&bars.full[slot]);
          }
        }
        at = (int64_t)(valid(pid1) ? pid1 : 0) * a.h_kv + p.kvh;
        ks = a.k_scale[at];
        vs = a.v_scale[at];
        pid0 = pid1;
        pid1 = look_up(t + 2 * NB);
      }
      if (!ok) break;
    }
    // every copy has landed before the CTA ends (so it has, unless a wait ran out)
    if (lane == 0)
      for (uint32_t j = i < kStages ? 0 : i - kStages; j < i; ++j)
        mbar_wait_drain(&bars.full[j % kStages], (j / kStages) & 1, nullptr);
  } else if (role == 3) {
    // ======================================================== products
    // S of a tile is issued one tile ahead of O: S(0), S(1), O(0), S(2), O(1), ..
    constexpr uint32_t idesc_s = idesc_f16_f32(128, kKeys, false, false);
    constexpr uint32_t idesc_o = idesc_f16_f32(128, D, false, true);
    const uint32_t lo = sdesc_lo(smem_u32(smem), 16), lo_v = sdesc_lo(smem_u32(smem + C::kHalf), C::kBlock64);
    uint32_t i = 0, n = 0;
    bool ok = true;
    while (ok && walk.next(a, p, lane == 0, warp_sync)) {
      const int tiles = (p.t1 - p.t0 + NB - 1) / NB;
      ok = wait_on(&bars.q_full, n & 1, ctx);
      auto scores = [&](uint32_t j) {
        const int slot = j % kStages;
        // its buffer holds P of two tiles before
        if (ok && j >= 2) ok = wait_on(&bars.o_done[j & 1], ((j >> 1) - 1) & 1, ctx);
        if (ok) ok = wait_on(&bars.k_full[slot], (j / kStages) & 1, ctx);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && lane == 0) {
          tc_fence_after();
          const uint32_t b = lo + ((slot * C::kStage) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ts_lo(tmem + C::col_s + (j & 1) * kKeys, tmem + kk * 8,
                      b + (((kk >> 2) * C::kBlock64 + (kk & 3) * 32) >> 4), idesc_s, kk > 0 ? 1u : 0u);
          mma_commit(&bars.s_full[j & 1]);
        }
        __syncwarp();
      };
      if (ok) scores(i);
      for (int u = 0; u < tiles && ok; ++u) {
        if (u + 1 < tiles) scores(i + u + 1);
        const uint32_t j = i + u;
        const int slot = j % kStages;
        if (ok) ok = wait_on(&bars.v_full[slot], (j / kStages) & 1, ctx);
        if (ok) ok = wait_on(&bars.p_full[j & 1], (j >> 1) & 1, ctx);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && lane == 0) {
          tc_fence_after();
          const uint32_t b = lo_v + ((slot * C::kStage) >> 4);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_ts_lo(tmem + C::col_o, tmem + C::col_s + (j & 1) * kKeys + kk * 8, b + ((kk * 2048) >> 4), idesc_o,
                      kk > 0 || u > 0 ? 1u : 0u);
          mma_commit(&bars.o_done[j & 1]);
          mma_commit(&bars.free[slot]);
        }
        __syncwarp();
      }
      i += tiles;
      ++n;
    }
    if (lane == 0) {
      mma_commit(&bars.drain);
      mbar_wait_drain(&bars.drain, 0, nullptr);
    }
  } else if (role < 2) {
    // ======================================================== widening
    const bool is_v = role == 1;
    const int wb = warp & 3;  // the block of the tile
    uint32_t i = 0, n = 0;    // tiles and pieces so far
    bool ok = true;
    while (walk.next(a, p, (threadIdx.x & 127) == 0, group_sync)) {
      if (is_v) {
        if (ok && n > 1) ok = wait_on(&bars.done[n & 1], ((n >> 1) - 1) & 1, ctx);
        if (a.s_q > 1)
          for (int u = threadIdx.x & 127; u < D * 4; u += 128) s_nan(n)[u] = 0u;
        if ((threadIdx.x & 127) == 0) s_any_nan[n & 1] = 0;
        group_sync();
      }
      if (wb < NB)
        for (int t = p.t0; t < p.t1; t += NB, ++i) {
          const int slot = i % kStages;
          if (ok) ok = wait_on(&bars.full[slot], (i / kStages) & 1, ctx);
          __syncwarp();
          uint8_t* base = smem + slot * C::kStage + (is_v ? C::kHalf : 0) + wb * 4096;
          uint32_t w[D / 4];
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint4 x = *reinterpret_cast<const uint4*>(base + code_offset<D>(lane, c));
            w[4 * c] = x.x;
            w[4 * c + 1] = x.y;
            w[4 * c + 2] = x.z;
            w[4 * c + 3] = x.w;
          }
          const int2 block = s_block[slot][wb];
          if (is_v && !block.y) {
            const int key = block.x + lane;
            const bool some = s_ok[slot][2 * wb + (lane >> 4)] && key < p.span.hi &&
                              (key >= p.span.lo || key < p.span.sink_hi);  // any query sees it
            if (a.s_q > 1 && some) {
              // a NaN that not every query sees (0 * NaN is NaN) is left out of the
              // product and noted for those that do
              uint32_t any = 0u;
#pragma unroll
              for (int j = 0; j < D / 4; ++j) any |= nan_bytes(w[j]);
              if (any) {
                s_any_nan[n & 1] = 1;
                const int rows = min(a.rows - p.rt * R, R);
#pragma unroll 1
                for (int r32 = 0; r32 < rows; r32 += 32) {
                  uint32_t mask = 0u;
#pragma unroll 1
                  for (int r = r32; r < min(rows, r32 + 32); ++r) {
                    const int q = p.len - a.s_q + (p.rt * R + r) / a.g;
                    if (key <= q && (a.window < 0 || q - key <= a.window || key < a.sink)) mask |= 1u << (r & 31);
                  }
#pragma unroll 1
                  for (int d = 0; d < D; ++d)
                    if ((base[code_offset<D>(lane, d >> 4) + (d & 15)] & 0x7f) == 0x7f)
                      atomicOr(s_nan(n) + d * 4 + (r32 >> 5), mask);
                }
              }
#pragma unroll
              for (int j = 0; j < D / 4; ++j) w[j] &= ~nan_bytes(w[j]);
            }
            if (!some) {
#pragma unroll
              for (int j = 0; j < D / 4; ++j) w[j] = 0u;
            }
          }
          __syncwarp();
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {  // 8 d's
            uint4 f;
            f.x = widen_lo(w[2 * c]);
            f.y = widen_hi(w[2 * c]);
            f.z = widen_lo(w[2 * c + 1]);
            f.w = widen_hi(w[2 * c + 1]);
            *reinterpret_cast<uint4*>(base + (c >> 3) * C::kBlock64 + lane * 128 + (((c ^ lane) & 7) << 4)) = f;
          }
          fence_proxy_async_smem();
          mbar_arrive(is_v ? &bars.v_full[slot] : &bars.k_full[slot]);
        }
      if (is_v) mbar_arrive(&bars.widened[n & 1]);
      ++n;
    }
  } else {
    // ======================================================== softmax
    const int wq = warp & 3, r = threadIdx.x & 127;  // the row of this thread
    const uint32_t my_tmem = tmem + ((uint32_t)(wq * 32) << 16), t_o = my_tmem + C::col_o;
    uint32_t i = 0, n = 0;
    bool ok = true;
    while (walk.next(a, p, r == 0, group_sync)) {
      const int row = p.rt * R + r;
      const bool mine = row < a.rows;
      const bool busy = p.rt * R + wq * 32 < a.rows;  // this warp has rows
      const int tok = mine ? row / a.g : 0, head = p.kvh * a.g + (mine ? row - tok * a.g : 0);
      const int64_t orow = ((int64_t)p.seq * a.s_q + tok) * a.h_q + head;
      const int pos = mine ? p.len - a.s_q + tok : -1;
      // ---- q's row as f16, the largest value in [2^14, 2^15)
      float fac;
      {
        const uint4* src = reinterpret_cast<const uint4*>(a.q + orow * D);
        float amax = 0.f;
#pragma unroll 8
        for (int c = 0; c < D / 8; ++c) {
          const uint4 x = mine ? src[c] : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x0 = fabsf(__uint_as_float(w[j] << 16)), x1 = fabsf(__uint_as_float(w[j] & 0xffff0000u));
            if (x0 < INFINITY) amax = fmaxf(amax, x0);
            if (x1 < INFINITY) amax = fmaxf(amax, x1);
          }
        }
        const uint32_t bits = __float_as_uint(amax);
        const int ex = bits ? max((int)(bits >> 23) - 127, -100) - 14 : 0;
        const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
        fac = mine ? a.scale_log2 * __uint_as_float((uint32_t)(127 + ex) << 23) : 0.f;
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 16) {
          uint32_t f[16];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint4 x = mine ? src[c / 4 + u] : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              f[4 * u + j] =
                  pack_f16(__uint_as_float(w[j] << 16) * inv, __uint_as_float(w[j] & 0xffff0000u) * inv);
          }
          tmem_st16(my_tmem + c, f);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars.q_full);
      }
      // the references of P and of P * v_scale (negated; at first below every score),
      // 2^(m - mo + kShift), the sum of P
      float nm = FLT_MAX, nmo = FLT_MAX, b = 1.f, l = 0.f;

#pragma unroll 1
      for (int t = p.t0; t < p.t1; t += NB, ++i) {
        const int slot = i % kStages;
        const bool first = t == p.t0;
        const uint32_t t_s = my_tmem + C::col_s + (i & 1) * kKeys;
        if (ok) ok = wait_on(&bars.full[slot], (i / kStages) & 1, ctx);
        if (ok) ok = wait_on(&bars.s_full[i & 1], (i >> 1) & 1, ctx);
        __syncwarp();
        tc_fence_after();
        if (busy) {
          bool all_seen = true;
#pragma unroll
          for (int c = 0; c < NB; ++c) all_seen = all_seen && s_block[slot][c].y;
          auto sees = [&](int c, int j) {  // key j of block c
            const int key = s_block[slot][c].x + j;
            return s_ok[slot][2 * c + (j >> 4)] && key < p.span.hi && key <= pos &&
                   (a.window < 0 || pos - key <= a.window || key < a.sink);
          };
          uint32_t pk[kKeys / 2];
          float sum;
#pragma unroll 1
          for (bool again = false;; again = true) {
            float top = 0.f, top_o = 0.f, part[8] = {};
#pragma unroll
            for (int c = 0; c < NB; ++c) {
              float e[32];
              tmem_ld32(t_s + 32 * c, reinterpret_cast<uint32_t*>(e));
              const float2 ks = *reinterpret_cast<const float2*>(&s_ks[slot][2 * c]);
              const float2 vs = *reinterpret_cast<const float2*>(&s_vs[slot][2 * c]);
              const float f[2] = {fac * ks.x, fac * ks.y}, v[2] = {vs.x * b, vs.y * b};
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; j += 2)
                fma_f32x2(e[j], e[j + 1], e[j], e[j + 1], f[j >> 4], f[j >> 4], nm, nm);
              if (!all_seen) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (!sees(c, j)) e[j] = -INFINITY;
              }
#pragma unroll
              for (int j = 0; j < 32; ++j) e[j] = ex2(e[j]);
              // (maxima and sums in several chains: one warp per scheduler has nothing
              // else to fill their latency)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float m[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float* x = e + 16 * h + 4 * j;
                  m[j] = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                }
                const float most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
                top = fmaxf(top, most);
                top_o = fmaxf(top_o, most * v[h]);
              }
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                add_f32x2(part[j & 6], part[(j & 6) + 1], part[j & 6], part[(j & 6) + 1], e[j], e[j + 1]);
                mul_f32x2(e[j], e[j + 1], e[j], e[j + 1], v[j >> 4], v[j >> 4]);
                pk[16 * c + j / 2] = pack_f16(e[j], e[j + 1]);
              }
            }
            sum = ((part[0] + part[1]) + (part[2] + part[3])) + ((part[4] + part[5]) + (part[6] + part[7]));
            if (again || !__any_sync(0xffffffffu, top > 256.f || top_o > 32768.f)) break;

            // raise the references where a score passed them, to the tile's largest
            float x = -INFINITY, xo = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < NB; ++c) {
              float e[32];
              tmem_ld32(t_s + 32 * c, reinterpret_cast<uint32_t*>(e));
              tmem_wait_ld();
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float f = fac * s_ks[slot][2 * c + h], lv = lg2(s_vs[slot][2 * c + h]);
                float y = -INFINITY;
#pragma unroll
                for (int j = 16 * h; j < 16 * h + 16; ++j)
                  y = fmaxf(y, all_seen || sees(c, j) ? e[j] * f : -INFINITY);
                x = fmaxf(x, y);
                xo = fmaxf(xo, y + lv);
              }
            }
            const float nm1 = x + nm > 0.f ? -x : nm;
            // b stays a normal number (x <= m + 8 and lg2(v_scale) < 128, so x + lg2(v_scale)
            // passes mo <= m + 130 by no more than 6)
            const float nmo1 = fminf(fmaxf(xo + nmo > 0.f ? -xo : nmo, nm1 - 130.f), nm1 + 119.f);
            const float fo = ex2(nmo1 - nmo);
            l *= ex2(nm1 - nm);
            nm = nm1;
            nmo = nmo1;
            b = ex2(nmo1 - nm1 + kShift);
            if (!first) {
              if (ok) ok = wait_on(&bars.o_done[(i - 1) & 1], ((i - 1) >> 1) & 1, ctx);
              __syncwarp();
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_ld32(t_o + c, reinterpret_cast<uint32_t*>(o));
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] *= fo;
                tmem_st32(t_o + c, reinterpret_cast<const uint32_t*>(o));
              }
            }
          }
          l += sum;
#pragma unroll
          for (int c = 0; c < NB; ++c) tmem_st16(t_s + 16 * c, pk + 16 * c);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&bars.p_full[i & 1]);
      }
      if (ok) ok = wait_on(&bars.o_done[(i - 1) & 1], ((i - 1) >> 1) & 1, ctx);
      if (ok) ok = wait_on(&bars.widened[n & 1], (n >> 1) & 1, ctx);
      __syncwarp();
      tc_fence_after();

      // ---- the row's result; a piece that starts inside its item is the first of
      // this CTA, one that ends inside it the last: one slot each
      if (busy) {
        const int64_t part = 2 * (int64_t)blockIdx.x + (p.t0 == 0 ? 1 : 0);
        const float bad = __int_as_float(0x7fffffff);  // a wait ran out: no result
        const float inv = !ok ? bad : l == 0.f ? 0.f : ex2(nm - nmo - kShift) / l;
        const float lse2 = !ok ? bad : l == 0.f ? -INFINITY : log2f(l) - nm;
        if (mine) {
          if (p.whole)
            a.lse[((int64_t)p.seq * a.h_q + head) * a.s_q + tok] = lse2 * kLn2;
          else
            a.part_lse[part * R + r] = lse2;
        }
        const bool nans = s_any_nan[n & 1];
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(t_o + c, reinterpret_cast<uint32_t*>(o));
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] *= inv;
          if (nans) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if ((s_nan(n)[(c + j) * 4 + wq] >> lane) & 1u) o[j] = bad;
          }
          if (!mine) continue;
          if (p.whole && !a.out_fp32) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + orow * D + c);
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              dst[j / 8] = make_uint4(pack_bf16(o[j], o[j + 1]), pack_bf16(o[j + 2], o[j + 3]),
                                      pack_bf16(o[j + 4], o[j + 5]), pack_bf16(o[j + 6], o[j + 7]));
          } else {
            float4* dst = reinterpret_cast<float4*>(p.whole ? static_cast<float*>(a.out) + orow * D + c
                                                            : a.part_o + (part * R + r) * D + c);
#pragma unroll
            for (int j = 0; j < 32; j += 4) dst[j / 4] = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&bars.done[n & 1]);
      ++n;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}
