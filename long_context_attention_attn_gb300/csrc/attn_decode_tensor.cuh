// The kernel for more rows than the warp-level one is good for (drafted tokens
// times a large group): 64 or 128 rows per CTA on the tensor-memory path, included
// by attn_decode.cu.
//
//   S[rows, keys] = q K^T,  O[rows, d] += P V   (f16 in, fp32 sums)
//
// One CTA per SM, its warps by role:
//   loader    copies the codes of 16 keys at a time (TMA, swizzled) into a ring
//   widening  a thread per key, one group of warps for K and one for V: the codes,
//             exactly, into f16 rows of 64 d's; the V warps also q's rows, as f16
//             into tensor memory, once a piece
//   products  a thread for S, a thread for O
//   softmax   4 warps, a thread per row: scores out of tensor memory, P (f16) back
//             into it
// The products have 128 rows.  With 64 the rows are there twice, and each copy takes
// half of a tile's keys (the other half of its P is zero), with references, sums and
// an O of its own, put together at a piece's end: the softmax of a tile then takes a
// warp half the time.
//
// Every wait ends: after a second it gives up and so do the CTA's others.  A thread that
// gave up writes nothing that others read and arrives nowhere any more, so a softmax
// thread that got through a piece has a right result, and the others' are NaN.
//
// HBM would take 1410 cycles per 128 keys at d = 128.  The softmax takes 2900 with
// 128 rows and 1500 with 64 (one warp per scheduler, so latencies count), a thread's
// eight products and their commit 700 to 800, the widening 1200; what a piece costs
// besides its tiles is 8 us.  Instruction fetch is felt everywhere (no-instruction
// stalls 1.6 per issue, six loops at once), so what is rarely run is rolled.  Tried,
// d 128, us of 48 sequences of 100 to 12000 tokens, Hkv 8, at 64 / 128 rows (this
// one 221 / 303 at that time, 232 / 300 now): scales looked up tile by tile 247 /
// 321; P over S, codes widened in place 317 / 305; keys on the M side (a thread per
// key, votes over threads) 273 / 495.
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

// 32 lanes x 32 bit, 16 or 8 consecutive columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// mbar_wait, asleep once before the clock is read.
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, const WaitCtx& ctx) {
  if (mbar_try_wait_sleep(smem_u32(bar), parity, kSleepHintNs)) return true;
  if (*ctx.abort_flag) return false;
  return mbar_wait(bar, parity, ctx);
}

template <int D, int NT>
struct TensorCfg {
  using T = Tune<D, NT>;
  static constexpr int R = NT * 8;
  static constexpr int kCopies = 128 / R;  // of each row
  static constexpr int kThreads = 32 * 15;  // K 4, V 4, softmax 4, S, loader, O
  static constexpr int kKeys = D == 256 ? 64 : 128;  // per tile
  static constexpr int kBlocks = kKeys / 32;
  // Shared memory: tiles of codes as they come (K, then V; 128 bytes of a key after
  // another's), K and V in f16 (64 d's after another, a key's 128 bytes after
  // another's) for one or two products.
  static constexpr int kStages = T::kStages, kKBufs = D == 64 ? 2 : 1, kVBufs = 2;
  static constexpr int kCodes = kKeys * D;            // of K (V)
  static constexpr int kBlock64 = kKeys * 128;
  static constexpr int kHalf = D / 64 * kBlock64;     // K (V) in f16
  static constexpr int k_off = kStages * 2 * kCodes, v_off = k_off + kKBufs * kHalf;
  // Scales and the like of a tile are kept until its S has been read.  The loader
  // fills tile i once K of i - kStages has been read, after K of the tile before that
  // was stored, whose S needs the buffer of the one two (or a K buffer) before.
  static constexpr int kMeta = 16;
  static_assert(kStages + kKBufs + 3 <= kMeta, "tiles under way");
  static constexpr int nan_off = v_off + kVBufs * kHalf;  // of two pieces: [D][4] bits: rows that see a NaN of V
  static constexpr int row_off = nan_off + 2 * D * 16;        // output rows: int64 [R]
  static constexpr int sum_off = row_off + R * 8;             // copies' results, 32 d's at a time: [128][33]
  static constexpr int bytes = sum_off + (kCopies > 1 ? 128 * 33 * 4 : 0) + 1024;  // (and up to 1023 to align)
  // tensor memory: q [rows][D / 2], S [rows][kKeys] twice, P [rows][kKeys / 2] as often
  // as there is room (else in the first half of S), O [rows][D]
  static constexpr int kPBufs = D == 64 ? 2 : D == 128 ? 1 : 0;
  static constexpr uint32_t col_s = D / 2, col_p = col_s + 2 * kKeys, col_o = col_p + kPBufs * kKeys / 2;
  static constexpr uint32_t kCols = 512;
  static_assert(R == 64 || R == 128, "rows");
  static_assert(col_o + D <= kCols, "tensor memory");
  static_assert(bytes <= 232448 - 4096, "shared memory");
};

// Where 16-byte piece c of key `row` of a tile's codes lies (the copy's 64-byte or
// 128-byte swizzle).
template <int D>
__device__ __forceinline__ int code_offset(int row, int c) {
  if constexpr (D == 64)
    return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
  else
    return (c >> 3) * ((D == 256 ? 64 : 128) * 128) + row * 128 + (((c ^ row) & 7) << 4);
}

// The column of tile i's P.
template <typename C>
__device__ __forceinline__ uint32_t p_col(uint32_t i) {
  if constexpr (C::kPBufs > 0)
    return C::col_p + i % C::kPBufs * (C::kKeys / 2);
  else
    return C::col_s + (i & 1) * C::kKeys;
}

template <int D, int NT>
__global__ void __launch_bounds__(TensorCfg<D, NT>::kThreads, 1)
attn_decode_tensor_kernel(const DecodeArgs a, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v) {
  using C = TensorCfg<D, NT>;
  using T = typename C::T;
  constexpr int R = C::R, kStages = C::kStages, NB = C::kBlocks, kKeys = C::kKeys;
  extern __shared__ uint8_t smem_raw[];
  struct Bars {
    uint64_t full[kStages];        // a tile's codes are there
    uint64_t free[kStages];        // they have been read
    uint64_t k_full[C::kKBufs];    // its K is there in f16
    uint64_t v_full[C::kVBufs];    // its V is
    uint64_t meta_full[2];         // its scales are
    uint64_t q_full[2];        // of a piece: q is in tensor memory
    uint64_t s_full[2];        // S is there
    uint64_t s_free[2];        // S has been read
    uint64_t p_full[2];        // P is in its place
    uint64_t o_done[2];        // O has it
    uint64_t widened[2], done[2];  // of a piece: V, everything
    uint64_t drain[2];
  };
  __shared__ Bars bars;
  __shared__ TensorWalk<T> walks[6];
  __shared__ int64_t before[kThreads + 1];
  // of a tile's groups of 16 keys: scales and whether they have a page; of its
  // blocks: the first key and whether every query sees all of them
  __shared__ float s_ks[C::kMeta][2 * NB], s_vs[C::kMeta][2 * NB];
  __shared__ uint8_t s_ok[C::kMeta][2 * NB];
  __shared__ int2 s_block[C::kMeta][NB];
  __shared__ float s_end[C::kCopies][2][R];  // references and sums
  __shared__ float s_fac[2][128];  // of two pieces: what the scores of q's f16 rows are multiplied by
  __shared__ int s_any_nan[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.full[i], 2 * NB);
      mbar_init(&bars.free[i], 2 * kKeys);
    }
    for (int i = 0; i < C::kKBufs; ++i) mbar_init(&bars.k_full[i], kKeys);
    for (int i = 0; i < C::kVBufs; ++i) mbar_init(&bars.v_full[i], kKeys);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.meta_full[i], 1);
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.s_free[i], 128);
      mbar_init(&bars.q_full[i], 128);
      mbar_init(&bars.p_full[i], 128);
      mbar_init(&bars.o_done[i], 1);
      mbar_init(&bars.widened[i], 128);
      mbar_init(&bars.done[i], 128);
    }
    mbar_init(&bars.drain[0], 1);
    mbar_init(&bars.drain[1], 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, C::kCols);
    tmem_relinquish();
  }
  const Placement pl = place<T>(a, before);
  // roles: 0 K, 1 V, 2 softmax, 3 S, 4 loader, 5 O
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
    // 16 blocks of keys at a time, a lane per group of 16 keys: their pages are looked
    // up two turns and their scales one turn ahead (a turn per tile would wait for
    // memory in each)
    constexpr int kTurn = 16, kLanes = 2 * NB;  // blocks per turn, lanes per tile
    uint32_t i = 0;  // tiles so far
    bool ok = true;
    while (!a.withhold && walk.next(a, p, lane == 0, warp_sync)) {
      const int* table = a.table + (int64_t)p.seq * a.max_pages;
      const int page_mask = (1 << a.page_shift) - 1;
      const int p_first = p.len - a.s_q, p_last = p.len - 1;  // query positions
      auto key_of = [&](int t) { return p.span.block(t + (lane >> 1)) * 32 + (lane & 1) * 16; };
      auto look_up = [&](int t) {
        return t + (lane >> 1) < p.t1 && key_of(t) < p.span.hi ? table[key_of(t) >> a.page_shift] : -1;
      };
      auto valid = [&](int pid) { return pid >= 0 && pid < a.num_pages; };
      auto scale_at = [&](int pid) { return (int64_t)(valid(pid) ? pid : 0) * a.h_kv + p.kvh; };
      int pid0 = look_up(p.t0), pid1 = look_up(p.t0 + kTurn);
      float ks = a.k_scale[scale_at(pid0)], vs = a.v_scale[scale_at(pid0)];
      for (int t = p.t0; t < p.t1 && ok; t += kTurn) {
        const float ks1 = a.k_scale[scale_at(pid1)], vs1 = a.v_scale[scale_at(pid1)];
        const int pid2 = look_up(t + 2 * kTurn);
        const int key = key_of(t);
        const bool take = valid(pid0);
        const bool both = ((__ballot_sync(0xffffffffu, take) >> (lane & 30)) & 3u) == 3u;
        const bool all = both && key + 32 <= p.span.hi && (key >= p.span.lo || key + 32 <= p.span.sink_hi) &&
                         key + 31 <= p_first && (a.window < 0 || p_last - key <= a.window || key + 31 < a.sink);
        for (int u = 0; u < kTurn && t + u < p.t1; u += NB, ++i) {
          const int slot = i % kStages;
          if (i >= kStages) ok = wait_on(&bars.free[slot], (i / kStages - 1) & 1, ctx);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const int g = lane - 2 * u;  // this lane's group of the tile
          if (g >= 0 && g < kLanes) {
            const int m = i % C::kMeta;
            s_ks[m][g] = take ? ks : 0.f;
            s_vs[m][g] = take ? vs : 0.f;
            s_ok[m][g] = take;
            if (!(g & 1)) s_block[m][g >> 1] = make_int2(key, all);
            if (take) {
              mbar_arrive_expect_tx(&bars.full[slot], 2 * 16 * D);
              const int y = key & page_mask;
              const uint32_t dst = smem_u32(smem + slot * 2 * C::kCodes) + g * 16 * (D < 128 ? 64 : 128);
#pragma unroll
              for (int h = 0; h < (D + 127) / 128; ++h) {
                tma_load_4d(dst + h * C::kBlock64, &tm_k, h * 128, y, p.kvh, pid0, &bars.full[slot]);
                tma_load_4d(dst + C::kCodes + h * C::kBlock64, &tm_v, h * 128, y, p.kvh, pid0, &bars.full[slot]);
              }
            } else {
              mbar_arrive(&bars.full[slot]);
            }
          }
        }
        pid0 = pid1;
        pid1 = pid2;
        ks = ks1;
        vs = vs1;
      }
      if (!ok) break;
    }
    // every copy has landed before the CTA ends (so it has, unless a wait ran out)
    if (lane == 0)
      for (uint32_t j = i < kStages ? 0 : i - kStages; j < i; ++j)
        mbar_wait_drain(&bars.full[j % kStages], (j / kStages) & 1, nullptr);
  } else if (role == 3) {
    // ======================================================== S = q K^T
    constexpr uint32_t idesc = idesc_f16_f32(128, kKeys, false, false);
    const uint32_t lo = sdesc_lo(smem_u32(smem + C::k_off), 16);
    uint32_t i = 0, n = 0;
    bool ok = true;
    while (ok && walk.next(a, p, lane == 0, warp_sync)) {
      ok = __all_sync(0xffffffffu, wait_on(&bars.q_full[n & 1], (n >> 1) & 1, ctx));
      for (int t = p.t0; t < p.t1 && ok; t += NB, ++i) {
        const int buf = i % C::kKBufs;
        // its buffer holds S (or P) of two tiles before
        if (ok && i >= 2)
          ok = wait_on(C::kPBufs > 0 ? &bars.s_free[i & 1] : &bars.o_done[i & 1], ((i >> 1) - 1) & 1, ctx);
        if (ok) ok = wait_on(&bars.k_full[buf], (i / C::kKBufs) & 1, ctx);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && lane == 0) {
          tc_fence_after();
          mbar_arrive(&bars.meta_full[i & 1]);
          const uint32_t b = lo + ((buf * C::kHalf) >> 4), d_s = tmem + C::col_s + (i & 1) * kKeys;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ts_lo(d_s, tmem + kk * 8, b + (((kk >> 2) * C::kBlock64 + (kk & 3) * 32) >> 4), idesc,
                      kk > 0 ? 1u : 0u);
          mma_commit(&bars.s_full[i & 1]);
        }
        __syncwarp();
      }
      ++n;
    }
    if (lane == 0) {
      mma_commit(&bars.drain[0]);
      mbar_wait_drain(&bars.drain[0], 0, nullptr);
    }
  } else if (role == 5) {
    // ======================================================== O += P V
    constexpr uint32_t idesc = idesc_f16_f32(128, D, false, true);
    const uint32_t lo = sdesc_lo(smem_u32(smem + C::v_off), C::kBlock64);
    uint32_t i = 0;
    bool ok = true;
    while (ok && walk.next(a, p, lane == 0, warp_sync)) {
      for (int t = p.t0; t < p.t1 && ok; t += NB, ++i) {
        const int buf = i % C::kVBufs;
        ok = wait_on(&bars.v_full[buf], (i / C::kVBufs) & 1, ctx);
        if (ok) ok = wait_on(&bars.p_full[i & 1], (i >> 1) & 1, ctx);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && lane == 0) {
          tc_fence_after();
          const uint32_t b = lo + ((buf * C::kHalf) >> 4), p16 = tmem + p_col<C>(i);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_ts_lo(tmem + C::col_o, p16 + kk * 8, b + ((kk * 2048) >> 4), idesc, kk > 0 || t > p.t0 ? 1u : 0u);
          mma_commit(&bars.o_done[i & 1]);
        }
        __syncwarp();
      }
    }
    if (lane == 0) {
      mma_commit(&bars.drain[1]);
      mbar_wait_drain(&bars.drain[1], 0, nullptr);
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
        if (ok && a.s_q > 1)
          for (int u = threadIdx.x & 127; u < D * 4; u += 128) s_nan(n)[u] = 0u;
        if (ok && (threadIdx.x & 127) == 0) s_any_nan[n & 1] = 0;
        group_sync();
        // ---- q's rows (a thread per row and copy) as f16, the largest value in [2^14,
        // 2^15), after the last S with the rows before them
        if (ok && i > 0) ok = wait_on(&bars.s_full[(i - 1) & 1], ((i - 1) >> 1) & 1, ctx);
        ok = __all_sync(0xffffffffu, ok);
      }
      if (is_v && ok) {
        tc_fence_after();
        const int th = threadIdx.x & 127, row = p.rt * R + th % R;
        const bool mine = row < a.rows;
        const int tok = mine ? row / a.g : 0, head = p.kvh * a.g + (mine ? row - tok * a.g : 0);
        const int64_t orow = ((int64_t)p.seq * a.s_q + tok) * a.h_q + head;
        const uint32_t my_tmem = tmem + ((uint32_t)((warp & 3) * 32) << 16);
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
        s_fac[n & 1][th] = mine ? a.scale_log2 * __uint_as_float((uint32_t)(127 + ex) << 23) : 0.f;
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
        mbar_arrive(&bars.q_full[n & 1]);
      }
      for (int t = p.t0; t < p.t1; t += NB, ++i) {
        if (wb >= NB) continue;
        const int slot = i % kStages;
        if (ok) ok = wait_on(&bars.full[slot], (i / kStages) & 1, ctx);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        const uint8_t* base = smem + slot * 2 * C::kCodes + (is_v ? C::kCodes : 0);
        const int k = wb * 32 + lane, m = i % C::kMeta;  // this thread's key of the tile
        uint32_t w[D / 4];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(base + code_offset<D>(k, c));
          w[4 * c] = x.x;
          w[4 * c + 1] = x.y;
          w[4 * c + 2] = x.z;
          w[4 * c + 3] = x.w;
        }
        const int2 block = s_block[m][wb];
        if (is_v && !block.y) {
          const int key = block.x + lane;
          const bool some = s_ok[m][2 * wb + (lane >> 4)] && key < p.span.hi &&
                            (key >= p.span.lo || key < p.span.sink_hi);  // any query sees it
          if (a.s_q > 1 && some) {
            // a NaN that not every query sees (0 * NaN is NaN) is left out of the
            // product and noted for those that do
            uint32_t any = 0u;
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              const uint4 x = *reinterpret_cast<const uint4*>(base + code_offset<D>(k, c));
              any |= nan_bytes(x.x) | nan_bytes(x.y) | nan_bytes(x.z) | nan_bytes(x.w);
            }
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
                  if ((base[code_offset<D>(k, d >> 4) + (d & 15)] & 0x7f) == 0x7f)
                    atomicOr(s_nan(n) + d * 4 + (r32 >> 5), mask);
              }
#pragma unroll
              for (int j = 0; j < D / 4; ++j) w[j] &= ~nan_bytes(w[j]);
            }
          }
          if (!some) {
#pragma unroll
            for (int j = 0; j < D / 4; ++j) w[j] = 0u;
          }
        }
        mbar_arrive(&bars.free[slot]);
        // the f16 tile that was there has been multiplied
        if (is_v) {
          if (i >= C::kVBufs) ok = wait_on(&bars.o_done[i & 1], ((i >> 1) - 1) & 1, ctx);
        } else if (i >= C::kKBufs) {
          const uint32_t j = i - C::kKBufs;
          ok = wait_on(&bars.s_full[j & 1], (j >> 1) & 1, ctx);
        }
        if (!ok) continue;
        uint8_t* dst = smem + (is_v ? C::v_off + i % C::kVBufs * C::kHalf : C::k_off + i % C::kKBufs * C::kHalf);
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
        mbar_arrive(is_v ? &bars.v_full[i % C::kVBufs] : &bars.k_full[i % C::kKBufs]);
      }
      if (is_v && ok) mbar_arrive(&bars.widened[n & 1]);
      ++n;
    }
  } else {
    // ======================================================== softmax
    constexpr int W = kKeys / C::kCopies, CH = 32;  // this thread's keys of a tile, in chunks
    const int wq = warp & 3, th = threadIdx.x & 127;
    const int r = th % R, copy = th / R;  // the row of this thread, and which copy of it
    const int col0 = copy * W;
    const uint32_t my_tmem = tmem + ((uint32_t)(wq * 32) << 16), t_o = my_tmem + C::col_o;
    if constexpr (C::kCopies > 1 && C::kPBufs > 0) {
      // (what this thread's copy does not write stays zero)
      const uint32_t zero[8] = {};
      for (int c = 0; c < C::kPBufs * kKeys / 2; c += 8) tmem_st8(my_tmem + C::col_p + c, zero);
      tmem_wait_st();
    }
    uint32_t i = 0, n = 0;
    bool ok = true;
    while (walk.next(a, p, th == 0, group_sync)) {
      const int row = p.rt * R + r;
      const bool mine = row < a.rows;
      const bool busy = p.rt * R + (wq * 32) % R < a.rows;  // this warp has rows
      const int tok = mine ? row / a.g : 0, head = p.kvh * a.g + (mine ? row - tok * a.g : 0);
      const int64_t orow = ((int64_t)p.seq * a.s_q + tok) * a.h_q + head;
      const int pos = mine ? p.len - a.s_q + tok : -1;
      if (ok) ok = wait_on(&bars.q_full[n & 1], (n >> 1) & 1, ctx);
      const float fac = s_fac[n & 1][th];
      // the references of P and of P * v_scale (negated; at first below every score),
      // 2^(m - mo + kShift), the sum of P
      float nm = FLT_MAX, nmo = FLT_MAX, b = 1.f, l = 0.f;

#pragma unroll 1
      for (int t = p.t0; t < p.t1; t += NB, ++i) {
        const int m = i % C::kMeta;
        const bool first = t == p.t0;
        const uint32_t t_s = my_tmem + C::col_s + (i & 1) * kKeys;
        if (ok) ok = wait_on(&bars.meta_full[i & 1], (i >> 1) & 1, ctx);
        if (ok) ok = wait_on(&bars.s_full[i & 1], (i >> 1) & 1, ctx);
        __syncwarp();
        tc_fence_after();
        uint32_t pk[W / 2];
        if (busy) {
          bool all_seen = true;
#pragma unroll
          for (int c = 0; c < W / 32; ++c) all_seen = all_seen && s_block[m][col0 / 32 + c].y;
          auto sees = [&](int j) {  // key j of the tile
            const int key = s_block[m][j >> 5].x + (j & 31);
            return s_ok[m][j >> 4] && key < p.span.hi && key <= pos &&
                   (a.window < 0 || pos - key <= a.window || key < a.sink);
          };
          float sum;
#pragma unroll 1
          for (bool again = false;; again = true) {
            float top = 0.f, top_o = 0.f, part[8] = {};
#pragma unroll
            for (int c = 0; c < W; c += CH) {
              float e[CH];
              tmem_ld32(t_s + col0 + c, reinterpret_cast<uint32_t*>(e));
              // (b * v_scale may pass fp32's range, where keys are out of sight or of next to
              // no weight: infinite it still tells below that a weight calls for a raise, but
              // 0 * infinity is NaN, so P takes the largest finite value)
              float f[CH / 16], v[CH / 16], v_all[CH / 16];
#pragma unroll
              for (int h = 0; h < CH / 16; ++h) {
                f[h] = fac * s_ks[m][(col0 + c) / 16 + h];
                v_all[h] = b * s_vs[m][(col0 + c) / 16 + h];
                v[h] = fminf(v_all[h], FLT_MAX);
              }
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < CH; j += 2)
                fma_f32x2(e[j], e[j + 1], e[j], e[j + 1], f[j >> 4], f[j >> 4], nm, nm);
              if (!all_seen) {
#pragma unroll
                for (int j = 0; j < CH; ++j)
                  if (!sees(col0 + c + j)) e[j] = -INFINITY;
              }
#pragma unroll
              for (int j = 0; j < CH; ++j) e[j] = ex2(e[j]);
              // (maxima and sums in several chains: one warp per scheduler has nothing
              // else to fill their latency)
#pragma unroll
              for (int h = 0; h < CH / 16; ++h) {
                float y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float* x = e + 16 * h + 4 * j;
                  y[j] = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                }
                const float most = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
                top = fmaxf(top, most);
                top_o = fmaxf(top_o, most * v_all[h]);  // (0 * infinity counts as nothing)
              }
#pragma unroll
              for (int j = 0; j < CH; j += 2) {
                add_f32x2(part[j & 6], part[(j & 6) + 1], part[j & 6], part[(j & 6) + 1], e[j], e[j + 1]);
                mul_f32x2(e[j], e[j + 1], e[j], e[j + 1], v[j >> 4], v[j >> 4]);
                pk[(c + j) / 2] = pack_f16(e[j], e[j + 1]);
              }
            }
            sum = ((part[0] + part[1]) + (part[2] + part[3])) + ((part[4] + part[5]) + (part[6] + part[7]));
            if (again || !__any_sync(0xffffffffu, top > 256.f || top_o > 32768.f)) break;

            // raise the references where a score passed them, to the tile's largest
            float x = -INFINITY, xo = -INFINITY;
#pragma unroll 1
            for (int c = col0; c < col0 + W; c += 16) {
              float e[16];
              tmem_ld16(t_s + c, reinterpret_cast<uint32_t*>(e));
              tmem_wait_ld();
              const float f = fac * s_ks[m][c / 16], lv = lg2(s_vs[m][c / 16]);
              float y = -INFINITY;
#pragma unroll
              for (int j = 0; j < 16; ++j) y = fmaxf(y, all_seen || sees(c + j) ? e[j] * f : -INFINITY);
              x = fmaxf(x, y);
              xo = fmaxf(xo, y + lv);
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
        }
        if constexpr (C::kPBufs > 0) {
          tc_fence_before();
          if (ok) mbar_arrive(&bars.s_free[i & 1]);
          // P's place is free after its last O
          if (ok && i >= C::kPBufs) {
            const uint32_t j = i - C::kPBufs;
            ok = wait_on(&bars.o_done[j & 1], (j >> 1) & 1, ctx);
          }
          __syncwarp();
        }
        if (busy) {
          // P of this copy's keys; zeros for the others, where S was
          const uint32_t t_p = my_tmem + p_col<C>(i);
          if constexpr (C::kCopies > 1 && C::kPBufs == 0) {
            const uint32_t zero[8] = {};
#pragma unroll
            for (int g = 0; g < kKeys / 16; ++g)
              if (g < col0 / 16 || g >= (col0 + W) / 16) tmem_st8(t_p + 8 * g, zero);
          }
#pragma unroll
          for (int g = 0; g < W / 16; ++g) tmem_st8(t_p + col0 / 2 + 8 * g, pk + 8 * g);
          tmem_wait_st();
        }
        tc_fence_before();
        if (ok) mbar_arrive(&bars.p_full[i & 1]);
      }
      if (ok) ok = wait_on(&bars.o_done[(i - 1) & 1], ((i - 1) >> 1) & 1, ctx);
      if (ok) ok = wait_on(&bars.widened[n & 1], (n >> 1) & 1, ctx);
      __syncwarp();
      tc_fence_after();

      // ---- the row's result; a piece that starts inside its item is the first of
      // this CTA, one that ends inside it the last: one slot each
      const int64_t part = 2 * (int64_t)blockIdx.x + (p.t0 == 0 ? 1 : 0);
      const float bad = __int_as_float(0x7fffffff);  // (a wait that ran out: no result)
      if (!ok) l = bad;
      float ref = -nm, z = l;
      if constexpr (C::kCopies > 1) {
        s_end[copy][0][r] = nm;
        s_end[copy][1][r] = l;
        if (copy == 0) reinterpret_cast<int64_t*>(smem + C::row_off)[r] = orow;
        group_sync();
#pragma unroll
        for (int c = 0; c < C::kCopies; ++c) ref = fmaxf(ref, -s_end[c][0][r]);
        z = 0.f;
#pragma unroll
        for (int c = 0; c < C::kCopies; ++c) z += s_end[c][1][r] * ex2(-s_end[c][0][r] - ref);
      }
      // of this copy's O: 2^(mo - ref) / z, as w * w2 (for small V alone the product is
      // below fp32's normal numbers)
      const float w2 = ex2(0.5f * (-nmo - ref - kShift));
      const float w = (z == 0.f ? 0.f : 1.f / z) * w2;
      const float lse2 = z == 0.f ? -INFINITY : ref + log2f(z);
      if (mine && copy == 0) {
        if (p.whole)
          a.lse[((int64_t)p.seq * a.h_q + head) * a.s_q + tok] = lse2 * kLn2;
        else
          a.part_lse[part * R + r] = lse2;
      }
      const bool nans = s_any_nan[n & 1];
      if constexpr (C::kCopies == 1) {
#pragma unroll 1
        for (int c = 0; c < D && busy; c += 32) {
          float o[32];
          tmem_ld32(t_o + c, reinterpret_cast<uint32_t*>(o));
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            mul_f32x2(o[j], o[j + 1], o[j], o[j + 1], w, w);
            mul_f32x2(o[j], o[j + 1], o[j], o[j + 1], w2, w2);
          }
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
      } else {
        // the copies' sum through shared memory, a d per lane
        float* buf = reinterpret_cast<float*>(smem + C::sum_off);
        const int64_t* s_orow = reinterpret_cast<const int64_t*>(smem + C::row_off);
        const int rows = min(a.rows - p.rt * R, R);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(t_o + c, reinterpret_cast<uint32_t*>(o));
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            mul_f32x2(o[j], o[j + 1], o[j], o[j + 1], w, w);
            mul_f32x2(buf[th * 33 + j], buf[th * 33 + j + 1], o[j], o[j + 1], w2, w2);
          }
          group_sync();
          for (int q = wq; q < rows; q += kWarps) {
            float x = 0.f;
#pragma unroll
            for (int u = 0; u < C::kCopies; ++u) x += buf[(u * R + q) * 33 + lane];
            if (nans && ((s_nan(n)[(c + lane) * 4 + (q >> 5)] >> (q & 31)) & 1u)) x = bad;
            if (!p.whole)
              a.part_o[(part * R + q) * D + c + lane] = x;
            else if (a.out_fp32)
              static_cast<float*>(a.out)[s_orow[q] * D + c + lane] = x;
            else
              static_cast<__nv_bfloat16*>(a.out)[s_orow[q] * D + c + lane] = __float2bfloat16_rn(x);
          }
          group_sync();
        }
      }
      tc_fence_before();
      if (ok) mbar_arrive(&bars.done[n & 1]);
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
