// Turning pairs of values by pos * frequency: exact angles, and the rows of a head.
//
// An angle is a fraction of a full turn in 64-bit fixed point: frequency / 2 pi is
// taken from the frequency's 53 bits once, and pos * fraction modulo 2^64 is the
// angle modulo a turn without any rounding, for every 32-bit position.  (In fp32
// the angle of position 10^6 would be off by 0.03 radians.)  What is left is the
// rounding of frequency / 2 pi to 2^-64 of a turn and below 2^-60 of itself.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace gb300 {

// frequency (radians per position) / 2 pi modulo 1, times 2^64.  m * 2^e with the
// 53-bit m: m * (2^64 / 2 pi) is a 117-bit product, shifted by e.
__device__ __forceinline__ uint64_t turns_of(double frequency) {
  constexpr uint64_t kInvTwoPi = 0x28be60db9391054aull;  // floor(2^64 / (2 pi))
  const uint64_t bits = (uint64_t)__double_as_longlong(frequency);
  const int ex = (int)(bits >> 52) & 0x7ff;
  const uint64_t m = (bits & 0xfffffffffffffull) | (ex ? 1ull << 52 : 0ull);
  const int e = (ex ? ex : 1) - 1075;
  const uint64_t hi = __umul64hi(m, kInvTwoPi), lo = m * kInvTwoPi;
  uint64_t t;
  if (e >= 0)
    t = e < 64 ? lo << e : 0ull;
  else if (e > -64)
    t = lo >> -e | hi << (64 + e);
  else
    t = e > -128 ? hi >> (-64 - e) : 0ull;
  return bits >> 63 ? 0ull - t : t;
}

// amp * (cos, sin) of pos * turns.  The angle's upper 32 bits (2^-32 of a turn, 1.5e-9
// radians) as a quadrant and a rest x in [-pi/4, pi/4], and there the two series up to
// x^10 and x^9: the first term left out is below 2e-9.
__device__ __forceinline__ float2 cos_sin(int pos, uint64_t turns, float amp) {
  // upper half of the 64-bit product with a signed position
  const uint32_t lo = (uint32_t)turns, u = (uint32_t)pos;
  const uint32_t angle = __umulhi(u, lo) + u * (uint32_t)(turns >> 32) - (pos < 0 ? lo : 0u);
  const uint32_t quadrant = (angle + 0x20000000u) >> 30;
  const float x = (float)(int)(angle - (quadrant << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float y = x * x;
  float s = fmaf(y, 1.f / 362880.f, -1.f / 5040.f);
  s = fmaf(y, s, 1.f / 120.f);
  s = fmaf(y, s, -1.f / 6.f);
  s = fmaf(y * x, s, x) * amp;
  float c = fmaf(y, -1.f / 3628800.f, 1.f / 40320.f);
  c = fmaf(y, c, -1.f / 720.f);
  c = fmaf(y, c, 1.f / 24.f);
  c = fmaf(y, c, -0.5f);
  c = fmaf(y, c, 1.f) * amp;
  // a quarter turn: (c, s) -> (-s, c)
  const float c1 = (quadrant & 1u) ? s : c, s1 = (quadrant & 1u) ? c : s;
  return make_float2(((quadrant + 1u) & 2u) ? -c1 : c1, (quadrant & 2u) ? -s1 : s1);
}

// What of a head turns.
struct Turning {
  const double* freqs;
  int rot, offset;
  float amp;
  bool inverse;
};

// (16384 tokens of 20 heads of 128, forward and backward: 59 us with evict-first loads, 61 us without;
// the rotated append of 65536 tokens 259 and 254 us)
template <bool kEvictFirst>
__device__ __forceinline__ uint4 load_rows(const void* p) {
  return kEvictFirst ? __ldcs(static_cast<const uint4*>(p)) : *static_cast<const uint4*>(p);
}
__device__ __forceinline__ void store_stream(void* p, uint4 v) { __stcs(static_cast<uint4*>(p), v); }

// A head's values in units of 32 bytes, two vectors of 16: first the units that turn
// (their pairs are the units' own), then those that are copied.  bf16 has 8 pairs to
// a unit, fp32 4.
template <typename E, bool kInterleaved>
struct HeadUnits {
  static constexpr int kVec = 16 / sizeof(E);  // values per vector, pairs per unit
  int turning, all;                            // units that turn, all of them
  // (in place: what does not turn stays)
  __device__ __forceinline__ HeadUnits(int d, int rot, bool copy)
      : turning(rot / (2 * kVec)), all(turning + (copy ? (d - rot) / (2 * kVec) : 0)) {}
  // first value of the unit's vector w (0, 1)
  __device__ __forceinline__ int at(int unit, int w, int rot, int offset) const {
    if (unit < turning)
      return offset + (kInterleaved ? (2 * unit + w) * kVec : unit * kVec + w * (rot / 2));
    const int v = (2 * (unit - turning) + w) * kVec;
    return v < offset ? v : v + rot;
  }
};

__device__ __forceinline__ float2 widen_bf16x2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Turns the pairs of one unit, in place: c, s per pair.
template <bool kInterleaved>
__device__ __forceinline__ void turn_unit(const __nv_bfloat16*, uint4& a, uint4& b, const float* c, const float* s) {
  uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if constexpr (kInterleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = widen_bf16x2(x[i]);
      x[i] = pack_bf16(v.x * c[i] - v.y * s[i], v.y * c[i] + v.x * s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = widen_bf16x2(x[i]), w = widen_bf16x2(x[4 + i]);
      x[i] = pack_bf16(v.x * c[2 * i] - w.x * s[2 * i], v.y * c[2 * i + 1] - w.y * s[2 * i + 1]);
      x[4 + i] = pack_bf16(w.x * c[2 * i] + v.x * s[2 * i], w.y * c[2 * i + 1] + v.y * s[2 * i + 1]);
    }
  }
  a = make_uint4(x[0], x[1], x[2], x[3]);
  b = make_uint4(x[4], x[5], x[6], x[7]);
}
template <bool kInterleaved>
__device__ __forceinline__ void turn_unit(const float*, uint4& a, uint4& b, const float* c, const float* s) {
  float x[8] = {__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w),
                __uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = kInterleaved ? 2 * i : i, q = kInterleaved ? 2 * i + 1 : i + 4;
    const float v = x[p], w = x[q];
    x[p] = v * c[i] - w * s[i];
    x[q] = w * c[i] + v * s[i];
  }
  a = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  b = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
}

constexpr int kMaxRot = 256;  // values of a head that turn, at most

// The heads [h0, h1) of one token by one warp: heads below h_q lie in q, the others in
// k (each row: the token's first value).  The warp's lanes first share the token's
// angles through `tab` (kMaxRot floats of shared memory, its own): cos, then sin, of
// pair lane + 32 i from turns[i].  Then a lane has one unit of every (32 / units)-th
// head, so its factors stay in registers; kBatch heads' loads are in flight together.
template <typename E, bool kInterleaved, int kBatch, bool kEvictFirst>
__device__ __forceinline__ void turn_token(const E* q_in, E* q_out, const E* k_in, E* k_out, int d, int h_q, int h0,
                                           int h1, bool copy, const Turning& t, int pos, const uint64_t (&turns)[4],
                                           float* tab) {
  using U = HeadUnits<E, kInterleaved>;
  const U units(d, t.rot, copy);
  const int lane = threadIdx.x & 31, half = t.rot / 2;
  const int per = 32 / units.all;  // heads at a time
  const int u = lane % units.all, r = lane / units.all;
  const int va = units.at(u, 0, t.rot, t.offset), vb = units.at(u, 1, t.rot, t.offset);
  __syncwarp();  // the last token's factors have been read
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (lane + 32 * i < half) {
      const float2 f = cos_sin(pos, turns[i], t.amp);
      tab[lane + 32 * i] = f.x;
      tab[half + lane + 32 * i] = t.inverse ? -f.y : f.y;
    }
  }
  __syncwarp();
  float c[U::kVec], s[U::kVec];
  const bool turns_here = u < units.turning;
  if (turns_here) {
#pragma unroll
    for (int i = 0; i < U::kVec; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(tab + u * U::kVec + i);
      const float4 y = *reinterpret_cast<const float4*>(tab + half + u * U::kVec + i);
      c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
      s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
    }
  }
  if (r >= per) return;
  for (int h = h0 + r; h < h1; h += kBatch * per) {
    uint4 a[kBatch], b[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int hh = h + i * per;
      if (hh < h1) {
        const E* row = hh < h_q ? q_in + (int64_t)hh * d : k_in + (int64_t)(hh - h_q) * d;
        a[i] = load_rows<kEvictFirst>(row + va);
        b[i] = load_rows<kEvictFirst>(row + vb);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int hh = h + i * per;
      if (hh < h1) {
        E* row = hh < h_q ? q_out + (int64_t)hh * d : k_out + (int64_t)(hh - h_q) * d;
        if (turns_here) turn_unit<kInterleaved>(row, a[i], b[i], c, s);
        store_stream(row + va, a[i]);
        store_stream(row + vb, b[i]);
      }
    }
  }
}

// The lane's pairs' turns: pair lane + 32 i.
__device__ __forceinline__ void load_turns(const Turning& t, uint64_t (&turns)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) turns[i] = lane + 32 * i < t.rot / 2 ? turns_of(t.freqs[lane + 32 * i]) : 0ull;
}

}  // namespace gb300
