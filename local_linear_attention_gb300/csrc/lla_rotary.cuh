// Rotary positions: a pair (x0, x1) of a head's features, at position pos, becomes scale times
//   (x0 cos a - x1 sin a, x0 sin a + x1 cos a),   a = pos * freq(pair),
// and its gradient goes back by the transpose (sin a with the other sign). Pairs are (i, i + rot/2) or
// (2i, 2i + 1), i < rot/2; features from rot on are copied.
//
// Angles. A far position times a frequency needs more bits than fp32 has (a million times 1 rad: the
// product is off by 0.03 rad), and fp64 is slow here. So a frequency is held in turns as a 64-bit fraction,
// pos times it wraps around modulo a turn by itself, exactly, in integers: off by pos * 2^-65 turns. The two
// highest bits of the sum with an eighth are the quadrant; what is left, within an eighth of a turn, goes to
// fp32 (off by little more than 2^-28 turns at its ends) and to sine and cosine.
#pragma once

#include "lla_internal.cuh"

namespace lla {
namespace rotary {

constexpr int kMaxPairs = 64;
// Heads that a position's threads go over: their indices, and those of a last group of them, stay within 31 bits.
constexpr long long kMostHeads = (1LL << 31) - (1 << 17);

// Passed to kernels by value.
struct Turn {
  unsigned long long turns[kMaxPairs];  // per position, in units of 2^-64 turns
  float scale;
  int half;  // pairs
  int back;  // the transpose
};

__device__ __forceinline__ float2 fast_cos_sin(float x) { return make_float2(__cosf(x), __sinf(x)); }
// scale * (cos, sin) of a pair's angle. FAST (bf16): the hardware's sine and cosine, off by 2^-21 at most
// where a feature is rounded to 2^-9 of its value; else CUDA's sincospif.
template <bool FAST>
__device__ __forceinline__ void cos_sin(const Turn& t, int pair, long long pos, float& c, float& s) {
  const unsigned long long at = (unsigned long long)pos * t.turns[pair];
  const unsigned q = (unsigned)((at + (1ull << 61)) >> 62);
  const float f = (float)(int)((long long)(at - ((unsigned long long)q << 62)) >> 32) * 0x1p-31f;  // half turns
  float s0, c0;
  if (FAST) {
    const float2 x = fast_cos_sin(f * 3.14159265358979f);
    c0 = x.x;
    s0 = x.y;
  } else {
    sincospif(f, &s0, &c0);
  }
  c0 *= t.scale;
  s0 *= t.scale;
  c = q & 1 ? s0 : c0;
  s = q & 1 ? c0 : s0;
  if (q == 1 || q == 2) c = -c;
  if ((q >> 1) != (unsigned)t.back) s = -s;
}

// N elements of T as one word of 2 to 16 bytes.
template <int BYTES>
struct Word;
template <> struct Word<16> { using type = uint4; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<2> { using type = uint16_t; };
template <typename T, int N>
struct Elements {
  union {
    typename Word<N * (int)sizeof(T)>::type word;
    T x[N];
  };
  __device__ Elements() {}
};

// What one thread does of a row of d features: an item is N pairs of the halves layout (N elements of each
// half), or N elements of interleaved pairs; or N elements that are copied. items(d) of them make a row.
template <typename T, int N, bool HALVES>
struct Item {
  static constexpr bool kFast = sizeof(T) == 2;
  static constexpr int P = HALVES ? N : N / 2;  // pairs
  static_assert(HALVES || N >= 2, "a pair to an item");
  // Heads whose loads are in flight together, 128 bytes where an item is 16 or 32 (prompts of 16k tokens, 24 heads of 128
  // rotated, interleaved: 59 us with 4, 50 with 8).
  static constexpr int kAhead = HALVES && N * sizeof(T) == 16 ? 4 : 8;
  using E = Elements<T, N>;
  struct Piece {
    E a, b;
  };
  int at, other;  // first elements; other: of the second half, or -1
  int first;      // first pair; kMaxPairs: none
  float c[P], s[P];
  static __host__ __device__ int items(int half, int d) { return HALVES ? half / N + (d - 2 * half) / N : d / N; }

  __device__ __forceinline__ Item(const Turn& t, int item) {
    other = -1;
    if (HALVES) {
      const int turned = t.half / N;
      first = item < turned ? item * N : kMaxPairs;
      at = item < turned ? item * N : 2 * t.half + (item - turned) * N;
      if (item < turned) other = t.half + item * N;
    } else {
      at = item * N;
      first = at / 2;
    }
  }
  // The cosines and sines of the item's pairs; before the first store.
  __device__ __forceinline__ void angles(const Turn& t, long long pos) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (first + i < t.half) cos_sin<kFast>(t, first + i, pos, c[i], s[i]);
  }
  __device__ __forceinline__ void load(const T* row, Piece& p) const {
    p.a.word = *reinterpret_cast<const decltype(p.a.word)*>(row + at);
    if (HALVES && other >= 0) p.b.word = *reinterpret_cast<const decltype(p.b.word)*>(row + other);
  }
  __device__ __forceinline__ void store(const Turn& t, T* row, Piece& p) const {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (first + i >= t.half) continue;  // copied as it is, infinities too
      T& u = HALVES ? p.a.x[i] : p.a.x[2 * i];
      T& v = HALVES ? p.b.x[i] : p.a.x[2 * i + 1];
      const float x = ldf(&u, 0), y = ldf(&v, 0);
      stf(&u, 0, fmaf(x, c[i], -(y * s[i])));
      stf(&v, 0, fmaf(x, s[i], y * c[i]));
    }
    *reinterpret_cast<decltype(p.a.word)*>(row + at) = p.a.word;
    if (HALVES && other >= 0) *reinterpret_cast<decltype(p.b.word)*>(row + other) = p.b.word;
  }
};

// Checks a spec for heads of d features and lays it out for the kernels.
int make_turn(const lla_rotary_spec* spec, int d, bool back, Turn* out);

// Calls go(Item type tag) with the widest item that the layout allows: in the halves layout its words have to
// divide half, so that both halves are aligned to them.
template <typename T, typename Go>
void pick_item(const Turn& t, int layout, Go&& go) {
  constexpr int W = 16 / (int)sizeof(T);
  if (layout == LLA_ROTARY_INTERLEAVED) return go((Item<T, W, false>*)nullptr);
  if (t.half % W == 0) return go((Item<T, W, true>*)nullptr);
  if (sizeof(T) == 2 && t.half % 4 == 0) return go((Item<T, 4, true>*)nullptr);
  if (t.half % 2 == 0) return go((Item<T, 2, true>*)nullptr);
  return go((Item<T, 1, true>*)nullptr);
}

}  // namespace rotary
}  // namespace lla
