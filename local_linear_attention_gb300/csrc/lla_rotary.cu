// Rotary positions of [B, H, T, d] tensors (q, k and the probe of an attention, or their gradients) and the
// frequencies.
//
// What bounds it: HBM, each element read once and written once. A thread keeps the cosines and sines of its
// pairs and takes the same features of several heads, of all the tensors, one after the other, so that an
// angle's sine and cosine (some 30 instructions with the integer product) are found once for `per` heads, while the
// first of them are on their way;
// the loads of several heads are in flight together. Measured: q, k and r of B4 H8 T4096 d64,
// 18 us, 5.6 TB/s (82 % of the copy bandwidth); fp32, two of B2 H8 T2047, 6.3 us.
#include <cmath>
#include <type_traits>

#include "lla_rotary.cuh"
#include "lla_turns.h"

namespace lla {
namespace rotary {

int make_turn(const lla_rotary_spec* spec, int d, bool back, Turn* out) {
  if (!spec) return LLA_ERR_INVALID_ARG;
  for (int r : spec->reserved)
    if (r != 0) return LLA_ERR_INVALID_ARG;
  if (spec->layout != LLA_ROTARY_HALVES && spec->layout != LLA_ROTARY_INTERLEAVED) return LLA_ERR_INVALID_ARG;
  if (spec->rot < 2 || spec->rot % 2 || spec->rot > d || !std::isfinite(spec->scale)) return LLA_ERR_INVALID_ARG;
  *out = Turn{};
  out->scale = spec->scale;
  out->half = spec->rot / 2;
  out->back = back;
  for (int i = 0; i < out->half; ++i) {
    if (!(std::fabs(spec->freq[i]) <= 0x1p20)) return LLA_ERR_INVALID_ARG;
    out->turns[i] = turns_of(spec->freq[i]);
  }
  return LLA_OK;
}

namespace {

struct Tensors {
  const void* x[3];
  void* y[3];
  int upto[3];  // heads of this tensor and those before it
  int heads, T, d, items, per;
  long long rows;  // B * T
  const int* positions;
};

template <typename I, typename T>
__global__ void __launch_bounds__(256) rotary_kernel(const __grid_constant__ Turn turn, const __grid_constant__ Tensors a) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, row = i / a.items;
  if (row >= a.rows) return;
  const int b = (int)(row / a.T), t = (int)(row - (long long)b * a.T);
  I item(turn, (int)(i - row * a.items));
  const int pos = a.positions ? a.positions[row] : t;
  const int h0 = blockIdx.y * a.per, h1 = min(a.heads, h0 + a.per);
  // element offset of head h's row, and which tensor it is in
  auto place = [&](int h, int& which) {
    which = h >= a.upto[1] ? 2 : h >= a.upto[0] ? 1 : 0;
    const int before = which ? a.upto[which - 1] : 0, heads = a.upto[which] - before;
    return (((long long)b * heads + h - before) * a.T + t) * a.d;
  };
  constexpr int U = I::kAhead;
  for (int h = h0; h < h1; h += U) {
    typename I::Piece p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u >= h1) break;
      int w;
      const long long at = place(h + u, w);
      item.load(static_cast<const T*>(a.x[w]) + at, p[u]);
    }
    if (h == h0) item.angles(turn, pos);  // while the first heads are on their way
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u >= h1) break;
      int w;
      const long long at = place(h + u, w);
      item.store(turn, static_cast<T*>(a.y[w]) + at, p[u]);
    }
  }
}

template <typename T>
cudaError_t launch(const Turn& turn, int layout, Tensors a, cudaStream_t s) {
  cudaError_t err = cudaErrorInvalidConfiguration;
  pick_item<T>(turn, layout, [&](auto* tag) {
    using I = std::remove_pointer_t<decltype(tag)>;
    a.items = I::items(turn.half, a.d);
    // Heads to a thread: as many as leave every SM five hundred threads, 8 at most.
    const long long threads = a.rows * a.items, all = threads * a.heads;
    const long long per = all / (152 * 512);
    a.per = per < 1 ? 1 : per > 8 ? 8 : (int)per;
    if (a.per < (a.heads + 65534) / 65535) a.per = (a.heads + 65534) / 65535;  // (the grid's limit)
    const long long blocks = (threads + 255) / 256, groups = (a.heads + a.per - 1) / a.per;
    if (blocks > 0x7fffffffLL) return;
    rotary_kernel<I, T><<<dim3((unsigned)blocks, (unsigned)groups), 256, 0, s>>>(turn, a);
    count_launch();
    err = cudaGetLastError();
  });
  return err;
}

}  // namespace
}  // namespace rotary
}  // namespace lla

using namespace lla;

extern "C" {

int lla_rotary_frequencies(lla_rotary_spec* spec, int rot, int layout, double base, int stretch, double factor,
                           int context, double slow, double fast) {
  if (!spec || rot < 2 || rot % 2 || rot > 2 * rotary::kMaxPairs) return LLA_ERR_INVALID_ARG;
  if (layout != LLA_ROTARY_HALVES && layout != LLA_ROTARY_INTERLEAVED) return LLA_ERR_INVALID_ARG;
  if (stretch < LLA_STRETCH_NONE || stretch > LLA_STRETCH_WAVELENGTHS) return LLA_ERR_INVALID_ARG;
  if (!(std::isfinite(base) && base >= 1.0)) return LLA_ERR_INVALID_ARG;
  if (stretch != LLA_STRETCH_NONE && !(std::isfinite(factor) && factor >= 1.0)) return LLA_ERR_INVALID_ARG;
  if (stretch == LLA_STRETCH_BASE) {
    if (rot == 2) return LLA_ERR_INVALID_ARG;
    base *= std::pow(factor, rot / (rot - 2.0));
    if (!std::isfinite(base)) return LLA_ERR_INVALID_ARG;
  }
  if (stretch == LLA_STRETCH_WAVELENGTHS && !(context > 0 && std::isfinite(slow) && std::isfinite(fast) && fast > slow))
    return LLA_ERR_INVALID_ARG;
  *spec = lla_rotary_spec{};
  spec->rot = rot;
  spec->layout = layout;
  spec->scale = stretch == LLA_STRETCH_WAVELENGTHS ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (stretch == LLA_STRETCH_POSITIONS) f /= factor;
    if (stretch == LLA_STRETCH_WAVELENGTHS) {
      const double turns = context * f / 6.283185307179586;
      double keep = (turns - slow) / (fast - slow);
      keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      f *= keep + (1 - keep) / factor;
    }
    spec->freq[i] = f;
  }
  return LLA_OK;
}

int lla_rotary(const lla_rotary_spec* spec, const void* const* x, void* const* y, const int* heads, int count,
               const int* positions, int B, int T, int d, int backward, int dtype, void* stream) {
  if (dtype != LLA_F32 && dtype != LLA_BF16) return LLA_ERR_INVALID_ARG;
  if (count < 1 || count > 3 || !x || !y || !heads || B < 0 || T < 0) return LLA_ERR_INVALID_ARG;
  if (d != 16 && d != 32 && d != 64 && d != 128) return LLA_ERR_UNSUPPORTED;
  rotary::Turn turn;
  const int st = rotary::make_turn(spec, d, backward != 0, &turn);
  if (st != LLA_OK) return st;
  rotary::Tensors a = {};
  long long all = 0;
  for (int i = 0; i < count; ++i) {
    if (heads[i] < 0) return LLA_ERR_INVALID_ARG;
    all += heads[i];
  }
  if (all > rotary::kMostHeads || all * B >= (1LL << 31) || all * B * T >= (1LL << 31)) return LLA_ERR_UNSUPPORTED;
  if (all * B * T == 0) return LLA_OK;
  for (int i = 0; i < 3; ++i) {
    a.upto[i] = (i ? a.upto[i - 1] : 0) + (i < count ? heads[i] : 0);
    a.x[i] = i < count ? x[i] : nullptr;
    a.y[i] = i < count ? y[i] : nullptr;
    if (i < count && heads[i] > 0 &&
        (!x[i] || !y[i] || (reinterpret_cast<uintptr_t>(x[i]) & 15u) || (reinterpret_cast<uintptr_t>(y[i]) & 15u)))
      return LLA_ERR_INVALID_ARG;
  }
  for (int i = 0; i < count; ++i)  // what is written is nobody else's
    for (int j = 0; j < count; ++j)
      if (i != j && heads[i] > 0 && heads[j] > 0 && (y[i] == y[j] || y[i] == x[j])) return LLA_ERR_INVALID_ARG;
  a.heads = (int)all;
  a.T = T;
  a.d = d;
  a.rows = (long long)B * T;
  a.positions = positions;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return (dtype == LLA_F32 ? rotary::launch<float>(turn, spec->layout, a, s)
                           : rotary::launch<__nv_bfloat16>(turn, spec->layout, a, s)) == cudaSuccess
             ? LLA_OK
             : LLA_ERR_CUDA;
}

}  // extern "C"
