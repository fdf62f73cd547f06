// Append with rotary positions: the new tokens' keys go rotated into the slots of a paged cache, their values
// as they are, and the queries (and the probe) of the same tokens come out rotated, in one launch.
//
// Data movement like lla_paged_append, bound by HBM and, for the few tokens of a drafting step, by the launch
// and the chain starts - page - slot. A thread has one item of a token's features (lla_rotary.cuh) and goes
// over `per` of the token's heads with the same cosines and sines.
#include <type_traits>

#include "lla_paged.cuh"
#include "lla_rotary.cuh"

namespace lla {
namespace paged {
namespace {

struct Rows {
  const void *k, *v, *q, *r;  // q, r: may be nullptr
  void *q_out, *r_out;
  const int* offsets;  // [tokens] or nullptr
  int Hq;              // heads of q (0 without), and of r where there is one
  int units;           // Hkv (a key with its value), then the heads of q and of r
  int items, per, vw;  // vw: 16-byte words of a value
};

template <typename I, typename T>
__global__ void __launch_bounds__(256) append_rotary_kernel(const __grid_constant__ rotary::Turn turn, Params p,
                                                            const __grid_constant__ Rows a) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int token = (int)(i / a.items), mine_ = (int)(i - (long long)token * a.items);
  if (token >= p.tokens) return;
  int b = 0, e = p.B;  // the last sequence with starts[b] <= token
  while (e - b > 1) {
    const int mid = (b + e) / 2;
    if (__ldg(p.starts + mid) <= token) b = mid;
    else e = mid;
  }
  const Seq sq = load_seq(p, b);
  if (token < sq.t0 || token >= sq.t0 + sq.n) return;
  const int index = token - sq.t0, j = sq.first + index;
  const I item(turn, mine_, sq.first + (a.offsets ? __ldg(a.offsets + token) : index));
  const int u0 = blockIdx.y * a.per, u1 = min(a.units, u0 + a.per);
  const int pg = u0 < p.Hkv && j >= 0 ? load_page(p, b, j >> p.page_shift) : -1;
  const long long slot0 = ((long long)pg * p.Hkv) * p.page + (j & (p.page - 1));
  const int d = p.d;
  auto src = [&](int u) -> const T* {
    if (u < p.Hkv) return static_cast<const T*>(a.k) + ((long long)token * p.Hkv + u) * d;
    u -= p.Hkv;
    return u < a.Hq ? static_cast<const T*>(a.q) + ((long long)token * a.Hq + u) * d
                    : static_cast<const T*>(a.r) + ((long long)token * a.Hq + u - a.Hq) * d;
  };
  auto dst = [&](int u) -> T* {
    if (u < p.Hkv) return pg < 0 ? nullptr : static_cast<T*>(p.k) + (slot0 + (long long)u * p.page) * d;
    u -= p.Hkv;
    return u < a.Hq ? static_cast<T*>(a.q_out) + ((long long)token * a.Hq + u) * d
                    : static_cast<T*>(a.r_out) + ((long long)token * a.Hq + u - a.Hq) * d;
  };
  constexpr int U = 4;
  for (int u = u0; u < u1; u += U) {
    typename I::Piece x[U];
#pragma unroll
    for (int c = 0; c < U; ++c)
      if (u + c < u1) item.load(src(u + c), x[c]);
#pragma unroll
    for (int c = 0; c < U; ++c) {
      if (u + c >= u1) break;
      T* const to = dst(u + c);
      if (to) item.store(turn, to, x[c]);
      if (u + c < p.Hkv && pg >= 0) {
        const uint4* vs = static_cast<const uint4*>(a.v) + ((long long)token * p.Hkv + u + c) * a.vw;
        uint4* vd = static_cast<uint4*>(p.v) + (slot0 + (long long)(u + c) * p.page) * a.vw;
        for (int w = mine_; w < a.vw; w += a.items) vd[w] = vs[w];
        if (mine_ == 0 && p.mass) p.mass[slot0 + (long long)(u + c) * p.page] = 0.f;
      }
    }
  }
}

template <typename T>
cudaError_t launch_t(const Params& p, const rotary::Turn& turn, int layout, Rows a, cudaStream_t s) {
  cudaError_t err = cudaErrorInvalidConfiguration;
  rotary::pick_item<T>(turn, layout, [&](auto* tag) {
    using I = std::remove_pointer_t<decltype(tag)>;
    a.items = I::items(turn.half, p.d);
    // Heads to a thread: as many as leave every SM a thousand threads, 8 at most.
    const long long threads = (long long)p.tokens * a.items, per = threads * a.units / (152 * 1024);
    a.per = per < 1 ? 1 : per > 8 ? 8 : (int)per;
    const long long blocks = (threads + 255) / 256, groups = (a.units + a.per - 1) / a.per;
    if (blocks > 0x7fffffffLL || groups > 65535) return;
    append_rotary_kernel<I, T><<<dim3((unsigned)blocks, (unsigned)groups), 256, 0, s>>>(turn, p, a);
    count_launch();
    err = cudaGetLastError();
  });
  return err;
}

}  // namespace

cudaError_t launch_append_rotary(const Params& p, const rotary::Turn& turn, int layout, const void* k, const void* v,
                                 const void* q, const void* r, void* q_out, void* r_out, int q_heads,
                                 const int* offsets, int dtype, cudaStream_t s) {
  Rows a = {};
  a.k = k;
  a.v = v;
  a.q = q;
  a.r = r;
  a.q_out = q_out;
  a.r_out = r_out;
  a.offsets = offsets;
  a.Hq = q ? q_heads : 0;
  a.units = p.Hkv + a.Hq + (r ? a.Hq : 0);
  a.vw = p.dv * (dtype == LLA_F32 ? 4 : 2) / 16;
  return dtype == LLA_F32 ? launch_t<float>(p, turn, layout, a, s) : launch_t<__nv_bfloat16>(p, turn, layout, a, s);
}

}  // namespace paged
}  // namespace lla
