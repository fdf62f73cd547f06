// Append with rotary positions: the new tokens' keys go rotated into the slots of a paged cache, their values
// as they are, and the queries (and the probe) of the same tokens come out rotated, in one launch.
//
// Data movement like lla_paged_append, bound by HBM and, for the few tokens of a drafting step, by the launch
// and the chain starts - page - slot. A thread has one item of a token's features (lla_rotary.cuh) and goes
// over `per` of the token's heads with the same cosines and sines, or has as much of `per` of its values. What it
// moves does not depend on where that goes, so the first heads are on their way before the search for the
// token's sequence, in a copy of starts in shared memory where it fits.
// Measured: 4 prompts of 4096, 8 heads of 128 of k, v, q and r, 50 us, 5.3 TB/s (78 % of the copy bandwidth); 16 drafts
// of 32 nodes, 32 heads over 8 of 128, 6.2 us.
#include <type_traits>

#include "lla_paged.cuh"
#include "lla_rotary.cuh"

namespace lla {
namespace paged {
namespace {

constexpr int kStarts = 1024;  // entries of starts in shared memory

struct Rows {
  const void *k, *v, *q, *r;  // q, r: may be nullptr
  void *q_out, *r_out;
  const int* offsets;  // [tokens] or nullptr
  int Hq;              // heads of q (0 without), and of r where there is one
  int units;           // rotated heads of a token: of k, q and r
  int items, per, vw;  // vw: 16-byte words of a value
  int groups;          // of `per` rotated heads; behind them those of values
};

// A token's place: index and position among its sequence's, page (-1: none) and slot of head 0.
struct Place {
  int index, first, pg;
  long long slot;
};
// All threads of a block call; false: no sequence covers the token.
__device__ __forceinline__ bool find_place(const Params& p, int token, bool cached, int* starts_s, Place* out) {
  const bool staged = p.B <= kStarts;
  if (staged) {
    for (int b = threadIdx.x; b < p.B; b += 256) starts_s[b] = p.starts[b];
    __syncthreads();
  }
  if (token >= p.tokens) return false;
  int b = 0, e = p.B;  // the last sequence with starts[b] <= token
  while (e - b > 1) {
    const int mid = (b + e) / 2;
    if ((staged ? starts_s[mid] : __ldg(p.starts + mid)) <= token) b = mid;
    else e = mid;
  }
  const Seq sq = load_seq(p, b);
  if (token < sq.t0 || token >= sq.t0 + sq.n) return false;
  out->index = token - sq.t0;
  out->first = sq.first;
  const int j = sq.first + out->index;
  out->pg = cached && j >= 0 ? load_page(p, b, j >> p.page_shift) : -1;
  out->slot = ((long long)out->pg * p.Hkv) * p.page + (j & (p.page - 1));
  return true;
}

template <typename I, typename T>
__global__ void __launch_bounds__(256, 3) append_rotary_kernel(const __grid_constant__ rotary::Turn turn, Params p,
                                                               const __grid_constant__ Rows a) {
  __shared__ int starts_s[kStarts];
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int token = (int)min(i / a.items, (long long)p.tokens), lane = (int)(i - i / a.items * a.items);
  const bool there = token < p.tokens;
  Place at;
  if ((int)blockIdx.y >= a.groups) {  // values: words lane, lane + items, .. of `per` heads
    const int h0 = (blockIdx.y - a.groups) * a.per, heads = min(p.Hkv - h0, a.per);
    const int each = (a.vw - lane + a.items - 1) / a.items, count = there ? heads * each : 0;
    const uint4* src = static_cast<const uint4*>(a.v) + ((long long)token * p.Hkv + h0) * a.vw + lane;
    constexpr int U = 8;
    uint4 w[U];
    auto load = [&](int j0) {
#pragma unroll
      for (int c = 0; c < U; ++c)
        if (j0 + c < count) w[c] = src[(j0 + c) / each * a.vw + (j0 + c) % each * a.items];
    };
    load(0);
    if (!find_place(p, token, true, starts_s, &at) || at.pg < 0) return;
    for (int j0 = 0; j0 < count; j0 += U) {
      if (j0) load(j0);
#pragma unroll
      for (int c = 0; c < U; ++c) {
        if (j0 + c >= count) break;
        const int h = h0 + (j0 + c) / each, word = lane + (j0 + c) % each * a.items;
        const long long slot = at.slot + (long long)h * p.page;
        static_cast<uint4*>(p.v)[slot * a.vw + word] = w[c];
        if (word == 0 && p.mass) p.mass[slot] = 0.f;
      }
    }
    return;
  }
  const int u0 = blockIdx.y * a.per, u1 = there ? min(a.units, u0 + a.per) : 0;
  I item(turn, lane);
  constexpr int U = I::kAhead;
  typename I::Piece x[U];
  auto load = [&](int v0) {
#pragma unroll
    for (int c = 0; c < U; ++c) {
      if (v0 + c >= u1) break;
      int u = v0 + c;
      const T* row = static_cast<const T*>(a.k) + ((long long)token * p.Hkv + u) * p.d;
      if (u >= p.Hkv) {
        u -= p.Hkv;
        row = u < a.Hq ? static_cast<const T*>(a.q) + ((long long)token * a.Hq + u) * p.d
                       : static_cast<const T*>(a.r) + ((long long)token * a.Hq + u - a.Hq) * p.d;
      }
      item.load(row, x[c]);
    }
  };
  load(u0);
  if (!find_place(p, token, u0 < p.Hkv, starts_s, &at)) return;
  item.angles(turn, (long long)at.first + (a.offsets ? __ldg(a.offsets + token) : at.index));
  for (int v0 = u0; v0 < u1; v0 += U) {
    if (v0 > u0) load(v0);
#pragma unroll
    for (int c = 0; c < U; ++c) {
      if (v0 + c >= u1) break;
      int u = v0 + c;
      T* row = static_cast<T*>(p.k) + (at.slot + (long long)u * p.page) * p.d;
      if (u >= p.Hkv) {
        u -= p.Hkv;
        row = u < a.Hq ? static_cast<T*>(a.q_out) + ((long long)token * a.Hq + u) * p.d
                       : static_cast<T*>(a.r_out) + ((long long)token * a.Hq + u - a.Hq) * p.d;
      } else if (at.pg < 0) {
        continue;
      }
      item.store(turn, row, x[c]);
    }
  }
}

template <typename T>
cudaError_t launch_t(const Params& p, const rotary::Turn& turn, int layout, Rows a, cudaStream_t s) {
  cudaError_t err = cudaErrorInvalidConfiguration;
  rotary::pick_item<T>(turn, layout, [&](auto* tag) {
    using I = std::remove_pointer_t<decltype(tag)>;
    a.items = I::items(turn.half, p.d);
    // Heads to a thread: as many as leave every SM five hundred threads, 8 at most (16 drafts of 32 nodes, 40 rotated
    // heads of 128: 8.4 us with a thousand, 6.1 so).
    const long long threads = (long long)p.tokens * a.items, per = threads * a.units / (152 * 512);
    a.per = per < 1 ? 1 : per > 8 ? 8 : (int)per;
    if (a.per < (a.units + p.Hkv + 65532) / 65533) a.per = (a.units + p.Hkv + 65532) / 65533;  // (the grid's limit)
    const long long blocks = (threads + 255) / 256;
    a.groups = (a.units + a.per - 1) / a.per;
    const long long groups = a.groups + (p.Hkv + a.per - 1) / a.per;
    if (blocks > 0x7fffffffLL) return;
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
