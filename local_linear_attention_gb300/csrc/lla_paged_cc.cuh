// Attention of new tokens over a paged cache on the CUDA cores, head sizes 16, 32, 64, 128, keys and
// values independent: the attention of bf16 where it is asked to (LLA_PATH_CUDA_CORE), with more than 128
// heads to a key/value head, or for chunks of more than 2048 sequences at once; the join of splits, for
// fp32 too; the weight tracking that does not go by the attention's logits (fp32: more than 256 rows to a
// sequence, or logits of more than 2 GiB; bf16 where the tensor cores do not take it).
//
// Mathematics, per row with visible keys j (logit s_j = q.k_j / h, probe t_j = r.k_j):
//   m = max s, p_j = exp(s_j - m), d1 = sum p, O1 = sum p v, and with a probe d2 = sum p t,
//   O2 = sum p t v;  o = (1 + d2/d1) O1/d1 - O2/d1  (softmax attention without one: O1/d1).
// One pass over the keys with the running m; the sums are fp32 whatever the inputs' type.
//
// A block takes BM rows (tokens x grouped heads of one key/value head, so that each key tile is
// read once for all of them) and key tiles of 64 staged in shared memory as fp32. 256 threads form
// a 16 x 16 grid: thread (ty, tx) computes the logits of BM/16 rows x 4 keys, then the products
// with the values for BM/16 rows x DV/16 columns. Bound: FP32 FMA.
// BM = 64, or 16 when no sequence brings more than 16 rows: a decode step would waste three
// quarters of the larger tile.
#pragma once

#include "lla_paged.cuh"

namespace lla {
namespace paged {
namespace {

constexpr int KT = 64;
constexpr int NT = 256;

template <int BM, int D, int DV, bool PROBE>
struct Smem {
  static constexpr int QP = D + 4, KP = D + 4, PP = BM + 4;
  static constexpr int q = 0;
  static constexpr int r = q + BM * QP;
  static constexpr int k = r + (PROBE ? BM * QP : 0);
  static constexpr int v = k + KT * KP;
  static constexpr int p = v + KT * DV;        // transposed: [key][row]
  static constexpr int p2 = p + KT * PP;
  static constexpr int floats = p2 + (PROBE ? KT * PP : 0);
  static constexpr int bytes = floats * 4;
};

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
}

// Stages ROWS rows of a [.., W] array as fp32; addr(row) gives a row's first element or nullptr
// (zeros). All loads of a thread are issued before the first store.
template <int W, int PITCH, int ROWS, typename T, typename Addr>
__device__ __forceinline__ void stage(float* dst, Addr addr) {
  constexpr int N = (ROWS * (W / 4) + NT - 1) / NT;
  float4 x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = threadIdx.x + i * NT, row = e / (W / 4), c = (e % (W / 4)) * 4;
    const T* src = row < ROWS ? addr(row) : nullptr;
    x[i] = src ? ld4(src + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = threadIdx.x + i * NT, row = e / (W / 4), c = (e % (W / 4)) * 4;
    if (row < ROWS) *reinterpret_cast<float4*>(dst + row * PITCH + c) = x[i];
  }
}

// s[i][j] += sum_c a[row0 + i][c] b[tx + 16 j][c]
template <int RM, int D, int P>
__device__ __forceinline__ void dots(const float* a, const float* b, float (&s)[RM][4]) {
  for (int c = 0; c < D; c += 4) {
    float4 x[RM], y[4];
#pragma unroll
    for (int i = 0; i < RM; ++i) x[i] = *reinterpret_cast<const float4*>(a + i * P + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + 16 * j * P + c);
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[i][j] = fmaf(x[i].w, y[j].w, fmaf(x[i].z, y[j].z, fmaf(x[i].y, y[j].y, fmaf(x[i].x, y[j].x, s[i][j]))));
  }
}

template <typename T, int D, int DV, bool PROBE, int BM>
__global__ void __launch_bounds__(NT) attend_cc_kernel(Params p) {
  using S = Smem<BM, D, DV, PROBE>;
  constexpr int RM = BM / 16;                          // rows per thread
  constexpr int VC = DV / 16, VW = VC < 4 ? VC : 4;    // value columns per thread, in vectors of VW
  extern __shared__ float sm[];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int hk = blockIdx.x % p.Hkv, part = blockIdx.y;
  const int per = max(1, BM / p.g);                    // tokens per tile (g > BM: several tiles a token)
  const int slices = (p.g + BM - 1) / BM;              // tiles per token
  int b, tile;
  const int index = blockIdx.x / p.Hkv;
  if (!find_tile(p, per, index / slices, &b, &tile)) return;
  const Seq sq = load_seq_or_tree(p, b);
  if (sq.n == 0) return;                     // an impossible length (find_tile counts by the starts)
  const int u0 = (index % slices) * BM;      // first grouped head of this tile (g > BM)
  const int tok0 = tile * per, ntok = min(per, sq.n - tok0);
  const int width = min(p.g - u0, BM);                 // grouped heads per token in this tile
  const int nrows = ntok * width;
  const T* qg = static_cast<const T*>(p.q);
  const T* rg = static_cast<const T*>(p.r);
  const T* kg = static_cast<const T*>(p.k);
  const T* vg = static_cast<const T*>(p.v);
  auto rowid = [&](int row) -> long long {             // row of q, r, out (flat [tokens * Hq])
    return (long long)(sq.t0 + tok0 + row / width) * p.Hq + hk * p.g + u0 + row % width;
  };
  stage<D, S::QP, BM, T>(sm + S::q, [&](int row) { return row < nrows ? qg + rowid(row) * D : (const T*)nullptr; });
  if (PROBE)
    stage<D, S::QP, BM, T>(sm + S::r, [&](int row) { return row < nrows ? rg + rowid(row) * D : (const T*)nullptr; });

  // (With trees the rows' positions lie between the first node's and this, and `visible` goes by their bits.)
  const int p0 = p.parents ? sq.first : sq.first + tok0, p1 = sq.first + tok0 + ntok - 1;
  const TileRange<KT> range(p, p0, p1);
  const int chunk = (range.count + p.split - 1) / p.split;
  const int i0 = part * chunk, i1 = min(range.count, i0 + chunk);

  int pos[RM];
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int row = ty * RM + i;
    pos[i] = row < nrows ? p0 + row / width : -1;      // a row past the end sees nothing
    if (p.parents && row < nrows) pos[i] = sq.first + p.depth[sq.t0 + tok0 + row / width];
  }
  auto see = [&](int i, int j) {
    if (!p.parents || pos[i] < 0) return visible(p, pos[i], j);
    return j < sq.len && node_sees(p, sq.first, sq.t0 + tok0 + (ty * RM + i) / width, pos[i], j);
  };
  float m[RM], d1[RM], d2[RM], o1[RM][VC], o2[PROBE ? RM : 1][VC];
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    m[i] = -CUDART_INF_F;
    d1[i] = d2[i] = 0.f;
#pragma unroll
    for (int c = 0; c < VC; ++c) {
      o1[i][c] = 0.f;
      if (PROBE) o2[i][c] = 0.f;
    }
  }

  for (int it = i0; it < i1; ++it) {
    const int k0 = range.tile(it) * KT;
    __syncthreads();  // the previous tile's products are done
    auto slot = [&](int row) -> long long {
      const int j = k0 + row;
      if (j >= sq.len) return -1;
      const int pg = load_page(p, b, j >> p.page_shift);
      return pg < 0 ? -1 : ((long long)pg * p.Hkv + hk) * p.page + (j & (p.page - 1));
    };
    stage<D, S::KP, KT, T>(sm + S::k, [&](int row) { const long long s = slot(row); return s < 0 ? (const T*)nullptr : kg + s * D; });
    stage<DV, DV, KT, T>(sm + S::v, [&](int row) { const long long s = slot(row); return s < 0 ? (const T*)nullptr : vg + s * DV; });
    __syncthreads();
    float s[RM][4] = {}, t[PROBE ? RM : 1][4] = {};
    dots<RM, D, S::KP>(sm + S::q + ty * RM * S::QP, sm + S::k + tx * S::KP, s);
    if constexpr (PROBE) dots<RM, D, S::KP>(sm + S::r + ty * RM * S::QP, sm + S::k + tx * S::KP, t);
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      float tm = -CUDART_INF_F;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = see(i, k0 + tx + 16 * j) ? s[i][j] : -CUDART_INF_F;
        tm = fmaxf(tm, s[i][j]);
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, o));
      const float mn = fmaxf(m[i], tm);
      // no visible key so far: weights exp(-inf - 0) = 0
      const float ref = mn == -CUDART_INF_F ? 0.f : mn;
      if (mn != m[i]) {
        const float sc = expf((m[i] - ref) * p.inv_h);
        d1[i] *= sc;
        d2[i] *= sc;
#pragma unroll
        for (int c = 0; c < VC; ++c) {
          o1[i][c] *= sc;
          if (PROBE) o2[i][c] *= sc;
        }
        m[i] = mn;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float w = expf((s[i][j] - ref) * p.inv_h);
        d1[i] += w;  // this thread's keys only; summed over tx at the end
        sm[S::p + (tx + 16 * j) * S::PP + ty * RM + i] = w;
        if constexpr (PROBE) {
          const float wt = s[i][j] == -CUDART_INF_F ? 0.f : w * t[i][j];
          d2[i] += wt;
          sm[S::p2 + (tx + 16 * j) * S::PP + ty * RM + i] = wt;
        }
      }
    }
    __syncthreads();
    for (int j = 0; j < KT; ++j) {
      float w[RM], wt[PROBE ? RM : 1], x[VC];
#pragma unroll
      for (int i = 0; i < RM; ++i) w[i] = sm[S::p + j * S::PP + ty * RM + i];
      if constexpr (PROBE) {
#pragma unroll
        for (int i = 0; i < RM; ++i) wt[i] = sm[S::p2 + j * S::PP + ty * RM + i];
      }
#pragma unroll
      for (int c = 0; c < VC; ++c) x[c] = sm[S::v + j * DV + ((c / VW) * 16 + tx) * VW + c % VW];
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int c = 0; c < VC; ++c) {
          o1[i][c] = fmaf(w[i], x[c], o1[i][c]);
          if constexpr (PROBE) o2[i][c] = fmaf(wt[i], x[c], o2[i][c]);
        }
    }
  }

  unsigned again = 0;  // rows of this warp whose result is not finite
#pragma unroll
  for (int i = 0; i < RM; ++i) {
#pragma unroll
    for (int o = 8; o; o >>= 1) {
      d1[i] += __shfl_xor_sync(0xffffffffu, d1[i], o);
      d2[i] += __shfl_xor_sync(0xffffffffu, d2[i], o);
    }
    const int row = ty * RM + i;
    if (p.split > 1) {
      if (row < nrows) {
        const long long id = (long long)part * p.tokens * p.Hq + rowid(row);
        if (tx == 0) p.part_s[id] = make_float4(m[i], d1[i], d2[i], 0.f);
        float* dst = p.part_o + id * (PROBE ? 2 : 1) * DV;
#pragma unroll
        for (int c = 0; c < VC; ++c) {
          dst[((c / VW) * 16 + tx) * VW + c % VW] = o1[i][c];
          if constexpr (PROBE) dst[DV + ((c / VW) * 16 + tx) * VW + c % VW] = o2[i][c];
        }
      }
      continue;
    }
    const float inv = d1[i] == 0.f ? 0.f : 1.f / d1[i], f1 = (1.f + d2[i] * inv) * inv;
    float bad = 0.f;
    if (row < nrows) {
      bad = d1[i] * 0.f;
      T* dst = static_cast<T*>(p.out) + rowid(row) * DV;
#pragma unroll
      for (int c = 0; c < VC; ++c) {
        float o = o1[i][c] * (PROBE ? f1 : inv);
        if constexpr (PROBE) o = fmaf(-o2[i][c], inv, o);
        bad += o * 0.f;
        stf(dst, ((c / VW) * 16 + tx) * VW + c % VW, o);
      }
      if (p.lse && tx == 0)
        p.lse[rowid(row)] = d1[i] == 0.f ? -CUDART_INF_F : m[i] * p.inv_h + logf(d1[i]);
    }
    const unsigned hit = __ballot_sync(0xffffffffu, !(bad == 0.f));
    if (hit & 0xFFFFu) again |= 1u << i;
    if (hit >> 16) again |= 1u << (16 + i);
  }
  while (again) {  // the warp holds rows of two ty
    const int bit = __ffs(again) - 1, i = bit & 15;
    again &= again - 1;
    const int row = ((threadIdx.x >> 5) * 2 + (bit >> 4)) * RM + i;
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < RM; ++u)
      if (u == i) sum = d1[u];
    sum = __shfl_sync(0xffffffffu, sum, bit & 16);
    const long long id = rowid(row);
    repair_row<T, KT>(p, sq, b, p0, p1, (int)(id / p.Hq), (int)(id % p.Hq), sum);
  }
}

// mass[j] += sum over the rows that see key j of exp(s_j - lse): a block owns 64 keys of one
// key/value head and goes over the row tiles in order, so the sums do not depend on scheduling.
template <typename T, int D>
__global__ void __launch_bounds__(NT) mass_cc_kernel(Params p) {
  constexpr int BM = 64, RM = 4;
  using S = Smem<BM, D, 16, false>;
  extern __shared__ float sm[];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int hk = blockIdx.y, b = blockIdx.z, k0 = blockIdx.x * KT;
  const Seq sq = load_seq(p, b);
  if (k0 >= sq.len || !mine(p, sq.n)) return;
  const T* qg = static_cast<const T*>(p.q);
  const T* kg = static_cast<const T*>(p.k);
  stage<D, S::KP, KT, T>(sm + S::k, [&](int row) {
    const int j = k0 + row;
    const int pg = j < sq.len ? load_page(p, b, j >> p.page_shift) : -1;
    return pg < 0 ? (const T*)nullptr : kg + (((long long)pg * p.Hkv + hk) * p.page + (j & (p.page - 1))) * D;
  });
  const int rows = sq.n * p.g;
  float got[4] = {};
  for (int r0 = 0; r0 < rows; r0 += BM) {
    const int p0 = sq.first + r0 / p.g, p1 = sq.first + min(rows - 1, r0 + BM - 1) / p.g;
    if (p1 < k0 || !(k0 + KT > p0 - p.window || k0 < p.sinks)) continue;
    __syncthreads();
    stage<D, S::QP, BM, T>(sm + S::q, [&](int row) {
      const int x = r0 + row;
      return x < rows ? qg + ((long long)(sq.t0 + x / p.g) * p.Hq + hk * p.g + x % p.g) * D : (const T*)nullptr;
    });
    __syncthreads();
    float s[RM][4] = {};
    dots<RM, D, S::KP>(sm + S::q + ty * RM * S::QP, sm + S::k + tx * S::KP, s);
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const int x = r0 + ty * RM + i;
      if (x >= rows) continue;
      const float lse = subtrahend(p.lse[(long long)(sq.t0 + x / p.g) * p.Hq + hk * p.g + x % p.g]);
      const int pos = sq.first + x / p.g;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (visible(p, pos, k0 + tx + 16 * j)) got[j] += expf(fmaf(s[i][j], p.inv_h, -lse));
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j) sm[S::p + (tx + 16 * j) * S::PP + ty] = got[j];
  __syncthreads();
  if (threadIdx.x < KT) {
    const int j = k0 + threadIdx.x;
    if (j < sq.len) {
      float a = 0.f;
      for (int y = 0; y < 16; ++y) a += sm[S::p + threadIdx.x * S::PP + y];
      const int pg = load_page(p, b, j >> p.page_shift);
      if (pg >= 0) p.mass[((long long)pg * p.Hkv + hk) * p.page + (j & (p.page - 1))] += a;
    }
  }
}

// One warp per row: o and lse from the splits' {m, d1, d2}, O1 (and O2).
template <typename T, int DV, bool PROBE>
__global__ void __launch_bounds__(128) join_kernel(Params p) {
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)p.tokens * p.Hq;
  const long long id = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (id >= rows) return;
  const int token = (int)(id / p.Hq);
  int b = 0, e = p.B;  // the row's sequence: the last with starts[b] <= token
  while (e - b > 1) {
    const int mid = (b + e) / 2;
    if (p.starts[mid] <= token) b = mid;
    else e = mid;
  }
  const Seq sq = load_seq_or_tree(p, b);
  if (token < sq.t0 || token >= sq.t0 + sq.n || !mine(p, sq.n)) return;
  float m = -CUDART_INF_F;
  for (int s = lane; s < p.split; s += 32) m = fmaxf(m, p.part_s[s * rows + id].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float ref = m == -CUDART_INF_F ? 0.f : m;
  float d1 = 0.f, d2 = 0.f;
  constexpr int NC = (DV + 31) / 32;
  float o1[NC] = {}, o2[NC] = {};
#pragma unroll 4
  for (int s = 0; s < p.split; ++s) {
    const float4 st = p.part_s[s * rows + id];
    const float sc = expf((st.x - ref) * p.inv_h);  // 0 where the split saw nothing
    d1 = fmaf(st.y, sc, d1);
    d2 = fmaf(st.z, sc, d2);
    const float* src = p.part_o + (s * rows + id) * (PROBE ? 2 : 1) * DV;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (lane + 32 * c < DV) {
        o1[c] = fmaf(src[lane + 32 * c], sc, o1[c]);
        if (PROBE) o2[c] = fmaf(src[DV + lane + 32 * c], sc, o2[c]);
      }
  }
  const float inv = d1 == 0.f ? 0.f : 1.f / d1, f1 = (1.f + d2 * inv) * inv;
  T* dst = static_cast<T*>(p.out) + id * DV;
  float bad = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
    if (lane + 32 * c < DV) {
      float o = o1[c] * (PROBE ? f1 : inv);
      if (PROBE) o = fmaf(-o2[c], inv, o);
      bad += o * 0.f;
      stf(dst, lane + 32 * c, o);
    }
  if (p.lse && lane == 0) p.lse[id] = d1 == 0.f ? -CUDART_INF_F : m * p.inv_h + logf(d1);
  if (__any_sync(0xffffffffu, !(bad == 0.f))) {
    const int first = sq.first + (token - sq.t0) / 64 * 64;  // (a block's rows are at most 64 tokens)
    repair_row<T, KT>(p, sq, b, p.parents ? sq.first : max(first - 64, sq.first), min(first + 127, sq.len - 1), token,
                      (int)(id % p.Hq), d1);
  }
}

template <typename T, int D, int DV, bool PROBE, int BM>
cudaError_t launch_cc(const Params& p, cudaStream_t s) {
  auto kern = attend_cc_kernel<T, D, DV, PROBE, BM>;
  constexpr int bytes = Smem<BM, D, DV, PROBE>::bytes;
  static_assert(bytes <= 227 * 1024, "shared memory");
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err != cudaSuccess) return err;
  const int per = p.g < BM ? BM / p.g : 1, slices = (p.g + BM - 1) / BM;
  const long long blocks = ((long long)p.tokens / per + p.B) * slices * p.Hkv;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  kern<<<dim3((unsigned)blocks, p.split), NT, bytes, s>>>(p);
  count_launch();
  return cudaGetLastError();
}

template <typename T, int D, int DV>
cudaError_t pick_cc(const Params& p, cudaStream_t s) {
  const bool few = p.max_rows <= 16;
  if (p.r) return few ? launch_cc<T, D, DV, true, 16>(p, s) : launch_cc<T, D, DV, true, 64>(p, s);
  return few ? launch_cc<T, D, DV, false, 16>(p, s) : launch_cc<T, D, DV, false, 64>(p, s);
}

template <typename T, int D>
cudaError_t pick_dv(const Params& p, int dv, cudaStream_t s) {
  switch (dv) {
    case 16: return pick_cc<T, D, 16>(p, s);
    case 32: return pick_cc<T, D, 32>(p, s);
    case 64: return pick_cc<T, D, 64>(p, s);
    default: return pick_cc<T, D, 128>(p, s);
  }
}

template <typename T>
cudaError_t pick_d(const Params& p, int d, int dv, cudaStream_t s) {
  switch (d) {
    case 16: return pick_dv<T, 16>(p, dv, s);
    case 32: return pick_dv<T, 32>(p, dv, s);
    case 64: return pick_dv<T, 64>(p, dv, s);
    default: return pick_dv<T, 128>(p, dv, s);
  }
}

template <typename T, int D>
cudaError_t launch_mass_t(const Params& p, cudaStream_t s) {
  auto kern = mass_cc_kernel<T, D>;
  constexpr int bytes = Smem<64, D, 16, false>::bytes;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err != cudaSuccess) return err;
  const long long tiles = (((long long)p.max_pages << p.page_shift) + KT - 1) / KT;
  if (p.Hkv > 65535 || p.B > 65535) return cudaErrorInvalidConfiguration;
  kern<<<dim3((unsigned)tiles, p.Hkv, p.B), NT, bytes, s>>>(p);
  count_launch();
  return cudaGetLastError();
}

template <typename T>
cudaError_t pick_mass(const Params& p, int d, cudaStream_t s) {
  switch (d) {
    case 16: return launch_mass_t<T, 16>(p, s);
    case 32: return launch_mass_t<T, 32>(p, s);
    case 64: return launch_mass_t<T, 64>(p, s);
    default: return launch_mass_t<T, 128>(p, s);
  }
}

template <typename T, int DV>
cudaError_t launch_join_t(const Params& p, cudaStream_t s) {
  const long long blocks = ((long long)p.tokens * p.Hq + 3) / 4;
  if (p.r) join_kernel<T, DV, true><<<(unsigned)blocks, 128, 0, s>>>(p);
  else join_kernel<T, DV, false><<<(unsigned)blocks, 128, 0, s>>>(p);
  count_launch();
  return cudaGetLastError();
}

template <typename T>
cudaError_t pick_join(const Params& p, int dv, cudaStream_t s) {
  switch (dv) {
    case 16: return launch_join_t<T, 16>(p, s);
    case 32: return launch_join_t<T, 32>(p, s);
    case 64: return launch_join_t<T, 64>(p, s);
    default: return launch_join_t<T, 128>(p, s);
  }
}

}  // namespace
}  // namespace paged
}  // namespace lla
