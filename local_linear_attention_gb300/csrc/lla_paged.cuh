// The paged-cache operators (append, attention of a chunk of new tokens, eviction): problem
// description, the mask's key ranges and the row arithmetic their kernels share.
//
// Sequence b's position j lives in slot j % page_size of page table[b][j / page_size]; its new
// tokens starts[b] .. starts[b+1]-1 (rows of q, r, out: [tokens, q_heads, d]) are its last
// positions, pos = lens[b] - n + i. Query heads u of key/value head hk are hk*g .. hk*g + g-1, so
// the rows of a (sequence, key/value head) pair are numbered row = i*g + u: one key/value stream
// serves all of them.
#pragma once

#include <cuda.h>
#include <math_constants.h>

#include "lla_internal.cuh"

namespace lla {
namespace paged {

constexpr int kNoWindow = 1 << 30;  // lengths stay below this (checked on the host)

// Raises the dynamic shared memory limit of a kernel on the current device (lla_paged_api.cu).
cudaError_t ensure_smem(const void* kern, size_t bytes);

// Passed to kernels by value.
struct Params {
  const void* q;      // [tokens, Hq, d]
  const void* r;      // [tokens, Hq, d] or nullptr: softmax attention
  void* k;            // [num_pages, Hkv, page, d]
  void* v;            // [num_pages, Hkv, page, dv]
  float* mass;        // [num_pages, Hkv, page] or nullptr
  void* out;          // [tokens, Hq, dv]
  float* lse;         // [tokens, Hq] or nullptr
  const int* starts;  // [B + 1]
  const int* table;   // [B, max_pages]
  const int* lens;    // [B]
  int* status;
  int B, tokens, Hq, Hkv, g, d, dv;
  int page, page_shift, max_pages, num_pages;
  int window, sinks;  // window = kNoWindow when there is none
  float inv_h;
  int max_rows;       // most rows (new tokens x g) of any sequence, as the caller states
  int lo, hi;         // this launch takes the sequences with lo < rows <= hi
  int beside;         // few-rows kernel: launched behind the tensor-core kernel, may overlap it
  // Blocks that share a row's keys (tensor-core kernel: CTAs of the launch), and their partial
  // results: {m, d1, d2, d1 of the rounded weights (bf16 with a probe)} with m the reference of the
  // weights (raw q.k), and unnormalised O1 (and O2). CUDA cores and few rows (split > 1): [split][rows], rows = tokens * Hq with O rows of dv, or
  // B * Hkv * row_cap with O rows of D. Tensor cores: [CTA][2 slots][rows of a tile], O rows of D.
  int split;
  float* part_o;
  float4* part_s;
  int4* pieces;      // tensor-core kernel: [CTA][2 slots] {sequence, tile, head, there is one}
  float* logits;     // [B * Hkv][row_cap][keys_cap]  raw q.k of the few-rows kernel, by the key's
                     // place among the visible 16-key steps (weight tracking)
  int row_cap, keys_cap;
};

struct Seq {
  int t0, n;     // first new token's index, number of new tokens
  int len;       // positions in the cache, the new tokens included
  int first;     // position of the first new token (negative when n > len)
};

// Sequence b; one with impossible starts or length is treated as having no positions and no new tokens,
// and reported once per reader. (Cut to the nearest possible length instead, it would write to whatever
// its row of the table ends in.)
__device__ __forceinline__ Seq load_seq(const Params& p, int b) {
  Seq s;
  const int t0 = p.starts[b], t1 = p.starts[b + 1];
  const int len = p.lens[b], cap = p.max_pages << p.page_shift;
  const bool bad = t0 < 0 || t1 < t0 || t1 > p.tokens || len < 0 || len > cap;
  s.t0 = bad ? 0 : t0;
  s.n = bad ? 0 : t1 - t0;
  s.len = bad ? 0 : len;
  s.first = s.len - s.n;
  if (bad) atomicOr(p.status, kStatusBadIndex);
  return s;
}

// Page index of a position's page, or -1 (reported) when the table's entry is out of range.
__device__ __forceinline__ int load_page(const Params& p, int b, int slot) {
  const int pg = __ldg(p.table + (long long)b * p.max_pages + slot);
  if ((unsigned)pg < (unsigned)p.num_pages) return pg;
  atomicOr(p.status, kStatusBadIndex);
  return -1;
}

__device__ __forceinline__ bool visible(const Params& p, int pos, int j) {
  return j <= pos && (j > pos - p.window || j < p.sinks);
}

// The key tiles of KT positions that rows at positions p0 .. p1 see: tiles 0 .. n1-1 hold the
// first tokens, tiles w0 .. the window; count of both. tile(i) is the i-th of them.
template <int KT>
struct TileRange {
  int n1, w0, count;
  __device__ __forceinline__ TileRange(const Params& p, int p0, int p1) {
    const int kend = p1 + 1;
    const int wstart = max(0, p0 - p.window + 1);
    const int send = min(p.sinks, kend);
    n1 = (send + KT - 1) / KT;
    w0 = wstart / KT;
    if (w0 <= n1) n1 = w0 = 0;
    count = kend <= 0 ? 0 : n1 + (kend + KT - 1) / KT - w0;
  }
  __device__ __forceinline__ int tile(int i) const { return i < n1 ? i : w0 + i - n1; }
};
// Keys k0 .. k1-1 are visible to every row at positions p0 .. p1 (no mask needed).
__device__ __forceinline__ bool all_visible(const Params& p, int p0, int p1, int k0, int k1) {
  return k1 - 1 <= p0 && (k0 > p1 - p.window || k1 <= p.sinks);
}

// Whether sequence rows `n` x g are this launch's.
__device__ __forceinline__ bool mine(const Params& p, int n) {
  return n > 0 && n * p.g > p.lo && n * p.g <= p.hi;
}

// Row tiles of this launch's sequences, `per` tokens each: finds the sequence and tile of linear
// index `x` (every warp does the search by itself; all lanes return the same). False when x is
// past the last tile.
__device__ __forceinline__ bool find_tile(const Params& p, int per, int x, int* b_out, int* tile_out) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int base = 0; base < p.B; base += 32) {
    const int b = base + lane;
    int cnt = 0;
    if (b < p.B) {
      const int t0 = p.starts[b], t1 = p.starts[b + 1];
      if (t0 >= 0 && t1 > t0 && t1 <= p.tokens && mine(p, t1 - t0)) cnt = (t1 - t0 + per - 1) / per;
    }
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, x < before + incl);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int upto = __shfl_sync(0xffffffffu, incl, l), c = __shfl_sync(0xffffffffu, cnt, l);
      *b_out = base + l;
      // the last tiles of a prompt see the most keys: first
      *tile_out = c - 1 - (x - (before + upto - c));
      return true;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// What a weight exp(s - lse) of the finished row is taken with: a row without any weight (lse -infinity)
// gives none either, not even to keys whose logit is -infinity as well.
__device__ __forceinline__ float subtrahend(float lse) { return lse == -CUDART_INF_F ? CUDART_INF_F : lse; }

// One row computed by one warp straight from the definition, skipping every key that the row does
// not see (see repair_row). Slow, and off every ordinary path.
template <typename T>
__device__ __noinline__ void exact_row(const Params& p, int b, int pos, int token, int head) {
  const int d = p.d, dv = p.dv;
  const int lane = threadIdx.x & 31, hk = head / p.g;
  const T* q = static_cast<const T*>(p.q) + ((long long)token * p.Hq + head) * d;
  const T* r = p.r ? static_cast<const T*>(p.r) + ((long long)token * p.Hq + head) * d : nullptr;
  const T* kp = static_cast<const T*>(p.k);
  const T* vp = static_cast<const T*>(p.v);
  float m = -CUDART_INF_F, d1 = 0.f, d2 = 0.f, o1[4] = {}, o2[4] = {};
  const TileRange<32> range(p, pos, pos);
  for (int i = 0; i < range.count; ++i) {
    const int j = range.tile(i) * 32 + lane;
    const bool see = visible(p, pos, j);
    float s = -CUDART_INF_F, t = 0.f;
    long long slot = -1;
    if (see) {
      const int pg = load_page(p, b, j >> p.page_shift);
      s = 0.f;
      if (pg >= 0) {
        slot = ((long long)pg * p.Hkv + hk) * p.page + (j & (p.page - 1));
        for (int c = 0; c < d; ++c) {
          const float kv = ldf(kp, slot * d + c);
          s = fmaf(ldf(q, c), kv, s);
          if (r) t = fmaf(ldf(r, c), kv, t);
        }
      }
      s *= p.inv_h;
    }
    float tm = s;
    for (int o = 16; o; o >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, tm, o);
      tm = (tm != tm || y != y) ? CUDART_NAN_F : fmaxf(tm, y);
    }
    const float mn = (m != m || tm != tm) ? CUDART_NAN_F : fmaxf(m, tm);
    if (mn == -CUDART_INF_F) continue;
    const float sc = m == -CUDART_INF_F ? 0.f : expf(m - mn);
    const float w = see ? expf(s - mn) : 0.f, wt = see ? w * t : 0.f;
    m = mn;
    float a = w, e = wt;
    for (int o = 16; o; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      e += __shfl_xor_sync(0xffffffffu, e, o);
    }
    d1 = fmaf(d1, sc, a);
    d2 = fmaf(d2, sc, e);
    for (int c = 0; c < 4; ++c) { o1[c] *= sc; o2[c] *= sc; }
    for (int l = 0; l < 32; ++l) {
      const float wl = __shfl_sync(0xffffffffu, w, l), tl = __shfl_sync(0xffffffffu, wt, l);
      const long long sl = __shfl_sync(0xffffffffu, slot, l);
      if (sl < 0) continue;
      for (int c = 0; c < 4; ++c)
        if (lane + 32 * c < dv) {
          const float x = ldf(vp, sl * dv + lane + 32 * c);
          o1[c] = fmaf(wl, x, o1[c]);
          o2[c] = fmaf(tl, x, o2[c]);
        }
    }
  }
  const float inv = d1 == 0.f ? 0.f : 1.f / d1, f1 = (1.f + d2 * inv) * inv;
  T* out = static_cast<T*>(p.out) + ((long long)token * p.Hq + head) * dv;
  for (int c = 0; c < 4; ++c)
    if (lane + 32 * c < dv)
      stf(out, lane + 32 * c, r ? fmaf(o1[c], f1, -o2[c] * inv) : o1[c] * inv);
  if (p.lse && lane == 0)
    p.lse[(long long)token * p.Hq + head] = d1 == 0.f ? -CUDART_INF_F : m + logf(d1);
}

// Whether a key that the row at position `pos` does not see, in the KT-key tiles that its row block
// (positions p0 .. p1) goes over, has a value that is not finite. One warp.
template <typename T, int KT>
__device__ __noinline__ bool hides_bad(const Params& p, const Seq& sq, int b, int hk, int pos, int p0, int p1) {
  const int lane = threadIdx.x & 31;
  const TileRange<KT> range(p, p0, p1);
  const T* vp = static_cast<const T*>(p.v);
  for (int base = 0; base < range.count; base += 32) {
    const int k0 = base + lane < range.count ? range.tile(base + lane) * KT : 0;
    unsigned masked = __ballot_sync(0xffffffffu, base + lane < range.count && !all_visible(p, pos, pos, k0, k0 + KT));
    while (masked) {
      const int t0 = __shfl_sync(0xffffffffu, k0, __ffs(masked) - 1);
      masked &= masked - 1;
      bool bad = false;
      for (int j = t0; j < min(t0 + KT, sq.len); ++j) {
        if (visible(p, pos, j)) continue;
        const int pg = load_page(p, b, j >> p.page_shift);
        if (pg < 0) continue;
        const long long slot = ((long long)pg * p.Hkv + hk) * p.page + (j & (p.page - 1));
        for (int c = lane; c < p.dv; c += 32) bad |= !isfinite(ldf(vp, slot * p.dv + c));
      }
      if (__any_sync(0xffffffffu, bad)) return true;
    }
  }
  return false;
}

// A row that came out not finite (d1: its sum of weights), by one warp. The kernels multiply the values
// of keys that a row does not see by a zero weight, which is not zero when such a value is infinite
// or NaN; and a weight may pass the range of fp32 where the reference it is taken against is a step
// old (d1 is infinite then). Either way the row is taken again from the definition. A NaN sum of
// weights comes from a key that the row sees, and so does everything else that is not finite: those
// rows stay as they are.
template <typename T, int KT>
__device__ __forceinline__ void repair_row(const Params& p, const Seq& sq, int b, int pos, int p0, int p1, int token,
                                           int head, float d1) {
  __syncwarp();
  if (isnan(d1)) return;
  if (isinf(d1) || hides_bad<T, KT>(p, sq, b, head / p.g, pos, p0, p1)) exact_row<T>(p, b, pos, token, head);
}

// ------------------------------------------------------------------------------------- arithmetic
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The two values of a pair of bf16.
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// Packed pairs of fp32 (one instruction per pair on this architecture).
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// ------------------------------------------------------------------------------------- launches
// Launches `kern` on `s`. `smem` bytes of dynamic shared memory (the opt-in above 48 KB is set once
// per kernel and device: an attribute of the function, which stays); `cluster` blocks per cluster
// (1: none); `after`: the kernel may be set up while the stream's previous kernel drains, and waits
// itself (wait_previous) before it reads what that one wrote.
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, int cluster, bool after,
                   cudaStream_t s, Args&&... args) {
  if (smem > 40 * 1024) {  // 48 KB, less what the kernel declares
    cudaError_t err = ensure_smem(reinterpret_cast<const void*>(kern), smem);
    if (err != cudaSuccess) return err;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  int n = 0;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = (unsigned)cluster;
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
  }
  if (after) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, KArgs(args)...);
  if (err == cudaSuccess) count_launch();
  return err;
}
// A kernel that may be set up early: everything before this call may not touch what the previous
// kernel of the stream writes (or reads, where this one writes it).
__device__ __forceinline__ void wait_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// From here on the next kernel of the stream may be set up (it still waits for this one's end).
__device__ __forceinline__ void let_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launchers (each returns the launch error, if any).
// CUDA cores, every supported size (one set per type): the attention; mass += the rows' weights from
// q, k and the finished lse; the join of the splits' partial results into out and lse.
cudaError_t attend_cc_bf16(const Params& p, int d, int dv, cudaStream_t s);
cudaError_t mass_cc_f32(const Params& p, int d, cudaStream_t s);
cudaError_t mass_cc_bf16(const Params& p, int d, cudaStream_t s);
cudaError_t join_f32(const Params& p, int dv, cudaStream_t s);
cudaError_t join_bf16(const Params& p, int dv, cudaStream_t s);
inline cudaError_t launch_mass_cc(const Params& p, int d, int dtype, cudaStream_t s) {
  return dtype == LLA_F32 ? mass_cc_f32(p, d, s) : mass_cc_bf16(p, d, s);
}
inline cudaError_t launch_join(const Params& p, int dv, int dtype, cudaStream_t s) {
  return dtype == LLA_F32 ? join_f32(p, dv, s) : join_bf16(p, dv, s);
}
// The tensor-core kernels (bf16) are built for head sizes D = 64 and 128 and take smaller ones
// padded with zeros in shared memory: zero features add nothing to a product. D of a call:
inline int padded(int d) { return d > 64 ? 128 : 64; }
// Sequences of few rows (p.hi = rows_limit of them at most): the attention, the join of its splits
// and, with p.logits, the weight tracking. D = padded(max(d, dv)).
constexpr int kRowsCluster = 8;  // splits that join within a cluster (the portable size)
inline int rows_limit(bool probe) { return probe ? 8 : 16; }
cudaError_t launch_attend_rows(const Params& p, int D, cudaStream_t s);
// fp32: the attention of every sequence in tiles of kF32Rows rows, at most f32_tiles a key/value head;
// the weight tracking of the sequences of at most p.row_cap rows, whose logits are in p.logits.
constexpr int kF32Rows = 16, kF32MassRows = 256;
long long f32_tiles(long long tokens, long long max_new, int B, int g);
cudaError_t launch_attend_f32(const Params& p, long long tiles, int D, cudaStream_t s);
cudaError_t launch_mass_f32(const Params& p, cudaStream_t s);
// Sequences of many rows: the attention on p.split CTAs, the join of the tiles that their shares
// cut; the weight tracking (D = padded(d)).
struct TcPlan {
  int ctas = 0;            // 0: not for these kernels
  size_t rows = 0;         // rows of partial results (part_s, part_o), row_floats of part_o each
  int row_floats = 0;
  bool cuts = false;       // whether a tile may have enough steps to be cut
};
TcPlan plan_tc(int D, bool probe, long long tokens, int B, int Hkv, int g, long long keys);
cudaError_t launch_attend_tc(const Params& p, int D, cudaStream_t s);
cudaError_t launch_join_tc(const Params& p, int D, cudaStream_t s);
cudaError_t launch_mass_tc(const Params& p, int D, cudaStream_t s);
cudaError_t encode_query_map(const Params& p, const void* q, CUtensorMap* map);
cudaError_t encode_page_map(const Params& p, void* pages, int d, int kt, CUtensorMap* map);
cudaError_t launch_append(const Params& p, const void* k_new, const void* v_new, int d, int dv,
                          int dtype, cudaStream_t s);
// `p` is the source cache; the other arguments the destination and the choice.
cudaError_t launch_evict(const Params& p, void* k, void* v, float* mass, const int* table, int* lens,
                         int max_pages, int num_pages, int budget, int sinks, int recent, int* kept,
                         int d, int dv, int dtype, cudaStream_t s);

}  // namespace paged
}  // namespace lla
