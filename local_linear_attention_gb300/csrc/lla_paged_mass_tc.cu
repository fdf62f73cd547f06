// Weight tracking of sequences with many rows, bf16, d up to D = 64 or 128, on the tensor cores:
//   mass[j] += sum over the rows i that see key j of exp(q_i.k_j / h - lse_i),
// from the finished lse. The product is taken transposed, S^T = K Q^T (128 keys x 128 rows in
// tensor memory, a thread per key), so that a key's sum runs along a thread's registers: no
// shuffles, no atomics, and a CTA that owns its keys adds its row blocks up in one fixed order.
// What bounds it: the exponentials, one per (row, key) pair (32 a cycle and SM); the product is
// half as long. Two CTAs a SM (two score buffers each) hide each other's waits.
// Measured: prompts B4 T4096, 8 heads of 64, 68 us (268 M row-key pairs, 3.9 T a second; the limit of
// the exponentials would be 27 us). Half a block's scores per buffer, so that the product refills one
// while the other is read, was slower: its N = 64 products take about as long as N = 128 ones.
// An item is a 128-key tile of one key/value head; CTAs take items in turn (their number depends on
// the lengths, which only the device knows), those with the most rows first where the sequences are few
// (prompts B4 T4096: the busiest CTA had 1.65 times the mean in the order of the sequences, 75 us).
// Warps 0-3 and 4-7: two consumer groups, alternate row blocks; 8: TMA loader (keys by page fragment; queries as [per tokens][g heads] boxes, rows in the
// order token * g + head); 9: MMA issuer. All mbarrier waits are bounded.
#include "lla_paged.cuh"
#include "lla_tc_ptx.cuh"
#include "lla_tmap.cuh"

namespace lla {
namespace paged {
namespace {

using namespace tc;

constexpr int KT = 128, BR = 128;
constexpr int NTHREADS = 320;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Cfg {
  static constexpr int tile = KT * D * 2;
  static constexpr int sm_q = tile;                  // two stages of row blocks
  static constexpr int sm_lse = 3 * tile;            // [8 warps][128] -lse * log2(e)
  static constexpr int sm_sum = sm_lse + 8 * BR * 4; // [2][2 groups][128]
  static constexpr int sm_bar = sm_sum + 2 * 2 * KT * 4;
  static constexpr int bytes = sm_bar + 128 + 1024;
};
static_assert(2 * (Cfg<128>::bytes + 1024) <= 227 * 1024, "two CTAs a SM");

struct Barriers {
  uint64_t kfull, qfull[2], qempty[2], sfull[2], sfree[2], done;
};
static_assert(sizeof(Barriers) <= 128, "barrier region");

// Key tiles of sequence b, if it is this launch's.
__device__ __forceinline__ int key_tiles(const Params& p, int b) {
  if (b >= p.B) return 0;
  const int t0 = p.starts[b], t1 = p.starts[b + 1];
  return t0 >= 0 && t1 > t0 && t1 <= p.tokens && mine(p, t1 - t0)
             ? (min(max(p.lens[b], 0), p.max_pages << p.page_shift) + KT - 1) / KT
             : 0;
}

// Key tiles of up to 32 sequences, the first tiles of all before the second ones: a prompt's first keys
// have the most rows, so the work of a tile declines along this order. A lane has its sequence's `count`
// and `below`, how many tiles come before tile number `count`.
struct Ranks {
  int count, below;
  __device__ __forceinline__ explicit Ranks(int n) : count(n), below(0) {
    for (int l = 0; l < 32; ++l) below += min(count, __shfl_sync(0xffffffffu, count, l));
  }
  __device__ __forceinline__ bool find(int x, int* b_out, int* tile_out) const {
    // sequences that end before x; between two ends every tile number has the same sequences
    const bool ended = below <= x;
    const int from = (int)__reduce_max_sync(0xffffffffu, ended ? (unsigned)count : 0u);
    const int at = (int)__reduce_max_sync(0xffffffffu, ended ? (unsigned)below : 0u);
    unsigned there = __ballot_sync(0xffffffffu, count > from);
    if (!there) return false;
    const int n = __popc(there);
    *tile_out = from + (x - at) / n;
    for (int skip = (x - at) % n; skip > 0; --skip) there &= there - 1;
    *b_out = __ffs(there) - 1;
    return true;
  }
};

// Key tile `x` of this launch's sequences (as find_tile, over keys).
__device__ __forceinline__ bool find_keys(const Params& p, int x, int* b_out, int* tile_out) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int base = 0; base < p.B; base += 32) {
    const int cnt = key_tiles(p, base + lane);
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
      *tile_out = x - (before + upto - c);  // the first keys of a prompt have the most rows: first
      return true;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// Whether key j, whose sum came out NaN, is not finite itself: its products with the zero rows past a
// block's `width` are NaN then, whatever its weights are.
__device__ __noinline__ bool infinite_key(const Params& p, int b, int hk, int j) {
  const int pg = load_page(p, b, j >> p.page_shift);
  bool finite = true;
  const long long at = (((long long)pg * p.Hkv + hk) * p.page + (j & (p.page - 1))) * p.d;
  for (int c = 0; c < p.d && pg >= 0; ++c) finite &= isfinite(ldf(static_cast<const __nv_bfloat16*>(p.k), at + c)) != 0;
  return !finite;
}
// The sum of such a key over every second block of `per` tokens, from token tok0 to before tok1, row by row;
// one warp.
__device__ __noinline__ float key_again(const Params& p, const Seq& sq, int b, int hk, int j, int tok0, int tok1, int per) {
  const int pg = load_page(p, b, j >> p.page_shift);
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k) + (((long long)pg * p.Hkv + hk) * p.page + (j & (p.page - 1))) * p.d;
  float sum = 0.f;
  for (; tok0 < tok1; tok0 += 2 * per)
    for (int r = threadIdx.x & 31; r < min(per, tok1 - tok0) * p.g; r += 32) {
      if (!visible(p, sq.first + tok0 + r / p.g, j)) continue;
      const long long row = (long long)(sq.t0 + tok0 + r / p.g) * p.Hq + hk * p.g + r % p.g;
      float s = 0.f;
      for (int c = 0; c < p.d; ++c) s = fmaf(ldf(static_cast<const __nv_bfloat16*>(p.q), row * p.d + c), ldf(k, c), s);
      sum += ex2((s * p.inv_h - subtrahend(p.lse[row])) * kLog2e);
    }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 2)
mass_tc_kernel(Params p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Barriers& bar = *reinterpret_cast<Barriers*>(smem + C::sm_bar);
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int per = BR / p.g, width = per * p.g;  // tokens and rows of a block
  int* const status = p.status;
  constexpr int TO = kStatusTimeout;

  // The rows past `width` of the row-block stages are never loaded: zeros.
  for (int e = tid; e < 2 * (D / 64) * (BR - width) * 8; e += NTHREADS) {
    const int c = e & 7, row = width + (e >> 3) % (BR - width), half = (e >> 3) / (BR - width);
    *reinterpret_cast<uint4*>(smem + C::sm_q + half * 16384 + row * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  if (tid == 0) {
    mbar_init(&bar.kfull, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.qfull[s], 1);
      mbar_init(&bar.qempty[s], 1);
      mbar_init(&bar.sfull[s], 1);
      mbar_init(&bar.sfree[s], 4);
    }
    mbar_init(&bar.done, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&tmem_base_s, 256);
    tmem_relinquish();
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = __shfl_sync(0xffffffffu, tmem_base_s, 0);
  volatile int* abort_p = &abort_flag;

  int lse_tok[4], lse_head[4];  // of rows lane, lane + 32, ..: token within the block, grouped head
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int row = u * 32 + lane;
    lse_tok[u] = row < width ? row / p.g : -1;
    lse_head[u] = row % p.g;
  }
  int done = 0, items = 0;  // row blocks and items so far (every thread counts the same)
  bool used = false;
  const bool ranked = p.B <= 32;
  const Ranks ranks(ranked ? key_tiles(p, lane) : 0);
  for (int turn = 0;; ++turn) {
    // rows of one item per CTA that run back and forth, which levels a steady decline
    const int x = turn * gridDim.x + (turn & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    int b, tile;
    if (!(ranked ? ranks.find(x / p.Hkv, &b, &tile) : find_keys(p, x / p.Hkv, &b, &tile))) break;
    const int hk = x % p.Hkv;
    const Seq sq = load_seq(p, b);
    const int k0 = tile * KT;
    // blocks of rows that see any of these keys
    const int from = max(0, k0 - sq.first) / per;
    int last = sq.n - 1;
    if (k0 >= p.sinks) last = (int)min((long long)last, (long long)k0 + KT - 2 + p.window - sq.first);
    const int nblk = last < 0 ? 0 : last / per - from + 1;
    if (nblk <= 0) continue;
    used = true;

    if (warp == 9) {
      // Warp-uniform, only the instructions under elect_one() (see lla_paged_tc.cu).
      const uint64_t kd = smem_desc_sw128(smem_u32(smem), 1024);
      const uint64_t qd = smem_desc_sw128(smem_u32(smem + C::sm_q), 1024);
      constexpr uint32_t id = idesc_bf16(KT, BR, false, false);
      auto wait = [&](uint64_t* x, uint32_t par) { return warp_wait(x, par, status, TO, abort_p); };
      const int first = __shfl_sync(0xffffffffu, done, 0), count = __shfl_sync(0xffffffffu, nblk, 0);
      bool ok = wait(&bar.kfull, items & 1);
      for (int i = 0; i < count && ok; ++i) {
        const int c = first + i, st = c & 1;
        ok = wait(&bar.qfull[st], (c >> 1) & 1) && (c < 2 || wait(&bar.sfree[st], ((c >> 1) - 1) & 1));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t o = (s >> 2) * 1024 + (s & 3) * 2;
            mma_ss(tbase + st * BR, kd + o, qd + (uint64_t)(st * (C::tile >> 4)) + o, id, s > 0);
          }
          mma_commit(&bar.sfull[st]);
          mma_commit(&bar.qempty[st]);
        }
        __syncwarp();
      }
      if (!ok) *abort_p = 1;
      __syncwarp();
    } else if (warp == 8) {
      const int frag = min(p.page, KT), nfrag = KT / frag;
      const int j = k0 + lane * frag;
      int c2 = p.num_pages * p.Hkv;  // out of range: zeros
      if (lane < nfrag && j < sq.len) {
        const int pg = load_page(p, b, j >> p.page_shift);
        if (pg >= 0) c2 = pg * p.Hkv + hk;
      }
      if (lane == 0) mbar_arrive_expect_tx(&bar.kfull, C::tile);
      __syncwarp();
      if (lane < nfrag)
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(smem + c * 16384 + lane * frag * 128, &kmap, c * 64, j & (p.page - 1), c2, &bar.kfull);
      if (lane == 0) {
        int issued = 0;
        for (int i = 0; i < nblk; ++i) {
          const int c = done + i, st = c & 1;
          if (c >= 2 && !mbar_wait(&bar.qempty[st], ((c >> 1) - 1) & 1, status, TO, abort_p)) break;
          mbar_arrive_expect_tx(&bar.qfull[st], width * D * 2);
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(smem + C::sm_q + st * C::tile + h * 16384, &qmap, h * 64, hk * p.g,
                        sq.t0 + (from + i) * per, &bar.qfull[st]);
          issued = i + 1;
        }
        // the copies of this item have landed before the CTA goes on (or leaves)
        volatile int never = 0;
        mbar_wait(&bar.kfull, items & 1, status, TO, &never);
        for (int i = max(0, issued - 2); i < issued; ++i) {
          const int c = done + i;
          mbar_wait(&bar.qfull[c & 1], (c >> 1) & 1, status, TO, &never);
        }
      }
      __syncwarp();
    } else {
      const int grp = warp >> 2, r = (warp & 3) * 32 + lane;
      const uint32_t lanes = tbase + ((uint32_t)((warp & 3) * 32) << 16);
      float* const lse = reinterpret_cast<float*>(smem + C::sm_lse) + warp * BR;
      const float c2 = p.inv_h * kLog2e;
      const int j = k0 + r;
      float got = 0.f;
      auto release = [&](int buf) {  // the scores have been read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.sfree[buf]);
      };
      // -lse log2(e) of a block's rows, four to a lane (-infinity past the rows there are); loaded a
      // block ahead, so that its latency is not in front of the sums
      float ahead[4];
      auto load_lse = [&](int i) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int t = (from + i) * per + lse_tok[u];
          ahead[u] = i < nblk && lse_tok[u] >= 0 && t < sq.n
                         ? subtrahend(p.lse[(long long)(sq.t0 + t) * p.Hq + hk * p.g + lse_head[u]]) * -kLog2e
                         : -CUDART_INF_F;
        }
      };
      load_lse((done ^ grp) & 1);
      for (int i = (done ^ grp) & 1; i < nblk; i += 2) {  // block counts of this group's parity
        const int c = done + i, tok0 = (from + i) * per;
#pragma unroll
        for (int u = 0; u < 4; ++u) lse[u * 32 + lane] = ahead[u];
        __syncwarp();
        load_lse(i + 2);
        if (!warp_wait(&bar.sfull[grp], (c >> 1) & 1, status, TO, abort_p)) break;
        tc_fence_after();
        const int p0 = sq.first + tok0, p1 = p0 + per - 1;
        // (the columns past `width` are products with zero rows, with -lse = -infinity: nothing, unless the
        // key is infinite, see key_again)
        const bool full = tok0 + per <= sq.n && all_visible(p, p0, p1, k0, k0 + KT);
        uint32_t s[2][32];
        tmem_ld32(lanes + grp * BR, s[0]);
        if (full) {
          // the next 32 columns are on their way while these are added up
          uint64_t a[2] = {};
          const uint64_t c22 = pair(c2, c2);
#pragma unroll
          for (int q = 0; q < BR / 32; ++q) {
            tmem_ld_wait();
            if (q + 1 < BR / 32) tmem_ld32(lanes + grp * BR + (q + 1) * 32, s[(q + 1) & 1]);
            else release(grp);
            const uint32_t(&x)[32] = s[q & 1];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 l = *reinterpret_cast<const float4*>(lse + q * 32 + e);
              float y[4];
              unpair(fma2(pair(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), c22, pair(l.x, l.y)), y[0], y[1]);
              unpair(fma2(pair(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), c22, pair(l.z, l.w)), y[2], y[3]);
              a[0] = add2(a[0], pair(ex2(y[0]), ex2(y[1])));
              a[1] = add2(a[1], pair(ex2(y[2]), ex2(y[3])));
            }
          }
          float y0, y1;
          unpair(add2(a[0], a[1]), y0, y1);
          got += y0 + y1;
        } else {
          // The rows that see key j are a range: e0 <= row < e1. As bits, then a select each (a branch per
          // row took several times as long).
          const long long g = p.g, end = j < p.sinks ? width : ((long long)j + p.window - p0) * g;
          const int e0 = (int)min(max(((long long)j - p0) * g, 0ll), (long long)BR);
          const int e1 = (int)min(max(end, 0ll), min((long long)width, (long long)(sq.n - tok0) * g));
          auto below = [](int x) { return x <= 0 ? 0u : x >= 32 ? 0xFFFFFFFFu : (1u << x) - 1u; };
          float a[2] = {};
#pragma unroll
          for (int q = 0; q < BR / 32; ++q) {
            tmem_ld_wait();
            if (q + 1 < BR / 32) tmem_ld32(lanes + grp * BR + (q + 1) * 32, s[(q + 1) & 1]);
            else release(grp);
            const unsigned seen = below(e1 - q * 32) & ~below(e0 - q * 32);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float y = ex2(fmaf(__uint_as_float(s[q & 1][e]), c2, lse[q * 32 + e]));
              a[e & 1] += seen & (1u << e) ? y : 0.f;
            }
          }
          got += a[0] + a[1];
        }
      }
      if (width < BR) {
        unsigned again = __ballot_sync(0xffffffffu, got != got && j < sq.len && infinite_key(p, b, hk, j));
        for (; again; again &= again - 1) {
          const int l = __ffs(again) - 1, first = from + ((done ^ grp) & 1);
          const float sum = key_again(p, sq, b, hk, j - lane + l, first * per, min(sq.n, (from + nblk) * per), per);
          if (lane == l) got = sum;
        }
      }
      reinterpret_cast<float*>(smem + C::sm_sum)[((items & 1) * 2 + grp) * KT + r] = got;
    }
    __syncthreads();  // the item's sums are there, its scores have been read
    if (*abort_p) break;
    if (tid < KT && k0 + tid < sq.len) {
      const float* sum = reinterpret_cast<const float*>(smem + C::sm_sum) + (items & 1) * 2 * KT;
      const int j = k0 + tid, pg = load_page(p, b, j >> p.page_shift);
      if (pg >= 0) p.mass[((long long)pg * p.Hkv + hk) * p.page + (j & (p.page - 1))] += sum[tid] + sum[KT + tid];
    }
    done += nblk;
    ++items;
  }
  if (warp == 9 && used) {  // after an abort there may be products in flight
    if (elect_one()) mma_commit(&bar.done);
    __syncwarp();
    volatile int never = 0;
    mbar_wait(&bar.done, 0, status, TO, &never);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 256);
  }
}

template <int D>
cudaError_t launch_t(const Params& p, cudaStream_t s) {
  CUtensorMap kmap, qmap;
  cudaError_t err = encode_page_map(p, p.k, p.d, KT, &kmap);
  if (err != cudaSuccess) return err;
  err = encode_query_map(p, p.q, &qmap);
  if (err != cudaSuccess) return err;
  const long long most = ((((long long)p.max_pages << p.page_shift) + KT - 1) / KT) * p.B * p.Hkv;
  return launch(mass_tc_kernel<D>, dim3((unsigned)(most < 304 ? most : 304)), NTHREADS, Cfg<D>::bytes, 1, false, s,
                p, kmap, qmap);
}

}  // namespace

cudaError_t launch_mass_tc(const Params& p, int D, cudaStream_t s) {
  return D == 128 ? launch_t<128>(p, s) : launch_t<64>(p, s);
}

}  // namespace paged
}  // namespace lla
