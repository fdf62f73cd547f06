// Attention over a paged cache for sequences with many rows (prompts and chunks), bf16, d = dv = 64
// or 128, on the tensor cores (tcgen05, tensor memory, TMA).
//
// One pass over the keys with a running row maximum. Per 128-key tile a CTA runs two 128-row score
// products and two 128-row value products, X and Y:
//   softmax attention: X and Y are two blocks of 128 rows (tokens x grouped heads of one key/value
//     head), S = Q K^T, P = exp(S - m), O += P V, each block with its own softmax warpgroup, so one
//     block's exponentials run while the tensor core works for the other;
//   with a probe: X is Q, Y is R of the same 128 rows; P1 = exp(S_X - m), P2 = P1 .* S_Y, O1 += P1 V,
//     O2 += P2 V. Each warpgroup takes 64 of a tile's 128 keys; the row maximum goes through shared
//     memory.
// Warps 0-3 and 4-7: the two softmax warpgroups (a thread is a row, so row sums need no shuffles);
// 8: TMA loader (one lane per page fragment: a tile spans 128 / page_size pages; rows past the
// sequence's end and bad pages are loaded as zeros by an out-of-range coordinate); 9: MMA issuer.
// Tensor memory: S_X, S_Y (128 columns each), O_X, O_Y (d each); bf16 P has columns of its own at
// d = 64, and overwrites its S at d = 128 (512 columns are all there are), where the next S product
// is issued behind the P V product that reads them.
// The accumulators are rescaled only when a row's maximum grows by more than 2^8 (the weights then
// stay below 2^8, exact in scale; d1 is fp32): after the first tiles this hardly happens.
// Rounding: p and p t enter the value products as bf16, d1 and d2 sum the unrounded fp32 weights.
// What bounds it: the tensor pipe and the exponentials are near balance at d = 128 (2048 cycles of
// MMA against 2048 of ex2 per 256 rows x 128 keys).
// All mbarrier waits are bounded.
#include "lla_paged.cuh"
#include "lla_tc_ptx.cuh"
#include "lla_tmap.cuh"

namespace lla {
namespace paged {
namespace {

using namespace tc;

constexpr int BM = 128, KT = 128;
constexpr int NTHREADS = 320;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D>
struct Cfg {
  static constexpr int tile = BM * D * 2;        // bytes of a [128][D] bf16 tile: D/64 blocks of 16 KiB
  static constexpr int stages = D == 128 ? 4 : 8;
  static constexpr int sm_y = tile, sm_ring = 2 * tile;
  static constexpr int sm_bar = sm_ring + stages * tile;
  static constexpr int sm_x = sm_bar + 512;      // row exchange: [2 buffers][2 groups][128] maxima
  static constexpr int bytes = sm_x + 2048 + 1024;  // 1024: aligning the base
  static constexpr bool overlay = D == 128;
  static constexpr uint32_t t_o = 256, t_p = overlay ? 0 : 384, p_stride = overlay ? 128 : 64;
};
static_assert(Cfg<128>::bytes <= 227 * 1024 && Cfg<64>::bytes <= 227 * 1024, "shared memory");

struct Barriers {
  uint64_t full[8], empty[8];
  uint64_t sfull[2], sfree[2], pfull[2], pvdone[2];
  uint64_t rowx, done;
};
static_assert(sizeof(Barriers) <= 512, "barrier region");

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

template <int D, bool PROBE>
__global__ void __launch_bounds__(NTHREADS, 1)
attend_tc_kernel(Params p, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Barriers& bar = *reinterpret_cast<Barriers*>(smem + C::sm_bar);
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.x % p.Hkv, part = blockIdx.y;
  const int per = BM / p.g, tokens = PROBE ? per : 2 * per;  // tokens per block and per tile
  int b, tile;
  if (!find_tile(p, tokens, blockIdx.x / p.Hkv, &b, &tile)) return;
  const Seq sq = load_seq(p, b);
  const int tok0 = tile * tokens, ntok = min(tokens, sq.n - tok0);
  const int p0 = sq.first + tok0, p1 = p0 + ntok - 1;
  const TileRange<KT> range(p, p0, p1);
  const int chunk = (range.count + p.split - 1) / p.split;
  const int i0 = min(range.count, part * chunk), n = min(range.count, i0 + chunk) - i0;

  // Row r of block h: token and head; -1 when there is none.
  auto token_of = [&](int h, int r) {
    const int t = (PROBE ? 0 : h * per) + r / p.g;
    return r < per * p.g && t < ntok ? t : -1;
  };
  auto rowid = [&](int t, int r) -> long long {
    return (long long)(sq.t0 + tok0 + t) * p.Hq + hk * p.g + r % p.g;
  };

  // X and Y tiles in the 128-byte swizzled layout (rows that do not exist are zero).
  for (int e = tid; e < 2 * BM * (D / 8); e += NTHREADS) {
    const int h = e / (BM * (D / 8)), r = (e / (D / 8)) % BM, c = e % (D / 8);
    const int t = token_of(h, r);
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(PROBE && h ? p.r : p.q);
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (t >= 0) x = *reinterpret_cast<const uint4*>(src + rowid(t, r) * D + c * 8);
    *reinterpret_cast<uint4*>(smem + h * C::tile + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) * 16)) = x;
  }
  if (tid == 0) {
    for (int s = 0; s < C::stages; ++s) { mbar_init(&bar.full[s], 1); mbar_init(&bar.empty[s], 1); }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.sfull[s], 1);
      mbar_init(&bar.sfree[s], PROBE ? 8 : 4);
      mbar_init(&bar.pfull[s], PROBE ? 8 : 4);
      mbar_init(&bar.pvdone[s], 1);
    }
    mbar_init(&bar.rowx, 8);
    mbar_init(&bar.done, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&tmem_base_s, 512);
    tmem_relinquish();
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_base_s;
  volatile int* abort_p = &abort_flag;
  int* const status = p.status;
  constexpr int TO = kStatusTimeout;

  if (warp == 9) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0 && n > 0) {
      const uint64_t xd = smem_desc_sw128(smem_u32(smem), 1024);
      const uint64_t kd = smem_desc_sw128(smem_u32(smem + C::sm_ring), 1024);
      const uint64_t vd = smem_desc_sw128_mn(smem_u32(smem + C::sm_ring), 16384, 1024);
      constexpr uint32_t id_s = idesc_bf16(BM, KT, false, false);
      constexpr uint32_t id_o = idesc_bf16(BM, D, false, true);
      constexpr uint32_t tile16 = C::tile >> 4;
      auto stage = [](int i) { return (uint32_t)(i % C::stages); };
      auto parity = [](int i) { return (uint32_t)((i / C::stages) & 1); };
      auto scores = [&](int h, int i) {  // S_h = (X or Y) K_i^T
        const uint64_t a = xd + (uint64_t)(h * tile16), k = kd + (uint64_t)(stage(2 * i) * tile16);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t o = (s >> 2) * 1024 + (s & 3) * 2;
          mma_ss(tbase + h * 128, a + o, k + o, id_s, s > 0);
        }
        mma_commit(&bar.sfull[h]);
      };
      auto values = [&](int h, int i) {  // O_h += P_h V_i
        const uint64_t v = vd + (uint64_t)(stage(2 * i + 1) * tile16);
#pragma unroll
        for (int s = 0; s < KT / 16; ++s)
          mma_ts(tbase + C::t_o + h * D, tbase + C::t_p + h * C::p_stride + s * 8,
                 v + (uint64_t)(s * (2048 >> 4)), id_o, (i > 0 || s > 0) ? 1u : 0u);
        mma_commit(&bar.pvdone[h]);
      };
      auto wait = [&](uint64_t* x, uint32_t par) { return mbar_wait(x, par, status, TO, abort_p); };
      bool ok = wait(&bar.full[0], 0);
      if (ok) {
        tc_fence_after();
        scores(0, 0);
        scores(1, 0);
        mma_commit(&bar.empty[0]);
      }
      for (int i = 0; i < n && ok; ++i) {
        const bool more = i + 1 < n;
        if (more) ok = wait(&bar.full[stage(2 * i + 2)], parity(2 * i + 2));
        if (!C::overlay && more && ok) {
          // S has its own columns: the next scores as soon as the softmax has read these
          for (int h = 0; h < 2 && ok; ++h) {
            ok = wait(&bar.sfree[h], i & 1);
            tc_fence_after();
            if (ok) scores(h, i + 1);
          }
          if (ok) mma_commit(&bar.empty[stage(2 * i + 2)]);
        }
        ok = ok && wait(&bar.full[stage(2 * i + 1)], parity(2 * i + 1));
        for (int h = 0; h < 2 && ok; ++h) {
          if (!PROBE || h == 0) ok = wait(&bar.pfull[h], i & 1);
          if (!ok) break;
          tc_fence_after();
          values(h, i);
          if (h == 1) mma_commit(&bar.empty[stage(2 * i + 1)]);
          // P overwrote S: the next scores follow the product that reads P (MMAs run in order)
          if (C::overlay && more && !(PROBE && h == 0)) {
            if (PROBE) scores(0, i + 1);
            scores(h, i + 1);
            if (h == 1) mma_commit(&bar.empty[stage(2 * i + 2)]);
          }
        }
      }
      if (!ok) *abort_p = 1;
      mma_commit(&bar.done);
      volatile int never = 0;
      mbar_wait(&bar.done, 0, status, TO, &never);
    }
    __syncwarp();
  } else if (warp == 8) {
    // ------------------------------------------------------------------ K/V loader
    const int frag = min(p.page, KT), nfrag = KT / frag;
    if (lane == 0) {
      tma_prefetch_map(&kmap);
      tma_prefetch_map(&vmap);
    }
    int issued = 0;
    for (int i = 0; i < n; ++i) {
      const int j = range.tile(i0 + i) * KT + lane * frag;
      int c2 = p.num_pages * p.Hkv;  // out of range: zeros
      if (lane < nfrag && j < sq.len) {
        const int pg = load_page(p, b, j >> p.page_shift);
        if (pg >= 0) c2 = pg * p.Hkv + hk;
      }
      bool ok = true;
      for (int kv = 0; kv < 2 && ok; ++kv) {
        const int x = 2 * i + kv, st = x % C::stages;
        if (x >= C::stages) ok = warp_wait(&bar.empty[st], ((x / C::stages) - 1) & 1, status, TO, abort_p);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar.full[st], C::tile);
        __syncwarp();
        if (lane < nfrag) {
          uint8_t* dst = smem + C::sm_ring + st * C::tile + lane * frag * 128;
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(dst + c * 16384, kv ? &vmap : &kmap, c * 64, j & (p.page - 1), c2, &bar.full[st]);
        }
        issued = x + 1;
      }
      if (!ok) break;
    }
    // Nothing may land in this CTA's shared memory after it exits.
    if (lane == 0) {
      volatile int never = 0;
      for (int x = issued > C::stages ? issued - C::stages : 0; x < issued; ++x)
        mbar_wait(&bar.full[x % C::stages], (x / C::stages) & 1, status, TO, &never);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax + output
    const int grp = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = tbase + ((uint32_t)((warp & 3) * 32) << 16);
    const int h = PROBE ? 0 : grp;                 // which row block this thread's row is in
    const int t = token_of(h, r);
    const int pos = t >= 0 ? p0 + t : p1;          // rows that do not exist are not written
    const int q0 = PROBE ? p0 : min(p0 + h * per, p1), q1 = PROBE ? p1 : min(q0 + per - 1, p1);
    const float c2 = p.inv_h * kLog2e, slack = 8.f / c2;
    float m = -CUDART_INF_F, d1 = 0.f, d2 = 0.f;
    float* const xm = reinterpret_cast<float*>(smem + C::sm_x);
    int xphase = 0;  // phases of rowx used so far
    auto exchange = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.rowx);
      return warp_wait(&bar.rowx, (xphase++) & 1, status, TO, abort_p);
    };
    bool ok = true;
    constexpr int NC = PROBE ? 64 : 128;           // keys of a tile per thread
    for (int i = 0; i < n; ++i) {
      ok = warp_wait(&bar.sfull[h], i & 1, status, TO, abort_p);
      if (PROBE) ok = ok && warp_wait(&bar.sfull[1], i & 1, status, TO, abort_p);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[NC / 32][32], tt[PROBE ? 2 : 1][32];
#pragma unroll
      for (int c = 0; c < NC / 32; ++c) tmem_ld32(lanes + h * 128 + (PROBE ? grp * 64 : 0) + c * 32, s[c]);
      if constexpr (PROBE) {
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32(lanes + 128 + grp * 64 + c * 32, tt[c]);
      }
      tmem_ld_wait();
      if (!C::overlay) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar.sfree[h]);
          if (PROBE) mbar_arrive(&bar.sfree[1]);
        }
      }
      const int k0 = range.tile(i0 + i) * KT, kb = k0 + (PROBE ? grp * 64 : 0);
      if (!all_visible(p, q0, q1, k0, k0 + KT)) {
        // column c is visible when c <= hi and (c > lo or c < first)
        const int hi = pos - kb, lo = pos - p.window - kb, first = p.sinks - kb;
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (!(c <= hi && (c > lo || c < first))) s[c >> 5][c & 31] = 0xFF800000u;
      }
      float tm = -CUDART_INF_F;
#pragma unroll
      for (int c = 0; c < NC; ++c) tm = fmaxf(tm, __uint_as_float(s[c >> 5][c & 31]));
      if (PROBE) {
        float* buf = xm + (i & 1) * 256;
        buf[grp * 128 + r] = tm;
        if (!(ok = exchange())) break;  // also: both groups have read S_X and S_Y
        tm = fmaxf(buf[r], buf[128 + r]);
      }
      if (!C::overlay && i > 0) {
        // the products that read the previous P (overlay: they precede this S in the pipe)
        ok = warp_wait(&bar.pvdone[h], (i - 1) & 1, status, TO, abort_p);
        if (PROBE) ok = ok && warp_wait(&bar.pvdone[1], (i - 1) & 1, status, TO, abort_p);
        if (!ok) break;
        tc_fence_after();
      }
      const bool grow = tm > m + slack || (m == -CUDART_INF_F && tm > m);
      if (__any_sync(0xffffffffu, grow)) {
        float sc = 1.f;
        if (grow) {
          sc = ex2((m - tm) * c2);  // 0 from -infinity
          m = tm;
          d1 *= sc;
          d2 *= sc;
        }
        if (i > 0) {
          const uint32_t o = lanes + C::t_o + grp * D;  // with a probe: each group one accumulator
#pragma unroll
          for (int c = 0; c < D; c += 16) {
            uint32_t x[16];
            tmem_ld16(o + c, x);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * sc);
            tmem_st16(o + c, x);
          }
        }
      }
      const float ref = m == -CUDART_INF_F ? 0.f : m * c2;
#pragma unroll
      for (int c = 0; c < NC / 32; ++c) {
        uint32_t w[16], wt[PROBE ? 16 : 1];
        float sum = 0.f, sumt = 0.f;
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float y0 = ex2(fmaf(__uint_as_float(s[c][e]), c2, -ref));
          const float y1 = ex2(fmaf(__uint_as_float(s[c][e + 1]), c2, -ref));
          sum += y0 + y1;
          w[e / 2] = pack_bf16(y0, y1);
          if constexpr (PROBE) {
            const float z0 = s[c][e] == 0xFF800000u ? 0.f : y0 * __uint_as_float(tt[c][e]);
            const float z1 = s[c][e + 1] == 0xFF800000u ? 0.f : y1 * __uint_as_float(tt[c][e + 1]);
            sumt += z0 + z1;
            wt[e / 2] = pack_bf16(z0, z1);
          }
        }
        d1 += sum;
        d2 += sumt;
        tmem_st16(lanes + C::t_p + h * C::p_stride + (PROBE ? grp * 32 : 0) + c * 16, w);
        if constexpr (PROBE) tmem_st16(lanes + C::t_p + C::p_stride + grp * 32 + c * 16, wt);
      }
      if (k0 + KT > sq.len) {
        // the last page's slots past the sequence's end may hold anything: their weight is zero,
        // and so must be the values (both groups write the same zeros; the products wait for both)
        const int x = 2 * i + 1, st = x % C::stages;
        if (!(ok = warp_wait(&bar.full[st], (x / C::stages) & 1, status, TO, abort_p))) break;
        for (int e = tid & 127; e < (k0 + KT - sq.len) * (D / 8); e += 128) {
          const int row = sq.len - k0 + e / (D / 8), c = e % (D / 8);
          *reinterpret_cast<uint4*>(smem + C::sm_ring + st * C::tile + (c >> 3) * 16384 + row * 128 + (c & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.pfull[h]);
    }

    if (PROBE && ok) {  // the groups' sums
      float* buf = xm;
      ok = exchange();  // the last maxima have been read
      if (ok) {
        buf[grp * 128 + r] = d1;
        buf[256 + grp * 128 + r] = d2;
        ok = exchange();
        d1 = buf[r] + buf[128 + r];
        d2 = buf[256 + r] + buf[384 + r];
      }
    }
    if (ok && n > 0) {
      ok = warp_wait(&bar.pvdone[h], (n - 1) & 1, status, TO, abort_p);
      if (PROBE) ok = ok && warp_wait(&bar.pvdone[1], (n - 1) & 1, status, TO, abort_p);
      tc_fence_after();
    }
    if (ok) {
      const float inv = d1 == 0.f ? 0.f : 1.f / d1, f1 = (1.f + d2 * inv) * inv;
      const long long id = t >= 0 ? rowid(t, r) : 0;
      const long long pid = (long long)part * p.tokens * p.Hq + id;
      float bad = 0.f;
      constexpr int NO = PROBE ? D / 2 : D;  // output columns per thread
      const int c0 = PROBE ? grp * NO : 0;
#pragma unroll 1
      for (int c = c0; c < c0 + NO; c += 16) {
        uint32_t a[16], e[16];
        if (n > 0) {
          tmem_ld16(lanes + C::t_o + h * D + c, a);
          if (PROBE) tmem_ld16(lanes + C::t_o + D + c, e);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int u = 0; u < 16; ++u) a[u] = e[u] = 0u;
        }
        if (t < 0) continue;
        if (p.split > 1) {
          float* dst = p.part_o + pid * (PROBE ? 2 : 1) * D + c;
#pragma unroll
          for (int u = 0; u < 16; u += 4) {
            *reinterpret_cast<uint4*>(dst + u) = make_uint4(a[u], a[u + 1], a[u + 2], a[u + 3]);
            if (PROBE) *reinterpret_cast<uint4*>(dst + D + u) = make_uint4(e[u], e[u + 1], e[u + 2], e[u + 3]);
          }
          continue;
        }
        uint32_t w[8];
#pragma unroll
        for (int u = 0; u < 16; u += 2) {
          float y0 = __uint_as_float(a[u]) * (PROBE ? f1 : inv);
          float y1 = __uint_as_float(a[u + 1]) * (PROBE ? f1 : inv);
          if (PROBE) {
            y0 = fmaf(-__uint_as_float(e[u]), inv, y0);
            y1 = fmaf(-__uint_as_float(e[u + 1]), inv, y1);
          }
          bad += (y0 + y1) * 0.f;
          w[u / 2] = pack_bf16(y0, y1);
        }
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + id * D + c);
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
      if (t >= 0 && (!PROBE || grp == 0)) {
        if (p.split > 1) p.part_s[pid] = make_float4(m, d1, d2, 0.f);
        else if (p.lse) p.lse[id] = d1 == 0.f ? -CUDART_INF_F : (m * c2 + log2f(d1)) * kLn2;
      }
      if (p.split == 1) {
        // rows that are not finite, again by themselves (with a probe: once both groups have
        // written their columns, by the first)
        if (PROBE) {
          ok = exchange();  // the sums have been read
          if (ok) xm[grp * 128 + r] = bad;
          ok = ok && exchange();
          bad = xm[r] + xm[128 + r];
        }
        unsigned again = __ballot_sync(0xffffffffu, ok && t >= 0 && !(bad == 0.f) && (!PROBE || grp == 0));
        while (again) {
          const int row = (warp & 3) * 32 + __ffs(again) - 1;
          again &= again - 1;
          const int tk = token_of(h, row);
          __syncwarp();
          exact_row<__nv_bfloat16>(p, D, D, b, p0 + tk, sq.t0 + tok0 + tk, hk * p.g + row % p.g);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D, bool PROBE>
cudaError_t launch_tc_t(const Params& p, cudaStream_t s) {
  CUtensorMap kmap, vmap;
  cudaError_t err = encode_page_map(p, p.k, D, &kmap);
  if (err == cudaSuccess) err = encode_page_map(p, p.v, D, &vmap);
  if (err != cudaSuccess) return err;
  auto kern = attend_tc_kernel<D, PROBE>;
  err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::bytes);
  if (err != cudaSuccess) return err;
  const int per = BM / p.g * (PROBE ? 1 : 2);
  const long long blocks = ((long long)p.tokens / per + p.B) * p.Hkv;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  kern<<<dim3((unsigned)blocks, p.split), NTHREADS, Cfg<D>::bytes, s>>>(p, kmap, vmap);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

// Tensor map of the pages ([num_pages * Hkv][page][d] bf16; boxes of one page fragment x 64
// features, 128-byte swizzled).
cudaError_t encode_page_map(const Params& p, void* pages, int d, CUtensorMap* map) {
  auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint32_t ones[3] = {1, 1, 1};
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)p.page, (cuuint64_t)p.num_pages * p.Hkv};
  const cuuint64_t str[2] = {(cuuint64_t)d * 2, (cuuint64_t)p.page * d * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)(p.page < 128 ? p.page : 128), 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, pages, dims, str, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

cudaError_t launch_attend_tc(const Params& p, int d, cudaStream_t s) {
  if (p.r) return d == 128 ? launch_tc_t<128, true>(p, s) : launch_tc_t<64, true>(p, s);
  return d == 128 ? launch_tc_t<128, false>(p, s) : launch_tc_t<64, false>(p, s);
}

}  // namespace paged
}  // namespace lla
