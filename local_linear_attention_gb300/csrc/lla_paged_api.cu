// C ABI of the paged-cache operators: argument validation, choice of kernels and splits, scratch.
#include <cmath>

#include "lla_paged.cuh"
#include "lla_smem_limits.h"

namespace lla {
namespace paged {

cudaError_t ensure_smem(const void* kern, size_t bytes) {
  static SmemLimits limits;
  int dev = 0;
  const cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  return limits.ensure(
      kern, dev, bytes,
      [&](size_t* held) {
        cudaFuncAttributes at;
        const cudaError_t e = cudaFuncGetAttributes(&at, kern);
        if (e == cudaSuccess) *held = (size_t)at.maxDynamicSharedSizeBytes;
        return e;
      },
      [&](size_t most) { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most); });
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool head_size(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// Fields of the cache description that do not depend on pointers.
int check_cache_shape(const lla_paged_cache* c) {
  if (!c) return LLA_ERR_INVALID_ARG;
  if (c->num_seqs < 0 || c->kv_heads <= 0 || c->max_pages < 0 || c->num_pages < 0)
    return LLA_ERR_INVALID_ARG;
  if (c->dtype != LLA_F32 && c->dtype != LLA_BF16) return LLA_ERR_INVALID_ARG;
  for (int r : c->reserved)
    if (r != 0) return LLA_ERR_INVALID_ARG;
  if (!head_size(c->d) || !head_size(c->dv)) return LLA_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
    return LLA_ERR_UNSUPPORTED;
  if ((long long)c->max_pages * c->page_size >= kNoWindow) return LLA_ERR_UNSUPPORTED;
  if ((long long)c->num_pages * c->kv_heads >= (1LL << 31)) return LLA_ERR_UNSUPPORTED;
  if (c->num_seqs > 65535 || c->kv_heads > 65535 || (long long)c->num_seqs * c->kv_heads >= (1LL << 28))
    return LLA_ERR_UNSUPPORTED;
  return LLA_OK;
}

int check_cache_pointers(const lla_paged_cache* c, bool need_mass) {
  if (!c->k_pages || !c->v_pages || !c->page_table || !c->lens) return LLA_ERR_INVALID_ARG;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages)) return LLA_ERR_INVALID_ARG;
  if (need_mass && (!c->mass || !aligned16(c->mass))) return LLA_ERR_INVALID_ARG;
  return LLA_OK;
}

Params cache_params(const lla_paged_cache* c) {
  Params p = {};
  p.k = c->k_pages;
  p.v = c->v_pages;
  p.mass = c->mass;
  p.table = c->page_table;
  p.lens = c->lens;
  p.B = c->num_seqs;
  p.Hkv = p.Hq = c->kv_heads;
  p.g = 1;
  p.page = c->page_size;
  while ((1 << p.page_shift) < c->page_size) ++p.page_shift;
  p.d = c->d;
  p.dv = c->dv;
  p.max_pages = c->max_pages;
  p.num_pages = c->num_pages;
  p.window = kNoWindow;
  p.split = 1;
  p.hi = 0x7fffffff;
  return p;
}

int check_query(const lla_paged_cache* c, const lla_paged_query* a) {
  int st = check_cache_shape(c);
  if (st != LLA_OK) return st;
  if (!a || a->tokens < 0 || a->max_new < 0 || a->q_heads <= 0 || a->window < 0 || a->sinks < 0)
    return LLA_ERR_INVALID_ARG;
  for (int r : a->reserved)
    if (r != 0) return LLA_ERR_INVALID_ARG;
  if (!(std::isfinite(a->h) && a->h > 0.f)) return LLA_ERR_INVALID_ARG;
  if (a->path < LLA_PATH_AUTO || a->path > LLA_PATH_TENSOR_CORE) return LLA_ERR_INVALID_ARG;
  if (a->q_heads % c->kv_heads != 0) return LLA_ERR_INVALID_ARG;
  if ((long long)a->tokens * a->q_heads >= (1LL << 31) || a->tokens >= kNoWindow)
    return LLA_ERR_UNSUPPORTED;
  return LLA_OK;
}

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// The weights of sequences of few rows come from the logits that the attention leaves in scratch, sized
// by the table's capacity. Above this much scratch they are computed again from q and k, as those of
// longer sequences are. (32 sequences of 4k to 16k, 32 heads over 8 of 128: 249 us with a table as wide as
// the longest, 289 with one of 262144 positions and 1 GiB of logits, 493 computed again; 16 of 2k to 4k in
// fp32, 16 heads over 4: 53, 335 with a table of a million, 1224 computed again.)
constexpr size_t kMostLogits = (size_t)1 << 31;

// How one call runs: the kernels it takes, their splits and scratch (byte offsets).
struct Plan {
  bool rows = false;   // the few-rows kernel takes the sequences of at most rows_limit rows
  bool tiles = false;  // a tiled kernel the others: tensor cores (tc) or CUDA cores
  long long f32 = 0;   // fp32: one kernel's tiles; `rows` and `tiles` are the weight tracking's parts
  bool tc = false;
  bool join = false;   // tensor cores: tiles may be cut
  bool logits_kept = false;  // weight tracking: of the sequences of at most row_cap rows from their logits
  bool mass_tc = false;      // of the others (or all) on the tensor cores
  int D = 0;           // head size of the tensor-core kernels
  int rows_split = 1, tiles_split = 1;
  int row_cap = 0, keys_cap = 0;
  size_t rows_s = 0, rows_o = 0, logits = 0, pieces = 0, tiles_s = 0, tiles_o = 0, lse = 0;
  size_t bytes = 0;
};

// Blocks to a tile of the fp32 kernel: the number with the least time of a block (its keys in rounds of
// 128, its start, and beyond a cluster the join through scratch) times the waves of blocks, in halves:
// two blocks fit an SM and share its FMAs. Clusters stay within a GPC (19 SMs), whose slots their size
// may not divide. Measured: 42 sequences of 3.5k, window 1052, 2 heads, 21 us with the 3 that it takes, 26
// with 2, 30 with 4; 62 of 12k to 18k, 2 heads, 1.00 ms as it takes, 1.21 with 2, 1.29 with 64; 7 of 16k to
// 24k, 96 us with 64, 184 with 16. It is not always the best: 34 of 10k, one tile each, with weights, 178 us,
// 146 with 20; 10 of 11k to 23k with weights 224, 190 with 20.
int f32_splits(long long tiles, long long keys, long long rows, int D, bool probe) {
  if (tiles <= 0) return 1;
  const double rate = 8.0 * 16 / (rows < 4 ? 4 : rows > 16 ? 16 : rows) * 128 / D * (probe ? 1 : 1.6);  // keys a us
  const double start = 8 * rate, join = 4 * rate;
  long long most = keys / 128 < 64 ? keys / 128 : 64;
  if (most > 16 * 304 / tiles) most = 16 * 304 / tiles;
  int best = 1;
  double least = 0;
  for (int n = 1; n == 1 || n <= most; ++n) {
    const int slots = n == 1 || n > kRowsCluster ? 304 : 8 * (38 / n * n);
    const long long halves = (2 * tiles * n + slots - 1) / slots;
    const double waves = halves < 2 ? 1 : halves * 0.5;
    const long long rounds = ((keys + n - 1) / n + 127) / 128;
    const double cost = waves * (rounds * 128 + start) + (n > kRowsCluster ? join : 0);
    if (n == 1 || cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

Plan make_plan(const lla_paged_cache* c, const lla_paged_query* a) {
  Plan pl;
  const int g = a->q_heads / c->kv_heads;
  const long long cap = (long long)c->max_pages * c->page_size;
  const long long max_new = a->max_new < a->tokens ? a->max_new : a->tokens;
  const long long reach = a->window ? (long long)a->window + a->sinks + max_new : cap;
  const long long keys = reach < cap ? reach : cap;  // most keys that a row may see
  const long long rows = max_new * g, pairs = (long long)c->num_seqs * c->kv_heads;
  const bool tc = c->dtype == LLA_BF16 && a->path != LLA_PATH_CUDA_CORE;
  pl.D = padded(c->d > c->dv ? c->d : c->dv);
  const int limit = c->dtype == LLA_F32 ? kF32Rows : rows_limit(a->r != nullptr);
  const int branches = a->r ? 2 : 1;
  // The few-rows kernel, unless the counts leave no sequence for it: a sequence of at most limit / g
  // new tokens falls short of max_new by more than all sequences together do.
  const long long short_of = max_new * c->num_seqs - a->tokens;
  pl.rows = (tc || c->dtype == LLA_F32) && g <= limit && (rows <= limit || short_of >= max_new - limit / g);
  pl.tiles = !pl.rows || rows > limit;
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t o = at; at += align_up(bytes); return o; };
  auto splits = [&](long long blocks, long long want, long long least) {
    long long n = blocks > 0 ? (want + blocks - 1) / blocks : 1;
    if (n > keys / least) n = keys / least;
    return n < 1 ? 1 : n > 512 ? 512 : (int)n;
  };
  if (c->dtype == LLA_F32) {
    pl.f32 = f32_tiles(a->tokens, max_new, c->num_seqs, g);
    // (the bound counts a part tile for every sequence: as likely as not there is one)
    const long long likely = pl.f32 - (pl.f32 > 2 * c->num_seqs ? c->num_seqs / 2 : 0);
    pl.tiles_split = f32_splits(likely * c->kv_heads, keys, rows, pl.D, a->r != nullptr);
    if (pl.tiles_split > kRowsCluster) {
      const size_t all = (size_t)a->tokens * a->q_heads * pl.tiles_split;
      pl.tiles_s = take(all * sizeof(float4));
      pl.tiles_o = take(all * branches * c->dv * sizeof(float));
    }
    if (a->track_mass) {
      // The weights of sequences of up to kF32MassRows rows come from their logits, which cost 8 bytes
      // of traffic each against 2 d flops to compute them again; those of longer ones, or where the
      // scratch would be too much, from q and k.
      pl.keys_cap = (int)((keys + 64 < cap ? keys + 64 : cap) + 15) / 16 * 16;
      const size_t row_bytes = (size_t)pairs * pl.keys_cap * sizeof(float);
      const long long few = rows < limit ? rows : limit;
      if (rows <= kF32MassRows && rows * row_bytes <= kMostLogits) {
        pl.row_cap = (int)rows;
        pl.rows = true;
        pl.tiles = false;
      } else if (pl.rows && few * row_bytes <= kMostLogits) {
        pl.row_cap = (int)few;
      } else {
        pl.rows = false;
        pl.tiles = true;
      }
      if (pl.rows) pl.logits = take(pl.row_cap * row_bytes);
    }
    if (a->track_mass && !a->lse) pl.lse = take((size_t)a->tokens * a->q_heads * sizeof(float));
    pl.bytes = at;
    return pl;
  }
  if (pl.rows) {
    pl.row_cap = (int)(rows < limit ? rows : limit);
    // Two blocks per SM first, down to 128 keys each (one sequence, 8 heads of 64, L 1000: 6.4 us
    // with 8 blocks a head, 8.8 with 2); then, so that uneven lengths level out, four waves of them,
    // but no block under 1024 keys (48 sequences, 4 heads, window 1024: 19.5 us with 2 blocks a head,
    // 37 with 7). More than a cluster of 8 only where its blocks would have over 1024 keys each:
    // below that, the launch that joins costs more than shorter blocks save.
    const int fill = splits(pairs, 304, 128), level = splits(pairs, pl.D == 128 ? 1216 : 1824, 1024);
    pl.rows_split = fill > level ? fill : level;
    if (pl.rows_split > kRowsCluster && keys <= kRowsCluster * 1024) pl.rows_split = kRowsCluster;
    if (pl.rows_split > kRowsCluster) {
      pl.rows_s = take((size_t)pairs * pl.row_cap * pl.rows_split * sizeof(float4));
      pl.rows_o = take((size_t)pairs * pl.row_cap * pl.rows_split * branches * pl.D * sizeof(float));
    }
    if (a->track_mass) {
      pl.keys_cap = (int)((keys + 64 < cap ? keys + 64 : cap) + 15) / 16 * 16;
      const size_t bytes = (size_t)pairs * pl.row_cap * pl.keys_cap * sizeof(float);
      pl.logits_kept = bytes <= kMostLogits;
      if (pl.logits_kept) pl.logits = take(bytes);
    }
  }
  const TcPlan t = tc ? plan_tc(pl.D, a->r != nullptr, a->tokens, c->num_seqs, c->kv_heads, g, keys) : TcPlan();
  pl.mass_tc = t.ctas > 0;
  if (pl.tiles) {
    pl.tc = t.ctas > 0;
    if (pl.tc) {
      pl.tiles_split = t.ctas;
      pl.join = t.cuts;
      pl.pieces = take((size_t)t.ctas * 2 * sizeof(int4));
      pl.tiles_s = take(t.rows * sizeof(float4));
      pl.tiles_o = take(t.rows * t.row_floats * sizeof(float));
    } else {
      // CUDA cores: few tiles' keys are split until every SM has two blocks, down to one step of 64.
      const long long BM = rows <= 16 ? 16 : 64, per = g < BM ? BM / g : 1, slices = (g + BM - 1) / BM;
      const long long by_tokens = (a->tokens + per - 1) / per;
      const long long tiles = (by_tokens > c->num_seqs ? by_tokens : c->num_seqs) * slices * c->kv_heads;
      pl.tiles_split = splits(tiles, 304, 64);
      if (pl.tiles_split > 1) {
        const size_t all = (size_t)a->tokens * a->q_heads * pl.tiles_split;
        pl.tiles_s = take(all * sizeof(float4));
        pl.tiles_o = take(all * branches * c->dv * sizeof(float));
      }
    }
  }
  if (a->track_mass && !a->lse) pl.lse = take((size_t)a->tokens * a->q_heads * sizeof(float));
  pl.bytes = at;
  return pl;
}

int run_f32(const Params& p, const Plan& pl, int track_mass, char* ws, cudaStream_t s) {
  Params f = p;
  f.hi = p.max_rows;
  f.split = pl.tiles_split;
  f.row_cap = pl.row_cap;
  f.keys_cap = pl.keys_cap;
  if (f.split > kRowsCluster) {
    f.part_s = reinterpret_cast<float4*>(ws + pl.tiles_s);
    f.part_o = reinterpret_cast<float*>(ws + pl.tiles_o);
  }
  if (track_mass && pl.rows) f.logits = reinterpret_cast<float*>(ws + pl.logits);
  cudaError_t err = launch_attend_f32(f, pl.f32, pl.D, s);
  if (err == cudaSuccess && f.split > kRowsCluster) err = launch_join(f, p.dv, LLA_F32, s);
  if (track_mass && pl.rows && err == cudaSuccess) {
    f.hi = pl.row_cap;
    err = launch_mass_f32(f, s);
  }
  if (track_mass && pl.tiles && err == cudaSuccess) {
    f.lo = pl.row_cap;
    f.hi = p.max_rows;
    err = launch_mass_cc(f, p.d, LLA_F32, s);
  }
  return err == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
}

int run_attention(const lla_paged_cache* c, const lla_paged_query* a, const Plan& pl, char* ws,
                  cudaStream_t s) {
  Params p = cache_params(c);
  if (device_status(&p.status) != cudaSuccess) return LLA_ERR_CUDA;
  p.q = a->q;
  p.r = a->r;
  p.out = a->out;
  p.lse = a->lse;
  p.starts = a->starts;
  p.tokens = a->tokens;
  p.Hq = a->q_heads;
  p.g = a->q_heads / c->kv_heads;
  p.window = a->window && a->window < kNoWindow ? a->window : kNoWindow;
  p.sinks = a->sinks < kNoWindow ? a->sinks : kNoWindow;
  p.inv_h = 1.f / a->h;
  const long long rows = (long long)a->max_new * p.g;
  p.max_rows = rows < 0x7fffffffLL ? (int)rows : 0x7fffffff;
  if (a->track_mass && !a->lse) p.lse = reinterpret_cast<float*>(ws + pl.lse);
  if (c->dtype == LLA_F32) return run_f32(p, pl, a->track_mass, ws, s);
  Params f = p;  // the few-rows kernel's
  p.lo = pl.rows ? pl.row_cap : 0;
  p.split = pl.tiles_split;
  if (pl.tiles) {
    if (pl.tc || p.split > 1) {
      p.part_s = reinterpret_cast<float4*>(ws + pl.tiles_s);
      p.part_o = reinterpret_cast<float*>(ws + pl.tiles_o);
    }
    if (pl.tc) p.pieces = reinterpret_cast<int4*>(ws + pl.pieces);
    if ((pl.tc ? launch_attend_tc(p, pl.D, s) : attend_cc_bf16(p, c->d, c->dv, s)) != cudaSuccess)
      return LLA_ERR_CUDA;
  }
  if (pl.rows) {
    f.lo = 0;
    f.hi = f.row_cap = pl.row_cap;
    f.split = pl.rows_split;
    f.beside = pl.tiles && pl.tc;
    if (pl.rows_split > kRowsCluster) {
      f.part_s = reinterpret_cast<float4*>(ws + pl.rows_s);
      f.part_o = reinterpret_cast<float*>(ws + pl.rows_o);
    }
    if (a->track_mass && pl.logits_kept) {
      f.keys_cap = pl.keys_cap;
      f.logits = reinterpret_cast<float*>(ws + pl.logits);
    }
    if (launch_attend_rows(f, pl.D, s) != cudaSuccess) return LLA_ERR_CUDA;
  }
  if (pl.tiles) {
    if (pl.tc ? pl.join && launch_join_tc(p, pl.D, s) != cudaSuccess
              : p.split > 1 && launch_join(p, c->dv, c->dtype, s) != cudaSuccess)
      return LLA_ERR_CUDA;
  }
  if (a->track_mass && (pl.tiles || !pl.logits_kept)) {
    p.lo = pl.logits_kept ? pl.row_cap : 0;
    if (!pl.tiles) p.hi = pl.row_cap;
    if ((pl.mass_tc ? launch_mass_tc(p, padded(c->d), s) : launch_mass_cc(p, c->d, c->dtype, s)) != cudaSuccess)
      return LLA_ERR_CUDA;
  }
  return LLA_OK;
}

}  // namespace
}  // namespace paged
}  // namespace lla

using namespace lla;
using namespace lla::paged;

extern "C" {

int lla_paged_append(const lla_paged_cache* cache, const void* k_new, const void* v_new,
                     const int* starts, int tokens, void* stream) {
  int st = check_cache_shape(cache);
  if (st != LLA_OK) return st;
  if (tokens < 0) return LLA_ERR_INVALID_ARG;
  if ((long long)tokens * cache->kv_heads >= (1LL << 31) || tokens >= kNoWindow)
    return LLA_ERR_UNSUPPORTED;
  if (tokens == 0 || cache->num_seqs == 0) return LLA_OK;
  st = check_cache_pointers(cache, false);
  if (st != LLA_OK) return st;
  if (!k_new || !v_new || !starts || !aligned16(k_new) || !aligned16(v_new)) return LLA_ERR_INVALID_ARG;
  Params p = cache_params(cache);
  if (device_status(&p.status) != cudaSuccess) return LLA_ERR_CUDA;
  p.starts = starts;
  p.tokens = tokens;
  return launch_append(p, k_new, v_new, cache->d, cache->dv, cache->dtype,
                       static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? LLA_OK
             : LLA_ERR_CUDA;
}

size_t lla_paged_workspace_size(const lla_paged_cache* cache, const lla_paged_query* query) {
  if (check_query(cache, query) != LLA_OK) return 0;
  if (query->tokens == 0 || cache->num_seqs == 0) return 0;
  return make_plan(cache, query).bytes;
}

int lla_paged_attention(const lla_paged_cache* cache, const lla_paged_query* query, void* workspace,
                        size_t workspace_bytes, void* stream) {
  int st = check_query(cache, query);
  if (st != LLA_OK) return st;
  if (query->tokens == 0 || cache->num_seqs == 0) return LLA_OK;
  if (query->max_new == 0) return LLA_ERR_INVALID_ARG;
  st = check_cache_pointers(cache, query->track_mass != 0);
  if (st != LLA_OK) return st;
  if (!query->q || !query->out || !query->starts || !aligned16(query->q) || !aligned16(query->out) ||
      (query->r && !aligned16(query->r)))
    return LLA_ERR_INVALID_ARG;
  const Plan pl = make_plan(cache, query);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (workspace || pl.bytes == 0) {
    if (workspace && ((reinterpret_cast<uintptr_t>(workspace) % 256) != 0 || workspace_bytes < pl.bytes))
      return LLA_ERR_INVALID_ARG;
    return run_attention(cache, query, pl, static_cast<char*>(workspace), s);
  }
  if (ensure_pool() != cudaSuccess) return LLA_ERR_CUDA;
  void* ws = nullptr;
  if (cudaMallocAsync(&ws, pl.bytes, s) != cudaSuccess) return LLA_ERR_CUDA;
  st = run_attention(cache, query, pl, static_cast<char*>(ws), s);
  if (cudaFreeAsync(ws, s) != cudaSuccess && st == LLA_OK) st = LLA_ERR_CUDA;
  return st;
}

int lla_paged_evict(const lla_paged_cache* from, const lla_paged_cache* to, int budget, int sinks,
                    int recent, int* kept, void* stream) {
  int st = check_cache_shape(from);
  if (st == LLA_OK) st = check_cache_shape(to);
  if (st != LLA_OK) return st;
  if (to->num_seqs != from->num_seqs || to->kv_heads != from->kv_heads ||
      to->page_size != from->page_size || to->d != from->d || to->dv != from->dv ||
      to->dtype != from->dtype)
    return LLA_ERR_INVALID_ARG;
  if (budget < 1 || sinks < 0 || recent < 0 || (long long)sinks + recent > budget)
    return LLA_ERR_INVALID_ARG;
  const long long cap = (long long)from->max_pages * from->page_size;
  if ((budget < cap ? budget : cap) > (long long)to->max_pages * to->page_size)
    return LLA_ERR_INVALID_ARG;
  if (from->num_seqs == 0) return LLA_OK;
  st = check_cache_pointers(from, true);
  if (st == LLA_OK) st = check_cache_pointers(to, true);
  if (st != LLA_OK) return st;
  if (!kept || from->lens == to->lens || from->page_table == to->page_table)
    return LLA_ERR_INVALID_ARG;
  Params p = cache_params(from);
  if (device_status(&p.status) != cudaSuccess) return LLA_ERR_CUDA;
  return launch_evict(p, to->k_pages, to->v_pages, to->mass, to->page_table, to->lens, to->max_pages,
                      to->num_pages, budget, sinks, recent, kept, from->d, from->dv, from->dtype,
                      static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? LLA_OK
             : LLA_ERR_CUDA;
}

}  // extern "C"
