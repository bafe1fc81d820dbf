// cache_attn.cuh -- what the cache attention kernels share: the arguments, the
// split of the work over the CTAs, and a row's last step.
//
// Work split.  A unit is (sequence b, row tile, KV head h): up to kRows of the
// group's G * q_len query rows (row r is token r / G of query head h G + r % G,
// so that a tile covers few tokens and a causal tile stops early) against the
// slots they see, in tiles of kTile slots.  The units' tiles, laid end to end,
// are cut into one equal range per CTA, so that ragged lengths leave no CTA
// behind; the lengths are device data, so every CTA finds its range itself
// with one scan over the (b, row tile) items.  A unit that lies within one
// range is finished there; a unit that is cut leaves one partial per CTA (the
// unnormalised O, the reference maximum m and the sum l of each row), which
// k_attn_merge joins in the order of the slots.  (The tile kernel keeps parts of a
// long unit's O there, too, until the unit is finished.)
#pragma once

#include "cache.cuh"

namespace dropkv {

struct AttnDev {
  CacheDev c;
  const void* q;
  void* out;
  float* lse;
  int64_t qs[3], os[3];
  int32_t Hq, G, T, causal;
  FastDiv fG;
  int32_t nrt;      // row tiles a sequence can have: ceil(G T / kRows)
  float c_log2;     // scale * log2(e)
  const int32_t* lengths;
  const int32_t* q_lengths;
  float* part;      // [2 grid][rows][pstride]
  int32_t pstride;  // floats of a partial row: O (d rounded up to 4), m, l, pad
  int32_t* status;
  long long wait_clocks;  // limit of every wait on an mbarrier
  int32_t withhold;       // 1 in the self-test alone: the first unit's queries are never handed over
};
// Of a wait: two seconds at least.
constexpr long long kWaitClocks = 4000000000ll;

// An attention kernel's first step.  It may be launched while its predecessor in
// the stream ends (those of the tensor path are), and waits for that here; only then may the join be launched,
// which reads the lengths before its own wait.
__device__ __forceinline__ void attn_begin() {
  pdl_wait();
  pdl_trigger();
}

// ex2 and the row statistics are in units of log2.
__device__ __forceinline__ float attn_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Weights x, y >= 0 as two bf16 parts each, for products whose V is bf16: the upper
// part is cut off, the lower is what it leaves of (1 + 2^-20) x, rounded.  Together
// they are within 2^-15 + 2^-20 of x (the lower is at most 2^-7 x, its rounding 2^-8
// of that); one part alone, rounded, is within 2^-8, as large an error as the output's
// own rounding to bf16 (in all 2.4e-3 of the norm against 1.7e-3).  The 2^-20 keeps
// the lower part of a positive weight above zero, since V may hold an infinity and
// 0 * inf is NaN (weights under 2^-113 do lose theirs to underflow).  The second
// part's products and instructions cost 1 to 6 % of a call of few rows, 9 to 16 % up
// to 128 rows and 19 to 28 % above (64 e4m3 sequences 118 to 125 us, 16 drafted tokens
// x 8 152 to 165, 512 tokens over 32K bf16 slots 310 to 388).
__device__ __forceinline__ uint32_t upper_bf16x2(float x, float y) {
  return __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
}
__device__ __forceinline__ float minus_upper(float x) {  // x >= 0
  return __uint_as_float((__float_as_uint(x) & 0xFFFF0000u) ^ 0x80000000u);
}
constexpr float kAboveOne = 1.f + 0x1p-20f;
__device__ __forceinline__ uint32_t lower_bf16x2(float x, float y) {
  return pack_bf16(fmaf(x, kAboveOne, minus_upper(x)), fmaf(y, kAboveOne, minus_upper(y)));
}

// Sequence b's slots and chunk, clamped to what there is.
__device__ __forceinline__ void attn_lengths(const AttnDev& a, int b, int& L, int& n) {
  L = __ldg(a.lengths + b);
  n = a.q_lengths ? __ldg(a.q_lengths + b) : a.T;
  if ((uint32_t)L > (uint32_t)a.c.cap || (uint32_t)n > (uint32_t)a.T) {
    raise_arg(a.status);
    L = min(max(L, 0), a.c.cap);
    n = min(max(n, 0), a.T);
  }
}
// n / d of non-negative values, which mostly fit 32 bits: the 64-bit division is a
// long routine, and the CTAs' ranges take several one after the other.
__device__ __forceinline__ int64_t attn_div(int64_t n, int64_t d) {
  if (((uint64_t)n | (uint64_t)d) >> 32) return n / d;
  return (int64_t)((uint32_t)n / (uint32_t)d);
}
// Slots that row r (token r / G) sees.
__device__ __forceinline__ int attn_seen(const AttnDev& a, int L, int n, int r) {
  return a.causal ? max(0, L - n + (int)a.fG.div((uint32_t)r) + 1) : L;
}
// Tiles of a unit of item (b, rt): those of its last row, and one at least, so
// that rows that see nothing are written too; 0 if the item has no rows.
template <int kRows, int kTile>
__device__ __forceinline__ int attn_tiles(const AttnDev& a, int item) {
  const int b = item / a.nrt, rt = item - b * a.nrt;
  int L, n;
  attn_lengths(a, b, L, n);
  const int rows = a.G * n;
  if (rt * kRows >= rows) return 0;
  const int seen = attn_seen(a, L, n, min((rt + 1) * kRows, rows) - 1);
  return max(1, (seen + kTile - 1) / kTile);
}

// A CTA's place in the work: item, head, the tiles [t0, t1) of the unit's `nt`
// that belong to the CTA, and what is left of the CTA's range after the unit.
struct AttnWalk {
  int item, h, nt, t0, t1;
  int64_t g0;        // first tile of the unit among all tiles
  int64_t left;      // tiles of the range from t0 on
};

struct AttnPlanShared {
  int64_t warp_sum[33];
  int64_t g0;        // of the item
  int item, nt;
};

// The unit of one tile of the work (kThreads threads, all call it): pick(total)
// names the tile, < 0 for none (then false).  Sets w but for left and t1.
template <int kRows, int kTile, int kThreads, typename Pick>
__device__ __forceinline__ bool attn_seek(const AttnDev& a, AttnPlanShared& sh, AttnWalk& w,
                                          int64_t& total, Pick pick) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int items = a.c.B * a.nrt;
  // pass 1: all tiles; with no more items than threads its scan also places
  // the tile
  int64_t sum = 0, incl = 0, base = 0;
  int mine = 0;
  for (int i0 = 0; i0 < items; i0 += kThreads) {
    const int it = i0 + (int)threadIdx.x;
    mine = it < items ? attn_tiles<kRows, kTile>(a, it) : 0;
    sum += (int64_t)mine * a.c.Hkv;
  }
  incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) sh.warp_sum[warp] = incl;
  __syncthreads();
  total = 0;
  for (int i = 0; i < kWarps; ++i) {
    if (i == warp) base = total;
    total += sh.warp_sum[i];
  }
  const int64_t at = pick(total);
  if (at < 0) return false;
  if (items <= kThreads) {
    const int64_t e = base + incl - sum;  // tiles before this thread's item
    if (at >= e && at < e + sum) {
      sh.item = threadIdx.x;
      sh.nt = mine;
      sh.g0 = e;
    }
    __syncthreads();
  } else {
    // pass 2: the same scan chunk by chunk until the tile
    int64_t before = 0;
    for (int i0 = 0; i0 < items; i0 += kThreads) {
      const int it = i0 + (int)threadIdx.x;
      const int nt = it < items ? attn_tiles<kRows, kTile>(a, it) : 0;
      const int64_t own = (int64_t)nt * a.c.Hkv;
      int64_t s = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += x;
      }
      __syncthreads();
      if (lane == 31) sh.warp_sum[warp] = s;
      __syncthreads();
      int64_t all = 0, wb = 0;
      for (int i = 0; i < kWarps; ++i) {
        if (i == warp) wb = all;
        all += sh.warp_sum[i];
      }
      const int64_t e = before + wb + s - own;
      if (at >= e && at < e + own) {
        sh.item = it;
        sh.nt = nt;
        sh.g0 = e;
      }
      before += all;
      if (at < before) break;  // the same for every thread
    }
    __syncthreads();
  }
  w.item = sh.item;
  w.nt = sh.nt;
  const int64_t in_item = at - sh.g0;
  w.h = (int)attn_div(in_item, w.nt);
  w.t0 = (int)(in_item - (int64_t)w.h * w.nt);
  w.g0 = sh.g0 + (int64_t)w.h * w.nt;
  return true;
}

// CTAs that have a range (every one of them a non-empty one), of `ctas`, and
// the ranges' ends.
__device__ __forceinline__ int attn_grid(int64_t total, int ctas) {
  return (int)min((int64_t)ctas, total);
}
__device__ __forceinline__ int64_t attn_range(int64_t total, int grid, int cta) {
  return attn_div(total * cta, grid);
}

// The range of this CTA (kThreads threads, all call it).
template <int kRows, int kTile, int kThreads>
__device__ __forceinline__ bool attn_plan(const AttnDev& a, AttnPlanShared& sh, AttnWalk& w) {
  int64_t total, first = 0, last = 0;
  const bool some = attn_seek<kRows, kTile, kThreads>(a, sh, w, total, [&](int64_t all) -> int64_t {
    const int grid = attn_grid(all, gridDim.x);
    if ((int)blockIdx.x >= grid) return -1;
    first = attn_range(all, grid, blockIdx.x);
    last = attn_range(all, grid, blockIdx.x + 1);
    return first;
  });
  if (!some) return false;
  w.left = last - first;
  w.t1 = (int)min((int64_t)w.nt, w.t0 + w.left);
  return true;
}

// The next unit of the range; false at its end.
template <int kRows, int kTile>
__device__ __forceinline__ bool attn_next(const AttnDev& a, AttnWalk& w) {
  w.left -= w.t1 - w.t0;
  if (w.left <= 0) return false;
  w.g0 += w.nt;
  if (++w.h == a.c.Hkv) {
    w.h = 0;
    do {
      ++w.item;
      w.nt = attn_tiles<kRows, kTile>(a, w.item);
    } while (w.nt == 0);
  }
  w.t0 = 0;
  w.t1 = (int)min((int64_t)w.nt, w.left);
  return true;
}

// Where the unit's rows go: -1 to the output (the unit is whole), or the
// partial's slot: 2 cta + 1 for the unit that begins in the CTA and does not
// end there, 2 cta for the one that began in an earlier CTA.
__device__ __forceinline__ int attn_slot(const AttnWalk& w) {
  if (w.t0 == 0 && w.t1 == w.nt) return -1;
  return 2 * (int)blockIdx.x + (w.t0 == 0 ? 1 : 0);
}
// A row's output position.
struct AttnRow {
  int b, hq, t;
};
__device__ __forceinline__ AttnRow attn_row(const AttnDev& a, int b, int h, int r) {
  AttnRow x;
  x.b = b;
  x.t = (int)a.fG.div((uint32_t)r);
  x.hq = h * a.G + (r - x.t * a.G);
  return x;
}
// m ln 2 + log l, with ln 2 as two fp32 values: one rounding behind logf's, where the
// approximate log2 and a product of the sum left three.
__device__ __forceinline__ void attn_put_lse(const AttnDev& a, const AttnRow& x, float m, float l) {
  constexpr float kLn2 = 0.69314718055994531, kLn2Rest = 0.69314718055994531 - kLn2;
  if (a.lse)
    a.lse[((int64_t)x.b * a.Hq + x.hq) * a.T + x.t] =
        l > 0.f ? fmaf(m, kLn2, fmaf(m, kLn2Rest, logf(l))) : (l == 0.f ? -CUDART_INF_F : l);
}

// The page and the offset in it of slot `slot` < end of the sequence with this
// page table row; off -1: no slot.  Volatile: requested here, a tile before it is
// used.
struct Look {
  int page, off;
};
__device__ __forceinline__ Look look_up(const AttnDev& a, const int32_t* table, int slot, int end) {
  Look k = {-1, -1};
  if (slot < end) {
    const int pi = (int)a.c.fpage.div((uint32_t)slot);
    asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(k.page) : "l"(table + pi));
    k.off = slot - pi * a.c.page;
  }
  return k;
}
// Its pool row, or -1 (32 bits: the tensor path's host side checked the size).
__device__ __forceinline__ int pool_row(const AttnDev& a, int h, Look k) {
  if ((uint32_t)k.page < (uint32_t)a.c.n_pages) return (k.page * a.c.Hkv + h) * a.c.page + k.off;
  if (k.off >= 0) raise_arg(a.status);
  return -1;
}

// 16 bytes global -> shared, asynchronously; zeros instead of the source's bytes
// (which are not read) when !on.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  const int n = on ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct AttnGrid {
  int ctas, rows, tile;  // of a unit
};
// Grid and unit rows of each kernel (host); launchers of one call's kernels.
AttnGrid attn_grid_simt(int64_t rows, int d);  // rows a KV head can have
AttnGrid attn_grid_rows();
AttnGrid attn_grid_few(int page_dtype);
AttnGrid attn_grid_tile(bool alt);
cudaError_t launch_attn_simt(const AttnDev& a, AttnGrid g, int page_dtype, int q_dtype,
                             cudaStream_t st);
cudaError_t launch_attn_rows(const AttnDev& a, int page_dtype, cudaStream_t st);
cudaError_t launch_attn_few(const AttnDev& a, int page_dtype, cudaStream_t st);
cudaError_t launch_attn_tile(const AttnDev& a, int page_dtype, bool alt, cudaStream_t st);
// The join of the units that the kernel of this grid cut.
cudaError_t launch_attn_merge(const AttnDev& a, AttnGrid g, int q_dtype, cudaStream_t st);

}  // namespace dropkv
