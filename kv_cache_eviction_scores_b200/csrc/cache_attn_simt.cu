// cache_attn_simt.cu -- cache attention on CUDA cores (any head dim up to 256,
// any page size, stride and storage type, fp32 arithmetic), and the merge of
// cut units that every path ends with.
//
// k_attn_simt: 128 threads; a unit is 16 query rows against tiles of 32 slots.
// K and V rows are widened to fp32 in shared memory; each warp owns four rows:
// its lane j holds the four logits of slot j (fp32 dot products over float4
// pieces), the running maximum and sum of a row are kept in the log2 domain
// and reduced by shuffles, and its lanes hold the four rows' O, a column in
// each 32.  The rows' stride is an odd number of 16-byte pieces, so that the
// lanes' float4 reads of 32 rows touch every bank evenly.  Bound by latency at
// small sizes (37 tokens, 6 / 2 heads over two caches of up to 1501 fp32 slots: 28 us,
// then the join; 0.44 instructions a cycle, the stalls on global memory, on shared
// memory and on dependent results about equal) and by shared-memory reads at large ones.
#include "cache_attn.cuh"
#include "tc_ptx.cuh"

namespace dropkv {

namespace {

constexpr int kSRows = 16, kSTile = 32, kSThreads = 128;
constexpr int kSCtas = 592;                  // four CTAs an SM
constexpr int kLCtas = 296, kLCtas3 = 444;   // of the 64-row kernel two, for d <= 64 three

__device__ __forceinline__ float4 four(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float single(const float* p) { return *p; }
__device__ __forceinline__ float single(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float single(const E4M3* p) { return unpack_e4m3(p->bits).x; }
__device__ __forceinline__ void store_out(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ uint64_t lo2(const float4& v) { return tc::pk2(v.x, v.y); }
__device__ __forceinline__ uint64_t hi2(const float4& v) { return tc::pk2(v.z, v.w); }

// Floats between rows in shared memory: d in whole float4s, an odd number of them.
__host__ __device__ __forceinline__ int row_stride(int d) { return (((d + 3) / 4) | 1) * 4; }

// Four values as they are stored.
template <typename TP>
struct Four {};
template <>
struct Four<float> {
  float4 w;
  __device__ __forceinline__ float4 get() const { return w; }
};
template <>
struct Four<__nv_bfloat16> {
  uint2 w;
  __device__ __forceinline__ float4 get() const {
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
  }
};
template <>
struct Four<E4M3> {
  uint32_t w;
  __device__ __forceinline__ float4 get() const {
    const float2 a = unpack_e4m3(w & 0xFFFFu), b = unpack_e4m3(w >> 16);
    return make_float4(a.x, a.y, b.x, b.y);
  }
};

// The kSTile / 4 rows of K and of V that are this warp's, to fp32 in shared memory
// (zeros where there is no row).  All of a column block's loads are in flight
// together: one after the other, their latencies were most of the kernel's time.
template <typename TP>
__device__ __forceinline__ void widen_rows(const AttnDev& a, float* sK, float* sV, int ds,
                                           const int64_t (&srow)[kSTile], int warp, int lane) {
  constexpr int kMine = kSTile / 4;
  const int d = a.c.d, d4 = (d + 3) & ~3;
  const TP* pool[2] = {reinterpret_cast<const TP*>(a.c.k), reinterpret_cast<const TP*>(a.c.v)};
  int64_t row[kMine];
  float f[2][kMine];
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    row[j] = srow[warp + 4 * j];
    f[0][j] = f[1][j] = 1.f;
    if (sizeof(TP) == 1 && row[j] >= 0) {
      f[0][j] = scale_of(__ldg(a.c.ks + row[j]));
      f[1][j] = scale_of(__ldg(a.c.vs + row[j]));
    }
  }
  if (d % 4 == 0) {
    for (int i = lane * 4; i < d; i += 128) {
      Four<TP> x[2][kMine];
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          x[v][j] = Four<TP>{};
          if (row[j] >= 0) x[v][j] = *reinterpret_cast<const Four<TP>*>(pool[v] + row[j] * d + i);
        }
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          const float4 y = x[v][j].get();
          const float s = f[v][j];
          *reinterpret_cast<float4*>((v ? sV : sK) + (warp + 4 * j) * ds + i) =
              make_float4(y.x * s, y.y * s, y.z * s, y.w * s);
        }
    }
  } else {
    for (int i = lane; i < d4; i += 32) {
      float x[2][kMine];
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int j = 0; j < kMine; ++j)
          x[v][j] = row[j] >= 0 && i < d ? single(pool[v] + row[j] * d + i) : 0.f;
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int j = 0; j < kMine; ++j) (v ? sV : sK)[(warp + 4 * j) * ds + i] = x[v][j] * f[v][j];
    }
  }
}

template <typename TQ, typename TP>
__global__ void __launch_bounds__(kSThreads, 4) k_attn_simt(const AttnDev a) {
  extern __shared__ __align__(16) float sm[];
  __shared__ AttnPlanShared plan;
  __shared__ int64_t srow[2][kSTile];  // pool rows of a tile's slots, -1: none
  attn_begin();
  const int d = a.c.d, ds = row_stride(d);
  float* sQ = sm;
  float* sK = sQ + kSRows * ds;
  float* sV = sK + kSTile * ds;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* sP = sV + kSTile * ds + warp * (kSTile * 4);  // this warp's [slot][4 rows]
  AttnWalk w;
  bool more = attn_plan<kSRows, kSTile, kSThreads>(a, plan, w);
  while (more) {
    const int b = w.item / a.nrt, rt = w.item - b * a.nrt;
    int L, n;
    attn_lengths(a, b, L, n);
    const int rows = min(kSRows, a.G * n - rt * kSRows);
    const int seen_all = attn_seen(a, L, n, rt * kSRows + rows - 1);
    __syncthreads();  // the last unit's reads of shared memory
    for (int r = warp; r < kSRows; r += 4) {
      const AttnRow x = attn_row(a, b, w.h, rt * kSRows + (r < rows ? r : 0));
      const TQ* q = reinterpret_cast<const TQ*>(a.q) + x.b * a.qs[0] + x.hq * a.qs[1] + x.t * a.qs[2];
      for (int i = lane; i < ((d + 3) & ~3); i += 32)
        sQ[r * ds + i] = r < rows && i < d ? single(q + i) : 0.f;
    }
    auto place = [&](int t) {  // warp 0: the pool rows of tile t
      const int slot = t * kSTile + lane;
      int64_t row = -1;
      if (slot < seen_all) {
        row = cache_row(a.c, b, w.h, slot);
        if (row < 0) raise_arg(a.status);
      }
      srow[t & 1][lane] = row;
    };
    if (warp == 0) place(w.t0);
    int seen[4];
    bool live[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = warp * 4 + k;
      live[k] = r < rows;
      seen[k] = live[k] ? attn_seen(a, L, n, rt * kSRows + r) : 0;
    }
    float m[4], l[4], o[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      m[k] = -CUDART_INF_F;
      l[k] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[k][i] = 0.f;
    }
    __syncthreads();
    for (int t = w.t0; t < w.t1; ++t) {
      widen_rows<TP>(a, sK, sV, ds, srow[t & 1], warp, lane);
      const bool absent = srow[t & 1][lane] < 0;
      if (warp == 0 && t + 1 < w.t1) place(t + 1);
      __syncthreads();
      if (warp * 4 < rows) {
        const int slot = t * kSTile + lane;
        // four sums per logit: packed products, and shorter chains of roundings
        uint64_t sa[4] = {0ull, 0ull, 0ull, 0ull}, sb[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 4
        for (int i = 0; i < d; i += 4) {
          const float4 k4 = four(sK + lane * ds + i);
          const uint64_t ka = lo2(k4), kb = hi2(k4);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 q4 = four(sQ + (warp * 4 + k) * ds + i);
            sa[k] = tc::ffma2(lo2(q4), ka, sa[k]);
            sb[k] = tc::ffma2(hi2(q4), kb, sb[k]);
          }
        }
        float s[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x, y;
          tc::upk2(tc::fadd2(sa[k], sb[k]), x, y);
          s[k] = x + y;
        }
        float p[4];
        bool partly = false;  // some row of the warp does not see some slot
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool hid = slot >= seen[k] || absent;
          partly = partly || (live[k] && hid);
          // c > 0 commutes with the max; the one rounding of s c - mu is relative to
          // that difference, and mu's own is the same for the whole row
          const float mt = fmaxf(m[k], warp_max(hid ? -CUDART_INF_F : s[k]) * a.c_log2);
          const float mu = mt == -CUDART_INF_F ? 0.f : mt;
          const float fac = attn_ex2(m[k] - mu);
          p[k] = hid ? 0.f : attn_ex2(fmaf(s[k], a.c_log2, -mu));
          m[k] = mt;
          l[k] = l[k] * fac + warp_sum(p[k]);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[k][i] *= fac;
        }
        partly = __any_sync(0xffffffffu, partly);
        *reinterpret_cast<float4*>(sP + lane * 4) = make_float4(p[0], p[1], p[2], p[3]);
        __syncwarp();
        if (!partly) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int col = lane + 32 * i;
            if (32 * i >= d) break;
            const float* v = sV + (col < d ? col : 0);
            // the tile's slots by themselves: a chain over all of a long cache's slots
            // loses bits (7e-4 of a sum of 64K equal terms)
            float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
            for (int j = 0; j < kSTile; ++j) {
              const float4 p4 = four(sP + j * 4);
              const float x = v[j * ds];
              y[0] = fmaf(p4.x, x, y[0]);
              y[1] = fmaf(p4.y, x, y[1]);
              y[2] = fmaf(p4.z, x, y[2]);
              y[3] = fmaf(p4.w, x, y[3]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k][i] += y[k];
          }
        } else {
          // a slot that a row does not see may hold anything: 0 * NaN must not
          // reach that row
#pragma unroll 1
          for (int j = 0; j < kSTile; ++j) {
            const float4 p4 = four(sP + j * 4);
            const float* v = sV + j * ds;
            const int sj = t * kSTile + j;
            const bool u0 = sj < seen[0], u1 = sj < seen[1], u2 = sj < seen[2], u3 = sj < seen[3];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (lane + 32 * i >= d) break;
              const float x = v[lane + 32 * i];
              if (u0) o[0][i] = fmaf(p4.x, x, o[0][i]);
              if (u1) o[1][i] = fmaf(p4.y, x, o[1][i]);
              if (u2) o[2][i] = fmaf(p4.z, x, o[2][i]);
              if (u3) o[3][i] = fmaf(p4.w, x, o[3][i]);
            }
          }
        }
      }
      __syncthreads();
    }
    const int slot = attn_slot(w);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!live[k]) continue;
      const int r = warp * 4 + k;
      if (slot < 0) {
        const AttnRow x = attn_row(a, b, w.h, rt * kSRows + r);
        TQ* out = reinterpret_cast<TQ*>(a.out) + x.b * a.os[0] + x.hq * a.os[1] + x.t * a.os[2];
        const float inv = l[k] == 0.f ? 0.f : 1.f / l[k];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (lane + 32 * i < d) store_out(out + lane + 32 * i, o[k][i] * inv);
        if (lane == 0) attn_put_lse(a, x, m[k], l[k]);
      } else {
        float* out = a.part + ((size_t)slot * kSRows + r) * a.pstride;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (lane + 32 * i < d) out[lane + 32 * i] = o[k][i];
        if (lane == 0) *reinterpret_cast<float2*>(out + a.pstride - 4) = make_float2(m[k], l[k]);
      }
    }
    more = attn_next<kSRows, kSTile>(a, w);
  }
}

// ---- many rows per KV head -----------------------------------------------------
//
// k_attn_simt_tile: a unit is 64 query rows against tiles of 32 slots, 128 threads.
// Thread (ty, tx) computes the logits of rows 4 ty .. 4 ty + 3 and slots tx + 8 j (j
// < 4) from float4 pieces, eight 16-byte loads for 64 multiply-adds (32 packed
// ones), keeps those rows' statistics with its seven neighbours, and owns columns 4
// tx .. 4 tx + 3 of every 32 of those rows' O.  The rows' stride, an odd number of
// 16-byte pieces, keeps the eight slots' loads in different banks.
constexpr int kLRows = 64, kPStride = kSTile + 4;

template <typename TQ, typename TP, int kCols>  // kCols: blocks of 32 columns
__global__ void __launch_bounds__(kSThreads, kCols > 4 ? 1 : kCols > 2 ? 2 : 3) k_attn_simt_tile(const AttnDev a) {
  extern __shared__ __align__(16) float sm[];
  __shared__ AttnPlanShared plan;
  __shared__ int64_t srow[2][kSTile];  // pool rows of a tile's slots, -1: none
  attn_begin();
  const int d = a.c.d, ds = row_stride(d), d4 = (d + 3) & ~3;
  float* sQ = sm;
  float* sK = sQ + kLRows * ds;
  float* sV = sK + kSTile * ds;
  float* sP = sV + kSTile * ds;  // [kLRows][kPStride]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ty = threadIdx.x >> 3, tx = threadIdx.x & 7;
  AttnWalk w;
  bool more = attn_plan<kLRows, kSTile, kSThreads>(a, plan, w);
  while (more) {
    const int b = w.item / a.nrt, rt = w.item - b * a.nrt;
    int L, n;
    attn_lengths(a, b, L, n);
    const int rows = min(kLRows, a.G * n - rt * kLRows);
    const int seen_all = attn_seen(a, L, n, rt * kLRows + rows - 1);
    const int seen_min = attn_seen(a, L, n, rt * kLRows);
    __syncthreads();  // the last unit's reads of shared memory
#pragma unroll 4
    for (int r = warp; r < kLRows; r += 4) {
      const AttnRow x = attn_row(a, b, w.h, rt * kLRows + (r < rows ? r : 0));
      const TQ* q = reinterpret_cast<const TQ*>(a.q) + x.b * a.qs[0] + x.hq * a.qs[1] + x.t * a.qs[2];
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int col = lane + 32 * i;
        if (col < d4) sQ[r * ds + col] = r < rows && col < d ? single(q + col) : 0.f;
      }
    }
    auto place = [&](int t) {  // warp 0: the pool rows of tile t
      const int slot = t * kSTile + lane;
      int64_t row = -1;
      if (slot < seen_all) {
        row = cache_row(a.c, b, w.h, slot);
        if (row < 0) raise_arg(a.status);
      }
      srow[t & 1][lane] = row;
    };
    if (warp == 0) place(w.t0);
    int seen[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      seen[k] = 4 * ty + k < rows ? attn_seen(a, L, n, rt * kLRows + 4 * ty + k) : 0;
    float m[4], l[4];
    uint64_t o[4][kCols][2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      m[k] = -CUDART_INF_F;
      l[k] = 0.f;
#pragma unroll
      for (int i = 0; i < kCols; ++i) o[k][i][0] = o[k][i][1] = 0ull;
    }
    __syncthreads();
    for (int t = w.t0; t < w.t1; ++t) {
      widen_rows<TP>(a, sK, sV, ds, srow[t & 1], warp, lane);
      // the slots of the tile that are there
      const uint32_t there = __ballot_sync(0xffffffffu, srow[t & 1][lane] >= 0);
      if (warp == 0 && t + 1 < w.t1) place(t + 1);
      __syncthreads();
      if (4 * 4 * warp < rows) {
        uint64_t acc[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[k][j] = 0ull;
#pragma unroll 2
        for (int i = 0; i < d; i += 4) {
          uint64_t ka[4], kb[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 k4 = four(sK + (tx + 8 * j) * ds + i);
            ka[j] = lo2(k4);
            kb[j] = hi2(k4);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 q4 = four(sQ + (4 * ty + k) * ds + i);
            const uint64_t qa = lo2(q4), qb = hi2(q4);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[k][j] = tc::ffma2(qb, kb[j], tc::ffma2(qa, ka[j], acc[k][j]));
          }
        }
        // some row of the unit does not see some slot of the tile
        const bool partly = there != 0xFFFFFFFFu || (t + 1) * kSTile > seen_min;
        const int lim = t * kSTile;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float s[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x, y;
            tc::upk2(acc[k][j], x, y);
            s[j] = x + y;
          }
          bool hid[4] = {false, false, false, false};
          float top = -CUDART_INF_F;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (partly) hid[j] = lim + tx + 8 * j >= seen[k] || !((there >> (tx + 8 * j)) & 1);
            if (!hid[j]) top = fmaxf(top, s[j]);
          }
#pragma unroll
          for (int x = 1; x < 8; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          // as in the kernel above: one rounding, relative to the difference
          const float mt = fmaxf(m[k], top * a.c_log2);
          const float mu = mt == -CUDART_INF_F ? 0.f : mt;
          if (mt != m[k]) {  // the same for the eight threads of the row
            const float fac = attn_ex2(m[k] - mu);
            m[k] = mt;
            l[k] *= fac;
            const uint64_t f2 = tc::pk2(fac, fac);
#pragma unroll
            for (int i = 0; i < kCols; ++i) {
              o[k][i][0] = tc::fmul2(o[k][i][0], f2);
              o[k][i][1] = tc::fmul2(o[k][i][1], f2);
            }
          }
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p = hid[j] ? 0.f : attn_ex2(fmaf(s[j], a.c_log2, -mu));
            sum += p;
            sP[(4 * ty + k) * kPStride + tx + 8 * j] = p;
          }
          l[k] += sum;
        }
        __syncwarp();
        if (!partly) {
          // the tile's slots by themselves, as in the kernel above; 128 columns at a
          // time, so that the sums fit the registers (d = 256 then reads P twice: 505 us
          // against 451 for 300 rows x 8 over 3000 fp32 slots; d = 128 199 and 201)
          constexpr int kPart = kCols < 4 ? kCols : 4;
#pragma unroll
          for (int i0 = 0; i0 < kCols; i0 += kPart) {
            uint64_t y[4][kPart][2];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int i = 0; i < kPart; ++i) y[k][i][0] = y[k][i][1] = 0ull;
#pragma unroll 1
            for (int j = 0; j < kSTile; j += 4) {
              float4 p[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) p[k] = four(sP + (4 * ty + k) * kPStride + j);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float* v = sV + (j + e) * ds;
#pragma unroll
                for (int i = 0; i < kPart; ++i) {
                  const float4 x = four(v + min(4 * tx + 32 * (i0 + i), d4 - 4));
                  const uint64_t xa = lo2(x), xb = hi2(x);
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const float pe = e == 0 ? p[k].x : e == 1 ? p[k].y : e == 2 ? p[k].z : p[k].w;
                    const uint64_t p2 = tc::pk2(pe, pe);
                    y[k][i][0] = tc::ffma2(p2, xa, y[k][i][0]);
                    y[k][i][1] = tc::ffma2(p2, xb, y[k][i][1]);
                  }
                }
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int i = 0; i < kPart; ++i) {
                o[k][i0 + i][0] = tc::fadd2(o[k][i0 + i][0], y[k][i][0]);
                o[k][i0 + i][1] = tc::fadd2(o[k][i0 + i][1], y[k][i][1]);
              }
          }
        } else {
          // a slot that a row does not see may hold anything: 0 * NaN must not
          // reach that row
#pragma unroll 1
          for (int j = 0; j < kSTile; ++j) {
            const float* v = sV + j * ds;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (lim + j >= seen[k] || !((there >> j) & 1)) continue;
              const float pe = sP[(4 * ty + k) * kPStride + j];
              const uint64_t p2 = tc::pk2(pe, pe);
#pragma unroll
              for (int i = 0; i < kCols; ++i) {
                const float4 x = four(v + min(4 * tx + 32 * i, d4 - 4));
                o[k][i][0] = tc::ffma2(p2, lo2(x), o[k][i][0]);
                o[k][i][1] = tc::ffma2(p2, hi2(x), o[k][i][1]);
              }
            }
          }
        }
      }
      __syncthreads();
    }
    const int slot = attn_slot(w);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int x = 1; x < 8; x <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], x);
      const int r = 4 * ty + k;
      if (r >= rows) continue;
      const AttnRow x = attn_row(a, b, w.h, rt * kLRows + r);
      TQ* out = reinterpret_cast<TQ*>(a.out) + x.b * a.os[0] + x.hq * a.os[1] + x.t * a.os[2];
      float* part = a.part + ((size_t)(slot < 0 ? 0 : slot) * kLRows + r) * a.pstride;
      const float inv = l[k] == 0.f ? 0.f : 1.f / l[k];
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int col = 4 * tx + 32 * i;
        float y[4];
        tc::upk2(o[k][i][0], y[0], y[1]);
        tc::upk2(o[k][i][1], y[2], y[3]);
        if (slot >= 0) {
          if (col < d) *reinterpret_cast<float4*>(part + col) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col + e < d) store_out(out + col + e, y[e] * inv);
        }
      }
      if (tx == 0) {
        if (slot < 0)
          attn_put_lse(a, x, m[k], l[k]);
        else
          *reinterpret_cast<float2*>(part + a.pstride - 4) = make_float2(m[k], l[k]);
      }
    }
    more = attn_next<kLRows, kSTile>(a, w);
  }
}

// Joins the partials of the cut unit that began in CTA blockIdx.x: a warp per
// row, the pieces in the order of their slots:
//   M = max m_i, l = sum l_i 2^(m_i - M), O = sum O_i 2^(m_i - M) / l.
// A piece whose row saw nothing has m = -inf and l = 0 and is left out (its O is
// 0).  Which unit and how many pieces follows from the lengths alone and is found
// before the wait for the kernel that writes the partials; after it, the first
// kFly pieces of O travel together with the (m, l) pairs.
template <typename TQ, int kRows, int kTile>
__global__ void __launch_bounds__(128) k_attn_merge(const AttnDev a, int ctas) {
  constexpr int kFly = 12;
  __shared__ AttnPlanShared plan;
  pdl_trigger();  // the next call's kernel waits for this one's end
  AttnWalk w;
  int64_t total, first = 0, last = 0;
  int grid = 0;
  const int c0 = (int)blockIdx.x;
  const bool some = attn_seek<kRows, kTile, 128>(a, plan, w, total, [&](int64_t all) -> int64_t {
    grid = attn_grid(all, ctas);
    if (c0 >= grid) return -1;
    first = attn_range(all, grid, c0);
    last = attn_range(all, grid, c0 + 1);
    return last - 1;
  });
  // the unit of the range's last tile, if it begins here and ends elsewhere
  if (!some || w.g0 < first || w.g0 + w.nt <= last) {
    pdl_wait();
    return;
  }
  const int c1 = (int)attn_div((w.g0 + w.nt) * grid - 1, total);  // the CTA of its last tile
  const int pieces = c1 - c0 + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = w.item / a.nrt, rt = w.item - b * a.nrt;
  int L, n;
  attn_lengths(a, b, L, n);
  const int rows = min(kRows, a.G * n - rt * kRows);
  const int d = a.c.d;
  pdl_wait();
  if (kRows >= 128 && pieces <= 4) {
    // large units are cut into few pieces: four rows at a time, lane 4 k + i with
    // row k's (m, l) of piece i (4 x 2048 tokens over e4m3 905 us, 922 by the form below)
    for (int r0 = (blockIdx.y * 4 + warp) * 4; r0 < rows; r0 += gridDim.y * 16) {
      auto from = [&](int k, int i) {
        const int slot = i == 0 ? 2 * c0 + 1 : 2 * (c0 + i);
        return a.part + ((size_t)slot * kRows + r0 + k) * a.pstride;
      };
      const int col = lane * 4;
      float4 v[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (r0 + k < rows && i < pieces && col < d)
            v[k][i] = *reinterpret_cast<const float4*>(from(k, i) + col);
        }
      float2 ml = make_float2(-CUDART_INF_F, 0.f);
      if (lane < 16 && r0 + (lane >> 2) < rows && (lane & 3) < pieces)
        ml = *reinterpret_cast<const float2*>(from(lane >> 2, lane & 3) + a.pstride - 4);
      float M = fmaxf(ml.x, __shfl_xor_sync(0xffffffffu, ml.x, 1));
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 2));
      const float wt = ml.x == -CUDART_INF_F ? 0.f : attn_ex2(ml.x - M);
      float l = ml.x == -CUDART_INF_F ? ml.y : ml.y * wt;
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (lane < 16 && (lane & 3) == 0 && r0 + (lane >> 2) < rows)
        attn_put_lse(a, attn_row(a, b, w.h, rt * kRows + r0 + (lane >> 2)), M, l);
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = __shfl_sync(0xffffffffu, wt, 4 * k + i);
          o.x = fmaf(f, v[k][i].x, o.x);
          o.y = fmaf(f, v[k][i].y, o.y);
          o.z = fmaf(f, v[k][i].z, o.z);
          o.w = fmaf(f, v[k][i].w, o.w);
        }
        const float f = __shfl_sync(0xffffffffu, inv, 4 * k);
        if (r0 + k < rows && col < d) {
          const AttnRow x = attn_row(a, b, w.h, rt * kRows + r0 + k);
          __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + x.b * a.os[0] +
                               x.hq * a.os[1] + x.t * a.os[2];
          *reinterpret_cast<uint2*>(out + col) =
              make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
        }
      }
    }
    return;
  }
  for (int r = blockIdx.y * 4 + warp; r < rows; r += gridDim.y * 4) {
    auto piece = [&](int i) {
      const int slot = i == 0 ? 2 * c0 + 1 : 2 * (c0 + i);
      return a.part + ((size_t)slot * kRows + r) * a.pstride;
    };
    float4 v[kFly];
#pragma unroll
    for (int k = 0; k < kFly; ++k)
      if (k < pieces && lane * 4 < d) v[k] = *reinterpret_cast<const float4*>(piece(k) + lane * 4);
    auto stats = [&](int i) {
      return i < pieces ? *reinterpret_cast<const float2*>(piece(i) + a.pstride - 4)
                        : make_float2(-CUDART_INF_F, 0.f);
    };
    float2 ml = stats(lane);  // of piece i0 + lane
    float M = ml.x;
    for (int i0 = 32; i0 < pieces; i0 += 32) M = fmaxf(M, stats(i0 + lane).x);
    M = warp_max(M);
    auto weight = [&](float2 y) { return y.x == -CUDART_INF_F ? 0.f : attn_ex2(y.x - M); };
    auto sum_of = [&](float2 y) { return y.x == -CUDART_INF_F ? y.y : y.y * weight(y); };
    float l = sum_of(ml);
    for (int i0 = 32; i0 < pieces; i0 += 32) l += sum_of(stats(i0 + lane));
    l = warp_sum(l);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const AttnRow x = attn_row(a, b, w.h, rt * kRows + r);
    TQ* out = reinterpret_cast<TQ*>(a.out) + x.b * a.os[0] + x.hq * a.os[1] + x.t * a.os[2];
    for (int c = 0; c < d; c += 128) {
      const int col = c + lane * 4;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i0 = 0; i0 < pieces; i0 += 32) {
        const float wt = weight(i0 == 0 ? ml : stats(i0 + lane));
        const int end = min(32, pieces - i0);
        for (int k0 = 0; k0 < end; k0 += kFly) {
          if (i0 + k0 + c > 0) {
#pragma unroll
            for (int k = 0; k < kFly; ++k)
              if (k0 + k < end && col < d)
                v[k] = *reinterpret_cast<const float4*>(piece(i0 + k0 + k) + col);
          }
#pragma unroll
          for (int k = 0; k < kFly; ++k) {
            const float f = __shfl_sync(0xffffffffu, wt, (k0 + k) & 31);
            if (k0 + k < end && col < d) {
              o.x = fmaf(f, v[k].x, o.x);
              o.y = fmaf(f, v[k].y, o.y);
              o.z = fmaf(f, v[k].z, o.z);
              o.w = fmaf(f, v[k].w, o.w);
            }
          }
        }
      }
      const float y[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
      if (sizeof(TQ) == 2 && d % 4 == 0 && ((uintptr_t)out & 7) == 0) {
        if (col < d)
          *reinterpret_cast<uint2*>(out + col) =
              make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (col + k < d) store_out(out + col + k, y[k]);
      }
    }
    if (lane == 0) attn_put_lse(a, x, M, l);
  }
}

// Both kernels are launched after their predecessor's end, unlike the others: with the
// programmatic launch a call of one token took up to 1.7 times as long for head dims of
// 65 to 128 (8 sequences of 2500 to 5000 slots, 8 heads: fp32, d = 128 137 us against 95;
// bf16, d = 80 96 against 64, and 371 against 223 for 16K slots), while the others won a
// microsecond or two.  The SMs keep their
// split between shared memory and L1 while a kernel is on them, so fewer of these CTAs
// fit (with the largest share of shared memory asked for, the loss was gone, at 2 to 3 %
// of every call for the smaller L1).
constexpr bool kSimtEarly = false;

template <typename TQ, typename TP>
cudaError_t launch_simt(const AttnDev& a, cudaStream_t st) {
  auto bytes = [](int d) {
    return ((size_t)(kSRows + 2 * kSTile) * row_stride(d) + 4 * kSTile * 4) * sizeof(float);
  };
  const size_t smem = bytes(a.c.d);
  const auto kern = k_attn_simt<TQ, TP>;
  cudaError_t e = allow_smem<k_attn_simt<TQ, TP>>((int)bytes(256));
  if (e != cudaSuccess) return e;
  return launch_ex(kern, dim3(kSCtas), dim3(kSThreads), smem, st, kSimtEarly, 1, a);
}

template <typename TQ, typename TP, int kCols>
cudaError_t launch_simt_cols(const AttnDev& a, int ctas, cudaStream_t st) {
  auto bytes = [](int d) {
    return ((size_t)(kLRows + 2 * kSTile) * row_stride(d) + kLRows * kPStride) * sizeof(float);
  };
  cudaError_t e = allow_smem<k_attn_simt_tile<TQ, TP, kCols>>((int)bytes(32 * kCols));
  if (e != cudaSuccess) return e;
  return launch_ex(k_attn_simt_tile<TQ, TP, kCols>, dim3(ctas), dim3(kSThreads), bytes(a.c.d), st,
                   kSimtEarly, 1, a);
}

template <typename TQ, typename TP>
cudaError_t launch_simt_tile(const AttnDev& a, int ctas, cudaStream_t st) {
  if (a.c.d <= 32) return launch_simt_cols<TQ, TP, 1>(a, ctas, st);
  if (a.c.d <= 64) return launch_simt_cols<TQ, TP, 2>(a, ctas, st);
  if (a.c.d <= 128) return launch_simt_cols<TQ, TP, 4>(a, ctas, st);
  return launch_simt_cols<TQ, TP, 8>(a, ctas, st);
}

}  // namespace

// Tiles of 64 rows where they are filled twice; below that, pieces of 16, which
// read K and V again but leave more CTAs at work.  Both measured (fp32 slots, d = 64, us
// by 16 and by 64 rows): two sequences of 1501 with 111 rows x 2 heads 35 and 43, one of
// 4000 with 70 x 4 41 and 61, with 72 x 8 66 and 68, one of 3000 with 420 x 8 199 and
// 125, one of 1000 with 1200 x 2 58 and 59; 300 x 8 over 3000 with d = 128 232 and 158,
// with d = 256 490 and 517.
AttnGrid attn_grid_simt(int64_t rows, int d) {
  if (rows <= 128) return {kSCtas, kSRows, kSTile};
  return {d <= 64 ? kLCtas3 : kLCtas, kLRows, kSTile};
}

template <typename TQ, typename TP>
static cudaError_t launch_simt_types(const AttnDev& a, AttnGrid g, cudaStream_t st) {
  return g.rows == kSRows ? launch_simt<TQ, TP>(a, st) : launch_simt_tile<TQ, TP>(a, g.ctas, st);
}

cudaError_t launch_attn_simt(const AttnDev& a, AttnGrid g, int page_dtype, int q_dtype,
                             cudaStream_t st) {
  if (q_dtype == DROPKV_BF16) {
    if (page_dtype == DROPKV_BF16) return launch_simt_types<__nv_bfloat16, __nv_bfloat16>(a, g, st);
    if (page_dtype == DROPKV_F32) return launch_simt_types<__nv_bfloat16, float>(a, g, st);
    return launch_simt_types<__nv_bfloat16, E4M3>(a, g, st);
  }
  if (page_dtype == DROPKV_BF16) return launch_simt_types<float, __nv_bfloat16>(a, g, st);
  if (page_dtype == DROPKV_F32) return launch_simt_types<float, float>(a, g, st);
  return launch_simt_types<float, E4M3>(a, g, st);
}

template <typename TQ, int kRows, int kTile>
cudaError_t launch_merge(const AttnDev& a, int ctas, cudaStream_t st) {
  // a warp per row or two; per eight rows of the largest units, which are cut
  // into few pieces
  const int most = a.G * a.T < kRows ? a.G * a.T : kRows;
  const int per = kRows == 256 ? 32 : kRows > 16 ? 8 : 4;
  return launch_ex(k_attn_merge<TQ, kRows, kTile>, dim3(ctas, (most + per - 1) / per), dim3(128), 0,
                   st, true, 1, a, ctas);
}

cudaError_t launch_attn_merge(const AttnDev& a, AttnGrid g, int q_dtype, cudaStream_t st) {
  if (g.tile == kSTile && g.rows == kLRows)
    return q_dtype == DROPKV_F32 ? launch_merge<float, kLRows, kSTile>(a, g.ctas, st)
                                 : launch_merge<__nv_bfloat16, kLRows, kSTile>(a, g.ctas, st);
  if (q_dtype == DROPKV_F32) return launch_merge<float, kSRows, kSTile>(a, g.ctas, st);
  if (g.tile == kSTile) return launch_merge<__nv_bfloat16, kSRows, kSTile>(a, g.ctas, st);
  if (g.rows == 8) return launch_merge<__nv_bfloat16, 8, 128>(a, g.ctas, st);
  if (g.rows == 16) return launch_merge<__nv_bfloat16, 16, 128>(a, g.ctas, st);
  if (g.rows == 128) return launch_merge<__nv_bfloat16, 128, 128>(a, g.ctas, st);
  return launch_merge<__nv_bfloat16, 256, 128>(a, g.ctas, st);
}

}  // namespace dropkv
