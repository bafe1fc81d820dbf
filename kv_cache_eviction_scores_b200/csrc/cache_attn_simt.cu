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
// lanes' float4 reads of 32 rows touch every bank evenly.
#include "cache_attn.cuh"

namespace dropkv {

namespace {

constexpr int kSRows = 16, kSTile = 32, kSThreads = 128, kSCtas = 592;  // four CTAs an SM

__device__ __forceinline__ float4 four(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 four(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ float4 four(const E4M3* p) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  const float2 a = unpack_e4m3(w & 0xFFFFu), b = unpack_e4m3(w >> 16);
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float single(const float* p) { return *p; }
__device__ __forceinline__ float single(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float single(const E4M3* p) { return unpack_e4m3(p->bits).x; }
__device__ __forceinline__ void store_out(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Floats between rows in shared memory: d in whole float4s, an odd number of them.
__host__ __device__ __forceinline__ int row_stride(int d) { return (((d + 3) / 4) | 1) * 4; }

// One pool row (or zeros) to fp32 in shared memory, by one warp.
template <typename TP>
__device__ __forceinline__ void widen_row(float* dst, const TP* pool, int64_t row, float f, int d,
                                          int lane) {
  const int d4 = (d + 3) & ~3;
  if (row < 0) {
    for (int i = lane; i < d4; i += 32) dst[i] = 0.f;
    return;
  }
  const TP* p = pool + row * d;
  if ((d & 3) == 0) {
    for (int i = lane * 4; i < d; i += 128) {
      float4 x = four(p + i);
      *reinterpret_cast<float4*>(dst + i) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
    }
  } else {
    for (int i = lane; i < d4; i += 32) dst[i] = i < d ? single(p + i) * f : 0.f;
  }
}

template <typename TQ, typename TP>
__global__ void __launch_bounds__(kSThreads) k_attn_simt(const AttnDev a) {
  extern __shared__ __align__(16) float sm[];
  __shared__ AttnPlanShared plan;
  __shared__ int64_t srow[2][kSTile];  // pool rows of a tile's slots, -1: none
  pdl_trigger();
  const int d = a.c.d, ds = row_stride(d);
  float* sQ = sm;
  float* sK = sQ + kSRows * ds;
  float* sV = sK + kSTile * ds;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* sP = sV + kSTile * ds + warp * (kSTile * 4);  // this warp's [slot][4 rows]
  int64_t total;
  int grid;
  AttnWalk w;
  bool more = attn_plan<kSRows, kSTile, kSThreads>(a, plan, w, total, grid);
  bool described = false;
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
      for (int j = warp; j < kSTile; j += 4) {
        const int64_t row = srow[t & 1][j];
        float fk = 1.f, fv = 1.f;
        if (sizeof(TP) == 1 && row >= 0) {
          fk = scale_of(a.c.ks[row]);
          fv = scale_of(a.c.vs[row]);
        }
        widen_row(sK + j * ds, reinterpret_cast<const TP*>(a.c.k), row, fk, d, lane);
        widen_row(sV + j * ds, reinterpret_cast<const TP*>(a.c.v), row, fv, d, lane);
      }
      const bool absent = srow[t & 1][lane] < 0;
      if (warp == 0 && t + 1 < w.t1) place(t + 1);
      __syncthreads();
      if (warp * 4 < rows) {
        const int slot = t * kSTile + lane;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < d; i += 4) {
          const float4 k4 = four(sK + lane * ds + i);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 q4 = four(sQ + (warp * 4 + k) * ds + i);
            s[k] = fmaf(q4.x, k4.x, s[k]);
            s[k] = fmaf(q4.y, k4.y, s[k]);
            s[k] = fmaf(q4.z, k4.z, s[k]);
            s[k] = fmaf(q4.w, k4.w, s[k]);
          }
        }
        float p[4];
        bool partly = false;  // some row of the warp does not see some slot
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool hid = slot >= seen[k] || absent;
          partly = partly || (live[k] && hid);
          const float y = hid ? -CUDART_INF_F : s[k] * a.c_log2;
          const float mt = fmaxf(m[k], warp_max(y));
          const float mu = mt == -CUDART_INF_F ? 0.f : mt;
          const float fac = attn_ex2(m[k] - mu);
          p[k] = hid ? 0.f : attn_ex2(y - mu);
          m[k] = mt;
          l[k] = l[k] * fac + warp_sum(p[k]);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[k][i] *= fac;
        }
        partly = __any_sync(0xffffffffu, partly);
        *reinterpret_cast<float4*>(sP + lane * 4) = make_float4(p[0], p[1], p[2], p[3]);
        __syncwarp();
        for (int j = 0; j < kSTile; ++j) {
          const float4 p4 = four(sP + j * 4);
          const float* v = sV + j * ds;
          const int sj = t * kSTile + j;
          // a slot that a row does not see may hold anything: 0 * NaN must not
          // reach that row
          const bool u0 = !partly || sj < seen[0], u1 = !partly || sj < seen[1];
          const bool u2 = !partly || sj < seen[2], u3 = !partly || sj < seen[3];
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
    if (slot >= 0 && (slot & 1)) {
      if (threadIdx.x == 0) attn_describe(a, w, total, grid);
      described = true;
    }
    more = attn_next<kSRows, kSTile>(a, w);
  }
  if (!described && threadIdx.x == 0) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
}

// Joins the partials of the cut unit that began in CTA blockIdx.x: a warp per
// row, the pieces in the order of their slots:
//   M = max m_i, l = sum l_i 2^(m_i - M), O = sum O_i 2^(m_i - M) / l.
// Loads of up to four pieces are in flight.  A piece whose row saw nothing has
// m = -inf and l = 0 and is left out (its O is 0).
template <typename TQ>
__global__ void __launch_bounds__(128) k_attn_merge(const AttnDev a, int unit_rows) {
  pdl_wait();
  const int4 de = a.desc[blockIdx.x];
  if (de.x < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = de.x / a.nrt, rt = de.x - b * a.nrt;
  int L, n;
  attn_lengths(a, b, L, n);
  const int rows = min(unit_rows, a.G * n - rt * unit_rows);
  const int c0 = (int)blockIdx.x, pieces = de.z - c0 + 1;
  const int d = a.c.d;
  for (int r = blockIdx.y * 4 + warp; r < rows; r += gridDim.y * 4) {
    auto piece = [&](int i) {
      const int slot = i == 0 ? 2 * c0 + 1 : 2 * (c0 + i);
      return a.part + ((size_t)slot * unit_rows + r) * a.pstride;
    };
    float M = -CUDART_INF_F, ls = 0.f;
    for (int i = lane; i < pieces; i += 32) {
      const float2 ml = *reinterpret_cast<const float2*>(piece(i) + a.pstride - 4);
      const float nm = fmaxf(M, ml.x);
      if (nm != -CUDART_INF_F || !(ml.y == 0.f)) {
        const float mu = nm == -CUDART_INF_F ? 0.f : nm;
        ls = ls * attn_ex2(M - mu) + ml.y * attn_ex2(ml.x - mu);
      }
      M = nm;
    }
    const float Mall = warp_max(M);
    const float mu = Mall == -CUDART_INF_F ? 0.f : Mall;
    const float l = warp_sum(ls * attn_ex2(M - mu));
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const AttnRow x = attn_row(a, b, de.y, rt * unit_rows + r);
    TQ* out = reinterpret_cast<TQ*>(a.out) + x.b * a.os[0] + x.hq * a.os[1] + x.t * a.os[2];
    for (int col = lane * 4; col < d; col += 128) {
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i0 = 0; i0 < pieces; i0 += 4) {
        float4 v[4];
        float wt[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (i0 + k >= pieces) break;
          const float* p = piece(i0 + k);
          v[k] = *reinterpret_cast<const float4*>(p + col);
          wt[k] = p[a.pstride - 4];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (i0 + k >= pieces) break;
          const float f = wt[k] == -CUDART_INF_F ? 0.f : attn_ex2(wt[k] - mu);
          o.x = fmaf(f, v[k].x, o.x);
          o.y = fmaf(f, v[k].y, o.y);
          o.z = fmaf(f, v[k].z, o.z);
          o.w = fmaf(f, v[k].w, o.w);
        }
      }
      const float y[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (col + k < d) store_out(out + col + k, y[k]);
    }
    if (lane == 0) attn_put_lse(a, x, Mall, l);
  }
}

template <typename TQ, typename TP>
cudaError_t launch_simt(const AttnDev& a, cudaStream_t st) {
  const size_t smem =
      ((size_t)(kSRows + 2 * kSTile) * row_stride(a.c.d) + 4 * kSTile * 4) * sizeof(float);
  const auto kern = k_attn_simt<TQ, TP>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<kSCtas, kSThreads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

AttnGrid attn_grid_simt() { return {kSCtas, kSRows}; }

cudaError_t launch_attn_simt(const AttnDev& a, int page_dtype, int q_dtype, cudaStream_t st) {
  if (q_dtype == DROPKV_BF16) {
    if (page_dtype == DROPKV_BF16) return launch_simt<__nv_bfloat16, __nv_bfloat16>(a, st);
    if (page_dtype == DROPKV_F32) return launch_simt<__nv_bfloat16, float>(a, st);
    return launch_simt<__nv_bfloat16, E4M3>(a, st);
  }
  if (page_dtype == DROPKV_BF16) return launch_simt<float, __nv_bfloat16>(a, st);
  if (page_dtype == DROPKV_F32) return launch_simt<float, float>(a, st);
  return launch_simt<float, E4M3>(a, st);
}

cudaError_t launch_attn_merge(const AttnDev& a, int ctas, int rows, int q_dtype, cudaStream_t st) {
  const dim3 grid((unsigned)ctas, (unsigned)((rows + 15) / 16));
  if (q_dtype == DROPKV_BF16)
    return launch_ex(k_attn_merge<__nv_bfloat16>, grid, dim3(128), 0, st, true, 1, a, rows);
  return launch_ex(k_attn_merge<float>, grid, dim3(128), 0, st, true, 1, a, rows);
}

}  // namespace dropkv
