// cache_attn_rows.cu -- cache attention for few query rows per KV head
// (decoding, short drafts): bf16 queries, bf16 or e4m3 pages, head dim 64/128;
// k_attn_few up to eight rows, k_attn_rows up to 16.
//
// Mathematics: the online softmax, per row with reference maximum m (log2
// units) and sum l: P = 2^(c q.k_j - m), l += sum P, O += P V; the reference
// moves only when a logit exceeds it by more than 8 (2^8 fits every type
// here), so O is rarely rescaled.  l sums the fp32 P; the P that meets V is
// taken as two bf16 parts (lower_bf16x2).  e4m3 pages: a value is widened exactly
// to bf16, K's row scale multiplies the logit and V's multiplies P before it is
// split (a power of two: exact), so nothing else is rounded.  (The products cut O's sums
// off, about 2^-24 of them a time: V of one sign comes out 1.2e-4 too small over 128K
// slots that one CTA sums, n / 64 products a warp.)
//
// What bounds it: reading the pages.  Layout: a unit of 16 rows is one
// m16n8k16 row block, so each K/V byte is used for 16 rows' products by the
// warp-level matrix instructions, whose operands come from shared memory by
// ldmatrix; eight warps of a CTA take 16 slots each of a 128-slot tile, every
// warp with its own ring of asynchronous copies (no block barrier in the
// loop).  The rows' page lookups run one step ahead of the copies, the scale
// bytes one step ahead of their use.  A 128-row tcgen05 tile would be 1/8 full
// here; the matrix work below it is a quarter of the copy's time.
#include "cache_attn.cuh"

namespace dropkv {

namespace {

constexpr int kRRows = 16, kRWarps = 8, kRThreads = 32 * kRWarps, kRTile = 16 * kRWarps;
constexpr int kRCtas = 148, kFRows = 8;

template <typename TP>
constexpr int ring_depth() {
  return sizeof(TP) == 2 ? 3 : 4;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two e4m3 bytes of x to a bf16 pair (the NaN code becomes 480; a stored NaN row
// carries it in its scale).
template <uint32_t kSel>
__device__ __forceinline__ uint32_t widen2(uint32_t x) {
  return widen_e4m3x2<kSel>(x, 0x7B807B80u);  // 2^120
}

// Byte offset of 16-byte piece `c` of row `row` in a swizzled tile of rows of
// kPieces pieces: eight consecutive rows' equal pieces fall into eight
// different 16-byte bank groups.
template <int kPieces>
__device__ __forceinline__ uint32_t swz(int row, int c) {
  const int x = kPieces >= 8 ? (c ^ (row & 7)) : (c ^ ((row >> 1) & 3));
  return (uint32_t)(row * kPieces + x) * 16u;
}

template <typename TP, int D>
struct RowsShared {
  static constexpr int kDepth = ring_depth<TP>();
  static constexpr int kRowBytes = D * (int)sizeof(TP);
  static constexpr int kHalf = 16 * kRowBytes;        // K or V of 16 slots
  static constexpr int kRing = kRWarps * kDepth * 2 * kHalf;
  static constexpr int kJoin = kRWarps * kRRows * (D + 4) * 4;  // the warps' O, over the ring
  static constexpr int kBytes = kRing > kJoin ? kRing : kJoin;
};

// A unit's rows from its warps' scaled O (all: [warp][kRows][D + 4]) and (m, l):
// to the output, or to the cut unit's partial.
template <int D, int kRows>
__device__ __forceinline__ void put_joined(const AttnDev& a, const AttnWalk& w, int b, int rt,
                                           int rows, const float2 (&sml)[kRWarps][kRows],
                                           const float* all) {
  const int slot = attn_slot(w);
  for (int i = threadIdx.x; i < rows * (D / 4); i += kRThreads) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    float M = -CUDART_INF_F;
#pragma unroll
    for (int k = 0; k < kRWarps; ++k) M = fmaxf(M, sml[k][r].x);
    float l = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kRWarps; ++k) {
      const float2 ml = sml[k][r];
      l += ml.x == -CUDART_INF_F ? ml.y : ml.y * attn_ex2(ml.x - M);
      const float4 z = *reinterpret_cast<const float4*>(all + (k * kRows + r) * (D + 4) + c);
      y.x += z.x;
      y.y += z.y;
      y.z += z.z;
      y.w += z.w;
    }
    if (slot < 0) {
      const AttnRow x = attn_row(a, b, w.h, rt * kRows + r);
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + x.b * a.os[0] +
                           x.hq * a.os[1] + x.t * a.os[2];
      const float inv = l == 0.f ? 0.f : 1.f / l;
      *reinterpret_cast<uint2*>(out + c) =
          make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
      if (c == 0) attn_put_lse(a, x, M, l);
    } else {
      float* out = a.part + ((size_t)slot * kRows + r) * a.pstride;
      *reinterpret_cast<float4*>(out + c) = y;
      if (c == 0) *reinterpret_cast<float2*>(out + a.pstride - 4) = make_float2(M, l);
    }
  }
}

template <typename TP, int D>
__global__ void __launch_bounds__(kRThreads, 1) k_attn_rows(const AttnDev a) {
  using S = RowsShared<TP, D>;
  constexpr int kDepth = S::kDepth;
  constexpr bool kScaled = sizeof(TP) == 1;
  constexpr int kPieces = S::kRowBytes / 16;
  constexpr int kPerPass = 32 / kPieces > 0 ? 32 / kPieces : 1;  // rows a warp copies at once
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ AttnPlanShared plan;
  __shared__ int srow[kRWarps][kDepth][16];       // pool rows of the ring's slots, -1: none
  __shared__ float sscale[kRWarps][2][2][16];     // K's scale times c_log2, V's scale
  __shared__ float2 sml[kRWarps][kRRows];
  attn_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, tq = lane & 3;
  uint8_t* ring = sm + warp * kDepth * 2 * S::kHalf;
  const uint32_t ring_s = smem_addr(ring);
  const uint8_t* kp = reinterpret_cast<const uint8_t*>(a.c.k);
  const uint8_t* vp = reinterpret_cast<const uint8_t*>(a.c.v);
  AttnWalk w;
  bool more = attn_plan<kRRows, kRTile, kRThreads>(a, plan, w);
  while (more) {
    const int b = w.item / a.nrt, rt = w.item - b * a.nrt;
    int L, n;
    attn_lengths(a, b, L, n);
    const int rows = min(kRRows, a.G * n - rt * kRRows);
    const int seen_all = attn_seen(a, L, n, rt * kRRows + rows - 1);
    const int seen_min = attn_seen(a, L, n, rt * kRRows);
    const int32_t* table = a.c.table + (size_t)b * a.c.max_pages;

    // the page of this lane's slot (lane & 15) of tile t: looked up one step
    // before its copy is issued
    auto look = [&](int t) {
      return look_up(a, table, t * kRTile + warp * 16 + (lane & 15), t < w.t1 ? seen_all : 0);
    };
    auto issue = [&](int st, const Look& at_) {
      const int row = pool_row(a, w.h, at_);
      if (lane < 16) srow[warp][st][lane] = row;
      const uint32_t dk = ring_s + st * 2 * S::kHalf, dv = dk + S::kHalf;
      const int c = lane % kPieces;
#pragma unroll
      for (int i = 0; i < 16 / kPerPass; ++i) {
        const int r = lane / kPieces + i * kPerPass;
        const int at = __shfl_sync(0xffffffffu, row, r);
        const size_t off = at < 0 ? 0 : (size_t)at * S::kRowBytes + c * 16;
        copy16(dk + swz<kPieces>(r, c), kp + off, at >= 0);
        copy16(dv + swz<kPieces>(r, c), vp + off, at >= 0);
      }
    };
    // the first tiles' lookups travel together
    Look first[kDepth - 1], nxt;
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) first[i] = look(w.t0 + i);
    nxt = look(w.t0 + kDepth - 1);
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) {
      issue(i, first[i]);
      copy_commit();
    }

    // the two rows of this lane's quad, and their queries as A fragments
    const int r0 = rt * kRRows + g, r1 = r0 + 8;
    const bool live0 = g < rows, live1 = g + 8 < rows;
    const int seen0 = live0 ? attn_seen(a, L, n, r0) : 0;
    const int seen1 = live1 ? attn_seen(a, L, n, r1) : 0;
    uint32_t qa[D / 16][4];
    {
      const AttnRow x0 = attn_row(a, b, w.h, live0 ? r0 : rt * kRRows);
      const AttnRow x1 = attn_row(a, b, w.h, live1 ? r1 : rt * kRRows);
      const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q);
      const __nv_bfloat16* q0 = q + x0.b * a.qs[0] + x0.hq * a.qs[1] + x0.t * a.qs[2];
      const __nv_bfloat16* q1 = q + x1.b * a.qs[0] + x1.hq * a.qs[1] + x1.t * a.qs[2];
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        if constexpr (kScaled) {
          // the product's k order follows the widened bytes: k = 2t, 2t+1 are
          // dims 4t, 4t+1, and k = 2t+8, 2t+9 dims 4t+2, 4t+3 of the 16
          uint2 u0 = make_uint2(0, 0), u1 = u0;
          if (live0) u0 = *reinterpret_cast<const uint2*>(q0 + ks * 16 + 4 * tq);
          if (live1) u1 = *reinterpret_cast<const uint2*>(q1 + ks * 16 + 4 * tq);
          qa[ks][0] = u0.x;
          qa[ks][2] = u0.y;
          qa[ks][1] = u1.x;
          qa[ks][3] = u1.y;
        } else {
          const uint32_t* p0 = reinterpret_cast<const uint32_t*>(q0 + ks * 16 + 2 * tq);
          const uint32_t* p1 = reinterpret_cast<const uint32_t*>(q1 + ks * 16 + 2 * tq);
          qa[ks][0] = live0 ? p0[0] : 0u;
          qa[ks][2] = live0 ? p0[4] : 0u;
          qa[ks][1] = live1 ? p1[0] : 0u;
          qa[ks][3] = live1 ? p1[4] : 0u;
        }
      }
    }
    float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F, l0 = 0.f, l1 = 0.f;
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.f;

    // scale bytes of the first tile (lanes 0..15 K's, 16..31 V's)
    uint32_t sbyte = 0;
    auto scale_load = [&](int st) {
      const int row = srow[warp][st][lane & 15];
      sbyte = 0;
      if (row >= 0) sbyte = __ldg((lane < 16 ? a.c.ks : a.c.vs) + row);
    };
    __syncwarp();
    if (kScaled) scale_load(0);

    int st = 0;
    for (int t = w.t0; t < w.t1; ++t) {
      copy_wait<kDepth - 2>();
      __syncwarp();  // the tile has landed for every lane, and the last one is read out
      const uint32_t valid = __ballot_sync(0xffffffffu, srow[warp][st][lane & 15] >= 0) & 0xFFFFu;
      const int base = t * kRTile + warp * 16;
      if (kScaled)
        sscale[warp][t & 1][lane >> 4][lane & 15] = scale_of(sbyte) * (lane < 16 ? a.c_log2 : 1.f);
      const int stn = st + kDepth - 1 >= kDepth ? st - 1 : st + kDepth - 1;
      issue(stn, nxt);
      copy_commit();
      nxt = look(t + kDepth);
      __syncwarp();
      const int st1 = st + 1 == kDepth ? 0 : st + 1;
      if (kScaled && t + 1 < w.t1) scale_load(st1);
      const uint32_t tk = ring_s + st * 2 * S::kHalf, tv = tk + S::kHalf;

      if (valid) {  // some slot of the 16 is there
        // S = Q K^T for slots base + {0..7} (s[0]) and {8..15} (s[1])
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const int mi = lane >> 3, mr = lane & 7;  // ldmatrix: matrix and row of this lane
        if constexpr (kScaled) {
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
            uint32_t r[4];  // slots 0-7 and 8-15 of piece c, then of piece c + 1
            ldsm4(r, tk + swz<kPieces>((mi & 1) * 8 + mr, c + (mi >> 1)));
#pragma unroll
            for (int u = 0; u < 4; ++u)
              mma16816(s[u & 1], qa[c + (u >> 1)], widen2<kBytes01>(r[u]), widen2<kBytes23>(r[u]));
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t r[4];
            ldsm4(r, tk + swz<kPieces>((mi >> 1) * 8 + mr, ks * 2 + (mi & 1)));
            mma16816(s[0], qa[ks], r[0], r[1]);
            mma16816(s[1], qa[ks], r[2], r[3]);
          }
        }
        float vs[2][2];  // V's scales of this lane's slots
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float2 kf = make_float2(a.c_log2, a.c_log2);
          if (kScaled) {
            kf = *reinterpret_cast<const float2*>(&sscale[warp][t & 1][0][x * 8 + 2 * tq]);
            const float2 vf = *reinterpret_cast<const float2*>(&sscale[warp][t & 1][1][x * 8 + 2 * tq]);
            vs[x][0] = vf.x;
            vs[x][1] = vf.y;
          }
          s[x][0] *= kf.x;
          s[x][1] *= kf.y;
          s[x][2] *= kf.x;
          s[x][3] *= kf.y;
        }
        // Slots that some row of the unit does not see.
        const bool partly = valid != 0xFFFFu || base + 16 > seen_min;
        uint32_t hid = 0;  // bit 4 x + e: s[x][e] is hidden
        if (partly) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = x * 8 + 2 * tq + (e & 1);
              const bool h = base + j >= (e < 2 ? seen0 : seen1) || !((valid >> j) & 1);
              if (h) {
                hid |= 1u << (4 * x + e);
                s[x][e] = -CUDART_INF_F;
              }
            }
        }
        float t0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        float t1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
          t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
          t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
        }
        if (__any_sync(0xffffffffu, t0 > m0 + 8.f || t1 > m1 + 8.f)) {
          const float n0 = t0 > m0 + 8.f ? t0 : m0, n1 = t1 > m1 + 8.f ? t1 : m1;
          const float f0 = m0 == -CUDART_INF_F ? 0.f : attn_ex2(m0 - n0);
          const float f1 = m1 == -CUDART_INF_F ? 0.f : attn_ex2(m1 - n1);
          m0 = n0;
          m1 = n1;
          l0 *= f0;
          l1 *= f1;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[i][0] *= f0;
            o[i][1] *= f0;
            o[i][2] *= f1;
            o[i][3] *= f1;
          }
        }
        const float u0 = m0 == -CUDART_INF_F ? 0.f : m0, u1 = m1 == -CUDART_INF_F ? 0.f : m1;
        float p[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          p[x][0] = attn_ex2(s[x][0] - u0);
          p[x][1] = attn_ex2(s[x][1] - u0);
          p[x][2] = attn_ex2(s[x][2] - u1);
          p[x][3] = attn_ex2(s[x][3] - u1);
          l0 += p[x][0] + p[x][1];
          l1 += p[x][2] + p[x][3];
          if (kScaled) {
            p[x][0] *= vs[x][0];
            p[x][1] *= vs[x][1];
            p[x][2] *= vs[x][0];
            p[x][3] *= vs[x][1];
            if (partly) {  // a NaN scale of a hidden slot
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if ((hid >> (4 * x + e)) & 1) p[x][e] = 0.f;
            }
          }
        }
        const uint32_t pa[4] = {upper_bf16x2(p[0][0], p[0][1]), upper_bf16x2(p[0][2], p[0][3]),
                                upper_bf16x2(p[1][0], p[1][1]), upper_bf16x2(p[1][2], p[1][3])};
        const uint32_t pl[4] = {lower_bf16x2(p[0][0], p[0][1]), lower_bf16x2(p[0][2], p[0][3]),
                                lower_bf16x2(p[1][0], p[1][1]), lower_bf16x2(p[1][2], p[1][3])};
        if (!kScaled && partly) {
          // A hidden slot's V may be an infinity or a NaN, and 0 * NaN must not
          // reach the rows that do not see it: such values are added to the rows
          // that do, and the products go without them.
          bool odd = false;
          const int c = lane % kPieces;
          auto piece = [&](int i) {
            return reinterpret_cast<uint4*>(ring + st * 2 * S::kHalf + S::kHalf +
                                            swz<kPieces>(lane / kPieces + i * kPerPass, c));
          };
#pragma unroll
          for (int i = 0; i < 16 / kPerPass; ++i) {
            const uint4 v = *piece(i);
            odd = odd || non_finite(v.x) || non_finite(v.y) || non_finite(v.z) || non_finite(v.w);
          }
          if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
            for (int j = 0; j < 16; ++j) {
              const int from = (lane & ~3) | ((j & 7) >> 1);
              float w0 = 0.f, w1 = 0.f;
              uint32_t h0 = 0;
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (x == (j >> 3) && e == (j & 1)) {
                    w0 = p[x][e];
                    w1 = p[x][2 + e];
                    h0 = ((hid >> (4 * x + e)) & 1) | ((hid >> (4 * x + 2 + e)) & 1) << 1;
                  }
              w0 = __shfl_sync(0xffffffffu, w0, from);
              w1 = __shfl_sync(0xffffffffu, w1, from);
              h0 = __shfl_sync(0xffffffffu, h0, from);
#pragma unroll
              for (int cc = 0; cc < D / 8; ++cc) {
                const uint32_t v2 = *reinterpret_cast<const uint32_t*>(
                    ring + st * 2 * S::kHalf + S::kHalf + swz<kPieces>(j, cc % kPieces) + 4 * tq);
                const uint32_t x2[2] = {v2 << 16, v2 & 0xFFFF0000u};
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if ((x2[e] & 0x7F800000u) == 0x7F800000u) {
                    if (!(h0 & 1)) o[cc][e] = fmaf(w0, __uint_as_float(x2[e]), o[cc][e]);
                    if (!(h0 & 2)) o[cc][2 + e] = fmaf(w1, __uint_as_float(x2[e]), o[cc][2 + e]);
                  }
              }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16 / kPerPass; ++i) {
              const uint4 v = *piece(i);
              *piece(i) = make_uint4(without_non_finite(v.x), without_non_finite(v.y),
                                     without_non_finite(v.z), without_non_finite(v.w));
            }
            __syncwarp();
          }
        }
        if constexpr (kScaled) {
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
            uint32_t r[4];  // slots 0-7 and 8-15 of piece c, then of piece c + 1
            ldsm4t(r, tv + swz<kPieces>((mi & 1) * 8 + mr, c + (mi >> 1)));
#pragma unroll
            for (int u = 0; u < 2; ++u) {  // even dims of the piece, then the odd ones
              const uint32_t e0 = widen2<kBytes02>(r[2 * u]), e1 = widen2<kBytes02>(r[2 * u + 1]);
              const uint32_t d0 = widen2<kBytes13>(r[2 * u]), d1 = widen2<kBytes13>(r[2 * u + 1]);
              mma16816(o[2 * (c + u)], pa, e0, e1);
              mma16816(o[2 * (c + u) + 1], pa, d0, d1);
              mma16816(o[2 * (c + u)], pl, e0, e1);
              mma16816(o[2 * (c + u) + 1], pl, d0, d1);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 8; c += 2) {
            uint32_t r[4];
            ldsm4t(r, tv + swz<kPieces>((mi & 1) * 8 + mr, c + (mi >> 1)));
            mma16816(o[c], pa, r[0], r[1]);
            mma16816(o[c + 1], pa, r[2], r[3]);
            mma16816(o[c], pl, r[0], r[1]);
            mma16816(o[c + 1], pl, r[2], r[3]);
          }
        }
      }
      st = st1;
    }
    copy_wait<0>();

    // join the warps: row maxima and sums, then the scaled O
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, x);
      l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }
    if (tq == 0) {
      sml[warp][g] = make_float2(m0, l0);
      sml[warp][g + 8] = make_float2(m1, l1);
    }
    __syncthreads();  // every warp's ring is read out, too
    float M0 = -CUDART_INF_F, M1 = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < kRWarps; ++i) {
      M0 = fmaxf(M0, sml[i][g].x);
      M1 = fmaxf(M1, sml[i][g + 8].x);
    }
    const float f0 = m0 == -CUDART_INF_F ? (l0 == 0.f ? 0.f : l0) : attn_ex2(m0 - M0);
    const float f1 = m1 == -CUDART_INF_F ? (l1 == 0.f ? 0.f : l1) : attn_ex2(m1 - M1);
    float* join = reinterpret_cast<float*>(sm) + warp * kRRows * (D + 4);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (!(half ? live1 : live0)) continue;
      float* to = join + (g + 8 * half) * (D + 4);
      const float f = half ? f1 : f0;
      const int e = 2 * half;
      if constexpr (kScaled) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
          *reinterpret_cast<float4*>(to + c * 16 + 4 * tq) =
              make_float4(o[2 * c][e] * f, o[2 * c + 1][e] * f, o[2 * c][e + 1] * f,
                          o[2 * c + 1][e + 1] * f);
      } else {
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<float2*>(to + c * 8 + 2 * tq) = make_float2(o[c][e] * f, o[c][e + 1] * f);
      }
    }
    __syncthreads();
    put_joined<D, kRRows>(a, w, b, rt, rows, sml, reinterpret_cast<const float*>(sm));
    more = attn_next<kRRows, kRTile>(a, w);
    if (more) __syncthreads();  // the joined rows are read out
  }
}

// ---- up to eight rows per KV head -------------------------------------------------
//
// The products the other way round: S^T = K Q^T with 16 slots as the rows of
// m16n8k16 and the (at most eight) query rows as its columns, and O^T = V^T P^T
// with 16 dims as rows.  Half the matrix instructions and half the registers of
// the kernel above, whose row block would be half empty; with e4m3 pages, whose
// tiles are half the bytes, two CTAs then fit an SM, and their warps hide each
// other's latencies, which bound that kernel there (8 rows over 64 sequences of 2K
// slots: e4m3 91 us by 16 rows, 66 by eight; bf16 97 and 95).  Four 128K bf16 caches,
// 4 rows each: 2.15 GB in 324 us, 6.6 TB/s, what reads alone reach (the copy that the
// other figures are held against, half of it writes, has 6.46).
template <typename TP, int D>
struct FewShared {
  static constexpr int kDepth = 3;
  static constexpr int kRowBytes = D * (int)sizeof(TP);
  static constexpr int kHalf = 16 * kRowBytes;  // K or V of 16 slots
  static constexpr int kRing = kRWarps * kDepth * 2 * kHalf;
  static constexpr int kJoin = kRWarps * kFRows * (D + 4) * 4;
  static constexpr int kBytes = kRing > kJoin ? kRing : kJoin;
};

template <typename TP>
constexpr int few_ctas_per_sm() {
  return sizeof(TP) == 1 ? 2 : 1;
}

// Transposes an 8 x 8 matrix of 16-bit values held by a warp as ldmatrix leaves it.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <typename TP, int D>
__global__ void __launch_bounds__(kRThreads, few_ctas_per_sm<TP>()) k_attn_few(const AttnDev a) {
  using S = FewShared<TP, D>;
  constexpr int kDepth = S::kDepth;
  constexpr bool kScaled = sizeof(TP) == 1;
  constexpr int kPieces = S::kRowBytes / 16;
  constexpr int kPerPass = 32 / kPieces;  // rows a warp copies at once
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ AttnPlanShared plan;
  __shared__ int srow[kRWarps][kDepth][16];    // pool rows of the ring's slots, -1: none
  __shared__ float sscale[kRWarps][2][2][16];  // K's scale times c_log2, V's scale
  __shared__ float2 sml[kRWarps][kFRows];
  attn_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, tq = lane & 3;
  uint8_t* ring = sm + warp * kDepth * 2 * S::kHalf;
  const uint32_t ring_s = smem_addr(ring);
  const uint8_t* kp = reinterpret_cast<const uint8_t*>(a.c.k);
  const uint8_t* vp = reinterpret_cast<const uint8_t*>(a.c.v);
  AttnWalk w;
  bool more = attn_plan<kFRows, kRTile, kRThreads>(a, plan, w);
  while (more) {
    const int b = w.item / a.nrt, rt = w.item - b * a.nrt;
    int L, n;
    attn_lengths(a, b, L, n);
    const int rows = min(kFRows, a.G * n - rt * kFRows);
    const int seen_all = attn_seen(a, L, n, rt * kFRows + rows - 1);
    const int seen_min = attn_seen(a, L, n, rt * kFRows);
    const int32_t* table = a.c.table + (size_t)b * a.c.max_pages;

    // the page of this lane's slot (lane & 15) of tile t: looked up one step
    // before its copy is issued
    auto look = [&](int t) {
      return look_up(a, table, t * kRTile + warp * 16 + (lane & 15), t < w.t1 ? seen_all : 0);
    };
    auto issue = [&](int st, const Look& at_) {
      const int row = pool_row(a, w.h, at_);
      if (lane < 16) srow[warp][st][lane] = row;
      const uint32_t dk = ring_s + st * 2 * S::kHalf, dv = dk + S::kHalf;
      const int c = lane % kPieces;
#pragma unroll
      for (int i = 0; i < 16 / kPerPass; ++i) {
        const int r = lane / kPieces + i * kPerPass;
        const int at = __shfl_sync(0xffffffffu, row, r);
        const size_t off = at < 0 ? 0 : (size_t)at * S::kRowBytes + c * 16;
        copy16(dk + swz<kPieces>(r, c), kp + off, at >= 0);
        copy16(dv + swz<kPieces>(r, c), vp + off, at >= 0);
      }
    };
    // the first tiles' lookups travel together
    Look first[kDepth - 1], nxt;
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) first[i] = look(w.t0 + i);
    nxt = look(w.t0 + kDepth - 1);
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) {
      issue(i, first[i]);
      copy_commit();
    }

    // query row g as a B fragment (k: dims, n: rows), and the two rows whose
    // logits this lane holds
    uint32_t qb[D / 16][2];
    {
      const bool on = g < rows;
      const AttnRow x = attn_row(a, b, w.h, rt * kFRows + (on ? g : 0));
      const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + x.b * a.qs[0] +
                               x.hq * a.qs[1] + x.t * a.qs[2];
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        if constexpr (kScaled) {
          // k in the order of the widened bytes: 2t, 2t+1 are dims 4t, 4t+1, and
          // 2t+8, 2t+9 dims 4t+2, 4t+3 of the 16
          const uint2 u = on ? *reinterpret_cast<const uint2*>(q + ks * 16 + 4 * tq) : make_uint2(0, 0);
          qb[ks][0] = u.x;
          qb[ks][1] = u.y;
        } else {
          const uint32_t* p = reinterpret_cast<const uint32_t*>(q + ks * 16 + 2 * tq);
          qb[ks][0] = on ? p[0] : 0u;
          qb[ks][1] = on ? p[4] : 0u;
        }
      }
    }
    const int q0 = 2 * tq, q1 = q0 + 1;
    const int seen0 = q0 < rows ? attn_seen(a, L, n, rt * kFRows + q0) : 0;
    const int seen1 = q1 < rows ? attn_seen(a, L, n, rt * kFRows + q1) : 0;
    float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F, l0 = 0.f, l1 = 0.f;
    float o[D / 16][4];  // dims g, g + 8 (e4m3: 2 g, 2 g + 1) of each 16; rows q0, q1
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.f;

    // scale bytes of the first tile (lanes 0..15 K's, 16..31 V's)
    uint32_t sbyte = 0;
    auto scale_load = [&](int st) {
      const int row = srow[warp][st][lane & 15];
      sbyte = 0;
      if (row >= 0)
        asm volatile("ld.global.nc.u8 %0, [%1];"
                     : "=r"(sbyte)
                     : "l"((lane < 16 ? a.c.ks : a.c.vs) + row));
    };
    __syncwarp();
    if (kScaled) scale_load(0);

    int st = 0;
    for (int t = w.t0; t < w.t1; ++t) {
      copy_wait<kDepth - 2>();
      __syncwarp();  // the tile has landed for every lane, and the last one is read out
      const uint32_t valid = __ballot_sync(0xffffffffu, srow[warp][st][lane & 15] >= 0) & 0xFFFFu;
      const int base = t * kRTile + warp * 16;
      if (kScaled)
        sscale[warp][t & 1][lane >> 4][lane & 15] = scale_of(sbyte) * (lane < 16 ? a.c_log2 : 1.f);
      const int stn = st + kDepth - 1 >= kDepth ? st - 1 : st + kDepth - 1;
      issue(stn, nxt);
      copy_commit();
      nxt = look(t + kDepth);
      __syncwarp();
      const int st1 = st + 1 == kDepth ? 0 : st + 1;
      if (kScaled && t + 1 < w.t1) scale_load(st1);
      const uint32_t tk = ring_s + st * 2 * S::kHalf, tv = tk + S::kHalf;
      if (valid) {  // some slot of the 16 is there
        const int mi = lane >> 3, mr = lane & 7;  // ldmatrix: matrix and row of this lane
        // S^T of slots g (s[0], s[1]) and g + 8 (s[2], s[3]) for rows q0, q1
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
        if constexpr (kScaled) {
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
            uint32_t r[4];  // slots 0-7 and 8-15 of piece c, then of piece c + 1
            ldsm4(r, tk + swz<kPieces>((mi & 1) * 8 + mr, c + (mi >> 1)));
            const uint32_t ka[4] = {widen2<kBytes01>(r[0]), widen2<kBytes01>(r[1]),
                                    widen2<kBytes23>(r[0]), widen2<kBytes23>(r[1])};
            const uint32_t kb[4] = {widen2<kBytes01>(r[2]), widen2<kBytes01>(r[3]),
                                    widen2<kBytes23>(r[2]), widen2<kBytes23>(r[3])};
            mma16816(s, ka, qb[c][0], qb[c][1]);
            mma16816(s2, kb, qb[c + 1][0], qb[c + 1][1]);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < D / 16; ks += 2) {
            uint32_t r[4], r2[4];
            ldsm4(r, tk + swz<kPieces>((mi & 1) * 8 + mr, ks * 2 + (mi >> 1)));
            ldsm4(r2, tk + swz<kPieces>((mi & 1) * 8 + mr, ks * 2 + 2 + (mi >> 1)));
            mma16816(s, r, qb[ks][0], qb[ks][1]);
            mma16816(s2, r2, qb[ks + 1][0], qb[ks + 1][1]);
          }
        }
        float kf0 = a.c_log2, kf1 = a.c_log2, vf0 = 1.f, vf1 = 1.f;  // slots g, g + 8
        if (kScaled) {
          kf0 = sscale[warp][t & 1][0][g];
          kf1 = sscale[warp][t & 1][0][g + 8];
          vf0 = sscale[warp][t & 1][1][g];
          vf1 = sscale[warp][t & 1][1][g + 8];
        }
        s[0] = (s[0] + s2[0]) * kf0;
        s[1] = (s[1] + s2[1]) * kf0;
        s[2] = (s[2] + s2[2]) * kf1;
        s[3] = (s[3] + s2[3]) * kf1;
        // slots that some row of the unit does not see
        const bool partly = valid != 0xFFFFu || base + 16 > seen_min;
        uint32_t hid = 0;  // bit e: s[e] is hidden
        if (partly) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = g + 8 * (e >> 1);
            if (base + j >= (e & 1 ? seen1 : seen0) || !((valid >> j) & 1)) {
              hid |= 1u << e;
              s[e] = -CUDART_INF_F;
            }
          }
        }
        float t0 = fmaxf(s[0], s[2]), t1 = fmaxf(s[1], s[3]);
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
          t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
        }
        if (__any_sync(0xffffffffu, t0 > m0 + 8.f || t1 > m1 + 8.f)) {
          const float n0 = t0 > m0 + 8.f ? t0 : m0, n1 = t1 > m1 + 8.f ? t1 : m1;
          const float f0 = m0 == -CUDART_INF_F ? 0.f : attn_ex2(m0 - n0);
          const float f1 = m1 == -CUDART_INF_F ? 0.f : attn_ex2(m1 - n1);
          m0 = n0;
          m1 = n1;
          l0 *= f0;
          l1 *= f1;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            o[i][0] *= f0;
            o[i][1] *= f1;
            o[i][2] *= f0;
            o[i][3] *= f1;
          }
        }
        const float u0 = m0 == -CUDART_INF_F ? 0.f : m0, u1 = m1 == -CUDART_INF_F ? 0.f : m1;
        float p[4] = {attn_ex2(s[0] - u0), attn_ex2(s[1] - u1), attn_ex2(s[2] - u0),
                      attn_ex2(s[3] - u1)};
        l0 += p[0] + p[2];
        l1 += p[1] + p[3];
        if (kScaled) {
          p[0] *= vf0;
          p[1] *= vf0;
          p[2] *= vf1;
          p[3] *= vf1;
          if (partly) {  // a NaN scale of a hidden slot
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((hid >> e) & 1) p[e] = 0.f;
          }
        }
        // P^T as a B fragment (k: slots, n: rows)
        const uint32_t pb0 = transpose8(upper_bf16x2(p[0], p[1]));
        const uint32_t pb1 = transpose8(upper_bf16x2(p[2], p[3]));
        const uint32_t pl0 = transpose8(lower_bf16x2(p[0], p[1]));
        const uint32_t pl1 = transpose8(lower_bf16x2(p[2], p[3]));
        if (!kScaled && partly) {
          // A hidden slot's V may be an infinity or a NaN, and 0 * NaN must not
          // reach the rows that do not see it: such values are added to the rows
          // that do, and the products go without them.
          bool odd = false;
          const int c = lane % kPieces;
          auto piece = [&](int i) {
            return reinterpret_cast<uint4*>(ring + st * 2 * S::kHalf + S::kHalf +
                                            swz<kPieces>(lane / kPieces + i * kPerPass, c));
          };
#pragma unroll
          for (int i = 0; i < 16 / kPerPass; ++i) {
            const uint4 v = *piece(i);
            odd = odd || non_finite(v.x) || non_finite(v.y) || non_finite(v.z) || non_finite(v.w);
          }
          if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
            for (int j = 0; j < 16; ++j) {
              const int from = (j & 7) * 4 + tq;
              const float w0 = __shfl_sync(0xffffffffu, j < 8 ? p[0] : p[2], from);
              const float w1 = __shfl_sync(0xffffffffu, j < 8 ? p[1] : p[3], from);
              const uint32_t h = __shfl_sync(0xffffffffu, j < 8 ? hid : hid >> 2, from);
#pragma unroll
              for (int cc = 0; cc < D / 16; ++cc)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t x = (uint32_t) * reinterpret_cast<const uint16_t*>(
                      ring + st * 2 * S::kHalf + S::kHalf + swz<kPieces>(j, (2 * cc + e) % kPieces) +
                      2 * g) << 16;
                  if ((x & 0x7F800000u) == 0x7F800000u) {
                    if (!(h & 1)) o[cc][2 * e] = fmaf(w0, __uint_as_float(x), o[cc][2 * e]);
                    if (!(h & 2)) o[cc][2 * e + 1] = fmaf(w1, __uint_as_float(x), o[cc][2 * e + 1]);
                  }
                }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16 / kPerPass; ++i) {
              const uint4 v = *piece(i);
              *piece(i) = make_uint4(without_non_finite(v.x), without_non_finite(v.y),
                                     without_non_finite(v.z), without_non_finite(v.w));
            }
            __syncwarp();
          }
        }
        if constexpr (kScaled) {
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
            uint32_t r[4];  // slots 0-7 and 8-15 of piece c, then of piece c + 1
            ldsm4t(r, tv + swz<kPieces>((mi & 1) * 8 + mr, c + (mi >> 1)));
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t va[4] = {widen2<kBytes02>(r[2 * u]), widen2<kBytes13>(r[2 * u]),
                                      widen2<kBytes02>(r[2 * u + 1]), widen2<kBytes13>(r[2 * u + 1])};
              mma16816(o[c + u], va, pb0, pb1);
              mma16816(o[c + u], va, pl0, pl1);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t r[4];  // dims 0-7 and 8-15 of slots 0-7, then of slots 8-15
            ldsm4t(r, tv + swz<kPieces>((mi >> 1) * 8 + mr, 2 * c + (mi & 1)));
            mma16816(o[c], r, pb0, pb1);
            mma16816(o[c], r, pl0, pl1);
          }
        }
      }
      st = st1;
    }
    copy_wait<0>();

    // join the warps: row maxima and sums, then the scaled O
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, x);
      l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }
    if (g == 0) {
      sml[warp][q0] = make_float2(m0, l0);
      sml[warp][q1] = make_float2(m1, l1);
    }
    __syncthreads();  // every warp's ring is read out, too
    float M0 = -CUDART_INF_F, M1 = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < kRWarps; ++i) {
      M0 = fmaxf(M0, sml[i][q0].x);
      M1 = fmaxf(M1, sml[i][q1].x);
    }
    const float f0 = m0 == -CUDART_INF_F ? (l0 == 0.f ? 0.f : l0) : attn_ex2(m0 - M0);
    const float f1 = m1 == -CUDART_INF_F ? (l1 == 0.f ? 0.f : l1) : attn_ex2(m1 - M1);
    float* join = reinterpret_cast<float*>(sm) + warp * kFRows * (D + 4);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if ((e ? q1 : q0) >= rows) continue;
      float* to = join + (e ? q1 : q0) * (D + 4);
      const float f = e ? f1 : f0;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        if constexpr (kScaled) {
          *reinterpret_cast<float2*>(to + c * 16 + 2 * g) = make_float2(o[c][e] * f, o[c][2 + e] * f);
        } else {
          to[c * 16 + g] = o[c][e] * f;
          to[c * 16 + 8 + g] = o[c][2 + e] * f;
        }
      }
    }
    __syncthreads();
    put_joined<D, kFRows>(a, w, b, rt, rows, sml, reinterpret_cast<const float*>(sm));
    more = attn_next<kFRows, kRTile>(a, w);
    if (more) __syncthreads();  // the joined rows are read out
  }
}

template <typename TP, int D>
cudaError_t launch_rows(const AttnDev& a, cudaStream_t st) {
  const auto kern = k_attn_rows<TP, D>;
  constexpr int smem = RowsShared<TP, D>::kBytes;
  cudaError_t e = allow_smem<k_attn_rows<TP, D>>(smem);
  if (e != cudaSuccess) return e;
  return launch_ex(kern, dim3(kRCtas), dim3(kRThreads), smem, st, true, 1, a);
}

template <typename TP, int D>
cudaError_t launch_few(const AttnDev& a, cudaStream_t st) {
  constexpr int smem = FewShared<TP, D>::kBytes;
  cudaError_t e = allow_smem<k_attn_few<TP, D>>(smem);
  if (e != cudaSuccess) return e;
  return launch_ex(k_attn_few<TP, D>, dim3(kRCtas * few_ctas_per_sm<TP>()), dim3(kRThreads), smem, st,
                   true, 1, a);
}

}  // namespace

AttnGrid attn_grid_rows() { return {kRCtas, kRRows, kRTile}; }
AttnGrid attn_grid_few(int page_dtype) {
  const int per = page_dtype == DROPKV_E4M3 ? few_ctas_per_sm<E4M3>() : few_ctas_per_sm<__nv_bfloat16>();
  return {kRCtas * per, kFRows, kRTile};
}

cudaError_t launch_attn_rows(const AttnDev& a, int page_dtype, cudaStream_t st) {
  if (page_dtype == DROPKV_BF16)
    return a.c.d == 128 ? launch_rows<__nv_bfloat16, 128>(a, st)
                        : launch_rows<__nv_bfloat16, 64>(a, st);
  return a.c.d == 128 ? launch_rows<E4M3, 128>(a, st) : launch_rows<E4M3, 64>(a, st);
}

cudaError_t launch_attn_few(const AttnDev& a, int page_dtype, cudaStream_t st) {
  if (page_dtype == DROPKV_BF16)
    return a.c.d == 128 ? launch_few<__nv_bfloat16, 128>(a, st)
                        : launch_few<__nv_bfloat16, 64>(a, st);
  return a.c.d == 128 ? launch_few<E4M3, 128>(a, st) : launch_few<E4M3, 64>(a, st);
}

}  // namespace dropkv
