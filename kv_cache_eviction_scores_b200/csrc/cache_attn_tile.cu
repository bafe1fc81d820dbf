// cache_attn_tile.cu -- cache attention for many query rows per KV head (chunks
// of a prompt, long drafts): bf16 queries, bf16 or e4m3 pages, head dim 64/128,
// on tcgen05 with the accumulators in TMEM.
//
// Mathematics: the online softmax of the row kernel (reference maximum in
// log2 units that moves only when a logit exceeds it by more than 8; fp32 P
// summed into l, P as two bf16 parts for P V), one query row per thread.
// e4m3 pages are widened to bf16 with their scale as they are staged: a
// 4-bit significand times a power of two is a bf16 exactly, wherever bf16 has
// the exponent (a row whose scale is under 2^-119 holds nothing above 2^-110,
// and rounds there).
//
// Layout: a unit of 256 rows is two query tiles of 128 rows against tiles of
// 128 slots; a staged K/V tile serves both, so the staging (four producer
// warps there: page lookups, asynchronous 16-byte copies or, for e4m3, loads, the
// widening and stores) is paid once per 256 rows.  Per query tile u: S_u = Q_u
// K^T (M = N = 128) in TMEM columns 128 u, P_u over it (each half of P over the
// half of S that it comes from; of each 16 slots eight columns of upper parts, then
// eight of lower ones), O_u at 256 + 128 u, all 512 columns.  One softmax warpgroup
// per query tile; while one tile's softmax runs, the other tile's MMAs fill the
// tensor pipe.  P V of a tile begins when the upper half of P is there.
// kAlt (units of at most 128 rows, which read more than they compute): one query
// tile, one softmax warpgroup and eight producer warps; S of the next slot tile
// goes to the other of two S/P buffers while this one's softmax runs, so that the
// softmax waits for no product.
//
// Every role walks the CTA's range by itself, so that staging runs on into the
// next unit while the last one is finished.  A slot without a page and the
// slots that no row of the unit sees are staged as zeros and hidden by a mask
// bit each.  Slots that only some rows see can hold an infinity or a NaN, and
// 0 * NaN must not reach the other rows: the producers stage such values as 0
// and raise the unit's flag, and the rows that do see them add them at the end.
//
// Every wait on an mbarrier is bounded (kWaitClocks, or the self-test's limit); on expiry the
// kernel records DROPKV_ERR_TIMEOUT, every role leaves, and TMEM is freed.
#include <type_traits>

#include "cache_attn.cuh"
#include "tc_ptx.cuh"

namespace dropkv {

namespace {

using namespace tc;

constexpr int kTTile = 128, kTCtas = 148;
constexpr int kTMmaWarp = 12;  // the softmax warps, the producers, then the MMA issuers
constexpr uint32_t kTColO = 256;
// The tensor core cuts its sums off, by 1.7 x 2^-24 of them on average at each of a slot
// tile's 16 P V steps: always downwards, so that O over 128K slots of V of one sign came
// out 1.6e-3 too small (half a step of bf16 is 2e-3 to 3.9e-3).  So every kFold slot
// tiles the softmax threads add O to their rows in the workspace, rounding to nearest,
// and P V begins from 0: 1.2e-4 then, for 0 to 3 % of the time (256 tokens x 8 over 64K
// bf16 slots 777 us, 748 to 781 without; 16 tokens x 8 over 128K e4m3 slots 963 and 967).
// Every 64 tiles: 8e-5, and 4 to 7 % (807 us).
constexpr int kFold = 128;

template <typename TP, int D, bool kAlt>
struct TileShared {
  static constexpr int kSoftmax = kAlt ? 4 : 8, kProd = kTMmaWarp - kSoftmax;  // warps
  static constexpr int kThreads = 32 * (kTMmaWarp + (kAlt ? 1 : 2));
  static constexpr bool kScaled = sizeof(TP) == 1;
  static constexpr int kStages = kAlt && !kScaled ? 3 : 2;
  static constexpr int kRing = !kScaled ? 0 : kAlt ? 4 : 2;  // e4m3 K or V tiles on their way
  static constexpr int kQTiles = kAlt ? 1 : 2;
  static constexpr int kBox = 128 * 128;                   // 128 rows x 64 bf16, 128-byte swizzle
  static constexpr int kTileBytes = D / 64 * kBox;
  static constexpr int kBars = 2 + 4 * kStages + 11;
  static constexpr int oK = kQTiles * kTileBytes;
  static constexpr int oV = oK + kStages * kTileBytes;
  static constexpr int oRaw = oV + kStages * kTileBytes;
  static constexpr int oBars = oRaw + kRing * 128 * D;
  static constexpr int oMask = oBars + (kBars + 1) / 2 * 16;  // [8][kProd] words of a bit a slot, 16 bytes a tile
  static constexpr int oOdd = oMask + 128;                    // int [2]
  static constexpr int oMisc = oOdd + 16;                     // TMEM base
  static constexpr int oPlan = oMisc + 16;
  static constexpr int kBytes = oPlan + (int)sizeof(AttnPlanShared);
};

__device__ __forceinline__ float f32(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t u32(float f) { return __float_as_uint(f); }

// A wait has run out: this role leaves, and the waits on it run out in turn.
__device__ __forceinline__ void fail(const AttnDev& a) {
  if (a.status) atomicMax(a.status, (int)DROPKV_ERR_TIMEOUT);
}
// Waits are bounded by the SM's clock: reading %globaltimer takes too long for
// loops that have to see a barrier at once.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, long long limit) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > limit) return false;
  return true;
}

__device__ __forceinline__ void sts16(uint32_t dst, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(src)
               : "memory");
  return v;
}

// 64 consecutive 32-bit columns for every lane, in two loads with one wait.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
#define DKV_O32(i) DKV_O8(i), DKV_O8(i + 8), DKV_O8(i + 16), DKV_O8(i + 24)
#define DKV_O8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
                  "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, "
      "%8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, "
      "%24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, "
      "%40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, "
      "%56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : DKV_O32(0), DKV_O32(32)
      : "r"(taddr), "r"(taddr + 32u)
      : "memory");
#undef DKV_O8
#undef DKV_O32
}
// One byte, or 0 when !on; volatile, so that it is requested here and not where
// it is used.
__device__ __forceinline__ uint32_t ldg1(const uint8_t* p, bool on) {
  uint32_t v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t"
      "@p ld.global.nc.u8 %0, [%1];\n\t}"
      : "=&r"(v)
      : "l"(p), "r"((int)on));
  return v;
}

// Byte offset of 16-byte piece c (eight bf16) of row r in a staged tile.
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  return (uint32_t)((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// A row scale 2^(byte - 127) as two bf16 factors for the bits of e4m3 on their
// way to bf16 (the seven magnitude bits at the bottom of the exponent: the value
// times 2^-120): 2^(byte - 7), 2^127 at most, in the lower half; the rest, 1 but
// for bytes above 134, in the upper.  NaN for 255.
__device__ __forceinline__ uint32_t widen_factors(uint32_t byte) {
  if (byte == 255u) return 0x3F807FC0u;
  return ((min(byte, 134u) + 120u) << 7) | (byte <= 134u ? 0x3F80u : (byte - 134u + 127u) << 7) << 16;
}
// The rows of one unit as a role sees them.
struct Unit {
  int b, rt, rows, seen_all, seen_min, L, n;
};
template <int kRows>
__device__ __forceinline__ Unit unit_of(const AttnDev& a, const AttnWalk& w) {
  Unit x;
  x.b = w.item / a.nrt;
  x.rt = w.item - x.b * a.nrt;
  attn_lengths(a, x.b, x.L, x.n);
  x.rows = min(kRows, a.G * x.n - x.rt * kRows);
  x.seen_all = attn_seen(a, x.L, x.n, x.rt * kRows + x.rows - 1);
  x.seen_min = attn_seen(a, x.L, x.n, x.rt * kRows);
  return x;
}

__device__ __forceinline__ void prefetch_l2(const float* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
// o += 2^(mp - m) from, and to = o, over 32 columns.
__device__ __forceinline__ void add_part(uint32_t (&o)[32], const float* from, float mp, float m, bool on) {
  if (!on) return;
  const float f = mp == -CUDART_INF_F ? 0.f : attn_ex2(mp - m);
  float4 z[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) z[k] = reinterpret_cast<const float4*>(from)[k];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    o[4 * k] = u32(fmaf(z[k].x, f, f32(o[4 * k])));
    o[4 * k + 1] = u32(fmaf(z[k].y, f, f32(o[4 * k + 1])));
    o[4 * k + 2] = u32(fmaf(z[k].z, f, f32(o[4 * k + 2])));
    o[4 * k + 3] = u32(fmaf(z[k].w, f, f32(o[4 * k + 3])));
  }
}
__device__ __forceinline__ void put_part(float* to, const uint32_t (&o)[32]) {
#pragma unroll
  for (int k = 0; k < 32; k += 4)
    *reinterpret_cast<float4*>(to + k) = make_float4(f32(o[k]), f32(o[k + 1]), f32(o[k + 2]), f32(o[k + 3]));
}

// The infinities and NaNs of V that a row sees, of its unit's partly seen
// slots: added to 32 columns of its O from column c0 on (rare).
template <typename TP, int D>
__device__ __forceinline__ void add_non_finite(const AttnDev& a, int b, int h, int j0, int j1, int c0,
                                            uint32_t (&o)[32]) {
#pragma unroll 1
  for (int j = j0; j < j1; ++j) {
    const int64_t row = cache_row(a.c, b, h, j);
    if (row < 0) continue;
    if (sizeof(TP) == 1) {
      const uint32_t byte = a.c.vs[row];
      const uint8_t* v = reinterpret_cast<const uint8_t*>(a.c.v) + row * D + c0;
#pragma unroll
      for (int x = 0; x < 32; ++x) {
        const float y = unpack_e4m3(v[x]).x * scale_of(byte);
        if (byte == 255u || isinf(y)) o[x] = u32(f32(o[x]) + y);
      }
    } else {
      const uint16_t* v = reinterpret_cast<const uint16_t*>(a.c.v) + row * D + c0;
#pragma unroll
      for (int x = 0; x < 32; ++x)
        if ((v[x] & 0x7F80u) == 0x7F80u) o[x] = u32(f32(o[x]) + f32((uint32_t)v[x] << 16));
    }
  }
}

template <typename TP, int D, bool kAlt>
__global__ void __launch_bounds__(TileShared<TP, D, kAlt>::kThreads, 1) k_attn_tile(const AttnDev a) {
  using S = TileShared<TP, D, kAlt>;
  constexpr int kStages = S::kStages, kRows = kAlt ? 128 : 256;
  constexpr bool kScaled = sizeof(TP) == 1;
  constexpr int kPieces = D / 8;  // of a staged row
  constexpr int kProd = S::kProd, kMine = 128 / kProd;  // producers, rows of a tile of each
  // The half of P whose end starts the second query tile.  Measured (512 tokens
  // over 32K bf16 slots; 4 x 2048 over e4m3): no delay, upper half, lower half 403,
  // 398, 388 and 941, 898, 936 us.  (Exponentials in part on the FMA pipe, by a
  // polynomial, gained nothing when P was one part: 311 us without, 314 and 319
  // with a quarter and three eighths of them there.)
  constexpr int kGoHalf = kScaled ? 1 : 0;
  extern __shared__ __align__(1024) uint8_t sm[];
  attn_begin();
  const uint32_t base = smem_u32(sm);
  if (base & 1023u) {  // the swizzled tiles need 1 KB alignment
    if (threadIdx.x == 0 && a.status) atomicMax(a.status, (int)DROPKV_ERR_CUDA);
    return;
  }
  AttnPlanShared& plan = *reinterpret_cast<AttnPlanShared*>(sm + S::oPlan);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + S::oMisc);
  using Bits = typename std::conditional<kAlt, uint16_t, uint32_t>::type;  // of a producer's slots
  volatile Bits* smask = reinterpret_cast<volatile Bits*>(sm + S::oMask);
  volatile int* sodd = reinterpret_cast<volatile int*>(sm + S::oOdd);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return base + S::oBars + 8 * i; };
  // the outcome is the same for every lane, so the warp stays converged
  auto warp_wait = [&](uint32_t b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait_on(b, parity, a.wait_clocks));
  };
  // Q full / empty; K and V full / empty per stage; per query tile (or, kAlt,
  // S/P buffer): S there, P's upper and lower half there, P V done
  const uint32_t QF = bar(0), QE = bar(1);
  auto KF = [&](int s) { return bar(2 + s); };
  auto KE = [&](int s) { return bar(2 + kStages + s); };
  auto VF = [&](int s) { return bar(2 + 2 * kStages + s); };
  auto VE = [&](int s) { return bar(2 + 3 * kStages + s); };
  constexpr int kB0 = 2 + 4 * kStages;
  auto SF = [&](int u) { return bar(kB0 + u); };
  auto PA = [&](int u) { return bar(kB0 + 2 + u); };
  auto PB = [&](int u) { return bar(kB0 + 4 + u); };
  auto PD = [&](int u) { return bar(kB0 + 6 + u); };
  // units of even / odd number finished by the softmax warps
  auto UE = [&](int p) { return bar(kB0 + 8 + p); };
  // a unit's second query tile begins
  const uint32_t GO = bar(kB0 + 10);
  if (threadIdx.x == 0) {
    mbar_init(GO, 1);
    mbar_init(QF, kProd);
    mbar_init(QE, kAlt ? 1 : 2);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(KF(s), kProd);
      mbar_init(KE(s), kAlt ? 1 : 2);
      mbar_init(VF(s), kProd);
      mbar_init(VE(s), kAlt ? 1 : 2);
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(SF(u), 1);
      mbar_init(PA(u), 4);
      mbar_init(PB(u), 4);
      mbar_init(PD(u), 1);
      mbar_init(UE(u), S::kSoftmax);
      sodd[u] = 0;
    }
    fence_mbar_init();
  }
  if (warp == kTMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  AttnWalk w;
  bool more = attn_plan<kRows, kTTile, S::kThreads>(a, plan, w);
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  if (warp >= kTMmaWarp) {
    // ---------------- MMA issuers ----------------
    // Warp u: S and P V of query tile u, so that no tile's products wait for the
    // other's softmax.  Measured against one warp for both, in turn or as they
    // became ready, when P was one part: 331 against 350 and 377 us for 512 tokens
    // over 32K bf16 slots (an MMA is issued as it executes, 64 clocks, and a barrier seen some 100
    // clocks late).  kAlt: one warp, S a tile ahead of P V.
    const int u = warp - kTMmaWarp;
    constexpr uint32_t IDS = idesc_bf16(128, 128, false, false);  // S = Q K^T
    constexpr uint32_t IDP = idesc_bf16(128, D, false, true);     // O += P V (V MN-major)
    const SDesc qd = sdesc_split(base + u * S::kTileBytes, 16, 1024);
    const SDesc kd = sdesc_split(base + S::oK, 16, 1024);
    const SDesc vd = sdesc_split(base + S::oV, S::kBox, 1024);
    const uint32_t dO = tbase + kTColO + 128u * u;
    uint32_t tiles = 0, units = 0;  // of the range so far
    uint32_t n = 0;                 // P V issued by this warp
    bool ok = true;
    while (more && ok) {
      const Unit x = unit_of<kRows>(a, w);
      const int T = w.t1 - w.t0;
      // a stage is handed back by both warps; a single query tile's does it twice
      const bool twice = !kAlt && x.rows <= 128;
      ok = warp_wait(QF, units & 1);
      ++units;
      tc_fence_after();
      // S, this warp's k-th, of tile j, once the P V that reads the last P from
      // its columns (the buffer's last one) is done
      auto issue_S = [&](int j, uint32_t k) {
        const uint32_t i = tiles + j, s = i % kStages;
        const int f = kAlt ? k & 1 : u;
        if (!warp_wait(KF(s), (i / kStages) & 1)) return false;
        if (kAlt ? k >= 2 && !warp_wait(PD(f), ((k >> 1) - 1) & 1)
                 : k >= 1 && !warp_wait(PD(f), (k - 1) & 1))
          return false;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t klo = kd.lo + s * (S::kTileBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t at = (uint32_t)((kk >> 2) * (S::kBox >> 4) + (kk & 3) * 2);
            mma_ss_w(tbase + 128u * f, qd.lo + at, qd.hi, klo + at, kd.hi, IDS, kk > 0 ? 1u : 0u);
          }
          mma_commit(SF(f));
          mma_commit(KE(s));
          if (twice) mma_commit(KE(s));
          if (j == T - 1) mma_commit(QE);
        }
        __syncwarp();
        return true;
      };
      if (kAlt || 128 * u < x.rows) {
        // The second query tile begins half a tile late: in step, the two would
        // take turns to leave the tensor pipe and the special-function unit idle.
        if (!kAlt && u == 1) ok = ok && warp_wait(GO, (units - 1) & 1);
        ok = ok && issue_S(0, n);
        for (int j = 0; j < T && ok; ++j) {
          if (kAlt && j + 1 < T) ok = issue_S(j + 1, n + 1);
          // O (+)= P V of tile j, as the halves of P come
          const uint32_t i = tiles + j, s = i % kStages;
          const uint32_t vlo = vd.lo + s * (S::kTileBytes >> 4);
          const int f = kAlt ? n & 1 : u;
          ok = ok && warp_wait(VF(s), (i / kStages) & 1);
#pragma unroll
          for (int half = 1; half >= 0; --half) {
            ok = ok && warp_wait(half ? PA(f) : PB(f), (kAlt ? n >> 1 : n) & 1);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)  // both parts of P for each V slice of 16 rows, 2 KB
                mma_ts_w(dO, tbase + 128u * f + 64u * half + 8u * kk, vlo + 128u * (4 * half + (kk >> 1)),
                         vd.hi, IDP, (j % kFold > 0 || half == 0 || kk > 0) ? 1u : 0u);
            }
          }
          if (!ok) break;
          if (lane == 0) {
            mma_commit(PD(f));
            mma_commit(VE(s));
            if (twice) mma_commit(VE(s));
          }
          __syncwarp();
          ++n;
          if (!kAlt && j + 1 < T) ok = issue_S(j + 1, n);
        }
      } else if (lane == 0) {
        mbar_arrive(QE);  // nothing to read; but no unit passes without this warp
      }
      tiles += T;
      more = attn_next<kRows, kTTile>(a, w);
    }
    if (!ok && lane == 0) fail(a);
  } else if (warp >= S::kSoftmax) {
    // ---------------- producers ----------------
    // Warp pw stages the kMine slots from kMine pw on of every tile, and so the
    // query rows; lane i looks up slot i mod kMine.
    const int pw = warp - S::kSoftmax, row0 = pw * kMine;
    const int mine = lane % kMine;
    uint32_t tc_ = 0, units = 0;  // tiles and units so far
    bool ok = true;
    const uint8_t* kp = reinterpret_cast<const uint8_t*>(a.c.k);
    const uint8_t* vp = reinterpret_cast<const uint8_t*>(a.c.v);
    auto arrive = [&](uint32_t b) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
    };
    auto hand_over_q = [&]() {
      if (!(a.withhold && units == 0 && pw == 0)) arrive(QF);
    };
    auto load_q = [&](const Unit& x) {
      // the unit's query rows, zeros behind the last
      constexpr int kPer = 32 / kPieces;  // rows a warp copies at once
      const int c = lane % kPieces;
      for (int q = 0; q < S::kQTiles; ++q) {
#pragma unroll 4
        for (int i = 0; i < kMine / kPer; ++i) {
          const int r = row0 + i * kPer + lane / kPieces, ur = q * 128 + r;
          const bool on = ur < x.rows;
          const AttnRow y = attn_row(a, x.b, w.h, x.rt * kRows + (on ? ur : 0));
          const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(a.q) + y.b * a.qs[0] +
                                     y.hq * a.qs[1] + y.t * a.qs[2] + c * 8;
          copy16(base + q * S::kTileBytes + piece_at(r, c), src, on);
        }
      }
      copy_commit();
    };
    while (more && ok) {
      // at most one unit ahead of the softmax warps: they read sodd at a unit's end
      ok = units < 2 || warp_wait(UE(units & 1), ((units >> 1) - 1) & 1);
      if (!ok) break;
      const Unit x = unit_of<kRows>(a, w);
      const int32_t* table = a.c.table + (size_t)x.b * a.c.max_pages;
      // lane's slot of tile t, and the word of the tile's slots that are there
      auto look = [&](int t) {
        return look_up(a, table, t * kTTile + row0 + mine, t < w.t1 ? x.seen_all : 0);
      };
      auto odd = [&]() { sodd[units & 1] = (int)units + 1; };
      Look nxt = look(w.t0);
      if constexpr (!kScaled) {
        constexpr int kPer = 32 / kPieces;
        const int c = lane % kPieces;
        // non-finite values of partly seen slots of V, as they landed in stage s
        auto clean = [&](int t, uint32_t s) {
          if ((t + 1) * kTTile <= x.seen_min) return;
          bool any = false;
          for (int i = 0; i < kMine / kPer; ++i) {
            const int r = row0 + i * kPer + lane / kPieces;
            if (t * kTTile + r < x.seen_min) continue;
            const uint32_t at = base + S::oV + s * S::kTileBytes + piece_at(r, c);
            uint4 v = lds16(at);
            if (non_finite(v.x) || non_finite(v.y) || non_finite(v.z) || non_finite(v.w)) {
              any = true;
              sts16(at, make_uint4(without_non_finite(v.x), without_non_finite(v.y),
                                   without_non_finite(v.z), without_non_finite(v.w)));
            }
          }
          if (any) odd();
        };
        for (int t = w.t0; t < w.t1 && ok; ++t) {
          const int row = pool_row(a, w.h, nxt);
          nxt = look(t + 1);
          const uint32_t s = tc_ % kStages, ph = (tc_ / kStages) & 1;
          const uint32_t word = __ballot_sync(0xffffffffu, row >= 0);
          // K of this tile, then the last tile's V is handed over; V, then K
          ok = warp_wait(KE(s), ph ^ 1);
          if (!ok) break;
          if (lane == 0) smask[(tc_ & 7) * kProd + pw] = (Bits)word;
          auto issue = [&](const uint8_t* pool, uint32_t dst) {
#pragma unroll 4
            for (int i = 0; i < kMine / kPer; ++i) {
              const int at = __shfl_sync(0xffffffffu, row, i * kPer + lane / kPieces);
              copy16(dst + piece_at(row0 + i * kPer + lane / kPieces, c),
                     pool + (at < 0 ? 0 : (size_t)at * (D * 2) + c * 16), at >= 0);
            }
            copy_commit();
          };
          issue(kp, base + S::oK + s * S::kTileBytes);
          if (t == w.t0) {
            // the last unit's rows are read out: this one's
            ok = warp_wait(QE, (units & 1) ^ 1);
            if (!ok) break;
            load_q(x);
            copy_wait<0>();
            hand_over_q();
            arrive(KF(s));
          } else {
            copy_wait<1>();
            const uint32_t sl = (tc_ - 1) % kStages;
            clean(t - 1, sl);
            arrive(VF(sl));
          }
          ok = warp_wait(VE(s), ph ^ 1);
          if (!ok) break;
          issue(vp, base + S::oV + s * S::kTileBytes);
          if (t != w.t0) {
            copy_wait<1>();
            arrive(KF(s));
          }
          ++tc_;
        }
        copy_wait<0>();
        if (ok) {
          const uint32_t sl = (tc_ - 1) % kStages;
          clean(w.t1 - 1, sl);
          arrive(VF(sl));
        }
      } else {
        // a row of D bytes is D / 16 loads; a warp's pass covers kPer rows
        constexpr int kIn = D / 16, kPer = 32 / kIn, kPass = kMine / kPer;
        const int c = lane % kIn;
        // Jobs: K and V of a tile in turn, by the same code (one copy of it: see
        // the softmax's loops).  A ring holds the next kRing jobs' bytes as the
        // asynchronous copies land; a lane widens what it has copied.
        constexpr int kRing = S::kRing, kAhead = kRing / 2;  // jobs, tiles
        const uint32_t ring = base + S::oRaw + pw * (kMine * D) + lane * 16;
        auto issue = [&](int job, int row) {
          if (job < 2 * w.t1) {
            const uint8_t* pool = (job & 1 ? vp : kp) + c * 16;
            const uint32_t dst = ring + (uint32_t)(job % kRing) * (128 * D);
            int at[kPass];
#pragma unroll
            for (int i = 0; i < kPass; ++i)
              at[i] = __shfl_sync(0xffffffffu, row, i * kPer + lane / kIn);
#pragma unroll
            for (int i = 0; i < kPass; ++i)
              copy16(dst + i * 512, pool + (size_t)max(at[i], 0) * D, at[i] >= 0);
          }
          copy_commit();
        };
        // widened into a stage
        auto put = [&](const uint32_t (&y)[8], int i, uint32_t dst) {
          // lanes of the second box store their odd piece first: eight lanes of a
          // row then hit eight different 16-byte bank groups
          const int r = row0 + i * kPer + lane / kIn;
          const bool swap = D == 128 && c >= kIn / 2;
          const uint4 p0 = make_uint4(y[0], y[1], y[2], y[3]), p1 = make_uint4(y[4], y[5], y[6], y[7]);
          sts16(dst + piece_at(r, 2 * c + swap), swap ? p1 : p0);
          sts16(dst + piece_at(r, 2 * c + !swap), swap ? p0 : p1);
        };
        auto widen = [&](const uint4& v, uint32_t f, uint32_t (&y)[8]) {
          const uint32_t in[4] = {v.x, v.y, v.z, v.w};
          const uint32_t f2 = __byte_perm(f, 0, 0x1010);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            y[2 * k] = widen_e4m3x2<kBytes01>(in[k], f2);
            y[2 * k + 1] = widen_e4m3x2<kBytes23>(in[k], f2);
          }
        };
        auto store = [&](uint32_t src, uint32_t byte, uint32_t dst, int part) {
          constexpr int kBatch = kPass < 4 ? kPass : 4;
          const uint32_t own = widen_factors(byte);
          // some passes' loads before their conversions: a warp alone on its
          // scheduler has nobody else to hide their latency
#pragma unroll 1
          for (int i0 = 0; i0 < kPass; i0 += kBatch) {
            uint4 in[kBatch];
            uint32_t f[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              in[i] = lds16(src + (i0 + i) * 512);
              f[i] = __shfl_sync(0xffffffffu, own, (i0 + i) * kPer + lane / kIn);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              uint32_t y[8];
              widen(in[i], f[i], y);
              put(y, i0 + i, dst);
            }
          }
          if (part >= kTTile && __all_sync(0xffffffffu, own >> 16 == 0x3F80u)) return;
          // large scales, or partly seen slots (from row `part` of the tile on),
          // whose values that are not finite are staged as 0
          bool any = false;
#pragma unroll 1
          for (int i = 0; i < kPass; ++i) {
            const int r = row0 + i * kPer + lane / kIn;
            const uint32_t f = __byte_perm(__shfl_sync(0xffffffffu, own, r - row0), 0, 0x3232);
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
              const uint32_t at = dst + piece_at(r, 2 * c + e);
              const uint4 v = lds16(at);
              uint32_t y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                y[k] = mul_bf16x2(y[k], f);
                any = any || (r >= part && non_finite(y[k]));
                if (r >= part) y[k] = without_non_finite(y[k]);
              }
              sts16(at, make_uint4(y[0], y[1], y[2], y[3]));
            }
          }
          if (any) odd();
        };
        uint32_t words[kAhead + 1], bk, bv, nk = 0, nv = 0;  // the lane's scale bytes, the next tile's
        int row = 0;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          row = pool_row(a, w.h, nxt);
          nxt = look(w.t0 + i + 1);
          words[i] = __ballot_sync(0xffffffffu, row >= 0);
          issue(2 * (w.t0 + i), row);
          issue(2 * (w.t0 + i) + 1, row);
          if (i == 0) {
            bk = ldg1(a.c.ks + max(row, 0), row >= 0);
            bv = ldg1(a.c.vs + max(row, 0), row >= 0);
          }
        }
#pragma unroll 1
        for (int job = 2 * w.t0; job < 2 * w.t1; ++job) {
          const int t = job >> 1, v = job & 1;
          const uint32_t s = tc_ % kStages, ph = (tc_ / kStages) & 1;
          if (!v) {
            int r1 = row;  // row of the lane's slot in tile t + 1
            row = pool_row(a, w.h, nxt);  // and in tile t + kAhead
            nxt = look(t + kAhead + 1);
            words[kAhead] = __ballot_sync(0xffffffffu, row >= 0);
            if (kAhead == 1) r1 = row;
            nk = ldg1(a.c.ks + max(r1, 0), r1 >= 0);
            nv = ldg1(a.c.vs + max(r1, 0), r1 >= 0);
          }
          ok = warp_wait(v ? VE(s) : KE(s), ph ^ 1);
          if (!ok) break;
          if (!v && lane == 0) smask[(tc_ & 7) * kProd + pw] = (Bits)words[0];
          copy_wait<kRing - 1>();
          store(ring + (uint32_t)(job % kRing) * (128 * D), v ? bv : bk,
                base + (v ? S::oV : S::oK) + s * S::kTileBytes,
                v ? x.seen_min - t * kTTile : kTTile);
          arrive(v ? VF(s) : KF(s));
          issue(job + kRing, row);
          if (job == 2 * w.t0) {
            ok = warp_wait(QE, (units & 1) ^ 1);
            if (!ok) break;
            load_q(x);
            copy_wait<0>();
            hand_over_q();
          }
          if (v) {
            ++tc_;
            bk = nk;
            bv = nv;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) words[i] = words[i + 1];
          }
        }
      }
      if (!ok) break;
      ++units;
      more = attn_next<kRows, kTTile>(a, w);
    }
    if (!ok && lane == 0) fail(a);
    copy_wait<0>();
  } else {
    // ---------------- softmax ----------------
    const int u = warp >> 2, ql = warp & 3;
    const int crow = 128 * u + ql * 32 + lane;       // row of the unit
    const uint32_t lane_off = (uint32_t)(ql * 32) << 16;
    const uint32_t tO = tbase + kTColO + 128u * u + lane_off;
    const float c = a.c_log2;
    const uint64_t c2 = pk2(c, c), above2 = pk2(kAboveOne, kAboveOne);
    uint32_t n = 0;              // slot tiles of this query tile so far
    uint32_t tiles = 0, units = 0;
    bool live = true;            // no wait has run out
    auto alive = [&](bool got) {
      if (!got) {
        if (live && lane == 0) fail(a);
        live = false;
      }
    };
    while (more) {
      const Unit x = unit_of<kRows>(a, w);
      const int T = w.t1 - w.t0;
      const bool warp_rows = 128 * u + ql * 32 < x.rows;
      const bool has = crow < x.rows;
      const int r = x.rt * kRows + crow;
      const int seen = has ? attn_seen(a, x.L, x.n, r) : 0;
      float m = -CUDART_INF_F, l = 0.f;
      const bool mine = 128 * u < x.rows;  // this query tile exists
      // Where O goes on the way: the unit's partial, or for a whole unit that of the CTA's
      // last one, which is written behind it.  mp: the reference that O has there.
      auto part_row = [&]() {
        const int slot = attn_slot(w);
        return a.part + ((size_t)(slot < 0 ? 2 * (int)blockIdx.x + 1 : slot) * kRows + crow) * a.pstride;
      };
      float mp = -CUDART_INF_F;
      for (int j = 0; j < T && live && mine; ++j) {
        const int f = kAlt ? n & 1 : u;  // S/P buffer
        const uint32_t tS = tbase + 128u * f + lane_off;
        if (warp_rows && j > 0 && j % kFold == 0) {
          // O, complete up to the last tile, to its row in the workspace
          if (!warp_wait(PD(kAlt ? f ^ 1 : u), (kAlt ? (n - 1) >> 1 : n - 1) & 1)) {
            alive(false);
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < D / 32; ++k) {
            uint32_t o[32];
            tmem_ld32(tO + 32u * k, o);
            if (j > kFold) add_part(o, part_row() + 32 * k, mp, m, has);
            if (has) put_part(part_row() + 32 * k, o);
            __syncwarp();
          }
          mp = m;
        }
        if (has && j >= kFold && ((j + 1) % kFold == 0 || j + 1 == T)) {
          // what the next tile's fold, or the unit's end, reads: behind the copies in
          // flight its way from memory takes microseconds
#pragma unroll
          for (int k = 0; k < D; k += 32) prefetch_l2(part_row() + k);
        }
        alive(warp_wait(SF(f), (kAlt ? n >> 1 : n) & 1));
        if (!live) break;
        if (warp_rows) {
          tc_fence_after();
          const int tok0 = (w.t0 + j) * kTTile, lim = seen - tok0;
          const uint4 there = lds16(base + S::oMask + ((tiles + j) & 7) * 16);
          if (tok0 + kTTile > x.seen_min || (there.x & there.y & there.z & there.w) != ~0u) {
            // hidden slots: -inf over their logits
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
              uint32_t o[16];
              tmem_ld16(tS + 16u * k, o);
              const uint32_t two = k < 2 ? there.x : k < 4 ? there.y : k < 6 ? there.z : there.w;
              const uint32_t word = two >> (16 * (k & 1));
#pragma unroll
              for (int y = 0; y < 16; ++y)
                if (16 * k + y >= lim || !((word >> y) & 1)) o[y] = 0xFF800000u;
              tmem_st16(tS + 16u * k, o);
            }
            tmem_st_wait();
          }
          // Rolled loops over the halves of the row: straight-line code for all
          // of it (with the producers' beside it) ran out of the instruction
          // caches, which cost more than the second TMEM read of a half.
          uint32_t sr[64];
          float ya = -CUDART_INF_F, yb = -CUDART_INF_F;
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            tmem_ld64(tS + 64u * half, sr);
#pragma unroll
            for (int k = 0; k < 64; k += 4) {
              ya = fmax3(ya, f32(sr[k]), f32(sr[k + 1]));
              yb = fmax3(yb, f32(sr[k + 2]), f32(sr[k + 3]));
            }
          }
          const float mt = fmaxf(ya, yb) * c;  // c > 0
          float fac = 1.f;
          if (mt > m + 8.f) {
            fac = m == -CUDART_INF_F ? 0.f : attn_ex2(m - mt);
            m = mt;
            l *= fac;
          }
          // rows whose reference moved: O, complete up to the last tile, by fac
          if (__any_sync(0xffffffffu, fac != 1.f) && j >= 1) {
            if (!warp_wait(PD(kAlt ? f ^ 1 : u), (kAlt ? (n - 1) >> 1 : n - 1) & 1)) {
              alive(false);
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < D / 16; ++k) {
              uint32_t o[16];
              tmem_ld16(tO + 16u * k, o);
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = u32(f32(o[y]) * fac);
              tmem_st16(tO + 16u * k, o);
            }
            tmem_st_wait();
          }
          const float mu = m == -CUDART_INF_F ? 0.f : m;
          const uint64_t nmu2 = pk2(-mu, -mu);
          uint64_t l2 = 0ull;  // of this tile: a chain over all slots would lose bits
#pragma unroll 1
          for (int half = 1; half >= 0; --half) {
            if (half == 0) tmem_ld64(tS, sr);  // the upper half is still there
#pragma unroll
            for (int z = 0; z < 4; ++z) {  // 16 slots at a time: there are no registers for more
              uint32_t pw[16];  // the upper parts, the lower parts
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int i = 16 * z + 2 * k;
                float d0, d1;
                upk2(ffma2(pk2(f32(sr[i]), f32(sr[i + 1])), c2, nmu2), d0, d1);
                const float e0 = attn_ex2(d0), e1 = attn_ex2(d1);
                const uint64_t e2 = pk2(e0, e1);
                l2 = fadd2(l2, e2);
                pw[k] = upper_bf16x2(e0, e1);
                upk2(ffma2(e2, above2, pk2(minus_upper(e0), minus_upper(e1))), d0, d1);
                pw[8 + k] = pack_bf16(d0, d1);
              }
              tmem_st16(tS + 64u * half + 16u * z, pw);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(half ? PA(f) : PB(f));
            if (!kAlt && half == kGoHalf && j == 0 && threadIdx.x == 0) mbar_arrive(GO);
          }
          float la, lb;
          upk2(l2, la, lb);
          l += la + lb;
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(PA(f));
            mbar_arrive(PB(f));
          }
        }
        ++n;
      }
      // ---- the unit's rows: O / l, or the cut unit's partial ----
      const AttnRow at = attn_row(a, x.b, w.h, has ? r : x.rt * kRows);
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + at.b * a.os[0] +
                           at.hq * a.os[1] + at.t * a.os[2];
      const int j0 = max(w.t0 * kTTile, x.seen_min), j1 = min(w.t1 * kTTile, seen);
      const int slot = attn_slot(w);
      float* part = part_row();
      auto finish = [&](uint32_t (&o)[32], int c0, bool fix, float inv) {
        if (T > kFold) add_part(o, part + c0, mp, m, has);
        if (fix) add_non_finite<TP, D>(a, x.b, w.h, j0, j1, c0, o);
        if (!has) return;
        if (slot < 0) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[e] = pack_bf16(f32(o[k + 2 * e]) * inv, f32(o[k + 2 * e + 1]) * inv);
            *reinterpret_cast<uint4*>(out + c0 + k) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else {
          put_part(part + c0, o);
        }
      };
      auto put_stats = [&](float mm, float ll) {
        if (!has) return;
        if (slot < 0)
          attn_put_lse(a, at, mm, ll);
        else
          *reinterpret_cast<float2*>(part + a.pstride - 4) = make_float2(mm, ll);
      };
      if (mine && live)
        alive(warp_wait(PD(kAlt ? (n - 1) & 1 : u), (kAlt ? (n - 1) >> 1 : n - 1) & 1));
      if (mine && live && warp_rows) {
        tc_fence_after();
        const bool fix = sodd[units & 1] == (int)units + 1;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          uint32_t o[32];
          tmem_ld32(tO + 32u * k, o);
          finish(o, 32 * k, fix, inv);
        }
        put_stats(m, l);
      }
      tc_fence_before();
      // a warpgroup without rows does not run ahead: its arrivals belong to units
      if (!kAlt && x.rows <= 128) named_barrier_sync(1, 256);
      __syncwarp();
      if (lane == 0) mbar_arrive(UE(units & 1));
      tiles += T;
      ++units;
      more = attn_next<kRows, kTTile>(a, w);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kTMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <typename TP, int D, bool kAlt>
cudaError_t launch_tile(const AttnDev& a, cudaStream_t st) {
  const auto kern = k_attn_tile<TP, D, kAlt>;
  constexpr int smem = TileShared<TP, D, kAlt>::kBytes;
  static_assert(smem <= 232448, "shared memory of a CTA");
  cudaError_t e = allow_smem<k_attn_tile<TP, D, kAlt>>(smem);
  if (e != cudaSuccess) return e;
  return launch_ex(kern, dim3(kTCtas), dim3(TileShared<TP, D, kAlt>::kThreads), smem, st, true, 1, a);
}

template <bool kAlt>
cudaError_t launch_tiles(const AttnDev& a, int page_dtype, cudaStream_t st) {
  if (page_dtype == DROPKV_BF16)
    return a.c.d == 128 ? launch_tile<__nv_bfloat16, 128, kAlt>(a, st)
                        : launch_tile<__nv_bfloat16, 64, kAlt>(a, st);
  return a.c.d == 128 ? launch_tile<E4M3, 128, kAlt>(a, st) : launch_tile<E4M3, 64, kAlt>(a, st);
}

}  // namespace

AttnGrid attn_grid_tile(bool alt) { return {kTCtas, alt ? 128 : 256, kTTile}; }

cudaError_t launch_attn_tile(const AttnDev& a, int page_dtype, bool alt, cudaStream_t st) {
  return alt ? launch_tiles<true>(a, page_dtype, st) : launch_tiles<false>(a, page_dtype, st);
}

}  // namespace dropkv
