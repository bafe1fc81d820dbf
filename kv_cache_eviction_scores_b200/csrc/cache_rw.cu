// cache_rw.cu -- rows to pages and back: dropkv_cache_write gathers dense K/V
// rows (all, or the kept positions of a list) into consecutive slots, as they
// are or quantised to e4m3; dropkv_cache_read takes slots back to dense rows.
//
// Mathematics.  E4M3: byte = e + 127 with e the least integer >= -127 such
// that max |x| <= 448 2^e, values RNE(x 2^-e); reading multiplies by 2^e.
//
// What bounds it: memory traffic, each row once in and once out, once the
// instructions are few enough.  One group of lanes owns a row (8 values a lane,
// 16-byte loads and stores; the row's maximum by shuffles inside the group) and
// moves K and V of that row together; kRowsInFlight rows per group keep their
// loads in flight, as they are stored; the list, page table and slot arithmetic
// are done once per row, by one thread.  Measured (one call after the other): 0.74 GB
// of bf16 rows to e4m3 in 141 us (5.3 TB/s, 81 % of the measured copy; 188 us with four
// rows placed by every lane and fp32 arithmetic; 143 to 150 as calls over changing
// inputs), 0.2 GB of e4m3 back to bf16 in 37 us (5.4; 38).  Rows that 16-byte pieces do
// not fit (d = 33) move value by value, one row in flight: 32K x 8 bf16 rows 100 us,
// their bytes 11.
#include "cache.cuh"

namespace dropkv {

namespace {

constexpr int kThreads = 256;

struct RowsDev {
  void* k;
  void* v;
  int64_t ks[3], vs[3];
  int32_t n, m;
  const int32_t* rows;
  const int32_t* start;
  const int32_t* counts;
  int32_t* status;
  int32_t nblk;    // blocks per (b, h)
  int32_t lanes;   // lanes per row, a power of two
};

// The eight values of a row that a lane owns: values 8 lane + j in one piece
// (kVec), or values lane + 32 j.
template <bool kVec>
__device__ __forceinline__ int value_at(int lane, int j) {
  return kVec ? lane * 8 + j : lane + 32 * j;
}

template <typename T>
struct Eight {};  // eight values of a row as they are stored
template <>
struct Eight<__nv_bfloat16> {
  uint4 w;
};
template <>
struct Eight<float> {
  float4 a, b;
};
template <>
struct Eight<E4M3> {
  uint2 w;
};

__device__ __forceinline__ void widen(const Eight<__nv_bfloat16>& s, float (&x)[8]) {
  const uint32_t w[4] = {s.w.x, s.w.y, s.w.z, s.w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void widen(const Eight<float>& s, float (&x)[8]) {
  x[0] = s.a.x; x[1] = s.a.y; x[2] = s.a.z; x[3] = s.a.w;
  x[4] = s.b.x; x[5] = s.b.y; x[6] = s.b.z; x[7] = s.b.w;
}
__device__ __forceinline__ void widen(const Eight<E4M3>& s, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_e4m3(((i < 2 ? s.w.x : s.w.y) >> (16 * (i & 1))) & 0xFFFFu);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void narrow(Eight<__nv_bfloat16>& s, const float (&x)[8]) {
  s.w = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                   pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void narrow(Eight<float>& s, const float (&x)[8]) {
  s.a = make_float4(x[0], x[1], x[2], x[3]);
  s.b = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void narrow(Eight<E4M3>& s, const float (&x)[8]) {
  s.w = make_uint2(pack_e4m3(x[0], x[1]) | pack_e4m3(x[2], x[3]) << 16,
                   pack_e4m3(x[4], x[5]) | pack_e4m3(x[6], x[7]) << 16);
}
__device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float one(const float* p) { return *p; }
__device__ __forceinline__ float one(const E4M3* p) { return unpack_e4m3(p->bits).x; }
__device__ __forceinline__ void put_one(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put_one(float* p, float x) { *p = x; }
__device__ __forceinline__ void put_one(E4M3* p, float x) { p->bits = (uint8_t)pack_e4m3(x, 0.f); }

// A lane's eight values of a row: as they are stored (kVec), or widened one by
// one; values past d are 0.
template <bool kVec, typename T>
struct Piece {};
template <typename T>
struct Piece<true, T> {
  Eight<T> s;
  __device__ __forceinline__ void load(const T* p, int lane, int d) {
    s = Eight<T>{};
    if (lane * 8 < d) s = *reinterpret_cast<const Eight<T>*>(p + lane * 8);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const { widen(s, x); }
};
template <typename T>
struct Piece<false, T> {
  float v[8];
  __device__ __forceinline__ void load(const T* p, int lane, int d) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = lane + 32 * j < d ? one(p + lane + 32 * j) : 0.f;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = v[j];
  }
};
template <bool kVec, typename T>
__device__ __forceinline__ void store8(T* p, int lane, int d, const float (&x)[8]) {
  if (kVec) {
    if (lane * 8 < d) {
      Eight<T> s;
      narrow(s, x);
      *reinterpret_cast<Eight<T>*>(p + lane * 8) = s;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (lane + 32 * j < d) put_one(p + lane + 32 * j, x[j]);
  }
}

// Scales the row that the `lanes` lanes of a group hold, for e4m3 pages, and
// returns its scale byte.  Every lane of the warp calls it.
__device__ __forceinline__ uint32_t to_scaled(float (&x)[8], int lanes) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
  for (int o = lanes >> 1; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const uint32_t byte = scale_byte(top);
  const float f = inv_scale_of(byte);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] *= f;
  return byte;
}

// The same for bf16 values of K and V on their way to e4m3, packed throughout: the
// kernel issues instructions most of its time, and this takes two thirds of them.
// |x| of bf16 orders like its bits, so one chain of shuffles finds both rows'
// maxima as 16-bit halves.  The product with a power of two is exact in bf16, too,
// where it matters: what falls below its range is far under e4m3's smallest step.
__device__ __forceinline__ uint32_t abs_max(const uint4& w) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  const uint32_t m = __vmaxu2(__vmaxu2(w.x & kAbs, w.y & kAbs), __vmaxu2(w.z & kAbs, w.w & kAbs));
  return max(m & 0xFFFFu, m >> 16);
}
__device__ __forceinline__ uint2 scaled_e4m3(const uint4& w, uint32_t byte) {
  const uint32_t f = (byte == 255u ? 0x7FC0u : (254u - byte) << 7) * 0x10001u;
  const uint32_t y[4] = {mul_bf16x2(w.x, f), mul_bf16x2(w.y, f), mul_bf16x2(w.z, f), mul_bf16x2(w.w, f)};
  uint32_t z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    z[i] = pack_e4m3(__uint_as_float(y[i] << 16), __uint_as_float(y[i] & 0xFFFF0000u));
  return make_uint2(__byte_perm(z[0], z[1], 0x5410), __byte_perm(z[2], z[3], 0x5410));
}

// What a group of lanes moves in one go: its dense row and its row of the pools.
struct Move {
  int64_t held;   // row of the pools
  int32_t dense;  // row of the dense tensors, < 0: nothing
};

// Item i of (b, h), whose list entry (i without a list) is `at`.  kWrite: dense row
// at, slot start + i; else dense row i, slot start + at.
template <bool kWrite>
__device__ __forceinline__ Move find(const CacheDev& c, const RowsDev& r, int b, int h, int i,
                                     int at, int cnt, int base) {
  Move mv = {-1, -1};
  if (i >= cnt || (r.rows && at == -1)) return mv;
  const int64_t slot = (int64_t)base + (kWrite ? i : at);
  const int dense = kWrite ? at : i;
  bool bad = at < 0 || dense >= r.n || slot < 0 || slot >= c.cap;
  if (!bad) {
    mv.held = cache_row(c, b, h, (int)slot);
    bad = mv.held < 0;
  }
  if (bad) {
    raise_arg(r.status);
    return mv;
  }
  mv.dense = dense;
  return mv;
}

template <bool kFirst, typename A, typename B>
struct Pick {
  using type = A;
};
template <typename A, typename B>
struct Pick<false, A, B> {
  using type = B;
};

// Reads to bf16 run with five blocks an SM (a 32K e4m3 cache 38.7 us, 40.6 with
// the four that their registers would give); writes lose by it (165 against 141).
template <bool kWrite, bool kVec, typename TD, typename TP, int kRowsInFlight>
__global__ void __launch_bounds__(kThreads, !kWrite && sizeof(TD) == 2 ? 5 : 1) k_cache_rows(const CacheDev c, const RowsDev r) {
  const int bh = blockIdx.x / r.nblk, blk = blockIdx.x - bh * r.nblk;
  const int b = bh / c.Hkv, h = bh - b * c.Hkv;
  const int lane = threadIdx.x & (r.lanes - 1);
  const int per = kThreads / r.lanes;
  const int grp = threadIdx.x / r.lanes;
  // the first list entry is requested together with the count and the start
  const int first = blk * per * kRowsInFlight;
  auto entry = [&](int i) {
    return r.rows && i < r.m ? __ldg(r.rows + ((size_t)b * c.Hkv + h) * r.m + i) : i;
  };
  int at = entry(first + (int)threadIdx.x);
  int cnt = r.counts ? __ldg(r.counts + b) : r.m;
  if (cnt < 0 || cnt > r.m) {
    if (threadIdx.x == 0) raise_arg(r.status);
    cnt = min(max(cnt, 0), r.m);
  }
  const int base = r.start ? __ldg(r.start + b) : 0;
  constexpr bool kScaled = sizeof(TP) == 1;
  if (first >= cnt) return;  // the whole block

  TD* const dk = reinterpret_cast<TD*>(r.k) + b * r.ks[0] + h * r.ks[1];
  TD* const dv = reinterpret_cast<TD*>(r.v) + b * r.vs[0] + h * r.vs[1];
  TP* const pk = reinterpret_cast<TP*>(c.k);
  TP* const pv = reinterpret_cast<TP*>(c.v);
  // each of the block's rows is placed by one thread; done by every lane that
  // moves a row, this was half of all instructions
  __shared__ Move place[kThreads * kRowsInFlight];
  for (int i = threadIdx.x; i < per * kRowsInFlight; i += kThreads) {
    if (i >= kThreads) at = entry(first + i);
    place[i] = find<kWrite>(c, r, b, h, first + i, at, cnt, base);
  }
  __syncthreads();
  Move mv[kRowsInFlight];
#pragma unroll
  for (int u = 0; u < kRowsInFlight; ++u) mv[u] = place[u * per + grp];
  using From = typename Pick<kWrite, TD, TP>::type;
  Piece<kVec, From> xk[kRowsInFlight], xv[kRowsInFlight];
  uint32_t bk[kRowsInFlight], bv[kRowsInFlight];
#pragma unroll
  for (int u = 0; u < kRowsInFlight; ++u) {
    const bool on = mv[u].dense >= 0;  // a row of nothing loads nothing
    const int dd = on ? c.d : 0;
    if constexpr (kWrite) {
      const int64_t row = on ? mv[u].dense : 0;
      xk[u].load(dk + row * r.ks[2], lane, dd);
      xv[u].load(dv + row * r.vs[2], lane, dd);
    } else {
      const int64_t row = on ? mv[u].held : 0;
      xk[u].load(pk + row * c.d, lane, dd);
      xv[u].load(pv + row * c.d, lane, dd);
      if (kScaled && on) {
        bk[u] = __ldg(c.ks + row);
        bv[u] = __ldg(c.vs + row);
      }
    }
  }
  if constexpr (kWrite && kVec && kScaled && sizeof(TD) == 2) {
    uint32_t top[kRowsInFlight];
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u) top[u] = abs_max(xk[u].s.w) | abs_max(xv[u].s.w) << 16;
    for (int o = r.lanes >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int u = 0; u < kRowsInFlight; ++u)
        top[u] = __vmaxu2(top[u], __shfl_xor_sync(0xffffffffu, top[u], o));
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u) {
      if (mv[u].dense < 0) continue;
      const uint32_t bk = scale_byte(top[u] << 16), bv = scale_byte(top[u] & 0xFFFF0000u);
      if (lane * 8 < c.d) {
        const int64_t at = mv[u].held * c.d + lane * 8;
        *reinterpret_cast<uint2*>(pk + at) = scaled_e4m3(xk[u].s.w, bk);
        *reinterpret_cast<uint2*>(pv + at) = scaled_e4m3(xv[u].s.w, bv);
      }
      if (lane == 0) {
        c.ks[mv[u].held] = (uint8_t)bk;
        c.vs[mv[u].held] = (uint8_t)bv;
      }
    }
  } else {
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u) {
      float yk[8], yv[8];
      xk[u].get(yk);
      xv[u].get(yv);
      if (kWrite && kScaled) {  // every lane of the warp
        bk[u] = to_scaled(yk, r.lanes);
        bv[u] = to_scaled(yv, r.lanes);
      }
      if (mv[u].dense < 0) continue;
      if constexpr (kWrite) {
        store8<kVec>(pk + mv[u].held * c.d, lane, c.d, yk);
        store8<kVec>(pv + mv[u].held * c.d, lane, c.d, yv);
        if (kScaled && lane == 0) {
          c.ks[mv[u].held] = (uint8_t)bk[u];
          c.vs[mv[u].held] = (uint8_t)bv[u];
        }
      } else {
        if (kScaled) {
          const float fk = scale_of(bk[u]), fv = scale_of(bv[u]);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            yk[j] *= fk;
            yv[j] *= fv;
          }
        }
        store8<kVec>(dk + mv[u].dense * r.ks[2], lane, c.d, yk);
        store8<kVec>(dv + mv[u].dense * r.vs[2], lane, c.d, yv);
      }
    }
  }
}

template <bool kWrite, bool kVec, typename TD, typename TP>
cudaError_t launch_rows(const CacheDev& c, RowsDev r, cudaStream_t st) {
  constexpr int kFly = kVec ? 4 : 1;
  if (kVec) {
    r.lanes = 1;
    while (r.lanes * 8 < c.d) r.lanes *= 2;
  } else {
    r.lanes = 32;
  }
  const int per = kThreads / r.lanes * kFly;
  r.nblk = (r.m + per - 1) / per;
  const int64_t blocks = (int64_t)c.B * c.Hkv * r.nblk;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  k_cache_rows<kWrite, kVec, TD, TP, kFly><<<(unsigned)blocks, kThreads, 0, st>>>(c, r);
  return cudaGetLastError();
}

template <bool kWrite, bool kVec, typename TD>
cudaError_t launch_pages(int dtype, const CacheDev& c, const RowsDev& r, cudaStream_t st) {
  if (dtype == DROPKV_BF16) return launch_rows<kWrite, kVec, TD, __nv_bfloat16>(c, r, st);
  if (dtype == DROPKV_F32) return launch_rows<kWrite, kVec, TD, float>(c, r, st);
  return launch_rows<kWrite, kVec, TD, E4M3>(c, r, st);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <bool kWrite>
dropkv_status run_rows(const dropkv_cache* cp, const dropkv_cache_rows* rp, int32_t* status_dev,
                       void* stream) {
  dropkv_status s = check_cache(cp, true);
  if (s != DROPKV_OK) return s;
  if (!rp) return DROPKV_ERR_ARG;
  const dropkv_cache& c = *cp;
  const dropkv_cache_rows& r = *rp;
  if (!r.k || !r.v || r.n < 1 || r.m < 1 || r.reserved != 0) return DROPKV_ERR_ARG;
  if (r.dtype != DROPKV_BF16 && r.dtype != DROPKV_F32) return DROPKV_ERR_ARG;
  if ((!r.rows || !kWrite) && r.m > r.n) return DROPKV_ERR_ARG;
  // the kernel counts a block's items in 32 bits past the last one (slots end there, too)
  if (r.m > 0x7FFF0000) return DROPKV_ERR_ARG;
  const int esz = r.dtype == DROPKV_BF16 ? 2 : 4;
  if (((uintptr_t)r.k | (uintptr_t)r.v) % esz) return DROPKV_ERR_ARG;
  if (((uintptr_t)r.rows | (uintptr_t)r.start | (uintptr_t)r.counts | (uintptr_t)status_dev) & 3u)
    return DROPKV_ERR_ARG;
  for (int i = 0; i < 3; ++i)
    if (r.k_stride[i] < 0 || r.v_stride[i] < 0) return DROPKV_ERR_ARG;
  s = device_ok();
  if (s != DROPKV_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (status_dev)
    if (cudaError_t e = cudaMemsetAsync(status_dev, 0, sizeof(int32_t), st)) return cuda_fail(e);
  RowsDev d = {};
  d.k = r.k;
  d.v = r.v;
  // 16-byte pieces need whole pieces per row, and dense rows on 16-byte borders
  bool vec = c.d % 8 == 0 && aligned16(r.k) && aligned16(r.v);
  for (int i = 0; i < 3; ++i) {
    d.ks[i] = r.k_stride[i];
    d.vs[i] = r.v_stride[i];
    vec = vec && r.k_stride[i] * esz % 16 == 0 && r.v_stride[i] * esz % 16 == 0;
  }
  d.n = r.n;
  d.m = r.m;
  d.rows = r.rows;
  d.start = r.start;
  d.counts = r.counts;
  d.status = status_dev;
  const CacheDev cd = cache_dev(c);
  cudaError_t e;
  if (r.dtype == DROPKV_BF16)
    e = vec ? launch_pages<kWrite, true, __nv_bfloat16>(c.dtype, cd, d, st)
            : launch_pages<kWrite, false, __nv_bfloat16>(c.dtype, cd, d, st);
  else
    e = vec ? launch_pages<kWrite, true, float>(c.dtype, cd, d, st)
            : launch_pages<kWrite, false, float>(c.dtype, cd, d, st);
  return e == cudaSuccess ? DROPKV_OK : cuda_fail(e);
}

}  // namespace

dropkv_status check_cache(const dropkv_cache* cp, bool pointers) {
  if (!cp) return DROPKV_ERR_ARG;
  const dropkv_cache& c = *cp;
  if (c.B < 1 || c.Hkv < 1 || c.d < 1 || c.d > 256 || c.n_pages < 1) return DROPKV_ERR_ARG;
  if (c.page_size < 1 || c.page_size > 1024 || c.max_pages < 1 || c.reserved != 0)
    return DROPKV_ERR_ARG;
  if (c.dtype != DROPKV_BF16 && c.dtype != DROPKV_F32 && c.dtype != DROPKV_E4M3)
    return DROPKV_ERR_ARG;
  // slots are 32-bit; rows of the pools and bytes are 64-bit
  if ((int64_t)c.max_pages * c.page_size > 0x7FFF0000) return DROPKV_ERR_ARG;
  if ((double)c.n_pages * c.Hkv * c.page_size * c.d > 4.0e18) return DROPKV_ERR_ARG;
  if ((double)c.B * c.Hkv > 1.0e9) return DROPKV_ERR_ARG;
  if (!pointers) return DROPKV_OK;
  if (!c.k_pages || !c.v_pages || !c.page_table) return DROPKV_ERR_ARG;
  if (!aligned16(c.k_pages) || !aligned16(c.v_pages) || ((uintptr_t)c.page_table & 3u))
    return DROPKV_ERR_ARG;
  const bool scaled = c.dtype == DROPKV_E4M3;
  if (scaled != (c.k_scale != nullptr) || scaled != (c.v_scale != nullptr)) return DROPKV_ERR_ARG;
  return DROPKV_OK;
}

CacheDev cache_dev(const dropkv_cache& c) {
  CacheDev d;
  d.B = c.B;
  d.Hkv = c.Hkv;
  d.d = c.d;
  d.n_pages = c.n_pages;
  d.page = c.page_size;
  d.max_pages = c.max_pages;
  d.cap = c.max_pages * c.page_size;
  d.fpage = FastDiv::of((uint32_t)c.page_size);
  d.k = c.k_pages;
  d.v = c.v_pages;
  d.ks = c.k_scale;
  d.vs = c.v_scale;
  d.table = c.page_table;
  return d;
}

}  // namespace dropkv

using namespace dropkv;

extern "C" dropkv_status dropkv_cache_write(const dropkv_cache* cache,
                                            const dropkv_cache_rows* rows, int32_t* status_dev,
                                            void* stream) {
  NvtxRange range("dropkv_cache_write");
  return run_rows<true>(cache, rows, status_dev, stream);
}

extern "C" dropkv_status dropkv_cache_read(const dropkv_cache* cache,
                                           const dropkv_cache_rows* rows, int32_t* status_dev,
                                           void* stream) {
  NvtxRange range("dropkv_cache_read");
  return run_rows<false>(cache, rows, status_dev, stream);
}
