// cache_attn.cu -- dropkv_cache_attention's entry points: argument checks, the
// choice of the path, the workspace and the launches.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "cache_attn.cuh"

namespace dropkv {

namespace {

constexpr double kLog2E = 1.4426950408889634;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

dropkv_status check_attn(const dropkv_cache* c, const dropkv_cache_attn* t, bool pointers) {
  dropkv_status s = check_cache(c, pointers);
  if (s != DROPKV_OK) return s;
  if (!t || t->Hq < 1 || t->Hq % c->Hkv != 0 || t->T < 1) return DROPKV_ERR_ARG;
  if (t->dtype != DROPKV_BF16 && t->dtype != DROPKV_F32) return DROPKV_ERR_ARG;
  if (t->causal != 0 && t->causal != 1) return DROPKV_ERR_ARG;
  if (!(t->scale >= 0.f) || t->scale * kLog2E > FLT_MAX) return DROPKV_ERR_ARG;
  if (t->path != DROPKV_PATH_AUTO && t->path != DROPKV_PATH_SIMT && t->path != DROPKV_PATH_TENSOR)
    return DROPKV_ERR_ARG;
  // rows of a group and (sequence, row tile) items are 32-bit
  if ((double)(t->Hq / c->Hkv) * t->T > 1.0e9) return DROPKV_ERR_ARG;
  if ((double)c->B * (t->Hq / c->Hkv) * t->T > 1.6e10) return DROPKV_ERR_ARG;
  for (int i = 0; i < 3; ++i)
    if (t->q_stride[i] < 0 || t->out_stride[i] < 0) return DROPKV_ERR_ARG;
  if (!pointers) return DROPKV_OK;
  const int esz = t->dtype == DROPKV_BF16 ? 2 : 4;
  if (!t->q || !t->out || !t->lengths) return DROPKV_ERR_ARG;
  if (((uintptr_t)t->q | (uintptr_t)t->out) % esz) return DROPKV_ERR_ARG;
  if (((uintptr_t)t->lse | (uintptr_t)t->lengths | (uintptr_t)t->q_lengths) & 3u)
    return DROPKV_ERR_ARG;
  return DROPKV_OK;
}

// The tensor path's sizes: pool rows that fit 32 bits, and the types and head
// dims its kernels are built for.
bool tensor_sizes(const dropkv_cache& c, const dropkv_cache_attn& t) {
  return t.dtype == DROPKV_BF16 && (c.dtype == DROPKV_BF16 || c.dtype == DROPKV_E4M3) &&
         (c.d == 64 || c.d == 128) &&
         (double)c.n_pages * c.Hkv * c.page_size < 2147483648.0;
}
// 16-byte loads of q and stores of out
bool tensor_aligned(const dropkv_cache_attn& t) {
  bool ok = aligned16(t.q) && aligned16(t.out);
  for (int i = 0; i < 3; ++i) ok = ok && t.q_stride[i] % 8 == 0 && t.out_stride[i] % 8 == 0;
  return ok;
}
int path_of(const dropkv_cache& c, const dropkv_cache_attn& t) {
  if (t.path == DROPKV_PATH_SIMT) return DROPKV_PATH_SIMT;
  if (tensor_sizes(c, t) && tensor_aligned(t)) return DROPKV_PATH_TENSOR;
  return t.path == DROPKV_PATH_TENSOR ? -1 : DROPKV_PATH_SIMT;
}

// Query rows a KV head can have.
int64_t group_rows(const dropkv_cache& c, const dropkv_cache_attn& t) {
  return (int64_t)(t.Hq / c.Hkv) * t.T;
}

// The tensor path's kernel by the rows a KV head can have: eight as columns, or
// 16 as rows, of warp-level products; or query tiles of 128 rows.  Both sides of each
// border, in us over 8 sequences of 16K slots, 8 heads, d = 128, bf16 / e4m3:
//   8 rows   few 92 / 62      rows 98 / 83
//   12       few 167 / 108    rows 98 / 84        one query tile 124 / 141
//   16                        rows 98 / 85        one 124 / 141
//   20                        rows 174 / 153      one 124 / 141      two 159 / 175
//   128                                           one 135 / 148      two 165 / 181
//   132                                           one 238 / 266      two 207 / 222
// (64 sequences of 2K alike.  One of 32K, where nothing fills the GPU: 20 rows take 41 /
// 46 as 16-row blocks and 46 / 48 in a query tile, 64 rows 64 / 82 and 49 / 51.)
enum class Tensor { kFew, kRows, kTile128, kTile256 };
Tensor tensor_of(const dropkv_cache& c, const dropkv_cache_attn& t) {
  const int64_t rows = group_rows(c, t);
  return rows <= 8     ? Tensor::kFew
         : rows <= 16  ? Tensor::kRows
         : rows <= 128 ? Tensor::kTile128
                       : Tensor::kTile256;
}
AttnGrid grid_of(Tensor k, int page_dtype) {
  return k == Tensor::kFew    ? attn_grid_few(page_dtype)
         : k == Tensor::kRows ? attn_grid_rows()
                              : attn_grid_tile(k == Tensor::kTile128);
}

size_t layout(const dropkv_cache& c, const AttnGrid& g) {
  return (size_t)2 * g.ctas * g.rows * ((c.d + 3) / 4 * 4 + 4) * sizeof(float);
}

}  // namespace

}  // namespace dropkv

using namespace dropkv;

extern "C" size_t dropkv_cache_attention_workspace_bytes(const dropkv_cache* cache,
                                                         const dropkv_cache_attn* attn) {
  if (check_attn(cache, attn, false) != DROPKV_OK) return 0;
  // the alignment of q and out is not known here: enough for either path
  const size_t simt = layout(*cache, attn_grid_simt(group_rows(*cache, *attn), cache->d));
  if (attn->path == DROPKV_PATH_SIMT || !tensor_sizes(*cache, *attn)) return simt;
  const size_t tensor = layout(*cache, grid_of(tensor_of(*cache, *attn), cache->dtype));
  return std::max(simt, tensor);
}

extern "C" int32_t dropkv_cache_attention_path(const dropkv_cache* cache,
                                               const dropkv_cache_attn* attn) {
  if (check_attn(cache, attn, false) != DROPKV_OK) return -1;
  return path_of(*cache, *attn);
}

// The call; `limit_ns` > 0: the tile kernel's self-test, with a wait that runs out.
static dropkv_status run_attention(const dropkv_cache* cache, const dropkv_cache_attn* attn,
                                   void* workspace, size_t workspace_bytes, int32_t* status_dev,
                                   uint64_t limit_ns, void* stream) {
  dropkv_status s = check_attn(cache, attn, true);
  if (s != DROPKV_OK) return s;
  const dropkv_cache& c = *cache;
  const dropkv_cache_attn& t = *attn;
  if ((uintptr_t)status_dev & 3u) return DROPKV_ERR_ARG;
  const int path = path_of(c, t);
  if (path < 0) return DROPKV_ERR_UNSUPPORTED;
  const bool tensor = path == DROPKV_PATH_TENSOR;
  const Tensor kind = tensor_of(c, t);
  if (limit_ns > 0 && (!tensor || kind == Tensor::kFew || kind == Tensor::kRows))
    return DROPKV_ERR_UNSUPPORTED;  // no waits to run out
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < dropkv_cache_attention_workspace_bytes(cache, attn))
    return DROPKV_ERR_WORKSPACE;
  s = device_ok();
  if (s != DROPKV_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (status_dev)
    if (cudaError_t e = cudaMemsetAsync(status_dev, 0, sizeof(int32_t), st)) return cuda_fail(e);

  const AttnGrid g = tensor ? grid_of(kind, c.dtype) : attn_grid_simt(group_rows(c, t), c.d);
  AttnDev a = {};
  a.c = cache_dev(c);
  a.q = t.q;
  a.out = t.out;
  a.lse = t.lse;
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = t.q_stride[i];
    a.os[i] = t.out_stride[i];
  }
  a.Hq = t.Hq;
  a.G = t.Hq / c.Hkv;
  a.T = t.T;
  a.causal = t.causal;
  a.fG = FastDiv::of((uint32_t)a.G);
  a.nrt = (a.G * t.T + g.rows - 1) / g.rows;
  const double scale = t.scale > 0.f ? (double)t.scale : 1.0 / sqrt((double)c.d);
  a.c_log2 = (float)(scale * kLog2E);
  a.lengths = t.lengths;
  a.q_lengths = t.q_lengths;
  a.part = reinterpret_cast<float*>(workspace);
  a.pstride = (c.d + 3) / 4 * 4 + 4;
  a.status = status_dev;
  a.withhold = limit_ns > 0;
  // the SM clock stays below 2 GHz
  a.wait_clocks = limit_ns > 0 ? 2 * (long long)limit_ns : kWaitClocks;
  cudaError_t e;
  if (!tensor)
    e = launch_attn_simt(a, g, c.dtype, t.dtype, st);
  else if (kind == Tensor::kFew)
    e = launch_attn_few(a, c.dtype, st);
  else if (kind == Tensor::kRows)
    e = launch_attn_rows(a, c.dtype, st);
  else
    e = launch_attn_tile(a, c.dtype, kind == Tensor::kTile128, st);
  if (e == cudaSuccess) e = launch_attn_merge(a, g, t.dtype, st);
  return e == cudaSuccess ? DROPKV_OK : cuda_fail(e);
}

extern "C" dropkv_status dropkv_cache_attention(const dropkv_cache* cache,
                                                const dropkv_cache_attn* attn, void* workspace,
                                                size_t workspace_bytes, int32_t* status_dev,
                                                void* stream) {
  NvtxRange range("dropkv_cache_attention");
  return run_attention(cache, attn, workspace, workspace_bytes, status_dev, 0, stream);
}

extern "C" dropkv_status dropkv_selftest_cache_attention_timeout(
    const dropkv_cache* cache, const dropkv_cache_attn* attn, void* workspace,
    size_t workspace_bytes, int32_t* status_dev, uint64_t limit_ns, void* stream) {
  if (!status_dev || limit_ns == 0 || limit_ns > 1000000000ull) return DROPKV_ERR_ARG;
  return run_attention(cache, attn, workspace, workspace_bytes, status_dev, limit_ns, stream);
}
