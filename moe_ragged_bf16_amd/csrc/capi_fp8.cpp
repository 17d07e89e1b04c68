// C ABI of the ragged grouped product in 8 bits (include/moe_ragged_bf16.h):
// argument checks before anything is enqueued, launch sizes, launches.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "fp8.h"
#include "grouped_gemm.h"
#include "host_common.h"
#include "moe_ragged_bf16.h"

namespace mdg {
namespace {

size_t align256(size_t b) { return (b + 255) / 256 * 256; }
int64_t blocks_of(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }
int64_t rows_scale_bytes(int64_t m_rows, int64_t k) { return (blocks_of(k) + 3) / 4 * m_rows * 4; }

bool real_dtype(int dtype) { return dtype == MDG_BF16 || dtype == MDG_FP32; }
int64_t dtype_bytes(int dtype) { return dtype == MDG_E4M3 ? 1 : dtype == MDG_FP32 ? 4 : 2; }

int check_device(DeviceInfo* dev) {
  int device = -1;
  const int st = query_device(dev, &device);
  if (st != MDG_OK) return st;
  return dev->gfx950 ? MDG_OK : MDG_EUNSUPPORTED;
}

int check_rows(int64_t m_rows, int64_t k) {
  if (m_rows < 0 || k <= 0) return MDG_EINVAL;
  if (k % kKAlign != 0 || k > (1 << 20) || m_rows > kMaxRows) return MDG_EUNSUPPORTED;
  return MDG_OK;
}

int check_weight(int32_t experts, int64_t n, int64_t k) {
  if (experts <= 0 || n <= 0 || k <= 0) return MDG_EINVAL;
  if (experts > kMaxGroups || n % kNAlign != 0 || k % kKAlign != 0) return MDG_EUNSUPPORTED;
  if (n > (1 << 20) || k > (1 << 20) || fp8_pitch(n) * fp8_pitch(k) > INT32_MAX) return MDG_EUNSUPPORTED;
  return MDG_OK;
}

// Workspace of a product whose x is not in 8 bits yet: q, then its scales.
struct XSpace {
  size_t scale_off, total;
};
XSpace x_space(int64_t m_rows, int64_t k, int x_dtype) {
  XSpace w{0, 0};
  if (x_dtype == MDG_E4M3) return w;
  w.scale_off = align256((size_t)(m_rows * fp8_pitch(k)));
  w.total = align256(w.scale_off + (size_t)rows_scale_bytes(m_rows, k));
  return w;
}

Fp8RowsParams rows_params(const void* x, int dtype, void* q, void* scale, int64_t m_rows, int64_t k) {
  Fp8RowsParams p{};
  p.x = x;
  p.q = static_cast<uint8_t*>(q);
  p.scale = static_cast<uint8_t*>(scale);
  p.m_rows = m_rows;
  p.k = (int32_t)k;
  p.pitch = (int32_t)fp8_pitch(k);
  p.blocks = (int32_t)blocks_of(k);
  p.fp32 = dtype == MDG_FP32;
  return p;
}

mdg_status launched(hipError_t err) { return status(err == hipSuccess ? MDG_OK : MDG_EHIP); }

}  // namespace
}  // namespace mdg

using namespace mdg;

extern "C" {

MDG_API mdg_status grouped_fp8_quantize_rows(const void* x, int dtype, void* q, void* scale, int64_t m_rows,
                                             int64_t k, void* stream) {
  int st = check_rows(m_rows, k);
  if (st != MDG_OK) return status(st);
  if (!real_dtype(dtype) || (m_rows > 0 && (!x || !q || !scale))) return status(MDG_EINVAL);
  if (!aligned16(x) || !aligned16(q) || !aligned4(scale)) return status(MDG_EINVAL);
  const Range rx = range_of(x, m_rows * k * dtype_bytes(dtype)), rq = range_of(q, m_rows * fp8_pitch(k));
  const Range rs = range_of(scale, rows_scale_bytes(m_rows, k));
  if (overlaps(rq, rx) || overlaps(rs, rx) || overlaps(rq, rs)) return status(MDG_EOVERLAP);
  if (m_rows == 0) return status(MDG_OK);
  DeviceInfo dev;
  if ((st = check_device(&dev)) != MDG_OK) return status(st);
  return launched(launch_fp8_quantize_rows(rows_params(x, dtype, q, scale, m_rows, k),
                                           static_cast<hipStream_t>(stream)));
}

MDG_API mdg_status grouped_fp8_quantize_weight(const void* w, int dtype, void* q, void* scale, void* q_t,
                                               void* scale_t, int32_t num_groups, int64_t n, int64_t k,
                                               void* stream) {
  int st = check_weight(num_groups, n, k);
  if (st != MDG_OK) return status(st);
  if (!real_dtype(dtype) || !w || !q || !scale || !q_t != !scale_t) return status(MDG_EINVAL);
  if (!aligned16(w) || !aligned16(q) || !aligned16(q_t)) return status(MDG_EINVAL);
  const int64_t values = num_groups * n * k, scales = num_groups * blocks_of(n) * blocks_of(k);
  const Range in = range_of(w, values * dtype_bytes(dtype));
  const Range out[4] = {range_of(q, num_groups * n * fp8_pitch(k)), range_of(scale, scales),
                        range_of(q_t, q_t ? num_groups * k * fp8_pitch(n) : 0),
                        range_of(scale_t, scale_t ? scales : 0)};
  for (int i = 0; i < 4; ++i) {
    if (overlaps(out[i], in)) return status(MDG_EOVERLAP);
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i], out[j])) return status(MDG_EOVERLAP);
  }
  DeviceInfo dev;
  if ((st = check_device(&dev)) != MDG_OK) return status(st);
  Fp8WeightParams p{};
  p.w = w;
  p.q = static_cast<uint8_t*>(q);
  p.scale = static_cast<uint8_t*>(scale);
  p.qt = static_cast<uint8_t*>(q_t);
  p.scale_t = static_cast<uint8_t*>(scale_t);
  p.experts = num_groups;
  p.n = (int32_t)n;
  p.k = (int32_t)k;
  p.pitch = (int32_t)fp8_pitch(k);
  p.pitch_t = (int32_t)fp8_pitch(n);
  p.fp32 = dtype == MDG_FP32;
  return launched(launch_fp8_quantize_weight(p, static_cast<hipStream_t>(stream)));
}

MDG_API size_t grouped_fp8_gemm_fwd_workspace_bytes(int64_t m_rows, int64_t n, int64_t k, int32_t num_groups,
                                                    int x_dtype) {
  if (check_rows(m_rows, k) != MDG_OK || check_weight(num_groups, n, k) != MDG_OK) return 0;
  if (!real_dtype(x_dtype) && x_dtype != MDG_E4M3) return 0;
  return x_space(m_rows, k, x_dtype).total;
}

MDG_API mdg_status grouped_fp8_gemm_fwd(const void* x, int x_dtype, const void* x_scale, const void* w,
                                        const void* w_scale, const int32_t* offs, void* y, int64_t m_rows,
                                        int64_t n, int64_t k, int32_t num_groups, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  int st = check_rows(m_rows, k);
  if (st != MDG_OK || (st = check_weight(num_groups, n, k)) != MDG_OK) return status(st);
  const bool quantized = x_dtype == MDG_E4M3;
  if (!quantized && !real_dtype(x_dtype)) return status(MDG_EINVAL);
  if (!w || !w_scale || !offs || (m_rows > 0 && (!x || !y))) return status(MDG_EINVAL);
  if (quantized ? (m_rows > 0 && !x_scale) : x_scale != nullptr) return status(MDG_EINVAL);
  if (!aligned16(x) || !aligned4(x_scale) || !aligned16(w) || !aligned4(offs) || !aligned16(y))
    return status(MDG_EINVAL);
  const XSpace xs = x_space(m_rows, k, x_dtype);
  if (xs.total > 0) {
    if (!workspace || workspace_bytes < xs.total) return status(MDG_EWORKSPACE);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return status(MDG_EINVAL);
  }
  const Range in[5] = {range_of(x, m_rows * (quantized ? fp8_pitch(k) : k) * dtype_bytes(x_dtype)),
                       range_of(x_scale, quantized ? rows_scale_bytes(m_rows, k) : 0),
                       range_of(w, num_groups * n * fp8_pitch(k)),
                       range_of(w_scale, num_groups * blocks_of(n) * blocks_of(k)),
                       range_of(offs, (int64_t)num_groups * 4)};
  const Range ry = range_of(y, m_rows * n * 2), rws = range_of(workspace, (int64_t)xs.total);
  for (const Range& r : in)
    if (overlaps(ry, r) || overlaps(rws, r)) return status(MDG_EOVERLAP);
  if (overlaps(ry, rws)) return status(MDG_EOVERLAP);
  if (m_rows == 0) return status(MDG_OK);
  DeviceInfo dev;
  if ((st = check_device(&dev)) != MDG_OK) return status(st);

  const hipStream_t s = static_cast<hipStream_t>(stream);
  Fp8GemmParams p{};
  p.x = static_cast<const uint8_t*>(x);
  p.xs = static_cast<const uint32_t*>(x_scale);
  p.w = static_cast<const uint8_t*>(w);
  p.ws = static_cast<const uint8_t*>(w_scale);
  p.offs = offs;
  p.y = static_cast<uint16_t*>(y);
  p.m_rows = m_rows;
  p.n = (int32_t)n;
  p.k = (int32_t)fp8_pitch(k);
  p.num_groups = num_groups;
  p.blocks = (int32_t)blocks_of(k);
  const int64_t active = std::min<int64_t>(num_groups, m_rows);  // groups with rows, at most
  if (!quantized) {
    uint8_t* q = static_cast<uint8_t*>(workspace);
    if (launch_fp8_quantize_rows(rows_params(x, x_dtype, q, q + xs.scale_off, m_rows, k), s) != hipSuccess)
      return status(MDG_EHIP);
    p.x = q;
    p.xs = reinterpret_cast<const uint32_t*>(q + xs.scale_off);
  }
  const int64_t cus = dev.cus > 0 ? dev.cus : 256;
  // Pieces of a kernel's rows, at most: whole ones and a partial one of every group.
  const auto pieces = [&](int64_t rows) { return (m_rows + rows - 1) / rows + active; };
  const auto columns = [&](int64_t cols) { return (n + cols - 1) / cols; };
  // Few rows: the weights are read at the memory's rate either way, and the small
  // kernel starts and ends faster; with more rows it reads weights that the middle
  // kernel would read once again, and x through the caches.  64 groups of 1536 x 2048,
  // small against middle: 2 rows on average 33 / 40 us, 8 rows 44 / 44, 16 rows
  // 51 / 44; where all its units run at once it gains at more rows: 1 group of
  // 4096 x 4096, 128 rows 16 / 23, 200 rows 26 / 23; 16 of 1000 x 2000, 20 rows 12 / 15.
  // The rules go by the most groups that can have rows, as offs is not read here.  Where
  // all rows are one group's, the small kernel reads that group's weight once for each
  // 64 of them: 1536 x 2048, 300 rows in one of 64 groups 9 us (in a call of that group alone,
  // by the middle kernel, 14), 512 rows 14 (14), 2000 rows in one of 256 groups 80 (15).
  const int64_t small = active + m_rows / kFp8SmallRows;
  if (m_rows <= 8 * active || (m_rows <= 128 * active && small * columns(kFp8SmallCols) <= 3 * cus))
    return launched(launch_fp8_small(p, (int)small, s));
  // The tile kernel where groups fill half a tile on average and its tiles (half of
  // each group's last one, on average, is counted) 5/8 of the CUs.  Middle against
  // tile: 64 groups of 1536 x 2048, 96 rows on average 57 / 65 us, 128 rows 68 / 67, 512
  // rows 159 / 129; 8 of 4096 x 4096, 128 rows (128 tiles) 48 / 57, 192 rows (160 tiles)
  // 65 / 59, 384 rows 86 / 65.
  const int64_t mid = (pieces(kFp8MidTile) * columns(kFp8MidTile) + 7) / 8 * 8;
  const bool fits = mid * 256 <= UINT32_MAX;  // a launch's work-items; the tile kernel walks its tiles
  if (fits && (m_rows < 128 * active || (m_rows / 128 + active) * columns(kTileJ) * 4 < 5 * cus))
    return launched(launch_fp8_mid(p, (int)mid, s));
  return launched(launch_fp8_gemm(p, (int)std::min(pieces(kTileI) * columns(kTileJ), cus), s));
}

}  // extern "C"
