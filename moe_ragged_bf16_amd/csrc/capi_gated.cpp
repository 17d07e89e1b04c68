// C ABI of the experts' gated feed-forward (include/moe_ragged_bf16.h): argument
// checks before anything is enqueued, launch sizes, launches.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gated.h"
#include "grouped_gemm.h"
#include "host_common.h"
#include "moe_ragged_bf16.h"

namespace mdg {
namespace {

int check_sizes(int64_t m_rows, int64_t n, int64_t f, int32_t num_groups) {
  if (m_rows < 0 || n <= 0 || f <= 0 || num_groups <= 0) return MDG_EINVAL;
  if (num_groups > kMaxGroups || m_rows > kMaxRows) return MDG_EUNSUPPORTED;
  if (n % kKAlign != 0 || f % kNAlign != 0) return MDG_EUNSUPPORTED;
  if (n > (1 << 20) || f > (1 << 19) || 2 * n * f > INT32_MAX) return MDG_EUNSUPPORTED;
  return MDG_OK;
}

static_assert(MDG_SILU == kActSilu && MDG_GELU_TANH == kActGeluTanh, "activations");

bool activation(int act, GatedParams* p) {
  p->act = act;
  return act == MDG_SILU || act == MDG_GELU_TANH;
}

// Units of the tile kernel, at most: row tiles of every group, the last one of each
// possibly partial, times column tiles.
int64_t units_of(Op op, int64_t m_rows, int64_t f, int32_t num_groups) {
  const int64_t cols = op == kFwd ? kGatedCols : kTileJ;
  return ((m_rows + kTileI - 1) / kTileI + num_groups) * ((f + cols - 1) / cols);
}

// fp32 partial tiles of the tail split (as for the plain products).
int64_t slots_of(int64_t units) { return std::min<int64_t>(units * kMaxSplit, kBalanceSlots); }

enum Kernel { kSmall, kMid, kTile };

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The middle kernel's tiles: 64 x 64 where there are few of them, at most two to a CU (dgrad
// 3.5), as a tile of 128 x 128 alone on a CU takes 0.75 us for a stage of 64 (dgrad 1.1) and one of 64 x 64
// 0.45 (0.65).  64 against 128, fwd: one group of 2 x 2048 x 2048, 100 rows 12.6 / 20; 4 of 2 x 520 x 1624,
// 1111 rows (357 tiles) 18.4 / 19.7; one of 2 x 4096 x 4096, 300 rows (640) 50 / 44.  dgrad: one of 2048
// x 2048, 1500 rows (768) 28 / 33; 2 of 456 x 280, 11127 rows (875) 16.6 / 19.7; 2 of 1000 x 1000, 4000
// rows (1024) 25.5 / 24.2; 4 of 2048 x 2048, 2048 rows (1152) 54 / 44.
int mid_tile(Op op, int64_t m_rows, int64_t f, int64_t active, int64_t cus) {
  constexpr int kHalf = kGatedMidTile / 2;
  const int64_t tiles = (m_rows / kHalf + active) * up(f, op == kFwd ? kHalf / 2 : kHalf);
  return tiles * 2 <= (op == kFwd ? 4 : 7) * cus ? kHalf : kGatedMidTile;
}

// Which kernel takes a launch (one takes all of its groups).  The rules go by the most
// groups that can have rows, as offs is not read here.  n: what is summed over (k in the forward).
// Times in us, weights from memory.
Kernel kernel_of(Op op, int64_t m_rows, int64_t n, int64_t f, int64_t active, int64_t cus) {
  // tiles of the tile kernel, twice over (half of each group's last one is counted)
  const int64_t half_tiles = (m_rows / (kTileI / 2) + active) * up(f, op == kFwd ? kGatedCols : kTileJ);
  if (op == kFwd) {
    // Few rows: the small kernel starts and ends faster and fills the GPU where the middle
    // one has too few tiles; with more rows it reads weights again for each 64 of them and
    // x through the caches, and with many units the middle kernel streams as well.  Small
    // against middle: one group of 2 x 4096 x 4096, 12 rows 20 / 30, 32 27 / 30, 64 51 / 31; 24 of 2 x
    // 8192 x 4096 41 / 35; 80 over 4 of 2 x 1024 x 4096 25 / 30; 200 over 8 of 2 x 512 x 1024 12.3 / 8.7;
    // 15 over 8 of 2 x 416 x 2176 10 / 13; 200 over 8 of 2 x 2048 x 2048 47 / 36; 2 over 8 of 2 x 14336
    // x 4096 84 / 92, 16 310 / 303; 512 over 64 of 2 x 1536 x 2048 152 / 140.  Around the second half's
    // bound of 8 units to a CU, each row in a group of its own (units to a CU in brackets): 16 of 2 x
    // 4096 x 4096, 8 rows [8] 101 / 107, 9 [9] 112 / 130, 12 [12] 146 / 139, 16 [16] 189 / 175; 64 of
    // 2 x 1536 x 2048, 21 rows [7.9] 61 / 61, 24 [9] 69 / 73, 32 [12] 88 / 79; 32 of 2 x 2048 x 2048, 16
    // rows [8] 66 / 63, 24 [12] 92 / 87; 8 of 2 x 14336 x 4096, 3 rows [10.5] 128 / 130, 5 [17.5] 200 /
    // 222, 8 [28] 308 / 310.
    const int64_t units = (active + m_rows / kGatedSmallRows) * up(f, kGatedSmallCols);
    if ((m_rows <= 32 * active && units * 4 <= 5 * cus) || (m_rows <= 16 * active && units <= 8 * cus)) return kSmall;
    // The tile kernel where groups fill a 256-row tile on average and its tiles 5/8 of the CUs, 9/8
    // where k has up to 32 of its stages, over which it fills its pipeline and ends.  Middle
    // against tile: 64 groups of 2 x 1536 x 2048, 128 rows on average 200 / 226, 256 rows 295 /
    // 289; 4 and 8 of 2 x 4096 x 4096, 500 rows 175 / 163 and 329 / 287; 16 of 2 x 1000 x 2000, 188 rows 58 / 83;
    // one of 2 x 2048 x 2048, 1500 rows 33 / 51; 2 of 2 x 2048 x 4096, 1000 rows 47 / 56; one of
    // 2 x 8192 x 2048, 600 rows 59 / 57; 4 of 2 x 2048 x 2048, 3000 rows 69 / 62.  k up to 1024: 3 of 2 x
    // 5904 x 600, 902 rows 35 / 48; 8 of 2 x 1024 x 1024, 8192 rows 54 / 64; one of 2 x 4096 x 1024, 2000 rows
    // 39 / 35; 4 of 2 x 2048 x 1024, 4096 rows 49 / 57, 8192 86 / 88; 2 of 2 x 1024 x 512, 16000 rows 47 / 42.
    return m_rows < 256 * active || half_tiles * 4 <= (n <= 1024 ? 9 : 5) * cus ? kMid : kTile;
  }
  // dgrad, whose tiles have twice the hidden columns, cut along n by the tile kernel where there
  // are few.  Middle against tile, tiles of 64: one group of 4096 x 4096, 300 rows 50 / 43; 4 of 4096 x
  // 512, 600 rows 39 / 33; 2 of 3000 x 1024, 200 rows 29 / 28; 8 of 2560 x 1024, 1200 rows 37 / 39; one of
  // 2048 x 2048, 1500 rows 28 / 41; 8 of 1024 x 512, 125 rows 13 / 21.
  if (mid_tile(op, m_rows, f, active, cus) != kGatedMidTile) return n <= 2560 ? kMid : kTile;
  // Tiles of 128: 64 groups of 2048 x 1536, 64 rows on average 113 / 131, 128 rows 147 / 144, 256 rows 198 /
  // 187; 16 of 2000 x 1000, 188 rows 48 / 49; 4 of 2048 x 2048, 3000 rows 46 / 55, 4096 73 / 68; one of
  // 2048 x 8192, 600 rows 43 / 51; 8 of 2048 x 1024, 8192 rows 74 / 65, of 1024 x 1024 45 / 45; 2 of 1000 x 1000,
  // 4000 rows 24 / 39; 4 of 512 x 2048, 8192 rows 49 / 57; one of 512 x 4096, 16384 rows 204 / 151.
  if (m_rows < 96 * active || (half_tiles <= cus && n <= 2048)) return kMid;
  return half_tiles * 4 <= 9 * cus && n <= 1024 ? kMid : kTile;
}

// What a call of valid sizes comes to on the current device.
struct Call {
  int device;           // a status: whether it can run there
  int64_t cus, active;  // active: groups that can have rows
  Kernel which;
  int tile;             // rows and columns of the middle kernel's tiles
  int64_t grid;         // and its workgroups
  size_t workspace;     // the plan's head (never 0), and the tile kernel's partial tiles where it takes the call
};
Call call_of(Op op, int64_t m_rows, int64_t n, int64_t f, int32_t num_groups) {
  DeviceInfo dev;
  Call c{};
  c.device = check_device(&dev);
  c.cus = dev.cus > 0 ? dev.cus : 256;
  c.active = std::min<int64_t>(num_groups, m_rows);
  c.which = kernel_of(op, m_rows, n, f, c.active, c.cus);
  c.tile = mid_tile(op, m_rows, f, c.active, c.cus);
  const int64_t row_tiles = (m_rows + c.tile - 1) / c.tile + c.active;
  c.grid = up(row_tiles * up(f, op == kFwd ? c.tile / 2 : c.tile), 8) * 8;
  if (c.which == kMid && c.grid * 256 > UINT32_MAX) c.which = kTile;  // (a launch's work-items)
  c.workspace = kTailHeadBytes;
  if (c.which == kTile || c.device != MDG_OK)  // (without a device any kernel could take it)
    c.workspace += (size_t)slots_of(units_of(op, m_rows, f, num_groups)) * kTileI * kTileJ * sizeof(float);
  return c;
}

size_t workspace_of(Op op, int64_t m_rows, int64_t n, int64_t f, int32_t num_groups) {
  return check_sizes(m_rows, n, f, num_groups) == MDG_OK ? call_of(op, m_rows, n, f, num_groups).workspace : 0;
}

int run(Op op, const Call& c, GatedParams* p, int64_t m_rows, int64_t f, int32_t num_groups, void* workspace,
        void* stream) {
  if (c.device != MDG_OK) return c.device;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t err = hipSuccess;
  if (c.which == kSmall) {
    err = launch_gated_small(*p, (int)(c.active + m_rows / kGatedSmallRows), s);
  } else if (c.which == kMid) {
    err = launch_gated_mid(op, *p, c.tile, (int)c.grid, s);
  } else {
    const int64_t units = units_of(op, m_rows, f, num_groups), slots = slots_of(units);
    char* ws = static_cast<char*>(workspace);
    p->g.tail_head = reinterpret_cast<int32_t*>(ws);
    p->g.partial = reinterpret_cast<float*>(ws + kTailHeadBytes);
    p->g.tail_slots = (int32_t)slots;
    int64_t grid = std::min<int64_t>(units + slots, c.cus);
    if (grid >= 8) grid -= grid % 8;
    err = launch_gated(op, *p, (int)grid, s);
    if (err == hipSuccess && slots >= 2)
      err = launch_gated_reduce(op, *p, 8, (int)std::min<int64_t>(kBalanceSlots / 2, slots / 2), s);
  }
  return err == hipSuccess ? MDG_OK : MDG_EHIP;
}

}  // namespace
}  // namespace mdg

using namespace mdg;

extern "C" {

MDG_API size_t grouped_gated_gemm_fwd_workspace_bytes(int64_t m_rows, int64_t f, int64_t k, int32_t num_groups) {
  return workspace_of(kFwd, m_rows, k, f, num_groups);
}

MDG_API size_t grouped_gated_gemm_dgrad_workspace_bytes(int64_t m_rows, int64_t n, int64_t f, int32_t num_groups) {
  return workspace_of(kDgrad, m_rows, n, f, num_groups);
}

MDG_API mdg_status grouped_gated_gemm_fwd(const void* x, const void* w, const int32_t* offs, void* h, void* gate_up,
                                          int activation_code, int64_t m_rows, int64_t f, int64_t k,
                                          int32_t num_groups, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_sizes(m_rows, k, f, num_groups);
  if (st != MDG_OK) return status(st);
  GatedParams p{};
  if (!activation(activation_code, &p)) return status(MDG_EINVAL);
  if (!w || !offs || (m_rows > 0 && (!x || !h))) return status(MDG_EINVAL);
  if (!aligned16(x) || !aligned16(w) || !aligned4(offs) || !aligned16(h) || !aligned16(gate_up)) return status(MDG_EINVAL);
  const Call c = call_of(kFwd, m_rows, k, f, num_groups);
  const size_t need = c.workspace;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MDG_OK) return status(st);
  const Range in[3] = {range_of(x, m_rows * k * 2), range_of(w, (int64_t)num_groups * 2 * f * k * 2),
                       range_of(offs, (int64_t)num_groups * 4)};
  const Range out[3] = {range_of(h, m_rows * f * 2), range_of(gate_up, gate_up ? m_rows * f * 4 : 0),
                        range_of(workspace, (int64_t)need)};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : in)
      if (overlaps(out[i], r)) return status(MDG_EOVERLAP);
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i], out[j])) return status(MDG_EOVERLAP);
  }
  if (m_rows == 0) return status(MDG_OK);
  p.g.a = static_cast<const uint16_t*>(x);
  p.g.b = static_cast<const uint16_t*>(w);
  p.g.offs = offs;
  p.g.out = h;
  p.g.m_rows = m_rows;
  p.g.n = (int32_t)(2 * f);
  p.g.k = (int32_t)k;
  p.g.num_groups = num_groups;
  p.keep = static_cast<uint16_t*>(gate_up);
  p.f = (int32_t)f;
  return status(run(kFwd, c, &p, m_rows, f, num_groups, workspace, stream));
}

MDG_API mdg_status grouped_gated_gemm_dgrad(const void* dy, const void* w_down, const void* gate_up,
                                            const int32_t* offs, void* dgate_up, int activation_code, int64_t m_rows,
                                            int64_t n, int64_t f, int32_t num_groups, void* workspace,
                                            size_t workspace_bytes, void* stream) {
  int st = check_sizes(m_rows, n, f, num_groups);
  if (st != MDG_OK) return status(st);
  GatedParams p{};
  if (!activation(activation_code, &p)) return status(MDG_EINVAL);
  if (!w_down || !offs || (m_rows > 0 && (!dy || !gate_up || !dgate_up))) return status(MDG_EINVAL);
  if (!aligned16(dy) || !aligned16(w_down) || !aligned16(gate_up) || !aligned4(offs) || !aligned16(dgate_up))
    return status(MDG_EINVAL);
  const Call c = call_of(kDgrad, m_rows, n, f, num_groups);
  const size_t need = c.workspace;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MDG_OK) return status(st);
  const Range in[4] = {range_of(dy, m_rows * n * 2), range_of(w_down, (int64_t)num_groups * n * f * 2),
                       range_of(gate_up, m_rows * f * 4), range_of(offs, (int64_t)num_groups * 4)};
  const Range out = range_of(dgate_up, m_rows * f * 4), ws = range_of(workspace, (int64_t)need);
  for (const Range& r : in)
    if (overlaps(out, r) || overlaps(ws, r)) return status(MDG_EOVERLAP);
  if (overlaps(out, ws)) return status(MDG_EOVERLAP);
  if (m_rows == 0) return status(MDG_OK);
  p.g.a = static_cast<const uint16_t*>(dy);
  p.g.b = static_cast<const uint16_t*>(w_down);
  p.g.offs = offs;
  p.g.out = dgate_up;
  p.g.m_rows = m_rows;
  p.g.n = (int32_t)n;
  p.g.k = (int32_t)f;
  p.g.num_groups = num_groups;
  p.gate_up = static_cast<const uint16_t*>(gate_up);
  p.f = (int32_t)f;
  return status(run(kDgrad, c, &p, m_rows, f, num_groups, workspace, stream));
}

}  // extern "C"
