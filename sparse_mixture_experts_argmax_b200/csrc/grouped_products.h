// Internal interface of the grouped products: the plan that the device makes
// from the group offsets, and the launchers of the kernels that run on it.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"

namespace swl {

// One call's sizes: rows of the buffers, width of x, width of y, groups.
struct GroupedShape {
  int64_t R, K, O, N;
  int dtype;
};

// Workspace of a call (device).
struct GroupedPlan {
  WsHeader* hdr;       // err, next_tile
  int* tile_prefix;    // [N + 1] row tiles of groups before e (tile_rows rows each)
  float* bias_part;    // [row tiles, at most][O] partial bias gradients
  float* sums;         // bf16 sums of many pieces: a CTA's half of D, [CTA][256][128]
  void* maps;          // bf16: [2 N] tensor maps, dy's and x's rows up to each group's end
};

enum GroupedWhich : int { kGroupedFwd = 0, kGroupedDx = 1, kGroupedDw = 2 };

// Reads and checks the offsets (0 <= off[0] <= ... <= off[N] <= R), counts the row
// tiles and resets the header.  Bad offsets: kDevIndexOutOfRange and no tiles, so
// that the kernels behind it touch nothing.  maps: dW's two templates, or NULL.
cudaError_t launch_grouped_plan(const GroupedShape& s, const GroupedPlan& p, const int* offsets,
                                int tile_rows, const CUtensorMap* maps, cudaStream_t stream);

// Bound of a kernel's waits: some last for a whole tile, whose steps go 64 deep along the
// summed axis (2^30 rows of one group in dW, at most), so the limit grows with them:
// 20 us a step, of which the slowest (fp32) takes 2.2.
inline unsigned long long grouped_wait_ns(int64_t depth) {
  return wait_limit_ns() + 20000ull * static_cast<unsigned long long>((depth + 63) / 64);
}

// The products of fp32 tensors.  which: y = x W^T + b (kGroupedFwd: a = x, b = W,
// bias), dx = dy W (kGroupedDx: a = dy, b = W) or dW = dy^T x (kGroupedDw: a = dy, b = x;
// every group written, empty ones zero).
int grouped_f32_tile_rows();
cudaError_t launch_grouped_f32(const GroupedShape& s, const GroupedPlan& p, GroupedWhich which,
                               const int* offsets, const void* a, const void* b, const void* bias,
                               void* out, int num_sms, cudaStream_t stream);

// The same of bf16 tensors; templates: dW's maps for the plan.
bool grouped_sm100_templates(const GroupedShape& s, const void* dy, const void* x, CUtensorMap* out);
int grouped_sm100_tile_rows(const GroupedShape& s);
// CTAs whose sums may have to be kept between pieces (0: no sum is that long).
int grouped_sm100_summing_ctas(const GroupedShape& s);
constexpr size_t kSumsPerCta = 256 * 128;
// Row tiles of a call with up to R rows, at most (fewer rows may take smaller tiles).
int64_t grouped_sm100_most_tiles(const GroupedShape& s);
cudaError_t launch_grouped_sm100(const GroupedShape& s, const GroupedPlan& p, GroupedWhich which,
                                 const int* offsets, const void* a, const void* b,
                                 const void* bias, void* out, int num_sms, cudaStream_t stream);

// The forward product for a few rows, without a plan: checks the offsets and writes the
// device status itself.  Taken for 8 bf16 rows, 16 when there are as many groups (they
// are then spread, about one each), and 32 fp32 rows.  8 / 16 / 32 rows over 128 groups of
// 4096 x 1024 bf16 take 18 / 24 / 46 us with it and 21 / 32 / 45 us on the tensor cores,
// 16 in one group of 1024 x 1024 26 and 18 us; 16 / 32 over 128 groups of 2048 x 1024 fp32
// 22 / 43 us and 72 / 117 us.
inline bool grouped_few(const GroupedShape& s) {
  return s.R > 0 && s.R <= (s.dtype == 0 ? 32 : s.N >= s.R ? 16 : 8);
}
cudaError_t launch_grouped_few(const GroupedShape& s, const GroupedPlan& p, const int* offsets,
                               const void* x, const void* W, const void* bias, void* y,
                               cudaStream_t stream);

// db[e] = sum of the group's rows of dy (fp32 sums in a fixed order); tile_rows as
// given to the plan.
cudaError_t launch_grouped_bias_grad(const GroupedShape& s, const GroupedPlan& p,
                                     const int* offsets, const void* dy, void* db, int tile_rows,
                                     cudaStream_t stream);

}  // namespace swl
