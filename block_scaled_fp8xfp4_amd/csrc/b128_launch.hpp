// Internal launchers of the experts' tokens and of FP8 products with a scale
// for each block of 128 (api.cpp validates, these launch).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mx {

constexpr int B128 = 128;                         // elements that share a scale along the reduction
constexpr int64_t TOKEN_MAX_CHUNKS = int64_t(1) << 31;   // threads of one call
constexpr int TOKEN_MAX_H = 1 << 30;              // columns, so that one a batch of pieces past the last is still an int

struct PermuteArgs {
  const uint8_t* x; int64_t x_ld; int64_t row;    // rows of `row` bytes, x_ld bytes apart
  const uint8_t* x_sc; int64_t sc;                // their scales, `sc` bytes a row (0: none)
  const int32_t* slot_pos; int T, k;
  uint8_t* out; uint8_t* out_sc; int64_t out_rows;
};
int64_t permute_chunks(int64_t row, int64_t sc);  // threads per row
hipError_t launch_permute(const PermuteArgs& a, hipStream_t stream);

struct UnpermuteArgs {
  const void* o; bool o_bf16; int64_t o_rows;     // [o_rows][H]
  const float* w; const int32_t* slot_pos;        // [T][k]; w NULL: ones
  int T, k, H;
  void* y; bool y_bf16;                           // [T][H]; the gradient's dy
  void* d_o; float* dw;                           // gradient: [o_rows][H] of o's type, [T][k]; each may be NULL
};
hipError_t launch_unpermute(const UnpermuteArgs& a, hipStream_t stream);
hipError_t launch_unpermute_grad(const UnpermuteArgs& a, hipStream_t stream);

// codes and scales of rows (swiglu: of silu(gate) * up of rows of 2 cols), 1 x 128 blocks
hipError_t launch_quantize128_rows(const void* src, bool bf16, int64_t ld, int64_t rows, int64_t cols, bool swiglu,
                                   uint8_t* q, float* sc, hipStream_t stream);
// 128 x 128 blocks of count matrices [rows][cols], rows ld elements apart
hipError_t launch_quantize128_tiles(const void* src, bool bf16, int64_t ld, int64_t count, int64_t rows, int64_t cols,
                                    uint8_t* q, float* sc, hipStream_t stream);
// 128 rows of one column, groups of rows apart: q [cols][q_ld], sc [cols][q_ld / 128]
hipError_t launch_quantize128_t(const void* src, bool bf16, int64_t ld, int64_t rows, int cols, const int32_t* offsets,
                                int E, uint8_t* q, float* sc, int64_t q_ld, hipStream_t stream);

// y[m][n] = sum over blocks of sa[m][b] * sw[n or n / 128][b] * (the block's sum of a w)
struct B128Args {
  const uint8_t* a; const float* a_sc;            // rows of ld bytes, and of ld_sc scales
  const uint8_t* w; const float* w_sc;
  int64_t ld, ld_sc;
  int M, N, K;                                    // M: rows in all (grouped), or one matrix's
  const int32_t* offsets; int E;                  // groups: of rows, or of K (weight gradient); NULL: none
  void* y; bool bf16_out;
  bool far;                                       // set by launch_b128: results go past the caches
};
constexpr int64_t B128_MAX_LD = int64_t(1) << 23;
enum class B128Mode { dense, grouped, wgrad };
bool b128_fits(const B128Args& a, B128Mode mode);   // whether one launch holds it
hipError_t launch_b128(B128Args a, B128Mode mode, bool w_rows, hipStream_t stream, const char** variant);

}  // namespace mx
