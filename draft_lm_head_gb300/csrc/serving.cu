// C entry points of the serving operators (include/lmhead.h): host-side
// validation and launches.
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "lmhead.h"

using namespace lmhead;

namespace {

constexpr int kMaxRows = 1 << 20;

inline int status(cudaError_t e) { return e == cudaSuccess ? LMHEAD_OK : LMHEAD_ERR_CUDA; }

}  // namespace

extern "C" {

int lmhead_page_plan(const int32_t* lens, const int32_t* new_lens, int S, int32_t* table,
                     int width, const int32_t* free_pages, int free_cap,
                     const int32_t* free_count, int page_size, int max_tokens,
                     int32_t* out_slots, int32_t* out_positions, int32_t* out_cu,
                     int32_t* out_granted, int32_t* out_free_left, lmhead_stream stream) {
  if (!lens || !new_lens || !table || !free_pages || !free_count || !out_slots ||
      !out_positions || !out_cu || !out_granted || !out_free_left)
    return LMHEAD_ERR_NULL;
  if (S < 1 || S > kMaxRows || width < 1 || free_cap < 0 || page_size < 1 || page_size > 65536 ||
      max_tokens < 1 || (int64_t)S * width > INT32_MAX)
    return LMHEAD_ERR_SHAPE;
  if (out_free_left == free_count) return LMHEAD_ERR_SHAPE;
  return status(launch_page_plan(lens, new_lens, S, table, width, free_pages, free_cap, free_count,
                                 page_size, max_tokens, out_slots, out_positions, out_cu,
                                 out_granted, out_free_left, device_error_word(),
                                 (cudaStream_t)stream));
}

}  // extern "C"
