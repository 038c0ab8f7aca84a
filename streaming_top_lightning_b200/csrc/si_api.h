// Host helpers that the files of the C ABI share (defined in api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "streamindex.h"

namespace si {

struct DevInfo {
  bool init = false;
  bool ok = false;
  int sms = 0;
  int max_smem = 0;
  uint32_t* err = nullptr;
  unsigned long long* role = nullptr;  // profiling build: role counters
};

// The current device, checked to be an sm_100 part; SI_OK or an error.
int dev_info(DevInfo** out);

// Shared memory and SM count to plan with: the current device's, or the
// sm_100 limits on a host with no usable device.
void plan_limits(int* max_smem, int* sms);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// 2-D row-major [rows, cols] tensor map with a {box_inner, box_rows} box and
// the given swizzle; out-of-range rows read as zero.
int make_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, uint64_t rows,
             uint64_t cols, uint32_t esz, uint32_t box_inner, uint32_t box_rows,
             CUtensorMapSwizzle sw);

// Tensor map of a bf16 [d3, d2, d1, d0] tensor (d0 fastest) with 64-element
// rows in the 128-byte swizzle: a {64, box1, box2, 1} box; what lies outside
// reads as zero.  d2 of pitch2 such planes are in it.
int make_map4(CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t d3,
              uint32_t box1, uint32_t box2, uint64_t pitch2);

struct Opts {
  int key_chunk, scratch_mb, grid_ctas, timeout_ms, debug_flags, row_finish, key_tile,
      strip_slots;
  cudaEvent_t ev_begin, ev_end;
  cudaEvent_t* ev_list;  // [2i], [2i+1] around query block i's score launch
  int ev_count;
  int plan_heads, plan_dim, plan_fp8;  // si_topk_scores: the fused kernel's plan
};

// The options of a call, checked; o may be null.
int read_opts(const si_options* o, Opts* out);

}  // namespace si
