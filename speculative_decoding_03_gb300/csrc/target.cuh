// What the target's side of a step shares (cache.cu, tree_attention.cu, tree_verify.cu): the
// requests' rows, their trees and their places in a paged cache.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace dspark {

struct RequestRows {
  int row0, n;   // rows row0 .. row0 + n - 1 (n = 0: none, or none that can be used)
};

// Rows of request b: packed (starts) or padded (counts, or all N of them).  Counts outside
// [0, N] and rows outside the batch are reported and give no rows.
__device__ __forceinline__ RequestRows request_rows(const TargetRows& t, int b, int* err) {
  RequestRows r;
  if (t.starts) {
    r.row0 = t.starts[b];
    r.n = t.starts[b + 1] - r.row0;
    if (r.row0 < 0 || r.n < 0 || r.n > t.N || r.row0 > t.rows - r.n) {
      set_device_error(err, DSPARK_ERR_DEVICE_CHECK);
      r.n = 0;
    }
  } else {
    r.row0 = b * t.N;
    r.n = t.counts ? t.counts[b] : t.N;
    if (r.n < 0 || r.n > t.N) {
      set_device_error(err, DSPARK_ERR_DEVICE_CHECK);
      r.n = 0;
    }
  }
  return r;
}

// A request's tokens in the cache before the step; -1 (reported) where they and `more` others
// do not fit its pages.
__device__ __forceinline__ int checked_length(const TargetSlots& s, int len, int more, int* err) {
  if (len < 0 || (long long)len + more > (long long)s.max_pages << s.page_shift) {
    set_device_error(err, DSPARK_ERR_DEVICE_CHECK);
    return -1;
  }
  return len;
}
__device__ __forceinline__ int request_length(const TargetSlots& s, int b, int more, int* err) {
  return checked_length(s, s.lengths[b], more, err);
}

// The page of a slot; -1 (reported) where the table names none of the cache's.
__device__ __forceinline__ int slot_page(const TargetSlots& s, int b, int slot, int* err) {
  const int page = s.pages[(long long)b * s.max_pages + (slot >> s.page_shift)];
  if (page < 0 || page >= s.n_pages) {
    set_device_error(err, DSPARK_ERR_DEVICE_CHECK);
    return -1;
  }
  return page;
}

// A token's parent by its place i in the request: a chain's, or the table's (one that is not
// before the token is reported and counts as none).
__device__ __forceinline__ int parent_of(const int32_t* parents, int row, int i, int* err) {
  if (!parents) return i - 1;
  const int p = parents[row];
  if (p < -1 || p >= i) {
    set_device_error(err, DSPARK_ERR_DEVICE_CHECK);
    return -1;
  }
  return p;
}

}  // namespace dspark
