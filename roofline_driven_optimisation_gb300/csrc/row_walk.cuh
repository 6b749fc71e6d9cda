// A thread's places among rows of `width` values: place number `first`, and every
// `step`-th after it, row by row.  Counted as row and place in the row, because the rows
// of one page may hold more than 2^31 values.
#ifndef G3_ROW_WALK_CUH
#define G3_ROW_WALK_CUH

namespace g3 {

struct RowWalk {
  unsigned row;                      // behind the last one at the end: up to 2^31 and more
  int at, width, step_rows, step_at;
  __host__ __device__ __forceinline__ RowWalk(int first, int step, int w)
      : row(first / w), at(first % w), width(w), step_rows(step / w), step_at(step % w) {}
  __host__ __device__ __forceinline__ bool within(int rows) const { return row < (unsigned)rows; }
  __host__ __device__ __forceinline__ void next() {
    at += step_at;
    row += step_rows;
    if (at >= width) {
      at -= width;
      ++row;
    }
  }
};

}  // namespace g3

#endif  // G3_ROW_WALK_CUH
