// Extents of the arrays that a call of the selective block may touch, and the check of one
// access against them.  The bounds-checked build (-DS4_BOUNDS_CHECK) makes it for every access
// to global memory; host code may include this header alone.
#pragma once

#ifdef __CUDACC__
#define S4_HOST_DEVICE __host__ __device__
#else
#define S4_HOST_DEVICE
#endif

namespace s4impl {

// An array of blocks of `width` consecutive bytes in up to three strided dimensions, the largest
// stride first; what lies between the blocks belongs to others.
struct Extent {
  unsigned long long at;
  long long stride[3], count[3], width;
  bool read, write;
};

S4_HOST_DEVICE inline bool extent_holds(const Extent& e, unsigned long long at, long long bytes) {
  if (at < e.at) return false;
  long long off = (long long)(at - e.at);
  for (int d = 0; d < 3; ++d) {
    if (e.stride[d] <= 0) continue;
    const long long i = off / e.stride[d];
    off -= (i < e.count[d] ? i : e.count[d] - 1) * e.stride[d];
  }
  return off + bytes <= e.width;
}

// Whether an access of `bytes` bytes lies inside one block of an array that may be accessed so,
// at a multiple of `align`.
S4_HOST_DEVICE inline bool access_ok(const Extent* list, int n, unsigned long long at, long long bytes, int align,
                                     bool write) {
  if (at % align != 0) return false;
  for (int i = 0; i < n; ++i)
    if ((write ? list[i].write : list[i].read) && extent_holds(list[i], at, bytes)) return true;
  return false;
}

// The arrays of one call (to be made as Extents x{}).  Without constructors: a copy lies in device memory.
struct Extents {
  static constexpr int kMost = 32;
  Extent list[kMost];
  int n;

  // `c` elements of `e` bytes, [c0][c1][c2] of them at strides (in elements)
  void add(const void* p, int e, bool read, bool write, long long c, long long c0 = 1, long long s0 = 0, long long c1 = 1,
           long long s1 = 0, long long c2 = 1, long long s2 = 0) {
    if (!p || n == kMost) return;
    Extent x{(unsigned long long)p, {s0 * e, s1 * e, s2 * e}, {c0, c1, c2}, c * e, read, write};
    for (int d = 0; d < 3; ++d)
      if (x.count[d] <= 1) x.stride[d] = 0;
    for (int i = 0; i < 2; ++i)
      for (int d = 0; d < 2; ++d)
        if (x.stride[d] < x.stride[d + 1]) {
          const long long s = x.stride[d], k = x.count[d];
          x.stride[d] = x.stride[d + 1], x.count[d] = x.count[d + 1];
          x.stride[d + 1] = s, x.count[d + 1] = k;
        }
    list[n++] = x;
  }
  void in(const void* p, int e, long long c, long long rows = 1) { add(p, e, true, false, c, rows, c); }
  void out(const void* p, int e, long long c, long long rows = 1) { add(p, e, false, true, c, rows, c); }
  void scratch(const void* p, int e, long long c, long long rows = 1) { add(p, e, true, true, c, rows, c); }
  // [batch][L][c] with the strides of s4_rows, s4_rows_out
  template <typename Rows>
  void in_rows(const Rows& r, int e, int batch, int L, long long c) { add(r.p, e, true, false, c, batch, r.batch, L, r.row); }
  template <typename Rows>
  void out_rows(const Rows& r, int e, int batch, int L, long long c) { add(r.p, e, false, true, c, batch, r.batch, L, r.row); }
};

}  // namespace s4impl
