// host_checks.h -- what the entry points check their arguments with.
#pragma once

#include <cstddef>
#include <cstdint>

#include "gdn.h"

namespace gdn {

struct Range {
  uintptr_t lo, hi;  // [lo, hi); empty when lo == hi
};

inline Range range_of(const void *p, size_t bytes) {
  uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, a + (p ? bytes : 0)};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Bytes from the first row's first element to the last row's last.
inline size_t rows_bytes(long long rows, long long ld, long long cols, size_t el) {
  return rows < 1 ? 0 : ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * el;
}

// Whether rows of wa bytes at a and of wb bytes at b, both `pitch` bytes apart,
// are disjoint column blocks of one buffer.
inline bool column_blocks(const void *a, size_t wa, const void *b, size_t wb, size_t pitch) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  const size_t d = x <= y ? (y - x) % pitch : (pitch - (x - y) % pitch) % pitch;  // b's column, from a's
  return d >= wa && d + wb <= pitch;
}

// The device error word and the SM count of the current device, looked up once
// per device: the smallest calls take a few microseconds, of which the look-up
// would be one.  GDN_ERR_NO_DEVICE where it is not an sm_103 GPU.
struct DeviceInfo {
  unsigned int *err;
  int sms;
};
gdn_status device_info(DeviceInfo *out);

}  // namespace gdn
