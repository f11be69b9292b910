// kda_check.h -- host-side argument checks shared by the C ABI files.
#pragma once
#include <stdint.h>

namespace {

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

Range range_of(const void* p, int64_t bytes) {
  uintptr_t a = (uintptr_t)p;
  return Range{a, a + (uintptr_t)(bytes > 0 ? bytes : 0)};
}

bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

bool misaligned(const void* p, unsigned bytes = 16) { return ((uintptr_t)p & (bytes - 1)) != 0; }

// Rows of a call: up to 2^32.  B, T >= 0, H >= 1; the product of all three may pass 64 bits.
bool too_many_rows(int64_t B, int64_t T, int64_t H) { return B * T > (int64_t(1) << 32) / H; }

bool supported_width(int d) { return d == 64 || d == 128; }

}  // namespace
