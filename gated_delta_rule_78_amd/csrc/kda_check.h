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

bool supported_width(int d) { return d == 64 || d == 128; }

}  // namespace
