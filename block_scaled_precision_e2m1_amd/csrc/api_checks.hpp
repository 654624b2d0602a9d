// Checks of an entry point's buffers, before any HIP call.
#pragma once

#include <stdint.h>

#include <initializer_list>

#include "../../include/fp4gemm.h"

namespace fp4g {

struct Buffer {
  const void* p;
  uint64_t bytes;   // unsigned: a workspace may be said to hold any size_t
  uintptr_t align;
};

// Every buffer present and aligned, every output clear of the inputs and the other outputs.
inline fp4g_status check_buffers(std::initializer_list<Buffer> ins, std::initializer_list<Buffer> outs) {
  for (const auto* list : {&ins, &outs})
    for (const Buffer& b : *list)
      if (b.bytes > 0 && !b.p) return FP4G_EINVAL;
  for (const auto* list : {&ins, &outs})
    for (const Buffer& b : *list)
      if (b.bytes > 0 && reinterpret_cast<uintptr_t>(b.p) % b.align != 0) return FP4G_EALIGN;
  auto clash = [](const Buffer& a, const Buffer& b) {
    // By the distance of the starts: an end may pass 2^64.
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.bytes > 0 && b.bytes > 0 && (x < y ? y - x < a.bytes : x - y < b.bytes);
  };
  for (const Buffer* o = outs.begin(); o != outs.end(); ++o) {
    for (const Buffer& i : ins)
      if (clash(*o, i)) return FP4G_EINVAL;
    for (const Buffer* q = outs.begin(); q != o; ++q)
      if (clash(*o, *q)) return FP4G_EINVAL;
  }
  return FP4G_OK;
}

// Buffers of zero elements are not there.
inline Buffer buf(const void* p, uint64_t bytes, uintptr_t align = 16) { return Buffer{p, bytes, align}; }

}  // namespace fp4g
