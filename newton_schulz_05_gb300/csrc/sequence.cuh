// What the operators over sequences (scan.cu, heads.cu, log_probs.cu, policy.cu)
// share on the host.
#pragma once

#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "pieces.cuh"

namespace muon {

namespace {

inline bool off(const void* p, size_t es) { return reinterpret_cast<uintptr_t>(p) % es != 0; }
template <typename... P> bool any_off(size_t es, const P*... p) { return (off(p, es) || ...); }

// f(value of the element type)
template <typename F> auto by_type(int dtype, F f) {
  if (dtype == MUON_BF16) return f(__nv_bfloat16());
  return f(float());
}
inline size_t size_of(int dtype) { return dtype == MUON_BF16 ? 2 : 4; }
inline bool known(int dtype) { return dtype == MUON_BF16 || dtype == MUON_F32; }

}  // namespace

}  // namespace muon
