// gmm_tensor.hpp -- what the argument checks need to know about a gmm_tensor
// (plain host C++, no HIP).
#pragma once

#include <stdint.h>

#include <string>

#include "gmm.h"

namespace gmmh {

inline std::string shape_str(const gmm_tensor* t) {
  std::string s = "(";
  for (int i = 0; i < t->ndim && i < 4; ++i) {
    if (i) s += ",";
    s += std::to_string(t->shape[i]);
  }
  return s + ")";
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int elem_size(int dtype) {
  switch (dtype) {
    case GMM_F32: return 4;
    case GMM_BF16: return 2;
    case GMM_F8E4M3FN: return 1;
    case GMM_F8E5M2: return 1;
    case GMM_E8M0: return 1;
    case GMM_I8: return 1;
    case GMM_I32: return 4;
    case GMM_I64: return 8;
    default: return 0;
  }
}

inline long long numel(const gmm_tensor* t) {
  long long n = 1;
  for (int i = 0; i < t->ndim; ++i) n *= t->shape[i];
  return n;
}

inline bool four_bit(int dtype) { return dtype == GMM_I4 || dtype == GMM_U4 || dtype == GMM_F4E2M1; }

// bytes of a tensor's data (four-bit types: two elements to a byte)
inline long long tensor_bytes(const gmm_tensor* t) {
  return four_bit(t->dtype) ? (numel(t) + 1) / 2 : numel(t) * elem_size(t->dtype);
}

inline bool overlaps(const gmm_tensor* a, const gmm_tensor* b) {
  if (!a || !b || !a->data || !b->data) return false;
  const char* a0 = static_cast<const char*>(a->data);
  const char* b0 = static_cast<const char*>(b->data);
  const char* a1 = a0 + tensor_bytes(a);
  const char* b1 = b0 + tensor_bytes(b);
  return a0 < b1 && b0 < a1;
}

}  // namespace gmmh
