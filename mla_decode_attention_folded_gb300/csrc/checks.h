// Host checks shared by the entry points (api.cu): MLA_OK or an error.
#pragma once

#include <cstddef>
#include <cstdint>

#include "internal.h"

namespace mlafold {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int check_shape(const mla_shape* s);
int check_device();
bool scales_ok(float bmm1, float bmm2);   // bmm1 finite and positive, bmm2 finite

}  // namespace mlafold
