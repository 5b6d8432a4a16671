// Sizes of the parts of a workspace.
#pragma once
#include <cstddef>

namespace cpattn {

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace cpattn
