// What the host sides of the C ABI entry points share: the error detail, the
// checks of pointers and workspaces, and the status of a launch.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/moe.h"

namespace moe {

// Record the detail of a failed validation (moe_last_error_detail) and return s.
moe_status fail(moe_status s, const char* fmt, ...);

constexpr size_t kAlign = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The workspace is there, aligned and at least `need` bytes long.
moe_status check_ws(const void* ws, size_t ws_bytes, size_t need);
// MOE_ERR_CUDA with its text when a launch before this call failed.
moe_status cuda_status();
// MOE_ERR_CUDA with its text for a launch that returned e.  The runtime's last error is
// taken too: the next call's cuda_status would report it as its own.
moe_status launch_status(cudaError_t e, const char* what);

template <typename T> T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

}  // namespace moe

#define MOE_CHECK(x) do { moe_status s_ = (x); if (s_ != MOE_OK) return s_; } while (0)
#define MOE_NONNULL(p) do { if (!(p)) return moe::fail(MOE_ERR_INVALID_ARG, #p " is NULL"); \
    if (!moe::aligned16(p)) return moe::fail(MOE_ERR_INVALID_ARG, #p " is not 16-byte aligned"); } while (0)
#define MOE_ALIGNED(p) do { if ((p) && !moe::aligned16(p)) return moe::fail(MOE_ERR_INVALID_ARG, #p " is not 16-byte aligned"); } while (0)
#define MOE_ALIGNED4(p) do { if ((p) && (reinterpret_cast<uintptr_t>(p) & 3u)) return moe::fail(MOE_ERR_INVALID_ARG, #p " is not 4-byte aligned"); } while (0)
#define MOE_NONNULL4(p) do { if (!(p)) return moe::fail(MOE_ERR_INVALID_ARG, #p " is NULL"); MOE_ALIGNED4(p); } while (0)
