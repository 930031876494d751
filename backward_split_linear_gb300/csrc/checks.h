// Argument checks that every C entry point shares (see the conventions in zb.h).
#pragma once

#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/zb.h"
#include "launch.h"

namespace zbk {

constexpr int32_t kMaxFeature = 1 << 20;
constexpr int32_t kMaxTokens = 1 << 24;

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A tensor with `tokens` rows: may be NULL when there are no rows.
inline bool rows_ok(const void* p, int32_t tokens) { return tokens == 0 ? (p == nullptr || aligned16(p)) : (p && aligned16(p)); }

// A tensor whose size does not depend on the tokens.
inline bool fixed_ok(const void* p) { return p && aligned16(p); }

inline bool feature_ok(int32_t f) { return f > 0 && f <= kMaxFeature && f % 64 == 0; }

inline bool tokens_ok(int32_t t) { return t >= 0 && t <= kMaxTokens; }

inline bool heads_ok(int32_t nh, int32_t nkv, int32_t hd) {
    if (nh <= 0 || nkv <= 0 || hd <= 0 || hd % 8 != 0 || nh % nkv != 0) return false;
    if (nh > kMaxFeature / hd) return false;  // the products below would pass 32 bits
    if (!feature_ok(nh * hd) || !feature_ok((nh + 2 * nkv) * hd)) return false;
    return true;
}

// Floats per head row of the attention statistics (lse, rowsum): whole 128-row blocks.
inline int32_t stat_stride(int32_t tokens) { return std::max<int32_t>(128, (tokens + 127) / 128 * 128); }

inline zb_status device_ok() {
    const int arch = device_arch();
    if (arch < 0) return ZB_ERR_CUDA;
    return arch == 103 ? ZB_OK : ZB_ERR_DEVICE;
}

inline zb_status cuda_status(cudaError_t e) { return e == cudaSuccess ? ZB_OK : ZB_ERR_CUDA; }

}  // namespace zbk

#define ZB_TRY(expr)                        \
    do {                                    \
        const zb_status zb_s_ = (expr);     \
        if (zb_s_ != ZB_OK) return zb_s_;   \
    } while (0)
