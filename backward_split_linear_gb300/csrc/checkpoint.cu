// Packing activations into 8 bits, and back.  The format is checkpoint.cuh's.
#include "chained.cuh"
#include "checkpoint.cuh"
#include "checks.h"
#include "operators.h"

namespace zbk {

namespace {

constexpr int kPackThreads = 256;

// Two threads a block of 32: each loads 16 elements (two 16-byte words), the larger of
// their largest magnitudes gives the scale.  Bound by HBM.
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const uint16_t* x, uint8_t* codes, uint8_t* scales, int64_t halves) {
    release_next();
    wait_for_previous();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kPackThreads + threadIdx.x;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (i < halves) {
        a = reinterpret_cast<const uint4*>(x)[2 * i];
        b = reinterpret_cast<const uint4*>(x)[2 * i + 1];
    }
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t top2 = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top2 = pack_top2(top2, w[e]);
    uint32_t top = pack_top(top2);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    if (i >= halves) return;
    const uint32_t scale = pack_scale(top);
    const uint32_t f = pack_factor(scale);
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        c[e] = top < kPackLargest ? pack_codes(w[2 * e], w[2 * e + 1], f) : pack_codes_slow(w[2 * e], w[2 * e + 1], f, scale);
    reinterpret_cast<uint4*>(codes)[i] = make_uint4(c[0], c[1], c[2], c[3]);
    if ((threadIdx.x & 1) == 0) scales[i >> 1] = static_cast<uint8_t>(scale);
}

// 16 elements a thread.  Bound by HBM.
__global__ void __launch_bounds__(kPackThreads) unpack_kernel(const uint8_t* codes, const uint8_t* scales, uint16_t* x,
                                                              int64_t halves) {
    release_next();
    wait_for_previous();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kPackThreads + threadIdx.x;
    if (i >= halves) return;
    const uint4 cv = reinterpret_cast<const uint4*>(codes)[i];
    const uint32_t unit = unpack_unit(scales[i >> 1]);
    const uint32_t c[4] = {cv.x, cv.y, cv.z, cv.w};
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        w[2 * e] = unpack_pair<0>(c[e], unit);
        w[2 * e + 1] = unpack_pair<1>(c[e], unit);
    }
    reinterpret_cast<uint4*>(x)[2 * i] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(x)[2 * i + 1] = make_uint4(w[4], w[5], w[6], w[7]);
}

bool halves_of(int tokens, int width, int64_t* halves, unsigned* grid) {
    *halves = static_cast<int64_t>(tokens) * (width / 16);
    const int64_t blocks = (*halves + kPackThreads - 1) / kPackThreads;
    *grid = static_cast<unsigned>(blocks);
    return blocks <= 0x7fffffff;
}

}  // namespace

cudaError_t launch_unpack(const void* codes, const void* scales, void* x, int tokens, int width, cudaStream_t stream) {
    int64_t halves;
    unsigned grid;
    if (!halves_of(tokens, width, &halves, &grid)) return cudaErrorInvalidValue;
    return launch_chained(unpack_kernel, grid, kPackThreads, 0, stream, static_cast<const uint8_t*>(codes),
                          static_cast<const uint8_t*>(scales), static_cast<uint16_t*>(x), halves);
}

}  // namespace zbk

extern "C" zb_status zb_op_checkpoint_pack(const void* x, const zb_checkpoint* packed, int32_t tokens, int32_t width,
                                           void* stream) {
    using namespace zbk;
    int64_t halves;
    unsigned grid;
    if (!tokens_ok(tokens) || !feature_ok(width) || !halves_of(tokens, width, &halves, &grid)) return ZB_ERR_SHAPE;
    if (!packed || !rows_ok(x, tokens) || !rows_ok(packed->codes, tokens) || !rows_ok(packed->scales, tokens))
        return ZB_ERR_ARG;
    ZB_TRY(device_ok());
    if (tokens == 0) return ZB_OK;
    return cuda_status(launch_chained(pack_kernel, grid, kPackThreads, 0, as_stream(stream), static_cast<const uint16_t*>(x),
                                      static_cast<uint8_t*>(packed->codes), static_cast<uint8_t*>(packed->scales), halves));
}

extern "C" zb_status zb_op_checkpoint_unpack(const zb_checkpoint* packed, void* x, int32_t tokens, int32_t width,
                                             void* stream) {
    using namespace zbk;
    int64_t halves;
    unsigned grid;
    if (!tokens_ok(tokens) || !feature_ok(width) || !halves_of(tokens, width, &halves, &grid)) return ZB_ERR_SHAPE;
    if (!packed || !rows_ok(x, tokens) || !rows_ok(packed->codes, tokens) || !rows_ok(packed->scales, tokens))
        return ZB_ERR_ARG;
    ZB_TRY(device_ok());
    if (tokens == 0) return ZB_OK;
    return cuda_status(launch_unpack(packed->codes, packed->scales, x, tokens, width, as_stream(stream)));
}
