// fd_copy.cu -- pages copied within the pools of every layer (fd_page_copy).
//
// Bound by HBM: each byte is read once and written once.  Work is dealt in chunks
// of a page of a pool; the list's length is read on the GPU.
#include "../../include/fd.h"
#include "fd_device.cuh"
#include "fd_internal.h"

namespace fdk {

namespace {

__device__ unsigned int g_status = 0;   // this file's bits of the device status word

constexpr int kCopyThreads = 256;
constexpr int kAhead = 4;               // loads of a thread in flight

// U: the unit that a thread moves.  A page is extent0 x extent1 rows of `per_row` units.
template <typename U>
__global__ void __launch_bounds__(kCopyThreads) fd_page_copy_kernel(const CopyParams p, int64_t page_units, int chunks) {
    grid_dependency_trigger();
    grid_dependency_wait();
    const int n = p.count != nullptr ? min(max(*p.count, 0), p.n_pairs) : p.n_pairs;
    const int64_t items = static_cast<int64_t>(n) * p.n_pools * chunks;
    const int64_t per_row = p.row_bytes / static_cast<int64_t>(sizeof(U));
    const bool flat = p.extent0 == 1 && p.extent1 == 1;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t pp = item / chunks;
        const int chunk = static_cast<int>(item - pp * chunks);
        const int pair = static_cast<int>(pp / p.n_pools), pool = static_cast<int>(pp - static_cast<int64_t>(pair) * p.n_pools);
        const int src = p.src[pair], dst = p.dst[pair];
        if (src < 0 || dst < 0 || src == dst) continue;
        if (src >= p.n_pages || dst >= p.n_pages) {
            if (threadIdx.x == 0) atomicOr(&g_status, kStatusPageBit);
            continue;
        }
        const char* from = p.base[pool] + src * p.page_stride;
        char* to = p.base[pool] + dst * p.page_stride;
        const int64_t u0 = static_cast<int64_t>(chunk) * (kCopyThreads * kAhead) + threadIdx.x;
        U v[kAhead];
        int64_t at[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t u = u0 + k * kCopyThreads;
            if (u >= page_units) continue;
            if (flat) {
                at[k] = u * static_cast<int64_t>(sizeof(U));
            } else {
                const int64_t row = u / per_row;
                const int i = static_cast<int>(row / p.extent1), j = static_cast<int>(row - static_cast<int64_t>(i) * p.extent1);
                at[k] = i * p.stride0 + j * p.stride1 + (u - row * per_row) * static_cast<int64_t>(sizeof(U));
            }
            v[k] = *reinterpret_cast<const U*>(from + at[k]);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (u0 + k * kCopyThreads < page_units) *reinterpret_cast<U*>(to + at[k]) = v[k];
    }
}

template <typename U>
cudaError_t launch_copy_u(const CopyParams& p, cudaStream_t stream) {
    const int64_t units = static_cast<int64_t>(p.extent0) * p.extent1 * (p.row_bytes / static_cast<int64_t>(sizeof(U)));
    const int64_t chunks = (units + kCopyThreads * kAhead - 1) / (kCopyThreads * kAhead);
    if (chunks > INT32_MAX) return cudaErrorInvalidValue;
    const int sms = fd_num_sms(-1);
    if (sms < 1) return cudaErrorInvalidDevice;
    const int64_t items = chunks * p.n_pools * p.n_pairs, most = static_cast<int64_t>(sms) * 8;
    return launch_pdl(fd_page_copy_kernel<U>, dim3(static_cast<unsigned>(items < most ? items : most)), dim3(kCopyThreads), 0,
                      stream, p, units, static_cast<int>(chunks));
}

}  // namespace

cudaError_t launch_page_copy(const CopyParams& p, cudaStream_t stream) {
    switch (p.unit) {
        case 16: return launch_copy_u<uint4>(p, stream);
        case 8: return launch_copy_u<uint2>(p, stream);
        case 4: return launch_copy_u<uint32_t>(p, stream);
        case 2: return launch_copy_u<uint16_t>(p, stream);
        default: return launch_copy_u<uint8_t>(p, stream);
    }
}

cudaError_t status_word_copy(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_status);
}

}  // namespace fdk
