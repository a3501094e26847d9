// fd_copy.cu -- pages copied within the pools of every layer (fd_page_copy).
//
// Bound by HBM: each byte is read once and written once.  Work is dealt in pieces
// of a page of a pool; the list's length is read on the GPU.  Rows of 8 KB and
// more of 16-byte units go by bulk copies through shared memory (500 pages of 32 KB in 64
// pools, 2.1 GB: 320 us, 6.6 TB/s, 97 % of a plain copy's rate; by registers 330), all others
// by registers.
//
// Pools of several shapes are a launch each, and every launch waits for the one before
// it before its first read: what wrote the list and the pages is visible to a grid
// only by a wait of its own, so none may rely on that of the call's first launch.
// (12 pages of 64 KB in 32 pools and the scales of 32 more: 12.6 us; 10.8 without that wait.)
#include "../../include/fd.h"
#include "fd_device.cuh"
#include "fd_internal.h"

namespace fdk {

namespace {

__device__ unsigned int g_status = 0;   // this file's bits of the device status word

constexpr int kCopyThreads = 256;
constexpr int kAhead = 4;               // loads of a thread in flight
// Bulk copies: bytes at a time, stages of a CTA, loads among them, CTAs per SM.  16 KB,
// 6 stages, 3 loads, 2 CTAs 319.6 us; 12 / 8 / 1 324.6; 32 KB, 6 / 3 / 1 320.8; 8 KB, 6 / 3 / 4
// 322.3, 24 / 12 / 1 540 (one thread issues too slowly); 4 KB, 12 / 6 / 4 333.
constexpr int kPiece = 16384, kStages = 6, kAheadLoads = 3, kBulkCtas = 2;
// Shorter rows by registers: a thread asks for one piece in about 0.3 us.  250 pages of 32 KB in 32
// pools, as rows of 2 / 4 / 8 KB apart from each other, us: bulk 265 / 138 / 82, registers 87 / 86 / 86.
constexpr int kBulkRow = 8192;

// U: the unit that a thread moves.  A page is extent0 x extent1 rows of `per_row` units;
// 2^TEAM threads take up to kAhead units each of it at a time.
template <typename U, int TEAM>
__global__ void __launch_bounds__(kCopyThreads) fd_page_copy_kernel(const CopyParams p, int64_t page_units, int chunks) {
    grid_dependency_trigger();
    grid_dependency_wait();
    const int n = p.count != nullptr ? min(max(*p.count, 0), p.n_pairs) : p.n_pairs;
    const int64_t items = static_cast<int64_t>(n) * p.n_pools * chunks;
    const int64_t per_row = p.row_bytes / static_cast<int64_t>(sizeof(U));
    const bool flat = p.extent0 == 1 && p.extent1 == 1;
    constexpr int kTeams = kCopyThreads >> TEAM, kTeam = 1 << TEAM;
    const int me = threadIdx.x & (kTeam - 1);
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * kTeams + (threadIdx.x >> TEAM); item < items;
         item += static_cast<int64_t>(gridDim.x) * kTeams) {
        const int64_t pp = item / chunks;
        const int chunk = static_cast<int>(item - pp * chunks);
        const int pair = static_cast<int>(pp / p.n_pools), pool = static_cast<int>(pp - static_cast<int64_t>(pair) * p.n_pools);
        const int src = p.src[pair], dst = p.dst[pair];
        if (src < 0 || dst < 0 || src == dst) continue;
        if (src >= p.n_pages || dst >= p.n_pages) {
            if (me == 0) atomicOr(&g_status, kStatusPageBit);
            continue;
        }
        const char* from = p.base[pool] + src * p.page_stride;
        char* to = p.base[pool] + dst * p.page_stride;
        const int64_t u0 = static_cast<int64_t>(chunk) * (kAhead * kTeam) + me;
        U v[kAhead];
        int64_t at[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t u = u0 + k * kTeam;
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
            if (u0 + k * kTeam < page_units) *reinterpret_cast<U*>(to + at[k]) = v[k];
    }
}

// One thread a CTA asks for pieces of up to kPiece bytes of a row and sends them
// on from shared memory, kAheadLoads loads and the other stages' stores in flight.
__global__ void __launch_bounds__(32) fd_page_bulk_kernel(const __grid_constant__ CopyParams p, int pieces) {
    extern __shared__ __align__(128) unsigned char s_stage[];    // [kStages][kPiece]
    __shared__ __align__(8) uint64_t s_bar[kStages];
    const uint32_t stages = smem_u32(s_stage), bars = smem_u32(s_bar);
    if (threadIdx.x != 0) return;
    for (int s = 0; s < kStages; ++s) mbar_init(bars + 8 * s, 1);
    fence_barrier_init();
    grid_dependency_trigger();
    grid_dependency_wait();
    const int n = p.count != nullptr ? min(max(*p.count, 0), p.n_pairs) : p.n_pairs;
    const int64_t per_page = static_cast<int64_t>(p.extent0) * p.extent1 * pieces;
    const int64_t items = static_cast<int64_t>(n) * p.n_pools * per_page;

    char* to[kStages];                  // of the pieces in the stages (unrolled: registers)
    int bytes[kStages];                 // 0: none
    int64_t item = blockIdx.x;
    // asks for the next piece of a pair that counts, if there is one left
    auto load = [&](int s, char*& where, int& size) {
        size = 0;
        for (; item < items && size == 0; item += gridDim.x) {
            const int64_t pp = item / per_page, in_page = item - pp * per_page;
            const int pair = static_cast<int>(pp / p.n_pools), pool = static_cast<int>(pp - static_cast<int64_t>(pair) * p.n_pools);
            const int src = p.src[pair], dst = p.dst[pair];
            if (src < 0 || dst < 0 || src == dst) continue;
            if (src >= p.n_pages || dst >= p.n_pages) {
                atomicOr(&g_status, kStatusPageBit);
                continue;
            }
            const int64_t row = in_page / pieces, piece = in_page - row * pieces;
            const int64_t i = row / p.extent1, j = row - i * p.extent1;
            const int64_t at = i * p.stride0 + j * p.stride1 + piece * kPiece;
            size = static_cast<int>(min(static_cast<int64_t>(kPiece), p.row_bytes - piece * kPiece));
            where = p.base[pool] + dst * p.page_stride + at;
            mbar_arrive_expect_tx(bars + 8 * s, size);
            bulk_load(stages + s * kPiece, p.base[pool] + src * p.page_stride + at, size, bars + 8 * s);
        }
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) bytes[s] = 0;
#pragma unroll
    for (int s = 0; s < kAheadLoads; ++s) load(s, to[s], bytes[s]);
    bool late = false;                  // a wait ran out: nothing more is asked for or sent
    int phase = 0;
    for (bool more = true; more; phase ^= 1) {
#pragma unroll
        for (int s = 0; s < kStages; ++s) {
            bulk_wait_read<kStages - kAheadLoads - 1>();    // the stage that the next load goes to has been sent
            constexpr int kTurn = kAheadLoads;
            const int ahead = (s + kTurn) % kStages;
            if (late) bytes[ahead] = 0;
            else load(ahead, to[ahead], bytes[ahead]);
            if (bytes[s] == 0) {
                more = false;           // (and none behind it)
                break;
            }
            if (!mbar_wait(bars + 8 * s, phase)) late = true;
            if (late) continue;         // (the loads behind it are waited for all the same)
            bulk_store(to[s], stages + s * kPiece, bytes[s]);
            bulk_commit();
        }
    }
    if (late) atomicOr(&g_status, kStatusTimeoutBit);
    bulk_wait<0>();
}

cudaError_t launch_copy_bulk(const CopyParams& p, cudaStream_t stream) {
    const int sms = fd_num_sms(-1);
    if (sms < 1) return cudaErrorInvalidDevice;
    static std::atomic<unsigned long long> configured_ctx{0};
    const cudaError_t e = allow_smem(fd_page_bulk_kernel, kStages * kPiece, configured_ctx);
    if (e != cudaSuccess) return e;
    const int64_t pieces = (p.row_bytes + kPiece - 1) / kPiece;
    if (pieces > INT32_MAX) return cudaErrorInvalidValue;
    const int64_t items = pieces * p.extent0 * p.extent1 * p.n_pools * p.n_pairs, most = static_cast<int64_t>(sms) * kBulkCtas;
    return launch_pdl(fd_page_bulk_kernel, dim3(static_cast<unsigned>(items < most ? items : most)), dim3(32), kStages * kPiece, stream,
                      p, static_cast<int>(pieces));
}

template <typename U, int TEAM>
cudaError_t launch_copy_team(const CopyParams& p, int64_t units, cudaStream_t stream) {
    constexpr int64_t kTeams = kCopyThreads >> TEAM, kChunk = kAhead << TEAM;
    const int64_t chunks = (units + kChunk - 1) / kChunk;
    if (chunks > INT32_MAX) return cudaErrorInvalidValue;
    const int sms = fd_num_sms(-1);
    if (sms < 1) return cudaErrorInvalidDevice;
    const int64_t ctas = (chunks * p.n_pools * p.n_pairs + kTeams - 1) / kTeams, most = static_cast<int64_t>(sms) * 8;
    return launch_pdl(fd_page_copy_kernel<U, TEAM>, dim3(static_cast<unsigned>(ctas < most ? ctas : most)), dim3(kCopyThreads), 0,
                      stream, p, units, static_cast<int>(chunks));
}

template <typename U>
cudaError_t launch_copy_u(const CopyParams& p, cudaStream_t stream) {
    // A page gets as many threads, whole warps, as it has kAhead units for.  8.2 MB of pages
    // of 1 / 2 / 4 KB in each of 32 pools, us: 430 / 219 / 130 with 256 threads a page, 90 / 86 / 84 so.
    const int64_t units = static_cast<int64_t>(p.extent0) * p.extent1 * (p.row_bytes / static_cast<int64_t>(sizeof(U)));
    if (units <= kAhead << 5) return launch_copy_team<U, 5>(p, units, stream);
    if (units <= kAhead << 6) return launch_copy_team<U, 6>(p, units, stream);
    return launch_copy_team<U, 8>(p, units, stream);
}

}  // namespace

cudaError_t launch_page_copy(const CopyParams& p, cudaStream_t stream) {
    if (p.unit == 16 && p.row_bytes >= kBulkRow) return launch_copy_bulk(p, stream);
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
