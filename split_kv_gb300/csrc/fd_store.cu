// fd_store.cu -- new K/V rows into an E4M3 cache with one power-of-two scale
// per (block of tokens, KV head) (fd_cache_store).
//
// For the new rows x of one (block, head): amax = max |x|, the scale they need
// is the smallest power of two s with amax <= 448 s, i.e. with amax = f 2^e,
// f in [0.5, 1): 448 = 0.875 * 2^9, so s = 2^(e - 9) if f <= 0.875, else
// 2^(e - 8).  A stored value is round(x / s) to E4M3.  Powers of two cost no
// precision in a floating format (at most one bit of range), make x / s exact,
// so that every value is rounded once, and let a block whose scale grows be
// rewritten without loss (a second rounding only among subnormals).
//
// Bound by HBM for many rows (2 bytes in, 1 out per value) and by latency for
// few: slots -> rows and old scale -> maximum -> stores.  10194 rows of 8 heads
// (62.7 MB): 20 us, 3.1 TB/s; 64 single rows: 3.4 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <initializer_list>
#include <type_traits>

#include "fd_device.cuh"
#include "fd_internal.h"

namespace fdk {

namespace {

__device__ unsigned int g_status = 0;   // this file's bits of the device status word

constexpr unsigned kFullMask = 0xffffffffu;
constexpr int kStoreWarps = 8;
constexpr int kKeep = 8;                // 16-byte pieces of the rows a lane keeps between the two passes

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    __half2 h;
    memcpy(&h, &w, 4);
    return __half22float2(h);
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// the smallest power of two s >= 2^-126 with amax <= 448 s
__device__ __forceinline__ float scale_for(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 126;   // amax = f 2^e, f in [0.5, 1)
    const int k = (u & 0x7fffffu) <= 0x600000u ? e - 9 : e - 8;
    return __uint_as_float(static_cast<uint32_t>(max(k, -126) + 127) << 23);
}

// two values to E4M3, nearest even; NaN stays NaN, and with SPECIAL infinities
// become NaN (the conversion would make them 448)
template <bool SPECIAL>
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    if constexpr (SPECIAL) {
        const float nan = __uint_as_float(0x7fc00000u);
        a = fabsf(a) <= 3.402823466e38f ? a : nan;
        b = fabsf(b) <= 3.402823466e38f ? b : nan;
    }
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Quotient by s: exact through the reciprocal where s is a power of two (the
// scales this file writes), a division for a scale of another origin.
struct Quotient {
    float s, inv;
    bool pow2;
    __device__ __forceinline__ explicit Quotient(float scale) : s(scale) {
        const uint32_t u = __float_as_uint(scale);
        pow2 = (u & 0x7fffffu) == 0 && u >= 0x00800000u && u < 0x7f000000u;
        inv = __uint_as_float(0x7f000000u - u);
    }
    __device__ __forceinline__ float operator()(float x) const { return pow2 ? x * inv : __fdiv_rn(x, s); }
};

struct Reciprocal {
    float inv;
    __device__ __forceinline__ float operator()(float x) const { return x * inv; }
};

// Patterns of infinity; a larger one with the sign cleared is a NaN.
template <typename T>
constexpr uint32_t kInfBits = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;

// The larger magnitudes, as patterns: those of 16-bit floats order like integers.
__device__ __forceinline__ uint32_t max_bits(uint32_t m, const uint4& r) {
    constexpr uint32_t abs2 = 0x7fff7fffu;
    return __vmaxu2(__vmaxu2(__vmaxu2(r.x & abs2, r.y & abs2), __vmaxu2(r.z & abs2, r.w & abs2)), m);
}

// The same without infinities and NaN.
template <typename T>
__device__ __forceinline__ uint32_t finite_max_bits(uint32_t m, const uint4& r) {
    for (const uint32_t w : {r.x, r.y, r.z, r.w})
        for (const uint32_t x : {w & 0x7fffu, (w >> 16) & 0x7fffu})
            if (x < kInfBits<T>) m = max(m, x);
    return m;
}

template <typename T, bool SPECIAL, typename Q>
__device__ __forceinline__ uint2 quantise(const uint4& r, const Q& q) {
    const float2 a = unpack2<T>(r.x), b = unpack2<T>(r.y), c = unpack2<T>(r.z), d = unpack2<T>(r.w);
    return make_uint2(to_e4m3x2<SPECIAL>(q(a.x), q(a.y)) | (to_e4m3x2<SPECIAL>(q(b.x), q(b.y)) << 16),
                      to_e4m3x2<SPECIAL>(q(c.x), q(c.y)) | (to_e4m3x2<SPECIAL>(q(d.x), q(d.y)) << 16));
}

// four stored values re-expressed for a scale `ratio` = old / new as large
__device__ __forceinline__ uint32_t requantise(uint32_t w, float ratio) {
    uint32_t out = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const __half2_raw raw = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * h)), __NV_E4M3);
        const float2 f = __half22float2(__half2(raw));
        out |= to_e4m3x2<true>(f.x * ratio, f.y * ratio) << (16 * h);
    }
    return out;
}

// Row r of an item: whether the list has it (a skipped row leaves its place).
__device__ __forceinline__ bool has_row(const int64_t* at, int r) { return at == nullptr || at[r] == at[0] + r; }

// The stores of an item with infinities or NaN, skipped rows or a scale that is
// no power of two: rare, so compact rather than fast.
template <typename T>
__device__ __noinline__ void store_rows_any(const T* from, int64_t src_t, uint8_t* to, int64_t dst_t, int run,
                                            const int64_t* at, int r, int r_step, float now) {
    const Quotient q(now);
#pragma unroll 1
    for (; r < run; r += r_step)
        if (has_row(at, r))
            *reinterpret_cast<uint2*>(to + r * dst_t) =
                quantise<T, true>(__ldg(reinterpret_cast<const uint4*>(from + r * src_t)), q);
}

template <typename T>
__device__ __noinline__ uint32_t max_rows_any(const T* from, int64_t src_t, int run, const int64_t* at, int r, int r_step) {
    uint32_t m = 0;
#pragma unroll 1
    for (; r < run; r += r_step)
        if (has_row(at, r)) m = finite_max_bits<T>(m, __ldg(reinterpret_cast<const uint4*>(from + r * src_t)));
    return m;
}

// The largest of W warps' values (the same W for every warp of the CTA).
__device__ __forceinline__ uint32_t share_max(uint32_t m, int W, int w, int lane, uint32_t* s_max, int base) {
    m = __reduce_max_sync(kFullMask, m);
    if (W > 1) {
        __syncthreads();
        if (lane == 0) s_max[base + w] = m;
        __syncthreads();
        for (int x = 0; x < W; ++x) m = max(m, s_max[base + x]);
    }
    return m;
}

// One item: the `run` rows from one row of the list on, which go to one block
// from its row `row0` on, for one head.  W warps share it, this is number w;
// with W > 1 every warp of the CTA makes the call (the item's part of s_max is
// [base, base + W); run = 0: no rows, only the barriers).  Half a warp takes a
// row, 8 values a lane; up to kKeep pieces stay in registers between the pass
// for the maximum and the one that stores, the rest is read again (from the caches).
// at: the item's slots, null unless rows between its first and last are skipped.
template <typename T>
__device__ __forceinline__ void store_item(const T* src, int64_t src_t, uint8_t* dst, int64_t dst_t, float* scale,
                                           int row0, int run, const int64_t* at, int W, int w, int lane, uint32_t* s_max,
                                           int base) {
    const int c = lane & 15;
    const T* from = src + 8 * c;
    const int r_first = 2 * w + (lane >> 4), r_step = 2 * W;
    const T* first = from + r_first * src_t;
    const int64_t src_step = r_step * src_t;
    uint4 keep[kKeep];
    float old = 0.f;
    if (row0 > 0 && run > 0) old = *scale;
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
        keep[i] = r_first + i * r_step < run ? __ldg(reinterpret_cast<const uint4*>(first + i * src_step))
                                             : make_uint4(0u, 0u, 0u, 0u);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kKeep; ++i) m = max_bits(m, keep[i]);
#pragma unroll 4
    for (int r = r_first + kKeep * r_step; r < run; r += r_step)
        m = max_bits(m, __ldg(reinterpret_cast<const uint4*>(from + r * src_t)));
    m = share_max(max(m & 0xffffu, m >> 16), W, w, lane, s_max, base);
    // rare: infinities, NaN or skipped rows, whose values have no part
    const bool any_special = m >= kInfBits<T> || at != nullptr;
    bool again = any_special;
    if (W > 1) again = __syncthreads_or(any_special);
    if (again) {
        const uint32_t f = share_max(max_rows_any<T>(from, src_t, run, at, r_first, r_step), W, w, lane, s_max, base);
        if (any_special) m = f;
    }
    if (run == 0) return;
    const float need = scale_for(unpack2<T>(m).x);
    const float now = row0 > 0 ? fmaxf(old, need) : need;
    if (row0 > 0 && now != old) {
        // rows before the new ones, 16 bytes a lane, four rows a warp
        const float ratio = __fdiv_rn(old, now);
        for (int r = 4 * w + (lane >> 3); r < row0; r += 4 * W) {
            uint4* piece = reinterpret_cast<uint4*>(dst + (r - row0) * dst_t) + (lane & 7);
            uint4 v = *piece;
            v.x = requantise(v.x, ratio);
            v.y = requantise(v.y, ratio);
            v.z = requantise(v.z, ratio);
            v.w = requantise(v.w, ratio);
            *piece = v;
        }
    }
    if (w == 0 && lane == 0 && now != old) *scale = now;
    uint8_t* to = dst + 8 * c;
    const Quotient q(now);
    if (any_special || !q.pow2) {
        store_rows_any<T>(from, src_t, to, dst_t, run, at, r_first, r_step, now);
        return;
    }
    const Reciprocal inv{q.inv};
    uint8_t* to_first = to + r_first * dst_t;
    const int64_t dst_step = r_step * dst_t;
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
        if (r_first + i * r_step < run)
            *reinterpret_cast<uint2*>(to_first + i * dst_step) = quantise<T, false>(keep[i], inv);
#pragma unroll 4
    for (int r = r_first + kKeep * r_step; r < run; r += r_step)
        *reinterpret_cast<uint2*>(to + r * dst_t) =
            quantise<T, false>(__ldg(reinterpret_cast<const uint4*>(from + r * src_t)), inv);
}

// Grid (tiles of TILE rows of the list, groups of kHeads heads, K and V).  A row
// begins a unit unless the row before it in the list (the last one that is not
// skipped) precedes it in its block at the same distance; the tile's units
// times its heads are the CTA's items.  Items of more than kLong rows (a
// prompt's) are shared by as many warps as keep all their rows in registers,
// then the short ones (a step's) are taken by a warp each, in turn.  The slots
// of the tile and of the rows that its last unit may go on with are read once
// into shared memory, so that the chain is slots -> rows and old scale -> stores.
// (Heads per CTA 1 / 2 / 4 / 8: 10194 prompt rows of 8 heads 26.2 / 20.2 / 23.9 / 32.2 us,
// 256 single rows 6.7 / 5.0 / 5.7 / 9.1, 64 2.9 / 3.4 / 4.2 / 6.5.)
constexpr int kHeads = 2;
constexpr int kAhead = 256;             // slots in shared memory
constexpr int kLong = 2 * kKeep;        // rows that one warp keeps

template <typename T, int TILE>
__global__ void __launch_bounds__(kStoreWarps * 32, 3) fd_store_kernel(const StoreParams p) {
    static_assert(kAhead == kStoreWarps * 32 && TILE <= kAhead, "one slot a thread");
    constexpr int kMaskWords = (TILE + 31) / 32;
    __shared__ int64_t s_slot[kAhead];
    __shared__ unsigned s_starts[2][kStoreWarps];   // short units, long ones
    __shared__ uint32_t s_max[kStoreWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = blockIdx.x * TILE, g0 = blockIdx.y * kHeads;
    const StoreSide& sd = p.side[blockIdx.z];
    grid_dependency_trigger();
    grid_dependency_wait();

    auto in_row = [&](int64_t s) {       // token within the page or sequence
        return static_cast<int>(p.row_shift >= 0 ? s & (p.row_tokens - 1) : s % p.row_tokens);
    };
    const int t = t0 + tid;
    const bool mine = tid < TILE && t < p.n_tokens;
    const int64_t before = mine && t > 0 ? p.slots[t - 1] : -1;
    const int64_t slot_t = t < p.n_tokens ? p.slots[t] : -1;
    s_slot[tid] = slot_t;
    bool start = false;
    if (mine && slot_t >= p.n_slots) {
        atomicOr(&g_status, kStatusPageBit);
    } else if (mine && slot_t >= 0) {
        const int back = min(in_row(slot_t) & (p.block - 1), t);
        start = true;
        if (back > 0) {
            int64_t b = before;
            int d = 1;
            while ((b < 0 || b >= p.n_slots) && d < back) b = p.slots[t - ++d];   // skipped rows
            start = b != slot_t - d;
        }
    }
    __syncthreads();
    const bool is_long = start && tid + kLong < kAhead && s_slot[tid + kLong] == slot_t + kLong &&
                         (in_row(slot_t) & (p.block - 1)) + kLong < p.block;
    const unsigned shorts = __ballot_sync(kFullMask, start && !is_long), longs = __ballot_sync(kFullMask, is_long);
    if (lane == 0) {
        s_starts[0][warp] = shorts;
        s_starts[1][warp] = longs;
    }
    if (!__syncthreads_or(start)) return;
    auto slot_at = [&](int i) {          // of list row t0 + i (inside the list)
        return i < kAhead ? s_slot[i] : p.slots[t0 + i];
    };
    const int heads = min(kHeads, p.n_kv_heads - g0);
    auto process = [&](const unsigned* starts, int W) {
        unsigned mask[kMaskWords];
        int items = 0;
#pragma unroll
        for (int i = 0; i < kMaskWords; ++i) {
            mask[i] = starts[i];
            items += __popc(mask[i]) * heads;
        }
        const int sets = kStoreWarps / W, set = warp / W;
        for (int first = 0; first < items; first += sets) {
            const int item = first + set;
            const bool any = item < items;
            if (W == 1 && !any) break;
            int u = any ? item / heads : 0;
            const int g = g0 + (any ? item - u * heads : 0);
            int iu = 0;                             // the tile's u-th unit
#pragma unroll
            for (int i = 0; i < kMaskWords; ++i) {
                const int n = __popc(mask[i]);
                if (u >= 0 && u < n) {
                    unsigned m = mask[i];
                    for (; u > 0; --u) m &= m - 1;
                    iu = 32 * i + __ffs(m) - 1;
                    u = -1;
                } else {
                    u -= u >= 0 ? n : 0;
                }
            }
            const int tu = t0 + iu;
            const int64_t slot = s_slot[iu];
            const int in = in_row(slot);
            const int64_t lead = p.row_shift >= 0 ? slot >> p.row_shift : slot / p.row_tokens;
            const int row0 = in & (p.block - 1);
            const int most = min(min(p.block - row0, p.row_tokens - in), p.n_tokens - tu);
            int run = 1;                            // rows of the list that go on from here in this block
            bool skips = false;
            for (int r = 1; r < most; r += 32) {
                const int64_t s = r + lane < most ? slot_at(iu + r + lane) : slot;
                const bool on = s == slot + r + lane;
                const bool skip = s < 0 || s >= p.n_slots;
                const unsigned go = __ballot_sync(kFullMask, on), stop = __ballot_sync(kFullMask, !on && !skip);
                const unsigned in_run = stop == 0 ? kFullMask : (1u << (__ffs(stop) - 1)) - 1u;
                if ((go & in_run) != 0) {
                    const int upto = r + 32 - __clz(go & in_run);
                    skips |= upto - run != __popc(go & in_run);
                    run = upto;
                }
                if (stop != 0) break;
            }
            const T* src = static_cast<const T*>(sd.src) + tu * sd.src_t + g * sd.src_h;
            uint8_t* dst = sd.dst + lead * sd.dst_b + g * sd.dst_h + in * sd.dst_t;
            float* scale = sd.scale + lead * sd.scale_b + g * sd.scale_h + (in >> p.block_shift) * sd.scale_n;
            store_item<T>(src, sd.src_t, dst, sd.dst_t, scale, row0, any ? run : 0, any && skips ? p.slots + tu : nullptr, W,
                          warp % W, lane, s_max, set * W);
        }
    };
    process(s_starts[1], p.block >= 8 * kLong ? 8 : p.block >= 4 * kLong ? 4 : 2);
    process(s_starts[0], 1);
}

template <typename T, int TILE>
cudaError_t launch_store_tile(const StoreParams& p, cudaStream_t stream) {
    return launch_pdl(fd_store_kernel<T, TILE>,
                      dim3((p.n_tokens + TILE - 1) / TILE, (p.n_kv_heads + kHeads - 1) / kHeads, 2),
                      dim3(kStoreWarps * 32), 0, stream, p);
}

template <typename T>
cudaError_t launch_store_t(const StoreParams& p, cudaStream_t stream) {
    // Rows of the list per CTA.  Single rows of many requests (a decode step) are
    // a unit each, so that small tiles keep a warp to few items; a prompt's rows
    // are few units, of which large tiles leave hardly a CTA without one.  From
    // rows alone the two cannot be told apart, and the first lose more.  8 heads,
    // tiles of 4 / 8 / 64: 256 single rows 5.0 / 5.7 / 23.3 us, of one prompt 3.3 /
    // 3.0 / 3.1 (blocks of 16); 400: 6.3 / 5.8 / 23.6, 3.7 / 3.0 / 3.2; 1024: 13.3 /
    // 12.4 / 35.5, 6.2 / 4.8 / 4.2; 4000 of one prompt 18.5 / 12.9 / 6.5.
    if (p.n_tokens <= 256) return launch_store_tile<T, 4>(p, stream);
    if (p.n_tokens <= 1024) return launch_store_tile<T, 8>(p, stream);
    return launch_store_tile<T, 64>(p, stream);
}

}  // namespace

cudaError_t launch_store(const StoreParams& p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_store_t<__nv_bfloat16>(p, stream) : launch_store_t<__half>(p, stream);
}

cudaError_t status_word_store(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_status);
}

}  // namespace fdk
