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
// few: slots -> rows and old scale -> maximum -> stores.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "fd_device.cuh"
#include "fd_internal.h"

namespace fdk {

namespace {

__device__ unsigned int g_status = 0;   // this file's bits of the device status word

constexpr unsigned kFullMask = 0xffffffffu;
constexpr int kStoreWarps = 8;
constexpr int kKeep = 4;                // 16-byte pieces of the rows a lane keeps between the two passes

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

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.f;
}

// the smallest power of two s >= 2^-126 with amax <= 448 s
__device__ __forceinline__ float scale_for(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 126;   // amax = f 2^e, f in [0.5, 1)
    const int k = (u & 0x7fffffu) <= 0x600000u ? e - 9 : e - 8;
    return __uint_as_float(static_cast<uint32_t>(max(k, -126) + 127) << 23);
}

// two values to E4M3, nearest even; infinities and NaN become NaN
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    const float nan = __uint_as_float(0x7fc00000u);
    a = fabsf(a) <= 3.402823466e38f ? a : nan;
    b = fabsf(b) <= 3.402823466e38f ? b : nan;
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

template <typename T>
__device__ __forceinline__ float piece_amax(const uint4& r) {
    const float2 a = unpack2<T>(r.x), b = unpack2<T>(r.y), c = unpack2<T>(r.z), d = unpack2<T>(r.w);
    return fmaxf(fmaxf(fmaxf(finite_abs(a.x), finite_abs(a.y)), fmaxf(finite_abs(b.x), finite_abs(b.y))),
                 fmaxf(fmaxf(finite_abs(c.x), finite_abs(c.y)), fmaxf(finite_abs(d.x), finite_abs(d.y))));
}

template <typename T>
__device__ __forceinline__ uint2 quantise(const uint4& r, const Quotient& q) {
    const float2 a = unpack2<T>(r.x), b = unpack2<T>(r.y), c = unpack2<T>(r.z), d = unpack2<T>(r.w);
    return make_uint2(to_e4m3x2(q(a.x), q(a.y)) | (to_e4m3x2(q(b.x), q(b.y)) << 16),
                      to_e4m3x2(q(c.x), q(c.y)) | (to_e4m3x2(q(d.x), q(d.y)) << 16));
}

// four stored values re-expressed for a scale `ratio` = old / new as large
__device__ __forceinline__ uint32_t requantise(uint32_t w, float ratio) {
    uint32_t out = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const __half2_raw raw = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * h)), __NV_E4M3);
        const float2 f = __half22float2(__half2(raw));
        out |= to_e4m3x2(f.x * ratio, f.y * ratio) << (16 * h);
    }
    return out;
}

// One unit: the `run` rows from row t of the list, which go to one block from
// its row `row0` on, for one head.  W warps share it (w is this warp's number;
// W = 8: the whole CTA, with s_max).  Half a warp takes a row, 8 values a lane.
// at: the unit's slots, null unless rows between its first and last are skipped.
template <typename T, int W>
__device__ __forceinline__ void store_unit(const T* src, int64_t src_t, uint8_t* dst, int64_t dst_t, float* scale,
                                           int row0, int run, const int64_t* at, int w, int lane, float* s_max) {
    const int half = lane >> 4, c = lane & 15;
    auto here = [&](int r) { return r < run && (at == nullptr || at[r] == at[0] + r); };
    const float old = row0 > 0 ? *scale : 0.f;
    const T* from = src + 8 * c;
    uint4 keep[kKeep];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        const int r = 2 * (i * W + w) + half;
        if (here(r)) keep[i] = __ldg(reinterpret_cast<const uint4*>(from + r * src_t));
    }
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
        if (here(2 * (i * W + w) + half)) amax = fmaxf(amax, piece_amax<T>(keep[i]));
#pragma unroll 4
    for (int r = 2 * (kKeep * W + w) + half; r < run; r += 2 * W)
        if (here(r)) amax = fmaxf(amax, piece_amax<T>(__ldg(reinterpret_cast<const uint4*>(from + r * src_t))));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, o));
    if (W > 1) {
        if (lane == 0) s_max[w] = amax;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < W; ++x) amax = fmaxf(amax, s_max[x]);
    }
    const float need = scale_for(amax);
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
    const Quotient q(now);
    uint8_t* to = dst + 8 * c;
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        const int r = 2 * (i * W + w) + half;
        if (here(r)) *reinterpret_cast<uint2*>(to + r * dst_t) = quantise<T>(keep[i], q);
    }
#pragma unroll 4
    for (int r = 2 * (kKeep * W + w) + half; r < run; r += 2 * W)
        if (here(r)) *reinterpret_cast<uint2*>(to + r * dst_t) =
            quantise<T>(__ldg(reinterpret_cast<const uint4*>(from + r * src_t)), q);
}

// Grid (tiles of TILE rows of the list, heads, K and V).  A row begins a unit
// unless the row before it in the list (the last one that is not skipped)
// precedes it in its block at the same distance.  A tile with
// one unit (a prompt's rows) is shared by the CTA's warps, otherwise each warp
// takes units of its own.
template <typename T, int TILE>
__global__ void __launch_bounds__(kStoreWarps * 32) fd_store_kernel(const StoreParams p) {
    __shared__ float s_max[kStoreWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = blockIdx.x * TILE, g = blockIdx.y;
    const StoreSide& sd = p.side[blockIdx.z];
    grid_dependency_trigger();
    grid_dependency_wait();

    const int t = t0 + lane;
    bool start = false;
    if (lane < TILE && t < p.n_tokens) {
        const int64_t s = p.slots[t];
        if (s >= p.n_slots) {
            atomicOr(&g_status, kStatusPageBit);
        } else if (s >= 0) {
            const int row0 = static_cast<int>(s % p.row_tokens) & (p.block - 1);
            start = true;
            for (int d = 1; d <= min(row0, t); ++d) {
                const int64_t before = p.slots[t - d];
                if (before < 0 || before >= p.n_slots) continue;   // skipped
                start = before != s - d;
                break;
            }
        }
    }
    const unsigned starts = __ballot_sync(kFullMask, start);
    if (starts == 0) return;
    const bool alone = __popc(starts) == 1;
    unsigned left = starts;
    for (int u = 0; left != 0; ++u, left &= left - 1) {
        if (!alone && u % kStoreWarps != warp) continue;
        const int tu = t0 + __ffs(left) - 1;
        const int64_t slot = p.slots[tu];
        const int64_t lead = slot / p.row_tokens;
        const int in = static_cast<int>(slot - lead * p.row_tokens);
        const int row0 = in & (p.block - 1);
        const int most = min(min(p.block - row0, p.row_tokens - in), p.n_tokens - tu);
        int run = 1;                            // rows of the list that go on from here in this block
        bool skips = false;
        for (int r = 1; r < most; r += 32) {
            const int64_t s = r + lane < most ? p.slots[tu + r + lane] : slot;
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
        float* scale = sd.scale + lead * sd.scale_b + g * sd.scale_h + (in / p.block) * sd.scale_n;
        if (alone)
            store_unit<T, kStoreWarps>(src, sd.src_t, dst, sd.dst_t, scale, row0, run, skips ? p.slots + tu : nullptr, warp, lane,
                                       s_max);
        else
            store_unit<T, 1>(src, sd.src_t, dst, sd.dst_t, scale, row0, run, skips ? p.slots + tu : nullptr, 0, lane, s_max);
    }
}

template <typename T>
cudaError_t launch_store_t(const StoreParams& p, cudaStream_t stream) {
    constexpr int kTile = 8;
    return launch_pdl(fd_store_kernel<T, kTile>, dim3((p.n_tokens + kTile - 1) / kTile, p.n_kv_heads, 2),
                      dim3(kStoreWarps * 32), 0, stream, p);
}

}  // namespace

cudaError_t launch_store(const StoreParams& p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_store_t<__nv_bfloat16>(p, stream) : launch_store_t<__half>(p, stream);
}

cudaError_t status_store(unsigned* value, bool clear) { return read_status_word(g_status, value, clear); }

}  // namespace fdk
