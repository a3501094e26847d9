// fd_rope.cu -- norms and rotation of a step's queries and keys, head by head,
// and the way of its keys and values into a cache (fd_qkv_rope).
//
// For a row x of 128:  n = x (sum x^2 / 128 + eps)^-1/2 w, then each pair (a, b) of
// its first rot_dim elements is turned by the angle position * inv_freq_i.
//
// Eight lanes hold a row, 16 elements each in two pieces of 16 bytes, chosen so
// that both elements of every pair are in one lane: for pairs (i, i + rot/2)
// pieces l and l + rot/16, for pairs (2i, 2i + 1) any two.  So the rotation needs
// no exchange and the norm three shuffles; a warp takes four rows at a time,
// each a whole 256 bytes.
//
// Angles: a turn is 2^64.  inv_freq / 2 pi is made a 64-bit fraction once per
// thread (24 bits of inv_freq times 2^64 / 2 pi, shifted), position times
// that, modulo 2^64, is the angle with the whole turns gone: one integer
// product, as exact for position 10^6 as for 1 (an error of 2^-32 of a turn from
// the bits that the conversion to 32-bit floats leaves).  The sines and
// cosines of a token are shared by the rows of an item: each of a warp's four
// row groups computes a quarter of them.
#include "../../include/fd.h"
#include "fd_convert.cuh"
#include "fd_device.cuh"
#include "fd_internal.h"

namespace fdk {

namespace {

__device__ unsigned int g_status = 0;   // this file's bits of the device status word

constexpr unsigned kFullMask = 0xffffffffu;
constexpr int kRopeWarps = 8;

// inv_freq as a fraction of a turn per position, modulo 1, times 2^64.
__device__ __forceinline__ uint64_t turns_of(float f) {
    const uint32_t u = __float_as_uint(f);
    const int e = static_cast<int>((u >> 23) & 255u);
    const uint64_t m = (u & 0x7fffffu) | (e != 0 ? 0x800000u : 0u);      // |f| = m 2^(max(e, 1) - 150)
    constexpr uint64_t kTurn = 2935890503282001226ull;                    // 2^64 / (2 pi)
    const uint64_t lo = m * kTurn, hi = __umul64hi(m, kTurn);
    const int s = 150 - max(e, 1);
    uint64_t t;
    if (s >= 128) t = 0;
    else if (s >= 64) t = hi >> (s - 64);
    else if (s > 0) t = (lo >> s) | (hi << (64 - s));
    else t = s > -64 ? lo << -s : 0;
    return (u >> 31) != 0 ? 0 - t : t;
}

// The 128 elements of a head's weights that a lane needs: its two pieces.
__device__ __forceinline__ void load_weights(float* w, const void* base, int64_t at, int c0, int c1, int dtype) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t i = at + 8 * (h == 0 ? c0 : c1);
        float* to = w + 8 * h;
        if (dtype == 2) {
            const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
            const float4 a = __ldg(f), b = __ldg(f + 1);
            to[0] = a.x, to[1] = a.y, to[2] = a.z, to[3] = a.w;
            to[4] = b.x, to[5] = b.y, to[6] = b.z, to[7] = b.w;
        } else {
            const uint4 r = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i));
            const uint32_t g[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = dtype == 1 ? unpack2<__nv_bfloat16>(g[j]) : unpack2<__half>(g[j]);
                to[2 * j] = v.x;
                to[2 * j + 1] = v.y;
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ void unpack8(float* x, const uint4& r) {
    const float2 a = unpack2<T>(r.x), b = unpack2<T>(r.y), c = unpack2<T>(r.z), d = unpack2<T>(r.w);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y, x[4] = c.x, x[5] = c.y, x[6] = d.x, x[7] = d.y;
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
}

// Eight values into a cache: the 16-bit type, or E4M3 of value * inv.
template <typename T, bool F8>
__device__ __forceinline__ void put8(void* cache, int64_t at, const float* x, float inv) {
    if constexpr (F8) {
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            w[h] = to_e4m3x2<true>(x[4 * h] * inv, x[4 * h + 1] * inv) |
                   (to_e4m3x2<true>(x[4 * h + 2] * inv, x[4 * h + 3] * inv) << 16);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + at) = make_uint2(w[0], w[1]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<T*>(cache) + at) = pack8<T>(x);
    }
}

// A warp takes an item: one token's rows [first, first + 4 ITERS) of its queries, its
// keys or its values.
template <typename T, int ITERS, bool PAIRS, bool F8>
__global__ void __launch_bounds__(kRopeWarps * 32, 2) fd_rope_kernel(const RopeParams p) {
    constexpr int kRows = 4 * ITERS;
    const int lane = threadIdx.x & 31, l = lane & 7, sub = lane >> 3;
    const int half_rot = p.rot_dim / 2, n_rot = p.rot_dim / 16;
    // the lane's two pieces of 8 elements, and whether they are rotated
    int c0, c1;
    bool rot0, rot1;
    if constexpr (PAIRS) {
        c0 = l;
        c1 = l + 8;
        rot0 = c0 < 2 * n_rot;
        rot1 = c1 < 2 * n_rot;
    } else {
        rot0 = rot1 = l < n_rot;
        c0 = rot0 ? l : 2 * l;          // 2 n_rot + 2 (l - n_rot)
        c1 = rot0 ? l + n_rot : c0 + 1;
    }
    const int groups_q = (p.n_q_heads + kRows - 1) / kRows, groups_kv = (p.n_kv_heads + kRows - 1) / kRows;
    const int per_token = groups_q + (p.k_cache != nullptr ? 2 : 1) * groups_kv;
    const int warps = gridDim.x * kRopeWarps;
    const int w0 = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    int64_t t = w0 / per_token;
    int g = w0 % per_token;
    const int dt = warps / per_token, dg = warps % per_token;
    grid_dependency_trigger();
    grid_dependency_wait();

    // of the token's pairs this lane turns eight, indices pair(0 .. 7); it computes two
    auto pair = [&](int e) {
        if constexpr (PAIRS) return e < 4 ? 4 * c0 + e : 4 * c1 + e - 4;
        else return 8 * l + e;
    };
    uint64_t turns[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = pair(2 * sub + j);
        turns[j] = i < half_rot ? turns_of(__ldg(p.inv_freq + i)) : 0;
    }

    for (; t < p.n_tokens; t += dt, g += dg) {
        if (g >= per_token) {
            g -= per_token;
            if (++t >= p.n_tokens) break;
        }
        const int kind = g < groups_q ? 0 : g < groups_q + groups_kv ? 1 : 2;
        const int first = (g - (kind == 0 ? 0 : kind == 1 ? groups_q : groups_q + groups_kv)) * kRows;
        const int heads = kind == 0 ? p.n_q_heads : p.n_kv_heads;
        const T* src = static_cast<const T*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
                       t * (kind == 0 ? p.q_t : kind == 1 ? p.k_t : p.v_t);
        const int64_t src_h = kind == 0 ? p.q_h : kind == 1 ? p.k_h : p.v_h;
        uint4 raw[ITERS][2];
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int h = first + 4 * i + sub;
            raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
            if (h < heads) {
                raw[i][0] = *reinterpret_cast<const uint4*>(src + h * src_h + 8 * c0);
                raw[i][1] = *reinterpret_cast<const uint4*>(src + h * src_h + 8 * c1);
            }
        }
        const int pos = p.positions[t];
        // where the token's keys and values go in the caches
        int64_t lead = 0, in = -1;
        if (kind != 0 && p.k_cache != nullptr) {
            const int64_t slot = p.slots[t];
            if (slot >= 0 && slot < p.n_slots) {
                lead = p.row_shift >= 0 ? slot >> p.row_shift : slot / p.row_tokens;
                in = slot - lead * p.row_tokens;
            } else if (slot >= 0 && pos >= 0) {
                atomicOr(&g_status, kStatusPageBit);
            }
        }
        if (pos < 0) continue;
        if (kind == 2) {
            if (in < 0) continue;
            const int64_t to = lead * p.vc_b + in * p.vc_t;
#pragma unroll
            for (int i = 0; i < ITERS; ++i) {
                const int h = first + 4 * i + sub;
                if (h >= heads) continue;
                float x[16];
                unpack8<T>(x, raw[i][0]);
                unpack8<T>(x + 8, raw[i][1]);
                put8<T, F8>(p.v_cache, to + h * p.vc_h + 8 * c0, x, p.v_inv);
                put8<T, F8>(p.v_cache, to + h * p.vc_h + 8 * c1, x + 8, p.v_inv);
            }
            continue;
        }
        float cs[8], sn[8];
        if (half_rot > 0) {
            float c[2], s[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint64_t a = turns[j] * static_cast<uint32_t>(pos);
                const float half_turns = static_cast<float>(static_cast<int32_t>(a >> 32)) * 0x1p-31f;
                sincospif(half_turns, &s[j], &c[j]);
                s[j] *= p.rot_scale;
                c[j] *= p.rot_scale;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                cs[e] = __shfl_sync(kFullMask, c[e & 1], (e >> 1) * 8 + l);
                sn[e] = __shfl_sync(kFullMask, s[e & 1], (e >> 1) * 8 + l);
            }
        }
        const bool norm = (p.norm & (kind == 0 ? FD_NORM_Q : FD_NORM_K)) != 0;
        const void* weights = kind == 0 ? p.q_w : p.k_w;
        const int64_t w_h = kind == 0 ? p.qw_h : p.kw_h;
        float w[16];
        if (norm && weights != nullptr && w_h == 0) load_weights(w, weights, 0, c0, c1, p.w_dtype);
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int h = first + 4 * i + sub;
            if (first + 4 * i >= heads) break;
            float x[16];
            unpack8<T>(x, raw[i][0]);
            unpack8<T>(x + 8, raw[i][1]);
            if (norm) {
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) sum = fmaf(x[e], x[e], sum);
                sum += __shfl_xor_sync(kFullMask, sum, 1);
                sum += __shfl_xor_sync(kFullMask, sum, 2);
                sum += __shfl_xor_sync(kFullMask, sum, 4);
                const float r = rsqrtf(fmaf(sum, 1.f / 128.f, p.eps));
                if (weights != nullptr) {
                    if (w_h != 0 && h < heads) load_weights(w, weights, h * w_h, c0, c1, p.w_dtype);
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = x[e] * r * w[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] *= r;
                }
            }
            if constexpr (PAIRS) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (e < 4 ? rot0 : rot1) {
                        const float a = x[2 * e], b = x[2 * e + 1];
                        x[2 * e] = a * cs[e] - b * sn[e];
                        x[2 * e + 1] = b * cs[e] + a * sn[e];
                    }
                }
            } else if (rot0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = x[e], b = x[e + 8];
                    x[e] = a * cs[e] - b * sn[e];
                    x[e + 8] = b * cs[e] + a * sn[e];
                }
            }
            if (h >= heads) continue;
            T* row = nullptr;
            if (kind == 0) row = static_cast<T*>(p.q_out) + t * p.qo_t + h * p.qo_h;
            else if (p.k_out != nullptr) row = static_cast<T*>(p.k_out) + t * p.ko_t + h * p.ko_h;
            if (row != nullptr) {
                *reinterpret_cast<uint4*>(row + 8 * c0) = pack8<T>(x);
                *reinterpret_cast<uint4*>(row + 8 * c1) = pack8<T>(x + 8);
            }
            if (kind == 1 && in >= 0) {
                const int64_t to = lead * p.kc_b + h * p.kc_h + in * p.kc_t;
                put8<T, F8>(p.k_cache, to + 8 * c0, x, p.k_inv);
                put8<T, F8>(p.k_cache, to + 8 * c1, x + 8, p.k_inv);
            }
        }
    }
}

template <typename T, int ITERS, bool PAIRS, bool F8>
cudaError_t launch_rope_v(const RopeParams& p, cudaStream_t stream) {
    constexpr int kRows = 4 * ITERS;
    const int64_t per_token = (p.n_q_heads + kRows - 1) / kRows +
                              static_cast<int64_t>(p.k_cache != nullptr ? 2 : 1) * ((p.n_kv_heads + kRows - 1) / kRows);
    const int sms = fd_num_sms(-1);
    if (sms < 1) return cudaErrorInvalidDevice;
    const int64_t ctas = (per_token * p.n_tokens + kRopeWarps - 1) / kRopeWarps;
    const int64_t most = static_cast<int64_t>(sms) * 2;
    return launch_pdl(fd_rope_kernel<T, ITERS, PAIRS, F8>, dim3(static_cast<unsigned>(ctas < most ? ctas : most)),
                      dim3(kRopeWarps * 32), 0, stream, p);
}

template <typename T, int ITERS>
cudaError_t launch_rope_t(const RopeParams& p, bool interleaved, bool fp8_cache, cudaStream_t stream) {
    if (interleaved)
        return fp8_cache ? launch_rope_v<T, ITERS, true, true>(p, stream) : launch_rope_v<T, ITERS, true, false>(p, stream);
    return fp8_cache ? launch_rope_v<T, ITERS, false, true>(p, stream) : launch_rope_v<T, ITERS, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, bool bf16, bool interleaved, bool fp8_cache, cudaStream_t stream) {
    return bf16 ? launch_rope_t<__nv_bfloat16, 1>(p, interleaved, fp8_cache, stream)
                : launch_rope_t<__half, 1>(p, interleaved, fp8_cache, stream);
}

cudaError_t status_word_rope(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_status);
}

}  // namespace fdk
