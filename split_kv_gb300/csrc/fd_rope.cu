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
// product, as exact for position 10^6 as for 1.  Its upper half becomes a 32-bit float of
// half turns: the cut is off by up to 2^-32 of a turn, the conversion by up to 2^-26 (half a
// step next to half a turn, about 1e-7 radians).  The sines and
// cosines of a token are shared by the rows of an item: each of a warp's four
// row groups computes a quarter of them.
#include <algorithm>

#include "../../include/fd.h"
#include "fd_convert.cuh"
#include "fd_device.cuh"
#include "fd_internal.h"

namespace fdk {

namespace {

__device__ unsigned int g_status = 0;   // this file's bits of the device status word

constexpr unsigned kFullMask = 0xffffffffu;
// 4 warps of 128 registers in 4 CTAs an SM, 3 stages of 16 rows (4 KB) each: 192 KB
// of rows on their way.  16384 tokens, 32 / 8 heads, bf16, into a cache (403 MB): 68.7 us, 5.9
// TB/s.  By the way there: 12 warps an SM with 4 stages 76 against 71.5, 20 with 8-row
// stages 120 (spills); all rows through registers instead, 2 / 3 / 4 groups
// ahead, 96 / 105 / 125; two groups' sums and roots side by side, no change; keys and
// values of eight heads as one item, 70.4 against 69 (8 / 1 heads, 60000 tokens: 100 against 109).
constexpr int kRopeWarps = 4;
constexpr int kRopeCtas = 4;            // per SM
constexpr int kRopeStages = 3;          // items of rows that a warp has in flight
constexpr int kRopeGroups = 4;          // groups of four rows in an item

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

// The elements of a head's weights at the lane's two pieces.
__device__ __forceinline__ void load_weights(float2 (&w)[8], const void* base, int64_t at, int c0, int c1, int dtype) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t i = at + 8 * (h == 0 ? c0 : c1);
        float2* to = w + 4 * h;
        if (dtype == 2) {
            const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
            const float4 a = __ldg(f), b = __ldg(f + 1);
            to[0] = make_float2(a.x, a.y), to[1] = make_float2(a.z, a.w);
            to[2] = make_float2(b.x, b.y), to[3] = make_float2(b.z, b.w);
        } else {
            const uint4 r = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i));
            const uint32_t g[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) to[j] = dtype == 1 ? unpack2<__nv_bfloat16>(g[j]) : unpack2<__half>(g[j]);
        }
    }
}

template <typename T>
__device__ __forceinline__ void unpack8(float2* x, const uint4& r) {
    x[0] = unpack2<T>(r.x), x[1] = unpack2<T>(r.y), x[2] = unpack2<T>(r.z), x[3] = unpack2<T>(r.w);
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float2* x) {
    return make_uint4(pack2<T>(x[0].x, x[0].y), pack2<T>(x[1].x, x[1].y), pack2<T>(x[2].x, x[2].y), pack2<T>(x[3].x, x[3].y));
}

// A product that overflows is of a finite value: 448, as the conversion makes it.
__device__ __forceinline__ uint32_t quantised2(float2 x, float inv) {
    return to_e4m3x2<false>(nan_for_inf(x.x) * inv, nan_for_inf(x.y) * inv);
}

__device__ __forceinline__ uint2 quantised8(const float2* x, float inv) {
    return make_uint2(quantised2(x[0], inv) | (quantised2(x[1], inv) << 16), quantised2(x[2], inv) | (quantised2(x[3], inv) << 16));
}

// An item is up to 4 GROUPS rows of one token: of its queries, its keys or its
// values.  The items of all tokens, in order, are dealt to the warps in equal runs, so
// that sines and cosines are computed once for several; with more than one group, the rows of the items ahead are on
// their way into the warp's stages of shared memory meanwhile (a bulk copy a row,
// issued by a lane each, so that no register is spent on it).
//
// Weight, cosine and sine are multiplied once per item into coefficients A and B,
// so that a row costs y = A (r x) + B (r x's partner), two elements an
// instruction.  FULL: whole rows are rotated; else the elements that
// are not never meet their B (an infinity times 0 would be a NaN).
//
// Large calls are bound by HBM and by their ends (65536 tokens 6.2 TB/s, 16384 5.9, 4096
// 5.0): a plain copy of the same 403 MB takes about 65 us.  56 % of the issue slots are taken.
template <typename T, int GROUPS, bool PAIRS, bool F8, bool FULL>
__global__ void __launch_bounds__(kRopeWarps * 32, kRopeCtas)
    fd_rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr bool kStaged = GROUPS > 1;
    constexpr int kRows = 4 * GROUPS, kStageBytes = kRows * 256, kStages = kStaged ? kRopeStages : 1;
    extern __shared__ __align__(128) unsigned char s_rows[];    // [warps][stages][rows][256]
    __shared__ __align__(8) uint64_t s_bar[kRopeWarps][kStages];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7, sub = lane >> 3;
    const int half_rot = p.rot_dim / 2, n_rot = p.rot_dim / 16;
    // the lane's two pieces of 8 elements, and whether they are rotated
    int c0 = l, c1 = l + 8;
    bool rot0 = true, rot1 = true;
    if constexpr (!FULL) {
        if constexpr (PAIRS) {
            rot0 = c0 < 2 * n_rot;
            rot1 = c1 < 2 * n_rot;
        } else {
            rot0 = rot1 = l < n_rot;
            c0 = rot0 ? l : 2 * l;      // 2 n_rot + 2 (l - n_rot)
            c1 = rot0 ? l + n_rot : c0 + 1;
        }
    }
    const int items_q = (p.side[0].heads + kRows - 1) / kRows, items_k = (p.side[1].heads + kRows - 1) / kRows;
    const int items = items_q + items_k + (p.side[2].cache != nullptr ? items_k : 0);
    const unsigned warps = gridDim.x * kRopeWarps, w0 = blockIdx.x * kRopeWarps + warp;
    const int64_t all = static_cast<int64_t>(p.n_tokens) * items;
    const int64_t begin = all * w0 / warps;
    int left = static_cast<int>(all * (w0 + 1) / warps - begin);   // items of this warp that are not done, and not asked for
    int left_ahead = left;
    // Heads that lie end to end may come in one copy, which starts sooner, or in one a row, which
    // keeps more of them on their way.  A row / one, us: 32 / 8 heads, 1024 tokens 6.9 / 6.2, 4096
    // 20.7 / 20.2, 16384 68.7 / 71.4; 8 / 8 heads, 2048 7.0 / 6.4; 64 / 8, 8192 58.3 / 62.5.
    const bool few = all <= 8 * static_cast<int64_t>(warps);
    const uint32_t bars = smem_u32(s_bar[warp]);
    const uint32_t stages = smem_u32(s_rows) + warp * (kStages * kStageBytes);
    if constexpr (kStaged) {
        if (lane < kStages) mbar_init(bars + 8 * lane, 1);
        fence_barrier_init();
        __syncwarp();
    }
    grid_dependency_trigger();
    grid_dependency_wait();

    struct Place {                      // an item of a token
        unsigned t;
        int i;
    };
    auto advance = [&](Place& x) {
        if (++x.i == items) {
            x.i = 0;
            ++x.t;
        }
    };
    auto kind_of = [&](const Place& x) { return x.i < items_q ? 0 : x.i < items_q + items_k ? 1 : 2; };
    auto first_of = [&](const Place& x, int kind) {
        return (x.i - (kind == 0 ? 0 : kind == 1 ? items_q : items_q + items_k)) * kRows;
    };
    int pos[kStages];                   // of the items in flight
    int64_t slot[kStages];
    uint4 direct[2];                    // (without stages: the item's rows)
    auto load = [&](const Place& x, int stage) {
        if (left_ahead == 0) return;
        --left_ahead;
        const int kind = kind_of(x), first = first_of(x, kind);
        const RopeSide& sd = p.side[kind];
        const int n = min(kRows, sd.heads - first);
        const T* src = static_cast<const T*>(sd.src) + x.t * sd.src_t;
        if constexpr (kStaged) {
            if (lane == 0) mbar_arrive_expect_tx(bars + 8 * stage, n * 256);
            const bool dense = few && sd.src_h == kHeadDim;
            if (lane < (dense ? 1 : n))
                bulk_load(stages + stage * kStageBytes + lane * 256, src + (first + lane) * sd.src_h, dense ? n * 256 : 256, bars + 8 * stage);
        } else {
            const uint4* row = reinterpret_cast<const uint4*>(src + (first + min(sub, n - 1)) * sd.src_h);
            direct[0] = row[c0];
            direct[1] = row[c1];
        }
        pos[kStages - 1] = p.positions[x.t];
        slot[kStages - 1] = sd.cache != nullptr ? p.slots[x.t] : -1;
    };

    Place cur = {static_cast<unsigned>(begin / items), static_cast<int>(begin % items)};
    Place ahead = cur;
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
#pragma unroll
        for (int j = 0; j + 1 < kStages; ++j) {
            pos[j] = pos[j + 1];
            slot[j] = slot[j + 1];
        }
        load(ahead, s);
        advance(ahead);
    }
    // of a token's pairs this lane turns eight, indices pair(0 .. 7); it computes two
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
    unsigned turned = 0xffffffffu;      // the token that cs and sn belong to,
    int folded = -1;                    // and the kind that A and B, with its weights, do
    float cs[8], sn[8];
    float2 A[8], B[8];
    auto fold = [&](const float2 (&w)[8]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (PAIRS) {      // elements 2e, 2e + 1 of each piece are a pair
                const float2 c = make_float2(cs[e], cs[e]), d = make_float2(cs[4 + e], cs[4 + e]);
                A[e] = rot0 ? __fmul2_rn(w[e], c) : w[e];
                B[e] = make_float2(-w[e].y * sn[e], w[e].x * sn[e]);
                A[4 + e] = rot1 ? __fmul2_rn(w[4 + e], d) : w[4 + e];
                B[4 + e] = make_float2(-w[4 + e].y * sn[4 + e], w[4 + e].x * sn[4 + e]);
            } else {                    // element i of one piece and i of the other
                const float2 c = make_float2(cs[2 * e], cs[2 * e + 1]), s = make_float2(sn[2 * e], sn[2 * e + 1]);
                A[e] = rot0 ? __fmul2_rn(w[e], c) : w[e];
                A[4 + e] = rot0 ? __fmul2_rn(w[4 + e], c) : w[4 + e];
                B[e] = __fmul2_rn(make_float2(-w[4 + e].x, -w[4 + e].y), s);
                B[4 + e] = __fmul2_rn(w[e], s);
            }
        }
    };
    int stage = 0, phase = 0;
    for (; left > 0; --left, advance(cur)) {
        if (kStaged && __any_sync(kFullMask, !mbar_wait(bars + 8 * stage, phase))) {
            // the copies never came: say so, give those behind the same time, leave
            if (lane == 0) atomicOr(&g_status, kStatusTimeoutBit);
            for (int s = 1; s < kStages && --left > 0; ++s) {
                if (++stage == kStages) stage = 0, phase ^= 1;
                mbar_wait(bars + 8 * stage, phase);
            }
            return;
        }
        const unsigned char* from = s_rows + (warp * kStages + stage) * kStageBytes + sub * 256;
        auto piece = [&](int i, int c) {            // 8 elements of the row of group i
            if constexpr (kStaged) return *reinterpret_cast<const uint4*>(from + i * 1024 + 16 * (c == 0 ? c0 : c1));
            else return direct[c];
        };
        const int my_pos = pos[0];
        const int64_t my_slot = slot[0];
#pragma unroll
        for (int j = 0; j + 1 < kStages; ++j) {
            pos[j] = pos[j + 1];
            slot[j] = slot[j + 1];
        }
        const int kind = kind_of(cur), first = first_of(cur, kind);
        const RopeSide& sd = p.side[kind];
        const int heads = sd.heads;
        // where the token's keys and values go in the caches
        unsigned char* cache = nullptr;
        if (my_slot >= 0 && my_pos >= 0) {
            if (my_slot < p.n_slots) {
                const int64_t lead = p.row_shift >= 0 ? my_slot >> p.row_shift : my_slot / p.row_tokens;
                const int64_t in = my_slot - lead * p.row_tokens;
                cache = static_cast<unsigned char*>(sd.cache) +
                        (lead * sd.cache_b + in * sd.cache_t + (first + sub) * sd.cache_h) * (F8 ? 1 : 2);
            } else if (lane == 0) {
                atomicOr(&g_status, kStatusPageBit);
            }
        }
        const int64_t cache_step = 4 * sd.cache_h * (F8 ? 1 : 2);
        if (my_pos >= 0 && kind == 2) {
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) {
                if (first + 4 * i + sub >= heads || cache == nullptr) break;
                const uint4 ra = piece(i, 0), rb = piece(i, 1);
                if constexpr (F8) {
                    float2 x[8];
                    unpack8<T>(x, ra);
                    unpack8<T>(x + 4, rb);
                    *reinterpret_cast<uint2*>(cache + i * cache_step + 8 * c0) = quantised8(x, sd.inv);
                    *reinterpret_cast<uint2*>(cache + i * cache_step + 8 * c1) = quantised8(x + 4, sd.inv);
                } else {
                    *reinterpret_cast<uint4*>(cache + i * cache_step + 16 * c0) = ra;
                    *reinterpret_cast<uint4*>(cache + i * cache_step + 16 * c1) = rb;
                }
            }
        } else if (my_pos >= 0) {
            if (turned != cur.t) {
                turned = cur.t;
                folded = -1;
                float c[2], s[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint64_t a = turns[j] * static_cast<uint32_t>(my_pos);
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
            if (folded != kind) {
                folded = kind;
                float2 w[8];
                if (sd.weights != nullptr && sd.w_h == 0) {
                    load_weights(w, sd.weights, 0, c0, c1, p.w_dtype);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = make_float2(1.f, 1.f);
                }
                fold(w);
            }
            T* row = sd.out == nullptr ? nullptr : static_cast<T*>(sd.out) + cur.t * sd.out_t + (first + sub) * sd.out_h;
            const int64_t row_step = 4 * sd.out_h;
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) {
                const int h = first + 4 * i + sub;
                if (first + 4 * i >= heads) break;
                // (behind the last head: what the stage held before; it is not stored)
                float2 x[8], y[8];
                unpack8<T>(x, piece(i, 0));
                unpack8<T>(x + 4, piece(i, 1));
                if (sd.norm != 0) {
                    float2 s2 = __fmul2_rn(x[0], x[0]);
#pragma unroll
                    for (int e = 1; e < 8; ++e) s2 = __ffma2_rn(x[e], x[e], s2);
                    float sum = s2.x + s2.y;
                    sum += __shfl_xor_sync(kFullMask, sum, 1);
                    sum += __shfl_xor_sync(kFullMask, sum, 2);
                    sum += __shfl_xor_sync(kFullMask, sum, 4);
                    const float r = rsqrtf(fmaf(sum, 1.f / 128.f, p.eps));
                    if (sd.w_h != 0) {  // a head's own weights
                        float2 w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[e] = make_float2(1.f, 1.f);
                        if (h < heads) load_weights(w, sd.weights, h * sd.w_h, c0, c1, p.w_dtype);
                        fold(w);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = __fmul2_rn(x[e], make_float2(r, r));
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = __fmul2_rn(x[e], A[e]);
                if constexpr (PAIRS) {
                    if (rot0) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = __ffma2_rn(make_float2(x[e].y, x[e].x), B[e], y[e]);
                    }
                    if (rot1) {
#pragma unroll
                        for (int e = 4; e < 8; ++e) y[e] = __ffma2_rn(make_float2(x[e].y, x[e].x), B[e], y[e]);
                    }
                } else if (rot0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = __ffma2_rn(x[e ^ 4], B[e], y[e]);
                }
                if (h < heads) {
                    if (row != nullptr) {
                        *reinterpret_cast<uint4*>(row + i * row_step + 8 * c0) = pack8<T>(y);
                        *reinterpret_cast<uint4*>(row + i * row_step + 8 * c1) = pack8<T>(y + 4);
                    }
                    if (cache != nullptr) {
                        if constexpr (F8) {
                            *reinterpret_cast<uint2*>(cache + i * cache_step + 8 * c0) = quantised8(y, sd.inv);
                            *reinterpret_cast<uint2*>(cache + i * cache_step + 8 * c1) = quantised8(y + 4, sd.inv);
                        } else {
                            *reinterpret_cast<uint4*>(cache + i * cache_step + 16 * c0) = pack8<T>(y);
                            *reinterpret_cast<uint4*>(cache + i * cache_step + 16 * c1) = pack8<T>(y + 4);
                        }
                    }
                }
            }
        }
        __syncwarp();                   // (every lane has read the stage)
        load(ahead, stage);
        advance(ahead);
        if (++stage == kStages) stage = 0, phase ^= 1;
    }
}

template <typename T, int GROUPS, bool PAIRS, bool F8, bool FULL>
cudaError_t launch_rope_v(const RopeParams& p, cudaStream_t stream) {
    constexpr int kRows = 4 * GROUPS;
    constexpr size_t kSmem = GROUPS > 1 ? static_cast<size_t>(kRopeWarps) * kRopeStages * kRows * 256 : 0;
    const int64_t kv_items = (p.side[1].heads + kRows - 1) / kRows;
    const int64_t items = (p.side[0].heads + kRows - 1) / kRows + (p.side[2].cache != nullptr ? 2 : 1) * kv_items;
    const int sms = fd_num_sms(-1);
    if (sms < 1) return cudaErrorInvalidDevice;
    auto kern = fd_rope_kernel<T, GROUPS, PAIRS, F8, FULL>;
    static std::atomic<unsigned long long> configured_ctx{0};
    const cudaError_t e = allow_smem(kern, kSmem, configured_ctx);
    if (e != cudaSuccess) return e;
    const int64_t ctas = (static_cast<int64_t>(p.n_tokens) * items + kRopeWarps - 1) / kRopeWarps;
    return launch_pdl(kern, dim3(static_cast<unsigned>(std::min<int64_t>(ctas, sms * kRopeCtas))), dim3(kRopeWarps * 32), kSmem,
                      stream, p);
}

template <typename T, int GROUPS, bool PAIRS>
cudaError_t launch_rope_p(const RopeParams& p, bool fp8_cache, cudaStream_t stream) {
    const bool full = p.rot_dim == kHeadDim;
    if (fp8_cache)
        return full ? launch_rope_v<T, GROUPS, PAIRS, true, true>(p, stream) : launch_rope_v<T, GROUPS, PAIRS, true, false>(p, stream);
    return full ? launch_rope_v<T, GROUPS, PAIRS, false, true>(p, stream) : launch_rope_v<T, GROUPS, PAIRS, false, false>(p, stream);
}

template <typename T, int GROUPS>
cudaError_t launch_rope_t(const RopeParams& p, bool interleaved, bool fp8_cache, cudaStream_t stream) {
    return interleaved ? launch_rope_p<T, GROUPS, true>(p, fp8_cache, stream) : launch_rope_p<T, GROUPS, false>(p, fp8_cache, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, bool bf16, bool interleaved, bool fp8_cache, cudaStream_t stream) {
    // While every group of four rows has a warp of its own, a warp loads it
    // directly: what counts is the time of one group.  Beyond that, staged items
    // of 16 rows.  Direct / staged, us: 64 tokens of 32 / 8 heads 2.8 / 3.8, 128 2.9 / 4.1, 256
    // 4.2 / 4.2, 512 5.7 / 4.3; 8 / 8 heads 256 2.8 / 3.7, 512 4.0 / 3.8; 64 / 8 128 4.0 / 4.5, 256 5.5 / 4.7.
    const int sms = fd_num_sms(-1);
    if (sms < 1) return cudaErrorInvalidDevice;
    const int64_t groups = (p.side[0].heads + 3) / 4 + static_cast<int64_t>(p.side[2].cache != nullptr ? 2 : 1) * ((p.side[1].heads + 3) / 4);
    if (groups * p.n_tokens <= static_cast<int64_t>(sms) * kRopeCtas * kRopeWarps)
        return bf16 ? launch_rope_t<__nv_bfloat16, 1>(p, interleaved, fp8_cache, stream)
                    : launch_rope_t<__half, 1>(p, interleaved, fp8_cache, stream);
    return bf16 ? launch_rope_t<__nv_bfloat16, kRopeGroups>(p, interleaved, fp8_cache, stream)
                : launch_rope_t<__half, kRopeGroups>(p, interleaved, fp8_cache, stream);
}

cudaError_t status_word_rope(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_status);
}

}  // namespace fdk
