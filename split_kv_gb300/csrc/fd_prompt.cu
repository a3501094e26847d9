// fd_prompt.cu -- attention over whole prompts (fd_prompt): packed sequences
// of different lengths, causal or full, grouped heads, on 5th-generation
// tensor cores.
//
//   s_ij = q_i . k_j / sqrt(128),  out_i = sum_j p_ij v_j / l_i,
//   p_ij = 2^(t_ij - m_i),  t = s log2(e),  l_i = sum_j p_ij,  lse_i = ln2 (m_i + log2 l_i)
// in one pass over the keys: m_i is a running reference that follows the row's
// maximum lazily (it moves when a tile's maximum passes it by more than 8, so
// p stays below 2^8 and O is rescaled only then); any reference gives the same
// result up to rounding.
//
// One CTA takes two query tiles of 128 rows and walks the key tiles of 128 they
// see.  The two tiles are the same positions of two heads of one group where
// the group is even (both then see the same keys, and a causal pair wastes
// half a tile on the diagonal, not one and a half), else 256 positions of one
// head.  Per key tile and query tile:
//   S[128 x 128] = Q K^T      8 MMAs of 16 dims, operands in shared memory
//   O[128 x 128] += P V       8 MMAs of 16 keys, P from tensor memory
// Warps 0-3 and 4-7 are the softmax of tile 0 and 1, a thread per row: it reads
// its row of S from tensor memory, writes P (16 bits; the sums l keep the
// unrounded weights) over it, in two halves so that PV starts on the first
// while the second is computed.  Warp 8 streams K and V tiles with TMA through
// a ring of five 32 KB slots, warp 9 issues the MMAs: while one tile's softmax
// runs, the tensor cores work on the other tile's PV and next S.  Warp 10
// guards the masked tiles (below).
// Tensor memory (512 columns): S/P of tile 0, 1 at 0, 128; O at 256, 384.
//
// Masked places: scores past a row's limit are replaced by -inf before they
// are used, so what K holds there does not matter.  P is 0 there, but 0 * NaN
// is NaN, so in the (last) tiles where some row's limit falls, warp 10 zeroes
// the V rows past the sequence's end and looks for infinities and NaN in the
// others; only if it finds one are the CTA's rows computed again by a plain
// loop over the keys each row sees.
//
// Bound by the tensor cores when sequences are long: 4 * 128 flops per visible
// pair and head against 2 bytes per element read once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "../../include/fd.h"
#include "fd_device.cuh"
#include "fd_internal.h"

namespace fdk {

namespace {

__device__ unsigned int g_status = 0;   // this file's bits of the device status word

constexpr unsigned kFullMask = 0xffffffffu;
constexpr float kLn2 = 0.693147180559945309f;
constexpr int kTile = 128;              // queries per tile, keys per tile
constexpr int kSlots = 5;
constexpr int kSlotBytes = kTile * 256; // [128 x 64 dims] low half, high half
constexpr int kHalf = kSlotBytes / 2;
constexpr int kOffRing = 2 * kSlotBytes;
constexpr int kOffBar = kOffRing + kSlots * kSlotBytes;
constexpr int kSmem = kOffBar + 512 + 1024;
constexpr int kPromptThreads = 11 * 32;
constexpr float kLazy = 8.f;

// mbarriers, 8 bytes each from kOffBar
enum Bar : int {
    kBarQ = 0,                  // [2] a tile's Q landed
    kBarFull = 2,               // [kSlots]
    kBarEmpty = kBarFull + kSlots,
    kBarS = kBarEmpty + kSlots, // [2] S written (MMA commit)
    kBarP = kBarS + 2,          // [2 tiles][2 halves] P written (and O rescaled), one arrival per warp
    kBarO = kBarP + 4,          // [2] PV done (MMA commit)
    kBarV = kBarO + 2,          // [4] a masked tile's V is guarded, by its number mod 4
    kBarG = kBarV + 4,          // [4] a masked tile's V landed and waits for the guard
    kBarDrain = kBarG + 4,      // every MMA done
    kBars
};
static_assert(kBars * 8 <= 256, "barriers");

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    if (mbar_wait(bar, parity)) return true;
    atomicOr(&g_status, kStatusTimeoutBit);
    *abort_flag = 1;
    return false;
}

// A value that every lane has, known to the compiler as warp-uniform.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(kFullMask, x, 0); }
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(kFullMask, x, 0); }

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// wait_bar by a whole warp, which leaves it together.
__device__ __forceinline__ bool wait_bar_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    if (__all_sync(kFullMask, mbar_try_wait(bar, parity))) return true;
    return __all_sync(kFullMask, wait_bar(bar, parity, abort_flag));
}

// umma_idesc_f16 of 128 x 128 as a constant
constexpr uint32_t umma_idesc(bool bf16, bool b_mn_major) {
    return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (b_mn_major ? 1u << 16 : 0u) | (128u >> 3) << 17 | (128u >> 4) << 24;
}

// What one CTA does: two query tiles and the key tiles [j0, j1) of one sequence.
struct Work {
    int b;                      // -1: nothing
    int q0, k0, nq, nk;         // the sequence's rows
    int head[2], pos[2];        // of the two query tiles
    int n[2];                   // key tiles each sees, from 0 (0: inactive)
    int j0, j1;                 // key tiles of this split
    int guard;                  // first key tile where some row's limit falls
    int split;
};

__device__ __forceinline__ int seen_by(const PromptParams& p, int nq, int nk, int i) {
    return p.causal ? min(max(nk - nq + 1 + i, 0), nk) : nk;
}

// The work of block `block`, found by one warp.  Blocks are (query tile, head
// unit, split), splits fastest; a sequence's tiles come last first, since the
// last ones see the most keys.
__device__ __forceinline__ void find_work(const PromptParams& p, int64_t block, int lane, Work& w, bool report) {
    const int split = static_cast<int>(block % p.n_splits);
    const int64_t rest = block / p.n_splits;
    const int unit = static_cast<int>(rest % p.head_units);
    int tile = static_cast<int>(rest / p.head_units);
    w.b = -1;
    const int span = p.pair_heads ? kTile : 2 * kTile;   // positions per CTA
    for (int base = 0; base < p.batch; base += 32) {
        const int b = base + lane;
        int a = 0, e = 0, ka = 0, ke = 0;
        if (b < p.batch) {
            a = p.cu_q[b];
            e = p.cu_q[b + 1];
            ka = p.cu_k[b];
            ke = p.cu_k[b + 1];
        }
        const bool ok = a >= 0 && e >= a && e <= p.total_q && ka >= 0 && ke >= ka && ke <= p.total_k;
        if (!ok && report) atomicOr(&g_status, kStatusSeqlenBit);
        const int tiles = ok ? (e - a + span - 1) / span : 0;
        int upto = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFullMask, upto, o);
            if (lane >= o) upto += y;
        }
        const unsigned hit = __ballot_sync(kFullMask, tile < upto);
        const int all = __shfl_sync(kFullMask, upto, 31);
        if (hit != 0 && w.b < 0) {
            const int src = __ffs(hit) - 1;
            const int mine = tile - (upto - tiles);      // this lane's view of the tile's number
            w.b = base + src;
            w.q0 = __shfl_sync(kFullMask, a, src);
            w.nq = __shfl_sync(kFullMask, e, src) - w.q0;
            w.k0 = __shfl_sync(kFullMask, ka, src);
            w.nk = __shfl_sync(kFullMask, ke, src) - w.k0;
            const int from_end = __shfl_sync(kFullMask, mine, src);
            tile = __shfl_sync(kFullMask, tiles, src) - 1 - from_end;
            if (!report) break;
        } else if (w.b < 0) {
            tile -= all;
        }
    }
    if (w.b < 0) return;
    w.split = split;
    int most = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        w.head[t] = p.pair_heads ? 2 * unit + t : unit;
        w.pos[t] = tile * span + (p.pair_heads ? 0 : t * kTile);
        const int last = min(w.pos[t] + kTile, w.nq) - 1;
        const int keys = last >= w.pos[t] ? seen_by(p, w.nq, w.nk, last) : 0;
        w.n[t] = (keys + kTile - 1) / kTile;
        most = max(most, w.n[t]);
    }
    const int each = most / p.n_splits, more = most % p.n_splits;
    w.j0 = split * each + min(split, more);
    w.j1 = w.j0 + each + (split < more ? 1 : 0);
    w.n[0] = min(w.n[0], w.j1);
    w.n[1] = min(w.n[1], w.j1);
    w.guard = max(w.j0, seen_by(p, w.nq, w.nk, w.pos[0]) / kTile);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
                 "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
                 "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    uint32_t r;
    memcpy(&r, &h, 4);
    return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    uint32_t r;
    memcpy(&r, &h, 4);
    return r;
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (std::is_same<T, __half>::value) {
        __half2 h;
        memcpy(&h, &w, 4);
        return __half22float2(h);
    } else {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
}

__device__ __forceinline__ int64_t out_row(const PromptParams& p, const Work& w, int t, int i) {
    return (static_cast<int64_t>(w.q0) + i) * p.n_q_heads + w.head[t];
}

// N consecutive dims of a row of out, from dim d (a multiple of N, N = 4 or 16)
template <int N>
__device__ __forceinline__ void put_out(const PromptParams& p, int64_t row, int d, const float* o) {
    const int64_t at = row * kHeadDim + d;
    if (p.out_dtype == 2) {
        float* dst = static_cast<float*>(p.out) + at;
        if (p.out_vec) {
#pragma unroll
            for (int e = 0; e < N; e += 4)
                *reinterpret_cast<float4*>(dst + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) dst[e] = o[e];
        }
        return;
    }
    uint32_t w[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e)
        w[e] = p.out_dtype == 0 ? pack2<__half>(o[2 * e], o[2 * e + 1]) : pack2<__nv_bfloat16>(o[2 * e], o[2 * e + 1]);
    uint16_t* dst = static_cast<uint16_t*>(p.out) + at;
    if (p.out_vec) {
        if constexpr (N == 4) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int e = 0; e < N / 2; e += 4)
                *reinterpret_cast<uint4*>(dst + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
            dst[2 * e] = static_cast<uint16_t>(w[e]);
            dst[2 * e + 1] = static_cast<uint16_t>(w[e] >> 16);
        }
    }
}

// A row again, by one warp over the keys [j0, j1): lane l holds dims 4l .. 4l + 3.
template <typename T>
__device__ __noinline__ void plain_row(const PromptParams& p, const Work& w, int t, int i, int lane) {
    const int j0 = w.j0 * kTile, j1 = min(w.j1 * kTile, seen_by(p, w.nq, w.nk, i));
    const int g = w.head[t] / p.group;
    const T* q = static_cast<const T*>(p.q) + (static_cast<int64_t>(w.q0) + i) * p.q_st + w.head[t] * p.q_sh + 4 * lane;
    const uint2 qw = *reinterpret_cast<const uint2*>(q);
    const float2 qa = unpack2<T>(qw.x), qb = unpack2<T>(qw.y);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = j0; j < j1; ++j) {
        const int64_t row = static_cast<int64_t>(w.k0) + j;
        const uint2 kw = *reinterpret_cast<const uint2*>(static_cast<const T*>(p.k) + row * p.k_st + g * p.k_sh + 4 * lane);
        const uint2 vw = *reinterpret_cast<const uint2*>(static_cast<const T*>(p.v) + row * p.v_st + g * p.v_sh + 4 * lane);
        const float2 ka = unpack2<T>(kw.x), kb = unpack2<T>(kw.y), va = unpack2<T>(vw.x), vb = unpack2<T>(vw.y);
        float s = fmaf(qa.x, ka.x, fmaf(qa.y, ka.y, fmaf(qb.x, kb.x, qb.y * kb.y)));
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(kFullMask, s, x);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s), mu = mn == -INFINITY ? 0.f : mn;
        const float a = fast_exp2(m - mu), e = fast_exp2(s - mu);
        m = mn;
        l = fmaf(l, a, e);
        o[0] = fmaf(o[0], a, e * va.x);
        o[1] = fmaf(o[1], a, e * va.y);
        o[2] = fmaf(o[2], a, e * vb.x);
        o[3] = fmaf(o[3], a, e * vb.y);
    }
    const int64_t row = out_row(p, w, t, i);
    const bool empty = j1 <= j0;
    if (p.n_splits == 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = empty ? 0.f : o[e] / l;
        put_out<4>(p, row, 4 * lane, o);
        if (lane == 0 && p.lse != nullptr) p.lse[row] = empty ? -INFINITY : (m + log2f(l)) * kLn2;
    } else {
        const int64_t at = row * p.n_splits + w.split;
        *reinterpret_cast<float4*>(p.ws_u + at * kHeadDim + 4 * lane) = make_float4(o[0], o[1], o[2], o[3]);
        if (lane == 0) {
            p.ws_m[at] = m;
            p.ws_l[at] = l;
        }
    }
}

// Any infinity or NaN among the eight 16-bit values of a piece: an exponent of
// all ones carries into the sign bit when one more is added.
template <typename T>
__device__ __forceinline__ bool any_special(const uint4& r) {
    constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
    constexpr uint32_t one = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
    return ((((r.x & e) + one) | ((r.y & e) + one) | ((r.z & e) + one) | ((r.w & e) + one)) & 0x80008000u) != 0;
}

template <typename T>
__global__ void __launch_bounds__(kPromptThreads, 1)
    fd_prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const PromptParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t bar0 = smem_u32(smem + kOffBar);
    auto bar = [&](int i) { return bar0 + 8u * i; };
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + kOffBar + 256);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffBar + 260);
    volatile int* special = reinterpret_cast<volatile int*>(smem + kOffBar + 264);
    Work* shared_work = reinterpret_cast<Work*>(smem + kOffBar + 272);
    static_assert(272 + sizeof(Work) <= 512, "work");

    if (threadIdx.x == 256) {
        for (int i = 0; i < kBars; ++i) mbar_init(bar(i), i >= kBarP && i < kBarP + 4 ? 4 : 1);
        *abort_flag = 0;
        *special = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    grid_dependency_trigger();
    grid_dependency_wait();
    if (warp == 0) {
        Work w;
        find_work(p, blockIdx.x, lane, w, blockIdx.x == 0);
        if (lane == 0) *shared_work = w;
    }
    __syncthreads();
    const Work w = *shared_work;
    if (w.b < 0) return;
    const int n0 = w.n[0], n1 = w.n[1], j0 = w.j0;
    const int n = max(n0, n1);
    const bool run0 = n0 > j0, run1 = n1 > j0;

    if (warp == 1) tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 8) {
        // ---- producer: Q of both tiles, then K and V of each key tile
        if (lane == 0 && n > j0) {
            const int g = w.head[0] / p.group;
            auto load = [&](uint8_t* dst, const CUtensorMap* map, uint32_t b, int row, int head) {
                mbar_arrive_expect_tx(b, kSlotBytes);
                tma_load_4d(smem_u32(dst), map, b, 0, row, head, 0);
                tma_load_4d(smem_u32(dst + kHalf), map, b, 64, row, head, 0);
            };
            if (run0) load(smem, &tmQ, bar(kBarQ), w.q0 + w.pos[0], w.head[0]);
            int i = 0;
            bool ok = true;
            auto tile = [&](const CUtensorMap* map, int j) {
                const int s = i % kSlots;
                if (i >= kSlots) ok = ok && wait_bar(bar(kBarEmpty + s), (i / kSlots - 1) & 1, abort_flag);
                if (!ok || *abort_flag) {
                    ok = false;
                    return;
                }
                load(smem + kOffRing + s * kSlotBytes, map, bar(kBarFull + s), w.k0 + j * kTile, g);
                ++i;
            };
            tile(&tmK, j0);
            if (run1) load(smem + kSlotBytes, &tmQ, bar(kBarQ + 1), w.q0 + w.pos[1], w.head[1]);
            for (int j = j0; ok && j < n; ++j) {
                tile(&tmV, j);
                if (ok && j + 1 < n) tile(&tmK, j + 1);
            }
            // nothing may be in flight towards this CTA when it exits
            if (run0) wait_bar(bar(kBarQ), 0, abort_flag);
            if (run1) wait_bar(bar(kBarQ + 1), 0, abort_flag);
            for (int x = max(0, i - kSlots); x < i; ++x) wait_bar(bar(kBarFull + x % kSlots), (x / kSlots) & 1, abort_flag);
        }
        __syncwarp();
    } else if (warp == 9) {
        // ---- MMA issue: the whole warp walks the tiles, one elected lane issues.
        // Everything the MMAs take is warp-uniform for the compiler (the
        // shuffles), so that descriptors stay in uniform registers: from inside
        // a one-lane branch an MMA cost its thread 113 cycles, with 64 the tensor
        // cores' own time.
        const int m_n0 = uniform(n0), m_n1 = uniform(n1), m_j0 = uniform(j0), m_guard = uniform(w.guard);
        const int m_n = max(m_n0, m_n1);
        if (m_n > m_j0) {
            constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
            constexpr uint32_t id_s = umma_idesc(kBf16, false), id_o = umma_idesc(kBf16, true);
            const uint32_t sm = uniform(smem_u32(smem)), tm = uniform(tmem), b0 = uniform(bar0);
            const uint64_t dq = umma_desc_sw128(sm, 16, 1024);
            const uint64_t dk = umma_desc_sw128(sm + kOffRing, 16, 1024);
            const uint64_t dv = umma_desc_sw128(sm + kOffRing, kHalf, 1024);
            const bool leader = elect_one();
            bool ok = true;
            auto wait = [&](int i, uint32_t parity) {
                if (ok) ok = wait_bar_warp(b0 + 8u * i, parity, abort_flag);
            };
            int slot = 0;                        // ring slot of the entry at hand, and the parity of its use
            uint32_t use = 0;
            auto next_slot = [&]() {
                if (++slot == kSlots) {
                    slot = 0;
                    use ^= 1u;
                }
            };
            // S of tile t from the K at `slot`
            auto issue_s = [&](auto tile, bool last) {
                constexpr int t = decltype(tile)::value;
                if (!ok) return;
                tc_fence_after();
                const uint64_t a = dq + static_cast<uint32_t>(t * (kSlotBytes >> 4));
                const uint64_t b = dk + static_cast<uint32_t>(slot) * (kSlotBytes >> 4);
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32u) >> 4;
                        umma_f16(tm + 128u * t, a + off, b + off, id_s, kk > 0);
                    }
                    umma_commit(b0 + 8u * (kBarS + t));
                    if (last) umma_commit(b0 + 8u * (kBarEmpty + slot));
                }
                __syncwarp();
            };
            // half h of PV of tile t from the V at `slot`
            auto issue_pv = [&](auto tile, int h, bool first) {
                constexpr int t = decltype(tile)::value;
                if (!ok) return;
                tc_fence_after();
                const uint64_t b = dv + static_cast<uint32_t>(slot) * (kSlotBytes >> 4) + static_cast<uint32_t>(h * 4 * (2048 >> 4));
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_f16_ta(tm + 256u + 128u * t, tm + 128u * t + 32u * h + 8u * kk,
                                    b + static_cast<uint32_t>(kk * (2048 >> 4)), id_o, !(first && kk == 0));
                }
                __syncwarp();
            };
            using Tile0 = std::integral_constant<int, 0>;
            using Tile1 = std::integral_constant<int, 1>;
            const bool act0 = m_n0 > m_j0, act1 = m_n1 > m_j0;
            if (act0) wait(kBarQ, 0);
            wait(kBarFull, 0);
            if (act0) issue_s(Tile0{}, !act1);
            if (act1) {
                wait(kBarQ + 1, 0);
                issue_s(Tile1{}, true);
            }
            next_slot();
            uint32_t turn = 0;                   // parity of the tile's number
            for (int j = m_j0; ok && j < m_n; ++j, turn ^= 1u) {
                // `slot` is V of tile j; the next one is K of tile j + 1
                const int v_slot = slot;
                const uint32_t v_use = use;
                const bool more0 = j + 1 < m_n0, more1 = j + 1 < m_n1;
                wait(kBarFull + v_slot, v_use);
                if (j >= m_guard) {              // some row's limit falls in this tile
                    const int g = (j - m_guard) & 3;
                    if (leader) mbar_arrive(b0 + 8u * (kBarG + g));
                    __syncwarp();
                    wait(kBarV + g, ((j - m_guard) >> 2) & 1);
                }
                next_slot();
                const int k_slot = slot;
                const uint32_t k_use = use;
                if (j < m_n0) {
                    slot = v_slot;
                    wait(kBarP, turn);
                    issue_pv(Tile0{}, 0, j == m_j0);
                    wait(kBarP + 1, turn);
                    issue_pv(Tile0{}, 1, false);
                    if (ok && leader) {
                        umma_commit(b0 + 8u * kBarO);
                        if (j >= m_n1) umma_commit(b0 + 8u * (kBarEmpty + v_slot));
                    }
                    __syncwarp();
                    slot = k_slot;
                    if (more0) {
                        wait(kBarFull + k_slot, k_use);
                        issue_s(Tile0{}, !more1);
                    }
                }
                if (j < m_n1) {
                    slot = v_slot;
                    wait(kBarP + 2, turn);
                    issue_pv(Tile1{}, 0, j == m_j0);
                    wait(kBarP + 3, turn);
                    issue_pv(Tile1{}, 1, false);
                    if (ok && leader) {
                        umma_commit(b0 + 8u * (kBarO + 1));
                        umma_commit(b0 + 8u * (kBarEmpty + v_slot));
                    }
                    __syncwarp();
                    slot = k_slot;
                    if (more1) {
                        if (!more0) wait(kBarFull + k_slot, k_use);
                        issue_s(Tile1{}, true);
                    }
                }
                slot = k_slot;
                use = k_use;
                next_slot();
            }
            if (leader) umma_commit(b0 + 8u * kBarDrain);
            __syncwarp();
            wait_bar_warp(b0 + 8u * kBarDrain, 0, abort_flag);
        }
    } else if (warp == 10) {
        // ---- guard of V in the tiles where some row's limit falls
        for (int j = max(j0, w.guard); j < n; ++j) {
            const int i = 2 * (j - j0) + 1, s = i % kSlots;
            // (the MMA thread says when: a warp that waits for a phase of the ring's
            // barrier long before it begins would take an older phase for it)
            const uint32_t x4 = (j - w.guard) & 3, par = ((j - w.guard) >> 2) & 1;
            const bool ok = wait_bar(bar(kBarG + x4), par, abort_flag) &&
                            wait_bar(bar(kBarFull + s), (i / kSlots) & 1, abort_flag);
            if (!__all_sync(kFullMask, ok)) break;
            uint8_t* v = smem + kOffRing + s * kSlotBytes;
            const int rows = min(kTile, w.nk - j * kTile);   // of this sequence
            bool bad = false;
#pragma unroll 8
            for (int x = lane; x < kSlotBytes / 16; x += 32) {
                uint4* at = reinterpret_cast<uint4*>(v) + x;
                if (((x >> 3) & (kTile - 1)) < rows) bad |= any_special<T>(*at);
                else *at = make_uint4(0u, 0u, 0u, 0u);
            }
            if (bad) *special = 1;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarV + x4));
        }
        __syncwarp();
    } else {
        // ---- softmax of tile t, a thread per row
        const int t = warp >> 2, r = threadIdx.x & 127;
        const int i = w.pos[t] + r;
        const bool real = i < w.nq;
        const int seen = real ? seen_by(p, w.nq, w.nk, i) : 0;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + 128u * t, to = tmem + lanes + 256u + 128u * t;
        const float sc = p.scale_log2;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
#pragma unroll 1
        for (int j = j0; j < w.n[t]; ++j) {
            const int x = j - j0;
            ok = __all_sync(kFullMask, wait_bar(bar(kBarS + t), x & 1, abort_flag));
            if (!ok) break;
            tc_fence_after();
            float s[kTile];
            {
                uint32_t (&lo)[64] = *reinterpret_cast<uint32_t(*)[64]>(s);
                uint32_t (&hi)[64] = *reinterpret_cast<uint32_t(*)[64]>(s + 64);
                tmem_ld64(ts, lo);
                tmem_ld64(ts + 64u, hi);
                tmem_wait_ld();
            }
            const int lim = seen - j * kTile;
            if (__any_sync(kFullMask, lim < kTile)) {
#pragma unroll
                for (int c = 0; c < kTile; ++c) s[c] = c < lim ? s[c] : -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int c = 4; c < kTile; c += 8)
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = c + e + 4 < kTile ? fmaxf(mx[e], fmaxf(s[c + e], s[c + e + 4])) : fmaxf(mx[e], s[c + e]);
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
            if (__any_sync(kFullMask, top > m + kLazy)) {
                const float mn = fmaxf(m, top);
                const float a = fast_exp2(m - (mn == -INFINITY ? 0.f : mn));
                m = mn;
                l *= a;
                if (x > 0) {                     // O of the tiles before takes the new reference
                    ok = __all_sync(kFullMask, wait_bar(bar(kBarO + t), (x - 1) & 1, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < kHeadDim; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(to + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                        tmem_st32(to + c, o);
                    }
                    tmem_wait_st();
                }
            }
            const float mu = m == -INFINITY ? 0.f : m;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t pw[32];
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    const float a = fast_exp2(fmaf(s[64 * h + c], sc, -mu));
                    const float b = fast_exp2(fmaf(s[64 * h + c + 1], sc, -mu));
                    sum[c & 3] += a;
                    sum[(c & 3) + 1] += b;
                    pw[c / 2] = pack2<T>(a, b);
                }
                tmem_st32(ts + 32u * h, pw);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarP + 2 * t + h));
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        // ---- the result of a row, or its state (u, m, l) where the keys are split
        const int done = w.n[t] - j0;            // key tiles this query tile walked
        if (ok && done > 0) ok = __all_sync(kFullMask, wait_bar(bar(kBarO + t), (done - 1) & 1, abort_flag));
        tc_fence_after();
        // the guard ends before the last PV, which the wait above covered
        if (ok && *special != 0) {
            for (int rr = 0; rr < 32; ++rr) {
                const int ii = w.pos[t] + (warp & 3) * 32 + rr;
                if (ii < w.nq) plain_row<T>(p, w, t, ii, lane);
            }
        } else if (ok) {
            const bool empty = seen <= j0 * kTile || done <= 0;
            const float inv = empty ? 0.f : 1.f / l;
            const int64_t row = out_row(p, w, t, i);
            const int64_t at = row * p.n_splits + w.split;
#pragma unroll 1
            for (int c = 0; c < kHeadDim; c += 16) {
                float o[16];
                if (done > 0) {
                    tmem_ld16(to + c, *reinterpret_cast<uint32_t(*)[16]>(o));
                    tmem_wait_ld();
                }
                if (!real) continue;
                if (p.n_splits == 1) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = empty ? 0.f : o[e] * inv;
                    put_out<16>(p, row, c, o);
                } else {
                    float4* dst = reinterpret_cast<float4*>(p.ws_u + at * kHeadDim + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        dst[e] = empty ? make_float4(0.f, 0.f, 0.f, 0.f)
                                       : make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
            }
            if (real && p.n_splits == 1) {
                if (p.lse != nullptr) p.lse[row] = empty ? -INFINITY : (m + log2f(l)) * kLn2;
            } else if (real) {
                p.ws_m[at] = empty ? -INFINITY : m;
                p.ws_l[at] = empty ? 0.f : l;
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Joins the splits of each row: M = max m_s, out = sum 2^(m_s - M) u_s / L,
// L = sum 2^(m_s - M) l_s, in split order.  The blocks of the split kernel
// without its splits; a warp per row, 4 dims a lane.
__global__ void __launch_bounds__(256) fd_prompt_join_kernel(const PromptParams p) {
    grid_dependency_trigger();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Work w;
    find_work(p, static_cast<int64_t>(blockIdx.x) * p.n_splits, lane, w, false);
    if (w.b < 0) return;
    const int S = p.n_splits;
    for (int x = blockIdx.y * 8 + warp; x < 2 * kTile; x += 8 * gridDim.y) {
        const int t = x / kTile, i = w.pos[t] + x % kTile;
        if (i >= w.nq) continue;
        const int64_t row = out_row(p, w, t, i);
        float M = -INFINITY;
        for (int s = 0; s < S; ++s) M = fmaxf(M, p.ws_m[row * S + s]);
        const float mu = M == -INFINITY ? 0.f : M;
        float L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < S; ++s) {
            const float e = fast_exp2(p.ws_m[row * S + s] - mu);
            L = fmaf(e, p.ws_l[row * S + s], L);
            const float4 u = *reinterpret_cast<const float4*>(p.ws_u + (row * S + s) * kHeadDim + 4 * lane);
            o[0] = fmaf(e, u.x, o[0]);
            o[1] = fmaf(e, u.y, o[1]);
            o[2] = fmaf(e, u.z, o[2]);
            o[3] = fmaf(e, u.w, o[3]);
        }
        const bool empty = seen_by(p, w.nq, w.nk, i) == 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = empty ? 0.f : o[e] / L;
        put_out<4>(p, row, 4 * lane, o);
        if (lane == 0 && p.lse != nullptr) p.lse[row] = empty ? -INFINITY : (M + log2f(L)) * kLn2;
    }
}

template <typename T>
cudaError_t launch_prompt_t(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                            const PromptParams& p, int64_t tiles, cudaStream_t stream) {
    auto kern = fd_prompt_kernel<T>;
    static std::atomic<unsigned long long> configured_ctx{0};
    const unsigned long long ctx = current_context_id();
    if (ctx == 0 || configured_ctx.load(std::memory_order_acquire) != ctx) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        if (ctx != 0) configured_ctx.store(ctx, std::memory_order_release);
    }
    const int64_t units = tiles * p.head_units;
    cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>(units * p.n_splits)), dim3(kPromptThreads), kSmem, stream,
                               tmQ, tmK, tmV, p);
    if (e != cudaSuccess || p.n_splits == 1) return e;
    return launch_pdl(fd_prompt_join_kernel, dim3(static_cast<unsigned>(units), 8), dim3(256), 0, stream, p);
}

}  // namespace

cudaError_t launch_prompt(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV, const PromptParams& p,
                          bool bf16, int64_t tiles, cudaStream_t stream) {
    return bf16 ? launch_prompt_t<__nv_bfloat16>(tmQ, tmK, tmV, p, tiles, stream)
                : launch_prompt_t<__half>(tmQ, tmK, tmV, p, tiles, stream);
}

cudaError_t status_prompt(unsigned* value, bool clear) { return read_status_word(g_status, value, clear); }

}  // namespace fdk
