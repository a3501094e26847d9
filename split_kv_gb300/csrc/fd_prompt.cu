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
// An item is two query tiles of 128 rows and the key tiles of 128 they see.  The
// two tiles are the same positions of two heads of one group where the group is
// even (both then see the same keys, and a causal pair wastes half a tile on the
// diagonal, not one and a half), else 256 positions of one head.  Per key tile
// and query tile:
//   S[128 x 128] = Q K^T      8 MMAs of 16 dims, operands in shared memory
//   O[128 x 128] += P V       8 MMAs of 16 keys, P from tensor memory
// Warps 0-3 and 4-7 are the softmax of tile 0 and 1, a thread per row: it reads
// its row of S from tensor memory, writes P over it, in two halves so that PV
// starts on the first while the second is computed.  P is rounded to the inputs'
// type (the sums l keep the unrounded weights): a second product with the low
// parts, as the decode kernels have it, would be half as many MMAs again, where
// they bind the kernel, and the roundings' signs vary: 16-bit results are 1.2 to
// 1.3 times as far from the exact ones as out's own rounding alone puts them.
// Warp 8 streams K and V tiles with TMA through a ring of four 32 KB slots, warp
// 9 issues the MMAs: while one tile's softmax runs, the tensor cores work on the
// other tile's PV and next S.  Warp 10 guards the masked tiles (below), warp 11
// hands out the items.
// Tensor memory (512 columns): S/P of tile 0, 1 at 0, 128; O at 256, 384.
//
// Persistent: one CTA per SM takes items in turn.  The roles run ahead of each
// other: the next item's Q and K are loaded and its first S is computed while
// the softmax warps still write out the item before (only its first PV waits
// until they have read O).  Items come largest first (by the key tiles they
// see, over all sequences; found by bisection over the sequences' lengths) and
// are dealt out back and forth, which leaves the CTAs about equal sums.
//
// Masked places: scores past a row's limit are replaced by -inf before they
// are used, so what K holds there does not matter.  P is 0 there, but 0 * NaN
// is NaN: V's rows past the sequence's end are zeroed in shared memory in the
// one tile that has some (warp 10), and a row of O that comes out with an
// infinity or NaN is looked into: if a key that the row does not see but whose
// tile it walked has one in V, and the row is not NaN by right, it is computed
// again by a plain loop over the keys that it sees, once the CTA's items are done.
//
// Bound by the tensor cores when sequences are long: 4 * 128 flops per visible
// pair and head against 2 bytes per element read once.  16384 tokens, 32 / 8
// heads, causal, bf16: 1306 us, 1684 TFLOP/s (87 % of the measured burst rate of
// a library product); called for seconds, under the power cap, 1407 us, 1563
// TFLOP/s (91 % of the sustained one).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
constexpr int kSlots = 4;
constexpr int kSlotBytes = kTile * 256; // [128 x 64 dims] low half, high half
constexpr int kHalf = kSlotBytes / 2;
constexpr int kOffRing = 2 * kSlotBytes;
constexpr int kOffStage = kOffRing + kSlots * kSlotBytes;   // the epilogue's, 4 KB a softmax warp
constexpr int kOffBar = kOffStage + 8 * 4096;
constexpr int kOffWork = kOffBar + 384; // [kWorks] Work, 64 bytes each
constexpr int kWorks = 4;
constexpr int kOffMisc = kOffWork + kWorks * 64;    // tensor memory address, abort flag, redo flags
constexpr int kSorted = 128;            // batches up to this are handed out largest first
constexpr int kSmem = kOffMisc + 32 + 1024;
static_assert(kSmem <= 232448, "shared memory");
constexpr int kPromptThreads = 12 * 32;
constexpr float kLazy = 8.f;

// mbarriers, 8 bytes each from kOffBar.  Every role keeps its own counts of the
// uses of a barrier across items; a wait's parity is that of the use.
enum Bar : int {
    kBarQ = 0,                  // [2] a tile's Q landed
    kBarQE = 2,                 // [2] the last S of an item's tile done: Q's place is free (MMA commit)
    kBarFull = 4,               // [kSlots]
    kBarEmpty = kBarFull + kSlots,
    kBarS = kBarEmpty + kSlots, // [2] S written (MMA commit)
    kBarP = kBarS + 2,          // [2 tiles][2 halves] P written (and O rescaled), one arrival per warp
    kBarO = kBarP + 4,          // [2] an item's last PV done (MMA commit)
    kBarOF = kBarO + 2,         // [2] an item's O read out, one arrival per warp
    kBarG = kBarOF + 2,         // the V of a tile with a sequence's end landed
    kBarV = kBarG + 1,          // its rows past the end are zero
    kBarWF = kBarV + 1,         // [kWorks] an item is handed out
    kBarWE = kBarWF + kWorks,   // [kWorks] every role is done with it: producer, MMA, guard, 8 softmax warps
    kBarDrain = kBarWE + kWorks,// every MMA done
    kBars
};
static_assert(kBars * 8 <= 384, "barriers");

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    if (mbar_wait(bar, parity)) return true;
    atomicOr(&g_status, kStatusTimeoutBit);
    *abort_flag = 1;
    return false;
}

// A descriptor moved on by `off` 16-byte units (no operand crosses 256 KB, so
// the low word never carries).
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t off) {
    return (d & 0xffffffff00000000ull) | (static_cast<uint32_t>(d) + off);
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

// One item: two query tiles and the key tiles [j0, j1) of one sequence.
struct Work {
    int b;                      // -1: no more items
    int q0, k0, nq, nk;         // the sequence's rows
    int head[2], pos[2];        // of the two query tiles
    int n[2];                   // key tiles each sees, from 0 (<= j0: inactive)
    int j0, j1;                 // key tiles of this split
    int tail;                   // the key tile where the sequence ends, past the last one if that is full
    int split;
};
static_assert(sizeof(Work) <= 64, "work");

__device__ __forceinline__ int seen_by(const PromptParams& p, int nq, int nk, int i) {
    return p.causal ? min(max(nk - nq + 1 + i, 0), nk) : nk;
}

__device__ __forceinline__ int span_shift(const PromptParams& p) { return p.pair_heads ? 7 : 8; }
static_assert(kTile == 1 << 7, "span_shift");

// Whether a sequence's offsets hold; its numbers of queries and keys.
__device__ __forceinline__ bool read_seq(const PromptParams& p, const int* cq, const int* ck, int& q0, int& nq, int& k0,
                                         int& nk) {
    q0 = cq[0];
    k0 = ck[0];
    nq = cq[1] - q0;
    nk = ck[1] - k0;
    return q0 >= 0 && cq[1] >= q0 && cq[1] <= p.total_q && k0 >= 0 && ck[1] >= k0 && ck[1] <= p.total_k;
}

// The item (tile `tile` of the sequence in w, head unit, split): the rest of w.
__device__ __forceinline__ void fill_work(const PromptParams& p, int tile, int unit, int split, Work& w) {
    w.split = split;
    int most = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        w.head[t] = p.pair_heads ? 2 * unit + t : unit;
        w.pos[t] = (tile << span_shift(p)) + (p.pair_heads ? 0 : t * kTile);
        const int last = min(w.pos[t] + kTile, w.nq) - 1;
        const int keys = last >= w.pos[t] ? seen_by(p, w.nq, w.nk, last) : 0;
        w.n[t] = (keys + kTile - 1) / kTile;
        most = max(most, w.n[t]);
    }
    w.j0 = 0;
    w.j1 = most;
    if (p.n_splits > 1) {
        const int each = most / p.n_splits, more = most % p.n_splits;
        w.j0 = split * each + min(split, more);
        w.j1 = w.j0 + each + (split < more ? 1 : 0);
    }
    w.n[0] = min(w.n[0], w.j1);
    w.n[1] = min(w.n[1], w.j1);
    w.tail = w.nk % kTile != 0 ? w.nk / kTile : INT32_MAX;
}

// Hands out items by their rank, one warp.  Ranks count (query tile, head unit,
// split), splits fastest.  Up to kSorted sequences (sorted): tiles in order of
// the key tiles they see, most first, the lanes holding the sequences' lengths;
// beyond: as the sequences come, each one's last tile first (ranks have to
// ascend).
struct Dealer {
    static constexpr int kPer = kSorted / 32;
    bool sorted;
    int q0[kPer], nq[kPer], k0[kPer], nk[kPer];     // sorted: sequences 32 c + lane (lengths 0: none)
    int top;                    // sorted: the most key tiles any sequence has
    int base, before;           // else: the chunk of 32 sequences looked at, tiles before it

    // tiles of a sequence that see at least `need` key tiles
    __device__ __forceinline__ int tiles_seeing(const PromptParams& p, int n, int m, int need) const {
        const int shift = span_shift(p), round = (1 << shift) - 1, tiles = (n + round) >> shift;
        if (need <= 0) return tiles;
        const int x = (need - 1) * kTile + 1;       // keys
        if (m < x) return 0;
        if (!p.causal) return tiles;
        const int rows = x - m + n;                  // the first so many rows see fewer, but for the last of them
        return rows <= 0 ? tiles : tiles - (((rows + round) >> shift) - 1);
    }
    __device__ __forceinline__ int all_seeing(const PromptParams& p, int need) const {
        int sum = 0;
#pragma unroll
        for (int c = 0; c < kPer; ++c) sum += tiles_seeing(p, nq[c], nk[c], need);
        return __reduce_add_sync(kFullMask, sum);
    }
    __device__ __forceinline__ void start(const PromptParams& p, int lane, bool report) {
        sorted = p.batch <= kSorted;
        base = before = top = 0;
        if (!sorted) return;
        int most = 0;
        bool bad = false;
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
            const int b = 32 * c + lane;
            q0[c] = nq[c] = k0[c] = nk[c] = 0;
            if (b < p.batch && !read_seq(p, p.cu_q + b, p.cu_k + b, q0[c], nq[c], k0[c], nk[c])) {
                bad = true;
                nq[c] = nk[c] = 0;
            }
            most = max(most, (nk[c] + kTile - 1) / kTile);
        }
        top = __reduce_max_sync(kFullMask, most);
        if (report && bad) atomicOr(&g_status, kStatusSeqlenBit);
    }
    // Among the sequences b, b + lane.. of one chunk with `mine` tiles each, the
    // one of tile idx - before; false: not in this chunk.
    __device__ __forceinline__ bool find(int idx, int mine, int& src, int& i) {
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFullMask, upto, o);
            if ((threadIdx.x & 31) >= o) upto += y;
        }
        const unsigned hit = __ballot_sync(kFullMask, idx - before < upto);
        if (hit == 0) {
            before += __shfl_sync(kFullMask, upto, 31);
            return false;
        }
        src = __ffs(hit) - 1;
        i = idx - before - __shfl_sync(kFullMask, upto - mine, src);
        return true;
    }
    __device__ __forceinline__ void take(Work& w, int b, int src, int q, int n, int k, int m) {
        w.b = b + src;
        w.q0 = __shfl_sync(kFullMask, q, src);
        w.nq = __shfl_sync(kFullMask, n, src);
        w.k0 = __shfl_sync(kFullMask, k, src);
        w.nk = __shfl_sync(kFullMask, m, src);
    }
    // (every lane gets the item; b = -1 past the last one)
    __device__ __forceinline__ void item(const PromptParams& p, uint32_t rank, int lane, Work& w) {
        int split = 0;
        if (p.n_splits > 1) {
            split = static_cast<int>(rank % p.n_splits);
            rank /= p.n_splits;
        }
        const int unit = static_cast<int>(rank % p.head_units);
        const int at = static_cast<int>(rank / p.head_units);   // the tile's rank
        w.b = -1;
        int src, i;
        if (!sorted) {
            for (; base < p.batch; base += 32) {
                int q = 0, n = 0, k = 0, m = 0;
                const bool ok = base + lane < p.batch && read_seq(p, p.cu_q + base + lane, p.cu_k + base + lane, q, n, k, m);
                const int mine = ok ? tiles_seeing(p, n, m, 0) : 0;
                if (find(at, mine, src, i)) {
                    take(w, base, src, q, n, k, m);
                    fill_work(p, __shfl_sync(kFullMask, mine, src) - 1 - i, unit, split, w);
                    return;
                }
            }
            return;
        }
        if (at >= all_seeing(p, 0)) return;
        int need = 0, hi = top + 1;                      // key tiles of the tile with that rank
        while (hi - need > 1) {
            const int mid = (need + hi) >> 1;
            if (all_seeing(p, mid) > at) need = mid;
            else hi = mid;
        }
        const int idx = at - all_seeing(p, need + 1);    // among those that see exactly `need`
        before = 0;
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
            const int from = tiles_seeing(p, nq[c], nk[c], need), mine = from - tiles_seeing(p, nq[c], nk[c], need + 1);
            if (w.b < 0 && find(idx, mine, src, i)) {
                take(w, 32 * c, src, q0[c], nq[c], k0[c], nk[c]);
                const int tile0 = tiles_seeing(p, nq[c], nk[c], 0) - from;   // the first of these tiles
                fill_work(p, __shfl_sync(kFullMask, tile0, src) + i, unit, split, w);
            }
        }
    }
    // unsorted: offsets of every sequence
    __device__ __forceinline__ void report_all(const PromptParams& p, int lane) const {
        if (sorted) return;
        for (int c = lane; c < p.batch; c += 32) {
            int q, n, k, m;
            if (!read_seq(p, p.cu_q + c, p.cu_k + c, q, n, k, m)) atomicOr(&g_status, kStatusSeqlenBit);
        }
    }
};

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

// Four consecutive dims of a row of out, from dim d.
__device__ __forceinline__ void put_out4(const PromptParams& p, int64_t row, int d, const float (&o)[4]) {
    const int64_t at = row * kHeadDim + d;
    if (p.out_dtype == 2) {
        float* dst = static_cast<float*>(p.out) + at;
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[e] = o[e];
        return;
    }
    const bool half = p.out_dtype == 0;
    const uint32_t a = half ? pack2<__half>(o[0], o[1]) : pack2<__nv_bfloat16>(o[0], o[1]);
    const uint32_t b = half ? pack2<__half>(o[2], o[3]) : pack2<__nv_bfloat16>(o[2], o[3]);
    uint16_t* dst = static_cast<uint16_t*>(p.out) + at;
    if (p.out_vec) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(a, b);
    } else {
        dst[0] = static_cast<uint16_t>(a);
        dst[1] = static_cast<uint16_t>(a >> 16);
        dst[2] = static_cast<uint16_t>(b);
        dst[3] = static_cast<uint16_t>(b >> 16);
    }
}

// Up to four rows again, by one warp, each over the keys that it sees in the
// item's key tiles (lim: one past the last; at most j0: no such row): lane l
// holds dims 4l .. 4l + 3.  Four keys at a time, so that their products and
// the exchanges that add them up run beside each other.
template <typename T>
__device__ __noinline__ void plain_rows(const PromptParams& p, const Work& w, int t, const int (&row)[4], int lane) {
    const int j0 = w.j0 * kTile, g = w.head[t] / p.group;
    const T* kp = static_cast<const T*>(p.k) + static_cast<int64_t>(w.k0) * p.k_st + g * p.k_sh + 4 * lane;
    const T* vp = static_cast<const T*>(p.v) + static_cast<int64_t>(w.k0) * p.v_st + g * p.v_sh + 4 * lane;
    float q[4][4], o[4][4], m[4], l[4];
    int lim[4], most = j0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        lim[r] = row[r] >= 0 ? min(w.j1 * kTile, seen_by(p, w.nq, w.nk, row[r])) : 0;
        most = max(most, lim[r]);
        uint2 qw = make_uint2(0u, 0u);
        if (row[r] >= 0)
            qw = *reinterpret_cast<const uint2*>(static_cast<const T*>(p.q) + (static_cast<int64_t>(w.q0) + row[r]) * p.q_st +
                                                 w.head[t] * p.q_sh + 4 * lane);
        const float2 a = unpack2<T>(qw.x), b = unpack2<T>(qw.y);
        q[r][0] = a.x, q[r][1] = a.y, q[r][2] = b.x, q[r][3] = b.y;
        o[r][0] = o[r][1] = o[r][2] = o[r][3] = 0.f;
        m[r] = -INFINITY;
        l[r] = 0.f;
    }
    uint2 kw[4], vw[4];                            // four keys ahead
    auto load = [&](int j) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            kw[x] = vw[x] = make_uint2(0u, 0u);
            if (j + x < most) {
                kw[x] = *reinterpret_cast<const uint2*>(kp + (j + x) * p.k_st);
                vw[x] = *reinterpret_cast<const uint2*>(vp + (j + x) * p.v_st);
            }
        }
    };
    load(j0);
#pragma unroll 1
    for (int j = j0; j < most; j += 4) {
        float k[4][4], v[4][4], s[4][4];           // [key], [key], [key][row]
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float2 ka = unpack2<T>(kw[x].x), kb = unpack2<T>(kw[x].y), va = unpack2<T>(vw[x].x), vb = unpack2<T>(vw[x].y);
            k[x][0] = ka.x, k[x][1] = ka.y, k[x][2] = kb.x, k[x][3] = kb.y;
            v[x][0] = va.x, v[x][1] = va.y, v[x][2] = vb.x, v[x][3] = vb.y;
        }
        load(j + 4);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                s[x][r] = fmaf(q[r][0], k[x][0], fmaf(q[r][1], k[x][1], fmaf(q[r][2], k[x][2], q[r][3] * k[x][3])));
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1)
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int r = 0; r < 4; ++r) s[x][r] += __shfl_xor_sync(kFullMask, s[x][r], d);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float mn = m[r];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                s[x][r] = j + x < lim[r] ? s[x][r] * p.scale_log2 : -INFINITY;
                mn = fmaxf(mn, s[x][r]);
            }
            const float mu = mn == -INFINITY ? 0.f : mn, a = fast_exp2(m[r] - mu);
            m[r] = mn;
            l[r] *= a;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][e] *= a;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (j + x < lim[r]) {              // (the same for the whole warp)
                    const float e = fast_exp2(s[x][r] - mu);
                    l[r] += e;
#pragma unroll
                    for (int d = 0; d < 4; ++d) o[r][d] = fmaf(e, v[x][d], o[r][d]);
                }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (lim[r] <= j0) continue;
        const int64_t to = out_row(p, w, t, row[r]);
        if (p.n_splits == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][e] /= l[r];
            put_out4(p, to, 4 * lane, o[r]);
            if (lane == 0 && p.lse != nullptr) p.lse[to] = (m[r] + __log2f(l[r])) * kLn2;
        } else {
            const int64_t at = to * p.n_splits + w.split;
            *reinterpret_cast<float4*>(p.ws_u + at * kHeadDim + 4 * lane) = make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
            if (lane == 0) {
                p.ws_m[at] = m[r];
                p.ws_l[at] = l[r];
            }
        }
    }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Four running maxima over 64 scores (set by the first call).
template <bool FIRST>
__device__ __forceinline__ void row_max(const uint32_t (&s)[64], float (&mx)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a = __uint_as_float(s[e]), b = __uint_as_float(s[e + 4]);
        mx[e] = FIRST ? fmaxf(a, b) : max3(mx[e], a, b);
    }
#pragma unroll
    for (int c = 8; c < 64; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], __uint_as_float(s[c + e]), __uint_as_float(s[c + e + 4]));
}

// The weights 2^(s sc + b) of 64 scores as 16-bit pairs, and their 32-bit sums;
// two at a time where the arithmetic has a form for it.
template <typename T>
__device__ __forceinline__ void weights(const uint32_t (&s)[64], float sc, float b, uint32_t (&pw)[32], float2 (&sum)[2]) {
    const float2 sc2 = make_float2(sc, sc), b2 = make_float2(b, b);
#pragma unroll
    for (int c = 0; c < 64; c += 2) {
        const float2 t = __ffma2_rn(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, b2);
        const float2 e = make_float2(fast_exp2(t.x), fast_exp2(t.y));
        sum[(c >> 1) & 1] = __fadd2_rn(sum[(c >> 1) & 1], e);
        pw[c / 2] = pack2<T>(e.x, e.y);
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

// Whether V has an infinity or NaN in a key tile that some row of this query
// tile does not see whole (one warp).
template <typename T>
__device__ __noinline__ bool hidden_special(const PromptParams& p, const Work& w, int t, int lane) {
    const int first = max(w.j0 * kTile, seen_by(p, w.nq, w.nk, w.pos[t]) / kTile * kTile);
    const int last = min(w.n[t] * kTile, w.nk);
    const int g = w.head[t] / p.group;
    bool bad = false;
    for (int j = first + (lane >> 4); j < last; j += 2)
        bad |= any_special<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) + (static_cast<int64_t>(w.k0) + j) * p.v_st +
                                                              g * p.v_sh + 8 * (lane & 15)));
    return __any_sync(kFullMask, bad);
}

// Rank of the k-th item of this CTA: back and forth over the CTAs.
__device__ __forceinline__ uint32_t item_rank(int k) {
    return k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// One item's rows of one warp (32 of query tile t, from 32 * quarter on) that an
// infinity or NaN of V reached which they do not see.  Lane l looks through
// dims 4l .. 4l + 3 for the last special value of the key tiles that some row
// does not see whole, and for the key from which on a row's result is NaN by
// right: the first NaN, or the later of the first +inf and -inf.  A row is
// computed again if a dim of it has the one hidden and not yet the other; so
// where V is NaN throughout hardly any is, and a first NaN in the middle costs
// the rows of one tile.
template <typename T>
__device__ __noinline__ void redo_item(const PromptParams& p, const Work& w, int t, int quarter, int lane) {
    constexpr uint32_t inf = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    const int from = w.j0 * kTile;
    const int first = max(from, seen_by(p, w.nq, w.nk, w.pos[t]) / kTile * kTile), last = min(w.n[t] * kTile, w.nk);
    const T* vp = static_cast<const T*>(p.v) + static_cast<int64_t>(w.k0) * p.v_st + w.head[t] / p.group * p.v_sh + 4 * lane;
    int nan_at[4], up_at[4], down_at[4], hidden[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        nan_at[d] = up_at[d] = down_at[d] = INT32_MAX;
        hidden[d] = -1;
    }
    auto look = [&](int j, const uint2& vw, bool masked) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const uint32_t x = ((d < 2 ? vw.x : vw.y) >> (16 * (d & 1))) & 0xffffu, a = x & 0x7fffu;
            if (a < inf) continue;
            if (masked) hidden[d] = max(hidden[d], j);
            if (a > inf) nan_at[d] = min(nan_at[d], j);
            else if (x == a) up_at[d] = min(up_at[d], j);
            else down_at[d] = min(down_at[d], j);
        }
    };
    auto nan_from = [&](int d) { return min(nan_at[d], max(up_at[d], down_at[d])); };
#pragma unroll 4
    for (int j = first; j < last; ++j) look(j, *reinterpret_cast<const uint2*>(vp + j * p.v_st), true);
#pragma unroll 1
    for (int j = from; j < first; j += 8) {          // (whole tiles)
        bool known = true;
#pragma unroll
        for (int d = 0; d < 4; ++d) known = known && (hidden[d] < 0 || nan_from(d) < first);
        if (__all_sync(kFullMask, known)) break;
        uint2 vw[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) vw[x] = *reinterpret_cast<const uint2*>(vp + (j + x) * p.v_st);
#pragma unroll
        for (int x = 0; x < 8; ++x) look(j + x, vw[x], false);
    }
    int row[4], rows = 0;
    const int i0 = w.pos[t] + 32 * quarter;
#pragma unroll 1
    for (int i = i0; i < i0 + 32; ++i) {
        bool reached = false;
        if (i < w.nq) {
            const int seen = seen_by(p, w.nq, w.nk, i);
#pragma unroll
            for (int d = 0; d < 4; ++d) reached = reached || (seen > from && hidden[d] >= seen && nan_from(d) >= seen);
        }
        const bool again = __any_sync(kFullMask, reached);
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (again && x == rows) row[x] = i;
        rows += again;
        if (rows == 4 || (rows > 0 && i == i0 + 31)) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (x >= rows) row[x] = -1;
            plain_rows<T>(p, w, t, row, lane);
            rows = 0;
        }
    }
}

// All items of the CTA again, for such rows.  Runs when they are done: nothing
// waits for this warp but the CTA's end, however long its rows take.  16384
// tokens, 32 / 8 heads: 17 ms with one NaN in the middle of one KV head, 2.2
// with NaN throughout, 254 with +inf throughout (every row again), 1.3 without.
template <typename T>
__device__ __noinline__ void redo_rows(const PromptParams& p, int t, int quarter, int lane) {
    Dealer dealer;
    dealer.start(p, lane, false);
    for (int k = 0;; ++k) {
        Work w;
        dealer.item(p, item_rank(k), lane, w);
        if (w.b < 0) break;
        if (w.n[t] > w.j0 && hidden_special<T>(p, w, t, lane)) redo_item<T>(p, w, t, quarter, lane);
    }
}

// 16 bytes of output at an address that has only its element's alignment
__device__ __forceinline__ void put_odd(uint8_t* dst, const uint4& q, bool wide) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (wide) {
            reinterpret_cast<uint32_t*>(dst)[e] = w[e];
        } else {
            reinterpret_cast<uint16_t*>(dst)[2 * e] = static_cast<uint16_t>(w[e]);
            reinterpret_cast<uint16_t*>(dst)[2 * e + 1] = static_cast<uint16_t>(w[e] >> 16);
        }
    }
}

// A warp's 32 rows of O, times inv, to rows at0, at0 + row_step, .. of out or of
// the states u: 64 (16-bit) or 32 (32-bit) dims at a time, each lane's row to the
// warp's staging area, 128 bytes a row, swizzled; from there eight lanes a row to
// memory (a lane writing its own row touches 32 lines a store: 3.4 us an item).
// Returns NaN if an infinity or NaN was among the lane's row, else 0.
// (One body for both widths: a second one, or a call, cost the softmax loop
// its registers, and 18 % of the kernel's rate.)
__device__ __forceinline__ float write_rows(const PromptParams& p, uint8_t* stage, uint32_t to, int64_t at0,
                                            int64_t row_step, int rows, bool done, bool empty, float inv, int lane) {
    const bool wide = p.n_splits > 1 || p.out_dtype == 2;
    const int64_t bytes = wide ? 4 : 2;
    uint8_t* dst = static_cast<uint8_t*>(p.n_splits > 1 ? static_cast<void*>(p.ws_u) : p.out) +
                   at0 * kHeadDim * bytes + (lane & 7) * 16;
    const int64_t step = row_step * kHeadDim * bytes;
    const float2 inv2 = make_float2(inv, inv), none = make_float2(0.f, 0.f);
    const bool some_empty = __any_sync(kFullMask, empty);
    float2 odd = none;
#pragma unroll 1
    for (int c = 0; c < kHeadDim; c += 32) {
        uint32_t o[32];
        if (done) {
            tmem_ld32(to + c, o);
            tmem_wait_ld();
        }
        if (some_empty) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = empty ? 0u : o[e];
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            const float2 f = __fmul2_rn(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), inv2);
            odd = __ffma2_rn(f, none, odd);
            o[e] = __float_as_uint(f.x);
            o[e + 1] = __float_as_uint(f.y);
        }
        int unit = 0;
        if (!wide) {
            unit = (c & 32) >> 3;
            if (p.out_dtype == 0) {
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = pack2<__half>(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    o[e] = pack2<__nv_bfloat16>(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
            }
        }
        uint8_t* mine = stage + lane * 128;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            *reinterpret_cast<uint4*>(mine + (((unit + u) ^ (lane & 7)) << 4)) =
                make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
        if (wide) {
#pragma unroll
            for (int u = 4; u < 8; ++u)
                *reinterpret_cast<uint4*>(mine + ((u ^ (lane & 7)) << 4)) =
                    make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
        }
        if (!wide && (c & 32) == 0) continue;
        __syncwarp();
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            const int rr = 4 * y + (lane >> 3);
            const uint4 q = *reinterpret_cast<const uint4*>(stage + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
            if (rr < rows) {
                if (p.n_splits > 1 || p.out_vec) *reinterpret_cast<uint4*>(dst + rr * step) = q;
                else put_odd(dst + rr * step, q, wide);
            }
        }
        dst += 128;
        __syncwarp();
    }
    return odd.x + odd.y;
}

template <typename T>
__global__ void __launch_bounds__(kPromptThreads, 1)
    fd_prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PromptParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t bar0 = smem_u32(smem + kOffBar);
    auto bar = [&](int i) { return bar0 + 8u * i; };
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
    auto work_at = [&](int k) { return reinterpret_cast<Work*>(smem + kOffWork + 64 * (k % kWorks)); };

    if (threadIdx.x == 256) {
        for (int i = 0; i < kBars; ++i)
            mbar_init(bar(i), (i >= kBarP && i < kBarP + 4) || (i >= kBarOF && i < kBarOF + 2) ? 4
                              : i >= kBarWE && i < kBarWE + kWorks                             ? 11
                                                                                               : 1);
        *abort_flag = 0;
        *reinterpret_cast<volatile uint64_t*>(smem + kOffMisc + 8) = 0;   // the softmax warps' flags to redo rows
        fence_barrier_init();
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == 1) tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
    grid_dependency_trigger();
    grid_dependency_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*const_cast<uint32_t*>(tmem_slot));

    // The softmax warps take registers from the others: 256 * 208 + 128 * 88 =
    // 384 * 168, what the launch has.
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 8) {
            // ---- producer: Q of both tiles, then K and V of each key tile
            if (lane == 0) {
                auto load = [&](uint8_t* dst, const CUtensorMap* map, uint32_t b, int row, int head) {
                    mbar_arrive_expect_tx(b, kSlotBytes);
                    tma_load_4d(smem_u32(dst), map, b, 0, row, head, 0);
                    tma_load_4d(smem_u32(dst + kHalf), map, b, 64, row, head, 0);
                };
                int i = 0, nq[2] = {0, 0};           // ring entries, Q tiles loaded
                bool ok = true;
                auto tile = [&](const CUtensorMap* map, int row, int head) {
                    const int s = i % kSlots;
                    if (i >= kSlots) ok = ok && wait_bar(bar(kBarEmpty + s), (i / kSlots - 1) & 1, abort_flag);
                    if (!ok || *abort_flag) {
                        ok = false;
                        return;
                    }
                    load(smem + kOffRing + s * kSlotBytes, map, bar(kBarFull + s), row, head);
                    ++i;
                };
                auto load_q = [&](const Work& w, int t) {
                    if (!ok || w.n[t] <= w.j0) return;
                    if (nq[t] > 0) ok = wait_bar(bar(kBarQE + t), (nq[t] - 1) & 1, abort_flag);
                    if (!ok) return;
                    load(smem + t * kSlotBytes, &tmQ, bar(kBarQ + t), w.q0 + w.pos[t], w.head[t]);
                    ++nq[t];
                };
                for (int k = 0; ok; ++k) {
                    ok = wait_bar(bar(kBarWF + k % kWorks), (k / kWorks) & 1, abort_flag);
                    if (!ok) break;
                    const Work w = *work_at(k);
                    mbar_arrive(bar(kBarWE + k % kWorks));
                    if (w.b < 0) break;
                    const int n = max(w.n[0], w.n[1]), g = w.head[0] / p.group;
                    if (n <= w.j0) continue;
                    // the first K before the Qs: its slot is free sooner than theirs
                    tile(&tmK, w.k0 + w.j0 * kTile, g);
                    load_q(w, 0);
                    load_q(w, 1);
                    for (int j = w.j0; ok && j < n; ++j) {
                        tile(&tmV, w.k0 + j * kTile, g);
                        if (ok && j + 1 < n) tile(&tmK, w.k0 + (j + 1) * kTile, g);
                    }
                }
                // nothing may be in flight towards this CTA when it exits
                for (int t = 0; t < 2; ++t)
                    if (nq[t] > 0) wait_bar(bar(kBarQ + t), (nq[t] - 1) & 1, abort_flag);
                for (int x = max(0, i - kSlots); x < i; ++x) wait_bar(bar(kBarFull + x % kSlots), (x / kSlots) & 1, abort_flag);
            }
            __syncwarp();
        } else if (warp == 9) {
            // ---- MMA issue: the whole warp walks the tiles, one elected lane issues.
            // Everything the MMAs take is warp-uniform for the compiler (the
            // shuffles), so that descriptors stay in uniform registers: from inside
            // a one-lane branch the MMAs' issue bound the kernel (16384 tokens, 32 / 8
            // heads: 2386 us against 1384).
            constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
            constexpr uint32_t id_s = umma_idesc(kBf16, false), id_o = umma_idesc(kBf16, true);
            const uint32_t sm = uniform(smem_u32(smem)), b0 = uniform(bar0);
            const uint64_t dq = umma_desc_sw128(sm, 16, 1024);
            const uint64_t dk = umma_desc_sw128(sm + kOffRing, 16, 1024);
            const uint64_t dv = umma_desc_sw128(sm + kOffRing, kHalf, 1024);
            const bool leader = elect_one();
            bool ok = true;
            auto wait = [&](int i, uint32_t parity) {
                if (ok) ok = wait_bar_warp(b0 + 8u * i, parity, abort_flag);
            };
            auto commit = [&](int i) { umma_commit(b0 + 8u * i); };
            int slot = 0;                            // ring slot of the entry at hand, and the parity of its use
            uint32_t use = 0;
            auto next_slot = [&]() {
                if (++slot == kSlots) {
                    slot = 0;
                    use ^= 1u;
                }
            };
            uint32_t turn0 = 0, turn1 = 0;           // parities: P of tile 0, 1,
            int items0 = 0, items1 = 0;              // items in which tile 0, 1 ran
            int tails = 0;                           // tiles with a sequence's end
            // (by the elected lane) S of tile t from the K at `ks`
            auto issue_s = [&](auto tile, int ks) {
                constexpr int t = decltype(tile)::value;
                const uint64_t b = dk + static_cast<uint32_t>(ks) * (kSlotBytes >> 4);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32u) >> 4;
                    umma_f16(tmem + 128u * t, desc_at(dq, t * (kSlotBytes >> 4) + off), desc_at(b, off), id_s, kk > 0);
                }
            };
            // One tile's turn: PV(j) from the V at `vs`, each half of P as it comes, then
            // (`more`) S(j + 1) from the K at `ks`.  MMAs run in issue order, so S
            // overwrites P only after PV has read it, and a softmax warp that sees S(j + 1)
            // done knows that PV(j) is: O is signalled apart only at an item's end.
            // last_v, last_k: no other tile reads the slot after this.
            auto turn = [&](auto tile, int vs, int ks, uint32_t parity, bool first, bool more, bool last_v, bool last_k,
                            bool end) {
                constexpr int t = decltype(tile)::value;
                const uint64_t b = dv + static_cast<uint32_t>(vs) * (kSlotBytes >> 4);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    wait(kBarP + 2 * t + h, parity);
                    if (!ok) return;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
                            umma_f16_ta(tmem + 256u + 128u * t, tmem + 128u * t + 8u * kk, desc_at(b, kk * (2048 >> 4)),
                                        id_o, !(first && kk == 0));
                        if (h == 1) {
                            if (more) {
                                issue_s(tile, ks);
                                commit(kBarS + t);
                                if (last_k) commit(kBarEmpty + ks);
                                if (end) commit(kBarQE + t);
                            } else {
                                commit(kBarO + t);
                            }
                            if (last_v) commit(kBarEmpty + vs);
                        }
                    }
                    __syncwarp();
                }
            };
            using Tile0 = std::integral_constant<int, 0>;
            using Tile1 = std::integral_constant<int, 1>;
            for (int k = 0; ok; ++k) {
                wait(kBarWF + k % kWorks, (k / kWorks) & 1);
                if (!ok) break;
                const Work* w = work_at(k);
                const int n0 = uniform(w->n[0]), n1 = uniform(w->n[1]), j0 = uniform(w->j0), tail = uniform(w->tail);
                const bool stop = uniform(w->b) < 0;
                if (leader) mbar_arrive(b0 + 8u * (kBarWE + k % kWorks));
                __syncwarp();
                if (stop) break;
                const int n = max(n0, n1);
                if (n <= j0) continue;
                const bool act0 = n0 > j0, act1 = n1 > j0;
                wait(kBarFull + slot, use);
                if (act0) {
                    wait(kBarQ, items0 & 1);
                    tc_fence_after();
                    if (ok && leader) {
                        issue_s(Tile0{}, slot);
                        commit(kBarS);
                        if (!act1) commit(kBarEmpty + slot);
                        if (j0 + 1 >= n0) commit(kBarQE);
                    }
                    __syncwarp();
                }
                if (act1) {
                    wait(kBarQ + 1, items1 & 1);
                    tc_fence_after();
                    if (ok && leader) {
                        issue_s(Tile1{}, slot);
                        commit(kBarS + 1);
                        commit(kBarEmpty + slot);
                        if (j0 + 1 >= n1) commit(kBarQE + 1);
                    }
                    __syncwarp();
                }
                next_slot();
                for (int j = j0; ok && j < n; ++j) {
                    // `slot` is V of tile j, the entry behind it K of tile j + 1
                    const int vs = slot;
                    const bool more0 = j + 1 < n0, more1 = j + 1 < n1;
                    wait(kBarFull + vs, use);
                    if (j == tail) {                 // the sequence ends in this tile
                        if (leader) mbar_arrive(b0 + 8u * kBarG);
                        __syncwarp();
                        wait(kBarV, tails & 1);
                        ++tails;
                    }
                    next_slot();
                    const int ks = slot;
                    if (more0 || more1) {
                        wait(kBarFull + ks, use);
                        next_slot();
                    }
                    if (j == j0) {                   // O's places: read out by the softmax warps
                        if (act0 && items0 > 0) wait(kBarOF, (items0 - 1) & 1);
                        if (act1 && items1 > 0) wait(kBarOF + 1, (items1 - 1) & 1);
                    }
                    if (j < n0) turn(Tile0{}, vs, ks, turn0, j == j0, more0, j >= n1, !more1, j + 2 >= n0), turn0 ^= 1u;
                    if (j < n1) turn(Tile1{}, vs, ks, turn1, j == j0, more1, true, true, j + 2 >= n1), turn1 ^= 1u;
                }
                items0 += act0;
                items1 += act1;
            }
            if (leader) commit(kBarDrain);
            __syncwarp();
            wait_bar_warp(b0 + 8u * kBarDrain, 0, abort_flag);
        } else if (warp == 10) {
            // ---- zeroes V's rows past a sequence's end
            bool ok = true;
            int tails = 0, i = 0;                    // tiles with an end, ring entries before the item
            for (int k = 0; ok; ++k) {
                ok = wait_bar_warp(bar(kBarWF + k % kWorks), (k / kWorks) & 1, abort_flag);
                if (!ok) break;
                const Work w = *work_at(k);
                if (w.b < 0) break;
                const int n = max(w.n[0], w.n[1]);
                if (w.tail >= w.j0 && w.tail < n) {
                    const int e = i + 2 * (w.tail - w.j0) + 1;
                    // (the MMA warp says when: a warp that waits for a phase of the ring's
                    // barrier long before it begins would take an older phase for it)
                    ok = wait_bar_warp(bar(kBarG), tails & 1, abort_flag) &&
                         wait_bar_warp(bar(kBarFull + e % kSlots), (e / kSlots) & 1, abort_flag);
                    if (!ok) break;
                    uint8_t* v = smem + kOffRing + e % kSlots * kSlotBytes;
                    for (int r = w.nk % kTile + (lane >> 3); r < kTile; r += 4)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            *reinterpret_cast<uint4*>(v + h * kHalf + r * 128 + (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBarV));
                    ++tails;
                }
                i += 2 * max(n - w.j0, 0);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarWE + k % kWorks));
            }
            __syncwarp();
        } else if (warp == 11) {
            // ---- dealer
            Dealer dealer;
            dealer.start(p, lane, blockIdx.x == 0);
            bool ok = true;
            for (int k = 0; ok; ++k) {
                if (k >= kWorks) ok = wait_bar_warp(bar(kBarWE + k % kWorks), (k / kWorks - 1) & 1, abort_flag);
                if (!ok) break;
                Work w;
                dealer.item(p, item_rank(k), lane, w);
                if (lane == 0) {
                    *work_at(k) = w;
                    mbar_arrive(bar(kBarWF + k % kWorks));
                }
                __syncwarp();
                if (w.b < 0) break;
            }
            if (blockIdx.x == 0) dealer.report_all(p, lane);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ---- softmax of tile t, a thread per row
        const int t = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + 128u * t, to = tmem + lanes + 256u + 128u * t;
        const float sc = p.scale_log2;
        volatile uint8_t* redo = smem + kOffMisc + 8 + warp;   // (a register less in the loop)
        uint32_t walked = 0, ran = 0;            // key tiles, and items with any: parities of S and O
        bool ok = true;
        for (int k = 0; ok; ++k) {
            ok = __all_sync(kFullMask, wait_bar(bar(kBarWF + k % kWorks), (k / kWorks) & 1, abort_flag));
            if (!ok) break;
            const Work& w = *work_at(k);         // stays until this warp's arrival below
            if (w.b < 0) break;
            const int i = w.pos[t] + r;
            const bool real = i < w.nq;
            const int seen = real ? seen_by(p, w.nq, w.nk, i) : 0;
            const int j0 = w.j0, jn = w.n[t];
            float m = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int j = j0; j < jn; ++j, ++walked) {
                ok = __all_sync(kFullMask, wait_bar(bar(kBarS + t), walked & 1, abort_flag));
                if (!ok) break;
                tc_fence_after();
                uint32_t lo[64], hi[64];         // the row's scores
                tmem_ld64(ts, lo);
                tmem_wait_ld();
                tmem_ld64(ts + 64u, hi);
                const int lim = seen - j * kTile;
                const bool masked = __any_sync(kFullMask, lim < kTile);
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) lo[c] = c < lim ? lo[c] : 0xff800000u;
                }
                float mx[4];
                row_max<true>(lo, mx);
                tmem_wait_ld();
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) hi[c] = c + 64 < lim ? hi[c] : 0xff800000u;
                }
                row_max<false>(hi, mx);
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
                if (__any_sync(kFullMask, top > m + kLazy)) {
                    const float mn = fmaxf(m, top);
                    const float a = fast_exp2(m - (mn == -INFINITY ? 0.f : mn));
                    m = mn;
                    l *= a;
                    if (j > j0) {                // O, which holds the tiles before, takes the new reference
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
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pw[32];
                    weights<T>(h == 0 ? lo : hi, sc, -mu, pw, sum);
                    tmem_st32(ts + 32u * h, pw);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBarP + 2 * t + h));
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            }
            if (!ok) break;
            // ---- the result of a row, or its state (u, m, l) where the keys are split
            const bool done = jn > j0;           // this query tile walked some key tiles
            if (done) ok = __all_sync(kFullMask, wait_bar(bar(kBarO + t), ran++ & 1, abort_flag));
            if (!ok) break;
            tc_fence_after();
            const bool empty = seen <= j0 * kTile || !done;
            // (an empty row's O is nothing: 1 keeps its zeros)
            const float inv = p.n_splits > 1 || empty ? 1.f : __frcp_rn(l);
            const int rows = min(32, w.nq - w.pos[t] - 32 * (warp & 3));   // of this warp that exist
            const int64_t row0 = out_row(p, w, t, i - lane);
            const int64_t row_step = p.n_splits > 1 ? static_cast<int64_t>(p.n_q_heads) * p.n_splits : p.n_q_heads;
            const int64_t at0 = p.n_splits > 1 ? row0 * p.n_splits + w.split : row0;   // rows of out, or of the states
            const float odd = write_rows(p, smem + kOffStage + warp * 4096, to, at0, row_step, rows, done, empty, inv, lane);
            tc_fence_before();
            __syncwarp();
            if (done && lane == 0) mbar_arrive(bar(kBarOF + t));
            if (real && p.n_splits == 1) {
                if (p.lse != nullptr) p.lse[at0 + lane * row_step] = empty ? -INFINITY : (m + __log2f(l)) * kLn2;
            } else if (real) {
                p.ws_m[at0 + lane * row_step] = empty ? -INFINITY : m;
                p.ws_l[at0 + lane * row_step] = empty ? 0.f : l;
            }
            // rows that a value they do not see may have reached: done again at the
            // end, so that no wait of the other roles depends on how long that takes
            if (__any_sync(kFullMask, real && odd != odd) && hidden_special<T>(p, w, t, lane)) *redo = 1;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarWE + k % kWorks));
        }
        __syncwarp();
        if (ok && *redo) redo_rows<T>(p, t, warp & 3, lane);
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Joins the splits of each row: M = max m_s, out = sum 2^(m_s - M) u_s / L,
// L = sum 2^(m_s - M) l_s, in split order.  The blocks of the split kernel
// without its splits; a warp per row, 4 dims a lane.
__global__ void __launch_bounds__(256) fd_prompt_join_kernel(const __grid_constant__ PromptParams p) {
    grid_dependency_trigger();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Dealer dealer;
    dealer.start(p, lane, false);
    Work w;
    dealer.item(p, blockIdx.x * static_cast<uint32_t>(p.n_splits), lane, w);
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
        put_out4(p, row, 4 * lane, o);
        if (lane == 0 && p.lse != nullptr) p.lse[row] = empty ? -INFINITY : (M + log2f(L)) * kLn2;
    }
}

template <typename T>
cudaError_t launch_prompt_t(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                            const PromptParams& p, int64_t tiles, cudaStream_t stream) {
    auto kern = fd_prompt_kernel<T>;
    static std::atomic<unsigned long long> configured_ctx{0};
    cudaError_t e = allow_smem(kern, kSmem, configured_ctx);
    if (e != cudaSuccess) return e;
    const int64_t units = tiles * p.head_units;
    const int64_t items = units * p.n_splits;
    const int sms = fd_num_sms(-1);
    if (sms < 1) return cudaErrorInvalidDevice;
    e = launch_pdl(kern, dim3(static_cast<unsigned>(items < sms ? items : sms)), dim3(kPromptThreads), kSmem,
                               stream, tmQ, tmK, tmV, p);
    if (e != cudaSuccess || p.n_splits == 1) return e;
    return launch_pdl(fd_prompt_join_kernel, dim3(static_cast<unsigned>(units), 8), dim3(256), 0, stream, p);
}

}  // namespace

cudaError_t launch_prompt(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV, const PromptParams& p,
                          bool bf16, int64_t tiles, cudaStream_t stream) {
    return bf16 ? launch_prompt_t<__nv_bfloat16>(tmQ, tmK, tmV, p, tiles, stream)
                : launch_prompt_t<__half>(tmQ, tmK, tmV, p, tiles, stream);
}

cudaError_t status_word_prompt(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_status);
}

}  // namespace fdk
