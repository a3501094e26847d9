// fd_pages.cu -- the life of a cache's pages after fd_page_tables has given them
// out: shared by forks (fd_page_fork), given back by trims (fd_page_trim), moved
// together by a compaction (fd_page_compact).
//
// Nothing here is bound by bandwidth (4 to 28 bytes per page); the time is the
// chain of dependent reads, atomics and barriers.  So what CTAs have to agree on
// each computes for itself (prefix sums over the sequences or forks): that is all
// a fork needs, which runs on the whole grid.  Trims and compactions need more and are one
// cluster, whose CTAs write into each other's shared memory (counts, ranges of the bitmap of
// held pages) and meet at the hardware's cluster barrier: one launch, no spin, no
// workspace.  Outputs that may alias inputs are written behind every CTA's reads of
// them: behind a barrier of the cluster, and by a fork of more than one CTA in a second launch.
//
// Which page gets what never depends on the order of atomics: a trim's sequences
// and pages are numbered, and the largest number wins by an atomic minimum of its code.
#include "../../include/fd.h"
#include "fd_cluster.cuh"
#include "fd_device.cuh"
#include "fd_internal.h"

namespace fdk {

namespace {

__device__ unsigned int g_status = 0;   // this file's bits of the device status word

constexpr unsigned kFullMask = 0xffffffffu;
constexpr int kMaxCtas = 16;            // of a cluster
constexpr int kSegment = 128;           // table entries that a warp takes at a time

__device__ __forceinline__ void raise(unsigned bit) { atomicOr(&g_status, bit); }

// The i with first[i] <= x < first[i + 1], of n ascending starts.
__device__ __forceinline__ int find(const int32_t* first, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Entries of the free stack, of the count as read; one out of range raises a bit and is cut.
// (Apart from the read, whose latency other reads share.)
__device__ __forceinline__ int free_entries(const PagePlanParams& p, int count) {
    if ((count < 0 || count > p.n_free_max) && blockIdx.x == 0 && threadIdx.x == 0) raise(kStatusSeqlenBit);
    return min(max(count, 0), p.n_free_max);
}

// Inclusive prefix sums over the CTA, one barrier each: two buffers of warp sums
// take turns.
struct Scan {
    long long (*sums)[32];              // [2][32], shared
    int turn = 0;
    __device__ __forceinline__ long long operator()(long long x, long long& total) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(kFullMask, x, o);
            if (lane >= o) x += y;
        }
        long long* s = sums[turn];
        turn ^= 1;
        if (lane == 31) s[warp] = x;
        __syncthreads();
        long long w = lane < warps ? s[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(kFullMask, w, o);
            if (lane >= o) w += y;
        }
        total = __shfl_sync(kFullMask, w, 31);
        const long long before = __shfl_sync(kFullMask, w, max(warp - 1, 0));
        return x + (warp > 0 ? before : 0);
    }
};
__device__ __forceinline__ long long two(int hi, int lo) { return (static_cast<long long>(hi) << 32) | static_cast<unsigned>(lo); }
__device__ __forceinline__ int high(long long x) { return static_cast<int>(x >> 32); }
__device__ __forceinline__ int low(long long x) { return static_cast<int>(x & 0xffffffffll); }

// ---------------------------------------------------------------- forks
// Every CTA checks and numbers all forks (one prefix sum: the pages that parts of
// a page need, and the rows' segments), then the warps of the grid copy the
// rows, a segment each.  Forks of one parent with as many full pages count their
// sharers together: the first of them adds for all, so that 64 samples of a
// prompt cost one atomic a page.
constexpr int kForkRows = 1, kForkFinish = 2;

__global__ void __launch_bounds__(1024) fd_page_fork_kernel(const PagePlanParams p, int what) {
    extern __shared__ int32_t s_mem[];
    int32_t* s_owner = s_mem;                   // [batch] the fork that has this child
    int32_t* s_lead = s_owner + p.batch;        // [batch] the first fork of this parent
    int32_t* s_keep = s_lead + p.batch;         // [n_forks] tokens, -1: left out
    int32_t* s_add = s_keep + p.n_forks;        // [n_forks] sharers that it adds
    int32_t* s_seg = s_add + p.n_forks;         // [n_forks + 1] first segment
    __shared__ long long s_sums[2][32];
    Scan scan{s_sums};
    const int tid = threadIdx.x, lane = tid & 31, rank = blockIdx.x;
    // the last CTA writes what is one for all; the others (it too, if it is alone) copy rows
    const bool scribe = rank == static_cast<int>(gridDim.x) - 1;
    const int ps1 = (1 << p.page_shift) - 1;
    const int64_t capacity = static_cast<int64_t>(p.max_pages) << p.page_shift;
    grid_dependency_trigger();
    grid_dependency_wait();

    const int count_read = *p.free_count;
    for (int b = tid; b < p.batch; b += blockDim.x) s_owner[b] = s_lead[b] = INT32_MAX;
    __syncthreads();
    bool bad = false;
    for (int i = tid; i < p.n_forks; i += blockDim.x) {
        const int from = p.parents[i], to = p.children[i];
        int keep = -1;
        if (from >= 0 && from < p.batch && to >= 0 && to < p.batch && from != to) {
            const int len = p.seqlens[from], there = p.seqlens[to];
            keep = p.keep != nullptr ? p.keep[i] : len;
            if (len < 0 || len > capacity || there != 0 || keep > len) keep = -1;
            if (keep >= 0) atomicMin(&s_owner[to], i);
        }
        s_keep[i] = max(keep, -1);
        s_add[i] = 0;
    }
    __syncthreads();
    const int count = free_entries(p, count_read);
    int pages = 0, segments = 0;
    for (int base = 0; base < p.n_forks; base += blockDim.x) {
        const int i = base + tid;
        int keep = -1, from = 0, to = 0;
        if (i < p.n_forks && s_keep[i] >= 0) {
            from = p.parents[i];
            to = p.children[i];
            keep = s_owner[to] == i ? s_keep[i] : -1;
        }
        const int part = keep > 0 && (keep & ps1) != 0, full = keep >= 0 ? keep >> p.page_shift : 0;
        const int segs = (full + kSegment - 1) / kSegment;
        long long all;
        const long long upto = scan(two(part, segs), all);
        const int page_number = pages + high(upto);
        const bool fits = !part || page_number <= count;   // (segments of one that does not: walked without effect)
        if (i < p.n_forks) {
            bad |= keep < 0 || !fits;
            s_keep[i] = fits ? keep : -1;
            s_seg[i] = segments + low(upto) - segs;
            if (full > 0 && fits) atomicMin(&s_lead[from], i);
            if (scribe && (what & kForkRows) && part && fits) {
                const int src = p.block_table[static_cast<int64_t>(from) * p.max_pages + full];
                const int dst = p.free_in[count - page_number];
                if (src < 0 || src >= p.n_pages || dst < 0 || dst >= p.n_pages) raise(kStatusPageBit);
                p.block_table[static_cast<int64_t>(to) * p.max_pages + full] = dst;
                p.copy_src[page_number - 1] = src;
                p.copy_dst[page_number - 1] = dst;
            }
        }
        pages += high(all);
        segments += low(all);
    }
    if (tid == 0) s_seg[p.n_forks] = segments;
    __syncthreads();
    if (what & kForkRows) {
        if (bad && scribe) raise(kStatusSeqlenBit);
        for (int i = tid; i < p.n_forks; i += blockDim.x) {
            const int full = s_keep[i] >> p.page_shift;
            if (s_keep[i] < 0 || full == 0) continue;
            const int lead = s_lead[p.parents[i]];
            atomicAdd(&s_add[s_keep[lead] >> p.page_shift == full ? lead : i], 1);
        }
        __syncthreads();
        const int warps = max(static_cast<int>(gridDim.x) - 1, 1) * (blockDim.x >> 5);
        for (int s = scribe && gridDim.x > 1 ? segments : rank * (blockDim.x >> 5) + (tid >> 5); s < segments; s += warps) {
            const int i = find(s_seg, p.n_forks, s);
            const int j0 = (s - s_seg[i]) * kSegment, full = s_keep[i] >= 0 ? s_keep[i] >> p.page_shift : 0, add = s_add[i];
            const int32_t* from = p.block_table + static_cast<int64_t>(p.parents[i]) * p.max_pages;
            int32_t* to = p.block_table + static_cast<int64_t>(p.children[i]) * p.max_pages;
            int page[kSegment / 32];
#pragma unroll
            for (int k = 0; k < kSegment / 32; ++k) {
                const int j = j0 + 32 * k + lane;
                page[k] = j < full ? from[j] : -1;
            }
#pragma unroll
            for (int k = 0; k < kSegment / 32; ++k) {
                const int j = j0 + 32 * k + lane;
                if (j >= full) continue;
                to[j] = page[k];
                if (page[k] < 0 || page[k] >= p.n_pages) raise(kStatusPageBit);
                else if (add > 0) atomicAdd(&p.shares[page[k]], add);
            }
        }
    }
    if (!(what & kForkFinish) || !scribe) return;
    for (int b = tid; b < p.batch; b += blockDim.x) {
        const int i = s_owner[b];
        p.seqlens_out[b] = i != INT32_MAX && s_keep[i] >= 0 ? s_keep[i] : p.seqlens[b];
    }
    if (tid == 0) {
        const int taken = min(pages, count);
        *p.free_count_out = count - taken;
        *p.copy_count = taken;
    }
}

// ---------------------------------------------------------------- trims
// References let go are numbered 0 .. E - 1 (sequences in order, their pages in
// order), claims (a sequence that keeps a part of its last page) E + b; together,
// the events.  Each adds 2^16 - 1 to shares[page]: the word then holds the
// events k and the holders s - k that are left beyond the first, as k 2^16 + (s - k).
// An event that finds (0, 0) is the page's only holder and decides for it alone.
// If every event does, one barrier (for the counts) is all; else the pages that
// nobody holds any more (s - k = -1) are decided by a bid: the largest
// number, a claim if there is one, leaves its code there by an atomic minimum.
// (A claim keeps the page, a reference gives it back.)
constexpr int kCode = 1 << 30;
__device__ __forceinline__ int code_of(int number) { return -kCode - number; }
constexpr int kEvent = 0xffff;          // what an event adds; also the word of a page with one event and no other holder
__device__ __forceinline__ int events_of(int word) { return (word + 0x8000) >> 16; }
__device__ __forceinline__ int left_of(int word) { return word - (events_of(word) << 16); }

constexpr int kHeld = 8;                // pages a thread keeps in registers between the phases

__global__ void __launch_bounds__(1024) fd_page_trim_kernel(const PagePlanParams p) {
    extern __shared__ int32_t s_mem[];
    int32_t* s_keep = s_mem;                    // [batch] tokens kept, -1: left as it is
    int32_t* s_first = s_keep + p.batch;        // [batch + 1] number of its first reference let go
    int32_t* s_new = s_first + p.batch + 1;     // [batch] the page that replaces a claim's, kNone: none (its own thread's)
    constexpr int32_t kNone = INT32_MIN;
    __shared__ long long s_sums[2][32];
    __shared__ uint32_t s_given[kMaxCtas], s_any[kMaxCtas];   // of each CTA: references that give a page back, events that were not alone
    Scan scan{s_sums};
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x, ranks = gridDim.x;
    const int ps1 = (1 << p.page_shift) - 1;
    const int64_t capacity = static_cast<int64_t>(p.max_pages) << p.page_shift;
    const bool shared = p.shares != nullptr;
    cluster_arrive();                   // (waited for before the first access to another CTA's memory)
    grid_dependency_trigger();
    grid_dependency_wait();

    const int count_read = *p.free_count;
    bool bad = false, bad_page = false;
    auto tail_page = [&](int b) {       // the page that a sequence keeps a part of, -1: none
        const int keep = s_keep[b];
        if (keep < 0 || (keep & ps1) == 0) return -1;
        const int page = p.block_table[static_cast<int64_t>(b) * p.max_pages + (keep >> p.page_shift)];
        return page >= 0 && page < p.n_pages ? page : -1;
    };
    auto let_go = [&](int len, int keep) { return keep >= 0 ? ((len + ps1) >> p.page_shift) - ((keep + ps1) >> p.page_shift) : 0; };
    int claims = 0, E = 0;              // (E < 2^30, the host's check)
    int my_len = 0;                     // of sequence tid
    for (int base = 0; base < p.batch; base += blockDim.x) {
        const int b = base + tid;
        int len = 0, keep = -1;
        if (b < p.batch) {
            len = p.seqlens[b];
            keep = p.keep[b];
            if (len < 0 || len > capacity) {
                bad = true;
                keep = -1;
            }
            if (keep >= len) keep = -1;
            keep = max(keep, -1);
            s_keep[b] = keep;
            if (base == 0) my_len = len;
        }
        const int n = let_go(len, keep);
        long long all;
        const long long upto = scan(two(shared && keep >= 0 && (keep & ps1) != 0, n), all);
        if (b < p.batch) s_first[b] = E + low(upto) - n;
        claims += high(all);
        E += low(all);
    }
    const int count = free_entries(p, count_read);
    __syncwarp();
    cluster_wait();
    if (claims > count) {
        // not sure that every claim that needs a page gets one: those of pages that
        // are shared now count, in order, and what does not fit is left as it is
        int may_need = 0;
        E = 0;
        for (int base = 0; base < p.batch; base += blockDim.x) {
            const int b = base + tid;
            const int tail = b < p.batch ? tail_page(b) : -1;
            const int may = tail >= 0 && __ldcg(p.shares + tail) > 0;
            long long all;
            const int number = may_need + low(scan(may, all));
            may_need += low(all);
            int n = 0;
            if (b < p.batch) {
                if (may && number > count) {
                    bad = true;
                    s_keep[b] = -1;
                }
                n = let_go(p.seqlens[b], s_keep[b]);
            }
            const int end = E + low(scan(n, all));
            E += low(all);
            if (b < p.batch) s_first[b] = end - n;
        }
        cluster_barrier();              // every CTA has looked at the shares as they were
    }
    if (tid == 0) s_first[p.batch] = E;
    if (rank == 0 && bad) raise(kStatusSeqlenBit);
    __syncthreads();

    // a warp's references: [e0, e1)
    const int warps = ranks * (blockDim.x >> 5);
    const int per_warp = ((E + warps - 1) / warps + 31) / 32 * 32;
    const int e0 = min(static_cast<int64_t>(rank * (blockDim.x >> 5) + warp) * per_warp, static_cast<int64_t>(E));
    const int e1 = min(e0 + per_warp, E);
    // the pages of the thread's references first + 32 k + lane, -1 behind the warp's last or outside the pool
    auto load_pages = [&](int first, auto& page) {
        constexpr int K = sizeof(page) / sizeof(int);
        int b = -1;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = first + 32 * k + lane;
            page[k] = -2;
            if (first + 32 * k >= e1) break;
            if (e >= e1) continue;
            if (b < 0) b = find(s_first, p.batch, e);
            for (int steps = 0; e >= s_first[b + 1]; ++steps) {     // most often the same sequence or one soon behind it
                if (steps < 4) ++b;
                else b = find(s_first, p.batch, e);
            }
            const int j = ((s_keep[b] + ps1) >> p.page_shift) + e - s_first[b];
            page[k] = p.block_table[static_cast<int64_t>(b) * p.max_pages + j];
        }
#pragma unroll
        for (int k = 0; k < K && first + 32 * k < e1; ++k) {
            if (page[k] >= 0 && page[k] < p.n_pages) continue;
            bad_page |= first + 32 * k + lane < e1;
            page[k] = -1;
        }
    };
    // calls f(first, pages) for the warp's references: the first kHeld of a thread at once,
    // whose pages stay in registers from phase to phase, others one by one
    int held[kHeld], words[kHeld];      // (and the pages' words, once every event has happened)
    auto for_references = [&](auto f) {
        if (e0 < e1) f(e0, held, words);
#pragma unroll 1
        for (int first = e0 + 32 * kHeld; first < e1; first += 32) {
            int page[1], word[1];
            load_pages(first, page);
            f(first, page, word);
        }
    };
    // calls f(b, page) for the thread's claims
    const int b0 = rank * blockDim.x + tid;
    int tail0 = -1;                     // the first claim's page, read together with the references'
    const bool claim0 = b0 < p.batch && s_keep[b0] >= 0 && (s_keep[b0] & ps1) != 0;
    if (claim0) tail0 = p.block_table[static_cast<int64_t>(b0) * p.max_pages + (s_keep[b0] >> p.page_shift)];
    auto for_claims = [&](auto f) {
        if (tail0 >= 0) f(b0, tail0);
        for (int b = b0 + ranks * blockDim.x; b < p.batch; b += ranks * blockDim.x) {
            const int page = tail_page(b);
            if (page >= 0) f(b, page);
        }
    };
    if (e0 < e1) load_pages(e0, held);
    if (tail0 < 0 || tail0 >= p.n_pages) tail0 = -1;
    int given = 0;                      // references of this thread that give a page back
    bool any = false;
    if (shared) {
        auto happened = [&](int was) {
            any |= was != 0;
            if (left_of(was) < 0) raise(kStatusPageBit);      // let go more often than held
        };
        const int was0 = tail0 >= 0 ? atomicAdd(&p.shares[tail0], kEvent) : 0;
        for_references([&](int first, auto& page, auto& word) {
            constexpr int K = sizeof(page) / sizeof(int);
            int was[K];
#pragma unroll
            for (int k = 0; k < K && first + 32 * k < e1; ++k) was[k] = page[k] >= 0 ? atomicAdd(&p.shares[page[k]], kEvent) : 0;
#pragma unroll
            for (int k = 0; k < K && first + 32 * k < e1; ++k) {
                happened(was[k]);
                given += page[k] >= 0 && was[k] == 0;
            }
        });
        happened(was0);
        for_claims([&](int b, int page) {
            if (b != b0) happened(atomicAdd(&p.shares[page], kEvent));
        });
        for (int b = b0; b < p.batch; b += ranks * blockDim.x) bad_page |= s_keep[b] >= 0 && (s_keep[b] & ps1) != 0 && (b == b0 ? tail0 : tail_page(b)) < 0;
    } else {
        for_references([&](int first, auto& page, auto& word) {
            constexpr int K = sizeof(page) / sizeof(int);
#pragma unroll
            for (int k = 0; k < K && first + 32 * k < e1; ++k) given += page[k] >= 0;
        });
    }
    long long cta_given;
    long long upto = scan(two(any, given), cta_given);
    if (tid < ranks) {
        remote_store(remote_smem(smem_u32(&s_given[rank]), tid), static_cast<uint32_t>(low(cta_given)));
        remote_store(remote_smem(smem_u32(&s_any[rank]), tid), static_cast<uint32_t>(high(cta_given)));
    }
    cluster_barrier();
    uint32_t others = 0;
    for (int r = 0; r < ranks; ++r) others |= s_any[r];
    int taken = 0;
    if (others != 0) {
        cluster_barrier();              // (the counts are read before they are written again)
        auto bid = [&](int number, int page, int word) {
            const bool bids = word != kEvent && (word <= -kCode || left_of(word) < 0);
            if (bids) atomicMin(&p.shares[page], code_of(number));
            return bids;
        };
        for_references([&](int first, auto& page, auto& word) {
            constexpr int K = sizeof(page) / sizeof(int);
#pragma unroll
            for (int k = 0; k < K && first + 32 * k < e1; ++k) word[k] = page[k] >= 0 ? __ldcg(p.shares + page[k]) : 0;
#pragma unroll
            for (int k = 0; k < K && first + 32 * k < e1; ++k)
                if (page[k] >= 0 && bid(first + 32 * k + lane, page[k], word[k])) word[k] = -kCode;   // (to be read again)
        });
        for_claims([&](int b, int page) { bid(E + b, page, __ldcg(p.shares + page)); });
        cluster_barrier();
        given = 0;
        for_references([&](int first, auto& page, auto& word) {
            constexpr int K = sizeof(page) / sizeof(int);
#pragma unroll
            for (int k = 0; k < K && first + 32 * k < e1; ++k)
                if (page[k] >= 0 && (K == 1 || word[k] == -kCode)) word[k] = __ldcg(p.shares + page[k]);
#pragma unroll
            for (int k = 0; k < K && first + 32 * k < e1; ++k) given += page[k] >= 0 && (word[k] == kEvent || word[k] == code_of(first + 32 * k + lane));
        });
        upto = scan(given, cta_given);
        if (tid < ranks) remote_store(remote_smem(smem_u32(&s_given[rank]), tid), static_cast<uint32_t>(low(cta_given)));
        // which claims get copies
        for (int base = 0; base < p.batch; base += blockDim.x) {
            const int b = base + tid;
            const int page = b < p.batch ? tail_page(b) : -1;
            const int word = page >= 0 ? __ldcg(p.shares + page) : 0;
            const int moves = page >= 0 && word != kEvent && word != code_of(E + b);
            long long all;
            const int number = taken + low(scan(moves, all));
            taken += low(all);
            if (base / static_cast<int>(blockDim.x) % ranks != rank || b >= p.batch) continue;   // (b is a claim of this very thread)
            s_new[b] = kNone;
            if (moves && number > count) {      // (shares that were less than the holders: the page stays as it is)
                raise(kStatusPageBit);
            } else if (moves) {
                const int to = p.free_in[count - number];
                if (to < 0 || to >= p.n_pages) raise(kStatusPageBit);
                p.copy_src[number - 1] = page;
                p.copy_dst[number - 1] = to;
                s_new[b] = to;
            }
        }
        taken = min(taken, count);
        cluster_barrier();
    }
    // where this warp's pages go: behind those of the CTAs and warps before it
    int before = low(upto) - given;     // (of this thread; its warp's first lane starts the warp)
    before = __shfl_sync(kFullMask, before, 0);
    int all_given = 0;
    for (int r = 0; r < ranks; ++r) {
        if (r < rank) before += static_cast<int>(s_given[r]);
        all_given += static_cast<int>(s_given[r]);
    }
    const int base = count - taken;
    if (rank == 0) {
        for (int b = tid; b < p.batch; b += blockDim.x) p.seqlens_out[b] = s_keep[b] >= 0 ? s_keep[b] : b == tid ? my_len : p.seqlens[b];
        if (tid == 0) {
            *p.free_count_out = static_cast<int>(min(static_cast<int64_t>(base) + all_given, static_cast<int64_t>(p.n_free_max)));
            if (p.copy_count != nullptr) *p.copy_count = taken;
        }
    }
    // whether the event decides for the page; its word is made a count again
    auto settle = [&](int number, int page, int word) {
        const bool mine = word == kEvent || word == code_of(number);
        if (mine) p.shares[page] = 0;
        else if (word > -kCode) p.shares[page] = left_of(word);   // (all of the page's events write the same)
        return mine;
    };
    if (shared)
        for_claims([&](int b, int page) {
            settle(E + b, page, others != 0 ? __ldcg(p.shares + page) : kEvent);
            if (others != 0 && s_new[b] != kNone)
                p.block_table[static_cast<int64_t>(b) * p.max_pages + (s_keep[b] >> p.page_shift)] = s_new[b];
        });
    for_references([&](int first, auto& page, auto& word) {
        constexpr int K = sizeof(page) / sizeof(int);
#pragma unroll
        for (int k = 0; k < K && first + 32 * k < e1; ++k) {
            if (others == 0) word[k] = kEvent;
            else if (K == 1 && page[k] >= 0) word[k] = __ldcg(p.shares + page[k]);
        }
#pragma unroll
        for (int k = 0; k < K && first + 32 * k < e1; ++k) {
            bool mine = page[k] >= 0;
            if (mine && shared) mine = settle(first + 32 * k + lane, page[k], word[k]);
            const unsigned votes = __ballot_sync(kFullMask, mine);
            if (mine) {
                const int64_t place = static_cast<int64_t>(base) + all_given - 1 - (before + __popc(votes & ((1u << lane) - 1u)));
                if (place < p.n_free_max) p.free_pages[place] = page[k];
                else raise(kStatusPageBit);
            }
            before += __popc(votes);
        }
    });
    if (bad_page) raise(kStatusPageBit);
}

// ---------------------------------------------------------------- compaction
// Held pages from n_keep on are bits of a map.  Each CTA marks those of its share of
// the tables in a map of its own; then each joins one range of all the maps,
// counts its bits, and sends the range and its prefix sums to every CTA, so that a
// page's number among the held ones (its word's prefix and the bits below
// it) is looked up in the CTA's own memory.  The free stack is filtered in rounds of
// what the cluster's registers hold, read before it is written; the first round's
// entries are on their way while the maps are made.
// (One map over all CTAs, marked and looked up remotely, was slower: 38 against 32 us
// for 61000 held pages of a pool of 131072, half of it given up.)
constexpr int kEntries = 16;            // entries of the free stack a thread holds in a round

__global__ void __launch_bounds__(512) fd_page_compact_kernel(const PagePlanParams p, int words_per_cta) {
    extern __shared__ int32_t s_mem[];
    int32_t* s_seg = s_mem;                                             // [batch + 1] first segment of the row
    int32_t* s_pages = s_seg + p.batch + 1;                             // [batch] pages of the row
    const int words = words_per_cta * gridDim.x;
    uint32_t* s_bits = reinterpret_cast<uint32_t*>(s_pages + p.batch);  // [words] this CTA's marks, then the joined map
    uint32_t* s_pref = s_bits + words;                                  // [words] held pages of the words before
    __shared__ long long s_sums[2][32];
    __shared__ uint32_t s_held[kMaxCtas], s_kept[2][kMaxCtas];          // of each CTA's range, and of its entries
    Scan scan{s_sums};
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x, ranks = gridDim.x;
    const int ps1 = (1 << p.page_shift) - 1, threads = blockDim.x;
    const int64_t capacity = static_cast<int64_t>(p.max_pages) << p.page_shift;
    cluster_arrive();               // (waited for before the first access to another CTA's memory)
    grid_dependency_trigger();
    grid_dependency_wait();

    const int warps = ranks * (threads >> 5), w0 = rank * (threads >> 5) + warp;
    const int count_read = *p.free_count;
    int entry[kEntries];
    auto load_entries = [&](int64_t base) {
#pragma unroll
        for (int k = 0; k < kEntries; ++k) {
            const int64_t i = base + static_cast<int64_t>(w0) * (32 * kEntries) + 32 * k + lane;
            entry[k] = i < p.n_free_max ? p.free_pages[i] : 0;     // (not looked at here: other reads share the latency)
        }
    };
    load_entries(0);
    for (int w = tid; w < words; w += threads) s_bits[w] = 0;
    int segments = 0;
    bool bad = false;
    for (int base = 0; base < p.batch; base += threads) {
        const int b = base + tid;
        int n = 0;
        if (b < p.batch) {
            const int len = p.seqlens[b];
            if (len < 0 || len > capacity) bad = true;
            else n = (len + ps1) >> p.page_shift;
        }
        long long all;
        const int end = segments + low(scan((n + kSegment - 1) / kSegment, all));
        segments += low(all);
        if (b < p.batch) {
            s_seg[b] = end - (n + kSegment - 1) / kSegment;
            s_pages[b] = n;
        }
    }
    if (tid == 0) s_seg[p.batch] = segments;
    if (bad && rank == 0) raise(kStatusSeqlenBit);
    __syncthreads();
    cluster_wait();                 // every CTA has started

    const uint32_t bits = smem_u32(s_bits), pref = smem_u32(s_pref);
    // A warp's segments of the rows; the first kCached of them stay in registers.
    constexpr int kPer = kSegment / 32, kCached = 2;
    struct Segment {
        int32_t* row;               // the lane's first entry
        int n;                      // entries from there on
        int page[kPer];
    };
    auto load_segment = [&](int s, Segment& x) {
        const int b = find(s_seg, p.batch, s);
        const int j0 = (s - s_seg[b]) * kSegment + lane;
        x.n = s_pages[b] - j0;
        x.row = p.block_table + static_cast<int64_t>(b) * p.max_pages + j0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) x.page[k] = 32 * k < x.n ? x.row[32 * k] : 0;
    };
    bool bad_page = false;
    auto moves = [&](const Segment& x, int k) { return 32 * k < x.n && x.page[k] >= p.n_keep && x.page[k] < p.n_pages; };
    auto mark = [&](const Segment& x) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            bad_page |= 32 * k < x.n && (x.page[k] < 0 || x.page[k] >= p.n_pages);
            const int bit = x.page[k] - p.n_keep;
            if (moves(x, k)) atomicOr(&s_bits[bit >> 5], 1u << (bit & 31));
        }
    };
    Segment cached[kCached];
#pragma unroll
    for (int c = 0; c < kCached; ++c)
        if (w0 + c * warps < segments) load_segment(w0 + c * warps, cached[c]);
#pragma unroll
    for (int c = 0; c < kCached; ++c)
        if (w0 + c * warps < segments) mark(cached[c]);
#pragma unroll 1
    for (int s = w0 + kCached * warps; s < segments; s += warps) {
        Segment x;
        load_segment(s, x);
        mark(x);
    }
    // the entries of the free stack that stay in it or are used up
    const int count = free_entries(p, count_read);
    int kept = 0, at = 0;               // of the rounds before; where this warp's go
    unsigned votes[kEntries];
    auto count_entries = [&](int64_t base, uint32_t* counts) {
        int n = 0;
#pragma unroll
        for (int k = 0; k < kEntries; ++k) {
            const int64_t i = base + static_cast<int64_t>(w0) * (32 * kEntries) + 32 * k + lane;
            bad_page |= i < count && (entry[k] < 0 || entry[k] >= p.n_pages);
            votes[k] = __ballot_sync(kFullMask, i < count && entry[k] >= 0 && entry[k] < p.n_keep);
            n += __popc(votes[k]);
        }
        long long all;
        at = __shfl_sync(kFullMask, low(scan(lane == 0 ? n : 0, all)), 0) - n;
        if (tid < ranks) remote_store(remote_smem(smem_u32(counts + rank), tid), static_cast<uint32_t>(low(all)));
    };
    auto write_entries = [&](const uint32_t* counts) {
        at += kept;
        for (int r = 0; r < ranks; ++r) {
            if (r < rank) at += static_cast<int>(counts[r]);
            kept += static_cast<int>(counts[r]);
        }
#pragma unroll
        for (int k = 0; k < kEntries; ++k) {
            if ((votes[k] >> lane) & 1u) p.free_pages[at + __popc(votes[k] & ((1u << lane) - 1u))] = entry[k];
            at += __popc(votes[k]);
        }
    };
    count_entries(0, s_kept[0]);
    cluster_barrier();              // the maps are marked, and every CTA has read its entries

    write_entries(s_kept[0]);
    const int round = ranks * threads * kEntries;
    int turn = 1;
    for (int64_t base = round; base < count; base += round, turn ^= 1) {
        load_entries(base);
        count_entries(base, s_kept[turn]);
        cluster_barrier();
        write_entries(s_kept[turn]);
    }
    // this CTA's range of the maps, joined; a thread takes words that follow each other
    const int per_thread = (words_per_cta + threads - 1) / threads;
    const int wa = min(tid * per_thread, words_per_cta), wb = min(wa + per_thread, words_per_cta);
    const int range = rank * words_per_cta;
    int mine = 0;
    for (int w = wa; w < wb; ++w) {
        uint32_t word = 0;
#pragma unroll 8
        for (int r = 0; r < ranks; ++r) word |= remote_load(remote_smem(bits + 4 * (range + w), r));
        s_pref[range + w] = word;   // (kept here until every CTA has read the marks)
        mine += __popc(word);
    }
    long long cta_held;
    int upto = low(scan(mine, cta_held)) - mine;
    if (tid < ranks) remote_store(remote_smem(smem_u32(&s_held[rank]), tid), static_cast<uint32_t>(low(cta_held)));
    cluster_barrier();              // the marks are read
    int held = 0;
    for (int r = 0; r < ranks; ++r) {
        if (r < rank) upto += static_cast<int>(s_held[r]);
        held += static_cast<int>(s_held[r]);
    }
    for (int w = wa; w < wb; ++w) {
        const uint32_t word = s_pref[range + w];
        for (int r = 0; r < ranks; ++r) {
            remote_store(remote_smem(bits + 4 * (range + w), r), word);
            remote_store(remote_smem(pref + 4 * (range + w), r), upto);
        }
        upto += __popc(word);
    }
    cluster_barrier();              // the map, its numbers and the filtered stack are there for everyone

    const int moved = min(min(held, kept), p.n_copies);
    auto rename = [&](const Segment& x) {
        int number[kPer], to[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int bit = x.page[k] - p.n_keep;
            number[k] = INT32_MAX;
            if (moves(x, k)) number[k] = static_cast<int>(s_pref[bit >> 5]) + __popc(s_bits[bit >> 5] & ((1u << (bit & 31)) - 1u));
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) to[k] = number[k] < moved ? __ldcg(p.free_pages + kept - 1 - number[k]) : 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (number[k] < moved) x.row[32 * k] = to[k];
    };
#pragma unroll
    for (int c = 0; c < kCached; ++c)
        if (w0 + c * warps < segments) rename(cached[c]);
#pragma unroll 1
    for (int s = w0 + kCached * warps; s < segments; s += warps) {
        Segment x;
        load_segment(s, x);
        rename(x);
    }
    // each CTA writes its range's part of the list and moves the counts, eight pages a thread at a time
    for (int x0 = tid; x0 < words_per_cta * 32; x0 += 8 * threads) {
        int number[8], to[8], held_by[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int x = x0 + k * threads;
            number[k] = INT32_MAX;
            if (x >= words_per_cta * 32) continue;
            const uint32_t word = s_bits[range + (x >> 5)];
            if ((word >> lane) & 1u)
                number[k] = static_cast<int>(s_pref[range + (x >> 5)]) + __popc(word & ((1u << lane) - 1u));
        }
        const int page0 = p.n_keep + range * 32 + x0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            to[k] = number[k] < moved ? __ldcg(p.free_pages + kept - 1 - number[k]) : 0;
            held_by[k] = p.shares != nullptr && number[k] < moved ? p.shares[page0 + k * threads] : 0;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (number[k] >= moved) continue;
            p.copy_src[number[k]] = page0 + k * threads;
            p.copy_dst[number[k]] = to[k];
            if (p.shares != nullptr) {
                p.shares[to[k]] = held_by[k];
                p.shares[page0 + k * threads] = 0;
            }
        }
    }
    if (rank == 0 && tid == 0) {
        if (moved < held) raise(kStatusPageBit);
        *p.free_count_out = kept - moved;
        *p.copy_count = moved;
    }
    if (bad_page) raise(kStatusPageBit);
}

// One cluster of `ctas` CTAs; more than 8 have to be allowed, once per context (large_ctx: the kernel's own).
template <typename Kern, typename... Args>
cudaError_t launch_cluster(Kern kern, std::atomic<unsigned long long>& large_ctx, int ctas, int threads, size_t smem,
                           cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaSuccess;
    if (ctas > 8) {
        const unsigned long long ctx = current_context_id();
        if (ctx == 0 || large_ctx.load(std::memory_order_acquire) != ctx) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e == cudaSuccess && ctx != 0) large_ctx.store(ctx, std::memory_order_release);
        }
    }
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_page_fork(const PagePlanParams& p, cudaStream_t stream) {
    static std::atomic<unsigned long long> configured_ctx{0};
    cudaError_t e = allow_smem(fd_page_fork_kernel, (5 * FD_MAX_TABLE_BATCH + 1) * sizeof(int32_t), configured_ctx);
    if (e != cudaSuccess) return e;
    const int sms = fd_num_sms(-1);
    if (sms < 1) return cudaErrorInvalidDevice;
    const size_t smem = (2 * static_cast<size_t>(p.batch) + 3 * static_cast<size_t>(p.n_forks) + 1) * sizeof(int32_t);
    // Forks and sequences are walked by every CTA, so that many want many threads; few
    // threads start and meet faster (12 forks of 755 pages, 64 of 8001, us: 128 threads
    // 4.7 / 8.9, 256 4.8 / 7.6, 512 5.3 / 7.1, 1024 6.3 / 8.1).
    const int threads = p.n_forks <= 1024 && p.batch <= 1024 ? 256 : 1024;
    // a warp for each segment that the rows can have
    const int64_t segments = static_cast<int64_t>(p.n_forks) * ((p.max_pages + kSegment - 1) / kSegment);
    const int64_t want = (segments + threads / 32 - 1) / (threads / 32);
    const int ctas = want <= 1 ? 1 : static_cast<int>(want < sms ? want + 1 : sms);
    // lengths or the count in place: they are written when every CTA has read them
    const bool in_place = p.seqlens == p.seqlens_out || p.free_count == p.free_count_out;
    if (ctas == 1 || !in_place) return launch_pdl(fd_page_fork_kernel, dim3(ctas), dim3(threads), smem, stream, p, kForkRows | kForkFinish);
    e = launch_pdl(fd_page_fork_kernel, dim3(ctas), dim3(threads), smem, stream, p, kForkRows);
    return e != cudaSuccess ? e : launch_pdl(fd_page_fork_kernel, dim3(1), dim3(threads), smem, stream, p, kForkFinish);
}

cudaError_t launch_page_trim(const PagePlanParams& p, cudaStream_t stream) {
    static std::atomic<unsigned long long> configured_ctx{0}, large_ctx{0};
    cudaError_t e = allow_smem(fd_page_trim_kernel, (3 * FD_MAX_TABLE_BATCH + 1) * sizeof(int32_t), configured_ctx);
    if (e != cudaSuccess) return e;
    const size_t smem = (3 * static_cast<size_t>(p.batch) + 1) * sizeof(int32_t);
    // Eight CTAs of 256 threads while a thread cannot get more than 16 references, else as
    // many as a cluster has, of 512.  Drafts of 64 sequences / 37600 references (pages of six
    // sequences among them, parts of which others keep), us with the copy that restores the
    // state (1.3): 8 x 128 7.0 / 75, 8 x 256 7.1 / 45, 8 x 512 7.3 / 33, 16 x 256 7.2 / 29, 16 x 512 7.5 / 19,
    // 16 x 768 7.9 / 21; since then 8 x 256 5.6 to 6.1, 16 x 512 16.4.
    const bool small = static_cast<int64_t>(p.batch) * p.max_pages <= 16 * 8 * 256;
    return launch_cluster(fd_page_trim_kernel, large_ctx, small ? 8 : kMaxCtas, small ? 256 : 512, smem, stream, p);
}

cudaError_t launch_page_compact(const PagePlanParams& p, cudaStream_t stream) {
    constexpr int kMaxWords = FD_MAX_COMPACT_PAGES / 32 + kMaxCtas;
    static std::atomic<unsigned long long> configured_ctx{0}, large_ctx{0};
    cudaError_t e = allow_smem(fd_page_compact_kernel, (2 * FD_MAX_TABLE_BATCH + 1 + 2 * kMaxWords) * sizeof(int32_t), configured_ctx);
    if (e != cudaSuccess) return e;
    // As many threads as hold tables and free stack in registers, within a cluster's.
    // 32 sequences in a pool of 2048 / 61000 pages in one of 131072, us with the copy that
    // restores the state (1.2 / 1.7): 8 x 128 8.9 / 72, 8 x 256 9.2 / 42, 16 x 256 9.7 / 26, 16 x 512 10.5 / 19; since
    // then 8 x 128 8.3, 16 x 512 17.4.
    const bool small = static_cast<int64_t>(p.batch) * p.max_pages <= 16384 && p.n_free_max <= 16384;
    const int ctas = small ? 8 : kMaxCtas;
    const int64_t words = (static_cast<int64_t>(p.n_pages) - p.n_keep + 31) / 32;
    const int words_per_cta = static_cast<int>(words < ctas ? 1 : (words + ctas - 1) / ctas);
    const size_t smem = (2 * static_cast<size_t>(p.batch) + 1 + 2 * static_cast<size_t>(words_per_cta) * ctas) * sizeof(int32_t);
    return launch_cluster(fd_page_compact_kernel, large_ctx, ctas, small ? 128 : 512, smem, stream, p, words_per_cta);
}

cudaError_t status_word_pages(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_status);
}

}  // namespace fdk
