// fd_pages.cu -- the life of a cache's pages after fd_page_tables has given them
// out: shared by forks (fd_page_fork), given back by trims (fd_page_trim), moved
// together by a compaction (fd_page_compact).
//
// Each call is one launch of one cluster of up to 8 CTAs.  Nothing here is bound
// by bandwidth (4 to 28 bytes per page); the time is the chain of dependent
// reads, atomics and barriers, which the hardware's cluster barrier keeps
// within one launch, without a spin and without a workspace: what the CTAs have
// to agree on they either compute each for itself (prefix sums over the
// sequences or forks) or keep in each other's shared memory (the bitmap of
// held pages, counts).  Outputs that may alias inputs are written behind a
// barrier that follows every CTA's reads of them.
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
constexpr int kMaxCtas = 8;
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

// Entries of the free stack; out of range counts raise a bit and are cut.
__device__ __forceinline__ int free_entries(const PagePlanParams& p) {
    const int count = *p.free_count;
    if ((count < 0 || count > p.n_free_max) && blockIdx.x == 0 && threadIdx.x == 0) raise(kStatusSeqlenBit);
    return min(max(count, 0), p.n_free_max);
}

// ---------------------------------------------------------------- forks
// Every CTA checks and numbers all forks (one prefix sum for the pages that
// parts of a page need), then the warps of the cluster copy the rows, a segment
// each.  Forks of one parent with as many full pages count their sharers together:
// the first of them adds for all, so that 64 samples of a prompt cost one
// atomic a page.
__global__ void __launch_bounds__(1024) fd_page_fork_kernel(const PagePlanParams p) {
    extern __shared__ int32_t s_mem[];
    int32_t* s_owner = s_mem;                   // [batch] the fork that has this child
    int32_t* s_lead = s_owner + p.batch;        // [batch] the first fork of this parent
    int32_t* s_keep = s_lead + p.batch;         // [n_forks] tokens, -1: left out
    int32_t* s_add = s_keep + p.n_forks;        // [n_forks] sharers that it adds
    int32_t* s_seg = s_add + p.n_forks;         // [n_forks + 1] first segment
    __shared__ long long s_sums[32];
    const int tid = threadIdx.x, lane = tid & 31, rank = blockIdx.x, ranks = gridDim.x;
    const int ps1 = (1 << p.page_shift) - 1;
    const int64_t capacity = static_cast<int64_t>(p.max_pages) << p.page_shift;
    grid_dependency_trigger();
    grid_dependency_wait();

    const int count = free_entries(p);
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
    long long pages = 0, segments = 0;
    for (int base = 0; base < p.n_forks; base += blockDim.x) {
        const int i = base + tid;
        int keep = -1, from = 0, to = 0;
        if (i < p.n_forks && s_keep[i] >= 0) {
            from = p.parents[i];
            to = p.children[i];
            keep = s_owner[to] == i ? s_keep[i] : -1;
        }
        const int part = keep > 0 && (keep & ps1) != 0;
        long long all;
        const long long upto = pages + block_scan(part, s_sums, all);
        pages += all;
        if (part && upto > count) keep = -1;
        const int full = keep >= 0 ? keep >> p.page_shift : 0;
        const long long seg_end = segments + block_scan((full + kSegment - 1) / kSegment, s_sums, all);
        if (i < p.n_forks) {
            bad |= keep < 0;
            s_keep[i] = keep;
            s_seg[i] = static_cast<int32_t>(seg_end - (full + kSegment - 1) / kSegment);
            if (full > 0) atomicMin(&s_lead[from], i);
            if (rank == 0 && part && keep >= 0) {
                const int src = p.block_table[static_cast<int64_t>(from) * p.max_pages + full];
                const int dst = p.free_in[count - upto];
                if (src < 0 || src >= p.n_pages || dst < 0 || dst >= p.n_pages) raise(kStatusPageBit);
                p.block_table[static_cast<int64_t>(to) * p.max_pages + full] = dst;
                p.copy_src[upto - 1] = src;
                p.copy_dst[upto - 1] = dst;
            }
        }
        segments += all;
    }
    if (tid == 0) s_seg[p.n_forks] = static_cast<int32_t>(segments);
    if (bad && rank == 0) raise(kStatusSeqlenBit);
    __syncthreads();
    cluster_arrive();           // every CTA has read the lengths and the free count
    for (int i = tid; i < p.n_forks; i += blockDim.x) {
        const int full = s_keep[i] >> p.page_shift;
        if (s_keep[i] < 0 || full == 0) continue;
        const int lead = s_lead[p.parents[i]];
        atomicAdd(&s_add[s_keep[lead] >> p.page_shift == full ? lead : i], 1);
    }
    __syncthreads();
    const int total = s_seg[p.n_forks];
    const int warps = ranks * (blockDim.x >> 5);
    for (int s = rank * (blockDim.x >> 5) + (tid >> 5); s < total; s += warps) {
        const int i = find(s_seg, p.n_forks, s);
        const int j0 = (s - s_seg[i]) * kSegment, full = s_keep[i] >> p.page_shift, add = s_add[i];
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
    __syncwarp();
    cluster_wait();
    if (rank != 0) return;
    for (int b = tid; b < p.batch; b += blockDim.x) {
        const int i = s_owner[b];
        p.seqlens_out[b] = i != INT32_MAX && s_keep[i] >= 0 ? s_keep[i] : p.seqlens[b];
    }
    if (tid == 0) {
        const int taken = static_cast<int>(pages < count ? pages : count);
        *p.free_count_out = count - taken;
        *p.copy_count = taken;
    }
}

// ---------------------------------------------------------------- trims
// References let go are numbered 0 .. E - 1 (sequences in order, their pages in
// order), claims (a sequence that keeps a part of its last page) E + b.  Each
// takes one from shares[page]: at -1 nobody else holds the page, and the largest
// number, a claim if there is one, leaves its code there by an atomic minimum: it
// decides for the page (a claim keeps it, a reference gives it back).
constexpr int kCode = 1 << 30;
__device__ __forceinline__ int code_of(int number) { return -kCode - number; }

__global__ void __launch_bounds__(1024) fd_page_trim_kernel(const PagePlanParams p) {
    extern __shared__ int32_t s_mem[];
    int32_t* s_keep = s_mem;                    // [batch] tokens kept, -1: left as it is
    int32_t* s_first = s_keep + p.batch;        // [batch + 1] number of its first reference let go
    __shared__ long long s_sums[32];
    __shared__ uint32_t s_given[kMaxCtas];      // references of each CTA that give a page back
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x, ranks = gridDim.x;
    const int ps1 = (1 << p.page_shift) - 1;
    const int64_t capacity = static_cast<int64_t>(p.max_pages) << p.page_shift;
    grid_dependency_trigger();
    grid_dependency_wait();

    const int count = free_entries(p);
    bool bad = false, bad_page = false;
    auto tail_page = [&](int b, int keep) {     // the page that a sequence keeps a part of, -1: none
        if (keep < 0 || (keep & ps1) == 0) return -1;
        const int page = p.block_table[static_cast<int64_t>(b) * p.max_pages + (keep >> p.page_shift)];
        return page >= 0 && page < p.n_pages ? page : -1;
    };
    long long may_need = 0, let_go = 0;
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
        }
        int tail = -1;
        if (p.shares != nullptr && keep >= 0) {
            tail = tail_page(b, keep);
            bad_page |= tail < 0 && (keep & ps1) != 0;
        }
        const int may = tail >= 0 && __ldcg(p.shares + tail) > 0;
        long long all;
        const long long upto = may_need + block_scan(may, s_sums, all);
        may_need += all;
        if (may && upto > count) {
            bad = true;
            keep = -1;
        }
        const int n = keep >= 0 ? ((len + ps1) >> p.page_shift) - ((keep + ps1) >> p.page_shift) : 0;
        const long long end = let_go + block_scan(n, s_sums, all);
        let_go += all;
        if (b < p.batch) {
            s_keep[b] = keep;
            s_first[b] = static_cast<int32_t>(end - n);
        }
    }
    const int E = static_cast<int>(let_go);     // (< 2^30, the host's check)
    if (tid == 0) s_first[p.batch] = E;
    if (rank == 0 && bad) raise(kStatusSeqlenBit);
    if (rank == 0 && bad_page) raise(kStatusPageBit);
    __syncthreads();

    // a warp's references: [e0, e1)
    const int warps = ranks * (blockDim.x >> 5);
    const int per_warp = ((E + warps - 1) / warps + 31) / 32 * 32;
    const int e0 = min(static_cast<int64_t>(rank * (blockDim.x >> 5) + warp) * per_warp, static_cast<int64_t>(E));
    const int e1 = min(e0 + per_warp, E);
    auto page_of = [&](int e) {
        const int b = find(s_first, p.batch, e);
        const int j = ((s_keep[b] + ps1) >> p.page_shift) + e - s_first[b];
        const int page = p.block_table[static_cast<int64_t>(b) * p.max_pages + j];
        return page >= 0 && page < p.n_pages ? page : -1;
    };
    const int step = ranks * blockDim.x, b_first = rank * blockDim.x + tid;
    if (p.shares != nullptr) {
        cluster_barrier();          // every CTA has looked at the shares before
        for (int e = e0 + lane; e < e1; e += 32) {
            const int page = page_of(e);
            if (page >= 0) atomicSub(&p.shares[page], 1);
        }
        for (int b = b_first; b < p.batch; b += step) {
            const int page = tail_page(b, s_keep[b]);
            if (page >= 0) atomicSub(&p.shares[page], 1);
        }
        cluster_barrier();
        auto bid = [&](int page, int number) {
            if (__ldcg(p.shares + page) >= 0) return;
            const int was = atomicMin(&p.shares[page], code_of(number));
            if (was < -1 && was > -kCode) raise(kStatusPageBit);   // let go more often than held
        };
        for (int e = e0 + lane; e < e1; e += 32) {
            const int page = page_of(e);
            if (page >= 0) bid(page, e);
        }
        for (int b = b_first; b < p.batch; b += step) {
            const int page = tail_page(b, s_keep[b]);
            if (page >= 0) bid(page, E + b);
        }
        cluster_barrier();
    }
    auto given_back = [&](int e, int page) {
        return page >= 0 && (p.shares == nullptr || __ldcg(p.shares + page) == code_of(e));
    };
    int given = 0;
    for (int e = e0 + lane; e < e1 + lane; e += 32) {       // (whole warps)
        const int page = e < e1 ? page_of(e) : -1;
        if (e < e1 && page < 0) raise(kStatusPageBit);
        given += __popc(__ballot_sync(kFullMask, given_back(e, page)));
    }
    long long cta_given;
    const long long warp_end = block_scan(lane == 0 ? given : 0, s_sums, cta_given);
    int before = __shfl_sync(kFullMask, static_cast<int>(warp_end), 0) - given;     // of this CTA's warps before
    if (tid < ranks)
        remote_store(remote_smem(smem_u32(&s_given[rank]), tid), static_cast<uint32_t>(cta_given));
    long long taken = 0;
    if (p.shares != nullptr) {
        // which claims get copies; the first CTA writes them down
        for (int base = 0; base < p.batch; base += blockDim.x) {
            const int b = base + tid;
            const int page = b < p.batch ? tail_page(b, s_keep[b]) : -1;
            const int moves = page >= 0 && __ldcg(p.shares + page) != code_of(E + b);
            long long all;
            const long long upto = taken + block_scan(moves, s_sums, all);
            taken += all;
            if (rank == 0 && moves) {
                const int to = p.free_in[count - upto];
                if (to < 0 || to >= p.n_pages) raise(kStatusPageBit);
                p.copy_src[upto - 1] = page;
                p.copy_dst[upto - 1] = to;
                // (the entry is read as a tail by every CTA: written behind the barrier)
            }
        }
    }
    cluster_barrier();
    int all_given = 0;
    for (int r = 0; r < ranks; ++r) {
        if (r < rank) before += static_cast<int>(s_given[r]);
        all_given += static_cast<int>(s_given[r]);
    }
    const int base = count - static_cast<int>(taken);
    if (rank == 0 && p.shares != nullptr) {
        long long at = 0;
        for (int b0 = 0; b0 < p.batch; b0 += blockDim.x) {
            const int b = b0 + tid;
            const int page = b < p.batch ? tail_page(b, s_keep[b]) : -1;
            const bool stays = page >= 0 && __ldcg(p.shares + page) == code_of(E + b);
            const int moves = page >= 0 && !stays;
            long long all;
            const long long upto = at + block_scan(moves, s_sums, all);
            at += all;
            if (moves)
                p.block_table[static_cast<int64_t>(b) * p.max_pages + (s_keep[b] >> p.page_shift)] = p.copy_dst[upto - 1];
            if (stays) p.shares[page] = 0;      // (only its own claim looks for this code)
        }
    }
    int at = before;
    for (int e = e0 + lane; e < e1 + lane; e += 32) {
        const int page = e < e1 ? page_of(e) : -1;
        const bool mine = given_back(e, page);
        const unsigned votes = __ballot_sync(kFullMask, mine);
        if (mine) {
            const int64_t place = static_cast<int64_t>(base) + all_given - 1 - (at + __popc(votes & ((1u << lane) - 1u)));
            if (p.shares != nullptr) p.shares[page] = 0;
            if (place < p.n_free_max) p.free_pages[place] = page;
            else raise(kStatusPageBit);
        }
        at += __popc(votes);
    }
    if (rank != 0) return;
    for (int b = tid; b < p.batch; b += blockDim.x) p.seqlens_out[b] = s_keep[b] >= 0 ? s_keep[b] : p.seqlens[b];
    if (tid == 0) {
        *p.free_count_out = static_cast<int>(min(static_cast<int64_t>(base) + all_given, static_cast<int64_t>(p.n_free_max)));
        if (p.copy_count != nullptr) *p.copy_count = static_cast<int>(taken);
    }
}

// ---------------------------------------------------------------- compaction
// Held pages from n_keep on are bits of a map that lies over the CTAs' shared
// memories (range by range); a page's number among them is its CTA's start, its
// word's prefix and the bits below it.  The free stack is filtered in rounds of
// what the cluster's registers hold, read before it is written.
constexpr int kKeepEntries = 8;         // entries of the free stack a thread holds in a round

__global__ void __launch_bounds__(1024) fd_page_compact_kernel(const PagePlanParams p, int words_per_cta) {
    extern __shared__ int32_t s_mem[];
    int32_t* s_seg = s_mem;                                             // [batch + 1] first segment of the row
    uint32_t* s_bits = reinterpret_cast<uint32_t*>(s_seg + p.batch + 1);   // [words_per_cta]
    uint32_t* s_pref = s_bits + words_per_cta;                          // [words_per_cta] held pages of the words before
    __shared__ long long s_sums[32];
    __shared__ uint32_t s_held[kMaxCtas], s_kept[kMaxCtas];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x, ranks = gridDim.x;
    const int ps1 = (1 << p.page_shift) - 1, threads = blockDim.x;
    const int64_t capacity = static_cast<int64_t>(p.max_pages) << p.page_shift;
    grid_dependency_trigger();
    grid_dependency_wait();

    for (int w = tid; w < words_per_cta; w += threads) s_bits[w] = 0;
    const int count = free_entries(p);
    long long segments = 0;
    bool bad = false;
    for (int base = 0; base < p.batch; base += threads) {
        const int b = base + tid;
        int n = 0;
        if (b < p.batch) {
            const int len = p.seqlens[b];
            if (len < 0 || len > capacity) bad = true;
            else n = (((len + ps1) >> p.page_shift) + kSegment - 1) / kSegment;
        }
        long long all;
        const long long end = segments + block_scan(n, s_sums, all);
        segments += all;
        if (b < p.batch) s_seg[b] = static_cast<int32_t>(end - n);
    }
    if (tid == 0) s_seg[p.batch] = static_cast<int32_t>(segments);
    if (bad && rank == 0) raise(kStatusSeqlenBit);
    __syncthreads();
    cluster_barrier();              // the map is empty everywhere

    const int total = s_seg[p.batch], warps = ranks * (threads >> 5), w0 = rank * (threads >> 5) + warp;
    const uint32_t bits = smem_u32(s_bits), pref = smem_u32(s_pref);
    // calls f(table entry, page) for the live entries of this warp's segments that hold a page from n_keep on
    auto for_held = [&](auto f) {
        for (int s = w0; s < total; s += warps) {
            const int b = find(s_seg, p.batch, s);
            const int j0 = (s - s_seg[b]) * kSegment;
            const int n = (p.seqlens[b] + ps1) >> p.page_shift;
            int32_t* row = p.block_table + static_cast<int64_t>(b) * p.max_pages;
            int page[kSegment / 32];
#pragma unroll
            for (int k = 0; k < kSegment / 32; ++k) {
                const int j = j0 + 32 * k + lane;
                page[k] = j < n ? row[j] : 0;
                if (page[k] < 0 || page[k] >= p.n_pages) {
                    raise(kStatusPageBit);
                    page[k] = -1;
                } else if (j >= n) {
                    page[k] = -1;
                }
            }
#pragma unroll
            for (int k = 0; k < kSegment / 32; ++k)
                if (page[k] >= p.n_keep) f(row + j0 + 32 * k + lane, page[k]);
        }
    };
    for_held([&](int32_t*, int page) {
        const int x = page - p.n_keep, w = x >> 5;
        remote_or(remote_smem(bits + 4 * (w % words_per_cta), w / words_per_cta), 1u << (x & 31));
    });
    cluster_barrier();

    // numbers: prefix sums of the words' bits
    const int per_thread = (words_per_cta + threads - 1) / threads;
    const int wa = min(tid * per_thread, words_per_cta), wb = min(wa + per_thread, words_per_cta);
    int mine = 0;
    for (int w = wa; w < wb; ++w) mine += __popc(s_bits[w]);
    long long cta_held;
    int upto = static_cast<int>(block_scan(mine, s_sums, cta_held)) - mine;
    for (int w = wa; w < wb; ++w) {
        s_pref[w] = upto;
        upto += __popc(s_bits[w]);
    }
    if (tid < ranks) remote_store(remote_smem(smem_u32(&s_held[rank]), tid), static_cast<uint32_t>(cta_held));

    // the free stack without the pages from n_keep on
    int kept = 0;
    const int round = ranks * threads * kKeepEntries;
    for (int64_t base = 0; base == 0 || base < count; base += round) {
        int entry[kKeepEntries];
        const int64_t a = base + static_cast<int64_t>(w0) * (32 * kKeepEntries);
        int n = 0;
        unsigned votes[kKeepEntries];
#pragma unroll
        for (int k = 0; k < kKeepEntries; ++k) {
            const int64_t i = a + 32 * k + lane;
            entry[k] = i < count ? p.free_pages[i] : -1;
            if (i < count && (entry[k] < 0 || entry[k] >= p.n_pages)) raise(kStatusPageBit);
        }
#pragma unroll
        for (int k = 0; k < kKeepEntries; ++k) {
            votes[k] = __ballot_sync(kFullMask, entry[k] >= 0 && entry[k] < p.n_keep);
            n += __popc(votes[k]);
        }
        long long cta_kept;
        int at = __shfl_sync(kFullMask, static_cast<int>(block_scan(lane == 0 ? n : 0, s_sums, cta_kept)), 0) - n;
        if (tid < ranks) remote_store(remote_smem(smem_u32(&s_kept[rank]), tid), static_cast<uint32_t>(cta_kept));
        cluster_barrier();          // every CTA has read its entries
        at += kept;
        for (int r = 0; r < ranks; ++r) {
            if (r < rank) at += static_cast<int>(s_kept[r]);
            kept += static_cast<int>(s_kept[r]);
        }
#pragma unroll
        for (int k = 0; k < kKeepEntries; ++k) {
            if ((votes[k] >> lane) & 1u) p.free_pages[at + __popc(votes[k] & ((1u << lane) - 1u))] = entry[k];
            at += __popc(votes[k]);
        }
        cluster_barrier();          // (s_kept is free again, the entries are written)
    }
    int held = 0, my_start = 0;
    for (int r = 0; r < ranks; ++r) {
        if (r < rank) my_start += static_cast<int>(s_held[r]);
        held += static_cast<int>(s_held[r]);
    }
    const int moved = min(min(held, kept), p.n_copies);

    for_held([&](int32_t* entry, int page) {
        const int x = page - p.n_keep, w = x >> 5, owner = w / words_per_cta, in = w % words_per_cta;
        int number = static_cast<int>(remote_load(remote_smem(pref + 4 * in, owner))) +
                     __popc(remote_load(remote_smem(bits + 4 * in, owner)) & ((1u << (x & 31)) - 1u));
        for (int r = 0; r < owner; ++r) number += static_cast<int>(s_held[r]);
        if (number < moved) *entry = __ldcg(p.free_pages + kept - 1 - number);
    });
    for (int w = tid; w < words_per_cta; w += threads) {
        int number = my_start + static_cast<int>(s_pref[w]);
        for (uint32_t left = s_bits[w]; left != 0 && number < moved; left &= left - 1, ++number) {
            const int page = p.n_keep + (rank * words_per_cta + w) * 32 + __ffs(left) - 1;
            const int to = __ldcg(p.free_pages + kept - 1 - number);
            p.copy_src[number] = page;
            p.copy_dst[number] = to;
            if (p.shares != nullptr) {
                p.shares[to] = p.shares[page];
                p.shares[page] = 0;
            }
        }
    }
    if (rank == 0 && tid == 0) {
        if (moved < held) raise(kStatusPageBit);
        *p.free_count_out = kept - moved;
        *p.copy_count = moved;
    }
    cluster_barrier();              // nobody reads this CTA's shared memory any more
}

// One cluster of `ctas` CTAs.
template <typename Kern, typename... Args>
cudaError_t launch_cluster(Kern kern, int ctas, int threads, size_t smem, cudaStream_t stream, const Args&... args) {
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_page_fork(const PagePlanParams& p, cudaStream_t stream) {
    static std::atomic<unsigned long long> configured_ctx{0};
    cudaError_t e = allow_smem(fd_page_fork_kernel, (5 * FD_MAX_TABLE_BATCH + 1) * sizeof(int32_t), configured_ctx);
    if (e != cudaSuccess) return e;
    const size_t smem = (2 * static_cast<size_t>(p.batch) + 3 * static_cast<size_t>(p.n_forks) + 1) * sizeof(int32_t);
    const bool small = static_cast<int64_t>(p.n_forks) * p.max_pages <= 8192;
    return launch_cluster(fd_page_fork_kernel, small ? 1 : kMaxCtas, small ? 256 : 1024, smem, stream, p);
}

cudaError_t launch_page_trim(const PagePlanParams& p, cudaStream_t stream) {
    static std::atomic<unsigned long long> configured_ctx{0};
    cudaError_t e = allow_smem(fd_page_trim_kernel, (2 * FD_MAX_TABLE_BATCH + 1) * sizeof(int32_t), configured_ctx);
    if (e != cudaSuccess) return e;
    const size_t smem = (2 * static_cast<size_t>(p.batch) + 1) * sizeof(int32_t);
    const bool small = static_cast<int64_t>(p.batch) * p.max_pages <= 8192;
    return launch_cluster(fd_page_trim_kernel, small ? 1 : kMaxCtas, small ? 256 : 1024, smem, stream, p);
}

cudaError_t launch_page_compact(const PagePlanParams& p, cudaStream_t stream) {
    constexpr int kMaxWords = FD_MAX_COMPACT_PAGES / 32 / kMaxCtas;
    static std::atomic<unsigned long long> configured_ctx{0};
    cudaError_t e = allow_smem(fd_page_compact_kernel, (FD_MAX_TABLE_BATCH + 1 + 2 * (kMaxWords + 1)) * sizeof(int32_t),
                               configured_ctx);
    if (e != cudaSuccess) return e;
    const int64_t words = (static_cast<int64_t>(p.n_pages) - p.n_keep + 31) / 32;
    const int words_per_cta = static_cast<int>((words + kMaxCtas - 1) / kMaxCtas) + 1;
    const size_t smem = (static_cast<size_t>(p.batch) + 1 + 2 * static_cast<size_t>(words_per_cta)) * sizeof(int32_t);
    return launch_cluster(fd_page_compact_kernel, kMaxCtas, 1024, smem, stream, p, words_per_cta);
}

cudaError_t status_word_pages(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_status);
}

}  // namespace fdk
