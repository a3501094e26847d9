// fd_tables.cu -- page tables, slot map and positions of one serving step from
// the requests' lengths (fd_page_tables).
//
// With L_b tokens held, n_b new ones and pages of P tokens, sequence b needs
// ceil((L_b + n_b) / P) - ceil(L_b / P) new pages; the exclusive prefix sums of
// n_b and of the pages say which row of the step's ragged list and which entry
// of the free stack each token and page is.
//
// Nothing here is bound by bandwidth (12 bytes per token): the time is the
// chain lengths -> sums -> search -> table entry -> slot.  So it is one launch
// of one cluster of up to 8 CTAs; every CTA computes the (small) prefix sums
// for itself and then maps its share of the tokens, each thread finding its
// token's sequence by bisection in shared memory.  The outputs that may alias
// inputs are written behind a cluster barrier, after every CTA has read them.
// 64 requests of one token: 3.1 us; 60000 tokens of 8 requests: 10.5 us.
#include "../../include/fd.h"
#include "fd_cluster.cuh"
#include "fd_device.cuh"
#include "fd_internal.h"

namespace fdk {

namespace {

__device__ unsigned int g_status = 0;   // this file's bits of the device status word

__global__ void __launch_bounds__(1024) fd_page_tables_kernel(const PageParams p) {
    // per sequence: first new token of the step, first new page (-1: the
    // sequence gets nothing), tokens held
    extern __shared__ int32_t s_tab[];
    int32_t* s_tok = s_tab;                     // [batch + 1]
    int32_t* s_page = s_tok + p.batch + 1;      // [batch]
    int32_t* s_len = s_page + p.batch;          // [batch]
    __shared__ long long s_sums[32];
    grid_dependency_trigger();
    grid_dependency_wait();
    const int rank = blockIdx.x, ranks = gridDim.x;
    const int64_t capacity = static_cast<int64_t>(p.max_pages) << p.page_shift;
    const int ps1 = p.page_size - 1;
    int count = *p.free_count;
    bool bad = count < 0 || count > p.n_free_max;
    count = min(max(count, 0), p.n_free_max);

    long long tokens = 0, pages = 0;            // of the sequences before this round's
    int taken = 0;                              // pages given out (this thread's sequences)
    for (int base = 0; base < p.batch; base += blockDim.x) {
        const int b = base + threadIdx.x;
        int len = 0, n = 0;
        if (b < p.batch) {
            len = p.seqlens[b];
            n = p.new_tokens[b];
        }
        bool ok = len >= 0 && n >= 0 && static_cast<int64_t>(len) + n <= capacity;
        n = max(n, 0);
        long long all;
        const long long tok_end = tokens + block_scan(n, s_sums, all);
        tokens += all;
        ok = ok && tok_end <= p.n_slots;
        int have = 0, need = 0;
        if (ok) {
            have = (len >> p.page_shift) + ((len & ps1) != 0);
            need = static_cast<int>((static_cast<int64_t>(len) + n + ps1) >> p.page_shift) - have;
        }
        const long long page_end = pages + block_scan(need, s_sums, all);
        pages += all;
        ok = ok && (need == 0 || page_end <= count);
        if (ok && need > 0) taken = max(taken, static_cast<int>(page_end));
        bad |= b < p.batch && !ok;
        if (b < p.batch) {
            const long long start = tok_end - n;
            s_tok[b] = static_cast<int32_t>(start < INT32_MAX ? start : INT32_MAX);
            s_page[b] = ok ? static_cast<int32_t>(page_end - need) : -1;
            s_len[b] = len;
        }
    }
    if (threadIdx.x == 0) s_tok[p.batch] = static_cast<int32_t>(tokens < INT32_MAX ? tokens : INT32_MAX);
    if (bad && rank == 0) atomicOr(&g_status, kStatusSeqlenBit);
    // the prefix tables are complete, and (for the outputs that may alias
    // inputs) every CTA of the cluster has read its inputs
    __syncthreads();
    cluster_arrive();

    const int total = s_tok[p.batch];
    for (int64_t t = static_cast<int64_t>(rank) * blockDim.x + threadIdx.x; t < p.n_slots;
         t += static_cast<int64_t>(ranks) * blockDim.x) {
        int64_t slot = -1;
        int pos = -1;
        if (t < total) {
            int lo = 0, hi = p.batch;           // s_tok[lo] <= t < s_tok[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_tok[mid] <= t) lo = mid;
                else hi = mid;
            }
            const int len = s_len[lo], first = s_page[lo];
            const int i = static_cast<int>(t) - s_tok[lo];
            // (unsigned: a bad length may wrap; its position says nothing)
            pos = static_cast<int>(static_cast<unsigned>(len) + static_cast<unsigned>(i));
            if (first >= 0) {
                const int pi = pos >> p.page_shift, off = pos & ps1;
                const int have = (len >> p.page_shift) + ((len & ps1) != 0);
                int32_t* entry = p.block_table + static_cast<int64_t>(lo) * p.max_pages + pi;
                int page;
                if (pi < have) {
                    page = *entry;
                } else {
                    page = p.free_pages[count - 1 - (first + pi - have)];
                    if (off == 0) *entry = page;   // the page's first token, always a new one
                }
                if (page >= 0 && page < p.n_pages)
                    slot = (static_cast<int64_t>(page) << p.page_shift) + off;
                else
                    atomicOr(&g_status, kStatusPageBit);
            }
        }
        p.slots[t] = slot;
        if (p.positions != nullptr) p.positions[t] = pos;
    }

    __syncwarp();
    cluster_wait();
    if (rank != 0) return;
    for (int b = threadIdx.x; b <= p.batch; b += blockDim.x) {
        if (p.cu_tokens != nullptr) p.cu_tokens[b] = s_tok[b];
        if (b < p.batch)
            p.seqlens_out[b] = s_page[b] >= 0 ? s_len[b] + (s_tok[b + 1] - s_tok[b]) : s_len[b];
    }
    __shared__ int s_taken;
    if (threadIdx.x == 0) s_taken = 0;
    __syncthreads();
    if (taken > 0) atomicMax(&s_taken, taken);
    __syncthreads();
    if (threadIdx.x == 0) *p.free_count_out = count - s_taken;
}

}  // namespace

cudaError_t launch_page_tables(const PageParams& p, cudaStream_t stream) {
    // Time is latency: more threads mean longer barriers and scans, fewer mean
    // more rounds in turn; more CTAs share the rounds, up to the portable 8.
    // Threads 256 / 512 / 1024: 64 requests of one token 3.2 / 3.8 / 6.2 us, 300
    // 5.3 / 4.2 / 6.6, 8000 35.0 / 28.8 / 34.9; 8000 tokens of 8 requests 4.3 / 4.0 /
    // 6.1, 32000 10.1 / 7.2 / 8.1, 60000 17.0 / 10.8 / 10.5.  Tokens per CTA 512 / 1024 /
    // 2048 (512 threads): 2000 tokens of 8 requests 3.5 / 4.1 / 5.0, 8000 4.0 / 4.0 / 5.1.
    constexpr int64_t kTokensPerCta = 512;
    const int64_t want = (p.n_slots + kTokensPerCta - 1) / kTokensPerCta;
    const int ctas = want <= 1 ? 1 : want <= 2 ? 2 : want <= 4 ? 4 : 8;
    const int threads = p.n_slots <= 256 && p.batch <= 256 ? 256 : p.n_slots <= 49152 ? 512 : 1024;
    const size_t smem = (3 * static_cast<size_t>(p.batch) + 1) * sizeof(int32_t);
    // the limit of the largest batch, whatever this call's is (the default of
    // 48 KB counts the static arrays too): calls of two threads never lower it
    // under each other
    static std::atomic<unsigned long long> configured_ctx{0};
    cudaError_t e = allow_smem(fd_page_tables_kernel, (3 * FD_MAX_TABLE_BATCH + 1) * sizeof(int32_t), configured_ctx);
    if (e != cudaSuccess) return e;
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
    e = cudaLaunchKernelEx(&cfg, fd_page_tables_kernel, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t status_word_tables(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_status);
}

}  // namespace fdk
