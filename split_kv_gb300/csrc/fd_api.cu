// fd_api.cu -- the C ABI of the decode library (declared in include/fd.h):
// host-side validation, workspace layout, TMA descriptors and launches.
// Nothing here allocates device memory or synchronises a stream except
// fd_device_status(), which is documented to.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <mutex>

#include "../../include/fd.h"
#include "fd_internal.h"

namespace {

using fdk::kHeadDim;

constexpr size_t kAlign = 256;
constexpr int64_t kKeyTile = 128;   // keys per tile of fd_prompt

size_t round_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

struct WsLayout {
    size_t off_u, off_m, off_l, total;
};

WsLayout ws_layout(int64_t rows, int64_t splits) {
    WsLayout w;
    w.off_u = 0;
    w.off_m = round_up(static_cast<size_t>(rows * splits * kHeadDim) * sizeof(float));
    w.off_l = w.off_m + round_up(static_cast<size_t>(rows * splits) * sizeof(float));
    w.total = w.off_l + round_up(static_cast<size_t>(rows * splits) * sizeof(float));
    return w;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool aligned_to(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Addresses of out and lse: multiples of their elements' size.
bool outputs_aligned(int32_t out_dtype, const void* out, const float* lse) {
    return aligned_to(out, out_dtype == FD_F32 ? 4 : 2) && aligned_to(lse, 4);
}

// A stride in elements of `esize` bytes is usable by TMA: a multiple of 16 bytes.
bool stride_ok(int64_t s, int esize = 2) {
    return s >= 0 && (s * esize) % 16 == 0 && s < (int64_t(1) << 38);
}

// A stride of 0 over several entries (rows shared, as by torch's expand): a
// tensor map has none, whatever stride it was given instead would read other rows.
bool shared_rows(int64_t stride, int64_t entries) { return stride == 0 && entries > 1; }

int log2_of(int32_t x) {   // of a power of two
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

bool is_fp8(const fd_desc* d) { return d->kv_dtype == FD_E4M3; }
int cache_esize(const fd_desc* d) { return is_fp8(d) ? 1 : 2; }
// the type of q (and of the MMA operands): kv_dtype, or q_dtype for an fp8 cache
int q_type_of(const fd_desc* d) { return is_fp8(d) ? d->q_dtype : d->kv_dtype; }

int q_len_of(const fd_desc* d) { return d->q_len <= 1 ? 1 : d->q_len; }

int64_t rows_of(const fd_desc* d) {
    return static_cast<int64_t>(d->batch) * q_len_of(d) * d->n_q_heads;
}

int cols_of(const fd_desc* d) { return (d->n_q_heads / d->n_kv_heads) * q_len_of(d); }

bool umma_of(const fd_desc* d) {
    return fdk::use_umma(is_fp8(d), (d->flags & FD_FLAG_CUDA_CORES) != 0, cols_of(d));
}

int col_blocks_of(const fd_desc* d) { return umma_of(d) ? 1 : fdk::column_blocks(cols_of(d)); }

// Shape / layout checks shared by every entry point.  Pointer checks are
// done by the callers, which know which pointers they use.
fd_status check_desc(const fd_desc* d) {
    if (d == nullptr) return FD_ERR_INVALID_ARG;
    if ((d->flags & ~(FD_FLAG_CUDA_CORES | FD_FLAG_TEST_DROP_FIRST_STAGE)) != 0)
        return FD_ERR_INVALID_ARG;
    if (d->q_len < 0) return FD_ERR_INVALID_ARG;
    if (d->batch < 0 || d->n_q_heads < 1 || d->n_kv_heads < 1 || d->head_dim < 1)
        return FD_ERR_INVALID_ARG;
    if (d->n_q_heads % d->n_kv_heads != 0) return FD_ERR_INVALID_ARG;
    if (d->kv_dtype != FD_F16 && d->kv_dtype != FD_BF16 && d->kv_dtype != FD_E4M3)
        return d->kv_dtype == FD_F32 ? FD_ERR_UNSUPPORTED : FD_ERR_INVALID_ARG;
    if (d->reserved != 0) return FD_ERR_INVALID_ARG;
    if (is_fp8(d)) {
        if (d->q_dtype != FD_F16 && d->q_dtype != FD_BF16) return FD_ERR_INVALID_ARG;
        if (!std::isfinite(d->k_scale) || !std::isfinite(d->v_scale)) return FD_ERR_INVALID_ARG;
        if ((d->flags & FD_FLAG_CUDA_CORES) != 0) return FD_ERR_UNSUPPORTED;
    }
    if (d->out_dtype != FD_F16 && d->out_dtype != FD_BF16 && d->out_dtype != FD_F32)
        return FD_ERR_INVALID_ARG;
    if (d->head_dim != kHeadDim) return FD_ERR_UNSUPPORTED;
    const int G = d->n_q_heads / d->n_kv_heads;
    const int ql = q_len_of(d);
    if (ql > 16 || static_cast<int64_t>(G) * ql > 256) return FD_ERR_UNSUPPORTED;
    if ((d->flags & FD_FLAG_CUDA_CORES) != 0 && ((G != 1 && G != 2 && G != 4 && G != 8) || ql != 1))
        return FD_ERR_UNSUPPORTED;
    if (ql > 1 && !stride_ok(d->q_stride_t)) return FD_ERR_INVALID_ARG;
    if (d->n_splits > FD_MAX_SPLITS) return FD_ERR_UNSUPPORTED;
    if (d->page_size < 0) return FD_ERR_INVALID_ARG;
    if (d->page_size > 0) {
        if ((d->page_size & (d->page_size - 1)) != 0 || d->page_size > (1 << 20))
            return FD_ERR_INVALID_ARG;
        if (d->page_size < 8) return FD_ERR_UNSUPPORTED;
        if (d->max_pages_per_seq < 1) return FD_ERR_INVALID_ARG;
        if (static_cast<int64_t>(d->max_pages_per_seq) * d->page_size > INT32_MAX)
            return FD_ERR_INVALID_ARG;
    }
    if (d->kv_extent < 1 || d->kv_extent > INT32_MAX) return FD_ERR_INVALID_ARG;
    if (!stride_ok(d->q_stride_b) || !stride_ok(d->q_stride_h)) return FD_ERR_INVALID_ARG;
    const int es = cache_esize(d);
    if (!stride_ok(d->k_stride_b, es) || !stride_ok(d->k_stride_h, es) || !stride_ok(d->k_stride_t, es))
        return FD_ERR_INVALID_ARG;
    if (!stride_ok(d->v_stride_b, es) || !stride_ok(d->v_stride_h, es) || !stride_ok(d->v_stride_t, es))
        return FD_ERR_INVALID_ARG;
    if (d->k_stride_t < kHeadDim || d->v_stride_t < kHeadDim) return FD_ERR_INVALID_ARG;
    if (d->max_seqlen < 0) return FD_ERR_INVALID_ARG;
    return FD_OK;
}

// Split count a call uses: the descriptor's, or the planner's.
int32_t splits_for(const fd_desc* d) {
    if (d->n_splits >= 1) return d->n_splits;
    return fdk::plan_launch(d->batch, d->n_kv_heads, cols_of(d), is_fp8(d),
                            (d->flags & FD_FLAG_CUDA_CORES) != 0, d->max_seqlen, 0);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

typedef CUresult (*CtxGetCurrentFn)(CUcontext*);
typedef CUresult (*CtxGetIdFn)(CUcontext, unsigned long long*);

template <typename Fn>
Fn driver_fn(const char* name, int version) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion(name, &p, version, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
        return reinterpret_cast<Fn>(p);
    return nullptr;
}

// 4-D map over one cache: dims (head_dim, tokens, kv heads, sequences|pages),
// 128-byte swizzle, zero fill outside.  Box: (64 dims, rows, 1, 1) of 16-bit
// elements, or (128 dims, rows, 1, 1) of 8-bit ones -- 128 bytes a row either way.
fd_status make_map(CUtensorMap* map, const fd_desc* d, const void* base, int64_t sb, int64_t sh,
                   int64_t st) {
    EncodeTiledFn enc = encode_fn();
    if (enc == nullptr) return FD_ERR_CUDA;
    const bool paged = d->page_size > 0;
    const int64_t n_tok = paged ? d->page_size : d->kv_extent;
    const int64_t n_outer = paged ? d->kv_extent : (d->batch > 0 ? d->batch : 1);
    const int cols = (d->n_q_heads / d->n_kv_heads) * q_len_of(d);
    const int rows = paged ? (d->page_size < fdk::kPagedBoxRows ? d->page_size : fdk::kPagedBoxRows)
                           : fdk::stage_tokens(is_fp8(d), cols);
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(n_tok),
                          static_cast<cuuint64_t>(d->n_kv_heads), static_cast<cuuint64_t>(n_outer)};
    // byte strides of dims 1..3; a stride of a size-1 dim is never used, but
    // must still be a valid multiple of 16 (other strides of 0 are refused)
    const int es = cache_esize(d);
    auto bs = [es](int64_t s) { return static_cast<cuuint64_t>(s > 0 ? s * es : 16); };
    cuuint64_t strides[3] = {bs(st), bs(sh), bs(sb)};
    cuuint32_t box[4] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(rows), 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUtensorMapDataType dt = is_fp8(d) ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : d->kv_dtype == FD_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                           : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUresult r = enc(map, dt, 4, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FD_OK : FD_ERR_INVALID_ARG;
}

// direct (S = 1 only): the split kernel writes out / lse itself, no combine.
fd_status split_impl(const fd_desc* d, int32_t S, const void* q, const void* k, const void* v,
                     const int32_t* seqlens, const int32_t* block_table, void* workspace,
                     size_t workspace_bytes, cudaStream_t stream, bool direct = false,
                     void* out = nullptr, float* lse = nullptr, const fd_kv_scales* scales = nullptr) {
    // a direct one-split launch given no workspace never touches one
    const bool no_ws = direct && S == 1 && out != nullptr && workspace == nullptr;
    if (q == nullptr || k == nullptr || v == nullptr || seqlens == nullptr ||
        (workspace == nullptr && !no_ws))
        return FD_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v)) return FD_ERR_INVALID_ARG;
    const bool paged = d->page_size > 0;
    if (paged != (block_table != nullptr)) return FD_ERR_INVALID_ARG;
    const int64_t outer = paged ? d->kv_extent : d->batch;
    if (shared_rows(d->k_stride_b, outer) || shared_rows(d->v_stride_b, outer) ||
        shared_rows(d->k_stride_h, d->n_kv_heads) || shared_rows(d->v_stride_h, d->n_kv_heads))
        return FD_ERR_INVALID_ARG;
    const int64_t rows = rows_of(d);
    const WsLayout w = ws_layout(rows, S);
    if ((reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0) return FD_ERR_WORKSPACE;
    if (!no_ws && workspace_bytes < w.total) return FD_ERR_WORKSPACE;
    if (d->batch == 0) return FD_OK;
    if (d->batch > 65535 || d->n_kv_heads > 65535)   // grid (S * col_blocks, n_kv_heads, batch)
        return FD_ERR_UNSUPPORTED;

    CUtensorMap tmK, tmV;
    fd_status st = make_map(&tmK, d, k, d->k_stride_b, d->k_stride_h, d->k_stride_t);
    if (st != FD_OK) return st;
    st = make_map(&tmV, d, v, d->v_stride_b, d->v_stride_h, d->v_stride_t);
    if (st != FD_OK) return st;

    fdk::SplitParams p;
    p.q = q;
    p.q_sb = d->q_stride_b;
    p.q_sh = d->q_stride_h;
    p.q_st = q_len_of(d) > 1 ? d->q_stride_t : 0;
    p.group = d->n_q_heads / d->n_kv_heads;
    p.q_len = q_len_of(d);
    p.cols = p.group * p.q_len;
    p.col_blocks = col_blocks_of(d);
    p.seqlens = seqlens;
    p.block_table = block_table;
    p.max_pages = paged ? d->max_pages_per_seq : 0;
    p.page_size = paged ? d->page_size : 0;
    int shift = 0;
    while (paged && (1 << shift) < d->page_size) ++shift;
    p.page_shift = shift;
    p.capacity = paged ? d->max_pages_per_seq * d->page_size : static_cast<int32_t>(d->kv_extent);
    p.n_pages = paged ? static_cast<int32_t>(d->kv_extent) : 0;
    p.n_q_heads = d->n_q_heads;
    p.n_kv_heads = d->n_kv_heads;
    p.batch = d->batch;
    p.n_splits = S;
    // whole 16-token units (8-token pages: 8), the paged box height, so a
    // TMA box never crosses a page and paged and contiguous caches split alike
    p.split_unit = paged && d->page_size < fdk::kSplitUnit ? d->page_size : fdk::kSplitUnit;
    p.drop_first_stage = (d->flags & FD_FLAG_TEST_DROP_FIRST_STAGE) != 0 ? 1 : 0;
    // fp8 cache: key = k_scale x stored, so the scale folds into the score
    // scale; value = v_scale x stored, applied to the split's u
    p.score_scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(kHeadDim)) *
                                            (is_fp8(d) ? static_cast<double>(d->k_scale) : 1.0));
    p.v_scale = is_fp8(d) ? d->v_scale : 1.0f;
    char* ws = static_cast<char*>(workspace);
    p.ws_u = no_ws ? nullptr : reinterpret_cast<float*>(ws + w.off_u);
    p.ws_m = no_ws ? nullptr : reinterpret_cast<float*>(ws + w.off_m);
    p.ws_l = no_ws ? nullptr : reinterpret_cast<float*>(ws + w.off_l);
    p.direct = direct && S == 1 && out != nullptr ? 1 : 0;
    p.out_dtype = d->out_dtype == FD_F16 ? 0 : d->out_dtype == FD_BF16 ? 1 : 2;
    p.out = out;
    p.lse = lse;
    p.scale_k = p.scale_v = nullptr;
    if (scales != nullptr) {
        p.scale_k = scales->k;
        p.scale_v = scales->v;
        p.scale_kb = scales->k_stride_b;
        p.scale_kh = scales->k_stride_h;
        p.scale_kn = scales->k_stride_n;
        p.scale_vb = scales->v_stride_b;
        p.scale_vh = scales->v_stride_h;
        p.scale_vn = scales->v_stride_n;
        p.scale_shift = log2_of(scales->block);
    }
    const cudaError_t e = fdk::launch_split(tmK, tmV, p, q_type_of(d), is_fp8(d),
                                            (d->flags & FD_FLAG_CUDA_CORES) != 0, d->batch,
                                            d->n_kv_heads, stream);
    return e == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

// The block scales of an E4M3 cache with `page_size`-token pages (0: contiguous).
fd_status check_scales(const fd_kv_scales* s, int32_t page_size) {
    if (s == nullptr || s->k == nullptr || s->v == nullptr || s->reserved != 0) return FD_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(s->k) & 3u) != 0 || (reinterpret_cast<uintptr_t>(s->v) & 3u) != 0)
        return FD_ERR_INVALID_ARG;
    if (s->block < 1 || (s->block & (s->block - 1)) != 0) return FD_ERR_INVALID_ARG;
    if (s->block > 1024) return FD_ERR_UNSUPPORTED;
    if (page_size > 0 && s->block > page_size) return FD_ERR_INVALID_ARG;
    for (const int64_t st : {s->k_stride_b, s->k_stride_h, s->k_stride_n, s->v_stride_b, s->v_stride_h, s->v_stride_n})
        if (st < 0 || st >= (int64_t(1) << 38)) return FD_ERR_INVALID_ARG;
    return FD_OK;
}

fd_status combine_impl(const fd_desc* d, int32_t S, const void* workspace, size_t workspace_bytes,
                       void* out, float* lse, cudaStream_t stream) {
    if (workspace == nullptr || out == nullptr) return FD_ERR_INVALID_ARG;
    const int64_t rows = rows_of(d);
    const WsLayout w = ws_layout(rows, S);
    if ((reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0) return FD_ERR_WORKSPACE;
    if (workspace_bytes < w.total) return FD_ERR_WORKSPACE;
    if (rows == 0) return FD_OK;
    if (rows > INT32_MAX) return FD_ERR_UNSUPPORTED;
    const char* ws = static_cast<const char*>(workspace);
    fdk::CombineParams p;
    p.ws_u = reinterpret_cast<const float*>(ws + w.off_u);
    p.ws_m = reinterpret_cast<const float*>(ws + w.off_m);
    p.ws_l = reinterpret_cast<const float*>(ws + w.off_l);
    p.out = out;
    p.lse = lse;
    p.rows = static_cast<int32_t>(rows);
    p.n_splits = S;
    p.out_dtype = d->out_dtype == FD_F16 ? 0 : d->out_dtype == FD_BF16 ? 1 : 2;
    const cudaError_t e = fdk::launch_combine(p, stream);
    return e == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

// ---- prompts
fd_status check_prompt(const fd_prompt_desc* d) {
    if (d == nullptr || d->batch < 0 || d->n_q_heads < 1 || d->n_kv_heads < 1 || d->head_dim < 1 || d->total_q < 0 ||
        d->total_k < 0 || d->max_q < 0 || d->max_k < 0)
        return FD_ERR_INVALID_ARG;
    if (d->n_q_heads % d->n_kv_heads != 0) return FD_ERR_INVALID_ARG;
    if (d->flags != 0 || d->reserved != 0 || (d->causal != 0 && d->causal != 1)) return FD_ERR_INVALID_ARG;
    if (d->dtype != FD_F16 && d->dtype != FD_BF16)
        return d->dtype == FD_F32 || d->dtype == FD_E4M3 ? FD_ERR_UNSUPPORTED : FD_ERR_INVALID_ARG;
    if (d->out_dtype != FD_F16 && d->out_dtype != FD_BF16 && d->out_dtype != FD_F32) return FD_ERR_INVALID_ARG;
    if (d->head_dim != kHeadDim) return FD_ERR_UNSUPPORTED;
    if (d->n_splits > FD_MAX_SPLITS || d->n_q_heads > 65535) return FD_ERR_UNSUPPORTED;
    for (const int64_t s : {d->q_stride_t, d->q_stride_h, d->k_stride_t, d->k_stride_h, d->v_stride_t, d->v_stride_h})
        if (!stride_ok(s)) return FD_ERR_INVALID_ARG;
    if (d->q_stride_t < kHeadDim || d->k_stride_t < kHeadDim || d->v_stride_t < kHeadDim) return FD_ERR_INVALID_ARG;
    if (shared_rows(d->q_stride_h, d->n_q_heads) || shared_rows(d->k_stride_h, d->n_kv_heads) ||
        shared_rows(d->v_stride_h, d->n_kv_heads))
        return FD_ERR_INVALID_ARG;
    return FD_OK;
}

bool pair_heads_of(const fd_prompt_desc* d) { return (d->n_q_heads / d->n_kv_heads) % 2 == 0; }

// Query tiles per head unit: every sequence may end inside one.
int64_t prompt_tiles(const fd_prompt_desc* d) {
    return d->total_q / (pair_heads_of(d) ? 128 : 256) + d->batch;
}

// Key splits per query tile.  Few tiles over long keys leave SMs idle, so the
// keys are cut where that pays, by the time it takes in microseconds: an item
// walks its key tiles at 1.5 each, and each wave of items costs 8 beside them
// (first loads, epilogues); joining the parts takes 8, and 0.3 a split.  The
// walk is the longest sequence's part or, if that is more, an average part
// (total_k / batch keys) in each wave.  The query tiles are the most that the
// sequences can have.  A part has four key tiles at least, there are 32 parts at
// most, and cutting has to save an eighth.
// One split against planned, measured: 64 queries over 9000 keys, 8 / 2 heads
// 116 -> 30 us; 200 over 12000, 32 / 8, 152 -> 66; 512 over 4000, 8 / 8,
// 54 -> 36; 4 single queries, 32 / 8, all over 9000 keys 124 -> 78, one over
// 9000 and three over 100 124 -> 49.  Left whole: 64 sequences of 2 queries, 32 /
// 8, one over 9000 keys and the others over 300 (175; in two 233, in nine 367);
// 16 single queries over 2500, 8 / 8 (40; in two 54).
int32_t prompt_splits(const fd_prompt_desc* d) {
    if (d->n_splits >= 1) return d->n_splits;
    const int64_t span = pair_heads_of(d) ? 128 : 256;
    const int64_t seqs = std::min(d->batch, d->total_q);   // (with queries, at most)
    if (seqs < 1) return 1;
    const double units = static_cast<double>((d->total_q + seqs * (span - 1)) / span) *
                         (pair_heads_of(d) ? d->n_q_heads / 2 : d->n_q_heads);
    const double all_tiles = static_cast<double>(d->total_k) / kKeyTile / d->batch;   // of a sequence on average
    const int64_t key_tiles = ((d->max_k > 0 ? d->max_k : (d->total_k + d->batch - 1) / d->batch) + kKeyTile - 1) / kKeyTile;
    if (key_tiles < 16) return 1;
    const int sms = fd_num_sms(-1);
    if (sms < 1) return 1;
    auto time = [&](int64_t s) {
        const double waves = std::ceil(units * s / sms);
        const double walk = std::max(static_cast<double>((key_tiles + s - 1) / s), waves * all_tiles / s);
        return 1.5 * walk + 8.0 * waves + (s > 1 ? 8.0 + 0.3 * s : 0.0);
    };
    int64_t best = 1;
    for (int64_t s = 2; s <= std::min(key_tiles / 4, static_cast<int64_t>(32)); ++s)
        if (time(s) < time(best)) best = s;
    return time(best) < 0.875 * time(1) ? static_cast<int32_t>(best) : 1;
}

// 3-D map over packed rows: dims (head_dim, rows, heads), boxes of 64 dims x
// 128 rows with 128-byte swizzle, zero fill outside.
fd_status make_rows_map(CUtensorMap* map, bool bf16, const void* base, int64_t rows, int64_t heads, int64_t st, int64_t sh) {
    EncodeTiledFn enc = encode_fn();
    if (enc == nullptr) return FD_ERR_CUDA;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(rows),
                          static_cast<cuuint64_t>(heads), 1};
    // (a stride of 0 belongs to a size-1 dim here, see shared_rows)
    auto bs = [](int64_t s) { return static_cast<cuuint64_t>(s > 0 ? s * 2 : 16); };
    cuuint64_t strides[3] = {bs(st), bs(sh), 16};
    cuuint32_t box[4] = {64, 128, 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                           const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FD_OK : FD_ERR_INVALID_ARG;
}

// What fd_page_fork, fd_page_trim and fd_page_compact ask of a descriptor.
fd_status check_pages(const fd_page_desc* d) {
    if (d == nullptr || d->batch < 0 || d->page_size < 1 || (d->page_size & (d->page_size - 1)) != 0 ||
        d->page_size > (1 << 20) || d->max_pages_per_seq < 1 || d->n_pages < 1 || d->n_free_max < 0 || d->n_slots < 0)
        return FD_ERR_INVALID_ARG;
    if (d->page_size < 8 || d->batch > FD_MAX_TABLE_BATCH) return FD_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(d->max_pages_per_seq) * d->page_size > INT32_MAX) return FD_ERR_INVALID_ARG;
    return FD_OK;
}

// Addresses of int32 arrays; `needed` ones may not be null.
bool ints_ok(std::initializer_list<const void*> needed, std::initializer_list<const void*> may_be_null) {
    for (const void* x : needed)
        if (x == nullptr || !aligned_to(x, 4)) return false;
    for (const void* x : may_be_null)
        if (!aligned_to(x, 4)) return false;
    return true;
}

fdk::PagePlanParams page_plan(const fd_page_desc* d) {
    fdk::PagePlanParams p = {};
    p.batch = d->batch;
    p.page_shift = log2_of(d->page_size);
    p.max_pages = d->max_pages_per_seq;
    p.n_pages = d->n_pages;
    p.n_free_max = d->n_free_max;
    p.n_copies = d->n_slots;
    return p;
}

fd_status check_rope(const fd_rope_desc* d, bool cached, bool k_rows) {
    if (d == nullptr || d->n_tokens < 0 || d->n_q_heads < 0 || d->n_kv_heads < 0 || d->n_q_heads + static_cast<int64_t>(d->n_kv_heads) < 1 ||
        d->head_dim < 1)
        return FD_ERR_INVALID_ARG;
    if (d->flags != 0 || d->reserved != 0 || (d->interleaved != 0 && d->interleaved != 1) ||
        (d->norm & ~(FD_NORM_Q | FD_NORM_K)) != 0)
        return FD_ERR_INVALID_ARG;
    if (d->dtype != FD_F16 && d->dtype != FD_BF16)
        return d->dtype == FD_F32 || d->dtype == FD_E4M3 ? FD_ERR_UNSUPPORTED : FD_ERR_INVALID_ARG;
    if (d->norm != 0 && d->w_dtype != FD_F16 && d->w_dtype != FD_BF16 && d->w_dtype != FD_F32)
        return d->w_dtype == FD_E4M3 ? FD_ERR_UNSUPPORTED : FD_ERR_INVALID_ARG;
    if (d->head_dim != kHeadDim) return FD_ERR_UNSUPPORTED;
    if (d->rot_dim < 0 || d->rot_dim > kHeadDim || d->rot_dim % 2 != 0) return FD_ERR_INVALID_ARG;
    if (d->rot_dim % 16 != 0 || d->n_q_heads > 65535 || d->n_kv_heads > 65535) return FD_ERR_UNSUPPORTED;
    if (!(d->eps >= 0.f) || !std::isfinite(d->eps) || !std::isfinite(d->rot_scale)) return FD_ERR_INVALID_ARG;
    for (const int64_t s : {d->q_stride_t, d->q_stride_h, d->k_src_stride_t, d->k_src_stride_h, d->v_src_stride_t,
                            d->v_src_stride_h, d->q_out_stride_t, d->q_out_stride_h, d->k_out_stride_t,
                            d->k_out_stride_h, d->q_w_stride_h, d->k_w_stride_h})
        if (!stride_ok(s)) return FD_ERR_INVALID_ARG;
    // what is written has a place of its own
    if (d->n_q_heads > 0 && ((d->q_out_stride_t < kHeadDim && d->n_tokens > 1) || (d->q_out_stride_h < kHeadDim && d->n_q_heads > 1)))
        return FD_ERR_INVALID_ARG;
    if (k_rows && ((d->k_out_stride_t < kHeadDim && d->n_tokens > 1) || (d->k_out_stride_h < kHeadDim && d->n_kv_heads > 1)))
        return FD_ERR_INVALID_ARG;
    if (!cached) return FD_OK;
    if (d->n_kv_heads < 1) return FD_ERR_INVALID_ARG;
    const bool fp8 = d->cache_dtype == FD_E4M3;
    if (!fp8 && d->cache_dtype != d->dtype)
        return d->cache_dtype == FD_F16 || d->cache_dtype == FD_BF16 || d->cache_dtype == FD_F32 ? FD_ERR_UNSUPPORTED
                                                                                               : FD_ERR_INVALID_ARG;
    if (fp8)
        for (const float s : {d->k_scale, d->v_scale})
            if (!(s > 0.f) || !std::isnormal(s)) return FD_ERR_INVALID_ARG;
    if (d->page_size < 0) return FD_ERR_INVALID_ARG;
    if (d->page_size > 0) {
        if ((d->page_size & (d->page_size - 1)) != 0 || d->page_size > (1 << 20)) return FD_ERR_INVALID_ARG;
        if (d->page_size < 8) return FD_ERR_UNSUPPORTED;
    } else if (d->batch < 1) {
        return FD_ERR_INVALID_ARG;
    }
    if (d->kv_extent < 1 || d->kv_extent > INT32_MAX) return FD_ERR_INVALID_ARG;
    const int es = fp8 ? 1 : 2;
    for (const int64_t s : {d->k_stride_b, d->k_stride_h, d->k_stride_t, d->v_stride_b, d->v_stride_h, d->v_stride_t})
        if (!stride_ok(s, es)) return FD_ERR_INVALID_ARG;
    if (d->k_stride_t < kHeadDim || d->v_stride_t < kHeadDim) return FD_ERR_INVALID_ARG;
    const int64_t lead = d->page_size > 0 ? d->kv_extent : d->batch;
    if (shared_rows(d->k_stride_b, lead) || shared_rows(d->v_stride_b, lead) || shared_rows(d->k_stride_h, d->n_kv_heads) ||
        shared_rows(d->v_stride_h, d->n_kv_heads))
        return FD_ERR_INVALID_ARG;
    return FD_OK;
}

// A pool with its dimensions joined where one goes on in the next, and the
// largest unit that divides all it is addressed by.
struct PoolShape {
    int64_t page_stride, stride0, stride1;
    int64_t extent0, extent1, row_bytes;
    bool operator==(const PoolShape& o) const {
        return page_stride == o.page_stride && stride0 == o.stride0 && stride1 == o.stride1 && extent0 == o.extent0 &&
               extent1 == o.extent1 && row_bytes == o.row_bytes;
    }
};

PoolShape pool_shape(const fd_pool& x) {
    PoolShape s = {x.page_stride, x.stride[0], x.stride[1], x.extent[0], x.extent[1], x.row_bytes};
    // rows in the order of their addresses (a copy does not care which index is the outer one)
    if (s.extent1 == 1 || (s.extent0 > 1 && s.stride0 < s.stride1)) {
        std::swap(s.stride0, s.stride1);
        std::swap(s.extent0, s.extent1);
    }
    for (int i = 0; i < 2; ++i)
        if (s.extent1 == 1 || s.stride1 == s.row_bytes) {   // the inner rows lie end to end: one row
            s.row_bytes *= s.extent1;
            s.stride1 = s.stride0;
            s.extent1 = s.extent0;
            s.stride0 = 0;
            s.extent0 = 1;
        }
    if (s.extent0 == 1) s.stride0 = 0;
    if (s.extent1 == 1) s.stride1 = 0;
    return s;
}

bool same_shape(const fd_pool& a, const fd_pool& b) {
    if (a.page_stride != b.page_stride) return false;
    if (a.stride[0] == b.stride[0] && a.stride[1] == b.stride[1] &&
        a.extent[0] == b.extent[0] && a.extent[1] == b.extent[1] && a.row_bytes == b.row_bytes)
        return true;
    return pool_shape(a) == pool_shape(b);
}

int pool_unit(const PoolShape& s, const void* base) {
    const uint64_t bits = static_cast<uint64_t>(s.page_stride) | static_cast<uint64_t>(s.stride0) |
                          static_cast<uint64_t>(s.stride1) | static_cast<uint64_t>(s.row_bytes) |
                          reinterpret_cast<uintptr_t>(base);
    int unit = 16;
    while ((bits & static_cast<uint64_t>(unit - 1)) != 0) unit /= 2;
    return unit;
}

fd_status check_pool(const fd_pool& x, int32_t n_pages) {
    if (x.base == nullptr || x.reserved != 0 || x.row_bytes < 1) return FD_ERR_INVALID_ARG;
    int64_t last = x.row_bytes;             // bytes from a page's first to behind its last
    for (int i = 0; i < 2; ++i) {
        if (x.extent[i] < 1 || x.stride[i] < 0 || x.stride[i] >= (int64_t(1) << 40)) return FD_ERR_INVALID_ARG;
        if (x.extent[i] > 1 && x.stride[i] < x.row_bytes) return FD_ERR_INVALID_ARG;   // rows on top of each other
        last += static_cast<int64_t>(x.extent[i] - 1) * x.stride[i];
        if (last > (int64_t(1) << 42)) return FD_ERR_INVALID_ARG;
    }
    if (x.page_stride < 1 || x.page_stride >= (int64_t(1) << 40)) return FD_ERR_INVALID_ARG;
    if (n_pages > 1 && x.page_stride < x.row_bytes) return FD_ERR_INVALID_ARG;
    if (x.page_stride > (int64_t(1) << 46) / n_pages) return FD_ERR_INVALID_ARG;         // (offsets stay within 64 bits)
    return FD_OK;
}

// ---- fixed workspace for fd_decode_static (callers that cannot allocate)
// The split states of fd_decode_static live here instead of in a caller
// buffer.  Every device that loads the library holds this array until exit.
static __device__ __align__(256) unsigned char g_static_workspace[FD_STATIC_WORKSPACE_BYTES];

// The array's device address in each CUDA context that used it, looked up
// once per context: the address belongs to the context, and a context that
// is destroyed and created again (cudaDeviceReset) may place it elsewhere.
// (In host code the symbol is only a host-side stand-in; handing it to a
// kernel would read the wrong memory.)
constexpr int kStaticSlots = 64;
std::mutex g_static_mutex;
unsigned long long g_static_ctx[kStaticSlots] = {};
void* g_static_ptr[kStaticSlots] = {};
int g_static_next = 0;

fd_status static_workspace(void** ptr) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FD_ERR_CUDA;
    const unsigned long long ctx = fdk::current_context_id();
    std::lock_guard<std::mutex> lock(g_static_mutex);
    if (ctx != 0) {
        for (int i = 0; i < kStaticSlots; ++i)
            if (g_static_ctx[i] == ctx) {
                *ptr = g_static_ptr[i];
                return FD_OK;
            }
    }
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_static_workspace) != cudaSuccess || p == nullptr) return FD_ERR_CUDA;
    if (ctx != 0) {   // without a context id every call looks the address up again
        g_static_ctx[g_static_next] = ctx;
        g_static_ptr[g_static_next] = p;
        g_static_next = (g_static_next + 1) % kStaticSlots;
    }
    *ptr = p;
    return FD_OK;
}

}  // namespace

namespace fdk {

unsigned long long current_context_id() {
    static CtxGetCurrentFn get_current = nullptr;
    static CtxGetIdFn get_id = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        get_current = driver_fn<CtxGetCurrentFn>("cuCtxGetCurrent", 4000);
        get_id = driver_fn<CtxGetIdFn>("cuCtxGetId", 12000);
    });
    if (get_current == nullptr || get_id == nullptr) return 0;
    CUcontext c = nullptr;
    if (get_current(&c) != CUDA_SUCCESS || c == nullptr) return 0;
    unsigned long long id = 0;
    return get_id(c, &id) == CUDA_SUCCESS ? id : 0;
}

}  // namespace fdk

extern "C" {

int32_t fd_abi_version(void) { return FD_ABI_VERSION; }

const char* fd_status_string(int32_t s) {
    switch (s) {
        case FD_OK: return "ok";
        case FD_ERR_INVALID_ARG: return "invalid argument";
        case FD_ERR_UNSUPPORTED: return "unsupported shape or dtype";
        case FD_ERR_WORKSPACE: return "workspace missing, too small or misaligned";
        case FD_ERR_CUDA: return "CUDA error";
        case FD_ERR_DEVICE_TIMEOUT: return "a device wait timed out";
        case FD_ERR_DEVICE_BOUNDS: return "a sequence length or page index was out of range";
        default: return "unknown status";
    }
}

size_t fd_workspace_size(const fd_desc* desc, int32_t n_splits) {
    if (check_desc(desc) != FD_OK) return 0;
    int32_t S = n_splits;
    if (S <= 0) S = splits_for(desc);
    if (S < 1 || S > FD_MAX_SPLITS) return 0;
    return ws_layout(rows_of(desc), S).total;
}

fd_status fd_split_states(const fd_desc* desc, const void* q, const void* k_cache,
                          const void* v_cache, const int32_t* seqlens, const int32_t* block_table,
                          void* workspace, size_t workspace_bytes, void* stream) {
    fd_status st = check_desc(desc);
    if (st != FD_OK) return st;
    const int32_t S = splits_for(desc);
    if (S < 1) return static_cast<fd_status>(S < 0 ? S : FD_ERR_INVALID_ARG);
    return split_impl(desc, S, q, k_cache, v_cache, seqlens, block_table, workspace,
                      workspace_bytes, static_cast<cudaStream_t>(stream));
}

fd_status fd_combine_states(const fd_desc* desc, const void* workspace, size_t workspace_bytes,
                            void* out, float* lse, void* stream) {
    fd_status st = check_desc(desc);
    if (st != FD_OK) return st;
    if (desc->n_splits < 1) return FD_ERR_INVALID_ARG;
    return combine_impl(desc, desc->n_splits, workspace, workspace_bytes, out, lse,
                        static_cast<cudaStream_t>(stream));
}

fd_status fd_decode(const fd_desc* desc, const void* q, const void* k_cache, const void* v_cache,
                    const int32_t* seqlens, const int32_t* block_table, void* out, float* lse,
                    void* workspace, size_t workspace_bytes, void* stream) {
    fd_status st = check_desc(desc);
    if (st != FD_OK) return st;
    if (out == nullptr) return FD_ERR_INVALID_ARG;
    const int32_t S = splits_for(desc);
    if (S < 1) return static_cast<fd_status>(S < 0 ? S : FD_ERR_INVALID_ARG);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // one split: the split kernel writes the result itself (no combine launch)
    st = split_impl(desc, S, q, k_cache, v_cache, seqlens, block_table, workspace, workspace_bytes, s,
                    S == 1, out, lse);
    if (st != FD_OK || S == 1) return st;
    return combine_impl(desc, S, workspace, workspace_bytes, out, lse, s);
}

fd_status fd_decode_scaled(const fd_desc* desc, const fd_kv_scales* scales, const void* q,
                           const void* k_cache, const void* v_cache, const int32_t* seqlens,
                           const int32_t* block_table, void* out, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
    fd_status st = check_desc(desc);
    if (st != FD_OK) return st;
    if (!is_fp8(desc)) return FD_ERR_INVALID_ARG;
    st = check_scales(scales, desc->page_size);
    if (st != FD_OK) return st;
    if (desc->batch == 0) return FD_OK;   // (an empty tensor's address is null)
    if (out == nullptr || !outputs_aligned(desc->out_dtype, out, lse) || !aligned_to(seqlens, 4) ||
        !aligned_to(block_table, 4))
        return FD_ERR_INVALID_ARG;
    const int32_t S = splits_for(desc);
    if (S < 1) return static_cast<fd_status>(S < 0 ? S : FD_ERR_INVALID_ARG);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = split_impl(desc, S, q, k_cache, v_cache, seqlens, block_table, workspace, workspace_bytes, s,
                    S == 1, out, lse, scales);
    if (st != FD_OK || S == 1) return st;
    return combine_impl(desc, S, workspace, workspace_bytes, out, lse, s);
}

fd_status fd_decode_static(const fd_desc* desc, const void* q, const void* k_cache,
                           const void* v_cache, const int32_t* seqlens, const int32_t* block_table,
                           void* out, float* lse, void* stream) {
    fd_status st = check_desc(desc);
    if (st != FD_OK) return st;
    if (out == nullptr) return FD_ERR_INVALID_ARG;
    const int32_t S = splits_for(desc);
    if (S < 1) return static_cast<fd_status>(S < 0 ? S : FD_ERR_INVALID_ARG);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (S == 1) {
        // one split: the split kernel writes out and lse itself and uses no
        // workspace, so neither the size limit nor the array applies
        return split_impl(desc, 1, q, k_cache, v_cache, seqlens, block_table, nullptr, 0, s, true,
                          out, lse);
    }
    const size_t need = ws_layout(rows_of(desc), S).total;
    if (need > FD_STATIC_WORKSPACE_BYTES) return FD_ERR_WORKSPACE;
    void* ws = nullptr;
    st = static_workspace(&ws);
    if (st != FD_OK) return st;
    st = split_impl(desc, S, q, k_cache, v_cache, seqlens, block_table, ws,
                    FD_STATIC_WORKSPACE_BYTES, s, false, out, lse);
    if (st != FD_OK) return st;
    return combine_impl(desc, S, ws, FD_STATIC_WORKSPACE_BYTES, out, lse, s);
}

fd_status fd_cache_store(const fd_store_desc* d, const fd_kv_scales* scales, const void* k, const void* v,
                         const int64_t* slots, void* k_cache, void* v_cache, void* stream) {
    if (d == nullptr || d->n_tokens < 0 || d->n_kv_heads < 1 || d->head_dim < 1) return FD_ERR_INVALID_ARG;
    if (d->src_dtype != FD_F16 && d->src_dtype != FD_BF16)
        return d->src_dtype == FD_F32 || d->src_dtype == FD_E4M3 ? FD_ERR_UNSUPPORTED : FD_ERR_INVALID_ARG;
    if (d->head_dim != kHeadDim) return FD_ERR_UNSUPPORTED;
    if (d->page_size < 0) return FD_ERR_INVALID_ARG;
    if (d->page_size > 0) {
        if ((d->page_size & (d->page_size - 1)) != 0 || d->page_size > (1 << 20)) return FD_ERR_INVALID_ARG;
        if (d->page_size < 8) return FD_ERR_UNSUPPORTED;
    } else if (d->batch < 1) {
        return FD_ERR_INVALID_ARG;
    }
    if (d->kv_extent < 1 || d->kv_extent > INT32_MAX) return FD_ERR_INVALID_ARG;
    if (!stride_ok(d->k_src_stride_t) || !stride_ok(d->k_src_stride_h) || !stride_ok(d->v_src_stride_t) ||
        !stride_ok(d->v_src_stride_h))
        return FD_ERR_INVALID_ARG;
    if (!stride_ok(d->k_stride_b, 1) || !stride_ok(d->k_stride_h, 1) || !stride_ok(d->k_stride_t, 1) ||
        !stride_ok(d->v_stride_b, 1) || !stride_ok(d->v_stride_h, 1) || !stride_ok(d->v_stride_t, 1))
        return FD_ERR_INVALID_ARG;
    if (d->k_stride_t < kHeadDim || d->v_stride_t < kHeadDim) return FD_ERR_INVALID_ARG;
    const fd_status st = check_scales(scales, d->page_size);
    if (st != FD_OK) return st;
    if (d->n_kv_heads > 65535) return FD_ERR_UNSUPPORTED;
    // what is written has a place of its own
    const int64_t lead = d->page_size > 0 ? d->kv_extent : d->batch;
    const int64_t blocks = ((d->page_size > 0 ? d->page_size : d->kv_extent) + scales->block - 1) / scales->block;
    if (shared_rows(d->k_stride_b, lead) || shared_rows(d->v_stride_b, lead) ||
        shared_rows(d->k_stride_h, d->n_kv_heads) || shared_rows(d->v_stride_h, d->n_kv_heads) ||
        shared_rows(scales->k_stride_b, lead) || shared_rows(scales->v_stride_b, lead) ||
        shared_rows(scales->k_stride_h, d->n_kv_heads) || shared_rows(scales->v_stride_h, d->n_kv_heads) ||
        shared_rows(scales->k_stride_n, blocks) || shared_rows(scales->v_stride_n, blocks))
        return FD_ERR_INVALID_ARG;
    if (d->n_tokens == 0) return FD_OK;   // (an empty tensor's address is null)
    if (k == nullptr || v == nullptr || slots == nullptr || k_cache == nullptr || v_cache == nullptr)
        return FD_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
        return FD_ERR_INVALID_ARG;
    fdk::StoreParams p;
    p.side[0] = {k, static_cast<uint8_t*>(k_cache), scales->k, d->k_src_stride_t, d->k_src_stride_h,
                 d->k_stride_b, d->k_stride_h, d->k_stride_t, scales->k_stride_b, scales->k_stride_h, scales->k_stride_n};
    p.side[1] = {v, static_cast<uint8_t*>(v_cache), scales->v, d->v_src_stride_t, d->v_src_stride_h,
                 d->v_stride_b, d->v_stride_h, d->v_stride_t, scales->v_stride_b, scales->v_stride_h, scales->v_stride_n};
    p.slots = slots;
    const bool paged = d->page_size > 0;
    p.row_tokens = paged ? d->page_size : static_cast<int32_t>(d->kv_extent);
    p.n_slots = (paged ? d->kv_extent : static_cast<int64_t>(d->batch)) * p.row_tokens;
    p.row_shift = paged ? log2_of(d->page_size) : -1;
    p.block = scales->block;
    p.block_shift = log2_of(scales->block);
    p.n_tokens = d->n_tokens;
    p.n_kv_heads = d->n_kv_heads;
    return fdk::launch_store(p, d->src_dtype == FD_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FD_OK
                                                                                                      : FD_ERR_CUDA;
}

fd_status fd_page_tables(const fd_page_desc* d, const int32_t* seqlens, const int32_t* new_tokens,
                         const int32_t* free_pages, const int32_t* free_count, int32_t* block_table,
                         int32_t* seqlens_out, int32_t* free_count_out, int32_t* cu_tokens, int64_t* slots,
                         int32_t* positions, void* stream) {
    if (d == nullptr || d->batch < 0 || d->page_size < 1 || (d->page_size & (d->page_size - 1)) != 0 ||
        d->page_size > (1 << 20) || d->max_pages_per_seq < 1 || d->n_pages < 1 || d->n_free_max < 0 || d->n_slots < 0)
        return FD_ERR_INVALID_ARG;
    if (d->page_size < 8 || d->batch > FD_MAX_TABLE_BATCH) return FD_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(d->max_pages_per_seq) * d->page_size > INT32_MAX) return FD_ERR_INVALID_ARG;
    if (free_count == nullptr || free_count_out == nullptr || (d->n_free_max > 0 && free_pages == nullptr) ||
        (d->n_slots > 0 && slots == nullptr))
        return FD_ERR_INVALID_ARG;
    if (d->batch > 0 && (seqlens == nullptr || new_tokens == nullptr || block_table == nullptr || seqlens_out == nullptr))
        return FD_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(slots) & 7u) != 0) return FD_ERR_INVALID_ARG;
    for (const void* x : {static_cast<const void*>(seqlens), static_cast<const void*>(new_tokens),
                          static_cast<const void*>(free_pages), static_cast<const void*>(free_count),
                          static_cast<const void*>(block_table), static_cast<const void*>(seqlens_out),
                          static_cast<const void*>(free_count_out), static_cast<const void*>(cu_tokens),
                          static_cast<const void*>(positions)})
        if ((reinterpret_cast<uintptr_t>(x) & 3u) != 0) return FD_ERR_INVALID_ARG;
    fdk::PageParams p;
    p.seqlens = seqlens;
    p.new_tokens = new_tokens;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.block_table = block_table;
    p.seqlens_out = seqlens_out;
    p.free_count_out = free_count_out;
    p.cu_tokens = cu_tokens;
    p.slots = slots;
    p.positions = positions;
    p.batch = d->batch;
    p.page_size = d->page_size;
    p.page_shift = log2_of(d->page_size);
    p.max_pages = d->max_pages_per_seq;
    p.n_pages = d->n_pages;
    p.n_free_max = d->n_free_max;
    p.n_slots = d->n_slots;
    return fdk::launch_page_tables(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

fd_status fd_qkv_rope(const fd_rope_desc* d, const void* q, const void* k, const void* v, const void* q_weight,
                      const void* k_weight, const float* inv_freq, const int32_t* positions, const int64_t* slots,
                      void* q_out, void* k_out, void* k_cache, void* v_cache, void* stream) {
    if ((k_cache == nullptr) != (v_cache == nullptr)) return FD_ERR_INVALID_ARG;
    const bool cached = k_cache != nullptr;
    const fd_status st = check_rope(d, cached, k_out != nullptr);
    if (st != FD_OK) return st;
    if (d->n_tokens == 0) return FD_OK;   // (an empty tensor's address is null)
    if (positions == nullptr || (d->rot_dim > 0 && inv_freq == nullptr) || (d->n_q_heads > 0 && (q == nullptr || q_out == nullptr)) ||
        (d->n_kv_heads > 0 && (k == nullptr || (k_out == nullptr && !cached))) || (cached && (v == nullptr || slots == nullptr)))
        return FD_ERR_INVALID_ARG;
    for (const void* x : {q, k, v, q_weight, k_weight, const_cast<const void*>(q_out), const_cast<const void*>(k_out),
                          const_cast<const void*>(k_cache), const_cast<const void*>(v_cache)})
        if (!aligned16(x)) return FD_ERR_INVALID_ARG;
    if (!aligned_to(positions, 4) || !aligned_to(inv_freq, 4) || !aligned_to(slots, 8)) return FD_ERR_INVALID_ARG;
    // in place: with the input's strides
    if (q != nullptr && q == q_out && (d->q_stride_t != d->q_out_stride_t || d->q_stride_h != d->q_out_stride_h)) return FD_ERR_INVALID_ARG;
    if (k != nullptr && k == k_out && (d->k_src_stride_t != d->k_out_stride_t || d->k_src_stride_h != d->k_out_stride_h))
        return FD_ERR_INVALID_ARG;
    const bool fp8 = cached && d->cache_dtype == FD_E4M3;
    const bool norm_q = (d->norm & FD_NORM_Q) != 0, norm_k = (d->norm & FD_NORM_K) != 0;
    fdk::RopeParams p = {};
    p.side[0] = {q, q_out, nullptr, norm_q ? q_weight : nullptr, d->q_stride_t, d->q_stride_h, d->q_out_stride_t,
                 d->q_out_stride_h, 0, 0, 0, norm_q && q_weight != nullptr ? d->q_w_stride_h : 0, d->n_q_heads, norm_q, 1.f};
    p.side[1] = {k, k_out, k_cache, norm_k ? k_weight : nullptr, d->k_src_stride_t, d->k_src_stride_h, d->k_out_stride_t,
                 d->k_out_stride_h, d->k_stride_b, d->k_stride_h, d->k_stride_t,
                 norm_k && k_weight != nullptr ? d->k_w_stride_h : 0, d->n_kv_heads, norm_k, fp8 ? 1.f / d->k_scale : 1.f};
    p.side[2] = {v, nullptr, v_cache, nullptr, d->v_src_stride_t, d->v_src_stride_h, 0, 0, d->v_stride_b, d->v_stride_h,
                 d->v_stride_t, 0, d->n_kv_heads, 0, fp8 ? 1.f / d->v_scale : 1.f};
    p.inv_freq = inv_freq;
    p.positions = positions;
    p.slots = slots;
    if (cached) {
        const bool paged = d->page_size > 0;
        p.row_tokens = paged ? d->page_size : static_cast<int32_t>(d->kv_extent);
        p.n_slots = (paged ? d->kv_extent : static_cast<int64_t>(d->batch)) * p.row_tokens;
        p.row_shift = paged ? log2_of(d->page_size) : -1;
    }
    p.n_tokens = d->n_tokens;
    p.rot_dim = d->rot_dim;
    p.w_dtype = d->w_dtype == FD_F16 ? 0 : d->w_dtype == FD_BF16 ? 1 : 2;
    p.eps = d->eps;
    p.rot_scale = d->rot_scale;
    return fdk::launch_rope(p, d->dtype == FD_BF16, d->interleaved != 0, fp8, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FD_OK
               : FD_ERR_CUDA;
}

fd_status fd_page_fork(const fd_page_desc* d, int32_t n_forks, const int32_t* parents, const int32_t* children,
                       const int32_t* keep, const int32_t* seqlens, const int32_t* free_pages, const int32_t* free_count,
                       int32_t* block_table, int32_t* shares, int32_t* seqlens_out, int32_t* free_count_out,
                       int32_t* copy_src, int32_t* copy_dst, int32_t* copy_count, void* stream) {
    const fd_status st = check_pages(d);
    if (st != FD_OK) return st;
    if (n_forks < 0 || d->n_slots < n_forks) return FD_ERR_INVALID_ARG;
    if (n_forks > FD_MAX_TABLE_BATCH) return FD_ERR_UNSUPPORTED;
    if (!ints_ok({free_count, free_count_out, shares, copy_count},
                 {parents, children, keep, seqlens, free_pages, block_table, seqlens_out, copy_src, copy_dst}))
        return FD_ERR_INVALID_ARG;
    if ((n_forks > 0 && (parents == nullptr || children == nullptr || copy_src == nullptr || copy_dst == nullptr)) ||
        (d->batch > 0 && (seqlens == nullptr || block_table == nullptr || seqlens_out == nullptr)) ||
        (d->n_free_max > 0 && free_pages == nullptr))
        return FD_ERR_INVALID_ARG;
    fdk::PagePlanParams p = page_plan(d);
    p.n_forks = n_forks;
    p.parents = parents;
    p.children = children;
    p.keep = keep;
    p.seqlens = seqlens;
    p.free_in = free_pages;
    p.free_count = free_count;
    p.block_table = block_table;
    p.shares = shares;
    p.seqlens_out = seqlens_out;
    p.free_count_out = free_count_out;
    p.copy_src = copy_src;
    p.copy_dst = copy_dst;
    p.copy_count = copy_count;
    return fdk::launch_page_fork(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

fd_status fd_page_trim(const fd_page_desc* d, const int32_t* keep, const int32_t* seqlens, int32_t* free_pages,
                       const int32_t* free_count, int32_t* block_table, int32_t* shares, int32_t* seqlens_out,
                       int32_t* free_count_out, int32_t* copy_src, int32_t* copy_dst, int32_t* copy_count, void* stream) {
    const fd_status st = check_pages(d);
    if (st != FD_OK) return st;
    if (static_cast<int64_t>(d->batch) * (static_cast<int64_t>(d->max_pages_per_seq) + 1) >= (int64_t(1) << 30)) return FD_ERR_UNSUPPORTED;
    if (shares != nullptr && d->n_slots < d->batch) return FD_ERR_INVALID_ARG;
    if (!ints_ok({free_count, free_count_out}, {keep, seqlens, free_pages, block_table, shares, seqlens_out, copy_src, copy_dst, copy_count}))
        return FD_ERR_INVALID_ARG;
    if ((d->batch > 0 && (keep == nullptr || seqlens == nullptr || block_table == nullptr || seqlens_out == nullptr)) ||
        (d->n_free_max > 0 && free_pages == nullptr) ||
        (shares != nullptr && (copy_count == nullptr || (d->batch > 0 && (copy_src == nullptr || copy_dst == nullptr)))))
        return FD_ERR_INVALID_ARG;
    fdk::PagePlanParams p = page_plan(d);
    p.keep = keep;
    p.seqlens = seqlens;
    p.free_in = free_pages;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.block_table = block_table;
    p.shares = shares;
    p.seqlens_out = seqlens_out;
    p.free_count_out = free_count_out;
    p.copy_src = copy_src;
    p.copy_dst = copy_dst;
    p.copy_count = copy_count;
    return fdk::launch_page_trim(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

fd_status fd_page_compact(const fd_page_desc* d, int32_t n_keep, const int32_t* seqlens, int32_t* free_pages,
                          const int32_t* free_count, int32_t* block_table, int32_t* shares, int32_t* free_count_out,
                          int32_t* copy_src, int32_t* copy_dst, int32_t* copy_count, void* stream) {
    const fd_status st = check_pages(d);
    if (st != FD_OK) return st;
    if (n_keep < 0 || n_keep > d->n_pages) return FD_ERR_INVALID_ARG;
    if (d->n_pages - n_keep > FD_MAX_COMPACT_PAGES) return FD_ERR_UNSUPPORTED;
    if (!ints_ok({free_count, free_count_out, copy_count}, {seqlens, free_pages, block_table, shares, copy_src, copy_dst}))
        return FD_ERR_INVALID_ARG;
    if ((d->batch > 0 && (seqlens == nullptr || block_table == nullptr)) || (d->n_free_max > 0 && free_pages == nullptr) ||
        (d->n_slots > 0 && (copy_src == nullptr || copy_dst == nullptr)))
        return FD_ERR_INVALID_ARG;
    fdk::PagePlanParams p = page_plan(d);
    p.n_keep = n_keep;
    p.seqlens = seqlens;
    p.free_in = free_pages;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.block_table = block_table;
    p.shares = shares;
    p.free_count_out = free_count_out;
    p.copy_src = copy_src;
    p.copy_dst = copy_dst;
    p.copy_count = copy_count;
    return fdk::launch_page_compact(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

fd_status fd_page_copy(const fd_pool* pools, int32_t n_pools, int32_t n_pages, int32_t n_pairs, const int32_t* copy_src,
                       const int32_t* copy_dst, const int32_t* copy_count, void* stream) {
    if (n_pools < 0 || n_pages < 1 || n_pairs < 0 || (n_pools > 0 && pools == nullptr)) return FD_ERR_INVALID_ARG;
    for (int i = 0; i < n_pools; ++i) {
        const fd_status st = check_pool(pools[i], n_pages);
        if (st != FD_OK) return st;
    }
    if (!ints_ok({}, {copy_src, copy_dst, copy_count})) return FD_ERR_INVALID_ARG;
    if (n_pools == 0 || n_pairs == 0) return FD_OK;   // (an empty tensor's address is null)
    if (copy_src == nullptr || copy_dst == nullptr) return FD_ERR_INVALID_ARG;
    // One launch for (up to kPoolsPerLaunch) pools of one shape, wherever they are among kPoolsAtOnce:
    // a launch waits for the one before it, and no two pools share memory.
    constexpr int kPoolsAtOnce = 1024;
    for (int base = 0; base < n_pools; base += kPoolsAtOnce) {
        const int end = std::min(n_pools - base, kPoolsAtOnce);
        const fd_pool* at = pools + base;
        bool taken[kPoolsAtOnce] = {};
        for (int first = 0; first < end; ++first) {
            if (taken[first]) continue;
            const PoolShape s = pool_shape(at[first]);
            fdk::CopyParams p = {};
            p.page_stride = s.page_stride;
            p.stride0 = s.stride0;
            p.stride1 = s.stride1;
            p.extent0 = static_cast<int32_t>(s.extent0);
            p.extent1 = static_cast<int32_t>(s.extent1);
            p.row_bytes = s.row_bytes;
            p.unit = 16;
            for (int i = first; i < end && p.n_pools < fdk::kPoolsPerLaunch; ++i) {
                if (taken[i] || !same_shape(at[i], at[first])) continue;
                taken[i] = true;
                p.base[p.n_pools++] = static_cast<char*>(at[i].base);
                p.unit = std::min(p.unit, pool_unit(s, at[i].base));
            }
            p.n_pages = n_pages;
            p.n_pairs = n_pairs;
            p.src = copy_src;
            p.dst = copy_dst;
            p.count = copy_count;
            if (fdk::launch_page_copy(p, static_cast<cudaStream_t>(stream)) != cudaSuccess) return FD_ERR_CUDA;
        }
    }
    return FD_OK;
}

size_t fd_prompt_workspace_size(const fd_prompt_desc* desc) {
    if (check_prompt(desc) != FD_OK) return 0;
    const int32_t S = prompt_splits(desc);
    if (S <= 1) return 0;
    return ws_layout(static_cast<int64_t>(desc->total_q) * desc->n_q_heads, S).total;
}

fd_status fd_prompt(const fd_prompt_desc* d, const void* q, const void* k, const void* v, const int32_t* cu_q,
                    const int32_t* cu_k, void* out, float* lse, void* workspace, size_t workspace_bytes,
                    void* stream) {
    fd_status st = check_prompt(d);
    if (st != FD_OK) return st;
    if (d->batch == 0 || d->total_q == 0) return FD_OK;
    if (q == nullptr || out == nullptr || cu_q == nullptr || cu_k == nullptr ||
        (d->total_k > 0 && (k == nullptr || v == nullptr)))
        return FD_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v)) return FD_ERR_INVALID_ARG;
    if (!aligned_to(cu_q, 4) || !aligned_to(cu_k, 4) || !outputs_aligned(d->out_dtype, out, lse)) return FD_ERR_INVALID_ARG;
    const int32_t S = prompt_splits(d);
    if (S < 1) return static_cast<fd_status>(S < 0 ? S : FD_ERR_INVALID_ARG);
    const WsLayout w = ws_layout(static_cast<int64_t>(d->total_q) * d->n_q_heads, S);
    if (S > 1 && (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0 ||
                  workspace_bytes < w.total))
        return FD_ERR_WORKSPACE;
    fdk::PromptParams p;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_st = d->q_stride_t;
    p.q_sh = d->q_stride_h;
    p.k_st = d->k_stride_t;
    p.k_sh = d->k_stride_h;
    p.v_st = d->v_stride_t;
    p.v_sh = d->v_stride_h;
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    p.out = out;
    p.lse = lse;
    char* ws = static_cast<char*>(workspace);
    p.ws_u = S > 1 ? reinterpret_cast<float*>(ws + w.off_u) : nullptr;
    p.ws_m = S > 1 ? reinterpret_cast<float*>(ws + w.off_m) : nullptr;
    p.ws_l = S > 1 ? reinterpret_cast<float*>(ws + w.off_l) : nullptr;
    p.batch = d->batch;
    p.n_q_heads = d->n_q_heads;
    p.group = d->n_q_heads / d->n_kv_heads;
    p.total_q = d->total_q;
    p.total_k = d->total_k;
    p.causal = d->causal;
    p.n_splits = S;
    p.pair_heads = pair_heads_of(d) ? 1 : 0;
    p.head_units = p.pair_heads ? d->n_q_heads / 2 : d->n_q_heads;
    p.out_dtype = d->out_dtype == FD_F16 ? 0 : d->out_dtype == FD_BF16 ? 1 : 2;
    p.out_vec = aligned16(out) ? 1 : 0;
    p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(kHeadDim)));
    const int64_t tiles = prompt_tiles(d);
    if (tiles * p.head_units * S > INT32_MAX) return FD_ERR_UNSUPPORTED;
    const bool bf16 = d->dtype == FD_BF16;
    CUtensorMap tmQ, tmK, tmV;
    st = make_rows_map(&tmQ, bf16, q, d->total_q, d->n_q_heads, d->q_stride_t, d->q_stride_h);
    if (st != FD_OK) return st;
    if (d->total_k > 0) {
        st = make_rows_map(&tmK, bf16, k, d->total_k, d->n_kv_heads, d->k_stride_t, d->k_stride_h);
        if (st != FD_OK) return st;
        st = make_rows_map(&tmV, bf16, v, d->total_k, d->n_kv_heads, d->v_stride_t, d->v_stride_h);
        if (st != FD_OK) return st;
    } else {
        tmK = tmV = tmQ;             // no key is ever read
    }
    return fdk::launch_prompt(tmQ, tmK, tmV, p, bf16, tiles, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FD_OK
               : FD_ERR_CUDA;
}

int32_t fd_plan_desc(const fd_desc* desc, const int32_t* seqlens_host, int32_t num_sms) {
    fd_status st = check_desc(desc);
    if (st != FD_OK) return st;
    if (desc->batch < 1 || seqlens_host == nullptr) return FD_ERR_INVALID_ARG;
    int64_t max_len = 0;
    for (int32_t b = 0; b < desc->batch; ++b) {
        if (seqlens_host[b] < 0) return FD_ERR_INVALID_ARG;
        if (seqlens_host[b] > max_len) max_len = seqlens_host[b];
    }
    return fdk::plan_launch(desc->batch, desc->n_kv_heads, cols_of(desc), is_fp8(desc),
                            (desc->flags & FD_FLAG_CUDA_CORES) != 0, max_len, num_sms);
}

fd_status fd_decode_status(void* stream) { return fd_device_status(stream, 1); }

fd_status fd_device_status(void* stream, int32_t clear) {
    unsigned v = 0;
    if (fdk::read_status(&v, static_cast<cudaStream_t>(stream), clear != 0) != cudaSuccess)
        return FD_ERR_CUDA;
    if (v & fdk::kStatusTimeoutBit) return FD_ERR_DEVICE_TIMEOUT;
    if (v != 0) return FD_ERR_DEVICE_BOUNDS;
    return FD_OK;
}

}  // extern "C"
