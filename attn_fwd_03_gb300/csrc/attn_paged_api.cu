// attn_paged_api.cu — entry points of the paged cache (include/attn.h): argument
// checks and launches. What the host can see is checked here, before anything is
// launched; lengths, pages and slots live on the device and are checked by the
// kernels that read them.
#include <cmath>
#include <cstdint>

#include "internal.h"

using namespace attn;

namespace {

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Device array of 32-bit integers.
attn_status_t check_ints(const char* name, const void* p) {
    if (!p) return report_error(ATTN_ERR_INVALID, "%s is NULL", name);
    if (misaligned(p, 4)) return report_error(ATTN_ERR_ALIGN, "%s is not 4-byte aligned", name);
    return ATTN_OK;
}

// 16-bit tensor with `n` strides over the extents `dims`; the last dimension is contiguous.
attn_status_t check_strided(const char* name, const void* p, const int64_t* st, const int64_t* dims, int n) {
    if (!p) return report_error(ATTN_ERR_INVALID, "%s is NULL", name);
    if (misaligned(p, 16)) return report_error(ATTN_ERR_ALIGN, "%s is not 16-byte aligned", name);
    for (int i = 0; i < n; ++i) {
        if (dims[i] <= 1) continue;
        if (st[i] <= 0)
            return report_error(ATTN_ERR_INVALID, "%s stride[%d] = %lld is not positive", name, i, (long long)st[i]);
        if (st[i] % 8 != 0)
            return report_error(ATTN_ERR_ALIGN, "%s stride[%d] = %lld elements is not a multiple of 16 bytes", name, i,
                                (long long)st[i]);
        if (st[i] >= (1ll << 38)) return report_error(ATTN_ERR_UNSUPPORTED, "%s stride[%d] too large", name, i);
    }
    return ATTN_OK;
}

attn_status_t check_page_size(int32_t page_size) {
    if (page_size < 1) return report_error(ATTN_ERR_INVALID, "page_size must be positive, got %d", page_size);
    if (page_size < 16 || (page_size & (page_size - 1)) != 0)
        return report_error(ATTN_ERR_UNSUPPORTED, "page_size %d not built (a power of two, 16 or more)", page_size);
    return ATTN_OK;
}

attn_status_t check_16bit(int32_t dtype, int32_t d) {
    if (dtype == ATTN_F32 || dtype == ATTN_E4M3)
        return report_error(ATTN_ERR_UNSUPPORTED, "the paged cache is built for bf16 and fp16 only");
    if (dtype != ATTN_BF16 && dtype != ATTN_F16) return report_error(ATTN_ERR_INVALID, "unknown dtype %d", dtype);
    if (d != 64 && d != 128) return report_error(ATTN_ERR_UNSUPPORTED, "head dim %d not built (64 or 128)", d);
    return ATTN_OK;
}

// Keys of a sequence: the kernels add up to a few tiles to such a number in 32 bits.
constexpr int64_t kMaxLength = (int64_t)INT32_MAX - 1023;

// The kernels step through the sequences, and through a sequence's rows, in 32 bits, some hundred at a time.
attn_status_t check_count(const char* name, int32_t n) {
    if (n > INT32_MAX - 1023) return report_error(ATTN_ERR_UNSUPPORTED, "%s must not exceed 2^31 - 1024, got %d", name, n);
    return ATTN_OK;
}

attn_status_t check_table(int32_t max_pages, int32_t page_size) {
    if (max_pages < 1) return report_error(ATTN_ERR_INVALID, "max_pages must be at least 1, got %d", max_pages);
    if ((int64_t)max_pages * page_size > kMaxLength)
        return report_error(ATTN_ERR_UNSUPPORTED, "max_pages * page_size must not exceed 2^31 - 1024");
    return ATTN_OK;
}

attn_status_t check_cache(int32_t num_pages, int32_t page_size, int32_t heads, const void* k, const void* v,
                          const int64_t* ks, const int64_t* vs) {
    if (num_pages < 1) return report_error(ATTN_ERR_INVALID, "num_pages must be at least 1, got %d", num_pages);
    if ((int64_t)num_pages * page_size > INT32_MAX)
        return report_error(ATTN_ERR_UNSUPPORTED, "num_pages * page_size must stay below 2^31");
    const int64_t dims[3] = {num_pages, heads, page_size};
    const attn_status_t st = check_strided("k_cache", k, ks, dims, 3);
    return st != ATTN_OK ? st : check_strided("v_cache", v, vs, dims, 3);
}

// All of a paged attention call but the workspace. *empty = nothing to compute.
attn_status_t check_paged(const attn_paged_params* p, bool* empty) {
    if (!p) return report_error(ATTN_ERR_INVALID, "params is NULL");
    if (p->num_seqs < 0 || p->total_q < 0 || p->num_q_heads < 1 || p->num_kv_heads < 1)
        return report_error(ATTN_ERR_INVALID, "bad size num_seqs=%d total_q=%d num_q_heads=%d num_kv_heads=%d", p->num_seqs,
                            p->total_q, p->num_q_heads, p->num_kv_heads);
    if (p->reserved0[0] != 0 || p->reserved0[1] != 0) return report_error(ATTN_ERR_INVALID, "reserved0 must be 0");
    if (p->causal != 0 && p->causal != 1)
        return report_error(ATTN_ERR_INVALID, "causal must be 0 or 1, got %d", p->causal);
    if (!std::isfinite(p->scale) || !(p->scale > 0.f))
        return report_error(ATTN_ERR_INVALID, "scale must be positive and finite");
    if (p->max_q < 1) return report_error(ATTN_ERR_INVALID, "max_q must be at least 1, got %d", p->max_q);
    attn_status_t st;
    if ((st = check_count("num_seqs", p->num_seqs)) != ATTN_OK) return st;
    if ((st = check_count("total_q", p->total_q)) != ATTN_OK) return st;
    if ((st = check_16bit(p->dtype, p->d)) != ATTN_OK) return st;
    if ((st = check_page_size(p->page_size)) != ATTN_OK) return st;
    if (p->num_q_heads % p->num_kv_heads != 0)
        return report_error(ATTN_ERR_INVALID, "num_q_heads %d is not a multiple of num_kv_heads %d", p->num_q_heads,
                            p->num_kv_heads);
    if (p->num_q_heads / p->num_kv_heads > 128)
        return report_error(ATTN_ERR_UNSUPPORTED, "more than 128 query heads to a key/value head");
    if (p->num_q_heads > 65535) return report_error(ATTN_ERR_UNSUPPORTED, "num_q_heads is limited to 65535");
    *empty = p->num_seqs == 0 || p->total_q == 0;
    if (*empty) return ATTN_OK;
    if ((st = check_table(p->max_pages, p->page_size)) != ATTN_OK) return st;
    if (p->table_stride < 0) return report_error(ATTN_ERR_INVALID, "table_stride must not be negative");
    const int64_t rows[2] = {p->total_q, p->num_q_heads};
    if ((st = check_strided("q", p->q, p->q_stride, rows, 2)) != ATTN_OK) return st;
    if ((st = check_strided("o", p->o, p->o_stride, rows, 2)) != ATTN_OK) return st;
    if ((st = check_cache(p->num_pages, p->page_size, p->num_kv_heads, p->k_cache, p->v_cache, p->k_stride,
                          p->v_stride)) != ATTN_OK)
        return st;
    if ((st = check_ints("lse", p->lse)) != ATTN_OK) return st;
    if ((st = check_ints("cu_q", p->cu_q)) != ATTN_OK) return st;
    if ((st = check_ints("kv_len", p->kv_len)) != ATTN_OK) return st;
    return check_ints("block_table", p->block_table);
}

// 32-bit integers that a table call reads or writes: `rows` of `n` side by side, `stride` apart.
struct Ints {
    const char* name;
    const void* p;
    int64_t n, rows = 1, stride = 0;
};

// Whether a row of `a` and the array `b` share an element.
bool overlap(const Ints& a, const Ints& b) {
    if (a.n <= 0 || a.rows <= 0 || b.n <= 0) return false;
    // b in elements from a's first; row r of a is [r * stride, r * stride + n)
    const int64_t lo = ((int64_t)reinterpret_cast<uintptr_t>(b.p) - (int64_t)reinterpret_cast<uintptr_t>(a.p)) / 4, hi = lo + b.n;
    if (hi <= 0) return false;
    if (a.rows == 1) return lo < a.n;
    const int64_t first = lo < a.n ? 0 : (lo - a.n) / a.stride + 1;  // the first row that ends behind lo
    return first < a.rows && first * a.stride < hi;
}

// The blocks of the table kernels read and write in no order: an array that is written (the first
// `written` of them) shares no element with any other. Only one of them may have several rows.
template <int N>
attn_status_t check_apart(const Ints (&a)[N], int written) {
    for (int i = 0; i < written; ++i)
        for (int j = i + 1; j < N; ++j)
            if (a[j].rows > 1 ? overlap(a[j], a[i]) : overlap(a[i], a[j]))
                return report_error(ATTN_ERR_INVALID, "%s and %s overlap", a[i].name, a[j].name);
    return ATTN_OK;
}

attn_status_t launched(cudaError_t e, const char* what) {
    return e == cudaSuccess ? ATTN_OK : report_error(ATTN_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

}  // namespace

extern "C" {

size_t attn_paged_workspace_size(const attn_paged_params* p) {
    bool empty = false;
    if (check_paged(p, &empty) != ATTN_OK || empty) return 0;
    LaunchCommon lc;
    if (launch_setup(&lc) != ATTN_OK) return 0;
    return paged_workspace_bytes(*p, lc.num_sms);
}

attn_status_t attn_paged(const attn_paged_params* p, void* stream) {
    bool empty = false;
    attn_status_t st = check_paged(p, &empty);
    if (st != ATTN_OK || empty) return st;
    LaunchCommon lc;
    if ((st = launch_setup(&lc)) != ATTN_OK) return st;
    const size_t need = paged_workspace_bytes(*p, lc.num_sms);
    if (!p->workspace || p->workspace_bytes < need)
        return report_error(ATTN_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", p->workspace_bytes, need);
    if (misaligned(p->workspace, 256)) return report_error(ATTN_ERR_ALIGN, "workspace is not 256-byte aligned");
    return launch_paged(*p, lc, static_cast<cudaStream_t>(stream));
}

attn_status_t attn_pages_write(const attn_pages_write_params* p, void* stream) {
    if (!p) return report_error(ATTN_ERR_INVALID, "params is NULL");
    if (p->rows < 0 || p->num_kv_heads < 1)
        return report_error(ATTN_ERR_INVALID, "bad size rows=%d num_kv_heads=%d", p->rows, p->num_kv_heads);
    if (p->reserved0[0] != 0 || p->reserved0[1] != 0) return report_error(ATTN_ERR_INVALID, "reserved0 must be 0");
    attn_status_t st;
    if ((st = check_16bit(p->dtype, p->d)) != ATTN_OK) return st;
    if ((st = check_page_size(p->page_size)) != ATTN_OK) return st;
    if (p->num_kv_heads > 65535) return report_error(ATTN_ERR_UNSUPPORTED, "num_kv_heads is limited to 65535");
    if (p->rows == 0) return ATTN_OK;
    const int64_t dims[2] = {p->rows, p->num_kv_heads};
    if ((st = check_strided("k", p->k, p->k_row_stride, dims, 2)) != ATTN_OK) return st;
    if ((st = check_strided("v", p->v, p->v_row_stride, dims, 2)) != ATTN_OK) return st;
    if ((st = check_ints("slots", p->slots)) != ATTN_OK) return st;
    if ((st = check_cache(p->num_pages, p->page_size, p->num_kv_heads, p->k_cache, p->v_cache, p->k_stride,
                          p->v_stride)) != ATTN_OK)
        return st;
    LaunchCommon lc;
    if ((st = launch_setup(&lc)) != ATTN_OK) return st;
    return launched(launch_pages_write(*p, lc, static_cast<cudaStream_t>(stream)), "attn_pages_write");
}

attn_status_t attn_pages_plan(const attn_pages_plan_params* p, void* stream) {
    if (!p) return report_error(ATTN_ERR_INVALID, "params is NULL");
    if (p->num_seqs < 0 || p->total_q < 0 || p->free_capacity < 0)
        return report_error(ATTN_ERR_INVALID, "negative size num_seqs=%d total_q=%d free_capacity=%d", p->num_seqs,
                            p->total_q, p->free_capacity);
    if (p->reserved0 != 0) return report_error(ATTN_ERR_INVALID, "reserved0 must be 0");
    attn_status_t st;
    if ((st = check_count("num_seqs", p->num_seqs)) != ATTN_OK) return st;
    if ((st = check_page_size(p->page_size)) != ATTN_OK) return st;
    if ((st = check_table(p->max_pages, p->page_size)) != ATTN_OK) return st;
    if (p->table_stride < p->max_pages)
        return report_error(ATTN_ERR_INVALID, "table_stride must be at least max_pages");
    if ((st = check_ints("free_count", p->free_count)) != ATTN_OK) return st;
    if ((st = check_ints("free_left", p->free_left)) != ATTN_OK) return st;
    if ((st = check_ints("cu_q", p->cu_q)) != ATTN_OK) return st;
    if (p->num_seqs > 0) {
        if ((st = check_ints("q_len", p->q_len)) != ATTN_OK) return st;
        if ((st = check_ints("kv_len", p->kv_len)) != ATTN_OK) return st;
        if ((st = check_ints("new_len", p->new_len)) != ATTN_OK) return st;
        if ((st = check_ints("block_table", p->block_table)) != ATTN_OK) return st;
    }
    if (p->total_q > 0) {
        if ((st = check_ints("slots", p->slots)) != ATTN_OK) return st;
        if ((st = check_ints("positions", p->positions)) != ATTN_OK) return st;
    }
    if (p->free_capacity > 0 && (st = check_ints("free_pages", p->free_pages)) != ATTN_OK) return st;
    const int64_t seqs = p->num_seqs;
    const Ints arrays[] = {{"block_table", p->block_table, p->max_pages, seqs, p->table_stride}, {"cu_q", p->cu_q, seqs + 1},
                           {"new_len", p->new_len, seqs}, {"slots", p->slots, p->total_q}, {"positions", p->positions, p->total_q},
                           {"free_left", p->free_left, 1}, {"q_len", p->q_len, seqs}, {"kv_len", p->kv_len, seqs},
                           {"free_pages", p->free_pages, p->free_capacity}, {"free_count", p->free_count, 1}};
    if ((st = check_apart(arrays, 6)) != ATTN_OK) return st;
    LaunchCommon lc;
    if ((st = launch_setup(&lc)) != ATTN_OK) return st;
    return launched(launch_pages_plan(*p, lc, static_cast<cudaStream_t>(stream)), "attn_pages_plan");
}

attn_status_t attn_pages_release(const attn_pages_release_params* p, void* stream) {
    if (!p) return report_error(ATTN_ERR_INVALID, "params is NULL");
    if (p->num_seqs < 0 || p->free_capacity < 0)
        return report_error(ATTN_ERR_INVALID, "negative size num_seqs=%d free_capacity=%d", p->num_seqs,
                            p->free_capacity);
    attn_status_t st;
    if ((st = check_count("num_seqs", p->num_seqs)) != ATTN_OK) return st;
    if ((st = check_page_size(p->page_size)) != ATTN_OK) return st;
    if ((st = check_table(p->max_pages, p->page_size)) != ATTN_OK) return st;
    if (p->table_stride < p->max_pages)
        return report_error(ATTN_ERR_INVALID, "table_stride must be at least max_pages");
    if ((st = check_ints("free_count", p->free_count)) != ATTN_OK) return st;
    if ((st = check_ints("free_left", p->free_left)) != ATTN_OK) return st;
    if (p->num_seqs > 0) {
        if ((st = check_ints("done", p->done)) != ATTN_OK) return st;
        if ((st = check_ints("kv_len", p->kv_len)) != ATTN_OK) return st;
        if ((st = check_ints("new_len", p->new_len)) != ATTN_OK) return st;
        if ((st = check_ints("block_table", p->block_table)) != ATTN_OK) return st;
    }
    if (p->free_capacity > 0 && (st = check_ints("free_pages", p->free_pages)) != ATTN_OK) return st;
    const int64_t seqs = p->num_seqs;
    const Ints arrays[] = {{"free_pages", p->free_pages, p->free_capacity}, {"new_len", p->new_len, seqs},
                           {"free_left", p->free_left, 1}, {"done", p->done, seqs}, {"kv_len", p->kv_len, seqs},
                           {"block_table", p->block_table, p->max_pages, seqs, p->table_stride},
                           {"free_count", p->free_count, 1}};
    if ((st = check_apart(arrays, 3)) != ATTN_OK) return st;
    LaunchCommon lc;
    if ((st = launch_setup(&lc)) != ATTN_OK) return st;
    return launched(launch_pages_release(*p, lc, static_cast<cudaStream_t>(stream)), "attn_pages_release");
}

}  // extern "C"
