// C-ABI entry points of the softmax-attention layer (declared in include/gdn.h): every
// argument is checked here, on the host, before anything is enqueued.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <initializer_list>

#include "gdn.h"
#include "gdn_attn.h"
#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace {

bool misaligned(const void* p, unsigned bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }
gdn_status from_cuda(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

// A scale of 0 selects 1; negative, infinite or NaN ones are refused.
bool scale_of(float s, float* out) {
    *out = s == 0.0f ? 1.0f : s;
    return isfinite(s) && s >= 0.0f;
}

gdn_status check_attn_config(const gdn_attn_config* c, gdn::AttnShape* sh) {
    if (!c) return GDN_ERR_INVALID_ARGUMENT;
    if (c->num_q_heads <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0 || c->page_size <= 0)
        return GDN_ERR_INVALID_ARGUMENT;
    if (c->num_q_heads % c->num_kv_heads != 0) return GDN_ERR_INVALID_ARGUMENT;
    if (c->rotary_dim < 0 || c->rotary_dim % 2 != 0 || c->rotary_dim > c->head_dim) return GDN_ERR_INVALID_ARGUMENT;
    if (c->rope_interleaved != 0 && c->rope_interleaved != 1) return GDN_ERR_INVALID_ARGUMENT;
    if (c->kv_dtype != GDN_KV_BF16 && c->kv_dtype != GDN_KV_E4M3) return GDN_ERR_INVALID_ARGUMENT;
    if (c->window < 0) return GDN_ERR_INVALID_ARGUMENT;
    if (!(c->norm_eps >= 0.0f) || !isfinite(c->norm_eps) || !isfinite(c->norm_offset) || !isfinite(c->sm_scale))
        return GDN_ERR_INVALID_ARGUMENT;
    if (!(c->softcap >= 0.0f) || !isfinite(c->softcap)) return GDN_ERR_INVALID_ARGUMENT;
    if (!scale_of(c->rope_scale, &sh->rope_scale) || !scale_of(c->k_scale, &sh->k_scale) ||
        !scale_of(c->v_scale, &sh->v_scale))
        return GDN_ERR_INVALID_ARGUMENT;
    if (c->kv_dtype == GDN_KV_BF16 && (sh->k_scale != 1.0f || sh->v_scale != 1.0f)) return GDN_ERR_INVALID_ARGUMENT;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return GDN_ERR_UNSUPPORTED;
    if (c->num_q_heads / c->num_kv_heads > 16 || c->num_q_heads > 1024 || c->page_size > 65536)
        return GDN_ERR_UNSUPPORTED;
    sh->Hq = c->num_q_heads;
    sh->Hkv = c->num_kv_heads;
    sh->d = c->head_dim;
    sh->G = sh->Hq / sh->Hkv;
    sh->R = c->rotary_dim;
    sh->interleaved = c->rope_interleaved != 0;
    sh->fp8 = c->kv_dtype == GDN_KV_E4M3;
    sh->page_size = c->page_size;
    sh->window = c->window;
    sh->norm_eps = c->norm_eps;
    sh->norm_offset = c->norm_offset;
    sh->sm_scale = c->sm_scale != 0.0f ? c->sm_scale : 1.0f / sqrtf((float)c->head_dim);
    sh->softcap = c->softcap;
    return GDN_OK;
}

// Sizes that do not depend on a pointer: B, T (1..16), rows.
gdn_status check_rows(int32_t B, int32_t T, const int32_t* cu, int32_t total) {
    if (B < 0 || T <= 0 || total < 0) return GDN_ERR_INVALID_ARGUMENT;
    if (T > gdn::kMaxTokens || B > gdn::kAttnMaxBatch) return GDN_ERR_UNSUPPORTED;
    if (!cu && total != B * T) return GDN_ERR_INVALID_ARGUMENT;
    if (misaligned(cu, 4)) return GDN_ERR_MISALIGNED;
    return GDN_OK;
}

gdn_status check_cache(const gdn_kv_cache* c, const gdn::AttnShape& sh, gdn::PagedCache* out) {
    if (!c || !c->k_pages || !c->v_pages || !c->page_table || !c->seq_lens) return GDN_ERR_INVALID_ARGUMENT;
    if (c->num_pages <= 0 || c->table_rows <= 0 || c->max_pages <= 0) return GDN_ERR_INVALID_ARGUMENT;
    if (misaligned(c->k_pages, 16) || misaligned(c->v_pages, 16) || misaligned(c->page_table, 4) ||
        misaligned(c->seq_lens, 4))
        return GDN_ERR_MISALIGNED;
    // token numbers (page * page_size + offset) and positions are 32-bit in the kernels, which look up to
    // a tile past a sequence's end
    if ((long)c->num_pages * sh.page_size > 0x7fffffffL || (long)c->max_pages * sh.page_size > 0x7fff0000L)
        return GDN_ERR_UNSUPPORTED;
    *out = gdn::PagedCache{c->k_pages, c->v_pages, c->num_pages, c->page_table, c->table_rows, c->max_pages, c->seq_lens};
    return GDN_OK;
}

gdn_status check_heads(const gdn_heads* h, gdn::Heads* out) {
    if (!h || !h->ptr || h->row_stride < 0 || h->head_stride < 0) return GDN_ERR_INVALID_ARGUMENT;
    if (misaligned(h->ptr, 16) || h->row_stride % 8 != 0 || h->head_stride % 8 != 0) return GDN_ERR_MISALIGNED;
    *out = gdn::Heads{h->ptr, (long)h->row_stride, (long)h->head_stride};
    return GDN_OK;
}

gdn_status check_tables(int32_t page_size, int32_t n, const int32_t* table, int32_t rows, int32_t max_pages,
                        const int32_t* refs, int32_t num_pages, const int32_t* err_flag) {
    if (page_size <= 0 || n < 0 || rows <= 0 || max_pages <= 0 || num_pages <= 0) return GDN_ERR_INVALID_ARGUMENT;
    if (n > gdn::kPagesMaxBatch || page_size > 65536 || (long)max_pages * page_size > 0x7fffffffL)
        return GDN_ERR_UNSUPPORTED;
    if (num_pages > gdn::kPagesMost || max_pages > gdn::kPagesMost) return GDN_ERR_UNSUPPORTED;
    if (n == 0) return GDN_OK;
    if (!table || !refs) return GDN_ERR_INVALID_ARGUMENT;
    if (misaligned(table, 4) || misaligned(refs, 4) || misaligned(err_flag, 4)) return GDN_ERR_MISALIGNED;
    return GDN_OK;
}

gdn_status check_ints(std::initializer_list<const int32_t*> required) {
    for (const int32_t* p : required)
        if (!p) return GDN_ERR_INVALID_ARGUMENT;
    for (const int32_t* p : required)
        if (misaligned(p, 4)) return GDN_ERR_MISALIGNED;
    return GDN_OK;
}

}  // namespace

namespace gdn {
cudaError_t device_sms(int* device, int* sms) {
    static std::atomic<int> cached[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    *device = dev;
    *sms = n;
    return cudaSuccess;
}
}  // namespace gdn

extern "C" {

gdn_status gdn_qk_rope_append(const gdn_attn_config* cfg, const gdn_kv_cache* cache, int32_t B, int32_t T,
                              const int32_t* cu_seqlens, int32_t total_tokens, const gdn_heads* q, const gdn_heads* k,
                              const gdn_heads* v, const uint16_t* q_norm_w, const uint16_t* k_norm_w,
                              const float* inv_freq, const int32_t* slots, uint16_t* q_out, int32_t* err_flag,
                              void* stream) {
    gdn::AppendArgs a{};
    gdn_status st = check_attn_config(cfg, &a.sh);
    if (st != GDN_OK) return st;
    if ((st = check_rows(B, T, cu_seqlens, total_tokens)) != GDN_OK) return st;
    if (B == 0 || total_tokens == 0) return GDN_OK;
    if ((st = check_cache(cache, a.sh, &a.c)) != GDN_OK) return st;
    if ((st = check_heads(q, &a.q)) != GDN_OK || (st = check_heads(k, &a.k)) != GDN_OK ||
        (st = check_heads(v, &a.v)) != GDN_OK)
        return st;
    if (!q_out || !slots || (a.sh.R > 0 && !inv_freq)) return GDN_ERR_INVALID_ARGUMENT;
    if (misaligned(q_out, 16) || misaligned(q_norm_w, 16) || misaligned(k_norm_w, 16) || misaligned(inv_freq, 4) ||
        misaligned(slots, 4) || misaligned(err_flag, 4))
        return GDN_ERR_MISALIGNED;
    a.B = B;
    a.T = T;
    a.total = total_tokens;
    a.cu = cu_seqlens;
    a.qw = q_norm_w;
    a.kw = k_norm_w;
    a.inv_freq = inv_freq;
    a.slots = slots;
    a.q_out = q_out;
    a.err_flag = err_flag;
    return from_cuda(gdn::launch_qk_rope_append(a, (cudaStream_t)stream));
}

gdn_status gdn_attn_decode(const gdn_attn_config* cfg, const gdn_kv_cache* cache, int32_t B, int32_t T,
                           const int32_t* cu_seqlens, int32_t total_tokens, const gdn_heads* q, const gdn_heads* gate,
                           const int32_t* slots, uint16_t* out, float* lse, int32_t* err_flag, void* workspace,
                           void* stream) {
    gdn::AttnArgs a{};
    gdn_status st = check_attn_config(cfg, &a.sh);
    if (st != GDN_OK) return st;
    if ((st = check_rows(B, T, cu_seqlens, total_tokens)) != GDN_OK) return st;
    if (B == 0 || total_tokens == 0) return GDN_OK;
    if ((st = check_cache(cache, a.sh, &a.c)) != GDN_OK) return st;
    if ((st = check_heads(q, &a.q)) != GDN_OK) return st;
    if (gate && (st = check_heads(gate, &a.gate)) != GDN_OK) return st;
    if (!slots || !out || !workspace) return GDN_ERR_INVALID_ARGUMENT;
    // (a broadcast row or head, stride 0, has no tensor map: the kernel for few rows takes it, whose
    // partial results are smaller)
    const int rows = T * a.sh.G;
    const bool broadcast = (a.q.row == 0 && total_tokens > 1) || (a.q.head == 0 && a.sh.Hq > 1);
    const bool many = gdn::attn_rows_supported(a.sh.d, a.sh.fp8, a.sh.page_size, rows) && !broadcast;
    // the kernels number the batch's work (token tiles of a row tile of a head) in 32 bits; the host knows
    // the lengths' bound only
    if (B * (many ? gdn::attn_rows_places(a.sh, a.c, T) : gdn::attn_decode_places(a.sh, a.c, T)) > gdn::kAttnMaxPlaces)
        return GDN_ERR_UNSUPPORTED;
    if (misaligned(out, 16) || misaligned(lse, 4) || misaligned(slots, 4) || misaligned(err_flag, 4) ||
        misaligned(workspace, 16))
        return GDN_ERR_MISALIGNED;
    a.B = B;
    a.T = T;
    a.total = total_tokens;
    a.cu = cu_seqlens;
    a.slots = slots;
    a.out = out;
    a.lse = lse;
    a.err_flag = err_flag;
    a.counters = static_cast<unsigned int*>(workspace);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    a.split = reinterpret_cast<gdn::Piece*>(ws + gdn::kAttnCounters * sizeof(unsigned int));
    a.partial = reinterpret_cast<float*>(ws + gdn::kAttnPartialAt);
    return from_cuda(many ? gdn::launch_attn_rows(a, (cudaStream_t)stream) : gdn::launch_attn_decode(a, (cudaStream_t)stream));
}

size_t gdn_attn_decode_workspace_bytes(const gdn_attn_config* cfg, int32_t B, int32_t T) {
    gdn::AttnShape sh;
    if (check_attn_config(cfg, &sh) != GDN_OK) return 0;
    if (B < 0 || B > gdn::kAttnMaxBatch || T <= 0 || T > gdn::kMaxTokens) return 0;
    return gdn::attn_workspace_bytes(sh.d, sh.fp8, sh.page_size, T * sh.G);
}

gdn_status gdn_rope_inv_freq_host(int32_t rotary_dim, double theta, double factor, int32_t yarn, int32_t original_len,
                                  float* inv_freq, float* rope_scale) {
    const int R = rotary_dim;
    if (R < 0 || R % 2 != 0 || !(theta > 1.0) || !isfinite(theta) || !(factor >= 1.0) || !isfinite(factor))
        return GDN_ERR_INVALID_ARGUMENT;
    if (yarn != 0 && (yarn != 1 || original_len <= 0)) return GDN_ERR_INVALID_ARGUMENT;
    if ((R > 0 && !inv_freq) || !rope_scale) return GDN_ERR_INVALID_ARGUMENT;
    const double two_pi = 2.0 * acos(-1.0);
    // the pair that turns `n` times over original_len tokens
    auto pair_of = [&](double n) { return R * log(original_len / (n * two_pi)) / (2.0 * log(theta)); };
    double lo = 0.0, hi = 0.0;
    if (yarn) {
        lo = fmax(floor(pair_of(32.0)), 0.0);
        hi = fmin(ceil(pair_of(1.0)), R - 1.0);
    }
    for (int i = 0; i < R / 2; ++i) {
        const double f = pow(theta, -2.0 * i / R);
        double slow = 1.0;  // share of the interpolated speed
        if (yarn) slow = fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
        inv_freq[i] = (float)(f / factor * slow + f * (1.0 - slow));
    }
    *rope_scale = yarn ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    return GDN_OK;
}

gdn_status gdn_pages_reserve(int32_t page_size, int32_t n, const int32_t* slots, const int32_t* n_tokens, int32_t T,
                             int32_t* page_table, int32_t table_rows, int32_t max_pages, const int32_t* seq_lens,
                             int32_t* page_refs, int32_t num_pages, int32_t* err_flag, void* stream) {
    gdn_status st = check_tables(page_size, n, page_table, table_rows, max_pages, page_refs, num_pages, err_flag);
    if (st != GDN_OK) return st;
    if (T < 0) return GDN_ERR_INVALID_ARGUMENT;
    if (n == 0) return GDN_OK;
    if ((st = check_ints({slots, seq_lens})) != GDN_OK) return st;
    if (misaligned(n_tokens, 4)) return GDN_ERR_MISALIGNED;
    gdn::PageArgs a{};
    a.page_size = page_size;
    a.n = n;
    a.slots = slots;
    a.n_tokens = n_tokens;
    a.T = T;
    a.table = page_table;
    a.rows = table_rows;
    a.max_pages = max_pages;
    a.seq_lens = const_cast<int32_t*>(seq_lens);
    a.refs = page_refs;
    a.num_pages = num_pages;
    a.err_flag = err_flag;
    return from_cuda(gdn::launch_pages_reserve(a, (cudaStream_t)stream));
}

gdn_status gdn_pages_fork(int32_t page_size, int32_t n, const int32_t* src, const int32_t* dst, int32_t* page_table,
                          int32_t table_rows, int32_t max_pages, int32_t* seq_lens, int32_t* page_refs,
                          int32_t num_pages, int32_t* copy_src, int32_t* copy_dst, int32_t* err_flag, void* stream) {
    gdn_status st = check_tables(page_size, n, page_table, table_rows, max_pages, page_refs, num_pages, err_flag);
    if (st != GDN_OK || n == 0) return st;
    if ((st = check_ints({src, dst, seq_lens, copy_src, copy_dst})) != GDN_OK) return st;
    gdn::PageArgs a{};
    a.page_size = page_size;
    a.n = n;
    a.slots = dst;
    a.src_slots = src;
    a.table = page_table;
    a.rows = table_rows;
    a.max_pages = max_pages;
    a.seq_lens = seq_lens;
    a.refs = page_refs;
    a.num_pages = num_pages;
    a.copy_src = copy_src;
    a.copy_dst = copy_dst;
    a.err_flag = err_flag;
    return from_cuda(gdn::launch_pages_fork(a, (cudaStream_t)stream));
}

gdn_status gdn_pages_free(int32_t n, const int32_t* slots, int32_t* page_table, int32_t table_rows, int32_t max_pages,
                          int32_t* seq_lens, int32_t* page_refs, int32_t num_pages, int32_t* err_flag, void* stream) {
    gdn_status st = check_tables(1, n, page_table, table_rows, max_pages, page_refs, num_pages, err_flag);
    if (st != GDN_OK || n == 0) return st;
    if ((st = check_ints({slots, seq_lens})) != GDN_OK) return st;
    gdn::PageArgs a{};
    a.n = n;
    a.slots = slots;
    a.table = page_table;
    a.rows = table_rows;
    a.max_pages = max_pages;
    a.seq_lens = seq_lens;
    a.refs = page_refs;
    a.num_pages = num_pages;
    a.err_flag = err_flag;
    return from_cuda(gdn::launch_pages_free(a, (cudaStream_t)stream));
}

gdn_status gdn_pages_compact(int32_t* page_table, int32_t table_rows, int32_t max_pages, int32_t* page_refs,
                             int32_t num_pages, int32_t* copy_src, int32_t* copy_dst, int32_t* n_copies,
                             int32_t* remap, int32_t* err_flag, void* stream) {
    gdn_status st = check_tables(1, 1, page_table, table_rows, max_pages, page_refs, num_pages, err_flag);
    if (st != GDN_OK) return st;
    if ((st = check_ints({copy_src, copy_dst, n_copies, remap})) != GDN_OK) return st;
    gdn::PageArgs a{};
    a.n = 1;
    a.table = page_table;
    a.rows = table_rows;
    a.max_pages = max_pages;
    a.refs = page_refs;
    a.num_pages = num_pages;
    a.copy_src = copy_src;
    a.copy_dst = copy_dst;
    a.n_copies = n_copies;
    a.remap = remap;
    a.err_flag = err_flag;
    return from_cuda(gdn::launch_pages_compact(a, (cudaStream_t)stream));
}

gdn_status gdn_copy_rows(const gdn_copy_buffer* buffers, int32_t n_buffers, int32_t rows, int32_t n,
                         const int32_t* src_ids, const int32_t* dst_ids, const int32_t* n_dev, int32_t* err_flag,
                         void* stream) {
    if (n_buffers < 0 || rows <= 0 || n < 0) return GDN_ERR_INVALID_ARGUMENT;
    if (n_buffers > gdn::kCopyMaxBuffers) return GDN_ERR_UNSUPPORTED;
    if (n_buffers == 0 || n == 0) return GDN_OK;
    if (!buffers) return GDN_ERR_INVALID_ARGUMENT;
    gdn_status st = check_ints({src_ids, dst_ids});
    if (st != GDN_OK) return st;
    gdn::CopyArgs a{};
    for (int i = 0; i < n_buffers; ++i) {
        if (!buffers[i].base || buffers[i].row_bytes <= 0) return GDN_ERR_INVALID_ARGUMENT;
        if (misaligned(buffers[i].base, 16) || buffers[i].row_bytes % 16 != 0) return GDN_ERR_MISALIGNED;
        if (buffers[i].row_bytes > (1L << 32)) return GDN_ERR_UNSUPPORTED;
        a.base[i] = static_cast<unsigned char*>(buffers[i].base);
        a.row_bytes[i] = (long)buffers[i].row_bytes;
    }
    if (misaligned(n_dev, 4) || misaligned(err_flag, 4)) return GDN_ERR_MISALIGNED;
    a.n_bufs = n_buffers;
    a.rows = rows;
    a.n_max = n;
    a.src = src_ids;
    a.dst = dst_ids;
    a.n_dev = n_dev;
    a.err_flag = err_flag;
    return from_cuda(gdn::launch_copy_rows(a, (cudaStream_t)stream));
}

}  // extern "C"
