// Internal interface of the softmax-attention layer (norm + rotary + append, paged
// attention, page tables, row copies) between the C-ABI layer and the kernel
// launchers. Nothing here is exported.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {

constexpr int GDN_DEVICE_ERR_PAGE_BIT = 16;

// Heads of a token row: element (row, head, i) at ptr[row * row_stride + head * head_stride + i].
struct Heads {
    const uint16_t* ptr;
    long row, head;
};

struct AttnShape {
    int Hq, Hkv, d, G;  // G = Hq / Hkv query heads per key/value head
    int R;              // rotated leading dimensions of a head
    bool interleaved, fp8;
    int page_size, window;
    float norm_eps, norm_offset, rope_scale, sm_scale, softcap, k_scale, v_scale;
};

// One layer's pages and the tables that the layers share.
struct PagedCache {
    void* k;
    void* v;
    int num_pages;
    const int32_t* table;  // [rows][max_pages]
    int rows, max_pages;
    const int32_t* seq_lens;  // [rows]
};

struct AppendArgs {
    AttnShape sh;
    PagedCache c;
    int B, T, total;
    const int32_t* cu;
    Heads q, k, v;
    const uint16_t* qw;
    const uint16_t* kw;
    const float* inv_freq;
    const int32_t* slots;
    uint16_t* q_out;
    int32_t* err_flag;
};

// A CTA's piece of a unit, as its loading warps describe it to the computing ones.
struct Piece {
    int n, first, past, lo, base;  // of the sequence
    int h, rt;                     // key/value head, row tile
    int tile, count;               // its first tile and how many
    int last;                      // the share ends with it
    int c0, c1;                    // the CTAs that share the unit
};

struct AttnArgs {
    AttnShape sh;
    PagedCache c;
    int B, T, total;
    const int32_t* cu;
    Heads q, gate;  // gate.ptr null: no gate
    const int32_t* slots;
    uint16_t* out;
    float* lse;
    int32_t* err_flag;
    unsigned int* counters;  // workspace: kAttnCounters zeroed counters, left zeroed
    Piece* split;            // workspace: kAttnMaxCtas units that go on in the next CTA (many rows)
    float* partial;          // workspace: two partial results per CTA
};

// CTAs of the attention kernel (one per SM, at most this many) and the workspace.
constexpr int kAttnMaxCtas = 192;
constexpr int kAttnCounters = 3 * kAttnMaxCtas;  // arrivals at units, and at groups of their pieces
constexpr size_t kAttnPartialAt = kAttnCounters * sizeof(unsigned int) + kAttnMaxCtas * sizeof(Piece);  // workspace offset
constexpr int kAttnMaxBatch = 2048;
// Places of the schedule (a unit's token tiles and what it costs beside them) of one sequence that fills
// its table row, or its window, for either kernel; a batch's are numbered in 32 bits.
constexpr long kAttnMaxPlaces = (1L << 31) - (1L << 16);
constexpr int kAttnUnitPlaces = 13;  // a tile at the window's edge, and more than either kernel's cost of a unit
long attn_decode_places(const AttnShape& sh, const PagedCache& c, int T);
long attn_rows_places(const AttnShape& sh, const PagedCache& c, int T);
inline long attn_places(const AttnShape& sh, const PagedCache& c, int T, int tile, int row_tile) {
    long positions = (long)c.max_pages * sh.page_size;
    if (sh.window > 0 && (long)sh.window + T < positions) positions = (long)sh.window + T;
    return ((positions + tile - 1) / tile + kAttnUnitPlaces) * ((T * sh.G + row_tile - 1) / row_tile) * sh.Hkv;
}
size_t attn_workspace_bytes(int d, bool fp8, int page_size, int rows);

cudaError_t launch_qk_rope_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t stream);
// The kernel for many rows on the tensor cores: whether it takes the shape, and its launch.
bool attn_rows_supported(int d, bool fp8, int page_size, int rows);
cudaError_t launch_attn_rows(const AttnArgs& a, cudaStream_t stream);

struct PageArgs {
    int page_size, n;           // sequences (or parent/child pairs) of this call
    const int32_t* slots;       // children for fork
    const int32_t* src_slots;   // fork: parents
    const int32_t* n_tokens;    // reserve: nullable per-sequence counts
    int T;                      // reserve: the count where n_tokens is null
    int32_t* table;
    int rows, max_pages;
    int32_t* seq_lens;
    int32_t* refs;
    int num_pages;
    int32_t* copy_src;
    int32_t* copy_dst;
    int32_t* n_copies;
    int32_t* remap;
    int32_t* err_flag;
};
constexpr int kPagesMaxBatch = 2048;
// Pages, and entries of a table row, at most: the kernels walk both in 32 bits, up to 2^14 at a time.
constexpr int kPagesMost = 0x7fffffff - (1 << 15);
cudaError_t launch_pages_reserve(const PageArgs& a, cudaStream_t stream);
cudaError_t launch_pages_fork(const PageArgs& a, cudaStream_t stream);
cudaError_t launch_pages_free(const PageArgs& a, cudaStream_t stream);
cudaError_t launch_pages_compact(const PageArgs& a, cudaStream_t stream);

constexpr int kCopyMaxBuffers = 64;
struct CopyArgs {
    unsigned char* base[kCopyMaxBuffers];
    long row_bytes[kCopyMaxBuffers];
    long first_chunk[kCopyMaxBuffers + 1];  // chunks of a pair that the buffers before this one hold
    int n_bufs, rows, n_max;
    const int32_t* src;
    const int32_t* dst;
    const int32_t* n_dev;
    int32_t* err_flag;
};
cudaError_t launch_copy_rows(CopyArgs& a, cudaStream_t stream);

// A tiled tensor map of bf16 values or bytes, swizzled over its inner dimension of 128 or 64 bytes;
// wide: misses in L2 fetch 256 bytes (128 otherwise).
bool encode_tensor_map(CUtensorMap* m, bool bytes, int rank, void* ptr, const cuuint64_t* dims, const cuuint64_t* strides,
                       const cuuint32_t* box, int inner_bytes, bool wide);

// The number of SMs of the current device (looked up once per device).
cudaError_t device_sms(int* device, int* sms);

}  // namespace gdn
