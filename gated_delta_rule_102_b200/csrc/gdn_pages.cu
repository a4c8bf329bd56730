// Page tables of the paged cache on the device (reserve, fork, free, compact) and the
// copy of pool rows that forks and compactions ask for.
//
// Whole numbers only. What a call allocates is always the lowest free page, in the order
// of the call's sequences, so two runs give the same tables. One CTA does the part that
// needs an order (how many pages each sequence lacks, which pages are free): it walks the
// reference counters 8192 at a time, a warp's ballot giving each free page its rank, and
// stops as soon as enough are found; a second launch over the whole GPU does the part that
// does not (copying table rows, renumbering entries). The work is a few dependent passes
// over small arrays: bound by latency, not bandwidth (free, fork and reserve of 2 children: 8 us
// together). The copies are bound by HBM: 500 moves in a pool of 2000 pages (four buffers of 64 KB a
// page, 131 MB read and as many written) take 46 us, 5.7 TB/s.
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_attn.h"
#include "gdn_device.cuh"

namespace gdn {
namespace {

constexpr int kT = 1024, kWarps = kT / 32, kPer = 8;
constexpr int kChunk = kT * kPer;  // counters looked at in one step

__device__ __forceinline__ void flag(int32_t* err, int bit) {
    if (err) atomicOr(err, bit);
}
__device__ __forceinline__ void pdl_wait() {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
}

// Sums of counts stay at 2^31 - 1 once they get there: more than any pool has, in any order.
__device__ __forceinline__ int add_sat(int a, int b) { return (int)min((unsigned)a + (unsigned)b, 0x7fffffffu); }

// Exclusive prefix sum of counts over the block (kT threads); *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x = add_sat(x, y);
    }
    if (lane == 31) warp_sums[warp] = x;
    const int left = __shfl_up_sync(0xffffffffu, x, 1);
    __syncthreads();
    if (warp == 0) {
        int s = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s = add_sat(s, y);
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    const int before = warp ? warp_sums[warp - 1] : 0;
    *total = warp_sums[kWarps - 1];
    __syncthreads();
    return add_sat(before, lane ? left : 0);
}

// Calls take(rank, page) for the lowest `want` pages whose counter is 0, in any order of
// calls; returns how many there are (at most `want`). All threads of the block.
template <typename Take>
__device__ __forceinline__ int lowest_free(const int32_t* refs, int num_pages, int want, int* warp_sums, Take take) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int found = 0;
    for (int base = 0; base < num_pages && found < want; base += kChunk) {
        const int at = base + warp * (32 * kPer) + lane;
        int r[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) r[i] = at + 32 * i < num_pages ? refs[at + 32 * i] : 1;
        unsigned m[kPer];
        int mine = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            m[i] = __ballot_sync(0xffffffffu, r[i] == 0);
            mine += __popc(m[i]);
        }
        int total;
        int rank = found + block_scan(lane == 0 ? mine : 0, warp_sums, &total);
        rank = __shfl_sync(0xffffffffu, rank, 0);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int k = rank + __popc(m[i] & ((1u << lane) - 1u));
            if (r[i] == 0 && k < want) take(k, at + 32 * i);
            rank += __popc(m[i]);
        }
        found += total;
    }
    return found < want ? found : want;
}

// The sequence whose pages have ranks prefix[i] .. prefix[i+1]-1.
__device__ __forceinline__ int owner(const int* prefix, int n, int rank) {
    int lo = 0, hi = n;  // prefix[lo] <= rank < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= rank) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kT) pages_reserve_kernel(const PageArgs p) {
    __shared__ int warp_sums[kWarps], prefix[kPagesMaxBatch + 1], start[kPagesMaxBatch];
    pdl_wait();
    const int ps = p.page_size;
    int total = 0;
    for (int base = 0; base < p.n; base += kT) {
        const int i = base + threadIdx.x;
        int need = 0, from = 0;
        if (i < p.n) {
            const int slot = p.slots[i];
            if (slot < 0 || slot >= p.rows) {
                flag(p.err_flag, GDN_DEVICE_ERR_SLOT_RANGE_BIT);
            } else {
                const long len = p.seq_lens[slot], more = p.n_tokens ? p.n_tokens[i] : p.T;
                const long want = (len + more + ps - 1) / ps;
                if (len < 0 || more < 0 || want > p.max_pages) {
                    flag(p.err_flag, GDN_DEVICE_ERR_SEQLEN_BIT);
                } else {
                    from = (int)((len + ps - 1) / ps);
                    while (from < want && p.table[(long)slot * p.max_pages + from] >= 0) ++from;  // held already
                    need = (int)want - from;
                }
            }
        }
        int sum;
        const int before = block_scan(need, warp_sums, &sum);
        if (i < p.n) {
            prefix[i] = add_sat(total, before);
            start[i] = from;
        }
        total = add_sat(total, sum);
    }
    if (threadIdx.x == 0) prefix[p.n] = total;
    __syncthreads();
    const int found = lowest_free(p.refs, p.num_pages, total, warp_sums, [&](int k, int page) {
        const int i = owner(prefix, p.n, k);
        p.table[(long)p.slots[i] * p.max_pages + start[i] + (k - prefix[i])] = page;
        p.refs[page] = 1;
    });
    if (found < total) {  // too few: a sequence gets all its pages or none
        __syncthreads();
        const int i = owner(prefix, p.n, found);
        for (int k = prefix[i] + threadIdx.x; k < found; k += kT) {
            int32_t* e = p.table + (long)p.slots[i] * p.max_pages + start[i] + (k - prefix[i]);
            p.refs[*e] = 0;
            *e = -1;
        }
        if (threadIdx.x == 0) flag(p.err_flag, GDN_DEVICE_ERR_PAGE_BIT);
    }
}

// copy_dst of a pair that was skipped (-1: forked, nothing to copy)
constexpr int kSkipped = -2;

// The whole pages of a forked child: the parent's, with one holder more. Threads begin, begin + step, ..
__device__ __forceinline__ void share_pages(const PageArgs& p, int i, int begin, int step) {
    if (p.copy_dst[i] == kSkipped) return;
    const int src = p.src_slots[i], full = p.seq_lens[src] / p.page_size;
    const int32_t* parent = p.table + (long)src * p.max_pages;
    int32_t* child = p.table + (long)p.slots[i] * p.max_pages;
    for (int j = begin; j < full; j += step) {
        const int e = parent[j];
        child[j] = e;
        if (e >= 0 && e < p.num_pages) atomicAdd(p.refs + e, 1);
        else flag(p.err_flag, GDN_DEVICE_ERR_PAGE_BIT);
    }
}

__global__ void __launch_bounds__(kT) pages_fork_kernel(const PageArgs p, const bool share) {
    __shared__ int warp_sums[kWarps], prefix[kPagesMaxBatch + 1];
    pdl_wait();
    const int ps = p.page_size;
    int total = 0;
    for (int base = 0; base < p.n; base += kT) {
        const int i = base + threadIdx.x;
        int need = 0;
        if (i < p.n) {
            const int src = p.src_slots[i], dst = p.slots[i];
            int from = -1, to = kSkipped;
            if (src < 0 || src >= p.rows || dst < 0 || dst >= p.rows || src == dst) {
                flag(p.err_flag, GDN_DEVICE_ERR_SLOT_RANGE_BIT);
            } else {
                const int32_t* parent = p.table + (long)src * p.max_pages;
                int32_t* child = p.table + (long)dst * p.max_pages;
                const int len = p.seq_lens[src], full = len / ps;
                const bool part = len > 0 && len % ps != 0;
                if (len < 0 || full + (part ? 1 : 0) > p.max_pages) {
                    flag(p.err_flag, GDN_DEVICE_ERR_SEQLEN_BIT);
                } else if (p.seq_lens[dst] != 0 || child[0] >= 0) {
                    flag(p.err_flag, GDN_DEVICE_ERR_PAGE_BIT);
                } else if (part && (parent[full] < 0 || parent[full] >= p.num_pages)) {
                    flag(p.err_flag, GDN_DEVICE_ERR_PAGE_BIT);
                } else if (part) {
                    need = 1;
                    from = parent[full];
                } else {
                    to = -1;
                }
            }
            p.copy_src[i] = from;
            p.copy_dst[i] = to;
        }
        int sum;
        const int before = block_scan(need, warp_sums, &sum);
        if (i < p.n) prefix[i] = add_sat(total, before);
        total = add_sat(total, sum);
    }
    if (threadIdx.x == 0) prefix[p.n] = total;
    __syncthreads();
    const int found = lowest_free(p.refs, p.num_pages, total, warp_sums, [&](int k, int page) {
        const int i = owner(prefix, p.n, k);
        p.copy_dst[i] = page;
        p.refs[page] = 1;
        p.table[(long)p.slots[i] * p.max_pages + p.seq_lens[p.src_slots[i]] / ps] = page;
    });
    if (found < total && threadIdx.x == 0) flag(p.err_flag, GDN_DEVICE_ERR_PAGE_BIT);
    __syncthreads();
    for (int i = threadIdx.x; i < p.n; i += kT) {
        if (p.copy_dst[i] != kSkipped) p.seq_lens[p.slots[i]] = p.seq_lens[p.src_slots[i]];
        else p.copy_src[i] = -1;
    }
    if (!share) return;
    __syncthreads();
    for (int i = threadIdx.x >> 5; i < p.n; i += kWarps) share_pages(p, i, threadIdx.x & 31, 32);
}

__global__ void __launch_bounds__(256) pages_share_kernel(const PageArgs p) {
    pdl_wait();
    share_pages(p, blockIdx.x, blockIdx.y * 256 + threadIdx.x, gridDim.y * 256);
}

__global__ void __launch_bounds__(256) pages_free_kernel(const PageArgs p) {
    pdl_wait();
    const int slot = p.slots[blockIdx.x];
    if (slot < 0 || slot >= p.rows) {
        if (blockIdx.y == 0 && threadIdx.x == 0) flag(p.err_flag, GDN_DEVICE_ERR_SLOT_RANGE_BIT);
        return;
    }
    int32_t* row = p.table + (long)slot * p.max_pages;
    for (int j = blockIdx.y * 256 + threadIdx.x; j < p.max_pages; j += gridDim.y * 256) {
        if (row[j] < 0) continue;
        const int e = atomicExch(row + j, -1);  // one release even if the slot is listed twice
        if (e >= p.num_pages) flag(p.err_flag, GDN_DEVICE_ERR_PAGE_BIT);
        else if (e >= 0) atomicSub(p.refs + e, 1);
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) p.seq_lens[slot] = 0;
}

__global__ void __launch_bounds__(kT) pages_compact_kernel(const PageArgs p) {
    __shared__ int warp_sums[kWarps], live_total;
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, P = p.num_pages;
    // how many pages are in use: they end up as pages 0 .. live-1
    int mine = 0;
    for (int base = threadIdx.x; base < P; base += kChunk) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) mine += base + i * kT < P && p.refs[base + i * kT] > 0;
    }
    int live;
    block_scan(mine, warp_sums, &live);
    if (threadIdx.x == 0) live_total = live;
    __syncthreads();
    live = live_total;
    // the k-th used page from `live` on moves to the k-th free one before it; in a step, a
    // warp's pages lie on one side or the other except in one step, so both ranks are kept
    int holes = 0, movers = 0;
    for (int base = 0; base < P; base += kChunk) {
        const int at = base + warp * (32 * kPer) + lane;
        bool used[kPer];
        unsigned mh[kPer], mm[kPer];
        int nh = 0, nm = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) used[i] = at + 32 * i < P && p.refs[at + 32 * i] > 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int id = at + 32 * i;
            mh[i] = __ballot_sync(0xffffffffu, id < live && !used[i]);
            mm[i] = __ballot_sync(0xffffffffu, id >= live && used[i]);
            nh += __popc(mh[i]);
            nm += __popc(mm[i]);
        }
        int th, tm;
        int rh = holes + block_scan(lane == 0 ? nh : 0, warp_sums, &th);
        int rm = movers + block_scan(lane == 0 ? nm : 0, warp_sums, &tm);
        rh = __shfl_sync(0xffffffffu, rh, 0);
        rm = __shfl_sync(0xffffffffu, rm, 0);
        const unsigned below = (1u << lane) - 1u;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int id = at + 32 * i;
            if (id < P) p.remap[id] = used[i] ? id : -1;
            if ((mh[i] >> lane) & 1u) p.copy_dst[rh + __popc(mh[i] & below)] = id;
            if ((mm[i] >> lane) & 1u) p.copy_src[rm + __popc(mm[i] & below)] = id;
            rh += __popc(mh[i]);
            rm += __popc(mm[i]);
        }
        holes += th;
        movers += tm;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < P; i += kT) {
        if (i < movers) {
            const int from = p.copy_src[i], to = p.copy_dst[i];
            p.remap[from] = to;
            p.refs[to] = p.refs[from];
            p.refs[from] = 0;
        } else {
            p.copy_src[i] = -1;
            p.copy_dst[i] = -1;
        }
    }
    if (threadIdx.x == 0) *p.n_copies = movers;
}

__global__ void __launch_bounds__(256) pages_renumber_kernel(const PageArgs p) {
    pdl_wait();
    const long n = (long)p.rows * p.max_pages;
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) {
        const int e = p.table[i];
        if (e < 0) continue;
        if (e >= p.num_pages) flag(p.err_flag, GDN_DEVICE_ERR_PAGE_BIT);
        else p.table[i] = p.remap[e];
    }
}

// ---------------------------------------------------------------------------------
// Rows of many buffers at once. A warp takes pieces of 4 KB (eight 16-byte words a lane,
// all loaded before the first store); with 32 warps an SM keeps 128 KB in flight, above
// what latency times bandwidth needs (about 45 KB), and rows of any size, one page or a
// 2 MB state, spread over the whole GPU. Bound by HBM: each byte is read and written once.
constexpr int kWords = 8, kPiece = kWords * 512, kCtas = 4;

__global__ void __launch_bounds__(256, kCtas) copy_rows_kernel(const __grid_constant__ CopyArgs p) {
    pdl_wait();
    int n = p.n_max;
    if (p.n_dev) {
        n = __ldg(p.n_dev);
        if (n < 0 || n > p.n_max) {
            if (blockIdx.x == 0 && threadIdx.x == 0) flag(p.err_flag, GDN_DEVICE_ERR_BATCH_BIT);
            return;
        }
    }
    const int lane = threadIdx.x & 31;
    const long per = p.first_chunk[p.n_bufs], items = per * n;
    for (long it = (long)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += (long)gridDim.x * 8) {
        const int pair = (int)(it / per);
        const long c = it - (long)pair * per;
        int lo = 0, hi = p.n_bufs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.first_chunk[mid] <= c) lo = mid; else hi = mid;
        }
        const int src = __ldg(p.src + pair), dst = __ldg(p.dst + pair);
        if (src < 0 || dst < 0) continue;
        if (src >= p.rows || dst >= p.rows) {
            if (lane == 0) flag(p.err_flag, GDN_DEVICE_ERR_SLOT_RANGE_BIT);
            continue;
        }
        const long at = (c - p.first_chunk[lo]) * kPiece, bytes = p.row_bytes[lo];
        const int words = (int)((bytes - at < kPiece ? bytes - at : kPiece) / 16);
        const uint4* s = reinterpret_cast<const uint4*>(p.base[lo] + src * bytes + at);
        uint4* d = reinterpret_cast<uint4*>(p.base[lo] + dst * bytes + at);
        uint4 w[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            if (lane + 32 * i < words) w[i] = __ldcs(s + lane + 32 * i);
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            if (lane + 32 * i < words) __stcs(d + lane + 32 * i, w[i]);
    }
}

template <typename K, typename... A>
cudaError_t launch(K kernel, dim3 grid, int threads, cudaStream_t stream, const A&... a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a...);
}

// CTAs that share one table row of up to max_pages entries (four entries a thread).
int row_ctas(int max_pages) {
    const int c = (max_pages + 1023) / 1024;
    return c < 1 ? 1 : (c > 64 ? 64 : c);
}

}  // namespace

cudaError_t launch_pages_reserve(const PageArgs& a, cudaStream_t stream) {
    return launch(pages_reserve_kernel, dim3(1), kT, stream, a);
}

cudaError_t launch_pages_fork(const PageArgs& a, cudaStream_t stream) {
    // a few thousand table entries are shared by the CTA that allocates; more pay for a launch of their own
    const bool share = (long)a.n * a.max_pages <= 4096;
    const cudaError_t e = launch(pages_fork_kernel, dim3(1), kT, stream, a, share);
    if (e != cudaSuccess || share) return e;
    return launch(pages_share_kernel, dim3(a.n, row_ctas(a.max_pages)), 256, stream, a);
}

cudaError_t launch_pages_free(const PageArgs& a, cudaStream_t stream) {
    return launch(pages_free_kernel, dim3(a.n, row_ctas(a.max_pages)), 256, stream, a);
}

cudaError_t launch_pages_compact(const PageArgs& a, cudaStream_t stream) {
    int dev, sms;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    if ((e = launch(pages_compact_kernel, dim3(1), kT, stream, a)) != cudaSuccess) return e;
    const long n = ((long)a.rows * a.max_pages + 1023) / 1024;
    return launch(pages_renumber_kernel, dim3((unsigned)(n < sms * 8 ? n : sms * 8)), 256, stream, a);
}

cudaError_t launch_copy_rows(CopyArgs& a, cudaStream_t stream) {
    int dev, sms;
    const cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    long chunks = 0;
    for (int i = 0; i < a.n_bufs; ++i) {
        a.first_chunk[i] = chunks;
        chunks += (a.row_bytes[i] + kPiece - 1) / kPiece;
    }
    a.first_chunk[a.n_bufs] = chunks;
    const long ctas = (chunks * a.n_max + 7) / 8;
    return launch(copy_rows_kernel, dim3((unsigned)(ctas < sms * kCtas ? ctas : sms * kCtas)), 256, stream, a);
}

}  // namespace gdn
