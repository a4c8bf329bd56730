// Building blocks of the paged-attention kernels: copies and matrix instructions, the layout
// of a tile of tokens in shared memory, the schedule that spreads a batch's work over the
// CTAs, and the join of units that several CTAs share.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_attn.h"
#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kJoinFlat = 12, kJoinGroup = 8;  // pieces of a unit that one CTA joins at once, and groups of more
constexpr int kJoinMost = (kAttnMaxCtas + kJoinGroup - 1) / kJoinGroup;
static_assert(kJoinMost >= kJoinFlat, "pieces joined at once");

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
    const int n = valid ? 16 : 0;  // 0: the 16 bytes are filled with zeros and nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;\n" ::: "memory"); }
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int c3, int c4, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, "
        "%4}], [%5];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
}
// The matrix loads are not volatile, so that the compiler may move them between the products;
// what keeps them behind the wait for their data and before its release is after_wait() on the
// address that they use and before_release() on the accumulators that depend on them.
__device__ __forceinline__ void after_wait(uint32_t& addr) { asm volatile("" : "+r"(addr)::"memory"); }
template <int N>
__device__ __forceinline__ void before_release(float (&acc)[N][4]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile("" : "+f"(acc[i][0]), "+f"(acc[i][1]), "+f"(acc[i][2]), "+f"(acc[i][3])::"memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// An 8 x 8 tile of 16-bit elements, two a lane in rows, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// c += a b, 16x8x16, bf16 or fp16 operands (both the same), fp32 sums.
template <bool HALF>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (HALF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
            "%2, %3};\n"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, "
            "%1, %2, %3};\n"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two e4m3 bytes (the low or high half of w) as two fp16, exactly.
__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t w, bool high) {
    uint32_t r;
    const uint16_t h = (uint16_t)(high ? w >> 16 : w);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool HALF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (HALF) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of 16-byte chunk c of token row r in a tile's keys (or values): atoms of eight
// rows by 128 bytes in which chunk c is stored at c ^ (r % 8) (64-byte rows: two to a line,
// c ^ (r / 2 % 4)), the swizzles that the TMA unit applies. Eight rows, eight bank groups.
template <int CPR>
__device__ __forceinline__ int chunk_at(int r, int c) {
    if (CPR >= 8) return ((r >> 3) * (CPR / 8) + (c >> 3)) * 1024 + (r & 7) * 128 + (((c ^ r) & 7) << 4);
    return r * 64 + (((c ^ (r >> 1)) & 3) << 4);
}

__device__ __forceinline__ int load_acquire(const int* at) {
    int v;
    asm volatile("ld.acquire.cta.shared::cta.b32 %0, [%1];\n" : "=r"(v) : "r"(smem_addr(at)) : "memory");
    return v;
}
__device__ __forceinline__ void add_release(int* at) {
    asm volatile("red.release.cta.shared::cta.add.u32 [%0], 1;\n" ::"r"(smem_addr(at)) : "memory");
}
__device__ __forceinline__ float sigmoid_fast(float x) { return __fdividef(1.0f, 1.0f + exp2_fast(-x * kLog2e)); }

// Raises the call's timeout flag and makes every role of the CTA leave at its next wait.
static __device__ __noinline__ void attn_abort(int32_t* err_flag, volatile int* stop) {
    if (err_flag) atomicOr(err_flag, GDN_DEVICE_ERR_TIMEOUT_BIT);
    *stop = 1;
}

// ---------------------------------------------------------------------------------
// The schedule. The G query heads of a key/value head and a sequence's n new tokens form
// n * G query rows that read the same keys, so a work unit is (sequence, row tile,
// key/value head) and costs its number of tiles of ST tokens, plus some for its
// beginning and end. All units' costs in a row are "places"; the CTAs get equal,
// contiguous shares of them. It follows from the lengths alone, which are read on the
// device: every CTA sums the batch.

// A sequence as the schedule sees it.
struct Seq {
    int n, first, past, slot;  // tokens of this call, their first row, tokens before them
    int lo, base, tiles;       // first position any row attends, the tiles' first position, tiles
    int cost;                  // places of a unit beside its tiles'
    int row_tiles;
};

// Tiles of ST tokens; a unit of at most SHORT tiles costs SHORT_COST more, any other COST.
template <int ST, int SHORT, int SHORT_COST, int COST>
struct Share {
    const AttnArgs& p;
    const int row_tile;  // query rows of a unit
    const int* prefix;  // [B + 1] (shared memory) places before each sequence
    int Hkv, total, ctas, per, more, lo, hi;
    Seq s;
    int b, unit, place, tile;  // where we are: unit = row_tile * Hkv + head, the place of its first tile, the tile

    __device__ __forceinline__ Share(const AttnArgs& args, int row_tile_, const int* prefix_) : p(args), row_tile(row_tile_), prefix(prefix_), Hkv(args.sh.Hkv) {}

    __device__ __forceinline__ Seq load(int i, bool report) const {
        Seq q;
        q.tiles = 0;
        q.cost = 0;
        q.row_tiles = 0;
        q.slot = __ldg(p.slots + i);
        q.first = i * p.T;
        q.n = p.T;
        if (p.cu) {
            q.first = __ldg(p.cu + i);
            q.n = __ldg(p.cu + i + 1) - q.first;
        }
        q.past = 0;
        q.lo = 0;
        q.base = 0;
        if (q.n < 0 || q.n > p.T || q.first < 0 || q.first > p.total - q.n) {
            if (report && p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_SEQLEN_BIT);
            q.n = 0;
            return q;
        }
        if (q.n == 0) return q;
        if (q.slot < 0 || q.slot >= p.c.rows) {
            if (report && p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_SLOT_RANGE_BIT);
            return q;
        }
        q.past = __ldg(p.c.seq_lens + q.slot);
        if (q.past < 0 || q.past > p.c.max_pages * p.sh.page_size - q.n) {
            if (report && p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_SEQLEN_BIT);
            return q;
        }
        if (p.sh.window > 0 && q.past + 1 > p.sh.window) q.lo = q.past + 1 - p.sh.window;
        q.base = q.lo & ~(ST - 1);
        q.tiles = (q.past + q.n - q.base + ST - 1) / ST;
        q.cost = q.tiles <= SHORT ? SHORT_COST : COST;
        q.row_tiles = (q.n * p.sh.G + row_tile - 1) / row_tile;
        return q;
    }

    // All NT threads of the block: fills `places` (the prefix array) and `total`. `sums`: NT / 32 ints.
    template <int NT>
    __device__ __forceinline__ void sum_batch(int* places, int* sums) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        total = 0;
        for (int base = 0; base < p.B; base += NT) {
            const int i = base + tid;
            int t = 0;
            if (i < p.B) {
                const Seq q = load(i, blockIdx.x == 0);
                t = (q.tiles + q.cost) * q.row_tiles * Hkv;
            }
            int x = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) sums[warp] = x;
            __syncthreads();
            int before = total, sum = 0;
#pragma unroll
            for (int w = 0; w < NT / 32; ++w) {
                if (w < warp) before += sums[w];
                sum += sums[w];
            }
            if (i < p.B) places[i] = before + x - t;
            total += sum;
            __syncthreads();
        }
        if (tid == 0) places[p.B] = total;
        __syncthreads();
    }

    // This CTA's share and its first tile; false when it has none. No more CTAs than SMs, and
    // no fewer than `least` places a CTA. CTA c has the places c * per + min(c, more) on: per of
    // them, one more for the first ones.
    __device__ __forceinline__ bool begin(int least) {
        ctas = min((int)gridDim.x, (total + least - 1) / least);
        if ((int)blockIdx.x >= ctas) return false;
        per = total / ctas;
        more = total - per * ctas;
        lo = blockIdx.x * per + min((int)blockIdx.x, more);
        hi = lo + per + ((int)blockIdx.x < more);
        int end = p.B;
        b = 0;
        while (end - b > 1) {
            const int mid = (b + end) >> 1;
            if (prefix[mid] <= lo) b = mid; else end = mid;
        }
        s = load(b, false);  // the last sequence that starts at or before the share: it has units
        unit = (lo - prefix[b]) / (s.tiles + s.cost);
        place = prefix[b] + unit * (s.tiles + s.cost) + s.cost;
        tile = max(lo - place, 0);
        return place + tile < hi;  // or nothing but a unit's overhead
    }

    __device__ __forceinline__ int cta_of(int at) const {
        const int big = more * (per + 1);
        return at < big ? at / (per + 1) : more + (at - big) / per;
    }

    // To the next unit's first place (`tile` is the caller's); false when it lies past the share.
    __device__ __forceinline__ bool next_unit() {
        place += s.tiles;  // the unit's end
        if (place >= hi) return false;
        if (++unit == s.row_tiles * Hkv) {
            unit = 0;
            do {
                ++b;
            } while (prefix[b + 1] == prefix[b]);
            s = load(b, false);
        }
        place += s.cost;
        return place < hi;
    }

    // `by` tiles on; false past the end of the share.
    __device__ __forceinline__ bool advance(int by) {
        tile += by;
        while (tile >= s.tiles) {
            tile -= s.tiles;
            if (!next_unit()) return false;
        }
        return place + tile < hi;
    }

    // Token number (page * page_size + offset) of the `len` tokens from position `pos` on, which
    // lie in one page; -1 where the sequence has none of them or the table no page.
    __device__ __forceinline__ int look_up(int pos, int len) const {
        if (pos + len <= s.lo || pos >= s.past + s.n) return -1;
        const int at = pos / p.sh.page_size;
        const int page = __ldg(p.c.table + (size_t)s.slot * p.c.max_pages + at);
        if (page >= 0 && page < p.c.num_pages) return page * p.sh.page_size + (pos - at * p.sh.page_size);
        if (p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_PAGE_BIT);
        return -1;
    }
};

// The cap c tanh(x / c) of scores, in log2 units. Up to kPlainCap it is c - 2 c / (1 + e^(2 x / c)), off by
// 1.2 c 2^-22 at most (the exponential by 2^-22 of itself, the reciprocal by 2^-23 and a rounding):
// less than what products in 32 bits leave of a score. For larger caps that would not do. With y = x / c,
// below a half the odd series x (1 + u (a0 + a1 u + a2 u^2 + a3 u^3)), u = y^2, whose coefficients
// interpolate (tanh(y) / y - 1) / u at the Chebyshev points of u in [0, 1/4] (off by 2^-24), and from
// there on the quotient of |x| with x's sign: each is off by at most 2^-20 of x, the quotient because c is
// at most 2.2 times the result there. That is a call of its own, through local memory: in line, for every
// cap, 16 drafted tokens of 64 sequences of 1000 to 8000 tokens (d = 256) took 240 us at a cap of 3, so
// 138; in line for large caps only it took uncapped calls up to 15 % longer by the code between their
// instructions, so 1 % (5 % with 32 rows of d = 64). At a cap of 100 the drafted tokens take 255 us, and
// one token of each sequence 87, so 86 without a cap.
constexpr float kPlainCap = 64.0f;
// A factor of scores for a cap next to zero: a score of zero stays one.
__device__ __forceinline__ float finite(float x) { return fminf(fmaxf(x, -3e38f), 3e38f); }
// A warp's scores, N a lane (log2 units, not yet capped), by a cap above kPlainCap.
template <int N>
__device__ __noinline__ void cap_large(float (&x)[N], float softcap) {
    const float c = fminf(softcap * kLog2e, 0x1p126f), inv = 1.0f / c;  // (twice c is finite, too)
#pragma unroll 16
    for (int i = 0; i < N; ++i) {
        const float y = x[i] * inv, u = y * y;
        const float near = fmaf(x[i] * u, fmaf(u, fmaf(u, fmaf(u, 0.01798874f, -0.05338711f), 0.13330476f), -0.33333311f), x[i]);
        const float far = fmaf(-2.0f * c, rcp_fast(1.0f + exp2_fast(fabsf(y) * (2.0f * kLog2e))), c);
        x[i] = fabsf(y) >= 0.5f ? copysignf(far, x[i]) : near;
    }
}

// With an e4m3 cache the probabilities are fp16, whose normal numbers end at 2^-14 and whose smallest
// is 2^-24. So a row's reference lies kUp below its maximum: P goes up to 2^15, is rounded once to 11
// bits down to 2^-29 of the row's largest, and vanishes below 2^-40 of it. (With the maximum itself the
// same came at 2^-14 and 2^-25, which a flat tail of many tokens below a sink reaches.) Sums and outputs
// carry the factor, and their quotient cancels it. A reference may be any number near the maximum as
// long as one row uses one; beyond 2^22, where 32 bits cannot place it to a quarter, it is the maximum.
constexpr float kUp = 15.0f;
__device__ __forceinline__ float fp16_reference(float top) { return fabsf(top) < 0x1p22f ? top - kUp : top; }
// The natural logarithm of a row's sum from its reference and the sum of exp2(x - reference). (The factor
// goes first: the logarithm of a sum of 2^15 has four bits fewer behind the point.)
template <bool FP8>
__device__ __forceinline__ float log_sum(float ref, float sum) {
    return FP8 ? ((ref + kUp) + log2f(sum * 0x1p-15f)) * kLn2 : (ref + log2f(sum)) * kLn2;
}

// Four columns of an output row: their gates (read apart, so that many are in flight), and the
// values normalised, gated and rounded once.
__device__ __forceinline__ uint2 gate_of4(const AttnArgs& p, size_t row, int head, int col) {
    return __ldg(reinterpret_cast<const uint2*>(p.gate.ptr + row * p.gate.row + (size_t)head * p.gate.head + col));
}
template <bool FP8>
__device__ __forceinline__ void write_out4(const AttnArgs& p, size_t row, int head, int d, int col, float4 o, float inv, uint2 z) {
    o.x *= inv;
    o.y *= inv;
    o.z *= inv;
    o.w *= inv;
    if (FP8) {  // the cache's scale by itself: a tiny one over the sum might not be a normal number
        o.x *= p.sh.v_scale;
        o.y *= p.sh.v_scale;
        o.z *= p.sh.v_scale;
        o.w *= p.sh.v_scale;
    }
    if (p.gate.ptr) {
        o.x *= sigmoid_fast(__uint_as_float(z.x << 16));
        o.y *= sigmoid_fast(__uint_as_float(z.x & 0xffff0000u));
        o.z *= sigmoid_fast(__uint_as_float(z.y << 16));
        o.w *= sigmoid_fast(__uint_as_float(z.y & 0xffff0000u));
    }
    *reinterpret_cast<uint2*>(p.out + (row * p.sh.Hq + head) * d + col) = make_uint2(pack2<false>(o.x, o.y), pack2<false>(o.z, o.w));
}

// ---------------------------------------------------------------------------------
// Units over several CTAs. Each leaves its piece (fp32, unnormalised: [BM][D], then the rows'
// maxima and sums) in the workspace, at 2 c + 1 for the unit that ends CTA c's share and 2 c
// for the one that begins it; the last CTA to get here joins a unit's pieces, in their order:
// the result does not depend on which one that is. More than kJoinFlat pieces are joined in
// groups of kJoinGroup first (by the last CTA of the group, into its first piece's place),
// then the groups: at 74 pieces of 8 KB one CTA alone would read 600 KB.
// All NT threads that meet() joins, after each has written its part of the pieces.
// shared_pieces: the share's first and last split piece; wt: BM * (kJoinMost + 2) floats and
// flag: one int of shared memory.
template <int D, bool FP8, int BM, int NT, typename Meet>
__device__ __forceinline__ bool join_units(const AttnArgs& p, const Piece* shared_pieces, bool split_first, bool split_last,
                                           float* wt, volatile int* flag, Meet meet) {
    constexpr int WP = kJoinMost + 2, PSTRIDE = BM * (D + 2);
    const int tid = threadIdx.x, G = p.sh.G, inv_g = 65536 / G + 1;  // r / G = r * inv_g >> 16 for r < 320, G <= 16
    if (!split_first && !split_last) return true;
    __threadfence();
    if (!meet()) return false;
    for (int which = 0; which < 2; ++which) {
        if (!(which ? split_last : split_first)) continue;
        const Piece u = shared_pieces[which];
        const int rows = min(BM, u.n * G - u.rt * BM), all = u.c1 - u.c0 + 1;
        auto place_of = [&](int i) { return p.partial + (size_t)((u.c0 + i) * 2 + (i == 0)) * PSTRIDE; };
        const bool flat = all <= kJoinFlat;
        for (int level = flat ? 1 : 0; level < 2; ++level) {
            // level 0: this CTA's group of pieces; level 1: all pieces, or the groups' first places
            const int step = level == 1 && !flat ? kJoinGroup : 1;
            const int from = level == 0 ? ((int)blockIdx.x - u.c0) / kJoinGroup * kJoinGroup : 0;
            const int count = level == 0 ? min(kJoinGroup, all - from) : (all + step - 1) / step;
            unsigned int* counter = p.counters + (level == 1 ? u.c0 : kAttnMaxCtas + (u.c0 + from) * 2 + (from == 0));
            if (tid == 0) *flag = atomicAdd(counter, 1u) == (unsigned)(count - 1);
            if (!meet()) return false;
            if (!*flag) break;  // (written next after another meeting)
            __threadfence();
            const float* first = place_of(from);
            const float* rest = place_of(from + step);  // of the second piece, the others at equal distances
            const size_t stride = (size_t)step * 2 * PSTRIDE;
            auto part = [&](int i) { return i == 0 ? first : rest + (size_t)(i - 1) * stride; };
            // (never more than kAttnMaxCtas / kJoinGroup pieces here: a thread a row)
            if (tid < rows) {
                float* w = wt + tid * WP;
                float top = -INFINITY, tot = 0.0f;
#pragma unroll 8
                for (int i = 0; i < count; ++i) {
                    w[i] = __ldcg(part(i) + BM * D + tid);
                    top = fmaxf(top, w[i]);
                }
#pragma unroll 8
                for (int i = 0; i < count; ++i) {
                    const float f = w[i] == -INFINITY ? 0.0f : exp2_fast(w[i] - top);
                    tot = fmaf(f, __ldcg(part(i) + BM * D + BM + tid), tot);
                    w[i] = f;
                }
                w[kJoinMost] = tot;
                w[kJoinMost + 1] = top;
            }
            if (!meet()) return false;
            // four columns by kItems rows a thread, so that their loads are in flight together
            constexpr int kItems = BM > 16 ? 4 : 2, kPieces = 4;
            const int items = rows * (D / 4);
            for (int k0 = tid; k0 < items; k0 += kItems * NT) {
                float4 o[kItems];
                uint2 z[kItems];
#pragma unroll
                for (int y = 0; y < kItems; ++y) {
                    const int k = k0 + y * NT, r = k / (D / 4), rr = u.rt * BM + r, t = (rr * inv_g) >> 16;
                    o[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    z[y] = make_uint2(0, 0);
                    if (p.gate.ptr && level == 1 && k < items) z[y] = gate_of4(p, (size_t)u.first + t, u.h * G + rr - t * G, (k % (D / 4)) * 4);
                }
                for (int i0 = 0; i0 < count; i0 += kPieces) {
                    float4 x[kPieces][kItems];
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const float* at = part(i0 + i);
#pragma unroll
                        for (int y = 0; y < kItems; ++y) {
                            const int k = k0 + y * NT;
                            x[i][y] = i0 + i < count && k < items ? __ldcg(reinterpret_cast<const float4*>(at) + k)
                                                                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
#pragma unroll
                        for (int y = 0; y < kItems; ++y) {
                            const int k = k0 + y * NT;
                            const float f = i0 + i < count && k < items ? wt[k / (D / 4) * WP + i0 + i] : 0.0f;
                            o[y].x = fmaf(f, x[i][y].x, o[y].x);
                            o[y].y = fmaf(f, x[i][y].y, o[y].y);
                            o[y].z = fmaf(f, x[i][y].z, o[y].z);
                            o[y].w = fmaf(f, x[i][y].w, o[y].w);
                        }
                    }
                }
#pragma unroll
                for (int y = 0; y < kItems; ++y) {
                    const int k = k0 + y * NT;
                    if (k >= items) continue;
                    if (level == 0) {
                        reinterpret_cast<float4*>(place_of(from))[k] = o[y];
                        continue;
                    }
                    const int r = k / (D / 4), col = (k % (D / 4)) * 4;
                    const int rr = u.rt * BM + r, t = (rr * inv_g) >> 16, head = u.h * G + rr - t * G;
                    const size_t row = (size_t)u.first + t;
                    const float* w = wt + r * WP;
                    write_out4<FP8>(p, row, head, D, col, o[y], 1.0f / w[kJoinMost], z[y]);
                    if (p.lse && col == 0) p.lse[row * p.sh.Hq + head] = log_sum<FP8>(w[kJoinMost + 1], w[kJoinMost]);
                }
            }
            if (tid == 0) *counter = 0;
            if (level == 0 && tid < rows) {  // the group's maximum and sum, in place of its first piece's
                float* to = place_of(from) + BM * D;
                to[tid] = wt[tid * WP + kJoinMost + 1];
                to[BM + tid] = wt[tid * WP + kJoinMost];
            }
            if (level == 0) __threadfence();
            if (!meet()) return false;  // the next weights go where these are
        }
        if (which == 0 && split_last && !meet()) return false;  // *flag is written again
    }
    return true;
}

// A tensor map over a pool of pages as [head][token / 8][128-byte block][token % 8][byte],
// in boxes of `box` tokens of one head: the atoms that the kernels read, in their order.
inline bool make_pool_map(CUtensorMap* m, void* pool, const AttnArgs& a, int row_bytes, int box) {
    const int inner = row_bytes < 128 ? row_bytes : 128, blocks = row_bytes / inner, esz = a.sh.fp8 ? 1 : 2;
    const cuuint64_t token = (cuuint64_t)a.sh.Hkv * row_bytes;
    const cuuint64_t dims[5] = {(cuuint64_t)(inner / esz), 8, (cuuint64_t)blocks, (cuuint64_t)a.c.num_pages * a.sh.page_size / 8,
                                (cuuint64_t)a.sh.Hkv};
    const cuuint64_t strides[4] = {token, (cuuint64_t)inner, token * 8, (cuuint64_t)row_bytes};
    const cuuint32_t boxes[5] = {(cuuint32_t)(inner / esz), 8, (cuuint32_t)blocks, (cuuint32_t)box / 8, 1};
    // A token's row of a head that is 128 bytes long lies alone: fetching 256 would bring another head's,
    // too (d = 64 bf16, 64 x 6700 tokens: 223 us, 177 with 128).
    return encode_tensor_map(m, a.sh.fp8, 5, pool, dims, strides, boxes, inner, row_bytes >= 256);
}

}  // namespace gdn
