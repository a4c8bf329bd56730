// Attention of 1..16 new tokens per sequence over the paged key/value cache
// ("metrale_model_layers/forward/qwen3_5/full_attention.rs": the decode attention and
// the sigmoid output gate), one launch.
//
//   x = sm_scale q.k (capped: c tanh(x / c));  P = softmax(x);  out = (P v) sigmoid(gate)
//
// The G query heads of a key/value head and the call's n tokens form n*G query rows that
// read the same keys, so a work unit is (sequence, row tile, key/value head) and a unit's
// cost is its number of token tiles. One CTA per SM takes an equal, contiguous share of
// all token tiles of the launch (the schedule follows from the lengths, which are read on
// the device: every CTA sums the tile counts of the batch). A unit that spans CTAs leaves
// one partial result (running maximum, sum, unnormalised output, fp32) per CTA in the
// workspace, and the last CTA to finish joins them in CTA order: the result does not
// depend on which one that is. A CTA has at most two partial pieces, one at each end of
// its share, so the workspace does not grow with the lengths.
//
// Within a CTA the warps form WM row groups of 16 by WN token groups; a warp runs its own
// online softmax over its tokens (scores and probabilities never leave registers) and the
// token groups are joined once per unit. Tiles arrive through a ring of shared-memory
// stages filled by 16-byte asynchronous copies, each token row addressed through the page
// table, so any page size works, and rows past the sequence are filled with zeros: what
// the pool holds there (NaN included) is never used. The ring runs across units.
//
// Bound by HBM for few query rows: 2 G n flop for each byte of a bf16 cache (8 query heads
// per key/value head, one token: 8 flop per byte).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "gdn_attn.h"
#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Geometry: D head size, WM x WN warps, KS 16-token steps of a warp per tile.
template <int D, bool FP8, int WM>
struct Geo {
    static constexpr int ESZ = FP8 ? 1 : 2;
    static constexpr int WARPS = D == 256 ? 4 : 8;
    static constexpr int WN = WARPS / WM;
    static constexpr int NT = WARPS * 32;
    static constexpr int BM = 16 * WM;
    // tokens per tile: the largest whose ring below keeps three stages
    static constexpr int BN = D == 256 ? (WM == 1 || FP8 ? 64 : 32) : (D == 128 && WM == 4 && !FP8 ? 64 : 128);
    static constexpr int KS = BN / (16 * WN);
    static constexpr int ROWB = D * ESZ;          // bytes of a token's key (value)
    static constexpr int TILEB = BN * ROWB;       // bytes of a tile of keys (values)
    static constexpr int QB = BM * D * 2;         // bytes of a unit's queries
    static constexpr int STAGEB = 2 * TILEB;
    static constexpr int BUDGET = 218 * 1024;  // 227 KB less the schedule (8 KB) and row data
    static constexpr int FIT = BUDGET / (STAGEB + QB);
    static constexpr int STAGES = FIT > 6 ? 6 : FIT;
    static constexpr int JOIN = WARPS * 16 > 2 * BM ? WARPS * 16 : 2 * BM;  // maxima and sums
    static constexpr int CPR = ROWB / 16;         // 16-byte chunks of a token row
    static constexpr int ROWS_PER_PASS = NT / CPR;
    static_assert(STAGES >= 3 && KS >= 1 && BN % ROWS_PER_PASS == 0, "ring");
    // joining the token groups goes through the stage that has just been used
    static_assert(WN == 1 || (WN / 2) * BM * D * 4 <= STAGEB, "join scratch");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
    const int n = valid ? 16 : 0;  // 0: the 16 bytes are filled with zeros and nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// c += a b, 16x8x16, bf16 or fp16 operands (both the same), fp32 sums.
template <bool HALF>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (HALF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
            "%2, %3};\n"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, "
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
template <bool HALF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (HALF) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of 16-byte chunk c of token row r in a tile whose rows are CPR chunks: the
// chunks of eight consecutive rows fall into different bank groups for every c.
template <int CPR>
__device__ __forceinline__ int chunk_at(int r, int c) {
    if (CPR >= 8) return (r * CPR + (c ^ (r & 7))) * 16;
    const int line = r >> 1, pos = ((r & 1) * 4 + c) ^ (line & 7);  // two 64-byte rows a line
    return (line * 8 + pos) * 16;
}

// A sequence as the schedule sees it.
struct Seq {
    int n, first, past, slot;  // tokens of this call, their first row, tokens before them
    int lo, tiles;             // first position any row attends, token tiles from there
    int row_tiles;
};

template <int BM, int BN>
__device__ __forceinline__ Seq load_seq(const AttnArgs& p, int b, bool report) {
    Seq s;
    s.tiles = 0;
    s.row_tiles = 0;
    s.slot = __ldg(p.slots + b);
    s.first = b * p.T;
    s.n = p.T;
    if (p.cu) {
        s.first = __ldg(p.cu + b);
        s.n = __ldg(p.cu + b + 1) - s.first;
    }
    s.past = 0;
    s.lo = 0;
    if (s.n < 0 || s.n > p.T || s.first < 0 || s.first > p.total - s.n) {
        if (report && p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_SEQLEN_BIT);
        s.n = 0;
        return s;
    }
    if (s.n == 0) return s;
    if (s.slot < 0 || s.slot >= p.c.rows) {
        if (report && p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_SLOT_RANGE_BIT);
        return s;
    }
    s.past = __ldg(p.c.seq_lens + s.slot);
    if (s.past < 0 || s.past > p.c.max_pages * p.sh.page_size - s.n) {
        if (report && p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_SEQLEN_BIT);
        return s;
    }
    if (p.sh.window > 0 && s.past + 1 > p.sh.window) s.lo = s.past + 1 - p.sh.window;
    s.tiles = (s.past + s.n - s.lo + BN - 1) / BN;
    s.row_tiles = (s.n * p.sh.G + BM - 1) / BM;
    return s;
}

// One CTA's place in its share: the sequence, the unit within it and the tile within that.
struct Cursor {
    Seq s;
    int b, unit, tile;  // unit = row_tile * Hkv + kv head
};

template <int D, bool FP8, int WM>
__global__ void __launch_bounds__(Geo<D, FP8, WM>::NT, 1) attn_decode_kernel(const __grid_constant__ AttnArgs p) {
    using Gm = Geo<D, FP8, WM>;
    constexpr int BM = Gm::BM, BN = Gm::BN, WN = Gm::WN, KS = Gm::KS, NT = Gm::NT, CPR = Gm::CPR;
    constexpr int STAGES = Gm::STAGES, TILEB = Gm::TILEB, QB = Gm::QB, ND = D / 8;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* stages = smem;
    unsigned char* qbuf = smem + STAGES * Gm::STAGEB;
    float* qexp = reinterpret_cast<float*>(qbuf + STAGES * QB);  // [BM] power of two taken out of a query row (e4m3)
    float* join = qexp + BM;                                     // [JOIN] maximum and sum of joined groups
    int* misc = reinterpret_cast<int*>(join + Gm::JOIN);   // [40] scan scratch and broadcast
    int* prefix = misc + 40;                                     // [B + 1] tiles before each sequence
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wm = warp % WM, wn = warp / WM;
    const int g = lane >> 2, j = lane & 3;
    const int Hkv = p.sh.Hkv, G = p.sh.G, ps = p.sh.page_size;

    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

    // ---- the schedule: tiles of every sequence, summed ----
    int total = 0;
    for (int base = 0; base < p.B; base += NT) {
        const int b = base + tid;
        int t = 0;
        if (b < p.B) {
            const Seq s = load_seq<BM, BN>(p, b, blockIdx.x == 0);
            t = s.tiles * s.row_tiles * Hkv;
        }
        int x = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) misc[warp] = x;
        __syncthreads();
        int before = total, sum = 0;
#pragma unroll
        for (int w = 0; w < Gm::WARPS; ++w) {
            if (w < warp) before += misc[w];
            sum += misc[w];
        }
        if (b < p.B) prefix[b] = before + x - t;
        total += sum;
        __syncthreads();
    }
    if (tid == 0) prefix[p.B] = total;
    __syncthreads();
    const int ctas = total < (int)gridDim.x ? total : (int)gridDim.x;
    if ((int)blockIdx.x >= ctas) return;
    const int share_lo = (int)((long)blockIdx.x * total / ctas);
    const int share_n = (int)((long)(blockIdx.x + 1) * total / ctas) - share_lo;

    // the sequence, unit and tile of the share's first tile
    auto seek = [&](Cursor& c) {
        int lo = 0, hi = p.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= share_lo) lo = mid; else hi = mid;
        }
        c.b = lo;  // the last sequence that starts at or before: it has tiles, as those that do not are empty ranges
        c.s = load_seq<BM, BN>(p, lo, false);
        const int off = share_lo - prefix[lo];
        c.unit = off / c.s.tiles;
        c.tile = off - c.unit * c.s.tiles;
    };
    // one tile on; loads the next sequence's data when the unit was the sequence's last
    auto advance = [&](Cursor& c) {
        if (++c.tile < c.s.tiles) return;
        c.tile = 0;
        if (++c.unit < c.s.row_tiles * Hkv) return;
        c.unit = 0;
        do {
            ++c.b;
        } while (prefix[c.b + 1] == prefix[c.b]);
        c.s = load_seq<BM, BN>(p, c.b, false);
    };

    // ---- the ring ----
    const int chunk = tid % CPR, row0 = tid / CPR;
    const size_t token_stride = (size_t)Hkv * Gm::ROWB;
    Cursor ld, cm;
    seek(ld);
    cm = ld;
    int ld_left = share_n, ld_stage = 0, ld_slot = 0;
    bool ld_first = true;
    int tok[BN / 32];  // this lane's token numbers (page * page_size + offset) of the tile to load, -1: none
    auto find_tokens = [&]() {
#pragma unroll
        for (int i = 0; i < BN / 32; ++i) {
            const int pos = ld.s.lo + ld.tile * BN + i * 32 + lane;
            int t = -1;
            if (pos < ld.s.past + ld.s.n) {
                const int pg = pos / ps;
                const int page = __ldg(p.c.table + (size_t)ld.s.slot * p.c.max_pages + pg);
                if (page >= 0 && page < p.c.num_pages) t = page * ps + (pos - pg * ps);
                else if (p.err_flag && ld.unit == 0) atomicOr(p.err_flag, GDN_DEVICE_ERR_PAGE_BIT);
            }
            tok[i] = t;
        }
    };
    // issues the copies of the next tile (and of its unit's queries, when it is the first
    // of them here), then looks up the pages of the one after it
    auto load_next = [&]() {
        if (ld_left > 0) {
            const int h = ld.unit % Hkv, rt = ld.unit / Hkv;
            const uint32_t st = smem_addr(stages + ld_stage * Gm::STAGEB);
            const unsigned char* kb = static_cast<const unsigned char*>(p.c.k) + (size_t)h * Gm::ROWB + chunk * 16;
            const unsigned char* vb = static_cast<const unsigned char*>(p.c.v) + (size_t)h * Gm::ROWB + chunk * 16;
#pragma unroll
            for (int i = 0; i < BN / Gm::ROWS_PER_PASS; ++i) {
                const int r = row0 + i * Gm::ROWS_PER_PASS;
                int t = -1;
#pragma unroll
                for (int u = 0; u < BN / 32; ++u) {
                    const int v = __shfl_sync(0xffffffffu, tok[u], r & 31);
                    if ((r >> 5) == u) t = v;
                }
                const size_t off = t < 0 ? 0 : (size_t)t * token_stride;
                const uint32_t at = st + chunk_at<CPR>(r, chunk);
                cp16(at, kb + off, t >= 0);
                cp16(at + TILEB, vb + off, t >= 0);
            }
            if (ld_first || ld.tile == 0) {
                // queries: row r is token r / G, query head h * G + r % G
                const uint32_t qs = smem_addr(qbuf + ld_slot * QB);
                const int rows = ld.s.n * G;
                for (int i = tid; i < BM * (D / 8); i += NT) {
                    const int r = i / (D / 8), c = i % (D / 8), rr = rt * BM + r;
                    const int t = rr / G;
                    const uint16_t* src = p.q.ptr;
                    if (rr < rows) src += (size_t)(ld.s.first + t) * p.q.row + (size_t)(h * G + rr - t * G) * p.q.head + c * 8;
                    cp16(qs + (r * (D / 8) + (c ^ (r & 7))) * 16, src, rr < rows);
                }
                ld_slot = ld_slot + 1 == STAGES ? 0 : ld_slot + 1;
                ld_first = false;
            }
            ld_stage = ld_stage + 1 == STAGES ? 0 : ld_stage + 1;
            if (--ld_left > 0) {
                advance(ld);
                find_tokens();
            }
        }
        cp_commit();
    };
    find_tokens();
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) load_next();

    // ---- the share ----
    float O[ND][4];
    float m[2], l[2];  // rows g and g + 8: running maximum (log2 units) and sum
    const bool capped = p.sh.softcap > 0.0f;
    const float qk_scale = p.sh.sm_scale * p.sh.k_scale;
    const float to_log2 = capped ? p.sh.softcap * kLog2e : qk_scale * kLog2e;  // after the cap, or at once
    const float cap_in = capped ? 2.0f * kLog2e * qk_scale / p.sh.softcap : 0.0f;
    int stage = 0, slot = -1;
    bool first = true;
    for (int left = share_n; left > 0; --left) {
        const bool begin = first || cm.tile == 0;
        first = false;
        cp_wait<STAGES - 2>();
        __syncthreads();
        load_next();
        const int h = cm.unit % Hkv, rt = cm.unit / Hkv;
        if (begin) {
            slot = slot + 1 == STAGES ? 0 : slot + 1;
#pragma unroll
            for (int i = 0; i < ND; ++i) O[i][0] = O[i][1] = O[i][2] = O[i][3] = 0.0f;
            m[0] = m[1] = -INFINITY;
            l[0] = l[1] = 0.0f;
            if (FP8) {
                // e4m3 keys become fp16, so the queries do too: a power of two per row brings its
                // largest element to 2^14 .. 2^15, exact for every element above 2^-38 of that
                for (int r = warp; r < BM; r += Gm::WARPS) {
                    uint32_t* row = reinterpret_cast<uint32_t*>(qbuf + slot * QB + r * D * 2);
                    uint32_t w[D / 64];
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) {
                        w[i] = row[lane + 32 * i];
                        top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
                    }
                    top = __reduce_max_sync(0xffffffffu, top);
                    const int e = top == 0 || top >= 0x7f80u ? 0 : max((int)(top >> 7), 1) - 127 - 14;
                    const float up = ldexpf(1.0f, -e);
#pragma unroll
                    for (int i = 0; i < D / 64; ++i)
                        row[lane + 32 * i] = pack2<true>(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
                    if (lane == 0) qexp[r] = ldexpf(1.0f, e);
                }
                __syncthreads();
            }
        }
        const unsigned char* kt = stages + stage * Gm::STAGEB;
        const uint32_t ks = smem_addr(kt), vs = ks + TILEB, qs = smem_addr(qbuf + slot * QB);
        const int tok0 = wn * (KS * 16);  // this warp's tokens of the tile
        const int pos0 = cm.s.lo + cm.tile * BN + tok0;
        const int kv_len = cm.s.past + cm.s.n;

        // scores: two accumulators per 8 tokens (even and odd steps) keep the chain short
        float S[KS * 2][4];
#pragma unroll
        for (int i = 0; i < KS * 2; ++i) S[i][0] = S[i][1] = S[i][2] = S[i][3] = 0.0f;
        if (!FP8) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t a[4];
                const int qr = wm * 16 + (lane & 15), qc = kk * 2 + (lane >> 4);
                ldsm4(a, qs + (qr * (D / 8) + (qc ^ (qr & 7))) * 16);
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    uint32_t b[4];
                    const int r = tok0 + s * 16 + (lane & 7) + ((lane >> 4) << 3), c = kk * 2 + ((lane >> 3) & 1);
                    ldsm4(b, ks + chunk_at<CPR>(r, c));
                    mma<false>(S[2 * s], a, b[0], b[1]);
                    mma<false>(S[2 * s + 1], a, b[2], b[3]);
                }
            }
        } else {
            // a 16-byte chunk is 16 elements of the head: a lane's four bytes are elements 4j..4j+3,
            // taken as the operand's columns 2j, 2j+1, 2j+8, 2j+9; the queries are read to match
#pragma unroll
            for (int kk = 0; kk < D / 16; kk += 2) {
                uint32_t a[2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = (kk + u) * 2 + (j >> 1), r0 = wm * 16 + g, r1 = r0 + 8;
                    const uint2 q0 = *reinterpret_cast<const uint2*>(qbuf + slot * QB + (r0 * (D / 8) + (c ^ (r0 & 7))) * 16 + (j & 1) * 8);
                    const uint2 q1 = *reinterpret_cast<const uint2*>(qbuf + slot * QB + (r1 * (D / 8) + (c ^ (r1 & 7))) * 16 + (j & 1) * 8);
                    a[u][0] = q0.x;
                    a[u][1] = q1.x;
                    a[u][2] = q0.y;
                    a[u][3] = q1.y;
                }
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    uint32_t b[4];  // tokens 0-7 and 8-15 of chunk kk, then of chunk kk + 1
                    const int r = tok0 + s * 16 + (lane & 15), c = kk + (lane >> 4);
                    ldsm4(b, ks + chunk_at<CPR>(r, c));
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        mma<true>(S[2 * s], a[u], e4m3_to_half2(b[2 * u], false), e4m3_to_half2(b[2 * u], true));
                        mma<true>(S[2 * s + 1], a[u], e4m3_to_half2(b[2 * u + 1], false), e4m3_to_half2(b[2 * u + 1], true));
                    }
                }
            }
        }

        // masks: row r attends positions row_lo .. row_hi-1
        const int r0 = rt * BM + wm * 16 + g, t0 = r0 / G, t1 = (r0 + 8) / G;
        const int hi0 = min(cm.s.past + t0 + 1, kv_len), hi1 = min(cm.s.past + t1 + 1, kv_len);
        const int lo0 = p.sh.window > 0 ? cm.s.past + t0 + 1 - p.sh.window : 0;
        const int lo1 = p.sh.window > 0 ? cm.s.past + t1 + 1 - p.sh.window : 0;
        float e0 = 1.0f, e1 = 1.0f;
        if (FP8) {
            e0 = qexp[wm * 16 + g];
            e1 = qexp[wm * 16 + g + 8];
        }
        // every row of the unit attends positions all_lo .. all_hi-1
        const int all_lo = p.sh.window > 0 ? max(0, cm.s.past + cm.s.n - p.sh.window) : 0, all_hi = cm.s.past + 1;
        const bool whole = pos0 >= all_lo && pos0 + KS * 16 <= all_hi;
        float mx0 = m[0], mx1 = m[1];
#pragma unroll
        for (int i = 0; i < KS * 2; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = S[i][e] * (e < 2 ? e0 : e1);
                if (capped) x = 1.0f - __fdividef(2.0f, 1.0f + exp2_fast(x * cap_in));  // tanh
                x *= to_log2;
                if (!whole) {
                    const int pos = pos0 + i * 8 + 2 * j + (e & 1);
                    const bool in = e < 2 ? pos < hi0 && pos >= lo0 : pos < hi1 && pos >= lo1;
                    x = in ? x : -INFINITY;
                }
                S[i][e] = x;
                if (e < 2) mx0 = fmaxf(mx0, x); else mx1 = fmaxf(mx1, x);
            }
        }
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
        const float ref0 = mx0 == -INFINITY ? 0.0f : mx0, ref1 = mx1 == -INFINITY ? 0.0f : mx1;  // nothing seen yet
        if (__any_sync(0xffffffffu, mx0 != m[0] || mx1 != m[1])) {
            const float f0 = exp2_fast(m[0] - ref0), f1 = exp2_fast(m[1] - ref1);
            l[0] *= f0;
            l[1] *= f1;
#pragma unroll
            for (int i = 0; i < ND; ++i) {
                O[i][0] *= f0;
                O[i][1] *= f0;
                O[i][2] *= f1;
                O[i][3] *= f1;
            }
            m[0] = mx0;
            m[1] = mx1;
        }
#pragma unroll
        for (int i = 0; i < KS * 2; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                S[i][e] = exp2_fast(S[i][e] - (e < 2 ? ref0 : ref1));
                l[e >> 1] += S[i][e];
            }
        }

        // a tile that some rows may not see in full: a value that is not finite must not reach
        // the rows whose mask leaves it out (0 * inf), so such tiles go token by token
        bool plain = true;
        if (!whole) {
            bool bad = false;
            for (int i = lane; i < KS * 16 * CPR; i += 32) {
                const int r = tok0 + i / CPR;
                const uint4 w = *reinterpret_cast<const uint4*>(kt + TILEB + chunk_at<CPR>(r, i % CPR));
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (FP8) {
                        const uint32_t t = u[q] & 0x7f7f7f7fu;  // e4m3: only 0x7f is not finite
                        bad |= ((t + 0x01010101u) & 0x80808080u) != 0;
                    } else {
                        bad |= (u[q] & 0x7f80u) == 0x7f80u || (u[q] & 0x7f800000u) == 0x7f800000u;
                    }
                }
            }
            plain = !__any_sync(0xffffffffu, bad);
        }
        if (plain) {
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const uint32_t a[4] = {pack2<FP8>(S[2 * s][0], S[2 * s][1]), pack2<FP8>(S[2 * s][2], S[2 * s][3]),
                                       pack2<FP8>(S[2 * s + 1][0], S[2 * s + 1][1]), pack2<FP8>(S[2 * s + 1][2], S[2 * s + 1][3])};
                const int r = tok0 + s * 16 + (lane & 15);
                if (!FP8) {
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t b[4];
                        ldsm4t(b, vs + chunk_at<CPR>(r, c * 2 + (lane >> 4)));
                        mma<false>(O[2 * c], a, b[0], b[1]);
                        mma<false>(O[2 * c + 1], a, b[2], b[3]);
                    }
                } else {
                    // a transposed pair of bytes is columns 2n, 2n+1 of one token: tile 2c takes the
                    // even columns of chunk c, tile 2c + 1 the odd ones
#pragma unroll
                    for (int c = 0; c < D / 16; c += 2) {
                        uint32_t b[4];
                        ldsm4t(b, vs + chunk_at<CPR>(r, c + (lane >> 4)));
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const uint32_t x0 = e4m3_to_half2(b[2 * u], false), y0 = e4m3_to_half2(b[2 * u], true);
                            const uint32_t x1 = e4m3_to_half2(b[2 * u + 1], false), y1 = e4m3_to_half2(b[2 * u + 1], true);
                            mma<true>(O[2 * (c + u)], a, __byte_perm(x0, y0, 0x5410), __byte_perm(x1, y1, 0x5410));
                            mma<true>(O[2 * (c + u) + 1], a, __byte_perm(x0, y0, 0x7632), __byte_perm(x1, y1, 0x7632));
                        }
                    }
                }
            }
        } else {
            for (int t = 0; t < KS * 16; ++t) {
                float p0 = 0.0f, p1 = 0.0f;
#pragma unroll
                for (int i = 0; i < KS * 2; ++i) {
                    if (i == (t >> 3)) {
                        p0 = (t & 1) ? S[i][1] : S[i][0];
                        p1 = (t & 1) ? S[i][3] : S[i][2];
                    }
                }
                p0 = __shfl_sync(0xffffffffu, p0, (lane & ~3) | ((t >> 1) & 3));
                p1 = __shfl_sync(0xffffffffu, p1, (lane & ~3) | ((t >> 1) & 3));
                const int pos = pos0 + t;
                const bool in0 = pos < hi0 && pos >= lo0, in1 = pos < hi1 && pos >= lo1;
#pragma unroll
                for (int i = 0; i < ND; ++i) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v;
                        if (!FP8) {
                            const int col = i * 8 + 2 * j + e;
                            v = bf16_bits_to_float(*reinterpret_cast<const uint16_t*>(kt + TILEB + chunk_at<CPR>(tok0 + t, col >> 3) + (col & 7) * 2));
                        } else {
                            const int col = (i >> 1) * 16 + 4 * j + 2 * e + (i & 1);
                            const uint32_t w = *(kt + TILEB + chunk_at<CPR>(tok0 + t, col >> 4) + (col & 15));
                            const uint32_t hh = e4m3_to_half2(w, false);
                            v = __low2float(*reinterpret_cast<const __half2*>(&hh));
                        }
                        if (in0) O[i][e] = fmaf(p0, v, O[i][e]);
                        if (in1) O[i][e + 2] = fmaf(p1, v, O[i][e + 2]);
                    }
                }
            }
        }

        const bool unit_done = cm.tile + 1 == cm.s.tiles || left == 1;
        if (unit_done) {
            // sums over the four lanes of a row, then over the token groups
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            }
            float* scratch = reinterpret_cast<float*>(stages + stage * Gm::STAGEB);
#pragma unroll
            for (int half = WN / 2; half >= 1; half >>= 1) {
                __syncthreads();
                const int to = (wn - half) * WM + wm;  // place of an upper warp's data
                if (wn >= half && wn < 2 * half) {
                    float4* d = reinterpret_cast<float4*>(scratch) + (size_t)to * ND * 32 + lane;
#pragma unroll
                    for (int i = 0; i < ND; ++i) d[i * 32] = make_float4(O[i][0], O[i][1], O[i][2], O[i][3]);
                    if (j == 0) {
                        join[to * 32 + g] = m[0];
                        join[to * 32 + g + 8] = m[1];
                        join[to * 32 + 16 + g] = l[0];
                        join[to * 32 + 24 + g] = l[1];
                    }
                }
                __syncthreads();
                if (wn < half) {
                    const int from = wn * WM + wm;
                    const float om0 = join[from * 32 + g], om1 = join[from * 32 + g + 8];
                    const float n0 = fmaxf(m[0], om0), n1 = fmaxf(m[1], om1);
                    const float z0 = n0 == -INFINITY ? 0.0f : n0, z1 = n1 == -INFINITY ? 0.0f : n1;
                    const float a0 = exp2_fast(m[0] - z0), a1 = exp2_fast(m[1] - z1);
                    const float b0 = exp2_fast(om0 - z0), b1 = exp2_fast(om1 - z1);
                    l[0] = l[0] * a0 + join[from * 32 + 16 + g] * b0;
                    l[1] = l[1] * a1 + join[from * 32 + 24 + g] * b1;
                    m[0] = n0;
                    m[1] = n1;
                    const float4* s = reinterpret_cast<const float4*>(scratch) + (size_t)from * ND * 32 + lane;
#pragma unroll
                    for (int i = 0; i < ND; ++i) {
                        const float4 o = s[i * 32];
                        O[i][0] = O[i][0] * a0 + o.x * b0;
                        O[i][1] = O[i][1] * a0 + o.y * b0;
                        O[i][2] = O[i][2] * a1 + o.z * b1;
                        O[i][3] = O[i][3] * a1 + o.w * b1;
                    }
                }
            }
            // whose piece of the unit this is
            const int unit_lo = prefix[cm.b] + cm.unit * cm.s.tiles, unit_hi = unit_lo + cm.s.tiles;
            const int c0 = (int)(((long)(unit_lo + 1) * ctas - 1) / total), c1 = (int)(((long)unit_hi * ctas - 1) / total);
            const int rows = min(BM, cm.s.n * G - rt * BM);
            auto finish = [&](int r, int col, float4 o, float mx, float sum) {  // four columns of row r, normalised
                const int rr = rt * BM + r, t = rr / G, head = h * G + rr - t * G;
                const size_t row = (size_t)cm.s.first + t;
                if (p.gate.ptr) {
                    const uint2 w = *reinterpret_cast<const uint2*>(p.gate.ptr + row * p.gate.row + (size_t)head * p.gate.head + col);
                    o.x *= sigmoid(__uint_as_float(w.x << 16));
                    o.y *= sigmoid(__uint_as_float(w.x & 0xffff0000u));
                    o.z *= sigmoid(__uint_as_float(w.y << 16));
                    o.w *= sigmoid(__uint_as_float(w.y & 0xffff0000u));
                }
                const size_t at = row * p.sh.Hq + head;
                *reinterpret_cast<uint2*>(p.out + at * D + col) = make_uint2(pack2<false>(o.x, o.y), pack2<false>(o.z, o.w));
                if (p.lse && col == 0) p.lse[at] = (mx + log2f(sum)) * kLn2;
            };
            // the unit's result (unnormalised) as rows of D floats, in the stage's memory or the workspace
            const bool split = c0 != c1;
            const int piece = split && (int)blockIdx.x != c0 && share_lo > unit_lo ? 0 : 1;
            constexpr int PSTRIDE = BM * (D + 2);
            // (a whole unit too large for the stage goes through the CTA's last piece: it is written
            // for good only at the end of the share)
            constexpr bool IN_STAGE = BM * D * 4 <= Gm::STAGEB;
            float* mine = split || !IN_STAGE ? p.partial + (size_t)(blockIdx.x * 2 + piece) * PSTRIDE : scratch;
            if (!split) __syncthreads();  // the join's reads of the stage are done
            if (wn == 0) {
#pragma unroll
                for (int i = 0; i < ND; ++i) {
                    const int col = FP8 ? 0 : i * 8 + 2 * j;
                    if (!FP8) {
                        const int a = wm * 16 + g;
                        if (a < rows) *reinterpret_cast<float2*>(mine + a * D + col) = make_float2(O[i][0], O[i][1]);
                        if (a + 8 < rows) *reinterpret_cast<float2*>(mine + (a + 8) * D + col) = make_float2(O[i][2], O[i][3]);
                    } else if ((i & 1) == 0) {
                        const int a = wm * 16 + g, c4 = (i >> 1) * 16 + 4 * j;
                        if (a < rows) *reinterpret_cast<float4*>(mine + a * D + c4) = make_float4(O[i][0], O[i + 1][0], O[i][1], O[i + 1][1]);
                        if (a + 8 < rows) *reinterpret_cast<float4*>(mine + (a + 8) * D + c4) = make_float4(O[i][2], O[i + 1][2], O[i][3], O[i + 1][3]);
                    }
                }
                if (j == 0) {
                    const int a = wm * 16 + g;
                    float* st = split ? mine + BM * D : join;
                    st[a] = m[0];
                    st[a + 8] = m[1];
                    st[BM + a] = l[0];
                    st[BM + a + 8] = l[1];
                }
            }
            if (!split) {
                __syncthreads();
                for (int i = tid; i < rows * (D / 4); i += NT) {
                    const int r = i / (D / 4), col = (i % (D / 4)) * 4;
                    const float inv = p.sh.v_scale / join[BM + r];
                    const float4 o = *reinterpret_cast<const float4*>(mine + r * D + col);
                    finish(r, col, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv), join[r], join[BM + r]);
                }
            } else {
                __threadfence();
                __syncthreads();
                if (tid == 0) misc[32] = atomicAdd(p.counters + c0, 1u) == (unsigned)(c1 - c0);
                __syncthreads();
                if (misc[32]) {
                    __threadfence();
                    auto part = [&](int c) {  // CTA c's piece of this unit
                        const long c_lo = (long)c * total / ctas;
                        return p.partial + (size_t)(c * 2 + (c != c0 && c_lo > unit_lo ? 0 : 1)) * PSTRIDE;
                    };
                    for (int i = tid; i < rows * (D / 4); i += NT) {
                        const int r = i / (D / 4), col = (i % (D / 4)) * 4;
                        float mx = -INFINITY;
                        for (int c = c0; c <= c1; ++c) mx = fmaxf(mx, __ldcg(part(c) + BM * D + r));
                        const float z = mx == -INFINITY ? 0.0f : mx;
                        float sum = 0.0f;
                        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                        for (int c = c0; c <= c1; ++c) {
                            const float* q = part(c);
                            const float w = exp2_fast(__ldcg(q + BM * D + r) - z);
                            const float4 x = __ldcg(reinterpret_cast<const float4*>(q + r * D + col));
                            sum = fmaf(w, __ldcg(q + BM * D + BM + r), sum);
                            o.x = fmaf(w, x.x, o.x);
                            o.y = fmaf(w, x.y, o.y);
                            o.z = fmaf(w, x.z, o.z);
                            o.w = fmaf(w, x.w, o.w);
                        }
                        const float inv = p.sh.v_scale / sum;
                        finish(r, col, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv), mx, sum);
                    }
                    if (tid == 0) p.counters[c0] = 0;
                }
            }
        }
        if (left > 1) advance(cm);
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    cp_wait<0>();
}

template <int D, bool FP8, int WM>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
    using Gm = Geo<D, FP8, WM>;
    auto kern = attn_decode_kernel<D, FP8, WM>;
    int dev, sms;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    const size_t smem = Gm::STAGES * (size_t)(Gm::STAGEB + Gm::QB) + (Gm::BM + Gm::JOIN) * 4 + 40 * 4 + ((size_t)a.B + 1) * 4;
    static std::once_flag once[kMaxDevices];
    std::call_once(once[dev], [&] {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms < kAttnMaxCtas ? sms : kAttnMaxCtas));
    cfg.blockDim = dim3(Gm::NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

// Row groups for `rows` query rows per key/value head.
int row_groups(int rows) { return rows <= 16 ? 1 : (rows <= 32 ? 2 : 4); }

// Calls f(integral_constant-like geometry) for the kernel that a shape selects.
template <typename F>
auto with_geometry(int d, bool fp8, int rows, F f) {
    const int wm = row_groups(rows);
#define GDN_PICK(D)                                                                     \
    if (fp8) return wm == 1 ? f(Geo<D, true, 1>{}) : wm == 2 ? f(Geo<D, true, 2>{}) : f(Geo<D, true, 4>{}); \
    return wm == 1 ? f(Geo<D, false, 1>{}) : wm == 2 ? f(Geo<D, false, 2>{}) : f(Geo<D, false, 4>{});
    switch (d) {
        case 64: GDN_PICK(64)
        case 128: GDN_PICK(128)
        default: GDN_PICK(256)
    }
#undef GDN_PICK
}

template <int D, bool FP8>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t stream) {
    switch (row_groups(a.T * a.sh.G)) {
        case 1: return launch<D, FP8, 1>(a, stream);
        case 2: return launch<D, FP8, 2>(a, stream);
        default: return launch<D, FP8, 4>(a, stream);
    }
}

}  // namespace

int attn_row_tile(int d, bool fp8, int rows) {
    return with_geometry(d, fp8, rows, [](auto g) { return decltype(g)::BM; });
}
int attn_token_tile(int d, bool fp8, int rows) {
    return with_geometry(d, fp8, rows, [](auto g) { return decltype(g)::BN; });
}
size_t attn_workspace_bytes(int d, bool fp8, int rows) {
    return kAttnMaxCtas * sizeof(unsigned int) + (size_t)kAttnMaxCtas * 2 * attn_row_tile(d, fp8, rows) * (d + 2) * sizeof(float);
}

cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t stream) {
    switch (a.sh.d) {
        case 64: return a.sh.fp8 ? launch_rows<64, true>(a, stream) : launch_rows<64, false>(a, stream);
        case 128: return a.sh.fp8 ? launch_rows<128, true>(a, stream) : launch_rows<128, false>(a, stream);
        case 256: return a.sh.fp8 ? launch_rows<256, true>(a, stream) : launch_rows<256, false>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
