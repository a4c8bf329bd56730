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
// Within a CTA four warps load and eight compute. The ring holds slots of 16 KB, the keys
// and values of 16 KS tokens; each loading warp fills every fourth slot by itself with
// 16-byte asynchronous copies, each token row addressed through the page table (any page
// size works), looks up the pages of its next slot meanwhile, and the one that meets a
// unit's first slot also brings the unit's queries and its description. Rows past the
// sequence are filled with zeros: what the pool holds there (NaN included) is never used.
// The computing warps form WM row groups of 16 rows by 8 / WM token groups; a token group
// takes every (8 / WM)-th slot and runs its own online softmax on it (scores and
// probabilities never leave registers), so no warp waits for another one until a unit
// ends, where the groups are joined through shared memory. The ring runs across units.
//
// Bound by HBM for few query rows: 2 G n flop for each byte of a bf16 cache (8 query heads
// per key/value head, one token: 8 flop per byte). Every wait is bounded.
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

// Geometry: D head size, WM row groups of 16 query rows.
template <int D, bool FP8, int WM>
struct Geo {
    static constexpr int ROWB = D * (FP8 ? 1 : 2);  // bytes of a token's key (value)
    static constexpr int SLOTB = 16 * 1024;
    static constexpr int ST = SLOTB / 2 / ROWB;     // tokens of a slot
    static constexpr int KS = ST / 16;
    static constexpr int NG = 8 / WM;               // token groups
    static constexpr int BM = 16 * WM;
    static constexpr int QB = BM * D * 2;           // bytes of a unit's queries
    static constexpr int NQ = QB >= 32768 ? 2 : 3;  // units whose queries are held
    static constexpr int CPR = ROWB / 16;           // 16-byte chunks of a token row
    static constexpr int CH = 32;                   // columns of the output joined at a time
    static constexpr int JROW = CH + 8;             // floats of a joined row: eight rows, eight bank groups
    static constexpr int JOINB = 2 * 8 * 16 * JROW * 4;  // two buffers
    static constexpr int FIXED = 1024 + (2 * BM + 2 * 8 * 16) * 4;
    static constexpr int FIT = (227 * 1024 - (kAttnMaxBatch + 1) * 4 - FIXED - JOINB - NQ * QB) / SLOTB;
    static constexpr int SLOTS = FIT > 12 ? 12 : FIT;
    static_assert(SLOTS >= 6 && KS >= 1, "ring");
};
constexpr int kLoadWarps = 4, kComputeWarps = 8, kAttnThreads = (kLoadWarps + kComputeWarps) * 32;

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
    int lo, tiles;             // first position any row attends, slots of tokens from there
    int row_tiles;
};

template <int BM, int ST>
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
    s.tiles = (s.past + s.n - s.lo + ST - 1) / ST;
    s.row_tiles = (s.n * p.sh.G + BM - 1) / BM;
    return s;
}

// A unit as the loading warps describe it to the computing ones.
struct Unit {
    Seq s;
    int h, rt;         // key/value head, row tile
    int tile, count;   // this CTA's piece: its first slot and how many
    int lo;            // number of the unit's first slot in the launch
};

__device__ __forceinline__ int load_acquire(const int* at) {
    int v;
    asm volatile("ld.acquire.cta.shared::cta.b32 %0, [%1];\n" : "=r"(v) : "r"(smem_addr(at)) : "memory");
    return v;
}
__device__ __forceinline__ void add_release(int* at) {
    asm volatile("red.release.cta.shared::cta.add.u32 [%0], 1;\n" ::"r"(smem_addr(at)) : "memory");
}

// Raises the call's timeout flag and makes every role of the CTA leave at its next wait.
__device__ __noinline__ void attn_abort(int32_t* err_flag, volatile int* stop) {
    if (err_flag) atomicOr(err_flag, GDN_DEVICE_ERR_TIMEOUT_BIT);
    *stop = 1;
}

template <int D, bool FP8, int WM>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_decode_kernel(const __grid_constant__ AttnArgs p) {
    using Gm = Geo<D, FP8, WM>;
    constexpr int BM = Gm::BM, ST = Gm::ST, KS = Gm::KS, NG = Gm::NG, CPR = Gm::CPR, SLOTS = Gm::SLOTS, NQ = Gm::NQ;
    constexpr int QB = Gm::QB, HALF = Gm::SLOTB / 2, ND = D / 8, CH = Gm::CH, JROW = Gm::JROW;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* ring = smem;
    unsigned char* qbuf = ring + SLOTS * Gm::SLOTB;
    float* jbuf = reinterpret_cast<float*>(qbuf + NQ * QB);       // [2][8][16][JROW]
    float* jm = jbuf + Gm::JOINB / 4;                             // [8][16] maxima of the computing warps
    float* jl = jm + 8 * 16;                                      // [8][16] sums
    float* qexp = jl + 8 * 16;                                    // [NQ][BM] (e4m3) power of two taken out of a query row
    Unit* units = reinterpret_cast<Unit*>(qexp + NQ * BM);        // [NQ]
    uint64_t* full = reinterpret_cast<uint64_t*>(units + 4);      // [SLOTS]
    uint64_t* qfull = full + SLOTS;                               // [NQ]
    uint64_t* cbar = qfull + NQ;                                  // the computing warps' barrier
    // Releases are counted, not phased: a warp comes back to a place only every few turns, and
    // a barrier's phase parity cannot tell a turn from the one two before it.
    int* freed = reinterpret_cast<int*>(cbar + 1);                // [SLOTS] warps that are done with a slot, all turns
    int* qfreed = freed + SLOTS;                                  // [NQ] the same for a unit's queries
    int* misc = qfreed + NQ;                 // [16] sums of the schedule's warps, 14: last, 15: stop
    int* prefix = misc + 16;                                      // [B + 1] slots before each sequence
    volatile int* stop = misc + 15;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hkv = p.sh.Hkv, G = p.sh.G, ps = p.sh.page_size;

    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(full + i, 32);
            freed[i] = 0;
        }
        for (int i = 0; i < NQ; ++i) {
            mbar_init(qfull + i, FP8 ? 32 : 64);
            qfreed[i] = 0;
        }
        mbar_init(cbar, kComputeWarps);
        *stop = 0;
        mbar_init_fence();
    }
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

    // ---- the schedule: slots of every sequence, summed ----
    int total = 0;
    for (int base = 0; base < p.B; base += kAttnThreads) {
        const int b = base + tid;
        int t = 0;
        if (b < p.B) {
            const Seq s = load_seq<BM, ST>(p, b, blockIdx.x == 0);
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
        for (int w = 0; w < kAttnThreads / 32; ++w) {
            if (w < warp) before += misc[w];
            sum += misc[w];
        }
        if (b < p.B) prefix[b] = before + x - t;
        total += sum;
        __syncthreads();
    }
    if (tid == 0) prefix[p.B] = total;
    __syncthreads();
    // as many CTAs as there are SMs, but no fewer slots a CTA than token groups
    const int ctas = min((int)gridDim.x, (total + NG - 1) / NG);
    if ((int)blockIdx.x >= ctas) return;
    const int share_lo = (int)((long)blockIdx.x * total / ctas);
    const int share_n = (int)((long)(blockIdx.x + 1) * total / ctas) - share_lo;
    auto give_up = [&] { return *stop != 0; };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_wait_deadline(bar, parity, kWaitTimeoutCycles, give_up)) return true;
        if (*stop == 0) attn_abort(p.err_flag, stop);
        return false;
    };
    auto wait_count = [&](const int* at, int count) {
        if (load_acquire(at) >= count) return true;
        const uint64_t begin = clock64();
        for (uint32_t i = 1; load_acquire(at) < count; ++i) {
            if ((i & 15) != 0) continue;
            if (*stop != 0) return false;
            if ((uint64_t)clock64() - begin > kWaitTimeoutCycles) {
                attn_abort(p.err_flag, stop);
                return false;
            }
        }
        return true;
    };

    if (warp >= kComputeWarps) {
        // ================= loading =================
        if (D == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
        const int pw = warp - kComputeWarps;
        if (pw >= share_n) return;
        int b, unit, tile, ord = 0;
        {
            int lo = 0, hi = p.B;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (prefix[mid] <= share_lo) lo = mid; else hi = mid;
            }
            b = lo;  // the last sequence that starts at or before the share: it has slots
        }
        Seq s = load_seq<BM, ST>(p, b, false);
        {
            const int off = share_lo - prefix[b];
            unit = off / s.tiles;
            tile = off - unit * s.tiles;
        }
        // `by` slots on; counts the units passed
        auto advance = [&](int by) {
            tile += by;
            while (tile >= s.tiles) {
                tile -= s.tiles;
                ++ord;
                if (++unit < s.row_tiles * Hkv) continue;
                unit = 0;
                do {
                    ++b;
                } while (prefix[b + 1] == prefix[b]);
                s = load_seq<BM, ST>(p, b, false);
            }
        };
        int tok[(ST + 31) / 32];  // this lane's token numbers (page * page_size + offset) of the slot, -1: none
        auto find_tokens = [&] {
#pragma unroll
            for (int i = 0; i < (ST + 31) / 32; ++i) {
                const int r = i * 32 + lane, pos = s.lo + tile * ST + r;
                int t = -1;
                if (r < ST && pos < s.past + s.n) {
                    const int pg = pos / ps;
                    const int page = __ldg(p.c.table + (size_t)s.slot * p.c.max_pages + pg);
                    if (page >= 0 && page < p.c.num_pages) t = page * ps + (pos - pg * ps);
                    else if (p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_PAGE_BIT);
                }
                tok[i] = t;
            }
        };
        const size_t token_stride = (size_t)Hkv * Gm::ROWB;
        constexpr int RPP = 32 / CPR;  // token rows of one warp-wide copy
        const int chunk = lane % CPR, sub = lane / CPR;
        if (pw > 0) advance(pw);
        find_tokens();
        for (int i = pw; i < share_n; i += kLoadWarps) {
            const int h = unit % Hkv, rt = unit / Hkv;
            const int st = i % SLOTS, turn = i / SLOTS;
            if (i == 0 || tile == 0) {
                // the unit's queries: row r is token r / G, query head h * G + r % G
                const int qs = ord % NQ, qturn = ord / NQ;
                if (!wait_count(qfreed + qs, qturn * kComputeWarps)) break;
                if (lane == 0) {
                    Unit u;
                    u.s = s;
                    u.h = h;
                    u.rt = rt;
                    u.tile = tile;
                    u.count = min(s.tiles - tile, share_n - i);
                    u.lo = prefix[b] + unit * s.tiles;
                    units[qs] = u;
                }
                const int rows = s.n * G;
                unsigned char* q = qbuf + qs * QB;
                if (!FP8) {
                    for (int k = lane; k < BM * (D / 8); k += 32) {
                        const int r = k / (D / 8), c = k % (D / 8), rr = rt * BM + r, t = rr / G;
                        const uint16_t* src = p.q.ptr;
                        if (rr < rows) src += (size_t)(s.first + t) * p.q.row + (size_t)(h * G + rr - t * G) * p.q.head + c * 8;
                        cp16(smem_addr(q + (r * (D / 8) + (c ^ (r & 7))) * 16), src, rr < rows);
                    }
                    cp_async_arrive(qfull + qs);
                } else {
                    // e4m3 keys become fp16, so the queries do too: a power of two per row brings its
                    // largest element to 2^14 .. 2^15, exact for every element above 2^-38 of that
#pragma unroll 2
                    for (int r = 0; r < BM; ++r) {
                        const int rr = rt * BM + r, t = rr / G;
                        const uint32_t* src = reinterpret_cast<const uint32_t*>(
                            p.q.ptr + (size_t)(s.first + t) * p.q.row + (size_t)(h * G + rr - t * G) * p.q.head);
                        uint32_t w[D / 64], top = 0;
#pragma unroll
                        for (int k = 0; k < D / 64; ++k) {
                            w[k] = rr < rows ? __ldg(src + lane + 32 * k) : 0;
                            top = max(top, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
                        }
                        top = __reduce_max_sync(0xffffffffu, top);
                        const int e = top == 0 || top >= 0x7f80u ? 0 : max((int)(top >> 7), 1) - 127 - 14;
                        const float up = ldexpf(1.0f, -e);
#pragma unroll
                        for (int k = 0; k < D / 64; ++k) {
                            const int x = lane + 32 * k;  // pair of elements; four pairs a chunk
                            *reinterpret_cast<uint32_t*>(q + (r * (D / 8) + ((x >> 2) ^ (r & 7))) * 16 + (x & 3) * 4) =
                                pack2<true>(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xffff0000u) * up);
                        }
                        if (lane == 0) qexp[qs * BM + r] = ldexpf(1.0f, e);
                    }
                }
                mbar_arrive(qfull + qs);
            }
            if (!wait_count(freed + st, turn * WM)) break;
            const uint32_t at = smem_addr(ring + st * Gm::SLOTB);
            const unsigned char* kb = static_cast<const unsigned char*>(p.c.k) + (size_t)h * Gm::ROWB + chunk * 16;
            const unsigned char* vb = static_cast<const unsigned char*>(p.c.v) + (size_t)h * Gm::ROWB + chunk * 16;
#pragma unroll
            for (int k = 0; k < ST / RPP; ++k) {
                const int r = k * RPP + sub;
                const int t = __shfl_sync(0xffffffffu, tok[(k * RPP) / 32], r & 31);
                const size_t off = t < 0 ? 0 : (size_t)t * token_stride;
                const uint32_t to = at + chunk_at<CPR>(r, chunk);
                cp16(to, kb + off, t >= 0);
                cp16(to + HALF, vb + off, t >= 0);
            }
            cp_async_arrive(full + st);
            if (i + kLoadWarps < share_n) {
                advance(kLoadWarps);
                find_tokens();
            }
        }
        cp_commit();
        cp_wait<0>();
        return;
    }

    // ================= computing =================
    if (D == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;\n");
    const int wm = warp % WM, grp = warp / WM;
    const int g = lane >> 2, j = lane & 3;
    const bool capped = p.sh.softcap > 0.0f;
    const float qk_scale = p.sh.sm_scale * p.sh.k_scale;
    const float to_log2 = capped ? p.sh.softcap * kLog2e : qk_scale * kLog2e;  // after the cap, or at once
    const float cap_in = capped ? 2.0f * kLog2e * qk_scale / p.sh.softcap : 0.0f;
    uint32_t cphase = 0;
    // all computing warps; what they wrote to shared memory before is visible after it
    auto meet = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(cbar);
        const bool ok = wait(cbar, cphase);
        cphase ^= 1;
        return ok;
    };

    for (int done = 0, ord = 0; done < share_n; ++ord) {
        const int qs = ord % NQ;
        if (!wait(qfull + qs, (ord / NQ) & 1)) return;
        const Unit u = units[qs];
        const uint32_t qaddr = smem_addr(qbuf + qs * QB);
        const unsigned char* qrow = qbuf + qs * QB;
        const int kv_len = u.s.past + u.s.n;
        // row r attends positions lo .. hi-1; every row of the unit those from all_lo to all_hi
        const int r0 = u.rt * BM + wm * 16 + g, t0 = r0 / G, t1 = (r0 + 8) / G;
        const int hi0 = min(u.s.past + t0 + 1, kv_len), hi1 = min(u.s.past + t1 + 1, kv_len);
        const int lo0 = p.sh.window > 0 ? u.s.past + t0 + 1 - p.sh.window : 0;
        const int lo1 = p.sh.window > 0 ? u.s.past + t1 + 1 - p.sh.window : 0;
        const int all_lo = p.sh.window > 0 ? max(0, kv_len - p.sh.window) : 0, all_hi = u.s.past + 1;
        float e0 = 1.0f, e1 = 1.0f;
        if (FP8) {
            e0 = qexp[qs * BM + wm * 16 + g];
            e1 = qexp[qs * BM + wm * 16 + g + 8];
        }
        float O[ND][4];
#pragma unroll
        for (int i = 0; i < ND; ++i) O[i][0] = O[i][1] = O[i][2] = O[i][3] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};  // rows g, g + 8: maximum (log2 units), sum

        // this group's slots of the piece: those whose number in the share is grp modulo NG
        for (int i = (grp - done % NG + NG) % NG; i < u.count; i += NG) {
            const int n = done + i, st = n % SLOTS, turn = n / SLOTS;
            // the turn before is over (it may be another group's), so the parity is this turn's
            if (!wait_count(freed + st, turn * WM) || !wait(full + st, turn & 1)) return;
            const unsigned char* kt = ring + st * Gm::SLOTB;
            const uint32_t ks = smem_addr(kt), vs = ks + HALF;
            const int pos0 = u.s.lo + (u.tile + i) * ST;
            float S[KS * 2][4];
#pragma unroll
            for (int x = 0; x < KS * 2; ++x) S[x][0] = S[x][1] = S[x][2] = S[x][3] = 0.0f;
            if (!FP8) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t a[4];
                    const int qr = wm * 16 + (lane & 15), qc = kk * 2 + (lane >> 4);
                    ldsm4(a, qaddr + (qr * (D / 8) + (qc ^ (qr & 7))) * 16);
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        uint32_t b[4];
                        const int r = s * 16 + (lane & 7) + ((lane >> 4) << 3), c = kk * 2 + ((lane >> 3) & 1);
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
                    for (int x = 0; x < 2; ++x) {
                        const int c = (kk + x) * 2 + (j >> 1), ra = wm * 16 + g, rb = ra + 8;
                        const uint2 q0 = *reinterpret_cast<const uint2*>(qrow + (ra * (D / 8) + (c ^ (ra & 7))) * 16 + (j & 1) * 8);
                        const uint2 q1 = *reinterpret_cast<const uint2*>(qrow + (rb * (D / 8) + (c ^ (rb & 7))) * 16 + (j & 1) * 8);
                        a[x][0] = q0.x;
                        a[x][1] = q1.x;
                        a[x][2] = q0.y;
                        a[x][3] = q1.y;
                    }
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        uint32_t b[4];  // tokens 0-7 and 8-15 of chunk kk, then of chunk kk + 1
                        ldsm4(b, ks + chunk_at<CPR>(s * 16 + (lane & 15), kk + (lane >> 4)));
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            mma<true>(S[2 * s], a[x], e4m3_to_half2(b[2 * x], false), e4m3_to_half2(b[2 * x], true));
                            mma<true>(S[2 * s + 1], a[x], e4m3_to_half2(b[2 * x + 1], false), e4m3_to_half2(b[2 * x + 1], true));
                        }
                    }
                }
            }
            const bool whole = pos0 >= all_lo && pos0 + ST <= all_hi;
            float mx0 = m[0], mx1 = m[1];
#pragma unroll
            for (int x = 0; x < KS * 2; ++x) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float y = FP8 ? S[x][e] * (e < 2 ? e0 : e1) : S[x][e];
                    if (capped) y = 1.0f - __fdividef(2.0f, 1.0f + exp2_fast(y * cap_in));  // tanh
                    y *= to_log2;
                    if (!whole) {
                        const int pos = pos0 + x * 8 + 2 * j + (e & 1);
                        const bool in = e < 2 ? pos < hi0 && pos >= lo0 : pos < hi1 && pos >= lo1;
                        y = in ? y : -INFINITY;
                    }
                    S[x][e] = y;
                    if (e < 2) mx0 = fmaxf(mx0, y); else mx1 = fmaxf(mx1, y);
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
                for (int x = 0; x < ND; ++x) {
                    O[x][0] *= f0;
                    O[x][1] *= f0;
                    O[x][2] *= f1;
                    O[x][3] *= f1;
                }
                m[0] = mx0;
                m[1] = mx1;
            }
#pragma unroll
            for (int x = 0; x < KS * 2; ++x) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    S[x][e] = exp2_fast(S[x][e] - (e < 2 ? ref0 : ref1));
                    l[e >> 1] += S[x][e];
                }
            }

            // a slot that some rows may not see in full: a value that is not finite must not reach
            // the rows whose mask leaves it out (0 * inf), so such slots go token by token
            bool plain = true;
            if (!whole) {
                bool bad = false;
                for (int x = lane; x < ST * CPR; x += 32) {
                    const uint4 w = *reinterpret_cast<const uint4*>(kt + HALF + x * 16);
                    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (FP8) bad |= (((v[q] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;  // only 0x7f is not finite
                        else bad |= (v[q] & 0x7f80u) == 0x7f80u || (v[q] & 0x7f800000u) == 0x7f800000u;
                    }
                }
                plain = !__any_sync(0xffffffffu, bad);
            }
            if (plain) {
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const uint32_t a[4] = {pack2<FP8>(S[2 * s][0], S[2 * s][1]), pack2<FP8>(S[2 * s][2], S[2 * s][3]),
                                           pack2<FP8>(S[2 * s + 1][0], S[2 * s + 1][1]), pack2<FP8>(S[2 * s + 1][2], S[2 * s + 1][3])};
                    const int r = s * 16 + (lane & 15);
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
                            for (int x = 0; x < 2; ++x) {
                                const uint32_t x0 = e4m3_to_half2(b[2 * x], false), y0 = e4m3_to_half2(b[2 * x], true);
                                const uint32_t x1 = e4m3_to_half2(b[2 * x + 1], false), y1 = e4m3_to_half2(b[2 * x + 1], true);
                                mma<true>(O[2 * (c + x)], a, __byte_perm(x0, y0, 0x5410), __byte_perm(x1, y1, 0x5410));
                                mma<true>(O[2 * (c + x) + 1], a, __byte_perm(x0, y0, 0x7632), __byte_perm(x1, y1, 0x7632));
                            }
                        }
                    }
                }
            } else {
#pragma unroll 1
                for (int t = 0; t < ST; ++t) {
                    float p0 = 0.0f, p1 = 0.0f;
#pragma unroll
                    for (int x = 0; x < KS * 2; ++x) {
                        if (x == (t >> 3)) {
                            p0 = (t & 1) ? S[x][1] : S[x][0];
                            p1 = (t & 1) ? S[x][3] : S[x][2];
                        }
                    }
                    p0 = __shfl_sync(0xffffffffu, p0, (lane & ~3) | ((t >> 1) & 3));
                    p1 = __shfl_sync(0xffffffffu, p1, (lane & ~3) | ((t >> 1) & 3));
                    const int pos = pos0 + t;
                    const bool in0 = pos < hi0 && pos >= lo0, in1 = pos < hi1 && pos >= lo1;
#pragma unroll
                    for (int x = 0; x < ND; ++x) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float v;
                            if (!FP8) {
                                const int col = x * 8 + 2 * j + e;
                                v = bf16_bits_to_float(*reinterpret_cast<const uint16_t*>(kt + HALF + chunk_at<CPR>(t, col >> 3) + (col & 7) * 2));
                            } else {
                                const int col = (x >> 1) * 16 + 4 * j + 2 * e + (x & 1);
                                const uint32_t hh = e4m3_to_half2(*(kt + HALF + chunk_at<CPR>(t, col >> 4) + (col & 15)), false);
                                v = __low2float(*reinterpret_cast<const __half2*>(&hh));
                            }
                            if (in0) O[x][e] = fmaf(p0, v, O[x][e]);
                            if (in1) O[x][e + 2] = fmaf(p1, v, O[x][e + 2]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) add_release(freed + st);
        }
        done += u.count;
        __syncwarp();
        if (lane == 0) add_release(qfreed + qs);

        // ---- the piece's token groups joined: a common maximum, then CH columns at a time ----
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        }
        // (the last readers of jm and jl left their previous use at a later barrier than this one's arrival)
        if (j == 0) {
            jm[warp * 16 + g] = m[0];
            jm[warp * 16 + g + 8] = m[1];
            jl[warp * 16 + g] = l[0];
            jl[warp * 16 + g + 8] = l[1];
        }
        if (!meet()) return;
        auto top_of = [&](int w, int r) {  // row r of row group w
            float x = jm[w * 16 + r];
#pragma unroll
            for (int k = 1; k < NG; ++k) x = fmaxf(x, jm[(k * WM + w) * 16 + r]);
            return x;
        };
        {
            const float a = top_of(wm, g), b = top_of(wm, g + 8);
            const float f0 = m[0] == -INFINITY ? 0.0f : exp2_fast(m[0] - a), f1 = m[1] == -INFINITY ? 0.0f : exp2_fast(m[1] - b);
#pragma unroll
            for (int x = 0; x < ND; ++x) {
                O[x][0] *= f0;
                O[x][1] *= f0;
                O[x][2] *= f1;
                O[x][3] *= f1;
            }
        }
        const int unit_hi = u.lo + u.s.tiles;
        const int c0 = (int)(((long)(u.lo + 1) * ctas - 1) / total), c1 = (int)(((long)unit_hi * ctas - 1) / total);
        const bool split = c0 != c1;
        const int rows = min(BM, u.s.n * G - u.rt * BM);
        constexpr int PSTRIDE = BM * (D + 2);  // floats of a partial result: [BM][D], then maxima and sums
        float* mine = p.partial + (size_t)(blockIdx.x * 2 + (split && (int)blockIdx.x != c0 && share_lo > u.lo ? 0 : 1)) * PSTRIDE;
        auto gate_of = [&](int r, int col) -> uint2 {
            const int rr = u.rt * BM + r, t = rr / G, head = u.h * G + rr - t * G;
            return __ldg(reinterpret_cast<const uint2*>(p.gate.ptr + (size_t)(u.s.first + t) * p.gate.row + (size_t)head * p.gate.head + col));
        };
        auto finish = [&](int r, int col, float4 o, float mx, float sum, uint2 w) {  // four normalised columns of row r
            const int rr = u.rt * BM + r, t = rr / G, head = u.h * G + rr - t * G;
            const size_t at = (size_t)(u.s.first + t) * p.sh.Hq + head;
            if (p.gate.ptr) {
                o.x *= sigmoid(__uint_as_float(w.x << 16));
                o.y *= sigmoid(__uint_as_float(w.x & 0xffff0000u));
                o.z *= sigmoid(__uint_as_float(w.y << 16));
                o.w *= sigmoid(__uint_as_float(w.y & 0xffff0000u));
            }
            *reinterpret_cast<uint2*>(p.out + at * D + col) = make_uint2(pack2<false>(o.x, o.y), pack2<false>(o.z, o.w));
            if (p.lse && col == 0) p.lse[at] = (mx + log2f(sum)) * kLn2;
        };
        constexpr int ITEMS = BM * (CH / 4);          // float4 columns of a joined chunk
        constexpr int PER = (ITEMS + 255) / 256;      // of one thread
        float mx[PER], sum[PER];
        uint2 gt[PER];
#pragma unroll
        for (int x = 0; x < PER; ++x) {
            const int k = tid + x * 256, r = k / (CH / 4), col = (k % (CH / 4)) * 4;
            mx[x] = sum[x] = 0.0f;
            gt[x] = make_uint2(0, 0);
            if (k < ITEMS && r < rows) {
                const int w = r >> 4, rr = r & 15;
                mx[x] = top_of(w, rr);
#pragma unroll
                for (int q = 0; q < NG; ++q) {
                    const float mq = jm[(q * WM + w) * 16 + rr];
                    if (mq != -INFINITY) sum[x] += jl[(q * WM + w) * 16 + rr] * exp2_fast(mq - mx[x]);
                }
                if (!split && p.gate.ptr) gt[x] = gate_of(r, col);
                if (split && col == 0) {
                    mine[BM * D + r] = mx[x];
                    mine[BM * D + BM + r] = sum[x];
                }
            }
        }
#pragma unroll
        for (int c = 0; c < D / CH; ++c) {
            float* jb = jbuf + (c & 1) * (8 * 16 * JROW);
            float* to = jb + warp * 16 * JROW;
#pragma unroll
            for (int x = 0; x < CH / 8; ++x) {
                const int i = c * (CH / 8) + x;
                if (!FP8) {
                    *reinterpret_cast<float2*>(to + g * JROW + x * 8 + 2 * j) = make_float2(O[i][0], O[i][1]);
                    *reinterpret_cast<float2*>(to + (g + 8) * JROW + x * 8 + 2 * j) = make_float2(O[i][2], O[i][3]);
                } else if ((x & 1) == 0) {
                    *reinterpret_cast<float4*>(to + g * JROW + x * 8 + 4 * j) = make_float4(O[i][0], O[i + 1][0], O[i][1], O[i + 1][1]);
                    *reinterpret_cast<float4*>(to + (g + 8) * JROW + x * 8 + 4 * j) = make_float4(O[i][2], O[i + 1][2], O[i][3], O[i + 1][3]);
                }
            }
            if (!meet()) return;
#pragma unroll
            for (int x = 0; x < PER; ++x) {
                const int k = tid + x * 256, r = k / (CH / 4), col = (k % (CH / 4)) * 4;
                if (k >= ITEMS || r >= rows) continue;
                float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int q = 0; q < NG; ++q) {
                    const float4 v = *reinterpret_cast<const float4*>(jb + ((q * WM + (r >> 4)) * 16 + (r & 15)) * JROW + col);
                    o.x += v.x;
                    o.y += v.y;
                    o.z += v.z;
                    o.w += v.w;
                }
                if (split) {
                    *reinterpret_cast<float4*>(mine + r * D + c * CH + col) = o;
                } else {
                    const uint2 w = gt[x];
                    if (p.gate.ptr && c + 1 < D / CH) gt[x] = gate_of(r, (c + 1) * CH + col);
                    const float inv = p.sh.v_scale / sum[x];
                    finish(r, c * CH + col, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv), mx[x], sum[x], w);
                }
            }
        }
        if (!split) continue;

        // ---- a unit over several CTAs: the last of them to get here joins the pieces, in their order ----
        __threadfence();
        if (!meet()) return;
        if (tid == 0) misc[14] = atomicAdd(p.counters + c0, 1u) == (unsigned)(c1 - c0);
        if (!meet()) return;
        if (!misc[14]) continue;
        __threadfence();
        const int pieces = c1 - c0 + 1;
        auto part = [&](int i) {  // the i-th piece
            const int c = c0 + i;
            return p.partial + (size_t)(c * 2 + (i > 0 && (long)c * total / ctas > u.lo ? 0 : 1)) * PSTRIDE;
        };
        float* wt = jbuf;  // [16][kAttnMaxCtas] weights of the pieces, then their sum's inverse and the maximum
        static_assert(16 * (kAttnMaxCtas + 2) * 4 <= Gm::JOINB, "weights");
        for (int base = 0; base < rows; base += 16) {
            const int n = min(16, rows - base);
            if (!meet()) return;  // the weights' previous readers are done
            for (int r = warp; r < n; r += kComputeWarps) {
                float* w = wt + r * (kAttnMaxCtas + 2);
                float top = -INFINITY, tot = 0.0f;
                for (int i = lane; i < pieces; i += 32) {
                    w[i] = __ldcg(part(i) + BM * D + base + r);
                    top = fmaxf(top, w[i]);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                for (int i = lane; i < pieces; i += 32) {
                    w[i] = w[i] == -INFINITY ? 0.0f : exp2_fast(w[i] - top);
                    tot = fmaf(w[i], __ldcg(part(i) + BM * D + BM + base + r), tot);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
                if (lane == 0) {
                    w[kAttnMaxCtas] = tot;
                    w[kAttnMaxCtas + 1] = top;
                }
            }
            if (!meet()) return;
            for (int k = tid; k < n * (D / 4); k += 256) {
                const int r = k / (D / 4), col = (k % (D / 4)) * 4;
                const float* w = wt + r * (kAttnMaxCtas + 2);
                const uint2 gw = p.gate.ptr ? gate_of(base + r, col) : make_uint2(0, 0);
                float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 16
                for (int i = 0; i < pieces; ++i) {
                    const float4 x = __ldcg(reinterpret_cast<const float4*>(part(i) + (base + r) * D + col));
                    o.x = fmaf(w[i], x.x, o.x);
                    o.y = fmaf(w[i], x.y, o.y);
                    o.z = fmaf(w[i], x.z, o.z);
                    o.w = fmaf(w[i], x.w, o.w);
                }
                const float inv = p.sh.v_scale / w[kAttnMaxCtas];
                finish(base + r, col, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv), w[kAttnMaxCtas + 1], w[kAttnMaxCtas], gw);
            }
        }
        if (tid == 0) p.counters[c0] = 0;
        if (!meet()) return;
    }
}

template <int D, bool FP8, int WM>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
    using Gm = Geo<D, FP8, WM>;
    auto kern = attn_decode_kernel<D, FP8, WM>;
    int dev, sms;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    const size_t smem = Gm::SLOTS * (size_t)Gm::SLOTB + Gm::NQ * (size_t)Gm::QB + Gm::JOINB + Gm::FIXED + ((size_t)a.B + 1) * 4;
    static std::once_flag once[kMaxDevices];
    std::call_once(once[dev], [&] {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms < kAttnMaxCtas ? sms : kAttnMaxCtas));
    cfg.blockDim = dim3(kAttnThreads);
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
    return with_geometry(d, fp8, rows, [](auto g) { return decltype(g)::ST; });
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
