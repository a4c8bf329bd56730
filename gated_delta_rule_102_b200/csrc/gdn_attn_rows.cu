// Attention of many query rows per key/value head (several new tokens of a sequence, as in
// the verification of a draft) over a paged bf16 cache, on the fifth-generation tensor
// cores: the same result, schedule and workspace as the kernel for few rows, which its
// matrix instructions hold back beyond 16 rows.
//
//   S = Q K^T;  P = exp2(c S - m);  O = P V
//
// A work unit has up to 128 query rows, the M of one tcgen05.mma; unused rows cost
// nothing but the products. Per tile of 64 tokens: S (128 x 64, fp32) accumulates in TMEM,
// twice, so that the next tile's scores are formed while this one's softmax runs; a thread
// owns a row (no shuffles); P goes to shared memory as bf16 and O (128 x d, fp32) stays in
// TMEM. O is rescaled only when a row's maximum has grown by more than 2^8 since the last
// time (P and the sums stay within range until then, and the quotient is the same).
// Warps: four of softmax, one issues the products, three load keys, values and queries by TMA.
// Units of several CTAs leave fp32 parts that a second launch joins over the whole GPU.
//
// Bound: a tile of 64 tokens at d = 256 is 64 KB of HBM, about 2700 cycles of an SM's share;
// its products take about 1000 and the softmax of 128 rows about 1900. Measured at 32 sequences of
// 1000 to 8000 tokens, 128 rows (234 MB): 77 us, 3.0 TB/s: 3300 cycles a tile while it runs, the
// rest the way to the first tile, the parts written (128 KB each) and the join. At d = 128 and 64
// the softmax is what a tile takes.
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "gdn_attn.h"
#include "gdn_attn_device.cuh"
#include "gdn_tcgen05.cuh"

namespace gdn {
namespace {

constexpr int kTile = 64, kRowTile = 128, kThreads = 256, kSoftmaxWarps = 4;
// Places of a unit beside its tiles' (4: 82 us where 32 sequences of 1000 to 8000 tokens check 16
// drafted ones, 8: 77), and of a CTA at least (8 sequences of 100 to 800 tokens, 8: 34 us, 3: 28).
constexpr int kCost = 8, kMinShare = 3;
// Growth of a row's maximum (log2) that makes it the new reference. Until then its largest probability is
// no power of two and is rounded to bf16 like the others (with the few-rows kernel it is exactly 1):
// outputs are off by 0.0021 of their size (rms; 4000 tokens, scores of variance 5), 0.0017 there and by
// their own rounding alone.
constexpr float kRescale = 8.0f;

template <int D>
struct RowsGeo {
    static constexpr int NB = D / 64;               // 128-byte blocks of a token's key
    static constexpr int TILEB = kTile * D * 2;     // bytes of a tile of keys (values)
    static constexpr int SLOTS = D == 256 ? 2 : (D == 128 ? 5 : 8);  // tiles of keys, and of values, in flight
    static constexpr int QB = kRowTile * D * 2, PB = kRowTile * kTile * 2;
    static constexpr int O_COL = 128;               // TMEM columns: S at 0 and 64, O from here
    static constexpr int FIXED = 1024;
    static constexpr size_t SMEM = QB + PB + 2 * SLOTS * TILEB + FIXED;
};

// Instruction descriptor of kind::f16: D fp32, A and B bf16, A K-major, B K-major or
// MN-major, M = 128, N = n.
constexpr uint32_t idesc_of(int n, int b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kRowTile >> 4) << 24);
}
// Shared-memory descriptor of a tile in 8-row by 128-byte atoms with the 128-byte swizzle.
// K-major: `stride` from one 8-row group to the next. MN-major: `lead` from one 64-element
// block to the next, `stride` from one group of 8 along K to the next.
__device__ __forceinline__ uint64_t atoms_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// LARGE: the scores' cap is above kPlainCap.
template <int D, bool LARGE>
__global__ void __launch_bounds__(kThreads, 1)
attn_rows_kernel(const __grid_constant__ AttnArgs p, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_q, const int box,
                 const int q_tokens) {
    using Gm = RowsGeo<D>;
    constexpr int NB = Gm::NB, TILEB = Gm::TILEB, SLOTS = Gm::SLOTS, CPR = D / 8;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* kring = smem;
    unsigned char* vring = kring + SLOTS * TILEB;
    unsigned char* qbuf = vring + SLOTS * TILEB;   // [NB blocks][128 rows][128 bytes], swizzled
    unsigned char* pbuf = qbuf + Gm::QB;           // [128 rows][128 bytes], swizzled
    uint64_t* kfull = reinterpret_cast<uint64_t*>(pbuf + Gm::PB);  // [SLOTS] each
    uint64_t* kempty = kfull + SLOTS;
    uint64_t* vfull = kempty + SLOTS;
    uint64_t* vempty = vfull + SLOTS;
    uint64_t* sfull = vempty + SLOTS;   // [2] scores formed
    uint64_t* sfree = sfull + 2;        // [2] scores read
    uint64_t* pready = sfree + 2;       // probabilities written (and O rescaled)
    uint64_t* pvdone = pready + 1;      // O complete up to a tile
    uint64_t* qfull = pvdone + 1;       // a unit's queries are there
    uint64_t* qfree = qfull + 1;        // its scores are all formed
    uint64_t* sbar = qfree + 1;         // the softmax warps' own barrier
    uint64_t* drain = sbar + 1;         // every product is complete
    int* misc = reinterpret_cast<int*>(drain + 1);  // [16] sums; 8, 9: tile skipped by the products; 10: TMEM; 15: stop
    int* prefix = misc + 16;                       // [B + 1]
    volatile int* stop = misc + 15;
    volatile int* skip = misc + 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hkv = p.sh.Hkv, G = p.sh.G;

    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(kfull + i, 1);
            mbar_init(kempty + i, 1);
            mbar_init(vfull + i, 1);
            mbar_init(vempty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sfull + i, 1);
            mbar_init(sfree + i, kSoftmaxWarps);
            skip[i] = 0;
        }
        mbar_init(pready, kSoftmaxWarps);
        mbar_init(pvdone, 1);
        mbar_init(qfull, 1);
        mbar_init(qfree, 1);
        mbar_init(sbar, kSoftmaxWarps);
        mbar_init(drain, 1);
        *stop = 0;
        mbar_init_fence();
        fence_proxy_async_smem();
    }
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

    // a unit's rows are whole tokens, so that a TMA box brings them
    const int row_tile = kRowTile / G * G, inv_g = 65536 / G + 1;  // r / G = r * inv_g >> 16 for r < 320, G <= 16
    Share<kTile, 0, kCost, kCost> at(p, row_tile, prefix);
    at.template sum_batch<kThreads>(prefix, misc);
    const bool any = at.begin(kMinShare);
    if (tid == 0) p.split[blockIdx.x].count = 0;  // no unit to join from here on, unless one is found
    if (!any) return;
    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&map_v)) : "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&map_q)) : "memory");
    }
    if (warp == 4) tmem_alloc(smem_addr(misc + 10), 512);
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(misc + 10);

    auto give_up = [&] { return *stop != 0; };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_wait_deadline(bar, parity, kWaitTimeoutCycles, give_up)) return true;
        if (*stop == 0) attn_abort(p.err_flag, stop);
        return false;
    };
    // the share's pieces in order: every role walks them by itself
    auto next_piece = [&](Piece& u) {
        const Seq c = at.s;
        const int rt = at.unit / Hkv, place = at.place, from = at.tile;
        u = Piece{c.n, c.first, c.past, c.lo, c.base, at.unit - rt * Hkv, rt, from, min(c.tiles - from, at.hi - place - from), 0,
                  at.cta_of(place), at.cta_of(place + c.tiles - 1)};
        // the CTA with the first piece of a unit that goes on tells the launch that joins them
        if (u.c0 != u.c1 && (int)blockIdx.x == u.c0 && tid == 0) p.split[blockIdx.x] = u;
        u.last = !at.next_unit();
        at.tile = 0;
    };

    if (warp == 5 || warp == 7) {
        // ================= loading: tile n's keys, or values =================
        // (a warp each: values are held until the softmax is done, keys are not, and neither waits for
        // the other's place)
        const bool v = warp == 7;
        uint64_t *full = v ? vfull : kfull, *empty = v ? vempty : kempty;
        unsigned char* ring = v ? vring : kring;
        const CUtensorMap* map = v ? &map_v : &map_k;
        const int x = lane * box < kTile ? lane : -1;  // this lane's part of a tile
        int n = 0;
        for (bool more = true; more; ++n) {
            const int st = n % SLOTS, turn = n / SLOTS, h = at.unit % Hkv;
            const int tok = x >= 0 ? at.look_up(at.s.base + at.tile * kTile + x * box, box) : -1;
            const unsigned bytes = __popc(__ballot_sync(0xffffffffu, tok >= 0)) * box * D * 2;
            if (turn > 0 && !wait(empty + st, (turn - 1) & 1)) break;
            if (lane == 0) mbar_arrive_expect_tx(full + st, bytes);
            __syncwarp();
            if (tok >= 0) tma_load_5d(smem_addr(ring + st * TILEB) + x * box * D * 2, map, tok >> 3, h, smem_addr(full + st));
            more = at.advance(1);
        }
        // what is still in flight lands before the block leaves (all of it has, unless a wait ran out)
        for (int i = max(0, n - SLOTS); i < n; ++i) mbar_wait_bounded(full + i % SLOTS, (i / SLOTS) & 1);
    } else if (warp == 4) {
        // ================= products: one thread =================
        if (lane == 0) {
            constexpr uint32_t qk = idesc_of(kTile, 0), pv = idesc_of(D, 1);
            const uint32_t q0 = smem_addr(qbuf), p0 = smem_addr(pbuf);
            bool ok = true, started = false;
            auto accumulate = [&](int n) {  // O += P V of tile n
                const int st = n % SLOTS;
                if (!wait(pready, n & 1) || !wait(vfull + st, (n / SLOTS) & 1)) return false;
                tcgen05_fence_after();
                if (!skip[n & 1]) {
                    const uint32_t v = smem_addr(vring + st * TILEB);
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        umma_bf16(tmem + Gm::O_COL, atoms_desc(p0 + k * 32, 16, 1024), atoms_desc(v + k * 2 * NB * 1024, 1024, NB * 1024), pv,
                                  started || k > 0);
                }
                skip[n & 1] = 0;
                started = true;
                umma_commit(smem_addr(vempty + st));
                umma_commit(smem_addr(pvdone));
                return true;
            };
            int n = 0;
            Piece u;
            u.last = 0;
            for (int ord = 0; ok && !u.last; ++ord) {
                next_piece(u);
                if (!(ok = wait(qfull, ord & 1))) break;
                started = false;
                for (int i = 0; i < u.count; ++i, ++n) {
                    const int st = n % SLOTS;
                    if (!(ok = wait(kfull + st, (n / SLOTS) & 1) && (n < 2 || wait(sfree + (n & 1), ((n >> 1) - 1) & 1)))) break;
                    tcgen05_fence_after();
                    const uint32_t k = smem_addr(kring + st * TILEB);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        umma_bf16(tmem + (n & 1) * kTile, atoms_desc(q0 + (kk / 4) * (kRowTile * 128) + (kk % 4) * 32, 16, 1024),
                                  atoms_desc(k + (kk / 4) * 1024 + (kk % 4) * 32, 16, NB * 1024), qk, kk > 0);
                    umma_commit(smem_addr(kempty + st));
                    umma_commit(smem_addr(sfull + (n & 1)));
                    if (i == u.count - 1) umma_commit(smem_addr(qfree));
                    if (i > 0 && !(ok = accumulate(n - 1))) break;
                }
                if (ok) ok = accumulate(n - 1);
            }
            // also where a wait ran out, here or in another role: nothing runs when the tensor memory goes back
            umma_commit(smem_addr(drain));
            mbar_wait_bounded(drain, 0);
        }
        __syncwarp();
    } else if (warp < kSoftmaxWarps) {
        // ================= softmax: thread = row =================
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        const bool capped = !LARGE && p.sh.softcap > 0.0f;
        const float to_log2 = capped ? p.sh.softcap * kLog2e : p.sh.sm_scale * kLog2e;
        const float factor = capped ? finite(2.0f * kLog2e * p.sh.sm_scale / p.sh.softcap) : to_log2;
        unsigned char* prow = pbuf + tid * 128;
        uint32_t sphase = 0;
        auto arrive = [&](uint64_t* bar) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        bool ok = true;
        int n = 0;
        Piece u;
        u.last = 0;
        for (int ord = 0; ok && !u.last; ++ord) {
            next_piece(u);
            const int rows = min(row_tile, u.n * G - u.rt * row_tile), kv_len = u.past + u.n;
            const int rr = u.rt * row_tile + tid, t = (rr * inv_g) >> 16, head = u.h * G + rr - t * G;
            if (p.gate.ptr && tid < rows) {  // the gates' lines into L2: they are read when the unit ends
                const uint16_t* line = p.gate.ptr + (size_t)(u.first + t) * p.gate.row + (size_t)head * p.gate.head;
#pragma unroll
                for (int i = 0; i < NB; ++i) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(line + i * 64));
            }
            const bool active = warp * 32 < rows;
            // this row attends positions lo .. hi-1; every row of the unit those from all_lo to all_hi
            const int hi = min(u.past + t + 1, kv_len), lo = p.sh.window > 0 ? u.past + t + 1 - p.sh.window : 0;
            const int all_lo = p.sh.window > 0 ? max(0, kv_len - p.sh.window) : 0, all_hi = u.past + 1;
            float ref = -INFINITY, sum = 0.0f;  // the row's reference (log2 units) and sum
            for (int i = 0; i < u.count; ++i, ++n) {
                const int pos0 = u.base + (u.tile + i) * kTile;
                const bool whole = pos0 >= all_lo && pos0 + kTile <= all_hi;
                if (!(ok = wait(sfull + (n & 1), (n >> 1) & 1))) break;
                tcgen05_fence_after();
                float x[kTile];
                if (active) {
                    tmem_ld32(lanes + (n & 1) * kTile, *reinterpret_cast<float(*)[32]>(x));
                    tmem_ld32(lanes + (n & 1) * kTile + 32, *reinterpret_cast<float(*)[32]>(x + 32));
                }
                tcgen05_fence_before();
                arrive(sfree + (n & 1));
                float top = -INFINITY;
                if (active) {
                    if (capped) {
#pragma unroll
                        for (int c = 0; c < kTile; ++c)  // c tanh(y) = c - 2 c / (1 + e^2y)
                            x[c] = fmaf(-2.0f * to_log2, rcp_fast(1.0f + exp2_fast(x[c] * factor)), to_log2);
                    } else {
#pragma unroll
                        for (int c = 0; c < kTile; ++c) x[c] *= factor;
                    }
                    if (LARGE) cap_large<kTile>(x, p.sh.softcap);
                    if (!whole) {
#pragma unroll
                        for (int c = 0; c < kTile; ++c) x[c] = pos0 + c < hi && pos0 + c >= lo ? x[c] : -INFINITY;
                    }
#pragma unroll
                    for (int c = 0; c < kTile; ++c) top = fmaxf(top, x[c]);
                }
                // the tile before is in O, and its probabilities are read
                if (i > 0 && !(ok = wait(pvdone, (n - 1) & 1))) break;
                if (active) {
                    const bool grow = i == 0 || top > ref + kRescale || ref == -INFINITY;
                    const float next = grow ? fmaxf(top, ref) : ref;
                    if (i > 0 && __any_sync(0xffffffffu, next != ref)) {
                        const float f = next == -INFINITY ? 1.0f : exp2_fast(ref - next);
                        sum *= f;
                        tcgen05_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            uint32_t z[32];
                            tmem_ld32(lanes + Gm::O_COL + c, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) z[e] = __float_as_uint(o[e] * f);
                            tmem_st32(lanes + Gm::O_COL + c, z);
                        }
                        tmem_wait_st();
                    }
                    ref = next;
                    const float from = ref == -INFINITY ? 0.0f : ref;  // nothing seen yet
#pragma unroll
                    for (int c = 0; c < kTile; c += 8) {
                        uint32_t z[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float a = exp2_fast(x[c + 2 * e] - from), b = exp2_fast(x[c + 2 * e + 1] - from);
                            sum += a + b;
                            z[e] = pack2<false>(a, b);
                        }
                        *reinterpret_cast<uint4*>(prow + ((((c >> 3) ^ tid) & 7) << 4)) = make_uint4(z[0], z[1], z[2], z[3]);
                    }
                }
                if (!whole) {
                    // Values outside the sequence become zeros. A value that is not finite must not reach
                    // the rows whose mask leaves it out (0 * inf): such a tile skips the products and goes
                    // token by token.
                    if (!(ok = wait(vfull + n % SLOTS, (n / SLOTS) & 1))) break;
                    unsigned char* vt = vring + (n % SLOTS) * TILEB;
                    bool bad = false;
                    for (int k = lane; k < 16 * CPR; k += 32) {
                        const int r = warp * 16 + k / CPR;
                        uint4* word = reinterpret_cast<uint4*>(vt + chunk_at<CPR>(r, k % CPR));
                        if (pos0 + r < u.lo || pos0 + r >= kv_len) {
                            *word = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        const uint4 w = *word;
                        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) bad |= (v[e] & 0x7f80u) == 0x7f80u || (v[e] & 0x7f800000u) == 0x7f800000u;
                    }
                    if (__any_sync(0xffffffffu, bad) && lane == 0) skip[n & 1] = 1;
                    arrive(sbar);
                    if (!(ok = wait(sbar, sphase))) break;
                    sphase ^= 1;
                    if (skip[n & 1] && active) {
                        tcgen05_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            uint32_t z[32];
                            if (i > 0) tmem_ld32(lanes + Gm::O_COL + c, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = i > 0 ? o[e] : 0.0f;
#pragma unroll 1
                            for (int k = 0; k < kTile; ++k) {
                                if (pos0 + k >= hi || pos0 + k < lo) continue;
                                const float f = bf16_bits_to_float(*reinterpret_cast<const uint16_t*>(prow + ((((k >> 3) ^ tid) & 7) << 4) + (k & 7) * 2));
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    o[e] = fmaf(f, bf16_bits_to_float(*reinterpret_cast<const uint16_t*>(vt + chunk_at<CPR>(k, (c + e) >> 3) + (e & 7) * 2)), o[e]);
                            }
                            __syncwarp();
#pragma unroll
                            for (int e = 0; e < 32; ++e) z[e] = __float_as_uint(o[e]);
                            tmem_st32(lanes + Gm::O_COL + c, z);
                        }
                        tmem_wait_st();
                    }
                }
                tcgen05_fence_before();
                fence_proxy_async_smem();
                arrive(pready);
            }
            if (!ok || !(ok = wait(pvdone, (n - 1) & 1))) break;
            tcgen05_fence_after();
            if (active) {
                float* mine = p.partial + (size_t)(blockIdx.x * 2 + ((int)blockIdx.x == u.c0)) * (kRowTile * (D + 2));
                const bool split = u.c0 != u.c1;
                const size_t row = (size_t)u.first + t;
                const float inv = 1.0f / sum;
                // a row's 32 columns through this warp's part of the probabilities' memory, so that
                // eight lanes write a row together
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint2 z[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int r = warp * 32 + e * 4 + (lane >> 3), qr = u.rt * row_tile + r, qt = (qr * inv_g) >> 16;
                        z[e] = make_uint2(0, 0);
                        if (!split && p.gate.ptr && r < rows) z[e] = gate_of4(p, (size_t)u.first + qt, u.h * G + qr - qt * G, c + (lane & 7) * 4);
                    }
                    float o[32];
                    tmem_ld32(lanes + Gm::O_COL + c, o);
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<float4*>(prow + (((e ^ tid) & 7) << 4)) = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int r = warp * 32 + e * 4 + (lane >> 3), q = lane & 7;
                        const float4 v = *reinterpret_cast<const float4*>(pbuf + r * 128 + (((q ^ r) & 7) << 4));
                        const float scale = __shfl_sync(0xffffffffu, inv, e * 4 + (lane >> 3));
                        if (r >= rows) continue;
                        if (split) {
                            *reinterpret_cast<float4*>(mine + r * D + c + q * 4) = v;
                        } else {
                            const int qr = u.rt * row_tile + r, qt = (qr * inv_g) >> 16;
                            write_out4<false>(p, (size_t)u.first + qt, u.h * G + qr - qt * G, D, c + q * 4, v, scale, z[e]);
                        }
                    }
                }
                if (tid < rows) {
                    if (split) {
                        mine[kRowTile * D + tid] = ref;
                        mine[kRowTile * D + kRowTile + tid] = sum;
                    } else if (p.lse) {
                        p.lse[row * p.sh.Hq + head] = log_sum<false>(ref, sum);
                    }
                }
            }
            tcgen05_fence_before();  // O is read before the next unit's products overwrite it (they wait for its queries)
        }
    } else if (warp == 6) {
        // ================= queries =================
        Piece u;
        u.last = 0;
        int ord = 0;
        for (; !u.last; ++ord) {
            next_piece(u);
            if (ord > 0 && !wait(qfree, (ord - 1) & 1)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(qfull, NB * G * q_tokens * 128);
                // q_tokens tokens of G heads, a 128-byte block at a time; what lies past the sequence's
                // tokens is other rows (or zeros), whose products touch no row of this unit
                for (int k = 0; k < NB; ++k) {
                    asm volatile(
                        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
                        "%3, %4, %5}], [%6];\n" ::"r"(smem_addr(qbuf + k * (kRowTile * 128))),
                        "l"(reinterpret_cast<uint64_t>(&map_q)), "r"(0), "r"(u.h * G), "r"(u.first + u.rt * (kRowTile / G)), "r"(k),
                        "r"(smem_addr(qfull))
                        : "memory");
                }
            }
            __syncwarp();
        }
        if (ord > 0) mbar_wait_bounded(qfull, (ord - 1) & 1);  // as for the tiles
    }
    // all roles are done (or have given up): the tensor memory goes back
    __syncthreads();
    if (warp == 4) {
        tcgen05_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------------
// The units that several CTAs share, joined by a launch of its own: a partial result is
// 128 KB here (128 rows of 256), and the last CTA of a unit alone took 25 us for its
// pieces while the others had nothing left to do; spread over all SMs, 16 rows of a unit
// a block, it is a few. Block (c, y): rows 16 y on of the unit whose first piece ends the
// share of CTA c.
constexpr int kJoinRows = 16;

template <int D>
__global__ void __launch_bounds__(kThreads) attn_rows_join_kernel(const __grid_constant__ AttnArgs p) {
    constexpr int PSTRIDE = kRowTile * (D + 2), WP = kAttnMaxCtas + 2;
    constexpr int ITEMS = kJoinRows * (D / 4) / kThreads;  // float4s of a thread
    __shared__ float wt[kJoinRows * WP];  // weights of a row's pieces, then their sum and maximum
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = p.sh.G;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const Piece u = p.split[blockIdx.x];
    if (u.count == 0) return;
    const int row_tile = kRowTile / G * G, rows = min(row_tile, u.n * G - u.rt * row_tile), base = blockIdx.y * kJoinRows;
    if (base >= rows) return;
    const int pieces = u.c1 - u.c0 + 1, inv_g = 65536 / G + 1;
    const float* first = p.partial + (size_t)(u.c0 * 2 + 1) * PSTRIDE;
    const float* rest = p.partial + (size_t)(u.c0 + 1) * 2 * PSTRIDE;
    auto part = [&](int i) { return i == 0 ? first : rest + (size_t)(i - 1) * (2 * PSTRIDE); };
    for (int r = warp; r < kJoinRows; r += kThreads / 32) {
        float* w = wt + r * WP;
        float top = -INFINITY, tot = 0.0f;
        for (int i = lane; i < pieces; i += 32) {
            w[i] = __ldcg(part(i) + kRowTile * D + base + r);
            top = fmaxf(top, w[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        for (int i = lane; i < pieces; i += 32) {
            w[i] = w[i] == -INFINITY ? 0.0f : exp2_fast(w[i] - top);
            tot = fmaf(w[i], __ldcg(part(i) + kRowTile * D + kRowTile + base + r), tot);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
        if (lane == 0) {
            w[kAttnMaxCtas] = tot;
            w[kAttnMaxCtas + 1] = top;
        }
    }
    float4 o[ITEMS];
    uint2 z[ITEMS];
#pragma unroll
    for (int y = 0; y < ITEMS; ++y) {
        const int k = tid + y * kThreads, rr = u.rt * row_tile + base + k / (D / 4), t = (rr * inv_g) >> 16;
        o[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        z[y] = make_uint2(0, 0);
        if (p.gate.ptr && base + k / (D / 4) < rows) z[y] = gate_of4(p, (size_t)u.first + t, u.h * G + rr - t * G, k % (D / 4) * 4);
    }
    __syncthreads();
    for (int i0 = 0; i0 < pieces; i0 += 4) {
        float4 x[4][ITEMS];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4* at = reinterpret_cast<const float4*>(part(min(i0 + i, pieces - 1)) + base * D);
#pragma unroll
            for (int y = 0; y < ITEMS; ++y) x[i][y] = __ldcg(at + tid + y * kThreads);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i0 + i >= pieces) break;
#pragma unroll
            for (int y = 0; y < ITEMS; ++y) {
                const float f = wt[(tid + y * kThreads) / (D / 4) * WP + i0 + i];
                if (f == 0.0f) continue;  // (a piece without a token for the row says nothing, whatever it holds)
                o[y].x = fmaf(f, x[i][y].x, o[y].x);
                o[y].y = fmaf(f, x[i][y].y, o[y].y);
                o[y].z = fmaf(f, x[i][y].z, o[y].z);
                o[y].w = fmaf(f, x[i][y].w, o[y].w);
            }
        }
    }
#pragma unroll
    for (int y = 0; y < ITEMS; ++y) {
        const int k = tid + y * kThreads, r = k / (D / 4), col = k % (D / 4) * 4;
        if (base + r >= rows) continue;
        const int rr = u.rt * row_tile + base + r, t = (rr * inv_g) >> 16, head = u.h * G + rr - t * G;
        const size_t row = (size_t)u.first + t;
        const float* w = wt + r * WP;
        write_out4<false>(p, row, head, D, col, o[y], 1.0f / w[kAttnMaxCtas], z[y]);
        if (p.lse && col == 0) p.lse[row * p.sh.Hq + head] = log_sum<false>(w[kAttnMaxCtas + 1], w[kAttnMaxCtas]);
    }
}

template <int D, bool LARGE>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
    using Gm = RowsGeo<D>;
    auto kern = attn_rows_kernel<D, LARGE>;
    static_assert((4 * Gm::SLOTS + 10) * 8 + 16 * 4 <= Gm::FIXED, "small data");
    static_assert(Gm::SMEM + (kAttnMaxBatch + 1) * 4 <= 227 * 1024, "shared memory");
    int dev, sms;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    static std::once_flag once[kMaxDevices];
    static cudaError_t set[kMaxDevices];
    std::call_once(once[dev], [&] {
        set[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    });
    if (set[dev] != cudaSuccess) return set[dev];
    int box = a.sh.page_size & -a.sh.page_size;
    if (box > kTile) box = kTile;
    CUtensorMap map_k{}, map_v{};
    if (!make_pool_map(&map_k, a.c.k, a, D * 2, box) || !make_pool_map(&map_v, a.c.v, a, D * 2, box)) return cudaErrorInvalidValue;
    // queries as [128-byte block][token][head][byte], in boxes of a unit's tokens by G heads
    const int q_tokens = a.T < kRowTile / a.sh.G ? a.T : kRowTile / a.sh.G;
    CUtensorMap map_q{};
    {
        // (a single row or head may come with a stride of 0, which no map takes and nothing uses)
        const cuuint64_t dims[4] = {64, (cuuint64_t)a.sh.Hq, (cuuint64_t)a.total, (cuuint64_t)Gm::NB};
        const cuuint64_t strides[3] = {(cuuint64_t)(a.q.head ? a.q.head * 2 : 16), (cuuint64_t)(a.q.row ? a.q.row * 2 : 16), 128};
        const cuuint32_t boxes[4] = {64, (cuuint32_t)a.sh.G, (cuuint32_t)q_tokens, 1};
        if (!encode_tensor_map(&map_q, false, 4, const_cast<uint16_t*>(a.q.ptr), dims, strides, boxes, 128, true)) return cudaErrorInvalidValue;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms < kAttnMaxCtas ? sms : kAttnMaxCtas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Gm::SMEM + ((size_t)a.B + 1) * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, kern, a, map_k, map_v, map_q, box, q_tokens)) != cudaSuccess) return e;
    cfg.gridDim.y = (unsigned)(((a.T * a.sh.G < kRowTile ? a.T * a.sh.G : kRowTile) + kJoinRows - 1) / kJoinRows);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attn_rows_join_kernel<D>, a);
}

}  // namespace

// The rows per key/value head from which this kernel is the faster one on long contexts. Its time
// hardly depends on them, the other kernel's does (two key/value heads, 64 sequences of 2000 to
// 8000 tokens, us, this | other): d = 256: 32 rows 133 | 171, 64 rows 137 | 317; d = 128: 32 rows
// 97 | 67, 64 rows 99 | 108; d = 64: 32 rows 82 | 48, 64 rows 82 | 78. (At 100 to 800 tokens, 8
// sequences, the other one is ahead by 3 to 12 us throughout; the host does not know the lengths.)
bool attn_rows_supported(int d, bool fp8, int page_size, int rows) {
    const int few = d == 256 ? 16 : (d == 128 ? 32 : 64);
    return !fp8 && page_size % 8 == 0 && rows > few;
}

long attn_rows_places(const AttnShape& sh, const PagedCache& c, int T) {
    static_assert(kCost < kAttnUnitPlaces, "places of a unit");
    return attn_places(sh, c, T, kTile, kRowTile / sh.G * sh.G);
}

cudaError_t launch_attn_rows(const AttnArgs& a, cudaStream_t stream) {
    const bool large = a.sh.softcap > kPlainCap;
    switch (a.sh.d) {
        case 64: return large ? launch<64, true>(a, stream) : launch<64, false>(a, stream);
        case 128: return large ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
        case 256: return large ? launch<256, true>(a, stream) : launch<256, false>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
