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
// one partial result (reference of its scores, sum, unnormalised output, fp32) per CTA in the
// workspace, and the last CTA to finish joins them in CTA order: the result does not
// depend on which one that is. A CTA has at most two partial pieces, one at each end of
// its share, so the workspace does not grow with the lengths.
//
// Within a CTA three warps load keys and values, one brings each unit's queries and its
// description, and eight compute. The ring holds slots of 16 KB, the keys and values of ST
// tokens; each loading warp fills every third slot by itself and looks up the pages of its
// next slot meanwhile. When the page size is a multiple of 8 a
// slot is a few TMA tiles (one for the keys and one for the values when a page holds whole
// slots); any other page size takes 16-byte asynchronous copies, row by row. Both write
// the same layout: atoms of 8 tokens by 128 bytes, 128-byte swizzle.
// The computing warps form WM row groups of 16 rows by CS column halves by NG token groups.
// A token group takes every NG-th slot of a unit and runs its own online softmax on it
// (scores and probabilities never leave registers), so no warp waits for another one until
// the unit ends, where the token groups are joined through shared memory; a short unit is
// one group's alone. (At head size 256 two warps compute the same scores and half of the
// output each: that halves the registers and the data to join, for 1.5 times the products.)
//
// Bound by HBM for few query rows: 2 G n flop for each byte of a bf16 cache (8 query heads
// per key/value head, one token: 16 flop per byte). Two key/value heads of 256 with 8 query heads
// each, bf16: 256 sequences of 500 to 16000 tokens 358 us (2351 MB, 6.56 TB/s), 64 of 200 to 12000
// 80 us (4.7 TB/s: 3 us until every CTA knows its share, 5 us of joins, CTAs that end unevenly),
// one of 262143 96 us, one of 509 12 us (all latency: lookups, a slot, two joins). An e4m3 cache
// moves half the bytes for the same conversions and products: 8 heads of 128, 64 sequences of 2000
// to 16000 tokens 170 us (5.2 TB/s), bound by the instructions that widen the keys and values.
// Every wait is bounded.
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "gdn_attn.h"
#include "gdn_attn_device.cuh"

namespace gdn {
namespace {

constexpr int kLoadWarps = 3, kComputeWarps = 8, kAttnThreads = (kLoadWarps + 1 + kComputeWarps) * 32;
constexpr int kLaunchRegs = 168;
// What a unit costs beside its slots, in slots: its queries, the join of the token groups, the
// output. Measured as a whole: with 4 for every unit 256 sequences of 500 to 16000 tokens take 383
// us, with 12 for the longer ones 360; a mix of many short ones takes 80 with 12 for all, 62 with
// 6 for the short ones.
constexpr int kShortCost = 6, kUnitCost = 12;
// A piece of so many slots or fewer is one token group's alone (4: one sequence of 509 tokens takes
// 14.5 us, 2: 12.6), and places of a CTA at least: fewer CTAs, and pieces to join, for little work
// (8: 12.6 us, 4: 11.7, 2: 15.8).
constexpr int kSingle = 2, kMinShare = 4;

// Geometry: D head size, WM row groups of 16 query rows (0: eight rows).
template <int D, bool FP8, int WM>
struct Geo {
    static constexpr int ROWB = D * (FP8 ? 1 : 2);  // bytes of a token's key (value)
    static constexpr int SLOTB = 16 * 1024, HALF = SLOTB / 2;
    static constexpr int ST = HALF / ROWB;          // tokens of a slot
    static constexpr int KU = ST >= 32 ? 2 : 1, SUB = KU * 16;  // tokens that a warp works on at a time
    static constexpr bool T8 = WM == 0;             // eight rows, transposed products
    static constexpr int CS = D == 256 && !T8 ? 2 : 1;     // column halves
    static constexpr int ND = T8 ? D / 16 : D / CS / 8;    // tiles of a warp's output (16 columns by 8 rows, or 8 by 16)
    static constexpr int READERS = T8 ? 1 : WM * CS;       // warps that read a slot
    static constexpr int NG = kComputeWarps / READERS;     // token groups
    static constexpr int BM = T8 ? 8 : 16 * WM;
    static constexpr int OUTP = 36;                 // (T8) floats of a row of 32 columns on the way out
    static constexpr int OUTB = T8 ? kComputeWarps * 8 * OUTP * 4 : 0;
    static constexpr int QP = D * 2 + 16;           // bytes from one query row to the next: eight rows, eight bank groups
    static constexpr int QB = BM * QP;
    static constexpr int NQ = WM == 4 ? 2 : (WM == 2 ? 3 : 6);  // units whose queries are held
    static constexpr int CPR = ROWB / 16;           // 16-byte chunks of a token row
    // The join of the token groups, so many columns of every group's output at a time, in rows that
    // spread a warp's stores over the banks.
    static constexpr int ROUNDS = ND > 8 ? ND / 8 : 1, RND = ND / ROUNDS;
    static constexpr int WCOLS = RND * (T8 ? 16 : 8), COLS = WCOLS * CS, JPITCH = COLS + (T8 ? 4 : (FP8 ? 16 : 8));
    static constexpr int JOINB = NG == 1 ? 0 : NG * BM * JPITCH * 4;
    static constexpr int FIXED = 4096;              // everything small (checked at the launch)
    static constexpr int FIT = (227 * 1024 - (kAttnMaxBatch + 1) * 4 - FIXED - JOINB - OUTB - NQ * QB) / SLOTB;
    static constexpr int SLOTS = FIT > 12 ? 12 : FIT;
    static_assert(SLOTS >= 8 && ST % SUB == 0 && NG >= 1, "ring");
};

template <int D, bool FP8, int WM>
__global__ void __launch_bounds__(kAttnThreads, 1)
attn_decode_kernel(const __grid_constant__ AttnArgs p, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const int box) {
    using Gm = Geo<D, FP8, WM>;
    constexpr int BM = Gm::BM, ST = Gm::ST, KU = Gm::KU, SUB = Gm::SUB, NG = Gm::NG, CS = Gm::CS, CPR = Gm::CPR, SLOTS = Gm::SLOTS;
    constexpr int NQ = Gm::NQ, QB = Gm::QB, QP = Gm::QP, HALF = Gm::HALF, ND = Gm::ND;
    constexpr bool T8 = Gm::T8;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* ring = smem;
    unsigned char* qbuf = ring + SLOTS * Gm::SLOTB;
    float* jbuf = reinterpret_cast<float*>(qbuf + NQ * QB);       // [NG][BM][JPITCH] outputs to be joined
    float* obuf = reinterpret_cast<float*>(qbuf + NQ * QB + Gm::JOINB);  // (T8) [8 warps][8][OUTP]
    float* jm = reinterpret_cast<float*>(qbuf + NQ * QB + Gm::JOINB + Gm::OUTB);  // [NG][2][BM] their references and sums
    float* qexp = jm + NG * 2 * BM;                                   // [NQ][BM] (e4m3) power of two taken out of a query row
    Piece* pieces = reinterpret_cast<Piece*>(qexp + NQ * BM);     // [NQ], then the share's first and last split ones
    uint64_t* full = reinterpret_cast<uint64_t*>(pieces + NQ + 2 + ((NQ + 2) & 1));  // [SLOTS]
    uint64_t* qfull = full + SLOTS;                               // [NQ]
    uint64_t* qraw = qfull + NQ;                                  // [NQ] (e4m3) the queries as they came
    uint64_t* cbar = qraw + NQ;                                   // the computing warps' barrier
    // Releases are counted, not phased: a warp comes back to a place only every few turns, and
    // a barrier's phase parity cannot tell a turn from the one two before it.
    uint64_t* rbar = cbar + 1;                                    // their reads of the last join
    int* freed = reinterpret_cast<int*>(rbar + 1);                // [SLOTS] warps that are done with a slot, all turns
    int* qfreed = freed + SLOTS;                                  // [NQ] the same for a unit's queries
    int* misc = qfreed + NQ;                                      // [16] sums of the schedule's warps; 12: last to arrive; 15: stop
    int* prefix = misc + 16;                                      // [B + 1] cost of the sequences before each
    volatile int* stop = misc + 15;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hkv = p.sh.Hkv, G = p.sh.G;

    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(full + i, box ? 1 : 32);
            freed[i] = 0;
        }
        for (int i = 0; i < NQ; ++i) {
            mbar_init(qfull + i, 1);
            mbar_init(qraw + i, 1);
            qfreed[i] = 0;
        }
        mbar_init(cbar, kComputeWarps);
        mbar_init(rbar, kComputeWarps);
        *stop = 0;
        if (box) {
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&map_v)) : "memory");
        }
        mbar_init_fence();
        fence_proxy_async_smem();
    }
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

    Share<ST, kSingle, kShortCost, kUnitCost> at(p, BM, prefix);
    at.template sum_batch<kAttnThreads>(prefix, misc);
    if (!at.begin(kMinShare)) return;

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

    // The block's registers (launched with kLaunchRegs a thread, which the launch checks) go to
    // the warps that need them: 4 warps * 88 + 8 * 208 = 12 * 168.
    if (warp >= kComputeWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;\n");

    if (warp == kComputeWarps + kLoadWarps) {
        // ================= queries =================
        // As many units' queries are on their way as there is room for; those of an e4m3 cache are
        // converted when they have come (one unit at a time, load and conversion, 96 sequences of up
        // to 16000 tokens took 62 us, so 60: its CTAs of many short units waited for queries).
        bool more_units = true;
        int sent = 0, converted = 0;
        const int inv_g = 65536 / G + 1;  // r / G = r * inv_g >> 16 for r < 320, G <= 16
        while (true) {
            const bool to_convert = FP8 && converted < sent;
            if (more_units && (!to_convert || __shfl_sync(0xffffffffu, load_acquire(qfreed + sent % NQ), 0) >= sent / NQ * kComputeWarps)) {
                const Seq c = at.s;
                const int rt = at.unit / Hkv, h = at.unit - rt * Hkv, place = at.place, from = at.tile;
                more_units = at.next_unit();  // before this one is described: it may be the last
                at.tile = 0;
                // the unit's queries: row r is token r / G, query head h * G + r % G; rows past the last
                // are left as they are (a row's products touch no other row)
                const int qs = sent % NQ, rows = min(BM, c.n * G - rt * BM);
                if (!wait_count(qfreed + qs, sent / NQ * kComputeWarps)) break;
                ++sent;
                unsigned char* q = qbuf + qs * QB;
                uint64_t* bar = (FP8 ? qraw : qfull) + qs;
                if (lane == 0) {
                    pieces[qs] = Piece{c.n, c.first, c.past, c.lo, c.base, h, rt, from, min(c.tiles - from, at.hi - place - from),
                                       !more_units, at.cta_of(place), at.cta_of(place + c.tiles - 1)};
                    mbar_arrive_expect_tx(bar, rows * D * 2);
                }
                __syncwarp();
                for (int r = lane; r < rows; r += 32) {
                    const int rr = rt * BM + r, t = (rr * inv_g) >> 16;
                    tma_load_1d(q + r * QP, p.q.ptr + (size_t)(c.first + t) * p.q.row + (size_t)(h * G + rr - t * G) * p.q.head, D * 2, bar);
                }
                if (p.gate.ptr) {  // the gates' lines into L2: they are read when the unit ends
                    for (int i = lane; i < rows * (D / 64); i += 32) {
                        const int r = i / (D / 64), rr = rt * BM + r, t = (rr * inv_g) >> 16;
                        const uint16_t* line = p.gate.ptr + (size_t)(c.first + t) * p.gate.row + (size_t)(h * G + rr - t * G) * p.gate.head;
                        asm volatile("prefetch.global.L2 [%0];\n" ::"l"(line + i % (D / 64) * 64));
                    }
                }
                continue;
            }
            if (!to_convert) break;
            // e4m3 keys become fp16, so the queries do too: a power of two per row brings its largest
            // element to 2^14 .. 2^15. Elements down to 2^-31 of that stay exact (eight bits above fp16's
            // smallest, 2^-24), smaller ones are off by 2^-39 of it at most.
            constexpr int LPR = D / 8, RPW = 32 / LPR;  // lanes a row, rows at a time
            const int qs = converted % NQ;
            if (!wait(qraw + qs, (converted / NQ) & 1)) break;
            const int rows = min(BM, pieces[qs].n * G - pieces[qs].rt * BM);
            unsigned char* q = qbuf + qs * QB;
#pragma unroll 1  // (unrolled by four, 256 short sequences take 69 us instead of 62: the instruction caches)
            for (int r0 = 0; r0 < rows; r0 += RPW) {
                const int r = r0 + lane / LPR, ch = lane % LPR;
                uint4* word = reinterpret_cast<uint4*>(q + r * QP + ch * 16);
                const uint4 in = r < rows ? *word : make_uint4(0, 0, 0, 0);
                const uint32_t v[4] = {in.x, in.y, in.z, in.w};
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) top = max(top, max(v[k] & 0x7fffu, (v[k] >> 16) & 0x7fffu));
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int e = top == 0 || top >= 0x7f80u ? 0 : max((int)(top >> 7), 1) - 127 - 14;
                // 2^-e: e is at most 113, and at least -140, where the exponent field ends
                const float up = __uint_as_float((uint32_t)(127 - max(e, -127)) << 23);
                uint32_t z[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) z[k] = pack2<true>(__uint_as_float(v[k] << 16) * up, __uint_as_float(v[k] & 0xffff0000u) * up);
                if (r < rows) {
                    *word = make_uint4(z[0], z[1], z[2], z[3]);
                    if (ch == 0) qexp[qs * BM + r] = 1.0f / up;
                }
            }
            fence_proxy_async_smem();  // before queries come to this place again
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull + qs);
            ++converted;
        }
        // What is in flight lands before the block leaves, which it may at any time now: a role whose wait
        // ran out does not wait for this one. What was read has landed (and its place may be turns ahead, where
        // the phase's parity says nothing any more).
        for (int i = FP8 ? converted : max(0, sent - NQ); i < sent; ++i) {
            auto was_read = [&] { return load_acquire(qfreed + i % NQ) >= (i / NQ + 1) * kComputeWarps; };
            if (!was_read()) mbar_wait_deadline((FP8 ? qraw : qfull) + i % NQ, (i / NQ) & 1, kWaitTimeoutCycles, was_read);
        }
        return;
    }

    if (warp >= kComputeWarps) {
        // ================= loading =================
        const int pw = warp - kComputeWarps;
        const size_t token_stride = (size_t)Hkv * Gm::ROWB;
        // With TMA, lane x (16 + x) fetches chunk x of the slot's keys (values), `box` tokens of
        // one page; otherwise a lane looks tokens up for everybody.
        constexpr int LOOK = (ST + 31) / 32;
        int tok[LOOK];  // token numbers (page * page_size + offset), -1: none
        auto find_tokens = [&] {
            const int pos0 = at.s.base + at.tile * ST;
            if (box) {
                const int x = lane & 15;
                tok[0] = x * box < ST ? at.look_up(pos0 + x * box, box) : -1;
            } else {
#pragma unroll
                for (int i = 0; i < LOOK; ++i) tok[i] = i * 32 + lane < ST ? at.look_up(pos0 + i * 32 + lane, 1) : -1;
            }
        };
        constexpr int RPP = 32 / CPR;  // token rows of one warp-wide copy
        const int chunk = lane % CPR, sub = lane / CPR;
        bool more_slots = pw == 0 || at.advance(pw);
        if (more_slots) find_tokens();
        int sent = -1;
        for (int i = pw; more_slots; i += kLoadWarps) {
            const int h = at.unit % Hkv, st = i % SLOTS, turn = i / SLOTS;
            if (!wait_count(freed + st, turn * Gm::READERS)) break;
            const uint32_t dst = smem_addr(ring + st * Gm::SLOTB);
            sent = i;
            if (box) {
                const unsigned got = __ballot_sync(0xffffffffu, tok[0] >= 0);
                if (lane == 0) mbar_arrive_expect_tx(full + st, __popc(got) * box * Gm::ROWB);
                __syncwarp();
                if (tok[0] >= 0)
                    tma_load_5d(dst + (lane >> 4) * HALF + (lane & 15) * box * Gm::ROWB, lane < 16 ? &map_k : &map_v, tok[0] >> 3, h,
                                smem_addr(full + st));
            } else {
                const unsigned char* kb = static_cast<const unsigned char*>(p.c.k) + (size_t)h * Gm::ROWB + chunk * 16;
                const unsigned char* vb = static_cast<const unsigned char*>(p.c.v) + (size_t)h * Gm::ROWB + chunk * 16;
#pragma unroll 1
                for (int k = 0; k < ST / RPP; k += 8) {
                    int t[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const int r = (k + x) * RPP;
                        int v = tok[0];
#pragma unroll
                        for (int y = 1; y < LOOK; ++y) v = (r >> 5) == y ? tok[y] : v;
                        t[x] = __shfl_sync(0xffffffffu, v, (r + sub) & 31);
                    }
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const size_t off = t[x] < 0 ? 0 : (size_t)t[x] * token_stride;
                        const uint32_t to = dst + chunk_at<CPR>((k + x) * RPP + sub, chunk);
                        cp16(to, kb + off, t[x] >= 0);
                        cp16(to + HALF, vb + off, t[x] >= 0);
                    }
                }
                cp_async_arrive(full + st);
            }
            more_slots = at.advance(kLoadWarps);
            if (more_slots) find_tokens();
        }
        cp_wait_all();
        if (box) {  // as above: a place's slot of the turn that has not been read, if this warp has filled it
#pragma unroll 1
            for (int st = 0; st < SLOTS; ++st) {
                const int turn = load_acquire(freed + st) / Gm::READERS, i = turn * SLOTS + st;
                auto was_read = [&] { return load_acquire(freed + st) >= (turn + 1) * Gm::READERS; };
                if (i <= sent && i % kLoadWarps == pw) mbar_wait_deadline(full + st, turn & 1, kWaitTimeoutCycles, was_read);
            }
        }
        return;
    }

    // ================= computing =================
    constexpr int WMX = T8 ? 1 : WM;
    const int wm = warp % WMX, cs = warp / WMX % CS, grp = warp / (WMX * CS);
    const int g = lane >> 2, j = lane & 3;
    // A lane's two query rows, and whose element e of an accumulator is: rows g and g + 8 of 16
    // (elements 0, 1 and 2, 3); or, transposed, rows 2j and 2j + 1 of 8 (even and odd elements).
    const int ra = T8 ? 2 * j : wm * 16 + g, rb = T8 ? ra + 1 : ra + 8;
    auto second = [](int e) { return T8 ? (e & 1) : (e >> 1); };
    // over the lanes that share rows
    constexpr int XOR0 = T8 ? 4 : 1, XOR1 = T8 ? 32 : 4;
    const bool capped = p.sh.softcap > 0.0f;
    const float qk_scale = p.sh.sm_scale * p.sh.k_scale;
    const bool large_cap = p.sh.softcap > kPlainCap;
    const float to_log2 = capped ? p.sh.softcap * kLog2e : 0.0f;
    const float score_in = capped && !large_cap ? 2.0f * kLog2e * qk_scale / p.sh.softcap : qk_scale * kLog2e;
    uint32_t cphase = 0;
    // all computing warps; what they wrote before is visible to them after it
    auto meet = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(cbar);
        const bool ok = wait(cbar, cphase);
        cphase ^= 1;
        return ok;
    };
    constexpr int PSTRIDE = BM * (D + 2);  // floats of a partial result: [BM][D], then maxima and sums
    bool split_first = false, split_last = false;

    bool last = false;
    for (int done = 0, ord = 0, joins = 0; !last; ++ord) {
        const int qs = ord % NQ;
        if (!wait(qfull + qs, (ord / NQ) & 1)) return;
        const Piece u = pieces[qs];
        last = u.last != 0;
        uint32_t qaddr = smem_addr(qbuf + qs * QB);
        after_wait(qaddr);
        const unsigned char* qrow = qbuf + qs * QB;
        const int kv_len = u.past + u.n;
        // row r attends positions lo .. hi-1; every row of the unit those from all_lo to all_hi
        const int t0 = (u.rt * BM + ra) / G, t1 = (u.rt * BM + rb) / G;
        const int hi0 = min(u.past + t0 + 1, kv_len), hi1 = min(u.past + t1 + 1, kv_len);
        const int lo0 = p.sh.window > 0 ? u.past + t0 + 1 - p.sh.window : 0;
        const int lo1 = p.sh.window > 0 ? u.past + t1 + 1 - p.sh.window : 0;
        const int all_lo = p.sh.window > 0 ? max(0, kv_len - p.sh.window) : 0, all_hi = u.past + 1;
        // what a product is multiplied by: to log2 units, or to twice the cap's argument
        float f0 = score_in, f1 = f0;
        if (FP8) {
            f0 *= qexp[qs * BM + ra];
            f1 *= qexp[qs * BM + rb];
        }
        if (capped) {
            f0 = finite(f0);
            f1 = finite(f1);
        }
        float O[ND][4];
#pragma unroll
        for (int i = 0; i < ND; ++i) O[i][0] = O[i][1] = O[i][2] = O[i][3] = 0.0f;
        // rows ra, rb: reference (log2 units: the maximum so far, or near it with an e4m3 cache), sum
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

        // this group's slots: all of a short piece, in turn with the other groups, or every NG-th
        const bool single = NG == 1 || u.count <= kSingle;
        const int owner = single ? ord % NG : -1;
        for (int i = single ? (grp == owner ? 0 : u.count) : (grp + NG - done % NG) % NG; i < u.count; i += single ? 1 : NG) {
            const int n = done + i, st = n % SLOTS, turn = n / SLOTS;
            // the turn before is over (it may be another group's), so the parity is this turn's
            if (!wait_count(freed + st, turn * Gm::READERS) || !wait(full + st, turn & 1)) return;
            unsigned char* slot = ring + st * Gm::SLOTB;
            uint32_t slot_addr = smem_addr(slot);
            after_wait(slot_addr);
            const int slot_pos = u.base + (u.tile + i) * ST;
            if (slot_pos < u.lo || slot_pos + ST > kv_len) {
                // values of places outside the sequence become zeros
                for (int x = lane; x < ST * CPR; x += 32) {
                    const int r = x / CPR;
                    if (slot_pos + r < u.lo || slot_pos + r >= kv_len)
                        *reinterpret_cast<uint4*>(slot + HALF + chunk_at<CPR>(r, x % CPR)) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();  // before the slot is filled again
                __syncwarp();
            }
            // in steps of SUB tokens, a loop: unrolled over a slot the code would not stay in the
            // instruction caches
#pragma unroll 1
            for (int sub = 0; sub < ST; sub += SUB) {
                const int pos0 = slot_pos + sub;
                if (pos0 >= kv_len || pos0 + SUB <= u.lo) continue;  // nobody's
                const unsigned char* kt = slot + sub * Gm::ROWB;
                const uint32_t ks = slot_addr + sub * Gm::ROWB, vs = ks + HALF;
                const bool whole = pos0 >= all_lo && pos0 + SUB <= all_hi;
                // with few tokens a slot, even and odd steps go to accumulators of their own (a product waits
                // for the one before it of the same accumulator)
                constexpr int NS = T8 ? KU : 2 * KU;  // accumulators of SUB tokens
                constexpr int SETS = FP8 ? 1 : (T8 && KU == 1 ? 4 : 2);
                float S[SETS * NS][4];
#pragma unroll
                for (int x = 0; x < SETS * NS; ++x) S[x][0] = S[x][1] = S[x][2] = S[x][3] = 0.0f;
                if (T8) {
                    // S^T = K Q^T: 16 tokens by 8 rows a product, half of what 16 rows would take
#pragma unroll
                    for (int kk = 0; kk < D / 16; kk += 2) {
                        uint32_t q[4];  // the rows' operands of steps kk and kk + 1
                        if (!FP8) {
                            ldsm4(q, qaddr + (lane & 7) * QP + (kk * 2 + (lane >> 3)) * 16);
                        } else {
                            const uint2 q0 = *reinterpret_cast<const uint2*>(qrow + g * QP + kk * 32 + j * 8);
                            const uint2 q1 = *reinterpret_cast<const uint2*>(qrow + g * QP + kk * 32 + 32 + j * 8);
                            q[0] = q0.x;
                            q[1] = q0.y;
                            q[2] = q1.x;
                            q[3] = q1.y;
                        }
#pragma unroll
                        for (int x = 0; x < KU; ++x) {
                            if (!FP8) {
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    uint32_t a[4];
                                    ldsm4(a, ks + chunk_at<CPR>(x * 16 + (lane & 15), (kk + y) * 2 + (lane >> 4)));
                                    mma<false>(S[(kk + y) % SETS * NS + x], a, q[2 * y], q[2 * y + 1]);
                                }
                            } else {
                                uint32_t v[4];  // tokens 0-7 and 8-15 of chunk kk, then of chunk kk + 1 (see below)
                                ldsm4(v, ks + chunk_at<CPR>(x * 16 + (lane & 15), kk + (lane >> 4)));
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const uint32_t a[4] = {e4m3_to_half2(v[2 * y], false), e4m3_to_half2(v[2 * y + 1], false),
                                                           e4m3_to_half2(v[2 * y], true), e4m3_to_half2(v[2 * y + 1], true)};
                                    mma<true>(S[x], a, q[2 * y], q[2 * y + 1]);
                                }
                            }
                        }
                    }
                } else if (!FP8) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const int o = kk % SETS * NS;
                        uint32_t a[4];
                        ldsm4(a, qaddr + (wm * 16 + (lane & 15)) * QP + (kk * 2 + (lane >> 4)) * 16);
#pragma unroll
                        for (int x = 0; x < KU; ++x) {
                            uint32_t v[4];
                            ldsm4(v, ks + chunk_at<CPR>(x * 16 + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)));
                            mma<false>(S[o + 2 * x], a, v[0], v[1]);
                            mma<false>(S[o + 2 * x + 1], a, v[2], v[3]);
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
                            const uint2 q0 = *reinterpret_cast<const uint2*>(qrow + (wm * 16 + g) * QP + (kk + x) * 32 + j * 8);
                            const uint2 q1 = *reinterpret_cast<const uint2*>(qrow + (wm * 16 + g + 8) * QP + (kk + x) * 32 + j * 8);
                            a[x][0] = q0.x;
                            a[x][1] = q1.x;
                            a[x][2] = q0.y;
                            a[x][3] = q1.y;
                        }
#pragma unroll
                        for (int y = 0; y < KU; ++y) {
                            uint32_t v[4];  // tokens 0-7 and 8-15 of chunk kk, then of chunk kk + 1
                            ldsm4(v, ks + chunk_at<CPR>(y * 16 + (lane & 15), kk + (lane >> 4)));
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                mma<true>(S[2 * y], a[x], e4m3_to_half2(v[2 * x], false), e4m3_to_half2(v[2 * x], true));
                                mma<true>(S[2 * y + 1], a[x], e4m3_to_half2(v[2 * x + 1], false), e4m3_to_half2(v[2 * x + 1], true));
                            }
                        }
                    }
                }
#pragma unroll
                for (int o = 1; o < SETS; ++o) {
#pragma unroll
                    for (int x = 0; x < NS; ++x) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) S[x][e] += S[o * NS + x][e];
                    }
                }
                float mx0 = FP8 ? -INFINITY : m[0], mx1 = FP8 ? -INFINITY : m[1];
                if (capped && !large_cap) {
#pragma unroll
                    for (int x = 0; x < NS; ++x) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)  // c tanh(y) = c - 2 c / (1 + e^2y)
                            S[x][e] = fmaf(-2.0f * to_log2, rcp_fast(1.0f + exp2_fast(S[x][e] * (second(e) ? f1 : f0))), to_log2);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < NS; ++x) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) S[x][e] *= second(e) ? f1 : f0;
                    }
                    if (__builtin_expect(large_cap, 0)) {
                        float y[NS * 4];
#pragma unroll
                        for (int x = 0; x < NS * 4; ++x) y[x] = S[x / 4][x % 4];
                        cap_large<NS * 4>(y, p.sh.softcap);
#pragma unroll
                        for (int x = 0; x < NS * 4; ++x) S[x / 4][x % 4] = y[x];
                    }
                }
                if (!whole) {
#pragma unroll
                    for (int x = 0; x < NS; ++x) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int pos = pos0 + (T8 ? x * 16 + g + (e >> 1) * 8 : x * 8 + 2 * j + (e & 1));
                            const bool in = second(e) ? pos < hi1 && pos >= lo1 : pos < hi0 && pos >= lo0;
                            S[x][e] = in ? S[x][e] : -INFINITY;
                        }
                    }
                }
#pragma unroll
                for (int x = 0; x < NS; ++x) {
                    mx0 = fmaxf(mx0, T8 ? fmaxf(S[x][0], S[x][2]) : fmaxf(S[x][0], S[x][1]));
                    mx1 = fmaxf(mx1, T8 ? fmaxf(S[x][1], S[x][3]) : fmaxf(S[x][2], S[x][3]));
                }
#pragma unroll
                for (int o = XOR0; o < XOR1; o <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
                }
                if (FP8) {
                    mx0 = fmaxf(m[0], fp16_reference(mx0));
                    mx1 = fmaxf(m[1], fp16_reference(mx1));
                }
                const float ref0 = mx0 == -INFINITY ? 0.0f : mx0, ref1 = mx1 == -INFINITY ? 0.0f : mx1;  // nothing seen yet
                if (__any_sync(0xffffffffu, mx0 != m[0] || mx1 != m[1])) {
                    const float a0 = exp2_fast(m[0] - ref0), a1 = exp2_fast(m[1] - ref1);
                    l[0] *= a0;
                    l[1] *= a1;
#pragma unroll
                    for (int x = 0; x < ND; ++x) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) O[x][e] *= second(e) ? a1 : a0;
                    }
                    m[0] = mx0;
                    m[1] = mx1;
                }
#pragma unroll
                for (int x = 0; x < NS; ++x) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        S[x][e] = exp2_fast(S[x][e] - (second(e) ? ref1 : ref0));
                        l[second(e)] += S[x][e];
                    }
                }

                // The probabilities meet the values in the 16 bits that the products take, rounded once: bf16
                // with a bf16 cache (by 2^-8 of each at most; the row's largest so far is 1, exact), fp16 with
                // an e4m3 one (2^-11). The sums are of the unrounded ones.
                // A slot that some rows may not see in full: a value that is not finite must not reach
                // the rows whose mask leaves it out (0 * inf), so such slots go token by token.
                bool plain = true;
                if (!whole) {
                    bool bad = false;
                    for (int x = lane; x < SUB * CPR; x += 32) {
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
                if (plain && T8) {
                    // O^T += V^T P^T: 16 columns by 8 rows a product; the probabilities' operand is their
                    // accumulator transposed
#pragma unroll
                    for (int x = 0; x < KU; ++x) {
                        const uint32_t b0 = transpose8(pack2<FP8>(S[x][0], S[x][1])), b1 = transpose8(pack2<FP8>(S[x][2], S[x][3]));
                        if (!FP8) {
#pragma unroll
                            for (int c = 0; c < ND; ++c) {
                                uint32_t a[4];
                                ldsm4t(a, vs + chunk_at<CPR>(x * 16 + (lane & 7) + ((lane >> 4) << 3), c * 2 + ((lane >> 3) & 1)));
                                mma<false>(O[c], a, b0, b1);
                            }
                        } else {
                            // rows g of the operand take the even columns of chunk c, rows g + 8 the odd ones
#pragma unroll
                            for (int c = 0; c < ND; c += 2) {
                                uint32_t v[4];
                                ldsm4t(v, vs + chunk_at<CPR>(x * 16 + (lane & 15), c + (lane >> 4)));
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const uint32_t x0 = e4m3_to_half2(v[2 * y], false), y0 = e4m3_to_half2(v[2 * y], true);
                                    const uint32_t x1 = e4m3_to_half2(v[2 * y + 1], false), y1 = e4m3_to_half2(v[2 * y + 1], true);
                                    const uint32_t a[4] = {__byte_perm(x0, y0, 0x5410), __byte_perm(x0, y0, 0x7632),
                                                           __byte_perm(x1, y1, 0x5410), __byte_perm(x1, y1, 0x7632)};
                                    mma<true>(O[c + y], a, b0, b1);
                                }
                            }
                        }
                    }
                } else if (plain) {
#pragma unroll
                    for (int x = 0; x < KU; ++x) {
                        const uint32_t a[4] = {pack2<FP8>(S[2 * x][0], S[2 * x][1]), pack2<FP8>(S[2 * x][2], S[2 * x][3]),
                                               pack2<FP8>(S[2 * x + 1][0], S[2 * x + 1][1]), pack2<FP8>(S[2 * x + 1][2], S[2 * x + 1][3])};
                        const int r = x * 16 + (lane & 15);
                        if (!FP8) {
#pragma unroll
                            for (int c = 0; c < ND / 2; ++c) {
                                uint32_t v[4];
                                ldsm4t(v, vs + chunk_at<CPR>(r, cs * ND + c * 2 + (lane >> 4)));
                                mma<false>(O[2 * c], a, v[0], v[1]);
                                mma<false>(O[2 * c + 1], a, v[2], v[3]);
                            }
                        } else {
                            // a transposed pair of bytes is columns 2n, 2n+1 of one token: tile 2c takes the
                            // even columns of chunk c, tile 2c + 1 the odd ones
#pragma unroll
                            for (int c = 0; c < ND / 2; c += 2) {
                                uint32_t v[4];
                                ldsm4t(v, vs + chunk_at<CPR>(r, cs * (ND / 2) + c + (lane >> 4)));
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const uint32_t x0 = e4m3_to_half2(v[2 * y], false), y0 = e4m3_to_half2(v[2 * y], true);
                                    const uint32_t x1 = e4m3_to_half2(v[2 * y + 1], false), y1 = e4m3_to_half2(v[2 * y + 1], true);
                                    mma<true>(O[2 * (c + y)], a, __byte_perm(x0, y0, 0x5410), __byte_perm(x1, y1, 0x5410));
                                    mma<true>(O[2 * (c + y) + 1], a, __byte_perm(x0, y0, 0x7632), __byte_perm(x1, y1, 0x7632));
                                }
                            }
                        }
                    }
                } else {
#pragma unroll 1
                    for (int t = 0; t < SUB; ++t) {
                        uint32_t b0 = 0, b1 = 0;  // by masks: an index known at run time only would put S into local memory
#pragma unroll
                        for (int x = 0; x < NS; ++x) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {  // this lane's elements of token t, if it has them
                                uint32_t mask = (T8 ? x == (t >> 4) && (e >> 1) == ((t >> 3) & 1) : x == (t >> 3) && (e & 1) == (t & 1)) ? ~0u : 0u;
                                asm("" : "+r"(mask));  // (or the compiler makes an index of it after all)
                                const uint32_t bits = __float_as_uint(S[x][e]) & mask;
                                if (second(e)) b1 |= bits; else b0 |= bits;
                            }
                        }
                        const int holder = T8 ? (t & 7) * 4 + j : (lane & ~3) | ((t >> 1) & 3);
                        const float p0 = __uint_as_float(__shfl_sync(0xffffffffu, b0, holder));
                        const float p1 = __uint_as_float(__shfl_sync(0xffffffffu, b1, holder));
                        const int pos = pos0 + t;
                        const bool in0 = pos < hi0 && pos >= lo0, in1 = pos < hi1 && pos >= lo1;
#pragma unroll
                        for (int x = 0; x < ND; ++x) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {  // the lane's two columns of tile x
                                float v;
                                if (!FP8) {
                                    const int col = T8 ? x * 16 + g + 8 * e : cs * (ND * 8) + x * 8 + 2 * j + e;
                                    v = bf16_bits_to_float(*reinterpret_cast<const uint16_t*>(kt + HALF + chunk_at<CPR>(t, col >> 3) + (col & 7) * 2));
                                } else {
                                    const int col = T8 ? x * 16 + 2 * g + e : cs * (ND * 8) + (x >> 1) * 16 + 4 * j + 2 * e + (x & 1);
                                    const uint32_t hh = e4m3_to_half2(*(kt + HALF + chunk_at<CPR>(t, col >> 4) + (col & 15)), false);
                                    v = __low2float(*reinterpret_cast<const __half2*>(&hh));
                                }
                                const int ea = T8 ? 2 * e : e, eb = T8 ? 2 * e + 1 : e + 2;
                                if (in0) O[x][ea] = fmaf(p0, v, O[x][ea]);
                                if (in1) O[x][eb] = fmaf(p1, v, O[x][eb]);
                            }
                        }
                    }
                }
            }
            before_release(O);
            __syncwarp();
            if (lane == 0) add_release(freed + st);
        }
        done += u.count;
        __syncwarp();
        if (lane == 0) add_release(qfreed + qs);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int o = XOR0; o < XOR1; o <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
        }

        const bool split = u.c0 != u.c1;
        const int rows = min(BM, u.n * G - u.rt * BM);
        if (split) {
            // the first CTA's piece ends its share, the others' begin theirs
            const int which = (int)blockIdx.x == u.c0;
            if (which) split_last = true; else split_first = true;
            if (warp == 0 && lane == 0) pieces[NQ + which] = u;
        }
        // where a piece goes (fp32, unnormalised)
        float* mine = p.partial + (size_t)(blockIdx.x * 2 + ((int)blockIdx.x == u.c0)) * PSTRIDE;

        // ---- the token groups joined: each leaves its output in shared memory, every thread sums
        // four columns of a row over the groups and writes them (by a tree down to one group, which
        // then wrote alone, 256 sequences of 16 to 300 tokens took 67 us, so 53) ----
        if (NG > 1 && !single) {
            constexpr int RND = Gm::RND, COLS = Gm::COLS, WCOLS = Gm::WCOLS, JPITCH = Gm::JPITCH, NT = kComputeWarps * 32;
            constexpr int ITEMS = (BM * COLS / 4 + NT - 1) / NT;  // of a thread and round
            auto column = [&](int round, int c) { return c / WCOLS * (D / CS) + round * WCOLS + c % WCOLS; };
            uint2 z[Gm::ROUNDS][ITEMS];  // the gates, on their way meanwhile
#pragma unroll
            for (int y = 0; y < ITEMS; ++y) {
                const int k = tid + y * NT, r = k / (COLS / 4), rr = u.rt * BM + r, t = rr / G;
#pragma unroll
                for (int round = 0; round < Gm::ROUNDS; ++round)
                    z[round][y] = !split && p.gate.ptr && r < rows ? gate_of4(p, (size_t)u.first + t, u.h * G + rr - t * G, column(round, k % (COLS / 4) * 4))
                                                                   : make_uint2(0, 0);
            }
            if (joins > 0 && !wait(rbar, (joins - 1) & 1)) return;  // the last join's reads are done
            float* part = jbuf + grp * BM * JPITCH + cs * WCOLS;
            if (cs == 0 && (T8 ? g == 0 : j == 0)) {
                float* stat = jm + grp * 2 * BM;
                stat[ra] = m[0];
                stat[rb] = m[1];
                stat[BM + ra] = l[0];
                stat[BM + rb] = l[1];
            }
#pragma unroll
            for (int round = 0; round < Gm::ROUNDS; ++round) {
                if (round > 0 && !meet()) return;
#pragma unroll
                for (int x = 0; x < RND; ++x) {
                    const float(&o)[4] = O[round * RND + x];
                    if (T8 && !FP8) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) part[(ra + (e & 1)) * JPITCH + x * 16 + g + 8 * (e >> 1)] = o[e];
                    } else if (T8) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<float2*>(part + (ra + e) * JPITCH + x * 16 + 2 * g) = make_float2(o[e], o[2 + e]);
                    } else if (!FP8) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<float2*>(part + (e ? rb : ra) * JPITCH + x * 8 + 2 * j) = make_float2(o[2 * e], o[2 * e + 1]);
                    } else if (x % 2 == 0) {  // tile x has the even columns, tile x + 1 the odd ones
                        const float(&o1)[4] = O[round * RND + (x | 1)];
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<float4*>(part + (e ? rb : ra) * JPITCH + x * 8 + 4 * j) = make_float4(o[2 * e], o1[2 * e], o[2 * e + 1], o1[2 * e + 1]);
                    }
                }
                if (!meet()) return;
#pragma unroll
                for (int y = 0; y < ITEMS; ++y) {
                    const int k = tid + y * NT, r = k / (COLS / 4), c = k % (COLS / 4) * 4, rr = u.rt * BM + r, t = rr / G;
                    if (r >= rows) continue;
                    float top = jm[r], w[NG], tot = 0.0f;
#pragma unroll
                    for (int i = 1; i < NG; ++i) top = fmaxf(top, jm[i * 2 * BM + r]);
                    const float ref = top == -INFINITY ? 0.0f : top;
                    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        w[i] = exp2_fast(jm[i * 2 * BM + r] - ref);
                        tot = fmaf(w[i], jm[i * 2 * BM + BM + r], tot);
                        const float4 o = *reinterpret_cast<const float4*>(jbuf + (i * BM + r) * JPITCH + c);
                        sum.x = fmaf(w[i], o.x, sum.x);
                        sum.y = fmaf(w[i], o.y, sum.y);
                        sum.z = fmaf(w[i], o.z, sum.z);
                        sum.w = fmaf(w[i], o.w, sum.w);
                    }
                    const int head = u.h * G + rr - t * G;
                    const size_t row = (size_t)u.first + t;
                    if (split) *reinterpret_cast<float4*>(mine + r * D + column(round, c)) = sum;
                    else write_out4<FP8>(p, row, head, D, column(round, c), sum, 1.0f / tot, z[round][y]);
                    if (round == 0 && c == 0) {
                        if (split) {
                            mine[BM * D + r] = top;
                            mine[BM * D + BM + r] = tot;
                        } else if (p.lse) {
                            p.lse[row * p.sh.Hq + head] = log_sum<FP8>(top, tot);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(rbar);
            ++joins;
        }

        // ---- or the one group that has a short piece, or all of a unit, writes the result or the piece ----
        if (T8 && grp == owner) {
            // 32 columns at a time through this warp's part of shared memory, rows by rows: a lane holds
            // columns of two rows, but eight lanes write a row together
            float* mem = obuf + warp * (8 * Gm::OUTP);
            const float inv0 = 1.0f / l[0], inv1 = 1.0f / l[1];
            uint2 z[D / 32][2];
            float inv[2];
            int head[2];
            size_t row[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int r = y * 4 + (lane >> 3), rr = u.rt * BM + r, t = rr / G;
                const float a = __shfl_sync(0xffffffffu, inv0, r >> 1), b = __shfl_sync(0xffffffffu, inv1, r >> 1);
                inv[y] = (r & 1) ? b : a;
                head[y] = u.h * G + rr - t * G;
                row[y] = (size_t)u.first + t;
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    z[c][y] = !split && p.gate.ptr && r < rows ? gate_of4(p, row[y], head[y], c * 32 + (lane & 7) * 4) : make_uint2(0, 0);
            }
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 2; ++x) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int col = x * 16 + (FP8 ? 2 * g + (e >> 1) : g + 8 * (e >> 1));
                        mem[(2 * j + (e & 1)) * Gm::OUTP + col] = O[c * 2 + x][e];
                    }
                }
                __syncwarp();
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int r = y * 4 + (lane >> 3), col = c * 32 + (lane & 7) * 4;
                    const float4 o = *reinterpret_cast<const float4*>(mem + r * Gm::OUTP + (lane & 7) * 4);
                    if (r >= rows) continue;
                    if (split) *reinterpret_cast<float4*>(mine + r * D + col) = o;
                    else write_out4<FP8>(p, row[y], head[y], D, col, o, inv[y], z[c][y]);
                }
            }
            if (g == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 2 * j + e, rr = u.rt * BM + r, t = rr / G;
                    if (r >= rows) continue;
                    if (split) {
                        mine[BM * D + r] = m[e];
                        mine[BM * D + BM + r] = l[e];
                    } else if (p.lse) {
                        p.lse[((size_t)u.first + t) * p.sh.Hq + u.h * G + rr - t * G] = log_sum<FP8>(m[e], l[e]);
                    }
                }
            }
        }
        if (!T8 && grp == owner) {
            const int a = wm * 16 + g, r0 = u.rt * BM + a;
            const bool in0 = a < rows, in1 = a + 8 < rows;
            if (split) {
#pragma unroll
                for (int x = 0; x < ND; x += 2) {
                    const int col = cs * (ND * 8) + x * 8;
                    if (!FP8) {
                        if (in0) {
                            *reinterpret_cast<float2*>(mine + a * D + col + 2 * j) = make_float2(O[x][0], O[x][1]);
                            *reinterpret_cast<float2*>(mine + a * D + col + 8 + 2 * j) = make_float2(O[x + 1][0], O[x + 1][1]);
                        }
                        if (in1) {
                            *reinterpret_cast<float2*>(mine + (a + 8) * D + col + 2 * j) = make_float2(O[x][2], O[x][3]);
                            *reinterpret_cast<float2*>(mine + (a + 8) * D + col + 8 + 2 * j) = make_float2(O[x + 1][2], O[x + 1][3]);
                        }
                    } else {
                        if (in0) *reinterpret_cast<float4*>(mine + a * D + col + 4 * j) = make_float4(O[x][0], O[x + 1][0], O[x][1], O[x + 1][1]);
                        if (in1) *reinterpret_cast<float4*>(mine + (a + 8) * D + col + 4 * j) = make_float4(O[x][2], O[x + 1][2], O[x][3], O[x + 1][3]);
                    }
                }
                if (j == 0 && cs == 0) {
                    mine[BM * D + a] = m[0];
                    mine[BM * D + a + 8] = m[1];
                    mine[BM * D + BM + a] = l[0];
                    mine[BM * D + BM + a + 8] = l[1];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (!(e ? in1 : in0)) continue;
                    const int t = e ? t1 : t0, head = u.h * G + (r0 + 8 * e) - t * G;
                    const size_t row = (size_t)u.first + t, at = row * p.sh.Hq + head;
                    uint16_t* out = p.out + at * D + cs * (ND * 8);
                    const uint16_t* gate = p.gate.ptr + row * p.gate.row + (size_t)head * p.gate.head + cs * (ND * 8);
                    const float inv = 1.0f / l[e];
                    if (!FP8) {
                        uint32_t z[ND];
                        if (p.gate.ptr) {
#pragma unroll
                            for (int x = 0; x < ND; ++x) z[x] = __ldg(reinterpret_cast<const uint32_t*>(gate + x * 8 + 2 * j));
                        }
#pragma unroll
                        for (int x = 0; x < ND; ++x) {
                            float v0 = O[x][2 * e] * inv, v1 = O[x][2 * e + 1] * inv;
                            if (p.gate.ptr) {
                                v0 *= sigmoid_fast(__uint_as_float(z[x] << 16));
                                v1 *= sigmoid_fast(__uint_as_float(z[x] & 0xffff0000u));
                            }
                            *reinterpret_cast<uint32_t*>(out + x * 8 + 2 * j) = pack2<false>(v0, v1);
                        }
                    } else {
                        uint2 z[ND / 2];
                        if (p.gate.ptr) {
#pragma unroll
                            for (int x = 0; x < ND / 2; ++x) z[x] = __ldg(reinterpret_cast<const uint2*>(gate + x * 16 + 4 * j));
                        }
#pragma unroll
                        for (int x = 0; x < ND / 2; ++x) {
                            const float s = p.sh.v_scale;  // (by itself, as in write_out4)
                            float v0 = O[2 * x][2 * e] * inv * s, v1 = O[2 * x + 1][2 * e] * inv * s;
                            float v2 = O[2 * x][2 * e + 1] * inv * s, v3 = O[2 * x + 1][2 * e + 1] * inv * s;
                            if (p.gate.ptr) {
                                v0 *= sigmoid_fast(__uint_as_float(z[x].x << 16));
                                v1 *= sigmoid_fast(__uint_as_float(z[x].x & 0xffff0000u));
                                v2 *= sigmoid_fast(__uint_as_float(z[x].y << 16));
                                v3 *= sigmoid_fast(__uint_as_float(z[x].y & 0xffff0000u));
                            }
                            *reinterpret_cast<uint2*>(out + x * 16 + 4 * j) = make_uint2(pack2<false>(v0, v1), pack2<false>(v2, v3));
                        }
                    }
                    if (p.lse && cs == 0 && j == 0) p.lse[at] = log_sum<FP8>(m[e], l[e]);
                }
            }
        }
    }

    static_assert(BM * (kJoinMost + 2) * 4 <= SLOTS * Gm::SLOTB, "weights");
    join_units<D, FP8, BM, kComputeWarps * 32>(p, pieces + NQ, split_first, split_last, reinterpret_cast<float*>(ring), misc + 12, meet);
}

template <int D, bool FP8, int WM>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
    using Gm = Geo<D, FP8, WM>;
    auto kern = attn_decode_kernel<D, FP8, WM>;
    int dev, sms;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    const size_t smem = Gm::SLOTS * (size_t)Gm::SLOTB + Gm::NQ * (size_t)Gm::QB + Gm::JOINB + Gm::OUTB + Gm::FIXED + ((size_t)a.B + 1) * 4;
    static_assert(Gm::NG * 2 * Gm::BM * 4 + Gm::NQ * Gm::BM * 4 + (Gm::NQ + 3) * (int)sizeof(Piece) + (Gm::SLOTS + 2 * Gm::NQ + 2) * 8 +
                      (Gm::SLOTS + Gm::NQ + 16) * 4 <= Gm::FIXED, "small data");
    static std::once_flag once[kMaxDevices];
    static cudaError_t set[kMaxDevices];
    std::call_once(once[dev], [&] {
        cudaFuncAttributes attr;
        set[dev] = cudaFuncGetAttributes(&attr, kern);
        // the kernel hands registers from one role to the others: fewer at the launch and it would wait for good
        if (set[dev] == cudaSuccess && attr.numRegs != kLaunchRegs) set[dev] = cudaErrorLaunchOutOfResources;
        if (set[dev] == cudaSuccess)
            set[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    });
    if (set[dev] != cudaSuccess) return set[dev];
    // TMA tiles of whole atoms when pages are whole atoms; otherwise row copies
    int box = a.sh.page_size % 8 == 0 ? a.sh.page_size & -a.sh.page_size : 0;
    if (box > Gm::ST) box = Gm::ST;
    CUtensorMap map_k{}, map_v{};
    if (box && !(make_pool_map(&map_k, a.c.k, a, Gm::ROWB, box) && make_pool_map(&map_v, a.c.v, a, Gm::ROWB, box)))
        return cudaErrorInvalidValue;
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
    return cudaLaunchKernelEx(&cfg, kern, a, map_k, map_v, box);
}

// Row groups for `rows` query rows per key/value head (0: up to eight rows, transposed).
int row_groups(int rows) { return rows <= 8 ? 0 : (rows <= 16 ? 1 : (rows <= 32 ? 2 : 4)); }

template <int D, bool FP8>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t stream) {
    switch (row_groups(a.T * a.sh.G)) {
        case 0: return launch<D, FP8, 0>(a, stream);
        case 1: return launch<D, FP8, 1>(a, stream);
        case 2: return launch<D, FP8, 2>(a, stream);
        default: return launch<D, FP8, 4>(a, stream);
    }
}

}  // namespace

size_t attn_workspace_bytes(int d, bool fp8, int page_size, int rows) {
    const int tile = attn_rows_supported(d, fp8, page_size, rows) ? 128 : 16 * (row_groups(rows) ? row_groups(rows) : 1);
    return kAttnPartialAt + (size_t)kAttnMaxCtas * 2 * tile * (d + 2) * sizeof(float);
}

long attn_decode_places(const AttnShape& sh, const PagedCache& c, int T) {
    static_assert(kShortCost < kAttnUnitPlaces && kUnitCost < kAttnUnitPlaces, "places of a unit");
    const int groups = row_groups(T * sh.G);
    return attn_places(sh, c, T, Geo<64, true, 0>::HALF / (sh.d * (sh.fp8 ? 1 : 2)), groups ? 16 * groups : 8);
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
