// RMSNorm of each q and k head, rotary positions and the append to the paged cache, one
// launch ("metrale_model_layers/forward/qwen3_5/full_attention.rs": the per-head q/k
// norms, RoPE and the KV append, three launches on that page).
//
//   x <- x / sqrt(mean x^2 + eps) * (offset + w);  (x_i, x_j) <- (x_i c - x_j s, x_j c + x_i s)
//
// A head vector is held by d/16 lanes in two 16-byte words each, so every load and store is a
// whole word and the norm's sum is a few shuffles. A CTA holds all heads of a row (up to 384
// threads); with many rows it keeps several of a sequence, so that a lane group's weights
// and addresses and the sequence's lookups are set up once, with the next rows' words on their
// way to shared memory. Cosines and sines depend on the row alone: once a CTA, in
// shared memory. Everything is fp32 and rounded once, on the way out; the angle is formed in
// 64 bits and in turns (a 32-bit product is off by a thousandth of a radian at position 10^4
// already), only its fraction goes to the 32-bit sine and cosine.
// Measured: 256 sequences of 16 rows, 16 query and 2 key/value heads of 256, bf16: 18.5 us for 84 MB
// (4.5 TB/s), 256 equal CTAs on 148 SMs, of which 108 have two and 40 one; about 200 instructions a warp
// and row. 200 sequences of up to 16 rows, 32 and 8 heads of 128 to e4m3: 16.9 us where the bytes take 5.6
// and the instructions (430 a warp and row, set-up among them) 7: the 400 CTAs have 1 to 8 rows each or
// none, so that an SM is without work for a third of the time, and while it has some the chain of a row
// (its words, the norm's shuffles, the rotation, the store) leaves half of the issue slots empty. One row
// takes 3.3 us, dependent lookups.
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "gdn_attn.h"
#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kRows = kMaxTokens;  // most token rows of one CTA
constexpr int kMostThreads = 384;
constexpr int kAhead = 4;  // rows whose words are in flight

// Two floats to two e4m3 bytes (round to nearest even, saturated; `a` in the low byte).
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

// How the pairs of a head lie: neighbours in a lane; halves whose partner is the same
// element of another lane's first word (R <= d/2), or of the lane's other word (R = d);
// halves of any other even R, exchanged through shared memory.
enum Pairs { kNeighbours, kFirstWord, kOtherWord, kAnywhere };

// A head vector is held by LPH = D / 16 lanes in two 16-byte words: lane `sub` has elements
// 8 sub .. 8 sub + 7 and D/2 more on. `cs` are the row's cosines and sines, `ex` the lane
// group's exchange area of D floats.
// Pair i's cosine and sine lie at cs_at(i): the four float4s that a lane with pairs 8 k .. 8 k + 7
// reads are apart, so that neighbouring lanes' reads are neighbours (no bank conflicts).
template <int D>
__device__ __forceinline__ int cs_at(int i) {
    return ((i >> 1) & 3) * (D / 8) + (i >> 3) * 2 + (i & 1);
}
template <int D>
__device__ __forceinline__ void rotate_head(float (&x)[2][8], int sub, int R, Pairs pairs, const float2* cs, float* ex) {
    constexpr int LPH = D / 16;
    const int h = R >> 1, e0 = sub * 8;
    const float4* cs4 = reinterpret_cast<const float4*>(cs);
    if (pairs == kNeighbours) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
#pragma unroll
            for (int u = 0; u < 8; u += 2) {
                const int e = w * (D / 2) + e0 + u;
                if (e < R) {
                    const float2 t = cs[cs_at<D>(e >> 1)];
                    const float a = x[w][u], b = x[w][u + 1];
                    x[w][u] = fmaf(a, t.x, -b * t.y);
                    x[w][u + 1] = fmaf(b, t.x, a * t.y);
                }
            }
        }
    } else if (pairs == kFirstWord) {
        const bool low = e0 < h;
        const int from = (low ? sub + (h >> 3) : sub - (h >> 3)) & (LPH - 1);
        const int k = (low ? sub : from) & (LPH - 1);  // the lane whose pairs these are
        float y[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) y[u] = __shfl_sync(0xffffffffu, x[0][u], from, LPH);
        if (e0 < R) {
            const uint32_t flip = low ? 0x80000000u : 0u;  // the first element of a pair subtracts
#pragma unroll
            for (int u = 0; u < 8; u += 2) {
                const float4 t = cs4[(u / 2) * LPH + k];
                x[0][u] = fmaf(__uint_as_float(__float_as_uint(y[u]) ^ flip), t.y, x[0][u] * t.x);
                x[0][u + 1] = fmaf(__uint_as_float(__float_as_uint(y[u + 1]) ^ flip), t.w, x[0][u + 1] * t.z);
            }
        }
    } else if (pairs == kOtherWord) {
#pragma unroll
        for (int u = 0; u < 8; u += 2) {
            const float4 t = cs4[(u / 2) * LPH + sub];
            const float a = x[0][u], b = x[1][u], c = x[0][u + 1], d = x[1][u + 1];
            x[0][u] = fmaf(a, t.x, -b * t.y);
            x[1][u] = fmaf(b, t.x, a * t.y);
            x[0][u + 1] = fmaf(c, t.z, -d * t.w);
            x[1][u + 1] = fmaf(d, t.z, c * t.w);
        }
    } else {
        __syncwarp();
#pragma unroll
        for (int w = 0; w < 2; ++w) {
#pragma unroll
            for (int u = 0; u < 8; ++u) ex[w * (D / 2) + e0 + u] = x[w][u];
        }
        __syncwarp();
#pragma unroll
        for (int w = 0; w < 2; ++w) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int e = w * (D / 2) + e0 + u;
                if (e < R) {
                    const float2 t = cs[cs_at<D>(e < h ? e : e - h)];
                    const float y = ex[e < h ? e + h : e - h];
                    x[w][u] = e < h ? fmaf(x[w][u], t.x, -y * t.y) : fmaf(x[w][u], t.x, y * t.y);
                }
            }
        }
    }
}

// A division by the cache's scale whose result is rounded to e4m3. A power of two: the product with
// its inverse, exact (results so small that they are not are zeros). Else the product, off by at
// most 2^-23 of itself: where the values 2^-21 to both sides of it round to the same, so does the
// quotient, and only the rest is divided (a division an element took 18.1 us for 200 sequences of up
// to 16 rows, so 16.8).
struct Divisor {
    float scale, inverse;
    bool exact, near;
    __device__ __forceinline__ explicit Divisor(float s) : scale(s), inverse(1.0f / s) {
        const uint32_t bits = __float_as_uint(s), e = bits >> 23;
        near = e >= 64 && e <= 190;  // the inverse is a normal number with room to either side
        exact = near && (bits & 0x7fffffu) == 0;
    }
};
// A lane's sixteen elements divided by the scale, as e4m3 (nowhere: a null pointer).
template <int D>
__device__ __forceinline__ void store_e4m3(const float (&x)[2][8], const Divisor& by, unsigned char* to) {
    if (!to) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t z[4];
        bool sure = by.near;
#pragma unroll
        for (int u = 0; u < 8; u += 2) {
            const float a = x[i][u] * by.inverse, b = x[i][u + 1] * by.inverse;
            z[u / 2] = e4m3x2(a, b);
            if (!by.exact) {
                constexpr float kLess = 1.0f - 0x1p-21f, kMore = 1.0f + 0x1p-21f;
                z[u / 2] = e4m3x2(a * kLess, b * kLess);
                sure = sure && z[u / 2] == e4m3x2(a * kMore, b * kMore);
            }
        }
        if (!sure) {
#pragma unroll
            for (int u = 0; u < 8; u += 2) z[u / 2] = e4m3x2(__fdiv_rn(x[i][u], by.scale), __fdiv_rn(x[i][u + 1], by.scale));
        }
        *reinterpret_cast<uint2*>(to + i * (D / 2)) = make_uint2(z[0] | (z[1] << 16), z[2] | (z[3] << 16));
    }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kMostThreads, 2) qk_rope_append_kernel(const AppendArgs p, const int rpc) {
    constexpr int LPH = D / 16;
    __shared__ __align__(16) float2 cs[kRows][D / 2];
    __shared__ long token[kRows];  // where a row's key and value go (page * page_size + offset), -1: nowhere
    extern __shared__ __align__(16) unsigned char dynamic[];  // [kAhead][2][threads] words, then the exchange areas
    const int tid = threadIdx.x, threads = blockDim.x, sub = tid % LPH, group = tid / LPH;
    const int Hq = p.sh.Hq, Hkv = p.sh.Hkv, V = Hq + 2 * Hkv, R = p.sh.R, h = R >> 1;
    // this lane group's head vector, of every row of the CTA: q's, then k's, then v's
    const int v = blockIdx.y * (threads / LPH) + group;
    const bool active = v < V, is_q = v < Hq, is_v = v >= Hq + Hkv;

    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int parts = (p.T + rpc - 1) / rpc;
    const int b = blockIdx.x / parts, t0 = (blockIdx.x - b * parts) * rpc;
    const bool report = t0 == 0 && blockIdx.y == 0 && tid == 0 && p.err_flag;
    int first = b * p.T, n = p.T;
    const int slot = __ldg(p.slots + b);
    if (p.cu) {
        first = __ldg(p.cu + b);
        n = __ldg(p.cu + b + 1) - first;
        if (n < 0 || n > p.T || first < 0 || first > p.total - n) {
            if (report) atomicOr(p.err_flag, GDN_DEVICE_ERR_SEQLEN_BIT);
            return;
        }
        if (t0 >= n) return;
    }
    if (slot < 0 || slot >= p.c.rows) {
        if (report) atomicOr(p.err_flag, GDN_DEVICE_ERR_SLOT_RANGE_BIT);
        return;
    }
    const int rows = min(rpc, n - t0);
    const long row0 = first + t0;
    const Heads& from = is_q ? p.q : (is_v ? p.v : p.k);
    const int head = is_q ? v : (is_v ? v - Hq - Hkv : v - Hq);
    const uint4* src = reinterpret_cast<const uint4*>(from.ptr + row0 * from.row + head * from.head) + sub;
    const long src_step = from.row / 8;
    // The words of the next kAhead rows are on their way to shared memory, a lane's own for itself:
    // in registers there is no room for them, and it takes that many to keep HBM busy.
    uint4* ring = reinterpret_cast<uint4*>(dynamic) + tid;
    float* exchange = reinterpret_cast<float*>(dynamic + kAhead * 2 * 16 * threads);
    auto fetch = [&](int t) {
        if (active && t < rows) {
            cp_async_16(ring + (t % kAhead) * 2 * threads, src + t * src_step);
            cp_async_16(ring + (t % kAhead) * 2 * threads + threads, src + t * src_step + LPH);
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(i);
    const int past = __ldg(p.c.seq_lens + slot);
    const bool fits = past >= 0 && past <= p.c.max_pages * p.sh.page_size - n;
    if (!fits && report) atomicOr(p.err_flag, GDN_DEVICE_ERR_SEQLEN_BIT);
    if (!fits) {
        // The words on their way land before the CTA's memory is another's. (In one branch with the flag
        // above, and wait_all for wait_group, the rows of every other sequence took 3 % longer.)
        asm volatile("cp.async.wait_group 0;\n");
        return;
    }
    if (tid < rows) {
        const int pos = past + t0 + tid, at = pos / p.sh.page_size;
        const int page = __ldg(p.c.table + (long)slot * p.c.max_pages + at);
        const bool ok = page >= 0 && page < p.c.num_pages;
        if (!ok && p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_PAGE_BIT);
        token[tid] = ok ? (long)page * p.sh.page_size + (pos - at * p.sh.page_size) : -1;
    }
    // cosines and sines in turns: position * speed / 2 pi in 64 bits, whose fraction the 32-bit
    // functions take
    for (int i = tid; i < rows * h; i += threads) {
        const int r = i / h, e = i - r * h;
        const double turns = (double)(past + t0 + r) * ((double)__ldg(p.inv_freq + e) * 0.15915494309189535);
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cs[r][cs_at<D>(e)] = make_float2(c * p.sh.rope_scale, s * p.sh.rope_scale);
    }
    const uint16_t* norm = is_q ? p.qw : (is_v ? nullptr : p.kw);
    float weight[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (norm) unpack8(__ldg(reinterpret_cast<const uint4*>(norm) + sub + i * LPH), weight[i]);
#pragma unroll
        for (int u = 0; u < 8; ++u) weight[i][u] = norm ? p.sh.norm_offset + weight[i][u] : 1.0f;
    }
    // (both for the whole warp, so that it takes the shuffles together)
    const bool only_values = __all_sync(0xffffffffu, is_v || !active), normed = __any_sync(0xffffffffu, norm != nullptr);
    const Pairs pairs = p.sh.interleaved ? kNeighbours : (R == D ? kOtherWord : ((h & 7) == 0 && R <= D / 2 ? kFirstWord : kAnywhere));
    // where a row's result goes: q_out + row * Hq * D, or pool + token * Hkv * D, in bytes from here
    constexpr int ESZ = FP8 ? 1 : 2;
    unsigned char* to = is_q ? reinterpret_cast<unsigned char*>(p.q_out + (row0 * Hq + head) * D + sub * 8)
                             : static_cast<unsigned char*>(is_v ? p.c.v : p.c.k) + ((size_t)head * D + sub * 8) * ESZ;
    const long to_step = is_q ? (long)Hq * D * 2 : (long)Hkv * D * ESZ;
    const Divisor by(is_v ? p.sh.v_scale : p.sh.k_scale);
    __syncthreads();

    for (int t = 0; t < rows; ++t) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(kAhead - 1) : "memory");
        const uint4 w[2] = {ring[(t % kAhead) * 2 * threads], ring[(t % kAhead) * 2 * threads + threads]};
        fetch(t + kAhead);
        uint4 z[2] = {w[0], w[1]};  // values as they came
        if (!only_values) {
            float x[2][8];
            unpack8(w[0], x[0]);
            unpack8(w[1], x[1]);
            if (normed) {
                float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    s0 = fmaf(x[0][u], x[0][u], s0);
                    s1 = fmaf(x[1][u], x[1][u], s1);
                }
                float ss = s0 + s1;
#pragma unroll
                for (int off = LPH / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
                const float f = norm ? rsqrtf(ss * (1.0f / D) + p.sh.norm_eps) : 1.0f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int u = 0; u < 8; ++u) x[i][u] *= f * weight[i][u];
                }
            }
            if (R > 0) rotate_head<D>(x, sub, R, pairs, cs[t], exchange + group * D);
            if (FP8 && !is_q) {
                // (below, from x)
                if (is_v) {
                    unpack8(w[0], x[0]);
                    unpack8(w[1], x[1]);
                }
                store_e4m3<D>(x, by, active && token[t] >= 0 ? to + token[t] * to_step : nullptr);
            } else if (!is_v) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    z[i] = make_uint4(bf16x2(x[i][0], x[i][1]), bf16x2(x[i][2], x[i][3]), bf16x2(x[i][4], x[i][5]), bf16x2(x[i][6], x[i][7]));
            }
        } else if (FP8) {
            float x[2][8];
            unpack8(w[0], x[0]);
            unpack8(w[1], x[1]);
            store_e4m3<D>(x, by, active && token[t] >= 0 ? to + token[t] * to_step : nullptr);
        }
        if (active && (is_q || (!FP8 && token[t] >= 0))) {
            uint4* at = reinterpret_cast<uint4*>(is_q ? to + t * to_step : to + token[t] * to_step);
            at[0] = z[0];
            at[LPH] = z[1];
        }
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");
}

template <int D>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    // A lane group a head vector, kMostThreads a CTA at most (more vectors: more CTAs a row). A CTA
    // keeps several rows of a sequence when there are more than two rows an SM: as many as make
    // two CTAs an SM, in equal parts of the sequence.
    int dev, sms;
    const cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    const int V = a.sh.Hq + 2 * a.sh.Hkv, most = kMostThreads / (D / 16), ys = (V + most - 1) / most, each = (V + ys - 1) / ys;
    const int threads = (each * (D / 16) + 31) / 32 * 32, per_y = threads / (D / 16);
    const long want = ((long)a.total * ys + 2 * sms - 1) / (2 * sms);  // rows a CTA
    const int parts = want >= a.T ? 1 : (int)(a.T / (want > 0 ? want : 1)), rpc = (a.T + parts - 1) / parts;
    cfg.gridDim = dim3((unsigned)(a.B * ((a.T + rpc - 1) / rpc)), (unsigned)((V + per_y - 1) / per_y));
    cfg.blockDim = dim3((unsigned)threads);
    const bool anywhere = !a.sh.interleaved && a.sh.R != D && ((a.sh.R / 2) % 8 != 0 || a.sh.R > D / 2);
    cfg.dynamicSmemBytes = kAhead * 2 * 16 * threads + (anywhere ? per_y * D * sizeof(float) : 0);
    static std::once_flag once[kMaxDevices];
    static cudaError_t set[kMaxDevices];
    std::call_once(once[dev], [&] {
        const int most_bytes = kAhead * 2 * 16 * kMostThreads + most * D * (int)sizeof(float);
        set[dev] = cudaFuncSetAttribute(qk_rope_append_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most_bytes);
        if (set[dev] == cudaSuccess)
            set[dev] = cudaFuncSetAttribute(qk_rope_append_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most_bytes);
    });
    if (set[dev] != cudaSuccess) return set[dev];
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return a.sh.fp8 ? cudaLaunchKernelEx(&cfg, qk_rope_append_kernel<D, true>, a, rpc)
                    : cudaLaunchKernelEx(&cfg, qk_rope_append_kernel<D, false>, a, rpc);
}

}  // namespace

cudaError_t launch_qk_rope_append(const AppendArgs& a, cudaStream_t stream) {
    switch (a.sh.d) {
        case 64: return launch<64>(a, stream);
        case 128: return launch<128>(a, stream);
        case 256: return launch<256>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
