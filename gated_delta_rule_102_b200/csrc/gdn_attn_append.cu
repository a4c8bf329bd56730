// RMSNorm of each q and k head, rotary positions and the append to the paged cache, one
// launch ("metrale_model_layers/forward/qwen3_5/full_attention.rs": the per-head q/k
// norms, RoPE and the KV append, three launches on that page).
//
//   x <- x / sqrt(mean x^2 + eps) * (offset + w);  (x_i, x_j) <- (x_i c - x_j s, x_j c + x_i s)
//
// One CTA per token row, or per four rows of a sequence when there are many. A head vector
// is held by d/16 lanes in two 16-byte words each, so every load and store is a whole word
// and the norm's sum is a few shuffles; the next vector's words are in flight while one is
// worked on. The angles depend on the row alone: the cosines and sines are computed once
// into shared memory while the first vectors are on their way.
// The angle p * f is formed and reduced to a turn in 64 bits (a 32-bit product is off by
// a thousandth of a radian at position 10^4 already); only the remainder goes to the
// 32-bit sine and cosine. Everything else is fp32 and is rounded once, on the way out.
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_attn.h"
#include "gdn_device.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;  // most token rows of one CTA

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
template <int D>
__device__ __forceinline__ void rotate_head(float (&x)[2][8], int sub, int R, Pairs pairs, const float2* cs, float* ex) {
    constexpr int LPH = D / 16;
    const int h = R >> 1, e0 = sub * 8;
    if (pairs == kNeighbours) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
#pragma unroll
            for (int u = 0; u < 8; u += 2) {
                const int e = w * (D / 2) + e0 + u;
                if (e < R) {
                    const float2 t = cs[e >> 1];
                    const float a = x[w][u], b = x[w][u + 1];
                    x[w][u] = fmaf(a, t.x, -b * t.y);
                    x[w][u + 1] = fmaf(b, t.x, a * t.y);
                }
            }
        }
    } else if (pairs == kFirstWord) {
        const bool low = e0 < h;
        const int from = (low ? sub + (h >> 3) : sub - (h >> 3)) & (LPH - 1);
        const float2* c = cs + (low ? e0 : e0 - h);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float y = __shfl_sync(0xffffffffu, x[0][u], from, LPH);
            if (e0 < R) {
                const float2 t = c[u];
                x[0][u] = low ? fmaf(x[0][u], t.x, -y * t.y) : fmaf(x[0][u], t.x, y * t.y);
            }
        }
    } else if (pairs == kOtherWord) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float2 t = cs[e0 + u];
            const float a = x[0][u], b = x[1][u];
            x[0][u] = fmaf(a, t.x, -b * t.y);
            x[1][u] = fmaf(b, t.x, a * t.y);
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
                    const float2 t = cs[e < h ? e : e - h];
                    const float y = ex[e < h ? e + h : e - h];
                    x[w][u] = e < h ? fmaf(x[w][u], t.x, -y * t.y) : fmaf(x[w][u], t.x, y * t.y);
                }
            }
        }
    }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads, 3) qk_rope_append_kernel(const AppendArgs p, const int rpc) {
    constexpr int LPH = D / 16, GROUPS = kThreads / LPH;
    __shared__ float2 cs[kRows][D / 2];
    __shared__ long token[kRows];  // where a row's key and value go (page * page_size + offset), -1: nowhere
    extern __shared__ float exchange[];
    const int tid = threadIdx.x, sub = tid % LPH, group = tid / LPH;
    const int Hq = p.sh.Hq, Hkv = p.sh.Hkv, V = Hq + 2 * Hkv, R = p.sh.R;

    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int parts = (p.T + rpc - 1) / rpc;
    const int b = blockIdx.x / parts, t0 = (blockIdx.x - b * parts) * rpc;
    int first = b * p.T, n = p.T;
    const int slot = __ldg(p.slots + b);
    if (p.cu) {
        first = __ldg(p.cu + b);
        n = __ldg(p.cu + b + 1) - first;
        if (n < 0 || n > p.T || first < 0 || first > p.total - n) {
            if (t0 == 0 && tid == 0 && p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_SEQLEN_BIT);
            return;
        }
        if (t0 >= n) return;
    }
    if (slot < 0 || slot >= p.c.rows) {
        if (t0 == 0 && tid == 0 && p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_SLOT_RANGE_BIT);
        return;
    }
    const int rows = min(rpc, n - t0);
    const long row0 = first + t0;

    // this lane group's vectors: numbers group, group + GROUPS, .. of the CTA's rows * V
    int v = group, t = 0;  // head vector of row t
    while (v >= V) v -= V, ++t;
    uint4 w[2];
    auto fetch = [&](int t, int v) {
        if (t >= rows) return;
        const Heads& h = v < Hq ? p.q : (v < Hq + Hkv ? p.k : p.v);
        const int head = v < Hq ? v : (v < Hq + Hkv ? v - Hq : v - Hq - Hkv);
        const uint4* src = reinterpret_cast<const uint4*>(h.ptr + (row0 + t) * h.row + head * h.head) + sub;
        w[0] = __ldg(src);
        w[1] = __ldg(src + LPH);
    };
    w[0] = w[1] = make_uint4(0, 0, 0, 0);
    fetch(t, v);
    const int past = __ldg(p.c.seq_lens + slot);
    if (past < 0 || past > p.c.max_pages * p.sh.page_size - n) {
        if (t0 == 0 && tid == 0 && p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_SEQLEN_BIT);
        return;
    }
    if (tid < rows) {
        const int pos = past + t0 + tid, at = pos / p.sh.page_size;
        const int page = __ldg(p.c.table + (long)slot * p.c.max_pages + at);
        const bool ok = page >= 0 && page < p.c.num_pages;
        if (!ok && p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_PAGE_BIT);
        token[tid] = ok ? (long)page * p.sh.page_size + (pos - at * p.sh.page_size) : -1;
    }
    const int h = R >> 1;
    for (int i = tid; i < rows * h; i += kThreads) {
        const int r = i / h, e = i - r * h;
        const double a = (double)(past + t0 + r) * (double)__ldg(p.inv_freq + e);
        const double turns = rint(a * 0.15915494309189535);  // 1 / (2 pi)
        const double x = fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586, a));  // 2 pi in two parts
        float s, c;
        sincosf((float)x, &s, &c);
        cs[r][e] = make_float2(c * p.sh.rope_scale, s * p.sh.rope_scale);
    }
    uint4 wq[2], wk[2];
    wq[0] = wq[1] = wk[0] = wk[1] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (p.qw) wq[i] = __ldg(reinterpret_cast<const uint4*>(p.qw) + sub + i * LPH);
        if (p.kw) wk[i] = __ldg(reinterpret_cast<const uint4*>(p.kw) + sub + i * LPH);
    }
    const Pairs pairs = p.sh.interleaved ? kNeighbours : (R == D ? kOtherWord : ((h & 7) == 0 && R <= D / 2 ? kFirstWord : kAnywhere));
    __syncthreads();

    // warps take every pass that any of their groups needs (the shuffles want all lanes)
    const int total = rows * V;
    for (int base = 0; base + (tid / 32) * (32 / LPH) < total; base += GROUPS) {
        const bool active = t < rows;
        const int tr = active ? t : 0, vr = v;
        float x[2][8];
        unpack8(w[0], x[0]);
        unpack8(w[1], x[1]);
        const uint4 raw0 = w[0], raw1 = w[1];
        // the next vector's words are on their way while this one is worked on
        v += GROUPS;
        while (v >= V) v -= V, ++t;
        fetch(t, v);
        const bool is_q = vr < Hq, is_v = vr >= Hq + Hkv;
        float ss = 0.0f;
#pragma unroll
        for (int u = 0; u < 8; ++u) ss = fmaf(x[0][u], x[0][u], fmaf(x[1][u], x[1][u], ss));
#pragma unroll
        for (int off = LPH / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        if (is_q ? p.qw != nullptr : p.kw != nullptr) {
            const float r = rsqrtf(ss * (1.0f / D) + p.sh.norm_eps);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float f[8];
                unpack8(is_q ? wq[i] : wk[i], f);
#pragma unroll
                for (int u = 0; u < 8; ++u) x[i][u] = x[i][u] * r * (p.sh.norm_offset + f[u]);
            }
        }
        if (R > 0) rotate_head<D>(x, sub, R, pairs, cs[tr], exchange + group * D);
        if (!active) continue;
        if (is_q) {
            uint4* out = reinterpret_cast<uint4*>(p.q_out + ((row0 + tr) * Hq + vr) * D) + sub;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                out[i * LPH] = make_uint4(bf16x2(x[i][0], x[i][1]), bf16x2(x[i][2], x[i][3]), bf16x2(x[i][4], x[i][5]), bf16x2(x[i][6], x[i][7]));
            continue;
        }
        if (token[tr] < 0) continue;
        if (is_v) {
            unpack8(raw0, x[0]);
            unpack8(raw1, x[1]);
        }
        const long dst = (token[tr] * Hkv + (is_v ? vr - Hq - Hkv : vr - Hq)) * D + sub * 8;
        void* pool = is_v ? p.c.v : p.c.k;
        if (!FP8) {
#pragma unroll
            for (int i = 0; i < 2; ++i)  // (exact for values: bf16 to fp32 and back)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(pool) + dst + i * (D / 2)) =
                    is_v ? (i ? raw1 : raw0)
                         : make_uint4(bf16x2(x[i][0], x[i][1]), bf16x2(x[i][2], x[i][3]), bf16x2(x[i][4], x[i][5]), bf16x2(x[i][6], x[i][7]));
        } else {
            const float scale = is_v ? p.sh.v_scale : p.sh.k_scale;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int u = 0; u < 8; ++u) x[i][u] /= scale;
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + dst + i * (D / 2)) =
                    make_uint2(e4m3x2(x[i][0], x[i][1]) | (e4m3x2(x[i][2], x[i][3]) << 16),
                               e4m3x2(x[i][4], x[i][5]) | (e4m3x2(x[i][6], x[i][7]) << 16));
            }
        }
    }
}

template <int D>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    // A row a CTA until every SM has its three; then a CTA keeps up to four rows of a
    // sequence, whose lengths and pages are looked up together.
    int dev, sms;
    const cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    const int rpc = a.B * a.T <= 3 * sms ? 1 : (a.T < kRows ? a.T : kRows);
    cfg.gridDim = dim3((unsigned)(a.B * ((a.T + rpc - 1) / rpc)));
    cfg.blockDim = dim3(kThreads);
    const bool anywhere = !a.sh.interleaved && a.sh.R != D && ((a.sh.R / 2) % 8 != 0 || a.sh.R > D / 2);
    cfg.dynamicSmemBytes = anywhere ? kThreads / (D / 16) * D * sizeof(float) : 0;
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
