// RMSNorm of each q and k head, rotary positions and the append to the paged cache, one
// launch ("metrale_model_layers/forward/qwen3_5/full_attention.rs": the per-head q/k
// norms, RoPE and the KV append, three launches on that page).
//
//   x <- x / sqrt(mean x^2 + eps) * (offset + w);  (x_i, x_j) <- (x_i c - x_j s, x_j c + x_i s)
//
// One CTA per token row. A head vector is held by d/8 lanes, 16 bytes each, so every
// load and store is a whole 16-byte word (8 bytes into an e4m3 cache) and the norm's sum
// is a few shuffles. The angles depend on the row alone: the first R/2 threads compute
// the cosines and sines once into shared memory while the head vectors are in flight.
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
constexpr int kBatch = 4;  // head vectors of a lane group whose loads are in flight together

// Two floats to two e4m3 bytes (round to nearest even, saturated; `a` in the low byte).
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
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
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = (uint32_t)float_to_bf16_bits(x[2 * i]) | ((uint32_t)float_to_bf16_bits(x[2 * i + 1]) << 16);
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// y[u] = x[(u + r) % 8] for a run-time r.
__device__ __forceinline__ void rotate8(const float (&x)[8], int r, float (&y)[8]) {
    float a[8], b[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) a[u] = (r & 1) ? x[(u + 1) & 7] : x[u];
#pragma unroll
    for (int u = 0; u < 8; ++u) b[u] = (r & 2) ? a[(u + 2) & 7] : a[u];
#pragma unroll
    for (int u = 0; u < 8; ++u) y[u] = (r & 4) ? b[(u + 4) & 7] : b[u];
}

// Rotates the eight elements e0..e0+7 of a head held by this lane; the head's other
// elements are in the neighbouring lanes of the same group of LPH.
template <int LPH>
__device__ __forceinline__ void rotate_head(float (&x)[8], int sub, int R, bool interleaved, const float2* cs) {
    const int e0 = sub * 8;
    if (interleaved) {
        if (e0 < R) {
#pragma unroll
            for (int u = 0; u < 8; u += 2) {
                if (e0 + u < R) {
                    const float2 t = cs[(e0 + u) >> 1];
                    const float a = x[u], b = x[u + 1];
                    x[u] = fmaf(a, t.x, -b * t.y);
                    x[u + 1] = fmaf(b, t.x, a * t.y);
                }
            }
        }
        return;
    }
    const int h = R >> 1;
    if ((h & 7) == 0) {  // a lane's elements are all in one half, its partner's lane is fixed
        const bool low = e0 < h;
        const int from = low ? sub + (h >> 3) : sub - (h >> 3);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float y = __shfl_sync(0xffffffffu, x[u], from & (LPH - 1), LPH);
            if (e0 < R) {
                const float2 t = cs[low ? e0 + u : e0 + u - h];
                x[u] = low ? fmaf(x[u], t.x, -y * t.y) : fmaf(x[u], t.x, y * t.y);
            }
        }
        return;
    }
    // any even R: element e's partner is e + h or e - h, at the same place (u +- h) % 8 of
    // its lane for every lane
    float up[8], dn[8], z[8];
    rotate8(x, h & 7, up);
    rotate8(x, (8 - h) & 7, dn);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const float a = __shfl_sync(0xffffffffu, up[u], (sub + ((u + h) >> 3)) & (LPH - 1), LPH);
        const float b = __shfl_sync(0xffffffffu, dn[u], (sub + ((u - h) >> 3)) & (LPH - 1), LPH);
        const int e = e0 + u;
        z[u] = x[u];
        if (e < R) {
            const float2 t = cs[e < h ? e : e - h];
            z[u] = e < h ? fmaf(x[u], t.x, -a * t.y) : fmaf(x[u], t.x, b * t.y);
        }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = z[u];
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) qk_rope_append_kernel(const AppendArgs p) {
    constexpr int LPH = D / 8, GROUPS = kThreads / LPH;
    __shared__ float2 cs[D / 2];
    const int tid = threadIdx.x, sub = tid % LPH, group = tid / LPH;
    const int Hq = p.sh.Hq, Hkv = p.sh.Hkv, V = Hq + 2 * Hkv, R = p.sh.R;

    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int b = blockIdx.x / p.T, t = blockIdx.x - b * p.T;
    int first = b * p.T, n = p.T;
    const int slot = __ldg(p.slots + b);
    if (p.cu) {
        first = __ldg(p.cu + b);
        n = __ldg(p.cu + b + 1) - first;
        if (n < 0 || n > p.T || first < 0 || first > p.total - n) {
            if (t == 0 && tid == 0 && p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_SEQLEN_BIT);
            return;
        }
        if (t >= n) return;
    }
    if (slot < 0 || slot >= p.c.rows) {
        if (t == 0 && tid == 0 && p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_SLOT_RANGE_BIT);
        return;
    }
    const long row = first + t;
    auto source = [&](int v) -> const uint16_t* {
        if (v < Hq) return p.q.ptr + row * p.q.row + v * p.q.head;
        if (v < Hq + Hkv) return p.k.ptr + row * p.k.row + (v - Hq) * p.k.head;
        return p.v.ptr + row * p.v.row + (v - Hq - Hkv) * p.v.head;
    };
    uint4 w[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        const int v = group + i * GROUPS;
        w[i] = v < V ? __ldg(reinterpret_cast<const uint4*>(source(v)) + sub) : make_uint4(0, 0, 0, 0);
    }
    const int past = __ldg(p.c.seq_lens + slot);
    if (past < 0 || past > p.c.max_pages * p.sh.page_size - n) {
        if (t == 0 && tid == 0 && p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_SEQLEN_BIT);
        return;
    }
    const int pos = past + t, at = pos / p.sh.page_size;
    const int page = __ldg(p.c.table + (long)slot * p.c.max_pages + at);
    const bool store = page >= 0 && page < p.c.num_pages;
    if (!store && tid == 0 && p.err_flag) atomicOr(p.err_flag, GDN_DEVICE_ERR_PAGE_BIT);
    const long token = (long)page * p.sh.page_size + (pos - at * p.sh.page_size);
    for (int i = tid; i < R / 2; i += kThreads) {
        const double a = (double)pos * (double)__ldg(p.inv_freq + i);
        const double turns = rint(a * 0.15915494309189535);  // 1 / (2 pi)
        const double r = fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586, a));  // 2 pi in two parts
        float s, c;
        sincosf((float)r, &s, &c);
        cs[i] = make_float2(c * p.sh.rope_scale, s * p.sh.rope_scale);
    }
    float wq[8], wk[8];
    if (p.qw) unpack8(__ldg(reinterpret_cast<const uint4*>(p.qw) + sub), wq);
    if (p.kw) unpack8(__ldg(reinterpret_cast<const uint4*>(p.kw) + sub), wk);
    __syncthreads();

    for (int base = 0; base < V; base += kBatch * GROUPS) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int v = base + group + i * GROUPS;
            if (base + i * GROUPS >= V) break;  // the same for every thread
            const bool is_q = v < Hq, is_v = v >= Hq + Hkv;
            float x[8];
            unpack8(w[i], x);
            float ss = 0.0f;
#pragma unroll
            for (int u = 0; u < 8; ++u) ss = fmaf(x[u], x[u], ss);
#pragma unroll
            for (int off = LPH / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            if (!is_v && (is_q ? p.qw : p.kw)) {
                const float r = rsqrtf(ss * (1.0f / D) + p.sh.norm_eps);
#pragma unroll
                for (int u = 0; u < 8; ++u) x[u] = x[u] * r * (p.sh.norm_offset + (is_q ? wq[u] : wk[u]));
            }
            float raw[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) raw[u] = x[u];
            if (R > 0) rotate_head<LPH>(x, sub, R, p.sh.interleaved, cs);  // shuffles: every lane takes part
            if (v >= V) continue;
            if (is_q) {
                reinterpret_cast<uint4*>(p.q_out + (row * Hq + v) * D)[sub] = pack8(x);
                continue;
            }
            if (!store) continue;
            const int h = is_v ? v - Hq - Hkv : v - Hq;
            const long dst = (token * Hkv + h) * D + sub * 8;
            void* pool = is_v ? p.c.v : p.c.k;
            if (!FP8) {
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(pool) + dst) = is_v ? w[i] : pack8(x);
            } else {
                const float scale = is_v ? p.sh.v_scale : p.sh.k_scale;
#pragma unroll
                for (int u = 0; u < 8; ++u) x[u] = (is_v ? raw[u] : x[u]) / scale;
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + dst) =
                    make_uint2(e4m3x2(x[0], x[1]) | (e4m3x2(x[2], x[3]) << 16),
                               e4m3x2(x[4], x[5]) | (e4m3x2(x[6], x[7]) << 16));
            }
        }
        if (base + kBatch * GROUPS < V) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int v = base + kBatch * GROUPS + group + i * GROUPS;
                w[i] = v < V ? __ldg(reinterpret_cast<const uint4*>(source(v)) + sub) : make_uint4(0, 0, 0, 0);
            }
        }
    }
}

template <int D>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * a.T));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return a.sh.fp8 ? cudaLaunchKernelEx(&cfg, qk_rope_append_kernel<D, true>, a)
                    : cudaLaunchKernelEx(&cfg, qk_rope_append_kernel<D, false>, a);
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
