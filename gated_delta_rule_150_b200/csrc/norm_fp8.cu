// norm_fp8.cu -- the producers of 8-bit operands: RMSNorm of the residual
// stream with the residual's addition, the mixer's gated per-head RMSNorm, and
// the weights' block quantisation.
//
// All three read every input once and write every output once: a row (or a
// group, or a 128 x 128 block) stays in registers from its load to its codes.
// They are bound by HBM.  A thread holds octets (eight consecutive channels,
// one 16-byte load of bf16); octet j of a row belongs to the row's group j / 16,
// so an aligned half warp holds exactly one group and finds its maximum by four
// shuffles.
#include "fp8.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace gdr {
namespace {

// ---------------------------------------------------------------------------
// y = h / sqrt(mean h^2 + eps) * w with h = x + residual.
// TPR threads own a row (a warp, or a whole CTA), each up to IT octets of it,
// kept in registers as fp32 between the sum of squares and the codes.
// ---------------------------------------------------------------------------
template <typename T, bool RES, int TPR, int IT>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
norm_fp8_kernel(int rows, int width, const T* x, const T* residual, const float* __restrict__ weight,
                float eps, T* residual_out, uint8_t* __restrict__ y, float* __restrict__ y_scale) {
    constexpr int kWarps = TPR / 32;
    __shared__ float part[kWarps];
    pdl_wait();
    pdl_launch_dependents();
    const int t = threadIdx.x % TPR;
    const int row = blockIdx.x * (blockDim.x / TPR) + threadIdx.x / TPR;
    if (TPR == 32 && row >= rows) return;          // whole warps; with TPR > 32 the grid is exact
    const int n8 = width >> 3;
    const int64_t base = (int64_t)row * width;
    Octet<T> a[IT], b[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int j = t + i * TPR;
        a[i].zero();
        b[i].zero();
        if (j < n8) {
            a[i].load(x + base + 8 * j);
            if (RES) b[i].load(residual + base + 8 * j);
        }
    }
    float h[IT][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        a[i].to_float(h[i]);
        if (RES) {
            float r[8];
            b[i].to_float(r);
#pragma unroll
            for (int c = 0; c < 8; ++c) h[i][c] += r[c];
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) ss = fmaf(h[i][c], h[i][c], ss);
    }
    if (RES && residual_out) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int j = t + i * TPR;
            if (j < n8) Octet<T>::store(residual_out + base + 8 * j, h[i]);
        }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
    if (kWarps > 1) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
        __syncthreads();
        ss = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) ss += part[w];
    }
    const float inv = rsqrtf(ss / (float)width + eps);
    const int groups = (width + kFp8Group - 1) / kFp8Group;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int j = t + i * TPR;
        if (i > 0 && (j & ~31) >= n8) break;       // the same for a whole warp
        if (j < n8) {
            const float4 w0 = __ldg(reinterpret_cast<const float4*>(weight) + 2 * j);
            const float4 w1 = __ldg(reinterpret_cast<const float4*>(weight) + 2 * j + 1);
            const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int c = 0; c < 8; ++c) h[i][c] = h[i][c] * inv * w[c];
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) h[i][c] = 0.f;      // past the row: 0 * inv may be NaN
        }
        const float s = fp8_scale(half_warp_max(abs_bits_max(h[i])));
        if (j < n8) {
            *reinterpret_cast<uint2*>(y + base + 8 * j) = fp8_codes(h[i], 1.f / s);
            if ((j & 15) == 0) y_scale[(int64_t)row * groups + (j >> 4)] = s;
        }
    }
}

// ---------------------------------------------------------------------------
// y = o / sqrt(mean_d o^2 + eps) * w * sigmoid(gate), per head of D channels.
// A half warp owns one group of 128 channels of a token (one head at D 128, two
// at D 64); each thread works on U groups at once, a grid stride apart, so that
// the loads of all of them are in flight together.
// ---------------------------------------------------------------------------
constexpr int kGatedThreads = 256;

template <typename TO, typename TG, int D, int U>
__global__ void __launch_bounds__(kGatedThreads)
gated_norm_fp8_kernel(int64_t tasks, int groups, int n8, const TO* __restrict__ o,
                      const TG* __restrict__ gate, const float* __restrict__ weight, float eps,
                      uint8_t* __restrict__ y, float* __restrict__ y_scale) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 15;
    const int64_t first = ((int64_t)blockIdx.x * kGatedThreads + threadIdx.x) >> 4;
    const int64_t stride = (int64_t)gridDim.x * (kGatedThreads / 16);
    float w[8];
    {
        const int c = (lane * 8) % D;
        const float4 w0 = __ldg(reinterpret_cast<const float4*>(weight + c));
        const float4 w1 = __ldg(reinterpret_cast<const float4*>(weight + c) + 1);
        w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
        w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
    }
    Octet<TO> a[U];
    Octet<TG> b[U];
    int64_t at[U];                                   // first channel of the octet, -1: none
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t task = first + u * stride;
        const int64_t row = task / groups;
        const int j = (int)(task - row * groups) * 16 + lane;
        at[u] = task < tasks && j < n8 ? (row * n8 + j) * 8 : -1;
        a[u].zero();
        b[u].zero();
        if (at[u] >= 0) {
            a[u].load(o + at[u]);
            b[u].load(gate + at[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float f[8], g[8];
        a[u].to_float(f);
        b[u].to_float(g);
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) ss = fmaf(f[c], f[c], ss);
#pragma unroll
        for (int s = D / 16; s > 0; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
        const float inv = rsqrtf(ss * (1.f / D) + eps);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            f[c] = at[u] >= 0 ? __fdividef(f[c] * inv * w[c], 1.f + __expf(-g[c])) : 0.f;
        const float s = fp8_scale(half_warp_max(abs_bits_max(f)));
        if (at[u] >= 0) {
            *reinterpret_cast<uint2*>(y + at[u]) = fp8_codes(f, 1.f / s);
            if (lane == 0) y_scale[first + u * stride] = s;
        }
    }
}

// ---------------------------------------------------------------------------
// Weights: one CTA per 128 x 128 block, 16 threads across a row, 8 rows each.
// ---------------------------------------------------------------------------
constexpr int kQuantThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kQuantThreads)
quantize_weight_kernel(int n, int k, int k_groups, const T* __restrict__ w, uint8_t* __restrict__ codes,
                       float* __restrict__ scales) {
    __shared__ uint32_t part[kQuantThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int bn = blockIdx.x / k_groups, bk = blockIdx.x - bn * k_groups;
    const int col = bk * kFp8Group + (threadIdx.x & 15) * 8;
    const int row0 = bn * kFp8Group + (threadIdx.x >> 4);
    Octet<T> a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = row0 + 16 * i;
        a[i].zero();
        if (row < n && col < k) a[i].load(w + (int64_t)row * k + col);
    }
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f[8];
        a[i].to_float(f);
        m = max(m, abs_bits_max(f));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQuantThreads / 32; ++i) m = max(m, part[i]);
    const float s = fp8_scale(m), inv = 1.f / s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = row0 + 16 * i;
        float f[8];
        a[i].to_float(f);
        if (row < n && col < k)
            *reinterpret_cast<uint2*>(codes + (int64_t)row * k + col) = fp8_codes(f, inv);
    }
    if (threadIdx.x == 0) scales[blockIdx.x] = s;
}

template <typename T, bool RES, int TPR, int IT>
cudaError_t launch_norm_shape(const gdr_norm_fp8_args& a, cudaStream_t st) {
    constexpr int threads = TPR < 128 ? 128 : TPR;
    constexpr int rows_per_cta = threads / TPR;
    const unsigned grid = (unsigned)((a.rows + rows_per_cta - 1) / rows_per_cta);
    return launch_pdl(true, norm_fp8_kernel<T, RES, TPR, IT>, dim3(grid), dim3(threads), 0, st,
                      (int)a.rows, a.width, (const T*)a.x, (const T*)a.residual, a.norm_weight,
                      a.norm_eps, (T*)a.residual_out, (uint8_t*)a.y, a.y_scale);
}

template <typename T, bool RES>
cudaError_t launch_norm_typed(const gdr_norm_fp8_args& a, cudaStream_t st) {
    const int n8 = a.width / 8;
    if (n8 <= 32 * 4) return launch_norm_shape<T, RES, 32, 4>(a, st);
    if (n8 <= 128 * 4) return launch_norm_shape<T, RES, 128, 4>(a, st);
    if (n8 <= 512 * 2) return launch_norm_shape<T, RES, 512, 2>(a, st);
    return launch_norm_shape<T, RES, 512, 8>(a, st);
}

template <typename TO, typename TG>
cudaError_t launch_gated_typed(const gdr_gated_norm_fp8_args& a, cudaStream_t st) {
    constexpr int U = 2;
    const int width = a.n_heads * a.d_v;
    const int groups = fp8_groups(width);
    const int64_t tasks = a.rows * groups;
    constexpr int64_t per_cta = kGatedThreads / 16 * U;
    const int64_t grid = (tasks + per_cta - 1) / per_cta;
    if (grid > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
    auto kern = a.d_v == 64 ? gated_norm_fp8_kernel<TO, TG, 64, U> : gated_norm_fp8_kernel<TO, TG, 128, U>;
    return launch_pdl(true, kern, dim3((unsigned)grid), dim3(kGatedThreads), 0, st, tasks, groups,
                      width / 8, (const TO*)a.o, (const TG*)a.gate_raw, a.norm_weight, a.norm_eps,
                      (uint8_t*)a.y, a.y_scale);
}

}  // namespace

cudaError_t launch_norm_fp8(const gdr_norm_fp8_args& a, cudaStream_t st) {
    if (a.io_dtype == GDR_BF16)
        return a.residual ? launch_norm_typed<__nv_bfloat16, true>(a, st)
                          : launch_norm_typed<__nv_bfloat16, false>(a, st);
    return a.residual ? launch_norm_typed<float, true>(a, st) : launch_norm_typed<float, false>(a, st);
}

cudaError_t launch_gated_norm_fp8(const gdr_gated_norm_fp8_args& a, cudaStream_t st) {
    if (a.o_dtype == GDR_BF16)
        return a.gate_dtype == GDR_BF16 ? launch_gated_typed<__nv_bfloat16, __nv_bfloat16>(a, st)
                                        : launch_gated_typed<__nv_bfloat16, float>(a, st);
    return a.gate_dtype == GDR_BF16 ? launch_gated_typed<float, __nv_bfloat16>(a, st)
                                    : launch_gated_typed<float, float>(a, st);
}

cudaError_t launch_quantize_weight_fp8(int n, int k, gdr_dtype dt, const void* w, void* codes,
                                       float* scales, cudaStream_t st) {
    const int k_groups = fp8_groups(k);
    const int64_t grid = (int64_t)fp8_groups(n) * k_groups;
    if (grid > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
    return dt == GDR_BF16
        ? launch_pdl(true, quantize_weight_kernel<__nv_bfloat16>, dim3((unsigned)grid), dim3(kQuantThreads),
                     0, st, n, k, k_groups, (const __nv_bfloat16*)w, (uint8_t*)codes, scales)
        : launch_pdl(true, quantize_weight_kernel<float>, dim3((unsigned)grid), dim3(kQuantThreads), 0, st,
                     n, k, k_groups, (const float*)w, (uint8_t*)codes, scales);
}

}  // namespace gdr
