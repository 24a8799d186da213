// norm_fp8.cu -- the producers of 8-bit operands: RMSNorm of the residual
// stream with the residual's addition, the mixer's gated per-head RMSNorm, and
// the weights' block quantisation.
//
// All three read every input once and write every output once: a row (or a
// group, or a 128 x 128 block) stays in registers from its load to its codes.
// They are bound by HBM.  A thread holds octets (eight consecutive channels,
// one 16-byte load of bf16).
#include "fp8.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace gdr {
namespace {

// ---------------------------------------------------------------------------
// y = h / sqrt(mean h^2 + eps) * w with h = x + residual.
// A row belongs to half a warp (ROWS = 8 rows per CTA, up to 16 octets), to a warp
// (ROWS = 4, up to 64) or to a whole CTA (ROWS = 1), each thread with up to IT octets
// of it, kept in registers as fp32 between the sum of squares and the codes.  Octet j of a row belongs to the
// row's group j / 16, so an aligned half warp holds exactly one group.
// ---------------------------------------------------------------------------
template <typename T, bool RES, int ROWS, int IT>
__global__ void __launch_bounds__(ROWS > 1 ? 128 : IT > 2 ? 512 : 1024)
norm_fp8_kernel(int rows, int width, const T* x, const T* residual, const float* __restrict__ weight,
                float eps, T* residual_out, uint8_t* __restrict__ y, float* __restrict__ y_scale) {
    __shared__ float part[32];
    pdl_wait();
    pdl_launch_dependents();
    const int TPR = ROWS > 1 ? 128 / ROWS : blockDim.x;
    const int t = ROWS > 1 ? threadIdx.x % (128 / ROWS) : threadIdx.x;
    const int row = ROWS > 1 ? blockIdx.x * ROWS + threadIdx.x / (128 / ROWS) : blockIdx.x;
    if (ROWS == 4 && row >= rows) return;          // whole warps
    const int n8 = ROWS > 4 && row >= rows ? 0 : width >> 3;
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
    for (int s = ROWS > 1 ? 64 / ROWS : 16; s > 0; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
    if (ROWS == 1) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
        __syncthreads();
        ss = 0.f;
        const int warps = blockDim.x >> 5;
        for (int w = 0; w < warps; ++w) ss += part[w];
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
        const float s = fp8_scale(lanes_max<16>(abs_bits_max(h[i])));
        if (j < n8) {
            *reinterpret_cast<uint2*>(y + base + 8 * j) = fp8_codes(h[i], fp8_inverse(s));
            if ((j & 15) == 0) y_scale[(int64_t)row * groups + (j >> 4)] = s;
        }
    }
}

// ---------------------------------------------------------------------------
// y = o / sqrt(mean_d o^2 + eps) * w * sigmoid(gate), per head of D channels.
// Eight lanes own one group of 128 channels of a token (one head at D 128, two at
// D 64), 16 channels each: half the shuffles and divisions per channel of eight
// channels a lane.  Bound by HBM with the issue slots close behind (16384 tokens of
// 32 x 128, bf16: 66 us in a stream of calls or 0.78 of the copy rate, 62 in a graph;
// in the stream 82 us with eight channels a lane, 71 with one channel to an instruction).
// ---------------------------------------------------------------------------
constexpr int kGatedThreads = 128;

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// CTAs per SM that the registers have to leave room for: eight, at which all loads are
// issued before the first is used (in graphs, inputs rotating past L2: 16384 x 7 x 64
// with fp32 gates 10.0 us, 12.0 when the compiler chooses; 8192 x 32 x 128 with fp32 o
// 41.5 against 43.5; 2048 x 14 x 64 bf16 3.7 against 4.2), and ten for bf16 heads of
// 128, where more warps hide more (16384 x 32 x 128: 62.1 us, 65.5 with eight).
template <typename TO, typename TG, int D>
constexpr int gated_ctas() { return sizeof(TO) + sizeof(TG) == 4 && D == 128 ? 10 : 8; }

template <typename TO, typename TG, int D>
__global__ void __launch_bounds__(kGatedThreads, gated_ctas<TO, TG, D>())
gated_norm_fp8_kernel(int64_t tasks, int groups, int n16, const TO* __restrict__ o,
                      const TG* __restrict__ gate, const float* __restrict__ weight, float eps,
                      uint8_t* __restrict__ y, float* __restrict__ y_scale) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 7;
    const int64_t task = ((int64_t)blockIdx.x * kGatedThreads + threadIdx.x) >> 3;
    int64_t at = -1;                                 // first of this thread's 16 channels, -1: none
    if (n16 == groups * 8) {                         // no shorter last group: groups lie end to end
        if (task < tasks) at = (task * 8 + lane) * 16;
    } else {
        const int64_t row = task / groups;
        const int j = (int)(task - row * groups) * 8 + lane;
        if (task < tasks && j < n16) at = (row * n16 + j) * 16;
    }
    Octet<TO> a[2];
    Octet<TG> b[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        a[u].zero();
        b[u].zero();
        if (at >= 0) {
            a[u].load(o + at + 8 * u);
            b[u].load(gate + at + 8 * u);
        }
    }
    // two channels per instruction
    float f[16], g[16];
    float2* f2 = reinterpret_cast<float2*>(f);
    float2* g2 = reinterpret_cast<float2*>(g);
    a[0].to_float(f);
    a[1].to_float(f + 8);
    b[0].to_float(g);
    b[1].to_float(g + 8);
    float2 sq = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < 8; ++c) sq = __ffma2_rn(f2[c], f2[c], sq);
    float ss = sq.x + sq.y;
#pragma unroll
    for (int s = D / 32; s > 0; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
    const float inv = rsqrtf(ss * (1.f / D) + eps);
    const float2 inv2 = make_float2(inv, inv), neg = make_float2(-1.44269504f, -1.44269504f), one = make_float2(1.f, 1.f);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const float2 w = __ldg(reinterpret_cast<const float2*>(weight + (lane * 16) % D) + c);
        f2[c] = __fmul2_rn(__fmul2_rn(f2[c], inv2), w);
        // 1 / (1 + 2^(-g log2 e)): 0 where the power overflows
        g2[c] = __fmul2_rn(g2[c], neg);
        g2[c] = __fadd2_rn(make_float2(exp2_approx(g2[c].x), exp2_approx(g2[c].y)), one);
        f2[c] = __fmul2_rn(f2[c], make_float2(rcp_approx(g2[c].x), rcp_approx(g2[c].y)));
    }
    if (at < 0) {                                    // 0 times an infinite inverse
#pragma unroll
        for (int c = 0; c < 16; ++c) f[c] = 0.f;
    }
    const float s = fp8_scale(lanes_max<8>(abs_bits_max(f)));
    if (at >= 0) {
        const float si = fp8_inverse(s);
        const uint2 lo = fp8_codes(f, si), hi = fp8_codes(f + 8, si);
        *reinterpret_cast<uint4*>(y + at) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        if (lane == 0) y_scale[task] = s;
    }
}

// ---------------------------------------------------------------------------
// Weights: one CTA per 128 x 128 block, 16 threads across a row, 8 rows each
// (16416 x 4096 bf16: 34.8 us or 0.88 of the copy rate in a stream of calls; in a graph
// on matrices rotating past L2 33.0 with four CTAs per SM, 35.5 with three, 42.0 with
// the two that the registers would leave otherwise).
// ---------------------------------------------------------------------------
constexpr int kQuantThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 2 ? 4 : 2)
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
            *reinterpret_cast<uint2*>(codes + (int64_t)row * k + col) = fp8_codes_divided(f, s, inv);
    }
    if (threadIdx.x == 0) scales[blockIdx.x] = s;
}

template <typename T, bool RES, int ROWS, int IT>
cudaError_t launch_norm_shape(const gdr_norm_fp8_args& a, int threads, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.rows + ROWS - 1) / ROWS);
    return launch_pdl(true, norm_fp8_kernel<T, RES, ROWS, IT>, dim3(grid), dim3(threads), 0, st, (int)a.rows,
                      a.width, (const T*)a.x, (const T*)a.residual, a.norm_weight, a.norm_eps,
                      (T*)a.residual_out, (uint8_t*)a.y, a.y_scale);
}

// Two octets a thread (graphs of calls on inputs rotating past L2, bf16 with residual):
// 65536 rows of 2048 take 142 us with 128 threads a row, 152 with a warp, 165 with 256;
// at 8192 rows of 896 it makes no difference (64 threads 12.0 us, one warp of four
// octets 12.4, 128 of one 11.8).  Several rows to a CTA of 256 threads were 8 % slower:
// they load and wait together.  With too few rows to fill the SMs one octet a thread (a
// single row of 896: 1.6 against 2.0 us).  Rows of one group would leave half of a warp
// idle: two to a warp (65536 rows of 64: 10.0 against 20.3 us; 100000 of 128: 16.5
// against 30.2).
template <typename T, bool RES>
cudaError_t launch_norm_typed(const gdr_norm_fp8_args& a, cudaStream_t st) {
    const int n8 = a.width / 8;
    const auto warps = [n8](int it) { return 32 * ((n8 + 32 * it - 1) / (32 * it)); };
    if (a.rows <= 2 * 148 && n8 <= 1024) return launch_norm_shape<T, RES, 1, 1>(a, warps(1), st);
    if (n8 <= 16) return launch_norm_shape<T, RES, 8, 1>(a, 128, st);
    if (n8 <= 64) return launch_norm_shape<T, RES, 4, 2>(a, 128, st);
    if (n8 <= 2048) return launch_norm_shape<T, RES, 1, 2>(a, warps(2), st);
    return launch_norm_shape<T, RES, 1, 8>(a, warps(8), st);
}

template <typename TO, typename TG>
cudaError_t launch_gated_typed(const gdr_gated_norm_fp8_args& a, cudaStream_t st) {
    const int width = a.n_heads * a.d_v;
    const int groups = fp8_groups(width);
    const int64_t tasks = a.rows * groups;
    constexpr int64_t per_cta = kGatedThreads / 8;
    const int64_t grid = (tasks + per_cta - 1) / per_cta;
    if (grid > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
    auto kern = a.d_v == 64 ? gated_norm_fp8_kernel<TO, TG, 64> : gated_norm_fp8_kernel<TO, TG, 128>;
    return launch_pdl(true, kern, dim3((unsigned)grid), dim3(kGatedThreads), 0, st, tasks, groups,
                      width / 16, (const TO*)a.o, (const TG*)a.gate_raw, a.norm_weight, a.norm_eps,
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
