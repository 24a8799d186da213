// linear_fp8.cu -- y = (x codes * x scales) (w codes * w scales)^T with e4m3
// codes, one fp32 scale per token and 128 channels (x) and per 128 x 128 block
// (w):
//     y[m, c] = sum_b sx[m, b] sw[c / 128, b] sum_{j in b} x[m, j] w[c, j].
//
// The scales differ from one 128-channel group to the next, so the tensor core
// sums one group (four K = 32 MMAs) into a TMEM accumulator, and the epilogue
// warps add it into fp32 registers with its factor while the next group's MMAs
// run into a second accumulator.
#include <cstring>
#include <cuda.h>

#include "fp8.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace gdr {
namespace {

constexpr int kSms = 148;

// Set by a kernel that gave up a bounded wait (1), or a wait for what it had in
// flight then (2); read and cleared by gdr_linear_fp8_status.
__device__ uint32_t g_linear_error;

// The output's column ranges: columns begin[i] .. begin[i + 1] - 1 go to the
// dense tensor ptr[i].
struct OutRanges {
    int n_outs;
    int begin[GDR_LINEAR_MAX_OUTS + 1];
    int f32[GDR_LINEAR_MAX_OUTS];
    void* ptr[GDR_LINEAR_MAX_OUTS];
};

// One output column: where its tensor's row 0 holds it, and that tensor's row
// length (0: past the last column).
struct OutColumn {
    void* p;
    int pitch;
    int f32;
    __device__ __forceinline__ OutColumn(const OutRanges& r, int c) : p(nullptr), pitch(0), f32(0) {
        for (int i = 0; i < r.n_outs; ++i)
            if (c >= r.begin[i] && c < r.begin[i + 1]) {
                pitch = r.begin[i + 1] - r.begin[i];
                f32 = r.f32[i];
                const int64_t off = c - r.begin[i];
                p = f32 ? (void*)((float*)r.ptr[i] + off) : (void*)((__nv_bfloat16*)r.ptr[i] + off);
            }
    }
    __device__ __forceinline__ void store(int64_t row, float v) const {
        if (f32) ((float*)p)[row * pitch] = v;
        else ((__nv_bfloat16*)p)[row * pitch] = __float2bfloat16_rn(v);
    }
};

// A whole warp's wait that ends: true once the phase completed, false when the
// tries ran out (then the error word is set and the warp's role stops).  A try
// suspends the warp for up to about a microsecond, so the limit is about a
// second.  The loop is kept this small because it is on every role's critical
// path: with a look at the timer in it the many-token kernel ran 10 to 30 %
// slower, with one more store after the limit 2 to 4 %.
#ifdef GDR_TEST_WAIT_LIMIT_NS
constexpr int kWaitTries = 1 << 11;      // the test copy
#else
constexpr int kWaitTries = 1 << 20;
#endif

template <bool CLUSTER = false>          // whether the phase orders other CTAs' writes
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
    for (int i = 0; i < kWaitTries; ++i)
        if (__all_sync(0xffffffffu, CLUSTER ? mbar_try_wait_cluster(a, parity) : mbar_try_wait(a, parity))) return true;
    atomicOr(&g_linear_error, 1u);
    return false;
}

// After a give-up: wait, again with a limit, for what this CTA has in flight.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
    if (!mbar_wait(bar, parity)) atomicOr(&g_linear_error, 2u);
}

// The test copy: one role (0: MMAs, 1: loads, 2: loads of odd CTAs, 3: sums; of CTA
// pairs also 4: stores, 5: loads of even CTAs) waits, at its second group, for a
// barrier that nothing arrives on.
#ifdef GDR_TEST_WAIT_LIMIT_NS
__device__ int g_linear_test_role;
#define GDR_TEST_STALLS(role, i) \
    ((i) == 1 && *(volatile int*)&g_linear_test_role == (role) && !wait(&never, 0))
#else
#define GDR_TEST_STALLS(role, i) false
#endif

// The warp's number from one lane, so that the compiler knows it to be the same in
// all of them and keeps what depends on it in uniform registers (the many-token
// kernel runs 7 % faster).
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0); }

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 16 bytes to another CTA's shared memory (shared::cluster addresses), counted on
// a barrier there.
__device__ __forceinline__ void st_async4(uint32_t cluster_dst, const float4& v, uint32_t cluster_bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
                 ::"r"(cluster_dst), "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)),
                   "r"(__float_as_uint(v.w)), "r"(cluster_bar) : "memory");
}

// ---------------------------------------------------------------------------
// Few tokens: the weights take the MMA's 128-row side and BN tokens its other
// side, so a decode step's few tokens do not leave the tensor core's rows empty
// and every weight is fetched once per BN tokens.  A cluster of `split` CTAs
// shares one 128-column tile: each sums a range of the K groups and sends its
// part of every four tokens to the CTA that owns them (4-token group q: CTA
// q % split), which adds the parts in rank order and stores.  The parts arrive in
// a place of their own and are counted on a barrier, so nobody waits for the
// whole cluster before its sums: no atomics, no workspace.  Bound by load latency and
// by launches where K is short (one token, 3598 x 896: 3.2 us, 2.5 with the weights in
// L2), by HBM and the way to it where the weights are large (one token, 16416 x 4096:
// 13.4 us, 5.0 TB/s).  Times here and at the choices of kernels below: graphs of calls
// whose operands rotate past L2.
//   warps 0-3   a thread owns an output column, BN fp32 sums (one per token)
//   warp 4      TMA loads
//   warp 5      TMEM allocation, MMAs
// ---------------------------------------------------------------------------
constexpr int kFewThreads = 192;
constexpr int kFewAccs = 4;             // TMEM accumulators: groups between an MMA and its sums

template <int BN>
struct FewLayout {
    static constexpr uint32_t kStageBytes = 16384u + BN * 128u;
    static constexpr int kStages = BN <= 16 ? 5 : BN <= 32 ? 4 : 3;     // two CTAs per SM
    static constexpr int kGroups = BN / 4;                              // of four tokens
    static constexpr uint32_t kParts = kStages * kStageBytes;           // [slot][rank][column] x 4 tokens
    static constexpr uint32_t kPartBytes = 2048u;
    static constexpr uint32_t kFactors = kParts + (kGroups < 8 ? 8 : kGroups) * kPartBytes;
    static constexpr uint32_t kBytes = kFactors + 4u * 2u * BN * 4u;    // 4 warps x 2 x BN floats
    static constexpr uint32_t kDynBytes = kBytes + 1024u;               // 1024-byte alignment
    static constexpr uint32_t kTmemCols = kFewAccs * BN;
};

template <int BN>
__global__ void __launch_bounds__(kFewThreads)
linear_few_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                  const float* __restrict__ sx, const float* __restrict__ sw, int M, int groups,
                  int split, const __grid_constant__ OutRanges out) {
    using Lay = FewLayout<BN>;
    constexpr int ST = Lay::kStages;
    extern __shared__ uint8_t dyn[];
    uint8_t* smem = align_smem<1024>(dyn);
    __shared__ uint64_t full[ST], empty[ST], acc_full[kFewAccs], acc_empty[kFewAccs], drained, parts_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up;
#ifdef GDR_TEST_WAIT_LIMIT_NS
    __shared__ uint64_t never;
    if (threadIdx.x == 0) mbar_init(&never, 1);
#endif
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int tile = blockIdx.x / split, part = blockIdx.x - tile * split;
    const int n0 = tile * 128, m0 = blockIdx.y * BN;
    const int tokens = M - m0 < BN ? M - m0 : BN;
    const int g0 = (int)((int64_t)groups * part / split), g1 = (int)((int64_t)groups * (part + 1) / split);
    const int count = g1 - g0;
    const int quads = (tokens + 3) >> 2;
    const int owned = quads > part ? (quads - part + split - 1) / split : 0;     // quads part, part + split, ...

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
        for (int i = 0; i < kFewAccs; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], 4); }
        mbar_init(&drained, 1);
        mbar_init(&parts_bar, 1);
        gave_up = 0;
        fence_mbar_init();
        if (split > 1) mbar_arrive_expect_tx(&parts_bar, (uint32_t)(owned * split) * Lay::kPartBytes);
    }
    // Every CTA's barrier must be ready for its peers' parts.  TMEM is held only
    // where no other CTA or kernel is waited for (from the previous kernel's end to the
    // sums), so that clusters which share SMs cannot wait for each other's columns, nor
    // a previous kernel, which may let this one start before it allocates, for this
    // one's.  The loads start beside the allocation (some 320 cycles).
    __syncwarp();
    if (split > 1) cluster_sync();
    else __syncthreads();
    pdl_wait();
    bool parts_due = false;              // this warp gave up its wait for the parts
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (warp_wait(bar, parity)) return true;
        gave_up = 1;
        return false;
    };
    if (warp == 4) {
        int i = 0;
        // the first loads need no TMEM; no wait with a limit starts before it is there
        bool allocated = false;
        const auto after_alloc = [&] {
            if (!allocated) asm volatile("bar.sync 2, 192;" ::: "memory");
            allocated = true;
        };
        for (int s = 0, phase = 1; i < count; ++i) {
            if (i == ST) after_alloc();
            if (GDR_TEST_STALLS(1, i) || (part % 2 == 1 && GDR_TEST_STALLS(2, i)) ||
                (i >= ST && !wait(&empty[s], phase))) break;
            if (elect_one()) {
                uint8_t* st = smem + s * Lay::kStageBytes;
                mbar_arrive_expect_tx(&full[s], Lay::kStageBytes);
                tma_load_2d(st, &map_w, (g0 + i) * kFp8Group, n0, &full[s]);
                tma_load_2d(st + 16384, &map_x, (g0 + i) * kFp8Group, m0, &full[s]);
            }
            __syncwarp();
            if (++s == ST) { s = 0; phase ^= 1; }
        }
        // no copy may still be in flight when the CTA ends, whichever role gave up
        after_alloc();
        for (int j = i < ST ? 0 : i - ST; j < i; ++j) drain_wait(&full[j % ST], (j / ST) & 1);
    } else if (warp == 5) {
        constexpr uint32_t idesc = idesc_e4m3_f32(128, BN);
        tmem_alloc(&tmem_slot, Lay::kTmemCols);
        pdl_launch_dependents();                             // not before: the next kernel may want TMEM too
        __syncwarp();
        tc_fence_before_sync();
        asm volatile("bar.arrive 2, 192;" ::: "memory");     // for the other warps
        const uint32_t tmem = *(volatile uint32_t*)&tmem_slot;
        for (int i = 0, s = 0, phase = 0; i < count; ++i) {
            const int buf = (unsigned)i % kFewAccs;
            if (GDR_TEST_STALLS(0, i) || !wait(&full[s], phase) ||
                (i >= kFewAccs && !wait(&acc_empty[buf], (((unsigned)i / kFewAccs) & 1) ^ 1))) break;
            tc_fence_after_sync();
            if (elect_one()) {
                const uint32_t a = smem_u32(smem + s * Lay::kStageBytes);
#pragma unroll
                for (int j = 0; j < 4; ++j)      // 32 codes = 32 bytes = 16 of the descriptor's 2-byte columns
                    mma_e4m3(tmem + buf * BN, sw128_desc(a, 128, 0, 16 * j),
                             sw128_desc(a + 16384, BN, 0, 16 * j), idesc, j > 0);
                mma_commit(&empty[s]);
                mma_commit(&acc_full[buf]);
            }
            __syncwarp();
            if (++s == ST) { s = 0; phase ^= 1; }
        }
        __syncwarp();
        asm volatile("bar.sync 1, 160;" ::: "memory");       // warps 0-3 have read their sums
        tc_fence_after_sync();
        if (*(volatile int*)&gave_up) {                      // this warp, or one of them: MMAs may be under way
            if (elect_one()) mma_commit(&drained);           // a commit counts its own thread's MMAs only
            drain_wait(&drained, 0);
            __syncwarp();
        }
        tmem_dealloc(tmem, Lay::kTmemCols);
    } else {
        float acc[BN];
#pragma unroll
        for (int m = 0; m < BN; ++m) acc[m] = 0.f;
        float* factors = reinterpret_cast<float*>(smem + Lay::kFactors) + warp * 2 * BN;
        constexpr int kPer = (BN + 31) / 32, kLoad = BN < 32 ? BN : 32;
        float next[kPer];
        const float* swp = sw + (int64_t)tile * groups;
        const auto fetch = [&](int g) {
            const float w = __ldg(swp + g);
#pragma unroll
            for (int p = 0; p < kPer; ++p) {
                const int m = p * 32 + lane;
                next[p] = m < tokens ? __ldg(sx + (int64_t)(m0 + m) * groups + g) * w : 0.f;
            }
        };
        fetch(g0);
        const OutColumn o(out, n0 + threadIdx.x);    // while the first loads are on their way
        asm volatile("bar.sync 2, 192;" ::: "memory");       // warp 5 has allocated
        tc_fence_after_sync();
        const uint32_t tmem = *(volatile uint32_t*)&tmem_slot;
        for (int i = 0; i < count; ++i) {
            const int buf = (unsigned)i % kFewAccs;
            float* f = factors + (i & 1) * BN;
#pragma unroll
            for (int p = 0; p < kPer; ++p)
                if (BN >= 32 || lane < BN) f[p * 32 + lane] = next[p];
            if (i + 1 < count) fetch(g0 + i + 1);
            __syncwarp();
            if (GDR_TEST_STALLS(3, i) || !wait(&acc_full[buf], ((unsigned)i / kFewAccs) & 1)) break;
            tc_fence_after_sync();
            const uint32_t at = tmem + ((uint32_t)(warp * 32) << 16) + buf * BN;
            float d[BN / kLoad][kLoad];
#pragma unroll
            for (int c = 0; c < BN / kLoad; ++c) tmem_ld(at + c * kLoad, d[c]);
#pragma unroll
            for (int c = 0; c < BN / kLoad; ++c) {
                tmem_ld_wait_for(d[c]);
#pragma unroll
                for (int q = 0; q < kLoad; q += 4) {
                    const float4 w = *reinterpret_cast<const float4*>(f + c * kLoad + q);
                    float* o = acc + c * kLoad + q;
                    o[0] = fmaf(d[c][q], w.x, o[0]);
                    o[1] = fmaf(d[c][q + 1], w.y, o[1]);
                    o[2] = fmaf(d[c][q + 2], w.z, o[2]);
                    o[3] = fmaf(d[c][q + 3], w.w, o[3]);
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
        }
        tc_fence_before_sync();
        asm volatile("bar.arrive 1, 160;" ::: "memory");
        if (split == 1) {
            if (o.pitch)
#pragma unroll
                for (int m = 0; m < BN; ++m)
                    if (m < tokens) o.store(m0 + m, acc[m]);
        } else {
            const uint32_t to = smem_u32(smem + Lay::kParts) + part * Lay::kPartBytes + threadIdx.x * 16;
            const uint32_t bar = smem_u32(&parts_bar);
            int owner = 0, slot = 0;                 // of quad q: q % split, q / split
#pragma unroll
            for (int q = 0; q < Lay::kGroups; ++q) {
                if (q < quads)
                    st_async4(cluster_addr(to + slot * split * Lay::kPartBytes, owner),
                              make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]),
                              cluster_addr(bar, owner));
                if (++owner == split) { owner = 0; ++slot; }
            }
            parts_due = owned > 0 && !warp_wait<true>(&parts_bar, 0);
            if (owned > 0 && !parts_due) {
                const float4* parts = reinterpret_cast<const float4*>(smem + Lay::kParts) + threadIdx.x;
                for (int j = 0; j < owned; ++j) {
                    float4 v = parts[(j * split) * 128];
                    for (int r = 1; r < split; ++r) {
                        const float4 p = parts[(j * split + r) * 128];
                        v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
                    }
                    const int m = (part + j * split) * 4;
                    if (o.pitch) {
                        o.store(m0 + m, v.x);
                        if (m + 1 < tokens) o.store(m0 + m + 1, v.y);
                        if (m + 2 < tokens) o.store(m0 + m + 2, v.z);
                        if (m + 3 < tokens) o.store(m0 + m + 3, v.w);
                    }
                }
            }
        }
    }
    if (split > 1) {
        // no CTA may end while a part is on its way to it; owners have waited for
        // theirs, so nothing else has to be ordered here.  Every CTA sends all its
        // parts, whatever it gave up, so after this they have at least been sent.
        __syncwarp();
        asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
        if (parts_due) drain_wait(&parts_bar, 0);
    }
}

// ---------------------------------------------------------------------------
// Many tokens: CTA pairs on tiles of 256 tokens x NT columns.  Each CTA loads
// 128 tokens and half of the columns per K group (32 KB at NT 256; two single CTAs
// on 128 x 256 tiles would pull 96 KB through L2), holds its 128 tokens x NT columns
// in TMEM, 512 / NT times, and adds each finished group into registers with its
// factor.
//   warps 0-7   a thread owns a token (row) and one half of the tile's columns, which
//               lie in one weight block: a group's factor sx sw is one number per
//               thread
//   warp 8      TMA loads
//   warps 9, 10 (even CTA) the MMAs: of one half each at NT 256, of every other group
//               at NT 128
//   warp 11     stores the outputs that warps 0-7 leave in shared memory, while
//               they are at the next tile
// The way from an MMA's end through the register sums to the next MMA into the same
// columns (commit, sums, arrival at the even CTA: about 750 cycles) has to fit into
// the MMA time of the rest of TMEM.  At NT 256 (two accumulators) it bounds the
// kernel; each half of an accumulator has its own barriers and issuing warp there, so
// that a half waits for itself only (whole accumulators were 3 % slower).  At NT 128
// (four) the 24 KB a group that a CTA takes in at about 61 bytes a cycle do.  NT 128 is
// for products whose tiles do not fill the SMs (512 x 4096 x 4096: 13.4 us against
// 16.6; 8192 x 4096 x 4096: 159 against 127).  Long runs are held at 1.3 GHz by the
// power limit.  Persistent: a pair takes tiles a grid stride apart.
// ---------------------------------------------------------------------------
constexpr int kPairThreads = 384;
constexpr int kPairRowGroup = 8;                             // token tiles that take their column tiles together

template <int NT>
struct PairLayout {
    static constexpr bool kSplit = NT == 256;                // an issuing warp per half
    static constexpr int kHalf = NT / 2;                     // columns of a CTA's loads and of an adder's sums
    static constexpr int kAccs = 512 / NT;                   // TMEM accumulators, of two halves each
    static constexpr int kStages = NT == 256 ? 5 : 6;
    static constexpr uint32_t kStageBytes = 16384u + kHalf * 128u;
    static constexpr uint32_t kSlots = kStages * kStageBytes;
    static constexpr uint32_t kSlotBytes = 32768u;           // 128 rows x 256 bytes of outputs, per half
    static constexpr uint32_t kBytes = kSlots + 2u * kSlotBytes;
    static constexpr uint32_t kDynBytes = kBytes + 1024u;
};

// acc += f * v, two columns per instruction.
template <int N>
__device__ __forceinline__ void add_scaled(float2* acc, const float (&v)[N], float2 f) {
#pragma unroll
    for (int q = 0; q < N / 2; ++q) acc[q] = __ffma2_rn(make_float2(v[2 * q], v[2 * q + 1]), f, acc[q]);
}

// Tile t of a tile grid: bands of kPairRowGroup token tiles, column by column,
// so that the tiles in flight share few rows of x and of w in L2.
__device__ __forceinline__ void pair_tile(int t, int tiles_m, int tiles_n, int* tm, int* tn) {
    const int band = t / (kPairRowGroup * tiles_n);
    const int first = band * kPairRowGroup;
    const int rows = tiles_m - first < kPairRowGroup ? tiles_m - first : kPairRowGroup;
    const int r = t - first * tiles_n;
    *tn = r / rows;
    *tm = first + (r - *tn * rows);
}

// Where the 16-byte chunk c (0 .. 15) of a row's 256 bytes lies in an output slot:
// two boxes of 128 rows x 128 bytes, 128-byte swizzle (no bank conflicts, and the
// layout a TMA store reads).
__device__ __forceinline__ uint32_t slot_chunk(int row, int c) {
    return (uint32_t)((c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}

// The tensors of the output ranges; a range whose base or rows are not 16-byte
// aligned has none.
struct OutMaps {
    CUtensorMap map[GDR_LINEAR_MAX_OUTS];
    int valid[GDR_LINEAR_MAX_OUTS];
};

// A warp's view of the output ranges, a lane per range: what a block of columns is
// then takes a vote instead of a walk through the parameters (which took the store
// warp 900 cycles a block, longer than a short K's sums).
struct RangeLane {
    int begin, end;
    bool f32, mapped, last;
    __device__ __forceinline__ RangeLane(const OutRanges& out, const OutMaps& maps, int lane)
        : begin(0), end(0), f32(false), mapped(false), last(lane == out.n_outs - 1) {
        if (lane < out.n_outs) {
            begin = out.begin[lane];
            end = out.begin[lane + 1];
            f32 = out.f32[lane] != 0;
            mapped = maps.valid[lane] != 0;
        }
    }
    // Whether any of the `cols` columns from c0 on goes to an fp32 tensor: their outputs
    // then pass through shared memory as fp32 (64 columns at a time), otherwise as bf16.
    __device__ __forceinline__ bool wide(int c0, int cols) const {
        return __any_sync(0xffffffffu, f32 && begin < c0 + cols && end > c0);
    }
    // The range that a slot of outputs goes to by TMA (`cols` columns from c0, all in
    // one range with a map, at a 16-byte boundary of its rows, where a TMA store has to
    // start, and not before the range, where it may not), or -1.  What lies past the
    // last range's columns is dropped by the store.
    __device__ __forceinline__ int slot_range(bool is_wide, int c0, int cols) const {
        const bool mine = begin <= c0 && c0 < end && (c0 + cols <= end || last) && f32 == is_wide && mapped &&
                          ((c0 - begin) * (is_wide ? 4 : 2) & 15) == 0;
        return __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
    }
};

// The other slots: a warp's 32 rows (from `first` of the CTA's 128), a lane per
// column.
__device__ __forceinline__ void store_rows(const OutRanges& out, const uint8_t* slot, bool wide, int c0, int cols,
                                           int row0, int first, int M, int lane) {
    const int rows = M - row0 - first < 32 ? M - row0 - first : 32;
    const int elem = wide ? 4 : 2;
    for (int q = lane; q < cols; q += 32) {
        const OutColumn o(out, c0 + q);
        if (!o.pitch) continue;
        const int chunk = q * elem >> 4, in = q * elem & 15;
        const uint8_t* at = slot + (chunk >> 3) * 16384 + first * 128 + in;
        const int64_t pitch = o.pitch;
        const int64_t start = (int64_t)(row0 + first) * pitch;
        if (!wide) {
            uint16_t* p = (uint16_t*)o.p + start;
#pragma unroll 8
            for (int j = 0; j < rows; ++j)
                p[j * pitch] = *reinterpret_cast<const uint16_t*>(at + j * 128 + (((chunk & 7) ^ (j & 7)) << 4));
        } else if (o.f32) {
            float* p = (float*)o.p + start;
#pragma unroll 8
            for (int j = 0; j < rows; ++j)
                p[j * pitch] = *reinterpret_cast<const float*>(at + j * 128 + (((chunk & 7) ^ (j & 7)) << 4));
        } else {
            __nv_bfloat16* p = (__nv_bfloat16*)o.p + start;
#pragma unroll 8
            for (int j = 0; j < rows; ++j)
                p[j * pitch] = __float2bfloat16_rn(
                    *reinterpret_cast<const float*>(at + j * 128 + (((chunk & 7) ^ (j & 7)) << 4)));
        }
    }
}

// After its loading warp gave up, on the even CTA, whose `full` barriers count both
// CTAs' loads: wait for all that were issued (`mine` groups here, *peers_plus_1 - 1 by
// the odd CTA, once its loading warp ended).  The CTAs may have stopped at different
// groups, at most STAGES apart: a stage is loaded anew only after both CTAs' last loads
// of it were used, so all but the last STAGES loads have landed.  Bytes that this CTA
// announced for loads its peer never made are taken off the barrier, and loads that
// only the peer made are announced.  (If this warp did not give up, it saw every stage
// used: both CTAs' loads have landed.)
template <int STAGES>
__device__ void drain_pair_loads(uint64_t* full, uint32_t stage_bytes, int mine, const volatile int* peers_plus_1) {
    const uint64_t t0 = global_timer_ns();
    while (*peers_plus_1 == 0)
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            atomicOr(&g_linear_error, 2u);
            return;
        }
    const int peers = *peers_plus_1 - 1;
    const int last = mine > peers ? mine : peers;
    for (int j = last < STAGES ? 0 : last - STAGES; j < last; ++j) {
        uint64_t* bar = &full[j % STAGES];
        if (j >= peers) mbar_complete_tx(bar, stage_bytes);
        if (j >= mine) mbar_arrive_expect_tx(bar, stage_bytes);
        drain_wait(bar, (j / STAGES) & 1);
    }
}

template <int NT>
__global__ void __launch_bounds__(kPairThreads, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                   const float* __restrict__ sx, const float* __restrict__ sw, int M, int N, int groups,
                   int tiles_m, int tiles_n, const __grid_constant__ OutRanges out,
                   const __grid_constant__ OutMaps maps) {
    using Lay = PairLayout<NT>;
    constexpr int ST = Lay::kStages, A = Lay::kAccs, H = Lay::kHalf;
    extern __shared__ uint8_t dyn[];
    uint8_t* smem = align_smem<1024>(dyn);
    __shared__ uint64_t full[ST], empty[ST];
    __shared__ uint64_t acc_full[2 * A], acc_empty[2 * A];   // 2 * accumulator + half (not split: half 0 for both)
    __shared__ uint64_t slot_full[2], slot_free[2], drained[2];
    __shared__ uint32_t tmem_slot;
    __shared__ int peers_plus_1;                             // even CTA: groups that the odd one loaded, + 1
#ifdef GDR_TEST_WAIT_LIMIT_NS
    __shared__ uint64_t never;
    if (threadIdx.x == 0) mbar_init(&never, 1);
#endif
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int tiles = tiles_m * tiles_n;

    if (threadIdx.x == 0) {
        // full: the even CTA's, one arrival (its producer) and both CTAs' bytes;
        // empty: a commit of each MMA warp that reads the stage; acc_empty: the
        // even CTA's, four warps of each CTA for a half
        for (int i = 0; i < ST; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], Lay::kSplit ? 2 : 1); }
        for (int i = 0; i < 2 * A; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], Lay::kSplit ? 8 : 16); }
        for (int i = 0; i < 2; ++i) { mbar_init(&slot_full[i], 4); mbar_init(&slot_free[i], 1); mbar_init(&drained[i], 1); }
        peers_plus_1 = 0;
        fence_mbar_init();
    }
    __syncwarp();
    cluster_sync();
    // Wait, allocation, start of the next kernel: in this order, as in the few-token
    // kernel.  Every warp takes up both CTAs' allocation (tmem_ready) before its first
    // wait with a limit and after what needs no TMEM.
    pdl_wait();
    if (warp == 9) {
        tmem_alloc_pair(&tmem_slot, 512);
        pdl_launch_dependents();
        __syncwarp();
    }
    tc_fence_before_sync();
    cluster_arrive();
    const auto tmem_ready = [&] {
        cluster_wait();
        tc_fence_after_sync();
        return *(volatile uint32_t*)&tmem_slot;
    };

    // registers: 256 threads x 216 + 128 x 72 = the launch's 384 x 168
    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const auto wait = [](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity); };
    if (warp == 8) {
        int i = 0, s = 0, phase = 1;
        bool ok = true, allocated = false;
        const auto after_alloc = [&] {
            if (!allocated) tmem_ready();
            allocated = true;
        };
        for (int t = pair; t < tiles && ok; t += pairs) {
            int tm, tn;
            pair_tile(t, tiles_m, tiles_n, &tm, &tn);
            const int m0 = tm * 256 + (int)rank * 128, n0 = tn * NT + (int)rank * 64;
            for (int g = 0; g < groups; ++g, ++i) {
                if (i == ST) after_alloc();
                if (GDR_TEST_STALLS(1, i) || GDR_TEST_STALLS(rank == 1 ? 2 : 5, i) ||
                    (i >= ST && !wait(&empty[s], phase))) { ok = false; break; }
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * Lay::kStageBytes);
                    const uint32_t bar = cluster_addr(smem_u32(&full[s]), 0);
                    uint8_t* st = smem + s * Lay::kStageBytes;
                    tma_load_2d_pair(st, &map_x, g * kFp8Group, m0, bar);
                    tma_load_2d_pair(st + 16384, &map_w, g * kFp8Group, n0, bar);
                    if (Lay::kSplit) tma_load_2d_pair(st + 24576, &map_w, g * kFp8Group, n0 + H, bar);
                }
                __syncwarp();
                if (++s == ST) { s = 0; phase ^= 1; }
            }
        }
        after_alloc();
        // the last stages' releases must have landed before this CTA's shared memory goes
        for (int j = i < ST ? 0 : i - ST; j < i && ok; ++j) ok = wait(&empty[j % ST], (j / ST) & 1);
        if (lane == 0) {
            if (rank == 1) st_cluster(cluster_addr(smem_u32(&peers_plus_1), 0), i + 1);
            else if (!ok) drain_pair_loads<ST>(full, Lay::kStageBytes, i, &peers_plus_1);
        }
        __syncwarp();
    } else if (warp == 9 || warp == 10) {
        const uint32_t tmem = tmem_ready();
        if (rank == 0) {
            // 128 columns at a time: of half `mine` in every group, or of every group
            // whose last bit is `mine`
            constexpr uint32_t idesc = idesc_e4m3_f32(256, 128);
            const int mine = warp - 9;
            int i = 0, s = 0, phase = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                for (int g = 0; g < groups; ++g, ++i) {
                    if (Lay::kSplit || (i & 1) == mine) {
                        const int buf = (unsigned)i % A, half = Lay::kSplit ? mine : 0;
                        if (GDR_TEST_STALLS(0, i) || !wait(&full[s], phase) ||
                            (i >= A && !wait(&acc_empty[2 * buf + half], (((unsigned)i / A) & 1) ^ 1))) { ok = false; break; }
                        tc_fence_after_sync();
                        if (elect_one()) {
                            const uint32_t a = smem_u32(smem + s * Lay::kStageBytes);
#pragma unroll
                            for (int j = 0; j < 4; ++j)      // 32 codes = 16 of the descriptor's 2-byte columns
                                mma_e4m3_pair(tmem + buf * NT + half * 128, sw128_desc(a, 128, 0, 16 * j),
                                              sw128_desc(a + 16384 + half * 8192, 64, 0, 16 * j), idesc, j > 0);
                            mma_commit_pair(&acc_full[2 * buf + half]);
                            mma_commit_pair(&empty[s]);
                        }
                        __syncwarp();
                    }
                    if (++s == ST) { s = 0; phase ^= 1; }
                }
            }
            // no MMA may still be under way when tensor memory is released, whichever role
            // gave up; a commit counts its own thread's MMAs only
            if (elect_one()) mma_commit_pair(&drained[mine]);
            drain_wait(&drained[mine], 0);
        }
    } else if (warp == 11) {
        // A slot is given back once its store has read it; while a store is under way
        // the other slot's is started (`pending`: the slot still to be given back).
        // The warp blocks on a slot only when it owes none, so no adder can wait for it
        // in a circle.
        int jobs[2] = {0, 0}, pending = -1;
        bool ok = true;
        const auto give_back = [&] {
            if (pending >= 0 && elect_one()) {
                bulk_wait_group_read0();
                mbar_arrive(&slot_free[pending]);
            }
            __syncwarp();
            pending = -1;
        };
        const RangeLane ranges(out, maps, lane);
        tmem_ready();
        for (int t = pair; t < tiles && ok; t += pairs) {
            int tm, tn;
            pair_tile(t, tiles_m, tiles_n, &tm, &tn);
            const int row0 = tm * 256 + (int)rank * 128;
            const bool wides[2] = {ranges.wide(tn * NT, H), ranges.wide(tn * NT + H, H)};
            for (int q = 0; q < H && ok; q += 64) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const bool wide = wides[half];
                    if (!ok || (q > 0 && !wide)) continue;
                    const int cols = wide ? 64 : H, c = tn * NT + half * H + q;
                    const int r = ranges.slot_range(wide, c, cols);
                    if (r < 0) continue;                     // past the columns, or warps 0-7 store it
                    if (pending >= 0 && !__all_sync(0xffffffffu, mbar_test_wait(smem_u32(&slot_full[half]), jobs[half] & 1)))
                        give_back();
                    if (GDR_TEST_STALLS(4, jobs[0] + jobs[1]) || !wait(&slot_full[half], jobs[half] & 1)) { ok = false; break; }
                    if (elect_one()) {
                        const int off = c - out.begin[r], box = wide ? 32 : 64;
                        const uint8_t* slot = smem + Lay::kSlots + half * Lay::kSlotBytes;
                        if (row0 < M) {                      // a box starts inside its tensor
                            tma_store_2d(&maps.map[r], slot, off, row0);
                            if (box < cols && c + box < out.begin[r + 1]) tma_store_2d(&maps.map[r], slot + 16384, off + box, row0);
                        }
                        bulk_commit_group();
                        if (pending >= 0) {
                            bulk_wait_group_read<1>();
                            mbar_arrive(&slot_free[pending]);
                        }
                    }
                    __syncwarp();
                    pending = half;
                    ++jobs[half];
                }
            }
        }
        give_back();
        if (elect_one()) bulk_wait_group0();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int half = warp >> 2;                          // columns half * H .. + H - 1 of the tile
        const int row = (warp & 3) * 32 + lane;              // row of the CTA's 128
        uint8_t* slot = smem + Lay::kSlots + half * Lay::kSlotBytes;
        const int side = Lay::kSplit ? half : 0;
        const uint32_t bars = cluster_addr(smem_u32(&acc_empty[side]), 0);
        const bool vec = (groups & 3) == 0 &&
                         ((reinterpret_cast<uint64_t>(sx) | reinterpret_cast<uint64_t>(sw)) & 15) == 0;
        int i = 0, jobs = 0;
        bool ok = true;
        // this tile's factor rows; the first four groups' factors are fetched a tile ahead
        const float *sxp = sx, *swp = sw;
        int c0 = 0, m0 = 0;
        float4 nx, nw;
        const auto fetch = [&](int g) {
            if (vec) {
                nx = __ldg(reinterpret_cast<const float4*>(sxp + g));
                nw = __ldg(reinterpret_cast<const float4*>(swp + g));
            } else {
                const int last = groups - 1;
                nx = make_float4(__ldg(sxp + g), __ldg(sxp + min(g + 1, last)), __ldg(sxp + min(g + 2, last)),
                                 __ldg(sxp + min(g + 3, last)));
                nw = make_float4(__ldg(swp + g), __ldg(swp + min(g + 1, last)), __ldg(swp + min(g + 2, last)),
                                 __ldg(swp + min(g + 3, last)));
            }
        };
        const RangeLane ranges(out, maps, lane);
        int tm = 0, tn = 0;                                  // the tile that enter() goes to
        const auto enter = [&] {
            m0 = tm * 256 + (int)rank * 128;
            const int m = m0 + row;
            c0 = tn * NT + half * H;
            sxp = sx + (int64_t)(m < M ? m : 0) * groups;
            swp = sw + (int64_t)(c0 < N ? c0 / kFp8Group : 0) * groups;
            fetch(0);
        };
        if (pair < tiles) {
            pair_tile(pair, tiles_m, tiles_n, &tm, &tn);
            enter();
        }
        const uint32_t at0 = tmem_ready() + ((uint32_t)((warp & 3) * 32) << 16) + half * H;
        for (int t = pair; t < tiles && ok; t += pairs) {
            const int c_out = c0, m_tile = m0;
            const bool wide = ranges.wide(c_out, H);
            if (t + pairs < tiles) pair_tile(t + pairs, tiles_m, tiles_n, &tm, &tn);
            float2 acc[H / 2];
#pragma unroll
            for (int c = 0; c < H / 2; ++c) acc[c] = make_float2(0.f, 0.f);
            float4 fs = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int g = 0; g < groups; ++g, ++i) {
                const int buf = (unsigned)i % A;
                if ((g & 3) == 0) {
                    fs = make_float4(nx.x * nw.x, nx.y * nw.y, nx.z * nw.z, nx.w * nw.w);
                    if (g + 4 < groups) fetch(g + 4);
                }
                const float2 f = make_float2(fs.x, fs.x);
                fs.x = fs.y;
                fs.y = fs.z;
                fs.z = fs.w;
                if (GDR_TEST_STALLS(3, i) || !wait(&acc_full[2 * buf + side], ((unsigned)i / A) & 1)) { ok = false; break; }
                tc_fence_after_sync();
                const uint32_t at = at0 + buf * NT;
                // the next load under way while one is added
                float u[32], v[16];
                tmem_ld32(at, u);
                tmem_ld_wait_for(u);
                tmem_ld16(at + 32, v);
                add_scaled<32>(acc, u, f);
                tmem_ld_wait_for(v);
                if constexpr (H == 128) {            // 32 + 16 + 32 + 16 + 32 columns
                    tmem_ld32(at + 48, u);
                    add_scaled<16>(acc + 16, v, f);
                    tmem_ld_wait_for(u);
                    tmem_ld16(at + 80, v);
                    add_scaled<32>(acc + 24, u, f);
                    tmem_ld_wait_for(v);
                    tmem_ld32(at + 96, u);
                    add_scaled<16>(acc + 40, v, f);
                    tmem_ld_wait_for(u);
                    add_scaled<32>(acc + 48, u, f);
                } else {                             // 32 + 16 + 16
                    float w[16];
                    tmem_ld16(at + 48, w);
                    add_scaled<16>(acc + 16, v, f);
                    tmem_ld_wait_for(w);
                    add_scaled<16>(acc + 24, w, f);
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(bars + buf * 16);
            }
            if (t + pairs < tiles) enter();
            if (!ok || c_out >= N) continue;
            const int cols = wide ? 64 : H;
#pragma unroll
            for (int q = 0; q < H; q += 64) {
                if (q >= 64 && !wide) break;
                // the slot's last TMA store has read it
                if (jobs > 0 && !wait(&slot_free[half], (jobs - 1) & 1)) { ok = false; break; }
                if (wide) {
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        *reinterpret_cast<float4*>(slot + slot_chunk(row, c)) =
                            make_float4(acc[q / 2 + 2 * c].x, acc[q / 2 + 2 * c].y, acc[q / 2 + 2 * c + 1].x,
                                        acc[q / 2 + 2 * c + 1].y);
                } else {
#pragma unroll
                    for (int c = 0; c < H / 8; ++c)
                        *reinterpret_cast<uint4*>(slot + slot_chunk(row, c)) =
                            make_uint4(pack_bf16(acc[4 * c].x, acc[4 * c].y), pack_bf16(acc[4 * c + 1].x, acc[4 * c + 1].y),
                                       pack_bf16(acc[4 * c + 2].x, acc[4 * c + 2].y), pack_bf16(acc[4 * c + 3].x, acc[4 * c + 3].y));
                }
                const int c = c_out + q;
                if (ranges.slot_range(wide, c, cols) >= 0) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&slot_full[half]);
                    ++jobs;
                } else {
                    __syncwarp();
                    store_rows(out, slot, wide, c, cols, m_tile, (warp & 3) * 32, M, lane);
                    __syncwarp();
                }
            }
        }
    }
    __syncthreads();
    cluster_sync();
    if (warp == 9) tmem_dealloc_pair(tmem_slot, 512);
    __syncwarp();
    cluster_sync();
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, fetched through the runtime once.
cudaError_t tensor_map_encoder(EncodeTiledFn* fn) {
    static EncodeTiledFn cached = nullptr;
    if (!cached) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (q != cudaDriverEntryPointSuccess || p == nullptr) return cudaErrorSymbolNotFound;
        cached = reinterpret_cast<EncodeTiledFn>(p);
    }
    *fn = cached;
    return cudaSuccess;
}

// Map of [rows][k] codes, box `box_rows` rows x 128 codes, 128-byte swizzle;
// rows and codes past the tensor's ends read as zero.
cudaError_t codes_map(EncodeTiledFn enc, CUtensorMap* m, const void* base, int64_t rows, int k, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)k};
    const cuuint32_t box[2] = {(cuuint32_t)kFp8Group, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1u, 1u};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
                           estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Map of an output tensor [rows][cols], box 128 rows x 128 bytes, 128-byte swizzle.
cudaError_t out_map(EncodeTiledFn enc, CUtensorMap* m, void* base, int64_t rows, int cols, int elem) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)cols * elem};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / elem), 128u};
    const cuuint32_t estr[2] = {1u, 1u};
    const CUresult r = enc(m, elem == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base,
                           dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Launch with the cluster size and programmatic stream serialization.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster,
                           cudaStream_t st, Args&&... args) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

OutRanges out_ranges(const gdr_linear_fp8_args& a) {
    OutRanges o{};
    o.n_outs = a.n_outs;
    for (int i = 0; i < a.n_outs; ++i) {
        o.begin[i + 1] = o.begin[i] + a.out_cols[i];
        o.f32[i] = a.out_dtype[i] == GDR_F32;
        o.ptr[i] = a.out[i];
    }
    return o;
}

template <int BN>
cudaError_t launch_few(const gdr_linear_fp8_args& a, EncodeTiledFn enc, cudaStream_t st) {
    const int groups = fp8_groups(a.k), tiles = fp8_groups(a.n);
    const int64_t token_tiles = (a.rows + BN - 1) / BN;
    if (token_tiles > 65535) return cudaErrorInvalidValue;
    // K in a power of two of parts, none without work: as many as fill the SMs once
    // (4096 x 4096 for one token: 5.7 us, filled twice 7.3; for 36 tokens, eight groups
    // a CTA, 7.9 and 9.4; the next kernel's start then overlaps this one), and twice
    // where a CTA would otherwise have 32 groups or more of 64 tokens to add up (16416
    // columns for 36 tokens, K 8192: 27.8 against 32.9 us; K 4096, where the groups
    // just reach that, 17.2 against 17.7, but 19.6 against 18.7 for 64 tokens).
    int split = 1;
    while (split < 8 && 2 * split <= groups) {
        const int64_t ctas = 2 * split * tiles * token_tiles;
        if (ctas > kSms && !(BN == 64 && groups >= 32 * split && ctas <= 2 * kSms)) break;
        split *= 2;
    }
    if ((int64_t)tiles * split > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
    CUtensorMap mw, mx;
    cudaError_t e;
    if ((e = codes_map(enc, &mw, a.w, a.n, a.k, 128)) != cudaSuccess) return e;
    if ((e = codes_map(enc, &mx, a.x, a.rows, a.k, BN)) != cudaSuccess) return e;
    return launch_cluster(linear_few_kernel<BN>, dim3((unsigned)(tiles * split), (unsigned)token_tiles),
                          dim3(kFewThreads), FewLayout<BN>::kDynBytes, split, st, mw, mx, a.x_scale,
                          a.w_scale, (int)a.rows, groups, split, out_ranges(a));
}

template <int NT>
cudaError_t launch_pair(const gdr_linear_fp8_args& a, EncodeTiledFn enc, cudaStream_t st) {
    const int groups = fp8_groups(a.k);
    const int64_t tiles_m = (a.rows + 255) / 256, tiles_n = ((int64_t)a.n + NT - 1) / NT;
    if (tiles_m * tiles_n > (int64_t)INT32_MAX - 1024) return cudaErrorInvalidValue;
    CUtensorMap mw, mx;
    cudaError_t e;
    if ((e = codes_map(enc, &mw, a.w, a.n, a.k, 64)) != cudaSuccess) return e;
    if ((e = codes_map(enc, &mx, a.x, a.rows, a.k, 128)) != cudaSuccess) return e;
    OutMaps maps;
    memset(&maps, 0, sizeof(maps));
    for (int i = 0; i < a.n_outs; ++i) {
        const int elem = a.out_dtype[i] == GDR_F32 ? 4 : 2;
        if ((int64_t)a.out_cols[i] * elem % 16 != 0 || (reinterpret_cast<uintptr_t>(a.out[i]) & 15u) != 0) continue;
        if ((e = out_map(enc, &maps.map[i], a.out[i], a.rows, a.out_cols[i], elem)) != cudaSuccess) return e;
        maps.valid[i] = 1;
    }
    const int64_t pairs = tiles_m * tiles_n < kSms / 2 ? tiles_m * tiles_n : kSms / 2;
    return launch_cluster(linear_pair_kernel<NT>, dim3((unsigned)(2 * pairs)), dim3(kPairThreads), PairLayout<NT>::kDynBytes, 2, st,
                          mw, mx, a.x_scale, a.w_scale, (int)a.rows, a.n, groups, (int)tiles_m, (int)tiles_n,
                          out_ranges(a), maps);
}

}  // namespace

cudaError_t launch_linear_fp8(const gdr_linear_fp8_args& a, cudaStream_t st) {
    EncodeTiledFn enc = nullptr;
    cudaError_t e = tensor_map_encoder(&enc);
    if (e != cudaSuccess) return e;
    if (a.rows <= 16) return launch_few<16>(a, enc, st);
    if (a.rows <= 32) return launch_few<32>(a, enc, st);
    // Up to 64 tokens, and more while the tiles of 64 tokens x 128 columns fill no more
    // than half of the SMs (K is then split: 128 x 4096 x 4096 12.0 us, on CTA pairs
    // 12.7), or all of them where K is short (256 x 3598 x 896: 6.4 against 7.1 us; 256 x
    // 4096 x 4096: 17.4 against 12.9).  Beyond that each weight would be fetched again
    // for every 64 tokens (256 x 16416 x 4096: 60 us against 22).
    const int64_t small_tiles = fp8_groups(a.n) * ((a.rows + 63) / 64);
    if (a.rows <= 64 || small_tiles <= kSms / 2 || (small_tiles <= kSms && fp8_groups(a.k) <= 12))
        return launch_few<64>(a, enc, st);
    // tiles of 256 x 128 where they fit the CTA pairs at once, else of 256 x 256
    if ((a.rows + 255) / 256 * fp8_groups(a.n) <= kSms / 2) return launch_pair<128>(a, enc, st);
    return launch_pair<256>(a, enc, st);
}

}  // namespace gdr

extern "C" gdr_status gdr_linear_fp8_status(void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &cs) != cudaSuccess || cs != cudaStreamCaptureStatusNone) {
        (void)cudaGetLastError();
        return GDR_ERR_CUDA;
    }
    uint32_t word = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&word, gdr::g_linear_error, sizeof(word), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess) {
        (void)cudaGetLastError();
        return GDR_ERR_CUDA;
    }
    if (word == 0) return GDR_OK;
    if (cudaMemcpyToSymbolAsync(gdr::g_linear_error, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess) {
        (void)cudaGetLastError();
        return GDR_ERR_CUDA;
    }
    return GDR_ERR_TIMEOUT;
}

#ifdef GDR_TEST_WAIT_LIMIT_NS
// The test copy's role that waits for nothing, and the error word as it is (cleared).
extern "C" int gdr_linear_fp8_test_role(int role) {
    return (int)cudaMemcpyToSymbol(gdr::g_linear_test_role, &role, sizeof(role));
}

extern "C" int gdr_linear_fp8_test_word(void) {
    uint32_t word = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&word, gdr::g_linear_error, sizeof(word)) != cudaSuccess ||
        cudaMemcpyToSymbol(gdr::g_linear_error, &zero, sizeof(zero)) != cudaSuccess) return -1;
    return (int)word;
}
#endif
