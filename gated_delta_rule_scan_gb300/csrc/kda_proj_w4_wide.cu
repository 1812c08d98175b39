// kda_proj_w4_wide.cu -- kda_proj_w4 for batches: the products on the tcgen05 tensor cores.
//
// Mathematics.  Codes minus 8 are whole numbers, exact in f16; x is scaled by a power of two per
// token (its largest magnitude to [2^7, 2^8)) and split into f16 hi + lo (22 significant bits; of a
// bf16 x hi alone, whose 8 bits are exact down to 2^-24 of that magnitude; both are off by at most
// 2^-32 of it below).  The tensor cores sum code * x over one group of G k into f32, and the
// group's scale multiplies that sum in f32:
//     acc[r][s] += c[r][g] * D_g[r][s] + (8 - z[r][g]) c[r][g] * xsum_g[s],
// so neither weights nor scales are ever rounded, whatever their type.  (The two terms are rounded
// apart: a group whose codes all equal its zero point leaves their rounding errors, not 0.)
//
// What bounds it: the codes' bytes from HBM up to about 48 rows, then the tensor cores (every
// product is made twice, for hi and lo).  Layout: a tile is 128 weight rows (the MMA's M = TMEM
// lanes) against all tokens of the block (N <= 128), in units of 128 k.  The warps have roles:
//   * one thread streams the codes of 128 rows x 128 k (8 KB, 64-byte swizzle) through a ring of
//     shared-memory stages, one the x images; one warp fetches the units' scales and zero points
//     (strided: a few bytes of each row) two units ahead;
//   * the dequantising warps read their row's codes (thread = row = TMEM lane, conflict-free
//     through the swizzle), turn 8 codes into four f16 pairs with nine instructions and store them
//     as the MMA's A operand in tensor memory, the warpgroups taking units in turn: shared memory
//     carries 4-bit codes only;
//   * one thread issues the MMAs, group by group, into two accumulators in turn;
//   * the epilogue warps read a finished group's accumulator and add it, scaled, to the f32 sums
//     that they hold in registers (thread = weight row, up to 64 tokens each).
// A unit passes through six hand-overs of 100 to 200 cycles each, against 512 cycles of MMAs at 64
// tokens: up to 64 tokens two blocks share an SM, so that one's hand-overs overlap the other's
// work (one block: MMAs alone 818 cycles a unit, epilogue 800, dequantising 570).
// Persistent blocks: the (tile, unit) pairs are dealt out evenly and in order, so a tile may be
// cut between blocks.  Its parts meet in the workspace, added in block order whoever adds them, so
// results do not depend on timing: usually the block that holds a tile's first units ends last,
// finds the other parts there, and adds them to its registers.
// At 64 heads x 6144 with groups of 128: 16 rows 34 us, 64 rows 45 (the tensor pipe active 41 % of
// the time), 256 rows 117 (60 %); of a bf16 x, half the products, 64 rows 43, 256 rows 101.
#include <cuda_fp16.h>

#include "kda_chunk_common.cuh"
#include "kda_device.cuh"
#include "kda_tc.cuh"

namespace kda {

namespace {

constexpr int kRows = 128;                     // weight rows of a tile
constexpr int kUnit = 128;                     // k of a unit: one stage of codes
constexpr int kGran = 64;                      // k of one x image row in shared memory (128 bytes)
constexpr int kCodeStage = kRows * kUnit / 2;  // 8 KB
constexpr int kMaxCodeStages = 8, kMaxXStages = 4, kMaxParStages = 8, kMaxABufs = 4;
constexpr int kBarBytes = 2048;                // barriers and token factors, in front of the stages
constexpr int kFactorAt = 1024;
constexpr int kTokBlock = 128;                 // tokens of one block at most

// One or two blocks on an SM.
template <int CTAS>
struct Cfg;
template <>
struct Cfg<1> {                                // 65 .. 128 tokens
    static constexpr int kDeqGroups = 3, kEpiGroups = 2, kABufs = 4, kCodeStages = 8;
    static constexpr int kTmem = 512, kDCols = 128;
    static constexpr int kDeqRegs = 56, kEpiRegs = 112;   // of 80: 384 * 24 >= 256 * 32
    static constexpr int kSmem = 226 * 1024;
};
template <>
struct Cfg<2> {                                // up to 64 tokens
    static constexpr int kDeqGroups = 2, kEpiGroups = 1, kABufs = 2, kCodeStages = 4;
    static constexpr int kTmem = 256, kDCols = 64;
    static constexpr int kDeqRegs = 40, kEpiRegs = 112;   // of 64: 256 * 24 = 128 * 48
    static constexpr int kSmem = 112 * 1024;
};
template <int CTAS>
__host__ __device__ constexpr int cfg_threads() {
    return 128 * (Cfg<CTAS>::kDeqGroups + Cfg<CTAS>::kEpiGroups + 1);
}
// stages of the ring of scales, zero terms and group sums of x
__host__ __device__ constexpr int par_stages(int group) { return group == 32 ? 4 : kMaxParStages; }

struct WideMaps {
    CUtensorMap w[kW4MaxWeights];
    CUtensorMap xh, xl;
};

struct WideParams {
    const void* scale[kW4MaxWeights];
    const void* zero[kW4MaxWeights];
    float* out[kW4MaxWeights];
    int rows[kW4MaxWeights];
    int tile_start[kW4MaxWeights + 1];
    int nw, t, in_f, scale_bf16, has_zero;
    int t_blk, t_rows;                         // tokens of a block (a multiple of 16), of the images
    int x_stages;
    int x_bf16;
    const float* tok_factor;                   // [t_rows] 2^(e - 7)
    const float* xsum;                         // [in_f / G][t_rows], in units of the factor
    float* partial;                            // [blocks][2][t_blk][128]
    int* counter;                              // [blocks][epilogue warps]: parts in the workspace
    int* err;
};

struct WideWs {
    size_t hi, lo, factor, counter, xsum, partial, total;
};
__host__ inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
// token blocks, tokens of a block, rows of the images
__host__ inline void token_blocks(int t, int& ny, int& t_blk) {
    ny = (t + kTokBlock - 1) / kTokBlock;
    t_blk = ((t + ny - 1) / ny + 15) / 16 * 16;
}
// blocks of a launch at most: two per SM up to 64 tokens
__host__ inline int max_blocks(int t_blk) { return t_blk <= 64 ? 2 * kW4MaxSms : kW4MaxSms; }
WideWs wide_ws(int t, int in_f) {
    int ny, t_blk;
    token_blocks(t, ny, t_blk);
    const size_t rows = (size_t)ny * t_blk;
    WideWs w;
    w.hi = 0;
    w.lo = w.hi + up256(rows * in_f * 2);
    w.factor = w.lo + up256(rows * in_f * 2);
    w.counter = w.factor + up256(rows * 4);
    w.xsum = w.counter + up256(kW4MaxBlocks * 8 * 4);
    w.partial = w.xsum + up256(rows * (in_f / 32) * 4);
    w.total = w.partial + (size_t)max_blocks(t_blk) * 2 * t_blk * kRows * 4;
    return w;
}

// ---- x into images --------------------------------------------------------------------------

// One block per image row: the token's largest magnitude, then hi and lo with each 8 k in the
// order in which a word's codes come out (0 4 1 5 2 6 3 7), and the group sums.  Thread = 8 k, kept
// in registers between the two passes when one round covers the row (in_f <= 8192).  Rows past t
// are zero.  Block 0 also clears the counters.
constexpr int kSplitThreads = 1024;
template <bool XBF16>
__global__ void __launch_bounds__(kSplitThreads) kda_proj_w4_split_kernel(
    const void* __restrict__ x, int t, int in_f, int group, int has_zero, int t_rows,
    __half* __restrict__ hi, __half* __restrict__ lo, float* __restrict__ factor,
    float* __restrict__ xsum, int* __restrict__ counter) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ uint32_t warp_max[kSplitThreads / 32];
    const int s = blockIdx.x, tid = threadIdx.x, threads = blockDim.x;
    if (s == 0)
        for (int i = tid; i < kW4MaxBlocks * 8; i += threads) counter[i] = 0;
    const int vecs = in_f / 8;
    uint4* h4 = reinterpret_cast<uint4*>(hi + (size_t)s * in_f);
    uint4* l4 = reinterpret_cast<uint4*>(lo + (size_t)s * in_f);
    const bool row_live = s < t;
    auto load8 = [&](int v, float (&f)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = 0.0f;
        if (v >= vecs || !row_live) return;
        if constexpr (XBF16) {
            const uint4 r = __ldg(reinterpret_cast<const uint4*>(x) + (size_t)s * vecs + v);
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[2 * j] = __uint_as_float(w[j] << 16);
                f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        } else {
            const float4* p = reinterpret_cast<const float4*>(x) + ((size_t)s * vecs + v) * 2;
            const float4 a = __ldg(p), b = __ldg(p + 1);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        }
    };
    uint32_t m = 0;
    float f[8];
    const int rounds = (vecs + threads - 1) / threads;
    for (int i = rounds - 1; i >= 0; --i) {      // the first round last: it stays in f
        load8(tid + i * threads, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0) warp_max[tid >> 5] = m;
    __syncthreads();
    m = (tid & 31) < threads / 32 ? warp_max[tid & 31] : 0u;
    m = __reduce_max_sync(0xffffffffu, m);
    // exponent of the largest magnitude, at least -100; a row that is not finite stays as it is
    const int e = max((int)(m >> 23) - 127, -100);
    const bool fin = m < 0x7f800000u;
    const float up = fin ? __uint_as_float((uint32_t)(127 + 7 - e) << 23) : 1.0f;
    if (tid == 0) factor[s] = fin ? __uint_as_float((uint32_t)(127 - 7 + e) << 23) : 1.0f;
    for (int i = 0; i < rounds; ++i) {
        const int v = tid + i * threads;
        if (i > 0) load8(v, f);
        float sum = 0.0f;
        __half a[8], b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float y = __fmul_rn(f[j], up);
            sum += y;
            const int at = j < 4 ? 2 * j : 2 * (j - 4) + 1;
            a[at] = __float2half_rn(y);
            b[at] = __float2half_rn(y - __half2float(a[at]));
        }
        if (v < vecs) {
            h4[v] = *reinterpret_cast<const uint4*>(a);
            if (!XBF16) l4[v] = *reinterpret_cast<const uint4*>(b);
        }
        if (has_zero) {
            for (int o = 1; o < group / 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (v < vecs && v % (group / 8) == 0) xsum[(size_t)(v / (group / 8)) * t_rows + s] = sum;
        }
    }
}

// ---- the products ---------------------------------------------------------------------------

// 8 codes as four f16 pairs of whole numbers -8 .. 7 (k order 0 4 | 1 5 | 2 6 | 3 7), each or-ed into
// the mantissa of 1024 (the publication named in kda_proj_w4.cu)
__device__ __forceinline__ void codes8(uint32_t w, uint32_t* o) {
    const __half2 k1032 = __float2half2_rn(1032.0f), k16 = __float2half2_rn(0.0625f),
                  k72 = __float2half2_rn(-72.0f);
#pragma unroll
    for (int h = 0; h < 2; ++h, w >>= 8) {
        const uint32_t a = (w & 0x000f000fu) | 0x64006400u, b = (w & 0x00f000f0u) | 0x64006400u;
        const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), k1032);
        const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&b), k16, k72);
        o[2 * h] = *reinterpret_cast<const uint32_t*>(&x);
        o[2 * h + 1] = *reinterpret_cast<const uint32_t*>(&y);
    }
}

// Barriers by shared-memory address.  A try that finds the phase complete costs about 60 cycles of
// latency, one that does not suspends the thread for up to 4 us; the limit is about a second.
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, int* err) {
    for (int n = 0; n < 250000; ++n)
        if (bar_try(bar, parity)) return true;
    if (err) atomicOr(err, kDevErrTimeout);
    return false;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, int* err) {
    return bar_try(bar, parity) || bar_wait_slow(bar, parity, err);
}
// Two or three barriers, tried together so that their latencies overlap.
__device__ __forceinline__ bool bar_wait2(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, int* err) {
    const bool r0 = bar_try(b0, p0), r1 = bar_try(b1, p1);
    if (r0 && r1) return true;
    return (r0 || bar_wait_slow(b0, p0, err)) && (r1 || bar_wait_slow(b1, p1, err));
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void bulk_1d(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
        : "memory");
}
__device__ __forceinline__ float lds(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ float4 lds4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds4u(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts(uint32_t a, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// Unit n of the block (from 0) uses slot n % S of a ring of S slots, for the (n / S)-th time: a
// consumer waits for parity (n / S) & 1 of the slot's `full`, a producer for the other one of its
// `empty`.
__device__ __forceinline__ uint32_t full_par(int n, int stages) { return (uint32_t)(n / stages) & 1u; }
__device__ __forceinline__ uint32_t empty_par(int n, int stages) { return full_par(n, stages) ^ 1u; }

// Waits for the last copies of a producer that filled n units, so that none is in flight when the
// block ends.
__device__ __forceinline__ void drain(uint32_t full, int n, int stages, int* err) {
    for (int j = n > stages ? n - stages : 0; j < n; ++j) bar_wait(full + 8 * (j % stages), full_par(j, stages), err);
}

// The 128 / G parameters of a row in one unit: one aligned load.
template <int G>
__device__ __forceinline__ void load_params(const void* base, long row, int ng, int unit, int bf16,
                                            float (&v)[kUnit / G]) {
    const long i = row * ng + unit * (kUnit / G);
    if (bf16) {
        const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(base) + i;
        if constexpr (G == 32) {
            const uint2 r = __ldg(reinterpret_cast<const uint2*>(p));
            v[0] = __uint_as_float(r.x << 16); v[1] = __uint_as_float(r.x & 0xffff0000u);
            v[2] = __uint_as_float(r.y << 16); v[3] = __uint_as_float(r.y & 0xffff0000u);
        } else if constexpr (G == 64) {
            const uint32_t r = __ldg(reinterpret_cast<const uint32_t*>(p));
            v[0] = __uint_as_float(r << 16); v[1] = __uint_as_float(r & 0xffff0000u);
        } else {
            v[0] = __bfloat162float(*p);
        }
    } else {
        const float* p = reinterpret_cast<const float*>(base) + i;
        if constexpr (G == 32) {
            const float4 r = __ldg(reinterpret_cast<const float4*>(p));
            v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
        } else if constexpr (G == 64) {
            const float2 r = __ldg(reinterpret_cast<const float2*>(p));
            v[0] = r.x; v[1] = r.y;
        } else {
            v[0] = __ldg(p);
        }
    }
}

// Where block b's part of the tile that block `first` begins lies, from token chunk c0 on.
__device__ __forceinline__ long part_row(const WideParams& p, int b, int first, int c0) {
    const long slot = (long)(blockIdx.y * gridDim.x + b) * 2 + (b == first ? 1 : 0);
    return (slot * p.t_blk + 16 * c0) * kRows;
}

template <int G, int CTAS, bool ZERO>
__global__ void __launch_bounds__(cfg_threads<CTAS>(), CTAS)
kda_proj_w4_wide_kernel(const __grid_constant__ WideMaps maps, const __grid_constant__ WideParams p) {
    extern __shared__ unsigned char smem_raw[];
    constexpr int NG = kUnit / G;                  // groups of a unit
    using C = Cfg<CTAS>;
    constexpr int kParStages = par_stages(G), kCodeStages = C::kCodeStages, kABufs = C::kABufs;
    constexpr int kDeqWarps = 4 * C::kDeqGroups, kEpiWarps = 4 * C::kEpiGroups;
    constexpr uint32_t kABase = 2 * C::kDCols;     // TMEM: two accumulators, then the A operands
    const bool x_lo = p.x_bf16 == 0;
    constexpr int kParStage = NG * kRows * 4 * (ZERO ? 2 : 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int x_image = p.t_blk * kGran * 2;       // 64 k of hi or lo
    const int x_stage = 2 * x_image * (x_lo ? 2 : 1);
    const int xs_stage = NG * p.t_blk * 4;
    // shared memory, by address: barriers at fixed offsets, then the stages
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t c_full = base, c_empty = c_full + 8 * kMaxCodeStages;
    const uint32_t x_full = c_empty + 8 * kMaxCodeStages, x_empty = x_full + 8 * kMaxXStages;
    const uint32_t p_full = x_empty + 8 * kMaxXStages, p_empty = p_full + 8 * kMaxParStages;
    const uint32_t s_full = p_empty + 8 * kMaxParStages;
    const uint32_t a_full = s_full + 8 * kMaxParStages, a_empty = a_full + 8 * kMaxABufs;
    const uint32_t d_full = a_empty + 8 * kMaxABufs, d_empty = d_full + 16, done = d_empty + 16;
    const uint32_t tmem_slot = done + 8;
    const uint32_t codes = base + kBarBytes;
    const uint32_t pars = codes + kCodeStages * kCodeStage;       // f32 [stage][c, corr][group][row]
    const uint32_t xst = pars + kParStages * kParStage;           // [stage][hi 0, hi 1, lo 0, lo 1]
    const uint32_t xss = xst + p.x_stages * x_stage;              // f32 [stage][group][token]

    // the epilogue warpgroups share the block's tokens in chunks of 16
    const int chunks = p.t_blk / 16;
    const int chunks0 = CTAS == 2 ? chunks : (chunks + 1) / 2;
    constexpr int epi_warps = kEpiWarps;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tmem_slot), "n"(C::kTmem) : "memory");
        tmem_relinquish();
    }
    if (tid == 32) {
        auto init = [](uint32_t bar, int n, int count) {
            for (int i = 0; i < n; ++i)
                asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar + 8 * i), "r"(count) : "memory");
        };
        init(c_full, kMaxCodeStages, 1);
        init(c_empty, kMaxCodeStages, 4);
        init(x_full, kMaxXStages, 1);
        init(x_empty, kMaxXStages, 1);
        init(p_full, kMaxParStages, 1);
        init(p_empty, kMaxParStages, epi_warps);
        init(s_full, kMaxParStages, 1);
        init(a_full, kMaxABufs, 4);
        init(a_empty, kMaxABufs, 1);
        init(d_full, 2, 1);
        init(d_empty, 2, epi_warps);
        init(done, 1, 1);
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    uint32_t tbase;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tbase) : "r"(tmem_slot));

    // units [u0, u1) of tiles x nk in order; a tile's parts are the blocks that touch it
    const int nk = p.in_f / kUnit;
    const int total = p.tile_start[p.nw] * nk;      // below 2^31: the entry checks it
    const int nb = gridDim.x, blk = blockIdx.x;
    const int u0 = (int)((long)total * blk / nb), u1 = (int)((long)total * (blk + 1) / nb);
    const int tok0 = blockIdx.y * p.t_blk;

    // The epilogue warps hold the sums: registers move to them from the dequantising warps.
    if (warp < kDeqWarps)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kDeqRegs));
    else if (warp < kDeqWarps + kEpiWarps)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kEpiRegs));

    if (warp < kDeqWarps) {
        // ---- codes -> A operand: the warpgroups take the block's units in turn
        const int wg = warp >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t tl = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + kABase;
        const uint32_t src0 = codes + row * (kUnit / 2);
        const uint32_t sw = (uint32_t)((row >> 1) & 3) << 4;
        const int count = u1 - u0;
        bool ok = true;
        for (int n = wg; n < count && ok; n += C::kDeqGroups) {
            const int i = n % kCodeStages, a = n % kABufs;
            ok = bar_wait2(c_full + 8 * i, full_par(n, kCodeStages), a_empty + 8 * a, empty_par(n, kABufs), p.err);
            tc_fence_after();
            const uint32_t src = src0 + i * kCodeStage;
            // (rolled: the roles' loops share a small instruction cache)
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                const uint4 w = lds4u(src + (((uint32_t)j << 4) ^ sw));
                uint32_t o[16];
                codes8(w.x, o);
                codes8(w.y, o + 4);
                codes8(w.z, o + 8);
                codes8(w.w, o + 12);
                tmem_st16u(tl + 64 * a + 16 * j, o);
            }
            __syncwarp();
            if (lane == 0) bar_arrive(c_empty + 8 * i);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(a_full + 8 * a);
        }
    } else if (warp < kDeqWarps + kEpiWarps) {
        // ---- group sums -> scaled f32 sums -> outputs
        const int e = (warp - kDeqWarps) >> 2, r_in = 32 * (warp & 3) + lane;
        const int c0 = e == 0 ? 0 : chunks0, nc = e == 0 ? chunks0 : chunks - chunks0;
        if (nc > 0) {
            const uint32_t tl = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + 16 * c0;
            float acc[4][16];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[i][j] = 0.0f;
            // the split's results: factors here, counters at the end of a part
            asm volatile("griddepcontrol.wait;" ::: "memory");
            for (int j = lane; j < 16 * nc; j += 32)        // (each warp all it needs, the same values)
                sts(base + kFactorAt + 4 * (16 * c0 + j), p.tok_factor[tok0 + 16 * c0 + j]);
            __syncwarp();
            bool ok = true;
            int k = u0 % nk;
            uint32_t dph = 0;                       // parity of both accumulators' next fill
            int d = 0;
            for (int u = u0; u < u1 && ok; ++u) {
                const int n = u - u0, ps = n % kParStages;
                const uint32_t pph = full_par(n, kParStages);
                const uint32_t par = pars + ps * kParStage + 4 * r_in;
                const uint32_t xs = xss + ps * xs_stage + 64 * c0;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    if (g == 0) {
                        ok = bar_wait2(p_full + 8 * ps, pph, d_full + 8 * d, dph, p.err);
                        if constexpr (ZERO) ok = ok && bar_wait(s_full + 8 * ps, pph, p.err);
                    } else {
                        ok = ok && bar_wait(d_full + 8 * d, dph, p.err);
                    }
                    tc_fence_after();
                    const float c = lds(par + 4 * g * kRows);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i < nc) {
                            float v[16];
                            tmem_ld16(tl + C::kDCols * d + 16 * i, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) acc[i][j] = fmaf(v[j], c, acc[i][j]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(d_empty + 8 * d);
                    dph ^= (uint32_t)d;
                    d ^= 1;
                    if constexpr (ZERO) {
                        const float corr = lds(par + 4 * (NG + g) * kRows);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (i < nc) {
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const float4 s = lds4(xs + 4 * (g * p.t_blk + 16 * i + 4 * j));
                                    acc[i][4 * j] = fmaf(corr, s.x, acc[i][4 * j]);
                                    acc[i][4 * j + 1] = fmaf(corr, s.y, acc[i][4 * j + 1]);
                                    acc[i][4 * j + 2] = fmaf(corr, s.z, acc[i][4 * j + 2]);
                                    acc[i][4 * j + 3] = fmaf(corr, s.w, acc[i][4 * j + 3]);
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) bar_arrive(p_empty + 8 * ps);
                if (++k < nk && u + 1 < u1) continue;

                // ---- end of this block's part of the tile
                k = 0;
                const int tile = u / nk;
                int wi = 0;
                while (wi + 1 < p.nw && tile >= p.tile_start[wi + 1]) ++wi;
                const int rows = p.rows[wi];
                const long row = (long)(tile - p.tile_start[wi]) * kRows + r_in;
                const long t0 = (long)tile * nk;
                const int first = (int)(((t0 + 1) * nb - 1) / total);
                const int last = (int)(((t0 + nk) * nb - 1) / total);
                // The sums step aside to local memory, so that what follows, once or twice a block,
                // does not press on the loop's registers.
                float own[64];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 16; ++j) own[16 * i + j] = acc[i][j];
                // Each warp's rows and tokens meet on their own: no warp waits for another.  The
                // counter holds the parts in the workspace.  The block's last part, when it finds
                // all the others there, need not be stored; every other one is.
                const int others = last - first;
                int* count = &p.counter[(blockIdx.y * nb + first) * 8 + warp - kDeqWarps];
                bool write = others == 0, mine = true;    // mine: this part is not in the workspace
                if (others > 0) {
                    int seen = 0;
                    if (u + 1 == u1 && lane == 0)
                        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(seen) : "l"(count) : "memory");
                    write = __shfl_sync(0xffffffffu, seen, 0) == others;
                    if (!write) {
                        // slot 0: a part that continues an earlier block's, slot 1: the first part
                        mine = false;
                        float* part = p.partial + part_row(p, blk, first, c0) + r_in;
#pragma unroll 1
                        for (int i = 0; i < nc; ++i)
#pragma unroll
                            for (int j = 0; j < 16; ++j, part += kRows) __stcg(part, own[16 * i + j]);
                        __threadfence();
                        __syncwarp();
                        seen = -1;
                        if (lane == 0 && ok) seen = atomicAdd(count, 1);
                        write = __shfl_sync(0xffffffffu, seen, 0) == others;
                    }
                    // lane 0 has seen the other parts' counts: its fence and the warp's barrier order
                    // every lane's reads of them behind that (a shuffle orders no memory)
                    __threadfence();
                    __syncwarp();
                }
                if (write && ok) {
#pragma unroll 1
                    for (int i = 0; i < nc; ++i) {
                        float v[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = 0.0f;
                        // in block order, whoever adds
#pragma unroll 1
                        for (int b = first; b <= last; ++b) {
                            float q[16];
                            if (mine && b == blk) {
#pragma unroll
                                for (int j = 0; j < 16; ++j) q[j] = own[16 * i + j];
                            } else {
                                const float* src = p.partial + part_row(p, b, first, c0 + i) + r_in;
#pragma unroll
                                for (int j = 0; j < 16; ++j) q[j] = __ldcg(src + j * kRows);
                            }
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] += q[j];
                        }
                        const int s = tok0 + 16 * (c0 + i);
                        float* o = p.out[wi] + (long)s * rows + row;
                        if (row < rows) {
#pragma unroll
                            for (int j = 0; j < 16; ++j, o += rows)
                                if (s + j < p.t) *o = v[j] * lds(base + kFactorAt + 4 * (16 * (c0 + i) + j));
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[i][j] = 0.0f;
            }
        }
    } else if (warp == kDeqWarps + kEpiWarps) {
        // ---- codes producer
        if (elect_one()) {
            int wi = 0, tile = u0 / nk, k = u0 % nk, n = 0;
            for (; n < u1 - u0; ++n) {
                while (wi + 1 < p.nw && tile >= p.tile_start[wi + 1]) ++wi;
                const int i = n % kCodeStages;
                if (!bar_wait(c_empty + 8 * i, empty_par(n, kCodeStages), p.err)) break;
                bar_expect(c_full + 8 * i, kCodeStage);
                tma_2d(codes + i * kCodeStage, &maps.w[wi], k * (kUnit / 2),
                       (tile - p.tile_start[wi]) * kRows, c_full + 8 * i);
                if (++k == nk) {
                    k = 0;
                    ++tile;
                }
            }
            drain(c_full, n, kCodeStages, p.err);
        }
    } else if (warp == kDeqWarps + kEpiWarps + 1) {
        // ---- x producer
        if (elect_one()) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            int k = u0 % nk, n = 0, ns = 0;
            for (; n < u1 - u0; ++n) {
                if constexpr (ZERO) {
                    // (the stage of the unit's group sums is free with the stage of its scales)
                    const int i = n % kParStages;
                    if (!bar_wait(p_empty + 8 * i, empty_par(n, kParStages), p.err)) break;
                    bar_expect(s_full + 8 * i, (uint32_t)xs_stage);
                    for (int g = 0; g < NG; ++g)
                        bulk_1d(xss + i * xs_stage + g * p.t_blk * 4,
                                p.xsum + (long)(k * NG + g) * p.t_rows + tok0, (uint32_t)(p.t_blk * 4),
                                s_full + 8 * i);
                    ++ns;
                }
                const int i = n % p.x_stages;
                if (!bar_wait(x_empty + 8 * i, empty_par(n, p.x_stages), p.err)) break;
                const uint32_t st = xst + i * x_stage, bar = x_full + 8 * i;
                bar_expect(bar, (uint32_t)x_stage);
                tma_2d(st, &maps.xh, k * kUnit, tok0, bar);
                tma_2d(st + x_image, &maps.xh, k * kUnit + kGran, tok0, bar);
                if (x_lo) {
                    tma_2d(st + 2 * x_image, &maps.xl, k * kUnit, tok0, bar);
                    tma_2d(st + 3 * x_image, &maps.xl, k * kUnit + kGran, tok0, bar);
                }
                if (++k == nk) k = 0;
            }
            drain(x_full, n, p.x_stages, p.err);
            if constexpr (ZERO) drain(s_full, ns, kParStages, p.err);
        }
    } else if (warp == kDeqWarps + kEpiWarps + 2) {
        // ---- MMA issuer: D_g = sum over the group of codes x (hi + lo).  The whole warp waits, and
        //      one thread is elected for each group's instructions.
        const uint32_t idesc = tc_idesc_f16(kRows, p.t_blk);
        const uint64_t desc0 = tc_smem_desc_sw128(xst);
        uint32_t dph = 1;
        int d = 0, xi = 0;
        uint32_t xph = 0;
        bool ok = true;
        for (int n = 0; n < u1 - u0 && ok; ++n) {
            const int a = n % kABufs;
            ok = bar_wait2(a_full + 8 * a, full_par(n, kABufs), x_full + 8 * xi, xph, p.err);
            const uint64_t hi = tc_desc_advance(desc0, (uint32_t)(xi * x_stage));
            const uint64_t lo = tc_desc_advance(hi, (uint32_t)(2 * x_image));
            const uint32_t at = tbase + kABase + 64 * a;
#pragma unroll 1
            for (int g = 0; g < NG; ++g) {
                ok = ok && bar_wait(d_empty + 8 * d, dph, p.err);
                tc_fence_after();
                const uint32_t dt = tbase + C::kDCols * d;
                if (ok && elect_one()) {
                    const uint64_t gh = tc_desc_advance(hi, (uint32_t)((g * G / kGran) * x_image + (g * G % kGran) * 2));
                    const uint64_t gl = tc_desc_advance(lo, (uint32_t)((g * G / kGran) * x_image + (g * G % kGran) * 2));
                    const uint32_t ga = at + g * (G / 2);
#pragma unroll 2
                    for (int kk = 0; kk < G; kk += 16) {                 // k within the group
                        const uint32_t off = (uint32_t)((kk / kGran) * x_image + (kk % kGran) * 2);
                        tc_mma_ts(dt, ga + kk / 2, tc_desc_advance(gh, off), idesc, kk > 0);
                        if (x_lo) tc_mma_ts(dt, ga + kk / 2, tc_desc_advance(gl, off), idesc, true);
                    }
                    bar_commit(d_full + 8 * d);
                    if (g + 1 == NG) {
                        bar_commit(a_empty + 8 * a);
                        bar_commit(x_empty + 8 * xi);
                    }
                }
                __syncwarp();
                dph ^= (uint32_t)d;
                d ^= 1;
            }
            if (++xi == p.x_stages) {
                xi = 0;
                xph ^= 1;
            }
        }
        // every MMA has completed: a commit follows those of the thread that issued them, and one
        // thread of a converged warp is elected every time
        if (elect_one()) bar_commit(done);
        __syncwarp();
        bar_wait(done, 0, p.err);
    } else {
        // ---- scales and zero terms of the units, row by row: lane l fetches rows l, l + 32, ..,
        //      two units ahead of the one it hands on
        const int ng = p.in_f / G, count = u1 - u0;
        float c[2][4][NG], z[2][4][NG];
        int wi = 0, tile = u0 / nk, k = u0 % nk;   // of the next unit to fetch
        bool ok = true;
        for (int n0 = -2; n0 < count && ok; n0 += 2) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int n = n0 + q;
                if (n >= 0 && n < count) {
                    const int i = n % kParStages;
                    ok = ok && bar_wait(p_empty + 8 * i, empty_par(n, kParStages), p.err);
                    const uint32_t par = pars + i * kParStage + 4 * lane;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            sts(par + 4 * (g * kRows + 32 * j), c[q][j][g]);
                            if constexpr (ZERO)
                                sts(par + 4 * ((NG + g) * kRows + 32 * j), (8.0f - z[q][j][g]) * c[q][j][g]);
                        }
                    __syncwarp();
                    if (lane == 0) bar_arrive(p_full + 8 * i);
                }
                if (n + 2 < count) {
                    while (wi + 1 < p.nw && tile >= p.tile_start[wi + 1]) ++wi;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        // rows past the weight repeat its last one; their sums are not written
                        const long row = min((tile - p.tile_start[wi]) * kRows + 32 * j + lane, p.rows[wi] - 1);
                        load_params<G>(p.scale[wi], row, ng, k, p.scale_bf16, c[q][j]);
                        if constexpr (ZERO) load_params<G>(p.zero[wi], row, ng, k, p.scale_bf16, z[q][j]);
                    }
                    if (++k == nk) {
                        k = 0;
                        ++tile;
                    }
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tbase, C::kTmem);
}

template <int G, int CTAS, bool ZERO>
cudaError_t launch_wide(const WideMaps& maps, WideParams& p, int units, int sms, int ny, cudaStream_t s) {
    using C = Cfg<CTAS>;
    const int x_stage = p.t_blk * kUnit * 2 * (p.x_bf16 ? 1 : 2);
    constexpr int ng = kUnit / G;
    const int fixed = 1024 + kBarBytes + C::kCodeStages * kCodeStage +
                      par_stages(G) * ng * 4 * (kRows * (p.has_zero ? 2 : 1) + (p.has_zero ? p.t_blk : 0));
    int xn = (C::kSmem - fixed) / x_stage;
    xn = xn > kMaxXStages ? kMaxXStages : (xn < 1 ? 1 : xn);
    p.x_stages = xn;
    const int smem = fixed + xn * x_stage;
    const auto kernel = kda_proj_w4_wide_kernel<G, CTAS, ZERO>;
    static PerDevice<int> done;
    const cudaError_t e = set_smem(kernel, kMaxBlockSmem, done);
    if (e != cudaSuccess) return e;
    int nb = sms * CTAS / ny;
    if (nb > units) nb = units;
    // a programmatic dependent of the split: codes stream and unpack while x is being split
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)nb, (unsigned)ny);
    cfg.blockDim = dim3(cfg_threads<CTAS>());
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    KernelTimer kt(kKProjW4Wide, s);
    return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

template <int G>
cudaError_t launch_wide_t(const WideMaps& maps, WideParams& p, int units, int sms, int ny, cudaStream_t s) {
    if (p.has_zero)
        return p.t_blk <= 64 ? launch_wide<G, 2, true>(maps, p, units, sms, ny, s)
                             : launch_wide<G, 1, true>(maps, p, units, sms, ny, s);
    return p.t_blk <= 64 ? launch_wide<G, 2, false>(maps, p, units, sms, ny, s)
                         : launch_wide<G, 1, false>(maps, p, units, sms, ny, s);
}

}  // namespace

size_t proj_w4_wide_workspace_bytes(int t, int in_f) { return wide_ws(t, in_f).total; }

cudaError_t launch_proj_w4_wide(const ProjW4Args& a, cudaStream_t s) {
    int ny, t_blk;
    token_blocks(a.t, ny, t_blk);
    const WideWs w = wide_ws(a.t, a.in_f);
    unsigned char* ws = static_cast<unsigned char*>(a.ws);
    WideMaps maps;
    WideParams p{};
    int tiles = 0;
    for (int i = 0; i < a.nw; ++i) {
        p.scale[i] = a.scale[i];
        p.zero[i] = a.zero[i];
        p.out[i] = a.out[i];
        p.rows[i] = a.rows[i];
        p.tile_start[i] = tiles;
        tiles += (a.rows[i] + kRows - 1) / kRows;
        if (!make_tensor_map_2d_u8_sw64(&maps.w[i], a.w[i], a.rows[i], a.in_f / 2, kRows))
            return cudaErrorInvalidValue;
    }
    p.tile_start[a.nw] = tiles;
    const int t_rows = ny * t_blk;
    __half* hi = reinterpret_cast<__half*>(ws + w.hi);
    __half* lo = reinterpret_cast<__half*>(ws + w.lo);
    if (!make_tensor_map_2d_bf16_sw128(&maps.xh, hi, t_rows, a.in_f, t_blk) ||
        !make_tensor_map_2d_bf16_sw128(&maps.xl, lo, t_rows, a.in_f, t_blk))
        return cudaErrorInvalidValue;
    p.nw = a.nw; p.t = a.t; p.in_f = a.in_f; p.scale_bf16 = a.scale_bf16; p.has_zero = a.has_zero;
    p.t_blk = t_blk; p.t_rows = t_rows; p.x_bf16 = a.x_bf16;
    p.tok_factor = reinterpret_cast<float*>(ws + w.factor);
    p.counter = reinterpret_cast<int*>(ws + w.counter);
    p.xsum = reinterpret_cast<float*>(ws + w.xsum);
    p.partial = reinterpret_cast<float*>(ws + w.partial);
    p.err = a.err;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (sms > kW4MaxSms) sms = kW4MaxSms;
    const int units = tiles * (a.in_f / kUnit);      // below 2^31: the entry checks it
    {
        KernelTimer kt(kKProjW4Split, s);
        float* factor = reinterpret_cast<float*>(ws + w.factor);
        float* xsum = reinterpret_cast<float*>(ws + w.xsum);
        const int vecs = a.in_f / 8;
        const int threads = vecs >= kSplitThreads ? kSplitThreads : (vecs + 31) / 32 * 32;
        if (a.x_bf16)
            kda_proj_w4_split_kernel<true><<<t_rows, threads, 0, s>>>(a.x, a.t, a.in_f, a.group, a.has_zero,
                                                                   t_rows, hi, lo, factor, xsum, p.counter);
        else
            kda_proj_w4_split_kernel<false><<<t_rows, threads, 0, s>>>(a.x, a.t, a.in_f, a.group, a.has_zero,
                                                                    t_rows, hi, lo, factor, xsum, p.counter);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    switch (a.group) {
        case 32: return launch_wide_t<32>(maps, p, units, sms, ny, s);
        case 64: return launch_wide_t<64>(maps, p, units, sms, ny, s);
        default: return launch_wide_t<128>(maps, p, units, sms, ny, s);
    }
}

}  // namespace kda
