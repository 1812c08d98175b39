// kda_proj_w4_wide.cu -- kda_proj_w4 for batches: the products on the tcgen05 tensor cores.
//
// Mathematics.  Codes minus 8 are whole numbers, exact in f16; x is scaled by a power of two per
// token (its largest magnitude to [2^7, 2^8)) and split into f16 hi + lo (22 significant bits; a
// bf16 x needs hi only).  The tensor cores sum code * x over one group of G k into f32, and the
// group's scale multiplies that sum in f32:
//     acc[r][s] += c[r][g] * D_g[r][s] + (8 - z[r][g]) c[r][g] * xsum_g[s],
// so neither weights nor scales are ever rounded, whatever their type.
//
// What bounds it: the codes' bytes from HBM up to about 48 rows, then the tensor cores (every
// product is made twice, for hi and lo).  Layout: a tile is 128 weight rows (the MMA's M = TMEM
// lanes) against all tokens of the block (N <= 128), in units of 128 k.  The warps have roles:
//   * one thread streams the codes of 128 rows x 128 k (8 KB, 64-byte swizzle) through a ring of
//     shared-memory stages that reaches 64 KB ahead, one the x images; one warp fetches the units'
//     scales and zero points (strided: a few bytes of each row) four units ahead;
//   * 8 dequantising warps read their row's codes (thread = row = TMEM lane, conflict-free through
//     the swizzle), turn 8 codes into four f16 pairs with nine instructions and store them as the
//     MMA's A operand in tensor memory, each warpgroup every other unit: shared memory carries
//     4-bit codes only;
//   * one thread issues the MMAs, group by group, into two accumulators in turn;
//   * 8 epilogue warps read a finished group's accumulator and add it, scaled, to the f32 sums that
//     they hold in registers (thread = weight row, up to 64 tokens each).
// One block per SM, persistent: the (tile, 128 k) units are dealt out evenly and in order, so a
// tile may be cut between blocks; its parts meet in the workspace, and the one that finishes last
// adds them in block order, so results do not depend on timing.
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
constexpr int kCodeStages = 8;
constexpr int kMaxXStages = 4;
constexpr int kMaxParStages = 8;
// stages of the ring of scales, zero terms and group sums of x
__host__ __device__ constexpr int par_stages(int group) { return group == 32 ? 4 : kMaxParStages; }
constexpr int kABufs = 4;                      // A operands in tensor memory, 64 columns each
constexpr uint32_t kABase = 256;               // their first column; accumulators in 0 .. 255
constexpr int kDeqWarps = 8, kEpiWarps = 8;
constexpr int kThreads = 32 * (kDeqWarps + kEpiWarps + 4);
constexpr int kParAhead = 4;                   // units whose parameters are on their way
constexpr int kBarBytes = 1024;                // barriers, in front of the stages
constexpr int kSmemBudget = 226 * 1024;
constexpr int kTokBlock = 128;                 // tokens of one block at most

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
    const float* tok_factor;                   // [t_rows] 2^(e - 7)
    const float* xsum;                         // [in_f / G][t_rows], in units of the factor
    float* partial;                            // [blocks][2][t_blk][128]
    int* counter;                              // [blocks][epilogue warps]
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
WideWs wide_ws(int t, int in_f) {
    int ny, t_blk;
    token_blocks(t, ny, t_blk);
    const size_t rows = (size_t)ny * t_blk;
    WideWs w;
    w.hi = 0;
    w.lo = w.hi + up256(rows * in_f * 2);
    w.factor = w.lo + up256(rows * in_f * 2);
    w.counter = w.factor + up256(rows * 4);
    w.xsum = w.counter + up256(kW4MaxBlocks * kEpiWarps * 4);
    w.partial = w.xsum + up256(rows * (in_f / 32) * 4);
    w.total = w.partial + (size_t)kW4MaxBlocks * 2 * t_blk * kRows * 4;
    return w;
}

// ---- x into images --------------------------------------------------------------------------

// One block per image row: the token's largest magnitude, then hi and lo with each 8 k in the
// order in which a word's codes come out (0 4 1 5 2 6 3 7), and the group sums.  Rows past t are
// zero.  Block 0 also clears the counters.
template <bool XBF16>
__global__ void __launch_bounds__(256) kda_proj_w4_split_kernel(
    const void* __restrict__ x, int t, int in_f, int group, int has_zero, int t_rows,
    __half* __restrict__ hi, __half* __restrict__ lo, float* __restrict__ factor,
    float* __restrict__ xsum, int* __restrict__ counter) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ uint32_t warp_max[8];
    const int s = blockIdx.x, tid = threadIdx.x;
    if (s == 0)
        for (int i = tid; i < kW4MaxBlocks * kEpiWarps; i += 256) counter[i] = 0;
    const int vecs = in_f / 8;
    uint4* h4 = reinterpret_cast<uint4*>(hi + (size_t)s * in_f);
    uint4* l4 = reinterpret_cast<uint4*>(lo + (size_t)s * in_f);
    if (s >= t) {
        for (int v = tid; v < vecs; v += 256) {
            h4[v] = make_uint4(0u, 0u, 0u, 0u);
            if (!XBF16) l4[v] = make_uint4(0u, 0u, 0u, 0u);
        }
        if (has_zero)
            for (int g = tid; g < in_f / group; g += 256) xsum[(size_t)g * t_rows + s] = 0.0f;
        if (tid == 0) factor[s] = 0.0f;
        return;
    }
    auto load8 = [&](int v, float (&f)[8]) {
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
    for (int v = tid; v < vecs; v += 256) {
        float f[8];
        load8(v, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0) warp_max[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, warp_max[w]);
    // exponent of the largest magnitude, at least -100; a row that is not finite stays as it is
    const int e = max((int)(m >> 23) - 127, -100);
    const bool fin = m < 0x7f800000u;
    const float up = fin ? __uint_as_float((uint32_t)(127 + 7 - e) << 23) : 1.0f;
    if (tid == 0) factor[s] = fin ? __uint_as_float((uint32_t)(127 - 7 + e) << 23) : 1.0f;
    const int steps = (vecs + 255) / 256;      // whole warps, for the shuffles
    for (int i = 0; i < steps; ++i) {
        const int v = tid + 256 * i;
        const bool live = v < vecs;
        float f[8] = {};
        if (live) load8(v, f);
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
        if (live) {
            h4[v] = *reinterpret_cast<const uint4*>(a);
            if (!XBF16) l4[v] = *reinterpret_cast<const uint4*>(b);
        }
        if (has_zero) {
            for (int o = 1; o < group / 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (live && v % (group / 8) == 0) xsum[(size_t)(v / (group / 8)) * t_rows + s] = sum;
        }
    }
}

// ---- the products ---------------------------------------------------------------------------

// 8 codes as four f16 pairs of whole numbers -8 .. 7 (k order 0 4 | 1 5 | 2 6 | 3 7)
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

// mbar_wait_bounded with the tries in a tight loop: a try that finds the phase complete costs about
// 60 cycles, and one that does not suspends the thread for up to 4 us, so the limit is over a second.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, int* err) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .pred q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, 1000000;\n"
        "WAIT_%=:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE_%=;\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.ne.u32 q, n, 0;\n\t"
        "@q bra WAIT_%=;\n"
        "DONE_%=:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (!ok && err) atomicOr(err, kDevErrTimeout);
    return ok != 0;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, "
        "%9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, "
        "%21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
        "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
        "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

// Position in a ring of `n` stages: index and the parity of its current pass.
struct Ring {
    int i = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++i == n) {
            i = 0;
            phase ^= 1;
        }
    }
};

// Waits for the last copies of a producer that filled n stages and stands at r, so that none is in
// flight when the block ends.
__device__ __forceinline__ void drain(uint64_t* full, Ring r, int n, int stages, int* err) {
    for (int j = n < stages ? n : stages; j > 0; --j) {
        if (r.i == 0) {
            r.i = stages;
            r.phase ^= 1;
        }
        --r.i;
        mbar_wait(&full[r.i], r.phase, err);
    }
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

__device__ __forceinline__ void rotate(float (&acc)[4][16]) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[i][j] = acc[i + 1][j];
}

// Where block b's part of the tile that block `first` begins lies, from token chunk c0 on.
__device__ __forceinline__ long part_row(const WideParams& p, int b, int first, int c0) {
    const long slot = (long)(blockIdx.y * gridDim.x + b) * 2 + (b == first ? 1 : 0);
    return (slot * p.t_blk + 16 * c0) * kRows;
}

template <int G, bool XBF16, bool ZERO>
__global__ void __launch_bounds__(kThreads, 1)
kda_proj_w4_wide_kernel(const __grid_constant__ WideMaps maps, const __grid_constant__ WideParams p) {
    extern __shared__ unsigned char smem_raw[];
    // the barriers lie at fixed offsets in front of the stages, so that every role forms their
    // addresses from one base
    unsigned char* base = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr int NG = kUnit / G;                  // groups of a unit
    constexpr int kParStages = par_stages(G);
    constexpr int kParStage = NG * kRows * 4 * (ZERO ? 2 : 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int x_image = p.t_blk * kGran * 2;       // 64 k of hi or lo
    const int x_stage = 2 * x_image * (XBF16 ? 1 : 2);
    const int xs_stage = NG * p.t_blk * 4;
    unsigned char* const codes = base + kBarBytes;
    unsigned char* const pars = codes + kCodeStages * kCodeStage;     // f32 [stage][c, corr][group][row]
    unsigned char* const xst = pars + kParStages * kParStage;         // [stage][hi 0, hi 1, lo 0, lo 1]
    unsigned char* const xss = xst + p.x_stages * x_stage;            // f32 [stage][group][token]
    uint64_t* const c_full = reinterpret_cast<uint64_t*>(base);
    uint64_t* const c_empty = c_full + kCodeStages;
    uint64_t* const x_full = c_empty + kCodeStages;
    uint64_t* const x_empty = x_full + kMaxXStages;
    uint64_t* const p_full = x_empty + kMaxXStages;
    uint64_t* const p_empty = p_full + kMaxParStages;
    uint64_t* const a_full = p_empty + kMaxParStages;
    uint64_t* const a_empty = a_full + kABufs;
    uint64_t* const d_full = a_empty + kABufs;
    uint64_t* const d_empty = d_full + 2;
    uint64_t* const s_full = d_empty + 2;
    uint64_t* const done = s_full + kMaxParStages;
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(done + 1);

    // the two epilogue warpgroups share the block's tokens in chunks of 16
    const int chunks = p.t_blk / 16;
    const int chunks0 = (chunks + 1) / 2;
    const int epi_warps = chunks > 1 ? 8 : 4;

    if (warp == 0) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (tid == 32) {
        for (int i = 0; i < kCodeStages; ++i) {
            mbar_init(&c_full[i], 1);
            mbar_init(&c_empty[i], 4);
        }
        for (int i = 0; i < kMaxXStages; ++i) {
            mbar_init(&x_full[i], 1);
            mbar_init(&x_empty[i], 1);
        }
        for (int i = 0; i < kParStages; ++i) {
            mbar_init(&p_full[i], 1);
            mbar_init(&p_empty[i], epi_warps);
            mbar_init(&s_full[i], 1);
        }
        for (int i = 0; i < kABufs; ++i) {
            mbar_init(&a_full[i], 4);
            mbar_init(&a_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&d_full[i], 1);
            mbar_init(&d_empty[i], epi_warps);
        }
        mbar_init(done, 1);
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;

    // units [u0, u1) of tiles x nk in order; a tile's parts are the blocks that touch it
    const int nk = p.in_f / kUnit;
    const int total = p.tile_start[p.nw] * nk;      // below 2^31: the entry checks it
    const int nb = gridDim.x, blk = blockIdx.x;
    const int u0 = (int)((long)total * blk / nb), u1 = (int)((long)total * (blk + 1) / nb);
    const int tok0 = blockIdx.y * p.t_blk;

    // The epilogue warps hold the sums: registers move to them from the dequantising warps.  The
    // launch gives every thread 96: 256 * 64 + 256 * 128 = 512 * 96.
    if (warp < kDeqWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        // ---- codes -> A operand: warpgroup wg takes the block's units wg, wg + 2, ..
        const int wg = warp >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t tl = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + kABase;
        const unsigned char* src0 = codes + row * (kUnit / 2);
        const int sw = (row >> 1) & 3;
        int i = wg;                                // code stage; A buffer i & 3
        uint32_t ph = 0, aph = 1;
        bool ok = true;
        for (int u = u0 + wg; u < u1 && ok; u += 2) {
            ok = mbar_wait(&c_full[i], ph, p.err);
            const unsigned char* src = src0 + i * kCodeStage;
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint4*>(src + ((j ^ sw) << 4));
            uint32_t o[32];
            codes8(w[0].x, o);
            codes8(w[0].y, o + 4);
            codes8(w[0].z, o + 8);
            codes8(w[0].w, o + 12);
            codes8(w[1].x, o + 16);
            codes8(w[1].y, o + 20);
            codes8(w[1].z, o + 24);
            codes8(w[1].w, o + 28);
            __syncwarp();
            if (lane == 0) mbar_arrive(&c_empty[i]);
            const int a = i & (kABufs - 1);
            ok = ok && mbar_wait(&a_empty[a], aph, p.err);
            tc_fence_after();
            tmem_st32u(tl + 64 * a, o);
            codes8(w[2].x, o);
            codes8(w[2].y, o + 4);
            codes8(w[2].z, o + 8);
            codes8(w[2].w, o + 12);
            codes8(w[3].x, o + 16);
            codes8(w[3].y, o + 20);
            codes8(w[3].z, o + 24);
            codes8(w[3].w, o + 28);
            tmem_st32u(tl + 64 * a + 32, o);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&a_full[a]);
            // stages 0 2 4 6 | 1 3 5 7: the code ring turns every 4 steps, the A ring every 2
            if (i & 2) aph ^= 1;
            i += 2;
            if (i >= kCodeStages) {
                i -= kCodeStages;
                ph ^= 1;
            }
        }
    } else if (warp < kDeqWarps + kEpiWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
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
            Ring rp;
            int d = 0;
            uint32_t dph = 0;
            bool ok = true;
            int k = u0 % nk;
            for (int u = u0; u < u1 && ok; ++u) {
                ok = mbar_wait(&p_full[rp.i], rp.phase, p.err);
                if constexpr (ZERO) ok = ok && mbar_wait(&s_full[rp.i], rp.phase, p.err);
                const float* par = reinterpret_cast<const float*>(pars + rp.i * kParStage) + r_in;
                const float* xs = reinterpret_cast<const float*>(xss + rp.i * xs_stage) + 16 * c0;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float c = par[g * kRows];
                    ok = ok && mbar_wait(&d_full[d], dph, p.err);
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i < nc) {
                            float v[16];
                            tmem_ld16(tl + (d ? 128 : 0) + 16 * i, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) acc[i][j] = fmaf(v[j], c, acc[i][j]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&d_empty[d]);
                    if (d == 1) dph ^= 1;
                    d ^= 1;
                    if constexpr (ZERO) {
                        const float corr = par[(NG + g) * kRows];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (i < nc) {
                                const float4* s4 = reinterpret_cast<const float4*>(xs + g * p.t_blk + 16 * i);
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const float4 s = s4[j];
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
                if (lane == 0) mbar_arrive(&p_empty[rp.i]);
                rp.next(kParStages);
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
                asm volatile("griddepcontrol.wait;" ::: "memory");
                // one chunk of 16 tokens at a time, the next one moved to the front
                const bool whole = first == last;
                bool write = whole;
                if (!whole) {
                    // slot 0: the part that continues an earlier block's, slot 1: the first part
                    float* part = p.partial + part_row(p, blk, first, c0) + r_in;
#pragma unroll 1
                    for (int i = 0; i < nc; ++i) {
#pragma unroll
                        for (int j = 0; j < 16; ++j, part += kRows) __stcg(part, acc[0][j]);
                        rotate(acc);
                    }
                    // each warp's rows and tokens meet on their own: no warp waits for another
                    __threadfence();
                    __syncwarp();
                    int seen = -1;
                    if (lane == 0 && ok)
                        seen = atomicAdd(&p.counter[(blockIdx.y * nb + first) * kEpiWarps + warp - kDeqWarps], 1);
                    write = __shfl_sync(0xffffffffu, seen, 0) == last - first;
                    __threadfence();
                }
                if (write && ok) {
#pragma unroll 1
                    for (int i = 0; i < nc; ++i) {
                        if (!whole) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) acc[0][j] = 0.0f;
                            for (int b = first; b <= last; ++b) {
                                const float* q = p.partial + part_row(p, b, first, c0 + i) + r_in;
#pragma unroll
                                for (int j = 0; j < 16; ++j) acc[0][j] += __ldcg(q + j * kRows);
                            }
                        }
                        const int s0 = tok0 + 16 * (c0 + i);
                        float* o = p.out[wi] + (long)s0 * rows + row;
                        if (row < rows) {
#pragma unroll
                            for (int j = 0; j < 16; ++j, o += rows)
                                if (s0 + j < p.t) *o = acc[0][j] * p.tok_factor[s0 + j];
                        }
                        rotate(acc);
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
            Ring r;
            int wi = 0, tile = u0 / nk, k = u0 % nk, n = 0;
            for (int u = u0; u < u1; ++u, ++n) {
                while (wi + 1 < p.nw && tile >= p.tile_start[wi + 1]) ++wi;
                if (!mbar_wait(&c_empty[r.i], r.phase ^ 1, p.err)) break;
                mbar_arrive_expect_tx(&c_full[r.i], kCodeStage);
                tma_load_2d(codes + r.i * kCodeStage, &maps.w[wi], k * (kUnit / 2),
                            (tile - p.tile_start[wi]) * kRows, &c_full[r.i]);
                r.next(kCodeStages);
                if (++k == nk) {
                    k = 0;
                    ++tile;
                }
            }
            drain(c_full, r, n, kCodeStages, p.err);
        }
    } else if (warp == kDeqWarps + kEpiWarps + 1) {
        // ---- x producer
        if (elect_one()) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            Ring r, rs;
            int k = u0 % nk, n = 0, ns = 0;
            for (int u = u0; u < u1; ++u) {
                if constexpr (ZERO) {
                    // (the stage of the unit's group sums is free with the stage of its scales)
                    if (!mbar_wait(&p_empty[rs.i], rs.phase ^ 1, p.err)) break;
                    mbar_arrive_expect_tx(&s_full[rs.i], (uint32_t)xs_stage);
                    for (int g = 0; g < NG; ++g)
                        bulk_load(xss + rs.i * xs_stage + g * p.t_blk * 4,
                                  p.xsum + (long)(k * NG + g) * p.t_rows + tok0,
                                  (uint32_t)(p.t_blk * 4), &s_full[rs.i]);
                    rs.next(kParStages);
                    ++ns;
                }
                if (!mbar_wait(&x_empty[r.i], r.phase ^ 1, p.err)) break;
                unsigned char* st = xst + r.i * x_stage;
                mbar_arrive_expect_tx(&x_full[r.i], (uint32_t)x_stage);
                tma_load_2d(st, &maps.xh, k * kUnit, tok0, &x_full[r.i]);
                tma_load_2d(st + x_image, &maps.xh, k * kUnit + kGran, tok0, &x_full[r.i]);
                if constexpr (!XBF16) {
                    tma_load_2d(st + 2 * x_image, &maps.xl, k * kUnit, tok0, &x_full[r.i]);
                    tma_load_2d(st + 3 * x_image, &maps.xl, k * kUnit + kGran, tok0, &x_full[r.i]);
                }
                r.next(p.x_stages);
                ++n;
                if (++k == nk) k = 0;
            }
            drain(x_full, r, n, p.x_stages, p.err);
            if constexpr (ZERO) drain(s_full, rs, ns, kParStages, p.err);
        }
    } else if (warp == kDeqWarps + kEpiWarps + 2) {
        // ---- MMA issuer: D_g = sum over the group of codes x (hi + lo)
        if (elect_one()) {
            const uint32_t idesc = tc_idesc_f16(kRows, p.t_blk);
            const uint64_t desc0 = tc_smem_desc_sw128(smem_u32(xst));
            Ring rx;
            int a = 0, d = 0;
            uint32_t aph = 0, dph = 1;
            bool ok = true;
            for (int u = u0; u < u1; ++u) {
                ok = mbar_wait(&a_full[a], aph, p.err) && mbar_wait(&x_full[rx.i], rx.phase, p.err);
                const uint64_t hi = tc_desc_advance(desc0, (uint32_t)(rx.i * x_stage));
                const uint64_t lo = tc_desc_advance(hi, (uint32_t)(2 * x_image));
                const uint32_t at = tbase + kABase + 64 * a;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    ok = ok && mbar_wait(&d_empty[d], dph, p.err);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t dt = tbase + (d ? 128 : 0);
#pragma unroll
                    for (int ks = 0; ks < G / 16; ++ks) {
                        const int kk = g * G + ks * 16;              // k within the unit
                        const uint32_t off = (uint32_t)((kk / kGran) * x_image + (kk % kGran) * 2);
                        tc_mma_ts(dt, at + kk / 2, tc_desc_advance(hi, off), idesc, ks > 0);
                        if constexpr (!XBF16)
                            tc_mma_ts(dt, at + kk / 2, tc_desc_advance(lo, off), idesc, true);
                    }
                    tc_commit(&d_full[d]);
                    if (d == 1) dph ^= 1;
                    d ^= 1;
                }
                if (!ok) break;
                tc_commit(&a_empty[a]);
                tc_commit(&x_empty[rx.i]);
                rx.next(p.x_stages);
                if (++a == kABufs) {
                    a = 0;
                    aph ^= 1;
                }
            }
            tc_commit(done);
            mbar_wait(done, 0, p.err);             // every MMA has completed
        }
    } else {
        // ---- scales and zero terms of the units, row by row: lane l fetches rows l, l + 32, ..,
        //      kParAhead units ahead of the one it hands on
        const int ng = p.in_f / G;
        float c[kParAhead][4][NG], z[kParAhead][4][NG];
        int wi = 0, tile = u0 / nk, k = u0 % nk;   // of the next unit to fetch
        auto fetch = [&](float (&cv)[4][NG], float (&zv)[4][NG]) {
            while (wi + 1 < p.nw && tile >= p.tile_start[wi + 1]) ++wi;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // rows past the weight repeat its last one; their sums are not written
                const long row = min((tile - p.tile_start[wi]) * kRows + 32 * j + lane, p.rows[wi] - 1);
                load_params<G>(p.scale[wi], row, ng, k, p.scale_bf16, cv[j]);
                if constexpr (ZERO) load_params<G>(p.zero[wi], row, ng, k, p.scale_bf16, zv[j]);
            }
            if (++k == nk) {
                k = 0;
                ++tile;
            }
        };
#pragma unroll
        for (int q = 0; q < kParAhead; ++q)
            if (u0 + q < u1) fetch(c[q], z[q]);
        Ring rp;
        bool ok = true;
        for (int u = u0; u < u1 && ok; u += kParAhead) {
#pragma unroll
            for (int q = 0; q < kParAhead; ++q) {
                if (u + q < u1 && ok) {
                    ok = mbar_wait(&p_empty[rp.i], rp.phase ^ 1, p.err);
                    float* par = reinterpret_cast<float*>(pars + rp.i * kParStage) + lane;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            par[g * kRows + 32 * j] = c[q][j][g];
                            if constexpr (ZERO)
                                par[(NG + g) * kRows + 32 * j] = (8.0f - z[q][j][g]) * c[q][j][g];
                        }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[rp.i]);
                    rp.next(kParStages);
                    if (u + q + kParAhead < u1) fetch(c[q], z[q]);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tbase, 512);
}

template <int G, bool XBF16, bool ZERO>
cudaError_t launch_wide(const WideMaps& maps, const WideParams& p, int nb, int ny, size_t smem,
                        cudaStream_t s) {
    static PerDevice<int> smem_set_for;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const auto kernel = kda_proj_w4_wide_kernel<G, XBF16, ZERO>;
    const bool cached = dev >= 0 && dev < kMaxDevices;
    if (!cached || smem_set_for[dev].load(std::memory_order_acquire) < (int)smem) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        if (cached) {
            int cur = smem_set_for[dev].load(std::memory_order_acquire);
            while (cur < (int)smem &&
                   !smem_set_for[dev].compare_exchange_weak(cur, (int)smem, std::memory_order_acq_rel)) {
            }
        }
    }
    // a programmatic dependent of the split: codes stream and unpack while x is being split
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)nb, (unsigned)ny);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
cudaError_t launch_wide_x(const WideMaps& maps, const WideParams& p, bool bf16, int nb, int ny,
                          size_t smem, cudaStream_t s) {
    if (p.has_zero)
        return bf16 ? launch_wide<G, true, true>(maps, p, nb, ny, smem, s)
                    : launch_wide<G, false, true>(maps, p, nb, ny, smem, s);
    return bf16 ? launch_wide<G, true, false>(maps, p, nb, ny, smem, s)
                : launch_wide<G, false, false>(maps, p, nb, ny, smem, s);
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
    p.t_blk = t_blk; p.t_rows = t_rows;
    p.tok_factor = reinterpret_cast<float*>(ws + w.factor);
    p.counter = reinterpret_cast<int*>(ws + w.counter);
    p.xsum = reinterpret_cast<float*>(ws + w.xsum);
    p.partial = reinterpret_cast<float*>(ws + w.partial);
    p.err = a.err;
    const int x_stage = t_blk * kUnit * 2 * (a.x_bf16 ? 1 : 2);
    const int ng = kUnit / a.group;
    const int xs = a.has_zero ? par_stages(a.group) * ng * t_blk * 4 : 0;
    const int fixed = 1024 + kBarBytes + kCodeStages * kCodeStage +
                      par_stages(a.group) * ng * kRows * 4 * (a.has_zero ? 2 : 1) + xs;
    int xn = (kSmemBudget - fixed) / x_stage;
    xn = xn > kMaxXStages ? kMaxXStages : (xn < 1 ? 1 : xn);
    p.x_stages = xn;
    const size_t smem = (size_t)fixed + (size_t)xn * x_stage;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (sms > kW4MaxBlocks) sms = kW4MaxBlocks;
    const long units = (long)tiles * (a.in_f / kUnit);
    int nb = sms / ny;
    if (nb > units) nb = (int)units;
    {
        KernelTimer kt(kKProjW4Split, s);
        float* factor = reinterpret_cast<float*>(ws + w.factor);
        float* xsum = reinterpret_cast<float*>(ws + w.xsum);
        if (a.x_bf16)
            kda_proj_w4_split_kernel<true><<<t_rows, 256, 0, s>>>(a.x, a.t, a.in_f, a.group, a.has_zero,
                                                                   t_rows, hi, lo, factor, xsum, p.counter);
        else
            kda_proj_w4_split_kernel<false><<<t_rows, 256, 0, s>>>(a.x, a.t, a.in_f, a.group, a.has_zero,
                                                                    t_rows, hi, lo, factor, xsum, p.counter);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    switch (a.group) {
        case 32: return launch_wide_x<32>(maps, p, a.x_bf16 != 0, nb, ny, smem, s);
        case 64: return launch_wide_x<64>(maps, p, a.x_bf16 != 0, nb, ny, smem, s);
        default: return launch_wide_x<128>(maps, p, a.x_bf16 != 0, nb, ny, smem, s);
    }
}

}  // namespace kda
