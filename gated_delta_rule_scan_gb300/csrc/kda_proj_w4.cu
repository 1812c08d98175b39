// kda_proj_w4.cu -- projections of t token rows by weights of 4 bits with group scales:
//
//     out_i[s][r] = sum_k (q_i[r][k] - z_i[r][k / G]) * c_i[r][k / G] * x[s][k]
//
// for up to 8 weights that read one x.  q is a 4-bit code (two to a byte, the even k in the low
// nibble), c the scale and z the zero point of G consecutive k (z = 8 without zero points).
//
// Mathematics.  A code minus 8 is an integer of -8 .. 7, exact in f16, so the products run on the
// tensor cores with the integers themselves and the scale multiplies each group's f32 sum: no
// weight is ever rounded.  x is split over 128 k at a time into f16 hi + lo after scaling by the
// power of two that brings the largest of the 128 magnitudes to [2^14, 2^15); hi + lo hold 22
// significant bits of every element that matters to the sum, and the power of two goes back in
// with the group's scale.  A bf16 x needs the hi part only: its 8 bits fit.  Zero points other
// than 8 add (8 - z) c sum_group(x), from f32 sums of x over each group.
//
// The form for few rows (t <= 8 per pass).  The weights' bytes are read once and bound the launch,
// so the kernel is built around their stream: a warp takes 16 weight rows x 128 k (1 KB of codes,
// two wide loads a lane straight into registers, the next 1 KB requested before the present one is
// used), and turns them into mma.sync m16n8k16 operands with two logical operations and two f16
// multiply-adds for 8 weights each way.  The order of k inside an MMA is free as long as both
// operands agree, so x is laid out in shared memory once per block in the order in which the
// nibbles of a word come out, and one 16-byte shared load feeds two MMAs.  The 8 columns of the
// MMA carry hi and lo of 4 tokens (f32 x) or 8 tokens (bf16 x).
// Blocks are persistent over 16-row tiles; the 8 warps of a block split K, and their partial sums
// meet in shared memory in warp order.  Where x of all of K does not fit, the CTAs of a cluster
// split K further and add their sums through distributed shared memory in rank order.  No atomics:
// results do not depend on timing.
#include <cuda_fp16.h>

#include "kda_device.cuh"
#include "kda_tc.cuh"

namespace kda {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 16;                    // weight rows of a tile: the MMA's M
constexpr int kChunk = 128;                  // k of one warp step
constexpr int kTok = 8;                      // tokens of one pass
// Rows up to which this form is taken: one launch and no workspace.  At 64 heads x 6144 it runs 33
// us at one row but 91 at eight (two MMA tiles), the form for batches 34 at any of them.
constexpr int kSmallT = 4;
constexpr int kXSmem = 72 * 1024;            // x of one block: three blocks per SM

struct W4Params {
    const void* x;
    const uint8_t* w[kW4MaxWeights];
    const void* scale[kW4MaxWeights];
    const void* zero[kW4MaxWeights];
    float* out[kW4MaxWeights];
    int rows[kW4MaxWeights];
    int tile_start[kW4MaxWeights + 1];
    int nw, t, in_f, scale_bf16, has_zero, ksplit;
};

// Bytes of the block's shared memory for `chunks` chunks of k and `cols` MMA columns.
struct W4Smem {
    int x, factor, xsum, red, total;
};
__host__ __device__ inline W4Smem w4_smem(int chunks, int cols, int group) {
    W4Smem m;
    m.x = 0;                                                   // f16 [chunk][4][cols][4][8]
    m.factor = chunks * kChunk * cols * 2;                     // f32 [chunk][8]
    m.xsum = m.factor + chunks * kTok * 4;                     // f32 [group][8]
    m.red = m.xsum + chunks * (kChunk / group) * kTok * 4;     // f32 [2][warps][8][16]
    m.total = m.red + 2 * kWarps * kTok * kRows * 4;
    return m;
}

// Nibbles p and p + 4 (lo) or p + 1 and p + 5 (hi) of the word w >> 4p as f16 pairs minus 8.  A
// nibble or-ed into the mantissa of 1024 (0x6400) is 1024 + q in its low place and 1024 + 16 q one
// place up; both corrections are exact.
__device__ __forceinline__ uint32_t nib_lo(uint32_t w) {
    const uint32_t v = (w & 0x000f000fu) | 0x64006400u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(1032.0f));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t nib_hi(uint32_t w) {
    const uint32_t v = (w & 0x00f000f0u) | 0x64006400u;
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(0.0625f),
                              __float2half2_rn(-72.0f));
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 4, 8 or 16 bytes (G / 8) of streamed weights into the words w[0 ..].
template <int BYTES>
__device__ __forceinline__ void load_words(uint32_t* w, const uint8_t* p) {
    if constexpr (BYTES == 16) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (BYTES == 8) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
        w[0] = v.x; w[1] = v.y;
    } else {
        w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
    }
}

__device__ __forceinline__ float load_param(const void* p, long i, int bf16) {
    return bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i])
                : reinterpret_cast<const float*>(p)[i];
}

// Codes, scales and zero points of 16 rows x 128 k as one warp holds them: lane 4g + c has, of rows
// g and g + 8 and of each group, the c-th quarter's codes.
template <int G>
struct W4Frag {
    uint32_t w[2][4];
    float c[2][kChunk / G];
    float z[2][kChunk / G];
};

template <int G>
__device__ __forceinline__ void frag_load(W4Frag<G>& f, const W4Params& p, int tile, int chunk,
                                          int lane) {
    int wi = 0;
    while (wi + 1 < p.nw && tile >= p.tile_start[wi + 1]) ++wi;
    const int row0 = (tile - p.tile_start[wi]) * kRows;
    const int g = lane >> 2, c = lane & 3;
    const int ng = p.in_f / G;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        // rows past the weight repeat its last one; their sums are not written
        const long row = min(row0 + g + 8 * r, p.rows[wi] - 1);
        const uint8_t* base = p.w[wi] + row * (p.in_f / 2) + chunk * (kChunk / 2) + c * (G / 8);
#pragma unroll
        for (int q = 0; q < kChunk / G; ++q) {
            load_words<G / 8>(&f.w[r][q * (G / 32)], base + q * (G / 2));
            const long gi = row * ng + chunk * (kChunk / G) + q;
            f.c[r][q] = load_param(p.scale[wi], gi, p.scale_bf16);
            f.z[r][q] = p.has_zero ? load_param(p.zero[wi], gi, p.scale_bf16) : 8.0f;
        }
    }
}

// x of the block's chunks [ch0, ch0 + chunks) and tokens [tok0, tok0 + nt): MMA operands, power-of-
// two factors and group sums.  A half warp takes one (chunk, token): lane u holds k = 8u .. 8u+7.
template <int G, bool XBF16>
__device__ __forceinline__ void stage_x(const W4Params& p, unsigned char* smem, const W4Smem& lay,
                                        int ch0, int chunks, int tok0, int nt, int cols) {
    const int half = threadIdx.x >> 4, u = threadIdx.x & 15;
    float* factor = reinterpret_cast<float*>(smem + lay.factor);
    float* xsum = reinterpret_cast<float*>(smem + lay.xsum);
    const int total = chunks * nt;
    for (int i0 = 0; i0 < total; i0 += kThreads / 16) {
        const int i = i0 + half;
        const bool live = i < total;
        const int ch = live ? i / nt : 0, tk = live ? i % nt : 0;
        float v[8];
        const long at = (long)(tok0 + tk) * p.in_f + (long)(ch0 + ch) * kChunk + 8 * u;
        if constexpr (XBF16) {
            const uint4 r = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.x) + at));
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        } else {
            const float4* x4 = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.x) + at);
            const float4 a = __ldg(x4), b = __ldg(x4 + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
        uint32_t m = 0;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
            sum += v[j];
        }
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
        for (int o = 1; o < G / 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        // 2^(14 - e) for the largest magnitude's exponent e (at least -100); 1 when it is not finite
        const int e = max((int)(m >> 23) - 127, -100);
        const bool fin = m < 0x7f800000u;
        const float up = fin ? __uint_as_float((uint32_t)(127 + 14 - e) << 23) : 1.0f;
        if (!live) continue;
        __half hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float y = __fmul_rn(v[j], up);
            const int at8 = j < 4 ? 2 * j : 2 * (j - 4) + 1;     // nibble order (0 4 1 5 2 6 3 7)
            hi[at8] = __float2half_rn(y);
            lo[at8] = __float2half_rn(y - __half2float(hi[at8]));
        }
        // k = 8u is word jj of quarter c of its group
        const int k0 = 8 * u, q = k0 / G, c = (k0 % G) / (G / 4), jj = q * (G / 32) + (k0 % (G / 4)) / 8;
        uint4* xs = reinterpret_cast<uint4*>(smem + lay.x);
        const long base = (long)(ch * 4 + jj) * cols * 4 + c;
        if constexpr (XBF16) {
            xs[base + tk * 4] = *reinterpret_cast<const uint4*>(hi);
        } else {
            xs[base + (2 * tk) * 4] = *reinterpret_cast<const uint4*>(hi);
            xs[base + (2 * tk + 1) * 4] = *reinterpret_cast<const uint4*>(lo);
        }
        if (u == 0) factor[ch * kTok + tk] = fin ? __uint_as_float((uint32_t)(127 - 14 + e) << 23) : 1.0f;
        if (u % (G / 8) == 0) xsum[(ch * (kChunk / G) + u / (G / 8)) * kTok + tk] = sum;
    }
}

// NT: 8-column MMA tiles (f32 x: 4 tokens each; bf16 x: 8).
template <int G, bool XBF16, int NT>
__global__ void __launch_bounds__(kThreads, 3) kda_proj_w4_kernel(const __grid_constant__ W4Params p) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int rank = blockIdx.x % p.ksplit, group_id = blockIdx.x / p.ksplit;
    const int stride = gridDim.x / p.ksplit;
    const int tok0 = blockIdx.y * kTok, nt = min(kTok, p.t - tok0);
    const int cols = XBF16 ? nt : 2 * nt;
    const int all = p.in_f / kChunk;
    const int ch0 = all * rank / p.ksplit, ch1 = all * (rank + 1) / p.ksplit;
    const int chunks = ch1 - ch0;
    const W4Smem lay = w4_smem((all + p.ksplit - 1) / p.ksplit, cols, G);
    const int tiles = p.tile_start[p.nw];
    const float* factor = reinterpret_cast<const float*>(smem + lay.factor);
    const float* xsum = reinterpret_cast<const float*>(smem + lay.xsum);
    const uint4* xs = reinterpret_cast<const uint4*>(smem + lay.x);
    float* red = reinterpret_cast<float*>(smem + lay.red);

    const int w0 = chunks * warp / kWarps, w1 = chunks * (warp + 1) / kWarps;
    W4Frag<G> cur;
    if (group_id < tiles && w0 < w1) frag_load<G>(cur, p, group_id, ch0 + w0, lane);
    stage_x<G, XBF16>(p, smem, lay, ch0, chunks, tok0, nt, cols);
    __syncthreads();

    int buf = 0;
    for (int tile = group_id; tile < tiles; tile += stride, buf ^= 1) {
        // acc[i][r][e]: f32 x: token 4 i + c of row g + 8 r (e = 0); bf16: token 2 c + e
        float acc[NT][2][2] = {};
        for (int ch = w0; ch < w1; ++ch) {
            W4Frag<G> nxt;
            const bool last = ch + 1 == w1;
            const int ntile = last ? tile + stride : tile;
            const bool more = ntile < tiles;
            if (more) frag_load<G>(nxt, p, ntile, ch0 + (last ? w0 : ch + 1), lane);
#pragma unroll
            for (int q = 0; q < kChunk / G; ++q) {
                float d[NT][4] = {};
#pragma unroll
                for (int j = q * (G / 32); j < (q + 1) * (G / 32); ++j) {
                    const uint32_t u0 = cur.w[0][j], u1 = cur.w[1][j];
                    const uint32_t a0 = nib_lo(u0), a1 = nib_lo(u1), a2 = nib_hi(u0), a3 = nib_hi(u1);
                    const uint32_t e0 = nib_lo(u0 >> 8), e1 = nib_lo(u1 >> 8);
                    const uint32_t e2 = nib_hi(u0 >> 8), e3 = nib_hi(u1 >> 8);
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        uint4 b = make_uint4(0u, 0u, 0u, 0u);
                        if (8 * i + g < cols) b = xs[((ch * 4 + j) * cols + 8 * i + g) * 4 + c];
                        mma_16816(d[i], a0, a1, a2, a3, b.x, b.y);
                        mma_16816(d[i], e0, e1, e2, e3, b.z, b.w);
                    }
                }
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < (XBF16 ? 2 : 1); ++e) {
                        const int tk = XBF16 ? 2 * c + e : 4 * i + c;
                        const float f = factor[ch * kTok + tk];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float s = XBF16 ? d[i][2 * r + e] : d[i][2 * r] + d[i][2 * r + 1];
                            acc[i][r][e] = fmaf(s * f, cur.c[r][q], acc[i][r][e]);
                            if (p.has_zero)
                                acc[i][r][e] = fmaf((8.0f - cur.z[r][q]) * cur.c[r][q],
                                                    xsum[(ch * (kChunk / G) + q) * kTok + tk],
                                                    acc[i][r][e]);
                        }
                    }
            }
            if (more) cur = nxt;
        }
        // this tile's sums of all warps, in warp order
        float* rb = red + buf * (kWarps * kTok * kRows);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < (XBF16 ? 2 : 1); ++e)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    rb[(warp * kTok + (XBF16 ? 2 * c + e : 4 * i + c)) * kRows + g + 8 * r] = acc[i][r][e];
        __syncthreads();
        int wi = 0;
        while (wi + 1 < p.nw && tile >= p.tile_start[wi + 1]) ++wi;
        const int tk = threadIdx.x / kRows, r = threadIdx.x % kRows;
        const int row = (tile - p.tile_start[wi]) * kRows + r;
        float sum = 0.0f;
        if (tk < nt) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += rb[(w * kTok + tk) * kRows + r];
        }
        if (p.ksplit > 1) {
            // the cluster's CTAs: each leaves its sums where warp 0's were, then rank 0 adds them.
            // Its reads of this buffer end before any CTA passes the next tile's barrier and fills
            // the buffer after that one.
            __syncthreads();
            if (tk < nt) rb[tk * kRows + r] = sum;
            cluster_sync_all();
            if (rank == 0 && tk < nt) {
                sum = 0.0f;
                for (int k = 0; k < p.ksplit; ++k) sum += ld_cluster_f32(&rb[tk * kRows + r], (uint32_t)k);
            }
        }
        if (rank == 0 && tk < nt && row < p.rows[wi])
            p.out[wi][(long)(tok0 + tk) * p.rows[wi] + row] = sum;
    }
    if (p.ksplit > 1) cluster_sync_all();        // rank 0 has read the last tile's sums
}

template <int G, bool XBF16, int NT>
cudaError_t launch_rows(const W4Params& p, int grid, size_t smem, cudaStream_t s) {
    static PerDevice<int> smem_set_for;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const auto kernel = kda_proj_w4_kernel<G, XBF16, NT>;
    const bool cached = dev >= 0 && dev < kMaxDevices;
    if (smem > 48 * 1024 && (!cached || smem_set_for[dev].load(std::memory_order_acquire) < (int)smem)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        if (cached) {
            int cur = smem_set_for[dev].load(std::memory_order_acquire);
            while (cur < (int)smem &&
                   !smem_set_for[dev].compare_exchange_weak(cur, (int)smem, std::memory_order_acq_rel)) {
            }
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, (unsigned)((p.t + kTok - 1) / kTok));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.ksplit;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.ksplit > 1 ? 1 : 0;
    KernelTimer kt(kKProjW4, s);
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int G>
cudaError_t launch_group(const W4Params& p, bool x_bf16, int grid, size_t smem, cudaStream_t s) {
    if (x_bf16) return launch_rows<G, true, 1>(p, grid, smem, s);
    return p.t <= 4 ? launch_rows<G, false, 1>(p, grid, smem, s)
                    : launch_rows<G, false, 2>(p, grid, smem, s);
}

}  // namespace

size_t proj_w4_workspace_bytes(int t, int in_f) {
    return t > kSmallT ? proj_w4_wide_workspace_bytes(t, in_f) : 0;
}

cudaError_t launch_proj_w4(const ProjW4Args& a, cudaStream_t s) {
    if (a.t > kSmallT) return launch_proj_w4_wide(a, s);
    W4Params p{};
    p.x = a.x;
    int tiles = 0;
    for (int i = 0; i < a.nw; ++i) {
        p.w[i] = static_cast<const uint8_t*>(a.w[i]);
        p.scale[i] = a.scale[i];
        p.zero[i] = a.zero[i];
        p.out[i] = a.out[i];
        p.rows[i] = a.rows[i];
        p.tile_start[i] = tiles;
        tiles += (a.rows[i] + kRows - 1) / kRows;
    }
    p.tile_start[a.nw] = tiles;
    if (tiles == 0) return cudaSuccess;
    p.nw = a.nw; p.t = a.t; p.in_f = a.in_f; p.scale_bf16 = a.scale_bf16; p.has_zero = a.has_zero;
    // the fewest CTAs along K whose share of x fits
    const int nt = a.t < kTok ? a.t : kTok, cols = a.x_bf16 ? nt : 2 * nt;
    const int all = a.in_f / kChunk;
    int ks = 1;
    while (ks < 8 && (all + ks - 1) / ks * (kChunk * cols * 2) > kXSmem) ks *= 2;
    p.ksplit = ks;
    const W4Smem lay = w4_smem((all + ks - 1) / ks, cols, a.group);
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    int per_sm = 220 * 1024 / (lay.total + 1024);
    per_sm = per_sm > 3 ? 3 : (per_sm < 1 ? 1 : per_sm);
    int groups = sms * per_sm / ks;
    if (groups > tiles) groups = tiles;
    if (groups < 1) groups = 1;
    switch (a.group) {
        case 32: return launch_group<32>(p, a.x_bf16 != 0, groups * ks, (size_t)lay.total, s);
        case 64: return launch_group<64>(p, a.x_bf16 != 0, groups * ks, (size_t)lay.total, s);
        default: return launch_group<128>(p, a.x_bf16 != 0, groups * ks, (size_t)lay.total, s);
    }
}

}  // namespace kda
