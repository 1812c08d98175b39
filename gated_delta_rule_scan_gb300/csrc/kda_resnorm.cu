// kda_resnorm.cu -- the norms after and before a block, fused with the block's gate, its scale and the
// residual sum:
//     h = res_scale * x + block_scale * act(gate) * (rms(y) * block_w),    z = rms(h) * norm_w
// with rms(a) = a / sqrt(mean a^2 + eps) along a row.  Both sums run over a row that stays in registers
// (8 elements a thread and step), so a row is read once and written once; h enters the second norm
// before its rounding to the stream's type.  Bound by HBM for many rows, by the two dependent
// reductions for one.  Measured: 4096 rows x 6144 with a gate 49.2 us, 5.1 TB/s (16384
// rows: 158 us, 6.4 TB/s); one row of f32 6.1 us.  Persistent CTAs with bulk copies three rows ahead and the
// weights in registers took 70 us: two of them on an SM do not hide a row's sums and its gate's exponentials.
#include "kda_device.cuh"

namespace kda {

namespace {

struct V8 {
    float x[8];
};

// Eight elements as they lie in memory: 16 bytes of bf16, 32 of f32.
template <bool BF16>
struct Raw8 {
    uint4 w[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void* base, long i) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + i * (BF16 ? 2 : 4));
        w[0] = __ldcs(p);
        if constexpr (!BF16) w[1] = __ldcs(p + 1);
    }
    __device__ __forceinline__ V8 get() const {
        const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
        V8 v;
        if constexpr (BF16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v.x[2 * j] = __uint_as_float(u[j] << 16);
                v.x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v.x[j] = __uint_as_float(u[j]);
        }
        return v;
    }
};

__device__ __forceinline__ void store8(void* base, long i, const V8& v, bool bf16) {
    if (bf16) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v.x[2 * j], v.x[2 * j + 1]);
            u[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + i) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
        p[0] = make_float4(v.x[0], v.x[1], v.x[2], v.x[3]);
        p[1] = make_float4(v.x[4], v.x[5], v.x[6], v.x[7]);
    }
}

__device__ __forceinline__ V8 load_w(const float* w, int i) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w + i));
    const float4 b = __ldg(reinterpret_cast<const float4*>(w + i + 4));
    return V8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// The sum over a row's threads; every one of them gets it.  part: one float a warp.
template <int THR>
__device__ __forceinline__ float row_sum(float x, float* part) {
    x = warp_sum(x);
    if constexpr (THR > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
        __syncthreads();
        x = 0.0f;
#pragma unroll
        for (int w = 0; w < THR / 32; ++w) x += part[w];
    }
    return x;
}

// One row by THR threads (a CTA, or with THR = 32 each of its kThrNarrow / 32 warps), STEPS times 8
// elements each.
constexpr int kThrNarrow = 128;

template <int THR, int STEPS, bool XB, bool RB>
__global__ void __launch_bounds__(THR == 32 ? kThrNarrow : THR, THR == 256 && STEPS <= 3 && XB && RB ? 4 : 1)
kda_residual_rmsnorm_kernel(const ResNormArgs a) {
    __shared__ float part[2][THR / 32];
    const int t = THR == 32 ? threadIdx.x & 31 : threadIdx.x;
    const long row = THR == 32 ? (long)blockIdx.x * (kThrNarrow / 32) + (threadIdx.x >> 5) : (long)blockIdx.x;
    if (row >= a.rows) return;                   // (THR = 32: whole warps; else never)
    const long base = row * a.F;
    // everything a row needs is on its way before the first sum
    Raw8<XB> y[STEPS], gate[STEPS];
    Raw8<RB> x[STEPS];
    const bool row_gate = a.gate != nullptr && a.gate_per_row;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int i = (s * THR + t) * 8;
        if (i < a.F) {
            if (a.block != nullptr) y[s].load(a.block, base + i);
            x[s].load(a.residual, base + i);
            if (row_gate) gate[s].load(a.gate, base + i);
        }
    }
    float inv = a.block_scale;
    if (a.block_w != nullptr) {
        float ss = 0.0f;
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            if ((s * THR + t) * 8 < a.F) {
                const V8 v = y[s].get();
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(v.x[j], v.x[j], ss);
            }
        ss = row_sum<THR>(ss, part[0]);
        inv = a.block_scale * rsqrtf(ss / (float)a.F + a.eps);
    }
    V8 h[STEPS];
    float ss = 0.0f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int i = (s * THR + t) * 8;
        if (i >= a.F) continue;
        h[s] = x[s].get();
#pragma unroll
        for (int j = 0; j < 8; ++j) h[s].x[j] *= a.res_scale;
        if (a.block != nullptr) {
            V8 v = y[s].get();
#pragma unroll
            for (int j = 0; j < 8; ++j) v.x[j] *= inv;
            if (a.block_w != nullptr) {
                const V8 w = load_w(a.block_w, i);
#pragma unroll
                for (int j = 0; j < 8; ++j) v.x[j] *= w.x[j];
            }
            if (a.gate != nullptr) {
                V8 g = row_gate ? gate[s].get() : load_w(static_cast<const float*>(a.gate), i);
                if (a.gate_act != 0)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float sg = __fdividef(1.0f, 1.0f + expf(-g.x[j]));
                        g.x[j] = a.gate_act == 2 ? g.x[j] * sg : sg;
                    }
#pragma unroll
                for (int j = 0; j < 8; ++j) v.x[j] *= g.x[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) h[s].x[j] += v.x[j];
        }
        if (a.h != nullptr) store8(a.h, base + i, h[s], RB);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(h[s].x[j], h[s].x[j], ss);
    }
    if (a.z == nullptr) return;
    ss = row_sum<THR>(ss, part[1]);
    inv = rsqrtf(ss / (float)a.F + a.eps);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int i = (s * THR + t) * 8;
        if (i >= a.F) continue;
        const V8 w = load_w(a.norm_w, i);
        V8 z;
#pragma unroll
        for (int j = 0; j < 8; ++j) z.x[j] = h[s].x[j] * inv * w.x[j];
        store8(a.z, base + i, z, a.z_bf16);
    }
}

template <int THR, int STEPS>
cudaError_t launch(const ResNormArgs& a, cudaStream_t s) {
    constexpr int rows_per = THR == 32 ? kThrNarrow / 32 : 1;
    const unsigned blocks = (unsigned)((a.rows + rows_per - 1) / rows_per);
    const int thr = THR == 32 ? kThrNarrow : THR;
    KernelTimer kt(kKResNorm, s);
    if (a.block_bf16 && a.residual_bf16) kda_residual_rmsnorm_kernel<THR, STEPS, true, true><<<blocks, thr, 0, s>>>(a);
    else if (a.block_bf16) kda_residual_rmsnorm_kernel<THR, STEPS, true, false><<<blocks, thr, 0, s>>>(a);
    else if (a.residual_bf16) kda_residual_rmsnorm_kernel<THR, STEPS, false, true><<<blocks, thr, 0, s>>>(a);
    else kda_residual_rmsnorm_kernel<THR, STEPS, false, false><<<blocks, thr, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_residual_rmsnorm(const ResNormArgs& a, cudaStream_t s) {
    const int pieces = (a.F + 7) / 8;            // 8 elements each
    if (pieces <= 32) return launch<32, 1>(a, s);
    if (pieces <= 64) return launch<32, 2>(a, s);
    if (pieces <= 256) return launch<256, 1>(a, s);
    if (pieces <= 512) return launch<256, 2>(a, s);
    if (pieces <= 768) return launch<256, 3>(a, s);
    if (pieces <= 1024) return launch<256, 4>(a, s);
    return launch<512, 4>(a, s);
}

}  // namespace kda
