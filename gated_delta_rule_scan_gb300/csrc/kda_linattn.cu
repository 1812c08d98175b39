// kda_linattn.cu -- linear attention with one log-decay a head, the recurrent form: for each sequence
// and value head, token by token,
//     S <- e^g S + k_t v_t^T,    o_t = scale * S^T q_t
// (the state is stored [value][key]).  One kernel serves the decode / verify step on a pool of states
// and prompts of few tokens (bf16 below 20, f32 below 32) or of callers who ask for it, so that a T-token call
// equals T one-token calls bit for bit.
//
// A value column's recurrence needs only its own 128 state elements, so a state is cut into blocks of
// kRows columns, one CTA each: 8 lanes own a column (16 keys a lane, four runs of 4), 4 columns a warp
// at a time, and the readout of a column is a butterfly over its 8 lanes.  A thread's whole share of
// the state sits in registers for all T tokens, and all of its loads go out before anything waits.  A
// decode step is bound by the state's bytes, read and written once: blocks of 32 columns leave enough
// CTAs per SM to keep HBM busy, and a single sequence spreads over 4 CTAs a head.
// Measured: 64 sequences x 64 heads, one token: 83.7 us, 6.5 TB/s; 37 x 16 heads of 256 values, 3 f32 tokens
// each: 24.7 us, 5.6 TB/s; one sequence x 64 heads 4.4 us, three of them a launch's.
#include "kda_q8.cuh"

namespace kda {

namespace {

constexpr int kThr = 128;
constexpr int kRows = 32;                        // value columns (state rows) of a CTA
constexpr int kBlocks = kHeadDim / kRows;        // CTAs of a 128-wide unit
constexpr int kTile = 16;                        // tokens staged at a time
constexpr int kRowsPerLane = kRows * 8 / kThr;   // columns a lane works on

template <bool BF16>
struct Raw;
template <>
struct Raw<false> {
    using T = float;
    static __device__ __forceinline__ float4 load4(const T* p) { return *reinterpret_cast<const float4*>(p); }
    static __device__ __forceinline__ float load(const T* p) { return *p; }
};
template <>
struct Raw<true> {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ float4 load4(const T* p) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                           __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
    }
    static __device__ __forceinline__ float load(const T* p) { return __bfloat162float(*p); }
};

template <typename T>
struct __align__(16) Stage {
    T q[kTile][kHeadDim], k[kTile][kHeadDim], v[kTile][kRows];
};

template <bool BF16, bool POOL>
__global__ void __launch_bounds__(kThr) kda_linattn_step_kernel(const LinArgs a) {
    using R = Raw<BF16>;
    using T = typename R::T;
    constexpr int kStages = POOL ? 1 : 2;        // a decode step is at most one tile
    __shared__ Stage<T> stage[kStages];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x / kBlocks, rb = blockIdx.x % kBlocks, n = blockIdx.y;
    const int units = a.H * a.m, hv = unit / a.m, hk = hv % a.Hk;

    long begin, in_row = n, out_row = n;
    int len, rows_stride;
    if constexpr (POOL) {
        const int in = a.slots ? a.slots[n] : n;
        const int out = a.slots_out ? a.slots_out[n] : in;
        if (in < 0 || out < 0) return;                        // padding
        if (in >= a.pool_rows || out >= a.pool_rows) {
            if (tid == 0 && a.err) atomicOr(a.err, kDevErrSlot);
            return;
        }
        in_row = in;
        out_row = out;
        rows_stride = a.seq.T_uniform;
        begin = (long)n * rows_stride;
        len = a.keep ? min(max(a.keep[n], 0), rows_stride) : rows_stride;
    } else if (a.seq.cu_seqlens != nullptr) {
        begin = a.seq.cu_seqlens[n];
        len = a.seq.cu_seqlens[n + 1] - (int)begin;
    } else {
        begin = (long)n * a.seq.T_uniform;
        len = a.seq.T_uniform;
    }

    // the state: lane (column c, part p) keeps keys 32 i + 4 p .. + 3 (i < 4) of columns c + 4 warp ...
    const int part = lane & 7;
    const int col = warp * (4 * kRowsPerLane) + (lane >> 3);  // its columns: col + 4 r
    const long soff = (long)rb * kRows * kHeadDim + 4 * part;
    float2 S[kRowsPerLane][8];
    if (a.state_in != nullptr) {
        const float* src = a.state_in + (in_row * units + unit) * (long)(kHeadDim * kHeadDim) + soff;
#pragma unroll
        for (int r = 0; r < kRowsPerLane; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 x = __ldcs(reinterpret_cast<const float4*>(
                    src + (col + 4 * r) * kHeadDim + 32 * i));
                S[r][2 * i] = make_float2(x.x, x.y);
                S[r][2 * i + 1] = make_float2(x.z, x.w);
            }
    } else {
#pragma unroll
        for (int r = 0; r < kRowsPerLane; ++r)
#pragma unroll
            for (int i = 0; i < 8; ++i) S[r][i] = make_float2(0.0f, 0.0f);
    }

    // token rows through shared memory, kTile at a time
    const T* q = static_cast<const T*>(a.q) + begin * a.q_stride + hk * kHeadDim;
    const T* k = static_cast<const T*>(a.k) + begin * a.k_stride + hk * kHeadDim;
    const T* v = static_cast<const T*>(a.v) + begin * a.v_stride + (long)unit * kHeadDim + rb * kRows;
    constexpr int kPer16 = 16 / sizeof(T);
    constexpr int kQ = kHeadDim / kPer16, kV = kRows / kPer16, kRow = 2 * kQ + kV;   // 16-byte pieces
    auto fetch = [&](int t0, int st) {
        const int nt = min(kTile, len - t0);
        for (int x = tid; x < nt * kRow; x += kThr) {
            const int t = x / kRow, c = x % kRow;
            const long row = t0 + t;
            if (c < kQ) cp_async16(&stage[st].q[t][c * kPer16], q + row * a.q_stride + c * kPer16);
            else if (c < 2 * kQ)
                cp_async16(&stage[st].k[t][(c - kQ) * kPer16], k + row * a.k_stride + (c - kQ) * kPer16);
            else cp_async16(&stage[st].v[t][(c - 2 * kQ) * kPer16], v + row * a.v_stride + (c - 2 * kQ) * kPer16);
        }
        cp_async_commit();
    };
    if (len > 0) fetch(0, 0);

    if constexpr (POOL) {
        // the whole batch is looked over for a row that reads this one's output slot or writes it
        // first, while the state is on its way
        bool clash = false;
        if (a.slots || a.slots_out)
            for (int x = lane; x < (int)gridDim.y; x += 32) {
                const int im = a.slots ? a.slots[x] : x;
                clash |= pool_rows_clash(im, a.slots_out ? a.slots_out[x] : im, n, (int)out_row, x, a.pool_rows);
            }
        if (__any_sync(0xffffffffu, clash)) {
            if (tid == 0 && a.err) atomicOr(a.err, kDevErrSlot);
            cp_async_wait_all();
            return;                                           // every warp sees the same slots
        }
    }

    // e^g S: for e^g above a half as S + (e^g - 1) S, so that a decay next to 1 keeps its distance
    // from 1 to 24 bits (rounded to f32 it would be off by up to 2^-25 at each of many thousand steps)
    const float g = a.log_decay[hv], lam = expf(g);
    const bool near1 = lam > 0.5f;
    const float fa = near1 ? 1.0f : lam, fd = near1 ? expm1f(g) : 0.0f;
    const float2 fa2 = make_float2(fa, fa), fd2 = make_float2(fd, fd);

    float* o = a.o + begin * units * kHeadDim + (long)unit * kHeadDim + rb * kRows;
    int st = 0;
    for (int t0 = 0; t0 < len; t0 += kTile) {
        cp_async_wait_all();
        __syncthreads();
        if (kStages > 1 && t0 + kTile < len) fetch(t0 + kTile, st ^ 1);
        const Stage<T>& sm = stage[st];
        const int nt = min(kTile, len - t0);
#pragma unroll 2
        for (int t = 0; t < nt; ++t) {
            float4 kk[4], qq[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                kk[i] = R::load4(&sm.k[t][32 * i + 4 * part]);
                qq[i] = R::load4(&sm.q[t][32 * i + 4 * part]);
            }
            float out[kRowsPerLane];
#pragma unroll
            for (int r = 0; r < kRowsPerLane; ++r) {
                const float vv = R::load(&sm.v[t][col + 4 * r]);
                const float2 v2 = make_float2(vv, vv);
                float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 k0 = make_float2(kk[i].x, kk[i].y), k1 = make_float2(kk[i].z, kk[i].w);
                    float2& s0 = S[r][2 * i];
                    float2& s1 = S[r][2 * i + 1];
                    s0 = __ffma2_rn(fa2, s0, __ffma2_rn(fd2, s0, __fmul2_rn(v2, k0)));
                    s1 = __ffma2_rn(fa2, s1, __ffma2_rn(fd2, s1, __fmul2_rn(v2, k1)));
                    acc[0] = __ffma2_rn(s0, make_float2(qq[i].x, qq[i].y), acc[0]);
                    acc[1] = __ffma2_rn(s1, make_float2(qq[i].z, qq[i].w), acc[1]);
                }
                out[r] = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
            }
#pragma unroll
            for (int r = 0; r < kRowsPerLane; ++r) out[r] = group8_sum(out[r]);
            if (part == 0) {
#pragma unroll
                for (int r = 0; r < kRowsPerLane; ++r)
                    o[(long)(t0 + t) * units * kHeadDim + col + 4 * r] = __fmul_rn(a.scale, out[r]);
            }
        }
        __syncthreads();
        st ^= kStages - 1;
    }

    float* dst = a.state_out + (out_row * units + unit) * (long)(kHeadDim * kHeadDim) + soff;
#pragma unroll
    for (int r = 0; r < kRowsPerLane; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            __stcs(reinterpret_cast<float4*>(dst + (col + 4 * r) * kHeadDim + 32 * i),
                   make_float4(S[r][2 * i].x, S[r][2 * i].y, S[r][2 * i + 1].x, S[r][2 * i + 1].y));
}

template <bool POOL>
cudaError_t launch(const LinArgs& a, cudaStream_t s) {
    const dim3 grid((unsigned)(a.H * a.m * kBlocks), (unsigned)a.seq.N);
    KernelTimer kt(kKLinStep, s);
    if (a.bf16) kda_linattn_step_kernel<true, POOL><<<grid, kThr, 0, s>>>(a);
    else kda_linattn_step_kernel<false, POOL><<<grid, kThr, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linattn_decode(const LinArgs& a, cudaStream_t s) { return launch<true>(a, s); }
cudaError_t launch_linattn_seq(const LinArgs& a, cudaStream_t s) { return launch<false>(a, s); }

}  // namespace kda
