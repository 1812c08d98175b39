// kda_state_q8.cu -- the 8-bit pool of recurrent states: kda_state_store_q8 writes f32 states
// (and conv rings) into pool slots as codes and row scales, kda_state_load_q8 reads them back.
//
// Mathematics and storage: kda_q8.cuh.  Both directions are pure streams, bound by HBM: 4 bytes of
// state on one side, 1 byte of code and 1/32 byte of scale on the other, for about ten
// instructions an element.  One CTA owns one (row, 128-wide value unit), 64 KB of f32 state, and
// extra CTAs of each row copy its ring.  A warp owns whole state rows: lane l holds elements
// 4l .. 4l+3, so a row is one 512-byte access on the f32 side and one 128-byte access on the code
// side, and the row maximum is one warp-wide integer maximum over magnitude bits.  The warp's 16
// rows are issued in two batches of 8, so that 4 KB of each warp is in flight.
// A block looks its row's indices over before its first access; other blocks of the SM stream
// meanwhile.  64 sequences x 64 heads: 59.5 us a store, 59.9 us a load, 93 and 92 % of the copy
// bandwidth.
#include "kda_q8.cuh"

namespace kda {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;                    // state rows of a warp in flight
constexpr int kRingVecs = 4;                 // float4 of a ring row per thread
constexpr int kUnit = kHeadDim * kHeadDim;   // elements of one unit

// Row n's source and destination rows.  A negative index is padding.  An index past its end, or a
// destination that an earlier row writes already, raises the error word; nothing is written.  (Rows
// that are padding or have an index past its end write nothing and claim no destination.)
__device__ __forceinline__ bool move_ok(const StateQ8Args& a, int n, long& src, long& dst) {
    src = a.src ? a.src[n] : n;
    dst = a.dst ? a.dst[n] : n;
    bool bad = src >= a.src_rows || dst >= a.dst_rows;
    if (a.dst && dst >= 0) {
        bool taken = false;
        for (int i = threadIdx.x; i < n; i += kThreads)
            taken |= a.dst[i] == (int)dst && (unsigned)(a.src ? a.src[i] : i) < (unsigned)a.src_rows;
        bad |= taken;
    }
    const bool live = src >= 0 && dst >= 0;
    const bool any = __syncthreads_or(bad && live) != 0;
    if (any && threadIdx.x == 0 && a.err) atomicOr(a.err, kDevErrSlot);
    return live && !any;
}

__device__ __forceinline__ void copy_ring(const StateQ8Args& a, int n, int block) {
    long src, dst;
    if (!move_ok(a, n, src, dst)) return;
    const long vecs = a.ring_row / 4;
    const float4* in = reinterpret_cast<const float4*>(a.ring_src + src * a.ring_row);
    float4* out = reinterpret_cast<float4*>(a.ring_dst + dst * a.ring_row);
    const long i0 = (long)block * (kThreads * kRingVecs) + threadIdx.x;
    float4 v[kRingVecs];
#pragma unroll
    for (int j = 0; j < kRingVecs; ++j)
        if (i0 + j * kThreads < vecs) v[j] = __ldcs(in + i0 + j * kThreads);
#pragma unroll
    for (int j = 0; j < kRingVecs; ++j)
        if (i0 + j * kThreads < vecs) __stcs(out + i0 + j * kThreads, v[j]);
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) kda_state_store_q8_kernel(const StateQ8Args a) {
    const int n = blockIdx.y, unit = blockIdx.x;
    if (unit >= a.units) {
        copy_ring(a, n, unit - a.units);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = warp * (kHeadDim / (kThreads / 32));
    long src, dst;
    const bool ok = move_ok(a, n, src, dst);
    if (!ok) return;
    const float* in = a.state_in + (src * a.units + unit) * kUnit + 4 * lane;
    uint32_t* codes = reinterpret_cast<uint32_t*>(a.codes) + (dst * a.units + unit) * (kUnit / 4) + lane;
    float* scales = a.scales + (dst * a.units + unit) * kHeadDim;
#pragma unroll
    for (int b = 0; b < kHeadDim / (kThreads / 32); b += kBatch) {
        float4 x[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            x[j] = __ldcs(reinterpret_cast<const float4*>(in + (row0 + b + j) * kHeadDim));
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const uint32_t m = max(max(mag_bits(x[j].x), mag_bits(x[j].y)),
                                   max(mag_bits(x[j].z), mag_bits(x[j].w)));
            float scale, mul;
            q8_row<FMT>(__reduce_max_sync(0xffffffffu, m), scale, mul);
            __stcs(codes + (row0 + b + j) * (kHeadDim / 4), q8_encode4<FMT>(x[j], mul));
            if (lane == 0) scales[row0 + b + j] = scale;
        }
    }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) kda_state_load_q8_kernel(const StateQ8Args a) {
    const int n = blockIdx.y, unit = blockIdx.x;
    if (unit >= a.units) {
        copy_ring(a, n, unit - a.units);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = warp * (kHeadDim / (kThreads / 32));
    long src, dst;
    if (!move_ok(a, n, src, dst)) return;
    const uint32_t* codes =
        reinterpret_cast<const uint32_t*>(a.codes) + (src * a.units + unit) * (kUnit / 4) + lane;
    const float* scales = a.scales + (src * a.units + unit) * kHeadDim;
    float* out = a.state_out + (dst * a.units + unit) * kUnit + 4 * lane;
#pragma unroll
    for (int b = 0; b < kHeadDim / (kThreads / 32); b += kBatch) {
        uint32_t w[kBatch];
        float s[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            w[j] = __ldcs(codes + (row0 + b + j) * (kHeadDim / 4));
            s[j] = scales[row0 + b + j];
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            __stcs(reinterpret_cast<float4*>(out + (row0 + b + j) * kHeadDim),
                   q8_decode4<FMT>(w[j], s[j]));
    }
}

dim3 move_grid(const StateQ8Args& a) {
    const long per = (long)kThreads * kRingVecs;
    const long ring_blocks = a.ring_row > 0 ? (a.ring_row / 4 + per - 1) / per : 0;
    return dim3((unsigned)(a.units + ring_blocks), (unsigned)a.N);
}

}  // namespace

cudaError_t launch_state_store_q8(const StateQ8Args& a, cudaStream_t s) {
    KernelTimer kt(kKStateStoreQ8, s);
    if (a.fmt == kQ8E4m3)
        kda_state_store_q8_kernel<kQ8E4m3><<<move_grid(a), kThreads, 0, s>>>(a);
    else
        kda_state_store_q8_kernel<kQ8Int8><<<move_grid(a), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_state_load_q8(const StateQ8Args& a, cudaStream_t s) {
    KernelTimer kt(kKStateLoadQ8, s);
    if (a.fmt == kQ8E4m3)
        kda_state_load_q8_kernel<kQ8E4m3><<<move_grid(a), kThreads, 0, s>>>(a);
    else
        kda_state_load_q8_kernel<kQ8Int8><<<move_grid(a), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
