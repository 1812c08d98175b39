// kda_decode_q8.cuh -- what the two forms of the decode step on the 8-bit pool share.
#pragma once

#include "kda_q8.cuh"

namespace kda {

// The form for up to kDecodeQ8FewT tokens (kda_decode_q8_few.cu).
constexpr int kDecodeQ8FewT = 4;
cudaError_t launch_decode_q8_few(const DecodeQ8Args& a, cudaStream_t s);

namespace {

// The conv of one channel: K taps over the ring slots and the new samples, oldest first.  KT = 4
// is a conv of exactly 4 taps (16-byte weights); KT = 8 any width up to 8.
template <int KT>
struct Conv {
    float w[KT], x[KT];
    __device__ __forceinline__ void weights(const float* conv_w, long ch, int K) {
        if constexpr (KT == 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(conv_w + ch * 4));
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else {
#pragma unroll
            for (int m = 0; m < KT; ++m) {
                const int jj = m - (KT - K);
                w[m] = jj >= 0 ? conv_w[ch * K + jj] : 0.0f;
            }
        }
    }
    __device__ __forceinline__ void load(const float* ring, long ch, int K) {
        if constexpr (KT == 4) {
            const float* p = ring + ch * 3;
            x[0] = 0.0f; x[1] = p[0]; x[2] = p[1]; x[3] = p[2];
        } else {
            const float* p = ring + ch * (K - 1);
#pragma unroll
            for (int m = 0; m < KT; ++m) {
                const int d = KT - m;
                x[m] = d <= K - 1 ? p[K - 1 - d] : 0.0f;
            }
        }
    }
    __device__ __forceinline__ float step(float v, int K) {
        window_push(x, v);
        return silu_f(conv_taps_f(w, x, KT == 4 ? 4 : K));
    }
    // the last K - 1 samples
    __device__ __forceinline__ void store(float* ring, long ch, int K) const {
        if constexpr (KT == 4) {
            float* p = ring + ch * 3;
            p[0] = x[1]; p[1] = x[2]; p[2] = x[3];
        } else {
            float* p = ring + ch * (K - 1);
#pragma unroll
            for (int m = 0; m < KT; ++m) {
                const int d = KT - 1 - m;
                if (d < K - 1) p[K - 2 - d] = x[m];
            }
        }
    }
};

}  // namespace

}  // namespace kda
