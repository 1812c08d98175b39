// kda_decode_q8.cu -- one decode step, speculative verify or rollback on the 8-bit state pool:
// kda_decode_fused's computation, with each sequence's state and conv ring in a pool slot, the
// state read as 8-bit codes and row scales (kda_q8.cuh) and written back the same way.
//
// Mathematics, for each (sequence, value head) and token, with the state's value column j as the
// row S_j of 128 keys:
//     P_j = a * S_j,   u_j = v_j - P_j . k,   S_j <- P_j + (beta u_j) k,
//     o_j = scale * (P_j . q + (beta u_j) (q . k)),
// the last line being S_j . q written with the state from before the update, so that one reduction
// finishes both dot products of a column and the readout needs no second pass; q . k is one number
// per token.  The state is f32 in registers over all tokens of the call and is rounded to 8 bits
// once, at the end.
//
// GB300 layout.  The bytes are a quarter of the f32 decode's (33 KB of state per (sequence, head)
// read and written, against 131 KB), so the fixed work of a CTA weighs more, and the f32 layout (a
// whole 64 KB state in the registers of two CTAs per SM) would leave the memory idle between its
// phases.  Here a warp owns 16 value columns as two batches of 8 and lane l keys 4l .. 4l+3: the
// codes of all 16 columns wait in 16 registers as they came (one 128-byte access a column), only 8
// columns are unpacked at a time, and k, q and the decay are 12 registers that serve every column.
// That fits three CTAs on an SM.  The 16 sums of a batch (8 columns, P.k and P.q) are finished by
// one transposed butterfly of 16 shuffles, which leaves value index i in lanes 2i and 2i+1.
#include "kda_q8.cuh"

namespace kda {

namespace {

constexpr int kThreads = 256;
constexpr int kColsPerWarp = kHeadDim / (kThreads / 32);   // 16
constexpr int kBatch = 8;                                   // columns unpacked at a time
constexpr int kMinBlocks = 3;

// Transposed butterfly over the warp for 16 values per lane: lane l ends with the full sum of value
// index l >> 1.
__device__ __forceinline__ float reduce16(const float (&v)[16], int lane) {
    float k8[8], k4[4], k2[2];
    const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4, b1 = lane & 2;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        k8[i] = (b4 ? v[8 + i] : v[i]) + __shfl_xor_sync(0xffffffffu, b4 ? v[i] : v[8 + i], 16);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        k4[i] = (b3 ? k8[4 + i] : k8[i]) + __shfl_xor_sync(0xffffffffu, b3 ? k8[i] : k8[4 + i], 8);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        k2[i] = (b2 ? k4[2 + i] : k4[i]) + __shfl_xor_sync(0xffffffffu, b2 ? k4[i] : k4[2 + i], 4);
    float s = (b1 ? k2[1] : k2[0]) + __shfl_xor_sync(0xffffffffu, b1 ? k2[0] : k2[1], 2);
    return s + __shfl_xor_sync(0xffffffffu, s, 1);
}

__device__ __forceinline__ float dot4(float4 a, float4 b) {
    const float2 p = __ffma2_rn(make_float2(a.z, a.w), make_float2(b.z, b.w),
                                __fmul2_rn(make_float2(a.x, a.y), make_float2(b.x, b.y)));
    return p.x + p.y;
}
__device__ __forceinline__ float4 mul4(float4 a, float4 b) {
    const float2 lo = __fmul2_rn(make_float2(a.x, a.y), make_float2(b.x, b.y));
    const float2 hi = __fmul2_rn(make_float2(a.z, a.w), make_float2(b.z, b.w));
    return make_float4(lo.x, lo.y, hi.x, hi.y);
}
// a * s + c
__device__ __forceinline__ float4 fma4(float4 a, float s, float4 c) {
    const float2 s2 = make_float2(s, s);
    const float2 lo = __ffma2_rn(make_float2(a.x, a.y), s2, make_float2(c.x, c.y));
    const float2 hi = __ffma2_rn(make_float2(a.z, a.w), s2, make_float2(c.z, c.w));
    return make_float4(lo.x, lo.y, hi.x, hi.y);
}

// KW: register window of the conv (4 when K <= 4, else 8).  WIDE: value heads of d.vsub > 1 units,
// one cluster of vsub CTAs each.
template <int FMT, int GATE_MODE, int KW, bool WIDE>
__global__ void __launch_bounds__(kThreads, kMinBlocks) kda_decode_q8_kernel(const DecodeQ8Args p) {
    extern __shared__ __align__(16) float rows_s[];
    __shared__ float beta_s[kDecodeMaxT], ascal[kDecodeMaxT], qk_s[kDecodeMaxT];
    __shared__ float part[3][2][kDecodeMaxT];     // q.q, k.k and q.k of two warps each
    __shared__ float inv_s[2][kDecodeMaxT];
    __shared__ float nss[kDecodeMaxT];            // this unit's RMSNorm sums of squares (WIDE)
    const DecodeArgs& a = p.d;
    float* qh = rows_s;                           // [T][128] each
    float* kh = qh + a.T * kHeadDim;
    float* vh = kh + a.T * kHeadDim;
    float* os = vh + a.T * kHeadDim;
    float* av = os + a.T * kHeadDim;              // per-channel gate only

    // unit h: value column block h % vs of value head gh, which reads q/k head hq
    const int h = blockIdx.x, n = blockIdx.y;
    const int vs = WIDE ? a.vsub : 1;
    const int gh = WIDE ? h / vs : h;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = a.H, K = a.K, R = a.K - 1;
    const long C = (long)H * kHeadDim;
    const int Hg = H / vs;
    const long Cg = (long)Hg * kHeadDim;
    const int Hkq = prep_qk_heads(Hg, a.Hk);
    const int hq = gh % Hkq;
    const long row0 = (long)n * a.T;
    const int T = a.keep != nullptr ? min(max(a.keep[n], 0), a.T) : a.T;

    // ---- raw rows on their way to shared memory; they do not depend on the slots
    const int task = tid >> 6, i0 = 2 * (tid & 63);
    const int cg = gh * kHeadDim + i0;
    float* dst = task == 0 ? qh : (task == 1 ? kh : vh);
    if (task < 3) {
        const void* raw = task == 0 ? a.q_raw : (task == 1 ? a.k_raw : a.v_raw);
        const long Cp = plane_width(H, a.Hk, task);
        const int cp = (task < 2 ? hq : h) * kHeadDim + i0;
        for (int t = 0; t < T; ++t) {
            if (a.raw_bf16)
                cp_async_4(dst + t * kHeadDim + i0,
                           reinterpret_cast<const __nv_bfloat16*>(raw) + (row0 + t) * Cp + cp);
            else
                cp_async_8(dst + t * kHeadDim + i0,
                           reinterpret_cast<const float*>(raw) + (row0 + t) * Cp + cp);
        }
    } else if (GATE_MODE == 0) {
        for (int t = 0; t < T; ++t)
            cp_async_8(av + t * kHeadDim + i0, a.f_raw + (row0 + t) * Cg + cg);
    }
    int slot_in, slot_out;
    const bool ok = pool_row(p.slots, p.slots_out, n, a.N, p.pool_rows, kThreads, a.err, slot_in,
                             slot_out);
    if (!ok) {                                    // uniform over the cluster: n decides alone
        cp_async_commit_wait();
        return;
    }

    // ---- this warp's codes and scales
    const long unit_in = ((long)slot_in * H + h) * kHeadDim + warp * kColsPerWarp;
    const long unit_out = ((long)slot_out * H + h) * kHeadDim + warp * kColsPerWarp;
    const uint32_t* cin = reinterpret_cast<const uint32_t*>(p.codes) + unit_in * (kHeadDim / 4) + lane;
    uint32_t* cout = reinterpret_cast<uint32_t*>(p.codes) + unit_out * (kHeadDim / 4) + lane;
    uint32_t code[kColsPerWarp];
#pragma unroll
    for (int c = 0; c < kColsPerWarp; ++c) code[c] = __ldcs(cin + c * (kHeadDim / 4));
    const float scales = p.scales[unit_in + (lane & (kColsPerWarp - 1))];

    // ---- conv weights, ring slots, gate inputs
    float wr[2][KW], win[2][KW];
    long ring_row = 0;
    bool ring_owner = false;
    float braw = 0.0f, fgate = 0.0f, dtb = 0.0f, alog = 0.0f;
    float2 dt = make_float2(0.0f, 0.0f);
    const long ring_len = ring_channels(H, a.Hk) * R;
    if (task < 3) {
        const long ch = plane_offset(H, a.Hk, task) + (task < 2 ? hq : h) * kHeadDim + i0;
        // a q / k ring row that several units read is rolled by one of them, and only into
        // another slot: in place it is left to the roll kernel that follows
        ring_owner = task == 2 || (h == gh * vs && gh < Hkq && (Hkq == H || slot_in != slot_out));
        ring_row = ch * R;
        const float* ring = a.ring_out + (long)slot_in * ring_len + ring_row;
#pragma unroll
        for (int m = 0; m < KW; ++m) {
            const int jj = m - (KW - K);
            const int d = KW - m;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                wr[e][m] = jj >= 0 ? a.conv_w[(ch + e) * K + jj] : 0.0f;
                win[e][m] = d <= R ? ring[e * R + (R - d)] : 0.0f;
            }
        }
        if (task == 2 && (tid & 63) < T) {
            const long rw = (row0 + (tid & 63)) * Hg + gh;
            braw = a.beta_raw[rw];
            if (GATE_MODE == 1) {
                fgate = a.f_raw[rw];
                dtb = a.dt_bias[gh];
                alog = a.a_log[gh];
            }
        }
    } else if (GATE_MODE == 0) {
        alog = a.a_log[gh];
        dt = *reinterpret_cast<const float2*>(a.dt_bias + cg);
    }

    if (T == 0) {       // nothing accepted: the slot passes through unchanged (in place: untouched)
        cp_async_commit_wait();
        if (slot_in != slot_out) {
#pragma unroll
            for (int c = 0; c < kColsPerWarp; ++c) __stcs(cout + c * (kHeadDim / 4), code[c]);
            if (lane < kColsPerWarp) p.scales[unit_out + lane] = scales;
            if (ring_owner) {
                float* ring = a.ring_out + (long)slot_out * ring_len + ring_row;
#pragma unroll
                for (int m = 0; m < KW; ++m) {
                    const int d = KW - m;
                    if (d <= R) {
                        ring[R - d] = win[0][m];
                        ring[R + R - d] = win[1][m];
                    }
                }
            }
        }
        return;
    }

    // ---- prologue: conv + SiLU and the ring roll, beta, the gate
    if (task < 3) {
        cp_async_commit_wait();
        for (int t = 0; t < T; ++t) {
            float* x2 = dst + t * kHeadDim + i0;
            float2 x;
            if (a.raw_bf16) x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(x2));
            else x = *reinterpret_cast<const float2*>(x2);
            window_push(win[0], x.x);
            window_push(win[1], x.y);
            *reinterpret_cast<float2*>(x2) =
                make_float2(silu_f(conv_taps_f(wr[0], win[0], K)), silu_f(conv_taps_f(wr[1], win[1], K)));
        }
        if (ring_owner) {
            float* ring = a.ring_out + (long)slot_out * ring_len + ring_row;
#pragma unroll
            for (int m = 0; m < KW; ++m) {
                const int d = KW - 1 - m;
                if (d < R) {
                    ring[R - 1 - d] = win[0][m];
                    ring[R + R - 1 - d] = win[1][m];
                }
            }
        }
        if (task == 2 && (tid & 63) < T) {
            const int t = tid & 63;
            beta_s[t] = sigmoid_f(braw);
            if (GATE_MODE == 1) ascal[t] = decay_f(gdn_gate_f(fgate, dtb, alog));
        }
    } else if (GATE_MODE == 0) {
        const float rate = expf(alog);
        cp_async_commit_wait();
        for (int t = 0; t < T; ++t) {
            float2* f2 = reinterpret_cast<float2*>(av + t * kHeadDim + i0);
            const float2 f = *f2;
            *f2 = make_float2(decay_f(kda_gate_f(f.x, dt.x, rate, a.gate_lb)),
                              decay_f(kda_gate_f(f.y, dt.y, rate, a.gate_lb)));
        }
    }
    __syncthreads();
    // ---- q.q (warps 0-1), k.k (warps 2-3) and q.k (warps 4-5) of the conv outputs
    if (task < 3) {
        const float* xa = task == 1 ? kh : qh;
        const float* xb = task == 0 ? qh : kh;
        for (int t = 0; t < T; ++t) {
            const float2 u = *reinterpret_cast<const float2*>(xa + t * kHeadDim + i0);
            const float2 w = *reinterpret_cast<const float2*>(xb + t * kHeadDim + i0);
            const float s = warp_sum(__fmul_rn(u.x, w.x) + __fmul_rn(u.y, w.y));
            if (lane == 0) part[task][warp & 1][t] = s;
        }
    }
    __syncthreads();
    if (tid < T) {
        const float iq = l2_inv_f(part[0][0][tid] + part[0][1][tid], a.l2_eps);
        const float ik = l2_inv_f(part[1][0][tid] + part[1][1][tid], a.l2_eps);
        inv_s[0][tid] = iq;
        inv_s[1][tid] = ik;
        qk_s[tid] = (part[2][0][tid] + part[2][1][tid]) * iq * ik;
    }
    __syncthreads();

    // ---- the recurrence, 8 columns at a time; q and k are scaled as they are read
    const float* vcol = vh + warp * kColsPerWarp;
    float* ocol = os + warp * kColsPerWarp;
#pragma unroll
    for (int b = 0; b < kColsPerWarp; b += kBatch) {
        float4 S[kBatch];
#pragma unroll
        for (int c = 0; c < kBatch; ++c)
            S[c] = q8_decode4<FMT>(code[b + c], __shfl_sync(0xffffffffu, scales, b + c));
        for (int t = 0; t < T; ++t) {
            const float iq = inv_s[0][t], ik = inv_s[1][t];
            float4 q = *reinterpret_cast<const float4*>(qh + t * kHeadDim + 4 * lane);
            float4 k = *reinterpret_cast<const float4*>(kh + t * kHeadDim + 4 * lane);
            q = make_float4(q.x * iq, q.y * iq, q.z * iq, q.w * iq);
            k = make_float4(k.x * ik, k.y * ik, k.z * ik, k.w * ik);
            float4 dec;
            if (GATE_MODE == 0) dec = *reinterpret_cast<const float4*>(av + t * kHeadDim + 4 * lane);
            else dec = make_float4(ascal[t], ascal[t], ascal[t], ascal[t]);
            float v16[16];
#pragma unroll
            for (int c = 0; c < kBatch; ++c) {
                S[c] = mul4(S[c], dec);
                v16[c] = dot4(S[c], k);
                v16[8 + c] = dot4(S[c], q);
            }
            const float red = reduce16(v16, lane);
            const int c_own = (lane >> 1) & 7;
            // lanes 0-15 hold P.k of column lane >> 1, lanes 16-31 P.q of column (lane - 16) >> 1
            const float w = beta_s[t] * (vcol[t * kHeadDim + b + c_own] - red);
            const float wk = __shfl_sync(0xffffffffu, w, lane & 15);
            if (lane >= 16 && (lane & 1) == 0)
                ocol[t * kHeadDim + b + c_own] = __fmul_rn(a.scale, fmaf(wk, qk_s[t], red));
#pragma unroll
            for (int c = 0; c < kBatch; ++c)
                S[c] = fma4(k, __shfl_sync(0xffffffffu, w, 2 * c), S[c]);
        }
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
            const uint32_t m = max(max(mag_bits(S[c].x), mag_bits(S[c].y)),
                                   max(mag_bits(S[c].z), mag_bits(S[c].w)));
            float scale, mul;
            q8_row<FMT>(__reduce_max_sync(0xffffffffu, m), scale, mul);
            __stcs(cout + (b + c) * (kHeadDim / 4), q8_encode4<FMT>(S[c], mul));
            if (lane == 0) p.scales[unit_out + b + c] = scale;
        }
    }
    __syncthreads();
    // ---- epilogue: gated RMSNorm, one warp per token row (as in kda_decode_fused)
    const float4 w4 = *reinterpret_cast<const float4*>(
        a.norm_w + (WIDE ? (int)blockIdx.x % a.vsub : 0) * kHeadDim + 4 * lane);
    if constexpr (WIDE) {
        for (int t = warp; t < T; t += kThreads / 32) {
            const float4 o4 = *reinterpret_cast<const float4*>(os + t * kHeadDim + 4 * lane);
            const float ss = warp_sum(dot4(o4, o4));
            if (lane == 0) nss[t] = ss;
        }
        cluster_sync_all();
    }
    for (int t = warp; t < T; t += kThreads / 32) {
        const float4 o4 = *reinterpret_cast<const float4*>(os + t * kHeadDim + 4 * lane);
        float inv;
        if constexpr (WIDE) {
            float tot = 0.0f;
            for (int b = 0; b < a.vsub; ++b) tot = tot + ld_cluster_f32(&nss[t], (uint32_t)b);
            inv = rms_inv_w(tot, a.rms_eps, a.vsub * kHeadDim);
        } else {
            inv = rms_inv_f(warp_sum(dot4(o4, o4)), a.rms_eps);
        }
        const long base = (row0 + t) * C + h * kHeadDim + 4 * lane;
        const float4 z4 = *reinterpret_cast<const float4*>(a.gate_raw + base);
        float4 y4;
        if (a.norm_silu) {
            y4.x = gated_norm_f<true>(o4.x, inv, w4.x, z4.x);
            y4.y = gated_norm_f<true>(o4.y, inv, w4.y, z4.y);
            y4.z = gated_norm_f<true>(o4.z, inv, w4.z, z4.z);
            y4.w = gated_norm_f<true>(o4.w, inv, w4.w, z4.w);
        } else {
            y4.x = gated_norm_f(o4.x, inv, w4.x, z4.x);
            y4.y = gated_norm_f(o4.y, inv, w4.y, z4.y);
            y4.z = gated_norm_f(o4.z, inv, w4.z, z4.z);
            y4.w = gated_norm_f(o4.w, inv, w4.w, z4.w);
        }
        *reinterpret_cast<float4*>(a.y + base) = y4;
    }
    if constexpr (WIDE) cluster_sync_all();       // the other units have read this unit's sums
}

// The q and k ring rows of in-place rows whose q/k heads several units read: rolled after every
// unit has read them.  One thread per channel.
__global__ void __launch_bounds__(kThreads) kda_ring_roll_q8_kernel(const DecodeQ8Args p) {
    const DecodeArgs& a = p.d;
    const int n = blockIdx.y, R = a.K - 1;
    int slot_in, slot_out;
    // (the decode kernel has reported bad slots already)
    if (!pool_row(p.slots, p.slots_out, n, a.N, p.pool_rows, kThreads, nullptr, slot_in, slot_out))
        return;
    const int T = a.keep != nullptr ? min(max(a.keep[n], 0), a.T) : a.T;
    if (slot_in != slot_out || T == 0) return;
    const int width = (int)plane_width(a.H, a.Hk, 0);
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= 2 * width) return;
    const int plane = c >= width, cp = c - plane * width;
    const void* raw = plane ? a.k_raw : a.q_raw;
    float* ring = a.ring_out + ((long)slot_in * ring_channels(a.H, a.Hk) + c) * R;
    for (int j = 0; j < R; ++j) {
        const int s = j + T;                      // slot s of (ring, new rows)
        float x;
        if (s < R) x = ring[s];
        else if (a.raw_bf16) x = load_raw<true>(raw, ((long)n * a.T + s - R) * width + cp);
        else x = load_raw<false>(raw, ((long)n * a.T + s - R) * width + cp);
        ring[j] = x;
    }
}

template <typename Kern>
cudaError_t launch_kernel(Kern kernel, const DecodeQ8Args& a, size_t smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.d.H, (unsigned)a.d.N);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.d.vsub;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.d.vsub > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int FMT, int GM>
cudaError_t launch_t(const DecodeQ8Args& a, cudaStream_t s) {
    // at most 5 * 16 rows of 512 bytes: 40 KB, within the default limit
    const size_t smem = (size_t)(GM == 0 ? 5 : 4) * a.d.T * kHeadDim * sizeof(float);
    KernelTimer kt(kKDecodeQ8, s);
    if (a.d.vsub > 1)
        return a.d.K <= 4 ? launch_kernel(kda_decode_q8_kernel<FMT, GM, 4, true>, a, smem, s)
                          : launch_kernel(kda_decode_q8_kernel<FMT, GM, kMaxConvK, true>, a, smem, s);
    return a.d.K <= 4 ? launch_kernel(kda_decode_q8_kernel<FMT, GM, 4, false>, a, smem, s)
                      : launch_kernel(kda_decode_q8_kernel<FMT, GM, kMaxConvK, false>, a, smem, s);
}

}  // namespace

cudaError_t launch_decode_q8(const DecodeQ8Args& a, cudaStream_t s) {
    if (a.d.N == 0) return cudaSuccess;
    cudaError_t e;
    if (a.fmt == kQ8E4m3)
        e = a.d.gate_mode == 0 ? launch_t<kQ8E4m3, 0>(a, s) : launch_t<kQ8E4m3, 1>(a, s);
    else
        e = a.d.gate_mode == 0 ? launch_t<kQ8Int8, 0>(a, s) : launch_t<kQ8Int8, 1>(a, s);
    if (e != cudaSuccess || a.d.Hk == a.d.H) return e;
    KernelTimer kt(kKRingRollQ8, s);
    const int blocks = (int)((2 * plane_width(a.d.H, a.d.Hk, 0) + kThreads - 1) / kThreads);
    kda_ring_roll_q8_kernel<<<dim3((unsigned)blocks, (unsigned)a.d.N), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
