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
// Up to four tokens take the form of kda_decode_q8_few.cu, which reads the state once for all of
// them; this one serves longer verify windows (and a positive gate bound): its state stays in
// registers from token to token, whatever their number.
//
// GB300 layout.  The bytes are a quarter of the f32 decode's (33 KB of state per (sequence, head)
// read and written, against 131 KB), so the instructions around them bound this kernel: at 64
// sequences x 64 heads x 8 tokens it runs 161 us, where its bytes need 38.  One CTA owns one
// (sequence, unit), in four warps: thread = channel of q, k, v and the gate in the prologue, so its
// address work is done by few warps.  8 lanes share 8 value columns, lane r keys 16r .. 16r + 15 of
// each, so that a column's codes are one 16-byte access a lane, its reductions take three steps, and
// every k, decay and q value read from shared memory serves four columns at a time (two: 172 us; the
// shared reads were the most used unit, 69 % of their peak at four tokens); the rows of q, k and the
// decay lie in shared memory in the order that makes those reads conflict-free (key 16r + 4m + e at
// 32m + 4r + e).  The codes of the next four columns are on their way meanwhile.  The l2 norms scale
// the finished sums instead of the vectors.  Of a reduction's lanes each finishes one column: one
// division a lane rounds the state, not two a column.
#include "kda_decode_q8.cuh"

namespace kda {

namespace {

constexpr int kThreads = 128;
constexpr int kCols = 8;                     // value columns of a group of 8 lanes
constexpr int kB = 4;                        // of them unpacked at a time

// Where key i of a q, k or decay row lies in shared memory.
__device__ __forceinline__ int key_pos(int i) { return 32 * ((i >> 2) & 3) + 4 * (i >> 4) + (i & 3); }

// 16 codes (keys 16r ..) of one column as pairs: s[2m], s[2m + 1] are keys 4m .. 4m + 3.
template <int FMT>
__device__ __forceinline__ void unpack16(float2 (&s)[8], uint4 w, float scale) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const float4 v = q8_decode4<FMT>(u[m], scale);
        s[2 * m] = make_float2(v.x, v.y);
        s[2 * m + 1] = make_float2(v.z, v.w);
    }
}
template <int FMT>
__device__ __forceinline__ uint4 pack16(const float2 (&s)[8], float mul) {
    uint32_t u[4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
        u[m] = q8_encode4_once<FMT>(make_float4(s[2 * m].x, s[2 * m].y, s[2 * m + 1].x, s[2 * m + 1].y), mul);
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// The 16 keys of a lane in a q, k or decay row.
__device__ __forceinline__ float4 row4(const float* row, int r, int m) {
    return *reinterpret_cast<const float4*>(row + 32 * m + 4 * r);
}

// Four columns' sums over the four lanes that differ in bits 0 and 1: lane j of them ends with column
// j's.
__device__ __forceinline__ float reduce_columns(const float (&s)[4], int lane) {
    const bool b1 = lane & 2, b0 = lane & 1;
    const float x = (b1 ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, b1 ? s[0] : s[2], 2);
    const float y = (b1 ? s[3] : s[1]) + __shfl_xor_sync(0xffffffffu, b1 ? s[1] : s[3], 2);
    return (b0 ? y : x) + __shfl_xor_sync(0xffffffffu, b0 ? x : y, 1);
}

// WIDE: value heads of d.vsub > 1 units, one cluster of vsub CTAs each.
template <int FMT, int GATE_MODE, int KT, bool WIDE>
__global__ void __launch_bounds__(kThreads, 3) kda_decode_q8_kernel(const DecodeQ8Args p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(16) float rows_s[];
    __shared__ float beta_s[kDecodeMaxT], ascal[kDecodeMaxT];
    __shared__ float part[3][4][kDecodeMaxT];     // q.q, q.k and k.k of four warps
    __shared__ float nss[kDecodeMaxT];            // this unit's RMSNorm sums of squares (WIDE)
    __shared__ int2 row_s;                        // slots in (-1: left out) and out
    const DecodeArgs& a = p.d;
    float* qh = rows_s;                           // [T][128] each; q, k, decay in key_pos order
    float* kh = qh + a.T * kHeadDim;
    float* vh = kh + a.T * kHeadDim;
    float* os = vh + a.T * kHeadDim;
    float* av = os + a.T * kHeadDim;              // per-channel gate only

    // unit h: value column block h % vs of value head gh, which reads q/k head hq
    const int h = blockIdx.x, n = blockIdx.y;
    const int vs = WIDE ? a.vsub : 1;
    const int gh = WIDE ? h / vs : h;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = a.H, K = a.K;
    const int Hg = H / vs;
    const int Hkq = prep_qk_heads(Hg, a.Hk);
    const int hq = gh < Hkq ? gh : gh % Hkq;
    const long row0 = (long)n * a.T;
    const int T = a.keep != nullptr ? min(max(a.keep[n], 0), a.T) : a.T;

    // ---- raw rows on their way to shared memory; they do not depend on the slots.  Thread tid has
    //      channel tid of q, k, v and the gate; two bf16 channels are one copy: the pair's even
    //      thread copies q and v, the odd one k.
    const int pos = key_pos(tid), pair = key_pos(tid & ~1);
    const long wq = plane_width(H, a.Hk, 0), wv = (long)H * kHeadDim, wg = (long)Hg * kHeadDim;
    if (a.raw_bf16) {
        const bool odd = tid & 1;
        const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(odd ? a.k_raw : a.q_raw) +
                                 row0 * wq + hq * kHeadDim + (tid & ~1);
        const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(a.v_raw) + row0 * wv +
                                 (long)h * kHeadDim + tid;
        float* dst = (odd ? kh : qh) + pair;
        for (int t = 0; t < T; ++t) {
            cp_async_4(dst + t * kHeadDim, x + t * wq);
            if (!odd) cp_async_4(vh + t * kHeadDim + tid, v + t * wv);
        }
    } else {
        const long at = row0 * wq + hq * kHeadDim + tid;
        const float* q = reinterpret_cast<const float*>(a.q_raw) + at;
        const float* k = reinterpret_cast<const float*>(a.k_raw) + at;
        const float* v = reinterpret_cast<const float*>(a.v_raw) + row0 * wv + (long)h * kHeadDim + tid;
        for (int t = 0; t < T; ++t) {
            cp_async_4(qh + t * kHeadDim + pos, q + t * wq);
            cp_async_4(kh + t * kHeadDim + pos, k + t * wq);
            cp_async_4(vh + t * kHeadDim + tid, v + t * wv);
        }
    }
    if (GATE_MODE == 0) {
        const float* f = a.f_raw + row0 * wg + (long)gh * kHeadDim + tid;
        for (int t = 0; t < T; ++t) cp_async_4(av + t * kHeadDim + pos, f + t * wg);
    }
    // ---- warp 3 looks the slots over
    if (warp == 3) {
        int in, out;
        const bool ok = pool_row_warp(p.slots, p.slots_out, n, a.N, p.pool_rows, a.err, in, out);
        if (lane == 0) row_s = make_int2(ok ? in : -1, out);
    }
    // ---- what does not depend on them either: conv weights, gate inputs
    const int chq = hq * kHeadDim + tid, chk = (int)plane_offset(H, a.Hk, 1) + chq;
    const int chv = (int)plane_offset(H, a.Hk, 2) + h * kHeadDim + tid;
    Conv<KT> cq, ck, cv;
    cq.weights(a.conv_w, chq, K);
    ck.weights(a.conv_w, chk, K);
    cv.weights(a.conv_w, chv, K);
    const float alog = a.a_log[gh];
    const float dt = GATE_MODE == 0 ? a.dt_bias[(long)gh * kHeadDim + tid] : a.dt_bias[gh];
    if (tid < T) {
        const long rw = (row0 + tid) * Hg + gh;
        beta_s[tid] = sigmoid_f(a.beta_raw[rw]);
        if (GATE_MODE == 1) ascal[tid] = decay_f(gdn_gate_f(a.f_raw[rw], dt, alog));
    }
    __syncthreads();
    const int slot_in = row_s.x, slot_out = row_s.y;
    if (slot_in < 0) {                            // uniform over the cluster: n decides alone
        cp_async_commit_wait();
        return;
    }

    // ---- this group's codes and scales: 8 columns of 16 codes a lane, the first 4 now
    const int grp = lane >> 3, r = lane & 7;
    const int col0 = warp * 32 + grp * kCols;
    const long unit_in = ((long)slot_in * H + h) * kHeadDim + col0;
    const long unit_out = ((long)slot_out * H + h) * kHeadDim + col0;
    const uint4* cin = reinterpret_cast<const uint4*>(p.codes) + unit_in * (kHeadDim / 16) + r;
    uint4* cout = reinterpret_cast<uint4*>(p.codes) + unit_out * (kHeadDim / 16) + r;
    uint4 code[kB];                               // the batch's, then the next one's
#pragma unroll
    for (int c = 0; c < kB; ++c) code[c] = __ldcs(cin + c * (kHeadDim / 16));
    const float scale_l = p.scales[unit_in + r];  // lane r: column r's

    // ---- ring slots
    // a q / k ring row that several units read is rolled by one of them, and only into another
    // slot: in place it is left to the roll kernel that follows
    const bool roll_qk = h == gh * vs && gh < Hkq && (Hkq == H || slot_in != slot_out);
    const long ring_len = ring_channels(H, a.Hk) * (K - 1);
    const float* ring_in = a.ring_out + (long)slot_in * ring_len;
    float* ring_out = a.ring_out + (long)slot_out * ring_len;
    cq.load(ring_in, chq, K);
    ck.load(ring_in, chk, K);
    cv.load(ring_in, chv, K);

    if (T == 0) {       // nothing accepted: the slot passes through unchanged (in place: untouched)
        cp_async_commit_wait();
        if (slot_in != slot_out) {
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                __stcs(cout + c * (kHeadDim / 16), c < kB ? code[c < kB ? c : 0] : __ldcs(cin + c * (kHeadDim / 16)));
            p.scales[unit_out + r] = scale_l;
            cv.store(ring_out, chv, K);
            if (roll_qk) {
                cq.store(ring_out, chq, K);
                ck.store(ring_out, chk, K);
            }
        }
        return;
    }

    // ---- prologue: conv + SiLU and the ring roll, the sums of q and k, the gate
    cp_async_commit_wait();
    __syncwarp();                                 // a pair's two threads copied for each other
    const float rate = GATE_MODE == 0 ? expf(alog) : 0.0f;
    for (int t = 0; t < T; ++t) {
        float* qr = qh + t * kHeadDim;
        float* kr = kh + t * kHeadDim;
        float* vr = vh + t * kHeadDim;
        float q, k, v;
        if (a.raw_bf16) {
            const __nv_bfloat162 q2 = *reinterpret_cast<const __nv_bfloat162*>(qr + pair);
            const __nv_bfloat162 k2 = *reinterpret_cast<const __nv_bfloat162*>(kr + pair);
            const __nv_bfloat162 v2 = *reinterpret_cast<const __nv_bfloat162*>(vr + (tid & ~1));
            q = __bfloat162float(tid & 1 ? q2.y : q2.x);
            k = __bfloat162float(tid & 1 ? k2.y : k2.x);
            v = __bfloat162float(tid & 1 ? v2.y : v2.x);
        } else {
            q = qr[pos];
            k = kr[pos];
            v = vr[tid];
        }
        q = cq.step(q, K);
        k = ck.step(k, K);
        v = cv.step(v, K);
        __syncwarp();                             // both threads have read the pair's raw samples
        qr[pos] = q;
        kr[pos] = k;
        vr[tid] = v;
        if (GATE_MODE == 0) {
            float* ar = av + t * kHeadDim + pos;
            *ar = decay_f(kda_gate_f(*ar, dt, rate, a.gate_lb));
        }
        // three sums over the warp: lanes 0-7 end with q.q, 8-15 with q.k, 16-23 with k.k
        const float qq = q * q, kk = k * k, qk = q * k;
        const bool b4 = lane & 16, b3 = lane & 8;
        const float h0 = (b4 ? kk : qq) + __shfl_xor_sync(0xffffffffu, b4 ? qq : kk, 16);
        const float h1 = (b4 ? 0.0f : qk) + __shfl_xor_sync(0xffffffffu, b4 ? qk : 0.0f, 16);
        float s = (b3 ? h1 : h0) + __shfl_xor_sync(0xffffffffu, b3 ? h0 : h1, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        if ((lane & 7) == 0 && lane < 24) part[lane >> 3][warp][t] = s;
    }
    cv.store(ring_out, chv, K);
    if (roll_qk) {
        cq.store(ring_out, chq, K);
        ck.store(ring_out, chk, K);
    }
    // the epilogue's norm weight and first gate row, requested ahead of the recurrence
    const long C = (long)H * kHeadDim;
    const float4 w4 = __ldg(reinterpret_cast<const float4*>(
        a.norm_w + (WIDE ? (int)blockIdx.x % a.vsub : 0) * kHeadDim + 4 * lane));
    float4 z_first = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (warp < T)
        z_first = __ldcs(reinterpret_cast<const float4*>(a.gate_raw + (row0 + warp) * C + h * kHeadDim + 4 * lane));
    __syncthreads();
    // lane t holds token t's l2 scales, normalised q.k and beta
    float iq_l = 0.0f, ik_l = 0.0f, qk_l = 0.0f, beta_l = 0.0f;
    if (lane < T) {
        float s[3];
#pragma unroll
        for (int j = 0; j < 3; ++j)
            s[j] = (part[j][0][lane] + part[j][1][lane]) + (part[j][2][lane] + part[j][3][lane]);
        iq_l = l2_inv_f(s[0], a.l2_eps);
        ik_l = l2_inv_f(s[2], a.l2_eps);
        qk_l = s[1] * iq_l * ik_l;
        beta_l = beta_s[lane];
    }

    // ---- the recurrence, four columns of each group at a time
    // (rolled: four copies of it would not fit the instruction cache)
    const bool b2 = lane & 4;
    const int own = lane & 3;                     // the column whose sums end here
#pragma unroll 1
    for (int b = 0; b < kCols; b += kB) {
        float2 S[kB][8];
#pragma unroll
        for (int c = 0; c < kB; ++c)
            unpack16<FMT>(S[c], code[c], __shfl_sync(0xffffffffu, scale_l, (lane & ~7) + b + c));
#pragma unroll
        for (int c = 0; c < kB; ++c)
            if (b + kB + c < kCols) code[c] = __ldcs(cin + (b + kB + c) * (kHeadDim / 16));
#pragma unroll 1
        for (int t = 0; t < T; ++t) {
            const float* krow = kh + t * kHeadDim;
            const float* qrow = qh + t * kHeadDim;
            const float* arow = av + t * kHeadDim;
            const float as = GATE_MODE == 0 ? 0.0f : ascal[t];
            float4 k4[4];
            float2 dk[kB][2], dq[kB][2];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                k4[m] = row4(krow, r, m);
                const float4 q4 = row4(qrow, r, m);
                const float4 a4 = GATE_MODE == 0 ? row4(arow, r, m) : make_float4(as, as, as, as);
                const float2 al = make_float2(a4.x, a4.y), ah = make_float2(a4.z, a4.w);
                const float2 kl = make_float2(k4[m].x, k4[m].y), kh2 = make_float2(k4[m].z, k4[m].w);
                const float2 ql = make_float2(q4.x, q4.y), qh2 = make_float2(q4.z, q4.w);
#pragma unroll
                for (int c = 0; c < kB; ++c) {
                    S[c][2 * m] = __fmul2_rn(S[c][2 * m], al);
                    S[c][2 * m + 1] = __fmul2_rn(S[c][2 * m + 1], ah);
                    if (m == 0) {
                        dk[c][0] = __fmul2_rn(S[c][0], kl);
                        dk[c][1] = __fmul2_rn(S[c][1], kh2);
                        dq[c][0] = __fmul2_rn(S[c][0], ql);
                        dq[c][1] = __fmul2_rn(S[c][1], qh2);
                    } else {
                        dk[c][0] = __ffma2_rn(S[c][2 * m], kl, dk[c][0]);
                        dk[c][1] = __ffma2_rn(S[c][2 * m + 1], kh2, dk[c][1]);
                        dq[c][0] = __ffma2_rn(S[c][2 * m], ql, dq[c][0]);
                        dq[c][1] = __ffma2_rn(S[c][2 * m + 1], qh2, dq[c][1]);
                    }
                }
            }
            // 8 sums over the 8 lanes: lanes with bit 2 clear end with P.k, the others with P.q, of
            // column `own`
            float sum[kB];
#pragma unroll
            for (int c = 0; c < kB; ++c) {
                const float sk = (dk[c][0].x + dk[c][0].y) + (dk[c][1].x + dk[c][1].y);
                const float sq = (dq[c][0].x + dq[c][0].y) + (dq[c][1].x + dq[c][1].y);
                sum[c] = (b2 ? sq : sk) + __shfl_xor_sync(0xffffffffu, b2 ? sk : sq, 4);
            }
            const float red = reduce_columns(sum, lane);
            const float iq = __shfl_sync(0xffffffffu, iq_l, t), ik = __shfl_sync(0xffffffffu, ik_l, t);
            const float qk = __shfl_sync(0xffffffffu, qk_l, t), beta = __shfl_sync(0xffffffffu, beta_l, t);
            const int col = col0 + b + own;
            const float w = beta * (vh[t * kHeadDim + col] - ik * red);      // in lanes of P.k
            const float wo = __shfl_xor_sync(0xffffffffu, w, 4);
            if (b2) os[t * kHeadDim + col] = __fmul_rn(a.scale, fmaf(wo, qk, iq * red));
            const float wk = w * ik;
#pragma unroll
            for (int c = 0; c < kB; ++c) {
                const float wc = __shfl_sync(0xffffffffu, wk, (lane & ~7) + c);
                const float2 w2 = make_float2(wc, wc);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    S[c][2 * m] = __ffma2_rn(make_float2(k4[m].x, k4[m].y), w2, S[c][2 * m]);
                    S[c][2 * m + 1] = __ffma2_rn(make_float2(k4[m].z, k4[m].w), w2, S[c][2 * m + 1]);
                }
            }
        }
        // back to 8 bits: lane l of a group finishes column l / 2; even lanes form the scale, odd ones
        // the multiplier
        float mx[kB];
#pragma unroll
        for (int c = 0; c < kB; ++c) {
            float m = mag_max(S[c][0].x, S[c][0].y);
#pragma unroll
            for (int i = 1; i < 8; ++i) m = mag_max3(m, S[c][i].x, S[c][i].y);
            mx[c] = m;
        }
        const bool b1 = lane & 2;
        const float m0 = mag_max(b2 ? mx[2] : mx[0], __shfl_xor_sync(0xffffffffu, b2 ? mx[0] : mx[2], 4));
        const float m1 = mag_max(b2 ? mx[3] : mx[1], __shfl_xor_sync(0xffffffffu, b2 ? mx[1] : mx[3], 4));
        float top = mag_max(b1 ? m1 : m0, __shfl_xor_sync(0xffffffffu, b1 ? m0 : m1, 2));
        top = mag_max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        const float f = q8_row_part<FMT>(mag_bits(top), lane & 1);
#pragma unroll
        for (int c = 0; c < kB; ++c)
            __stcs(cout + (b + c) * (kHeadDim / 16),
                   pack16<FMT>(S[c], __shfl_sync(0xffffffffu, f, (lane & ~7) + 2 * c + 1)));
        if (!(lane & 1)) p.scales[unit_out + b + r / 2] = f;
    }
    __syncthreads();
    // ---- epilogue: gated RMSNorm, one warp per token row (as in kda_decode_fused)
    if constexpr (WIDE) {
        for (int t = warp; t < T; t += kThreads / 32) {
            const float4 o4 = *reinterpret_cast<const float4*>(os + t * kHeadDim + 4 * lane);
            const float ss = warp_sum((o4.x * o4.x + o4.y * o4.y) + (o4.z * o4.z + o4.w * o4.w));
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
            inv = rms_inv_f(warp_sum((o4.x * o4.x + o4.y * o4.y) + (o4.z * o4.z + o4.w * o4.w)), a.rms_eps);
        }
        const long base = (row0 + t) * C + h * kHeadDim + 4 * lane;
        const float4 z4 = t == warp ? z_first : *reinterpret_cast<const float4*>(a.gate_raw + base);
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
// unit has read them.  One thread per channel.  Launched as the decode kernel's programmatic dependent.
__global__ void __launch_bounds__(kThreads) kda_ring_roll_q8_kernel(const DecodeQ8Args p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const DecodeArgs& a = p.d;
    const int n = blockIdx.y, R = a.K - 1;
    int slot_in, slot_out;
    // (the decode kernel has reported bad slots already)
    if (!pool_row_warp(p.slots, p.slots_out, n, a.N, p.pool_rows, nullptr, slot_in, slot_out)) return;
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
    if (a.d.vsub > 1)
        return a.d.K == 4 ? launch_kernel(kda_decode_q8_kernel<FMT, GM, 4, true>, a, smem, s)
                          : launch_kernel(kda_decode_q8_kernel<FMT, GM, kMaxConvK, true>, a, smem, s);
    return a.d.K == 4 ? launch_kernel(kda_decode_q8_kernel<FMT, GM, 4, false>, a, smem, s)
                      : launch_kernel(kda_decode_q8_kernel<FMT, GM, kMaxConvK, false>, a, smem, s);
}

}  // namespace

cudaError_t launch_decode_q8(const DecodeQ8Args& a, cudaStream_t s) {
    if (a.d.N == 0) return cudaSuccess;
    cudaError_t e;
    {
        KernelTimer kt(kKDecodeQ8, s);
        // (a positive gate bound lets decays grow past 1, out of the range of the form for few,
        // which reads a slot before it knows whether the pool has it)
        if (a.d.T <= kDecodeQ8FewT && a.pool_rows > 0 && (a.d.gate_mode != 0 || a.d.gate_lb <= 0.0f))
            e = launch_decode_q8_few(a, s);
        else if (a.fmt == kQ8E4m3)
            e = a.d.gate_mode == 0 ? launch_t<kQ8E4m3, 0>(a, s) : launch_t<kQ8E4m3, 1>(a, s);
        else
            e = a.d.gate_mode == 0 ? launch_t<kQ8Int8, 0>(a, s) : launch_t<kQ8Int8, 1>(a, s);
    }
    if (e != cudaSuccess || a.d.Hk == a.d.H) return e;
    KernelTimer kt(kKRingRollQ8, s);
    const int blocks = (int)((2 * plane_width(a.d.H, a.d.Hk, 0) + kThreads - 1) / kThreads);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)a.d.N);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kda_ring_roll_q8_kernel, a);
}

}  // namespace kda
