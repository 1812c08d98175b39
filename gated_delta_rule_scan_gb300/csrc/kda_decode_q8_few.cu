// kda_decode_q8_few.cu -- the decode step on the 8-bit pool (kda_decode_q8.cu) for up to four tokens,
// with the state's codes as a tensor-core operand.
//
// Mathematics.  Unrolled over the call's tokens, everything that token t wants of the state is a dot
// product of the state that came in: with A_t the product of the decays up to token t, D_st that of
// the tokens after s up to t, and k, q normalised,
//     S_j,t-1 decayed, . k_t = S_j . (A_t k_t) + sum_{s<t} w_s (D_st k_s . k_t),
//     w_t = beta_t (v_t - that),      o_t = scale (S_j . (A_t q_t) + sum_{s<=t} w_s (D_st k_s . q_t)),
//     S_j out = A_T S_j + sum_s w_s (D_sT k_s).
// The products D_st k_s . k_t and D_st k_s . q_t belong to the token rows, not to a value column: at
// four tokens they are 16 sums over 128 channels for the whole unit.  The products with the incoming
// state are a matrix product, 128 columns x 128 keys by 2 T vectors: its left side are the codes
// themselves, whole numbers or e4m3 values, exact in f16, the row scale going on afterwards; its
// right side the vectors A_t k_t and A_t q_t, each times the power of two that brings its largest
// element (read to 8 bits) to [2^11, 2^13), as f16 hi + lo: an element is held to 2^-23 of itself or
// 2^-36 of the vector's largest, whichever is more, and mma.sync sums in f32.  (One power of two for
// all vectors loses the readout of a state that has faded, where nothing new covers it: relative
// errors of 2e-2 behind a decay of e^-20, of 1 behind e^-25.)  Decays are at most 1, which keeps the
// vectors finite; a positive gate bound takes the other form.  The new state is formed once, in f32,
// from the codes, and rounded back to 8 bits.
//
// What it saves: one pass over the state's f32 values for all tokens instead of two per token.
// GB300 layout.  One CTA of four warps owns one (sequence, unit).  Thread = channel of q, k, v and
// the gate, and = value column: its v, its row scale and its solve stay in registers.  A warp owns
// 32 columns as two 16-row MMA tiles; lane 4g + c holds of rows g and g + 8 the key words that the MMA
// wants of it, chosen as keys 64 half + 16c .. 16c + 15 so that a row is read and written in 16-byte
// pieces; the same words are the MMA's left side and, unpacked, the state.  Everything a block reads
// is asked for at once, before its slots have been looked over; codes and output gates wait in shared
// memory (in registers: 4 blocks an SM and spills, 45 us at one token and 85 at four, 64 x 64 heads).
// There it runs 40 us at one token, 48 at two, 60 at three and 66 at four, where its bytes need 27 to 32; the
// other form takes 53 at one, 70 at two and 118 at five.  (The vectors' own powers of two cost 0.5 us at one
// token and 3.5 at four, 4 % more instructions.)  What is left is the wait for a block's first bytes, about
// a third of its life, overlapped by four other blocks only.  (Persistent blocks that fetch the next unit by bulk
// copies meanwhile: 62 us; issuing some fifteen small copies a unit takes longer than the wait.)
#include <cuda_fp16.h>

#include "kda_decode_q8.cuh"

namespace kda {

namespace {

constexpr int kThreads = 128;
constexpr int kVecBytes = 320;               // one f16 vector: 256 bytes, and 64 against bank conflicts
constexpr int kDotRow = 136;                 // floats: four lanes' columns land in different banks
constexpr int kVecExp = 11;                  // exponent of a vector's largest element in f16
constexpr int kMinBlocks = 5;                // an SM: 64 x 64 heads, with one power of two for all
                                             // vectors, 39.5 us at one token and 62 at four (4
                                             // blocks: 43 and 67, 6: 40 and 71)

// Key i is byte e of word m (0 .. 7) of lane c: i = 64 (m / 4) + 16 c + 4 (m % 4) + e.
__device__ __forceinline__ int key_word(int i) { return ((i >> 6) << 2) | ((i >> 2) & 3); }
__device__ __forceinline__ int key_lane(int i) { return (i >> 4) & 3; }
// Where it lies in an f32 row (a lane's word is 16 bytes) and in an f16 vector (two words are).
__device__ __forceinline__ int key_pos32(int i) { return (key_word(i) * 4 + key_lane(i)) * 4 + (i & 3); }
__device__ __forceinline__ int key_pos16(int i) {
    const int m = key_word(i);
    return ((m >> 1) * 4 + key_lane(i)) * 8 + (m & 1) * 4 + (i & 3);
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four codes as two f16 pairs, exact.
template <int FMT>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (FMT == kQ8E4m3) {
        const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
        const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
        lo = *reinterpret_cast<const uint32_t*>(&a);
        hi = *reinterpret_cast<const uint32_t*>(&b);
    } else {
        // code + 128 in the mantissa of 1024
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t x = __byte_perm(u, 0x64646464u, 0x4140), y = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 off = __float2half2_rn(1152.0f);
        const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&x), off);
        const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&y), off);
        lo = *reinterpret_cast<const uint32_t*>(&a);
        hi = *reinterpret_cast<const uint32_t*>(&b);
    }
}

__device__ __forceinline__ void cp_async_16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// N sums over the warp's lanes, N a power of two: lane l ends with sum l / (32 / N).
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N], int lane) {
    int bit = 16;
#pragma unroll
    for (int n = N / 2; n >= 1; n /= 2, bit /= 2) {
        const bool up = lane & bit;
#pragma unroll
        for (int j = 0; j < n; ++j)
            v[j] = (up ? v[j + n] : v[j]) + __shfl_xor_sync(0xffffffffu, up ? v[j] : v[j + n], bit);
    }
    float s = v[0];
#pragma unroll
    for (int b = 16 / N; b >= 1; b /= 2) s += __shfl_xor_sync(0xffffffffu, s, b);
    return s;
}

// A raw sample as it lies in memory, and its value.  (Converted when used: a conversion next to the
// load waits for it, token by token: 93 us against 85 at four tokens, 64 x 64 heads.)
__device__ __forceinline__ uint32_t raw_bits(const void* p, long i, bool bf16) {
    if (bf16) return reinterpret_cast<const unsigned short*>(p)[i];
    return reinterpret_cast<const uint32_t*>(p)[i];
}
__device__ __forceinline__ float raw_value(uint32_t x, bool bf16) { return __uint_as_float(bf16 ? x << 16 : x); }

// Two magnitudes by their upper 16 bits, as a bf16 pair; the larger of two pairs, NaN above all.
__device__ __forceinline__ uint32_t mag_pair(float lo, float hi) {
    return __byte_perm(mag_bits(lo), mag_bits(hi), 0x7632);
}
// The power of two that brings magnitude m to [2^kVecExp, 2^(kVecExp + 1)), or one below 2^-100 as
// far as 2^-100 would come; 1 where m is not finite.
__device__ __forceinline__ float vec_factor(float m) {
    const uint32_t bits = mag_bits(m);
    const int e = max((int)(bits >> 23) - 127, -100);
    return bits < 0x7f800000u ? __uint_as_float((uint32_t)(127 + kVecExp - e) << 23) : 1.0f;
}

// TT: tokens of the call at most.  The sums over channels are numbered q.q (t), k.k (TT + t), then
// D k_s . k_t for s < t and D k_s . q_t for s <= t, by t and then s.
template <int TT>
struct Sums {
    static constexpr int kk = TT, kt = 2 * TT, qt = kt + TT * (TT - 1) / 2, n = qt + TT * (TT + 1) / 2;
    static constexpr int padded = n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : 32;
    static constexpr int lanes = 32 / padded;
    __host__ __device__ static constexpr int kk_at(int s, int t) { return kt + t * (t - 1) / 2 + s; }
    __host__ __device__ static constexpr int qk_at(int s, int t) { return qt + t * (t + 1) / 2 + s; }
};

template <int TT>
struct FewSmem {
    uint4 code[kHeadDim * 8];
    static constexpr int kTiles = (TT + 1) / 2;              // MMA tiles of 8 columns: two tokens each
    uint4 vec[8 * kTiles * kVecBytes / 16];                  // hi, lo of k, then of q, token by token
    float row[(TT + 1) * kHeadDim];                          // D_sT k_s, then A_T
    float dot[4 * kTiles * kDotRow];                         // (token, k or q) x columns
    float part[4][Sums<TT>::padded];
    uint4 top[2 * TT];                           // largest |A q| of each token, then |A k|: four warps'
    float z[TT][kHeadDim];
    float beta[TT], nss[TT], osum[4][TT];
};

template <int FMT, int GATE_MODE, int KT, bool WIDE, int TT>
__global__ void __launch_bounds__(kThreads, kMinBlocks) kda_decode_q8_few_kernel(const DecodeQ8Args p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");    // (the ring roll, if one follows)
    __shared__ __align__(16) FewSmem<TT> sm;
    using S_ = Sums<TT>;
    const DecodeArgs& a = p.d;

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

    // ---- raw samples, conv weights and gate inputs: nothing of them depends on the slots
    const long wq = plane_width(H, a.Hk, 0), wv = (long)H * kHeadDim, wg = (long)Hg * kHeadDim;
    const bool bf16 = a.raw_bf16 != 0;
    uint32_t qr[TT], kr[TT], vr[TT];
    float ga[TT];
    {
        const long aq = row0 * wq + hq * kHeadDim + tid, av = row0 * wv + (long)h * kHeadDim + tid;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            qr[t] = kr[t] = vr[t] = 0u;
            ga[t] = 0.0f;
            if (t >= T) continue;
            qr[t] = raw_bits(a.q_raw, aq + t * wq, bf16);
            kr[t] = raw_bits(a.k_raw, aq + t * wq, bf16);
            vr[t] = raw_bits(a.v_raw, av + t * wv, bf16);
            ga[t] = GATE_MODE == 0 ? a.f_raw[(row0 + t) * wg + gh * kHeadDim + tid] : a.f_raw[(row0 + t) * Hg + gh];
            cp_async_4(&sm.z[t][tid], a.gate_raw + av + t * wv);
        }
    }
    const float nw = __ldg(a.norm_w + (WIDE ? (int)blockIdx.x % a.vsub : 0) * kHeadDim + tid);
    // ---- codes, scales and ring of the slot in, asked for before the slots are looked over: what a
    //      row that is left out reads so is dropped
    const int slot_in = p.slots ? p.slots[n] : n;
    const int slot_out = p.slots_out ? p.slots_out[n] : slot_in;
    const int from = min(max(slot_in, 0), p.pool_rows - 1);
    const int g = lane >> 2, c = lane & 3;
    const long unit_in = ((long)from * H + h) * kHeadDim;
    // [row g, row g + 8][half]: 8 pieces of 16 bytes a row, this lane's at c and 4 + c
    const uint4* cin = reinterpret_cast<const uint4*>(p.codes) + (unit_in + warp * 32 + g) * 8 + c;
    // (a lane reads what it copied itself, so its pieces lie 32 lanes apart: no bank conflicts)
    uint4* code_s = sm.code + warp * 256 + lane;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int f = 0; f < 2; ++f) cp_async_16(code_s + (2 * r + f) * 32, cin + r * 64 + f * 4);
    const float scale_l = p.scales[unit_in + tid];

    const long ring_len = ring_channels(H, a.Hk) * (K - 1);
    const float* ring_in = a.ring_out + (long)from * ring_len;
    const int chq = hq * kHeadDim + tid, chk = (int)plane_offset(H, a.Hk, 1) + chq;
    const int chv = (int)plane_offset(H, a.Hk, 2) + h * kHeadDim + tid;
    Conv<KT> cq, ck, cv;
    cq.weights(a.conv_w, chq, K);
    ck.weights(a.conv_w, chk, K);
    cv.weights(a.conv_w, chv, K);
    cq.load(ring_in, chq, K);
    ck.load(ring_in, chk, K);
    cv.load(ring_in, chv, K);
    const float alog = a.a_log[gh];
    const float dt = GATE_MODE == 0 ? a.dt_bias[(long)gh * kHeadDim + tid] : a.dt_bias[gh];
    const float beta_raw = tid < T ? a.beta_raw[(row0 + tid) * Hg + gh] : 0.0f;
    // the first rows' slots that this thread looks over below
    const int other = min(tid, a.N - 1);
    const int im = p.slots ? p.slots[other] : other, om = p.slots_out ? p.slots_out[other] : im;
    // ---- conv + SiLU, the gate, the sums over channels
    const float rate = GATE_MODE == 0 ? expf(alog) : 0.0f;
    float q[TT], k[TT], v[TT];
    float kd[TT], cum[TT];                        // D_st k_s so far, A_t
    {
        float sum[S_::padded] = {};
        uint32_t top[TT] = {};
        float run = 1.0f;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            q[t] = k[t] = v[t] = kd[t] = cum[t] = 0.0f;
            if (t >= T) continue;
            q[t] = cq.step(raw_value(qr[t], bf16), K);
            k[t] = ck.step(raw_value(kr[t], bf16), K);
            v[t] = cv.step(raw_value(vr[t], bf16), K);
            const float dec = decay_f(GATE_MODE == 0 ? kda_gate_f(ga[t], dt, rate, a.gate_lb)
                                                     : gdn_gate_f(ga[t], dt, alog));
            run *= dec;
            cum[t] = run;
            // (no products fused into sums: a call's results do not depend on TT)
            sum[t] = __fmul_rn(q[t], q[t]);
            sum[S_::kk + t] = __fmul_rn(k[t], k[t]);
#pragma unroll
            for (int s = 0; s < t; ++s) {
                kd[s] *= dec;
                sum[S_::kk_at(s, t)] = __fmul_rn(kd[s], k[t]);
                sum[S_::qk_at(s, t)] = __fmul_rn(kd[s], q[t]);
            }
            kd[t] = k[t];
            sum[S_::qk_at(t, t)] = __fmul_rn(k[t], q[t]);
            top[t] = mag_pair(__fmul_rn(k[t], run), __fmul_rn(q[t], run));
        }
        const float s = warp_sums(sum, lane);
        if (lane % S_::lanes == 0) sm.part[warp][lane / S_::lanes] = s;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const uint32_t mq = __reduce_max_sync(0xffffffffu, top[t] >> 16);
            const uint32_t mk = __reduce_max_sync(0xffffffffu, top[t] & 0xffffu);
            if (lane == 0) {
                reinterpret_cast<uint32_t*>(&sm.top[t])[warp] = mq << 16;
                reinterpret_cast<uint32_t*>(&sm.top[TT + t])[warp] = mk << 16;
            }
        }
    }
    if (tid < T) sm.beta[tid] = sigmoid_f(beta_raw);
    // The slots (the rules of pool_row_warp, here looked over by the whole block).
    const bool live = slot_in >= 0 && slot_out >= 0;
    bool bad = slot_in >= p.pool_rows || slot_out >= p.pool_rows;
    if (p.slots || p.slots_out) {
        if (tid < a.N) bad |= pool_rows_clash(im, om, n, slot_out, tid, p.pool_rows);
        for (int m = tid + kThreads; m < a.N; m += kThreads) {
            const int mi = p.slots ? p.slots[m] : m;
            bad |= pool_rows_clash(mi, p.slots_out ? p.slots_out[m] : mi, n, slot_out, m, p.pool_rows);
        }
    }
    const bool clash = __syncthreads_or(live && bad);
    if (clash && tid == 0 && a.err) atomicOr(a.err, kDevErrSlot);
    if (!live || clash) {                         // uniform over the cluster: n decides alone
        cp_async_commit_wait();
        return;
    }

    const long unit_out = ((long)slot_out * H + h) * kHeadDim;
    uint4* cout = reinterpret_cast<uint4*>(p.codes) + (unit_out + warp * 32 + g) * 8 + c;
    // a q / k ring row that several units read is rolled by one of them, and only into another slot:
    // in place it is left to the roll kernel that follows
    const bool roll_qk = h == gh * vs && gh < Hkq && (Hkq == H || slot_in != slot_out);
    float* ring_out = a.ring_out + (long)slot_out * ring_len;

    if (T == 0) {       // nothing accepted: the slot passes through unchanged (in place: untouched)
        cp_async_commit_wait();
        if (slot_in != slot_out) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int f = 0; f < 2; ++f) __stcs(cout + r * 64 + f * 4, code_s[(2 * r + f) * 32]);
            p.scales[unit_out + tid] = scale_l;
            cv.store(ring_out, chv, K);
            if (roll_qk) {
                cq.store(ring_out, chq, K);
                ck.store(ring_out, chk, K);
            }
        }
        return;
    }
    cv.store(ring_out, chv, K);
    if (roll_qk) {
        cq.store(ring_out, chq, K);
        ck.store(ring_out, chk, K);
    }
    // lane l: sum l / lanes of the unit; then the l2 scales in its place for q.q and k.k
    const int own = lane / S_::lanes;
    const float total = (sm.part[0][own] + sm.part[1][own]) + (sm.part[2][own] + sm.part[3][own]);
    const float coef = own < 2 * TT ? l2_inv_f(total, a.l2_eps) : total;
    const auto coef_at = [&](int i) { return __shfl_sync(0xffffffffu, coef, i * S_::lanes); };
    // and each vector's factor, by the very products that form its elements below
    float up = 1.0f;
    if (own < 2 * TT && own % TT < T) {
        const uint4 m = sm.top[own];
        up = vec_factor(__fmul_rn(__uint_as_float(max(max(m.x, m.y), max(m.z, m.w))), coef));
    }
    const float coef_up = __fmul_rn(coef, up);
    const auto coef_up_at = [&](int i) { return __shfl_sync(0xffffffffu, coef_up, i * S_::lanes); };
    float iq[TT], ik[TT];
    {
        float run = 0.0f;
        __half* vec = reinterpret_cast<__half*>(sm.vec) + key_pos16(tid);
        float* row = sm.row + key_pos32(tid);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            iq[t] = coef_at(t);
            ik[t] = coef_at(S_::kk + t);
            // (tokens from T on are zeros)
            const float kc = coef_up_at(S_::kk + t), qc = coef_up_at(t);
            const float x = __fmul_rn(__fmul_rn(k[t], cum[t]), t < T ? kc : 0.0f);
            const float y = __fmul_rn(__fmul_rn(q[t], cum[t]), t < T ? qc : 0.0f);
            const __half xh = __float2half_rn(x), yh = __float2half_rn(y);
            __half* at = vec + 4 * t * (kVecBytes / 2);
            at[0] = xh;
            at[kVecBytes / 2] = __float2half_rn(x - __half2float(xh));
            at[2 * (kVecBytes / 2)] = yh;
            at[3 * (kVecBytes / 2)] = __float2half_rn(y - __half2float(yh));
            row[t * kHeadDim] = t < T ? kd[t] * ik[t] : 0.0f;
            if (t < T) run = cum[t];
        }
        if (GATE_MODE == 0) row[TT * kHeadDim] = run;
        else if (tid == 0) row[TT * kHeadDim] = run;
    }
    __syncthreads();

    // ---- the incoming state's products, 16 columns at a time
    cp_async_commit_wait();                       // (each lane reads what it copied)
    constexpr int kTiles = FewSmem<TT>::kTiles;
    const int cols = 4 * TT;                      // columns past them repeat the last one
    // this lane's columns of tile i are those of vector 4 i + c: one over its factor
    float down[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
        const int v = 2 * i + (c >> 1);
        const float u = __shfl_sync(0xffffffffu, up, (c & 1 ? v : S_::kk + v) * S_::lanes);
        down[i] = __uint_as_float((254u << 23) - __float_as_uint(u));
    }
#pragma unroll 1
    for (int mt = 0; mt < 2; ++mt) {
        float d[kTiles][4] = {};
        uint4 cur[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int f = 0; f < 2; ++f) cur[r][f] = code_s[(4 * mt + 2 * r + f) * 32];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const uint32_t u[2][4] = {{cur[0][f].x, cur[0][f].y, cur[0][f].z, cur[0][f].w},
                                      {cur[1][f].x, cur[1][f].y, cur[1][f].z, cur[1][f].w}};
#pragma unroll
            for (int m = 0; m < 4; m += 2) {
                uint4 b[kTiles];
#pragma unroll
                for (int i = 0; i < kTiles; ++i)
                    b[i] = sm.vec[min(8 * i + g, cols - 1) * (kVecBytes / 16) + (f * 2 + m / 2) * 4 + c];
                uint32_t a0, a1, a2, a3;
                codes_f16<FMT>(u[0][m], a0, a2);
                codes_f16<FMT>(u[1][m], a1, a3);
#pragma unroll
                for (int i = 0; i < kTiles; ++i) mma_16816(d[i], a0, a1, a2, a3, b[i].x, b[i].y);
                codes_f16<FMT>(u[0][m + 1], a0, a2);
                codes_f16<FMT>(u[1][m + 1], a1, a3);
#pragma unroll
                for (int i = 0; i < kTiles; ++i) mma_16816(d[i], a0, a1, a2, a3, b[i].z, b[i].w);
            }
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
            if (TT > 1 || c < 2) {
                float* o = sm.dot + (4 * i + c) * kDotRow + warp * 32 + mt * 16 + g;
                o[0] = __fmul_rn(d[i][0] + d[i][1], down[i]);
                o[8] = __fmul_rn(d[i][2] + d[i][3], down[i]);
            }
    }
    __syncwarp();

    // ---- the solve: thread = value column
    float w[TT], o[TT];
    {
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            float x = __fmul_rn(sm.dot[2 * t * kDotRow + tid], scale_l);
            float y = __fmul_rn(sm.dot[(2 * t + 1) * kDotRow + tid], scale_l);
#pragma unroll
            for (int s = 0; s < t; ++s) {
                x = fmaf(w[s], coef_at(S_::kk_at(s, t)) * (ik[s] * ik[t]), x);
                y = fmaf(w[s], coef_at(S_::qk_at(s, t)) * (ik[s] * iq[t]), y);
            }
            const float qk = coef_at(S_::qk_at(t, t)) * (ik[t] * iq[t]);
            w[t] = t < T ? __fmul_rn(sm.beta[t], v[t] - x) : 0.0f;
            o[t] = __fmul_rn(a.scale, fmaf(w[t], qk, y));
            const float ss = t < T ? warp_sum(__fmul_rn(o[t], o[t])) : 0.0f;
            if (lane == 0) sm.osum[warp][t] = ss;
        }
    }

    // ---- the new state, 16 columns at a time
#pragma unroll 1
    for (int mt = 0; mt < 2; ++mt) {
        float2 S[2][16];
        float wr[2][TT], sr[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int src = 16 * mt + 8 * r + g;
            sr[r] = __shfl_sync(0xffffffffu, scale_l, src);
#pragma unroll
            for (int t = 0; t < TT; ++t) wr[r][t] = __shfl_sync(0xffffffffu, w[t], src);
        }
        const float as = GATE_MODE == 0 ? 0.0f : sm.row[TT * kHeadDim];
        uint4 w4[2];
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            if (m % 4 == 0) {
#pragma unroll
                for (int r = 0; r < 2; ++r) w4[r] = code_s[(4 * mt + 2 * r + m / 4) * 32];
            }
            const float4* rows = reinterpret_cast<const float4*>(sm.row) + m * 4 + c;
            const float4 a4 = GATE_MODE == 0 ? rows[TT * (kHeadDim / 4)] : make_float4(as, as, as, as);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t word = m % 4 == 0 ? w4[r].x : m % 4 == 1 ? w4[r].y : m % 4 == 2 ? w4[r].z : w4[r].w;
                const float4 x = q8_decode4<FMT>(word, sr[r]);
                S[r][2 * m] = __fmul2_rn(make_float2(x.x, x.y), make_float2(a4.x, a4.y));
                S[r][2 * m + 1] = __fmul2_rn(make_float2(x.z, x.w), make_float2(a4.z, a4.w));
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const float4 k4 = rows[t * (kHeadDim / 4)];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 w2 = make_float2(wr[r][t], wr[r][t]);
                    S[r][2 * m] = __ffma2_rn(make_float2(k4.x, k4.y), w2, S[r][2 * m]);
                    S[r][2 * m + 1] = __ffma2_rn(make_float2(k4.z, k4.w), w2, S[r][2 * m + 1]);
                }
            }
        }
        // back to 8 bits: of a row pair's four lanes 0 and 2 form the scales, 1 and 3 the multipliers
        float mx[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float x = mag_max(S[r][0].x, S[r][0].y);
#pragma unroll
            for (int i = 1; i < 16; ++i) x = mag_max3(x, S[r][i].x, S[r][i].y);
            mx[r] = x;
        }
        const bool up = c & 2;
        float top = mag_max(up ? mx[1] : mx[0], __shfl_xor_sync(0xffffffffu, up ? mx[0] : mx[1], 2));
        top = mag_max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        const float f = q8_row_part<FMT>(mag_bits(top), c & 1);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float mul = __shfl_sync(0xffffffffu, f, 4 * g + 2 * r + 1);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                uint32_t u[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float2 lo = S[r][2 * (4 * y + m)], hi = S[r][2 * (4 * y + m) + 1];
                    u[m] = q8_encode4_once<FMT>(make_float4(lo.x, lo.y, hi.x, hi.y), mul);
                }
                __stcs(cout + mt * 128 + r * 64 + y * 4, make_uint4(u[0], u[1], u[2], u[3]));
            }
        }
        if (!(c & 1)) p.scales[unit_out + warp * 32 + mt * 16 + 4 * c + g] = f;
    }
    __syncthreads();

    // ---- epilogue: gated RMSNorm, thread = channel
    float ss[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t)
        ss[t] = (sm.osum[0][t] + sm.osum[1][t]) + (sm.osum[2][t] + sm.osum[3][t]);
    if constexpr (WIDE) {
        if (tid == 0) {
#pragma unroll
            for (int t = 0; t < TT; ++t) sm.nss[t] = ss[t];
        }
        cluster_sync_all();
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        if (t >= T) continue;
        float inv;
        if constexpr (WIDE) {
            float tot = 0.0f;
            for (int b = 0; b < a.vsub; ++b) tot = tot + ld_cluster_f32(&sm.nss[t], (uint32_t)b);
            inv = rms_inv_w(tot, a.rms_eps, a.vsub * kHeadDim);
        } else {
            inv = rms_inv_f(ss[t], a.rms_eps);
        }
        a.y[(row0 + t) * wv + h * kHeadDim + tid] =
            a.norm_silu ? gated_norm_f<true>(o[t], inv, nw, sm.z[t][tid]) : gated_norm_f(o[t], inv, nw, sm.z[t][tid]);
    }
    if constexpr (WIDE) cluster_sync_all();       // the other units have read this unit's sums
}

template <int FMT, int GM, int KT, bool WIDE, int TT>
cudaError_t launch_one(const DecodeQ8Args& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.d.H, (unsigned)a.d.N);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.d.vsub;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = WIDE ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kda_decode_q8_few_kernel<FMT, GM, KT, WIDE, TT>, a);
}

template <int FMT, int GM, int TT>
cudaError_t launch_t(const DecodeQ8Args& a, cudaStream_t s) {
    if (a.d.vsub > 1)
        return a.d.K == 4 ? launch_one<FMT, GM, 4, true, TT>(a, s) : launch_one<FMT, GM, kMaxConvK, true, TT>(a, s);
    return a.d.K == 4 ? launch_one<FMT, GM, 4, false, TT>(a, s) : launch_one<FMT, GM, kMaxConvK, false, TT>(a, s);
}

template <int FMT, int GM>
cudaError_t launch_gm(const DecodeQ8Args& a, cudaStream_t s) {
    if (a.d.T == 1) return launch_t<FMT, GM, 1>(a, s);
    if (a.d.T == 2) return launch_t<FMT, GM, 2>(a, s);
    return a.d.T == 3 ? launch_t<FMT, GM, 3>(a, s) : launch_t<FMT, GM, 4>(a, s);
}

}  // namespace

cudaError_t launch_decode_q8_few(const DecodeQ8Args& a, cudaStream_t s) {
    if (a.fmt == kQ8E4m3)
        return a.d.gate_mode == 0 ? launch_gm<kQ8E4m3, 0>(a, s) : launch_gm<kQ8E4m3, 1>(a, s);
    return a.d.gate_mode == 0 ? launch_gm<kQ8Int8, 0>(a, s) : launch_gm<kQ8Int8, 1>(a, s);
}

}  // namespace kda
