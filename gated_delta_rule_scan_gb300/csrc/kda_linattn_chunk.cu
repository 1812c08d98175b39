// kda_linattn_chunk.cu -- linear attention with one log-decay g a head, the chunked form for bf16
// prompts, on the tcgen05 tensor cores.
//
// Mathematics.  Over a chunk of C = 64 tokens with incoming state S (stored [value j][key i]):
//     O^T = scale * ( V^T P^T + e^{g (t+1)} S Q^T ),   P[t][s] = e^{g (t-s)} q_t . k_s  for s <= t,
//     S  <- e^{g C} S + V^T Kd,                        Kd[s]   = e^{g (C-1-s)} k_s.
// Every decay is a power e^{g n} with 0 <= n <= C, at most 1, whatever g is.  q, k and v enter as the
// bf16 values they are; what is f32 (P, Kd and the state) enters as three bf16 parts, 24 bits in all,
// so that the result is an f32 one: P = 3 products, S = 3, Kd = 3 beside q k's one.  (Two parts would
// leave errors of 2^-17 to save 3 of the 10 product passes.)  The state itself stays in f32 registers.
//
// One CTA per (sequence, 128-wide value unit), chunk after chunk, the values on the MMA's M = 128 TMEM
// lanes.  That way the state parts are an A operand in tensor memory, written by the threads that hold
// the state rows, v is read as it lies (MN-major), and k's and q's tiles are B operands as TMA brings
// them.  The 512 TMEM columns are full: S parts 3 x 64, V^T Kd 128, S Q^T 64, V^T P^T 64, q k 64.
// 64 tokens, not 128: the parts of P and Kd then fit beside two stages of q, k, v.
// Warps have roles: 8 hold the state (64 f32 a thread) and write o, 8 turn k into Kd and q k into P,
// one issues the MMAs, one the TMA loads; they meet on mbarriers only, so the loads, the MMAs and both
// groups' register work overlap across chunks.
#include "kda_tc.cuh"

namespace kda {

namespace {

constexpr int kC = 64;                           // tokens of a chunk
constexpr int kStages = 2;
constexpr int kHalf = kC * 128;                  // bytes of 64 tokens x 64 columns, 128-byte swizzle
constexpr int kTileBytes = 2 * kHalf;            // 64 tokens x 128 columns
constexpr int kStageBytes = 3 * kTileBytes;      // q, k, v
constexpr int kKdAt = kStages * kStageBytes;     // Kd: 3 parts
constexpr int kPAt = kKdAt + 3 * kTileBytes;     // P: 3 parts of [64 t][64 s]
constexpr int kTailAt = kPAt + 3 * kHalf;
constexpr int kStateWarps = 8, kConvWarps = 8;
constexpr int kMmaWarp = kStateWarps + kConvWarps, kTmaWarp = kMmaWarp + 1;
constexpr int kThr = 32 * (kMmaWarp + 4);        // whole warpgroups: registers move between them
constexpr int kStateRegs = 136, kConvRegs = 80, kOtherRegs = 48;   // of 96 each at launch
static_assert(32 * (kStateWarps * kStateRegs + kConvWarps * kConvRegs + 4 * kOtherRegs) <= kThr * 96, "");

struct Tail {
    float pw[kC + 2];                            // e^{g n}, n = 0 .. 64
    uint64_t full[kStages], empty[kStages];
    uint64_t sc_full, sc_free, kd_full, u_full, u_free, sp_full, oi_full, p_full, oa_full, o_free;
    uint32_t tmem;
    int failed;
};
constexpr int kSmemBytes = 1024 + kTailAt + (int)sizeof(Tail);

// TMEM columns
constexpr uint32_t kTSp = 0, kTU = 192, kTOi = 320, kTOa = 384, kTSc = 448;

// Two f32 as three bf16x2 words whose sum they are to 24 bits.
__device__ __forceinline__ void split3(float2 x, uint32_t& a, uint32_t& b, uint32_t& c) {
    const float2 neg = make_float2(-1.0f, -1.0f);
    const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
    a = *reinterpret_cast<const uint32_t*>(&h);
    x = __ffma2_rn(make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u)), neg, x);
    const __nv_bfloat162 m = __floats2bfloat162_rn(x.x, x.y);
    b = *reinterpret_cast<const uint32_t*>(&m);
    x = __ffma2_rn(make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u)), neg, x);
    const __nv_bfloat162 l = __floats2bfloat162_rn(x.x, x.y);
    c = *reinterpret_cast<const uint32_t*>(&l);
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A warp's arrival: its lanes' TMEM and shared memory accesses before it are done.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Shares of the 32 pieces of 32 x 16 bytes of a k tile among the 8 converting warps.  Warps 0, 1 and 5
// also turn a 32 x 32 block of q k into P (about 5 pieces' worth); warps w and w + 4 share a scheduler.
__device__ constexpr int kKdFirst[kConvWarps + 1] = {0, 2, 3, 8, 14, 19, 20, 26, 32};

__global__ void __launch_bounds__(kThr, 1)
kda_linattn_chunk_kernel(const LinArgs a, const __grid_constant__ CUtensorMap tq,
                         const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* const base = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Tail& sm = *reinterpret_cast<Tail*>(base + kTailAt);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x, n = blockIdx.y;
    const int units = a.H * a.m, hv = unit / a.m, hk = hv % a.Hk;
    long begin;
    int len;
    if (a.seq.cu_seqlens != nullptr) {
        begin = a.seq.cu_seqlens[n];
        len = a.seq.cu_seqlens[n + 1] - (int)begin;
    } else {
        begin = (long)n * a.seq.T_uniform;
        len = a.seq.T_uniform;
    }
    const int chunks = (len + kC - 1) / kC;
    const float g = a.log_decay[hv];

    if (warp == kMmaWarp) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    if (warp == kTmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < kStages; ++i) {
                mbar_init(&sm.full[i], 1);
                mbar_init(&sm.empty[i], 1);
            }
            mbar_init(&sm.sc_full, 1);
            mbar_init(&sm.sc_free, 3);
            mbar_init(&sm.kd_full, kConvWarps);
            mbar_init(&sm.u_full, 1);
            mbar_init(&sm.u_free, kStateWarps);
            mbar_init(&sm.sp_full, kStateWarps);
            mbar_init(&sm.oi_full, 1);
            mbar_init(&sm.p_full, 3);
            mbar_init(&sm.oa_full, 1);
            mbar_init(&sm.o_free, kStateWarps);
            sm.failed = 0;
            fence_mbar_init();
            prefetch_tensormap(&tq);
            prefetch_tensormap(&tk);
            prefetch_tensormap(&tv);
        }
        // e^{g n}; n = 0 apart, so that a log-decay of -infinity is a plain reset
        for (int i = lane; i <= kC; i += 32) sm.pw[i] = i == 0 ? 1.0f : expf(g * (float)i);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    bool ok = true;

    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kTmaWarp) {
        // ---- loads ---------------------------------------------------------------------------
        for (int c = 0; c < chunks && ok; ++c) {
            const int st = c % kStages;
            if (c >= kStages)
                ok = mbar_wait_bounded(&sm.empty[st], (uint32_t)((c / kStages - 1) & 1), a.err);
            if (ok && elect_one()) {
                unsigned char* s = base + st * kStageBytes;
                const int row = (int)(begin + (long)c * kC);
                mbar_arrive_expect_tx(&sm.full[st], kStageBytes);
                for (int h = 0; h < 2; ++h) {
                    tma_load_2d(s + kTileBytes + h * kHalf, &tk, hk * kHeadDim + 64 * h, row, &sm.full[st]);
                    tma_load_2d(s + h * kHalf, &tq, hk * kHeadDim + 64 * h, row, &sm.full[st]);
                    tma_load_2d(s + 2 * kTileBytes + h * kHalf, &tv, unit * kHeadDim + 64 * h, row, &sm.full[st]);
                }
            }
            __syncwarp();
        }
        if (!ok)                                 // no load may land after the CTA has left
            for (int i = 0; i < kStages; ++i)
                for (uint32_t p = 0; p < 2; ++p) mbar_wait_bounded(&sm.full[i], p, nullptr);
    } else if (warp == kMmaWarp) {
        // ---- MMAs ----------------------------------------------------------------------------
        constexpr uint32_t id_sc = tc_idesc_bf16(128, kC);                        // q k
        constexpr uint32_t id_u = tc_idesc_bf16(128, 128) | kTcAMajorMN | kTcBMajorMN;   // V^T Kd
        constexpr uint32_t id_oi = tc_idesc_bf16(128, kC);                        // S Q^T
        constexpr uint32_t id_oa = tc_idesc_bf16(128, kC) | kTcAMajorMN;          // V^T P^T
        const uint32_t b0 = smem_u32(base);
        // q_t . k_s on lanes t < 64.  (M = 128 reads 64 rows more, whatever lies there: lanes 64 .. 127
        // are never read.)
        auto qk = [&](int c) {
            const uint32_t s = b0 + (c % kStages) * kStageBytes;
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t off = (ks >> 2) * kHalf + (ks & 3) * 32;
                    tc_mma_ss(tmem + kTSc, tc_smem_desc_sw128(s + off),
                              tc_smem_desc_sw128(s + kTileBytes + off), id_sc, ks > 0);
                }
                tc_commit(&sm.sc_full);
            }
            __syncwarp();
        };
        if (chunks > 0) {
            ok = mbar_wait_bounded(&sm.full[0], 0, a.err);
            tc_fence_after();
            if (ok) qk(0);
        }
        for (int c = 0; c < chunks && ok; ++c) {
            const int st = c % kStages;
            const uint32_t s = b0 + st * kStageBytes, v = s + 2 * kTileBytes;
            const uint32_t par = (uint32_t)(c & 1);
            // V^T Kd
            ok = mbar_wait_bounded(&sm.kd_full, par, a.err) &&
                 (c == 0 || mbar_wait_bounded(&sm.u_free, par ^ 1u, a.err));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int p = 2; p >= 0; --p)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        tc_mma_ss(tmem + kTU, tc_smem_desc_sw128_mn(v + 2048 * ks, kHalf),
                                  tc_smem_desc_sw128_mn(b0 + kKdAt + p * kTileBytes + 2048 * ks, kHalf),
                                  id_u, p < 2 || ks > 0);
                tc_commit(&sm.u_full);
            }
            __syncwarp();
            // the next chunk's q k
            if (c + 1 < chunks) {
                ok = mbar_wait_bounded(&sm.full[(c + 1) % kStages], (uint32_t)(((c + 1) / kStages) & 1), a.err) &&
                     mbar_wait_bounded(&sm.sc_free, par, a.err);
                if (!ok) break;
                tc_fence_after();
                qk(c + 1);
            }
            // S Q^T
            ok = mbar_wait_bounded(&sm.sp_full, par, a.err) &&
                 (c == 0 || mbar_wait_bounded(&sm.o_free, par ^ 1u, a.err));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int p = 2; p >= 0; --p)
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        tc_mma_ts(tmem + kTOi, tmem + kTSp + 64 * p + 8 * ks,
                                  tc_smem_desc_sw128(s + (ks >> 2) * kHalf + (ks & 3) * 32), id_oi,
                                  p < 2 || ks > 0);
                tc_commit(&sm.oi_full);
            }
            __syncwarp();
            // V^T P^T
            ok = mbar_wait_bounded(&sm.p_full, par, a.err);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int p = 2; p >= 0; --p)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        tc_mma_ss(tmem + kTOa, tc_smem_desc_sw128_mn(v + 2048 * ks, kHalf),
                                  tc_smem_desc_sw128(b0 + kPAt + p * kHalf + 32 * ks), id_oa,
                                  p < 2 || ks > 0);
                tc_commit(&sm.oa_full);
                tc_commit(&sm.empty[st]);
            }
            __syncwarp();
        }
        }
    } else if (warp >= kStateWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
        // ---- k into Kd, q k into P -----------------------------------------------------------
        const int cw = warp - kStateWarps;
        const bool has_p = cw == 0 || cw == 1 || cw == 5;
        const int prow = 32 * (cw & 1) + lane;   // token t of P, = TMEM lane
        const int pcol = cw == 5 ? 32 : 0;       // its tokens s
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        if (cw == 4) {                           // t < 32 <= s: P is 0 there, once and for all
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
                for (int q = 4; q < 8; ++q)
                    *reinterpret_cast<uint4*>(base + kPAt + p * kHalf + lane * 128 + ((q ^ (lane & 7)) * 16)) =
                        make_uint4(0u, 0u, 0u, 0u);
        }
        for (int c = 0; c < chunks && ok; ++c) {
            const int st = c % kStages;
            const uint32_t par = (uint32_t)(c & 1);
            const int nt = min(kC, len - c * kC);
            unsigned char* s = base + st * kStageBytes;
            ok = mbar_wait_bounded(&sm.full[st], (uint32_t)((c / kStages) & 1), a.err) &&
                 (c == 0 || mbar_wait_bounded(&sm.u_full, par ^ 1u, a.err));
            if (!ok) break;
            for (int u = kKdFirst[cw]; u < kKdFirst[cw + 1]; ++u) {
                const int at = (u * 32 + lane) * 16;
                const int t = (at >> 7) & (kC - 1);          // 128-byte rows are tokens
                const uint4 w = *reinterpret_cast<const uint4*>(s + kTileBytes + at);
                const float d = t < nt ? sm.pw[nt - 1 - t] : 0.0f;
                const float2 d2 = make_float2(d, d);
                const uint32_t in[4] = {w.x, w.y, w.z, w.w};
                uint32_t o[3][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 x = make_float2(__uint_as_float(in[j] << 16), __uint_as_float(in[j] & 0xffff0000u));
                    x = t < nt ? __fmul2_rn(x, d2) : make_float2(0.0f, 0.0f);
                    split3(x, o[0][j], o[1][j], o[2][j]);
                }
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    *reinterpret_cast<uint4*>(base + kKdAt + p * kTileBytes + at) =
                        make_uint4(o[p][0], o[p][1], o[p][2], o[p][3]);
                // rows past the sequence's end are another's: 0 times a NaN there is not 0
                if (t >= nt) *reinterpret_cast<uint4*>(s + 2 * kTileBytes + at) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            warp_arrive(&sm.kd_full);
            if (!has_p) continue;
            ok = mbar_wait_bounded(&sm.sc_full, par, a.err);
            if (!ok) break;
            tc_fence_after();
            float x[32];
            tmem_ld16(tl + kTSc + pcol, *reinterpret_cast<float(*)[16]>(x));
            tmem_ld16(tl + kTSc + pcol + 16, *reinterpret_cast<float(*)[16]>(x + 16));
            tmem_ld_wait();
            tc_fence_before();
            warp_arrive(&sm.sc_free);
            if (c > 0) ok = mbar_wait_bounded(&sm.oa_full, par ^ 1u, a.err);
            if (!ok) break;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t o[3][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int s0 = pcol + 8 * q + 2 * j, gap = prow - s0;
                    float2 y;
                    y.x = gap >= 0 ? x[8 * q + 2 * j] * sm.pw[max(gap, 0)] : 0.0f;
                    y.y = gap >= 1 ? x[8 * q + 2 * j + 1] * sm.pw[max(gap - 1, 0)] : 0.0f;
                    split3(y, o[0][j], o[1][j], o[2][j]);
                }
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    *reinterpret_cast<uint4*>(base + kPAt + p * kHalf + prow * 128 +
                                              (((pcol / 8 + q) ^ (prow & 7)) * 16)) =
                        make_uint4(o[p][0], o[p][1], o[p][2], o[p][3]);
            }
            fence_proxy_async_smem();
            warp_arrive(&sm.p_full);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStateRegs));
        // ---- the state and o -----------------------------------------------------------------
        const int j = 32 * (warp & 3) + lane, hf = warp >> 2;     // value row, half of its keys / tokens
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        float S[64];                             // keys 64 hf ..
        if (a.state_in != nullptr) {
            const float4* src = reinterpret_cast<const float4*>(
                a.state_in + (((long)n * units + unit) * kHeadDim + j) * kHeadDim + 64 * hf);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float4 x = __ldg(src + i);
                S[4 * i] = x.x; S[4 * i + 1] = x.y; S[4 * i + 2] = x.z; S[4 * i + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) S[i] = 0.0f;
        }
        auto put_state = [&]() {
#pragma unroll
            for (int b = 0; b < 4; ++b) {        // 16 keys: 8 columns of each part
                uint32_t w[3][8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    split3(make_float2(S[16 * b + 2 * i], S[16 * b + 2 * i + 1]), w[0][i], w[1][i], w[2][i]);
#pragma unroll
                for (int p = 0; p < 3; ++p) tmem_st8(tl + kTSp + 64 * p + 32 * hf + 8 * b, w[p]);
            }
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&sm.sp_full);
        };
        if (chunks > 0) put_state();
        float* o = a.o + begin * units * kHeadDim + (long)unit * kHeadDim + j;
        for (int c = 0; c < chunks && ok; ++c) {
            const uint32_t par = (uint32_t)(c & 1);
            const int nt = min(kC, len - c * kC);
            // S <- e^{g nt} S + U; above a half as S + (e^{g nt} - 1) S, which keeps a decay next to 1
            const float lam = sm.pw[nt];
            const bool near1 = lam > 0.5f;
            const float fa = near1 ? 1.0f : lam, fd = near1 ? expm1f(g * (float)nt) : 0.0f;
            ok = mbar_wait_bounded(&sm.u_full, par, a.err);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                float u[16];
                tmem_ld16(tl + kTU + 64 * hf + 16 * b, u);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float x = S[16 * b + i];
                    S[16 * b + i] = fmaf(fa, x, fmaf(fd, x, u[i]));
                }
            }
            tc_fence_before();
            warp_arrive(&sm.u_free);
            ok = mbar_wait_bounded(&sm.oi_full, par, a.err);
            if (!ok) break;
            tc_fence_after();
            if (c + 1 < chunks) put_state();
            ok = mbar_wait_bounded(&sm.oa_full, par, a.err);
            if (!ok) break;
            tc_fence_after();
            float* oc = o + ((long)c * kC + 32 * hf) * units * kHeadDim;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float x[16], y[16];
                tmem_ld16(tl + kTOi + 32 * hf + 16 * b, x);
                tmem_ld16(tl + kTOa + 32 * hf + 16 * b, y);
                tmem_ld_wait();
                if (b == 1) {
                    tc_fence_before();
                    warp_arrive(&sm.o_free);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int t = 16 * b + i;
                    if (32 * hf + t < nt)
                        __stcs(oc + (long)t * units * kHeadDim,
                               a.scale * fmaf(sm.pw[32 * hf + t + 1], x[i], y[i]));
                }
            }
        }
        if (ok) {
            float4* dst = reinterpret_cast<float4*>(
                a.state_out + (((long)n * units + unit) * kHeadDim + j) * kHeadDim + 64 * hf);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                dst[i] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
        }
    }
    // every role has seen its last barrier; after a wait that gave up, MMAs may still be running
    if (!ok) sm.failed = 1;
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        if (sm.failed) {
            if (elect_one()) tc_commit(&sm.sc_full);
            __syncwarp();
            for (uint32_t p = 0; p < 2; ++p) mbar_wait_bounded(&sm.sc_full, p, nullptr);
        }
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

cudaError_t launch_linattn_chunk(const LinArgs& a, cudaStream_t s) {
    const long qk = (long)a.Hk * kHeadDim, vw = (long)a.H * a.m * kHeadDim;
    CUtensorMap tq, tk, tv;
    if (!make_tensor_map_2d_bf16_sw128(&tq, a.q, a.seq.total_rows, qk, kC, a.q_stride) ||
        !make_tensor_map_2d_bf16_sw128(&tk, a.k, a.seq.total_rows, qk, kC, a.k_stride) ||
        !make_tensor_map_2d_bf16_sw128(&tv, a.v, a.seq.total_rows, vw, kC, a.v_stride))
        return cudaErrorInvalidValue;
    static PerDevice<int> done;
    const cudaError_t e = set_smem(kda_linattn_chunk_kernel, kSmemBytes, done);
    if (e != cudaSuccess) return e;
    KernelTimer kt(kKLinChunk, s);
    kda_linattn_chunk_kernel<<<dim3((unsigned)(a.H * a.m), (unsigned)a.seq.N), kThr, kSmemBytes, s>>>(a, tq, tk, tv);
    return cudaGetLastError();
}

}  // namespace kda
