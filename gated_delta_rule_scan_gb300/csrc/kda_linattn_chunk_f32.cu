// kda_linattn_chunk_f32.cu -- linear attention with one log-decay g a head, the chunked form for f32 prompts, on the
// tcgen05 tensor cores.
//
// Mathematics.  Over a chunk of C = 64 tokens with incoming state S (stored [value j][key i]), relative to the middle
// of the chunk: with V'[s] = e^{g (31-s)} v_s and the state kept as S' = e^{32 g} S,
//     o_t = scale e^{g (t-31)} ( sum_{s <= t} V'[s] (q_t . k_s) + S' q_t ),
//     S' <- e^{g C} (S' + sum_s V'[s] k_s^T).
// All of a chunk's decays are in V' and in factors of whole rows, so that q and k enter every product as they are.
// Heads that decay faster (g < -1, where e^{32 |g|} might overflow) take v itself with e^{g (t-s)} in the scores, then
// e^{g (C-1-s)} v_s for the state, and o in two sums.
// f32 factors enter as three bf16 parts, 24 bits, whatever their size, and a product as its six terms down to 2^-16
// (hi lo, mid mid, lo hi, then hi mid, mid hi, hi hi): what is left out is 2^-24 of a product, less than what the tensor
// cores' sums truncate.  They truncate at each step, to 24 bits of what has come together, so that o gets all small terms
// of S' q first and its largest last.  q and k are split by a launch before, V', the scores and the state in registers here.
// The state itself stays in f32 registers.
//
// A NaN or an infinity at one token does not reach the tokens before it: scores that are not seen are 0 by selection,
// and in v it is replaced by 0 and its value column made NaN from that token on.  k rows behind the sequence's end,
// which are another's, are cleared.
//
// One CTA per (sequence, 128-wide value unit), chunk after chunk, the values on the MMA's 128 TMEM lanes; a thread that
// converts v has one value, 32 of whose tokens it reads from global memory a chunk ahead (rows of 128 bytes a warp) and
// writes to its own TMEM lane.  k is K-major for the scores and MN-major for the state's update, in the same tile.
// Shared memory holds two stages of q's and k's parts and the scores' parts, 216 KB; of the 512 TMEM columns the state
// takes 192, the update 128 (in turn with the scores), V' 96, o 64.
// The warps' roles are those of the bf16 form: 16 hold the state and write o, 8 convert v and the scores, three issue
// MMAs, one the loads.  Long sequences of few heads are cut into segments as there.
//
// Measured: 16384 tokens x 32 heads 579 us (the split 209, at a copy's rate, pieces' states 107, their sums 10, chunks
// 273), off by 2.9e-7, plain f32 sums by 2.6e-7; 16 x 4096 tokens x 64 heads 3.52 ms, 5.8 TB/s of what the chunks read and write.  With every SM
// busy a chunk takes 8150 cycles and waits for v from memory; what its MMAs take, one after the other, is 6800: the
// scores 2500, the update 1500, S' q 1900, V' P 900.  Two bf16 parts of everything took as long, off by 6.6e-6.
// v converted by four warps a chunk in turn, 16 tokens at a time, took 808 us; the scores with M = 128, half of its
// rows unused, 604.
#include "kda_linattn_chunk.cuh"

#include <algorithm>

namespace kda {

using namespace linattn;

namespace {

constexpr int kStages = 2;
constexpr int kHalfBytes = kParts * kHalf;                       // 64 columns of q or k: their parts one after the other
constexpr int kPlaneBytes = 2 * kHalfBytes;                      // a stage of q or k
constexpr int kKAt = 0, kQAt = kStages * kPlaneBytes;
constexpr int kPAt = kQAt + kStages * kPlaneBytes;               // the scores' parts, [64 t][64 s] each
constexpr int kStAt = kQAt + kPlaneBytes;                        // states on their way: q's second stage, scores
constexpr int kTailAt = kPAt + kParts * kHalf;
static_assert(kStAt + 4 * kStTile <= kTailAt, "");
// TMEM columns
constexpr uint32_t kTSp = 0, kTU = 64 * kParts, kTSc = kTU, kTO = kTU + 128, kTV = kTO + 64;
static_assert(kTV + 32 * kParts <= 512, "");
// the parts of A and B in term x of a product, the smallest first
constexpr int kTerms = 6;
__device__ __forceinline__ int a_part(int x) { return 0x001012 >> (4 * x) & 3; }
__device__ __forceinline__ int b_part(int x) { return 0x010210 >> (4 * x) & 3; }

struct __align__(16) Tail {
    float pw[kC + 4];                            // e^{g n}, n = 0 .. 64
    float down[kC];                              // v's factors: e^{g (31-s)}
    float up[kC];                                // the outputs': scale * e^{g (t-31)}, or scale * e^{g (t+1)}
    uint64_t k_full[2], k_free[2], q_full[2], q_free[2];
    // (two each, by the chunk's parity: some wait for a chunk's only after the next one's may have come)
    uint64_t v_full[2], v_free[2], vu_full[2], sc_full[2], oa_full[2];
    uint64_t sc_free, u_full, u_free, sp_full, p_full, os_full, oa_free, o_full, o_free;
    uint64_t st_full, st_free, st_out[4];        // the state on its way in and out
    uint64_t drain[3];
    uint32_t tmem;
    int bad[kHeadDim];                           // by value: the first token whose v is no number
};
constexpr int kSmemBytes = 1024 + kTailAt + (int)sizeof(Tail);
static_assert(kSmemBytes <= kMaxBlockSmem, "");

constexpr int kStateRegs = 72, kConvRegs = 96;   // (32 tokens of v are held ahead)
static_assert(regs_fit(kStateRegs, kConvRegs), "");
constexpr int kScoreWarps = 7;                   // converting warps with a share of the scores

// 16 lanes x 16 columns of TMEM: lane l gets rows l / 4 and l / 4 + 8, columns 2 (l % 4) and the next, then 8 columns on.
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

struct Maps {
    CUtensorMap q[kParts], k[kParts], in, parts, out;            // out: the parts in the STATE launch, else state_out
};

// e^{g n}, with what g n's rounding leaves: three such factors of a token together are 1 or so, each up to e^{64 |g|}
// away from it, where the rounding alone is 2^-19.
__device__ __forceinline__ float power(float g, int n) {
    const float x = g * (float)n, e = expf(x);
    return n == 0 || e == 0.0f ? (n == 0 ? 1.0f : 0.0f) : fmaf(e, fmaf(g, (float)n, -x), e);
}

template <bool STATE>
__global__ void __launch_bounds__(kThr, 1)
kda_linattn_chunk_f32_kernel(const LinArgs a, const Cut cut, const __grid_constant__ Maps maps) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* const base = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Tail& sm = *reinterpret_cast<Tail*>(base + kTailAt);
    // (shuffled from lane 0, what is the same in a warp is known to be: it goes to uniform registers)
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int unit = blockIdx.x, seg = blockIdx.z;
    const int units = a.H * a.m, hv = unit / a.m, hk = hv % a.Hk;
    const Part at = locate<STATE>(a.seq, cut, lane);
    if (at.len < 0) return;                      // (the whole CTA)
    const int n = at.n, len = at.len;
    const long begin = at.begin;
    const int chunks = (len + kC - 1) / kC;
    const float g = a.log_decay[hv];
    const bool strong = g < -1.0f;
    const int mid = strong ? 0 : kMid;           // the state is kept as e^{mid g} S
    const bool starts = !STATE && (seg > 0 || a.state_in != nullptr);

    if (warp == kUWarp) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    const auto load = [&](int at_byte, const CUtensorMap* map, uint64_t* bar, int c) {   // by one thread
        unsigned char* s = base + at_byte + c % kStages * kPlaneBytes;
        mbar_arrive_expect_tx(bar + c % kStages, kPlaneBytes);
        for (int p = 0; p < kParts; ++p)
            for (int h = 0; h < 2; ++h)
                tma_load_2d(s + h * kHalfBytes + p * kHalf, map + p, hk * kHeadDim + 64 * h,
                            (int)(begin + (long)c * kC), bar + c % kStages);
    };
    const auto load_k = [&](int c) { load(kKAt, maps.k, sm.k_full, c); };
    const auto load_q = [&](int c) { load(kQAt, maps.q, sm.q_full, c); };
    // into L2: what chunk c has no stage for yet
    const auto prefetch = [&](int c) {
        for (int p = 0; p < kParts; ++p)
            for (int h = 0; h < 2; ++h) {
                tma_prefetch_2d(&maps.k[p], hk * kHeadDim + 64 * h, (int)(begin + (long)c * kC));
                if (!STATE) tma_prefetch_2d(&maps.q[p], hk * kHeadDim + 64 * h, (int)(begin + (long)c * kC));
            }
    };
    // the next launch may be set up meanwhile; it waits for the end of this one before it reads what this one writes
    if (STATE) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == kTmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sm.k_full[i], 1);
                mbar_init(&sm.k_free[i], STATE ? 1 : 2);
                mbar_init(&sm.q_full[i], 1);
                mbar_init(&sm.q_free[i], 2);
                mbar_init(&sm.v_full[i], kConvWarps);
                mbar_init(&sm.v_free[i], STATE ? 1 : 2);
                mbar_init(&sm.vu_full[i], kConvWarps);
                mbar_init(&sm.sc_full[i], 1);
                mbar_init(&sm.oa_full[i], 1);
            }
            mbar_init(&sm.sc_free, kScoreWarps);
            mbar_init(&sm.u_full, 1);
            mbar_init(&sm.u_free, kStateWarps);
            mbar_init(&sm.sp_full, kStateWarps);
            mbar_init(&sm.p_full, kScoreWarps);
            mbar_init(&sm.os_full, 1);
            mbar_init(&sm.oa_free, kStateWarps);
            mbar_init(&sm.o_full, 1);
            mbar_init(&sm.o_free, kStateWarps);
            mbar_init(&sm.st_full, 1);
            mbar_init(&sm.st_free, kStateWarps);
            for (int i = 0; i < 4; ++i) mbar_init(&sm.st_out[i], 4);
            for (int i = 0; i < 3; ++i) mbar_init(&sm.drain[i], 1);
            fence_mbar_init();
            for (int p = 0; p < kParts; ++p) {
                prefetch_tensormap(&maps.k[p]);
                if (!STATE) prefetch_tensormap(&maps.q[p]);
            }
        }
        __syncwarp();
        // (n = 0 apart, so that a log-decay of -infinity is a plain reset)
        for (int i = lane; i <= kC; i += 32) sm.pw[i] = power(g, i);
        for (int i = lane; i < kC; i += 32) {
            sm.down[i] = strong ? 1.0f : power(g, kMid - 1 - i);
            sm.up[i] = a.scale * power(g, strong ? i + 1 : i - kMid + 1);
        }
        if (lane == 0) {
            // the launches before have written these: q and k split, the state that a segment starts from
            asm volatile("griddepcontrol.wait;" ::: "memory");
            for (int c = 0; c < kStages && c < chunks; ++c) {
                load_k(c);
                if (!STATE && (c == 0 || !starts)) load_q(c);
            }
            if (starts) {
                const long st = seg > 0 ? piece_state(cut, n, seg * cut.subs - 1, units) : (long)n * units;
                mbar_arrive_expect_tx(&sm.st_full, 4 * kStTile);
                for (int i = 0; i < 4; ++i)
                    tma_load_2d(base + kStAt + i * kStTile, seg > 0 ? &maps.parts : &maps.in, 32 * i,
                                (int)(st + unit) * kHeadDim, &sm.st_full);
            }
        }
        __syncwarp();
    }
    if (warp >= kConvWarp0 && warp < kConvWarp0 + 4) sm.bad[32 * (warp - kConvWarp0) + lane] = 0x7fffffff;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
    bool ok = true;

    if (warp == kTmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        // ---- loads ---------------------------------------------------------------------------
        if (starts && chunks > 1) {              // (the state came where q's second stage is)
            ok = mbar_wait(&sm.st_free, 0, a.err);
            if (ok && elect_one()) load_q(1);
            __syncwarp();
        }
        if (chunks > kStages && elect_one()) prefetch(kStages);
        __syncwarp();
        for (int c = kStages; c < chunks && ok; ++c) {
            const uint32_t was = (uint32_t)((c / kStages - 1) & 1);
            ok = mbar_wait(&sm.k_free[c % kStages], was, a.err);
            if (ok && elect_one()) {
                load_k(c);
                if (c + 1 < chunks) prefetch(c + 1);
            }
            __syncwarp();
            if (STATE) continue;
            ok = ok && mbar_wait(&sm.q_free[c % kStages], was, a.err);
            if (ok && elect_one()) load_q(c);
            __syncwarp();
        }
        if (!ok)                                 // no load may land after the CTA has left
            for (uint32_t p = 0; p < 2; ++p) {
                for (int i = 0; i < 2; ++i) mbar_wait(&sm.k_full[i], p, nullptr);
                for (int i = 0; !STATE && i < 2; ++i) mbar_wait(&sm.q_full[i], p, nullptr);
                if (starts) mbar_wait(&sm.st_full, 0, nullptr);
            }
    } else if (warp < kTmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        // ---- MMAs: scores and the state's update by one warp, S' Q^T by the next, V'^T P^T by the third ----
        constexpr uint32_t id_sc = tc_idesc_bf16(kC, kC), id_sc2 = tc_idesc_bf16(kC, 2 * kC);
        constexpr uint32_t id_u = tc_idesc_bf16(128, 128) | kTcBMajorMN;
        constexpr uint32_t id_o = tc_idesc_bf16(128, kC);
        const uint32_t b0 = __shfl_sync(0xffffffffu, smem_u32(base), 0);
        if (warp == kUWarp) {
            for (int c = 0; c < chunks; ++c) {
                const int st = c % kStages, odd = c & 1;
                const uint32_t par = (uint32_t)(c & 1), pc = (uint32_t)((c >> 1) & 1);
                ok = mbar_wait(&sm.k_full[st], pc, a.err) && (c == 0 || mbar_wait(&sm.u_free, par ^ 1u, a.err));
                if (!STATE) {
                    ok = ok && mbar_wait(&sm.q_full[st], pc, a.err);
                    if (!ok) break;
                    tc_fence_after();
                    // (M = 64: token t's row of scores is on lane 32 (t / 16) + t % 16)
                    const uint64_t q0 = tc_smem_desc_sw128(b0 + kQAt + st * kPlaneBytes);
                    const uint64_t k0 = tc_smem_desc_sw128(b0 + kKAt + st * kPlaneBytes);
                    if (elect_one()) {
// mid (hi, mid) into both halves of the columns; hi lo and lo hi into the first; hi (hi, mid) into
                        // both, 64 keys each time: of k two parts in one MMA, whose time hardly grows with them
#pragma unroll 1
                        for (int x = 0; x < 8; ++x) {
                            const int term = x >> 1;
                            const uint32_t h = (x & 1) * kHalfBytes;
                            const uint64_t q = tc_desc_advance(q0, (term == 0 ? 1 : term == 2 ? 2 : 0) * kHalf + h);
                            const uint64_t k = tc_desc_advance(k0, (term == 1 ? 2 : 0) * kHalf + h);
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                tc_mma_ss(tmem + kTSc, tc_desc_advance(q, 32 * ks), tc_desc_advance(k, 32 * ks),
                                          term == 0 || term == 3 ? id_sc2 : id_sc, x > 0 || ks > 0);
                        }
                        tc_commit(&sm.sc_full[odd]);
                        tc_commit(&sm.k_free[st]);
                        tc_commit(&sm.q_free[st]);
                    }
                    __syncwarp();
                    ok = mbar_wait(&sm.sc_free, par, a.err);
                }
                ok = ok && mbar_wait(strong && !STATE ? &sm.vu_full[odd] : &sm.v_full[odd], pc, a.err);
                if (!ok) break;
                tc_fence_after();
                const uint64_t km = tc_smem_desc_sw128_mn(b0 + kKAt + st * kPlaneBytes, kHalfBytes);
                if (elect_one()) {
#pragma unroll 1
                    for (int x = 0; x < kTerms; ++x) {
                        const uint32_t v = tmem + kTV - (STATE && (c & 1) ? kTV : 0u) + 32 * a_part(x);
                        const uint64_t k = tc_desc_advance(km, b_part(x) * kHalf);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            tc_mma_ts(tmem + kTU, v + 8 * ks, tc_desc_advance(k, 2048 * ks), id_u, x > 0 || ks > 0);
                    }
                    tc_commit(&sm.u_full);
                    tc_commit(&sm.k_free[st]);
                    tc_commit(&sm.v_free[odd]);
                }
                __syncwarp();
            }
            // no arrival of the tensor pipe on a barrier of a CTA that has left: each warp sees its last
            if (ok && chunks > 0)
                ok = mbar_wait(&sm.v_free[(chunks - 1) & 1], (uint32_t)(((chunks - 1) >> 1) & 1), a.err);
        } else if (STATE) {
        } else if (warp == kOiWarp) {
            for (int c = 0; c < chunks; ++c) {
                const int st = c % kStages;
                const uint32_t par = (uint32_t)(c & 1), pc = (uint32_t)((c >> 1) & 1);
                const uint64_t q0 = tc_smem_desc_sw128(b0 + kQAt + st * kPlaneBytes);
                const auto terms = [&](int x, int end) {
#pragma unroll 1
                    for (bool first = x == 0; x < end; ++x) {
                        const uint32_t sp = tmem + kTSp + 64 * a_part(x);
                        const uint64_t q = tc_desc_advance(q0, b_part(x) * kHalf);
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks, first = false)
                            tc_mma_ts(tmem + kTO, sp + 8 * ks, tc_desc_advance(q, (ks >> 2) * kHalfBytes + (ks & 3) * 32),
                                      id_o, !first);
                    }
                };
                // (the state's parts come after o of the chunk before is read)
                ok = mbar_wait(&sm.q_full[st], pc, a.err) && mbar_wait(&sm.sp_full, par, a.err);
                if (!ok) break;
                tc_fence_after();
                if (!strong) {
                    if (elect_one()) {
                        terms(0, kTerms - 1);
                        tc_commit(&sm.os_full);
                    }
                    __syncwarp();
                }
                ok = mbar_wait(&sm.oa_full[c & 1], pc, a.err) && (!strong || mbar_wait(&sm.oa_free, par, a.err));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    terms(strong ? 0 : kTerms - 1, kTerms);
                    tc_commit(&sm.o_full);
                    tc_commit(&sm.q_free[st]);
                }
                __syncwarp();
            }
            if (ok && chunks > 0)
                ok = mbar_wait(&sm.q_free[(chunks - 1) % kStages], (uint32_t)(((chunks - 1) / kStages) & 1), a.err);
        } else {
            const uint64_t p0 = tc_smem_desc_sw128(b0 + kPAt);
            for (int c = 0; c < chunks; ++c) {
                const uint32_t par = (uint32_t)(c & 1);
                ok = mbar_wait(&sm.v_full[c & 1], (uint32_t)((c >> 1) & 1), a.err) &&
                     mbar_wait(&sm.p_full, par, a.err) &&
                     (strong ? c == 0 || mbar_wait(&sm.o_free, par ^ 1u, a.err) : mbar_wait(&sm.os_full, par, a.err));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll 1
                    for (int x = 0; x < kTerms; ++x) {
                        const uint32_t v = tmem + kTV + 32 * a_part(x);
                        const uint64_t p = tc_desc_advance(p0, b_part(x) * kHalf);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            tc_mma_ts(tmem + kTO, v + 8 * ks, tc_desc_advance(p, 32 * ks), id_o,
                                      !strong || x > 0 || ks > 0);
                    }
                    tc_commit(&sm.oa_full[c & 1]);
                    tc_commit(&sm.v_free[c & 1]);
                }
                __syncwarp();
            }
            if (ok && chunks > 0)
                ok = mbar_wait(&sm.v_free[(chunks - 1) & 1], (uint32_t)(((chunks - 1) >> 1) & 1), a.err);
        }
        if (!ok) {                               // a wait gave up: whatever still runs ends first
            if (elect_one()) tc_commit(&sm.drain[warp]);
            __syncwarp();
            mbar_wait(&sm.drain[warp], 0, nullptr);
        }
    } else if (warp >= kConvWarp0) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConvRegs));
        // ---- v and the scores into bf16 parts: 32 tokens of each chunk a group of warps --------
        const int quarter = (warp - kConvWarp0) & 3, group = (warp - kConvWarp0) / kGroupWarps;
        const int j = 32 * quarter + lane, own = 32 * group;
        const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16);
        const long vs = a.v_stride;
        const float* const v = static_cast<const float*>(a.v) + (begin + own) * vs + (long)unit * kHeadDim + j;
        // a chunk's 32 tokens of this thread's value
        const auto load_v = [&](float (&x)[32], int c) {
            const float* p = v + (long)c * kC * vs;
            const int live = len - c * kC - own;
            if (live >= 32) {
#pragma unroll
                for (int i = 0; i < 32; ++i, p += vs) x[i] = __ldcs(p);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i, p += vs) x[i] = i < live ? __ldcs(p) : 0.0f;
            }
        };
        // as parts, times their factors; nt tokens of the chunk are the sequence's.  The first token at which v is no
        // number, if any
        const auto put_v = [&](float (&x)[32], int c, int nt, bool late) {
            const float2 zero2 = make_float2(0.0f, 0.0f);
            float2 odd = zero2;                  // 0 times v, summed: 0 unless one is no number
            int bad = 0x7fffffff;
#pragma unroll
            for (int i = 0; i < 16; ++i) odd = __ffma2_rn(make_float2(x[2 * i], x[2 * i + 1]), zero2, odd);
            if (__any_sync(0xffffffffu, !(odd.x + odd.y == 0.0f)))
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (!(fabsf(x[i]) < __int_as_float(0x7f800000))) {
                        bad = min(bad, own + i);
                        x[i] = 0.0f;
                    }
            const uint32_t to = tl + kTV - (STATE && (c & 1) ? kTV : 0u) + 16 * group;
#pragma unroll
            for (int b = 0; b < 4; ++b) {        // 8 tokens: 4 columns of each part
                uint32_t w[4][kParts];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 8 * b + 2 * i, s = own + r;
                    const float2 f = late ? make_float2(sm.pw[max(nt - 1 - s, 0)], sm.pw[max(nt - 2 - s, 0)])
                                          : *reinterpret_cast<const float2*>(sm.down + s);
                    split(__fmul2_rn(make_float2(x[r], x[r + 1]), f), w[i]);
                }
#pragma unroll
                for (int p = 0; p < kParts; ++p) tmem_st4(to + 32 * p + 4 * b, {w[0][p], w[1][p], w[2][p], w[3][p]});
            }
            tmem_st_wait();
            tc_fence_before();
            return bad;
        };
        float x[32];
        load_v(x, 0);
        for (int c = 0; c < chunks; ++c) {
            const int st = c % kStages;
            const uint32_t pc = (uint32_t)((c >> 1) & 1);
            const int nt = min(kC, len - c * kC);
            constexpr int kBehind = STATE ? 2 : 1;                        // chunks ahead of V's buffer
            ok = c < kBehind || mbar_wait(&sm.v_free[(c - kBehind) & 1], (uint32_t)(((c - kBehind) >> 1) & 1), a.err);
            if (!ok) break;
            tc_fence_after();
            const int bad = put_v(x, c, nt, STATE && strong);
            if (bad != 0x7fffffff) atomicMin(&sm.bad[j], c * kC + bad);
            if (nt < kC) {                       // 0 times a NaN of another sequence's k is not 0
                ok = mbar_wait(&sm.k_full[st], pc, a.err);
                if (!ok) break;
                unsigned char* k = base + kKAt + st * kPlaneBytes + nt * 128;
                for (int h = 0; h < 2 * kParts; ++h, k += kHalf)
                    for (int i = 4 * own + j; i < (kC - nt) * 8; i += 32 * kConvWarps)
                        *reinterpret_cast<uint4*>(k + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
            }
            warp_arrive(&sm.v_full[c & 1]);
            // the next chunk's on its way, the one after it into L2: a row's 128 bytes a lane
            if (c + 1 < chunks && (STATE || !strong)) load_v(x, c + 1);
            if ((c + 2) * kC + own + lane < len)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(v - lane + ((long)(c + 2) * kC + lane) * vs));
            if (STATE) continue;
            if (group <= quarter) {
                // rows 16 quarter .. of the scores, every other 16 of the tokens s that they see
                const int r0 = 16 * quarter + (lane >> 2), s0 = 2 * (lane & 3);
                const int prow = 16 * quarter + (lane & 15), piece = lane >> 4;  // whose address this lane gives
                unsigned char* const row = base + kPAt + prow * 128;
                ok = mbar_wait(&sm.sc_full[c & 1], pc, a.err) &&
                     (c > 0 ? mbar_wait(&sm.oa_full[(c - 1) & 1], (uint32_t)(((c - 1) >> 1) & 1), a.err)
                            : !starts || mbar_wait(&sm.st_free, 0, a.err));
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int b = group; b <= quarter; b += 2) {
                    float y[8], y2[8];
                    tmem_ld_16x256b_x2(tl + kTSc + 16 * b, y);
                    tmem_ld_16x256b_x2(tl + kTSc + kC + 16 * b, y2);
                    tmem_ld_wait();
                    if (b + 2 > quarter) {
                        tc_fence_before();
                        warp_arrive(&sm.sc_free);
                    }
                    uint32_t w[4][kParts];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = r0 + 8 * (i & 1), s = 16 * b + s0 + 8 * (i >> 1);
                        float2 z = __fadd2_rn(make_float2(y[2 * i], y[2 * i + 1]), make_float2(y2[2 * i], y2[2 * i + 1]));
                        if (strong) z = __fmul2_rn(z, make_float2(sm.pw[max(t - s, 0)], sm.pw[max(t - s - 1, 0)]));
                        // (where s > t not 0 times q k: it is what it is for tokens to come, and another sequence's
                        // behind the end)
                        split(make_float2(s <= t ? z.x : 0.0f, s + 1 <= t ? z.y : 0.0f), w[i]);
                    }
                    const uint32_t to = smem_u32(row) + (((2 * b + piece) ^ (prow & 7)) * 16);
#pragma unroll
                    for (int p = 0; p < kParts; ++p) stsm4(to + p * kHalf, {w[0][p], w[1][p], w[2][p], w[3][p]});
                }
                if (c == 0 && group == 0)        // tokens that none of these rows sees: 0 once and for all
                    for (int q = 2 * (quarter + 1) + piece; q < 8; q += 2)
                        for (int p = 0; p < kParts; ++p)
                            *reinterpret_cast<uint4*>(row + p * kHalf + ((q ^ (prow & 7)) * 16)) =
                                make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                warp_arrive(&sm.p_full);
            }
            if (strong) {
                load_v(x, c);
                ok = mbar_wait(&sm.oa_full[c & 1], pc, a.err);
                if (!ok) break;
                tc_fence_after();
                put_v(x, c, nt, true);
                warp_arrive(&sm.vu_full[c & 1]);
                if (c + 1 < chunks) load_v(x, c + 1);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStateRegs));
        // ---- the state and o -----------------------------------------------------------------
        // value row j; keys 32 part .. of its state, tokens 16 part .. of its outputs
        const int j = 32 * (warp & 3) + lane, part = (warp - kStateWarp0) >> 2;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        float2 S[16];                            // times e^{mid g}
        unsigned char* const tile = base + kStAt + part * kStTile + j * 128;
        if (starts) {
            ok = mbar_wait(&sm.st_full, 0, a.err);
            const float in = chunks > 0 ? sm.pw[mid] : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 x = *reinterpret_cast<const float4*>(tile + ((i ^ (j & 7)) * 16));
                S[2 * i] = make_float2(x.x * in, x.y * in);
                S[2 * i + 1] = make_float2(x.z * in, x.w * in);
            }
            // (scores or q's second tile come there next: by ordinary stores, by TMA)
            fence_proxy_async_smem();
            warp_arrive(&sm.st_free);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) S[i] = make_float2(0.0f, 0.0f);
        }
        auto put_state = [&]() {
#pragma unroll
            for (int b = 0; b < 4; ++b) {        // 8 keys: 4 columns of each part
                uint32_t w[4][kParts];
#pragma unroll
                for (int i = 0; i < 4; ++i) split(S[4 * b + i], w[i]);
#pragma unroll
                for (int p = 0; p < kParts; ++p)
                    tmem_st4(tl + kTSp + 64 * p + 16 * part + 4 * b, {w[0][p], w[1][p], w[2][p], w[3][p]});
            }
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&sm.sp_full);
        };
        if (!STATE && chunks > 0 && ok) put_state();
        const float2 whole = decay_pair(g * (float)kC);
        const long step = (long)units * kHeadDim;
        // (rows by 32-bit offsets from an address that the whole warp shares: one addition a store)
        float* o = a.o + (begin + 16 * part) * step + (long)unit * kHeadDim;
        const uint32_t step4 = (uint32_t)step * 4;
        const float4* up = reinterpret_cast<const float4*>(sm.up + 16 * part);
        for (int c = 0; c < chunks && ok; ++c, o += kC * step) {
            const uint32_t par = (uint32_t)(c & 1);
            const int nt = min(kC, len - c * kC), live = nt - 16 * part;
            const uint32_t to = tl + kTO + 16 * part;
            const float2 f = nt == kC ? whole : decay_pair(g * (float)nt);
            const float2 fa2 = make_float2(f.x, f.x), fd2 = make_float2(f.y, f.y);
            const float fu = strong ? 1.0f : sm.pw[nt];
            const float2 fu2 = make_float2(fu, fu);
            ok = mbar_wait(&sm.u_full, par, a.err);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float u[16];
                tmem_ld16(tl + kTU + 32 * part + 16 * b, u);
                tmem_ld_wait();
                if (b == 1) {
                    tc_fence_before();
                    warp_arrive(&sm.u_free);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float2& y = S[8 * b + i];
                    const float2 add = __fmul2_rn(fu2, make_float2(u[2 * i], u[2 * i + 1]));
                    y = __ffma2_rn(fa2, y, __ffma2_rn(fd2, y, add));
                }
            }
            const int bad = sm.bad[j];
            const bool any_bad = __any_sync(0xffffffffu, bad < (c + 1) * kC);
            if (any_bad) {
                const float nan = bad < (c + 1) * kC ? __int_as_float(0x7fffffff) : 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) S[i] = make_float2(S[i].x + nan, S[i].y + nan);
            }
            if (STATE) continue;
            if (strong) {                        // V^T P^T by itself: stored, and S Q^T added to it below
                ok = mbar_wait(&sm.oa_full[c & 1], (uint32_t)((c >> 1) & 1), a.err);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int t = 0; t < 16; t += 4) {
                    float x[4];
                    tmem_ld4(to + t, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (t + i < live) o[(t + i) * step + j] = a.scale * x[i];
                }
                tc_fence_before();
                warp_arrive(&sm.oa_free);
            }
            ok = mbar_wait(&sm.o_full, par, a.err);      // O is whole, S Q^T has read the parts
            if (!ok) break;
            tc_fence_after();
            float x[16];                         // (first, so that V^T P^T of the next chunk may start)
            tmem_ld16(to, x);
            tmem_ld_wait();
            tc_fence_before();
            warp_arrive(&sm.o_free);
            if (c + 1 < chunks) put_state();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = up[i];
                const float2 u = __fmul2_rn(make_float2(x[4 * i], x[4 * i + 1]), make_float2(f.x, f.y));
                const float2 w = __fmul2_rn(make_float2(x[4 * i + 2], x[4 * i + 3]), make_float2(f.z, f.w));
                x[4 * i] = u.x; x[4 * i + 1] = u.y; x[4 * i + 2] = w.x; x[4 * i + 3] = w.y;
            }
            if (any_bad)
#pragma unroll
                for (int t = 0; t < 16; ++t)
                    if (c * kC + 16 * part + t >= bad) x[t] = __int_as_float(0x7fffffff);
            uint32_t at_o = (uint32_t)j * 4;
            if (live >= 16 && !strong) {
#pragma unroll
                for (int t = 0; t < 16; ++t, at_o += step4)
                    __stcs(reinterpret_cast<float*>(reinterpret_cast<char*>(o) + at_o), x[t]);
            } else {
#pragma unroll
                for (int t = 0; t < 16; ++t, at_o += step4)
                    if (t < live) {
                        float* ob = reinterpret_cast<float*>(reinterpret_cast<char*>(o) + at_o);
                        *ob = strong ? *ob + x[t] : x[t];
                    }
            }
        }
        if (ok && (STATE || at.ends)) {
            const float out = chunks > 0 ? 1.0f / sm.pw[mid] : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float4*>(tile + ((i ^ (j & 7)) * 16)) =
                    make_float4(S[2 * i].x * out, S[2 * i].y * out, S[2 * i + 1].x * out, S[2 * i + 1].y * out);
            fence_proxy_async_smem();
            warp_arrive(&sm.st_out[part]);       // one of the tile's four warps
            if ((warp & 3) == 0 && mbar_wait(&sm.st_out[part], 0, a.err) && elect_one()) {
                const long st = STATE ? piece_state(cut, n, seg, units) : (long)n * units;
                tma_store_2d(&maps.out, base + kStAt + part * kStTile, 32 * part, (int)(st + unit) * kHeadDim);
                bulk_commit();
                bulk_wait_read0();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kUWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// f32 rows as three bf16 parts, each packed: a plane's first [rows][cols], its second, its third.
constexpr int kSplitThr = 256;

struct SplitPlane {
    const float* src; uint2* parts;
    long stride;                                 // elements between rows
};
struct SplitArgs {
    SplitPlane p[2];                             // q, k
    long rows; int heads;                        // groups of 128 in a row
};

// A warp takes kSplitAhead heads at a time, their loads ahead of their stores.
constexpr int kSplitAhead = 4;

__global__ void __launch_bounds__(kSplitThr) kda_linattn_split_kernel(const __grid_constant__ SplitArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const SplitPlane& p = a.p[blockIdx.y];
    const int lane = threadIdx.x & 31, heads = a.heads;
    const long n = a.rows * heads, step = (long)gridDim.x * (kSplitThr / 32) * kSplitAhead;
    for (long i = ((long)blockIdx.x * (kSplitThr / 32) + (threadIdx.x >> 5)) * kSplitAhead; i < n; i += step) {
        long row = i / heads;
        int head = (int)(i - row * heads);
        float4 x[kSplitAhead];
#pragma unroll
        for (int u = 0; u < kSplitAhead; ++u) {
            if (i + u < n) x[u] = __ldcs(reinterpret_cast<const float4*>(p.src + row * p.stride) + head * 32 + lane);
            if (++head == heads) { head = 0; ++row; }
        }
#pragma unroll
        for (int u = 0; u < kSplitAhead; ++u) {
            if (i + u >= n) break;
            uint32_t w[2][kParts];
            split(make_float2(x[u].x, x[u].y), w[0]);
            split(make_float2(x[u].z, x[u].w), w[1]);
#pragma unroll
            for (int q = 0; q < kParts; ++q) p.parts[(q * n + i + u) * 32 + lane] = make_uint2(w[0][q], w[1][q]);
        }
    }
}

template <bool STATE>
cudaError_t launch(const LinArgs& a, const Cut& cut, const Maps& maps, cudaStream_t s) {
    static PerDevice<int> done;
    const cudaError_t e = set_smem(kda_linattn_chunk_f32_kernel<STATE>, kSmemBytes, done);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.H * a.m), (unsigned)a.seq.N, (unsigned)(STATE ? cut.pieces() : cut.segs));
    return launch_as(STATE ? kKLinState : kKLinChunk, true, kda_linattn_chunk_f32_kernel<STATE>, grid, kThr, kSmemBytes,
                     s, a, cut, maps);
}

}  // namespace

size_t linattn::f32_split_bytes(long rows, int Hk) { return (size_t)rows * 2 * Hk * kHeadDim * kParts * 2; }

cudaError_t linattn::launch_chunks_f32(const LinArgs& a, const Cut& cut, const StateMaps& states, void* workspace,
                                       cudaStream_t s) {
    const long rows = a.seq.total_rows, qk = (long)a.Hk * kHeadDim;
    Maps maps;
    SplitArgs sp;
    sp.rows = rows;
    sp.heads = a.Hk;
    for (int i = 0; i < 2; ++i) {
        unsigned char* const at = static_cast<unsigned char*>(workspace) + (size_t)i * rows * qk * kParts * 2;
        sp.p[i] = SplitPlane{static_cast<const float*>(i ? a.k : a.q), reinterpret_cast<uint2*>(at),
                             i ? a.k_stride : a.q_stride};
        for (int p = 0; p < kParts; ++p)
            if (!make_tensor_map_2d_bf16_sw128(i ? &maps.k[p] : &maps.q[p], at + (size_t)p * rows * qk * 2, rows, qk, kC))
                return cudaErrorInvalidValue;
    }
    maps.in = states.in;
    maps.parts = maps.out = states.parts;
    {
        KernelTimer kt(kKLinSplit, s);
        const long blocks = (rows * a.Hk + kSplitThr / 32 * kSplitAhead - 1) / (kSplitThr / 32 * kSplitAhead);
        kda_linattn_split_kernel<<<dim3((unsigned)std::min(blocks, 152L * 8), 2), kSplitThr, 0, s>>>(sp);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (cut.segs > 1) {
        cudaError_t e = launch<true>(a, cut, maps, s);
        if (e == cudaSuccess) e = launch_join(a, cut, s);
        if (e != cudaSuccess) return e;
    }
    maps.out = states.out;
    return launch<false>(a, cut, maps, s);
}

}  // namespace kda
