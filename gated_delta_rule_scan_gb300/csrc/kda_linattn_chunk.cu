// kda_linattn_chunk.cu -- linear attention with one log-decay g a head, the chunked form for bf16 prompts, on the
// tcgen05 tensor cores; and how prompts of either type are cut (kda_linattn_chunk_f32.cu has f32's form).
//
// Mathematics.  Over a chunk of C = 64 tokens with incoming state S (stored [value j][key i]):
//     O^T = scale * ( V^T P^T + e^{g (t+1)} S Q^T ),   P[t][s] = e^{g (t-s)} q_t . k_s  for s <= t,
//     S  <- e^{g C} S + V^T Kd,                        Kd[s]   = e^{g (C-1-s)} k_s.
// Both parts of O are one sum in the tensor cores when its rows share a factor: with everything
// relative to the middle of the chunk, P[t][s] = e^{g (31-s)} q_t . k_s, the state kept as e^{32 g} S
// (and Kd 32 further on), a token's output is e^{g (t-31)} times that sum.  These factors stay within
// e^{32 |g|}, 8e13 at |g| = 1.  Heads that decay faster (g < -1) take the parts one after the other, with
// the powers as they stand, all of them at most 1, and a slower pipeline: there S Q^T matters to a few tens
// of tokens at most, but overflow must not.
// q, k and v enter as they are; what is f32 (P, Kd and the state) enters as three bf16 parts, 24 bits of it: o is off
// by 4e-7 to 8e-7 of a head's norm, most of it the tensor cores' truncated sums (two parts: 3e-6).  The state itself
// stays in f32 registers.
//
// A NaN or an infinity at one token does not reach the tokens before it: where q k is not seen P is 0 by
// selection, and in v, whose products with P = 0 would be NaN, it is replaced by 0 and its value column made
// NaN from that token on (by an infinity too).
//
// One CTA per (sequence, 128-wide value unit), chunk after chunk, the values on the MMA's M = 128 TMEM
// lanes.  Shared memory carries what the tensor cores read of it at 128 bytes a cycle, so the A
// operands lie in tensor memory: the state parts, written by the threads that hold the state rows, and
// v, transposed on the way (from shared memory as an MN-major operand it cost twice its bytes: U 140
// cycles an MMA against 64).  B operands are q's tile as TMA brings it, P, and Kd transposed to
// [key][token] while it is formed.  The 512 TMEM columns are full: S parts 3 x 64, V^T Kd 128, the
// outputs 64, q k 64, v 2 x 32.
// 64 tokens, not 128: the parts of P and Kd then fit beside two stages of q, k, v.
// Warps have roles: 16 hold the state (32 f32 a thread) and write o, 8 turn k into Kd and q k into P (4 of
// them a chunk, in turn), three issue MMAs, one the TMA loads; they meet on mbarriers only, so the loads,
// the MMAs and the groups' register work overlap across chunks.  (One issuing warp took 50 to 100 cycles an
// MMA beside six busy warps on its scheduler, twice the tensor pipe's time.)
// The roles' loops run at once, so their code has to share the instruction caches: unrolled, every fourth
// stall was for an instruction, the worse the more SMs were busy (152 heads x 4096 tokens: 210 us; with the
// loops over terms, halves and columns rolled up 164).
//
// Measured: 152 heads x 4096 tokens (a CTA an SM) 164 us, 4.9 TB/s of what it reads and writes; 16 ragged
// prompts, 64 heads, 73722 tokens: 1222 us, 5.1 TB/s, 75% of a copy's rate.  Issue slots are 64% taken, the
// tensor pipe 56%: a chunk takes 2.0 to 2.4 us where the MMAs take 1.3, bound by the state's warps, which are
// busy throughout: 870 cycles for V^T Kd, 1360 for the state's parts, 1540 for o.
//
// Few sequences and heads leave SMs idle, so long sequences are then cut into segments: a first launch
// (STATE) forms each segment's own contribution to the state from k and v alone, in pieces where that leaves SMs
// idle, a second adds them up to the state that each segment starts from, and the third is the kernel above with
// a CTA a segment.  The cut is chosen by a cost model (plan()).
#include "kda_linattn_chunk.cuh"

#include <algorithm>
#include <cstring>

namespace kda {

using namespace linattn;

namespace {

constexpr int kStages = 2;
constexpr int kPWarps = 3;                       // of the converting warps of a chunk, those with a share of P
constexpr int kStateRegs = 80, kConvRegs = 80;
static_assert(regs_fit(kStateRegs, kConvRegs), "");
// barriers of k and v: a chunk's comes two chunks later again at the earliest, since its group of warps knows
// only of its own chunks that they have passed
constexpr int kBars = 2;
constexpr int kKvBytes = 2 * kTileBytes, kVAt = kTileBytes;      // a stage: k, v
constexpr int kQAt = kStages * kKvBytes;
constexpr int kKdBytes = kParts * kTileBytes;                    // Kd's parts, two buffers
constexpr int kKdAt = kQAt + kStages * kTileBytes;
constexpr int kPAt = kKdAt + 2 * kKdBytes;                       // P's parts, [64 t][64 s] each
constexpr int kTailAt = kPAt + kParts * kHalf;
// TMEM columns; v has two buffers
constexpr uint32_t kTSp = 0, kTU = 64 * kParts, kTO = kTU + 128, kTSc = kTO + 64, kTVt = kTSc + 64, kVtCols = 32;
static_assert(kTVt + 2 * kVtCols <= 512 && 4 * kStTile <= 2 * kKdBytes, "");

struct __align__(16) Tail {
    float pw[kC + kMid + 4];                     // e^{g n}, n = 0 .. 96
    float down[kC];                              // P's factors: e^{g (31-s)}
    float up[kC];                                // the outputs': scale * e^{g (t-31)}, or scale * e^{g (t+1)}
    uint64_t kv_full[2], kv_free[2], q_full[2], q_free[2];
    uint64_t kd_full[2], kd_free[2];
    uint64_t sc_full[2], sc_free, u_full, u_free, sp_full, p_full, oa_full[2], oa_free, o_full, o_free;
    uint64_t st_full, st_free, st_out[4];        // the state on its way in and out
    uint64_t drain[3];
    uint32_t tmem;
    int bad[kHeadDim];                           // by value: the first token whose v is no number
};
constexpr int kSmemBytes = 1024 + kTailAt + (int)sizeof(Tail);
static_assert(kSmemBytes <= kMaxBlockSmem, "");

// Four 8 x 8 blocks of bf16 from shared memory, transposed: lane l gets elements (2 (l % 4), l / 4) and
// the one below of each, 8 lanes giving the addresses of a block's rows.
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 16 lanes x 16 columns of TMEM: lane l's words 2 i and 2 i + 1 go to lanes l / 4 and l / 4 + 8, column
// 4 i + l % 4.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

struct Maps {
    CUtensorMap q, k, v, in, parts, out;         // out: the parts in the STATE launch, else state_out
};

template <bool STATE>
__global__ void __launch_bounds__(kThr, 1)
kda_linattn_chunk_kernel(const LinArgs a, const Cut cut, const __grid_constant__ Maps maps) {
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
    const bool ends = at.ends;
    const int chunks = (len + kC - 1) / kC;
    const float g = a.log_decay[hv];
    const bool strong = g < -1.0f;
    const int mid = strong ? 0 : kMid;           // the state is kept as e^{mid g} S

    // what this CTA starts from; it comes through shared memory, where Kd will be: 4 tiles of 128 rows x 32 keys
    const bool starts = !STATE && (seg > 0 || a.state_in != nullptr);

    if (warp == kUWarp) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    const auto load_kv = [&](int c) {            // by one thread
        unsigned char* s = base + c % kStages * kKvBytes;
        uint64_t* bar = &sm.kv_full[c % kBars];
        const int row = (int)(begin + (long)c * kC);
        mbar_arrive_expect_tx(bar, kKvBytes);
        for (int h = 0; h < 2; ++h) {
            tma_load_2d(s + h * kHalf, &maps.k, hk * kHeadDim + 64 * h, row, bar);
            tma_load_2d(s + kVAt + h * kHalf, &maps.v, unit * kHeadDim + 64 * h, row, bar);
        }
    };
    const auto load_q = [&](int c) {
        unsigned char* s = base + kQAt + c % kStages * kTileBytes;
        uint64_t* bar = &sm.q_full[c % kStages];
        mbar_arrive_expect_tx(bar, kTileBytes);
        for (int h = 0; h < 2; ++h)
            tma_load_2d(s + h * kHalf, &maps.q, hk * kHeadDim + 64 * h, (int)(begin + (long)c * kC), bar);
    };
    // Into L2: what chunk c has no stage for yet.  (Further ahead it only pushed other CTAs' out: 4 chunks cost 1%.)
    const auto prefetch = [&](int c) {
        for (int h = 0; h < 2; ++h)
            if (!STATE) tma_prefetch_2d(&maps.q, hk * kHeadDim + 64 * h, (int)(begin + (long)c * kC));
    };
    const auto first_loads = [&]() {
        for (int c = 0; c < kStages && c < chunks; ++c) load_kv(c);
        for (int c = 0; !STATE && c < kStages && c < chunks; ++c) load_q(c);
        if (chunks > kStages) prefetch(kStages);
    };
    // the next launch may be set up meanwhile; it waits for the end of this one before it reads what this one writes
    if (STATE) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == kTmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sm.kv_full[i], 1);
                mbar_init(&sm.kv_free[i], kGroupWarps + !STATE);
                mbar_init(&sm.q_full[i], 1);
                mbar_init(&sm.q_free[i], 2);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sm.kd_full[i], kGroupWarps);
                mbar_init(&sm.kd_free[i], STATE ? 1 : 2);
            }
            for (int i = 0; i < 2; ++i) mbar_init(&sm.sc_full[i], 1);
            mbar_init(&sm.sc_free, kPWarps);
            mbar_init(&sm.u_full, 1);
            mbar_init(&sm.u_free, kStateWarps);
            mbar_init(&sm.sp_full, kStateWarps);
            mbar_init(&sm.o_full, 1);
            mbar_init(&sm.p_full, kPWarps);
            for (int i = 0; i < 2; ++i) mbar_init(&sm.oa_full[i], 1);
            mbar_init(&sm.oa_free, kStateWarps);
            mbar_init(&sm.o_free, kStateWarps);
            for (int i = 0; i < 3; ++i) mbar_init(&sm.drain[i], 1);
            mbar_init(&sm.st_full, 1);
            mbar_init(&sm.st_free, kStateWarps);
            for (int i = 0; i < 4; ++i) mbar_init(&sm.st_out[i], 4);
            fence_mbar_init();
            first_loads();
        }
        __syncwarp();
        // e^{g n}; n = 0 apart, so that a log-decay of -infinity is a plain reset
        for (int i = lane; i <= kC + kMid; i += 32) sm.pw[i] = i == 0 ? 1.0f : expf(g * (float)i);
        for (int i = lane; i < kC; i += 32) {
            sm.down[i] = strong || i == kMid - 1 ? 1.0f : expf(g * (float)(kMid - 1 - i));
            const int n = strong ? i + 1 : i - kMid + 1;
            sm.up[i] = a.scale * (n == 0 ? 1.0f : expf(g * (float)n));
        }
        if (lane == 0) {
            // the launch before has written the state that a segment starts from
            if (seg > 0) asm volatile("griddepcontrol.wait;" ::: "memory");
            if (starts) {
                const long st = seg > 0 ? piece_state(cut, n, seg * cut.subs - 1, units) : (long)n * units;
                mbar_arrive_expect_tx(&sm.st_full, 4 * kStTile);
                for (int i = 0; i < 4; ++i)
                    tma_load_2d(base + kKdAt + i * kStTile, seg > 0 ? &maps.parts : &maps.in, 32 * i,
                                (int)(st + unit) * kHeadDim, &sm.st_full);
            }
        }
        __syncwarp();
    }
    if (warp >= kConvWarp0 && warp < kConvWarp0 + 4) sm.bad[32 * (warp - kConvWarp0) + lane] = 0x7fffffff;
    if (warp == kConvWarp0) {                    // t < 32 <= s: P is 0 there, once and for all
#pragma unroll
        for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int q = 4; q < 8; ++q)
                *reinterpret_cast<uint4*>(base + kPAt + p * kHalf + lane * 128 + ((q ^ (lane & 7)) * 16)) =
                    make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
    bool ok = true;

    if (warp == kTmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        // ---- loads ---------------------------------------------------------------------------
        // (in the order in which the stages come free: k and v are done with a product earlier than q)
        for (int c = kStages; c < chunks && ok; ++c) {
            const int was = c - kStages;
            ok = mbar_wait(&sm.kv_free[was % kBars], (uint32_t)((was / kBars) & 1), a.err);
            if (ok && elect_one()) {
                load_kv(c);
                if (c + 1 < chunks) prefetch(c + 1);
            }
            __syncwarp();
            if (STATE || c < kStages) continue;
            ok = ok && mbar_wait(&sm.q_free[c % kStages], (uint32_t)((c / kStages - 1) & 1), a.err);
            if (ok && elect_one()) load_q(c);
            __syncwarp();
        }
        if (!ok)                                 // no load may land after the CTA has left
            for (uint32_t p = 0; p < 2; ++p) {
                for (int i = 0; i < kBars; ++i) mbar_wait(&sm.kv_full[i], p, nullptr);
                for (int i = 0; !STATE && i < kStages; ++i) mbar_wait(&sm.q_full[i], p, nullptr);
                if (starts) mbar_wait(&sm.st_full, 0, nullptr);
            }
    } else if (warp < kTmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        // ---- MMAs: V^T Kd by one warp, S Q^T by the next, q k and V^T P^T by the third -------
        constexpr uint32_t id_sc = tc_idesc_bf16(128, kC / 2);                           // q k
        constexpr uint32_t id_u = tc_idesc_bf16(128, 128);                               // V^T Kd
        constexpr uint32_t id_o = tc_idesc_bf16(128, kC);                                // S Q^T, V^T P^T
        // descriptors by byte offset in shared memory (the address field is the low one, in 16 bytes)
        const uint64_t d0 = tc_smem_desc_sw128(__shfl_sync(0xffffffffu, smem_u32(base), 0));
        if (warp == kUWarp) {
            for (int c = 0; c < chunks; ++c) {
                const int skv = c % kStages, bkv = c % kBars, sq = c % kStages;
                const uint32_t par = (uint32_t)(c & 1);
                // q_t . k_s, s < 32 with q on the lanes 0 .. 63, s >= 32 with q on 64 .. 127: the threads of
                // three lane quarters then share the work on P.  (M = 128 covers twice the rows of q's tile,
                // those behind it, or before it, being whatever lies there: their lanes are never read.)
                if (!STATE) {
                    ok = mbar_wait(&sm.kv_full[bkv], (uint32_t)((c / kBars) & 1), a.err) &&
                         mbar_wait(&sm.q_full[sq], (uint32_t)((c / kStages) & 1), a.err) &&
                         (c == 0 || mbar_wait(&sm.sc_free, par ^ 1u, a.err));
                    if (!ok) break;
                    tc_fence_after();
                }
                const uint64_t k0 = tc_desc_advance(d0, skv * kKvBytes);
                const uint64_t q0 = tc_desc_advance(d0, kQAt + sq * kTileBytes);
                if (!STATE && elect_one()) {
#pragma unroll 1
                    for (int x = 0; x < 2; ++x) {         // 64 keys each time
                        const uint64_t q = tc_desc_advance(q0, x * kHalf), k = tc_desc_advance(k0, x * kHalf);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            tc_mma_ss(tmem + kTSc, tc_desc_advance(q, 32 * ks), tc_desc_advance(k, 32 * ks), id_sc,
                                      x > 0 || ks > 0);
                            tc_mma_ss(tmem + kTSc + 32, tc_desc_advance(q, 32 * ks) - (kHalf >> 4),
                                      tc_desc_advance(k, kHalf / 2 + 32 * ks), id_sc, x > 0 || ks > 0);
                        }
                    }
                    tc_commit(&sm.sc_full[c & 1]);
                    tc_commit(&sm.kv_free[bkv]);
                    tc_commit(&sm.q_free[sq]);
                }
                __syncwarp();
                const uint64_t kd = tc_desc_advance(d0, kKdAt + (c & 1) * kKdBytes);
                const uint32_t vt = tmem + kTVt + kVtCols * (c & 1);
                ok = mbar_wait(&sm.kd_full[c & 1], (uint32_t)((c >> 1) & 1), a.err) &&
                     (c == 0 || mbar_wait(&sm.u_free, par ^ 1u, a.err));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll 1
                    for (int x = 0; x < kParts; ++x) {
                        const int p = kParts - 1 - x;
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            tc_mma_ts(tmem + kTU, vt + 8 * ks,
                                      tc_desc_advance(kd, p * kTileBytes + 32 * ks), id_u, x > 0 || ks > 0);
                    }
                    tc_commit(&sm.u_full);
                    tc_commit(&sm.kd_free[c & 1]);
                }
                __syncwarp();
            }
            // no arrival of the tensor pipe on a barrier of a CTA that has left: each warp sees its last
            if (ok && chunks > 0)
                ok = STATE ? mbar_wait(&sm.kd_free[(chunks - 1) & 1], (uint32_t)(((chunks - 1) >> 1) & 1), a.err)
                           : mbar_wait(&sm.kv_free[(chunks - 1) % kBars],
                                       (uint32_t)(((chunks - 1) / kBars) & 1), a.err);
        } else if (STATE) {
        } else if (warp == kOiWarp) {
            for (int c = 0; c < chunks; ++c) {
                const int st = c % kStages;
                const uint64_t q = tc_desc_advance(d0, kQAt + st * kTileBytes);
                const uint32_t par = (uint32_t)(c & 1);
                ok = mbar_wait(&sm.q_full[st], (uint32_t)((c / kStages) & 1), a.err) &&
                     mbar_wait(&sm.sp_full, par, a.err) &&
                     mbar_wait(&sm.oa_full[c & 1], (uint32_t)((c >> 1) & 1), a.err) &&
                     (!strong || mbar_wait(&sm.oa_free, par, a.err));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll 1
                    for (int x = 0; x < kParts; ++x) {
                        const int p = kParts - 1 - x;
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            tc_mma_ts(tmem + kTO, tmem + kTSp + 64 * p + 8 * ks,
                                      tc_desc_advance(q, (ks >> 2) * kHalf + (ks & 3) * 32), id_o,
                                      !strong || x > 0 || ks > 0);
                    }
                    tc_commit(&sm.o_full);
                    tc_commit(&sm.q_free[st]);
                }
                __syncwarp();
            }
            if (ok && chunks > 0)
                ok = mbar_wait(&sm.q_free[(chunks - 1) % kStages],
                               (uint32_t)(((chunks - 1) / kStages) & 1), a.err);
        } else {
            for (int c = 0; c < chunks; ++c) {
                const uint64_t pp = tc_desc_advance(d0, kPAt);
                const uint32_t vt = tmem + kTVt + kVtCols * (c & 1), par = (uint32_t)(c & 1);
                // (v's last quarter comes from a warp without a share of P)
                ok = mbar_wait(&sm.p_full, par, a.err) &&
                     mbar_wait(&sm.kd_full[c & 1], (uint32_t)((c >> 1) & 1), a.err) &&
                     (c == 0 || mbar_wait(&sm.o_free, par ^ 1u, a.err));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll 1
                    for (int x = 0; x < kParts; ++x) {
                        const int p = kParts - 1 - x;
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            tc_mma_ts(tmem + kTO, vt + 8 * ks,
                                      tc_desc_advance(pp, p * kHalf + 32 * ks), id_o, x > 0 || ks > 0);
                    }
                    tc_commit(&sm.oa_full[c & 1]);
                    tc_commit(&sm.kd_free[c & 1]);
                }
                __syncwarp();
            }
            if (ok && chunks > 0)
                ok = mbar_wait(&sm.kd_free[(chunks - 1) & 1], (uint32_t)(((chunks - 1) >> 1) & 1), a.err);
        }
        if (!ok) {                               // a wait gave up: whatever still runs ends first
            if (elect_one()) tc_commit(&sm.drain[warp]);
            __syncwarp();
            mbar_wait(&sm.drain[warp], 0, nullptr);
        }
    } else if (warp >= kConvWarp0) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConvRegs));
        // ---- k into Kd, q k into P -----------------------------------------------------------
        const int quarter = (warp - kConvWarp0) & 3, r = lane & 7;
        const int prow = 32 * (quarter != 0) + lane;                  // token t of P
        const int pcol = 32 * (quarter == 3);                         // the first of its 32 tokens s
        const int last = prow - pcol;                                 // the last of them that t sees
        const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t b0 = __shfl_sync(0xffffffffu, smem_u32(base), 0);
        for (int c = (warp - kConvWarp0) / kGroupWarps; c < chunks; c += 2) {
            const int st = c % kStages, bkv = c % kBars;
            const uint32_t pc = (uint32_t)((c >> 1) & 1);
            const int nt = min(kC, len - c * kC);
            const uint32_t stage = b0 + st * kKvBytes, kd = b0 + kKdAt + (c & 1) * kKdBytes;
            // (in this order: the MMAs of chunk c - 2, and with them those of c - 3, are done, so that the barrier of
            // the loads is not a phase behind)
            ok = (c >= 2 ? mbar_wait(&sm.kd_free[c & 1], pc ^ 1u, a.err)
                         : !starts || mbar_wait(&sm.st_free, 0, a.err)) &&
                 mbar_wait(&sm.kv_full[bkv], (uint32_t)((c / kBars) & 1), a.err);
            if (!ok) break;
            // v^T: values of this warp's lane quarter, 16 and 16, tokens 0 .. 31 and 32 ..
            const auto v_words = [&](uint32_t (&w)[8], int h) {
                const int half = (h >> 1) & 1;
                const int jc = 4 * quarter + 2 * (h & 1) + ((lane >> 3) & 1);     // 16-byte piece of the row
                const int vs = 32 * half + 8 * (lane >> 4) + r;                   // + 16 for the second pair
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    ldsm4_t(*reinterpret_cast<uint32_t(*)[4]>(w + 4 * q),
                            stage + kVAt + (jc >> 3) * kHalf + (vs + 16 * q) * 128 +
                                (((jc ^ vs) & 7) * 16));
                if (nt < kC)      // rows past the sequence's end are another's: 0 times a NaN there is not 0
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int t = 32 * half + 8 * (i >> 1) + 2 * (lane & 3);
                        w[i] = t >= nt ? 0u : t + 1 >= nt ? w[i] & 0xffffu : w[i];
                    }
            };
            const auto v_store = [&](const uint32_t (&w)[8], int h) {
                tmem_st_16x128b_x4(tl + ((uint32_t)(16 * (h & 1)) << 16) + kTVt + kVtCols * (c & 1) +
                                       16 * ((h >> 1) & 1), w);
            };
            const __nv_bfloat162 zero2 = __floats2bfloat162_rn(0.0f, 0.0f);
            __nv_bfloat162 odd[2] = {zero2, zero2};          // 0 times v, summed: 0 unless one is no number
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {
                uint32_t w[8];
                v_words(w, h);
                v_store(w, h);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    odd[i & 1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(w + i), zero2, odd[i & 1]);
            }
            const uint32_t odd_bits =
                *reinterpret_cast<const uint32_t*>(odd) | *reinterpret_cast<const uint32_t*>(odd + 1);
            if (__any_sync(0xffffffffu, (odd_bits & 0x7fff7fffu) != 0)) {
#pragma unroll 1
                for (int h = 0; h < 4; ++h) {
                    uint32_t w[8];
                    v_words(w, h);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        int* bad = &sm.bad[32 * quarter + 16 * (h & 1) + 8 * (i & 1) + (lane >> 2)];
                        const int t = c * kC + 32 * ((h >> 1) & 1) + 8 * (i >> 1) + 2 * (lane & 3);
                        if ((w[i] & 0x7f800000u) == 0x7f800000u) { w[i] &= 0xffffu; atomicMin(bad, t + 1); }
                        if ((w[i] & 0x7f80u) == 0x7f80u) { w[i] &= 0xffff0000u; atomicMin(bad, t); }
                    }
                    v_store(w, h);
                }
            }
            // Kd: tokens 16 quarter .., 8 and 8, transposed to [key][token]
            const auto k_words = [&](uint32_t (&w)[4], int h, int q) {
                const int ic = 4 * q + (lane >> 3);                               // 16-byte piece of k's row
                ldsm4_t(w, stage + (ic >> 3) * kHalf + (16 * quarter + 8 * h + r) * 128 +
                               (((ic ^ r) & 7) * 16));
            };
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int sb = 2 * quarter + h, t = 8 * sb + 2 * (lane & 3);
                const float2 d = make_float2(sm.pw[mid + max(nt - 1 - t, 0)], sm.pw[mid + max(nt - 2 - t, 0)]);
                const uint32_t live = t + 1 < nt ? 0xffffffffu : t < nt ? 0xffffu : 0u;
                uint32_t kw[4][4];
#pragma unroll
                for (int q = 0; q < 4; ++q) k_words(kw[q], h, q);
                if (h == 1) warp_arrive(&sm.kv_free[bkv]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int ic = 4 * q + (lane >> 3);
                    uint32_t o[4][kParts];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t w = kw[q][i] & live;
                        const float2 x = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
                        split(__fmul2_rn(x, d), o[i]);
                    }
#pragma unroll
                    for (int p = 0; p < kParts; ++p)
                        stsm4(kd + p * kTileBytes + (8 * ic + r) * 128 + ((sb ^ r) * 16),
                              {o[0][p], o[1][p], o[2][p], o[3][p]});
                }
            }
            tmem_st_wait();
            tc_fence_before();
            fence_proxy_async_smem();
            warp_arrive(&sm.kd_full[c & 1]);
            if (STATE || quarter == 2) continue;
            ok = mbar_wait(&sm.sc_full[c & 1], pc, a.err);
            if (!ok) break;
            tc_fence_after();
            if (c > 0) ok = mbar_wait(&sm.oa_full[(c & 1) ^ 1], (uint32_t)(((c - 1) >> 1) & 1), a.err);
            if (!ok) break;
#pragma unroll 1
            for (int b = 0; b < 32; b += 16) {
                float x[16];
                tmem_ld16(tl + kTSc + pcol + b, x);
                tmem_ld_wait();
                if (strong)
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] *= sm.pw[max(last - b - i, 0)];
                uint32_t o[8][kParts];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 f = *reinterpret_cast<const float2*>(sm.down + pcol + b + 2 * i);
                    float2 y = __fmul2_rn(make_float2(x[2 * i], x[2 * i + 1]), f);
                    // (where s > t not 0 times q k: it is what it is for tokens to come, and another sequence's
                    // behind the end)
                    y.x = quarter == 1 || b + 2 * i <= last ? y.x : 0.0f;
                    y.y = quarter == 1 || b + 2 * i + 1 <= last ? y.y : 0.0f;
                    split(y, o[i]);
                }
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int p = 0; p < kParts; ++p)
                        *reinterpret_cast<uint4*>(base + kPAt + p * kHalf + prow * 128 +
                                                  ((((pcol + b) / 8 + q) ^ (prow & 7)) * 16)) =
                            make_uint4(o[4 * q][p], o[4 * q + 1][p], o[4 * q + 2][p], o[4 * q + 3][p]);
            }
            tc_fence_before();
            warp_arrive(&sm.sc_free);
            fence_proxy_async_smem();
            warp_arrive(&sm.p_full);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStateRegs));
        // ---- the state and o -----------------------------------------------------------------
        // value row j; keys 32 part .. of its state, tokens 16 part .. of its outputs
        const int j = 32 * (warp & 3) + lane, part = (warp - kStateWarp0) >> 2;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        float2 S[16];                            // times e^{mid g}
        unsigned char* const tile = base + kKdAt + part * kStTile + j * 128;
        if (starts) {
            ok = mbar_wait(&sm.st_full, 0, a.err);
            const float in = chunks > 0 ? sm.pw[mid] : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 x = *reinterpret_cast<const float4*>(tile + ((i ^ (j & 7)) * 16));
                S[2 * i] = make_float2(x.x * in, x.y * in);
                S[2 * i + 1] = make_float2(x.z * in, x.w * in);
            }
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
                    y = __ffma2_rn(fa2, y, __ffma2_rn(fd2, y, make_float2(u[2 * i], u[2 * i + 1])));
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
            uint32_t at = (uint32_t)j * 4;
            if (live >= 16 && !strong) {
#pragma unroll
                for (int t = 0; t < 16; ++t, at += step4)
                    __stcs(reinterpret_cast<float*>(reinterpret_cast<char*>(o) + at), x[t]);
            } else {
#pragma unroll
                for (int t = 0; t < 16; ++t, at += step4)
                    if (t < live) {
                        float* ob = reinterpret_cast<float*>(reinterpret_cast<char*>(o) + at);
                        *ob = strong ? *ob + x[t] : x[t];
                    }
            }
        }
        if (ok && (STATE || ends)) {
            const float out = chunks > 0 ? 1.0f / sm.pw[mid] : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float4*>(tile + ((i ^ (j & 7)) * 16)) =
                    make_float4(S[2 * i].x * out, S[2 * i].y * out, S[2 * i + 1].x * out, S[2 * i + 1].y * out);
            fence_proxy_async_smem();
            warp_arrive(&sm.st_out[part]);       // one of the tile's four warps
            if ((warp & 3) == 0 && mbar_wait(&sm.st_out[part], 0, a.err) && elect_one()) {
                const long st = STATE ? piece_state(cut, n, seg, units) : (long)n * units;
                tma_store_2d(&maps.out, base + kKdAt + part * kStTile, 32 * part, (int)(st + unit) * kHeadDim);
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

// The contributions of a sequence's pieces into the states after them, in place; a thread owns four elements
// of a unit's state.
constexpr int kJoinThr = 256;
constexpr int kJoinAhead = 4;

__global__ void __launch_bounds__(kJoinThr) kda_linattn_join_kernel(const LinArgs a, const Cut cut) {
    constexpr int kPieces = kHeadDim * kHeadDim / 4;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int units = a.H * a.m, n = blockIdx.y;
    const long piece = (long)blockIdx.x * kJoinThr + threadIdx.x;     // kPieces is a multiple of kJoinThr
    const int unit = (int)(piece / kPieces);
    const int len = a.seq.cu_seqlens ? a.seq.cu_seqlens[n + 1] - a.seq.cu_seqlens[n] : a.seq.T_uniform;
    const int seg_len = cut.seg_chunks * kC;
    // (the last segment's are not formed)
    const int parts = min(((len + seg_len - 1) / seg_len - 1) * cut.subs, cut.pieces());
    if (parts <= 0) return;
    const float2 f = decay_pair(a.log_decay[unit / a.m] * (float)(seg_len / cut.subs));
    const long stride = (long)units * kPieces;
    float4* at = reinterpret_cast<float4*>(cut.parts) + piece_state(cut, n, 0, units) * kPieces + piece;
    float4 S = a.state_in ? __ldg(reinterpret_cast<const float4*>(a.state_in) + (long)n * stride + piece)
                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int p = 0; p < parts; p += kJoinAhead) {
        float4 u[kJoinAhead];
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i)
            if (p + i < parts) u[i] = at[(p + i) * stride];
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i)
            if (p + i < parts) {
                S.x = fmaf(f.x, S.x, fmaf(f.y, S.x, u[i].x));
                S.y = fmaf(f.x, S.y, fmaf(f.y, S.y, u[i].y));
                S.z = fmaf(f.x, S.z, fmaf(f.y, S.z, u[i].z));
                S.w = fmaf(f.x, S.w, fmaf(f.y, S.w, u[i].w));
                at[(p + i) * stride] = S;
            }
    }
}

// Segments of a call and their pieces, by the time of their waves of CTAs in us: a chunk of the main kernel 2.3 (f32:
// 3.9), of the state kernel 1.1 (f32: 1.5), a CTA's start and end 6, the two further launches 4.5.  (bf16, 4096 tokens
// x 64 heads: whole 145 us, 2 segments of 2 pieces 113; 8192 x 8 heads: whole 272, 19 segments 47.)
constexpr int kMaxSegs = 32;
long most_segs(long chains, long chunks, int sms) {
    return std::max(1L, std::min({(long)kMaxSegs, chunks, 4L * sms / std::max(1L, chains)}));
}

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

long seq_chunks(const SeqLayout& s, const int* cu_host, int n) {
    const long len = cu_host ? cu_host[n + 1] - cu_host[n] : s.T_uniform;
    return (len + kC - 1) / kC;
}

// Chains of (sequence, unit) that are cut at all: with two on each SM they fill it.
bool may_cut(long chains, int sms) { return chains < 2L * sms; }

Cut plan(const SeqLayout& s, const int* cu_host, int units, bool bf16) {
    const double main_us = bf16 ? 2.3 : 3.9, state_us = bf16 ? 1.1 : 1.5, ends_us = 6.0, launches_us = 4.5;
    const int sms = sm_count();
    long most = 1;
    for (int n = 0; n < s.N; ++n) most = std::max(most, seq_chunks(s, cu_host, n));
    Cut best{(int)most, 1, 1, nullptr};
    if (!may_cut((long)s.N * units, sms)) return best;
    double least = 0.0;
    const long limit = most_segs((long)s.N * units, most, sms);
    for (long segs = 1; segs <= limit; ++segs)
        for (long subs = 1; segs * subs <= limit && (segs > 1 || subs == 1); ++subs) {
            const long per = ((most + segs - 1) / segs + subs - 1) / subs * subs;
            if (segs > 1 && (most + per - 1) / per != segs) continue;
            long blocks = 0, cut_seqs = 0;
            for (int n = 0; n < s.N; ++n) {
                const long k = (seq_chunks(s, cu_host, n) + per - 1) / per;
                blocks += k;
                cut_seqs += k > 0;
            }
            const auto waves = [&](long b) { return (double)((b * units + sms - 1) / sms); };
            const double cost = waves(blocks) * (per * main_us + ends_us) +
                                (segs > 1 ? waves((blocks - cut_seqs) * subs) * (per / subs * state_us + ends_us) +
                                                launches_us : 0.0);
            if (segs > 1 && cost >= least) continue;
            least = cost;
            best = Cut{(int)per, (int)segs, (int)subs, nullptr};
        }
    return best;
}

template <bool STATE>
cudaError_t launch(const LinArgs& a, const Cut& cut, const Maps& maps, bool after, cudaStream_t s) {
    static PerDevice<int> done;
    const cudaError_t e = set_smem(kda_linattn_chunk_kernel<STATE>, kSmemBytes, done);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.H * a.m), (unsigned)a.seq.N, (unsigned)(STATE ? cut.pieces() : cut.segs));
    return launch_as(STATE ? kKLinState : kKLinChunk, after, kda_linattn_chunk_kernel<STATE>, grid, kThr, kSmemBytes, s,
                     a, cut, maps);
}

size_t states_bytes(long states) { return (size_t)states * kHeadDim * kHeadDim * sizeof(float); }

}  // namespace

cudaError_t linattn::launch_join(const LinArgs& a, const Cut& cut, cudaStream_t s) {
    const unsigned blocks = (unsigned)((long)a.H * a.m * kHeadDim * kHeadDim / 4 / kJoinThr);
    return launch_as(kKLinJoin, true, kda_linattn_join_kernel, dim3(blocks, (unsigned)a.seq.N), kJoinThr, 0, s, a, cut);
}

// The workspace: parts of q and k (f32), then the segments' states.
size_t linattn_chunk_workspace_bytes(const SeqLayout& seq, const int* cu_host, int Hk, int units, bool bf16) {
    return (bf16 ? 0 : f32_split_bytes(seq.total_rows, Hk)) +
           states_bytes((long)seq.N * plan(seq, cu_host, units, bf16).pieces() * units);
}

// (more than any cut of total_T tokens into N sequences takes: the cut of the longest possible one; for f32 4 bytes an
// element of q, k and v, which the 6 of q and k never pass)
size_t linattn_chunk_workspace_bound(int N, long total_T, int Hk, int units, bool bf16) {
    const int sms = sm_count();
    const long chains = (long)N * units;
    const size_t split = bf16 ? 0 : (size_t)total_T * (2L * Hk + units) * kHeadDim * 4;
    if (!may_cut(chains, sms)) return split;
    return split + states_bytes(chains * (most_segs(chains, (total_T + kC - 1) / kC, sms) - 1));
}

cudaError_t launch_linattn_chunk(const LinArgs& a, const int* cu_host, void* workspace, cudaStream_t s) {
    const int units = a.H * a.m;
    const long rows = a.seq.total_rows, qk = (long)a.Hk * kHeadDim, vw = (long)units * kHeadDim;
    Cut cut = plan(a.seq, cu_host, units, a.bf16);
    cut.parts = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) +
                                         (a.bf16 ? 0 : f32_split_bytes(rows, a.Hk)));
    StateMaps states;
    std::memset(&states, 0, sizeof(states));
    const auto rows_of = [&](CUtensorMap* m, const float* base, long seqs) {
        return make_tensor_map_2d_f32_sw128(m, base, seqs * units * kHeadDim, kHeadDim, kHeadDim);
    };
    if ((a.state_in != nullptr && !rows_of(&states.in, a.state_in, a.seq.N)) ||
        !rows_of(&states.out, a.state_out, a.seq.N) ||
        (cut.segs > 1 && !rows_of(&states.parts, cut.parts, (long)a.seq.N * cut.pieces())))
        return cudaErrorInvalidValue;
    if (!a.bf16) return launch_chunks_f32(a, cut, states, workspace, s);
    Maps maps;
    if (!make_tensor_map_2d_bf16_sw128(&maps.q, a.q, rows, qk, kC, a.q_stride) ||
        !make_tensor_map_2d_bf16_sw128(&maps.k, a.k, rows, qk, kC, a.k_stride) ||
        !make_tensor_map_2d_bf16_sw128(&maps.v, a.v, rows, vw, kC, a.v_stride))
        return cudaErrorInvalidValue;
    maps.in = states.in;
    maps.parts = maps.out = states.parts;
    if (cut.segs > 1) {
        cudaError_t e = launch<true>(a, cut, maps, false, s);
        if (e == cudaSuccess) e = launch_join(a, cut, s);
        if (e != cudaSuccess) return e;
    }
    maps.out = states.out;
    return launch<false>(a, cut, maps, cut.segs > 1, s);
}

}  // namespace kda
