// kda_linattn_chunk.cuh -- what the chunked forms of linear attention for bf16 (kda_linattn_chunk.cu) and f32
// (kda_linattn_chunk_f32.cu) share: the tiles, the warps' roles, waits, the cut of long sequences into segments.
#pragma once

#include "kda_tc.cuh"

namespace kda {

namespace linattn {

constexpr int kC = 64;                           // tokens of a chunk
constexpr int kMid = kC / 2;
constexpr int kHalf = kC * 128;                  // bytes of 64 tokens x 64 columns, 128-byte swizzle
constexpr int kTileBytes = 2 * kHalf;            // 64 tokens x 128 columns
constexpr int kStTile = kHeadDim * 128;          // 128 state rows x 32 keys, f32
constexpr int kParts = 3;                        // bf16 parts of what is f32: 24 bits

constexpr int kStateWarps = 16, kConvWarps = 8;
// The first warpgroup issues the MMAs and the loads; whole warpgroups: registers move between them.
constexpr int kUWarp = 0, kOiWarp = 1, kTmaWarp = 3, kStateWarp0 = 4;
constexpr int kConvWarp0 = kStateWarp0 + kStateWarps;
constexpr int kThr = 32 * (kConvWarp0 + kConvWarps);
constexpr int kGroupWarps = 4;                   // converting warps that cover the TMEM lanes
constexpr int kLaunchRegs = 72, kOtherRegs = 24;
// registers of a state warp's and a converting warp's threads: what the launch has
constexpr bool regs_fit(int state, int conv) {
    return 32 * (kStateWarps * state + kConvWarps * conv + 4 * kOtherRegs) <= kThr * kLaunchRegs;
}

constexpr int kMaxRanked = 32;                   // packed sequences that are taken longest first

// Two f32 as bf16x2 words, each the rest of those before it rounded.
__device__ __forceinline__ void split(float2 x, uint32_t (&w)[kParts]) {
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
        w[p] = *reinterpret_cast<const uint32_t*>(&h);
        if (p + 1 < kParts) x = __ffma2_rn(make_float2(__uint_as_float(w[p] << 16), __uint_as_float(w[p] & 0xffff0000u)),
                           make_float2(-1.0f, -1.0f), x);
    }
}

// mbar_wait_bounded for two dozen warps that wait most of the time: the suspended wait is left to the
// hardware (polling took issue slots from the warps that work), and a clock bounds it.
__device__ __forceinline__ bool mbar_wait_long(uint64_t* bar, uint32_t parity, int* err) {
    unsigned long long t0;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
            : "memory");
        if (done) return true;
        unsigned long long t;
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
        if (t - t0 > 1000000000ull) break;
    }
    if (err) atomicOr(err, kDevErrTimeout);
    return false;
}
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, int* err) {
    return mbar_try_wait(bar, parity) || mbar_wait_long(bar, parity, err);
}

__device__ __forceinline__ void tma_prefetch_2d(const void* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A warp's arrival: its lanes' TMEM and shared memory accesses before it are done.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Four 8 x 8 blocks of bf16 to shared memory, 8 lanes giving the addresses of a block's rows: lane l has elements
// (l / 4, 2 (l % 4)) and the one behind of each.
__device__ __forceinline__ void stsm4(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

// How the sequences are cut: segments of seg_chunks chunks, at most segs of one sequence, each in subs pieces for the
// STATE launch; parts: [N][(segs - 1) subs][units][128][128] f32, first the pieces' contributions to the state, then
// the states after them.
struct Cut {
    int seg_chunks, segs, subs;
    float* parts;
    __host__ __device__ int pieces() const { return (segs - 1) * subs; }
};

// the first unit's state of a piece among the parts
__device__ __forceinline__ long piece_state(const Cut& cut, int n, int piece, int units) {
    return ((long)n * cut.pieces() + piece) * units;
}

// a + b is e^x: a step S <- e^x S + U is S <- a S + (b S + U).  Above a half a = 1 and b = e^x - 1, which
// keeps a decay next to 1: rounded itself, e^x would be off by up to 2^-25 at every step.
__device__ __forceinline__ float2 decay_pair(float x) {
    const float lam = expf(x);
    return lam > 0.5f ? make_float2(1.0f, expm1f(x)) : make_float2(lam, 0.0f);
}

// What a CTA works on: segment blockIdx.z (with STATE: a piece of one) of the blockIdx.y-th sequence, packed ones
// in the order of their lengths; len < 0: nothing.  By whole warps.
struct Part {
    long begin;                                  // its first token's row
    int n, len;
    bool ends;                                   // the sequence ends with it
};
template <bool STATE>
__device__ __forceinline__ Part locate(const SeqLayout& seq, const Cut& cut, int lane) {
    const int seg = blockIdx.z;
    Part p;
    p.n = blockIdx.y;
    int len;
    if (seq.cu_seqlens != nullptr) {
        const int* cu = seq.cu_seqlens;
        if (seq.N <= kMaxRanked) {               // the longest sequences first
            const int mine = lane < seq.N ? cu[lane + 1] - cu[lane] : -1;
            int rank = 0;
            for (int k = 0; k < seq.N; ++k) {
                const int other = __shfl_sync(0xffffffffu, mine, k);
                rank += other > mine || (other == mine && k < lane);
            }
            p.n = __ffs(__ballot_sync(0xffffffffu, lane < seq.N && rank == p.n)) - 1;
        }
        p.begin = __shfl_sync(0xffffffffu, cu[p.n], 0);
        len = __shfl_sync(0xffffffffu, cu[p.n + 1], 0) - (int)p.begin;
    } else {
        p.begin = (long)p.n * seq.T_uniform;
        len = seq.T_uniform;
    }
    const int whole_len = cut.seg_chunks * kC, seg_len = STATE ? whole_len / cut.subs : whole_len;
    p.ends = (seg + 1) * (long)seg_len >= len;
    p.begin += (long)seg * seg_len;
    // (with STATE a piece whose segment nothing follows has no use)
    const bool none = (seg > 0 && seg * (long)seg_len >= len) ||
                      (STATE && (seg / cut.subs + 1) * (long)whole_len >= len);
    p.len = none ? -1 : min(len - seg * seg_len, seg_len);
    return p;
}

// `after`: as the programmatic dependent of the launch before, a launch of this file that it waits for itself.
template <typename... P, typename... A>
cudaError_t launch_as(int id, bool after, void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t s,
                      const A&... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = after ? 1 : 0;
    KernelTimer kt(id, s);
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Tensor maps of the states as rows of 128 keys, one a value: state_in, the parts, state_out.
struct StateMaps {
    CUtensorMap in, parts, out;
};
// The pieces' contributions into the states after them (kda_linattn_chunk.cu).
cudaError_t launch_join(const LinArgs& a, const Cut& cut, cudaStream_t s);
// The launches for f32 (kda_linattn_chunk_f32.cu); the workspace's first f32_split_bytes are theirs.
size_t f32_split_bytes(long rows, int Hk);
cudaError_t launch_chunks_f32(const LinArgs& a, const Cut& cut, const StateMaps& states, void* workspace,
                              cudaStream_t s);

}  // namespace linattn
}  // namespace kda
