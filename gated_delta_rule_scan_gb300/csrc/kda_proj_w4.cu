// kda_proj_w4.cu -- projections of t token rows by weights of 4 bits with group scales:
//
//     out_i[s][r] = sum_k (q_i[r][k] - z_i[r][k / G]) * c_i[r][k / G] * x[s][k]
//
// for up to 8 weights that read one x.  q is a 4-bit code (two to a byte, the even k in the low
// nibble), c the scale and z the zero point of G consecutive k (z = 8 without zero points).
//
// Mathematics.  Codes become f16 integers and the products run on the tensor cores with them: no
// weight is ever rounded.  The zero point comes off each group's f32 sum, which the scale then
// multiplies:
//     out = sum over groups of c (sum_k q x - z / 8 sum_k 8 x).
// x is scaled over 128 k at a time by the power of two that brings the largest magnitude of the 128
// to [2^14, 2^15), split into f16 hi + lo, and the power of two goes back in with the group's scale.
// hi is a whole number, so that sum_k q hi and sum_k 8 hi are exact in f32, and so is their
// difference, as long as they stay below 2^24: 128 elements of a quarter of the largest's magnitude,
// all of one sign, still do; larger sums are rounded as any f32 sum.  Subtracting after the sum
// then loses nothing, and a code needs no more than a logical operation to become a number (taking 8
// off each code first: 22.8 us against 19.1 at one row x 6144, 64 heads).  hi + lo is x within 2^-23
// of the element's own magnitude or 2^-27 of the largest of the 128, whichever is more.
//     5 rows or more of a bf16 x take hi alone, for half the MMA's columns: its 8 bits are exact down to
// 2^-31 of the largest of the 128, and smaller elements are off by at most 2^-39 of it.  Its sums are
// rounded, so there the codes have 8 taken off first.
//
// The form for few rows: up to 16, by the rule at its launch.  The weights' bytes are read once and bound the
// launch, so the kernel is built around their stream: a warp takes 16 weight rows x 128 k (1 KB of
// codes, wide loads straight into registers, the next 1 KB asked for before the present one is used;
// two ahead: 19.1 us against 17.7), and turns them into mma.sync m16n8k16 operands.  The order of k
// inside an MMA is free as long as both operands agree, so x is laid out in shared memory once per
// block in the order in which the nibbles of a word come out, and one 16-byte shared load feeds two
// MMAs.
// The MMA's 8 columns carry hi and lo of 4 tokens, or hi of 8; up to four such tiles go over one
// fetch of the codes.
// One block per SM holds x for up to three teams of 8 warps (three blocks staged it three times: 32
// us against 25 at four rows, before the codes' centring went).  Each team takes tiles of 16 rows in
// turn; its warps split K, and their partial sums meet in shared memory in warp order.  Where x of
// all of K does not fit, the CTAs of a cluster split K further and add their sums through
// distributed shared memory in rank order.  No atomics: results do not depend on timing.
// At 64 heads x 6144 and groups of 128: one row 17.9 to 20.3 us from machine to machine (4.4 to 3.9 TB/s of
// codes and scales: the shared loads, MMAs and logical operations of a chunk cost about half its bytes'
// time again), four rows 20.7 to 22.6, eight bf16 rows 25.0 to 25.8, five f32 rows 28.
#include <cuda_fp16.h>

#include "kda_device.cuh"
#include "kda_tc.cuh"

namespace kda {

namespace {

constexpr int kWarps = 8;                    // warps of a team: they split K of a tile
constexpr int kTeam = kWarps * 32;
constexpr int kRows = 16;                    // weight rows of a tile: the MMA's M
constexpr int kChunk = 128;                  // k of one warp step
// Tokens that NT MMA tiles of 8 columns hold.
template <bool ONE, int NT>
constexpr int kTok = (ONE ? 8 : 4) * NT;
constexpr float kMagic = 12582912.0f;        // 1.5 * 2^23
constexpr int kXSmem = 152 * 1024;           // x of one block at most

struct W4Params {
    const void* x;
    const uint8_t* w[kW4MaxWeights];
    const void* scale[kW4MaxWeights];
    const void* zero[kW4MaxWeights];
    float* out[kW4MaxWeights];
    int rows[kW4MaxWeights];
    int tile_start[kW4MaxWeights + 1];
    int nw, t, in_f, x_bf16, scale_bf16, has_zero, ksplit;
};

// Bytes of the block's shared memory for `chunks` chunks of k and `cols` MMA columns.
struct W4Smem {
    int x, factor, eights, red, total;
};
__host__ __device__ inline W4Smem w4_smem(int chunks, int cols, int group, int teams, int tok, int nt) {
    W4Smem m;
    m.x = 0;                                                   // f16 [chunk][4][cols][4][8]
    m.factor = chunks * kChunk * cols * 2;                     // f32 [chunk][tok]
    m.eights = m.factor + chunks * tok * 4;                    // f32 [group][8 nt columns]
    m.red = m.eights + chunks * (kChunk / group) * 8 * nt * 4; // f32 [teams][2][warps][tok][16]
    m.total = m.red + teams * (2 * kWarps * tok * kRows * 4);
    return m;
}

// Nibbles 0 and 4 (lo) or 1 and 5 (hi) of a word as f16 pairs.  Alone in its place of the mantissa,
// with no exponent, a code q is the f16 number q 2^-24 or 16 q 2^-24.  CENTRED: q - 8, from 1024 + q
// and 1024 + 16 q (the code or-ed into the mantissa of 1024: Kim, Henry, Fahim and Awadalla, "Who Says
// Elephants Can't Run", 2022); both corrections are exact.
template <bool CENTRED>
__device__ __forceinline__ uint32_t nib_lo(uint32_t w) {
    if constexpr (!CENTRED) return w & 0x000f000fu;
    const uint32_t v = (w & 0x000f000fu) | 0x64006400u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(1032.0f));
    return *reinterpret_cast<const uint32_t*>(&r);
}
template <bool CENTRED>
__device__ __forceinline__ uint32_t nib_hi(uint32_t w) {
    if constexpr (!CENTRED) return w & 0x00f000f0u;
    const uint32_t v = (w & 0x00f000f0u) | 0x64006400u;
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(0.0625f),
                              __float2half2_rn(-72.0f));
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 4, 8 or 16 bytes (G / 8) of streamed weights into the words w[0 ..].
template <int BYTES>
__device__ __forceinline__ void load_words(uint32_t* w, const uint8_t* p) {
    if constexpr (BYTES == 16) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (BYTES == 8) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
        w[0] = v.x; w[1] = v.y;
    } else {
        w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
    }
}

// N = 1, 2 or 4 consecutive scales or zero points as they lie in memory; value() is the i-th.
template <int N, bool BF16>
struct W4Par {
    static constexpr int kWords = BF16 ? (N + 1) / 2 : N;
    uint32_t u[kWords];
    __device__ __forceinline__ void load(const void* p) {
        if constexpr (BF16 && N == 1) {
            u[0] = __ldg(reinterpret_cast<const unsigned short*>(p));
        } else if constexpr (kWords == 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
            u[0] = v.x; u[1] = v.y; u[2] = v.z; u[3] = v.w;
        } else if constexpr (kWords == 2) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
            u[0] = v.x; u[1] = v.y;
        } else {
            u[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
        }
    }
    __device__ __forceinline__ float value(int i) const {
        if constexpr (BF16) return __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
        else return __uint_as_float(u[i]);
    }
};

// Codes, scales and zero points of 16 rows x 128 k as one warp holds them: lane 4g + c has, of rows
// g and g + 8 and of each group, the c-th quarter's codes.  (Groups of 32 are loaded two at a time,
// 8 bytes a lane, and sorted by a shuffle when used: 28.4 us against 31.9 with 4-byte loads.)
template <int G, bool SBF16, bool ZERO>
struct W4Frag {
    uint32_t w[2][4];
    W4Par<kChunk / G, SBF16> c[2];
    W4Par<kChunk / G, SBF16> z[ZERO ? 2 : 1];
};

// The chunks of one warp in the order of their use: its share of K for each of its block's tiles.
template <int G, bool SBF16, bool ZERO>
struct W4Stream {
    const uint8_t* w[2];                         // rows g and g + 8 at the next chunk
    const uint8_t* c[2];
    const uint8_t* z[ZERO ? 2 : 1];
    int tile, left;                              // its tile, its chunks left

    __device__ __forceinline__ void open(const W4Params& p, int chunk, int chunks, int lane) {
        constexpr int kSize = SBF16 ? 2 : 4;
        int wi = 0;
        while (wi + 1 < p.nw && tile >= p.tile_start[wi + 1]) ++wi;
        const int row0 = (tile - p.tile_start[wi]) * kRows + (lane >> 2);
        left = chunks;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // rows past the weight repeat its last one; their sums are not written
            const long row = min(row0 + 8 * i, p.rows[wi] - 1);
            const long par = (row * (p.in_f / G) + chunk * (kChunk / G)) * kSize;
            w[i] = p.w[wi] + row * (p.in_f / 2) + chunk * (kChunk / 2) + (lane & 3) * (G == 32 ? 8 : G / 8);
            c[i] = static_cast<const uint8_t*>(p.scale[wi]) + par;
            if constexpr (ZERO) z[i] = static_cast<const uint8_t*>(p.zero[wi]) + par;
        }
    }
    __device__ __forceinline__ void fetch(W4Frag<G, SBF16, ZERO>& f) {
        constexpr int kStep = kChunk / G * (SBF16 ? 2 : 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (G == 32) {
#pragma unroll
                for (int q = 0; q < 2; ++q) load_words<8>(&f.w[i][q * 2], w[i] + q * 32);
            } else {
#pragma unroll
                for (int q = 0; q < kChunk / G; ++q)
                    load_words<G / 8>(&f.w[i][q * (G / 32)], w[i] + q * (G / 2));
            }
            f.c[i].load(c[i]);
            w[i] += kChunk / 2;
            c[i] += kStep;
            if constexpr (ZERO) {
                f.z[i].load(z[i]);
                z[i] += kStep;
            }
        }
    }
};

// Teams of a block, at most: three (four of 64 registers a thread are as fast: 17.7 us at one row x
// 6144 and 64 heads either way), but two where f32 scales and zero points of 32 k each need more
// registers (34 us against 36 at one row).
constexpr int w4_teams(int group, bool scale_bf16, bool zero, int nt) {
    return nt == 4 || (group == 32 && !scale_bf16 && zero) ? 2 : 3;
}

__device__ __forceinline__ void team_sync(int team) {
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(kTeam) : "memory");
}

// x of the block's chunks [ch0, ch0 + chunks): MMA operands and power-of-two factors.  A half warp
// takes one (chunk, token): lane u holds k = 8u .. 8u+7.
template <int G, bool ONE, int TOK>
__device__ __forceinline__ void stage_x(const W4Params& p, unsigned char* smem, const W4Smem& lay,
                                        int ch0, int chunks, int nt, int cols) {
    const int half = threadIdx.x >> 4, u = threadIdx.x & 15;
    float* factor = reinterpret_cast<float*>(smem + lay.factor);
    const int total = chunks * nt;
    for (int i0 = 0; i0 < total; i0 += blockDim.x / 16) {
        const int i = i0 + half;
        const bool live = i < total;
        const int ch = live ? i / nt : 0, tk = live ? i % nt : 0;
        float v[8];
        const long at = (long)tk * p.in_f + (long)(ch0 + ch) * kChunk + 8 * u;
        if (ONE || p.x_bf16) {
            const uint4 r = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.x) + at));
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        } else {
            const float4* x4 = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.x) + at);
            const float4 a = __ldg(x4), b = __ldg(x4 + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        // 2^(14 - e) for the largest magnitude's exponent e (at least -100); 1 when it is not finite
        const int e = max((int)(m >> 23) - 127, -100);
        const bool fin = m < 0x7f800000u;
        const float up = fin ? __uint_as_float((uint32_t)(127 + 14 - e) << 23) : 1.0f;
        if (!live) continue;
        __half hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float y = __fmul_rn(v[j], up);
            const int at8 = j < 4 ? 2 * j : 2 * (j - 4) + 1;     // nibble order (0 4 1 5 2 6 3 7)
            if constexpr (ONE) {
                hi[at8] = __float2half_rn(y);
            } else {
                // to a whole number (a step of f32 at 2^23), then to f16's 11 bits
                const float h = __half2float(__float2half_rn(__fsub_rn(__fadd_rn(y, kMagic), kMagic)));
                const float w = j & 1 ? 0.0625f : 1.0f;          // odd codes come times 16
                hi[at8] = __float2half_rn(h * w);
                lo[at8] = __float2half_rn(__fsub_rn(y, h) * w);
            }
        }
        // k = 8u is word jj of quarter c of its group
        const int k0 = 8 * u, q = k0 / G, c = (k0 % G) / (G / 4), jj = q * (G / 32) + (k0 % (G / 4)) / 8;
        uint4* xs = reinterpret_cast<uint4*>(smem + lay.x);
        // (G = 32: after the trade, lanes 1 and 2 hold words 2 and 1 of their group)
        const long base = (long)(ch * 4 + jj) * cols * 4 + (G == 32 ? (c >> 1) + 2 * (c & 1) : c);
        if constexpr (ONE) {
            xs[base + tk * 4] = *reinterpret_cast<const uint4*>(hi);
        } else {
            xs[base + (2 * tk) * 4] = *reinterpret_cast<const uint4*>(hi);
            xs[base + (2 * tk + 1) * 4] = *reinterpret_cast<const uint4*>(lo);
        }
        if (u == 0) factor[ch * TOK + tk] = fin ? __uint_as_float((uint32_t)(127 - 14 + e) << 23) : 1.0f;
    }
}

template <int G, bool ONE, bool SBF16, bool ZERO, int NT>
__global__ void __launch_bounds__(kTeam * w4_teams(G, SBF16, ZERO, NT)) kda_proj_w4_kernel(const __grid_constant__ W4Params p) {
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int TOK = kTok<ONE, NT>;
    const int team = threadIdx.x / kTeam, teams = blockDim.x / kTeam;
    const int warp = threadIdx.x % kTeam >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int rank = blockIdx.x % p.ksplit;
    const int blocks = gridDim.x / p.ksplit, stride = blocks * teams;
    const int first = team * blocks + blockIdx.x / p.ksplit;
    const int nt = p.t, cols = ONE ? nt : 2 * nt;
    const int all = p.in_f / kChunk;
    const int ch0 = all * rank / p.ksplit, ch1 = all * (rank + 1) / p.ksplit;
    const int chunks = ch1 - ch0;
    const W4Smem lay = w4_smem((all + p.ksplit - 1) / p.ksplit, cols, G, teams, TOK, NT);
    const int tiles = p.tile_start[p.nw];
    const float* factor = reinterpret_cast<const float*>(smem + lay.factor);
    float* eights = reinterpret_cast<float*>(smem + lay.eights);
    float* red = reinterpret_cast<float*>(smem + lay.red) + team * (2 * kWarps * TOK * kRows);

    const int w0 = chunks * warp / kWarps, w1 = chunks * (warp + 1) / kWarps;
    const int mine = w1 - w0;
    W4Stream<G, SBF16, ZERO> in;
    in.tile = first;
    if (mine > 0 && in.tile < tiles) in.open(p, ch0 + w0, mine, lane);
    const auto fetch = [&](W4Frag<G, SBF16, ZERO>& f) {
        if (mine == 0 || in.tile >= tiles) return;
        in.fetch(f);
        if (--in.left == 0) {
            in.tile += stride;
            if (in.tile < tiles) in.open(p, ch0 + w0, mine, lane);
        }
    };
    W4Frag<G, SBF16, ZERO> f0, f1;
    fetch(f0);
    stage_x<G, ONE, TOK>(p, smem, lay, ch0, chunks, nt, cols);
    __syncthreads();

    // Columns of the MMA past the batch repeat its last one: a column of the result depends on its
    // own column of x alone.
    const uint4* xs0 = reinterpret_cast<const uint4*>(smem + lay.x) + c;
    int col[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) col[i] = min(8 * i + g, cols - 1) * 4;
    // The sums of a group whose codes are all 8, by the very steps that sum the groups below: what
    // a zero point of 8 takes off.  A group that holds nothing but its zero point comes out as 0.
    for (int ch = !ONE || ZERO ? threadIdx.x >> 5 : chunks; ch < chunks; ch += blockDim.x >> 5) {
#pragma unroll
        for (int q = 0; q < kChunk / G; ++q) {
            float d[NT][4] = {};
#pragma unroll
            for (int j = q * (G / 32); j < (q + 1) * (G / 32); ++j) {
                const uint32_t lo = ONE ? 0x48004800u : nib_lo<false>(0x88888888u);      // 8 in f16
                const uint32_t hi = ONE ? 0x48004800u : nib_hi<false>(0x88888888u);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const uint4 b = xs0[(ch * 4 + j) * 4 * cols + col[i]];
                    mma_16816(d[i], lo, lo, hi, hi, b.x, b.y);
                    mma_16816(d[i], lo, lo, hi, hi, b.z, b.w);
                }
            }
            if (g == 0) {
                float* o = eights + (ch * (kChunk / G) + q) * (8 * NT) + 2 * c;
#pragma unroll
                for (int i = 0; i < NT; ++i) *reinterpret_cast<float2*>(o + 8 * i) = make_float2(d[i][0], d[i][1]);
            }
        }
    }
    __syncthreads();
    int buf = 0;
    // All teams of a cluster go through the same number of tiles, the last one past the end maybe.
    for (int tile = first; tile - team * blocks < tiles; tile += stride, buf ^= 1) {
        // acc[i][r][e]: token 4 i + c of row g + 8 r (e = 0), ONE: token 8 i + 2 c + e
        float acc[NT][2][2] = {};
        const uint4* xs = xs0 + w0 * 16 * cols;
        for (int ch = tile < tiles ? w0 : w1; ch < w1; ++ch, xs += 16 * cols) {
            fetch(f1);
            // groups of 32: the lane's 8 bytes are of one group; trade for a word of either
            if constexpr (G == 32) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int q = 0; q < 4; q += 2) {
                        uint32_t& a = f0.w[i][q];
                        uint32_t& b = f0.w[i][q + 1];
                        const bool up = c >= 2;
                        const uint32_t r = __shfl_xor_sync(0xffffffffu, up ? a : b, 2);
                        a = up ? r : a;
                        b = up ? b : r;
                    }
            }
#pragma unroll
            for (int q = 0; q < kChunk / G; ++q) {
                float d[NT][4] = {};
#pragma unroll
                for (int j = q * (G / 32); j < (q + 1) * (G / 32); ++j) {
                    const uint32_t u0 = f0.w[0][j], u1 = f0.w[1][j];
                    const uint32_t a0 = nib_lo<ONE>(u0), a1 = nib_lo<ONE>(u1), a2 = nib_hi<ONE>(u0), a3 = nib_hi<ONE>(u1);
                    const uint32_t a4 = nib_lo<ONE>(u0 >> 8), a5 = nib_lo<ONE>(u1 >> 8);
                    const uint32_t a6 = nib_hi<ONE>(u0 >> 8), a7 = nib_hi<ONE>(u1 >> 8);
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const uint4 b = xs[j * 4 * cols + col[i]];
                        mma_16816(d[i], a0, a1, a2, a3, b.x, b.y);
                        mma_16816(d[i], a4, a5, a6, a7, b.z, b.w);
                    }
                }
                const float* o = eights + (ch * (kChunk / G) + q) * (8 * NT) + 2 * c;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    float2 o2 = make_float2(0.0f, 0.0f);
                    if constexpr (!ONE || ZERO) o2 = *reinterpret_cast<const float2*>(o + 8 * i);
#pragma unroll
                    for (int e = 0; e < (ONE ? 2 : 1); ++e) {
                        const float f = factor[ch * TOK + (ONE ? 8 * i + 2 * c + e : 4 * i + c)];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            float v;
                            if constexpr (ONE) {
                                v = d[i][2 * r + e];
                                if constexpr (ZERO)
                                    v = fmaf(1.0f - 0.125f * f0.z[r].value(q), e ? o2.y : o2.x, v);
                            } else if constexpr (ZERO) {
                                // hi and lo apart: the difference of the hi sums is exact
                                const float z = -0.125f * f0.z[r].value(q);
                                v = fmaf(z, o2.x, d[i][2 * r]) + fmaf(z, o2.y, d[i][2 * r + 1]);
                            } else {
                                v = (d[i][2 * r] - o2.x) + (d[i][2 * r + 1] - o2.y);
                            }
                            acc[i][r][e] = fmaf(v * f, f0.c[r].value(q), acc[i][r][e]);
                        }
                    }
                }
            }
            f0 = f1;
        }
        // this tile's sums of all warps, in warp order
        float* rb = red + buf * (kWarps * TOK * kRows);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < (ONE ? 2 : 1); ++e)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    rb[(warp * TOK + (ONE ? 8 * i + 2 * c + e : 4 * i + c)) * kRows + g + 8 * r] =
                        ONE ? acc[i][r][e] : acc[i][r][e] * 16777216.0f;
        team_sync(team);
        int wi = 0;
        while (wi + 1 < p.nw && tile >= p.tile_start[wi + 1]) ++wi;
        const int tk = threadIdx.x % kTeam / kRows, r = threadIdx.x % kRows;
        const int row = (tile - p.tile_start[wi]) * kRows + r;
        float sum = 0.0f;
        if (tk < nt) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += rb[(w * TOK + tk) * kRows + r];
        }
        if (p.ksplit > 1) {
            // the cluster's CTAs: each leaves its sums where warp 0's were, then rank 0 adds them.
            // Its reads of this buffer end before any CTA passes the next tile's barrier and fills
            // the buffer after that one.
            team_sync(team);
            if (tk < nt) rb[tk * kRows + r] = sum;
            cluster_sync_all();
            if (rank == 0 && tk < nt) {
                sum = 0.0f;
                for (int k = 0; k < p.ksplit; ++k) sum += ld_cluster_f32(&rb[tk * kRows + r], (uint32_t)k);
            }
        }
        if (rank == 0 && tk < nt && tile < tiles && row < p.rows[wi])
            p.out[wi][(long)tk * p.rows[wi] + row] = sum;
    }
    if (p.ksplit > 1) cluster_sync_all();        // rank 0 has read the last tile's sums
}

template <int G, bool ONE, bool SBF16, bool ZERO, int NT>
cudaError_t launch_rows(const W4Params& p, int grid, int teams, size_t smem, cudaStream_t s) {
    const auto kernel = kda_proj_w4_kernel<G, ONE, SBF16, ZERO, NT>;
    static PerDevice<int> done;
    const cudaError_t e = set_smem(kernel, kMaxBlockSmem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)(teams * kTeam));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.ksplit;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.ksplit > 1 ? 1 : 0;
    KernelTimer kt(kKProjW4, s);
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int G, bool ONE, int NT>
cudaError_t launch_params(const W4Params& p, int grid, int teams, size_t smem, cudaStream_t s) {
    if (p.has_zero)
        return p.scale_bf16 ? launch_rows<G, ONE, true, true, NT>(p, grid, teams, smem, s)
                            : launch_rows<G, ONE, false, true, NT>(p, grid, teams, smem, s);
    return p.scale_bf16 ? launch_rows<G, ONE, true, false, NT>(p, grid, teams, smem, s)
                        : launch_rows<G, ONE, false, false, NT>(p, grid, teams, smem, s);
}

template <int G>
cudaError_t launch_group(const W4Params& p, bool one, int nt, int grid, int teams, size_t smem, cudaStream_t s) {
    if (one)
        return nt == 1 ? launch_params<G, true, 1>(p, grid, teams, smem, s)
                       : launch_params<G, true, 2>(p, grid, teams, smem, s);
    return nt == 1   ? launch_params<G, false, 1>(p, grid, teams, smem, s)
           : nt == 2 ? launch_params<G, false, 2>(p, grid, teams, smem, s)
                     : launch_params<G, false, 4>(p, grid, teams, smem, s);
}

}  // namespace

size_t proj_w4_workspace_bytes(int t, int in_f) {
    // (more than a call of up to 16 rows needs whose weights are few)
    return t > 4 ? proj_w4_wide_workspace_bytes(t, in_f) : 0;
}

cudaError_t launch_proj_w4(const ProjW4Args& a, cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const bool one = a.x_bf16 && a.t > 4;
    const int cols = one ? a.t : 2 * a.t, nt = cols <= 8 ? 1 : cols <= 16 ? 2 : 4;
    const int all = a.in_f / kChunk;
    W4Params p{};
    p.x = a.x;
    int tiles = 0;
    for (int i = 0; i < a.nw; ++i) {
        p.w[i] = static_cast<const uint8_t*>(a.w[i]);
        p.scale[i] = a.scale[i];
        p.zero[i] = a.zero[i];
        p.out[i] = a.out[i];
        p.rows[i] = a.rows[i];
        p.tile_start[i] = tiles;
        tiles += (a.rows[i] + kRows - 1) / kRows;
    }
    p.tile_start[a.nw] = tiles;
    if (tiles == 0) return cudaSuccess;
    // the fewest CTAs along K whose share of x fits
    int ks = 1;
    while (ks < 8 && (all + ks - 1) / ks * (kChunk * cols * 2) > kXSmem) ks *= 2;
    // This form or the one for batches.  With one MMA tile of columns this one is faster at any size
    // (64 heads x 6144: 25 us against 34 at eight bf16 rows).  With two, while x of all of K fits into
    // one block (28 against 34 us at five f32 rows; cut along K: 35 at eight, 40 at sixteen bf16
    // rows); with two or four, while the weights are few, where its single launch tells: 128 chunks of
    // 1 KB an SM (16 heads x 2176: 8 against 14 us at eight f32 rows), or 64 of them (13 against 14 at
    // 13 rows; 32 heads x 2048, 83 chunks an SM: 14 - 16 against 14.5).
    const long work = (long)tiles * all;
    const bool few = nt == 1 || (nt == 2 && ks == 1) || work <= (long)sms * (nt == 4 ? 64 : 128);
    if (a.t > 16 || !few || (all + ks - 1) / ks * (kChunk * cols * 2) > kXSmem)
        return launch_proj_w4_wide(a, s);
    p.nw = a.nw; p.t = a.t; p.in_f = a.in_f; p.x_bf16 = a.x_bf16; p.scale_bf16 = a.scale_bf16; p.has_zero = a.has_zero;
    p.ksplit = ks;
    const int blocks = tiles < sms / ks ? tiles : (sms / ks < 1 ? 1 : sms / ks);
    const int most = w4_teams(a.group, a.scale_bf16 != 0, a.has_zero != 0, nt);
    const int want = (tiles + blocks - 1) / blocks, teams = want < most ? want : most;
    const W4Smem lay = w4_smem((all + ks - 1) / ks, cols, a.group, teams, one ? 8 * nt : 4 * nt, nt);
    switch (a.group) {
        case 32: return launch_group<32>(p, one, nt, blocks * ks, teams, (size_t)lay.total, s);
        case 64: return launch_group<64>(p, one, nt, blocks * ks, teams, (size_t)lay.total, s);
        default: return launch_group<128>(p, one, nt, blocks * ks, teams, (size_t)lay.total, s);
    }
}

}  // namespace kda
