// kda_accept.cu -- verification of drafted tokens against the target's probabilities: drafts of a
// sequence are accepted in turn while u_i q_i(x_i) < p_i(x_i), then one more token is drawn, from
// max(p - q, 0) where a draft was refused and from p after the last one, as the first index whose
// running sum of weights passes r times their total.
//
// The work is the one row (two with the draft's) that a sequence draws from; everything before it is a
// few dependent reads.  A cluster of CTAs shares a sequence's row, so that one user's 131072 weights
// are read by 8 SMs.  The row is read once: each warp sums tiles of 1024 weights, the tile sums give
// the tile that holds the drawn index, and only that tile is read again (from L2).
//
// Which index is drawn must not hang on the order of summation: next to a border an f32 running sum
// over a flat row is off by several indices.  A lane sums its weights as an exact f32 pair (value and
// error of each addition and of p - q), about 2^-46 of the sum, and everything above a lane is in f64.
// (f64 throughout would be 4 operations a weight at a rate far below HBM's.)
#include "kda_device.cuh"

namespace kda {

namespace {

constexpr int kThr = 256;
constexpr int kWarps = kThr / 32;
constexpr int kTileElems = 1024;                 // weights of a tile: 32 a lane
constexpr int kMaxTiles = 1024;                  // tiles whose sums a CTA keeps; longer rows: more a sum

struct Pair {                                    // hi + lo
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float x, float xe) {
        const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
        const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b));
        hi = s;
        lo = __fadd_rn(lo, __fadd_rn(e, xe));
    }
    __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

template <bool BF16>
__device__ __forceinline__ float prob(const void* row, long i) {
    return load_raw<BF16>(row, i);
}

// One weight and its rounding error: p - q where positive, else 0 (so is a NaN or an infinity).
__device__ __forceinline__ void weight(float p, float q, float& w, float& e) {
    const float d = __fsub_rn(p, q);
    const bool on = d > 0.0f && d < __int_as_float(0x7f800000);
    w = on ? d : 0.0f;
    e = on ? __fsub_rn(__fsub_rn(p, d), q) : 0.0f;   // exact: p > q >= 0
}

struct Row {                                     // what a sequence draws from
    const void* p;
    const void* q;                               // or null
    int skip;                                    // index that weighs nothing, or -1
};

template <bool BF16>
__device__ __forceinline__ float q_at(const Row& row, long i) {
    const float q = row.q ? prob<BF16>(row.q, i) : 0.0f;
    return q > 0.0f ? q : 0.0f;
}

template <bool BF16>
__device__ __forceinline__ double weight_at(const Row& row, long i) {
    float w, e;
    weight(prob<BF16>(row.p, i), q_at<BF16>(row, i), w, e);
    return i == row.skip ? 0.0 : (double)w + (double)e;
}

// 4 consecutive probabilities, their address a multiple of 4 elements
template <bool BF16>
__device__ __forceinline__ float4 prob4(const void* row, long i) {
    if constexpr (BF16) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(row) + i));
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                           __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
    } else {
        return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(row) + i));
    }
}

// The sum of weights b .. e - 1 (at most kTileElems), by one warp; every lane returns it.
template <bool BF16>
__device__ __forceinline__ double tile_sum(const Row& row, long b, long e, bool vec, int lane) {
    Pair acc;
    if (vec && e - b == kTileElems) {
        float4 p[8], q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = prob4<BF16>(row.p, b + 128 * i + 4 * lane);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            q[i] = row.q ? prob4<BF16>(row.q, b + 128 * i + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float pp[4] = {p[i].x, p[i].y, p[i].z, p[i].w};
            const float qq[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float w, we;
                weight(pp[j], qq[j] > 0.0f ? qq[j] : 0.0f, w, we);
                const bool skip = b + 128 * i + 4 * lane + j == row.skip;
                acc.add(skip ? 0.0f : w, skip ? 0.0f : we);
            }
        }
    } else {
        for (long i0 = b + lane; i0 < e; i0 += 32 * 8) {
            float p[8], q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const long i = i0 + 32 * j;
                p[j] = i < e ? prob<BF16>(row.p, i) : 0.0f;
                q[j] = i < e ? q_at<BF16>(row, i) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float w, we;
                weight(p[j], q[j], w, we);
                const bool skip = i0 + 32 * j == row.skip;
                acc.add(skip ? 0.0f : w, skip ? 0.0f : we);
            }
        }
    }
    double x = acc.value();
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

__device__ __forceinline__ double ld_cluster_f64(const double* local, uint32_t rank) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(remote) : "memory");
    return v;
}

template <bool BF16>
__global__ void __launch_bounds__(kThr) kda_draft_accept_kernel(const AcceptArgs a) {
    __shared__ double tiles[kMaxTiles];
    __shared__ double total[2];                  // of this CTA, by attempt
    __shared__ int s_taken, s_count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = blockIdx.y, rank = blockIdx.x, ranks = gridDim.x;   // the cluster is the x extent
    const int drafts = a.T - 1;
    constexpr size_t kElem = BF16 ? 2 : 4;
    const unsigned char* target = static_cast<const unsigned char*>(a.target) +
                                  (size_t)n * a.T * a.target_stride * kElem;
    const unsigned char* draft = a.draft ? static_cast<const unsigned char*>(a.draft) +
                                               (size_t)n * drafts * a.draft_stride * kElem
                                         : nullptr;

    // how many drafts hold: lane i tests draft i
    if (warp == 0) {
        int count = a.n_draft ? a.n_draft[n] : drafts;
        const bool live = count >= 0;
        count = min(max(count, 0), drafts);
        bool good = false;
        int tok = -1;
        if (lane < count) {
            tok = a.tokens[(long)n * drafts + lane];
            if (tok >= 0 && tok < a.V) {
                const float p = prob<BF16>(target + (size_t)lane * a.target_stride * kElem, tok);
                const float q = draft ? prob<BF16>(draft + (size_t)lane * a.draft_stride * kElem, tok) : 1.0f;
                // the product of two f32 is exact in f64
                good = (double)a.u[(long)n * drafts + lane] * (double)q < (double)p;
            }
        }
        const unsigned refused = ~__ballot_sync(0xffffffffu, good);
        const int taken = live ? min(__ffs(refused) - 1, count) : -1;
        if (lane == 0) {
            s_taken = taken;
            s_count = count;
        }
        if (rank == 0) {
            if (lane == 0) a.keep[n] = taken + 1;
            if (lane < a.T && lane != taken)
                a.out_tokens[(long)n * a.T + lane] = lane < taken ? tok : -1;
        }
    }
    __syncthreads();
    const int taken = s_taken;
    if (taken < 0) return;                       // padding: the whole cluster leaves
    const bool refused = taken < s_count;

    const void* p_row = target + (size_t)taken * a.target_stride * kElem;
    Row row{p_row, nullptr, -1};
    if (refused) {
        if (draft) row.q = draft + (size_t)taken * a.draft_stride * kElem;
        else row.skip = a.tokens[(long)n * drafts + taken];
    }
    // this CTA's slice, in spans of whole tiles; a span's sum is one entry of tiles[]
    const long all_tiles = (a.V + kTileElems - 1) / kTileElems;
    const long per_cta = (all_tiles + ranks - 1) / ranks;
    const long tile0 = min(all_tiles, rank * per_cta), tile1 = min(all_tiles, tile0 + per_cta);
    const long group = (per_cta + kMaxTiles - 1) / kMaxTiles;         // tiles of a span
    const int spans = (int)((tile1 - tile0 + group - 1) / group);

    double before = 0.0, mine = 0.0, sum = 0.0;
    for (int attempt = 0; attempt < 2; ++attempt) {
        const bool vec = ((reinterpret_cast<uintptr_t>(row.p) | reinterpret_cast<uintptr_t>(row.q)) &
                          (4 * kElem - 1)) == 0;
        for (int sp = warp; sp < spans; sp += kWarps) {
            double x = 0.0;
            for (long t = tile0 + sp * group; t < min(tile1, tile0 + (sp + 1) * group); ++t)
                x += tile_sum<BF16>(row, t * kTileElems, min((long)a.V, (t + 1) * kTileElems), vec, lane);
            if (lane == 0) tiles[sp] = x;
        }
        __syncthreads();
        if (warp == 0) {
            double x = 0.0;
            for (int sp = lane; sp < spans; sp += 32) x += tiles[sp];
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
            if (lane == 0) total[attempt] = x;
        }
        cluster_sync_all();
        before = mine = sum = 0.0;
        for (int k = 0; k < ranks; ++k) {
            if (k == rank) before = sum;
            sum += ld_cluster_f64(&total[attempt], k);
            if (k == rank) mine = sum;           // the running sum past this CTA
        }
        if (sum > 0.0 || (row.q == nullptr && row.skip < 0)) break;
        row = Row{p_row, nullptr, -1};           // nothing is left of p - q: p itself
    }
    // r in [0, 1): the whole sum is passed at the last weight at the latest
    const double aim = (double)fminf(fmaxf(a.r[n], 0.0f), 0x1.fffffep-1f) * sum;
    if (!(sum > 0.0)) {
        if (rank == 0 && tid == 0) a.out_tokens[(long)n * a.T + taken] = -1;
    } else if (aim >= before && aim < mine && warp == 0) {
        // the span, then the tile, then the lane's 32 weights in which the running sum passes aim
        double run = before;
        int sp = 0;
        for (; sp < spans - 1; ++sp) {
            if (run + tiles[sp] > aim) break;
            run += tiles[sp];
        }
        const bool vec = ((reinterpret_cast<uintptr_t>(row.p) | reinterpret_cast<uintptr_t>(row.q)) &
                          (4 * kElem - 1)) == 0;
        long t = tile0 + sp * group;
        const long t_end = min(tile1, t + group);
        for (; t < t_end - 1; ++t) {
            const double x = tile_sum<BF16>(row, t * kTileElems, (t + 1) * kTileElems, vec, lane);
            if (run + x > aim) break;
            run += x;
        }
        const long b = t * kTileElems, e = min((long)a.V, b + kTileElems);
        const long lb = b + 32 * lane, le = min(e, lb + 32);
        double x = 0.0;
        int last = -1;
        for (long i = lb; i < le; ++i) {
            const double w = weight_at<BF16>(row, i);
            x += w;
            if (w > 0.0) last = (int)i;
        }
        double upto = x;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, run + upto > aim);
        int pick = -1;
        if (past != 0) {
            if (lane == __ffs(past) - 1) {
                double at = run + (upto - x);
                for (long i = lb; i < le; ++i) {
                    const double w = weight_at<BF16>(row, i);
                    at += w;
                    if (w > 0.0) pick = (int)i;
                    if (at > aim && w > 0.0) break;
                }
            }
        }
        // (rounding between the two ways of summing may leave aim past the tile: its last weight)
        pick = __reduce_max_sync(0xffffffffu, past != 0 ? pick : last);
        if (lane == 0) a.out_tokens[(long)n * a.T + taken] = pick;
    }
    cluster_sync_all();                          // no CTA leaves while another reads its total
}

template <bool BF16>
cudaError_t launch(const AcceptArgs& a, cudaStream_t s) {
    // CTAs a sequence: up to 8 tiles each stay one warp's work apiece; more sequences than SMs need
    // no sharing
    const long tiles = ((long)a.V + kTileElems - 1) / kTileElems;
    int ranks = 1;
    while (ranks < 8 && (long)a.N * ranks < 1216 && tiles > (long)ranks * kWarps) ranks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ranks, (unsigned)a.N);
    cfg.blockDim = dim3(kThr);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ranks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    KernelTimer kt(kKDraftAccept, s);
    return cudaLaunchKernelEx(&cfg, kda_draft_accept_kernel<BF16>, a);
}

}  // namespace

cudaError_t launch_draft_accept(const AcceptArgs& a, cudaStream_t s) {
    return a.bf16 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace kda
