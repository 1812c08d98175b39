// kda_accept.cu -- verification of drafted tokens against the target's probabilities: drafts of a
// sequence are accepted in turn while u_i q_i(x_i) < p_i(x_i), then one more token is drawn, from
// max(p - q, 0) where a draft was refused and from p after the last one, as the first index whose
// running sum of weights passes r times their total.
//
// The work is the one row (two with the draft's) that a sequence draws from; everything before it is a
// few dependent reads.  A cluster of CTAs shares a sequence's row, so that one user's 131072 weights
// are read by 8 SMs.  The row is read once: each warp sums tiles of 512 weights, the tile sums give
// the tile that holds the drawn index, and only that tile is read again (from L2).
//
// Which index is drawn must not hang on the order of summation: next to a border an f32 running sum
// over a flat row is off by several indices.  All sums are of f32 pairs (a value and what its rounding left,
// the exact error of p - q among it), about 2^-45 of the sum.  (f64 has the same bits, but its additions took
// some 600 cycles each here: 10 us of a call's 12.)  A row of finite weights whose sum is past f32 is drawn from by one
// warp, in another unit.
// Measured, vocabulary 131072: one sequence 10.3 us in a stream of calls (three dependent reads, a reduction over
// the cluster, a tile's read), 64 sequences x 4 drafts 19.3 us, 3.0 TB/s.
#include "kda_device.cuh"

namespace kda {

namespace {

constexpr int kThr = 512;
constexpr int kWarps = kThr / 32;
constexpr int kTileElems = 512;                  // weights of a tile
constexpr int kPerLane = kTileElems / 32;
constexpr int kMaxTiles = 1024;                  // tiles whose sums a CTA keeps; longer rows: more a sum

// An unevaluated sum hi + lo; "whole" when hi is that sum rounded, which comparisons and products need.
struct Pair {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float x, float xe) {
        const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
        const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b));
        hi = s;
        lo = __fadd_rn(lo, __fadd_rn(e, xe));
    }
    __device__ __forceinline__ Pair whole() const {
        Pair r;
        r.hi = __fadd_rn(hi, lo);
        r.lo = __fsub_rn(lo, __fsub_rn(r.hi, hi));
        return r;
    }
};

__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    a.add(b.hi, b.lo);
    return a.whole();
}
__device__ __forceinline__ bool operator>(Pair a, Pair b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
__device__ __forceinline__ Pair operator*(float r, Pair a) {
    Pair p;
    p.hi = __fmul_rn(r, a.hi);
    p.lo = fmaf(r, a.lo, fmaf(r, a.hi, -p.hi));
    return p.whole();
}

__device__ __forceinline__ Pair shfl(Pair x, int from) {
    x.hi = __shfl_sync(0xffffffffu, x.hi, from);
    x.lo = __shfl_sync(0xffffffffu, x.lo, from);
    return x;
}

// the sum over the warp, the same in every lane
__device__ __forceinline__ Pair warp_pair_sum(Pair x) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
        const float h = __shfl_xor_sync(0xffffffffu, x.hi, m), l = __shfl_xor_sync(0xffffffffu, x.lo, m);
        x.add(h, l);
    }
    // (the lanes may differ in the last bits of lo: all take lane 0's, and so the same branches)
    return shfl(x.whole(), 0);
}

// the sums over the lanes up to each, and (before) those up to the one before it
__device__ __forceinline__ Pair warp_scan(Pair x, int lane, Pair& before) {
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        Pair y;
        y.hi = __shfl_up_sync(0xffffffffu, x.hi, m);
        y.lo = __shfl_up_sync(0xffffffffu, x.lo, m);
        const Pair z = y + x;
        if (lane >= m) x = z;
    }
    before.hi = __shfl_up_sync(0xffffffffu, x.hi, 1);
    before.lo = __shfl_up_sync(0xffffffffu, x.lo, 1);
    if (lane == 0) before = Pair();
    return x;
}

// One weight and its rounding error: p - q where positive, else 0 (so is a NaN or an infinity).
__device__ __forceinline__ void weight(float p, float q, float& w, float& e) {
    q = q > 0.0f ? q : 0.0f;
    const float d = __fsub_rn(p, q);
    const bool on = d > 0.0f && d < __int_as_float(0x7f800000);
    w = on ? d : 0.0f;
    e = on ? __fsub_rn(__fsub_rn(p, d), q) : 0.0f;   // exact: p > q >= 0
}

struct Row {                                     // what a sequence draws from
    const void* p;
    const void* q;                               // or null
    int skip;                                    // index that weighs nothing, or -1
    // tiles begin `lead` elements before the row, where p's address is a multiple of 4 elements; q_vec: so
    // is q's
    int lead;
    bool q_vec;
    template <bool BF16>
    __device__ __forceinline__ void align() {
        constexpr int kElem = BF16 ? 2 : 4;
        lead = (int)(reinterpret_cast<uintptr_t>(p) / kElem % 4);
        q_vec = q == nullptr || (int)(reinterpret_cast<uintptr_t>(q) / kElem % 4) == lead;
    }
};

template <bool BF16>
__device__ __forceinline__ void weight_at(const Row& row, long i, long V, float& w, float& e) {
    const bool in = i >= 0 && i < V && i != row.skip;
    weight(in ? load_raw<BF16>(row.p, i) : 0.0f, in && row.q ? load_raw<BF16>(row.q, i) : 0.0f, w, e);
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

// A lane's share of the weights b .. b + kTileElems - 1: with `runs` its 16 are consecutive, else 4 times 4 at
// distances of 128.  Their sum.  By the whole warp.  Whole tiles go two weights an instruction (64 sequences x
// 131072: 22.9 -> 20.3 us), with max(p, max(q, 0)) - max(q, 0) for the weight, which a NaN leaves 0; a tile
// with an infinity is summed again one by one.
template <bool BF16>
__device__ __forceinline__ Pair lane_sum(const Row& row, long b, long V, int lane, bool runs) {
    Pair acc;
    const int at = runs ? kPerLane * lane : 4 * lane, step = runs ? 4 : 128;
    if (b >= 0 && b + kTileElems <= V && !(row.skip >= b && row.skip < b + kTileElems)) {
        float4 p[kPerLane / 4], q[kPerLane / 4];
#pragma unroll
        for (int i = 0; i < kPerLane / 4; ++i) p[i] = prob4<BF16>(row.p, b + at + step * i);
#pragma unroll
        for (int i = 0; i < kPerLane / 4; ++i) {
            const long x = b + at + step * i;
            q[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row.q != nullptr) {
                if (row.q_vec) q[i] = prob4<BF16>(row.q, x);
                else q[i] = make_float4(load_raw<BF16>(row.q, x), load_raw<BF16>(row.q, x + 1),
                                        load_raw<BF16>(row.q, x + 2), load_raw<BF16>(row.q, x + 3));
            }
        }
        const float2 neg = make_float2(-1.0f, -1.0f);
        const auto sub = [&](float2 x, float2 y) { return __ffma2_rn(y, neg, x); };
        float2 hi = make_float2(0.f, 0.f), lo = hi;
#pragma unroll
        for (int i = 0; i < kPerLane / 2; ++i) {
            const float4 p4 = p[i / 2], q4 = q[i / 2];
            float2 pp = i % 2 ? make_float2(p4.z, p4.w) : make_float2(p4.x, p4.y);
            float2 qq = i % 2 ? make_float2(q4.z, q4.w) : make_float2(q4.x, q4.y);
            qq = make_float2(fmaxf(qq.x, 0.0f), fmaxf(qq.y, 0.0f));
            pp = make_float2(fmaxf(pp.x, qq.x), fmaxf(pp.y, qq.y));
            const float2 d = sub(pp, qq), de = sub(sub(pp, d), qq);
            const float2 s = __fadd2_rn(hi, d), t = sub(s, hi);
            lo = __fadd2_rn(lo, __fadd2_rn(__fadd2_rn(sub(hi, sub(s, t)), sub(d, t)), de));
            hi = s;
        }
        acc.hi = hi.x;
        acc.lo = lo.x;
        acc.add(hi.y, lo.y);
        if (!__any_sync(0xffffffffu, !(acc.hi < __int_as_float(0x7f800000)))) return acc;
        acc = Pair();
    }
#pragma unroll 4
    for (int i = 0; i < kPerLane; ++i) {
        float w, e;
        weight_at<BF16>(row, b + (runs ? kPerLane * lane + i : 32 * i + lane), V, w, e);
        acc.add(w, e);
    }
    return acc;
}

// The index that a row's weights give whose sum is past f32, by one warp: with all of them times 2^-40, in which unit the
// sum of 2^31 is not (what the smallest of them lose is below 2^-180 of it).
template <bool BF16>
__device__ __noinline__ int draw_scaled(const Row row, long V, float r, int lane) {
    const auto at = [&](long i) {
        const bool in = i < V && i != row.skip;
        Pair w;
        weight(in ? load_raw<BF16>(row.p, i) * 0x1p-40f : 0.0f,
               in && row.q ? load_raw<BF16>(row.q, i) * 0x1p-40f : 0.0f, w.hi, w.lo);
        return w;
    };
    const auto tile_sum = [&](long b) {
        Pair x;
        for (int i = 0; i < kPerLane; ++i) {
            const Pair w = at(b + 32 * i + lane);
            x.add(w.hi, w.lo);
        }
        return warp_pair_sum(x);
    };
    Pair sum, run;
    for (long b = 0; b < V; b += kTileElems) sum = sum + tile_sum(b);
    const Pair aim = r * sum;
    long b = 0;
    for (;; b += kTileElems) {
        const Pair x = run + tile_sum(b);
        if (x > aim || b + kTileElems >= V) break;
        run = x;
    }
    int last = -1;
    for (long i = b; i < min(V, b + kTileElems); ++i) {
        const Pair w = at(i);
        if (!(w.hi > 0.0f)) continue;
        last = (int)i;
        run = run + w;
        if (run > aim) break;
    }
    return last;
}

__device__ __forceinline__ Pair ld_cluster_pair(const Pair* local, uint32_t rank) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
    Pair v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.hi), "=f"(v.lo) : "r"(remote) : "memory");
    return v;
}

template <bool BF16>
__global__ void __launch_bounds__(kThr, 2) kda_draft_accept_kernel(const AcceptArgs a) {
    __shared__ __align__(8) Pair tiles[kMaxTiles];
    __shared__ __align__(8) Pair total[2];       // of this CTA, by attempt
    __shared__ int s_taken, s_count, s_token;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = blockIdx.y, rank = blockIdx.x, ranks = gridDim.x;   // the cluster is the x extent
    const int drafts = a.T - 1;
    constexpr size_t kElem = BF16 ? 2 : 4;
    const unsigned char* target = static_cast<const unsigned char*>(a.target) +
                                  (size_t)n * a.T * a.target_stride * kElem;
    const unsigned char* draft = a.draft ? static_cast<const unsigned char*>(a.draft) +
                                               (size_t)n * drafts * a.draft_stride * kElem
                                         : nullptr;

    const float r = a.r[n];
    // how many drafts hold: lane i tests draft i
    if (warp == 0) {
        // (two rounds of reads, not four: what a draft beyond the count would need is read too)
        int count = a.n_draft ? a.n_draft[n] : drafts;
        const int tok = lane < drafts ? a.tokens[(long)n * drafts + lane] : -1;
        const float u = lane < drafts ? a.u[(long)n * drafts + lane] : 0.0f;
        float p = 0.0f, q = 1.0f;
        const bool known = tok >= 0 && tok < a.V;
        if (known) {
            p = load_raw<BF16>(target + (size_t)lane * a.target_stride * kElem, tok);
            if (draft) q = load_raw<BF16>(draft + (size_t)lane * a.draft_stride * kElem, tok);
        }
        const bool live = count >= 0;
        count = min(max(count, 0), drafts);
        bool good = false;
        if (known && lane < count) {
            // u q < p exactly: where the rounded product equals p its error decides (small ones are taken times
            // 2^100, or that error would be lost among denormals)
            if (fmaxf(p, q) < 0x1p-60f) {
                p *= 0x1p100f;
                q *= 0x1p100f;
            }
            const float x = __fmul_rn(u, q);
            good = x < p || (x == p && fmaf(u, q, -x) < 0.0f);
        }
        const unsigned refused = ~__ballot_sync(0xffffffffu, good);
        const int taken = live ? min(__ffs(refused) - 1, count) : -1;
        if (lane == 0) {
            s_taken = taken;
            s_count = count;
        }
        if (lane == taken) s_token = tok;        // the refused one
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
    Row row{p_row, nullptr, -1, 0, true};
    if (refused) {
        if (draft) row.q = draft + (size_t)taken * a.draft_stride * kElem;
        else row.skip = s_token;
    }
    row.template align<BF16>();
    // this CTA's slice, in spans of whole tiles; a span's sum is one entry of tiles[]
    const long all_tiles = ((long)a.V + row.lead + kTileElems - 1) / kTileElems;
    const long per_cta = (all_tiles + ranks - 1) / ranks;
    const long tile0 = min(all_tiles, rank * per_cta), tile1 = min(all_tiles, tile0 + per_cta);
    const long group = (per_cta + kMaxTiles - 1) / kMaxTiles;         // tiles of a span
    const int spans = (int)((tile1 - tile0 + group - 1) / group);

    Pair before, mine, sum;
    for (int attempt = 0; attempt < 2; ++attempt) {
        for (int sp = warp; sp < spans; sp += kWarps) {
            Pair x;
            for (long t = tile0 + sp * group; t < min(tile1, tile0 + (sp + 1) * group); ++t)
                x = x + lane_sum<BF16>(row, t * kTileElems - row.lead, a.V, lane, false);
            x = warp_pair_sum(x);
            if (lane == 0) tiles[sp] = x;
        }
        __syncthreads();
        if (warp == 0) {
            Pair x;
            for (int sp = lane; sp < spans; sp += 32) x = x + tiles[sp];
            x = warp_pair_sum(x);
            if (lane == 0) total[attempt] = x;
        }
        __syncwarp();
        cluster_sync_all();
        Pair of[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < ranks) of[k] = ld_cluster_pair(&total[attempt], k);
        before = mine = sum = Pair();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k == rank) before = sum;
            if (k < ranks) sum = sum + of[k];
            if (k == rank) mine = sum;           // the running sum past this CTA
        }
        if (!(sum.hi == 0.0f) || (row.q == nullptr && row.skip < 0)) break;
        row.q = nullptr;                         // nothing is left of p - q: p itself
        row.skip = -1;
        row.q_vec = true;
    }
    // r in [0, 1): the whole sum is passed at the last weight at the latest.  (Small sums, exact among denormals, are
    // compared times 2^100: r times them is not.)
    const float up = sum.hi < 0x1p-60f ? 0x1p100f : 1.0f;
    const auto scaled = [&](Pair x) {
        x.hi *= up;
        x.lo *= up;
        return x;
    };
    const float r01 = fminf(fmaxf(r, 0.0f), 0x1.fffffep-1f);
    const Pair aim = r01 * scaled(sum);
    const auto passes = [&](const Pair& x) { return scaled(x) > aim; };
    if (!(sum.hi > 0.0f && sum.hi < __int_as_float(0x7f800000))) {       // nothing, or more than f32 holds
        if (rank == 0 && warp == 0) {
            const int token = sum.hi == 0.0f ? -1 : draw_scaled<BF16>(row, a.V, r01, lane);
            if (lane == 0) a.out_tokens[(long)n * a.T + taken] = token;
        }
    } else if (!passes(before) && passes(mine) && warp == 0) {
        // the span, the tile, the lane's 16 weights and the one of them at which the running sum passes aim.
        // (Where rounding between two ways of summing leaves aim past a piece, its last part is taken.)
        Pair run = before, below;
        int sp = 0;
        for (;; sp += 32) {
            const Pair x = sp + lane < spans ? tiles[sp + lane] : Pair();
            const Pair upto = run + warp_scan(x, lane, below);
            const unsigned past = __ballot_sync(0xffffffffu, passes(upto));
            const bool done = past != 0 || sp + 32 >= spans;
            const int at = past != 0 ? __ffs(past) - 1 : done ? spans - 1 - sp : 31;
            const Pair at_below = run + shfl(below, at);
            run = done ? at_below : shfl(upto, at);
            if (done) {
                sp += at;
                break;
            }
        }
        long t = tile0 + sp * group;
        const long t_end = min(tile1, t + group);
        for (; t < t_end - 1; ++t) {
            const Pair x = run + warp_pair_sum(lane_sum<BF16>(row, t * kTileElems - row.lead, a.V, lane, false));
            if (passes(x)) break;
            run = x;
        }
        const long b = t * kTileElems - row.lead;
        const Pair of_lane = lane_sum<BF16>(row, b, a.V, lane, true).whole();
        const Pair upto = run + warp_scan(of_lane, lane, below);
        unsigned past = __ballot_sync(0xffffffffu, passes(upto));
        const unsigned any = __ballot_sync(0xffffffffu, of_lane.hi > 0.0f);
        const int pick_lane = past != 0 ? __ffs(past) - 1 : any != 0 ? 31 - __clz(any) : 31;
        run = run + shfl(below, pick_lane);
        Pair w;
        weight_at<BF16>(row, lane < kPerLane ? b + kPerLane * pick_lane + lane : -1, a.V, w.hi, w.lo);
        const Pair at_lane = run + warp_scan(w, lane, below);        // (every lane takes part)
        past = __ballot_sync(0xffffffffu, w.hi > 0.0f && passes(at_lane));
        const unsigned on = __ballot_sync(0xffffffffu, w.hi > 0.0f);
        const int at = past != 0 ? __ffs(past) - 1 : on != 0 ? 31 - __clz(on) : 0;
        if (lane == 0) a.out_tokens[(long)n * a.T + taken] = (int)(b + kPerLane * pick_lane + at);
    }
    __syncwarp();
    cluster_sync_all();                          // no CTA leaves while another reads its total
}

template <bool BF16>
cudaError_t launch(const AcceptArgs& a, cudaStream_t s) {
    // CTAs a sequence: of at least a tile a warp, and as many as run at once (two on an SM; clusters of 8 leave
    // some of the 152 SMs out)
    const long tiles = ((long)a.V + kTileElems - 1) / kTileElems;
    int ranks = 1;
    while (ranks < 8 && 2L * a.N * ranks <= 256 && tiles > (long)ranks * kWarps) ranks *= 2;
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
