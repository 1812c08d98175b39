// kda_internal.h -- host-side launch interface between the C ABI (kda_api.cu) and the kernels.
// Every launcher assumes its arguments already passed the ABI's contract checks and returns the
// cudaError_t of its launch(es).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace kda {

constexpr int kHeadDim = 128;      // the only head width the kernels are built for
constexpr int kMaxConvK = 8;       // conv window held in registers (taps 2..8)
// device error word bits (written by kernels, read by kda_device_status)
constexpr int kDevErrTimeout = 1;  // a bounded wait gave up
constexpr int kDevErrSlot = 2;     // a slot outside its pool, or named twice
constexpr int kMaxDevices = 64;    // per-device caches (symbol addresses, function attributes)

// A value looked up once per device (a symbol address, an attribute that was set).  Every slot
// is an atomic, so host threads that make their first call on one device at the same time each
// look the value up and store the same result: no data race.  The cache is not invalidated by
// cudaDeviceReset; a process that resets a device must not call the library on it afterwards.
template <typename T>
using PerDevice = std::atomic<T>[kMaxDevices];

constexpr int kMaxBlockSmem = 227 * 1024;   // dynamic shared memory one block can opt into

// Opt a kernel into `bytes` of dynamic shared memory once per device; `done` is the caller's own
// per-device flag array (one per template instantiation).  `bytes` is one constant for a kernel,
// whatever a launch needs: the call sets a value, not a maximum, so that host threads with different
// values would undo one another's.
template <typename K>
inline cudaError_t set_smem(K kernel, size_t bytes, PerDevice<int>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool cached = dev >= 0 && dev < kMaxDevices;
    if (cached && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && cached) done[dev].store(1, std::memory_order_release);
    return e;
}

// Row ranges of the packed token-major arrays.  When cu_seqlens is null every sequence has
// T_uniform tokens and sequence n owns rows [n*T, (n+1)*T).
struct SeqLayout {
    const int* cu_seqlens;   // device int32 [N+1] or null
    int T_uniform;
    int N;
    long total_rows;
};

struct PrepArgs {
    const void* q_raw; const void* k_raw; const void* v_raw; int raw_bf16;
    const float* conv_w;                 // [3C, K] or null (no conv, no SiLU)
    const float* ring_in; float* ring_out;  // [N, 3C, K-1]
    const float* f_raw; const float* dt_bias; const float* a_log; int gate_mode; float gate_lb;
    const float* beta_raw;
    float* q_hat; float* k_hat; float* v_hat; float* g; float* beta;
    SeqLayout seq;
    int H; int K; float l2_eps;
    int Hk;                  // heads of the q and k planes (grouped queries: value head h reads
                             // q/k head h % Hk); 0 means H
    int Hg;                  // heads of the gate and beta (a value head wider than 128 is H / Hg
                             // 128-wide sub-heads that share them); 0 means H
};

// Gate / beta heads of a prep call (the value heads); H counts 128-wide value sub-heads.
__host__ __device__ inline int prep_gate_heads(const PrepArgs& a) { return a.Hg > 0 ? a.Hg : a.H; }

// Channel layout of the three conv planes under grouped queries: q and k hold Hk heads, v holds H;
// conv_w rows and ring rows are [q | k | v] = [Hk*D | Hk*D | H*D] (gdn_ops.rs gdn_delta_rule_into
// doc: q, k are [num_k_heads * head_k_dim], v is [num_v_heads * head_v_dim]).
__host__ __device__ inline int prep_qk_heads(int H, int Hk) { return Hk > 0 ? Hk : H; }
__host__ __device__ inline long plane_width(int H, int Hk, int p) {
    return (long)(p < 2 ? prep_qk_heads(H, Hk) : H) * kHeadDim;
}
__host__ __device__ inline long plane_offset(int H, int Hk, int p) {
    return (long)p * prep_qk_heads(H, Hk) * kHeadDim;
}
__host__ __device__ inline long ring_channels(int H, int Hk) {
    return (2L * prep_qk_heads(H, Hk) + H) * kHeadDim;
}

struct ScanArgs {
    const float* q; const float* k; const float* v; const float* g; int gate_mode;
    const float* beta;
    const float* state_in; float* state_out; float* o;
    SeqLayout seq;
    int H; float scale;
    const int* order;        // device-side order of sequences (longest first) or null
    int* err;                // device error word
    int Hk;                  // heads of q and k (grouped queries: value head h reads q/k head
                             // h % Hk; rows of q and k are Hk * D wide); 0 means H
    int vsub;                // 128-wide sub-heads per value head (value width vsub * 128): unit h
                             // is value head h / vsub, which owns the gate and beta and reads q/k
                             // head (h / vsub) % Hk; 0 means 1
    // the gated RMSNorm folded into the chunked scan's readout (fused prefill, 128-wide value
    // heads): with norm_y set the chunk kernel writes y = rmsnorm(o) * w * gate(z) in place of o
    const float* norm_w; const float* norm_z; float* norm_y; float norm_eps;
    int norm_silu;           // gate: 0 sigmoid (KDA), 1 SiLU (GDN's gated_rmsnorm)
};

// the heads of q and k, and the one value head h reads
__host__ __device__ inline int qk_heads(const ScanArgs& a) { return a.Hk > 0 ? a.Hk : a.H; }
__host__ __device__ inline int value_sub(const ScanArgs& a) { return a.vsub > 0 ? a.vsub : 1; }
// the value head (gate and beta head) of unit h, the number of such heads, and the q/k head
__host__ __device__ inline int gate_head(const ScanArgs& a, int h) { return h / value_sub(a); }
__host__ __device__ inline int gate_heads(const ScanArgs& a) { return a.H / value_sub(a); }
__host__ __device__ inline int unit_qk_head(const ScanArgs& a, int h) {
    return gate_head(a, h) % qk_heads(a);
}

struct NormArgs {
    const float* o; const float* w; const float* z; float* y; long rows; float eps;
    int silu;                // gate: 0 sigmoid (KDA), 1 SiLU (GDN's gated_rmsnorm)
    int width;               // row length, a multiple of 128 (0 means 128)
};

struct DecodeArgs {
    const void* q_raw; const void* k_raw; const void* v_raw; int raw_bf16;
    const float* conv_w; const float* ring_in; float* ring_out;
    const float* f_raw; const float* dt_bias; const float* a_log; int gate_mode; float gate_lb;
    const float* beta_raw;
    const float* state_in; float* state_out;
    const float* norm_w; const float* gate_raw; float* y;
    int N; int T; int H; int K; float l2_eps; float scale; float rms_eps;
    const int* keep;         // rollback: tokens of sequence n to take (device [N], clamped to
                             // 0..T; rows keep their stride T), or null for all T
    int Hk;                  // heads of the q and k planes (grouped queries); 0 means H
    int norm_silu;           // RMSNorm gate: 0 sigmoid (KDA), 1 SiLU (GDN's gated_rmsnorm)
    int* err;                // device error word (bounded waits)
    int vsub;                // 128-wide units per value head (H counts units); 0 means 1.  A
                             // value head's units run as one thread-block cluster, which sums the
                             // RMSNorm's squares over the whole value row
};

cudaError_t launch_prep(const PrepArgs& a, cudaStream_t s);
cudaError_t launch_wait_selftest(int* err, cudaStream_t s);
cudaError_t launch_scan_seq(const ScanArgs& a, cudaStream_t s);
cudaError_t launch_scan_chunk(const ScanArgs& a, const int* cu_host, void* workspace,
                              cudaStream_t s);
// exact workspace the chunked scan needs for this layout (cu_host: host copy of cu_seqlens)
size_t chunk_workspace_bytes(const SeqLayout& s, const int* cu_host, int H);
long chunk_count(const SeqLayout& s, const int* cu_host);
// pieces of the chunked form for the fused prefill (kda_scan_chunk.cu): the varlen chunk offsets
// at the head of the workspace (blocks = where the per-(chunk, head) blocks start), and the
// inter-chunk kernel over filled blocks
cudaError_t launch_chunk_offsets(const SeqLayout& seq, void* workspace, int** chunk_off,
                                 unsigned char** blocks, cudaStream_t s);
cudaError_t launch_chunk_inter(const ScanArgs& a, const int* chunk_off,
                               const unsigned char* blocks, cudaStream_t s,
                               const PrepArgs* ring = nullptr);
// the fused prefill's prep + intra-chunk kernel, then the ring roll (kda_chunk_prep.cu)
cudaError_t launch_prefill_chunk(const PrepArgs& p, const ScanArgs& a, const int* cu_host,
                                 void* workspace, cudaStream_t s);
// the conv ring roll alone (kda_prep.cu)
cudaError_t launch_ring_roll(const PrepArgs& a, cudaStream_t s);

// Fixed device scratch for kda_scan_varlen_static (kda_scan_static.cu): its byte size, and the
// address of this device's copy (looked up once per device, on the first call with it current).
constexpr size_t kStaticScratchBytes = (size_t)32 << 20;
cudaError_t static_scratch(void** ptr);
constexpr int kChunkTokens = 32;        // tokens per chunk of the chunked scan
constexpr size_t kChunkBlockBytes = 43520;  // workspace bytes per (chunk, head)

// 2-D f32 tensor map over [rows, cols] (row stride = cols), box [box_rows, box_cols], no swizzle.
bool make_tensor_map_2d(CUtensorMap* m, const float* base, long rows, long cols, int box_cols,
                        int box_rows);
// The same over bf16 (bf16 = true) or f32 elements.
bool make_tensor_map_2d_any(CUtensorMap* m, const void* base, bool bf16, long rows, long cols,
                            int box_cols, int box_rows);
// The U rows of the chunked scan's workspace blocks: f32 [nblocks][32 tokens][128 values] at
// `base` (the first block's U region), block stride block_bytes; box [1][32][32], 128-byte swizzle.
bool make_tensor_map_blocks_ut(CUtensorMap* m, void* base, long nblocks, size_t block_bytes);
// The layer input's six projections (kda_proj.cu).  Weights are bf16 [rows_i, in_f]; outputs f32
// [t, rows_i]; x f32 [t, in_f]; ws holds x split into bf16 hi / lo images of t_pad rows.
struct Proj6Args {
    const float* x;
    const void* w[6];
    float* out[6];
    int rows[6];
    int t; int in_f;
    void* ws;
    int* err;
};
constexpr int kProjMaxT = 256;          // token rows per call: the MMA's N
constexpr int kProjKAlign = 128;        // in_f must be a multiple of this
inline int proj_t_pad(int t) { return (t + 15) / 16 * 16; }
inline size_t proj_workspace_bytes(int t, int in_f) {
    return 2 * (size_t)proj_t_pad(t) * (size_t)in_f * 2;   // x hi and x lo, bf16
}
cudaError_t launch_proj6(const Proj6Args& a, cudaStream_t s);
// 2-D bf16 tensor map over [rows, cols], rows row_stride elements apart (0: cols), with a [box_rows][64]
// box in the 128-byte swizzle
bool make_tensor_map_2d_bf16_sw128(CUtensorMap* m, const void* base, long rows, long cols,
                                   int box_rows, long row_stride = 0);
// 2-D f32 tensor map over [rows, cols] with a [box_rows][32] box in the 128-byte swizzle
bool make_tensor_map_2d_f32_sw128(CUtensorMap* m, const void* base, long rows, long cols, int box_rows);
cudaError_t launch_gated_rmsnorm(const NormArgs& a, cudaStream_t s);
cudaError_t launch_decode_fused(const DecodeArgs& a, cudaStream_t s);

constexpr int kDecodeMaxT = 16;   // tokens one fused decode/verify call may carry

// The 8-bit state pool (kda_q8.cuh, kda_state_q8.cu, kda_decode_q8.cu).
constexpr int kQ8Int8 = 0, kQ8E4m3 = 1;
// Store: f32 rows of state_in / ring_src -> pool rows; load: pool rows -> f32 rows of state_out.
// src / dst: device int32 [N] row indices (null: row n), negative for padding.
struct StateQ8Args {
    const float* state_in; float* state_out;
    void* codes; float* scales; int fmt;
    const int* src; const int* dst;
    int src_rows; int dst_rows;
    int N; int units;                       // 128-wide value units of a row
    const float* ring_src; float* ring_dst; long ring_row;   // floats of one ring row; 0: no ring
    int* err;
};
cudaError_t launch_state_store_q8(const StateQ8Args& a, cudaStream_t s);
cudaError_t launch_state_load_q8(const StateQ8Args& a, cudaStream_t s);
// The decode step on the pool: DecodeArgs with state and ring rows in pool slots (state_in,
// state_out, ring_in unused; ring_out is the ring pool).
struct DecodeQ8Args {
    DecodeArgs d;
    void* codes; float* scales; int fmt;
    const int* slots; const int* slots_out; int pool_rows;
};
cudaError_t launch_decode_q8(const DecodeQ8Args& a, cudaStream_t s);

// Projections by 4-bit weights with group scales (kda_proj_w4.cu).
constexpr int kW4MaxWeights = 8;        // weights of one call
constexpr int kW4MaxInF = 32768;        // widest x
struct ProjW4Args {
    const void* x; int x_bf16;
    const void* w[kW4MaxWeights]; const void* scale[kW4MaxWeights]; const void* zero[kW4MaxWeights];
    float* out[kW4MaxWeights];
    int rows[kW4MaxWeights];
    int nw; int t; int in_f; int group; int scale_bf16; int has_zero;
    void* ws;
    int* err;
};
size_t proj_w4_workspace_bytes(int t, int in_f);
cudaError_t launch_proj_w4(const ProjW4Args& a, cudaStream_t s);
// the form for batches, on tcgen05 (kda_proj_w4_wide.cu)
constexpr int kW4MaxSms = 152;
constexpr int kW4MaxBlocks = 2 * kW4MaxSms;   // its blocks: two per SM at most
size_t proj_w4_wide_workspace_bytes(int t, int in_f);
cudaError_t launch_proj_w4_wide(const ProjW4Args& a, cudaStream_t s);
// 2-D byte tensor map over [rows, cols] with a [box_rows][64] box in the 64-byte swizzle
bool make_tensor_map_2d_u8_sw64(CUtensorMap* m, const void* base, long rows, long cols, int box_rows);

// Linear attention with one log-decay a head (kda_linattn.cu: the recurrent form; kda_linattn_chunk.cu:
// the chunked form on tcgen05).
struct LinArgs {
    const void* q; const void* k; const void* v; int bf16;
    long q_stride, k_stride, v_stride;   // elements between token rows
    const float* log_decay;              // [H]
    const float* state_in;               // null: zero (prefill)
    float* state_out;
    float* o;
    SeqLayout seq;
    int H; int Hk; int m;                // value heads, q/k heads, 128-wide units of a value head
    float scale;
    // decode on a pool (state_in == state_out): rows by slot, as in DecodeQ8Args
    const int* slots; const int* slots_out; const int* keep; int pool_rows;
    int* err;
};
cudaError_t launch_linattn_decode(const LinArgs& a, cudaStream_t s);
cudaError_t launch_linattn_seq(const LinArgs& a, cudaStream_t s);
// total_rows > 0; workspace: linattn_chunk_workspace_bytes for these lengths, which the bound covers for any
// lengths of total_T tokens in all
cudaError_t launch_linattn_chunk(const LinArgs& a, const int* cu_host, void* workspace, cudaStream_t s);
size_t linattn_chunk_workspace_bytes(const SeqLayout& seq, const int* cu_host, int Hk, int units, bool bf16);
size_t linattn_chunk_workspace_bound(int N, long total_T, int Hk, int units, bool bf16);

// Verification of drafted tokens (kda_accept.cu).
struct AcceptArgs {
    const void* target; const void* draft; int bf16;
    long target_stride, draft_stride;    // elements between probability rows
    const int* tokens; const float* u; const float* r; const int* n_draft;
    int* keep; int* out_tokens;
    int N; int T; int V;
};
cudaError_t launch_draft_accept(const AcceptArgs& a, cudaStream_t s);

// The norms around a block with its gate and residual (kda_resnorm.cu).
constexpr int kResNormMaxF = 16384;      // widest row
struct ResNormArgs {
    const void* residual; int residual_bf16;
    const void* block; int block_bf16;
    const float* block_w; const void* gate; int gate_per_row; int gate_act;
    float res_scale, block_scale;
    const float* norm_w; void* h; void* z; int z_bf16;
    long rows; int F; float eps;
};
cudaError_t launch_residual_rmsnorm(const ResNormArgs& a, cudaStream_t s);

// ---- optional per-kernel timing (kda_timer.cu): a KernelTimer scoped around a launch records a
// CUDA event before and after it on the launch stream while timing is enabled.
enum KernelId {
    kKPrep, kKRingRoll, kKScanSeq, kKChunkOffsets, kKChunkIntra, kKChunkInter, kKRmsNorm,
    kKDecode, kKPrepIntra, kKProjSplit, kKProj6, kKStateStoreQ8, kKStateLoadQ8, kKDecodeQ8,
    kKRingRollQ8, kKProjW4, kKProjW4Split, kKProjW4Wide, kKLinStep, kKLinSplit, kKLinState, kKLinJoin,
    kKLinChunk, kKDraftAccept, kKResNorm, kKernelCount
};
class KernelTimer {
public:
    KernelTimer(int id, cudaStream_t s);
    ~KernelTimer();
    KernelTimer(const KernelTimer&) = delete;
    KernelTimer& operator=(const KernelTimer&) = delete;
private:
    int id_; cudaStream_t s_; bool on_;
};

}  // namespace kda
