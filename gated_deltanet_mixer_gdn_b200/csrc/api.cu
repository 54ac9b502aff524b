// C ABI of the Gated DeltaNet mixer (declared in include/gdn.h): argument
// checks, workspace carving, TMA descriptor set-up and kernel launches.
// This is the library's only translation unit; the kernels are included.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <new>
#include <utility>
#include <vector>

#include "../../include/gdn.h"
#include "chunk.cuh"
#include "chunk_pair.cuh"
#include "common.cuh"
#include "decode.cuh"
#include "gemm.cuh"
#include "inproj.cuh"
#include "pool.cuh"
#include "prep.cuh"
#include "qproj.cuh"
#include "quant.cuh"

namespace {

using namespace gdn;

// An NVTX range over one ABI call (named after the entry point), so host timelines of a
// profiler show each call and the launches it enqueued; free when no tool is attached.
struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

constexpr size_t kAlign = 256;
constexpr int kMaxDevices = 64;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_dims(const gdn_dims* d) {
    if (d == nullptr) return GDN_ERR_INVALID_ARG;
    if (d->num_k_heads <= 0 || d->num_v_heads <= 0) return GDN_ERR_INVALID_ARG;
    if (d->head_dim != 128 || d->conv_width != 4) return GDN_ERR_UNSUPPORTED;
    if (d->num_v_heads % d->num_k_heads != 0) return GDN_ERR_UNSUPPORTED;
    if (d->num_v_heads / d->num_k_heads > 8) return GDN_ERR_UNSUPPORTED;
    if (d->num_v_heads > 1024 || d->num_k_heads > 1024) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

int check_weights(const gdn_weights* w) {
    if (w == nullptr || w->conv_w == nullptr || w->A_log == nullptr || w->dt_bias == nullptr || w->norm_w == nullptr)
        return GDN_ERR_INVALID_ARG;
    if (!aligned16(w->conv_w) || !aligned16(w->norm_w)) return GDN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(w->A_log) & 3u) || (reinterpret_cast<uintptr_t>(w->dt_bias) & 3u))
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

int check_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
    int major = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) return GDN_ERR_CUDA;
    return major == 10 ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// 2-D row-major map over [rows][cols] 16-bit elements, box {box_cols, box_rows}.
bool make_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, uint64_t cols, uint64_t rows, uint32_t box_cols,
              uint32_t box_rows, CUtensorMapSwizzle swz) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols * 2};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

struct Workspace {
    size_t off_q, off_k, off_ql, off_kl, off_v, off_g, off_b, off_cb, off_rec, bytes;
};

// Chunks over all rows: exact for uniform rows, and an upper bound for N rows
// of `total` tokens in all (each row adds at most one partial chunk).
int64_t chunk_bound(int64_t N, int64_t total) { return (total + 63 * N) / 64; }

Workspace plan_workspace(const gdn_dims* d, int64_t total, int64_t N, int64_t nchunks) {
    Workspace w{};
    const size_t qk = (size_t)total * d->num_k_heads * 128 * 2;
    const size_t vv = (size_t)total * d->num_v_heads * 128 * 2;
    const size_t gb = (size_t)total * d->num_v_heads * 4;
    w.off_q = 0;
    w.off_k = align_up(qk);
    w.off_ql = w.off_k + align_up(qk);
    w.off_kl = w.off_ql + align_up(qk);
    w.off_v = w.off_kl + align_up(qk);
    w.off_g = w.off_v + align_up(vv);
    w.off_b = w.off_g + align_up(gb);
    w.off_cb = w.off_b + align_up(gb);
    w.off_rec = w.off_cb + align_up((size_t)(2 * N + 1) * 4);  // chunk bases [N+1], then the row order [N]
    w.bytes = w.off_rec + align_up((size_t)nchunks * d->num_v_heads * wy::REC_BYTES);
    return w;
}

// Internal streams of the overlapped dense prefill, one set per device: the
// recurrence runs on a high-priority stream while the load stage and the WY
// records of the next segment run on a low-priority one.  Created on the
// first overlapped call on the device.
constexpr int kMaxSegments = 8;
struct SideStreams {
    bool ready = false;
    cudaStream_t prod = nullptr, chain = nullptr, tail = nullptr;  // priorities: chain > prod > tail
    cudaEvent_t fork = nullptr, prod_done = nullptr, chain_done = nullptr, tail_done = nullptr;
    cudaEvent_t seg[kMaxSegments] = {};   // WY records of a segment written (prod -> chain)
    cudaEvent_t rec[kMaxSegments] = {};   // recurrence of a segment done (chain -> prod)
};
std::mutex g_side_mu;
SideStreams g_side[kMaxDevices];

int side_streams(int dev, SideStreams** out) {
    if (dev < 0 || dev >= kMaxDevices) return GDN_ERR_UNSUPPORTED;
    SideStreams& st = g_side[dev];
    if (!st.ready) {
        int least = 0, greatest = 0;
        if (cudaDeviceGetStreamPriorityRange(&least, &greatest) != cudaSuccess) return GDN_ERR_CUDA;
        // (numerically lower is higher priority; with a single level all three are equal)
        const int middle = greatest < least ? greatest + 1 : greatest;
        if (cudaStreamCreateWithPriority(&st.prod, cudaStreamNonBlocking, middle) != cudaSuccess ||
            cudaStreamCreateWithPriority(&st.chain, cudaStreamNonBlocking, greatest) != cudaSuccess ||
            cudaStreamCreateWithPriority(&st.tail, cudaStreamNonBlocking, least) != cudaSuccess)
            return GDN_ERR_CUDA;
        cudaEvent_t* evs[4] = {&st.fork, &st.prod_done, &st.chain_done, &st.tail_done};
        for (cudaEvent_t* e : evs)
            if (cudaEventCreateWithFlags(e, cudaEventDisableTiming) != cudaSuccess) return GDN_ERR_CUDA;
        for (auto& e : st.seg)
            if (cudaEventCreateWithFlags(&e, cudaEventDisableTiming) != cudaSuccess) return GDN_ERR_CUDA;
        for (auto& e : st.rec)
            if (cudaEventCreateWithFlags(&e, cudaEventDisableTiming) != cudaSuccess) return GDN_ERR_CUDA;
        st.ready = true;
    }
    *out = &st;
    return GDN_OK;
}

// Dynamic shared memory opt-in of a kernel (the attribute belongs to the device's context):
// once per kernel and device, under a lock.
int smem_optin(const void* kernel_fn, uint32_t bytes) {
    static std::mutex mu;
    static std::vector<std::pair<const void*, int>> done;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mu);
    for (auto& d : done)
        if (d.first == kernel_fn && d.second == dev) return GDN_OK;
    if (cudaFuncSetAttribute(kernel_fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
        return GDN_ERR_CUDA;
    done.emplace_back(kernel_fn, dev);
    return GDN_OK;
}

// The load stage fused into the in_proj GEMM: the hidden states and the
// stacked in_proj weights go in; the staged operands, z and the rows' last
// pre-conv tokens come out (z and the latter into workspace buffers).
struct FusedLoad {
    const uint16_t* x;     // bf16 [total][hidden]
    const uint16_t* w_in;  // bf16 [C + Vh*128 + 2*Vh][hidden]
    int hidden;
    uint16_t* z;           // bf16 [total][Vh*128]
    float* conv_last;      // f32 [N][3][C]
};

// out_proj after the mixer (gdn_prefill_out): out[t] = y[t] w_out^T for every token t,
// y being the mixer's gated-norm output.
struct OutProjTail {
    const uint16_t* w_out;  // bf16 [hidden][Vh*128]
    int hidden;
    uint16_t* out;          // bf16 [tokens][hidden]
};

int gemm_launch(const uint16_t* A, const uint16_t* W, struct GemmParams gp, cudaStream_t stream);

// out_proj of tokens [t0, t1) of the call (rows of y and of out).
int out_proj_range(const OutProjTail& op, const uint16_t* y, int VD, int64_t t0, int64_t t1, cudaStream_t st) {
    if (t1 <= t0) return GDN_OK;
    GemmParams gp{};
    gp.M = (int)(t1 - t0);
    gp.N = op.hidden;
    gp.K = VD;
    gp.nseg = 1;
    gp.seg[0] = GemmSegment{0, op.hidden, op.out + t0 * op.hidden};
    return gemm_launch(y + t0 * VD, op.w_out, gp, st);
}

// Segment plan of the overlapped dense prefill.  The load stage runs over all
// tokens first; segment 0's WY records run on every SM; after that, the recurrence
// of segment k (one CTA per row and value head) runs beside the WY records of
// segment k+1 on the remaining SMs.  The plan is picked on the host by simulating
// candidate plans with a cost model of this library's kernels measured on B200: a
// WY launch takes about 11.2 us per wave of tasks (a task: one chunk, one q/k head,
// up to 3 of its value heads) plus 4 us; a recurrence launch about 9.5 us plus 2.3 us
// per chunk (the WY figure as measured beside a running recurrence; erring slow keeps
// the recurrence from waiting).  Candidates: segment sizes growing or shrinking
// geometrically (s_k = s_0 rho^k: rho > 1 lets the recurrence start early when it
// bounds the call, rho < 1 runs most WY records on every SM first when they bound
// it), 2..kMaxSegments segments of at least one chunk, and the plain schedule.
// (Running the load stage per segment on the WY stream as well was measured no
// faster at one row and slower at two.)
namespace seg_model {
constexpr double kWaveUs = 11.2, kWyFixedUs = 4.0, kChainFixedUs = 9.5;
constexpr double kChainChunkUs = 2.3, kPairChainChunkUs = 1.9;  // one CTA per head; CTA pairs
}

// The recurrence runs on CTA pairs (each 64 of a head's value channels, a shorter per-chunk
// chain) when the pairs fit in one wave of SMs; with more rows one CTA per head does more work
// per SM (measured: 8 packed rows 0.60 ms against 0.87 ms on pairs, 2 x 65,536 tokens 2.28
// against 3.62 ms; one row of 8192 tokens 0.297 ms against 0.242 ms).
bool use_pair(int N, int Vh, int nsm) { return 2 * (int64_t)N * Vh <= nsm; }

struct SegPlan {
    int S = 1;  // segments (1: the plain schedule on the caller's stream)
    int cs[kMaxSegments + 1] = {};
};

// Time from the end of the load stage to the end of the last recurrence launch.
double simulate_plan(const SegPlan& pl, int tasks_per_chunk, int nsm, int chain_ctas, double chunk_us) {
    using namespace seg_model;
    const int P = pl.S > 1 ? nsm - chain_ctas : nsm;  // SMs of the WY stream beside a running recurrence
    auto wy_us = [&](int chunks, int sms) {
        const int64_t tasks = (int64_t)chunks * tasks_per_chunk;
        return kWaveUs * (double)((tasks + sms - 1) / sms) + kWyFixedUs;
    };
    double wy_end = wy_us(pl.cs[1], nsm), chain_end = 0.0;
    for (int k = 0; k < pl.S; ++k) {
        const double start = chain_end > wy_end ? chain_end : wy_end;
        chain_end = start + kChainFixedUs + chunk_us * (pl.cs[k + 1] - pl.cs[k]);
        if (k + 1 < pl.S) wy_end += wy_us(pl.cs[k + 2] - pl.cs[k + 1], P);
    }
    return chain_end;
}

// The plan for N dense rows of T tokens: overlap needs a recurrence that leaves at least
// 32 SMs to the WY records and rows of at least 16 chunks.
SegPlan dense_plan(int Kh, int Vh, int N, int T, int nsm, bool pair) {
    const int per = (T + 63) / 64;
    SegPlan best;
    best.cs[1] = per;
    const int chain_ctas = (pair ? 2 : 1) * N * Vh;
    const double chunk_us = pair ? seg_model::kPairChainChunkUs : seg_model::kChainChunkUs;
    if (chain_ctas + 32 > nsm || per < 16) return best;
    const int tasks_per_chunk = N * Kh * ((Vh / Kh + wy::kHeads - 1) / wy::kHeads);
    double best_t = simulate_plan(best, tasks_per_chunk, nsm, chain_ctas, chunk_us);
    static const double kRho[] = {0.2, 0.3, 0.4, 0.5, 0.6, 0.7, 0.8, 0.9, 1.0, 1.1, 1.2, 1.35, 1.5, 1.75, 2.0};
    const int max_S = per < kMaxSegments ? per : kMaxSegments;
    for (int S = 2; S <= max_S; ++S) {
        for (double rho : kRho) {
            SegPlan c;
            c.S = S;
            double total = 0.0, f = 1.0;
            for (int k = 0; k < S; ++k, f *= rho) total += f;
            double acc = 0.0;
            f = 1.0;
            for (int k = 1; k <= S; ++k, f *= rho) {
                acc += f / total * per;
                const int v = (int)(acc + 0.5);
                const int lo = c.cs[k - 1] + 1, hi = per - (S - k);  // every segment keeps at least one chunk
                c.cs[k] = v < lo ? lo : (v > hi ? hi : v);
            }
            c.cs[S] = per;
            const double t = simulate_plan(c, tasks_per_chunk, nsm, chain_ctas, chunk_us);
            if (t < best_t) {
                best_t = t;
                best = c;
            }
        }
    }
    return best;
}

// Kernels one dense call launches under a plan: the load stage (or the fused in_proj GEMM),
// the history writer, then WY records and recurrence per segment.
int plan_launches(const SegPlan& pl) { return 2 + 2 * pl.S; }

// Everything one prefill call launches, with the workspace carved and the
// tensor maps built once.
struct PrefillPlan {
    int Kh, Vh, C, N, uniform_T, total, nsm;
    SeqIndex seq;
    const gdn_weights* w;
    const uint16_t *qkv, *a, *b;
    const float* init_conv;
    float* final_conv;
    uint16_t* out;
    const float* norm_w;
    const int* slots;  // state / history row of each packed row, or nullptr
    const FusedLoad* fused;  // load stage inside the in_proj GEMM (dense rows), or nullptr
    __half *Qs, *Ks, *Ql, *Kl, *Vs;
    float *Gs, *Bs;
    int* chunk_base;
    int* order;  // recurrence row order (packed rows), or nullptr
    uint8_t* rec;
    int rec_chunks;  // chunks the record array holds
    int state_rows;  // rows of the state / history arrays (the pool's, with slots)
    bool pair;       // recurrence on CTA pairs (64 value channels each), else one CTA per head
    CUtensorMap mK, mQ, mKl, mQl, mV, mZ, mO;

    int prep(int tok_begin, int tok_end, cudaStream_t st) const {
        if (tok_end <= tok_begin) return GDN_OK;
        if (fused != nullptr) return fused_prep(st);  // always the whole range
        PrepParams pp{};
        pp.Kh = Kh;
        pp.Vh = Vh;
        pp.C = C;
        pp.total = total;
        pp.tok_begin = tok_begin;
        pp.tok_end = tok_end;
        pp.seq = seq;
        pp.qkv = qkv;
        pp.a = a;
        pp.b = b;
        pp.conv_w = w->conv_w;
        pp.A_log = w->A_log;
        pp.dt_bias = w->dt_bias;
        pp.init_conv = init_conv;
        pp.slots = slots;
        pp.Qs = Qs;
        pp.Ks = Ks;
        pp.Ql = Ql;
        pp.Kl = Kl;
        pp.Vs = Vs;
        pp.Gs = Gs;
        pp.Bs = Bs;
        CUtensorMap mX;  // the CTAs' input rows x 256-channel boxes (rows outside the tensor read as zero)
        if (!make_map(&mX, qkv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)C, (uint64_t)total, kPrepBox, kPrepRows,
                      CU_TENSOR_MAP_SWIZZLE_NONE))
            return GDN_ERR_CUDA;
        int rc = smem_optin(reinterpret_cast<const void*>(gdn_prep_kernel), kPrepSmem);
        if (rc != GDN_OK) return rc;
        dim3 grid((tok_end - tok_begin + kPrepTokens - 1) / kPrepTokens, (2 * Kh + Vh + kPrepSlots - 1) / kPrepSlots);
        gdn_prep_kernel<<<grid, 256, kPrepSmem, st>>>(mX, pp);
        return cuda_status(cudaGetLastError());
    }
    // in_proj + load stage over all tokens: 128-row tiles advancing by 125 tokens
    int fused_prep(cudaStream_t st) const {
        GemmParams gp{};
        gp.M = total;
        gp.N = C + Vh * 128 + 2 * Vh;
        gp.K = fused->hidden;
        FusedPrep f{};
        f.Kh = Kh;
        f.Vh = Vh;
        f.T = uniform_T;
        f.cu = seq.cu;
        f.N = N;
        f.conv_w = w->conv_w;
        f.A_log = w->A_log;
        f.dt_bias = w->dt_bias;
        f.init_conv = init_conv;
        f.Qs = Qs;
        f.Ks = Ks;
        f.Ql = Ql;
        f.Kl = Kl;
        f.Vs = Vs;
        f.Gs = Gs;
        f.Bs = Bs;
        f.z = fused->z;
        f.conv_last = fused->conv_last;
        CUtensorMap mA, mW;
        if (!make_map(&mA, fused->x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)gp.K, (uint64_t)gp.M, gemm::BK,
                      gemm::BM, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !make_map(&mW, fused->w_in, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)gp.K, (uint64_t)gp.N, gemm::BK,
                      gemm::BN, CU_TENSOR_MAP_SWIZZLE_128B))
            return GDN_ERR_CUDA;
        int rc = smem_optin(reinterpret_cast<const void*>(gdn_gemm_kernel<1>), gemm::SMEM_BYTES);
        if (rc != GDN_OK) return rc;
        const int64_t ntiles = (int64_t)((gp.M + gemm::BM - 4) / (gemm::BM - 3)) * ((gp.N + gemm::BN - 1) / gemm::BN);
        const int grid = (int)(ntiles < nsm ? ntiles : nsm);
        gdn_gemm_kernel<1><<<grid, gemm::kThreads, gemm::SMEM_BYTES, st>>>(mA, mW, gp, f);
        return cuda_status(cudaGetLastError());
    }
    int conv_out(cudaStream_t st) const {
        if (final_conv == nullptr) return GDN_OK;
        if (fused != nullptr) {  // the rows' last tokens, staged by the fused load stage, and the history
            dim3 grid((C + 255) / 256, N);
            gdn_conv_merge_kernel<<<grid, 256, 0, st>>>(seq, C, fused->conv_last, init_conv, final_conv);
            return cuda_status(cudaGetLastError());
        }
        ConvOutParams cp{};
        cp.C = C;
        cp.N = N;
        cp.total = total;
        cp.seq = seq;
        cp.qkv = qkv;
        cp.init_conv = init_conv;
        cp.final_conv = final_conv;
        cp.slots = slots;
        dim3 grid((C + 255) / 256, N);
        gdn_conv_out_kernel<<<grid, 256, 0, st>>>(cp);
        return cuda_status(cudaGetLastError());
    }
    // WY records of nch chunks: all of them (win 0), or the window [c0, c0 + win) of every uniform row
    int wy_records(int64_t nch, int c0, int win, int grid_cap, cudaStream_t st) const {
        if (nch <= 0) return GDN_OK;
        WyParams wp{};
        wp.Kh = Kh;
        wp.Vh = Vh;
        wp.total = total;
        wp.seq = seq;
        wp.chunk_base = chunk_base;
        wp.nchunks = (int)nch;
        wp.c0 = c0;
        wp.win = win;
        wp.Gs = Gs;
        wp.Bs = Bs;
        wp.rec = rec;
        wp.rec_chunks = rec_chunks;
        int rc = smem_optin(reinterpret_cast<const void*>(gdn_wy_kernel), wy::SMEM_BYTES);
        if (rc != GDN_OK) return rc;
        const int ratio = Vh / Kh;
        const int64_t ntasks = nch * Kh * ((ratio + wy::kHeads - 1) / wy::kHeads);
        const int grid = (int)(ntasks < grid_cap ? ntasks : grid_cap);
        gdn_wy_kernel<<<grid, wy::kThreads, wy::SMEM_BYTES, st>>>(mK, mQ, mKl, mQl, wp);
        return cuda_status(cudaGetLastError());
    }
    // the recurrence over the chunk window [c0, c1) of every row (c1 < 0: to the end)
    int recurrence(int c0, int c1, const float* init_state, float* final_state, cudaStream_t st) const {
        ChunkParams cp{};
        cp.Kh = Kh;
        cp.Vh = Vh;
        cp.total = total;
        cp.seq = seq;
        cp.chunk_base = chunk_base;
        cp.order = order;
        cp.rec = rec;
        cp.init_state = init_state;
        cp.final_state = final_state;
        cp.norm_w = norm_w;
        cp.out = out;
        cp.c0 = c0;
        cp.c1 = c1;
        cp.slots = slots;
        cp.rec_chunks = rec_chunks;
        cp.state_rows = state_rows;
        if (pair) {
            int rc = smem_optin(reinterpret_cast<const void*>(gdn_chunk_pair_kernel), pair::SMEM_BYTES);
            if (rc != GDN_OK) return rc;
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(2 * Vh, N);
            cfg.blockDim = dim3(pair::kThreads);
            cfg.dynamicSmemBytes = pair::SMEM_BYTES;
            cfg.stream = st;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            return cuda_status(cudaLaunchKernelEx(&cfg, gdn_chunk_pair_kernel, mV, mQ, mK, mZ, mO, cp));
        }
        int rc = smem_optin(reinterpret_cast<const void*>(gdn_chunk_kernel), chunk::SMEM_BYTES);
        if (rc != GDN_OK) return rc;
        dim3 grid(Vh, N);
        gdn_chunk_kernel<<<grid, chunk::kThreads, chunk::SMEM_BYTES, st>>>(mV, mQ, mK, mZ, mO, cp);
        return cuda_status(cudaGetLastError());
    }
};

int prefill_impl(const gdn_dims* d, const gdn_weights* w, int32_t N, const int32_t* cu_dev, int32_t uniform_T,
                 int32_t total, int64_t nchunks, int64_t nchunks_planned, const uint16_t* qkv, const uint16_t* z,
                 const uint16_t* a, const uint16_t* b, const float* init_state, const float* init_conv, uint16_t* out,
                 float* final_state, float* final_conv, void* workspace, size_t workspace_bytes, cudaStream_t stream,
                 bool may_overlap, const int32_t* slots_dev = nullptr, const FusedLoad* fused = nullptr,
                 const OutProjTail* op = nullptr, int32_t pool_rows = 0) {
    const int Kh = d->num_k_heads, Vh = d->num_v_heads;
    const int C = (2 * Kh + Vh) * 128;
    const size_t state_bytes = (size_t)N * Vh * 128 * 128 * 4;
    const size_t conv_bytes = (size_t)N * 3 * C * 4;
    SeqIndex seq{cu_dev, uniform_T, N};

    if (N == 0) return GDN_OK;
    if (total == 0) {
        // Nothing to run: states and histories pass through.
        if (final_state != nullptr && final_state != init_state) {
            cudaError_t e = init_state ? cudaMemcpyAsync(final_state, init_state, state_bytes, cudaMemcpyDeviceToDevice, stream)
                                       : cudaMemsetAsync(final_state, 0, state_bytes, stream);
            if (e != cudaSuccess) return GDN_ERR_CUDA;
        }
        if (final_conv != nullptr && final_conv != init_conv) {
            cudaError_t e = init_conv ? cudaMemcpyAsync(final_conv, init_conv, conv_bytes, cudaMemcpyDeviceToDevice, stream)
                                      : cudaMemsetAsync(final_conv, 0, conv_bytes, stream);
            if (e != cudaSuccess) return GDN_ERR_CUDA;
        }
        return GDN_OK;
    }

    const Workspace ws = plan_workspace(d, total, N, nchunks_planned);
    if (nchunks > nchunks_planned || nchunks > INT32_MAX / d->num_v_heads) return GDN_ERR_INVALID_ARG;
    if (workspace == nullptr || workspace_bytes < ws.bytes) return GDN_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GDN_ERR_INVALID_ARG;
    uint8_t* wsb = static_cast<uint8_t*>(workspace);
    int dev = 0, nsm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return GDN_ERR_CUDA;

    PrefillPlan P{};
    P.Kh = Kh;
    P.Vh = Vh;
    P.C = C;
    P.N = N;
    P.uniform_T = uniform_T;
    P.total = total;
    P.nsm = nsm;
    P.seq = seq;
    P.w = w;
    P.qkv = qkv;
    P.a = a;
    P.b = b;
    P.init_conv = init_conv;
    P.final_conv = final_conv;
    P.out = out;
    P.norm_w = w->norm_w;
    P.slots = slots_dev;
    P.fused = fused;
    P.Qs = reinterpret_cast<__half*>(wsb + ws.off_q);
    P.Ks = reinterpret_cast<__half*>(wsb + ws.off_k);
    P.Ql = reinterpret_cast<__half*>(wsb + ws.off_ql);
    P.Kl = reinterpret_cast<__half*>(wsb + ws.off_kl);
    P.Vs = reinterpret_cast<__half*>(wsb + ws.off_v);
    P.Gs = reinterpret_cast<float*>(wsb + ws.off_g);
    P.Bs = reinterpret_cast<float*>(wsb + ws.off_b);
    P.chunk_base = cu_dev ? reinterpret_cast<int*>(wsb + ws.off_cb) : nullptr;
    P.order = cu_dev ? P.chunk_base + N + 1 : nullptr;
    P.rec = wsb + ws.off_rec;
    P.rec_chunks = (int)nchunks_planned;
    P.state_rows = slots_dev != nullptr ? pool_rows : N;
    P.pair = use_pair(N, Vh, nsm);
    if (!make_map(&P.mK, P.Ks, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (uint64_t)Kh * 128, total, 64, 64,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&P.mKl, P.Kl, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (uint64_t)Kh * 128, total, 64, 64,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&P.mQl, P.Ql, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (uint64_t)Kh * 128, total, 64, 64,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&P.mQ, P.Qs, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (uint64_t)Kh * 128, total, 64, 64,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&P.mV, P.Vs, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (uint64_t)Vh * 128, total, 64, 64,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&P.mZ, z, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)Vh * 128, total, P.pair ? 64 : 128, 64,
                  P.pair ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !make_map(&P.mO, out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)Vh * 128, total, P.pair ? 64 : 128, 64,
                  P.pair ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE))
        return GDN_ERR_CUDA;

    // Overlapped schedule (dense rows that leave most SMs idle during the recurrence):
    // the load stage runs over all tokens first; then the rows' chunks are cut into S
    // segments and the WY records of segment s+1 run on the low-priority stream (a
    // persistent grid that leaves the recurrence its SMs) while the recurrence of
    // segment s runs on the high-priority one, each segment's recurrence starting from
    // the state the previous one left in final_state.
    const int chain_ctas = (P.pair ? 2 : 1) * N * Vh;
    SegPlan plan;
    if (may_overlap && cu_dev == nullptr && final_state != nullptr)
        plan = dense_plan(Kh, Vh, N, uniform_T, nsm, P.pair);
    const int S = plan.S;
    const int* cs = plan.cs;
    if (S > 1) {
        std::lock_guard<std::mutex> lock(g_side_mu);
        SideStreams* ss = nullptr;
        int st = side_streams(dev, &ss);
        if (st != GDN_OK) return st;
        if (cudaEventRecord(ss->fork, stream) != cudaSuccess || cudaStreamWaitEvent(ss->prod, ss->fork, 0) != cudaSuccess ||
            cudaStreamWaitEvent(ss->chain, ss->fork, 0) != cudaSuccess)
            return GDN_ERR_CUDA;
        if ((st = P.prep(0, total, ss->prod)) != GDN_OK) return st;
        for (int k = 0; k < S; ++k) {
            const int win = cs[k + 1] - cs[k];
            const int cap = k == 0 ? nsm : nsm - chain_ctas;  // leave the recurrence its SMs
            if ((st = P.wy_records((int64_t)N * win, cs[k], win, cap, ss->prod)) != GDN_OK) return st;
            if (cudaEventRecord(ss->seg[k], ss->prod) != cudaSuccess ||
                cudaStreamWaitEvent(ss->chain, ss->seg[k], 0) != cudaSuccess)
                return GDN_ERR_CUDA;
            if ((st = P.recurrence(cs[k], k + 1 < S ? cs[k + 1] : -1, k == 0 ? init_state : final_state, final_state,
                                   ss->chain)) != GDN_OK)
                return st;
            if (op != nullptr && cudaEventRecord(ss->rec[k], ss->chain) != cudaSuccess) return GDN_ERR_CUDA;
        }
        // out_proj on the lowest-priority stream: when the recurrence leaves at least half the
        // SMs, each segment's tokens as soon as that segment's recurrence has written them (it
        // takes the SMs the WY records leave); otherwise all tokens after the last segment (a
        // persistent GEMM grid between segments holds SMs the next recurrence launch needs:
        // one row on CTA pairs, 96 SMs, measured 0.86 ms per segment against 0.82 ms after)
        const bool per_segment = 2 * chain_ctas <= nsm;
        for (int k = per_segment ? 0 : S - 1; op != nullptr && k < S; ++k) {
            if (cudaStreamWaitEvent(ss->tail, ss->rec[k], 0) != cudaSuccess) return GDN_ERR_CUDA;
            const int64_t a0 = per_segment ? (int64_t)cs[k] * 64 : 0;
            const int64_t a1 = k + 1 < S ? (int64_t)cs[k + 1] * 64 : uniform_T;
            for (int n = 0; n < N; ++n)
                if ((st = out_proj_range(*op, out, Vh * 128, (int64_t)n * uniform_T + a0,
                                         (int64_t)n * uniform_T + (a1 < uniform_T ? a1 : uniform_T), ss->tail)) != GDN_OK)
                    return st;
        }
        // the final histories: after the load stage has read the old ones, off the path to the
        // first recurrence segment (beside the last one)
        if ((st = P.conv_out(ss->prod)) != GDN_OK) return st;
        if (cudaEventRecord(ss->prod_done, ss->prod) != cudaSuccess ||
            cudaEventRecord(ss->chain_done, ss->chain) != cudaSuccess ||
            cudaStreamWaitEvent(stream, ss->prod_done, 0) != cudaSuccess ||
            cudaStreamWaitEvent(stream, ss->chain_done, 0) != cudaSuccess)
            return GDN_ERR_CUDA;
        if (op != nullptr && (cudaEventRecord(ss->tail_done, ss->tail) != cudaSuccess ||
                              cudaStreamWaitEvent(stream, ss->tail_done, 0) != cudaSuccess))
            return GDN_ERR_CUDA;
        return GDN_OK;
    }

    // Plain schedule on the caller's stream.
    int st = P.prep(0, total, stream);  // 1. load stage: conv + silu, L2 norms, gates
    if (st != GDN_OK) return st;
    if ((st = P.conv_out(stream)) != GDN_OK) return st;  // 2. final history (after the load stage read it)
    if (P.chunk_base != nullptr) {                        // 3. first chunk of every packed row
        gdn_chunk_base_kernel<<<1, 1024, 0, stream>>>(cu_dev, N, P.chunk_base, P.order);
        if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    }
    if ((st = P.wy_records(nchunks, 0, 0, nsm, stream)) != GDN_OK) return st;  // 4. WY records, all chunks
    if ((st = P.recurrence(0, -1, init_state, final_state, stream)) != GDN_OK) return st;  // 5. recurrence + gated norm
    return op != nullptr ? out_proj_range(*op, out, Vh * 128, 0, total, stream) : GDN_OK;  // 6. out_proj
}

int check_io(int32_t total, const uint16_t* qkv, const uint16_t* z, const uint16_t* a, const uint16_t* b,
             const uint16_t* out, const float* init_state, const float* init_conv, const float* final_state,
             const float* final_conv) {
    if (total > 0) {
        if (!qkv || !z || !a || !b || !out) return GDN_ERR_INVALID_ARG;
        if (!aligned16(qkv) || !aligned16(z) || !aligned16(out)) return GDN_ERR_INVALID_ARG;
        if ((reinterpret_cast<uintptr_t>(a) & 1u) || (reinterpret_cast<uintptr_t>(b) & 1u)) return GDN_ERR_INVALID_ARG;
    }
    const void* fs[4] = {init_state, init_conv, final_state, final_conv};
    for (const void* p : fs)
        if (p != nullptr && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// Scratch of gdn_prefill_noalloc: one fixed array per device, never freed.
// Host code must not pass g_noalloc_scratch itself to a kernel (on the host
// it names a stand-in, not the device address): its device address is looked
// up once per device below.
static __device__ __align__(256) uint8_t g_noalloc_scratch[GDN_NOALLOC_SCRATCH_BYTES];

// The address is cached per CUDA context (by the driver's unique context id), so a
// context that replaced an earlier one on the same device (after cudaDeviceReset) gets
// its own lookup instead of a stale pointer.
std::mutex g_noalloc_mu;
struct NoallocEntry {
    unsigned long long ctx_id;
    void* addr;
};
std::vector<NoallocEntry> g_noalloc_addr;

using PfnCtxGetCurrent = CUresult (*)(CUcontext*);
using PfnCtxGetId = CUresult (*)(CUcontext, unsigned long long*);

void* driver_fn(const char* name) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion(name, &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return nullptr;
    return p;
}

// Unique id of the current context (0 if there is none or the driver cannot say).
unsigned long long current_ctx_id() {
    static PfnCtxGetCurrent get_cur = nullptr;
    static PfnCtxGetId get_id = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        get_cur = reinterpret_cast<PfnCtxGetCurrent>(driver_fn("cuCtxGetCurrent"));
        get_id = reinterpret_cast<PfnCtxGetId>(driver_fn("cuCtxGetId"));
    });
    CUcontext ctx = nullptr;
    unsigned long long id = 0;
    if (get_cur == nullptr || get_id == nullptr || get_cur(&ctx) != CUDA_SUCCESS || ctx == nullptr ||
        get_id(ctx, &id) != CUDA_SUCCESS)
        return 0;
    return id;
}

// Device address of g_noalloc_scratch in the current context (resolved on first use there;
// cudaGetSymbolAddress also makes the device's primary context current if it was not).
int noalloc_scratch(void** out) {
    std::lock_guard<std::mutex> lock(g_noalloc_mu);
    unsigned long long id = current_ctx_id();
    for (const NoallocEntry& e : g_noalloc_addr)
        if (id != 0 && e.ctx_id == id) {
            *out = e.addr;
            return GDN_OK;
        }
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || p == nullptr) return GDN_ERR_CUDA;
    if (id == 0) id = current_ctx_id();
    if (id != 0) g_noalloc_addr.push_back(NoallocEntry{id, p});
    *out = p;
    return GDN_OK;
}

// Host check of a slot table: 0 <= slots[r] < pool_rows, no slot twice.
int check_slots(const int32_t* slots_host, int32_t rows, int32_t pool_rows) {
    if (slots_host == nullptr || pool_rows <= 0) return GDN_ERR_INVALID_ARG;
    std::vector<unsigned char> seen((size_t)pool_rows, 0);
    for (int32_t r = 0; r < rows; ++r) {
        const int32_t sl = slots_host[r];
        if (sl < 0 || sl >= pool_rows || seen[(size_t)sl]) return GDN_ERR_INVALID_ARG;
        seen[(size_t)sl] = 1;
    }
    return GDN_OK;
}

// The decode launch: rows batch rows, state / history rows through slots (or nullptr).
int decode_impl(const gdn_dims* dims, const gdn_weights* w, int32_t rows, const uint16_t* qkv, const uint16_t* z,
                const uint16_t* a, const uint16_t* b, float* state, float* conv, uint16_t* out, const int32_t* slots,
                int32_t ntok, void* stream, int32_t pool_rows) {
    int st = GDN_OK;
    if (!state || !conv || !aligned16(state) || !aligned16(conv)) return GDN_ERR_INVALID_ARG;
    if ((st = check_io(rows, qkv, z, a, b, out, nullptr, nullptr, nullptr, nullptr)) != GDN_OK) return st;
    if ((st = check_device()) != GDN_OK) return st;
    DecodeParams p{};
    p.Kh = dims->num_k_heads;
    p.Vh = dims->num_v_heads;
    p.C = (2 * p.Kh + p.Vh) * 128;
    p.rows = rows;
    p.qkv = qkv;
    p.z = z;
    p.a = a;
    p.b = b;
    p.conv_w = w->conv_w;
    p.A_log = w->A_log;
    p.dt_bias = w->dt_bias;
    p.norm_w = w->norm_w;
    p.state = state;
    p.conv = conv;
    p.out = out;
    p.slots = slots;
    p.pool_rows = pool_rows;
    p.ntok = ntok;
    const void* kernels[4] = {reinterpret_cast<const void*>(gdn_decode_kernel<1, false>),
                              reinterpret_cast<const void*>(gdn_decode_kernel<dec::kMaxTokens, false>),
                              reinterpret_cast<const void*>(gdn_decode_kernel<1, true>),
                              reinterpret_cast<const void*>(gdn_decode_kernel<dec::kMaxTokens, true>)};
    for (const void* k : kernels)
        if ((st = smem_optin(k, dec::kSmemLimit)) != GDN_OK) return st;
    int dev = 0, nsm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return GDN_ERR_CUDA;
    // Work item = (row, q/k head) with its value heads, persistent CTAs walking the items.  A batch
    // small enough that one CTA per value head still fits in one wave splits each q/k group over a
    // cluster of Vh/Kh CTAs, one value head each (one item per CTA): 1 row 9.6 -> 6.3 us, 2 rows
    // 9.9 -> 6.5 us; with more than one wave the persistent grouping is faster.
    const int Gfull = p.Vh / p.Kh;
    const bool split = Gfull > 1 && rows * p.Kh * Gfull <= nsm;
    const int kmax = ntok == 1 ? 1 : dec::kMaxTokens;  // the kernel instantiation
    const dec::Plan dplan = dec::plan(split ? 1 : Gfull, ntok, dec::groups(kmax));
    if (dplan.stages < 2) return GDN_ERR_UNSUPPORTED;  // the group's inputs of ntok tokens leave no room
    p.nitems = rows * p.Kh * (split ? Gfull : 1);
    const int grid = split ? p.nitems : (p.nitems < nsm ? p.nitems : nsm);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(dec::threads(kmax));
    cfg.dynamicSmemBytes = dplan.smem_bytes;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = Gfull;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = split ? attr : nullptr;
    cfg.numAttrs = split ? 1 : 0;
    if (split)
        return cuda_status(ntok == 1 ? cudaLaunchKernelEx(&cfg, gdn_decode_kernel<1, true>, p)
                                     : cudaLaunchKernelEx(&cfg, gdn_decode_kernel<dec::kMaxTokens, true>, p));
    return cuda_status(ntok == 1 ? cudaLaunchKernelEx(&cfg, gdn_decode_kernel<1, false>, p)
                                 : cudaLaunchKernelEx(&cfg, gdn_decode_kernel<dec::kMaxTokens, false>, p));
}


// C = A W^T over bf16 A [M][K] and W [N][K], columns routed to the segments of gp.
int gemm_launch(const uint16_t* A, const uint16_t* W, GemmParams gp, cudaStream_t stream) {
    if (gp.M == 0 || gp.N == 0) return GDN_OK;
    if (gp.K <= 0 || gp.K % gemm::BK != 0) return GDN_ERR_UNSUPPORTED;
    if (!A || !W || !aligned16(A) || !aligned16(W)) return GDN_ERR_INVALID_ARG;
    for (int i = 0; i < gp.nseg; ++i)
        if (gp.seg[i].dst == nullptr || (reinterpret_cast<uintptr_t>(gp.seg[i].dst) & 1u)) return GDN_ERR_INVALID_ARG;
    int st = check_device();
    if (st != GDN_OK) return st;
    CUtensorMap mA, mW;
    if (!make_map(&mA, A, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)gp.K, (uint64_t)gp.M, gemm::BK, gemm::BM,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&mW, W, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)gp.K, (uint64_t)gp.N, gemm::BK, gemm::BN,
                  CU_TENSOR_MAP_SWIZZLE_128B))
        return GDN_ERR_CUDA;
    st = smem_optin(reinterpret_cast<const void*>(gdn_gemm_kernel<0>), gemm::SMEM_BYTES);
    if (st != GDN_OK) return st;
    int dev = 0, nsm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return GDN_ERR_CUDA;
    const int64_t ntiles = (int64_t)((gp.M + gemm::BM - 1) / gemm::BM) * ((gp.N + gemm::BN - 1) / gemm::BN);
    const int grid = (int)(ntiles < nsm ? ntiles : nsm);
    gdn_gemm_kernel<0><<<grid, gemm::kThreads, gemm::SMEM_BYTES, stream>>>(mA, mW, gp, FusedPrep{});
    return cuda_status(cudaGetLastError());
}

// Workspace of gdn_prefill_hidden: the prefill workspace, then z, then either the
// rows' staged histories (fused load stage) or the unfused in_proj outputs.
struct HiddenLayout {
    bool fused;
    size_t off_z, off_conv, off_qkv, off_b, off_a, bytes;
};

// The fused load stage needs whole 256-column tiles of qkv and of z, and b and a in one tile.
bool fused_load_ok(const gdn_dims* d) {
    const int Kh = d->num_k_heads, Vh = d->num_v_heads;
    return (2 * Kh + Vh) % 2 == 0 && Vh % 2 == 0 && 2 * Vh <= gemm::BN;
}

// rows: N packed rows (or B dense rows) of `total` tokens in all; nchunks: the prefill's chunk plan
HiddenLayout hidden_layout(const gdn_dims* d, int32_t rows, int64_t total, int64_t nchunks) {
    HiddenLayout L{};
    const int Kh = d->num_k_heads, Vh = d->num_v_heads;
    const size_t C = (size_t)(2 * Kh + Vh) * 128;
    L.fused = fused_load_ok(d);
    L.off_z = plan_workspace(d, total, rows, nchunks).bytes;
    size_t o = L.off_z + align_up((size_t)total * Vh * 128 * 2);
    if (L.fused) {
        L.off_conv = o;
        o += align_up((size_t)rows * 3 * C * 4);
    } else {
        L.off_qkv = o;
        o += align_up((size_t)total * C * 2);
        L.off_b = o;
        o += align_up((size_t)total * Vh * 2);
        L.off_a = o;
        o += align_up((size_t)total * Vh * 2);
    }
    L.bytes = o;
    return L;
}

// The prefill from hidden states over dense rows (cu_dev == nullptr, uniform_T) or packed rows:
// the fused in_proj + load stage where the head counts allow, else in_proj then the prefill.
int prefill_hidden_impl(const gdn_dims* dims, const gdn_weights* w, int32_t N, const int32_t* cu_dev,
                        int32_t uniform_T, int32_t total, int64_t nch, int64_t nch_planned, int32_t hidden,
                        const uint16_t* x, const uint16_t* w_in, const float* init_state, const float* init_conv,
                        uint16_t* out, float* final_state, float* final_conv, void* workspace,
                        size_t workspace_bytes, void* stream) {
    int st = GDN_OK;
    if (hidden % gemm::BK != 0) return GDN_ERR_UNSUPPORTED;
    if (total > 0 && (!x || !w_in || !out || !aligned16(x) || !aligned16(w_in) || !aligned16(out)))
        return GDN_ERR_INVALID_ARG;
    const void* fs[4] = {init_state, init_conv, final_state, final_conv};
    for (const void* p : fs)
        if (p != nullptr && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    if ((st = check_device()) != GDN_OK) return st;
    const HiddenLayout L = hidden_layout(dims, N, total, nch_planned);
    if (total > 0 && (workspace == nullptr || workspace_bytes < L.bytes)) return GDN_ERR_WORKSPACE;
    if (workspace != nullptr && !aligned16(workspace)) return GDN_ERR_INVALID_ARG;
    uint8_t* wsb = static_cast<uint8_t*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool dense = cu_dev == nullptr;
    uint16_t* z = total > 0 ? reinterpret_cast<uint16_t*>(wsb + L.off_z) : nullptr;
    if (total > 0 && L.fused) {
        FusedLoad fl{x, w_in, hidden, z, reinterpret_cast<float*>(wsb + L.off_conv)};
        return prefill_impl(dims, w, N, cu_dev, uniform_T, total, nch, nch_planned, nullptr, z, nullptr, nullptr,
                            init_state, init_conv, out, final_state, final_conv, workspace, L.off_z, s, dense,
                            nullptr, &fl);
    }
    // head counts the fused tiles do not cover: in_proj into the workspace, then the prefill over it
    uint16_t* qkv = total > 0 ? reinterpret_cast<uint16_t*>(wsb + L.off_qkv) : nullptr;
    uint16_t* bb = total > 0 ? reinterpret_cast<uint16_t*>(wsb + L.off_b) : nullptr;
    uint16_t* aa = total > 0 ? reinterpret_cast<uint16_t*>(wsb + L.off_a) : nullptr;
    if (total > 0 && (st = gdn_in_proj(dims, total, hidden, x, w_in, qkv, z, bb, aa, stream)) != GDN_OK) return st;
    return prefill_impl(dims, w, N, cu_dev, uniform_T, total, nch, nch_planned, qkv, z, aa, bb, init_state,
                        init_conv, out, final_state, final_conv, workspace, total > 0 ? L.off_z : 0, s, dense);
}

}  // namespace

extern "C" {

int gdn_in_proj(const gdn_dims* dims, int32_t T, int32_t hidden, const uint16_t* x, const uint16_t* w_in,
                uint16_t* qkv, uint16_t* z, uint16_t* b, uint16_t* a, void* stream) {
    NvtxRange nvtx_range("gdn_in_proj");
    int st = check_dims(dims);
    if (st != GDN_OK) return st;
    if (T < 0 || hidden <= 0) return GDN_ERR_INVALID_ARG;
    if (T == 0) return GDN_OK;
    const int Vh = dims->num_v_heads, D = dims->head_dim;
    const int C = (2 * dims->num_k_heads + Vh) * D;
    GemmParams gp{};
    gp.M = T;
    gp.N = C + Vh * D + 2 * Vh;
    gp.K = hidden;
    gp.nseg = 4;
    gp.seg[0] = GemmSegment{0, C, qkv};
    gp.seg[1] = GemmSegment{C, Vh * D, z};
    gp.seg[2] = GemmSegment{C + Vh * D, Vh, b};
    gp.seg[3] = GemmSegment{C + Vh * D + Vh, Vh, a};
    return gemm_launch(x, w_in, gp, static_cast<cudaStream_t>(stream));
}

int gdn_out_proj(const gdn_dims* dims, int32_t T, int32_t hidden, const uint16_t* y, const uint16_t* w_out,
                 uint16_t* out, void* stream) {
    NvtxRange nvtx_range("gdn_out_proj");
    int st = check_dims(dims);
    if (st != GDN_OK) return st;
    if (T < 0 || hidden <= 0) return GDN_ERR_INVALID_ARG;
    if (T == 0) return GDN_OK;
    GemmParams gp{};
    gp.M = T;
    gp.N = hidden;
    gp.K = dims->num_v_heads * dims->head_dim;
    gp.nseg = 1;
    gp.seg[0] = GemmSegment{0, hidden, out};
    return gemm_launch(y, w_out, gp, static_cast<cudaStream_t>(stream));
}


size_t gdn_prefill_hidden_workspace_size(const gdn_dims* dims, int32_t B, int32_t T) {
    if (check_dims(dims) != GDN_OK || B < 0 || T < 0) return 0;
    const int64_t total = (int64_t)B * T;
    if (total > INT32_MAX) return 0;
    return hidden_layout(dims, B, total, (int64_t)B * ((T + 63) / 64)).bytes;
}

int gdn_prefill_hidden(const gdn_dims* dims, const gdn_weights* w, int32_t B, int32_t T, int32_t hidden,
                       const uint16_t* x, const uint16_t* w_in, const float* init_state, const float* init_conv,
                       uint16_t* out, float* final_state, float* final_conv, void* workspace, size_t workspace_bytes,
                       void* stream) {
    NvtxRange nvtx_range("gdn_prefill_hidden");
    int st = check_dims(dims);
    if (st != GDN_OK) return st;
    if ((st = check_weights(w)) != GDN_OK) return st;
    if (B < 0 || T < 0 || B > 65535 || hidden <= 0) return GDN_ERR_INVALID_ARG;
    const int64_t total = (int64_t)B * T;
    if (total > INT32_MAX) return GDN_ERR_INVALID_ARG;
    const int64_t nch = (int64_t)B * ((T + 63) / 64);
    return prefill_hidden_impl(dims, w, B, nullptr, T, (int32_t)total, nch, nch, hidden, x, w_in, init_state,
                               init_conv, out, final_state, final_conv, workspace, workspace_bytes, stream);
}

size_t gdn_prefill_hidden_varlen_workspace_size(const gdn_dims* dims, int32_t N, int32_t total_T) {
    if (check_dims(dims) != GDN_OK || N < 0 || total_T < 0) return 0;
    return hidden_layout(dims, N, total_T, chunk_bound(N, total_T)).bytes;
}

int gdn_prefill_hidden_varlen(const gdn_dims* dims, const gdn_weights* w, int32_t N, const int32_t* cu_host,
                              const int32_t* cu_dev, int32_t total_T, int32_t hidden, const uint16_t* x,
                              const uint16_t* w_in, const float* init_state, const float* init_conv, uint16_t* out,
                              float* final_state, float* final_conv, void* workspace, size_t workspace_bytes,
                              void* stream) {
    NvtxRange nvtx_range("gdn_prefill_hidden_varlen");
    int st = check_dims(dims);
    if (st != GDN_OK) return st;
    if ((st = check_weights(w)) != GDN_OK) return st;
    if (N < 0 || N > 65535 || total_T < 0 || hidden <= 0) return GDN_ERR_INVALID_ARG;
    if (cu_host == nullptr || (N > 0 && cu_dev == nullptr)) return GDN_ERR_INVALID_ARG;
    if (cu_host[0] != 0 || cu_host[N] != total_T) return GDN_ERR_INVALID_ARG;
    for (int32_t i = 0; i < N; ++i)
        if (cu_host[i + 1] < cu_host[i]) return GDN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(cu_dev) & 3u) != 0) return GDN_ERR_INVALID_ARG;
    int64_t nch = 0;
    for (int32_t i = 0; i < N; ++i) nch += (cu_host[i + 1] - cu_host[i] + 63) / 64;
    return prefill_hidden_impl(dims, w, N, cu_dev, 0, total_T, nch, chunk_bound(N, total_T), hidden, x, w_in,
                               init_state, init_conv, out, final_state, final_conv, workspace, workspace_bytes,
                               stream);
}

// The schedule of a dense prefill on a device with nsm SMs (arguments already checked).
void schedule_for(const gdn_dims* dims, int32_t B, int32_t T, int32_t from_hidden, int nsm, int32_t* segments,
                  int32_t* launches) {
    const bool fused = from_hidden != 0 && fused_load_ok(dims);
    const SegPlan pl =
        dense_plan(dims->num_k_heads, dims->num_v_heads, B, T, nsm, use_pair(B, dims->num_v_heads, nsm));
    *segments = pl.S;
    *launches = plan_launches(pl) + (from_hidden != 0 && !fused ? 1 : 0);  // + the unfused in_proj
}

int schedule_args(const gdn_dims* dims, int32_t B, int32_t T, int32_t* segments, int32_t* launches) {
    int st = check_dims(dims);
    if (st != GDN_OK) return st;
    if (B < 0 || T < 0 || B > 65535 || (int64_t)B * T > INT32_MAX || !segments || !launches)
        return GDN_ERR_INVALID_ARG;
    *segments = 0;
    *launches = 0;
    return GDN_OK;
}

int gdn_prefill_schedule(const gdn_dims* dims, int32_t B, int32_t T, int32_t from_hidden, int32_t* segments,
                         int32_t* launches) {
    int st = schedule_args(dims, B, T, segments, launches);
    if (st != GDN_OK || B == 0 || T == 0) return st;
    if ((st = check_device()) != GDN_OK) return st;
    int dev = 0, nsm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return GDN_ERR_CUDA;
    schedule_for(dims, B, T, from_hidden, nsm, segments, launches);
    return GDN_OK;
}

int gdn_prefill_schedule_nsm(const gdn_dims* dims, int32_t B, int32_t T, int32_t from_hidden, int32_t nsm,
                             int32_t* segments, int32_t* launches) {
    int st = schedule_args(dims, B, T, segments, launches);
    if (st != GDN_OK) return st;
    if (nsm < 1) return GDN_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return GDN_OK;
    schedule_for(dims, B, T, from_hidden, nsm, segments, launches);
    return GDN_OK;
}

size_t gdn_prefill_workspace_size(const gdn_dims* dims, int32_t B, int32_t T) {
    if (check_dims(dims) != GDN_OK || B < 0 || T < 0) return 0;
    const int64_t total = (int64_t)B * T;
    if (total > INT32_MAX) return 0;
    return plan_workspace(dims, total, B, (int64_t)B * ((T + 63) / 64)).bytes;
}

size_t gdn_prefill_out_workspace_size(const gdn_dims* dims, int32_t B, int32_t T) {
    if (check_dims(dims) != GDN_OK || B < 0 || T < 0) return 0;
    const int64_t total = (int64_t)B * T;
    if (total > INT32_MAX) return 0;
    return plan_workspace(dims, total, B, (int64_t)B * ((T + 63) / 64)).bytes +
           align_up((size_t)total * dims->num_v_heads * 128 * 2);
}

int gdn_prefill_out(const gdn_dims* dims, const gdn_weights* w, int32_t B, int32_t T, int32_t hidden,
                    const uint16_t* qkv, const uint16_t* z, const uint16_t* a, const uint16_t* b,
                    const float* init_state, const float* init_conv, const uint16_t* w_out, uint16_t* out,
                    float* final_state, float* final_conv, void* workspace, size_t workspace_bytes, void* stream) {
    NvtxRange nvtx_range("gdn_prefill_out");
    int st = check_dims(dims);
    if (st != GDN_OK) return st;
    if ((st = check_weights(w)) != GDN_OK) return st;
    if (B < 0 || T < 0 || B > 65535 || hidden <= 0) return GDN_ERR_INVALID_ARG;
    if (hidden % 8 != 0) return GDN_ERR_UNSUPPORTED;
    const int64_t total = (int64_t)B * T;
    if (total > INT32_MAX) return GDN_ERR_INVALID_ARG;
    if ((st = check_io((int32_t)total, qkv, z, a, b, out, init_state, init_conv, final_state, final_conv)) != GDN_OK)
        return st;
    if (total > 0 && (w_out == nullptr || !aligned16(w_out))) return GDN_ERR_INVALID_ARG;
    if ((st = check_device()) != GDN_OK) return st;
    const int64_t nch = (int64_t)B * ((T + 63) / 64);
    const size_t ws_mixer = plan_workspace(dims, total, B, nch).bytes;
    if (total > 0 && (workspace == nullptr || workspace_bytes < gdn_prefill_out_workspace_size(dims, B, T)))
        return GDN_ERR_WORKSPACE;
    uint16_t* y = total > 0 ? reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + ws_mixer) : nullptr;
    const OutProjTail op{w_out, hidden, out};
    return prefill_impl(dims, w, B, nullptr, T, (int32_t)total, nch, nch, qkv, z, a, b, init_state, init_conv, y,
                        final_state, final_conv, workspace, ws_mixer, static_cast<cudaStream_t>(stream), true, nullptr,
                        nullptr, &op);
}

size_t gdn_prefill_varlen_workspace_size(const gdn_dims* dims, int32_t N, int32_t total_T) {
    if (check_dims(dims) != GDN_OK || N < 0 || total_T < 0) return 0;
    return plan_workspace(dims, total_T, N, chunk_bound(N, total_T)).bytes;
}

int gdn_prefill(const gdn_dims* dims, const gdn_weights* w, int32_t B, int32_t T, const uint16_t* qkv,
                const uint16_t* z, const uint16_t* a, const uint16_t* b, const float* init_state,
                const float* init_conv, uint16_t* out, float* final_state, float* final_conv, void* workspace,
                size_t workspace_bytes, void* stream) {
    NvtxRange nvtx_range("gdn_prefill");
    int st = check_dims(dims);
    if (st != GDN_OK) return st;
    if ((st = check_weights(w)) != GDN_OK) return st;
    if (B < 0 || T < 0 || B > 65535) return GDN_ERR_INVALID_ARG;
    const int64_t total = (int64_t)B * T;
    if (total > INT32_MAX) return GDN_ERR_INVALID_ARG;
    if ((st = check_io((int32_t)total, qkv, z, a, b, out, init_state, init_conv, final_state, final_conv)) != GDN_OK)
        return st;
    if ((st = check_device()) != GDN_OK) return st;
    const int64_t nch = (int64_t)B * ((T + 63) / 64);
    return prefill_impl(dims, w, B, nullptr, T, (int32_t)total, nch, nch, qkv, z, a, b, init_state, init_conv, out,
                        final_state, final_conv, workspace, workspace_bytes, static_cast<cudaStream_t>(stream), true);
}

int gdn_prefill_varlen(const gdn_dims* dims, const gdn_weights* w, int32_t N, const int32_t* cu_host,
                       const int32_t* cu_dev, int32_t total_T, const uint16_t* qkv, const uint16_t* z,
                       const uint16_t* a, const uint16_t* b, const float* init_state, const float* init_conv,
                       uint16_t* out, float* final_state, float* final_conv, void* workspace, size_t workspace_bytes,
                       void* stream) {
    NvtxRange nvtx_range("gdn_prefill_varlen");
    int st = check_dims(dims);
    if (st != GDN_OK) return st;
    if ((st = check_weights(w)) != GDN_OK) return st;
    if (N < 0 || N > 65535 || total_T < 0) return GDN_ERR_INVALID_ARG;
    if (cu_host == nullptr || (N > 0 && cu_dev == nullptr)) return GDN_ERR_INVALID_ARG;
    if (cu_host[0] != 0 || cu_host[N] != total_T) return GDN_ERR_INVALID_ARG;
    for (int32_t i = 0; i < N; ++i)
        if (cu_host[i + 1] < cu_host[i]) return GDN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(cu_dev) & 3u) != 0) return GDN_ERR_INVALID_ARG;
    if ((st = check_io(total_T, qkv, z, a, b, out, init_state, init_conv, final_state, final_conv)) != GDN_OK)
        return st;
    if ((st = check_device()) != GDN_OK) return st;
    int64_t nch = 0;
    for (int32_t i = 0; i < N; ++i) nch += (cu_host[i + 1] - cu_host[i] + 63) / 64;
    return prefill_impl(dims, w, N, cu_dev, 0, total_T, nch, chunk_bound(N, total_T), qkv, z, a, b, init_state,
                        init_conv, out, final_state, final_conv, workspace, workspace_bytes,
                        static_cast<cudaStream_t>(stream), false);
}

int gdn_decode(const gdn_dims* dims, const gdn_weights* w, int32_t rows, const uint16_t* qkv, const uint16_t* z,
               const uint16_t* a, const uint16_t* b, float* state, float* conv, uint16_t* out, void* stream) {
    NvtxRange nvtx_range("gdn_decode");
    int st = check_dims(dims);
    if (st != GDN_OK) return st;
    if ((st = check_weights(w)) != GDN_OK) return st;
    if (rows < 0 || rows > 65535) return GDN_ERR_INVALID_ARG;
    if (rows == 0) return GDN_OK;
    return decode_impl(dims, w, rows, qkv, z, a, b, state, conv, out, nullptr, 1, stream, rows);
}

int gdn_decode_multi(const gdn_dims* dims, const gdn_weights* w, int32_t rows, int32_t ntok, const uint16_t* qkv,
                     const uint16_t* z, const uint16_t* a, const uint16_t* b, float* state, float* conv, uint16_t* out,
                     void* stream) {
    NvtxRange nvtx_range("gdn_decode_multi");
    int st = check_dims(dims);
    if (st != GDN_OK) return st;
    if ((st = check_weights(w)) != GDN_OK) return st;
    if (rows < 0 || rows > 65535 || ntok < 1) return GDN_ERR_INVALID_ARG;
    if (ntok > dec::kMaxTokens) return GDN_ERR_UNSUPPORTED;
    if (rows == 0) return GDN_OK;
    return decode_impl(dims, w, rows, qkv, z, a, b, state, conv, out, nullptr, ntok, stream, rows);
}


int gdn_decode_slots(const gdn_dims* dims, const gdn_weights* w, int32_t rows, const int32_t* slots_host,
                     const int32_t* slots_dev, int32_t pool_rows, const uint16_t* qkv, const uint16_t* z,
                     const uint16_t* a, const uint16_t* b, float* state_pool, float* conv_pool, uint16_t* out,
                     void* stream) {
    NvtxRange nvtx_range("gdn_decode_slots");
    int st = check_dims(dims);
    if (st != GDN_OK) return st;
    if ((st = check_weights(w)) != GDN_OK) return st;
    if (rows < 0 || rows > 65535) return GDN_ERR_INVALID_ARG;
    if (rows == 0) return GDN_OK;
    if ((st = check_slots(slots_host, rows, pool_rows)) != GDN_OK) return st;
    if (slots_dev == nullptr || (reinterpret_cast<uintptr_t>(slots_dev) & 3u)) return GDN_ERR_INVALID_ARG;
    return decode_impl(dims, w, rows, qkv, z, a, b, state_pool, conv_pool, out, slots_dev, 1, stream, pool_rows);
}

int gdn_prefill_varlen_slots(const gdn_dims* dims, const gdn_weights* w, int32_t N, const int32_t* cu_host,
                             const int32_t* cu_dev, int32_t total_T, const int32_t* slots_host,
                             const int32_t* slots_dev, int32_t pool_rows, const uint16_t* qkv, const uint16_t* z,
                             const uint16_t* a, const uint16_t* b, float* state_pool, float* conv_pool,
                             uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
    NvtxRange nvtx_range("gdn_prefill_varlen_slots");
    int st = check_dims(dims);
    if (st != GDN_OK) return st;
    if ((st = check_weights(w)) != GDN_OK) return st;
    if (N < 0 || N > 65535 || total_T < 0) return GDN_ERR_INVALID_ARG;
    if (cu_host == nullptr || (N > 0 && cu_dev == nullptr)) return GDN_ERR_INVALID_ARG;
    if (cu_host[0] != 0 || cu_host[N] != total_T) return GDN_ERR_INVALID_ARG;
    for (int32_t i = 0; i < N; ++i)
        if (cu_host[i + 1] < cu_host[i]) return GDN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(cu_dev) & 3u) != 0) return GDN_ERR_INVALID_ARG;
    if (N == 0) return GDN_OK;
    if ((st = check_slots(slots_host, N, pool_rows)) != GDN_OK) return st;
    if (slots_dev == nullptr || (reinterpret_cast<uintptr_t>(slots_dev) & 3u)) return GDN_ERR_INVALID_ARG;
    if (state_pool == nullptr || conv_pool == nullptr) return GDN_ERR_INVALID_ARG;
    if ((st = check_io(total_T, qkv, z, a, b, out, state_pool, conv_pool, state_pool, conv_pool)) != GDN_OK)
        return st;
    if ((st = check_device()) != GDN_OK) return st;
    if (total_T == 0) return GDN_OK;  // the pool rows stay as they are
    int64_t nch = 0;
    for (int32_t i = 0; i < N; ++i) nch += (cu_host[i + 1] - cu_host[i] + 63) / 64;
    return prefill_impl(dims, w, N, cu_dev, 0, total_T, nch, chunk_bound(N, total_T), qkv, z, a, b, state_pool,
                        conv_pool, out, state_pool, conv_pool, workspace, workspace_bytes,
                        static_cast<cudaStream_t>(stream), false, slots_dev, nullptr, nullptr, pool_rows);
}

int gdn_prefill_noalloc(const gdn_dims* dims, const gdn_weights* w, int32_t B, int32_t T, const uint16_t* qkv,
                        const uint16_t* z, const uint16_t* a, const uint16_t* b, const float* init_state,
                        const float* init_conv, uint16_t* out, float* final_state, float* final_conv, void* stream) {
    NvtxRange nvtx_range("gdn_prefill_noalloc");
    int st = check_dims(dims);
    if (st != GDN_OK) return st;
    if ((st = check_weights(w)) != GDN_OK) return st;
    if (B < 0 || T < 0 || B > 65535) return GDN_ERR_INVALID_ARG;
    const int64_t total = (int64_t)B * T;
    if (total > INT32_MAX) return GDN_ERR_INVALID_ARG;
    if ((st = check_io((int32_t)total, qkv, z, a, b, out, init_state, init_conv, final_state, final_conv)) != GDN_OK)
        return st;
    const int64_t nch = (int64_t)B * ((T + 63) / 64);
    if (plan_workspace(dims, total, B, nch).bytes > (size_t)GDN_NOALLOC_SCRATCH_BYTES) return GDN_ERR_WORKSPACE;
    if ((st = check_device()) != GDN_OK) return st;
    void* scratch = nullptr;
    if ((st = noalloc_scratch(&scratch)) != GDN_OK) return st;
    return prefill_impl(dims, w, B, nullptr, T, (int32_t)total, nch, nch, qkv, z, a, b, init_state, init_conv, out,
                        final_state, final_conv, scratch, (size_t)GDN_NOALLOC_SCRATCH_BYTES,
                        static_cast<cudaStream_t>(stream), false);
}

int gdn_set_decode_wait_limit(uint64_t ns) {
    if (cudaDeviceSynchronize() != cudaSuccess) return GDN_ERR_CUDA;
    const unsigned long long v = ns;
    if (cudaMemcpyToSymbol(gdn::g_decode_wait_limit_ns, &v, sizeof(v)) != cudaSuccess) return GDN_ERR_CUDA;
    return cudaDeviceSynchronize() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_test_decode_stop_copies_at(int32_t unit) {
    if (unit < -1) return GDN_ERR_INVALID_ARG;
    if (cudaDeviceSynchronize() != cudaSuccess) return GDN_ERR_CUDA;
    const int v = unit;
    if (cudaMemcpyToSymbol(gdn::g_decode_stop_copies_at, &v, sizeof(v)) != cudaSuccess) return GDN_ERR_CUDA;
    return cudaDeviceSynchronize() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_last_device_error(void) {
    int v = 0;
    if (cudaDeviceSynchronize() != cudaSuccess) return GDN_ERR_CUDA;
    if (cudaMemcpyFromSymbol(&v, gdn::g_device_error, sizeof(int)) != cudaSuccess) return GDN_ERR_CUDA;
    const int zero = 0;
    if (cudaMemcpyToSymbol(gdn::g_device_error, &zero, sizeof(int)) != cudaSuccess) return GDN_ERR_CUDA;
    return v;
}

const char* gdn_status_string(int status) {
    switch (status) {
        case GDN_OK: return "ok";
        case GDN_ERR_INVALID_ARG: return "invalid argument";
        case GDN_ERR_UNSUPPORTED: return "unsupported dimensions or device";
        case GDN_ERR_CUDA: return "CUDA error";
        case GDN_ERR_WORKSPACE: return "workspace missing or too small";
        case GDN_ERR_TIMEOUT: return "bounded device wait expired";
        case GDN_ERR_HOST_MEMORY: return "out of host memory";
        default: return "unknown status";
    }
}

int gdn_version(void) { return 200; }

}  // extern "C"

namespace {

// ---------------------------------------------------------------- 4-bit operands
int sm_count(int* nsm) {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess &&
                   cudaDeviceGetAttribute(nsm, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
}

int check_format(int32_t format) {
    return format == GDN_NVFP4 || format == GDN_MXFP4 ? GDN_OK : GDN_ERR_INVALID_ARG;
}

// Contraction widths the 4-bit operands support: whole products of 64 elements.
bool quant_width_ok(int32_t K) { return K > 0 && K % qproj::kMmaK == 0; }

size_t quant_scale_bytes(int format, int64_t rows, int K) {
    return (size_t)((rows + 127) / 128) * quant::scale_tiles(format, K) * quant::kTileBytes;
}

// Launch that may overlap the end of the stream's previous kernel: the kernels launched so call grid_wait before
// they touch global memory (the projections: before they touch what the call's quantisation wrote).  attr[0] is
// filled in; n attributes in all.
cudaLaunchConfig_t early_launch(dim3 grid, dim3 block, uint32_t smem, cudaStream_t stream, cudaLaunchAttribute* attr,
                                int n = 1) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cfg;
}

// Launch shape of the row kernels: one unit (of `unit` elements) per thread up to 512 threads a row (then two or
// more), at least 160 threads a CTA, `threads` of them per SM over the persistent grid.
int quant_shape(int32_t rows, int32_t K, int unit, int threads, dim3* grid, dim3* block) {
    int nsm = 0;
    const int st = sm_count(&nsm);
    if (st != GDN_OK) return st;
    const int units = K / unit;
    const int gx = units >= quant::kMaxGroup ? quant::kMaxGroup : (units + 31) / 32 * 32;
    const int gy = gx > 128 ? 1 : 256 / gx;
    const int64_t groups = ((int64_t)rows + gy - 1) / gy, resident = (int64_t)nsm * (threads / (gx * gy));
    *block = dim3(gx, gy);
    *grid = dim3((unsigned)(groups < resident ? groups : resident));
    return GDN_OK;
}

int quantize_launch(int format, int32_t rows, int32_t K, const uint16_t* x, uint8_t* codes, uint8_t* scales,
                    float* row_scale, cudaStream_t stream) {
    const quant::Params p{x, codes, scales, row_scale, rows, K, quant::scale_tiles(format, K)};
    dim3 grid, block;
    const int st = quant_shape(rows, K, quant::kUnit, 2048, &grid, &block);
    if (st != GDN_OK) return st;
    auto kernel = format == GDN_NVFP4 ? gdn_quantize_kernel<quant::kNvfp4> : gdn_quantize_kernel<quant::kMxfp4>;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = early_launch(grid, block, 0, stream, attr);
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

// 2-D map over packed 4-bit codes [rows][K / 2 bytes], box of 128 bytes (256 elements) x box_rows.
bool make_code_map(CUtensorMap* m, const uint8_t* base, int32_t K, int64_t rows, uint32_t box_rows) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[2] = {(cuuint64_t)K / 2, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)K / 2};
    cuuint32_t box[2] = {128, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The scale tiles as rows of 512 bytes, `stage` of them per box.
bool make_scale_map(CUtensorMap* m, const uint8_t* base, int64_t tiles, uint32_t stage) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[2] = {quant::kTileBytes / 4, (cuuint64_t)tiles};
    cuuint64_t strides[1] = {quant::kTileBytes};
    cuuint32_t box[2] = {quant::kTileBytes / 4, stage};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT>
int qproj_pairs(const uint8_t* cx, const uint8_t* cw, const qproj::Params& p, int nsm, cudaStream_t stream) {
    CUtensorMap mW, mX, mSw, mSx;
    const int stage = qproj::kTilesPerStage(FMT);
    if (!make_code_map(&mW, cw, p.K, p.N, 128) || !make_code_map(&mX, cx, p.K, p.T, 128) ||
        !make_scale_map(&mSw, p.sw, (int64_t)((p.N + 127) / 128) * p.tiles, stage) ||
        !make_scale_map(&mSx, p.sx, (int64_t)((p.T + 127) / 128) * p.tiles, stage))
        return GDN_ERR_CUDA;
    auto kernel = gdn_qproj_pair_kernel<FMT>;
    int st = smem_optin(reinterpret_cast<const void*>(kernel), qproj::duo::SMEM_BYTES);
    if (st != GDN_OK) return st;
    const int64_t ntiles = (int64_t)((p.T + qproj::duo::kTileM - 1) / qproj::duo::kTileM) *
                           ((p.N + qproj::duo::kTileN - 1) / qproj::duo::kTileN);
    const int pairs = (int)(ntiles < nsm / 2 ? ntiles : nsm / 2);
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = early_launch(dim3(2 * pairs), qproj::duo::kDuoThreads, qproj::duo::SMEM_BYTES, stream, attr, 1);
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, mW, mX, mSw, mSx, p));
}

// Clusters of `cfg`'s size that the current device runs at once (0: unknown); asked once per kernel, device and
// size while the table has room.
int resident_clusters(const void* kernel, int size, const cudaLaunchConfig_t& cfg) {
    struct Known {
        const void* kernel;
        int dev, size, clusters;
    };
    static std::mutex mu;
    static Known known[256];
    static int count = 0;
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < count; ++i)
        if (known[i].kernel == kernel && known[i].dev == dev && known[i].size == size) return known[i].clusters;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();  // (not the launch's error)
        n = 0;
    }
    if (count < 256) known[count++] = Known{kernel, dev, size, n};
    return n;
}

template <int FMT, int BN, bool kFuse>
int qproj_few(const uint8_t* cx, const uint8_t* cw, const qproj::Params& p, int nsm, cudaStream_t stream) {
    using C = qproj::few::Cfg<BN, kFuse>;
    CUtensorMap mW, mX;
    if (!make_code_map(&mW, cw, p.K, p.N, qproj::few::kTileN)) return GDN_ERR_CUDA;
    if (kFuse) mX = mW;  // (not read)
    else if (!make_code_map(&mX, cx, p.K, p.T, BN)) return GDN_ERR_CUDA;
    auto kernel = gdn_qproj_few_kernel<FMT, BN, kFuse>;
    const int st = smem_optin(reinterpret_cast<const void*>(kernel), C::SMEM_BYTES);
    if (st != GDN_OK) return st;
    // Clusters that share a tile's K while the tiles leave SMs idle, at least two stages per CTA, and only as large as
    // lets all of them run at once: a cluster lies inside one group of SMs, so 37 tiles by 4 take two rounds (12.3 us)
    // where 37 by 3 take one (8.3 us).
    const int tiles = (p.N + qproj::few::kTileN - 1) / qproj::few::kTileN, steps = (p.K + qproj::BK - 1) / qproj::BK;
    int split = nsm / tiles;
    if (split > steps / 2) split = steps / 2;
    if (split > qproj::few::kMaxSplit) split = qproj::few::kMaxSplit;
    cudaLaunchAttribute attr[2];
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = 1;
    for (;; --split) {
        if (split < 1) split = 1;
        attr[1].val.clusterDim.z = split;
        const cudaLaunchConfig_t cfg = early_launch(dim3(tiles, 1, split), C::kThreads, C::SMEM_BYTES, stream, attr, split > 1 ? 2 : 1);
        if (split > 1 && resident_clusters(reinterpret_cast<const void*>(kernel), split, cfg) < tiles) continue;
        return cuda_status(cudaLaunchKernelEx(&cfg, kernel, mW, mX, p));
    }
}

template <int FMT>
int qproj_launch(const uint8_t* cx, const uint8_t* cw, const qproj::Params& p, int nsm, cudaStream_t stream) {
    if (p.T <= 16) return qproj_few<FMT, 16, false>(cx, cw, p, nsm, stream);
    if (p.T <= 32) return qproj_few<FMT, 32, false>(cx, cw, p, nsm, stream);
    if (p.T <= 64) return qproj_few<FMT, 64, false>(cx, cw, p, nsm, stream);
    // Up to 96 tokens one pass over the weights by single CTAs; up to 128 too, unless the pairs' tiles keep two thirds
    // of them busy.  us by single CTAs / by pairs, nvfp4, at 65, 96 and 128 tokens: 16480 x 5120 (65 pair tiles)
    // 15.5 / 16.8, 16.4 / 16.9, 17.9 / 17.4; 12352 x 5120 (49) 15.2 / 15.9, 15.9 / 15.9, 17.2 / 16.4; 10240 x 6144 (40)
    // 14.9 / 16.4, 15.5 / 16.5, 16.5 / 17.1; 12288 x 6144 (48) 15.4 / 17.0, 15.9 / 17.0, 16.9 / 17.6; 5120 x 6144 (20) 10.3 / 14.4, 11.3 / 14.9, 12.1 / 15.2.
    if (p.T <= 96 || (p.T <= 128 && (p.N + qproj::duo::kTileN - 1) / qproj::duo::kTileN < nsm / 3))
        return qproj_few<FMT, 128, false>(cx, cw, p, nsm, stream);
    return qproj_pairs<FMT>(cx, cw, p, nsm, stream);
}

// Whether a projection quantises its few tokens itself: at most 16 tokens and 16384 elements, which fit its threads'
// registers, of rows that fit its shared memory.  The rule is in T and K alone because the workspace's size, which the
// caller asks for by T and K, follows from it: such calls need none.  Every CTA repeats the quantisation, so it pays
// where its weights' loads cover it.  us so / by a launch of its own, nvfp4: 16480 x 5120, 1 token 11.3 / 12.3, 2 tokens
// 11.3 / 12.5, 3 tokens 12.3 / 12.4; 16480 x 1024, 1 token 5.1 / 5.6, 4 tokens 5.2 / 5.7, 8 tokens 5.7 / 5.2, 16 tokens
// 6.2 / 5.7; 5120 x 6144 (K shared by 3 CTAs, each scanning whole rows), 1 token 7.7 / 7.7, 2 tokens 8.2 / 7.7;
// 4120 x 1088, 1 token 5.7 / 5.7, 15 tokens 7.2 / 5.7.  More elements would lose everywhere (before it had this bound:
// 16480 x 5120, 8 tokens 16.3 against 13.4).
bool few_fuse(int64_t T, int K) {
    return T <= 16 && T * (K / 16) <= qproj::few::kRowThreads * qproj::few::kHold &&
           K <= qproj::few::kMaxSteps * qproj::BK;
}

// Workspace of a 4-bit projection: the quantised tokens, none where it quantises them itself.
struct QuantRows {
    size_t off_scales, off_row_scale, bytes;
};
QuantRows quant_rows(int format, int64_t T, int K) {
    QuantRows q{};
    if (few_fuse(T, K)) return q;
    q.off_scales = align_up((size_t)T * (K / 2));
    q.off_row_scale = q.off_scales + align_up(quant_scale_bytes(format, T, K));
    q.bytes = q.off_row_scale + align_up((size_t)T * 4);
    return q;
}

// y = x W^T on 4-bit operands: x [T][K] quantised into the workspace, then the product.
int proj_quant(int format, int32_t T, int32_t K, int32_t N, const uint16_t* x, const uint8_t* w_codes,
               const uint8_t* w_scales, const float* w_row_scale, const GemmSegment* seg, int nseg, void* workspace,
               size_t workspace_bytes, void* stream) {
    if (!x || !w_codes || !w_scales || !w_row_scale || !aligned16(x) || !aligned16(w_codes) || !aligned16(w_scales) ||
        (reinterpret_cast<uintptr_t>(w_row_scale) & 3u))
        return GDN_ERR_INVALID_ARG;
    for (int i = 0; i < nseg; ++i)
        if (seg[i].dst == nullptr || !aligned16(seg[i].dst)) return GDN_ERR_INVALID_ARG;
    const QuantRows q = quant_rows(format, T, K);
    if (workspace_bytes < q.bytes || (workspace == nullptr && q.bytes > 0)) return GDN_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GDN_ERR_INVALID_ARG;
    int st = check_device(), nsm = 0;
    if (st != GDN_OK || (st = sm_count(&nsm)) != GDN_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* wsb = static_cast<uint8_t*>(workspace);
    qproj::Params p{};
    p.T = T;
    p.N = N;
    p.K = K;
    p.tiles = quant::scale_tiles(format, K);
    p.x = x;
    p.sx = wsb + q.off_scales;
    p.sw = w_scales;
    p.gx = reinterpret_cast<const float*>(wsb + q.off_row_scale);
    p.gw = w_row_scale;
    p.nseg = nseg;
    for (int i = 0; i < nseg; ++i) p.seg[i] = seg[i];
    try {
        if (few_fuse(T, K))
            return format == GDN_NVFP4 ? qproj_few<quant::kNvfp4, 16, true>(nullptr, w_codes, p, nsm, s)
                                       : qproj_few<quant::kMxfp4, 16, true>(nullptr, w_codes, p, nsm, s);
        if ((st = quantize_launch(format, T, K, x, wsb, wsb + q.off_scales,
                                  reinterpret_cast<float*>(wsb + q.off_row_scale), s)) != GDN_OK)
            return st;
        return format == GDN_NVFP4 ? qproj_launch<quant::kNvfp4>(wsb, w_codes, p, nsm, s)
                                   : qproj_launch<quant::kMxfp4>(wsb, w_codes, p, nsm, s);
    } catch (const std::bad_alloc&) {  // (the list of kernels whose shared memory has been opted in)
        return GDN_ERR_HOST_MEMORY;
    }
}

// ---------------------------------------------------------------- pool rows
// Pairs (src[i], dst[i]) of pool rows, src -1 = clear, all reads before all writes.  Checked by the caller.
struct RowPair {
    int32_t src, dst;
};

int pool_flush(pool::Params& p, int nsm, cudaStream_t stream) {
    if (p.nset == 0) return GDN_OK;
    int st = smem_optin(reinterpret_cast<const void*>(gdn_pool_kernel), pool::SMEM_BYTES);
    if (st != GDN_OK) return st;
    const int ctas = pool::kCtasPerSm * nsm;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = early_launch(dim3(p.ntask < ctas ? p.ntask : ctas), dim3(32), pool::SMEM_BYTES, stream, attr);
    st = cuda_status(cudaLaunchKernelEx(&cfg, gdn_pool_kernel, p));
    p.nset = p.ntask = 0;
    return st;
}

// Groups the pairs into sets linked by a shared row and launches them, at most pool::kMaxOps
// destinations a launch.  Sets share no rows, so launches do not depend on one another.
int pool_launch(const gdn_dims* dims, std::vector<RowPair> pairs, int32_t pool_rows, float* state, float* conv,
                cudaStream_t stream) {
    // a row kept in place is neither read nor written
    size_t n = 0;
    for (const RowPair& r : pairs)
        if (r.src != r.dst) pairs[n++] = r;
    pairs.resize(n);
    if (n == 0) return GDN_OK;
    int dev = 0, nsm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return GDN_ERR_CUDA;
    std::vector<int32_t> root((size_t)pool_rows);
    for (int32_t i = 0; i < pool_rows; ++i) root[i] = i;
    auto find = [&](int32_t i) {
        while (root[i] != i) i = root[i] = root[root[i]];
        return i;
    };
    std::vector<unsigned char> is_dst((size_t)pool_rows, 0);
    for (const RowPair& r : pairs) {
        if (r.src >= 0) root[find(r.src)] = find(r.dst);
        is_dst[r.dst] = 1;
    }
    // pairs of a set next to each other, a set's pairs by source
    std::vector<std::pair<int64_t, int32_t>> key(n);
    for (size_t i = 0; i < n; ++i) key[i] = {((int64_t)find(pairs[i].dst) << 32) | (uint32_t)(pairs[i].src + 1), (int32_t)i};
    std::sort(key.begin(), key.end());
    auto set_end = [&](size_t i) {
        size_t j = i;
        while (j < n && (key[j].first >> 32) == (key[i].first >> 32)) ++j;
        return j;
    };
    // a set that overwrites one of its sources is moved by one launch
    auto overwrites = [&](size_t i, size_t j) {
        for (size_t k = i; k < j; ++k) {
            const int32_t src = pairs[key[k].second].src;
            if (src >= 0 && is_dst[src]) return true;
        }
        return false;
    };
    for (size_t i = 0; i < n; i = set_end(i))
        if (set_end(i) - i > (size_t)pool::kMaxOps && overwrites(i, set_end(i))) return GDN_ERR_UNSUPPORTED;

    pool::Params p{};
    p.base[0] = reinterpret_cast<uint8_t*>(state);
    p.base[1] = reinterpret_cast<uint8_t*>(conv);
    p.row_bytes[0] = (uint32_t)dims->num_v_heads * 128 * 128 * 4;
    p.row_bytes[1] = 3u * (2 * dims->num_k_heads + dims->num_v_heads) * 128 * 4;
    p.pool_rows = pool_rows;
    // Bytes loaded per task: what gives every CTA one task, up to a whole stage (a fork of one 27B row to four 5.2 ->
    // 4.1 us against 8 KB tasks, of which some CTAs had two).
    uint64_t loads = 0;  // rows loaded (or cleared, in a set that loads none)
    for (size_t i = 0; i < n; i = set_end(i)) {
        uint64_t distinct = 0;
        for (size_t k = i; k < set_end(i); ++k) {
            const int32_t src = pairs[key[k].second].src;
            distinct += src >= 0 && (k == i || src != pairs[key[k - 1].second].src);
        }
        loads += distinct > 0 ? distinct : 1;
    }
    const uint64_t share = loads * (p.row_bytes[0] + p.row_bytes[1]) / ((uint64_t)pool::kCtasPerSm * nsm);
    const uint32_t stage = share >= pool::kStageBytes ? pool::kStageBytes : share < 4096 ? 4096 : ((uint32_t)share + 127) & ~127u;
    int nsrc = 0, nop = 0;
    for (size_t i = 0; i < n;) {
        size_t j = set_end(i);
        if (j - i > (size_t)pool::kMaxOps) j = i + pool::kMaxOps;  // (one source, or clears: any part of it)
        if (nop + (int)(j - i) > pool::kMaxOps) {
            const int st = pool_flush(p, nsm, stream);
            if (st != GDN_OK) return st;
            nsrc = nop = 0;
        }
        pool::Set& e = p.set[p.nset++];
        e.task0 = p.ntask;
        e.src0 = (uint16_t)nsrc;
        e.op0 = (uint16_t)nop;
        for (size_t k = i; k < j; ++k) {
            const RowPair& r = pairs[key[k].second];
            if (r.src >= 0 && (nsrc == e.src0 || p.src[nsrc - 1] != r.src)) p.src[nsrc++] = r.src;
            p.op[nop++] = pool::Op{r.dst, r.src >= 0 ? nsrc - 1 - e.src0 : pool::kZero};
        }
        e.nsrc = (uint16_t)(nsrc - e.src0);
        e.nop = (uint16_t)(nop - e.op0);
        uint32_t chunk = stage / (e.nsrc > 1 ? e.nsrc : 1);
        if (chunk < 256) chunk = pool::kStageBytes / e.nsrc;  // (many sources: the whole stage)
        e.chunk = chunk >= 128 ? chunk & ~127u : chunk & ~15u;
        for (int k = 0; k < 2; ++k) p.ntask += (int32_t)((p.row_bytes[k] + e.chunk - 1) / e.chunk);
        i = j;
    }
    return pool_flush(p, nsm, stream);
}

int check_pool(const gdn_dims* dims, int32_t pool_rows, const float* state, const float* conv) {
    const int st = check_dims(dims);
    if (st != GDN_OK) return st;
    if (pool_rows < 0) return GDN_ERR_INVALID_ARG;
    if (pool_rows > 0 && (!state || !conv || !aligned16(state) || !aligned16(conv))) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

}  // namespace

extern "C" {

size_t gdn_quant_scale_bytes(int32_t format, int32_t rows, int32_t K) {
    if (check_format(format) != GDN_OK || rows < 0 || !quant_width_ok(K)) return 0;
    return quant_scale_bytes(format, rows, K);
}

int gdn_quantize(int32_t format, int32_t rows, int32_t K, const uint16_t* x, uint8_t* codes, uint8_t* scales,
                 float* row_scale, void* stream) {
    NvtxRange nvtx_range("gdn_quantize");
    int st = check_format(format);
    if (st != GDN_OK) return st;
    if (rows < 0 || K <= 0) return GDN_ERR_INVALID_ARG;
    if (!quant_width_ok(K)) return GDN_ERR_UNSUPPORTED;
    if (rows == 0) return GDN_OK;
    if (!x || !codes || !scales || !row_scale || !aligned16(x) || !aligned16(codes) || !aligned16(scales) ||
        (reinterpret_cast<uintptr_t>(row_scale) & 3u))
        return GDN_ERR_INVALID_ARG;
    if ((st = check_device()) != GDN_OK) return st;
    return quantize_launch(format, rows, K, x, codes, scales, row_scale, static_cast<cudaStream_t>(stream));
}

int gdn_dequantize(int32_t format, int32_t rows, int32_t K, const uint8_t* codes, const uint8_t* scales,
                   const float* row_scale, uint16_t* out, void* stream) {
    NvtxRange nvtx_range("gdn_dequantize");
    int st = check_format(format);
    if (st != GDN_OK) return st;
    if (rows < 0 || K <= 0) return GDN_ERR_INVALID_ARG;
    if (!quant_width_ok(K)) return GDN_ERR_UNSUPPORTED;
    if (rows == 0) return GDN_OK;
    if (!out || !codes || !scales || !row_scale || !aligned16(out) || !aligned16(codes) || !aligned16(scales) ||
        (reinterpret_cast<uintptr_t>(row_scale) & 3u))
        return GDN_ERR_INVALID_ARG;
    if ((st = check_device()) != GDN_OK) return st;
    const int tiles = quant::scale_tiles(format, K);
    dim3 grid, block;
    if ((st = quant_shape(rows, K, 16, 1280, &grid, &block)) != GDN_OK) return st;
    auto kernel = format == GDN_NVFP4 ? gdn_dequantize_kernel<quant::kNvfp4> : gdn_dequantize_kernel<quant::kMxfp4>;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = early_launch(grid, block, 0, static_cast<cudaStream_t>(stream), attr);
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, codes, scales, row_scale, rows, K, tiles, out));
}

size_t gdn_proj_quant_workspace_size(int32_t format, int32_t T, int32_t K) {
    if (check_format(format) != GDN_OK || T < 0 || !quant_width_ok(K)) return 0;
    return quant_rows(format, T, K).bytes;
}

int gdn_in_proj_quant(const gdn_dims* dims, int32_t format, int32_t T, int32_t hidden, const uint16_t* x,
                      const uint8_t* w_codes, const uint8_t* w_scales, const float* w_row_scale, uint16_t* qkv,
                      uint16_t* z, uint16_t* b, uint16_t* a, void* workspace, size_t workspace_bytes, void* stream) {
    NvtxRange nvtx_range("gdn_in_proj_quant");
    int st = check_dims(dims);
    if (st != GDN_OK || (st = check_format(format)) != GDN_OK) return st;
    if (T < 0 || hidden <= 0) return GDN_ERR_INVALID_ARG;
    if (!quant_width_ok(hidden)) return GDN_ERR_UNSUPPORTED;
    if (T == 0) return GDN_OK;
    const int Vh = dims->num_v_heads, D = dims->head_dim;
    const int C = (2 * dims->num_k_heads + Vh) * D;
    const GemmSegment seg[4] = {GemmSegment{0, C, qkv}, GemmSegment{C, Vh * D, z}, GemmSegment{C + Vh * D, Vh, b},
                                GemmSegment{C + Vh * D + Vh, Vh, a}};
    return proj_quant(format, T, hidden, C + Vh * D + 2 * Vh, x, w_codes, w_scales, w_row_scale, seg, 4, workspace,
                      workspace_bytes, stream);
}

int gdn_out_proj_quant(const gdn_dims* dims, int32_t format, int32_t T, int32_t hidden, const uint16_t* y,
                       const uint8_t* w_codes, const uint8_t* w_scales, const float* w_row_scale, uint16_t* out,
                       void* workspace, size_t workspace_bytes, void* stream) {
    NvtxRange nvtx_range("gdn_out_proj_quant");
    int st = check_dims(dims);
    if (st != GDN_OK || (st = check_format(format)) != GDN_OK) return st;
    if (T < 0 || hidden <= 0) return GDN_ERR_INVALID_ARG;
    if (T == 0) return GDN_OK;
    const GemmSegment seg[1] = {GemmSegment{0, hidden, out}};
    return proj_quant(format, T, dims->num_v_heads * dims->head_dim, hidden, y, w_codes, w_scales, w_row_scale, seg, 1,
                      workspace, workspace_bytes, stream);
}

int gdn_copy_slots(const gdn_dims* dims, int32_t n, const int32_t* src_host, const int32_t* dst_host, int32_t pool_rows,
                   float* state_pool, float* conv_pool, void* stream) {
    NvtxRange nvtx_range("gdn_copy_slots");
    int st = check_pool(dims, pool_rows, state_pool, conv_pool);
    if (st != GDN_OK) return st;
    if (n < 0) return GDN_ERR_INVALID_ARG;
    if (n == 0) return GDN_OK;
    if (src_host == nullptr) return GDN_ERR_INVALID_ARG;
    try {
        if ((st = check_slots(dst_host, n, pool_rows)) != GDN_OK) return st;
        std::vector<RowPair> pairs((size_t)n);
        for (int32_t i = 0; i < n; ++i) {
            if (src_host[i] < -1 || src_host[i] >= pool_rows) return GDN_ERR_INVALID_ARG;
            pairs[i] = RowPair{src_host[i], dst_host[i]};
        }
        if ((st = check_device()) != GDN_OK) return st;
        return pool_launch(dims, std::move(pairs), pool_rows, state_pool, conv_pool,
                           static_cast<cudaStream_t>(stream));
    } catch (const std::bad_alloc&) {
        return GDN_ERR_HOST_MEMORY;
    }
}

int gdn_compact_slots(const gdn_dims* dims, int32_t pool_rows, const uint8_t* live_host, int32_t clear,
                      float* state_pool, float* conv_pool, int32_t* remap_host, void* stream) {
    NvtxRange nvtx_range("gdn_compact_slots");
    int st = check_pool(dims, pool_rows, state_pool, conv_pool);
    if (st != GDN_OK) return st;
    if (pool_rows == 0) return GDN_OK;
    if (live_host == nullptr || remap_host == nullptr) return GDN_ERR_INVALID_ARG;
    if ((st = check_device()) != GDN_OK) return st;
    int32_t nlive = 0;
    for (int32_t i = 0; i < pool_rows; ++i) nlive += live_host[i] != 0;
    try {
        std::vector<RowPair> pairs;
        int32_t hole = 0;
        for (int32_t i = 0; i < pool_rows; ++i) {
            remap_host[i] = live_host[i] ? i : -1;
            if (live_host[i] && i >= nlive) {
                while (live_host[hole]) ++hole;
                remap_host[i] = hole;
                pairs.push_back(RowPair{i, hole++});
            }
            if (clear && i >= nlive) pairs.push_back(RowPair{-1, i});
        }
        return pool_launch(dims, std::move(pairs), pool_rows, state_pool, conv_pool,
                           static_cast<cudaStream_t>(stream));
    } catch (const std::bad_alloc&) {
        return GDN_ERR_HOST_MEMORY;
    }
}

}  // extern "C"
