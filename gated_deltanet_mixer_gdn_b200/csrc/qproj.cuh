// Projections on microscaled 4-bit operands (quant.cuh), on the block-scaled tcgen05 products:
//     y[t][n] = gx[t] gw[n] sum_k (cx[t][k] sx[t][k/B]) (cw[n][k] sw[n][k/B])
// The products and block scales are applied by the tensor core (kind::mxf4nvf4 with E4M3 scales per
// 16, kind::mxf4 with power-of-two scales per 32), summed in f32 in tensor memory; the row scales
// multiply the sum, which is rounded once to bf16.
#pragma once

#include "common.cuh"
#include "gemm.cuh"
#include "quant.cuh"

namespace gdn {
namespace qproj {

constexpr int BK = 256;                 // elements of K per stage: 128 bytes, one swizzled row
constexpr int kMmaK = 64;               // elements of K per tcgen05.mma
__host__ __device__ constexpr int kTilesPerStage(int fmt) { return BK / (4 * quant::block_of(fmt)); }  // scale tiles per 128 rows: 4 or 2

// One lane of the (converged) warp.  The loads and products are issued from code that the whole warp runs,
// inside one elected block per stage with every descriptor formed from warp-uniform values: the operands
// then stay in uniform registers.  Issued by a lane picked with `lane == 0`, from loops, a product took
// about 73 issue cycles and a scale copy 60; so, 4 products and 12 copies take under 300 (M = 256, N = 256:
// 512 of tensor time).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
    return r != 0;
}

// Instruction descriptor of the block-scaled 4-bit kinds: E2M1 operands, both K-major, f32 sums;
// scale type E4M3 (0) or power of two (1).  The scale ids (bits 4-5 and 29-30: which bytes of a
// scale word a product reads) are or'ed in.
__host__ __device__ constexpr uint32_t idesc(int fmt, int M, int N) {
    return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
           ((fmt == quant::kMxfp4 ? 1u : 0u) << 23) | (static_cast<uint32_t>(M >> 7) << 27);
}
__host__ __device__ constexpr uint32_t scale_id(uint32_t id) { return (id << 4) | (id << 29); }

// Shared-memory descriptor of a 512-byte scale tile: 32 rows of 16 bytes, no swizzle, 8-row groups
// 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128 >> 4) << 32) |
           (static_cast<uint64_t>(1) << 46);
}

// A scale tile into 4 columns of tensor memory, repeated in the four lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <int FMT>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sa, uint32_t sb,
                                           uint32_t accumulate) {
    if constexpr (FMT == quant::kNvfp4)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}

struct Params {
    int T, N, K;                 // tokens, output features, contraction width (a multiple of 64)
    int tiles;                   // scale tiles per row of either operand
    const uint16_t* x;           // the tokens [T][K] bf16 (where the projection quantises them itself)
    const uint8_t *sx, *sw;      // block scales
    const float *gx, *gw;        // row scales [T], [N]
    int nseg;                    // output segments over the features, as in the bf16 projections
    GemmSegment seg[4];
};

// The segment of feature n, by selects (indexing the parameter array would copy it to local memory).
__device__ __forceinline__ GemmSegment segment_of(const Params& p, int n, int& end) {
    GemmSegment g = p.seg[0];
    end = p.nseg > 1 ? p.seg[1].col0 : p.N;
#pragma unroll
    for (int i = 1; i < 4; ++i)
        if (i < p.nseg && n >= p.seg[i].col0) {
            g = p.seg[i];
            end = i + 1 < p.nseg ? p.seg[i < 3 ? i + 1 : 3].col0 : p.N;
        }
    return g;
}

__device__ __forceinline__ uint16_t* output_at(const Params& p, int n, int t) {
    int end;
    const GemmSegment g = segment_of(p, n, end);
    if (!GDN_CHECK(t >= 0 && t < p.T && n >= g.col0 && n - g.col0 < g.ld)) return g.dst;
    return g.dst + (size_t)t * g.ld + (n - g.col0);
}

// Sums times the row scales: a token's gx is a power of two in [2^-100, 2^117], 1, or NaN, a feature's gw any finite
// number.  Their product may leave f32's range where v gx gw does not (2^114 2^15 over a sum that cancels, 2^-100
// 2^-50 under a large one), so a sum v (in nvfp4 0 or 2^-20 <= |v| <= 2^40) is scaled as ((v x) gw) y with gx = x y:
// up to gx = 2^+-79 v gx is in range, and y = 1; beyond, half of gx's exponent comes before gw and half after it, so
// that nothing overflows unless the result does, and nothing is lost that it still shows.  The factors x and y are
// exact: the result has gw's one rounding.
__device__ __forceinline__ float2 split_scale(float gx) {
    const int e = static_cast<int>(__float_as_uint(gx) >> 23) - 127;
    if ((e > -80 && e < 80) || e == 128) return make_float2(gx, 1.0f);
    return make_float2(quant::pow2f(e >> 1), quant::pow2f(e - (e >> 1)));
}

// Two sums of a token times the row scales, as a bf16 pair.
__device__ __forceinline__ uint32_t scale_pack2(float v0, float v1, float2 gx, float gw0, float gw1) {
    const float2 r = mul2(mul2(mul2(make_float2(v0, v1), make_float2(gx.x, gx.x)), make_float2(gw0, gw1)),
                          make_float2(gx.y, gx.y));
    return pack_bf16x2(r.x, r.y);
}

constexpr uint32_t S_BYTES = 4 * quant::kTileBytes;  // scales of 128 rows and a stage, at most

// ---------------------------------------------------------------- few tokens: the weights' rows as lanes
namespace few {
constexpr int kTileN = 128;                           // features per tile (rows of the A operand)
constexpr uint32_t W_BYTES = kTileN * BK / 2;         // 16 KB
constexpr int kMaxSplit = 8;                          // CTAs of a cluster that share a tile's K
// The tokens quantised by the projection itself (kFuse): kRowThreads threads hold kHold units of 16 elements
// each, and a CTA's part of K is at most kMaxSteps stages (its codes and scales stay in shared memory).
constexpr int kRowThreads = 512, kHold = 2, kMaxSteps = 24;

template <int BN, bool kFuse>
struct Cfg {
    static constexpr uint32_t X_BYTES = BN * BK / 2;
    static constexpr uint32_t X_STAGE = X_BYTES + S_BYTES;  // a stage's token codes and scales
    static constexpr uint32_t STAGE_BYTES = W_BYTES + S_BYTES + (kFuse ? 0 : X_STAGE);
    static constexpr int kStages = kFuse ? 7 : 6;  // (more: 64 tokens 14.5 us with 7 against 14.4, 32 tokens 13.6 with 9 against 13.2)
    static constexpr uint32_t OFF_X = kStages * STAGE_BYTES;  // (kFuse) all stages' tokens
    static constexpr uint32_t OFF_MISC = OFF_X + (kFuse ? kMaxSteps * X_STAGE : 0);
    static constexpr uint32_t OFF_AMAX = OFF_MISC + 256 + BN * 8;  // (kFuse) behind the row scales
    static constexpr uint32_t SMEM_BYTES = OFF_AMAX + (kFuse ? BN * 4 : 0) + 1024;
    static constexpr int kThreads = 64 + (kFuse ? kRowThreads : 256);  // warp 0 loads, warp 1 products, rows and sums
    // tensor memory: the sums (BN columns), then per stage 16 columns of weight scales and 16 of token
    // scales; a stage's columns are free when its shared memory is
    static constexpr uint32_t TMEM_COLS = 512;
    static_assert(BN + 32 * kStages <= 512, "tensor memory");
    static_assert(X_BYTES % 1024 == 0 && STAGE_BYTES % 1024 == 0, "swizzle atoms");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
    static_assert(kStages * STAGE_BYTES >= BN * kTileN * 4, "the partial sums reuse the ring");
};
}  // namespace few
}  // namespace qproj

// (kFuse) The tokens' rows, held in registers by kRowThreads threads: row maxima, then the codes (swizzled
// rows of 128 bytes per stage) and scale tiles of stages [k0, k0 + ksteps) into shared memory at `out`, and
// the split row scales.  The same values as gdn_quantize_kernel's.
template <int FMT, class C>
__device__ __forceinline__ void quantize_tokens(const qproj::Params& p, uint8_t* out, uint32_t* s_amax, float2* s_gx,
                                                uint64_t* rows_ready, int tid, int k0, int ksteps) {
    using namespace qproj;
    using namespace qproj::few;
    const int per_row = p.K / 16, units = p.T * per_row;  // units <= kRowThreads * kHold
    const uint32_t inv = (0xffffffffu / per_row) + 1;  // u / per_row by the high word, exact below 2^16 (per_row >= 4)
    auto row_of = [&](int u) { return static_cast<int>(__umulhi(static_cast<uint32_t>(u), inv)); };
    const uint4* src = reinterpret_cast<const uint4*>(p.x);
    uint4 a[kHold], b[kHold];
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
        const int u = tid + h * kRowThreads;
        a[h] = b[h] = make_uint4(0, 0, 0, 0);
        if (u < units && GDN_CHECK(u >= 0 && row_of(u) < p.T)) {
            a[h] = src[2 * u];
            b[h] = src[2 * u + 1];
        }
    }
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
        if (h * kRowThreads < units) {
            const int u = tid + h * kRowThreads, u0 = u & ~31;
            const uint32_t um = quant::amax_bits16(a[h], b[h]);
            if (u0 < units && row_of(u0) == row_of(min(u0 + 31, units - 1))) {  // the warp's units are in one row
                const uint32_t wm = __reduce_max_sync(0xffffffffu, um);
                if ((tid & 31) == 0) atomicMax(&s_amax[row_of(u0)], wm);
            } else if (u < units) {
                atomicMax(&s_amax[row_of(u)], um);
            }
        }
    }
    named_barrier_sync(1, kRowThreads);
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
        const int u = tid + h * kRowThreads;
        if (h * kRowThreads < units) {  // (whole warps: blocks of two units exchange their maxima)
            const int t = u < units ? row_of(u) : 0, ku = u - t * per_row;
            uint32_t um = quant::amax_bits16(a[h], b[h]);
            if constexpr (FMT == quant::kMxfp4) um = max(um, __shfl_xor_sync(0xffffffffu, um, 1));
            const int stage = ku / (BK / 16) - k0;
            if (u < units && stage >= 0 && stage < ksteps) {
                const uint32_t rm = s_amax[t];
                uint32_t scale;
                const float inv = quant::block_scale<FMT>(um, FMT == quant::kNvfp4 ? quant::inv_row_scale(rm) : 1.0f, scale);
                uint2 codes = quant::codes16<FMT>(a[h], b[h], inv);
                if (rm >= 0x7f80u) codes = make_uint2(0u, 0u), scale = 0u;
                uint8_t* st = out + stage * C::X_STAGE;
                const int in = ku % (BK / 16);  // the unit's 8 bytes in the stage's 128
                *reinterpret_cast<uint2*>(st + sw128_chunk(t, in >> 1) + 8 * (in & 1)) = codes;
                const int blk = in / (quant::block_of(FMT) / 16);
                if (FMT == quant::kNvfp4 || (in & 1) == 0)
                    st[C::X_BYTES + (blk >> 2) * quant::kTileBytes + t * 16 + (blk & 3)] = static_cast<uint8_t>(scale);
            }
        }
    }
    fence_proxy_async_smem();
    mbar_arrive(rows_ready);
    if (tid < p.T) s_gx[tid] = split_scale(quant::row_scale_of<FMT>(s_amax[tid]));
}

// At most 128 tokens: a tile is 128 features x all BN (>= T) tokens, the weights the A operand, so that few
// tokens still fill the tensor core's 128 lanes.  Bound: reading the weights once.  Where the tiles are fewer
// than the SMs a cluster of gridDim.z CTAs shares one tile's K; each leaves its sums in shared memory and adds
// the others' for its part of the tokens, in rank order.
// kFuse (few elements in all): every CTA quantises the tokens itself, its part of K into shared memory, while
// its weights arrive: no second launch (3 us) and no workspace; all CTAs repeat the work, so it stays at what
// their registers hold.  Else the tokens were quantised by the call's previous launch, and the loads of the
// first stages' weights, and all of the prologue, run before its end is waited for.
template <int FMT, int BN, bool kFuse>
__global__ void __launch_bounds__(qproj::few::Cfg<BN, kFuse>::kThreads, 1)
    gdn_qproj_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                         const qproj::Params p) {
    using namespace qproj;
    using namespace qproj::few;
    using C = Cfg<BN, kFuse>;
    constexpr int kTiles = kTilesPerStage(FMT);
    constexpr uint32_t ID = idesc(FMT, kTileN, BN);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_MISC);
    uint64_t* empty = full + C::kStages;
    uint64_t* done = empty + C::kStages;
    uint64_t* rows_ready = done + 1;  // (kFuse) the tokens' codes and scales are in shared memory
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 192);
    float2* s_gx = reinterpret_cast<float2*>(smem + C::OFF_MISC + 256);        // [BN] the tokens' row scales, split
    uint32_t* s_amax = reinterpret_cast<uint32_t*>(smem + C::OFF_AMAX);        // (kFuse) the tokens' largest magnitudes
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n0 = blockIdx.x * kTileN;
    const int split = gridDim.z, rank = blockIdx.z;  // (the cluster spans z)
    const int all = (p.K + BK - 1) / BK;
    const int k0 = static_cast<int>(static_cast<int64_t>(all) * rank / split);
    const int ksteps = static_cast<int>(static_cast<int64_t>(all) * (rank + 1) / split) - k0;

    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        mbar_init(rows_ready, kRowThreads);
        fence_barrier_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmX);
    }
    if (kFuse && tid < BN) s_amax[tid] = 0;
    if (warp == 1) {
        tmem_alloc(s_tmem, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *s_tmem;
    bool broken = false;
    auto wait1 = [&](uint64_t* bar, uint32_t parity, int code) {
        if (!broken && !mbar_wait(bar, parity)) {
            broken = true;
            record_error(code);
        }
    };
    const int n = n0 + 4 * lane;  // a lane's four features of the output, and their row scales
    float gw[4];

    if (warp == 0) {
        // ---------------- loads; a stage's bytes: codes of 128 features and BN tokens, their scale tiles
        auto scale_bytes = [&](int ks) { return min(kTiles, p.tiles - (k0 + ks) * kTiles) * quant::kTileBytes; };
        auto tile_ok = [&](int ks) { return GDN_CHECK(k0 + ks >= 0 && (k0 + ks) * kTiles < p.tiles && n0 < p.N); };
        auto load_w = [&](int ks, int s) {
            uint8_t* st = smem + s * C::STAGE_BYTES;
            mbar_arrive_expect_tx(&full[s], W_BYTES + (kFuse ? 0 : C::X_BYTES) + (kFuse ? 1 : 2) * scale_bytes(ks));
            tma_load_2d(st, &tmW, (k0 + ks) * (BK / 2), n0, &full[s]);
            bulk_load(st + W_BYTES,
                      p.sw + (tile_ok(ks) ? ((size_t)blockIdx.x * p.tiles + (k0 + ks) * kTiles) * quant::kTileBytes : 0),
                      scale_bytes(ks), &full[s]);
        };
        auto load_x = [&](int ks, int s) {
            if (kFuse) return;
            uint8_t* st = smem + s * C::STAGE_BYTES + W_BYTES + S_BYTES;
            tma_load_2d(st, &tmX, (k0 + ks) * (BK / 2), 0, &full[s]);
            bulk_load(st + C::X_BYTES, p.sx + (tile_ok(ks) ? (size_t)(k0 + ks) * kTiles * quant::kTileBytes : 0),
                      scale_bytes(ks), &full[s]);
        };
        const int head = min(C::kStages, ksteps);
        if (kFuse) grid_wait();
        if (elect_one())
            for (int ks = 0; ks < head; ++ks) load_w(ks, ks);
        __syncwarp();
        if (!kFuse) grid_wait();
        if (elect_one())
            for (int ks = 0; ks < head; ++ks) load_x(ks, ks);
        __syncwarp();
        int issued = head;
        uint32_t s = 0, ph = 0;
        for (; issued < ksteps; ++issued) {
            wait1(&empty[s], ph, kErrTimeoutTma);
            if (broken) break;
            if (elect_one()) {
                load_w(issued, s);
                load_x(issued, s);
            }
            __syncwarp();
            if (++s == C::kStages) s = 0, ph ^= 1;
        }
        // no copy is in flight when the CTA exits, whatever the other warps did
        for (int ks = max(issued - C::kStages, 0); ks < issued; ++ks)
            mbar_wait(&full[ks % C::kStages], (ks / C::kStages) & 1);
    } else if (warp == 1) {
        grid_wait();  // (a bounded wait starts only when the kernel before this one has ended)
        const uint64_t kDesc = sw128_desc(0, 16, 1024), sDesc = scale_desc(0);
        uint32_t s = 0, ph = 0;
        if (kFuse) wait1(rows_ready, 0, kErrTimeoutTma);
        for (int ks = 0; ks < ksteps; ++ks) {
            wait1(&full[s], ph, kErrTimeoutTma);
            if (broken) break;
            tc_fence_after();
            const uint32_t aW = sbase + s * C::STAGE_BYTES;
            const uint32_t aX = kFuse ? sbase + C::OFF_X + ks * C::X_STAGE : aW + W_BYTES + S_BYTES;
            const uint64_t dW = desc_at(kDesc, aW), dX = desc_at(kDesc, aX);
            const uint64_t dSw = desc_at(sDesc, aW + W_BYTES), dSx = desc_at(sDesc, aX + C::X_BYTES);
            const uint32_t cW = tbase + BN + 32 * s, cX = cW + 16;
            const int nk = min(BK / kMmaK, (p.K - (k0 + ks) * BK) / kMmaK);
            const uint32_t more = ks > 0;
            if (elect_one()) {
                // (at the end of K some tiles hold an earlier stage's scales: no product reads them)
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    copy_scales(cW + 4 * i, dSw + 32 * i);
                    copy_scales(cX + 4 * i, dSx + 32 * i);
                }
#pragma unroll
                for (int kk = 0; kk < BK / kMmaK; ++kk) {
                    constexpr bool nv = FMT == quant::kNvfp4;
                    const int tile = nv ? kk : kk >> 1;
                    if (kk < nk)
                        mma_scaled<FMT>(tbase, dW + 2 * kk, dX + 2 * kk, nv ? ID : ID | scale_id(2 * (kk & 1)), cW + 4 * tile,
                                        cX + 4 * tile, kk > 0 ? 1u : more);
                }
                mma_commit(&empty[s]);
                if (ks + 1 == ksteps) mma_commit(done);
            }
            __syncwarp();
            if (++s == C::kStages) s = 0, ph ^= 1;
        }
    } else {
        grid_wait();
        if constexpr (kFuse) quantize_tokens<FMT, C>(p, smem + C::OFF_X, s_amax, s_gx, rows_ready, tid - 64, k0, ksteps);
        // (the features' row scales, used behind the sums, are loaded ahead of them, but not ahead of the tokens: 3 tokens
        // 12.4 us, 13.2 so)
#pragma unroll
        for (int e = 0; e < 4; ++e) gw[e] = n + e < p.N ? p.gw[n + e] : 0.0f;
        // ---------------- sums -> shared memory [token][feature] (the ring: every product has read it)
        const int q4 = warp & 3;  // TMEM lane quarter of this warp
        float* part = reinterpret_cast<float*>(smem);
        if constexpr (!kFuse) {
            if (tid - 64 < p.T) s_gx[tid - 64] = split_scale(p.gx[tid - 64]);  // (T <= BN <= 128 threads)
        }
        wait1(done, 0, kErrTimeoutMma);
        __syncwarp();
        tc_fence_after();
        constexpr int kWays = (C::kThreads - 64) / 128;  // warps per lane quarter
#pragma unroll 1
        for (int j = (warp - 2) >> 2; j < BN / 16; j += kWays) {
            float v[16];
            tmem_ld16(tbase + (static_cast<uint32_t>(32 * q4) << 16) + 16 * j, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) part[(16 * j + e) * kTileN + 32 * q4 + lane] = v[e];
        }
    }
    tc_fence_before();
    if (split > 1) cluster_sync();
    else __syncthreads();
    if (warp >= 2) {
        // ---------------- this rank's tokens: four features per lane, a token's 128 per warp
        constexpr int kWarps = C::kThreads / 32 - 2, kBatch = 4;  // a warp's tokens, kBatch of them at once
        int end;
        const GemmSegment g = segment_of(p, n, end);
        const bool whole = n + 4 <= end && (((n - g.col0) | g.ld) & 3) == 0;  // (segments start on 16 bytes)
        for (int t0 = rank + split * (warp - 2); t0 < p.T; t0 += kBatch * kWarps * split) {
            float4 a[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) a[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int r = 0; r < split; ++r) {
                uint32_t at = sbase + 16 * lane;
                if (split > 1) asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(r));
                float4 b[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    b[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    const int t = t0 + i * kWarps * split;
                    if (t < p.T)
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(b[i].x), "=f"(b[i].y), "=f"(b[i].z), "=f"(b[i].w)
                                     : "r"(at + t * kTileN * 4)
                                     : "memory");
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    a[i].x += b[i].x;
                    a[i].y += b[i].y;
                    a[i].z += b[i].z;
                    a[i].w += b[i].w;
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int t = t0 + i * kWarps * split;
                if (t < p.T && GDN_CHECK(t >= 0 && (n >= p.N || (n >= g.col0 && n - g.col0 < g.ld)))) {
                    const float2 gx = s_gx[t];
                    const uint32_t lo = scale_pack2(a[i].x, a[i].y, gx, gw[0], gw[1]);
                    const uint32_t hi = scale_pack2(a[i].z, a[i].w, gx, gw[2], gw[3]);
                    if (whole) {
                        *reinterpret_cast<uint2*>(g.dst + (size_t)t * g.ld + (n - g.col0)) = make_uint2(lo, hi);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n + e < p.N)
                                *output_at(p, n + e, t) = static_cast<uint16_t>((e < 2 ? lo : hi) >> (16 * (e & 1)));
                    }
                }
            }
        }
    }
    if (split > 1) cluster_sync();  // the other CTAs have read this one's sums
    if (warp == 1) tmem_dealloc(tbase, C::TMEM_COLS);
}

// ---------------------------------------------------------------- many tokens: pairs of SMs
namespace qproj {
namespace duo {
constexpr int kTileM = 256, kTileN = 256;             // tokens x features of a pair's tile
constexpr uint32_t kCodeBytes = 128 * BK / 2;         // one CTA's 128 tokens, or its 128 of the features
constexpr int kStages = 5;
constexpr uint32_t STAGE_BYTES = 2 * kCodeBytes + 3 * S_BYTES;  // + scales of 128 tokens and 256 features
constexpr uint32_t OFF_MISC = kStages * STAGE_BYTES;
constexpr uint32_t OFF_GW = OFF_MISC + 256;           // the tile's feature row scales, two buffers
constexpr uint32_t kOutBytes = 32 * 128;              // a warp's 32 tokens x 64 features on their way out
constexpr uint32_t OFF_OUT = OFF_GW + 2 * kTileN * 4;
constexpr uint32_t SMEM_BYTES = OFF_OUT + 8 * kOutBytes + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
constexpr int kDuoThreads = 320;                      // warp 0 loads, warp 1 products, warps 2-9 epilogue
// Tensor memory: two accumulators of 256 columns that share columns [kAcc1, 256), and two buffers of
// scales behind them (16 columns of token scales, 32 of feature scales each).
constexpr uint32_t kAcc1 = 160, kScales = kAcc1 + kTileN, kScaleCols = 48;
static_assert(kScales + 2 * kScaleCols <= 512, "tensor memory");
constexpr int kWalkM = 32;                            // M tiles swept across all N tiles: 8192 tokens, whose codes stay in L2 (16: 272 us, 32: 265)
}  // namespace duo

// Address of this variable's counterpart in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* local, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(local)), "r"(rank));
    return r;
}

// TMA load into this CTA that completes bytes of a barrier in either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void* smem_dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void copy_scales_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Arrive on the barrier at this offset in both CTAs when the pair's products issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

template <int FMT>
__device__ __forceinline__ void mma_scaled_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sa, uint32_t sb,
                                                uint32_t accumulate) {
    if constexpr (FMT == quant::kNvfp4)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}

// 32 sums of one token (features c0 ..) times the row scales, as bf16 pairs.
__device__ __forceinline__ void scale_pack32(const float (&v)[32], float2 gx, const float* gw, uint32_t (&o)[16]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float4 g = reinterpret_cast<const float4*>(gw)[e];
        o[2 * e] = scale_pack2(v[4 * e], v[4 * e + 1], gx, g.x, g.y);
        o[2 * e + 1] = scale_pack2(v[4 * e + 2], v[4 * e + 3], gx, g.z, g.w);
    }
}

// A warp's 32 tokens x 64 features into the output segments: lane l holds token t0 + l, features c0 .. c0 + 63
// as bf16 pairs.  Inside one segment with 16-byte rows they go through shared memory (32 rows of 128 bytes,
// 16-byte chunks swizzled by row: no bank conflicts), so that eight lanes store one token's 128 contiguous
// bytes (stored by each lane straight to its own row, the output cost 37 of 322 us at 8192 x 16480 x 5120).
__device__ __forceinline__ void store_tile32x64(const Params& p, int t0, int c0, const uint32_t (&lo)[16],
                                                const uint32_t (&hi)[16], uint8_t* stage, int lane) {
    int end;
    const GemmSegment g = segment_of(p, c0, end);
    const int col = c0 - g.col0;
    if (c0 + 64 <= end && ((col | g.ld) & 7) == 0) {  // (segments start on 16 bytes)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            *reinterpret_cast<uint4*>(stage + sw128_chunk(lane, c)) = make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
            *reinterpret_cast<uint4*>(stage + sw128_chunk(lane, 4 + c)) = make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
        }
        __syncwarp();
        uint16_t* dst = g.dst + (size_t)t0 * g.ld + col + (lane & 7) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            const uint4 v = *reinterpret_cast<const uint4*>(stage + sw128_chunk(r, lane & 7));
            if (t0 + r < p.T && GDN_CHECK(t0 >= 0 && col >= 0 && col + 64 <= g.ld)) *reinterpret_cast<uint4*>(dst + (size_t)r * g.ld) = v;
        }
    } else if (t0 + lane < p.T) {  // segment boundaries, the last features, rows off 16 bytes
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int n = c0 + 8 * c;
            if (n >= p.N) break;
            const uint32_t(&w)[16] = c < 4 ? lo : hi;
            const GemmSegment sg = segment_of(p, n, end);
            uint16_t* dst = sg.dst + (size_t)(t0 + lane) * sg.ld + (n - sg.col0);
            if (n + 8 <= end && (((n - sg.col0) | sg.ld) & 7) == 0) {
                if (!GDN_CHECK(n >= sg.col0 && n + 8 - sg.col0 <= sg.ld)) continue;
                *reinterpret_cast<uint4*>(dst) =
                    make_uint4(w[4 * (c & 3)], w[4 * (c & 3) + 1], w[4 * (c & 3) + 2], w[4 * (c & 3) + 3]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (n + e < p.N)
                        *output_at(p, n + e, t0 + lane) =
                            static_cast<uint16_t>(w[4 * (c & 3) + (e >> 1)] >> (16 * (e & 1)));
            }
        }
    }
    __syncwarp();
}

}  // namespace qproj

// Clusters of two CTAs walk 256 x 256 tiles of tokens x features: each CTA holds 128 tokens' rows and
// 128 of the features' rows in shared memory and the sums of its 128 tokens x 256 features in tensor
// memory; the products (cta_group::2, M = 256, N = 256) read both CTAs' shared memory, so each SM loads
// half the weights of the tile.  Rank 0 issues the products; both CTAs load and run their epilogue.
template <int FMT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(qproj::duo::kDuoThreads, 1)
    gdn_qproj_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                          const __grid_constant__ CUtensorMap tmSw, const __grid_constant__ CUtensorMap tmSx,
                          const qproj::Params p) {
    using namespace qproj;
    using namespace qproj::duo;
    constexpr int kTiles = kTilesPerStage(FMT);
    constexpr uint32_t kScaleBytes = kTiles * quant::kTileBytes;  // scale bytes of 128 rows and a stage
    constexpr uint32_t TX = 2 * (2 * kCodeBytes + 3 * kScaleBytes);
    constexpr uint32_t ID = idesc(FMT, kTileM, kTileN);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_MISC);  // rank 0: both CTAs' loads of a stage
    uint64_t* empty = full + kStages;                               // the stage's products are done
    uint64_t* acc_full = empty + kStages;                           // [2] a tile's sums are complete
    uint64_t* acc_free = acc_full + 2;                              // rank 0: the shared columns are drained
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + OFF_MISC + 128);
    float* s_gw = reinterpret_cast<float*>(smem + OFF_GW);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int tiles_m = (p.T + kTileM - 1) / kTileM, tiles_n = (p.N + kTileN - 1) / kTileN;
    const int ntiles = tiles_m * tiles_n, first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const int ksteps = (p.K + BK - 1) / BK;
    auto coords = [&](int t, int& tm, int& tn) {
        const int per_group = kWalkM * tiles_n;
        const int g = t / per_group, r = t - g * per_group;
        const int gm = min(kWalkM, tiles_m - g * kWalkM);
        tn = r / gm;
        tm = g * kWalkM + (r - tn * gm);
    };

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&acc_full[0], 1);
        mbar_init(&acc_full[1], 1);
        mbar_init(acc_free, 16);  // the epilogue warps of both CTAs
        fence_barrier_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmX);
        prefetch_tensormap(&tmSw);
        prefetch_tensormap(&tmSx);
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tbase = *s_tmem;
    bool broken = false;
    auto wait1 = [&](uint64_t* bar, uint32_t parity, int code) {
        if (!broken && !mbar_wait(bar, parity)) {
            broken = true;
            record_error(code);
        }
    };

    if (warp == 0) {
        // ---------------- loads: this CTA's rows; the bytes of both CTAs complete on rank 0's barrier
        grid_wait();
        uint32_t q = 0;
        for (int t = first; t < ntiles && !broken; t += step) {
            int tm, tn;
            coords(t, tm, tn);
            const int m0 = tm * kTileM + 128 * rank, n0 = tn * kTileN + 128 * rank;
            const int yx = (m0 >> 7) * p.tiles, yw = 2 * tn * p.tiles;
            for (int ks = 0; ks < ksteps; ++ks, ++q) {
                const int s = q % kStages;
                if (q >= kStages) wait1(&empty[s], ((q / kStages) - 1) & 1, kErrTimeoutTma);
                if (broken) break;
                uint8_t* st = smem + s * STAGE_BYTES;
                uint8_t* sc = st + 2 * kCodeBytes;
                const uint32_t bar = cluster_addr(&full[s], 0);
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], TX);
                    tma_load_2d_pair(st, &tmX, ks * (BK / 2), m0, bar);
                    tma_load_2d_pair(st + kCodeBytes, &tmW, ks * (BK / 2), n0, bar);
                    tma_load_2d_pair(sc, &tmSx, 0, yx + ks * kTiles, bar);
                    tma_load_2d_pair(sc + S_BYTES, &tmSw, 0, yw + ks * kTiles, bar);
                    tma_load_2d_pair(sc + 2 * S_BYTES, &tmSw, 0, yw + p.tiles + ks * kTiles, bar);
                }
                __syncwarp();
            }
        }
        // no copy is in flight when the pair exits
        if (rank == 0)
            for (uint32_t i = q > kStages ? q - kStages : 0; i < q; ++i) mbar_wait(&full[i % kStages], (i / kStages) & 1);
    } else if (warp == 1) {
        // ---------------- products (rank 0)
        if (rank == 0) {
            grid_wait();  // (as above: before the first bounded wait)
            const uint64_t kDesc = sw128_desc(0, 16, 1024), sDesc = scale_desc(0);
            // stage s of the ring, its phase; the stage two back, its phase
            uint32_t s = 0, ph = 0, s2 = kStages - 2, ph2 = 1, it = 0, cS = tbase + kScales;
            bool primed = false;  // two stages have been issued
            for (int t = first; t < ntiles && !broken; t += step, ++it) {
                // the accumulators share columns: those of the previous tile are drained first (and with
                // them, in order, everything of the tile before it)
                if (it >= 1 && !mbar_wait_cluster(acc_free, (it - 1) & 1)) {
                    broken = true;
                    record_error(kErrTimeoutMma);
                }
                tc_fence_after();
                const uint32_t d = tbase + ((it & 1) ? kAcc1 : 0);
                for (int ks = 0; ks < ksteps; ++ks) {
                    // the stage is loaded, and the scale buffer's last readers, two stages back, are done (both
                    // asked at once: a wait that succeeds costs about 80 cycles)
                    const bool loaded = mbar_try_wait(smem_u32(&full[s]), ph);
                    const bool done2 = mbar_try_wait(smem_u32(&empty[s2]), ph2);
                    if (!loaded) wait1(&full[s], ph, kErrTimeoutTma);
                    if (!done2 && primed) wait1(&empty[s2], ph2, kErrTimeoutMma);
                    if (broken) break;
                    tc_fence_after();
                    const uint32_t aX = sbase + s * STAGE_BYTES, aS = aX + 2 * kCodeBytes;
                    const uint64_t dX = desc_at(kDesc, aX), dW = desc_at(kDesc, aX + kCodeBytes), dS = desc_at(sDesc, aS);
                    const uint32_t cX = cS, cW = cX + 16;
                    const int nk = min(BK / kMmaK, (p.K - ks * BK) / kMmaK);
                    const uint32_t more = ks > 0;
                    if (elect_one()) {
                        // (at the end of K some tiles hold other rows' scales: no product reads them)
#pragma unroll
                        for (int i = 0; i < kTiles; ++i) {
                            copy_scales_pair(cX + 4 * i, dS + 32 * i);
                            copy_scales_pair(cW + 8 * i, dS + (S_BYTES >> 4) + 32 * i);
                            copy_scales_pair(cW + 8 * i + 4, dS + (2 * S_BYTES >> 4) + 32 * i);
                        }
#pragma unroll
                        for (int kk = 0; kk < BK / kMmaK; ++kk) {
                            constexpr bool nv = FMT == quant::kNvfp4;
                            const int tile = nv ? kk : kk >> 1;
                            if (kk < nk)
                                mma_scaled_pair<FMT>(d, dX + 2 * kk, dW + 2 * kk, nv ? ID : ID | scale_id(2 * (kk & 1)),
                                                     cX + 4 * tile, cW + 8 * tile, kk > 0 ? 1u : more);
                        }
                        commit_pair(&empty[s]);
                        if (ks + 1 == ksteps) commit_pair(&acc_full[it & 1]);
                    }
                    __syncwarp();
                    cS = cS == tbase + kScales ? cS + kScaleCols : tbase + kScales;
                    if (++s == kStages) s = 0, ph ^= 1;
                    if (++s2 == kStages) s2 = 0, ph2 ^= 1, primed = true;
                }
            }
        }
    } else {
        // ---------------- epilogue: this CTA's 128 tokens
        const int q4 = warp & 3, et = tid - 64;
        const bool upper = warp >= 6;  // two warps per lane quarter share the tile's columns
        const uint32_t tl = static_cast<uint32_t>(32 * q4) << 16;
        const uint32_t free_bar = cluster_addr(acc_free, 0);
        grid_wait();
        uint32_t it = 0;
        for (int t = first; t < ntiles; t += step, ++it) {
            int tm, tn;
            coords(t, tm, tn);
            const int row = tm * kTileM + 128 * rank + 32 * q4 + lane, n0 = tn * kTileN;
            float* gw = s_gw + (it & 1) * kTileN;
            for (int i = et; i < kTileN; i += 256) gw[i] = n0 + i < p.N ? p.gw[n0 + i] : 0.0f;
            const float2 gx = split_scale(row < p.T ? p.gx[row] : 1.0f);
            named_barrier_sync(1, 256);
            wait1(&acc_full[it & 1], (it >> 1) & 1, kErrTimeoutMma);
            __syncwarp();
            tc_fence_after();
            const uint32_t acc = tbase + tl + ((it & 1) ? kAcc1 : 0);
            // the shared columns first, into registers, and the next tile's products may start: columns 160 .. 255
            // of the first accumulator, 0 .. 95 of the second.  A warp stores its columns in two parts of 64: one
            // that holds its shared columns, then one that holds none.
            const bool second = (it & 1) != 0;
            const int part0 = second ? (upper ? 0 : 64) : (upper ? 192 : 128);
            const int part1 = (second ? 128 : 0) + (upper ? 64 : 0);
            float v0[32], v1[32];
            if (upper) {  // all 64 of its first part are shared
                tmem_ld32(acc + part0, v0);
                tmem_ld32(acc + part0 + 32, v1);
            } else {      // 32 are: its last (160 .. 191) or first (64 .. 95)
                tmem_ld32(acc + part0 + (second ? 0 : 32), v0);
            }
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            // Relaxed: the order that the next products need does not come from the arrival's own semantics.  Tensor
            // memory is ordered by the tcgen05 operations: wait::ld completes the loads, fence::before_thread_sync
            // orders them before whatever instruction signals the other thread, and the issuer's
            // fence::after_thread_sync behind its wait orders its products after that.  Nothing else is handed over
            // (the row scales in s_gw are this CTA's epilogue's own); a release at cluster scope would wait for the
            // previous tile's output stores, about 1,300 cycles a tile.
            if (lane == 0)
                asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(free_bar) : "memory");
            uint8_t* stage = smem + OFF_OUT + (warp - 2) * kOutBytes;
            const int t0 = row - lane;
            uint32_t lo[16], hi[16];
            auto from_tmem = [&](int c, uint32_t(&o)[16]) {
                tmem_ld32(acc + c, v1);
                tmem_ld_wait();
                scale_pack32(v1, gx, gw + c, o);
            };
            auto emit = [&](int c) {
                if (n0 + c < p.N) store_tile32x64(p, t0, n0 + c, lo, hi, stage, lane);
            };
            if (upper) {
                scale_pack32(v0, gx, gw + part0, lo);
                scale_pack32(v1, gx, gw + part0 + 32, hi);
            } else if (second) {
                scale_pack32(v0, gx, gw + part0, lo);
                from_tmem(part0 + 32, hi);
            } else {
                scale_pack32(v0, gx, gw + part0 + 32, hi);
                from_tmem(part0, lo);
            }
            emit(part0);
            from_tmem(part1, lo);
            from_tmem(part1 + 32, hi);
            emit(part1);
        }
    }
    tc_fence_before();
    cluster_sync();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(512u) : "memory");
}

}  // namespace gdn
