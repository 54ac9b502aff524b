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
    const uint8_t *sx, *sw;      // block scales
    const float *gx, *gw;        // row scales [T], [N]
    int nseg;                    // output segments over the features, as in the bf16 projections
    GemmSegment seg[4];
};

__device__ __forceinline__ uint16_t* output_at(const Params& p, int n, int t) {
    int sg = 0;
#pragma unroll
    for (int i = 1; i < 4; ++i)
        if (i < p.nseg && n >= p.seg[i].col0) sg = i;
    return p.seg[sg].dst + (size_t)t * p.seg[sg].ld + (n - p.seg[sg].col0);
}

constexpr int BM = 128;                              // features per tile (rows of the A operand)
constexpr uint32_t W_BYTES = BM * BK / 2;            // 16 KB
constexpr uint32_t S_BYTES = 4 * quant::kTileBytes;  // scales of 128 rows, at most
constexpr int kThreads = 192;                        // warp 0 loads, warp 1 products, warps 2-5 epilogue

template <int BN>
struct Cfg {
    static constexpr uint32_t X_BYTES = BN * BK / 2;
    static constexpr uint32_t STAGE_BYTES = W_BYTES + X_BYTES + 2 * S_BYTES;
    static constexpr int kStages = 6;
    static constexpr uint32_t OFF_MISC = kStages * STAGE_BYTES;
    static constexpr uint32_t SMEM_BYTES = OFF_MISC + 256 + 1024;
    // tensor memory: the sums (BN columns), then per stage 16 columns of weight scales and 16 of token scales
    static constexpr uint32_t TMEM_COLS = 512;
    static_assert(BN + 32 * kStages <= 512, "tensor memory");
    static_assert(X_BYTES % 1024 == 0, "swizzle atoms");
};

}  // namespace qproj

// One CTA per 128 features x BN tokens: the weights are the A operand (128 rows), the tokens the B
// operand, so that few tokens still fill the tensor core's 128 lanes.  Token tiles start at multiples
// of 128 rows (BN = 128), or there is one (BN < 128), so that their scales are whole tiles.
template <int FMT, int BN>
__global__ void __launch_bounds__(qproj::kThreads, 1)
    gdn_qproj_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                     const qproj::Params p) {
    using namespace qproj;
    using C = Cfg<BN>;
    constexpr int kTiles = kTilesPerStage(FMT);
    constexpr uint32_t ID = idesc(FMT, BM, BN);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_MISC);
    uint64_t* empty = full + C::kStages;
    uint64_t* done = empty + C::kStages;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 128);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n0 = blockIdx.x * BM, t0 = blockIdx.y * BN;
    const int ksteps = (p.K + BK - 1) / BK;

    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        fence_barrier_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmX);
    }
    if (warp == 0) {
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

    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (int ks = 0; ks < ksteps; ++ks) {
                const int s = ks % C::kStages;
                if (ks >= C::kStages) wait1(&empty[s], ((ks / C::kStages) - 1) & 1, kErrTimeoutTma);
                if (broken) break;  // nothing more is requested
                uint8_t* st = smem + s * C::STAGE_BYTES;
                const uint32_t sbytes = min(kTiles, p.tiles - ks * kTiles) * quant::kTileBytes;
                mbar_arrive_expect_tx(&full[s], W_BYTES + C::X_BYTES + 2 * sbytes);
                tma_load_2d(st, &tmW, ks * (BK / 2), n0, &full[s]);
                tma_load_2d(st + W_BYTES, &tmX, ks * (BK / 2), t0, &full[s]);
                bulk_load(st + W_BYTES + C::X_BYTES,
                          p.sw + ((size_t)(n0 >> 7) * p.tiles + ks * kTiles) * quant::kTileBytes, sbytes, &full[s]);
                bulk_load(st + W_BYTES + C::X_BYTES + S_BYTES,
                          p.sx + ((size_t)(t0 >> 7) * p.tiles + ks * kTiles) * quant::kTileBytes, sbytes, &full[s]);
                issued = ks + 1;
            }
            // no copy is in flight when the CTA exits, whatever the other warps did
            for (int ks = max(issued - C::kStages, 0); ks < issued; ++ks)
                mbar_wait(&full[ks % C::kStages], (ks / C::kStages) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            for (int ks = 0; ks < ksteps; ++ks) {
                const int s = ks % C::kStages;
                wait1(&full[s], (ks / C::kStages) & 1, kErrTimeoutTma);
                if (broken) break;
                tc_fence_after();
                const uint32_t aW = sbase + s * C::STAGE_BYTES, aX = aW + W_BYTES, aSw = aX + C::X_BYTES;
                const uint32_t cS = tbase + BN + 32 * s;
                const int tiles = min(kTiles, p.tiles - ks * kTiles);
                for (int i = 0; i < tiles; ++i) {
                    copy_scales(cS + 4 * i, scale_desc(aSw + i * quant::kTileBytes));
                    copy_scales(cS + 16 + 4 * i, scale_desc(aSw + S_BYTES + i * quant::kTileBytes));
                }
                const int nk = min(BK / kMmaK, (p.K - ks * BK) / kMmaK);
                for (int kk = 0; kk < nk; ++kk) {
                    const int tile = FMT == quant::kNvfp4 ? kk : kk >> 1;
                    const uint32_t id = FMT == quant::kNvfp4 ? ID : ID | scale_id(2 * (kk & 1));
                    mma_scaled<FMT>(tbase, sw128_desc(aW + kk * 32, 16, 1024), sw128_desc(aX + kk * 32, 16, 1024), id,
                                    cS + 4 * tile, cS + 16 + 4 * tile, (ks > 0 || kk > 0) ? 1u : 0u);
                }
                mma_commit(&empty[s]);
            }
            mma_commit(done);
        }
        __syncwarp();
    } else {
        const int q4 = warp & 3;  // TMEM lane quarter of this warp
        const uint32_t tl = static_cast<uint32_t>(32 * q4) << 16;
        const int n = n0 + 32 * q4 + lane;
        const float gw = n < p.N ? __ldg(p.gw + n) : 0.0f;
        wait1(done, 0, kErrTimeoutMma);
        __syncwarp();
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; j < BN / 16; ++j) {
            float v[16];
            tmem_ld16(tbase + tl + 16 * j, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int t = t0 + 16 * j + e;
                if (n < p.N && t < p.T) *output_at(p, n, t) = float_to_bf16_bits(v[e] * (gw * __ldg(p.gx + t)));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tbase, C::TMEM_COLS);
}

}  // namespace gdn
