// Microscaled 4-bit rows: quantisation of bf16 rows to E2M1 codes with a scale per block, and the
// values the codes stand for.
//
//   value[r][k] = e2m1(code[r][k]) * scale[r][k / B] * row_scale[r],   e2m1 in +-{0, .5, 1, 1.5, 2, 3, 4, 6}
//
// nvfp4 (B = 16, E4M3 scales): row_scale g = the least power of two >= amax_row / (448 * 6) (at least
// 2^-100), so that every block scale s = rn_e4m3(amax_block / (6 g)) is at most 448; code =
// rn_e2m1(x / (s g)).  A power of two costs the block scales nothing (E4M3 has as many fraction bits at
// any exponent), makes x / g exact, and makes value exact in bf16 (2 + 4 significant bits).
// mxfp4 (B = 32, power-of-two scales): s = 2^max(-127, floor(log2 amax_block) - 2), code =
// rn_e2m1(x / s), saturating at 6; g = 1.
// A row that holds an infinity or a NaN gets row_scale NaN and codes 0, so all its values are NaN.
//
// Layout: codes [rows][K / 2], element 2i in the low nibble of byte i.  Scales in tiles of 128 rows x 4
// blocks, 512 bytes each, the order in which the tensor core's scale operands are copied to tensor
// memory: tile (r / 128, b / 4) at ((r / 128) * tiles_per_row + b / 4) * 512, and in it row r, block b at
// (r % 32) * 16 + (r / 32 % 4) * 4 + b % 4.
#pragma once

#include "common.cuh"

namespace gdn {
namespace quant {

constexpr int kNvfp4 = 0, kMxfp4 = 1;  // enum gdn_quant_format
constexpr uint32_t kTileBytes = 512;
constexpr int kUnit = 16;        // elements per thread and step
constexpr int kMaxGroup = 512;   // threads per row

__host__ __device__ constexpr int block_of(int fmt) { return fmt == kNvfp4 ? 16 : 32; }
// scale tiles across a row of K elements
__host__ __device__ constexpr int scale_tiles(int fmt, int K) { return (K + 4 * block_of(fmt) - 1) / (4 * block_of(fmt)); }

// Byte offset of the scale of row r, block b.
__host__ __device__ __forceinline__ size_t scale_offset(size_t r, int b, int tiles) {
    return ((r >> 7) * tiles + (b >> 2)) * kTileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// 8 floats -> 8 E2M1 codes (round to nearest even, saturating), element i in nibble i.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float* v) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}\n"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

__device__ __forceinline__ uint32_t e4m3_bits(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return r & 0xffu;
}

__device__ __forceinline__ float e4m3_value(uint32_t b) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xffffu)));
}

// Largest bf16 magnitude of 16 packed elements, as bits (a NaN among them: 0x7fff, above infinity).
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t amax_bits16(const uint4& a, const uint4& b) {
    const uint32_t m = 0x7fff7fffu;
    uint32_t r = max_bf16x2(max_bf16x2(a.x & m, a.y & m), max_bf16x2(a.z & m, a.w & m));
    r = max_bf16x2(r, max_bf16x2(max_bf16x2(b.x & m, b.y & m), max_bf16x2(b.z & m, b.w & m)));
    return max(r & 0xffffu, r >> 16);
}

// v rounded to 16 significant bits.  A quotient formed with a rounded reciprocal may miss an exact tie by a
// relative 2^-22; the quotients taken here (8 bits over at most 4) are ties of the format rounded to next
// or at least a relative 1/255 away from one, so this restores the former and keeps the latter apart (and
// keeps the sign of a zero).
__device__ __forceinline__ float snap16(float v) { return __uint_as_float((__float_as_uint(v) + 0x80u) & 0xffffff00u); }

// A row's scale from its largest magnitude (bf16 bits).
template <int FMT>
__device__ __forceinline__ float row_scale_of(uint32_t row_max) {
    if (row_max >= 0x7f80u) return __uint_as_float(0x7fc00000u);
    if (FMT != kNvfp4) return 1.0f;
    // amax = (1 + m / 128) 2^e against 2688 = (1 + 40 / 128) 2^11
    return pow2f(max(static_cast<int>(row_max >> 7) - 127 - 11 + ((row_max & 127u) > 40u ? 1 : 0), -100));
}

// The 16 codes of one thread's unit and its block's scale byte, from the unit, the block's and the
// row's largest magnitudes.
template <int FMT>
__device__ __forceinline__ void quantize_unit(const uint4& a, const uint4& b, uint32_t block_max, uint32_t row_max,
                                              uint2& codes, uint32_t& scale) {
    const bool finite = row_max < 0x7f80u;
    float inv;  // 1 / (s g)
    if constexpr (FMT == kNvfp4) {
        const int j = max(static_cast<int>(row_max >> 7) - 127 - 11 + ((row_max & 127u) > 40u ? 1 : 0), -100);
        const float inv_g = pow2f(-j);
        scale = e4m3_bits(snap16(bf16_bits_to_float(static_cast<uint16_t>(block_max)) * inv_g * (1.0f / 6.0f)));
        const float s = e4m3_value(scale);
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
        inv = s > 0.0f ? r * inv_g : 0.0f;
    } else {
        const int e = max(static_cast<int>(block_max >> 7) - 127 - 2, -127);
        scale = static_cast<uint32_t>(e + 127);
        inv = pow2f(-e);
    }
    if (!finite) {
        scale = 0;
        codes = make_uint2(0u, 0u);
        return;
    }
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16) * inv;
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * inv;
    }
    if constexpr (FMT == kNvfp4) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = snap16(v[i]);
    }
    codes.x = pack_e2m1x8(v);
    codes.y = pack_e2m1x8(v + 8);
}

struct Params {
    const uint16_t* x;  // bf16 [rows][K]
    uint8_t* codes;
    uint8_t* scales;
    float* row_scale;
    int rows, K, tiles;
};

}  // namespace quant

// One row per group of blockDim.x threads (a multiple of 32), blockDim.y rows per CTA and step; persistent
// CTAs walk the rows.  A thread takes units of 16 elements, blockDim.x units apart; a row is read once while
// it fits in kHold units per thread (K <= 16384) and twice above.  The next row's first units are requested
// before this row's largest magnitude is known, so a row's load latency overlaps the previous row's
// arithmetic.  kHold is 1 up to K = 8192, else 2 (registers that a short row leaves empty cost occupancy:
// 16480 x 5120 rows 49 us with 1, 60 us with 2).  Bound: HBM (2 bytes read and about 0.57 written per element).
template <int FMT, int kHold>
__global__ void __launch_bounds__(quant::kMaxGroup) gdn_quantize_kernel(const quant::Params p) {
    using namespace quant;
    __shared__ uint32_t s_max[2][kMaxGroup / 32];
    // a projection launched behind this kernel may start its prologue (it waits for this grid's end before
    // it reads what is written here)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int units = p.K / kUnit, step = blockDim.x, lane = threadIdx.x & 31;
    const int groups = (p.rows + blockDim.y - 1) / blockDim.y;  // steps of all CTAs
    uint4 a[kHold], b[kHold];
    auto load = [&](int g) {
        const int row = g * blockDim.y + threadIdx.y;
        const uint4* src = reinterpret_cast<const uint4*>(p.x + (size_t)row * p.K);
#pragma unroll
        for (int h = 0; h < kHold; ++h) {
            const int u = threadIdx.x + h * step;
            a[h] = b[h] = make_uint4(0, 0, 0, 0);
            if (row < p.rows && u < units) {
                a[h] = __ldg(src + 2 * u);
                b[h] = __ldg(src + 2 * u + 1);
            }
        }
    };
    int buf = 0;
    load(blockIdx.x);
    for (int g = blockIdx.x; g < groups; g += gridDim.x, buf ^= 1) {
        const int row = g * blockDim.y + threadIdx.y;
        const bool active = row < p.rows;  // (rows do not share a warp)
        const uint4* src = reinterpret_cast<const uint4*>(p.x + (size_t)(active ? row : 0) * p.K);
        uint4 ca[kHold], cb[kHold];
        uint32_t bm[kHold], rm = 0;
#pragma unroll
        for (int h = 0; h < kHold; ++h) {
            ca[h] = a[h];
            cb[h] = b[h];
            bm[h] = amax_bits16(ca[h], cb[h]);
            rm = max(rm, bm[h]);
        }
        for (int u = threadIdx.x + kHold * step; u < units; u += step)
            if (active) rm = max(rm, amax_bits16(__ldg(src + 2 * u), __ldg(src + 2 * u + 1)));
        if (g + gridDim.x < groups) load(g + gridDim.x);
        rm = __reduce_max_sync(0xffffffffu, rm);
        if (step > 32) {  // the row's warps (blockDim.y rows of step / 32 warps, at most kMaxGroup threads in all)
            const int w = threadIdx.x >> 5, nw = step >> 5;
            if (lane == 0) s_max[buf][threadIdx.y * nw + w] = rm;
            __syncthreads();  // (two buffers: the next row's maxima do not overwrite those still being read)
            rm = __reduce_max_sync(0xffffffffu, s_max[buf][threadIdx.y * nw + (lane < nw ? lane : 0)]);
        }
        if (!active) continue;
        auto emit = [&](int u, const uint4& ua, const uint4& ub, uint32_t um) {
            uint2 codes;
            uint32_t scale;
            if constexpr (FMT == kMxfp4) um = max(um, __shfl_xor_sync(0xffffffffu, um, 1));  // a block is two units
            quantize_unit<FMT>(ua, ub, um, rm, codes, scale);
            if (u < units) *reinterpret_cast<uint2*>(p.codes + (size_t)row * (p.K / 2) + (size_t)u * 8) = codes;
            // 4 scales of a tile row are one aligned word
            constexpr int kPer = block_of(FMT) / kUnit;  // units per block
            uint32_t word = u < units ? scale << (8 * ((lane / kPer) & 3)) : 0u;
            word = (lane % kPer == 0) ? word : 0u;
#pragma unroll
            for (int off = kPer; off < 4 * kPer; off <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, off);
            if (lane % (4 * kPer) == 0 && u < units)
                *reinterpret_cast<uint32_t*>(p.scales + scale_offset(row, u / kPer, p.tiles)) = word;
        };
        const int u0 = static_cast<int>(threadIdx.x & ~31u);
#pragma unroll
        for (int h = 0; h < kHold; ++h)
            if (u0 + h * step < units) emit(threadIdx.x + h * step, ca[h], cb[h], bm[h]);
        for (int v0 = u0 + kHold * step; v0 < units; v0 += step) {
            const int u = v0 + lane;
            uint4 ua = make_uint4(0, 0, 0, 0), ub = ua;
            if (u < units) {
                ua = __ldg(src + 2 * u);
                ub = __ldg(src + 2 * u + 1);
            }
            emit(u, ua, ub, amax_bits16(ua, ub));
        }
        if (threadIdx.x == 0) p.row_scale[row] = row_scale_of<FMT>(rm);
    }
}

// 16 codes -> 16 bf16 values per thread and step (exact: see the header), rows and threads as above.
// Bound: HBM.
template <int FMT>
__global__ void __launch_bounds__(quant::kMaxGroup)
    gdn_dequantize_kernel(const uint8_t* codes, const uint8_t* scales, const float* row_scale, int rows, int K, int tiles,
                          uint16_t* out) {
    using namespace quant;
    const int units = K / kUnit;
    for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < rows; row += (int64_t)gridDim.x * blockDim.y) {
        const float g = __ldg(row_scale + row);
        const uint2* src = reinterpret_cast<const uint2*>(codes + (size_t)row * (K / 2));
        uint4* dst = reinterpret_cast<uint4*>(out + (size_t)row * K);
        for (int u = threadIdx.x; u < units; u += blockDim.x) {
            const uint2 c = __ldg(src + u);
            const uint32_t sb = __ldg(scales + scale_offset(row, FMT == kNvfp4 ? u : u >> 1, tiles));
            float s;
            if (FMT == kNvfp4) s = e4m3_value(sb);
            else s = sb == 255u ? __uint_as_float(0x7fc00000u) : (sb == 0u ? __uint_as_float(1u << 22) : __uint_as_float(sb << 23));
            s *= g;
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t byte = ((j < 4 ? c.x : c.y) >> (8 * (j & 3))) & 0xffu;
                uint32_t h;
                asm("{\n\t.reg .b8 b0, b1;\n\tmov.b16 {b0, b1}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\t}\n"
                    : "=r"(h)
                    : "h"(static_cast<uint16_t>(byte)));
                const __half2 h2 = *reinterpret_cast<__half2*>(&h);
                o[j] = pack_bf16x2(__low2float(h2) * s, __high2float(h2) * s);
            }
            dst[2 * u] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[2 * u + 1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

}  // namespace gdn
