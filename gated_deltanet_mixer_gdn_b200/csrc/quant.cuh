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
constexpr int kUnit = 32;        // elements per thread and step of the quantisation
constexpr int kMaxGroup = 512;   // threads per row

__host__ __device__ constexpr int block_of(int fmt) { return fmt == kNvfp4 ? 16 : 32; }
// scale tiles across a row of K elements
__host__ __device__ constexpr int scale_tiles(int fmt, int K) { return (K + 4 * block_of(fmt) - 1) / (4 * block_of(fmt)); }

// Byte offset of the scale of row r, block b.
__host__ __device__ __forceinline__ size_t scale_offset(size_t r, int b, int tiles) {
    return ((r >> 7) * tiles + (b >> 2)) * kTileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

// 32 bytes to a 32-byte boundary: one sector per lane (stored as two halves, 32 bytes apart between lanes, each
// sector goes to L2 twice: 16480 x 5120 values 41 us against 38).
__device__ __forceinline__ void store32(void* p, const uint4& a, const uint4& b) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
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

// A quotient formed with a rounded reciprocal may miss an exact tie by a relative 2^-21.  The quotients taken here
// (8 bits over at most 4) are ties of the format rounded to next, or at least a relative 1/255 away from one: taken
// kAbove times too large (2^-17), and their last 8 bits dropped, ties come out exact, the others stay on their side,
// and a zero keeps its sign.
constexpr float kAbove = 0x1.00008p0f;
__device__ __forceinline__ float snap16(float v) { return __uint_as_float(__float_as_uint(v) & 0xffffff00u); }

// A row's scale from its largest magnitude (bf16 bits).
template <int FMT>
__device__ __forceinline__ float row_scale_of(uint32_t row_max) {
    if (row_max >= 0x7f80u) return __uint_as_float(0x7fc00000u);
    if (FMT != kNvfp4) return 1.0f;
    // amax = (1 + m / 128) 2^e against 2688 = (1 + 40 / 128) 2^11
    return pow2f(max(static_cast<int>(row_max >> 7) - 127 - 11 + ((row_max & 127u) > 40u ? 1 : 0), -100));
}

// 1 / row scale (nvfp4), from the row's largest magnitude.
__device__ __forceinline__ float inv_row_scale(uint32_t row_max) {
    return pow2f(-max(static_cast<int>(row_max >> 7) - 127 - 11 + ((row_max & 127u) > 40u ? 1 : 0), -100));
}

// A block's scale byte from its largest magnitude, and what its elements are multiplied by: 1 / (s g) (nvfp4:
// kAbove times that, for snap16).
template <int FMT>
__device__ __forceinline__ float block_scale(uint32_t block_max, float inv_g, uint32_t& byte) {
    if constexpr (FMT == kNvfp4) {
        byte = e4m3_bits(snap16(bf16_bits_to_float(static_cast<uint16_t>(block_max)) * inv_g * (kAbove / 6.0f)));
        const float s = e4m3_value(byte);
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
        return s > 0.0f ? r * inv_g * kAbove : 0.0f;
    } else {
        const int e = max(static_cast<int>(block_max >> 7) - 127 - 2, -127);
        byte = static_cast<uint32_t>(e + 127);
        return pow2f(-e);
    }
}

// 16 codes of bf16 elements times inv.
template <int FMT>
__device__ __forceinline__ uint2 codes16(const uint4& a, const uint4& b, float inv) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16) * inv;
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * inv;
    }
    if constexpr (FMT == kNvfp4) {  // (mxfp4: inv is a power of two, the quotients are exact)
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = snap16(v[i]);
    }
    return make_uint2(pack_e2m1x8(v), pack_e2m1x8(v + 8));
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
// CTAs walk the rows.  A thread takes units of 32 elements (two blocks of 16 or one of 32), blockDim.x units
// apart; a row is read once up to K = 16384 (one unit per thread) and twice above.  The next row is requested
// before this row's largest magnitude is known, so a row's load latency overlaps the previous row's
// arithmetic.  Bound: HBM (2 bytes read and about 0.57 written per element) and, close behind, issue: units
// of 16 elements, with the row's bookkeeping on half as much data, took 242 instructions each.
template <int FMT>
__global__ void __launch_bounds__(quant::kMaxGroup) gdn_quantize_kernel(const quant::Params p) {
    using namespace quant;
    __shared__ uint32_t s_max[2][kMaxGroup / 32];
    grid_wait();
    launch_dependents();  // a projection behind this kernel may start its prologue and load its weights
    const int units = p.K / kUnit, step = blockDim.x, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int groups = (p.rows + blockDim.y - 1) / blockDim.y;  // steps of all CTAs
    const int w = tid >> 5, nw = step >> 5;                     // the row's warps
    uint4 next[4];
    // Past the row its last unit is loaded, past the last row that one: neither changes a maximum, and nothing is stored.
    // (Predicated loads of zeros cost 16480 x 5120 nvfp4 40.2 us against 38.9; clamped addresses on the first load, whose
    // latency few rows wait for, 8 x 6144 2.7 us against 2.1.)
    auto load = [&](int g, int u, uint4(&x)[4]) {
        const int row = min(static_cast<int>(g * blockDim.y + threadIdx.y), p.rows - 1), uu = min(u, units - 1);
        const bool ok = GDN_CHECK(row >= 0 && row < p.rows && uu >= 0 && (uu + 1) * kUnit <= p.K);
        const uint4* src = reinterpret_cast<const uint4*>(p.x + (ok ? (size_t)row * p.K : 0)) + (ok ? 4 * uu : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = src[i];
    };
    auto load_first = [&](int g, int u, uint4(&x)[4]) {
        const int row = g * blockDim.y + threadIdx.y;
        const uint4* src = reinterpret_cast<const uint4*>(p.x + (size_t)row * p.K) + 4 * u;
        const bool in = row < p.rows && u < units && GDN_CHECK(row >= 0 && u >= 0 && (u + 1) * kUnit <= p.K);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = in ? src[i] : make_uint4(0, 0, 0, 0);
    };
    load_first(blockIdx.x, tid, next);
    for (int g = blockIdx.x, buf = 0; g < groups; g += gridDim.x, buf ^= 1) {
        const int row = g * blockDim.y + threadIdx.y;
        const bool active = row < p.rows;  // (rows do not share a warp)
        uint4 x[4] = {next[0], next[1], next[2], next[3]};
        uint32_t m0 = amax_bits16(x[0], x[1]), m1 = amax_bits16(x[2], x[3]);
        uint32_t rm = max(m0, m1);
        for (int u = tid + step; u < units; u += step) {
            uint4 y[4];
            load(g, u, y);
            rm = max(rm, max(amax_bits16(y[0], y[1]), amax_bits16(y[2], y[3])));
        }
        if (g + gridDim.x < groups) load(g + gridDim.x, tid, next);
        rm = __reduce_max_sync(0xffffffffu, rm);
        if (step > 32) {
            if (lane == 0) s_max[buf][threadIdx.y * nw + w] = rm;
            __syncthreads();  // (two buffers: the next row's maxima do not overwrite those still being read)
            rm = __reduce_max_sync(0xffffffffu, s_max[buf][threadIdx.y * nw + (lane < nw ? lane : 0)]);
        }
        if (!active) continue;
        const bool finite = rm < 0x7f80u;
        const float inv_g = FMT == kNvfp4 ? inv_row_scale(rm) : 1.0f;
        uint8_t* codes = p.codes + (size_t)row * (p.K / 2);
        uint8_t* scales = p.scales + scale_offset(row, 0, p.tiles);
        auto emit = [&](int u) {
            uint32_t b0, b1, word;
            float i0, i1;
            if constexpr (FMT == kNvfp4) {
                i0 = block_scale<FMT>(m0, inv_g, b0);
                i1 = block_scale<FMT>(m1, inv_g, b1);
                word = b0 | (b1 << 8);
            } else {
                i0 = i1 = block_scale<FMT>(max(m0, m1), 1.0f, b0);
                word = b0;
            }
            uint2 lo = codes16<FMT>(x[0], x[1], i0), hi = codes16<FMT>(x[2], x[3], i1);
            if (!finite) lo = hi = make_uint2(0u, 0u), word = 0u;
            // 4 scales of a tile row are one aligned word: of 2 lanes, or of 4 (past the row: zeros)
            if (u >= units) word = 0u;
            if constexpr (FMT == kNvfp4) {
                word |= __shfl_down_sync(0xffffffffu, word, 1) << 16;
            } else {
                word |= __shfl_down_sync(0xffffffffu, word, 1) << 8;
                word |= __shfl_down_sync(0xffffffffu, word, 2) << 16;
            }
            constexpr int kLanes = FMT == kNvfp4 ? 2 : 4;
            if (u < units && GDN_CHECK(u >= 0 && row < p.rows && (u + 1) * kUnit <= p.K && u / kLanes < p.tiles)) {
                *reinterpret_cast<uint4*>(codes + 16 * u) = make_uint4(lo.x, lo.y, hi.x, hi.y);
                if ((lane & (kLanes - 1)) == 0)
                    *reinterpret_cast<uint32_t*>(scales + (u / kLanes) * kTileBytes) = word;
            }
        };
        if (32 * w < units) emit(tid);
        for (int u0 = 32 * w + step; u0 < units; u0 += step) {  // (whole warps)
            load(g, u0 + lane, x);
            m0 = amax_bits16(x[0], x[1]);
            m1 = amax_bits16(x[2], x[3]);
            emit(u0 + lane);
        }
        if (tid == 0) p.row_scale[row] = row_scale_of<FMT>(rm);
    }
}

// 16 codes -> 16 bf16 values per thread and step (exact: see the header), rows and threads as above.
// Bound: HBM.
template <int FMT>
__global__ void __launch_bounds__(quant::kMaxGroup)
    gdn_dequantize_kernel(const uint8_t* codes, const uint8_t* scales, const float* row_scale, int rows, int K, int tiles,
                          uint16_t* out) {
    using namespace quant;
    grid_wait();
    const int units = K / 16;
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;  // (rows are multiples of 128 bytes)
    for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < rows; row += (int64_t)gridDim.x * blockDim.y) {
        const float g = row_scale[row];
        const uint2* src = reinterpret_cast<const uint2*>(codes + (size_t)row * (K / 2));
        uint4* dst = reinterpret_cast<uint4*>(out + (size_t)row * K);
        for (int u = threadIdx.x; u < units; u += blockDim.x) {
            if (!GDN_CHECK(row >= 0 && (u + 1) * 16 <= K && (FMT == kNvfp4 ? u : u >> 1) / 4 < tiles)) break;
            const uint2 c = src[u];
            const uint32_t sb = scales[scale_offset(row, FMT == kNvfp4 ? u : u >> 1, tiles)];
            float s;
            if (FMT == kNvfp4) s = e4m3_value(sb);
            else s = sb == 255u ? __uint_as_float(0x7fc00000u) : (sb == 0u ? __uint_as_float(1u << 22) : __uint_as_float(sb << 23));
            // code * (s g); where s g overflows (row scales made elsewhere) (code * s) g: a code of 0 stays 0, and small
            // codes may have finite values
            const bool far = fabsf(s * g) > 0x1.fffffep127f;  // (not for a NaN)
            const float2 f0 = far ? make_float2(s, s) : make_float2(s * g, s * g);
            const float2 f1 = far ? make_float2(g, g) : make_float2(1.0f, 1.0f);
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t byte = ((j < 4 ? c.x : c.y) >> (8 * (j & 3))) & 0xffu;
                uint32_t h;
                asm("{\n\t.reg .b8 b0, b1;\n\tmov.b16 {b0, b1}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\t}\n"
                    : "=r"(h)
                    : "h"(static_cast<uint16_t>(byte)));
                const float2 v = mul2(mul2(__half22float2(*reinterpret_cast<__half2*>(&h)), f0), f1);
                o[j] = pack_bf16x2(v.x, v.y);
            }
            const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
            if (wide) {
                store32(dst + 2 * u, lo, hi);
            } else {
                dst[2 * u] = lo;
                dst[2 * u + 1] = hi;
            }
        }
    }
}

}  // namespace gdn
