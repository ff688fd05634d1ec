// MXFP4 quantize and expand for gfx950.
//
// Quantize: b = max(E - 2, 0) with E the exponent field of the block's largest magnitude, which is
// 2^(floor(log2 amax) - 2) as an E8M0 byte, then code = nearest E2M1 of v 2^(127 - b).  The product with
// a power of two is exact (v 2^(127 - b) lies below 8), so the only rounding is the conversion to
// E2M1.  Nothing outside a block is needed: one pass, one launch.
//
// Bound by HBM: source bytes in, 17/32 byte out per element.  A lane takes 8 elements (16 bytes of a
// 16-bit source; 16 elements of a one-byte one), the four (two) lanes of a block agree on its largest
// magnitude by DPP moves, and codes leave as one dword (two) per lane, consecutive lanes to consecutive
// addresses; four chunks per lane are loaded before the first is used.  12288 x 4096, calls in a row over inputs of 1 GB
// in turn, which the Infinity Cache does not hold: fp32 41.4 us (5.5 TB/s), bf16 25.0 us (5.1 TB/s); expand to bf16
// 23.2 us (5.5 TB/s), to fp32 44.6 us (5.1 TB/s).  The same input again and again: 33.6, 21.6, 20.8 and 37.4 us.  A
// device copy of 1 GiB moves 5.07 TB/s.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "mx.h"

namespace nvfp4 {

namespace {

constexpr int kPerLane = 4;  // chunks per lane per pass, all loaded before the first is used

// Elements per chunk: 16 of a one-byte source (4096 x 12288 E4M3: 19.6 us with 8), else 8.
template <int DT>
constexpr int chunk_elems() { return DT == NVFP4_E4M3 ? 16 : 8; }

template <int DT>
struct RawChunk {  // a chunk as loaded
    u32x4 v[DT == NVFP4_F32 ? 2 : 1];
};

template <int DT>
__device__ __forceinline__ void widen(const RawChunk<DT> &r, float s, float *v) {
    if constexpr (DT == NVFP4_E4M3) {
        // one rounding per element, as nvfp4_quantize widens an FP8 source
#pragma unroll
        for (int d = 0; d < 4; d++) {
            const int w = (int)r.v[0][d];
            v[4 * d] = __builtin_amdgcn_cvt_f32_fp8(w, 0) * s;
            v[4 * d + 1] = __builtin_amdgcn_cvt_f32_fp8(w, 1) * s;
            v[4 * d + 2] = __builtin_amdgcn_cvt_f32_fp8(w, 2) * s;
            v[4 * d + 3] = __builtin_amdgcn_cvt_f32_fp8(w, 3) * s;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
        if constexpr (DT == NVFP4_F32) {
            v[i] = u2f(r.v[i / 4][i % 4]);
        } else if constexpr (DT == NVFP4_BF16) {
            const uint32_t w = r.v[0][i / 2];
            v[i] = u2f(i % 2 ? w & 0xFFFF0000u : w << 16);
        } else if constexpr (DT == NVFP4_F16) {
            const uint32_t w = r.v[0][i / 2];
            v[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(i % 2 ? w >> 16 : w));
        }
    }
}

// cpr: chunks per row.
template <int DT>
__global__ __launch_bounds__(256) void k_mx_quant(const uint8_t *__restrict__ x, int64_t ld_bytes, int contiguous,
                                                  uint64_t nchunks, uint32_t cpr, const float *__restrict__ src_scale,
                                                  uint32_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                  int32_t *__restrict__ flags) {
    constexpr int CH = chunk_elems<DT>(), LPB = kMxBlock / CH;  // lanes per block
    constexpr int CB = CH * (DT == NVFP4_F32 ? 4 : DT == NVFP4_E4M3 ? 1 : 2);
    const float s = src_scale ? *src_scale : 1.0f;
    const uint64_t stride = (uint64_t)gridDim.x * blockDim.x;
    bool bad = false;
    for (uint64_t i0 = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i0 < nchunks; i0 += kPerLane * stride) {
        RawChunk<DT> raw[kPerLane];
#pragma unroll
        for (int j = 0; j < kPerLane; j++) {
            const uint64_t i = i0 + j * stride;
            raw[j] = RawChunk<DT>{};
            if (i < nchunks) {
                uint64_t off = i * CB;
                if (!contiguous) {
                    const uint64_t r = nchunks <= 0xFFFFFFFFull ? (uint32_t)i / cpr : i / cpr;
                    off = r * (uint64_t)ld_bytes + (i - r * cpr) * CB;
                }
#pragma unroll
                for (int d = 0; d < CB / 16; d++) raw[j].v[d] = *reinterpret_cast<const u32x4 *>(x + off + 16 * d);
            }
        }
#pragma unroll
        for (int j = 0; j < kPerLane; j++) {
            const uint64_t i = i0 + j * stride;
            // nchunks is a multiple of LPB (cols % 32 == 0), so the lanes of a block stay together
            if (i >= nchunks) break;
            float v[CH];
            widen<DT>(raw[j], s, v);
            uint32_t m = 0;
#pragma unroll
            for (int q = 0; q < CH; q++) m = max(m, f2u(v[q]) & 0x7FFFFFFFu);
            m = max(m, dpp_u32<kDppXor1>(m));
            if constexpr (LPB == 4) m = max(m, dpp_u32<kDppXor2>(m));
            const uint32_t e = m >> 23;
            uint32_t b = e > 2 ? e - 2 : 0;
            const float inv = u2f((254u - b) << 23);
#pragma unroll
            for (int q = 0; q < CH; q++) v[q] *= inv;
            uint32_t w[CH / 8];
#pragma unroll
            for (int d = 0; d < CH / 8; d++) w[d] = fp4_pack8(v + 8 * d);
            if (e == 255) {
                b = 255;
#pragma unroll
                for (int d = 0; d < CH / 8; d++) w[d] = 0;
                bad = true;
            }
            if constexpr (CH == 16) reinterpret_cast<u32x2 *>(codes)[i] = u32x2{w[0], w[1]};
            else codes[i] = w[0];
            if (i % LPB == 0) scales[i / LPB] = (uint8_t)b;
        }
    }
    if (flags && __any(bad) && (threadIdx.x & 63) == 0) atomicOr(flags, 1);
}

template <bool BF16_OUT>
__global__ __launch_bounds__(256) void k_mx_dequant(const uint32_t *__restrict__ codes,
                                                    const uint8_t *__restrict__ scales, uint64_t nchunks, uint32_t cpr,
                                                    int64_t ld_out, int contiguous, void *__restrict__ out) {
    const uint64_t stride = (uint64_t)gridDim.x * blockDim.x;
    for (uint64_t i0 = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i0 < nchunks; i0 += kPerLane * stride) {
        uint32_t w[kPerLane], sb[kPerLane];
#pragma unroll
        for (int j = 0; j < kPerLane; j++) {
            const uint64_t i = i0 + j * stride;
            w[j] = i < nchunks ? codes[i] : 0u;
            sb[j] = i < nchunks ? scales[i >> 2] : 0u;
        }
#pragma unroll
        for (int j = 0; j < kPerLane; j++) {
            const uint64_t i = i0 + j * stride;
            if (i >= nchunks) break;
            const float s = e8m0_to_f32(sb[j]);
            float v[8];
            fp4_unpack8_f32(w[j], v);
#pragma unroll
            for (int q = 0; q < 8; q++) v[q] *= s;
            uint64_t e = i * 8;
            if (!contiguous) {
                const uint64_t r = nchunks <= 0xFFFFFFFFull ? (uint32_t)i / cpr : i / cpr;
                e = r * (uint64_t)ld_out + (i - r * cpr) * 8;
            }
            if constexpr (BF16_OUT) {
                bf16x8 o;
#pragma unroll
                for (int q = 0; q < 8; q++) o[q] = (__bf16)v[q];
                *reinterpret_cast<bf16x8 *>(reinterpret_cast<__bf16 *>(out) + e) = o;
            } else {
                f32x4 *dst = reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(out) + e);
                dst[0] = f32x4{v[0], v[1], v[2], v[3]};
                dst[1] = f32x4{v[4], v[5], v[6], v[7]};
            }
        }
    }
}

unsigned codec_grid(uint64_t nchunks) {
    uint64_t grid = (nchunks + 256 * kPerLane - 1) / (256 * kPerLane);
    if (grid > ((uint64_t)1 << 20)) grid = (uint64_t)1 << 20;
    return (unsigned)(grid < 1 ? 1 : grid);
}

template <int DT>
void launch_quant_t(const void *x, int64_t ld_x, const float *src_scale, const mxfp4_tensor *out, int32_t *flags,
                    hipStream_t stream) {
    constexpr int EB = DT == NVFP4_F32 ? 4 : DT == NVFP4_E4M3 ? 1 : 2, CH = chunk_elems<DT>();
    const uint64_t nchunks = (uint64_t)out->rows * (uint64_t)(out->cols / CH);
    hipLaunchKernelGGL(k_mx_quant<DT>, dim3(codec_grid(nchunks)), dim3(256), 0, stream,
                       reinterpret_cast<const uint8_t *>(x), ld_x * EB, ld_x == out->cols || out->rows == 1 ? 1 : 0,
                       nchunks, (uint32_t)(out->cols / CH), src_scale, reinterpret_cast<uint32_t *>(out->codes),
                       out->scales, flags);
}

}  // namespace

hipError_t launch_mx_quantize(const void *x, nvfp4_dtype dt, int64_t ld_x, const float *src_scale,
                              const mxfp4_tensor *out, int32_t *flags, hipStream_t stream) {
    switch (dt) {
    case NVFP4_F32: launch_quant_t<NVFP4_F32>(x, ld_x, src_scale, out, flags, stream); break;
    case NVFP4_BF16: launch_quant_t<NVFP4_BF16>(x, ld_x, src_scale, out, flags, stream); break;
    case NVFP4_F16: launch_quant_t<NVFP4_F16>(x, ld_x, src_scale, out, flags, stream); break;
    default: launch_quant_t<NVFP4_E4M3>(x, ld_x, src_scale, out, flags, stream); break;
    }
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const mxfp4_tensor *in, void *out, nvfp4_dtype out_dtype, int64_t ld_out,
                                hipStream_t stream) {
    const uint64_t nchunks = (uint64_t)in->rows * (uint64_t)(in->cols / 8);
    const uint32_t cpr = (uint32_t)(in->cols / 8);
    const int contiguous = ld_out == in->cols || in->rows == 1 ? 1 : 0;
    const uint32_t *codes = reinterpret_cast<const uint32_t *>(in->codes);
    if (out_dtype == NVFP4_BF16)
        hipLaunchKernelGGL(k_mx_dequant<true>, dim3(codec_grid(nchunks)), dim3(256), 0, stream, codes, in->scales,
                           nchunks, cpr, ld_out, contiguous, out);
    else
        hipLaunchKernelGGL(k_mx_dequant<false>, dim3(codec_grid(nchunks)), dim3(256), 0, stream, codes, in->scales,
                           nchunks, cpr, ld_out, contiguous, out);
    return hipGetLastError();
}

}  // namespace nvfp4
