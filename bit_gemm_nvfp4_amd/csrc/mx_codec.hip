// MXFP4 quantize and expand for gfx950.
//
// Quantize: b = max(E - 2, 0) with E the exponent field of the block's largest magnitude, which is
// 2^(floor(log2 amax) - 2) as an E8M0 byte, then code = nearest E2M1 of v 2^(127 - b).  The product with
// a power of two is exact (v 2^(127 - b) lies below 8), so the only rounding is the conversion to
// E2M1.  Nothing outside a block is needed: one pass, one launch.
//
// Bound by HBM: source bytes in, 17/32 byte out per element.  A lane takes 8 elements (16 bytes of a
// 16-bit source), four lanes hold a block and agree on its largest magnitude by two DPP moves; codes
// leave as one dword per lane, consecutive lanes to consecutive addresses.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "mx.h"

namespace nvfp4 {

namespace {

constexpr int kPerLane = 4;  // chunks of 8 elements per lane per pass, all loaded before the first is used

template <int DT>
struct Raw8 {  // 8 source elements as loaded
    u32x4 v[DT == NVFP4_F32 ? 2 : 1];
};

template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const uint8_t *p) {
    Raw8<DT> r;
    if constexpr (DT == NVFP4_F32) {
        r.v[0] = *reinterpret_cast<const u32x4 *>(p);
        r.v[1] = *reinterpret_cast<const u32x4 *>(p + 16);
    } else if constexpr (DT == NVFP4_E4M3) {
        const u32x2 t = *reinterpret_cast<const u32x2 *>(p);
        r.v[0] = u32x4{t[0], t[1], 0, 0};
    } else {
        r.v[0] = *reinterpret_cast<const u32x4 *>(p);
    }
    return r;
}

template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT> &r, float s, float *v) {
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
    if constexpr (DT == NVFP4_E4M3) {
        // one rounding per element, as nvfp4_quantize widens an FP8 source
        const int lo = (int)r.v[0][0], hi = (int)r.v[0][1];
        v[0] = __builtin_amdgcn_cvt_f32_fp8(lo, 0) * s; v[1] = __builtin_amdgcn_cvt_f32_fp8(lo, 1) * s;
        v[2] = __builtin_amdgcn_cvt_f32_fp8(lo, 2) * s; v[3] = __builtin_amdgcn_cvt_f32_fp8(lo, 3) * s;
        v[4] = __builtin_amdgcn_cvt_f32_fp8(hi, 0) * s; v[5] = __builtin_amdgcn_cvt_f32_fp8(hi, 1) * s;
        v[6] = __builtin_amdgcn_cvt_f32_fp8(hi, 2) * s; v[7] = __builtin_amdgcn_cvt_f32_fp8(hi, 3) * s;
    }
}

template <int DT>
__global__ __launch_bounds__(256) void k_mx_quant(const uint8_t *__restrict__ x, int64_t ld_bytes, int contiguous,
                                                  uint64_t nchunks, uint32_t cpr, const float *__restrict__ src_scale,
                                                  uint32_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                  int32_t *__restrict__ flags) {
    constexpr int EB = DT == NVFP4_F32 ? 4 : DT == NVFP4_E4M3 ? 1 : 2;
    const float s = src_scale ? *src_scale : 1.0f;
    const uint64_t stride = (uint64_t)gridDim.x * blockDim.x;
    bool bad = false;
    for (uint64_t i0 = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i0 < nchunks; i0 += kPerLane * stride) {
        Raw8<DT> raw[kPerLane];
#pragma unroll
        for (int j = 0; j < kPerLane; j++) {
            const uint64_t i = i0 + j * stride;
            raw[j] = Raw8<DT>{};
            if (i < nchunks) {
                uint64_t off = i * (8 * EB);
                if (!contiguous) {
                    const uint64_t r = nchunks <= 0xFFFFFFFFull ? (uint32_t)i / cpr : i / cpr;
                    off = r * (uint64_t)ld_bytes + (i - r * cpr) * (8 * EB);
                }
                raw[j] = load8<DT>(x + off);
            }
        }
#pragma unroll
        for (int j = 0; j < kPerLane; j++) {
            const uint64_t i = i0 + j * stride;
            // nchunks is a multiple of 4 (cols % 32 == 0), so the four lanes of a block stay together
            if (i >= nchunks) break;
            float v[8];
            widen8<DT>(raw[j], s, v);
            uint32_t m = 0;
#pragma unroll
            for (int q = 0; q < 8; q++) m = max(m, f2u(v[q]) & 0x7FFFFFFFu);
            m = max(m, dpp_u32<kDppXor1>(m));
            m = max(m, dpp_u32<kDppXor2>(m));
            const uint32_t e = m >> 23;
            uint32_t b = e > 2 ? e - 2 : 0;
            const float inv = u2f((254u - b) << 23);
#pragma unroll
            for (int q = 0; q < 8; q++) v[q] *= inv;
            uint32_t w = fp4_pack8(v);
            if (e == 255) {
                b = 255;
                w = 0;
                bad = true;
            }
            codes[i] = w;
            if ((i & 3) == 0) scales[i >> 2] = (uint8_t)b;
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
    constexpr int EB = DT == NVFP4_F32 ? 4 : DT == NVFP4_E4M3 ? 1 : 2;
    const uint64_t nchunks = (uint64_t)out->rows * (uint64_t)(out->cols / 8);
    hipLaunchKernelGGL(k_mx_quant<DT>, dim3(codec_grid(nchunks)), dim3(256), 0, stream,
                       reinterpret_cast<const uint8_t *>(x), ld_x * EB, ld_x == out->cols || out->rows == 1 ? 1 : 0,
                       nchunks, (uint32_t)(out->cols / 8), src_scale, reinterpret_cast<uint32_t *>(out->codes),
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
