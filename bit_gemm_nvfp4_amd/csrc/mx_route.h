// A router's row of logits held by one wave: order, largest entries, ranks (gfx950).
#pragma once

#include "common.h"

namespace nvfp4 {

// Order of fp32 values as unsigned keys (-0 counts as +0); NaN lies beyond the infinities.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = f2u(v + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_to_f32(uint32_t k) { return u2f(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
constexpr uint32_t kKeyNegInf = 0x007FFFFFu, kKeyPosInf = 0xFF800000u;

// A row of logits as keys, one wave: lane l holds entries c * 64 + l.  Entries past E and masked ones are
// kKeyNegInf.
template <int EC>
struct RowKeys {
    uint32_t k[EC];
};

template <bool BF16, int EC>
__device__ __forceinline__ RowKeys<EC> load_row_keys(const void *logits, int64_t ld, int E, int64_t t, int lane) {
    RowKeys<EC> r;
#pragma unroll
    for (int c = 0; c < EC; c++) {
        const int j = c * 64 + lane;
        const int64_t at = t * ld + min(j, E - 1);
        float v;
        if constexpr (BF16) v = (float)reinterpret_cast<const __bf16 *>(logits)[at];
        else v = reinterpret_cast<const float *>(logits)[at];
        r.k[c] = j < E ? key_of(v) : kKeyNegInf;
    }
    return r;
}

// Whether a row holds a NaN or +infinity (a NaN's key is above +infinity's or below -infinity's).
template <int EC>
__device__ __forceinline__ bool row_bad(const RowKeys<EC> &r) {
    bool b = false;
#pragma unroll
    for (int c = 0; c < EC; c++) b = b || r.k[c] >= kKeyPosInf || r.k[c] < kKeyNegInf;
    return __ballot(b) != 0;
}

template <int EC>
__device__ __forceinline__ uint32_t row_max(const RowKeys<EC> &r) {
    uint32_t m = r.k[0];
#pragma unroll
    for (int c = 1; c < EC; c++) m = max(m, r.k[c]);
    return wave_max_u32(m);
}

// Entry e of the row.
template <int EC>
__device__ __forceinline__ uint32_t row_at(const RowKeys<EC> &r, int e) {
    uint32_t v = 0;
#pragma unroll
    for (int c = 0; c < EC; c++)
        if (e / 64 == c) v = readlane_u32(r.k[c], e % 64);
    return v;
}

// Takes the largest entry out of the row (ties: the lowest index); its index, or -1 when none is left.
template <int EC>
__device__ __forceinline__ int pop_max(RowKeys<EC> &r, int lane, uint32_t &key) {
    key = row_max(r);
    if (key == kKeyNegInf) return -1;
    int e = -1;
#pragma unroll
    for (int c = 0; c < EC; c++) {
        const uint64_t m = __ballot(r.k[c] == key);
        if (e < 0 && m != 0) {
            const int l = __builtin_ctzll(m);
            e = c * 64 + l;
            if (lane == l) r.k[c] = kKeyNegInf;
        }
    }
    return e;
}

// Number of entries ahead of entry e, whose key is ke.
template <int EC>
__device__ __forceinline__ int rank_of(const RowKeys<EC> &r, int e, uint32_t ke, int lane) {
    int n = 0;
#pragma unroll
    for (int c = 0; c < EC; c++)
        n += __popcll(__ballot(r.k[c] > ke || (r.k[c] == ke && c * 64 + lane < e)));
    return n;
}

}  // namespace nvfp4
