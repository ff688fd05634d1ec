// Router of a mixture-of-experts layer for any number of tokens, the sort of rows by group behind it, and the weighted
// sum of what the groups give back (gfx950).
//
// k_mx_route: top-k choices and softmax weights, four rows of logits per wave: a row sits in the registers of 16 lanes as
//   unsigned keys and gives its largest entry k times.
// k_mx_count, k_mx_place: a counting sort of the (row, choice) pairs by group, stable in the pairs' order.  A
//   workgroup has a run of pairs; its counts per group (k_mx_route makes them as it goes, k_mx_count for choices that
//   are given) go to the workspace, and k_mx_place adds up those of the workgroups before its own, so that every pair's
//   place follows from counts alone.  No place comes from an atomic (counts are integer sums), so the order never
//   depends on timing.  Few rows are
//   done by one workgroup in one launch.
// k_mx_combine: y[t] = sum_j w[t][j] z[places[t][j]] in fp32, in the order of j.  Bound by reading z: 4096 x 4096, four rows
// each, bf16 27 us: z's 134 MB at 4.9 TB/s, with y's 34 MB 6.2 TB/s (part of z is in the caches).
// The router is bound by latency: 16 rows 6.8 us, 4096 x 64 6.4 + 7.2 us (two launches), 16384 x 128, top 8 7.8 + 8.1 us.  A row has
// registers for 64, 128, 256 or 512 entries, so just above one of them it costs as much as at the next: 16384 rows, top 8, of 64,
// 65, 128, 129, 256 and 257 entries 12.5, 15.3, 15.8, 20.9, 22.0 and 33.1 us.
// The sort alone, eight choices of 64 groups: 64 rows 4.8 us, 512 9.6 (one workgroup), 513 13.9 (two launches); 2^20 rows of two
// choices, 128 groups 34 us.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.h"
#include "mx.h"
#include "mx_route.h"

namespace nvfp4 {

namespace {

constexpr int kMaxG = MXFP4_MOE_MAX_EXPERTS;
constexpr int kWaves = 16, kThreads = 64 * kWaves;
constexpr int kMaxBlocks = 256;      // runs of pairs
// Rows of logits that one workgroup routes and sorts in one launch, a row per wave: 16 x 64 6.8 us, in two launches 9; 64 x 64
// 13.6 and 9.1.
constexpr int kOneBlockRows = 16;
constexpr int kOneBlockPairs = 4096; // given choices that one workgroup sorts

struct RouteDev {
    const void *logits;
    int64_t ld;
    int64_t T, P;
    int E, k, renorm;
    const int32_t *ids;  // the choices to sort
    int32_t *out_ids;    // k_mx_route: where they are written (= ids)
    float *weights;
    int32_t *offsets, *rows, *places;
    int32_t *hist;  // [blocks][E]
    int blocks;
    bool rest;    // choices outside the groups belong to the last one
    int64_t run;  // pairs per workgroup; whole rows for k_mx_route
};

struct SortShared {
    uint32_t cnt[kWaves][kMaxG];
    uint32_t tot[kThreads], pre[kThreads];
    uint32_t wave_sum[kWaves];
};

// Lanes of the wave whose group is the lane's own (of the lanes with `ok`).
__device__ __forceinline__ uint64_t same_group(int g, bool ok, int bits) {
    uint64_t m = __ballot(ok);
    for (int b = 0; b < bits; b++) {
        const uint64_t set = __ballot(g >> b & 1);
        m &= g >> b & 1 ? set : ~set;
    }
    return m;
}

// Sums over the waves of the counts of each group.
__device__ __forceinline__ uint32_t group_count(const SortShared &s, int e) {
    uint32_t n = 0;
#pragma unroll
    for (int w = 0; w < kWaves; w++) n += s.cnt[w][e];
    return n;
}

// The wave's part of the workgroup's n pairs: whole batches of 64, so that waves hold consecutive runs.
__device__ __forceinline__ void wave_part(int64_t n, int wave, int64_t &lo, int64_t &hi) {
    const int64_t q = ((n + kWaves - 1) / kWaves + 63) / 64 * 64;
    lo = min(n, wave * q);
    hi = min(n, lo + q);
}

// The group of pair i, outside 0 .. E - 1 where it has none.
__device__ __forceinline__ int group_of(const RouteDev &a, int64_t i) {
    const int g = a.ids[i];
    return a.rest && (unsigned)g >= (unsigned)a.E - 1 ? a.E - 1 : g;
}

__device__ __forceinline__ void clear_counts(const RouteDev &a, SortShared &s, int lane, int wave) {
    for (int e = lane; e < a.E; e += 64) s.cnt[wave][e] = 0;  // a wave's own line
    wave_exchange();
}

// The wave's pairs a block of kAhead x 64 at a time, their groups loaded side by side: each(place of the lane's pair, or -1
// behind the last; its group).  (One at a time, the two passes over 4096 pairs in one workgroup waited eight times.)
constexpr int kAhead = 4;
template <class Each>
__device__ __forceinline__ void each_pair(const RouteDev &a, int64_t n0, int64_t n, Each each) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t lo, hi;
    wave_part(n, wave, lo, hi);
    for (int64_t i = lo; i < hi; i += 64 * kAhead) {
        int g[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; q++) g[q] = i + 64 * q + lane < hi ? group_of(a, n0 + i + 64 * q + lane) : -1;
#pragma unroll
        for (int q = 0; q < kAhead; q++)
            if (i + 64 * q < hi) each(i + 64 * q + lane < hi ? n0 + i + 64 * q + lane : -1, g[q]);
    }
}

// Counts per wave and group of the workgroup's pairs n0 .. n0 + n - 1.  Lanes of one group let the first of them add.
__device__ __forceinline__ void count_pairs(const RouteDev &a, SortShared &s, int64_t n0, int64_t n, int bits) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    clear_counts(a, s, lane, wave);
    each_pair(a, n0, n, [&](int64_t, int g) {
        const bool ok = (unsigned)g < (unsigned)a.E;
        const uint64_t m = same_group(g, ok, bits);
        if (ok && lane == __builtin_ctzll(m)) s.cnt[wave][g] += __popcll(m);
        wave_exchange();
    });
    __syncthreads();
}

// Places of the workgroup's pairs, whose counts are in s.cnt; offsets by workgroup 0.
__device__ void place_pairs(const RouteDev &a, SortShared &s, int block, int64_t n0, int64_t n, int bits) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // totals of each group, and of the workgroups before this one: parts of the table's rows per thread
    int width = 64;
    while (width < a.E) width *= 2;
    const int parts = kThreads / width, e = tid & (width - 1), part = tid / width;
    uint32_t total = 0, before = 0;
    if (a.blocks > 1 && e < a.E) {
        // rows part, part + parts, ... of the table, eight loads side by side
        for (int b0 = part; b0 < a.blocks; b0 += 8 * parts) {
            uint32_t v[8];
#pragma unroll
            for (int q = 0; q < 8; q++) {
                const int b = b0 + q * parts;
                v[q] = b < a.blocks ? (uint32_t)a.hist[(int64_t)b * a.E + e] : 0;
            }
#pragma unroll
            for (int q = 0; q < 8; q++) {
                total += v[q];
                before += b0 + q * parts < block ? v[q] : 0;
            }
        }
    } else if (a.blocks == 1 && part == 0 && e < a.E) {
        total = group_count(s, e);
    }
    s.tot[tid] = total;
    s.pre[tid] = before;
    __syncthreads();
    total = before = 0;
    if (tid < a.E) {
        for (int p = 0; p < parts; p++) {
            total += s.tot[p * width + tid];
            before += s.pre[p * width + tid];
        }
    }
    uint32_t upto = total;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t v = __shfl_up(upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 63) s.wave_sum[wave] = upto;
    __syncthreads();
    uint32_t first = upto - total, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
        if (w < wave) first += s.wave_sum[w];
        all += s.wave_sum[w];
    }
    if (tid < a.E) {
        if (block == 0) a.offsets[tid] = (int32_t)first;
        uint32_t run = first + before;
#pragma unroll
        for (int w = 0; w < kWaves; w++) {
            const uint32_t c = s.cnt[w][tid];
            s.cnt[w][tid] = run;
            run += c;
        }
    }
    if (block == 0 && tid == 0) a.offsets[a.E] = (int32_t)all;
    __syncthreads();
    each_pair(a, n0, n, [&](int64_t i, int g) {
        const bool ok = (unsigned)g < (unsigned)a.E;
        const uint64_t m = same_group(g, ok, bits);
        int at = -1;
        const uint32_t base = ok ? s.cnt[wave][g] : 0;
        wave_exchange();  // all lanes of the group have read it
        if (ok && lane == __builtin_ctzll(m)) s.cnt[wave][g] = base + __popcll(m);
        wave_exchange();
        if (ok) {
            at = (int)(base + __popcll(m & ((1ull << lane) - 1)));
            a.rows[at] = a.k == 1 ? (int32_t)i : (int32_t)((uint32_t)i / (uint32_t)a.k);
        }
        if (i >= 0 && a.places) a.places[i] = at;
    });
    // positions behind the last group
    for (int64_t i = all + (int64_t)block * kThreads + tid; i < a.P; i += (int64_t)a.blocks * kThreads) a.rows[i] = -1;
}

__device__ __forceinline__ int group_bits(int E) {
    return 32 - __builtin_clz((unsigned)E);
}

// Four rows of logits per wave, one per row of 16 lanes: lane l of it holds entries c * 16 + l as keys.  Entries past E and
// masked ones are kKeyNegInf.  (A wave per row spends its instructions on one choice at a time: 16384 x 128, top 8, 15 us.)
template <int EC>
struct Keys16 {
    uint32_t k[EC];
};

template <bool BF16, int EC>
__device__ __forceinline__ Keys16<EC> load_keys16(const RouteDev &a, int64_t t, int l) {
    Keys16<EC> r;
#pragma unroll
    for (int c = 0; c < EC; c++) {
        const int j = c * 16 + l;
        const int64_t at = t * a.ld + min(j, a.E - 1);
        float v;
        if constexpr (BF16) v = (float)reinterpret_cast<const __bf16 *>(a.logits)[at];
        else v = reinterpret_cast<const float *>(a.logits)[at];
        r.k[c] = j < a.E ? key_of(v) : kKeyNegInf;
    }
    return r;
}

// Over the 16 lanes of a row, the result in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    v = max(v, dpp_u32<kDppXor1>(v));
    v = max(v, dpp_u32<kDppXor2>(v));
    v = max(v, dpp_u32<kDppHalfMirror>(v));
    return max(v, dpp_u32<kDppMirror>(v));
}
__device__ __forceinline__ uint32_t min16(uint32_t v) {
    v = min(v, dpp_u32<kDppXor1>(v));
    v = min(v, dpp_u32<kDppXor2>(v));
    v = min(v, dpp_u32<kDppHalfMirror>(v));
    return min(v, dpp_u32<kDppMirror>(v));
}
__device__ __forceinline__ float sum16(float v) {
    v += u2f(dpp_u32<kDppXor1>(f2u(v)));
    v += u2f(dpp_u32<kDppXor2>(f2u(v)));
    v += u2f(dpp_u32<kDppHalfMirror>(f2u(v)));
    return v + u2f(dpp_u32<kDppMirror>(f2u(v)));
}

// The rows of a wave: lane j < k of each gets its choice j, the id and weight.  A row with a NaN or +infinity has no choices,
// and NaN for weights.
template <int EC>
__device__ __forceinline__ void route_rows(const RouteDev &a, Keys16<EC> r, int l, int &id, float &w) {
    uint32_t hi = r.k[0], lo = r.k[0];
#pragma unroll
    for (int c = 1; c < EC; c++) {
        hi = max(hi, r.k[c]);
        lo = min(lo, r.k[c]);
    }
    hi = max16(hi);
    // a NaN's key is above +infinity's or below -infinity's
    const bool bad = hi >= kKeyPosInf || min16(lo) < kKeyNegInf;
    const float top = key_to_f32(hi);
    float s = 0.0f;
    if (!a.renorm) {
#pragma unroll
        for (int c = 0; c < EC; c++) s += r.k[c] > kKeyNegInf ? expf(key_to_f32(r.k[c]) - top) : 0.0f;
    }
    id = -1;
    uint32_t mine = kKeyNegInf;
    for (int j = 0; j < a.k; j++) {
        uint32_t m = r.k[0];
#pragma unroll
        for (int c = 1; c < EC; c++) m = max(m, r.k[c]);
        m = max16(m);
        uint32_t at = 0xFFFFFFFFu;  // the lowest entry that holds it
#pragma unroll
        for (int c = EC - 1; c >= 0; c--) at = r.k[c] == m ? (uint32_t)(c * 16) + l : at;
        at = min16(at);
        if (l == j && m > kKeyNegInf) {
            id = (int)at;
            mine = m;
        }
#pragma unroll
        for (int c = 0; c < EC; c++) r.k[c] = at == (uint32_t)(c * 16) + l ? kKeyNegInf : r.k[c];
    }
    const float p = mine > kKeyNegInf ? expf(key_to_f32(mine) - top) : 0.0f;
    const float den = sum16(a.renorm ? p : s);
    w = bad ? __builtin_nanf("") : id >= 0 ? p / den : 0.0f;
    if (bad) id = -1;
}

template <bool BF16, int EC>
__global__ __launch_bounds__(kThreads) void k_mx_route(RouteDev a) {
    __shared__ SortShared s;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane & 15;
    const int64_t n0 = blockIdx.x * a.run, n = min(a.run, a.P - n0);
    clear_counts(a, s, lane, wave);
    // rows of a workgroup are dealt to the waves first
    constexpr int ROWS = 4 * kWaves;
    const int64_t t0 = n0 / a.k, t1 = t0 + n / a.k;
    int64_t t = t0 + (lane >> 4) * kWaves + wave;
    Keys16<EC> next;
    if (t0 + wave < t1) next = load_keys16<BF16, EC>(a, min(t, t1 - 1), l);  // (rows behind the last repeat it)
    for (int64_t f = t0 + wave; f < t1; f += ROWS, t += ROWS) {
        const Keys16<EC> rows = next;
        if (f + ROWS < t1) next = load_keys16<BF16, EC>(a, min(t + ROWS, t1 - 1), l);
        int id;
        float w;
        route_rows<EC>(a, rows, l, id, w);
        if (l < a.k && t < t1) {
            a.out_ids[t * a.k + l] = id;
            a.weights[t * a.k + l] = w;
            if (id >= 0) atomicAdd(&s.cnt[wave][id], 1u);  // rows of a wave may choose the same
        }
    }
    __syncthreads();
    if (a.blocks > 1) {
        if (tid < a.E) a.hist[(int64_t)blockIdx.x * a.E + tid] = (int32_t)group_count(s, tid);
        return;
    }
    const int bits = group_bits(a.E);
    count_pairs(a, s, n0, n, bits);  // again by runs of pairs, the order of their places
    place_pairs(a, s, 0, n0, n, bits);
}

__global__ __launch_bounds__(kThreads) void k_mx_count(RouteDev a) {
    __shared__ SortShared s;
    const int64_t n0 = blockIdx.x * a.run, n = min(a.run, a.P - n0);
    count_pairs(a, s, n0, n, group_bits(a.E));
    if ((int)threadIdx.x < a.E) a.hist[(int64_t)blockIdx.x * a.E + threadIdx.x] = (int32_t)group_count(s, threadIdx.x);
}

__global__ __launch_bounds__(kThreads) void k_mx_place(RouteDev a) {
    __shared__ SortShared s;
    const int64_t n0 = blockIdx.x * a.run, n = min(a.run, a.P - n0);
    const int bits = group_bits(a.E);
    count_pairs(a, s, n0, n, bits);
    place_pairs(a, s, blockIdx.x, n0, n, bits);
}

// 16 bytes of a row of z as fp32 values.
template <class T>
struct Piece;
template <>
struct Piece<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void add(float w, u32x4 r, float *s) {
#pragma unroll
        for (int i = 0; i < 4; i++) s[i] += w * u2f(r[i]);
    }
};
template <>
struct Piece<__bf16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void add(float w, u32x4 r, float *s) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t v = r[i];
            s[2 * i] += w * u2f(v << 16);
            s[2 * i + 1] += w * u2f(v & 0xFFFF0000u);
        }
    }
};

// Rows of y by blockIdx.y and up, a piece of 16 bytes of z per thread.  A last piece that ends behind the row's columns,
// and rows of z (z_wide) or y (y_wide) that are not 16-byte aligned, go element by element.
template <class ZT, class YT>
__global__ __launch_bounds__(256) void k_mx_combine(const ZT *__restrict__ z, int64_t ld_z, int64_t z_rows,
                                                    const int32_t *__restrict__ places, const float *__restrict__ weights,
                                                    int64_t T, int k, int64_t cols, YT *__restrict__ y, int64_t ld_y,
                                                    int z_wide, int y_wide) {
    constexpr int N = Piece<ZT>::N;
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * N;
    if (c >= cols) return;
    const int left = (int)min((int64_t)N, cols - c);
    for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
        float s[N] = {};
        for (int j0 = 0; j0 < k; j0 += 4) {
            u32x4 r[4];
            float w[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                r[j] = u32x4{0, 0, 0, 0};
                w[j] = 0.0f;
                if (j0 + j >= k) continue;
                const int64_t at = places[t * k + j0 + j];
                w[j] = weights[t * k + j0 + j];
                if (at < 0 || at >= z_rows) continue;  // counts as a row of zeros
                const ZT *p = z + at * ld_z + c;
                if (z_wide && left == N) {
                    r[j] = *reinterpret_cast<const u32x4 *>(p);
                } else {
                    ZT v[N] = {};
#pragma unroll
                    for (int i = 0; i < N; i++)
                        if (i < left) v[i] = p[i];
                    r[j] = *reinterpret_cast<const u32x4 *>(v);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; j++) Piece<ZT>::add(w[j], r[j], s);
        }
        YT *dst = y + t * ld_y + c;
        if (y_wide && left == N) {
            constexpr int PER = 16 / sizeof(YT) < N ? 16 / sizeof(YT) : N;
            typedef YT vec __attribute__((ext_vector_type(PER)));
#pragma unroll
            for (int q = 0; q < N / PER; q++) {
                vec o;
#pragma unroll
                for (int i = 0; i < PER; i++) o[i] = (YT)s[q * PER + i];
                *reinterpret_cast<vec *>(dst + q * PER) = o;
            }
        } else {
            for (int i = 0; i < left; i++) dst[i] = (YT)s[i];
        }
    }
}

int64_t runs_of(int64_t n, int64_t least, int64_t &run) {
    run = std::max<int64_t>(least, (n + kMaxBlocks - 1) / kMaxBlocks);
    return (n + run - 1) / run;
}

// Workgroups and pairs per workgroup of a router's call, and of a sort of given choices.
int64_t route_blocks(int64_t tokens, int top_k, int64_t &run) {
    if (tokens <= kOneBlockRows) {
        run = tokens * top_k;
        return 1;
    }
    const int64_t blocks = runs_of(tokens, kWaves, run);
    run *= top_k;
    return blocks;
}

int64_t sort_blocks(int64_t pairs, int64_t &run) { return runs_of(pairs, kOneBlockPairs, run); }

template <bool BF16>
void launch_route_t(const RouteDev &a, hipStream_t stream) {
    const dim3 grid((unsigned)a.blocks), block(kThreads);
    if (a.E <= 64) hipLaunchKernelGGL((k_mx_route<BF16, 4>), grid, block, 0, stream, a);
    else if (a.E <= 128) hipLaunchKernelGGL((k_mx_route<BF16, 8>), grid, block, 0, stream, a);
    else if (a.E <= 256) hipLaunchKernelGGL((k_mx_route<BF16, 16>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((k_mx_route<BF16, 32>), grid, block, 0, stream, a);
}

}  // namespace

size_t mx_route_ws_bytes(int64_t tokens, int64_t top_k, int64_t experts) {
    if (tokens <= 0 || top_k <= 0 || experts <= 0) return 0;
    int64_t run;
    const int64_t blocks = route_blocks(tokens, (int)top_k, run);
    return blocks > 1 ? (size_t)(blocks * experts * 4) : 0;
}

size_t mx_sort_ws_bytes(int64_t pairs, int64_t groups) {
    if (pairs <= 0 || groups <= 0) return 0;
    int64_t run;
    const int64_t blocks = sort_blocks(pairs, run);
    return blocks > 1 ? (size_t)(blocks * groups * 4) : 0;
}

hipError_t launch_mx_route(const MxRouteArgs &p, void *workspace, hipStream_t stream) {
    RouteDev a{};
    a.logits = p.logits;
    a.ld = p.ld_logits;
    a.T = p.tokens;
    a.P = p.tokens * p.top_k;
    a.E = (int)p.experts;
    a.k = p.top_k;
    a.renorm = p.renormalize;
    a.ids = a.out_ids = p.ids;
    a.weights = p.weights;
    a.offsets = p.offsets;
    a.rows = p.rows;
    a.places = p.places;
    a.hist = reinterpret_cast<int32_t *>(workspace);
    a.blocks = (int)route_blocks(p.tokens, p.top_k, a.run);
    if (p.logits_bf16) launch_route_t<true>(a, stream);
    else launch_route_t<false>(a, stream);
    if (a.blocks > 1) hipLaunchKernelGGL(k_mx_place, dim3((unsigned)a.blocks), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_mx_sort(const int32_t *ids, int64_t rows, int per_row, int64_t groups, int32_t *offsets, int32_t *out_rows,
                          int32_t *places, bool rest, void *workspace, hipStream_t stream) {
    RouteDev a{};
    a.rest = rest;
    a.T = rows;
    a.P = rows * per_row;
    a.E = (int)groups;
    a.k = per_row;
    a.ids = ids;
    a.offsets = offsets;
    a.rows = out_rows;
    a.places = places;
    a.hist = reinterpret_cast<int32_t *>(workspace);
    a.blocks = (int)std::max<int64_t>(1, sort_blocks(a.P, a.run));  // without pairs: the offsets
    if (a.blocks > 1) hipLaunchKernelGGL(k_mx_count, dim3((unsigned)a.blocks), dim3(kThreads), 0, stream, a);
    hipLaunchKernelGGL(k_mx_place, dim3((unsigned)a.blocks), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_mx_combine(const void *z, nvfp4_dtype z_dtype, int64_t z_rows, int64_t ld_z, const int32_t *places,
                             const float *weights, int64_t tokens, int top_k, int64_t cols, void *y, nvfp4_dtype y_dtype,
                             int64_t ld_y, hipStream_t stream) {
    const int per = z_dtype == NVFP4_F32 ? 4 : 8, yeb = y_dtype == NVFP4_F32 ? 4 : 2;
    const int y_wide = reinterpret_cast<uintptr_t>(y) % 16 == 0 && ld_y * yeb % 16 == 0;
    const int z_wide = reinterpret_cast<uintptr_t>(z) % 16 == 0 && ld_z * (16 / per) % 16 == 0;
    const dim3 grid((unsigned)((cols + 256 * per - 1) / (256 * per)), (unsigned)std::min<int64_t>(tokens, 65535));
#define MX_COMBINE(ZT, YT)                                                                                                \
    hipLaunchKernelGGL((k_mx_combine<ZT, YT>), grid, dim3(256), 0, stream, reinterpret_cast<const ZT *>(z), ld_z, z_rows, \
                       places, weights, tokens, top_k, cols, reinterpret_cast<YT *>(y), ld_y, z_wide, y_wide)
    if (z_dtype == NVFP4_F32) {
        if (y_dtype == NVFP4_F32) MX_COMBINE(float, float);
        else MX_COMBINE(float, __bf16);
    } else {
        if (y_dtype == NVFP4_F32) MX_COMBINE(__bf16, float);
        else MX_COMBINE(__bf16, __bf16);
    }
#undef MX_COMBINE
    return hipGetLastError();
}

}  // namespace nvfp4
