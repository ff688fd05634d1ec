// Mixture-of-experts layer with MXFP4 experts for a few tokens (gfx950), in two kernels:
//   y[t] = sum_e p[t][e] . Wd[e] (silu(Wg[e] x[t]) * (Wu[e] x[t])), e over the top-k of logits[t].
//
// Bound by streaming the chosen experts' weights (17/32 byte per element) once from HBM; everything else
// is small.  Weights go from memory to registers in the matrix instructions' operand layout (MxGroup),
// are expanded exactly to bf16 (half an instruction per element) and multiply up to 16 tokens at a time with
// v_mfma_f32_16x16x32_bf16.  Each wave has the weights of its next groups in flight while it works on one.
// Measured with 64 experts of 4096 x 1536, kernel times and rate of the weights' bytes:
//   1 token, 8 experts each    up 15.5 us (3.5 TB/s), down 11.2 us (2.4 TB/s)
//   33 tokens, 4 experts each  up 92 us (4.2 TB/s), down 66 us (2.9 TB/s)
// with the same weights again and again: the 80 MB of the one token come from the Infinity Cache, the 565 MB of the 33
// do not fit it.  The layer's calls for one token: 26.6 us, over nine sets of weights in turn 28.5 us.
// Figures marked "two planes" below compare forms as they were before h had its third one.
// A copy of 1 GiB moves 5.07 TB/s.  What is lost: about 4 us of each launch pass before its first weights arrive
// and after the last (logits or slot lists, sums over the waves), and k_moe_down deals whole units to the waves
// (6 rounds for 5.3 units a wave with 33 tokens).
//
// Routing needs no kernel of its own: an expert's rank in a row is the number of entries ahead of it
// (larger, or equal with a lower index), so a workgroup of the first kernel finds which tokens chose its
// expert by counting, and one further workgroup per token writes that token's choices and softmax sum.
//   k_moe_up:   workgroup (slot, a run of 16-row tiles of the intermediate size): gate and up products of
//               the slot's expert for the tokens that chose it, h = silu(g) u exp(logit - row max), stored
//               as three bf16 planes that add up to its fp32 value, per (token, choice).  With tokens * top_k <
//               experts a slot is a (token, choice) pair, and a pair whose expert an earlier token chose
//               is left empty; otherwise a slot is an expert.  The first run of a slot lists its tokens.
//   k_moe_down: workgroup (16 rows of Wd): (slot, 512-column group) items dealt to the waves.  h carries the
//               softmax weight, so a wave adds its items into its own [token][16 rows] sums in LDS; these are
//               joined in wave order and divided by the softmax sum.  No sum is made by atomics (one counter
//               per row block says which workgroup joins the parts): the result does not depend on the order
//               of execution.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.h"
#include "mx.h"

namespace nvfp4 {

namespace {

constexpr int kMaxT = MXFP4_MOE_MAX_TOKENS, kMaxE = MXFP4_MOE_MAX_EXPERTS;
constexpr int kUpWaves = 8, kDownWaves = 8;
// k_moe_down's tall form: row tiles per workgroup, and the average tokens per expert from which it is taken.
constexpr int kTallTiles = 4, kTallTokens = 2, kTallRows = 16 * kTallTiles;
constexpr int kPlanes = 3;  // bf16 values that carry the 24 bits of an fp32 one
constexpr int kUpTiles = 4;  // tiles whose sums a wave keeps before the waves join them

struct MoeDev {
    const __bf16 *x;
    const void *logits;
    int64_t ld_x, ld_logits;
    const uint8_t *gu_codes, *gu_scales, *dn_codes, *dn_scales;
    int H, I;
    void *y;
    int64_t ld_y;
    int32_t *ids;    // user's, may be null
    float *weights;  // user's, may be null
    // workspace
    float *den;          // [T] softmax sum; NaN for a row with NaN or +inf
    int32_t *slot_n;     // [slots] tokens of the slot | expert << 16
    uint16_t *slot_tok;  // [slots][T] token | choice << 8
    __bf16 *h;           // [T * k][kPlanes][I]: the planes of a (token, choice)
    float *parts;        // [workgroups of k_moe_down][T][64], with several tokens per expert
    uint32_t *arrived;   // [64-row blocks of H], zeroed by k_moe_up
    int row_blocks;
    int T, E, k, renorm, slots, pair_slots, tiles, tile_run, runs;
};

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
__device__ __forceinline__ RowKeys<EC> load_row(const MoeDev &a, int t, int lane) {
    RowKeys<EC> r;
#pragma unroll
    for (int c = 0; c < EC; c++) {
        const int j = c * 64 + lane;
        const int64_t at = (int64_t)t * a.ld_logits + min(j, a.E - 1);
        float v;
        if constexpr (BF16) v = (float)reinterpret_cast<const __bf16 *>(a.logits)[at];
        else v = reinterpret_cast<const float *>(a.logits)[at];
        r.k[c] = j < a.E ? key_of(v) : kKeyNegInf;
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

// One token's choices, weights and softmax sum (one wave).
template <bool BF16, int EC>
__device__ __forceinline__ void route_token(const MoeDev &a, int t, int lane) {
    RowKeys<EC> r = load_row<BF16, EC>(a, t, lane);
    const bool bad = row_bad(r);
    const uint32_t top = row_max(r);
    const float ftop = key_to_f32(top);
    float s = 0.0f;
    if (!a.renorm) {
#pragma unroll
        for (int c = 0; c < EC; c++) s += r.k[c] > kKeyNegInf ? expf(key_to_f32(r.k[c]) - ftop) : 0.0f;
    }
    int id = -1;     // lane j < k holds choice j
    float p = 0.0f;
    for (int j = 0; j < a.k && !bad; j++) {
        uint32_t key;
        const int e = pop_max(r, lane, key);
        if (e < 0) break;
        if (lane == j) {
            id = e;
            p = expf(key_to_f32(key) - ftop);
        }
    }
    const float den = wave_sum_f32(a.renorm ? p : s);
    if (lane == 0) a.den[t] = bad ? __builtin_nanf("") : top == kKeyNegInf ? 0.0f : den;
    if (lane < a.k) {
        if (a.ids) a.ids[t * a.k + lane] = id;
        if (a.weights) a.weights[t * a.k + lane] = id >= 0 ? p / den : 0.0f;
    }
}

// lane i takes lane (i - N) mod 16 of its row of 16
template <int N>
constexpr int kDppRowRor = 0x120 + N;

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// (13 to 61 scalar values live in lanes of vector registers; nothing goes to memory.)
// XREG: H has no more 512-column groups than there are waves, so that a wave's activations are the same for
// all its tiles and stay in registers.
template <bool LBF16, int EC, bool XREG>
__global__ __launch_bounds__(64 * kUpWaves) void k_moe_up(MoeDev a) {
    __shared__ int sh_tok[kMaxT], sh_rank[kMaxT];
    __shared__ float sh_p[kMaxT];
    __shared__ __align__(16) float red[kUpWaves][kUpTiles][2][256];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if ((int)blockIdx.x < a.T) {
        if (wave == 0) route_token<LBF16, EC>(a, blockIdx.x, lane);
        if (blockIdx.x == 0)
            for (int j = tid; j < a.row_blocks; j += 64 * kUpWaves) a.arrived[j] = 0;
        return;
    }
    const int block = blockIdx.x - a.T;
    const int slot = block / a.runs, run = block % a.runs;
    int e = slot, t0 = 0;
    if (a.pair_slots) {  // the slot's expert: choice slot % k of token slot / k
        t0 = slot / a.k;
        RowKeys<EC> r = load_row<LBF16, EC>(a, t0, lane);
        const bool bad = row_bad(r);
        uint32_t key;
        e = -1;
        for (int j = slot % a.k; j >= 0 && !bad; j--) {
            e = pop_max(r, lane, key);
            if (e < 0) break;
        }
        if (e < 0) {
            if (run == 0 && tid == 0) a.slot_n[slot] = 0;
            return;
        }
    }
    e = __builtin_amdgcn_readfirstlane(e);

    const int r = lane & 15, lg = lane >> 4;
    const int kb = a.H / kMxBlock, full = a.H / kGroup, tail = kb - full * kGroupBlocks;
    const int groups = full + (tail > 0 ? 1 : 0);
    const int tile0 = run * a.tile_run, ntile = min(a.tile_run, a.tiles - tile0);
    struct Pair {
        MxGroup t[2];  // a tile of gate rows and one of up rows
    };
    // the wave's items: groups wave, wave + kUpWaves, ... of tile 0, 1, ...
    const int gw = wave < groups ? (groups - wave + kUpWaves - 1) / kUpWaves : 0, items = ntile * gw;
    // An item's codes are read through buffers of its sixteen gate and its sixteen up rows, so that blocks past a
    // row's end and items past the last one load nothing, without a branch.
    struct Item {
        __amdgpu_buffer_rsrc_t rsrc[2];
        int soff, left;  // of the group: byte offset, and the blocks from its start to the row's end
    };
    const int row_bytes = a.H / 2;
    const uint32_t voff = (uint32_t)(r * row_bytes + lg * 16);
    auto item_row = [&](int it) -> int64_t { return (int64_t)e * 2 * a.I + (tile0 + (XREG ? it : it / gw)) * 16; };
    auto item_group = [&](int it) -> int { return XREG ? wave : wave + it % gw * kUpWaves; };
    auto item_of = [&](int it) -> Item {
        if (it >= items) return Item{{uniform_rsrc(a.gu_codes, 0), uniform_rsrc(a.gu_codes, 0)}, 0, 0};
        const uint8_t *gc = a.gu_codes + item_row(it) * row_bytes;
        const int g = item_group(it);
        return Item{{uniform_rsrc(gc, 16 * row_bytes), uniform_rsrc(gc + (int64_t)a.I * row_bytes, 16 * row_bytes)},
                    g * (kGroup / 2), kb - g * kGroupBlocks};
    };
    auto load_scales = [&](int it, Pair &w) {
        if (it >= items) return;
        const int g = item_group(it);
        const uint8_t *gs = a.gu_scales + (item_row(it) + r) * kb, *us = gs + (int64_t)a.I * kb;
        if (g < full) {
            w.t[0].s = *reinterpret_cast<const u32x4_u *>(gs + g * kGroupBlocks);
            w.t[1].s = *reinterpret_cast<const u32x4_u *>(us + g * kGroupBlocks);
        } else {
            w.t[0].s = load_mx_tail_scales(gs, g, tail);
            w.t[1].s = load_mx_tail_scales(us, g, tail);
        }
    };
    auto load_chunk = [&](const Item &m, int i, Pair &w) {
        const uint32_t o = i * 4 + lg < m.left ? voff + i * 64 : kOffsetPastRange;
#pragma unroll
        for (int j = 0; j < 2; j++)
            w.t[j].c[i] = __builtin_amdgcn_raw_buffer_load_b128(m.rsrc[j], (int)o, m.soff, 0);
    };
    auto load_w = [&](int it, Pair &w) {
        const Item m = item_of(it);
#pragma unroll
        for (int i = 0; i < kGroupChunks; i++) load_chunk(m, i, w);
        load_scales(it, w);
    };
    // two items in flight while the tokens are looked up
    Pair w[2] = {};
    load_w(0, w[0]);
    load_w(1, w[1]);

    // the tokens that chose e
    for (int t = wave; t < a.T; t += kUpWaves) {
        const RowKeys<EC> row = load_row<LBF16, EC>(a, t, lane);
        const uint32_t ke = row_at(row, e);
        const int n = rank_of(row, e, ke, lane);
        const float top = key_to_f32(row_max(row));
        if (lane == 0) {
            sh_rank[t] = row_bad(row) || ke == kKeyNegInf || n >= a.k ? -1 : n;
            sh_p[t] = expf(key_to_f32(ke) - top);
        }
    }
    __syncthreads();
    const bool in = lane < a.T && sh_rank[lane] >= 0;  // every wave, the same
    const uint64_t chosen = __ballot(in);
    const int n = __popcll(chosen);
    const bool leader = n > 0 && (!a.pair_slots || __builtin_ctzll(chosen) == t0);
    const int at = __popcll(chosen & ((1ull << lane) - 1));
    if (run == 0 && wave == 0) {
        if (lane == 0) a.slot_n[slot] = leader ? n | e << 16 : 0;
        if (leader && in) a.slot_tok[slot * a.T + at] = (uint16_t)(lane | sh_rank[lane] << 8);
    }
    if (!leader) return;
    if (in && wave == 0) sh_tok[at] = lane;
    __syncthreads();

    // Sixteen tokens at a time; more read the weights again, which are in the caches then.
    for (int q = 0; q < n; q += 16) {
        const int cols = min(16, n - q);
        // columns past the last token repeat the first; their results are not stored
        const __bf16 *xr = a.x + (int64_t)sh_tok[q + (r < cols ? r : 0)] * a.ld_x;
        auto load_x = [&](int g) { return g < full ? load_bf16_group<false>(xr, g, lg) : load_bf16_group<true>(xr, g, lg, tail); };
        Bf16Group x;
        if (XREG && gw > 0) x = load_x(wave);
        if (q > 0) {
            load_w(0, w[0]);
            load_w(1, w[1]);
        }
        // One item: its products, each chunk's registers taking the chunk of the item after next as they get free
        // (with a third set of registers for it the kernel spilled: 1 token 28.7 -> 27.0 us for the layer, 33
        // tokens 152 -> 149 us).
        auto step = [&](Pair &p, int it, f32x4(&acc)[2]) {
            if constexpr (!XREG) x = load_x(item_group(it));
            const u32x4 s0 = p.t[0].s, s1 = p.t[1].s;
            const Item m = item_of(it + 2);
            load_scales(it + 2, p);
#pragma unroll
            for (int i = 0; i < kGroupChunks; i++) {
                chunk_product<2>(p.t, {s0[i], s1[i]}, x, i, lg, acc);
                __builtin_amdgcn_sched_barrier(0);
                load_chunk(m, i, p);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        int it = 0;
        for (int c0 = 0; c0 < ntile; c0 += kUpTiles) {
            f32x4 acc[kUpTiles][2] = {};
#pragma unroll
            for (int t = 0; t < kUpTiles; t++) {
                if (c0 + t >= ntile) break;
                if constexpr (XREG) {
                    static_assert(kUpTiles % 2 == 0, "item it is in w[it % 2]");
                    if (gw > 0) step(w[t % 2], it++, acc[t]);
                } else {
                    for (int j = 0; j < gw; j++, it++) {
                        step(w[0], it, acc[t]);
                        const Pair next = w[1];
                        w[1] = w[0];
                        w[0] = next;
                    }
                }
            }
            if (c0 > 0 || q > 0) __syncthreads();  // the previous sums have been read
#pragma unroll
            for (int t = 0; t < kUpTiles; t++)
#pragma unroll
                for (int i = 0; i < 2; i++) *reinterpret_cast<f32x4 *>(&red[wave][t][i][lane * 4]) = acc[t][i];
            __syncthreads();
            // element (row il of a tile, column j) sits in lane j + 16 (il / 4), register il % 4
            const int rows = min(kUpTiles, ntile - c0) * 16;
            for (int o = tid; o < cols * rows; o += 64 * kUpWaves) {
                const int ir = o % rows, j = o / rows, il = ir % 16;
                const int src = (j + 16 * (il / 4)) * 4 + il % 4;
                float gs = 0.0f, us = 0.0f;
#pragma unroll
                for (int v = 0; v < kUpWaves; v++) {
                    gs += red[v][ir / 16][0][src];
                    us += red[v][ir / 16][1][src];
                }
                const int t = sh_tok[q + j];
                const float h = silu(gs) * us * sh_p[t];
                // Three planes of eight bits each, cut off, so that none rounds beyond bf16's range and their sum is
                // h itself (to 2^-133 where its last bits lie below that); an infinity or NaN has no rest.
                const bool finite = (f2u(h) & 0x7F800000u) != 0x7F800000u;
                const float hi = u2f(f2u(h) & 0xFFFF0000u), rest = finite ? h - hi : 0.0f;
                const float mid = u2f(f2u(rest) & 0xFFFF0000u);
                __bf16 *dst = a.h + (int64_t)(t * a.k + sh_rank[t]) * kPlanes * a.I + (tile0 + c0) * 16 + ir;
                dst[0] = (__bf16)(finite ? hi : h);
                dst[a.I] = (__bf16)mid;
                dst[2 * a.I] = (__bf16)(rest - mid);
            }
        }
    }
}

// Five tokens at a time: columns 0-4 of the matrix instruction take the high planes of their h, columns 5-9 and 10-14
// the others, and the three parts of the result are added (column 15 repeats a value that is not used).  A unit of work
// is five tokens of a slot and a 512-column group; units are dealt to the waves in turn.
constexpr int kDownTokens = 16 / kPlanes;
constexpr int kDownEntries = kMaxE + kMaxT * MXFP4_MOE_MAX_TOP_K / kDownTokens;

// RT: tiles of 16 rows that share a unit's activations.  RT = 1: one workgroup has all the units of its rows.
// RT = 4, for several tokens per expert: the h of all tokens passes through every workgroup, so fewer, taller
// ones read less of it (64 tokens, 8 of 64 experts, 4096 x 1536, with two planes: 131 us with RT = 1); RT workgroups then share
// the units of 64 rows, each leaves its sums in the workspace, and the one that finishes last adds them in
// order.  The tall form needs eight registers more than there are and keeps them in memory, 28 bytes a lane: 3 of the 5.3
// MiB that a launch for 33 tokens writes.
template <class OT, int RT>
__global__ __launch_bounds__(64 * kDownWaves) void k_moe_down(MoeDev a) {
    extern __shared__ __align__(16) float sums[];  // [waves][T][16 RT]
    __shared__ uint32_t sh_entry[kDownEntries];    // slot | pass over the tokens << 9 | tokens of the slot << 16
    __shared__ int sh_expert[kMaxE], sh_cnt[kDownWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    static_assert(kMaxE <= 64 * kDownWaves && kMaxE <= 512, "one thread per slot, nine bits");
    // entries in the order of the slots: the passes of the slots before give each its place
    const int info = tid < a.slots ? a.slot_n[tid] : 0;
    const int n_slot = info & 0xFFFF, passes = (n_slot + kDownTokens - 1) / kDownTokens;
    int upto = passes;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 63) sh_cnt[wave] = upto;
    float *mine = sums + wave * a.T * 16 * RT;
    for (int j = lane; j < a.T * 16 * RT; j += 64) mine[j] = 0.0f;
    __syncthreads();
    int at = upto - passes, entries = 0;
#pragma unroll
    for (int v = 0; v < kDownWaves; v++) {
        if (v < wave) at += sh_cnt[v];
        entries += sh_cnt[v];
    }
    if (tid < a.slots) sh_expert[tid] = info >> 16;
    for (int q = 0; q < passes; q++) sh_entry[at + q] = (uint32_t)(tid | q << 9 | n_slot << 16);
    __syncthreads();
    entries = __builtin_amdgcn_readfirstlane(entries);

    const int r = lane & 15, lg = lane >> 4, plane = min(r / kDownTokens, kPlanes - 1);
    const int kb = a.I / kMxBlock, full = a.I / kGroup, tail = kb - full * kGroupBlocks;
    const int groups = full + (tail > 0 ? 1 : 0), units = entries * groups;
    const int part = blockIdx.x % RT, n0 = blockIdx.x / RT * (16 * RT);
    struct Tile {
        MxGroup t[RT];
    };
    auto load_w = [&](int u) -> Tile {
        const int g = u % groups;
        const int64_t row0 = (int64_t)sh_expert[sh_entry[u / groups] & 511] * a.H;
        Tile w;
#pragma unroll
        for (int t = 0; t < RT; t++) {
            // H is a multiple of 32: rows past it repeat the last one, and are not stored
            const int64_t row = row0 + (RT == 1 ? n0 + r : min(n0 + 16 * t + r, a.H - 1));
            const uint8_t *c = a.dn_codes + row * (a.I / 2), *s = a.dn_scales + row * kb;
            w.t[t] = g < full ? load_mx_group(c, s, g, lg) : load_mx_tail(c, s, g, lg, tail);
        }
        return w;
    };
    // the lane's token | choice << 8; columns past the last token repeat the first (not used in the end)
    auto load_tok = [&](int u) -> int {
        const uint32_t en = sh_entry[u / groups];
        const int j = (en >> 9 & 127) * kDownTokens + r % kDownTokens, n = en >> 16;
        return a.slot_tok[(en & 511) * a.T + (j < n ? j : 0)] | (j < n ? 0 : 1 << 16);
    };
    auto load_h = [&](int u, int tok) -> Bf16Group {
        const int g = u % groups;
        const __bf16 *row = a.h + ((int64_t)((tok & 255) * a.k + (tok >> 8 & 255)) * kPlanes + plane) * a.I;
        if (g < full) return load_bf16_group<false>(row, g, lg);
        return load_bf16_group<true>(row, g, lg, tail);
    };
    auto product = [&](const Tile &w, const Bf16Group &h, int tok) {
        f32x4 acc[RT] = {};
        group_product<RT>(w.t, h, lg, acc);
#pragma unroll
        for (int t = 0; t < RT; t++) {
            // columns c, c + 5 and c + 10 of a row of 16 lanes, the smallest first
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float v = acc[t][i];
                acc[t][i] = v + (u2f(dpp_u32<kDppRowRor<16 - kDownTokens>>(f2u(v))) +
                                 u2f(dpp_u32<kDppRowRor<16 - 2 * kDownTokens>>(f2u(v))));
            }
            if (r < kDownTokens && tok >> 16 == 0) {
                f32x4 *dst = reinterpret_cast<f32x4 *>(&mine[(tok & 255) * (16 * RT) + t * 16 + lg * 4]);
                f32x4 s = *dst;
                s += acc[t];
                *dst = s;
            }
        }
    };
    constexpr int STEP = kDownWaves * RT;
    const int u0 = part * kDownWaves + wave;
    if constexpr (RT == 1) {
        // Loads return in order, so they are issued in the order of use: behind a unit's product come the
        // activations of the next unit, the token of the one after and its weights.
        if (u0 < units) {
            const int u1 = min(u0 + STEP, units - 1);
            int tok = load_tok(u0), tok1 = load_tok(u1);
            Tile w = load_w(u0), w1 = load_w(u1);
            Bf16Group h = load_h(u0, tok);
            int u = u0;
            for (; u + 2 * STEP < units; u += STEP) {
                const Bf16Group h1 = load_h(u + STEP, tok1);
                const int tok2 = load_tok(u + 2 * STEP);
                __builtin_amdgcn_sched_barrier(0);
                const Tile w2 = load_w(u + 2 * STEP);
                __builtin_amdgcn_sched_barrier(0);
                product(w, h, tok);
                tok = tok1;
                tok1 = tok2;
                w = w1;
                w1 = w2;
                h = h1;
            }
            if (u + STEP < units) {
                const Bf16Group h1 = load_h(u + STEP, tok1);
                __builtin_amdgcn_sched_barrier(0);
                product(w, h, tok);
                tok = tok1;
                w = w1;
                h = h1;
            }
            product(w, h, tok);
        }
    } else if (u0 < units) {
        // A unit's four tiles are enough to have one unit in flight ahead.  Refilling a chunk's registers as its
        // products are done, as k_moe_up does, was no faster here (with two planes): 33 tokens 148 -> 151 us, 1 token
        // 27.0 -> 27.9 us.
        int tok = load_tok(u0);
        Tile w = load_w(u0);
        int u = u0;
        for (; u + STEP < units; u += STEP) {
            const Bf16Group h = load_h(u, tok);
            const int tok1 = load_tok(u + STEP);
            __builtin_amdgcn_sched_barrier(0);
            const Tile w1 = load_w(u + STEP);
            __builtin_amdgcn_sched_barrier(0);
            product(w, h, tok);
            tok = tok1;
            w = w1;
        }
        product(w, load_h(u, tok), tok);
    }
    __syncthreads();
    OT *y = reinterpret_cast<OT *>(a.y);
    const int cells = a.T * 16 * RT;
    // no expert: 0; a row with NaN or +inf has den = NaN
    auto store_y = [&](int t, int n, float s) {
        const float den = a.den[t];
        y[(int64_t)t * a.ld_y + n] = (OT)(den == 0.0f ? 0.0f : s / den);
    };
    auto joined = [&](int o) {
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < kDownWaves; v++) s += sums[v * cells + o];
        return s;
    };
    if constexpr (RT == 1) {
        for (int o = tid; o < cells; o += 64 * kDownWaves) store_y(o / 16, n0 + o % 16, joined(o));
    } else {
        // Sums of the parts: written and read past the caches that are not shared between XCDs (relaxed
        // atomics of agent scope).  Every wave waits for its stores before the workgroup counts itself in, so
        // whoever counts RT - 1 before it finds all of them.
        float *mine_p = a.parts + (int64_t)blockIdx.x * cells;
        for (int o = tid; o < cells; o += 64 * kDownWaves)
            __hip_atomic_store(mine_p + o, joined(o), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
        __syncthreads();
        if (tid == 0)
            sh_cnt[0] = (int)__hip_atomic_fetch_add(a.arrived + blockIdx.x / RT, 1u, __ATOMIC_RELAXED,
                                                    __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (sh_cnt[0] != RT - 1) return;
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
        const float *p = a.parts + (int64_t)(blockIdx.x - part) * cells;
        for (int o = tid; o < cells; o += 64 * kDownWaves) {
            const int t = o / (16 * RT), n = n0 + o % (16 * RT);
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < RT; v++)
                s += __hip_atomic_load(p + (int64_t)v * cells + o, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (n < a.H) store_y(t, n, s);
        }
    }
}

size_t align256(size_t b) { return (b + 255) / 256 * 256; }

template <bool LBF16, bool XREG>
void launch_up_x(const MoeDev &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.T + a.slots * a.runs)), block(64 * kUpWaves);
    if (a.E <= 64) hipLaunchKernelGGL((k_moe_up<LBF16, 1, XREG>), grid, block, 0, stream, a);
    else if (a.E <= 128) hipLaunchKernelGGL((k_moe_up<LBF16, 2, XREG>), grid, block, 0, stream, a);
    else if (a.E <= 256) hipLaunchKernelGGL((k_moe_up<LBF16, 4, XREG>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((k_moe_up<LBF16, 8, XREG>), grid, block, 0, stream, a);
}

template <bool LBF16>
void launch_up(const MoeDev &a, hipStream_t stream) {
    if (a.H <= kUpWaves * kGroup) launch_up_x<LBF16, true>(a, stream);
    else launch_up_x<LBF16, false>(a, stream);
}

template <class OT, int RT>
void launch_down(const MoeDev &a, int grid, hipStream_t stream) {
    const size_t lds = (size_t)kDownWaves * a.T * 16 * RT * 4;  // at most 128 KiB
    hipLaunchKernelGGL((k_moe_down<OT, RT>), dim3((unsigned)grid), dim3(64 * kDownWaves), lds, stream, a);
}

}  // namespace

// Sized from the number of (token, choice) pairs, which bounds the tokens.
size_t mx_moe_ws_bytes(int64_t pairs, int64_t hidden, int64_t inter) {
    if (pairs <= 0 || hidden <= 0 || inter <= 0) return 0;
    const size_t tokens = (size_t)std::min<int64_t>(pairs, kMaxT), blocks = (size_t)(hidden + kTallRows - 1) / kTallRows;
    return align256(kMaxT * 4) + align256(kMaxE * 4) + align256(kMaxE * tokens * 2) +
           align256((size_t)pairs * inter * kPlanes * 2) + align256(blocks * 4) + blocks * kTallTiles * tokens * kTallRows * 4;
}

hipError_t launch_mx_moe(const MoeArgs &p, void *workspace, int num_cus, hipStream_t stream) {
    MoeDev a{};
    a.x = reinterpret_cast<const __bf16 *>(p.x);
    a.logits = p.logits;
    a.ld_x = p.ld_x;
    a.ld_logits = p.ld_logits;
    a.gu_codes = p.w_gate_up->codes;
    a.gu_scales = p.w_gate_up->scales;
    a.dn_codes = p.w_down->codes;
    a.dn_scales = p.w_down->scales;
    a.H = (int)p.w_gate_up->cols;
    a.I = (int)p.w_down->cols;
    a.y = p.y;
    a.ld_y = p.ld_y;
    a.ids = p.ids;
    a.weights = p.weights;
    a.T = (int)p.tokens;
    a.E = (int)p.experts;
    a.k = p.top_k;
    a.renorm = p.renormalize;
    uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
    a.den = reinterpret_cast<float *>(ws);
    ws += align256(kMaxT * 4);
    a.slot_n = reinterpret_cast<int32_t *>(ws);
    ws += align256(kMaxE * 4);
    a.slot_tok = reinterpret_cast<uint16_t *>(ws);
    ws += align256((size_t)kMaxE * a.T * 2);
    a.h = reinterpret_cast<__bf16 *>(ws);
    ws += align256((size_t)a.T * a.k * a.I * kPlanes * 2);
    const int blocks = (a.H + kTallRows - 1) / kTallRows;
    a.arrived = reinterpret_cast<uint32_t *>(ws);
    a.parts = reinterpret_cast<float *>(ws + align256((size_t)blocks * 4));
    a.pair_slots = a.T * a.k < a.E ? 1 : 0;
    a.slots = a.pair_slots ? a.T * a.k : a.E;
    a.tiles = a.I / 16;
    // Tiles per workgroup: an even share of one round over the device, at most 12.  Starting a workgroup costs about
    // as much as one tile, and long runs leave CUs without work in the last round.  Layers of 4096 x 1536, runs of 8,
    // 12, 16 tiles at most, with two planes: 4 tokens, 8 of 64 experts 82.8, 72.0, 72 us; 8 tokens 130, 128, 143 us; 33
    // tokens, 4 of 64 157, 152, 165 us; 64 tokens, 8 of 64 202, 207, 195 us.  Measured at H = 4096 only, which is also where
    // the eight waves have a 512-column group each; with smaller H fewer of them work.
    a.tile_run = (int)std::min<int64_t>(12, std::max<int64_t>(1, ((int64_t)a.slots * a.tiles + num_cus - 1) / num_cus));
    a.runs = (a.tiles + a.tile_run - 1) / a.tile_run;
    const bool tall = a.T * a.k >= kTallTokens * a.E;
    a.row_blocks = tall ? blocks : 0;
    if (p.logits_bf16) launch_up<true>(a, stream);
    else launch_up<false>(a, stream);
    if (tall) {
        if (p.y_bf16) launch_down<__bf16, kTallTiles>(a, blocks * kTallTiles, stream);
        else launch_down<float, kTallTiles>(a, blocks * kTallTiles, stream);
    } else {
        if (p.y_bf16) launch_down<__bf16, 1>(a, a.H / 16, stream);
        else launch_down<float, 1>(a, a.H / 16, stream);
    }
    return hipGetLastError();
}

}  // namespace nvfp4
