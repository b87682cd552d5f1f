// rope.cuh -- rotary positions of q and k, alone (forward, and with the angle's
// sign turned its backward) and on the way into the paged cache.
//
// Pair i of a head's rot_dim leading columns turns by the angle of its token's
// position: y1 = x1 c - x2 s, y2 = x2 c + x1 s, with c = table[p][i],
// s = table[p][rot_dim / 2 + i] and p the token's position on the pair's axis
// (one axis, or up to four: time, height, width of image and video tokens).
// A pair is the columns (i, i + rot_dim / 2), or (2 i, 2 i + 1) interleaved;
// rotary, partial and interleaved, stands among the options of "[CUDA]
// PagedAttention: add SM<80 fp16 fallback via memory-efficient attention".
// Each product and sum is rounded to fp32 by itself (no contraction), and the
// result once to bf16, so the value does not depend on which kernel computes it.
//
// HBM bound: 2 bytes read and 2 written for 6 flops a pair.  A head is D / 16
// units of two 16-byte pieces (the two halves of 8 pairs, or 8 interleaved
// pairs); a lane keeps one unit of every head its warp takes, so that the
// cosines and sines are loaded once for a token and stay in registers.  The rows
// are loaded before the positions are looked up, heads of one type after another
// (a loop over all heads with a choice of tensor in it took 127 us where this
// takes 107).
//
// Measured: 33700 tokens of 32 + 8 heads of 128, 107 us, 6.6 TB/s, the rate of a
// copy.  11103 tokens of 16 + 16 heads of 64 with three axes, 21 us, 4.3 TB/s: a
// warp lives for its three dependent look-ups (position, row of the table, the
// heads behind them), and four rounds of warps fill the call.  128 threads a
// block: with 64 the same, with 256 2 us more on both.
// One token: 6 us, a launch.
#pragma once

#include "ptx.cuh"
#include "prefill.cuh"   // kPageRows

namespace attn {

constexpr int kRopeThreads = 128;
constexpr int kRopeMaxAxes = 4;
// kErrRope*: a position outside the table, an axis outside the given ones.
// kErrAppend* as in append.cuh.
enum : int { kErrRopePosition = 521, kErrRopeAxis = 522 };
enum : int { kCacheBf16 = 0, kCacheE4m3 = 1, kCacheQ4 = 2 };

struct RopeTable {
    const float* table;      // [max_pos][rot]: cosines, then sines; null: no rotation
    int max_pos, rot;
    const int* positions;    // [axes][total]; null (append only): the cache position
    int axes;
    const int* pair_axis;    // [rot / 2], or null: axis 0
    int interleaved;
    float sign;              // -1: the inverse rotation (the gradient)
};

// Cosines, sines and minus sines of the pairs 2 i and 2 i + 1 of eight, for packed arithmetic.
struct RopeAngles {
    float2 c[4], s[4], n[4];
};

// The eight pairs 8 u .. 8 u + 7 of token t.
__device__ __forceinline__ RopeAngles rope_angles(const RopeTable& r, long long t, long long total, int u, int seq_pos) {
    const int half = r.rot / 2;
    // the token's position on every axis, and the axes of the eight pairs (all loads first)
    int p[kRopeMaxAxes], ax[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int a = 0; a < kRopeMaxAxes; ++a) p[a] = a < r.axes ? r.positions ? __ldg(r.positions + a * total + t) : seq_pos : 0;
    if (r.pair_axis) {
        const int4 a0 = __ldg(reinterpret_cast<const int4*>(r.pair_axis + 8 * u));
        const int4 a1 = __ldg(reinterpret_cast<const int4*>(r.pair_axis + 8 * u + 4));
        ax[0] = a0.x, ax[1] = a0.y, ax[2] = a0.z, ax[3] = a0.w, ax[4] = a1.x, ax[5] = a1.y, ax[6] = a1.z, ax[7] = a1.w;
    }
#pragma unroll
    for (int a = 0; a < kRopeMaxAxes; ++a)
        if (p[a] < 0 || p[a] >= r.max_pos) {
            record_data_error(kErrRopePosition);       // reported, the nearest row used
            p[a] = min(max(p[a], 0), r.max_pos - 1);
        }
    bool one = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (ax[i] < 0 || ax[i] >= r.axes) {
            record_data_error(kErrRopeAxis);
            ax[i] = 0;
        }
        one = one && ax[i] == ax[0];
    }
    auto place = [&](int a) { return a == 0 ? p[0] : a == 1 ? p[1] : a == 2 ? p[2] : p[3]; };
    RopeAngles g;
    if (one) {
        const float* row = r.table + (long long)place(ax[0]) * r.rot + 8 * u;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const float4 cv = __ldg(reinterpret_cast<const float4*>(row + 2 * i));
            const float4 sv = __ldg(reinterpret_cast<const float4*>(row + half + 2 * i));
            g.c[i] = make_float2(cv.x, cv.y), g.c[i + 1] = make_float2(cv.z, cv.w);
            g.s[i] = make_float2(sv.x, sv.y), g.s[i + 1] = make_float2(sv.z, sv.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* r0 = r.table + (long long)place(ax[2 * i]) * r.rot + 8 * u + 2 * i;
            const float* r1 = r.table + (long long)place(ax[2 * i + 1]) * r.rot + 8 * u + 2 * i + 1;
            g.c[i] = make_float2(__ldg(r0), __ldg(r1));
            g.s[i] = make_float2(__ldg(r0 + half), __ldg(r1 + half));
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        g.s[i] = make_float2(g.s[i].x * r.sign, g.s[i].y * r.sign);
        g.n[i] = make_float2(-g.s[i].x, -g.s[i].y);
    }
    return g;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float2 bf16_pair(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

// Turns two pairs (x1, x2) by the angles 2 i and 2 i + 1: packed, every operation rounded by itself.
__device__ __forceinline__ void rope_turn(float2& x1, float2& x2, const RopeAngles& g, int i) {
    const float2 y1 = fadd2(fmul2(x1, g.c[i]), fmul2(x2, g.n[i]));
    x2 = fadd2(fmul2(x2, g.c[i]), fmul2(x1, g.s[i]));
    x1 = y1;
}

// Turns a unit: pieces a and b hold the first and second columns of the eight
// pairs, or eight interleaved pairs in order.
__device__ __forceinline__ void rope_unit(uint4& a, uint4& b, const RopeAngles& g, bool interleaved) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (interleaved) {
            float2 x1 = make_float2(bf16_lo(w[2 * i]), bf16_lo(w[2 * i + 1]));
            float2 x2 = make_float2(bf16_hi(w[2 * i]), bf16_hi(w[2 * i + 1]));
            rope_turn(x1, x2, g, i);
            w[2 * i] = pack_bf16(x1.x, x2.x);
            w[2 * i + 1] = pack_bf16(x1.y, x2.y);
        } else {
            float2 x1 = bf16_pair(w[i]), x2 = bf16_pair(w[4 + i]);
            rope_turn(x1, x2, g, i);
            w[i] = pack_bf16(x1.x, x1.y);
            w[4 + i] = pack_bf16(x2.x, x2.y);
        }
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
}

// Columns of unit u's two pieces.  Units past rot / 16 hold the columns that do
// not turn.
__device__ __forceinline__ void rope_columns(const RopeTable& r, int u, int* ca, int* cb) {
    const int nrot = r.table ? r.rot / 16 : 0;
    if (u < nrot && !r.interleaved) {
        *ca = 8 * u;
        *cb = r.rot / 2 + 8 * u;
    } else {
        *ca = 16 * u;
        *cb = 16 * u + 8;
    }
}

struct HeadRows {            // [token][head][D] with element strides
    const __nv_bfloat16* p;
    long long row, head;
};

// Eight bf16 values times `inv`, as e4m3 (nearest even, saturating at +-448).
__device__ __forceinline__ uint2 bf16x8_to_e4m3(uint4 x, float inv) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 lo = fmul2(bf16_pair(w[2 * i]), make_float2(inv, inv));
        const float2 hi = fmul2(bf16_pair(w[2 * i + 1]), make_float2(inv, inv));
        o[i] = pack_e4m3x4(lo.x, lo.y, hi.x, hi.y);
    }
    return make_uint2(o[0], o[1]);
}

// One token's rows of H heads (q, k or v) on their way: a warp takes every parts-th group of
// HP heads, a lane its unit (pieces at columns ca and cb) of each.  N groups' loads are in
// flight together; start() issues the first ones, before the caller looks the token up.
template <int D, int N>
struct RopeRows {
    static constexpr int U = D / 16, HP = 32 / U;
    const __nv_bfloat16* src;            // this lane's first group, piece a
    long long pitch;                     // elements to its next group
    int left, apart;                     // heads from its first one on, heads between its groups
    int cb_ca;                           // piece b behind piece a
    uint4 xa[N], xb[N];

    __device__ __forceinline__ void load() {
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (n * apart < left) {
                xa[n] = *reinterpret_cast<const uint4*>(src + n * pitch);
                xb[n] = *reinterpret_cast<const uint4*>(src + n * pitch + cb_ca);
            }
    }
    __device__ __forceinline__ void start(const HeadRows& x, long long t, int H, int first, int parts, int ca, int cb) {
        src = x.p + t * x.row + first * x.head + ca;
        pitch = parts * HP * x.head;
        left = H - first;
        apart = parts * HP;
        cb_ca = cb - ca;
        load();
    }
    // Writes them to dst (this lane's first group, piece a; `step` bytes to its next one) as bf16, or
    // as e4m3 times inv; turned where `turns`.
    template <int CACHE>
    __device__ __forceinline__ void finish(uint8_t* dst, long long step, bool turns, const RopeAngles& g, bool interleaved,
                                           float inv) {
        constexpr int E = CACHE == kCacheE4m3 ? 1 : 2;
        while (left > 0) {
#pragma unroll
            for (int n = 0; n < N; ++n)
                if (n * apart < left) {
                    if (turns) rope_unit(xa[n], xb[n], g, interleaved);
                    uint8_t* to = dst + n * step;
                    if (CACHE == kCacheE4m3) {
                        *reinterpret_cast<uint2*>(to) = bf16x8_to_e4m3(xa[n], inv);
                        *reinterpret_cast<uint2*>(to + cb_ca) = bf16x8_to_e4m3(xb[n], inv);
                    } else {
                        *reinterpret_cast<uint4*>(to) = xa[n];
                        *reinterpret_cast<uint4*>(to + E * cb_ca) = xb[n];
                    }
                }
            src += N * pitch;
            dst += N * step;
            left -= N * apart;
            load();
        }
    }
};

struct RopeArgs {
    HeadRows q, k;           // k.p null: q alone
    __nv_bfloat16 *q_out, *k_out;
    long long qo_row, qo_head, ko_row, ko_head;
    int total, Hq, Hkv;
    int parts;               // warps that share a token's heads
    RopeTable r;
};

template <int D>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
    constexpr int U = D / 16;            // units of a head
    constexpr int HP = 32 / U;           // heads a warp takes at once
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const long long t = w / a.parts;
    const int part = (int)(w % a.parts);
    if (t >= a.total) return;
    const int u = lane % U;
    const bool turns = u < a.r.rot / 16;
    int ca, cb;
    rope_columns(a.r, u, &ca, &cb);
    const int first = part * HP + lane / U;
    RopeRows<D, D == 64 ? 2 : 4> q;      // (two groups of narrow heads are 16: at four, 22.5 us in place of 20.5
    RopeRows<D, 2> k;                    // for 11103 tokens of 16 + 16 heads)
    q.start(a.q, t, a.Hq, first, a.parts, ca, cb);     // in flight while the angles are looked up
    k.start(a.k, t, a.Hkv, first, a.parts, ca, cb);
    RopeAngles g;
    if (turns) g = rope_angles(a.r, t, a.total, u, 0);
    q.template finish<kCacheBf16>(reinterpret_cast<uint8_t*>(a.q_out + t * a.qo_row + first * a.qo_head + ca),
                                  2 * a.parts * HP * a.qo_head, turns, g, a.r.interleaved, 1.0f);
    k.template finish<kCacheBf16>(reinterpret_cast<uint8_t*>(a.k_out + t * a.ko_row + first * a.ko_head + ca),
                                  2 * a.parts * HP * a.ko_head, turns, g, a.r.interleaved, 1.0f);
}

// ---------------------------------------------------------------- append
struct RopeAppendArgs {
    HeadRows q, k, v;        // q.p null: keys and values alone
    void* q_out;             // [total_new][Hq][D], bf16 or e4m3 (the cache's type; bf16 for 4-bit pages)
    uint8_t *k_cache, *v_cache;   // bf16, e4m3: [num_blocks][16][Hkv][D]; 4-bit: [num_blocks][Hkv][16 D / 2] bytes
    uint16_t *k_meta, *v_meta;    // 4-bit: [num_blocks][Hkv][16][D / group]
    const float *descale_q, *descale_k, *descale_v;   // e4m3
    const int* block_table;
    int max_blocks, num_blocks;
    const int* cu_new;       // [B + 1], or null: one new token per sequence
    const int* seqused_k;
    int* seqused_k_out;      // or null
    int B, total_new, Hq, Hkv;
    int parts;
    RopeTable r;
};

// The sequence of new token t (-1: behind the last sequence), its position in
// the cache and the page that holds it (-1: not to be written).
struct NewToken {
    int b, pos;
    long long page;
};

__device__ __forceinline__ NewToken find_new_token(const RopeAppendArgs& a, int t, int lane) {
    NewToken n;
    int first = t;
    n.b = t;
    n.page = -1;
    n.pos = 0;
    if (a.cu_new) {
        const int begin = __ldg(&a.cu_new[0]), end = __ldg(&a.cu_new[a.B]);
        // the largest b with cu_new[b] <= t, 32 candidates at a time
        int b = 0;
        first = begin;
        for (int len = a.B; len > 0;) {
            const int step = (len + 31) / 32, i = lane * step;
            const int c = i < len ? __ldg(&a.cu_new[b + i]) : 0;
            const int k = max(__popc(__ballot_sync(0xffffffffu, i < len && c <= t)) - 1, 0);
            first = __shfl_sync(0xffffffffu, c, k);
            b += k * step;
            len = step == 1 ? 0 : min(step, len - k * step);
        }
        n.b = t < begin || t >= end ? -1 : b;
        if (n.b < 0) return n;
    }
    n.pos = __ldg(&a.seqused_k[n.b]) + (t - first);
    const int slot = n.pos >= 0 ? n.pos / kPageRows : -1;
    if (slot < 0 || slot >= a.max_blocks) {
        if (lane == 0) record_data_error(kErrAppendSlot);
        return n;
    }
    const int page = __ldg(&a.block_table[(long long)n.b * a.max_blocks + slot]);
    if (page < 0 || page >= a.num_blocks) {
        if (lane == 0) record_data_error(kErrAppendPage);
        return n;
    }
    n.page = page;
    return n;
}

__device__ __forceinline__ void append_lengths(const RopeAppendArgs& a) {
    if (!a.seqused_k_out) return;
    for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < a.B; b += gridDim.x * blockDim.x)
        a.seqused_k_out[b] = a.seqused_k[b] + (a.cu_new ? a.cu_new[b + 1] - a.cu_new[b] : 1);
}

// New tokens into bf16 or e4m3 pages: q turned into q_out, k turned into its
// page, v into its page.  A warp takes `1 / parts` of one token's heads.  HBM
// bound over long chunks, latency bound over a decode step: the token's sequence
// (a search 32 candidates wide: two round trips up to 1024 sequences), its page
// and its angles hang on one another, so q's rows are asked for first.
// 10100 tokens of 32 + 8 + 8 heads of 128 into e4m3 pages: 39 to 41 us, 4.7 TB/s
// (48 with the rows loaded after the look-ups; 80 registers for six blocks on an
// SM spill and gain nothing).  32 tokens, one each: 8 us.
template <int D, int CACHE>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeAppendArgs a) {
    constexpr int U = D / 16, HP = 32 / U;
    constexpr int E = CACHE == kCacheE4m3 ? 1 : 2;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    append_lengths(a);
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const long long t = w / a.parts;
    const int part = (int)(w % a.parts);
    if (t >= a.total_new) return;
    const int u = lane % U;
    const bool turns = a.r.table && u < a.r.rot / 16;
    int ca, cb;
    rope_columns(a.r, u, &ca, &cb);
    const int first = part * HP + lane / U;
    RopeRows<D, 4> q;
    RopeRows<D, 2> k, v;                 // (fewer heads)
    q.start(a.q, t, a.Hq, first, a.parts, ca, cb);     // in flight while the token's page and angles are looked up
    const NewToken nt = find_new_token(a, (int)t, lane);
    if (nt.b < 0) return;
    RopeAngles g;
    if (turns) g = rope_angles(a.r, t, a.total_new, u, nt.pos);
    float iq = 1.0f, ik = 1.0f, iv = 1.0f;
    if (CACHE == kCacheE4m3) {
        if (a.q.p) iq = __frcp_rn(__ldg(a.descale_q));
        ik = __frcp_rn(__ldg(a.descale_k));
        iv = __frcp_rn(__ldg(a.descale_v));
    }
    const long long step = (long long)a.parts * HP * D * E;
    q.template finish<CACHE>(static_cast<uint8_t*>(a.q_out) + ((t * a.Hq + first) * D + ca) * E, step, turns, g, a.r.interleaved, iq);
    if (nt.page < 0) return;
    k.start(a.k, t, a.Hkv, first, a.parts, ca, cb);
    v.start(a.v, t, a.Hkv, first, a.parts, ca, cb);
    const long long at = (((nt.page * kPageRows + nt.pos % kPageRows) * a.Hkv + first) * D + ca) * E;
    k.template finish<CACHE>(a.k_cache + at, step, turns, g, a.r.interleaved, ik);
    v.template finish<CACHE>(a.v_cache + at, step, false, g, false, iv);
}

}  // namespace attn
