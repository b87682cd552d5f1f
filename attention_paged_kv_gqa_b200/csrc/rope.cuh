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
// cosines and sines are loaded once for a token and stay in registers.
#pragma once

#include "ptx.cuh"
#include "prefill.cuh"   // kPageRows

namespace attn {

constexpr int kRopeThreads = 256;
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

// Cosines and sines of the eight pairs 8 u .. 8 u + 7 of token t.
__device__ __forceinline__ void rope_angles(const RopeTable& r, long long t, long long total, int u, int seq_pos,
                                            float (&c)[8], float (&s)[8]) {
    const int half = r.rot / 2;
    auto place = [&](int axis) {
        int p = r.positions ? __ldg(r.positions + axis * total + t) : seq_pos;
        if (p < 0 || p >= r.max_pos) {
            record_data_error(kErrRopePosition);   // reported, the nearest row used
            p = min(max(p, 0), r.max_pos - 1);
        }
        return p;
    };
    int ax[8];
    bool one = true;
    if (r.pair_axis) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            ax[i] = __ldg(r.pair_axis + 8 * u + i);
            if (ax[i] < 0 || ax[i] >= r.axes) {
                record_data_error(kErrRopeAxis);
                ax[i] = 0;
            }
            one = one && ax[i] == ax[0];
        }
    } else {
        ax[0] = 0;
    }
    if (one) {
        const float* row = r.table + (long long)place(ax[0]) * r.rot + 8 * u;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 cv = __ldg(reinterpret_cast<const float4*>(row + i));
            const float4 sv = __ldg(reinterpret_cast<const float4*>(row + half + i));
            c[i] = cv.x, c[i + 1] = cv.y, c[i + 2] = cv.z, c[i + 3] = cv.w;
            s[i] = sv.x, s[i + 1] = sv.y, s[i + 2] = sv.z, s[i + 3] = sv.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float* row = r.table + (long long)place(ax[i]) * r.rot + 8 * u + i;
            c[i] = __ldg(row);
            s[i] = __ldg(row + half);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] *= r.sign;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Turns the pair (x1, x2); every operation rounded by itself.
__device__ __forceinline__ void rope_turn(float& x1, float& x2, float c, float s) {
    const float y1 = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
    x2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
    x1 = y1;
}

// Turns a unit: pieces a and b hold the first and second columns of the eight
// pairs, or eight interleaved pairs in order.
__device__ __forceinline__ void rope_unit(uint4& a, uint4& b, const float (&c)[8], const float (&s)[8], bool interleaved) {
    uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
    uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x1 = bf16_lo(wa[i]), x2 = bf16_hi(wa[i]);
            rope_turn(x1, x2, c[i], s[i]);
            wa[i] = pack_bf16(x1, x2);
            x1 = bf16_lo(wb[i]), x2 = bf16_hi(wb[i]);
            rope_turn(x1, x2, c[4 + i], s[4 + i]);
            wb[i] = pack_bf16(x1, x2);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x1 = bf16_lo(wa[i]), x2 = bf16_lo(wb[i]);
            float z1 = bf16_hi(wa[i]), z2 = bf16_hi(wb[i]);
            rope_turn(x1, x2, c[2 * i], s[2 * i]);
            rope_turn(z1, z2, c[2 * i + 1], s[2 * i + 1]);
            wa[i] = pack_bf16(x1, z1);
            wb[i] = pack_bf16(x2, z2);
        }
    }
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
    float c[8], s[8];
    if (turns) rope_angles(a.r, t, a.total, u, 0, c, s);
    int ca, cb;
    rope_columns(a.r, u, &ca, &cb);
    const int H = a.Hq + a.Hkv;
    constexpr int N = 4;                 // head groups whose loads are in flight together
    for (int h0 = part * HP + lane / U; h0 < H; h0 += a.parts * HP * N) {
        uint4 xa[N], xb[N];
        __nv_bfloat16* dst[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int h = h0 + n * a.parts * HP;
            if (h < H) {
                const bool isq = h < a.Hq;
                const __nv_bfloat16* src = isq ? a.q.p + t * a.q.row + h * a.q.head
                                               : a.k.p + t * a.k.row + (h - a.Hq) * a.k.head;
                dst[n] = isq ? a.q_out + t * a.qo_row + h * a.qo_head
                             : a.k_out + t * a.ko_row + (h - a.Hq) * a.ko_head;
                xa[n] = *reinterpret_cast<const uint4*>(src + ca);
                xb[n] = *reinterpret_cast<const uint4*>(src + cb);
            }
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int h = h0 + n * a.parts * HP;
            if (h < H) {
                if (turns) rope_unit(xa[n], xb[n], c, s, a.r.interleaved);
                *reinterpret_cast<uint4*>(dst[n] + ca) = xa[n];
                *reinterpret_cast<uint4*>(dst[n] + cb) = xb[n];
            }
        }
    }
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

__device__ __forceinline__ NewToken find_new_token(const RopeAppendArgs& a, int t, bool report) {
    NewToken n;
    int first = t;
    n.b = t;
    n.page = -1;
    n.pos = 0;
    if (a.cu_new) {
        if (t < __ldg(&a.cu_new[0]) || t >= __ldg(&a.cu_new[a.B])) {
            n.b = -1;
            return n;
        }
        int lo = 0, hi = a.B;           // the largest b with cu_new[b] <= t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(&a.cu_new[mid]) <= t) lo = mid; else hi = mid;
        }
        n.b = lo;
        first = __ldg(&a.cu_new[lo]);
    }
    n.pos = __ldg(&a.seqused_k[n.b]) + (t - first);
    const int slot = n.pos >= 0 ? n.pos / kPageRows : -1;
    if (slot < 0 || slot >= a.max_blocks) {
        if (report) record_data_error(kErrAppendSlot);
        return n;
    }
    const int page = __ldg(&a.block_table[(long long)n.b * a.max_blocks + slot]);
    if (page < 0 || page >= a.num_blocks) {
        if (report) record_data_error(kErrAppendPage);
        return n;
    }
    n.page = page;
    return n;
}

// Eight bf16 values times `inv`, as e4m3 (nearest even, saturating at +-448).
__device__ __forceinline__ uint2 bf16x8_to_e4m3(uint4 x, float inv) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        o[i] = pack_e4m3x4(bf16_lo(w[2 * i]) * inv, bf16_hi(w[2 * i]) * inv, bf16_lo(w[2 * i + 1]) * inv,
                           bf16_hi(w[2 * i + 1]) * inv);
    return make_uint2(o[0], o[1]);
}

__device__ __forceinline__ void append_lengths(const RopeAppendArgs& a) {
    if (!a.seqused_k_out) return;
    for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < a.B; b += gridDim.x * blockDim.x)
        a.seqused_k_out[b] = a.seqused_k[b] + (a.cu_new ? a.cu_new[b + 1] - a.cu_new[b] : 1);
}

// New tokens into bf16 or e4m3 pages: q turned into q_out, k turned into its
// page, v into its page.  A warp takes `1 / parts` of one token's heads.
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
    const NewToken nt = find_new_token(a, (int)t, lane == 0);
    if (nt.b < 0) return;
    const int u = lane % U;
    const bool turns = a.r.table && u < a.r.rot / 16;
    float c[8], s[8];
    if (turns) rope_angles(a.r, t, a.total_new, u, nt.pos, c, s);
    int ca, cb;
    rope_columns(a.r, u, &ca, &cb);
    float iq = 1.0f, ik = 1.0f, iv = 1.0f;
    if (CACHE == kCacheE4m3) {
        if (a.q.p) iq = __frcp_rn(__ldg(a.descale_q));
        ik = __frcp_rn(__ldg(a.descale_k));
        iv = __frcp_rn(__ldg(a.descale_v));
    }
    const long long row0 = (nt.page * kPageRows + nt.pos % kPageRows) * a.Hkv;   // cache row of KV head 0
    const int H = a.Hq + 2 * a.Hkv;
    constexpr int N = 4;
    for (int h0 = part * HP + lane / U; h0 < H; h0 += a.parts * HP * N) {
        uint4 xa[N], xb[N];
        uint8_t* dst[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int h = h0 + n * a.parts * HP;
            dst[n] = nullptr;
            if (h >= H) continue;
            const __nv_bfloat16* src;
            if (h < a.Hq) {
                src = a.q.p + t * a.q.row + h * a.q.head;
                dst[n] = static_cast<uint8_t*>(a.q_out) + (t * a.Hq + h) * (D * E);
            } else if (nt.page >= 0) {
                const bool isk = h < a.Hq + a.Hkv;
                const int g = h - a.Hq - (isk ? 0 : a.Hkv);
                src = isk ? a.k.p + t * a.k.row + g * a.k.head : a.v.p + t * a.v.row + g * a.v.head;
                dst[n] = (isk ? a.k_cache : a.v_cache) + (row0 + g) * (D * E);
            } else {
                continue;
            }
            xa[n] = *reinterpret_cast<const uint4*>(src + ca);
            xb[n] = *reinterpret_cast<const uint4*>(src + cb);
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if (!dst[n]) continue;
            const int h = h0 + n * a.parts * HP;
            if (turns && h < a.Hq + a.Hkv) rope_unit(xa[n], xb[n], c, s, a.r.interleaved);
            if (CACHE == kCacheE4m3) {
                const float inv = h < a.Hq ? iq : h < a.Hq + a.Hkv ? ik : iv;
                *reinterpret_cast<uint2*>(dst[n] + ca) = bf16x8_to_e4m3(xa[n], inv);
                *reinterpret_cast<uint2*>(dst[n] + cb) = bf16x8_to_e4m3(xb[n], inv);
            } else {
                *reinterpret_cast<uint4*>(dst[n] + 2 * ca) = xa[n];
                *reinterpret_cast<uint4*>(dst[n] + 2 * cb) = xb[n];
            }
        }
    }
}

}  // namespace attn
