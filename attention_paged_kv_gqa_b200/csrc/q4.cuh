// q4.cuh -- the KV cache held in 4 bits: appending to it, reading it back, and
// attention over it for one or a few query tokens per sequence.
//
// Format.  Along head_dim every `group` (32, 64 or 128) values x of a token and
// head share a step and a zero code: with lo = min(x, 0), hi = max(x, 0), step is
// (hi - lo) / 15 rounded up to 4 significant bits (0 below 2^-100; NaN where the
// group holds a NaN or an infinity) and zero = nearest(-lo / step).  The code of x
// is nearest(x / step) + zero (ties to even) held within 0 .. 15 and stands for
// step * (code - zero): at most 4 x 4 significant bits, so a bf16 number exactly,
// at most half a step from x.  A meta is the 16 bits of step as bf16, whose
// lowest four are free and hold zero.
//   k_cache, v_cache  bytes  [num_blocks][Hkv][16 * D / 2]
//   k_meta, v_meta    uint16 [num_blocks][Hkv][16][D / group]
// K tile: 16 rows (tokens) of D nibbles; dim d = 32 w + 8 c + e is nibble e of the
// row's 32-bit word c * (D / 32) + w.  V tile: token 8 a + 2 c + h, dim
// 32 u + 8 j + r is nibble j of the 16-bit piece
// (((a * 8 + r) * 4 + c) * (D / 32) + u) * 2 + h.
// Both orders are those in which a lane of the warp MMA below wants its operand:
// lane 4 r + c reads its words of a tile with one or two vector loads, without
// bank conflicts and without a transposition.
#pragma once

#include "append.cuh"
#include "decode.cuh"
#include "rope.cuh"

namespace attn {

enum : int { kErrQ4Rows = 531, kErrQ4Full = 541, kErrQ4Empty = 542 };

// ---------------------------------------------------------------- quantiser
struct Q4Group {
    float step, inv;         // inv = 1 / step, or 0
    float zero;
    uint32_t meta;
};

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// nearest(x / step) as an integer-valued float plus kQ4Magic (its low bits are
// the integer), for |x / step| <= 16.  x has 8 significant bits and step 4, so
// x / step lies either on a half-integer or further than 2^-12 from one: the sum
// with 768, rounded to 2^-14, makes ties exact again whatever the rounding of
// inv, and the second sum rounds them to even.
constexpr float kQ4Magic = 12582912.0f;     // 1.5 * 2^23
__device__ __forceinline__ float q4_nearest(float x, float inv) {
    return __fadd_rn(__fmaf_rn(x, inv, 768.0f), kQ4Magic - 768.0f);
}

// Step and zero of a group from its lo <= 0 and hi >= 0 (NaN where it has one).
__device__ __forceinline__ Q4Group q4_group(float lo, float hi) {
    Q4Group g;
    const float s = __fdiv_rn(__fsub_rn(hi, lo), 15.0f);
    uint32_t bits = (__float_as_uint(s) + 0xfffffu) & 0xfff00000u;
    if (!(s < INFINITY)) bits = 0x7fc00000u;         // NaN or an infinity in the group
    else if (__uint_as_float(bits) < 7.888609052210118e-31f) bits = 0;   // 2^-100
    g.step = __uint_as_float(bits);
    const bool live = bits != 0 && bits != 0x7fc00000u;
    g.inv = live ? __frcp_rn(g.step) : 0.0f;
    g.zero = live ? __fsub_rn(q4_nearest(-lo, g.inv), kQ4Magic) : 0.0f;
    g.meta = (bits >> 16) | (uint32_t)(int)g.zero;
    return g;
}

// The codes of eight values, value i in nibble i.
__device__ __forceinline__ uint32_t q4_codes(const float (&x)[8], const Q4Group& g) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // (zero is added after the rounding, whose ties are to even; a NaN is held to the
        // lower bound, its group's step is NaN)
        const float v = fminf(fmaxf(__fadd_rn(q4_nearest(x[i], g.inv), g.zero), kQ4Magic), kQ4Magic + 15.0f);
        w |= (__float_as_uint(v) & 15u) << (4 * i);
    }
    return w;
}

__device__ __forceinline__ float q4_step(uint32_t meta) { return __uint_as_float((meta << 16) & 0xfff00000u); }
__device__ __forceinline__ float q4_zero(uint32_t meta) { return (float)(meta & 15u); }

// ---------------------------------------------------------------- append
// New tokens into 4-bit pages: q turned into q_out (bf16), k turned, rounded to
// bf16 as attn_rope would, and quantised, v quantised.  A warp takes 1 / parts of
// one token's heads.  For k and v a lane holds eight consecutive columns (the
// partner columns of a half-split pair come from another lane), a group's
// smallest and largest are found across its group / 8 lanes, a K word is one
// lane's eight codes, and the V pieces are regrouped among the four lanes that
// hold the dims 32 u .. 32 u + 31.
template <int D, int GS>
__global__ void __launch_bounds__(kRopeThreads) rope_append_q4_kernel(const RopeAppendArgs a) {
    constexpr int U = D / 16, HP = 32 / U;        // q: units, heads at once
    constexpr int LPH = D / 8, HV = 32 / LPH;     // k, v: lanes of a head, heads at once
    constexpr int W = D / 32, G = D / GS;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    append_lengths(a);
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const long long t = w / a.parts;
    const int part = (int)(w % a.parts);
    if (t >= a.total_new) return;
    const NewToken nt = find_new_token(a, (int)t, lane == 0);
    if (nt.b < 0) return;
    const int nrot = a.r.table ? a.r.rot / 16 : 0;

    const int nq = (a.Hq + HP - 1) / HP, nk = (a.Hkv + HV - 1) / HV;   // passes over q; over k, over v
    {
        const int u = lane % U;
        const bool turns = u < nrot;
        float c[8], s[8];
        if (turns && part < nq) rope_angles(a.r, t, a.total_new, u, nt.pos, c, s);
        int ca, cb;
        rope_columns(a.r, u, &ca, &cb);
        for (int i = part; i < nq; i += a.parts) {
            const int h = i * HP + lane / U;
            if (h >= a.Hq) continue;
            const __nv_bfloat16* src = a.q.p + t * a.q.row + h * a.q.head;
            uint4 xa = *reinterpret_cast<const uint4*>(src + ca), xb = *reinterpret_cast<const uint4*>(src + cb);
            if (turns) rope_unit(xa, xb, c, s, a.r.interleaved);
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.q_out) + (t * a.Hq + h) * D;
            *reinterpret_cast<uint4*>(dst + ca) = xa;
            *reinterpret_cast<uint4*>(dst + cb) = xb;
        }
    }
    if (nt.page < 0) return;
    const int v = lane % LPH;                      // columns 8 v .. 8 v + 7
    const int row = nt.pos % kPageRows;
    // first pass of this part among the k and v passes nq .. nq + 2 nk
    int i = part;
    if (i < nq) i += (nq - i + a.parts - 1) / a.parts * a.parts;
    for (; i < nq + 2 * nk; i += a.parts) {
        const bool isk = i < nq + nk;
        const int h = (isk ? i - nq : i - nq - nk) * HV + lane / LPH;
        const bool live = h < a.Hkv;
        const HeadRows& x = isk ? a.k : a.v;
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (live) raw = *reinterpret_cast<const uint4*>(x.p + t * x.row + h * x.head + 8 * v);
        const uint32_t wd[4] = {raw.x, raw.y, raw.z, raw.w};
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[2 * e] = bf16_lo(wd[e]);
            f[2 * e + 1] = bf16_hi(wd[e]);
        }
        if (isk && nrot) {
            if (a.r.interleaved) {
                if (v < 2 * nrot) {
                    // pairs 4 v .. 4 v + 3: half of the eight whose angles start at 8 (v / 2)
                    float c[8], s[8];
                    rope_angles(a.r, t, a.total_new, v / 2, nt.pos, c, s);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        rope_turn(f[2 * e], f[2 * e + 1], v & 1 ? c[4 + e] : c[e], v & 1 ? s[4 + e] : s[e]);
                }
            } else {
                // columns 8 v .. of the first half turn with those 8 (v + nrot) .. of the second
                const int mate = lane - v + (v < nrot ? v + nrot : v < 2 * nrot ? v - nrot : v);
                uint32_t pw[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) pw[e] = __shfl_sync(0xffffffffu, wd[e], mate);
                if (v < 2 * nrot) {
                    const bool first = v < nrot;
                    float c[8], s[8];
                    rope_angles(a.r, t, a.total_new, first ? v : v - nrot, nt.pos, c, s);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float m = e & 1 ? bf16_hi(pw[e / 2]) : bf16_lo(pw[e / 2]);
                        float x1 = first ? f[e] : m, x2 = first ? m : f[e];
                        rope_turn(x1, x2, c[e], s[e]);
                        f[e] = first ? x1 : x2;
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const uint32_t p = pack_bf16(f[e], f[e + 1]);
                f[e] = bf16_lo(p);
                f[e + 1] = bf16_hi(p);
            }
        }
        float lo = 0.0f, hi = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            lo = min_nan(lo, f[e]);
            hi = max_nan(hi, f[e]);
        }
#pragma unroll
        for (int o = 1; o < GS / 8; o <<= 1) {
            lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        const Q4Group g = q4_group(lo, hi);
        uint32_t codes = q4_codes(f, g);
        const long long tile = nt.page * a.Hkv + h;
        if (isk) {
            if (live) {
                uint32_t* kt = reinterpret_cast<uint32_t*>(a.k_cache + tile * (kPageRows * D / 2)) + row * (D / 8);
                kt[(v % 4) * W + v / 4] = codes;
            }
        } else {
            // lane j of a quad holds nibble r of dims 32 u + 8 j + r; it takes pieces r = 2 j, 2 j + 1
            const int j = lane & 3;
            uint32_t q[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t other = __shfl_sync(0xffffffffu, codes, (lane & ~3) + e);
                q[e] = (other >> (8 * j)) & 0xffu;
            }
            const uint32_t even = (q[0] & 15u) | (q[1] & 15u) << 4 | (q[2] & 15u) << 8 | (q[3] & 15u) << 12;
            const uint32_t odd = q[0] >> 4 | (q[1] >> 4) << 4 | (q[2] >> 4) << 8 | (q[3] >> 4) << 12;
            if (live) {
                uint16_t* vt = reinterpret_cast<uint16_t*>(a.v_cache + tile * (kPageRows * D / 2));
                const int at = (((row / 8) * 8 * 4 + row % 8 / 2) * W + v / 4) * 2 + row % 2;   // piece r = 0
                vt[at + 2 * j * 4 * W * 2] = (uint16_t)even;
                vt[at + (2 * j + 1) * 4 * W * 2] = (uint16_t)odd;
            }
        }
        if (live && v % (GS / 8) == 0)
            (isk ? a.k_meta : a.v_meta)[(tile * kPageRows + row) * G + v / (GS / 8)] = (uint16_t)g.meta;
    }
}

// ---------------------------------------------------------------- read back
struct Q4GatherArgs {
    const uint8_t *k_cache, *v_cache;
    const uint16_t *k_meta, *v_meta;
    const int* block_table;
    int max_blocks, num_blocks;
    const int* cu;           // [B + 1] rows of each sequence in the output; null: all of each (lens)
    const int* starts;       // [B] first token of each, or null: 0
    const int* lens;         // [B] (cu null)
    int* cu_out;             // [B + 1] (cu null): the rows' offsets, held within `total`
    int B, total, Hkv;
    __nv_bfloat16 *k_out, *v_out;   // [total][Hkv][D]
};

// Two codes (nibbles at bits 0 and 16 of w) as step * (code - zero) in bf16x2.
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, float step, float zero) {
    return pack_bf16(((float)(w & 15u) - zero) * step, ((float)((w >> 16) & 15u) - zero) * step);
}

// The rows of packed K and V from 4-bit pages: a warp takes the K and V tile of
// one page and head.  The values are bf16 numbers, so nothing is lost.
template <int D, int GS>
__global__ void __launch_bounds__(256) q4_gather_kernel(const Q4GatherArgs a) {
    constexpr int W = D / 32, G = D / GS;
    extern __shared__ int smem_tab[];
    int* pages = smem_tab;                  // [B + 1] pages before sequence b
    int* rows = smem_tab + a.B + 1;         // [B + 1] output rows before it
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < 32) {
        int run_p = 0, run_r = 0;
        for (int base = 0; base < a.B; base += 32) {
            const int b = base + lane;
            int n = 0, np = 0, s0 = 0;
            if (b < a.B) {
                if (a.starts) s0 = max(a.starts[b], 0);
                n = a.cu ? a.cu[b + 1] - a.cu[b] : a.lens[b];
                n = min(max(n, 0), max(a.max_blocks * kPageRows - s0, 0));
                np = n > 0 ? (s0 + n - 1) / kPageRows - s0 / kPageRows + 1 : 0;
            }
            int ip = np, ir = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, ip, o), y = __shfl_up_sync(0xffffffffu, ir, o);
                if (lane >= o) ip += x, ir += y;
            }
            if (b < a.B) {
                pages[b] = run_p + ip - np;
                rows[b] = a.cu ? a.cu[b] : run_r + ir - n;
            }
            run_p += __shfl_sync(0xffffffffu, ip, 31);
            run_r += __shfl_sync(0xffffffffu, ir, 31);
        }
        if (lane == 0) {
            pages[a.B] = run_p;
            rows[a.B] = a.cu ? a.cu[a.B] : run_r;
            if (blockIdx.x == 0 && rows[a.B] > a.total) record_data_error(kErrQ4Rows);
        }
    }
    __syncthreads();
    if (a.cu_out && blockIdx.x == 0)
        for (int b = threadIdx.x; b <= a.B; b += blockDim.x) a.cu_out[b] = min(rows[b], a.total);
    const long long items = (long long)pages[a.B] * a.Hkv;
    const int warps = gridDim.x * (blockDim.x >> 5);
    for (long long it = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items; it += warps) {
        const int g = (int)(it / a.Hkv), h = (int)(it % a.Hkv);
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pages[mid] <= g) lo = mid; else hi = mid;
        }
        const int b = lo;
        const int s0 = a.starts ? max(a.starts[b], 0) : 0;
        const int slot = s0 / kPageRows + (g - pages[b]);
        int n = a.cu ? a.cu[b + 1] - a.cu[b] : a.lens[b];
        n = min(n, a.max_blocks * kPageRows - s0);
        int page = __ldg(&a.block_table[(long long)b * a.max_blocks + slot]);
        if (page < 0 || page >= a.num_blocks) {
            if (lane == 0) record_data_error(kErrDecPageRange);
            page = 0;
        }
        const long long tile = (long long)page * a.Hkv + h;
        const int tok0 = slot * kPageRows;
        // output row of page row y, or -1
        auto out_row = [&](int y) -> long long {
            const int i = tok0 + y - s0;
            if (i < 0 || i >= n) return -1;
            const long long r = rows[b] + (long long)i;
            return r >= 0 && r < a.total ? r : -1;
        };
        const uint16_t* km = a.k_meta + tile * kPageRows * G;
        const uint16_t* vm = a.v_meta + tile * kPageRows * G;
        // K: 4 units (16-byte piece c) of W words in each of the 16 rows
        const uint32_t* kt = reinterpret_cast<const uint32_t*>(a.k_cache + tile * (kPageRows * D / 2));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int y = (lane + 32 * i) / 4, c = lane % 4;
            const long long r = out_row(y);
            if (r < 0) continue;
            __nv_bfloat16* dst = a.k_out + (r * a.Hkv + h) * D;
#pragma unroll
            for (int wi = 0; wi < W; ++wi) {
                const uint32_t w = __ldg(kt + (y * 4 + c) * W + wi);
                const uint32_t m = __ldg(km + y * G + 32 * wi / GS);
                const float st = q4_step(m), z = q4_zero(m);
                // nibble e at bits 4 e: pairs (0, 1), (2, 3) ...
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t p = w >> (8 * e);
                    o[e] = q4_pair((p & 15u) | (p & 0xf0u) << 12, st, z);
                }
                *reinterpret_cast<uint4*>(dst + 32 * wi + 8 * c) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        // V: lane (token pair p = 4 a + c, word u): the eight words r = 0 .. 7 hold its two
        // tokens' dims 32 u + 8 j + r
        const uint32_t* vt = reinterpret_cast<const uint32_t*>(a.v_cache + tile * (kPageRows * D / 2));
        const int u = lane % W, p = lane / W;
        if (p < 8) {
            const int y = 2 * p;
            uint32_t wr[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) wr[r] = __ldg(vt + (((p / 4) * 8 + r) * 4 + p % 4) * W + u);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const long long r = out_row(y + half);
                if (r < 0) continue;
                const uint32_t m = __ldg(vm + (y + half) * G + 32 * u / GS);
                const float st = q4_step(m), z = q4_zero(m);
                __nv_bfloat16* dst = a.v_out + (r * a.Hkv + h) * D + 32 * u;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int sh = 16 * half + 4 * j;
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[e] = q4_pair(((wr[2 * e] >> sh) & 15u) | ((wr[2 * e + 1] >> sh) & 15u) << 16, st, z);
                    *reinterpret_cast<uint4*>(dst + 8 * j) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
    }
}

// ---------------------------------------------------------------- attention
// A few query rows per sequence (R = tokens x query heads of a KV head <= 8 NT)
// over 4-bit pages: the page stream of decode.cuh with another consumer.
//
// The pages of the batch, for one block of HB KV heads after another, are cut
// into one contiguous equal share per CTA.  A page's HB tiles of K, V and their
// metas are four contiguous runs, fetched by four bulk copies into a ring of
// stages.  Of the SUB warps of a KV head each takes every SUB-th page and keeps an
// online softmax of its own; where a sequence or the share ends they are joined
// through shared memory, and the partial (O normalised, LSE) goes to slot
// CTA + sequence for the combine kernel.
//
// Score: s = step (q . c - zero sum q), c the codes: the code, shifted to the
// low or second nibble of a 16-bit half, IS the f16 number c 2^-24 or c 2^-20
// (subnormal, exact), so a K word becomes four A registers with four ANDs and a
// shift.  q is exact in f16 after a power of two per row, divided by 16 for the
// dims that meet second nibbles.  The output: O = sum_j w_j c_j - sum_j w_j zero_j
// with w_j = p_j step_j, again on the codes as they are; w is rounded to f16
// (11 bits) after a power of two that keeps the largest step in range.  Groups
// smaller than the head repeat the two sums per group.
// The first sum is far larger than the difference where p is spread over many
// keys, and the tensor cores truncate when they add; every 16 pages the second
// sum is therefore taken out of the accumulators, which stay near their final size.
// The running maximum moves only when a score exceeds it by 2^8, which a page
// shows by one vote.
constexpr int kQ4MaxHeads = 8;           // KV heads of a CTA's block
constexpr float kQ4Slack = 8.0f;         // p <= 2^8 between moves of the maximum
constexpr int kQ4Recentre = 16;          // pages

struct Q4AttnArgs {
    int B, Hq, Hkv, group;
    int HB, SUB, nhb;        // KV heads of a block, warps of a head, blocks
    const __nv_bfloat16* q;  // rows of queries [..][Hq][D]
    const int* cu_q;         // [B + 1], or null: one query per sequence
    int max_q;               // query tokens a sequence may have (group * max_q <= 8 NT)
    int total_q;
    const uint8_t *k_cache, *v_cache;
    const uint16_t *k_meta, *v_meta;
    const int* block_table;
    int max_blocks, num_blocks;
    const int* seqused_k;
    float scale;
    int causal;              // 0: every query sees every key
    int window;              // < 0: none
    float softcap;           // 0: none
    float* o_part;           // [slots][HB][8 NT][D]
    float* lse_part;         // [slots][HB][8 NT]
    int* meta;               // [B + 1] page prefix, then pages per CTA
    int nstages;
    __nv_bfloat16* o;        // as q
    float* lse;              // [Hq][total_q], or [B][Hq] (cu_q null); or null
};

template <int D, int GS>
struct Q4Cfg {
    static constexpr int TILE = kPageRows * D / 2;              // bytes of a head's K or V tile
    static constexpr int META = kPageRows * (D / GS) * 2;       // bytes of its metas
    __host__ __device__ static constexpr int stage_bytes(int HB) { return 2 * HB * (TILE + META); }
    __host__ __device__ static constexpr int merge_bytes(int HB, int SUB, int NT) {
        // per exchange slot: the accumulators of a warp, its maxima and sums
        return SUB > 1 ? HB * ((SUB + 1) / 2) * 32 * (D / 16 * NT * 4 + NT * 4) * 4 : 0;
    }
    __host__ __device__ static constexpr int table_bytes(int B) { return ((2 * B + 2) * 4 + 15) / 16 * 16; }
    __host__ __device__ static constexpr int smem_bytes(int HB, int SUB, int NT, int B, int ns) {
        return 128 + ns * stage_bytes(HB) + merge_bytes(HB, SUB, NT) + table_bytes(B) + 2 * ns * 8;
    }
};

// n contiguous bytes (a multiple of 16, both sides 16-byte aligned) into shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t n, uint64_t* bar, uint64_t pol) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(n), "r"(smem_u32(bar)), "l"(pol)
        : "memory");
}

// Keys the sequence's queries can see start here (the window of its first query).
__device__ __forceinline__ int q4_first_key(int L, int n, int window) {
    return window >= 0 ? max(0, L - n - window) : 0;
}

template <int D, int GS, int NT>
__global__ void __launch_bounds__(NT == 1 ? 544 : 288, 1) q4_attn_kernel(const Q4AttnArgs a) {
    using C = Q4Cfg<D, GS>;
    constexpr int W = D / 32;            // words of a lane's K row piece; V words per token pair
    constexpr int G = D / GS;            // groups of a head
    constexpr int WG = W / G;            // words of a group
    constexpr int MT = D / 16;           // 16-column output tiles
    const int NS = a.nstages, HB = a.HB, SUB = a.SUB, SB = C::stage_bytes(HB);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    float* mrg = reinterpret_cast<float*>(smem + NS * SB);
    int* prefix = reinterpret_cast<int*>(smem + NS * SB + C::merge_bytes(HB, SUB, NT));   // [B + 1]
    int* lenv = prefix + (a.B + 1);                                                     // [B]
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + NS * SB + C::merge_bytes(HB, SUB, NT) + C::table_bytes(a.B));
    uint64_t* empty = full + NS;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cap = a.max_blocks * kPageRows;
    auto queries = [&](int b) { return a.cu_q ? min(max(__ldg(&a.cu_q[b + 1]) - __ldg(&a.cu_q[b]), 0), a.max_q) : 1; };
    if (warp == 0) {
        int run = 0;
        for (int base = 0; base < a.B; base += 32) {
            const int b = base + lane;
            int cnt = 0;
            if (b < a.B) {
                const int L = min(max(a.seqused_k[b], 0), cap), n = queries(b);
                lenv[b] = L;
                if (n > 0) cnt = (L + kPageRows - 1) / kPageRows - q4_first_key(L, n, a.window) / kPageRows;
            }
            int incl = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (b < a.B) prefix[b] = run + incl - cnt;
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) prefix[a.B] = run;
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], HB);
        }
        fence_mbar_init();
    }
    __syncthreads();
    const int P = prefix[a.B];                       // pages of one head block
    const long long total = (long long)P * a.nhb;
    const long long ppc = (total + gridDim.x - 1) / gridDim.x;
    const long long p0 = min(total, blockIdx.x * ppc), p1 = min(total, p0 + ppc);
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b <= a.B; b += blockDim.x) a.meta[b] = prefix[b];
        if (threadIdx.x == 0) a.meta[a.B + 1] = (int)ppc;
    }
    auto seq_of = [&](int g) {                       // the largest b with prefix[b] <= g
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= g) lo = mid; else hi = mid;
        }
        return lo;
    };
    const int npages = (int)(p1 - p0);

    if (warp == HB * SUB) {
        // ------------------------------------------------------------ producer
        const uint64_t pol = policy_evict_first();
        int issued = 0;
        for (int base = 0; base < npages; base += 32) {
            int phys = 0, hb = 0;
            if (base + lane < npages) {
                const long long vg = p0 + base + lane;
                hb = (int)(vg / P);
                const int g = (int)(vg % P);
                const int b = seq_of(g);
                const int slot = g - prefix[b] + q4_first_key(lenv[b], queries(b), a.window) / kPageRows;
                phys = a.block_table[(long long)b * a.max_blocks + slot];
                if (phys < 0 || phys >= a.num_blocks) {
                    record_data_error(kErrDecPageRange);   // outside the cache: reported, page 0 read
                    phys = 0;
                }
            }
            const int cnt = min(32, npages - base);
            bool ok = true;
            for (int i = 0; i < cnt; ++i, ++issued) {
                const long long tile = (long long)__shfl_sync(0xffffffffu, phys, i) * a.Hkv +
                                       __shfl_sync(0xffffffffu, hb, i) * HB;
                const int st = issued % NS;
                ok = mbar_wait(&empty[st], ((issued / NS) & 1) ^ 1, kErrQ4Empty);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                uint8_t* dst = smem + st * SB;
                if (lane == 0) mbar_arrive_expect_tx(&full[st], SB);
                __syncwarp();
                if (lane < 2)
                    bulk_load(dst + lane * HB * C::TILE, (lane ? a.v_cache : a.k_cache) + tile * C::TILE, HB * C::TILE,
                              &full[st], pol);
                else if (lane < 4)
                    bulk_load(dst + 2 * HB * C::TILE + (lane - 2) * HB * C::META,
                              (lane == 3 ? a.v_meta : a.k_meta) + tile * (C::META / 2), HB * C::META, &full[st], pol);
            }
            if (!ok) break;
        }
        if (lane == 0) {
            for (int st = 0; st < NS && st < issued; ++st) {
                const int last = st + ((issued - 1 - st) / NS) * NS;
                mbar_wait_drain(&full[st], (last / NS) & 1, kErrQ4Full);
            }
        }
        return;
    }
    if (warp > HB * SUB) return;
    // ---------------------------------------------------------------- consumers
    const int h = warp / SUB, sub = warp % SUB;      // head of the block, this warp's share of its pages
    const int r8 = lane >> 2, t4 = lane & 3;
    const bool capped = a.softcap > 0.0f;
    uint32_t qb[NT][W][4];               // B fragments of Q^T: (dims e = 0, 4), (1, 5), (2, 6), (3, 7)
    float qs[NT][2][G];                  // sum of q over a group, in units of the raw score
    float kf[NT][2];                     // score in natural units = raw score * kf
    float acc[MT][NT][4];                // sum w c: tile rows r8 in units of 2^-24, r8 + 8 of 2^-20
    float zac[NT][2][G];                 // sum w zero, this lane's keys
    float m[NT][2], l[NT][2];            // maximum (log2 units) and sum (this lane's keys)
    float beta = 1.0f, cap_step = 0.0f;  // w = p step beta; steps below cap_step are in range
    int since = 0;
    auto load_q = [&](int b, int n, int hq0) {
        const long long tok0 = a.cu_q ? __ldg(&a.cu_q[b]) : b;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = nt * 8 + r8;
            const int tok = row / a.group;
            const bool live = tok < n;
            const __nv_bfloat16* qr = a.q + ((tok0 + (live ? tok : 0)) * a.Hq + hq0 + (live ? row % a.group : 0)) * D;
            uint4 x[W];
#pragma unroll
            for (int w = 0; w < W; ++w)
                x[w] = live ? __ldg(reinterpret_cast<const uint4*>(qr + 32 * w + 8 * t4)) : make_uint4(0, 0, 0, 0);
            float big = 0.0f, sum[G];
#pragma unroll
            for (int g = 0; g < G; ++g) sum[g] = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const uint32_t xs[4] = {x[w].x, x[w].y, x[w].z, x[w].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    big = fmaxf(big, fmaxf(fabsf(bf16_lo(xs[e])), fabsf(bf16_hi(xs[e]))));
                    sum[w / WG] += bf16_lo(xs[e]) + bf16_hi(xs[e]);
                }
            }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
#pragma unroll
            for (int g = 0; g < G; ++g) {
                sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
                sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
            }
            // the largest q of the row to [2^13, 2^14)
            const int ex = min(max((int)(__float_as_uint(big) >> 23) - 127, -100), 115);
            const float up = __uint_as_float((uint32_t)(127 + 13 - ex) << 23);
            const float down = __uint_as_float((uint32_t)(127 + 11 + ex) << 23);    // 2^24 / up
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float f[8] = {bf16_lo(x[w].x), bf16_hi(x[w].x), bf16_lo(x[w].y), bf16_hi(x[w].y),
                                    bf16_lo(x[w].z), bf16_hi(x[w].z), bf16_lo(x[w].w), bf16_hi(x[w].w)};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float s = e & 1 ? up * 0.0625f : up;
                    qb[nt][w][e] = pack_f16(f[e] * s, f[e + 4] * s);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int src = (2 * t4 + e) * 4;
                kf[nt][e] = __shfl_sync(0xffffffffu, down, src);
#pragma unroll
                for (int g = 0; g < G; ++g) qs[nt][e][g] = __shfl_sync(0xffffffffu, sum[g], src) / kf[nt][e];
            }
        }
    };
    auto reset = [&]() {
#pragma unroll
        for (int c = 0; c < MT; ++c)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[c][nt][0] = acc[c][nt][1] = acc[c][nt][2] = acc[c][nt][3] = 0.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nt][e] = -INFINITY;
                l[nt][e] = 0.0f;
#pragma unroll
                for (int g = 0; g < G; ++g) zac[nt][e][g] = 0.0f;
            }
        beta = 1.0f;
        cap_step = 0.0f;
        since = 0;
    };
    // takes sum w zero out of the accumulators
    auto recentre = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    float z = zac[nt][e][g];
                    z += __shfl_xor_sync(0xffffffffu, z, 4);
                    z += __shfl_xor_sync(0xffffffffu, z, 8);
                    z += __shfl_xor_sync(0xffffffffu, z, 16);
                    zac[nt][e][g] = 0.0f;
#pragma unroll
                    for (int c = g * (MT / G); c < (g + 1) * (MT / G); ++c) {
                        acc[c][nt][e] = fmaf(z, -5.9604644775390625e-8f, acc[c][nt][e]);             // 2^-24
                        acc[c][nt][2 + e] = fmaf(z, -9.5367431640625e-7f, acc[c][nt][2 + e]);        // 2^-20
                    }
                }
        since = 0;
    };
    // the end of a sequence or of the share: join the SUB warps of the head, write the partial
    auto flush_partial = [&](int vb, int n) {
        recentre();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float s = l[nt][e];
                s += __shfl_xor_sync(0xffffffffu, s, 4);
                s += __shfl_xor_sync(0xffffffffu, s, 8);
                s += __shfl_xor_sync(0xffffffffu, s, 16);
                l[nt][e] = s;
            }
        const float back = 1.0f / beta;              // a power of two
#pragma unroll
        for (int c = 0; c < MT; ++c)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[c][nt][e] = acc[c][nt][e] * (e < 2 ? 16777216.0f : 1048576.0f) * back;
        constexpr int FL = MT * NT * 4 + NT * 4;     // floats a lane exchanges
        const int slots = (SUB + 1) / 2;
        float* mine = mrg + (long long)h * slots * 32 * FL;
        int width = 1;
        while (width < SUB) width <<= 1;
        for (int st = width / 2; st > 0; st >>= 1) {
            if (sub >= st && sub < 2 * st) {
                float* x = mine + (sub - st) * 32 * FL + lane;
                int i = 0;
#pragma unroll
                for (int c = 0; c < MT; ++c)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[32 * i++] = acc[c][nt][e];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        x[32 * i++] = m[nt][e];
                        x[32 * i++] = l[nt][e];
                    }
            }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + h), "r"(32 * SUB) : "memory");
            if (sub < st && sub + st < SUB) {
                const float* x = mine + sub * 32 * FL + lane;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float m2 = x[32 * (MT * NT * 4 + (nt * 2 + e) * 2)];
                        const float l2 = x[32 * (MT * NT * 4 + (nt * 2 + e) * 2 + 1)];
                        const float mn = fmaxf(m[nt][e], m2);
                        const float f1 = mn == -INFINITY ? 1.0f : ex2(m[nt][e] - mn);
                        const float f2 = mn == -INFINITY ? 1.0f : ex2(m2 - mn);
                        m[nt][e] = mn;
                        l[nt][e] = l[nt][e] * f1 + l2 * f2;
#pragma unroll
                        for (int c = 0; c < MT; ++c) {
                            acc[c][nt][e] = acc[c][nt][e] * f1 + x[32 * ((c * NT + nt) * 4 + e)] * f2;
                            acc[c][nt][2 + e] = acc[c][nt][2 + e] * f1 + x[32 * ((c * NT + nt) * 4 + 2 + e)] * f2;
                        }
                    }
            }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + h), "r"(32 * SUB) : "memory");
        }
        if (sub != 0) return;
        const long long row0 = (((long long)blockIdx.x + vb) * HB + h) * (8 * NT);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = nt * 8 + 2 * t4 + e;
                if (row >= n * a.group) continue;
                const float s = l[nt][e];
                const float inv = s > 0.0f ? 1.0f / s : s == s ? 0.0f : s;    // a NaN stays one
                float* rp = a.o_part + (row0 + row) * D;
#pragma unroll
                for (int c = 0; c < MT; ++c) {
                    rp[16 * c + r8] = acc[c][nt][e] * inv;
                    rp[16 * c + 8 + r8] = acc[c][nt][2 + e] * inv;
                }
                if (r8 == 0)
                    a.lse_part[row0 + row] = s > 0.0f ? (m[nt][e] + log2f(s)) * kLn2 : s == s ? -INFINITY : s;
            }
    };
    bool ok = true;
    int i = sub;                                     // this warp's next page of the share
    for (int seg = 0; seg < npages;) {
        const long long vg = p0 + seg;
        const int hb = (int)(vg / P), g0 = (int)(vg % P);
        const int b = seq_of(g0);
        const int seg_end = (int)min((long long)npages, (long long)hb * P + prefix[b + 1] - p0);
        const int L = lenv[b], n = queries(b);
        // first key of the share's page `seg`
        const int key0 = (g0 - prefix[b] + q4_first_key(L, n, a.window) / kPageRows) * kPageRows;
        load_q(b, n, (hb * HB + h) * a.group);
        reset();
        // pages whose keys every query sees: key0 of the page in [all_lo, all_hi]
        const int all_hi = (a.causal ? L - n : L - 1) - (kPageRows - 1);
        const int all_lo = a.window >= 0 ? L - 1 - a.window : 0;
        for (; i < seg_end; i += SUB) {
            const int st = i % NS;
            if (ok) {
                ok = mbar_wait(&full[st], (i / NS) & 1, kErrQ4Full);
                ok = __all_sync(0xffffffffu, ok);
            }
            if (ok) {
                const int tok0 = key0 + (i - seg) * kPageRows;
                const uint8_t* stage = smem + st * SB;
                const uint32_t* kt = reinterpret_cast<const uint32_t*>(stage + h * C::TILE) + r8 * (D / 8) + t4 * W;
                const uint32_t* vt = reinterpret_cast<const uint32_t*>(stage + (HB + h) * C::TILE) + lane * W;
                const uint16_t* km = reinterpret_cast<const uint16_t*>(stage + 2 * HB * C::TILE + h * C::META) + r8 * G;
                const uint16_t* vm = km + HB * C::META / 2;
                uint32_t k0[W], k1[W];
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    k0[w] = kt[w];
                    k1[w] = kt[D + w];
                }
                float sc[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.0f;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    float raw[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) raw[nt][0] = raw[nt][1] = raw[nt][2] = raw[nt][3] = 0.0f;
#pragma unroll
                    for (int w = g * WG; w < (g + 1) * WG; ++w) {
                        const uint32_t lo[4] = {k0[w] & 0x000f000fu, k1[w] & 0x000f000fu, k0[w] & 0x00f000f0u,
                                                k1[w] & 0x00f000f0u};
                        const uint32_t s0 = k0[w] >> 8, s1 = k1[w] >> 8;
                        const uint32_t hi[4] = {s0 & 0x000f000fu, s1 & 0x000f000fu, s0 & 0x00f000f0u, s1 & 0x00f000f0u};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16_16816(raw[nt], lo, qb[nt][w][0], qb[nt][w][1]);
                            mma_f16_16816(raw[nt], hi, qb[nt][w][2], qb[nt][w][3]);
                        }
                    }
                    const uint32_t m0 = km[g], m1 = km[8 * G + g];
                    const float s0 = q4_step(m0), s1 = q4_step(m1), z0 = -q4_zero(m0), z1 = -q4_zero(m1);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            sc[nt][e] = fmaf(fmaf(z0, qs[nt][e][g], raw[nt][e]), s0, sc[nt][e]);
                            sc[nt][2 + e] = fmaf(fmaf(z1, qs[nt][e][g], raw[nt][2 + e]), s1, sc[nt][2 + e]);
                        }
                }
                // to log2 units
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = sc[nt][e] * (kf[nt][e & 1] * a.scale);
                        if (capped) x = a.softcap * tanh_ex2(x / a.softcap);
                        sc[nt][e] = x * kLog2e;
                    }
                float vs[2][G], vz[2][G];
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const uint32_t m0 = vm[g], m1 = vm[8 * G + g];
                    vs[0][g] = q4_step(m0), vs[1][g] = q4_step(m1), vz[0][g] = q4_zero(m0), vz[1][g] = q4_zero(m1);
                }
                if (tok0 > all_hi || tok0 < all_lo) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int key = tok0 + r8 + 8 * y;
                        if (key >= L) {                // not data of the sequence
#pragma unroll
                            for (int g = 0; g < G; ++g) vs[y][g] = vz[y][g] = 0.0f;
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int tok = (nt * 8 + 2 * t4 + e) / a.group;
                                const int last = a.causal ? L - n + tok : L - 1;
                                if (key > last || key >= L || (a.window >= 0 && key < last - a.window))
                                    sc[nt][2 * y + e] = -INFINITY;
                            }
                    }
                }
                // does a score exceed its row's maximum by the slack, or a step the range?
                bool over = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        over = over || fmaxf(sc[nt][e], sc[nt][2 + e]) > m[nt][e] + kQ4Slack;
                float top = 0.0f;
#pragma unroll
                for (int g = 0; g < G; ++g) top = fmaxf(top, fmaxf(vs[0][g], vs[1][g]));
                over = over || (top >= cap_step && top > 0.0f && top < INFINITY);
                if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    float resc = 1.0f;
                    if (top >= cap_step && top > 0.0f && top < INFINITY) {
                        // 2^ex <= top < 2^(ex + 1): beta puts it below 2^7
                        const int ex = (int)(__float_as_uint(top) >> 23) - 127;
                        const float nb = __uint_as_float((uint32_t)(127 + 6 - ex) << 23);
                        cap_step = ex < 127 ? __uint_as_float((uint32_t)(127 + 1 + ex) << 23) : INFINITY;
                        resc = nb / beta;
                        beta = nb;
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float mx = fmaxf(sc[nt][e], sc[nt][2 + e]);
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                            const float mn = fmaxf(m[nt][e], mx);
                            const float al = mn == -INFINITY ? 1.0f : ex2(m[nt][e] - mn);
                            m[nt][e] = mn;
                            l[nt][e] *= al;
                            const float f = al * resc;
#pragma unroll
                            for (int g = 0; g < G; ++g) zac[nt][e][g] *= f;
#pragma unroll
                            for (int c = 0; c < MT; ++c) {
                                acc[c][nt][e] *= f;
                                acc[c][nt][2 + e] *= f;
                            }
                        }
                }
                float p[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float mu = m[nt][e] == -INFINITY ? 0.0f : m[nt][e];
                        p[nt][e] = ex2(sc[nt][e] - mu);
                        p[nt][2 + e] = ex2(sc[nt][2 + e] - mu);
                        l[nt][e] += p[nt][e] + p[nt][2 + e];
                    }
                uint32_t v0[W], v1[W];
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    v0[w] = vt[w];
                    v1[w] = vt[32 * W + w];
                }
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float w0 = vs[0][g] * beta, w1 = vs[1][g] * beta;
                    uint32_t pb[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float x0 = p[nt][0] * w0, x1 = p[nt][1] * w0, x2 = p[nt][2] * w1, x3 = p[nt][3] * w1;
                        zac[nt][0][g] = fmaf(x0, vz[0][g], fmaf(x2, vz[1][g], zac[nt][0][g]));
                        zac[nt][1][g] = fmaf(x1, vz[0][g], fmaf(x3, vz[1][g], zac[nt][1][g]));
                        pb[nt][0] = movmatrix_trans(pack_f16(x0, x1));
                        pb[nt][1] = movmatrix_trans(pack_f16(x2, x3));
                    }
#pragma unroll
                    for (int w = g * WG; w < (g + 1) * WG; ++w) {
                        const uint32_t lo[4] = {v0[w] & 0x000f000fu, v0[w] & 0x00f000f0u, v1[w] & 0x000f000fu,
                                                v1[w] & 0x00f000f0u};
                        const uint32_t s0 = v0[w] >> 8, s1 = v1[w] >> 8;
                        const uint32_t hi[4] = {s0 & 0x000f000fu, s0 & 0x00f000f0u, s1 & 0x000f000fu, s1 & 0x00f000f0u};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16_16816(acc[2 * w][nt], lo, pb[nt][0], pb[nt][1]);
                            mma_f16_16816(acc[2 * w + 1][nt], hi, pb[nt][0], pb[nt][1]);
                        }
                    }
                }
                if (++since == kQ4Recentre) recentre();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
        }
        flush_partial(hb * a.B + b, n);
        seg = seg_end;
    }
}

// Joins the partials: a warp per output row.  The partials of sequence b and head
// block hb sit in slots c + hb B + b for the CTAs c whose shares covered it.
template <int D, int NT>
__global__ void __launch_bounds__(256) q4_combine_kernel(const Q4AttnArgs a) {
    constexpr int V = D / 32;            // columns of a lane
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int per = a.max_q * a.Hq;      // rows of a sequence
    if (w >= (long long)a.B * per) return;
    const int b = (int)(w / per), tok = (int)(w % per) / a.Hq, hq = (int)(w % per) % a.Hq;
    const long long q0 = a.cu_q ? __ldg(&a.cu_q[b]) : b;
    if (a.cu_q && tok >= __ldg(&a.cu_q[b + 1]) - q0) return;
    const int hkv = hq / a.group, hb = hkv / a.HB, h = hkv % a.HB;
    const int row = tok * a.group + hq % a.group;
    const long long P = a.meta[a.B], ppc = max(a.meta[a.B + 1], 1);
    const long long pb = hb * P + a.meta[b], pe = hb * P + a.meta[b + 1];
    const long long c0 = pb / ppc;
    const int ns = pe > pb ? (int)((pe - 1) / ppc - c0 + 1) : 0;
    const long long first = ((c0 + (long long)hb * a.B + b) * a.HB + h) * (8 * NT) + row;
    const long long step = (long long)a.HB * 8 * NT;
    float M = -INFINITY;
    bool nan = false;
    for (int s = lane; s < ns; s += 32) {
        const float x = a.lse_part[first + s * step];
        nan = nan || x != x;
        M = fmaxf(M, x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    nan = __any_sync(0xffffffffu, nan);
    float sum = 0.0f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.0f;
    if (M != -INFINITY) {
#pragma unroll 4
        for (int s = 0; s < ns; ++s) {
            const float f = ex2((a.lse_part[first + s * step] - M) * kLog2e);
            sum += f;
            const float* src = a.o_part + (first + s * step) * D + lane * V;
            float x[V];
            if constexpr (V == 4) {
                const float4 t = *reinterpret_cast<const float4*>(src);
                x[0] = t.x, x[1] = t.y, x[2] = t.z, x[3] = t.w;
            } else {
                const float2 t = *reinterpret_cast<const float2*>(src);
                x[0] = t.x, x[1] = t.y;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = fmaf(f, x[v], acc[v]);
        }
    }
    const float inv = nan ? NAN : sum > 0.0f ? 1.0f / sum : 0.0f;
    __nv_bfloat16* dst = a.o + ((q0 + tok) * a.Hq + hq) * D + lane * V;
    if constexpr (V == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16(acc[0] * inv, acc[1] * inv);
    if (a.lse && lane == 0)
        a.lse[a.cu_q ? (long long)hq * a.total_q + q0 + tok : (long long)b * a.Hq + hq] =
            nan ? NAN : sum > 0.0f ? M + logf(sum) : -INFINITY;
}

}  // namespace attn
