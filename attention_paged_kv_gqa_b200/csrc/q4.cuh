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

#include <type_traits>

#include "append.cuh"
#include "decode.cuh"
#include "rope.cuh"

namespace attn {

enum : int { kErrQ4Rows = 531, kErrQ4Queries = 532, kErrQ4Full = 541, kErrQ4Empty = 542 };

// ---------------------------------------------------------------- quantiser
struct Q4Group {
    float inv;               // 1 / step, or 0
    float zero;
    uint32_t meta;
};

// Of two bf16 pairs the smaller and the larger elements; a NaN wins.
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// nearest(x / step) + kQ4Magic, for |x / step| <= 16.  x has 8 significant bits and
// step 4, so x / step lies either on a half-integer or further than 2^-12 from one: the
// sum with 768, rounded to 2^-14, makes ties exact again whatever the rounding of inv,
// and the second sum rounds them to even.
constexpr float kQ4Magic = 12582912.0f;     // 1.5 * 2^23
__device__ __forceinline__ float q4_nearest(float x, float inv) {
    return __fadd_rn(__fmaf_rn(x, inv, 768.0f), kQ4Magic - 768.0f);
}

// Step and zero of a group from its lo <= 0 and hi >= 0 (NaN where it has one).  width / 15
// up to 4 significant bits without a division: a candidate from a product that is a little
// low, and one notch more where 15 of them still fall short.
__device__ __forceinline__ Q4Group q4_group(float lo, float hi) {
    Q4Group g;
    const float width = __fsub_rn(hi, lo);
    const float s = __fmul_rn(width, 0.06666663f);   // 1 / 15 less 2^-21 of it
    uint32_t bits = (__float_as_uint(s) + 0xfffffu) & 0xfff00000u;
    if (__fmaf_rn(-15.0f, __uint_as_float(bits), width) > 0.0f) bits += 0x100000u;
    const bool live = bits >= 0x0d800000u && width < INFINITY;       // 2^-100; a NaN is not less
    g.inv = live ? rcp_approx(__uint_as_float(bits)) : 0.0f;         // (see q4_nearest)
    const float z = live ? q4_nearest(-lo, g.inv) : kQ4Magic;
    g.zero = __fsub_rn(z, kQ4Magic);
    g.meta = live ? (bits >> 16) | (__float_as_uint(z) & 15u) : width < INFINITY ? 0u : 0x7fc0u;
    return g;
}

// The codes of eight values, value i in nibble i.  No code is below 0: the smallest value's
// quotient rounds to minus zero.  The nibbles are put together as numbers (16-bit halves
// are exact), and the sum with 2^23 leaves a half in the low bits.  (A NaN gives some code;
// its group's step is NaN.)
__device__ __forceinline__ uint32_t q4_codes(const float2 (&x)[4], const Q4Group& g) {
    float c[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 n = fadd2(ffma2(x[i], make_float2(g.inv, g.inv), make_float2(768.0f, 768.0f)),
                               make_float2(kQ4Magic - 768.0f, kQ4Magic - 768.0f));
        const float2 v = fadd2(n, make_float2(g.zero - kQ4Magic, g.zero - kQ4Magic));
        c[2 * i] = fminf(v.x, 15.0f);
        c[2 * i + 1] = fminf(v.y, 15.0f);
    }
    const float lo = fmaf(fmaf(fmaf(c[3], 16.0f, c[2]), 16.0f, c[1]), 16.0f, c[0]) + 8388608.0f;
    const float hi = fmaf(fmaf(fmaf(c[7], 16.0f, c[6]), 16.0f, c[5]), 16.0f, c[4]) + 8388608.0f;
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410);
}

__device__ __forceinline__ float q4_step(uint32_t meta) { return __uint_as_float((meta << 16) & 0xfff00000u); }
// (as a float whose significand ends in the integer: a conversion would go to the
// quarter-rate unit that the exponentials need)
__device__ __forceinline__ float q4_zero(uint32_t meta) { return __uint_as_float((meta & 15u) | 0x4b000000u) - 8388608.0f; }

// ---------------------------------------------------------------- append
// New tokens into 4-bit pages: q turned into q_out (bf16), k turned, rounded to
// bf16 as attn_rope would, and quantised, v quantised.  A warp takes 1 / parts of
// one token's heads.  For k and v a lane holds eight consecutive columns (the
// partner columns of a half-split pair come from another lane), a group's
// smallest and largest are found across its group / 8 lanes, a K word is one
// lane's eight codes, and the V pieces are regrouped among the four lanes that
// hold the dims 32 u .. 32 u + 31.
// Bound by HBM and, close behind, by the issue of instructions (55 % of the slots,
// the logic pipe 47 %): 16955 tokens of 32 + 8 + 8 heads of 128, 70 to 74 us, of
// which the bytes take 57.  It was 106: the division by the step became a product
// with its approximate reciprocal whose ties are made exact (see q4_nearest), the
// minimum and the negated maximum of a group travel in one register, and codes
// are put together by fused multiply-adds.  Four passes' loads in flight (two:
// 4 us more); 64 or 256 threads a block: 12 and 18 us more.
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
    const int nrot = a.r.table ? a.r.rot / 16 : 0;
    NewToken nt;
    {
        const int u = lane % U, first = part * HP + lane / U;
        const bool turns = u < nrot;
        int ca, cb;
        rope_columns(a.r, u, &ca, &cb);
        RopeRows<D, 4> q;
        q.start(a.q, t, a.Hq, first, a.parts, ca, cb);     // in flight while the page and the angles are looked up
        nt = find_new_token(a, (int)t, lane);
        if (nt.b < 0) return;
        RopeAngles g;
        if (turns && a.q.p) g = rope_angles(a.r, t, a.total_new, u, nt.pos);
        q.template finish<kCacheBf16>(static_cast<uint8_t*>(a.q_out) + ((t * a.Hq + first) * D + ca) * 2,
                                      2LL * a.parts * HP * D, turns, g, a.r.interleaved, 1.0f);
    }
    if (nt.page < 0) return;
    const int v = lane % LPH;                      // columns 8 v .. 8 v + 7
    const int row = nt.pos % kPageRows;
    // This lane's angles: of eight pairs (columns 8 v of one half), or of pairs 4 v .. 4 v + 3
    // (interleaved: the first or second half of the eight from 8 (v / 2)).
    const bool turns = v < 2 * nrot, front = v < nrot;
    RopeAngles g;
    if (turns) {
        g = rope_angles(a.r, t, a.total_new, a.r.interleaved ? v / 2 : front ? v : v - nrot, nt.pos);
        if (a.r.interleaved && (v & 1)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) g.c[e] = g.c[2 + e], g.s[e] = g.s[2 + e], g.n[e] = g.n[2 + e];
        }
        if (!a.r.interleaved && front) {           // the first half's column: x1 c - x2 s; the second's: x2 c + x1 s
#pragma unroll
            for (int e = 0; e < 4; ++e) g.s[e] = g.n[e];
        }
    }
    constexpr int N = 4;                           // passes whose loads are in flight together
    auto rows = [&](const HeadRows& x, uint8_t* cache, uint16_t* metas, auto is_k) {
        constexpr bool K = decltype(is_k)::value;
        int h = part * HV + lane / LPH;
        const int apart = a.parts * HV;
        const __nv_bfloat16* src = x.p + t * x.row + h * x.head + 8 * v;
        const long long pitch = apart * x.head;
        const long long tile0 = nt.page * a.Hkv;
        // the lane's word of a K row, or its pieces r = 2 j and 2 j + 1 of a V tile
        uint8_t* code = cache + (tile0 + h) * (kPageRows * D / 2) +
                        (K ? row * (D / 2) + ((v % 4) * W + v / 4) * 4
                           : ((((row / 8) * 8 + 2 * (lane & 3)) * 4 + row % 8 / 2) * W + v / 4) * 4 + row % 2 * 2);
        uint16_t* meta = metas + ((tile0 + h) * kPageRows + row) * G + v / (GS / 8);
        // (the number of passes is the warp's, so that all lanes shuffle)
        for (int h0 = part * HV; h0 < a.Hkv; h0 += N * apart) {
            uint4 raw[N];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                raw[n] = make_uint4(0, 0, 0, 0);
                if (h + n * apart < a.Hkv) raw[n] = *reinterpret_cast<const uint4*>(src + n * pitch);
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if (h0 + n * apart >= a.Hkv) break;
                const bool live = h + n * apart < a.Hkv;
                uint32_t wd[4] = {raw[n].x, raw[n].y, raw[n].z, raw[n].w};
                if (K && nrot) {
                    if (a.r.interleaved) {
                        if (turns) {
#pragma unroll
                            for (int e = 0; e < 4; e += 2) {
                                float2 x1 = make_float2(bf16_lo(wd[e]), bf16_lo(wd[e + 1]));
                                float2 x2 = make_float2(bf16_hi(wd[e]), bf16_hi(wd[e + 1]));
                                rope_turn(x1, x2, g, e / 2);
                                wd[e] = pack_bf16(x1.x, x2.x);
                                wd[e + 1] = pack_bf16(x1.y, x2.y);
                            }
                        }
                    } else {
                        // columns 8 v .. of the first half turn with those 8 (v + nrot) .. of the second
                        const int mate = lane + (!turns ? 0 : front ? nrot : -nrot);
                        uint32_t pw[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) pw[e] = __shfl_sync(0xffffffffu, wd[e], mate);
                        if (turns) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 y = fadd2(fmul2(bf16_pair(wd[e]), g.c[e]), fmul2(bf16_pair(pw[e]), g.s[e]));
                                wd[e] = pack_bf16(y.x, y.y);
                            }
                        }
                    }
                }
                // the group's smallest and, negated, largest value side by side, across its lanes
                const uint32_t lo2 = min_bf16x2(min_bf16x2(wd[0], wd[1]), min_bf16x2(wd[2], wd[3]));
                const uint32_t hi2 = max_bf16x2(max_bf16x2(wd[0], wd[1]), max_bf16x2(wd[2], wd[3])) ^ 0x80008000u;
                uint32_t ends = min_bf16x2(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));
                ends = min_bf16x2(ends, 0u);           // (a group's range includes zero)
#pragma unroll
                for (int o = 1; o < GS / 8; o <<= 1) ends = min_bf16x2(ends, __shfl_xor_sync(0xffffffffu, ends, o));
                const Q4Group q = q4_group(bf16_lo(ends), -bf16_hi(ends));
                const float2 f[4] = {bf16_pair(wd[0]), bf16_pair(wd[1]), bf16_pair(wd[2]), bf16_pair(wd[3])};
                const uint32_t codes = q4_codes(f, q);
                uint8_t* to = code + (long long)n * apart * (kPageRows * D / 2);
                if (K) {
                    if (live) *reinterpret_cast<uint32_t*>(to) = codes;
                } else {
                    // lane j of a quad holds nibble r of dims 32 u + 8 j + r; it takes byte j of the
                    // quad's four words
                    const int j = lane & 3;
                    uint32_t b[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) b[e] = __shfl_sync(0xffffffffu, codes, (lane & ~3) + e);
                    const uint32_t sel = j | (4 + j) << 4;
                    const uint32_t all = __byte_perm(__byte_perm(b[0], b[1], sel), __byte_perm(b[2], b[3], sel), 0x5410);
                    const uint32_t e4 = all & 0x0f0f0f0fu, o4 = (all >> 4) & 0x0f0f0f0fu;
                    const uint32_t even = (e4 | e4 >> 4) & 0x00ff00ffu, odd = (o4 | o4 >> 4) & 0x00ff00ffu;
                    if (live) {
                        *reinterpret_cast<uint16_t*>(to) = (uint16_t)(even | even >> 8);
                        *reinterpret_cast<uint16_t*>(to + 16 * W) = (uint16_t)(odd | odd >> 8);
                    }
                }
                if (live && v % (GS / 8) == 0) meta[(long long)n * apart * (kPageRows * G)] = (uint16_t)q.meta;
            }
            h += N * apart;
            src += N * pitch;
            code += (long long)N * apart * (kPageRows * D / 2);
            meta += (long long)N * apart * (kPageRows * G);
        }
    };
    rows(a.k, a.k_cache, a.k_meta, std::true_type());
    rows(a.v, a.v_cache, a.v_meta, std::false_type());
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

// N consecutive words (N = 2 or 4, aligned).
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        w[0] = x.x, w[1] = x.y;
    }
}

// The N metas (1, 2 or 4) of a token.
template <int N>
__device__ __forceinline__ void load_metas(const uint8_t* p, uint32_t (&m)[N]) {
    if constexpr (N == 4) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        m[0] = x.x & 0xffffu, m[1] = x.x >> 16, m[2] = x.y & 0xffffu, m[3] = x.y >> 16;
    } else if constexpr (N == 2) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(p);
        m[0] = x & 0xffffu, m[1] = x >> 16;
    } else {
        m[0] = *reinterpret_cast<const uint16_t*>(p);
    }
}

// The codes at the low nibbles of w's halves as step * (code - zero) in bf16: 128 + code has
// 8 bits, its difference with 128 + zero is exact, and so is the product.
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, uint32_t step2, uint32_t zero2) {
    uint32_t r = (w & 0x000f000fu) | 0x43004300u;
    asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(zero2));
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(step2));
    return r;
}
// Steps, and 128 + zeros, of two metas (low and high half) in bf16.
__device__ __forceinline__ uint32_t q4_steps(uint32_t m2) { return m2 & 0xfff0fff0u; }
__device__ __forceinline__ uint32_t q4_zeros(uint32_t m2) { return (m2 & 0x000f000fu) | 0x43004300u; }

// The rows of packed K and V from 4-bit pages: a warp takes the K and V tile of
// one page and head.  The values are bf16 numbers, so nothing is lost.  HBM bound
// by what it writes (4 bytes for each byte read): 59000 tokens of 8 heads of 128,
// 55 us, 5.4 TB/s (65 when a lane wrote 16 bytes of V 64 bytes apart from the
// next lane's); the arithmetic is two packed bf16 operations for two values.  A
// warp that takes several looks its next page up while it unpacks this one.
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
        // (rows are held at 2^31 - 1, past any output: the lengths' sum may be more)
        constexpr uint32_t kMost = 0x7fffffffu;
        int run_p = 0;
        uint32_t run_r = 0;
        for (int base = 0; base < a.B; base += 32) {
            const int b = base + lane;
            int n = 0, np = 0, s0 = 0;
            if (b < a.B) {
                if (a.starts) s0 = max(a.starts[b], 0);
                n = a.cu ? a.cu[b + 1] - a.cu[b] : a.lens[b];
                n = min(max(n, 0), max(a.max_blocks * kPageRows - s0, 0));
                np = n > 0 ? (s0 + n - 1) / kPageRows - s0 / kPageRows + 1 : 0;
            }
            int ip = np;
            uint32_t ir = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, ip, o);
                const uint32_t y = __shfl_up_sync(0xffffffffu, ir, o);
                if (lane >= o) ip += x, ir = min(ir + y, kMost);
            }
            const uint32_t before = __shfl_up_sync(0xffffffffu, ir, 1);
            if (b < a.B) {
                pages[b] = run_p + ip - np;
                rows[b] = a.cu ? a.cu[b] : (int)min(run_r + (lane ? before : 0u), kMost);
            }
            run_p += __shfl_sync(0xffffffffu, ip, 31);
            run_r = min(run_r + __shfl_sync(0xffffffffu, ir, 31), kMost);
        }
        if (lane == 0) {
            pages[a.B] = run_p;
            rows[a.B] = a.cu ? a.cu[a.B] : (int)run_r;
            if (blockIdx.x == 0 && rows[a.B] > a.total) record_data_error(kErrQ4Rows);
        }
    }
    __syncthreads();
    if (a.cu_out && blockIdx.x == 0)
        for (int b = threadIdx.x; b <= a.B; b += blockDim.x) a.cu_out[b] = min(rows[b], a.total);
    const long long items = (long long)pages[a.B] * a.Hkv;
    const int warps = gridDim.x * (blockDim.x >> 5);
    struct Item {
        int h, b, s0, slot, n, page;
    };
    auto look_up = [&](long long it) {
        Item x;
        const int g = (int)(it / a.Hkv);
        x.h = (int)(it - (long long)g * a.Hkv);
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pages[mid] <= g) lo = mid; else hi = mid;
        }
        x.b = lo;
        x.s0 = a.starts ? max(__ldg(&a.starts[lo]), 0) : 0;
        x.slot = x.s0 / kPageRows + (g - pages[lo]);
        x.n = min(a.cu ? __ldg(&a.cu[lo + 1]) - rows[lo] : a.lens[lo], a.max_blocks * kPageRows - x.s0);
        x.page = __ldg(&a.block_table[(long long)lo * a.max_blocks + x.slot]);
        return x;
    };
    long long it = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    Item next;
    if (it < items) next = look_up(it);
    for (; it < items; it += warps) {
        const Item x = next;
        if (it + warps < items) next = look_up(it + warps);      // in flight beside this one
        const int h = x.h, b = x.b, s0 = x.s0, slot = x.slot, n = x.n;
        // (all further rows lie behind the output's last: lengths past `total` cost no time)
        if (!a.cu && (long long)rows[b] + slot * kPageRows >= a.total) break;
        int page = x.page;
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
        // K: 4 units (16-byte piece c) of W words in each of the 16 rows; V: lane (token pair
        // p = 4 a + c, nibble j) takes its two tokens' dims 32 u + 8 j + r, so that four lanes
        // write 64 bytes of a row side by side.  All of it is loaded first.
        const uint32_t* kt = reinterpret_cast<const uint32_t*>(a.k_cache + tile * (kPageRows * D / 2));
        const uint32_t* vt = reinterpret_cast<const uint32_t*>(a.v_cache + tile * (kPageRows * D / 2));
        const int j = lane % 4, p = lane / 4;
        uint32_t kw[2][W], kmeta[2][G], vw[8][W], vm0[G], vm1[G];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            load_words<W>(reinterpret_cast<const uint8_t*>(kt + (lane + 32 * i) * W), kw[i]);
            load_metas<G>(reinterpret_cast<const uint8_t*>(km + (lane + 32 * i) / 4 * G), kmeta[i]);
        }
#pragma unroll
        for (int r = 0; r < 8; ++r)
            load_words<W>(reinterpret_cast<const uint8_t*>(vt + (((p / 4) * 8 + r) * 4 + p % 4) * W), vw[r]);
        load_metas<G>(reinterpret_cast<const uint8_t*>(vm + 2 * p * G), vm0);
        load_metas<G>(reinterpret_cast<const uint8_t*>(vm + (2 * p + 1) * G), vm1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int y = (lane + 32 * i) / 4, c = lane % 4;
            const long long r = out_row(y);
            if (r < 0) continue;
            __nv_bfloat16* dst = a.k_out + (r * a.Hkv + h) * D + 8 * c;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const uint32_t m2 = kmeta[i][32 * w / GS] * 0x10001u, st = q4_steps(m2), z = q4_zeros(m2);
                uint32_t x[4];                     // dims e and e + 4
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = q4_pair(kw[i][w] >> (4 * e), st, z);
                *reinterpret_cast<uint4*>(dst + 32 * w) =
                    make_uint4(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410), __byte_perm(x[0], x[1], 0x7632),
                               __byte_perm(x[2], x[3], 0x7632));
            }
        }
        const long long r0 = out_row(2 * p), r1 = out_row(2 * p + 1);
#pragma unroll
        for (int u = 0; u < W; ++u) {
            const uint32_t m2 = vm0[32 * u / GS] | vm1[32 * u / GS] << 16, st = q4_steps(m2), z = q4_zeros(m2);
            uint32_t x[8];                         // dim 32 u + 8 j + r of both tokens
#pragma unroll
            for (int r = 0; r < 8; ++r) x[r] = q4_pair(vw[r][u] >> (4 * j), st, z);
            if (r0 >= 0)
                *reinterpret_cast<uint4*>(a.v_out + (r0 * a.Hkv + h) * D + 32 * u + 8 * j) =
                    make_uint4(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410), __byte_perm(x[4], x[5], 0x5410),
                               __byte_perm(x[6], x[7], 0x5410));
            if (r1 >= 0)
                *reinterpret_cast<uint4*>(a.v_out + (r1 * a.Hkv + h) * D + 32 * u + 8 * j) =
                    make_uint4(__byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632), __byte_perm(x[4], x[5], 0x7632),
                               __byte_perm(x[6], x[7], 0x7632));
        }
    }
}

// ---------------------------------------------------------------- attention
// A few query rows per sequence (tokens x query heads of a KV head) over 4-bit pages: the
// page stream of decode.cuh with another consumer.
//
// Split.  The pages of the batch, for one block of HB KV heads after another, are cut into
// one contiguous share of equal cost per CTA, a change of sequence counted as kQ4Switch
// pages.  A page's HB tiles of K, V and their metas are four contiguous runs, which three
// producer warps fetch by bulk copies into a ring of stages; a fourth prepares the queries
// of the share's next sequence.  The query rows are in RT tiles of 8 NT, and of the SUB warps
// of a KV head and tile each takes every SUB-th page, two at a time (with NT = 2 one, whose
// two tiles' chains run side by side), and keeps an online softmax of its own.  Where a
// sequence or the share ends they are joined through shared memory, in a fixed order, and
// the partial (O normalised, LSE) goes to slot CTA + sequence for the combine kernel, which
// follows as a programmatic dependent.  No atomics: the result does not depend on timing.
//
// Score: s = step (q . c - zero sum q), c the codes: the code, shifted to the
// low or second nibble of a 16-bit half, IS the f16 number c 2^-24 or c 2^-20
// (subnormal, exact), so a K word becomes four A registers with four ANDs and a
// shift.  q is exact in f16 after a power of two per row, divided by 16 for the
// dims that meet second nibbles.  The output: O = sum_j w_j c_j - sum_j w_j zero_j
// with w_j = p_j step_j, again on the codes as they are; w is rounded to f16 (what
// the MMA takes) after a scale per row and group that follows the largest w, not the
// largest step, which may belong to a key of no weight or to another group's columns;
// everything else is held in fp32.  Both sums take the rounded w, so that its error,
// at most 2^-11 of each weight, meets the value c - zero and not the code c: the
// weights of keys of equal scores all err alike (with the sum of the zeros over the
// unrounded w the output over 113000 such keys was off by up to 7 %).
// Groups smaller than the head repeat the two sums per group.
// The first sum is far larger than the difference where p is spread over many
// keys, and the tensor cores truncate when they add; every 16 pages the second
// sum is therefore taken out of the accumulators, which stay near their final size
// (every 4 or every 64 pages take the same time, within 2 %).  The running maximum of
// the scores, and that of the weights, moves only when one exceeds it by 2^8, which a
// page shows by one vote (the second case below takes 91 us if they move with every
// larger one, against 77).
//
// Bound.  Bytes would take 20 us for 32 sequences of 4100 keys (32 + 8 heads of 128, groups
// of 128) and 35 us for 3 of 65000 (64 + 8, groups of 32).  With cold caches, as are all
// figures here that do not say otherwise, the calls take 45 to 46 and 76 to 79 us; in a row,
// each beginning while the one before ends, 39 and 70.  About 14 us are fixed: 4 to 5 until
// the first page is there (launch, lengths, table, page), 1.5 to 2 for the join, 4 to 6 for
// the combine kernel.  A page of four heads then costs 0.26 us of a CTA's time, where its
// bytes take 0.19: taking the codes apart keeps the logic pipe at 49 and 57 % of its rate
// over the whole call, and the chain from score to weight does not leave it busy throughout.
// The tensor pipe is at 21 and 18 %, DRAM at half.  The scales per row and group cost the
// second case 2 us, the sum of the zeros over rounded weights another 2 (each 1 or less in
// the first case).  A change of sequence costs 3 to 4 us (kQ4Switch: with 0, 6 and 20 in
// place of 13 the first case takes 50, 48 and 46 us against 46, 600 sequences of 100 keys
// 118, 97 and 88 against 90).
// Tried and slower: MMAs on e4m3 codes (the warp form is emulated: 1.6 times), shifts on the
// multiplier, the next pages' scores ahead of this pair's softmax (with twelve warps 49 us
// against 45, at the time).
constexpr float kQ4Slack = 8.0f;         // p <= 2^8 between moves of the maximum, and w <= 2^8 of its own
constexpr float kQ4Top = 7.0f;           // the largest w seen is 2^7 (one of 2^15 still fits)
constexpr float kQ4Range = 111.0f;       // w's maximum is held at 2^-111 of p's or more: p scale <= 2^126
constexpr int kQ4Recentre = 16;          // pages
constexpr int kQ4Producers = 4;          // warps that fetch K, V, their metas, the queries
constexpr int kQ4Scan = 4;               // sequences that a lane looks up at once
constexpr int kQ4Rows = 128;             // query rows of a KV head at most
// A tile is 8 NT rows, NT = 1 where that holds them all, or 2; a CTA has this many consumer warps.
__host__ __device__ constexpr int q4_warps(int NT) { return NT == 1 ? 12 : 8; }
constexpr int kQ4Switch = 13;            // pages that a change of sequence costs a CTA (for equal shares)
constexpr float kQ4NoMax = -3.0e38f;     // the maximum before the first key (finite: differences with it stay numbers)

struct Q4AttnArgs {
    int B, Hq, Hkv, group;
    int HB, RT, SUB, nhb;    // KV heads of a block, row tiles, warps of a head and tile, blocks
    const __nv_bfloat16* q;  // rows of queries [..][Hq][D]
    const int* cu_q;         // [B + 1], or null: one query per sequence
    int max_q;               // query tokens a sequence may have (group * max_q <= 8 NT RT)
    int total_q;
    int total_k;             // < 0, or what the caller takes the lengths' sum to be at most
    const uint8_t *k_cache, *v_cache;
    const uint16_t *k_meta, *v_meta;
    const int* block_table;
    int max_blocks, num_blocks;
    const int* seqused_k;
    float scale;
    int causal;              // 0: every query sees every key
    int window;              // < 0: none
    float softcap;           // 0: none
    int rows;                // query rows of a KV head: group * max_q
    float* o_part;           // [slots][HB][rows][D]
    float* lse_part;         // [slots][HB][rows]
    int2* table;             // [B + 1] pages and the cost before each sequence, for the combine kernel; or null
    int grid;                // CTAs
    int nstages;
    int wpr;                 // combine: warps of a row (1, 2, 4 or 8)
    __nv_bfloat16* o;        // as q
    float* lse;              // [Hq][total_q], or [B][Hq] (cu_q null); or null
};

template <int D, int GS, int NT>
struct Q4Cfg {
    static constexpr int TILE = kPageRows * D / 2;              // bytes of a head's K or V tile
    static constexpr int META = kPageRows * (D / GS) * 2;       // bytes of its metas
    __host__ __device__ static constexpr int stage_bytes(int HB) { return 2 * HB * (TILE + META); }
    // pairs that a lane exchanges: outputs, maxima, sums
    static constexpr int PAIRS = D / 16 * 2 * NT + 2 * NT;
    // (U: heads x row tiles)
    __host__ __device__ static constexpr int merge_bytes(int U, int SUB) {
        return SUB > 1 ? U * ((SUB + 1) / 2) * 32 * PAIRS * 8 : 0;
    }
    // the queries of a segment, twice: the B fragments of Q^T, then per row the units and sums
    static constexpr int QROWS = 1 + D / GS;
    static constexpr int FRAG = NT * (D / 32) * 512, ROWS = QROWS * 32 * NT;
    __host__ __device__ static constexpr int query_bytes(int U) { return U * (FRAG + ROWS); }
    // a warp's scales: per row and group the limit of w, the factor of p and the maximum of w
    static constexpr int SCALES = NT * (D / GS) * 8 * 3 * 4;
    __host__ __device__ static constexpr int table_bytes(int B) { return ((3 * B + 2) * 4 + 15) / 16 * 16; }
    __host__ __device__ static constexpr int smem_bytes(int HB, int U, int SUB, int B, int ns) {
        return ns * stage_bytes(HB) + 2 * query_bytes(U) + merge_bytes(U, SUB) + U * SUB * SCALES + table_bytes(B) + (2 * ns + 4) * 8;
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

// The two halves of an f16x2 in fp32 (exact).
__device__ __forceinline__ float2 f16_pair(uint32_t x) {
    float2 r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.f32.f16 %0, lo;\n\t"
        "cvt.f32.f16 %1, hi;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(x));
    return r;
}

// 1 / s of a sum of weights, or 0 without any; a NaN stays one.
__device__ __forceinline__ float q4_over(float s) { return s > 0.0f ? 1.0f / s : s == s ? 0.0f : s; }

// D += A B and D = A B (no accumulator to clear), not volatile: free to be scheduled.
__device__ __forceinline__ void q4_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void q4_mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void q4_mma2(float2 (&d)[2], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0].x), "+f"(d[0].y), "+f"(d[1].x), "+f"(d[1].y)
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Keys the sequence's queries can see start here (the window of its first query).
__device__ __forceinline__ int q4_first_key(int L, int n, int window) {
    return window >= 0 ? max(0, L - n - window) : 0;
}

// Queries of sequence b (those within total_q and max_q).
__device__ __forceinline__ int q4_queries(const Q4AttnArgs& a, int b) {
    if (!a.cu_q) return 1;
    const int q0 = __ldg(&a.cu_q[b]), q1 = __ldg(&a.cu_q[b + 1]);
    return q0 < 0 ? 0 : min(max(min(q1, a.total_q) - q0, 0), a.max_q);
}
// Pages that they read, of one block of KV heads.
__device__ __forceinline__ int q4_pages(const Q4AttnArgs& a, int b, int len) {
    const int L = min(max(len, 0), a.max_blocks * kPageRows), n = q4_queries(a, b);
    return n > 0 ? (L + kPageRows - 1) / kPageRows - q4_first_key(L, n, a.window) / kPageRows : 0;
}
// The cost of a CTA's share, PC that of all pages of one block of heads: equal ones, of a
// pair of pages per warp at least.
__device__ __forceinline__ int q4_share(int PC, const Q4AttnArgs& a) {
    return max((int)(((uint32_t)(PC * a.nhb) + a.grid - 1) / (uint32_t)a.grid), 2 * a.SUB);   // (below 2^31)
}

// The queries of a sequence of n as the consumers want them: `units` (KV head of the block,
// row tile) of NT times eight rows, of whose eights this warp takes every step-th from `first`
// on.  Per eight rows the B fragments (dims e = 0, 4), (1, 5), (2, 6), (3, 7) of each word in
// f16 (second nibbles' dims over 16), and per row the unit of its raw scores in log2 units and
// minus the sums of q over the groups.  Rows past the last query are zero.  The loads of N
// eights are in flight together.
template <int D, int GS, int NT, int N>
__device__ __noinline__ void q4_prepare(const __nv_bfloat16* q, int Hq, int group, float unit, int n, int RT, int units, int first,
                                        int step, uint32_t frag_at, uint32_t rows_at) {
    // (q: the first query of the sequence, at the block's first query head; offsets in shared memory)
    extern __shared__ __align__(128) uint8_t q4_smem[];
    using C = Q4Cfg<D, GS, NT>;
    const int lane = threadIdx.x & 31;
    constexpr int W = D / 32, G = D / GS, WG = W / G;
    const int r8 = lane >> 2, t4 = lane & 3;
    for (int t0 = first; t0 < units * NT; t0 += N * step) {
        uint4 x[N][W];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int t = t0 + i * step, h = t / (RT * NT), row = t % (RT * NT) * 8 + r8;
            const int tok = n == 1 ? row >= group : row / group;
            const bool live = t < units * NT && tok < n;
            const __nv_bfloat16* qr = q + (live ? ((long long)tok * Hq + h * group + row - tok * group) * D : 0);
#pragma unroll
            for (int w = 0; w < W; ++w)
                x[i][w] = live ? __ldg(reinterpret_cast<const uint4*>(qr + 32 * w + 8 * t4)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int t = t0 + i * step;
            if (t >= units * NT) break;
            float big = 0.0f, sum[G];
#pragma unroll
            for (int g = 0; g < G; ++g) sum[g] = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const uint32_t xs[4] = {x[i][w].x, x[i][w].y, x[i][w].z, x[i][w].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    big = fmax3(big, fabsf(bf16_lo(xs[e])), fabsf(bf16_hi(xs[e])));
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
            const float up = __uint_as_float((uint32_t)(127 + 13 - ex) << 23), up1 = up * 0.0625f;
            const float down = __uint_as_float((uint32_t)(127 + 11 + ex) << 23);    // 2^24 / up
            uint4* frag = reinterpret_cast<uint4*>(q4_smem + frag_at + t * (C::FRAG / NT));
            float* rows = reinterpret_cast<float*>(q4_smem + rows_at + t / NT * C::ROWS + t % NT * 32);
#pragma unroll
            for (int w = 0; w < W; ++w)
                frag[w * 32 + lane] = make_uint4(pack_f16(bf16_lo(x[i][w].x) * up, bf16_lo(x[i][w].z) * up),
                                                 pack_f16(bf16_hi(x[i][w].x) * up1, bf16_hi(x[i][w].z) * up1),
                                                 pack_f16(bf16_lo(x[i][w].y) * up, bf16_lo(x[i][w].w) * up),
                                                 pack_f16(bf16_hi(x[i][w].y) * up1, bf16_hi(x[i][w].w) * up1));
            if (t4 == 0) {
                rows[r8] = fmaxf(down * unit, 1e-33f);   // (with 0 a masked score's minus infinity would give a NaN)
#pragma unroll
                for (int g = 0; g < G; ++g) rows[(1 + g) * 8 * NT + r8] = -sum[g] / down;
            }
        }
    }
}

template <int D, int GS, int NT>
__global__ void __launch_bounds__(32 * (q4_warps(NT) + kQ4Producers), 1) q4_attn_kernel(const Q4AttnArgs a) {
    using C = Q4Cfg<D, GS, NT>;
    constexpr int W = D / 32;            // words of a lane's K row piece; V words per token pair
    constexpr int G = D / GS;            // groups of a head
    constexpr int WG = W / G;            // words of a group
    constexpr int MT = D / 16;           // 16-column output tiles
    constexpr int NP = NT == 1 ? 2 : 1;  // pages a warp takes at once: two chains of dependent operations side by side
    const int NS = a.nstages, HB = a.HB, SUB = a.SUB, U = HB * a.RT, SB = C::stage_bytes(HB);
    extern __shared__ __align__(128) uint8_t q4_smem[];
    uint8_t* smem = q4_smem;
    uint8_t* tail = smem + NS * SB;
    uint8_t* qarea = tail;                           // two of: [U][NT][W][32] uint4, [U][QROWS][8 NT] float
    const int QB = C::query_bytes(U);
    tail += 2 * QB;
    float* mrg = reinterpret_cast<float*>(tail);
    tail += C::merge_bytes(U, SUB);
    float2* scales = reinterpret_cast<float2*>(tail);
    tail += U * SUB * C::SCALES;
    int* prefix = reinterpret_cast<int*>(tail);      // [B + 1] pages before sequence b
    int* cost = prefix + (a.B + 1);                  // [B + 1] their cost
    int* lenv = cost + (a.B + 1);                    // [B]
    uint64_t* full = reinterpret_cast<uint64_t*>(tail + C::table_bytes(a.B));
    uint64_t* empty = full + NS;
    uint64_t *qfull = empty + NS, *qempty = qfull + 2;
    __shared__ int bounds[2], first_place[2];        // the share's first page and the one behind it; its first sequence

    // Launched as a programmatic dependent of whatever precedes it.  Only then may the combine
    // kernel start, which reads the lengths before it waits for this one.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // (by way of a shuffle: what depends on the warp alone then stays off the vector units)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    auto queries = [&](int b) { return q4_queries(a, b); };
    if (warp == 0) {
        int run = 0, with_any = 0;
        long long keys = 0;
        for (int base = 0; base < a.B; base += 32 * kQ4Scan) {
            int cnts[kQ4Scan];
#pragma unroll
            for (int i = 0; i < kQ4Scan; ++i) {
                const int b = base + 32 * i + lane;
                cnts[i] = 0;
                if (b < a.B) {
                    const int len = a.seqused_k[b];
                    lenv[b] = min(max(len, 0), a.max_blocks * kPageRows);
                    keys += max(len, 0);
                    cnts[i] = q4_pages(a, b, len);
                    if (a.cu_q && blockIdx.x == 0 && q4_queries(a, b) != max(__ldg(&a.cu_q[b + 1]) - __ldg(&a.cu_q[b]), 0))
                        record_data_error(kErrQ4Queries);
                }
            }
#pragma unroll
            for (int i = 0; i < kQ4Scan; ++i) {
                if (base + 32 * i >= a.B) break;
                const int b = base + 32 * i + lane, cnt = cnts[i];
                int incl = cnt;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += v;
                }
                const uint32_t any = __ballot_sync(0xffffffffu, cnt > 0);
                if (b < a.B) {
                    prefix[b] = run + incl - cnt;
                    cost[b] = run + incl - cnt + kQ4Switch * (with_any + __popc(any & ((1u << lane) - 1u)));
                    if (a.table && blockIdx.x == 0) a.table[b] = make_int2(cnt, cost[b]);
                }
                run += __shfl_sync(0xffffffffu, incl, 31);
                with_any += __popc(any);
            }
        }
        if (a.total_k >= 0 && blockIdx.x == 0) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) keys += __shfl_xor_sync(0xffffffffu, keys, o);
            if (keys > a.total_k) record_data_error(kErrQ4Rows);
        }
        if (lane == 0) {
            prefix[a.B] = run;
            cost[a.B] = run + kQ4Switch * with_any;
            if (a.table && blockIdx.x == 0) a.table[a.B] = make_int2(0, cost[a.B]);
        }
        __syncwarp();
        // The pages of one head block after another, each sequence's behind kQ4Switch units for
        // the change to it, are cut into equal shares of this cost (their number stays below
        // 2^31, as the host checks).  Where this CTA's share starts and ends:
        const int PC = run + kQ4Switch * with_any, share = q4_share(PC, a);
        for (int e = 0; e < 2; ++e) {
            const uint32_t c = (blockIdx.x + e) * (uint32_t)share;       // (below 2^32)
            int hb = 0, at = run * a.nhb, b = 0;
            if (c < (uint32_t)(PC * a.nhb)) {
                hb = a.nhb == 1 ? 0 : c / (uint32_t)PC;
                const int r = (int)c - hb * PC;
                // the largest b with cost[b] <= r, 32 candidates at a time
                for (int len = a.B; len > 1;) {
                    const int step = (len + 31) / 32, i = lane * step;
                    const int k = __popc(__ballot_sync(0xffffffffu, i < len && cost[b + min(i, len - 1)] <= r)) - 1;
                    b += k * step;
                    len = min(step, len - k * step);
                }
                at = hb * run + prefix[b] + max(r - cost[b] - kQ4Switch, 0);
            }
            if (lane == 0) {
                bounds[e] = at;
                if (e == 0) {
                    first_place[0] = hb;
                    first_place[1] = b;
                }
            }
        }
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 3);
            mbar_init(&empty[i], U);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qfull[i], 1);
            mbar_init(&qempty[i], U * SUB);
        }
        fence_mbar_init();
    }
    __syncthreads();
    const int P = prefix[a.B], p0 = bounds[0], npages = bounds[1] - p0;
    if (npages == 0) return;

    // The queries of the share's sequences as the consumers want them, in two areas by turns:
    // the first sequence's by the consumers themselves, the others one sequence ahead by the
    // fourth producer warp.
    auto prepare = [&](int turn, int hb, int b, int first, int step, auto at_once) {
        const uint32_t to = (uint32_t)(qarea - smem) + (turn & 1) * QB;
        const __nv_bfloat16* q = a.q + ((long long)(a.cu_q ? __ldg(&a.cu_q[b]) : b) * a.Hq + hb * HB * a.group) * D;
        q4_prepare<D, GS, NT, decltype(at_once)::value>(q, a.Hq, a.group, a.scale * kLog2e, queries(b), a.RT, U, first, step, to, to + U * C::FRAG);
    };
    // The sequences of the share in order: (block of heads, sequence), and the page at which each ends.
    struct Place {
        int hb, b, end;
    };
    auto ends = [&](int hb, int b) { return min(npages, hb * P + prefix[b + 1] - p0); };
    auto next_place = [&](Place x) {                 // the next sequence that has pages
        do {
            if (++x.b == a.B) {
                x.b = 0;
                ++x.hb;
            }
        } while (prefix[x.b + 1] == prefix[x.b]);
        x.end = ends(x.hb, x.b);
        return x;
    };
    const Place start = {first_place[0], first_place[1], ends(first_place[0], first_place[1])};

    if (warp >= q4_warps(NT)) {
        // ------------------------------------------------------------ producers: K, V, metas, queries
        const int which = warp - q4_warps(NT);
        if (which == 3) {
            Place x = start;
            for (int turn = 1; x.end < npages; ++turn) {
                x = next_place(x);
                bool ok = mbar_wait(&qempty[turn & 1], (turn >> 1 & 1) ^ 1, kErrQ4Empty);
                if (!__all_sync(0xffffffffu, ok)) break;
                prepare(turn, x.hb, x.b, 0, 1, std::integral_constant<int, 2>());
                __syncwarp();
                if (lane == 0) mbar_arrive(&qfull[turn & 1]);
            }
            return;
        }
        const uint8_t* src = which == 0 ? a.k_cache : which == 1 ? a.v_cache : reinterpret_cast<const uint8_t*>(a.k_meta);
        const uint8_t* src2 = reinterpret_cast<const uint8_t*>(a.v_meta);
        const int unit = which < 2 ? C::TILE : C::META, bytes = HB * unit;
        uint8_t* dst0 = smem + which * HB * C::TILE;
        const uint64_t pol = policy_evict_first();
        int issued = 0, st = 0;
        uint32_t ph = 1;
        Place x = start;
        for (int base = 0; base < npages; base += 32) {
            long long mine = 0;                      // this lane's page of the next 32: its first tile
            if (base + lane < npages) {
                while (x.end <= base + lane) x = next_place(x);
                const int hb = x.hb, b = x.b, g = p0 + base + lane - hb * P;
                const int slot = g - prefix[b] + q4_first_key(lenv[b], queries(b), a.window) / kPageRows;
                int phys = a.block_table[(long long)b * a.max_blocks + slot];
                if (phys < 0 || phys >= a.num_blocks) {
                    record_data_error(kErrDecPageRange);   // outside the cache: reported, page 0 read
                    phys = 0;
                }
                mine = ((long long)phys * a.Hkv + hb * HB) * unit;
            }
            const int cnt = min(32, npages - base);
            bool ok = true;
            for (int i = 0; i < cnt; ++i, ++issued) {
                const long long at = __shfl_sync(0xffffffffu, mine, i);
                ok = mbar_wait(&empty[st], ph, kErrQ4Empty);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[st], which < 2 ? bytes : 2 * bytes);
                    bulk_load(dst0 + st * SB, src + at, bytes, &full[st], pol);
                    if (which == 2) bulk_load(dst0 + st * SB + bytes, src2 + at, bytes, &full[st], pol);
                }
                if (++st == NS) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (!ok) break;
        }
        if (lane == 0) {
            for (int s = 0; s < NS && s < issued; ++s) {
                const int last = s + ((issued - 1 - s) / NS) * NS;
                mbar_wait_drain(&full[s], (last / NS) & 1, kErrQ4Full);
            }
        }
        return;
    }
    if (warp >= U * SUB) return;
    // ---------------------------------------------------------------- consumers
    const int unit = warp / SUB, sub = warp % SUB;   // head and row tile, this warp's share of their pages
    const int h = unit / a.RT, row0 = unit % a.RT * 8 * NT;
    const int r8 = lane >> 2, t4 = lane & 3;
    const bool capped = a.softcap > 0.0f;
    // this lane's B fragments of Q^T, (dims e = 0, 4), (1, 5), (2, 6), (3, 7) of each word: in
    // shared memory, which spares registers
    uint32_t qb = 0;                     // (its offset in shared memory)
    // of the columns 2 t4 and 2 t4 + 1 (x, y) of each 8-row tile:
    float2 qs[NT][G];                    // minus the sum of q over a group, in units of the raw score
    float2 kf[NT];                       // score in log2 units = raw score * kf
    float2 acc[MT][NT][2];               // sum w c: tile rows r8 in units of 2^-24, r8 + 8 of 2^-20
    float2 zac[NT][G];                   // sum w zero, this lane's keys
    float2 m[NT], l[NT];                 // minus the maximum (log2 units); sum, this lane's keys
    // Per row and group, in shared memory: w_max, the largest log2 of p step seen (the maximum of
    // the scores not taken off: acc stays in its units when m moves), and by it w = p beta step with
    // beta = 2^(7 + max - w_max), and the limit of log2(p step) that moves it.
    float2* const lim = scales + warp * (C::SCALES / 8) + t4;
    float2* const beta = lim + NT * G * 4;
    float2* const wmax = beta + NT * G * 4;
    int since = 0;
    auto reset = [&]() {
        const float2 zero2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < MT; ++c)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[c][nt][0] = acc[c][nt][1] = zero2;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt] = make_float2(-kQ4NoMax, -kQ4NoMax);
            l[nt] = zero2;
#pragma unroll
            for (int g = 0; g < G; ++g) zac[nt][g] = zero2;
        }
        __syncwarp();
        if (r8 == 0) {
#pragma unroll
            for (int i = 0; i < NT * G; ++i) {
                lim[4 * i] = make_float2(INFINITY, INFINITY);        // (the first key moves m)
                beta[4 * i] = make_float2(1.0f, 1.0f);
                wmax[4 * i] = make_float2(kQ4NoMax, kQ4NoMax);
            }
        }
        __syncwarp();
        since = 0;
    };
    auto over_rows = [&](float2 v) {                 // the sum over the lanes of a column
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
        return v;
    };
    // takes sum w zero out of the accumulators
    auto recentre = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float2 z = over_rows(zac[nt][g]);
                zac[nt][g] = make_float2(0.0f, 0.0f);
                const float lo = -5.9604644775390625e-8f, hi = -9.5367431640625e-7f;     // -2^-24, -2^-20
#pragma unroll
                for (int c = g * (MT / G); c < (g + 1) * (MT / G); ++c) {
                    acc[c][nt][0] = ffma2(z, make_float2(lo, lo), acc[c][nt][0]);
                    acc[c][nt][1] = ffma2(z, make_float2(hi, hi), acc[c][nt][1]);
                }
            }
        since = 0;
    };
    // the end of a sequence or of the share: join the SUB warps of the head, write the partial
    auto flush_partial = [&](int vb, int n) {
        recentre();
        // this warp's output: acc, in units of w, over l
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            l[nt] = over_rows(l[nt]);
            const float2 inv = make_float2(q4_over(l[nt].x), q4_over(l[nt].y));
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float2 w = fadd2(wmax[4 * (nt * G + g)], m[nt]);
                const float2 half = make_float2(ex2(0.5f * w.x), ex2(0.5f * w.y));     // (2^w may not be a float)
                const float2 f = fmul2(inv, half);
#pragma unroll
                for (int c = g * (MT / G); c < (g + 1) * (MT / G); ++c) {
                    acc[c][nt][0] = fmul2(fmul2(fmul2(acc[c][nt][0], make_float2(131072.0f, 131072.0f)), f), half);  // 2^(24 - 7)
                    acc[c][nt][1] = fmul2(fmul2(fmul2(acc[c][nt][1], make_float2(8192.0f, 8192.0f)), f), half);      // 2^(20 - 7)
                }
            }
        }
        constexpr int FL = C::PAIRS;                 // pairs a lane exchanges
        const int slots = (SUB + 1) / 2;
        float2* mine = reinterpret_cast<float2*>(mrg) + unit * slots * 32 * FL;
        int width = 1;
        while (width < SUB) width <<= 1;
        for (int st = width / 2; st > 0; st >>= 1) {
            if (sub >= st && sub < 2 * st) {
                float2* x = mine + (sub - st) * 32 * FL + lane;
#pragma unroll
                for (int c = 0; c < MT; ++c)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        x[32 * (c * NT + nt) * 2] = acc[c][nt][0];
                        x[32 * ((c * NT + nt) * 2 + 1)] = acc[c][nt][1];
                    }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    x[32 * (MT * NT + nt) * 2] = m[nt];
                    x[32 * ((MT * NT + nt) * 2 + 1)] = l[nt];
                }
            }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + unit), "r"(32 * SUB) : "memory");
            if (sub < st && sub + st < SUB) {
                const float2* x = mine + sub * 32 * FL + lane;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float2 m2 = x[32 * (MT * NT + nt) * 2], l2 = x[32 * ((MT * NT + nt) * 2 + 1)];
                    const float2 mn = make_float2(fminf(m[nt].x, m2.x), fminf(m[nt].y, m2.y));
                    float2 f1 = make_float2(ex2(mn.x - m[nt].x), ex2(mn.y - m[nt].y));
                    float2 f2 = make_float2(ex2(mn.x - m2.x), ex2(mn.y - m2.y));
                    m[nt] = mn;
                    f1 = fmul2(l[nt], f1);
                    f2 = fmul2(l2, f2);
                    l[nt] = fadd2(f1, f2);
                    const float2 inv = make_float2(q4_over(l[nt].x), q4_over(l[nt].y));
                    f1 = fmul2(f1, inv);
                    f2 = fmul2(f2, inv);
#pragma unroll
                    for (int c = 0; c < MT; ++c)
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            acc[c][nt][y] = ffma2(acc[c][nt][y], f1, fmul2(x[32 * ((c * NT + nt) * 2 + y)], f2));
                }
            }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + unit), "r"(32 * SUB) : "memory");
        }
        if (sub > 0) return;
        const long long base = (((long long)blockIdx.x + vb) * HB + h) * a.rows;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = row0 + nt * 8 + 2 * t4 + e;
                if (row >= n * a.group) continue;
                const float s = e ? l[nt].y : l[nt].x;
                float* rp = a.o_part + (base + row) * D;
#pragma unroll
                for (int c = 0; c < MT; ++c) {
                    rp[16 * c + r8] = e ? acc[c][nt][0].y : acc[c][nt][0].x;
                    rp[16 * c + 8 + r8] = e ? acc[c][nt][1].y : acc[c][nt][1].x;
                }
                if (r8 == 0)
                    a.lse_part[base + row] = s > 0.0f ? (log2f(s) - (e ? m[nt].y : m[nt].x)) * kLn2 : s == s ? -INFINITY : s;
            }
    };
    bool ok = true;
    int i = sub, st = sub;                           // this warp's next page of the share, and its stage
    uint32_t ph = 0;
    while (st >= NS) {
        st -= NS;
        ph ^= 1;
    }
    const uint8_t* kbase = smem + h * C::TILE + r8 * (D / 2) + t4 * W * 4;
    const uint8_t* vbase = smem + (HB + h) * C::TILE + lane * W * 4;
    const uint8_t* mbase = smem + 2 * HB * C::TILE + h * C::META + r8 * G * 2;
    // raw scores of a page's keys r8 and r8 + 8 against the tile's columns
    auto scores = [&](int so, float2 (&sc)[NT][2]) {
        uint32_t k0[W], k1[W], km0[G], km1[G];
        load_words<W>(kbase + so, k0);
        load_words<W>(kbase + so + 4 * D, k1);
        load_metas<G>(mbase + so, km0);
        load_metas<G>(mbase + so + 16 * G, km1);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float raw[NT][4], raw2[NT][4];
#pragma unroll
            for (int w = g * WG; w < (g + 1) * WG; ++w) {
                const uint32_t lo[4] = {k0[w] & 0x000f000fu, k1[w] & 0x000f000fu, k0[w] & 0x00f000f0u, k1[w] & 0x00f000f0u};
                const uint32_t x0 = k0[w] >> 8, x1 = k1[w] >> 8;
                const uint32_t hi[4] = {x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 qw = *reinterpret_cast<const uint4*>(smem + qb + (nt * W + w) * 512);
                    if (WG == 1) {
                        q4_mma_first(raw[nt], lo, qw.x, qw.y);
                        q4_mma(raw[nt], hi, qw.z, qw.w);
                    } else if (w == g * WG) {
                        q4_mma_first(raw[nt], lo, qw.x, qw.y);
                        q4_mma_first(raw2[nt], hi, qw.z, qw.w);
                    } else {
                        q4_mma(raw[nt], lo, qw.x, qw.y);
                        q4_mma(raw2[nt], hi, qw.z, qw.w);
                    }
                }
            }
            const float s0 = q4_step(km0[g]), s1 = q4_step(km1[g]), z0 = q4_zero(km0[g]), z1 = q4_zero(km1[g]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float2 d0 = make_float2(raw[nt][0], raw[nt][1]), d1 = make_float2(raw[nt][2], raw[nt][3]);
                if (WG > 1) {
                    d0 = fadd2(d0, make_float2(raw2[nt][0], raw2[nt][1]));
                    d1 = fadd2(d1, make_float2(raw2[nt][2], raw2[nt][3]));
                }
                const float2 y0 = ffma2(make_float2(z0, z0), qs[nt][g], d0), y1 = ffma2(make_float2(z1, z1), qs[nt][g], d1);
                sc[nt][0] = g == 0 ? fmul2(y0, make_float2(s0, s0)) : ffma2(y0, make_float2(s0, s0), sc[nt][0]);
                sc[nt][1] = g == 0 ? fmul2(y1, make_float2(s1, s1)) : ffma2(y1, make_float2(s1, s1), sc[nt][1]);
            }
        }
    };
    int turn = 0;                                    // sequences of the share so far
    Place place = start;
    for (int seg = 0; seg < npages; ++turn) {
        if (turn) place = next_place(place);
        const int hb = place.hb, b = place.b, seg_end = place.end, g0 = p0 + seg - hb * P;
        const int L = lenv[b], n = queries(b);
        // first key of the share's page `seg`
        const int key0 = (g0 - prefix[b] + q4_first_key(L, n, a.window) / kPageRows) * kPageRows;
        reset();
        if (turn == 0) {
            prepare(0, hb, b, warp, U * SUB, std::integral_constant<int, 1>());
            asm volatile("bar.sync 15, %0;" ::"r"(32 * U * SUB) : "memory");
        } else if (ok) {
            ok = mbar_wait(&qfull[turn & 1], (turn >> 1 & 1) ^ (turn & 1 ^ 1), kErrQ4Full);
            ok = __all_sync(0xffffffffu, ok);
        }
        {
            const uint8_t* q = qarea + (turn & 1) * QB;
            qb = (uint32_t)(qarea - smem) + (turn & 1) * QB + unit * C::FRAG + lane * 16;
            const float* rows = reinterpret_cast<const float*>(q + U * C::FRAG + unit * C::ROWS) + 2 * t4;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                kf[nt] = *reinterpret_cast<const float2*>(rows + 8 * nt);
#pragma unroll
                for (int g = 0; g < G; ++g) qs[nt][g] = *reinterpret_cast<const float2*>(rows + (1 + g) * 8 * NT + 8 * nt);
            }
        }
        // pages whose keys every query sees: key0 of the page in [all_lo, all_hi]
        const int all_hi = (a.causal ? L - n : L - 1) - (kPageRows - 1);
        const int all_lo = a.window >= 0 ? L - 1 - a.window : 0;
        // waits for this warp's next page (and the one after); their stages go to `at`
        auto take = [&](int (&at)[NP]) {
            const bool two = NP > 1 && i + SUB < seg_end;
#pragma unroll
            for (int x = 0; x < NP; ++x) {
                if (x == 0 || two) {
                    if (ok) {
                        ok = mbar_wait(&full[st], ph, kErrQ4Full);
                        ok = __all_sync(0xffffffffu, ok);
                    }
                    at[x] = st;
                    st += SUB;
                    while (st >= NS) {
                        st -= NS;
                        ph ^= 1;
                    }
                } else {
                    at[x] = at[0];                               // no second page: masked below
                }
            }
            i += two ? 2 * SUB : SUB;
            return two;
        };
        int at[NP];
        float2 sc[NP][NT][2];
        while (i < seg_end) {
            const int tok0 = key0 + (i - seg) * kPageRows;
            const bool two = take(at);
#pragma unroll
            for (int x = 0; x < NP; ++x) scores(at[x] * SB, sc[x]);
            uint32_t vm0[NP][G], vm1[NP][G];
#pragma unroll
            for (int x = 0; x < NP; ++x) {
                load_metas<G>(mbase + at[x] * SB + HB * C::META, vm0[x]);
                load_metas<G>(mbase + at[x] * SB + HB * C::META + 16 * G, vm1[x]);
            }
            if (capped) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float b0 = kf[nt].x * kLn2, b1 = kf[nt].y * kLn2;             // to natural units
                    const float i0 = b0 / a.softcap, i1 = b1 / a.softcap, o0 = a.softcap / b0, o1 = a.softcap / b1;
#pragma unroll
                    for (int x = 0; x < NP; ++x)
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            sc[x][nt][y] = make_float2(softcap_raw(sc[x][nt][y].x, i0, o0), softcap_raw(sc[x][nt][y].y, i1, o1));
                }
            }
            if ((NP > 1 && !two) || tok0 + (NP - 1) * SUB * kPageRows > all_hi || tok0 < all_lo) {
#pragma unroll
                for (int x = 0; x < NP; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int key = x == 0 || two ? tok0 + x * SUB * kPageRows + r8 + 8 * y : L;
                        if (key >= L) {                // not data of the sequence
#pragma unroll
                            for (int g = 0; g < G; ++g) (y ? vm1 : vm0)[x][g] = 0;
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int tok = (row0 + nt * 8 + 2 * t4 + e) / a.group;
                                const int last = a.causal ? L - n + tok : L - 1;
                                if (key > last || key >= L || (a.window >= 0 && key < last - a.window))
                                    (e ? sc[x][nt][y].y : sc[x][nt][y].x) = -INFINITY;
                            }
                        // A NaN step reaches the rows that see its key, by way of the sums, and no weight of 0.
#pragma unroll
                        for (int g = 0; g < G; ++g) {
                            uint32_t& meta = (y ? vm1 : vm0)[x][g];
                            if ((meta & 0x7f80u) != 0x7f80u) continue;
                            meta = 0;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                if (sc[x][nt][y].x != -INFINITY) zac[nt][g].x = NAN;
                                if (sc[x][nt][y].y != -INFINITY) zac[nt][g].y = NAN;
                            }
                        }
                    }
            }
            // Does a score exceed its row's maximum by the slack, or a weight its own?  (Of the weights a
            // bound from above, the lane's largest score by its largest step, whose bits count 128 to the
            // octave and stay at most 0.09 below its logarithm; a step of 0 counts as 2^-127, too little.)
            bool over = false;
            float top[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                uint32_t most = max(vm0[0][g], vm1[0][g]);
                if (NP > 1) most = max(most, max(vm0[NP - 1][g], vm1[NP - 1][g]));
                top[g] = fmaf(__uint_as_float(most | 0x4b000000u), 0.0078125f, -65663.0f);
            }
            float2 mx[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mx[nt] = make_float2(fmaxf(sc[0][nt][0].x, sc[0][nt][1].x), fmaxf(sc[0][nt][0].y, sc[0][nt][1].y));
                if (NP > 1) {
                    mx[nt].x = fmax3(mx[nt].x, sc[NP - 1][nt][0].x, sc[NP - 1][nt][1].x);
                    mx[nt].y = fmax3(mx[nt].y, sc[NP - 1][nt][0].y, sc[NP - 1][nt][1].y);
                }
                const float2 u = ffma2(mx[nt], kf[nt], m[nt]);
                over = over || u.x > kQ4Slack || u.y > kQ4Slack;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float2 w = fadd2(u, make_float2(top[g], top[g])), most = lim[4 * (nt * G + g)];
                    over = over || w.x > most.x || w.y > most.y;
                }
            }
            if (__any_sync(0xffffffffu, over)) {
                // (a NaN among the steps takes no part: it makes its weights and its group NaN)
                auto largest = [&](float2 y) {       // over the keys of a column
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        y.x = fmaxf(y.x, __shfl_xor_sync(0xffffffffu, y.x, o));
                        y.y = fmaxf(y.y, __shfl_xor_sync(0xffffffffu, y.y, o));
                    }
                    return y;
                };
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float2 y = largest(mx[nt]);
                    const float2 mn = make_float2(fminf(m[nt].x, -y.x * kf[nt].x), fminf(m[nt].y, -y.y * kf[nt].y));
                    l[nt] = fmul2(l[nt], make_float2(ex2(mn.x - m[nt].x), ex2(mn.y - m[nt].y)));
                    m[nt] = mn;
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        float2 w = make_float2(-INFINITY, -INFINITY);
#pragma unroll
                        for (int x = 0; x < NP; ++x)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const float s = __log2f(q4_step((y ? vm1 : vm0)[x][g]));       // (of 0 minus infinity)
                                const float2 v = ffma2(sc[x][nt][y], kf[nt], make_float2(s, s));
                                w.x = fmaxf(w.x, v.x);
                                w.y = fmaxf(w.y, v.y);
                            }
                        w = largest(w);
                        float2 &at = wmax[4 * (nt * G + g)], old = at;
                        w.x = fmax3(old.x, w.x, -mn.x - kQ4Range);
                        w.y = fmax3(old.y, w.y, -mn.y - kQ4Range);
                        const float2 f = make_float2(ex2(old.x - w.x), ex2(old.y - w.y)), d = fadd2(w, mn);
                        zac[nt][g] = fmul2(zac[nt][g], f);
#pragma unroll
                        for (int c = g * (MT / G); c < (g + 1) * (MT / G); ++c) {
                            acc[c][nt][0] = fmul2(acc[c][nt][0], f);
                            acc[c][nt][1] = fmul2(acc[c][nt][1], f);
                        }
                        __syncwarp();
                        if (r8 == 0) {
                            at = w;
                            lim[4 * (nt * G + g)] = make_float2(d.x + kQ4Slack, d.y + kQ4Slack);
                            beta[4 * (nt * G + g)] = make_float2(ex2(kQ4Top - d.x), ex2(kQ4Top - d.y));
                        }
                    }
                }
                __syncwarp();
            }
#pragma unroll
            for (int x = 0; x < NP; ++x) {
                float2 p[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float2 d = ffma2(sc[x][nt][y], kf[nt], m[nt]);
                        p[nt][y] = make_float2(ex2(d.x), ex2(d.y));
                        l[nt] = fadd2(l[nt], p[nt][y]);
                    }
                uint32_t v0[W], v1[W];
                load_words<W>(vbase + at[x] * SB, v0);
                load_words<W>(vbase + at[x] * SB + 128 * W, v1);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float s0 = q4_step(vm0[x][g]), s1 = q4_step(vm1[x][g]);
                    const float z0 = q4_zero(vm0[x][g]), z1 = q4_zero(vm1[x][g]);
                    uint32_t pb[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float2 bt = beta[4 * (nt * G + g)];
                        const float2 x0 = fmul2(fmul2(p[nt][0], bt), make_float2(s0, s0));
                        const float2 x1 = fmul2(fmul2(p[nt][1], bt), make_float2(s1, s1));
                        const uint32_t h0 = pack_f16(x0.x, x0.y), h1 = pack_f16(x1.x, x1.y);
                        zac[nt][g] = ffma2(f16_pair(h0), make_float2(z0, z0),
                                           ffma2(f16_pair(h1), make_float2(z1, z1), zac[nt][g]));
                        pb[nt][0] = movmatrix_trans(h0);
                        pb[nt][1] = movmatrix_trans(h1);
                    }
#pragma unroll
                    for (int w = g * WG; w < (g + 1) * WG; ++w) {
                        const uint32_t lo[4] = {v0[w] & 0x000f000fu, v0[w] & 0x00f000f0u, v1[w] & 0x000f000fu,
                                                v1[w] & 0x00f000f0u};
                        const uint32_t y0 = v0[w] >> 8, y1 = v1[w] >> 8;
                        const uint32_t hi[4] = {y0 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x000f000fu, y1 & 0x00f000f0u};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            q4_mma2(acc[2 * w][nt], lo, pb[nt][0], pb[nt][1]);
                            q4_mma2(acc[2 * w + 1][nt], hi, pb[nt][0], pb[nt][1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&empty[at[0]]);
                if (two) mbar_arrive(&empty[at[NP - 1]]);
            }
            since += NP;
            if (since >= kQ4Recentre) recentre();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&qempty[turn & 1]);
        flush_partial(hb * a.B + b, n);
        seg = seg_end;
    }
}

// Joins the partials: a.wpr warps per output row (one for each eight partials, whose loads
// are in flight together): bound by its launch and two round trips, 4 to 6 us.  The partials
// of sequence b and head block hb sit in slots c + hb B + b for the CTAs c whose shares
// covered it.
template <int D>
__global__ void __launch_bounds__(256) q4_combine_kernel(const Q4AttnArgs a) {
    constexpr int V = D / 32;            // columns of a lane
    constexpr int N = 8;                 // partials whose loads are in flight together
    __shared__ float part[8][32 * V + 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp % a.wpr;        // this warp's share of the row's partials
    const long long w = (long long)blockIdx.x * (8 / a.wpr) + warp / a.wpr;
    const int per = a.max_q * a.Hq;      // rows of a sequence
    bool live = w < (long long)a.B * per;
    const int b = live ? (int)(w / per) : 0, tok = live ? (int)(w % per) / a.Hq : 0, hq = live ? (int)(w % per) % a.Hq : 0;
    const long long q0 = a.cu_q ? __ldg(&a.cu_q[b]) : b;
    live = live && tok < q4_queries(a, b);
    const int hkv = hq / a.group, hb = hkv / a.HB, h = hkv % a.HB;
    const int row = tok * a.group + hq % a.group;
    // The shares follow from the lengths alone: few are worked out while the attention kernel
    // still runs (which began after whatever wrote the lengths had ended), many taken from it.
    int PC = 0, cb = 0, mine = 0;
    if (!a.table) {
#pragma unroll 1
        for (int base = 0; base < a.B; base += 32 * kQ4Scan)
#pragma unroll
            for (int i = 0; i < kQ4Scan; ++i) {
                if (base + 32 * i >= a.B) break;
                const int s = base + 32 * i + lane;
                const int pages = s < a.B ? q4_pages(a, s, a.seqused_k[s]) : 0, c = pages > 0 ? pages + kQ4Switch : 0;
                PC += c;
                cb += s < b ? c : 0;
                mine += s == b ? pages : 0;
            }
        PC = __reduce_add_sync(0xffffffffu, PC);
        cb = __reduce_add_sync(0xffffffffu, cb);
        mine = __reduce_add_sync(0xffffffffu, mine);
    }
    int ns = 0;
    long long first = 0;
    auto slots = [&]() {
        const int share = q4_share(PC, a);
        const int c0 = (hb * PC + cb + kQ4Switch) / share;        // the CTAs of its first and last page
        ns = live && mine > 0 ? (hb * PC + cb + kQ4Switch + mine - 1) / share - c0 + 1 : 0;
        first = (((long long)c0 + hb * a.B + b) * a.HB + h) * a.rows + row;
    };
    if (!a.table) slots();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (a.table) {
        const int2 x = a.table[b];
        mine = x.x;
        cb = x.y;
        PC = a.table[a.B].y;
        slots();
    }
    const long long step = (long long)a.HB * a.rows * a.wpr;      // rows between this warp's partials
    float M = -INFINITY, sum = 0.0f, acc[V];
    bool nan = false;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.0f;
    for (int s0 = sub; s0 < ns; s0 += N * a.wpr) {
        const long long at = first + (long long)s0 * a.HB * a.rows;
        float x[N], y[N][V];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool has = s0 + i * a.wpr < ns;
            x[i] = has ? a.lse_part[at + i * step] : -INFINITY;
            const float* src = a.o_part + (at + i * step) * D + lane * V;
            if constexpr (V == 4) {
                const float4 f = has ? *reinterpret_cast<const float4*>(src) : make_float4(0, 0, 0, 0);
                y[i][0] = f.x, y[i][1] = f.y, y[i][2] = f.z, y[i][3] = f.w;
            } else {
                const float2 f = has ? *reinterpret_cast<const float2*>(src) : make_float2(0, 0);
                y[i][0] = f.x, y[i][1] = f.y;
            }
        }
        float mn = M;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            nan = nan || x[i] != x[i];
            mn = fmaxf(mn, x[i]);
        }
        if (mn == -INFINITY) continue;
        const float al = ex2((M - mn) * kLog2e);
        M = mn;
        sum *= al;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] *= al;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float f = ex2((x[i] - mn) * kLog2e);
            sum += f;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = fmaf(f, y[i][v], acc[v]);
        }
    }
    if (a.wpr > 1) {
        // the row's warps through shared memory, in order (the sum does not depend on their speed)
#pragma unroll
        for (int v = 0; v < V; ++v) part[warp][v * 32 + lane] = acc[v];
        if (lane == 0) {
            part[warp][32 * V] = nan ? NAN : M;
            part[warp][32 * V + 1] = sum;
        }
        __syncthreads();
        if (sub != 0) return;
        for (int s = 1; s < a.wpr; ++s) {
            const float m2 = part[warp + s][32 * V];
            if (m2 != m2) nan = true;
            const float mn = fmaxf(M, m2);
            if (mn == -INFINITY) continue;
            const float f1 = ex2((M - mn) * kLog2e), f2 = ex2((m2 - mn) * kLog2e);
            M = mn;
            sum = sum * f1 + part[warp + s][32 * V + 1] * f2;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = acc[v] * f1 + part[warp + s][v * 32 + lane] * f2;
        }
    }
    if (!live) return;
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
