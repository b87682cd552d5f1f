// api_rope_q4.cuh -- the C entry points of the rotary positions, the rotating KV
// appends and the 4-bit cache (included by attn_api.cu, whose helpers it uses).
#pragma once

#include <climits>

#include "q4.cuh"

namespace {

bool stride8(const int64_t* s, int n) {
    for (int i = 0; i < n; ++i)
        if (s[i] % 8) return false;
    return true;
}

// Do the heads of an output with these {token, head} strides lie apart: a token's all before the
// next token's, or a head's tokens all before the next head's?
bool own_places(const int64_t* s, int total, int H, int D) {
    auto within = [D](int64_t outer, int64_t inner, int n) { return n <= 1 || (outer - D) / (n - 1) >= inner; };
    return s[0] >= D && s[1] >= D && (within(s[0], s[1], H) || within(s[1], s[0], total));
}

// Strides of the same layout, where there is more than one token and head.
bool same_places(const int64_t* a, const int64_t* b, int total, int H) {
    return (total <= 1 || a[0] == b[0]) && (H <= 1 || a[1] == b[1]);
}

// Arguments of the table: cos_sin null means no rotation (where `optional`).
attn_status_t check_rope(const float* cos_sin, int max_position, int rot_dim, const int32_t* positions, int n_axes,
                         const int32_t* pair_axis, int D, bool optional) {
    if (!cos_sin) return optional ? ATTN_OK : ATTN_ERR_INVALID_ARG;
    if (max_position <= 0 || rot_dim <= 0 || rot_dim > D || n_axes < 1) return ATTN_ERR_INVALID_ARG;
    if (rot_dim % 16 || n_axes > kRopeMaxAxes) return ATTN_ERR_UNSUPPORTED;
    if (!positions && !optional) return ATTN_ERR_INVALID_ARG;
    if (n_axes > 1 && (!positions || !pair_axis)) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(cos_sin) || (n_axes > 1 && !aligned16(pair_axis))) return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

RopeTable rope_table(const float* cos_sin, int max_position, int rot_dim, const int32_t* positions, int n_axes,
                     const int32_t* pair_axis, int interleaved, int inverse) {
    RopeTable r;
    r.table = cos_sin;
    r.max_pos = max_position;
    r.rot = cos_sin ? rot_dim : 0;
    r.positions = positions;
    r.axes = n_axes;
    r.pair_axis = n_axes > 1 ? pair_axis : nullptr;
    r.interleaved = interleaved ? 1 : 0;
    r.sign = inverse ? -1.0f : 1.0f;
    return r;
}

HeadRows head_rows(const void* p, const int64_t* strides) {
    HeadRows h;
    h.p = static_cast<const __nv_bfloat16*>(p);
    h.row = p ? strides[0] : 0;
    h.head = p ? strides[1] : 0;
    return h;
}

// Warps that share a token's heads: one, unless that leaves an SM with fewer than eight,
// too few loads in flight.  (1024 tokens of 32 + 8 + 8 heads of 128 into 4-bit pages:
// 12.3 us with a warp per token, 10.2 at eight warps per SM, 14.3 at sixteen, which repeats
// the look-up of page and angles too often; 2048: 14.3, 14.3 and 16.4.)
int rope_parts(long long tokens, int passes, int sms) {
    const long long want = (long long)sms * 8;
    long long parts = tokens > 0 ? (want + tokens - 1) / tokens : 1;
    return (int)std::max<long long>(1, std::min<long long>(parts, passes));
}

constexpr int kQ4Few = 32 * kQ4Scan;
constexpr int kQ4Smem = 227 * 1024 - 256;      // (some is static)

// Eights of query rows that a warp holds.  Up to eight rows: one, which at 128 registers leaves
// room for twelve warps, and those hide each other's waits best (3 sequences of 65000 keys 77
// us, with eight warps 79; 32 of 4100 46 and 48).  More: two, so that half as many warps take
// the codes of a page apart; they need 168 registers, eight warps (16 sequences of 3700 keys,
// groups of four: 8 queries 73 us, one eight to each of eight warps 85, of twelve 91; 16 queries
// 126, 155, 155).
int q4_tile(int rows) { return rows <= 8 ? 1 : 2; }

// Row tiles of a KV head, KV heads of a CTA's block, and warps of a head and row tile: the
// block with the most of the CTA's warps at work, the largest such one (its copies are
// longest), but of two eights to a warp at most four heads: with eight, whose queries take
// twice as long to prepare, 4 queries take 50 us in place of 44 (with two 49).
void q4_split(int Hkv, int rows, int* RT, int* HB, int* SUB) {
    const int NT = q4_tile(rows), warps = q4_warps(NT);
    *RT = (rows + 8 * NT - 1) / (8 * NT);
    int best = 1;
    for (int hb = 2; hb <= std::min(Hkv, std::min(NT == 1 ? warps : 4, warps / *RT)); ++hb)
        if (Hkv % hb == 0 && hb * (warps / (hb * *RT)) >= best * (warps / (best * *RT))) best = hb;
    *HB = best;
    *SUB = warps / (best * *RT);
}

// SMs of the current device; without one more than any has.
int sm_count_or_most() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 1024;
    }
    return sm_count(dev);
}

// The combine kernel takes the shares of more than kQ4Few sequences from a table that the
// attention kernel leaves behind the partials (600 sequences of 100 keys: 106 us without it,
// 90 with), those of fewer from the lengths, while the attention kernel still runs (32
// sequences of 4100 keys, calls in a row: 40.1 us, with the table 40.8).
size_t q4_table_bytes(int B) { return B > kQ4Few ? 8 + (size_t)(B + 1) * sizeof(int2) : 0; }

size_t q4_workspace(int B, int Hkv, int D, int rows, int sms) {
    int RT, HB, SUB;
    q4_split(Hkv, rows, &RT, &HB, &SUB);
    // a partial for every (CTA, sequence and block of heads) that meet
    return ((size_t)sms + (size_t)(Hkv / HB) * B) * HB * rows * (D + 1) * sizeof(float) + q4_table_bytes(B);
}

bool q4_group_ok(int group_size, int D) {
    return (group_size == 32 || group_size == 64 || group_size == 128) && group_size <= D;
}

template <int D, int GS, int NT>
attn_status_t launch_q4_tiles(Q4AttnArgs a, int sms, void* workspace, size_t workspace_bytes, cudaStream_t st) {
    static std::atomic<uint64_t> attr_mask{0};   // one bit per device
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (!(attr_mask.load() & bit)) {
        const attn_status_t s = set_smem(q4_attn_kernel<D, GS, NT>, kQ4Smem);
        if (s != ATTN_OK) return s;
        attr_mask.fetch_or(bit);
    }
    q4_split(a.Hkv, a.rows, &a.RT, &a.HB, &a.SUB);
    const int U = a.HB * a.RT;
    a.nhb = a.Hkv / a.HB;
    const long long bound = (long long)a.B * (a.max_blocks + kQ4Switch) * a.nhb;    // of the cost
    if (bound >= (1LL << 31)) return ATTN_ERR_UNSUPPORTED;
    const int grid = (int)std::min<long long>(sms, bound);
    const size_t rows = ((size_t)grid + (size_t)a.nhb * a.B) * a.HB * a.rows;      // of partials
    if (!workspace || !aligned16(workspace)) return ATTN_ERR_INVALID_ARG;
    if (workspace_bytes < rows * (D + 1) * sizeof(float) + q4_table_bytes(a.B))
        return ATTN_ERR_WORKSPACE_TOO_SMALL;
    a.o_part = static_cast<float*>(workspace);
    a.lse_part = a.o_part + rows * D;
    if (a.B > kQ4Few) a.table = reinterpret_cast<int2*>(a.o_part + (rows * (D + 1) + 1) / 2 * 2);
    a.grid = grid;
    using C = Q4Cfg<D, GS, NT>;
    int ns = 0;
    while (ns < 64 && C::smem_bytes(a.HB, U, a.SUB, a.B, ns + 1) <= kQ4Smem) ++ns;
    // A multiple of SUB: a stage then holds the pages of the same warps in every round, so a warp
    // that waits for a stage's next round has itself seen the one before end.  (Otherwise a warp
    // whose pages came early would take a barrier still in the round before, for another warp's
    // late page, for one that had passed.)  Two rounds: a warp holds one page of a pair while it
    // waits for the other, SUB pages on.
    ns = ns / a.SUB * a.SUB;
    if (ns < 2 * a.SUB) return ATTN_ERR_UNSUPPORTED;
    a.nstages = ns;
    const int per_row = grid / (a.nhb * a.B);
    a.wpr = per_row <= 8 ? 1 : per_row <= 16 ? 2 : per_row <= 32 ? 4 : 8;
    attn_status_t s = launch_maybe_pdl(q4_attn_kernel<D, GS, NT>, dim3(grid), dim3(32 * (q4_warps(NT) + kQ4Producers)),
                                       C::smem_bytes(a.HB, U, a.SUB, a.B, ns), st, true, a);
    if (s != ATTN_OK) return s;
    // a sequence's pages are spread over about grid / (B nhb) CTAs: eight partials to a warp,
    // whose loads are then all in flight together
    const long long rows_out = (long long)a.B * a.max_q * a.Hq;
    return launch_maybe_pdl(q4_combine_kernel<D>, dim3((unsigned)((rows_out * a.wpr + 7) / 8)), dim3(256), 0, st, true, a);
}

template <int D, int GS>
attn_status_t launch_q4_rows(Q4AttnArgs a, int sms, void* ws, size_t ws_bytes, cudaStream_t st) {
    a.rows = a.max_q * a.group;
    return q4_tile(a.rows) == 1 ? launch_q4_tiles<D, GS, 1>(a, sms, ws, ws_bytes, st)
                                : launch_q4_tiles<D, GS, 2>(a, sms, ws, ws_bytes, st);
}

attn_status_t launch_q4(const Q4AttnArgs& a, int D, int GS, int sms, void* ws, size_t ws_bytes, cudaStream_t st) {
    if (D == 128)
        return GS == 128  ? launch_q4_rows<128, 128>(a, sms, ws, ws_bytes, st)
               : GS == 64 ? launch_q4_rows<128, 64>(a, sms, ws, ws_bytes, st)
                          : launch_q4_rows<128, 32>(a, sms, ws, ws_bytes, st);
    return GS == 64 ? launch_q4_rows<64, 64>(a, sms, ws, ws_bytes, st) : launch_q4_rows<64, 32>(a, sms, ws, ws_bytes, st);
}

template <int D, int GS>
attn_status_t launch_q4_gather_t(const Q4GatherArgs& a, int sms, cudaStream_t st) {
    // A page and head per warp.  Every block builds the tables, which is cheap for up to 64
    // sequences: then sixteen blocks to an SM, of which three are there at once and the next follows
    // where one ends (8 sequences of 16000 tokens 112 us, with two lasting blocks to an SM 125; 24
    // of 4000 86 and 94; 64 of 4000 222 and 244; 32 of 500 19 and 18), and no more, since `total`
    // may be far above the rows there are (8 of 500 under a total 64 times theirs, forward included:
    // 30.7 us, with a block for each eight pages of the total 56).  For more sequences two lasting
    // blocks (128 of 2000: 243 us, with a block for each eight pages 244; 512 of 100: 59 and 90).
    const long long items = ((long long)a.total / kPageRows + 2LL * a.B) * a.Hkv, blocks = (items + 7) / 8;
    const int grid = (int)std::max<long long>(1, std::min<long long>(blocks, (long long)sms * (a.B <= 64 ? 16 : 2)));
    q4_gather_kernel<D, GS><<<grid, 256, 2 * (a.B + 1) * sizeof(int), st>>>(a);
    return launch_status();
}

attn_status_t launch_q4_gather(const Q4GatherArgs& a, int D, int GS, int sms, cudaStream_t st) {
    if (D == 128)
        return GS == 128  ? launch_q4_gather_t<128, 128>(a, sms, st)
               : GS == 64 ? launch_q4_gather_t<128, 64>(a, sms, st)
                          : launch_q4_gather_t<128, 32>(a, sms, st);
    return GS == 64 ? launch_q4_gather_t<64, 64>(a, sms, st) : launch_q4_gather_t<64, 32>(a, sms, st);
}

// Checks of a 4-bit cache that every entry point shares.
attn_status_t check_q4_cache(const void* k_cache, const void* v_cache, const void* k_meta, const void* v_meta,
                             const int32_t* block_table, int max_blocks, int num_blocks, int block_size, int B, int Hkv,
                             int D, int group_size) {
    if (!k_cache || !v_cache || !k_meta || !v_meta || !block_table) return ATTN_ERR_INVALID_ARG;
    if (B < 0 || Hkv <= 0 || max_blocks <= 0 || num_blocks <= 0) return ATTN_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if (block_size != kPageRows || !q4_group_ok(group_size, D)) return ATTN_ERR_UNSUPPORTED;
    if (B > kDecMaxSeqs) return ATTN_ERR_UNSUPPORTED;
    if ((long long)num_blocks * block_size >= (1LL << 31)) return ATTN_ERR_UNSUPPORTED;
    if ((long long)max_blocks * block_size >= (1LL << 30)) return ATTN_ERR_UNSUPPORTED;
    if ((long long)B * max_blocks >= (1LL << 31)) return ATTN_ERR_UNSUPPORTED;   // the page prefix is 32 bits
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_meta) || !aligned16(v_meta))
        return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

attn_status_t check_append(const void* q, const void* q_out, const void* k_new, const void* v_new, const int64_t* sq,
                           const int64_t* sk, const int64_t* sv, const int32_t* cu_new, const int32_t* seqused_k,
                           const int32_t* seqused_k_out, int B, int total_new, int Hq, int Hkv) {
    if (!k_new || !v_new || !sk || !sv || !seqused_k) return ATTN_ERR_INVALID_ARG;
    if ((q != nullptr) != (q_out != nullptr) || (q && !sq)) return ATTN_ERR_INVALID_ARG;
    if (B < 0 || total_new < 0 || Hkv <= 0 || (q ? Hq <= 0 : Hq != 0)) return ATTN_ERR_INVALID_ARG;
    if (!cu_new && total_new != B) return ATTN_ERR_INVALID_ARG;
    if (seqused_k_out && seqused_k_out == seqused_k) return ATTN_ERR_INVALID_ARG;
    if ((q && (!aligned16(q) || !aligned16(q_out) || !stride8(sq, 2))) || !aligned16(k_new) || !aligned16(v_new) ||
        !stride8(sk, 2) || !stride8(sv, 2))
        return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

// Blocks of a kernel whose warp takes 1 / parts of a token; at least enough threads
// for the lengths.
attn_status_t append_grid(const RopeAppendArgs& a, unsigned* grid) {
    const long long warps = std::max<long long>((long long)a.total_new * a.parts, 1);
    const long long g = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    if (g >= (1LL << 31)) return ATTN_ERR_UNSUPPORTED;
    *grid = (unsigned)g;
    return ATTN_OK;
}

}  // namespace

attn_status_t attn_rope(const void* q, void* q_out, const void* k, void* k_out, const int64_t* strides_q,
                        const int64_t* strides_q_out, const int64_t* strides_k, const int64_t* strides_k_out, int total,
                        int Hq, int Hkv, int D, const float* cos_sin, int max_position, int rot_dim,
                        const int32_t* positions, int n_axes, const int32_t* pair_axis, int interleaved, int inverse,
                        attn_stream_t stream) {
    if (!q || !q_out || !strides_q || !strides_q_out) return ATTN_ERR_INVALID_ARG;
    if ((k != nullptr) != (k_out != nullptr) || (k && (!strides_k || !strides_k_out))) return ATTN_ERR_INVALID_ARG;
    if (total < 0 || Hq <= 0 || (k ? Hkv <= 0 : Hkv != 0)) return ATTN_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    attn_status_t s = check_rope(cos_sin, max_position, rot_dim, positions, n_axes, pair_axis, D, false);
    if (s != ATTN_OK) return s;
    if (!aligned16(q) || !aligned16(q_out) || !stride8(strides_q, 2) || !stride8(strides_q_out, 2))
        return ATTN_ERR_INVALID_ARG;
    if (k && (!aligned16(k) || !aligned16(k_out) || !stride8(strides_k, 2) || !stride8(strides_k_out, 2)))
        return ATTN_ERR_INVALID_ARG;
    if (!own_places(strides_q_out, total, Hq, D) || (k && !own_places(strides_k_out, total, Hkv, D)))
        return ATTN_ERR_INVALID_ARG;
    if ((q == q_out && !same_places(strides_q, strides_q_out, total, Hq)) ||
        (k && k == k_out && !same_places(strides_k, strides_k_out, total, Hkv)))
        return ATTN_ERR_INVALID_ARG;
    int dev = 0;
    if ((s = current_device_ok(&dev)) != ATTN_OK) return s;
    if (total == 0) return ATTN_OK;
    RopeArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = head_rows(q, strides_q);
    a.k = head_rows(k, strides_k);
    a.q_out = static_cast<__nv_bfloat16*>(q_out);
    a.k_out = static_cast<__nv_bfloat16*>(k_out);
    a.qo_row = strides_q_out[0];
    a.qo_head = strides_q_out[1];
    a.ko_row = k ? strides_k_out[0] : 0;
    a.ko_head = k ? strides_k_out[1] : 0;
    a.total = total;
    a.Hq = Hq;
    a.Hkv = k ? Hkv : 0;
    a.r = rope_table(cos_sin, max_position, rot_dim, positions, n_axes, pair_axis, interleaved, inverse);
    const int heads_at_once = 512 / D;
    a.parts = rope_parts(total, (a.Hq + a.Hkv + heads_at_once - 1) / heads_at_once, sm_count(dev));
    const long long grid = ((long long)total * a.parts + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    if (grid >= (1LL << 31)) return ATTN_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (D == 128) rope_kernel<128><<<(unsigned)grid, kRopeThreads, 0, st>>>(a);
    else rope_kernel<64><<<(unsigned)grid, kRopeThreads, 0, st>>>(a);
    return launch_status();
}

attn_status_t attn_kv_append_rope_paged(const void* q, void* q_out, const void* k_new, const void* v_new,
                                        const int64_t* strides_q, const int64_t* strides_k, const int64_t* strides_v,
                                        void* k_cache, void* v_cache, const int32_t* block_table, int max_blocks_per_seq,
                                        int num_blocks, int block_size, const int32_t* cu_seqlens_new,
                                        const int32_t* seqused_k, int32_t* seqused_k_out, int B, int total_new, int Hq,
                                        int Hkv, int D, const float* cos_sin, int max_position, int rot_dim,
                                        const int32_t* positions, int n_axes, const int32_t* pair_axis, int interleaved,
                                        int dtype, const float* descale_q, const float* descale_k,
                                        const float* descale_v, attn_stream_t stream) {
    attn_status_t s = check_append(q, q_out, k_new, v_new, strides_q, strides_k, strides_v, cu_seqlens_new, seqused_k,
                                   seqused_k_out, B, total_new, Hq, Hkv);
    if (s != ATTN_OK) return s;
    if (!k_cache || !v_cache || !block_table || max_blocks_per_seq <= 0 || num_blocks <= 0) return ATTN_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return ATTN_ERR_INVALID_ARG;
    if (dtype == ATTN_FP8_E4M3 && (!descale_k || !descale_v || (q && !descale_q))) return ATTN_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if (block_size != kPageRows) return ATTN_ERR_UNSUPPORTED;
    if ((long long)num_blocks * block_size >= (1LL << 31) || (long long)max_blocks_per_seq * block_size >= (1LL << 30))
        return ATTN_ERR_UNSUPPORTED;
    if ((s = check_rope(cos_sin, max_position, rot_dim, positions, n_axes, pair_axis, D, true)) != ATTN_OK) return s;
    if (!aligned16(k_cache) || !aligned16(v_cache)) return ATTN_ERR_INVALID_ARG;
    int dev = 0;
    if ((s = current_device_ok(&dev)) != ATTN_OK) return s;
    if (B == 0) return ATTN_OK;
    RopeAppendArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = head_rows(q, strides_q);
    a.k = head_rows(k_new, strides_k);
    a.v = head_rows(v_new, strides_v);
    a.q_out = q_out;
    a.k_cache = static_cast<uint8_t*>(k_cache);
    a.v_cache = static_cast<uint8_t*>(v_cache);
    a.descale_q = descale_q;
    a.descale_k = descale_k;
    a.descale_v = descale_v;
    a.block_table = block_table;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.cu_new = cu_seqlens_new;
    a.seqused_k = seqused_k;
    a.seqused_k_out = seqused_k_out;
    a.B = B;
    a.total_new = total_new;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.r = rope_table(cos_sin, max_position, rot_dim, positions, n_axes, pair_axis, interleaved, 0);
    const int heads_at_once = 512 / D;
    a.parts = rope_parts(total_new, (Hq + 2 * Hkv + heads_at_once - 1) / heads_at_once, sm_count(dev));
    unsigned grid;
    if ((s = append_grid(a, &grid)) != ATTN_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == ATTN_BF16) {
        if (D == 128) rope_append_kernel<128, kCacheBf16><<<grid, kRopeThreads, 0, st>>>(a);
        else rope_append_kernel<64, kCacheBf16><<<grid, kRopeThreads, 0, st>>>(a);
    } else {
        if (D == 128) rope_append_kernel<128, kCacheE4m3><<<grid, kRopeThreads, 0, st>>>(a);
        else rope_append_kernel<64, kCacheE4m3><<<grid, kRopeThreads, 0, st>>>(a);
    }
    return launch_status();
}

attn_status_t attn_kv_append_paged_q4(const void* q, void* q_out, const void* k_new, const void* v_new,
                                      const int64_t* strides_q, const int64_t* strides_k, const int64_t* strides_v,
                                      void* k_cache, void* v_cache, void* k_meta, void* v_meta,
                                      const int32_t* block_table, int max_blocks_per_seq, int num_blocks,
                                      int block_size, const int32_t* cu_seqlens_new, const int32_t* seqused_k,
                                      int32_t* seqused_k_out, int B, int total_new, int Hq, int Hkv, int D,
                                      int group_size, const float* cos_sin, int max_position, int rot_dim,
                                      const int32_t* positions, int n_axes, const int32_t* pair_axis, int interleaved,
                                      attn_stream_t stream) {
    attn_status_t s = check_append(q, q_out, k_new, v_new, strides_q, strides_k, strides_v, cu_seqlens_new, seqused_k,
                                   seqused_k_out, B, total_new, Hq, Hkv);
    if (s != ATTN_OK) return s;
    if ((s = check_q4_cache(k_cache, v_cache, k_meta, v_meta, block_table, max_blocks_per_seq, num_blocks, block_size, B,
                            Hkv, D, group_size)) != ATTN_OK)
        return s;
    if ((s = check_rope(cos_sin, max_position, rot_dim, positions, n_axes, pair_axis, D, true)) != ATTN_OK) return s;
    int dev = 0;
    if ((s = current_device_ok(&dev)) != ATTN_OK) return s;
    if (B == 0) return ATTN_OK;
    RopeAppendArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = head_rows(q, strides_q);
    a.k = head_rows(k_new, strides_k);
    a.v = head_rows(v_new, strides_v);
    a.q_out = q_out;
    a.k_cache = static_cast<uint8_t*>(k_cache);
    a.v_cache = static_cast<uint8_t*>(v_cache);
    a.k_meta = static_cast<uint16_t*>(k_meta);
    a.v_meta = static_cast<uint16_t*>(v_meta);
    a.block_table = block_table;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.cu_new = cu_seqlens_new;
    a.seqused_k = seqused_k;
    a.seqused_k_out = seqused_k_out;
    a.B = B;
    a.total_new = total_new;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.r = rope_table(cos_sin, max_position, rot_dim, positions, n_axes, pair_axis, interleaved, 0);
    const int hq = 512 / D, hv = 256 / D;      // heads at once: of q, of k or v
    a.parts = rope_parts(total_new, (Hq + hq - 1) / hq + 2 * ((Hkv + hv - 1) / hv), sm_count(dev));
    unsigned grid;
    if ((s = append_grid(a, &grid)) != ATTN_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (D == 128) {
        if (group_size == 128) rope_append_q4_kernel<128, 128><<<grid, kRopeThreads, 0, st>>>(a);
        else if (group_size == 64) rope_append_q4_kernel<128, 64><<<grid, kRopeThreads, 0, st>>>(a);
        else rope_append_q4_kernel<128, 32><<<grid, kRopeThreads, 0, st>>>(a);
    } else {
        if (group_size == 64) rope_append_q4_kernel<64, 64><<<grid, kRopeThreads, 0, st>>>(a);
        else rope_append_q4_kernel<64, 32><<<grid, kRopeThreads, 0, st>>>(a);
    }
    return launch_status();
}

attn_status_t attn_kv_gather_paged_q4(const void* k_cache, const void* v_cache, const void* k_meta, const void* v_meta,
                                      const int32_t* block_table, int max_blocks_per_seq, int num_blocks,
                                      int block_size, const int32_t* cu_seqlens, const int32_t* starts, int B, int total,
                                      int Hkv, int D, int group_size, void* k_out, void* v_out, attn_stream_t stream) {
    attn_status_t s = check_q4_cache(k_cache, v_cache, k_meta, v_meta, block_table, max_blocks_per_seq, num_blocks,
                                     block_size, B, Hkv, D, group_size);
    if (s != ATTN_OK) return s;
    if (!cu_seqlens || !k_out || !v_out || total < 0) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(k_out) || !aligned16(v_out)) return ATTN_ERR_INVALID_ARG;
    int dev = 0;
    if ((s = current_device_ok(&dev)) != ATTN_OK) return s;
    if (B == 0 || total == 0) return ATTN_OK;
    Q4GatherArgs a;
    std::memset(&a, 0, sizeof(a));
    a.k_cache = static_cast<const uint8_t*>(k_cache);
    a.v_cache = static_cast<const uint8_t*>(v_cache);
    a.k_meta = static_cast<const uint16_t*>(k_meta);
    a.v_meta = static_cast<const uint16_t*>(v_meta);
    a.block_table = block_table;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.cu = cu_seqlens;
    a.starts = starts;
    a.B = B;
    a.total = total;
    a.Hkv = Hkv;
    a.k_out = static_cast<__nv_bfloat16*>(k_out);
    a.v_out = static_cast<__nv_bfloat16*>(v_out);
    return launch_q4_gather(a, D, group_size, sm_count(dev), static_cast<cudaStream_t>(stream));
}

size_t attn_decode_q4_workspace_size(int B, int Hq, int Hkv, int D) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || D <= 0 || Hq / Hkv > 64) return 0;
    return q4_workspace(B, Hkv, D, Hq / Hkv, sm_count_or_most()) + 16;
}

attn_status_t attn_decode_paged_q4(const void* q, const void* k_cache, const void* v_cache, const void* k_meta,
                                   const void* v_meta, const int32_t* block_table, int max_blocks_per_seq,
                                   int num_blocks, int block_size, const int32_t* seqused_k, int B, int Hq, int Hkv,
                                   int D, int group_size, float softmax_scale, int window_left, float softcap, void* o,
                                   float* lse, void* workspace, size_t workspace_bytes, attn_stream_t stream) {
    if (!q || !o || !seqused_k) return ATTN_ERR_INVALID_ARG;
    attn_status_t s = check_q4_cache(k_cache, v_cache, k_meta, v_meta, block_table, max_blocks_per_seq, num_blocks,
                                     block_size, B, Hkv, D, group_size);
    if (s != ATTN_OK) return s;
    if ((s = check_score_mods(ATTN_MASK_CAUSAL, window_left, softcap)) != ATTN_OK) return s;
    if (Hq <= 0 || Hq % Hkv) return ATTN_ERR_INVALID_ARG;
    if (Hq / Hkv > 64) return ATTN_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(o)) return ATTN_ERR_INVALID_ARG;
    int dev = 0;
    if ((s = current_device_ok(&dev)) != ATTN_OK) return s;
    if (B == 0) return ATTN_OK;
    Q4AttnArgs a;
    std::memset(&a, 0, sizeof(a));
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.group = Hq / Hkv;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.max_q = 1;
    a.total_q = B;
    a.total_k = -1;
    a.k_cache = static_cast<const uint8_t*>(k_cache);
    a.v_cache = static_cast<const uint8_t*>(v_cache);
    a.k_meta = static_cast<const uint16_t*>(k_meta);
    a.v_meta = static_cast<const uint16_t*>(v_meta);
    a.block_table = block_table;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.seqused_k = seqused_k;
    a.scale = resolve_scale(softmax_scale, D);
    a.causal = 1;
    a.window = window_left < 0 ? -1 : std::min(window_left, 1 << 30);
    a.softcap = softcap;
    a.o = static_cast<__nv_bfloat16*>(o);
    a.lse = lse;
    return launch_q4(a, D, group_size, sm_count(dev), workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

// The page stream serves up to 128 query rows per KV head; above that the pages are read back
// as packed bf16 rows (exact) and the tensor-core forward runs on those.  (Groups of four, 2
// sequences of 40000 keys: 24 and 32 queries 300 and 304 us, read back 843; 16 sequences of 3700:
// 17 to 32 queries 222 to 232 us, read back 220; 16 queries 126 and 220.)
static bool q4_fwd_streams(int max_seqlen_q, int group) { return (long long)max_seqlen_q * group <= kQ4Rows; }

size_t attn_fwd_q4_workspace_size(int B, int max_seqlen_q, int Hq, int Hkv, int D, int total_k) {
    if (B <= 0 || max_seqlen_q <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || D <= 0 || total_k < 0) return 0;
    const int group = Hq / Hkv;
    if (q4_fwd_streams(max_seqlen_q, group))
        return q4_workspace(B, Hkv, D, max_seqlen_q * group, sm_count_or_most()) + 16;
    return 2 * (size_t)std::max(total_k, 1) * Hkv * D * 2 + (size_t)(B + 1) * sizeof(int) + 16;
}

attn_status_t attn_fwd_varlen_paged_q4(const void* q, const void* k_cache, const void* v_cache, const void* k_meta,
                                       const void* v_meta, const int32_t* block_table, int max_blocks_per_seq,
                                       int num_blocks, int block_size, const int32_t* cu_seqlens_q,
                                       const int32_t* seqused_k, int B, int total_q, int total_k, int max_seqlen_q,
                                       int Hq, int Hkv, int D, int group_size, float softmax_scale, int mask,
                                       int window_left, float softcap, void* o, float* lse, void* workspace,
                                       size_t workspace_bytes, attn_stream_t stream) {
    if (!q || !o || !seqused_k || !cu_seqlens_q) return ATTN_ERR_INVALID_ARG;
    attn_status_t s = check_q4_cache(k_cache, v_cache, k_meta, v_meta, block_table, max_blocks_per_seq, num_blocks,
                                     block_size, B, Hkv, D, group_size);
    if (s != ATTN_OK) return s;
    if (mask < ATTN_MASK_NONE || mask > ATTN_MASK_PATCH) return ATTN_ERR_INVALID_ARG;
    if ((s = check_score_mods(mask, window_left, softcap)) != ATTN_OK) return s;
    if (mask == ATTN_MASK_PATCH) return ATTN_ERR_UNSUPPORTED;
    if (Hq <= 0 || Hq % Hkv || total_q < 0 || total_k < 0 || max_seqlen_q < 0) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(o)) return ATTN_ERR_INVALID_ARG;
    int dev = 0;
    if ((s = current_device_ok(&dev)) != ATTN_OK) return s;
    if (B == 0 || total_q == 0 || max_seqlen_q == 0) return ATTN_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int group = Hq / Hkv;
    if (q4_fwd_streams(max_seqlen_q, group)) {
        Q4AttnArgs a;
        std::memset(&a, 0, sizeof(a));
        a.B = B;
        a.Hq = Hq;
        a.Hkv = Hkv;
        a.group = group;
        a.q = static_cast<const __nv_bfloat16*>(q);
        a.cu_q = cu_seqlens_q;
        a.max_q = max_seqlen_q;
        a.total_q = total_q;
        a.total_k = total_k;
        a.k_cache = static_cast<const uint8_t*>(k_cache);
        a.v_cache = static_cast<const uint8_t*>(v_cache);
        a.k_meta = static_cast<const uint16_t*>(k_meta);
        a.v_meta = static_cast<const uint16_t*>(v_meta);
        a.block_table = block_table;
        a.max_blocks = max_blocks_per_seq;
        a.num_blocks = num_blocks;
        a.seqused_k = seqused_k;
        a.scale = resolve_scale(softmax_scale, D);
        a.causal = mask == ATTN_MASK_CAUSAL ? 1 : 0;
        a.window = window_left < 0 ? -1 : std::min(window_left, 1 << 30);
        a.softcap = softcap;
        a.o = static_cast<__nv_bfloat16*>(o);
        a.lse = lse;
        return launch_q4(a, D, group_size, sm_count(dev), workspace, workspace_bytes, st);
    }
    if (!workspace || !aligned16(workspace)) return ATTN_ERR_INVALID_ARG;
    if (workspace_bytes < attn_fwd_q4_workspace_size(B, max_seqlen_q, Hq, Hkv, D, total_k))
        return ATTN_ERR_WORKSPACE_TOO_SMALL;
    const size_t rows = (size_t)std::max(total_k, 1) * Hkv * D;
    __nv_bfloat16* kw = static_cast<__nv_bfloat16*>(workspace);
    __nv_bfloat16* vw = kw + rows;
    int* cu_k = reinterpret_cast<int*>(vw + rows);
    Q4GatherArgs g;
    std::memset(&g, 0, sizeof(g));
    g.k_cache = static_cast<const uint8_t*>(k_cache);
    g.v_cache = static_cast<const uint8_t*>(v_cache);
    g.k_meta = static_cast<const uint16_t*>(k_meta);
    g.v_meta = static_cast<const uint16_t*>(v_meta);
    g.block_table = block_table;
    g.max_blocks = max_blocks_per_seq;
    g.num_blocks = num_blocks;
    g.lens = seqused_k;
    g.cu_out = cu_k;
    g.B = B;
    g.total = total_k;
    g.Hkv = Hkv;
    g.k_out = kw;
    g.v_out = vw;
    if ((s = launch_q4_gather(g, D, group_size, sm_count(dev), st)) != ATTN_OK) return s;
    return fwd_varlen_paged_impl(q, kw, vw, nullptr, 0, 0, 0, cu_seqlens_q, cu_k, nullptr, B, total_q, total_k,
                                 max_seqlen_q, Hq, Hkv, D, softmax_scale, mask, nullptr, window_left, softcap, ATTN_BF16,
                                 nullptr, nullptr, nullptr, o, lse, stream, 0);
}
