"""Cases of the rotary positions, the rotating KV appends and the attention over a 4-bit paged cache.

``run`` makes one pass through an operator: with ``own`` false in its plain form
(elementary torch operations in 32 bits), with ``own`` true through the entry
points of attention_paged_kv_gqa_b200.

The 4-bit cache.  A page holds 16 tokens.  Along head_dim every ``group`` values
x share a step and a zero code: with lo = min(x, 0) and hi = max(x, 0), step is
(hi - lo) / 15 rounded up to 4 significant bits (0 below 2^-100) and zero is the
integer nearest to -lo / step; the code of x is the integer nearest to x / step
(ties to even) plus zero, held within 0 .. 15, and stands for step * (code - zero),
which is a bf16 number exactly.  Tensors:
    k_cache, v_cache  uint8 [num_blocks, Hkv, 16, D / 2]
    k_meta, v_meta    int16 [num_blocks, Hkv, 16, D / group]: the bits of step as
                      bf16, whose lowest four bits are free and hold zero
Nibble order of a token's K row: dim d = 32 w + 8 c + e is nibble e of the 32-bit
word c * (D / 32) + w.  Nibble order of a page's V tile (16 tokens x D): token
t = 8 a + 2 c + h, dim d = 32 u + 8 j + r is nibble j of 16-bit piece
(((a * 8 + r) * 4 + c) * (D / 32) + u) * 2 + h.
"""
import math
import random

import torch

own = False

PAGE = 16


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the rotation of q and k before a varlen prefill or training step (16 ragged sequences, GQA 32/8)
        dict(name="rope_fwd_varlen_gqa", kind="rope", B=16, lmin=64, lmax=4096, lens_seed=3, Hq=32, Hkv=8, D=128,
             rot=128, axes=1, interleaved=False, inverse=False, packed=False),
        # its gradient for image/video tokens: three position axes, q and k views of one packed QKV tensor,
        # partial rotation, interleaved pairs
        dict(name="rope_bwd_video_axes", kind="rope", B=5, lmin=1500, lmax=3001, lens_seed=4, Hq=16, Hkv=16, D=64,
             rot=48, axes=3, interleaved=True, inverse=True, packed=True),
        # one decode step of a single short chat: latency
        dict(name="rope_one_token", kind="rope", B=1, lmin=1, lmax=1, lens_seed=1, Hq=8, Hkv=2, D=64,
             rot=64, axes=1, interleaved=False, inverse=False, packed=False),
        # a decode step of a batch: one new token a sequence into bf16 pages
        dict(name="append_rope_decode", kind="append", B=32, lmin=1, lmax=255, nmin=1, nmax=1, lens_seed=5, Hq=32,
             Hkv=8, D=128, rot=128, axes=1, interleaved=False, cache="bf16", group=0, packed=False),
        # a prefill chunk of ragged length into e4m3 pages, from a packed QKV projection
        dict(name="append_rope_chunk_e4m3", kind="append", B=7, lmin=0, lmax=700, nmin=300, nmax=2048, lens_seed=6,
             Hq=32, Hkv=8, D=128, rot=64, axes=1, interleaved=True, cache="e4m3", group=0, packed=True),
        # a decode step into 4-bit pages, and the new rows read back
        dict(name="append_q4_decode", kind="append", B=32, lmin=1, lmax=255, nmin=1, nmax=1, lens_seed=7, Hq=32,
             Hkv=8, D=128, rot=128, axes=1, interleaved=False, cache="q4", group=64, packed=False),
        # a whole ragged prefill into 4-bit pages, and the rows read back
        dict(name="append_q4_prefill", kind="append", B=9, lmin=0, lmax=40, nmin=64, nmax=4096, lens_seed=8, Hq=32,
             Hkv=8, D=128, rot=128, axes=1, interleaved=False, cache="q4", group=128, packed=True),
        # decode of a serving batch over 4-bit pages, lengths as in the library's paged decode workload
        dict(name="decode_q4_batch", kind="decode", B=32, lmin=1, lmax=8192, lens_seed=9, Hq=32, Hkv=8, D=128,
             group=128, window=-1, softcap=0.0),
        # decode of a few long contexts, fine groups
        dict(name="decode_q4_long", kind="decode", B=3, lmin=60001, lmax=70003, lens_seed=10, Hq=64, Hkv=8, D=128,
             group=32, window=-1, softcap=0.0),
        # decode of one short sequence: latency; narrow heads, softcap and a sliding window
        dict(name="decode_q4_one", kind="decode", B=1, lmin=333, lmax=333, lens_seed=1, Hq=8, Hkv=2, D=64,
             group=32, window=255, softcap=30.0),
        # a chunked-prefill step over long 4-bit contexts
        dict(name="fwd_q4_chunk", kind="fwd", B=6, lmin=2500, lmax=8192, qmin=200, qmax=512, lens_seed=11, Hq=32,
             Hkv=8, D=128, group=128, window=-1, softcap=0.0, causal=True),
        # verification of a few drafted tokens a sequence
        dict(name="fwd_q4_draft", kind="fwd", B=16, lmin=100, lmax=6000, qmin=2, qmax=4, lens_seed=12, Hq=32,
             Hkv=8, D=128, group=64, window=-1, softcap=0.0, causal=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "append", "append", "decode", "decode", "fwd"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 8])
    c = dict(kind=kind, Hq=Hkv * G, Hkv=Hkv, D=D, lens_seed=rng.randrange(1 << 20))
    rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= D])
    if kind == "rope":
        c.update(B=_log_int(rng, 1, 16), lmin=1, lmax=_log_int(rng, 1, 3000), rot=rot, axes=rng.choice([1, 1, 3]),
                 interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, packed=rng.random() < 0.5)
    elif kind == "append":
        cache = rng.choice(["bf16", "e4m3", "q4", "q4"])
        n = _log_int(rng, 1, 2000)
        c.update(B=_log_int(rng, 1, 12), lmin=0, lmax=_log_int(rng, 1, 600), nmin=1, nmax=n, rot=rot,
                 axes=rng.choice([1, 1, 3]), interleaved=rng.random() < 0.5, cache=cache,
                 group=rng.choice([g for g in (32, 64, 128) if g <= D]) if cache == "q4" else 0,
                 packed=rng.random() < 0.5)
    elif kind == "decode":
        c.update(B=_log_int(rng, 1, 32), lmin=1, lmax=_log_int(rng, 1, 8192),
                 group=rng.choice([g for g in (32, 64, 128) if g <= D]),
                 window=rng.choice([-1, -1, 0, 1000]), softcap=rng.choice([0.0, 0.0, 50.0]))
    else:
        q = _log_int(rng, 1, 400)
        c.update(B=_log_int(rng, 1, 6), lmin=q, lmax=q + _log_int(rng, 1, 6000), qmin=1, qmax=q,
                 group=rng.choice([g for g in (32, 64, 128) if g <= D]), window=rng.choice([-1, -1, 500]),
                 softcap=rng.choice([0.0, 0.0, 50.0]), causal=True)
        if rng.random() < 0.3:
            c.update(causal=False, window=-1)
    return c


def _lengths(case):
    """(keys cached before or used, new or query tokens) of each sequence."""
    r = random.Random(case["lens_seed"])
    lens = [r.randint(case["lmin"], case["lmax"]) for _ in range(case["B"])]
    lo, hi = (case["nmin"], case["nmax"]) if "nmin" in case else (case["qmin"], case["qmax"]) if "qmin" in case else (0, 0)
    return lens, [r.randint(lo, hi) for _ in range(case["B"])]


# ------------------------------------------------------------------ work
def work(case):
    lens, new = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["kind"] == "rope":
        T = sum(lens)
        return dict(bytes=T * (Hq + Hkv) * D * 4 + T * (case["rot"] * 4 + case["axes"] * 4),
                    flops=T * (Hq + Hkv) * case["rot"] * 3)
    if case["kind"] == "append":
        T = sum(new)
        io = T * (Hq + 2 * Hkv) * D * 2 + T * (case["rot"] * 4 + case["axes"] * 4)     # read
        if case["cache"] == "q4":
            held = T * Hkv * (D + 2 * 2 * (D // case["group"]))
            # written, read back, and the values of the new rows written
            io += T * Hq * D * 2 + 2 * held + T * 2 * Hkv * D * 2
        else:
            io += T * (Hq + 2 * Hkv) * D * (1 if case["cache"] == "e4m3" else 2)
        return dict(bytes=io, flops=T * (Hq + Hkv) * case["rot"] * 3)
    held = Hkv * (D + 2 * 2 * (D // case["group"]))
    w = case["window"]
    if case["kind"] == "decode":
        seen = [min(L, w + 1) if w >= 0 else L for L in lens]
        return dict(bytes=sum(seen) * held + case["B"] * Hq * (D * 4 + 4), flops=sum(seen) * 4 * D * Hq)
    pairs = keys = 0
    for L, n in zip(lens, new):
        if not case["causal"]:
            pairs, keys = pairs + n * L, keys + L
            continue
        counts = [max(0, min(L - n + i + 1, w + 1 if w >= 0 else L)) for i in range(n)]
        pairs += sum(counts)
        keys += min(L, n + w) if w >= 0 else L
    return dict(bytes=keys * held + sum(new) * Hq * (D * 4 + 4), flops=pairs * 4 * D * Hq)


# ------------------------------------------------------------------ the plain forms
def _positions(case, lens, starts, dev):
    """int32 [axes, T]: of one axis the place in the sequence, of three the frame, row and column on a 40 x 25 grid."""
    place = torch.cat([torch.arange(s, s + n, device=dev) for s, n in zip(starts, lens)])
    if case["axes"] == 1:
        return place[None].to(torch.int32).contiguous()
    return torch.stack([place // 1000, place // 25 % 40, place % 25]).to(torch.int32).contiguous()


def _table(n, rot, dev):
    """cos and sin of place * 10000^(-2 i / rot), fp32 [n, rot] (cos of the pairs, then sin)."""
    i = torch.arange(rot // 2, device=dev, dtype=torch.float64)
    a = torch.arange(n, device=dev, dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


def _rotate(x, table, positions, pair_axis, interleaved, inverse):
    """x [T, H, D] -> the rotated values in 32 bits."""
    half = table.shape[1] // 2
    i = torch.arange(half, device=x.device)
    axis = pair_axis.long() if pair_axis is not None else torch.zeros_like(i)
    place = positions.long()[axis].t()                                  # [T, half]
    c, s = table[place, i][:, None], table[place, half + i][:, None]     # [T, 1, half]
    if inverse:
        s = -s
    f = x.float()
    rotated, rest = f[..., : 2 * half], f[..., 2 * half:]
    if interleaved:
        a, b = rotated[..., 0::2], rotated[..., 1::2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = rotated[..., :half], rotated[..., half:]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, rest], -1)


def _quantise(x, group):
    """x [..., D] (bf16 values in 32 bits) -> codes [..., D], metas [..., D / group]."""
    g = x.unflatten(-1, (-1, group))
    lo, hi = g.amin(-1, keepdim=True).clamp(max=0), g.amax(-1, keepdim=True).clamp(min=0)
    width = torch.full((), 15.0, device=x.device)      # a tensor: a division, and not a product with 1 / 15
    step = ((((hi - lo) / width).view(torch.int32) + 0xFFFFF) & -0x100000).view(torch.float32)
    step = torch.where(step < 2.0 ** -100, torch.zeros_like(step), step)
    by = torch.where(step > 0, step, torch.ones_like(step))
    zero = torch.where(step > 0, torch.round(-lo / by), torch.zeros_like(step))
    code = torch.where(step > 0, torch.round(g / by), torch.zeros_like(g)) + zero
    meta = (step.view(torch.int32) >> 16) + zero.to(torch.int32)
    return code.clamp(0, 15).to(torch.uint8).flatten(-2), meta[..., 0].to(torch.int16)


def _pack(nibbles):
    """[..., n] codes in nibble order -> [..., n / 2] bytes."""
    return nibbles[..., 0::2] | (nibbles[..., 1::2] << 4)


def _unpack(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _k_nibbles(code):
    """codes [..., D] of tokens -> in the nibble order of K rows."""
    return code.unflatten(-1, (-1, 4, 8)).transpose(-3, -2).flatten(-3)


def _k_codes(k):
    """K rows [..., D / 2] bytes -> codes [..., D]."""
    n = _unpack(k)
    return n.unflatten(-1, (4, -1, 8)).transpose(-3, -2).flatten(-3)


def _v_nibbles(code):
    """codes [..., 16, D] of pages -> [..., 16 D] in the nibble order of V tiles."""
    t = code.unflatten(-1, (-1, 4, 8)).unflatten(-4, (2, 4, 2))          # a c h u j r
    n = t.dim()
    return t.permute(*range(n - 6), n - 6, n - 1, n - 5, n - 3, n - 4, n - 2).flatten(-6)


def _v_codes(v):
    """V tiles [..., 16, D / 2] bytes -> codes [..., 16, D]."""
    D = 2 * v.shape[-1]
    t = _unpack(v.flatten(-2)).unflatten(-1, (2, 8, 4, D // 32, 2, 4))    # a r c u h j
    n = t.dim()
    return t.permute(*range(n - 6), n - 6, n - 4, n - 2, n - 3, n - 1, n - 5).flatten(-6, -4).flatten(-3)


def _values(code, meta):
    """codes [..., D] and metas [..., D / group] -> what they stand for, in 32 bits."""
    m = meta.to(torch.int32)[..., None]
    step, zero = ((m & -16) << 16).view(torch.float32), (m & 15).float()
    return ((code.float().unflatten(-1, (meta.shape[-1], -1)) - zero) * step).flatten(-2)


def _slots(s):
    """(page, row in the page) of each new token."""
    p = s["places"]
    return s["block_table"].long()[s["owner"], p // PAGE], p % PAGE


def _append_plain(s, case):
    q = _rotate(s["q"], s["table"], s["positions"], s["pair_axis"], case["interleaved"], False).to(torch.bfloat16)
    k = _rotate(s["k"], s["table"], s["positions"], s["pair_axis"], case["interleaved"], False).to(torch.bfloat16)
    v = s["v"]
    page, row = _slots(s)
    used = s["lens"] + s["new"]
    if case["cache"] == "bf16":
        s["k_cache"][page, row], s["v_cache"][page, row] = k, v
        return q, s["k_cache"], s["v_cache"], used
    if case["cache"] == "e4m3":
        def e4m3(x, d):
            return (x.float() * (1 / d)).clamp(-448, 448).to(torch.float8_e4m3fn)
        for cache, x, d in ((s["k_cache"], k, s["descale_k"]), (s["v_cache"], v, s["descale_v"])):
            cache.view(torch.uint8)[page, row] = e4m3(x, d).view(torch.uint8)
        return e4m3(q, s["descale_q"]), s["k_cache"], s["v_cache"], used
    kc, km = _quantise(k.float(), case["group"])
    vc, vm = _quantise(v.float(), case["group"])
    head = torch.arange(case["Hkv"], device=q.device)[None]
    at = (page[:, None], head, row[:, None])
    s["k_cache"][at] = _pack(_k_nibbles(kc))
    s["k_meta"][at], s["v_meta"][at] = km, vm
    D = case["D"]
    halves = _pack(vc.unflatten(-1, (-1, 4, 8)).permute(0, 1, 4, 2, 3).contiguous())                 # [T, Hkv, 8 r, u, 2 bytes]
    tiles = s["v_cache"].view(-1, case["Hkv"], 2, 8, 4, D // 32, 2, 2)
    tiles[page, :, row // 8, :, row % 8 // 2, :, row % 2] = halves
    # the new rows read back
    k_back = _values(_k_codes(s["k_cache"][at]), s["k_meta"][at]).to(torch.bfloat16)
    codes = _unpack(tiles[page, :, row // 8, :, row % 8 // 2, :, row % 2]).permute(0, 1, 3, 4, 2).flatten(-3)
    v_back = _values(codes, s["v_meta"][at]).to(torch.bfloat16)
    return q, k_back, v_back, used


def _attend_plain(s, case):
    """Queries [T, Hq, D], padded to a batch, over all pages of their sequences."""
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    bt = s["block_table"].long()
    k = _values(_k_codes(s["k_cache"][bt]), s["k_meta"][bt]).transpose(1, 2).flatten(2, 3)           # [B, Hkv, keys, D]
    v = _values(_v_codes(s["v_cache"][bt]), s["v_meta"][bt]).transpose(1, 2).flatten(2, 3)
    n = s["new"].long() if case["kind"] == "fwd" else torch.ones(B, dtype=torch.int64, device=k.device)
    most = int(case["most_q"])
    i = torch.arange(most, device=k.device)
    first = torch.cumsum(n, 0) - n
    at = (first[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().view(B, most, Hkv, G, D).permute(0, 2, 3, 1, 4).flatten(2, 3)             # [B, Hkv, G most, D]
    x = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    if case["softcap"] > 0:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    x = x.view(B, Hkv, G, most, -1)
    L = s["lens"].long()
    j = torch.arange(x.shape[-1], device=k.device)
    seen = (j < L[:, None])[:, None]                                                                  # [B, 1, keys]
    if case.get("causal", True):
        diagonal = (L[:, None] - n[:, None] + i)[:, :, None]
        seen = seen & (j <= diagonal)
        if case["window"] >= 0:
            seen = seen & (j >= diagonal - case["window"])
    x = torch.where(seen[:, None, None], x, torch.full_like(x[..., :1, :1], -math.inf))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).view(B, Hkv, G, most, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = torch.log(total[..., 0]) + top[..., 0]                                                      # [B, Hkv, G, most]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, most, Hq, D).to(torch.bfloat16)
    lse = lse.reshape(B, Hq, most)
    if case["kind"] == "decode":
        return o[:, 0], lse[..., 0]
    return o.flatten(0, 1)[s["rows"]], lse.transpose(0, 1).flatten(1)[:, s["rows"]].contiguous()


# ------------------------------------------------------------------ state
def _qkv(case, T, gen, dev):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=gen, device=dev)
    x[:, Hq:Hq + Hkv] *= torch.exp(0.5 * torch.randn(1, Hkv, D, generator=gen, device=dev))    # keys have strong channels
    x = x.to(torch.bfloat16)
    if case["packed"]:
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    return x[:, :Hq].contiguous(), x[:, Hq:Hq + Hkv].contiguous(), x[:, Hq + Hkv:].contiguous()


def _pair_axis(case, dev):
    if case["axes"] == 1:
        return None
    half = case["rot"] // 2
    cut = [half // 4, half // 4 + (half - half // 4) // 2]       # a quarter for time, the rest for height and width
    return torch.tensor([sum(i >= c for c in cut) for i in range(half)], dtype=torch.int32, device=dev)


def _pages(lens, gen, dev):
    """A block table over a shuffled pool that the sequences fill about nine tenths of."""
    need = [max(1, -(-L // PAGE)) for L in lens]
    pool = sum(need) + max(2, sum(need) // 10)
    order = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pool


def _cache(pool, case, gen, dev, shift):
    """4-bit pages of N(0, 1) values whose channels differ in strength."""
    Hkv, D, g = case["Hkv"], case["D"], case["group"]
    x = torch.randn(pool, Hkv, PAGE, D, generator=gen, device=dev)
    x = (x * torch.exp(shift * torch.randn(1, Hkv, 1, D, generator=gen, device=dev))).to(torch.bfloat16).float()
    return _quantise(x, g)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    lens, new = _lengths(case)
    s = dict(case=case)
    i32 = dict(dtype=torch.int32, device=dev)
    s["lens"] = torch.tensor(lens, **i32)
    if case["kind"] == "rope":
        q, k, _ = _qkv(case, sum(lens), gen, dev)
        s.update(q=q, k=k, positions=_positions(case, lens, [0] * len(lens), dev),
                 table=_table(max(max(lens), 40), case["rot"], dev), pair_axis=_pair_axis(case, dev))
        return s
    if case["kind"] == "append":
        ends = [a + b for a, b in zip(lens, new)]
        q, k, v = _qkv(case, sum(new), gen, dev)
        table, pool = _pages(ends, gen, dev)
        s.update(q=q, k=k, v=v, new=torch.tensor(new, **i32), block_table=table,
                 positions=_positions(case, new, lens, dev), table=_table(max(max(ends), 40), case["rot"], dev),
                 pair_axis=_pair_axis(case, dev),
                 places=torch.cat([torch.arange(a, b, device=dev) for a, b in zip(lens, ends)]),
                 owner=torch.repeat_interleave(torch.arange(len(new), device=dev), torch.tensor(new, device=dev)),
                 cu_new=torch.cat([torch.zeros(1, **i32), torch.cumsum(torch.tensor(new, **i32), 0).to(torch.int32)]))
        shape = (pool, PAGE, case["Hkv"], case["D"])
        if case["cache"] == "q4":
            code, s["k_meta"] = _cache(pool, case, gen, dev, 0.5)
            s["k_cache"] = _pack(_k_nibbles(code)).contiguous()
            code, s["v_meta"] = _cache(pool, case, gen, dev, 0.0)
            s["v_cache"] = _pack(_v_nibbles(code)).view(pool, case["Hkv"], PAGE, case["D"] // 2).contiguous()
        else:
            kind = torch.bfloat16 if case["cache"] == "bf16" else torch.float8_e4m3fn
            for name in ("k_cache", "v_cache"):
                s[name] = torch.randn(shape, generator=gen, device=dev).to(torch.bfloat16).to(kind)
            for name, d in (("descale_q", 0.011), ("descale_k", 0.023), ("descale_v", 0.0125)):
                s[name] = torch.tensor([d], dtype=torch.float32, device=dev)
        return s
    table, pool = _pages(lens, gen, dev)
    code, s["k_meta"] = _cache(pool, case, gen, dev, 0.3)
    s["k_cache"] = _pack(_k_nibbles(code)).contiguous()
    code, s["v_meta"] = _cache(pool, case, gen, dev, 0.0)
    s["v_cache"] = _pack(_v_nibbles(code)).view(pool, case["Hkv"], PAGE, case["D"] // 2).contiguous()
    del code
    n = new if case["kind"] == "fwd" else [1] * case["B"]
    s["case"] = dict(case, most_q=max(n), total_k=sum(lens))
    s.update(block_table=table, new=torch.tensor(n, **i32), scale=1.0 / math.sqrt(case["D"]),
             q=torch.randn(sum(n), case["Hq"], case["D"], generator=gen, device=dev).to(torch.bfloat16),
             cu_q=torch.cat([torch.zeros(1, **i32), torch.cumsum(torch.tensor(n, **i32), 0).to(torch.int32)]))
    if case["kind"] == "fwd":
        s["rows"] = torch.cat([torch.arange(b * max(n), b * max(n) + m) for b, m in enumerate(n)]).to(dev)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    kind = case["kind"]
    if not own:
        if kind == "rope":
            return tuple(_rotate(s[x], s["table"], s["positions"], s["pair_axis"], case["interleaved"], case["inverse"]).to(torch.bfloat16)
                         for x in ("q", "k"))
        return _append_plain(s, case) if kind == "append" else _attend_plain(s, case)
    from attention_paged_kv_gqa_b200 import binding as A
    if kind == "rope":
        return A.attn_rope(s["q"], s["k"], cos_sin=s["table"], positions=s["positions"], pair_axis=s["pair_axis"],
                           interleaved=case["interleaved"], inverse=case["inverse"])
    if kind == "append":
        rope = dict(cos_sin=s["table"], positions=s["positions"], pair_axis=s["pair_axis"],
                    interleaved=case["interleaved"], cu_seqlens_new=s["cu_new"])
        if case["cache"] == "q4":
            q, used = A.attn_kv_append_paged_q4(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_meta"],
                                                s["v_meta"], s["block_table"], s["lens"], **rope)
            k, v = A.attn_kv_gather_paged_q4(s["k_cache"], s["v_cache"], s["k_meta"], s["v_meta"], s["block_table"],
                                             s["cu_new"], s["q"].shape[0], starts=s["lens"])
            return q, k, v, used
        if case["cache"] == "e4m3":
            rope.update(descale_q=s["descale_q"], descale_k=s["descale_k"], descale_v=s["descale_v"])
        q, used = A.attn_kv_append_rope_paged(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"],
                                              s["lens"], **rope)
        return q, s["k_cache"], s["v_cache"], used
    if kind == "decode":
        return A.attn_decode_paged_q4(s["q"], s["k_cache"], s["v_cache"], s["k_meta"], s["v_meta"], s["block_table"],
                                      s["lens"], scale=s["scale"], window_left=case["window"], softcap=case["softcap"])
    return A.attn_fwd_varlen_paged_q4(s["q"], s["k_cache"], s["v_cache"], s["k_meta"], s["v_meta"],
                                      block_table=s["block_table"], cu_seqlens_q=s["cu_q"],
                                      max_seqlen_q=case["most_q"], seqused_k=s["lens"], total_k=case["total_k"],
                                      mask=A.MASK_CAUSAL if case["causal"] else A.MASK_NONE, scale=s["scale"],
                                      window_left=case["window"], softcap=case["softcap"])


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _turn64(x, s, case, sign):
    """The rotation as a product with e^(i angle): pairs as complex numbers."""
    half = case["rot"] // 2
    axis = [0] * half if s["pair_axis"] is None else s["pair_axis"].tolist()
    t = s["table"].double()
    turn = torch.stack([torch.complex(t[s["positions"][a].long(), i], sign * t[s["positions"][a].long(), half + i])
                        for i, a in enumerate(axis)], 1)[:, None]
    y = x.double().clone()
    first = slice(0, 2 * half, 2) if case["interleaved"] else slice(0, half)
    second = slice(1, 2 * half, 2) if case["interleaved"] else slice(half, 2 * half)
    z = torch.complex(y[..., first].clone(), y[..., second].clone()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _held64(x, group):
    """What the 4-bit form of the values x stands for."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    low = torch.minimum(g.min(-1, keepdim=True).values, torch.zeros((), dtype=x.dtype, device=x.device))
    high = torch.maximum(g.max(-1, keepdim=True).values, torch.zeros((), dtype=x.dtype, device=x.device))
    part, power = torch.frexp((high - low) / torch.full((), 15.0, dtype=x.dtype, device=x.device))
    step = torch.ldexp(torch.ceil(part * 16) / 16, power)
    step = step.where(step >= 2.0 ** -100, torch.zeros_like(step))
    held = step.where(step > 0, torch.ones_like(step))
    zero = torch.round(-low / held)
    return ((torch.round(g / held) + zero).clamp(0, 15) - zero).mul(step).reshape(x.shape)


def _read64(s, b, L):
    """K and V [L, Hkv, D] of sequence b, nibble by nibble from the page layout."""
    case = s["case"]
    D, Hkv = case["D"], case["Hkv"]
    dev = s["q"].device
    t, d = torch.arange(L, device=dev), torch.arange(D, device=dev)
    page, row = s["block_table"][b].long()[t // PAGE], t % PAGE
    out = []
    for name in ("k", "v"):
        tiles = s[name + "_cache"].reshape(-1, Hkv, PAGE * D // 2)[page]                    # [L, Hkv, bytes]
        if name == "k":
            nib = row[:, None] * D + ((d % 32 // 8) * (D // 32) + d // 32) * 8 + d % 8
        else:
            a, c, h = row[:, None] // 8, row[:, None] % 8 // 2, row[:, None] % 2
            nib = ((((a * 8 + d % 8) * 4 + c) * (D // 32) + d // 32) * 2 + h) * 4 + d % 32 // 8
        byte = torch.gather(tiles, 2, (nib // 2)[:, None].expand(L, Hkv, D)).long()
        code = (byte >> (4 * (nib % 2))[:, None]) % 16
        m = s[name + "_meta"][page, :, row].int().repeat_interleave(case["group"], 2)       # [L, Hkv, D]
        step = (m & 0xFFF0).to(torch.int16).view(torch.bfloat16)
        out.append((code - m % 16).double() * step.double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "rope":
        return tuple(_turn64(s[x], s, case, -1.0 if case["inverse"] else 1.0) for x in ("q", "k"))
    if kind == "append":
        q = _turn64(s["q"], s, case, 1.0)
        k = _turn64(s["k"], s, case, 1.0).to(torch.bfloat16).double()
        v = s["v"].double()
        used = s["lens"] + s["new"]
        if case["cache"] == "q4":
            return q, _held64(k, case["group"]), _held64(v, case["group"]), used
        d = [s["descale_" + x].double() for x in "qkv"] if case["cache"] == "e4m3" else [1.0, 1.0, 1.0]
        caches = []
        for name, x, u in (("k_cache", k, d[1]), ("v_cache", v, d[2])):
            c = s[name].to(torch.float32).double()
            c[s["block_table"][s["owner"], s["places"] // PAGE].long(), s["places"] % PAGE] = x / u
            caches.append(c)
        return q / d[0], caches[0], caches[1], used
    G = case["Hq"] // case["Hkv"]
    outs, sums, first = [], [], 0
    for b in range(case["B"]):
        L, n = int(s["lens"][b]), int(s["new"][b])
        k, v = _read64(s, b, L)
        q = s["q"][first:first + n].double()
        first += n
        at = torch.arange(L - n, L, device=q.device)[:, None]
        j = torch.arange(L, device=q.device)[None]
        if kind == "fwd" and not case["causal"]:
            hidden = torch.zeros(n, L, dtype=torch.bool, device=q.device)
        else:
            hidden = (j > at) | (j < at - case["window"] if case["window"] >= 0 else j < 0)
        o = torch.zeros(n, case["Hq"], case["D"], dtype=torch.float64, device=q.device)
        lse = torch.zeros(case["Hq"], n, dtype=torch.float64, device=q.device)
        for h in range(case["Hkv"]):
            x = torch.einsum("ngd,ld->gnl", q[:, h * G:(h + 1) * G], k[:, h]) / math.sqrt(case["D"])
            if case["softcap"] > 0:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            x = x.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(x, -1)
            w = torch.exp(x - z.clamp(min=-1e300)[..., None])
            lse[h * G:(h + 1) * G] = z
            o[:, h * G:(h + 1) * G] = torch.einsum("gnl,ld->ngd", w, v[:, h])
        outs.append(o)
        sums.append(lse)
    o, lse = torch.cat(outs), torch.cat(sums, 1)
    return (o, lse) if kind == "fwd" else (o, lse.t().contiguous())
