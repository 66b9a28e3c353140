"""What is measured of the paged, quantised KV cache: writing tokens into it,
reading them back, and attention of new tokens over it.

The operators, for the newest ``n_b`` tokens of each sequence ``b`` of a batch
(``seq_lens`` counts them in):

write   rotate each new key and value vector by the Sylvester Hadamard matrix,
        quantise groups of 32 to b bits with one fp16 scale each, and store them
        in the sequence's pages; then read the same tokens back (a chunk of a
        prompt, whose attention runs on the values the cache stands for).
read    the whole sequences back out of their pages.
attend  causal attention of the new tokens' queries over the whole sequence in
        the cache, with grouped heads and an optional sliding window.
decode  one step of a serving loop: write the new tokens, then attend.

The cache is int32 ``[pages, kv_heads, page_size / 32, words]``: one record per
32 tokens of one head, holding K codes, K scales, V codes and V scales.
"""
import math
import random

import numpy as np
import torch

own = False

TILE = 32


# ------------------------------------------------------------------ the cases

def _case(name, op, dtype, batch, length, new, q_heads, kv_heads, head_dim, k_bits, v_bits, page, ragged, window=0):
    return dict(name=name, op=op, dtype=dtype, batch=batch, length=length, new=new, q_heads=q_heads,
                kv_heads=kv_heads, head_dim=head_dim, k_bits=k_bits, v_bits=v_bits, page=page, ragged=ragged,
                window=window)


def listed():
    return [
        # one user's chat turn, short context: launch latency is all there is (Llama-3-70B's heads)
        _case("attend 1x509", "attend", "float16", 1, 509, 1, 64, 8, 128, 4, 4, 64, False),
        # one user with a long document: the cache of one sequence split over the whole GPU
        _case("attend 1x131072", "attend", "float16", 1, 131072, 1, 64, 8, 128, 4, 4, 256, False),
        # a serving batch of uneven conversations
        _case("attend 64x<=4096", "attend", "bfloat16", 64, 4096, 1, 64, 8, 128, 4, 4, 64, True),
        # the largest: many long contexts, keys held wider than values
        _case("attend 32x<=24576 k6v4", "attend", "bfloat16", 32, 24576, 1, 64, 8, 128, 6, 4, 256, True),
        # small heads, 8-bit cache, local layers that see the last 1000 tokens
        _case("attend 48x<=6000 d64 window", "attend", "float16", 48, 6000, 1, 32, 8, 64, 8, 8, 32, True, 1000),
        # verification of drafted tokens: five queries per sequence, large heads, three-bit values
        _case("attend 12x<=5000 d256 drafts", "attend", "bfloat16", 12, 5000, 5, 6, 2, 256, 5, 3, 64, True),
        # one step of a decoding loop: write the token, then attend
        _case("decode 16x<=8192", "decode", "float16", 16, 8192, 1, 64, 8, 128, 4, 4, 128, True),
        # the write of one decode step
        _case("write 8x1", "write", "float16", 8, 700, 1, 64, 8, 128, 4, 4, 64, True),
        # uneven chunks of prompts, rotated K next to V in odd widths
        _case("write 5x<=1501 k5v3", "write", "bfloat16", 5, 4000, 1501, 32, 8, 128, 5, 3, 64, True),
        # one long prompt
        _case("write 1x32768", "write", "bfloat16", 1, 32768, 32768, 64, 8, 128, 4, 4, 256, False),
        # short contexts fetched again, small heads, two bits
        _case("read 7x<=333 d64", "read", "float16", 7, 333, 333, 16, 4, 64, 2, 2, 32, True),
        # a prompt's whole context fetched for the next chunk's attention
        _case("read 4x<=16384", "read", "bfloat16", 4, 16384, 16384, 64, 8, 128, 4, 4, 128, True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "decode", "write", "read"])
    head_dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 12, 16])
    k_bits, v_bits = rng.choice([2, 3, 4, 4, 5, 6, 8]), rng.choice([2, 3, 4, 4, 5, 6, 8])
    page = rng.choice([32, 64, 128, 256])
    batch = _log_int(rng, 1, 64)
    drafts = rng.choice([1, 1, 1, 2, 3, 5, 8])
    # at most 2^18 tokens of 8 heads of 128, about two thirds of the largest listed case; fewer for many rows
    most = min(131072, (1 << 28) // (batch * kv_heads * head_dim) * 16 // max(16, drafts * group))
    if op in ("write", "read"):
        most = min(most, (1 << 25) // (batch * kv_heads * head_dim))
    length = _log_int(rng, 1, max(2, most))
    if op in ("attend", "decode"):
        new = min(length, drafts)
    else:
        new = length if op == "read" else _log_int(rng, 1, length)
    window = rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]) if op in ("attend", "decode") else 0
    c = _case("", op, rng.choice(["float16", "bfloat16"]), batch, length, new, kv_heads * group, kv_heads, head_dim,
              k_bits, v_bits, page, rng.random() < 0.7, window)
    del c["name"]
    return c


def _lengths(case):
    """Tokens in the cache and new ones of each sequence: part of the case, whatever the seed."""
    B, L, n = case["batch"], case["length"], case["new"]
    if not case["ragged"]:
        return [L] * B, [n] * B
    r = random.Random(B * 1000003 + L * 7 + n)
    lens = [L] + [r.randint(max(1, L // 16), L) for _ in range(B - 1)]
    if case["op"] == "read":
        return lens, list(lens)
    if case["op"] == "write":
        return lens, [min(l, r.randint(max(1, n // 4), n)) for l in lens]
    return lens, [min(l, n) for l in lens]


def work(case):
    lens, news = _lengths(case)
    D, Hk, Hq = case["head_dim"], case["kv_heads"], case["q_heads"]
    T, per = sum(news), D * (case["k_bits"] + case["v_bits"]) / 8 + 4 * (D // 32)
    rotation = 2 * T * Hk * D * int(math.log2(D))
    if case["op"] == "write":
        return {"bytes": T * Hk * (8 * D + per), "flops": 2 * rotation + 8 * T * Hk * D}
    if case["op"] == "read":
        return {"bytes": T * Hk * (4 * D + per), "flops": rotation + 4 * T * Hk * D}
    W = case["window"]
    seen, pairs = 0, 0
    for l, n in zip(lens, news):
        first = max(0, l - n - W + 1) if W else 0
        seen += l - first
        pairs += sum(min(p + 1, W) if W else p + 1 for p in range(l - n, l))
    total = {"bytes": seen * Hk * per + T * Hq * (4 * D + 4), "flops": 4.0 * D * Hq * pairs}
    if case["op"] == "decode":
        total["bytes"] += T * Hk * 4 * D
        total["flops"] += rotation
    return total


# ---------------------------------------------------------- the records' layout
# A record is 32 lane streams of K codes, K scales [t % 8][t / 8][group], 32
# lane streams of V codes and V scales [j][group][t / 8][u] (t = 8 tt + 2 j + u).
# Streams are made of units of 8 codes (b bytes, little-endian) and stored in
# chunks, chunk c of lane l at c * 32 + l.

WIDE_ORDER = [0, 1, 4, 5, 2, 3, 6, 7]  # K codes of 5 bits and more: the dims a unit's slots hold


def _chunk(D, b):
    return math.gcd(16, D * b // 16)


def _parts(D, kb, vb):
    a, s, v = 4 * D * kb, 2 * D, 4 * D * vb
    return a, s, v, s


def _to_bytes(codes, b):  # [..., 8] -> [..., b]
    x = (codes << (b * torch.arange(8, device=codes.device))).sum(-1)
    return x.unsqueeze(-1).view(torch.uint8)[..., :b]


def _to_codes(by, b):  # [..., b] -> [..., 8]
    wide = torch.nn.functional.pad(by, (0, 8 - b)).view(torch.int64)
    return (wide >> (b * torch.arange(8, device=by.device))) & ((1 << b) - 1)


def _pack_units(codes, D, b):
    """codes int64 [..., 32 lanes, D / 8 units, 8] -> bytes [..., 4 D b]."""
    by = _to_bytes(codes, b)
    c = _chunk(D, b)
    by = by.reshape(*by.shape[:-3], 32, D * b // 8 // c, c)
    return by.transpose(-3, -2).reshape(*by.shape[:-3], 4 * D * b)


def _unpack_units(by, D, b):
    """bytes [..., 4 D b] -> codes int64 [..., 32 lanes, D / 8 units, 8]."""
    c = _chunk(D, b)
    by = by.reshape(*by.shape[:-1], D * b // 8 // c, 32, c).transpose(-3, -2)
    return _to_codes(by.reshape(*by.shape[:-3], 32, D // 8, b), b)


def _k_to_units(codes, D, b):
    """[..., 32 tokens, D] -> [..., 32 lanes, D / 8, 8]."""
    lead = codes.shape[:-2]
    x = codes.reshape(*lead, 4, 8, D // 32, 4, 8)  # tt, r, g, j, i
    n = len(lead)
    x = x.permute(*range(n), n + 1, n + 3, n, n + 2, n + 4).reshape(*lead, 32, D // 8, 8)
    return x[..., WIDE_ORDER] if b >= 5 else x


def _k_from_units(x, D, b):
    lead = x.shape[:-3]
    if b >= 5:
        x = x[..., WIDE_ORDER]  # its own inverse
    n = len(lead)
    x = x.reshape(*lead, 8, 4, 4, D // 32, 8)  # r, j, tt, g, i
    return x.permute(*range(n), n + 2, n, n + 3, n + 1, n + 4).reshape(*lead, 32, D)


def _v_to_units(codes, D):
    lead = codes.shape[:-2]
    n = len(lead)
    x = codes.reshape(*lead, 4, 4, 2, D // 64, 2, 8, 4)  # tt, j, u, h, l2, r, i
    x = x.permute(*range(n), n + 5, n + 1, n, n + 2, n + 3, n + 4, n + 6)
    return x.reshape(*lead, 32, D // 8, 8)


def _v_from_units(x, D):
    lead = x.shape[:-3]
    n = len(lead)
    x = x.reshape(*lead, 8, 4, 4, 2, D // 64, 2, 4)  # r, j, tt, u, h, l2, i
    return x.permute(*range(n), n + 2, n + 1, n + 3, n + 4, n + 5, n, n + 6).reshape(*lead, 32, D)


def _records(k_codes, k_scales, v_codes, v_scales, D, kb, vb):
    """Codes [..., 32, D] and scales [..., 32, D / 32] of K and V -> records int32 [..., words]."""
    lead, n, G = k_codes.shape[:-2], k_codes.dim() - 2, D // 32
    ks = k_scales.reshape(*lead, 4, 8, G).transpose(-3, -2)
    vs = v_scales.reshape(*lead, 4, 4, 2, G).permute(*range(n), n + 1, n + 3, n, n + 2)
    parts = [_pack_units(_k_to_units(k_codes, D, kb), D, kb),
             ks.reshape(*lead, D).contiguous().view(torch.uint8),
             _pack_units(_v_to_units(v_codes, D), D, vb),
             vs.reshape(*lead, D).contiguous().view(torch.uint8)]
    return torch.cat(parts, dim=-1).view(torch.int32)


def _from_records(rec, D, kb, vb):
    """Records int32 [..., words] -> rotated K and V, float32 [..., 32, D]."""
    by = rec.contiguous().view(torch.uint8)
    kc, ks, vc, vs = torch.split(by, _parts(D, kb, vb), dim=-1)
    lead, n, G = by.shape[:-1], by.dim() - 1, D // 32
    ks = ks.contiguous().view(torch.float16).reshape(*lead, 8, 4, G).transpose(-3, -2).reshape(*lead, 32, G, 1)
    vs = vs.contiguous().view(torch.float16).reshape(*lead, 4, G, 4, 2).permute(*range(n), n + 2, n, n + 3, n + 1)
    vs = vs.reshape(*lead, 32, G, 1)
    k = _k_from_units(_unpack_units(kc, D, kb), D, kb).float() - 2 ** (kb - 1)
    v = _v_from_units(_unpack_units(vc, D, vb), D).float() - 2 ** (vb - 1)
    k = k.reshape(*lead, 32, G, 32) * ks.float()
    v = v.reshape(*lead, 32, G, 32) * vs.float()
    return k.reshape(*lead, 32, D), v.reshape(*lead, 32, D)


def _hadamard(D, device, dtype=torch.float32):
    i = torch.arange(D, device=device)
    x = i[:, None] & i[None, :]
    x = x ^ (x >> 4)
    x = x ^ (x >> 2)
    x = x ^ (x >> 1)
    return (1 - 2 * (x & 1)).to(dtype)


def _butterflies(x):
    """H_D x in single precision, in the order that defines the codes (strides 1, 2, ..., D / 2, each sum
    rounded): a code next to a border is decided by these roundings, so every form takes the same ones."""
    D, st = x.shape[-1], 1
    while st < D:
        y = x.reshape(*x.shape[:-1], D // (2 * st), 2, st)
        x = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], dim=-2).reshape(x.shape)
        st *= 2
    return x


def _quantise(u, b):
    """Rotated vectors u float32 [..., D] -> codes int64 [..., D] and fp16 scales [..., D / 32]."""
    z = 2 ** (b - 1)
    g = u.reshape(*u.shape[:-1], u.shape[-1] // 32, 32)
    # divided by a tensor: a number would be applied as a product with its reciprocal
    s = (g.abs().amax(-1) / torch.full((), z - 1.0, device=u.device)).to(torch.float16)
    inv = torch.where(s == 0, torch.zeros_like(g[..., 0]), 1 / s.float())
    q = (torch.round(g * inv.unsqueeze(-1)) + z).clamp(0, 2 * z - 1)
    return q.reshape(u.shape).to(torch.int64), s


# ------------------------------------------------------------------ the inputs

def prepare(case, seed):
    dev, dt = torch.device("cuda"), getattr(torch, case["dtype"])
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    D, Hk, Hq, kb, vb, page = (case[k] for k in ("head_dim", "kv_heads", "q_heads", "k_bits", "v_bits", "page"))
    lens, news = _lengths(case)
    B, T = len(lens), sum(news)
    used = [-(-l // page) for l in lens]
    pages = sum(used) + 3

    def randn(*shape):
        return torch.randn(*shape, device=dev, generator=gen)

    # what earlier steps left in the pages: rotated vectors are close to normal,
    # with a spread over heads; slots behind a sequence's end hold old tokens
    def content(b):
        u = randn(pages, Hk, page // TILE, TILE, D) * math.sqrt(D)
        u *= torch.exp(0.3 * randn(1, Hk, 1, 1, 1))
        return _quantise(u, b)

    kc, ks = content(kb)
    vc, vs = content(vb)
    cache = _records(kc, ks, vc, vs, D, kb, vb)
    del kc, ks, vc, vs

    order = torch.randperm(pages, device=dev, generator=gen).to(torch.int32)
    table = torch.zeros(B, max(used), dtype=torch.int32, device=dev)
    row = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(used, device=dev))
    starts = torch.tensor(np.cumsum([0] + used[:-1]), device=dev)
    col = torch.arange(sum(used), device=dev) - starts[row]
    table[row, col] = order[:sum(used)]

    def tokens(heads):  # a view of a fused projection's rows, as a model's attention layer has it
        return randn(T, heads * D).to(dt).view(T, heads, D)

    qkv = torch.cat([tokens(Hq), tokens(Hk) * torch.exp(0.3 * randn(1, Hk, 1)).to(dt), tokens(Hk)], dim=1)
    return {
        "case": dict(case), "cache": cache, "table": table,
        "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
        "cu": torch.tensor(np.cumsum([0] + news), device=dev).to(torch.int32),
        "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hk], "v": qkv[:, Hq + Hk:],
        # a serving loop's own buffers and its handle of the cache (made on the first pass)
        "out": torch.empty(T, Hq, D, dtype=dt, device=dev), "lse": torch.empty(T, Hq, device=dev),
        "k_back": torch.empty(T, Hk, D, dtype=dt, device=dev), "v_back": torch.empty(T, Hk, D, dtype=dt, device=dev),
        "longest": max(lens), "most_new": max(news), "handles": {},
    }


# ------------------------------------------------------------------ the passes

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    import mixed_bitwidth_weight_b200 as lib
    c, h = st["case"], st["handles"]
    if not h:  # the cache's handle and the workspace: made once, kept as long as the cache
        h["cache"] = lib.KVCache(st["cache"], c["page"], c["kv_heads"], c["head_dim"], c["k_bits"], c["v_bits"])
        h["ws"] = lib.kv_workspace(h["cache"], c["q_heads"])
    cache, batch = h["cache"], lib.KVBatch(st["table"], st["lens"], st["cu"])
    if c["op"] in ("write", "decode"):
        lib.qgemm_kv_append(st["k"], st["v"], cache, batch)
    if c["op"] in ("write", "read"):
        lib.qgemm_kv_gather(cache, batch, st["k_back"], st["v_back"])
        return {"k": st["k_back"], "v": st["v_back"]}
    lib.qgemm_kv_attend(st["q"], cache, batch, st["out"], h["ws"], window=c["window"], lse=st["lse"])
    return {"out": st["out"], "lse": st["lse"]}


def _rows(st):
    """For each new token: its sequence and its position there."""
    cu, lens = st["cu"].long(), st["lens"].long()
    t = torch.arange(st["q"].shape[0], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, lens[b] - cu[b + 1] + t


def _places(D, kb, vb, dev):
    """[32, n]: the byte places, in a record, of each token slot's n bytes: its K units (group, j), K scales,
    V units (r, pair of groups) and V scales."""
    G = D // 32

    def stream(lane, unit, b):  # -> [32, units, b]
        y = unit.unsqueeze(-1) * b + torch.arange(b, device=dev)
        c = _chunk(D, b)
        return ((y // c * 32 + lane.unsqueeze(-1)) * c + y % c).reshape(32, -1)

    def two(at):  # the two bytes of each fp16 scale
        return (2 * at.unsqueeze(-1) + torch.arange(2, device=dev)).reshape(32, -1)

    t = torch.arange(TILE, device=dev)[:, None, None]
    g, j, r, h = (torch.arange(n, device=dev) for n in (G, 4, 8, D // 64))
    flat = t[:, :, 0]
    k = stream((4 * (t % 8) + j + 0 * g[:, None]).reshape(32, -1), (t // 8 * G + g[:, None] + 0 * j).reshape(32, -1), kb)
    ks = two((flat % 8 * 4 + flat // 8) * G + g)
    v = stream((4 * r[:, None] + t // 2 % 4 + 0 * h).reshape(32, -1),
               ((t // 8 * 2 + t % 2) * (D // 64) + h + 0 * r[:, None]).reshape(32, -1), vb)
    vs = two(((flat // 2 % 4 * G + g) * 4 + flat // 8) * 2 + flat % 2)
    first = np.cumsum((0,) + _parts(D, kb, vb)).tolist()
    return torch.cat([k + first[0], ks + first[1], v + first[2], vs + first[3]], dim=1)


def _token_addresses(st):
    """[T, heads, n]: where in the cache's bytes the new tokens' bytes are."""
    c = st["case"]
    D, page, Hk = c["head_dim"], c["page"], c["kv_heads"]
    b, pos = _rows(st)
    tiles, size = page // TILE, 4 * st["cache"].shape[-1]
    heads = torch.arange(Hk, device=pos.device)
    rec = (st["table"][b, pos // page].long()[:, None] * Hk + heads) * tiles + (pos % page // TILE)[:, None]
    return (rec * size)[..., None] + _places(D, c["k_bits"], c["v_bits"], pos.device)[pos % TILE][:, None, :]


def _write_plain(st):
    c = st["case"]
    D, kb, vb = c["head_dim"], c["k_bits"], c["v_bits"]
    kc, ks = _quantise(_butterflies(st["k"].float()), kb)
    vc, vs = _quantise(_butterflies(st["v"].float()), vb)
    kc = kc.reshape(*kc.shape[:2], D // 8, 8)
    kc = kc[..., WIDE_ORDER] if kb >= 5 else kc
    vc = vc.reshape(*vc.shape[:2], D // 64, 2, 8, 4).permute(0, 1, 4, 2, 3, 5).reshape(*vc.shape[:2], D // 8, 8)
    mine = torch.cat([_to_bytes(kc, kb).flatten(2), ks.view(torch.uint8), _to_bytes(vc, vb).flatten(2),
                      vs.view(torch.uint8)], dim=2)
    st["cache"].view(torch.uint8).view(-1)[_token_addresses(st)] = mine


def _read_tokens(st):
    c = st["case"]
    D, kb, vb = c["head_dim"], c["k_bits"], c["v_bits"]
    by = st["cache"].view(torch.uint8).view(-1)[_token_addresses(st)]      # [T, heads, n]
    kc, ks, vc, vs = torch.split(by, (D * kb // 8, D // 16, D * vb // 8, D // 16), dim=2)
    lead = by.shape[:2]
    kc, vc = _to_codes(kc.reshape(*lead, D // 8, kb), kb), _to_codes(vc.reshape(*lead, D // 8, vb), vb)
    kc = kc[..., WIDE_ORDER] if kb >= 5 else kc
    vc = vc.reshape(*lead, 8, D // 64, 2, 4).permute(0, 1, 3, 4, 2, 5)

    def back(codes, scales, b):
        x = codes.reshape(*lead, D // 32, 32).float() - 2 ** (b - 1)
        x = x * scales.contiguous().view(torch.float16).float().unsqueeze(-1)
        return (x.reshape(*lead, D) @ (_hadamard(D, x.device) / D)).to(st["k"].dtype)

    return {"k": back(kc, ks, kb), "v": back(vc, vs, vb)}


def _context(st):
    """K and V of every sequence, rotated back, float32 [B, heads, tokens, D] (tokens: whole pages)."""
    c = st["case"]
    D, Hk, B = c["head_dim"], c["kv_heads"], c["batch"]
    rec = st["cache"][st["table"].long()]                                  # [B, pages, heads, tiles, words]
    k, v = _from_records(rec.transpose(1, 2), D, c["k_bits"], c["v_bits"])
    had = _hadamard(D, k.device) / D
    return (k.reshape(B, Hk, -1, D) @ had), (v.reshape(B, Hk, -1, D) @ had)


def _run_plain(st):
    c = st["case"]
    if c["op"] in ("write", "decode"):
        _write_plain(st)
    if c["op"] == "write":  # only the new tokens' records
        return _read_tokens(st)
    if c["op"] == "read":
        k, v = _context(st)
        b, pos = _rows(st)
        return {"k": k[b, :, pos].to(st["q"].dtype), "v": v[b, :, pos].to(st["q"].dtype)}
    return _attend_plain(st)


def _attend_plain(st):
    c = st["case"]
    D, Hk, Hq, B, n = c["head_dim"], c["kv_heads"], c["q_heads"], c["batch"], st["most_new"]
    G = Hq // Hk
    cu, lens = st["cu"].long(), st["lens"].long()
    k, v = _context(st)
    L = k.shape[2]
    new = cu[1:] - cu[:-1]
    i = torch.arange(n, device=cu.device)
    rows = (cu[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)             # [B, n], the last ones padding
    q = st["q"][rows].float().reshape(B, n, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, n * G, D)
    score = (q @ k.transpose(-1, -2)) / math.sqrt(D)
    pos = (lens - new)[:, None] + i                                        # [B, n]
    t = torch.arange(L, device=cu.device)
    seen = t <= pos[..., None]
    if c["window"]:
        seen &= t > pos[..., None] - c["window"]
    seen = seen[:, None, :, None, :].expand(B, Hk, n, G, L).reshape(B, Hk, n * G, L)
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = top + torch.log(total)
    out = out.reshape(B, Hk, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)
    lse = lse.reshape(B, Hk, n, G).permute(0, 2, 1, 3).reshape(B, n, Hq)
    b, _ = _rows(st)
    at = torch.arange(st["q"].shape[0], device=cu.device) - cu[b]
    return {"out": out[b, at].to(st["q"].dtype), "lse": lse[b, at]}


# ------------------------------------------------------------- in 64 bits, apart

def _exact_side(by, t, D, b, keys):
    """One part of records by [..., bytes] -> rotated values, float64 [..., len(t), D], written from the
    layout's definition: for each token and dim its lane, unit and slot, and from them its bits."""
    d = torch.arange(D, device=by.device)[None, :]
    t = t[:, None]
    G = D // 32
    if keys:
        lane, unit, slot = 4 * (t % 8) + d % 32 // 8, t // 8 * G + d // 32, (d % 8).expand(t.shape[0], D)
        if b >= 5:
            slot = torch.tensor([0, 1, 4, 5, 2, 3, 6, 7], device=by.device)[slot]
        at = (t % 8 * 4 + t // 8) * G + d // 32
    else:
        lane = 4 * (d % 32 // 4) + t // 2 % 4
        unit = (t // 8 * 2 + t % 2) * (D // 64) + d // 64
        slot = (d // 32 % 2 * 4 + d % 4).expand(t.shape[0], D)
        at = ((t // 2 % 4 * G + d // 32) * 4 + t // 8) * 2 + t % 2
    bit = slot * b
    inner = unit * b + bit // 8                       # byte of the lane's stream
    ch = [n for n in (16, 8, 4) if D * b // 16 % n == 0][0]
    place = lambda y: (y // ch * 32 + lane) * ch + y % ch  # noqa: E731
    low = by[..., place(inner)].long()
    high = by[..., place((inner + 1).clamp(max=D * b // 8 - 1))].long()
    code = ((low | (high << 8)) >> (bit % 8)) & ((1 << b) - 1)
    scale = by[..., 4 * D * b:4 * D * b + 2 * D].contiguous().view(torch.float16)[..., at]
    return (code - 2 ** (b - 1)).double() * scale.double()


def _exact_sequence(st, b, lo, hi, keys):
    """Values of tokens lo .. hi of sequence b, float64 [heads, hi - lo, D], rotated back."""
    c = st["case"]
    D, kb, vb, page = c["head_dim"], c["k_bits"], c["v_bits"], c["page"]
    dev = st["cache"].device
    first, last = lo // TILE, -(-hi // TILE)
    tile = torch.arange(first, last, device=dev)
    rec = st["cache"][st["table"][b, tile // (page // TILE)].long(), :, tile % (page // TILE)]
    by = rec.contiguous().view(torch.uint8)
    cut = 4 * D * kb + 2 * D
    part = by[..., :cut] if keys else by[..., cut:]
    x = _exact_side(part, torch.arange(TILE, device=dev), D, kb if keys else vb, keys)
    x = x.transpose(0, 1).reshape(c["kv_heads"], -1, D) @ _hadamard(D, dev, torch.float64) / D
    return x[:, lo - first * TILE:hi - first * TILE]


def _exact_quantised(x, b):
    """The values a written vector x [..., D] stands for, float64. The codes are defined by single-precision steps
    (numpy's here); what they stand for is exact."""
    D, G, lead = x.shape[-1], x.shape[-1] // 32, tuple(x.shape[:-1])
    u = x.float().cpu().numpy()
    u = np.ascontiguousarray(u).reshape((-1,) + (2,) * int(math.log2(D)))
    for axis in range(u.ndim - 1, 0, -1):
        a, c = np.take(u, 0, axis), np.take(u, 1, axis)
        u = np.stack([a + c, a - c], axis)
    u = u.reshape(-1, G, 32)
    top = np.float32(2 ** (b - 1) - 1)
    s = (np.abs(u).max(-1, keepdims=True) / top).astype(np.float16).astype(np.float32)
    inv = np.divide(np.float32(1), s, out=np.zeros_like(s), where=s > 0)
    q = np.clip(np.rint(u * inv), -2.0 ** (b - 1), top)
    w = torch.from_numpy(q.astype(np.float64) * s.astype(np.float64)).to(x.device).reshape(*lead, D)
    return w @ _hadamard(D, x.device, torch.float64) / D


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    D, Hk, Hq, W = c["head_dim"], c["kv_heads"], c["q_heads"], c["window"]
    lens, news = _lengths(case)
    if c["op"] == "write":
        return {"k": _exact_quantised(st["k"], c["k_bits"]),
                "v": _exact_quantised(st["v"], c["v_bits"])}
    ks, vs, outs, lses, at = [], [], [], [], 0
    for b, (l, n) in enumerate(zip(lens, news)):
        lo = max(0, l - n - W + 1) if W and c["op"] != "read" else 0
        k, v = _exact_sequence(st, b, lo, l, True), _exact_sequence(st, b, lo, l, False)
        if c["op"] == "read":
            ks.append(k.transpose(0, 1))
            vs.append(v.transpose(0, 1))
            continue
        if c["op"] == "decode":
            k[:, l - n - lo:] = _exact_quantised(st["k"][at:at + n], c["k_bits"]).transpose(0, 1)
            v[:, l - n - lo:] = _exact_quantised(st["v"][at:at + n], c["v_bits"]).transpose(0, 1)
        q = st["q"][at:at + n].double()
        t = torch.arange(lo, l, device=k.device)
        for i in range(n):
            p = l - n + i
            see = (t <= p) & ((t > p - W) if W else (t >= 0))
            s = torch.einsum("hgd,htd->hgt", q[i].reshape(Hk, Hq // Hk, D), k[:, see]) * D ** -0.5
            e = torch.logsumexp(s, dim=-1)
            outs.append(torch.einsum("hgt,htd->hgd", torch.exp(s - e[..., None]), v[:, see]).reshape(1, Hq, D))
            lses.append(e.reshape(1, Hq))
        at += n
    if c["op"] == "read":
        return {"k": torch.cat(ks), "v": torch.cat(vs)}
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
