"""Cases and plain forms of the attention-side operators: rotary positions with
per-head norms, appending to a paged 4-bit key/value cache, reading it back,
and attention over it.

Conventions. Token rows q_start[b] .. q_start[b + 1] - 1 belong to sequence
b; lens[b] is that sequence's cache length, these tokens included; its token
i sits at position lens[b] - n_b + i. A page holds P tokens: per kv head the
key codes (P rows of hd / 2 bytes), the key scales (hd / 32 rows of P fp16),
then the value codes and value scales. Eight channels share a dword, channel
c in nibble (c >> 1) + 4 (c & 1); a nibble n stands for d (n - 8).
"""
import math

import torch

own = False

BLOCK = 32


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of a 0.5B-class model: the smallest call of a decode step
        dict(name="rope_decode", op="rope", n_tok=1, H=14, hd=64, rot=64, inter=False, norm=False, first=777),
        # a long prompt's queries far into a long context, normed, interleaved pairs
        dict(name="rope_prompt", op="rope", n_tok=4096, H=32, hd=128, rot=128, inter=True, norm=True, first=120000),
        # one new token of an 8B-class model: rotate q and k, store k and v
        dict(name="append_decode_1", op="append", n_seq=1, q_tok=1, ctx=8192, H=32, Hk=8, hd=128, rot=128,
             inter=False, norm=False, page=64),
        # a batch of decoding sequences, normed heads, half of each head rotated
        dict(name="append_decode_48", op="append", n_seq=48, q_tok=1, ctx=2111, H=14, Hk=2, hd=64, rot=32,
             inter=False, norm=True, page=16),
        # two prompts of different lengths stored at once
        dict(name="append_prompt", op="append", n_seq=2, q_tok=4096, ctx=5001, H=32, Hk=8, hd=128, rot=128,
             inter=True, norm=True, page=128),
        # a short sequence handed to another path
        dict(name="read_short", op="read", n_seq=1, ctx=333, Hk=2, hd=64, page=16),
        # a batch of long sequences moved out of the cache
        dict(name="read_long", op="read", n_seq=8, ctx=8000, Hk=8, hd=128, page=64),
        # decode, short context, a 0.5B-class model (seven query heads a kv head)
        dict(name="decode_short", op="attn", n_seq=1, q_tok=1, ctx=333, H=14, Hk=2, hd=64, page=16, causal=True, window=0),
        # decode, one sequence of an 8B-class model
        dict(name="decode_8k", op="attn", n_seq=1, q_tok=1, ctx=8192, H=32, Hk=8, hd=128, page=64, causal=True, window=0),
        # decode, a serving batch with lengths from 8k to 16k
        dict(name="decode_32x16k", op="attn", n_seq=32, q_tok=1, ctx=16384, H=32, Hk=8, hd=128, page=64, causal=True,
             window=0),
        # one prompt chunk of 64 positions late in a long context
        dict(name="chunk_64_16k", op="attn", n_seq=1, q_tok=64, ctx=16384, H=32, Hk=8, hd=128, page=64, causal=True,
             window=0),
        # two whole prompts of different lengths, odd sizes
        dict(name="prompt_4k", op="attn", n_seq=2, q_tok=4096, ctx=4099, H=32, Hk=8, hd=128, page=128, causal=True,
             window=0),
    ]


HEADS = [(14, 2), (9, 3), (32, 8), (8, 4), (16, 16), (40, 8), (12, 2)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attn", "attn"])
    H, Hk = rng.choice(HEADS)
    hd = rng.choice([64, 96, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    rot = rng.choice([hd, hd, hd // 2])
    inter, norm = rng.random() < 0.5, rng.random() < 0.5
    if op == "rope":
        n = min(_log(rng, 1, 8192), 4096 * 32 * 128 // (H * hd))
        return dict(op=op, n_tok=n, H=H, hd=hd, rot=rot, inter=inter, norm=norm, first=_log(rng, 1, 300000))
    if op == "append":
        if rng.random() < 0.5:
            n_seq, q_tok = _log(rng, 1, 128), 1
        else:
            n_seq, q_tok = rng.randint(1, 4), _log(rng, 2, 4096)
        q_tok = max(1, min(q_tok, 8192 * 40 * 128 // ((H + Hk) * hd * n_seq)))
        return dict(op=op, n_seq=n_seq, q_tok=q_tok, ctx=q_tok + _log(rng, 1, 4096), H=H, Hk=Hk, hd=hd, rot=rot,
                    inter=inter, norm=norm, page=page)
    if op == "read":
        n_seq = _log(rng, 1, 32)
        ctx = min(_log(rng, 1, 16384), 8 * 8000 * 8 * 128 // (n_seq * Hk * hd))
        return dict(op=op, n_seq=n_seq, ctx=max(1, ctx), Hk=Hk, hd=hd, page=page)
    if rng.random() < 0.5:
        n_seq, q_tok = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3])
        ctx = q_tok + min(_log(rng, 1, 16384), 32 * 16384 * 8 * 128 // (n_seq * Hk * hd) - 4)
    else:
        n_seq, q_tok = rng.randint(1, 4), _log(rng, 2, 4096)
        q_tok = max(2, min(q_tok, int((4096 * 4096 * 32 / H * 128 / hd / n_seq) ** 0.5)))
        room = 4096 * 4096 * 32 * 128 // (H * hd * n_seq * q_tok) - q_tok
        ctx = q_tok + min(_log(rng, 1, 16384), max(0, room), 64 * 4096 * 8 // (n_seq * Hk))
    return dict(op=op, n_seq=n_seq, q_tok=q_tok, ctx=ctx, H=H, Hk=Hk, hd=hd, page=page, causal=rng.random() < 0.85,
                window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]))


def _ragged(case):
    """New tokens and cache length of every sequence."""
    n_seq, q_tok, ctx = case["n_seq"], case.get("q_tok", 0), case["ctx"]
    if case["op"] == "read":
        lens = [ctx - (b * 977) % (ctx // 3 + 1) for b in range(n_seq)]
        return lens, lens
    n = [q_tok - (b * 1201) % (q_tok // 2 + 1) for b in range(n_seq)]
    lens = [max(n[b], ctx - (b * 1571) % (ctx // 2 + 1)) for b in range(n_seq)]
    return n, lens


def _page_bytes(case):
    return case["page"] * case["Hk"] * (case["hd"] + case["hd"] // 8)


# ----------------------------------------------------------------- prepare
def _freqs(case):
    """Inverse frequencies in fp32, the positions interpolated by two."""
    rot = case["rot"]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) / 2.0
    return f.to(torch.float32).cuda()


def _cache(case, lens, gen):
    """A filled pool whose pages are handed out in random order."""
    P, Hk, hd = case["page"], case["Hk"], case["hd"]
    per = -(-max(lens) // P)
    n_pages = case["n_seq"] * per + 3
    table = torch.randperm(n_pages, generator=gen, device="cuda")[: case["n_seq"] * per].to(torch.int32)
    code_b, scale_n = P * hd // 2, P * hd // BLOCK
    pool = torch.empty((n_pages, Hk, 2, code_b + 2 * scale_n), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (Hk * P * hd))
    for p in range(0, n_pages, step):
        part = pool[p: p + step]
        m = part.shape[0]
        c = torch.randn((m, Hk, 2, code_b, 2), generator=gen, device="cuda").mul_(2.9).round_().clamp_(-8, 7).add_(8)
        c = c.to(torch.uint8)
        part[..., :code_b] = c[..., 0] | (c[..., 1] << 4)
        d = torch.randn((m, Hk, 2, scale_n), generator=gen, device="cuda").mul_(0.4).add_(2.1).abs_().div_(8)
        d = d * (torch.randint(0, 2, d.shape, generator=gen, device="cuda") * 2 - 1)
        part[..., code_b:] = d.to(torch.bfloat16).to(torch.float16).view(torch.uint8)
    return pool.view(n_pages, -1), table.view(case["n_seq"], per)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    if case["op"] == "rope":
        s["x"] = randn(case["n_tok"], case["H"], case["hd"])
        s["pos"] = (torch.arange(case["n_tok"], device="cuda") + case["first"]).to(torch.int32)
        s["freqs"] = _freqs(case)
        s["w"] = 1 + 0.1 * randn(case["hd"]) if case["norm"] else None
        return s
    n, lens = _ragged(case)
    s["pages"], s["table"] = _cache(case, lens, gen)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    start = [0]
    for m in n:
        start.append(start[-1] + m)
    s["q_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    s["n_tok"], s["max_q"], s["max_len"] = start[-1], max(n), max(lens)
    if case["op"] == "append":
        # the rows of a fused q | k | v projection
        H, Hk, hd = case["H"], case["Hk"], case["hd"]
        s["qkv"] = randn(s["n_tok"], (H + 2 * Hk), hd)
        s["freqs"] = _freqs(case)
        s["qw"] = 1 + 0.1 * randn(hd) if case["norm"] else None
        s["kw"] = 1 + 0.1 * randn(hd) if case["norm"] else None
    elif case["op"] == "attn":
        s["q"] = 1.5 * randn(s["n_tok"], case["H"], case["hd"])
    return s


# ------------------------------------------------------------- plain forms
def _rope_plain(x, pos, freqs, rot, inter, w, wide):
    """Norm and rotation of [n, heads, hd]; angles in 64 bits, the rest too where `wide`."""
    a = pos.double()[:, None] * freqs.double()
    t = torch.float64 if wide else torch.float32
    cos, sin, x = torch.cos(a).to(t)[:, None], torch.sin(a).to(t)[:, None], x.to(t)
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.to(t)
    y = x.clone()
    if inter:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = u * cos - v * sin, v * cos + u * sin
    else:
        u, v = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2], y[..., rot // 2: rot] = u * cos - v * sin, v * cos + u * sin
    return y


def _quantised_plain(x):
    """The values that 4-bit blocks of 32 channels hold for x (64 bits: codes and scales sit next to borders)."""
    b = x.double().unflatten(-1, (-1, BLOCK))
    a = b.gather(-1, b.abs().argmax(-1, keepdim=True))
    d = -a / 8
    _, e = torch.frexp(d)
    q = torch.ldexp(torch.ones_like(d), torch.clamp(e - 8, min=-24))
    d = (torch.round(d / q) * q).clamp(-8160, 8160)
    c = torch.where(d == 0, 0.0, torch.round(b / d).clamp(-8, 7))
    return (d * c).flatten(-2).float()


def _unpacked_plain(s):
    """Keys and values of every table entry: [n_seq, kv heads, tokens, hd] each."""
    P, Hk, hd = s["page"], s["Hk"], s["hd"]
    code_b = P * hd // 2
    t = s["pages"][s["table"].long()].unflatten(-1, (Hk, 2, -1))  # n_seq, pages, Hk, 2, bytes
    codes = t[..., :code_b].unflatten(-1, (P, hd // 8, 4))
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)  # the dword's nibbles in order
    val = nib.unflatten(-1, (2, 4)).transpose(-1, -2).flatten(-3)  # channels in order
    d = t[..., code_b:].contiguous().view(torch.float16).unflatten(-1, (hd // BLOCK, P)).transpose(-1, -2).float()
    val = (val.float() - 8).unflatten(-1, (-1, BLOCK)) * d[..., None]
    val = val.flatten(-2).permute(3, 0, 2, 1, 4, 5).flatten(3, 4)  # 2, n_seq, Hk, tokens, hd
    return val[0], val[1]


def _rows(s):
    """Sequence, place in it and position of every token row."""
    row = torch.arange(s["n_tok"], device="cuda")
    start, lens = s["q_start"].long(), s["lens"].long()
    b = torch.searchsorted(start[1:].contiguous(), row, right=True)
    i = row - start[b]
    return b, i, lens[b] - (start[b + 1] - start[b]) + i


def _attn_plain(s):
    H, Hk, hd, mq = s["H"], s["Hk"], s["hd"], s["max_q"]
    K, V = _unpacked_plain(s)
    start, lens = s["q_start"].long(), s["lens"].long()
    n = start[1:] - start[:-1]
    place = torch.arange(mq, device="cuda")
    tok = (start[:-1, None] + place).clamp(max=s["n_tok"] - 1)
    q = s["q"][tok].unflatten(2, (Hk, H // Hk)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # n_seq, Hk, G mq, hd
    sc = torch.matmul(q, K.transpose(-1, -2)) * hd ** -0.5
    key = torch.arange(K.shape[2], device="cuda")
    pos = (lens - n)[:, None] + place
    seen = (key < lens[:, None, None]).expand(-1, mq, -1)
    if s["causal"]:
        seen = seen & (key <= pos[..., None])
    if s["window"]:
        seen = seen & (key > pos[..., None] - s["window"])
    sc = sc.unflatten(2, (H // Hk, mq)).masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True).clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), V).unflatten(2, (H // Hk, mq))
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).flatten(2, 3)  # n_seq, mq, H, hd
    b, i, _ = _rows(s)
    return o[b, i]


# --------------------------------------------------------------------- run
def _handles(s):
    """The framework's handles that a program keeps: made on a state's first pass."""
    import gguf_block_quant_gq_amd as gq

    if "gq" not in s:
        s["gq"] = gq
        if "pages" in s:
            s["cache"] = gq.KV4Cache(s["pages"], s["table"], s["page"], s["Hk"], s["hd"])
        if "freqs" in s:
            s["rope"] = gq.Rope(s["freqs"], interleaved=s["inter"])
    return gq


def run(s):
    if s["op"] == "rope":
        if own:
            gq = _handles(s)
            return gq.gq_qk_rope(s["x"], s["pos"], s["rope"], norm=s["w"], eps=1e-6)
        return _rope_plain(s["x"], s["pos"], s["freqs"], s["rot"], s["inter"], s["w"], False)
    if s["op"] == "append":
        H, Hk = s["H"], s["Hk"]
        q, k, v = s["qkv"][:, :H], s["qkv"][:, H: H + Hk], s["qkv"][:, H + Hk:]
        if own:
            gq = _handles(s)
            qr = gq.gq_kv4_append(s["cache"], k, v, s["lens"], s["q_start"], rope=s["rope"], k_norm=s["kw"], q=q,
                                  q_norm=s["qw"], eps=1e-6)
            kc, vc = gq.gq_kv4_read(s["cache"], s["lens"], s["n_tok"], s["q_start"])
            return {"q": qr, "k": kc, "v": vc}
        _, _, pos = _rows(s)
        return {"q": _rope_plain(q, pos, s["freqs"], s["rot"], s["inter"], s["qw"], False),
                "k": _quantised_plain(_rope_plain(k, pos, s["freqs"], s["rot"], s["inter"], s["kw"], True)),
                "v": _quantised_plain(v)}
    if s["op"] == "read":
        if own:
            gq = _handles(s)
            kc, vc = gq.gq_kv4_read(s["cache"], s["lens"], s["n_tok"], s["q_start"])
            return {"k": kc, "v": vc}
        K, V = _unpacked_plain(s)
        b, _, pos = _rows(s)
        return {"k": K[b, :, pos], "v": V[b, :, pos]}
    if own:
        gq = _handles(s)
        return gq.gq_kv4_attn(s["cache"], s["q"], s["lens"], s["q_start"], max_q=s["max_q"], max_len=s["max_len"],
                              causal=s["causal"], window=s["window"])
    return _attn_plain(s)


# -------------------------------------------------------------------- work
def work(case):
    hd = case["hd"]
    if case["op"] == "rope":
        n = case["n_tok"] * case["H"] * hd
        return {"bytes": 8 * n + 4 * case["n_tok"] + 2 * case["rot"], "flops": 6 * n}
    n, lens = _ragged(case)
    Hk = case["Hk"]
    if case["op"] == "read":
        vals = 2 * sum(lens) * Hk * hd
        return {"bytes": vals * (0.5625 + 4), "flops": vals}
    if case["op"] == "append":
        q, kv = sum(n) * case["H"] * hd, 2 * sum(n) * Hk * hd
        # q rotated; k and v stored, then read back as the values they hold
        return {"bytes": 8 * q + kv * (4 + 0.5625 + 0.5625 + 4), "flops": 6 * q + 8 * kv}
    pairs = keys = 0
    for m, L in zip(n, lens):
        # the row at position p sees the keys lo .. hi - 1
        p = torch.arange(L - m, L, dtype=torch.int64)
        hi = p + 1 if case["causal"] else torch.full_like(p, L)
        lo = (p + 1 - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(p)
        pairs += int((hi - lo).clamp(min=0).sum())
        keys += int(hi.max() - lo.min())
    return {"bytes": 1.125 * keys * Hk * hd + 8 * sum(n) * case["H"] * hd, "flops": 4 * pairs * case["H"] * hd}


# ------------------------------------------------------------------- exact
def _rope_exact(x, pos, freqs, rot, inter, w):
    """The rotation as a product of complex numbers, in 64 bits."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * w.double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.outer(pos.double(), freqs.double()))[:, None]
    head, rest = x[..., :rot], x[..., rot:]
    z = torch.complex(*(head.unflatten(-1, (-1, 2)).unbind(-1) if inter else head.chunk(2, -1))) * turn
    head = torch.view_as_real(z).flatten(-2) if inter else torch.cat((z.real, z.imag), -1)
    return torch.cat((head, rest), -1)


def _held_exact(x):
    """What the cache holds for x: the scale's 8 bits taken by adding and subtracting a large number."""
    b = x.double().reshape(-1, BLOCK)
    top, bot = b.max(1).values, b.min(1).values
    first = (b == b.abs().max(1, keepdim=True).values[:, :1]).to(torch.int8).argmax(1)
    last = (b == -b.abs().max(1, keepdim=True).values[:, :1]).to(torch.int8).argmax(1)
    a = torch.where(top > -bot, top, torch.where(top < -bot, bot, torch.where(first <= last, top, bot)))
    d = a * -0.125
    unit = torch.clamp(torch.exp2(torch.floor(torch.log2(d.abs().clamp(min=1e-30))) - 7), min=2.0 ** -24)
    big = unit * (1.5 * 2.0 ** 52)
    d = ((d + big) - big).clamp(-8160, 8160)[:, None]
    c = torch.clamp(torch.nan_to_num(b / d).round(), -8, 7)
    return (c * d).reshape(x.shape)


def _tokens_exact(s, b):
    """Keys and values of sequence b, [tokens, kv heads, hd] each, nibble by nibble."""
    P, Hk, hd, L = s["page"], s["Hk"], s["hd"], int(s["lens"][b])
    pages = s["pages"][s["table"][b, : -(-L // P)].long()]
    got = []
    for kv in range(2):
        part = pages.reshape(pages.shape[0], Hk, 2, -1)[:, :, kv]
        words = part[..., : P * hd // 2].contiguous().view(torch.int32).reshape(-1, Hk, P, hd // 8)
        d = part[..., P * hd // 2:].contiguous().view(torch.float16).double().reshape(-1, Hk, hd // BLOCK, P)
        x = torch.empty((pages.shape[0], Hk, P, hd), dtype=torch.float64, device="cuda")
        for c in range(8):
            x[..., c::8] = ((words >> (4 * ((c >> 1) + 4 * (c & 1)))) & 15).double() - 8
        x *= d.repeat_interleave(BLOCK, 2).transpose(2, 3)
        got.append(x.transpose(1, 2).reshape(-1, Hk, hd)[:L])
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _rope_exact(s["x"], s["pos"], s["freqs"], s["rot"], s["inter"], s["w"])
    n, lens = _ragged(case)
    if case["op"] == "append":
        H, Hk = s["H"], s["Hk"]
        pos = torch.cat([torch.arange(L - m, L) for m, L in zip(n, lens)]).cuda()
        q, k, v = s["qkv"].split((H, Hk, Hk), 1)
        turn = lambda x, w: _rope_exact(x, pos, s["freqs"], s["rot"], s["inter"], w)  # noqa: E731
        return {"q": turn(q, s["qw"]), "k": _held_exact(turn(k, s["kw"])), "v": _held_exact(v)}
    if case["op"] == "read":
        parts = [_tokens_exact(s, b) for b in range(case["n_seq"])]
        return {"k": torch.cat([p[0] for p in parts]), "v": torch.cat([p[1] for p in parts])}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (m, L) in enumerate(zip(n, lens)):
        K, V = _tokens_exact(s, b)
        j = torch.arange(L, device="cuda")
        for t in range(0, m, 1024):
            p = torch.arange(L - m + t, L - m + min(m, t + 1024), device="cuda")[:, None]
            seen = torch.ones((len(p), L), dtype=torch.bool, device="cuda")
            if case["causal"]:
                seen &= j <= p
            if case["window"]:
                seen &= p - j < case["window"]
            for h in range(case["H"]):
                g = h // (case["H"] // case["Hk"])
                z = s["q"][at + t: at + t + len(p), h].double() @ K[:, g].T.contiguous() / math.sqrt(case["hd"])
                out[at + t: at + t + len(p), h] = torch.softmax(z.masked_fill(~seen, -math.inf), -1).nan_to_num() @ V[:, g]
        at += m
    return out
