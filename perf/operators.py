"""The paged-cache operators as measured workloads: appending rotated keys and values to the pages,
attention over a page table (whole, or a sliding window with the first tokens kept), and attention
for a batch that shares one long prefix.

Every case is a dict of plain values.  ``prepare`` makes its inputs on the GPU from a seed, ``run``
makes one pass: in plain torch operations where ``own`` is false, through the package's own calls
where it is true.  ``exact`` gives the result from the definition in 64 bits.

The page format (one 3,200-byte block holds 32 tokens of one kv-head; ``pages`` is uint8
[num_pages, kv_heads, page_tokens / 32, 3200]):
    bytes    0 ..  511   key sign bits, u32 [32 rows][4]; row 8 i + 2 t + e is token 8 t + 2 i + e; bit
                         i of word w is 1 iff rotated channel 32 w + i is >= 0
    bytes  512 ..  639   f32 [32]: the key's norm times its correction, N * (128 N / sum |y|)
    bytes  640 ..  895   f16 [4][32]: value scale per 32-channel group and token
    bytes  896 .. 1151   f16 [4][32]: value minimum per group and token
    bytes 1152 .. 3199   value codes, u32 [128 channels][4]; nibble p of word w is token 8 w + 2 p for
                         p < 4 and token 8 w + 2 (p - 4) + 1 for p >= 4
"""
import math

import torch

own = False

D = 128
BLOCK = 32
BLOCK_BYTES = 3200
F16_MAX = 65504.0
TABLE_POSITIONS = 131072


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one sequence: the append of a single-user decode step, launch latency counts
        dict(name="append decode b1", op="append", batch=1, tokens=1, past=4999, kv_heads=8, group=4, page=128, dtype="bf16",
             rot=128, axes=1, interleaved=False),
        # one token for each of 64 sequences of uneven length
        dict(name="append decode b64", op="append", batch=64, tokens=64, past=32000, kv_heads=8, group=4, page=64, dtype="bf16",
             rot=128, axes=1, interleaved=False),
        # a prefill chunk whose tokens carry three positions each (time, height, width)
        dict(name="append chunk 3-axis", op="append", batch=1, tokens=4096, past=1001, kv_heads=8, group=4, page=128, dtype="fp16",
             rot=128, axes=3, interleaved=False),
        # uneven prompts of eight sequences packed behind one another, a part of the channels rotated
        dict(name="append ragged prompts", op="append", batch=8, tokens=32768, past=37, kv_heads=8, group=4, page=128, dtype="bf16",
             rot=64, axes=1, interleaved=True),
        # a chat just begun: a few hundred odd tokens, latency counts
        dict(name="attend short", op="attend", batch=1, length=397, kv_heads=8, group=4, page=128, dtype="bf16", window=0, sinks=0),
        # a serving batch of uneven long contexts
        dict(name="attend b8 32k", op="attend", batch=8, length=32768, kv_heads=8, group=4, page=128, dtype="bf16", window=0, sinks=0),
        # one context of a million tokens
        dict(name="attend 1M", op="attend", batch=1, length=1048576, kv_heads=8, group=4, page=128, dtype="bf16", window=0, sinks=0),
        # a sliding-window layer: 4,096 recent tokens and the first 4, eight query heads a kv-head
        dict(name="attend window", op="attend", batch=32, length=32768, kv_heads=8, group=8, page=64, dtype="fp16", window=4096, sinks=4),
        # a few short answers under a common instruction
        dict(name="shared small", op="shared", batch=4, prefix=1000, length=61, kv_heads=8, group=4, page=64, dtype="bf16"),
        # every head its own keys, sixteen samples of one prompt
        dict(name="shared b16 32 heads", op="shared", batch=16, prefix=8192, length=300, kv_heads=32, group=1, page=128, dtype="fp16"),
        # many requests over one long document
        dict(name="shared b64 128k", op="shared", batch=64, prefix=131072, length=512, kv_heads=8, group=4, page=128, dtype="bf16"),
    ]


MOST_TOKEN_HEADS = 8 << 20  # the cache of the largest listed case


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "shared"])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 8, 16, 32])
    group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    page = rng.choice([32, 64, 128, 256])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "append":
        batch = _log(rng, 1, 64)
        tokens = _log(rng, batch, 32768)
        while tokens * kv_heads > 32768 * 8:
            kv_heads //= 2
        axes = rng.choice([1, 1, 3])
        return dict(op=op, batch=batch, tokens=tokens, past=rng.randrange(0, 4000), kv_heads=kv_heads, group=min(group, max(1, 64 // kv_heads)),
                    page=page, dtype=dtype, rot=rng.choice([32, 64, 96, 128, 128]), axes=axes, interleaved=rng.random() < 0.3)
    if op == "attend":
        batch = _log(rng, 1, 64)
        length = _log(rng, 1, MOST_TOKEN_HEADS // (batch * kv_heads))
        window = 0 if rng.random() < 0.5 else _log(rng, 1, max(2, length))
        return dict(op=op, batch=batch, length=length, kv_heads=kv_heads, group=group, page=page, dtype=dtype, window=window,
                    sinks=rng.choice([0, 1, 4, 33]) if window else 0)
    batch = _log(rng, 2, 64)
    prefix = _log(rng, 1, max(2, min(131072, (1 << 28) // (batch * kv_heads * group))))
    length = _log(rng, 1, 512)
    return dict(op=op, batch=batch, prefix=prefix, length=length, kv_heads=kv_heads, group=group, page=page, dtype=dtype)


def _uneven(total_each, batch):
    """One length per sequence, between a half and the whole of total_each; the first has it all."""
    return [max(1, total_each - (total_each * ((i * 37) % 64)) // 128) for i in range(batch)]


def _new_tokens(case):
    """How many of case["tokens"] each sequence appends (uneven; one each where tokens == batch)."""
    n, batch = case["tokens"], case["batch"]
    weights = [1 + (i * 5) % 7 for i in range(batch)]
    spare = n - batch
    got = [1 + spare * w // sum(weights) for w in weights]
    got[0] += n - sum(got)
    return got


def _past(case):
    return [(case["past"] * (64 - (i * 29) % 64)) // 64 for i in range(case["batch"])]


def _sections(case):
    half = case["rot"] // 2
    if case["axes"] == 1:
        return [half]
    hw = (3 * half) // 8
    return [half - 2 * hw, hw, hw]


# ----------------------------------------------------------------------------------------- inputs
def _dtype(case):
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[case["dtype"]]


def _table(gen, lengths, page, spare=3):
    """A page table over shuffled pages: int32 [batch, most pages], -1 behind a sequence's pages."""
    counts = [(n + page - 1) // page for n in lengths]
    total = sum(counts) + spare
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), max(max(counts), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    return table, total, order[at:]


def _fields(pages):
    """The planes of the page blocks as views of the buffer."""
    return (pages[..., :512].view(torch.int32), pages[..., 512:640].view(torch.float32), pages[..., 640:896].view(torch.float16),
            pages[..., 896:1152].view(torch.float16), pages[..., 1152:].view(torch.int32))


def _random_pages(gen, total, kv_heads, page):
    """Pages as encoded Gaussian keys and values give them: random signs and codes, norms near
    sqrt(128), scales and minima of 32 normal values."""
    shape = (total, kv_heads, page // BLOCK)
    pages = torch.empty(shape + (BLOCK_BYTES,), dtype=torch.uint8, device="cuda")
    bits, nc, scale, least, codes = _fields(pages)
    pages.view(torch.int32).random_(-2 ** 31, 2 ** 31 - 1, generator=gen)
    spread = torch.randn(nc.shape, generator=gen, device="cuda")
    nc.copy_(math.sqrt(128.0) * 1.2533 * torch.exp(0.25 * spread))
    scale.copy_(0.27 + 0.05 * torch.randn(scale.shape, generator=gen, device="cuda").clamp_(-3, 3))
    least.copy_(-2.05 + 0.4 * torch.randn(least.shape, generator=gen, device="cuda"))
    return pages


def _signs(gen):
    s = torch.zeros((3, D), device="cuda")
    s[0] = torch.randint(0, 2, (D,), generator=gen, device="cuda") * 2.0 - 1.0
    return s


def _align_some(gen, pages, q, signs, kv_heads):
    """Every 37th block's first key gets the signs of a query (three of four words), so that a few
    tokens draw much of the attention."""
    z = _rotate(q.float(), signs)[:, :: max(1, q.shape[1] // kv_heads)][:, :kv_heads]    # [batch, kv_heads, 128]
    word = _pack_bits((z[0] >= 0).to(torch.int64))                                       # [kv_heads, 4]
    bits = _fields(pages)[0].view(pages.shape[:-1] + (BLOCK, 4))
    flat = torch.arange(pages.shape[0], device="cuda")[::5]
    bits[flat, :, 0, 0, :3] = word[None, :, :3]


def _pack_bits(b):
    """int64 0 / 1 [..., 128] to int32 words [..., 4]."""
    w = (b.reshape(b.shape[:-1] + (4, 32)) << torch.arange(32, device=b.device)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:  # the handles a serving program keeps: the cache over its pages, the rotary table
        import long_context_decode_kv1b_b200 as kv

        st["cache"] = kv.PagedCache.wrap(st["pages"], st["signs"])
        if case["op"] == "append":
            st["rope"] = kv.Rope(st["cos_sin"], sections=_sections(case), interleaved=case["interleaved"])
    return st


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, H, G, page = _dtype(case), case["kv_heads"], case["group"], case["page"]
    st = dict(case=case, signs=_signs(gen))
    if case["op"] == "append":
        n, past = _new_tokens(case), _past(case)
        T = case["tokens"]
        table, total, _ = _table(gen, [a + b for a, b in zip(past, n)], page)
        st["pages"] = _random_pages(gen, total, H, page)
        st["table"] = table
        st["start"] = torch.tensor(past, dtype=torch.int32, device="cuda")
        cu = [0]
        for x in n:
            cu.append(cu[-1] + x)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        # q, k and v as one projection writes them: rows of (Hq + 2 Hkv) heads
        qkv = torch.randn((T, H * G + 2 * H, D), generator=gen, device="cuda").to(dt)
        st["q"], st["k"], st["v"] = qkv[:, :H * G], qkv[:, H * G:H * G + H], qkv[:, H * G + H:]
        half = case["rot"] // 2
        freq = 1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        angle = torch.arange(TABLE_POSITIONS, device="cuda", dtype=torch.float64)[:, None] * freq
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        pos = torch.cat([torch.arange(p, p + x, device="cuda") for p, x in zip(past, n)])
        if case["axes"] == 3:  # rows and columns of images 24 wide
            pos = torch.stack([pos, pos - pos % 24 + (pos // 24) % 24, pos - pos % 24 + pos % 24])
        else:
            pos = pos[None]
        st["positions"] = pos.to(torch.int32)
        return st
    lengths = _uneven(case["length"], case["batch"])
    if case["op"] == "attend":
        table, total, _ = _table(gen, lengths, page)
    else:
        np_ = (case["prefix"] + page - 1) // page
        table, total, rest = _table(gen, lengths, page, spare=np_)
        st["prefix_pages"] = rest[:np_].contiguous()
        st["prefix_length"] = torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda")
    st["pages"] = _random_pages(gen, total, H, page)
    st["table"] = table
    st["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    st["q"] = torch.randn((case["batch"], H * G, D), generator=gen, device="cuda").to(dt)
    _align_some(gen, st["pages"], st["q"], st["signs"], H)
    return st


# ------------------------------------------------------------------------------------- plain forms
def _rotate(x, signs):
    """y = H (D x) in float32: butterflies of stride 1, 2, ..., 64 (the cases use one rotation round)."""
    x = x * signs[0]
    for h in (1, 2, 4, 8, 16, 32, 64):
        y = x.reshape(x.shape[:-1] + (D // (2 * h), 2, h))
        a, c = y[..., 0, :], y[..., 1, :]
        x = torch.stack([a + c, a - c], -2).reshape(x.shape)
    return x


def _tree_sum(a):
    """Sum of 128 channels in float32: a[i] += a[i + h] for h = 64, 32, ..., 1."""
    for h in (64, 32, 16, 8, 4, 2, 1):
        a = a[..., :h] + a[..., h:2 * h]
    return a[..., 0]


def _rope(x, st):
    """Channels [0, rot) of x [T, heads, 128] (float32) turned by each pair's angle."""
    case = st["case"]
    rot, half = case["rot"], case["rot"] // 2
    sec = _sections(case)
    axis = torch.repeat_interleave(torch.arange(len(sec), device=x.device), torch.tensor(sec, device=x.device), output_size=half)
    row = st["cos_sin"][st["positions"].long()]                    # [axes, T, rot]
    pick = axis[None, None].expand(1, row.shape[1], half)
    c = row[:, :, :half].gather(0, pick)[0][:, None]               # [T, 1, half]
    s = row[:, :, half:].gather(0, pick)[0][:, None]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _half_order(h):
    i = h.contiguous().view(torch.int16).to(torch.int32)
    return torch.where(i >= 0, i, -(i & 0x7FFF))


def _half_of(o):
    return torch.where(o >= 0, o, (-o) | 0x8000).to(torch.int16).view(torch.float16)


def _quantise(v):
    """v float32 [..., 128] to (codes int32 [..., 128], scale f16 [..., 4], min f16 [..., 4])."""
    v = v.clamp(-F16_MAX, F16_MAX).reshape(v.shape[:-1] + (4, 32))
    mn, mx = v.amin(-1), v.amax(-1)
    h = mn.half()
    least = _half_of(_half_order(h) - (h.float() > mn).int())
    lf = least.float()
    span = mx.double() - lf.double()
    o = _half_order((span / 15.0).half())
    o = o + (_half_of(o).double() * 15.0 < span).int()
    o = o - ((_half_of((o - 1).clamp(min=0)).double() * 15.0 >= span) & (o > 0)).int()
    o = o - (lf.double() + 15.0 * _half_of(o).double() > F16_MAX).int()
    scale = _half_of(o)
    sf = scale.float()[..., None]
    y = torch.floor((v - lf[..., None]) / sf + 0.5)
    codes = torch.where(sf > 0, y.clamp(0, 15), torch.zeros_like(y)).to(torch.int32)
    return codes.flatten(-2), scale, least


def _nibble_shift(device):
    j = torch.arange(8, device=device)
    return 4 * (j // 2 + 4 * (j % 2))   # token j of a word sits at this bit


def _bit_row(tok):
    return 8 * ((tok >> 1) & 3) + 2 * (tok >> 3) + (tok & 1)


def _plain_append(st):
    case, pages = st["case"], st["pages"]
    dev = pages.device
    bits, nc, scale, least, codes = _fields(pages)
    n = st["cu"][1:] - st["cu"][:-1]
    T = case["tokens"]
    seq = torch.repeat_interleave(torch.arange(case["batch"], device=dev), n.long(), output_size=T)
    at = torch.arange(T, device=dev) - st["cu"].long()[seq] + st["start"].long()[seq]
    pg = st["table"].long()[seq, at // case["page"]]
    blk, tok = (at % case["page"]) // BLOCK, at % BLOCK
    k = _rope(st["k"].float(), st)
    y = _rotate(k, st["signs"])
    norm = _tree_sum(k * k).sqrt()
    total = _tree_sum(y.abs())
    cinv = torch.where(total > 0, 128.0 * norm / total, torch.ones_like(total))
    nc[pg, :, blk, tok] = norm * cinv
    bits.view(bits.shape[:-1] + (BLOCK, 4))[pg, :, blk, _bit_row(tok)] = _pack_bits((y >= 0).to(torch.int64))
    c, s, m = _quantise(st["v"].float())
    scale.view(scale.shape[:-1] + (4, BLOCK))[pg, :, blk, :, tok] = s
    least.view(least.shape[:-1] + (4, BLOCK))[pg, :, blk, :, tok] = m
    # the codes: whole words of the touched blocks taken apart and put together again
    words = codes.view(codes.shape[:-1] + (D, 4))
    touched = (pg * (case["page"] // BLOCK) + blk).unique()
    tp, tb = touched // (case["page"] // BLOCK), touched % (case["page"] // BLOCK)
    where = torch.searchsorted(touched, pg * (case["page"] // BLOCK) + blk)
    sh = _nibble_shift(dev)
    nib = ((words[tp, :, tb].long()[..., None] >> sh) & 15).flatten(-2)         # [blocks, H, 128, 32]
    nib[where, :, :, tok] = c.long()
    w = (nib.unflatten(-1, (4, 8)) << sh).sum(-1)
    words[tp, :, tb] = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
    return _rope(st["q"].float(), st).to(st["q"].dtype)


def _query(q, signs):
    """Rotated query as 4-bit codes: (codes, origin, step) in float32."""
    z = _rotate(q.float(), signs)
    lo, hi = z.amin(-1, keepdim=True), z.amax(-1, keepdim=True)
    step = (hi - lo) / torch.full_like(hi, 15.0)
    y = torch.floor((z - lo) / step + 0.5).clamp(0, 15)
    return torch.where(step > 0, y, torch.zeros_like(y)), lo, step


def _unpack(pages, table, kv_heads):
    """Signs +-1 and values, float32 [batch, kv_heads, tokens, 128], and N / C [batch, kv_heads, tokens]."""
    got = pages[table.long().clamp(min=0)].transpose(1, 2)       # [batch, H, pages, blocks, bytes]
    bits, nc, scale, least, codes = _fields(got.contiguous())
    dev = pages.device
    row = _bit_row(torch.arange(BLOCK, device=dev))
    b = bits.unflatten(-1, (BLOCK, 4))[..., row, :]
    sign = (((b[..., None] >> torch.arange(32, device=dev, dtype=torch.int32)) & 1) * 2 - 1).float().flatten(-2)
    w = codes.unflatten(-1, (D, 4))
    c = ((w[..., None] >> _nibble_shift(dev).to(torch.int32)) & 15).flatten(-2).float()      # [.., 128, 32]
    sc = scale.unflatten(-1, (4, BLOCK)).float().repeat_interleave(32, -2)
    mn = least.unflatten(-1, (4, BLOCK)).float().repeat_interleave(32, -2)
    v = (mn + sc * c).transpose(-1, -2)
    flat = lambda x: x.flatten(2, 4)  # noqa: E731
    return flat(sign), flat(v), nc.flatten(2)


def _weights(q, signs, kv_heads, scale, sign, nc, visible):
    """exp(logit - max) [batch, kv_heads, queries, tokens] and the max; `visible` broadcasts."""
    code, lo, step = _query(q, signs)
    part = lambda x: x.unflatten(1, (kv_heads, -1))  # noqa: E731
    dot = part(step) * (part(code) @ sign.transpose(-1, -2)) + part(lo) * sign.sum(-1)[:, :, None]
    s = dot * nc[:, :, None] * (scale / 128.0)
    s = s.masked_fill(~visible, -math.inf)
    m = s.amax(-1, keepdim=True)
    return torch.exp(s - m.clamp(min=-1e30)), m


def _plain_attend(st):
    case = st["case"]
    sign, v, nc = _unpack(st["pages"], st["table"], case["kv_heads"])
    t = torch.arange(sign.shape[2], device=sign.device)
    n = st["lengths"][:, None]
    visible = t < n
    if case["window"]:
        visible = visible & ((t >= n - case["window"]) | (t < case["sinks"]))
    p, _ = _weights(st["q"], st["signs"], case["kv_heads"], D ** -0.5, sign, nc, visible[:, None, None])
    v = v.masked_fill(~visible[:, None, :, None], 0.0)
    out = (p @ v) / p.sum(-1, keepdim=True)
    return out.flatten(1, 2).to(st["q"].dtype)


def _plain_shared(st):
    case = st["case"]
    B, H, G = case["batch"], case["kv_heads"], case["group"]
    # the prefix: one matrix of all sequences' queries per kv-head
    sign, v, nc = _unpack(st["pages"], st["prefix_pages"][None], H)
    t = torch.arange(sign.shape[2], device=sign.device)
    all_q = st["q"].unflatten(1, (H, G)).transpose(0, 1).reshape(1, H * B * G, D)
    visible = t < st["prefix_length"]
    p, m = _weights(all_q, st["signs"], H, D ** -0.5, sign, nc, visible)
    v = v.masked_fill(~visible[:, None], 0.0)
    back = lambda x: x[0].unflatten(1, (B, G)).transpose(0, 1)  # noqa: E731
    m0, l0, o0 = back(m), back(p.sum(-1, keepdim=True)), back(p @ v)
    sign, v, nc = _unpack(st["pages"], st["table"], H)
    t = torch.arange(sign.shape[2], device=sign.device)
    visible = t < st["lengths"][:, None]
    p, m1 = _weights(st["q"], st["signs"], H, D ** -0.5, sign, nc, visible[:, None, None])
    v = v.masked_fill(~visible[:, None, :, None], 0.0)
    m = torch.maximum(m0, m1)
    e0, e1 = torch.exp(m0 - m), torch.exp(m1 - m)
    out = (e0 * o0 + e1 * (p @ v)) / (e0 * l0 + e1 * p.sum(-1, keepdim=True))
    return out.flatten(1, 2).to(st["q"].dtype)


# ------------------------------------------------------------------------------------------- a pass
def _append_outputs(st, q_rot):
    """The rotated queries and the whole updated pages, as views: the packed words are whole numbers
    (equal words hold equal signs and codes), the scalars are floats."""
    bits, nc, scale, least, codes = _fields(st["pages"])
    return {"q": q_rot, "bits": bits, "nc": nc, "scale": scale, "min": least, "codes": codes}


def run(state):
    case = state["case"]
    if own:
        cache = state["cache"]
        if case["op"] == "append":
            q = cache.append(state["k"], state["v"], state["table"], state["start"], state["cu"], rope=state["rope"],
                             positions=state["positions"], q=state["q"])
            return _append_outputs(state, q)
        if case["op"] == "attend":
            return cache.attend(state["q"], D ** -0.5, state["table"], state["lengths"], window=case["window"], sinks=case["sinks"])
        return cache.attend_shared(state["q"], D ** -0.5, state["prefix_pages"], state["prefix_length"], state["table"], state["lengths"])
    if case["op"] == "append":
        return _append_outputs(state, _plain_append(state))
    return _plain_attend(state) if case["op"] == "attend" else _plain_shared(state)


def work(case):
    H, G, es = case["kv_heads"], case["group"], 2
    if case["op"] == "append":
        T = case["tokens"]
        heads = T * H
        return {"bytes": heads * (2 * D * es + 100) + 2 * T * H * G * D * es + T * case["rot"] * 4 + T * 4 * case["axes"],
                "flops": heads * (7 * D + 12 * D) + (heads * (1 + G)) * 3 * case["rot"]}
    lengths = _uneven(case["length"], case["batch"])
    seen = sum(lengths)
    if case.get("window"):
        seen = sum(min(n, case["window"] + min(case["sinks"], max(0, n - case["window"]))) for n in lengths)
    flops = 4 * D * G * H * seen
    bytes_ = 100 * H * seen + 2 * case["batch"] * H * G * D * es
    if case["op"] == "shared":
        flops += 4 * D * G * H * case["batch"] * case["prefix"]
        bytes_ += 100 * H * case["prefix"]
    return {"bytes": bytes_, "flops": flops}


# ---------------------------------------------------------------------------------- 64-bit results
def _exact_rope(x, st):
    """x float64 [T, heads, 128]; each pair as a complex number times cos + i sin."""
    case = st["case"]
    rot, half = case["rot"], case["rot"] // 2
    tab = st["cos_sin"].double()
    turn = torch.empty((x.shape[0], half), dtype=torch.complex128, device=x.device)
    lo = 0
    for a, width in enumerate(_sections(case)):
        rows = tab[st["positions"][a].long()]
        turn[:, lo:lo + width] = torch.complex(rows[:, lo:lo + width], rows[:, half + lo:half + lo + width])
        lo += width
    out = x.clone()
    if case["interleaved"]:
        z = torch.view_as_complex(x[..., :rot].reshape(x.shape[:-1] + (half, 2)).contiguous()) * turn[:, None]
        out[..., :rot] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :half].contiguous(), x[..., half:rot].contiguous()) * turn[:, None]
        out[..., :half], out[..., half:rot] = z.real, z.imag
    return out


def _hadamard(signs):
    i = torch.arange(D, device=signs.device)
    ones = (i[:, None] & i[None]).unsqueeze(-1) >> torch.arange(7, device=signs.device) & 1
    return (1 - 2 * (ones.sum(-1) % 2)).double() * signs[0].double()     # H diag(D)


def _exact_append(st):
    case = st["case"]
    _, nc, scale, least, _ = _fields(st["pages"].clone())
    nc, scale, least = nc.double(), scale.double(), least.double()
    page = case["page"]
    k = _exact_rope(st["k"].double(), st)
    y = k @ _hadamard(st["signs"]).T
    norm2 = (k * k).sum(-1)
    new_nc = 128.0 * norm2 / y.abs().sum(-1)
    v = st["v"].double().clamp(-F16_MAX, F16_MAX).unflatten(-1, (4, 32))
    grid = torch.arange(0x7C00, device=v.device, dtype=torch.int32).to(torch.int16).view(torch.float16).double()
    lo, hi = v.amin(-1), v.amax(-1)
    every = torch.cat([-grid.flip(0), grid[1:]])
    m = every[torch.searchsorted(every, lo.contiguous(), right=True) - 1]
    at = torch.searchsorted(15.0 * grid, (hi - m).contiguous())
    s = grid[at]
    s = torch.where(m + 15.0 * s > F16_MAX, grid[(at - 1).clamp(min=0)], s)
    cu, start = st["cu"].tolist(), st["start"].tolist()
    seq = torch.cat([torch.full((cu[b + 1] - cu[b],), b, device=v.device) for b in range(case["batch"])])
    at = torch.cat([torch.arange(start[b], start[b] + cu[b + 1] - cu[b], device=v.device) for b in range(case["batch"])])
    pg, blk, tok = st["table"][seq, at // page].long(), at % page // BLOCK, at % BLOCK
    nc[pg, :, blk, tok] = new_nc
    for g in range(4):
        scale[pg, :, blk, 32 * g + tok] = s[..., g]
        least[pg, :, blk, 32 * g + tok] = m[..., g]
    return {"q": _exact_rope(st["q"].double(), st), "bits": None, "nc": nc, "scale": scale, "min": least, "codes": None}


def _exact_tokens(pages, table_row, h, t):
    """Signs, values and N / C in float64 of tokens t (a tensor) of one sequence and kv-head."""
    page = pages.shape[2] * BLOCK
    blocks = pages[table_row[t // page].long(), h, t % page // BLOCK]        # [tokens, 3200]
    tok = (t % BLOCK)[:, None]
    byte = torch.arange(16, device=t.device)[None]
    row = 8 * ((tok >> 1) % 4) + 2 * (tok >> 3) + tok % 2
    bits = blocks.gather(1, 16 * row + byte).long()
    sign = 2.0 * ((bits[..., None] >> torch.arange(8, device=t.device)) & 1).double().flatten(1) - 1.0
    ch = torch.arange(D, device=t.device)[None]
    j = tok % 8
    nibble = j // 2 + 4 * (j % 2)
    code = blocks.gather(1, 1152 + 16 * ch + 4 * (tok // 8) + nibble // 2).long()
    code = torch.where(nibble % 2 == 1, code >> 4, code & 15).double()
    half = blocks[:, 640:1152].contiguous().view(torch.float16).double()     # [tokens, 256]: scales, then minima
    group = 32 * (ch // 32) + tok
    v = half.gather(1, 128 + group) + half.gather(1, group) * code
    nc = blocks[:, 512:640].contiguous().view(torch.float32).double().gather(1, tok)[:, 0]
    return sign, v, nc


def _exact_rows(q, had, sign, v, nc):
    """(max, sum, weighted values) of softmax over the tokens for query rows q [rows, 128]."""
    z = q.double() @ had.T
    lo = z.amin(-1, keepdim=True)
    step = (z.amax(-1, keepdim=True) - lo) / 15.0
    code = torch.where(step > 0, torch.floor((z - lo) / step + 0.5).clamp(0, 15), torch.zeros_like(z))
    est = (lo + step * code) @ sign.T * nc / 128.0 * D ** -0.5
    m = est.amax(-1, keepdim=True)
    p = (est - m).exp()
    return m, p.sum(-1, keepdim=True), p @ v


def _exact_over(pages, table_row, h, tokens, q, had):
    m = torch.full((q.shape[0], 1), -math.inf, dtype=torch.float64, device=q.device)
    l, o = torch.zeros_like(m), torch.zeros((q.shape[0], D), dtype=torch.float64, device=q.device)
    for part in tokens.split(65536):
        m2, l2, o2 = _exact_rows(q, had, *_exact_tokens(pages, table_row, h, part))
        top = torch.maximum(m, m2)
        a, b = (m - top).exp(), (m2 - top).exp()
        m, l, o = top, a * l + b * l2, a * o + b * o2
    return m, l, o


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    B, H, G = case["batch"], case["kv_heads"], case["group"]
    had = _hadamard(st["signs"])
    out = torch.empty((B, H * G, D), dtype=torch.float64, device="cuda")
    lengths = st["lengths"].tolist()
    for h in range(H):
        heads = slice(h * G, (h + 1) * G)
        if case["op"] == "shared":
            t = torch.arange(case["prefix"], device="cuda")
            pre = _exact_over(st["pages"], st["prefix_pages"], h, t, st["q"][:, heads].reshape(B * G, D), had)
        for b in range(B):
            n = lengths[b]
            t = torch.arange(n, device="cuda")
            if case.get("window"):
                t = t[(t >= n - case["window"]) | (t < case["sinks"])]
            m, l, o = _exact_over(st["pages"], st["table"][b], h, t, st["q"][b, heads], had)
            if case["op"] == "shared":
                m0, l0, o0 = (x[b * G:(b + 1) * G] for x in pre)
                top = torch.maximum(m, m0)
                a, c = (m - top).exp(), (m0 - top).exp()
                l, o = a * l + c * l0, a * o + c * o0
            out[b, heads] = o / l
    return out
