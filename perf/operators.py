"""The serving and training operators around the attention kernels, as measurable cases.

Four kinds of pass, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and as the library's calls:

* ``norm_rope``      -- RMS norm of every query and key head with the rotary
  position embedding in the same pass (packed batches, before the attention);
* ``norm_rope_bwd``  -- its gradients: dQ, dK and the two norm weights';
* ``append``         -- new keys (normed, rotated) and values into a paged KV
  cache, the new queries rotated along;
* ``attend``         -- attention of new tokens (a prompt chunk, or one token a
  sequence) over the paged cache.

Head counts, head sizes and lengths are the library's own workloads' (32 or 16
heads, head sizes 64 and 128, packed batches of 16,384 tokens, caches of 4,096
to 32,768 tokens) and their grouped-head variants.
"""

import random

import torch

own = False

_EPS = 1e-6
_BASE = 10000.0


# ------------------------------------------------------------------ cases --

def _rows(name, op, tokens, heads, kv_heads, dim, rotary, interleaved, norm, max_pos):
    return dict(name=name, op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim,
                rotary=rotary, interleaved=interleaved, norm=norm, max_pos=max_pos)


def _paged(name, op, seqs, new_lo, new_hi, ctx_lo, ctx_hi, heads, kv_heads, dim, page, lens,
           **more):
    return dict(name=name, op=op, seqs=seqs, new_lo=new_lo, new_hi=new_hi, ctx_lo=ctx_lo,
                ctx_hi=ctx_hi, heads=heads, kv_heads=kv_heads, dim=dim, page=page, lens=lens,
                **more)


def listed():
    return [
        # The new tokens of 32 sequences in one decoding step of one layer.
        _rows("norm_rope decode step", "norm_rope", 32, 32, 8, 128, 128, False, True, 32768),
        # One packed training micro-batch, as many key heads as query heads.
        _rows("norm_rope packed 16k", "norm_rope", 16384, 32, 32, 128, 128, False, True, 16384),
        # Its backward pass.
        _rows("norm_rope_bwd packed 16k", "norm_rope_bwd", 16384, 32, 32, 128, 128, False, True,
              16384),
        # A ragged micro-batch of a small model: grouped heads, half of each head rotated.
        _rows("norm_rope_bwd ragged", "norm_rope_bwd", 4999, 15, 5, 64, 32, True, True, 8192),
        # One decoding step: a token each of 64 sequences, norms, rotation and append.
        _paged("append decode step", "append", 64, 1, 1, 4095, 32767, 32, 8, 128, 16, 1,
               rotary=128, interleaved=False, norm=True),
        # Prompt chunks of several requests, rotation only.
        _paged("append prompt chunks", "append", 5, 1000, 5000, 0, 8192, 32, 8, 128, 64, 2,
               rotary=128, interleaved=False, norm=False),
        # One user's short conversation, one token: latency.
        _paged("attend one short", "attend", 1, 1, 1, 999, 999, 32, 8, 128, 16, 3),
        # The decoding step of a full server: 64 caches of 4,096 to 32,768 tokens.
        _paged("attend decode 64", "attend", 64, 1, 1, 4095, 32767, 32, 8, 128, 64, 4),
        # Drafted tokens checked together: a few new tokens each, odd groups, head size 64.
        _paged("attend drafts", "attend", 17, 2, 5, 1, 20001, 20, 4, 64, 32, 5),
        # A long prompt in chunks: 2,048 new tokens over 32,768 cached ones.
        _paged("attend chunk over 32k", "attend", 1, 2048, 2048, 32768, 32768, 32, 8, 128, 64, 6),
        # Chunks of requests that share a step, ragged, some of them only started.
        _paged("attend ragged chunks", "attend", 7, 1, 1500, 0, 6000, 16, 4, 64, 16, 7),
        # A whole prompt at once, as many KV heads as query heads.
        _paged("attend whole prompt", "attend", 1, 8192, 8192, 0, 0, 16, 16, 128, 128, 8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "attend", "attend", "attend"])
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    heads = kv_heads * group
    turn = dict(rotary=rng.choice([dim, dim // 2]), interleaved=rng.random() < 0.4,
                norm=rng.random() < 0.7)
    if op.startswith("norm_rope"):
        tokens = _log(rng, 1, max(1, (1 << 27) // ((heads + kv_heads) * dim)))
        c = _rows("", op, min(tokens, 32768), heads, kv_heads, dim, turn["rotary"],
                  turn["interleaved"], turn["norm"], 32768)
    elif op == "append":
        seqs = _log(rng, 1, 100)
        hi = _log(rng, 1, max(1, 20000 // seqs))
        c = _paged("", op, seqs, rng.randint(1, hi), hi, 0, _log(rng, 16, 8192), heads, kv_heads,
                   dim, rng.choice([16, 32, 64, 128]), rng.randrange(1 << 20), **turn)
    else:
        page = rng.choice([16, 32, 64, 128])
        if rng.random() < 0.5:  # one or a few new tokens each
            seqs = _log(rng, 1, 100)
            ctx = _log(rng, 100, min(65536, 1600000 // seqs))
            hi = rng.choice([1, 1, 2, 4, 9])
        else:  # chunks
            seqs = _log(rng, 1, 9)
            ctx = _log(rng, 16, 24000 // seqs)
            hi = _log(rng, 10, 4000 // seqs)
        c = _paged("", op, seqs, rng.randint(1, hi), hi, ctx // 3, ctx, heads, kv_heads, dim,
                   page, rng.randrange(1 << 20))
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs --

def _lengths(c):
    r = random.Random(c["lens"])
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["seqs"])]
    kv = [n + r.randint(c["ctx_lo"], c["ctx_hi"]) for n in new]
    return new, kv


def _table(max_pos, rotary, device):
    j = torch.arange(rotary // 2, device=device, dtype=torch.float64)
    angle = torch.arange(max_pos, device=device, dtype=torch.float64)[:, None] * _BASE ** (
        -2.0 * j / rotary)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _weight(dim, g, device):
    return (1 + 0.2 * torch.randn(dim, generator=g, device=device)).to(torch.bfloat16)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0):
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
        return x.mul_(std) if std != 1.0 else x

    s = dict(case=dict(c))
    heads, kv_heads, dim = c["heads"], c["kv_heads"], c["dim"]
    if c["op"].startswith("norm_rope"):
        tokens = c["tokens"]
        # Samples of a few hundred to a few thousand tokens, packed; a decoding
        # step's tokens stand anywhere in their contexts.
        r = random.Random(seed)
        if tokens <= 256:
            pos = [r.randrange(c["max_pos"]) for _ in range(tokens)]
        else:
            pos = []
            while len(pos) < tokens:
                pos.extend(range(min(r.randint(64, 4096), tokens - len(pos), c["max_pos"])))
        s["pos"] = torch.tensor(pos, dtype=torch.int32, device=dev)
        s["table"] = _table(c["max_pos"], c["rotary"], dev)
        # Q and K as slices of one projection's output, [tokens, (Q + K + V) heads, dim].
        qkv = normal(tokens, heads + 2 * kv_heads, dim, std=1.5)
        s["q"], s["k"] = qkv[:, :heads], qkv[:, heads:heads + kv_heads]
        s["wq"] = _weight(dim, g, dev) if c["norm"] else None
        s["wk"] = _weight(dim, g, dev) if c["norm"] else None
        if c["op"] == "norm_rope_bwd":
            s["gq"], s["gk"] = normal(tokens, heads, dim), normal(tokens, kv_heads, dim)
        return s

    new, kv = _lengths(c)
    page = c["page"]
    counts = [-(-n // page) for n in kv]
    total, most = sum(counts), max(counts)
    pages = total + 7
    order = torch.randperm(pages, generator=g, device=dev)[:total].to(torch.int32)
    at = torch.arange(most, device=dev)[None, :]
    n = torch.tensor(counts, device=dev)[:, None]
    first = (n.cumsum(0) - n)
    s["pages"] = torch.where(at < n, order[(first + at).clamp(max=total - 1)],
                             torch.zeros((), dtype=torch.int32, device=dev)).contiguous()
    s["kc"] = normal(pages, page, kv_heads, dim)
    s["vc"] = normal(pages, page, kv_heads, dim)
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["kv"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    s["most_new"], s["most_kv"] = max(new), max(kv)
    if c["op"] == "append":
        qkv = normal(cu[-1], heads + 2 * kv_heads, dim, std=1.5)
        s["q"], s["k"], s["v"] = qkv.split([heads, kv_heads, kv_heads], 1)
        s["table"] = _table(max(kv), c["rotary"], dev)
        s["wq"] = _weight(dim, g, dev) if c["norm"] else None
        s["wk"] = _weight(dim, g, dev) if c["norm"] else None
    else:
        s["q"] = normal(cu[-1], heads, dim)
    return s


# ------------------------------------------------------------ plain forms --

def _turn(x, cos, sin, interleaved):
    """The rotation of the first 2 * cos.shape[-1] features; [T, H, D] by [T, 1, R / 2]."""
    half = cos.shape[-1]
    a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
    if interleaved:
        pair = x[..., :2 * half].unflatten(-1, (half, 2))
        a, b = pair[..., 0], pair[..., 1]
    y0, y1 = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([y0, y1], -1).flatten(-2) if interleaved else torch.cat([y0, y1], -1)
    return torch.cat([y, rest], -1)


def _angles(table, pos):
    row = table[pos.long()][:, None, :]
    return row.chunk(2, -1)


def _norm_turn(x, w, cos, sin, interleaved):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * w.float()
    return _turn(x, cos, sin, interleaved)


def _norm_turn_grad(dy, x, w, cos, sin, interleaved):
    g = _turn(dy.float(), cos, -sin, interleaved)
    if w is None:
        return g.to(dy.dtype), None
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS)
    hat = x * r
    u = g * w.float()
    dx = r * (u - hat * (u * hat).mean(-1, keepdim=True))
    # The weight's gradient is a sum over every token and head.
    return dx.to(dy.dtype), (g * hat).sum((0, 1), dtype=torch.float64).float()


def _sequence_of(s):
    """Each new token's sequence and position."""
    t = torch.arange(s["q"].shape[0], device=s["q"].device)
    b = torch.searchsorted(s["cu"].long(), t, right=True) - 1
    pos = s["kv"].long()[b] - (s["cu"].long()[b + 1] - t)
    return b, pos


def _append_plain(s):
    c = s["case"]
    b, pos = _sequence_of(s)
    cos, sin = _angles(s["table"], pos)
    page, slot = s["pages"].long()[b, pos // c["page"]], pos % c["page"]
    k = _norm_turn(s["k"], s["wk"], cos, sin, c["interleaved"])
    s["kc"][page, slot] = k.to(s["kc"].dtype)
    s["vc"][page, slot] = s["v"]
    q = _norm_turn(s["q"], s["wq"], cos, sin, c["interleaved"]).to(s["q"].dtype)
    return q, s["kc"], s["vc"]


def _attend_plain(s):
    c = s["case"]
    heads, kv_heads, dim = c["heads"], c["kv_heads"], c["dim"]
    group, seqs, most_new, most_kv = heads // kv_heads, c["seqs"], s["most_new"], s["most_kv"]
    dev = s["q"].device
    b, pos = _sequence_of(s)
    i = torch.arange(len(b), device=dev) - s["cu"].long()[b]
    # Every sequence padded to the longest: queries [B, KV heads, group * new, D].
    q = torch.zeros(seqs, most_new, heads, dim, device=dev)
    q[b, i] = s["q"].float() * dim ** -0.5
    q = q.view(seqs, most_new, kv_heads, group, dim).permute(0, 2, 3, 1, 4).flatten(2, 3)
    at = torch.full((seqs, most_new), -1, device=dev)
    at[b, i] = pos
    key = torch.arange(most_kv, device=dev)
    seen = (key <= at[..., None])[:, None, None]
    pages = s["pages"].long()
    k = s["kc"][pages].flatten(1, 2)[:, :most_kv].permute(0, 2, 3, 1).float()
    x = torch.matmul(q, k).view(seqs, kv_heads, group, most_new, most_kv)
    del k
    x = x.masked_fill_(~seen, -torch.inf)
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = s["vc"][pages].flatten(1, 2)[:, :most_kv].permute(0, 2, 1, 3)
    v = torch.where((key < s["kv"][:, None])[:, None, :, None], v, 0).float()
    o = torch.matmul(p.flatten(2, 3), v).view(seqs, kv_heads, group, most_new, dim)
    o = (o / total).permute(0, 3, 1, 2, 4).flatten(2, 3)[b, i].to(s["q"].dtype)
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[b, i]
    return o, lse.contiguous()


# ------------------------------------------------------------------- pass --

def run(state):
    s = state
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "norm_rope":
        cos, sin = _angles(s["table"], s["pos"])
        return tuple(_norm_turn(x, w, cos, sin, c["interleaved"]).to(x.dtype)
                     for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])))
    if c["op"] == "norm_rope_bwd":
        cos, sin = _angles(s["table"], s["pos"])
        dq, dwq = _norm_turn_grad(s["gq"], s["q"], s["wq"], cos, sin, c["interleaved"])
        dk, dwk = _norm_turn_grad(s["gk"], s["k"], s["wk"], cos, sin, c["interleaved"])
        return dq, dk, dwq, dwk
    return _append_plain(s) if c["op"] == "append" else _attend_plain(s)


def _run_own(s, c):
    from long_context_gb300 import cpattn
    if c["op"] == "norm_rope":
        return cpattn.qk_norm_rope(s["q"], s["k"], s["pos"], s["table"], q_weight=s["wq"],
                                   k_weight=s["wk"], eps=_EPS, interleaved=c["interleaved"])
    if c["op"] == "norm_rope_bwd":
        return cpattn.qk_norm_rope_bwd(s["gq"], s["gk"], s["q"], s["k"], s["pos"], s["table"],
                                       q_weight=s["wq"], k_weight=s["wk"], eps=_EPS,
                                       interleaved=c["interleaved"])
    if c["op"] == "append":
        q = cpattn.paged_append(s["k"], s["v"], s["kc"], s["vc"], s["pages"], s["cu"], s["kv"],
                                rope_table=s["table"], interleaved=c["interleaved"], q=s["q"],
                                q_weight=s["wq"], k_weight=s["wk"], eps=_EPS)
        return q, s["kc"], s["vc"]
    return cpattn.paged_attn(s["q"], s["kc"], s["vc"], s["pages"], s["cu"], s["kv"],
                             max_seqlen=s["most_new"], max_kv_len=s["most_kv"])


# ------------------------------------------------------------------- work --

def work(case):
    c = case
    heads, kv_heads, dim = c["heads"], c["kv_heads"], c["dim"]
    if c["op"].startswith("norm_rope"):
        elements = c["tokens"] * (heads + kv_heads) * dim
        passes = 2 if c["op"] == "norm_rope" else 3
        if c["op"] == "norm_rope_bwd" and not c["norm"]:
            passes = 2  # rotated back; the inputs are not needed
        rows = min(c["tokens"], c["max_pos"])
        return dict(bytes=2 * passes * elements + 4 * c["tokens"] + 4 * rows * c["rotary"],
                    flops=(12 if passes == 2 else 24) * elements)
    new, kv = _lengths(c)
    n = sum(new)
    if c["op"] == "append":
        elements = n * (heads + 2 * kv_heads) * dim
        pages = sum(-(-b // c["page"]) - (b - a) // c["page"] for a, b in zip(new, kv))
        return dict(bytes=4 * elements + 4 * pages + 8 * c["seqs"] + 4 * c["rotary"] * n,
                    flops=12 * n * (heads + kv_heads) * dim)
    pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(new, kv))
    pages = sum(-(-b // c["page"]) for b in kv)
    return dict(bytes=4 * n * heads * dim + 4 * n * heads + 4 * sum(kv) * kv_heads * dim
                + 4 * pages + 8 * c["seqs"], flops=4 * dim * heads * pairs)


# ------------------------------------------------------------------ exact --

def _complex_rows(x, R, interleaved):
    """The first R features as R / 2 complex numbers, and the rest."""
    z = x[..., :R]
    z = (torch.complex(z[..., 0::2].contiguous(), z[..., 1::2].contiguous()) if interleaved
         else torch.complex(z[..., :R // 2].contiguous(), z[..., R // 2:].contiguous()))
    return z, x[..., R:]


def _from_complex(z, rest, interleaved):
    y = torch.view_as_real(z).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)
    return torch.cat([y, rest], -1)


def _exact_rows(x, w, unit, c):
    """A normed and turned block of rows, by multiplication with unit complex numbers."""
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / c["dim"] + _EPS).sqrt() * w.double()
    z, rest = _complex_rows(x, c["rotary"], c["interleaved"])
    return _from_complex(z * unit, rest, c["interleaved"])


def _exact_grads(dy, x, w, unit, c):
    """The gradients through the complex form: the product's transpose is the conjugate."""
    z, rest = _complex_rows(dy.double(), c["rotary"], c["interleaved"])
    back = _from_complex(z * unit.conj(), rest, c["interleaved"])
    if w is None:
        return back, None
    x, w = x.double(), w.double()
    d = c["dim"]
    square = x.pow(2).sum(-1, keepdim=True) / d + _EPS
    inner = (back * w * x).sum(-1, keepdim=True)
    dx = back * w / square.sqrt() - x * inner / (d * square * square.sqrt())
    return dx, (back * x / square.sqrt()).sum((0, 1))


def _unit(table, pos):
    row = table.double()[pos.long()]
    cos, sin = row[:, :row.shape[1] // 2], row[:, row.shape[1] // 2:]
    return torch.complex(cos.contiguous(), sin.contiguous())[:, None, :]


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "norm_rope":
        u = _unit(s["table"], s["pos"])
        return _exact_rows(s["q"], s["wq"], u, c), _exact_rows(s["k"], s["wk"], u, c)
    if c["op"] == "norm_rope_bwd":
        u = _unit(s["table"], s["pos"])
        dq, dwq = _exact_grads(s["gq"], s["q"], s["wq"], u, c)
        dk, dwk = _exact_grads(s["gk"], s["k"], s["wk"], u, c)
        return dq, dk, dwq, dwk
    new, kv = _lengths(c)
    heads, kv_heads, dim, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    out, row = [], 0
    if c["op"] == "append":
        kc, vc = s["kc"].double(), s["vc"].double()
        for b, (n, total) in enumerate(zip(new, kv)):
            pos = torch.arange(total - n, total, device="cuda")
            u = _unit(s["table"], pos)
            where = s["pages"][b].long()[pos // page] * page + pos % page
            kc.view(-1, kv_heads, dim)[where] = _exact_rows(s["k"][row:row + n], s["wk"], u, c)
            vc.view(-1, kv_heads, dim)[where] = s["v"][row:row + n].double()
            out.append(_exact_rows(s["q"][row:row + n], s["wq"], u, c))
            row += n
        return torch.cat(out), kc, vc
    lses = []
    for b, (n, total) in enumerate(zip(new, kv)):
        used = s["pages"][b, :-(-total // page)].long()
        k = s["kc"][used].flatten(0, 1)[:total].double()
        v = s["vc"][used].flatten(0, 1)[:total].double()
        q = s["q"][row:row + n].double()
        row += n
        hidden = (torch.arange(total, device="cuda")[None, :]
                  > torch.arange(total - n, total, device="cuda")[:, None])
        o = torch.empty(n, heads, dim, dtype=torch.float64, device="cuda")
        lse = torch.empty(n, heads, dtype=torch.float64, device="cuda")
        for h in range(heads):
            kh, vh = k[:, h * kv_heads // heads], v[:, h * kv_heads // heads]
            x = (q[:, h] @ kh.T) / dim ** 0.5
            x.masked_fill_(hidden, -torch.inf)
            lse[:, h] = torch.logsumexp(x, 1)
            o[:, h] = (x - lse[:, h, None]).exp_() @ vh
        out.append(o)
        lses.append(lse)
    return torch.cat(out), torch.cat(lses)
