"""Operators measured on a GPU: the 16-bit paged key/value cache (rotating
write, read back, attention over it) and latent attention (its paged cache, the
absorbed form over it and the expanded form for prompts).

``run`` computes a case in elementary torch operations, or, where ``own`` is
true, through attention_forward_gb300.fa.  Lengths and counts follow from the
case alone, values from the seed.

Kinds of cases
  write     fa_paged_write: a chunk's queries and keys are rotated to their
            positions, keys and values go into the pages; with ``read``,
            fa_paged_read of the sequences so far
  paged     fa_fwd_paged: the newest tokens' attention over the pages
  lwrite    fa_latent_write: latent rows of 512 + 64 channels, the 64 rotated,
            go into the pages and the queries' 64 are rotated into place; with
            ``read``, fa_latent_read of the sequences so far
  absorbed  fa_fwd_latent: the newest tokens' attention over latent rows, whose
            first 512 channels are the values too
  expanded  fa_fwd_expanded: attention of a block of rows over keys of 128
            channels a head + 64 that the heads share, values of 128

The caches: K and V [pages, Hkv, page_size, D], latent [pages, page_size, 576];
token n of sequence b is in slot n % page_size of page table[b, n // page_size].
"""
import math
import random

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16}
LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128


def listed():
    return [
        # a batch of prompts goes into the cache, grouped heads, and comes back for
        # the attention of the chunk
        dict(name="write_B4S4096", kind="write", B=4, H=32, Hkv=8, S=4096, L=4096, page=64, D=128,
             rot=128, pairs=False, read=True, dtype="bf16"),
        # one decode step's tokens of a batch: latency; half of each head rotated
        dict(name="write_token_B32", kind="write", B=32, H=32, Hkv=8, S=1, L=701, page=16, D=128,
             rot=64, pairs=True, read=False, dtype="fp16"),
        # a serving batch's decode step over long cached sequences
        dict(name="paged_B32L8192", kind="paged", B=32, H=32, Hkv=8, Sq=1, L=8192, page=64, D=128,
             dtype="bf16", cap=0.0, bias=False),
        # one long conversation, capped scores
        dict(name="paged_B1L16384", kind="paged", B=1, H=32, Hkv=8, Sq=1, L=16384, page=16, D=128,
             dtype="bf16", cap=50.0, bias=False),
        # four drafted tokens at once, ungrouped small heads, distance bias, odd lengths
        dict(name="paged_draft_B4L701", kind="paged", B=4, H=16, Hkv=16, Sq=4, L=701, page=16,
             D=64, dtype="fp16", cap=0.0, bias=True),
        # prompts into the latent cache, and read back to be expanded
        dict(name="lwrite_B4S4096", kind="lwrite", B=4, H=16, S=4096, L=4096, page=64, width=192,
             pairs=True, read=True, dtype="bf16"),
        # one decode step's tokens
        dict(name="lwrite_token_B32", kind="lwrite", B=32, H=16, S=1, L=1500, page=64, width=576,
             pairs=True, read=False, dtype="bf16"),
        # a decode step with few heads: bytes
        dict(name="absorbed_B64H16L4096", kind="absorbed", B=64, H=16, Sq=1, L=4096, page=64,
             dtype="bf16"),
        # with many heads: the products weigh as much as the bytes
        dict(name="absorbed_B32H128L8192", kind="absorbed", B=32, H=128, Sq=1, L=8192, page=64,
             dtype="bf16"),
        # two drafted tokens of a few short sequences, fp16, small pages
        dict(name="absorbed_draft_B3L701", kind="absorbed", B=3, H=16, Sq=2, L=701, page=16,
             dtype="fp16"),
        # prompts of a training-length batch
        dict(name="expanded_B2S4096", kind="expanded", B=2, H=16, Sq=4096, Skv=4096, causal=True,
             dtype="bf16"),
        # an odd chunk of one prompt behind earlier tokens
        dict(name="expanded_chunk_B1S509", kind="expanded", B=1, H=16, Sq=509, Skv=1500,
             causal=True, dtype="fp16"),
    ]


def _spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["write", "paged", "paged", "lwrite", "absorbed", "absorbed", "expanded"])
    dtype = rng.choice(["bf16", "fp16"])
    if kind == "expanded":
        Skv, H = _spread(rng, 2, 8192), rng.choice([1, 5, 16, 32])
        Sq = rng.choice([Skv, rng.randint(1, Skv), min(Skv, rng.randint(1, 300))])
        most = 1 << 28
        B = max(1, min(8, most // (H * Sq * Skv)))
        if H * Sq * Skv > most:
            H = max(1, most // (Sq * Skv))
        return dict(kind=kind, B=rng.randint(1, B), H=H, Sq=Sq, Skv=Skv,
                    causal=rng.random() < 0.75, dtype=dtype)
    L, page = _spread(rng, 17, 16384), rng.choice([16, 32, 64, 128])
    B = rng.randint(1, 32)
    if kind == "absorbed":
        B = max(1, min(B, 131072 // L))
        return dict(kind=kind, B=B, H=rng.choice([1, 8, 16, 24, 40, 64, 128]),
                    Sq=rng.choice([1, 1, 1, 2, 3]), L=L, page=page, dtype=dtype)
    if kind == "lwrite":
        B = max(1, min(B, 16384 // L))
        return dict(kind=kind, B=B, H=rng.choice([1, 16, 40]), S=rng.choice([1, L, rng.randint(1, L)]),
                    L=L, page=page, width=rng.choice([192, 576]), pairs=rng.random() < 0.5,
                    read=rng.random() < 0.5, dtype=dtype)
    D, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    if kind == "paged":
        B = max(1, min(B, 1048576 // (L * Hkv)))
        return dict(kind=kind, B=B, H=Hkv * rng.choice([1, 3, 4, 8]), Hkv=Hkv,
                    Sq=rng.choice([1, 1, 2, 5]), L=L, page=page, D=D, dtype=dtype,
                    cap=rng.choice([0.0, 30.0]), bias=rng.random() < 0.3)
    B = max(1, min(B, 65536 // (L * Hkv)))
    return dict(kind=kind, B=B, H=Hkv * rng.choice([1, 3, 4]), Hkv=Hkv,
                S=rng.choice([1, L, rng.randint(1, L)]), L=L, page=page, D=D,
                rot=rng.choice([D, D // 2, 32]), pairs=rng.random() < 0.5,
                read=rng.random() < 0.5, dtype=dtype)


# ------------------------------------------------------------ what a case fixes

def _lengths(c):
    """Tokens of each sequence, the newest included: full, and shorter by up to a third."""
    rng = random.Random("lengths %d %d" % (c["B"], c["L"]))
    least = min(c["L"], max(c.get("Sq", 1), 2 * c["L"] // 3))
    return [c["L"]] + [rng.randint(least, c["L"]) for _ in range(c["B"] - 1)]


def _counts(c):
    """Tokens of a chunk that each sequence writes, the last ones of its length."""
    if c["S"] == 1:
        return [1] * c["B"]
    rng = random.Random("counts %d %d" % (c["B"], c["S"]))
    return [min(c["S"], n) if b == 0 else rng.randint(1, min(c["S"], n))
            for b, n in enumerate(_lengths(c))]


def _slopes(H):
    return [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]


def work(case):
    c = case
    if c["kind"] == "expanded":
        off, n = c["Skv"] - c["Sq"], c["Sq"] * c["Skv"]
        if c["causal"]:
            n = sum(max(0, i + off + 1) for i in range(c["Sq"]))
        rows, keys = c["B"] * c["H"] * c["Sq"], c["B"] * c["Skv"]
        return {"bytes": rows * (2 * (NOPE + ROPE + VALUE) + 4)
                + keys * 2 * (c["H"] * (NOPE + VALUE) + ROPE),
                "flops": 2.0 * (NOPE + ROPE + VALUE) * c["B"] * c["H"] * n}
    tokens = sum(_lengths(c))
    pages = sum(-(-n // c["page"]) for n in _lengths(c))
    if c["kind"] in ("paged", "absorbed"):
        rows = c["B"] * c["H"] * c["Sq"]
        pairs = c["H"] * sum(n * c["Sq"] - c["Sq"] * (c["Sq"] - 1) // 2 for n in _lengths(c))
        if c["kind"] == "paged":
            return {"bytes": tokens * c["Hkv"] * 4 * c["D"] + rows * (4 * c["D"] + 4) + 4 * pages,
                    "flops": 4.0 * c["D"] * pairs}
        return {"bytes": tokens * 2 * (LATENT + ROPE) + rows * (2 * (2 * LATENT + ROPE) + 4)
                + 4 * pages,
                "flops": 2.0 * (2 * LATENT + ROPE) * pairs}
    new = sum(_counts(c))
    if c["kind"] == "write":
        row, q, turned = 2 * c["Hkv"] * c["D"], c["H"] * c["D"], (c["H"] + c["Hkv"]) * c["rot"]
    else:
        row, q, turned = LATENT + ROPE, c["H"] * ROPE, (c["H"] + 1) * ROPE
    return {"bytes": 4 * new * (row + q) + (4 * tokens * row if c["read"] else 0),
            "flops": 3.0 * new * turned}


# ------------------------------------------------------------ inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _frequencies(rot):
    j = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    return (10000.0 ** (-2.0 * j / rot)).float()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, B, kind = DTYPE[c["dtype"]], c["B"], c["kind"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)

    s = {"case": c}
    if kind == "expanded":
        s["q"] = normal(B, c["H"], c["Sq"], NOPE + ROPE)
        s["kv"] = normal(B, c["H"], c["Skv"], NOPE + VALUE)
        s["k_rope"] = normal(B, c["Skv"], ROPE)
        return s
    page = c["page"]
    per = -(-c["L"] // page)
    pages = B * per + 3
    order = torch.randperm(pages, generator=gen, device="cuda")
    s["table"] = order[:B * per].view(B, per).to(torch.int32).contiguous()
    if kind in ("write", "paged"):
        s["cache"] = [normal(pages, c["Hkv"], page, c["D"]) for _ in range(2)]
    else:
        s["cache"] = normal(pages, page, LATENT + ROPE)
    s["length"] = _ints(_lengths(c))
    if kind == "paged":
        s["q"] = normal(B, c["H"], c["Sq"], c["D"]) * (2.0 if c["cap"] else 1.0)
        if c["bias"]:
            s["slopes"] = torch.tensor(_slopes(c["H"]), dtype=torch.float32, device="cuda")
    elif kind == "absorbed":
        # the latent part of a query is a product over 128 channels
        s["q"] = normal(B, c["H"], c["Sq"], LATENT + ROPE) * 0.5
    else:
        S = c["S"]
        s["count"] = _ints(_counts(c))
        s["start"] = s["length"] - s["count"]
        if kind == "write":
            s["q"] = normal(B, c["H"], S, c["D"])
            s["k"], s["v"] = normal(B, c["Hkv"], S, c["D"]), normal(B, c["Hkv"], S, c["D"])
            s["freqs"] = _frequencies(c["rot"])
            s["q_out"] = torch.zeros_like(s["q"])
        else:
            s["q"] = normal(B, c["H"], S, ROPE)
            s["c"], s["k_rope"] = normal(B, S, LATENT), normal(B, S, ROPE)
            s["freqs"] = _frequencies(ROPE)
            s["q_out"] = normal(B, c["H"], S, c["width"])  # its first channels are there already
        if c["read"]:
            shapes = ([(B, c["Hkv"], c["L"], c["D"])] * 2 if kind == "write"
                      else [(B, c["L"], LATENT), (B, c["L"], ROPE)])
            s["out"] = [torch.zeros(shape, dtype=dt, device="cuda") for shape in shapes]
    return s


# ------------------------------------------------------------ one pass

def run(state):
    if own:
        return _own(state)
    return _plain(state)


def _own(s):
    from attention_forward_gb300 import fa
    c = s["case"]
    if c["kind"] == "expanded":
        return fa.fa_fwd_expanded(s["q"], s["kv"], s["k_rope"], causal=c["causal"])
    if c["kind"] == "paged":
        return fa.fa_fwd_paged(s["q"], s["cache"], s["table"], s["length"], softcap=c["cap"],
                               slopes=s.get("slopes"))
    if c["kind"] == "absorbed":
        return fa.fa_fwd_latent(s["q"], s["cache"], s["table"], s["length"])
    if c["kind"] == "write":
        fa.fa_paged_write(s["k"], s["v"], s["cache"], s["table"], s["start"], s["count"],
                          freqs=s["freqs"], interleaved=c["pairs"], q=s["q"], q_out=s["q_out"])
        if c["read"]:
            fa.fa_paged_read(s["cache"], s["table"], count=s["length"], out=s["out"])
        return [s["q_out"], *s["cache"], *s.get("out", [])]
    fa.fa_latent_write(s["c"], s["k_rope"], s["cache"], s["table"], s["start"], s["count"],
                       freqs=s["freqs"], interleaved=c["pairs"], q_rope=s["q"], q=s["q_out"])
    if c["read"]:
        fa.fa_latent_read(s["cache"], s["table"], count=s["length"], out=s["out"])
    return [s["q_out"], s["cache"], *s.get("out", [])]


def _plain(s):
    c = s["case"]
    if c["kind"] == "expanded":
        q, kv, k_rope = s["q"].float(), s["kv"].float(), s["k_rope"].float()
        B, H, Sq, _ = q.shape
        Skv = kv.shape[2]
        k = torch.cat([kv[..., :NOPE], k_rope[:, None].expand(B, H, Skv, ROPE)], -1)
        at = torch.arange(Sq, device="cuda")[:, None] + (Skv - Sq)
        j = torch.arange(Skv, device="cuda")
        seen = j <= at if c["causal"] else torch.ones((Sq, Skv), dtype=torch.bool, device="cuda")
        o, lse = _attend(q, k, kv[..., NOPE:], seen, (NOPE + ROPE) ** -0.5)
        return o.to(s["q"].dtype), lse
    if c["kind"] in ("paged", "absorbed"):
        if c["kind"] == "paged":
            k, v = (x[s["table"].long()].float().transpose(1, 2).flatten(2, 3) for x in s["cache"])
            scale = c["D"] ** -0.5
        else:
            k = s["cache"][s["table"].long()].float().flatten(1, 2)[:, None]
            v, scale = k[..., :LATENT], (NOPE + ROPE) ** -0.5
        j = torch.arange(k.shape[2], device="cuda")
        at = s["length"].view(-1, 1, 1, 1) - c["Sq"] + torch.arange(c["Sq"], device="cuda")[:, None]
        o, lse = _attend(s["q"].float(), k, v, j <= at, scale, (at - j).abs(), c.get("cap", 0.0),
                         s.get("slopes"))
        return o.to(s["q"].dtype), lse
    S = s["q"].shape[2]
    i = torch.arange(S, device="cuda")
    b, i = (i[None] < s["count"][:, None]).nonzero(as_tuple=True)
    at = s["start"][b].long() + i
    page, slot = s["table"][b, at // c["page"]].long(), at % c["page"]
    angle = at.double()[:, None] * s["freqs"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if c["kind"] == "write":
        s["q_out"][b, :, i] = _turned(s["q"][b, :, i], cos, sin, c["pairs"])
        s["cache"][0][page, :, slot] = _turned(s["k"][b, :, i], cos, sin, c["pairs"])
        s["cache"][1][page, :, slot] = s["v"][b, :, i]
    else:
        s["q_out"][b, :, i, -ROPE:] = _turned(s["q"][b, :, i], cos, sin, c["pairs"])
        s["cache"][page, slot, :LATENT] = s["c"][b, i]
        s["cache"][page, slot, LATENT:] = _turned(s["k_rope"][b, i, None], cos, sin, c["pairs"])[:, 0]
    if c["read"]:
        i = torch.arange(c["L"], device="cuda")
        b, i = (i[None] < s["length"][:, None]).nonzero(as_tuple=True)
        page, slot = s["table"][b, i // c["page"]].long(), i % c["page"]
        if c["kind"] == "write":
            for x, out in zip(s["cache"], s["out"]):
                out[b, :, i] = x[page, :, slot]
        else:
            rows = s["cache"][page, slot]
            s["out"][0][b, i], s["out"][1][b, i] = rows[:, :LATENT], rows[:, LATENT:]
    cache = s["cache"] if c["kind"] == "write" else [s["cache"]]
    return [s["q_out"], *cache, *s.get("out", [])]


def _turned(x, cos, sin, pairs):
    """Rows [n, heads, D] rotated over their first channels, in their type."""
    y, half = x.float(), cos.shape[-1]
    if pairs:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., 2 * half:]], -1).to(x.dtype)


def _attend(q, k, v, seen, scale, distance=None, cap=0.0, slopes=None):
    B, H, Sq, D = q.shape
    Hkv = k.shape[1]
    scores = torch.matmul(q.reshape(B, Hkv, (H // Hkv) * Sq, D), k.transpose(2, 3)) * scale
    scores = scores.view(B, H, Sq, -1)
    if cap:
        scores = cap * torch.tanh(scores / cap)
    if slopes is not None:
        scores = scores - slopes.view(1, -1, 1, 1) * distance
    scores = torch.where(seen, scores, -torch.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, -1, p.shape[-1]), v).view(B, H, Sq, v.shape[-1])
    return (o / torch.where(total > 0, total, 1.0),
            (top + torch.log(total)).squeeze(-1))


# ------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["kind"] in ("paged", "absorbed", "expanded"):
        return _exact_attention(s, c)
    return _exact_write(s, c)


def _exact_attention(s, c):
    B, H, Sq, D = s["q"].shape
    width = {"paged": D, "absorbed": LATENT, "expanded": VALUE}[c["kind"]]
    scale = 1.0 / math.sqrt(D if c["kind"] == "paged" else NOPE + ROPE)
    o = torch.zeros((B, H, Sq, width), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, Sq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        L = c["Skv"] if c["kind"] == "expanded" else int(s["length"][b])
        i = torch.arange(Sq, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None, :]
        gone = j > i + (L - Sq)
        if c["kind"] == "expanded":
            gone = gone & c["causal"]
        else:
            n = torch.arange(L, device="cuda")
            page, slot = s["table"][b][n // c["page"]].long(), n % c["page"]
        for h in range(H):
            q = s["q"][b, h].double()
            if c["kind"] == "expanded":
                row = s["kv"][b, h].double()
                x = q[:, :NOPE] @ row[:, :NOPE].T + q[:, NOPE:] @ s["k_rope"][b].double().T
                values = row[:, NOPE:]
            elif c["kind"] == "absorbed":
                if h == 0:
                    keys = s["cache"][page, slot].double()
                x, values = q @ keys.T, keys[:, :LATENT]
            else:
                if h % (H // c["Hkv"]) == 0:
                    keys, values = (y[page, h // (H // c["Hkv"]), slot].double() for y in s["cache"])
                x = q @ keys.T
            x = x * scale
            if c.get("cap"):
                x = c["cap"] * torch.tanh(x / c["cap"])
            if c.get("bias"):
                x = x - float(s["slopes"][h]) * (i + (L - Sq) - j).abs()
            x = x.masked_fill(gone, -math.inf)
            lse[b, h] = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(lse[b, h].isfinite(), lse[b, h], 0.0)[:, None])
            o[b, h] = p @ values
    return [o, lse]


def _exact_write(s, c):
    """By sequences, the pairs of a rotation as complex numbers."""
    paged = c["kind"] == "write"
    caches = [x.double() for x in (s["cache"] if paged else [s["cache"]])]
    q_out = s["q_out"].double()
    half = s["freqs"].numel()
    for b in range(c["B"]):
        first, many = int(s["start"][b]), int(s["count"][b])
        n = torch.arange(first, first + many, device="cuda")
        page, slot = s["table"][b][n // c["page"]].long(), n % c["page"]
        angle = n.double()[:, None] * s["freqs"].double()[None, :]
        unit = torch.polar(torch.ones_like(angle), angle)

        def turned(rows):  # [..., many, D] in 64 bits
            out = rows.double().clone()
            ch = torch.arange(half, device="cuda")
            one, two = (2 * ch, 2 * ch + 1) if c["pairs"] else (ch, ch + half)
            z = torch.complex(out[..., one], out[..., two]) * unit
            out[..., one], out[..., two] = z.real, z.imag
            return out

        if paged:
            q_out[b, :, :many] = turned(s["q"][b, :, :many])
            caches[0][page, :, slot] = turned(s["k"][b, :, :many]).transpose(0, 1)
            caches[1][page, :, slot] = s["v"][b, :, :many].double().transpose(0, 1)
        else:
            q_out[b, :, :many, -ROPE:] = turned(s["q"][b, :, :many])
            caches[0][page, slot] = torch.cat([s["c"][b, :many].double(),
                                               turned(s["k_rope"][b, :many])], -1)
    outs = []
    if c["read"]:
        outs = [torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in s["out"]]
        for b, many in enumerate(_lengths(c)):
            n = torch.arange(many, device="cuda")
            page, slot = s["table"][b][n // c["page"]].long(), n % c["page"]
            if paged:
                for x, out in zip(caches, outs):
                    out[b, :, :many] = x[page, :, slot].transpose(0, 1)
            else:
                rows = caches[0][page, slot]
                outs[0][b, :many], outs[1][b, :many] = rows[:, :LATENT], rows[:, LATENT:]
    return [q_out, *caches, *outs]
