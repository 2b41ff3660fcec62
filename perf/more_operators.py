"""Operators around a paged KV cache held in 4 bits: the cases that are measured, their plain form and their definition in 64 bits.

Four operators, as a serving step uses them:
  axes    RMS norm of every query and key head and the rotation by positions of several axes (time, height, width);
  store   new key / value rows into 4-bit codes with a scale and a minimum per (token, head), and the same rows read back, as a
          prompt's owner hands them on;
  read    rows of token ranges back from the cache (4 or 8 bits);
  attend  attention of 1..n query tokens per request over the 4-bit codes (grouped heads, ragged lengths, windows).
"""
import math
import random

import torch

own = False

FP8 = torch.float8_e4m3fn
LIMIT = 2.0 ** 120              # larger magnitudes are held as this one


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 48 requests, positions on three axes
        dict(name="axes_decode_b48", op="axes", T=48, H=32, Hk=8, D=128, rot=128, off=0, style="halves", axes=3, cut=False, far=32768),
        # patches of images and video beside text, an odd number of tokens, axes taken in turn pair by pair
        dict(name="axes_prompt", op="axes", T=6143, H=32, Hk=8, D=128, rot=128, off=0, style="halves", axes=3, cut=True, far=32768),
        # one new token for each of 48 requests, in the middle of their blocks
        dict(name="store_decode_b48", op="store", B=48, q=1, ctx=16384, ragged=True, Hk=8, D=128, bs=16),
        # prompts of up to 2,500 tokens at once
        dict(name="store_prompt", op="store", B=6, q=2500, ctx=4096, ragged=True, Hk=8, D=128, bs=32),
        # whole prefixes of 16 requests handed on
        dict(name="read_prefix_b16", op="read", bits=4, B=16, n=8192, ctx=8192, ragged=True, Hk=8, D=128, bs=16, shared=False),
        # the last 2,000 latent rows of 8 requests of the 8-bit cache
        dict(name="read_latent_8bit", op="read", bits=8, B=8, n=2000, ctx=32768, ragged=True, Hk=1, D=512, bs=64, shared=True),
        # one token over one context of 8K: the smallest call
        dict(name="attend_8k_b1", op="attend", B=1, q=1, ctx=8192, ragged=False, mixed=False, H=32, Hk=8, D=128, bs=64, window=0),
        # a decode batch, ragged contexts, small blocks
        dict(name="attend_decode_b64", op="attend", B=64, q=1, ctx=16384, ragged=True, mixed=False, H=32, Hk=8, D=128, bs=16, window=0),
        # verification of drafted tokens: up to 5 query tokens per request
        dict(name="attend_drafts_b16", op="attend", B=16, q=5, ctx=8192, ragged=True, mixed=False, H=64, Hk=8, D=128, bs=32, window=0),
        # prompt chunks of up to 1,024 tokens against their contexts: the compute-bound end
        dict(name="attend_chunk", op="attend", B=4, q=1024, ctx=8192, ragged=True, mixed=False, H=32, Hk=8, D=128, bs=64, window=0),
        # a server's mixed step: two prompt chunks among 30 requests that decode
        dict(name="attend_mixed_b32", op="attend", B=32, q=512, ctx=8192, ragged=True, mixed=True, H=32, Hk=8, D=128, bs=16, window=0),
        # wide heads with a sliding window over long contexts
        dict(name="attend_window_d256", op="attend", B=24, q=1, ctx=32768, ragged=True, mixed=False, H=16, Hk=4, D=256, bs=128, window=4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["axes", "store", "read", "attend", "attend", "attend"])
    bs = rng.choice([16, 32, 64, 128])
    if op == "axes":
        D = rng.choice([64, 96, 128, 256, 512])
        H = rng.choice([4, 12, 16, 24, 32, 64])
        Hk = rng.choice([1, 2, 4, 8])
        rot = rng.choice([r for r in (32, 64, D) if r <= D])
        return dict(op=op, T=_log(rng, 1, max(1, min(8000, 31000000 // ((H + Hk) * D)))), H=H, Hk=Hk, D=D, rot=rot,
                    off=rng.choice([0, D - rot]), style=rng.choice(["pairs", "halves"]), axes=rng.choice([2, 3, 3, 4]),
                    cut=rng.random() < 0.5, far=_log(rng, 1024, 1048576))
    if op == "store":
        D, Hk, B = rng.choice([128, 128, 256]), rng.choice([1, 2, 4, 8]), _log(rng, 1, 64)
        q = _log(rng, 1, max(1, min(2500, 14000000 // (B * Hk * D))))
        return dict(op=op, B=B, q=q, ctx=q + _log(rng, 16, 4096), ragged=True, Hk=Hk, D=D, bs=bs)
    if op == "read":
        bits = rng.choice([4, 4, 8])
        shared = bits == 8 and rng.random() < 0.5
        D = rng.choice([128, 256, 512]) if shared else rng.choice([128, 128, 256])
        Hk, B = 1 if shared else rng.choice([1, 2, 4, 8]), _log(rng, 1, 64)
        n = _log(rng, 1, max(1, min(16384, 60000000 // (B * Hk * D))))
        return dict(op=op, bits=bits, B=B, n=n, ctx=n + _log(rng, 16, 4096), ragged=True, Hk=Hk, D=D, bs=bs, shared=shared)
    D, Hk, G = rng.choice([128, 128, 256]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 12, 16])
    kind = rng.random()
    q = 1 if kind < 0.5 else _log(rng, 2, 8) if kind < 0.75 else _log(rng, 9, 600)
    # the products of the largest listed case, and its bytes, at most: B * H * q * ctx scores of D products
    B = _log(rng, 1, max(1, min(64, 200000 // (q * Hk * G))))
    most = max(64, min(32768, 900000000 // (B * Hk * D), int(2e11) // (4 * D * B * q * Hk * G)))
    ctx = max(q, _log(rng, 16, most))
    return dict(op=op, B=B, q=q, ctx=ctx, ragged=rng.random() < 0.8, mixed=q > 8 and B > 3 and rng.random() < 0.5, H=Hk * G, Hk=Hk,
                D=D, bs=bs, window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]))


def _lengths(c):
    """(lengths, new or wanted tokens) of each request: by the case alone, so that its work is known."""
    m = c["n"] if c["op"] == "read" else c["q"]
    r = random.Random(c["B"] * 7919 + c["ctx"] * 31 + m)
    if c.get("mixed"):
        q = [r.randint(max(1, m // 2), m) if i % 16 == 5 else 1 for i in range(c["B"])]
    else:
        q = [r.randint(max(1, m // 4), m) if c["ragged"] else m for _ in range(c["B"])]
        q[0] = m
    n = [max(qi, r.randint(max(1, c["ctx"] // 8), c["ctx"])) if c["ragged"] else c["ctx"] for qi in q]
    n[0] = max(c["ctx"], q[0])
    return n, q


# ---------------------------------------------------------------------------------------------- inputs
def _quantised(x):
    """bf16 rows [..., D]: codes 0..15 (uint8), scale and minimum (bf16), by the definition in 32 bits."""
    x = x.float()
    x = torch.where(torch.isfinite(x), x, 0.0).clamp(-LIMIT, LIMIT)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi - lo) / 15).bfloat16()
    n = torch.where(s > 0, torch.round((x - lo) / s.float()), 0.0).clamp(0, 15)
    return n.to(torch.uint8), s, lo.bfloat16()


def _packed(n):
    """Two codes to a byte, the even dim in the low half."""
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _filled(g, n_blocks, Hk, bs, D):
    """A filled 4-bit cache: rows whose sizes differ by a few powers of two, keys and values with a mean of their own per dim."""
    codes = torch.empty((n_blocks, Hk, bs, D // 2), dtype=torch.uint8, device="cuda")
    scale = torch.empty((n_blocks, Hk, bs, 2), dtype=torch.bfloat16, device="cuda")
    mean = 0.3 * torch.randn((Hk, 1, D), generator=g, device="cuda")
    step = max(1, (1 << 26) // (Hk * bs * D))
    for i in range(0, n_blocks, step):
        m = min(step, n_blocks - i)
        x = torch.randn((m, Hk, bs, D), generator=g, device="cuda") + mean
        x *= torch.exp2(torch.randint(-2, 2, (m, Hk, bs, 1), generator=g, device="cuda").float())
        n, s, lo = _quantised(x.bfloat16())
        codes[i:i + m] = _packed(n)
        scale[i:i + m] = torch.cat((s, lo), -1)
    return codes, scale


def _filled8(g, n_blocks, Hk, bs, D):
    """A filled 8-bit cache: e4m3 codes with a power-of-two scale per (block, head)."""
    x = torch.randn((n_blocks, Hk, bs, D), generator=g, device="cuda")
    scale = torch.exp2(torch.randint(-9, -5, (n_blocks, Hk), generator=g, device="cuda").float())
    return (x * 64).clamp(-448, 448).to(FP8).view(torch.uint8), scale


def _cache(c, s, g, n):
    """Block table (scattered blocks) for lengths n, with some blocks over."""
    bs, B = c["bs"], c["B"]
    need = [-(-x // bs) for x in n]
    width = max(need) + 2
    total = sum(need) + B + 3
    order = torch.randperm(total, generator=g, device="cuda").int()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(width, device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
    table[at] = order[:sum(need)]
    s.update(table=table, n_blocks=total, width=width)


def _handle(c, s):
    from sparse_retrieval_host_gb300.paged import PagedKV4, PagedKV8
    if c["op"] == "axes":       # any cache will do: the heads' shapes are the call's own
        return PagedKV4(batch=1, n_kv_heads=1, head_dim=128, block_tokens=64, n_blocks=1, max_blocks=1)
    held = {k: s[k] for k in ("k_codes", "k_scale", "v_codes", "v_scale", "table", "len") if k in s}
    more = dict(batch=c["B"], n_kv_heads=c["Hk"], head_dim=c["D"], block_tokens=c["bs"], n_blocks=s["n_blocks"], max_blocks=s["width"],
                buffers=held)
    return PagedKV8(shared_kv=c["shared"], **more) if c.get("bits") == 8 else PagedKV4(**more)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    s = dict(case=c)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    bf = lambda *shape: torch.randn(shape, generator=g, device="cuda").bfloat16()  # noqa: E731
    if c["op"] == "axes":
        T, H, Hk, D, half = c["T"], c["H"], c["Hk"], c["D"], c["rot"] // 2
        qkv = bf(T, (H + 2 * Hk) * D)                       # one projection's rows: queries, keys, values side by side
        s["q"] = qkv[:, :H * D].view(T, H, D)
        s["k"] = qkv[:, H * D:(H + Hk) * D].view(T, Hk, D)
        s["wq"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
        s["wk"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
        s["pos"] = torch.randint(0, c["far"], (c["axes"], T), generator=g, device="cuda", dtype=torch.int32)
        pair = torch.arange(half, device="cuda")
        # the pairs of each axis in a row, or in turn
        s["axis"] = (pair % c["axes"] if c["cut"] else pair * c["axes"] // half).to(torch.uint8)
        s["freq"] = 10000.0 ** (-pair.double() / half)
        s["oq"] = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
        s["ok"] = torch.empty((T, Hk, D), dtype=torch.bfloat16, device="cuda")
    else:
        n, q = _lengths(c)
        _cache(c, s, g, n)
        s["T"] = sum(q)
        s["max_q"], s["max_len"] = max(q), max(n)
        s["cu"] = i32([sum(q[:i]) for i in range(len(q) + 1)])
        s["len"] = i32(n)
        s["start"] = i32([a - b for a, b in zip(n, q)])
        fill = _filled8 if c.get("bits") == 8 else _filled
        s["k_codes"], s["k_scale"] = fill(g, s["n_blocks"], c["Hk"], c["bs"], c["D"])
        s["v_codes"], s["v_scale"] = (s["k_codes"], s["k_scale"]) if c.get("shared") else fill(g, s["n_blocks"], c["Hk"], c["bs"], c["D"])
        if c["op"] == "attend":
            s["q"] = bf(s["T"], c["H"], c["D"])
            s["out"] = torch.empty_like(s["q"])
        else:
            s["ok"] = torch.empty((s["T"], c["Hk"], c["D"]), dtype=torch.bfloat16, device="cuda")
            s["ov"] = None if c.get("shared") else torch.empty_like(s["ok"])
        if c["op"] == "store":
            s["k"], s["v"] = bf(s["T"], c["Hk"], c["D"]), bf(s["T"], c["Hk"], c["D"])
    s["handle"] = _handle(c, s) if own else None
    return s


# ---------------------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s["case"], s, s["handle"])
    return _PLAIN[op](s["case"], s)


def _own_axes(c, s, h):
    q, k = h.norm_rope(s["q"], s["k"], pos=s["pos"], axis=s["axis"], inv_freq=s["freq"], rot_dim=c["rot"], rot_off=c["off"],
                       style=c["style"], q_weight=s["wq"], k_weight=s["wk"], eps=1e-6, q_out=s["oq"], k_out=s["ok"])
    return dict(q=q, k=k)


def _own_store(c, s, h):
    h.append(s["k"], s["v"], s["cu"])
    k, v = h.read(s["start"], s["cu"], s["T"], k_out=s["ok"], v_out=s["ov"])
    return dict(k=k, v=v, ks=s["k_scale"], vs=s["v_scale"])


def _own_read(c, s, h):
    k, v = h.read(s["start"], s["cu"], s["T"], k_out=s["ok"], v_out=s["ov"])
    return dict(k=k) if c["shared"] else dict(k=k, v=v)


def _own_attend(c, s, h):
    return h.attend(s["q"], s["cu"], scale=c["D"] ** -0.5, window=c["window"], out=s["out"])


def _norm_rope(c, s, x, w):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    angle = s["pos"][s["axis"].long()].double().t() * s["freq"]            # [T, pairs]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    r = x[..., c["off"]:c["off"] + c["rot"]]
    if c["style"] == "pairs":
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = r[..., :c["rot"] // 2], r[..., c["rot"] // 2:]
        r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((x[..., :c["off"]], r, x[..., c["off"] + c["rot"]:]), -1).bfloat16()


def _plain_axes(c, s):
    return dict(q=_norm_rope(c, s, s["q"], s["wq"]), k=_norm_rope(c, s, s["k"], s["wk"]))


def _places(c, s):
    """(block, place in it) of each row's token: rows cu[b] .. of request b are its tokens start[b] .. on."""
    i = torch.arange(s["T"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"][1:].contiguous(), i, right=True)
    pos = (s["start"][b] + i - s["cu"][b]).long()
    return s["table"][b, pos // c["bs"]].long(), pos % c["bs"]


def _store(c, s, x, codes, scale):
    block, at = _places(c, s)
    n, sc, lo = _quantised(x)
    head = torch.arange(c["Hk"], device="cuda")[None]
    codes[block[:, None], head, at[:, None]] = _packed(n)
    scale[block[:, None], head, at[:, None]] = torch.cat((sc, lo), -1)


def _unpacked(codes, scale):
    """Values of codes [..., D / 2] with (scale, minimum) [..., 2], in fp32."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    return n * scale[..., :1].float() + scale[..., 1:].float()


def _rows(c, s, codes, scale):
    block, at = _places(c, s)
    head = torch.arange(c["Hk"], device="cuda")[None]
    x = codes[block[:, None], head, at[:, None]]
    if c.get("bits") == 8:
        return (x.view(FP8).float() * scale[block][..., None]).bfloat16()
    return _unpacked(x, scale[block[:, None], head, at[:, None]]).bfloat16()


def _plain_store(c, s):
    _store(c, s, s["k"], s["k_codes"], s["k_scale"])
    _store(c, s, s["v"], s["v_codes"], s["v_scale"])
    return dict(k=_rows(c, s, s["k_codes"], s["k_scale"]), v=_rows(c, s, s["v_codes"], s["v_scale"]), ks=s["k_scale"], vs=s["v_scale"])


def _plain_read(c, s):
    k = _rows(c, s, s["k_codes"], s["k_scale"])
    return dict(k=k) if c["shared"] else dict(k=k, v=_rows(c, s, s["v_codes"], s["v_scale"]))


def _held(c, s, codes, scale):
    """The cache's values of every request, [B, Hk, tokens, D] in fp32."""
    nb = -(-s["max_len"] // c["bs"])
    tab = s["table"][:, :nb].long().clamp(min=0)
    return _unpacked(codes[tab], scale[tab]).transpose(1, 2).reshape(c["B"], c["Hk"], nb * c["bs"], c["D"])


def _plain_attend(c, s):
    B, Hk, D, m = c["B"], c["Hk"], c["D"], s["max_q"]
    G = c["H"] // Hk
    k = _held(c, s, s["k_codes"], s["k_scale"])
    cu, ln = s["cu"].long(), s["len"].long()
    nq = cu[1:] - cu[:-1]
    i = torch.arange(m, device=k.device)
    q = s["q"][(cu[:-1, None] + i).clamp(max=s["T"] - 1)].float()          # [B, m, H, D]
    q = q.view(B, m, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, m * G, D)
    p = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).view(B, Hk, m, G, -1)
    t = torch.arange(k.shape[2], device=k.device)
    del k
    at = (ln - nq)[:, None] + i                                            # each query's own position
    see = (t <= at[..., None]) & (t < ln[:, None, None])
    if c["window"]:
        see &= t > at[..., None] - c["window"]
    p.masked_fill_(~see[:, None, :, None], float("-inf"))
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _held(c, s, s["v_codes"], s["v_scale"])
    v = torch.where((t < ln[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(p.view(B, Hk, m * G, -1), v).view(B, Hk, m, G, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B, m, c["H"], D)
    row = torch.arange(s["T"], device=o.device)
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    return o[b, row - cu[b]].bfloat16()


_PLAIN = dict(axes=_plain_axes, store=_plain_store, read=_plain_read, attend=_plain_attend)
_OWN = dict(axes=_own_axes, store=_own_store, read=_own_read, attend=_own_attend)


# ---------------------------------------------------------------------------------------------- what one pass cannot do without
def _visible(c, n, q):
    """(tokens read, query-token pairs) over all requests."""
    tokens = pairs = 0
    for a, m in zip(n, q):
        w = c["window"] or a
        tokens += min(a, w + m - 1)
        if w >= a:
            pairs += m * (a - m) + m * (m + 1) // 2
        else:
            pairs += sum(min(w, a - m + i + 1) for i in range(m))
    return tokens, pairs


def work(case):
    c = case
    if c["op"] == "axes":
        values = c["T"] * (c["H"] + c["Hk"]) * c["D"]
        return dict(bytes=values * 4 + c["T"] * 4 * c["axes"] + c["D"] * 8 + c["rot"] * 4 + c["rot"] // 2, flops=values * 6)
    n, q = _lengths(c)
    T, B, bs, row = sum(q), c["B"], c["bs"], c["Hk"] * c["D"]
    copies = 1 if c.get("shared") else 2
    held = c["Hk"] * (c["D"] // 2 + 4)                                     # of a token, in 4 bits
    if c["op"] == "store":
        blocks = sum(-(-a // bs) - (a - m) // bs for a, m in zip(n, q))
        return dict(bytes=2 * T * (row * 2 + 2 * held + row * 2) + B * 12 + blocks * 4, flops=2 * T * row * 6)
    if c["op"] == "read":
        blocks = sum(-(-a // bs) - (a - m) // bs for a, m in zip(n, q))
        here = T * held if c["bits"] == 4 else T * row + blocks * c["Hk"] * 4
        return dict(bytes=copies * (here + T * row * 2) + B * 12 + blocks * 4, flops=copies * T * row * 2)
    tokens, pairs = _visible(c, n, q)
    blocks = sum(-(-min(a, (c["window"] or a) + m - 1) // bs) for a, m in zip(n, q))
    return dict(bytes=2 * tokens * held + T * c["H"] * c["D"] * 4 + B * 8 + blocks * 4, flops=4 * c["D"] * c["H"] * pairs)


# ---------------------------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    c = dict(case)
    global own
    was, own = own, False
    s = prepare(c, seed)
    own = was
    if c["op"] == "axes":
        return dict(q=_exact_axes(c, s, s["q"], s["wq"]), k=_exact_axes(c, s, s["k"], s["wk"]))
    n, q = _lengths(c)
    tab = s["table"].tolist()
    if c["op"] == "store":
        got = {}
        for part in ("k", "v"):
            value, held = _exact_quantised(s[part].double())
            got[part] = value
            got[part + "s"] = _exact_held(c, s[part + "_scale"].double(), held, n, q, tab)
        return got
    if c["op"] == "read":
        got = {}
        for part in ("k",) if c["shared"] else ("k", "v"):
            rows = []
            for b in range(c["B"]):
                rows.append(_exact_rows(c, s, part, tab[b], n[b])[n[b] - q[b]:])
            got[part] = torch.cat(rows)
        return got
    return _exact_attend(c, s, n, q, tab)


def _exact_axes(c, s, x, w):
    x = x.double()
    y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["D"] + 1e-6) * w.double()
    half = c["rot"] // 2
    lo = torch.arange(half, device=x.device)
    ia, ib = (c["off"] + 2 * lo, c["off"] + 2 * lo + 1) if c["style"] == "pairs" else (c["off"] + lo, c["off"] + half + lo)
    pos = torch.stack([s["pos"][int(a)] for a in s["axis"].tolist()], 1).double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos * s["freq"][None])
    z = torch.complex(y[..., ia], y[..., ib]) * turn[:, None]
    out = y.clone()
    out[..., ia], out[..., ib] = z.real, z.imag
    return out


def _exact_quantised(x):
    """What rows stand for once held, and their (scale, minimum)."""
    lo, hi = torch.min(x, -1)[0], torch.max(x, -1)[0]
    m, e = torch.frexp((hi - lo) / 15)
    s = torch.ldexp(torch.round(m * 256) / 256, e)                         # 8 significant bits, ties to even
    n = torch.zeros_like(x)
    some = s > 0
    n[some] = torch.floor((x[some] - lo[some][:, None]) / s[some][:, None] + 0.5).clamp(max=15)
    # a value halfway between two codes goes to the even one
    half = n - 0.5 == (x - lo[..., None]) / torch.where(some, s, 1.0)[..., None]
    n = torch.where(half & (n % 2 == 1), n - 1, n)
    return lo[..., None] + n * s[..., None], torch.stack((s, lo), -1)


def _exact_held(c, scale, held, n, q, tab):
    at = 0
    for b in range(c["B"]):
        for j in range((n[b] - q[b]) // c["bs"], (n[b] - 1) // c["bs"] + 1):
            lo, hi = max(n[b] - q[b], j * c["bs"]), min(n[b], (j + 1) * c["bs"])
            scale[tab[b][j], :, lo - j * c["bs"]:hi - j * c["bs"]] = held[at:at + hi - lo].transpose(0, 1)
            at += hi - lo
    return scale


def _exact_rows(c, s, part, tab, n):
    """A request's n tokens, [n, Hk, D] in fp64."""
    blk = torch.tensor(tab[:-(-n // c["bs"])], device="cuda")
    codes, scale = s[part + "_codes"][blk], s[part + "_scale"][blk].double()
    if c.get("bits") == 8:
        x = codes.view(FP8).double() * scale[:, :, None, None]
    else:
        low = codes % 16
        x = torch.empty((*codes.shape[:-1], c["D"]), dtype=torch.float64, device="cuda")
        x[..., 0::2], x[..., 1::2] = low.double(), ((codes - low) // 16).double()
        x = scale[..., 1:] + x * scale[..., :1]
    return x.transpose(1, 2).reshape(-1, c["Hk"], c["D"])[:n]


def _exact_attend(c, s, n, q, tab):
    Hk, D = c["Hk"], c["D"]
    G, at, out = c["H"] // Hk, 0, []
    for b in range(c["B"]):
        k, v = (_exact_rows(c, s, part, tab[b], n[b]).transpose(0, 1) for part in ("k", "v"))
        got = []
        for lo in range(0, q[b], 256):
            hi = min(q[b], lo + 256)
            y = s["q"][at + lo:at + hi].double().view(hi - lo, Hk, G, D).permute(1, 2, 0, 3)
            a = torch.einsum("hgid,htd->hgit", y, k) / math.sqrt(D)
            own_pos = torch.arange(n[b] - q[b] + lo, n[b] - q[b] + hi, device="cuda")[:, None]
            t = torch.arange(n[b], device="cuda")[None]
            hide = (t > own_pos) | ((own_pos - t >= c["window"]) if c["window"] else False)
            a = torch.softmax(a.masked_fill(hide, float("-inf")), -1)
            got.append(torch.einsum("hgit,htd->ihgd", a, v).reshape(hi - lo, c["H"], D))
        out.append(torch.cat(got))
        at += q[b]
    return torch.cat(out)
