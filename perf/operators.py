"""The paged 8-bit KV cache's operators: the cases that are measured, their plain form and their definition in 64 bits.

Four operators, as one serving step uses them:
  resize     block tables, positions and slots on the GPU from request lengths (grow for drafted tokens, then roll back);
  norm_rope  RMS norm of every query and key head and the position rotation in one pass;
  append     new key / value rows into e4m3 codes with one power-of-two scale per (block of tokens, head);
  attend     attention of 1..n query tokens per request over the codes (grouped heads, or latent rows with K = V).
"""
import math
import random

import torch

own = False

FP8 = torch.float8_e4m3fn
E_MIN, E_MAX = -64, 64          # exponents a block's scale may take


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a small server's drafted tokens: 16 requests grow by up to 5 tokens and are rolled back
        dict(name="resize_drafts_b16", op="resize", B=16, ctx=8192, q=5, bs=64, ragged=True),
        # a large server admits prompts: 1,024 requests, up to 127 new tokens each
        dict(name="resize_prompts_b1024", op="resize", B=1024, ctx=4096, q=127, bs=16, ragged=True),
        # one decode step of the latent-row model: 32 requests, 64 query heads + the latent row, tail of 64 rotated
        dict(name="norm_decode_latent", op="norm", T=32, H=64, Hk=1, D=512, rot=64, off=448, style="pairs", far=262144),
        # a prompt chunk of a grouped-head model, whole heads rotated, an odd number of tokens
        dict(name="norm_prompt_gqa", op="norm", T=6143, H=32, Hk=8, D=128, rot=128, off=0, style="halves", far=32768),
        # one new latent row for each of 32 requests, in the middle of their blocks
        dict(name="append_decode_latent", op="append", B=32, q=1, ctx=32768, ragged=True, Hk=1, D=512, bs=64, shared=True),
        # prompts of up to 2,500 tokens written at once
        dict(name="append_prompt_gqa", op="append", B=6, q=2500, ctx=4096, ragged=True, Hk=8, D=128, bs=32, shared=False),
        # one token over a resident 8K context of ratio-4 chunks and the window: the smallest call
        dict(name="attend_latent_8k_b1", op="attend", B=1, q=1, ctx=2176, ragged=False, H=64, Hk=1, D=512, bs=64, shared=True, window=0),
        # the batch-32 sweep's 128K contexts as latent rows
        dict(name="attend_latent_128k_b32", op="attend", B=32, q=1, ctx=32768, ragged=False, H=64, Hk=1, D=512, bs=64, shared=True, window=0),
        # a decode batch of a grouped-head model, ragged contexts, small blocks
        dict(name="attend_gqa_decode_b64", op="attend", B=64, q=1, ctx=16384, ragged=True, H=32, Hk=8, D=128, bs=16, shared=False, window=0),
        # verification of drafted tokens: up to 5 query tokens per request
        dict(name="attend_gqa_drafts_b16", op="attend", B=16, q=5, ctx=8192, ragged=True, H=64, Hk=8, D=128, bs=32, shared=False, window=0),
        # prompt chunks of up to 1,024 tokens against their contexts: the compute-bound end
        dict(name="attend_chunk_gqa", op="attend", B=4, q=1024, ctx=8192, ragged=True, H=32, Hk=8, D=128, bs=64, shared=False, window=0),
        # wide heads with a sliding window over long contexts
        dict(name="attend_window_d256", op="attend", B=24, q=1, ctx=32768, ragged=True, H=16, Hk=4, D=256, bs=128, shared=False, window=4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["resize", "norm", "append", "attend", "attend", "attend"])
    bs = rng.choice([16, 32, 64, 128])
    if op == "resize":
        B = _log(rng, 1, 1024)
        return dict(op=op, B=B, ctx=_log(rng, 64, 8192), q=_log(rng, 1, max(1, min(1024, 65536 // B))), bs=bs, ragged=True)
    if op == "norm":
        D = rng.choice([64, 96, 128, 256, 512])
        H = rng.choice([4, 12, 16, 24, 32, 64])
        Hk = rng.choice([1, 2, 4, 8])
        rot = rng.choice([r for r in (32, 64, D) if r <= D])
        return dict(op=op, T=_log(rng, 1, max(1, min(8000, 31000000 // ((H + Hk) * D)))), H=H, Hk=Hk, D=D, rot=rot,
                    off=rng.choice([0, D - rot]), style=rng.choice(["pairs", "halves"]), far=_log(rng, 1024, 1048576))
    shared = rng.random() < 0.4
    D = rng.choice([128, 256, 512]) if shared else rng.choice([128, 128, 256])
    Hk = rng.choice([1, 1, 2]) if shared else rng.choice([1, 2, 4, 8])
    if op == "append":
        B = _log(rng, 1, 64)
        q = _log(rng, 1, max(1, min(2500, 14000000 // (B * Hk * D))))
        return dict(op=op, B=B, q=q, ctx=q + _log(rng, 16, 4096), ragged=True, Hk=Hk, D=D, bs=bs, shared=shared)
    G = rng.choice([1, 3, 4, 6, 8, 16]) if not shared else rng.choice([8, 16, 32, 64])
    kind = rng.random()
    q = 1 if kind < 0.5 else _log(rng, 2, 8) if kind < 0.75 else _log(rng, 9, 600)
    # the products of the largest listed case, and its bytes, at most: B * H * q * ctx scores of D products
    B = _log(rng, 1, max(1, min(48, 200000 // (q * Hk * G))))
    most = max(64, min(32768, 500000000 // (B * Hk * D * (1 if shared else 2)), int(2e11) // (4 * D * B * q * Hk * G)))
    ctx = max(q, _log(rng, 16, most))
    return dict(op=op, B=B, q=q, ctx=ctx, ragged=rng.random() < 0.8, H=Hk * G, Hk=Hk, D=D, bs=bs, shared=shared,
                window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]))


def _lengths(c):
    """(lengths after the step, new tokens) of each request: by the case alone, so that its work is known."""
    r = random.Random(c["B"] * 7919 + c["ctx"] * 31 + c["q"])
    q = [r.randint(max(1, c["q"] // 4), c["q"]) if c["ragged"] else c["q"] for _ in range(c["B"])]
    q[0] = c["q"]
    n = [max(qi, r.randint(max(1, c["ctx"] // 8), c["ctx"])) if c["ragged"] else c["ctx"] for qi in q]
    n[0] = max(c["ctx"], q[0])
    return n, q


# ---------------------------------------------------------------------------------------------- inputs
def _codes(g, n_blocks, Hk, bs, D, spread):
    """A filled cache: rows of normal values, block scales that differ by a few powers of two."""
    codes = torch.empty((n_blocks, Hk, bs, D), dtype=torch.uint8, device="cuda")
    scale = torch.empty((n_blocks, Hk), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (Hk * bs * D))
    for i in range(0, n_blocks, step):
        m = min(step, n_blocks - i)
        x = torch.randn((m, Hk, bs, D), generator=g, device="cuda")
        x *= torch.exp2(torch.randint(-spread, spread + 1, (m, Hk, 1, 1), generator=g, device="cuda").float())
        e = _exponent(x.abs().amax((2, 3)))
        scale[i:i + m] = _power(e)
        codes[i:i + m] = (x / scale[i:i + m, :, None, None]).to(FP8).view(torch.uint8)
    return codes, scale


def _power(e):
    """2^e in fp32, exactly, from its bits (e in -126..127)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, held to the range a scale may take."""
    m, e = torch.frexp(amax / 448)
    e = e - (m == 0.5).int()
    return torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX).int()


def _cache(c, s, g, n):
    """Block table (scattered blocks), codes and scales for lengths n, with some blocks over."""
    bs, B = c["bs"], c["B"]
    need = [-(-x // bs) for x in n]
    width = max(need) + 2
    total = sum(need) + B + 3
    order = torch.randperm(total, generator=g, device="cuda").int()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(width, device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
    table[at] = order[:sum(need)]
    s.update(table=table, n_blocks=total, width=width, rest=order[sum(need):].contiguous())


def _handle(c, s):
    from sparse_retrieval_host_gb300.paged import PagedKV8
    if c["op"] == "norm":       # any cache will do: the heads' shapes are the call's own
        return PagedKV8(batch=1, n_kv_heads=1, head_dim=128, block_tokens=64, n_blocks=1, max_blocks=1)
    return PagedKV8(batch=c["B"], n_kv_heads=c.get("Hk", 1), head_dim=c.get("D", 128), block_tokens=c["bs"],
                    n_blocks=s["n_blocks"], max_blocks=s["width"], shared_kv=c.get("shared", True),
                    buffers={k: s[k] for k in ("k_codes", "k_scale", "v_codes", "v_scale", "table", "len", "free", "n_free") if k in s})


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    s = dict(case=c)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    bf = lambda *shape: torch.randn(shape, generator=g, device="cuda").bfloat16()  # noqa: E731
    if c["op"] == "norm":
        T, H, Hk, D = c["T"], c["H"], c["Hk"], c["D"]
        qkv = bf(T, (H + 2 * Hk) * D)                       # one projection's rows: queries, keys, values side by side
        s["q"] = qkv[:, :H * D].view(T, H, D)
        s["k"] = qkv[:, H * D:(H + Hk) * D].view(T, Hk, D)
        s["wq"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
        s["wk"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
        s["pos"] = torch.randint(0, c["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        s["freq"] = 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
        s["oq"] = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
        s["ok"] = torch.empty((T, Hk, D), dtype=torch.bfloat16, device="cuda")
    else:
        n, q = _lengths(c)
        old = [a - b for a, b in zip(n, q)]
        _cache(c, s, g, old if c["op"] == "resize" else n)
        s["T"] = sum(q)
        s["max_q"], s["max_len"] = max(q), max(n)
        s["cu"] = i32([sum(q[:i]) for i in range(len(q) + 1)])
        if c["op"] == "resize":
            extra = sum(-(-a // c["bs"]) - -(-b // c["bs"]) for a, b in zip(n, old))
            more = s["n_blocks"] + torch.randperm(extra, generator=g, device="cuda").int()
            rest = torch.cat([s["rest"], more])
            s["n_blocks"] += extra
            width = max(-(-a // c["bs"]) for a in n)
            if width > s["width"]:
                s["table"] = torch.nn.functional.pad(s["table"], (0, width - s["width"]), value=-1)
                s["width"] = width
            s["free"] = torch.full((s["n_blocks"],), -1, dtype=torch.int32, device="cuda")
            s["free"][:rest.numel()] = rest
            s["n_free"] = i32([rest.numel()])
            s["len"], s["back"], s["new"] = i32(old), i32(old), i32(n)
        else:
            s["len"] = i32(n)
            s["k_codes"], s["k_scale"] = _codes(g, s["n_blocks"], c["Hk"], c["bs"], c["D"], 2)
            s["v_codes"], s["v_scale"] = (s["k_codes"], s["k_scale"]) if c["shared"] else \
                _codes(g, s["n_blocks"], c["Hk"], c["bs"], c["D"], 2)
            if c["op"] == "append":
                s["k"] = bf(s["T"], c["Hk"], c["D"])
                s["v"] = s["k"] if c["shared"] else bf(s["T"], c["Hk"], c["D"])
            else:
                s["q"] = bf(s["T"], c["H"], c["D"])
                s["out"] = torch.empty_like(s["q"])
    s["handle"] = _handle(c, s) if own else None
    return s


# ---------------------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s["case"], s, s["handle"])
    return _PLAIN[op](s["case"], s)


def _own_resize(c, s, h):
    cu, pos, slot = h.resize(s["new"], s["T"])
    h.resize(s["back"], 0)
    return dict(cu=cu, pos=pos, slot=slot, table=s["table"], len=s["len"], n_free=s["n_free"])


def _own_norm(c, s, h):
    q, k = h.norm_rope(s["q"], s["k"], pos=s["pos"], inv_freq=s["freq"], rot_dim=c["rot"], rot_off=c["off"], style=c["style"],
                       q_weight=s["wq"], k_weight=s["wk"], eps=1e-6, q_out=s["oq"], k_out=s["ok"])
    return dict(q=q, k=k)


def _own_append(c, s, h):
    h.append(s["k"], None if c["shared"] else s["v"], s["cu"])
    return _held(c, s)


def _own_attend(c, s, h):
    return h.attend(s["q"], s["cu"], scale=c["D"] ** -0.5, window=c["window"], out=s["out"])


def _held(c, s):
    got = dict(k=s["k_codes"].view(FP8), ks=s["k_scale"])
    if not c["shared"]:
        got.update(v=s["v_codes"].view(FP8), vs=s["v_scale"])
    return got


def _before(x):
    """Sums of what stands before each entry, and the whole sum last."""
    return torch.nn.functional.pad(torch.cumsum(x, 0), (1, 0))


def _resize(s, new, T):
    """Tables, lengths and the free stack to the lengths `new`; the new tokens' places."""
    bs, table, ln, free, n_free = s["case"]["bs"], s["table"], s["len"], s["free"], s["n_free"]
    have, need = (ln.long() + bs - 1) // bs, (new.long() + bs - 1) // bs
    j = torch.arange(table.shape[1], device=table.device)[None]
    gone = (j >= need[:, None]) & (j < have[:, None])
    come = (j >= have[:, None]) & (j < need[:, None])
    # released blocks: the first one in (request, block) order ends on top of the stack
    rank = torch.cumsum(gone.reshape(-1), 0).reshape(gone.shape) - 1
    top = n_free.long() + gone.sum()
    spare = free.numel()
    stack = torch.nn.functional.pad(free, (0, 1))
    stack.scatter_(0, torch.where(gone, top - 1 - rank, spare).reshape(-1), table.reshape(-1))
    rank = torch.cumsum(come.reshape(-1), 0).reshape(come.shape) - 1
    taken = stack[torch.where(come, top - 1 - rank, spare)]
    table.copy_(torch.where(come, taken, torch.where(gone, -1, table)))
    free.copy_(stack[:-1])
    n_free.copy_(top - come.sum())
    cu = _before((new.long() - ln).clamp(min=0)).int()
    i = torch.arange(T, device=table.device, dtype=torch.int32)
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    pos = (ln[b] + i - cu[b]).int()
    slot = table[b, pos.long() // bs].long() * bs + pos % bs
    ln.copy_(new)
    return cu, pos, slot


def _plain_resize(c, s):
    cu, pos, slot = _resize(s, s["new"], s["T"])
    _resize(s, s["back"], 0)
    return dict(cu=cu, pos=pos, slot=slot, table=s["table"], len=s["len"], n_free=s["n_free"])


def _norm_rope(c, s, x, w):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    angle = s["pos"].double()[:, None] * s["freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    r = x[..., c["off"]:c["off"] + c["rot"]]
    if c["style"] == "pairs":
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = r[..., :c["rot"] // 2], r[..., c["rot"] // 2:]
        r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((x[..., :c["off"]], r, x[..., c["off"] + c["rot"]:]), -1).bfloat16()


def _plain_norm(c, s):
    return dict(q=_norm_rope(c, s, s["q"], s["wq"]), k=_norm_rope(c, s, s["k"], s["wk"]))


def _append(c, s, x, codes, scale):
    bs, n_blocks, Hk, D = c["bs"], codes.shape[0], c["Hk"], c["D"]
    i = torch.arange(s["T"], device=x.device, dtype=torch.int32)
    cu, ln = s["cu"], s["len"]
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    first = ln - (cu[1:] - cu[:-1])                            # each request's first new position
    pos = (first[b] + i - cu[b]).long()
    block = s["table"][b, pos // bs].long()
    x = x.float()
    # a block begun before this call keeps at least its old scale; a fresh one starts from the smallest
    fresh = torch.ones(n_blocks, dtype=torch.bool, device=x.device)
    begun = s["table"].gather(1, (first.long() // bs)[:, None])[:, 0].long()
    some = (first % bs != 0) & (cu[1:] > cu[:-1])
    fresh[begun.clamp(min=0)] = ~some
    amax = torch.zeros((n_blocks, Hk), device=x.device)
    amax.scatter_reduce_(0, block[:, None].expand(-1, Hk), x.abs().amax(-1), "amax")
    want = _power(_exponent(amax))
    new = torch.where(fresh[:, None], want, torch.maximum(want, scale))
    at = begun[:, None, None, None].clamp(min=0)               # codes of the begun blocks to the new scale
    hs, ts = torch.arange(Hk, device=x.device)[None, :, None, None], torch.arange(bs, device=x.device)[None, None, :, None]
    held = codes[begun.clamp(min=0)]
    again = held.view(FP8).float() * (scale / new)[begun.clamp(min=0)][:, :, None, None]
    keep = some[:, None, None, None] & (ts < (first % bs)[:, None, None, None])
    codes[at, hs, ts, torch.arange(D, device=x.device)] = torch.where(keep, again.to(FP8).view(torch.uint8), held)
    y = (x / new[block][:, :, None]).clamp(-448, 448).to(FP8).view(torch.uint8)
    codes[block[:, None], torch.arange(Hk, device=x.device)[None], (pos % bs)[:, None]] = y
    touched = torch.zeros(n_blocks, dtype=torch.bool, device=x.device)
    touched[block] = True
    scale.copy_(torch.where(touched[:, None], new, scale))


def _plain_append(c, s):
    _append(c, s, s["k"], s["k_codes"], s["k_scale"])
    if not c["shared"]:
        _append(c, s, s["v"], s["v_codes"], s["v_scale"])
    return _held(c, s)


def _rows(c, s, codes, scale):
    """The cache's values of every request, [B, Hk, tokens, D] in fp32."""
    nb = -(-s["max_len"] // c["bs"])
    tab = s["table"][:, :nb].long().clamp(min=0)
    x = codes[tab].view(FP8).float() * scale[tab][..., None, None]
    return x.transpose(1, 2).reshape(c["B"], c["Hk"], nb * c["bs"], c["D"])


def _plain_attend(c, s):
    B, Hk, D, m = c["B"], c["Hk"], c["D"], s["max_q"]
    G = c["H"] // Hk
    k = _rows(c, s, s["k_codes"], s["k_scale"])
    v = k if c["shared"] else _rows(c, s, s["v_codes"], s["v_scale"])
    cu, ln = s["cu"].long(), s["len"].long()
    nq = cu[1:] - cu[:-1]
    i = torch.arange(m, device=k.device)
    q = s["q"][(cu[:-1, None] + i).clamp(max=s["T"] - 1)].float()          # [B, m, H, D]
    q = q.view(B, m, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, m * G, D)
    p = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).view(B, Hk, m, G, -1)
    t = torch.arange(k.shape[2], device=k.device)
    at = (ln - nq)[:, None] + i                                            # each query's own position
    see = (t <= at[..., None]) & (t < ln[:, None, None])
    if c["window"]:
        see &= t > at[..., None] - c["window"]
    p.masked_fill_(~see[:, None, :, None], float("-inf"))
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = torch.where((t < ln[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(p.view(B, Hk, m * G, -1), v).view(B, Hk, m, G, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B, m, c["H"], D)
    row = torch.arange(s["T"], device=k.device)
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    return o[b, row - cu[b]].bfloat16()


_PLAIN = dict(resize=_plain_resize, norm=_plain_norm, append=_plain_append, attend=_plain_attend)
_OWN = dict(resize=_own_resize, norm=_own_norm, append=_own_append, attend=_own_attend)


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
    if c["op"] == "norm":
        values = c["T"] * (c["H"] + c["Hk"]) * c["D"]
        return dict(bytes=values * 4 + c["T"] * 4 + c["D"] * 8 + c["rot"] * 4, flops=values * 6)
    n, q = _lengths(c)
    T, B, bs = sum(q), c["B"], c["bs"]
    if c["op"] == "resize":
        blocks = sum(-(-a // bs) - -(-(a - m) // bs) for a, m in zip(n, q))
        return dict(bytes=T * 12 + B * 4 * 7 + blocks * 4 * 6, flops=T * 4 + B * 8)
    copies = 1 if c["shared"] else 2
    if c["op"] == "append":
        blocks = sum(-(-a // bs) - (a - m) // bs for a, m in zip(n, q))
        return dict(bytes=copies * (T * c["Hk"] * c["D"] * 3 + blocks * c["Hk"] * 4) + B * 8 + blocks * 4,
                    flops=copies * T * c["Hk"] * c["D"] * 3)
    tokens, pairs = _visible(c, n, q)
    blocks = sum(-(-min(a, (c["window"] or a) + m - 1) // bs) for a, m in zip(n, q))
    return dict(bytes=copies * (tokens * c["Hk"] * c["D"] + blocks * c["Hk"] * 4) + T * c["H"] * c["D"] * 4 + B * 8 + blocks * 4,
                flops=4 * c["D"] * c["H"] * pairs)


# ---------------------------------------------------------------------------------------------- the definition in 64 bits
def _e4m3(v):
    """Nearest e4m3 value (ties to even) of 64-bit values within +-448."""
    m, e = torch.frexp(v)
    step = _power((e - 1).clamp(min=-6) - 3).double()
    return torch.round(v / step) * step


def exact(case, seed):
    c = dict(case)
    global own
    was, own = own, False
    s = prepare(c, seed)
    own = was
    if c["op"] == "resize":
        return _exact_resize(c, s)
    if c["op"] == "norm":
        return dict(q=_exact_norm(c, s, s["q"], s["wq"]), k=_exact_norm(c, s, s["k"], s["wk"]))
    n, q = _lengths(c)
    tab = s["table"].tolist()
    if c["op"] == "append":
        if c["B"] * max(q) > 40000:
            return None
        got = {}
        for name, part in (("k", "k"),) if c["shared"] else (("k", "k"), ("v", "v")):
            got[name], got[name + "s"] = _exact_append(c, s, s[part].double(), s[part + "_codes"], s[part + "_scale"], n, q, tab)
        return got
    return _exact_attend(c, s, n, q, tab)


def _exact_resize(c, s):
    bs, tab, ln = c["bs"], s["table"].tolist(), s["len"].tolist()
    free = s["free"].tolist()[:int(s["n_free"])]
    cu, pos, slot = [0], [], []
    for b, new in enumerate(s["new"].tolist()):
        for j in range(-(-ln[b] // bs), -(-new // bs)):
            tab[b][j] = free.pop()
        for p in range(ln[b], new):
            pos.append(p)
            slot.append(tab[b][p // bs] * bs + p % bs)
        cu.append(len(pos))
    t = lambda v, d: torch.tensor(v, dtype=d)  # noqa: E731
    # the roll-back gives every block back: tables, lengths and the count are as they were
    return dict(cu=t(cu, torch.int32), pos=t(pos, torch.int32), slot=t(slot, torch.int64), table=s["table"], len=s["len"],
                n_free=s["n_free"])


def _exact_norm(c, s, x, w):
    x = x.double()
    y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["D"] + 1e-6) * w.double()
    half = c["rot"] // 2
    lo = torch.arange(half, device=x.device)
    ia, ib = (c["off"] + 2 * lo, c["off"] + 2 * lo + 1) if c["style"] == "pairs" else (c["off"] + lo, c["off"] + half + lo)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), s["pos"].double()[:, None] * s["freq"][None])
    z = torch.complex(y[..., ia], y[..., ib]) * turn[:, None]
    out = y.clone()
    out[..., ia], out[..., ib] = z.real, z.imag
    return out


def _exact_append(c, s, x, codes, scale, n, q, tab):
    bs = c["bs"]
    value = codes.view(FP8).double().clone()
    scale = scale.double().clone()
    at = 0
    for b in range(c["B"]):
        first = n[b] - q[b]
        for j in range(first // bs, (n[b] - 1) // bs + 1):
            lo, hi = max(first, j * bs), min(n[b], (j + 1) * bs)
            rows = x[at:at + hi - lo].transpose(0, 1)            # [Hk, rows, D]
            at += hi - lo
            blk, o = tab[b][j], lo - j * bs
            amax = rows.abs().amax((1, 2))
            m, e = torch.frexp(amax / 448)
            e = torch.where(m > 0.5, e, e - 1).clamp(E_MIN, E_MAX)
            want = torch.where(amax > 0, _power(e).double(), 2.0 ** E_MIN)
            if o:
                want = torch.maximum(want, scale[blk])
                value[blk, :, :o] = _e4m3(value[blk, :, :o] * (scale[blk] / want)[:, None, None])
            scale[blk] = want
            value[blk, :, o:o + hi - lo] = _e4m3((rows / want[:, None, None]).clamp(-448, 448))
    return value, scale


def _exact_attend(c, s, n, q, tab):
    bs, Hk, D = c["bs"], c["Hk"], c["D"]
    G, at, out = c["H"] // Hk, 0, []
    for b in range(c["B"]):
        blk = torch.tensor(tab[b][:-(-n[b] // bs)], device="cuda")
        rows = []
        for part in ("k",) if c["shared"] else ("k", "v"):
            x = s[part + "_codes"][blk].view(FP8).double() * s[part + "_scale"][blk].double()[:, :, None, None]
            rows.append(x.permute(1, 0, 2, 3).reshape(Hk, -1, D)[:, :n[b]])
        k, v = rows[0], rows[-1]
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
