"""The paged cache in 4 bits (kv4_*), rows read back (kv4_read, kv8_read) and the rotation by several axes against plain
64-bit implementations, and a serving loop of them together."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def _abi():
    from sparse_retrieval_host_gb300 import abi
    return abi


def _kv4(**kw):
    from sparse_retrieval_host_gb300.paged import PagedKV4
    return PagedKV4(**kw)


def _kv8(**kw):
    from sparse_retrieval_host_gb300.paged import PagedKV8
    return PagedKV8(**kw)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def _cu(counts):
    return _i32([0] + list(np.cumsum(counts)))


# ---------------------------------------------------------------------------------------------- the form of a row
def _quantise(x):
    """numpy float32 rows [..., D] of bf16 values -> codes, s, m by the documented steps."""
    x = np.where(np.isfinite(x), x, np.float32(0)).astype(np.float32)
    x = np.clip(x, -np.float32(2.0 ** 120), np.float32(2.0 ** 120))
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    s = torch.from_numpy(((hi - lo) / np.float32(15)).astype(np.float32)).bfloat16().float().numpy()
    with np.errstate(divide="ignore", invalid="ignore"):
        n = np.rint((x - lo) / s)
    n = np.where(s > 0, np.clip(n, 0, 15), 0).astype(np.uint8)
    return n, s[..., 0], lo[..., 0]


def _codes(c, part, layer=0):
    """Codes [n_blocks][heads][tokens][D] and (s, m) as fp64, of a 4-bit cache."""
    b = (c.k_codes if part == "k" else c.v_codes)[layer]
    sm = (c.k_scale if part == "k" else c.v_scale)[layer]
    return torch.stack((b & 15, b >> 4), -1).flatten(-2), sm


def _values(c, part, b, n, layer=0):
    """Request b's first n tokens, fp64 [n][heads][D]."""
    codes, sm = _codes(c, part, layer)
    blk = c.table[b, :-(-n // c.bs)].long()
    v = codes[blk].double() * sm[blk][..., :1].double() + sm[blk][..., 1:].double()
    return v.transpose(1, 2).reshape(-1, c.Hk, c.D)[:n]


def _filled(c, g, lens, spread=2, mean=0.3, layer=0):
    """Fills a cache's tables and pools for lengths `lens` with quantised rows, by the test's own hand."""
    bs = c.bs
    need = [-(-n // bs) for n in lens]
    ids = torch.randperm(c.n_blocks, generator=g, device="cuda")[:sum(need)].int()
    at = 0
    c.table.fill_(-1)
    for b, k in enumerate(need):
        c.table[b, :k] = ids[at:at + k]
        at += k
    c.len[:len(lens)] = _i32(lens)
    for codes, scale in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)):
        codes[layer].copy_(torch.randint(0, 256, codes[layer].shape, generator=g, device="cuda", dtype=torch.uint8))
        sh = scale[layer].shape[:-1]
        s = 0.3 * torch.exp2(torch.randint(-spread, spread + 1, sh, generator=g, device="cuda").float())
        m = -7.5 * s * (1 + 0.2 * torch.randn(sh, generator=g, device="cuda")) + mean
        scale[layer].copy_(torch.stack((s, m), -1).bfloat16())


# ---------------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("bs,Hk,D,news", [(16, 1, 128, [1]), (16, 8, 128, [1, 5, 0, 33]), (32, 2, 256, [70, 1, 16]),
                                          (64, 3, 128, [129, 64, 2]), (128, 1, 256, [1] * 40), (16, 4, 128, [1, 0] * 600)])
def test_append_is_exact(bs, Hk, D, news):
    g = _gen(bs * Hk + len(news))
    rng = np.random.default_rng(bs + D)
    B = len(news)
    olds = [int(v) for v in rng.integers(0, 3 * bs, B)]
    lens = [a + b for a, b in zip(olds, news)]
    most = max(-(-n // bs) for n in lens) + 1
    c = _kv4(batch=B, n_kv_heads=Hk, head_dim=D, block_tokens=bs, n_blocks=sum(-(-n // bs) for n in lens) + 5, max_blocks=most)
    _filled(c, g, lens)
    T = sum(news)
    big = _bf16(g, T + 2, 3 * Hk * D) * torch.exp2(torch.randint(-20, 20, (T + 2, 1), generator=g, device="cuda").float()).bfloat16()
    k, v = big[:T, :Hk * D].view(T, Hk, D), big[:T, 2 * Hk * D:].view(T, Hk, D)      # strided rows
    cu = _cu(news)
    before = {p: [t.clone() for t in _codes(c, p)] for p in "kv"}
    c.append(k, v, cu)
    assert c.check_error() == 0
    table = c.table.tolist()
    for part, x in (("k", k), ("v", v)):
        want_n, want_s = before[part][0].cpu().numpy(), before[part][1].float().cpu().numpy()
        n, s, m = _quantise(x.float().cpu().numpy())
        at = 0
        for b in range(B):
            for i in range(news[b]):
                p = olds[b] + i
                blk = table[b][p // bs]
                want_n[blk, :, p % bs] = n[at]
                want_s[blk, :, p % bs, 0], want_s[blk, :, p % bs, 1] = s[at], m[at]
                at += 1
        got_n, got_s = _codes(c, part)
        assert np.array_equal(got_s.float().cpu().numpy(), want_s)
        # (x - m) / s in fp32 on both sides
        assert np.array_equal(got_n.cpu().numpy(), want_n)
    c.close()


def test_append_odd_values():
    abi = _abi()
    c = _kv4(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=2, max_blocks=2)
    cu, _, _ = c.resize(_i32([8]), 8)
    k = torch.zeros(8, 1, 128, device="cuda")
    k[0] = 3.25                                    # all equal: s = 0
    k[1, 0, 5] = float("inf")
    k[2, 0, 6] = float("nan")
    k[2, 0, 7] = 2.0
    k[3, 0, :] = torch.linspace(-1, 1, 128)
    k[4, 0, 0], k[4, 0, 1] = 3e38, -3e38
    k[5, 0, 0] = 2.0 ** -130                       # differences that bf16 holds as subnormals only
    k[6, 0, 0] = 2.0 ** -133 * 3
    k[7, 0, 0] = -0.0
    k = k.bfloat16()
    c.append(k, k, cu)
    assert c.check_error() == abi.SRH_ERR_RANGE and c.check_error() == 0
    n, s, m = _quantise(k.float().cpu().numpy())
    codes, sm = _codes(c, "k")
    blk = int(c.table[0, 0])
    assert np.array_equal(codes[blk, :, :8].transpose(0, 1).cpu().numpy(), n)
    assert np.array_equal(sm[blk, :, :8, 0].t().float().cpu().numpy(), s)
    assert np.array_equal(sm[blk, :, :8, 1].t().float().cpu().numpy(), m)
    out, _ = c.read(_i32([0]), cu, 8)
    assert bool(torch.isfinite(out).all()) and float(out[0].min()) == float(out[0].max()) == 3.25
    c.close()


@pytest.mark.parametrize("why", ["down", "rows", "short", "long", "negative", "entry"])
def test_append_leaves_out_what_is_out_of_bounds(why):
    abi = _abi()
    g = _gen(11)
    c = _kv4(batch=3, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=12, max_blocks=4)
    _filled(c, g, [20, 40, 30])
    cu, rows = [0, 4, 9, 12], 12
    touched = {0, 1, 2}
    if why == "down":
        cu, touched = [0, 9, 4, 12], set()
    if why == "rows":
        cu, touched = [0, 4, 9, 13], {0, 1}
    if why == "short":
        c.len[1] = 4
        touched = {0, 2}
    if why == "long":
        c.len[1] = 65
        touched = {0, 2}
    if why == "negative":
        c.len[1] = -1
        touched = {0, 2}
    if why == "entry":
        c.table[1, 2] = 12
        touched = {0, 1, 2}
    k = _bf16(g, rows, 2, 128)
    before = [t.clone() for t in (*_codes(c, "k"), *_codes(c, "v"))]
    c.append(k, k, _i32(cu))
    assert c.check_error() == abi.SRH_ERR_BOUNDS
    after = (*_codes(c, "k"), *_codes(c, "v"))
    n, s, m = _quantise(k.float().cpu().numpy())
    lens, table = c.len.tolist(), c.table.tolist()
    want = [t.clone() for t in before]
    for b in sorted(touched):
        nq = cu[b + 1] - cu[b]
        for i in range(nq):
            p = lens[b] - nq + i
            blk = table[b][p // 16]
            if not 0 <= blk < 12:
                continue
            for j in (0, 2):
                want[j][blk, :, p % 16] = torch.from_numpy(n[cu[b] + i]).cuda()
                want[j + 1][blk, :, p % 16] = torch.from_numpy(np.stack((s[cu[b] + i], m[cu[b] + i]), -1)).cuda().bfloat16()
    for x, y in zip(after, want):
        assert torch.equal(x, y)
    c.close()


# ---------------------------------------------------------------------------------------------- read
@pytest.mark.parametrize("bits,bs,Hk,D,shared", [(4, 16, 8, 128, False), (4, 128, 1, 256, False), (4, 32, 3, 128, False),
                                                 (8, 16, 2, 128, False), (8, 64, 1, 512, True), (8, 32, 4, 256, False),
                                                 (8, 16, 1, 512, False), (8, 128, 2, 128, True)])
def test_read_is_exact(bits, bs, Hk, D, shared):
    g = _gen(bits * bs + D)
    lens, starts, counts = [70, 1, 0, 300, 33], [3, 0, 0, 0, 32], [64, 1, 0, 300, 1]
    kw = dict(batch=6, n_kv_heads=Hk, head_dim=D, block_tokens=bs, n_blocks=60, max_blocks=30)
    if bits == 4:
        c = _kv4(**kw)
        _filled(c, g, lens)
    else:
        c = _kv8(shared_kv=shared, **kw)
        c.resize(_i32(lens))
        for codes, scale in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)):
            x = (100 * torch.randn(codes[0].shape, generator=g, device="cuda")).clamp(-448, 448)
            codes[0].copy_(x.to(FP8).view(torch.uint8))
            scale[0].copy_(0.1 + torch.rand(scale[0].shape, generator=g, device="cuda"))
    T = sum(counts)
    outs = torch.full((T + 3, 2, Hk, D + 0), 7.0, device="cuda", dtype=torch.bfloat16)    # K and V rows side by side
    k_out, v_out = outs[:, 0], outs[:, 1]
    got = c.read(_i32(starts), _cu(counts), T + 3, k_out=k_out, v_out=None if shared else v_out)
    assert c.check_error() == 0 and got[0] is k_out
    for part, out in (("k", k_out),) if shared else (("k", k_out), ("v", v_out)):
        at = 0
        for b, n in enumerate(counts):
            if bits == 4:
                want = _values(c, part, b, lens[b])[starts[b]:starts[b] + n].float().bfloat16()
            else:
                codes, scale = (c.k_codes[0], c.k_scale[0]) if part == "k" else (c.v_codes[0], c.v_scale[0])
                blk = c.table[b, :-(-lens[b] // bs)].long()
                x = codes[blk].view(FP8).float() * scale[blk][..., None, None]
                want = x.transpose(1, 2).reshape(-1, Hk, D)[starts[b]:starts[b] + n].bfloat16()
            assert torch.equal(out[at:at + n], want), (part, b)
            at += n
        assert bool((out[T:] == 7).all())
    if shared:
        assert bool((v_out == 7).all()) and got[1] is None
    else:
        k2, v2 = c.read(_i32(starts), _cu(counts), T)
        assert torch.equal(k2, k_out[:T]) and torch.equal(v2, v_out[:T])
    c.close()


@pytest.mark.parametrize("why", ["down", "behind", "before", "rows", "long", "entry"])
def test_read_leaves_out_what_is_out_of_bounds(why):
    abi = _abi()
    g = _gen(5)
    c = _kv4(batch=2, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=12, max_blocks=4)
    _filled(c, g, [20, 40])
    start, cu, left = [0, 10], [0, 8, 20], set()
    if why == "down":
        cu, left = [8, 0, 20], set(range(20))
    if why == "behind":
        start, left = [14, 10], {6, 7}
    if why == "before":
        start, left = [0, -3], {8, 9, 10}
    if why == "rows":
        cu = [0, 8, 25]
    if why == "long":
        c.len[1] = 65
        left = set(range(8, 20))
    if why == "entry":
        c.table[1, 1] = -1
        left = set(range(14, 20))
    full = _values(c, "k", 0, 20), _values(c, "k", 1, 40)
    k, v = (torch.full((20, 2, 128), 7.0, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    c.read(_i32(start), _i32(cu), 20, k_out=k, v_out=v)
    assert c.check_error() == abi.SRH_ERR_BOUNDS
    for r in range(20):
        b = int(r >= cu[1])
        if r in left:
            assert bool((k[r] == 7).all()) and bool((v[r] == 7).all()), r
        else:
            assert torch.equal(k[r], full[b][start[b] + r - cu[b]].float().bfloat16()), r
    c.close()


# ---------------------------------------------------------------------------------------------- attend
def _attend_64(c, q, cu, scale, window=0, layer=0):
    """(outputs, tolerance) in fp64. A row that sees nothing gives zeros.

    The tolerance: bf16's rounding of the output, 2^-8 of it; the fp16 rounding of a weight times V's scale, at most 2^-11 of
    it, on codes at most 8 from the middle; scores in fp32: a sum of 2 D products of up to |q| (|m| + 15 s) each, of which
    each addition rounds by 2^-24, moves a weight by 2^-24 2 D sum|q| max|K| scale at the very worst (an eighth of that is
    allowed: errors of a sum add up as a walk), and exponentials within 2^-21. Where many rows share a KV head, keys and
    values are rounded to fp16, 2^-11 of each at most: a score of D such products moves by 2^-11 |q| max|K| scale as a walk of
    equal steps (four times that is allowed), and a weight by as much of itself."""
    cus, lens = cu.tolist(), c.len.tolist()
    G = q.shape[1] // c.Hk
    out, tol = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b in range(len(cus) - 1):
        n, nq = lens[b], cus[b + 1] - cus[b]
        if nq == 0:
            continue
        k, v = _values(c, "k", b, n, layer), _values(c, "v", b, n, layer)
        sm = c.v_scale[layer][c.table[b, :-(-n // c.bs)].long()].double().transpose(1, 2).reshape(-1, c.Hk, 2)[:n]
        pos = torch.arange(n - nq, n, device="cuda")[:, None]
        t = torch.arange(n, device="cuda")[None]
        see = (t <= pos) & ((t > pos - window) if window else (t >= 0))
        x = q[cus[b]:cus[b + 1]].double().view(nq, c.Hk, G, c.D)
        a = torch.einsum("ihgd,thd->hgit", x, k) * scale
        a = a.masked_fill(~see, float("-inf"))
        w = torch.softmax(a, -1)
        w = torch.where(see.any(-1)[..., None], w, 0.0)
        o = torch.einsum("hgit,thd->ihgd", w, v)
        out[cus[b]:cus[b + 1]] = o.reshape(nq, -1, c.D)
        if n == 0:
            continue
        rounding = 2.0 ** -11 * 8 * torch.einsum("hgit,th->ihg", w, sm[..., 0])[..., None]
        reach = x.abs().sum(-1, keepdim=True) * k.abs().amax((0, 2))[None, :, None, None] * abs(scale)
        scores = (2.0 ** -24 * c.D / 4 * reach / c.D ** 0.5 + 2.0 ** -20) * torch.einsum("hgit,thd->ihgd", w, v.abs()) * 2
        if nq * G > (24 if c.D == 128 else 32):
            walk = 2.0 ** -9 * x.square().sum(-1, keepdim=True).sqrt() * k.abs().amax((0, 2))[None, :, None, None] * abs(scale)
            scores = scores + (2 * walk + 2.0 ** -11) * torch.einsum("hgit,thd->ihgd", w, v.abs())
        tol[cus[b]:cus[b + 1]] = (2.0 ** -8 * o.abs() + rounding + scores).reshape(nq, -1, c.D)
    return out, tol + 1e-30


def _check(c, q, cu, out, scale, window=0, layer=0):
    want, tol = _attend_64(c, q, cu, scale, window, layer)
    rows = slice(int(cu[0]), int(cu[-1]))
    err = (out.double() - want).abs()[rows]
    assert bool(torch.isfinite(out[rows]).all())
    assert bool((err <= tol[rows]).all()), float((err / tol[rows]).max())


@pytest.mark.parametrize("Hk,G,D,bs,lens,news,window", [
    (1, 1, 128, 16, [1], [1], 0),
    (8, 4, 128, 64, [2000], [1], 0),
    (2, 8, 128, 16, [300, 17, 1000, 128, 129], [1] * 5, 0),
    (1, 5, 128, 32, [77, 500], [3, 4], 0),
    (3, 7, 128, 128, [400, 90, 260], [5, 1, 60], 0),
    (2, 16, 128, 16, [700, 64, 3], [1, 1, 1], 0),
    (1, 32, 128, 64, [900], [2], 0),
    (4, 4, 256, 16, [333, 40, 1200], [1, 2, 1], 0),
    (1, 12, 256, 128, [600, 129], [1, 7], 0),
    (2, 1, 256, 32, [64, 63, 65], [64, 63, 65], 0),
    (2, 4, 128, 16, [300, 130], [300, 130], 0),
    (1, 3, 128, 64, [1500, 200], [1, 40], 100),
    (2, 2, 128, 16, [1000], [200], 1),
    (1, 8, 128, 16, [5000, 31], [1, 9], 4096),
    (2, 4, 256, 128, [3000, 260], [1, 30], 257),
    (1, 6, 128, 16, [20000], [1], 0),
    (1, 2, 128, 32, [90] * 60, [1] * 60, 0),
    (1, 1, 128, 16, [17], [17], 0),
    (1, 1, 128, 64, [128, 129, 127, 256, 257, 1000], [128, 129, 127, 256, 257, 255], 0),
    (2, 8, 128, 128, [4000, 200, 5], [40, 16, 3], 0),
    (8, 4, 128, 64, [1500, 700, 64], [300, 1, 64], 0),
    (1, 24, 128, 16, [9000], [1], 0),
    (1, 3, 128, 32, [2000, 130], [700, 100], 300),
    (4, 16, 128, 16, [513, 100], [33, 1], 64),
    (1, 300, 128, 16, [260, 3], [2, 1], 0),
    (1, 3, 256, 16, [2000, 129], [700, 129], 0),
    (2, 8, 256, 64, [513, 4000, 200], [33, 300, 1], 0),
    (4, 4, 256, 32, [3000], [1000], 300),
    (1, 20, 256, 128, [260, 9000], [1, 7], 0),
    (1, 17, 256, 16, [9000], [1], 0),
    (1, 129, 256, 16, [300, 20], [1, 2], 0),
    (8, 2, 256, 32, [1, 128, 129, 127, 640], [1, 64, 65, 127, 640], 0),
    (1, 24, 128, 16, [700, 300], [1, 2], 0),
    (2, 25, 128, 32, [700, 3000], [1, 1], 0),
    (2, 33, 256, 32, [700, 3000], [1, 1], 0),
    (1, 1, 256, 16, [4000, 100], [600, 33], 256),
])
def test_attend(Hk, G, D, bs, lens, news, window):
    g = _gen(Hk * 1000 + G * 100 + bs)
    B = len(lens)
    c = _kv4(batch=B, n_kv_heads=Hk, head_dim=D, block_tokens=bs, n_blocks=sum(-(-n // bs) for n in lens) + 3,
             max_blocks=max(-(-n // bs) for n in lens))
    _filled(c, g, lens)
    T = sum(news)
    big = _bf16(g, T, 2 * Hk * G * D) * 1.5
    q = big[:, Hk * G * D:].view(T, Hk * G, D)
    out = torch.full((T + 2, Hk * G + 1, D), 9.0, dtype=torch.bfloat16, device="cuda")
    view = out[:T, :Hk * G]
    cu = _cu(news)
    assert c.attend(q, cu, scale=D ** -0.5, window=window, out=view) is view
    assert c.check_error() == 0
    _check(c, q, cu, view, D ** -0.5, window)
    assert bool((out[T:] == 9).all()) and bool((out[:, -1] == 9).all())
    again = c.attend(q, cu, scale=D ** -0.5, window=window)
    assert torch.equal(again, view)                # the same sums in the same order
    c.close()


def test_attend_many_requests_of_all_kinds():
    rng = np.random.default_rng(3)
    B = 700
    lens = rng.integers(0, 200, B)
    news = np.minimum(rng.integers(0, 4, B), lens)
    lens[5], news[5] = 3000, 1
    lens[600], news[600] = 700, 90
    g = _gen(3)
    c = _kv4(batch=B, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=int((-(-lens // 16)).sum()), max_blocks=200)
    _filled(c, g, lens.tolist())
    q = _bf16(g, int(news.sum()), 6, 128)
    cu = _cu(news)
    out = c.attend(q, cu, scale=0.1)
    assert c.check_error() == 0
    _check(c, q, cu, out, 0.1)
    c.close()


@pytest.mark.parametrize("heads", [2, 4, 32, 96])
def test_attend_rows_that_see_nothing_give_zeros(heads):
    """More rows than tokens: the first ones lie before the request."""
    g = _gen(8)
    c = _kv4(batch=2, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=8, max_blocks=4)
    _filled(c, g, [3, 0])
    q = _bf16(g, 9, heads, 128)
    out = c.attend(q, _i32([0, 5, 9]), scale=0.1)
    assert bool((out[:2] == 0).all()) and bool((out[5:] == 0).all()) and bool((out[2:5] != 0).any())
    c.close()


@pytest.mark.parametrize("why", ["down", "long", "entry", "rows"])
def test_attend_leaves_out_what_is_out_of_bounds(why):
    abi = _abi()
    g = _gen(4)
    c = _kv4(batch=3, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=60, max_blocks=20)
    _filled(c, g, [200, 150, 90])
    q = _bf16(g, 9, 8, 128)
    cu = [0, 3, 5, 9]
    out = torch.full((9, 8, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    if why == "down":
        c.attend(q, _i32([0, 5, 3, 9]), scale=0.1, out=out)
        assert c.check_error() == abi.SRH_ERR_BOUNDS and bool((out == 9).all())
    elif why == "rows":
        c.attend(q, _i32([0, 3, 5, 12]), scale=0.1, out=out)
        assert c.check_error() == abi.SRH_ERR_BOUNDS
        _check(c, q[:5], _i32([0, 3, 5]), out[:5], 0.1)
    elif why == "long":
        c.len[1] = 321
        c.attend(q, _i32(cu), scale=0.1, out=out)
        assert c.check_error() == abi.SRH_ERR_BOUNDS and bool((out[3:5] == 9).all())
        c.len[1] = 0
        _check(c, q[:3], _i32([0, 3]), out[:3], 0.1)
    else:
        c.table[1, 2] = 60                         # tokens 32 .. 47 of request 1 are absent
        c.attend(q, _i32(cu), scale=0.1, out=out)
        assert c.check_error() == abi.SRH_ERR_BOUNDS
        c.table[1, 2] = 0
        k, v = _values(c, "k", 1, 150), _values(c, "v", 1, 150)
        keep = torch.tensor([t for t in range(149) if not 32 <= t < 48], device="cuda")
        x = q[3].double().view(2, 4, 128)
        w = torch.softmax(torch.einsum("hgd,thd->hgt", x, k[keep]) * 0.1, -1)
        want = torch.einsum("hgt,thd->hgd", w, v[keep]).reshape(8, 128)
        assert float((out[3].double() - want).abs().max()) < 2.0 ** -8 * float(want.abs().max()) + 0.01
    c.close()


@pytest.mark.parametrize("heads", [8, 24, 96])
def test_attend_whatever_lies_behind_a_request(heads):
    """Scales of NaN and infinity behind the length, in its last block and others, do not show."""
    g = _gen(21)
    c = _kv4(batch=2, n_kv_heads=2, head_dim=128, block_tokens=64, n_blocks=12, max_blocks=6)
    lens = [133, 65]
    _filled(c, g, lens)
    q = _bf16(g, 3, heads, 128)
    cu = _i32([0, 1, 3])
    want = c.attend(q, cu, scale=0.1)
    for scale in (c.k_scale[0], c.v_scale[0]):
        kept = torch.zeros(12, 64, dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens):
            for t in range(n):
                kept[int(c.table[b, t // 64]), t % 64] = True
        bad = ~kept[:, None, :, None]
        odd = torch.tensor([float("nan"), float("inf")], device="cuda").bfloat16()
        scale.copy_(torch.where(bad, odd, scale))
    assert torch.equal(c.attend(q, cu, scale=0.1), want)
    assert c.check_error() == 0
    c.close()


@pytest.mark.parametrize("offset", [0.0, 3.0])
@pytest.mark.parametrize("heads", [4, 24, 40])
def test_attend_equal_weights(offset, heads):
    """Where all tokens weigh the same, every weight rounds the same way: the mean of many values that nearly cancel must not
    show it. Per output: bf16's rounding, 2^-11 of the mean around V's middle, fp32 sums of 12,000 values of up to 7. With 40
    heads values are rounded to fp16 (2^-11 of each, and all weights alike: 2^-11 of the mean)."""
    g = _gen(77)
    n = 12000
    c = _kv4(batch=1, n_kv_heads=1, head_dim=128, block_tokens=32, n_blocks=400, max_blocks=400)
    _filled(c, g, [n], spread=0, mean=offset)
    c.v_scale[0][..., 0] = 0.3
    c.v_scale[0][..., 1] = offset - 2.25
    q = torch.zeros(1, heads, 128, device="cuda", dtype=torch.bfloat16)
    out = c.attend(q, _i32([0, 1]), scale=0.1).double()
    v = _values(c, "v", 0, n)[:, 0]
    want = v.mean(0)
    middle = float((c.v_scale[0][0, 0, 0, 1].double() + 8 * c.v_scale[0][0, 0, 0, 0].double()))
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -11 * (want - middle).abs() + 7 * 2.0 ** -20
    if heads > 24:
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -11 * want.abs() + 2.0 ** -11 * v.abs().mean(0) + 7 * 2.0 ** -20
    assert bool(((out[0] - want).abs() <= tol).all())
    c.close()


@pytest.mark.parametrize("heads", [1, 20, 40])
@pytest.mark.parametrize("share", [0.5, 0.999])
def test_attend_long_tail_behind_one_weight(share, heads):
    """One token with `share` of the weight in front of 30,000 equal ones that hold the rest between them."""
    g = _gen(78)
    n = 30001
    c = _kv4(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=2000, max_blocks=2000)
    _filled(c, g, [n], spread=0)
    # K: one dim decides; all others hold 0
    c.k_codes[0].zero_()
    c.k_scale[0][..., 0] = 1.0
    c.k_scale[0][..., 1] = 0.0
    first = int(c.table[0, 0])
    c.k_codes[0][first, 0, 0, 0] = 8               # token 0, dim 0
    lead = math.log(share / (1 - share) * (n - 1))
    q = torch.zeros(1, heads, 128, device="cuda", dtype=torch.bfloat16)
    q[0, :, 0] = lead / 8
    out = c.attend(q, _i32([0, 1]), scale=1.0)
    _check(c, q, _i32([0, 1]), out, 1.0)
    v = _values(c, "v", 0, n)[:, 0]
    assert float((v[1:].mean(0)).abs().max()) > 0.01
    c.close()


@pytest.mark.parametrize("G,D", [(2, 128), (12, 128), (40, 128), (3, 256), (24, 256), (40, 256)])
def test_attend_wide_scores_and_scales(G, D):
    """Scores over hundreds, rows of all sizes, constant rows (scale 0) of V, queries of 2^-40 to 2^40, scores of 10^14, scales
    below 0 and of 0."""
    g = _gen(79)
    c = _kv4(batch=2, n_kv_heads=2, head_dim=D, block_tokens=16, n_blocks=80, max_blocks=40)
    _filled(c, g, [600, 333], spread=9)
    c.v_scale[0][:, :, ::3, 0] = 0.0
    q = _bf16(g, 4, 2 * G, D)
    for k in (-40, 0, 6, 40, 7, 8, 9):
        x = (q.float() * 2.0 ** (k if k not in (7, 8, 9) else 0)).bfloat16()
        scale = {6: 0.1 * 2.0 ** -6 * 32, 7: 1e11, 8: -0.05, 9: 0.0}.get(k, 0.1 * 2.0 ** -k)
        cu = _i32([0, 1, 4])
        out = c.attend(x, cu, scale=scale)
        _check(c, x, cu, out, scale)
    c.close()


@pytest.mark.parametrize("extra,scale", [(0, 0.1), (30, 0.1), (0, 1e11), (30, 1e11)])
def test_attend_a_row_that_is_not_finite_is_nan_alone(extra, scale):
    g = _gen(80)
    c = _kv4(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=40, max_blocks=40)
    _filled(c, g, [500])
    q = _bf16(g, 2 + extra, 4, 128)
    q[0, 1, 7] = float("inf")
    q[1, 2, 3] = float("nan")
    cu = _i32([0, 2 + extra])
    out = c.attend(q, cu, scale=scale)
    nan = torch.isnan(out).all(-1)
    assert nan[:2].tolist() == [[False, True, False, False], [False, False, True, False]] and not bool(nan[2:].any())
    q[0, 1, 7], q[1, 2, 3] = 0, 0
    want = c.attend(q, cu, scale=scale)
    assert torch.equal(out[~nan], want[~nan])
    c.close()


def test_codes_past_32_bit_offsets():
    """Blocks 1.5 GB apart: offsets of codes pass 32 bits."""
    g = _gen(81)
    nb, stride = 5, 3 << 29
    codes = [torch.zeros(nb * stride, dtype=torch.uint8, device="cuda") for _ in "kv"]
    views = [t.as_strided((nb, 2, 16, 64), (stride, 16 * 64, 64, 1)) for t in codes]
    c = _kv4(batch=1, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=nb, max_blocks=nb,
             buffers=dict(k_codes=views[0], v_codes=views[1]))
    cu, _, _ = c.resize(_i32([75]), 75)
    k, v = _bf16(g, 75, 2, 128), _bf16(g, 75, 2, 128)
    c.append(k, v, cu)
    kb, vb = c.read(_i32([0]), cu, 75)
    assert float((kb.double() - k.double()).abs().max()) < 0.5 and float((vb.double() - v.double()).abs().max()) < 0.5
    q = _bf16(g, 2, 4, 128)
    out = c.attend(q, _i32([0, 2]), scale=0.1)
    _check(c, q, _i32([0, 2]), out, 0.1)
    c.close()


def test_graph_follows_new_lengths():
    g = _gen(82)
    lens = [300, 50, 1000]
    c = _kv4(batch=3, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=150, max_blocks=80)
    c.resize(_i32(lens))
    for codes, scale in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)):
        codes[0].copy_(torch.randint(0, 256, codes[0].shape, generator=g, device="cuda", dtype=torch.uint8))
        scale[0][..., 0], scale[0][..., 1] = 0.3, -2.0
    new, start = _i32(lens), _i32([0, 0, 0])
    q, k, v = _bf16(g, 3, 8, 128), _bf16(g, 3, 2, 128), _bf16(g, 3, 2, 128)
    out, kb, vb = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    cu, pos, slot = torch.empty(4, dtype=torch.int32, device="cuda"), _i32([0] * 3), torch.zeros(3, dtype=torch.int64, device="cuda")

    def step():
        start.copy_(c.len[:3])
        c.resize(new, 3, out=(cu, pos, slot))
        c.append(k, v, cu)
        c.read(start, cu, 3, k_out=kb, v_out=vb)
        c.attend(q, cu, scale=0.1, out=out)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        new += 1
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for add in ([1, 1, 1], [1, 0, 1], [0, 1, 0], [1, 1, 1]):
        new += _i32(add)
        k.copy_(_bf16(g, 3, 2, 128))
        graph.replay()
        assert c.check_error() == 0
        t = sum(add)
        assert int(cu[-1]) == t
        _check(c, q, cu, out, 0.1)
        assert float((kb[:t].double() - k[:t].double()).abs().max()) < 0.3
    c.close()


def test_calls_on_a_stream_of_their_own():
    g = _gen(83)
    c = _kv4(batch=1, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=150, max_blocks=150)
    s = torch.cuda.Stream()
    new = _i32([2000])
    k, v, q = _bf16(g, 2000, 2, 128), _bf16(g, 2000, 2, 128), _bf16(g, 1, 8, 128)
    torch.cuda.synchronize()
    cu, _, _ = c.resize(new, 2000, stream=s)
    c.append(k, v, cu, stream=s)
    with torch.cuda.stream(s):
        one, zero = _i32([0, 1]), _i32([0])
    kb, vb = c.read(zero, cu, 2000, stream=s)
    out = c.attend(q, one, scale=0.1, stream=s.cuda_stream)
    s.synchronize()
    _check(c, q, one, out, 0.1)
    assert torch.equal(kb, _values(c, "k", 0, 2000).float().bfloat16()) and torch.equal(vb, _values(c, "v", 0, 2000).float().bfloat16())
    c.close()


def test_layers_of_both_widths_on_one_table():
    """A 4-bit and an 8-bit pool on one handle's tables through the C entry points."""
    abi = _abi()
    g = _gen(84)
    c4 = _kv4(batch=2, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=20, max_blocks=10)
    c8 = _kv8(batch=2, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=20, max_blocks=10,
              buffers=dict(table=c4.table, len=c4.len, free=c4.free, n_free=c4.n_free))
    cu, _, _ = c4.resize(_i32([60, 100]), 160)
    k, v = _bf16(g, 160, 2, 128), _bf16(g, 160, 2, 128)
    c4.append(k, v, cu)
    c8.append(k, v, cu)
    q = _bf16(g, 2, 8, 128)
    a, b = c4.attend(q, _i32([0, 1, 2]), scale=0.1), c8.attend(q, _i32([0, 1, 2]), scale=0.1)
    _check(c4, q, _i32([0, 1, 2]), a, 0.1)
    assert float((a.double() - b.double()).abs().max()) < 0.2
    # the 8-bit pool through the 4-bit cache's handle
    lib = abi.load()
    k2 = torch.empty_like(k)
    v2 = torch.empty_like(v)
    start = _i32([0, 0])
    assert lib.kv8_read(c4.cache, c8._pool[0], c4.table.data_ptr(), c4.len.data_ptr(), start.data_ptr(), cu.data_ptr(), 2,
                        k2.data_ptr(), 256, v2.data_ptr(), 256, 160, torch.cuda.current_stream().cuda_stream) == 0
    want = c8.read(start, cu, 160)
    assert torch.equal(k2, want[0]) and torch.equal(v2, want[1])
    c4.close()
    c8.close()


def test_refusals():
    abi = _abi()
    c = _kv4(batch=2, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=20, max_blocks=10, layers=2)
    g = _gen(1)
    q, k = _bf16(g, 4, 8, 128), _bf16(g, 4, 2, 128)
    cu, start = _i32([0, 2, 4]), _i32([0, 0])
    for bad in (lambda: c.append(k, None, cu), lambda: c.append(k[:, :1], k, cu), lambda: c.append(k.float(), k, cu),
                lambda: c.append(k, k[:3], cu), lambda: c.attend(q[:, :, :64], cu, scale=1.0),
                lambda: c.attend(q, cu.long(), scale=1.0), lambda: c.read(start[:1], cu, 4), lambda: c.read(start, cu, -1),
                lambda: c.read(start, cu, 4, k_out=k[:3]), lambda: c.read(start, cu, 4, v_out=k.float()),
                lambda: c.read(start.cpu(), cu, 4)):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros(4, 7, 128, device="cuda", dtype=torch.bfloat16)
    for bad in (lambda: c.attend(odd, cu, scale=1.0), lambda: c.attend(q, cu, scale=float("nan")),
                lambda: c.attend(q, cu, scale=1.0, window=-1), lambda: c.attend(q, cu, scale=1.0, out=q),
                lambda: c.read(start, cu, 4, k_out=k, v_out=k)):
        with pytest.raises(abi.SrhError) as e:
            bad()
        assert e.value.code == abi.SRH_ERR_INVALID
    lib = abi.load()
    pool = abi.Kv4Pool(c.k_codes[0].data_ptr(), c.k_scale[0].data_ptr(), c.v_codes[0].data_ptr(), c.v_scale[0].data_ptr(), 0)

    def append(p, handle=c.cache):
        return lib.kv4_append(handle, p, c.table.data_ptr(), c.len.data_ptr(), cu.data_ptr(), 2, k.data_ptr(), 256,
                              k.data_ptr(), 256, 4, 0)
    for field, value in (("k_codes", 0), ("v_scale", 0), ("k_codes", pool.k_codes + 8), ("v_scale", pool.v_scale + 4),
                         ("block_stride", 2 * 16 * 64 - 16), ("block_stride", 2 * 16 * 64 + 8), ("block_stride", 1 << 40)):
        p = abi.Kv4Pool(*(getattr(pool, f) for f, _ in abi.Kv4Pool._fields_))
        setattr(p, field, value)
        assert append(p) == abi.SRH_ERR_INVALID, field
    assert append(None) == abi.SRH_ERR_INVALID
    shared = _kv8(batch=2, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=20, max_blocks=10, shared_kv=True)
    assert append(pool, shared.cache) == abi.SRH_ERR_INVALID
    wide = _kv8(batch=2, n_kv_heads=2, head_dim=512, block_tokens=16, n_blocks=20, max_blocks=10)
    assert append(pool, wide.cache) == abi.SRH_ERR_INVALID
    with pytest.raises(ValueError):
        _kv4(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=4, max_blocks=4,
             buffers=dict(k_codes=torch.zeros(4, 1, 16, 128, dtype=torch.uint8, device="cuda")))
    with pytest.raises(ValueError):
        _kv4(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=4, max_blocks=4,
             buffers=dict(k_scale=torch.zeros(4, 1, dtype=torch.float32, device="cuda")))
    assert c.check_error() == 0
    for x in (c, shared, wide):
        x.close()


# ---------------------------------------------------------------------------------------------- rotation by several axes
def _axes_64(x, w, pos, axis, freq, rot, off, style, eps):
    x = x.double()
    y = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * w.double()
    angle = pos.double()[axis.long()].t() * freq                # [tokens, pairs]
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    i = torch.arange(rot // 2, device="cuda")
    a, b = (off + 2 * i, off + 2 * i + 1) if style == "pairs" else (off + i, off + rot // 2 + i)
    out = y.clone()
    out[..., a] = y[..., a] * cos - y[..., b] * sin
    out[..., b] = y[..., a] * sin + y[..., b] * cos
    size = y.abs()
    size[..., a] = size[..., b] = torch.sqrt(y[..., a] ** 2 + y[..., b] ** 2)
    return out, size


@pytest.mark.parametrize("T,H,Hk,D,rot,off,style,axes", [
    (1, 4, 1, 128, 128, 0, "halves", 3), (77, 6, 2, 96, 32, 64, "pairs", 2), (300, 3, 3, 64, 64, 0, "halves", 8),
    (50, 2, 1, 256, 256, 0, "pairs", 3), (33, 5, 1, 512, 64, 448, "halves", 4), (9, 2, 2, 512, 512, 0, "pairs", 1),
    (2000, 8, 2, 128, 128, 0, "pairs", 3)])
def test_rotation_by_axes(T, H, Hk, D, rot, off, style, axes):
    """bf16's rounding (2^-8 of the result), the norm and the factors in fp32, cos and sin within 2^-22 and the angle's 2^-26
    of a turn, of the pair's length."""
    g = _gen(T + D)
    c = _kv4(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=1, max_blocks=1)
    q, k = _bf16(g, T, H, D), _bf16(g, T, Hk, D)
    wq, wk = (1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in "qk")
    big = torch.randint(-5000, 100000, (axes, T + 5), generator=g, device="cuda", dtype=torch.int32)
    pos = big[:, 2:T + 2]                                        # rows apart
    axis = torch.randint(0, axes, (rot // 2,), generator=g, device="cuda", dtype=torch.uint8)
    freq = 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) / (rot // 2))
    qo, ko = c.norm_rope(q, k, pos=pos, axis=axis, inv_freq=freq, rot_dim=rot, rot_off=off, style=style, q_weight=wq, k_weight=wk)
    assert c.check_error() == 0
    for x, w, out in ((q, wq, qo), (k, wk, ko)):
        want, size = _axes_64(x, w, pos, axis, freq, rot, off, style, 1e-6)
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -19 * size + 1e-30
        assert bool(((out.double() - want).abs() <= tol).all())
    # each axis the same positions: what one axis gives, bit for bit
    same = pos[:1].expand(axes, T).contiguous()
    q1, k1 = c.norm_rope(q, k, pos=same, axis=axis, inv_freq=freq, rot_dim=rot, rot_off=off, style=style, q_weight=wq, k_weight=wk)
    q2, k2 = c.norm_rope(q, k, pos=same[0].contiguous(), inv_freq=freq, rot_dim=rot, rot_off=off, style=style, q_weight=wq, k_weight=wk)
    assert torch.equal(q1, q2) and torch.equal(k1, k2)
    # in place, and to slots
    slot = torch.randperm(T + 3, generator=g, device="cuda")[:T]
    slot[0] = -1
    rows = torch.full((T + 3, Hk, D), 7.0, dtype=torch.bfloat16, device="cuda")
    x = q.clone()
    c.norm_rope(x, k, pos=pos, axis=axis, inv_freq=freq, rot_dim=rot, rot_off=off, style=style, q_weight=wq, k_weight=wk, q_out=x,
                k_out=rows, k_slot=slot)
    assert torch.equal(x, qo) and torch.equal(rows[slot[1:]], ko[1:])
    c.close()


def test_rotation_by_axes_refusals_and_an_axis_that_is_none():
    abi = _abi()
    g = _gen(2)
    c = _kv4(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=1, max_blocks=1)
    q = _bf16(g, 5, 2, 64)
    pos = torch.randint(0, 100, (3, 5), generator=g, device="cuda", dtype=torch.int32)
    freq = torch.ones(32, dtype=torch.float64, device="cuda")
    axis = torch.zeros(32, dtype=torch.uint8, device="cuda")
    axis[7] = 3
    out, _ = c.norm_rope(q, pos=pos, axis=axis, inv_freq=freq, rot_dim=64, style="pairs")
    assert c.check_error() == abi.SRH_ERR_BOUNDS
    still, _ = c.norm_rope(q)
    turned, _ = c.norm_rope(q, pos=pos[0].contiguous(), inv_freq=freq, rot_dim=64, style="pairs")
    turned[..., 14:16] = still[..., 14:16]
    assert torch.equal(out, turned)
    for kw in (dict(pos=pos, axis=axis.int()), dict(pos=pos, axis=axis[:31]), dict(pos=pos[0].contiguous(), axis=axis),
               dict(pos=pos.long(), axis=axis), dict(pos=pos.repeat(3, 1), axis=axis), dict(pos=pos[:, :4], axis=axis),
               dict(pos=pos.t().contiguous().t(), axis=axis), dict(pos=pos[:1].expand(3, 5), axis=axis)):
        with pytest.raises(ValueError):
            c.norm_rope(q, inv_freq=freq, rot_dim=64, style="pairs", **kw)
    assert c.check_error() == 0
    c.close()


# ---------------------------------------------------------------------------------------------- all of them
def test_serving_loop():
    """Prompts of text and images, decode steps, drafts that are taken back, a prefix handed on to an 8-bit cache."""
    rng = np.random.default_rng(9)
    g = _gen(9)
    B, Hk, G, D, bs, layers = 5, 2, 4, 128, 16, 2
    c = _kv4(batch=B, n_kv_heads=Hk, head_dim=D, block_tokens=bs, n_blocks=120, max_blocks=30, layers=layers)
    freq = 10000.0 ** (-torch.arange(D // 2, device="cuda", dtype=torch.float64) / (D // 2))
    axis = (torch.arange(D // 2, device="cuda") % 3).to(torch.uint8)
    lens = [0] * B
    rows = [[[] for _ in range(B)] for _ in range(layers)]      # what each request's keys and values were
    for step in range(8):
        if step == 0:
            new = rng.integers(1, 200, B)
        elif step == 4:
            new = rng.integers(20, 60, B)
        else:
            new = rng.integers(0, 6, B)
        lens = [a + int(n) for a, n in zip(lens, new)]
        T = int(new.sum())
        cu, p, slot = c.resize(_i32(lens), T)
        pos = torch.stack((p, p // 7, p % 7))
        for layer in range(layers):
            q, k, v = _bf16(g, T, Hk * G, D), _bf16(g, T, Hk, D), _bf16(g, T, Hk, D)
            q, k = c.norm_rope(q, k, pos=pos, axis=axis, inv_freq=freq, rot_dim=D, style="halves")
            c.append(k, v, cu, layer=layer)
            out = c.attend(q, cu, scale=D ** -0.5, layer=layer)
            assert c.check_error() == 0
            _check(c, q, cu, out, D ** -0.5, layer=layer)
            cl = cu.tolist()
            for b in range(B):
                rows[layer][b] += list(zip(k[cl[b]:cl[b + 1]], v[cl[b]:cl[b + 1]]))
        if step % 3 == 2:                                       # some drafts go back
            keep = [max(1, n - int(rng.integers(0, 4))) for n in lens]
            c.resize(_i32(keep))
            for layer in range(layers):
                for b in range(B):
                    del rows[layer][b][keep[b]:]
            lens = keep
    T = sum(lens)
    cu, start = _cu(lens), _i32([0] * B)
    c8 = _kv8(batch=B, n_kv_heads=Hk, head_dim=D, block_tokens=64, n_blocks=60, max_blocks=10)
    to, _, _ = c8.resize(_i32(lens), T)
    for layer in range(layers):
        k, v = c.read(start, cu, T, layer=layer)
        assert c.check_error() == 0
        for got, i in ((k, 0), (v, 1)):
            x = torch.stack([r[i] for b in range(B) for r in rows[layer][b]]).float()
            s = ((x.amax(-1) - x.amin(-1)) / 15)[..., None]
            # half a step (of a scale rounded by 2^-8, so that 15 steps may end half a step off), and bf16's rounding
            assert bool(((got.float() - x).abs() <= s * (0.5 + 16 * 2.0 ** -8) + 2.0 ** -8 * x.abs() + 1e-6).all())
        c8.append(k, v, to)
        k8, v8 = c8.read(start, to, T)
        assert c8.check_error() == 0
        for a, b in ((k, k8), (v, v8)):
            assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -4 * float(a.abs().max())
    c.close()
    c8.close()


@pytest.mark.parametrize("G,news", [(4, 1), (4, 30)])
def test_blocks_given_up_behind_a_window(G, news):
    """Table entries that no query sees any more may be gone: they are not reported."""
    g = _gen(85)
    c = _kv4(batch=1, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=70, max_blocks=64)
    _filled(c, g, [1000])
    q = _bf16(g, news, 2 * G, 128)
    cu = _i32([0, news])
    want = c.attend(q, cu, scale=0.1, window=200)
    c.table[0, :(1000 - news - 199) // 16] = -1
    c.table[0, 63:] = -1
    out = c.attend(q, cu, scale=0.1, window=200)
    assert c.check_error() == 0 and torch.equal(out, want)
    c.close()


@pytest.mark.parametrize("Hk,G,n,news", [(1, 8, 60000, 1), (1, 8, 60000, 5), (1, 16, 100000, 1), (1, 4, 40000, 60)])
def test_one_long_request_over_all_parts(Hk, G, n, news):
    """Parts of many CTAs, joined in groups."""
    g = _gen(86)
    c = _kv4(batch=1, n_kv_heads=Hk, head_dim=128, block_tokens=64, n_blocks=n // 64 + 1, max_blocks=n // 64 + 1)
    _filled(c, g, [n])
    q = _bf16(g, news, Hk * G, 128)
    cu = _i32([0, news])
    out = c.attend(q, cu, scale=0.1)
    _check(c, q, cu, out, 0.1)
    for _ in range(3):
        assert torch.equal(c.attend(q, cu, scale=0.1), out)
    c.close()


@pytest.mark.parametrize("D", [128, 256])
def test_a_mixed_batch_captured_and_replayed_with_other_lengths(D):
    """A mixed batch through both kernels in a captured call, replayed with other lengths; rows behind the last request stay."""
    g = _gen(87)
    B = 9
    lens, news = [900, 40, 700, 300, 1, 2000, 64, 512, 130], [200, 1, 1, 90, 1, 3, 64, 0, 1]
    c = _kv4(batch=B, n_kv_heads=2, head_dim=D, block_tokens=16, n_blocks=400, max_blocks=150)
    _filled(c, g, lens)
    T = sum(news)
    q = _bf16(g, T + 40, 8, D)
    cu = _cu(news)
    out = torch.full_like(q, 9.0)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c.attend(q, cu, scale=0.1, out=out)
    torch.cuda.synchronize()
    _check(c, q, cu, out, 0.1)
    assert bool((out[T:] == 9).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attend(q, cu, scale=0.1, out=out)
    for news in ([1] * B, [1, 40, 1, 300, 0, 9, 2, 30, 1], [0] * B, [230, 0, 0, 0, 0, 0, 0, 0, 0]):
        cu.copy_(_cu(news))
        out.fill_(9.0)
        graph.replay()
        assert c.check_error() == 0
        T = sum(news)
        if T:
            _check(c, q, cu, out, 0.1)
        assert bool((out[T:] == 9).all())
    c.close()


def test_two_handles_at_once():
    """Two caches on two streams: nothing of one shows in the other."""
    g = _gen(88)
    cs, outs, qs, cus = [], [], [], []
    for k in range(2):
        c = _kv4(batch=3, n_kv_heads=2, head_dim=128, block_tokens=32, n_blocks=200, max_blocks=100)
        _filled(c, g, [3000, 800 + k, 1500])
        cs.append(c)
        qs.append(_bf16(g, 42, 8, 128))
        cus.append(_i32([0, 1, 41, 42]))
    want = [c.attend(q, cu, scale=0.1) for c, q, cu in zip(cs, qs, cus)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        outs = [c.attend(q, cu, scale=0.1, stream=s) for c, q, cu, s in zip(cs, qs, cus, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    for c in cs:
        c.close()


def test_the_largest_batch():
    """4,096 requests: tables found by bisection, prefix sums over all of them."""
    g = _gen(89)
    rng = np.random.default_rng(89)
    B = 4096
    lens = rng.integers(1, 40, B)
    lens[4000] = 2500
    news = np.minimum(rng.integers(0, 3, B), lens)
    news[4000] = 70
    c = _kv4(batch=B, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=int((-(-lens // 16)).sum()), max_blocks=160)
    _filled(c, g, lens.tolist())
    T = int(news.sum())
    k, v, cu = _bf16(g, T, 1, 128), _bf16(g, T, 1, 128), _cu(news)
    c.append(k, v, cu)
    kb, vb = c.read(_i32((lens - news).tolist()), cu, T)
    assert c.check_error() == 0
    for a, b in ((kb, k), (vb, v)):
        step = ((b.float().amax(-1) - b.float().amin(-1)) / 15)[..., None]
        assert bool(((a.float() - b.float()).abs() <= step * (0.5 + 16 * 2.0 ** -8) + 2.0 ** -8 * b.float().abs()).all())
    q = _bf16(g, T, 4, 128)
    out = c.attend(q, cu, scale=0.1)
    assert c.check_error() == 0
    pick = [0, 1, 17, 500, 2047, 4000, 4094, 4095]
    cl = cu.tolist()
    for b in pick:
        if cl[b + 1] == cl[b]:
            continue
        one = _kv4(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=c.n_blocks, max_blocks=160,
                   buffers=dict(k_codes=c.k_codes[0], v_codes=c.v_codes[0], k_scale=c.k_scale[0], v_scale=c.v_scale[0],
                                table=c.table[b:b + 1].contiguous(), len=c.len[b:b + 1].contiguous()))
        x = q[cl[b]:cl[b + 1]]
        _check(one, x, _i32([0, x.shape[0]]), out[cl[b]:cl[b + 1]], 0.1)
        one.close()
    c.close()


@pytest.mark.parametrize("G,D", [(4, 128), (20, 128), (40, 128), (4, 256), (20, 256), (40, 256)])
def test_attend_constant_rows_of_large_values(G, D):
    """V rows without a scale, 600 values of up to 2^36 (2^45.3 in sum; 2^47 is allowed)."""
    g = _gen(90)
    c = _kv4(batch=1, n_kv_heads=1, head_dim=D, block_tokens=16, n_blocks=40, max_blocks=40)
    _filled(c, g, [600])
    c.v_scale[0][..., 0] = 0.0
    c.v_scale[0][..., 1] = (torch.rand(c.v_scale[0].shape[:-1], generator=g, device="cuda") * 2.0 ** 36).bfloat16()
    q = _bf16(g, 2, G, D)
    cu = _i32([0, 2])
    out = c.attend(q, cu, scale=0.1)
    _check(c, q, cu, out, 0.1)
    c.close()


# ---------------------------------------------------------------------------------------------- attend, closely
def _few(D):
    """Query rows per KV head up to which a request's codes enter the products as they are."""
    return 24 if D == 128 else 32


def _close_64(c, q, cu, scale, window=0, gone=()):
    """(outputs, tolerance) in fp64, of requests whose keys and values lie well within fp16's range. `gone`: (request, token) that
    are absent.

    Where a request has more than _few rows per KV head keys and values are rounded to fp16 first, as documented, here too
    (scaled by 2^8, away from fp16's subnormals, as the kernel scales by its own power of two); what is left then, per output:
      2^-8 |o|             bf16's rounding;
      2^-11 sum w |v|      a weight's rounding to fp16 (as it is where codes enter exactly: of w s |n - 8|, n - 8 at most 8);
      sum w d |v - o|      d: what a score is off by. fp32 sums of D products, 16 at a time, two roundings or truncations of
                           2^-23 of all magnitudes each (codes enter as s <q, n> + m sum q, of larger magnitudes);
                           2^-22 of the score itself for the factors and the difference from the reference; 2^-19 for
                           logarithm, exponential and reciprocal;
      n / 8 2^-23 sum w |v|  fp32 sums of n weighted values, 16 at a time;
      2^-30 max |v|        weights below 2^-35 of the row's largest."""
    cus, lens = cu.tolist(), c.len.tolist()
    Hk, D, G = c.Hk, c.D, q.shape[1] // c.Hk
    out, tol = (torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in "ot")
    for b in range(len(cus) - 1):
        n, nq = lens[b], cus[b + 1] - cus[b]
        if nq == 0 or n == 0:
            continue
        many = nq * G > _few(D)
        k, v = _values(c, "k", b, n), _values(c, "v", b, n)
        blk = c.table[b, :-(-n // c.bs)].long()
        ksm, vsm = (t[0][blk].double().transpose(1, 2).reshape(-1, Hk, 2)[:n].abs() for t in (c.k_scale, c.v_scale))
        mid = (vsm[..., :1] * 8).expand(n, Hk, D)
        size_k, size_v = k.abs(), v.abs()
        if many:
            k, v = ((x * 256).half().double() / 256 for x in (k, v))
            mid = size_v
        else:
            size_k = (k.abs() + 2 * ksm[..., 1:])
            size_v = size_v + 2 * mid
        pos = torch.arange(n - nq, n, device="cuda")[:, None]
        t = torch.arange(n, device="cuda")[None]
        see = (t <= pos) & ((t > pos - window) if window else (t >= 0))
        for r, tok in gone:
            if r == b:
                see[:, tok] = False
        for h in range(Hk):
            x = q[cus[b]:cus[b + 1], h * G:(h + 1) * G].double()
            a = torch.einsum("igd,td->igt", x, k[:, h]) * scale
            d = torch.einsum("igd,td->igt", x.abs(), size_k[:, h]) * (abs(scale) * D / 8 * 2.0 ** -23) + 2.0 ** -22 * a.abs() + 2.0 ** -19
            w = torch.softmax(a.masked_fill(~see[:, None], float("-inf")), -1)
            w = torch.where(see.any(-1)[:, None, None], w, 0.0)
            o = w @ v[:, h]
            e = 2.0 ** -8 * o.abs() + (2.0 ** -11 * (w @ mid[:, h])) + n / 8 * 2.0 ** -23 * (w @ size_v[:, h])
            e += (w * d) @ v[:, h].abs() + (w * d).sum(-1, keepdim=True) * o.abs()
            e += 2.0 ** -30 * size_v[:, h].amax()
            out[cus[b]:cus[b + 1], h * G:(h + 1) * G] = o
            tol[cus[b]:cus[b + 1], h * G:(h + 1) * G] = e
    return out, tol


def _check_close(c, q, cu, out, scale, window=0, gone=()):
    want, tol = _close_64(c, q, cu, scale, window, gone)
    rows = slice(int(cu[0]), int(cu[-1]))
    bad = ~((out.double() - want).abs() <= tol)[rows]
    assert not bool(bad.any()), (int(bad.sum()), [int(i) for i in torch.nonzero(bad)[0]],
                                 float(((out.double() - want).abs() / (tol + 1e-300))[rows].nan_to_num(1e30).max()))


_SHAPES = [
    # few rows per KV head
    (2, 4, 128, 16, [300, 129, 128, 1], [5, 5, 1, 1], 0),
    (2, 8, 128, 64, [1000], [3], 100),
    (8, 1, 128, 16, [400, 17], [20, 17], 33),
    (1, 24, 128, 32, [6000], [1], 0),
    (2, 4, 256, 16, [300, 257], [7, 8], 0),
    (1, 8, 256, 32, [700], [4], 65),
    # up to a row tile's half: lanes take every other tile of tokens
    (2, 25, 128, 32, [300, 9000], [1, 1], 0),
    (1, 8, 128, 128, [4000, 200], [13, 16], 0),
    (4, 4, 128, 16, [900, 129], [30, 32], 200),
    (2, 8, 256, 64, [513, 4000], [12, 16], 0),
    (1, 40, 256, 16, [300], [3], 64),
    # more
    (2, 4, 128, 16, [700, 260], [300, 130], 0),
    (1, 300, 128, 16, [260, 3], [2, 1], 0),
    (2, 1, 128, 64, [1000, 520], [400, 515], 150),
    (1, 3, 256, 16, [2000, 129], [200, 129], 0),
    (2, 1, 256, 128, [600], [600], 256),
    # both kernels in one call
    (2, 4, 128, 32, [700, 260, 40], [100, 1, 5], 0),
    (2, 4, 256, 16, [700, 260, 40], [100, 1, 5], 90),
]


def _shape(case, seed):
    Hk, G, D, bs, lens, news, window = case
    g = _gen(seed)
    c = _kv4(batch=len(lens), n_kv_heads=Hk, head_dim=D, block_tokens=bs, n_blocks=sum(-(-n // bs) for n in lens) + 3,
             max_blocks=max(-(-n // bs) for n in lens))
    _filled(c, g, lens)
    return g, c, _cu(news)


@pytest.mark.parametrize("case", _SHAPES)
def test_attend_closely(case):
    """Outputs within what the documented roundings explain: a token lost or a few percent of the sums show."""
    g, c, cu = _shape(case, 92)
    Hk, G, D, _, _, news, window = case
    q = _bf16(g, sum(news), Hk * G, D)
    out = c.attend(q, cu, scale=D ** -0.5, window=window)
    assert c.check_error() == 0
    _check_close(c, q, cu, out, D ** -0.5, window)
    c.close()


@pytest.mark.parametrize("case", _SHAPES)
def test_attend_each_query_finds_its_token(case):
    """Keys of random signs and queries that are one of them, so that a token has nearly all the weight: a row's own, the one behind
    it, the first of its window and the one before, the edges of tiles, any. One token too many or too few is another answer."""
    g, c, cu = _shape(case, 93)
    Hk, G, D, bs, lens, news, window = case
    rng = np.random.default_rng(93)
    c.k_codes[0].copy_(torch.randint(0, 2, c.k_codes[0].shape, generator=g, device="cuda", dtype=torch.uint8) * 15 +
                       torch.randint(0, 2, c.k_codes[0].shape, generator=g, device="cuda", dtype=torch.uint8) * 240)
    c.k_scale[0][..., 0] = 0.125
    c.k_scale[0][..., 1] = -0.9375
    q = torch.zeros(sum(news), Hk * G, D, device="cuda", dtype=torch.bfloat16)
    at = 0
    for b, (n, nq) in enumerate(zip(lens, news)):
        k = torch.sign(_values(c, "k", b, n)).bfloat16()
        w = window or n
        aim = np.zeros((nq, Hk, G), dtype=np.int64)
        for i in range(nq):
            p = n - nq + i
            some = [p, p + 1, p - w + 1, p - w, p // 128 * 128, p // 128 * 128 - 1, (p - w + 1) // 128 * 128, n - nq, 0]
            some = [t for t in some if 0 <= t < n]
            for h in range(Hk):
                for r in range(G):
                    aim[i, h, r] = some[rng.integers(len(some))] if rng.random() < 0.6 else rng.integers(0, n)
        aim = torch.from_numpy(aim).cuda()
        for h in range(Hk):
            q[at:at + nq, h * G:(h + 1) * G] = k[aim[:, h], h]
        at += nq
    out = c.attend(q, cu, scale=1.0, window=window)
    assert c.check_error() == 0
    _check_close(c, q, cu, out, 1.0, window)
    c.close()


@pytest.mark.parametrize("case", [_SHAPES[i] for i in (0, 4, 6, 8, 9, 11, 12, 14, 16)])
@pytest.mark.parametrize("entry", ["none", "beyond"])
def test_attend_blocks_that_are_not_there(case, entry):
    """Table entries that are no block, in what rows see: those tokens are absent, and reported."""
    g, c, cu = _shape(case, 94)
    Hk, G, D, bs, lens, news, window = case
    gone = []
    for b, n in enumerate(lens):
        for j in {0, (n - 1) // bs // 2, max(0, (n - 130) // bs), max(0, (n - 1) // bs - 1)}:
            if (j + 1) * bs >= n or (window and (j + 1) * bs <= n - news[b] - window + 1):
                continue                               # (a last block stays: each row sees something)
            c.table[b, j] = -1 if entry == "none" else c.n_blocks
            gone += [(b, t) for t in range(j * bs, (j + 1) * bs)]
    assert gone
    q = _bf16(g, sum(news), Hk * G, D)
    out = c.attend(q, cu, scale=D ** -0.5, window=window)
    assert c.check_error() == _abi().SRH_ERR_BOUNDS
    for b in range(len(lens)):                         # (the values of absent tokens, which do not count)
        c.table[b].clamp_(0, c.n_blocks - 1)
    _check_close(c, q, cu, out, D ** -0.5, window, gone)
    c.close()


@pytest.mark.parametrize("D,G,nq", [(128, 4, 1), (128, 32, 1), (128, 40, 4), (256, 40, 1)])
@pytest.mark.parametrize("B", [1, 160])
def test_attend_a_long_prefix_of_zero_values(B, D, G, nq):
    """35,000 tokens whose values are all 0, with scores 5 (log2) higher behind the first tile, before 5,000 of ordinary values: in one
    CTA's share of a request (160 requests over the same blocks) and over many."""
    g = _gen(95)
    n, zero = 40000, 35072
    c = _kv4(batch=B, n_kv_heads=1, head_dim=D, block_tokens=64, n_blocks=n // 64, max_blocks=n // 64)
    _filled(c, g, [n], spread=0, mean=3.0)
    c.table[:] = torch.arange(n // 64, dtype=torch.int32, device="cuda")
    c.len.fill_(n)
    c.k_codes[0].zero_()
    c.k_scale[0][..., 0] = 1.0
    c.k_scale[0][..., 1] = 0.0
    c.k_codes[0][2:, 0, :, 0] = 8                      # dim 0 of the tokens from 128 on
    c.v_scale[0][:zero // 64] = 0.0
    q = torch.zeros(B * nq, G, D, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 5 * math.log(2) / 8
    out = c.attend(q, _i32([b * nq for b in range(B + 1)]), scale=1.0)
    assert c.check_error() == 0
    c.len[1:] = 0
    want, tol = _close_64(c, q[:nq], _i32([0, nq]), 1.0)
    assert float(want.abs().min()) > 0.05
    err = (out.view(B, nq, G, D).double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    c.close()


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("G,news", [(4, 1), (8, 2), (40, 1)])
def test_blocks_behind_a_window_may_hold_anything(G, news, D):
    """Blocks that no query sees any more may have gone to someone else, who has not written every row: scales of NaN and infinity
    in them do not show, 16 tokens before the first that is seen."""
    g = _gen(96)
    c = _kv4(batch=1, n_kv_heads=2, head_dim=D, block_tokens=16, n_blocks=70, max_blocks=64)
    q, cu = _bf16(g, news, 2 * G, D), _i32([0, news])
    for first in range(784, 848, 16):                  # the first token that is seen
        _filled(c, g, [1000])
        window = 1000 - news + 1 - first
        want = c.attend(q, cu, scale=0.1, window=window)
        spare = sorted(set(range(70)) - set(c.table[0].tolist()))[0]
        odd = torch.tensor([float("nan"), float("inf")], device="cuda").bfloat16()
        c.k_scale[0][spare], c.v_scale[0][spare] = odd, odd
        c.table[0, :first // 16] = spare
        out = c.attend(q, cu, scale=0.1, window=window)
        assert c.check_error() == 0 and torch.equal(out, want)
    c.close()


@pytest.mark.parametrize("D,G", [(128, 4), (128, 40), (128, 150), (256, 40)])
def test_attend_small_values_beside_large_ones(D, G):
    """A row that only sees a token 2^-28 as large as its neighbour: values are within 2^-11, or 2^-34 of the tile's largest."""
    c = _kv4(batch=1, n_kv_heads=1, head_dim=D, block_tokens=16, n_blocks=1, max_blocks=1)
    c.resize(_i32([2]))
    blk = int(c.table[0, 0])
    for t in (c.k_codes[0], c.k_scale[0], c.v_codes[0], c.v_scale[0]):
        t.zero_()
    c.k_scale[0][blk, 0, :, 0] = 1.0
    c.k_codes[0][blk, 0, 0, 0] = 15                    # token 0, dim 0
    g = _gen(97)
    c.v_codes[0][blk, 0, :2] = torch.randint(0, 256, (2, D // 2), generator=g, device="cuda", dtype=torch.uint8)
    c.v_scale[0][blk, 0, 0, 0] = 0.125
    c.v_scale[0][blk, 0, 1, 0] = 1.125 * 2.0 ** -32
    q = torch.zeros(1, G, D, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = -20                                    # token 0 weighs e^-300
    out = c.attend(q, _i32([0, 1]), scale=1.0)
    v = _values(c, "v", 0, 2)[:, 0]
    tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -11) * v[1].abs() + 2.0 ** -34 * v[0].abs().max()
    if G <= _few(D):                                   # (codes enter as n - 8)
        tol = (2.0 ** -8 + 2.0 ** -11) * v[1].abs() + 2.0 ** -11 * 8 * 1.125 * 2.0 ** -32
    err = (out[0].double() - v[1]).abs()
    assert bool((err <= tol).all()), float((err / (tol + 1e-300)).max())
    c.close()


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("B", [3, 40])
def test_append_rows_of_no_request_are_not_reported(B, D):
    """Rows before the first request and behind the last one may hold anything: nothing of them is stored, nothing is reported."""
    g = _gen(91)
    c = _kv4(batch=B, n_kv_heads=2, head_dim=D, block_tokens=16, n_blocks=2 * B + 2, max_blocks=4)
    _filled(c, g, [20] * B)
    news = [2 + b % 3 for b in range(B)]
    T = sum(news)
    k, v = _bf16(g, T + 12, 2, D), _bf16(g, T + 12, 2, D)
    for x, odd in ((k, float("nan")), (v, float("inf"))):
        x[:5] = odd
        x[T + 5:] = -odd
    k[T + 6], v[2] = 3e38, -3e38
    cu = _cu(news) + 5
    before = [t.clone() for t in (*_codes(c, "k"), *_codes(c, "v"))]
    c.append(k, v, cu)
    assert c.check_error() == 0
    kb, vb = c.read(_i32([20 - n for n in news]), cu, T + 12)
    assert c.check_error() == 0
    for a, b in ((kb, k), (vb, v)):
        assert bool((a[:5] == 0).all()) and bool((a[T + 5:] == 0).all())
        x = b[5:T + 5].float()
        step = ((x.amax(-1) - x.amin(-1)) / 15)[..., None]
        assert bool(((a[5:T + 5].float() - x).abs() <= step * (0.5 + 16 * 2.0 ** -8) + 2.0 ** -8 * x.abs()).all())
    # nothing but the requests' tokens has changed
    table = c.table.tolist()
    for t, was in zip((*_codes(c, "k"), *_codes(c, "v")), before):
        for b in range(B):
            for p in range(20 - news[b], 20):
                was[table[b][p // 16], :, p % 16] = t[table[b][p // 16], :, p % 16]
        assert torch.equal(t, was)
    # one of a request's own is
    k[5, 1, 3] = float("nan")
    c.append(k, v, cu)
    assert c.check_error() == _abi().SRH_ERR_RANGE
    c.close()


@pytest.mark.parametrize("D,new", [(128, 60), (128, 63), (256, 40), (256, 63), (128, 64), (128, 30), (256, 64), (256, 20)])
def test_idle_rows_of_the_table_change_nothing(D, new):
    """A prompt among 63 table rows that have no new tokens. Of more than 128 rows per KV head, and of fewer than the table's: the
    same kernels, and so the same bits, as by itself."""
    g = _gen(98)
    c = _kv4(batch=64, n_kv_heads=2, head_dim=D, block_tokens=16, n_blocks=900, max_blocks=80)
    _filled(c, g, [100] * 40 + [1200] + [100] * 23)
    q = _bf16(g, new, 8, D)
    cu = _cu([0] * 40 + [new] + [0] * 23)
    out = c.attend(q, cu, scale=0.1)
    assert c.check_error() == 0
    _check(c, q, cu, out, 0.1)
    one = _kv4(batch=1, n_kv_heads=2, head_dim=D, block_tokens=16, n_blocks=900, max_blocks=80,
               buffers=dict(k_codes=c.k_codes[0], v_codes=c.v_codes[0], k_scale=c.k_scale[0], v_scale=c.v_scale[0],
                            table=c.table[40:41].contiguous(), len=c.len[40:41].contiguous()))
    alone = one.attend(q, _i32([0, new]), scale=0.1)
    _check_close(one, q, _i32([0, new]), alone, 0.1)
    if 128 < new * 4 and new < 64:
        assert bool((out == alone).all())
    one.close()
    c.close()


@pytest.mark.parametrize("D", [128, 256])
def test_layers_of_both_widths_attend_on_one_handle(D):
    """Attention over 8-bit and 4-bit pools in turn on one handle, whose scratch they share: the bits that handles of their own
    give, captured and replayed too."""
    abi = _abi()
    g = _gen(99)
    lens, news = [3000, 200, 700, 40], [1, 130, 9, 1]
    kw = dict(batch=4, n_kv_heads=2, head_dim=D, block_tokens=32, n_blocks=160, max_blocks=100)
    c4 = _kv4(**kw)
    _filled(c4, g, lens)
    c8 = _kv8(buffers=dict(table=c4.table, len=c4.len), **kw)
    for codes, scale in ((c8.k_codes, c8.k_scale), (c8.v_codes, c8.v_scale)):
        codes[0].copy_(torch.randn(codes[0].shape, generator=g, device="cuda").to(FP8).view(torch.uint8))
        scale[0].fill_(0.5)
    T = sum(news)
    q, cu = _bf16(g, T, 8, D), _cu(news)
    one = _i32([0, 1, 2, 3, 4])                        # a decode step
    want = [(c4.attend(q, x, scale=0.1), c8.attend(q, x, scale=0.1)) for x in (cu, one)]
    lib = abi.load()
    outs = [[torch.zeros_like(q) for _ in range(2)] for _ in range(2)]

    def call(fn, pool, x, out):
        rows = T if x is cu else 4
        assert fn(c8.cache, pool, c4.table.data_ptr(), c4.len.data_ptr(), x.data_ptr(), 4, q.data_ptr(), 8 * D, rows, 8, 0.1, 0,
                  out.data_ptr(), 8 * D, torch.cuda.current_stream().cuda_stream) == 0

    def step():
        for (a, b), x in zip(outs, (cu, one)):
            call(lib.kv4_attend, c4._pool[0], x, a)
            call(lib.kv8_attend, c8._pool[0], x, b)
            call(lib.kv4_attend, c4._pool[0], x, a)

    def check():
        assert c8.check_error() == 0
        for got, exp, rows in zip(outs, want, (T, 4)):
            for a, b in zip(got, exp):
                assert torch.equal(a[:rows], b[:rows])
                a.zero_()

    for _ in range(3):
        step()
        check()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        graph.replay()
        check()
    c4.close()
    c8.close()


def test_pools_whose_blocks_are_not_16_bytes_apart_are_refused_at_once():
    """As PagedKV8 refuses them: when the cache is made, not by its first call."""
    kw = dict(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=4, max_blocks=4)
    for make, width in ((_kv4, 64), (_kv8, 128)):
        n = 16 * width + 8
        codes = torch.zeros(4 * n, dtype=torch.uint8, device="cuda").as_strided((4, 1, 16, width), (n, 16 * width, width, 1))
        with pytest.raises((ValueError, _abi().SrhError)):
            make(buffers=dict(k_codes=codes), **kw)


@pytest.mark.parametrize("G,D", [(4, 128), (40, 128), (4, 256), (40, 256)])
def test_attend_queries_of_any_size(G, D):
    """Queries of 2^-98 and 2^98 with scales that make up for it: the bits of ordinary ones."""
    g = _gen(100)
    c = _kv4(batch=1, n_kv_heads=2, head_dim=D, block_tokens=16, n_blocks=20, max_blocks=20)
    _filled(c, g, [300])
    q, cu = _bf16(g, 2, 2 * G, D), _i32([0, 2])
    want = c.attend(q, cu, scale=0.0625)
    _check_close(c, q, cu, want, 0.0625)
    for k in (-98, 98):
        out = c.attend((q.double() * 2.0 ** k).bfloat16(), cu, scale=0.0625 * 2.0 ** -k)
        assert bool((out == want).all())
    c.close()
