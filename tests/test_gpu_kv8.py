"""The paged 8-bit cache (kv8_*) against plain 64-bit implementations: block
tables and slots, norm + rotation, quantised append, attention, and a serving
loop of all four."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn
NAN_CODE = 0x7F


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def _abi():
    from sparse_retrieval_host_gb300 import abi
    return abi


def _paged(**kw):
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


# ---------------------------------------------------------------------------------------------- resize
class ResizeOracle:
    """The free stack and the tables in plain Python."""

    def __init__(self, batch, bs, n_blocks):
        self.bs, self.free = bs, list(range(n_blocks - 1, -1, -1))
        self.len, self.table = [0] * batch, [[] for _ in range(batch)]

    def resize(self, new):
        bs = self.bs
        gone = []
        for b, n in enumerate(new):
            need = -(-n // bs)
            gone += self.table[b][need:]
            self.table[b] = self.table[b][:need]
        self.free += gone[::-1]
        cu, pos, slot = [0], [], []
        for b, n in enumerate(new):
            while len(self.table[b]) < -(-n // bs):
                self.table[b].append(self.free.pop())
            for p in range(self.len[b], n):
                pos.append(p)
                slot.append(self.table[b][p // bs] * bs + p % bs)
            self.len[b] = n
            cu.append(len(pos))
        return cu, pos, slot


def _same_tables(c, o, n):
    assert c.len[:n].tolist() == o.len[:n]
    table = c.table.tolist()
    for b in range(n):
        assert table[b] == o.table[b] + [-1] * (c.max_blocks - len(o.table[b])), b
    assert int(c.n_free) == len(o.free)
    assert c.free[:len(o.free)].tolist() == o.free


@pytest.mark.parametrize("batch,bs,most,steps", [(1, 16, 40, 8), (7, 16, 300, 12), (33, 64, 700, 8), (1500, 32, 70, 4),
                                                 (4096, 16, 33, 3), (3, 128, 9000, 4)])
def test_resize_follows_the_oracle(batch, bs, most, steps):
    rng = np.random.default_rng(batch * 131 + bs)
    max_blocks = -(-most // bs)
    n_blocks = batch * max_blocks
    c = _paged(batch=batch, n_kv_heads=1, head_dim=128, block_tokens=bs, n_blocks=n_blocks, max_blocks=max_blocks)
    o = ResizeOracle(batch, bs, n_blocks)
    for step in range(steps):
        new = rng.integers(0, most + 1, batch)
        if step % 3 == 1:       # a decode step: one token more where there is room
            new = np.minimum(np.array(o.len) + 1, most)
        if step % 3 == 2:       # some requests end
            new[rng.random(batch) < 0.5] = 0
        room = int(np.maximum(new - np.array(o.len), 0).sum())
        extra = int(rng.integers(0, 3))
        cu, pos, slot = (torch.full((k,), -7, dtype=t, device="cuda") for k, t in
                         ((batch + 1, torch.int32), (room + extra, torch.int32), (room + extra, torch.int64)))
        c.resize(_i32(new.tolist()), room + extra, out=(cu, pos, slot))
        want = o.resize(new.tolist())
        assert cu.tolist() == want[0]
        if room + extra:
            assert pos.tolist() == want[1] + [-7] * extra and slot.tolist() == want[2] + [-7] * extra
        _same_tables(c, o, batch)
        assert c.check_error() == 0
    c.close()


def test_resize_shrinks_back_exactly_and_reuses_in_order():
    c = _paged(batch=3, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=32, max_blocks=10)
    c.resize(_i32([20, 0, 40]), 60)
    table, free = c.table.clone(), c.free[:int(c.n_free)].clone()
    c.resize(_i32([100, 33, 41]), 200)
    c.resize(_i32([20, 0, 40]))
    assert torch.equal(c.table, table) and torch.equal(c.free[:int(c.n_free)], free)
    assert c.check_error() == 0
    c.close()


def test_resize_only_some_requests_leaves_the_others():
    c = _paged(batch=4, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=32, max_blocks=8)
    c.resize(_i32([17, 5, 90, 16]), 128)
    before, lens = c.table.clone(), c.len.clone()
    c.resize(_i32([40, 2]), 23)
    assert torch.equal(c.table[2:], before[2:]) and torch.equal(c.len[2:], lens[2:])
    assert c.len.tolist() == [40, 2, 90, 16]
    c.close()


@pytest.mark.parametrize("why", ["blocks", "cap", "negative", "long", "bad_len", "bad_entry", "depth"])
def test_resize_refuses_whole_calls(why):
    abi = _abi()
    c = _paged(batch=3, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=8, max_blocks=6)
    c.resize(_i32([30, 10, 0]), 40)
    new, cap, code = [40, 10, 20], 64, abi.SRH_ERR_BOUNDS
    if why == "blocks":
        new, cap, code = [90, 60, 10], 200, abi.SRH_ERR_NOMEM
    elif why == "cap":
        cap = 29
    elif why == "negative":
        new = [40, -1, 20]
    elif why == "long":
        new = [97, 10, 20]
    elif why == "bad_len":
        c.len[1] = -5
    elif why == "bad_entry":
        new = [30, 0, 0]
        c.table[1, 0] = 99
    elif why == "depth":
        c.n_free.fill_(9)
    table, lens, free, n_free = c.table.clone(), c.len.clone(), c.free.clone(), c.n_free.clone()
    cu, pos, slot = c.resize(_i32(new), cap, out=(_i32([5] * 4), _i32([-7] * cap), torch.full((cap,), -7, device="cuda")))
    assert cu.tolist() == [0] * 4 and (pos == -7).all() and (slot == -7).all()
    assert torch.equal(c.table, table) and torch.equal(c.len, lens) and torch.equal(c.free, free)
    assert torch.equal(c.n_free, n_free)
    assert c.check_error() == code and c.check_error() == abi.SRH_OK
    c.close()


# ---------------------------------------------------------------------------------------------- norm + rotation
def _norm_oracle(x, w, pos, freq, rot, off, style, eps):
    """(value, bound on what the norm and rotation may be off before rounding)."""
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.double()
    mag = y.abs()
    if rot:
        ang = pos.double()[:, None] * freq[None]
        cos, sin = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        i = torch.arange(rot // 2, device=x.device)
        a, b = (off + 2 * i, off + 2 * i + 1) if style == "pairs" else (off + i, off + rot // 2 + i)
        out, m = y.clone(), mag.clone()
        out[..., a] = y[..., a] * cos - y[..., b] * sin
        out[..., b] = y[..., a] * sin + y[..., b] * cos
        m[..., a] = m[..., b] = mag[..., a] + mag[..., b]
        y, mag = out, m
    return y, mag


def _norm_tol(y, mag, d):
    # bf16 output 2^-8; fp32 before it: a sum of d squares in a tree and a chain of 8 (relative (8 + 10) 2^-24 in the
    # sum, half of it in its root), rsqrt 2 ulp, three products, cos and sin within 2^-22 (their argument is a
    # fraction rounded to 2^-24), two products and a sum: under 40 * 2^-24 of the magnitudes
    return 2.0 ** -8 * y.abs() + 2.0 ** -18 * mag


@pytest.mark.parametrize("style", ["pairs", "halves"])
@pytest.mark.parametrize("T,H,Hk,D,rot,off", [(1, 1, 1, 128, 128, 0), (5, 64, 1, 512, 64, 448), (3, 24, 1, 128, 64, 64),
                                              (257, 32, 8, 128, 128, 0), (31, 7, 3, 96, 32, 8), (64, 12, 2, 64, 64, 0),
                                              (700, 5, 1, 256, 256, 0), (2, 3, 2, 80, 80, 0), (9, 2, 1, 8, 0, 0),
                                              (4, 600, 2, 64, 16, 40)])
def test_norm_rope(style, T, H, Hk, D, rot, off):
    g = _gen(T * 7 + D + rot)
    c = _paged(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=1, max_blocks=1)
    row = torch.randn((T, (H + 2 * Hk) * D), generator=g, device="cuda") * torch.exp(
        3 * torch.randn((T, 1), generator=g, device="cuda"))
    row = row.bfloat16()
    q, k = row[:, :H * D].view(T, H, D), row[:, H * D:(H + Hk) * D].view(T, Hk, D)
    kept = row.clone()
    w = 1 + 0.3 * torch.randn(D, generator=g, device="cuda")
    pos = torch.randint(-1000, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 0
    freq = 500000.0 ** (-torch.arange(0, max(rot, 2), 2, device="cuda", dtype=torch.float64) / max(rot, 1))[:rot // 2]
    oq, ok = c.norm_rope(q, k, pos=pos, inv_freq=freq, rot_dim=rot, rot_off=off, style=style, eps=1e-5, q_weight=w)
    for got, x, ww in ((oq, q, w), (ok, k, None)):
        y, mag = _norm_oracle(x, ww, pos, freq, rot, off, style, 1e-5)
        assert ((got.double() - y).abs() <= _norm_tol(y, mag, D)).all()
    assert torch.equal(row, kept) and c.check_error() == 0
    # in place, on a strided row, the same bits
    c.norm_rope(q, None, pos=pos, inv_freq=freq, rot_dim=rot, rot_off=off, style=style, eps=1e-5, q_weight=w, q_out=q)
    assert torch.equal(q, oq) and torch.equal(row[:, H * D:], kept[:, H * D:])
    c.close()


def test_norm_rope_writes_rows_to_slots():
    abi = _abi()
    g = _gen(3)
    c = _paged(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=1, max_blocks=1)
    k = _bf16(g, 6, 2, 128)
    pos, freq = _i32([5, 1, 2, 3, 9, 4]), torch.rand(32, generator=g, device="cuda", dtype=torch.float64)
    kw = dict(pos=pos, inv_freq=freq, rot_dim=64, style="halves")
    _, plain = c.norm_rope(None, k, **kw)
    out = torch.full((8, 2, 128), 3.0, device="cuda").bfloat16()
    slot = torch.tensor([7, 0, -1, 3, -(1 << 40), 2], device="cuda")
    c.norm_rope(None, k, k_out=out, k_slot=slot, **kw)
    want = torch.full_like(out, 3.0)
    for t, s in enumerate(slot.tolist()):
        if s >= 0:
            want[s] = plain[t]
    assert torch.equal(out, want) and c.check_error() == abi.SRH_OK
    slot[1], slot[0] = 8, 1 << 40          # past the end: left out and reported
    out.fill_(3.0)
    c.norm_rope(None, k, k_out=out, k_slot=slot, **kw)
    assert (out[[0, 1, 4, 5, 6, 7]] == 3).all() and torch.equal(out[3], plain[3])
    assert c.check_error() == abi.SRH_ERR_BOUNDS
    c.close()


# ---------------------------------------------------------------------------------------------- append
def _e4m3(v):
    m, e = torch.frexp(v)
    # 2^k from its bits: pow on the GPU is not exact at whole exponents
    step = ((((e - 1).clamp(min=-6) - 3).long() + 1023) << 52).view(torch.float64)
    return torch.round(v / step) * step


class AppendOracle:
    """Values (codes) and scales of a pool, block by block."""

    def __init__(self, codes, scale):
        self.code, self.scale = codes.view(FP8).double().clone(), scale.double().clone()

    def append(self, rows, first, n, table, bs):
        """rows [n, Hk, D] fp64 to positions first .. of the request with blocks `table`."""
        at = 0
        while at < n:
            p = first + at
            blk, o = table[p // bs], p % bs
            m = min(bs - o, n - at)
            x = rows[at:at + m].transpose(0, 1)
            amax = x.abs().amax((1, 2))
            want = torch.full_like(amax, 2.0 ** -64)
            for h in range(amax.numel()):
                a = float(amax[h])
                e = -64
                while e < 64 and a > 448 * 2.0 ** e:
                    e += 1
                want[h] = 2.0 ** e
            if o:
                new = torch.maximum(want, self.scale[blk])
                f = (self.scale[blk] / new)[:, None, None]
                self.code[blk, :, :o] = _e4m3(self.code[blk, :, :o] * f)
                want = new
            self.scale[blk] = want
            self.code[blk, :, o:o + m] = _e4m3((x / want[:, None, None]).clamp(-448, 448))
            at += m


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("B,Hk,D,bs,counts", [
    (1, 1, 128, 16, [[1], [1], [15], [2], [40]]),
    (3, 2, 256, 32, [[5, 0, 70], [1, 1, 1], [27, 31, 0], [1, 1, 1], [1, 64, 33]]),
    (5, 1, 512, 64, [[64, 63, 65, 1, 0], [1, 1, 1, 1, 1], [1, 0, 130, 2, 200]]),
    (40, 4, 128, 16, [[3] * 40, [1] * 40, [1] * 40, [17] * 40]),
    (2, 8, 128, 128, [[300, 1], [129, 500]]),
])
def test_append(shared, B, Hk, D, bs, counts):
    g = _gen(B + D + bs)
    longest = max(sum(c[b] for c in counts) for b in range(B))
    mb = -(-longest // bs)
    c = _paged(batch=B, n_kv_heads=Hk, head_dim=D, block_tokens=bs, n_blocks=B * mb + 2, max_blocks=mb, shared_kv=shared)
    for t in [c.k_codes[0], c.v_codes[0]]:
        t.fill_(NAN_CODE)
    for t in [c.k_scale[0], c.v_scale[0]]:
        t.fill_(float("nan"))
    ora = {p: AppendOracle(torch.zeros_like(t[0]), torch.ones_like(s[0]))
           for p, t, s in (("k", c.k_codes, c.k_scale), ("v", c.v_codes, c.v_scale))}
    ln = [0] * B
    written = torch.zeros((B * mb + 2, bs), dtype=torch.bool)
    for step, n in enumerate(counts):
        T = sum(n)
        first = list(ln)
        ln = [a + b for a, b in zip(ln, n)]
        cu, _, _ = c.resize(_i32(ln), T)
        # rows of growing size, so that begun blocks' scales grow; a padding row behind
        big = torch.exp(2 * torch.randn((T + 2, 1, 1), generator=g, device="cuda") + 2 * step)
        wide = (torch.randn((T + 2, 2 * Hk * D), generator=g, device="cuda").view(T + 2, 2, Hk * D) * big).bfloat16()
        k, v = wide[:, 0].view(T + 2, Hk, D), wide[:, 1].view(T + 2, Hk, D)
        k[T:] = float("nan")
        c.append(k, None if shared else v, cu)
        table, at = c.table.tolist(), 0
        for b in range(B):
            for p, x in (("k", k), ("v", v)):
                if p == "k" or not shared:
                    ora[p].append(x[at:at + n[b]].double(), first[b], n[b], table[b], bs)
            at += n[b]
            for q in range(first[b], ln[b]):
                written[table[b][q // bs], q % bs] = True
        for p, codes, scale in (("k", c.k_codes[0], c.k_scale[0]), ("v", c.v_codes[0], c.v_scale[0])):
            if p == "v" and shared:
                continue
            got = codes.view(FP8).double()
            m = written.cuda()[:, None, :, None].expand_as(got)
            used = written.any(1).cuda()
            # exact: dividing by a power of two rounds nothing, e4m3 rounds to nearest even
            assert torch.equal(scale.double()[used], ora[p].scale[used]), (step, p)
            assert torch.equal(got[m], ora[p].code[m]), (step, p)
            assert (codes[~m] == NAN_CODE).all() and torch.isnan(scale[~used]).all()
    assert c.check_error() == 0
    c.close()


def test_append_again_changes_nothing():
    g = _gen(5)
    c = _paged(batch=2, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=20, max_blocks=8)
    cu, _, _ = c.resize(_i32([20, 9]), 29)
    c.append(_bf16(g, 29, 2, 128), _bf16(g, 29, 2, 128), cu)
    cu, _, _ = c.resize(_i32([50, 12]), 33)
    k, v = _bf16(g, 33, 2, 128) * 9, _bf16(g, 33, 2, 128)
    c.append(k, v, cu)
    held = [t.clone() for t in (c.k_codes[0], c.k_scale[0], c.v_codes[0], c.v_scale[0])]
    c.append(k, v, cu)
    assert all(torch.equal(a, b) for a, b in zip(held, (c.k_codes[0], c.k_scale[0], c.v_codes[0], c.v_scale[0])))
    c.close()


def test_append_extremes_and_reports():
    abi = _abi()
    c = _paged(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=2, max_blocks=2, shared_kv=True)
    cu, _, _ = c.resize(_i32([3]), 3)
    x = torch.zeros((3, 1, 128), device="cuda").bfloat16()
    c.append(x, None, cu)                                   # all zero: the smallest scale, zero codes
    assert float(c.k_scale[0][c.table[0, 0], 0]) == 2.0 ** -64 and c.check_error() == 0
    x[0, 0, :4] = torch.tensor([448.0, -449.0, 2.0 ** -9, 1e-30])
    c.append(x, None, cu)
    blk = int(c.table[0, 0])
    # bf16's step between 256 and 512 is 2, and 449 is a tie: 448 = 224 * 2 is the even side, so 448 * 1 still holds it
    assert float(c.k_scale[0][blk, 0]) == 1.0
    assert c.k_codes[0].view(FP8)[blk, 0, 0, :4].float().tolist() == [448.0, -448.0, 2.0 ** -9, 0.0]
    x[0, 0, 1] = -450.0                                     # the next value does not fit
    c.append(x, None, cu)
    assert float(c.k_scale[0][blk, 0]) == 2.0
    assert c.k_codes[0].view(FP8)[blk, 0, 0, :4].float().tolist() == [224.0, -224.0, 0.0, 0.0]
    x.zero_()
    x[0, 0, 0], x[1, 0, 1], x[2, 0, 2] = float("inf"), float("nan"), 1.0
    c.append(x, None, cu)
    got = c.k_codes[0].view(FP8)[blk, 0, :3, :3].float() * c.k_scale[0][blk, 0]
    assert got.tolist() == [[0, 0, 0], [0, 0, 0], [0, 0, 1]]
    assert c.check_error() == abi.SRH_ERR_RANGE
    x[0, 0, 0] = 3e38
    c.append(x, None, cu)
    assert float(c.k_scale[0][blk, 0]) == 2.0 ** 64 and float(c.k_codes[0].view(FP8)[blk, 0, 0, 0]) == 448.0
    assert c.check_error() == abi.SRH_ERR_RANGE
    c.close()


def test_append_leaves_out_what_is_out_of_bounds():
    abi = _abi()
    g = _gen(8)
    c = _paged(batch=3, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=9, max_blocks=3, shared_kv=True)
    cu, _, _ = c.resize(_i32([20, 20, 20]), 60)
    k = _bf16(g, 60, 1, 128)
    for spoil in ("table", "len", "cu"):
        c.k_codes[0].zero_()
        table, ln, cu2 = c.table.clone(), c.len.clone(), cu.clone()
        if spoil == "table":
            c.table[1] = _i32([9, -1, 5])
        elif spoil == "len":
            c.len[1] = 49
        else:
            cu2[2] = 61
        c.append(k, None, cu2)
        assert c.check_error() == abi.SRH_ERR_BOUNDS
        c.table.copy_(table)
        c.len.copy_(ln)
        touched = (c.k_codes[0].view(9, -1) != 0).any(1)
        for b in ((0, 2) if spoil != "cu" else (0,)):
            assert touched[c.table[b, :2].long()].all()
        assert not touched[c.table[1, :2].long()].any()
    c.close()


# ---------------------------------------------------------------------------------------------- attention
def _filled(lens, Hk, D, bs, shared, seed, gap=0, spread=2, pow2=True):
    """A cache whose requests hold random codes; everything else is NaN codes and NaN scales."""
    g = _gen(seed)
    need = [-(-n // bs) for n in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").tolist()
    mb = max(need + [1]) + 1
    buf, flat = {}, Hk * bs * D
    # gap: K and V of a block side by side with room between
    both = torch.full((total, 2, flat + gap), NAN_CODE, dtype=torch.uint8, device="cuda")
    for i, p in enumerate("kv"):
        if p == "v" and shared:
            continue
        buf[p + "_codes"] = both[:, i, :flat].view(total, Hk, bs, D)
        buf[p + "_scale"] = torch.full((total, Hk), float("nan"), device="cuda")
    c = _paged(batch=len(lens), n_kv_heads=Hk, head_dim=D, block_tokens=bs, n_blocks=total, max_blocks=mb, shared_kv=shared,
               buffers=buf)
    c.len.copy_(_i32(lens))
    at = 0
    for b, n in enumerate(lens):
        ids = order[at:at + need[b]]
        at += need[b]
        if not ids:
            continue
        c.table[b, :need[b]] = _i32(ids)
        for p in "k" if shared else "kv":
            codes, scale = buf[p + "_codes"], buf[p + "_scale"]
            x = torch.randn((need[b], Hk, bs, D), generator=g, device="cuda") * 60
            y = x.clamp(-448, 448).to(FP8).view(torch.uint8)
            t = torch.arange(need[b] * bs, device="cuda").view(need[b], 1, bs, 1) < n
            codes[ids] = torch.where(t, y, torch.full_like(y, NAN_CODE))
            e = torch.randint(-spread, spread + 1, (need[b], Hk), generator=g, device="cuda").float()
            s = torch.exp2(e - 6)
            scale[ids] = s if pow2 else s * (1 + torch.rand(s.shape, generator=g, device="cuda"))
    return c, g


def _check_attend(c, q, cu, out, scale, window):
    """Every value within what the number formats allow.

    Weights are rounded to two e4m3 terms: relative 2^-4 * 2^-4 (and 2^-11 on the way, in fp16), or, for small ones, half of
    the smallest step 2^-9 where the row's largest weight is at least 2^5 (the reference is set 2^5 below the maximum):
    2^-15 of the largest w * vs per code. Queries are two e4m3 terms: exact, or 2^-17 of the row's
    largest times the sum of |K|; scores are fp32 sums of D products and a few fp32 steps on values up to |s|:
    (D + 8) 2^-24 of sum |q K| covers them. Weight errors reach the output through sum w |V| / l. bf16 output: 2^-8."""
    D, Hk, bs = c.D, c.Hk, c.bs
    H = q.shape[1]
    G = H // Hk
    cul, ln = cu.tolist(), c.len.tolist()
    for b in range(len(cul) - 1):
        nq, n = cul[b + 1] - cul[b], ln[b]
        if nq == 0:
            continue
        got = out[cul[b]:cul[b + 1]].double()
        y = q[cul[b]:cul[b + 1]].double().view(nq, Hk, G, D).permute(1, 2, 0, 3)
        if n == 0:
            assert (got == 0).all()
            continue
        ids = c.table[b, :-(-n // bs)].long()
        kc, vc = (t[0][ids].view(FP8).double().permute(1, 0, 2, 3).reshape(Hk, -1, D)[:, :n] for t in (c.k_codes, c.v_codes))
        ks, vs = (t[0][ids].double().t().repeat_interleave(bs, 1)[:, :n] for t in (c.k_scale, c.v_scale))
        k, v = kc * ks[..., None], vc * vs[..., None]
        s = torch.einsum("hgid,htd->hgit", y, k) * scale
        s_abs = torch.einsum("hgid,htd->hgit", y.abs(), k.abs()) * abs(scale)
        k_sum = k.abs().sum(-1)[:, None, None, :] * abs(scale)
        pos = torch.arange(n - nq, n, device="cuda")[:, None]
        t = torch.arange(n, device="cuda")[None]
        see = (t <= pos) & ((t > pos - window) if window else torch.ones_like(t, dtype=torch.bool))
        s = s.masked_fill(~see, float("-inf"))
        m = s.amax(-1, keepdim=True)
        w = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
        l = w.sum(-1, keepdim=True)
        ok = l > 0
        w = torch.where(ok, w / l, 0.0)
        want = torch.einsum("hgit,htd->hgid", w, v)
        eps_s = (D + 8) * 2.0 ** -24 * s_abs + 2.0 ** -17 * y.abs().amax(-1)[..., None] * k_sum
        rel = 2.0 ** -8 + 2.0 ** -11 + 2 * (eps_s * see).amax(-1, keepdim=True)
        contrib = (w * vs[:, None, None, :]).amax(-1, keepdim=True)
        tol = rel * torch.einsum("hgit,htd->hgid", w, v.abs())
        tol += 2.0 ** -15 * contrib * torch.einsum("hgit,htd->hgid", see.double().expand_as(w), vc.abs())
        tol += 2.0 ** -8 * want.abs()
        want, tol = (z.permute(2, 0, 1, 3).reshape(nq, H, D) for z in (want, tol))
        bad = ~((got - want).abs() <= tol)
        assert not bad.any(), (b, int(bad.sum()), float((got - want).abs().max()), float(want.abs().max()))


def _attend(lens, nq, H, Hk, D, bs, shared, window=0, seed=0, pad=0, scale=None, **kw):
    c, g = _filled(lens, Hk, D, bs, shared, seed, **kw)
    cu = _i32(np.concatenate([[0], np.cumsum(nq)]).tolist())
    T = sum(nq) + pad
    q = torch.randn((T, H, D), generator=g, device="cuda")
    q = (q * torch.exp(torch.randn((T, H, 1), generator=g, device="cuda"))).bfloat16()
    out = torch.full((T, H, D), 7.0, device="cuda").bfloat16()
    scale = D ** -0.5 / 4 if scale is None else scale
    c.attend(q, cu, scale=scale, window=window, out=out)
    assert c.check_error() == 0
    _check_attend(c, q, cu, out, scale, window)
    assert (out[sum(nq):] == 7).all()
    c.close()


@pytest.mark.parametrize("D,shared", [(128, False), (128, True), (256, False), (256, True), (512, True), (512, False)])
@pytest.mark.parametrize("G", [1, 16, 17, 40])
def test_attend_one_tile(D, shared, G):
    _attend([100], [1], G, 1, D, 16, shared, seed=D + G)


@pytest.mark.parametrize("D,shared", [(128, False), (256, False), (512, True), (128, True), (512, False)])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_attend_decode_lengths(D, shared, bs):
    lens = [1, 2, 15, 16, 17, 127, 128, 129, 255, 0, 1000, 3001, bs, bs + 1, 640]
    _attend(lens, [1] * len(lens), 8, 2, D, bs, shared, seed=bs + D, pad=2)


@pytest.mark.parametrize("H,Hk,D,shared,bs", [(8, 1, 128, False, 16), (6, 2, 128, False, 32), (64, 1, 512, True, 64),
                                              (16, 4, 256, False, 128), (65, 1, 128, True, 16), (5, 5, 256, True, 64),
                                              (128, 1, 512, True, 64), (64, 2, 512, False, 32)])
def test_attend_several_queries(H, Hk, D, shared, bs):
    lens = [1, 40, 128, 130, 300, 1111, 7, 64, 513]
    nq = [1, 4, 128, 5, 0, 3, 7, 2, 130]
    _attend(lens, nq, H, Hk, D, bs, shared, seed=H, pad=1)


@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 1000])
@pytest.mark.parametrize("D,shared,q", [(128, False, 1), (128, False, 150), (512, True, 3), (256, True, 40)])
def test_attend_window(window, D, shared, q):
    lens = [q, q + 1, 128 + q, 700, 2049 + q]
    _attend(lens, [min(q, n) for n in lens], 8, 2, D, 32, shared, window=window, seed=window)


@pytest.mark.parametrize("D,shared", [(128, False), (512, True)])
def test_attend_one_long_request_is_split_and_joined(D, shared):
    _attend([50001], [1], 16, 1, D, 64, shared, seed=1)
    _attend([9000, 1, 0, 20000], [2, 1, 1, 5], 8, 1, D, 64, shared, seed=2)


def test_attend_rows_before_the_request_see_nothing():
    # more queries than tokens: the first rows lie before the request
    _attend([3, 0, 129], [5, 2, 140], 8, 2, 128, 16, False, seed=4)
    _attend([3, 0, 129], [5, 2, 140], 64, 1, 512, 16, True, seed=4, window=7)


@pytest.mark.parametrize("D,shared", [(128, False), (256, False), (512, True)])
def test_attend_scales_far_apart_and_strided_blocks(D, shared):
    # scales are not powers of two here, and blocks' contributions differ by up to 2^40
    _attend([700, 33, 1500], [1, 2, 3], 8, 2, D, 32, shared, seed=9, spread=20, pow2=False, gap=48,
            scale=2.0 ** -14)


@pytest.mark.parametrize("D,shared", [(128, False), (512, True)])
def test_attend_peaked_and_flat_scores(D, shared):
    _attend([1000, 300], [1, 4], 16, 2, D, 16, shared, seed=11, scale=2.0)     # one token takes all
    _attend([1000, 300], [1, 4], 16, 2, D, 16, shared, seed=12, scale=0.0)     # a plain mean
    _attend([1000, 300], [1, 4], 16, 2, D, 16, shared, seed=13, scale=-0.02)


def test_attend_rising_scores_move_the_reference():
    # keys grow along the request, so every tile raises the maximum
    c, g = _filled([2000], 1, 128, 16, False, 21, spread=0)
    ids = c.table[0, :125].long()
    c.k_codes[0][ids] = torch.full((125, 1, 16, 128), 8.0, device="cuda").to(FP8).view(torch.uint8)
    c.k_scale[0][ids] = (torch.arange(125, device="cuda").float()[:, None] + 1) / 64
    q = torch.ones((1, 3, 128), device="cuda").bfloat16() * _i32([1, -1, 3]).bfloat16()[None, :, None]
    cu = _i32([0, 1])
    out = c.attend(q, cu, scale=128 ** -0.5)
    assert c.check_error() == 0
    _check_attend(c, q, cu, out, 128 ** -0.5, 0)
    c.close()


def test_attend_bad_rows_stay_alone():
    """Queries that are not finite give NaN in their rows only."""
    c, g = _filled([300, 200], 2, 128, 16, False, 31)
    q = _bf16(g, 5, 8, 128)
    cu = _i32([0, 3, 5])
    clean = c.attend(q, cu, scale=0.05)
    q2 = q.clone()
    q2[1, 2, 5], q2[3, 7, 0] = float("nan"), float("inf")
    out = c.attend(q2, cu, scale=0.05)
    assert torch.isnan(out[1, 2]).all() and torch.isnan(out[3, 7]).all()
    keep = torch.ones((5, 8), dtype=torch.bool, device="cuda")
    keep[1, 2] = keep[3, 7] = False
    assert torch.equal(out[keep], clean[keep])
    c.close()


def test_attend_reports_bad_tables_and_lengths():
    abi = _abi()
    c, g = _filled([300, 200], 1, 128, 16, True, 41)
    q, cu = _bf16(g, 2, 4, 128), _i32([0, 1, 2])
    good = c.attend(q, cu, scale=0.05)
    table = c.table.clone()
    c.table[0, 3], c.table[0, 5] = c.n_blocks, -2          # blocks that are not there: read as absent
    out = c.attend(q, cu, scale=0.05)
    assert c.check_error() == abi.SRH_ERR_BOUNDS
    assert torch.isfinite(out).all() and torch.equal(out[1], good[1]) and not torch.equal(out[0], good[0])
    c.table.copy_(table)
    c.len[0] = 1 << 30
    out = c.attend(q, cu, scale=0.05)
    assert c.check_error() == abi.SRH_ERR_BOUNDS and torch.equal(out[1], good[1])
    c.len[0] = 300
    out = c.attend(q, _i32([0, 1, 9]), scale=0.05)
    assert c.check_error() == abi.SRH_ERR_BOUNDS and torch.equal(out, good)
    out = torch.full_like(q, 5.0)
    c.attend(q, _i32([-4, 1, 2]), scale=0.05, out=out)
    assert c.check_error() == abi.SRH_ERR_BOUNDS and torch.equal(out, good)
    c.close()


def test_attend_repeats_bit_for_bit_on_streams_and_in_graphs():
    c, g = _filled([5000, 77, 1300], 2, 128, 32, False, 51)
    q, cu = _bf16(g, 6, 16, 128), _i32([0, 1, 4, 6])
    want = c.attend(q, cu, scale=0.08)
    torch.cuda.synchronize()
    for _ in range(3):
        assert torch.equal(c.attend(q, cu, scale=0.08), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = torch.zeros_like(q)
    c.attend(q, cu, scale=0.08, out=a, stream=s)
    s.synchronize()
    assert torch.equal(a, want)
    # captured: other lengths and queries, same graph
    out, graph = torch.zeros_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.attend(q, cu, scale=0.08, out=out)
    for ln in ([5000, 77, 1300], [4999, 12, 640]):
        c.len.copy_(_i32(ln))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _check_attend(c, q, cu, out, 0.08, 0)
    assert c.check_error() == 0
    c.close()


# ---------------------------------------------------------------------------------------------- together
@pytest.mark.parametrize("H,Hk,D,shared,rot,off,style", [(8, 2, 128, False, 128, 0, "halves"),
                                                         (64, 1, 512, True, 64, 448, "pairs")])
def test_a_serving_loop(H, Hk, D, shared, rot, off, style):
    """Prompts, decode steps with drafted tokens and their rejection, requests that
    end and start, two layers on one table: the attention agrees with the plain
    one over the values that the cache should hold."""
    rng = np.random.default_rng(7)
    g = _gen(7)
    B, bs, mb, layers = 5, 32, 24, 2
    c = _paged(batch=B, n_kv_heads=Hk, head_dim=D, block_tokens=bs, n_blocks=70, max_blocks=mb, shared_kv=shared,
               layers=layers)
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    ora = [{p: AppendOracle(t[i], s[i]) for p, t, s in (("k", c.k_codes, c.k_scale), ("v", c.v_codes, c.v_scale))}
           for i in range(layers)]
    ln = [0] * B
    for step in range(9):
        if step == 0:
            new = [200, 33, 1, 150, 64]
        elif step % 3 == 2:
            new = [max(1, n - int(rng.integers(0, 4))) for n in ln]       # drafted tokens rejected
        else:
            new = [n + int(rng.integers(1, 5)) for n in ln]
        if step == 4:
            new[1] = 0                                                    # a request ends ...
        if step == 5:
            new[1] = 300                                                  # ... and another takes its place
        T = sum(max(0, a - b) for a, b in zip(new, ln))
        cu, pos, slot = c.resize(_i32(new), T)
        if not T:
            ln = new
            continue
        qkv = _bf16(g, T, (H + 2 * Hk) * D)
        q, k = c.norm_rope(qkv[:, :H * D].view(T, H, D), qkv[:, H * D:(H + Hk) * D].view(T, Hk, D), pos=pos, inv_freq=freq,
                           rot_dim=rot, rot_off=off, style=style, q_weight=w, k_weight=w)
        want, mag = _norm_oracle(qkv[:, H * D:(H + Hk) * D].view(T, Hk, D), w, pos, freq, rot, off, style, 1e-6)
        assert ((k.double() - want).abs() <= _norm_tol(want, mag, D)).all()
        v = qkv[:, (H + Hk) * D:].view(T, Hk, D)
        cul, table = cu.tolist(), c.table.tolist()
        for layer in range(layers):
            kk, vv = (k, v) if layer == 0 else (-k, v * 2)
            c.append(kk, None if shared else vv, cu, layer=layer)
            out = c.attend(q, cu, scale=D ** -0.5, layer=layer)
            for b in range(B):
                n = cul[b + 1] - cul[b]
                for p, x in (("k", kk), ("v", vv)):
                    if p == "k" or not shared:
                        ora[layer][p].append(x[cul[b]:cul[b + 1]].double(), new[b] - n, n, table[b], bs)
            for p, codes, scale in (("k", c.k_codes, c.k_scale), ("v", c.v_codes, c.v_scale)):
                if p == "v" and shared:
                    continue
                for b in range(B):
                    for j in range(-(-new[b] // bs)):
                        m = min(bs, new[b] - j * bs)
                        assert torch.equal(scale[layer][table[b][j]].double(), ora[layer][p].scale[table[b][j]])
                        assert torch.equal(codes[layer][table[b][j]][:, :m].view(FP8).double(),
                                           ora[layer][p].code[table[b][j]][:, :m])
            one = type("OneLayer", (), dict(D=D, Hk=Hk, bs=bs, len=c.len, table=c.table,
                                            k_codes=[c.k_codes[layer]], v_codes=[c.v_codes[layer]],
                                            k_scale=[c.k_scale[layer]], v_scale=[c.v_scale[layer]]))
            _check_attend(one, q, cu, out, D ** -0.5, 0)
        ln = new
        assert c.check_error() == 0
    c.close()


def test_a_captured_step():
    """resize, append and attend in one CUDA graph, replayed with new lengths."""
    g = _gen(77)
    c = _paged(batch=4, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=80, max_blocks=20)
    cu, _, _ = c.resize(_i32([100, 3, 40, 250]), 393)
    c.append(_bf16(g, 393, 2, 128), _bf16(g, 393, 2, 128), cu)
    new = c.len + 1
    cu, pos, slot = _i32([0] * 5), _i32([0] * 4), torch.zeros(4, dtype=torch.int64, device="cuda")
    k, v, q = _bf16(g, 4, 2, 128), _bf16(g, 4, 2, 128), _bf16(g, 4, 8, 128)
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.resize(new, 4, out=(cu, pos, slot))
        c.append(k, v, cu)
        c.attend(q, cu, scale=0.09, out=out)
    for step in range(20):
        for t in (k, v, q):
            t.copy_(_bf16(g, *t.shape))
        new.copy_(c.len + 1)
        graph.replay()
        assert pos.tolist() == (new - 1).tolist() and cu.tolist() == [0, 1, 2, 3, 4]
        _check_attend(c, q, cu, out, 0.09, 0)
    assert c.len.tolist() == [120, 23, 60, 270] and c.check_error() == 0
    c.close()


# ---------------------------------------------------------------------------------------------- further shapes and uses
@pytest.mark.parametrize("n_req", [33, 200, 1500])
def test_attend_many_requests(n_req):
    rng = np.random.default_rng(n_req)
    lens = rng.integers(0, 90, n_req)
    nq = np.minimum(rng.integers(0, 4, n_req), lens)
    _attend(lens.tolist(), nq.tolist(), 4, 2, 128, 16, False, seed=n_req, pad=1)


@pytest.mark.parametrize("D,shared,G,q", [(128, False, 3, 700), (512, True, 64, 9), (512, False, 5, 90), (256, False, 33, 20),
                                          (256, True, 1, 1000), (128, True, 100, 7)])
@pytest.mark.parametrize("window", [0, 300, 2 ** 31 - 1])
def test_attend_many_row_tiles(D, shared, G, q, window):
    _attend([q + 5, 2 * q, 130, q // 2], [q, q, 1, q // 2 + 3], G, 1, D, 32, shared, window=window, seed=G, pad=3)


def test_attend_rows_that_come_into_sight_late():
    """Windows of one row tile that begin in different tiles: a row's reference is
    set by a tile that is not the segment's first."""
    _attend([1200], [600], 1, 1, 128, 16, False, window=40, seed=5)
    _attend([1200], [60], 8, 1, 256, 16, True, window=3, seed=6)


def test_attend_strided_queries_and_outputs():
    c, g = _filled([300, 77], 2, 128, 16, False, 61)
    row = _bf16(g, 5, 3, 8, 128)                           # queries between other things, outputs too
    q, cu = row[:, 1], _i32([0, 3, 5])
    want = c.attend(q.contiguous(), cu, scale=0.06)
    out = torch.full((5, 2, 8, 128), 9.0, device="cuda").bfloat16()
    c.attend(q, cu, scale=0.06, out=out[:, 1])
    assert torch.equal(out[:, 1], want) and (out[:, 0] == 9).all()
    one = row[:1, 1].expand(5, 8, 128)                     # the same query five times, without copies
    assert torch.equal(c.attend(one, cu, scale=0.06), c.attend(one.contiguous(), cu, scale=0.06))
    bits = q.contiguous().view(torch.int16)                # bit patterns, as DecodeStep holds them
    assert torch.equal(c.attend(bits, cu, scale=0.06).view(torch.bfloat16), want)
    c.close()


def test_two_caches_on_two_streams():
    a, ga = _filled([4000, 900], 2, 128, 16, False, 71)
    b, gb = _filled([3000, 50, 700], 1, 512, 64, True, 72)
    qa, qb = _bf16(ga, 2, 16, 128), _bf16(gb, 3, 64, 512)
    ca, cb = _i32([0, 1, 2]), _i32([0, 1, 2, 3])
    wa, wb = a.attend(qa, ca, scale=0.08), b.attend(qb, cb, scale=0.03)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(20):
        outs.append((a.attend(qa, ca, scale=0.08, stream=sa), b.attend(qb, cb, scale=0.03, stream=sb.cuda_stream)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, wa) and torch.equal(y, wb) for x, y in outs)
    a.close()
    b.close()


def test_block_table_order_does_not_show():
    """The same rows in other blocks give the same bits."""
    c, g = _filled([500, 260], 2, 128, 16, False, 81)
    q, cu = _bf16(g, 3, 8, 128), _i32([0, 1, 3])
    want = c.attend(q, cu, scale=0.07)
    perm = torch.randperm(c.n_blocks, generator=g, device="cuda")
    for t in (c.k_codes[0], c.v_codes[0], c.k_scale[0], c.v_scale[0]):
        t[perm] = t.clone()
    c.table.copy_(torch.where(c.table >= 0, perm[c.table.clamp(min=0).long()].int(), c.table))
    assert torch.equal(c.attend(q, cu, scale=0.07), want)
    c.close()


def test_refusals():
    abi = _abi()
    c = _paged(batch=2, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=8, max_blocks=4)
    s = _paged(batch=2, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=8, max_blocks=4, shared_kv=True)
    g = _gen(1)
    q, k, cu = _bf16(g, 3, 4, 128), _bf16(g, 3, 2, 128), _i32([0, 1, 3])
    freq, pos = torch.ones(16, dtype=torch.float64, device="cuda"), _i32([1, 2, 3])
    value = [lambda: c.attend(q[:, :, ::2], cu, scale=1.0), lambda: c.attend(q.float(), cu, scale=1.0),
             lambda: c.attend(q, cu.long(), scale=1.0), lambda: c.attend(q, _i32([0]), scale=1.0),
             lambda: c.attend(q, _i32([0, 1, 2, 3]), scale=1.0), lambda: c.attend(q.cpu(), cu, scale=1.0),
             lambda: c.attend(q, cu, scale=1.0, out=q[:2]), lambda: c.append(k, None, cu), lambda: s.append(k, k, cu),
             lambda: c.append(k, k[:2], cu), lambda: c.append(q, q, cu), lambda: c.resize(_i32([1, 2, 3])),
             lambda: c.resize(_i32([1, 2]), -1), lambda: c.norm_rope(q, style="spiral"), lambda: c.norm_rope(),
             lambda: c.norm_rope(q, k[:2]), lambda: c.norm_rope(q, pos=pos, inv_freq=freq, rot_dim=64),
             lambda: c.norm_rope(q, q_slot=pos.long()), lambda: c.norm_rope(q, q_weight=freq)]
    for f in value:
        with pytest.raises(ValueError):
            f()
    code = [lambda: c.attend(_bf16(g, 3, 3, 128), cu, scale=1.0), lambda: c.attend(q, cu, scale=float("nan")),
            lambda: c.attend(q, cu, scale=1.0, window=-1), lambda: c.attend(q, cu, scale=1.0, out=q),
            lambda: c.norm_rope(q, pos=pos, inv_freq=freq[:12], rot_dim=24), lambda: c.norm_rope(q, eps=-1.0),
            lambda: c.norm_rope(q, pos=pos, inv_freq=freq, rot_dim=32, rot_off=100),
            lambda: c.norm_rope(_bf16(g, 3, 4, 20)), lambda: c.norm_rope(_bf16(g, 3, 1, 520)),
            lambda: c.norm_rope(q, q_out=q, q_slot=pos.long()),
            lambda: c.attend(_bf16(g, 3, 4 * 128 + 4)[:, 4:].view(3, 4, 128), cu, scale=1.0)]
    for f in code:
        with pytest.raises(abi.SrhError) as ei:
            f()
        assert ei.value.code == abi.SRH_ERR_INVALID and str(ei.value)
    assert c.check_error() == 0
    # nothing to do is no error
    empty = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    assert c.attend(empty, cu, scale=1.0).shape == empty.shape
    c.append(empty[:, :2], empty[:, :2], cu)
    c.norm_rope(empty)
    c.close()
    s.close()
    c.close()


def test_blocks_past_four_gigabytes():
    """Blocks whose codes lie beyond 32-bit offsets: written, read back, attended."""
    n_blocks, Hk, bs = 34000, 8, 128                       # 131,072 bytes a block
    c = _paged(batch=2, n_kv_heads=Hk, head_dim=128, block_tokens=bs, n_blocks=n_blocks, max_blocks=40, shared_kv=True)
    g = _gen(91)
    c.free.copy_(torch.arange(n_blocks, dtype=torch.int32, device="cuda"))       # the last block on top
    cu, _, slot = c.resize(_i32([700, 300]), 1000)
    assert int(c.table[0, 0]) == n_blocks - 1 and int(slot.max()) >= n_blocks * bs - bs
    k = _bf16(g, 1000, Hk, 128)
    c.append(k, None, cu)
    ids = c.table[0, :6].long()
    got = (c.k_codes[0][ids].view(FP8).float() * c.k_scale[0][ids][:, :, None, None]).transpose(1, 2).reshape(-1, Hk, 128)[:700]
    # e4m3 after a power of two: 2^-4 of the value, or half of 2^-9 steps of the block's scale
    tol = 2.0 ** -4 * k[:700].float().abs() + 2.0 ** -10 * float(c.k_scale[0][ids].max())
    assert ((got - k[:700].float()).abs() <= tol).all()
    q, cq = _bf16(g, 3, 16, 128), _i32([0, 1, 3])
    out = c.attend(q, cq, scale=0.08)
    assert c.check_error() == 0
    _check_attend(c, q, cq, out, 0.08, 0)
    c.close()


def test_attend_chunks_taken_as_ctas_come_free():
    """Enough work that chunks are handed out while the kernel runs: the same bits
    every time, and the formula's values."""
    c, g = _filled([30000 + 77 * b for b in range(12)], 16, 128, 128, True, 95, spread=0)
    q, cu = _bf16(g, 12, 32, 128), _i32(list(range(13)))
    want = c.attend(q, cu, scale=0.01)
    for _ in range(4):
        assert torch.equal(c.attend(q, cu, scale=0.01), want)
    one = type("Some", (), dict(D=128, Hk=16, bs=128, len=c.len[[0, 11]], table=c.table[[0, 11]], k_codes=c.k_codes,
                                v_codes=c.v_codes, k_scale=c.k_scale, v_scale=c.v_scale))
    _check_attend(one, q[[0, 11]], _i32([0, 1, 2]), want[[0, 11]], 0.01, 0)
    assert c.check_error() == 0
    c.close()


def test_attend_scales_of_zero():
    """A block of zeros with a scale of 0: its tokens still take part in the softmax."""
    c, g = _filled([64, 40], 1, 128, 16, False, 97, spread=0)
    blk = int(c.table[0, 1])
    c.v_scale[0][blk] = 0
    c.v_codes[0][blk] = 0
    c.k_scale[0][int(c.table[1, 0])] = 0
    q, cu = _bf16(g, 2, 4, 128), _i32([0, 1, 2])
    out = c.attend(q, cu, scale=0.02)
    _check_attend(c, q, cu, out, 0.02, 0)
    c.close()


def test_pools_whose_blocks_overlap_are_refused():
    """A pool of repeated blocks (stride 0) or of overlapping ones: writes would meet, or leave the tensor."""
    flat = torch.zeros(4 * 16 * 128, dtype=torch.uint8, device="cuda")
    for stride in (0, 16, 16 * 128 - 16):
        t = flat.as_strided((4, 1, 16, 128), (stride, 16 * 128, 128, 1))
        with pytest.raises(ValueError, match="overlap"):
            _paged(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=4, max_blocks=4, shared_kv=True,
                   buffers={"k_codes": t})


@pytest.mark.parametrize("D,H,Hk,T", [(128, 5, 3, 7001), (64, 3, 0, 9000), (512, 3, 1, 2500), (256, 1, 1, 6000), (24, 1, 2, 11000)])
def test_norm_ranges_cross_tokens(D, H, Hk, T):
    """Warps whose heads belong to several tokens and to both kinds, begin and end inside one, with tokens left out."""
    g = _gen(101 + D)
    c = _paged(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=1, max_blocks=1)
    q, k = _bf16(g, T, H, D), _bf16(g, T, max(Hk, 1), D)
    w = torch.randn(D, generator=g, device="cuda")
    rot = 16 * (D // 32)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda").int()
    freq = 10000.0 ** (-torch.arange(rot // 2, device="cuda").double() / max(rot // 2, 1))
    slot = torch.arange(T, device="cuda")
    slot[::3] = -1
    k_out = torch.full((T, max(Hk, 1), D), 7.0, dtype=torch.bfloat16, device="cuda")
    kw = dict(pos=pos, inv_freq=freq, rot_dim=rot, rot_off=8 if D > 16 else 0, style="halves", eps=1e-5, q_weight=w)
    if Hk:
        kw.update(k_out=k_out, k_slot=slot)
    qo, _ = c.norm_rope(q, k if Hk else None, **kw)
    args = (pos, freq, rot, kw["rot_off"], "halves", 1e-5)
    want, mag = _norm_oracle(q, w, *args)
    assert ((qo.double() - want).abs() <= _norm_tol(want, mag, D)).all()
    if Hk:
        want, mag = _norm_oracle(k, None, *args)
        on = slot >= 0
        assert ((k_out.double() - want).abs() <= _norm_tol(want, mag, D))[on].all()
        assert (k_out[~on] == 7).all()
    assert c.check_error() == 0
    c.close()


def test_rotation_without_positions_is_refused():
    g = _gen(111)
    c = _paged(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=1, max_blocks=1)
    q, pos, freq = _bf16(g, 3, 2, 128), _i32([0, 1, 2]), torch.ones(16, dtype=torch.float64, device="cuda")
    for kw in ({}, {"pos": pos}, {"inv_freq": freq}):
        with pytest.raises(ValueError, match="rot_dim needs"):
            c.norm_rope(q, rot_dim=32, **kw)
    c.close()


def test_attend_prompt_in_rounds():
    """A prompt of so many units (2,000 row tiles of 4 KV heads) that the last quarter is handed out while the kernel runs."""
    c, g = _filled([4000], 4, 128, 64, True, 113, spread=1)
    q, cu = _bf16(g, 4000, 64, 128), _i32([0, 4000])
    want = c.attend(q, cu, scale=0.02)
    for _ in range(3):
        assert torch.equal(c.attend(q, cu, scale=0.02), want)
    for at in (2, 777, 2001, 4000):                        # the last two rows that see `at` tokens
        part = type("Some", (), dict(D=128, Hk=4, bs=64, len=_i32([at]), table=c.table, k_codes=c.k_codes, v_codes=c.v_codes,
                                     k_scale=c.k_scale, v_scale=c.v_scale))
        _check_attend(part, q[at - 2:at], _i32([0, 2]), want[at - 2:at], 0.02, 0)
    assert c.check_error() == 0
    c.close()


# ---------------------------------------------------------------------------------------------- rows with a long tail
def _tail(n, D, shared, G, depth, sd, bs=64, batch=1, outlier=0):
    """`batch` requests over the same n tokens: the first takes about exp(depth) times the weight of another one, whose scores
    spread by sd. Rows differ in how far. With `outlier`, a block's V scale is 2^outlier larger and its codes are 0 in the
    upper half of the dims."""
    from types import SimpleNamespace
    g = _gen(n + D + G)
    nb = -(-n // bs)
    rows = torch.randn((nb * bs, D), generator=g, device="cuda") * 0.3 + 1
    key = rows if shared else torch.randn((nb * bs, D), generator=g, device="cuda")
    key[:, 0] = sd * torch.randn(nb * bs, generator=g, device="cuda")
    rows[0] = 0
    key[0, 0] = depth
    scale = torch.ones((nb, 1), device="cuda")
    kc = key.to(FP8).view(torch.uint8).view(nb, 1, bs, D)
    vc = kc if shared else rows.to(FP8).view(torch.uint8).view(nb, 1, bs, D)
    vs = scale if shared else scale.clone()
    if outlier:
        at = nb // 2
        vs[at] = 2.0 ** outlier
        vc[at, :, :, D // 2:] = 0
    buf = dict(k_codes=kc, k_scale=scale, v_codes=vc, v_scale=vs) if not shared else dict(k_codes=kc, k_scale=scale)
    c = _paged(batch=batch, n_kv_heads=1, head_dim=D, block_tokens=bs, n_blocks=nb, max_blocks=nb, shared_kv=shared, buffers=buf)
    c.table.copy_(torch.arange(nb, device="cuda").int().expand(batch, nb))
    c.len.fill_(n)
    q = torch.zeros((G, D), device="cuda")
    q[:, 0] = 0.9 + 0.3 * torch.arange(G, device="cuda") / G
    q = q.bfloat16()
    # the formula in 64 bits
    k = kc.view(FP8).double().view(-1, D)[:n]
    v = vc.view(FP8).double().view(-1, D)[:n]
    w = torch.softmax(q.double() @ k.t(), -1)
    f = vs.double().repeat_interleave(bs)[:n]
    want, mag = (w * f) @ v, (w * f) @ v.abs()
    # Weights: fp16 (2^-11), then three terms, of which the last is rounded at 2^-9; scores here are one product of at most
    # 16, in fp32 (2^-24 * 16 and as much again for the steps behind it, and 2^-22 of the exponential): under 2^-11 with
    # fp16's. Steps of 2^-16 where the row's largest contribution is at least 2^10: 2^-27 of it per code. Sums of n / 32 steps
    # for each of three terms, 2^-23 each (they may truncate). bf16 output: 2^-8.
    tol = (2.0 ** -9 + 2 * 2.0 ** -11 + 3 * n / 32 * 2.0 ** -23) * mag + 2.0 ** -8 * want.abs()
    tol += 2.0 ** -27 * (w * f).amax(-1, keepdim=True) * v.abs().sum(0)
    return SimpleNamespace(c=c, q=q, want=want, tol=tol, mag=mag)


@pytest.mark.parametrize("D,shared,G", [(128, False, 8), (128, True, 32), (256, False, 4), (256, True, 24), (256, False, 64),
                                        (512, True, 64), (512, True, 16), (512, False, 32)])
@pytest.mark.parametrize("n,depth,sd", [(8192, 11.0, 0.0), (32768, 10.0, 0.0), (32768, 10.0, 0.3), (32768, 11.0, 1.0),
                                        (131072, 12.0, 0.3)])
def test_attend_keeps_the_tail_behind_one_large_weight(D, shared, G, n, depth, sd):
    """A first token with a large part of the weight (an attention sink) over a long flat tail, alone (cut into many parts)
    and in a batch (whole requests to a CTA): the tail's weights are far below the largest and count together."""
    got = []
    for batch in (1, 320):
        t = _tail(n, D, shared, G, depth, sd, batch=batch)
        out = t.c.attend(t.q.expand(batch, G, D), _i32(list(range(batch + 1))), scale=1.0).double()
        assert t.c.check_error() == 0
        bad = ~((out - t.want).abs() <= t.tol)
        assert not bad.any(), (batch, float(((out - t.want).abs() / t.mag).nan_to_num().max()))
        got.append(out[-1])
        t.c.close()
    assert ((got[0] - got[1]).abs() <= 2 * t.tol).all()


@pytest.mark.parametrize("D,G", [(128, 8), (128, 32), (256, 64), (512, 64), (512, 16)])
@pytest.mark.parametrize("outlier", [11, 15])
def test_attend_keeps_what_stands_beside_a_block_of_large_values(D, G, outlier):
    t = _tail(4096, D, False, G, 2.0, 1.0, outlier=outlier)
    out = t.c.attend(t.q[None], _i32([0, 1]), scale=1.0)[0].double()
    assert t.c.check_error() == 0
    assert ((out - t.want).abs() <= t.tol).all()
    # (the bound says something there: 2^-8 + 2^-9 + 2^-10, and 2^-27 * 2^15 of a weight of at most about e^4.3 times the mean,
    # for each of the tokens: under 2^-12 * 75, 2.6 % in all)
    assert (t.tol[:, D // 2:] < 0.03 * t.want[:, D // 2:].abs()).all()
    t.c.close()


def test_a_cache_made_beside_a_busy_default_stream():
    """The handle's own clears are over when it is there: its first call on a stream that does not wait for the default one
    finds them done."""
    c, g = _filled([5000, 77], 2, 128, 32, False, 121)
    q, cu2 = _bf16(g, 2, 16, 128), _i32([0, 1, 2])
    want = c.attend(q, cu2, scale=0.08)
    x = torch.randn((8192, 8192), device="cuda").bfloat16()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(40):                                     # some 25 ms
        y = x @ x
    busy = torch.cuda.Event()
    busy.record()
    buf = dict(k_codes=c.k_codes[0], k_scale=c.k_scale[0], v_codes=c.v_codes[0], v_scale=c.v_scale[0], table=c.table, len=c.len,
               free=c.free, n_free=c.n_free)
    with torch.cuda.stream(side):
        d = _paged(batch=2, n_kv_heads=2, head_dim=128, block_tokens=32, n_blocks=c.n_blocks, max_blocks=c.max_blocks, buffers=buf)
        assert busy.query()                                 # the clears come behind that work, and creation waits for them
        out = d.attend(q, cu2, scale=0.08)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and d.check_error() == 0 and y.shape == x.shape
    d.close()
    c.close()


@pytest.mark.parametrize("room", [40, 5000])               # one CTA, and a grid of its own
def test_slots_behind_the_last_token_name_no_row(room):
    """Arrays with room for more tokens than there are, used again and again as in a captured step: rows that are padding
    go nowhere, after a refused call too."""
    abi = _abi()
    g = _gen(131)
    c = _paged(batch=3, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=400, max_blocks=400)
    x, pos0 = _bf16(g, room, 1, 128), torch.zeros(room, dtype=torch.int32, device="cuda")
    held = torch.full((400 * 16, 1, 128), 5.0, device="cuda").bfloat16()
    out = (_i32([0] * 4), pos0, torch.full((room,), 3, dtype=torch.int64, device="cuda"))      # as memory used before
    for new, n in (([30, 4, 0], 34), ([31, 5, 1], 3), ([31, 5, 1], 0), ([room, 5, 1], room - 31), ([-1, 9, 9], 0),
                   ([32 + room, 5, 1], 32), ([0, 0, 0], 0)):
        cu, pos, slot = c.resize(_i32(new), room, out=out)
        code = abi.SRH_ERR_BOUNDS if new[0] < 0 else abi.SRH_OK
        assert c.check_error() == code and int(cu[3]) == n
        assert (slot[n:] == -1).all() and (slot[:n] >= 0).all()
        held.fill_(5.0)
        c.norm_rope(x, q_out=held, q_slot=slot)
        rows = torch.zeros(400 * 16, dtype=torch.bool, device="cuda")
        rows[slot[:n]] = True
        assert (held[~rows] == 5).all() and c.check_error() == abi.SRH_OK
    # refused for its cap: the slots of the call before name nothing either
    c.resize(_i32([20, 0, 0]), room, out=out)
    c.resize(_i32([20 + room + 1, 0, 0]), room, out=out)
    assert c.check_error() == abi.SRH_ERR_BOUNDS and (out[2] == -1).all()
    c.close()


def test_new_slot_arrays_hold_no_old_rows():
    c = _paged(batch=2, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=64, max_blocks=64)
    for n in (300, 9000):
        old = [torch.full((n,), 7, dtype=torch.int64, device="cuda") for _ in range(8)]
        del old                                             # (the allocator hands their memory out again)
        _, _, slot = c.resize(_i32([2, 1]), n)
        assert (slot[:3] >= 0).all() and (slot[3:] < 0).all()
        c.resize(_i32([0, 0]))
    c.close()


@pytest.mark.parametrize("bad", [99, -1, 1 << 30])
@pytest.mark.parametrize("new", [[33, 10, 20], [200, 0, 0], [0, 40, 200]])
def test_resize_refuses_a_stack_that_holds_no_block(bad, new):
    """An id to be taken that names no block: refused as a whole, as the other causes are; one deeper down is not looked at."""
    abi = _abi()
    c = _paged(batch=3, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=40, max_blocks=16)
    c.resize(_i32([30, 10, 0]), 40)
    have, need = [2, 1, 0], [-(-n // 16) for n in new]
    taken = sum(max(0, a - b) for a, b in zip(need, have)) - sum(max(0, b - a) for a, b in zip(need, have))
    depth = int(c.n_free)
    for at in (depth - 1, depth - taken):                   # the first and the last one from the stack
        good = c.free.clone()
        c.free[at] = bad
        before = [t.clone() for t in (c.table, c.len, c.free, c.n_free)]
        cu, pos, slot = c.resize(_i32(new), 300)
        assert cu.tolist() == [0] * 4 and (slot < 0).all()
        assert all(torch.equal(a, b) for a, b in zip(before, (c.table, c.len, c.free, c.n_free)))
        assert c.check_error() == abi.SRH_ERR_BOUNDS
        c.free.copy_(good)
    c.free[depth - taken - 1] = bad
    c.resize(_i32(new), 300)
    assert c.check_error() == abi.SRH_OK and c.len.tolist() == new
    c.close()


@pytest.mark.parametrize("cu", [[0, 5, 3, 8], [0, 5, 3, 4, 8], [8, 0], [0, 8, 8, 7] + [8] * 60])
def test_attend_refuses_rows_that_two_requests_would_write(cu):
    abi = _abi()
    n = len(cu) - 1
    c, g = _filled([60 + b for b in range(n)], 2, 128, 16, False, 141)
    q, out = _bf16(g, 8, 8, 128), torch.full((8, 8, 128), 7.0, device="cuda").bfloat16()
    c.attend(q, _i32(cu), scale=0.05, out=out)
    assert c.check_error() == abi.SRH_ERR_BOUNDS and (out == 7).all()
    c.attend(q, _i32(sorted(cu)), scale=0.05, out=out)
    assert c.check_error() == 0
    _check_attend(c, q, _i32(sorted(cu)), out, 0.05, 0)
    c.close()


@pytest.mark.parametrize("bad", [-1, 321, 1 << 30, -(1 << 31)])
def test_attend_leaves_out_requests_of_impossible_lengths(bad):
    abi = _abi()
    c, g = _filled([300, 200, 290], 1, 128, 16, True, 151)
    assert c.max_blocks * 16 == 320
    q, cu = _bf16(g, 6, 4, 128), _i32([0, 1, 4, 6])
    good = c.attend(q, cu, scale=0.05)
    c.len[1] = bad
    out = torch.full_like(q, 7.0)
    c.attend(q, cu, scale=0.05, out=out)
    assert c.check_error() == abi.SRH_ERR_BOUNDS
    assert (out[1:4] == 7).all() and torch.equal(out[:1], good[:1]) and torch.equal(out[4:], good[4:])
    c.close()


def test_attend_refuses_an_output_that_overlaps_its_queries():
    abi = _abi()
    c, g = _filled([300, 77], 2, 128, 16, False, 161)
    w = 6 * 128                                             # a row of 6 heads
    cu, n = _i32([0, 3, 5]), 5 * w
    flat = _bf16(g, 4 * n)
    q = flat[n:2 * n].view(5, 6, 128)
    for at in (n, n + 8, n - 8, n + w, 8, 2 * n - 8):       # the same rows, shifted either way by less than they hold
        with pytest.raises(abi.SrhError, match="overlap"):
            c.attend(q, cu, scale=0.06, out=flat[at:at + n].view(5, 6, 128))
    row = flat[:3 * n].view(5, 3 * w)                       # rows between each other's
    at = lambda o: row[:, o:o + w].view(5, 6, 128)  # noqa: E731
    for qa, oa in ((0, 0), (0, w - 8), (w - 8, 0), (8, 0), (w + 352, 2 * w - 8)):
        with pytest.raises(abi.SrhError, match="overlap"):
            c.attend(at(qa), cu, scale=0.06, out=at(oa))
    want, keep = None, q.reshape(5, w).clone()
    for qa, oa in ((0, w), (2 * w, 0), (8, w + 8), (2 * w, w)):
        row[:, qa:qa + w] = keep
        got = c.attend(at(qa), cu, scale=0.06, out=at(oa))
        want = got.clone() if want is None else want
        assert torch.equal(got, want) and torch.equal(row[:, qa:qa + w], keep)
    assert c.check_error() == 0
    c.close()


def test_norm_refuses_outputs_that_overlap_other_rows():
    abi = _abi()
    g = _gen(171)
    c = _paged(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=1, max_blocks=1)
    row = _bf16(g, 6, 2048)                                 # 4 query heads, 2 key heads, room
    q, k, slot = row[:, :512].view(6, 4, 128), row[:, 512:768].view(6, 2, 128), torch.arange(6, device="cuda")
    at = lambda o, h: row[:, o:o + h * 128].view(6, h, 128)  # noqa: E731
    new = lambda h: torch.empty((6, h, 128), device="cuda").bfloat16()  # noqa: E731
    for kw in (dict(q=q, q_out=at(8, 4)), dict(q=at(256, 4), q_out=at(0, 4)), dict(q=q, k=k, q_out=at(264, 4)),
               dict(q=q, k=k, q_out=at(1024, 4), k_out=at(1280, 2)), dict(q=q, k=k, k_out=at(0, 2)),
               dict(q=q, k=k, q_out=at(768, 4), k_out=at(1272, 2)), dict(k=k, k_out=at(640, 2), k_slot=slot),
               dict(q=q, k=k, q_out=q, k_out=q[:, :2]), dict(q=q, q_out=row.view(-1)[2560:2560 + 6 * 512].view(6, 4, 128))):
        with pytest.raises(abi.SrhError, match="overlap|in place"):
            c.norm_rope(**kw)
    wq, wk = c.norm_rope(q, k, q_out=new(4), k_out=new(2))
    # side by side in one row, in place beside the other, and with slots
    a, b = c.norm_rope(q, k, q_out=at(768, 4), k_out=at(1280, 2))
    assert torch.equal(a, wq) and torch.equal(b, wk)
    _, b = c.norm_rope(None, k, k_out=at(1536, 2), k_slot=slot)
    assert torch.equal(b, wk)
    a, b = c.norm_rope(q, k, q_out=q, k_out=k)
    assert torch.equal(a, wq) and torch.equal(b, wk) and c.check_error() == 0
    c.close()


def test_append_counts_no_further_than_its_blocks_go():
    """2,048 of 4,096 requests name the same 17 million rows (one row, repeated): more blocks than an int counts. Refused as a
    whole; no table entry is read, so none is set."""
    abi = _abi()
    n = (1 << 24) + 4096
    mb = n // 16 + 1
    buf = dict(table=torch.empty((4096, mb), dtype=torch.int32, device="cuda"))
    c = _paged(batch=4096, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=4, max_blocks=mb, shared_kv=True, buffers=buf)
    c.len.fill_(n)
    k = torch.ones((1, 1, 128), device="cuda").bfloat16().expand(n, 1, 128)
    c.append(k, None, _i32([0, n] * 2048 + [0]))
    assert c.check_error() == abi.SRH_ERR_BOUNDS
    assert (c.k_codes[0] == 0).all() and (c.k_scale[0] == 1).all()
    c.close()


@pytest.mark.parametrize("handle", [False, True])
def test_tensors_of_a_call_on_another_stream_may_be_let_go(handle):
    """Inputs that the caller drops while the call still waits on its stream: their memory is not handed out before."""
    g = _gen(181)
    c = _paged(batch=2, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=40, max_blocks=20)
    lens, n = [100, 60], 160
    q, k, v = _bf16(g, n, 8, 128), _bf16(g, n, 2, 128), _bf16(g, n, 2, 128)
    pos, freq, w = torch.arange(n, device="cuda").int(), torch.rand(64, device="cuda", dtype=torch.float64), torch.rand(128, device="cuda")

    def step(side, s):
        new = _i32(lens)
        if side:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for _ in range(20):
                    big @ big
        cu, _, _ = c.resize(new, n, stream=s)
        del new
        a = [t.clone() for t in (q, k, v, pos, freq, w)]
        if side:
            side.wait_stream(torch.cuda.current_stream())
        qq, kk = c.norm_rope(a[0], a[1], pos=a[3], inv_freq=a[4], rot_dim=128, q_weight=a[5], stream=s)
        c.append(kk, a[2], cu, stream=s)
        out = c.attend(qq, cu, scale=0.09, stream=s)
        del a, cu, qq, kk
        for m in (n * 1024, n * 256, n * 2, n, 64 * 4, 128 * 2, 6, 4, 2):          # what is free now is written over
            for _ in range(6):
                torch.full((m,), 77, dtype=torch.int16, device="cuda")
                hold.append(torch.full((m,), 77, dtype=torch.int16, device="cuda"))
        torch.cuda.synchronize()
        assert c.check_error() == 0
        return out

    big, hold = torch.randn((8192, 8192), device="cuda").bfloat16(), []
    want = step(None, None)
    c.resize(_i32([0, 0]))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side, side.cuda_stream if handle else side)
    assert torch.equal(got, want)
    c.close()


def test_a_call_that_names_the_capturing_stream():
    c, g = _filled([500, 77], 2, 128, 32, False, 191)
    q, cu = _bf16(g, 2, 16, 128), _i32([0, 1, 2])
    want, s = c.attend(q, cu, scale=0.08), torch.cuda.Stream()
    for how in (s, s.cuda_stream):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            twice = q * 2                                   # from the graph's own memory
            out = c.attend(twice, cu, scale=0.04, stream=how)
            del twice
            again = c.attend(q, cu, scale=0.08, stream=how)
        for _ in range(3):
            out.zero_()
            again.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(again, want)
        del out, again, graph
    assert c.check_error() == 0
    c.close()


def _check_closely(c, q, cu, out, scale, window):
    """Every value within what three e5m2 terms per weight allow, however many tokens there are: 2^-9 and fp16's 2^-11 of each
    weight, 2^-27 of the row's largest contribution (2^-17 where that is at least 2^10), n / 32 additions for each of three
    terms at 2^-23; scores as in _check_attend; bf16 output 2^-8."""
    D, Hk, bs, G = c.D, c.Hk, c.bs, q.shape[1] // c.Hk
    cul, ln = cu.tolist(), c.len.tolist()
    for b in range(len(cul) - 1):
        nq, n = cul[b + 1] - cul[b], ln[b]
        if nq == 0 or n == 0:
            continue
        ids = c.table[b, :-(-n // bs)].long()
        kc, vc = (t[0][ids].view(FP8).double().permute(1, 0, 2, 3).reshape(Hk, -1, D)[:, :n] for t in (c.k_codes, c.v_codes))
        ks, vs = (t[0][ids].double().t().repeat_interleave(bs, 1)[:, None, :n] for t in (c.k_scale, c.v_scale))
        y = q[cul[b]:cul[b + 1]].double().view(nq, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * nq, D)
        pos = torch.arange(n - nq, n, device="cuda").repeat(G)[:, None]
        t = torch.arange(n, device="cuda")
        see = (t <= pos) & (t > pos - (window or n + nq))
        s = torch.where(see, y @ (kc.transpose(1, 2) * ks) * scale, float("-inf"))
        eps = ((D + 8) * 2.0 ** -24 * (y.abs() @ kc.abs().transpose(1, 2)) +
               2.0 ** -17 * y.abs().amax(-1, keepdim=True) * kc.abs().sum(-1)[:, None]) * ks * abs(scale)
        w = torch.where(pos < 0, 0.0, torch.softmax(s, -1)) * vs           # contributions per code
        want, mag = w @ vc, w @ vc.abs()
        tol = (2.0 ** -9 + 2.0 ** -10 + 3 * n / 32 * 2.0 ** -23 + 2 * (eps * see).amax(-1, keepdim=True)) * mag
        tol += 2.0 ** -27 * w.amax(-1, keepdim=True) * (see.double() @ vc.abs()) + 2.0 ** -8 * want.abs()
        got = out[cul[b]:cul[b + 1]].double().view(nq, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * nq, D)
        bad = ~((got - want).abs() <= tol)
        assert not bad.any(), (b, int(bad.sum()), float(((got - want).abs() - tol).max()))


@pytest.mark.parametrize("H,Hk,D,shared,bs", [(16, 2, 128, False, 16), (48, 1, 128, True, 64), (8, 2, 256, False, 32),
                                              (24, 1, 256, True, 128), (64, 1, 256, False, 64), (16, 1, 512, True, 16),
                                              (32, 1, 512, False, 64), (64, 1, 512, True, 64)])
@pytest.mark.parametrize("spread,window", [(0, 0), (3, 0), (2, 700)])
def test_attend_is_as_close_over_long_requests(H, Hk, D, shared, bs, spread, window):
    """Block scales 2^spread apart either way, so that a row's tiles differ by many powers of two and its reference moves."""
    lens, nq = [20000, 3000, 129, 9000], [2, 40, 3, 1]
    c, g = _filled(lens, Hk, D, bs, shared, H + D + spread, spread=spread)
    q, cu = _bf16(g, 46, H, D), _i32([0, 2, 42, 45, 46])
    scale = D ** -0.5 / 2
    out = c.attend(q, cu, scale=scale, window=window)
    assert c.check_error() == 0
    _check_closely(c, q, cu, out, scale, window)
    c.close()


@pytest.mark.parametrize("room", [60, 6000])
def test_a_captured_resize_with_room(room):
    """Growth with room for more tokens, shrinking and a refusal, replayed from one graph each with other lengths."""
    abi = _abi()
    c = _paged(batch=40, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=2000, max_blocks=300)
    o = ResizeOracle(40, 16, 2000)
    rng = np.random.default_rng(room)
    new = torch.zeros(40, dtype=torch.int32, device="cuda")
    out = (_i32([0] * 41), torch.full((room,), 9, dtype=torch.int32, device="cuda"),
           torch.full((room,), 9, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.resize(new, room, out=out)
    for step in range(12):
        want = np.array(o.len)
        grow = rng.integers(0, max(2, 2 * room // 40), 40)
        while grow.sum() > room:
            grow[rng.integers(40)] = 0
        want = want + grow if step % 3 != 2 else want // 3
        if step % 4 == 3:                                   # no such length: refused
            new.copy_(_i32([-1] + [1] * 39))
            graph.replay()
            assert c.check_error() == abi.SRH_ERR_BOUNDS and (out[2] < 0).all() and not out[0].any()
        new.copy_(_i32(want.tolist()))
        graph.replay()
        cu, pos, slot = o.resize(want.tolist())
        assert c.check_error() == abi.SRH_OK
        assert out[0].tolist() == cu and out[1][:len(pos)].tolist() == pos and out[2][:len(pos)].tolist() == slot
        assert (out[2][len(pos):] == -1).all()
        _same_tables(c, o, 40)
    c.close()


@pytest.mark.parametrize("n_req,H,D,shared", [(4096, 2, 128, False), (700, 64, 512, True), (400, 40, 256, False), (300, 17, 512, False)])
def test_attend_as_many_requests_as_there_may_be(n_req, H, D, shared):
    rng = np.random.default_rng(n_req + D)
    lens = rng.integers(0, 40, n_req)
    nq = np.minimum(rng.integers(0, 3, n_req), lens)
    nq[-1] = lens[-1] = 33
    _attend(lens.tolist(), nq.tolist(), H, 1, D, 16, shared, seed=n_req, pad=2)


@pytest.mark.parametrize("D,shared", [(128, True), (256, False), (512, True)])
def test_attend_a_thousand_heads_on_one(D, shared):
    _attend([300, 1, 77], [2, 1, 3], 1024, 1, D, 32, shared, seed=D, pad=1)
    _attend([2000], [1], 1000, 1, D, 64, shared, seed=D + 1, window=150)
