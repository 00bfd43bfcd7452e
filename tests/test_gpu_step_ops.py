"""The operators of include/sbp_step.h against their definitions in 64 bits.

Tolerances.  With e = 2^-24 (half a step of fp32) a sum of n fp32 terms in any order is off by at
most (n - 1) e times the sum of their magnitudes, a product or sum by e, rsqrtf and a division by
2 ulp (4 e); an output in bf16 adds 2^-8 of its value.  Each bound below counts these."""
import numpy as np
import pytest
import torch

from memory_efficient_exact_chunk_b200 import sbp

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def close(got, want, bound):
    """|got - want| <= bound element by element (all fp64)."""
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (int(bad.sum()), float((err - bound).max()))


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def guarded(*shape, dtype=torch.float32, fill=7.0):
    """A buffer with sentinel elements before and behind it (16-byte aligned inside)."""
    n = int(np.prod(shape))
    buf = torch.full((n + 128,), fill, dtype=dtype, device="cuda")
    return buf, buf[64:64 + n].view(shape)


def untouched(buf, n, fill=7.0):
    assert (buf[:64] == fill).all() and (buf[64 + n:] == fill).all()


# ------------------------------------------------------------------------------- embedding
EMBED = [  # rows, cols, vocab, kind of ids
    (1, 1, 1, "same"), (1, 64, 512, "uniform"), (7, 5, 3, "uniform"), (256, 64, 512, "uniform"),
    (33, 8, 1000, "ends"), (300, 12, 40, "padded"), (128, 16, 9, "all_padding"),
    (1000, 1032, 77, "zipf"), (4100, 100, 50, "uniform"), (5000, 36, 1, "same"),
    (5000, 36, 130000, "two"), (8191, 4, 128256, "zipf"), (8193, 20, 152064, "zipf"),
    (20011, 132, 700, "padded"), (70001, 8, 200000, "zipf"), (40000, 3, 4096, "same"),
    (66000, 2, 1 << 22, "ends"), (17000, 24, 300, "sorted"), (16385, 24, 300, "reversed"),
    (256, 36, 1, "same"), (255, 130, 128256, "two"), (256, 4100, 30, "ends"), (257, 8, 4, "zipf"),
    (4096, 8, 5000, "zipf"), (4097, 8, 5000, "padded"), (300, 2, 200000, "uniform"),
    (700, 1447, 50, "padded"), (8192, 12, 100, "zipf"), (9000, 264, 300, "zipf"),
    (300000, 4, 1000, "zipf"), (2001, 666, 64, "uniform"), (5000, 2, 1, "same"),
]


def make_ids(rows, vocab, kind, g):
    u = torch.rand(rows, generator=g, device="cuda", dtype=torch.float64)
    if kind == "same":
        return torch.full((rows,), vocab - 1, dtype=torch.int32, device="cuda")
    if kind == "two":       # two long runs, interleaved
        return torch.where(u < 0.5, 3, vocab - 2).to(torch.int32)
    if kind == "zipf":
        ids = ((vocab + 1.0) ** u - 1.0).long().clamp_(0, vocab - 1).to(torch.int32)
    else:
        ids = (u * vocab).long().clamp_(0, vocab - 1).to(torch.int32)
    if kind == "sorted":
        ids = ids.sort().values
    if kind == "reversed":
        ids = ids.sort(descending=True).values
    if kind == "ends":      # values at and beyond both ends of the range
        ends = torch.tensor([0, vocab - 1, vocab, -1, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32,
                            device="cuda")
        ids[:len(ends)] = ends[:rows]
    if kind in ("padded", "all_padding"):
        ids[torch.rand(rows, generator=g, device="cuda") < (0.4 if kind == "padded" else 2.0)] = -1
    return ids.contiguous()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,vocab,kind", EMBED)
def test_embedding_scaled_forward(rows, cols, vocab, kind, dt):
    g = gen(rows + cols)
    ids = make_ids(rows, vocab, kind, g)
    table = torch.randn(vocab, cols, generator=g, device="cuda").to(DT[dt])
    buf, y = guarded(rows, cols, dtype=DT[dt])
    sbp.embedding_scaled_forward(ids, table, 1.7, y)
    ok = (ids >= 0) & (ids < vocab)
    want = table[torch.where(ok, ids, 0).long()].double() * float(np.float32(1.7)) * ok[:, None]
    close(y, want, want.abs() * (HALF_STEP[dt] * (1 + E) + E))
    assert (y[~ok] == 0).all()
    untouched(buf, rows * cols)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [3, 67, 257, 259, 511, 518, 521, 1001, 1027, 1030, 1156, 4097])
def test_embedding_scaled_forward_off_the_16_byte_grid(cols, dt):
    """Rows at every offset, the table's last elements among them; what lies around the table is
    not used, and a row of padding is +0 under a negative scale."""
    g = gen(cols)
    vocab, rows = 9, 75
    buf, table = guarded(vocab, cols, dtype=DT[dt], fill=float("nan"))
    table.copy_(torch.randn(vocab, cols, generator=g, device="cuda"))
    ids = torch.arange(rows, device="cuda", dtype=torch.int32) * 7 % (vocab + 1)
    ids[::5] = vocab - 1
    out, y = guarded(rows, cols, dtype=DT[dt])
    sbp.embedding_scaled_forward(ids, table, -1.7, y)
    ok = ids < vocab
    want = (table[torch.where(ok, ids, 0).long()].float() * float(np.float32(-1.7))).to(DT[dt])
    assert torch.equal(y[ok], want[ok])
    assert (y[~ok].float().view(torch.int32) == 0).all()
    untouched(out, rows * cols)


def grad_reference(ids, dy, scale, vocab, base):
    """d_table, the sum of the terms' magnitudes and the number of rows of each id, in fp64."""
    ok = (ids >= 0) & (ids < vocab)
    i, d = ids[ok].long(), dy[ok].double()
    s = float(np.float32(scale))
    z = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device="cuda")
    total = z.clone().index_add_(0, i, d) * s
    mag = z.index_add_(0, i, d.abs()) * abs(s)
    n = torch.bincount(i, minlength=vocab)
    return total + base, mag, n


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows,cols,vocab,kind", EMBED)
def test_embedding_scaled_backward(rows, cols, vocab, kind, accumulate):
    g = gen(rows + 3 * cols)
    ids = make_ids(rows, vocab, kind, g)
    dy = torch.randn(rows, cols, generator=g, device="cuda")
    dy[(ids < 0) | (ids >= vocab)] = float("nan")        # padding rows are not read
    buf, d = guarded(vocab, cols)
    base = torch.zeros((), dtype=torch.float64, device="cuda")
    if accumulate:
        d.normal_(generator=g)
        base = d.double().clone()
    else:
        d.fill_(float("nan"))
    first = d.clone()
    ws = sbp.embedding_scaled_backward(ids, dy, -0.37, d, accumulate=accumulate)
    want, mag, n = grad_reference(ids, dy, -0.37, vocab, base)
    # n rows' sum, the product with the scale and the sum with the old value
    close(d, want, mag * ((n[:, None] + 2) * E) + (want.abs() + mag) * E * 2)
    untouched(buf, vocab * cols)
    if accumulate:           # ids that do not occur keep their bits
        assert torch.equal(d[n == 0], first[n == 0])
    again = first
    sbp.embedding_scaled_backward(ids, dy, -0.37, again, accumulate=accumulate, ws=ws)
    assert torch.equal(again, d)


def test_embedding_scaled_backward_is_the_forwards_gradient():
    """<dy, F(E)> is linear in E: its gradient is compared with differences of the forward."""
    g = gen(3)
    rows, cols, vocab = 57, 12, 10
    ids = make_ids(rows, vocab, "padded", g)
    table = torch.randn(vocab, cols, generator=g, device="cuda")
    dy = torch.randn(rows, cols, generator=g, device="cuda")
    d = torch.empty(vocab, cols, device="cuda")
    sbp.embedding_scaled_backward(ids, dy, 2.5, d, accumulate=False)
    y0, y1 = torch.empty(rows, cols, device="cuda"), torch.empty(rows, cols, device="cuda")
    for _ in range(5):
        step = torch.randn(vocab, cols, generator=g, device="cuda")
        sbp.embedding_scaled_forward(ids, table + step, 2.5, y1)
        sbp.embedding_scaled_forward(ids, table - step, 2.5, y0)
        diff = float((dy.double() * (y1.double() - y0.double())).sum()) / 2
        form = float((d.double() * step.double()).sum())
        # each of the rows * cols products carries a few roundings of size e (table +- step,
        # scale, the gradient's own sum of at most rows terms)
        mag = float((dy.double().abs() * (y1.double().abs() + y0.double().abs())).sum()
                    + (d.double().abs() * step.double().abs()).sum())
        assert abs(diff - form) <= mag * (rows + 8) * E


# ------------------------------------------------------------------------- queries and keys
def qk_tables(n, hd, theta=1e4):
    return sbp.rope_table(n, hd, theta)


def qk_positions(kind, rows, g):
    if kind is None:
        return None, None, rows
    if isinstance(kind, int):
        return None, kind, kind
    if kind == "any":
        p = torch.randint(0, 97, (rows,), generator=g, device="cuda", dtype=torch.int32)
        return p, None, 97
    p = torch.randint(0, 40, (rows,), generator=g, device="cuda", dtype=torch.int32)
    p[::3] = torch.tensor([-1, 40, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32,
                          device="cuda")[torch.arange(len(p[::3]), device="cuda") % 4]
    return p, None, 40        # "outside": positions beyond the tables


def qk_inputs(rows, H, Hkv, hd, dt, layout, g):
    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda").to(DT[dt])
    if layout == "fused":
        x = randn(rows, H + 2 * Hkv, hd)
        return x[:, :H], x[:, H:H + Hkv]
    if layout == "odd":       # rows an odd number of elements apart, off the 16-byte grid
        ldq, ldk = H * hd + 1, Hkv * hd + 3
        xq, xk = randn(rows * ldq + 1), randn(rows * ldk + 1)
        return (xq[1:].view(rows, ldq)[:, :H * hd].unflatten(1, (H, hd)),
                xk[1:].view(rows, ldk)[:, :Hkv * hd].unflatten(1, (Hkv, hd)))
    return randn(rows, H, hd), randn(rows, Hkv, hd)


QK = [  # rows, heads, kv heads, head_dim, dtype, layout, positions
    (1, 1, 1, 2, "f32", "plain", None), (1, 32, 8, 128, "bf16", "fused", None),
    (3, 4, 4, 16, "f32", "plain", None), (64, 4, 4, 16, "bf16", "fused", 16),
    (5, 7, 1, 64, "bf16", "odd", "any"), (130, 6, 2, 80, "f32", "plain", "any"),
    (77, 6, 3, 96, "bf16", "fused", 11), (33, 8, 2, 256, "bf16", "plain", "outside"),
    (33, 8, 2, 256, "f32", "odd", None), (201, 28, 4, 128, "bf16", "fused", "outside"),
    (1031, 32, 8, 128, "bf16", "plain", 1031), (515, 12, 12, 128, "f32", "fused", "any"),
    (40, 5, 5, 210, "bf16", "fused", None), (900, 3, 1, 32, "bf16", "plain", 300),
    (9, 2, 1, 6, "f32", "odd", "outside"), (2050, 9, 3, 112, "f32", "plain", "any"),
    (3000, 1, 1, 64, "f32", "fused", None), (17, 64, 1, 48, "bf16", "plain", None),
    (700, 1, 512, 16, "bf16", "plain", 700), (999, 1, 3, 8, "f32", "fused", "outside"),
    (1500, 5, 2, 24, "bf16", "plain", "any"), (333, 3, 1, 256, "bf16", "fused", 111),
    (2000, 7, 1, 102, "bf16", "fused", "any"), (600, 2, 2, 254, "f32", "plain", None),
    (1, 1, 1, 80, "bf16", "plain", None), (515, 7, 3, 80, "bf16", "fused", "outside"),
    (1003, 12, 12, 80, "f32", "plain", "any"), (3001, 28, 4, 80, "bf16", "plain", 3001),
    (64, 32, 8, 96, "f32", "plain", 64), (2, 1, 11, 96, "bf16", "fused", "outside"),
    (1777, 5, 1, 96, "bf16", "plain", "any"), (31, 6, 2, 80, "bf16", "odd", None),
]


def qk_reference(x, gain, c, s, ok, eps, dy=None):
    """Definition in fp64 and, with dy, the gradients; magnitudes for the bounds."""
    x, gain = x.double(), gain.double()
    hd = x.shape[-1]
    h = hd // 2
    r = 1.0 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    xh = x * r
    if dy is None:
        n = xh * gain
        a, b = n[..., :h], n[..., h:]
        y = torch.cat((a * c - b * s, b * c + a * s), -1) * ok
        mag = torch.cat((a.abs() * c.abs() + b.abs() * s.abs(),
                         b.abs() * c.abs() + a.abs() * s.abs()), -1) * ok
        return y, mag
    dy = dy.double()
    a, b = dy[..., :h], dy[..., h:]
    u = torch.cat((a * c + b * s, b * c - a * s), -1) * ok
    um = torch.cat((a.abs() * c.abs() + b.abs() * s.abs(),
                    b.abs() * c.abs() + a.abs() * s.abs()), -1) * ok
    v = u * gain
    vm = um * gain.abs()
    dx = r * (v - xh * (xh * v).mean(-1, keepdim=True))
    dxm = r * (vm + xh.abs() * (xh.abs() * vm).mean(-1, keepdim=True))
    return dx, dxm, (u * xh).sum((0, 1)), (um * xh.abs()).sum((0, 1))


def qk_angles(pos, seq, table_len, cos, sin, rows):
    p = pos.long() if pos is not None else torch.arange(rows, device="cuda") % (seq or rows)
    ok = (p >= 0) & (p < table_len)
    p = torch.where(ok, p, 0)
    return cos[p].double()[:, None], sin[p].double()[:, None], ok.double()[:, None, None]


@pytest.mark.parametrize("rows,H,Hkv,hd,dt,layout,kind", QK)
def test_qk_norm_rope_forward(rows, H, Hkv, hd, dt, layout, kind):
    g = gen(rows * H + hd)
    q, k = qk_inputs(rows, H, Hkv, hd, dt, layout, g)
    gains = [(1 + 0.3 * torch.randn(hd, generator=g, device="cuda")).to(DT[dt]) for _ in "qk"]
    pos, seq, n = qk_positions(kind, rows, g)
    cos, sin = qk_tables(n, hd)
    bq, qo = guarded(rows, H, hd, dtype=DT[dt])
    bk, ko = guarded(rows, Hkv, hd, dtype=DT[dt])
    sbp.qk_norm_rope_forward(q, k, *gains, cos, sin, 1e-6, qo, ko, positions=pos, seq_len=seq)
    c, s, ok = qk_angles(pos, seq, n, cos, sin, rows)
    for x, gain, y in ((q, gains[0], qo), (k, gains[1], ko)):
        want, mag = qk_reference(x, gain, c, s, ok, 1e-6)
        # mean of hd squares (halved by the root), the root itself, three products and a sum
        close(y, want, mag * (hd / 2 + 16) * E + want.abs() * HALF_STEP[dt] * (1 + 2.0 ** -7))
    untouched(bq, rows * H * hd)
    untouched(bk, rows * Hkv * hd)
    # in place on the strided inputs, and the queries alone
    only = torch.empty_like(qo)
    sbp.qk_norm_rope_forward(q, None, gains[0], None, cos, sin, 1e-6, only, None, positions=pos,
                             seq_len=seq)
    assert torch.equal(only, qo)
    sbp.qk_norm_rope_forward(q, k, *gains, cos, sin, 1e-6, q, k, positions=pos, seq_len=seq)
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("rows,H,Hkv,hd,dt,layout,kind", QK)
def test_qk_norm_rope_backward(rows, H, Hkv, hd, dt, layout, kind):
    g = gen(rows * H + hd + 1)
    q, k = qk_inputs(rows, H, Hkv, hd, dt, layout, g)
    gains = [(1 + 0.3 * torch.randn(hd, generator=g, device="cuda")).to(DT[dt]) for _ in "qk"]
    pos, seq, n = qk_positions(kind, rows, g)
    cos, sin = qk_tables(n, hd)
    dqo, dko = qk_inputs(rows, H, Hkv, hd, "f32", layout, g)
    bq, dq = guarded(rows, H, hd)
    bk, dk = guarded(rows, Hkv, hd)
    dg = [torch.randn(hd, generator=g, device="cuda") for _ in "qk"]
    base = [t.clone() for t in dg]
    args = (q, k, *gains, cos, sin, 1e-6)
    ws = sbp.qk_norm_rope_backward(*args, dqo, dko, dq, dk, *dg, positions=pos, seq_len=seq)
    c, s, ok = qk_angles(pos, seq, n, cos, sin, rows)
    for x, gain, dy, dx, got, b in ((q, gains[0], dqo, dq, dg[0], base[0]),
                                    (k, gains[1], dko, dk, dg[1], base[1])):
        want, mag, wg, mg = qk_reference(x, gain, c, s, ok, 1e-6, dy)
        # the norm's factor (hd / 2 + 8 e) enters three times, the mean of hd products once
        close(dx, want, mag * (2.5 * hd + 40) * E)
        terms = rows * x.shape[1]
        close(got, wg + b.double(), mg * (terms + hd / 2 + 16) * E + (wg + b).abs() * 2 * E)
    untouched(bq, rows * H * hd)
    untouched(bk, rows * Hkv * hd)
    # again: the same bits; into the upstream gradients' own buffers too
    dg2 = [t.clone() for t in base]
    sbp.qk_norm_rope_backward(*args, dqo, dko, dqo, dko, *dg2, positions=pos, seq_len=seq, ws=ws)
    assert torch.equal(dqo, dq) and torch.equal(dko, dk)
    assert torch.equal(dg2[0], dg[0]) and torch.equal(dg2[1], dg[1])
    # the queries alone
    dq3, dg3 = torch.empty_like(dq), base[0].clone()
    qa = (q, None, gains[0], None, cos, sin, 1e-6)
    dqo3, _ = qk_inputs(rows, H, Hkv, hd, "f32", layout, g)
    sbp.qk_norm_rope_backward(*qa, dqo3, None, dq3, None, dg3, None, positions=pos, seq_len=seq)
    want, mag, wg, mg = qk_reference(q, gains[0], c, s, ok, 1e-6, dqo3)
    close(dq3, want, mag * (2.5 * hd + 40) * E)


def test_qk_norm_rope_backward_against_differences():
    """Central differences of the fp64 definition (step 1e-5: truncation and rounding below
    1e-9 relative) along random directions, against the kernel's gradients."""
    g = gen(11)
    rows, H, Hkv, hd = 9, 4, 2, 32
    q, k = qk_inputs(rows, H, Hkv, hd, "f32", "plain", g)
    gq, gk = (1 + 0.3 * torch.randn(hd, generator=g, device="cuda") for _ in "qk")
    cos, sin = qk_tables(rows, hd)
    c, s, ok = qk_angles(None, None, rows, cos, sin, rows)
    dqo, dko = qk_inputs(rows, H, Hkv, hd, "f32", "plain", g)
    dq, dk = torch.empty_like(dqo), torch.empty_like(dko)
    dg = [torch.zeros(hd, device="cuda") for _ in "qk"]
    sbp.qk_norm_rope_backward(q, k, gq, gk, cos, sin, 1e-6, dqo, dko, dq, dk, *dg)
    for x, gain, dy, dx, dgain in ((q, gq, dqo, dq, dg[0]), (k, gk, dko, dk, dg[1])):
        for _ in range(4):
            vx = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
            vg = torch.randn(hd, generator=g, device="cuda", dtype=torch.float64)
            h = 1e-5
            f = [float((qk_reference(x.double() + t * vx, gain.double() + t * vg, c, s, ok,
                                     1e-6)[0] * dy.double()).sum()) for t in (h, -h)]
            got = float((dx.double() * vx).sum() + (dgain.double() * vg).sum())
            mag = float((dx.double().abs() * vx.abs()).sum() + (dgain.double().abs() * vg.abs())
                        .sum())
            # per element (2.5 hd + 40) e of a magnitude a few times its own, and the differences
            assert abs(got - (f[0] - f[1]) / (2 * h)) <= mag * ((2.5 * hd + 40) * 4 * E + 1e-9)


def test_rope_table():
    cos, sin = sbp.rope_table(1000, 64, 5e5)
    j = torch.arange(0, 64, 2, device="cuda", dtype=torch.float64) / 64
    a = torch.arange(1000, device="cuda", dtype=torch.float64)[:, None] * (5e5 ** -j)[None]
    # fp64 angles up to 999 (error 1e-13 relative), rounded to fp32
    assert float((cos.double() - a.cos()).abs().max()) <= E + 1e-12
    assert float((sin.double() - a.sin()).abs().max()) <= E + 1e-12


# ------------------------------------------------------------------------------ clipping
def grad_list(sizes, g, scale=1.0, spread=2.0):
    out = []
    for i, n in enumerate(sizes):
        t = torch.randn(n, generator=g, device="cuda") * (scale * spread ** (i % 5 - 2))
        out.append(t)
    return out


SIZES = {
    "one": [1], "odd": [1, 2, 3, 4, 5, 0, 7, 1023, 16383, 16384, 16385, 0, 65537],
    "empty": [0, 0], "many": [(i * 37) % 1201 for i in range(700)], "large": [3_000_001, 17],
    "few": [131072], "above_few": [131073], "full_table": [5] * 64, "one_more": [5] * 65,
    "full_large_table": [130] * 1024, "one_more_large": [130] * 1025,
    "small_among_large": [1] * 900 + [2_000_001] + [3] * 200 + [4_000_000],
    "thousands": [3] * 2500, "pieces": [4 * 1024 * k + k % 3 for k in range(1, 70)],
}


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9])
@pytest.mark.parametrize("out", [False, True])
@pytest.mark.parametrize("name", list(SIZES))
def test_grad_clip_norm(name, out, max_norm):
    g = gen(len(SIZES[name]))
    grads = grad_list(SIZES[name], g)
    ref = [t.double() for t in grads]
    norm = torch.stack([t.square().sum() for t in ref]).sum().sqrt()
    coef = min(1.0, max_norm / (float(norm) + 1e-6))
    into = [torch.full_like(t, 3.0) for t in grads] if out else None
    got_norm = torch.full((1,), -1.0, device="cuda")
    keep = [t.clone() for t in grads]
    ws = sbp.grad_clip_norm(grads, max_norm, got_norm, out=into)
    assert abs(float(got_norm) - float(norm)) <= float(norm) * (E + 1e-12)
    for t, r, k in zip(into if out else grads, ref, keep):
        # the coefficient and the product are each rounded once (and an underflow step)
        close(t, r * coef, r.abs() * coef * (2 * E + 1e-12) + 2.0 ** -149)
        if coef == 1.0:
            assert torch.equal(t, k)
    if out:
        assert all(torch.equal(t, k) for t, k in zip(grads, keep))
        again = [torch.empty_like(t) for t in grads]
        sbp.grad_clip_norm(sbp.GradList(grads), max_norm, got_norm, out=sbp.GradList(again), ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(again, into))


@pytest.mark.parametrize("scale", [1e-30, 1e-42, 1e25, 3e38])
def test_grad_norm_far_from_one(scale):
    """Squares that fp32 cannot hold: the norm is formed in 64 bits."""
    g = gen(5)
    grads = [(torch.rand(1000, generator=g, device="cuda") - 0.5) * scale, torch.zeros(
        7, device="cuda")]
    norm = sum(float(t.double().square().sum()) for t in grads) ** 0.5
    sq = torch.zeros(1, dtype=torch.float64, device="cuda")
    sbp.grad_sqsum(grads, sq)
    assert abs(float(sq) - norm ** 2) <= norm ** 2 * 1e-12
    got = torch.zeros(1, device="cuda")
    ref = [t.double() for t in grads]
    sbp.grad_clip(grads, sq, 1.0, norm_out=got)
    if norm < 3.4e38:
        assert abs(float(got) - norm) <= norm * (E + 1e-12) + 2.0 ** -149
    coef = min(1.0, 1.0 / (norm + 1e-6))
    for t, r in zip(grads, ref):
        # a coefficient below the normal range of fp32 is rounded to a multiple of 2^-149
        close(t, r * coef, r.abs() * (coef * 3 * E + 2.0 ** -149) + 2.0 ** -149)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("out", [False, True])
def test_grad_clip_leaves_nonfinite_gradients_alone(bad, out):
    grads = [torch.ones(5000, device="cuda"), torch.ones(33, device="cuda")]
    grads[1][32] = bad
    keep = [t.clone() for t in grads]
    into = [torch.zeros_like(t) for t in grads] if out else None
    norm = torch.zeros(1, device="cuda")
    sbp.grad_clip_norm(grads, 0.1, norm, out=into)
    assert not torch.isfinite(norm).any()
    for t, k in zip(into if out else grads, keep):
        assert torch.equal(t.nan_to_num(nan=-5.0), k.nan_to_num(nan=-5.0))


def test_grad_lists_that_share_memory_are_refused():
    flat = torch.ones(1024, device="cuda")
    a, b, c = flat[:256], flat[256:512], flat[512:768]
    for bad in ([a, a], [a, flat[252:300]], [flat, b]):
        with pytest.raises(ValueError, match="share memory"):
            sbp.GradList(bad)
    norm = torch.zeros(1, device="cuda")
    for out in ([b, a], [b, c], [flat[4:260], c], [a], [c, flat[768:1000]]):
        with pytest.raises(ValueError, match="out must"):
            sbp.grad_clip_norm([a, b], 1.0, norm, out=out)
    assert (flat == 1).all()
    for out in ([a, b], [a, c], [c, b], [c, flat[768:]]):     # its own, or elsewhere
        flat.fill_(1.0)
        sbp.grad_clip_norm([a, b], 1.0, norm, out=out)
        assert all(torch.equal(t, torch.full_like(t, float(t[0]))) for t in out)
        assert abs(float(out[0][0]) - 1 / (512 ** 0.5)) < 1e-6


def test_grad_sqsum_of_shards_adds_up():
    """Two ranks' shares of the gradients: their sums of squares add, each clips its own."""
    g = gen(9)
    a, b = grad_list([700, 5, 30001], g), grad_list([1, 16384], g)
    sa, sb = (torch.zeros(1, dtype=torch.float64, device="cuda") for _ in "ab")
    sbp.grad_sqsum(a, sa)
    sbp.grad_sqsum(b, sb)
    whole = [t.clone() for t in a + b]
    norm = torch.zeros(1, device="cuda")
    sbp.grad_clip_norm(whole, 0.7, norm)
    total = sa + sb
    n2 = torch.zeros(1, device="cuda")
    sbp.grad_clip(a, total, 0.7, norm_out=n2)
    sbp.grad_clip(b, total, 0.7)
    assert abs(float(n2) - float(norm)) <= 2 * E * float(norm)
    for x, y in zip(a + b, whole):
        close(x, y.double(), y.double().abs() * 4 * E)


def test_sizes_the_library_refuses():
    """The wrappers pass the library's own status on."""
    f = torch.zeros(1, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    for call in (lambda: sbp.embedding_scaled_forward(none, f.view(1, 1), 1.0, f[:0].view(0, 1)),
                 lambda: sbp.embedding_scaled_backward(none, f[:0].view(0, 1), 1.0, f.view(1, 1))):
        with pytest.raises(sbp.SbpError) as e:
            call()
        assert e.value.code == 1
    table = f.expand((1 << 22) + 1).contiguous().view(-1, 1)
    with pytest.raises(sbp.SbpError) as e:
        sbp.embedding_scaled_backward(torch.zeros(1, dtype=torch.int32, device="cuda"),
                                      f.view(1, 1), 1.0, table)
    assert e.value.code == 2
    q, g, t = (torch.zeros(2, 1, 3, device="cuda"), torch.zeros(3, device="cuda"),
               torch.zeros(2, 1, device="cuda"))
    with pytest.raises(sbp.SbpError) as e:
        sbp.qk_norm_rope_forward(q, None, g, None, t, t, 1e-6, q, None)
    assert e.value.code == 2
    with pytest.raises(sbp.SbpError) as e:          # more positions than the tables hold
        sbp.qk_norm_rope_forward(torch.zeros(3, 1, 2, device="cuda"), None, g[:2], None, t, t,
                                 1e-6, torch.zeros(3, 1, 2, device="cuda"), None)
    assert e.value.code == 1
    with pytest.raises(sbp.SbpError) as e:          # a workspace that is not 256-byte aligned
        sbp.grad_sqsum([f], torch.zeros(1, dtype=torch.float64, device="cuda"),
                       ws=sbp.workspace(1 << 20)[1:])
    assert e.value.code == 1


# ------------------------------------------------------- offsets past 32 bits, masked places
def test_embedding_offsets_past_32_bits():
    """A table of 2.3 G elements (9.2 GB): the last rows of it are used."""
    vocab, cols = 140000, 16384
    g = gen(41)
    ids = torch.tensor([vocab - 1, 5, vocab - 2, vocab - 1, 0, 131073] * 50, dtype=torch.int32,
                       device="cuda")
    dy = torch.randn(len(ids), cols, generator=g, device="cuda")
    table = torch.full((vocab, cols), float("nan"), device="cuda")
    sbp.embedding_scaled_backward(ids, dy, 0.5, table, accumulate=False)
    for v in ids.unique().tolist():
        rows = dy[ids == v].double()
        close(table[v], rows.sum(0) * 0.5, rows.abs().sum(0) * 0.5 * (len(rows) + 4) * E)
    for v in (1, 100000, vocab - 3):
        assert (table[v] == 0).all()
    y = torch.empty_like(dy)
    sbp.embedding_scaled_forward(ids, table, 2.0, y)
    assert torch.equal(y, table[ids.long()] * 2.0)


def test_qk_offsets_past_32_bits():
    """Rows 8192 elements apart, 2.3 G elements from first to last."""
    rows, H, hd, ld = 280000, 2, 64, 8192
    x = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")
    q = x[:, 64:64 + H * hd].unflatten(1, (H, hd))
    q.normal_(generator=gen(42))
    gain = torch.ones(hd, dtype=torch.bfloat16, device="cuda")
    cos, sin = qk_tables(1000, hd)
    sbp.qk_norm_rope_forward(q, None, gain, None, cos, sin, 1e-6, q, None, seq_len=1000)
    tail = q[-2500:].clone()
    q.normal_(generator=gen(42))          # the inputs again
    c, s, ok = qk_angles(None, 1000, 1000, cos, sin, rows)
    want, mag = qk_reference(q[-2500:], gain, c[-2500:], s[-2500:], ok[-2500:], 1e-6)
    close(tail, want, mag * (hd / 2 + 16) * E + want.abs() * 2.0 ** -8 * (1 + 2.0 ** -7))


def test_clip_offsets_past_32_bits():
    n = 2 ** 31 + 5
    big, small = torch.full((n,), 1e-3, device="cuda"), torch.ones(3, device="cuda")
    norm = torch.zeros(1, device="cuda")
    v = float(np.float32(1e-3))
    want = (n * v * v + 3) ** 0.5
    sbp.grad_clip_norm([small, big], 1.0, norm)
    assert abs(float(norm) - want) <= want * 2 * E
    coef = 1.0 / (want + 1e-6)
    for t, x in ((big[:4], v), (big[-6:], v), (big[2 ** 31 - 2:2 ** 31 + 2], v), (small, 1.0)):
        close(t, torch.full_like(t, x, dtype=torch.float64) * coef, x * coef * 4 * E)
    assert float(big.min()) == float(big.max())


@pytest.mark.parametrize("hd,dt", [(128, "bf16"), (64, "f32"), (10, "bf16")])
def test_rows_outside_the_tables_are_not_looked_at(hd, dt):
    """NaN and infinities in rows whose position is outside stay where they are."""
    g = gen(hd)
    rows, H, Hkv = 41, 3, 1
    q, k = qk_inputs(rows, H, Hkv, hd, dt, "fused", g)
    gain = torch.ones(hd, dtype=DT[dt], device="cuda")
    pos = torch.arange(rows, device="cuda", dtype=torch.int32)
    pos[1::3] = -5
    bad = pos < 0
    cos, sin = qk_tables(rows, hd)
    q[bad], k[bad] = float("nan"), float("inf")
    qo, ko = torch.empty_like(q).contiguous(), torch.empty_like(k).contiguous()
    sbp.qk_norm_rope_forward(q, k, gain, gain, cos, sin, 1e-6, qo, ko, positions=pos)
    dqo, dko = qk_inputs(rows, H, Hkv, hd, "f32", "plain", g)
    dqo[bad], dko[bad] = float("inf"), float("nan")
    dq, dk, dg = torch.empty_like(dqo), torch.empty_like(dko), torch.zeros(2, hd, device="cuda")
    sbp.qk_norm_rope_backward(q, k, gain, gain, cos, sin, 1e-6, dqo, dko, dq, dk, dg[0], dg[1],
                              positions=pos)
    for t in (qo, ko, dq, dk):
        assert (t[bad] == 0).all() and torch.isfinite(t).all()
    assert torch.isfinite(dg).all() and (dg != 0).any()


# --------------------------------------------------------------- streams, capture, sharing
def step_calls(g):
    """One call of each operator with its own buffers: (run, outputs, inputs)."""
    ids = make_ids(9000, 3000, "zipf", g)
    table = torch.randn(3000, 40, generator=g, device="cuda")
    y = torch.empty(9000, 40, device="cuda")
    dy = torch.randn(9000, 40, generator=g, device="cuda")
    dt = torch.empty(3000, 40, device="cuda")
    q, k = qk_inputs(300, 8, 2, 128, "bf16", "fused", g)
    gq = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    cos, sin = qk_tables(300, 128)
    qo, ko = torch.empty_like(q).contiguous(), torch.empty_like(k).contiguous()
    dqo, dko = qk_inputs(300, 8, 2, 128, "f32", "plain", g)
    dq, dk, dg = torch.empty_like(dqo), torch.empty_like(dko), torch.zeros(2, 128, device="cuda")
    grads = sbp.GradList(grad_list([100, 70001, 3], g))
    into = sbp.GradList([torch.empty_like(t) for t in grads.tensors])
    norm = torch.zeros(1, device="cuda")
    ws = [sbp.workspace(8 << 20) for _ in range(3)]

    def run(stream=None):
        dg.zero_()
        sbp.embedding_scaled_forward(ids, table, 1.5, y, stream=stream)
        sbp.embedding_scaled_backward(ids, dy, 1.5, dt, accumulate=False, ws=ws[0], stream=stream)
        sbp.qk_norm_rope_forward(q, k, gq, gq, cos, sin, 1e-6, qo, ko, stream=stream)
        sbp.qk_norm_rope_backward(q, k, gq, gq, cos, sin, 1e-6, dqo, dko, dq, dk, dg[0], dg[1],
                                  ws=ws[1], stream=stream)
        sbp.grad_clip_norm(grads, 0.5, norm, out=into, ws=ws[2], stream=stream)
    return run, [y, dt, qo, ko, dq, dk, dg, norm, *into.tensors], [ids, table, dy, q, dqo, dko,
                                                                   *grads.tensors]


def test_calls_on_other_streams_at_once():
    a, outs_a, _ = step_calls(gen(21))
    b, outs_b, _ = step_calls(gen(22))
    a(), b()
    want = [t.clone() for t in outs_a + outs_b]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for t in outs_a + outs_b:
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            a()
        with torch.cuda.stream(s2):
            b(stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs_a + outs_b, want))


def test_captured_calls_replay_on_new_inputs():
    run, outs, ins = step_calls(gen(31))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    fresh, outs2, ins2 = step_calls(gen(32))
    fresh()
    for x, y in zip(ins, ins2):
        x.copy_(y)
    # k is a view of q's buffer: copy the whole projection
    ins[3]._base.copy_(ins2[3]._base)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, outs2))
