"""Calls at the edges of the operators of include/sbp_step.h and of the paths that use them:
streams that run beside one another, sizes next to a limit, aliased arguments, and gradients of few
summands, held to bounds that a single lost or foreign summand breaks."""
import numpy as np
import pytest
import torch

from memory_efficient_exact_chunk_b200 import sbp, synth
from tests.helpers import rel_fro, to_np

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
S = synth.LayerShape


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------- the layer's side streams
def layer_run(L, W, x, dy, D, reverse):
    """Gradients of the layer; weights with q_norm_g take the path with query/key norms."""
    B, T, d = x.shape
    code = sbp.SBP_BF16 if x.dtype == torch.bfloat16 else sbp.SBP_F32
    cfg = sbp.layer_cfg(B, T, d, L.n_heads, L.n_kv_heads, L.head_dim, L.ffn, L.rms_eps,
                        L.rope_theta, code, D)
    dx = torch.full(x.shape, float("nan"), device="cuda")
    g = {n: None if v is None else torch.zeros(v.shape, device="cuda") for n, v in W.items()}
    run = sbp.decoder_layer_backward_reverse if reverse else sbp.decoder_layer_backward
    sbp.device_status(run(cfg, W, x, dy, dx, g))
    return {"dx": dx, **{n: v for n, v in g.items() if v is not None}}


def layer_data(L, B, T, dtype, seed, norms):
    rng = np.random.default_rng(seed)
    W = synth.layer_weights(rng, L, dtype == "bf16", gamma_std=0.1)
    if norms:
        for n in sbp.QK_NORM_FIELDS:
            W[n] = 1.0 + 0.3 * rng.standard_normal(L.head_dim, dtype=np.float32)
    W = {n: None if v is None else torch.from_numpy(v).to(DT[dtype]).cuda() for n, v in W.items()}
    x = torch.randn(B, T, L.d_model, generator=gen(seed), device="cuda").to(DT[dtype])
    dy = torch.randn(B, T, L.d_model, generator=gen(seed + 1), device="cuda") * 1e-3
    return W, x, dy


@pytest.mark.parametrize("norms", [False, True])
def test_bias_sums_of_both_chunk_orders_while_the_weight_products_lag(norms):
    """The query bias is summed behind the weight products of a wide MLP on a side stream, the key
    and value biases on the caller's: in reverse order at the same time.  Calls repeat their bits,
    and the orders differ by fp32 roundings only (1e-5 per tensor, as D = 1 against D > 1)."""
    L = S(256, 2, 2, 128, 14336, 1e-6, 10000.0, qkv_bias=True)
    W, x, dy = layer_data(L, 1, 2048, "bf16", 3, norms)
    want = layer_run(L, W, x, dy, 2, reverse=False)
    first = layer_run(L, W, x, dy, 2, reverse=True)
    for n in ("bq", "bv"):
        assert rel_fro(to_np(first[n]), to_np(want[n])) <= 1e-5, n
    for _ in range(6):
        again = layer_run(L, W, x, dy, 2, reverse=True)
        for n, v in first.items():
            assert torch.equal(v, again[n]), n


# ------------------------------------------------------------------------------- embedding
NEAR_THE_DEFAULT = """
import torch
from memory_efficient_exact_chunk_b200 import sbp
rows, vocab = {rows}, {vocab}
g = torch.Generator(device="cuda").manual_seed(1)
ids = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
ids[:3] = torch.tensor([0, vocab - 1, vocab], dtype=torch.int32, device="cuda")
dy = torch.randn(rows, 4, generator=g, device="cuda")
d = torch.empty(vocab, 4, device="cuda")
sbp.embedding_scaled_backward(ids, dy, 1.0, d, accumulate=False)
ok = ids < vocab
i, v = ids[ok].long(), dy[ok].double()
z = torch.zeros(vocab, 4, dtype=torch.float64, device="cuda")
want, mag = z.index_add(0, i, v), z.index_add(0, i, v.abs())
n = torch.bincount(i, minlength=vocab)[:, None]
# a sum of n terms and the product with the scale
assert ((d.double() - want).abs() <= mag * (n + 1) * 2.0 ** -24).all()
"""


@pytest.mark.parametrize("rows,vocab", [(40000, 349184), (40000, 348673), (5000, 628736),
                                        (5000, 628225), (40000, 348672), (5000, 628737)])
def test_embedding_gradient_with_histograms_next_to_48_kb(rows, vocab):
    """The sort's histograms of these tables fill the 48 KB that a CTA may have without asking,
    to the last bytes.  A process of its own: an earlier call with a larger table would have asked
    already."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", NEAR_THE_DEFAULT.format(rows=rows, vocab=vocab)],
                       cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


# ---------------------------------------------------------------------- the gains' gradients
def gain_sums(x, dy, eps):
    """sum over rows and heads of dy * xhat at position 0 (where the rotation is the identity),
    and of its magnitude, in fp64."""
    x = x.double()
    xh = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    t = xh * dy.double()
    return t.sum((0, 1)), t.abs().sum((0, 1))


def gain_chain(heads, hd):
    """Additions between a summand of a gain's gradient and the result, at most: the heads that a
    lane adds one after the other (at least 4 CTAs of 4 warps per SM share them, of which a tensor
    gets at least half of its part), the heads of a warp, the 4 warps of a CTA, the partial rows (of
    at most 5 CTAs per SM) per warp of the joining CTA, its 32 warps, the old value."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    per_warp = 32 // max(1, 2 ** int(np.ceil(np.log2(hd / 16))))
    lane = 2 * -(-heads // (sms * 4 * 4 * per_warp))
    return lane + 31 + 3 + -(-sms * 5 // 32) + 31 + 1


def gain_close(got, want, mag, heads, hd):
    # a summand: the norm's factor (hd / 2 + 8), the rotation (a product that is exact at position 0
    # and a sum with zero) and two products
    bound = mag * (gain_chain(heads, hd) + hd / 2 + 12) * E + want.abs() * E
    err = (got.double() - want).abs()
    assert (err <= bound).all(), float((err - bound).max())


@pytest.mark.parametrize("rows,H,Hkv,hd,dt", [
    (3001, 28, 4, 80, "bf16"), (20011, 28, 4, 128, "bf16"), (4099, 12, 12, 96, "f32"),
    (9001, 8, 8, 10, "f32"), (2050, 32, 8, 128, "f32"), (3, 2, 1, 64, "bf16"), (700, 1, 300, 16, "bf16")])
def test_gain_gradients_lose_no_summand(rows, H, Hkv, hd, dt):
    """Sums of up to 600 thousand heads to within the roundings of their own additions: the queries
    alone (as the layer calls it), the queries with the keys, and one gain that both share."""
    g = gen(rows)
    x = {n: torch.randn(rows, h, hd, generator=g, device="cuda").to(DT[dt])
         for n, h in (("q", H), ("k", Hkv))}
    dy = {n: torch.randn(v.shape, generator=g, device="cuda") for n, v in x.items()}
    gain = (1 + 0.3 * torch.randn(hd, generator=g, device="cuda")).to(DT[dt])
    cos, sin = sbp.rope_table(1, hd, 1e4)
    want = {n: gain_sums(x[n], dy[n], 1e-6) for n in x}
    dx = {n: torch.empty_like(v) for n, v in dy.items()}

    def run(k, dq_g, dk_g):
        on = lambda t: t if k else None
        sbp.qk_norm_rope_backward(x["q"], on(x["k"]), gain, on(gain), cos, sin, 1e-6, dy["q"],
                                  on(dy["k"]), dx["q"], on(dx["k"]), dq_g, on(dk_g), seq_len=1)
    zero = lambda: torch.zeros(hd, device="cuda")
    a, b, c, shared = zero(), zero(), zero(), zero()
    run(False, a, None)
    gain_close(a, *want["q"], rows * H, hd)
    run(True, b, c)
    gain_close(b, *want["q"], rows * (H + Hkv), hd)
    gain_close(c, *want["k"], rows * (H + Hkv), hd)
    for _ in range(3):
        shared.fill_(0.0)
        run(True, shared, shared)
        gain_close(shared, want["q"][0] + want["k"][0], want["q"][1] + want["k"][1],
                   rows * (H + Hkv), hd)


# ------------------------------------------------------------- stacks of both kinds of layers
def test_stack_of_layers_with_and_without_norms():
    """bf16, head width 64: the layers without norms need the larger workspace there."""
    from memory_efficient_exact_chunk_b200 import stack
    L, T, V = S(128, 4, 2, 64, 256, 1e-6, 10000.0), 1024, 61
    layers = [layer_data(L, 1, 1, "bf16", i, norms)[0] for i, norms in enumerate((True, False))]
    cfg = sbp.layer_cfg(1, T, L.d_model, L.n_heads, L.n_kv_heads, L.head_dim, L.ffn, L.rms_eps,
                        L.rope_theta, sbp.SBP_BF16, 2)
    assert sbp.layer_workspace_size(cfg) > sbp.layer_workspace_size(cfg, True)
    table = (torch.randn(V, L.d_model, generator=gen(9), device="cuda") * 0.05).bfloat16()
    ids = torch.arange(T, device="cuda", dtype=torch.int32) * 7 % V
    w = torch.full((T,), 1.0 / T, device="cuda")
    fg = torch.ones(L.d_model, dtype=torch.bfloat16, device="cuda")
    got = [stack.stack_backward(cfg, table, order, fg, table, ids, ids, w, embed_scale=2.0)
           for order in (layers, layers[::-1])]
    for r in got:
        assert torch.isfinite(r.loss).all()
        assert all(torch.isfinite(t).all() and (t != 0).any()
                   for t in stack.grad_tensors(r.grads))


# ------------------------------------------------------------------------------------ streams
def test_workspaces_of_calls_on_another_stream():
    """While the current stream has yet to write to memory that its pool has back, a call on another
    stream without a workspace gets memory of its own."""
    rows, cols, vocab = 9000, 40, 3000
    g = gen(5)
    ids = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    dy = torch.randn(rows, cols, generator=g, device="cuda")
    want, got = torch.empty(vocab, cols, device="cuda"), torch.zeros(vocab, cols, device="cuda")
    need = sbp.embedding_scaled_backward(ids, dy, 1.5, want, accumulate=False).numel()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        torch.cuda._sleep(2_000_000)          # about a millisecond
        late = torch.empty(need, dtype=torch.uint8, device="cuda").fill_(255)
        at = late.data_ptr()
        del late
        ws = sbp.embedding_scaled_backward(ids, dy, 1.5, got, accumulate=False, stream=side)
        assert ws.data_ptr() != at
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        got.zero_()
        torch.cuda.synchronize()


def test_a_training_step_on_another_stream():
    """The whole step is on its stream: it does not wait for the current one, which is busy with
    memory that its pool has back, and its results are those of a step on the current stream."""
    from memory_efficient_exact_chunk_b200 import stack
    L, T, V = S(64, 4, 2, 16, 96, 1e-6, 10000.0), 64, 61
    W, _, _ = layer_data(L, 1, 1, "f32", 2, True)
    cfg = sbp.layer_cfg(1, T, L.d_model, L.n_heads, L.n_kv_heads, L.head_dim, L.ffn, L.rms_eps,
                        L.rope_theta, sbp.SBP_F32, 2)
    table = torch.randn(V, L.d_model, generator=gen(9), device="cuda") * 0.05
    ids = torch.arange(T, device="cuda", dtype=torch.int32) * 7 % V
    w = torch.full((T,), 1.0 / T, device="cuda")
    args = (cfg, table, [W], torch.ones(L.d_model, device="cuda"), table, ids, ids, w)
    opts = dict(embed_scale=2.0, max_grad_norm=0.05)
    want = stack.stack_backward(*args, **opts)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda._sleep(20_000_000)         # about ten milliseconds
        for n in (1 << 8, 1 << 12, 1 << 16, 1 << 20, 1 << 24):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
        got = stack.stack_backward(*args, **opts, stream=side)
        side.synchronize()
        with torch.cuda.stream(side):
            assert torch.equal(got.loss, want.loss) and torch.equal(got.grad_norm, want.grad_norm)
            for a, b in zip(stack.grad_tensors(got.grads), stack.grad_tensors(want.grads)):
                assert torch.equal(a, b)
        torch.cuda.synchronize()


# ------------------------------------------------- head widths between two powers of two lanes
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,H,Hkv,hd,layout,kind", [
    (1003, 12, 4, 72, "plain", "any"), (515, 7, 3, 72, "fused", "outside"),
    (31, 6, 2, 72, "odd", None), (1777, 5, 1, 88, "plain", "any"), (2, 1, 11, 88, "fused", "outside"),
    (64, 32, 8, 88, "plain", 64), (1, 1, 1, 88, "plain", None), (1, 1, 1, 72, "plain", None),
    (77, 3, 1, 66, "plain", None), (77, 3, 1, 94, "fused", "any"), (130, 4, 2, 104, "plain", 65),
    (130, 4, 2, 136, "plain", None), (77, 5, 1, 160, "fused", "any")])
def test_qk_norm_rope_of_widths_between(rows, H, Hkv, hd, layout, kind, dt):
    """Widths whose heads share a warp in sixes, fives and, off the vector grid or wider, in powers of
    two, against the definition in 64 bits with the bounds of the other widths."""
    from tests import test_gpu_step_ops as ops
    ops.test_qk_norm_rope_forward(rows, H, Hkv, hd, dt, layout, kind)
    ops.test_qk_norm_rope_backward(rows, H, Hkv, hd, dt, layout, kind)


# --------------------------------------------------------- gains of a bf16 layer, few summands
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("H,Hkv,B,T,D", [(1, 1, 1, 2, 2), (1, 1, 1, 2, 1), (2, 1, 1, 2, 2),
                                         (1, 1, 1, 3, 3), (1, 1, 2, 2, 2), (2, 2, 1, 3, 2)])
def test_bf16_gain_gradients_of_few_summands(H, Hkv, B, T, D, reverse):
    """The upstream gradient reaches the last token alone, so a gain's gradient is a sum of few
    products that hardly cancel (which is asserted), and rows of another chunk or of another
    rounding would show.  A summand passes ten roundings to bf16 on its way (n1, the projection,
    q, k, v, dy, dh, dO, O, and P or dS), of 2^-8 at most each: 5e-2 of the summands' magnitudes,
    a tenth of the result."""
    from tests import test_gpu_step_layer as layer
    L = S(256, H, Hkv, 128, 512, 1e-6, 10000.0)
    W = layer.make_layer(L, 10 * T + D + H, "bf16")
    g = gen(100 * B + 10 * T + H)
    x = torch.randn(B, T, L.d_model, generator=g, device="cuda").bfloat16()
    dy = torch.zeros(B, T, L.d_model, device="cuda")
    dy[:, -1] = torch.randn(B, L.d_model, generator=g, device="cuda") * 1e-3
    _, _, want, mags = layer.ref_backward(L, W, x, dy)
    _, _, got = layer.gpu_backward(L, W, x, dy, D, reverse)
    for n in sbp.QK_NORM_FIELDS:
        assert mags[n] <= 2 * float(want[n].norm()), n
        assert float((got[n].double() - want[n]).norm()) <= 5e-2 * mags[n], n
