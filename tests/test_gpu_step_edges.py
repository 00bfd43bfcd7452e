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
