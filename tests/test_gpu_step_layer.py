"""The decoder layer with per-head query/key norms, and a training step of a small stack that uses
every operator of include/sbp_step.h (scaled embedding, normed layers, clipping), against plain
definitions in 64 bits differentiated by torch.autograd.

Tolerances are those of the layer without norms: relative Frobenius 1e-5 (fp32), 1e-2 (bf16) per
tensor, D = 1 against D > 1 within 1e-5.  The gains' gradients are sums over tokens and heads with
cancellation; in bf16 they are held against the norm of the sum of the summands' magnitudes, the
error scale of a rounded sum."""
import numpy as np
import pytest
import torch

from memory_efficient_exact_chunk_b200 import dp, sbp, stack, synth
from tests.helpers import rel_fro, to_np

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {"f32": 1e-5, "bf16": 1e-2}


def make_layer(L, seed, dtype):
    rng = np.random.default_rng(seed)
    W = synth.layer_weights(rng, L, dtype == "bf16", gamma_std=0.1)
    for n in sbp.QK_NORM_FIELDS:
        g = 1.0 + 0.3 * rng.standard_normal(L.head_dim, dtype=np.float32)
        W[n] = synth.bf16_round(g) if dtype == "bf16" else g
    return {n: None if v is None else torch.from_numpy(v).to(DT[dtype]).cuda()
            for n, v in W.items()}


def rms(x, g, eps):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * g


def ref_layer(L, W, x, terms=None):
    """The layer's definition; W and x fp64.  terms (a list) collects what the gains multiply."""
    B, T, _ = x.shape
    H, Hkv, hd = L.n_heads, L.n_kv_heads, L.head_dim

    def lin(v, n, b=None):
        y = v @ W[n].t()
        return y if b is None or W.get(b) is None else y + W[b]
    n1 = rms(x, W["ln1_g"], L.rms_eps)
    q = lin(n1, "wq", "bq").view(B, T, H, hd)
    k = lin(n1, "wk", "bk").view(B, T, Hkv, hd)
    v = lin(n1, "wv", "bv").view(B, T, Hkv, hd)
    inv = L.rope_theta ** (-torch.arange(0, hd, 2, dtype=torch.float64, device=x.device) / hd)
    ang = torch.arange(T, dtype=torch.float64, device=x.device)[:, None] * inv
    # the library's tables are the fp64 angles' cosines rounded to fp32
    turn = torch.complex(ang.cos().float().double(), ang.sin().float().double())[:, None]

    def normed(y, g):
        y = y / (y.square().mean(-1, keepdim=True) + L.rms_eps).sqrt() * g
        if terms is not None:
            y.retain_grad()
            terms.append(y)
        z = torch.complex(y[..., :hd // 2].contiguous(), y[..., hd // 2:].contiguous()) * turn
        return torch.cat((z.real, z.imag), -1)
    q, k = normed(q, W["q_norm_g"]), normed(k, W["k_norm_g"])
    kk = k.repeat_interleave(H // Hkv, 2)
    vv = v.repeat_interleave(H // Hkv, 2)
    s = torch.einsum("bthd,bshd->bhts", q, kk) / hd ** 0.5
    s = s.masked_fill(torch.triu(torch.ones(T, T, dtype=torch.bool, device=x.device), 1),
                      float("-inf"))
    a = torch.einsum("bhts,bshd->bthd", s.softmax(-1), vv).reshape(B, T, H * hd)
    h = x + lin(a, "wo")
    n2 = rms(h, W["ln2_g"], L.rms_eps)
    return h + (torch.nn.functional.silu(lin(n2, "w_gate")) * lin(n2, "w_up")) @ W["w_down"].t()


def ref_backward(L, W, x, dy):
    W64 = {n: None if v is None else v.double().requires_grad_() for n, v in W.items()}
    x64 = x.double().requires_grad_()
    terms = []
    y = ref_layer(L, W64, x64, terms)
    y.backward(dy.double())
    mags = {}
    for n, t in zip(sbp.QK_NORM_FIELDS, terms):     # |u * xhat| summed over tokens and heads
        mags[n] = float((t.grad * (t / W64[n]).detach()).abs().sum((0, 1, 2)).norm())
    return y.detach(), x64.grad, {n: v.grad for n, v in W64.items() if v is not None}, mags


def gpu_backward(L, W, x, dy, D, reverse=False):
    B, T, d = x.shape
    code = sbp.SBP_BF16 if x.dtype == torch.bfloat16 else sbp.SBP_F32
    cfg = sbp.layer_cfg(B, T, d, L.n_heads, L.n_kv_heads, L.head_dim, L.ffn, L.rms_eps,
                        L.rope_theta, code, D)
    y = torch.full_like(x, float("nan"))
    sbp.device_status(sbp.decoder_layer_forward(cfg, W, x, y))
    dx = torch.full(x.shape, float("nan"), device="cuda")
    g = {n: None if v is None else torch.zeros(v.shape, device="cuda") for n, v in W.items()}
    run = sbp.decoder_layer_backward_reverse if reverse else sbp.decoder_layer_backward
    sbp.device_status(run(cfg, W, x, dy, dx, g))
    return y, dx, {n: v for n, v in g.items() if v is not None}


S = synth.LayerShape
CASES = [  # shape, batch, tokens, chunks, dtype
    (S(64, 4, 2, 16, 96, 1e-6, 10000.0), 1, 37, 3, "f32"),
    (S(64, 4, 4, 16, 172, 1e-6, 10000.0, qkv_bias=True), 2, 40, 4, "f32"),
    (S(48, 6, 3, 10, 40, 1e-5, 500000.0), 1, 1, 1, "f32"),
    (S(48, 6, 3, 10, 40, 1e-5, 500000.0), 3, 23, 23, "f32"),
    (S(256, 4, 2, 128, 512, 1e-5, 500000.0), 1, 300, 5, "bf16"),
    (S(256, 4, 1, 128, 512, 1e-6, 1000000.0, qkv_bias=True), 2, 131, 2, "bf16"),
    (S(128, 4, 2, 64, 256, 1e-6, 10000.0), 2, 70, 3, "bf16"),
]


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("L,B,T,D,dtype", CASES)
def test_layer_with_qk_norm(L, B, T, D, dtype, reverse):
    W = make_layer(L, T + D, dtype)
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(B, T, L.d_model, generator=gen, device="cuda").to(DT[dtype])
    dy = torch.randn(B, T, L.d_model, generator=gen, device="cuda") * 1e-3
    y0, dx0, g0, mags = ref_backward(L, W, x, dy)
    y, dx, g = gpu_backward(L, W, x, dy, D, reverse)
    assert rel_fro(to_np(y), y0.cpu().numpy()) <= TOL[dtype]
    assert rel_fro(to_np(dx), dx0.cpu().numpy()) <= TOL[dtype]
    assert set(g) == {n for n, v in W.items() if v is not None}
    for n, v in g.items():
        if dtype == "bf16" and n in mags:
            assert float((v.double() - g0[n]).norm()) <= TOL[dtype] * mags[n], n
        elif dtype == "bf16" and n == "bk":
            # the stated exception of the layer without norms: a column sum with cancellation
            assert rel_fro(to_np(v), g0[n].cpu().numpy()) <= 5e-2
        else:
            assert rel_fro(to_np(v), g0[n].cpu().numpy()) <= TOL[dtype], n


def test_layer_with_qk_norm_does_not_depend_on_the_chunks():
    L = S(256, 4, 2, 128, 512, 1e-5, 500000.0)
    W = make_layer(L, 7, "bf16")
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(1, 512, 256, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(1, 512, 256, generator=gen, device="cuda") * 1e-3
    y1, dx1, g1 = gpu_backward(L, W, x, dy, 1)
    for D, reverse in ((4, False), (4, True), (2, False)):
        y, dx, g = gpu_backward(L, W, x, dy, D, reverse)
        assert torch.equal(y, y1)
        assert rel_fro(to_np(dx), to_np(dx1)) <= 1e-5
        for n in g:
            assert rel_fro(to_np(g[n]), to_np(g1[n])) <= 1e-5, n


def test_layer_qk_norm_refusals():
    L = S(64, 4, 2, 16, 96, 1e-6, 10000.0)
    W = make_layer(L, 1, "f32")
    x = torch.zeros(1, 8, 64, device="cuda")
    cfg = sbp.layer_cfg(1, 8, 64, 4, 2, 16, 96, 1e-6, 1e4, sbp.SBP_F32, 2)
    with pytest.raises(ValueError, match="both"):
        sbp.decoder_layer_forward(cfg, {**W, "k_norm_g": None}, x, torch.empty_like(x))
    with pytest.raises(ValueError, match="shape"):
        sbp.decoder_layer_forward(cfg, {**W, "k_norm_g": torch.ones(8, device="cuda")}, x,
                                  torch.empty_like(x))
    with pytest.raises(TypeError):
        sbp.decoder_layer_forward(cfg, {**W, "q_norm_g": W["q_norm_g"].bfloat16()}, x,
                                  torch.empty_like(x))
    g = {n: None if v is None else torch.zeros_like(v) for n, v in W.items()}
    with pytest.raises(ValueError, match="missing"):
        sbp.decoder_layer_backward(cfg, W, x, x, torch.empty_like(x), {**g, "q_norm_g": None})
    small = sbp.workspace(sbp.layer_workspace_size(cfg))
    assert sbp.layer_workspace_size(cfg, True) > small.numel()
    with pytest.raises(sbp.SbpError) as e:
        sbp.decoder_layer_forward(cfg, W, x, torch.empty_like(x), ws=small)
    assert e.value.code == 3


def make_stack(dtype, n_layers, B, T, seed=5):
    L = S(64, 4, 2, 16, 96, 1e-6, 10000.0) if dtype == "f32" else \
        S(256, 4, 2, 128, 512, 1e-5, 500000.0)
    V = 61
    rng = np.random.default_rng(seed)

    def dev(*s):
        a = torch.from_numpy(rng.standard_normal(s, dtype=np.float32) * np.float32(0.05))
        return a.to(DT[dtype]).cuda()
    layers = [make_layer(L, seed + i, dtype) for i in range(n_layers)]
    ids = torch.from_numpy(rng.integers(0, V, B * T).astype(np.int32)).cuda()
    ids[::7] = 3                                       # a frequent token
    targets = torch.from_numpy(rng.integers(0, V, B * T).astype(np.int32)).cuda()
    w = torch.full((B * T,), 1.0 / (B * T), device="cuda")
    w[:5] = 0.0
    fg = torch.ones(L.d_model, dtype=DT[dtype], device="cuda")
    code = sbp.SBP_BF16 if dtype == "bf16" else sbp.SBP_F32
    cfg = sbp.layer_cfg(B, T, L.d_model, L.n_heads, L.n_kv_heads, L.head_dim, L.ffn, L.rms_eps,
                        L.rope_theta, code, 3)
    return L, cfg, dev(V, L.d_model), layers, fg, dev(V, L.d_model), ids, targets, w


def ref_stack(L, cfg, embed, layers, fg, lm, ids, targets, w, scale):
    leaves = {"embed": embed, "final_g": fg, "lm_head": lm}
    leaves = {n: v.double().requires_grad_() for n, v in leaves.items()}
    Ws = [{n: None if v is None else v.double().requires_grad_() for n, v in W.items()}
          for W in layers]
    x = (leaves["embed"][ids.long()] * scale).view(cfg.batch, cfg.seq_len, -1)
    for W in Ws:
        x = ref_layer(L, W, x)
    hf = rms(x, leaves["final_g"], L.rms_eps).view(-1, L.d_model)
    ce = torch.nn.functional.cross_entropy(hf @ leaves["lm_head"].t(), targets.long(),
                                           reduction="none")
    loss = (ce * w.double()).sum()
    loss.backward()
    return float(loss), {**{n: v.grad for n, v in leaves.items()},
                         "layers": [{n: v.grad for n, v in W.items() if v is not None}
                                    for W in Ws]}


@pytest.mark.parametrize("dtype,B,T", [("f32", 2, 45), ("bf16", 1, 200)])
def test_training_step_with_every_operator(dtype, B, T):
    args = make_stack(dtype, 2, B, T)
    L, cfg, embed, layers, fg, lm, ids, targets, w = args
    scale, max_norm = L.d_model ** 0.5, 0.05
    loss0, g0 = ref_stack(*args, scale)
    norm0 = float(sum(t.square().sum() for t in stack.grad_tensors(g0)) ** 0.5)
    assert norm0 > max_norm                              # the clipping bites
    keep = {}
    res = stack.stack_backward(cfg, embed, layers, fg, lm, ids, targets, w, keep_workspace=keep,
                               embed_scale=scale, max_grad_norm=max_norm)
    tol = TOL[dtype]
    assert abs(float(res.loss) - loss0) <= tol * abs(loss0)
    assert abs(float(res.grad_norm) - norm0) <= tol * norm0
    coef = max_norm / (norm0 + 1e-6)
    total = 0.0
    got, want = stack.grad_tensors(res.grads), stack.grad_tensors(g0)
    assert len(got) == len(want) == 3 + 2 * (9 + 2)
    for a, b in zip(got, want):
        assert a.shape == b.shape
        total += float(a.double().square().sum())
        if a.shape == (L.head_dim,) and dtype == "bf16":
            continue               # the gains' gradients: see test_layer_with_qk_norm
        assert rel_fro(to_np(a), (b * coef).cpu().numpy()) <= 2 * tol
    assert total ** 0.5 <= max_norm * (1 + 1e-5)
    again = stack.stack_backward(cfg, embed, layers, fg, lm, ids, targets, w,
                                 keep_workspace=keep, embed_scale=scale, max_grad_norm=max_norm)
    assert torch.equal(again.grads["embed"], res.grads["embed"])


def test_sharded_clipping_of_one_replica():
    """dp.dp_stack_step with scaled embedding and normed layers, then clip_sharded, equals the
    stack's own clipping."""
    L, cfg, embed, layers, fg, lm, ids, targets, w = make_stack("f32", 2, 1, 45)
    plan = dp.stack_buckets(layers, lm.shape, fg.shape, embed.shape)
    assert any(n == "q_norm_g" for _, ts in plan for n, _ in ts)
    g = dp.ShardedGrads(plan, 1, 0, "cuda")
    dp.dp_stack_step(cfg, embed, layers, fg, lm, ids, targets, w, g, dp.GradReducer(g),
                     embed_scale=8.0)
    norm = dp.clip_sharded(g, 0.05)
    res = stack.stack_backward(cfg, embed, layers, fg, lm, ids, targets, w, embed_scale=8.0,
                               max_grad_norm=0.05)
    assert abs(float(norm) - float(res.grad_norm)) <= 1e-6 * float(norm)
    off = g.offsets["layer1"]["q_norm_g"]
    mine = g.out["layer1"][off:off + L.head_dim]
    assert rel_fro(to_np(mine), to_np(res.grads["layers"][1]["q_norm_g"])) <= 1e-6
    assert rel_fro(to_np(g.out["embed"][:embed.numel()].view(embed.shape)),
                   to_np(res.grads["embed"])) <= 1e-6
