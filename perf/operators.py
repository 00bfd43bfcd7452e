"""Timed cases of the operators that stand around the streamed backward: the scaled embedding
and its gradient by sorted tokens, the per-head norm of queries and keys with RoPE in the same
pass, and the global gradient norm with clipping.

`own` False computes an operator from elementary torch operations in 32 bits, True calls the
framework.  `exact` restates each operator from its definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

#: Elements between the tensors of a flat gradient bucket (256 bytes, the layout of the
#: data-parallel buckets).
ALIGN = 64
#: Added to the norm before the division, so that a zero gradient is not divided by zero.
CLIP_EPS = 1e-6


# ------------------------------------------------------------------------------------- cases
def _embed(name, op, rows, cols, vocab, dt, ids="zipf", pad=0.0, scale=None):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "vocab": vocab, "dt": dt,
            "ids": ids, "pad": pad, "scale": float(scale or math.sqrt(cols))}


def _qk(name, op, rows, heads, kv_heads, hd, dt, seq_len, theta, eps, fused=True, packed=False):
    return {"name": name, "op": op, "rows": rows, "heads": heads, "kv_heads": kv_heads,
            "head_dim": hd, "dt": dt, "seq_len": seq_len, "theta": theta, "eps": eps,
            "fused": fused, "packed": packed}


def _clip(name, sizes, max_norm, out, tensors=0, total=0, shape_seed=0):
    return {"name": name, "op": "clip", "sizes": sizes, "tensors": tensors, "total": total,
            "shape_seed": shape_seed, "max_norm": max_norm, "out": out}


def listed():
    return [
        # token embedding of one 64K-token sequence of the Llama-3-8B-shaped stack
        _embed("embed_forward_64k", "embed_forward", 65536, 4096, 128256, "bf16"),
        # the tiny fp32 model's 256 tokens: a call whose launch is all it costs
        _embed("embed_forward_tiny", "embed_forward", 256, 64, 512, "f32", ids="uniform"),
        # its gradient at 64K tokens, written over the whole table: the largest case
        _embed("embed_backward_64k", "embed_backward", 65536, 4096, 128256, "bf16"),
        # a ragged batch: a third of the rows is padding, which no table row receives
        _embed("embed_backward_padded", "embed_backward", 20001, 3584, 152064, "bf16", pad=0.33),
        # the tiny fp32 model's gradient
        _embed("embed_backward_tiny", "embed_backward", 256, 64, 512, "f32", ids="uniform"),
        # one 4096-token chunk of the 64K stack at D = 16, out of the fused projection
        _qk("qk_forward_chunk", "qk_forward", 4096, 32, 8, 128, "bf16", 4096, 500000.0, 1e-5),
        # the tiny fp32 model's chunk of 64 tokens at D = 4
        _qk("qk_forward_tiny", "qk_forward", 64, 4, 4, 16, "f32", 64, 10000.0, 1e-6),
        # a chunk of the GRPO batch: 8 sequences of 16384 at D = 8, Qwen2.5-7B heads
        _qk("qk_backward_batch", "qk_backward", 16384, 28, 4, 128, "bf16", 2048, 1000000.0, 1e-6),
        # packed sequences of odd lengths, heads whose halves are no power of two, fp32
        _qk("qk_backward_packed", "qk_backward", 1003, 12, 12, 80, "f32", 1003, 10000.0, 1e-6,
            fused=False, packed=True),
        # the weight gradients of one Llama-3-8B-shaped layer, clipped into the optimizer's copy
        _clip("clip_layer", "llama_layer", 1.0, True),
        # the tiny model's gradients, under the limit: nothing has to be written
        _clip("clip_tiny", "tiny_stack", 1000.0, False),
        # many tensors of very uneven sizes
        _clip("clip_ragged", "ragged", 0.5, True, tensors=300, total=30_000_000, shape_seed=1),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed_forward", "embed_backward", "embed_backward", "qk_forward",
                     "qk_backward", "clip"])
    if op.startswith("embed"):
        dt = rng.choice(["bf16", "bf16", "f32"])
        rows = _log_int(rng, 1, 65536)
        vocab = _log_int(rng, 512, 152064)
        cols = _log_int(rng, 64, 4096)
        if rng.random() < 0.7:
            cols = (cols + 7) // 8 * 8
        c = _embed("", op, rows, cols, vocab, dt, ids=rng.choice(["zipf", "uniform"]),
                   pad=rng.choice([0.0, 0.0, round(rng.uniform(0.05, 0.6), 3)]),
                   scale=round(rng.uniform(0.1, 70.0), 3))
    elif op.startswith("qk"):
        hd = rng.choice([16, 32, 64, 80, 96, 128, 128, 128, 256, 2 * rng.randint(1, 128)])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 7])
        rows = _log_int(rng, 1, 24576)
        seq = rng.choice([rows, max(1, rows // rng.randint(1, 8))])
        c = _qk("", op, rows, heads, kv, hd, rng.choice(["bf16", "bf16", "f32"]), seq,
                rng.choice([10000.0, 500000.0, 1000000.0]), rng.choice([1e-5, 1e-6]),
                fused=rng.random() < 0.5, packed=rng.random() < 0.5)
    else:
        n = _log_int(rng, 1, 600)
        c = _clip("", "ragged", rng.choice([0.25, 1.0, 1e9]), rng.random() < 0.7, tensors=n,
                  total=max(n, _log_int(rng, 1, 200_000_000)), shape_seed=rng.randrange(1 << 30))
        if not c["out"]:
            c["max_norm"] = 1e9      # in place: repeated passes see the same gradients
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _dtype(case):
    return torch.bfloat16 if case["dt"] == "bf16" else torch.float32


def _id_probs(case):
    v = np.arange(case["vocab"], dtype=np.float64)
    p = 1.0 / (v + 2.7) if case["ids"] == "zipf" else np.ones_like(v)
    return p / p.sum()


def _make_ids(case, g):
    """Token ids: low ids are the frequent ones, as a byte-pair vocabulary numbers them; a
    share `pad` of the rows is padding, marked -1."""
    n = case["rows"]
    cdf = torch.from_numpy(np.cumsum(_id_probs(case))).cuda()
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    ids = torch.searchsorted(cdf, u).clamp_(max=case["vocab"] - 1).to(torch.int32)
    if case["pad"]:
        ids[torch.rand(n, generator=g, device="cuda") < case["pad"]] = -1
    return ids


def _sizes(case):
    """Element counts of the gradient tensors."""
    if case["sizes"] == "llama_layer":
        d, kv, f = 4096, 1024, 14336
        return [d, d * d, kv * d, kv * d, d * d, d, f * d, f * d, d * f]
    if case["sizes"] == "tiny_stack":
        d, f, v = 64, 172, 512
        return [v * d, d, d, d * d, d * d, d * d, d * d, d, f * d, f * d, d * f, v * d]
    r = random.Random(case["shape_seed"])
    w = [math.exp(r.uniform(0.0, 9.0)) for _ in range(case["tensors"])]
    return [max(1, int(case["total"] * x / sum(w))) for x in w]


def _prepare_embed(case, g):
    rows, cols, vocab = case["rows"], case["cols"], case["vocab"]
    s = {"ids": _make_ids(case, g), "scale": case["scale"]}
    if case["op"] == "embed_forward":
        s["table"] = (torch.randn(vocab, cols, generator=g, device="cuda") * 0.02).to(_dtype(case))
        s["y"] = torch.empty(rows, cols, dtype=_dtype(case), device="cuda")
    else:
        s["dy"] = torch.randn(rows, cols, generator=g, device="cuda") * 1e-3
        s["d_table"] = torch.empty(vocab, cols, device="cuda")
    return s


def _prepare_qk(case, g):
    rows, H, Hkv, hd = case["rows"], case["heads"], case["kv_heads"], case["head_dim"]
    dt = _dtype(case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["fused"]:        # queries, keys and values side by side, as one projection leaves them
        x = randn(rows, H + 2 * Hkv, hd).to(dt)
        q, k = x[:, :H], x[:, H:H + Hkv]
    else:
        q, k = randn(rows, H, hd).to(dt), randn(rows, Hkv, hd).to(dt)
    s = {"q": q, "k": k, "eps": case["eps"], "seq_len": case["seq_len"], "positions": None,
         "q_g": (1.0 + 0.1 * randn(hd)).to(dt), "k_g": (1.0 + 0.1 * randn(hd)).to(dt)}
    table = case["seq_len"]
    if case["packed"]:       # sequences of odd lengths one after the other
        cuts = torch.rand(rows, generator=g, device="cuda") < 5.0 / max(rows, 5)
        at = torch.arange(rows, device="cuda")
        s["positions"] = (at - torch.where(cuts, at, 0).cummax(0).values).to(torch.int32)
        table = rows
    inv = case["theta"] ** (-torch.arange(0, hd, 2, device="cuda", dtype=torch.float64) / hd)
    ang = torch.arange(table, device="cuda", dtype=torch.float64)[:, None] * inv[None, :]
    s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    if case["op"] == "qk_forward":
        s["q_out"] = torch.empty(rows, H, hd, dtype=dt, device="cuda")
        s["k_out"] = torch.empty(rows, Hkv, hd, dtype=dt, device="cuda")
    else:
        s["dq_out"], s["dk_out"] = randn(rows, H, hd) * 1e-3, randn(rows, Hkv, hd) * 1e-3
        s["dq"], s["dk"] = torch.empty_like(s["dq_out"]), torch.empty_like(s["dk_out"])
        s["dg"] = torch.zeros(2, max(hd, 4) + 3 & ~3, device="cuda")   # both gains' gradients
    return s


def _prepare_clip(case, g):
    sizes, at = _sizes(case), 0
    views = []
    for n in sizes:
        views.append((at, n))
        at += (n + ALIGN - 1) // ALIGN * ALIGN
    flat = torch.zeros(at, device="cuda")
    r = random.Random(g.initial_seed())
    for o, n in views:
        flat[o:o + n].normal_(generator=g)
        flat[o:o + n].mul_(1e-3 * math.exp(r.uniform(-2.0, 2.0)))
    s = {"flat": flat, "max_norm": case["max_norm"], "norm": torch.empty(1, device="cuda"),
         "out": torch.zeros_like(flat) if case["out"] else None}
    if own:      # the list of gradients that a training program keeps from step to step
        from memory_efficient_exact_chunk_b200 import sbp
        s["grads"] = sbp.GradList([flat[o:o + n] for o, n in views])
        s["into"] = sbp.GradList([s["out"][o:o + n] for o, n in views]) if case["out"] else None
    return s


def prepare(case, seed):
    g = _generator(seed)
    if case["op"].startswith("embed"):
        s = _prepare_embed(case, g)
    elif case["op"].startswith("qk"):
        s = _prepare_qk(case, g)
    else:
        s = _prepare_clip(case, g)
    s["op"] = case["op"]
    return s


# --------------------------------------------------------------------------------- plain forms
def _plain_embed_forward(s):
    ids, table = s["ids"], s["table"]
    ok = (ids >= 0) & (ids < table.shape[0])
    rows = table[torch.where(ok, ids, 0).long()].float() * s["scale"]
    return (rows * ok[:, None]).to(table.dtype)


def _plain_embed_backward(s):
    ids, vocab = s["ids"], s["d_table"].shape[0]
    keep = ((ids >= 0) & (ids < vocab)).nonzero()[:, 0]
    out = torch.zeros_like(s["d_table"])
    return out.index_add_(0, ids[keep].long(), s["dy"][keep] * s["scale"])


def _angles(s, rows):
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(rows, device="cuda") % s["seq_len"]
    return s["cos"][pos.long()][:, None, :], s["sin"][pos.long()][:, None, :]


def _plain_norm_rope(x, g, c, sn, eps):
    h = x.float()
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + eps) * g.float()
    half = x.shape[-1] // 2
    a, b = n[..., :half], n[..., half:]
    return torch.cat((a * c - b * sn, b * c + a * sn), -1).to(x.dtype)


def _plain_norm_rope_backward(x, g, c, sn, eps, dy):
    h, half = x.float(), x.shape[-1] // 2
    a, b = dy[..., :half], dy[..., half:]
    u = torch.cat((a * c + b * sn, b * c - a * sn), -1)
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + eps)
    xh, v = h * r, u * g.float()
    return r * (v - xh * (xh * v).mean(-1, keepdim=True)), (u * xh).sum((0, 1))


def _plain_clip(s):
    norm = s["flat"].square().sum().sqrt()
    coef = (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    return [norm[None], s["flat"] * coef]


def _run_plain(s):
    if s["op"] == "embed_forward":
        return _plain_embed_forward(s)
    if s["op"] == "embed_backward":
        return _plain_embed_backward(s)
    if s["op"] == "clip":
        return _plain_clip(s)
    c, sn = _angles(s, s["q"].shape[0])
    if s["op"] == "qk_forward":
        return [_plain_norm_rope(s["q"], s["q_g"], c, sn, s["eps"]),
                _plain_norm_rope(s["k"], s["k_g"], c, sn, s["eps"])]
    dq, dq_g = _plain_norm_rope_backward(s["q"], s["q_g"], c, sn, s["eps"], s["dq_out"])
    dk, dk_g = _plain_norm_rope_backward(s["k"], s["k_g"], c, sn, s["eps"], s["dk_out"])
    return [dq, dk, dq_g, dk_g]


# ----------------------------------------------------------------------------- the framework's
def _run_own(s):
    from memory_efficient_exact_chunk_b200 import sbp
    op = s["op"]
    if op == "embed_forward":
        sbp.embedding_scaled_forward(s["ids"], s["table"], s["scale"], s["y"])
        return s["y"]
    if op == "embed_backward":
        s["ws"] = sbp.embedding_scaled_backward(s["ids"], s["dy"], s["scale"], s["d_table"],
                                                accumulate=False, ws=s.get("ws"))
        return s["d_table"]
    if op == "clip":
        s["ws"] = sbp.grad_clip_norm(s["grads"], s["max_norm"], s["norm"], out=s["into"],
                                     ws=s.get("ws"))
        return [s["norm"], s["flat"] if s["out"] is None else s["out"]]
    if op == "qk_forward":
        sbp.qk_norm_rope_forward(s["q"], s["k"], s["q_g"], s["k_g"], s["cos"], s["sin"],
                                 s["eps"], s["q_out"], s["k_out"], positions=s["positions"],
                                 seq_len=s["seq_len"])
        return [s["q_out"], s["k_out"]]
    hd = s["q"].shape[-1]
    dg = s["dg"].zero_()      # weight gradients are accumulated
    s["ws"] = sbp.qk_norm_rope_backward(s["q"], s["k"], s["q_g"], s["k_g"], s["cos"], s["sin"],
                                        s["eps"], s["dq_out"], s["dk_out"], s["dq"], s["dk"],
                                        dg[0, :hd], dg[1, :hd], positions=s["positions"],
                                        seq_len=s["seq_len"], ws=s.get("ws"))
    return [s["dq"], s["dk"], dg[0, :hd], dg[1, :hd]]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------- work and definition
def work(case):
    es = 2 if case.get("dt") == "bf16" else 4
    if case["op"].startswith("embed"):
        rows, cols, vocab = case["rows"], case["cols"], case["vocab"]
        valid = rows * (1.0 - case["pad"])
        if case["op"] == "embed_forward":   # the distinct table rows, the ids, the output
            used = float((1.0 - (1.0 - _id_probs(case)) ** valid).sum())
            return {"bytes": 4 * rows + (used + rows) * cols * es, "flops": rows * cols}
        return {"bytes": 4 * rows + 4 * valid * cols + 4 * vocab * cols,
                "flops": 2 * valid * cols}
    if case["op"] == "clip":
        n = sum(_sizes(case))
        writes = n if case["out"] or case["max_norm"] < 1e3 else 0
        return {"bytes": 4 * (n + writes), "flops": 3 * n}
    rows, hd = case["rows"], case["head_dim"]
    n = rows * (case["heads"] + case["kv_heads"]) * hd
    table = 4 * min(rows, case["seq_len"] if not case["packed"] else rows) * hd
    if case["op"] == "qk_forward":
        return {"bytes": 2 * n * es + table + 2 * hd * es, "flops": 8 * n}
    return {"bytes": n * es + 8 * n + table + 2 * hd * (es + 4), "flops": 18 * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed_forward":
        t = torch.cat((s["table"].double(), torch.zeros(1, case["cols"], dtype=torch.float64,
                                                        device="cuda")))   # the padding row
        return torch.nn.functional.embedding(s["ids"].long() % (case["vocab"] + 1), t) * s["scale"]
    if case["op"] == "embed_backward":
        # products with the one-hot matrix of a few thousand rows at a time
        out = torch.zeros(case["vocab"] + 1, case["cols"], dtype=torch.float64, device="cuda")
        ids = s["ids"].long() % (case["vocab"] + 1)
        for at in range(0, case["rows"], 4096):
            part = ids[at:at + 4096]
            names, where = part.unique(return_inverse=True)
            hot = torch.zeros(len(names), len(part), dtype=torch.float64, device="cuda")
            hot[where, torch.arange(len(part), device="cuda")] = 1.0
            out[names] += hot @ s["dy"][at:at + 4096].double()
        return out[:-1] * s["scale"]
    if case["op"] == "clip":
        f = s["flat"].double()
        norm = torch.linalg.vector_norm(f)
        f *= min(1.0, case["max_norm"] / (float(norm) + CLIP_EPS))
        return [norm[None], f]
    rows, hd = case["rows"], case["head_dim"]
    pos = (torch.arange(rows, device="cuda") % case["seq_len"] if s["positions"] is None
           else s["positions"].long())
    turn = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None, :]

    def head(x, g):      # pairs (j, j + hd / 2) as complex numbers, turned by the position
        n = x / (x.square().sum(-1, keepdim=True) / hd + case["eps"]).sqrt() * g
        z = torch.complex(n[..., :hd // 2].contiguous(), n[..., hd // 2:].contiguous()) * turn
        return torch.cat((z.real, z.imag), -1)

    outs = []
    for x, g in (("q", "q_g"), ("k", "k_g")):
        x64, g64 = s[x].double().requires_grad_(), s[g].double().requires_grad_()
        y = head(x64, g64)
        if case["op"] == "qk_forward":
            outs.append(y.detach())
        else:
            outs.append(torch.autograd.grad(y, (x64, g64), s["d%s_out" % x].double()))
    return outs if case["op"] == "qk_forward" else [outs[0][0], outs[1][0], outs[0][1],
                                                    outs[1][1]]
