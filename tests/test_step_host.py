"""Refusals of the operators of include/sbp_step.h: everything here returns before any launch,
so no GPU is needed."""
import ctypes as C

import pytest
import torch

from memory_efficient_exact_chunk_b200 import build as sbp_build
from memory_efficient_exact_chunk_b200 import sbp

FAKE = 0x100000  # an aligned address that is never dereferenced (argument checks fail first)
OK_WS = 1 << 40


@pytest.fixture(scope="module")
def lib():
    sbp_build.build()
    return sbp.load()


def test_embedding_scaled_refusals(lib):
    def fwd(rows=8, cols=16, vocab=32, dt=1, ids=FAKE, table=FAKE, y=FAKE):
        return lib.sbp_embedding_scaled_forward(rows, cols, vocab, dt, 2.0, ids, table, y, None)

    def bwd(rows=8, cols=16, vocab=32, ids=FAKE, dy=FAKE, dt=FAKE, ws=FAKE, wsb=OK_WS):
        return lib.sbp_embedding_scaled_backward(rows, cols, vocab, 2.0, ids, dy, dt, 0, ws, wsb,
                                                 None)
    for bad in (dict(rows=0), dict(rows=-1), dict(cols=0), dict(vocab=0), dict(ids=None),
                dict(ids=FAKE + 4)):
        assert fwd(**bad) == 1 and bwd(**bad) == 1, bad
    assert fwd(dt=2) == 1 and fwd(table=None) == 1 and fwd(y=FAKE + 2) == 1
    assert bwd(dy=None) == 1 and bwd(dt=FAKE + 8) == 1 and bwd(ws=None) == 1
    assert bwd(ws=FAKE + 16) == 1 and bwd(wsb=8) == 3
    for bad in (dict(rows=1 << 30), dict(vocab=(1 << 22) + 1), dict(cols=1 << 30)):
        assert fwd(**bad) == 2 and bwd(**bad) == 2, bad
    size = lib.sbp_embedding_scaled_backward_workspace_size
    assert size(8, 16, 32) > 0 and size(0, 16, 32) == 0 and size(8, 16, 1 << 23) == 0
    assert size(1 << 16, 4096, 128256) > size(1 << 15, 4096, 128256)
    assert bwd(rows=1 << 16, wsb=size(1 << 16, 16, 32) - 1) == 3


def _qk_fwd(lib, rows=4, H=4, Hkv=2, hd=16, seq=4, table=8, eps=1e-6, dt=1, q=FAKE, ldq=64,
            k=FAKE, ldk=32, qg=FAKE, kg=FAKE, pos=None, cos=FAKE, sin=FAKE, qo=FAKE, ldqo=64,
            ko=FAKE, ldko=32):
    cfg = sbp.QkCfg(rows, H, Hkv, hd, seq, table, eps, dt)
    return lib.sbp_qk_norm_rope_forward(C.byref(cfg), q, ldq, k, ldk, qg, kg, pos, cos, sin, qo,
                                        ldqo, ko, ldko, None)


def _qk_bwd(lib, rows=4, H=4, Hkv=2, hd=16, seq=4, table=8, eps=1e-6, dt=1, q=FAKE, ldq=64,
            k=FAKE, ldk=32, qg=FAKE, kg=FAKE, pos=None, cos=FAKE, sin=FAKE, dqo=FAKE, lddqo=64,
            dko=FAKE, lddko=32, dq=FAKE, lddq=64, dk=FAKE, lddk=32, dqg=FAKE, dkg=FAKE, ws=FAKE,
            wsb=OK_WS):
    cfg = sbp.QkCfg(rows, H, Hkv, hd, seq, table, eps, dt)
    return lib.sbp_qk_norm_rope_backward(C.byref(cfg), q, ldq, k, ldk, qg, kg, pos, cos, sin, dqo,
                                         lddqo, dko, lddko, dq, lddq, dk, lddk, dqg, dkg, ws, wsb,
                                         None)


@pytest.mark.parametrize("call", [_qk_fwd, _qk_bwd])
def test_qk_norm_rope_refusals(lib, call):
    for bad in (dict(rows=0), dict(H=0), dict(Hkv=-1), dict(hd=0), dict(table=0), dict(seq=0),
                dict(seq=9), dict(eps=-1.0), dict(eps=float("nan")), dict(dt=3), dict(q=None),
                dict(k=None), dict(qg=None), dict(kg=None), dict(cos=None), dict(sin=None),
                dict(cos=FAKE + 4), dict(q=FAKE + 1), dict(ldq=63), dict(ldk=31),
                dict(pos=FAKE + 2)):
        assert call(lib, **bad) == 1, bad
    for bad in (dict(hd=15), dict(hd=258, ldq=2000, ldk=2000), dict(rows=1 << 30)):
        assert call(lib, **bad) == 2, bad


def test_qk_norm_rope_output_refusals(lib):
    for bad in (dict(qo=None), dict(ko=None), dict(qo=FAKE + 1), dict(ldqo=63), dict(ldko=31)):
        assert _qk_fwd(lib, **bad) == 1, bad
    for bad in (dict(dqo=None), dict(dko=None), dict(dq=None), dict(dk=None), dict(dqg=None),
                dict(dkg=None), dict(dq=FAKE + 2), dict(lddqo=63), dict(lddko=31), dict(lddq=63),
                dict(lddk=31), dict(ws=None), dict(ws=FAKE + 128)):
        assert _qk_bwd(lib, **bad) == 1, bad
    assert _qk_bwd(lib, wsb=16) == 3
    size = lib.sbp_qk_norm_rope_backward_workspace_size
    assert size(C.byref(sbp.QkCfg(4, 4, 2, 16, 4, 8, 1e-6, 1))) > 0
    assert size(C.byref(sbp.QkCfg(4, 4, 2, 15, 4, 8, 1e-6, 1))) == 0
    assert size(None) == 0
    f = lib.sbp_rope_table
    assert f(0, 16, 1e4, FAKE, FAKE, None) == 1 and f(4, 15, 1e4, FAKE, FAKE, None) == 2
    assert f(4, 16, 0.0, FAKE, FAKE, None) == 1 and f(4, 16, 1e4, None, FAKE, None) == 1
    assert f(4, 16, 1e4, FAKE, FAKE + 4, None) == 1


def _ptrs(*v):
    return (C.c_void_p * len(v))(*v)


def _nums(*v):
    return (C.c_int64 * len(v))(*v)


def test_grad_norm_refusals(lib):
    def sq(n=2, g=_ptrs(FAKE, FAKE), m=_nums(4, 5), out=FAKE, ws=FAKE, wsb=OK_WS):
        return lib.sbp_grad_sqsum(n, g, m, out, ws, wsb, None)

    def clip(n=2, g=_ptrs(FAKE, FAKE), o=None, m=_nums(4, 5), s=FAKE, mx=1.0, norm=FAKE):
        return lib.sbp_grad_clip(n, g, o, m, s, mx, norm, None)

    def both(n=2, g=_ptrs(FAKE, FAKE), o=None, m=_nums(4, 5), mx=1.0, norm=FAKE, ws=FAKE,
             wsb=OK_WS):
        return lib.sbp_grad_clip_norm(n, g, o, m, mx, norm, ws, wsb, None)
    for bad in (dict(n=-1), dict(g=None), dict(m=None), dict(g=_ptrs(FAKE, None)),
                dict(g=_ptrs(FAKE, FAKE + 4)), dict(m=_nums(4, -1))):
        assert sq(**bad) == 1 and clip(**bad) == 1 and both(**bad) == 1, bad
    for bad in (dict(o=_ptrs(FAKE, None)), dict(o=_ptrs(FAKE + 8, FAKE)), dict(mx=-1.0),
                dict(mx=float("nan"))):
        assert clip(**bad) == 1 and both(**bad) == 1, bad
    assert sq(out=None) == 1 and clip(s=None) == 1 and clip(s=FAKE + 4) == 1
    assert both(norm=None) == 1 and both(norm=FAKE + 2) == 1 and clip(norm=FAKE + 2) == 1
    assert sq(ws=None) == 1 and sq(wsb=16) == 3 and both(ws=FAKE + 8) == 1 and both(wsb=0) == 3
    assert lib.sbp_grad_norm_workspace_size(-1) == 0
    assert lib.sbp_grad_norm_workspace_size(5000) > lib.sbp_grad_norm_workspace_size(1)


def test_wrappers_refuse_before_the_library():
    """Shapes, types and devices are checked by the binding; CPU tensors never reach a kernel."""
    ids, table = torch.zeros(4, dtype=torch.int32), torch.zeros(8, 16)
    y, f = torch.zeros(4, 16), torch.float32
    with pytest.raises(ValueError, match="CUDA device"):
        sbp.embedding_scaled_forward(ids, table, 1.0, y)
    with pytest.raises(TypeError):
        sbp.embedding_scaled_forward(ids.long(), table, 1.0, y)
    with pytest.raises(ValueError, match="shape"):
        sbp.embedding_scaled_forward(ids, table, 1.0, torch.zeros(5, 16))
    with pytest.raises(ValueError, match="contiguous"):
        sbp.embedding_scaled_forward(ids, torch.zeros(16, 8).t(), 1.0, y)
    with pytest.raises(TypeError):
        sbp.embedding_scaled_forward(ids, table.half(), 1.0, y.half())
    with pytest.raises(TypeError):
        sbp.embedding_scaled_backward(ids, y.bfloat16(), 1.0, table)
    q, k, g = torch.zeros(4, 4, 16), torch.zeros(4, 2, 16), torch.ones(16)
    cos = torch.zeros(4, 8)

    def fwd(q=q, k=k, q_g=g, k_g=g, cos=cos, sin=cos, qo=None, ko=None, **kw):
        sbp.qk_norm_rope_forward(q, k, q_g, k_g, cos, sin, 1e-6, torch.empty_like(q) if qo is None
                                 else qo, torch.empty_like(k) if ko is None else ko, **kw)
    with pytest.raises(ValueError, match="CUDA device"):
        fwd()
    for bad in (dict(q_g=torch.ones(8)), dict(sin=torch.zeros(5, 8)), dict(cos=torch.zeros(4, 16)),
                dict(qo=torch.zeros(4, 4, 8)), dict(q=torch.zeros(16, 4, 4).permute(2, 1, 0)),
                dict(positions=torch.zeros(5, dtype=torch.int32)),
                dict(q=torch.zeros(1, 4, 16).expand(4, 4, 16))):
        with pytest.raises(ValueError):
            fwd(**bad)
    for bad in (dict(k=k.bfloat16()), dict(k_g=g.double()), dict(positions=torch.zeros(4)),
                dict(ko=k.bfloat16())):
        with pytest.raises(TypeError):
            fwd(**bad)
    with pytest.raises(ValueError, match="CUDA device"):
        sbp.GradList([torch.zeros(4)])
    with pytest.raises(TypeError):
        sbp.GradList([torch.zeros(4, dtype=torch.float64)])
    with pytest.raises(ValueError, match="contiguous"):
        sbp.GradList([torch.zeros(4, 4, dtype=f).t()])
    with pytest.raises(ValueError, match="no gradients"):
        sbp.grad_clip_norm([], 1.0, torch.zeros(1))


def test_layer_qk_norm_refusals(lib):
    cfg = sbp.layer_cfg(1, 256, 64, 4, 4, 16, 172, 1e-6, 1e4, sbp.SBP_F32, 4)
    none = ("bq", "bk", "bv")
    w = sbp.LayerWeights(**{n: (FAKE if n not in none else None) for n in sbp.WEIGHT_FIELDS})
    g = sbp.LayerGrads(**{n: (FAKE if n not in none else None) for n in sbp.WEIGHT_FIELDS})
    gains = sbp.QkGains(FAKE, FAKE)

    def fwd(c=cfg, gains=C.byref(gains), x=FAKE, y=FAKE, ws=FAKE, wsb=OK_WS):
        return lib.sbp_decoder_layer_qk_norm_forward_stream(C.byref(c), C.byref(w), gains, x, y,
                                                            ws, wsb, None)

    def bwd(c=cfg, gains=C.byref(gains), x=FAKE, dqg=FAKE, dkg=FAKE, ws=FAKE, wsb=OK_WS):
        return lib.sbp_decoder_layer_qk_norm_backward_stream(
            C.byref(c), C.byref(w), gains, x, FAKE, FAKE, C.byref(g), dqg, dkg, 0, ws, wsb, None)
    for bad in (dict(gains=None), dict(gains=C.byref(sbp.QkGains(FAKE, None))),
                dict(gains=C.byref(sbp.QkGains(FAKE + 2, FAKE))), dict(x=None),
                dict(ws=FAKE + 16)):
        assert fwd(**bad) == 1 and bwd(**bad) == 1, bad
    assert bwd(dqg=None) == 1 and bwd(dkg=FAKE + 4) == 1 and fwd(y=None) == 1
    size = lib.sbp_decoder_layer_qk_norm_workspace_size
    plain = lib.sbp_decoder_layer_workspace_size(C.byref(cfg))
    assert size(C.byref(cfg)) != plain and size(None) == 0
    assert fwd(wsb=size(C.byref(cfg)) - 1) == 3 and bwd(wsb=size(C.byref(cfg)) - 1) == 3
    odd = sbp.layer_cfg(1, 256, 64, 4, 4, 15, 172, 1e-6, 1e4, sbp.SBP_F32, 4)
    assert fwd(c=odd) == 2 and size(C.byref(odd)) == 0
    assert not sbp.has_qk_norm({"q_norm_g": None})
    with pytest.raises(ValueError, match="both"):
        sbp.has_qk_norm({"q_norm_g": 1})


class _FakeGrads:
    def __init__(self, tensors):
        self.tensors = list(tensors)


def _clip_worker(rank, world, port, q):
    """clip_sharded's exchange with the kernels replaced by their definitions."""
    import torch.distributed as dist
    from memory_efficient_exact_chunk_b200 import dp
    dist.init_process_group("gloo", init_method=f"tcp://127.0.0.1:{port}", rank=rank,
                            world_size=world)
    sbp.GradList = _FakeGrads
    sbp.grad_sqsum = lambda g, out, ws=None: out.copy_(
        sum(t.double().square().sum() for t in g.tensors).reshape(1))

    def clip(g, sqsum, max_norm, norm_out=None):
        norm_out.copy_(sqsum.sqrt())
        for t in g.tensors:
            t.mul_(min(1.0, max_norm / (float(sqsum.sqrt()) + 1e-6)))
    sbp.grad_clip = clip
    g = dp.ShardedGrads([("a", [("x", (10, 7))]), ("b", [("y", (300,))])], world, rank, "cpu")
    gen = torch.Generator().manual_seed(rank)
    before = []
    for name in g.order:
        g.out[name].normal_(generator=gen)
        before.append(g.out[name].clone())
    norm = dp.clip_sharded(g, 0.5)
    q.put((rank, float(norm), [t.tolist() for t in before], [g.out[n].tolist() for n in g.order]))
    dist.barrier()
    dist.destroy_process_group()


def test_clip_sharded_adds_the_ranks_sums():
    import socket

    import torch.multiprocessing as mp
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    ps = [ctx.Process(target=_clip_worker, args=(r, 2, port, q)) for r in range(2)]
    for p in ps:
        p.start()
    got = sorted(q.get(timeout=120) for _ in ps)
    for p in ps:
        p.join(timeout=60)
        assert p.exitcode == 0
    norm = sum(sum(v * v for v in t) for _, _, before, _ in got for t in before) ** 0.5
    for _, n, before, after in got:
        assert abs(n - norm) <= 1e-5 * norm
        for b, a in zip(before, after):
            assert all(abs(x * 0.5 / norm - y) <= 1e-5 for x, y in zip(b, a))
