"""Host side of the operators of include/sbp_step.h and of the paths that use them, at its edges:
nothing here reaches a kernel, so no GPU is needed."""
import pytest
import torch

from memory_efficient_exact_chunk_b200 import build as sbp_build
from memory_efficient_exact_chunk_b200 import sbp, stack


@pytest.fixture(scope="module")
def lib():
    sbp_build.build()
    return sbp.load()


# --------------------------------------------------------------------------------- workspaces
@pytest.mark.parametrize("head_dim,dtype", [(64, sbp.SBP_BF16), (128, sbp.SBP_BF16),
                                            (16, sbp.SBP_F32)])
def test_a_stack_of_both_kinds_of_layers_gets_the_larger_workspace(lib, head_dim, dtype):
    """Neither kind needs the larger workspace in every configuration."""
    cfg = sbp.layer_cfg(1, 4096, 128, 4, 2, head_dim, 256, 1e-6, 1e4, dtype, 2)
    normed = {n: torch.ones(head_dim) for n in sbp.QK_NORM_FIELDS}
    sizes = [sbp.layer_workspace_size(cfg), sbp.layer_workspace_size(cfg, True)]
    for layers, need in (([{}, normed], max(sizes)), ([normed, {}, normed], max(sizes)),
                         ([{}], sizes[0]), ([normed, normed], sizes[1])):
        ws = stack.Workspaces("cpu")
        assert stack._layer_ws(cfg, layers, ws).numel() == max(need, 256)


# ---------------------------------------------------------------------------- queries and keys
FAKE = 0x100000  # an aligned address that is never dereferenced (argument checks fail first)


def test_gain_gradients_that_overlap_in_part_are_refused(lib):
    """One vector for both gains is allowed, one that begins inside the other is not (the workspace
    of none, which is checked behind it, keeps the allowed calls from a launch)."""
    import ctypes as C
    cfg = sbp.QkCfg(4, 4, 2, 16, 4, 8, 1e-6, 1)

    def call(dqg, dkg):
        code = lib.sbp_qk_norm_rope_backward(
            C.byref(cfg), FAKE, 64, FAKE, 32, FAKE, FAKE, None, FAKE, FAKE, FAKE, 64, FAKE, 32,
            FAKE, 64, FAKE, 32, dqg, dkg, None, 0, None)
        return code, lib.sbp_last_error().decode()
    for dqg, dkg in ((FAKE, FAKE + 4), (FAKE + 60, FAKE)):
        code, msg = call(dqg, dkg)
        assert code == 1 and "overlap" in msg
    for dqg, dkg in ((FAKE, FAKE), (FAKE, FAKE + 64), (FAKE + 64, FAKE)):
        code, msg = call(dqg, dkg)
        assert code == 1 and "workspace" in msg


# ------------------------------------------------------------------------------------ streams
class _Streams:
    """torch.cuda.stream without a GPU: keeps the stream that allocations are made for."""

    def __init__(self, monkeypatch, makers=("empty",)):
        self.now, self.made = None, []
        monkeypatch.setattr(torch.cuda, "stream", self.use)
        for name in makers:
            monkeypatch.setattr(torch, name, self.counted(getattr(torch, name)))

    def counted(self, fn):
        def make(*a, **k):
            self.made.append(self.now)
            return fn(*a, **{**k, "device": "cpu"})
        return make

    def use(self, stream):
        import contextlib

        @contextlib.contextmanager
        def on():
            before, self.now = self.now, stream
            yield
            self.now = before
        return on()


class _Taker:
    """A library that takes every call and does nothing."""

    def __getattr__(self, name):
        return lambda *a: 512 if name.endswith("size") else 0


def test_workspaces_are_allocated_for_the_stream_they_are_used_on(monkeypatch):
    """The current stream's queued work may still use memory that its pool hands out again."""
    streams = _Streams(monkeypatch)
    need = lambda: 1000
    calls = []
    call = lambda p, n: calls.append(n) or 0
    sbp._with_ws(None, 0, "side", need, call)
    sbp._with_ws(None, 0, None, need, call)
    assert streams.made == ["side", None] and calls == [1000, 1000]
    # one that is too small is replaced by one for the stream
    small = torch.zeros(8, dtype=torch.uint8)
    monkeypatch.setattr(type(small), "get_device", lambda t: 0, raising=False)
    sbp._with_ws(small, 0, "side", need, lambda p, n: 3 if n < 1000 else 0)
    assert streams.made[2:] == ["side"]
    # the calls of sbp.h too
    x = torch.zeros(2, 2)
    del streams.made[:]
    monkeypatch.setattr(sbp, "load", _Taker)
    monkeypatch.setattr(sbp, "_stream", lambda s: None)
    sbp.rmsnorm_backward(x, x, x, x, x, x, stream="side")
    sbp.embedding_backward(torch.zeros(2, dtype=torch.int32), x, x, stream="side")
    sbp.lmhead_ce_backward(x, x, x, x, 1, x, x, x, stream="side")
    sbp.lmhead_ce_forward(x, x, x, x, 1, x, stream="side")
    cfg = sbp.layer_cfg(1, 4, 4, 1, 1, 2, 4, 1e-6, 1e4, sbp.SBP_F32, 1)
    sbp.decoder_layer_forward(cfg, {}, x, x, stream="side")
    sbp.decoder_layer_backward(cfg, {}, x, x, x, {}, stream="side")
    assert streams.made == ["side"] * 6


def test_the_stack_allocates_and_clears_on_its_stream(monkeypatch):
    """Gradients that the current stream clears are not ready for the calls on another one."""
    streams = _Streams(monkeypatch, ("empty", "zeros"))
    monkeypatch.setattr(sbp, "load", _Taker)
    monkeypatch.setattr(sbp, "_stream", lambda s: None)
    cfg = sbp.layer_cfg(1, 4, 4, 1, 1, 2, 4, 1e-6, 1e4, sbp.SBP_F32, 1)
    ids, w = torch.ones(4, dtype=torch.int32), torch.ones(4)
    table, g = torch.ones(3, 4), torch.ones(4)
    seen = []
    stack.stack_backward(cfg, table, [{}], g, table, ids, ids, w, stream="side")
    assert len(streams.made) > 5 and set(streams.made) == {"side"}
    del streams.made[:]
    ws = stack.Workspaces("cpu")
    xs, hf, rstd = stack.stack_forward(cfg, table, [{}], g, ids, ws, "side")     # by its place
    stack.stack_backward_from(cfg, [{}], g, table, ids, ids, w, xs, hf, rstd, ws, stream="side",
                              grads=stack.zero_grads([{}], table, g, "cpu", (3, 4)),
                              on_final=lambda name: seen.append((name, streams.now)))
    assert seen == [(n, "side") for n in ("head", "layer0", "embed")]
    assert set(streams.made[:3]) == {"side"}
    stack.stack_backward(cfg, table, [{}], g, table, ids, ids, w)
    assert streams.made[-1] is None and streams.now is None


# ----------------------------------------------------------------------------- gradient lists
@pytest.fixture
def clip_calls(monkeypatch):
    """The calls that reach the library, which is a fake; CPU tensors pass for device tensors."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 512 if name.endswith("size") else calls.append(name) or 0
    monkeypatch.setattr(sbp, "load", Lib)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(sbp, "_on_device", lambda stream, *t: (0, None))
    return calls


@pytest.mark.parametrize("n", [1, 12, 16, 17, 40])
def test_a_list_whose_tensors_got_other_memory_is_refused(clip_calls, n):
    ws, norm, sq = torch.empty(512, dtype=torch.uint8), torch.zeros(1), torch.zeros(1).double()
    turns = -(-n // sbp.GradList.LOOK)
    for k in {0, n // 2, n - 1}:
        for out in (False, True):
            old = [torch.full((8,), 3.0) for _ in range(2 * n)]
            grads, into = sbp.GradList(old[:n]), sbp.GradList(old[n:])
            for _ in range(2 * turns):
                sbp.grad_clip_norm(grads, 1.0, norm, out=into if out else None, ws=ws)
            moved = old[n + k if out else k]
            kept = (into if out else grads).memory[k]
            moved.data = torch.zeros(8)
            del clip_calls[:]
            with pytest.raises(ValueError, match="other memory"):
                for _ in range(turns):
                    sbp.grad_clip_norm(grads, 1.0, norm, out=into if out else None, ws=ws)
            assert len(clip_calls) == k // sbp.GradList.LOOK
            # what the calls worked on until then is not freed
            assert kept.data_ptr() == (into if out else grads).ptrs[k] and kept.nbytes() == 32
            assert torch.tensor([], dtype=torch.float32).set_(kept).tolist() == [3.0] * 8
    grads = sbp.GradList([moved])
    moved.data = torch.zeros(8)
    for call in (lambda: sbp.grad_sqsum(grads, sq, ws=ws),
                 lambda: sbp.grad_clip(grads, sq, 1.0, norm_out=norm)):
        with pytest.raises(ValueError, match="other memory"):
            call()


# ------------------------------------------------------------------------- sharded gradients
class _Tensors:
    def __init__(self, tensors):
        self.tensors = list(tensors)


def _subgroup_worker(rank, world, port, q):
    """Every rank a replica group of its own: the exchange must stay inside it.  The kernels are
    replaced by their definitions."""
    import torch.distributed as dist

    from memory_efficient_exact_chunk_b200 import dp
    dist.init_process_group("gloo", init_method=f"tcp://127.0.0.1:{port}", rank=rank,
                            world_size=world)
    sbp.GradList = _Tensors
    sbp.grad_sqsum = lambda g, out, ws=None: out.copy_(
        sum(t.double().square().sum() for t in g.tensors).reshape(1))
    sbp.grad_clip = lambda g, sqsum, max_norm, norm_out=None: norm_out.copy_(sqsum.sqrt())
    own = [dist.new_group([r]) for r in range(world)][rank]
    both = dist.new_group(list(range(world)))

    def grads(shards):
        g = dp.ShardedGrads([("a", [("x", (300,))])], shards, rank % shards, "cpu")
        g.out["a"].fill_(rank + 1.0)
        return g

    def refused(*args):
        try:
            dp.clip_sharded(*args)
        except ValueError:
            return True
        return False
    alone, halves, unreduced = grads(1), grads(world), grads(world)
    dp.GradReducer(alone, group=own)
    dp.GradReducer(halves, group=both)
    n = alone.out["a"].numel()
    got = {"alone": float(dp.clip_sharded(alone, 1.0)) / n ** 0.5,
           "halves": float(dp.clip_sharded(halves, 1.0)) / halves.out["a"].numel() ** 0.5,
           "by name": float(dp.clip_sharded(unreduced, 1.0, both)) /
           unreduced.out["a"].numel() ** 0.5,
           "refused": [refused(alone, 1.0, both), refused(halves, 1.0, own),
                       refused(unreduced, 1.0, own), refused(grads(1), 1.0)]}
    q.put((rank, got))
    dist.barrier()
    dist.destroy_process_group()


def test_clip_sharded_stays_in_the_reducers_group():
    import socket

    import torch.multiprocessing as mp
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    ps = [ctx.Process(target=_subgroup_worker, args=(r, 2, port, q)) for r in range(2)]
    for p in ps:
        p.start()
    got = dict(q.get(timeout=120) for _ in ps)
    for p in ps:
        p.join(timeout=60)
        assert p.exitcode == 0
    for rank, r in got.items():
        assert r["refused"] == [True] * 4
        assert abs(r["alone"] - (rank + 1)) < 1e-5
        for name in ("halves", "by name"):           # 1 and 2, in halves of equal size
            assert abs(r[name] - 5 ** 0.5) < 1e-5, name


# ------------------------------------------------------------------- the layer with the norms
@pytest.mark.parametrize("B,T,H,hd,D", [(1, 1 << 25, 64, 2, 1), (1, 1 << 30, 1, 8, 1),
                                        (1 << 20, 1 << 11, 4, 2, 4), (1, 8, 65537, 8, 1)])
def test_layers_whose_chunks_pass_the_norms_limits_are_refused(lib, B, T, H, hd, D):
    """The norms' kernels count rows and heads in 32 bits (no workspace is given, which is checked
    behind the sizes: no call gets to a launch)."""
    import ctypes as C
    cfg = sbp.layer_cfg(B, T, 64, H, H, hd, 64, 1e-6, 1e4, sbp.SBP_F32, D)
    none = ("bq", "bk", "bv")
    ptrs = {n: (FAKE if n not in none else None) for n in sbp.WEIGHT_FIELDS}
    w, g, gains = sbp.LayerWeights(**ptrs), sbp.LayerGrads(**ptrs), sbp.QkGains(FAKE, FAKE)
    assert lib.sbp_decoder_layer_qk_norm_workspace_size(C.byref(cfg)) == 0
    assert lib.sbp_decoder_layer_qk_norm_forward_stream(
        C.byref(cfg), C.byref(w), C.byref(gains), FAKE, FAKE, None, 0, None) == 2
    assert lib.sbp_decoder_layer_qk_norm_backward_stream(
        C.byref(cfg), C.byref(w), C.byref(gains), FAKE, FAKE, FAKE, C.byref(g), FAKE, FAKE, 0,
        None, 0, None) == 2
    assert "norms" in lib.sbp_last_error().decode()
    assert lib.sbp_decoder_layer_workspace_size(C.byref(cfg)) > 0      # without norms as before
    cfg.num_chunks = min(T, 4 * D) if H <= 65536 else D                # shorter chunks are taken
    assert (lib.sbp_decoder_layer_qk_norm_workspace_size(C.byref(cfg)) > 0) == (H <= 65536)


def test_the_backward_makes_its_own_gradients(monkeypatch):
    """Without gradient buffers it makes them all, the embedding's among them, or says at once what
    it needs."""
    monkeypatch.setattr(sbp, "load", _Taker)
    monkeypatch.setattr(sbp, "_stream", lambda s: None)
    cfg = sbp.layer_cfg(1, 4, 4, 1, 1, 2, 4, 1e-6, 1e4, sbp.SBP_F32, 1)
    ids, w = torch.ones(4, dtype=torch.int32), torch.ones(4)
    head, g, x = torch.ones(3, 4), torch.ones(4), torch.ones(4, 4)
    seen = []
    args = (cfg, [{"wq": x}], g, head, ids, ids, w, [x, x], x, w, stack.Workspaces("cpu"))
    r = stack.stack_backward_from(*args, embed_shape=(5, 4))
    assert r.grads["embed"].shape == (5, 4) and r.grads["lm_head"].shape == (3, 4)
    with pytest.raises(ValueError, match="embed_shape"):
        stack.stack_backward_from(*args, on_final=seen.append)
    assert not seen


# ------------------------------------------------------------------------------ memory model
def test_memory_model_counts_the_step_operators(lib):
    """The workspaces that the stack takes for scaled embeddings, normed layers and clipping, and the
    gains with their gradients."""
    import dataclasses

    from memory_efficient_exact_chunk_b200 import memory_model as MM
    from memory_efficient_exact_chunk_b200 import synth
    plain = MM.StackShape.from_workload(synth.WORKLOADS["llama3_8b_stack4_64k"])
    T, D, d, V = 65536, 8, plain.d_model, plain.vocab
    a = MM.stack_step_bytes(plain, T, D)
    with_all = dataclasses.replace(plain, qk_norm=True, embed_scaled=True, clipped=True)
    b = MM.stack_step_bytes(with_all, T, D)
    cfg = sbp.layer_cfg(1, T, d, 32, 8, 128, 14336, 1e-5, 500000.0, sbp.SBP_BF16, D)
    assert b["layer_workspace"] == sbp.layer_workspace_size(cfg, True) > a["layer_workspace"]
    assert b["small_workspaces"] - a["small_workspaces"] == (
        sbp.embedding_scaled_backward_workspace_size(T, d, V)
        - int(lib.sbp_embedding_backward_workspace_size(T, V))
        + sbp.grad_norm_workspace_size(3 + 4 * 11))
    assert b["small_workspaces"] - a["small_workspaces"] > 30e6        # the partial rows
    assert b["grads_fp32"] - a["grads_fp32"] == 4 * 4 * 2 * 128
    assert b["total"] == sum(v for k, v in b.items() if k != "total")
    assert MM.max_tokens(with_all, D, 150 * 10 ** 9) < MM.max_tokens(plain, D, 150 * 10 ** 9)


def test_a_workspace_for_another_stream_may_come_back_to_the_current_one(monkeypatch):
    """It is returned to the caller, who may use it on either: its memory is not handed out again
    before both have passed its end."""
    class Buffer:
        is_cuda, device, recorded = True, "cuda:0", []

        def record_stream(self, stream):
            self.recorded.append(stream)
    streams = _Streams(monkeypatch)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: Buffer())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: (d, streams.now))
    sbp.workspace(100, "cuda:0", "side")
    assert Buffer.recorded == [("cuda:0", None)]
    sbp.workspace(100, "cuda:0")
    assert len(Buffer.recorded) == 1
