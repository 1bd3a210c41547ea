"""The mixture-of-experts layer on the GPU against the oracle, and the chain
route -> experts as a serving program runs it.

Bound.  A hidden value is rounded to bf16 and then to a 4-bit level, so an
error of the fp32 sums before it, however small, can move a value next to a
border by a whole level.  The sums' error is at most e = K * 65 / 64 * 2^-23 of
their magnitude A (see test_gpu_mx.py), so only values within e of a border
can move, each by one step.  The oracle therefore recomputes the hidden values
of the library's own operators where it compares tightly: gate and up products
by lutq_mx_gemm (checked against the oracle elsewhere), silu in fp64; what is
left are the values whose fp64 silu product lies within 2^-20 of a bf16
rounding border, which are allowed either neighbour by the slack below: the
largest level step (a third of the block's largest magnitude) times the
weights it meets.
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import mx_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dequant_gemv_group_b200 as m
    return m


def _f64(t):
    return t.double().cpu().numpy()


class Layer:
    def __init__(self, lq, e, d, f, fmt, seed=0):
        self.lq, self.e, self.d, self.f, self.fmt = lq, e, d, f, fmt
        mk = lambda n, k, s: torch.stack([workloads.normal_weights(n, k, k ** -0.5, seed=s + 7 * i)  # noqa: E731
                                          for i in range(e)]).cuda()
        self.w = {"gate": mk(f, d, seed), "up": mk(f, d, seed + 1), "down": mk(d, f, seed + 2)}
        self.p = {n: lq.lutq_mx_quantize(w, fmt) for n, w in self.w.items()}
        self.v = {n: lq.lutq_mx_dequantize(self.p[n], w.shape[1], w.shape[2], fmt,
                                           dtype=torch.float32).double() for n, w in self.w.items()}

    def run(self, x, ids, weights, **kw):
        return self.lq.lutq_mx_experts(x, ids, weights, self.p["gate"], self.p["up"],
                                       self.p["down"], self.f, self.fmt, **kw)

    def reference(self, x, ids, weights, batch=None):
        """y in fp64 from the library's fp32 gate and up sums, and the slack per output; batch:
        the tokens of the call that these were part of."""
        batch = batch or len(x)
        lq, fmt, d, f = self.lq, self.fmt, self.d, self.f
        y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        slack = torch.zeros_like(y)
        for e in range(self.e):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if not t.numel():
                continue
            xp = lq.lutq_mx_quantize(x[t].contiguous(), fmt)
            g = lq.lutq_mx_gemm(xp, t.numel(), self.p["gate"][e], f, d, fmt).double()
            u = lq.lutq_mx_gemm(xp, t.numel(), self.p["up"][e], f, d, fmt).double()
            exact = g / (1 + torch.exp(-g)) * u
            h = exact.to(torch.bfloat16)
            hv = lq.lutq_mx_dequantize(lq.lutq_mx_quantize(h, fmt), t.numel(), f, fmt,
                                       dtype=torch.float32).double()
            w = weights[t, j].double().unsqueeze(1)
            down = self.v["down"][e]
            out = hv @ down.t()
            y.index_add_(0, t, w * out)
            if (x.dtype == torch.bfloat16 and batch > 64
                    and -(-batch * ids.shape[1] // self.e) > 32):
                # these rows are rounded to bf16: each off by half a step, 2^-8 of itself
                slack.index_add_(0, t, w.abs() * out.abs() * 2.0 ** -8)
            # values next to a bf16 border: within 2^-20 of halfway between two bf16 numbers
            near = exact * (1 + 2.0 ** -20)
            unsure = (exact * (1 - 2.0 ** -20)).to(torch.bfloat16) != near.to(torch.bfloat16)
            block = hv.abs().view(t.numel(), -1, O.BLOCK[fmt]).amax(2, keepdim=True)
            step = (block / 3 * 1.5).expand(-1, -1, O.BLOCK[fmt]).reshape(hv.shape)
            # a moved block maximum can move the block's scale: all its values may move
            hit = unsure.view(t.numel(), -1, O.BLOCK[fmt]).any(2, keepdim=True)
            hit = hit.expand(-1, -1, O.BLOCK[fmt]).reshape(hv.shape)
            moved = torch.where(unsure, step, torch.zeros_like(step))
            top = hv.abs() >= 0.99 * block.expand(-1, -1, O.BLOCK[fmt]).reshape(hv.shape)
            top = (unsure & top).view(t.numel(), -1, O.BLOCK[fmt]).any(2, keepdim=True)
            top = top.expand(-1, -1, O.BLOCK[fmt]).reshape(hv.shape)
            moved = torch.where(hit & top, step, moved)
            slack.index_add_(0, t, w.abs() * (moved @ down.abs().t()))
            mag = hv.abs() @ down.abs().t()
            slack.index_add_(0, t, w.abs() * mag * (f * 65 / 64 * 2.0 ** -23 + 2.0 ** -20))
        return y, slack


def _inputs(t, e, k, d, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, d, generator=g).to(dtype).cuda()
    z = torch.randn(t, e, generator=g).cuda()
    return x, z


def _close(y, ref, slack):
    eps = torch.finfo(y.dtype).eps / 2
    bound = slack + (eps * 1.01 + 2.0 ** -22) * (ref.abs() + slack)
    worst = ((y.double() - ref).abs() / bound.clamp(min=1e-300)).max()
    assert ((y.double() - ref).abs() <= bound).all(), float(worst)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("t,e,k,d,f", [
    (1, 4, 2, 256, 128), (1, 8, 8, 512, 96), (1, 2, 1, 1056, 512), (4, 9, 8, 608, 160), (2, 3, 1, 64, 32), (5, 8, 2, 288, 160),
    (16, 16, 4, 512, 256), (17, 6, 3, 256, 320), (40, 8, 2, 384, 192), (130, 4, 4, 256, 256),
    (333, 5, 2, 544, 416), (700, 3, 1, 256, 544)])
def test_layer(lq, fmt, t, e, k, d, f):
    layer = Layer(lq, e, d, f, fmt, seed=t)
    x, z = _inputs(t, e, k, d, seed=e)
    ids, w = lq.lutq_route(z, k, renormalize=True)
    st = lq.new_status()
    y = layer.run(x, ids, w, status=st)
    assert int(st.item()) == 0
    _close(y, *layer.reference(x, ids, w))
    assert torch.equal(layer.run(x, ids, w), y)


def test_against_the_plain_oracle(lq):
    """The whole chain in numpy, with the one input whose hidden values have no near border."""
    fmt, t, e, k, d, f = "mxfp4", 3, 4, 2, 128, 64
    layer = Layer(lq, e, d, f, fmt, seed=1)
    x, z = _inputs(t, e, k, d, seed=2)
    ids, w = lq.lutq_route(z, k, renormalize=True)
    xv = O.values(*O.quantize(_f64(x), fmt), fmt)
    v = {n: np.stack([O.values(*O.quantize(_f64(m), fmt), fmt) for m in layer.w[n]])
         for n in layer.w}
    ref = O.experts(xv, ids.cpu().numpy(), _f64(w), v["gate"], v["up"], v["down"], fmt)
    y, slack = layer.reference(x, ids, w)
    np.testing.assert_allclose(_f64(y), ref, rtol=0, atol=float(slack.max()) + 1e-12)
    _close(layer.run(x, ids, w), y, slack)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_types(lq, fmt, dtype):
    layer = Layer(lq, 5, 320, 96, fmt, seed=3)
    x, z = _inputs(21, 5, 2, 320, seed=4, dtype=dtype)
    x = x.bfloat16().to(dtype)
    ids, w = lq.lutq_route(z, 2)
    y = layer.run(x, ids, w)
    assert y.dtype == dtype
    _close(y, *layer.reference(x, ids, w))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_uneven_skipped_and_repeated(lq, fmt):
    """All tokens to one expert, experts without tokens, ids out of range, an expert twice."""
    t, e, k, d, f = 150, 9, 3, 256, 160
    layer = Layer(lq, e, d, f, fmt, seed=5)
    x, _ = _inputs(t, e, k, d, seed=6)
    g = torch.Generator().manual_seed(7)
    w = torch.rand(t, k, generator=g).cuda()
    ids = torch.full((t, k), 4, dtype=torch.int32)
    ids[:, 1] = 7
    ids[:, 2] = torch.where(torch.arange(t) % 3 == 0, 4, -1)      # twice, or skipped
    ids[10] = torch.tensor([-1, 9, 1 << 30])                       # none at all
    ids = ids.cuda()
    y = layer.run(x, ids, w)
    ref, slack = layer.reference(x, ids, w)
    _close(y, ref, slack)
    assert (y[10] == 0).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("t,e", [(60, 40), (100, 60), (200, 40)])
def test_most_tokens_to_one_expert(lq, fmt, t, e):
    """Few tokens an expert on average, but one has more than a tile holds."""
    d, f = 160, 96
    layer = Layer(lq, e, d, f, fmt, seed=e)
    x, z = _inputs(t, e, 1, d, seed=t)
    z[:, 3] += 3.5
    ids, w = lq.lutq_route(z, 2)
    _close(layer.run(x, ids, w), *layer.reference(x, ids, w))


def test_rows_do_not_depend_on_the_batch(lq):
    layer = Layer(lq, 6, 256, 224, "mxfp4", seed=8)
    x, z = _inputs(300, 6, 2, 256, seed=9)
    ids, w = lq.lutq_route(z, 2)
    y = layer.run(x, ids, w)
    for n in (1, 7, 40):
        part = layer.run(x[:n].contiguous(), ids[:n].contiguous(), w[:n].contiguous())
        _close(part, *layer.reference(x[:n], ids[:n], w[:n]))
        _close(y[:n], *layer.reference(x[:n], ids[:n], w[:n], batch=300))


def test_nonfinite_token_stays_alone(lq):
    layer = Layer(lq, 4, 256, 128, "nvfp4", seed=10)
    x, z = _inputs(12, 4, 2, 256, seed=11)
    ids, w = lq.lutq_route(z, 2)
    want = layer.run(x, ids, w)
    x[5, 3] = float("nan")
    st = lq.new_status()
    y = layer.run(x, ids, w, status=st)
    assert int(st.item()) == 5 and torch.isnan(y[5]).all()
    keep = [i for i in range(12) if i != 5]
    assert torch.equal(y[keep], want[keep])


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("t", [1, 12, 40, 300])
def test_every_size_with_streams_and_graphs(lq, fmt, t):
    """Few pairs an expert, some, many: a workspace of NaN bytes, two streams at once, a captured
    call replayed on new inputs.  Always the same bits."""
    e, k, d, f = 5, 2, 512, 288
    layer = Layer(lq, e, d, f, fmt, seed=22)
    nb = lq.lutq_mx_experts_workspace_bytes(t, k, e, d, f, fmt)
    sets = []
    for seed in (23, 24):
        x, z = _inputs(t, e, k, d, seed=seed)
        ids, w = lq.lutq_route(z, k)
        sets.append((x, ids, w, layer.run(x, ids, w)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.full((nb,), 255, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for s, sp, (x, ids, w, want) in zip(streams, spaces, sets):
            with torch.cuda.stream(s):
                got.append((layer.run(x, ids, w, workspace=sp), want))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y, want in got)
    x, ids, w = (v.clone() for v in sets[0][:3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.run(x, ids, w, workspace=spaces[0])
    for x2, ids2, w2, want in sets[::-1]:
        x.copy_(x2)
        ids.copy_(ids2)
        w.copy_(w2)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_offsets_beyond_32_bits(lq, fmt):
    """The last of 64 experts, 4.4 GB into its matrices, gives what the first one gives."""
    e, d, f = 64, 16384, 8192
    g = torch.Generator("cuda").manual_seed(2)
    mats = []
    for n, k in ((f, d), (f, d), (d, f)):
        a, b = (lq.lutq_mx_quantize(torch.randn(n, k, device="cuda", generator=g).bfloat16()
                                    * k ** -0.5, fmt) for _ in range(2))
        m = a.repeat(e, 1)
        m[0] = b
        mats.append(m)
    for t in (4, 600, 1100):
        x = torch.randn(t, d, device="cuda", generator=g).bfloat16()
        w = torch.rand(t, 1, device="cuda", generator=g)
        ids = torch.zeros(t, 1, dtype=torch.int32, device="cuda")
        y = lq.lutq_mx_experts(x, ids, w, *mats, f, fmt)
        other = lq.lutq_mx_experts(x, ids + 1, w, *mats, f, fmt)
        swap = torch.tensor([0, e - 1], device="cuda")
        for m in mats:
            m[swap] = m[swap.flip(0)]
        assert torch.equal(lq.lutq_mx_experts(x, ids + (e - 1), w, *mats, f, fmt), y)
        assert not torch.equal(y, other)
        for m in mats:
            m[swap] = m[swap.flip(0)]


def test_graph_streams_and_dirty_workspace(lq):
    """route -> experts captured and replayed; the workspace's old contents (NaN bytes) do not
    matter; two streams with their own workspaces."""
    fmt, t, e, k, d, f = "nvfp4", 20, 8, 2, 256, 192
    layer = Layer(lq, e, d, f, fmt, seed=12)
    nb = lq.lutq_mx_experts_workspace_bytes(t, k, e, d, f, fmt)
    x, z = _inputs(t, e, k, d, seed=13)
    ids, w = lq.lutq_route(z, k)
    want = layer.run(x, ids, w)
    for fill in (0, 255):
        ws = torch.full((nb,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(layer.run(x, ids, w, workspace=ws), want)
    zin, xin = z.clone(), x.clone()
    ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        i2, w2 = lq.lutq_route(zin, k)
        y = layer.run(xin, i2, w2, workspace=ws)
    for seed in (14, 15):
        x2, z2 = _inputs(t, e, k, d, seed=seed)
        xin.copy_(x2)
        zin.copy_(z2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, layer.run(x2, *lq.lutq_route(z2, k)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.empty(nb, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for s, sp in zip(streams, spaces):
            with torch.cuda.stream(s):
                got.append(layer.run(x, ids, w, workspace=sp))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("t,k", [(1, 1), (3, 2), (20, 4)])
def test_no_expert_at_all(lq, t, k):
    """Tokens without any expert get zeros, in every kernel's sum."""
    layer = Layer(lq, 6, 160, 64, "mxfp4")
    x, _ = _inputs(t, 6, k, 160, seed=1)
    w = torch.ones(t, k, device="cuda")
    y = torch.full((t, 160), 7.0, dtype=torch.bfloat16, device="cuda")
    layer.run(x, torch.full((t, k), -1, dtype=torch.int32, device="cuda"), w, y=y)
    assert (y == 0).all()
    ids = torch.full((t, k), 6, dtype=torch.int32, device="cuda")
    ids[t - 1, k - 1] = 5
    y.fill_(7.0)
    layer.run(x, ids, w, y=y)
    assert (y[:t - 1] == 0).all() and (y[t - 1] != 0).any()


def test_refusals(lq):
    layer = Layer(lq, 3, 64, 32, "mxfp4")
    x, z = _inputs(4, 3, 2, 64, seed=1)
    ids, w = lq.lutq_route(z, 2)
    small = torch.empty(lq.lutq_mx_experts_workspace_bytes(4, 2, 3, 64, 32, "mxfp4") - 1,
                        dtype=torch.uint8, device="cuda")
    with pytest.raises(lq.LutqError) as e:
        layer.run(x, ids, w, workspace=small)
    assert e.value.status == 9
    for bad in (lambda: layer.run(x, ids[:2], w[:2]), lambda: layer.run(x[:, :32].contiguous(), ids, w),
                lambda: layer.run(x, ids, w[:, :1].contiguous())):
        with pytest.raises(lq.LutqError):
            bad()
    with pytest.raises(ValueError):
        layer.run(x, ids.long(), w)
    with pytest.raises(ValueError):
        layer.run(x, ids, w.double())


def test_empty(lq):
    layer = Layer(lq, 3, 64, 32, "mxfp4")
    y = layer.run(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                  torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                  torch.empty(0, 2, device="cuda"))
    assert y.shape == (0, 64)
