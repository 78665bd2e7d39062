"""The layer for a few tokens on the GPU against its plain 64-bit statement
(tests/few_ref.py, which derives the tolerance), through the binding."""
import pytest
import torch

from tests import few_ref as ref

pytestmark = pytest.mark.gpu

# T, d, E, K, I, Is
SHAPES = [
    (1, 128, 1, 1, 128, 0), (1, 256, 8, 2, 512, 0), (2, 384, 6, 2, 256, 128),
    (3, 256, 5, 3, 384, 128), (8, 1024, 64, 6, 640, 1280), (16, 512, 16, 4, 256, 512),
    (4, 128, 40, 32, 128, 128), (13, 1152, 7, 7, 256, 896), (5, 128, 1024, 8, 128, 128),
    (16, 2048, 64, 8, 1408, 0), (9, 640, 3, 1, 2048, 384), (8, 256, 64, 16, 1408, 128),
    (16, 128, 1024, 32, 128, 128), (2, 16384, 2, 1, 128, 128), (2, 128, 2, 2, 16384, 16384)]
# widths that are odd numbers of 64: bf16 weights alone
ODD = [(1, 64, 1, 1, 64, 0), (3, 192, 5, 3, 320, 64), (16, 448, 300, 3, 64, 192),
       (7, 2112, 9, 4, 1344, 2688), (12, 64, 4, 2, 192, 0), (8, 192, 64, 16, 1472, 64),
       (15, 320, 64, 10, 1472, 192)]
FORMATS = ["bf16", "fp8", "blocks"]


@pytest.fixture(scope="module")
def moe():
    import sparse_expert_ffn_moe_gb300 as m
    return m


class Layer:
    def __init__(self, moe, c, fill=None):
        self.moe, self.c = moe, c
        self.g = {k: v.cuda() for k, v in c.items() if torch.is_tensor(v)}
        self.shape = moe.make_shape(c["T"], c["d"], c["E"], c["K"], c["I"], c["Is"], "bf16",
                                    c["router"])
        self.ws = moe.alloc_few_workspace(self.shape)
        if fill is not None:
            self.ws.fill_(fill)
        if c["fmt"] != "bf16":
            self.w = moe.make_fp8_experts(self.g)

    def __call__(self, y=None, stream=None, x=None):
        g, moe = self.g, self.moe
        x = g["x"] if x is None else x
        y = torch.full_like(x, 9) if y is None else y
        if self.c["fmt"] == "bf16":
            moe.moe_forward_few(self.shape, x, g["w_g"], g.get("bias"), g["w_gate"], g["w_up"],
                                g["w_down"], g.get("ws_gate"), g.get("ws_up"), g.get("ws_down"),
                                g.get("residual"), y, self.ws, stream)
        else:
            call = moe.moe_forward_few_fp8 if self.c["fmt"] == "fp8" else \
                moe.moe_forward_few_fp8_blocks
            call(self.shape, x, g["w_g"], g.get("bias"), self.w, g.get("residual"), y, self.ws,
                 stream)
        return y


def _check(moe, c, fill=255):
    layer = Layer(moe, c, fill)  # a workspace of NaNs: nothing may be read that was not written
    y = layer()
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(layer.ws) == 0
    want, tol = ref.layer(c)
    got = y.cpu().double()
    assert torch.isfinite(got).all()
    over = ((got - want).abs() - tol).max().item()
    assert over <= 0, (over, (got - want).abs().max().item(), want.abs().max().item())
    return layer, y


@pytest.mark.parametrize("router", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES + ODD)
def test_bf16(moe, shape, router):
    _check(moe, ref.inputs(*shape, router, "bf16", sum(shape)))


@pytest.mark.parametrize("router", ["softmax", "sigmoid"])
@pytest.mark.parametrize("fmt", ["fp8", "blocks"])
@pytest.mark.parametrize("shape", SHAPES)
def test_8_bit(moe, shape, fmt, router):
    _check(moe, ref.inputs(*shape, router, fmt, sum(shape)))


@pytest.mark.parametrize("fmt", FORMATS)
def test_without_bias_and_residual(moe, fmt):
    _check(moe, ref.inputs(6, 384, 12, 3, 256, 128, "softmax", fmt, 1, False, False))


@pytest.mark.parametrize("T", [2, 9, 16])
@pytest.mark.parametrize("fmt", FORMATS)
def test_all_tokens_at_the_same_experts(moe, fmt, T):
    _, y = _check(moe, ref.inputs(T, 512, 20, 4, 384, 256, "sigmoid", fmt, 2, True, False, True))
    assert (y == y[0]).all()


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("E", [102, 127, 200, 300])
def test_ties_go_to_the_lower_expert(moe, E, T):
    """Scores that are all equal choose what a bias that falls from expert to expert does (the
    sigmoid router's bias is not in its weights)."""
    c = ref.inputs(T, 128, E, 5, 128, 128, "sigmoid", "bf16", E + T)
    c["w_g"].zero_()
    c["bias"] = 0.01 * torch.arange(E, 0, -1)
    _, y = _check(moe, c)
    c["bias"] = None
    tied = Layer(moe, c, 255)()
    torch.cuda.synchronize()
    assert torch.equal(tied, y)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("E", [24, 150])
def test_one_token_that_is_not_finite(moe, fmt, E):
    """Its row is NaN, the call ends without an error and the next one is right."""
    c = ref.inputs(1, 256, E, 4, 256, 128, "softmax", fmt, E)
    layer, y = _check(moe, c)
    bad = torch.full_like(layer.g["x"], float("nan"))
    out = layer(x=bad)
    again = layer()
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(layer.ws) == 0
    assert torch.isnan(out).all() and torch.equal(again, y)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 8, 16])
def test_same_bits_on_every_run(moe, fmt, T):
    """Who takes which unit changes from run to run, the sums' order does not."""
    layer = Layer(moe, ref.inputs(T, 1024, 32, 4, 512, 1024, "softmax", fmt, 3))
    y = layer()
    for _ in range(30):
        assert torch.equal(layer(), y)


@pytest.mark.parametrize("fmt", FORMATS)
def test_residual_in_place(moe, fmt):
    layer = Layer(moe, ref.inputs(5, 256, 8, 2, 256, 128, "softmax", fmt, 4))
    y = layer()
    r = layer.g["residual"]
    layer(y=r)
    assert torch.equal(r, y)


@pytest.mark.parametrize("fmt", FORMATS)
def test_what_is_not_finite_stays_with_its_token(moe, fmt):
    """A row of NaNs, one of infinities, and an expert whose weights are NaN: tokens that do
    not pick it keep their bits, those that do show it."""
    c = ref.inputs(12, 256, 16, 2, 256, 128, "softmax", fmt, 5)
    y = Layer(moe, c)().cpu()
    bad = Layer(moe, c, 255)
    bad.g["x"] = bad.g["x"].clone()
    bad.g["x"][3] = float("nan")
    bad.g["x"][7, 5] = float("inf")
    idx, _, _ = ref.route(c["x"].double() @ c["w_g"].double().T, c["bias"], 2, "softmax")
    e = idx[0, 0].item()
    if fmt == "bf16":
        bad.g["w_down"][e, 7, 9] = float("nan")
    else:
        bad.g["w_down"][e, 7, 9] = 0x7F
    out = bad().cpu()
    assert bad.moe.moe_get_device_error(bad.ws) == 0
    hit = [t for t in range(12) if e in idx[t].tolist() and t not in (3, 7)]
    for t in range(12):
        if t in (3, 7):
            assert torch.isnan(out[t]).any()
        elif t in hit:
            assert torch.isnan(out[t, 7])
            assert torch.equal(out[t, :7], y[t, :7]) and torch.equal(out[t, 8:], y[t, 8:])
        else:
            assert torch.equal(out[t], y[t])
    assert 0 < len(hit) < 10


@pytest.mark.parametrize("fmt", FORMATS)
def test_captured_and_replayed(moe, fmt):
    layer = Layer(moe, ref.inputs(6, 512, 16, 3, 256, 256, "sigmoid", fmt, 6))
    x = layer.g["x"]
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    y = torch.empty_like(x)
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            layer(y=y)
    for seed in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(layer(), got)
        assert moe.moe_get_device_error(layer.ws) == 0


def test_calls_on_two_streams(moe):
    """Two layers at once, each with its own workspace, over and over: each gives its own
    bits and no wait runs out."""
    layers = [Layer(moe, ref.inputs(T, 1024, 32, 4, 768, 512, "softmax", fmt, 7 + T))
              for T, fmt in ((4, "bf16"), (9, "fp8"))]
    want = [layer() for layer in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    outs = [[torch.empty_like(w) for _ in range(40)] for w in want]
    for i in range(40):
        for layer, st, o in zip(layers, streams, outs):
            with torch.cuda.stream(st):
                layer(y=o[i])
    torch.cuda.synchronize()
    for layer, w, o in zip(layers, want, outs):
        assert all(torch.equal(v, w) for v in o)
        assert moe.moe_get_device_error(layer.ws) == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_wait_that_runs_out_is_reported(moe, fmt, monkeypatch):
    """With the copies held back (a switch for this test) the products' wait runs out: an
    error code, and the next call is sound."""
    layer = Layer(moe, ref.inputs(3, 256, 8, 2, 256, 128, "softmax", fmt, 8))
    want = layer()
    torch.cuda.synchronize()
    monkeypatch.setenv("MOE_TC_TEST_STALL", "1")
    monkeypatch.setenv("MOE_TC_TIMEOUT_MS", "30")
    layer()
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(layer.ws) == moe.MOE_ERR_TIMEOUT
    monkeypatch.delenv("MOE_TC_TEST_STALL")
    monkeypatch.delenv("MOE_TC_TIMEOUT_MS")
    assert torch.equal(layer(), want)
    assert moe.moe_get_device_error(layer.ws) == 0
