"""The 8-bit rows and product, the norms around a block and the group-limited choice as they
are used: a decoder layer with experts, captured and replayed, on several streams, with
shared workspaces in order."""
import numpy as np
import pytest

from tests import block_ref as R
from tests.gpu_util import require_gpu, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wob():
    require_gpu()
    import weight_only_bit_amd as w
    w.device_check()
    return w


class Layer:
    """norm -> 8-bit projection -> norm (gate, residual scale) -> router -> MXFP4 experts ->
    norm -> 8-bit feed-forward (gated rows quantised again) -> norm into MXFP4 -> 4-bit head."""

    def __init__(self, wob, T, H, I, E, topk, seed):
        torch = torch_mod()
        self.wob, self.topk = wob, topk
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*s, std=1.0, dtype=torch.bfloat16):
            return (torch.randn(s, device="cuda", generator=g) * std).to(dtype)
        self.x = normal(T, H)
        self.h = normal(T, H, dtype=torch.float32)
        self.norm = [(1 + normal(H, std=0.1, dtype=torch.float32)).bfloat16() for _ in range(6)]
        self.gate = normal(H)
        self.proj = wob.int8_quantize(normal(H, H, std=H ** -0.5))
        self.router = normal(E, H, std=H ** -0.5)
        self.bias = normal(E, std=0.05, dtype=torch.float32)
        self.w1 = wob.mxfp4_quantize(normal(E, 2 * I, H, std=H ** -0.5))
        self.w2 = wob.mxfp4_quantize(normal(E, H, I, std=I ** -0.5))
        self.up = wob.int8_quantize(normal(2 * I, H, std=H ** -0.5))
        self.down = wob.int8_quantize(normal(H, I, std=I ** -0.5))
        self.head = wob.mxfp4_quantize(normal(256, H, std=H ** -0.5))

    def run(self):
        wob, torch = self.wob, torch_mod()
        o = {}
        o["c0"], o["s0"], o["h0"] = wob.residual_norm(self.x, self.h, self.norm[0], quant=wob.QUANT_INT8)
        o["y0"] = wob.int8_gemm(o["c0"], o["s0"], *self.proj, out_dtype=torch.bfloat16)
        o["n1"], o["h1"] = wob.residual_norm(o["y0"], o["h0"], self.norm[1], post_weight=self.norm[2], gate=self.gate,
                                             alpha=0.5)
        o["logits"] = o["n1"] @ self.router.t()
        o["ids"], o["w"] = wob.moe_route(o["logits"], self.topk, bias=self.bias, groups=4, topk_groups=2, scale=1.5)
        o["a"] = wob.mxfp4_moe_gemm(o["n1"], o["ids"], *self.w1, act=wob.ACT_SILU_MUL)
        o["y1"] = wob.mxfp4_moe_stage2(o["a"], o["ids"], o["w"], *self.w2)
        o["c2"], o["s2"], o["h2"] = wob.residual_norm(o["y1"], o["h1"], self.norm[3], quant=wob.QUANT_INT8)
        o["gu"] = wob.int8_gemm(o["c2"], o["s2"], *self.up, out_dtype=torch.bfloat16)
        o["c3"], o["s3"] = wob.int8_quantize(o["gu"], act=wob.ACT_SILU_MUL)
        o["y3"] = wob.int8_gemm(o["c3"], o["s3"], *self.down, out_dtype=torch.bfloat16)
        o["c4"], o["s4"], o["h4"] = wob.residual_norm(o["y3"], o["h2"], self.norm[4], post_weight=self.norm[5],
                                                      quant=wob.QUANT_MXFP4)
        o["out"] = wob.mxfp4_gemm(o["c4"], o["s4"], *self.head, out_dtype=torch.float32)
        return o


def f64(t):
    return t.double().cpu().numpy()


def within(got, ref, bound, dtype):
    off = np.abs(f64(got) - ref)
    limit = bound + R.HALF_STEP[dtype] * (np.abs(ref) + bound) + R.TINY[dtype]
    assert (off <= limit).all(), (off - limit).max()


@pytest.mark.parametrize("T", (1, 5, 70, 300))
def test_layer_stage_by_stage(wob, T):
    """Each stage against the 64-bit reference on what the stage before it gave."""
    m = Layer(wob, T, 512, 256, 16, 4, T)
    o = m.run()

    def norm(y, r, w, post=None, gate=None, alpha=1.0):
        return R.norm(f64(y), f64(r), f64(w), None if post is None else f64(post), None if gate is None else f64(gate),
                      alpha, np.float64(np.float32(1e-6)))

    def rows8(c, s, n, dn):
        s64 = f64(s)[:, None]
        assert (np.abs(f64(c) * s64 - n) <= (0.5 + 127 * 3 * 2.0 ** -23) * s64 + dn + dn.max(-1, keepdims=True)).all()

    def product(y, c, s, w):
        ref, bound = R.product(c.cpu().numpy(), s.cpu().numpy(), w[0].cpu().numpy(), w[1].cpu().numpy(), None)
        within(y, ref, bound, "bf16")
    h, dh, n, dn = norm(m.x, m.h, m.norm[0])
    within(o["h0"], h, dh, "fp32")
    rows8(o["c0"], o["s0"], n, dn)
    product(o["y0"], o["c0"], o["s0"], m.proj)
    h, dh, n, dn = norm(o["y0"], o["h0"], m.norm[1], m.norm[2], m.gate, 0.5)
    within(o["h1"], h, dh, "fp32")
    within(o["n1"], n, dn, "bf16")
    ids, w = R.route(o["logits"].float().cpu().numpy(), 4, m.bias.cpu().numpy(), True, 4, 2, 2, True, 1.5)
    assert np.array_equal(o["ids"].cpu().numpy(), ids)
    assert (np.abs(f64(o["w"]) - w) <= R.route_bound(w, 4)).all()
    h, dh, n, dn = norm(o["y1"], o["h1"], m.norm[3])
    within(o["h2"], h, dh, "fp32")
    rows8(o["c2"], o["s2"], n, dn)
    product(o["gu"], o["c2"], o["s2"], m.up)
    v, dv = R.silu_mul(f64(o["gu"]))
    rows8(o["c3"], o["s3"], v, dv)
    product(o["y3"], o["c3"], o["s3"], m.down)
    h, dh, n, dn = norm(o["y3"], o["h2"], m.norm[4], m.norm[5])
    within(o["h4"], h, dh, "fp32")
    # the expert stages on these ids and weights (their own tests hold their bounds)
    torch = torch_mod()
    x, ref = o["n1"].double(), torch.zeros_like(o["y1"], dtype=torch.float64)
    for t in range(T):
        for s in range(4):
            e = int(o["ids"][t, s])
            if e < 0:
                continue
            w1 = wob.mxfp4_dequant(m.w1[0][e], m.w1[1][e]).double()
            w2 = wob.mxfp4_dequant(m.w2[0][e], m.w2[1][e]).double()
            gu = w1 @ x[t]
            a = gu[:256] * torch.sigmoid(gu[:256]) * gu[256:]
            ref[t] += o["w"][t, s].double() * (w2 @ a)
    err = float((o["y1"].double() - ref).norm() / ref.norm())
    assert err <= 2 * 2.0 ** -8  # two roundings to bf16: the activated rows and the result


@pytest.mark.parametrize("T", (1, 12, 200))
def test_layer_captured_and_replayed(wob, T):
    torch = torch_mod()
    m = Layer(wob, T, 512, 256, 16, 4, 7 + T)
    g = torch.Generator(device="cuda").manual_seed(T)
    new = [(torch.randn((T, 512), device="cuda", generator=g).bfloat16(),
            torch.randn((T, 512), device="cuda", generator=g)) for _ in range(4)]
    eager = []
    for x, h in new:
        m.x.copy_(x)
        m.h.copy_(h)
        eager.append({k: v.clone() for k, v in m.run().items()})
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.run()
    for k in (0, 1, 2, 3, 1, 0):
        m.x.copy_(new[k][0])
        m.h.copy_(new[k][1])
        graph.replay()
        torch.cuda.synchronize()
        for name, v in out.items():
            assert torch.equal(v, eager[k][name]), (k, name)
        m.run()  # eager work between the replays
        torch.cuda.synchronize()


def test_layers_on_two_streams_at_once(wob):
    torch = torch_mod()
    layers = [Layer(wob, T, 512, 256, 16, 4, 20 + T) for T in (3, 130)]
    want = [{k: v.clone() for k, v in m.run().items()} for m in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [[], []]
    for _ in range(5):
        for i, (s, m) in enumerate(zip(streams, layers)):
            with torch.cuda.stream(s):
                got[i].append(m.run())
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            for name, v in o.items():
                assert torch.equal(v, want[i][name]), (i, name)


@pytest.mark.parametrize("M,N,K", [(40, 2000, 8192), (250, 5376, 8208), (400, 5376, 21520)])
def test_products_share_a_workspace_in_order(wob, M, N, K):
    """Calls that are ordered on one stream may share one workspace, in two captured graphs too."""
    torch = torch_mod()
    need = wob.int8_gemm_workspace_size(M, N, K)
    assert need > 0
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randint(-127, 128, (N, K), device="cuda", generator=g, dtype=torch.int8)
    ws = torch.rand(N, device="cuda", generator=g)
    xs = torch.rand(M, device="cuda", generator=g)
    x = [torch.randint(-127, 128, (M, K), device="cuda", generator=g, dtype=torch.int8) for _ in range(2)]
    want = [(v.double() @ w.double().t()).float() * xs[:, None] * ws for v in x]
    y = [wob.int8_gemm(v, xs, w, ws, out_dtype=torch.float32, workspace=work) for v in x]
    assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])
    graphs, outs = [], []
    for v in x:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(wob.int8_gemm(v, xs, w, ws, out_dtype=torch.float32, workspace=work))
        graphs.append(graph)
    for k in (0, 1, 1, 0):
        work.fill_(0x55)
        graphs[k].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[k], want[k])
    graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_an_operand_on_another_device_is_refused(wob):
    torch = torch_mod()
    x = torch.zeros((4, 64), dtype=torch.int8, device="cuda")
    s = torch.ones(4, device="cuda")
    w, ws = torch.zeros((16, 64), dtype=torch.int8), torch.ones(16)
    with pytest.raises(ValueError):
        wob.int8_gemm(x, s, w, ws)
    with pytest.raises(ValueError):
        wob.int8_gemm(x, s, w.cuda(), ws.cuda(), out=torch.zeros((4, 16), dtype=torch.bfloat16))
    y = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(64, dtype=torch.bfloat16)
    for args, kw in (((y.cpu(), y, v.cuda()), {}), ((y, y.cpu(), v.cuda()), {}), ((y, y, v), {}),
                     ((y, y, v.cuda()), dict(gate=v)), ((y, y, v.cuda()), dict(post_weight=v)),
                     ((y, y, v.cuda()), dict(residual_out=y.cpu())), ((y, y, v.cuda()), dict(out=y.cpu()))):
        with pytest.raises(ValueError):
            wob.residual_norm(*args, **kw)
    l = torch.zeros((4, 16), device="cuda")
    with pytest.raises(ValueError):
        wob.moe_route(l, 2, bias=torch.zeros(16))
    with pytest.raises(ValueError):
        wob.int8_dequant(x, s.cpu())
    torch.cuda.synchronize()
