"""The row norms (forward, backward) against a float64 evaluation of their formulas.

Tolerances, from the number of roundings: a bf16 output of magnitude a is off by
at most a 2^-8 (its one rounding: 8 significant bits) plus the fp32 arithmetic in front of it.  A row
statistic of n terms is a sum of positive terms (or, for the mean, is compared on
the scale of its terms) taken as 8 consecutive fused steps per lane and then a tree:
at most 8 + 10 + 16 roundings of 2^-24, so 2^-18 relative covers it; an output needs a
handful of roundings more.  A column sum over r rows is off by at most
(rows per workgroup + 2 * 32 + 64) 2^-24 <= (r + 128) 2^-24 of the sum of magnitudes,
plus 2^-18 per term for the statistics inside it.
"""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu

EPS = 1e-5
F64 = torch.float64


@pytest.fixture(scope="module")
def fp8():
    import fp8_precision_amd
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return fp8_precision_amd


def inputs(rows, cols, f32, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)
    wide = torch.float32 if f32 else torch.bfloat16
    return {
        "x": (n(rows, cols) * 2 + 0.5).to(wide).cuda(), "add": n(rows, cols).to(torch.bfloat16).cuda(),
        "weight": (1 + 0.2 * n(cols)).to(torch.bfloat16).cuda(), "bias": n(cols).to(torch.bfloat16).cuda(),
        "dy": n(rows, cols).to(torch.bfloat16).cuda(), "dres": n(rows, cols).to(wide).cuda(),
    }


def forward64(x, add, weight, bias, rms):
    s = x.to(F64) + (0 if add is None else add.to(F64))
    mean = torch.zeros_like(s[:, :1]) if rms else s.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((s - mean) ** 2).mean(1, keepdim=True) + EPS)
    h = (s - mean) * rstd
    return h * weight.to(F64) + (0 if bias is None else bias.to(F64)), s, mean, rstd, h


SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 8), (2, 511), (2, 512), (4, 513), (7, 1000), (33, 1027), (300, 640),
          (9, 4096), (1025, 2048), (3, 8191), (2, 8192), (3, 8200), (2, 8203), (2, 16384), (600, 5120)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("joined", [True, False])
def test_forward(fp8, rows, cols, rms, f32, joined):
    say("norm forward", rows, cols, rms, f32, joined)
    t = inputs(rows, cols, f32, rows * 31 + cols)
    add, bias = (t["add"] if joined else None), (None if rms else t["bias"])
    top = torch.full((1,), 0.25, device="cuda")
    y, s, mean, rstd = fp8.norm(t["x"], t["weight"], bias, add=add, eps=EPS, rms=rms, absmax=top)
    y64, s64, m64, r64, h64 = forward64(t["x"], add, t["weight"], bias, rms)
    size = (h64 * t["weight"].to(F64)).abs() + (0 if bias is None else bias.to(F64).abs())
    # the mean's own error moves every element of a row by as much
    moved = (s64.abs().mean(1, keepdim=True) * r64 * 2.0 ** -18 * t["weight"].to(F64).abs()) if not rms else 0
    assert ((y.to(F64) - y64).abs() <= y64.abs() * 2.0 ** -8 * 1.01 + size * 2.0 ** -17 + moved * 2 + 1e-30).all()
    assert ((rstd.to(F64) - r64[:, 0]).abs() <= r64[:, 0] * 2.0 ** -18 * 4).all()
    if not rms:
        assert ((mean.to(F64) - m64[:, 0]).abs() <= s64.abs().mean(1) * 2.0 ** -18).all()
    else:
        assert mean is None
    if joined:
        rel = 2.0 ** -23 if f32 else 2.0 ** -8 * 1.01
        assert s.dtype == t["x"].dtype and ((s.to(F64) - s64).abs() <= s64.abs() * rel + 1e-30).all()
    else:
        assert s is t["x"]
    assert top.item() == max(0.25, y.float().abs().max().item())


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("joined", [True, False])
def test_backward(fp8, rows, cols, rms, f32, joined):
    say("norm backward", rows, cols, rms, f32, joined)
    t = inputs(rows, cols, f32, rows * 37 + cols)
    _, s, mean, rstd = fp8.norm(t["x"], t["weight"], None if rms else t["bias"], eps=EPS, rms=rms)
    dx, dw, db = fp8.norm_backward(t["dy"], s, t["weight"], mean, rstd, dres=t["dres"] if joined else None,
                                   want_dbias=not rms)
    h = ((s.to(F64) - (0 if rms else mean.to(F64)[:, None])) * rstd.to(F64)[:, None])
    dy = t["dy"].to(F64)
    g = dy * t["weight"].to(F64)
    along, flat = (g * h).mean(1, keepdim=True), (0 if rms else g.mean(1, keepdim=True))
    r = rstd.to(F64)[:, None]
    dx64 = r * (g - h * along - flat) + (t["dres"].to(F64) if joined else 0)
    size = r * (g.abs() + h.abs() * (g * h).abs().mean(1, keepdim=True) + (0 if rms else g.abs().mean(1, keepdim=True)))
    size = size + (t["dres"].to(F64).abs() if joined else 0)
    rel = 0 if f32 else 2.0 ** -8 * 1.01
    assert dx.dtype == t["x"].dtype
    assert ((dx.to(F64) - dx64).abs() <= dx64.abs() * rel + size * 2.0 ** -17 + 1e-30).all()
    col = (rows + 128) * 2.0 ** -24 + 2.0 ** -18
    assert ((dw.to(F64) - (dy * h).sum(0)).abs() <= (dy * h).abs().sum(0) * col + 1e-30).all()
    if rms:
        assert db is None
    else:
        assert ((db.to(F64) - dy.sum(0)).abs() <= dy.abs().sum(0) * col + 1e-30).all()


# Rows narrow enough that a workgroup takes several: one per head of a projection, as many
# as make its workgroups walk, and counts that leave the last set of rows ragged.
NARROW = [(16, 16), (17, 128), (5, 129), (9, 250), (1001, 64), (33, 300), (70, 480), (40003, 128), (20011, 200)]


@pytest.mark.parametrize("rows,cols", NARROW)
@pytest.mark.parametrize("rms,f32,joined", [(True, False, False), (False, False, True), (True, True, True),
                                            (False, True, False)])
def test_narrow_rows(fp8, rows, cols, rms, f32, joined):
    test_forward(fp8, rows, cols, rms, f32, joined)
    test_backward(fp8, rows, cols, rms, f32, joined)


@pytest.mark.parametrize("rms", [True, False])
def test_gradient_against_differences(fp8, rms):
    """dx, dweight and dbias against central differences of the float64 forward."""
    t = inputs(3, 40, True, 5)
    bias = None if rms else t["bias"]
    _, s, mean, rstd = fp8.norm(t["x"], t["weight"], bias, eps=EPS, rms=rms)
    dx, dw, db = fp8.norm_backward(t["dy"], s, t["weight"], mean, rstd, want_dbias=not rms)
    dy, step = t["dy"].to(F64), 1e-6

    def loss(x, w, b):
        return (forward64(x, None, w, b, rms)[0] * dy).sum()

    def difference(name):
        base = {"x": t["x"].to(F64), "w": t["weight"].to(F64), "b": None if rms else bias.to(F64)}
        grad = torch.zeros_like(base[name])
        for i in range(base[name].numel()):
            v = []
            for sign in (1, -1):
                moved = {k: (None if z is None else z.clone()) for k, z in base.items()}
                moved[name].view(-1)[i] += sign * step
                v.append(loss(moved["x"], moved["w"], moved["b"]))
            grad.view(-1)[i] = (v[0] - v[1]) / (2 * step)
        return grad

    # fp32 gradients of order 1; differences in float64 are good to about 1e-8
    assert (dx.to(F64) - difference("x")).abs().max() < 1e-4
    assert (dw.to(F64) - difference("w")).abs().max() < 1e-4
    if not rms:
        assert (db.to(F64) - difference("b")).abs().max() < 1e-4


def test_values_at_the_edge(fp8):
    """A row of zeros, one of a single huge value, one with an infinity and one with a
    NaN: each stays its own row's affair."""
    x = torch.ones(5, 256, device="cuda")
    x[1] = 0
    x[2, 3] = 1e15
    x[3, 7] = float("inf")
    x[4, 9] = float("nan")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    y, _, _, r = fp8.norm(x, w, rms=True, eps=1e-6)
    assert torch.isfinite(y[:3].float()).all() and (y[1] == 0).all()
    assert abs(y[2, 3].item() - 16) < 0.1 and r[1].item() == pytest.approx(1e3, rel=1e-6)
    assert torch.isnan(y[3, 7]) and torch.isnan(y[4].float()).all()
    y, _, m, _ = fp8.norm(x, w, rms=False, eps=1e-6)
    assert (y[:2] == 0).all() and m[0].item() == 1


def test_same_bytes_every_time_and_on_another_stream(fp8):
    t = inputs(700, 5120, False, 3)
    run = lambda: fp8.norm_backward(t["dy"], s, t["weight"], None, r, dres=t["dres"])
    _, s, _, r = fp8.norm(t["x"], t["weight"], rms=True)
    a = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = run()
    side.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals(fp8):
    t = inputs(4, 64, False, 1)
    x, w, dy = t["x"], t["weight"], t["dy"]
    with pytest.raises(TypeError):
        fp8.norm(x.half(), w)
    with pytest.raises(ValueError):
        fp8.norm(x.t(), w)
    with pytest.raises(ValueError):
        fp8.norm(x, w[:32])
    with pytest.raises(ValueError):
        fp8.norm(x, w, out_sum=torch.empty_like(x))
    with pytest.raises(fp8.Fp8Error, match="no mean and no bias"):
        fp8.norm(x, w, t["bias"], rms=True)
    with pytest.raises(fp8.Fp8Error, match="eps"):
        fp8.norm(x, w, eps=float("nan"))
    with pytest.raises(fp8.Fp8Error, match="overlapping"):
        fp8.norm(x, w, y=x)
    with pytest.raises(fp8.Fp8Error, match="positive"):
        fp8.norm(x[:0], w)
    wide = torch.zeros(1, 16385, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fp8.Fp8Error, match="16384"):
        fp8.norm(wide, wide[0])
    _, s, _, r = fp8.norm(x, w)
    with pytest.raises(ValueError):
        fp8.norm_backward(dy, s, w, None, r, want_dbias=True)
    with pytest.raises(TypeError):
        fp8.norm_backward(dy, s, w, None, r, dres=t["dres"].float())
    with pytest.raises(fp8.Fp8Error, match="overlapping"):
        fp8.norm_backward(dy, s, w, None, r, dx=dy)
