"""Layer norm and RMS norm with residual and gate on the GPU against their 64-bit definition."""

import pytest
import torch

import delta_ref as ref
import gated_delta_rule_56_gb300 as kda
from layers_cases import DEV, HALF, ULP32, close, d64, gen, near, strided

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
EPS = 1e-6


class Case:
    def __init__(self, dtype, shape, weight=True, bias=True, residual=False, gate=None, rms=False, seed=0, shift=0.5):
        r = gen(seed)
        D = shape[-1]
        self.dtype, self.rms, self.kind = dtype, rms, gate or "silu"
        self.x = (1.5 * r(*shape) + shift).to(dtype)
        self.res = (2 * r(*shape)).to(dtype) if residual else None
        self.z = (2 * r(*shape)).to(dtype) if gate else None
        self.w = (1 + 0.3 * r(D)).to(dtype) if weight else None
        self.b = (0.3 * r(D)).to(dtype) if bias else None
        self.dy, self.ds = r(*shape).to(dtype), r(*shape).to(dtype) if residual else None

    def more(self):
        return dict(bias=self.b, gate=self.z, activation=self.kind, norm="rms" if self.rms else "layer", eps=EPS)

    def forward(self, **out):
        return kda.layer_norm(self.x, self.w, residual=self.res, **self.more(), **out)

    def backward(self):
        return kda.layer_norm_backward(self.x, self.w, self.dy, d_sum=self.ds, **self.more())

    def tolerance(self):
        # A line's sums: chains of up to 32 values and 10 levels, so 42 half steps at most; the mean's error moves every difference by as
        # much of the line's largest value, the root halves the squares' error. Sigmoid and root: 8. Against |n| + 1, the size of a line.
        return 64 * ULP32

    def check_forward(self, y, s):
        yr, sr = ref.layer_norm(d64(self.x), d64(self.w), d64(self.b), d64(self.res), d64(self.z), self.kind, self.rms, EPS)
        big = 1 if self.z is None else ref.act(d64(self.z), self.kind).abs()
        wide = (1 if self.w is None else d64(self.w).abs()) * 2
        spread = sr.abs().amax(-1, keepdim=True) / (sr - (0 if self.rms else sr.mean(-1, keepdim=True))).square().mean(-1, keepdim=True).add(EPS).sqrt()
        close("y", y, yr, HALF[self.dtype] * 1.001 * yr.abs() + self.tolerance() * big * wide * (1 + spread) + 1e-30)
        if s is not None:
            close("sum", s, sr, HALF[self.dtype] * 1.001 * sr.abs() + 1e-30)
        assert (s is None) == (self.res is None)

    def check_backward(self, g):
        dx, dw, db, dz = ref.layer_norm_backward(d64(self.x), d64(self.w), d64(self.b), d64(self.z), self.kind, self.rms, EPS, d64(self.dy), d64(self.ds))
        # As above; the weights' sums run over chains of lines per block, of random signs: sqrt(lines) half steps of their own size
        lines = self.x.numel() // self.x.shape[-1]
        tol = self.tolerance()
        # dx = r (t - mean(t) - h r^2 mean(t h)): differences of terms of t's size, each right to tol, so dx is off by tol of r t, whatever
        # the difference leaves (at width 1 nothing but eps / h^2 of it).
        x = d64(self.x)
        h = x if self.rms else x - x.mean(-1, keepdim=True)
        t = d64(self.dy) * (1 if self.z is None else ref.act(d64(self.z), self.kind)) * (1 if self.w is None else d64(self.w))
        terms = (t / (h.square().mean(-1, keepdim=True) + EPS).sqrt()).norm()
        off = (d64(g["dx"]) - dx).norm()
        assert off <= 4 * tol * (dx.norm() + terms), f"dx: off by {off:.3e}, terms {terms:.3e}, value {dx.norm():.3e}"
        for name, want in (("dweight", dw), ("dbias", db)):
            assert (g[name] is None) == (want is None)
            if want is not None:
                near(name, g[name], want, 4 * tol + ULP32 * lines ** 0.5)
        assert (g["dgate"] is None) == (dz is None)
        if dz is not None:
            near("dgate", g["dgate"], dz, 4 * tol)


WIDTHS = [1, 2, 7, 8, 31, 32, 33, 64, 100, 128, 200, 256, 257, 512, 520, 1000, 1024, 1025, 1531, 2048, 2056, 4096, 4100, 8192, 8193, 16384, 16400, 32768,
          32767]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D", WIDTHS)
def test_every_width(dtype, D):
    lines = 3 if D > 4096 else 37
    c = Case(dtype, (lines, D), residual=True, seed=1)
    c.check_forward(*c.forward())
    r = Case(dtype, (lines, D), bias=False, gate="silu", rms=True, seed=2)
    r.check_forward(*r.forward())
    c.check_backward(c.backward())
    r.check_backward(r.backward())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("weight,bias,residual,gate,rms", [
    (False, False, False, None, False), (False, False, True, "sigmoid", True), (True, False, True, "silu", False),
    (False, True, False, "sigmoid", False), (True, True, True, "silu", True), (True, False, False, None, True)])
@pytest.mark.parametrize("shape", [(2, 5, 3, 128), (3, 700), (1100, 4, 64)])
def test_every_option(dtype, weight, bias, residual, gate, rms, shape):
    c = Case(dtype, shape, weight, bias, residual, gate, rms, seed=3)
    c.check_forward(*c.forward())
    g = c.backward()
    c.check_backward(g)
    again = c.backward()
    assert all(torch.equal(g[k], again[k]) for k in g if g[k] is not None), "the same bits every time"


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape,lead", [((2, 9, 4, 128), 2), ((21, 136), 1), ((2, 11, 72), 2)])
def test_strided_rows(dtype, shape, lead):
    c = Case(dtype, shape, residual=True, gate="silu", seed=4)
    y, s = c.forward()
    g = c.backward()
    for pad, offset in ((16, 8), (3, 1)):
        v = Case(dtype, shape, residual=True, gate="silu", seed=4)
        v.x, v.res, v.z = (strided(t, lead, pad, offset) for t in (c.x, c.res, c.z))
        y2, s2 = v.forward()
        v.check_forward(y2, s2)
        v.check_backward(v.backward())
        assert torch.equal(s, s2)
        mixed = Case(dtype, shape, residual=True, gate="silu", seed=4)
        mixed.z = v.z
        mixed.check_forward(*mixed.forward())
        mixed.check_backward(mixed.backward())
    assert g["dx"].shape == c.x.shape


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_in_place(dtype):
    for shape in ((40, 4, 128), (5, 4096), (6, 77)):
        c = Case(dtype, shape, residual=True, gate="sigmoid", seed=5)
        y, s = c.forward()
        for name in ("x", "res"):
            v = Case(dtype, shape, residual=True, gate="sigmoid", seed=5)
            y2, s2 = v.forward(sum_out=getattr(v, name))
            assert s2 is getattr(v, name) and torch.equal(y, y2) and torch.equal(s, s2)
            v = Case(dtype, shape, residual=True, gate="sigmoid", seed=5)
            y2, s2 = v.forward(y=getattr(v, name))
            assert torch.equal(y, y2) and torch.equal(s, s2)


def test_large_means_keep_the_variance():
    """A mean 1000 times the spread: the differences are taken before the squares."""
    c = Case(FP32, (8, 1000), seed=6, shift=1500.0)
    c.check_forward(*c.forward())
    c = Case(FP32, (8, 4096), bias=False, seed=6, shift=1500.0)
    c.check_forward(*c.forward())


def test_constant_zero_infinite_and_nan_rows():
    for dtype in (BF16, FP32):
        for D in (128, 300, 4096):
            for rms in (False, True):
                c = Case(dtype, (9, D), residual=False, rms=rms, seed=7)
                clean, _ = c.forward()
                gc = c.backward()
                c.x[2], c.x[4, 3], c.x[6, 5] = 0, float("nan"), float("inf")
                y, _ = c.forward()
                g = c.backward()
                ok = [0, 1, 3, 5, 7, 8]
                assert torch.equal(y[ok], clean[ok]) and torch.equal(g["dx"][ok], gc["dx"][ok])
                assert torch.equal(y[2], c.b) and torch.isfinite(g["dx"][2]).all()
                assert torch.isnan(y[4].float()).all() and torch.isnan(y[6].float()).any()


def test_no_rows():
    c = Case(BF16, (0, 128), residual=True, gate="silu", seed=8)
    y, s = c.forward()
    assert y.shape == s.shape == (0, 128)
    g = c.backward()
    assert g["dx"].shape == (0, 128) and not g["dweight"].any() and not g["dbias"].any()
    h = Case(FP32, (3, 0, 128), seed=8)
    assert h.forward()[0].shape == (3, 0, 128)
    assert not h.backward()["dweight"].any()


def test_captured_and_replayed_with_many_lines():
    c = Case(BF16, (5003, 4, 128), gate="silu", rms=True, bias=False, seed=9)
    y, _ = c.forward()
    g = c.backward()
    c.check_backward(g)
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append((c.forward()[0], c.backward()))
        graphs.append(graph)
    for i in (0, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    for y2, g2 in outs:
        assert torch.equal(y, y2) and all(torch.equal(g[k], g2[k]) for k in g if g[k] is not None)
    assert g["dx"].device == torch.device(DEV)
