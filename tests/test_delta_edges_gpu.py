"""The delta rule with one decay per value head and the layer norm at the ends of their ranges: neighbours that are not numbers, no value
heads, more than 2^31 elements, outputs that the caller gives."""

import pytest
import torch

import gated_delta_rule_56_gb300 as kda
from delta_cases import GRADS, Case
from layers_cases import DEV, gen

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("bad", [0, 1, 2])
def test_a_sequence_of_nan_leaves_its_neighbours_as_they_were(dtype, bad):
    """A neighbour's rows lie in the same tile as a sequence's last ones."""
    lengths = [70, 50, 130]
    c = Case(dtype, 1, 0, 1, 2, 128, 128, lengths, seed=21)
    o, fin = c.prefill()
    g = c.backward()
    start = sum(lengths[:bad])
    rows = slice(start, start + lengths[bad])
    for t in (c.q, c.k, c.v, c.g, c.beta, c.d_o):
        t[:, rows] = float("nan")
    o2, fin2 = c.prefill()
    g2 = c.backward()
    kda.check_status()
    rest = torch.ones(sum(lengths), dtype=torch.bool, device=DEV)
    rest[rows] = False
    others = [n for n in range(3) if n != bad]
    assert torch.equal(o[:, rest], o2[:, rest]) and torch.equal(fin[others], fin2[others])
    for name in GRADS:
        assert torch.equal(g[name][others], g2[name][others]) if name == "d_initial_state" else torch.equal(g[name][:, rest], g2[name][:, rest])
    assert torch.isnan(o2[:, rows].float()).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_no_value_heads(dtype):
    q = torch.ones(2, 70, 3, 64, dtype=dtype, device=DEV)
    v, g = torch.empty(2, 70, 0, 64, dtype=dtype, device=DEV), torch.empty(2, 70, 0, device=DEV)
    o, fin = kda.delta_prefill(q, q, v, g, g)
    assert o.shape == (2, 70, 0, 64) and fin.shape == (2, 0, 64, 64)
    grads = kda.delta_backward(q, q, v, g, g, v)
    kda.check_status()
    assert not grads["dq"].any() and not grads["dk"].any()


def test_more_than_2_to_the_31_values():
    T, H = 65600, 256
    r = gen(22)
    q, k = (torch.nn.functional.normalize(r(1, T, 1, 128), dim=-1).to(BF16) for _ in range(2))
    v = torch.empty(1, T, H, 128, dtype=BF16, device=DEV).normal_(generator=torch.Generator(device=DEV).manual_seed(23))
    g, beta = -0.1 * torch.rand(1, T, H, device=DEV), torch.rand(1, T, H, device=DEV)
    assert v.numel() > 2 ** 31
    o, fin = kda.delta_prefill(q, k, v, g, beta)
    one = [t[:, :, H - 1:].contiguous() for t in (v, g, beta)]
    o1, fin1 = kda.delta_prefill(q, k, *one)
    kda.check_status()
    assert torch.equal(o[:, -1000:, H - 1], o1[:, -1000:, 0]) and torch.equal(fin[:, H - 1], fin1[:, 0])
    del o, o1
    y, _ = kda.layer_norm(v, norm="rms")
    y1, _ = kda.layer_norm(v[:, -3:].contiguous(), norm="rms")
    assert torch.equal(y[:, -3:], y1)
    grads = kda.layer_norm_backward(v[:, :, :130], None, y[:, :, :130].contiguous(), norm="rms")
    g1 = kda.layer_norm_backward(v[:, -2:, :130], None, y[:, -2:, :130].contiguous(), norm="rms")
    assert torch.equal(grads["dx"][:, -2:], g1["dx"])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_rows_in_front_of_and_behind_the_outputs_stay(dtype):
    """Outputs given as parts of larger buffers: nothing beside them is written."""
    c = Case(dtype, 1, 0, 1, 2, 64, 64, [33, 0, 97], seed=24)
    T = 130
    buffer = torch.full((T + 2, 2, 64), 7.0, dtype=dtype, device=DEV)
    states = torch.full((5, 2, 64, 64), 7.0, device=DEV)
    o, fin = c.prefill(o=buffer[1:-1].unsqueeze(0), final_state=states[1:4])
    want, want_fin = c.prefill()
    kda.check_status()
    assert torch.equal(o, want) and torch.equal(fin, want_fin)
    assert (buffer[[0, -1]] == 7).all() and (states[[0, 4]] == 7).all()
    x = torch.randn(40, 96, device=DEV).to(dtype)
    ybuf = torch.full((42, 96), 7.0, dtype=dtype, device=DEV)
    y, _ = kda.layer_norm(x, y=ybuf[1:-1])
    assert torch.equal(y, kda.layer_norm(x)[0]) and (ybuf[[0, -1]] == 7).all()


def test_the_binding_refuses_what_does_not_fit():
    c = Case(BF16, 2, 8, 2, 4, 64, 32, seed=25)
    q, k, v, g, b = c.inputs()
    with pytest.raises(ValueError, match="shape"):
        kda.delta_prefill(q, k[:, :, :1], v, g, b)
    with pytest.raises(ValueError, match="shape"):
        kda.delta_prefill(q, k, v, g[:, :, :2], b)
    with pytest.raises(TypeError, match="dtype"):
        kda.delta_prefill(q, k, v, g.to(BF16), b)
    with pytest.raises(ValueError, match="contiguous"):
        kda.delta_prefill(q, k, v, g.mT.contiguous().mT, b)
    with pytest.raises(kda.KDAError, match="multiple"):
        kda.delta_prefill(q, k, v[:, :, :3].contiguous(), g[:, :, :3].contiguous(), b[:, :, :3].contiguous())
    with pytest.raises(kda.KDAError, match="supported"):
        kda.delta_prefill(q, k, torch.zeros(2, 8, 4, 48, dtype=BF16, device=DEV), g, b)
    with pytest.raises(ValueError, match="batch"):
        kda.delta_prefill(q, k, v, g, b, cu_seqlens=torch.tensor([0, 16], dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError, match="shape"):
        kda.delta_prefill(q, k, v, g, b, initial_state=torch.zeros(2, 4, 32, 64, device=DEV))
    with pytest.raises(ValueError, match="distance|dense"):
        kda.delta_prefill(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, g, b)
    x = torch.zeros(4, 8, device=DEV)
    with pytest.raises(ValueError, match="unknown norm"):
        kda.layer_norm(x, norm="max")
    with pytest.raises(ValueError, match="unknown activation"):
        kda.layer_norm(x, gate=x, activation="tanh")
    with pytest.raises(ValueError, match="residual"):
        kda.layer_norm(x, sum_out=x)
    with pytest.raises(ValueError, match="shape"):
        kda.layer_norm(x, torch.ones(4, device=DEV))
    with pytest.raises(ValueError, match="shape"):
        kda.layer_norm(x, gate=torch.zeros(4, 9, device=DEV))
    with pytest.raises(kda.KDAError, match="32768"):
        kda.layer_norm(torch.zeros(1, 32769, device=DEV))


@pytest.mark.parametrize("shape", [(80, 33, 2, 4, 128, 128), (2, 33, 2, 4, 128, 128), (80, 17, 1, 2, 64, 64), (1, 17, 1, 2, 64, 64),
                                   (160, 40, 1, 2, 32, 32), (160, 15, 1, 2, 32, 64), (3, 15, 1, 2, 128, 64)])
def test_fp32_with_many_and_with_few_states(shape):
    c = Case(FP32, *shape, seed=13)
    c.check_prefill(*c.prefill())
    c.check_backward(c.backward())
    kda.check_status()


@pytest.mark.parametrize("B", [2, 160])
def test_a_value_that_is_not_a_number_stays_behind_the_rows_before_it(B):
    c = Case(FP32, B, 40, 1, 2, 64, 64, seed=14)
    q, k, v, g, b = c.inputs()
    o, _ = c.prefill()
    for x in (k, v, g, b):
        y = x.clone()
        y[:, 21] = float("nan")
        got, _ = kda.delta_prefill(*(y if t is x else t for t in (q, k, v, g, b)), initial_state=c.state)
        assert torch.equal(got[:, :21], o[:, :21]) and got[:, 22:].isnan().any()
    kda.check_status()
