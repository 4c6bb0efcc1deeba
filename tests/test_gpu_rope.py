"""attn_qk_norm_rope against a 64-bit implementation.

Tolerance of an element: half a bf16 step of the result, plus 2^-19 of its pair's magnitude: the fp32
path is under 16 roundings of 2^-24 (norm: a sum of D <= 256 squares in a tree, whose relative error is below
12 * 2^-24 and halves under the root; two products and a sum) and a sine and cosine of an angle
rounded to fp32 (2^-24 of up to pi, plus 2 ulp)."""
import math

import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kp():
    from key_prefix_masked_b200 import build
    build.build()
    import key_prefix_masked_b200 as kp
    torch.cuda.init()
    assert kp.device_status() == kp.ATTN_OK
    return kp


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen).to(torch.bfloat16)


def _close(got, want, mag):
    got = got.detach().cpu().double()
    tol = want.abs() * ref.BF16_HALF_STEP + mag * 2.0 ** -19 + 1e-38
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {((got - want).abs() / tol).max():.3g} of the tolerance"


ROTARY = {32: (32, 8, 20, 2), 64: (64, 32, 0), 128: (128, 64, 36), 256: (256, 128, 254)}


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(D, R) for D, rs in ROTARY.items() for R in rs])
def test_packed_projection(kp, D, R, interleaved):
    """q and k as views of one packed [T, Hq + 2 Hkv, D] projection; norm of both."""
    g = torch.Generator().manual_seed(D + R)
    T, Hq, Hkv = 37, 6, 3
    qkv = _randn(g, T, Hq + 2 * Hkv, D)
    w = _randn(g, D) + 1
    wk = torch.randn(D, generator=g)                   # fp32 weights for k
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32)
    inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R) if R else None
    dev = qkv.cuda()
    qo, ko = kp.attn_qk_norm_rope(dev[:, :Hq], dev[:, Hq:Hq + Hkv], pos.cuda(), None if inv is None else inv.cuda(),
                                  q_weight=w.cuda(), k_weight=wk.cuda(), eps=1e-5, interleaved=interleaved, attn_factor=1.25)
    assert torch.equal(dev.cpu(), qkv)                 # the inputs stay
    for got, x, ww in ((qo, qkv[:, :Hq], w), (ko, qkv[:, Hq:Hq + Hkv], wk)):
        _close(got.transpose(0, 1), *ref.rope(x.transpose(0, 1), ww, pos, inv, 1e-5, interleaved, 1.25))


@pytest.mark.parametrize("layout", ["bhtd", "bthd", "inplace"])
@pytest.mark.parametrize("norm", ["both", "q", "none"])
def test_batched_layouts(kp, layout, norm):
    g = torch.Generator().manual_seed(5)
    B, H, Hk, T, D, R = 2, 5, 1, 19, 64, 48
    q, k = _randn(g, B, H, T, D), _randn(g, B, Hk, T, D)
    w = _randn(g, D)
    pos = torch.randint(0, 100000, (B, T), generator=g, dtype=torch.int32)
    inv = 500000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    put = (lambda t: t.transpose(1, 2).contiguous().cuda().transpose(1, 2)) if layout == "bthd" else (lambda t: t.cuda())
    qd, kd = put(q), put(k)
    wq, wk = (w if norm != "none" else None), (w if norm == "both" else None)
    kw = dict(q_out=qd, k_out=kd) if layout == "inplace" else {}
    qo, ko = kp.attn_qk_norm_rope(qd, kd, pos.cuda(), inv.cuda(), q_weight=None if wq is None else wq.cuda(),
                                  k_weight=None if wk is None else wk.cuda(), **kw)
    if layout == "inplace":
        assert qo.data_ptr() == qd.data_ptr() and ko.data_ptr() == kd.data_ptr()
    _close(qo, *ref.rope(q, wq, pos[:, None], inv, 1e-6, False, 1.0))
    _close(ko, *ref.rope(k, wk, pos[:, None], inv, 1e-6, False, 1.0))


def test_far_and_negative_positions(kp):
    """The angle in 64 bits over the whole int32 range; its own error there: 2^31 * 2^-52 / (2 pi) turns."""
    g = torch.Generator().manual_seed(6)
    pos = torch.tensor([0, 1, -1, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int32)
    inv = 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)
    q = _randn(g, 8, 2, 128)
    qo, none = kp.attn_qk_norm_rope(q.cuda(), None, pos.cuda(), inv.cuda())
    assert none is None
    want, mag = ref.rope(q.transpose(0, 1), None, pos, inv, 0.0, False, 1.0)
    _close(qo.transpose(0, 1), want, mag * 2)


@pytest.mark.parametrize("T", [1, 2, 591, 592, 1500])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (12, 12), (40, 7)])
def test_token_counts(kp, T, Hq, Hkv):
    """Few tokens spread their heads over blocks, many do not."""
    g = torch.Generator().manual_seed(T)
    D = 64 if Hq == 12 else 256
    q, k = _randn(g, T, Hq, D), _randn(g, T, Hkv, D)
    w = _randn(g, D)
    pos = torch.arange(T, dtype=torch.int32)
    inv = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    qo, ko = kp.attn_qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), inv.cuda(), q_weight=w.cuda())
    _close(qo.transpose(0, 1), *ref.rope(q.transpose(0, 1), w, pos, inv, 1e-6, False, 1.0))
    _close(ko.transpose(0, 1), *ref.rope(k.transpose(0, 1), None, pos, inv, 1e-6, False, 1.0))


def test_nonfinite_elements_stay_in_their_place(kp):
    """Without a norm, an infinity touches its own pair alone, and unrotated elements nothing."""
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    x[0, 0, 3], x[0, 0, 50] = math.inf, math.nan
    inv = torch.ones(16, dtype=torch.float64)
    y, _ = kp.attn_qk_norm_rope(x.cuda(), None, torch.zeros(1, dtype=torch.int32).cuda(), inv.cuda())
    y = y.cpu().flatten()
    odd = {3, 19, 50}
    assert all((not math.isfinite(y[i])) if i in (3, 50) else y[i] == 0 for i in range(64) if i != 19), odd


def test_on_another_stream_and_in_a_graph(kp):
    g = torch.Generator().manual_seed(7)
    q = _randn(g, 33, 4, 128).cuda()
    pos, inv = torch.arange(33, dtype=torch.int32).cuda(), torch.rand(64, dtype=torch.float64).cuda()
    want, _ = kp.attn_qk_norm_rope(q, None, pos, inv)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, _ = kp.attn_qk_norm_rope(q, None, pos, inv)
    s.synchronize()
    assert torch.equal(got, want)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
    with torch.cuda.graph(graph):
        kp.attn_qk_norm_rope(q, None, pos, inv, q_out=out)
    q.copy_(q.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, kp.attn_qk_norm_rope(q, None, pos, inv)[0])


def test_refusals(kp):
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos, inv = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(32, dtype=torch.float64, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(q=q.half()), dict(q=q[:, :, ::2]), dict(q=q[:0]), dict(k=q[:3]), dict(k=q[None]), dict(positions=pos.long()),
                dict(positions=pos[:3]), dict(inv_freq=inv.float()), dict(q_weight=w[:32]), dict(q_weight=w.half()),
                dict(q_out=q[:3]), dict(q_out=q[:, :1].expand(4, 2, 64)), dict(q=q[:1].expand(4, 2, 64)),
                dict(inv_freq=inv.cpu()), dict(positions=pos.cpu())):
        args = dict(q=q, k=None, positions=pos, inv_freq=inv)
        args.update(bad)
        with pytest.raises(ValueError):
            kp.attn_qk_norm_rope(**args)
    for bad in (dict(eps=-1.0), dict(attn_factor=math.inf),
                dict(inv_freq=torch.ones(33, dtype=torch.float64, device="cuda"))):
        args = dict(q=q, k=None, positions=pos, inv_freq=inv)
        args.update(bad)
        with pytest.raises(kp.AttnError):
            kp.attn_qk_norm_rope(**args)
    assert kp.device_status() == kp.ATTN_OK
