"""Host checks of the serving entry points, the reference's own pins, and the frequency helper (no GPU)."""
import ctypes
import math
import struct

import pytest
import torch

import paged_reference as ref

A = ctypes.c_void_p(0x10000)
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    from key_prefix_masked_b200 import build
    build.build()
    from key_prefix_masked_b200 import _binding
    return _binding.lib()


def _operand(x=0x10000, y=0x10000, w=0, H=2, w32=0, xs=(0, 0, 0), ys=(0, 0, 0)):
    return struct.pack("3P2i6q", x, y, w, H, w32, *xs, *ys)


def _rope(lib, q=None, k=None, pos=A, inv=A, B=1, T=4, D=64, R=64, inter=0, eps=1e-6, f=1.0):
    return lib.attn_qk_norm_rope(_operand() if q is None else q, k, pos, inv, B, T, D, R, inter, eps, f, NULL)


@pytest.mark.parametrize("kw,want", [
    (dict(q=_operand(x=0)), 1), (dict(q=_operand(y=0)), 1), (dict(q=_operand(x=0x10008)), 1),
    (dict(q=_operand(w=0x10004)), 1), (dict(q=_operand(H=0)), 1), (dict(q=_operand(xs=(0, 60, 64))), 1),
    (dict(q=_operand(ys=(0, 64, 32))), 1), (dict(k=_operand(y=0)), 1), (dict(pos=NULL), 1), (dict(inv=NULL), 1),
    (dict(inv=ctypes.c_void_p(0x10004)), 1), (dict(B=0), 1), (dict(T=0), 1), (dict(B=65536, T=65536), 1),
    (dict(R=63), 1), (dict(R=-2), 1), (dict(R=66), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(f=math.inf), 1),
    (dict(D=96), 2), (dict(D=48, R=16), 2),
])
def test_rope_rejects_bad_arguments(lib, kw, want):
    assert _rope(lib, **kw) == want


def _cache(k=0x10000, v=0x10000, ks=0, vs=0, kst=(0, 0, 0), vst=(0, 0, 0), P=4, page=16, H=2, D=64, fmt=0):
    return struct.pack("4P6q5i4x", k, v, ks, vs, *kst, *vst, P, page, H, D, fmt)


BAD_CACHES = [
    (dict(k=0), 1), (dict(v=0), 1), (dict(k=0x10008), 1), (dict(P=0), 1), (dict(page=0), 1), (dict(H=0), 1),
    (dict(P=1 << 20, page=1 << 12), 1), (dict(fmt=1), 1), (dict(fmt=1, ks=0x10000), 1), (dict(fmt=2), 2),
    (dict(page=12), 2), (dict(D=96), 2), (dict(kst=(1024, 60, 64)), 1), (dict(vst=(1024, 64, 32)), 1),
    (dict(kst=(4096, 72, 256)), 1),                                       # heads not a whole number of 64-column blocks apart
    (dict(fmt=1, ks=0x10000, vs=0x10000, kst=(1024, 72, 128)), 1),       # 8-byte rows in an e4m3 cache
    (dict(fmt=1, ks=0x10004, vs=0x10000), 1), (dict(fmt=1, ks=0x10000, vs=0x10001), 1),
    (dict(kst=(2048, 0, 64)), 1), (dict(vst=(0, 1024, 64)), 1),           # broadcast heads, pages
    (dict(D=32, H=65535, kst=(1 << 40, 1 << 39, 32)), 1),                 # more column blocks than an int counts
]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_every_cache_call_rejects_a_bad_cache(lib, kw, want):
    c = _cache(**kw)
    assert lib.attn_cache_write(c, A, A, None, None, A, 3, NULL) == want
    assert lib.attn_cache_read(c, A, 4, 4, A, A, A, None, None, 2, 32, NULL) == want
    assert lib.attn_paged_fwd(c, A, None, A, 4, 4, A, A, A, None, NULL, A, 2, 8, 4, 8, 1, 0.1, NULL) == want


def test_cache_calls_reject_bad_arguments(lib):
    c = _cache()
    w = lib.attn_cache_write
    assert w(c, NULL, A, None, None, A, 3, NULL) == 1
    assert w(c, A, ctypes.c_void_p(0x10008), None, None, A, 3, NULL) == 1
    assert w(c, A, A, None, None, NULL, 3, NULL) == 1
    assert w(c, A, A, None, None, ctypes.c_void_p(0x10002), 3, NULL) == 1
    assert w(c, A, A, None, None, A, 0, NULL) == 1
    assert w(c, A, A, struct.pack("3q", 0, 60, 128), None, A, 3, NULL) == 1
    r = lib.attn_cache_read
    assert r(c, NULL, 4, 4, A, A, A, None, None, 2, 32, NULL) == 1
    assert r(c, A, -4, 4, A, A, A, None, None, 2, 32, NULL) == 1
    assert r(c, A, 4, 0, A, A, A, None, None, 2, 32, NULL) == 1
    assert r(c, A, 4, 4, NULL, A, A, None, None, 2, 32, NULL) == 1
    assert r(c, A, 4, 4, A, A, NULL, None, None, 2, 32, NULL) == 1
    assert r(c, A, 4, 4, A, A, A, None, None, 0, 32, NULL) == 1
    assert r(c, A, 4, 4, A, A, A, None, None, 2, 0, NULL) == 1
    assert r(c, A, 4, 4, A, A, A, struct.pack("3q", 0, 2048, 32), None, 2, 32, NULL) == 1


def test_paged_rejects_bad_arguments(lib):
    c = _cache()

    def f(q=A, table=A, stride=4, n=4, kv=A, qs=A, out=A, lse=NULL, ws=A, B=2, T=8, Hq=4, mq=8, scale=0.1,
          qst=None):
        return lib.attn_paged_fwd(c, q, qst, table, stride, n, kv, qs, out, None, lse, ws, B, T, Hq, mq, 1, scale, NULL)

    bad = ctypes.c_void_p(0x10002)
    for kw in (dict(q=NULL), dict(q=ctypes.c_void_p(0x10008)), dict(out=NULL), dict(table=NULL), dict(table=bad), dict(kv=NULL),
               dict(kv=bad), dict(qs=bad), dict(lse=bad), dict(stride=-1), dict(n=0), dict(n=1 << 28), dict(B=0), dict(T=0),
               dict(Hq=0), dict(Hq=5), dict(Hq=2 * 129), dict(mq=0), dict(scale=math.nan),
               dict(qs=NULL), dict(ws=NULL, mq=1), dict(ws=ctypes.c_void_p(0x10008), mq=1), dict(qst=struct.pack("3q", 0, 64, 252)),
               dict(qst=struct.pack("3q", 0, 0, 256)), dict(qst=struct.pack("3q", 0, 64, 0))):
        assert f(**kw) == 1, kw


def test_workspace_of_any_size_of_work(lib):
    w = lib.attn_paged_workspace_bytes
    for D in (32, 64, 128, 256):
        for max_q, G in ((1, 1), (16, 1), (17, 1), (4096, 4), (2 ** 31 - 1, 1), (2 ** 31 - 1, 128)):
            small = w(1, 2 ** 31 - 1, G, 1, D, 16, 1, max_q)
            large = w(2 ** 20, 2 ** 31 - 1, 16 * G, 16, D, 16, 4096, max_q)
            most = w(2 ** 31 - 1, 2 ** 31 - 1, 65535 * G, 65535, D, 2 ** 20, 2 ** 11 - 1, max_q)     # products beyond 64 bits
            assert 0 < small <= large == most < 2 ** 28
    for bad in (dict(B=0), dict(T=0), dict(Hq=3), dict(Hkv=0), dict(D=0), dict(page=0), dict(pages=0), dict(mq=0)):
        a = dict(B=2, T=8, Hq=4, Hkv=2, D=64, page=16, pages=4, mq=8)
        a.update(bad)
        assert w(a["B"], a["T"], a["Hq"], a["Hkv"], a["D"], a["page"], a["pages"], a["mq"]) == 0


def test_python_checks_refuse(lib):
    import key_prefix_masked_b200 as kp
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        kp.attn_qk_norm_rope(x, None, torch.zeros(4, dtype=torch.int32), f)
    with pytest.raises(ValueError, match="CUDA"):
        kp.attn_cache_write(x, x, torch.zeros(4, dtype=torch.int32), x[None], x[None])
    with pytest.raises(ValueError, match="CUDA"):
        kp.attn_paged_fwd(x, x[None], x[None], None, None)
    for kw in (dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=2, scaling="ntk", factor=2.0), dict(rotary_dim=8, factor=0.5),
               dict(rotary_dim=8, scaling="yarn", factor=4.0), dict(rotary_dim=8, scaling="other")):
        with pytest.raises(ValueError):
            kp.rope_inv_freq(device="cpu", **kw)


def test_inv_freq():
    from key_prefix_masked_b200 import rope_inv_freq
    f, a = rope_inv_freq(8, device="cpu")
    assert a == 1.0 and f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-15)
    assert torch.equal(rope_inv_freq(8, scaling="linear", factor=4.0, device="cpu")[0], f / 4)
    n, _ = rope_inv_freq(8, scaling="ntk", factor=4.0, device="cpu")
    assert n[0] == 1.0 and abs(n[-1] / (f[-1] / 4) - 1) < 1e-12       # fastest kept, slowest interpolated
    y, a = rope_inv_freq(64, scaling="yarn", factor=8.0, original_context=4096, device="cpu")
    g, _ = rope_inv_freq(64, device="cpu")
    assert abs(a - (0.1 * math.log(8.0) + 1)) < 1e-15
    turns = 4096 * g / (2 * math.pi)
    assert torch.equal(y[turns >= 32], g[turns >= 32]) and torch.allclose(y[turns <= 1], g[turns <= 1] / 8, rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((y[mid] < g[mid]) & (y[mid] > g[mid] / 8)).all()


@pytest.mark.parametrize("base,context,factor,first,last", [
    # 128 ln(4096 / (32 * 2 pi)) / (2 ln 10^4) = 128 * 3.0142 / 18.4207 = 20.94, and 128 ln(4096 / (2 pi)) / 18.4207 =
    # 128 * 6.4799 / 18.4207 = 45.03: pairs up to 20 are kept, those from 46 on divided in full
    (1e4, 4096, 8.0, 20, 46),
    # 128 * 5.0936 / 27.6310 = 23.60 and 128 * 8.5594 / 27.6310 = 39.65
    (1e6, 32768, 4.0, 23, 40),
    # 128 * -1.1447 / 18.4207 = -7.95, cut to 0, and 128 * 2.3210 / 18.4207 = 16.13
    (1e4, 64, 16.0, 0, 17),
])
def test_yarn_ramps_over_the_pair_index(base, context, factor, first, last):
    from key_prefix_masked_b200 import rope_inv_freq
    f, a = rope_inv_freq(128, base=base, scaling="yarn", factor=factor, original_context=context, device="cpu")
    assert abs(a - (0.1 * math.log(factor) + 1)) < 1e-15
    for i in range(64):
        kept = min(max((last - i) / (last - first), 0.0), 1.0)
        want = base ** (-i / 64) * (kept + (1 - kept) / factor)
        assert abs(f[i].item() / want - 1) < 1e-12, i


def test_yarn_in_turns():
    """Pair 35 at base 10^4 and R 128 turns 4096 * 10^(-4 * 35 / 64) / (2 pi) = 4.2333 times over 4096 positions."""
    from key_prefix_masked_b200 import rope_inv_freq
    f, a = rope_inv_freq(128, scaling="yarn_turns", factor=8.0, original_context=4096, device="cpu")
    kept = (4.2333 - 1) / 31
    assert abs(f[35].item() / (10 ** (-4 * 35 / 64) * (kept + (1 - kept) / 8)) - 1) < 1e-5
    assert abs(a - (0.1 * math.log(8.0) + 1)) < 1e-15
    for kw in (dict(original_context=-4), dict(beta_fast=1.0), dict(beta_slow=0.0), dict(base=1.0)):
        for scaling in ("yarn", "yarn_turns"):
            with pytest.raises(ValueError):
                rope_inv_freq(**{**dict(rotary_dim=8, scaling=scaling, factor=4.0, original_context=64, device="cpu"), **kw})


def test_reference_table_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    t = codes.view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.nan_to_num(t, nan=7e7), torch.nan_to_num(ref.e4m3_table(), nan=7e7))


def test_reference_quantiser():
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(64, 32, generator=g) * 2.0 ** torch.randint(-20, 20, (64, 1), generator=g)).to(torch.bfloat16)
    c, s = ref.quantise(x)
    back = ref.dequantise(c, s)
    amax = x.double().abs().amax(-1, keepdim=True)
    # half a step: 2^-4 of a normal value, 2^-10 2^e below 2^-6 2^e (2^e < amax / 224)
    assert ((back - x.double()).abs() <= torch.maximum(x.double().abs() * 2.0 ** -4, amax / 224 * 2.0 ** -10)).all()
    assert ((amax[:, 0] / 2.0 ** (s.double() - 127) <= 448) & (amax[:, 0] / 2.0 ** (s.double() - 128) > 448)).all()
    assert torch.equal(back, back.to(torch.bfloat16).double())        # every stored value is a bf16 number


def test_reference_attention_against_sdpa():
    g = torch.Generator().manual_seed(2)
    B, Hq, Hkv, D, page, kv, n = 2, 4, 2, 32, 8, [21, 16], [5, 3]
    table = torch.tensor([[4, 0, 2], [5, 1, -1]])
    k, v = (torch.randn(6, Hkv, page, D, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(sum(n), Hq, D, generator=g).to(torch.bfloat16)
    start = [0, 5, 8]
    for causal in (False, True):
        out, lse, _, _ = ref.paged(q, k, v, table, kv, start, causal, 0.2)
        for b in range(B):
            kb, vb = (ref.gather(x, table[b], kv[b]).repeat_interleave(2, 0) for x in (k, v))
            mask = torch.ones(n[b], kv[b], dtype=torch.bool)
            if causal:
                mask = mask.tril(kv[b] - n[b])
            want = torch.nn.functional.scaled_dot_product_attention(
                q[start[b]:start[b + 1]].double().transpose(0, 1), kb, vb, attn_mask=mask, scale=0.2)
            assert (out[start[b]:start[b + 1]].transpose(0, 1) - want).abs().max() < 1e-12


def test_calls_run_on_their_tensors_device(monkeypatch):
    """With another device current, a call is made with the tensors' device current and on that one's stream."""
    from key_prefix_masked_b200 import paged
    current, seen = [0], []

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    monkeypatch.setattr(paged, "_current_device", lambda: current[0])
    monkeypatch.setattr(paged, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setitem(paged._functions, "f", lambda *args: seen.append((current[0], args)) or 0)
    for index in (0, 1, 0):
        paged._call("f", torch.device("cuda", index), 7)
        assert seen[-1] == (index, (7, 1000 + index)) and current[0] == 0
    monkeypatch.setitem(paged._functions, "f", lambda *args: 1)
    with pytest.raises(paged._binding.AttnError):
        paged._call("f", torch.device("cuda", 1), 7)
    assert current[0] == 0
