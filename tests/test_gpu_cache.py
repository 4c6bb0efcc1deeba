"""attn_cache_write and attn_cache_read: exact, so everything is compared for equality."""
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


def _pool(P, H, page, D, e4m3, layout="head", seed=0):
    """Caches with content; layout "slot": memory is [P, page, H, D]."""
    g = torch.Generator().manual_seed(seed)
    caches, scales = [], []
    for _ in range(2):
        x = torch.randint(0, 0x7F, (P, H, page, D), generator=g, dtype=torch.uint8)
        c = x if e4m3 else (x.double() - 60).to(torch.bfloat16)
        if layout == "slot":
            c = c.transpose(1, 2).contiguous().transpose(1, 2)
        caches.append(c)
        scales.append(torch.randint(100, 150, (P, H, page), generator=g, dtype=torch.uint8) if e4m3 else None)
    return caches, scales


def _dev(caches, scales):
    c = [x.cuda() for x in caches]
    if caches[0].dtype == torch.uint8:
        c = [x.view(torch.float8_e4m3fn) for x in c]
    return c, dict(zip(("k_scale", "v_scale"), (s.cuda() for s in scales))) if scales[0] is not None else {}


def _bytes(c):
    return c.view(torch.uint8).cpu() if c.dtype == torch.float8_e4m3fn else c.view(torch.int16).cpu()


def _rows(g, T, H, D):
    """Ordinary rows, and one each of zeros, NaN, infinity, the largest and the smallest numbers."""
    x = (torch.randn(T, H, D, generator=g) * 2.0 ** torch.randint(-12, 12, (T, H, 1), generator=g)).to(torch.bfloat16)
    f = x.view(-1, D)
    special = [0.0, math.nan, math.inf, 3.3895e38, 2.0 ** -126, 2.0 ** -133, 448.0, 449.0, 2.0 ** -120]
    for r, s in enumerate(special):
        if r < f.shape[0]:
            f[r] = 0.0
            f[r, (7 * r) % D] = s
            if s and math.isfinite(s):
                f[r, (7 * r + 1) % D] = -s / 2
    return x


@pytest.mark.parametrize("layout", ["head", "slot"])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,page,H,T", [(32, 8, 3, 11), (64, 16, 1, 1), (128, 24, 2, 40), (256, 128, 5, 33), (128, 16, 8, 100)])
def test_write_then_read(kp, D, page, H, T, e4m3, layout):
    g = torch.Generator().manual_seed(D + T)
    P = -(-T // page) + 3
    caches, scales = _pool(P, H, page, D, e4m3, layout)
    k, v = _rows(g, T, H, D), torch.flip(_rows(g, T, H, D), (0,))
    slots = torch.randperm(P * page, generator=g)[:T].to(torch.int32)
    if T > 4:
        slots[3] = -7                                  # skipped
    dc, ds = _dev(caches, scales)
    packed = torch.cat((k, v), 1).cuda()               # k and v as views of one tensor
    kp.attn_cache_write(packed[:, :H], packed[:, H:], slots.cuda(), dc[0], dc[1], **ds)
    want, want_s = [c.clone() for c in caches], [None if s is None else s.clone() for s in scales]
    for i, x in enumerate((k, v)):
        codes, sc = ref.quantise(x) if e4m3 else (x, None)
        for t, s in enumerate(slots.tolist()):
            if s >= 0:
                want[i][s // page, :, s % page] = codes[t]
                if e4m3:
                    want_s[i][s // page, :, s % page] = sc[t]
    for i in range(2):
        assert torch.equal(_bytes(dc[i]), want[i].view(torch.int16) if not e4m3 else want[i]), "stored rows"
        if e4m3:
            assert torch.equal(ds["kv"[i] + "_scale"].cpu(), want_s[i]), "scales"
    assert kp.device_status() == kp.ATTN_OK
    # read back: three sequences, one empty, one ending inside a page
    perm = torch.randperm(P, generator=g).to(torch.int32)
    n = min(P, 3)
    table = torch.full((3, n + 1), -1, dtype=torch.int32)
    table[0, :n], table[1, :1] = perm[:n], perm[-1:]
    lens = [n * page - 3, page - 5 if page > 5 else 1, 0]
    Tk = n * page + 2
    for out_layout in ("bhtd", "bthd"):
        shape = (3, H, Tk, D) if out_layout == "bhtd" else (3, Tk, H, D)
        outs = [torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        if out_layout == "bthd":
            outs = [o.transpose(1, 2) for o in outs]
        kp.attn_cache_read(dc[0], dc[1], table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), k_out=outs[0],
                           v_out=outs[1], **ds)
        for i in range(2):
            vals = ref.dequantise(want[i], want_s[i]) if e4m3 else want[i].double()
            exp = torch.full((3, H, Tk, D), 7.0, dtype=torch.float64)
            for b, m in enumerate(lens):
                exp[b, :, :m] = ref.gather(vals, table[b], m)
            got = outs[i].cpu().double()
            assert torch.equal(torch.isnan(got), torch.isnan(exp))
            assert torch.equal(torch.nan_to_num(got, nan=0.0, posinf=1e39, neginf=-1e39),
                               torch.nan_to_num(exp, nan=0.0, posinf=1e39, neginf=-1e39))
    assert kp.device_status() == kp.ATTN_OK


def test_every_code_and_scale_reads_back(kp):
    """All 256 codes under every scale that the writer makes."""
    codes = torch.arange(256, dtype=torch.uint8).view(1, 1, 1, 256).expand(31, 1, 8, 256).contiguous()
    scales = torch.arange(10, 10 + 31 * 8).clamp(max=247).to(torch.uint8).view(31, 1, 8)
    c = codes.cuda().view(torch.float8_e4m3fn)
    table = torch.arange(31, dtype=torch.int32).view(1, 31).cuda()
    k, _ = kp.attn_cache_read(c, c, table, torch.tensor([248], dtype=torch.int32).cuda(), k_scale=scales.cuda(), v_scale=scales.cuda())
    want = ref.dequantise(codes, scales).transpose(0, 1).reshape(1, 248, 256)
    got = k[0].cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    big = want.abs() > 3.3895e38               # 448 * 2^120 alone is above bf16's largest number
    assert (torch.isinf(got) == big).all() and torch.equal(got[~big & ~torch.isnan(want)], want[~big & ~torch.isnan(want)])


def test_slots_and_pages_out_of_range(kp):
    P, H, page, D = 4, 2, 8, 64
    for e4m3 in (False, True):
        caches, scales = _pool(P, H, page, D, e4m3)
        dc, ds = _dev(caches, scales)
        before = [_bytes(c).clone() for c in dc]
        k = torch.ones(3, H, D, dtype=torch.bfloat16, device="cuda")
        slots = torch.tensor([P * page, 2 ** 31 - 1, -1], dtype=torch.int32, device="cuda")
        kp.attn_cache_write(k, k, slots, dc[0], dc[1], **ds)
        assert kp.device_status() == kp.ATTN_ERR_CACHE_RANGE and kp.device_status() == kp.ATTN_OK
        assert all(torch.equal(_bytes(c), b) for c, b in zip(dc, before))
        table = torch.tensor([[1, P, -5, 2]], dtype=torch.int32, device="cuda")
        got, _ = kp.attn_cache_read(dc[0], dc[1], table, torch.tensor([4 * page], dtype=torch.int32, device="cuda"), **ds)
        assert kp.device_status() == kp.ATTN_ERR_CACHE_RANGE
        vals = ref.dequantise(caches[0], scales[0]) if e4m3 else caches[0].double()
        assert torch.equal(got[0].cpu().double(), ref.gather(vals, table[0].cpu(), 4 * page))
        for n in (-1, 4 * page + 1):
            kp.attn_cache_read(dc[0], dc[1], table[:, :1].expand(1, 4).contiguous(), torch.tensor([n], dtype=torch.int32, device="cuda"), **ds)
            assert kp.device_status() == kp.ATTN_ERR_KVLEN_RANGE


def test_long_pool(kp):
    """Element offsets past 32 bits: a pool of 5.4 GB, rows written near its end."""
    P, H, page, D = 20600, 1, 1024, 128
    c = torch.zeros(P, H, page, D, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(3)
    k = torch.randn(5, H, D, generator=g).to(torch.bfloat16)
    slots = torch.tensor([0, 16777216, 16777217, P * page - 1, P * page - 2], dtype=torch.int32)
    assert int(slots.max()) * D * 2 > 2 ** 32
    kp.attn_cache_write(k.cuda(), k.cuda(), slots.cuda(), c, c)
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(c[s // page, :, s % page].cpu(), k[t])
    table = torch.tensor([[P - 1, 16777216 // page]], dtype=torch.int32).cuda()
    out, _ = kp.attn_cache_read(c, c, table, torch.tensor([2 * page], dtype=torch.int32).cuda())
    assert torch.equal(out[0, :, page - 1].cpu(), k[3]) and torch.equal(out[0, :, page].cpu(), k[1])


def test_read_feeds_the_prefix_kernel(kp):
    """Pages -> prefix -> attn_prefix_fwd, rows behind kv_len NaN, against the 64-bit attention over the pages."""
    g = torch.Generator().manual_seed(9)
    P, H, page, D, lens = 12, 2, 16, 64, [70, 3]
    caches, scales = _pool(P, H, page, D, True)
    dc, ds = _dev(caches, scales)
    table = torch.randperm(P, generator=g)[:10].view(2, 5).to(torch.int32)
    q = torch.randn(2, H, 7, D, generator=g).to(torch.bfloat16) * 0.01
    outs = [torch.full((2, H, 128, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kv = torch.tensor(lens, dtype=torch.int32).cuda()
    k, v = kp.attn_cache_read(dc[0], dc[1], table.cuda(), kv, k_out=outs[0], v_out=outs[1], **ds)
    out, lse = kp.attn_prefix_fwd(q.cuda(), k, v, kv)
    vals = [ref.dequantise(c, s) for c, s in zip(caches, scales)]
    r = ref.paged(q.transpose(1, 2).reshape(14, H, D), vals[0], vals[1], table, lens, [0, 7, 14], False, D ** -0.5)
    ref.assert_paged_close(out.transpose(1, 2).reshape(14, H, D), lse.transpose(1, 2).reshape(14, H), r)


def test_in_a_graph_and_on_a_stream(kp):
    P, H, page, D = 6, 2, 16, 128
    caches, scales = _pool(P, H, page, D, True)
    dc, ds = _dev(caches, scales)
    g = torch.Generator().manual_seed(4)
    k = torch.randn(9, H, D, generator=g).to(torch.bfloat16).cuda()
    slots = torch.arange(20, 29, dtype=torch.int32).cuda()
    table, kv = torch.tensor([[1, 0]], dtype=torch.int32).cuda(), torch.tensor([30], dtype=torch.int32).cuda()
    outs = [torch.zeros(1, H, 32, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kp.attn_cache_write(k, k, slots, dc[0], dc[1], **ds)
        kp.attn_cache_read(dc[0], dc[1], table, kv, k_out=outs[0], v_out=outs[1], **ds)
    k.mul_(-2)
    graph.replay()
    torch.cuda.synchronize()
    got = outs[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kp.attn_cache_write(k, k, slots, dc[0], dc[1], **ds)
        again, _ = kp.attn_cache_read(dc[0], dc[1], table, kv, **ds)
    s.synchronize()
    assert torch.equal(got[:, :, :30], again[:, :, :30])
    assert torch.equal(got[0, :, 4:13].cpu().double(), ref.dequantise(*ref.quantise(k.cpu())).transpose(0, 1))


def test_refusals(kp):
    c = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    e = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.zeros(4, 2, 16, dtype=torch.uint8, device="cuda")
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    kp.attn_cache_write(k[:0], k[:0], slots[:0], c, c)                  # nothing to write
    for bad in (dict(k=k.float()), dict(v=k[:2]), dict(slots=slots.long()), dict(slots=slots[:2]), dict(k=k[:, :1], v=k[:, :1]),
                dict(k_cache=c.half()), dict(k_cache=c[:3]), dict(k_cache=e, v_cache=e), dict(k_cache=e, v_cache=e, k_scale=s, v_scale=s[:3]),
                dict(k_scale=s, v_scale=s), dict(k_cache=c[:1].expand(4, 2, 16, 64)), dict(v_cache=e)):
        args = dict(k=k, v=k, slots=slots, k_cache=c, v_cache=c)
        args.update(bad)
        with pytest.raises(ValueError):
            kp.attn_cache_write(**args)
    table, kv = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    o = torch.zeros(2, 2, 40, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(block_table=table.long()), dict(block_table=table.t()), dict(kv_len=kv[:1]), dict(k_out=o), dict(k_out=o, v_out=o[:1]),
                dict(k_out=o, v_out=o.float()), dict(Tk=41, k_out=o, v_out=o), dict(k_out=o[:, :1].expand(2, 2, 40, 64), v_out=o)):
        args = dict(k_cache=c, v_cache=c, block_table=table, kv_len=kv)
        args.update(bad)
        with pytest.raises(ValueError):
            kp.attn_cache_read(**args)
    odd = torch.zeros(4, 2, 12, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(kp.AttnError):
        kp.attn_cache_write(k, k, slots, odd, odd)                     # page_size not a multiple of 8
    assert kp.device_status() == kp.ATTN_OK
