"""attn_paged_fwd against a 64-bit implementation over the same pages (tolerances: paged_reference)."""
import math
import random

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


def make(kv, n_q, Hq, Hkv, D, page, e4m3, seed=0, std=1.0, slack=0, layout="head", spread=0):
    """A batch on the CPU: pages whose slots behind each sequence are NaN, and unused table entries that
    name no page.  slack: rows of q in front of the first and behind the last sequence."""
    g = torch.Generator().manual_seed(seed)
    rnd = random.Random(seed)
    need = [-(-n // page) for n in kv]
    P = sum(need) + 2
    order = list(range(P))
    rnd.shuffle(order)
    table = torch.full((len(kv), max(max(need), 1) + 1), -1, dtype=torch.int32)
    owned = torch.zeros(P, page, dtype=torch.bool)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
        for j in range(m):
            owned[order[at + j], :min(page, kv[b] - j * page)] = True
        at += m
    c = dict(kv=kv, causal=True, scale=D ** -0.5, table=table, Hq=Hq, Hkv=Hkv, D=D)
    for name in ("k", "v"):
        x = (torch.randn(P, Hkv, page, D, generator=g) * std).to(torch.bfloat16)
        if spread:
            x = (x.float() * 2.0 ** torch.randint(-spread, spread + 1, (P, Hkv, page, 1), generator=g)).to(torch.bfloat16)
        if e4m3:
            codes = x.float()
            m, e = torch.frexp(codes.abs().amax(-1))
            e = e - 9 + (m > 0.875).int()
            s = (e + 127).to(torch.uint8)
            codes = (codes * 2.0 ** (-e[..., None])).to(torch.float8_e4m3fn).view(torch.uint8)
            codes[~owned[:, None, :].expand(P, Hkv, page)] = 0x7F
            s[~owned[:, None, :].expand(P, Hkv, page)] = 255
            c[name + "s"], c[name + "vals"] = s, torch.nan_to_num(ref.dequantise(codes, s))
            c[name] = codes
        else:
            x[~owned[:, None, :].expand(P, Hkv, page)] = math.nan
            c[name + "s"], c[name + "vals"], c[name] = None, torch.nan_to_num(x.double()), x
        if layout == "slot":
            c[name] = c[name].transpose(1, 2).contiguous().transpose(1, 2)
    start = [slack]
    for n in n_q:
        start.append(start[-1] + n)
    c["start"] = start
    c["q"] = (torch.randn(start[-1] + slack, Hq, D, generator=g) * std).to(torch.bfloat16)
    return c


def call(kp, c, **kw):
    dc = [c[n].cuda() for n in ("k", "v")]
    ds = {}
    if c["ks"] is not None:
        dc = [x.view(torch.float8_e4m3fn) for x in dc]
        ds = dict(k_scale=c["ks"].cuda(), v_scale=c["vs"].cuda())
    T, Hq, D = c["q"].shape
    out = torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 5.0, device="cuda")
    args = dict(q_start=torch.tensor(c["start"], dtype=torch.int32).cuda(), max_q=max(b - a for a, b in zip(c["start"], c["start"][1:])),
                causal=c["causal"], scale=c["scale"], out=out, lse=lse)
    args.update(kw)
    args["max_q"] = max(args["max_q"] or 1, 1)
    return kp.attn_paged_fwd(c["q"].cuda(), dc[0], dc[1], c["table"].cuda(), torch.tensor(c["kv"], dtype=torch.int32).cuda(), **ds, **args)


def check(kp, c, **kw):
    out, lse = call(kp, c, **kw)
    assert kp.device_status() == kp.ATTN_OK
    r = ref.paged(c["q"], c["kvals"], c["vvals"], c["table"], c["kv"], c["start"], c["causal"], c["scale"])
    ref.assert_paged_close(out, lse, r)
    outside = torch.isnan(r[1])                    # rows of no sequence stay as they were
    assert (out.cpu()[outside] == 3.0).all() and (lse.cpu()[outside] == 5.0).all()
    return out, lse


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,page", [(4, 4, 16), (8, 2, 8), (6, 2, 24), (16, 1, 64), (5, 1, 256), (32, 1, 16)])
def test_single_tokens(kp, D, Hq, Hkv, page, e4m3):
    kv = [1, 0, 15, 16, 17, 64, 127, 128, 129, 700]
    c = make(kv, [1] * len(kv), Hq, Hkv, D, page, e4m3, seed=D + Hq)
    check(kp, c)
    assert torch.equal(call(kp, c)[0], call(kp, c, q_start=None, max_q=None)[0])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,page", [(2, 2, 16), (6, 2, 32), (5, 1, 8), (8, 1, 128)])
def test_chunks(kp, D, Hq, Hkv, page, causal, e4m3):
    """Chunks of 0 to 300 rows; sequences shorter than their chunk (rows without keys), and empty ones."""
    kv = [300, 0, 129, 128, 40, 1, 515, 90]
    n_q = [300, 3, 1, 128, 60, 2, 77, 0]
    c = make(kv, n_q, Hq, Hkv, D, page, e4m3, seed=D + Hq + page, slack=3)
    c["causal"] = causal
    check(kp, c)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n_q", [1, 4, 9, 150])
@pytest.mark.parametrize("kv", [[30000], [1], [0], [64, 20000, 0, 65], [1500, 130, 0, 1] * 40])
def test_sequences_shared_by_many_blocks(kp, kv, n_q, e4m3):
    """One long sequence over all of the GPU, a few of very different lengths, and more sequences than blocks."""
    check(kp, make(kv, [n_q] * len(kv), 4, 2, 64, 16, e4m3, seed=len(kv)))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 7, 64, 128])
def test_head_groups(kp, G, D):
    for n_q in (1, 2, 5, 40):
        c = make([333, 50], [n_q, min(n_q, 3)], G, 1, D, 16, False, seed=G + n_q)
        check(kp, c)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n_q", [1, 33, 200])
def test_layouts(kp, n_q, e4m3):
    """Pages with heads innermost ([P, page, H, D] memory), q out of a packed projection, out in another layout."""
    c = make([400, 7, 250], [n_q, 2, 1], 6, 2, 64, 16, e4m3, seed=n_q, layout="slot")
    want, wl = check(kp, c)
    T, Hq, D = c["q"].shape
    packed = torch.zeros(T, Hq + 4, D, dtype=torch.bfloat16)
    packed[:, 2:2 + Hq] = c["q"]
    d = dict(c)
    d["q"] = packed.cuda()[:, 2:2 + Hq]
    out = torch.zeros(Hq, T, D, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    lse = torch.zeros(T, Hq, device="cuda")
    got, gl = call(kp, d, out=out, lse=lse)
    live = slice(c["start"][0], c["start"][-1])
    assert torch.equal(got[live], want[live]) and torch.equal(gl[live], wl[live])


@pytest.mark.parametrize("n_q", [1, 100])
def test_scales_and_spread(kp, n_q):
    """Zero and negative scales; rows whose magnitudes differ by 2^16; an e4m3 cache with scales beyond 2^7."""
    for scale in (0.0, -0.3, 2.0):
        c = make([200, 65], [n_q, 1], 4, 2, 64, 16, False, seed=4)
        c["scale"] = scale
        check(kp, c)
    c = make([300], [n_q], 4, 2, 64, 16, True, seed=5, spread=8)
    c["scale"] = 1e-3
    check(kp, c)
    c = make([300], [n_q], 4, 2, 64, 16, True, seed=6, std=1e6)
    c["q"] = (c["q"].float() * 1e-6).to(torch.bfloat16)
    c["scale"] = 1e-6
    check(kp, c)


@pytest.mark.parametrize("n_q", [1, 100])
@pytest.mark.parametrize("up", [10, 20])
def test_large_values_with_small_weights(kp, n_q, up):
    """Blocks of keys whose values are 2^up times the others' and whose weights are 2^-up: both count alike."""
    c = make([3 * 256], [n_q], 2, 1, 64, 16, True, seed=12)
    c["causal"] = False
    c["q"] = torch.zeros_like(c["q"])
    c["q"][..., 0] = 1.0
    c["scale"] = math.log(2.0)                       # scores in powers of two: the key's first element
    for j in range(3 * 256):
        row = (int(c["table"][0, j // 16]), 0, j % 16)
        big = j // 256 == 1
        key = torch.zeros(1, 64, dtype=torch.bfloat16)
        key[0, 0] = -up if big else 0.0
        val = (c["vvals"][row].float() * (2.0 ** up if big else 1.0)).to(torch.bfloat16)[None]
        for n, x in (("k", key), ("v", val)):
            codes, s = ref.quantise(x)
            c[n][row], c[n + "s"][row], c[n + "vals"][row] = codes[0], s[0], ref.dequantise(codes, s)[0]
    check(kp, c)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n_q", [1, 60])
@pytest.mark.parametrize("D", [64, 256])
def test_nan_rows_reach_their_sequence_only(kp, D, n_q, e4m3):
    c = make([100, 130, 70], [n_q] * 3, 4, 2, D, 16, e4m3, seed=14)
    clean, _ = check(kp, c)
    for n in ("k", "v"):
        d = dict(c)
        d[n] = c[n].clone()
        at = (int(c["table"][1, 2]), 1, 5)                  # key 37 of sequence 1, key head 1
        if e4m3:
            d[n + "s"] = c[n + "s"].clone()
            d[n][at], d[n + "s"][at] = 0x7F, 255
        else:
            d[n][at] = math.nan
        out, lse = call(kp, d)
        assert torch.equal(out[:n_q], clean[:n_q]) and torch.equal(out[2 * n_q:], clean[2 * n_q:])
        assert torch.equal(out[n_q:2 * n_q, :2], clean[n_q:2 * n_q, :2])            # the other key head
        assert torch.isnan(out[n_q:2 * n_q, 2:]).all()
        assert torch.isnan(lse[n_q:2 * n_q, 2:]).all() == (n == "k")
    assert kp.device_status() == kp.ATTN_OK


@pytest.mark.parametrize("n_q", [1, 17])
def test_thousands_of_sequences(kp, n_q):
    rnd = random.Random(15)
    kv = [rnd.choice((0, 1, 7, 18, 40)) for _ in range(4200)]
    rows = [rnd.choice((0, n_q, n_q, n_q + 2)) if n_q > 1 else rnd.choice((0, 1)) for _ in kv]
    check(kp, make(kv, rows, 2, 1, 32, 8, n_q > 1, seed=16), max_q=max(rows))


def test_pages_shared_by_sequences(kp):
    for n_q in (1, 50):
        c = make([150, 150, 90], [n_q] * 3, 4, 2, 128, 16, False, seed=17)
        c["table"][1:] = c["table"][0]
        check(kp, c)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n_q", [1, 60])
@pytest.mark.parametrize("D", [64, 256])
def test_far_pages(kp, D, n_q, e4m3):
    """Pages 2^32 bytes apart: offsets beyond 32 bits."""
    c = make([40, 30], [n_q] * 2, 4, 2, D, 32, e4m3, seed=18)
    want, want_lse = check(kp, c)
    P, H, page, _ = c["k"].shape
    size = 1 if e4m3 else 2
    pool = torch.empty((P - 1) * 2 ** 32 // size + 2 * H * page * D, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda")
    k, v = (pool.as_strided((P, H, page, D), (2 ** 32 // size, page * D, D, 1), i * H * page * D) for i in range(2))
    k.copy_(c["k"])
    v.copy_(c["v"])
    d = {}
    if e4m3:
        k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
        d = dict(k_scale=c["ks"].cuda(), v_scale=c["vs"].cuda())
    out, lse = kp.attn_paged_fwd(c["q"].cuda(), k, v, c["table"].cuda(), torch.tensor(c["kv"], dtype=torch.int32).cuda(),
                                 torch.tensor(c["start"], dtype=torch.int32).cuda(), n_q, scale=c["scale"], **d)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert kp.device_status() == kp.ATTN_OK


def test_a_waiting_row_tile_is_no_timeout(kp):
    """17 rows leave a block's second row tile without work for milliseconds; the limit is on steps."""
    H, page, n = 148, 4096, 128
    k = torch.zeros(1, H, page, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(17, H, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(1, n, dtype=torch.int32, device="cuda")
    kv = torch.tensor([n * page], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 17], dtype=torch.int32, device="cuda")
    kp.set_wait_limit_ns(1_000_000)
    try:
        out, lse = kp.attn_paged_fwd(q, k, k, table, kv, start, 17, causal=False)
        assert kp.device_status() == kp.ATTN_OK
    finally:
        kp.set_wait_limit_ns(1_000_000_000)
    assert (out == 0).all() and (lse - math.log(n * page)).abs().max() < 1e-3


def test_work_beyond_the_counters_is_refused(kp):
    """32 sequences of 2^30 keys (one page again and again) over 32 key heads: 2^33 tiles."""
    k = torch.zeros(1, 32, 2 ** 16, 32, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(32 * 17, 32, 32, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(32, 2 ** 14, dtype=torch.int32, device="cuda")
    kv = torch.full((32,), 2 ** 30, dtype=torch.int32, device="cuda")
    start = torch.arange(0, 32 * 17 + 1, 17, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 3.0)
    kp.attn_paged_fwd(q, k, k, table, kv, start, 17, out=out)
    assert kp.device_status() == kp.ATTN_ERR_CACHE_RANGE
    assert (out == 3.0).all()


@pytest.mark.parametrize("n_q", [1, 150])
@pytest.mark.parametrize("D", [32, 128, 256])
def test_rows_of_far_scales(kp, D, n_q):
    """Scales from 2^-40 to 2^30 in one sequence, beyond what one bf16 factor reaches, and a page of ordinary ones."""
    c = make([250, 131], [n_q, n_q], 4, 2, D, 16, True, seed=19, spread=35)
    c["q"] = (c["q"].float() * 2.0 ** -35).to(torch.bfloat16)
    check(kp, c)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n_q", [1, 140])
def test_rising_scores(kp, n_q, e4m3):
    """Scores that grow along the keys, so that the running maximum moves in every tile."""
    c = make([900], [n_q], 2, 1, 64, 16, e4m3, seed=8)
    ramp = torch.ones(64, dtype=torch.float64)
    for j in range(900):
        row = (int(c["table"][0, j // 16]), 0, j % 16)
        val = torch.tensor(j / 900 * 3.0, dtype=torch.bfloat16)
        if e4m3:
            codes, s = ref.quantise(val.expand(1, 64))
            c["k"][row], c["ks"][row] = codes[0], s[0]
            c["kvals"][row] = ref.dequantise(codes, s)[0]
        else:
            c["k"][row], c["kvals"][row] = val * ramp, val.double() * ramp
    c["q"] = torch.ones_like(c["q"])
    c["scale"] = 1.0
    check(kp, c)


def test_ranges_are_clamped_and_flagged(kp):
    c = make([100, 60], [5, 4], 4, 2, 64, 16, False, seed=11)
    d = dict(c)
    d["kv"] = [100, 60]
    bad_table = c["table"].clone()
    bad_table[0, 1] = 10 ** 6
    d["table"] = bad_table
    out, lse = call(kp, d)
    assert kp.device_status() == kp.ATTN_ERR_CACHE_RANGE       # that page's keys and values count as zeros
    r = ref.paged(c["q"], c["kvals"], c["vvals"], bad_table, c["kv"], c["start"], True, c["scale"])
    ref.assert_paged_close(out, lse, r)
    for kv in (-3, 16 * c["table"].shape[1] + 1):
        d = dict(c)
        d["kv"] = [kv, 60]
        d["table"] = c["table"].clamp_min(0)
        call(kp, d)
        assert kp.device_status() == kp.ATTN_ERR_KVLEN_RANGE
    for start in ([0, 9, 5], [-1, 5, 9], [0, 5, 99]):
        d = dict(c)
        call(kp, d, q_start=torch.tensor(start, dtype=torch.int32).cuda(), max_q=9)
        assert kp.device_status() == kp.ATTN_ERR_CACHE_RANGE
    out, lse = call(kp, c, max_q=3)                             # rows beyond max_q are not computed
    assert kp.device_status() == kp.ATTN_ERR_CACHE_RANGE
    full, _ = call(kp, c)
    assert torch.equal(out[:3], full[:3]) and (out[3:5] == 3.0).all() and torch.equal(out[5:8], full[5:8])
    assert kp.device_status() == kp.ATTN_OK


@pytest.mark.parametrize("n_q", [1, 130])
def test_repeats_graphs_and_streams_agree(kp, n_q):
    c = make([2000, 31, 0, 700], [n_q, 1, 1, n_q], 8, 2, 128, 16, True, seed=12)
    want, wl = call(kp, c)
    for _ in range(2):
        a, al = call(kp, c)
        assert torch.equal(a, want) and torch.equal(al, wl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a, al = call(kp, c)
    s.synchronize()
    assert torch.equal(a, want) and torch.equal(al, wl)
    dev = dict(q=c["q"].cuda(), k=c["k"].cuda().view(torch.float8_e4m3fn), v=c["v"].cuda().view(torch.float8_e4m3fn), ks=c["ks"].cuda(),
               vs=c["vs"].cuda(), table=c["table"].cuda(), kv=torch.tensor(c["kv"], dtype=torch.int32).cuda(),
               start=torch.tensor(c["start"], dtype=torch.int32).cuda())
    outs = [torch.zeros_like(want) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            kp.attn_paged_fwd(dev["q"], dev["k"], dev["v"], dev["table"], dev["kv"], dev["start"], n_q, scale=c["scale"],
                              k_scale=dev["ks"], v_scale=dev["vs"], out=o)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    live = slice(0, c["start"][-1])
    assert all(torch.equal(o[live], want[live]) for o in outs)
    dev["kv"].copy_(torch.tensor([1000, 31, 5, 700], dtype=torch.int32))
    d = dict(c)
    d["kv"] = [1000, 31, 5, 700]
    d["table"] = c["table"].clone()
    d["table"][2, 0] = d["table"][0, -2]
    dev["table"].copy_(d["table"])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][live], call(kp, d)[0][live])
    assert kp.device_status() == kp.ATTN_OK


def test_a_whole_serving_step(kp):
    """PagedCache.step over prompt chunks and single tokens, against the 64-bit chain."""
    g = torch.Generator().manual_seed(20)
    Hq, Hkv, D, page = 4, 2, 64, 16
    for quantised in (False, True):
        cache = kp.PagedCache(20, page, Hkv, D, quantised=quantised)
        table = torch.randperm(20, generator=g)[:18].view(2, 9).to(torch.int32)
        inv, f = kp.rope_inv_freq(D, scaling="yarn", factor=4.0, original_context=64)
        wq, wk = (torch.randn(D, generator=g).to(torch.bfloat16) + 1 for _ in range(2))
        have = [0, 0]
        kvals = torch.zeros(20, Hkv, page, D, dtype=torch.float64)
        vvals = kvals.clone()
        for n_q in ([40, 17], [1, 1], [5, 60], [1, 1]):
            start = [0, n_q[0], sum(n_q)]
            q, k, v = (torch.randn(sum(n_q), h, D, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
            pos = torch.tensor([have[b] + i for b in range(2) for i in range(n_q[b])], dtype=torch.int32)
            seq = [b for b in range(2) for _ in range(n_q[b])]
            slots = torch.tensor([int(table[b, p // page]) * page + p % page for b, p in zip(seq, pos.tolist())], dtype=torch.int32)
            have = [have[b] + n_q[b] for b in range(2)]
            out, lse = cache.step(q.cuda(), k.cuda(), v.cuda(), pos.cuda(), slots.cuda(), table.cuda(),
                                  torch.tensor(have, dtype=torch.int32).cuda(), torch.tensor(start, dtype=torch.int32).cuda(),
                                  max(n_q), inv_freq=inv, rope=dict(q_weight=wq.cuda(), k_weight=wk.cuda(), attn_factor=f))
            # the rotated rows as the kernel rounds them (compared with 64 bits in test_gpu_rope)
            qr, kr = kp.attn_qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), inv, q_weight=wq.cuda(), k_weight=wk.cuda(), attn_factor=f)
            for x, vals in ((kr.cpu(), kvals), (v, vvals)):
                rows = ref.dequantise(*ref.quantise(x)) if quantised else x.double()
                for t, s in enumerate(slots.tolist()):
                    vals[s // page, :, s % page] = rows[t]
            r = ref.paged(qr.cpu(), kvals, vvals, table, have, start, True, D ** -0.5)
            ref.assert_paged_close(out, lse, r)
            kb, vb = cache.read(table.cuda(), torch.tensor(have, dtype=torch.int32).cuda())
            for b in range(2):
                assert torch.equal(kb[b, :, :have[b]].cpu().double(), ref.gather(kvals, table[b], have[b]))
                assert torch.equal(vb[b, :, :have[b]].cpu().double(), ref.gather(vvals, table[b], have[b]))
    assert kp.device_status() == kp.ATTN_OK


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_dropped_copy_times_out_and_context_survives(kp, D, e4m3):
    """A K tile that is announced and never delivered: the bounded waits end the kernel with its flag."""
    c = make([500], [200], 4, 2, D, 16, e4m3, seed=D)
    kp.set_wait_limit_ns(20_000_000)
    kp.set_debug_flags(kp.ATTN_DEBUG_DROP_COPY)
    try:
        call(kp, c)
        assert kp.device_status() == kp.ATTN_ERR_TIMEOUT
    finally:
        kp.set_debug_flags(0)
        kp.set_wait_limit_ns(1_000_000_000)
    check(kp, c)


def test_refusals(kp):
    c = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16, device="cuda")
    table, kv = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    ok = dict(q=q, k_cache=c, v_cache=c, block_table=table, kv_len=kv, q_start=start, max_q=3)
    kp.attn_paged_fwd(**ok)
    for bad in (dict(q=q.float()), dict(q=q[..., :32]), dict(q=q[:, :3]), dict(q_start=None), dict(q_start=start[:2]),
                dict(q_start=start.long()), dict(kv_len=kv.long()), dict(block_table=table[:1]), dict(out=q[:4]),
                dict(out=q.float()), dict(lse=torch.zeros(4, 4, device="cuda")), dict(q=q[:1].expand(5, 4, 64)),
                dict(out=torch.zeros(5, 1, 64, dtype=torch.bfloat16, device="cuda").expand(5, 4, 64))):
        with pytest.raises(ValueError):
            kp.attn_paged_fwd(**{**ok, **bad})
    for bad in (dict(max_q=0), dict(scale=math.inf)):
        with pytest.raises(kp.AttnError):
            kp.attn_paged_fwd(**{**ok, **bad})
    out, _ = kp.attn_paged_fwd(q[:0], c, c, table, kv, torch.zeros(3, dtype=torch.int32, device="cuda"))   # no rows
    assert out.shape == (0, 4, 64)
    assert kp.device_status() == kp.ATTN_OK


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_late_softmax_warps(kp, D, e4m3):
    """Warps that come to the end of a run's tiles long after the last product is complete: one, two and
    more tiles to a segment, several segments to a block, and the same bits as without the pause."""
    for kv, n_q in (([100], [40]), ([200], [200]), ([700, 130, 385], [300, 1, 140]), ([129, 500, 0, 260] * 30, [30, 77, 5, 1] * 30)):
        c = make(kv, n_q, 4, 1, D, 16, e4m3, seed=D + len(kv))
        want, want_lse = check(kp, c)
        kp.set_wait_limit_ns(20_000_000)
        kp.set_debug_flags(kp.ATTN_DEBUG_LATE_SOFTMAX)
        try:
            out, lse = call(kp, c)
            assert kp.device_status() == kp.ATTN_OK
        finally:
            kp.set_debug_flags(0)
            kp.set_wait_limit_ns(1_000_000_000)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("spread", [0, 8])
@pytest.mark.parametrize("n_q", [1, 60])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_nan_codes_under_ordinary_scales(kp, D, n_q, spread):
    """A single code of NaN (0x7F, 0xFF) in a row whose scale is an ordinary one, as another quantiser stores it:
    NaN for the rows and dims that the formula has it in, and nothing else changes.  spread: scales too far apart
    for f16 weights.  Keys in whole tiles and in a sequence's last one."""
    c = make([100, 300, 70], [n_q] * 3, 4, 2, D, 16, True, seed=21, spread=spread)
    c["causal"] = False
    if spread:
        c["q"] = (c["q"].float() * 2.0 ** -8).to(torch.bfloat16)
    clean, clean_lse = call(kp, c)
    assert kp.device_status() == kp.ATTN_OK and not torch.isnan(clean).any()
    rows = slice(n_q, 2 * n_q)                                  # of sequence 1
    for key, d, code in ((37, 0, 0x7F), (200, 5, 0xFF), (299, D - 1, 0x7F), (288, D // 2 + 2, 0xFF), (140, D - 16, 0x7F)):
        for n in ("k", "v"):
            m = dict(c)
            m[n] = c[n].clone()
            m[n][int(c["table"][1, key // 16]), 1, key % 16, d] = code
            out, lse = call(kp, m)
            want, want_lse = clean.clone(), clean_lse.clone()
            if n == "k":
                want[rows, 2:], want_lse[rows, 2:] = math.nan, math.nan
            else:
                want[rows, 2:, d] = math.nan
            bits = (x.view(torch.int16) for x in (out.nan_to_num(7.0), want.nan_to_num(7.0)))
            assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(*bits), (key, n)
            assert torch.equal(torch.isnan(lse), torch.isnan(want_lse)) and torch.equal(lse.nan_to_num(7.0), want_lse.nan_to_num(7.0))
            read = dict(k=0, v=1)[n]
            got = kp.attn_cache_read(*(m[x].cuda().view(torch.float8_e4m3fn) for x in ("k", "v")), m["table"][1:2].contiguous().cuda(),
                                     torch.tensor([300], dtype=torch.int32).cuda(), k_scale=m["ks"].cuda(), v_scale=m["vs"].cuda())[read]
            assert torch.isnan(got[0, 1, key, d]) and int(torch.isnan(got[0, :, :300]).sum()) == 1
    assert kp.device_status() == kp.ATTN_OK


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n_q", [1, 17])
@pytest.mark.parametrize("D", [32, 64, 256])
def test_longest_sequence(kp, D, n_q, e4m3):
    """2^31 - 13 keys: one page 16382 times, then one whose keys outweigh all of those and whose last five rows, behind the
    sequence, are NaN.  Tolerances as in paged_reference: the 2^31 weights of the first page sum to 2^-9 of
    the others' rounding at most, and the 131075 keys of the last one are added to 8192 at a time in fp32 (2^-11)."""
    page, n = 8 * 16385, 16383
    kv = page * n - 5
    assert kv == 2 ** 31 - 13
    g = torch.Generator().manual_seed(D + n_q)
    score = torch.randint(0, 4, (page,), generator=g) * 2.0 + 26.0         # every number here is one in e4m3, and in bf16
    val = torch.randint(-8, 9, (page, D), generator=g).double() / 4
    k = torch.zeros(2, 1, page, D)
    k[1, 0, :, 0] = score
    v = torch.ones(2, 1, page, D)
    v[1, 0] = val.float()
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kc, vc = k.cuda().to(dtype), v.cuda().to(dtype)
    ds = {}
    if e4m3:
        s = torch.full((2, 1, page), 127, dtype=torch.uint8)
        s[1, 0, -5:] = 255
        ds = dict(k_scale=s.cuda(), v_scale=s.cuda())
        for c in (kc, vc):
            c.view(torch.uint8)[1, 0, -5:] = 0x7F
    else:
        kc[1, 0, -5:] = vc[1, 0, -5:] = math.nan
    q = torch.zeros(n_q, 1, D, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    table = torch.zeros(1, n, dtype=torch.int32)
    table[0, -1] = 1
    out, lse = kp.attn_paged_fwd(q.cuda(), kc, vc, table.cuda(), torch.tensor([kv], dtype=torch.int32).cuda(),
                                 torch.tensor([0, n_q], dtype=torch.int32).cuda(), n_q, scale=1.0, **ds)
    assert kp.device_status() == kp.ATTN_OK
    w = (score - 32.0).double().exp()
    first = page * (n - 1) * math.exp(-32.0)
    r_out, mean, r_lse = torch.empty(n_q, 1, D, dtype=torch.float64), torch.empty(n_q, 1, D, dtype=torch.float64), torch.empty(n_q, 1, dtype=torch.float64)
    for i in range(n_q):
        m = page - 5 - (n_q - 1 - i)                                       # keys of the last page that row i sees
        total = w[:m].sum() + first
        r_out[i, 0], mean[i, 0] = (w[:m] @ val[:m] + first) / total, (w[:m] @ val[:m].abs() + first) / total
        r_lse[i, 0] = total.log() + 32.0
    err = torch.full((n_q, 1), (D + 4) * 2.0 ** -24 * 32.0, dtype=torch.float64)
    ref.assert_paged_close(out, lse, (r_out, r_lse, mean, err))


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("n_q,Hq,key", [(4, 4, 298), (300, 2, 290), (300, 4, 31)])
def test_nan_that_causal_hides(kp, D, n_q, Hq, key, e4m3):
    """A row of NaN that only later rows see.  In keys it does not matter to the others.  In values it reaches all who
    see it; the others, and only those of its sequence and key head, have their values or NaN, by the tiles."""
    c = make([90, 300, 70], [3, n_q, 2], Hq, 2, D, 16, e4m3, seed=22)
    clean, clean_lse = check(kp, c)
    rows = torch.arange(3, 3 + n_q)
    sees = rows - 3 + 300 - n_q >= key
    mine = torch.zeros(clean.shape[:2], dtype=torch.bool)                      # of key head 1 and this sequence
    mine[rows, Hq // 2:] = True
    seen = torch.zeros_like(mine)
    seen[rows[sees], Hq // 2:] = True
    assert seen.any() and (mine & ~seen).any()
    seen, mine = seen.cuda(), mine.cuda()
    at = (int(c["table"][1, key // 16]), 1, key % 16)
    for n in ("k", "v"):
        d = dict(c)
        d[n] = c[n].clone()
        if e4m3:
            d[n + "s"] = c[n + "s"].clone()
            d[n][at], d[n + "s"][at] = 0x7F, 255
        else:
            d[n][at] = math.nan
        out, lse = call(kp, d)
        assert torch.isnan(out[seen]).all()
        same = (out.view(torch.int16) == clean.view(torch.int16)).all(-1)
        hidden = mine & ~seen
        assert same[~mine].all() and (same | torch.isnan(out).all(-1))[hidden].all()
        assert torch.isnan(lse[seen]).all() if n == "k" else torch.equal(lse[seen], clean_lse[seen])
        assert torch.equal(lse[~seen], clean_lse[~seen])
        if n == "k":
            assert same[hidden].all()
    assert kp.device_status() == kp.ATTN_OK


def test_one_status_call_clears_the_flags_of_all_kernels(kp):
    """The prefix kernels' flag and the paged ones', raised together: the first call reports the one with priority,
    and none is left behind."""
    x = torch.zeros(1, 1, 64, 64, dtype=torch.bfloat16, device="cuda")
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    table = torch.full((1, 2), 9, dtype=torch.int32, device="cuda")
    for bad_kv in (True, False):
        if bad_kv:
            kp.attn_prefix_fwd(x, x, x, one * 65)
        kp.attn_paged_fwd(x[0, 0, :1, None], x, x, table, one)
        assert kp.device_status() == (kp.ATTN_ERR_KVLEN_RANGE if bad_kv else kp.ATTN_ERR_CACHE_RANGE)
        assert kp.device_status() == kp.ATTN_OK


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("G", [5, 33, 100])
def test_rows_beside_a_sequences_own_change_nothing(kp, G, D, e4m3):
    """Rows of a tile that are not the sequence's: the next sequence's queries, and (head counts that do not divide
    128) what an earlier launch left in shared memory.  Bit for bit the same whatever they are."""
    c = make([700, 600], [20, 300 // G], G, 1, D, 16, e4m3, seed=G)
    big, fill = dict(c), make([300], [256], 1, 1, D, 16, e4m3, seed=1)
    big["q"] = c["q"].clone()
    big["q"][20:] *= 64.0
    want = None
    for size, case in ((0.0, c), (64.0, c), (0.0, big), (64.0, big)):
        d = dict(fill)
        d["kv"], d["table"] = [300] * 148, fill["table"].expand(148, -1).contiguous()
        d["start"] = [256 * i for i in range(149)]
        d["q"] = fill["q"].repeat(148, 1, 1) * size
        call(kp, d)                                     # a block on every SM, all rows of its tiles
        out, lse = call(kp, case)
        got = out[:20].view(torch.int16).cpu(), lse[:20].cpu()
        want = want or got
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert kp.device_status() == kp.ATTN_OK


def test_threads_with_streams_of_their_own(kp):
    """Four threads, each writing, attending and reading over caches of its own on its own stream."""
    import threading
    results, errors = {}, []

    def work(i, key):
        try:
            g = torch.Generator(device="cuda").manual_seed(i)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                cache = kp.PagedCache(40, 16, 2, 64, quantised=i % 2 == 1)
                q = torch.randn(300, 6, 64, generator=g, device="cuda").to(torch.bfloat16)
                k, v = (torch.randn(300, 2, 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
                table = torch.randperm(40, generator=g, device="cuda").int()[:19].view(1, 19)
                j = torch.arange(300, device="cuda")
                slots = table[0][j // 16] * 16 + (j % 16).int()
                start = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
                inv, _ = kp.rope_inv_freq(64)
                kv = torch.tensor([300], dtype=torch.int32, device="cuda")
                for _ in range(20):
                    step = cache.step(q, k, v, j.int(), slots, table, kv, start, 300, inv_freq=inv)
                    one = cache.attend(q[:1], table, kv)
                read = cache.read(table, kv, 300)
            stream.synchronize()
            results[key] = [x.clone() for x in (*step, *one, *read)]
        except Exception as e:                          # noqa: BLE001  (reported by the test's thread)
            errors.append(e)

    for i in range(4):
        work(i, ("alone", i))
    threads = [threading.Thread(target=work, args=(i, ("together", i))) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in range(4):
        assert all(torch.equal(a, b) for a, b in zip(results["alone", i], results["together", i]))
    assert kp.device_status() == kp.ATTN_OK
