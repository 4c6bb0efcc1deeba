"""The paged-cache operators' measured cases, and what each of them computes in plain torch.

Three operators that one serving step calls in this order, on the keys and queries that
the prefix-masked attention of this library works on:

  rope    attn_qk_norm_rope: per-head RMS norm of q and k and the rotation by position.
  cache   attn_cache_write + attn_cache_read: new key and value rows stored in the pages
          of a cache, in bf16 or in e4m3 with one power-of-two scale a row, and the
          sequences read back from their pages as contiguous prefixes.
  paged   attn_paged_fwd: attention of each sequence's new tokens over its pages.

``run`` computes an operator in elementary torch operations where ``own`` is false and
calls the library where it is true.  ``exact`` is the same from the definition, in 64 bits.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
SCALE_MIN, SCALE_MAX = -117, 120     # exponents of the row scales


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step's rows: 8 requests, a token each; latency counts
        dict(name="rope_step", op="rope", T=8, Hq=32, Hkv=8, D=128, R=128, interleaved=False, norm=True,
             max_pos=4096, scaled=False),
        # 8 views of 973 tokens, 12 heads of 64 (the unmasked workload's small shape)
        dict(name="rope_views", op="rope", T=7784, Hq=12, Hkv=12, D=64, R=64, interleaved=True, norm=True,
             max_pos=7784, scaled=False),
        # a long prompt's rows at far positions: half of each head rotated, scaled frequencies
        dict(name="rope_prompt", op="rope", T=65536, Hq=32, Hkv=8, D=128, R=64, interleaved=False, norm=True,
             max_pos=1000000, scaled=True),
        # a decoding step on a small quantised cache
        dict(name="cache_step", op="cache", B=16, new=1, kv_max=300, Hkv=8, D=128, page=16, e4m3=True),
        # the ragged workload's lengths (one of them empty), chunks of new rows, quantised
        dict(name="cache_ragged_e4m3", op="cache", B=8, new=512, kv_max=32768, Hkv=8, D=128, page=64, e4m3=True),
        # 100000 context rows of head dim 256 (the icl workload's keys), bf16 pages
        dict(name="cache_context_bf16", op="cache", B=1, new=8192, kv_max=100000, Hkv=8, D=256, page=128, e4m3=False),
        # one request decoding: latency counts
        dict(name="decode_one", op="paged", B=1, q_max=1, kv_max=1000, Hq=32, Hkv=8, D=128, page=16, e4m3=False,
             causal=True),
        # a serving batch decoding, ragged lengths up to the ragged workload's 32768
        dict(name="decode_ragged_bf16", op="paged", B=64, q_max=1, kv_max=32768, Hq=32, Hkv=8, D=128, page=16,
             e4m3=False, causal=True),
        # the same with a quantised cache, longer contexts and eight queries to a key head
        dict(name="decode_ragged_e4m3", op="paged", B=32, q_max=1, kv_max=65536, Hq=64, Hkv=8, D=128, page=64,
             e4m3=True, causal=True),
        # a mixed batch: chunks of 1 to 512 new tokens, 12 heads of 64 on 4 key heads
        dict(name="chunk_mixed_e4m3", op="paged", B=16, q_max=512, kv_max=8192, Hq=12, Hkv=4, D=64, page=32,
             e4m3=True, causal=True),
        # a chunk of a long prompt
        dict(name="chunk_long_bf16", op="paged", B=1, q_max=2048, kv_max=32768, Hq=32, Hkv=8, D=128, page=16,
             e4m3=False, causal=True),
        # new rows against 100000 context rows kept in pages, no causal mask (the icl workload's context)
        dict(name="context_rows_bf16", op="paged", B=1, q_max=2000, kv_max=100000, Hq=8, Hkv=8, D=256, page=128,
             e4m3=False, causal=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "cache", "paged", "paged"))
    D = rng.choice((32, 64, 128, 256))
    if op == "rope":
        Hkv, G = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 5, 8))
        T = _log_int(rng, 1, max(1, 65536 * 40 * 128 // (Hkv * (G + 1) * D * 2)))
        return dict(op="rope", T=T, Hq=Hkv * G, Hkv=Hkv, D=D, R=2 * rng.randint(1, D // 2),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.7, max_pos=_log_int(rng, 64, 1000000),
                    scaled=rng.random() < 0.5)
    Hkv = rng.choice((1, 2, 3, 4, 8))
    page = rng.choice((8, 16, 24, 32, 64, 128, 256))
    e4m3 = rng.random() < 0.5
    B = _log_int(rng, 1, 64)
    if op == "cache":
        kv = _log_int(rng, 2, max(2, 100000 * 8 * 256 // (Hkv * D * B)))
        return dict(op="cache", B=B, new=_log_int(rng, 1, max(1, kv // 2)), kv_max=kv, Hkv=Hkv, D=D, page=page,
                    e4m3=e4m3)
    G = rng.choice((1, 2, 3, 4, 5, 8, 16))
    kv = _log_int(rng, 2, max(2, 64 * 32768 * 8 * 128 // (2 * Hkv * D * B * (2 if B > 8 else 1))))
    kv = min(kv, 131072)
    q = 1 if rng.random() < 0.4 else _log_int(rng, 1, max(1, min(4096, 2000 * 100000 * 8 * 256 // (2 * B * kv * Hkv * G * D))))
    return dict(op="paged", B=B, q_max=q, kv_max=kv, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, e4m3=e4m3,
                causal=rng.random() < 0.7)


# ------------------------------------------------------------------------------ inputs
def _normal(gen, shape, std=1.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return x.mul_(std).to(torch.bfloat16)


def _lengths(case, rnd):
    """Key counts: the longest one is kv_max, the others uniform; in a batch of 4 or more the last one is 0."""
    B, m = case["B"], case["kv_max"]
    kv = [m] + [rnd.randint(1, m) for _ in range(B - 1)]
    if B >= 4:
        kv[-1] = 0
    return kv


def _pages(kv, page, rnd):
    """A pool a little larger than needed, and each sequence's pages in no order; -1 behind them."""
    need = [-(-n // page) for n in kv]
    num = sum(need) + 3
    order = list(range(num))
    rnd.shuffle(order)
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (max(max(need), 1) - n))
        at += n
    return num, torch.tensor(table, dtype=torch.int32)


def _inv_freq(R, scaled):
    """Frequencies of base 10000; scaled: the slow half divided by 8 (a context 8 times as long)."""
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    if scaled:
        f[R // 4:] /= 8.0
    return f.cuda()


def _cache(gen, case, num):
    """Key and value pages with content, in the case's format: (values or codes, scales)."""
    shape = (num, case["Hkv"], case["page"], case["D"])
    made = []
    for _ in range(2):
        x = _normal(gen, shape)
        made.append(_quantise(x) if case["e4m3"] else (x, None))
    return made


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = random.Random(seed)
    if case["op"] == "rope":
        T, D = case["T"], case["D"]
        # one packed projection [T, Hq + 2 Hkv, D], as a user's program has it: q and k are views of it
        qkv = _normal(gen, (T, case["Hq"] + 2 * case["Hkv"], D))
        pos = torch.randint(0, case["max_pos"], (T,), generator=gen, device="cuda", dtype=torch.int32)
        w = [_normal(gen, (D,), 0.2) + 1.0 for _ in range(2)] if case["norm"] else [None, None]
        return dict(case=case, q=qkv[:, :case["Hq"]], k=qkv[:, case["Hq"]:case["Hq"] + case["Hkv"]], pos=pos,
                    wq=w[0], wk=w[1], inv_freq=_inv_freq(case["R"], case["scaled"]),
                    factor=1.2 if case["scaled"] else 1.0)
    kv = _lengths(case, rnd)
    num, table = _pages(kv, case["page"], rnd)
    (kc, ks), (vc, vs) = _cache(gen, case, num)
    st = dict(case=case, kc=kc, ks=ks, vc=vc, vs=vs, table=table.cuda(),
              kv_len=torch.tensor(kv, dtype=torch.int32).cuda())
    if case["op"] == "cache":
        new = [min(case["new"], n) for n in kv]      # the last rows of each sequence are written now
        slots = [int(table[b][j // case["page"]]) * case["page"] + j % case["page"]
                 for b in range(case["B"]) for j in range(kv[b] - new[b], kv[b])]
        T = len(slots)
        shape = (case["B"], case["Hkv"], case["kv_max"], case["D"])
        st.update(k=_normal(gen, (T, case["Hkv"], case["D"])), v=_normal(gen, (T, case["Hkv"], case["D"])),
                  slots=torch.tensor(slots, dtype=torch.int32).cuda(),
                  k_out=torch.zeros(shape, dtype=torch.bfloat16, device="cuda"),
                  v_out=torch.zeros(shape, dtype=torch.bfloat16, device="cuda"))
        return st
    by_case = random.Random(case["B"] * 65537 + case["q_max"])      # as many query rows for every seed
    ql = [min(case["q_max"], kv[0])] + [by_case.randint(1, case["q_max"]) for _ in range(case["B"] - 1)]
    start = [0]
    for n in ql:
        start.append(start[-1] + n)
    st.update(q=_normal(gen, (start[-1], case["Hq"], case["D"])),
              q_start=torch.tensor(start, dtype=torch.int32).cuda(), q_max=case["q_max"], scale=case["D"] ** -0.5)
    return st


# ------------------------------------------------------------------------------ plain forms
def _rope_plain(x, w, pos, inv_freq, factor, interleaved):
    R = 2 * inv_freq.numel()
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
    ang = pos.double()[:, None, None] * inv_freq          # 64 bits: far positions
    c, s = (ang.cos() * factor).float(), (ang.sin() * factor).float()
    rot, rest = y[..., :R], y[..., R:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = rot[..., :R // 2], rot[..., R // 2:]
        rot = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((rot, rest), -1).to(torch.bfloat16)


def _quantise(x):
    """e4m3 codes of x / 2^e and e + 127, e the least exponent with amax / 2^e <= 448, for each row of x."""
    y = x.float()
    m, e = torch.frexp(y.abs().amax(-1))                  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m == 0, 0, e - 9 + (m > 0.875).int()).clamp(SCALE_MIN, SCALE_MAX)
    return torch.ldexp(y, -e[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _values(c, s):
    """The bf16 values that codes and scales stand for (exact), or the values themselves."""
    return c if s is None else torch.ldexp(c.float(), s.int()[..., None] - 127).to(torch.bfloat16)


def _gather(pages, scales, table, L):
    """The first L rows of every sequence from its pages: [B, Hkv, L, D] bf16."""
    t = table.clamp_min(0).long()
    x = pages.view(torch.uint8)[t].view(pages.dtype) if scales is not None else pages[t]
    x = _values(x, None if scales is None else scales[t])   # [B, pages, Hkv, page, D]
    B, n, H, p, D = x.shape
    return x.transpose(1, 2).reshape(B, H, n * p, D)[:, :, :L]


def _cache_plain(st):
    page, D = st["case"]["page"], st["case"]["D"]
    pg, row = (st["slots"] // page).long(), (st["slots"] % page).long()
    out = []
    for x, c, s, o in ((st["k"], st["kc"], st["ks"], st["k_out"]), (st["v"], st["vc"], st["vs"], st["v_out"])):
        if s is not None:
            codes, e = _quantise(x)
            c.view(torch.uint8)[pg, :, row] = codes.view(torch.uint8)
            s[pg, :, row] = e
        else:
            c[pg, :, row] = x
        L = o.shape[2]
        live = (torch.arange(L, device="cuda") < st["kv_len"][:, None])[:, None, :, None]
        out.append(torch.where(live, _gather(c, s, st["table"], L), o))
    return out


def _paged_plain(st):
    case = st["case"]
    L, G, Q = case["kv_max"], case["Hq"] // case["Hkv"], case["q_max"]
    k, v = (_gather(c, s, st["table"], L).float() for c, s in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
    j = torch.arange(L, device="cuda")
    kv, start = st["kv_len"].long(), st["q_start"].long()
    v = torch.where((j < kv[:, None])[:, None, :, None], v, 0.0)
    n_q = start[1:] - start[:-1]
    i = torch.arange(Q, device="cuda")
    live = i < n_q[:, None]                                                     # [B, Q]
    row = (start[:-1, None] + i).clamp_max(st["q"].shape[0] - 1)
    q = st["q"][row].float()                                                    # [B, Q, Hq, D]
    B, D = q.shape[0], q.shape[-1]
    q = q.view(B, Q, -1, G, D).permute(0, 2, 1, 3, 4).reshape(B, -1, Q * G, D)  # [B, Hkv, Q G, D]
    last = kv[:, None] - n_q[:, None] + i if case["causal"] else (kv[:, None] - 1).expand(B, Q)
    seen = (j <= last[..., None]) & (j < kv[:, None, None])                     # [B, Q, L]
    s = (q @ k.transpose(-1, -2)).mul_(st["scale"]).view(B, -1, Q, G, L)
    s.masked_fill_(~seen[:, None, :, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(-1e38)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m + l.log()).squeeze(-1)                                             # [B, Hkv, Q, G]
    o = (p.view(B, -1, Q * G, L) @ v).view(B, -1, Q, G, D) / torch.where(l == 0, 1.0, l)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, Q, -1, D)[live].to(torch.bfloat16)
    return o, lse.permute(0, 2, 1, 3).reshape(B, Q, -1)[live]


def run(st):
    case = st["case"]
    if own:
        import key_prefix_masked_b200 as kp
        if case["op"] == "rope":
            return kp.attn_qk_norm_rope(st["q"], st["k"], st["pos"], st["inv_freq"], q_weight=st["wq"],
                                        k_weight=st["wk"], eps=1e-6, interleaved=case["interleaved"],
                                        attn_factor=st["factor"])
        if case["op"] == "cache":
            kp.attn_cache_write(st["k"], st["v"], st["slots"], st["kc"], st["vc"], k_scale=st["ks"], v_scale=st["vs"])
            return kp.attn_cache_read(st["kc"], st["vc"], st["table"], st["kv_len"], k_scale=st["ks"],
                                      v_scale=st["vs"], k_out=st["k_out"], v_out=st["v_out"])
        return kp.attn_paged_fwd(st["q"], st["kc"], st["vc"], st["table"], st["kv_len"], st["q_start"], st["q_max"],
                                 causal=case["causal"], scale=st["scale"], k_scale=st["ks"], v_scale=st["vs"])
    if case["op"] == "rope":
        a = (st["pos"], st["inv_freq"], st["factor"], case["interleaved"])
        return _rope_plain(st["q"], st["wq"], *a), _rope_plain(st["k"], st["wk"], *a)
    return _cache_plain(st) if case["op"] == "cache" else _paged_plain(st)


# ------------------------------------------------------------------------------ work
def work(case):
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "rope":
        n = case["T"] * (case["Hq"] + Hkv) * D
        return {"bytes": 4 * n + 4 * case["T"] + 4 * case["R"], "flops": 8 * n}
    # sums over the batch: the expected lengths (one full, the rest uniform, one empty)
    B, m = case["B"], case["kv_max"]
    uniform = max(0, B - 1 - (B >= 4))
    keys = m + uniform * (m + 1) / 2
    row = 2 * Hkv * ((D + 1) if case["e4m3"] else 2 * D)      # one token's keys and values in the cache
    if case["op"] == "cache":
        new = min(case["new"], m) * (1 + uniform)
        return {"bytes": new * (4 * Hkv * D + 4) + keys * (row + 4 * Hkv * D), "flops": 4 * new * Hkv * D}
    q1 = min(case["q_max"], m)
    q = q1 + (B - 1) * (case["q_max"] + 1) / 2
    # (query, key) pairs: without a mask every row sees its sequence; with one, half of its own chunk less
    pairs = q1 * m + uniform * (case["q_max"] + 1) / 2 * (m + 1) / 2
    if case["causal"]:
        pairs -= q1 * (q1 - 1) / 2 + uniform * case["q_max"] ** 2 / 6
    pairs = max(pairs, 1.0)
    return {"bytes": keys * row + q * case["Hq"] * (4 * D + 4) + 4 * B + 4 * keys / case["page"],
            "flops": 4 * D * case["Hq"] * pairs}


# ------------------------------------------------------------------------------ 64 bits
def _rope_exact(x, w, pos, inv_freq, factor, interleaved):
    y = x.double()
    T, H, D = y.shape
    if w is not None:
        y = y / (y.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
    n = inv_freq.numel()
    first = torch.arange(n, device="cuda") * 2 if interleaved else torch.arange(n, device="cuda")
    second = first + (1 if interleaved else n)
    turn = torch.polar(torch.full((T, 1, n), factor, dtype=torch.float64, device="cuda"),
                       (pos.double()[:, None] * inv_freq)[:, None])
    z = torch.complex(y[..., first], y[..., second]) * turn
    out = y.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _row_values_exact(x):
    """What rows of x read back as from e4m3 pages, from the grid of e4m3 numbers."""
    y = x.double()
    amax = y.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(amax.clamp_min(1e-300) / E4M3_MAX))
    e = torch.where(amax <= E4M3_MAX * 2.0 ** (e - 1), e - 1, e).clamp(SCALE_MIN, SCALE_MAX)   # log2 may be an ulp high
    z = y / 2.0 ** e
    step = torch.ldexp(torch.ones_like(z), torch.frexp(z.abs().clamp_min(2.0 ** -6))[1] - 4)   # 3 bits below the first
    return torch.round(z / step) * step * 2.0 ** e         # ties to even multiples of the step


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        a = (st["pos"], st["inv_freq"], st["factor"], case["interleaved"])
        return _rope_exact(st["q"], st["wq"], *a), _rope_exact(st["k"], st["wk"], *a)
    page, kv = case["page"], st["kv_len"].tolist()

    def rows(pages, scales, b, n):
        """[Hkv, n, D] in 64 bits: sequence b's first n rows."""
        at = st["table"][b, :-(-n // page)].long()
        x = pages.view(torch.uint8)[at].view(pages.dtype).double() if scales is not None else pages[at].double()
        if scales is not None:
            x = x * 2.0 ** (scales[at].double() - 127)[..., None]
        return x.transpose(0, 1).reshape(case["Hkv"], -1, case["D"])[:, :n]

    if case["op"] == "cache":
        outs = []
        for x, c, s, o in ((st["k"], st["kc"], st["ks"], st["k_out"]), (st["v"], st["vc"], st["vs"], st["v_out"])):
            o, at = o.double(), 0
            x = _row_values_exact(x) if case["e4m3"] else x.double()
            for b, n in enumerate(kv):
                new = min(case["new"], n)
                if n:
                    o[b, :, :n] = rows(c, s, b, n)
                    o[b, :, n - new:n] = x[at:at + new].transpose(0, 1)
                at += new
            outs.append(o)
        return outs
    start = st["q_start"].tolist()
    G = case["Hq"] // case["Hkv"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(kv):
        if n == 0:
            continue
        t0, t1 = start[b], start[b + 1]
        k, v = rows(st["kc"], st["ks"], b, n), rows(st["vc"], st["vs"], b, n)
        for h in range(case["Hq"]):
            s = st["q"][t0:t1, h].double() @ k[h // G].T * st["scale"]
            if case["causal"]:
                at = torch.arange(n - (t1 - t0), n, device="cuda")[:, None]
                s = s.masked_fill(torch.arange(n, device="cuda") > at, -math.inf)
            l = torch.logsumexp(s, -1, keepdim=True)
            some = l > -math.inf
            out[t0:t1, h] = torch.where(some, (s - torch.where(some, l, 0.0)).exp(), 0.0) @ v[h // G]
            lse[t0:t1, h] = l[:, 0]
    return out, lse
