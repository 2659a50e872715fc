"""What the paged key-value cache and the attention over it compute, as cases
to measure.

Row i of a batch has ``start[i]`` tokens in its cache; its new token t stands
at position p = start[i] + t.  The cache is pages of ``page`` tokens; the page
table says which page holds which part of a row.

* ``ssd_kv_append``: the keys of the new tokens, turned by their positions, and
  their values go into the cache; the queries are turned in the same pass.
* ``ssd_attn_step`` and ``ssd_attn_fwd``: attention of one new token per row,
  or of several, to every key at its own position or before it (with a window,
  to the last ``window`` of them):

      out = sum_j softmax_j(scale * q . k_j) v_j,   lse = log sum_j e^(scale * q . k_j)

``own`` chooses between the plain torch form and the library's kernels.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _append(name, b, L, Hq, Hk, N, R, page, ctx, dtype, interleaved=False, fused=True, ragged=False, some=False):
    c = dict(op="append", b=b, L=L, Hq=Hq, Hk=Hk, N=N, R=R, page=page, ctx=ctx, dtype=dtype,
             interleaved=interleaved, fused=fused, ragged=ragged, some=some)
    if name:
        c["name"] = name
    return c


def _attn(name, kind, b, L, Hq, Hk, N, page, ctx, dtype, window=0, ragged=False, some=False):
    c = dict(op="attn", kind=kind, b=b, L=L, Hq=Hq, Hk=Hk, N=N, page=page, ctx=ctx, dtype=dtype,
             window=window, ragged=ragged, some=some)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one request, one token: the latency of a decode step
        _append("append_step_b1", 1, 1, 32, 8, 128, 128, 16, 1000, "bf16"),
        # a full decode batch, each request at its own position
        _append("append_step_b256", 256, 1, 32, 8, 128, 128, 64, 4000, "bf16", ragged=True),
        # prompts: queries, keys and values are slices of one projection
        _append("append_prompt_b4", 4, 4096, 32, 8, 128, 128, 64, 0, "bf16"),
        # a padded fp32 batch behind caches of several lengths: an empty row, adjacent pairs, part of the head turned
        _append("append_ragged", 5, 333, 7, 1, 80, 40, 24, 5000, "f32", interleaved=True, ragged=True, some=True),
        # one request, one token, a short cache: the latency of a decode step
        _attn("step_b1", "step", 1, 1, 32, 8, 128, 16, 999, "bf16"),
        # a decode batch with caches from nearly nothing to 16384 tokens
        _attn("step_b128", "step", 128, 1, 32, 8, 128, 64, 16384, "bf16", ragged=True),
        # one request with a very long cache: only the cache's length can be split
        _attn("step_long", "step", 1, 1, 32, 8, 128, 128, 262143, "bf16"),
        # local attention between recurrences: wide heads, one key head, a window
        _attn("step_window", "step", 64, 1, 10, 1, 256, 16, 20000, "bf16", window=2048, ragged=True),
        # a few drafted tokens for each request, fp32, odd sizes, a row without any
        _attn("draft_f32", "fwd", 9, 5, 6, 2, 80, 24, 3001, "f32", ragged=True, some=True),
        # prompts from their first token on
        _attn("prompt_b4", "fwd", 4, 4096, 32, 8, 128, 64, 0, "bf16"),
        # one piece of a long prompt behind the pieces before it
        _attn("prompt_piece", "fwd", 1, 512, 32, 8, 128, 64, 32000, "bf16"),
        # padded prompts with a window, fp32, odd sizes
        _attn("prompt_window_f32", "fwd", 3, 777, 5, 1, 96, 100, 1500, "f32", window=500, ragged=True, some=True),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    e = 2 if dtype == "bf16" else 4
    N = rng.choice([16, 32, 64, 80, 96, 128, 128, 192, 256])
    Hk = _logint(rng, 1, 12)
    Hq = Hk * rng.choice([1, 2, 3, 4, 4, 7, 8, 10])
    page = rng.choice([1, 16, 16, 24, 32, 64, 64, 100, 128, 256])
    ragged, some = rng.random() < 0.6, rng.random() < 0.4
    if rng.random() < 0.35:
        b = _logint(rng, 1, 256)
        L = 1 if rng.random() < 0.4 else max(1, min(_logint(rng, 1, 8192), int(160e6 / (b * (Hq + 2 * Hk) * N * e))))
        ctx = min(_logint(rng, 1, 20000), max(1, int(2e9 / (2 * b * Hk * N * e))))
        return _append(None, b, L, Hq, Hk, N, rng.choice([N, N, N // 2, 0]) // 8 * 8, page, ctx, dtype,
                       interleaved=rng.random() < 0.5, fused=rng.random() < 0.6, ragged=ragged, some=some and L > 1)
    window = rng.choice([0, 0, 0, _logint(rng, 16, 4096)])
    if rng.random() < 0.6:
        b = _logint(rng, 1, 256)
        ctx = min(_logint(rng, 1, 262144), max(1, int(3e9 / (2 * b * Hk * N * e))))
        return _attn(None, "step", b, 1, Hq, Hk, N, page, ctx, dtype, window, ragged)
    b = _logint(rng, 1, 32)
    ctx = min(_logint(rng, 1, 32768), max(1, int(2e9 / (2 * b * Hk * N * e))))
    if rng.random() < 0.4:
        return _attn(None, "fwd", b, rng.randint(2, 16), Hq, Hk, N, page, ctx, dtype, window, ragged, some)
    if rng.random() < 0.5:
        ctx = 0
    # at most the products of the largest prompt above, a tenth of them in fp32
    cap = 4.0e11 * (1.0 if dtype == "bf16" else 0.1) / (4 * N * Hq * b)
    L = _logint(rng, 17, 8192)
    while L > 17 and L * (ctx + L / 2) > cap:
        L = max(17, L * 3 // 4)
    if L * (ctx + L / 2) > cap:
        ctx = max(1, int(cap / L))
    return _attn(None, "fwd", b, L, Hq, Hk, N, page, ctx, dtype, window, ragged, some)


def _starts(case):
    """Tokens in each row's cache before the call."""
    if not case["ragged"]:
        return [case["ctx"]] * case["b"]
    return [int(case["ctx"] * ((i + 1) * 0.6180339887498949 % 1.0)) for i in range(case["b"])]


def _tokens(case):
    """New tokens of each row, from none to all of L."""
    b, L = case["b"], case["L"]
    if not case["some"]:
        return [L] * b
    if b == 1:
        return [(2 * L + 2) // 3]
    return [L * i // (b - 1) for i in range(b)]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    b, L, Hq, Hk, N, page = (case[k] for k in ("b", "L", "Hq", "Hk", "N", "page"))
    dt = DTYPES[case["dtype"]]
    starts, tokens = _starts(case), _tokens(case)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    # pages dealt out in no order; the table is as wide as the longest row's, entries no row has yet are -1
    used = [-(-(s + n) // page) for s, n in zip(starts, tokens)]
    width, total = max(max(used), 1), max(sum(used), 1)
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.full((b, width), -1, dtype=torch.int32, device=dev)
    first = torch.tensor([sum(used[:i]) for i in range(b)], device=dev)
    have = torch.arange(width, device=dev)[None] < torch.tensor(used, device=dev)[:, None]
    src = first[:, None] + torch.arange(width, device=dev)[None]
    table[have] = order[src[have]]
    kc, vc = (torch.empty(total, page, Hk, N, dtype=dt, device=dev) for _ in range(2))
    for c in (kc, vc):
        per = max(1, (1 << 28) // (page * Hk * N))
        for i in range(0, total, per):
            c[i:i + per] = randn(min(per, total - i), page, Hk, N).to(dt)
    st = dict(case=case, table=table, kc=kc, vc=vc, starts=starts, counts=tokens,
              start=torch.tensor(starts, dtype=torch.int32, device=dev),
              tokens=torch.tensor(tokens, dtype=torch.int32, device=dev) if case["some"] else None)
    if case["op"] == "append":
        if case["fused"]:
            proj = randn(b, L, Hq + 2 * Hk, N).to(dt)
            st.update(q=proj[:, :, :Hq], k=proj[:, :, Hq:Hq + Hk], v=proj[:, :, Hq + Hk:])
        else:
            st.update(q=randn(b, L, Hq, N).to(dt), k=randn(b, L, Hk, N).to(dt), v=randn(b, L, Hk, N).to(dt))
        R = case["R"]
        st["freqs"] = None
        if R:
            j = torch.arange(R // 2, device=dev, dtype=torch.float64)
            st["freqs"] = (10000.0 ** (-2.0 * j / R)).float()
        # zeros, since the tokens a row does not have are left as they were
        st["q_out"] = torch.zeros(b, L, Hq, N, dtype=dt, device=dev)
        return st
    # scores of a few units, as of trained heads
    st["scale"] = 2.0 / math.sqrt(N)
    if case["kind"] == "step":
        st["q"] = randn(b, Hq, N).to(dt)
        return st
    st["q"] = randn(b, L, Hq, N).to(dt)
    st["out"] = torch.zeros(b, L, Hq, N, dtype=dt, device=dev)
    st["lse"] = torch.zeros(b, L, Hq, device=dev)
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    if state["case"]["op"] == "append":
        return _own_append(state) if own else _plain_append(state)
    return _own_attn(state) if own else _plain_attn(state)


def _own_append(s):
    from mamba_ssd_scan_05_amd import ssd
    q_out = ssd.ssd_kv_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["start"], q=s["q"], freqs=s["freqs"],
                              tokens=s["tokens"], interleaved=s["case"]["interleaved"], q_out=s["q_out"])
    return q_out, s["kc"], s["vc"]


def _own_attn(s):
    from mamba_ssd_scan_05_amd import ssd
    opts = dict(scale=s["scale"], window=s["case"]["window"])
    if s["case"]["kind"] == "step":
        return ssd.ssd_attn_step(s["q"], s["kc"], s["vc"], s["table"], s["start"], **opts)
    return ssd.ssd_attn_fwd(s["q"], s["kc"], s["vc"], s["table"], s["start"], tokens=s["tokens"], out=s["out"],
                            lse=s["lse"], **opts)


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def _turn(v, cos, sin, interleaved):
    R = 2 * cos.shape[-1]
    rot, rest = v[..., :R], v[..., R:]
    if interleaved:
        p, q = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([p * cos - q * sin, p * sin + q * cos], -1).flatten(-2)
    else:
        p, q = rot[..., :R // 2], rot[..., R // 2:]
        rot = torch.cat([p * cos - q * sin, p * sin + q * cos], -1)
    return torch.cat([rot, rest], -1)


def _plain_append(s):
    case, k, v, table = s["case"], s["k"], s["v"], s["table"]
    b, L, page = case["b"], case["L"], case["page"]
    pos = s["start"].long()[:, None] + torch.arange(L, device=k.device)[None]
    q, kk = s["q"].float(), k.float()
    if s["freqs"] is not None:
        ang = pos.double()[..., None] * s["freqs"].double()
        cos, sin = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]
        q, kk = _turn(q, cos, sin, case["interleaved"]), _turn(kk, cos, sin, case["interleaved"])
    entry = (pos // page).clamp(max=table.shape[1] - 1)
    where = torch.gather(table.long(), 1, entry) * page + pos % page
    kc, vc = s["kc"].flatten(0, 1), s["vc"].flatten(0, 1)
    if s["tokens"] is None:
        where = where.flatten()
        kc[where] = kk.to(kc.dtype).flatten(0, 1)
        vc[where] = v.flatten(0, 1)
        s["q_out"].copy_(q)
    else:
        new = torch.arange(L, device=k.device)[None] < s["tokens"][:, None]
        kc[where[new]] = kk.to(kc.dtype)[new]
        vc[where[new]] = v[new]
        s["q_out"].copy_(torch.where(new[..., None, None], q.to(k.dtype), s["q_out"]))
    return s["q_out"], s["kc"], s["vc"]


def _plain_attn(s):
    case, table = s["case"], s["table"]
    b, L, Hq, Hk, N, page, window = (case[k] for k in ("b", "L", "Hq", "Hk", "N", "page", "window"))
    step = case["kind"] == "step"
    q = s["q"].reshape(b, L, Hq, N)
    dev, G = q.device, Hq // Hk
    kc, vc = s["kc"].flatten(0, 1), s["vc"].flatten(0, 1)
    # the first key of each row that one of its tokens sees, and the keys from there on
    low = [max(0, a + 1 - window) if window else 0 for a in s["starts"]]
    span = [max(1, a + n - l) for a, n, l in zip(s["starts"], s["counts"], low)]
    out, lse = torch.empty(b, L, Hq, N, device=dev), torch.empty(b, L, Hq, device=dev)
    i = 0
    while i < b:
        S, j = span[i], i + 1  # as many rows at once as fit
        while j < b and (j + 1 - i) * max(S, span[j]) * max(Hk * N, Hq * L) <= 1 << 29:
            S, j = max(S, span[j]), j + 1
        first = (s["start"][i:j].long() + 1 - window).clamp(min=0) if window else torch.zeros(j - i, dtype=torch.long, device=dev)
        key = first[:, None] + torch.arange(S, device=dev)[None]
        entry = torch.gather(table[i:j].long(), 1, (key // page).clamp(max=table.shape[1] - 1))
        where = entry.clamp(min=0) * page + key % page
        k = kc[where].float().permute(0, 2, 3, 1).contiguous()               # rows, Hk, N, S
        v = vc[where].float().transpose(1, 2).contiguous()                   # rows, Hk, S, N
        qq = q[i:j].float().unflatten(2, (Hk, G)).permute(0, 2, 3, 1, 4).reshape(j - i, Hk, G * L, N)
        score = (torch.matmul(qq, k) * s["scale"]).unflatten(2, (G, L))      # rows, Hk, G, L, S
        pos = s["start"][i:j].long()[:, None] + torch.arange(L, device=dev)[None]
        seen = key[:, None, :] <= pos[:, :, None]
        if window:
            seen &= key[:, None, :] > pos[:, :, None] - window
        score = torch.where(seen[:, None, None], score, -math.inf)
        top = score.amax(-1, keepdim=True)
        w = torch.exp(score - top)
        total = w.sum(-1, keepdim=True)
        o = torch.matmul(w.flatten(2, 3), v).unflatten(2, (G, L)) / total
        out[i:j] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)
        lse[i:j] = (top + total.log())[..., 0].permute(0, 3, 1, 2).flatten(2, 3)
        i = j
    if step:
        return out.to(q.dtype).reshape(b, Hq, N)
    if s["tokens"] is not None:
        new = (torch.arange(L, device=dev)[None] < s["tokens"][:, None])[..., None]
        s["out"].copy_(torch.where(new[..., None], out.to(q.dtype), s["out"]))
        s["lse"].copy_(torch.where(new, lse, s["lse"]))
    else:
        s["out"].copy_(out)
        s["lse"].copy_(lse)
    return s["out"], s["lse"]


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    b, Hq, Hk, N, page = (case[k] for k in ("b", "Hq", "Hk", "N", "page"))
    starts, tokens = _starts(case), _tokens(case)
    new = sum(tokens)
    if case["op"] == "append":
        pages = sum(-(-(s + n) // page) - s // page for s, n in zip(starts, tokens) if n)
        return {"bytes": 2 * e * N * (Hq + 2 * Hk) * new + 2 * case["R"] + 4 * (b + pages),
                "flops": 3 * case["R"] * (Hq + Hk) * new}
    keys = pairs = pages = 0
    w = case["window"]
    for s, n in zip(starts, tokens):
        if n == 0:
            continue
        low = max(0, s + 1 - w) if w else 0
        keys += s + n - low
        pages += -(-(s + n) // page) - low // page
        pairs += sum(min(s + t + 1, w) for t in range(n)) if w else n * s + n * (n + 1) // 2
    size = 2 * e * N * Hk * keys + 2 * e * N * Hq * new + 4 * (b + pages)
    return {"bytes": size + (0 if case["kind"] == "step" else 4 * Hq * new), "flops": 4 * N * Hq * pairs}


# --------------------------------------------------------------------------
# the definitions in 64 bits, row by row
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attn(s)


def _slots(s, i, positions):
    """Where a row's positions lie in the cache seen as one list of tokens."""
    page = s["case"]["page"]
    return s["table"][i].long()[positions // page] * page + positions % page


def _exact_append(s):
    d64, case = torch.float64, s["case"]
    kc, vc = s["kc"].to(d64), s["vc"].to(d64)
    q_out = s["q_out"].to(d64)
    fk, fv = kc.flatten(0, 1), vc.flatten(0, 1)
    for i, (start, n) in enumerate(zip(s["starts"], s["counts"])):
        if n == 0:
            continue
        pos = torch.arange(start, start + n, device=kc.device)
        q, k = s["q"][i, :n].to(d64), s["k"][i, :n].to(d64)
        if s["freqs"] is not None:
            ang = pos.to(d64)[:, None, None] * s["freqs"].to(d64)
            e, half = torch.polar(torch.ones_like(ang), ang), s["freqs"].shape[0]
            for t in (q, k):
                a, c = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else (slice(0, half), slice(half, 2 * half))
                z = torch.complex(t[..., a].clone(), t[..., c].clone()) * e
                t[..., a], t[..., c] = z.real, z.imag
        at = _slots(s, i, pos)
        fk[at], fv[at], q_out[i, :n] = k, s["v"][i, :n].to(d64), q
    return q_out, kc, vc


def _exact_attn(s):
    d64, case = torch.float64, s["case"]
    b, L, Hq, Hk, N, window = (case[k] for k in ("b", "L", "Hq", "Hk", "N", "window"))
    q = s["q"].reshape(b, L, Hq, N)
    out = torch.zeros(b, L, Hq, N, dtype=d64, device=q.device)
    lse = torch.zeros(b, L, Hq, dtype=d64, device=q.device)
    kc, vc = s["kc"].flatten(0, 1), s["vc"].flatten(0, 1)
    for i, (start, n) in enumerate(zip(s["starts"], s["counts"])):
        if n == 0:
            continue
        low = max(0, start + 1 - window) if window else 0
        key = torch.arange(low, start + n, device=q.device)
        at = _slots(s, i, key)
        gone = key[None] > start + torch.arange(n, device=q.device)[:, None]
        if window:
            gone |= key[None] <= start + torch.arange(n, device=q.device)[:, None] - window
        for h in range(Hk):
            k, v = kc[at, h].to(d64), vc[at, h].to(d64)
            kt = k.t().contiguous()
            for j in range(h * (Hq // Hk), (h + 1) * (Hq // Hk)):
                z = (q[i, :n, j].to(d64) @ kt).mul_(s["scale"]).masked_fill_(gone, -math.inf)
                total = torch.logsumexp(z, -1)
                out[i, :n, j] = (z - total[:, None]).exp_() @ v
                lse[i, :n, j] = total
    return out[:, 0] if case["kind"] == "step" else (out, lse)
