"""Workloads of the 4-bit floating-point draft cache and of windowed verification.

Kinds of case
  write   rows of K and V quantised into the cache as they are written, then
          read back (vc_fp4_cache_write + vc_fp4_cache_read)
  read    rows of a cache brought back to 16 or 32 bits (vc_fp4_cache_read)
  draft   one query token per request over the 4-bit cache, optionally with a
          sliding window and first tokens that stay visible (vc_draft_attn_fp4)
  verify  nq causal rows per request over the full bf16 cache with a sliding
          window and first tokens that stay visible (vc_verify_attn_window)

The plain forms below are elementary torch operations; `exact` restates each
operator in 64 bits.  Cache layout (records of 16 tokens) as in include/vc.h.
"""

import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

#: Most work a drawn case may have: (request, head, token, channel) elements of K.
MOST = {"draft": 8 * 8 * 32768 * 128, "write": 8 * 8 * 8192 * 128, "read": 4 * 8 * 32768 * 128, "verify": 8 * 8 * 16384 * 128}


def listed():
    d = dict(Hq=32, Hkv=8, D=128, ragged=False, window=0, sinks=0, exps=False)
    return [
        # one drafted token of one short request: the smallest call, latency
        {**d, "name": "draft 1 x 512", "kind": "draft", "B": 1, "T": 512},
        # the repository's default workload: 8 requests x 32K keys
        {**d, "name": "draft 8 x 32K", "kind": "draft", "B": 8, "T": 32768},
        # one request with a very long context
        {**d, "name": "draft 1 x 262K", "kind": "draft", "B": 1, "T": 262144, "exps": True},
        # 8 query heads per KV head, requests of different lengths, only the window and the first tokens visible
        {**d, "name": "draft window 4096, g 8", "kind": "draft", "B": 4, "Hq": 64, "T": 131072, "ragged": True, "window": 4096, "sinks": 4},
        # small heads, 3 query heads per KV head, odd lengths
        {**d, "name": "draft 5 x 1999, D 64", "kind": "draft", "B": 5, "Hq": 6, "Hkv": 2, "D": 64, "T": 1999, "ragged": True, "exps": True},
        # one drafted token of 8 requests appended and read back
        {**d, "name": "write 8 x 1", "kind": "write", "B": 8, "T": 4096, "n": 1, "dtype": "bf16", "ragged": True},
        # a round's verified block, of which each request keeps its accepted part
        {**d, "name": "write 16 x 31, accepted part", "kind": "write", "B": 16, "D": 64, "T": 2048, "n": 31, "dtype": "fp16", "ragged": True, "exps": True},
        # a prompt's rows when the cache is built
        {**d, "name": "write 8 x 8K", "kind": "write", "B": 8, "T": 8192, "n": 8192, "dtype": "bf16"},
        # a long prefix brought back to bf16
        {**d, "name": "read 4 x 32K", "kind": "read", "B": 4, "T": 32768, "n": 32768, "dtype": "bf16"},
        # single-token decoding of a sliding-window layer
        {**d, "name": "verify 1 row, window 1024", "kind": "verify", "B": 1, "T": 5000, "nq": 1, "window": 1024, "sinks": 4},
        # a round's block of 31 rows, sliding-window layer, 8 requests
        {**d, "name": "verify 31 rows, window 4096", "kind": "verify", "B": 8, "T": 16384, "nq": 31, "window": 4096, "sinks": 4, "ragged": True},
        # 5 query heads per KV head (two row tiles), a window longer than most requests
        {**d, "name": "verify 31 rows, g 5", "kind": "verify", "B": 2, "Hq": 40, "T": 20001, "nq": 31, "window": 16000, "sinks": 130, "ragged": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["draft", "draft", "write", "read", "verify", "verify"])
    Hkv = rng.choice([1, 2, 4, 8])
    c = {"kind": kind, "B": _log(rng, 1, 24), "Hkv": Hkv, "Hq": Hkv * rng.randint(1, 8), "D": rng.choice([64, 128, 128]),
         "ragged": rng.random() < 0.6, "window": 0, "sinks": 0, "exps": rng.random() < 0.4}
    most = MOST[kind] // (c["B"] * c["Hkv"] * c["D"])
    if kind in ("draft", "verify"):
        c["T"] = max(40, _log(rng, 40, min(most, 262144)) - rng.randint(0, 15))
        if kind == "verify" or rng.random() < 0.5:
            c["window"] = _log(rng, 16, min(c["T"], 16384))
            c["sinks"] = rng.choice([0, 1, 4, 17, 64, 200])
        if kind == "verify":
            c["nq"] = rng.choice([1, 2, rng.randint(3, 30), 31, 32])
            most = min(8 * 8 * 8192 * 128, 2**32 // (c["Hq"] // Hkv * c["nq"]))  # keys' channels, and products of them
            c["window"] = max(1, min(c["window"], most // (c["B"] * Hkv * c["D"])))
    else:
        c["dtype"] = rng.choice(["bf16", "fp16", "fp32"] if kind == "read" else ["bf16", "fp16"])
        c["n"] = _log(rng, 1, min(most // (2 if c["dtype"] == "fp32" else 1), 32768))
        c["T"] = c["n"] + rng.randint(0, 100)
    return c


def lengths(case):
    """Rows that each request holds: all of T, or spread down to a tenth of it."""
    T, B = case["T"], case["B"]
    if not case["ragged"]:
        return [T] * B
    return [max(1, int(T * (1 - 0.9 * ((b * 61) % 100) / 100))) for b in range(B)]


def counts_of(case):
    """Rows that each request writes or reads, of n."""
    n, B = case["n"], case["B"]
    return [max(1, n - (b * 7) % n) for b in range(B)] if case["ragged"] else [n] * B


def _visible(case, length):
    """Distinct keys that one request's rows see, and (row, key) pairs that count."""
    nq = case.get("nq", 1)
    w, s = case["window"] or length, case["sinks"]
    pairs, lo = 0, length
    for p in range(max(0, length - nq), length):
        first = max(0, p - w + 1)
        pairs += p + 1 - first + min(s, first)
        lo = min(lo, first)
    return length - lo + min(s, lo), pairs


def work(case):
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    if case["kind"] in ("write", "read"):
        rows = sum(counts_of(case)) * Hkv
        wide = 4 if case["dtype"] == "fp32" else 2
        if case["kind"] == "write":  # K, V in; records out and in again; K, V out
            return {"bytes": rows * (2 * D * 2 * wide + 2 * 18 * D // 16), "flops": rows * 2 * D}
        return {"bytes": rows * (2 * D * wide + 18 * D // 16), "flops": rows * 2 * D}
    nq = case.get("nq", 1)
    seen = [_visible(case, n) for n in lengths(case)]
    keys, pairs = sum(k for k, _ in seen), sum(p for _, p in seen)
    per_key = 18 * D / 16 if case["kind"] == "draft" else 4 * D
    return {"bytes": keys * Hkv * per_key + B * nq * Hq * (6 * D + 4), "flops": 4 * Hq * D * pairs}


# ---------------------------------------------------------------- the layout
def _pack(codes, scales):
    """4-bit codes [2][B, H, T, D] (one per byte) and scale bytes [2][B, H, T, D/16]
    of K and V -> records [B, H, T/16, 18 D]."""
    B, H, T, D = codes[0].shape
    byte = [c[..., 0::2] | (c[..., 1::2] << 4) for c in codes]
    k = byte[0].reshape(B, H, T // 16, 8 * D)
    # V: [half of the tokens][token pair][token of the pair][channel group][bytes]
    v = byte[1].reshape(B, H, T // 16, 2, 4, 2, 8, D // 16)
    v = (v.permute(0, 1, 2, 3, 6, 4, 5, 7) if D == 128 else v.permute(0, 1, 2, 6, 4, 3, 5, 7)).reshape(B, H, T // 16, 8 * D)
    ks = scales[0].reshape(B, H, T // 16, 2, 8, 4, D // 64).permute(0, 1, 2, 4, 5, 3, 6).reshape(B, H, T // 16, D)
    vs = scales[1].reshape(B, H, T // 16, 2, 4, 2, D // 16).permute(0, 1, 2, 6, 4, 3, 5).reshape(B, H, T // 16, D)
    return torch.cat([k, v, ks, vs], -1)


def _unpack(records):
    """records [..., 18 D] -> (codes, scale bytes) of K and V, tokens in order: [..., 16, D] and [..., 16, D/16]."""
    D, lead = records.shape[-1] // 18, records.shape[:-1]
    n = len(lead)
    k, v, ks, vs = (records[..., a * D:b * D] for a, b in ((0, 8), (8, 16), (16, 17), (17, 18)))
    ax = lambda *p: (*range(n), *(n + i for i in p))  # noqa: E731
    k = k.reshape(*lead, 16, D // 2)
    v = (v.reshape(*lead, 2, 8, 4, 2, D // 16).permute(ax(0, 2, 3, 1, 4)) if D == 128
         else v.reshape(*lead, 8, 4, 2, 2, D // 16).permute(ax(2, 1, 3, 0, 4))).reshape(*lead, 16, D // 2)
    ks = ks.reshape(*lead, 8, 4, 2, D // 64).permute(ax(2, 0, 1, 3)).reshape(*lead, 16, D // 16)
    vs = vs.reshape(*lead, D // 16, 4, 2, 2).permute(ax(2, 1, 3, 0)).reshape(*lead, 16, D // 16)
    nib = lambda b: torch.stack([b & 15, b >> 4], -1).flatten(-2)  # noqa: E731
    return (nib(k), nib(v)), (ks, vs)


def _two(exp):
    """2^exp, exactly."""
    return torch.exp2(exp.double()).float()


def _quantise(x, exp):
    """x [B, H, T, D] -> (codes, scale bytes); exp int32 [H] or None."""
    xf = torch.nan_to_num(x.float(), nan=0.0, posinf=math.inf, neginf=-math.inf)
    if exp is not None:
        xf = xf * _two(-exp)[:, None, None]
    xb = xf.unflatten(-1, (-1, 16))
    a = xb.abs()
    s8 = (a.amax(-1) / torch.full((), 6.0, device=x.device)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()[..., None]
    code = ((a > 0.25 * s).to(torch.uint8) + (a >= 0.75 * s) + (a > 1.25 * s) + (a >= 1.75 * s) + (a > 2.5 * s)
            + (a >= 3.5 * s) + (a > 5.0 * s) + 8 * torch.signbit(xb).to(torch.uint8))
    code = torch.where(s == 0, torch.zeros_like(code), code)
    return code.flatten(-2), s8.view(torch.uint8)


def _values(codes, scales, exp):
    """fp32 values of codes [B, H, ..., D] with scale bytes [B, H, ..., D/16]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    x = table[codes.int()].unflatten(-1, (-1, 16)) * scales.contiguous().view(torch.float8_e4m3fn).float()[..., None]
    x = x.flatten(-2)
    return x if exp is None else x * _two(exp).view(-1, *[1] * (x.dim() - 2))


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 17)
    B, Hq, Hkv, D, T = (case[k] for k in ("B", "Hq", "Hkv", "D", "T"))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def kv(n, dtype):
        # keys with channel outliers, as in the repository's other workloads
        k = normal(B, Hkv, n, D) * torch.exp(normal(B, Hkv, 1, D))
        return k.to(dtype), normal(B, Hkv, n, D).to(dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    s = {"case": case, "keep": {}}
    if case["kind"] == "verify":
        s["k"], s["v"] = kv(T, torch.bfloat16)
        s["q"] = normal(B, case["nq"], Hq, D).to(torch.bfloat16)
        s["lens"] = ints(lengths(case)) if case["ragged"] else None
        s["out"] = torch.zeros(B, case["nq"], Hq, D, device=DEV)
        s["lse"] = torch.zeros(B, case["nq"], Hq, device=DEV)
        return s
    cap = -(-T // 16) * 16
    s["k_exp"] = torch.randint(-2, 3, (Hkv,), generator=g, device=DEV, dtype=torch.int32) if case["exps"] else None
    s["v_exp"] = torch.randint(-2, 3, (Hkv,), generator=g, device=DEV, dtype=torch.int32) if case["exps"] else None
    if case["kind"] == "write":
        s["records"] = torch.zeros(B, Hkv, cap // 16, 18 * D, dtype=torch.uint8, device=DEV)
        s["k"], s["v"] = kv(case["n"], DTYPES[case["dtype"]])
    else:
        k, v = kv(cap, torch.bfloat16)
        kc, ks = _quantise(k, s["k_exp"])
        vc_, vs = _quantise(v, s["v_exp"])
        s["records"] = _pack((kc, vc_), (ks, vs))
        del k, v, kc, vc_
    if case["kind"] == "draft":
        s["lens"] = ints(lengths(case)) if case["ragged"] else None
        s["q"] = normal(B, Hq, D).to(torch.bfloat16)
        s["out"] = torch.zeros(B, Hq, D, device=DEV)
        s["lse"] = torch.zeros(B, Hq, device=DEV)
        return s
    # each request's rows start at a place of its own
    s["pos"] = ints([(b * 5) % (T - case["n"] + 1) for b in range(B)])
    s["counts"] = ints(counts_of(case)) if case["ragged"] else None
    s["k_out"] = torch.zeros(B, Hkv, case["n"], D, dtype=DTYPES[case["dtype"]], device=DEV)
    s["v_out"] = torch.zeros_like(s["k_out"])
    return s


# ---------------------------------------------------------------- plain forms
def _rows_at(s):
    """Positions [B, n] of the rows and whether they count [B, n]."""
    case = s["case"]
    i = torch.arange(case["n"], device=DEV)
    live = i < (s["counts"][:, None] if s["counts"] is not None else case["n"])
    return s["pos"][:, None] + i, live.expand(case["B"], -1)


def _write(s):
    case = s["case"]
    B, Hkv, D, n = case["B"], case["Hkv"], case["D"], case["n"]
    at, live = _rows_at(s)
    (kc, vc_), (ks, vs) = _unpack(s["records"])
    where = at.long()[:, None, :, None]
    keep = live[:, None, :, None]
    new = [*_quantise(s["k"], s["k_exp"]), *_quantise(s["v"], s["v_exp"])]
    held = [x.flatten(2, 3) for x in (kc, ks, vc_, vs)]

    def put(old, x):
        i = where.expand(B, Hkv, n, x.shape[-1])
        return old.contiguous().scatter(2, i, torch.where(keep, x, old.gather(2, i)))

    kc, ks, vc_, vs = (put(o, x) for o, x in zip(held, new))
    s["records"].copy_(_pack((kc, vc_), (ks, vs)))


def _read(s):
    case = s["case"]
    at, live = _rows_at(s)
    (kc, vc_), (ks, vs) = _unpack(s["records"])

    def get(codes, scales, exp, out):
        pick = lambda x: x.flatten(2, 3).gather(2, at.long()[:, None, :, None].expand(case["B"], case["Hkv"], case["n"], x.shape[-1]))  # noqa: E731
        out.copy_(torch.where(live[:, None, :, None], _values(pick(codes), pick(scales), exp).to(out.dtype), out))

    get(kc, ks, s["k_exp"], s["k_out"])
    get(vc_, vs, s["v_exp"], s["v_out"])
    return s["k_out"], s["v_out"]


def _softmax_rows(q, k, v, seen, scale):
    """q [B, H, R, D], k, v [B, H, N, D], seen [B, R or 1, N] -> (o [B, H, R, D], lse [B, H, R])."""
    x = torch.matmul(q, k.transpose(-1, -2)) * scale
    x = torch.where(seen[:, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(l == 0, 1.0, l), (m + torch.log(l))[..., 0]


def _lens(s):
    c = s["case"]
    return s["lens"].long() if s["lens"] is not None else torch.full((c["B"],), c["T"], device=DEV)


def _draft(s):
    case = s["case"]
    B, Hq, Hkv, D = (case[k] for k in ("B", "Hq", "Hkv", "D"))
    n = _lens(s)[:, None]
    recs = s["records"]
    r = torch.arange(recs.shape[2], device=DEV)[None].expand(B, -1)
    ok = torch.ones_like(r, dtype=torch.bool)
    lo = torch.zeros_like(n)
    if case["window"]:  # the sinks' records, then the window's
        lo = (n - case["window"]).clamp(min=0)
        ns, nw = -(-case["sinks"] // 16), min(case["window"] // 16 + 2, recs.shape[2])
        head = torch.arange(ns, device=DEV)[None].expand(B, -1)
        tail = lo // 16 + torch.arange(nw, device=DEV)
        r = torch.cat([head, tail], 1)
        ok = torch.cat([head < lo // 16, tail < recs.shape[2]], 1)
        r = r.clamp(max=recs.shape[2] - 1)
        recs = recs.gather(2, r[:, None, :, None].expand(B, Hkv, -1, recs.shape[3]))
    (kc, vc_), (ks, vs) = _unpack(recs)
    k, v = _values(kc, ks, s["k_exp"]).flatten(2, 3), _values(vc_, vs, s["v_exp"]).flatten(2, 3)
    t = (r[..., None] * 16 + torch.arange(16, device=DEV)).flatten(1)
    seen = ok.repeat_interleave(16, 1) & (t < n) & ((t >= lo) | (t < case["sinks"]))
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    o, l = _softmax_rows(q, k, v, seen[:, None], 1 / math.sqrt(D))
    return o.reshape(B, Hq, D), l.reshape(B, Hq)


def _verify(s):
    case = s["case"]
    B, Hq, Hkv, D, T, nq = (case[k] for k in ("B", "Hq", "Hkv", "D", "T", "nq"))
    g, n = Hq // Hkv, _lens(s)[:, None]
    w, sinks = case["window"], case["sinks"]
    lo = (n - nq + 1 - w).clamp(min=0)  # first key of the first row's window
    head = torch.arange(min(sinks, T), device=DEV)[None].expand(B, -1)
    tail = lo + torch.arange(min(w + nq - 1, T), device=DEV)
    t = torch.cat([head, tail], 1)
    ok = torch.cat([head < lo, tail < n], 1)
    at = t.clamp(max=T - 1)[:, None, :, None].expand(B, Hkv, -1, D)
    k, v = s["k"].gather(2, at).float(), s["v"].gather(2, at).float()
    p = (n - nq + torch.arange(nq, device=DEV))[:, :, None]  # positions [B, nq, 1]
    seen = ok[:, None] & (t[:, None] <= p) & ((t[:, None] > p - w) | (t[:, None] < sinks))
    q = s["q"].float().view(B, nq, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, nq * g, D)
    o, l = _softmax_rows(q, k, v, seen.repeat_interleave(g, 1), 1 / math.sqrt(D))
    o = o.view(B, Hkv, nq, g, D).permute(0, 2, 1, 3, 4).reshape(B, nq, Hq, D)
    return o, l.view(B, Hkv, nq, g).permute(0, 2, 1, 3).reshape(B, nq, Hq)


# ---------------------------------------------------------------- one pass
def _handles(s):
    """What a program makes once per layer: the shape, the cache's descriptor, a workspace."""
    from lossless_draft_verify_vc_b200 import vc

    c, k = s["case"], s["keep"]
    if not k:
        k["vc"] = vc
        k["sh"] = vc.shape(c["B"], c["Hq"], c["Hkv"], c["D"])
        if c["kind"] == "verify":
            size = vc.vc_verify_attn_window_workspace_size(k["sh"], c["T"], c["nq"], c["window"], c["sinks"])
        else:
            k["fc"] = vc.fp4_cache(s["records"], T=c["T"], lens=s.get("lens"), k_exp=s["k_exp"], v_exp=s["v_exp"])
            size = vc.vc_draft_attn_fp4_workspace_size(k["sh"], k["fc"]) if c["kind"] == "draft" else vc.vc_compress_workspace_size()
        k["ws"] = vc.workspace(size)
    return k["vc"], k["sh"], k.get("fc"), k["ws"]


def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        vc, sh, fc, ws = _handles(s)
        if kind == "draft":
            vc.vc_draft_attn_fp4(sh, fc, s["q"], s["out"], ws, lse=s["lse"], window=case["window"], n_sink=case["sinks"])
            return s["out"], s["lse"]
        if kind == "verify":
            vc.vc_verify_attn_window(sh, s["q"], s["k"], s["v"], case["T"], case["nq"], s["out"], s["lse"], ws,
                                     window=case["window"], n_sink=case["sinks"], lens=s["lens"])
            return s["out"], s["lse"]
        if kind == "write":
            vc.vc_fp4_cache_write(sh, fc, s["k"], s["v"], case["n"], ws, pos=s["pos"], counts=s["counts"])
        vc.vc_fp4_cache_read(sh, fc, case["n"], s["k_out"], s["v_out"], ws, pos=s["pos"], counts=s["counts"])
        return s["k_out"], s["v_out"]
    if kind == "draft":
        return _draft(s)
    if kind == "verify":
        return _verify(s)
    if kind == "write":
        _write(s)
    return _read(s)


# ---------------------------------------------------------------- 64 bits
def _two64(e):
    return torch.tensor([2.0**i for i in e.tolist()], dtype=torch.float64, device=DEV).view(-1, 1, 1)


def _decode64(records, exp):
    """Values [2][H, T, D] in 64 bits of one request's records [H, R, 18 D], byte by byte from the layout's addresses."""
    H, R, nb = records.shape
    D = nb // 18
    t = torch.arange(16, device=DEV)[:, None]
    c = torch.arange(D, device=DEV)[None]
    blk, grp, pair = c // 16, c // (D // 8), (t % 8) // 2
    inner = (c % (D // 8)) // 2  # byte of the channel group
    k_at = t * (D // 2) + c // 2
    v_at = 8 * D + ((t // 8) * 512 + grp * 64 + pair * 16 + (t % 2) * 8 + inner if D == 128 else grp * 64 + pair * 16 + (t // 8) * 8 + (t % 2) * 4 + inner)
    ks_at = 16 * D + ((t % 8) * 16 + (blk // 2) * 4 + (t // 8) * 2 + blk % 2 if D == 128 else (t % 8) * 8 + blk * 2 + t // 8)
    vs_at = 17 * D + blk * 16 + pair * 4 + (t // 8) * 2 + t % 2

    def value(at, s_at, e):
        byte = records[:, :, at.flatten()].view(H, R * 16, D).long()
        code = torch.where(c % 2 == 0, byte % 16, byte // 16)
        exponent, half = (code % 8) // 2, code % 2
        mag = torch.where(exponent == 0, half * 0.5, (1 + half * 0.5) * (1 << exponent) / 2)
        sb = records[:, :, s_at.expand(16, D).flatten()].view(H, R * 16, D).long()
        se, sm = sb // 8, (sb % 8).double()
        scale = torch.where(se == 0, sm * 2.0**-9, (8 + sm) * (1 << se) * 2.0**-10)
        x = torch.where(code >= 8, -mag, mag) * scale
        return x if e is None else x * _two64(e)

    return value(k_at, ks_at, exp[0]), value(v_at, vs_at, exp[1])


def _attend64(q, k, v, pos, window, sinks):
    """q [H, g, D] at position pos over the first pos + 1 rows of k, v [H, N, D]; a position before the first row sees nothing."""
    pos = max(pos, -1)
    first = max(0, pos - window + 1) if window else 0
    keys = torch.cat([torch.arange(min(sinks, first)), torch.arange(first, pos + 1)]).to(DEV)
    if not len(keys):
        return torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    kk, vv = k[:, keys], v[:, keys]
    x = torch.einsum("hgd,hnd->hgn", q, kk) / math.sqrt(q.shape[-1])
    return torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), vv), torch.logsumexp(x, -1)


def _nearest64(x, table):
    """Index of the nearest entry of an ascending table, ties to the even index; x >= 0."""
    hi = torch.searchsorted(table, x).clamp(max=len(table) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = x - table[lo], table[hi] - x
    return torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def _round64(x, e):
    """What a cache holds of x [H, n, D]."""
    x = torch.nan_to_num(x.double(), nan=0.0, posinf=1e300, neginf=-1e300)
    if e is not None:
        x = x * _two64(-e)
    i = torch.arange(127, device=DEV)
    e4m3 = torch.where(i < 8, i * 2.0**-9, (8 + i % 8).double() * (1 << (i // 8)) * 2.0**-10)
    e2m1 = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    xb = x.unflatten(-1, (-1, 16))
    s = e4m3[_nearest64(xb.abs().amax(-1) / torch.full((), 6.0, dtype=torch.float64, device=DEV), e4m3)][..., None]
    y = torch.where(s > 0, xb.abs() / torch.where(s > 0, s, 1.0), 0.0)
    y = (torch.sign(xb) * e2m1[_nearest64(y.contiguous(), e2m1)] * s).flatten(-2)
    return y if e is None else y * _two64(e)


def exact(case, seed):
    s = prepare(case, seed)
    B, Hq, Hkv, D = (case[k] for k in ("B", "Hq", "Hkv", "D"))
    if case["kind"] in ("write", "read"):
        k, v = (torch.zeros(B, Hkv, case["n"], D, dtype=torch.float64, device=DEV) for _ in range(2))
        for b, (at, n) in enumerate(zip(s["pos"].tolist(), counts_of(case))):
            if case["kind"] == "write":
                k[b, :, :n], v[b, :, :n] = _round64(s["k"][b, :, :n], s["k_exp"]), _round64(s["v"][b, :, :n], s["v_exp"])
            else:
                kk, vv = _decode64(s["records"][b], (s["k_exp"], s["v_exp"]))
                k[b, :, :n], v[b, :, :n] = kk[:, at:at + n], vv[:, at:at + n]
        return k, v
    nq = case.get("nq", 1)
    o = torch.zeros(B, nq, Hkv, Hq // Hkv, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(B, nq, Hkv, Hq // Hkv, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lengths(case)):
        k, v = (s["k"][b].double(), s["v"][b].double()) if case["kind"] == "verify" else _decode64(s["records"][b], (s["k_exp"], s["v_exp"]))
        for i in range(nq):
            q = s["q"].view(B, nq, Hkv, Hq // Hkv, D)[b, i].double()
            o[b, i], lse[b, i] = _attend64(q, k, v, n - nq + i, case["window"], case["sinks"])
    shape = (B, Hq) if case["kind"] == "draft" else (B, nq, Hq)
    return o.reshape(*shape, D), lse.reshape(shape)
