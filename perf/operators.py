"""What is measured of the 4-bit block cache: writing drafted blocks and prompts into it, reading it
back, and the attention of a drafted block over it.

A cache holds keys and values as 4-bit floats (e2m1: 0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives) with
one 8-bit scale (e4m3) for every 16 channels of a token.  With g the head's calibration scale:

    y = x * (1/g)                       in fp32, 1/g rounded to fp32
    s = max(e4m3(max |y| / 6), 2^-9)    over 16 channels, the quotient in fp32, at most 448
    c = the e2m1 value nearest to y / s, ties to the even code, at most 6 in magnitude
    x~ = c * s * g

    attention of query token j of a block of L tokens that starts at position n, for one head:
    out = sum_t softmax_t(scale * q . k~_t) v~_t over the visible positions t of [0, n + L):
    t <= n + j, and t > n + j - window where a window is given.

Positions live in pages named by a table.  A page holds, for each key/value head, runs of 16 tokens;
a run is [d/32][16 tokens][16 bytes] of key codes (two channels a byte, the lower one in the low four
bits), [16 tokens][d/16] key scales, [d][8 bytes] of value codes (two tokens a byte, the earlier one in
the low four bits) and [d/16][16 tokens] value scales.
"""
import math
import random

import torch

own = False

_RUN = 16  # tokens of a run, and channels of a scale group


# ------------------------------------------------------------------ cases --

def _attend(name, B, T, hq, hkv, d, lo, hi, page, dtype="bf16", window=0, ragged=True):
    return dict(name=name, op="attend", B=B, T=T, hq=hq, hkv=hkv, d=d, lo=lo, hi=hi, page=page,
                dtype=dtype, window=window, ragged=ragged)


def _write(name, B, T, hkv, d, lo, hi, page, dtype="bf16", ragged=True):
    return dict(name=name, op="write", B=B, T=T, hkv=hkv, d=d, lo=lo, hi=hi, page=page, dtype=dtype,
                ragged=ragged)


def _read(name, B, hkv, d, lo, hi, page, dtype="bf16"):
    return dict(name=name, op="read", B=B, hkv=hkv, d=d, lo=lo, hi=hi, page=page, dtype=dtype)


def listed():
    return [
        # one user, one token, a short conversation: the latency of a call
        _attend("attend-one-token", 1, 1, 32, 8, 128, 700, 700, 16, ragged=False),
        # one user verifying a block of five drafts over a long document
        _attend("attend-long-document", 1, 6, 32, 8, 128, 100003, 100003, 64, ragged=False),
        # the verification step of a full server: blocks of up to five drafts, mixed contexts
        _attend("attend-verify-256", 256, 6, 32, 8, 128, 64, 4096, 64),
        # plain decoding beside it, eight query heads to a key head, small pages
        _attend("attend-decode-64", 64, 1, 64, 8, 128, 500, 8192, 16, "fp16", ragged=False),
        # layers with a sliding window and narrow heads, blocks of eight drafts
        _attend("attend-window-d64", 48, 9, 32, 4, 64, 300, 20000, 32, window=1024),
        # wide heads, two query heads to a key head
        _attend("attend-d256", 24, 4, 8, 4, 256, 200, 6000, 128, "fp16"),
        # the longest block the verifier takes (16 drafts), five query heads to a key head
        _attend("attend-block-17", 33, 17, 40, 8, 128, 100, 3500, 64),
        # one request's block written and read back
        _write("write-one-block", 1, 6, 8, 128, 1001, 1001, 16, ragged=False),
        # every request's block in a full server
        _write("write-blocks-256", 256, 6, 8, 128, 64, 4096, 64),
        # prompts entering the cache
        _write("write-prompts", 4, 8191, 8, 128, 0, 77, 64, "fp16"),
        # one prefix read back, for a step that runs on whole values
        _read("read-prefix", 1, 4, 64, 1999, 1999, 32),
        # a batch moved out of the cache
        _read("read-batch", 12, 8, 128, 1000, 16384, 64, "fp16"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "write", "read"])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 5, 8])
    if op == "attend":
        B = _logint(rng, 1, 256)
        T = rng.randint(1, 17)
        group = rng.choice([1, 2, 3, 4, 5, 7, 8])
        # all tokens x heads x channels at most those of attend-verify-256
        top = max(8, min(131072, int(256 * 2080 * 8 * 128 / (B * hkv * d) * min(1.0, 24 / (T * group)))))
        hi = _logint(rng, 2, top)
        lo = max(1, int(hi * rng.uniform(0.02, 1.0)))
        window = rng.choice([0, 0, 0, _logint(rng, 1, 4096)])
        return dict(op=op, B=B, T=T, hq=group * hkv, hkv=hkv, d=d, lo=lo, hi=hi, page=page, dtype=dtype,
                    window=window, ragged=rng.random() < 0.6)
    if op == "write":
        B = _logint(rng, 1, 256)
        T = _logint(rng, 1, max(2, min(16384, int(4 * 8191 * 8 * 128 / (B * hkv * d)))))
        hi = _logint(rng, 1, 4096)
        return dict(op=op, B=B, T=T, hkv=hkv, d=d, lo=int(hi * rng.random()), hi=hi, page=page,
                    dtype=dtype, ragged=rng.random() < 0.6)
    B = _logint(rng, 1, 64)
    hi = _logint(rng, 1, max(2, min(65536, int(12 * 8000 * 8 * 128 / (B * hkv * d)))))
    return dict(op=op, B=B, hkv=hkv, d=d, lo=max(1, int(hi * rng.random())), hi=hi, page=page, dtype=dtype)


def _lengths(case):
    """(positions in the cache before the block, tokens of the block) of every request: part of the
    case, so that its work is known without its data."""
    rng = random.Random("%(op)s %(B)d %(lo)d %(hi)d %(d)d" % case)
    n = [rng.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    if case["op"] == "read":
        return n, [0] * case["B"]
    T = case["T"]
    t = [rng.randint(max(1, T // 2), T) if case["ragged"] else T for _ in range(case["B"])]
    t[-1] = T
    return n, t


def work(case):
    n, t = _lengths(case)
    d, hkv = case["d"], case["hkv"]
    packed = 2 * d * (1 / 2 + 1 / 16)  # bytes of a token and head: key and value
    if case["op"] == "read":
        tok = sum(n)
        return {"bytes": tok * hkv * (packed + 2 * 2 * d), "flops": tok * hkv * 2 * d}
    if case["op"] == "write":
        tok = sum(t)
        # the rows in, the packed tokens out and in again, the values out
        return {"bytes": tok * hkv * (2 * 2 * 2 * d + 2 * packed), "flops": tok * hkv * 2 * 4 * d}
    hq, w = case["hq"], case["window"]
    tok = pairs = 0
    for a, b in zip(n, t):
        lo = max(0, a + 1 - w) if w else 0
        tok += a + b - lo
        pairs += sum((min(w, a + j + 1) if w else a + j + 1) for j in range(b))
    return {"bytes": tok * hkv * packed + sum(t) * hq * 2 * 2 * d, "flops": pairs * hq * 4 * d}


# ------------------------------------------------- the format, plain form --

def _quantise(x, g):
    """x [..., d] -> (e2m1 codes as bytes 0..15 [..., d], e4m3 scales [..., d/16]); g broadcasts over
    x's leading dimensions."""
    y = x.float() * (1.0 / g).unsqueeze(-1)
    y = y.view(y.shape[:-1] + (y.shape[-1] // _RUN, _RUN))
    a = y.abs()
    s = (a.amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = torch.maximum(s.float(), torch.full((), 2.0 ** -9, device=x.device))
    t = s.unsqueeze(-1)
    # nearest e2m1 value: the midpoints times s are exact, ties go to the even code
    c = (a > 0.25 * t).to(torch.uint8)
    c += a >= 0.75 * t
    c += a > 1.25 * t
    c += a >= 1.75 * t
    c += a > 2.5 * t
    c += a >= 3.5 * t
    c += a > 5.0 * t
    c += 8 * torch.signbit(y).to(torch.uint8)
    return c.flatten(-2), s.to(torch.float8_e4m3fn)


def _pack(kc, ks, vc, vs):
    """Codes [n, hkv, 16, d] and scales [n, hkv, 16, d/16] of whole runs -> bytes [n, hkv, 18 d]."""
    n, h, _, d = kc.shape
    kb = kc[..., 0::2] | (kc[..., 1::2] << 4)
    kb = kb.view(n, h, _RUN, d // 32, 16).transpose(2, 3).reshape(n, h, 8 * d)
    vb = vc[:, :, 0::2] | (vc[:, :, 1::2] << 4)
    vb = vb.transpose(2, 3).reshape(n, h, 8 * d)
    return torch.cat([kb, ks.view(torch.uint8).reshape(n, h, d), vb,
                      vs.view(torch.uint8).transpose(2, 3).reshape(n, h, d)], -1)


def _values(code):
    """e2m1 codes 0..15 -> fp32 values."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    table = torch.cat([table, -table])
    return table[code.long()]


def _unpack(raw, d):
    """Bytes [n, hkv, 18 d] of runs -> K, V [16 n, hkv, d] in fp32, before the heads' scales."""
    n, h, _ = raw.shape
    kb = raw[..., :8 * d].view(n, h, d // 32, _RUN, 16).transpose(2, 3).reshape(n, h, _RUN, d // 2)
    ks = raw[..., 8 * d:9 * d].contiguous().view(torch.float8_e4m3fn).float().view(n, h, _RUN, d // 16)
    vb = raw[..., 9 * d:17 * d].reshape(n, h, d, 8)
    vs = raw[..., 17 * d:].contiguous().view(torch.float8_e4m3fn).float().view(n, h, d // 16, _RUN)
    k = torch.stack([kb & 15, kb >> 4], -1).reshape(n, h, _RUN, d)
    k = _values(k) * ks.repeat_interleave(_RUN, -1)
    v = torch.stack([vb & 15, vb >> 4], -1).reshape(n, h, d, _RUN)
    v = _values(v) * vs.repeat_interleave(_RUN, 2)
    return (k.transpose(1, 2).reshape(n * _RUN, h, d), v.permute(0, 3, 1, 2).reshape(n * _RUN, h, d))


def _runs(st, i, lo, hi):
    """The packed runs [.., hkv, 18 d] of request i's positions [lo, hi), and the first one's position."""
    page, r0, r1 = st["page"], lo // _RUN, (hi + _RUN - 1) // _RUN
    ids = st["table"][i].long()
    r = torch.arange(r0, r1, device=ids.device)
    raw = st["pages"][ids[r * _RUN // page], :, r % (page // _RUN)]
    return raw, r0 * _RUN


# ----------------------------------------------------------------- prepare --

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    n, t = _lengths(case)
    B, hkv, d, page = case["B"], case["hkv"], case["d"], case["page"]
    T = case.get("T", 0)
    per = [(a + b + page - 1) // page for a, b in zip(n, t)]
    total, most = sum(per), max(per)
    # pages in the order in which a server's free list hands them out after a while: none
    ids = torch.randperm(total, generator=gen, device=dev).to(torch.int32).cpu()
    table = torch.full((B, most), -1, dtype=torch.int32)
    at = 0
    for i, m in enumerate(per):
        table[i, :m] = ids[at:at + m]
        at += m
    # calibration: a head's largest magnitude over 6 * 448, as found on other data
    k_scale = 0.004 * (0.5 + torch.rand(hkv, generator=gen, device=dev))
    v_scale = 0.002 * (0.5 + torch.rand(hkv, generator=gen, device=dev))
    # key channels of very unlike sizes, values alike: what rotary keys and their values look like
    k_size = torch.exp(0.7 * torch.randn(hkv, d, generator=gen, device=dev))
    st = dict(op=case["op"], B=B, T=T, n=n, t=t, page=page, d=d, hkv=hkv, dtype=_DT[case["dtype"]],
              table=table.to(dev), cache_len=torch.tensor(n, dtype=torch.int32, device=dev),
              block_len=torch.tensor(t, dtype=torch.int32, device=dev), k_scale=k_scale,
              v_scale=v_scale)
    runs = page // _RUN
    pages = torch.zeros((total, hkv, runs, 18 * d), dtype=torch.uint8, device=dev)
    flat = pages.view(total, hkv, runs * 18 * d)
    step = max(1, (1 << 25) // (hkv * page * d))
    for a in range(0, total, step):
        m = min(step, total - a)
        shape = (m * runs, hkv, _RUN, d)
        k = torch.randn(shape, generator=gen, device=dev) * k_size[:, None, :]
        v = torch.randn(shape, generator=gen, device=dev)
        raw = _pack(*_quantise(k.to(st["dtype"]), k_scale[:, None]),
                    *_quantise(v.to(st["dtype"]), v_scale[:, None]))
        flat[a:a + m] = raw.view(m, runs, hkv, 18 * d).transpose(1, 2).reshape(m, hkv, runs * 18 * d)
    st["pages"] = pages
    if case["op"] == "attend":
        st["hq"], st["window"] = case["hq"], case["window"]
        st["scale"] = d ** -0.5
        q = torch.randn((B, T, case["hq"], d), generator=gen, device=dev)
        st["q"] = q.to(st["dtype"])
    elif case["op"] == "write":
        k = torch.randn((B, T, hkv, d), generator=gen, device=dev) * k_size
        v = torch.randn((B, T, hkv, d), generator=gen, device=dev)
        st["k"], st["v"] = k.to(st["dtype"]), v.to(st["dtype"])
    if case["op"] == "read":
        st["start"] = torch.zeros(B, dtype=torch.int32, device=dev)
        st["count"], st["rows"] = st["cache_len"], max(n)
    elif case["op"] == "write":
        st["start"], st["count"], st["rows"] = st["cache_len"], st["block_len"], T
    # outputs are the caller's: rows behind a request's last token stay as they are
    if case["op"] == "attend":
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros((B, T, case["hq"]), dtype=torch.float32, device=dev)
    else:
        shape = (B, st["rows"], hkv, d)
        st["k_out"] = torch.zeros(shape, dtype=st["dtype"], device=dev)
        st["v_out"] = torch.zeros(shape, dtype=st["dtype"], device=dev)
    if own:
        from speculative_decoding_verification_86_b200 import binding
        st["cache"] = binding.BlockCache(dev, heads_q=case.get("hq", hkv), heads_kv=hkv, head_dim=d,
                                         page_size=page, max_batch=B)
    return st


# --------------------------------------------------------------------- run --

def _plain_attend(st):
    """One request after another: the cache's lengths differ."""
    out, lse = st["out"], st["lse"]
    d, hkv, group = st["d"], st["hkv"], st["hq"] // st["hkv"]
    for i in range(st["B"]):
        n, L, w = st["n"][i], st["t"][i], st["window"]
        raw, at = _runs(st, i, max(0, n + 1 - w) if w else 0, n + L)
        k, v = _unpack(raw, d)
        k, v = k * st["k_scale"][:, None], v * st["v_scale"][:, None]
        q = st["q"][i, :L].float().view(L, hkv, group, d).permute(1, 0, 2, 3).reshape(hkv, L * group, d)
        s = torch.matmul(q, k.permute(1, 2, 0)).view(hkv, L, group, -1) * st["scale"]
        pos = at + torch.arange(k.shape[0], device=k.device)
        j = n + torch.arange(L, device=k.device)[:, None]
        see = pos <= j
        if w:
            see &= pos > j - w
        s = s.masked_fill(~see[:, None, :], float("-inf"))
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        o = torch.matmul((p / z).view(hkv, L * group, -1), v.transpose(0, 1))
        out[i, :L] = o.view(hkv, L, group, d).transpose(0, 1).reshape(L, hkv * group, d).to(out.dtype)
        lse[i, :L] = (m + torch.log(z)).squeeze(-1).transpose(0, 1).reshape(L, hkv * group)
    return out, lse


def _plain_read(st, start, count):
    for i in range(st["B"]):
        a, c = start[i], count[i]
        if c == 0:
            continue
        raw, at = _runs(st, i, a, a + c)
        k, v = _unpack(raw, st["d"])
        st["k_out"][i, :c] = (k[a - at:a - at + c] * st["k_scale"][:, None]).to(st["dtype"])
        st["v_out"][i, :c] = (v[a - at:a - at + c] * st["v_scale"][:, None]).to(st["dtype"])
    return st["k_out"], st["v_out"]


def _merge(old, new, a, b, d):
    """Old runs [n, hkv, 18 d] with the tokens of [a, b) (counted from the first run) taken from new."""
    n = old.shape[0]
    pos = torch.arange(n * _RUN, device=old.device).view(n, _RUN)
    mine = (pos >= a) & (pos < b)
    low = torch.where(mine[:, 0::2], 0x0F, 0) | torch.where(mine[:, 1::2], 0xF0, 0)  # [n, 8]
    full = torch.where(mine, 0xFF, 0)
    mask = torch.cat([
        full[:, None, :, None].expand(n, d // 32, _RUN, 16).reshape(n, 8 * d),
        full[:, :, None].expand(n, _RUN, d // 16).reshape(n, d),
        low[:, None, :].expand(n, d, 8).reshape(n, 8 * d),
        full[:, None, :].expand(n, d // 16, _RUN).reshape(n, d)], -1).to(torch.uint8)[:, None, :]
    return (old & ~mask) | (new & mask)


def _plain_write(st):
    d, hkv, page = st["d"], st["hkv"], st["page"]
    for i in range(st["B"]):
        n, L = st["n"][i], st["t"][i]
        old, at = _runs(st, i, n, n + L)
        m = old.shape[0]
        rows = []
        for x, g in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])):
            full = torch.zeros((m * _RUN, hkv, d), dtype=torch.float32, device=x.device)
            full[n - at:n - at + L] = x[i, :L]
            c, s = _quantise(full, g)
            rows += [c.view(m, _RUN, hkv, d).transpose(1, 2), s.view(m, _RUN, hkv, d // 16).transpose(1, 2)]
        new = _pack(*rows)
        r = torch.arange(at // _RUN, at // _RUN + m, device=old.device)
        ids = st["table"][i].long()[r * _RUN // page]
        st["pages"][ids, :, r % (page // _RUN)] = _merge(old, new, n - at, n - at + L, d)
    return _plain_read(st, st["n"], st["t"])


def run(st):
    if not own:
        if st["op"] == "attend":
            return _plain_attend(st)
        if st["op"] == "write":
            return _plain_write(st)
        return _plain_read(st, [0] * st["B"], st["n"])
    cache = st["cache"]
    where = dict(table=st["table"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    if st["op"] == "attend":
        return cache.attend(st["q"], st["pages"], cache_len=st["cache_len"], block_len=st["block_len"],
                            scale=st["scale"], window=st["window"], out=st["out"], lse=st["lse"], **where)
    if st["op"] == "write":
        cache.write(st["k"], st["v"], st["pages"], cache_len=st["cache_len"], block_len=st["block_len"],
                    **where)
    return cache.read(st["pages"], start=st["start"], count=st["count"], out=(st["k_out"], st["v_out"]),
                      **where)


# ------------------------------------------------------------------- exact --

def _decode(st, i, pos, head_major=False):
    """Keys and values of request i at the positions `pos`, in fp64, byte by byte from the definition."""
    d, page = st["d"], st["page"]
    size = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=pos.device)
    page_id = st["table"][i].long()[pos // page]
    run, tok = (pos % page) // 16, pos % 16
    c = torch.arange(d, device=pos.device)

    def e4m3(b):
        b = b.long()
        e, m = (b >> 3) & 15, (b & 7).double()
        return torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))

    def code(b):
        b = b.long()
        return size[b & 7] * (1 - 2 * (b >> 3)).double()

    flat = st["pages"][page_id, :, run]  # [tokens, hkv, 18 d]

    def take(offset):  # offset [tokens, d]
        return torch.gather(flat, 2, offset[:, None, :].expand(-1, flat.shape[1], -1))

    t = tok[:, None]
    kb = take((c // 32) * 256 + t * 16 + (c % 32) // 2)
    ks = take(8 * d + t * (d // 16) + c // 16)
    vb = take(9 * d + c * 8 + t // 2)
    vs = take(17 * d + (c // 16) * 16 + t)
    k = code(torch.where(c % 2 == 0, kb & 15, kb >> 4)) * e4m3(ks)
    v = code(torch.where((t % 2 == 0)[:, None, :], vb & 15, vb >> 4)) * e4m3(vs)
    return k * st["k_scale"].double()[:, None], v * st["v_scale"].double()[:, None]


def exact(case, seed):
    st = prepare(case, seed)
    dev = st["pages"].device
    if case["op"] == "attend":
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device=dev)
        lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device=dev)
        group = st["hq"] // st["hkv"]
        head = torch.arange(st["hq"], device=dev) // group
        for i in range(st["B"]):
            n, L, w = st["n"][i], st["t"][i], st["window"]
            first = max(0, n + 1 - w) if w else 0
            k, v = _decode(st, i, torch.arange(first, n + L, device=dev))
            for h in range(st["hkv"]):
                rows = (head == h).nonzero().flatten()
                q = st["q"][i, :L][:, rows].double()  # [L, group, d]
                s = torch.einsum("jgd,td->jgt", q, k[:, h]) * st["scale"]
                for j in range(L):
                    a = max(first, n + j + 1 - w) if w else 0
                    x = s[j, :, a - first:n + j + 1 - first]
                    z = torch.logsumexp(x, -1)
                    lse[i, j, rows] = z
                    out[i, j, rows] = torch.exp(x - z[:, None]) @ v[a - first:n + j + 1 - first, h]
        return out, lse
    outs = [torch.zeros(st["k_out"].shape, dtype=torch.float64, device=dev) for _ in range(2)]
    for i in range(st["B"]):
        if case["op"] == "read":
            pair = _decode(st, i, torch.arange(st["n"][i], device=dev))
            for o, x in zip(outs, pair):
                o[i, :st["n"][i]] = x
            continue
        L = st["t"][i]
        for o, x, g in ((outs[0], st["k"], st["k_scale"]), (outs[1], st["v"], st["v_scale"])):
            # the definition rounds y and the quotient behind the scale to fp32; the rest is exact
            y = (x[i, :L].float() * (1.0 / g)[:, None]).double().unflatten(-1, (-1, 16))
            top = (y.abs().amax(-1).float() / 6.0).double().clamp(max=448.0)
            e = torch.floor(torch.log2(top.clamp(min=2.0 ** -30))).clamp(min=-6)
            unit = torch.exp2(e - 3)
            s = (torch.round(top / unit) * unit).clamp(min=2.0 ** -9, max=448.0)
            r = (y.abs() / s.unsqueeze(-1)).clamp(max=6.0)
            step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0)).double()
            c = torch.round(r / step) * step
            c = torch.copysign(c, y) * s.unsqueeze(-1)
            o[i, :L] = c.flatten(-2) * g.double()[:, None]
    return tuple(outs)
