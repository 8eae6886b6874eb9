"""The 4-bit block cache (spec_cache_*) against its definition in 64 bits: stored bytes and read-back
values exactly, attention within bounds derived from its roundings."""
import math

import numpy as np
import pytest
import torch

import cache_reference as ref
from speculative_decoding_verification_86_b200 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_device):
    return cuda_device


def make(dev, *, B, T, heads_q, heads_kv, d, page, lens, dtype=torch.bfloat16, seed=0, block=None, spare=2,
         scales=True, width=None):
    """A cache object, a pool of random bytes whose visible positions were written with the reference,
    a table of shuffled pages, and a block's q, k, v."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.RandomState(seed)
    per = [max(1, (n + T + page - 1) // page) for n in lens]
    width = width or max(per)
    num = sum(per) + spare
    ids = rng.permutation(num)
    table = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for i, m in enumerate(per):
        table[i, :m] = ids[at:at + m]
        at += m
    raw = rng.randint(0, 256, size=(num, heads_kv, page // 16, 18 * d)).astype(np.uint8)
    ks = (0.01 * (0.5 + rng.rand(heads_kv))).astype(np.float32) if scales else None
    vs = (0.003 * (0.5 + rng.rand(heads_kv))).astype(np.float32) if scales else None
    most = max(max(lens), 1)
    k = torch.randn((B, most, heads_kv, d), generator=g) * torch.exp(0.7 * torch.randn((heads_kv, d), generator=g))
    v = torch.randn((B, most, heads_kv, d), generator=g)
    raw = ref.write(raw, page, table, [0] * B, k.to(dtype), v.to(dtype), lens, ks, vs)
    q = torch.randn((B, T, heads_q, d), generator=g).to(dtype)
    kb = torch.randn((B, T, heads_kv, d), generator=g).to(dtype)
    vb = torch.randn((B, T, heads_kv, d), generator=g).to(dtype)
    return dict(cache=binding.BlockCache(dev, heads_q, heads_kv, d, page, max_batch=max(B, 1)), raw=raw, page=page,
                table=table, lens=lens, block=block, ks=ks, vs=vs, q=q, k=kb, v=vb, dev=dev)


def on(dev, x, dtype=torch.int32):
    return None if x is None else torch.as_tensor(np.asarray(x)).to(dtype).to(dev)


def device_args(s):
    dev = s["dev"]
    return dict(table=on(dev, s["table"]), cache_len=on(dev, s["lens"]), block_len=on(dev, s["block"]),
                k_scale=on(dev, s["ks"], torch.float32), v_scale=on(dev, s["vs"], torch.float32))


def check_attend(s, causal=True, window=0, scale=None, out=None, lse=None, q=None, cache=None):
    """Write the block with the library, attend, compare both with the reference."""
    dev = s["dev"]
    a = device_args(s)
    pages = torch.from_numpy(s["raw"]).to(dev)
    cache = cache or s["cache"]
    q = s["q"] if q is None else q
    cache.write(s["k"].to(dev), s["v"].to(dev), pages, **a)
    got, glse = cache.attend(q.to(dev), pages, causal=causal, window=window, scale=scale, out=out, lse=lse, **a)
    torch.cuda.synchronize(dev)
    assert cache.errors() == 0
    raw = ref.write(s["raw"], s["page"], s["table"], s["lens"], s["k"], s["v"], s["block"], s["ks"], s["vs"])
    assert np.array_equal(pages.cpu().numpy(), raw)
    compare(s, raw, q, got, glse, causal, window, scale)
    return got, glse


def compare(s, raw, q, got, glse, causal=True, window=0, scale=None):
    d = q.shape[-1]
    sc = d ** -0.5 if scale is None else scale
    out, l, a, size, done = ref.attend(raw, s["page"], s["table"], s["lens"], q, s["block"], sc, causal, window,
                                       s["ks"], s["vs"])
    tokens = max(s["lens"]) + q.shape[1]
    tol, tol_lse = ref.attend_bounds(out, l, a, size, tokens, d, q.dtype)
    g, gl = ref.to_np(got), ref.to_np(glse)
    nan = np.isnan(out) & done[..., None, None]
    assert np.array_equal(np.isnan(g) & done[..., None, None], nan)
    ok = done[..., None, None] & ~nan
    err = np.where(ok, np.abs(g - np.where(nan, 0, out)) - tol, -1)
    assert err.max() <= 0, (err.max(), np.unravel_index(err.argmax(), err.shape))
    nl = np.isnan(l) & done[..., None]
    assert np.array_equal(np.isnan(gl) & done[..., None], nl)
    inf = np.isneginf(l)
    assert np.all(np.isneginf(gl[inf & done[..., None]]))
    okl = done[..., None] & ~nl & ~inf
    errl = np.where(okl, np.abs(np.where(okl, gl, 0) - np.where(okl, l, 0)) - tol_lse, -1)
    assert errl.max() <= 0, (errl.max(), np.unravel_index(errl.argmax(), errl.shape))


# ------------------------------------------------------------ write and read --

@pytest.mark.parametrize("d,heads,page,T,lens,dtype,scales", [
    (128, 2, 16, 1, [0], torch.bfloat16, True),
    (128, 1, 64, 6, [0, 1, 15, 16, 17, 63, 64], torch.bfloat16, True),
    (64, 3, 32, 5, [31, 27, 40], torch.float16, True),
    (256, 1, 128, 17, [3, 120], torch.float32, True),
    (128, 2, 256, 35, [250, 5], torch.bfloat16, False),
    (64, 1, 16, 50, [7], torch.float32, False),
])
def test_write_stores_the_defined_bytes_and_read_returns_them(dev, d, heads, page, T, lens, dtype, scales):
    B = len(lens)
    block = [T, 0, 1, T, 2, T - 1, T][:B]
    s = make(dev, B=B, T=T, heads_q=heads, heads_kv=heads, d=d, page=page, lens=lens, dtype=dtype, block=block,
             scales=scales, seed=d + page)
    a = device_args(s)
    pages = torch.from_numpy(s["raw"]).to(dev)
    status = torch.zeros(B, dtype=torch.int32, device=dev)
    s["cache"].write(s["k"].to(dev), s["v"].to(dev), pages, status=status, **a)
    raw = ref.write(s["raw"], page, s["table"], lens, s["k"], s["v"], block, s["ks"], s["vs"])
    assert np.array_equal(pages.cpu().numpy(), raw)  # every other byte and half byte as it was
    assert status.tolist() == [0] * B
    # read the last positions back, from an odd start
    pool = ref.Pool(raw, page)
    start = [max(0, n - 3) for n in lens]
    count = [n + b - st for n, b, st in zip(lens, block, start)]
    rows = max(count) + 2
    for out_dtype in (torch.float32, torch.bfloat16, torch.float16):
        out = tuple(torch.full((B, rows, heads, d), 7.0, dtype=out_dtype, device=dev) for _ in range(2))
        s["cache"].read(pages, a["table"], start=on(dev, start), count=on(dev, count), out=out,
                        k_scale=a["k_scale"], v_scale=a["v_scale"], status=status)
        for i in range(B):
            for j in range(rows):
                got = [o[i, j].cpu() for o in out]
                if j >= count[i]:
                    assert all(bool((x == 7.0).all()) for x in got)
                    continue
                for x, val, gs in zip(got, pool.get(s["table"][i], start[i] + j), (s["ks"], s["vs"])):
                    gs = np.ones(heads, np.float32) if gs is None else gs
                    want = (val.astype(np.float32) * gs[:, None]).astype(np.float32)
                    assert torch.equal(x, torch.from_numpy(want).to(out_dtype))
    assert status.tolist() == [0] * B


def test_write_rounds_ties_to_even_and_keeps_signs_and_non_finite_groups(dev):
    """Values on the midpoints of the codes, at the scales' ends, zeros of both signs, the type's
    extremes, NaN and infinities: the stored bytes are the definition's."""
    d, page = 64, 16
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    rows = []
    for s in (1.0, 2.0 ** -9, 448.0, 0.0703125, 1.125, 2.0 ** -6):
        rows.append(np.concatenate([mids * s, -mids * s]))
        rows.append(np.concatenate([np.nextafter(np.float32(mids * s), np.float32(0)), -mids[::-1] * s]))
        rows.append(np.concatenate([np.nextafter(np.float32(mids * s), np.float32(1e9)), mids * s]))
    rows += [np.zeros(16), -np.zeros(16), np.full(16, 2.0 ** -12), np.full(16, -1e-30), np.full(16, 3e38),
             np.full(16, -2688.0), np.full(16, 2689.0)]
    for special in (np.nan, np.inf, -np.inf):
        x = np.linspace(-3, 3, 16)
        x[5] = special
        rows.append(x)
    rng = np.random.RandomState(3)
    while len(rows) % 4:
        rows.append(rng.randn(16))
    # e4m3 halfway cases of the scale itself
    x = np.concatenate(rows).astype(np.float32).reshape(1, -1, 1, d)
    T = x.shape[1]
    table = np.arange((T + page - 1) // page, dtype=np.int32)[None]
    raw = np.random.RandomState(0).randint(0, 256, size=(table.shape[1], 1, 1, 18 * d)).astype(np.uint8)
    for dtype in (torch.float32, torch.bfloat16):
        k = torch.from_numpy(x).to(dtype)
        v = torch.flip(k, dims=[3]).contiguous()
        for g in (None, np.array([0.37], np.float32)):
            with binding.BlockCache(dev, 1, 1, d, page, max_batch=1) as c:
                pages = torch.from_numpy(raw).to(dev)
                c.write(k.to(dev), v.to(dev), pages, on(dev, table), on(dev, [0]),
                        k_scale=on(dev, g, torch.float32), v_scale=on(dev, g, torch.float32))
                want = ref.write(raw, page, table, [0], k, v, None, g, g)
                assert np.array_equal(pages.cpu().numpy(), want)


def test_write_takes_slices_of_a_fused_projection(dev):
    s = make(dev, B=3, T=4, heads_q=4, heads_kv=2, d=64, page=16, lens=[5, 30, 0], seed=5)
    a = device_args(s)
    fused = torch.zeros((3, 4 + 2, 8 + 1, 64), dtype=torch.bfloat16, device=dev)
    fused[:, 1:5, 4:6] = s["k"].to(dev)
    fused[:, 1:5, 6:8] = s["v"].to(dev)
    fused[:, 1:5, 0:4] = s["q"].to(dev)
    part = fused[:, 1:5]
    pages = torch.from_numpy(s["raw"]).to(dev)
    s["cache"].write(part[:, :, 4:6], part[:, :, 6:8], pages, **a)
    raw = ref.write(s["raw"], 16, s["table"], s["lens"], s["k"], s["v"], None, s["ks"], s["vs"])
    assert np.array_equal(pages.cpu().numpy(), raw)
    # queries by heads first, outputs into a wider tensor
    by_head = part[:, :, 0:4].transpose(1, 2).contiguous().transpose(1, 2)
    wide = torch.full((3, 4, 6, 64), 9.0, dtype=torch.bfloat16, device=dev)
    out, lse = s["cache"].attend(by_head, pages, out=wide[:, :, 1:5], **a)
    compare(s, raw, s["q"], out, lse)
    assert bool((wide[:, :, 0] == 9).all()) and bool((wide[:, :, 5] == 9).all())


# ------------------------------------------------------------------ attention --

@pytest.mark.parametrize("d,hq,hkv,page,T,lens,dtype", [
    (128, 1, 1, 16, 1, [0], torch.bfloat16),
    (128, 4, 1, 64, 1, [1, 15, 16, 127, 128, 129], torch.bfloat16),
    (128, 8, 2, 16, 6, [0, 3, 122, 250, 255, 256, 300], torch.bfloat16),
    (128, 8, 2, 64, 6, [700, 0, 64], torch.float16),
    (64, 6, 2, 32, 5, [0, 11, 500, 129], torch.bfloat16),
    (64, 16, 1, 128, 2, [260, 1], torch.float16),
    (256, 4, 2, 16, 3, [0, 140, 257], torch.bfloat16),
    (256, 8, 1, 64, 4, [200, 30], torch.float16),
    (128, 5, 1, 256, 17, [90, 0, 250], torch.bfloat16),
    (128, 8, 1, 64, 17, [100, 333], torch.float16),
    (256, 16, 1, 32, 9, [77], torch.bfloat16),
    (64, 7, 7, 16, 40, [20, 0], torch.bfloat16),
])
@pytest.mark.parametrize("mask", ["causal", "all", "window"])
def test_attend_matches_its_definition(dev, d, hq, hkv, page, T, lens, dtype, mask):
    B = len(lens)
    block = None if B == 1 else [T, max(1, T // 2), T, 1, T, T, T][:B]
    s = make(dev, B=B, T=T, heads_q=hq, heads_kv=hkv, d=d, page=page, lens=lens, dtype=dtype, block=block,
             seed=d + hq + page)
    check_attend(s, causal=mask != "all", window=33 if mask == "window" else 0)


@pytest.mark.parametrize("window", [1, 2, 16, 17, 128, 200, 10 ** 9])
def test_attend_window_edges(dev, window):
    s = make(dev, B=3, T=7, heads_q=2, heads_kv=1, d=64, page=16, lens=[0, 150, 271], block=[7, 5, 7], seed=11)
    check_attend(s, window=window)
    check_attend(s, window=window, causal=False)


def test_attend_scale_signs_and_sizes(dev):
    """Scores of thousands (a softmax on one token), a negative scale, scale 0 (a plain mean)."""
    s = make(dev, B=2, T=3, heads_q=4, heads_kv=2, d=128, page=32, lens=[200, 33], seed=21)
    for scale in (40.0, -0.3, 0.0, 1e-6):
        check_attend(s, scale=scale)


def test_attend_growing_scores_move_the_maximum(dev):
    """Keys that grow along the context raise each row's running maximum again and again."""
    d, n = 64, 1000
    s = make(dev, B=1, T=2, heads_q=2, heads_kv=1, d=d, page=16, lens=[n], seed=31, scales=False)
    base = torch.randn(d, generator=torch.Generator().manual_seed(1))
    k = (base * torch.linspace(0.01, 9.0, n)[:, None]).view(1, n, 1, d)
    v = torch.randn((1, n, 1, d), generator=torch.Generator().manual_seed(2))
    s["raw"] = ref.write(s["raw"], 16, s["table"], [0], k, v)
    q = torch.stack([base, -base]).view(1, 1, 2, d).expand(1, 2, 2, d).to(torch.bfloat16).contiguous()
    check_attend(s, q=q, scale=0.25)


def test_attend_queries_of_all_sizes(dev):
    """Rows at the ends of bf16's range: the row's power-of-two scaling keeps their products exact."""
    s = make(dev, B=1, T=4, heads_q=4, heads_kv=1, d=128, page=16, lens=[100], seed=41, scales=False)
    q = s["q"].float()
    q[0, 0, 0] *= 1e30
    q[0, 0, 1] *= 1e-30
    q[0, 1, 2] = 0
    q[0, 1, 3] = -0.0
    q[0, 2, 0, :64] *= 1e-9
    q[0, 2, 1] *= 3e36
    q[0, 3, 1] = 1e-40
    q = q.to(torch.bfloat16)
    check_attend(s, q=q)
    s["q"] = q
    check_attend(s, q=(s["q"].float().clamp(-60000, 60000)).half(), scale=1e-3)


def test_nothing_behind_the_end_is_judged(dev):
    """Bytes of ones (NaN scales) in every position that no row sees, and a table whose other entries
    name no page."""
    s = make(dev, B=3, T=5, heads_q=4, heads_kv=2, d=128, page=64, lens=[70, 0, 129], block=[5, 2, 3], seed=51,
             width=9)
    raw = np.full_like(s["raw"], 255)
    keep = ref.Pool(s["raw"], 64)
    pool = ref.Pool(raw, 64)
    g = torch.Generator().manual_seed(8)
    for i, n in enumerate(s["lens"]):
        if n:
            k = torch.randn((1, n, 2, 128), generator=g)
            pool.raw = ref.write(pool.raw, 64, s["table"][i:i + 1], [0], k, k.flip(1), None, s["ks"], s["vs"])
    s["raw"] = pool.raw
    assert keep.raw.shape == pool.raw.shape
    s["table"][1, 3:] = 2 ** 31 - 1
    out = torch.full((3, 5, 4, 128), 5.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((3, 5, 4), 5.0, device=dev)
    check_attend(s, out=out, lse=lse)
    for i, b in enumerate(s["block"]):
        assert bool((out[i, b:] == 5).all()) and bool((lse[i, b:] == 5).all())


def test_nan_tokens_reach_only_the_rows_that_see_them(dev):
    """A NaN key, a NaN value group and an infinite query element; the rows before the token, and those
    whose window has left it, are as if it were not there."""
    s = make(dev, B=2, T=6, heads_q=4, heads_kv=2, d=128, page=16, lens=[140, 9], seed=61)
    s["k"][0, 3, 0, 17] = float("nan")
    s["v"][0, 4, 1, 40] = float("inf")
    s["v"][1, 2, 0, 3] = float("nan")
    check_attend(s)
    check_attend(s, window=2)
    check_attend(s, causal=False)
    q = s["q"].clone()
    q[0, 1, 2, 5] = float("inf")
    q[1, 0, 0, 5] = float("nan")
    q[1, 4, 3] = float("-inf")
    check_attend(s, q=q)


def test_bad_pages_are_masked_and_bad_lengths_skipped(dev):
    s = make(dev, B=5, T=4, heads_q=2, heads_kv=1, d=64, page=16, lens=[40, 100, 10, 60, 7], seed=71)
    s["table"][0, 1] = -1               # tokens 16..31 of request 0
    s["table"][2, 0] = s["raw"].shape[0]  # all of request 2
    s["lens"][1] = -3
    s["lens"][3] = 16 * s["table"].shape[1] - 3
    dev_, a = s["dev"], device_args(s)
    pages = torch.from_numpy(s["raw"]).to(dev_)
    status = torch.zeros(5, dtype=torch.int32, device=dev_)
    s["cache"].write(s["k"].to(dev_), s["v"].to(dev_), pages, status=status, **a)
    L, P = binding.DEV_BAD_LENGTH, binding.DEV_BAD_PAGE
    assert status.tolist() == [0, L, P, L, 0]
    raw = ref.write(s["raw"], 16, s["table"], s["lens"], s["k"], s["v"], None, s["ks"], s["vs"])
    assert np.array_equal(pages.cpu().numpy(), raw)
    out = torch.full((5, 4, 2, 64), 3.0, dtype=torch.bfloat16, device=dev_)
    lse = torch.full((5, 4, 2), 3.0, device=dev_)
    status.zero_()
    s["cache"].attend(s["q"].to(dev_), pages, out=out, lse=lse, status=status, **a)
    assert status.tolist() == [P, L, P, L, 0]
    compare(s, raw, s["q"], out, lse)
    assert bool((out[2] == 0).all()) and bool(torch.isneginf(lse[2]).all())
    for i in (1, 3):
        assert bool((out[i] == 3).all()) and bool((lse[i] == 3).all())
    status.zero_()
    o = tuple(torch.full((5, 40, 1, 64), 3.0, device=dev_) for _ in range(2))
    s["cache"].read(pages, a["table"], start=on(dev_, [0, -1, 0, 16 * 30, 0]), count=on(dev_, [40, 3, 3, 40, 7]),
                    out=o, status=status)
    assert status.tolist() == [P, L, P, L, 0]
    assert bool((o[0][0, 16:32] == 3).all()) and bool((o[1][2] == 3).all()) and bool((o[0][3] == 3).all())
    assert not bool((o[0][0, 32:40] == 3).any())


def test_attend_long_context_of_one_request(dev):
    """One request split over the whole GPU and joined; the reference runs on the device in fp64."""
    d, hq, hkv, page, n, T = 128, 8, 2, 64, 30011, 6
    rng = np.random.RandomState(0)
    width = (n + T + page - 1) // page
    cache = binding.BlockCache(dev, hq, hkv, d, page, max_batch=1)
    pages = cache.alloc(width + 3)
    table = torch.from_numpy(rng.permutation(width + 3)[:width].astype(np.int32)).to(dev)[None]
    g = torch.Generator(device=dev).manual_seed(3)
    k = torch.randn((1, n + T, hkv, d), generator=g, device=dev, dtype=torch.bfloat16)
    v = torch.randn((1, n + T, hkv, d), generator=g, device=dev, dtype=torch.bfloat16)
    q = torch.randn((1, T, hq, d), generator=g, device=dev, dtype=torch.bfloat16)
    cache.write(k, v, pages, table, torch.zeros(1, dtype=torch.int32, device=dev))
    length = torch.tensor([n], dtype=torch.int32, device=dev)
    kk, vv = cache.read(pages, table, rows=n + T, dtype=torch.float32)
    for window in (0, 20000):
        out, lse = cache.attend(q, pages, table, length, window=window)
        again, lse2 = cache.attend(q, pages, table, length, window=window)
        assert torch.equal(out, again) and torch.equal(lse, lse2)  # same call, same bits
        for h in range(hq):
            x = (q[0, :, h].double() @ kk[0, :, h // 4].double().T) * d ** -0.5
            pos = torch.arange(n + T, device=dev)
            j = n + torch.arange(T, device=dev)[:, None]
            see = (pos <= j) & ((pos > j - window) if window else True)
            x = x.masked_fill(~see, -math.inf)
            p = torch.softmax(x, -1)
            want, a = p @ vv[0, :, h // 4].double(), p @ vv[0, :, h // 4].double().abs()
            size = (q[0, :, h].double().abs() @ kk[0, :, h // 4].double().abs().T).max() * d ** -0.5
            # fp32 sums of a tile's 128 tokens and of the tiles: 128 + 30017 / 128 + parts terms deep
            tol, tol_lse = ref.attend_bounds(want.cpu().numpy(), torch.logsumexp(x, -1).cpu().numpy(),
                                             a.cpu().numpy(), np.full(T, float(size)), 600, d, q.dtype)
            assert np.all(np.abs(ref.to_np(out[0, :, h]) - want.cpu().numpy()) <= tol)
            assert np.all(np.abs(ref.to_np(lse[0, :, h]) - torch.logsumexp(x, -1).cpu().numpy()) <= tol_lse)
    assert cache.errors() == 0


def test_pages_behind_4_gib_and_rows_behind_2_gib(dev):
    """Page offsets and row offsets that pass 32 bits."""
    d, page = 256, 256
    s = make(dev, B=1, T=3, heads_q=2, heads_kv=2, d=d, page=page, lens=[300], seed=81)
    per = s["raw"][0].size
    num = (5 << 30) // per
    pages = torch.empty((num,) + s["raw"].shape[1:], dtype=torch.uint8, device=dev)
    high = {int(p): num - 1 - 7 * e for e, p in enumerate(s["table"][0])}
    for p, to in high.items():
        pages[to] = torch.from_numpy(s["raw"][p]).to(dev)
    a = device_args(s)
    a["table"] = on(dev, [[high[int(p)] for p in s["table"][0]]])
    big = torch.empty(3 * (1 << 29) + 3 * 2 * d, dtype=torch.bfloat16, device=dev)
    k = torch.as_strided(big, (1, 3, 2, d), (8, 1 << 29, d, 1))
    k.copy_(s["k"])
    s["cache"].write(k, s["v"].to(dev), pages, **a)
    k.copy_(s["q"])
    out, lse = s["cache"].attend(k, pages, **a)
    raw = ref.write(s["raw"], page, s["table"], s["lens"], s["k"], s["v"], None, s["ks"], s["vs"])
    for p, to in high.items():
        assert np.array_equal(pages[to].cpu().numpy(), raw[p])
    compare(s, raw, s["q"], out, lse)


def test_empty_calls_do_nothing(dev):
    c = binding.BlockCache(dev, 2, 1, 64, 16, max_batch=4)
    pages = c.alloc(2)
    pages.fill_(3)
    e = torch.zeros((0, 3), dtype=torch.int32, device=dev)
    n = torch.zeros(0, dtype=torch.int32, device=dev)
    k = torch.zeros((0, 2, 1, 64), dtype=torch.bfloat16, device=dev)
    c.write(k, k, pages, e, n)
    out, lse = c.attend(torch.zeros((0, 2, 2, 64), dtype=torch.bfloat16, device=dev), pages, e, n)
    assert out.shape == (0, 2, 2, 64) and lse.shape == (0, 2, 2)
    t = torch.zeros((2, 3), dtype=torch.int32, device=dev)
    n = torch.zeros(2, dtype=torch.int32, device=dev)
    k = torch.zeros((2, 0, 1, 64), dtype=torch.bfloat16, device=dev)
    c.write(k, k, pages, t, n)
    assert c.attend(torch.zeros((2, 0, 2, 64), dtype=torch.bfloat16, device=dev), pages, t, n)[0].numel() == 0
    assert c.read(pages, t, rows=0)[0].shape == (2, 0, 1, 64)
    assert bool((pages == 3).all())


def test_captured_step_replays_with_new_lengths(dev):
    """write + attend in a CUDA graph; cache_len, block_len, the table and the block change between the
    replays."""
    s = make(dev, B=3, T=4, heads_q=4, heads_kv=2, d=64, page=16, lens=[60, 7, 130], block=[4, 4, 4], seed=91)
    a = device_args(s)
    pages = torch.from_numpy(s["raw"]).to(dev)
    k, v, q = s["k"].to(dev), s["v"].to(dev), s["q"].to(dev)
    out = torch.zeros_like(q)
    lse = torch.zeros((3, 4, 4), device=dev)

    def step():
        s["cache"].write(k, v, pages, **a)
        s["cache"].attend(q, pages, out=out, lse=lse, **a)

    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream(dev).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    raw = s["raw"]
    for lens, block in (([60, 7, 130], [4, 4, 4]), ([2, 9, 40], [1, 4, 0]), ([61, 0, 133], [4, 2, 1])):
        s["lens"], s["block"] = lens, block
        a["cache_len"].copy_(on(dev, lens))
        a["block_len"].copy_(on(dev, block))
        pages.copy_(torch.from_numpy(raw))
        graph.replay()
        torch.cuda.synchronize(dev)
        want = ref.write(raw, 16, s["table"], lens, s["k"], s["v"], block, s["ks"], s["vs"])
        assert np.array_equal(pages.cpu().numpy(), want)
        compare(s, want, s["q"], out, lse)
    del graph


def test_two_streams_with_a_context_each(dev):
    s = make(dev, B=4, T=3, heads_q=8, heads_kv=2, d=128, page=16, lens=[300, 11, 800, 64], seed=101)
    a = device_args(s)
    pages = torch.from_numpy(s["raw"]).to(dev)
    s["cache"].write(s["k"].to(dev), s["v"].to(dev), pages, **a)
    q = s["q"].to(dev)
    want, wl = s["cache"].attend(q, pages, **a)
    other = binding.BlockCache(dev, 8, 2, 128, 16, max_batch=4)
    torch.cuda.synchronize(dev)
    streams = [torch.cuda.Stream(dev), torch.cuda.Stream(dev)]
    got = [[], []]
    for _ in range(20):
        for st, c, g in zip(streams, (s["cache"], other), got):
            with torch.cuda.stream(st):
                g.append(c.attend(q, pages, **a))
    torch.cuda.synchronize(dev)
    for g in got:
        for out, lse in g:
            assert torch.equal(out, want) and torch.equal(lse, wl)
    assert s["cache"].errors() == 0 and other.errors() == 0


def test_batches_larger_than_a_block_of_threads(dev):
    """1500 requests: the shares come from a scan in several rounds; many requests have nothing to do."""
    B, T = 1500, 2
    rng = np.random.RandomState(5)
    lens = [int(x) for x in rng.randint(0, 40, size=B)]
    block = [int(x) for x in rng.randint(-1, 4, size=B)]  # clamped to 0..2
    lens[700] = -1
    per = [max(1, (max(n, 0) + T + 15) // 16) for n in lens]
    table = np.full((B, 3), -1, dtype=np.int32)
    ids, at = rng.permutation(sum(per)), 0
    for i, m in enumerate(per):
        table[i, :m] = ids[at:at + m]
        at += m
    cache = binding.BlockCache(dev, 2, 1, 64, 16, max_batch=B)
    pages = cache.alloc(sum(per))
    g = torch.Generator(device=dev).manual_seed(9)
    k = torch.randn((B, 42, 1, 64), generator=g, device=dev)
    v = torch.randn((B, 42, 1, 64), generator=g, device=dev)
    t = on(dev, table)
    cache.write(k, v, pages, t, torch.zeros(B, dtype=torch.int32, device=dev),
                block_len=on(dev, [max(n, 0) + min(max(b, 0), T) for n, b in zip(lens, block)]))
    q = torch.randn((B, T, 2, 64), generator=g, device=dev).half()
    out = torch.full_like(q, 7.0)
    lse = torch.full((B, T, 2), 7.0, device=dev)
    status = torch.zeros(B, dtype=torch.int32, device=dev)
    cache.attend(q, pages, t, on(dev, lens), block_len=on(dev, block), out=out, lse=lse, status=status)
    assert status.nonzero().flatten().tolist() == [700] and int(status[700]) == binding.DEV_BAD_LENGTH
    kk, vv = cache.read(pages, t, rows=42, dtype=torch.float32)
    ok = torch.zeros((B, T), dtype=torch.bool)
    for i in range(B):
        for j in range(min(max(block[i], 0), T) if i != 700 else 0):
            ok[i, j] = True
            n = lens[i] + j + 1
            x = q[i, j].double() @ kk[i, :n, 0].double().T / 8
            p = torch.softmax(x, -1)
            want, a = p @ vv[i, :n, 0].double(), p @ vv[i, :n, 0].double().abs()
            size = (q[i, j].double().abs() @ kk[i, :n, 0].double().abs().T).amax(-1) / 8
            z = torch.logsumexp(x, -1)
            tol, tol_lse = ref.attend_bounds(want.cpu().numpy(), z.cpu().numpy(), a.cpu().numpy(), size.cpu().numpy(), 42,
                                             64, q.dtype)
            assert np.all(np.abs(ref.to_np(out[i, j]) - want.cpu().numpy()) <= tol)
            assert np.all(np.abs(ref.to_np(lse[i, j]) - z.cpu().numpy()) <= tol_lse)
    left = ~ok.to(dev)
    assert bool((out[left] == 7).all()) and bool((lse[left] == 7).all())
    assert cache.errors() == 0


@pytest.mark.parametrize("d,hq,hkv,T", [(128, 32, 1, 5), (64, 1, 1, 150), (256, 8, 2, 21), (128, 3, 3, 65)])
def test_blocks_of_several_row_tiles(dev, d, hq, hkv, T):
    """More query rows than a tile holds: every row tile reads its own span of positions."""
    s = make(dev, B=2, T=T, heads_q=hq, heads_kv=hkv, d=d, page=32, lens=[45, 210], block=[T, T - 2], seed=T)
    check_attend(s)
    check_attend(s, window=50)


def test_a_score_that_leaps_far_past_all_before_it(dev):
    """A key whose score passes the running maximum by thousands of powers of two: the sums so far overflow
    or vanish, and the row is that key's value."""
    d, n = 64, 700
    s = make(dev, B=1, T=1, heads_q=3, heads_kv=1, d=d, page=16, lens=[n], seed=77, scales=False)
    g = torch.Generator().manual_seed(3)
    k = torch.randn((1, n, 1, d), generator=g) * 0.01
    q = torch.randn((1, 1, 3, d), generator=g)
    k[0, 300, 0] = q[0, 0, 0] * 40.0
    k[0, 650, 0] = q[0, 0, 0] * 300.0
    k[0, 450, 0] = q[0, 0, 1] * 8.0
    v = torch.randn((1, n, 1, d), generator=g)
    s["raw"] = ref.write(s["raw"], 16, s["table"], [0], k, v)
    for scale in (0.05, 1.0, 30.0):
        check_attend(s, q=q.to(torch.bfloat16), scale=scale)


def test_outputs_on_the_callers_stream(dev):
    """Outputs that the call makes are filled on the stream that it runs on."""
    s = make(dev, B=2, T=3, heads_q=2, heads_kv=1, d=64, page=16, lens=[50, 3], block=[3, 1], seed=13)
    a = device_args(s)
    pages = torch.from_numpy(s["raw"]).to(dev)
    k, v, q = s["k"].to(dev), s["v"].to(dev), s["q"].to(dev)
    st = torch.cuda.Stream(dev)
    st.wait_stream(torch.cuda.current_stream(dev))
    s["cache"].write(k, v, pages, stream=st, **a)
    out, lse = s["cache"].attend(q, pages, stream=st, **a)
    kk, _ = s["cache"].read(pages, a["table"], rows=4, stream=st)
    st.synchronize()
    raw = ref.write(s["raw"], 16, s["table"], s["lens"], s["k"], s["v"], s["block"], s["ks"], s["vs"])
    compare(s, raw, s["q"], out, lse)
    assert bool((out[1, 1:] == 0).all()) and bool(torch.isneginf(lse[1, 1:]).all())
    assert kk.shape == (2, 4, 1, 64)


@pytest.mark.parametrize("captured", [False, True])
def test_calls_in_a_row_do_not_overtake_one_another(dev, captured):
    """Kernels start while the ones before them drain: inputs that the call before has just written, pages that
    the next call overwrites, a fork and a join of streams, memsets and copies between, all without a wait of
    the host, give the bits of the same calls made one by one."""
    s = make(dev, B=5, T=4, heads_q=8, heads_kv=2, d=64, page=16, lens=[900, 0, 250, 17, 1500], seed=57)
    a = device_args(s)
    start = a["cache_len"].clone()
    raw = torch.from_numpy(s["raw"]).to(dev)
    pages = raw.clone()
    k, v, q = s["k"].to(dev), s["v"].to(dev), s["q"].to(dev)
    kk, qq = torch.empty_like(k), torch.empty_like(q)
    side = torch.cuda.Stream(dev)

    def run(wait):
        main = torch.cuda.current_stream(dev)
        pages.copy_(raw)
        a["cache_len"].copy_(start)
        res = []
        for n in range(4):
            side.wait_stream(main)
            with torch.cuda.stream(side):
                torch.mul(q, 1.0 + n, out=qq)
            torch.mul(k, 2.0 - n, out=kk)
            s["cache"].write(kk, v, pages, **a)
            wait()
            main.wait_stream(side)
            out, lse = s["cache"].attend(qq, pages, **a)
            wait()
            back = s["cache"].read(pages, a["table"], a["cache_len"], rows=4, k_scale=a["k_scale"], v_scale=a["v_scale"])
            wait()
            twice = s["cache"].attend(qq, pages, window=100, **a)
            wait()
            res += [out, lse, back[0], back[1], twice[0], twice[1], out.clone()]
            a["cache_len"].add_(n % 2)  # the next block is written over this one, or one further
        return res + [pages.clone()]

    with torch.cuda.stream(torch.cuda.Stream(dev)):
        want = run(lambda: torch.cuda.synchronize(dev))
        torch.cuda.synchronize(dev)
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = run(lambda: None)
            for _ in range(3):
                graph.replay()
        else:
            for _ in range(3):
                got = run(lambda: None)
        torch.cuda.synchronize(dev)
    for n, (x, y) in enumerate(zip(got, want)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), n
    if captured:
        del graph


@pytest.mark.parametrize("d,hq,hkv,dtype", [(64, 6, 2, torch.bfloat16), (128, 3, 3, torch.float16),
                                            (256, 4, 1, torch.bfloat16)])
def test_a_prompt_as_one_block(dev, d, hq, hkv, dtype):
    """A block of many hundred tokens: dozens of row tiles, most of them cut into several CTAs' shares."""
    s = make(dev, B=2, T=1300, heads_q=hq, heads_kv=hkv, d=d, page=64, lens=[0, 70], block=[1300, 701], dtype=dtype,
             seed=d)
    check_attend(s)
    check_attend(s, window=300)


def test_out_may_be_the_queries(dev):
    """The outputs over the queries: whole segments, cut ones, rows that stay as they were."""
    s = make(dev, B=3, T=6, heads_q=8, heads_kv=2, d=128, page=32, lens=[9000, 40, 0], block=[6, 3, 6], seed=23)
    a = device_args(s)
    pages = torch.from_numpy(s["raw"]).to(dev)
    q = s["q"].to(dev)
    s["cache"].write(s["k"].to(dev), s["v"].to(dev), pages, **a)
    want, wl = s["cache"].attend(q, pages, **a)
    want[1, 3:] = q[1, 3:]
    out, lse = s["cache"].attend(q, pages, out=q, **a)
    assert out is q and torch.equal(q, want) and torch.equal(lse, wl)


def test_two_graphs_of_one_context_in_turn(dev):
    """Graphs share the context's workspace; replayed one behind the other they do not disturb one another."""
    s = make(dev, B=1, T=2, heads_q=8, heads_kv=1, d=128, page=64, lens=[20000], seed=29)
    a = device_args(s)
    pages = torch.from_numpy(s["raw"]).to(dev)
    s["cache"].write(s["k"].to(dev), s["v"].to(dev), pages, **a)
    qs = [s["q"].to(dev), torch.flip(s["q"], (1,)).contiguous().to(dev)]
    want = [s["cache"].attend(q, pages, window=w, **a) for q, w in zip(qs, (0, 5000))]
    outs = [(torch.zeros_like(qs[0]), torch.zeros_like(want[0][1])) for _ in qs]
    torch.cuda.synchronize(dev)
    graphs = []
    for q, w, (out, lse) in zip(qs, (0, 5000), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s["cache"].attend(q, pages, window=w, out=out, lse=lse, **a)
        graphs.append(g)
    for _ in range(10):
        for out, lse in outs:
            out.zero_()
            lse.zero_()
        for g in graphs:
            g.replay()
    torch.cuda.synchronize(dev)
    for (out, lse), (wo, wl) in zip(outs, want):
        assert torch.equal(out, wo) and torch.equal(lse, wl)
    del graphs


def test_gpu_refusals(dev):
    c = binding.BlockCache(dev, 4, 2, 64, 16, max_batch=2)
    pages = c.alloc(4)
    t = torch.zeros((2, 2), dtype=torch.int32, device=dev)
    n = torch.zeros(2, dtype=torch.int32, device=dev)
    k = torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16, device=dev)
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError):
        c.write(k, k[:, :2], pages, t, n)
    with pytest.raises(TypeError):
        c.write(k, k.half(), pages, t, n)
    with pytest.raises(TypeError):
        c.write(k.double(), k.double(), pages, t, n)
    with pytest.raises(ValueError):
        c.write(k[:, :, :1], k[:, :, :1], pages, t, n)
    with pytest.raises(ValueError):
        c.write(k.cpu(), k.cpu(), pages, t, n)
    with pytest.raises(ValueError):
        c.write(k, k, pages, t, None)
    with pytest.raises(ValueError):
        c.write(k, k, pages, t, n[:1])
    with pytest.raises(TypeError):
        c.write(k, k, pages, t.long(), n)
    with pytest.raises(ValueError):
        c.write(k, k, pages[:, :1], t, n)
    with pytest.raises(ValueError):
        c.write(k, k, pages, t.t().contiguous().t(), n)
    with pytest.raises(TypeError):
        c.attend(q.float(), pages, t, n)
    with pytest.raises(ValueError):
        c.attend(q, pages, t, n, out=q[:, :2])
    with pytest.raises(ValueError):
        c.attend(q, pages, t, n, out=q[:, :1].expand(2, 3, 4, 64))
    with pytest.raises(ValueError):
        c.attend(q, pages, t, n, lse=torch.zeros((2, 3, 2), device=dev))
    with pytest.raises(ValueError):
        c.attend(q, pages, t, n, k_scale=torch.ones(3, device=dev))
    with pytest.raises(binding.SpecVerifyError) as e:
        c.attend(q, pages, t, n, window=-1)
    assert e.value.status == binding.SPEC_ERR_INVALID_ARG
    with pytest.raises(binding.SpecVerifyError):
        c.attend(q, pages, t, n, scale=float("nan"))
    flat = torch.zeros(2 * 3 * 4 * 64 + 8, dtype=torch.bfloat16, device=dev)
    with pytest.raises(binding.SpecVerifyError) as e:
        c.attend(flat[1:1 + q.numel()].view(q.shape), pages, t, n)
    assert e.value.status == binding.SPEC_ERR_UNSUPPORTED
    with pytest.raises(binding.SpecVerifyError) as e:
        big = torch.zeros((3, 1, 2, 64), dtype=torch.bfloat16, device=dev)
        c.write(big, big, pages, torch.zeros((3, 1), dtype=torch.int32, device=dev), torch.zeros(3, dtype=torch.int32, device=dev))
    assert e.value.status == binding.SPEC_ERR_INVALID_ARG
    for bad in (dict(head_dim=96), dict(page_size=24), dict(page_size=8), dict(head_dim=512)):
        with pytest.raises(binding.SpecVerifyError) as e:
            binding.BlockCache(dev, **dict(dict(heads_q=4, heads_kv=2, head_dim=64, page_size=16), **bad))
        assert e.value.status == binding.SPEC_ERR_UNSUPPORTED
    with pytest.raises(binding.SpecVerifyError) as e:
        binding.BlockCache(dev, heads_q=5, heads_kv=2, head_dim=64, page_size=16)
    assert e.value.status == binding.SPEC_ERR_INVALID_ARG


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad,high", [(5, 200), (200, 5), (130, 260), (260, 130)])
def test_a_nan_key_far_below_the_maximum_is_not_lost(dev, d, bad, high):
    """A NaN key in one tile, and a score hundreds of powers of two above all others in the next: the first
    tile's sums weigh nothing beside the second's, and are NaN all the same.  Enough requests that a CTA takes
    whole segments (and some that are cut)."""
    B, T, h, n, page = 40, 2, 8, 300, 64
    cache = binding.BlockCache(dev, h, h, d, page, max_batch=B)
    width = (n + T + page - 1) // page
    pages = cache.alloc(B * width)
    table = torch.randperm(B * width, generator=torch.Generator().manual_seed(d)).to(torch.int32).view(B, width).to(dev)
    g = torch.Generator(device=dev).manual_seed(7)
    k = torch.randn((B, n + T, h, d), generator=g, device=dev)
    v = torch.randn((B, n + T, h, d), generator=g, device=dev)
    q = torch.randn((B, T, h, d), generator=g, device=dev).bfloat16()
    k[:, high] = 100.0 * q[:, 0].float().sign()
    k[::2, bad, :, 3] = float("nan")  # every other request
    zero = torch.zeros(B, dtype=torch.int32, device=dev)
    cache.write(k, v, pages, table, zero)
    q[:, 1] = q[:, 0]  # both rows meet the large key
    out, lse = cache.attend(q, pages, table, zero + n, scale=1.0)
    assert bool(out[::2].isnan().all()) and bool(lse[::2].isnan().all())
    assert bool(out[1::2].isfinite().all()) and bool(lse[1::2].isfinite().all())
    assert cache.errors() == 0


@pytest.fixture(scope="module")
def hasty(tmp_path_factory):
    """The library with waits of one try (1.4 us at most) instead of 2^22."""
    return build.build(extra_flags=["-DSV_WAIT_TRIES=1"], out=str(tmp_path_factory.mktemp("hasty") / "libhasty.so"))


@pytest.mark.parametrize("d,hq,hkv,T,lens", [
    (128, 32, 8, 6, [30000, 70, 0, 3000]),  # two softmax sets, cut segments and whole ones
    (64, 32, 8, 12, [30000, 400]),          # one set of two warpgroups
    (256, 48, 8, 4, [20000, 100, 2000]),    # one set of one
    (256, 8, 4, 3, [700] * 40),             # two sets, one K and one O buffer
    (64, 32, 8, 1, [300] * 400),            # more segments a CTA than the ring of plans holds
])
def test_a_wait_that_runs_out_ends_the_launch_and_says_so(dev, hasty, monkeypatch, d, hq, hkv, T, lens):
    """With less patience than the memory's latency, or a segment, needs, the roles leave one after another:
    the call returns, the requests' status and the error word say it, and what runs next is as ever."""
    B, page = len(lens), 64
    width = (max(lens) + T + page - 1) // page
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    table = torch.randperm(B * width, generator=torch.Generator().manual_seed(d)).to(torch.int32).view(B, width).to(dev)
    g = torch.Generator(device=dev).manual_seed(5)
    k = torch.randn((B, max(lens) + T, hkv, d), generator=g, device=dev, dtype=torch.bfloat16)
    q = torch.randn((B, T, hq, d), generator=g, device=dev, dtype=torch.bfloat16)
    with binding.BlockCache(dev, hq, hkv, d, page, max_batch=B) as cache:
        pages = cache.alloc(B * width)
        status = torch.zeros(B, dtype=torch.int32, device=dev)
        cache.write(k, k.flip(1), pages, table, torch.zeros_like(n), block_len=n + T)
        want, wl = cache.attend(q, pages, table, n, status=status)
        assert cache.errors() == 0 and not bool(status.any())
        with monkeypatch.context() as m:
            m.setattr(binding, "LIB_PATH", hasty)
            m.setattr(binding, "_lib", None)
            with binding.BlockCache(dev, hq, hkv, d, page, max_batch=B) as other:
                for _ in range(20):
                    status.zero_()
                    other.attend(q, pages, table, n, status=status)
                    other.attend(q, pages, table, n)
                    torch.cuda.synchronize(dev)
                    assert status.tolist() == [binding.DEV_INTERNAL] * B and other.errors() != 0
        status.zero_()
        out, lse = cache.attend(q, pages, table, n, status=status)
        assert torch.equal(out, want) and torch.equal(lse, wl)
        assert cache.errors() == 0 and not bool(status.any())


@pytest.mark.parametrize("group,T", [(1, 1), (8, 1), (3, 3), (8, 2), (17, 1), (8, 3), (5, 5), (8, 4), (11, 3), (8, 6),
                                     (7, 7), (8, 8)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_every_count_of_rows_that_changes_the_kernel(dev, d, group, T):
    """1, 8, 9, 16, 17, 24, 25, 32, 33, 48, 49 and 64 rows at every width: the first and the last count of rows
    of each instance of the attention (width 256 splits what is above 32)."""
    s = make(dev, B=2, T=T, heads_q=group, heads_kv=1, d=d, page=32, lens=[290, 17], block=[T, (T + 1) // 2],
             seed=group * T + d)
    check_attend(s)
    check_attend(s, window=70)


def crowd(s, copies, **how):
    """The requests of s among `copies` more that read the first one's pages: enough work that a CTA takes
    whole segments, where the few of s alone would be cut into the CTAs' shares."""
    dev, a = s["dev"], device_args(s)
    pages = torch.from_numpy(s["raw"]).to(dev)
    s["cache"].write(s["k"].to(dev), s["v"].to(dev), pages, **a)
    raw = ref.write(s["raw"], s["page"], s["table"], s["lens"], s["k"], s["v"], s["block"], s["ks"], s["vs"])
    B, T, hq, d = s["q"].shape
    first = torch.zeros(B + copies, dtype=torch.long)
    first[copies // 2:copies // 2 + B] = torch.arange(B)  # not at an end
    q = s["q"][first].contiguous()
    hkv = s["k"].shape[2]
    a["table"], a["cache_len"] = a["table"][first.to(dev)].contiguous(), a["cache_len"][first.to(dev)].contiguous()
    if a["block_len"] is not None:
        a["block_len"] = a["block_len"][first.to(dev)].contiguous()
    with binding.BlockCache(dev, hq, hkv, d, s["page"], max_batch=B + copies) as cache:
        out, lse = cache.attend(q.to(dev), pages, **a, **how)
        assert cache.errors() == 0
    mine = slice(copies // 2, copies // 2 + B)
    compare(s, raw, s["q"], out[mine], lse[mine], how.get("causal", True), how.get("window", 0))


@pytest.mark.parametrize("d,hq,hkv,T", [(64, 4, 2, 6), (64, 16, 2, 5), (128, 8, 2, 6), (128, 12, 2, 10),
                                        (256, 4, 2, 4), (256, 12, 2, 4), (256, 8, 2, 8)])
@pytest.mark.parametrize("copies", [0, 120])
def test_nan_tokens_in_every_form_of_the_kernel(dev, d, hq, hkv, T, copies):
    """NaN keys, value groups and queries at every width, with one and two softmax sets, in segments that are
    cut between CTAs (few requests) and in whole ones (many)."""
    s = make(dev, B=2, T=T, heads_q=hq, heads_kv=hkv, d=d, page=16, lens=[300, 9], seed=d + T)
    s["k"][0, 3, 0, 17] = float("nan")
    s["v"][0, 2, 1, 40] = float("inf")
    s["v"][0, 1, 0, d - 1] = float("nan")
    s["v"][1, 2, 0, 3] = float("nan")
    s["v"][1, 3, 1, d // 2] = float("-inf")
    # and one in the context, which whole rows of tiles before and behind it do not see with a window
    ctx_k = torch.randn((1, 1, hkv, d), generator=torch.Generator().manual_seed(1))
    ctx_v = ctx_k.clone()
    ctx_v[0, 0, 1, d - 20] = float("nan")
    s["raw"] = ref.write(s["raw"], 16, s["table"][:1], [150], ctx_k, ctx_v, None, s["ks"], s["vs"])
    q = s["q"]
    q[0, 1, 1, 5] = float("inf")
    q[1, 0, 0, 5] = float("nan")
    crowd(s, copies)
    crowd(s, copies, window=2)
    crowd(s, copies, causal=False, window=152)


@pytest.mark.parametrize("d,hq,hkv,T,lens", [
    (64, 4, 1, 2, [100003]),
    (64, 12, 1, 3, [40007, 0, 25003]),
    (128, 8, 2, 6, [30011]),
    (128, 8, 4, 1, [20000, 129, 20001]),
    (128, 40, 2, 2, [9999, 30000]),
    (256, 4, 2, 2, [12345, 4000]),
    (256, 12, 1, 2, [30011]),
])
@pytest.mark.parametrize("window", [0, 5000])
def test_every_token_counts_once_wherever_a_context_is_cut(dev, d, hq, hkv, T, lens, window):
    """Equal scores and a value of one channel for each token: a row's output is a count of its tokens by
    channel, its lse the logarithm of their number.  All sums are of integers below 2^24, so a token lost or
    counted twice at the border of a tile, a page or a share changes a count of a few hundred by one, and lse
    by 1 / N, far beyond the rounding of the results.  Two assignments of tokens to channels."""
    B, page = len(lens), 64
    width = (max(lens) + T + page - 1) // page
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    table = torch.randperm(B * width, generator=torch.Generator().manual_seed(d)).to(torch.int32).view(B, width).to(dev)
    t = torch.arange(max(lens) + T, device=dev)
    k = torch.randn((1, 1, hkv, d), device=dev, dtype=torch.bfloat16).expand(B, len(t), hkv, d)
    q = torch.zeros((B, T, hq, d), dtype=torch.float16, device=dev)
    with binding.BlockCache(dev, hq, hkv, d, page, max_batch=B) as cache:
        pages = cache.alloc(B * width)
        for channel in (t % d, t // d % d):
            v = (6.0 * torch.nn.functional.one_hot(channel, d)).bfloat16()  # 6 is a code, its scale 1
            cache.write(k, v[None, :, None].expand(B, len(t), hkv, d), pages, table, torch.zeros_like(n), block_len=n + T)
            out, lse = cache.attend(q, pages, table, n, window=window)
            assert cache.errors() == 0
            for i in range(B):
                for j in range(T):
                    end = lens[i] + j + 1
                    first = max(0, end - window) if window else 0
                    want = 6.0 * torch.bincount(channel[first:end], minlength=d).double() / (end - first)
                    # to fp16, and three roundings of the normalisation in fp32
                    off = (out[i, j].double() - want).abs() - want * (2.0 ** -11 + 2.0 ** -20)
                    assert float(off.max()) <= 0, (i, j)
                    # lg2 to 2^-22 absolute, a sum of at most 25 and a product rounded
                    assert float((lse[i, j].double() - math.log(end - first)).abs().max()) <= 2.0 ** -22 + 30 * 2.0 ** -23


@pytest.mark.parametrize("d,hq,T", [(64, 8, 1), (64, 32, 2), (128, 8, 3), (128, 32, 1), (128, 16, 4), (256, 8, 1),
                                    (256, 32, 1)])
def test_a_key_is_found_at_every_border(dev, d, hq, T):
    """Keys with one channel each at the borders of tiles, runs and shares of a long context, and rows that ask
    for one of them: each row's output is that token's value, its lse that score."""
    n, page, block = 30011, 16, hq * T
    rng = np.random.RandomState(d + hq)
    ends = [0, 1, n - 1, n - 2]
    spots = torch.tensor(ends + [128 * e + o for e in rng.permutation(np.arange(1, n // 128))[:2 * d] for o in (-1, 0)],
                         device=dev)
    width = (n + T + page - 1) // page
    table = torch.randperm(width, generator=torch.Generator().manual_seed(d)).to(torch.int32).view(1, width).to(dev)
    length = torch.tensor([n], dtype=torch.int32, device=dev)
    v = torch.randn((1, n + T, 1, d), generator=torch.Generator(device=dev).manual_seed(2), device=dev)
    with binding.BlockCache(dev, hq, 1, d, page, max_batch=1) as cache:
        pages = cache.alloc(width)
        for at in range(0, len(spots) // d * d, d):
            mine = spots[at:at + d]  # one channel each
            k = torch.zeros((1, n + T, 1, d), device=dev)
            k[0, mine, 0, torch.arange(d, device=dev)] = 96.0
            cache.write(k, v, pages, table, torch.zeros_like(length))
            _, vv = cache.read(pages, table, rows=n + T, dtype=torch.float32)
            for c in range(0, d, block):
                ask = (c + torch.arange(block, device=dev)) % d
                q = torch.nn.functional.one_hot(ask, d).view(1, T, hq, d).half().contiguous()
                out, lse = cache.attend(q, pages, table, length, scale=1.0)
                # 30,000 tokens of score 0 weigh exp(-96) each: nothing
                want = vv[0, mine[ask], 0].view(T, hq, d).double()
                assert float(((out[0].double() - want).abs() - want.abs() * (2.0 ** -11 + 2.0 ** -20)).max()) <= 2.0 ** -25
                assert float((lse - 96.0).abs().max()) <= 96 * 2.0 ** -22
        assert cache.errors() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_write_saturates_up_to_the_largest_finite_quotient(dev, dtype):
    """Around the x whose y = x / g is the largest finite number: below it +-6 * 448, above it a NaN group."""
    d, page = 64, 16
    g = np.array([0.25, 0.3], np.float32)
    top = np.float32(np.finfo(np.float32).max)
    x = torch.zeros((1, 16, 2, d), dtype=dtype)
    for h in range(2):
        edge = torch.tensor(float(top) * float(g[h])).to(dtype)
        for j in range(16):  # eight steps of the type on either side
            bits = edge.view(torch.int32 if dtype == torch.float32 else torch.int16) + (j - 8)
            x[0, j, h, 7] = bits.view(dtype)
            x[0, j, h, 8:12] = -bits.view(dtype)
            x[0, j, h, 33] = bits.view(dtype) / 2
            x[0, j, h, 34] = 1e-3
    table = np.zeros((1, 1), np.int32)
    raw = np.zeros((1, 2, 1, 18 * d), np.uint8)
    with binding.BlockCache(dev, 2, 2, d, page, max_batch=1) as c:
        pages = torch.from_numpy(raw).to(dev)
        gd = on(dev, g, torch.float32)
        c.write(x.to(dev), x.flip(1).to(dev), pages, on(dev, table), on(dev, [0]), k_scale=gd, v_scale=gd)
        want = ref.write(raw, page, table, [0], x, x.flip(1), None, g, g)
        assert np.array_equal(pages.cpu().numpy(), want)
        k, _ = c.read(pages, on(dev, table), rows=16, dtype=torch.float32, k_scale=gd)
    assert bool(k[0, 0, :, 7].isfinite().all()) and bool(k[0, 15, :, 7].isnan().all())
    assert bool(k[0, :, :, 32:48].isfinite().all())


def test_a_write_past_the_largest_grid_is_refused(dev):
    c = binding.BlockCache(dev, 1024, 1024, 256, 16, max_batch=1)
    k = torch.zeros((1, 1, 1024, 256), dtype=torch.bfloat16, device=dev).expand(1, 262144, 1024, 256)
    pages = c.alloc(1)
    with pytest.raises(binding.SpecVerifyError) as e:
        c.write(k, k, pages, torch.full((1, 1), -1, dtype=torch.int32, device=dev), on(dev, [0]))
    assert e.value.status == binding.SPEC_ERR_INVALID_ARG
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    few = k[:, :262113]  # the largest that fits: skipped, since the table does not hold it
    c.write(few, few, pages, torch.full((1, 1), -1, dtype=torch.int32, device=dev), on(dev, [0]), status=status)
    assert status.tolist() == [binding.DEV_BAD_LENGTH]


@pytest.mark.parametrize("d,hq,n", [(64, 4, 700), (128, 4, 1000), (128, 40, 650), (256, 4, 517), (256, 24, 900)])
def test_a_cut_row_has_the_lse_of_a_whole_one_where_its_sums_are_exact(dev, d, hq, n):
    """Equal scores and values of whole numbers: every sum is exact in any order, so a request alone (cut into
    the CTAs' shares) and its copies in a crowd (some cut, most whole) give the same lse, bit for bit.  (Outputs
    need not: a whole row's two sums are scaled by 1 / l before they are added, a cut one's behind it, which is
    one rounding of fp32 apart, or a step of the result where that passes a border: 2^-7 of a bf16.)"""
    copies, page, T = 300, 64, 1
    width = (n + T + page - 1) // page
    table = torch.randperm(width, generator=torch.Generator().manual_seed(d)).to(torch.int32).view(1, width).to(dev)
    length = torch.tensor([n], dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(3)
    k = torch.randn((1, n + T, 1, d), generator=g, device=dev)
    v = torch.randint(-2, 3, (1, n + T, 1, d), generator=g, device=dev) * 2.0
    v[..., 0::16] = 6.0  # the scale of each group is 1
    with binding.BlockCache(dev, hq, 1, d, page, max_batch=copies) as cache:
        pages = cache.alloc(width)
        cache.write(k, v, pages, table, torch.zeros_like(length))
        q = torch.zeros((copies, T, hq, d), dtype=torch.bfloat16, device=dev)
        one, one_lse = cache.attend(q[:1], pages, table, length)
        out, lse = cache.attend(q, pages, table.repeat(copies, 1), length.repeat(copies))
        assert torch.equal(lse, one_lse.expand_as(lse))
        off = (out.float() - one.float()).abs() - one.float().abs() * 2.0 ** -7
        assert float(off.max()) <= 6 * 2.0 ** -22  # of the largest value, where the sum is near 0
        assert cache.errors() == 0


def test_windows_wider_than_a_32_bit_number(dev):
    """A window that no position leaves is no window, whatever its size."""
    s = make(dev, B=2, T=3, heads_q=4, heads_kv=2, d=64, page=16, lens=[200, 7], seed=3)
    a = device_args(s)
    pages = torch.from_numpy(s["raw"]).to(dev)
    s["cache"].write(s["k"].to(dev), s["v"].to(dev), pages, **a)
    want, lse = s["cache"].attend(s["q"].to(dev), pages, **a)
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1):
        out, l2 = s["cache"].attend(s["q"].to(dev), pages, window=window, **a)
        assert torch.equal(out, want) and torch.equal(lse, l2), window
    for window in (-1, -2 ** 32 + 5):
        with pytest.raises(binding.SpecVerifyError):
            s["cache"].attend(s["q"].to(dev), pages, window=window, **a)


def test_the_longest_block(dev):
    """65535 query tokens (a row's number and head share 32 bits); one more is refused."""
    T, d, hq, page = 65535, 64, 2, 256
    g = torch.Generator(device=dev).manual_seed(1)
    width = (T + page) // page + 1
    with binding.BlockCache(dev, hq, 1, d, page, max_batch=1) as cache:
        pages = cache.alloc(width)
        table = torch.arange(width, dtype=torch.int32, device=dev).view(1, width)
        n = torch.full((1,), 3, dtype=torch.int32, device=dev)
        k = torch.randn((1, T + 3, 1, d), generator=g, device=dev, dtype=torch.bfloat16)
        v = torch.randn((1, T + 3, 1, d), generator=g, device=dev, dtype=torch.bfloat16)
        q = torch.randn((1, T, hq, d), generator=g, device=dev, dtype=torch.bfloat16)
        cache.write(k, v, pages, table, torch.zeros_like(n))
        kk, vv = cache.read(pages, table, rows=T + 3, dtype=torch.float32)
        out, lse = cache.attend(q, pages, table, n)
        for j in (0, 1, 125, 4095, 32768, 40000, T - 2, T - 1):
            x = q[0, j].double() @ kk[0, :j + 4, 0].double().T / 8
            p = torch.softmax(x, -1)
            want, a = p @ vv[0, :j + 4, 0].double(), p @ vv[0, :j + 4, 0].double().abs()
            size = (q[0, j].double().abs() @ kk[0, :j + 4, 0].double().abs().T).amax(-1) / 8
            z = torch.logsumexp(x, -1)
            # sums are 128 tokens deep in a tile and 512 tiles deep
            tol, tol_lse = ref.attend_bounds(want.cpu().numpy(), z.cpu().numpy(), a.cpu().numpy(), size.cpu().numpy(),
                                             800, d, q.dtype)
            assert np.all(np.abs(ref.to_np(out[0, j]) - want.cpu().numpy()) <= tol), j
            assert np.all(np.abs(ref.to_np(lse[0, j]) - z.cpu().numpy()) <= tol_lse), j
        assert cache.errors() == 0
        with pytest.raises(binding.SpecVerifyError) as e:
            cache.attend(torch.zeros((1, T + 1, hq, d), dtype=torch.bfloat16, device=dev), pages, table, n)
        assert e.value.status == binding.SPEC_ERR_INVALID_ARG
