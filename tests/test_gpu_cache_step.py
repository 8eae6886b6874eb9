"""The cache's entry points as a serving step uses them: verified lengths, the block into the cache, its
attention, the shared head with verification, the accepted tokens kept."""
import numpy as np
import pytest
import torch

import cache_reference as ref
from test_gpu_cache import compare
from speculative_decoding_verification_86_b200 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16])
def test_three_steps_from_lengths_to_the_next_context(cuda_device, dtype):
    dev = cuda_device
    B, k, hq, hkv, d, page, V, H = 5, 3, 4, 2, 64, 16, 2000, 256
    T = k + 1
    g = torch.Generator(device=dev).manual_seed(17)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev).to(dtype)

    lens = np.array([70, 0, 15, 33, 128], dtype=np.int32)
    width = 12
    table = torch.randperm(B * width, generator=g, device=dev).to(torch.int32).view(B, width)
    cache = binding.BlockCache(dev, hq, hkv, d, page, max_batch=B)
    pages = cache.alloc(B * width)
    pages.fill_(255)  # fresh pages may hold anything
    ks, vs = torch.rand(hkv, generator=g, device=dev) + 0.01, torch.rand(hkv, generator=g, device=dev) + 0.01
    scales = dict(k_scale=ks, v_scale=vs)
    cache_len = torch.from_numpy(lens.copy()).to(dev)
    raw = pages.cpu().numpy()
    tn, ksn, vsn = table.cpu().numpy(), ks.cpu().numpy(), vs.cpu().numpy()

    def write(pos, kk, vv, count=None):
        """The library's write and the reference's, on both copies of the cache."""
        nonlocal raw
        cache.write(kk, vv, pages, table, pos, block_len=count, **scales)
        raw = ref.write(raw, page, tn, pos.cpu().numpy(), kk, vv, None if count is None else count.cpu().numpy(), ksn,
                        vsn)
        assert np.array_equal(pages.cpu().numpy(), raw)

    write(torch.zeros_like(cache_len), normal(B, 128, hkv, d), normal(B, 128, hkv, d), cache_len)  # prompts
    ver = binding.SpecVerifier(dev, max_batch=B, max_k=k, max_vocab=V, mode="dense")
    lm = binding.LmHeadVerifier(ver, max_hidden=H)
    head = (torch.randn((V, H), generator=g, device=dev) / 4).to(dtype)
    w = normal(H)
    kept = 0
    for step in range(3):
        tokens = torch.randint(0, V, (B, k), generator=g, device=dev, dtype=torch.int32)
        draft = normal(B, k, H)
        conf = dict(hidden=draft, w=w, bias=4.0, threshold=0.2)
        L, _ = ver.lengths(conf, k)
        count = L + 1
        write(cache_len, normal(B, T, hkv, d), normal(B, T, hkv, d), count)
        q = normal(B, T, hq, d)
        out, lse = cache.attend(q, pages, table, cache_len, block_len=count, **scales)
        s = dict(page=page, table=tn, lens=cache_len.cpu().numpy().tolist(), block=count.cpu().numpy(), ks=ksn, vs=vsn)
        compare(s, raw, q.cpu(), out, lse)
        hidden = out.view(B, T, H)
        # drafts that agree with the target at some places
        agree = lm.logits(hidden[:, :k].contiguous(), head).argmax(-1).to(torch.int32)
        tokens = torch.where(torch.rand((B, k), generator=g, device=dev) < 0.7, agree, tokens).contiguous()
        t0 = torch.zeros(B, device=dev)
        o = lm.verify(hidden, None, head, tokens, verify_len=L, temperature=t0, seed=step)
        plain = ver.run(lm.logits(hidden, head), None, tokens, verify_len=L, temperature=t0, seed=step)
        assert torch.equal(o["accepted"], plain["accepted"]) and torch.equal(o["tokens"], plain["tokens"])
        assert bool((o["accepted"] >= 0).all()) and bool((o["accepted"] <= L).all())
        cache_len = cache_len + o["accepted"] + 1
        kept += int(o["accepted"].sum())
    assert kept > 0
    # what is kept reads back as the reference reads it
    rows = int(cache_len.max())
    kk, vv = cache.read(pages, table, count=cache_len, rows=rows, dtype=torch.float32, **scales)
    pool = ref.Pool(raw, page)
    for i in range(B):
        for t in range(int(cache_len[i])):
            a, b = pool.get(tn[i], t)
            assert np.array_equal(kk[i, t].cpu().numpy(), a.astype(np.float32) * ksn[:, None])
            assert np.array_equal(vv[i, t].cpu().numpy(), b.astype(np.float32) * vsn[:, None])
    assert cache.errors() == 0 and lm.errors() == 0
    cache.close()
    lm.close()
    ver.close()
