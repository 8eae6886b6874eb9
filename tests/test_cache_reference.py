"""CPU tests of the 4-bit block cache: its reference, its host-side refusals."""
import ctypes

import numpy as np
import pytest
import torch

import cache_reference as ref
from speculative_decoding_verification_86_b200 import binding, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


def test_e4m3_table_is_torchs():
    b = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.E4M3, b, equal_nan=True)


def test_scales_round_as_torch_rounds_them():
    x = np.float32(np.exp(np.random.RandomState(0).uniform(-9, 6.1, 20000)))
    x = np.concatenate([x, (ref.E4M3[:126] + ref.E4M3[1:127]) / 2]).astype(np.float32)
    x = np.minimum(x, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.nearest_even(x.astype(np.float64), ref.E4M3[:127]), want)


def test_codes_are_the_nearest_values_and_ties_go_to_the_even_code():
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -5.0, 0.0, -0.0, 0.26, 4.9, -6.0])
    c, s = ref.quantise(x, 1.0)
    assert s.tolist() == [0x38]
    assert c.tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 8, 10, 14, 0, 8, 1, 6, 15]
    r = np.random.RandomState(1).randn(50, 16).astype(np.float32)
    c, s = ref.quantise(r, 1.0)
    val = np.where(c & 8, -ref.MAG[c & 7], ref.MAG[c & 7]) * ref.E4M3[s]
    grid = np.concatenate([-ref.MAG, ref.MAG])
    best = np.abs(r[..., None] - grid * ref.E4M3[s][..., None]).min(-1)
    assert np.allclose(np.abs(val - r), best, rtol=0, atol=1e-12)


def test_a_pool_gives_back_what_was_put():
    rng = np.random.RandomState(2)
    raw = rng.randint(0, 256, size=(3, 2, 2, 18 * 64)).astype(np.uint8)
    table = np.array([[2, 0]])
    k = torch.randn((1, 40, 2, 64), generator=torch.Generator().manual_seed(0))
    new = ref.write(raw, 32, table, [11], k, -k)
    pool, old = ref.Pool(new, 32), ref.Pool(raw, 32)
    for t in range(64):
        a, b = pool.get(table[0], t), old.get(table[0], t)
        if 11 <= t < 51:
            assert np.array_equal(a[0], -a[1])
            # half the widest step (2) of a scale that may be rounded up by 2^-4
            x = k[0, t - 11].double().numpy().reshape(2, 4, 16)
            off = np.abs(a[0].reshape(2, 4, 16) - x)
            assert np.all(off <= np.abs(x).max(-1, keepdims=True) / 6 * (1 + 2.0 ** -4))
        else:
            assert np.array_equal(a[0], b[0], equal_nan=True) and np.array_equal(a[1], b[1], equal_nan=True)
    assert np.array_equal(new[1], raw[1])


def test_plain_forms_of_the_measured_cases_agree_with_the_reference():
    """perf/operators.py computes the format with torch operations; its bytes are the reference's."""
    from perf import operators as ops
    x = torch.randn((2, 3, 16, 128), generator=torch.Generator().manual_seed(4)) * 3
    g = torch.tensor([0.01, 0.3, 1.0])
    c, s = ops._quantise(x.transpose(1, 2), g)
    packed = ops._pack(c.transpose(1, 2), s.transpose(1, 2), c.transpose(1, 2), s.transpose(1, 2))
    raw = np.zeros((2, 3, 1, 18 * 128), dtype=np.uint8)
    table = np.array([[0], [1]])
    want = ref.write(raw, 16, table, [0, 0], x.transpose(1, 2), x.transpose(1, 2), None, g.numpy(), g.numpy())
    assert np.array_equal(packed.numpy()[:, :, None], want)
    k, v = ops._unpack(packed[:1], 128)
    kk, vv = ref.Pool(want, 16).get(table[0], 5)
    assert np.array_equal(k[5].double().numpy(), kk) and np.array_equal(v[5].double().numpy(), vv)


def test_page_bytes(L):
    assert binding.BlockCache.bytes_per_page(8, 128, 64) == 8 * 64 * 128 * 2 * 9 // 16
    assert binding.BlockCache.bytes_per_page(1, 64, 16) == 18 * 64
    n = ctypes.c_size_t(5)
    assert L.spec_cache_page_bytes(8, 96, 64, ctypes.byref(n)) == binding.SPEC_ERR_UNSUPPORTED and n.value == 0
    assert L.spec_cache_page_bytes(8, 128, 48, ctypes.byref(n)) == binding.SPEC_ERR_UNSUPPORTED
    assert L.spec_cache_page_bytes(0, 128, 64, ctypes.byref(n)) == binding.SPEC_ERR_UNSUPPORTED
    assert L.spec_cache_page_bytes(8, 128, 64, None) == binding.SPEC_ERR_INVALID_ARG


def test_null_cache_context_and_bad_geometry_are_rejected(L):
    inv = binding.SPEC_ERR_INVALID_ARG
    assert L.spec_cache_destroy(None) == binding.SPEC_OK
    assert L.spec_cache_errors(None, None) == inv
    assert L.spec_cache_write(None, None, None, None, 1, None, None, 1, 1, None, None) == inv
    assert L.spec_cache_read(None, None, None, None, 1, 1, 1, None, None, None, None) == inv
    assert L.spec_cache_attend(None, None, None, 1, None, None, 1, 1, 1.0, 1, 0, None, None, None, None) == inv
    h = ctypes.c_void_p()
    init = L.spec_cache_init
    assert init(None, 0, 1, 8, 8, 128, 64) == inv
    assert init(ctypes.byref(h), 0, 0, 8, 8, 128, 64) == inv
    assert init(ctypes.byref(h), 0, 65536, 8, 8, 128, 64) == inv
    assert init(ctypes.byref(h), 0, 1, 9, 8, 128, 64) == inv
    assert init(ctypes.byref(h), 0, 1, 4, 8, 128, 64) == inv
    assert init(ctypes.byref(h), 0, 1, 8, 8, 80, 64) == binding.SPEC_ERR_UNSUPPORTED
    assert init(ctypes.byref(h), 0, 1, 8, 8, 128, 100) == binding.SPEC_ERR_UNSUPPORTED
    assert not h.value


def test_cache_needs_a_cuda_device():
    with pytest.raises(ValueError):
        binding.BlockCache("cpu", 8, 8, 128, 64)


def test_values_that_overflow_behind_the_calibration_scale_are_nan():
    """y = x / g decides: the largest finite y saturates, one that overflows makes the group NaN."""
    big = np.float32(3e38)
    x = np.zeros(16, np.float32)
    x[3], x[4] = -big, 1.0
    c, s = ref.quantise(x, 1.0)
    assert s.tolist() == [0x7e] and c[3] == 15 and c[4] == 0  # -6 * 448
    c, s = ref.quantise(x, 0.5)
    assert s.tolist() == [0x7f] and not c.any()
    x[3] = np.inf
    assert ref.quantise(x, 4.0)[1].tolist() == [0x7f]
