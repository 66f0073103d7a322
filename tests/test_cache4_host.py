"""Host checks of the 4-bit caches and the windowed attention (no GPU): every
entry point of the two headers is exported, invalid calls are refused with the
documented status before any CUDA call, and the oracle's format holds by brute
force."""
import ctypes
import itertools
import os
import re
import subprocess

import numpy as np
import pytest

import sparse_decode_attention_basiskv_b200 as bkv
from oracle import span_oracle as SO

FAKE = 0x10000
BIG = 1 << 40


def _dims(**kw):
    base = dict(B=2, Hq=8, Hkv=2, d=128, hidden=256, r_v=64, r_k=32, page_size=16,
                max_pages_per_seq=64, num_phys_pages=128)
    base.update(kw)
    return bkv.Dims(**base)


@pytest.fixture(scope="module")
def lib():
    return bkv.load_library()


def test_headers_are_exported(lib):
    root = os.path.dirname(bkv.HEADER)
    names = []
    for f in ("basiskv_cache4.h", "basiskv_window.h"):
        with open(os.path.join(root, f)) as h:
            names += re.findall(r"BASISKV_API\s+[\w\s\*]*?\b(basiskv_\w+)\s*\(", h.read())
    assert len(names) == 7
    out = subprocess.run(["nm", "-D", "--defined-only", bkv.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    assert set(names) <= exported
    assert set(names) <= set(bkv._SIGNATURES)


def test_cache4_bytes(lib):
    d = _dims()
    for w in (128, 64, 32):
        assert bkv.cache4_bytes(d, w) == 128 * 2 * 16 * w * 9 // 16
    assert bkv.cache4_bytes(d, 96) == 0                       # not a width of these dims
    assert bkv.cache4_bytes(_dims(page_size=8), 128) == 0     # no 4-bit pages of 8
    assert bkv.cache4_bytes(_dims(cache_fp8=1), 128) == 0     # one element type


CACHE4_BAD_DIMS = [
    (dict(page_size=8), bkv.ERR_UNSUPPORTED_SHAPE),
    (dict(cache_fp8=1), bkv.ERR_INVALID_ARG),
    (dict(route_r_v=16, route_r_k=16), bkv.ERR_UNSUPPORTED_SHAPE),
    (dict(d=80), bkv.ERR_UNSUPPORTED_SHAPE),
    (dict(B=0), bkv.ERR_INVALID_ARG),
    (dict(Hq=6), bkv.ERR_UNSUPPORTED_SHAPE),
]


def _calls(lib, d):
    p = ctypes.byref(d)
    return {
        "write": (lib.basiskv_cache4_write, [p, FAKE, FAKE, FAKE, 4, FAKE, FAKE, FAKE, FAKE, FAKE,
                                             FAKE, None]),
        "read": (lib.basiskv_cache4_read, [p, FAKE, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                           FAKE, None]),
        "route": (lib.basiskv_cache4_route, [p, FAKE, FAKE, 100, FAKE, FAKE, FAKE, FAKE, FAKE, 8,
                                             FAKE, FAKE, FAKE, BIG, None]),
        "attend": (lib.basiskv_cache4_attend, [p, FAKE, FAKE, 100, FAKE, FAKE, FAKE, FAKE, 8,
                                               FAKE, FAKE, BIG, None]),
        "window": (lib.basiskv_attend_window, [p, FAKE, 4, FAKE, 100, FAKE, FAKE, FAKE, 1, 4, 16,
                                               FAKE, FAKE, BIG, None]),
    }


@pytest.mark.parametrize("bad,status", CACHE4_BAD_DIMS)
@pytest.mark.parametrize("name", ["write", "read", "route", "attend", "window"])
def test_bad_dims_are_refused(lib, name, bad, status):
    f, args = _calls(lib, _dims(**bad))[name]
    assert f(*args) == status


@pytest.mark.parametrize("name,i,value,status", [
    ("write", 1, None, bkv.ERR_INVALID_ARG), ("write", 1, FAKE + 8, bkv.ERR_INVALID_ARG),
    ("write", 2, None, bkv.ERR_INVALID_ARG), ("write", 3, None, bkv.ERR_INVALID_ARG),
    ("write", 4, 0, bkv.ERR_INVALID_ARG), ("write", 4, 64 * 16 + 1, bkv.ERR_INVALID_ARG),
    ("write", 5, None, bkv.ERR_INVALID_ARG), ("write", 6, FAKE + 1, bkv.ERR_INVALID_ARG),
    ("write", 7, FAKE + 2, bkv.ERR_INVALID_ARG), ("write", 8, FAKE + 8, bkv.ERR_INVALID_ARG),
    ("write", 10, None, bkv.ERR_INVALID_ARG),
    ("read", 1, None, bkv.ERR_INVALID_ARG), ("read", 2, 0, bkv.ERR_INVALID_ARG),
    ("read", 3, None, bkv.ERR_INVALID_ARG), ("read", 5, None, bkv.ERR_INVALID_ARG),
    ("read", 8, None, bkv.ERR_INVALID_ARG), ("read", 9, FAKE + 8, bkv.ERR_INVALID_ARG),
    ("route", 1, None, bkv.ERR_INVALID_ARG), ("route", 3, 0, bkv.ERR_INVALID_ARG),
    ("route", 3, 64 * 16 + 1, bkv.ERR_INVALID_ARG), ("route", 9, 1, bkv.ERR_INVALID_ARG),
    ("route", 7, None, bkv.ERR_INVALID_ARG), ("route", 10, FAKE + 1, bkv.ERR_INVALID_ARG),
    ("route", 12, FAKE + 16, bkv.ERR_INVALID_ARG),
    ("route", 13, 64, bkv.ERR_WORKSPACE_TOO_SMALL),
    ("attend", 5, None, bkv.ERR_INVALID_ARG), ("attend", 7, None, bkv.ERR_INVALID_ARG),
    ("attend", 8, 1, bkv.ERR_INVALID_ARG), ("attend", 9, FAKE + 8, bkv.ERR_INVALID_ARG),
    ("attend", 11, 64, bkv.ERR_WORKSPACE_TOO_SMALL),
    ("window", 1, None, bkv.ERR_INVALID_ARG), ("window", 2, 0, bkv.ERR_INVALID_ARG),
    ("window", 2, 64 * 16 + 1, bkv.ERR_INVALID_ARG), ("window", 4, 0, bkv.ERR_INVALID_ARG),
    ("window", 4, 64 * 16 + 1, bkv.ERR_INVALID_ARG), ("window", 6, FAKE + 8, bkv.ERR_INVALID_ARG),
    ("window", 8, 2, bkv.ERR_INVALID_ARG), ("window", 9, -1, bkv.ERR_INVALID_ARG),
    ("window", 10, -1, bkv.ERR_INVALID_ARG), ("window", 11, None, bkv.ERR_INVALID_ARG),
    ("window", 12, FAKE + 16, bkv.ERR_INVALID_ARG),
    ("window", 13, 64, bkv.ERR_WORKSPACE_TOO_SMALL),
])
def test_bad_arguments_are_refused(lib, name, i, value, status):
    f, args = _calls(lib, _dims())[name]
    args[i] = value
    assert f(*args) == status


def test_route_needs_an_output_and_read_a_cache(lib):
    f, args = _calls(lib, _dims())["route"]
    args[10] = args[11] = None
    assert f(*args) == bkv.ERR_INVALID_ARG
    f, args = _calls(lib, _dims())["read"]
    for i in (5, 6, 7, 8, 9, 10):
        args[i] = None
    assert f(*args) == bkv.ERR_INVALID_ARG


def test_window_workspace_size(lib):
    d = _dims()
    n = bkv.window_workspace_size(d, 1, 1000, 4, 100)
    assert n > 0 and n % 256 == 0
    assert bkv.window_workspace_size(d, 0, 1000, 4, 100) == 0
    assert bkv.window_workspace_size(d, 1, 64 * 16 + 1, 4, 100) == 0
    assert bkv.window_workspace_size(d, 1, 1000, -1, 100) == 0
    assert bkv.window_workspace_size(d, 1, 1000, 4, -1) == 0
    # page and router limits of the other entry points do not apply here
    assert bkv.window_workspace_size(_dims(page_size=8), 3, 400, 0, 0) > 0
    assert bkv.window_workspace_size(_dims(cache_fp8=1, Hq=2, page_size=8, r_k=16), 300, 400, 0,
                                     0) > 0
    assert bkv.window_workspace_size(_dims(cache_fp8=2), 1, 400, 0, 0) == 0
    # the scratch does not grow with the context
    assert bkv.window_workspace_size(d, 1, 1000, 0, 0) == bkv.window_workspace_size(d, 1, 100, 0, 0)


def test_scale_and_code_by_brute_force():
    """Every positive bf16 magnitude as a block's largest: the byte is the
    nearest representable number to amax / 6 (ties to even), and every code the
    nearest to x / scale, by search over all of them."""
    bits = np.arange(1, 0x7F80, 37, dtype=np.uint32)
    x = (bits << 16).view(np.float32).astype(np.float64)
    grid = SO.scale_value(np.arange(SO.MAX_SCALE_BYTE + 1))
    assert np.all(np.diff(grid) > 0) and grid[-1] == 10240.0
    for v in x[::7]:
        blk = np.zeros((1, 16))
        blk[0, 3] = -v
        blk[0, 4] = v / 3
        codes, byte = SO.quantise(blk)
        dist = np.abs(grid - v / 6)
        best = np.flatnonzero(dist == dist.min())
        assert byte[0, 0] in best and (len(best) == 1 or byte[0, 0] % 2 == 0)
        s = grid[byte[0, 0]]
        for col in (3, 4):
            if s == 0:
                assert codes[0, col] == 0
                continue
            d = np.abs(SO.E2M1 - abs(blk[0, col]) / s)
            best = np.flatnonzero(d == d.min())
            assert (codes[0, col] & 7) in best
            assert len(best) == 1 or (codes[0, col] & 1) == 0


def test_values_are_bf16_and_f16():
    byte = np.arange(SO.MAX_SCALE_BYTE + 1)
    v = SO.scale_value(byte)[:, None] * SO.E2M1[None]
    import torch
    t = torch.from_numpy(v)
    assert torch.equal(t.to(torch.bfloat16).double(), t)
    assert torch.equal(t.to(torch.float16).double(), t)
    # the byte is the top of a half
    h = torch.from_numpy((byte << 7).astype(np.int16)).view(torch.float16).double()
    assert torch.equal(h, torch.from_numpy(SO.scale_value(byte)))


def test_round4_is_idempotent_and_tiles_round_trip():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((16, 96)) * np.exp(rng.standard_normal((16, 1)) * 3)
    r = SO.round4(x)
    np.testing.assert_array_equal(SO.unpack_tile(SO.pack_tile(x), 16, 96), r)
    # the largest magnitude may round down (a saturated code), so the second
    # rounding sees the same or a smaller block; its codes are values already
    np.testing.assert_array_equal(SO.round4(r), SO.round4(SO.round4(r)))
    assert np.abs(r - x).max() <= np.abs(x).max() / 6 * (1 + 1 / 16) + 1e-12


def test_window_mask_by_definition():
    for L, n, W, s in itertools.product((1, 5, 9), (1, 4, 11), (0, 1, 3, 20), (0, 2)):
        m = SO.window_mask(L, n, W, s)
        for j, t in itertools.product(range(n), range(L)):
            p = L - n + j
            assert m[j, t] == (t <= p and (W == 0 or t > p - W or t < s))


def test_mix_equals_a_plain_softmax():
    rng = np.random.default_rng(1)
    q, K, Z = rng.standard_normal((3, 8)), rng.standard_normal((5, 8)), rng.standard_normal((5, 4))
    see = np.array([[1, 1, 0, 0, 0], [0, 0, 0, 0, 0], [1, 1, 1, 1, 1]], dtype=bool)
    a = SO.mix(q, K, Z, see)
    assert np.all(a[1] == 0)
    w = np.exp(K @ q[2] / np.sqrt(8))
    np.testing.assert_allclose(a[2], w @ Z / w.sum(), rtol=1e-12)
    w = np.exp(K[:2] @ q[0] / np.sqrt(8))
    np.testing.assert_allclose(a[0], w @ Z[:2] / w.sum(), rtol=1e-12)


def test_binding_refuses_tensors_elsewhere(monkeypatch):
    """Tensors in host memory, or on another device than the current one, never
    reach the library."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(bkv, "load_library", lambda *a: pytest.fail("the library was called"))
    monkeypatch.setattr(bkv, "_lib", None)
    t, d = torch.zeros(4), _dims()
    for call in (
            lambda: bkv.basiskv_cache4_write(d, t, t, t, 1, t, t, t, t, t, t),
            lambda: bkv.basiskv_cache4_write(d, t, t, None, 1, t, None, t, t, t, None),
            lambda: bkv.basiskv_cache4_read(d, t, 1, t, t, t, t, t, t, t, t),
            lambda: bkv.basiskv_cache4_route(d, t, t, 9, t, t, t, t, t, 2, t, t, t),
            lambda: bkv.basiskv_cache4_attend(d, t, t, 9, t, t, t, t, 2, t, t),
            lambda: bkv.basiskv_attend_window(d, t, 1, t, 9, t, t, t, 0, 0, t, t)):
        with pytest.raises(ValueError, match="current device"):
            call()

    class Elsewhere:  # a tensor of a second GPU
        shape, device = (4,), "cuda:1"
        get_device = staticmethod(lambda: 1)

    with pytest.raises(ValueError, match="cuda:1"):
        bkv._here(None, None, Elsewhere())


def test_window_workspace_is_bounded(lib):
    """Prompts: at most four runs an SM (148 of them here, where no GPU is found), and
    none where the split would gain less than its join costs."""
    sms, worst = 148, 0
    for r_v, B, Hq, n in itertools.product((64, 128), (1, 2, 3, 4, 5, 7, 9, 16), (8, 32, 64),
                                           (40, 130, 200, 257, 1000)):
        for bound in (400, 4096, 34000, 37000, 131072, 1 << 20):
            d = _dims(B=B, Hq=Hq, Hkv=8, r_v=r_v, page_size=32, max_pages_per_seq=1 << 15,
                      num_phys_pages=1 << 16)
            for window in (0, 4096):
                size = bkv.window_workspace_size(d, n, bound, 4, window)
                assert 256 <= size <= 4 * sms * 256 * (r_v + 2) * 4 + 256
                worst = max(worst, size)
    assert worst > 2 * sms * 256 * 66 * 4  # splits are taken
    for r_v in (64, 128):
        d = _dims(B=4, Hq=32, Hkv=8, r_v=r_v, max_pages_per_seq=4096, num_phys_pages=1 << 15)
        assert {bkv.window_workspace_size(d, 200, x, 0, 0) for x in (34000, 37000, 60000)} == {256}
