"""Host-side refusals of the 8-bit append, the read-back and the page-selecting decode: every bad argument
is answered before anything is enqueued. The calls carry fake device addresses, so the module runs only
where no GPU is visible."""
import ctypes

import pytest
import torch

from mla_compressed_latent_b200 import _lib as L
from mla_compressed_latent_b200 import build as B
from mla_compressed_latent_b200 import ops

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake device pointers: host-side checks run where no GPU is visible")

GOOD, ODD, BIG_WS = 4096, 4100, 1 << 50


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def _dims(**kw):
    d = dict(H=128, D=128, d_r=64, d_c=512, d_v=128, g=0, page_size=64, sm_scale=0.0, rms_eps=1e-6, rope_base=10000.0)
    d.update(kw)
    return L.MlaDims(*[d[f] for f, _ in L.MlaDims._fields_])


def _lc(**kw):
    c = dict(latent=GOOD, latent_stride=576, rope=GOOD + 1024, rope_stride=576, num_pages=10)
    c.update(kw)
    return L.MlaLatentCache(c["latent"], c["latent_stride"], c["rope"], c["rope_stride"], c["num_pages"])


def _fc(**kw):
    c = dict(codes=GOOD, code_stride=512, scales=GOOD, rope=GOOD + 1024, rope_stride=576, num_pages=10)
    c.update(kw)
    return L.MlaLatentCacheFp8(c["codes"], c["code_stride"], c["scales"], c["rope"], c["rope_stride"], c["num_pages"])


# name -> (arguments after dims; "P" a device pointer, "LC"/"FC" a cache), required pointers, sizes that must be
# positive, workspace index, optional pointers, has a dtype as its first argument
CALLS = {
    "mla_append_cache_fp8": ([1, 64, 1, "P", 7168, "P", "P", "P", "P", 64, "FC", "P", BIG_WS, None],
                             [3, 5, 7, 8], [1, 2, 4, 9], 11, [6]),
    "mla_read_latent_fp8": ([1, 64, "FC", "P", 64, "P", "P", 1000, "P", 576, None], [3, 6, 8], [1, 4, 7], None, [5]),
    "mla_update_page_keys": ([1, 64, 1, "LC", "P", 64, "P", "P", 576, None], [4, 6, 7], [1, 2, 5], None, []),
    "mla_update_page_keys_fp8": ([1, 64, 1, "FC", "P", 64, "P", "P", 576, None], [4, 6, 7], [1, 2, 5], None, []),
    "mla_score_pages": ([1, 64, 1, "P", "P", 576, 10, "P", 64, "P", "P", "P", BIG_WS, None], [3, 4, 7, 9, 10],
                        [1, 2, 6, 8], None, [11]),
    "mla_select_pages": ([64, 1, "P", 64, "P", 16, 1, 2, "P", "P", None], [2, 4, 8, 9], [0, 1, 3, 5], None, []),
    "mla_decode_absorbed_sparse": ([1, 64, 1, "P", "LC", "P", 64, "P", "P", "P", 16, "P", "P", "P", BIG_WS, None],
                                   [3, 5, 7, 8, 9, 11, 12], [1, 2, 6, 10], 13, []),
    "mla_decode_absorbed_sparse_fp8": ([1, 64, 1, "P", "FC", "P", 64, "P", "P", "P", 16, "P", "P", "P", BIG_WS, None],
                                       [3, 5, 7, 8, 9, 11, 12], [1, 2, 6, 10], 13, []),
}


def _call(lib, name, args, dims=None, lc=None, fc=None):
    conv = []
    for a in args:
        if a == "LC":
            conv.append(ctypes.byref(lc or _lc()))
        elif a == "FC":
            conv.append(ctypes.byref(fc or _fc()))
        elif a == "P":
            conv.append(GOOD)
        else:
            conv.append(a)
    return getattr(lib, name)(ctypes.byref(dims or _dims()), *conv)


def _cases():
    for name, (args, ptrs, sizes, ws, optional) in CALLS.items():
        for i in ptrs:
            yield name, i, None, L.MLA_ERR_INVALID_ARG
            yield name, i, ODD, L.MLA_ERR_INVALID_ARG
        for i in optional:
            yield name, i, ODD, L.MLA_ERR_INVALID_ARG
        for i in sizes:
            yield name, i, 0, L.MLA_ERR_INVALID_ARG
            yield name, i, -3, L.MLA_ERR_INVALID_ARG
        if ws is not None:
            yield name, ws, None, L.MLA_ERR_WORKSPACE
            yield name, ws + 1, 16, L.MLA_ERR_WORKSPACE
            yield name, ws, ODD, L.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("name,i,bad,want", list(_cases()), ids=lambda v: str(v))
def test_one_bad_argument_is_rejected(lib, name, i, bad, want):
    args = list(CALLS[name][0])
    args[i] = bad
    assert _call(lib, name, args) == want


@pytest.mark.parametrize("name", list(CALLS))
def test_bad_dims_dtype_and_token_counts_are_rejected(lib, name):
    args = CALLS[name][0]
    for bad in (_dims(H=0), _dims(d_c=-1), _dims(page_size=32), _dims(sm_scale=-1.0), _dims(sm_scale=float("nan"))):
        assert _call(lib, name, args, dims=bad) == L.MLA_ERR_INVALID_ARG
    if name != "mla_select_pages":
        assert _call(lib, name, [7] + args[1:]) == L.MLA_ERR_INVALID_ARG
    if name == "mla_read_latent_fp8":
        return
    at = 0 if name == "mla_select_pages" else 1
    big = list(args)
    big[at], big[at + 1] = 1 << 16, 1 << 16
    if "page_keys" in name:   # its grid: sequences times the pages that s_q positions touch
        big[at], big[at + 1], big[5] = 1 << 20, 1 << 20, 1 << 20
    assert _call(lib, name, big) == L.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("name", [n for n, v in CALLS.items() if "FC" in v[0]])
@pytest.mark.parametrize("field,value", [("codes", 0), ("scales", 0), ("rope", 0), ("codes", ODD), ("scales", ODD),
                                         ("code_stride", 500), ("code_stride", 520), ("rope_stride", 63),
                                         ("num_pages", 0)])
def test_bad_fp8_cache_is_rejected(lib, name, field, value):
    assert _call(lib, name, CALLS[name][0], fc=_fc(**{field: value})) == L.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("name", [n for n, v in CALLS.items() if "LC" in v[0]])
@pytest.mark.parametrize("field,value", [("latent", 0), ("rope", 0), ("latent", ODD), ("latent_stride", 577),
                                         ("num_pages", 0)])
def test_bad_latent_cache_is_rejected(lib, name, field, value):
    assert _call(lib, name, CALLS[name][0], lc=_lc(**{field: value})) == L.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["mla_append_cache_fp8", "mla_read_latent_fp8", "mla_update_page_keys_fp8"])
def test_codes_come_in_whole_16_value_rows(lib, name):
    args = list(CALLS[name][0])
    for i, a in enumerate(args):
        if a == 576:
            args[i] = 640
    assert _call(lib, name, args, dims=_dims(d_c=520), fc=_fc(code_stride=528)) == L.MLA_ERR_UNSUPPORTED


def test_selection_bounds(lib):
    args = list(CALLS["mla_select_pages"][0])
    for first, recent in [(-1, 1), (1, -1), (15, 2), (1 << 30, 1 << 30)]:
        bad = list(args)
        bad[6], bad[7] = first, recent
        assert _call(lib, "mla_select_pages", bad) == L.MLA_ERR_INVALID_ARG


def test_row_strides_are_checked(lib):
    for name, i in [("mla_read_latent_fp8", 9), ("mla_update_page_keys", 8), ("mla_score_pages", 5)]:
        for bad in (575, 577, 0, -576):
            args = list(CALLS[name][0])
            args[i] = bad
            assert _call(lib, name, args) == L.MLA_ERR_INVALID_ARG


def test_sparse_decode_refuses_shapes_without_a_kernel(lib):
    for name in ("mla_decode_absorbed_sparse", "mla_decode_absorbed_sparse_fp8"):
        assert _call(lib, name, CALLS[name][0], dims=_dims(H=12)) == L.MLA_ERR_UNSUPPORTED
        bad = list(CALLS[name][0])
        bad[10] = (1 << 31) - 1
        assert _call(lib, name, bad) == L.MLA_ERR_INVALID_ARG


def test_size_queries_answer_zero_for_bad_arguments(lib):
    d = _dims()
    for fn in (lib.mla_append_fp8_workspace_size, lib.mla_score_pages_workspace_size, lib.mla_decode_sparse_workspace_size,
               lib.mla_decode_sparse_fp8_workspace_size):
        for args in [(7, 1, 1, 16), (1, 0, 1, 16), (1, 1, 0, 16), (1, 1, 1, 0), (1, 1 << 16, 1 << 16, 16)]:
            assert fn(ctypes.byref(d), *args) == 0
    assert lib.mla_decode_sparse_workspace_size(ctypes.byref(d), 1, 64, 1, 16) > 0


def test_binding_refuses_host_tensors():
    dims = ops.Dims(8, 64, 16, 128, 64)
    z = torch.zeros(1, 1, 8)
    i = torch.zeros(1, dtype=torch.int32)
    t = torch.zeros(1, 8, dtype=torch.int32)
    rows = torch.zeros(8 * 64, 144)
    cache = ops.LatentCache(rows[:, :128], rows[:, 128:], 8)
    c8 = ops.LatentCacheFp8(torch.zeros(512, 128, dtype=torch.uint8), torch.zeros(512), rows[:, 128:], 8)
    q = torch.zeros(1, 1, 8, 144)
    with pytest.raises(ValueError):
        ops.mla_select_pages(dims, z, i, 4)
    with pytest.raises(ValueError):
        ops.mla_append_cache_fp8(dims, torch.zeros(1, 1, 64), torch.zeros(64, 144), None, i, t, c8)
    with pytest.raises(ValueError):
        ops.mla_read_latent_fp8(dims, c8, t, torch.zeros(2, dtype=torch.int32), torch.zeros(4, 144))
    with pytest.raises(ValueError):
        ops.mla_update_page_keys(dims, cache, t, i, 1, torch.zeros(8, 144))
    with pytest.raises(ValueError):
        ops.mla_score_pages(dims, q, torch.zeros(8, 144), t, i)
    with pytest.raises(ValueError):
        ops.mla_decode_absorbed_sparse(dims, q, cache, t, i, torch.zeros(1, 1, 2, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32))
