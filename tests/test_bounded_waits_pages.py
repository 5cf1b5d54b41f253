"""Bounded waits that run out inside the tensor-core decodes, the page scores and the projection of many tokens:
the kernel records MLA_ERR_TIMEOUT, everything in flight ends, the kernel returns, and the next call is clean and
gives what it gave before. As in test_bounded_waits.py nothing is faulted: the test-hooks build has a switch that
makes an issuer of products wait, with a 10 ms limit, for a barrier phase that only its own later commit
completes; here the step before which it does so is chosen too, so that loads, copies and products of
earlier steps are in flight or done."""
import ctypes
import functools
import time

import numpy as np
import pytest
import torch

from mla_compressed_latent_b200 import _lib as L
from mla_compressed_latent_b200.ops import Dims

from test_bounded_waits import _load_test_lib
from test_gpu_pages import _cache8, _cache16, _case, _lists

pytestmark = pytest.mark.gpu

LIMIT = 3.0   # seconds: 10 ms, the waits for what was in flight (50 ms each) and the host


def _stalls_then_clean(lib, call, outputs, which, step):
    """call() as it should be, then with the wait that runs out, then as it should be again."""
    stream = torch.cuda.current_stream().cuda_stream

    def run():
        for t in outputs:
            t.fill_(7)
        torch.cuda.synchronize()
        t0 = time.monotonic()
        assert call(stream) == L.MLA_OK
        status = lib.mla_check_status(stream)
        return status, time.monotonic() - t0, [t.clone() for t in outputs]

    assert run()[0] == L.MLA_OK
    status, _, before = run()
    assert status == L.MLA_OK
    assert lib.mla_test_set_stall(which | step << 8) == L.MLA_OK
    try:
        status, took, _ = run()
    finally:
        assert lib.mla_test_set_stall(0) == L.MLA_OK
    assert status == L.MLA_ERR_TIMEOUT and took < LIMIT, took
    status, _, after = run()
    assert status == L.MLA_OK
    for a, b in zip(before, after):
        assert torch.equal(a, b)


# one row cut over many pairs; one page a row, several rows to a pair; some tiles a row, several rows to a pair
ROWS = {"cut": ([64 * 300], 280), "one page": ([40 + i % 90 for i in range(300)], 1), "some pages": ([500 + i for i in range(150)], 7)}


@functools.lru_cache(maxsize=9)
def _decode_call(kind, rows):
    """A decode of the test build, its outputs, and what it keeps alive."""
    lib, (lens, k) = _load_test_lib(), ROWS[rows]
    case = _case("dsv3_b64_l4096", lens)
    w, dev = case.w, case.to_device()
    d = Dims.of(w).c()
    cache = _cache8(dev, case)[0] if kind == "8-bit" else _cache16(dev, case)
    cc = cache.c()
    o = torch.empty(w.B, 1, w.H, w.d_c, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(w.B, 1, w.H, device="cuda")
    pages, counts = (torch.from_numpy(x).cuda() for x in _lists(lens, 1, k, 3))
    table, seqlens, q = dev["table"].contiguous(), dev["seqlens"], dev["q_abs"]
    ws = torch.empty(96 << 20, dtype=torch.uint8, device="cuda")
    keep = (case, cache, pages, counts, table, seqlens, q, ws)
    tail = [o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel()]
    head = [ctypes.byref(d), L.MLA_BF16, w.B, 1, q.data_ptr(), ctypes.byref(cc), table.data_ptr(), table.shape[1], seqlens.data_ptr()]
    if kind == "dense":
        fn, args = lib.mla_decode_absorbed, head + tail
    else:
        fn = lib.mla_decode_absorbed_sparse_fp8 if kind == "8-bit" else lib.mla_decode_absorbed_sparse
        args = head + [pages.data_ptr(), counts.data_ptr(), k] + tail
    return lambda stream: fn(*args, stream), [o, lse], keep


@pytest.mark.parametrize("kind", ["dense", "16-bit", "8-bit"])
@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("which,step", [(1, 0), (2, 0), (1, 1), (2, 1), (2, 2)])
def test_decode(kind, rows, which, step):
    lib = _load_test_lib()
    call, outputs, _ = _decode_call(kind, rows)
    _stalls_then_clean(lib, call, outputs, which, step)


@pytest.mark.parametrize("n_tok,C,gamma", [(1000, 7168, True), (1300, 1216, False), (4096, 2048, False)])
@pytest.mark.parametrize("step", [0, 1, 3, 5])
def test_append_of_many_tokens(n_tok, C, gamma, step):
    lib = _load_test_lib()
    g = torch.Generator(device="cuda").manual_seed(n_tok)
    x = torch.randn(1, n_tok, C, device="cuda", generator=g).bfloat16()
    w = (torch.randn(C, 576, device="cuda", generator=g) * C ** -0.5).bfloat16()
    gm = torch.rand(512, device="cuda", generator=g).bfloat16() if gamma else None
    pages = n_tok // 64 + 1
    table = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)[None].contiguous()
    lens = torch.tensor([n_tok], dtype=torch.int32, device="cuda")
    codes = torch.empty(pages * 64, 512, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages * 64, device="cuda")
    rope = torch.empty(pages * 64, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    d = Dims(128, 128, 64, 512, 128).c()
    cc = L.MlaLatentCacheFp8(codes.data_ptr(), 512, scales.data_ptr(), rope.data_ptr(), 64, pages)

    def call(stream):
        return lib.mla_append_cache_fp8(ctypes.byref(d), L.MLA_BF16, 1, n_tok, x.data_ptr(), C, w.data_ptr(),
                                        gm.data_ptr() if gamma else None, lens.data_ptr(), table.data_ptr(), pages,
                                        ctypes.byref(cc), ws.data_ptr(), ws.numel(), stream)

    _stalls_then_clean(lib, call, [codes, scales, rope], 1, step)


@pytest.mark.parametrize("lens", [[64 * 50] * 3, [64 * 700, 64 * 1100], [64 * 60] * 200], ids=["short", "long", "two CTAs an SM"])
@pytest.mark.parametrize("step", [0, 1, 4, 8])
def test_scores(lens, step):
    lib = _load_test_lib()
    g = torch.Generator(device="cuda").manual_seed(len(lens))
    B, P = len(lens), max(lens) // 64
    keys = torch.randn(5000, 576, device="cuda", generator=g).bfloat16()
    q = torch.randn(B, 1, 128, 576, device="cuda", generator=g).bfloat16()
    table = torch.randint(0, 5000, (B, P), device="cuda", generator=g).to(torch.int32)
    seqlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    scores = torch.empty(B, 1, P, device="cuda")
    d = Dims(128, 128, 64, 512, 128).c()

    def call(stream):
        return lib.mla_score_pages(ctypes.byref(d), L.MLA_BF16, B, 1, q.data_ptr(), keys.data_ptr(), 576, 5000, table.data_ptr(), P,
                                   seqlens.data_ptr(), scores.data_ptr(), None, 0, stream)

    _stalls_then_clean(lib, call, [scores], 1, step)
