"""Edges of the 8-bit append, the read-back and the page-selecting decode: the two-launch fallback, a first
call inside a stream capture, streams other than the current one, pools past 2^32 bytes, queries and scales
of very different sizes. Tolerances as in test_gpu_pages.py."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import synth
from oracle import fp8_cache as F
from oracle import mla_oracle as O
from oracle import page_select as PS
from mla_compressed_latent_b200 import _lib as L
from mla_compressed_latent_b200 import ops
from mla_compressed_latent_b200.ops import Dims, LatentCache, LatentCacheFp8

from _cases import TOL, Case, max_rel_err
from test_bounded_waits import _load_test_lib
from test_gpu_pages import _cache8, _cache16, _case, _check_sparse, _f64, _lists, _rows, ok

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("lens,k", [([131072], 64), (list(np.random.default_rng(5).integers(1, 2000, 120)), 11)])
def test_sparse_decode_as_two_launches(lens, k, bits):
    """The fallback when the runtime refuses the cooperative launch: the decode, then the merge kernel."""
    lib = _load_test_lib()
    case = _case("dsv3_b64_l4096", lens)
    w, dev = case.w, case.to_device()
    cache, held = _cache8(dev, case) if bits == 8 else (_cache16(dev, case), None)
    pages, counts = _lists(lens, 1, k, 3)
    if len(lens) > 1:
        pages[1], counts[1] = -1, 0
    d, cc = Dims.of(w).c(), cache.c()
    tp, tc = torch.from_numpy(pages).cuda(), torch.from_numpy(counts).cuda()
    size = lib.mla_decode_sparse_fp8_workspace_size if bits == 8 else lib.mla_decode_sparse_workspace_size
    fn = lib.mla_decode_absorbed_sparse_fp8 if bits == 8 else lib.mla_decode_absorbed_sparse
    ws = torch.empty(size(ctypes.byref(d), L.MLA_BF16, w.B, 1, k), dtype=torch.uint8, device="cuda")
    o = torch.empty(w.B, 1, w.H, w.d_c, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(w.B, 1, w.H, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.mla_test_set_two_launches(1) == L.MLA_OK
    try:
        rc = fn(ctypes.byref(d), L.MLA_BF16, w.B, 1, dev["q_abs"].data_ptr(), ctypes.byref(cc), dev["table"].data_ptr(),
                dev["table"].shape[1], dev["seqlens"].data_ptr(), tp.data_ptr(), tc.data_ptr(), k, o.data_ptr(),
                lse.data_ptr(), ws.data_ptr(), ws.numel(), stream)
    finally:
        lib.mla_test_set_two_launches(0)
    assert rc == L.MLA_OK and lib.mla_check_status(stream) == L.MLA_OK
    _check_sparse(case, pages, counts, held, o, lse)


FIRST_CALL = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from test_gpu_pages import _case, _cache8, _cache16, _lists, _check_sparse, ok
from mla_compressed_latent_b200 import ops
from mla_compressed_latent_b200.ops import Dims
lens = [131072, 64 * 30 + 7]
case = _case("dsv3_b64_l4096", lens)
w, dev = case.w, case.to_device()
c8, held = _cache8(dev, case)
c8.rope = c8.rope.clone()   # (the append below writes it; the 16-bit cache keeps its own)
c16, dims, k = _cache16(dev, case), Dims.of(w), 40
pages, counts = (torch.from_numpy(x).cuda() for x in _lists(lens, 1, k, 5))
keys = torch.zeros(case.num_pages, 576, dtype=torch.bfloat16, device="cuda")
x = torch.randn(2, 1, 7168, device="cuda").bfloat16()
wt = torch.randn(7168, 576, device="cuda").bfloat16()
rows = torch.zeros(64, 576, dtype=torch.bfloat16, device="cuda")
off = torch.tensor([0, 20, 64], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
side = torch.cuda.Stream()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=side):   # the library's first calls in this process
    out = [ops.mla_decode_absorbed_sparse(dims, dev["q_abs"], c, dev["table"], dev["seqlens"], pages, counts) for c in (c16, c8)]
    ops.mla_read_latent_fp8(dims, c8, dev["table"], off, rows)
    ops.mla_update_page_keys(dims, c16, dev["table"], dev["seqlens"], 131072, keys)
    scores = ops.mla_score_pages(dims, dev["q_abs"], keys, dev["table"], dev["seqlens"])
    chosen = ops.mla_select_pages(dims, scores, dev["seqlens"], 8, 1, 2)
    ops.mla_append_cache_fp8(dims, x, wt, None, dev["seqlens"], dev["table"], c8)
for _ in range(2):
    g.replay()
ok()
_check_sparse(case, pages.cpu().numpy(), counts.cpu().numpy(), None, *out[0])
assert chosen[1].flatten().tolist() == [8, 8] and bool((rows != 0).any(1).all())
print("captured first")
"""


def test_first_calls_of_a_process_may_be_captured():
    code = FIRST_CALL.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_calls_on_a_stream_that_is_not_current():
    """stream=: workspaces and outputs made by the binding belong to that stream, whatever else is made and
    freed on the current one meanwhile."""
    lens = [131072]
    case = _case("dsv3_b64_l4096", lens)
    w, dev = case.w, case.to_device()
    dims, side = Dims.of(w), torch.cuda.Stream()
    pages, counts = _lists(lens, 1, 40, 4)
    tp, tc = torch.from_numpy(pages).cuda(), torch.from_numpy(counts).cuda()
    cache = _cache16(dev, case)
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(6):
        got.append(ops.mla_decode_absorbed_sparse(dims, dev["q_abs"], cache, dev["table"], dev["seqlens"], tp, tc, stream=side))
        torch.full((40 << 20,), float("nan"), device="cuda")   # takes what the current stream's pool has free
    keys = torch.zeros(case.num_pages, 576, dtype=torch.bfloat16, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    ops.mla_update_page_keys(dims, cache, dev["table"], dev["seqlens"], 131072, keys, stream=side)
    scores = ops.mla_score_pages(dims, dev["q_abs"], keys, dev["table"], dev["seqlens"], stream=side)
    chosen = ops.mla_select_pages(dims, scores, dev["seqlens"], 8, stream=side)
    side.synchronize()
    ok()
    for o, l in got:
        _check_sparse(case, pages, counts, None, o, l)
    assert PS.select(scores[0, 0].tolist(), 8, 0, 1) == chosen[0][0, 0].tolist()


@pytest.mark.parametrize("bits", [16, 8])
def test_pools_past_four_gigabytes(bits):
    """Pages whose bytes lie past 2^32 (and whose element offsets lie past 2^31)."""
    lens = [200, 64 * 9 + 3]
    case = _case("dsv3_b64_l4096", lens)
    w, dev = case.w, case.to_device()
    n = 140000   # pages: 10.3 GB of 16-bit rows, 4.6 GB of codes
    rows16 = torch.empty(n * 64, w.d_c + w.d_r, dtype=torch.bfloat16, device="cuda")
    where = torch.arange(case.num_pages) * 61 + (n - 1 - 61 * (case.num_pages - 1))   # the last of them is the pool's last
    dst = (where[:, None] * 64 + torch.arange(64)).flatten()
    rows16[dst.cuda()] = dev["pool"]
    table = where[torch.from_numpy(case.table).long()].to(torch.int32).cuda()
    dims, k = Dims.of(w), 4
    held = None
    if bits == 8:
        small, held = _cache8(dev, case)
        codes = torch.empty(n * 64, w.d_c, dtype=torch.uint8, device="cuda")
        scales = torch.empty(n * 64, device="cuda")
        codes[dst.cuda()], scales[dst.cuda()] = small.codes, small.scales
        cache = LatentCacheFp8(codes, scales, rows16[:, w.d_c:], n)
        out = torch.zeros(sum(lens), 576, dtype=torch.bfloat16, device="cuda")
        off = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
        ops.mla_read_latent_fp8(dims, cache, table, off, out)
        want = torch.zeros_like(out)
        ops.mla_read_latent_fp8(dims, small, dev["table"], off, want)
        ok()
        assert torch.equal(out, want)
    else:
        cache = LatentCache(rows16[:, :w.d_c], rows16[:, w.d_c:], n)
    pages, counts = _lists(lens, 1, k, 2)
    o, lse = ops.mla_decode_absorbed_sparse(dims, dev["q_abs"], cache, table, dev["seqlens"], torch.from_numpy(pages).cuda(),
                                            torch.from_numpy(counts).cuda())
    ok()
    _check_sparse(case, pages, counts, held, o, lse)
    keys = torch.zeros(n, 4096, dtype=torch.bfloat16, device="cuda")[:, :576]   # key rows far apart: past 2^30 bytes
    ops.mla_update_page_keys(dims, cache, table, dev["seqlens"], 1000, keys)
    scores = ops.mla_score_pages(dims, dev["q_abs"], keys, table, dev["seqlens"])
    ok()
    for b, L_b in enumerate(lens):
        ref = PS.page_keys(_rows(case, b, held))
        got = _f64(keys[table[b, :len(ref)].long()])
        assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 66 * 2.0 ** -24 * np.abs(_rows(case, b, held)).max())
        np.testing.assert_allclose(_f64(scores[b, 0, :len(ref)]), PS.page_scores(case.q_abs64[b, 0], got, w.sm_scale), rtol=1e-4)
    if bits == 8:
        x, wt = torch.randn(2, 1, 7168, device="cuda").bfloat16(), (torch.randn(7168, 576, device="cuda") / 85).bfloat16()
        ops.mla_append_cache_fp8(dims, x, wt, None, dev["seqlens"], table, cache)
        ops.mla_append_cache_fp8(dims, x, wt, None, dev["seqlens"], dev["table"], small)
        ok()
        for b, L_b in enumerate(lens):
            r, s = int(table[b, (L_b - 1) // 64]) * 64 + (L_b - 1) % 64, int(case.table[b, (L_b - 1) // 64]) * 64 + (L_b - 1) % 64
            assert torch.equal(codes[r], small.codes[s]) and torch.equal(scales[r], small.scales[s])


@pytest.mark.parametrize("how", ["scales of many sizes", "small latents", "small keys", "large scores", "zero rows", "zero queries"])
def test_sparse_fp8_decode_of_values_of_very_different_sizes(how):
    """The 8-bit decode holds queries in two E4M3 terms and multiplies scales into scores and weights: rows and
    heads of very different sizes, and rows and queries of zeros."""
    lens = [64 * 11 + 9, 300]
    case = _case("dsv3_b64_l4096", lens, 2)
    w, dev = case.w, case.to_device()
    cache, _ = _cache8(dev, case)
    g = np.random.default_rng(6)
    scales = cache.scales.cpu().numpy()
    q = case.q_abs64.copy()
    if how == "scales of many sizes":      # neighbouring rows up to 2^-30 apart: later tiles move the reference
        scales = scales * np.exp2(-g.integers(0, 30, scales.shape)).astype(np.float32)
    elif how == "small latents":
        scales = scales * np.float32(2.0 ** -40)
        q[..., :512] *= 2.0 ** 20
    elif how == "small keys":              # the head's size comes from the part the keys do not see
        q[..., :512] *= np.exp2(g.integers(-30, 1, q.shape[:-1]))[..., None]
    elif how == "large scores":
        q *= 6.0
    elif how == "zero rows":
        dead = g.random(scales.shape) < 0.5
        scales[dead] = 0
        cache.codes[torch.from_numpy(dead).cuda()] = 0
        scales[case.table[1].astype(np.int64)[:5].repeat(64) * 64 + np.tile(np.arange(64), 5)] = 0   # whole tiles of them
    else:
        q[0, 0, :64] = 0
        q[1, :, :, :512] = 0
    qt = torch.from_numpy(q).to(torch.bfloat16)
    case.q_abs64 = qt.double().numpy()
    cache.scales.copy_(torch.from_numpy(scales))
    held = F.dequantize_rows(cache.codes.cpu().numpy(), scales)
    pages, counts = _lists(lens, 2, 9, 1)
    o, lse = ops.mla_decode_absorbed_sparse(Dims.of(w), qt.cuda(), cache, dev["table"], dev["seqlens"],
                                            torch.from_numpy(pages).cuda(), torch.from_numpy(counts).cuda())
    ok()
    got_o, got_l = _f64(o), _f64(lse)
    for b in range(w.B):
        rows = _rows(case, b, held)
        for t in range(2):
            ro, rl = PS.sparse_decode(case.q_abs64[b, t], rows[:, :512], rows[:, 512:], pages[b, t, :counts[b, t]], lens[b] - 1 + t, w.sm_scale)
            # lse: 1e-3, and what the two E4M3 terms of a query (2^-18 of the head's largest value per element)
            # and fp32 sums of 576 terms may move a score
            mag = np.abs(case.q_abs64[b, t])
            terms = (mag @ np.abs(rows).T).max(1) * 576 * 2.0 ** -24 + mag.max(1) * 2.0 ** -18 * np.abs(rows).sum(1).max()
            assert np.all(np.abs(got_l[b, t] - rl) <= 1e-3 + w.sm_scale * terms), (b, t)
            # a head's output within the 16-bit decode's bar of its own largest value
            top = np.abs(ro).max(1, keepdims=True)
            assert np.all(np.abs(got_o[b, t] - ro) <= 2e-2 * top + 1e-30), (b, t)


def test_scores_do_not_read_keys_of_pages_that_no_token_sees():
    w = synth.workload("dsv3_b64_l4096", B=2, s_q=2, lengths=("list", (300, 64 * 20)), pages="random")
    table, n = synth.block_table(w, np.asarray([300, 1280], np.int32))
    keys = torch.full((n + 3, 576), float("nan"), dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(1)
    for b, m in enumerate((5, 20)):
        keys[torch.from_numpy(table[b, :m]).long()] = (torch.randn(m, 576, generator=g) * 0.3).bfloat16()
    q = torch.randn(2, 2, 128, 576, generator=g).bfloat16()
    s = ops.mla_score_pages(Dims.of(w), q.cuda(), keys.cuda(), torch.from_numpy(table).cuda(), torch.tensor([300, 1280], dtype=torch.int32, device="cuda"))
    ok()
    for b, m in enumerate((5, 20)):
        for t in range(2):
            ref = PS.page_scores(q[b, t].double().numpy(), keys[torch.from_numpy(table[b, :m]).long()].double().numpy(), w.sm_scale)
            np.testing.assert_allclose(_f64(s[b, t, :m]), ref, rtol=1e-4)


def test_two_streams_at_once():
    """Two decodes and a selection chain issued on two streams with nothing between them."""
    lens = [64 * 50 + 1] * 6
    case = _case("dsv3_b64_l4096", lens)
    w, dev = case.w, case.to_device()
    dims = Dims.of(w)
    c8, held = _cache8(dev, case)
    c16 = _cache16(dev, case)
    lists = [_lists(lens, 1, 12, s) for s in (1, 2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    args = [(torch.from_numpy(p).cuda(), torch.from_numpy(c).cuda()) for p, c in lists]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, (st, cache) in enumerate(zip(streams, (c16, c8))):
            got[i].append(ops.mla_decode_absorbed_sparse(dims, dev["q_abs"], cache, dev["table"], dev["seqlens"], *args[i], stream=st))
    for st in streams:
        st.synchronize()
    ok()
    for i, h in enumerate((None, held)):
        for o, l in got[i]:
            _check_sparse(case, *lists[i], h, o, l)


@pytest.mark.parametrize("d_c,d_r,C", [(512, 64, 320), (144, 16, 64), (208, 48, 704), (256, 8, 7168), (16, 8, 128)])
@pytest.mark.parametrize("n_tok", [512, 513, 767, 1025])
def test_append_fp8_of_many_tokens_at_odd_widths(d_c, d_r, C, n_tok):
    """Tiles whose features or tokens end inside them, one to many K chunks (the split of K included)."""
    g = torch.Generator().manual_seed(n_tok + C)
    x = torch.randn(1, n_tok, C, generator=g).bfloat16()
    w = (torch.randn(C, d_c + d_r, generator=g) * C ** -0.5).bfloat16()
    seqlen, pages = n_tok + 5, n_tok // 64 + 2
    table = torch.randperm(pages + 3, generator=g)[:pages].to(torch.int32)
    rows = (pages + 3) * 64
    codes = torch.full((rows, d_c), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows,), -2.0, device="cuda")
    rope = torch.full((rows, d_r), 3.0, dtype=torch.bfloat16, device="cuda")
    dims = Dims(8, 64, d_r, d_c, 64)
    ops.mla_append_cache_fp8(dims, x.cuda(), w.cuda(), None, torch.tensor([seqlen], dtype=torch.int32).cuda(),
                             table[None].cuda(), LatentCacheFp8(codes, scales, rope, pages + 3))
    ok()
    pos = np.arange(5, seqlen)
    at = table.numpy()[pos // 64].astype(np.int64) * 64 + pos % 64
    c, kr = O.latent_rows(x[0].double().numpy(), w[:, :d_c].double().numpy(), w[:, d_c:].double().numpy(), pos, None,
                          dims.rms_eps, dims.rope_base)
    got_s = scales.cpu().numpy().astype(np.float64)[at]
    got = F.e4m3_decode(codes.cpu().numpy()[at])
    top = np.abs(c).max(1)
    slack = 2.0 ** -13   # as in test_append_fp8
    assert np.all(np.abs(got_s - top / 448) <= slack * top / 448)
    bar = np.maximum(2.0 ** -4 * np.abs(c), 2.0 ** -10 * got_s[:, None]) + 2 * slack * top[:, None]
    assert np.all(np.abs(got * got_s[:, None] - c) <= bar)
    assert np.all(np.abs(_f64(rope)[at] - kr) <= 2.0 ** -8 * np.abs(kr) + slack * max(1.0, np.abs(kr).max()))
    keep = torch.ones(rows, dtype=torch.bool)
    keep[torch.from_numpy(at)] = False
    assert bool((codes.cpu()[keep] == 9).all() and (scales.cpu()[keep] == -2).all() and (rope.cpu()[keep] == 3).all())


def test_append_fp8_of_many_tokens_captured_and_on_two_streams():
    """An append of many tokens and one of a step, eagerly, on two streams at once, and replayed from a graph: the
    same bytes each time (no sum's order depends on the launch)."""
    g = torch.Generator().manual_seed(3)
    n, C, dims = 1600, 512, Dims(128, 128, 64, 512, 128)
    x = torch.randn(2, n // 2, C, generator=g).bfloat16().cuda()
    w = (torch.randn(C, 576, generator=g) * C ** -0.5).bfloat16().cuda()
    pages = n // 64 + 2
    table = torch.randperm(pages, generator=g)[:2 * (pages // 2)].to(torch.int32).view(2, -1).cuda()
    lens = torch.tensor([n // 2, n // 2 + 9], dtype=torch.int32).cuda()

    def cache():
        return LatentCacheFp8(torch.zeros(pages * 64, 512, dtype=torch.uint8, device="cuda"),
                              torch.zeros(pages * 64, device="cuda"),
                              torch.zeros(pages * 64, 64, dtype=torch.bfloat16, device="cuda"), pages)

    first, small = torch.ones(2, dtype=torch.int32).cuda(), x[:, :1].contiguous()

    def call(c, stream=None):   # many tokens, then a step's
        ops.mla_append_cache_fp8(dims, x, w, None, lens, table, c, stream=stream)
        ops.mla_append_cache_fp8(dims, small, w, None, first, table, c, stream=stream)

    eager, caches = cache(), [cache() for _ in range(3)]
    call(eager)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for st, c in zip(streams, caches):
            call(c, st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(caches[2])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    ok()
    for c in caches:
        assert torch.equal(c.codes, eager.codes) and torch.equal(c.scales, eager.scales) and torch.equal(c.rope, eager.rope)


def test_append_fp8_of_more_tokens_than_one_wave():
    g = torch.Generator().manual_seed(4)
    n, C, d_c, d_r = 16421, 128, 512, 64
    dims = Dims(128, 128, d_r, d_c, 128)
    x = torch.randn(1, n, C, generator=g).bfloat16()
    w = (torch.randn(C, d_c + d_r, generator=g) * C ** -0.5).bfloat16()
    pages = n // 64 + 1
    table = torch.randperm(pages, generator=g).to(torch.int32)
    codes = torch.zeros(pages * 64, d_c, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(pages * 64, device="cuda")
    rope = torch.zeros(pages * 64, d_r, dtype=torch.bfloat16, device="cuda")
    ops.mla_append_cache_fp8(dims, x.cuda(), w.cuda(), None, torch.tensor([n], dtype=torch.int32).cuda(), table[None].cuda(),
                             LatentCacheFp8(codes, scales, rope, pages))
    ok()
    pos = np.arange(n)
    at = table.numpy()[pos // 64].astype(np.int64) * 64 + pos % 64
    c, kr = O.latent_rows(x[0].double().numpy(), w[:, :d_c].double().numpy(), w[:, d_c:].double().numpy(), pos, None,
                          dims.rms_eps, dims.rope_base)
    got_s = scales.cpu().numpy().astype(np.float64)[at]
    top, slack = np.abs(c).max(1), 2.0 ** -13   # as in test_append_fp8
    bar = np.maximum(2.0 ** -4 * np.abs(c), 2.0 ** -10 * got_s[:, None]) + 2 * slack * top[:, None]
    assert np.all(np.abs(F.e4m3_decode(codes.cpu().numpy()[at]) * got_s[:, None] - c) <= bar)
    assert np.all(np.abs(_f64(rope)[at] - kr) <= 2.0 ** -8 * np.abs(kr) + slack * max(1.0, np.abs(kr).max()))


@pytest.mark.parametrize("n", [9, 300, 2048, 8200])
@pytest.mark.parametrize("k,first,recent", [(3, 1, 2), (8, 8, 0), (7, 0, 3)])
def test_select_when_forced_pages_fill_the_list_or_scores_differ_late(n, k, first, recent):
    """Every place forced; scores equal in all but the last bits (the search runs to its last digit); a tie that
    crosses the last place; nothing but NaN."""
    g = torch.Generator().manual_seed(n + k)
    late = (torch.full((n,), 0.37).view(torch.int32) + torch.randint(0, 3 * n, (n,), generator=g).int()).view(torch.float32)
    tie = torch.full((n,), 2.0)
    tie[torch.randperm(n, generator=g)[:k // 2]] = 5.0
    x = torch.stack([late, tie, torch.full((n,), float("nan")), torch.randn(n, generator=g)])[:, None].contiguous()
    lens = torch.full((4,), 64 * n, dtype=torch.int32, device="cuda")
    pages, counts = ops.mla_select_pages(Dims(128, 128, 64, 512, 128), x.cuda(), lens, k, first, recent)
    ok()
    for b in range(4):
        assert pages[b, 0].tolist() == PS.select(x[b, 0].tolist(), k, first, recent)
    assert counts.flatten().tolist() == [k] * 4
