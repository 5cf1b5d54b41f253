"""GPU parity of the 8-bit append, the read-back and the page-selecting decode against the fp64 oracle.

Tolerances. Storing rounds to nearest: within eps/2 of the value (bf16 2^-8, E4M3 2^-4 or half a subnormal
step, 2^-10 of the scale). A projection of C products summed 16 at a time by the tensor cores rounds its
partial sum C/16 times by at most 2^-23 of it: 7168/16 * 2^-23 = 2^-14.2 of a partial sum, which is held to
2^-13 of the row's largest value (the fp32 sums of the CUDA cores, at most 64 a slice, stay below that).
fp32 outputs of the decode are held to 1e-5 of the largest value, 16-bit ones and lse to the bars of the dense
decode (2e-2 and 1e-3)."""
import math

import numpy as np
import pytest
import torch

import synth
from oracle import fp8_cache as F
from oracle import mla_oracle as O
from oracle import page_select as PS
from mla_compressed_latent_b200 import ops
from mla_compressed_latent_b200.ops import Dims, LatentCache, LatentCacheFp8

from _cases import TOL, TORCH_DT, Case, max_rel_err

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # half a step, relative to the value


def ok():
    torch.cuda.synchronize()
    assert ops.mla_check_status() == 0


def _f64(t):
    return t.detach().double().cpu().numpy()


def _case(name, lens, s_q=1, pages="random", **kw):
    return Case(synth.workload(name, B=len(lens), s_q=s_q, lengths=("list", tuple(lens)), pages=pages, **kw),
                with_weights=kw.pop("with_weights", False))


def _cache16(dev, case):
    return LatentCache(dev["pool"][:, :case.w.d_c], dev["pool"][:, case.w.d_c:], case.num_pages)


def _cache8(dev, case):
    """The case's pool as an 8-bit cache (quantised by the oracle), and the rows it holds, in fp64."""
    w = case.w
    codes, scale = F.quantize_rows_f32(case.pool[:, :w.d_c].float().numpy())
    cache = LatentCacheFp8(torch.from_numpy(codes).cuda(), torch.from_numpy(scale.astype(np.float32)).cuda(),
                           dev["pool"][:, w.d_c:], case.num_pages)
    return cache, F.dequantize_rows(codes, scale)


def _rows(case, b, held):
    """fp64 [c ; k_r] of positions 0..L-1 of sequence b; held: the latent pool in fp64 (None: the 16-bit one)."""
    p = np.arange(int(case.lens[b]))
    idx = case.table[b, p // 64].astype(np.int64) * 64 + p % 64
    rows = case.pool[torch.from_numpy(idx)].double().numpy()
    if held is not None:
        rows[:, :case.w.d_c] = held[idx]
    return rows


# ---- append into the 8-bit cache ---------------------------------------------------------------------


@pytest.mark.parametrize("name,lens,s_q", [
    ("dsv3_b64_l4096", [4096 - 3 * i for i in range(64)], 1),
    ("dsv3_b64_l4096", [1], 1),
    ("dsv3_b64_l4096", [64, 65, 130], 3),
    ("dsv3_b64_l4096", [200, 333], 129),      # prefill: several pages and token blocks
    ("dsv3_b64_l4096", [1000, 777], 700),
    ("smallem_fp32", [512], 1),
    ("smallem_fp32", [64, 70, 3], 3),
    ("smallem_fp32", [100], 77),
])
@pytest.mark.parametrize("with_gamma", [False, True])
def test_append_fp8(name, lens, s_q, with_gamma):
    w = synth.workload(name, B=len(lens), s_q=s_q, lengths=("list", tuple(lens)), pages="random")
    case = Case(w)
    dev = case.to_device()
    n = w.B * s_q
    x = dev["x"].clone()
    x[0, 0] = 0   # an all-zero token stores scale 0, zero codes and a zero key
    gamma = torch.linspace(0.5, 1.5, w.d_c).to(TORCH_DT[w.dtype]) if with_gamma else None
    rows = case.num_pages * 64
    g = torch.Generator().manual_seed(5)
    codes = torch.randint(0, 256, (rows, w.d_c), dtype=torch.uint8, generator=g).cuda()
    scales = torch.randn(rows, generator=g).cuda()
    rope = torch.randn(rows, w.d_r, generator=g).to(TORCH_DT[w.dtype]).cuda()
    before = [t.clone() for t in (codes, scales, rope)]
    cache = LatentCacheFp8(codes, scales, rope, case.num_pages)
    ops.mla_append_cache_fp8(Dims.of(w), x, dev["w_dkv_kr"], None if gamma is None else gamma.cuda(), dev["seqlens"],
                             dev["table"], cache)
    ok()
    pos = (case.lens[:, None] - s_q + np.arange(s_q)).astype(np.int64)
    at = (case.table[np.arange(w.B)[:, None], pos // 64].astype(np.int64) * 64 + pos % 64).ravel()
    c, kr = O.latent_rows(_f64(x).reshape(n, -1), case.W64["W_DKV"], case.W64["W_KR"], pos.ravel(),
                          None if gamma is None else gamma.double().numpy(), w.rms_eps, w.rope_base)
    got_s, got = scales.cpu().numpy().astype(np.float64)[at], F.e4m3_decode(codes.cpu().numpy()[at])
    top = np.abs(c).max(1)
    slack = 2.0 ** -13
    assert np.all(np.abs(got_s - top / 448) <= slack * top / 448)
    # within half a step of E4M3 of c, and what the fp32 sums may be off; the largest magnitude has code 448
    bar = np.maximum(2.0 ** -4 * np.abs(c), 2.0 ** -10 * got_s[:, None]) + 2 * slack * top[:, None]
    assert np.all(np.abs(got * got_s[:, None] - c) <= bar)
    assert np.all(np.abs(got).max(1)[1:] == 448)
    assert got_s[0] == 0 and not codes.cpu().numpy()[at[0]].any()
    assert not np.any(codes.cpu().numpy()[at] == 0x80)   # no negative zeros
    assert np.all(np.abs(_f64(rope)[at] - kr) <= HALF[w.dtype] * np.abs(kr) + slack * max(1.0, np.abs(kr).max()))
    keep = torch.ones(rows, dtype=torch.bool)
    keep[torch.from_numpy(at)] = False
    for t, b in zip((codes, scales, rope), before):
        assert torch.equal(t.cpu()[keep], b.cpu()[keep])


def test_append_fp8_to_a_bad_page_or_position_is_reported_not_written():
    w = synth.workload("dsv3_b64_l4096", B=3, lengths=("list", (70, 10, 64)), pages="contiguous")
    case = Case(w)
    dev = case.to_device()
    rows = case.num_pages * 64
    codes = torch.full((rows, w.d_c), 7, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows,), 3.0, device="cuda")
    rope = torch.full((rows, w.d_r), 2.0, dtype=torch.bfloat16, device="cuda")
    cache = LatentCacheFp8(codes, scales, rope, case.num_pages)
    table = dev["table"].clone()
    table[0, 1] = case.num_pages          # past the pool
    table[1, 0] = -1
    seqlens = dev["seqlens"].clone()
    seqlens[2] = 64 * table.shape[1] + 1   # past the table row
    ops.mla_append_cache_fp8(Dims.of(w), dev["x"], dev["w_dkv_kr"], None, seqlens, table, cache)
    torch.cuda.synchronize()
    assert ops.mla_check_status() == 6
    assert bool((codes == 7).all()) and bool((scales == 3).all()) and bool((rope == 2).all())


# ---- read back ----------------------------------------------------------------------------------------


@pytest.mark.parametrize("name", ["dsv3_b64_l4096", "smallem_fp32"])
@pytest.mark.parametrize("lens,first,tail", [
    ([1], None, 0), ([300, 1, 64, 0, 65], None, 3), ([0, 0, 7, 0], None, 100), ([5] * 200, None, 1),
    ([130, 64, 20], [3, 0, 19], 0), ([64, 700], [63, 100], 70),
])
def test_read_back_is_exact(name, lens, first, tail):
    full = [max(1, v) for v in lens]
    case = _case(name, full)
    w, dev = case.w, case.to_device()
    cache, _ = _cache8(dev, case)
    n = [v - (first[b] if first else 0) for b, v in enumerate(lens)]
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    dt = TORCH_DT[w.dtype]
    wide = torch.full((int(off[-1]) + tail + 1, w.d_c + w.d_r + 16), 9.0, dtype=dt, device="cuda")
    out = wide[:, :w.d_c + w.d_r]   # rows further apart than they are wide
    ops.mla_read_latent_fp8(Dims.of(w), cache, dev["table"], torch.from_numpy(off).cuda(), out,
                            first=None if first is None else torch.tensor(first, dtype=torch.int32, device="cuda"))
    ok()
    value = torch.from_numpy(F.e4m3_decode(cache.codes.cpu().numpy()).astype(np.float32)) * cache.scales.cpu()[:, None]
    held = torch.cat([value.to(dt), cache.rope.cpu()], 1)
    for b in range(len(lens)):
        p = np.arange(n[b]) + (first[b] if first else 0)
        idx = case.table[b, p // 64].astype(np.int64) * 64 + p % 64
        assert torch.equal(out[int(off[b]):int(off[b + 1])].cpu(), held[torch.from_numpy(idx)]), b
    assert bool((out[int(off[-1]):] == 9).all()) and bool((wide[:, w.d_c + w.d_r:] == 9).all())


def test_read_back_reports_bad_pages_and_stays_inside_its_output():
    case = _case("dsv3_b64_l4096", [70, 64, 100], pages="contiguous")
    w, dev = case.w, case.to_device()
    cache, _ = _cache8(dev, case)
    table = dev["table"].clone()
    table[0, 1], table[1, 0] = case.num_pages, -5
    off = torch.tensor([0, 70, 134, 234], dtype=torch.int32, device="cuda")
    guard = torch.full((300, w.d_c + w.d_r), 9.0, dtype=torch.bfloat16, device="cuda")
    ops.mla_read_latent_fp8(Dims.of(w), cache, table, off, guard[:150])   # the offsets go on past the output
    torch.cuda.synchronize()
    assert ops.mla_check_status() == 6
    assert bool((guard[64:134] == 9).all()) and bool((guard[150:] == 9).all())
    assert bool((guard[:64] != 9).any(1).all()) and bool((guard[134:150] != 9).any(1).all())
    first = torch.tensor([0, 64 * table.shape[1] - 3, -2], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 0, 5, 9], dtype=torch.int32, device="cuda")
    guard.fill_(9.0)
    ops.mla_read_latent_fp8(Dims.of(w), cache, dev["table"], off, guard, first=first)
    torch.cuda.synchronize()
    assert ops.mla_check_status() == 6
    assert bool((guard[3:7] == 9).all()) and bool((guard[9:] == 9).all()) and bool((guard[7:9] != 9).any(1).all())


# ---- page keys ------------------------------------------------------------------------------------------


@pytest.mark.parametrize("name,over", [("dsv3_b64_l4096", {}), ("smallem_fp32", {}),
                                       ("smallem_fp32", {"d_c": 39, "d_r": 6, "dtype": "bf16"})])
@pytest.mark.parametrize("lens,s_q", [([1], 1), ([63, 64, 65], 1), ([130, 500], 3), ([200, 1, 64], 66),
                                      ([1000, 129, 64], 1000)])
@pytest.mark.parametrize("bits", [16, 8])
def test_page_keys(name, over, lens, s_q, bits):
    if bits == 8 and over:
        pytest.skip("codes come in rows of 16 values")
    case = _case(name, lens, **over)
    w = case.w
    W = w.d_c + w.d_r
    pad = 8 if W % 8 else 0
    # slots behind a sequence's last position may hold anything
    used = np.zeros(case.num_pages * 64, bool)
    used[case.pool_rows()] = True
    if pad:
        wide = torch.zeros(case.num_pages * 64, 56, dtype=case.pool.dtype)   # 16-byte row strides
        lat, rope = wide[:, :w.d_c], torch.zeros(case.num_pages * 64, 8, dtype=case.pool.dtype)
        lat.copy_(case.pool[:, :w.d_c])
        rope[:, :w.d_r] = case.pool[:, w.d_c:]
        wide, rope = wide.cuda(), rope.cuda()
        cache = LatentCache(wide[:, :w.d_c], rope[:, :w.d_r], case.num_pages)
        held = None
    else:
        dev = case.to_device()
        cache, held = _cache8(dev, case) if bits == 8 else (_cache16(dev, case), None)
        dead = torch.from_numpy(~used).cuda()
        dev["pool"][dead] = float("nan")
        if bits == 8:
            cache.codes[dead] = 0x7f
            cache.scales[dead] = float("nan")
    keys = torch.full((case.num_pages, W + (8 - W % 8) % 8), 7.0, dtype=TORCH_DT[w.dtype], device="cuda")
    table, seqlens = torch.from_numpy(case.table).cuda(), torch.from_numpy(case.lens).cuda()
    ops.mla_update_page_keys(Dims.of(w), cache, table, seqlens, s_q, keys[:, :W])
    ok()
    got, touched = _f64(keys[:, :W]), np.zeros(case.num_pages, bool)
    for b, L in enumerate(lens):
        rows = _rows(case, b, held)
        ref = PS.page_keys(rows)
        for p in range(max(0, L - s_q) // 64, (L - 1) // 64 + 1):
            page = case.table[b, p]
            touched[page] = True
            # 64 fp32 additions and a division, each 2^-24 of at most the sum of magnitudes, then the store
            mag = np.abs(rows[p * 64:p * 64 + 64]).mean(0)
            assert np.all(np.abs(got[page] - ref[p]) <= HALF[w.dtype] * np.abs(ref[p]) + 66 * 2.0 ** -24 * mag)
    assert np.all(got[~touched] == 7) and bool((keys[:, W:] == 7).all())


def test_page_keys_of_an_empty_sequence_and_a_bad_page():
    case = _case("dsv3_b64_l4096", [70, 64], pages="contiguous")
    w, dev = case.w, case.to_device()
    keys = torch.full((case.num_pages, w.d_c + w.d_r), 7.0, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    ops.mla_update_page_keys(Dims.of(w), _cache16(dev, case), dev["table"], lens, 100, keys)
    ok()
    assert bool((keys == 7).all())
    table = dev["table"].clone()
    table[0, 1], table[1, 0] = case.num_pages, -1
    ops.mla_update_page_keys(Dims.of(w), _cache16(dev, case), table, dev["seqlens"], 100, keys)
    torch.cuda.synchronize()
    assert ops.mla_check_status() == 6
    assert bool((keys[1:] == 7).all()) and bool((keys[0] != 7).any())


# ---- page scores ------------------------------------------------------------------------------------------


def _score_case(name, lens, s_q, seed, **over):
    w = synth.workload(name, B=len(lens), s_q=s_q, lengths=("list", tuple(lens)), pages="random", **over)
    table, num_pages = synth.block_table(w, np.asarray(lens, np.int32))
    g = torch.Generator().manual_seed(seed)
    W = w.d_c + w.d_r
    dt = TORCH_DT[w.dtype]
    keys = (torch.randn(num_pages, W, generator=g) * 0.4).to(dt)
    q = torch.randn(w.B, s_q, w.H, W, generator=g).to(dt)
    return w, torch.from_numpy(table), num_pages, keys, q


@pytest.mark.parametrize("name,lens,s_q,over", [
    ("dsv3_b64_l4096", [1], 1, {}),
    ("dsv3_b64_l4096", [63, 64, 65, 4096], 1, {}),
    ("dsv3_b64_l4096", [2, 66, 64 * 130 + 1], 3, {}),
    ("dsv3_b64_l4096", [64 * 700 + 5, 64 * 33], 2, {}),        # more pages than one CTA's accumulator holds
    ("dsv3_b64_l4096", [131072], 1, {}),
    ("dsv3_b64_l4096", [64 * 4200 + 9, 100], 1, {}),           # more pages than a cluster holds
    ("dsv3_b64_l4096", [777, 64 * 70], 2, {"H": 16}),          # fewer heads than a tile
    ("dsv3_b64_l4096", list(range(1, 64 * 128, 130)), 3, {}),   # many tokens of one tile of pages: two CTAs an SM
    ("dsv3_b64_l4096", [64 * 128] * 40 + [5, 64], 4, {"H": 24}),
    ("dsv3_b64_l4096", [777, 64 * 70], 1, {"H": 40, "d_c": 256, "d_r": 32}),
    ("dsv3_b64_l4096", [777], 1, {"H": 3, "d_c": 72, "d_r": 8}),
    ("dsv3_b64_l4096", [777, 64 * 9], 1, {"H": 192}),
    ("smallem_fp32", [1, 512, 65], 1, {}),
    ("smallem_fp32", [300, 64 * 40], 4, {"H": 5}),
])
def test_page_scores(name, lens, s_q, over):
    w, table, num_pages, keys, q = _score_case(name, lens, s_q, 3, **over)
    scores = torch.full((w.B, s_q, table.shape[1]), -7.0, device="cuda")
    ops.mla_score_pages(Dims.of(w), q.cuda(), keys.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), scores)
    ok()
    got = scores.cpu().numpy().astype(np.float64)
    for b, L in enumerate(lens):
        k64 = keys[table[b].long()].double().numpy()
        for t in range(s_q):
            n = PS.visible_pages(L, s_q, t)
            q64 = q[b, t].double().numpy()
            ref = PS.page_scores(q64, k64[:n], w.sm_scale)
            # u is off by at most W 2^-23 of the sum of its terms' magnitudes; a mass e^u / sum e^u by twice
            # that relative to itself, and 2^-20 for the exponentials, their sums and the sum over heads
            eps = w.sm_scale * (w.d_c + w.d_r) * 2.0 ** -23 * (np.abs(q64) @ np.abs(k64[:n]).T).max(initial=0)
            assert np.all(np.abs(got[b, t, :n] - ref) <= (2 * eps + 2.0 ** -20) * ref), (b, t)
            assert np.all(got[b, t, n:] == -7)


def test_page_scores_report_a_bad_page_and_score_it_as_zero():
    w, table, num_pages, keys, q = _score_case("dsv3_b64_l4096", [64 * 5], 1, 4)
    bad = table.clone()
    bad[0, 2] = num_pages
    bad[0, 4] = -3
    s = ops.mla_score_pages(Dims.of(w), q.cuda(), keys.cuda(), bad.cuda(), torch.tensor([320], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert ops.mla_check_status() == 6
    k64 = keys[table[0].long()].double().numpy()
    k64[[2, 4]] = 0
    np.testing.assert_allclose(s[0, 0].cpu().numpy(), PS.page_scores(q[0, 0].double().numpy(), k64, w.sm_scale), rtol=1e-4)


def test_page_scores_of_a_token_that_sees_nothing_are_not_written():
    w, table, num_pages, keys, q = _score_case("dsv3_b64_l4096", [130, 70], 3, 4)
    scores = torch.full((2, 3, table.shape[1]), -7.0, device="cuda")
    ops.mla_score_pages(Dims.of(w), q.cuda(), keys.cuda(), table.cuda(), torch.tensor([0, 2], dtype=torch.int32, device="cuda"), scores)
    ok()
    assert bool((scores[0] == -7).all()) and bool((scores[1, 0] == -7).all())
    assert scores[1, 1, 0].item() == pytest.approx(w.H, rel=1e-5) and bool((scores[:, :, 1:] == -7).all())


# ---- selection --------------------------------------------------------------------------------------------


def _select_ref(scores, lens, s_q, k, first, recent):
    B = len(lens)
    pages, counts = np.full((B, s_q, k), -1, np.int32), np.zeros((B, s_q), np.int32)
    for b in range(B):
        for t in range(s_q):
            n = min(PS.visible_pages(lens[b], s_q, t), scores.shape[2])
            got = PS.select(scores[b, t, :n].tolist(), k, first, recent)
            pages[b, t, :len(got)], counts[b, t] = got, len(got)
    return pages, counts


@pytest.mark.parametrize("max_pages", [1, 7, 64, 257, 2048, 2049, 8192, 9001])
@pytest.mark.parametrize("k,first,recent", [(1, 0, 1), (4, 1, 2), (16, 0, 0), (100, 3, 5)])
@pytest.mark.parametrize("kind", ["normal", "ties", "odd"])
def test_select(max_pages, k, first, recent, kind):
    g = torch.Generator().manual_seed(max_pages + k)
    lens = [1, 64 * max_pages, max(2, 40 * max_pages), min(130, 64 * max_pages)]
    s_q = 2
    x = torch.randn(4, s_q, max_pages, generator=g)
    if kind == "ties":
        x = (x * 2).round()
    elif kind == "odd":   # zeros of both signs, infinities, NaNs, denormals, neighbours in the last bit
        pick = torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan, 1e-42, -1e-42, 1.0, 1.0 + 2.0 ** -23, -1.0, -3e38])
        x = pick[torch.randint(0, len(pick), x.shape, generator=g)]
    pages, counts = ops.mla_select_pages(Dims(128, 128, 64, 512, 128), x.cuda(),
                                         torch.tensor(lens, dtype=torch.int32, device="cuda"), k, first, recent)
    ok()
    rp, rc = _select_ref(x.numpy(), lens, s_q, k, first, recent)
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert np.array_equal(pages.cpu().numpy(), rp)


def test_select_reports_a_sequence_longer_than_its_row():
    x = torch.arange(12, dtype=torch.float32, device="cuda").view(1, 1, 12)
    pages, counts = ops.mla_select_pages(Dims(128, 128, 64, 512, 128), x, torch.tensor([64 * 13], dtype=torch.int32, device="cuda"), 3)
    torch.cuda.synchronize()
    assert ops.mla_check_status() == 6
    assert pages[0, 0].tolist() == [9, 10, 11] and counts.item() == 3


# ---- decode over selected pages -----------------------------------------------------------------------------


def _lists(lens, s_q, k, seed, keep_last=True):
    """Random ascending lists of at most k visible pages (the last visible one among them)."""
    g = np.random.default_rng(seed)
    B = len(lens)
    pages, counts = np.full((B, s_q, k), -1, np.int32), np.zeros((B, s_q), np.int32)
    for b in range(B):
        for t in range(s_q):
            n = PS.visible_pages(lens[b], s_q, t)
            if n == 0:
                continue
            got = set(g.choice(n, min(k, n), replace=False).tolist())
            if keep_last and n - 1 not in got:
                got.remove(max(got))
                got.add(n - 1)
            pages[b, t, :len(got)], counts[b, t] = sorted(got), len(got)
    return pages, counts


def _run_sparse(case, pages, counts, bits=16, poison=True):
    """The decode over the lists and its reference; every row that no list names is NaN on the device."""
    w, dev = case.w, case.to_device()
    cache, held = _cache8(dev, case) if bits == 8 else (_cache16(dev, case), None)
    s_q = w.s_q
    if poison:
        named = np.zeros(case.num_pages * 64, bool)
        for b in range(w.B):
            for t in range(s_q):
                vis = int(case.lens[b]) - s_q + t + 1
                for p in pages[b, t, :counts[b, t]]:
                    n = min(64, vis - p * 64)
                    named[case.table[b, p] * 64:case.table[b, p] * 64 + n] = True
        dead = torch.from_numpy(~named).cuda()
        dev["pool"][dead] = float("nan")
        if bits == 8:
            cache.codes[dead] = 0x7f
            cache.scales[dead] = float("nan")
    o, lse = ops.mla_decode_absorbed_sparse(Dims.of(w), dev["q_abs"], cache, dev["table"], dev["seqlens"],
                                            torch.from_numpy(pages).cuda(), torch.from_numpy(counts).cuda())
    ok()
    _check_sparse(case, pages, counts, held, o, lse)
    return o, lse


def _check_sparse(case, pages, counts, held, o, lse):
    w, s_q = case.w, case.w.s_q
    got_o, got_l = _f64(o), _f64(lse)
    for b in range(w.B):
        rows = _rows(case, b, held)
        for t in range(s_q):
            vis = int(case.lens[b]) - s_q + t + 1
            ro, rl = PS.sparse_decode(case.q_abs64[b, t], rows[:, :w.d_c], rows[:, w.d_c:], pages[b, t, :counts[b, t]], vis, w.sm_scale)
            if counts[b, t] == 0:
                assert not got_o[b, t].any() and np.all(got_l[b, t] == -np.inf)
                continue
            assert max_rel_err(got_o[b, t], ro) <= TOL[w.dtype]["out"], (b, t)
            bar = TOL[w.dtype]["lse"] * (1 if w.dtype == "bf16" else max(1.0, np.abs(rl).max()))
            assert np.abs(got_l[b, t] - rl).max() <= bar, (b, t)


SPARSE = [
    ([1], 1, 1), ([63, 64, 65], 1, 2), ([4096], 1, 1), ([4096], 1, 32), ([131072], 1, 40),
    ([4096, 129, 2049, 64, 5000], 1, 20), ([700, 64 * 12 + 1], 2, 6), ([65, 130, 64 * 9], 4, 3),
    (list(np.random.default_rng(3).integers(1, 3000, 90)), 1, 13),
    (list(np.random.default_rng(4).integers(4, 3000, 40)), 4, 9),
    # whole rows, several to a pair; rows of very different lengths, cut between pairs
    (list(np.random.default_rng(5).integers(200, 700, 124)), 2, 4), ([300] * 80 + [6000] * 10, 1, 64),
]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("lens,s_q,k", SPARSE)
def test_sparse_decode(lens, s_q, k, bits):
    case = _case("dsv3_b64_l4096", lens, s_q)
    pages, counts = _lists(lens, s_q, k, 7)
    _run_sparse(case, pages, counts, bits)


@pytest.mark.parametrize("bits", [16, 8])
def test_sparse_decode_of_lists_without_the_last_page_and_empty_ones(bits):
    lens = [64 * 6 + 10, 64 * 40, 30, 64 * 3]
    case = _case("dsv3_b64_l4096", lens, 2)
    pages, counts = _lists(lens, 2, 4, 9, keep_last=False)
    pages[0, 0], counts[0, 0] = [0, 1, 2, 3], 4   # whole pages only
    pages[1, 1], counts[1, 1] = -1, 0
    pages[2], counts[2] = -1, 0
    _run_sparse(case, pages, counts, bits)
    pages[:], counts[:] = -1, 0                    # no token lists anything
    _run_sparse(case, pages, counts, bits)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("lens,s_q,k", [([512, 65, 1], 1, 3), ([2000, 300], 3, 20), ([4096], 1, 64)])
def test_sparse_decode_fp32(lens, s_q, k, bits):
    case = _case("smallem_fp32", lens, s_q)
    pages, counts = _lists(lens, s_q, k, 8)
    if len(lens) > 2:
        pages[2], counts[2] = -1, 0
    _run_sparse(case, pages, counts, bits)


@pytest.mark.parametrize("bits", [16, 8])
def test_sparse_decode_bf16_of_other_shapes(bits):
    case = _case("dsv3_b64_l4096", [700, 64 * 5 + 1], 2, H=16, d_c=256)
    pages, counts = _lists([700, 64 * 5 + 1], 2, 4, 8)
    _run_sparse(case, pages, counts, bits)


def test_sparse_decode_of_every_page_is_the_dense_decode():
    lens = [4096, 129, 2049, 64, 5000]
    case = _case("dsv3_b64_l4096", lens)
    w, dev = case.w, case.to_device()
    n = [PS.visible_pages(v, 1, 0) for v in lens]
    pages = np.full((5, 1, max(n) + 3), -1, np.int32)
    for b, m in enumerate(n):
        pages[b, 0, :m] = np.arange(m)
    o, lse = ops.mla_decode_absorbed_sparse(Dims.of(w), dev["q_abs"], _cache16(dev, case), dev["table"], dev["seqlens"],
                                            torch.from_numpy(pages).cuda(), torch.tensor(n, dtype=torch.int32, device="cuda")[:, None])
    ro, rl = ops.mla_decode_absorbed(Dims.of(w), dev["q_abs"], _cache16(dev, case), dev["table"], dev["seqlens"])
    ok()
    assert max_rel_err(_f64(o), _f64(ro)) <= TOL["bf16"]["out"] and float((lse - rl).abs().max()) <= TOL["bf16"]["lse"]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("name", ["dsv3_b64_l4096", "smallem_fp32"])
@pytest.mark.parametrize("bad", ["past the visible pages", "twice", "descending", "negative", "two negative", "count", "pool"])
def test_sparse_decode_reports_a_bad_list(name, bits, bad):
    """A bad entry is reported and not read; the other tokens' results stand."""
    lens = [64 * 6, 64 * 8 + 3]
    case = _case(name, lens)
    w, dev = case.w, case.to_device()
    cache, held = _cache8(dev, case) if bits == 8 else (_cache16(dev, case), None)
    pages = np.array([[[0, 2, 5]], [[1, 3, 8]]], np.int32)
    counts = np.full((2, 1), 3, np.int32)
    sent, n, table = pages.copy(), counts.copy(), dev["table"].clone()
    if bad == "past the visible pages":
        sent[0, 0, 2] = 6
    elif bad == "twice":
        sent[0, 0, 1] = 0
    elif bad == "descending":
        sent[0, 0] = [2, 0, 5]
    elif bad == "negative":
        sent[0, 0, 0] = -4
    elif bad == "two negative":   # ascending, but no page at all
        sent[0, 0] = [-4, -3, 5]
    elif bad == "count":
        n[0] = 4
    else:
        table[0, 2] = case.num_pages
    o, lse = ops.mla_decode_absorbed_sparse(Dims.of(w), dev["q_abs"], cache, table, dev["seqlens"],
                                            torch.from_numpy(sent).cuda(), torch.from_numpy(n).cuda())
    torch.cuda.synchronize()
    assert ops.mla_check_status() == 6
    rows = _rows(case, 1, held)
    ro, rl = PS.sparse_decode(case.q_abs64[1, 0], rows[:, :w.d_c], rows[:, w.d_c:], pages[1, 0], lens[1], w.sm_scale)
    assert max_rel_err(_f64(o[1, 0]), ro) <= TOL[w.dtype]["out"]


# ---- together ------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("s_q", [1, 2])
def test_append_keys_scores_selection_and_decode_together(bits, s_q):
    """One step as a serving loop makes it, run eagerly on a side stream and replayed from a CUDA graph: the
    cache grows by s_q tokens, the pages are chosen and attended; checked against the oracle on the cache's
    own contents and the pages that were chosen."""
    lens = [64 * 30 + 5, 64 * 7, 65 + s_q, s_q]
    w = synth.workload("dsv3_b64_l4096", B=4, s_q=s_q, lengths=("list", tuple(lens)), pages="random")
    case = Case(w)
    dims, k = Dims.of(w), 6
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        dev = case.to_device()
        cache = _cache8(dev, case)[0] if bits == 8 else _cache16(dev, case)
        keys = torch.zeros(case.num_pages, w.d_c + w.d_r, dtype=torch.bfloat16, device="cuda")
        ops.mla_update_page_keys(dims, cache, dev["table"], dev["seqlens"], max(lens), keys)
        x = dev["x"].clone()

        def step():
            if bits == 8:
                ops.mla_append_cache_fp8(dims, x, dev["w_dkv_kr"], None, dev["seqlens"], dev["table"], cache)
            else:
                ops.mla_append_cache(dims, x, dev["w_dkv_kr"], None, dev["seqlens"], dev["table"], cache)
            ops.mla_update_page_keys(dims, cache, dev["table"], dev["seqlens"], s_q, keys)
            scores = ops.mla_score_pages(dims, dev["q_abs"], keys, dev["table"], dev["seqlens"])
            pages, counts = ops.mla_select_pages(dims, scores, dev["seqlens"], k, 1, 2)
            return scores, pages, counts, ops.mla_decode_absorbed_sparse(dims, dev["q_abs"], cache, dev["table"], dev["seqlens"], pages, counts)

        def check(got):
            side.synchronize()
            assert ops.mla_check_status() == 0
            scores, pages, counts, (o, lse) = got
            pool = dev["pool"].cpu()
            held = F.dequantize_rows(cache.codes.cpu().numpy(), cache.scales.cpu().numpy()) if bits == 8 else None
            case.pool = pool
            keys64 = _f64(keys)
            for b, L in enumerate(lens):
                rows = _rows(case, b, held)
                ref = PS.page_keys(rows)
                at = case.table[b, :len(ref)]
                assert np.all(np.abs(keys64[at] - ref) <= 2.0 ** -8 * np.abs(ref) + 66 * 2.0 ** -24 * np.abs(rows).max())
                for t in range(s_q):
                    n = PS.visible_pages(L, s_q, t)
                    s = PS.page_scores(case.q_abs64[b, t], keys64[at[:n]], w.sm_scale)
                    np.testing.assert_allclose(_f64(scores[b, t, :n]), s, rtol=1e-4)
            assert np.array_equal(np.stack([pages.cpu().numpy()]), np.stack([_select_ref(scores.cpu().numpy(), lens, s_q, k, 1, 2)[0]]))
            _check_sparse(case, pages.cpu().numpy(), counts.cpu().numpy(), held, o, lse)

        check(step())
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
        for seed in (1, 2):
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)).to(x.dtype))
            graph.replay()
            check(out)


def test_two_captured_decodes_share_a_workspace():
    """Two graphs over one caller-given workspace, replayed in turn on one stream."""
    lens = [131072]
    case = _case("dsv3_b64_l4096", lens)
    w, dev = case.w, case.to_device()
    lists = [_lists(lens, 1, 40, s) for s in (1, 2)]
    ws = torch.empty(80 << 20, dtype=torch.uint8, device="cuda")
    args = [(torch.from_numpy(p).cuda(), torch.from_numpy(c).cuda()) for p, c in lists]
    outs = [(torch.empty(1, 1, w.H, w.d_c, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 1, w.H, device="cuda")) for _ in lists]
    graphs = []
    for (p, c), (o, l) in zip(args, outs):
        ops.mla_decode_absorbed_sparse(Dims.of(w), dev["q_abs"], _cache16(dev, case), dev["table"], dev["seqlens"], p, c, o, l, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.mla_decode_absorbed_sparse(Dims.of(w), dev["q_abs"], _cache16(dev, case), dev["table"], dev["seqlens"], p, c, o, l, ws)
        graphs.append(g)
    for o, l in outs:
        o.zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    ok()
    for (p, c), (o, l) in zip(lists, outs):
        _check_sparse(case, p, c, None, o, l)


def test_refusals():
    case = _case("dsv3_b64_l4096", [300])
    w, dev = case.w, case.to_device()
    dims, cache = Dims.of(w), _cache16(dev, case)
    pages = torch.zeros(1, 1, 2, dtype=torch.int32, device="cuda")
    counts = torch.ones(1, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        ops.mla_decode_absorbed_sparse(dims, dev["q_abs"], cache, dev["table"], dev["seqlens"], pages.long(), counts)
    with pytest.raises(ValueError):
        ops.mla_decode_absorbed_sparse(dims, dev["q_abs"], cache, dev["table"], dev["seqlens"], pages, counts[0])
    with pytest.raises(ValueError):
        ops.mla_decode_absorbed_sparse(dims, dev["q_abs"].transpose(1, 2), cache, dev["table"], dev["seqlens"], pages, counts)
    with pytest.raises(ops.MlaError):
        ops.mla_select_pages(dims, torch.zeros(1, 1, 8, device="cuda"), dev["seqlens"], 2, 2, 1)
    with pytest.raises(ValueError):
        ops.mla_update_page_keys(dims, cache, dev["table"], dev["seqlens"], 1, torch.zeros(1, 576, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        ops.mla_read_latent_fp8(dims, LatentCacheFp8(torch.zeros(64, 512, dtype=torch.uint8, device="cuda"), torch.zeros(64, device="cuda"), dev["pool"][:, 512:], 2), dev["table"], torch.zeros(2, dtype=torch.int32, device="cuda"), dev["pool"])
    short = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(ops.MlaError):
        ops.mla_decode_absorbed_sparse(dims, dev["q_abs"], cache, dev["table"], dev["seqlens"], pages, counts, workspace=short)
