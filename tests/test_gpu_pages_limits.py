"""The calls on 8-bit rows and on pages at the limits of what they take: thousands of uneven lists, scales
of very different sizes in one tile, sequences that outgrow their table row, RoPE widths of any even size, calls of
no rows, scores of -inf. Tolerances as in test_gpu_pages.py unless derived beside the test."""
import numpy as np
import pytest
import torch

from oracle import fp8_cache as F
from oracle import page_select as PS
from mla_compressed_latent_b200 import ops
from mla_compressed_latent_b200.ops import Dims, LatentCache, LatentCacheFp8

from _cases import TOL, TORCH_DT, max_rel_err
from test_gpu_pages import HALF, _cache8, _cache16, _case, _f64, _lists, _rows, _score_case, ok

pytestmark = pytest.mark.gpu

DIMS = Dims(128, 128, 64, 512, 128)


# ---- many uneven lists --------------------------------------------------------------------------------------


def _ramp(n, bits):
    """One sequence of n new tokens, each listing every page it sees: lists of 1 to n / 64 pages."""
    g = torch.Generator(device="cuda").manual_seed(n)
    P = n // 64
    rows = torch.randn(P * 64, 576, device="cuda", generator=g).bfloat16()
    q = (torch.randn(1, n, 128, 576, device="cuda", generator=g) * 0.4).bfloat16()
    table = torch.randperm(P, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    counts = (torch.arange(n, device="cuda", dtype=torch.int32) // 64 + 1)[None]
    pages = torch.arange(P, device="cuda", dtype=torch.int32).expand(1, n, P).contiguous()
    pages[pages >= counts[..., None]] = -1
    cache, held = LatentCache(rows[:, :512], rows[:, 512:], P), _f64(rows)
    if bits == 8:
        codes, scale = F.quantize_rows_f32(rows[:, :512].float().cpu().numpy())
        cache = LatentCacheFp8(torch.from_numpy(codes).cuda(), torch.from_numpy(scale.astype(np.float32)).cuda(), rows[:, 512:], P)
        held[:, :512] = F.dequantize_rows(codes, scale)
    logical = held.reshape(P, 64, 576)[table[0].cpu().numpy()].reshape(-1, 576)
    return q, cache, table, lens, pages, counts, logical


def _time(call, n=5):
    best = float("inf")
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("bits", [16, 8])
def test_thousands_of_uneven_lists(bits):
    """Joining the few rows that are cut must not add a step per pair of rows: the time is held to that of as many
    tiles in lists of one length, which nothing is cut for (a scan of all rows by every row made it 9 times
    that). The bar is 3.1: tiles are shared out evenly, 1824 to each of 73 pairs, and the pair at the start
    of the ramp takes them in 448 rows of 1 to 7 pages, where an even list's takes 56 of 33; a row costs about 14 tiles beyond
    its own, and (1824 + 448 * 14) / (56 * (33 + 14)) = 3.1."""
    n = 4096
    q, cache, table, lens, pages, counts, logical = _ramp(n, bits)
    o = torch.empty(1, n, 128, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, n, 128, device="cuda")

    def call():
        ops.mla_decode_absorbed_sparse(DIMS, q, cache, table, lens, pages, counts, o, lse)

    call()
    ok()
    for t in [0, 63, 64, 65, 1000, 2047, 2048, 3000, 3500, 3777, 3999, 4094, 4095] + list(range(2500, 2600, 7)):
        ro, rl = PS.sparse_decode(_f64(q[0, t]), logical[:, :512], logical[:, 512:], np.arange(t // 64 + 1), t + 1, (128 + 64) ** -0.5)
        assert max_rel_err(_f64(o[0, t]), ro) <= TOL["bf16"]["out"], t
        assert np.abs(_f64(lse[0, t]) - rl).max() <= TOL["bf16"]["lse"], t
    tiles = int(counts.sum())
    long = _time(call)
    even = torch.full_like(counts, tiles // n + 1)   # as many tiles in lists of one length, which nothing is cut for
    even_pages = torch.arange(pages.shape[-1], device="cuda", dtype=torch.int32).expand_as(pages).contiguous()
    even_lens = torch.tensor([n + 64 * pages.shape[-1]], dtype=torch.int32, device="cuda")   # (every token sees all of them)
    big = torch.cat([table, table], 1)

    def even_call():
        ops.mla_decode_absorbed_sparse(DIMS, q, cache, big, even_lens, even_pages, even, o, lse)

    even_call()
    ok()
    assert long <= 3.1 * _time(even_call)


# ---- scales of one tile --------------------------------------------------------------------------------------


@pytest.mark.parametrize("lens,k", [([64 * 9], 3), ([64 * 90], 40), ([64 * 6 + 3 + i for i in range(70)], 4)], ids=["one", "cut", "whole"])
@pytest.mark.parametrize("size", [-8, -20, -26, -32, -60, -90])
def test_a_small_row_that_takes_nearly_all_the_probability(lens, k, size):
    """One row of a tile holds all but 2^-130 of every head's probability while its scale is 2^size of its
    neighbours': the output is that row, however small."""
    case = _case("dsv3_b64_l4096", lens)
    w, dev = case.w, case.to_device()
    cache, _ = _cache8(dev, case)
    pages, counts = _lists(lens, 1, k, 3)
    scales = cache.scales.cpu().numpy()
    q = torch.zeros_like(case.q_abs)
    q[..., :512] = case.q_abs[..., :512]
    q[..., 512] = 8.0
    pool = case.pool.clone()
    pool[:, 512:] = 0
    chosen = []
    for b in range(w.B):
        r = int(case.table[b, pages[b, 0, counts[b, 0] // 2]]) * 64 + (b * 11) % 64   # (a tile that is not the last)
        chosen.append(r)
        scales[r] = np.float32(2.0 ** size) * scales[r]
        pool[r, 512] = 200.0   # q . k_r = 1600, times sm_scale = 1/sqrt(192): 115 above the others
    dev["pool"][:, 512:] = pool[:, 512:].cuda()
    cache.scales.copy_(torch.from_numpy(scales))
    held = F.dequantize_rows(cache.codes.cpu().numpy(), scales)
    case.pool, case.q_abs64 = pool, q.double().numpy()
    o, lse = ops.mla_decode_absorbed_sparse(Dims.of(w), q.cuda(), cache, dev["table"], dev["seqlens"],
                                            torch.from_numpy(pages).cuda(), torch.from_numpy(counts).cuda())
    ok()
    got, got_l = _f64(o)[:, 0], _f64(lse)[:, 0]
    for b in {0, w.B // 2, w.B - 1}:
        rows = _rows(case, b, held)
        ro, rl = PS.sparse_decode(case.q_abs64[b, 0], rows[:, :512], rows[:, 512:], pages[b, 0, :counts[b, 0]], lens[b], w.sm_scale)
        assert np.abs(ro - held[chosen[b]]).max() <= 1e-3 * np.abs(ro).max()   # (what the case is about)
        assert max_rel_err(got[b], ro) <= TOL["bf16"]["out"], b
        # lse: the bar and, as in the test of many sizes, what the query's second term may leave
        mag = np.abs(case.q_abs64[b, 0])
        terms = (mag @ np.abs(rows).T).max(1) * 576 * 2.0 ** -24 + mag.max(1) * 2.0 ** -18 * np.abs(rows).sum(1).max()
        assert np.all(np.abs(got_l[b] - rl) <= 1e-3 + w.sm_scale * terms), b


# ---- page keys ------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("s_q", [1, 64, 300, 100000])
def test_page_keys_report_a_sequence_longer_than_its_table_row(bits, s_q):
    case = _case("dsv3_b64_l4096", [256, 100])
    w, dev = case.w, case.to_device()
    cache = _cache8(dev, case)[0] if bits == 8 else _cache16(dev, case)
    keys = torch.full((case.num_pages, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    table = dev["table"].contiguous()
    lens = torch.tensor([64 * table.shape[1] + 1, 100], dtype=torch.int32, device="cuda")
    ops.mla_update_page_keys(Dims.of(w), cache, table, lens, s_q, keys)
    torch.cuda.synchronize()
    assert ops.mla_check_status() == 6
    assert bool((keys[int(case.table[1, 1])] != 7).any())   # the other sequence's key is written


@pytest.mark.parametrize("dtype,d_c,d_r", [("bf16", 64, 6), ("bf16", 512, 10), ("bf16", 16, 2), ("f32", 64, 6), ("f32", 128, 2),
                                           ("bf16", 144, 12)])
@pytest.mark.parametrize("lens,s_q", [([1], 1), ([63, 64, 65], 1), ([200, 1, 64], 66)])
def test_page_keys_of_an_8_bit_cache_with_any_even_rope_width(dtype, d_c, d_r, lens, s_q):
    case = _case("smallem_fp32", lens, dtype=dtype, d_c=d_c, d_r=d_r)
    w, W = case.w, d_c + d_r
    codes, scale = F.quantize_rows_f32(case.pool[:, :d_c].float().numpy())
    rope = torch.full((case.num_pages * 64, (d_r + 7) // 8 * 8), float("nan"), dtype=case.pool.dtype)
    rope[:, :d_r] = case.pool[:, d_c:]
    cache = LatentCacheFp8(torch.from_numpy(codes).cuda(), torch.from_numpy(scale.astype(np.float32)).cuda(), rope.cuda()[:, :d_r],
                           case.num_pages)
    held = F.dequantize_rows(codes, scale)
    keys = torch.full((case.num_pages, (W + 7) // 8 * 8), 7.0, dtype=TORCH_DT[dtype], device="cuda")
    ops.mla_update_page_keys(Dims.of(w), cache, torch.from_numpy(case.table).cuda(), torch.from_numpy(case.lens).cuda(), s_q, keys[:, :W])
    ok()
    got, touched = _f64(keys[:, :W]), np.zeros(case.num_pages, bool)
    for b, L in enumerate(lens):
        rows = _rows(case, b, held)
        ref = PS.page_keys(rows)
        for p in range(max(0, L - s_q) // 64, (L - 1) // 64 + 1):
            page = case.table[b, p]
            touched[page] = True
            mag = np.abs(rows[p * 64:p * 64 + 64]).mean(0)
            assert np.all(np.abs(got[page] - ref[p]) <= HALF[dtype] * np.abs(ref[p]) + 66 * 2.0 ** -24 * mag)
    assert np.all(got[~touched] == 7) and bool((keys[:, W:] == 7).all())


# ---- read back ------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("name", ["dsv3_b64_l4096", "smallem_fp32"])
def test_read_back_of_no_rows(name):
    """A ragged batch in which no sequence has rows: nothing to do, and the arguments are checked all the same."""
    case = _case(name, [70, 64])
    w, dev = case.w, case.to_device()
    cache, _ = _cache8(dev, case)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.empty(0, w.d_c + w.d_r, dtype=TORCH_DT[w.dtype], device="cuda")
    assert ops.mla_read_latent_fp8(Dims.of(w), cache, dev["table"], off, out) is out
    ok()
    with pytest.raises(ValueError):
        ops.mla_read_latent_fp8(Dims.of(w), cache, dev["table"], off[:2], out)
    with pytest.raises(ValueError):
        ops.mla_read_latent_fp8(Dims.of(w), cache, dev["table"], off, out[:, 1:])


# ---- scores ---------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("name,lens,far", [
    ("dsv3_b64_l4096", [64 * 65], [64]),                   # the only page of the second half of a tile
    ("dsv3_b64_l4096", [64 * 100], list(range(64))),       # a whole half
    ("dsv3_b64_l4096", [64 * 700], list(range(0, 128)) + [699]),
    ("dsv3_b64_l4096", [64 * 700], list(range(600))),      # all pages of most of the cluster's CTAs
    ("dsv3_b64_l4096", [64 * 65] + [64 * 3] * 200, [64]),  # two CTAs to an SM
    ("smallem_fp32", [64 * 65], [64]),
    ("dsv3_b64_l4096", [64 * 3, 64 * 9], [0, 2]),
])
def test_pages_whose_keys_score_minus_infinity_have_no_mass(name, lens, far):
    w, table, num_pages, keys, q = _score_case(name, lens, 1, 3)
    q[0, 0, :, 0] = q[0, 0, :, 0].abs().clamp_min(0.5)
    keys[table[0, far].long(), 0] = float("-inf")
    s = ops.mla_score_pages(Dims.of(w), q.cuda(), keys.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    ok()
    n = lens[0] // 64
    near = np.setdiff1d(np.arange(n), far)
    k64, q64 = keys[table[0, near].long()].double().numpy(), q[0, 0].double().numpy()
    ref = PS.page_scores(q64, k64, w.sm_scale)
    got = _f64(s[0, 0])
    eps = w.sm_scale * (w.d_c + w.d_r) * 2.0 ** -23 * (np.abs(q64) @ np.abs(k64).T).max()   # as in test_page_scores
    assert np.all(got[far] == 0)
    assert np.all(np.abs(got[near] - ref) <= (2 * eps + 2.0 ** -20) * ref)


# ---- several new tokens ---------------------------------------------------------------------------------------


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("L", [64 * 20 + 2, 64 * 20 + 40])   # the new tokens lie across two pages, or in one
def test_tokens_of_a_step_taken_one_by_one_choose_pages_without_the_later_ones(bits, L):
    """A page's key holds every row below seqlens, rows of later tokens of the same step among them. With the lengths
    lowered to each token's own, and its key brought up to date before its scores, a token chooses as if the
    later ones were not there, whatever they are; taken together, the scores of a token that shares a page with
    later ones change with them."""
    s_q, k = 4, 5
    case = _case("dsv3_b64_l4096", [L], s_q)
    w, dims = case.w, Dims.of(case.w)
    got = []
    for later in (0, 1):   # the same step with other rows for its last two tokens
        dev = case.to_device()
        if later:
            for p in (L - 2, L - 1):
                dev["pool"][int(case.table[0, p // 64]) * 64 + p % 64] *= -3
        cache = _cache16(dev, case)
        if bits == 8:
            codes, scale = F.quantize_rows_f32(dev["pool"][:, :512].float().cpu().numpy())
            cache = LatentCacheFp8(torch.from_numpy(codes).cuda(), torch.from_numpy(scale.astype(np.float32)).cuda(),
                                   dev["pool"][:, 512:], case.num_pages)
        q = dev["q_abs"] * 4
        keys = torch.zeros(case.num_pages, 576, dtype=torch.bfloat16, device="cuda")
        lens = [torch.tensor([L - s_q + t + 1], dtype=torch.int32, device="cuda") for t in range(s_q)]
        ops.mla_update_page_keys(dims, cache, dev["table"], lens[0], L, keys)
        alone = []
        for t in range(s_q):
            ops.mla_update_page_keys(dims, cache, dev["table"], lens[t], 1, keys)
            scores = ops.mla_score_pages(dims, q[:, t:t + 1].contiguous(), keys, dev["table"], lens[t])
            alone.append((scores, *ops.mla_select_pages(dims, scores, lens[t], k)))
        together = ops.mla_score_pages(dims, q, keys, dev["table"], dev["seqlens"])
        ok()
        ref = PS.page_keys(_rows(case, 0, None)) if not later and bits == 16 else None
        if ref is not None:   # the keys of the whole step are what the call for all of its tokens leaves
            whole = torch.zeros_like(keys)
            ops.mla_update_page_keys(dims, cache, dev["table"], dev["seqlens"], L, whole)
            ok()
            assert torch.equal(keys, whole)
        got.append((alone, together))
    for t in range(s_q - 2):
        for a, b in zip(got[0][0][t], got[1][0][t]):
            assert torch.equal(a, b), t
        shared = (L - s_q + t) // 64 == (L - 2) // 64   # its last page holds the later tokens' rows too
        assert torch.equal(got[0][1][:, t], got[1][1][:, t]) != shared, t
