"""NaN and infinite scores in the decodes. A head whose query, or any of whose scores, is NaN has NaN outputs and a
NaN lse, however the work was split; a position whose score is -inf weighs nothing; and only a token
without a score above -inf has zeros and lse = -inf. Tolerances as in test_gpu_pages.py."""
import copy
import functools

import numpy as np
import pytest
import torch

from oracle import page_select as PS
from mla_compressed_latent_b200 import ops
from mla_compressed_latent_b200.ops import Dims

from _cases import TOL, max_rel_err
from test_gpu_pages import _cache8, _cache16, _case, _f64, _lists, _rows, ok

pytestmark = pytest.mark.gpu

# one token whose list is cut over many workers, and many tokens whose lists are not
CUT = {"dsv3_b64_l4096": [64 * 40 - 3], "smallem_fp32": [64 * 40]}
WHOLE = {"dsv3_b64_l4096": [705 + 9 * i for i in range(70)], "smallem_fp32": [705 + i for i in range(300)]}
FORMS = [("dsv3_b64_l4096", 16), ("dsv3_b64_l4096", 8), ("smallem_fp32", 16), ("smallem_fp32", 8)]


@functools.lru_cache(maxsize=8)
def _base(name, bits, lens):
    """The case, its 8-bit cache on the device and the rows that holds."""
    case = _case(name, list(lens))
    return (case, *_cache8(case.to_device(), case)) if bits == 8 else (case, None, None)


def _sparse(name, bits, lens, k, change):
    """The decode of a case whose queries [B, H, W] and pool rows [rows, W] `change(case, q, rows, pages)` altered on the
    device first; the case that is returned holds them as altered."""
    case, cache, held = _base(name, bits, tuple(lens))
    case = copy.copy(case)
    w, dev = case.w, case.to_device()
    if bits == 8:
        cache = copy.copy(cache)
        cache.rope = dev["pool"][:, w.d_c:]
    else:
        cache = _cache16(dev, case)
    pages, counts = _lists(lens, 1, k, 7)
    q, rows = dev["q_abs"], dev["pool"]
    change(case, q[:, 0], rows, pages[:, 0])
    o, lse = ops.mla_decode_absorbed_sparse(Dims.of(w), q, cache, dev["table"], dev["seqlens"], torch.from_numpy(pages).cuda(),
                                            torch.from_numpy(counts).cuda())
    ok()
    case.q_abs64, case.pool = _f64(q), rows.cpu()
    return case, pages, counts, held, _f64(o)[:, 0], _f64(lse)[:, 0]


def _ref(case, b, pages, counts, held, keep=slice(None)):
    """The oracle's answer for token b, over the listed pages that `keep` selects."""
    rows, d_c = _rows(case, b, held), case.w.d_c
    return PS.sparse_decode(case.q_abs64[b, 0], rows[:, :d_c], rows[:, d_c:], pages[b, 0, :counts[b, 0]][keep], int(case.lens[b]),
                            case.w.sm_scale)


def _near(case, o, lse, ref):
    w = case.w
    assert max_rel_err(o, ref[0]) <= TOL[w.dtype]["out"]
    assert np.abs(lse - ref[1]).max() <= TOL[w.dtype]["lse"] * (1 if w.dtype == "bf16" else max(1.0, np.abs(ref[1]).max()))


def _pool_row(case, b, page, slot):
    return int(case.table[b, page]) * 64 + slot


@pytest.mark.parametrize("lens", [CUT, WHOLE], ids=["cut", "whole"])
@pytest.mark.parametrize("name,bits", FORMS)
@pytest.mark.parametrize("part", ["latent", "rope"])
def test_a_nan_query_head_has_nan_outputs(name, bits, lens, part):
    lens, head = lens[name], 5

    def change(case, q, rows, pages):
        q[0, head, 3 if part == "latent" else case.w.d_c + 3] = float("nan")

    case, pages, counts, held, o, lse = _sparse(name, bits, lens, 11, change)
    assert np.isnan(o[0, head]).all() and np.isnan(lse[0, head])
    case.q_abs64[0, 0, head] = 0   # (the oracle's other heads)
    others = np.arange(case.w.H) != head
    ro, rl = _ref(case, 0, pages, counts, held)
    _near(case, o[0, others], lse[0, others], (ro[others], rl[others]))
    if len(lens) > 1:
        _near(case, o[1], lse[1], _ref(case, 1, pages, counts, held))


@pytest.mark.parametrize("lens", [CUT, WHOLE], ids=["cut", "whole"])
@pytest.mark.parametrize("name,bits", FORMS)
@pytest.mark.parametrize("where", ["first", "middle", "last", "behind the last"])
def test_one_nan_row_makes_every_head_of_its_token_nan(name, bits, lens, where):
    """NaN in one position's key: every head of the token is NaN if it sees the position, and none if not."""
    lens = lens[name]
    if where == "behind the last" and lens[0] % 64 == 0:
        pytest.skip("the last page is full")
    i, slot = {"first": (0, 2), "middle": (5, 2), "last": (10, 0), "behind the last": (10, lens[0] % 64)}[where]

    def change(case, q, rows, pages):
        rows[_pool_row(case, 0, pages[0, i], slot), case.w.d_c + 1] = float("nan")

    case, pages, counts, held, o, lse = _sparse(name, bits, lens, 11, change)
    assert counts[0, 0] == 11 and pages[0, 0, 10] == (lens[0] - 1) // 64
    if where == "behind the last":
        _near(case, o[0], lse[0], _ref(case, 0, pages, counts, held))
    else:
        assert np.isnan(o[0]).all() and np.isnan(lse[0]).all()
    if len(lens) > 1:
        _near(case, o[1], lse[1], _ref(case, 1, pages, counts, held))


@pytest.mark.parametrize("lens", [CUT, WHOLE], ids=["cut", "whole"])
@pytest.mark.parametrize("name,bits", FORMS)
@pytest.mark.parametrize("away", [[0], [0, 1, 2], [4], [9, 10], list(range(11))], ids=str)
def test_positions_with_scores_of_minus_infinity_weigh_nothing(name, bits, lens, away):
    """Whole listed pages whose keys score -inf for every head: as if the list did not name them."""
    lens = lens[name]

    def change(case, q, rows, pages):
        q[0, :, case.w.d_c] = q[0, :, case.w.d_c].abs().clamp_min(0.5)
        for i in away:
            r = _pool_row(case, 0, pages[0, i], 0)
            rows[r:r + 64, case.w.d_c] = float("-inf")

    case, pages, counts, held, o, lse = _sparse(name, bits, lens, 11, change)
    keep = [i for i in range(11) if i not in away]
    if keep:
        _near(case, o[0], lse[0], _ref(case, 0, pages, counts, held, keep))
    else:
        assert not o[0].any() and np.all(lse[0] == -np.inf)


@pytest.mark.parametrize("lens", [CUT, WHOLE], ids=["cut", "whole"])
@pytest.mark.parametrize("name", ["dsv3_b64_l4096", "smallem_fp32"])
def test_dense_decode_keeps_nan_too(name, lens):
    lens, head = lens[name], 3
    case = _base(name, 16, tuple(lens))[0]
    w, dev = case.w, case.to_device()
    q = dev["q_abs"]
    q[0, 0, head, 1] = float("nan")
    dev["pool"][_pool_row(case, len(lens) - 1, 1, 9), w.d_c] = float("nan")
    o, lse = ops.mla_decode_absorbed(Dims.of(w), q, _cache16(dev, case), dev["table"], dev["seqlens"])
    ok()
    o, lse = _f64(o)[:, 0], _f64(lse)[:, 0]
    assert np.isnan(o[0, head]).all() and np.isnan(lse[0, head])
    assert np.isnan(o[-1]).all() and np.isnan(lse[-1]).all()
    if len(lens) > 1:
        assert np.isfinite(np.delete(o[0], head, 0)).all() and np.isfinite(o[1:-1]).all() and np.isfinite(lse[1:-1]).all()
