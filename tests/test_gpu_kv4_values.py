"""Magnitudes and values at the ends of their types in the cache operators:
queries of any finite size, values that only some of a tile's rows see,
infinities and NaN, scales of any size.

Tolerances.  What tests/test_gpu_kv4.py derives, by row: an element is off by
2^-8 of itself (bf16), by the weights' rounding (2^-10 of the sum of weight *
|v|, or bf16's 2^-8 + 2^-11 on the kernel for many rows), and by what lies below
f16's normal range: by 2^-25 * |code| a token, |code| <= 6, where a block's sums
are 1 and more (or the reference is within 2^8 of what the row needs, which is as
good): n tokens are off by n * 6 * 2^-25 of the block's largest |sum|, and that sum
is at most the sum of weight * (largest |v| of the block): n * 2^-22 of that.  Nothing counts that the row does not see."""
import math

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_fp8_b200 as fp8mm
from tests import gpu_util as gu
from tests import kv4_ref as ref
from tests.test_gpu_kv4 import BF16_WEIGHTS, MANY_ROWS, _i32, _kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gu.require_gpu()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert fp8mm.last_device_error() == 0


def _workspace(dim):
    return torch.zeros(fp8mm.mxfp4_kv_attention_workspace_bytes(dim), dtype=torch.uint8, device="cuda")


def _written(k, v, page_size=16):
    """One sequence's tokens appended: (cache, page table, length), and the stored fp64 keys and values."""
    n, heads, dim = k.shape
    pages = -(-n // page_size)
    table = _i32([torch.randperm(pages, generator=torch.Generator().manual_seed(n)).tolist()])
    cache = torch.full((pages, fp8mm.mxfp4_kv_page_bytes(page_size, heads, dim)), 255, dtype=torch.uint8, device="cuda")
    fp8mm.mxfp4_kv_append(k.cuda(), v.cuda(), cache, table, _i32([n]), page_size, cu_seqlens=_i32([0, n]))
    stored = []
    for x in (k, v):
        finite = torch.isfinite(x.float()).unflatten(-1, (-1, 32)).all(-1).repeat_interleave(32, -1)
        stored.append(torch.where(finite, ref.value(*ref.quantize(torch.where(finite, x, 0))), math.nan))
    return cache, table, stored


def _run(q, written, heads, scale, workspace, page_size=16):
    cache, table, (k, _) = written
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    out = fp8mm.mxfp4_kv_attention(q.cuda(), cache, table, _i32([k.shape[0]]), page_size, cu_seqlens=_i32([0, q.shape[0]]),
                                   scale=scale, lse=lse, workspace=workspace)
    return out.double().cpu(), lse.double().cpu()


def _check_row(out, lse, q, k, v, scale, weights):
    """One row of one head, q [dim], over the keys and values [n, dim] that it sees."""
    s = k @ q.double() * scale
    p = torch.softmax(s, 0)
    want, mag = p @ v, p @ v.abs()
    peak = (p[:, None] * v.unflatten(-1, (-1, 32)).abs().amax(-1)).sum(0).repeat_interleave(32)
    lim = 2.0 ** -8 * want.abs() + weights * mag + k.shape[0] * 2.0 ** -22 * peak + 1e-37
    bad = (out - want).abs() / lim
    assert torch.isfinite(out).all() and bad.max() <= 1, (bad.max(), want[bad.argmax()], out[bad.argmax()])
    wlse = torch.logsumexp(s, 0)
    assert (lse - wlse).abs() <= 2.0 ** -14 * (1 + wlse.abs()), (lse, wlse)


def _kinds(rows, group, dim):
    """(workspace, weights) of the calls that a test makes: cut or not, and which kernel the rows take."""
    many = rows * group >= MANY_ROWS
    return ((_workspace(dim), BF16_WEIGHTS if many else 2.0 ** -10), (None, 2.0 ** -10))


def _check_queries(dim, rows, sizes):
    """Rows whose largest magnitude is sizes[h] in query head h, zeros among them, three heads on each of two."""
    n, heads = 150, 2
    written = _written(*_kv(n, heads, dim, 4))
    g = torch.Generator().manual_seed(rows)
    q = torch.randn(rows, heads, 3, dim, generator=g)
    q = q / q.abs().amax(-1, keepdim=True) * torch.tensor(sizes).view(heads, 3, 1)
    q[..., ::7] = 0
    q = q.flatten(1, 2).bfloat16()
    assert (q.abs().amax(-1) > 0).all()
    for ws, weights in _kinds(rows, 3, dim):
        out, lse = _run(q, written, heads, dim ** -0.5, ws)
        for i in range(rows):
            for h in range(6):
                k, v = (x[:n - rows + i + 1, h // 3] for x in written[2])
                _check_row(out[i, h], lse[i, h], q[i, h], k, v, dim ** -0.5, weights)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_queries_of_tiny_size(dim, rows):
    """Down to bf16's smallest subnormal, beside rows of ordinary size."""
    _check_queries(dim, rows, (2.0 ** -113, 2.0 ** -114, 2.0 ** -126, 2.0 ** -133, 1.0, 2.0 ** -120))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_queries_of_huge_size(dim, rows):
    """The largest score takes all of the weight, whatever its rounding in fp32."""
    _check_queries(dim, rows, (2.0 ** 20, 2.0 ** 30, 2.0 ** 60, 2.0 ** 100, 1.0, 2.0 ** 110))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [1, 4, 40])
@pytest.mark.parametrize("step", [2.0 ** 20, 2.0 ** 26, 2.0 ** 40])
def test_scores_past_the_precision_of_fp32(dim, rows, step):
    """Scores of up to 120 steps whose rounding in fp32 is larger than one: tokens share the largest, in the first
    step, the last and between, and the softmax is theirs alone."""
    n, heads = 260, 1
    k = torch.zeros(n, heads, dim)
    k[:, :, 0] = (torch.arange(n) % 97).clamp(max=96)[:, None] // 24
    top = [30, 31, 140, n - rows]
    k[top, :, 0] = 6.0
    k[:, :, 1] = 0.5
    _, v = _kv(n, heads, dim, 8)
    written = _written(k.bfloat16(), v)
    assert torch.equal(written[2][0], k.double())
    q = torch.zeros(rows, 3, dim)
    q[..., 0] = torch.tensor([1.0, 1.2109375, 1.7578125]) * step
    q[..., 1] = 3.0 * step
    q = q.bfloat16()
    for ws, weights in _kinds(rows, 3, dim):
        out, lse = _run(q, written, heads, 0.7, ws)
        for i in range(rows):
            for h in range(3):
                kk, vv = (x[:n - rows + i + 1, 0] for x in written[2])
                _check_row(out[i, h], lse[i, h], q[i, h], kk, vv, 0.7, weights)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** 30, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("rows,group", [(2, 2), (4, 2), (5, 3), (40, 3)])
def test_outlier_values_that_other_rows_see(dim, size, rows, group):
    """The last token's values, which only the last row sees, and those of a token that only the first query head of
    each key/value head attends to, are 2^30 and more times the others': every row keeps its own precision."""
    n, heads, at = 130, 2, 77
    k, v = _kv(n, heads, dim, 6)
    k, v = 0.02 * k.float(), v.float()
    k[..., :32] = 0
    k[at, :, :32] = 6.0
    v[at, :, ::3] *= size
    v[n - 1] *= size
    written = _written(k.bfloat16(), v.bfloat16())
    q = torch.randn(rows, heads, group, dim, generator=torch.Generator().manual_seed(2))
    q[..., :32] = -1.0
    q[:, :, 0, :32] = 1.0
    q = q.flatten(1, 2).bfloat16()
    for ws, weights in _kinds(rows, group, dim):
        out, lse = _run(q, written, heads, 1.0, ws)
        for i in range(rows):
            for h in range(heads * group):
                kk, vv = (x[:n - rows + i + 1, h // group] for x in written[2])
                _check_row(out[i, h], lse[i, h], q[i, h], kk, vv, 1.0, weights)


POISON = {"inf": math.inf, "-inf": -math.inf, "nan": math.nan, "largest": 3.3895313892515355e38}


@pytest.mark.parametrize("kind", list(POISON))
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,group", [(1, 2), (4, 2), (6, 3), (70, 3)])
def test_poisoned_tokens_stay_with_the_rows_that_see_them(kind, where, dim, rows, group):
    """One element of the last two tokens (a padded step's) is infinite, NaN or the type's largest: rows before them are as without."""
    n, heads = 150, 2
    k, v = (x.float() for x in _kv(n, heads, dim, 6))
    (k if where == "k" else v)[n - 2:, :, 5] = POISON[kind]
    written = _written(k.bfloat16(), v.bfloat16())
    q = torch.randn(rows, heads * group, dim, generator=torch.Generator().manual_seed(2)).bfloat16()
    for ws, weights in _kinds(rows, group, dim):
        out, lse = _run(q, written, heads, dim ** -0.5, ws)
        for i in range(rows):
            seen = n - rows + i + 1
            for h in range(heads * group):
                kk, vv = (x[:seen, h // group] for x in written[2])
                if seen <= n - 2:
                    _check_row(out[i, h], lse[i, h], q[i, h], kk, vv, dim ** -0.5, weights)
                elif kind == "nan" and where == "k":
                    assert torch.isnan(out[i, h]).all() and torch.isnan(lse[i, h])
                elif kind != "largest" and where == "v":                   # the poisoned block, and no other
                    hit = out[i, h, :32]
                    assert (~torch.isfinite(hit) | (hit.abs() > 2.0 ** 100)).any()
                    _check_row(out[i, h, 32:], lse[i, h], q[i, h], kk, vv[:, 32:], dim ** -0.5, weights)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,group", [(1, 2), (6, 3), (70, 3)])
def test_poisoned_prefix(dim, rows, group):
    """A NaN that every row sees: in a key it makes the rows NaN, in a value its block of them."""
    n, heads = 150, 2
    q = torch.randn(rows, heads * group, dim, generator=torch.Generator().manual_seed(2)).bfloat16()
    for where in "kv":
        k, v = (x.float() for x in _kv(n, heads, dim, 6))
        (k if where == "k" else v)[9, :, 37] = math.nan
        written = _written(k.bfloat16(), v.bfloat16())
        for ws, weights in _kinds(rows, group, dim):
            out, lse = _run(q, written, heads, dim ** -0.5, ws)
            if where == "k":
                assert torch.isnan(out).all() and torch.isnan(lse).all()
                continue
            assert torch.isnan(out[..., 32:64]).all() and torch.isfinite(lse).all()
            rest = [d for d in range(dim) if not 32 <= d < 64]
            for i in range(rows):
                for h in range(heads * group):
                    kk, vv = (x[:n - rows + i + 1, h // group] for x in written[2])
                    s = torch.softmax(kk @ q[i, h].double() * dim ** -0.5, 0)
                    want, mag = s @ vv[:, rest], s @ vv[:, rest].abs()
                    assert ((out[i, h, rest] - want).abs() <= 2.0 ** -8 * want.abs() + (weights + 2.0 ** -20) * mag).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_nan_and_infinity_in_the_cache(dim):
    """A block that holds a NaN has exponent 255 and reads back as NaN; an infinity reads back as infinity; other
    blocks and tokens are as without."""
    k, v = _kv(20, 2, dim, 3)
    clean = _written(k, v)
    k, v = k.clone(), v.clone()
    k[3, 1, 40], v[17, 0, 1] = math.nan, math.nan
    k[4, 0, 2], v[0, 1, 33] = math.inf, -math.inf
    k[5, 0, 0] = torch.tensor([0x7F81], dtype=torch.int16).view(torch.bfloat16)[0]      # a NaN of the smallest mantissa
    written = _written(k, v)
    at = ref.places(dim)
    got, was = (c[0].cpu().view(2, 2, 17 * dim)[c[1][0].cpu().long()] for c in (written, clean))   # group, head, byte
    assert got[0, 1, at["ke"][3, 1]] == 255 and got[1, 0, at["ve"][1, 0]] == 255 and got[0, 0, at["ke"][5, 0]] == 255
    assert got[0, 0, at["ke"][4, 0]] == 253 and got[0, 1, at["ve"][0, 1]] == 253
    gk, gv = fp8mm.mxfp4_kv_gather(*written[:2], _i32([0, 20]), 16, dim, 20)
    wk, wv = fp8mm.mxfp4_kv_gather(*clean[:2], _i32([0, 20]), 16, dim, 20)
    assert torch.isnan(gk[3, 1, 32:64]).all() and torch.isnan(gv[17, 0, :32]).all() and torch.isnan(gk[5, 0, :32]).all()
    assert gk[4, 0, 2] == math.inf and gv[0, 1, 33] == -math.inf
    for x, y, blocks in ((gk, wk, ((3, 1, 1), (5, 0, 0), (4, 0, 0))), (gv, wv, ((17, 0, 0), (0, 1, 1)))):
        for t, h, b in blocks:
            y[t, h, 32 * b:32 * b + 32] = x[t, h, 32 * b:32 * b + 32]
        same = (x == y) | (torch.isnan(x) & torch.isnan(y))
        assert same.all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [2, 40])
@pytest.mark.parametrize("scale", [1e-35, -1e-35, 1e-40])
def test_scales_of_any_size(dim, rows, scale):
    """Scales below 1e-30 with queries that make scores of them."""
    n, heads, group = 150, 2, 3
    written = _written(*_kv(n, heads, dim, 6))
    # scores of some tens; for 1e-40 below 1e-2, since products have to be within fp32
    size = min(0.1 / abs(scale), 2.0 ** 117)
    q = torch.randn(rows, heads * group, dim, generator=torch.Generator().manual_seed(2)) * size
    q = q.bfloat16()
    for ws, weights in _kinds(rows, group, dim):
        out, lse = _run(q, written, heads, scale, ws)
        for i in range(rows):
            for h in range(heads * group):
                kk, vv = (x[:n - rows + i + 1, h // group] for x in written[2])
                # the call's scale is a float
                _check_row(out[i, h], lse[i, h], q[i, h], kk, vv, float(np.float32(scale)), weights)


def _scored(n, heads, dim, scores, sizes, seed=6):
    """Keys whose scores under a query of ones in its first 32 elements are `scores` (natural units, scale 1, to 3 bits),
    and values of magnitude `sizes`, by token."""
    g = torch.Generator().manual_seed(seed)
    k = 0.01 * torch.randn(n, heads, dim, generator=g)
    k[..., :32] = (torch.tensor(scores) / 32).view(n, 1, 1)
    v = torch.randn(n, heads, dim, generator=g) * torch.tensor(sizes).view(n, 1, 1)
    return _written(k.bfloat16(), v.bfloat16())


def _check_ones(written, rows, group, dim):
    n, heads, _ = written[2][0].shape
    q = 0.5 * torch.randn(rows, heads * group, dim, generator=torch.Generator().manual_seed(2))
    q[..., :32] = 1.0
    q = q.bfloat16()
    for ws, weights in _kinds(rows, group, dim):
        out, lse = _run(q, written, heads, 1.0, ws)
        for i in range(rows):
            for h in range(heads * group):
                k, v = (x[:n - rows + i + 1, h // group] for x in written[2])
                _check_row(out[i, h], lse[i, h], q[i, h], k, v, 1.0, weights)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,group", [(1, 1), (1, 4), (2, 4), (3, 5), (40, 3)])
@pytest.mark.parametrize("huge,large", [(3, 54), (19, 38), (3, 38), (35, 54), (54, 3)])
def test_huge_values_of_no_weight(dim, rows, group, huge, large):
    """A token of values 2^40 whose score is 40 below that of another one (2^-58 of its weight), in either half of a step of
    32 tokens, before it and after."""
    n = 64 + rows - 1
    scores, sizes = [-45.0] * n, [1.0] * n
    scores[huge], sizes[huge] = -40.0, 2.0 ** 40
    scores[large] = 0.0
    _check_ones(_scored(n, 2, dim, scores, sizes), rows, group, dim)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,group", [(1, 1), (1, 4), (2, 4), (3, 5), (40, 3)])
@pytest.mark.parametrize("size,score", [(2.0 ** -30, -22.0), (2.0 ** -20, -16.0), (2.0 ** -40, -28.0)])
def test_a_large_weight_of_small_values(dim, rows, group, size, score):
    """The first token has nearly all of the weight and values so small that the others', of 2^-23 to 2^-40 of its weight,
    matter as much."""
    n = 400
    g = torch.Generator().manual_seed(1)
    scores, sizes = (score + torch.rand(n, generator=g)).tolist(), [1.0] * n
    scores[0], sizes[0] = 0.0, size
    _check_ones(_scored(n, 2, dim, scores, sizes), rows, group, dim)
