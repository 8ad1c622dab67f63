"""The cache's kernels, which are launched early with programmatic dependent
launch, behind the kernel right before them on the stream: each reads what that
one wrote, and writes only what that one has read.  Every case runs a chain of
calls without a wait between them, and the same with a wait after each call: the
results have the same bits."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_fp8_b200 as fp8mm
from tests import gpu_util as gu
from tests.test_gpu_kv4 import _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gu.require_gpu()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert fp8mm.last_device_error() == 0


def _randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def _both(chain, times=3):
    """The chain's results with and without a wait after each call, several times."""
    want = [t.clone() for t in chain(torch.cuda.synchronize)]
    for _ in range(times):
        got = chain(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_norm_reads_and_writes_in_order():
    """Queries and positions written by the kernel right before; a result that the kernel right before still reads."""
    t, hq, hk, dim = 4096, 8, 2, 128
    x0, pos0 = _randn(t, hq + hk, dim, seed=1), torch.arange(t, dtype=torch.int32, device="cuda")
    ang = torch.arange(t, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, dim, 2, device="cuda").double() / dim)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()

    def chain(wait):
        x, pos, out, kept = torch.empty_like(x0), torch.empty_like(pos0), x0 * 2, []
        wait()
        for scale in (1.0, -3.0, 0.25):
            torch.mul(x0, scale, out=x)
            wait()
            pos.copy_(pos0 if scale > 0 else pos0.flip(0))
            wait()
            kept.append(out.clone())                           # reads what the next call overwrites
            wait()
            fp8mm.qk_norm_rope(x[:, :hq], x[:, hq:], cs, pos, q_out=out[:, :hq], k_out=out[:, hq:])
            wait()
            kept.append(out.clone())
            wait()
        return kept

    _both(chain)


@pytest.mark.parametrize("new,length", [(1, 3000), (70, 3000)])
def test_a_cache_is_read_and_rewritten_in_order(new, length):
    """Append, attention (either kernel and the join of cut tiles), append of other tokens over the same records, page
    copy over pages that the attention read, read back, attention."""
    dim, hq, hk, ps, batch = 128, 8, 2, 64, 4
    per = -(-length // ps)
    table = torch.randperm(2 * batch * per, generator=torch.Generator().manual_seed(1))
    first, second = (_i32(x.view(batch, per).tolist()) for x in (table[:batch * per], table[batch * per:]))
    lens, all_rows = _i32([length] * batch), _i32([i * length for i in range(batch + 1)])
    cu = _i32([i * new for i in range(batch + 1)])
    k, v = (_randn(batch * length, hk, dim, seed=i) for i in (2, 3))
    q = _randn(batch * new, hq, dim, seed=4)
    tails = [tuple(_randn(batch * new, hk, dim, seed=s + i) for i in (0, 1)) for s in (5, 7)]
    cache = torch.zeros(2 * batch * per, fp8mm.mxfp4_kv_page_bytes(ps, hk, dim), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(fp8mm.mxfp4_kv_attention_workspace_bytes(dim), dtype=torch.uint8, device="cuda")
    moves = first.flatten().tolist(), second.flatten().tolist()

    def chain(wait):
        kept, x = [], torch.empty_like(q)
        cache.zero_()
        wait()
        fp8mm.mxfp4_kv_append(k, v, cache, first, lens, ps, all_rows)
        wait()
        for i, (tk, tv) in enumerate(tails):
            torch.mul(q, 1.0 + i, out=x)                       # queries written right before
            wait()
            kept.append(fp8mm.mxfp4_kv_attention(x, cache, first, lens, ps, cu, workspace=ws))
            wait()
            fp8mm.mxfp4_kv_append(tk, tv, cache, first, lens, ps, cu)    # over records that the attention reads
            wait()
            kept.append(fp8mm.mxfp4_kv_attention(x, cache, first, lens, ps, cu))
            wait()
        fp8mm.kv_copy_pages(cache, *moves)
        wait()
        kept.append(fp8mm.mxfp4_kv_attention(x, cache, second, lens, ps, cu, workspace=ws))
        wait()
        fp8mm.kv_copy_pages(cache, moves[0][::-1], moves[1])   # over pages that the attention reads
        wait()
        kept += fp8mm.mxfp4_kv_gather(cache, second, all_rows, ps, dim, batch * length)
        wait()
        cache.fill_(17)                                        # over pages that the read back reads
        wait()
        return kept + [cache]

    _both(chain)
