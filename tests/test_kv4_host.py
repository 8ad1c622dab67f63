"""The cache operators without a GPU: what the library and the binding refuse,
the cache description's layout, the page pool, and the 64-bit references'
own checks."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_fp8_b200 as fp8mm
from mxfp8_block_scaled_fp8_b200 import fp8mm as binding
from tests import kv4_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20                                                 # never dereferenced
OK, NULL, SHAPE, ALIGN = 0, 1, 2, 3
FIELDS = ("pages", "page_stride", "num_pages", "page_size", "kv_heads", "head_dim", "page_table", "table_stride",
          "max_pages", "batch")
DESC = dict(pages=FAKE, page_stride=64 // 16 * 2 * 17 * 128, num_pages=9, page_size=64, kv_heads=2, head_dim=128,
            page_table=FAKE, table_stride=4, max_pages=4, batch=3)


def _desc(**change):
    return binding.KV_CACHE_DESC.pack(*({**DESC, **change}[f] or 0 for f in FIELDS))


BAD_CACHES = [(SHAPE, dict(head_dim=96)), (SHAPE, dict(page_size=24)), (SHAPE, dict(page_size=8)),
              (SHAPE, dict(page_size=8192, page_stride=1 << 30)), (SHAPE, dict(kv_heads=0)),
              (SHAPE, dict(kv_heads=65536, page_stride=1 << 40)), (SHAPE, dict(num_pages=-1)),
              (SHAPE, dict(num_pages=1 << 31)), (SHAPE, dict(batch=-1)), (SHAPE, dict(max_pages=-1)),
              (SHAPE, dict(table_stride=3)), (SHAPE, dict(max_pages=1 << 26, table_stride=1 << 26)),
              (SHAPE, dict(page_stride=DESC["page_stride"] - 16)), (NULL, dict(pages=None)), (NULL, dict(page_table=None)),
              (ALIGN, dict(pages=FAKE + 8)), (ALIGN, dict(page_stride=DESC["page_stride"] + 8)),
              (ALIGN, dict(page_table=FAKE + 2))]


def _append(desc=None, k=FAKE, kt=256, kh=128, v=FAKE, vt=256, vh=128, rows=3, cu=None, lens=FAKE):
    return binding.lib().mxfp4_kv_append(k, kt, kh, v, vt, vh, rows, cu, lens, desc or _desc(), None)


def _gather(desc=None, starts=None, cu=FAKE, rows=3, k=FAKE, kt=256, kh=128, v=FAKE, vt=256, vh=128):
    return binding.lib().mxfp4_kv_gather(desc or _desc(), starts, cu, rows, k, kt, kh, v, vt, vh, None)


def _attention(desc=None, q=FAKE, qt=512, qh=128, rows=3, heads=4, cu=None, lens=FAKE, scale=0.1, out=FAKE, ot=512, oh=128,
               lse=None, ls=4, ws=None, wsb=0):
    return binding.lib().mxfp4_kv_attention(q, qt, qh, rows, heads, cu, lens, desc or _desc(), scale, out, ot, oh, lse, ls,
                                            ws, wsb, None)


def _norm(q=FAKE, qt=512, qh=128, k=FAKE, kt=256, kh=128, tokens=3, hq=4, hk=2, dim=128, qw=None, kw=None, eps=1e-6,
          cs=FAKE, most=10, rot=64, css=64, inter=0, pos=FAKE, qo=FAKE, qot=512, qoh=128, ko=FAKE, kot=256, koh=128):
    return binding.lib().qk_norm_rope(q, qt, qh, k, kt, kh, tokens, hq, hk, dim, qw, kw, eps, cs, most, rot, css, inter, pos,
                                      qo, qot, qoh, ko, kot, koh, None)


def _copy(pages=FAKE, num=8, nbytes=64, stride=64, layers=2, layer_stride=512, src=(1, 2), dst=(3, 4), moves=None):
    a, b = ((ctypes.c_int32 * max(len(x), 1))(*x) for x in (src, dst))
    return binding.lib().kv_copy_pages(pages, num, nbytes, stride, layers, layer_stride, ctypes.addressof(a),
                                       ctypes.addressof(b), len(src) if moves is None else moves, None)


@pytest.mark.parametrize("status,change", BAD_CACHES)
def test_bad_caches(status, change):
    for call in (_append, _gather, _attention):
        assert call(_desc(**change)) == status, call


def test_no_cache():
    L = binding.lib()
    assert L.mxfp4_kv_append(FAKE, 256, 128, FAKE, 256, 128, 3, None, FAKE, None, None) == NULL
    assert L.mxfp4_kv_gather(None, None, FAKE, 3, FAKE, 256, 128, FAKE, 256, 128, None) == NULL
    assert L.mxfp4_kv_attention(FAKE, 512, 128, 3, 4, None, FAKE, None, 0.1, FAKE, 512, 128, None, 4, None, 0, None) == NULL


def test_append_refusals():
    assert _append(rows=-1) == SHAPE and _append(rows=4) == SHAPE and _append(rows=1 << 31, cu=FAKE) == SHAPE
    assert _append(lens=None) == NULL and _append(k=None) == NULL and _append(v=None) == NULL
    assert _append(kt=-256) == SHAPE and _append(kh=64) == SHAPE and _append(vh=-128) == SHAPE
    assert _append(k=FAKE + 8) == ALIGN and _append(vt=260) == ALIGN and _append(kh=132) == ALIGN
    assert _append(cu=FAKE + 1) == ALIGN and _append(lens=FAKE + 2) == ALIGN
    assert _append(k=None, v=None, lens=None, rows=0, cu=FAKE) == OK
    assert _append(_desc(batch=0), k=None, v=None, lens=None, rows=0) == OK


def test_gather_refusals():
    assert _gather(rows=-1) == SHAPE and _gather(cu=None) == NULL and _gather(k=None) == NULL and _gather(v=None) == NULL
    assert _gather(kt=64) == SHAPE and _gather(vh=64) == SHAPE                  # an output's rows may not overlap
    assert _gather(k=FAKE + 8) == ALIGN and _gather(vt=260) == ALIGN and _gather(starts=FAKE + 2) == ALIGN
    assert _gather(rows=0, cu=None, k=None, v=None) == OK


def test_attention_refusals():
    assert _attention(rows=-1) == SHAPE and _attention(rows=4) == SHAPE
    assert _attention(heads=0) == SHAPE and _attention(heads=3) == SHAPE and _attention(heads=1 << 17) == SHAPE
    for scale in (float("nan"), float("inf"), -3e38):                           # 3e38 log2 e is not a float
        assert _attention(scale=scale) == SHAPE, scale
    assert _attention(lens=None) == NULL and _attention(q=None) == NULL and _attention(out=None) == NULL
    assert _attention(ot=64) == SHAPE and _attention(oh=64) == SHAPE and _attention(qh=64) == SHAPE
    assert _attention(lse=FAKE, ls=3) == SHAPE
    assert _attention(q=FAKE + 8) == ALIGN and _attention(ot=516) == ALIGN and _attention(lse=FAKE + 2) == ALIGN
    assert _attention(cu=FAKE + 2) == ALIGN and _attention(lens=FAKE + 1) == ALIGN
    assert _attention(ws=FAKE + 128, wsb=1 << 30) == ALIGN
    assert _attention(rows=0, cu=FAKE, q=None, out=None, lens=None) == OK
    L = binding.lib()
    assert L.mxfp4_kv_attention_workspace_bytes(96) == 0
    assert 0 < L.mxfp4_kv_attention_workspace_bytes(64) < L.mxfp4_kv_attention_workspace_bytes(128)


def test_norm_refusals():
    assert _norm(tokens=-1) == SHAPE and _norm(dim=96) == SHAPE and _norm(hq=-1) == SHAPE and _norm(hq=65535) == SHAPE
    assert _norm(rot=8) == SHAPE and _norm(rot=24) == SHAPE and _norm(rot=256) == SHAPE and _norm(css=32) == SHAPE
    assert _norm(most=0) == SHAPE and _norm(most=1 << 31) == SHAPE and _norm(inter=2) == SHAPE
    assert _norm(eps=-1.0) == SHAPE and _norm(eps=float("nan")) == SHAPE and _norm(eps=float("inf")) == SHAPE
    assert _norm(cs=None) == NULL and _norm(pos=None) == NULL and _norm(qw=FAKE) == NULL and _norm(kw=FAKE) == NULL
    assert _norm(q=None) == NULL and _norm(ko=None) == NULL and _norm(qot=64) == SHAPE and _norm(kh=64) == SHAPE
    assert _norm(q=FAKE + 8) == ALIGN and _norm(kot=260) == ALIGN and _norm(cs=FAKE + 8) == ALIGN
    assert _norm(css=66) == ALIGN and _norm(pos=FAKE + 2) == ALIGN and _norm(qw=FAKE + 8, kw=FAKE) == ALIGN
    assert _norm(tokens=0, q=None, k=None, cs=None, pos=None, qo=None, ko=None) == OK
    assert _norm(hq=0, hk=0) == OK


def test_copy_refusals():
    assert _copy(num=-1) == SHAPE and _copy(nbytes=-16) == SHAPE and _copy(layers=-1) == SHAPE and _copy(moves=-1) == SHAPE
    assert _copy(moves=9) == SHAPE and _copy(nbytes=1 << 31, stride=1 << 31) == SHAPE
    assert _copy(stride=48) == SHAPE and _copy(layer_stride=48) == SHAPE
    assert _copy(layer_stride=64) == SHAPE and _copy(layer_stride=448) == SHAPE           # layers overlap
    assert _copy(pages=None) == NULL and _copy(pages=FAKE + 8) == ALIGN and _copy(nbytes=56) == ALIGN
    assert _copy(src=(1, 8)) == SHAPE and _copy(src=(-1, 2)) == SHAPE and _copy(dst=(3, 8)) == SHAPE
    assert _copy(dst=(3, 3)) == SHAPE                                                     # written twice
    assert _copy(dst=(3, 1)) == SHAPE and _copy(src=(1,), dst=(1,)) == SHAPE              # read and written
    assert _copy(src=(), dst=()) == OK and _copy(layers=0) == OK and _copy(nbytes=0) == OK


def test_page_bytes():
    for size in (16, 48, 4096):
        for dim in (64, 128):
            assert fp8mm.mxfp4_kv_page_bytes(size, 3, dim) == size * 3 * dim * 17 // 16     # 4.25 bits, keys and values
    for bad in ((8, 1, 64), (24, 1, 64), (16, 0, 64), (16, 1, 96), (-16, 1, 64)):
        assert fp8mm.mxfp4_kv_page_bytes(*bad) == 0


def test_description_layout(tmp_path):
    """The binding packs fp8mm_kv_cache by hand: field by field where the compiler has it."""
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fp8mm.h"\nint main(void) {\n'
                   '  printf("size %zu\\n", sizeof(fp8mm_kv_cache));\n'
                   + "".join(f'  printf("{f} %zu\\n", offsetof(fp8mm_kv_cache, {f}));\n' for f in FIELDS) + "  return 0;\n}\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(out["size"]) == binding.KV_CACHE_DESC.size
    packed = binding.KV_CACHE_DESC.pack(*range(1, len(FIELDS) + 1))
    for i, f in enumerate(FIELDS):
        assert np.frombuffer(packed, np.int64, 1, int(out[f]))[0] == i + 1, f


def test_binding_refuses_tensors_off_the_gpu():
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    cache = torch.zeros(4, fp8mm.mxfp4_kv_page_bytes(16, 2, 128), dtype=torch.uint8)
    table, n = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    calls = (lambda: fp8mm.mxfp4_kv_append(x, x, cache, table, n, 16),
             lambda: fp8mm.mxfp4_kv_gather(cache, table, torch.zeros(4, dtype=torch.int32), 16, 128, 3),
             lambda: fp8mm.mxfp4_kv_attention(x, cache, table, n, 16),
             lambda: fp8mm.kv_copy_pages(cache, [0], [1]),
             lambda: fp8mm.qk_norm_rope(x, x, torch.zeros(4, 128), n))
    for call in calls:
        with pytest.raises(TypeError):
            call()


# ------------------------------------------------------------------ the page pool

def test_pool_gives_and_takes():
    pool = fp8mm.KvPagePool(5, 16)
    assert [pool.pages_for(n) for n in (0, 1, 16, 17)] == [0, 1, 1, 2]
    a = pool.allocate(3)
    assert a == [0, 1, 2] and pool.free_pages == 2 and pool.allocate(0) == []
    with pytest.raises(MemoryError):
        pool.allocate(3)
    assert pool.free_pages == 2
    pool.free([1])
    assert pool.allocate(1) == [1]                              # the lowest first
    for bad in ([3], [5], [-1], [0, 0], [0, 3]):
        with pytest.raises(ValueError):
            pool.free(bad)
    assert [pool.references(p) for p in range(5)] == [1, 1, 1, 0, 0]
    for bad in (lambda: pool.allocate(-1), lambda: pool.pages_for(-1), lambda: pool.references(5),
                lambda: fp8mm.KvPagePool(-1, 16), lambda: fp8mm.KvPagePool(1, 24), lambda: fp8mm.KvPagePool(1, 8192)):
        with pytest.raises(ValueError):
            bad()
    empty = fp8mm.KvPagePool(0, 16)
    assert empty.allocate(0) == [] and empty.compact() == ([], [], {})


def test_pool_forks():
    pool = fp8mm.KvPagePool(6, 16)
    a = pool.allocate(3)
    child, src, dst = pool.fork(a, 40)                          # two full pages, half a third
    assert child == [0, 1, 3] and (src, dst) == ([2], [3])
    whole, src, dst = pool.fork(a, 32)                          # ends with a page: nothing to copy, the third is left
    assert whole == [0, 1] and src == dst == []
    assert [pool.references(p) for p in range(6)] == [3, 3, 1, 1, 0, 0]
    assert pool.fork([], 0) == ([], [], [])
    pool.free(a)
    assert [pool.references(p) for p in range(4)] == [2, 2, 0, 1] and pool.free_pages == 3
    pool.allocate(3)
    with pytest.raises(MemoryError):
        pool.fork(child, 33)                                    # no page for the copy
    assert [pool.references(p) for p in range(2)] == [2, 2]     # and nothing was shared
    for pages, n in (([0], 17), ([9], 3)):
        with pytest.raises(ValueError):
            pool.fork(pages, n)
    pool.free(child + whole)
    with pytest.raises(ValueError):
        pool.fork([0], 16)                                      # a free page


@pytest.mark.parametrize("seed", range(4))
def test_pool_compaction_moves_what_a_table_reads(seed):
    """Random lives of sequences against a plain model: the bytes that a list of pages reads survive forks, frees and
    compactions, and no move reads a page that another writes."""
    rng = np.random.default_rng(seed)
    pool, data = fp8mm.KvPagePool(40, 16), np.arange(40)
    live, stamp = {}, 1000
    for step in range(200):
        what = rng.integers(4)
        if what == 0 and pool.free_pages >= 4:
            pages = pool.allocate(int(rng.integers(5)))
            for p in pages:
                data[p] = stamp
                stamp += 1
            live[step] = (pages, [int(data[p]) for p in pages])
        elif what == 1 and live and pool.free_pages:
            pages, want = live[int(rng.choice(list(live)))]
            n = int(rng.integers(16 * len(pages) + 1))
            child, src, dst = pool.fork(pages, n)
            data[dst] = data[src]
            live[step] = (child, want[:len(child)])
        elif what == 2 and live:
            pool.free(live.pop(int(rng.choice(list(live))))[0])
        else:
            src, dst, moved = pool.compact()
            assert not set(src) & set(dst) and len(set(dst)) == len(dst)
            data[dst] = data[src]
            live = {k: ([moved.get(p, p) for p in pages], want) for k, (pages, want) in live.items()}
            held = {p for pages, _ in live.values() for p in pages}
            assert held == set(range(len(held)))
        for pages, want in live.values():
            assert [int(data[p]) for p in pages] == want
        count = np.bincount([p for pages, _ in live.values() for p in pages], minlength=40)
        assert [pool.references(p) for p in range(40)] == count.tolist()
        assert pool.free_pages == int((count == 0).sum())


# ------------------------------------------------------------------ the references

@pytest.mark.parametrize("dim", [64, 128])
def test_reference_places_fill_a_record(dim):
    """Every half byte of a record's codes belongs to one code, every byte of its exponents to one exponent."""
    at, halves = ref.places(dim), np.zeros((17 * dim, 2), dtype=int)
    for name in ("k", "v"):
        byte, shift = np.broadcast_arrays(*at[name])
        np.add.at(halves, (byte, shift // 4), 1)
    for name in ("ke", "ve"):
        np.add.at(halves, at[name], 1)
    assert (halves == 1).all()


def test_reference_quantizer_takes_the_smallest_exponent():
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(50, 64, generator=g) * torch.exp(torch.randn(50, 1, generator=g) * 8)).bfloat16()
    x[0] = 0
    codes, e = ref.quantize(x)
    amax = x.double().abs().reshape(50, 2, 32).amax(-1)
    e = e.double().reshape(50, 2)
    zero = amax == 0
    assert (e[zero] == 0).all()
    assert (6 * 2.0 ** (e - 127) >= amax).all() and (6 * 2.0 ** (e - 128) < amax)[~zero].all()


def test_page_bytes_of_sizes_that_calls_refuse():
    """0 for the sizes that append, gather and attention refuse, up to the largest that they take."""
    assert fp8mm.mxfp4_kv_page_bytes(4096, 65535, 128) == 4096 // 16 * 65535 * 17 * 128
    for bad in ((4112, 1, 64), (8192, 2, 128), (16, 65536, 64), (1 << 40, 1, 64), (16, 1 << 60, 128)):
        assert fp8mm.mxfp4_kv_page_bytes(*bad) == 0, bad
