"""Argument checks of the append and attention calls, in C and in the binding
(CPU only: no call here reaches the GPU)."""

import ctypes

import pytest
import torch

A = 1 << 20   # a 256-byte-aligned stand-in address (never dereferenced)


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_indexer_score_gb300 import build
    try:
        build.build()
    except RuntimeError as e:   # no nvcc on this machine
        pytest.skip(str(e))
    from sparse_attention_indexer_score_gb300 import dsa as d
    d._lib = None
    d.lib()
    return d


def cache(dsa, **kw):
    f = dict(k=A, v=A, k_page_stride=64 * 256, k_token_stride=256, k_head_stride=128, v_page_stride=64 * 256,
             v_token_stride=256, v_head_stride=128, num_pages=4, heads=2, dim=128, dtype=0)
    f.update(kw)
    return dsa.KvCache(**f)


APPEND = dict(k=A, kt=256, kh=128, v=A, vt=256, vh=128, q=A, qt=1024, qh=128, q_heads=8, q_out=A, ot=1024, oh=128,
              n=3, slots=A, positions=A, cos_sin=A, cs=128, max_pos=10, rot=128, inter=0, status=None, stream=None)
PAGED = dict(q=A, qr=1024, qh=128, heads=8, bt=A, bts=4, pages=4, starts=A, ends=A, R=1, rows=1, mq=1, pp=None, pl=0,
             scale=0.1, out=A, orow=1024, oh=128, lse=None, ws=A, wsb=1 << 40, status=None, stream=None)
SELECTED = dict(q=A, qr=1024, qh=128, heads=8, bt=A, bts=4, pages=4, starts=A, ends=A, R=1, rows=1, topk=A, ts=16,
                k=16, scale=0.1, out=A, orow=1024, oh=128, lse=None, ws=A, wsb=1 << 40, status=None, stream=None)


def call(dsa, fn, base, cache_kw=None, **kw):
    args = dict(base)
    assert set(kw) <= set(args)
    args.update(kw)
    c = cache(dsa, **(cache_kw or {}))
    return getattr(dsa.lib(), fn)(ctypes.addressof(c), *args.values())


BAD_CACHE = [(dict(num_pages=-1), -1), (dict(heads=0), -1), (dict(dim=0), -1), (dict(dim=100), -2),
             (dict(dim=528), -2), (dict(dtype=2), -2), (dict(k=None), -1), (dict(v=None), -1), (dict(k=A + 8), -1),
             (dict(v=A + 2), -1), (dict(k_page_stride=100), -1), (dict(v_token_stride=-256), -1),
             (dict(v_head_stride=4), -1), (dict(num_pages=1 << 31), -2)]


@pytest.mark.parametrize("kw,rc", BAD_CACHE)
def test_every_call_refuses_a_bad_cache(dsa, kw, rc):
    assert call(dsa, "dsa_kv_append", APPEND, kw) == rc
    assert call(dsa, "dsa_attend_paged", PAGED, kw) == rc
    assert call(dsa, "dsa_attend_selected", SELECTED, kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(n=-1), -1), (dict(rot=-16), -1), (dict(rot=144), -1), (dict(rot=24), -2), (dict(inter=2), -1),
    (dict(q=None), -1), (dict(q_out=None), -1), (dict(q_heads=0), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(slots=None), -1), (dict(positions=None), -1), (dict(cos_sin=None), -1), (dict(max_pos=0), -1),
    (dict(cs=64), -1), (dict(cs=130), -1), (dict(k=A + 2), -1), (dict(v=A + 4), -1), (dict(q=A + 8), -1),
    (dict(q_out=A + 8), -1), (dict(cos_sin=A + 4), -1), (dict(kt=257), -1), (dict(vh=132), -1), (dict(qt=1020), -1),
    (dict(oh=4), -1), (dict(n=0), 0)])
def test_append_arguments(dsa, kw, rc):
    assert call(dsa, "dsa_kv_append", APPEND, None, **kw) == rc


COMMON = [(dict(heads=0), -1), (dict(heads=9), -1), (dict(heads=2 * 129), -2), (dict(rows=-1), -1), (dict(R=-1), -1),
          (dict(pages=-1), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("inf")), -1),
          (dict(scale=float("nan")), -1), (dict(q=None), -1), (dict(out=None), -1), (dict(starts=None), -1),
          (dict(ends=None), -1), (dict(ws=None), -1), (dict(bt=None), -1), (dict(bts=3), -1), (dict(q=A + 2), -1),
          (dict(out=A + 8), -1), (dict(ws=A + 16), -1), (dict(qr=1028), -1), (dict(qh=4), -1), (dict(orow=1025), -1),
          (dict(oh=-128), -1), (dict(wsb=0), -1), (dict(rows=0), 0), (dict(rows=1 << 25), -2)]


@pytest.mark.parametrize("kw,rc", COMMON + [(dict(mq=-1), -1), (dict(pl=-1), -1), (dict(pl=64), -1)])
def test_attend_paged_arguments(dsa, kw, rc):
    assert call(dsa, "dsa_attend_paged", PAGED, None, **kw) == rc


@pytest.mark.parametrize("kw,rc", COMMON + [(dict(k=-1), -1), (dict(topk=None), -1), (dict(ts=15), -1)])
def test_attend_selected_arguments(dsa, kw, rc):
    assert call(dsa, "dsa_attend_selected", SELECTED, None, **kw) == rc


def test_attention_refuses_wide_heads(dsa):
    wide = dict(dim=144)
    assert call(dsa, "dsa_attend_paged", PAGED, wide) == -2
    assert call(dsa, "dsa_attend_selected", SELECTED, wide) == -2


def test_workspace_sizes(dsa):
    f = dsa.attend_workspace_size
    assert 0 < f(64, 64, 32, 8, 128, 1) <= f(128, 128, 32, 8, 128, 4)
    assert f(64, 64, 32, 8, 128, 1, 2048) > 0
    for bad in [(-1, 1, 8, 2, 128, 1), (1, -1, 8, 2, 128, 1), (1, 1, 9, 2, 128, 1), (1, 1, 8, 0, 128, 1),
                (1, 1, 8, 2, 100, 1), (1, 1, 8, 2, 144, 1), (1, 1, 129, 1, 128, 1), (1, 1, 8, 2, 128, -1)]:
        assert f(*bad) == 0


def tensors(dt=torch.bfloat16):
    z = torch.zeros
    return dict(q=z(2, 8, 64, dtype=dt), k_cache=z(3, 64, 2, 64, dtype=dt), v_cache=z(3, 64, 2, 64, dtype=dt),
                block_table=z(1, 3, dtype=torch.int32), starts=z(2, dtype=torch.int32),
                row_ends=z(2, dtype=torch.int32))


@pytest.mark.parametrize("name,value", [
    ("q", torch.zeros(2, 8, 64)), ("q", torch.zeros(2, 8, 32, dtype=torch.bfloat16)),
    ("q", torch.zeros(2, 64, 8, dtype=torch.bfloat16).transpose(1, 2)),
    ("k_cache", torch.zeros(3, 64, 2, 64)), ("v_cache", torch.zeros(3, 64, 2, 64, dtype=torch.float16)),
    ("k_cache", torch.zeros(3, 32, 2, 64, dtype=torch.bfloat16)),
    ("v_cache", torch.zeros(2, 64, 2, 64, dtype=torch.bfloat16)),
    ("block_table", torch.zeros(1, 3, dtype=torch.int64)), ("block_table", torch.zeros(2, 3, dtype=torch.int32)),
    ("block_table", torch.zeros(3, 1, dtype=torch.int32).t()[:, :0].expand(1, 0).t()),
    ("starts", torch.zeros(2, dtype=torch.int64)), ("row_ends", torch.zeros(3, dtype=torch.int32))])
def test_the_binding_refuses_other_tensors(dsa, name, value):
    t = tensors()
    t[name] = value
    with pytest.raises(ValueError):
        dsa.attend_paged(**t, max_query_len=1)
    with pytest.raises(ValueError):
        dsa.attend_selected(**t, topk=torch.zeros(2, 4, dtype=torch.int32))


def test_the_binding_refuses_other_lists(dsa):
    t = tensors()
    for topk in (torch.zeros(2, 4, dtype=torch.int64), torch.zeros(3, 4, dtype=torch.int32),
                 torch.zeros(4, 2, dtype=torch.int32).t()):
        with pytest.raises(ValueError):
            dsa.attend_selected(**t, topk=topk)
    for pages in (None, torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)):
        with pytest.raises(ValueError):
            dsa.attend_paged(**t, max_query_len=1, prefix_pages=pages, prefix_len=65)
    with pytest.raises(ValueError):
        dsa.attend_paged(**t, max_query_len=1, out=torch.zeros(2, 8, 64))


def test_the_binding_refuses_other_append_tensors(dsa):
    bf = torch.bfloat16
    good = dict(k=torch.zeros(3, 2, 64, dtype=bf), v=torch.zeros(3, 2, 64, dtype=bf),
                slots=torch.zeros(3, dtype=torch.int64), k_cache=torch.zeros(2, 64, 2, 64, dtype=bf),
                v_cache=torch.zeros(2, 64, 2, 64, dtype=bf), positions=torch.zeros(3, dtype=torch.int64),
                cos_sin=torch.zeros(9, 64), q=torch.zeros(3, 4, 64, dtype=bf))
    for name, value in [("k", torch.zeros(3, 2, 64)), ("v", torch.zeros(2, 2, 64, dtype=bf)),
                        ("k", torch.zeros(3, 1, 64, dtype=bf)), ("slots", torch.zeros(3, dtype=torch.int32)),
                        ("slots", torch.zeros(2, dtype=torch.int64)), ("positions", None),
                        ("positions", torch.zeros(3, dtype=torch.int32)), ("cos_sin", torch.zeros(9, 64).double()),
                        ("q", torch.zeros(2, 4, 64, dtype=bf)), ("q", torch.zeros(3, 4, 32, dtype=bf)),
                        ("q_out", torch.zeros(3, 4, 64))]:
        bad = dict(good)
        bad[name] = value
        with pytest.raises(ValueError):
            dsa.kv_append(**bad)
    with pytest.raises(ValueError):
        dsa.kv_append(**dict(good, q=None, q_out=torch.zeros(3, 4, 64, dtype=bf)))


def test_the_binding_fails_loudly_without_its_extension(dsa, monkeypatch):
    import builtins
    import sys

    monkeypatch.setattr(dsa, "_binding", None)
    monkeypatch.delitem(sys.modules, "sparse_attention_indexer_score_gb300._dsa_binding", raising=False)
    package = sys.modules["sparse_attention_indexer_score_gb300"]
    monkeypatch.delattr(package, "_dsa_binding", raising=False)
    real = builtins.__import__

    def missing(name, globals=None, locals=None, fromlist=(), level=0):
        if fromlist and "_dsa_binding" in fromlist:
            raise ImportError("no _dsa_binding")
        return real(name, globals, locals, fromlist, level)

    monkeypatch.setattr(builtins, "__import__", missing)
    with pytest.raises(RuntimeError, match="missing"):
        dsa.attend_paged(**tensors(), max_query_len=1)


def test_the_binding_refuses_cpu_tensors_and_other_numbers(dsa):
    t = tensors()
    with pytest.raises(ValueError, match="CUDA"):
        dsa.attend_paged(**t, max_query_len=1, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    for bad in (dict(max_query_len="1"), dict(max_query_len=1, scale="x"), dict(max_query_len=1, prefix_len=None),
                dict(max_query_len=1, status=torch.zeros(1)), dict(max_query_len=1, q=None)):
        with pytest.raises(ValueError):
            dsa.attend_paged(**{**t, **bad})
