"""Argument checks of the 4-bit cache's calls, in C and in the binding (CPU only: no call here reaches the GPU)."""

import ctypes

import pytest
import torch

A = 1 << 20   # a 256-byte-aligned stand-in address (never dereferenced)
BF, U8, I32, I64 = torch.bfloat16, torch.uint8, torch.int32, torch.int64


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


SECTION = 64 * (128 + 16)
APPEND = dict(dtype=0, k=A, kt=256, kh=128, v=A, vt=256, vh=128, q=A, qt=1024, qh=128, q_heads=8, q_out=A, ot=1024,
              oh=128, n=3, slots=A, positions=A, cos_sin=A, cs=128, max_pos=10, rot=128, inter=0, status=None, stream=None)
READ = dict(dtype=0, slots=A, n=3, k=A, kt=256, kh=128, v=A, vt=256, vh=128, status=None, stream=None)
PAGED = dict(dtype=0, q=A, qr=1024, qh=128, heads=8, bt=A, bts=4, pages=4, starts=A, ends=A, R=1, rows=1, mq=1,
             scale=0.1, out=A, orow=1024, oh=128, lse=None, ws=A, wsb=1 << 40, status=None, stream=None)
SELECTED = dict(dtype=0, q=A, qr=1024, qh=128, heads=8, bt=A, bts=4, pages=4, starts=A, ends=A, R=1, rows=1, topk=A,
                ts=16, k=16, scale=0.1, out=A, orow=1024, oh=128, lse=None, ws=A, wsb=1 << 40, status=None, stream=None)
CALLS = dict(append=("dsa_kv_append_fp4", APPEND), read=("dsa_kv_read_fp4", READ),
             paged=("dsa_attend_paged_fp4", PAGED), selected=("dsa_attend_selected_fp4", SELECTED))


def call(dsa, which, cache_kw=None, **kw):
    fn, base = CALLS[which]
    args = dict(base)
    assert set(kw) <= set(args)
    args.update(kw)
    f = dict(data=A, page_stride=2 * SECTION, head_stride=SECTION, num_pages=4, heads=2, dim=128, k_scale=1.0, v_scale=1.0)
    f.update(cache_kw or {})
    c = dsa.KvCacheFp4(**f)
    return getattr(dsa.lib(), fn)(ctypes.addressof(c), *args.values())


@pytest.mark.parametrize("which", list(CALLS))
@pytest.mark.parametrize("kw,rc", [
    (dict(num_pages=-1), -1), (dict(heads=0), -1), (dict(dim=0), -1), (dict(dim=100), -2), (dict(dim=144), -2),
    (dict(data=None), -1), (dict(data=A + 8), -1), (dict(page_stride=2 * SECTION + 8), -1), (dict(head_stride=-SECTION), -1),
    (dict(page_stride=0), -1), (dict(head_stride=0), -1), (dict(head_stride=SECTION - 16), -1),
    (dict(page_stride=SECTION - 16), -1), (dict(num_pages=1 << 31), -2), (dict(heads=65536), -2),
    (dict(k_scale=0.0), -1), (dict(v_scale=-1.0), -1), (dict(k_scale=float("nan")), -1), (dict(v_scale=float("inf")), -1),
    (dict(k_scale=2.0 ** -65), -1), (dict(v_scale=2.0 ** 65), -1)])
def test_every_call_refuses_a_bad_cache(dsa, which, kw, rc):
    assert call(dsa, which, kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(dtype=2), -2), (dict(n=-1), -1), (dict(rot=-16), -1), (dict(rot=144), -1), (dict(rot=24), -2), (dict(inter=2), -1),
    (dict(q=None), -1), (dict(q_out=None), -1), (dict(q_heads=0), -1), (dict(q_heads=65536), -2), (dict(k=None), -1),
    (dict(v=None), -1), (dict(slots=None), -1), (dict(positions=None), -1), (dict(cos_sin=None), -1), (dict(max_pos=0), -1),
    (dict(cs=64), -1), (dict(cs=130), -1), (dict(k=A + 2), -1), (dict(v=A + 4), -1), (dict(q=A + 8), -1),
    (dict(q_out=A + 8), -1), (dict(cos_sin=A + 4), -1), (dict(kt=257), -1), (dict(vh=132), -1), (dict(qt=1020), -1),
    (dict(oh=4), -1), (dict(ot=0), -1), (dict(oh=0), -1), (dict(n=0), 0)])
def test_append_arguments(dsa, kw, rc):
    assert call(dsa, "append", None, **kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(dtype=-1), -2), (dict(n=-1), -1), (dict(slots=None), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(k=A + 8), -1), (dict(v=A + 2), -1), (dict(kt=100), -1), (dict(vh=4), -1), (dict(kt=0), -1), (dict(vh=0), -1),
    (dict(n=1 << 41), -2), (dict(n=0), 0)])
def test_read_arguments(dsa, kw, rc):
    assert call(dsa, "read", None, **kw) == rc


COMMON = [(dict(dtype=3), -2), (dict(heads=0), -1), (dict(heads=9), -1), (dict(heads=2 * 129), -2), (dict(rows=-1), -1),
          (dict(R=-1), -1), (dict(pages=-1), -1), (dict(pages=1 << 25, bts=1 << 25), -2), (dict(scale=0.0), -1),
          (dict(scale=-1.0), -1), (dict(scale=float("inf")), -1), (dict(scale=float("nan")), -1), (dict(q=None), -1),
          (dict(out=None), -1), (dict(starts=None), -1), (dict(ends=None), -1), (dict(ws=None), -1), (dict(bt=None), -1),
          (dict(bts=3), -1), (dict(q=A + 2), -1), (dict(out=A + 8), -1), (dict(ws=A + 16), -1), (dict(qr=1028), -1),
          (dict(qh=4), -1), (dict(orow=1025), -1), (dict(oh=-128), -1), (dict(rows=2, orow=0), -1), (dict(oh=0), -1),
          (dict(wsb=0), -1), (dict(rows=0), 0), (dict(rows=1 << 25), -2)]


@pytest.mark.parametrize("kw,rc", COMMON + [(dict(mq=-1), -1)])
def test_paged_arguments(dsa, kw, rc):
    assert call(dsa, "paged", None, **kw) == rc


@pytest.mark.parametrize("kw,rc", COMMON + [(dict(k=-1), -1), (dict(topk=None), -1), (dict(ts=15), -1),
                                            (dict(k=1 << 25, ts=1 << 25), -2)])
def test_selected_arguments(dsa, kw, rc):
    assert call(dsa, "selected", None, **kw) == rc


def test_sizes(dsa):
    assert dsa.kv_section_bytes_fp4(128) == SECTION and dsa.kv_section_bytes_fp4(64) == 64 * 72
    assert dsa.kv_section_bytes_fp4(80) == 64 * 96 and dsa.kv_section_bytes_fp4(16) == 64 * 24
    for dim in (0, 8, 100, 144, -16):
        with pytest.raises(ValueError):
            dsa.kv_section_bytes_fp4(dim)
    assert dsa.new_kv_cache_fp4(3, 2, 96, "cpu").shape == (3, 2, 64 * 112)
    f = dsa.attend_workspace_size_fp4
    assert 0 < f(64, 64, 32, 8, 128, 1) <= f(128, 128, 32, 8, 128, 4)
    assert f(64, 64, 32, 8, 128, 1, 2048) > 0
    for bad in [(-1, 1, 8, 2, 128, 1), (1, -1, 8, 2, 128, 1), (1, 1, 9, 2, 128, 1), (1, 1, 8, 0, 128, 1),
                (1, 1, 8, 2, 100, 1), (1, 1, 8, 2, 144, 1), (1, 1, 129, 1, 128, 1), (1, 1, 8, 2, 128, -1)]:
        assert f(*bad) == 0


def z(*n, dtype=BF, device="cpu"):
    return torch.zeros(n, dtype=dtype, device=device)


def tensors(device="cpu"):
    """Arguments that pass every check but the one on the device."""
    cache = z(3, 2, 64 * 72, dtype=U8, device=device)
    d = dict(device=device)
    shared = dict(q=z(2, 8, 64, **d), cache=cache, block_table=z(1, 3, dtype=I32, **d), starts=z(2, dtype=I32, **d),
                  row_ends=z(2, dtype=I32, **d), out=z(2, 8, 64, **d), workspace=z(1 << 26, dtype=U8, **d),
                  status=z(1, dtype=I32, **d))
    return dict(
        append=dict(k=z(3, 2, 64, **d), v=z(3, 2, 64, **d), slots=z(3, dtype=I64, **d), cache=cache,
                    positions=z(3, dtype=I64, **d), cos_sin=z(9, 64, dtype=torch.float32, **d), q=z(3, 4, 64, **d),
                    q_out=z(3, 4, 64, **d), status=z(1, dtype=I32, **d)),
        read=dict(slots=z(3, dtype=I64, **d), cache=cache, dim=64, k_out=z(3, 2, 64, **d), v_out=z(3, 2, 64, **d),
                  status=z(1, dtype=I32, **d)),
        paged=dict(shared, max_query_len=2), selected=dict(shared, topk=z(2, 4, dtype=I32, **d)))


def function(dsa, which):
    return dict(append=dsa.kv_append_fp4, read=dsa.kv_read_fp4, paged=dsa.attend_paged_fp4,
                selected=dsa.attend_selected_fp4)[which]


@pytest.mark.parametrize("which", list(CALLS))
def test_cpu_tensors_and_tensors_elsewhere_are_refused(dsa, which):
    args = tensors()[which]
    with pytest.raises(ValueError, match="CUDA"):
        function(dsa, which)(**args)
    for name, value in args.items():
        if isinstance(value, torch.Tensor):
            with pytest.raises(ValueError, match="device"):
                function(dsa, which)(**dict(args, **{name: value.to("meta")}))


@pytest.mark.parametrize("which,name,value", [
    ("append", "k", z(3, 2, 64, dtype=torch.float32)), ("append", "k", z(3, 1, 64)), ("append", "v", z(2, 2, 64)),
    ("append", "v", z(3, 2, 64, dtype=torch.float16)), ("append", "k", z(3, 64, 2).transpose(1, 2)),
    ("append", "slots", z(3, dtype=I32)), ("append", "slots", z(2, dtype=I64)), ("append", "positions", None),
    ("append", "cos_sin", z(9, 64, dtype=torch.float64)), ("append", "q", z(2, 4, 64)), ("append", "q", z(3, 4, 32)),
    ("append", "q", z(3, 4, 64, dtype=torch.float16)), ("append", "q_out", z(3, 4, 64, dtype=torch.float32)),
    ("append", "q", None), ("append", "cache", z(3, 2, 64 * 72 + 16, dtype=U8)), ("append", "cache", z(3, 2, 4608)),
    ("append", "cache", z(3, 64 * 72, 2, dtype=U8).transpose(1, 2)), ("append", "k_scale", "x"),
    ("append", "interleaved", torch.zeros(2)), ("append", "status", torch.zeros(1)),
    ("read", "dim", 80), ("read", "dim", 63), ("read", "dim", "64"), ("read", "dtype", torch.float32), ("read", "dtype", 5),
    ("read", "slots", z(3, 1, dtype=I64)), ("read", "slots", z(6, dtype=I64)[::2]), ("read", "k_out", z(3, 2, 32)),
    ("read", "v_out", z(2, 2, 64)), ("read", "v_out", z(3, 2, 64, dtype=torch.float16)), ("read", "v_scale", None),
    ("paged", "q", z(2, 8, 64, dtype=torch.float32)), ("paged", "q", z(2, 8, 80)), ("paged", "q", z(2, 64, 8).transpose(1, 2)),
    ("paged", "cache", z(3, 2, 4600, dtype=U8)), ("paged", "block_table", z(1, 3, dtype=I64)),
    ("paged", "block_table", z(2, 3, dtype=I32)), ("paged", "starts", z(2, dtype=I64)),
    ("paged", "row_ends", z(3, dtype=I32)), ("paged", "out", z(2, 8, 64, dtype=torch.float16)),
    ("paged", "max_query_len", "1"), ("paged", "scale", "x"), ("paged", "want_lse", torch.zeros(2)),
    ("paged", "workspace", z(1 << 26, dtype=U8)[::2]), ("paged", "status", torch.zeros(1)),
    ("selected", "topk", z(2, 4, dtype=I64)), ("selected", "topk", z(3, 4, dtype=I32)),
    ("selected", "topk", z(4, 2, dtype=I32).t()), ("selected", "q", None)])
def test_the_binding_refuses(dsa, which, name, value):
    with pytest.raises(ValueError) as e:
        function(dsa, which)(**dict(tensors()[which], **{name: value}))
    assert "CUDA" not in str(e.value)                    # the argument's own check


def test_the_layer_refuses(dsa):
    from sparse_attention_indexer_score_gb300.attention import DecodeAttention

    with pytest.raises(ValueError, match="kv_format"):
        DecodeAttention(None, 8, 2, 64, torch.zeros(1, 64), 1, 1, kv_format="mxfp4")
