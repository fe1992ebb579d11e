"""Calls that drafted trees, their verification and the cache's compaction
refuse (no GPU: arguments are checked before anything is launched)."""
import ctypes

import pytest
import torch

from paged_kv_cache_318_gb300 import api

P = 1 << 20                       # a pointer that is never followed
NONE = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_318_gb300 import _build
    _build.build()
    return api.load_library()


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


class Scales(ctypes.Structure):
    _fields_ = [("k_block_scale", ctypes.c_void_p),
                ("v_block_scale", ctypes.c_void_p),
                ("strides", ctypes.c_int64 * 4),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


def options(**kw):
    o = api._Options()
    for k, v in kw.items():
        setattr(o, k, v)
    return ctypes.byref(o)


# ------------------------------------------------------------------- C ABI

def attend(lib, **kw):
    a = dict(q=P, qst=512, qsh=128, kc=P, vc=P,
             cs=strides(8192, 512, 128, 1), sc=None, out=P, ost=512, osh=128,
             cu=P, su=P, par=P, batch=1, total_q=5, max_q=5, max_k=16, bt=P,
             bts=1, maxb=1, Hq=4, Hkv=4, D=128, BS=16, NB=8, scale=0.125,
             causal=1, wl=-1, wr=-1, softcap=0.0, splits=0, lse=None, ws=None,
             wsb=0, dtype=1, stream=None, opts=None)
    assert not set(kw) - set(a)
    a.update(kw)
    # (a binding of its own: the package passes the structs as bytes)
    fn = ctypes.CDLL(lib._name).pkv_paged_attention_varlen_tree
    i, l, p, f = (ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
                  ctypes.c_float)
    fn.argtypes = [p, l, l, p, p, p, p, p, l, l, p, p, p, i, i, i, i, p, l, i,
                   i, i, i, i, l, f, i, i, i, f, i, p, p, ctypes.c_size_t, i,
                   p, p]
    fn.restype = i
    for k in ("cs", "sc"):
        if a[k] is not None:
            a[k] = ctypes.cast(ctypes.pointer(a[k]), p)
    if a["opts"] is not None:
        a["opts"] = ctypes.cast(a["opts"], p)
    return fn(*a.values())


@pytest.mark.parametrize("kw,status,text", [
    (dict(causal=0), 1, b"causal"),
    (dict(max_q=257, total_q=257), 2, b"256 rows"),
    (dict(splits=2), 2, b"num_splits"),
    (dict(splits=-1), 1, b"num_splits"),
    (dict(opts=options(fixed_split_size=64)), 2, b"fixed split"),
    (dict(opts=options(cu_seqlens_k=P, total_k=4)), 2, b"paged"),
    (dict(opts=options(q_fp8=1, kv_cache_fp8=1)), 2, b"16-bit query"),
    (dict(opts=options(kv_cache_fp8=1)), 1, b"k_scale"),
    (dict(opts=options(kv_cache_fp8=1, k_scale=P, v_scale=P),
          sc=Scales(P, P, (ctypes.c_int64 * 4)(512, 8, 128, 1), P, P)), 2,
     b"4-bit"),
    (dict(sc=Scales(P, None, (ctypes.c_int64 * 4)(512, 8, 128, 1), P, P)), 1,
     b"block scales"),
    (dict(par=None), 1, b"tree_parents"),
    (dict(q=None), 1, b"NULL"), (dict(su=None), 1, b"NULL"),
    (dict(bt=None), 1, b"NULL"), (dict(cs=None), 1, b"NULL"),
    (dict(NB=0), 1, b"no blocks"),
    (dict(maxb=0), 1, b"block_table"), (dict(bts=0), 1, b"block_table"),
    (dict(maxb=1 << 27, bts=1 << 27), 2, b"2^31"),
    (dict(max_q=256, total_q=256, Hq=4096, Hkv=1), 2, b"too many rows"),
    (dict(batch=1 << 26, Hq=128, Hkv=128), 2, b"too many rows"),
    (dict(Hq=6), 1, b"multiple"), (dict(Hkv=0), 1, b"num_kv_heads"),
    (dict(D=96), 2, b"head_size"), (dict(BS=24), 1, b"block_size"),
    (dict(dtype=2), 2, b"dtype"), (dict(batch=-1), 1, b"negative"),
    (dict(scale=float("inf")), 1, b"softmax_scale"),
    (dict(softcap=-1.0), 1, b"softcap"),
    (dict(cs=strides(8192, 512, 128, 2)), 1, b"contiguous"),
    (dict(cs=strides(8192, 516, 128, 1)), 2, b"16-byte"),
    (dict(q=P + 2), 2, b"16-byte"), (dict(ost=516), 2, b"16-byte"),
])
def test_attention_refuses(lib, kw, status, text):
    assert attend(lib, **kw) == status
    assert text in lib.pkv_last_error()


@pytest.mark.parametrize("cap", [4097.0, 1e6, 1e30, float("inf")])
def test_attention_refuses_large_soft_caps(lib, cap):
    assert attend(lib, softcap=cap) == 2
    assert b"softcap" in lib.pkv_last_error()


@pytest.mark.parametrize("kw", [dict(batch=0), dict(total_q=0),
                                dict(max_q=0, q=None, par=None)])
def test_nothing_to_attend_is_a_noop(lib, kw):
    assert attend(lib, **kw) == 0


@pytest.mark.parametrize("kw", [dict(max_q=257), dict(splits=2),
                                dict(splits=-1), dict(D=96), dict(Hq=6),
                                dict(BS=8), dict(batch=-1),
                                dict(opts=options(fixed_split_size=8)),
                                dict(opts=options(q_fp8=1))])
def test_workspace_size_refuses(lib, kw):
    a = dict(batch=1, total_q=5, max_q=5, max_k=500, Hq=4, Hkv=4, D=128,
             BS=16, splits=0, opts=None)
    a.update(kw)
    fn = ctypes.CDLL(lib._name).pkv_paged_attention_workspace_size_tree
    fn.argtypes = [ctypes.c_int] * 9 + [ctypes.c_void_p]
    fn.restype = ctypes.c_size_t
    if a["opts"] is not None:
        a["opts"] = ctypes.cast(a["opts"], ctypes.c_void_p)
    assert fn(*a.values()) == NONE


@pytest.mark.parametrize("kw", [dict(splits=1), dict(max_k=64), dict(max_q=0)])
def test_no_workspace_where_nothing_is_cut(lib, kw):
    a = dict(batch=1, total_q=5, max_q=5, max_k=500, Hq=4, Hkv=4, D=128,
             BS=16, splits=0, opts=None)
    a.update(kw)
    assert lib.pkv_paged_attention_workspace_size_tree(*a.values()) == 0


def check(lib, **kw):
    a = dict(tp=P, tst=1000, dp=P, dst=1000, ids=P, u=P, cu=P, par=P, batch=2,
             total_q=8, max_q=4, vocab=1000, out=P, rows=P, counts=P, dtype=1,
             stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.pkv_verify_draft_tokens(*a.values())


@pytest.mark.parametrize("kw,status,text", [
    (dict(dtype=3), 2, b"float32"), (dict(batch=-1), 1, b"negative"),
    (dict(total_q=-1), 1, b"negative"), (dict(max_q=-1), 1, b"negative"),
    (dict(vocab=0), 1, b"vocab"), (dict(vocab=(1 << 20) + 1), 2, b"vocab"),
    (dict(max_q=257), 2, b"256 rows"), (dict(max_q=0), 1, b"max_seqlen_q"),
    (dict(batch=65537), 2, b"65536"), (dict(tp=None), 1, b"NULL"),
    (dict(ids=None), 1, b"NULL"), (dict(u=None), 1, b"NULL"),
    (dict(cu=None), 1, b"NULL"), (dict(out=None), 1, b"NULL"),
    (dict(rows=None), 1, b"NULL"), (dict(counts=None), 1, b"NULL"),
    (dict(tp=P + 1), 1, b"misaligned"),
    (dict(dtype=2, dp=P + 2), 1, b"misaligned"),
])
def test_verification_refuses(lib, kw, status, text):
    assert check(lib, **kw) == status
    assert text in lib.pkv_last_error()


def test_verification_of_no_requests_is_a_noop(lib):
    assert check(lib, batch=0, tp=None, max_q=0) == 0


def move(lib, **kw):
    a = dict(c=(ctypes.c_void_p * 2)(P, 2 * P), n=2, cs=strides(8192, 512, 128),
             heads=4, row=128, BS=16, NB=8, bt=P, bts=4, maxb=4, cu=P, su=P,
             rows=P, rst=8, maxr=8, cnt=P, batch=2, total_q=16, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    fn = ctypes.CDLL(lib._name).pkv_compact_draft_cache
    i, l, p = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p
    fn.argtypes = [p, i, p, i, i, i, l, p, l, i, p, p, p, l, i, p, i, i, p]
    return fn(*a.values())


@pytest.mark.parametrize("kw,status,text", [
    (dict(n=-1), 1, b"negative"), (dict(batch=-1), 1, b"negative"),
    (dict(maxr=-1), 1, b"negative"), (dict(NB=-1), 1, b"negative"),
    (dict(heads=0), 1, b"num_heads"), (dict(row=0), 1, b"row_bytes"),
    (dict(heads=1 << 20, row=1 << 12), 2, b"1 GB"),
    (dict(BS=24), 1, b"block_size"), (dict(maxr=257, rst=257), 2, b"256"),
    (dict(cs=None), 1, b"cache_strides"), (dict(c=None), 1, b"NULL"),
    (dict(bt=None), 1, b"NULL"), (dict(rows=None), 1, b"NULL"),
    (dict(cnt=None), 1, b"NULL"), (dict(maxb=0), 1, b"block_table"),
    (dict(bts=3), 1, b"block_table"), (dict(rst=7), 1, b"rows_stride"),
    (dict(c=(ctypes.c_void_p * 2)(P, None)), 1, b"NULL cache"),
    (dict(c=(ctypes.c_void_p * 2)(P, P)), 1, b"cache 1 is cache 0"),
])
def test_compaction_refuses(lib, kw, status, text):
    assert move(lib, **kw) == status
    assert text in lib.pkv_last_error()


@pytest.mark.parametrize("kw", [dict(batch=0), dict(total_q=0),
                                dict(maxr=0, rst=0)])
def test_nothing_to_move_is_a_noop(lib, kw):
    assert move(lib, **kw) == 0


# ------------------------------------------------------------------ Python

bf, f32, i32, i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def zeros(*shape, t=i32):
    return torch.zeros(shape, dtype=t)


@pytest.fixture
def no_device(monkeypatch):
    """What gets past the checks of shapes and types ends here."""
    def passed(*_):
        raise AssertionError("not refused")
    monkeypatch.setattr(api, "_on_device", passed)


def tree(**kw):
    a = dict(q=zeros(5, 4, 64, t=bf), k=zeros(3, 16, 2, 64, t=bf),
             v=zeros(3, 16, 2, 64, t=bf), max_seqlen_q=3,
             cu_seqlens_q=zeros(3), max_seqlen_k=20, seqused_k=zeros(2),
             causal=True, block_table=zeros(2, 2), tree_parents=zeros(5))
    a.update(kw)
    return api.flash_attn_varlen_func(**a)


@pytest.mark.parametrize("kw,error", [
    (dict(cu_seqlens_k=zeros(3)), NotImplementedError),
    (dict(q=zeros(5, 4, 64, t=torch.float8_e4m3fn)), NotImplementedError),
    (dict(alibi_slopes=zeros(4, t=f32)), NotImplementedError),
    (dict(q=zeros(5, 4, 64, t=torch.float16)), NotImplementedError),
    (dict(v=zeros(3, 16, 2, 64, t=torch.float16)), NotImplementedError),
    (dict(q=zeros(5, 256, t=bf)), ValueError),
    (dict(q=zeros(5, 4, 128, t=bf)), ValueError),
    (dict(q=zeros(5, 4, 128, t=bf)[:, :, ::2]), ValueError),
    (dict(v=zeros(3, 16, 4, 64, t=bf)), ValueError),
    (dict(block_table=None), ValueError), (dict(seqused_k=None), ValueError),
    (dict(cu_seqlens_q=zeros(4)), ValueError),
    (dict(cu_seqlens_q=zeros(3, t=i64)), ValueError),
    (dict(seqused_k=zeros(2, t=i64)), ValueError),
    (dict(seqused_k=zeros(4)[::2]), ValueError),
    (dict(tree_parents=zeros(4)), ValueError),
    (dict(tree_parents=zeros(5, t=i64)), ValueError),
    (dict(tree_parents=zeros(10)[::2]), ValueError),
    (dict(block_table=zeros(3, 2)[:1]), ValueError),
    (dict(block_table=zeros(2, 2, t=i64)), ValueError),
    (dict(block_table=zeros(2, 4)[:, ::2]), ValueError),
    (dict(out=zeros(5, 4, 64, t=f32)), ValueError),
    (dict(out=zeros(4, 4, 64, t=bf)), ValueError),
    (dict(s_aux=zeros(4, t=bf)), ValueError),
    (dict(s_aux=zeros(3, t=f32)), ValueError),
    (dict(k=zeros(3, 16, 2, 64, t=torch.uint8),
          v=zeros(3, 16, 2, 64, t=torch.uint8)), ValueError),
])
def test_tree_attention_refuses(no_device, kw, error):
    with pytest.raises(error):
        tree(**kw)


def verify(**kw):
    a = dict(target_probs=zeros(5, 100, t=f32), draft_token_ids=zeros(5),
             cu_seqlens_q=zeros(3), max_seqlen_q=3, uniform=zeros(5, t=f32),
             tree_parents=zeros(5), draft_probs=zeros(5, 100, t=f32))
    a.update(kw)
    return api.verify_draft_tokens(**a)


@pytest.mark.parametrize("kw,error", [
    (dict(target_probs=zeros(500, t=f32)), ValueError),
    (dict(target_probs=zeros(5, 100, t=torch.float64)), NotImplementedError),
    (dict(target_probs=zeros(5, 200, t=f32)[:, ::2]), ValueError),
    (dict(draft_probs=zeros(5, 100, t=bf)), ValueError),
    (dict(draft_probs=zeros(4, 100, t=f32)), ValueError),
    (dict(draft_probs=zeros(5, 200, t=f32)[:, ::2]), ValueError),
    (dict(uniform=zeros(5, t=bf)), ValueError),
    (dict(uniform=zeros(4, t=f32)), ValueError),
    (dict(uniform=zeros(10, t=f32)[::2]), ValueError),
    (dict(draft_token_ids=zeros(4)), ValueError),
    (dict(draft_token_ids=zeros(5, t=i64)), ValueError),
    (dict(tree_parents=zeros(4)), ValueError),
    (dict(cu_seqlens_q=zeros(0)), ValueError),
    (dict(cu_seqlens_q=zeros(3, t=i64)), ValueError),
    (dict(out=(zeros(2, 4), zeros(2, 3), zeros(2))), ValueError),
    (dict(out=(zeros(2, 3), zeros(2, 3), zeros(2, t=i64))), ValueError),
    (dict(out=(zeros(2, 3), zeros(2, 6)[:, ::2], zeros(2))), ValueError),
])
def test_verify_refuses(no_device, kw, error):
    with pytest.raises(error):
        verify(**kw)


def compact(**kw):
    a = dict(caches=[zeros(3, 16, 2, 64, t=bf) for _ in range(2)],
             block_table=zeros(2, 2), cu_seqlens_q=zeros(3),
             seqused_k=zeros(2), rows=zeros(2, 4), counts=zeros(2))
    a.update(kw)
    return api.compact_draft_cache(**a)


@pytest.mark.parametrize("kw", [
    dict(caches=[zeros(3, 16, 128, t=bf)]),
    dict(caches=[zeros(3, 16, 2, 64, t=bf)[..., ::2]]),
    dict(caches=[zeros(3, 16, 2, 64, t=bf), zeros(3, 16, 2, 32, t=bf)]),
    dict(caches=[zeros(3, 16, 2, 64, t=bf),
                 zeros(3, 16, 2, 64, t=torch.float16)]),
    dict(caches=[zeros(3, 16, 2, 64, t=bf),
                 zeros(3, 2, 16, 64, t=bf).transpose(1, 2)]),
    dict(caches=zeros(1, 16, 2, 64, t=bf).expand(3, -1, -1, -1)),
    dict(rows=zeros(2, 4, t=i64)), dict(rows=zeros(8)),
    dict(rows=zeros(2, 8)[:, ::2]), dict(counts=zeros(1)),
    dict(counts=zeros(2, t=i64)), dict(seqused_k=zeros(3)),
    dict(cu_seqlens_q=zeros(2)), dict(block_table=zeros(1, 2)),
    dict(block_table=zeros(2, 2, t=i64)),
])
def test_compact_refuses(no_device, kw):
    with pytest.raises(ValueError):
        compact(**kw)


def test_compact_of_no_caches_is_a_noop():
    assert compact(caches=[]) is None


@pytest.mark.parametrize("call,kw", [
    (tree, dict(seqused_k=torch.zeros(2, dtype=i32, device="meta"))),
    (tree, dict(s_aux=torch.zeros(4, device="meta"))), (tree, {}),
    (verify, dict(uniform=torch.zeros(5, device="meta"))), (verify, {}),
    (compact, dict(counts=torch.zeros(2, dtype=i32, device="meta"))),
    (compact, {}),
])
def test_tensors_have_to_be_on_one_cuda_device(call, kw):
    with pytest.raises(ValueError, match="device"):
        call(**kw)
