"""Calls that the 4-bit cache and the rotation entry points refuse (no GPU:
arguments are checked before anything is launched)."""
import ctypes

import pytest
import torch

from paged_kv_cache_318_gb300 import api


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_318_gb300 import _build
    _build.build()
    return api.load_library()


P = 1 << 20                       # a pointer that is never followed


class Scales(ctypes.Structure):
    _fields_ = [("k_block_scale", ctypes.c_void_p),
                ("v_block_scale", ctypes.c_void_p),
                ("strides", ctypes.c_int64 * 4),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]

    def __init__(self, **kw):
        super().__init__(P, P, (ctypes.c_int64 * 4)(512, 8, 128, 1), P, P)
        for k, v in kw.items():
            setattr(self, k, v)


def strides(*s):
    return (ctypes.c_int64 * 4)(*s)


class RopeParams(ctypes.Structure):
    """pkv_rope_params (include/pkv.h)."""
    _fields_ = [("positions", ctypes.c_void_p),
                ("position_axis_stride", ctypes.c_int64),
                ("num_axes", ctypes.c_int),
                ("interleaved_axes", ctypes.c_int),
                ("sections", ctypes.c_int * 4), ("cos_sin", ctypes.c_void_p),
                ("cos_sin_stride", ctypes.c_int64),
                ("max_position", ctypes.c_int64),
                ("cos_sin_f32", ctypes.c_int), ("rot_dim", ctypes.c_int),
                ("is_neox", ctypes.c_int), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float)]


def rope(**kw):
    r = RopeParams(positions=P, position_axis_stride=8, num_axes=1,
                   cos_sin=P, cos_sin_stride=128, max_position=100,
                        cos_sin_f32=1, rot_dim=128, is_neox=1, q_weight=P,
                        k_weight=P, eps=1e-6, weight_offset=0.0)
    for k, v in kw.items():
        if k == "sections":
            for i, n in enumerate(v):
                r.sections[i] = n
        else:
            setattr(r, k, v)
    return r


# ------------------------------------------------------------------- C ABI

def write(lib, **kw):
    a = dict(k=P, v=P, kst=2048, ksh=128, vst=2048, vsh=128, kc=P, vc=P,
             cs=strides(4096, 64, 1024, 1), sc=ctypes.byref(Scales()),
             slots=P, n=4, H=4, D=128, BS=16, NB=8, dtype=1, stream=None)
    a.update(kw)
    return lib.pkv_reshape_and_cache_fp4(*a.values())


@pytest.mark.parametrize("kw,status,text", [
    (dict(sc=None), 1, b"scales"),
    (dict(D=96), 2, b"multiple of 64"),
    (dict(BS=24), 1, b"block_size"),
    (dict(dtype=2), 2, b"dtype"),
    (dict(n=-1), 1, b"negative"),
    (dict(H=0), 1, b"num_kv_heads"),
    (dict(cs=None), 1, b"cache_strides"),
    (dict(cs=strides(4096, 64, 1024, 2)), 1, b"contiguous"),
    (dict(cs=strides(4096, 72, 1024, 1)), 2, b"16-byte"),
    (dict(kc=P + 8), 2, b"16-byte"),
    (dict(k=P + 2), 2, b"16-byte"),
    (dict(vst=1004), 2, b"16-byte"),
    (dict(k=None), 1, b"NULL"),
    (dict(slots=None), 1, b"NULL"),
    (dict(sc=ctypes.byref(Scales(v_block_scale=None))), 1, b"block scales"),
    (dict(sc=ctypes.byref(Scales(k_scale=None))), 1, b"k_scale"),
    (dict(sc=ctypes.byref(Scales(k_block_scale=P + 1))), 2, b"8-byte"),
    (dict(sc=ctypes.byref(Scales(strides=strides(512, 8, 128, 2)))), 1,
     b"contiguous"),
    (dict(sc=ctypes.byref(Scales(strides=strides(512, 9, 128, 1)))), 2,
     b"8-byte"),
])
def test_write_refuses(lib, kw, status, text):
    assert write(lib, **kw) == status
    assert text in lib.pkv_last_error()


def test_write_of_no_tokens_is_a_noop(lib):
    assert write(lib, n=0, k=None, slots=None) == 0


def read(lib, **kw):
    a = dict(c=P, cs=strides(4096, 64, 1024, 1), f=P,
             fs=strides(512, 8, 128, 1), sc=P, ids=None, n=8, H=4, D=128,
             BS=16, NB=8, out=P, dtype=1, stream=None)
    a.update(kw)
    return lib.pkv_dequantize_fp4_cache(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(n=9), 1), (dict(D=32), 2), (dict(BS=8), 1), (dict(sc=None), 1),
    (dict(f=None), 1), (dict(c=None), 1), (dict(out=None), 1),
    (dict(out=P + 8), 2), (dict(c=P + 4), 2), (dict(fs=None), 1),
    (dict(dtype=2), 2), (dict(n=-3), 1)])
def test_read_back_refuses(lib, kw, status):
    assert read(lib, **kw) == status and lib.pkv_last_error()


def attend(lib, **kw):
    opts = api._Options()
    for k in [k for k in kw if hasattr(opts, k)]:
        setattr(opts, k, kw.pop(k))
    a = dict(q=P, qst=512, qsh=128, kc=P, vc=P,
             cs=strides(4096, 64, 1024, 1), sc=ctypes.byref(Scales()), out=P,
             ost=512, osh=128, cu=P, su=P, batch=1, total_q=1, max_q=1,
             max_k=16, bt=P, bts=1, maxb=1, Hq=4, Hkv=4, D=128, BS=16, NB=8,
             scale=0.125, causal=1, wl=-1, wr=-1, softcap=0.0, alibi=None,
             splits=0, lse=None, ws=None, wsb=0, dtype=1, stream=None,
             opts=ctypes.byref(opts))
    a.update(kw)
    return lib.pkv_paged_attention_varlen_fp4(*a.values())


@pytest.mark.parametrize("kw,status,text", [
    (dict(sc=None), 1, b"scales"),
    (dict(sc=ctypes.byref(Scales(k_scale=None))), 1, b"k_scale"),
    (dict(kv_cache_fp8=1, k_scale=P, v_scale=P), 2, b"4-bit"),
    (dict(cu_seqlens_k=P, total_k=4), 2, b"4-bit"),
    (dict(cs=strides(4096, 72, 1024, 1)), 2, b"16-byte"),
    (dict(q=P + 2), 2, b"16-byte"),
    (dict(Hq=6), 1, b"multiple"),
    (dict(D=192), 2, b"head_size"),
    (dict(BS=8), 1, b"block_size"),
    (dict(splits=-1), 1, b"num_splits"),
    (dict(splits=2, fixed_split_size=64), 1, b"exclusive"),
    (dict(softcap=-1.0), 1, b"softcap"),
    (dict(su=None), 1, b"NULL"),
    (dict(maxb=0), 1, b"block_table"),
    (dict(NB=0), 1, b"no blocks"),
    (dict(cs=strides(1 << 31, 64, 1024, 1)), 2, b"2 GB"),
    (dict(cs=strides(4096, 1 << 28, 1024, 1)), 2, b"2 GB"),
    (dict(cs=strides(4096, 1 << 60, 1024, 1)), 2, b"2 GB"),
])
def test_attention_refuses(lib, kw, status, text):
    assert attend(lib, **kw) == status
    assert text in lib.pkv_last_error()


def test_workspace_size_refuses(lib):
    opts = api._Options(kv_cache_fp8=1)
    n = lib.pkv_paged_attention_workspace_size_fp4(
        1, 1, 1, 16, 4, 4, 128, 16, 1, -1, -1, 0, 1, ctypes.byref(opts))
    assert n == ctypes.c_size_t(-1).value


def norm(lib, r=None, **kw):
    a = dict(q=P, qst=512, qsh=128, k=P, kst=512, ksh=128, qo=P, qost=512,
             qosh=128, ko=P, kost=512, kosh=128, n=4, Hq=4, Hkv=4, D=128,
             r=ctypes.byref(rope() if r is None else r), dtype=1,
             stream=None)
    a.update(kw)
    return lib.pkv_qk_norm_rope(*a.values())


ROPE = [
    (dict(rot_dim=129), b"rot_dim"), (dict(rot_dim=0), b"rot_dim"),
    (dict(rot_dim=130), b"rot_dim"), (dict(rot_dim=127), b"rot_dim"),
    (dict(num_axes=0), b"num_axes"), (dict(num_axes=5), b"num_axes"),
    (dict(num_axes=3, sections=(20, 20, 20)), b"sum"),
    (dict(num_axes=2, sections=(-1, 65)), b"section"),
    (dict(max_position=0), b"max_position"),
    (dict(cos_sin_stride=100), b"rot_dim"),
    (dict(q_weight=None), b"go together"),
    (dict(eps=-1.0), b"eps"), (dict(eps=float("nan")), b"eps"),
    (dict(weight_offset=float("inf")), b"weight_offset"),
    (dict(positions=None), b"NULL"), (dict(cos_sin=None), b"NULL"),
]


@pytest.mark.parametrize("kw,text", ROPE)
def test_rope_refuses(lib, kw, text):
    assert norm(lib, rope(**kw)) == 1
    assert text in lib.pkv_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(r=None), 1), (dict(D=120 + 4), 2), (dict(D=520), 2),
    (dict(dtype=2), 2), (dict(n=-1), 1), (dict(Hkv=0), 1), (dict(Hq=-1), 1),
    (dict(q=None), 1), (dict(ko=None), 1)])
def test_norm_rope_refuses(lib, kw, status):
    args = dict(kw)
    if "D" in args:
        r = rope(rot_dim=64)
        assert norm(lib, r, **args) == status
    elif "r" in args:
        a = [P, 512, 128] * 4 + [4, 4, 4, 128, None, 1, None]
        assert lib.pkv_qk_norm_rope(*a) == status
    else:
        assert norm(lib, **args) == status
    assert lib.pkv_last_error()


def append(lib, r=None, **kw):
    a = dict(q=P, qst=512, qsh=128, k=P, kst=512, ksh=128, v=P, vst=512,
             vsh=128, qo=P, qost=512, qosh=128, kc=P, vc=P,
             cs=strides(8192, 512, 128, 1), slots=P, n=4, Hq=4, Hkv=4, D=128,
             BS=16, NB=8, r=ctypes.byref(rope() if r is None else r),
             dtype=1, kind=b"auto", ks=None, vs=None, f=None, stream=None)
    a.update(kw)
    return lib.pkv_rope_reshape_and_cache(*a.values())


@pytest.mark.parametrize("kw,status,text", [
    (dict(kind=b"int8"), 2, b"int8"),
    (dict(kind=b"fp8"), 1, b"k_scale"),
    (dict(kind=b"fp4"), 1, b"scales"),
    (dict(kind=b"fp4", f=ctypes.byref(Scales()), D=96,
          r=rope(rot_dim=64)), 2, b"multiple of 64"),
    (dict(kind=b"fp4", f=ctypes.byref(Scales()), kc=P + 8), 2, b"16-byte"),
    (dict(BS=20), 1, b"block_size"),
    (dict(cs=strides(8192, 512, 128, 2)), 1, b"contiguous"),
    (dict(v=None), 1, b"NULL"), (dict(slots=None), 1, b"NULL"),
])
def test_rope_append_refuses(lib, kw, status, text):
    assert append(lib, **kw) == status
    assert text in lib.pkv_last_error()


# ------------------------------------------------------------------ Python

bf, i64, i32 = torch.bfloat16, torch.int64, torch.int32


def cache(nb=4, bs=16, h=2, d=128):
    return api.fp4_kv_cache(nb, bs, h, d, device="cpu")


def test_packed_structs_match_their_declarations():
    """The bytes the binding passes are the structs of the header."""
    r = rope(num_axes=3, sections=(1, 2, 3), is_neox=0, interleaved_axes=1)
    s = list(r.sections)
    assert api._PACK_ROPE(
        r.positions, r.position_axis_stride, r.num_axes, r.interleaved_axes,
        *s, r.cos_sin, r.cos_sin_stride, r.max_position, r.cos_sin_f32,
        r.rot_dim, r.is_neox, r.q_weight, r.k_weight, r.eps,
        r.weight_offset) == bytes(r)
    f = Scales()
    assert api._PACK_FP4(f.k_block_scale, f.v_block_scale, *f.strides,
                         f.k_scale, f.v_scale) == bytes(f)


def test_cache_layout():
    codes, sf = cache()
    assert codes.shape == (2, 4, 16, 2, 64) and codes.dtype == torch.uint8
    assert sf.shape == (2, 4, 16, 2, 8) and sf.dtype == torch.float8_e4m3fn
    assert codes[0].stride() == (2048, 64, 1024, 1)
    with pytest.raises(NotImplementedError, match="multiple of 64"):
        cache(d=80)
    with pytest.raises(ValueError, match="multiple of 16"):
        cache(bs=20)


def py_write(**kw):
    codes, sf = cache()
    one = torch.ones(1)
    a = dict(key=torch.zeros(3, 2, 128, dtype=bf),
             value=torch.zeros(3, 2, 128, dtype=bf), key_cache=codes[0],
             value_cache=codes[1], slot_mapping=torch.zeros(3, dtype=i64),
             kv_cache_dtype="fp4", k_scale=one, v_scale=one,
             k_block_scale=sf[0], v_block_scale=sf[1])
    a.update(kw)
    return api.reshape_and_cache_flash(**a)


@pytest.mark.parametrize("kw,text", [
    (dict(), "CUDA device"),
    (dict(slot_mapping=torch.zeros(3, dtype=i32)), "int64"),
    (dict(slot_mapping=torch.zeros(6, dtype=i64)[::2]), "contiguous"),
    (dict(slot_mapping=torch.zeros(4, dtype=i64)), "key must be"),
    (dict(key=torch.zeros(3, 2, 64, dtype=bf)), "key must be"),
    (dict(value=torch.zeros(3, 1, 128, dtype=bf)), "value must be"),
    (dict(key=torch.zeros(3, 128, 2, dtype=bf).transpose(1, 2)),
     "contiguous"),
    (dict(value=torch.zeros(3, 2, 128)), "share a dtype"),
    (dict(k_scale=None), "k_scale"),
    (dict(v_scale=torch.ones(1, dtype=bf)), "v_scale"),
    (dict(v_block_scale=None), "both block scales"),
    (dict(k_block_scale=cache(nb=3)[1][0]), "block scales must be"),
    (dict(k_block_scale=cache()[1][0].contiguous()), "share their strides"),
    (dict(key_cache=cache()[0][0].float(),
          value_cache=cache()[0][0].float()), "uint8"),
    (dict(kv_cache_dtype="auto"), "cache dtype|block scales"),
])
def test_python_write_refuses(lib, kw, text):
    with pytest.raises(ValueError, match=text):
        py_write(**kw)


def py_attend(**kw):
    codes, sf = cache()
    one = torch.ones(1)
    a = dict(q=torch.zeros(1, 4, 128, dtype=bf), k=codes[0], v=codes[1],
             max_seqlen_q=1, cu_seqlens_q=torch.tensor([0, 1], dtype=i32),
             max_seqlen_k=16, seqused_k=torch.tensor([3], dtype=i32),
             block_table=torch.zeros((1, 1), dtype=i32), k_descale=one,
             v_descale=one, k_block_scale=sf[0], v_block_scale=sf[1])
    a.update(kw)
    return api.flash_attn_varlen_func(**a)


@pytest.mark.parametrize("kw,text", [
    (dict(), "CUDA device"),
    (dict(k_descale=None), "k_scale"),
    (dict(v_block_scale=None), "both block scales"),
    (dict(k_block_scale=None, v_block_scale=None), "head_size differ"),
    (dict(seqused_k=torch.zeros(1, dtype=i64)), "int32"),
    (dict(block_table=None), "block_table"),
])
def test_python_attention_refuses(lib, kw, text):
    with pytest.raises(ValueError, match=text):
        py_attend(**kw)


def test_python_attention_refuses_fp8_queries_and_rows(lib):
    with pytest.raises(NotImplementedError, match="16-bit query"):
        py_attend(q=torch.zeros(1, 4, 128, dtype=torch.float8_e4m3fn))
    with pytest.raises(NotImplementedError, match="paged"):
        py_attend(k=torch.zeros(3, 2, 128, dtype=bf),
                  v=torch.zeros(3, 2, 128, dtype=bf),
                  cu_seqlens_k=torch.tensor([0, 3], dtype=i32))


def test_cascade_refuses_a_four_bit_cache(lib):
    codes, _ = cache()
    one = torch.ones(1)
    q = torch.zeros(8, 4, 128, dtype=bf)
    t = torch.zeros(8, dtype=i32)
    with pytest.raises(ValueError, match="4-bit"):
        api.cascade_attention(torch.zeros_like(q), q, codes[0], codes[1], t,
                              1, t, t, t, 64, 0.1, None, (-1, -1), 0.0,
                              torch.zeros((8, 4), dtype=i32), 16,
                              k_descale=one, v_descale=one)


def py_norm(**kw):
    a = dict(q=torch.zeros(3, 4, 128, dtype=bf),
             k=torch.zeros(3, 2, 128, dtype=bf),
             positions=torch.zeros(3, dtype=i64),
             cos_sin_cache=torch.zeros(10, 64))
    a.update(kw)
    return api.qk_norm_rope(**a)


@pytest.mark.parametrize("kw,text", [
    (dict(), "CUDA device"),
    (dict(q=torch.zeros(3, 512, dtype=bf)), "q and k must be"),
    (dict(k=torch.zeros(2, 2, 128, dtype=bf)), "k must be"),
    (dict(k=torch.zeros(3, 2, 128)), "share a dtype"),
    (dict(positions=torch.zeros(3, dtype=i32)), "int64"),
    (dict(positions=torch.zeros(2, dtype=i64)), "positions has 2"),
    (dict(positions=torch.zeros((2, 3), dtype=i64)), "need mrope_section"),
    (dict(mrope_section=[16, 16]), "one count"),
    (dict(positions=torch.zeros((5, 3), dtype=i64),
          mrope_section=[8, 8, 8, 4, 4]), "1 to 4"),
    (dict(cos_sin_cache=torch.zeros(10, 64, dtype=torch.float16)),
     "cos_sin_cache must be float32"),
    (dict(cos_sin_cache=torch.zeros(64)), "cos_sin_cache must be"),
    (dict(q_weight=torch.ones(128, dtype=bf)), "go together"),
    (dict(q_weight=torch.ones(64, dtype=bf),
          k_weight=torch.ones(64, dtype=bf)), "norm weights"),
    (dict(q_weight=torch.ones(128), k_weight=torch.ones(128)),
     "norm weights"),
    (dict(q_out=torch.zeros(3, 4, 64, dtype=bf)), "q_out must be"),
    (dict(q_out=torch.zeros(3, 4, 128)), "share a dtype"),
])
def test_python_norm_refuses(lib, kw, text):
    with pytest.raises(ValueError, match=text):
        py_norm(**kw)


def py_append(**kw):
    a = dict(q=torch.zeros(3, 4, 128, dtype=bf),
             k=torch.zeros(3, 2, 128, dtype=bf),
             v=torch.zeros(3, 2, 128, dtype=bf),
             key_cache=torch.zeros(4, 16, 2, 128, dtype=bf),
             value_cache=torch.zeros(4, 16, 2, 128, dtype=bf),
             slot_mapping=torch.zeros(3, dtype=i64),
             positions=torch.zeros(3, dtype=i64),
             cos_sin_cache=torch.zeros(10, 64))
    a.update(kw)
    return api.rope_reshape_and_cache(**a)


fp8 = dict(key_cache=torch.zeros(4, 16, 2, 128, dtype=torch.uint8),
           value_cache=torch.zeros(4, 16, 2, 128, dtype=torch.uint8))


@pytest.mark.parametrize("kw,text", [
    (dict(), "CUDA device"),
    (dict(k=torch.zeros(3, 4, 128, dtype=bf)), "k must be"),
    (dict(v=torch.zeros(2, 2, 128, dtype=bf)), "v must be"),
    (dict(key_cache=torch.zeros(4, 16, 2, 64, dtype=bf),
          value_cache=torch.zeros(4, 16, 2, 64, dtype=bf)),
     "head_size differ"),
    (dict(value_cache=torch.zeros(4, 16, 2, 128)), "cache dtype"),
    (fp8, "cache dtype"),
    (dict(kv_cache_dtype="fp8"), "fp8 cache must be"),
    (dict(kv_cache_dtype="fp8", **fp8), "k_scale"),
    (dict(kv_cache_dtype="fp4", **fp8), "both block scales"),
    (dict(k_block_scale=torch.zeros(1)), "need kv_cache_dtype"),
    (dict(slot_mapping=torch.zeros(3, dtype=i32)), "int64"),
])
def test_python_append_refuses(lib, kw, text):
    with pytest.raises(ValueError, match=text):
        py_append(**kw)


def test_python_read_back_refuses(lib):
    codes, sf = cache()
    one = torch.ones(1)
    call = api.dequantize_fp4_cache
    for text, args, kw in [
            ("CUDA device", (codes[0], sf[0], one), dict(dtype=bf)),
            ("dtype or out", (codes[0], sf[0], one), {}),
            ("codes must be", (codes, sf[0], one), dict(dtype=bf)),
            ("block scales must be", (codes[0], sf[0][:2], one),
             dict(dtype=bf)),
            ("out must be", (codes[0], sf[0], one),
             dict(out=torch.zeros(3, 16, 2, 128, dtype=bf))),
            ("int64", (codes[0], sf[0], one),
             dict(dtype=bf, block_ids=torch.zeros(2, dtype=i32)))]:
        with pytest.raises(ValueError, match=text):
            call(*args, **kw)
