"""Head norms, rotation and cache append on the GPU.

Two references: the float64 formula, within the rounding of the output type
(half a step) plus the float32 arithmetic before it; and the float32
definition (every operation rounded, sums pairwise), whose roundings to 16, 8
and 4 bits have to come out bit for bit, since a row is quantized after
arithmetic that leaves no freedom."""
import numpy as np
import pytest
import torch

from oracle.fp4 import dequantize_fp4_ref, quantize_fp4_ref
from oracle.fp8 import e4m3_encode
from oracle.rope import make_table, norm_rope_ref
from paged_kv_cache_318_gb300 import api

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built(cuda_device):
    from paged_kv_cache_318_gb300 import _build
    _build.build()
    api.load_library()
    api.check_device_errors(cuda_device)
    yield
    api.check_device_errors(cuda_device)


def f32(t):
    return t.detach().float().cpu().numpy()


class Case:
    """Inputs on the host and the device; q, k, v are views of one tensor."""

    def __init__(self, dev, T=5, Hq=4, Hkv=2, D=128, rot=None, dtype="bf16",
                 neox=True, sections=None, interleaved=False, norm=True,
                 offset=0.0, table="f32", max_pos=300, seed=0, shift=0,
                 extra=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        rot = D if rot is None else rot
        dt = DT[dtype]
        heads = Hq + 2 * Hkv
        # `shift` elements off the allocation and `extra` after each token:
        # rows that are not on 16-byte boundaries
        flat = torch.randn(T * (heads * D + extra) + shift, generator=g)
        flat = (flat * 2).to(dt)
        self.qkv = flat.to(dev)[shift:].view(T, heads * D + extra)
        rows = self.qkv[:, :heads * D].unflatten(1, (heads, D))
        self.q, self.k, self.v = (rows[:, :Hq], rows[:, Hq:Hq + Hkv],
                                  rows[:, Hq + Hkv:])
        axes = len(sections) if sections else 1
        pos = rng.integers(0, max_pos, (axes, T))
        self.pos = pos if axes > 1 else pos[0]
        tab = torch.from_numpy(make_table(max_pos, rot))
        self.table = tab.to(torch.float32 if table == "f32" else dt).to(dev)
        self.w = [None, None]
        if norm:
            self.w = [(torch.randn(D, generator=g) * 0.3 + 1 - offset)
                      .to(dt).to(dev) for _ in "qk"]
        self.kw = dict(q_weight=self.w[0], k_weight=self.w[1], is_neox=neox,
                       mrope_section=sections, mrope_interleaved=interleaved,
                       weight_offset=offset)
        self.ref_kw = dict(neox=neox, sections=sections,
                           interleaved=interleaved, offset=offset)
        self.dev, self.dt, self.T, self.D = dev, dt, T, D

    def positions(self):
        return torch.from_numpy(np.ascontiguousarray(self.pos)).to(self.dev)

    def ref(self, x, w, dtype):
        return norm_rope_ref(f32(x), None if w is None else f32(w), self.pos,
                             f32(self.table), dtype=dtype, **self.ref_kw)

    def check(self, got, x, w):
        """Bits against the float32 definition; distance to float64."""
        want = torch.from_numpy(self.ref(x, w, np.float32)).to(self.dt)
        assert torch.equal(got.cpu().view(torch.int16),
                           want.view(torch.int16))
        exact = self.ref(x, w, np.float64)
        # half a step of the type, and float32: the norm factor's relative
        # error (pairwise sum log2(D) + 4 roundings), two products and a sum
        half = torch.finfo(self.dt).eps / 2
        big = np.abs(exact).max(-1, keepdims=True) * 2
        tol = half * np.abs(exact) + big * 18 * 2.0 ** -24 + 2.0 ** -25
        assert np.all(np.abs(f32(got) - exact) <= tol)


CASES = [
    dict(),
    dict(T=1, Hq=1, Hkv=1),
    dict(T=3, Hq=32, Hkv=8, rot=64),
    dict(T=2, Hq=9, Hkv=3, rot=32, dtype="f16"),
    dict(T=7, Hq=8, Hkv=1, D=64, table="16"),
    dict(T=4, Hq=5, Hkv=5, D=64, rot=32, norm=False),
    dict(T=3, Hq=16, Hkv=8, D=256, offset=1.0),
    dict(T=3, Hq=6, Hkv=2, D=256, rot=128, dtype="f16", table="16"),
    dict(T=3, Hq=4, Hkv=2, D=256, rot=64),
    dict(T=6, neox=False),
    dict(T=6, neox=False, rot=64, norm=False),
    dict(T=6, neox=False, rot=24, dtype="f16"),
    dict(T=5, neox=False, D=64, rot=8, table="16"),
    dict(T=5, neox=False, D=256),
    # several axes
    dict(T=6, sections=[20, 22, 22]),
    dict(T=6, sections=[24, 20, 20], interleaved=True, dtype="f16"),
    dict(T=6, sections=[10, 0, 22, 32], table="16"),
    dict(T=6, sections=[40, 44, 44], interleaved=True, D=256),
    dict(T=6, neox=False, sections=[32, 32]),
    dict(T=6, neox=False, sections=[11, 11, 10], interleaved=True, D=64),
    # the kernel for every other shape
    dict(D=80), dict(D=96, rot=48, dtype="f16"), dict(D=8), dict(D=512),
    dict(D=128, rot=96), dict(D=128, rot=16), dict(D=128, rot=2),
    dict(D=64, rot=6, neox=False), dict(D=136, rot=136, neox=False),
    dict(D=80, sections=[13, 13, 14], interleaved=True),
    dict(shift=1), dict(extra=4), dict(shift=3, extra=6, neox=False),
    # many tokens: several passes a warp, a partly filled last block
    dict(T=1031, Hq=4, Hkv=2, D=64, max_pos=2000),
    dict(T=5003, Hq=3, Hkv=1, D=128, max_pos=2000),
    # keys alone, the last pass of each kind partly filled
    dict(T=5, Hq=0, Hkv=3), dict(T=5, Hq=0, Hkv=5, D=256, rot=64),
    dict(T=5003, Hq=5, Hkv=3, D=256, max_pos=2000),
    # more tokens than the grid takes at once
    dict(T=40003, Hq=1, Hkv=1, D=64, max_pos=2000),
    dict(T=6001, Hq=7, Hkv=1, D=8, max_pos=2000),
]


@pytest.mark.parametrize("kw", CASES, ids=range(len(CASES)))
def test_qk_norm_rope(cuda_device, kw):
    c = Case(cuda_device, seed=len(repr(kw)), **kw)
    q, k = api.qk_norm_rope(c.q, c.k, c.positions(), c.table, **c.kw)
    torch.cuda.synchronize()
    assert q.is_contiguous() and k.is_contiguous()
    c.check(q, c.q, c.w[0])
    c.check(k, c.k, c.w[1])


@pytest.mark.parametrize("kw", [dict(T=70, Hq=8, Hkv=2), dict(D=80)])
def test_in_place(cuda_device, kw):
    c = Case(cuda_device, **kw)
    want = api.qk_norm_rope(c.q, c.k, c.positions(), c.table, **c.kw)
    v = c.v.clone()
    got = api.qk_norm_rope(c.q, c.k, c.positions(), c.table, q_out=c.q,
                           k_out=c.k, **c.kw)
    torch.cuda.synchronize()
    assert got[0].data_ptr() == c.q.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(c.v, v)


@pytest.mark.parametrize("D", [128, 80])
def test_padding_and_bad_positions(cuda_device, D):
    """Negative positions: rows stay as they were.  Positions past the table:
    the same, and flagged."""
    c = Case(cuda_device, T=9, D=D)
    q = torch.full(c.q.shape, 7.0, dtype=c.dt, device=cuda_device)
    k = torch.full(c.k.shape, 7.0, dtype=c.dt, device=cuda_device)
    pos = c.pos.copy()
    pos[[2, 8]] = -1
    c.pos = pos
    api.qk_norm_rope(c.q, c.k, c.positions(), c.table, q_out=q, k_out=k,
                     **c.kw)
    api.check_device_errors(cuda_device)
    keep = pos >= 0
    assert (q[~torch.from_numpy(keep)] == 7).all()
    c.pos = np.where(keep, pos, 0)
    ref = api.qk_norm_rope(c.q, c.k, c.positions(), c.table, **c.kw)
    sel = torch.from_numpy(keep).to(cuda_device)
    assert torch.equal(q[sel], ref[0][sel]) and torch.equal(k[sel],
                                                            ref[1][sel])
    c.pos[4] = 300                       # the table has rows 0 .. 299
    q.fill_(7.0)
    api.qk_norm_rope(c.q, c.k, c.positions(), c.table, q_out=q, k_out=k,
                     **c.kw)
    with pytest.raises(api.PkvError, match="position past"):
        api.check_device_errors(cuda_device)
    api.check_device_errors(cuda_device)
    assert (q[4] == 7).all() and torch.equal(q[3], ref[0][3])


def test_row_of_zeros_and_infinities(cuda_device):
    """eps keeps a zero row zero; inf and NaN stay in their own rows."""
    c = Case(cuda_device, T=4, norm=True)
    c.q[1] = 0
    c.q[2, 0, 5] = float("inf")
    c.q[2, 1, 6] = float("nan")
    q, _ = api.qk_norm_rope(c.q, c.k, c.positions(), c.table, **c.kw)
    assert not q[1].any()
    assert torch.isnan(q[2, 1]).all()
    ok = torch.ones(4, 4, dtype=torch.bool)
    ok[2, :2] = False
    assert torch.isfinite(q[ok.to(cuda_device)]).all()


# ----------------------------------------------------------- cache append

STORES = [
    ("auto", dict(T=37, Hq=8, Hkv=2), 16, False),
    ("auto", dict(T=21, Hq=4, Hkv=3, D=64, dtype="f16", neox=False), 32,
     True),
    ("auto", dict(T=9, D=80, norm=False), 16, False),
    ("auto", dict(T=9, shift=1), 16, False),
    ("fp8", dict(T=37, Hq=8, Hkv=2), 16, False),
    ("fp8", dict(T=19, Hq=4, Hkv=4, D=256, offset=1.0), 48, True),
    ("fp8", dict(T=9, D=96, rot=48, dtype="f16"), 16, False),
    ("fp4", dict(T=37, Hq=8, Hkv=2), 16, True),
    ("fp4", dict(T=37, Hq=8, Hkv=5, D=64, rot=32), 16, False),
    ("fp4", dict(T=19, Hq=4, Hkv=1, D=256, dtype="f16", table="16"), 32,
     True),
    ("fp4", dict(T=19, neox=False, rot=64, norm=False), 16, True),
    ("fp4", dict(T=19, sections=[20, 22, 22]), 16, True),
    ("fp4", dict(T=9, D=128, rot=16), 16, True),
    ("fp4", dict(T=9, D=192, rot=192), 16, True),
    ("fp4", dict(T=9, extra=4), 64, True),
]


def make_cache(kind, nb, bs, hkv, D, dt, dev, hnd):
    """(codes, block scales) of K and V, filled with a pattern."""
    def one(last, dtype, fill):
        shape = (2, nb, hkv, bs, last) if hnd else (2, nb, bs, hkv, last)
        t = torch.full(shape, fill, dtype=dtype, device=dev)
        return t.transpose(2, 3) if hnd else t
    if kind == "auto":
        return one(D, dt, 9.0), None
    if kind == "fp8":
        return one(D, torch.uint8, 0xAB), None
    return one(D // 2, torch.uint8, 0xAB), one(D // 16, torch.uint8, 0x2C)


@pytest.mark.parametrize("idx", range(len(STORES)))
def test_rope_reshape_and_cache(cuda_device, idx):
    kind, kw, bs, hnd = STORES[idx]
    dev = cuda_device
    c = Case(dev, seed=idx, **kw)
    D, T, hkv = c.D, c.T, c.k.shape[1]
    nb = T // bs + 4
    rng = np.random.default_rng(idx)
    slots = rng.permutation(nb * bs)[:T]
    slots[[1, T - 1]] = -1
    codes, sf = make_cache(kind, nb, bs, hkv, D, c.dt, dev, hnd)
    before = codes.clone()
    ks, vs = (torch.tensor([x], dtype=torch.float32, device=dev)
              for x in (0.013, 0.021))
    q = api.rope_reshape_and_cache(
        c.q, c.k, c.v, codes[0], codes[1],
        torch.from_numpy(slots).to(dev), c.positions(), c.table,
        kv_cache_dtype=kind, k_scale=ks, v_scale=vs,
        k_block_scale=None if sf is None else sf[0],
        v_block_scale=None if sf is None else sf[1], **c.kw)
    api.check_device_errors(dev)
    c.check(q, c.q, c.w[0])              # every token, slot or not
    keep = slots >= 0
    b, o = slots[keep] // bs, slots[keep] % bs
    kf = c.ref(c.k, c.w[1], np.float32)[keep]
    vf = f32(c.v)[keep]
    written = np.zeros((nb, bs), bool)
    written[b, o] = True
    for m, (rows, scale) in enumerate(((kf, 0.013), (vf, 0.021))):
        got = codes[m].cpu()
        if kind == "auto":
            want = torch.from_numpy(rows).to(c.dt)
            assert torch.equal(got[b, o].view(torch.int16),
                               want.view(torch.int16))
        elif kind == "fp8":
            want = e4m3_encode(rows / np.float32(scale))
            assert np.array_equal(got.numpy()[b, o], want)
        else:
            want, wsf = quantize_fp4_ref(rows, scale)
            assert np.array_equal(got.numpy()[b, o], want)
            gsf = sf[m].cpu().numpy()
            assert np.array_equal(gsf[b, o], wsf)
            assert (gsf[~written] == 0x2C).all()
        rest = torch.from_numpy(~written)
        assert torch.equal(got[rest], before[m].cpu()[rest])


@pytest.mark.parametrize("kind", ["auto", "fp4"])
def test_append_bad_slots_and_positions(cuda_device, kind):
    dev = cuda_device
    c = Case(dev, T=6)
    codes, sf = make_cache(kind, 2, 16, 2, 128, c.dt, dev, True)
    before = codes.clone()
    one = torch.ones(1, dtype=torch.float32, device=dev)
    slots = torch.tensor([32, 5, 1 << 40, -7, 6, 7], device=dev)
    c.pos[5] = 1 << 33
    q = torch.full(c.q.shape, 7.0, dtype=c.dt, device=dev)
    api.rope_reshape_and_cache(
        c.q, c.k, c.v, codes[0], codes[1], slots, c.positions(), c.table,
        kv_cache_dtype=kind, k_scale=one, v_scale=one,
        k_block_scale=None if sf is None else sf[0],
        v_block_scale=None if sf is None else sf[1], q_out=q, **c.kw)
    with pytest.raises(api.PkvError) as e:
        api.check_device_errors(dev)
    assert "slot outside" in str(e.value) and "position past" in str(e.value)
    changed = (codes != before).any(-1).any(-1).any(0).flatten()
    assert changed.nonzero().flatten().tolist() == [5, 6]
    # queries: all but the token without a position
    assert (q[5] == 7).all() and not (q[:5] == 7).all(-1).any()


def test_padded_batch(cuda_device):
    """Rows past len(slot_mapping) are not read; 0 tokens is a no-op."""
    dev = cuda_device
    c = Case(dev, T=12)
    codes, _ = make_cache("auto", 2, 16, 2, 128, c.dt, dev, False)
    slots = torch.arange(8, device=dev)
    q = torch.full(c.q.shape, 7.0, dtype=c.dt, device=dev)
    api.rope_reshape_and_cache(c.q, c.k, c.v, codes[0], codes[1], slots,
                               c.positions(), c.table, q_out=q, **c.kw)
    assert (q[8:] == 7).all() and not (q[:8] == 7).all(-1).any()
    assert (codes[:, 0, 8:] == 9).all() and (codes[:, 1] == 9).all()
    before = codes.clone()
    api.rope_reshape_and_cache(c.q, c.k, c.v, codes[0], codes[1], slots[:0],
                               c.positions(), c.table, q_out=q, **c.kw)
    api.check_device_errors(dev)
    assert torch.equal(codes, before)


def test_graph_and_side_stream(cuda_device):
    """Captured and replayed with new inputs; run on another stream."""
    dev = cuda_device
    c = Case(dev, T=64, Hq=8, Hkv=2)
    codes, sf = make_cache("fp4", 8, 16, 2, 128, c.dt, dev, True)
    one = torch.full((1,), 0.01, dtype=torch.float32, device=dev)
    slots, pos = torch.arange(64, device=dev), c.positions()
    q = torch.empty(c.q.shape, dtype=c.dt, device=dev)

    def call():
        api.rope_reshape_and_cache(
            c.q, c.k, c.v, codes[0], codes[1], slots, pos, c.table,
            kv_cache_dtype="fp4", k_scale=one, v_scale=one,
            k_block_scale=sf[0], v_block_scale=sf[1], q_out=q, **c.kw)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    c.qkv.mul_(-0.5)
    pos.add_(1).clamp_(max=299)
    slots.add_(32)
    graph.replay()
    torch.cuda.synchronize()
    got = q.clone(), codes.clone(), sf.clone()
    codes[:, 2:6].zero_()
    sf[:, 2:6].zero_()
    q.zero_()
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(q, got[0])
    assert torch.equal(codes, got[1]) and torch.equal(sf, got[2])
    c.pos = pos.cpu().numpy()
    c.check(q, c.q, c.w[0])
    back = dequantize_fp4_ref(codes[1].cpu().numpy(), sf[1].cpu().numpy(),
                              0.01)[2:6].reshape(64, 2, 128)
    v = f32(c.v)
    top = np.abs(v).reshape(64, 2, 8, 16).max(-1).repeat(16, -1)
    assert np.all(np.abs(back - v) <= top * (1 / 6 * 1.0625 + 0.0625))
