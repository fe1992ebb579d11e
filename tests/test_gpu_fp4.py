"""The 4-bit KV cache on the GPU: the quantizing write and the read-back are
bit-exact; attention over it matches the float64 oracle on the values that
the codes stand for.

Tolerance of an attention output, from the arithmetic: the probabilities
round to f16 in the decode kernel (relative error at most half a step, eps/2)
or to the call's type in the prefill kernels, so the output moves by at most
that times the largest |v| among the keys; the output rounds once more, by
half a step of its type; and the logits carry a float32 error `d`, which
scales every probability by at most e^(2 d)."""
import numpy as np
import pytest
import torch

from oracle import paged_attention_ref
from oracle.fp4 import (dequantize_fp4_ref, quantize_fp4_ref,
                        reshape_and_cache_fp4_ref)
from oracle.fp8 import e4m3_decode
from oracle.rope import make_table, norm_rope_ref
from paged_kv_cache_318_gb300 import api, workloads

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
KS, VS = 0.0021, 0.0017


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


def scales(dev, k=KS, v=VS):
    return [torch.tensor([x], dtype=torch.float32, device=dev)
            for x in (k, v)]


def poisoned(wl, dev, nhd=False):
    """A cache whose unwritten scales are NaN (and codes are noise)."""
    NB, BS, H, D = wl.cache_shape()[1:]
    codes, sf = api.fp4_kv_cache(NB, BS, H, D, dev)
    if nhd:
        codes, sf = codes.contiguous(), sf.contiguous()
    codes.fill_(0x5B)
    sf.view(torch.uint8).fill_(0x7F)
    return codes, sf


def fill(wl, dev, nhd=False):
    codes, sf = poisoned(wl, dev, nhd)
    ks, vs = scales(dev)
    for k, v, slots in ((wl.k_ctx, wl.v_ctx, wl.slot_mapping_ctx),
                        (wl.k_new, wl.v_new, wl.slot_mapping_new)):
        if len(slots):
            api.reshape_and_cache_flash(
                k.to(dev), v.to(dev), codes[0], codes[1],
                torch.from_numpy(slots).to(dev), "fp4", ks, vs,
                k_block_scale=sf[0], v_block_scale=sf[1])
    torch.cuda.synchronize()
    return codes, sf, ks, vs


def oracle_cache(wl):
    """The workload's rows through the oracle's quantizing write, as values."""
    NB, BS, H, D = wl.cache_shape()[1:]
    kc, vc = (np.full((NB, BS, H, D // 2), 0x5B, np.uint8) for _ in "kv")
    kf, vf = (np.full((NB, BS, H, D // 16), 0x7F, np.uint8) for _ in "kv")
    for k, v, slots in ((wl.k_ctx, wl.v_ctx, wl.slot_mapping_ctx),
                        (wl.k_new, wl.v_new, wl.slot_mapping_new)):
        reshape_and_cache_fp4_ref(f32(k), f32(v), kc, vc, kf, vf, slots, KS,
                                  VS)
    return (kc, kf, vc, vf), (dequantize_fp4_ref(kc, kf, KS),
                              dequantize_fp4_ref(vc, vf, VS))


# ------------------------------------------------------- write and read-back

@pytest.mark.parametrize("D,Hkv,BS,dtype,nhd", [
    (128, 8, 16, "bf16", False), (64, 1, 48, "f16", False),
    (256, 2, 32, "bf16", True), (128, 40, 16, "f16", True),
    (192, 3, 64, "bf16", False)])
def test_write_bit_exact(cuda_device, D, Hkv, BS, dtype, nhd):
    dev = cuda_device
    T, NB = 61, 7
    g = torch.Generator().manual_seed(D + Hkv)
    # magnitudes from subnormal block scales to saturation, and specials
    mag = 10.0 ** torch.empty(T, Hkv, D // 16, 1).uniform_(-7, 4, generator=g)
    k = (torch.randn(T, Hkv, D // 16, 16, generator=g) * mag).flatten(2)
    v = torch.randn(T, Hkv, D, generator=g)
    v[3], v[4, 0, 5], v[5, 0, 7] = 0.0, float("nan"), float("-inf")
    v[6, 0, :16] = torch.tensor([6.0, -5, 3.5, -2.5, 1.75, 1.25, .75, .25,
                                 -.25, -.75, 0, 5, 2.5, -3.5, 1, 4]) * 64
    k, v = k.to(DT[dtype]), v.to(DT[dtype])
    slots = np.random.default_rng(1).permutation(NB * BS)[:T]
    slots[[0, 9]] = -1
    both = torch.cat([k, v], 1).to(dev)     # k and v side by side
    codes, sf = api.fp4_kv_cache(NB, BS, Hkv, D, dev)
    if nhd:
        codes, sf = codes.contiguous(), sf.contiguous()
    codes.fill_(0xAB)
    sf.view(torch.uint8).fill_(0x2C)
    ks, vs = scales(dev, 0.37, 1.0)
    api.reshape_and_cache_flash(
        both[:, :Hkv], both[:, Hkv:], codes[0], codes[1],
        torch.from_numpy(slots).to(dev), "fp4", ks, vs, k_block_scale=sf[0],
        v_block_scale=sf[1])
    api.check_device_errors(dev)
    want = [np.full((NB, BS, Hkv, n), x, np.uint8)
            for n, x in ((D // 2, 0xAB), (D // 2, 0xAB), (D // 16, 0x2C),
                         (D // 16, 0x2C))]
    reshape_and_cache_fp4_ref(f32(k), f32(v), *want, slots, 0.37, 1.0)
    got = [codes[0], codes[1], sf[0].view(torch.uint8),
           sf[1].view(torch.uint8)]
    got = [t.cpu().numpy() for t in got]
    assert np.array_equal(got[2], want[2]) and np.array_equal(got[3], want[3])
    assert np.array_equal(got[0], want[0])
    # codes of a group with a NaN scale say nothing
    nan = np.repeat((want[3] & 0x7F) == 0x7F, 8, axis=-1)
    assert nan.sum() == 8 and np.array_equal(got[1][~nan], want[1][~nan])
    # read back
    for m, s in ((0, ks), (1, vs)):
        out = api.dequantize_fp4_cache(codes[m], sf[m], s, dtype=DT[dtype])
        ref = dequantize_fp4_ref(got[m], got[2 + m])       # exact products
        ref = (ref.astype(np.float32) *
               np.float32(s.item())).astype(np.float32)
        ref = torch.from_numpy(ref).to(DT[dtype])
        assert torch.equal(out.cpu().nan_to_num(7.0), ref.nan_to_num(7.0))


def test_read_back_of_listed_blocks(cuda_device):
    dev = cuda_device
    wl = workloads.build_workload("r4", 5, [1, 1], [70, 33], 4, 2, 64, 16)
    codes, sf, ks, vs = fill(wl, dev)
    whole = api.dequantize_fp4_cache(codes[1], sf[1], vs,
                                     dtype=torch.bfloat16)
    ids = torch.tensor([3, 0, 3], device=dev)
    out = torch.full((3,) + tuple(whole.shape[1:]), 5.0, device=dev,
                     dtype=torch.bfloat16)
    api.dequantize_fp4_cache(codes[1], sf[1], vs, out=out, block_ids=ids)
    assert torch.equal(out.nan_to_num(9.0), whole[ids].nan_to_num(9.0))
    api.check_device_errors(dev)
    ids = torch.tensor([1, -1, codes.shape[1]], device=dev)
    api.dequantize_fp4_cache(codes[1], sf[1], vs, out=out, block_ids=ids)
    with pytest.raises(api.PkvError, match="block id outside"):
        api.check_device_errors(dev)
    assert not out[1:].any()


def test_write_flags_bad_slots(cuda_device):
    dev = cuda_device
    codes, sf = api.fp4_kv_cache(2, 16, 2, 128, dev)
    ks, vs = scales(dev)
    k = torch.ones(3, 2, 128, dtype=torch.bfloat16, device=dev)
    slots = torch.tensor([32, 4, 1 << 40], device=dev)
    api.reshape_and_cache_flash(k, k, codes[0], codes[1], slots, "fp4", ks,
                                vs, k_block_scale=sf[0], v_block_scale=sf[1])
    with pytest.raises(api.PkvError, match="slot outside"):
        api.check_device_errors(dev)
    assert codes.any(-1).any(-1).any(0).flatten().nonzero().tolist() == [[4]]


# --------------------------------------------------------------- attention

def attend(wl, dev, cache, lse=True, max_k=0, **kw):
    codes, sf, ks, vs = cache
    args = dict(softmax_scale=wl.softmax_scale, causal=wl.causal,
                window_size=wl.window_size, softcap=wl.softcap,
                num_splits=wl.num_splits)
    if wl.alibi_slopes is not None:
        args["alibi_slopes"] = torch.from_numpy(wl.alibi_slopes).to(dev)
    args.update(kw)
    return api.flash_attn_varlen_func(
        wl.q.to(dev), codes[0], codes[1], wl.max_seqlen_q,
        torch.from_numpy(wl.cu_seqlens_q).to(dev),
        max(wl.max_seqlen_k, max_k),
        seqused_k=torch.from_numpy(wl.seq_lens).to(dev),
        block_table=torch.from_numpy(wl.block_table).to(dev),
        return_softmax_lse=lse, k_descale=ks, v_descale=vs,
        k_block_scale=sf[0], v_block_scale=sf[1], **args)


def logit_error(wl, kref):
    """Bound of the float32 error of a logit: D products summed in the tensor
    core (2^-23 a term of the sum of magnitudes, which Cauchy-Schwarz
    bounds), the scalings after it, and exp and log (2^-21 relative)."""
    q = f32(wl.q).astype(np.float64)
    big = np.sqrt((q ** 2).sum(-1).max()) * \
        np.sqrt(np.nanmax((kref ** 2).sum(-1))) * wl.softmax_scale
    return (wl.head_size * 2.0 ** -23 + 2.0 ** -21) * big + 2.0 ** -20


def check(wl, out, lse, refs, sinks=None, keep=None):
    kref, vref = refs
    ro, rl = paged_attention_ref(
        f32(wl.q).astype(np.float64), kref, vref, wl.cu_seqlens_q,
        wl.seq_lens, wl.block_table, wl.softmax_scale, causal=wl.causal,
        window_size=wl.window_size, softcap=wl.softcap,
        alibi_slopes=wl.alibi_slopes, **({} if sinks is None else
                                         {"sinks": sinks}))
    if np.isnan(kref).all():             # no request has a key
        kref = vref = np.zeros_like(kref)
    d = logit_error(wl, kref)
    half = torch.finfo(wl.torch_dtype).eps / 2
    G = wl.num_heads // wl.num_kv_heads
    prefill = wl.max_seqlen_q * G > 16
    p_half = half if prefill else 2.0 ** -11
    if prefill and wl.softcap:
        # the prefill kernels' tanh has a relative error of 2^-10.987
        d += wl.softcap * 2.0 ** -10.9
    if wl.alibi_slopes is not None:
        d += 2.0 ** -22 * np.abs(wl.alibi_slopes).max() * wl.max_seqlen_k
    v_big = np.nanmax(np.abs(vref))
    tol = v_big * (p_half + 2 * d * 1.05 + 2.0 ** -20)
    o = f32(out)
    keep = slice(None) if keep is None else keep
    assert np.isfinite(o[keep]).all()
    err = np.abs(o - ro) - half * np.abs(ro)
    assert err[keep].max() <= tol, (err[keep].max(), tol)
    if lse is not None:
        got = lse.cpu().numpy()
        assert np.array_equal(np.isneginf(got), np.isneginf(rl))
        f = np.isfinite(rl)
        assert np.all(np.abs(got[f] - rl[f]) <=
                      2 * d + 2.0 ** -20 * np.abs(rl[f]))


CASES = [
    # q_lens, seq_lens, Hq, Hkv, D, BS, more
    ([1], [1], 1, 1, 64, 16, {}),
    ([1, 1], [37, 50], 4, 2, 64, 16, {}),
    ([1, 1, 1], [700, 3000, 9], 32, 8, 128, 16, {}),
    ([1, 1, 1], [15, 16, 17], 8, 1, 128, 16, dict(dtype="f16")),
    ([1, 1], [4000, 64], 16, 2, 128, 64, dict(num_splits=4)),
    ([1, 2, 3, 4], [500, 70, 1300, 4], 8, 2, 64, 48, dict(dtype="f16")),
    ([1, 2, 4], [33, 2049, 900], 16, 4, 128, 32, dict(num_splits=1)),
    ([2, 1], [900, 3000], 16, 8, 256, 32, {}),
    ([1, 1], [1, 129], 16, 1, 256, 128, dict(dtype="f16")),
    ([16, 1, 9], [16, 400, 1000], 3, 3, 128, 16, {}),
    ([5, 5], [300, 5], 12, 4, 256, 16, dict(num_splits=3)),
    ([1, 1, 1], [513, 511, 4100], 24, 8, 128, 16, dict(num_splits=7)),
    # windows, caps, slopes
    ([1, 1, 2], [700, 3000, 90], 16, 8, 256, 32,
     dict(window_size=(511, -1), softcap=50.0)),
    ([4, 1, 3], [700, 3000, 90], 8, 4, 128, 16,
     dict(window_size=(20, -1), dtype="f16")),
    ([3, 4], [200, 64], 8, 2, 64, 16,
     dict(causal=False, window_size=(30, 5))),
    ([2, 1], [100, 1000], 8, 8, 128, 16, dict(causal=False)),
    ([2, 1, 1], [100, 1000, 3], 8, 4, 128, 16, dict(alibi=True)),
    ([1, 4], [2000, 77], 4, 1, 256, 16, dict(alibi=True, softcap=20.0,
                                             window_size=(100, -1))),
    # more queries than keys: rows that see nothing; requests without keys
    ([4, 3, 1], [2, 0, 0], 4, 2, 128, 16, {}),
    ([0, 1, 0, 2], [40, 50, 0, 20], 8, 2, 64, 16, {}),
    # prefill-class requests, alone and beside decodes
    ([200, 1, 90], [900, 2000, 90], 32, 8, 128, 16, {}),
    ([70, 1], [600, 1200], 16, 8, 256, 32, dict(softcap=30.0)),
    ([130, 1, 40], [400, 800, 41], 16, 4, 64, 16, dict(dtype="f16")),
    ([33, 300], [100, 300], 8, 8, 128, 64, dict(window_size=(64, -1))),
]


def workload(name, seed, q_lens, seq_lens, Hq, *args, **kw):
    """build_workload, for requests with more queries than keys too."""
    if kw.pop("alibi", False):
        kw["alibi_slopes"] = np.linspace(0.01, 0.3, Hq).astype(np.float32)
    short = np.minimum(q_lens, seq_lens)
    wl = workloads.build_workload(name, seed, short, seq_lens, Hq, *args,
                                  **kw)
    if list(short) != list(q_lens):
        g = torch.Generator().manual_seed(seed)
        wl.q_lens = np.asarray(q_lens, np.int32)
        wl.cu_seqlens_q = workloads.cu_seqlens(q_lens)
        wl.q = torch.randn(int(sum(q_lens)), Hq, wl.head_size, generator=g) \
            .to(wl.torch_dtype)
    return wl


def build(idx):
    q_lens, seq_lens, Hq, Hkv, D, BS, kw = CASES[idx]
    return workload("a4_%d" % idx, 70 + idx, q_lens, seq_lens, Hq, Hkv, D, BS,
                    **kw)


@pytest.mark.parametrize("nhd", [False, True], ids=["hnd", "nhd"])
@pytest.mark.parametrize("idx", range(len(CASES)))
def test_attention(cuda_device, idx, nhd):
    wl = build(idx)
    cache = fill(wl, cuda_device, nhd)
    out, lse = attend(wl, cuda_device, cache)
    api.check_device_errors(cuda_device)
    check(wl, out, lse, oracle_cache(wl)[1])


@pytest.mark.parametrize("splits", [0, 1, 3])
def test_sinks(cuda_device, splits):
    wl = workload("s4", 3, [1, 2, 1], [600, 90, 0], 8, 2, 128, 16,
                  num_splits=splits)
    sinks = np.linspace(-2, 6, 8).astype(np.float32)
    out, lse = attend(wl, cuda_device, fill(wl, cuda_device),
                      s_aux=torch.from_numpy(sinks).to(cuda_device))
    check(wl, out, lse, oracle_cache(wl)[1], sinks=sinks)


def test_fixed_splits_are_batch_invariant(cuda_device):
    dev = cuda_device
    wl = workloads.build_workload("b4", 8, [1, 2, 1], [3000, 700, 64], 8, 2,
                                  128, 16)
    cache = fill(wl, dev)
    whole = attend(wl, dev, cache, fixed_split_size=256)
    check(wl, whole[0], whole[1], oracle_cache(wl)[1])
    codes, sf, ks, vs = cache
    for b in range(3):
        q = wl.q[wl.cu_seqlens_q[b]:wl.cu_seqlens_q[b + 1]].to(dev)
        n = q.shape[0]
        out, lse = api.flash_attn_varlen_func(
            q, codes[0], codes[1], n,
            torch.tensor([0, n], dtype=torch.int32, device=dev),
            int(wl.seq_lens[b]),
            seqused_k=torch.from_numpy(wl.seq_lens[b:b + 1]).to(dev),
            softmax_scale=wl.softmax_scale, causal=True,
            block_table=torch.from_numpy(wl.block_table[b:b + 1]).to(dev),
            return_softmax_lse=True, k_descale=ks, v_descale=vs,
            k_block_scale=sf[0], v_block_scale=sf[1], fixed_split_size=256)
        at = slice(wl.cu_seqlens_q[b], wl.cu_seqlens_q[b + 1])
        assert torch.equal(out, whole[0][at])
        assert torch.equal(lse, whole[1][:, at])


def test_runs_agree_bit_for_bit(cuda_device):
    wl = workloads.build_workload("d4", 8, [1] * 9, [900] * 9, 16, 4, 128, 16)
    cache = fill(wl, cuda_device)
    a = attend(wl, cuda_device, cache)
    b = attend(wl, cuda_device, cache, enable_pdl=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("matrix", [0, 1])
def test_nan_is_seen_only_by_its_rows(cuda_device, matrix, D):
    """A NaN in a key or value that some rows of a request see and others do
    not: only the rows that see it (and, for a value, only its 16 columns)
    read NaN."""
    dev = cuda_device
    wl = workloads.build_workload("n4", 8, [4, 1], [100, 300], 4, 2, D, 16)
    cache = fill(wl, dev)
    codes, sf, ks, vs = cache
    key = 98                                 # seen by the last two queries
    blk, off = wl.block_table[0, key // 16], key % 16
    sf[matrix].view(torch.uint8)[blk, off, 1, 1] = 0x7F
    out, lse = attend(wl, dev, cache)
    refs = list(oracle_cache(wl)[1])
    o = f32(out)
    nan = np.zeros(o.shape, bool)
    if matrix == 0:
        nan[2:4, 2:4] = True
    else:
        nan[2:4, 2:4, 16:32] = True
    assert np.array_equal(np.isnan(o), nan)
    assert np.array_equal(np.isnan(f32(lse)), nan.any(-1).T
                          if matrix == 0 else np.zeros(lse.shape, bool))
    check(wl, out, None, refs, keep=~nan)


def test_wide_query_magnitudes(cuda_device):
    """bf16 queries far outside f16's range, a zero row, an infinite row."""
    dev = cuda_device
    wl = workloads.build_workload("m4", 8, [4], [64], 4, 4, 128, 16)
    wl.q = wl.q.clone()
    wl.q[0] *= 1e-20
    wl.q[1] = 0
    wl.q[2, 1, 3] = float("inf")
    cache = fill(wl, dev)
    out, lse = attend(wl, dev, cache)
    assert torch.isnan(out[2, 1]).all()
    keep = np.ones((4, 4), bool)
    keep[2, 1] = False
    wl.q[2, 1] = 0
    check(wl, out, None, oracle_cache(wl)[1], keep=keep)
    # large ones: the largest logit takes the row
    big = wl.q.clone()
    big[3] *= 2.0 ** 30
    wl.q = big
    out, lse = attend(wl, dev, cache)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_bad_indices(cuda_device):
    dev = cuda_device
    wl = workloads.build_workload("i4", 8, [1, 1], [100, 300], 4, 2, 128, 16)
    cache = fill(wl, dev)
    ref = attend(wl, dev, cache)
    table = wl.block_table.copy()
    wl.block_table = table.copy()
    wl.block_table[0, 2] = -5
    wl.block_table[0, 3] = 1 << 30
    out, _ = attend(wl, dev, cache)
    with pytest.raises(api.PkvError, match="block id outside"):
        api.check_device_errors(dev)
    assert torch.isfinite(out).all() and torch.equal(out[1], ref[0][1])
    # its keys read as zero: a score of 0 and no value
    refs = [x.copy() for x in oracle_cache(wl)[1]]
    spare = int(wl.pad_block)
    for x in refs:
        x[spare] = 0
    wl.block_table[0, 2:4] = spare
    check(wl, out, None, refs)
    # a key range past the table row
    wl.block_table = table[:, :5].copy()
    attend(wl, dev, cache)
    with pytest.raises(api.PkvError, match="beyond the table"):
        api.check_device_errors(dev)


def test_understated_query_length(cuda_device):
    """max_seqlen_q says 1 while a request has 3 queries of 4 heads."""
    dev = cuda_device
    wl = workloads.build_workload("u4", 8, [1, 3], [40, 90], 4, 1, 128, 16)
    codes, sf, ks, vs = fill(wl, dev)
    out = torch.full(wl.q.shape, 7.0, dtype=wl.torch_dtype, device=dev)
    api.flash_attn_varlen_func(
        wl.q.to(dev), codes[0], codes[1], 1,
        torch.from_numpy(wl.cu_seqlens_q).to(dev), wl.max_seqlen_k,
        seqused_k=torch.from_numpy(wl.seq_lens).to(dev), causal=True,
        block_table=torch.from_numpy(wl.block_table).to(dev), out=out,
        k_descale=ks, v_descale=vs, k_block_scale=sf[0],
        v_block_scale=sf[1])
    with pytest.raises(api.PkvError, match="more queries than"):
        api.check_device_errors(dev)
    assert (out[1:] == 7).all() and not (out[0] == 7).all()


@pytest.mark.parametrize("q_lens,num_splits", [([1, 2], 0), ([1, 2], 3),
                                               ([40, 1], 0)])
def test_the_widest_windows(cuda_device, q_lens, num_splits):
    """Windows up to the largest int hide nothing."""
    dev = cuda_device
    wl = workloads.build_workload("w4", 5, q_lens, [700, 2500], 8, 2, 128, 16,
                                  causal=False, num_splits=num_splits)
    cache = fill(wl, dev)
    want = attend(wl, dev, cache)
    check(wl, want[0], want[1], oracle_cache(wl)[1])
    for window in ((2 ** 31 - 1, 2 ** 31 - 1), (-1, 2 ** 31 - 1),
                   (2 ** 31 - 1, -1)):
        out, lse = attend(wl, dev, cache, window_size=window)
        check(wl, out, lse, oracle_cache(wl)[1])


@pytest.mark.parametrize("which", ["PREFILL_TCGEN05", "PREFILL_MMA_SYNC"])
def test_both_prefill_kernels(cuda_device, which):
    dev = cuda_device
    wl = workloads.build_workload("p4", 6, [70, 1, 200], [600, 900, 200], 8, 2,
                                  128, 16, window_size=(300, -1))
    cache = fill(wl, dev)
    api.set_prefill_kernel(getattr(api, which))
    try:
        out, lse = attend(wl, dev, cache)
        api.check_device_errors(dev)
    finally:
        api.set_prefill_kernel(api.PREFILL_TCGEN05)
    check(wl, out, lse, oracle_cache(wl)[1])


def test_padded_rows_stay(cuda_device):
    """Rows of q and out behind the last sequence are left as they were."""
    dev = cuda_device
    wl = workloads.build_workload("p4", 8, [1, 1], [400, 90], 8, 2, 128, 16)
    codes, sf, ks, vs = fill(wl, dev)
    q = torch.full((5, 8, 128), float("nan"), dtype=wl.torch_dtype,
                   device=dev)
    q[:2] = wl.q.to(dev)
    out = torch.full_like(q, 7.0)
    _, lse = api.flash_attn_varlen_func(
        q, codes[0], codes[1], 1,
        torch.from_numpy(wl.cu_seqlens_q).to(dev), 400,
        seqused_k=torch.from_numpy(wl.seq_lens).to(dev), causal=True,
        block_table=torch.from_numpy(wl.block_table).to(dev), out=out,
        k_descale=ks, v_descale=vs, k_block_scale=sf[0],
        v_block_scale=sf[1], return_softmax_lse=True)
    assert (out[2:] == 7).all()
    check(wl, out[:2], lse[:, :2].contiguous(), oracle_cache(wl)[1])


def test_strided_queries_and_outputs(cuda_device):
    dev = cuda_device
    wl = workloads.build_workload("q4", 8, [1, 2], [400, 90], 8, 2, 128, 16)
    cache = fill(wl, dev)
    ref = attend(wl, dev, cache)
    wide = torch.zeros(3, 12, 128, dtype=wl.torch_dtype, device=dev)
    wide[:, 2:10] = wl.q.to(dev)
    out = torch.zeros(3, 8, 160, dtype=wl.torch_dtype, device=dev)
    keep = wl.q
    wl.q = wide[:, 2:10]
    got = attend(wl, dev, cache, out=out[..., :128])
    wl.q = keep
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert not out[..., 128:].any()


def test_offsets_past_32_bits(cuda_device):
    """Blocks beyond 4 GB of codes and past 2^31 bytes of scales."""
    dev = cuda_device
    H, D, BS = 8, 128, 64
    NB = (1 << 32) // (H * BS * D // 2) + 600
    codes, sf = api.fp4_kv_cache(NB, BS, H, D, dev)
    ks, vs = scales(dev)
    L = 300
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(L, H, D, generator=g).bfloat16() for _ in "kv")
    table = np.array([[NB - 1, 3, NB - 300, 131073, NB - 2]], np.int32)
    slots = table[0][np.arange(L) // BS].astype(np.int64) * BS + \
        np.arange(L) % BS
    api.reshape_and_cache_flash(
        k.to(dev), v.to(dev), codes[0], codes[1],
        torch.from_numpy(slots).to(dev), "fp4", ks, vs, k_block_scale=sf[0],
        v_block_scale=sf[1])
    q = torch.randn(1, 16, D, generator=g).bfloat16()
    out = api.flash_attn_varlen_func(
        q.to(dev), codes[0], codes[1], 1,
        torch.tensor([0, 1], dtype=torch.int32, device=dev), L,
        seqused_k=torch.tensor([L], dtype=torch.int32, device=dev),
        causal=True, block_table=torch.from_numpy(table).to(dev),
        k_descale=ks, v_descale=vs, k_block_scale=sf[0], v_block_scale=sf[1])
    back = api.dequantize_fp4_cache(
        codes[1], sf[1], vs, dtype=torch.bfloat16,
        block_ids=torch.tensor([NB - 1], device=dev))
    api.check_device_errors(dev)
    kv = []
    for x, s in ((k, KS), (v, VS)):
        p, f = quantize_fp4_ref(f32(x), s)
        kv.append(dequantize_fp4_ref(p, f, s))
    assert np.abs(f32(back)[0] - kv[1][:BS]).max() <= \
        2.0 ** -8 * np.abs(kv[1]).max()
    ref = np.empty((16, D))
    for h in range(16):
        x = kv[0][:, h // 2] @ f32(q)[0, h] * D ** -0.5
        p = np.exp(x - x.max())
        ref[h] = p @ kv[1][:, h // 2] / p.sum()
    tol = np.abs(kv[1]).max() * (2.0 ** -11 + 2.0 ** -14)
    assert np.all(np.abs(f32(out)[0] - ref) <= tol + 2.0 ** -8 * np.abs(ref))


def test_prefill_range_of_values_is_exact(cuda_device):
    """Block scales over E4M3's whole range (code * scale stays exact in 16
    bits): identical keys make the output the mean of the values."""
    dev = cuda_device
    for dtype, q_len in (("f16", 40), ("bf16", 40), ("f16", 1), ("bf16", 2)):
        codes, sf = api.fp4_kv_cache(1, 16, 1, 128, dev)
        one = torch.ones(1, dtype=torch.float32, device=dev)
        g = torch.Generator().manual_seed(4)
        codes[1] = torch.randint(0, 256, codes[1].shape, generator=g,
                                 dtype=torch.uint8).to(dev)
        byte = torch.randint(0, 0x7F, sf[1].shape, generator=g,
                             dtype=torch.uint8)
        sf[1].view(torch.uint8).copy_(byte.to(dev))
        q = torch.ones(q_len, 1, 128, dtype=DT[dtype], device=dev)
        out = api.flash_attn_varlen_func(
            q, codes[0], codes[1], q_len,
            torch.tensor([0, q_len], dtype=torch.int32, device=dev), 1,
            seqused_k=torch.tensor([1], dtype=torch.int32, device=dev),
            causal=False,
            block_table=torch.zeros((1, 1), dtype=torch.int32, device=dev),
            k_descale=one, v_descale=one, k_block_scale=sf[0],
            v_block_scale=sf[1])
        want = dequantize_fp4_ref(codes[1].cpu().numpy(), byte.numpy())
        assert np.array_equal(f32(out), np.broadcast_to(
            want[0, 0], (q_len, 1, 128)).astype(np.float32))
        assert np.isfinite(e4m3_decode(byte.numpy())).all()


# --------------------------------------------------- graphs, streams, chain

def shares(idx):
    """Calls whose key range is long enough (by max_seqlen_k) that every CTA
    takes an equal share of all units' keys."""
    g = np.random.default_rng(idx)
    q, more = None, {}
    if idx == 0:         # more requests than threads, empty ones among them
        k = g.integers(0, 150, 310)
        heads = (4, 2, 64, 16)
    elif idx == 1:       # up to 16 rows, requests without queries or keys
        q, k = g.integers(0, 5, 140), g.integers(0, 300, 140)
        heads = (8, 2, 128, 16)
        more = dict(dtype="f16")
    elif idx == 2:
        q, k = g.integers(1, 4, 40), g.integers(0, 900, 40)
        heads = (20, 4, 256, 48)
        more = dict(window_size=(2100, -1), softcap=30.0)
    elif idx == 3:       # one unit over many CTAs
        k, heads = [9001], (8, 1, 128, 32)
    elif idx == 4:       # ... over more than the join looks at in one step
        k, heads = [70000], (2, 2, 64, 64)
    elif idx == 5:       # beside prefill-class requests
        q, k = [1, 40, 2, 1, 90], [2500, 400, 1, 3000, 90]
        heads, more = (16, 4, 128, 16), dict(alibi=True)
    elif idx == 6:       # nothing to see at all
        k, heads = [0] * 9, (8, 4, 128, 16)
    elif idx == 7:       # one key each: the smallest shares
        k, heads = [1] * 5 + [3000] + [1] * 700, (8, 1, 256, 16)
    elif idx == 8:
        q, k = [3, 2] * 30, g.integers(3, 700, 60)
        heads, more = (4, 4, 64, 16), dict(causal=False,
                                           window_size=(2048, 40))
    q = [1] * len(k) if q is None else q
    return workload("sh_%d" % idx, 40 + idx, q, k, *heads, **more)


@pytest.mark.parametrize("kw", [
    {}, dict(num_splits=1), dict(num_splits=50), dict(num_splits=200),
    dict(fixed_split_size=512)], ids=["auto", "1", "50", "200", "fixed"])
@pytest.mark.parametrize("Hq,Hkv,D,q_lens,L", [
    (1, 1, 64, [1], [33000]), (2, 2, 64, [1], [70001]),
    (8, 1, 128, [1, 1], [40000, 11]), (16, 1, 256, [1], [20011]),
    (4, 1, 128, [3, 0, 2], [26000, 9, 5000]),
    (4, 2, 128, [40], [3000])])
def test_equal_weights(cuda_device, Hq, Hkv, D, q_lens, L, kw):
    """Queries of zero weigh every key alike: the output is the mean of the
    values a row sees and the LSE the logarithm of their number.  Here P is
    1 and a piece's sums (of multiples of 2^-1 below 2^23) are exact; what is
    left are the exp2 and log2 of the pieces' joins (2^-20 relative each) and
    the output's rounding, so a single piece that is lost or counted twice
    shows."""
    dev = cuda_device
    g = np.random.default_rng(L[0])
    BS, B = 16, len(L)
    blocks = [-(-n // BS) for n in L]
    NB = sum(blocks) + 1
    table = np.zeros((B, max(blocks)), np.int32)
    perm = g.permutation(NB)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    codes, sf = api.fp4_kv_cache(NB, BS, Hkv, D, dev)
    codes.copy_(torch.from_numpy(g.integers(0, 256, codes.shape, np.uint8)))
    sf.view(torch.uint8).fill_(0x38)                # 1.0
    one = torch.ones(1, device=dev)
    v = api.dequantize_fp4_cache(codes[1], sf[1], one, dtype=torch.bfloat16)
    v = f32(v).astype(np.float64)
    T = sum(q_lens)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    out, lse = api.flash_attn_varlen_func(
        torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=dev), codes[0],
        codes[1], max(q_lens), torch.from_numpy(cu).to(dev), max(L),
        seqused_k=torch.tensor(L, dtype=torch.int32, device=dev),
        softmax_scale=1.0, causal=True,
        block_table=torch.from_numpy(table).to(dev), return_softmax_lse=True,
        k_descale=one, v_descale=one, k_block_scale=sf[0],
        v_block_scale=sf[1], **kw)
    o, lse = f32(out).astype(np.float64), lse.cpu().numpy()
    for b in range(B):
        rows = v[table[b]].reshape(-1, Hkv, D)[:L[b]].cumsum(0)
        for i in range(q_lens[b]):
            n = L[b] - q_lens[b] + i + 1
            want = np.repeat(rows[n - 1] / n, Hq // Hkv, axis=0)
            assert np.abs(lse[:, cu[b] + i] - np.log(n)).max() <= 1e-5
            err = np.abs(o[cu[b] + i] - want)
            assert (err <= 2.0 ** -8 * np.abs(want) + 6 * 2.0 ** -18).all()


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("idx", range(9))
def test_shares(cuda_device, idx, sinks):
    dev = cuda_device
    wl = shares(idx)
    cache = fill(wl, dev)
    z = np.linspace(-3, 5, wl.num_heads).astype(np.float32) if sinks else None
    kw = dict(s_aux=torch.from_numpy(z).to(dev)) if sinks else {}
    out, lse = attend(wl, dev, cache, max_k=4096, **kw)
    api.check_device_errors(dev)
    check(wl, out, lse, oracle_cache(wl)[1], sinks=z)
    again = attend(wl, dev, cache, max_k=4096, enable_pdl=False, **kw)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_shares_need_their_workspace(cuda_device):
    """A workspace without room for the shares' parts: one CTA a unit."""
    dev = cuda_device
    wl = shares(0)
    out, lse = attend(wl, dev, fill(wl, dev), max_k=4096,
                      workspace=torch.empty(0, dtype=torch.uint8, device=dev))
    api.check_device_errors(dev)
    check(wl, out, lse, oracle_cache(wl)[1])


@pytest.mark.parametrize("matrix", [0, 1])
def test_shares_nan_is_seen_only_by_its_rows(cuda_device, matrix):
    dev = cuda_device
    wl = workloads.build_workload("ns4", 8, [4, 1, 2], [5000, 300, 70], 4, 2,
                                  128, 16)
    cache = fill(wl, dev)
    codes, sf, ks, vs = cache
    nan = np.zeros(wl.q.shape, bool)
    # (request, key, rows that see it)
    for b, key, rows in ((0, 4998, slice(2, 4)), (0, 7, slice(0, 4)),
                         (2, 69, slice(6, 7))):
        blk, off = wl.block_table[b, key // 16], key % 16
        sf[matrix].view(torch.uint8)[blk, off, 1, 1] = 0x7F
        nan[rows, 2:4, slice(0, 128) if matrix == 0 else slice(16, 32)] = True
    out, lse = attend(wl, dev, cache)
    o = f32(out)
    assert np.array_equal(np.isnan(o), nan)
    assert np.array_equal(np.isnan(f32(lse)), nan.any(-1).T
                          if matrix == 0 else np.zeros(lse.shape, bool))
    check(wl, out, None, oracle_cache(wl)[1], keep=~nan)


@pytest.mark.parametrize("own_workspace", [True, False])
def test_shares_in_a_graph_follow_the_lengths(cuda_device, own_workspace):
    """A captured call of equal shares, replayed with other lengths (none, a
    long one) and with queries moved from
    one request to another."""
    dev = cuda_device
    wl = workload("gs4", 8, [1] * 6, [5000, 40, 2000, 0, 1, 3000], 16, 4, 128,
                  16)
    cache = fill(wl, dev)
    codes, sf, ks, vs = cache
    refs = oracle_cache(wl)[1]
    q, cu = wl.q.to(dev), torch.from_numpy(wl.cu_seqlens_q).to(dev)
    k = torch.from_numpy(wl.seq_lens).to(dev)
    bt = torch.from_numpy(wl.block_table).to(dev)
    out = torch.empty_like(q)

    def call(work=None, out=out, max_q=2, max_k=5000):
        return api.flash_attn_varlen_func(
            q, codes[0], codes[1], max_q, cu, max_k, seqused_k=k,
            softmax_scale=wl.softmax_scale, causal=True, block_table=bt,
            out=out, workspace=work, k_descale=ks, v_descale=vs,
            k_block_scale=sf[0], v_block_scale=sf[1])
    work = torch.empty(64 << 20, dtype=torch.uint8, device=dev)
    call(work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(work if own_workspace else None)
    full = wl.seq_lens.copy()
    for lens, cus in ((full, [0, 1, 2, 3, 4, 5, 6]),
                      ([0, 0, 0, 0, 0, 1], [0, 1, 2, 3, 4, 5, 6]),
                      ([17, 40, 1999, 0, 1, 2999], [0, 2, 2, 4, 4, 5, 6]),
                      ([5000, 33, 0, 0, 0, 0], [0, 2, 4, 4, 4, 4, 6])):
        wl.seq_lens = np.array(lens, np.int32)
        wl.cu_seqlens_q = np.array(cus, np.int32)
        wl.q_lens = np.diff(wl.cu_seqlens_q)
        k.copy_(torch.from_numpy(wl.seq_lens))
        cu.copy_(torch.from_numpy(wl.cu_seqlens_q))
        work.fill_(0xFF)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        check(wl, out, None, refs)
    api.check_device_errors(dev)


def test_two_streams_at_once(cuda_device):
    """Calls of equal shares and their appends on two streams, each with a
    workspace of its own, many times over."""
    dev = cuda_device
    jobs = []
    for seed in (3, 4):
        wl = workloads.build_workload("ts%d" % seed, seed, [1] * 24,
                                      [2500 - 97 * i for i in range(24)], 16,
                                      4, 128, 16)
        cache = fill(wl, dev)
        want = attend(wl, dev, cache)
        jobs.append((wl, cache, want, torch.cuda.Stream(dev),
                     wl.q.to(dev), torch.from_numpy(wl.cu_seqlens_q).to(dev),
                     torch.from_numpy(wl.seq_lens).to(dev),
                     torch.from_numpy(wl.block_table).to(dev),
                     wl.k_new.to(dev), wl.v_new.to(dev),
                     torch.from_numpy(wl.slot_mapping_new).to(dev), []))
    torch.cuda.synchronize()
    for _ in range(20):
        for wl, (codes, sf, ks, vs), _, st, q, cu, k, bt, kn, vn, sl, \
                outs in jobs:
            with torch.cuda.stream(st):
                api.reshape_and_cache_flash(
                    kn, vn, codes[0], codes[1], sl, "fp4", ks, vs,
                    k_block_scale=sf[0], v_block_scale=sf[1])
                outs.append(api.flash_attn_varlen_func(
                    q, codes[0], codes[1], 1, cu, wl.max_seqlen_k,
                    seqused_k=k, softmax_scale=wl.softmax_scale, causal=True,
                    block_table=bt, k_descale=ks, v_descale=vs,
                    k_block_scale=sf[0], v_block_scale=sf[1]))
    torch.cuda.synchronize()
    for wl, _, want, *_, outs in jobs:
        for out in outs:
            assert torch.equal(out, want[0])


def test_two_graphs_share_a_workspace(cuda_device):
    """Two captured calls of different shapes over one workspace, replayed
    in turn on one stream, with new inputs."""
    dev = cuda_device
    wls = [workloads.build_workload("g4", 8, [1] * 3, [900, 70, 2000], 16, 4,
                                    128, 16),
           workloads.build_workload("h4", 9, [60, 1], [200, 3000], 16, 4, 128,
                                    16)]
    work = torch.empty(64 << 20, dtype=torch.uint8, device=dev)
    runs = []
    for wl in wls:
        cache = fill(wl, dev)
        eager = attend(wl, dev, cache)
        t = dict(q=wl.q.to(dev), cu=torch.from_numpy(wl.cu_seqlens_q).to(dev),
                 k=torch.from_numpy(wl.seq_lens).to(dev),
                 bt=torch.from_numpy(wl.block_table).to(dev))
        out = torch.empty_like(t["q"])

        def call(t=t, out=out, wl=wl, cache=cache):
            codes, sf, ks, vs = cache
            return api.flash_attn_varlen_func(
                t["q"], codes[0], codes[1], wl.max_seqlen_q, t["cu"],
                wl.max_seqlen_k, seqused_k=t["k"],
                softmax_scale=wl.softmax_scale, causal=True,
                block_table=t["bt"], out=out, workspace=work, k_descale=ks,
                v_descale=vs, k_block_scale=sf[0], v_block_scale=sf[1])
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((graph, out, eager[0], t, cache, wl))
    work.fill_(0xFF)
    for _ in range(3):
        for graph, out, want, *_ in runs:
            out.zero_()
            graph.replay()
            assert torch.equal(out, want)
    # shorter sequences than captured
    graph, out, _, t, cache, wl = runs[0]
    t["k"].copy_(torch.tensor([5, 70, 0], dtype=torch.int32))
    graph.replay()
    wl.seq_lens = np.array([5, 70, 0], np.int32)
    check(wl, out, None, oracle_cache(wl)[1])


def test_write_then_attend_on_a_side_stream(cuda_device):
    dev = cuda_device
    wl = workloads.build_workload("t4", 8, [1] * 8, [2000] * 8, 32, 8, 128,
                                  16)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        cache = poisoned(wl, dev)
        ks, vs = scales(dev)
        codes, sf = cache
        for k, v, slots in ((wl.k_ctx, wl.v_ctx, wl.slot_mapping_ctx),
                            (wl.k_new, wl.v_new, wl.slot_mapping_new)):
            api.reshape_and_cache_flash(
                k.to(dev), v.to(dev), codes[0], codes[1],
                torch.from_numpy(slots).to(dev), "fp4", ks, vs,
                k_block_scale=sf[0], v_block_scale=sf[1])
        out, lse = attend(wl, dev, (codes, sf, ks, vs))
    side.synchronize()
    want = attend(wl, dev, fill(wl, dev))
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("D,neox", [(128, True), (64, False)])
def test_the_whole_chain(cuda_device, D, neox):
    """What a serving step runs: the projection's q, k, v through the head
    norms and the rotation into the 4-bit cache, then attention: a prompt,
    then two decode steps (one of two tokens), against float64 on the cache
    that the definition gives."""
    dev = cuda_device
    Hq, H, BS, NB = 8, 2, 16, 12
    rng = np.random.default_rng(D)
    g = torch.Generator().manual_seed(D)
    dt = torch.bfloat16
    table = torch.from_numpy(make_table(256, D)).float()
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(dt) for _ in "qk"]
    codes, sf = api.fp4_kv_cache(NB, BS, H, D, dev)
    sf.view(torch.uint8).fill_(0x7F)
    ks, vs = scales(dev)
    bt = rng.permutation(NB)[:6].astype(np.int32)[None]
    kref = np.full((NB, BS, H, D), np.nan)
    vref = np.full((NB, BS, H, D), np.nan)
    done = 0
    for n in (50, 1, 2):
        qkv = torch.randn(n, Hq + 2 * H, D, generator=g).to(dt)
        pos = np.arange(done, done + n)
        slots = bt[0][pos // BS].astype(np.int64) * BS + pos % BS
        d = qkv.to(dev)
        q = api.rope_reshape_and_cache(
            d[:, :Hq], d[:, Hq:Hq + H], d[:, Hq + H:], codes[0], codes[1],
            torch.from_numpy(slots).to(dev), torch.from_numpy(pos).to(dev),
            table.to(dev), kv_cache_dtype="fp4", k_scale=ks, v_scale=vs,
            k_block_scale=sf[0], v_block_scale=sf[1],
            q_weight=w[0].to(dev), k_weight=w[1].to(dev), is_neox=neox)
        done += n
        out, lse = api.flash_attn_varlen_func(
            q, codes[0], codes[1], n,
            torch.tensor([0, n], dtype=torch.int32, device=dev), done,
            seqused_k=torch.tensor([done], dtype=torch.int32, device=dev),
            causal=True, block_table=torch.from_numpy(bt).to(dev),
            return_softmax_lse=True, k_descale=ks, v_descale=vs,
            k_block_scale=sf[0], v_block_scale=sf[1])
        api.check_device_errors(dev)
        args = dict(neox=neox, dtype=np.float32)
        kf = norm_rope_ref(f32(qkv[:, Hq:Hq + H]), f32(w[1]), pos, f32(table),
                           **args)
        b, o = slots // BS, slots % BS
        kref[b, o] = dequantize_fp4_ref(*quantize_fp4_ref(kf, KS), KS)
        vref[b, o] = dequantize_fp4_ref(
            *quantize_fp4_ref(f32(qkv[:, Hq + H:]), VS), VS)
        qf = norm_rope_ref(f32(qkv[:, :Hq]), f32(w[0]), pos, f32(table),
                           **args)
        qf = torch.from_numpy(qf).to(dt)
        assert torch.equal(q.cpu(), qf)
        wl = workloads.build_workload("c4", 1, [n], [done], Hq, H, D, BS)
        wl.q, wl.block_table = qf, bt
        check(wl, out, lse, (kref, vref))


# ------------------------------------------------------------------ limits

@pytest.mark.parametrize("L,window,max_k,kw", [
    (300, 100, 0, {}), (300, 100, 0, dict(num_splits=1)),
    (300, 100, 0, dict(num_splits=3)), (300, 270, 0, dict(num_splits=3)),
    (300, 100, 0, dict(fixed_split_size=64)), (5000, 2500, 8000, {}),
    (5000, 4950, 8000, {})],
    ids=["auto", "1", "3", "3-partly", "fixed", "shares", "shares-partly"])
def test_a_window_past_a_short_table(cuda_device, L, window, max_k, kw):
    """A table row of 5 columns, whose request's window starts past them (or
    in them, at a key that is no multiple of 16): no column behind the row is
    looked at.  The row is a view of a wider table, whose other columns hold
    ids outside the cache: they would be reported."""
    dev = cuda_device
    wl = workload("k4", 8, [1, 3, 1], [70, L, L], 8, 2, 128, 16,
                  window_size=(window, -1))
    codes, sf, ks, vs = fill(wl, dev)
    table = torch.from_numpy(wl.block_table).to(dev)
    table[:, 5:] = 1 << 30
    out, lse = api.flash_attn_varlen_func(
        wl.q.to(dev), codes[0], codes[1], 3,
        torch.from_numpy(wl.cu_seqlens_q).to(dev), max(L, max_k),
        seqused_k=torch.from_numpy(wl.seq_lens).to(dev),
        softmax_scale=wl.softmax_scale, causal=True,
        window_size=wl.window_size, block_table=table[:, :5],
        return_softmax_lse=True, k_descale=ks, v_descale=vs,
        k_block_scale=sf[0], v_block_scale=sf[1], **kw)
    with pytest.raises(api.PkvError, match="beyond the table") as e:
        api.check_device_errors(dev)
    assert "block id outside" not in str(e.value)
    # the keys that the columns hold are seen, as if they were all
    o, kref, vref = f32(out).astype(np.float64), *oracle_cache(wl)[1]
    tol = 2.0 ** -11 + 2 * 1.05 * logit_error(wl, kref) + 2.0 ** -20
    for b in range(3):
        page = wl.block_table[b, :5]
        k, v = (x[page].reshape(80, 2, 128) for x in (kref, vref))
        n = int(wl.q_lens[b])
        for i in range(n):
            t, at = wl.cu_seqlens_q[b] + i, int(wl.seq_lens[b]) - n + i
            lo, hi = max(0, at - window), min(80, at + 1)
            if lo >= hi:
                assert not o[t].any() and torch.isneginf(lse[:, t]).all()
                continue
            for h in range(8):
                x = k[lo:hi, h // 4] @ f32(wl.q)[t, h] * wl.softmax_scale
                p = np.exp(x - x.max())
                want = p @ v[lo:hi, h // 4] / p.sum()
                assert (np.abs(o[t, h] - want) <= 2.0 ** -8 * np.abs(want) +
                        tol * np.abs(v[lo:hi]).max()).all()


@pytest.mark.parametrize("kw", [dict(num_splits=3), dict(fixed_split_size=64),
                                dict(num_splits=1)],
                         ids=["3", "fixed", "1"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_refused_rows_stay_under_splits(cuda_device, D, kw):
    """max_seqlen_q says 1 while a request has 3 queries of 4 heads: its rows
    are not computed, and the join of the splits leaves them alone too."""
    dev = cuda_device
    wl = workloads.build_workload("v4", 8, [1, 3, 1], [400, 900, 300], 4, 1,
                                  D, 16)
    codes, sf, ks, vs = fill(wl, dev)
    out = torch.full(wl.q.shape, 7.0, dtype=wl.torch_dtype, device=dev)
    api.flash_attn_varlen_func(
        wl.q.to(dev), codes[0], codes[1], 1,
        torch.from_numpy(wl.cu_seqlens_q).to(dev), wl.max_seqlen_k,
        seqused_k=torch.from_numpy(wl.seq_lens).to(dev), causal=True,
        block_table=torch.from_numpy(wl.block_table).to(dev), out=out,
        workspace=torch.zeros(8 << 20, dtype=torch.uint8, device=dev),
        k_descale=ks, v_descale=vs, k_block_scale=sf[0],
        v_block_scale=sf[1], **kw)
    with pytest.raises(api.PkvError, match="more queries than"):
        api.check_device_errors(dev)
    assert (out[1:4] == 7).all()
    check(wl, out, None, oracle_cache(wl)[1],
          keep=np.array([True, False, False, False, True]))


@pytest.mark.parametrize("kw", [dict(fixed_split_size=256),
                                dict(num_splits=1)], ids=["fixed", "1"])
@pytest.mark.parametrize("more", [{}, dict(softcap=30.0), dict(alibi=True)],
                         ids=["plain", "cap", "slopes"])
@pytest.mark.parametrize("D,q_lens", [(64, [1, 2]), (128, [1, 2]),
                                      (256, [1, 2]), (128, [1, 40])])
def test_bits_do_not_depend_on_the_batch(cuda_device, D, q_lens, more, kw):
    """A request whose rows fill one tile of 8 (8 heads a KV head), alone and
    beside one that makes the call use two: its window starts inside a key
    tile, so that a masked tile comes before unmasked ones."""
    dev = cuda_device
    q_lens, L, window = q_lens + [1] * 3, [900, 700, 815, 301, 77], 187
    wl = workload("b8", 11, q_lens, L, 16, 2, D, 16,
                  window_size=(window, -1), **more)
    codes, sf, ks, vs = cache = fill(wl, dev)
    whole = attend(wl, dev, cache, **kw)
    check(wl, whole[0], whole[1], oracle_cache(wl)[1])
    slopes = None if wl.alibi_slopes is None else \
        torch.from_numpy(wl.alibi_slopes).to(dev)
    for b, n in enumerate(q_lens):
        at = slice(wl.cu_seqlens_q[b], wl.cu_seqlens_q[b + 1])
        out, lse = api.flash_attn_varlen_func(
            wl.q[at].to(dev), codes[0], codes[1], n,
            torch.tensor([0, n], dtype=torch.int32, device=dev), L[b],
            seqused_k=torch.from_numpy(wl.seq_lens[b:b + 1]).to(dev),
            softmax_scale=wl.softmax_scale, causal=True,
            window_size=wl.window_size, softcap=wl.softcap,
            alibi_slopes=slopes,
            block_table=torch.from_numpy(wl.block_table[b:b + 1]).to(dev),
            return_softmax_lse=True, k_descale=ks, v_descale=vs,
            k_block_scale=sf[0], v_block_scale=sf[1], **kw)
        assert torch.equal(out, whole[0][at])
        assert torch.equal(lse, whole[1][:, at])


def one_hot_call(dev, logit_of, v_codes, D, dtype, k_scale, **kw):
    """One request of one head whose query is (1, 0, ...): key j's logit is
    k_scale * logit_of[j] (in -6 .. 6, E2M1 values) and its value row the
    codes v_codes[j], all block and value scales 1.  Returns out [D] and the
    LSE as float64, and the values [L, D]."""
    L, BS = len(logit_of), 16
    NB = -(-L // BS)
    mags = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    k = np.zeros((NB * BS, D // 2), np.uint8)
    v = np.zeros((NB * BS, D // 2), np.uint8)
    k[:L, 0] = np.searchsorted(mags, np.abs(logit_of)) + 8 * (logit_of < 0)
    v[:L] = v_codes
    codes, sf = api.fp4_kv_cache(NB, BS, 1, D, dev)
    codes[0, :, :, 0] = torch.from_numpy(k).view(NB, BS, -1).to(dev)
    codes[1, :, :, 0] = torch.from_numpy(v).view(NB, BS, -1).to(dev)
    sf.view(torch.uint8).fill_(0x38)                # 1.0
    q = torch.zeros(1, 1, D, dtype=DT[dtype], device=dev)
    q[0, 0, 0] = 1
    ks, one = scales(dev, k_scale, 1.0)
    out, lse = api.flash_attn_varlen_func(
        q, codes[0], codes[1], 1,
        torch.tensor([0, 1], dtype=torch.int32, device=dev), L,
        seqused_k=torch.tensor([L], dtype=torch.int32, device=dev),
        softmax_scale=1.0, causal=True,
        block_table=torch.arange(NB, dtype=torch.int32, device=dev)[None],
        return_softmax_lse=True, k_descale=ks, v_descale=one,
        k_block_scale=sf[0], v_block_scale=sf[1], **kw)
    nib = np.stack([v & 15, v >> 4], -1).reshape(NB * BS, D)[:L]
    vals = mags[nib & 7] * np.where(nib & 8, -1, 1)
    return f32(out)[0, 0].astype(np.float64), float(lse[0, 0]), vals


@pytest.mark.parametrize("kw", [dict(num_splits=1), {},
                                dict(fixed_split_size=8192)],
                         ids=["1", "auto", "fixed"])
@pytest.mark.parametrize("at", [0, 40000])
@pytest.mark.parametrize("D,dtype,gap", [
    (64, "bf16", 17.5), (128, "f16", 17.5), (256, "bf16", 17.5),
    (128, "bf16", 8.0), (64, "f16", 15.25), (128, "f16", 20.0)])
def test_small_weights_are_kept(cuda_device, D, dtype, gap, at, kw):
    """One key `gap` nats above 70000 others, with a value of 0: the output is
    the others' share.  A weight is held in f16 relative to 2^-9 of the
    largest: off by half a step, 2^-11 of itself or 2^-25.  The output is off
    by that share of the values' magnitudes (they are positive), the float32
    logit (2^-22 of it), exp2 and joins (2^-18 in all), the sum of the
    weights, and its rounding.  The sum is float32: a lane of one of the 4
    warps adds the keys of each of its subtiles of 16 to its sum, so at most
    L / 64 roundings by half a step, 2^-24 of a sum that is at most the whole.
    (A weight below 2^-25 of the lane's sum is lost to it: 2188 keys of
    2.5e-8 in the lane that has the large one, 5.5e-5, of 6.5e-5 allowed.)"""
    dev = cuda_device
    L = 70001
    g = np.random.default_rng(D)
    logits = np.zeros(L)
    logits[at] = 1
    v = g.integers(0, 8, (L, D)).astype(np.uint8)       # positive
    v = v[:, ::2] | v[:, 1::2] << 4
    v[at] = 0
    out, lse, vals = one_hot_call(dev, logits, v, D, dtype, gap, **kw)
    w = np.exp(logits * gap - gap)
    want = w @ vals / w.sum()
    held = 2.0 ** (9 - gap * np.log2(np.e))
    adds = -(-L // 64) * 2.0 ** -24
    rel = max(2.0 ** -11, 2.0 ** -25 / held) + gap * 2.0 ** -22 + \
        2.0 ** -18 + adds
    half = torch.finfo(DT[dtype]).eps / 2
    assert (np.abs(out - want) <= want * (rel + half * (1 + rel))).all()
    assert abs(lse - gap - np.log(w.sum())) <= 2.0 ** -20 * gap + \
        2.0 ** -18 + adds


@pytest.mark.parametrize("size", [3e4, 2e7, 4e7, 7e7, 1e8, 1.2e8, 3e8, 1e12])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("kw", [dict(num_splits=1), {}], ids=["1", "auto"])
def test_logits_far_from_zero(cuda_device, sign, size, kw):
    """Equal logits whose float32 step is above 1: the mean of the values."""
    L = 50
    g = np.random.default_rng(5)
    v = g.integers(0, 256, (L, 64)).astype(np.uint8)
    out, lse, vals = one_hot_call(cuda_device, np.full(L, float(sign)), v,
                                  128, "bf16", size, **kw)
    want = vals.mean(0)
    assert (np.abs(out - want) <= 2.0 ** -8 * np.abs(want) +
            6 * 2.0 ** -18).all()
    # (the logit in base 2 and back, each product rounded, and the sum)
    assert abs(lse - sign * size) <= size * 2.0 ** -21 + 2 * np.log(L)


def test_logits_far_apart(cuda_device):
    """Rising logits, each key far above the ones before it: the last key's
    value, whatever the steps of the references were."""
    dev = cuda_device
    steps = np.array([-6, -4, -3, -2, -1.5, -1, -.5, 0, .5, 1, 1.5, 2, 3, 4,
                      6.])
    g = np.random.default_rng(6)
    for scale in (20.0, 11.0, 3e7):
        logits = np.repeat(steps, 40)
        v = g.integers(0, 256, (600, 64)).astype(np.uint8)
        out, lse, vals = one_hot_call(dev, logits, v, 128, "f16", scale,
                                      num_splits=1)
        w = np.exp((logits - 6) * scale)
        want = w @ vals / w.sum()
        assert (np.abs(out - want) <= 2.0 ** -11 * np.abs(want) +
                6 * (2.0 ** -11 + 2.0 ** -18)).all()


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f16"),
                                     (256, "bf16")])
@pytest.mark.parametrize("L", [40001, 65536])
def test_join_of_many_parts(cuda_device, D, dtype, L):
    """One request in more than 128 parts whose weights differ by up to e^9
    from one run of 500 keys to the next (a part that is read from another's
    place shows): P rounds by 2^-11, exp2, the sums (a part's own below 256
    keys) and the join take 2^-17, the output half a step."""
    g = np.random.default_rng(L + D)
    steps = g.choice([-6, -3, -1, 0, 1, 2, 3], -(-L // 500))
    logits = np.repeat(steps.astype(float), 500)[:L]
    v = g.integers(0, 256, (L, D // 2)).astype(np.uint8)
    # (values of one sign in a run, so that sums do not cancel)
    sign = np.repeat(g.integers(0, 2, len(steps)), 500)[:L, None]
    v = ((v & 0x77) | np.where(sign, 0x88, 0)).astype(np.uint8)
    out, lse, vals = one_hot_call(cuda_device, logits, v, D, dtype, 1.0)
    w = np.exp(logits)
    want = w @ vals / w.sum()
    size = w @ np.abs(vals) / w.sum()
    half = torch.finfo(DT[dtype]).eps / 2
    assert (np.abs(out - want) <= half * np.abs(want) +
            size * (2.0 ** -11 + 2.0 ** -17)).all()
    assert abs(lse - np.log(w.sum())) <= 2.0 ** -17


@pytest.mark.parametrize("window,seen", [
    ((2 ** 30 + 2 ** 27, -1), 2 ** 30 + 2 ** 27 + 1),
    ((-1, 2 ** 31 - 1), None), ((2 ** 31 - 1, 2 ** 30), None),
    ((2 ** 28, 2 ** 31 - 1), 2 ** 28 + 1)])
def test_windows_over_more_than_2_30_keys(cuda_device, window, seen):
    """A table whose columns all name one of two blocks, so that a request may
    have 1.3e9 keys: with a query of zero the LSE is the
    logarithm of the number of keys seen and the output their mean."""
    dev = cuda_device
    BS, D, L = 1 << 16, 64, 2 ** 30 + 2 ** 28 + 5
    codes, sf = api.fp4_kv_cache(2, BS, 1, D, dev)
    codes.fill_(0x22)                               # 1.0
    sf.view(torch.uint8).fill_(0x38)
    one = torch.ones(1, device=dev)
    cols = -(-L // BS)
    table = torch.arange(cols, device=dev, dtype=torch.int32)[None] % 2
    out, lse = api.flash_attn_varlen_func(
        torch.zeros(1, 1, D, dtype=torch.bfloat16, device=dev), codes[0],
        codes[1], 1, torch.tensor([0, 1], dtype=torch.int32, device=dev), L,
        seqused_k=torch.tensor([L], dtype=torch.int32, device=dev),
        softmax_scale=1.0, causal=False, window_size=window,
        block_table=table, return_softmax_lse=True, k_descale=one,
        v_descale=one, k_block_scale=sf[0], v_block_scale=sf[1])
    api.check_device_errors(dev)
    # (the parts' and the whole LSE round to float32 near 16: 2^-20 each, and
    # the join's exp2 and log2 2^-20)
    assert abs(float(lse[0, 0]) - np.log(seen or L)) <= 2.0 ** -17
    assert (out == 1).all()


def test_decode_windows_past_2_30_over_16_bits(cuda_device):
    """Over a 16-bit cache too, windows that reach past every key hide nothing
    and leave the bits as they are."""
    dev = cuda_device
    wl = workloads.build_workload("w16", 5, [1, 2, 40], [700, 2500, 90], 8, 2,
                                  128, 16, causal=False)
    NB, BS, H, D = wl.cache_shape()[1:]
    cache = torch.zeros(2, NB, BS, H, D, dtype=wl.torch_dtype, device=dev)
    for k, v, slots in ((wl.k_ctx, wl.v_ctx, wl.slot_mapping_ctx),
                        (wl.k_new, wl.v_new, wl.slot_mapping_new)):
        api.reshape_and_cache_flash(k.to(dev), v.to(dev), cache[0], cache[1],
                                    torch.from_numpy(slots).to(dev))

    def call(window):
        return api.flash_attn_varlen_func(
            wl.q.to(dev), cache[0], cache[1], wl.max_seqlen_q,
            torch.from_numpy(wl.cu_seqlens_q).to(dev), wl.max_seqlen_k,
            seqused_k=torch.from_numpy(wl.seq_lens).to(dev),
            softmax_scale=wl.softmax_scale, causal=False, window_size=window,
            block_table=torch.from_numpy(wl.block_table).to(dev),
            num_splits=1)
    want = call((-1, -1))
    for window in ((2 ** 31 - 1, 2 ** 31 - 1), (-1, 2 ** 31 - 1), (-1, 43),
                   (2 ** 31 - 1, -1), (2 ** 31 - 44, 2 ** 30)):
        assert torch.equal(call(window), want)
