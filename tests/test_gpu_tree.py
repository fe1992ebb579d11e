"""A speculative decoding step on the GPU against the float64 reference:
attention of drafted trees, verification, compaction, and a run of them.

Tolerance of an attention output, from the arithmetic: the probabilities round
to the call's type (relative error at most half a step, eps / 2), so the output
moves by at most that times the largest |v| of the request's keys; it rounds
once more, by half a step of itself; the logits carry a float32 error d of at
most (D + 8) roundings of the sum of their terms' magnitudes (the soft-cap adds
a few roundings of the cap, the exponential and the joins of pieces 2^-20),
which scales every probability by at most e^(2 d).  Codes of a quantized cache
widen exactly, and their scales are float32 factors.  An LSE moves by d, the
exponential's and logarithm's 2^-20 and the roundings of its own size.

Verified tokens are whole numbers and have to be the reference's: the numbers u
are drawn so that no comparison is nearer than 1e-5 of its size (the kernel's
entries of R carry float32 roundings, 2^-24 of the row's own entry each, its
sums about 1e-13)."""
import numpy as np
import pytest
import torch

from oracle.tree import compact, tree_attention, verify
from paged_kv_cache_318_gb300 import api

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])
KS, VS = np.float32(.021), np.float32(.013)


@pytest.fixture(scope="module", autouse=True)
def built(cuda_device):
    from paged_kv_cache_318_gb300 import _build
    _build.build()
    api.load_library()
    api.check_device_errors(cuda_device)
    yield
    api.check_device_errors(cuda_device)


def flagged(dev):
    with pytest.raises(api.PkvError) as e:
        api.check_device_errors(dev)
    assert e.value.status == 5


def f64(t):
    return t.detach().double().cpu().numpy()


def ints(x, dev):
    return torch.from_numpy(np.asarray(x, np.int32)).to(dev)


def cumulate(ns):
    return np.concatenate([[0], np.cumsum(ns)])


def trees(rng, ns, reach):
    """Parents of each request's rows, up to `reach` rows back."""
    out = []
    for n in ns:
        i = np.arange(n)
        out.append(np.where(
            i > 0, np.maximum(i - rng.integers(1, reach + 1, n), 0), -1))
    return out


def view(kind, nb, bs, h, x, dtype, dev, layout):
    """An uninitialised cache view [nb, bs, h, x]: pages token by token,
    pages head by head, or with gaps between rows, tokens and pages."""
    if layout == "nhd":
        return torch.empty((nb, bs, h, x), dtype=dtype, device=dev)
    if layout == "hnd":
        return torch.empty((nb, h, bs, x), dtype=dtype,
                           device=dev).transpose(1, 2)
    es = torch.empty(0, dtype=dtype).element_size()
    pad = 16 // es
    return torch.empty((nb, bs + 1, h + 1, x + pad), dtype=dtype,
                       device=dev)[:, :bs, :h, :x]


class Draft:
    """Requests with ns[b] drafted rows behind Ls[b] - ns[b] keys of context,
    in a shuffled paged cache whose other places hold NaN."""

    def __init__(self, dev, ns, Ls, hq, hkv, d, bs, dtype=BF, kind="auto",
                 layout="nhd", reach=4, seed=0, spread=1.0, empty_tail=0):
        self.rng = rng = np.random.default_rng(seed)
        self.dev, self.ns, self.Ls, self.kind = dev, ns, Ls, kind
        self.hq, self.hkv, self.d, self.bs = hq, hkv, d, bs
        self.dtype = dtype
        B = len(ns)
        blocks = [-(-max(l, 0) // bs) for l in Ls]
        self.nb = nb = sum(blocks) + 2
        perm = rng.permutation(nb)
        table = np.full((B, max(max(blocks), 1) + 1), perm[-1], np.int32)
        at = 0
        for b, m in enumerate(blocks):
            table[b, :m] = perm[at:at + m]
            at += m
        self.table = table
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        used = np.zeros((nb, bs), bool)
        for b, l in enumerate(Ls):
            pos = np.arange(max(l, 0))
            used[table[b][pos // bs], pos % bs] = True
        spare = torch.from_numpy(~used).to(dev)
        self.caches, self.vals, self.kw = [], [], {}
        for name, s in (("k", KS), ("v", VS)):
            if kind == "auto":
                x = torch.randn((nb, bs, hkv, d), device=dev, generator=g)
                x = (x * (spread if name == "k" else 1)).to(dtype)
                x[spare] = float("nan")
                val = f64(x)
            elif kind == "fp8":
                x = (torch.randn((nb, bs, hkv, d), device=dev, generator=g) /
                     float(s)).to(torch.float8_e4m3fn)
                val = f64(x.float()) * s
                x.view(torch.uint8)[spare] = 0x7F
            else:
                x = torch.randint(0, 256, (nb, bs, hkv, d // 2), device=dev,
                                  generator=g, dtype=torch.uint8)
                f = (torch.rand((nb, bs, hkv, d // 16), device=dev,
                                generator=g) * 20 + 2).to(torch.float8_e4m3fn)
                c = x.cpu().numpy()
                val = np.stack([E2M1[c & 15], E2M1[c >> 4]], -1).reshape(
                    nb, bs, hkv, d) * np.repeat(f64(f.float()), 16, -1) * s
                f.view(torch.uint8)[spare] = 0x7F
                fc = view(kind, nb, bs, hkv, d // 16, f.dtype, dev, layout)
                fc.copy_(f)
                self.kw[name + "_block_scale"] = fc
            c = view(kind, nb, bs, hkv, x.shape[-1], x.dtype, dev, layout)
            if c.dtype == torch.float8_e4m3fn:
                c.view(torch.uint8).copy_(x.view(torch.uint8))
            else:
                c.copy_(x)
            self.caches.append(c)
            self.vals.append(val)
            if kind != "auto":
                self.kw[name + "_descale"] = torch.tensor([s], device=dev)
        self.cu = cumulate(ns)
        T = int(self.cu[-1])
        self.q = torch.randn((T + empty_tail, hq, d), device=dev,
                             generator=g).to(dtype)
        self.parents = trees(rng, ns, reach)
        self.tail = empty_tail

    def meta(self):
        par = np.concatenate(self.parents + [np.full(self.tail, -1)])
        return dict(cu_seqlens_q=ints(self.cu, self.dev),
                    seqused_k=ints(self.Ls, self.dev),
                    block_table=ints(self.table, self.dev),
                    tree_parents=ints(par, self.dev))

    def args(self, **kw):
        meta = {} if set(kw) >= {"cu_seqlens_q", "seqused_k", "block_table",
                                 "tree_parents"} else self.meta()
        a = dict(q=self.q, k=self.caches[0], v=self.caches[1],
                 max_seqlen_q=max(self.ns), max_seqlen_k=max(self.Ls),
                 causal=True, return_softmax_lse=True, **meta,
                 **self.kw)
        a.update(kw)
        return a

    def run(self, **kw):
        return api.flash_attn_varlen_func(**self.args(**kw))

    def rows(self, b):
        pos = np.arange(max(self.Ls[b], 0))
        return [x[self.table[b][pos // self.bs], pos % self.bs]
                for x in self.vals]

    def check(self, out, lse, window=-1, softcap=0.0, sinks=None, scale=None,
              requests=None):
        scale = self.d ** -0.5 if scale is None else scale
        eps = torch.finfo(self.dtype).eps
        out, lse = f64(out), f64(lse)
        for b in range(len(self.ns)) if requests is None else requests:
            n, L = self.ns[b], self.Ls[b]
            if n == 0:
                continue
            at = slice(self.cu[b], self.cu[b + 1])
            q = f64(self.q[at])
            k, v = self.rows(b)
            o, l = tree_attention(q, k, v, self.parents[b], scale, softcap,
                                  window, None if sinks is None
                                  else f64(sinks))
            size = max((abs(scale) *
                        np.abs(q).max() *
                        np.abs(k).sum(-1).max()) if L > 0 else 0, 0)
            d = 2.0 ** -24 * ((self.d + 8) * size + 32 * softcap)
            top = np.abs(v).max() if L > 0 else 0.0
            tol = top * (eps / 2 + np.expm1(2 * d) + 2.0 ** -20) * (1 + eps) \
                + np.abs(o) * eps / 2 + 2.0 ** -24
            got = out[at]
            assert np.isfinite(got).all()
            assert (np.abs(got - o) <= tol).all(), (
                b, np.abs(got - o).max(), float(np.min(tol)))
            dead = np.isneginf(l)
            assert (np.isneginf(lse[:, at]) == dead).all()
            if not dead.all():
                e = np.abs(lse[:, at][~dead] - l[~dead])
                lt = d + 2.0 ** -20 + 2.0 ** -22 * np.abs(l[~dead])
                assert (e <= lt).all(), (b, e.max(), lt.min())


# --------------------------------------------------------------- attention

SHAPES = [
    # ns, Ls, hq, hkv, d, bs
    ([7, 7], [37, 50], 4, 2, 64, 16),
    ([1], [1], 4, 4, 128, 16),
    ([2, 1, 3], [2, 500, 3], 6, 2, 128, 48),
    ([33, 5, 64], [533, 1005, 764], 8, 2, 128, 32),
    ([80, 3, 50], [780, 23, 350], 8, 2, 64, 64),
    ([13, 40], [900, 331], 10, 2, 256, 32),
    ([9, 256], [1000, 300], 2, 1, 128, 128),
    ([31, 17], [257, 1300], 16, 1, 128, 256),
    ([5] * 40, list(range(5, 2005, 50)), 8, 8, 64, 16),
]


@pytest.mark.parametrize("kind", ["auto", "fp8", "fp4"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_trees(cuda_device, shape, kind):
    dtype = (BF, HF)[shape % 2]
    t = Draft(cuda_device, *SHAPES[shape], dtype=dtype, kind=kind, seed=shape)
    t.check(*t.run())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", ["auto", "fp8", "fp4"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_types(cuda_device, d, kind, dtype):
    t = Draft(cuda_device, [12, 70, 3], [300, 700, 1200], 8, 2, d, 16, dtype,
              kind)
    t.check(*t.run())


@pytest.mark.parametrize("kind", ["auto", "fp8", "fp4"])
@pytest.mark.parametrize("layout", ["hnd", "gaps"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_layouts(cuda_device, d, layout, kind):
    t = Draft(cuda_device, [12, 40], [300, 620], 8, 2, d, 32, BF, kind,
              layout)
    t.check(*t.run())


@pytest.mark.parametrize("kind", ["auto", "fp4"])
@pytest.mark.parametrize("window", [0, 1, 5, 100, 5000])
@pytest.mark.parametrize("softcap", [0.0, 15.0])
def test_window_and_softcap(cuda_device, window, softcap, kind):
    t = Draft(cuda_device, [30, 7, 100], [630, 8, 777], 8, 2, 128, 16, BF,
              kind, spread=3.0)
    t.check(*t.run(window_size=(window, -1), softcap=softcap), window=window,
            softcap=softcap)


def test_pages_before_the_window_are_not_read(cuda_device):
    t = Draft(cuda_device, [10], [1000], 8, 2, 128, 16)
    want = t.run(window_size=(64, -1))
    t.table[0, :(1000 - 10 - 64) // 16] = t.table[0, -1]      # (NaN)
    spare = sorted(set(range(t.nb)) - set(t.table[0].tolist()))
    for c in t.caches:
        c[spare] = float("nan")
    got = t.run(window_size=(64, -1))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("scale", [0.0, -0.2, 2.0])
def test_scales_and_sinks(cuda_device, scale, d):
    t = Draft(cuda_device, [30, 7], [530, 7], 8, 2, d, 16, HF)
    sinks = torch.linspace(-2, 12, 8, device=cuda_device)
    t.check(*t.run(softmax_scale=scale, s_aux=sinks), sinks=sinks,
            scale=scale)


@pytest.mark.parametrize("kind", ["auto", "fp8"])
@pytest.mark.parametrize("d", [64, 256])
def test_requests_without_keys_or_rows(cuda_device, d, kind):
    """No rows; fewer keys than rows (the first rows see nothing, or only the
    keys of their ancestors); no keys."""
    t = Draft(cuda_device, [0, 4, 3, 0, 2], [9, 2, 0, 0, 40], 4, 2, d, 16,
              kind=kind)
    sinks = torch.zeros(4, device=cuda_device)
    t.check(*t.run())
    t.check(*t.run(s_aux=sinks), sinks=sinks)
    out, lse = t.run()
    assert (out[4:7] == 0).all() and torch.isneginf(lse[:, 4:7]).all()


def test_rows_behind_the_last_request_stay(cuda_device):
    t = Draft(cuda_device, [5, 9], [200, 300], 8, 2, 128, 16, empty_tail=7)
    out = torch.full_like(t.q, 42.0)
    got, lse = t.run(out=out, num_splits=1)
    assert got is out and (out[14:] == 42.0).all()
    t.check(out[:14], lse[:, :14])
    # a padded batch: requests without rows behind the others
    out.fill_(42.0)
    pad = dict(cu_seqlens_q=ints([0, 5, 14, 14, 14], cuda_device),
               seqused_k=ints([200, 300, 0, 9], cuda_device),
               block_table=ints(np.concatenate([t.table, t.table]),
                                cuda_device))
    _, lse = t.run(out=out, **pad)
    assert (out[14:] == 42.0).all()
    t.check(out[:14], lse[:, :14])


@pytest.mark.parametrize("kind", ["auto", "fp8", "fp4"])
def test_a_chain_is_the_causal_call(cuda_device, kind):
    t = Draft(cuda_device, [20, 6], [320, 800], 8, 2, 128, 16, BF, kind,
              reach=1)
    t.check(*t.run())
    t.check(*t.run(tree_parents=None))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_hidden_key_does_not_matter(cuda_device, d):
    """Whatever stands in the key rows of a row's cousins, it sees the same:
    bit for bit."""
    t = Draft(cuda_device, [40], [340], 8, 2, d, 16, reach=40)
    want, lse = t.run()
    out = f64(want)
    par = t.parents[0]
    bad = [j for j in range(1, 40) if (par != j).all()][:5]      # leaves
    for j in bad:
        pos = 300 + j
        t.caches[0][t.table[0][pos // 16], pos % 16] = float("nan")
    got, lse2 = t.run()
    rest = [i for i in range(40) if i not in bad]
    assert torch.equal(got[rest], want[rest])
    assert torch.equal(lse2[:, rest], lse[:, rest])
    assert torch.isnan(got[bad].float()).all() and np.isfinite(out).all()


def test_large_logits(cuda_device):
    """Maxima that climb from tile to tile, by more than f16 could hold."""
    t = Draft(cuda_device, [20, 70], [1500, 900], 8, 2, 128, 16, HF,
              spread=12.0)
    t.check(*t.run())


def test_one_block_per_unit_does_not_depend_on_the_batch(cuda_device):
    ns, Ls = [9, 30, 4, 70, 12], [700, 1500, 30, 2000, 333]
    t = Draft(cuda_device, ns, Ls, 8, 2, 128, 16)
    out, lse = t.run(num_splits=1)
    t.check(out, lse)
    for b in range(5):
        at = slice(t.cu[b], t.cu[b + 1])
        o, l = t.run(q=t.q[at], num_splits=1,
                     cu_seqlens_q=ints([0, ns[b]], cuda_device),
                     seqused_k=ints([Ls[b]], cuda_device),
                     block_table=ints(t.table[b:b + 1], cuda_device),
                     tree_parents=ints(t.parents[b], cuda_device),
                     max_seqlen_q=ns[b], max_seqlen_k=Ls[b])
        assert torch.equal(o, out[at]) and torch.equal(l, lse[:, at])


def test_a_short_workspace_works_unsplit(cuda_device):
    t = Draft(cuda_device, [9, 30], [3000, 1500], 8, 2, 128, 16)
    want = t.run(num_splits=1)
    small = torch.empty(256, dtype=torch.uint8, device=cuda_device)
    got = t.run(workspace=small)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_used_workspace(cuda_device):
    """Nothing in the workspace has to be set before a call."""
    t = Draft(cuda_device, [9, 30], [3000, 1500], 8, 2, 128, 16)
    n = api.load_library().pkv_paged_attention_workspace_size_tree(
        2, 39, 30, 3000, 8, 2, 128, 16, 0, None)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=cuda_device)
    got = t.run(workspace=ws)
    t.check(*got)
    again = t.run(workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_views_of_queries_and_outputs(cuda_device):
    t = Draft(cuda_device, [20, 6], [320, 800], 6, 2, 64, 16)
    wide = torch.full((26, 9, 72), 3.0, dtype=BF, device=cuda_device)
    wide[:, 1:7, :64] = t.q
    out = torch.full((26, 6, 80), 5.0, dtype=BF, device=cuda_device)
    got, lse = t.run(q=wide[:, 1:7, :64], out=out[:, :, :64])
    t.check(got, lse)
    assert (out[:, :, 64:] == 5.0).all()
    heads = torch.empty((6, 26, 64), dtype=BF, device=cuda_device)
    heads.copy_(t.q.transpose(0, 1))
    t.check(*t.run(q=heads.transpose(0, 1)))


@pytest.mark.parametrize("kind", ["auto", "fp8", "fp4"])
def test_many_requests_of_all_lengths(cuda_device, kind):
    rng = np.random.default_rng(5)
    ns = rng.integers(0, 30, 700).tolist()
    Ls = [n + int(c) for n, c in zip(ns, rng.integers(0, 300, 700))]
    t = Draft(cuda_device, ns, Ls, 4, 2, 64, 16, HF, kind)
    t.check(*t.run(), requests=range(0, 700, 7))


def test_shared_pages(cuda_device):
    """Requests whose contexts lie in the same pages."""
    t = Draft(cuda_device, [8, 8, 8], [168, 168, 168], 8, 2, 128, 16)
    t.table[1, :10] = t.table[2, :10] = t.table[0, :10]
    t.check(*t.run())


def test_flagged_requests(cuda_device):
    t = Draft(cuda_device, [5, 9, 4], [200, 300, 100], 8, 2, 128, 16)
    want, lse = t.run(num_splits=1)
    # more rows than max_seqlen_q: not computed
    out = torch.full_like(t.q, 42.0)
    t.run(max_seqlen_q=8, out=out, num_splits=1)
    flagged(cuda_device)
    assert (out[5:14] == 42.0).all()
    assert torch.equal(out[:5], want[:5]) and torch.equal(out[14:], want[14:])
    # parents that are no earlier row count as none
    for bad in (3, 7, -2, 1 << 30):
        par = np.concatenate(t.parents)
        par[5 + 3] = bad
        got, _ = t.run(tree_parents=ints(par, cuda_device), num_splits=1)
        flagged(cuda_device)
        par[5 + 3] = -1
        ref, _ = t.run(tree_parents=ints(par, cuda_device), num_splits=1)
        assert torch.equal(got, ref)
    api.check_device_errors(cuda_device)
    # a page outside the cache, and a table that ends before the keys
    for col, kw in ((2, {}), (None, dict(seqused_k=ints([200, 3000, 100],
                                                        cuda_device)))):
        table = t.table.copy()
        if col is not None:
            table[1, col] = t.nb
        got, _ = t.run(block_table=ints(table, cuda_device), num_splits=1,
                       **kw)
        flagged(cuda_device)
        assert torch.equal(got[:5], want[:5])
        assert torch.equal(got[14:], want[14:])


def test_other_stream_and_plain_launches(cuda_device):
    t = Draft(cuda_device, [9, 30], [3000, 1500], 8, 2, 128, 16)
    want = t.run()
    assert all(torch.equal(a, b) for a, b in
               zip(t.run(enable_pdl=False), want))
    s = torch.cuda.Stream(cuda_device)
    s.wait_stream(torch.cuda.current_stream(cuda_device))
    with torch.cuda.stream(s):
        got = t.run()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_calls_at_once(cuda_device):
    """Two streams, a workspace each."""
    a = Draft(cuda_device, [9, 30], [3000, 1500], 8, 2, 128, 16)
    b = Draft(cuda_device, [70], [2500], 8, 2, 256, 16, kind="fp8")
    wa, wb = a.run(), b.run()
    sa, sb = (torch.cuda.Stream(cuda_device) for _ in range(2))
    torch.cuda.synchronize(cuda_device)
    got = []
    for _ in range(10):
        with torch.cuda.stream(sa):
            ga = a.run()
        with torch.cuda.stream(sb):
            gb = b.run()
        got.append((ga, gb))
    torch.cuda.synchronize(cuda_device)
    for ga, gb in got:
        assert all(torch.equal(x, y) for x, y in zip(ga, wa))
        assert all(torch.equal(x, y) for x, y in zip(gb, wb))


@pytest.mark.parametrize("kind", ["auto", "fp8", "fp4"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("empty", [0, 1000, 6000])
def test_a_wait_that_runs_out(cuda_device, empty, splits, d, kind):
    """With a limit of 0 a wait gives up at its second poll, some 8 us on:
    without empty requests on the way a few blocks at head size 256 do, half
    way; with 1000 some of those that have to search for their share; with
    6000 all, before their first piece.  The call ends and is flagged; no row
    is joined from pieces that were not written (the workspace holds NaN), so
    what is written is right, and so is the next call."""
    dev = cuda_device
    ns = [9, 30] + [0] * empty + [70, 12]
    t = Draft(dev, ns, [3000, 1500] + [0] * empty + [2100, 4000], 8, 2, d, 16,
              kind=kind)
    ws = torch.empty(api.load_library().
                     pkv_paged_attention_workspace_size_tree(
                         len(ns), 121, 70, 4000, 8, 2, d, 16, 0, None),
                     dtype=torch.uint8, device=dev)
    a = t.args(num_splits=splits, workspace=ws)
    out, lse = api.flash_attn_varlen_func(**a)
    t.check(out, lse)
    a["out"] = torch.empty_like(out)
    status = []
    try:
        api.set_wait_limit_ns(0)
        for _ in range(5):
            ws.fill_(255)
            a["out"].fill_(42.0)
            api.flash_attn_varlen_func(**a)
            try:
                api.check_device_errors(dev)
            except api.PkvError as e:
                status.append(e.status)
            assert ((a["out"] == 42.0) | (a["out"] == out)).all()
            if empty == 6000:
                assert (a["out"] == 42.0).all()
    finally:
        api.set_wait_limit_ns(api.WAIT_LIMIT_DEFAULT_NS)
    assert set(status) <= {api.PKV_ERR_TIMEOUT}
    assert status or empty < 6000
    got, lse2 = api.flash_attn_varlen_func(**a)
    api.check_device_errors(dev)
    assert torch.equal(got, out) and torch.equal(lse2, lse)


def test_captured_and_replayed(cuda_device):
    """A graph over largest sizes, replayed with other lengths."""
    ns, Ls = [9, 30, 4], [700, 1500, 30]
    t = Draft(cuda_device, ns, Ls, 8, 2, 128, 16)
    a = t.args(max_seqlen_q=64, max_seqlen_k=4096)
    out = torch.empty_like(t.q)
    ws = torch.empty(api.load_library().
                     pkv_paged_attention_workspace_size_tree(
                         3, 43, 64, 4096, 8, 2, 128, 16, 0, None),
                     dtype=torch.uint8, device=cuda_device)
    a.update(out=out, workspace=ws)
    s = torch.cuda.Stream(cuda_device)
    s.wait_stream(torch.cuda.current_stream(cuda_device))
    with torch.cuda.stream(s):
        api.flash_attn_varlen_func(**a)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, lse = api.flash_attn_varlen_func(**a)
    t.ns, t.Ls = [30, 4, 9], [1000, 8, 700]
    t.table = t.table[[1, 2, 0]]
    t.parents = trees(t.rng, t.ns, 5)
    t.cu = cumulate(t.ns)
    for k, v in t.meta().items():
        a[k].copy_(v)
    out.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize(cuda_device)
    t.check(out, lse)


def test_offsets_past_32_bits(cuda_device):
    """Pages 5 GB apart in a cache of codes; 2^31 elements and more behind
    one another in a 16-bit one."""
    d, bs, hkv = 128, 16, 1
    nb = 1 + (5 << 30) // (bs * d)
    big = torch.empty((nb, bs, hkv, d), dtype=torch.uint8, device=cuda_device)
    t = Draft(cuda_device, [9], [40], 4, hkv, d, bs, kind="fp8")
    far = [nb - 1 - 3 * i for i in range(t.nb)]
    for i, f in enumerate(far):
        big[f] = t.caches[0].view(torch.uint8)[i]
    k = big.view(torch.float8_e4m3fn)
    t.vals[1] = t.vals[0]
    got = t.run(k=k, v=k, v_descale=t.kw["k_descale"],
                block_table=ints(np.array(far)[t.table], cuda_device))
    t.check(*got)
    half = big.view(BF)                       # [nb, bs, 1, 64]
    u = Draft(cuda_device, [9], [40], 4, hkv, 64, bs)
    for i, f in enumerate(far[:u.nb]):
        half[f] = u.caches[0][i]
    u.vals[1] = u.vals[0]
    u.check(*u.run(k=half, v=half, block_table=ints(np.array(far)[u.table],
                                                    cuda_device)))


# ------------------------------------------------------------ verification

def clear(target, tokens, uniform, parents, draft):
    """Whether every comparison of the reference is farther than 1e-5 of its
    sides apart: the float64 walk, with a margin."""
    n, vocab = target.shape
    node, rest, mass = 0, np.maximum(target[0], 0.0), 1.0
    near = lambda a, b: abs(a - b) <= 1e-5 * max(abs(a), abs(b))
    for i in range(1, n):
        x = int(tokens[i])
        if parents[i] != node or not 0 <= x < vocab:
            continue
        likely = 1.0 if draft is None else draft[node, x]
        a = float(uniform[i]) * likely * mass
        if near(a, rest[x]) and max(a, rest[x]) > 0:
            return False
        if a < rest[x]:
            node, rest, mass = i, np.maximum(target[i], 0.0), 1.0
        elif draft is None:
            mass = max(mass - rest[x], 0.0)
            rest[x] = 0.0
        else:
            rest = np.maximum(rest - mass * draft[node], 0.0)
            mass = rest.sum()
    if not rest.sum() > 0:
        rest = np.maximum(target[node], 0.0)
    run = np.cumsum(rest)
    if not run[-1] > 0:
        return True
    at = float(uniform[0]) * run[-1]
    # (the nearest running sum, next to the entries' own roundings)
    return np.abs(run - at).min() > 1e-6 * run[-1] / max(
        1.0, vocab / 1000.0) or float(uniform[0]) == 0.0


class Check:
    def __init__(self, dev, ns, vocab, dtype=torch.float32, reach=3,
                 sampled=False, sharp=3.0, seed=0, chain=False, pad=(0, 0)):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        self.ns, self.dev, self.cu = ns, dev, cumulate(ns)
        T = int(self.cu[-1])
        lg = torch.randn((T, vocab), device=dev, generator=g) * sharp
        near = lg + torch.randn((T, vocab), device=dev, generator=g) * .7

        def rows(x, gap):
            y = torch.zeros((T, vocab + gap), dtype=dtype, device=dev)
            y = y[:, gap // 2:gap // 2 + vocab]
            return y.copy_(torch.softmax(x, -1))
        self.p = rows(lg, pad[0])
        self.q = rows(near, pad[1]) if sampled else None
        self.parents = trees(rng, ns, 1 if chain else reach)
        self.chain = chain
        self.tok = np.zeros(T, np.int32)
        cand = torch.topk(near, min(4, vocab)).indices.cpu().numpy()
        for b, n in enumerate(ns):
            for j in range(1, n):
                row = self.cu[b] + self.parents[b][j]
                self.tok[self.cu[b] + j] = rng.choice(cand[row]) \
                    if not sampled or j % 2 else int(torch.multinomial(
                        torch.softmax(near[row], -1), 1, generator=g))
        self.u = rng.random(T).astype(np.float32)
        p, q = f64(self.p), None if self.q is None else f64(self.q)
        self.want = []
        for b in range(len(ns)):
            at = slice(self.cu[b], self.cu[b + 1])
            a = lambda: (p[at], self.tok[at], self.u[at], self.parents[b],
                         None if q is None else q[at])
            while ns[b] and not clear(*a()):
                self.u[at] = rng.random(ns[b])
            self.want.append(verify(*a()) if ns[b] else ([], []))

    def args(self):
        return [self.p, ints(self.tok, self.dev), ints(self.cu, self.dev),
                max(self.ns), torch.from_numpy(self.u).to(self.dev),
                None if self.chain else ints(np.concatenate(self.parents),
                                             self.dev), self.q]

    def check(self, tokens, rows, counts):
        tokens, rows, counts = (t.cpu().numpy() for t in
                                (tokens, rows, counts))
        for b, (said, stand) in enumerate(self.want):
            k = len(stand)
            assert counts[b] == k
            assert rows[b, :k].tolist() == stand
            assert tokens[b, :k].tolist() == said
            assert (rows[b, k:] == -1).all() and (tokens[b, k:] == -1).all()


@pytest.mark.parametrize("sampled", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, BF, HF])
@pytest.mark.parametrize("vocab", [3, 17, 1003, 1024, 5000, 32001, 100003])
def test_verification(cuda_device, vocab, dtype, sampled):
    c = Check(cuda_device, [5, 1, 0, 24, 9, 13], vocab, dtype, 4, sampled,
              sharp=min(3.0, .5 + vocab / 3000))
    c.check(*api.verify_draft_tokens(*c.args()))


@pytest.mark.parametrize("sampled", [False, True])
@pytest.mark.parametrize("batch", [1, 7, 40, 100, 200])
def test_verification_of_batches(cuda_device, batch, sampled):
    """Every number of blocks to a request."""
    rng = np.random.default_rng(batch)
    c = Check(cuda_device, rng.integers(1, 12, batch).tolist(), 9001,
              reach=2, sampled=sampled, seed=batch)
    c.check(*api.verify_draft_tokens(*c.args()))


@pytest.mark.parametrize("sampled", [False, True])
def test_verification_of_chains(cuda_device, sampled):
    c = Check(cuda_device, [6, 2, 1, 8], 2000, sampled=sampled, chain=True)
    c.check(*api.verify_draft_tokens(*c.args()))


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("pad", [(3, 3), (2, 5), (7, 0), (0, 1)])
def test_verification_of_unaligned_rows(cuda_device, pad, dtype):
    c = Check(cuda_device, [6, 20, 3], 3001, dtype, sampled=True, pad=pad)
    c.check(*api.verify_draft_tokens(*c.args()))


def test_verification_of_the_largest_trees(cuda_device):
    c = Check(cuda_device, [256, 100, 1], 1500, reach=40, sampled=True,
              sharp=.4)
    c.check(*api.verify_draft_tokens(*c.args()))
    c = Check(cuda_device, [256, 255], 700, reach=250, sharp=.2)
    c.check(*api.verify_draft_tokens(*c.args()))


def test_verification_of_the_largest_vocabulary(cuda_device):
    c = Check(cuda_device, [3, 2], 1 << 20, BF, sampled=True)
    c.check(*api.verify_draft_tokens(*c.args()))


@pytest.mark.parametrize("max_n", [0, 3])
def test_verification_of_requests_without_rows(cuda_device, max_n):
    d = cuda_device
    tok, rows, cnt = api.verify_draft_tokens(
        torch.empty((0, 100), device=d), ints([], d), ints([0, 0, 0], d),
        max_n, torch.empty(0, device=d), ints([], d))
    assert tok.shape == rows.shape == (2, max_n)
    assert (tok == -1).all() and (rows == -1).all() and cnt.tolist() == [0, 0]


def test_attention_of_requests_without_rows(cuda_device):
    t = Draft(cuda_device, [0, 0], [9, 30], 4, 2, 64, 16)
    out, lse = t.run()
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)


def one(dev, p, tok, u, par, q=None):
    p = torch.tensor(p, dtype=torch.float32, device=dev)
    n = p.shape[0]
    out = api.verify_draft_tokens(
        p, ints(tok, dev), ints([0, n], dev), n,
        torch.tensor(u, dtype=torch.float32, device=dev), ints(par, dev),
        None if q is None else torch.tensor(q, dtype=torch.float32,
                                            device=dev))
    m = int(out[2][0])
    return out[0][0, :m].tolist(), out[1][0, :m].tolist()


def test_verification_at_the_edges(cuda_device):
    d = cuda_device
    P = [[.5, .25, .25, 0], [.125, .25, .375, .25], [0, 0, 1, 0]]
    Q = [[1.0] * 4] * 3
    # the draft covers the target: nothing is left, the target's row stays
    assert one(d, P, [0, 3, 0], [.6, .5, .9], [-1, 0, 1], Q) == ([1], [0])
    # a row without mass; numbers of 0, 1, more and less
    assert one(d, [[0.0] * 5], [0], [.5], [-1]) == ([-1], [0])
    assert one(d, [[0, .5, .5, 0]], [0], [0.0], [-1]) == ([1], [0])
    assert one(d, [[0, .5, .5, 0]], [0], [-1.0], [-1]) == ([1], [0])
    for u in (1.0, 7.0):
        assert one(d, [[0, .5, .5, 0]], [0], [u], [-1]) == ([2], [0])
    # equality does not stand; the same token twice is refused twice
    assert one(d, P, [0, 0, 1], [0., .5, .5], [-1, 0, 0]) == ([2], [0])
    assert one(d, P, [0, 0, 0], [0., .6, .0], [-1, 0, 0]) == ([1], [0])
    # negative and NaN probabilities count as none
    nan = float("nan")
    assert one(d, [[-1, nan, .5, -3]], [0], [.9], [-1]) == ([2], [0])
    assert one(d, [[.5, nan, .5, 0]] * 2, [0, 1], [.9, 0.], [-1, 0]) == \
        ([2], [0])
    api.check_device_errors(d)


@pytest.mark.parametrize("bad", [-.2, -1e30, float("-inf"), float("nan")])
@pytest.mark.parametrize("vocab", [4, 2000])
def test_negative_draft_probabilities_count_as_none(cuda_device, vocab, bad):
    """In 2000 entries: of the vectors that a row reads whole."""
    d = cuda_device

    def row(*x):
        return list(x) + [0.0] * (vocab - len(x))
    P = [row(.5, .5), row(0, 0, 1)]
    # a token of the draft below 0 that the target does not have either
    assert one(d, P, [0, 2], [.7, .5], [-1, 0], [row(.6, .6, bad, 0)] * 2) \
        == ([1], [0])
    # ... that the target has: it stands with whatever number
    assert one(d, P, [0, 1], [0., .99], [-1, 0], [row(1, bad)] * 2) == \
        ([1, 2], [0, 1])
    # entries below 0 beside a refused token add nothing to what is left:
    # [0, .25, .25] twice over, with u_0 at .4 and .6 of it
    P = [row(.5, .25, .25), row(1), row(1)]
    Q = [row(.75, bad, 0, bad)] * 3
    assert one(d, P[:2], [0, 0], [.4, .9], [-1, 0], Q[:2]) == ([1], [0])
    assert one(d, P, [0, 0, 0], [.6, .9, .9], [-1, 0, 0], Q) == ([2], [0])
    assert one(d, P, [0, 0, 3], [.6, .9, 0.], [-1, 0, 0], Q) == ([2], [0])
    api.check_device_errors(d)


@pytest.mark.parametrize("tok,par", [
    (1000, 0), (-1, 0), (1 << 30, 0), (3, 1), (3, 2), (3, -2), (3, 1 << 30)])
def test_verification_flags(cuda_device, tok, par):
    """A row with a token outside the vocabulary or a parent that is no
    earlier row never stands; the others do as without it."""
    c = Check(cuda_device, [4, 3, 5], 1000, seed=3)
    a = c.args()
    t, p = c.tok.copy(), np.concatenate(c.parents)
    t[c.cu[1] + 1], p[c.cu[1] + 1] = tok, par
    a[1], a[5] = ints(t, cuda_device), ints(p, cuda_device)
    got = api.verify_draft_tokens(*a)
    flagged(cuda_device)
    t[c.cu[1] + 1], p[c.cu[1] + 1] = 0, -1          # (a second root)
    at = slice(c.cu[1], c.cu[2])
    c.want[1] = verify(f64(c.p)[at], t[at], c.u[at], p[at])
    c.check(*got)


def test_verification_of_too_many_rows(cuda_device):
    c = Check(cuda_device, [4, 9, 5], 1000, seed=4)
    a = c.args()
    a[3] = 8
    got = api.verify_draft_tokens(*a)
    flagged(cuda_device)
    c.want[1] = ([], [])
    c.check(*got)


def test_verification_captured_elsewhere_and_twice(cuda_device):
    c = Check(cuda_device, [5, 1, 0, 24, 9, 13], 5000, sampled=True)
    a = c.args()
    want = api.verify_draft_tokens(*a)
    s = torch.cuda.Stream(cuda_device)
    s.wait_stream(torch.cuda.current_stream(cuda_device))
    with torch.cuda.stream(s):
        got = api.verify_draft_tokens(*a)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    out = tuple(torch.full_like(x, 7) for x in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = api.verify_draft_tokens(*a, out=out)
    other = Check(cuda_device, [5, 1, 0, 24, 9, 13], 5000, sampled=True,
                  seed=1)
    for x, y in zip(a, other.args()):
        if isinstance(x, torch.Tensor):
            x.copy_(y)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize(cuda_device)
    assert all(x is y for x, y in zip(res, out))
    other.check(*out)


# -------------------------------------------------------------- compaction

def drafts(rng, ns, ctxs, bs, spare=2):
    lens = [n + c for n, c in zip(ns, ctxs)]
    blocks = [-(-l // bs) for l in lens]
    perm = rng.permutation(sum(blocks) + spare)
    table = np.full((len(ns), max(max(blocks), 1)), perm[-1], np.int32)
    at = 0
    for b, m in enumerate(blocks):
        table[b, :m] = perm[at:at + m]
        at += m
    rows = np.full((len(ns), max(max(ns), 1)), -1, np.int32)
    cnt = np.zeros(len(ns), np.int32)
    for b, n in enumerate(ns):
        if n:
            k = int(rng.integers(0, n))
            rows[b, 0] = 0
            rows[b, 1:k + 1] = np.sort(rng.permutation(n - 1)[:k] + 1)
            cnt[b] = k + 1
    return lens, len(perm), table, rows, cnt


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("layout", ["nhd", "hnd", "gaps"])
@pytest.mark.parametrize("dtype,x", [
    (BF, 128), (HF, 64), (torch.uint8, 64), (torch.float8_e4m3fn, 8),
    (torch.float8_e4m3fn, 4), (torch.float32, 3), (BF, 3),
    (torch.uint8, 5)])
def test_compaction(cuda_device, dtype, x, layout):
    rng = np.random.default_rng(0)
    ns, ctxs, bs = [9, 1, 0, 100, 30, 256, 2], [0, 5, 7, 44, 16, 3, 31], 16
    lens, nb, table, rows, cnt = drafts(rng, ns, ctxs, bs)
    if layout == "gaps" and dtype == torch.uint8 and x == 5:
        x = 7
    caches = []
    for _ in range(3):
        c = view("", nb, bs, 3, x, dtype, cuda_device, layout)
        es = c.element_size()
        c.copy_(torch.from_numpy(rng.integers(
            0, 256, (nb, bs, 3, x * es), dtype=np.uint8)).to(
                cuda_device).view(dtype) if dtype != torch.float8_e4m3fn else
            torch.randn((nb, bs, 3, x), device=cuda_device).to(dtype))
        caches.append(c)
    want = [raw(c) for c in caches]
    for b, n in enumerate(ns):
        want = [compact(w, table[b], ctxs[b], rows[b, :cnt[b]]) for w in want]
    api.compact_draft_cache(caches, ints(table, cuda_device),
                            ints(cumulate(ns), cuda_device),
                            ints(lens, cuda_device), ints(rows, cuda_device),
                            ints(cnt, cuda_device))
    for w, c in zip(want, caches):
        np.testing.assert_array_equal(raw(c), w)


def test_compaction_of_many_caches(cuda_device):
    """More caches than a launch takes, and wide tables and rows."""
    rng = np.random.default_rng(1)
    ns, ctxs = [7, 12], [20, 3]
    lens, nb, table, rows, cnt = drafts(rng, ns, ctxs, 16)
    whole = torch.randn((300, 2, nb, 16, 2, 8), device=cuda_device).to(BF)
    caches = [whole[l, i] for l in range(300) for i in range(2)]
    want = [raw(c) for c in caches]
    for b in range(2):
        want = [compact(w, table[b], ctxs[b], rows[b, :cnt[b]]) for w in want]
    wide = np.full((2, 40), -7, np.int32)
    wide[:, :rows.shape[1]] = rows
    big = np.full((2, 90), 1 << 30, np.int32)
    big[:, :table.shape[1]] = table
    api.compact_draft_cache(
        caches, ints(big, cuda_device)[:, :table.shape[1]],
        ints(cumulate(ns), cuda_device), ints(lens, cuda_device),
        ints(wide, cuda_device)[:, :rows.shape[1]], ints(cnt, cuda_device))
    for w, c in zip(want, caches):
        np.testing.assert_array_equal(raw(c), w)


def test_compaction_flags(cuda_device):
    """Rows that do not grow or lie outside, pages outside the cache and keys
    behind the table: left out and flagged, the rest moves."""
    dev = cuda_device
    table = np.array([[1, 0], [2, 3]], np.int32)
    cu, lens = ints([0, 6, 12], dev), [20, 26]

    def run(rows, cnt, table=table, lens=lens):
        c = torch.arange(5 * 16, device=dev, dtype=torch.int32).view(
            5, 16, 1, 1).clone()
        api.compact_draft_cache(c, ints(table, dev), cu, ints(lens, dev),
                                ints(rows, dev), ints(cnt, dev))
        return raw(c).view(np.int32).ravel()

    base = np.arange(80)
    same = run([[0, 1, 2]] * 2, [3, 3])
    np.testing.assert_array_equal(same, base)
    api.check_device_errors(dev)
    for bad in ([0, 3, 2], [0, 6, 9], [0, -1, 3], [5, 1, 1]):
        got = run([bad, [0, 2, 5]], [3, 3])
        flagged(dev)
        # request 1 lies behind 20 keys of pages 2 and 3
        assert got[3 * 16 + 5] == 3 * 16 + 6
        assert got[3 * 16 + 6] == 3 * 16 + 9
    for t in (5, -1):
        got = run([[0, 2, 5], [0, 2, 5]], [3, 3],
                  np.array([[1, t], [2, 3]], np.int32))
        flagged(dev)
        assert got[1 * 16 + 15] == 1 * 16 + 15     # (its source is out)
        assert got[3 * 16 + 5] == 3 * 16 + 6
    got = run([[0, 2, 5], [0, 2, 5]], [3, 3], lens=[60, 26])
    flagged(dev)
    assert got[3 * 16 + 5] == 3 * 16 + 6 and (got[:32] == base[:32]).all()
    # no rows of the request, fewer keys than rows, no count
    got = run([[0, 2, 5], [0, 2, 5]], [0, -4])
    np.testing.assert_array_equal(got, base)
    api.check_device_errors(dev)
    got = run([[0, 2, 5], [0, 2, 5]], [3, 0], lens=[4, 26])
    flagged(dev)
    np.testing.assert_array_equal(got, base)


def test_compaction_of_more_rows_than_are_given(cuda_device):
    """The rows that are there move; the call is flagged, unless the request
    has no rows at all."""
    dev = cuda_device
    c = torch.arange(5 * 16, device=dev, dtype=torch.int32).view(5, 16, 1, 1)
    c = c.clone()
    a = (c, ints([[1, 0], [2, 3]], dev), ints([0, 6, 6], dev),
         ints([20, 26], dev), ints([[0, 2, 5], [0, 1, 2]], dev))
    api.compact_draft_cache(*a, ints([3, 4], dev))
    api.check_device_errors(dev)
    want = compact(np.arange(80).reshape(5, 16, 1, 1), np.array([1, 0]), 14,
                   [0, 2, 5]).ravel()
    np.testing.assert_array_equal(raw(c).view(np.int32).ravel(), want)
    for cnt in ([4, 0], [1 << 30, 3]):
        c.copy_(torch.arange(80, dtype=torch.int32).view_as(c))
        api.compact_draft_cache(*a, ints(cnt, dev))
        flagged(dev)
        np.testing.assert_array_equal(raw(c).view(np.int32).ravel(), want)


def test_compaction_past_32_bits(cuda_device):
    nb = 1 + (5 << 30) // (16 * 256)
    c = torch.zeros((nb, 16, 1, 256), dtype=torch.uint8, device=cuda_device)
    c[nb - 1, 3] = 9
    api.compact_draft_cache(
        c, ints([[nb - 2, nb - 1]], cuda_device), ints([0, 6], cuda_device),
        ints([21], cuda_device), ints([[0, 4]], cuda_device),
        ints([2], cuda_device))
    assert (c[nb - 1, 0] == 9).all() and (c[nb - 1, 3] == 9).all()
    assert (c[nb - 2] == 0).all() and (c[nb - 1, 1:3] == 0).all()


# ------------------------------------------------------- the step as a whole

def step(dev, kind, dtype, layers, ns, ctxs, hq, hkv, d, bs, vocab, seed,
         graph):
    """Attention over the drafts in every layer, verification, compaction;
    then what a next step reads has to be what a cache that never held the
    refused tokens gives."""
    layer = [Draft(dev, ns, [n + c for n, c in zip(ns, ctxs)], hq, hkv, d,
                   bs, dtype, kind, seed=seed) for _ in range(layers)]
    lead = layer[0]
    for i, l in enumerate(layer):
        l.q = torch.roll(l.q, i, 0)
        l.table, l.parents = lead.table, lead.parents
    ver = Check(dev, ns, vocab, sampled=True, reach=4, seed=seed, sharp=1.0)
    ver.parents = lead.parents
    meta = lead.meta()
    flat = [c for l in layer for c in l.caches]
    scales = [l.kw[k] for l in layer for k in ("k_block_scale",
                                               "v_block_scale")
              if k in l.kw]
    before = [raw(c) for c in flat + scales]

    def go():
        outs = [l.run(**meta) for l in layer]
        a = ver.args()
        tok, rows, cnt = api.verify_draft_tokens(
            a[0], ids, meta["cu_seqlens_q"], a[3], uni,
            meta["tree_parents"], a[6])
        for group in (flat, scales):
            api.compact_draft_cache(group, meta["block_table"],
                                    meta["cu_seqlens_q"], meta["seqused_k"],
                                    rows, cnt)
        return outs, tok, rows, cnt
    ids = ints(ver.tok, dev)
    uni = torch.from_numpy(ver.u).to(dev)
    if graph:
        keep = [c.clone() for c in flat + scales]
        s = torch.cuda.Stream(dev)
        s.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(s):
            go()
        s.synchronize()
        for c, k in zip(flat + scales, keep):
            c.copy_(k)
        g = torch.cuda.CUDAGraph()
        fixed = ver.args()
        ver.args = lambda: fixed
        with torch.cuda.graph(g):
            outs, tok, rows, cnt = go()
        g.replay()
        torch.cuda.synchronize(dev)
    else:
        outs, tok, rows, cnt = go()
    for l, o in zip(layer, outs):
        l.check(*o)
    p, q = f64(ver.p), f64(ver.q)
    stand = []
    for b, n in enumerate(ns):
        at = slice(lead.cu[b], lead.cu[b + 1])
        said, way = verify(p[at], ver.tok[at], ver.u[at], lead.parents[b],
                           q[at])
        k = int(cnt[b])
        assert tok[b, :k].tolist() == said and rows[b, :k].tolist() == way
        stand.append(way)
    for c, w in zip(flat + scales, before):
        for b in range(len(ns)):
            w = compact(w, lead.table[b], ctxs[b], stand[b])
        np.testing.assert_array_equal(raw(c), w)
    # the next step: a draft of m rows whose keys are written behind the
    # tokens that stand; its context has to be the kept rows
    lens = [c + len(w) for c, w in zip(ctxs, stand)]
    for l in layer:
        l.vals = [np.array(v) for v in l.vals]
        for v in l.vals:
            for b in range(len(ns)):
                v[:] = compact(v, l.table[b], ctxs[b], stand[b])
        rows_of = [len(w) for w in stand]
        nxt = torch.randn((sum(rows_of), hq, d), device=dev).to(dtype)
        l.q, l.ns, l.Ls = nxt, rows_of, lens
        l.cu, l.parents = cumulate(rows_of), trees(l.rng, rows_of, 1)
        # (the rows that stand are a chain now)
        l.check(*l.run())
        plain = l.run(tree_parents=None)
        l.check(*plain)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("kind,dtype", [("auto", BF), ("fp8", HF),
                                        ("fp4", BF)])
def test_a_speculative_step(cuda_device, kind, dtype, graph):
    step(cuda_device, kind, dtype, 3, [6, 1, 20, 9], [100, 7, 333, 0], 8, 2,
         128, 16, 3001, 2, graph)
