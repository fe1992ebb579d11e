"""Attention of drafted trees where the value rows at which a kernel can go
wrong (the draft's own, those beside tiles, pages and windows) are 64 times the
others, against the float64 reference and within a tolerance that such a row
would break were it lost or misplaced (test_tree_tolerance.py)."""
import numpy as np
import pytest
import torch

from _tree_util import borders, reference
from paged_kv_cache_318_gb300 import api
from test_gpu_tree import BF, E2M1, HF, VS, Draft, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built(cuda_device):
    from paged_kv_cache_318_gb300 import _build
    _build.build()
    api.load_library()
    api.check_device_errors(cuda_device)
    yield
    api.check_device_errors(cuda_device)


class Loud(Draft):
    def __init__(self, dev, ns, Ls, *args, window=-1, **kw):
        super().__init__(dev, ns, Ls, *args, **kw)
        self.q /= 4           # (no key's weight is far below the others')
        self.window = window
        at = [(self.table[b][j // self.bs], j % self.bs)
              for b, L in enumerate(Ls)
              for j in borders(self.parents[b], L - ns[b], L, window)]
        blk, off = (np.array(x) for x in zip(*at))
        v, vals = self.caches[1], self.vals[1]
        rng = np.random.default_rng(9)
        where = tuple(torch.from_numpy(x).to(dev) for x in (blk, off))
        if self.kind == "auto":
            new = torch.from_numpy(rng.standard_normal(
                (len(at), self.hkv, self.d)) * 64).to(dev, v.dtype)
            v[where] = new
            vals[blk, off] = f64(new)
        elif self.kind == "fp8":
            # (the others go down: codes end at 448)
            c = v.float() / 32
            c[where] = torch.from_numpy(np.clip(rng.standard_normal(
                (len(at), self.hkv, self.d)) * 160, -448, 448)).to(
                    dev, torch.float32)
            c = c.to(v.dtype)
            v.view(torch.uint8).copy_(c.view(torch.uint8))
            vals[:] = np.nan_to_num(f64(c.float())) * VS
        else:
            sf = self.kw["v_block_scale"]
            new = torch.from_numpy(rng.uniform(256, 448, (
                len(at), self.hkv, self.d // 16))).to(dev).float().to(sf.dtype)
            sf.view(torch.uint8)[where] = new.view(torch.uint8)
            c = v[where].cpu().numpy()
            code = np.stack([E2M1[c & 15], E2M1[c >> 4]], -1)
            vals[blk, off] = code.reshape(vals[blk, off].shape) * \
                np.repeat(f64(new.float()), 16, -1) * VS

    def hold(self, out, lse, softcap=0.0, sinks=None):
        out, lse = f64(out), f64(lse)
        eps = torch.finfo(self.dtype).eps
        for b, n in enumerate(self.ns):
            if n == 0:
                continue
            at = slice(self.cu[b], self.cu[b + 1])
            o, l, tol, ltol = reference(
                f64(self.q[at]), *self.rows(b), self.parents[b], eps,
                self.d ** -0.5, softcap, self.window,
                None if sinks is None else f64(sinks))
            off = np.abs(out[at] - o)
            assert np.isfinite(out[at]).all()
            assert (off <= tol).all(), (b, (off / tol).max())
            dead = np.isneginf(l)
            assert (np.isneginf(lse[:, at]) == dead).all()
            assert (np.abs(lse[:, at] - l)[~dead] <= ltol[~dead]).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", ["auto", "fp8", "fp4"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_rows(cuda_device, d, kind, dtype):
    """Up to 128 packed rows, more, and more than a block's, cut into pieces
    and not."""
    t = Loud(cuda_device, [20, 50, 7, 80], [620, 1350, 40, 333], 8, 2, d, 16,
             dtype, kind)
    for splits in (0, 1):
        t.hold(*t.run(num_splits=splits))


@pytest.mark.parametrize("kind", ["auto", "fp8", "fp4"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 3, 130, 1000])
def test_large_rows_beside_a_window(cuda_device, window, d, kind):
    t = Loud(cuda_device, [12, 45, 3], [812, 700, 1200], 8, 2, d, 32, BF,
             kind, window=window)
    for splits in (0, 1):
        t.hold(*t.run(window_size=(window, -1), num_splits=splits))


@pytest.mark.parametrize("kind", ["auto", "fp8", "fp4"])
@pytest.mark.parametrize("layout", ["hnd", "gaps"])
@pytest.mark.parametrize("bs", [16, 48, 128])
def test_large_rows_of_layouts(cuda_device, bs, layout, kind):
    t = Loud(cuda_device, [9, 70], [500, 401], 6, 2, 128, bs, HF, kind, layout)
    sinks = torch.linspace(-2, 4, 6, device=cuda_device)
    t.hold(*t.run(softcap=20.0, s_aux=sinks), softcap=20.0, sinks=sinks)


@pytest.mark.parametrize("kind", ["auto", "fp8", "fp4"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_rows_of_a_long_context(cuda_device, d, kind):
    """One request: every block's share is a piece of it."""
    t = Loud(cuda_device, [11], [6011], 4, 1, d, 16, BF, kind)
    t.hold(*t.run())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("softcap", [0.5, 50.0, 1000.0, 4096.0])
def test_soft_caps(cuda_device, softcap, d):
    """Small logits, and some of up to a hundred."""
    t = Loud(cuda_device, [12, 45], [300, 500], 8, 2, d, 16, HF)
    t.hold(*t.run(softcap=softcap), softcap=softcap)
    t = Draft(cuda_device, [12, 45], [300, 500], 8, 2, d, 16, HF, spread=8.0)
    t.window = -1
    Loud.hold(t, *t.run(softcap=softcap), softcap=softcap)
