"""Attention over the paged cache where keys weigh nothing: scores of minus
infinity beside finite ones, pages of very different size, and pages that no
row sees, in both kernels and with units cut between CTAs and whole."""
import math

import numpy as np
import pytest
import torch

import block_scaled_quantized_mx_gb300 as mx
from tests import _kv

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
TOP = {mx.E4M3: 448.0, mx.E5M2: 57344.0, mx.INT8: 128.0}


@pytest.fixture(scope="module", autouse=True)
def _built():
    mx.build()
    mx.lib()


class One:
    """One request of n keys in pages of `page` in a shuffled pool, one cache
    head, `rows` new tokens and two query heads.  key and value: K and V as n x d
    arrays; the planes may be changed afterwards."""

    def __init__(self, n, rows, page, key, value, q, fmt=mx.E4M3, seed=0):
        g = torch.Generator().manual_seed(seed)
        pages, d = -(-n // page), key.shape[1]
        ids = torch.randperm(pages + 2, generator=g)[:pages]
        self.n, self.rows, self.page, self.fmt, self.d, self.ids = n, rows, page, fmt, d, ids.numpy()
        self.cache = mx.empty_kv_cache(fmt, pages + 2, 1, page, d)
        for t in (self.cache.k, self.cache.v, self.cache.k_scales, self.cache.v_scales):
            t.zero_()
        j = torch.arange(n)
        slots = ids[j // page] * page + j % page
        mx.mx_kv_append(self.cache, key.to(BF).cuda().view(n, 1, d), value.to(BF).cuda().view(n, 1, d),
                        slots.cuda())
        self.table = ids.to(torch.int32).view(1, -1).cuda()
        self.q = q.to(BF).cuda().view(rows, 2, d)

    def run(self, window=0, ws=True, causal=True):
        i32 = dict(dtype=torch.int32, device="cuda")
        w = None
        if ws:
            w = torch.randint(0, 256, (mx.kv_attention_workspace_bytes(2, 1, self.d, self.rows),),
                              dtype=torch.uint8, device="cuda")
        r = mx.mx_kv_attention(self.q, self.cache, self.table, torch.tensor([self.n], **i32),
                               torch.tensor([0, self.rows], **i32), self.rows, causal=causal,
                               window=window, out_dtype=F32, workspace=w)
        torch.cuda.synchronize()
        assert mx.mx_last_error() == 0
        return r.double().cpu().numpy()

    def exact(self, window=0, skip=()):
        """64-bit outputs, and how far an fp32 output of the kernels may be
        from them.  A weight's product with its page's scale is rounded to f16:
        2^-11 relative, or half of f16's smallest step, 2^-25, in a unit in
        which the row's largest such product is 2^3 at least (it is brought to
        2^7, less the rounding of that power and three bits for pages that are
        taken as one); an error e of the scores, of d products and their
        scaling in fp32, changes a weight by 2 e relative; the sums of the
        weights and of O add 2^-23 for each step of 16 keys and for the joining.
        Keys in `skip` have no weight."""
        def of_keys(plane, scales):
            s = 2.0 ** (scales.cpu().numpy()[self.ids, 0].astype(float) - 127)
            x = _kv.TABLES[self.fmt][plane.cpu().numpy()[self.ids, 0]]
            return x.reshape(-1, self.d)[:self.n], np.repeat(s, self.page)[:self.n]

        k, ks = of_keys(self.cache.k, self.cache.k_scales)
        codes, vs = of_keys(self.cache.v, self.cache.v_scales)
        k = k * ks[:, None]
        q = self.q.double().cpu().numpy()
        out, tol = np.zeros((self.rows, 2, self.d)), np.zeros((self.rows, 2, self.d))
        j = np.arange(self.n)
        for i in range(self.rows):
            p = self.n - self.rows + i
            see = (j <= p) & (j > p - window if window else True) & ~np.isin(j, skip)
            for h in range(2):
                x = (k[see] @ q[i, h]) * self.d ** -0.5
                w = np.exp(x - x.max())
                w /= w.sum()
                ws = w * vs[see]
                out[i, h] = ws @ codes[see]
                ab = self.d ** -0.5 * ((self.d + 4.5) * (np.abs(k[see]) @ np.abs(q[i, h])).max() +
                                       0.5 * np.abs(q[i, h]).max() * np.abs(k[see]).sum(1).max()) * 2.0 ** -24
                rel = 2.0 ** -11 + 2 * ab + (see.sum() / 16 + 64) * 2.0 ** -23
                tol[i, h] = (ws @ np.abs(codes[see])) * rel + see.sum() * ws.max() * TOP[self.fmt] * 2.0 ** -28 + \
                    np.abs(out[i, h]) * 2.0 ** -24
        return out, tol


def _noise(n, d, seed=1):
    return torch.randn(n, d, generator=torch.Generator().manual_seed(seed)).clamp(-4, 4)


# (keys, rows): one tile of the kernel for few rows, several of its CTAs, the
# kernel for many rows in one unit and in one cut over all SMs
FEW, MANY = [(250, 1), (6000, 3)], [(300, 40), (9000, 70)]


@pytest.mark.parametrize("n,rows", FEW + MANY)
@pytest.mark.parametrize("ws", [True, False])
@pytest.mark.parametrize("page,d", [(16, 64), (64, 64), (32, 128)])
def test_keys_of_minus_infinity_beside_others(n, rows, ws, page, d):
    """Scores that overflow to -infinity weigh nothing where the row has
    finite ones, whoever else they share a warp, a segment or a part with."""
    far = np.arange(0, n // 2 // page * page)             # whole pages
    far = far[(far // page) % 7 != 3] if n > 1000 else far
    key = _noise(n, d) * 0.1
    key[far] = -4.0
    q = torch.ones(rows * 2, d) + 0.1 * _noise(rows * 2, d, seed=3)
    s = One(n, rows, page, key, _noise(n, d, seed=2), q)
    s.cache.k_scales[torch.from_numpy(s.ids[np.unique(far // page)])] = 254      # -2^135 and below: -infinity
    out, tol = s.exact(skip=far)
    got = s.run(ws=ws)
    assert (np.abs(got - out) <= tol).all()
    # a row that has no finite score at all is NaN still, and alone in it
    s.q[0, 1] = 0
    s.q[0, 1, 5] = 1
    s.cache.k.view(-1, d)[:, 5] = 0xFE                    # -448
    s.cache.k_scales.fill_(254)
    got = s.run(ws=ws)
    assert np.isnan(got[0, 1]).all()


@pytest.mark.parametrize("n,rows", FEW + MANY)
@pytest.mark.parametrize("ws", [True, False])
@pytest.mark.parametrize("page,d", [(16, 64), (64, 64), (16, 128), (32, 128)])
@pytest.mark.parametrize("fmt", [mx.E4M3, mx.INT8])
def test_large_values_of_no_weight(n, rows, ws, page, d, fmt):
    """Values of 2^33 in every third page, with weights of e^-40: what the
    other pages give has to survive beside them."""
    far = (np.arange(n) // page) % 3 == 1
    key, value = _noise(n, d) * 0.05 + 2.5, _noise(n, d, seed=2)
    key[far] -= 5.0 if d == 64 else 5.0 * 2 ** -0.5
    value[far] *= 2.0 ** 33
    s = One(n, rows, page, key, value, torch.ones(rows * 2, d), fmt=fmt)
    out, tol = s.exact()
    assert (np.abs(out) > 4 * tol).mean() > 0.5            # the bound can tell them from zero
    assert (np.abs(s.run(ws=ws) - out) <= tol).all()


@pytest.mark.parametrize("n,rows", [(259, 5), (6003, 5), (300, 40), (9000, 70)])
@pytest.mark.parametrize("ws", [True, False])
@pytest.mark.parametrize("up", [12, 40, 90])
@pytest.mark.parametrize("d", [64, 128])
def test_large_values_that_a_row_does_not_see(n, rows, ws, up, d):
    """The last page's values are 2^up times the others': rows in front of it
    do not know it.  The same in front of a window that begins inside a page
    and behind whole ones."""
    page = 16
    s = One(n, rows, page, _noise(n, d), _noise(n, d, seed=2), _noise(rows * 2, d, seed=3))
    s.cache.v_scales[int(s.ids[-1])] += up
    out, tol = s.exact()
    before = n - rows + np.arange(rows) < (n - 1) // page * page
    assert before.any() and not before.all()
    got = s.run(ws=ws)
    assert (np.abs(got - out) <= tol).all()
    s.cache.v_scales[int(s.ids[-1])] -= up
    window = 50
    first = n - rows + 1 - window
    s.cache.v_scales[torch.from_numpy(s.ids[:first // page])] += up
    out, tol = s.exact(window=window)
    assert (np.abs(s.run(window=window, ws=ws) - out) <= tol).all()


@pytest.mark.parametrize("n,rows,window", [(250, 1, 100), (6000, 3, 990), (300, 40, 70), (9000, 70, 100)])
@pytest.mark.parametrize("ws", [True, False])
@pytest.mark.parametrize("fmt,d", [(mx.E4M3, 64), (mx.E5M2, 64), (mx.E4M3, 128)])
def test_pages_in_front_of_the_window_are_not_followed(n, rows, window, ws, fmt, d):
    """Pages that no row sees may belong to another request by now, whatever
    the table still says: NaN codes and any scale in them change no bit."""
    page = 16
    s = One(n, rows, page, _noise(n, d), _noise(n, d, seed=2), _noise(rows * 2, d, seed=3), fmt=fmt)
    want = s.run(window=window, ws=ws)
    out, tol = s.exact(window=window)
    assert (np.abs(want - out) <= tol).all()
    gone = torch.from_numpy(s.ids[:(n - rows + 1 - window) // page])
    for code, scale in ((0x7F, 254), (0x7F, 255), (0x00, 254)):
        s.cache.k[gone] = s.cache.v[gone] = code
        s.cache.k_scales[gone] = s.cache.v_scales[gone] = scale
        assert np.array_equal(s.run(window=window, ws=ws), want)
