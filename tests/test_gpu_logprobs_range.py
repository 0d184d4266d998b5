"""token_logprobs over the whole range of its types: large common offsets, chunks and
rows of a type's lowest value (the usual mask), values near the largest.

The tolerances are those of test_gpu_logprobs.py: z - M is rounded once and everything
else depends on differences from the row's maximum only, so no bound grows with it."""
import numpy as np
import pytest
import torch

from test_gpu_logprobs import call

pytestmark = pytest.mark.gpu

OFFSETS = [100, 1e3, 1e4, 7e4, 1e6, 1e9, 1e20, 1e30]


def check(z, V, tokens, n, got):
    """As test_gpu_logprobs.check, with log sum e^(z - M) taken from z - M last: in 64 bits
    too M + log sum loses the sum beside a large M."""
    lp, ent, ids, tlp = got
    x = z[:, :V].double().numpy()
    d = x - x.max(1, keepdims=True)
    ref = d - np.log(np.exp(d).sum(1, keepdims=True))
    H = -(np.exp(ref) * ref).sum(1)
    order = np.argsort(-(x + 0.0), axis=1, kind="stable")[:, :n]
    assert np.array_equal(ids, order)
    pick = np.take_along_axis(ref, np.asarray(tokens)[:, None].astype(int), 1)[:, 0]
    for a, b in ((lp, pick), (tlp, np.take_along_axis(ref, order, 1))):
        off = np.abs(a - b) > 4e-6 + 2.0 ** -22 * np.abs(b)
        assert np.isfinite(a).all() and not off.any(), (np.argwhere(off)[:5], a[off][:5], b[off][:5])
    assert (np.abs(ent - H) <= 2e-5 * (1 + np.abs(H))).all(), np.nanmax(np.abs(ent - H))


def rows_of(dt, V, rng):
    """The rows of one test, most of them normal around an offset; each within its type's
    range, their log probabilities too."""
    lo = torch.finfo(dt).min
    normal = lambda: torch.from_numpy((3 * rng.standard_normal(V)).astype(np.float32))  # noqa: E731
    rows = []
    for off in OFFSETS:
        rows += [normal() + off, normal() - off]
        # as far apart in the type's own steps
        rows += [off * (1 + normal() / 300), -off * (1 + normal() / 300)]
    rows += [torch.full((V,), lo), torch.full((V,), -lo), torch.full((V,), -1e9)]
    high = torch.full((V,), 3e38)
    high[5:900] = 2.9e38
    rows += [high, high - 1e38]
    n = min(V, 2048)
    for at in range(0, V, n):          # one chunk masked, one chunk left
        a, b = normal(), torch.full((V,), lo)
        a[at:at + n] = lo
        b[at:at + n] = normal()[at:at + n]
        rows += [a, b] if n < V else [b]
    tail = normal() - 50               # a vocabulary padded to a round size, in the row's steps
    tail[V // 3:] = lo
    return torch.stack(rows + [tail]).to(dt)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("n", [0, 1, 20])
def test_offsets_and_masked_chunks(dt, many, n):
    rng = np.random.default_rng(n)
    for V in (1, 300, 2048 * 5 + 77):
        print(dt, many, n, V, flush=True)
        z = rows_of(dt, V, rng)
        if many:                       # enough rows for the kernel with a block a row
            z = z.repeat(-(-520 // len(z)), 1)
        k = min(n, V)
        tok = rng.integers(0, V, len(z))
        got = call(z, V, tok, k)
        check(z, V, tok, k, got)
        assert (got[0] <= 0).all() and (got[3] <= 0).all()


@pytest.mark.parametrize("many", [False, True])
def test_one_shift_for_all_changes_nothing(many):
    """Logits in steps of 1/4 shifted by whole numbers: the same differences exactly."""
    rng = np.random.default_rng(3)
    V, T = 5000, 520 if many else 7
    z = torch.from_numpy((rng.integers(-40, 40, (T, V)) / 4).astype(np.float32))
    tok = rng.integers(0, V, T)
    want = call(z, V, tok, 5)
    for off in (128.0, 4096.0, 2.0 ** 20, -2.0 ** 17):
        got = call(z + off, V, tok, 5)
        assert np.array_equal(got[2], want[2])
        for i, tol in ((0, 8e-6), (1, 4e-5), (3, 8e-6)):    # both within their bound
            a, b = got[i], want[i]
            assert (np.abs(a - b) <= tol * (1 + np.abs(b))).all(), (off, np.abs(a - b).max())


def test_infinity_beside_the_extremes():
    """+inf and NaN beside a type's lowest and largest values give NaN in their row alone."""
    for dt in (torch.float32, torch.bfloat16):
        for T in (4, 516):
            lo, V = torch.finfo(dt).min, 4500
            z = torch.randn((T, V)).to(dt)
            z[0, :2100] = lo
            z[1, :4096] = lo
            z[1, 4200] = float("inf")
            z[2, 2048:] = lo
            z[2, 9] = float("nan")
            tok = np.full(T, 7)
            lp, ent, ids, tlp = call(z, V, tok, 3)
            good = [0] + list(range(3, T))
            check(z[good], V, tok[good], 3, [a[good] for a in (lp, ent, ids, tlp)])
            assert np.isnan(lp[1:3]).all() and np.isnan(ent[1:3]).all() and np.isnan(tlp[1:3]).all()
            assert ids[1, 0] == 4200
