"""token_logprobs against 64-bit log-softmax.

Tolerance: a row's weight is summed in fp32 through at most 32 + 6 + V / 2^19 + 12
adds of positive terms, each exponential within 2^-22 (1 + |z - M| 2^-2) of its
value where it weighs anything: log l within 60 x 2^-24 = 4e-6; z - M is rounded
once.  The entropy's second sum has terms of up to (1 + |z - M|) times that."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_expert_ffn_moe_amd as moe  # noqa: E402

DEV = "cuda:0"


def call(z, V, tokens, n, entropy=True, status=0):
    """z [T][stride] on the CPU, the first V columns the row."""
    T, stride = z.shape
    zd = z.to(DEV)
    dt = moe.MOE_DT_BF16 if z.dtype == torch.bfloat16 else moe.MOE_DT_F32
    nb = moe.token_logprobs_workspace_bytes(T, V, n)
    assert nb > 0
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device=DEV)
    lp = torch.full((T,), 7.0, device=DEV)
    ent = torch.full((T,), 7.0, device=DEV)
    ids = torch.full((T, n), -7, dtype=torch.int32, device=DEV)
    tlp = torch.full((T, n), 7.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    tok = torch.as_tensor(tokens, dtype=torch.int32).to(DEV) if tokens is not None else None
    moe.token_logprobs(zd, dt, stride, T, V, tok, n, lp if tok is not None else None,
                       ent if entropy else None, ids if n else None, tlp if n else None, st, ws, nb)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    return [a.cpu().numpy() for a in (lp, ent, ids, tlp)]


def check(z, V, tokens, n, got):
    lp, ent, ids, tlp = got
    x = z[:, :V].double().numpy()
    with np.errstate(all="ignore"):
        M = x.max(1, keepdims=True)
        e = np.exp(x - M)
        lse = M + np.log(e.sum(1, keepdims=True))
        ref = x - lse
        p = np.exp(ref)
        H = -np.sum(np.where(p > 0, p * ref, 0), 1)
    order = np.argsort(-(x + 0.0), axis=1, kind="stable")[:, :n]
    assert np.array_equal(ids, order)
    tol = lambda r: 4e-6 + 2.0 ** -22 * np.abs(np.where(np.isfinite(r), r, 0))  # noqa: E731
    pick = np.take_along_axis(ref, np.asarray(tokens)[:, None].astype(int), 1)[:, 0]
    for a, b in ((lp, pick), (tlp, np.take_along_axis(ref, order, 1))):
        assert np.array_equal(np.isfinite(a), np.isfinite(b))
        f = np.isfinite(b)
        assert (np.abs(a - b)[f] <= tol(b)[f]).all(), np.abs(a - b)[f].max()
        assert (a[~f] == b[~f]).all()
    assert (np.abs(ent - H) <= 2e-5 * (1 + np.abs(H))).all(), np.abs(ent - H).max()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [0, 1, 5, 20, 64])
def test_matches_64_bit_log_softmax(dt, n):
    rng = np.random.default_rng(n)
    for T, V, pad in [(1, max(n, 1), 0), (3, 64 + n, 1), (2, 2047, 0), (5, 2049, 3), (2, 8192, 0),
                      (3, 50021, 0), (1, 131072, 5), (70, 1001, 0), (1, 600001, 0)]:
        print(dt, n, T, V, flush=True)
        z = torch.from_numpy((3 * rng.standard_normal((T, V + pad))).astype(np.float32)).to(dt)
        z[:, V:] = 1e30            # past the row: not read
        tok = rng.integers(0, V, T)
        tok[0] = V - 1
        check(z, V, tok, n, call(z, V, tok, n))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [0, 1, 7, 64])
def test_many_rows(dt, n):
    """Enough rows for the kernel that walks a row with one block: random rows, rows
    of few values (ties), sorted ones both ways, masked ones."""
    rng = np.random.default_rng(n)
    T = 600
    for V in (70, 2049, 9001, 20000):
        print(dt, n, V, flush=True)
        z = torch.from_numpy((3 * rng.standard_normal((T, V + 1))).astype(np.float32)).to(dt)
        z[5] = torch.round(z[5])
        z[6] = z[6].sort().values
        z[7] = z[7].sort(descending=True).values
        z[8, 40:] = -float("inf")
        z[9] = 1.5
        z[10, ::3] = -float("inf")
        z[:, V:] = 1e30
        tok = rng.integers(0, 40, T)
        check(z, V, tok, min(n, 40), call(z, V, tok, min(n, 40)))
        k = min(n, V)
        check(z[:8], V, tok[:8], k, [a[:8] for a in call(z, V, tok, k)])


def test_nan_rows_among_many():
    T, V, n = 520, 6000, 5
    z = torch.randn((T, V))
    z[3, 100] = float("nan")
    z[4, 5000] = float("inf")
    z[5] = float("nan")
    z[5, [70, 3000]] = torch.tensor([1.0, 2.0])
    tok = np.full(T, 7)
    lp, ent, ids, tlp = call(z, V, tok, n)
    ok = [i for i in range(T) if i not in (3, 4, 5)]
    check(z[ok], V, tok[ok], n, [a[ok] for a in (lp, ent, ids, tlp)])
    x = np.where(np.isnan(z.numpy()), -np.inf, z.numpy())
    for r in (3, 4):
        assert np.isnan(lp[r]) and np.isnan(ent[r])
        assert np.array_equal(ids[r], np.argsort(-x[r], kind="stable")[:n])
    assert np.array_equal(ids[5], [3000, 70, 0, 1, 2])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_ties_go_to_the_lowest_id(dt):
    rng = np.random.default_rng(1)
    for V in (100, 2048, 5000, 20000):
        z = torch.from_numpy(rng.integers(0, 3, (4, V)).astype(np.float32)).to(dt)
        z[1] = 2.0                 # all equal
        z[2] = torch.where(z[2] == 0, -0.0, 0.0)   # signed zeros are one value
        z[3, :] = 0.0
        z[3, V - 40:] = 1.0        # the best in one lane's reach
        tok = np.array([0, 1, 2, 3])
        check(z, V, tok, 64, call(z, V, tok, 64))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_one_lane_holds_all_the_best(dt):
    """The n best in the 32 elements of one lane, rising and falling."""
    V = 6000
    VE = 4 if dt == torch.float32 else 8
    z = torch.randn((2, V)).to(dt) * 0.1
    at = [2048 + (v * 64 + 9) * VE + i for v in range(32 // VE) for i in range(VE)]
    z[0, at] = torch.arange(32).to(dt) + 10
    z[1, at] = 50 - torch.arange(32).to(dt)
    check(z, V, np.array([0, 1]), 40, call(z, V, np.array([0, 1]), 40))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_infinities(dt):
    """-inf has probability 0; a row of -inf; few finite logits; one of the
    type's lowest value; +inf and NaN spoil their row alone."""
    V, n = 4100, 10
    inf = float("inf")
    z = torch.full((7, V), -inf).to(dt)
    z[0, 17] = 1.0
    z[1, [5, 4000, 4099]] = torch.tensor([1.0, 2.0, 2.0]).to(dt)
    z[2] = torch.randn(V).to(dt)
    z[2, ::2] = torch.finfo(dt).min
    z[4] = torch.randn(V).to(dt)
    z[4, 100] = inf
    z[5] = torch.randn(V).to(dt)
    z[5, 3000] = float("nan")
    z[6] = torch.randn(V).to(dt)
    tok = np.array([17, 6, 4, 9, 100, 7, 8])
    lp, ent, ids, tlp = call(z, V, tok, n)
    good = [0, 1, 2, 6]
    sub = lambda a: a[good]  # noqa: E731
    check(z[good], V, tok[good], n, [sub(a) for a in (lp, ent, ids, tlp)])
    # the empty row
    assert lp[3] == -inf and ent[3] == 0 and (tlp[3] == -inf).all()
    assert np.array_equal(ids[3], np.arange(n))
    for r in (4, 5):
        assert np.isnan(lp[r]) and np.isnan(ent[r])
    assert ids[4, 0] == 100
    x = z[5].double().numpy()
    assert np.array_equal(ids[5], np.argsort(np.where(np.isnan(x), inf, -x), kind="stable")[:n])
    assert np.isnan(tlp[5]).all()


def test_nan_ranks_last():
    V = 50
    z = torch.full((2, V + 3), float("nan"))
    z[0, [3, 40]] = torch.tensor([-float("inf"), 2.0])
    ids = call(z, V, np.array([0, 0]), V)[2]
    rest = [i for i in range(V) if i not in (3, 40)]
    assert np.array_equal(ids[0], [40, 3] + rest)
    assert np.array_equal(ids[1], np.arange(V))


def test_tokens_outside_the_vocabulary_and_optional_outputs():
    z = torch.randn((4, 300))
    full = call(z, 300, np.array([0, 5, 299, 7]), 2)
    got = call(z, 300, np.array([-1, 5, 300, 7]), 2, status=moe.MOE_STATUS_BAD_TOKEN)
    assert got[0][0] == 0 and got[0][2] == 0
    assert np.array_equal(got[0][[1, 3]], full[0][[1, 3]])
    assert call(z, 300, np.array([-1, -2, 3, 4]), 0)[0][0] == 0
    lp, ent, ids, tlp = call(z, 300, None, 2, entropy=False)
    assert (lp == 7).all() and (ent == 7).all() and np.array_equal(ids, full[2])


def test_large_rows_and_offsets():
    """Rows past 4 GiB from the first."""
    V, stride, T = 1000, (1 << 29) + 8, 3
    z = torch.zeros(T * stride, dtype=torch.float32, device=DEV)
    for t in range(T):
        z[t * stride:t * stride + V] = torch.randn(V, device=DEV)
    nb = moe.token_logprobs_workspace_bytes(T, V, 3)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    lp, ent = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    ids = torch.empty((T, 3), dtype=torch.int32, device=DEV)
    tlp = torch.empty((T, 3), device=DEV)
    tok = torch.tensor([1, 2, 3], dtype=torch.int32, device=DEV)
    moe.token_logprobs(z, moe.MOE_DT_F32, stride, T, V, tok, 3, lp, ent, ids, tlp, None, ws, nb)
    rows = torch.stack([z[t * stride:t * stride + V] for t in range(T)]).cpu()
    check(rows, V, np.array([1, 2, 3]), 3, [a.cpu().numpy() for a in (lp, ent, ids, tlp)])
