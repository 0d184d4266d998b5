"""attn_shared_prefix at values that stand out: V scales of an E4M3 cache that differ by powers
of two, NaN in queries and keys, positions up to the largest.  Shapes for the blocks of 16 and
32 rows and for those over key tiles in LDS.  Tolerances: test_gpu_attn.check, whose bound is
2^-8 of each weight, whatever the scales beside it."""
import numpy as np
import pytest
import torch

import ops_ref as ref
from test_gpu_attn import build, call, check, positions

pytestmark = pytest.mark.gpu

import bit_expert_ffn_moe_amd as moe  # noqa: E402

SHAPES = [  # B, Q, Hq, Hkv, D, page, P, own
    (3, 3, 4, 2, 64, 32, 45, [9, 40, 64]),               # blocks of 16 rows
    (2, 4, 8, 1, 128, 64, 700, [9, 90]),
    (20, 2, 8, 2, 128, 16, 333, list(range(2, 22))),     # shared keys: key tiles, two blocks
    (12, 2, 8, 2, 128, 32, 140, [2 + 9 * i for i in range(12)]),   # blocks of 32 rows
    (2, 140, 2, 1, 64, 16, 70, [140, 200]),              # both by key tiles
    (1, 150, 2, 2, 256, 64, 130, [333]),
]


def make(shape, fp8, seed=0):
    B, Q, Hq, Hkv, D, page, P, own = shape
    rng = np.random.default_rng(seed)
    kv, q, pre, table, n = build(rng, B, Q, Hq, Hkv, D, page, P, own, fp8)
    return rng, kv, q, pre, table, n, positions(own, P, Q)


def place(shape, pre, table, b, j):
    page, P = shape[5], shape[6]
    return int(pre[j // page] if j < P else table[b, j // page]), j % page


def run(shape, kv, q, pos, pre, table, n):
    Q, P, scale = shape[1], shape[6], shape[4] ** -0.5
    o, lse = call(kv, q, pos, pre, P, table, n, scale, Q)
    check(o, lse, q, kv, pos, pre, P, table, scale, Q, n)


# ---- V scales

@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("power", [16, 30, 100, -16, -60])
def test_v_scale_of_a_key_some_rows_do_not_see(shape, power):
    """The last token's key of every sequence: rows before it must not notice."""
    rng, kv, q, pre, table, n, pos = make(shape, True)
    print(shape, power, flush=True)
    for b in range(shape[0]):
        pg, s = place(shape, pre, table, b, shape[6] + shape[7][b] - 1)
        kv.t["vs"][pg, :, s] *= 2.0 ** power
    run(shape, kv, q, pos, pre, table, n)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("nats,power", [(64, 16), (64, 30), (14, 16), (14, 30), (300, 100), (0, 24),
                                        (-20, -30), (-20, -14)])
def test_v_scale_of_a_key_with_little_or_most_of_the_weight(shape, nats, power):
    """One shared key whose score lies `nats` below (or above) the others' and whose V scale
    is 2^power times theirs, in the first, a middle or the last key tile."""
    print(shape, nats, power, flush=True)
    for at in (0.0, 0.5, 1.0):
        rng, kv, q, pre, table, n, pos = make(shape, True)
        pg, s = place(shape, pre, table, 0, int(at * (shape[6] - 1)))
        q[:, :, 0] = 8.0
        if nats:
            kv.t["k"][pg, :, s] = 0
            kv.t["k"][pg, :, s, 0] = 0xFE if nats > 0 else 0x7E          # -+448
            kv.t["ks"][pg, :, s] = abs(nats) / (448 * 8 * shape[4] ** -0.5)
        kv.t["vs"][pg, :, s] *= 2.0 ** power
        run(shape, kv, q, pos, pre, table, n)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("spread", [8, 40])
def test_v_scales_all_different(shape, spread):
    rng, kv, q, pre, table, n, pos = make(shape, True)
    kv.t["vs"] *= torch.from_numpy(
        np.exp2(rng.uniform(-spread, spread, kv.t["vs"].shape)).astype(np.float32))
    run(shape, kv, q, pos, pre, table, n)


# ---- NaN

@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fp8", [False, True])
def test_nan_queries_show(shape, fp8):
    """A NaN in a query makes its own row NaN, out and lse, and no other; a padding row's
    query may hold anything."""
    B, Q, Hq, Hkv, D, page, P, own = shape
    print(shape, fp8, flush=True)
    rng, kv, q, pre, table, n, pos = make(shape, fp8)
    pos[3] = -1
    want = ref.attention(q.double().numpy(), kv, pos, pre, P, table, 0.125, Q, n)
    hit = np.zeros((B * Q, Hq), bool)
    for t, h in ((1, 0), (3, 1), (B * Q - 1, Hq - 1)):
        q[t, h, D // 2] = float("nan")
        hit[t, h] = t != 3
    o, lse = call(kv, q, pos, pre, P, table, n, 0.125, Q)
    assert np.isnan(o[hit]).all() and np.isnan(lse[hit]).all()
    assert (o[3] == 0).all() and (lse[3] == -np.inf).all()
    compare(o, lse, q, want, ~hit & (pos >= 0)[:, None])


def compare(o, lse, q, want, rows):
    """test_gpu_attn.check for some (token, head) rows, against values formed before."""
    eo, el, mag, qk = (a[rows] for a in want)
    d = 2 * q.shape[2] * 2.0 ** -23 * qk
    tol = 1.05 * 2.0 ** -8 * (mag + np.abs(eo)) + (2 * d[..., None] + 2.0 ** -16) * mag
    assert (np.abs(o[rows] - eo) <= tol).all()
    assert (np.abs(lse[rows] - el) <= d + 2.0 ** -20 * (1 + np.abs(el))).all()


ONLY = [  # the key spoilt is the only one of its own that the sequence's rows see, or one of many
    (2, 1, 4, 2, 64, 16, 40, [1, 30]),
    (1, 1, 2, 1, 128, 16, 0, [1]),
    (40, 1, 4, 1, 128, 16, 200, [1 + i % 3 for i in range(40)]),
    (30, 1, 4, 1, 128, 64, 0, [1 + i % 3 for i in range(30)]),
]


@pytest.mark.parametrize("shape", ONLY + SHAPES)
@pytest.mark.parametrize("fp8", [False, True])
def test_nan_keys_show(shape, fp8):
    """A NaN in K at the first own key of sequence 0: every row that sees it is NaN, out and
    lse, the others as before; the same at a shared key."""
    B, Q, Hq, Hkv, D, page, P, own = shape
    print(shape, fp8, flush=True)
    rng, kv, q, pre, table, n, pos = make(shape, fp8)
    if Q > 1:
        pos[1] = P // 2 if P else 0        # a row that ends before
    want = ref.attention(q.double().numpy(), kv, pos, pre, P, table, 0.125, Q, n)
    seq = np.arange(B * Q) // Q
    for j, who in ((P, seq == 0), (2 * P // 3 + 1, True)):
        if j > P or not P and who is True:
            continue
        pg, s = place(shape, pre, table, 0, j)
        name = "ks" if fp8 else "k"
        kept = kv.t[name][pg, :, s].clone()
        kv.t[name][pg, :, s] = float("nan")
        hit = who & (pos >= j)
        o, lse = call(kv, q, pos, pre, P, table, n, 0.125, Q)
        assert hit.any() and np.isnan(o[hit]).all() and np.isnan(lse[hit]).all()
        compare(o, lse, q, want, np.repeat(~hit[:, None], Hq, 1))
        kv.t[name][pg, :, s] = kept


# ---- positions

@pytest.mark.parametrize("shape", SHAPES)
def test_the_largest_position(shape):
    """A position past max_keys, up to the type's last, sees the keys below max_keys."""
    B, Q, Hq, Hkv, D, page, P, own = shape
    rng, kv, q, pre, table, n, pos = make(shape, False)
    b = int(np.argmax(own))                # the sequence that has all n keys
    pos[b * Q + Q - 1] = n - 1
    want = call(kv, q, pos, pre, P, table, n, 0.1, Q)
    check(*want, q, kv, pos, pre, P, table, 0.1, Q, n)
    for p in (n, 2 ** 31 - 1):
        pos[b * Q + Q - 1] = p
        got = call(kv, q, pos, pre, P, table, n, 0.1, Q, expect_status=moe.MOE_STATUS_BAD_PAGE)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]), p


# ---- V scales of 0

@pytest.mark.parametrize("shape", SHAPES)
def test_v_scales_of_zero(shape):
    """Rows of zeros in V, as appended: a key of most of the weight, every shared key, all."""
    print(shape, flush=True)
    for nats in (20, 40, 60):
        rng, kv, q, pre, table, n, pos = make(shape, True)
        q[:, :, 0] = 8.0
        pg, s = place(shape, pre, table, 0, shape[6] // 2)
        kv.t["k"][pg, :, s] = 0
        kv.t["k"][pg, :, s, 0] = 0x7E
        kv.t["ks"][pg, :, s] = nats / (448 * 8 * shape[4] ** -0.5)
        kv.t["v"][pg, :, s], kv.t["vs"][pg, :, s] = 0, 0.0
        run(shape, kv, q, pos, pre, table, n)
    for pages in (torch.from_numpy(np.asarray(pre)), slice(None)):
        kv.t["v"][pages], kv.t["vs"][pages] = 0, 0.0
        run(shape, kv, q, pos, pre, table, n)
