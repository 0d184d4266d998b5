"""attn_shared_prefix at the shapes that its kernels with many rows take: blocks of 256 (128 at
256 columns) rows over key tiles in LDS, for the shared keys and for a sequence's own, and
blocks of 32 rows at 64 and 128 columns; several key tiles and parts, more than one block of
rows, every page size.  Tolerances: test_gpu_attn.check."""
import numpy as np
import pytest
import torch

import ops_ref as ref
from test_gpu_attn import build, call, check, positions

pytestmark = pytest.mark.gpu

import bit_expert_ffn_moe_amd as moe  # noqa: E402

SHAPES = [  # B, Q, Hq, Hkv, D, page, P, own
    # shared keys by many rows (B Q G > 128), own keys by few
    (5, 7, 16, 2, 128, 16, 300, [7, 64, 150, 33, 90]),        # 280 rows: two blocks; 56 own
    (40, 1, 8, 2, 128, 64, 777, list(range(1, 41))),          # 160 rows, a third of a block
    (9, 4, 8, 1, 64, 512, 2100, [4, 700, 65, 30, 12, 5, 128, 129, 64]),
    (3, 11, 12, 2, 256, 32, 260, [11, 70, 200]),              # 198 rows at 256 columns
    (70, 2, 1, 1, 256, 256, 129, [2 + i % 9 for i in range(70)]),
    # a sequence's own keys by many rows (Q G > 128)
    (2, 150, 2, 2, 64, 16, 0, [150, 411]),                    # no prefix
    (2, 70, 8, 2, 128, 256, 77, [70, 300]),                   # 280 rows: two blocks, prefix ends in a page
    (1, 140, 1, 1, 256, 512, 130, [333]),                     # one sequence, both by many rows
    (2, 131, 1, 1, 128, 128, 40, [131, 1500]),
    # blocks of 32 rows: the shared keys', the own, both
    (20, 1, 8, 2, 128, 64, 333, list(range(1, 21))),
    (24, 1, 4, 1, 128, 32, 1500, [1 + 13 * i for i in range(24)]),
    (2, 20, 4, 1, 128, 16, 100, [20, 190]),                   # 160 shared, 80 own
    (1, 20, 4, 1, 128, 16, 300, [200]),                       # 80 and 80
    (3, 20, 4, 1, 64, 64, 0, [20, 190, 64]),
    (1, 20, 4, 1, 256, 64, 70, [140]),                        # 16-row blocks at 256 columns
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_64_bit_attention(shape, fp8):
    B, Q, Hq, Hkv, D, page, P, own = shape
    print(shape, fp8, flush=True)
    rng = np.random.default_rng(B * 1000 + P)
    kv, q, pre, table, n = build(rng, B, Q, Hq, Hkv, D, page, P, own, fp8)
    pos = positions(own, P, Q)
    scale = D ** -0.5
    o, lse = call(kv, q, pos, pre, P, table, n, scale, Q, extra=8)
    check(o, lse, q, kv, pos, pre, P, table, scale, Q, n)


@pytest.mark.parametrize("fp8", [False, True])
def test_only_the_shared_keys(fp8):
    """max_keys = prefix_len: no key of a sequence's own, no page table."""
    rng = np.random.default_rng(1)
    for B, G, D in ((40, 4, 128), (24, 4, 128), (3, 2, 64)):
        P = 200
        kv, q, pre, table, _ = build(rng, B, 1, G, 1, D, 32, P, [1] * B, fp8)
        pos = rng.integers(0, P, B)
        pos[1] = -1
        o, lse = call(kv, q, pos, pre, P, table, P, 0.1, 1)
        check(o, lse, q, kv, pos, pre, P, table, 0.1, 1, P)


MANY = [SHAPES[0], SHAPES[3], SHAPES[6], SHAPES[7], SHAPES[9], SHAPES[11]]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", MANY)
def test_limits_anywhere_and_empty_rows(shape, fp8):
    B, Q, Hq, Hkv, D, page, P, own = shape
    print(shape, fp8, flush=True)
    rng = np.random.default_rng(P)
    kv, q, pre, table, n = build(rng, B, Q, Hq, Hkv, D, page, P, own, fp8)
    top = np.repeat([P + m for m in own], Q)
    pos = np.minimum(rng.integers(-30, n, B * Q), top - 1)
    pos[:3] = (P - 1, 0, -1)
    o, lse = call(kv, q, pos, pre, P, table, n, 0.1, Q)
    check(o, lse, q, kv, pos, pre, P, table, 0.1, Q, n)
    o, lse = call(kv, q, np.full(B * Q, -1), pre, P, table, n, 0.1, Q)
    assert (o == 0).all() and (lse == -np.inf).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", ["nan", "inf"])
@pytest.mark.parametrize("shape", MANY)
def test_what_a_row_does_not_see_does_not_enter(shape, bad, fp8):
    """NaN or inf in K, V and scales in the free part of pages, and in V at the keys of the
    sequences' last rows: those rows alone turn non-finite, the others stay as they were within
    the tolerance (key groups with a non-finite V are multiplied in another order)."""
    B, Q, Hq, Hkv, D, page, P, own = shape
    print(shape, bad, fp8, flush=True)
    rng = np.random.default_rng(6)
    kv, q, pre, table, n = build(rng, B, Q, Hq, Hkv, D, page, P, own, fp8)
    pos = positions(own, P, Q)
    pos[0] = P // 2                       # a row that ends inside the prefix
    want = ref.attention(q.double().numpy(), kv, pos, pre, P, table, 0.125, Q, n)
    val = float(bad)
    used = {(int(pre[j // page]), j % page) for j in range(P)} | \
        {(int(table[b, j // page]), j % page) for b in range(B) for j in range(P, P + own[b])}

    def spoil(pg, s, names):
        for name in names:
            if fp8:
                kv.t[name][pg, :, s] = 0x7F
                kv.t[name + "s"][pg, :, s] = val
            else:
                kv.t[name][pg, :, s] = val

    for pg in range(kv.t["k"].shape[0]):
        for s in range(page):
            if (pg, s) not in used:
                spoil(pg, s, "kv")
    dirty = np.zeros(B * Q, bool)
    for b in range(B):
        j = P + own[b] - 1                # the key of the sequence's last token
        spoil(int(table[b, j // page]), j % page, "v")
        dirty |= (np.arange(B * Q) // Q == b) & (pos >= j)
    o, lse = call(kv, q, pos, pre, P, table, n, 0.125, Q)
    assert dirty.any() and not dirty.all()
    assert not np.isfinite(o[dirty]).any()
    compare(o, lse, q, want, ~dirty)
    j = 2 * P // 3                        # and one that the row inside the prefix does not see
    spoil(int(pre[j // page]), j % page, "v")
    o, lse = call(kv, q, pos, pre, P, table, n, 0.125, Q)
    assert not np.isfinite(o[pos >= j]).any()
    compare(o, lse, q, want, pos < j)


def compare(o, lse, q, want, rows):
    """test_gpu_attn.check for some rows, against values formed before."""
    eo, el, mag, qk = (a[rows] for a in want)
    d = 2 * q.shape[2] * 2.0 ** -23 * qk
    tol = 1.05 * 2.0 ** -8 * (mag + np.abs(eo)) + (2 * d[..., None] + 2.0 ** -16) * mag
    assert (np.abs(o[rows] - eo) <= tol).all()
    assert (np.abs(lse[rows] - el) <= d + 2.0 ** -20 * (1 + np.abs(el))).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", MANY)
def test_bad_pages(shape, fp8):
    """Pages outside the cache, of the shared list and of a sequence's, hide their keys."""
    B, Q, Hq, Hkv, D, page, P, own = shape
    print(shape, fp8, flush=True)
    rng = np.random.default_rng(9)
    kv, q, pre, table, n = build(rng, B, Q, Hq, Hkv, D, page, P, own, fp8)
    pos = positions(own, P, Q)
    pre, table = pre.copy(), table.copy()
    pre[len(pre) // 2] = 10 ** 6
    o, lse = call(kv, q, pos, pre, P, table, n, 0.1, Q, expect_status=moe.MOE_STATUS_BAD_PAGE)
    check(o, lse, q, kv, pos, pre, P, table, 0.1, Q, n)
    b = int(np.argmax(own))
    table[b, (P + own[b] - 1) // page] = -5
    o, lse = call(kv, q, pos, pre, P, table, n, 0.1, Q, expect_status=moe.MOE_STATUS_BAD_PAGE)
    check(o, lse, q, kv, pos, pre, P, table, 0.1, Q, n)


def test_graph_replays():
    """A captured call of both kernels, replayed with other positions between eager calls."""
    rng = np.random.default_rng(2)
    B, Q, Hq, Hkv, D, page, P, own = SHAPES[0]
    kv, q, pre, table, n = build(rng, B, Q, Hq, Hkv, D, page, P, own, True)
    dev = {k: t.to("cuda:0") for k, t in kv.t.items()}
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to("cuda:0")  # noqa: E731
    c = moe.make_kv_cache(moe.MOE_DT_FP8_E4M3, dev["k"].shape[0], page, Hkv, D, dev["k"], dev["v"],
                          dev["ks"], dev["vs"])
    qd, pre_d, tab_d, pos_d = q.to("cuda:0"), i32(pre), i32(table), i32(positions(own, P, Q))
    nb = moe.attn_workspace_bytes(c, B, Q, Hq, P, n)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda:0")
    out, lse = torch.empty_like(qd), torch.empty((B * Q, Hq), device="cuda:0")

    def step():
        moe.attn_shared_prefix(c, qd, Hq * D, B, Q, Hq, pos_d, pre_d, P, tab_d, table.shape[1], n,
                               0.1, out, lse, None, ws, nb)

    step()
    torch.cuda.synchronize()
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        step()
    for shift in (0, 3, 1, 40):
        pos_d.copy_(i32(np.maximum(positions(own, P, Q) - shift, -1)))
        step()
        torch.cuda.synchronize()
        want = out.clone(), lse.clone()
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
