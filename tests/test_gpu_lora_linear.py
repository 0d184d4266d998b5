"""lora_linear against 64 bits: every rank and split of its kernels, mixed adapters in a tile, tokens
without one, what lies past a rank, NaN and infinities of other tokens and adapters."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_expert_ffn_moe_amd as moe  # noqa: E402

DEV = "cuda:0"


def run(x, a, b, rank, scale, of, base, out, xs=None, ys=None, bs=None, in_place=False, stream=None):
    """x [T][stride] etc. on the CPU; returns y [T][N] (CPU) and the status."""
    T, (n, R, K), N = x.shape[0], a.shape, b.shape[1]
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    up = lambda t: t.to(DEV).contiguous() if t is not None else None  # noqa: E731
    xd, ad, bd, rd, sd, od = (up(t) for t in (x, a, b, rank, scale, of))
    based = up(base)
    ys = ys or N
    y = based if in_place else torch.full((T, ys), 5.0, dtype=dt, device=DEV)
    bs = base.shape[1] if base is not None else 0
    w = moe.make_lora(n, R, K, N, ad, bd, rd, sd)
    nb = moe.lora_workspace_bytes(w, T)
    assert nb > 0
    ws = torch.full((nb // 4,), float("nan"), device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.lora_linear(w, xd, x.shape[1], T, od, based, bs, y, bs if in_place else ys,
                    moe.MOE_DT_BF16 if out == "bf16" else moe.MOE_DT_F32, st, ws, nb, stream)
    torch.cuda.synchronize()
    if not in_place and ys > N:
        assert bool((y[:, N:] == 5).all())
    return y.cpu()[:, :N], int(st.item())


def expect(x, a, b, rank, scale, of, base, K):
    """y and the size of what it is summed from, in 64 bits."""
    T, n, R, N = x.shape[0], a.shape[0], a.shape[1], b.shape[1]
    y = base[:, :N].double().clone() if base is not None else torch.zeros((T, N), dtype=torch.float64)
    mag = torch.zeros((T, N), dtype=torch.float64)
    for i in range(n):
        t = torch.nonzero(of == i)[:, 0]
        if not len(t):
            continue
        r = max(0, min(int(rank[i]), R)) if rank is not None else R
        s = float(scale[i]) if scale is not None else 1.0
        xd, ad, bd = x[t, :K].double(), a[i, :r].double(), b[i, :, :r].double()
        y[t] += (xd @ ad.T) @ bd.T * s
        mag[t] = (xd.abs() @ ad.abs().T) @ bd.abs().T * abs(s)
    return y, mag


def check(x, a, b, rank, scale, of, base, out, status=0, **kw):
    K = a.shape[2]
    y, st = run(x, a, b, rank, scale, of, base, out, **kw)
    assert st == status
    e, mag = expect(x, a, b, rank, scale, of, base, K)
    # sums of K products, then of R, in fp32 (the matrix cores' additions within 2^-23 each), joined
    # over 8 waves and 16 parts; then one rounding of y
    tol = (K + a.shape[1] + 32) * 2.0 ** -23 * mag + (2.0 ** -8 if out == "bf16" else 2.0 ** -23) * e.abs()
    bad = ~((y.double() - e).abs() <= tol + 1e-30)
    assert not bool(bad.any()), (int(bad.sum()), float((y.double() - e).abs().max()))
    return y


def make(rng, T, K, N, n, R, out, ranks=False, pad=0, basis=True):
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    x, a, b = f(T, K + pad).to(torch.bfloat16), f(n, R, K).to(torch.bfloat16), f(n, N, R).to(torch.bfloat16)
    rank = torch.from_numpy(rng.integers(0, R + 1, n).astype(np.int32)) if ranks else None
    scale = torch.from_numpy((0.2 + rng.random(n)).astype(np.float32))
    of = torch.from_numpy(rng.integers(-1, n, T).astype(np.int32))
    base = (10 * f(T, N + pad)).to(torch.bfloat16 if out == "bf16" else torch.float32) if basis else None
    return x, a, b, rank, scale, of, base


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 96, 128])
def test_ranks(R, out):
    rng = np.random.default_rng(R)
    for T, K, N, n, ranks in [(1, 64, 64, 1, False), (1, 520, 100, 3, True), (16, 256, 1000, 5, True),
                              (37, 1000, 65, 40, True), (5, 8, 1, 2, False)]:
        print(R, out, T, K, N, n, flush=True)
        check(*make(rng, T, K, N, n, R, out, ranks), out)


@pytest.mark.parametrize("T,K,N,n,R", [(1, 4096, 300, 2, 16), (32, 2056, 500, 32, 64), (300, 600, 128, 6, 32),
                                       (1500, 264, 70, 3, 8), (4100, 72, 40, 9, 16), (3, 70000, 17, 3, 8)])
def test_sizes(T, K, N, n, R):
    """Few tokens and many (from 1024), several parts of x's columns, several passes a part."""
    rng = np.random.default_rng(T)
    x, a, b, rank, scale, of, base = make(rng, T, K, N, n, R, "bf16", True, pad=8)
    check(x, a, b, rank, scale, of, base, "bf16", ys=N + 3)
    of = torch.from_numpy((np.arange(T) * n // T).astype(np.int32))      # runs of one adapter
    check(x, a, b, rank, scale, of, base, "bf16", in_place=True)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("R", [8, 16, 32, 64, 104, 128])
def test_many_tokens(R, out):
    """Every rank's kernels for many tokens (from 1024): chunks of outputs cut short, a last block of few
    tokens, one or many adapters a block."""
    rng = np.random.default_rng(R)
    for T, K, N, n in [(1024, 1104, 700, 2), (1415, 72, 64, 30), (1090, 4104, 257, 5), (1025, 2048, 33, 1),
                       (2000, 136, 3, 70)]:
        print(R, out, T, K, N, n, flush=True)
        x, a, b, rank, scale, of, base = make(rng, T, K, N, n, R, out, True)
        check(x, a, b, rank, scale, of, base, out)
        of = torch.from_numpy((np.arange(T) * n // T).astype(np.int32))
        check(x, a, b, None, scale, of, base, out, in_place=True)


@pytest.mark.parametrize("T", [19, 270])      # in one launch (ranks up to 32) and in two
@pytest.mark.parametrize("R", [8, 16, 32, 64])
def test_exact_sums_keep_every_bit(R, T):
    """Whole numbers whose sums stay below 2^24: fp32 outputs are exact, so nothing of a x is lost on
    its way through the second product."""
    rng = np.random.default_rng(R)
    K, N, n = 640, 130, 4
    i = lambda lo, hi, *s: torch.from_numpy(rng.integers(lo, hi + 1, s).astype(np.float32))  # noqa: E731
    x, a, b = i(-9, 9, T, K), i(-9, 9, n, R, K), i(-3, 3, n, N, R)
    of = torch.from_numpy(rng.integers(-1, n, T).astype(np.int32))
    base = i(-1000, 1000, T, N)
    scale = torch.tensor([1.0, 2.0, 0.5, 4.0])
    y, st = run(x.to(torch.bfloat16), a.to(torch.bfloat16), b.to(torch.bfloat16), None, scale, of, base, "f32")
    e, mag = expect(x, a, b, None, scale, of, base, K)
    hm = max(float((x[t].double() @ a[int(of[t])].double().T).abs().max()) for t in range(T) if of[t] >= 0)
    assert hm > 2 ** 9 and float(mag.max()) < 2 ** 24      # more bits than a bf16 has, no sum is rounded
    assert st == 0 and torch.equal(y.double(), e)


def test_what_is_not_the_tokens_does_not_reach_it():
    """NaN and infinities in other adapters, past the ranks, in other tokens of the tile; NaN between
    the rows of x."""
    rng = np.random.default_rng(1)
    T, K, N, n, R = 20, 136, 90, 5, 32
    x, a, b, rank, scale, of, base = make(rng, T, K, N, n, R, "f32", pad=8)
    rank = torch.tensor([32, 7, 0, 17, 25], dtype=torch.int32)
    of = torch.from_numpy(np.tile(np.array([0, 1, 2, 3, -1], np.int32), 4))
    want = check(x, a, b, rank, scale, of, base, "f32")
    for i in range(n):
        r = int(rank[i])
        a[i, r:], b[i, :, r:] = float("nan"), float("inf")
    a[4], b[4], x[:, K:] = float("nan"), float("nan"), float("nan")
    scale[4] = float("nan")
    assert torch.equal(run(x, a, b, rank, scale, of, base, "f32")[0], want)
    x[0], x[6, 3], x[4] = float("nan"), float("inf"), float("nan")       # tokens of adapters 0, 1, none
    y, _ = run(x, a, b, rank, scale, of, base, "f32")
    same = torch.ones(T, dtype=torch.bool)
    same[0] = same[6] = False
    assert torch.equal(y[same], want[same])
    assert bool(y[0].isnan().all()) and not bool(y[6].isfinite().any())


def test_no_base_no_adapter_and_bad_numbers():
    rng = np.random.default_rng(2)
    T, K, N, n, R = 18, 64, 77, 3, 16
    x, a, b, rank, scale, of, base = make(rng, T, K, N, n, R, "bf16")
    check(x, a, b, None, None, of, None, "bf16")
    of[:] = -1
    y, st = run(x, a, b, None, None, of, base, "bf16")
    assert st == 0 and torch.equal(y, base)
    y, st = run(x, a, b, None, None, of, None, "bf16")
    assert st == 0 and bool((y == 0).all())
    of[3], of[17], of[4] = n, 2 ** 31 - 1, 1
    ok = of.clone()
    ok[3] = ok[17] = -1
    y, st = run(x, a, b, None, None, of, base, "bf16")
    assert st == moe.MOE_STATUS_BAD_INDEX
    assert torch.equal(y, run(x, a, b, None, None, ok, base, "bf16")[0])


def test_in_place_leaves_other_rows_alone():
    """Rows without an adapter are not written in place; rows behind the last token neither."""
    rng = np.random.default_rng(3)
    T, K, N, n, R = 21, 128, 96, 2, 8
    x, a, b, _, scale, of, base = make(rng, T, K, N, n, R, "f32")
    of[5] = -1
    base[5, 7] = float("nan")
    y = torch.cat([base, torch.full((3, N), 5.0)]).to(DEV)
    w = moe.make_lora(n, R, K, N, a.to(DEV), b.to(DEV), None, scale.to(DEV))
    nb = moe.lora_workspace_bytes(w, T)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    moe.lora_linear(w, x.to(DEV), K, T, of.to(DEV), y, N, y, N, moe.MOE_DT_F32, None, ws, nb)
    torch.cuda.synchronize()
    assert torch.equal(y[5].view(torch.int32).cpu(), base[5].view(torch.int32)) and bool((y[T:] == 5).all())


def test_stacks_past_4_gib():
    """Offsets past 32 bits in both stacks: the last of many adapters."""
    K, N, R = 8192, 8192, 64
    n = (1 << 32) // (R * K * 2) + 2
    a = torch.zeros((n, R, K), dtype=torch.bfloat16, device=DEV)
    b = torch.zeros((n, N, R), dtype=torch.bfloat16, device=DEV)
    a[-1, :, -1], b[-1, -1, :] = 1.0, 2.0
    x = torch.ones((1, K), dtype=torch.bfloat16, device=DEV)
    of = torch.tensor([n - 1], dtype=torch.int32, device=DEV)
    y = torch.empty((1, N), device=DEV)
    w = moe.make_lora(n, R, K, N, a, b)
    nb = moe.lora_workspace_bytes(w, 1)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    moe.lora_linear(w, x, K, 1, of, None, 0, y, N, moe.MOE_DT_F32, None, ws, nb)
    torch.cuda.synchronize()
    assert float(y[0, -1]) == 128.0 and float(y[0, :-1].abs().max()) == 0.0


def test_captured_beside_eager_calls_with_a_workspace_each():
    rng = np.random.default_rng(4)
    T, K, N, n, R = 40, 512, 300, 6, 32
    x, a, b, _, scale, of, base = (t.to(DEV) if t is not None else None for t in make(rng, T, K, N, n, R, "bf16"))
    w = moe.make_lora(n, R, K, N, a, b, None, scale)
    nb = moe.lora_workspace_bytes(w, T)
    ws = [torch.empty(nb, dtype=torch.uint8, device=DEV) for _ in range(2)]
    out = [torch.empty((T, N), dtype=torch.bfloat16, device=DEV) for _ in range(2)]

    def go(k):
        moe.lora_linear(w, x, K, T, of, base, N, out[k], N, moe.MOE_DT_BF16, None, ws[k], nb)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        go(0)
    for i in range(3):
        x.copy_(torch.randn_like(x))
        of.copy_(torch.randint(-1, n, (T,), dtype=torch.int32))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            go(1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], out[1])


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("R", [8, 16, 24, 32])
def test_one_launch_or_two(R, out):
    """Small adapters at both sides of the limits of tokens times outputs and of ranks times columns: one
    kernel for up to 256 blocks of 512 outputs, and up to 2^18 elements of a (2^17 past rank 16)."""
    rng = np.random.default_rng(R)
    for T, K, N, n in [(256, 72, 40, 7), (257, 72, 40, 7), (300, 1000, 65, 40), (1, 2048, 1500, 3), (2, 2056, 515, 2),
                       (1, 4096, 33, 2), (3, 4104, 100, 2), (19, 6000, 130, 30), (40, 264, 5000, 9),
                       (2, 16384 // R * 8, 70, 2), (2, 16384 // R * 8 + 8, 70, 2), (2, 32768 // R * 8, 70, 2),
                       (2, 32768 // R * 8 + 8, 70, 2)]:
        print(R, out, T, K, N, n, flush=True)
        x, a, b, rank, scale, of, base = make(rng, T, K, N, n, R, out, True, pad=8)
        check(x, a, b, rank, scale, of, base, out, ys=N + 1)
        check(x, a, b, None, None, of, base, out, in_place=True)


def test_two_launches_and_what_is_not_the_tokens():
    """The same of NaN, infinities and bad numbers in two launches: tokens enough."""
    rng = np.random.default_rng(12)
    T, K, N, n, R = 270, 136, 90, 5, 32
    x, a, b, rank, scale, of, base = make(rng, T, K, N, n, R, "f32", pad=8)
    rank = torch.tensor([32, 7, 0, 17, 25], dtype=torch.int32)
    of = torch.from_numpy(np.tile(np.array([0, 1, 2, 3, -1], np.int32), 54))
    want = check(x, a, b, rank, scale, of, base, "f32")
    for i in range(n):
        r = int(rank[i])
        a[i, r:], b[i, :, r:] = float("nan"), float("inf")
    a[4], b[4], x[:, K:], scale[4] = float("nan"), float("nan"), float("nan"), float("nan")
    x[0], x[6, 3], x[4] = float("nan"), float("inf"), float("nan")
    of[8], of[263] = n, 2 ** 31 - 1
    y, st = run(x, a, b, rank, scale, of, base, "f32")
    assert st == moe.MOE_STATUS_BAD_INDEX
    same = torch.ones(T, dtype=torch.bool)
    same[0] = same[6] = same[8] = same[263] = False
    assert torch.equal(y[same], want[same]) and torch.equal(y[[8, 263]], base[[8, 263], :N])
    assert bool(y[0].isnan().all()) and not bool(y[6].isfinite().any())


def test_the_workspace_of_a_large_batch_serves_smaller_ones():
    """One allocation for up to 2400 tokens, calls of fewer with the bytes that it has: several of them have
    more parts of x's columns than 2400 have.  Bytes behind it stay as they were."""
    rng = np.random.default_rng(14)
    K, N, n, R = 8192, 40, 3, 32
    w0 = moe.make_lora(n, R, K, N, 256, 256)
    nb = moe.lora_workspace_bytes(w0, 2400)
    ws = torch.full((nb + 4096,), 0xAB, dtype=torch.uint8, device=DEV)
    x, a, b, rank, scale, of, base = make(rng, 2400, K, N, n, R, "f32")
    w = moe.make_lora(n, R, K, N, a.to(DEV), b.to(DEV), None, scale.to(DEV))
    e, mag = expect(x, a, b, None, scale, of, base, K)
    tol = (K + R + 32) * 2.0 ** -23 * mag + 2.0 ** -23 * e.abs()       # as in check()
    xd, od, based = x.to(DEV), of.to(DEV), base.to(DEV)
    for T in (1, 33, 1000, 1023, 1024, 1500, 2336, 2337, 2400):
        print(T, flush=True)
        y = torch.full((T, N), 5.0, device=DEV)
        moe.lora_linear(w, xd, K, T, od, based, N, y, N, moe.MOE_DT_F32, None, ws, nb)
        torch.cuda.synchronize()
        assert bool(((y.cpu().double() - e[:T]).abs() <= tol[:T]).all())
        assert bool((ws[nb:] == 0xAB).all())


def cut3(h):
    """h (float32) as the kernels cut it: three bf16, 8 bits each, cut off."""
    p = [np.zeros_like(h)] * 3
    for k in range(3):
        p[k] = (h.view(np.uint32) & 0xffff0000).view(np.float32)
        h = h - p[k]
    return p


@pytest.mark.parametrize("T", [19, 270, 1100])      # one launch (ranks up to 32), two, three
@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 128])
def test_every_part_of_h_counts(R, T):
    """Whole numbers whose sums stay below 2^24, with a x of up to 20 bits: fp32 outputs are exact, and no
    fewer than three bf16 parts of a x hold it (shown here: without the last one y is another)."""
    rng = np.random.default_rng(R)
    K, N, n = 640, 70, 4
    i = lambda lo, hi, *s: torch.from_numpy(rng.integers(lo, hi + 1, s).astype(np.float32))  # noqa: E731
    x, a = i(-127, 127, T, K), i(-127, 127, n, R, K)
    b = torch.zeros((n, N, R))                       # four ranks an output, every rank in one of them
    for k in range(N):
        b[:, k, [(4 * k + j) % R for j in range(4)]] = 2 * i(0, 1, n, 4) - 1
    of = torch.from_numpy((np.arange(T) % (n + 1) - 1).astype(np.int32))
    base = i(-1000, 1000, T, N)
    scale = torch.tensor([1.0, 2.0, 0.5, 4.0])
    e, _ = expect(x, a, b, None, scale, of, base, K)
    assert float((x.abs() @ a.abs().flatten(0, 1).T).max()) < 2 ** 24
    for ad in range(n):
        t = of == ad
        h = ((x[t].double() @ a[ad].double().T) * float(scale[ad])).numpy()
        bd = b[ad].double().numpy().T
        assert (np.abs(h) @ np.abs(bd)).max() + 1000 < 2 ** 23      # (sums of halves too are exact)
        p = cut3(h.astype(np.float32))
        assert np.array_equal(p[0].astype(np.float64) + p[1] + p[2], h)
        less = base[t].double().numpy() + (p[0].astype(np.float64) + p[1]) @ bd
        assert (p[2] != 0).mean() > 0.1 and (less != e[t].numpy()).any(0).mean() > 0.5
        assert T < 100 or (p[2] != 0).any(0).all() and (less != e[t].numpy()).any(0).all()
    y, st = run(x.to(torch.bfloat16), a.to(torch.bfloat16), b.to(torch.bfloat16), None, scale, of, base, "f32")
    assert st == 0 and torch.equal(y.double(), e)


@pytest.mark.parametrize("R", [8, 16, 32, 64, 128])
def test_many_tokens_and_what_is_not_the_tokens(R):
    """NaN, infinities and bad numbers of other adapters and tokens from 1024 tokens on."""
    rng = np.random.default_rng(13)
    T, K, N, n = 1100, 136, 90, 5
    x, a, b, rank, scale, of, base = make(rng, T, K, N, n, R, "f32", pad=8)
    rank = torch.tensor([R, 7, 0, R // 2 + 1, R - 7], dtype=torch.int32)
    of = torch.from_numpy(np.tile(np.array([0, 1, 2, 3, -1], np.int32), T // 5))
    want = check(x, a, b, rank, scale, of, base, "f32")
    for i in range(n):
        r = int(rank[i])
        a[i, r:], b[i, :, r:] = float("nan"), float("inf")
    a[4], b[4], x[:, K:], scale[4] = float("nan"), float("nan"), float("nan"), float("nan")
    x[0], x[6, 3], x[4] = float("nan"), float("inf"), float("nan")
    of[8], of[1093] = n, 2 ** 31 - 1
    y, st = run(x, a, b, rank, scale, of, base, "f32")
    assert st == moe.MOE_STATUS_BAD_INDEX
    same = torch.ones(T, dtype=torch.bool)
    same[0] = same[6] = same[8] = same[1093] = False
    assert torch.equal(y[same], want[same]) and torch.equal(y[[8, 1093]], base[[8, 1093], :N])
    assert bool(y[0].isnan().all()) and not bool(y[6].isfinite().any())


@pytest.mark.parametrize("T,K,N,n,R", [(2048, 14336, 40, 4, 24), (4096, 9000, 70, 3, 64), (1056, 20000, 33, 9, 8),
                                       (8192, 4096, 64, 2, 16)])
def test_many_tokens_in_several_passes_a_part(T, K, N, n, R):
    """So many tokens and columns that a part of x's columns is 2048 or more: a block takes it in passes, the
    last of them cut short."""
    rng = np.random.default_rng(T)
    x, a, b, rank, scale, of, base = make(rng, T, K, N, n, R, "bf16", True, pad=8)
    check(x, a, b, rank, scale, of, base, "bf16")
    of = torch.from_numpy((np.arange(T) * n // T).astype(np.int32))      # runs of one adapter
    check(x, a, b, None, scale, of, base, "bf16", in_place=True)


@pytest.mark.parametrize("T,K,N,R", [(16, 4096, 4096, 32), (17, 4096, 4096, 32), (21, 4096, 4096, 24),
                                     (22, 4096, 4096, 24), (256, 2048, 300, 32), (250, 2096, 300, 32),
                                     (251, 2096, 300, 32)])
def test_one_launch_or_two_past_rank_16(T, K, N, R):
    """Both sides of 2^24 elements of a, read by all blocks of 512 outputs together."""
    rng = np.random.default_rng(T)
    x, a, b, rank, scale, of, base = make(rng, T, K, N, 3, R, "bf16", True)
    check(x, a, b, rank, scale, of, base, "bf16")
    check(x, a, b, None, None, of, base, "bf16", in_place=True)
