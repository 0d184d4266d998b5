"""kv_append_rope against the rotation in float32 with every operation rounded
(numpy float32) and torch's conversions: bit for bit, and nothing else of the
cache touched."""
import numpy as np
import pytest
import torch

import ops_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_expert_ffn_moe_amd as moe  # noqa: E402

DEV = "cuda:0"


def run(rng, T, Hq, Hkv, D, page, rot, pairs, fp8, seq, pos, table, n_pages, extra=0, rows=None,
        qkv=None, expect_status=0):
    rows = rows or int(max(pos.max(), 0)) + 1
    tab = ref.rope_table(rows, rot) if rot else None
    row = (Hq + 2 * Hkv) * D + extra
    if qkv is None:
        qkv = ref.bf16(rng.standard_normal((T, row)).astype(np.float32))
    kv = ref.Cache(rng, n_pages, page, Hkv, D, fp8)
    want = {n: t.clone() if t is not None else None for n, t in kv.t.items()}
    q_want = torch.full((T, Hq, D), 5.0, dtype=torch.bfloat16)
    x = qkv.float().numpy()[:, :row - extra].reshape(T, Hq + 2 * Hkv, D)
    for t in range(T):
        if seq[t] < 0 or pos[t] < 0 or seq[t] >= table.shape[0] or \
                pos[t] // page >= table.shape[1] or (rot and pos[t] >= rows):
            continue
        pg, sl = int(table[seq[t], pos[t] // page]), int(pos[t] % page)
        if pg < 0 or pg >= n_pages:
            continue
        r = ref.rotate_f32(x[t:t + 1, :Hq + Hkv], tab[pos[t]][None], rot, pairs) if rot else \
            x[t:t + 1, :Hq + Hkv]
        q_want[t] = ref.bf16(r[0, :Hq])
        for n, new in (("k", r[0, Hq:]), ("v", x[t, Hq + Hkv:])):
            if fp8:
                codes, s = ref.fp8_rows(new)
                want[n][pg, :, sl], want[n + "s"][pg, :, sl] = torch.from_numpy(codes), torch.from_numpy(s)
            else:
                want[n][pg, :, sl] = ref.bf16(new)
    d = {n: t.to(DEV) if t is not None else None for n, t in kv.t.items()}
    c = moe.make_kv_cache(moe.MOE_DT_FP8_E4M3 if fp8 else moe.MOE_DT_BF16, n_pages, page, Hkv, D,
                          d["k"], d["v"], d["ks"], d["vs"])
    qd = qkv.to(DEV)
    q_out = torch.full((T, Hq, D), 5.0, dtype=torch.bfloat16, device=DEV) if Hq else None
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)  # noqa: E731
    a, seq_d, pos_d, table_d = qd.data_ptr(), i32(seq), i32(pos), i32(table)
    tab_d = torch.from_numpy(tab).to(DEV) if rot else None
    moe.kv_append_rope(c, a if Hq else None, row, Hq, a + 2 * Hq * D, row, a + 2 * (Hq + Hkv) * D,
                       row, T, tab_d, rows, rot, moe.ROPE_PAIRS if pairs else moe.ROPE_HALF,
                       seq_d, pos_d, table_d, table.shape[0], table.shape[1], q_out, st)
    torch.cuda.synchronize()
    bits = lambda t: t.view(torch.int16) if t.dtype == torch.bfloat16 else t  # noqa: E731
    if Hq:
        assert torch.equal(bits(q_out.cpu()), bits(q_want))
    for n in ("k", "v", "ks", "vs"):
        if want[n] is not None:
            got = d[n].cpu()
            assert torch.equal(bits(got), bits(want[n])), n
    assert int(st.item()) == expect_status
    return d


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("pairs", [False, True])
def test_tokens_of_several_sequences(D, fp8, pairs):
    rng = np.random.default_rng(D + 2 * fp8 + pairs)
    for T, Hq, Hkv, page, rot, extra in [(1, 1, 1, 16, D, 0), (5, 6, 2, 16, D // 2, 8),
                                         (33, 32, 8, 64, 16, 0), (7, 0, 3, 32, 0, 16),
                                         (700, 3, 1, 128, D, 0)]:
        print(T, Hq, Hkv, D, page, rot, flush=True)
        B = min(T, 9)
        cols = 6
        n_pages = B * cols + 3
        table = rng.permutation(n_pages)[:B * cols].reshape(B, cols)
        # distinct (sequence, position) pairs
        flat = rng.permutation(B * cols * page)[:T]
        run(rng, T, Hq, Hkv, D, page, rot, pairs, fp8, flat // (cols * page), flat % (cols * page),
            table, n_pages, extra)


@pytest.mark.parametrize("fp8", [False, True])
def test_padding_and_out_of_range(fp8):
    """Negative sequence or position: silent; a sequence, position, table row or
    page out of range: skipped and reported.  Nothing is written for either."""
    rng = np.random.default_rng(1)
    table = np.array([[0, 1], [2, -1], [9, 3]])
    run(rng, 4, 2, 1, 64, 16, 64, False, fp8, np.array([-1, 0, 0, 1]), np.array([3, -5, 31, 4]),
        table, 4)
    for seq, pos in [(3, 0), (0, 32), (1, 16), (2, 5), (0, 2 ** 31 - 1)]:
        rows = 32
        run(rng, 2, 2, 1, 64, 16, 64, False, fp8, np.array([0, seq]), np.array([1, pos]), table, 4,
            rows=rows, expect_status=moe.MOE_STATUS_BAD_PAGE)
    # a position past the table of rotations
    run(rng, 1, 2, 1, 64, 16, 64, False, fp8, np.array([0]), np.array([20]), table, 4, rows=20,
        expect_status=moe.MOE_STATUS_BAD_PAGE)


def test_zero_rows_and_signed_zeros_in_fp8():
    rng = np.random.default_rng(2)
    T, D = 3, 64
    qkv = ref.bf16(rng.standard_normal((T, 3 * D)).astype(np.float32))
    qkv[0, D:] = 0
    qkv[1, 2 * D:] = -0.0
    run(rng, T, 1, 1, D, 16, 0, False, True, np.zeros(3, int), np.arange(3), np.array([[1]]), 2,
        qkv=qkv)


def test_cache_past_4_gib():
    """Byte offsets past 32 bits: the last page of a cache of over 4 GiB."""
    Hkv, D, page = 8, 128, 64
    n_pages = (1 << 32) // (Hkv * D * page * 2) + 3
    k = torch.zeros((n_pages, Hkv, page, D), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    c = moe.make_kv_cache(moe.MOE_DT_BF16, n_pages, page, Hkv, D, k, v)
    x = torch.randn((1, 2 * Hkv * D), device=DEV).to(torch.bfloat16)
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.tensor([[n_pages - 1]], dtype=torch.int32, device=DEV)
    pos = torch.tensor([63], dtype=torch.int32, device=DEV)
    moe.kv_append_rope(c, None, 0, 0, x, 2 * Hkv * D, x.data_ptr() + 2 * Hkv * D, 2 * Hkv * D, 1,
                       None, 0, 0, 0, one, pos, table, 1, 1, None, None)
    torch.cuda.synchronize()
    assert torch.equal(k[-1, :, 63].reshape(-1), x[0, :Hkv * D])
    assert torch.equal(v[-1, :, 63].reshape(-1), x[0, Hkv * D:])
    assert int((k != 0).sum()) == int((x[0, :Hkv * D] != 0).sum())
