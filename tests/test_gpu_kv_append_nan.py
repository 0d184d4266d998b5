"""kv_append_rope into an E4M3 cache with NaN and infinities in a head row: what the row reads
back as, code times scale, is NaN where a bf16 cache would read NaN, and the row's other
values are as they are without it; other rows are untouched."""
import numpy as np
import pytest
import torch

import ops_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_expert_ffn_moe_amd as moe  # noqa: E402

DEV = "cuda:0"
nan, inf = float("nan"), float("inf")


def append(x, T, D, Hkv, rot=None, pairs=False):
    """k and v rows of x [T][2 Hkv D] appended at slots 0.. of one page: codes and scales."""
    page = 16
    k, v = (torch.zeros((2, Hkv, page, D), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((2, Hkv, page), device=DEV) for _ in range(2))
    c = moe.make_kv_cache(moe.MOE_DT_FP8_E4M3, 2, page, Hkv, D, k, v, ks, vs)
    xd = x.to(DEV)
    seq = torch.zeros(T, dtype=torch.int32, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    table = torch.tensor([[1]], dtype=torch.int32, device=DEV)
    tab = torch.from_numpy(ref.rope_table(page, rot)).to(DEV) if rot else None
    moe.kv_append_rope(c, None, 0, 0, xd, 2 * Hkv * D, xd.data_ptr() + 2 * Hkv * D, 2 * Hkv * D, T,
                       tab, page if rot else 0, rot or 0,
                       (moe.ROPE_PAIRS if pairs else moe.ROPE_HALF) if rot else 0, seq, pos, table,
                       1, 1, None, None)
    torch.cuda.synchronize()
    return [t[1, :, :T].cpu() for t in (k, v, ks, vs)]


def values(codes, scales):
    return codes.view(torch.float8_e4m3fn).double() * scales.double()[..., None]


@pytest.mark.parametrize("D", [64, 128, 256])
def test_nan_reads_back_as_nan(D):
    rng = np.random.default_rng(D)
    T, Hkv = 6, 2
    x = ref.bf16(rng.standard_normal((T, 2 * Hkv * D)).astype(np.float32))
    clean = append(x, T, D, Hkv)
    r = x.view(T, 2, Hkv, D).clone()
    # token 0: one NaN in a K head; 1: several in a V head, the last element too; 2: a row of
    # NaN; 3: NaN beside zeros; others clean.  The rows' largest values stay
    big = r.float().abs().argmax(-1)
    at = (big[0, 0, 1] + 3) % D
    r[0, 0, 1, at] = nan
    spots = [int((big[1, 1, 0] + i) % D) for i in (1, 7, 12, 20)]
    r[1, 1, 0, spots] = nan
    r[2, 0, 0] = nan
    r[3, 1, 1] = 0
    r[3, 1, 1, D - 1] = nan
    got = append(r.view(T, -1), T, D, Hkv)
    for kind in (0, 1):
        g, c = values(got[kind], got[kind + 2]), values(clean[kind], clean[kind + 2])
        for t in range(T):
            for h in range(Hkv):
                row = r[t, kind, h].float()
                assert torch.equal(torch.isnan(g[h, t]), torch.isnan(row)), (kind, t, h)
                if (t, kind, h) == (3, 1, 1):
                    assert (g[h, t][:D - 1] == 0).all()
                elif not torch.isnan(row).all():
                    keep = ~torch.isnan(row)
                    assert torch.equal(g[h, t][keep], c[h, t][keep]), (kind, t, h)
                    assert torch.equal(got[kind + 2][h, t], clean[kind + 2][h, t])


@pytest.mark.parametrize("pairs", [False, True])
def test_nan_goes_through_the_rotation(pairs):
    """Both values of the rotated pair are NaN, none other."""
    D, T = 64, 4
    x = ref.bf16(np.random.default_rng(1).standard_normal((T, 2 * D)).astype(np.float32))
    x[2, 10] = nan
    got = append(x, T, D, 1, rot=D, pairs=pairs)
    g = values(got[0], got[2])[0]
    hit = torch.zeros((T, D), dtype=torch.bool)
    hit[2, [10, 11] if pairs else [10, 42]] = True
    assert torch.equal(torch.isnan(g), hit)


def test_infinity_leaves_no_finite_number():
    """E4M3 has no infinity: the row's scale is inf, and every value reads as NaN or inf."""
    D, T = 128, 3
    x = ref.bf16(np.random.default_rng(2).standard_normal((T, 2 * D)).astype(np.float32))
    clean = append(x, T, D, 1)
    x[1, 5] = -inf
    got = append(x, T, D, 1)
    g = values(got[0], got[2])[0]
    assert not torch.isfinite(g[1]).any()
    for t in (0, 2):
        assert torch.equal(got[0][0, t], clean[0][0, t])
    assert torch.equal(got[1], clean[1])
