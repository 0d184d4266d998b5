"""CPU tests of the decode-step operators' limits: what the launches could not hold is refused
with the arguments, not after kernels have been enqueued."""
import ctypes

import pytest

moe = pytest.importorskip("bit_expert_ffn_moe_amd")

P, BIG = 0x100000, 1 << 50


def cache(Hkv, D):
    return ctypes.byref(moe.make_kv_cache(moe.MOE_DT_BF16, 10, 16, Hkv, D, P, P))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,Q,Hq,Hkv", [(1 << 18, 1, 64, 64), (1 << 14, 1, 1024, 8),
                                        (1 << 8, 1 << 10, 64, 8)])
def test_attention_rows(B, Q, Hq, Hkv, D):
    """2^24 rows: blocks of 256 threads each would be a grid of 2^32 threads, which no launch
    takes.  One token or sequence fewer is accepted."""
    size = moe._lib.attn_workspace_bytes
    assert size(cache(Hkv, D), B, Q, Hq, 16, 64) == 0
    assert size(cache(Hkv, D), B - 1, Q, Hq, 16, 64) > 0
    assert moe.raw_call("attn_shared_prefix", cache(Hkv, D), P, Hq * D, B, Q, Hq, P, P, 16, P, 4, 64,
                        0.1, P, None, None, P, BIG, None) == moe.MOE_ENOTSUP
