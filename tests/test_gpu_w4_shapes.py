"""w4_linear where a block of the matrix-core kernel takes several tiles of rows: its ring of
loads, the sums joined one tile behind, the sums kept over passes of K, and the form for many
tiles a block; against the dequantised product in 64 bits (tolerances: test_gpu_w4_linear.check).
Rows are checked in full: a tile joined too early or late shows in its own rows."""
import numpy as np
import pytest
import torch

import ops_ref as ref
from test_gpu_w4_linear import call, check, make

pytestmark = pytest.mark.gpu

import bit_expert_ffn_moe_amd as moe  # noqa: E402

DEV = "cuda:0"


@pytest.mark.parametrize("fmt,group,zeros", [("fp4", 32, False), ("int4", 32, True),
                                             ("int4", 64, False), ("int4", 128, True)])
@pytest.mark.parametrize("N,K,Ts", [
    (70001, 96, (3, 20, 40)),        # 4376 tiles: many a block, K cut short
    (33005, 512, (3, 20, 40)),       # 2063 tiles, whole steps
    (40003, 1152, (40,)),            # two steps a wave
    (8211, 544, (6, 24, 64)),        # two or three tiles a block: the ring's start and end
    (5000, 2080, (17, 65)),          # a second block of tokens
    (9000, 4224, (5, 33)),           # several passes over K, two to three tiles each
])
def test_several_tiles_a_block(fmt, group, zeros, N, K, Ts):
    rng = np.random.default_rng(N + group)
    q, s, z = make(rng, fmt, N, K, group, zeros)
    w, mag = ref.w4_dequant(fmt, q, s, z, group)
    for T in Ts:
        print(fmt, group, N, K, T, flush=True)
        x = ref.bf16(rng.standard_normal((T, K)).astype(np.float32))
        f32 = T != 24
        check(call(fmt, N, K, group, q, s, z, x, K + 8, N + 5, f32), x, w, mag, K, f32)


@pytest.mark.parametrize("fmt,group", [("fp4", 32), ("int4", 128)])
def test_more_tiles_than_are_kept_over_the_passes(fmt, group):
    """Over 16 tiles a block with K in several passes: groups of 16 tiles."""
    rng = np.random.default_rng(1)
    N, K, T = 256 * 16 * 17 + 7, 2080, 33
    q, s, z = make(rng, fmt, N, K, group, True)
    x = ref.bf16(rng.standard_normal((T, K)).astype(np.float32))
    y = call(fmt, N, K, group, q, s, z, x)
    part = np.arange(0, N, 5)           # rows of every place in a tile, of every tile
    w, mag = ref.w4_dequant(fmt, q[part], s[part], z[part] if z is not None else None, group)
    check(y[:, part], x, w, mag, K, True)


@pytest.mark.parametrize("T", [1, 3, 20])
def test_graph_replays(T):
    """A captured call, replayed with new activations between eager calls."""
    rng = np.random.default_rng(9)
    N, K = 5000, 1024
    q, s, _ = make(rng, "fp4", N, K, 32)
    qd, sd = torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV)
    w = moe.make_w4(moe.MOE_W_FP4_E2M1_UE8M0_K32, N, K, 32, qd, sd)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    y, eager = (torch.empty((T, N), device=DEV) for _ in range(2))
    moe.w4_linear(w, x, K, T, y, N, moe.MOE_DT_F32)
    torch.cuda.synchronize()
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        moe.w4_linear(w, x, K, T, y, N, moe.MOE_DT_F32)
    for _ in range(4):
        x.copy_(ref.bf16(rng.standard_normal((T, K)).astype(np.float32)))
        y.fill_(-7.0)
        graph.replay()
        moe.w4_linear(w, x, K, T, eager, N, moe.MOE_DT_F32)
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and float(y.abs().max()) > 0
