"""GPU: rotation of the queries' rope columns against the rotation in 64 bits.  Two fp32
products and a sum of bf16 inputs, rounded once: off by at most half a bf16 step (2^-8 of the
value) and 2^-22 of the pair's size (three fp32 roundings, and cancellation of the two)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import dev
from spec_util import bf16_bits, bf16_value, freqs_table, rotate64

pytestmark = pytest.mark.gpu
FILL = 0x1234


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300  # noqa: F401


def problem(seed, rows, heads, P, seq):
    gen = np.random.default_rng(seed)
    x = bf16_bits(gen.standard_normal((rows, heads, P)))
    pos = gen.integers(0, seq, rows).astype(np.uint32)
    pos[:1] = seq - 1
    return x, pos, freqs_table(seq, P) * np.float32(1.25)  # scaled, as a long-context table is


def assert_rotated(got, x, pos, freqs, half):
    x64, cs = bf16_value(x), freqs.astype(np.float64)[pos][:, None]
    ref = rotate64(x64, cs, half)
    size = rotate64(np.abs(x64), np.abs(cs) * np.where(np.arange(cs.shape[-1]) % 2, -1.0, 1.0), half)
    size = np.maximum(np.abs(size), np.abs(ref)) + np.abs(x64).max()
    assert (np.abs(bf16_value(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * size).all()


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("rows,heads,P", [(1, 1, 8), (1, 128, 64), (37, 16, 64), (5, 3, 24),
                                          (300, 20, 32), (7, 130, 256), (2, 1000, 16),
                                          (64, 1, 48), (2, 33, 104)])
def test_packed(rows, heads, P, half):
    import paged_kv_mla_gb300 as pkm
    x, pos, freqs = problem(rows + heads + P, rows, heads, P, 777)
    y = torch.full((rows, heads, P), FILL, dtype=torch.int16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkm.mla_rope_heads(dev(x), dev(pos), torch.from_numpy(freqs).cuda(), y, half=half,
                       dev_status=status)
    assert status.item() == 0
    assert_rotated(y.cpu().numpy().view(np.uint16), x, pos, freqs, half)


@pytest.mark.parametrize("half", [False, True])
def test_strided_into_a_wider_row(half):
    """The last columns of [rows, heads, 128 + P] into the last of [rows, heads, 512 + P];
    the other columns stay."""
    import paged_kv_mla_gb300 as pkm
    rows, heads, P = 19, 12, 64
    x, pos, freqs = problem(1, rows, heads, P, 500)
    q = torch.zeros(rows, heads, 128 + P, dtype=torch.int16, device="cuda")
    q[..., 128:] = dev(x)
    y = torch.full((rows, heads, 512 + P), FILL, dtype=torch.int16, device="cuda")
    pkm.mla_rope_heads(q[..., 128:], dev(pos), torch.from_numpy(freqs).cuda(), y[..., 512:], half=half)
    out = y.cpu().numpy().view(np.uint16)
    assert (out[..., :512] == FILL).all()
    assert_rotated(out[..., 512:], x, pos, freqs, half)


@pytest.mark.parametrize("half", [False, True])
def test_in_place_heads_first_and_broadcast(half):
    import paged_kv_mla_gb300 as pkm
    rows, heads, P = 23, 6, 40
    x, pos, freqs = problem(2, rows, heads, P, 90)
    f, p = torch.from_numpy(freqs).cuda(), dev(pos)
    t = dev(x)
    pkm.mla_rope_heads(t, p, f, t, half=half)
    assert_rotated(t.cpu().numpy().view(np.uint16), x, pos, freqs, half)
    hf = torch.full((heads, rows, P), FILL, dtype=torch.int16, device="cuda")
    pkm.mla_rope_heads(dev(x), p, f, hf.transpose(0, 1), half=half)
    assert_rotated(hf.transpose(0, 1).cpu().numpy().view(np.uint16), x, pos, freqs, half)
    one = dev(x[:, :1]).expand(rows, heads, P)
    y = torch.empty(rows, heads, P, dtype=torch.int16, device="cuda")
    pkm.mla_rope_heads(one, p, f, y, half=half)
    assert_rotated(y.cpu().numpy().view(np.uint16), np.broadcast_to(x[:, :1], x.shape), pos, freqs, half)


def test_position_out_of_range_leaves_its_row():
    import paged_kv_mla_gb300 as pkm
    x, pos, freqs = problem(3, 9, 4, 32, 60)
    pos[[2, 7]] = [60, 0xFFFFFFFF]
    y = torch.full((9, 4, 32), FILL, dtype=torch.int16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkm.mla_rope_heads(dev(x), dev(pos), torch.from_numpy(freqs).cuda(), y, dev_status=status)
    assert status.item() == 4
    out = y.cpu().numpy().view(np.uint16)
    keep = [r for r in range(9) if r not in (2, 7)]
    assert (out[[2, 7]] == FILL).all()
    assert_rotated(out[keep], x[keep], pos[keep], freqs, False)


def test_captured_and_replayed_on_another_stream():
    import paged_kv_mla_gb300 as pkm
    x, pos, freqs = problem(4, 50, 16, 64, 200)
    t, p, f = dev(x), dev(pos), torch.from_numpy(freqs).cuda()
    y = torch.zeros(50, 16, 64, dtype=torch.int16, device="cuda")
    pkm.mla_rope_heads(t, p, f, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkm.mla_rope_heads(t, p, f, y)
    x2, pos2, _ = problem(5, 50, 16, 64, 200)
    t.copy_(dev(x2))
    p.copy_(dev(pos2))
    graph.replay()
    torch.cuda.synchronize()
    assert_rotated(y.cpu().numpy().view(np.uint16), x2, pos2, freqs, False)
