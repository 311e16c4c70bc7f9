"""The encode of a plan's sorted rows: rows past the rows in use are not read."""
import numpy as np
import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq
import fp4_reference as ref
from test_gpu_fp4 import read_operand, values_like

pytestmark = pytest.mark.gpu


def best_us(call, reps=7):
    """The least time of a call by events on its stream, the call before it waited for."""
    best = float("inf")
    for _ in range(reps):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


@pytest.mark.parametrize("pad", [0, 1])
def test_rows_past_the_rows_in_use_cost_nothing(pad):
    """200,000 rows of 4096 bf16 are 1.6 GB: some 300 us to read. With one of them in use the call is a launch; a quarter of
    the whole call's time lies far from both. Rows of either alignment (an odd stride takes another load)."""
    tokens, K, E = 200_000, 4096, 4
    buf = torch.empty(tokens * (K + pad), dtype=torch.bfloat16, device="cuda").normal_()
    x = torch.as_strided(buf, (tokens, K), (K + pad, 1))
    ids = torch.zeros(tokens, 1, dtype=torch.int32, device="cuda")
    every = pnq.expert_sort(ids, E)
    ids.fill_(-1)
    ids[tokens // 2] = 2
    one = pnq.expert_sort(ids, E)
    q = pnq.fp4_quantize(pnq.NVFP4, x, plan=every, sorted=True)
    whole = best_us(lambda: pnq.fp4_quantize(pnq.NVFP4, x, plan=every, sorted=True, out=q))
    single = best_us(lambda: pnq.fp4_quantize(pnq.NVFP4, x, plan=one, sorted=True, out=q))
    assert whole > 100 and single < whole / 4, (whole, single)


@pytest.mark.parametrize("kind", [pnq.NVFP4, pnq.MXFP4])
@pytest.mark.parametrize("tokens,slots,used", [(40, 2, 0), (40, 2, 1), (40, 2, 79), (3000, 3, 0), (3000, 3, 2), (3000, 3, 4999)])
def test_rows_in_use_are_encoded_and_no_others(kind, tokens, slots, used):
    """No row, one, or all but a few in use, few rows and many: what the buffers held past them stays."""
    K, E, n = 160, 7, tokens * slots
    ids = np.full(n, -1, np.int32)
    ids[np.random.default_rng(used).permutation(n)[:used]] = np.arange(used) % E
    plan = pnq.expert_sort(torch.from_numpy(ids.reshape(tokens, slots)).cuda(), E)
    x = values_like(max(used, 1), K, seed=used)[:used]
    xs = np.full((n, K), np.nan, np.float32)
    xs[:used] = x
    pitch, size = pnq.fp4_layout(kind, n, K, 1, E)
    codes = torch.full((n, pitch), 0xA5, dtype=torch.uint8, device="cuda")
    m = pnq.Fp4Matrix(kind, n, K, codes, torch.zeros(size, dtype=torch.uint8, device="cuda"), plan=plan)
    pnq.fp4_quantize(kind, torch.from_numpy(xs).cuda(), 1.0, plan=plan, sorted=True, out=m)
    got, words = read_operand(m, np.maximum(ref.plan(ids, E)[4], 0))
    want_codes, want_words = ref.quantize(x, kind, 1.0) if used else (got[:0], words[:0])
    assert np.array_equal(got[:used], want_codes) and np.array_equal(words[:used], want_words)
    assert bool((codes[used:] == 0xA5).all())
