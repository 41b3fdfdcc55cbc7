"""Attention over the paged cache at values that a long context brings: weights far below the largest over
E4M3 caches."""
import math

import pytest
import torch

from shared_routed_expert_b200 import _lib, build
from tests.serve_util import Paged, attention_ref
from tests.test_gpu_tree_attn import run

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


# B sequences of n new tokens, n n_q / n_kv rows of a kv head: up to 16 and up to 32 (warp-level products), more (tiles)
TAILS = [(80, 1, 12, 4, 128, 700), (80, 2, 48, 4, 64, 700), (40, 4, 24, 2, 128, 1400), (40, 30, 24, 2, 64, 1400),
         (80, 2, 8, 2, 256, 700), (80, 5, 8, 2, 256, 700), (40, 12, 8, 2, 256, 1400)]


@pytest.mark.parametrize("bits", [25.3, 23.5, 20.0])
@pytest.mark.parametrize("B,n,n_q,n_kv,d,ctx", TAILS)
def test_small_weights_over_e4m3_caches_count(B, n, n_q, n_kv, d, ctx, bits):
    """One key whose value is 0 outweighs each of the others by 2^bits; theirs are 1, so that the result is
    the others' share. Error allowed: a weight is rounded to fp16 beside a largest one of 2^7 or more, where
    its smallest step is 2^-24: 2^-25 2^-7 of the largest at most, for each key; and what attention_ref
    allows. As many items as blocks, so that few are cut."""
    P = Paged([n] * B, [ctx] * B, n_kv, d, 64, "e4m3", seed=40, k_scale=1.0, v_scale=1.0)
    one = 0x38                                              # 1.0
    P.k.fill_(0)
    P.v.fill_(one)
    for b in range(B):
        pg, sl = P.slots(b, 1)
        P.k[pg, :, sl] = one
        P.v[pg, :, sl] = 0
    q = torch.ones(P.T, n_q * d, dtype=torch.bfloat16, device=DEV)
    scale = bits * math.log(2) / d
    out, lse, st = run(P, q, n_q, scale=scale)
    assert st == _lib.MOE_OK
    ref, rl, to, tl = attention_ref(P, q, n_q, scale=scale)
    assert float(ref.max()) < 0.01 and float(ref.min()) > 0
    keys = ctx + n
    assert float(((out.view(P.T, n_q, d).double() - ref).abs() - to).max()) <= keys * 2.0 ** -32
    assert float(((lse.double() - rl).abs() - tl).max()) <= 0
