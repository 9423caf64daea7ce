"""The weights' gradients of the head norm, held to the additions that the kernels make."""
import numpy as np
import pytest
import torch

import paged_reference as ref
import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda
from test_gpu_qk_norm_rope import CASES, IDS, make

pytestmark = pytest.mark.gpu

# ... and with several items a group of lanes, up to hundreds of heads
LONG = [(5000, 16, 4, 128, 128, False, None, torch.bfloat16), (9001, 8, 8, 64, 64, True, None, torch.float32),
        (700, 258, 2, 64, 32, False, None, torch.bfloat16)]


def up(a, b):
    return -(-a // b)


def depth(T, Hq, Hkv, d, dtype):
    """Roundings on a term's way into the sum.  A term itself: below 32.  A group of lanes goes through a run of
    items, up to two heads of one token each; a block sums its groups, 32 threads the blocks' rows, one those 32."""
    lanes = d * (2 if dtype == torch.bfloat16 else 4) // 16
    groups = 256 // lanes
    items = T * (up(Hq, 2) + up(Hkv, 2))
    blocks = min(up(items, groups), 304)
    return 32 + 2 * up(items, blocks * groups) + groups + up(blocks, 32) + 32


@pytest.mark.parametrize("case", CASES + LONG, ids=IDS + ["long0", "long1", "long2"])
def test_weight_gradients(case):
    need_cuda()
    T, Hq, Hkv, d, rot, inter, sections, dt = case
    q, k, v, wq, wk, pos, table = make(case, seed=6, max_pos=10000)
    g = torch.Generator().manual_seed(4)
    gq, gk = torch.randn(T, Hq, d, generator=g).to(dt).cuda(), torch.randn(T, Hkv, d, generator=g).to(dt).cuda()
    got = rsa.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, pos, table, eps=1e-5, interleaved=inter, sections=sections)
    torch.cuda.synchronize()
    rsa.check_device_error()
    t = None if table is None else ref.to64(table)
    for name, dy, x, w, dw in (("q", gq, q, wq, got[2]), ("k", gk, k, wk, got[3])):
        _, want, _, size = ref.norm_rope_bwd(ref.to64(dy), ref.to64(x), ref.to64(w), pos.cpu().numpy(), t, 1e-5, inter, sections)
        worst = (np.abs(ref.to64(dw) - want) / (depth(T, Hq, Hkv, d, dt) * ref.U32 * size)).max()
        assert worst <= 1, f"dw of {name} is {worst:.3g} times its bound off"
