"""The backward, again and again on the same inputs, beside other work: the same
bits each time."""
import pytest
import torch

from tests import gpu_helpers as gh
from trained_kv_prefix_gb300 import cartattn as ca
from trained_kv_prefix_gb300 import synth

pytestmark = pytest.mark.gpu

CASES = [
    # id, B, n, Hq, Hkv, d, p, dtype, window: from three steps a key tile to many
    ("f32_d64", 1, 130, 4, 2, 64, 64, "f32", 0),
    ("few_steps", 1, 257, 4, 1, 64, 129, "bf16", 0),
    ("d128", 2, 300, 8, 2, 128, 200, "bf16", 0),
    ("window", 2, 260, 8, 2, 64, 150, "bf16", 96),
    ("many_steps", 6, 700, 16, 2, 128, 300, "bf16", 0),
]


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_bwd_repeats_bit_for_bit(case):
    name, B, n, Hq, Hkv, d, p, dt, window = case
    s = synth.TrainShape(name, B=B, n=n, Hq=Hq, Hkv=Hkv, d=d, p=p, dtype=dt, seed=161, qkv_std=0.5,
                         do_std=1.0)
    g = gh.to_gpu(synth.train_inputs(s))
    o, lse = ca.cart_attn_fwd(g["q"], g["k"], g["v"], g["kc"], g["vc"], theta=s.theta, window=window)
    x = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    y, side = torch.empty_like(x), torch.cuda.Stream()
    torch.cuda.synchronize()
    first = None
    for turn in range(60):
        if turn % 2:                                # copies beside every other one
            with torch.cuda.stream(side):
                for _ in range(4):
                    y.copy_(x)
        got = ca.cart_attn_bwd(g["q"], g["k"], g["v"], g["kc"], g["vc"], o, lse, g["do"],
                               theta=s.theta, window=window)
        first = first or [z.clone() for z in got]
        for nme, u, v in zip(("dq", "dk", "dv", "dkc", "dvc"), first, got):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8)), (nme, turn)
    assert ca.device_status(clear=True) == 0
