"""The 8-bit block's magnitudes belong to the weight that its product computes
with: wnorm and g against the fp64 norm of codes * scale + s B A.

The norm's tolerance is the acceptance bar of fp32 operands, 1e-4.  That of the
unquantised weight is off by more: a code's error of up to half a step, some
0.9% of a normal row's rms in the mean square, moves a norm over 512 columns by
about 0.009 / sqrt(512) = 4e-4, and more in the worst of 1024 rows.
"""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

from parity_utils import NORM_RTOL, check_rel, host64

pytestmark = pytest.mark.gpu


def test_the_blocks_norm_is_that_of_its_8_bit_weight():
    print("[example] norm of the 8-bit weight", file=sys.stderr, flush=True)
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "eight_bit_block.py")
    spec = importlib.util.spec_from_file_location("eight_bit_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    block = mod.Block(512, 1024, 8, torch.device("cuda:0"))
    torch.cuda.synchronize()
    W8 = host64(block.up_q) * host64(block.up_s)[:, None]
    W = W8 + block.up.spec.s * (host64(block.up.B) @ host64(block.up.A))
    wnorm = np.sqrt(np.sum(W * W, axis=1))
    check_rel(host64(block.up_wnorm), wnorm, NORM_RTOL[torch.float32], "wnorm")
    check_rel(host64(block.up_g), host64(block.up.m) / wnorm, NORM_RTOL[torch.float32], "g")
