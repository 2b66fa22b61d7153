"""Seeded random configurations of the gated recurrence and the convolution
against their definitions in 64 bits, beside the chosen ones: sizes that take
every shape of the kernels (long sequences over few channels, many sequences,
one or several parts of a warp, clusters), strided and odd rows, packed
sequences, carried states.  Limits as in test_gpu_block.py."""
import random

import pytest
import torch

from test_gpu_block import BF, F32, conv_case, conv_check, gated_all, gated_case, gated_check, gated_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(36))
def test_gated_scan_random(ssm, seed):
    r = random.Random(seed)
    form = seed % 4
    if form == 0:    # few channels, a long sequence
        b, L, d = r.randint(1, 2), r.randint(600, 2600), r.choice([8, 16, 24, 40, 7])
    elif form == 1:  # many sequences
        b, L, d = r.randint(100, 330), r.randint(20, 140), r.choice([64, 72, 33])
    elif form == 2:  # many channels
        b, L, d = r.randint(1, 3), r.randint(30, 400), r.randint(500, 1500)
    else:
        b, L, d = r.randint(1, 9), r.randint(1, 300), r.randint(1, 300)
    if r.random() < 0.5:
        d = max(8, d // 8 * 8)
    kw = dict(gate=r.random() < 0.5, carry=r.random() < 0.5, packed=r.random() < 0.5,
              bias=r.random() < 0.7, view=r.random() < 0.4)
    c, dout, dh = gated_case(b, L, d, r.choice([F32, BF]), seed=seed, **kw)
    gated_check(gated_all(ssm, c, dout, dh), gated_ref(c, dout, dh), c, dout, dh)


@pytest.mark.parametrize("seed", range(24))
def test_conv1d_random(ssm, seed):
    r = random.Random(100 + seed)
    form = seed % 3
    if form == 0:
        b, L, d = r.randint(1, 2), r.randint(300, 1500), r.choice([8, 16, 33, 40])
    elif form == 1:
        b, L, d = r.randint(50, 200), r.randint(3, 60), r.choice([64, 72, 50])
    else:
        b, L, d = r.randint(1, 5), r.randint(1, 200), r.randint(1, 700)
    if r.random() < 0.5:
        d = max(4, d // 4 * 4)
    kw = dict(carry=r.random() < 0.5, packed=r.random() < 0.5, bias=r.random() < 0.7,
              view=r.random() < 0.4)
    conv_check(ssm, *conv_case(b, L, d, r.randint(1, 8), r.choice([F32, BF]), seed=seed, **kw),
               silu=r.random() < 0.8)


def test_calls_on_a_raw_stream_handle(ssm):
    """stream= as the integer handle of another stream."""
    c, dout, dh = gated_case(2, 70, 40, BF, seed=1)
    a = gated_all(ssm, c, dout, dh)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = gated_all(ssm, c, dout, dh, stream=s.cuda_stream)
    s.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]), k
