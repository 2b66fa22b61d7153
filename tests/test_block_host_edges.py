"""Host-side tests of the operators around the scan at the ends of what a call
can be given: nothing here touches CUDA."""
import os
import subprocess
import sys

import torch

import test_block_host as H
from selective_state_space_25_b200 import ssmscan as S

# sizes far beyond any memory; the library only counts
WIDE = """
from selective_state_space_25_b200 import ssmscan as S
import torch

import test_block_host as H
L = S.lib()
for d in [2 ** k + e for k in range(30, 57) for e in (-1, 0, 1)]:
    for K in (1, 4, 8):
        n = L.ssm_conv1d_bwd_workspace_bytes(1, 1, d, K)
        assert n == H.NONE or n % ((K + 1) * d * 4) == 0, (d, K, n)
    for n, m in ((L.ssm_gated_scan_bwd_workspace_bytes(1, 1, d), 12 * d),
                 (L.ssm_gated_norm_bwd_workspace_bytes(1, d, 1), 4 * d),
                 (L.ssm_add_norm_bwd_workspace_bytes(1, d), 12 * d),
                 (L.ssm_gated_scan_states_bytes(1, 33, d), 8 * d)):
        assert n == H.NONE or n % m == 0, (d, n)
d = 2 ** 40  # 2^40 channels in 2^35 groups of 32
big = dict(b=1, d=d)
assert H.conv_bwd(**big, L=1, x_ld=d, dy_ld=d, dx_ld=d) == H.INV, S.last_error()
assert H.conv_bwd(**big, L=1, x=None) == H.INV, S.last_error()
assert H.conv_fwd(**big, L=0, x=None, y=None, cs=None, cso=H.at(20), bias=None, start=None, K=1,
                  w=2 ** 44) == H.UNS, S.last_error()
print("counted")
"""


def test_sizes_beyond_any_memory_are_counted_or_refused():
    """In a process of its own: a signal there ends that one only."""
    r = subprocess.run([sys.executable, "-c", WIDE], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, PYTHONPATH=":".join(sys.path)))
    assert r.returncode == 0 and "counted" in r.stdout, (r.returncode, r.stderr[-2000:])


def test_conv1d_of_an_empty_sequence_needs_its_weight():
    """With a window to write there is a launch, which takes the weight."""
    assert H.conv_fwd(L=0, w=None, x=None, y=None) == H.INV and "weight" in S.last_error()
    assert H.conv_fwd(L=0, w=None, x=None, y=None, cso=None) == H.OK
    assert H.conv_fwd(L=0, b=0, w=None, x=None, y=None) == H.OK


def test_binding_leaves_sizes_without_a_workspace_to_the_call(monkeypatch):
    """(size_t)-1, the library's answer for sizes that it refuses, is no number of
    bytes to allocate: the call goes on without a workspace, to the refusal."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)

    class Pool:
        device = torch.device("cuda", 0)

        def new(self, ref, shape, dtype):
            return torch.empty(shape, dtype=dtype)

    assert S._workspace(None, lambda: H.NONE, Pool(), None)[1:] == (None, 0)
    ws, ptr, n = S._workspace(None, lambda: 96, Pool(), None)
    assert ws.numel() == n == 96 and ptr == ws.data_ptr()
