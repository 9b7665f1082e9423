"""The bounds-check build on the dense products and the distillation loss: odd and
ragged shapes of every kernel, forward and backward; lq_check_device must report no
index out of range.  The library is loaded in a child process (one CUDA library
per process)."""
import os
import subprocess
import sys

import pytest

from bit_ptq_looped_b200 import build as B

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
sys.path.insert(0, ROOT)
import torch
from bit_ptq_looped_b200 import lq
lq.lib()
assert any('liblq_bounds.so' in l for l in open('/proc/self/maps')), 'bounds build not mapped'
r = lambda *s: torch.randn(s, device='cuda').to(torch.bfloat16)
for M, N, K in ((1, 1, 8), (3, 70, 264), (7, 65, 72), (16, 1000, 264), (17, 64, 64), (129, 257, 200),
                (300, 1001, 520), (1000, 264, 1024), (2300, 195, 72), (8192, 100, 136),
                (33, 5632, 264), (20, 195, 2048), (129, 1003, 2056), (100, 1040, 264)):
    x, w, w2, b, y, z, u = r(M, K), r(N, K), r(N, K), r(N), r(M, N), r(M, N), r(M, N)
    lq.lq_dense_linear(x, w, b, act=2, residual=y, want_z=True)
    lq.lq_gated_linear(x, w, w2, b, b, want_gu=True)
    for g in (torch.bfloat16, torch.float32):
        lq.lq_dense_linear_bwd(y, x, w, z, act=3, want_db=True, g_dtype=g)
        lq.lq_dense_linear_bwd(y, x, w, want_db=True, g_dtype=g)
        lq.lq_gated_linear_bwd(y, z, u, x, w, w2, want_db=True, g_dtype=g)
for M, V, k in ((1, 1, 1), (5, 31, 3), (130, 515, 9), (3, 50001, 700), (300, 20011, 50)):
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        l = torch.randn(M, V, device='cuda') * 3
        tv, ti = torch.topk(l, k, dim=1)
        lq.lq_distill_loss(l.to(dt), tv, ti, want_grad=True)
        lq.lq_distill_loss(l.to(dt), tv, ti, t_lse=torch.logsumexp(l, 1), want_grad=True)
torch.cuda.synchronize()
lq.lq_check_device()
print('bounds build: no index out of range')
""".replace("ROOT", repr(ROOT))


def test_dense_kernels_stay_in_range_under_the_bounds_check_build():
    lib = B.build_bounds_checked()
    env = dict(os.environ, LQ_LIB_PATH=lib)
    r = subprocess.run([sys.executable, "-c", CHILD], env=env, capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    assert "no index out of range" in r.stdout
