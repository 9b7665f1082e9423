"""The bounds-check build where stores are cut short: last pieces of unaligned rows in
every epilogue, saved factors, gradients over slices and into float32, rows of weight
zero and rows without an entry, and the rest class far below the list."""
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
r = lambda *s: torch.randn(*s, device='cuda').to(torch.float16)
for M in (2, 5, 16, 17, 31, 127, 130, 260, 700):
    for N in (1, 7, 63, 65, 127, 129, 195, 257):
        for K in (8, 264, 2048):
            x, w, w2, b, y, z, u = r(M, K), r(N, K), r(N, K), r(N), r(M, N), r(M, N), r(M, N)
            lq.lq_dense_linear(x, w, b, act=1, residual=y, want_z=True)
            lq.lq_gated_linear(x, w, w2, b, b, want_gu=True)
            lq.lq_dense_linear_bwd(y, x, w, z, act=2, want_db=True)
            dw, db = torch.zeros(N, K, device='cuda'), torch.zeros(N, device='cuda')
            lq.lq_gated_linear_bwd(y, z, u, x, w, w2, dwg=dw, dwu=dw.clone(), dbg=db, dbu=db.clone(),
                                   want_db=True, accumulate=True)
x, w, y = r(8192, 512), r(512, 512), r(8192, 512)
lq.lq_dense_linear_bwd(y, x, w, want_db=True)
for M, V, k in ((3, 1, 1), (3, 9, 2), (9, 1003, 20), (3, 50001, 700), (600, 2051, 9)):
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        l = torch.randn(M, V, device='cuda')
        tv, ti = torch.topk(l, k, dim=1)
        z = l.to(dt)
        z.scatter_add_(1, ti, torch.full_like(tv, 300.0).to(dt))
        wt = torch.ones(M, device='cuda')
        wt[1] = 0
        ti[2] = -1
        for lse in (None, torch.logsumexp(l, 1)):
            lq.lq_distill_loss(z, tv, ti, t_lse=lse, weight=wt, want_grad=True)
            lq.lq_distill_loss(z, tv, ti, t_lse=lse, weight=wt, grad=z.clone())
torch.cuda.synchronize()
lq.lq_check_device()
print('bounds build: no index out of range')
""".replace("ROOT", repr(ROOT))


def test_cut_stores_stay_in_range_under_the_bounds_check_build():
    lib = B.build_bounds_checked()
    env = dict(os.environ, LQ_LIB_PATH=lib)
    r = subprocess.run([sys.executable, "-c", CHILD], env=env, capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    assert "no index out of range" in r.stdout
