"""First calls of the tree attention from several threads of a new process at
once, every type and width among them."""

import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytestmark = pytest.mark.skip("needs a GPU")
else:
    pytestmark = pytest.mark.gpu

import __graft_entry__  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCRIPT = """
import threading, torch
import speculative_decoding_verification_decode_gb300 as sv
dev = torch.device("cuda", 0)
g = torch.Generator().manual_seed(0)
def inputs(dtype, D):
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).to(dev)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    return dict(q=r(12, 8, D), k=r(12, 2, D), v=r(12, 2, D), k_cache=r(30, 16, 2, D), v_cache=r(30, 16, 2, D),
                table=i([list(range(b, 30, 4))[:7] for b in range(4)]), lengths=i([100, 5, 0, 77]), n=3)
args = [inputs(dtype, D) for dtype in (torch.bfloat16, torch.float16) for D in (64, 128)]
torch.cuda.synchronize()
T, got, gate = 12, {}, threading.Barrier(12)
def work(t):
    with torch.cuda.stream(torch.cuda.Stream()):
        gate.wait()
        got[t] = sv.tree_attention(**args[t % 4])
        torch.cuda.current_stream().synchronize()
threads = [threading.Thread(target=work, args=(t,)) for t in range(T)]
[t.start() for t in threads]
[t.join() for t in threads]
assert len(got) == T
for t in range(T):
    want = sv.tree_attention(**args[t % 4])
    assert torch.equal(got[t].out, want.out) and torch.equal(got[t].lse, want.lse) and not got[t].status.any(), t
    assert want.out.float().abs().sum() > 0
"""


def test_first_calls_at_once():
    __graft_entry__.build()
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, env={**os.environ, "PYTHONPATH": ROOT}, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
