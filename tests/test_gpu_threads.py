"""The first calls of a process made by several threads at once, each on a stream of
its own: what the first call of a device sets up is there for all of them."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = r"""
import threading
import torch
import int4_gemm_gb300 as q4

N = 6
g = torch.Generator("cuda").manual_seed(3)
x, dy = (torch.randn((2500, 1040), device="cuda", generator=g).bfloat16() for _ in range(2))
qa = torch.randint(-128, 128, (2500, 1040), dtype=torch.int8, device="cuda", generator=g)
qb = torch.randint(-128, 128, (9000, 1040), dtype=torch.int8, device="cuda", generator=g)
sa, sb = torch.rand(2500, device="cuda", generator=g), torch.rand(9000, device="cuda", generator=g)
rstd = torch.rsqrt(x.float().square().mean(1) + 1e-6)
logits = torch.randn((30000, 64), device="cuda", generator=g)
ids = torch.randint(0, 64, (30000, 4), dtype=torch.int32, device="cuda", generator=g)
streams = [torch.cuda.Stream() for _ in range(N)]
torch.cuda.synchronize()
gate, results, errors = threading.Barrier(N), [None] * N, []

def work(i):
    try:
        torch.cuda.set_device(0)
        gate.wait()
        with torch.cuda.stream(streams[i]):
            out = [q4.gemm_w8a8_int8(qa, sa, qb, sb), q4.gemm_w8a8_int8(qa[:9].contiguous(), sa[:9].contiguous(), qb, sb)]
            out += q4.rms_norm_int8(x)[:2]
            out += q4.rms_norm_backward(dy, x, rstd)
            out += q4.quantize_int8(x)
            out += q4.moe_balance_loss(logits, ids)
        streams[i].synchronize()
        results[i] = out
    except BaseException as e:
        errors.append(e)

threads = [threading.Thread(target=work, args=(i,)) for i in range(N)]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert not errors, errors
for out in results[1:]:
    for a, b in zip(out, results[0]):
        assert torch.equal(a, b)
want = ((qa.double() @ qb.double().t()).float() * sa.unsqueeze(1) * sb).bfloat16()
assert torch.equal(results[0][0], want) and torch.equal(results[0][1], want[:9])
assert q4.sync_status() == 0
print("same")
"""


def test_first_calls_of_several_threads():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
