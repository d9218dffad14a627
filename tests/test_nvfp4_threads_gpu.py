"""A process's first calls over caches held in 4 bits, from two threads at once, take
the same way as later ones: bit-equal results."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import threading, torch
import __graft_entry__
__graft_entry__.build()
import sparse_attention_indexer_logits_gb300 as pml

g = torch.Generator(device="cuda").manual_seed(3)
_, *parts = pml.pml_nvfp4_pages(64, 8, 128)
for p in parts:
    p.copy_(torch.randint(0x20, 0x50, p.shape, generator=g, device="cuda", dtype=torch.uint8))
table = torch.randperm(64, generator=g, device="cuda").int()[None]
lens = torch.tensor([4000], dtype=torch.int32, device="cuda")
q = torch.randn((1, 32, 128), generator=g, device="cuda", dtype=torch.bfloat16)
streams = [torch.cuda.Stream() for _ in range(2)]
torch.cuda.synchronize()
start, out = threading.Barrier(2), [[None] * 3 for _ in range(2)]

def calls(i):
    start.wait()
    for k in range(3):
        out[i][k] = pml.pml_paged_attention_nvfp4(q, *parts, table, lens, stream=streams[i])

threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
want = pml.pml_paged_attention_nvfp4(q, *parts, table, lens)
assert all(torch.equal(o, want) for mine in out for o in mine)
assert torch.isfinite(want).all() and pml.pml_device_status() == 0
print("same")
"""


def test_first_calls_from_two_threads():
    for _ in range(3):
        done = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=300)
        assert done.returncode == 0 and done.stdout.endswith("same\n"), done.stderr[-2000:]
