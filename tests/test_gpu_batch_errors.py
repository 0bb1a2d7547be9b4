"""A launch that the runtime refuses is that call's error alone: the next calls do not report it."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
# The refused launch is one on a stream whose capture has been invalidated (by a synchronize during it): the runtime
# refuses that on the host.  In a process of its own, which ends with it.
CHILD = """
import sys
sys.path[:0] = [{here!r}, {root!r}]
import ctypes, glob, os
import torch
from host_streamed_paged_gb300 import kvs
from test_gpu_q4 import Filled

f = Filled([200, 90], 2, 64, 64, seed=1, spare=8)
q = torch.randn(2, 1, 4, 64, device="cuda")
p = torch.randn(100, 4, 64, device="cuda").half()
cu = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
w = torch.rand(2, 2, 256, device="cuda")
dst = torch.from_numpy(f.free[:4].reshape(2, 2).astype("int32").copy()).cuda()
want = f.cache.attend(f.table_t, f.lens_t, q), kvs.prompt_attend(p, p[:, :2], p[:, 2:], cu)
torch.cuda.synchronize()
names = sorted({{line.split()[-1] for line in open("/proc/self/maps") if "libcudart" in line}})
rt = ctypes.CDLL(names[0])
s = ctypes.c_void_p()
k = torch.zeros(1, 2, 64, device="cuda")
assert rt.cudaStreamCreateWithFlags(ctypes.byref(s), 1) == 0
def refused():
    assert rt.cudaStreamBeginCapture(s, 2) == 0
    assert rt.cudaStreamSynchronize(s) != 0
    rt.cudaGetLastError()  # (torch's runtime, which the library does not share)
    try:
        kvs.kvs_q4_append(f.cache.pool, f.lens_t.data_ptr() // 8 * 8, 1, k.data_ptr(), k.data_ptr(), kvs.KVS_F32, 128, 128, s.value)
        raise SystemExit("the launch was not refused")
    except kvs.KVSError as e:
        assert e.status == kvs.KVS_ERR_CUDA, e
    g = ctypes.c_void_p()
    rt.cudaStreamEndCapture(s, ctypes.byref(g))
    rt.cudaGetLastError()
refused()
kept, lens, _ = f.cache.evict(f.table_t, dst, f.lens_t, w, 100)
assert lens.tolist() == [100, 90]
refused()
out, lse = kvs.prompt_attend(p, p[:, :2], p[:, 2:], cu)
assert torch.equal(out, want[1][0]) and torch.equal(lse, want[1][1])
refused()
out, lse = f.cache.attend(f.table_t, f.lens_t, q)
assert torch.equal(out, want[0][0])
torch.cuda.synchronize()
print("done")
"""


def test_a_refused_launch_is_not_reported_by_the_next_calls():
    code = CHILD.format(here=HERE, root=os.path.dirname(HERE))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "done" in r.stdout, (r.stdout[-500:], r.stderr[-1500:])
