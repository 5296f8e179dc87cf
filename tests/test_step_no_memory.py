"""A C entry that runs out of host memory says so: it neither throws nor leaves an earlier call's message."""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))

# 2^24 empty tensors: the call's own table of them does not fit what the process may still take
CHILD = """
import ctypes, resource, sys
sys.path[:0] = [%r, %r]
import bit_nf4_quantized_09_amd as nf4
import step_abi as abi
L = abi.library()
assert L.qlora_grad_norm(None, 1, 1.0, None, None, None, 0, None) == nf4.NF4_ERR_ARG
count = 1 << 24
tensors = (abi.Tensor * count)()
pages = int(open("/proc/self/statm").read().split()[0])
resource.setrlimit(resource.RLIMIT_AS, (pages * resource.getpagesize() + (64 << 20),) * 2)
status = L.qlora_grad_norm(tensors, count, 1.0, 4096, None, 8192, 1 << 30, None)
print(status, L.nf4_last_error().decode())
""" % (os.path.dirname(HERE), HERE)


def test_out_of_host_memory_says_so():
    done = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
    assert done.stdout.strip() == "4 out of memory"
