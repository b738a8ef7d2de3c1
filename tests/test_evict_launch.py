"""Launch errors of the two-kernel calls with token weights, on the host: the library runs over
a stand-in for the CUDA runtime whose n-th launch fails.  The running sums cannot be formed
again, so a call whose first kernel did not start must not start the one that adds to them."""
import subprocess
import sys
import textwrap

import pytest

import bit_rotated_kv_tq_b200 as tq

RUNTIME = r"""
#include <cuda_runtime_api.h>
int launches = 0, fail_at = -1;
static cudaError_t last = cudaSuccess;
static cudaError_t launch(void) {
    if (launches++ == fail_at) return last = cudaErrorLaunchOutOfResources;
    return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int d) { (void)a; (void)d; *v = 148; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) { (void)f; (void)a; (void)v; return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(struct cudaFuncAttributes* a, const void* f) { (void)f; a->numRegs = 128; return cudaSuccess; }
cudaError_t cudaLaunchKernel(const void* f, dim3 g, dim3 b, void** a, size_t m, cudaStream_t s) {
    (void)f; (void)g; (void)b; (void)a; (void)m; (void)s;
    return launch();
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** a) { (void)c; (void)f; (void)a; return launch(); }
cudaError_t cudaGetLastError(void) { cudaError_t e = last; last = cudaSuccess; return e; }
const char* cudaGetErrorName(cudaError_t e) { (void)e; return "name"; }
const char* cudaGetErrorString(cudaError_t e) { (void)e; return "text"; }
"""

# One call per process; prints its code and the launches it made.
CALLS = """
import ctypes, sys
C, P = ctypes, ctypes.c_void_p
rt = C.CDLL({runtime!r}, mode=C.RTLD_GLOBAL)
L = C.CDLL({lib!r})
class Cache(C.Structure):
    _fields_ = [("num_blocks", C.c_int32), ("num_kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("flags", C.c_int32), ("data", P)]
fail_at, call, d, flags = int(sys.argv[1]), sys.argv[2], int(sys.argv[3]), int(sys.argv[4])
C.c_int.in_dll(rt, "fail_at").value = fail_at
cache, at, big = Cache(64, 2, d, flags, 4096), P(4096), C.c_size_t(1 << 34)
if call == "decode":
    rc = L.tq_decode_attention_weights(at, C.byref(cache), None, at, 64, at, 1, 8, 1000, C.c_float(0.1), at, at,
                                       C.c_int64(1000), at, big, 0, None, None)
else:  # 2 tokens: contexts in parts; 5000: whole ones
    n = int(call)
    rc = L.tq_prefill_attention_weights(at, C.byref(cache), None, at, 64, at, at, 1, 8, n, n, C.c_float(0.1), at, 0, at,
                                        C.c_int64(1000), at, big, None, None)
print(rc, C.c_int.in_dll(rt, "launches").value)
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    from bit_rotated_kv_tq_b200 import build

    build.build()
    at = tmp_path_factory.mktemp("runtime")
    (at / "rt.c").write_text(RUNTIME)
    lib = at / "librt.so"
    subprocess.run(["gcc", "-shared", "-fPIC", "-I/usr/local/cuda/include", "-o", str(lib), str(at / "rt.c")], check=True)
    code = textwrap.dedent(CALLS).format(runtime=str(lib), lib=tq.LIB_PATH)

    def call(*args):
        p = subprocess.run([sys.executable, "-c", code, *map(str, args)], capture_output=True, text=True, timeout=60)
        assert p.returncode == 0, p.stderr
        return tuple(int(x) for x in p.stdout.split())

    return call


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("call,flags", [("decode", 0), ("decode", tq.TQ_CACHE_BF16), ("2", 0), ("5000", 0)])
def test_no_sums_behind_a_launch_that_failed(run, call, flags, d):
    assert run(-1, call, d, flags) == (tq.TQ_OK, 2)
    assert run(0, call, d, flags) == (tq.TQ_ERR_CUDA, 1)  # the attention did not start: nothing is added
    assert run(1, call, d, flags) == (tq.TQ_ERR_CUDA, 2)
