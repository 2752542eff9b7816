"""Launches of the block codes at the largest sizes, without a GPU: the HIP calls
that the library makes go to a recorder, which notes each launch and runs
nothing. A dimension of a grid has to stay below 2^32 work items, and the
launches of one call together have to cover its work."""
import os
import subprocess
import sys

import pytest

import mini_means_amd as mm

RECORDER = r"""
#include <hip/hip_runtime_api.h>
#include <stdio.h>
#include <string.h>
static struct { const void* stub; char name[512]; } known[4096];
static int count;
static dim3 grid, block;
static size_t shared;
static hipStream_t stream;
void __hipRegisterFunction(void** m, const void* stub, char* d, const char* name, unsigned l,
                           void* t, void* b, void* bd, void* gd, int* w) {
  known[count].stub = stub;
  strncpy(known[count++].name, name, 511);
}
hipError_t __hipPushCallConfiguration(dim3 g, dim3 b, size_t s, hipStream_t st) {
  grid = g, block = b, shared = s, stream = st;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* g, dim3* b, size_t* s, hipStream_t* st) {
  *g = grid, *b = block, *s = shared, *st = stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 g, dim3 b, void** args, size_t s, hipStream_t st) {
  const char* name = "?";
  for (int i = 0; i < count; ++i)
    if (known[i].stub == f) name = known[i].name;
  printf("launch %s %u %u %u %u\n", name, g.x, g.y, g.z, b.x);
  return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipPointerGetAttributes(hipPointerAttribute_t* a, const void* p) {
  memset(a, 0, sizeof *a);
  a->type = hipMemoryTypeDevice;
  return hipSuccess;
}
hipError_t hipMallocAsync(void** p, size_t n, hipStream_t s) { *p = (void*)4096; return hipSuccess; }
hipError_t hipFreeAsync(void* p, hipStream_t s) { return hipSuccess; }
"""


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    if not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("no HIP headers")
    if not os.path.exists(mm.LIB_PATH):
        from mini_means_amd import build
        build.build(verbose=False)
    room = tmp_path_factory.mktemp("recorder")
    source, lib = room / "recorder.c", room / "recorder.so"
    source.write_text(RECORDER)
    subprocess.check_call(["gcc", "-shared", "-fPIC", "-w", "-D__HIP_PLATFORM_AMD__",
                           "-I/opt/rocm/include", str(source), "-o", str(lib)])
    root = os.path.dirname(os.path.dirname(os.path.abspath(mm.__file__)))

    def run(call):
        """(kernel, grid, workgroup) of each launch of one call of the C ABI."""
        program = (f"import ctypes, sys; sys.path.insert(0, {root!r})\n"
                   f"ctypes.CDLL({str(lib)!r}, mode=ctypes.RTLD_GLOBAL)\n"
                   f"import mini_means_amd as mm\nL, P = mm.lib(), 4096\n"
                   f"rc = {call}\nassert rc == 0, (rc, L.emeans_last_error())\n")
        text = subprocess.run([sys.executable, "-c", program], check=True, capture_output=True,
                              text=True).stdout
        found = []
        for line in text.splitlines():
            if line.startswith("launch "):
                name, *n = line.split()[1:]
                found.append((name, tuple(int(v) for v in n[:3]), int(n[3])))
        return found

    return run


# the call, the kernel, how many workgroups cover it
N = 2 ** 31 - 1
LONG = 2 ** 31 - 1024
CALLS = [
    # rows of 8 bf16 values; 32 blocks of 128 per workgroup
    (f"L.emeans_block_encode(P, 1, {N}, 8, 8, 0, P, 16, P, 4, None, 0, None, 0, None)",
     "encode_rows_kernel", -(-N // 32)),
    # rows of 2048 values in blocks of 16, 256 of them per workgroup, by slot
    (f"L.emeans_cache_write(P, 1, {2 ** 26}, 1, 2048, 2048, 2048, P, 8, P, P, {2 ** 26}, 16, 3, None)",
     "encode_rows_kernel", 2 ** 26 * 128 // 256),
    # two long fp32 rows, transposed too
    (f"L.emeans_block_encode(P, 0, 2, {LONG}, {LONG}, 0, P, {LONG}, P, {LONG}, P, 2, P, 1, None)",
     "encode_tile_kernel", -(-LONG // 128)),
    (f"L.emeans_block_encode(P, 0, 2, {LONG}, {LONG}, 1, P, {LONG}, P, {LONG}, P, 2, P, 1, None)",
     "encode_tile_kernel", -(-LONG // 128)),
    # 64 rows per workgroup, to bf16
    (f"L.emeans_cache_read(P, P, 100, 32, 32, 2, P, 4, {N}, P, 1, 32, None)",
     "decode_rows_kernel", -(-N // 64)),
    (f"L.emeans_cache_read_pages(P, P, 10, 10, 32, 32, 2, P, 4, 4, P, 2, {N}, P, 1, 32, None)",
     "decode_rows_kernel", -(-N // 64)),
    # one row against all: 64 rows of B per workgroup at two k-steps, 16 at eight or more
    (f"L.emeans_block_matmul(P, 256, P, 2, P, 256, P, 2, 0, 1, {N}, 256, P, 0, {N}, None, None)",
     "product_few_kernel", -(-N // 64)),
    (f"L.emeans_block_matmul(P, 1024, P, 8, P, 1024, P, 8, 1, 2, {2 ** 28}, 1024, P, 1, {2 ** 28}, "
     "None, None)", "product_few_kernel", 2 ** 28 // 16),
    (f"L.emeans_block_linear(P, 1, 128, P, 128, P, 1, 1, 1, {N}, 128, P, 1, {N}, None, None)",
     "product_few_kernel", -(-N // 128)),
    # 64 x 64 tiles at any pitch; 128 x 128 and 256 x 256 tiles; the same with long A
    (f"L.emeans_block_matmul(P, 17, P, 1, P, 17, P, 1, 1, 40, {N}, 17, P, 1, {N}, None, None)",
     "product_any_kernel", -(-N // 64)),
    (f"L.emeans_block_matmul(P, 17, P, 1, P, 17, P, 1, 1, {2 ** 18}, {2 ** 18}, 17, P, 1, {2 ** 18}, "
     "None, None)", "product_any_kernel", 2 ** 24),
    (f"L.emeans_block_matmul(P, 128, P, 1, P, 128, P, 1, 0, 17, {N}, 128, P, 0, {N}, None, None)",
     "product_tile_kernel", -(-N // 128)),
    (f"L.emeans_block_matmul(P, 128, P, 1, P, 128, P, 1, 0, {N}, 70, 128, P, 1, 70, None, None)",
     "product_tile_kernel", -(-N // 256)),
]


@pytest.mark.parametrize("call,kernel,groups", CALLS)
def test_no_launch_reaches_two_to_the_32(launches, call, kernel, groups):
    found = launches(call)
    assert found
    for name, grid, wg in found:
        for g, w in zip(grid, (wg, 1, 1)):
            assert g * w < 2 ** 32, (name, grid, wg)
    assert sum(g[0] * g[1] * g[2] for name, g, _ in found if kernel in name) >= groups, found


def test_common_sizes_are_one_launch(launches):
    for call in ("L.emeans_block_matmul(P, 128, P, 1, P, 128, P, 1, 0, 8192, 8192, 128, P, 0, 8192, "
                 "None, None)",
                 "L.emeans_block_encode(P, 1, 65536, 4096, 4096, 0, P, 4096, P, 32, None, 0, None, "
                 "0, None)",
                 "L.emeans_cache_read(P, P, 100, 768, 128, 3, P, 4, 1000000, P, 0, 768, None)"):
        assert len(launches(call)) == 1
