"""The release of shared pages where the device has no room for its cluster, by a fake of the runtime's
calls in a process of its own; and as the first call of a process, captured."""
import os
import shutil
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# No clusters fit, or the question itself fails; and a launch as a cluster of 16 is refused, as on
# such a device. What was asked and launched is counted in a file.
FAKE = r"""
#define _GNU_SOURCE
#include <cuda_runtime_api.h>
#include <dlfcn.h>
#include <stdio.h>
#include <stdlib.h>
static void note(const char* what) {
  FILE* f = fopen(getenv("FAKE_NOTES"), "a");
  if (f) fprintf(f, "%s\n", what), fclose(f);
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* c) {
  note("asked");
  *n = 0;
  return getenv("FAKE_ERROR") ? cudaErrorInvalidValue : cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) {
      note("cluster");
      return cudaErrorInvalidClusterSize;
    }
  cudaError_t (*next)(const cudaLaunchConfig_t*, const void*, void**) = dlsym(RTLD_NEXT, "cudaLaunchKernelExC");
  return next(c, f, args);
}
"""

RELEASES = """
import numpy as np
from tests.test_gpu_paged_share import Books
for r, page, longest in ((500, 16, 400), (12, 16, 60000), (4, 16, 50)):
    bk = Books(r, page, longest, r // 2, r)
    c = bk.cache()
    e, f = np.flatnonzero(bk.lens == 0), np.flatnonzero(bk.lens > 0)
    bk.fork(bk.rs.choice(f, len(e)), e)
    for part in (0, 1):
        bk.release(np.arange(r) % 2 == part)
        bk.check()
    assert bk.count == len(bk.free) and c.status() == 0
print("released")
"""

CAPTURED = """
import numpy as np
import torch
from tests.test_gpu_paged import ints
from tests.test_gpu_paged_share import Books
bk = Books(300, 16, 400, 3, 2)
c, d = bk.cache(), bk.d
done = ints(np.arange(300) % 3 == 0)
keep = {k: v.clone() for k, v in d.items()}
gr = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(gr):
    c.release(done, d["lens"], d["table"], d["free"], d["count"], shared=d["shared"])
bk.check()
for _ in range(2):
    for k, v in keep.items():
        d[k].copy_(v)
    gr.replay()
got = {k: v.clone() for k, v in d.items()}
for k, v in keep.items():
    d[k].copy_(v)
bk.release(done.cpu().numpy())
bk.check()
assert all(torch.equal(got[k], d[k]) for k in d) and c.status() == 0
print("released")
"""


def run(code, **env):
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=dict(os.environ, PYTHONPATH=ROOT, **env),
                       capture_output=True, text=True, timeout=240)
    assert p.returncode == 0 and p.stdout.strip().endswith("released"), p.stdout + p.stderr


@pytest.mark.parametrize("error", [False, True])
def test_large_releases_without_room_for_a_cluster(error, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc")))
    if not cc or not os.path.exists(os.path.join(cuda, "include", "cuda_runtime_api.h")):
        pytest.skip("no compiler for the fake")
    (tmp_path / "fake.c").write_text(FAKE)
    fake = str(tmp_path / "fake.so")
    subprocess.run([cc, "-shared", "-fPIC", "-I", os.path.join(cuda, "include"), "-o", fake, str(tmp_path / "fake.c"), "-ldl"],
                   check=True)
    notes = tmp_path / "notes"
    run(RELEASES, LD_PRELOAD=fake, FAKE_NOTES=str(notes), **({"FAKE_ERROR": "1"} if error else {}))
    assert notes.read_text().split() == ["asked"]  # once, and no cluster was launched


def test_the_first_call_of_a_process_may_be_captured():
    run(CAPTURED)
