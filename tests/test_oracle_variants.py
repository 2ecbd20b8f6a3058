"""A variant of the oracle with a mistake in its indices reads nothing but what it was given room for."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# in a process of its own: the down weights end where readable memory does
CHILD = r'''
import ctypes, mmap, sys
import numpy as np
from oracle import oracle as orc
from quantized_routed_expert_02_gb300 import synth
from tests.test_oracle_mutants import MUTANTS, SRC

before, after = MUTANTS["down_row_stride"]
src = sys.argv[1] + "/mutant.c"
open(src, "w").write(open(SRC).read().replace(before, after))
o = orc.Oracle(orc.load_variant(orc.build(force=True, src=src, out=sys.argv[1] + "/mutant.so")))
T, H, E, k, I = 3, 512, 4, 2, 256
shape = synth.custom_shape(T, H, E, k, I, cfg_id=5)
blobs = synth.expert_blobs(shape, 0)
down = blobs["down"].reshape(-1)
page = mmap.PAGESIZE
pages = -(-down.size // page)
room = mmap.mmap(-1, (pages + 1) * page)
held = np.frombuffer(room, dtype=np.uint8)
libc = ctypes.CDLL(None, use_errno=True)
assert libc.mprotect(ctypes.c_void_p(held.ctypes.data + pages * page), ctypes.c_size_t(page), 0) == 0
last = held[pages * page - down.size:pages * page]
last[:] = down
rng = np.random.default_rng(0)
x = rng.standard_normal((T, H)).astype(np.float32)
idx = np.array([[E - 1, 0]] * T, dtype=np.int32)
w = np.full((T, k), 0.5)
good = orc.Oracle().ffn(x, idx, w, blobs["gate"], blobs["up"], last, E, I)[0]
bad = o.ffn(x, idx, w, blobs["gate"], blobs["up"], last, E, I)[0]
assert np.isfinite(bad).all() and np.abs(good - bad).max() > 1e-3 * np.abs(good).max()
print("done")
sys.stdout.flush()
import os
os._exit(0)  # the guarded page stays as it is
'''


def test_a_row_stride_too_long_ends_no_process(tmp_path):
    r = subprocess.run([sys.executable, "-c", CHILD, str(tmp_path)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, (r.returncode, r.stderr[-2000:])
