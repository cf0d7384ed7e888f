"""GPU: a Talker call that fails on the host leaves its streams as they were. The failure is made on the host: a library
loaded before the CUDA runtime answers one call with an error."""
import os
import shutil
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKE = r"""
#include <dlfcn.h>
#include <stddef.h>
int fail_next = 0;   /* the next graph cannot be made: out of memory */
int cudaGraphInstantiate(void **exec, void *graph, unsigned long long flags) {
    static int (*real)(void **, void *, unsigned long long) = NULL;
    if (fail_next) { fail_next = 0; *exec = NULL; return 2; }
    if (!real) {
        void *lib = dlopen("libcudart.so.13", RTLD_LAZY | RTLD_NOLOAD);
        *(void **)&real = lib ? dlsym(lib, "cudaGraphInstantiate") : NULL;
    }
    return real ? real(exec, graph, flags) : 999;
}
"""

PROGRAM = r"""
import ctypes, sys
import torch
from kv_cached_qwen3_gb300 import inputs
from kv_cached_qwen3_gb300.talker import Talker, TalkerError

fake = ctypes.CDLL(sys.argv[1])
fail = ctypes.c_int.in_dll(fake, "fail_next")
kv = sys.argv[2]
g = inputs.Geometry(**{**inputs.TALKER.__dict__, "n_layers": 2, "kv_dtype": kv})
w = inputs.make_weights(g, 31)
dtype = torch.bfloat16 if kv == "bf16" else torch.float32
tk, ref = Talker(g, w), Talker(g, w)
n = 150
def export(t, s):
    k = torch.empty(g.n_layers, g.n_kv_heads, t.cur_len(s), g.head_dim, device="cuda", dtype=dtype)
    v = torch.empty_like(k)
    t.kv_export(s, k, v, t.cur_len(s))
    return k, v
for t in (tk, ref):
    t.kv_init_batched(3, 300)
    torch.manual_seed(1)
    for s in range(3):
        t.kv_import(s, torch.randn(g.n_layers, g.n_kv_heads, n, g.head_dim, device="cuda").to(dtype),
                    torch.randn(g.n_layers, g.n_kv_heads, n, g.head_dim, device="cuda").to(dtype), n)
    t.kv_reorder(torch.tensor([0, 0, 1], dtype=torch.int32).cuda(), 1, 3)
rows = [export(tk, s) for s in range(3)]

def unchanged():
    for s in range(3):
        assert tk.cur_len(s) == n, (s, tk.cur_len(s))
        for a, b in zip(export(tk, s), rows[s]):
            assert torch.equal(a, b), s

def refused(call):
    fail.value = 1
    try:
        call()
    except TalkerError:
        pass
    else:
        raise AssertionError("the call did not fail")
    assert fail.value == 0
    unchanged()

emb = torch.randn(70, g.hidden, device="cuda")
refused(lambda: tk.prefill(1, emb))
refused(lambda: tk.prefill(0, emb[:3].contiguous()))
refused(lambda: tk.prefill_batched(emb[:60].view(2, 30, -1).contiguous()))
refused(lambda: tk.prefill_append(2, emb))
# and goes on as if nothing had been
e = torch.randn(3, g.hidden, device="cuda")
assert torch.allclose(tk.decode(e)[0], ref.decode(e)[0], rtol=2e-2, atol=2e-2)
tk.prefill(1, emb)
assert tk.cur_len(1) == 70 and tk.sync_status() == 0
for s in (0, 2):
    for a, b in zip(export(tk, s), rows[s]):
        assert torch.equal(a[:, :, :n], b), s
print("ok")
"""


@pytest.mark.parametrize("kv", ["q4_0", "bf16"])
def test_a_prefill_whose_graph_cannot_be_made_leaves_shared_streams_as_they_were(tmp_path, kv):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cc = shutil.which("gcc") or pytest.skip("no C compiler")
    src, lib = tmp_path / "fake.c", tmp_path / "libfake.so"
    src.write_text(FAKE)
    subprocess.run([cc, "-shared", "-fPIC", "-O1", str(src), "-o", str(lib), "-ldl"], check=True)
    r = subprocess.run([sys.executable, "-c", PROGRAM, str(lib), kv], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "LD_PRELOAD": str(lib), "PYTHONPATH": ROOT})
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout[-1000:] + r.stderr[-3000:]
