"""CPU test of the host encoders where threads are refused, for certain: a preloaded
pthread_create gives the first few and then fails as a system without more does.
The parts without a thread are done on the caller's, none among them."""
import os
import shutil
import subprocess
import sys

import pytest

HOOK = r"""
#define _GNU_SOURCE
#include <dlfcn.h>
#include <errno.h>
#include <pthread.h>
static int left = -1, made = 0, refused = 0;   /* left < 0: all are given */
void hook_allow(int n) { left = n; made = refused = 0; }
int hook_made(void) { return made; }
int hook_refused(void) { return refused; }
int pthread_create(pthread_t* t, const pthread_attr_t* a, void* (*f)(void*), void* x) {
  static int (*real)(pthread_t*, const pthread_attr_t*, void* (*)(void*), void*);
  if (!real) real = (int (*)(pthread_t*, const pthread_attr_t*, void* (*)(void*), void*))dlsym(RTLD_NEXT, "pthread_create");
  if (left == 0) { ++refused; return EAGAIN; }
  if (left > 0) { --left; ++made; }
  return real(t, a, f, x);
}
"""

CODE = """
import ctypes, sys
import numpy as np
import unstructured_sparse_weight_amd as usw
hook = ctypes.CDLL(sys.argv[1])
rng = np.random.default_rng(1)
W = (rng.standard_normal((1024, 256)) * 0.05).astype(np.float16)
mask = rng.random((1024, 256)) < 0.5
encoders = (lambda: usw.w4_encode_host(W, 64), lambda: usw.encode_host(W, mask), lambda: usw.encode_host(W, mask, dtype="i4"))
want = [e() for e in encoders]
for allowed in (0, 1, 3):
    for e, w in zip(encoders, want):
        hook.hook_allow(allowed)
        got = e()
        made, refused = hook.hook_made(), hook.hook_refused()
        hook.hook_allow(-1)
        for name in ("codes", "values", "scales", "offsets", "bitmaps"):
            a, b = getattr(got, name, None), getattr(w, name, None)
            assert (a is None) == (b is None) and (a is None or np.array_equal(a, b)), name
        print(allowed, made, refused)
"""


def test_encoders(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    # Parts there are: one to a hardware thread, 16 at most, 4 where the number is unknown.
    if len(os.sched_getaffinity(0)) < 5:
        pytest.skip("needs five hardware threads, so that a fourth thread is asked for")
    src, so = tmp_path / "hook.c", tmp_path / "hook.so"
    src.write_text(HOOK)
    subprocess.run([cc, "-shared", "-fPIC", "-O1", str(src), "-o", str(so), "-ldl"], check=True)
    env = dict(os.environ, LD_PRELOAD=":".join(p for p in (str(so), os.environ.get("LD_PRELOAD", "")) if p))
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CODE, str(so)], capture_output=True, text=True, timeout=120, cwd=root, env=env)
    assert r.returncode == 0, r.stderr[-800:]
    rows = [[int(v) for v in line.split()] for line in r.stdout.splitlines()]
    assert len(rows) == 9
    for allowed, made, refused in rows:
        # Each parallel section asks again after a refusal, so only the first sections' threads are made.
        assert made == allowed and refused >= 1, (allowed, made, refused)
