"""The library's host side on a stand-in for the CUDA runtime (fake_cudart.cpp): the objects that
the build leaves are linked with it into a library of their own.  Pointers that a test passes as
device buffers are plain numbers that nobody follows."""
import ctypes
import os
import shutil
import subprocess

from kv_cache_incremental_gb300 import _build, _lib

HERE = os.path.dirname(os.path.abspath(__file__))
PTR = 1 << 40          # device buffers: any 16-byte aligned numbers


def build(directory):
    objs = [os.path.join(_build.OUT_DIR, s.replace(".cu", ".o")) for s in _build.SOURCES]
    _build.build(force=not all(map(os.path.exists, objs)))
    out = os.path.join(directory, "libkvinc_host.so")
    nvcc = os.path.realpath(shutil.which("nvcc"))
    include = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wl,-Bsymbolic",
                        "-Wl,-z,defs", f"-I{include}", os.path.join(HERE, "fake_cudart.cpp"),
                        *objs, "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(out)
    for name, (res, args) in _lib.SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    lib.fake_live_bytes.restype = ctypes.c_longlong
    lib.fake_launch_name.restype = ctypes.c_char_p
    return lib


def i32(values):
    return None if values is None else (ctypes.c_int32 * max(1, len(values)))(*values)


class Cache:
    """A cache of the host-side library; calls return the status code."""

    def __init__(self, lib, B=2, max_len=640, Hq=8, Hk=2, D=64, kinds=(0,), W=0, blocks=None):
        self.lib, self.B, self.max_len, self.Hq, self.Hk, self.D = lib, B, max_len, Hq, Hk, D
        self.kinds = list(kinds)
        self.h = ctypes.c_void_p()
        args = (ctypes.byref(self.h), B, max_len, Hq, Hk, D, W, len(kinds), i32(kinds), 1e4, 0)
        self.rc = (lib.kv_cache_create(*args) if blocks is None
                   else lib.kv_cache_create_paged(*args, blocks))

    def close(self):
        self.lib.kv_cache_destroy(self.h)

    def append(self, n_new, rows=None, layer=0, C=None):
        return self.lib.kv_append(self.h, layer, PTR, PTR, PTR, self.Hq, C or max(1, *n_new),
                                  i32(n_new), i32(rows), len(n_new), PTR, None)

    def advance(self, n_new, rows=None):
        return self.lib.kv_advance(self.h, i32(n_new), i32(rows), len(n_new), None)

    def fill(self, lens):
        for b, n in enumerate(lens):
            if n:
                assert self.lib.kv_import_row(self.h, b, n, PTR,
                                              self.lib.kv_export_bytes(self.h, n), None) == 0

    def sparse(self, n_new, top_k, sink=1, recent=2, rows=None, layer=0, selected=None):
        return self.lib.kv_append_sparse(self.h, layer, PTR, PTR, PTR, self.Hq, max(1, *n_new),
                                         i32(n_new), i32(rows), len(n_new), sink, top_k, recent,
                                         PTR, selected, None)

    def weights(self, n_new, acc_in=PTR, acc_out=PTR, last=1, rows=None, layer=0):
        return self.lib.kv_append_weights(self.h, layer, PTR, PTR, PTR, self.Hq, max(1, *n_new),
                                          i32(n_new), i32(rows), len(n_new), last, acc_in,
                                          acc_out, PTR, None)

    def evict(self, dst_rows, src, src_rows, keep, recent, acc_in, acc_out, kept):
        arr = lambda xs: None if xs is None else (ctypes.c_void_p * len(xs))(*xs)
        return self.lib.kv_evict_rows(self.h, i32(dst_rows), src.h, i32(src_rows), len(dst_rows),
                                      keep, recent, arr(acc_in), arr(acc_out), arr(kept), None)

    def table(self, row):
        n = ctypes.c_int()
        self.lib.kv_get_block_table(self.h, row, None, 0, ctypes.byref(n))
        out = (ctypes.c_int32 * max(1, n.value))()
        self.lib.kv_get_block_table(self.h, row, out, n.value, ctypes.byref(n))
        return list(out)[:n.value]

    def state(self):
        """Everything the host knows of the rows that a caller can ask for."""
        lens, slots = (ctypes.c_int32 * self.B)(), (ctypes.c_int32 * self.B)()
        assert self.lib.kv_get_lens(self.h, lens) == 0
        assert self.lib.kv_get_slots(self.h, slots) == 0
        return (list(lens), list(slots), [self.table(b) for b in range(self.B)],
                self.lib.kv_free_blocks(self.h))

    def launches(self):
        """(kernel, grid x) of the launches since the last call of this function."""
        out = []
        for i in range(self.lib.fake_launches()):
            mangled = self.lib.fake_launch_name(i).decode()
            out.append((next((k for k in KERNELS if k in mangled), "?"),
                        self.lib.fake_launch_grid(i)))
        self.lib.fake_reset()
        return out


KERNELS = ["append_kernel", "state_kernel", "table_kernel", "copy_kernel", "bounds_kernel",
           "select_kernel", "join_kernel", "weights_kernel", "evict_move", "evict_select",
           "decode_kernel", "prefill_merge", "prefill_tc", "prefill_kernel", "commit_kernel"]
KERNELS.sort(key=len, reverse=True)   # evict_select_kernel holds select_kernel's name
