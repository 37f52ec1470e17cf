"""Which kernels the library launches for a call, found without a GPU: its
objects are linked with a stand-in for the runtime that notes the kernels'
names in place of starting them. Addresses are never read, so any aligned
numbers serve as buffers."""
import ctypes
import glob
import os
import re
import subprocess

from combine_epx_get_amd import build

RUNTIME = r"""
#include <stddef.h>
#include <string.h>
typedef struct { unsigned x, y, z; } dim3_t;
static struct { const void *f; const char *name; } known[4096];
static int num_known, num_launched;
static const char *launched[64];
static dim3_t pushed_grid, pushed_block;
static size_t pushed_lds;
static void *pushed_stream;
int num_kernels(void) { return num_known; }
const char *kernel_name(int i) { return known[i].name; }
int num_launches(void) { return num_launched; }
const char *launch_name(int i) { return launched[i]; }
void forget(void) { num_launched = 0; }
void **__hipRegisterFatBinary(const void *d) { static void *h; (void)d; return &h; }
void __hipUnregisterFatBinary(void **h) { (void)h; }
void __hipRegisterVar(void **h, void *v, char *a, char *b, int e, size_t s, int c, int g)
{ (void)h; (void)v; (void)a; (void)b; (void)e; (void)s; (void)c; (void)g; }
void __hipRegisterFunction(void **h, const void *f, char *d, const char *name, unsigned t, void *a, void *b, void *c,
                           void *e, int *w)
{
    (void)h; (void)d; (void)t; (void)a; (void)b; (void)c; (void)e; (void)w;
    known[num_known].f = f;
    known[num_known++].name = name;
}
int __hipPushCallConfiguration(dim3_t g, dim3_t b, size_t lds, void *s)
{ pushed_grid = g; pushed_block = b; pushed_lds = lds; pushed_stream = s; return 0; }
int __hipPopCallConfiguration(dim3_t *g, dim3_t *b, size_t *lds, void **s)
{ *g = pushed_grid; *b = pushed_block; *lds = pushed_lds; *s = pushed_stream; return 0; }
static int note(const void *f)
{
    for (int i = 0; i < num_known; ++i)
        if (known[i].f == f && num_launched < 64) {
            launched[num_launched++] = known[i].name;
            return 0;
        }
    return 1;
}
int hipLaunchKernel(const void *f, dim3_t g, dim3_t b, void **a, size_t lds, void *s)
{ (void)g; (void)b; (void)a; (void)lds; (void)s; return note(f); }
int hipExtLaunchKernel(const void *f, dim3_t g, dim3_t b, void **a, size_t lds, void *s, void *x, void *y, int n)
{ (void)g; (void)b; (void)a; (void)lds; (void)s; (void)x; (void)y; (void)n; return note(f); }
int hipGetLastError(void) { return 0; }
int hipGetDevice(int *d) { *d = 0; return 0; }
int hipGetSymbolAddress(void **p, const void *s) { (void)p; (void)s; return 1; }
int hipMemcpyAsync(void *d, const void *s, size_t n, int k, void *q) { (void)d; (void)s; (void)n; (void)k; (void)q; return 1; }
int hipStreamSynchronize(void *q) { (void)q; return 1; }
"""


class Rows(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32), ("num_rows", ctypes.c_int32), ("row_offset", ctypes.c_void_p),
                ("row_count", ctypes.c_void_p)]


def objects():
    srcs = sorted(glob.glob(os.path.join(build.CSRC, "*.hip")))
    objs = [os.path.join(build.BUILD, os.path.basename(s) + ".o") for s in srcs]
    newest = max(os.path.getmtime(s) for s in glob.glob(os.path.join(build.CSRC, "*")))
    if not all(os.path.exists(o) and os.path.getmtime(o) >= newest for o in objs):
        build.build()
    return objs


class Recorder:
    """The library's entry points (`lib`), and the kernels that a call launches."""

    def __init__(self, folder):
        source, so = os.path.join(folder, "runtime.c"), os.path.join(folder, "librecorder.so")
        open(source, "w").write(RUNTIME)
        for cmd in (["gcc", "-O1", "-fPIC", "-c", source, "-o", source + ".o"],
                    ["g++", "-shared", "-Wl,-Bsymbolic", "-Wl,-z,defs", "-o", so, source + ".o", *objects()]):
            r = subprocess.run(cmd, capture_output=True, text=True)
            assert r.returncode == 0, r.stderr[-2000:]
        self.lib = ctypes.CDLL(so)
        for f in ("kernel_name", "launch_name"):
            getattr(self.lib, f).restype = ctypes.c_char_p
        mangled = [self.lib.kernel_name(i).decode() for i in range(self.lib.num_kernels())]
        plain = subprocess.run(["c++filt"], input="\n".join(mangled), capture_output=True, text=True, check=True).stdout
        # a template's name and arguments alone
        self.names = {m: re.sub(r"^void |epx::|\(anonymous namespace\)::|\((?!anonymous).*$", "", p)
                      for m, p in zip(mangled, plain.splitlines())}

    def kernels(self):
        return set(self.names.values())

    def launched(self, call):
        """Names of what `call`, a function of the library, launches; it has to succeed."""
        self.lib.forget()
        assert call(self.lib) == 0
        return [self.names[self.lib.launch_name(i).decode()] for i in range(self.lib.num_launches())]


def expert_calls(rows, experts, width, inner):
    """The experts' products on 8-bit rows by name, at addresses that are never read."""
    at = [ctypes.c_void_p((i + 1) << 20) for i in range(10)]
    x, xs, w, ws, kept, kept_scales, out, act, off, cnt = at
    r = Rows(experts, rows, off, cnt)
    ref = ctypes.byref(r)
    int8 = lambda act, *keep: lambda lib: lib.epx_expert_gemm_int8(   # noqa: E731
        ref, x, xs, w, ws, width, inner, act, *(keep or (None, None)), out, None)
    wgrad = lambda dtype: lambda lib: lib.epx_expert_gemm_wgrad_kept8(   # noqa: E731
        ref, x, kept, kept_scales, width, inner, dtype, 0, out, None)
    return {
        "int8": int8(0), "int8 gated": int8(1), "int8 kept": int8(1, kept, kept_scales),
        "keep8": lambda lib: lib.epx_expert_gemm_keep8(ref, x, w, width, inner, kept, kept_scales, out, None),
        "dgrad8": lambda lib: lib.epx_expert_gemm_dgrad_kept8(ref, x, w, width, inner, kept, kept_scales, act, out, None),
        "wgrad8 bf16": wgrad(0), "wgrad8 f32": wgrad(2),
    }
