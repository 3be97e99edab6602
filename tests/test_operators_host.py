"""The training and cache operators without a GPU: their headers' entry points
are exported, bad arguments are refused on the host before any launch, and
the split of a cache's length covers it."""
import ctypes
import os
import random
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
V = ctypes.c_void_p
A = 4096          # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def mods():
    from block_sparse_attention_aware_b200 import build, cache, fvattn, train
    build.build()
    train.load(), cache.load()
    return fvattn, train, cache


def _declared(header):
    src = open(os.path.join(ROOT, "include", header)).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(fvattn_[a-z_]+)\s*\(", src)))


def test_headers_and_bindings_name_the_same_entry_points(mods):
    fv, tr, ca = mods
    for header, mod in (("fvattn_train.h", tr), ("fvattn_cache.h", ca)):
        names = _declared(header)
        assert names == sorted(mod.EXPORTED)
        for n in names:
            assert hasattr(fv.load(), n), n


# ------------------------------------------------------------------ training

def _bwd(fv, g, **kw):
    p = dict(q=A, k=A, v=A, o=A, do=A, lse=A, idx=A, cnt=A, scale=0.125, dq=A, dk=A, dv=A, ws=A, bytes=1 << 40)
    p.update(kw)
    return fv.load().fvattn_sparse_attn_bwd(None if g is None else ctypes.byref(g), *[p[n] for n in (
        "q", "k", "v", "o", "do", "lse", "idx", "cnt", "scale", "dq", "dk", "dv", "ws", "bytes")], None)


def _lse(fv, g, **kw):
    p = dict(q=A, k=A, v=A, idx=A, cnt=A, scale=0.125, o=A, lse=A, stats=None, ws=A, bytes=1 << 40)
    p.update(kw)
    return fv.load().fvattn_sparse_attn_lse(None if g is None else ctypes.byref(g), *[p[n] for n in (
        "q", "k", "v", "idx", "cnt", "scale", "o", "lse", "stats", "ws", "bytes")], None)


def test_training_calls_refuse_bad_arguments(mods):
    fv = mods[0]
    g = fv.geom(1, 2, 64, 2, 8, 8, 2, 2, 4)
    for call, names in ((_bwd, ("q", "k", "v", "o", "do", "lse", "idx", "cnt", "dq", "dk", "dv", "ws")),
                        (_lse, ("q", "k", "v", "idx", "cnt", "o", "lse", "ws"))):
        assert call(fv, None) == fv.ERR_INVALID
        for n in names:
            assert call(fv, g, **{n: None}) == fv.ERR_INVALID, n
            assert call(fv, g, **{n: A + 4 if n not in ("idx", "cnt", "lse") else A + 2}) == fv.ERR_INVALID, n
        assert call(fv, g, bytes=16) == fv.ERR_INVALID
        for scale in (0.0, -1.0, float("inf"), float("nan")):
            assert call(fv, g, scale=scale) == fv.ERR_INVALID
        for field, value in (("D", 96), ("bs", 48), ("nb", 4000)):
            bad = fv.Geom.from_buffer_copy(g)
            setattr(bad, field, value)
            assert call(fv, bad) != fv.OK, field


def test_backward_workspace_holds_its_parts(mods):
    fv, tr, _ = mods
    size = tr.load().fvattn_sparse_attn_bwd_workspace_size
    assert size(None) == 0
    for args in ((1, 40, 128, 21, 45, 80, 2, 8, 8), (1, 2, 64, 2, 8, 8, 2, 2, 4), (2, 3, 64, 3, 5, 7, 2, 2, 4)):
        g = fv.geom(*args)
        heads, groups = g.B * g.H, -(-g.nb * g.bs // 128)
        assert size(ctypes.byref(g)) >= 9 * heads * g.Npad + 8 * heads * groups * g.nb + heads * g.nb * (g.nb // 8)
        assert size(ctypes.byref(g)) % 256 == 0


def test_training_bindings_refuse_host_tensors_and_wrong_shapes(mods):
    fv, tr, _ = mods
    g = fv.geom(1, 2, 64, 2, 8, 8, 2, 2, 4)
    x = torch.zeros((1, 2, g.Npad, 64), dtype=torch.bfloat16)
    i, c = torch.zeros((1, 2, g.nb, g.nb), dtype=torch.int32), torch.zeros((1, 2, g.nb), dtype=torch.int32)
    lse = torch.zeros((1, 2, g.Npad))
    with pytest.raises(ValueError, match="CUDA"):
        tr.sparse_attn_lse(g, x, x, x, i, c)
    with pytest.raises(ValueError, match="required"):
        tr.sparse_attn_lse(g, None, x, x, i, c)
    with pytest.raises(ValueError, match="CUDA"):
        tr.sparse_attn_bwd(g, x, x, x, x, x, lse, i, c)
    with pytest.raises(ValueError, match="CUDA"):
        tr.attention(g, x, x, x, i, c)
    with pytest.raises(ValueError, match="order"):
        tr.TrainLayer(g, 0.9, 1, order="spiral")


# ------------------------------------------------------------------ cache

def _append(fv, ca, cache={}, rot={}, **kw):
    c = dict(pages=4, Hkv=2, D=64, page=16, k=A, v=2 * A)
    c.update(cache)
    r = None
    if rot is not None:
        r = dict(table=A, rows=8, axes=2, pairs=(20, 12, 0), pos=A, halves=0)
        r.update(rot)
        r = ca._Rotation(r["table"], r["rows"], r["axes"], (ctypes.c_int * 3)(*r["pairs"]), r["pos"], r["halves"])
    p = dict(B=2, rows=5, cu=A, lens=A, table=A, width=2, k=A, ks=128, v=A, vs=128, q=A, qs=256, Hq=4, qo=A, qos=256)
    p.update(kw)
    return fv.load().fvattn_cache_append(
        ctypes.byref(ca._Cache(c["pages"], c["Hkv"], c["D"], c["page"], c["k"], c["v"])),
        *[p[n] for n in ("B", "rows", "cu", "lens", "table", "width", "k", "ks", "v", "vs", "q", "qs", "Hq", "qo", "qos")],
        None if r is None else ctypes.byref(r), None)


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(rows=-1), dict(rows=1 << 31), dict(width=0), dict(lens=None), dict(table=None), dict(k=None), dict(v=None),
    dict(cu=None, rows=1), dict(k=A + 2), dict(lens=A + 2), dict(cu=A + 2), dict(ks=120), dict(vs=132), dict(qs=248),
    dict(q=None), dict(qo=None), dict(Hq=0), dict(qos=100),
    dict(cache=dict(pages=0)), dict(cache=dict(Hkv=0)), dict(cache=dict(k=None)), dict(cache=dict(v=A)),
    dict(cache=dict(k=A + 8)),
    dict(rot=dict(table=None)), dict(rot=dict(pos=None)), dict(rot=dict(rows=0)), dict(rot=dict(axes=0)),
    dict(rot=dict(axes=4)), dict(rot=dict(pairs=(20, 11, 0))), dict(rot=dict(pairs=(-1, 33, 0))), dict(rot=dict(halves=2)),
], ids=str)
def test_append_refuses(mods, kw):
    fv, _, ca = mods
    assert _append(fv, ca, **kw) == fv.ERR_INVALID


def _attend(fv, ca, cache={}, **kw):
    c = dict(pages=4, Hkv=2, D=64, page=16, k=A, v=2 * A)
    c.update(cache)
    p = dict(B=2, Hq=4, q=A, qs=256, table=A, width=2, lens=A, longest=5000, scale=0.125, o=A, lse=A, ws=A, bytes=1 << 40)
    p.update(kw)
    return fv.load().fvattn_cache_attn(
        ctypes.byref(ca._Cache(c["pages"], c["Hkv"], c["D"], c["page"], c["k"], c["v"])),
        *[p[n] for n in ("B", "Hq", "q", "qs", "table", "width", "lens", "longest", "scale", "o", "lse", "ws", "bytes")], None)


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(B=65536), dict(width=0), dict(q=None), dict(table=None), dict(lens=None), dict(o=None), dict(Hq=1), dict(Hq=5),
    dict(longest=-1), dict(longest=1 << 31), dict(q=A + 2), dict(o=A + 2), dict(lens=A + 2), dict(lse=A + 2), dict(qs=248),
    dict(qs=260), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(ws=None), dict(ws=A + 16),
    dict(bytes=64), dict(cache=dict(pages=0)), dict(cache=dict(v=A)),
], ids=str)
def test_attend_refuses(mods, kw):
    fv, _, ca = mods
    assert _attend(fv, ca, **kw) == fv.ERR_INVALID


def test_unsupported_cache_shapes(mods):
    fv, _, ca = mods
    for bad in (dict(D=96), dict(page=24), dict(page=256)):
        assert _attend(fv, ca, cache=bad) == fv.ERR_UNSUPPORTED
        assert _append(fv, ca, cache=bad) == fv.ERR_UNSUPPORTED
    assert _attend(fv, ca, cache=dict(pages=1 << 28, page=16)) == fv.ERR_UNSUPPORTED      # rows past 2^31


def test_parts_cover_the_length(mods):
    fv, _, ca = mods
    L, rng, tk = ca.load(), random.Random(7), ctypes.c_int()
    for i in range(400):
        hkv, group = rng.randint(1, 64), rng.choice([1, 2, 4, 8, 17, 40])
        b = int(2 ** rng.uniform(0, 12))
        longest = 0 if i == 0 else int(2 ** rng.uniform(0, 31)) - 130 if i % 3 == 0 else rng.randint(1, 100000)
        longest = max(longest, 0)
        parts = L.fvattn_cache_attn_parts(b, hkv * group, hkv, 128, longest, ctypes.byref(tk))
        assert 1 <= parts <= 256 and tk.value % 64 == 0 and tk.value >= 64
        assert parts * tk.value >= longest and (parts == 1 or (parts - 1) * tk.value < longest)
        need = L.fvattn_cache_attn_workspace_size(b, hkv * group, hkv, 128, longest)
        assert need == 0 if parts == 1 else need >= b * hkv * group * parts * (128 * 4 + 8)
    for bad in ((0, 1, 1, 64, 1), (1, 3, 2, 64, 1), (1, 1, 1, 96, 1), (1, 1, 1, 64, -1), (1, 1, 0, 64, 1)):
        assert L.fvattn_cache_attn_parts(*bad, None) == 0 and L.fvattn_cache_attn_workspace_size(*bad) == 0


def test_cache_bindings_refuse_host_tensors(mods):
    _, _, ca = mods
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ca.PagedCache(k, k.clone())
    with pytest.raises(ValueError, match="add up"):
        ca.rotation_table(64, (20, 20), 8, device="cpu")


def test_rotation_table_keeps_the_phase_of_far_positions(mods):
    """cos and sin of n base^(-i/pairs) at n = 999999 to fp32 rounding (2^-24, values at most 1): an angle formed in
    32 bits would be off by up to 2^-24 * 10^6 = 0.06."""
    import math
    _, _, ca = mods
    t = ca.rotation_table(64, (20, 12), 1_000_000, device="cpu")
    assert t.shape == (1_000_000, 64) and t.dtype == torch.float32
    for n in (0, 1, 12345, 999_999):
        for i in range(32):
            pairs, j = (20, i) if i < 20 else (12, i - 20)
            a = n * 10000.0 ** (-j / pairs)
            # the angle itself is a 64-bit product of two roundings: 3 * 2^-53 * 10^6 more
            assert abs(t[n, i].item() - math.cos(a)) <= 2 ** -24 + 1e-9
            assert abs(t[n, 32 + i].item() - math.sin(a)) <= 2 ** -24 + 1e-9


def test_the_extension_leaves_all_but_the_plain_case_to_the_bindings(mods):
    fv, tr, _ = mods
    n = tr.native()
    t = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    g = fv.geom(1, 2, 64, 2, 8, 8, 2, 2, 4)
    for f, count in ((n.append, 13), (n.attend, 10), (n.sparse_attn_lse, 10), (n.sparse_attn_bwd, 11)):
        assert f() is NotImplemented and f(*[None] * count) is NotImplemented and f(*[1] * count) is NotImplemented
        assert f(*[t] * count) is NotImplemented                       # not on a GPU
        assert f(g, *[t] * (count - 1)) is NotImplemented


# ------------------------------------------------------------------ sources

CSRC = os.path.join(ROOT, "block_sparse_attention_aware_b200", "csrc")


def _code(name):
    src = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", src, flags=re.S))


@pytest.mark.parametrize("name", ["attn.cu", "cache.cu", "grad.cu", "route.cu", "common.cuh", "ptx.cuh"])
def test_kernels_that_start_early_read_with_plain_loads(name):
    """A kernel that waits for the one before it after its own start (pdl_wait) may have begun while its inputs were
    written: nothing in it goes through the read-only path, which takes inputs as constant from the kernel's start."""
    src = _code(name)
    if name == "route.cu":       # some of its kernels start after all before them have ended
        parts = [p for p in src.split("__global__")[1:] if "pdl_wait()" in p]
        assert len(parts) == 2
        src = "\n".join(parts)
    for path in (r"__ldg\s*\(", r"ld\.global\.nc", r"const\s+[\w:]+\s*\*\s*__restrict__"):
        assert not re.search(path, src), path


def test_append_into_fresh_queries_refuses(mods):
    fv, _, ca = mods

    class Fresh:         # _append's call under the other name
        def load(self):
            L = ca.load()
            return type("L", (), dict(fvattn_cache_append=staticmethod(L.fvattn_cache_append_fresh)))

    for kw in (dict(q=None, qo=None), dict(q=None), dict(qo=None), dict(q=A, qo=A), dict(B=0, qo=2 * A), dict(qos=100, qo=2 * A)):
        assert _append(Fresh(), ca, **kw) == fv.ERR_INVALID, kw


# ------------------------------------------------------------------ errors

# A stand-in for the CUDA runtime whose calls fail as often as it is told: it runs nothing and keeps the last error as
# the runtime does.
FAKE_RUNTIME = r"""
#include <stddef.h>
static int last = 0, left = 0;
void fake_fail_after(int calls) { left = calls; last = 0; }
int fake_last(void) { return last; }
static int result(void) { if (left-- > 0) return 0; return last = 719; }
int cudaGetLastError(void) { int e = last; last = 0; return e; }
int cudaGetDevice(int* d) { *d = 0; return result(); }
int cudaDeviceGetAttribute(int* v, int attr, int dev) { (void)attr; (void)dev; *v = 148; return result(); }
int cudaFuncGetAttributes(int* a, const void* f) { (void)f; for (int i = 0; i < 16; ++i) a[i] = 255; return result(); }
int cudaFuncSetAttribute(const void* f, int a, int v) { (void)f; (void)a; (void)v; return result(); }
static int encode(void) { return 0; }
int cudaGetDriverEntryPoint(const char* n, void** p, unsigned long long f, int* q) { (void)n; (void)f; *p = (void*)encode; *q = 0; return result(); }
int cudaGetSymbolAddress(void** p, const void* s) { (void)s; *p = (void*)4096; return result(); }
int cudaLaunchKernel(void) { return result(); }
int cudaLaunchKernelExC(void) { return result(); }
int cudaMemcpy2DAsync(void) { return result(); }
int cudaMemcpyFromSymbol(int* d) { *d = 0; return result(); }
int cudaMemcpyToSymbol(void) { return result(); }
int cudaStreamSynchronize(void) { return result(); }
int __cudaPushCallConfiguration(void) { return 0; }
int __cudaPopCallConfiguration(void) { return 0; }
static void* handle[4];
void** __cudaRegisterFatBinary(void* f) { (void)f; return handle; }
void __cudaRegisterFatBinaryEnd(void** h) { (void)h; }
void __cudaUnregisterFatBinary(void** h) { (void)h; }
void __cudaRegisterFunction(void) {}
void __cudaRegisterVar(void) {}
"""

CALLER = r"""
import ctypes, sys
fake, path = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL), sys.argv[2]
L = ctypes.CDLL(path)
I, P, F, LL, D, S = ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_longlong, ctypes.c_double, ctypes.c_size_t
A, BIG = P(4096), S(1 << 40)
geoms = []
for bs in ((2, 2, 4), (2, 8, 8)):
    g = ctypes.create_string_buffer(256)
    ctypes.memmove(g, (I * 9)(1, 2, 64, 4, 16, 16, *bs), 36)
    assert L.fvattn_geom_init(g) == 0
    geoms.append(g)
cache = ctypes.create_string_buffer(64)
ctypes.memmove(cache, (I * 4)(4, 2, 64, 16), 16)
ctypes.memmove(ctypes.byref(cache, 16), (P * 2)(4096, 8192), 16)
calls = {}
for n, g in enumerate(geoms):
    calls.update({
        f"lse {n}": lambda g=g: L.fvattn_sparse_attn_lse(g, A, A, A, A, A, F(0.125), A, A, None, A, BIG, None),
        f"attn {n}": lambda g=g: L.fvattn_sparse_attn(g, A, A, A, A, A, F(0.125), A, None, A, BIG, None),
        f"noalloc {n}": lambda g=g: L.fvattn_sparse_attn_noalloc(g, A, A, A, A, A, F(0.125), A, None, None),
        f"bwd {n}": lambda g=g: L.fvattn_sparse_attn_bwd(g, A, A, A, A, A, A, A, A, F(0.125), A, A, A, A, BIG, None),
        f"route {n}": lambda g=g: L.fvattn_route(g, A, A, D(0.9), I(1), F(0.125), A, A, None, None, None, A, BIG, None),
        f"reorder_route {n}": lambda g=g: L.fvattn_reorder_route(g, A, A, A, P(8192), D(0.9), I(1), I(0), F(0.125), A, A, None,
                                                                None, None, A, BIG, None),
        f"reorder {n}": lambda g=g: L.fvattn_reorder(g, A, P(8192), None),
        f"order {n}": lambda g=g: L.fvattn_block_order(g, A, None),
        f"heads {n}": lambda g=g: L.fvattn_copy_heads(g, I(0), I(1), A, P(8192), I(1), None)})
calls["append"] = lambda: L.fvattn_cache_append(cache, I(2), LL(2), None, A, A, I(2), A, LL(128), A, LL(128), None, LL(0), I(0), None,
                                                LL(0), None, None)
calls["attend"] = lambda: L.fvattn_cache_attn(cache, I(2), I(4), A, LL(256), A, I(2), A, LL(5000), F(0.125), A, A, A, BIG, None)
calls["status"] = lambda: L.fvattn_get_status(None)
for name, call in calls.items():
    for good in range(40):           # the runtime's calls fail from the good-th on
        fake.fake_fail_after(good)
        rc = call()
        assert fake.fake_last() == 0, (name, good, rc)
        if rc == 0:
            break
        assert rc == 3, (name, good, rc)
    else:
        raise AssertionError(name)
    assert good > 0, name
print("done")
"""


def test_failed_calls_leave_no_error_behind(mods, tmp_path):
    """Whichever call of the runtime fails, the entry point returns the error and clears the runtime's last one, which
    the next check of somebody else's launch would take for its own."""
    import subprocess
    import sys
    from block_sparse_attention_aware_b200 import fvattn
    src, lib = tmp_path / "fake.c", tmp_path / "libcudart.so.12"
    src.write_text(FAKE_RUNTIME)
    (tmp_path / "versions").write_text("libcudart.so.12 { global: *; };")
    subprocess.check_call(["gcc", "-shared", "-fPIC", "-O1", "-w", "-Wl,-soname,libcudart.so.12",
                           f"-Wl,--version-script={tmp_path}/versions", str(src), "-o", str(lib)])
    done = subprocess.run([sys.executable, "-S", "-c", CALLER, str(lib), fvattn.LIB_PATH], capture_output=True, text=True, timeout=120,
                          env=dict(os.environ, LD_LIBRARY_PATH=str(tmp_path)))
    assert done.returncode == 0 and "done" in done.stdout, done.stderr[-2000:]


# ------------------------------------------------------------------ the extension's build

def test_the_extension_is_built_again_for_another_torch(mods, tmp_path, monkeypatch):
    """Only the extension: the library does not know torch.  Nothing is built where nothing changed."""
    from block_sparse_attention_aware_b200 import build
    commands = []
    monkeypatch.setattr(build.subprocess, "check_call", lambda cmd, *a, **k: commands.append(cmd))
    monkeypatch.setattr(build.subprocess, "Popen", lambda cmd, *a, **k: pytest.fail("the library is built again"))
    monkeypatch.setattr(build.os, "replace", lambda a, b: None)
    build.build()
    assert commands == []
    stamp = tmp_path / "native.txt"
    monkeypatch.setattr(build, "STAMP", str(stamp))
    stamp.write_text("torch 1.0, Python 3.12")
    build.build()
    assert len(commands) == 1 and commands[0][0] == "g++" and stamp.read_text() == build.native_target()
    build.build()
    assert len(commands) == 1


def test_an_extension_for_another_torch_is_refused(mods, monkeypatch):
    import types
    import block_sparse_attention_aware_b200 as package
    tr = mods[1]
    assert tr.native().target == tr.build.native_target()
    monkeypatch.setattr(tr, "_fast", None)
    monkeypatch.setattr(package, "_native", types.SimpleNamespace(target="torch 1.0, Python 3.12"))
    with pytest.raises(ImportError, match="built for torch 1.0"):
        tr.native()
