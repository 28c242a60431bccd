"""The C ABI of the scan, the convolution and the group norm: exported symbols,
structure layouts, size queries and refusals before any device is touched (CPU
only); and the refusals of their Python bindings."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

from linear_rnn_sequence_wkv7_amd import groupnorm as N
from linear_rnn_sequence_wkv7_amd import shortconv as K
from linear_rnn_sequence_wkv7_amd import ssm as S
from linear_rnn_sequence_wkv7_amd import wkv7 as W

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(not os.path.exists(W.lib_path()), reason="libwkv7.so not built")

SP = 1 << 26          # 64 MiB between fake arrays: disjoint unless a test makes them overlap
BASE = 1 << 36        # never dereferenced: every case below fails validation, or has nothing to do


def declared(header):
    src = open(os.path.join(ROOT, "include", header)).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return set(re.findall(r"^\s*(?:int|int64_t)\s+(\w+)\s*\(", src, flags=re.M))


@pytest.mark.parametrize("header,mod", [("ssm.h", S), ("shortconv.h", K), ("groupnorm.h", N)])
def test_every_declared_symbol_is_exported(header, mod):
    names = declared(header)
    assert names == set(mod.EXPORTED_SYMBOLS)
    lib = W.load_library()
    for n in names:
        assert hasattr(lib, n), n


def test_structures_match_the_headers(tmp_path):
    """Sizes and offsets as a C compiler sees them."""
    prog = tmp_path / "layout.c"
    fields = {"ssm": S.SsmDesc, "shortconv": K.ShortconvDesc, "groupnorm": N.GroupnormDesc}
    lines = ['#include <stdio.h>', '#include <stddef.h>']
    lines += [f'#include "{n}.h"' for n in fields]
    lines.append("int main(void) {")
    for n, st in fields.items():
        lines.append(f'printf("{n} %zu\\n", sizeof({n}_desc));')
        lines += [f'printf("{n}.{f[0]} %zu\\n", offsetof({n}_desc, {f[0]}));' for f in st._fields_]
    lines.append("return 0; }")
    prog.write_text("\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    out = dict(l.split() for l in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    for n, st in fields.items():
        assert int(out[n]) == ctypes.sizeof(st)
        for f in st._fields_:
            assert int(out[f"{n}.{f[0]}"]) == getattr(st, f[0]).offset, f


# ---- calls with fake pointers -------------------------------------------------

CALLS = {
    # function: (descriptor maker, pointer names in order, optional ones, written ones)
    "ssm_forward": ("ssm", "x dt A Bm Cm D dt_bias z state_in y state_out checkpoints", "D dt_bias z state_in state_out checkpoints",
                    "y state_out checkpoints"),
    "ssm_step": ("ssm", "x dt A Bm Cm D dt_bias z state state_index y", "D dt_bias z state_index", "state y"),
    "ssm_backward": ("ssm", "x dt A Bm Cm D dt_bias z state_in dy dstate_out checkpoints dx ddt dA dBm dCm dD ddt_bias dz dstate_in workspace",
                     "D dt_bias z state_in dstate_out checkpoints dD ddt_bias dz dstate_in",
                     "dx ddt dA dBm dCm dD ddt_bias dz dstate_in workspace"),
    "shortconv_forward": ("conv", "x w bias state_in y state_out", "bias state_in state_out", "y state_out"),
    "shortconv_step": ("conv", "x w bias state state_index y", "bias state_index", "state y"),
    "shortconv_backward": ("conv", "x w bias state_in dy dstate_out dx dw dbias dstate_in workspace",
                           "bias state_in dstate_out dbias dstate_in", "dx dw dbias dstate_in workspace"),
    "groupnorm_forward": ("norm", "x weight bias gate y mean rstd workspace", "weight bias gate mean rstd", "y mean rstd workspace"),
    "groupnorm_backward": ("norm", "x weight bias gate dy mean rstd dx dweight dbias dgate workspace",
                           "weight bias gate dweight dbias dgate", "dx dweight dbias dgate workspace"),
}
# gradients that go with an input
PAIRS = {"ssm_backward": {"D": "dD", "dt_bias": "ddt_bias", "z": "dz"}, "shortconv_backward": {"bias": "dbias"},
         "groupnorm_backward": {"weight": "dweight", "bias": "dbias", "gate": "dgate"}, "groupnorm_forward": {"mean": "rstd"}}


def desc(kind, step=False, **kw):
    T = 1 if step else 70
    if kind == "ssm":
        d = dict(B=2, T=T, C=64, N=16, G=1, in_dtype=1, y_dtype=1, dt_softplus=1, S=5)
        return S.SsmDesc(**{**d, **kw})
    if kind == "conv":
        d = dict(B=2, T=T, C=64, K=4, in_dtype=1, y_dtype=1, act=1, S=5)
        return K.ShortconvDesc(**{**d, **kw})
    # positions past what one workgroup holds: the form with a workspace
    d = dict(B=2, T=9000, C=64, G=4, in_dtype=1, y_dtype=1, act=1, eps=1e-5)
    return N.GroupnormDesc(**{**d, **kw})


def call(fn, d=None, **over):
    kind, names, _, _ = CALLS[fn]
    S._lib(), K._lib(), N._lib()
    lib = W.load_library()
    d = desc(kind, fn.endswith("_step")) if d is None else d
    args = []
    for i, n in enumerate(names.split()):
        args.append(over[n] if n in over else BASE + i * SP)
        if n == "workspace":
            args.append(over.get("ws_bytes", SP))
    return getattr(lib, fn)(None if over.get("no_desc") else ctypes.byref(d), *args, None)


def message():
    return W.load_library().wkv7_last_error().decode()


@pytest.mark.parametrize("fn", CALLS)
def test_pointers(fn):
    _, names, optional, _ = CALLS[fn]
    assert call(fn, no_desc=True) == W.WKV7_EINVAL
    for n in names.split():
        if n not in optional.split():
            assert call(fn, **{n: None}) == W.WKV7_EINVAL, n
            assert f"{n} is NULL" in message()
        odd = BASE + 2 if n == "state_index" else BASE + 4
        assert call(fn, **{n: odd}) == W.WKV7_EINVAL, n
        assert f"{n} is not" in message(), n
    for a, b in PAIRS.get(fn, {}).items():
        assert call(fn, **{b: None}) == W.WKV7_EINVAL
        assert b in message()


@pytest.mark.parametrize("fn", CALLS)
def test_written_arrays_share_no_byte(fn):
    _, names, _, written = CALLS[fn]
    names = names.split()
    at = {n: BASE + i * SP for i, n in enumerate(names)}
    for w in written.split():
        for o in names:
            if o == w or (fn.startswith("groupnorm_forward") and {w, o} == {"mean", "rstd"}):
                continue
            if {w, o} == {"state_in", "state_out"}:
                continue   # in place is allowed
            assert call(fn, **{w: at[o]}) == W.WKV7_EINVAL, (w, o)
            assert "overlaps" in message(), (w, o)
    if "state_out" in names and "state_in" in names:   # in place, but not half
        assert call(fn, state_out=at["state_in"] + 16) == W.WKV7_EINVAL
        assert "overlaps" in message()


@pytest.mark.parametrize("fn", ["ssm_forward", "shortconv_forward"])
def test_nothing_else_joins_a_state_in_place(fn):
    """A state that is moved in place shares its bytes with no third array, at its start either."""
    _, names, _, _ = CALLS[fn]
    names = names.split()
    st = BASE + names.index("state_in") * SP
    for o in names:
        if o not in ("state_in", "state_out"):
            assert call(fn, state_out=st, **{o: st}) == W.WKV7_EINVAL, o
            assert "overlaps" in message() and o in message(), o


@pytest.mark.parametrize("fn", [f for f in CALLS if "workspace" in CALLS[f][1]])
def test_workspace_sizes(fn):
    kind = CALLS[fn][0]
    d = desc(kind)
    lib = W.load_library()
    S._lib(), K._lib(), N._lib()
    need = {"ssm_backward": lambda: lib.ssm_backward_workspace_bytes(ctypes.byref(d), 0),
            "shortconv_backward": lambda: lib.shortconv_backward_workspace_bytes(ctypes.byref(d)),
            "groupnorm_forward": lambda: lib.groupnorm_workspace_bytes(ctypes.byref(d)),
            "groupnorm_backward": lambda: lib.groupnorm_backward_workspace_bytes(ctypes.byref(d))}[fn]()
    assert need > 0
    assert call(fn, ws_bytes=need - 1) == W.WKV7_EINVAL
    assert f"{need} needed" in message()
    if fn == "ssm_backward":   # without checkpoints it needs room for them too
        more = lib.ssm_backward_workspace_bytes(ctypes.byref(d), 1)
        assert more >= need + lib.ssm_checkpoint_bytes(ctypes.byref(d))
        assert call(fn, checkpoints=None, ws_bytes=more - 1) == W.WKV7_EINVAL
        assert f"{more} needed" in message()


BAD = {
    "ssm": [(dict(B=-1), 1), (dict(T=-1), 1), (dict(C=-1), 1), (dict(G=-1), 1), (dict(N=0), 1), (dict(N=65), 2), (dict(G=3), 1),
            (dict(in_dtype=2), 1), (dict(y_dtype=-1), 1), (dict(dt_softplus=2), 1), (dict(reserved=1), 1), (dict(lengths=BASE + 2), 1),
            (dict(B=1 << 30, C=1 << 20), 2), (dict(T=2147483647), 2), (dict(C=1 << 22), 2), (dict(C=1 << 18, G=1 << 18, N=16), 2),
            (dict(B=1 << 15, T=1 << 12, C=1 << 10, G=1 << 10, N=64), 2)],
    "conv": [(dict(B=-1), 1), (dict(T=-1), 1), (dict(C=-1), 1), (dict(K=0), 1), (dict(K=1), 2), (dict(K=5), 2), (dict(in_dtype=2), 1),
             (dict(y_dtype=5), 1), (dict(act=2), 1), (dict(lengths=BASE + 1), 1), (dict(B=1 << 30, C=1 << 20), 2)],
    "norm": [(dict(B=-1), 1), (dict(T=-1), 1), (dict(C=-1), 1), (dict(G=0), 1), (dict(G=5), 1), (dict(in_dtype=2), 1), (dict(y_dtype=5), 1),
             (dict(act=-1), 1), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(lengths=BASE + 3), 1),
             (dict(B=1 << 30, C=1 << 20, G=1), 2)],
}


@pytest.mark.parametrize("fn", CALLS)
def test_descriptors(fn):
    kind = CALLS[fn][0]
    step = fn.endswith("_step")
    for kw, code in BAD[kind]:
        if step and "T" in kw:
            code = W.WKV7_EINVAL
        assert call(fn, desc(kind, step, **kw)) == code, kw
        assert message()
    if step:
        assert call(fn, desc(kind, True, T=2)) == W.WKV7_EINVAL
        assert call(fn, desc(kind, True, lengths=BASE)) == W.WKV7_EINVAL
        assert call(fn, desc(kind, True, S=-1)) == W.WKV7_EINVAL
        assert call(fn, desc(kind, True, S=1), state_index=None) == W.WKV7_EINVAL
        assert "state_index" in message()


def test_lengths_need_the_alignment_of_an_int32():
    """A slice of a tensor of lengths is taken (nothing to do here: no device call)."""
    for off in (4, 8, 12):
        assert call("ssm_forward", desc("ssm", B=0, lengths=BASE + off)) == W.WKV7_OK
        assert call("shortconv_forward", desc("conv", B=0, lengths=BASE + off)) == W.WKV7_OK
        assert call("groupnorm_forward", desc("norm", B=0, lengths=BASE + off)) == W.WKV7_OK
        assert call("ssm_step", desc("ssm", True, B=0), state_index=BASE + off) == W.WKV7_OK


WIDE = {
    # more threads than a launch takes, in arrays that fit a GPU's memory
    "ssm_forward": dict(B=1 << 14, T=16, C=1 << 12, G=1 << 12, N=1),
    "ssm_step": dict(B=1 << 27, C=1, N=1, S=1 << 27),
    "ssm_backward": dict(B=1 << 16, T=17, C=1 << 12, N=16, G=1),
    "shortconv_step": dict(B=1 << 26, C=1, K=2, S=1 << 26),
    "shortconv_backward": dict(B=1 << 25, T=2, C=1),
    "groupnorm_forward": dict(B=1 << 23, T=2, C=2, G=2),
    "groupnorm_backward": dict(B=1 << 23, T=2, C=2, G=2),
}


@pytest.mark.parametrize("fn", WIDE)
def test_refuses_more_threads_than_a_launch_takes(fn):
    kind, names, optional, _ = CALLS[fn]
    ptrs = {n: BASE + (i << 45) if n not in optional.split() else None for i, n in enumerate(names.split())}
    d = desc(kind, fn.endswith("_step"), **WIDE[fn])
    assert call(fn, d, **ptrs, ws_bytes=1 << 50) == W.WKV7_EUNSUPPORTED
    assert "2^32" in message()


def test_scan_without_tokens_still_needs_its_rates():
    """The kernel reads A whatever T is."""
    assert call("ssm_forward", desc("ssm", T=0), A=None) == W.WKV7_EINVAL
    assert call("ssm_backward", desc("ssm", T=0), A=None) == W.WKV7_EINVAL
    assert "A is NULL" in message()


def test_norm_size_queries_hold_for_both_dtypes():
    """The forms differ between the dtypes; the binding's query covers either."""
    for T in (1, 2, 600, 1100, 1700, 2100, 3000, 9000):
        for C, G in ((64, 4), (64, 1), (63, 1), (96, 2), (1024, 32)):
            for dt in (0, 1):
                d = ctypes.byref(desc("norm", T=T, C=C, G=G, in_dtype=dt, y_dtype=dt))
                assert N._lib().groupnorm_workspace_bytes(d) <= N.groupnorm_workspace_bytes(2, T, C, G)
                assert N._lib().groupnorm_backward_workspace_bytes(d) <= N.groupnorm_backward_workspace_bytes(2, T, C, G)


def test_size_queries():
    assert S.ssm_checkpoint_bytes(2, 65, 64, 16) == 2 * 3 * 64 * 16 * 4
    assert S.ssm_checkpoint_bytes(2, 0, 64, 16) == 0
    assert S.ssm_backward_workspace_bytes(0, 10, 64, 16) == 0
    assert K.shortconv_backward_workspace_bytes(2, 0, 64, 4) == 0
    assert N.groupnorm_workspace_bytes(2, 0, 64, 4) == 0
    for q in (lambda: S.ssm_checkpoint_bytes(2, -1, 64, 16), lambda: S.ssm_backward_workspace_bytes(2, 1, 64, 65),
              lambda: K.shortconv_backward_workspace_bytes(2, 1, 64, 9), lambda: N.groupnorm_workspace_bytes(2, 1, 64, 5),
              lambda: N.groupnorm_backward_workspace_bytes(2, 1, 64, 0)):
        with pytest.raises(W.Wkv7Error):
            q()


def test_norm_workspace_of_single_rows():
    """At T = 1 the forward needs none for the groups that the header names, and some past them."""
    for Cg in (1, 8, 63, 96, 512, 1000, 1023, 1024, 1026, 2046, 2048):
        for G in (1, 3):
            assert N.groupnorm_workspace_bytes(8, 1, G * Cg, G) == 0, Cg
    for Cg in (1025, 2047, 2049, 2050, 4096):
        assert N.groupnorm_workspace_bytes(8, 1, Cg, 1) > 0, Cg


def test_no_tokens_need_no_workspace():
    """The sizes that the headers give as 0 when B T C == 0."""
    for B, T, C in ((2, 0, 64), (0, 70, 64), (2, 70, 0)):
        for own in (True, False):
            assert S.ssm_backward_workspace_bytes(B, T, C, 16, checkpoints=own) == 0
        assert K.shortconv_backward_workspace_bytes(B, T, C, 4) == 0
        assert N.groupnorm_workspace_bytes(B, T, C, 4) == 0
        assert N.groupnorm_backward_workspace_bytes(B, T, C, 4) == 0


def test_nothing_to_do_needs_no_device():
    assert call("ssm_forward", desc("ssm", B=0)) == W.WKV7_OK
    assert call("ssm_forward", desc("ssm", T=0), state_out=None) == W.WKV7_OK
    assert call("ssm_step", desc("ssm", True, B=0)) == W.WKV7_OK
    assert call("shortconv_forward", desc("conv", B=0)) == W.WKV7_OK
    assert call("shortconv_step", desc("conv", True, B=0)) == W.WKV7_OK
    assert call("groupnorm_forward", desc("norm", B=0)) == W.WKV7_OK
    assert call("shortconv_backward", desc("conv", C=0)) == W.WKV7_OK
    assert call("groupnorm_backward", desc("norm", C=0, G=1)) == W.WKV7_OK


def test_bindings_import_without_torchs_private_names():
    """A torch without the short ways to the current stream and device: the modules are there and refuse as ever."""
    code = """
import torch
for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, n):
        delattr(torch._C, n)
from linear_rnn_sequence_wkv7_amd import _marshal, groupnorm, shortconv, ssm
assert _marshal._raw_stream is _marshal._public_stream and _marshal._device is torch.cuda.current_device
x = torch.zeros(2, 3, 8)
try:
    groupnorm.groupnorm_forward(x, 2)
except ValueError as e:
    assert "GPU" in str(e)
    print("refused")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr


def test_bindings_refuse_sizes_past_an_int32():
    """2^32 + 5 rows are not 5."""
    import torch
    x, many = torch.zeros(2, 3, 8), (1 << 32) + 5
    for q in (lambda n: S.ssm_checkpoint_bytes(n, 1, 1, 1), lambda n: S.ssm_checkpoint_bytes(1, n, 1, 1),
              lambda n: S.ssm_backward_workspace_bytes(1, 1, n, 1), lambda n: S.ssm_backward_workspace_bytes(1, 1, 1, 1, G=n),
              lambda n: K.shortconv_backward_workspace_bytes(n, 1, 1, 4), lambda n: N.groupnorm_workspace_bytes(n, 1, 1, 1),
              lambda n: N.groupnorm_backward_workspace_bytes(1, 1, n, 1),
              # what the calls make of their tensors' shapes
              lambda n: S._desc(x, x, n, 1, 1, 1, 1, True), lambda n: S._desc(x, x, 1, 1, 1, 1, 1, True, None, n),
              lambda n: K._desc(x, x, n, 1, 1, 4, "silu"), lambda n: K._desc(x, x, 1, 1, 1, 4, "silu", n),
              lambda n: N._desc(x, x, n, 1, 1, 1, "none", 1e-5, None)):
        with pytest.raises(ValueError, match="2\\^31"):
            q(many)
        q(1)


def test_gradients_under_other_names_are_refused():
    """A caller's output tensor under a name that is no gradient's would stay as it was."""
    import torch
    from linear_rnn_sequence_wkv7_amd import _marshal
    x, w = torch.zeros(2, 3, 8), torch.zeros(8, 4)
    wanted = (("x", x, None, None), ("w", w, None, None), ("bias", None, None, None))
    out = _marshal.gradients({"x": x.clone(), "w": None, "bias": None}, wanted, x.device)
    assert out["w"] is not None and out["bias"] is None
    for name in ("X", "dw", "dx"):
        with pytest.raises(ValueError, match=f"no {name}; its keys are x, w, bias"):
            _marshal.gradients({name: x}, wanted, x.device)


def test_python_bindings_refuse_wrong_tensors():
    """Shapes, types and devices are checked before the library is called."""
    import torch
    x = torch.zeros(2, 3, 8)
    A, Bm = torch.zeros(8, 4), torch.zeros(2, 3, 1, 4)
    with pytest.raises(ValueError, match="GPU"):
        S.ssm_forward(x, x, A, Bm, Bm)
    with pytest.raises(ValueError, match="dimensions"):
        S.ssm_forward(x[0], x, A, Bm, Bm)
    with pytest.raises(ValueError, match="dimensions"):
        S.ssm_step(x, x, A, Bm, Bm, torch.zeros(2, 8, 4))
    with pytest.raises(ValueError, match="GPU"):
        K.shortconv_forward(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="GPU"):
        N.groupnorm_forward(x, 2)
