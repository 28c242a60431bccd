"""The C ABI of linear attention and the layer norm: exported symbols, structure layouts, size queries and
refusals before any device is touched (CPU only); the refusals of their Python bindings; and the rules on
linear attention's kernel sources."""
import ctypes
import os
import re
import subprocess

import pytest

from linear_rnn_sequence_wkv7_amd import layernorm as N
from linear_rnn_sequence_wkv7_amd import linattn as L
from linear_rnn_sequence_wkv7_amd import wkv7 as W
from tests.test_seq_abi import declared

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KERNELS = os.path.join(ROOT, "linear_rnn_sequence_wkv7_amd", "csrc", "linattn")
needs_library = pytest.mark.skipif(not os.path.exists(W.lib_path()), reason="libwkv7.so not built")

SP = 1 << 26          # 64 MiB between fake arrays: disjoint unless a test makes them overlap
BASE = 1 << 36        # never dereferenced: every case below fails validation, or has nothing to do

CALLS = {
    # function: (pointer names in order, optional ones, written ones, pairs that may be one array)
    "linattn_forward": ("q k v g state_in y state_out workspace", "state_in state_out", "y state_out workspace", ("state_out", "state_in")),
    "linattn_step": ("q k v g state state_index y", "state_index", "state y", ()),
    "linattn_backward": ("q k v g state_in dy dstate_out dq dk dv dg dstate_in workspace", "state_in dstate_out dg dstate_in",
                         "dq dk dv dg dstate_in workspace", ()),
    "layernorm_forward": ("x residual weight bias h y mean rstd", "residual weight bias h mean rstd", "h y mean rstd", ("h", "residual")),
    "layernorm_backward": ("h weight bias dy dh mean rstd dresidual dx dweight dbias workspace", "weight bias dh dx dweight dbias",
                           "dresidual dx dweight dbias workspace", ("dresidual", "dh")),
}
TOGETHER = {"layernorm_forward": [("residual", "h"), ("h", "residual"), ("mean", "rstd"), ("rstd", "mean")],
            "layernorm_backward": [("dweight", "weight"), ("dbias", "bias")]}


def desc(fn, **kw):
    if fn.startswith("linattn"):
        step = fn.endswith("step")
        d = dict(B=2, T=1 if step else 4000, H=4, Hq=2, Hk=1, Hv=4, Dk=24, Dv=40, in_dtype=1, y_dtype=1, g_per_token=1, S=5, scale=1.0)
        return L.LinattnDesc(**{**d, **kw})
    return N.LayernormDesc(**{**dict(B=2, T=70, C=64, x_dtype=1, h_dtype=1, y_dtype=1, eps=1e-5), **kw})


def call(fn, d=None, **over):
    names = CALLS[fn][0]
    L._lib(), N._lib()
    d = desc(fn) if d is None else d
    args = []
    for i, n in enumerate(names.split()):
        args.append(over[n] if n in over else BASE + i * SP)
        if n == "workspace":
            args.append(over.get("ws_bytes", SP))
    return getattr(W.load_library(), fn)(None if over.get("no_desc") else ctypes.byref(d), *args, None)


def message():
    return W.load_library().wkv7_last_error().decode()


@needs_library
@pytest.mark.parametrize("header,mod", [("linattn.h", L), ("layernorm.h", N)])
def test_every_declared_symbol_is_exported(header, mod):
    names = declared(header)
    assert names == set(mod.EXPORTED_SYMBOLS)
    for n in names:
        assert hasattr(W.load_library(), n), n


def test_structures_match_the_headers(tmp_path):
    """Sizes and offsets as a C compiler sees them."""
    fields = {"linattn": L.LinattnDesc, "layernorm": N.LayernormDesc}
    lines = ['#include <stdio.h>', '#include <stddef.h>'] + [f'#include "{n}.h"' for n in fields] + ["int main(void) {"]
    for n, st in fields.items():
        lines.append(f'printf("{n} %zu\\n", sizeof({n}_desc));')
        lines += [f'printf("{n}.{f[0]} %zu\\n", offsetof({n}_desc, {f[0]}));' for f in st._fields_]
    prog, exe = tmp_path / "layout.c", tmp_path / "layout"
    prog.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    out = dict(l.split() for l in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    for n, st in fields.items():
        assert int(out[n]) == ctypes.sizeof(st)
        for f in st._fields_:
            assert int(out[f"{n}.{f[0]}"]) == getattr(st, f[0]).offset, f


@needs_library
@pytest.mark.parametrize("fn", CALLS)
def test_pointers(fn):
    names, optional = CALLS[fn][0].split(), CALLS[fn][1].split()
    assert call(fn, no_desc=True) == W.WKV7_EINVAL
    for n in names:
        if n not in optional:
            assert call(fn, **{n: None}) == W.WKV7_EINVAL, n
            assert f"{n} is NULL" in message()
        assert call(fn, **{n: BASE + 2 if n == "state_index" else BASE + 4}) == W.WKV7_EINVAL, n
        assert f"{n} is not" in message(), n
    for a, b in TOGETHER.get(fn, ()):
        assert call(fn, **{a: None}) == W.WKV7_EINVAL, (a, b)
        assert a in message()


@needs_library
@pytest.mark.parametrize("fn", CALLS)
def test_written_arrays_share_no_byte(fn):
    names, _, written, pair = CALLS[fn]
    names = names.split()
    at = {n: BASE + i * SP for i, n in enumerate(names)}
    for w in written.split():
        for o in names:
            if o == w or {w, o} == set(pair):
                continue   # in place is allowed
            assert call(fn, **{w: at[o]}) == W.WKV7_EINVAL, (w, o)
            assert "overlaps" in message(), (w, o)
    if pair:   # in place, but not half, and with no third array
        moved, source = pair
        assert call(fn, **{moved: at[source] + 16}) == W.WKV7_EINVAL and "overlaps" in message()
        for o in names:
            if o not in pair:
                assert call(fn, **{moved: at[source], o: at[source]}) == W.WKV7_EINVAL, o
                assert "overlaps" in message() and o in message(), o


@needs_library
@pytest.mark.parametrize("fn", ["linattn_forward", "linattn_backward", "layernorm_backward"])
def test_workspace_sizes(fn):
    d = desc(fn)
    lib = (L._lib(), N._lib())[0]
    need = {"linattn_forward": lib.linattn_workspace_bytes, "linattn_backward": lib.linattn_backward_workspace_bytes,
            "layernorm_backward": lib.layernorm_backward_workspace_bytes}[fn](ctypes.byref(d))
    assert need > 0
    assert call(fn, ws_bytes=need - 1) == W.WKV7_EINVAL
    assert f"{need} needed" in message()


ATTN_BAD = [(dict(B=-1), 1), (dict(T=-1), 1), (dict(H=-1), 1), (dict(Hq=-1), 1), (dict(Hk=-4), 1), (dict(Hv=-1), 1), (dict(Hq=3), 1), (dict(Hk=8), 1),
            (dict(Hv=3), 1), (dict(H=0), 1), (dict(Dk=0), 1), (dict(Dv=-1), 1), (dict(Dk=129), 2), (dict(Dv=256), 2), (dict(in_dtype=2), 1),
            (dict(y_dtype=-1), 1), (dict(g_per_token=2), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(reserved=1), 1),
            (dict(lengths=BASE + 2), 1), (dict(H=1 << 16), 2), (dict(B=1 << 28, H=1 << 12), 2), (dict(T=2147483647), 2),
            (dict(B=1 << 30, T=1 << 10), 2)]
NORM_BAD = [(dict(B=-1), 1), (dict(T=-1), 1), (dict(C=-1), 1), (dict(x_dtype=2), 1), (dict(h_dtype=-1), 1), (dict(y_dtype=7), 1), (dict(eps=0.0), 1),
            (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(reserved=2), 1), (dict(lengths=BASE + 3), 1), (dict(C=1 << 24), 2),
            (dict(B=1 << 30, T=1 << 20), 2)]


@needs_library
@pytest.mark.parametrize("fn", CALLS)
def test_descriptors(fn):
    for kw, code in ATTN_BAD if fn.startswith("linattn") else NORM_BAD:
        if fn == "linattn_step" and "T" in kw:
            code = W.WKV7_EINVAL
        assert call(fn, desc(fn, **kw)) == code, kw
        assert message()
    if fn == "linattn_step":
        assert call(fn, desc(fn, T=2)) == W.WKV7_EINVAL
        assert call(fn, desc(fn, lengths=BASE)) == W.WKV7_EINVAL
        assert call(fn, desc(fn, S=-1)) == W.WKV7_EINVAL
        assert call(fn, desc(fn, S=1), state_index=None) == W.WKV7_EINVAL
        assert "state_index" in message()
    if fn == "layernorm_forward":
        assert call(fn, desc(fn, x_dtype=0), residual=None, h=None) == W.WKV7_EINVAL
        assert "h_dtype" in message()


@needs_library
def test_refuses_more_threads_than_a_launch_takes():
    far = lambda fn: {n: BASE + (i << 45) if n not in CALLS[fn][1].split() else None for i, n in enumerate(CALLS[fn][0].split())}
    wide = dict(H=1, Hq=1, Hk=1, Hv=1, Dk=1, Dv=1)
    for fn, kw in (("linattn_forward", dict(B=1 << 25, T=1)), ("linattn_step", dict(B=1 << 26, T=1, S=1 << 26)), ("linattn_backward", dict(B=1 << 25, T=1))):
        assert call(fn, desc(fn, **{**wide, **kw}), **far(fn), ws_bytes=1 << 50) == W.WKV7_EUNSUPPORTED, fn
        assert "2^32" in message()


@needs_library
def test_lengths_need_the_alignment_of_an_int32():
    for off in (4, 8, 12):
        assert call("linattn_forward", desc("linattn_forward", B=0, lengths=BASE + off)) == W.WKV7_OK
        assert call("layernorm_forward", desc("layernorm_forward", B=0, lengths=BASE + off)) == W.WKV7_OK
        assert call("linattn_step", desc("linattn_step", B=0), state_index=BASE + off) == W.WKV7_OK


@needs_library
def test_nothing_to_do_needs_no_device():
    none = dict(H=0, Hq=0, Hk=0, Hv=0)
    assert call("linattn_forward", desc("linattn_forward", B=0)) == W.WKV7_OK
    assert call("linattn_forward", desc("linattn_forward", T=0), state_out=None) == W.WKV7_OK
    assert call("linattn_forward", desc("linattn_forward", **none)) == W.WKV7_OK
    assert call("linattn_step", desc("linattn_step", B=0)) == W.WKV7_OK
    assert call("linattn_backward", desc("linattn_backward", **none)) == W.WKV7_OK
    assert call("layernorm_forward", desc("layernorm_forward", T=0)) == W.WKV7_OK
    assert call("layernorm_forward", desc("layernorm_forward", C=0), mean=None, rstd=None) == W.WKV7_OK
    assert call("layernorm_backward", desc("layernorm_backward", C=0)) == W.WKV7_OK


@needs_library
def test_size_queries():
    for dims in ((2, 0, 4, 8, 8), (0, 70, 4, 8, 8), (2, 70, 0, 8, 8)):
        assert L.linattn_backward_workspace_bytes(*dims) == 0
    assert L.linattn_workspace_bytes(64, 4096, 32, 64, 64) == 0          # enough heads: one part
    assert L.linattn_workspace_bytes(1, 4096, 1, 64, 64) > 0
    one, shared = (L.linattn_backward_workspace_bytes(64, 64, 32, 64, 64, Hq=h) for h in (32, 8))
    assert shared >= one + 64 * 64 * 32 * 64 * 4                         # each head's dq
    for dims in ((2, 0, 64), (0, 70, 64), (2, 70, 0)):
        assert N.layernorm_backward_workspace_bytes(*dims) == 0
    assert N.layernorm_backward_workspace_bytes(1, 1, 5) >= 2 * 5 * 4
    for q in (lambda: L.linattn_workspace_bytes(2, -1, 4, 8, 8), lambda: L.linattn_backward_workspace_bytes(2, 1, 4, 8, 129),
              lambda: L.linattn_workspace_bytes(2, 1, 4, 8, 8, Hq=3), lambda: N.layernorm_backward_workspace_bytes(-1, 1, 1)):
        with pytest.raises(W.Wkv7Error):
            q()


@needs_library
def test_bindings_refuse_sizes_past_an_int32():
    """2^32 + 5 rows are not 5."""
    import torch
    x, many = torch.zeros(2, 3, 8), (1 << 32) + 5
    for q in (lambda n: L.linattn_workspace_bytes(n, 1, 1, 1, 1), lambda n: L.linattn_backward_workspace_bytes(1, n, 1, 1, 1),
              lambda n: L._desc(x, x, x, (None, n, 1, 1, 1, 1, 1, 1, 1), 1.0), lambda n: L._desc(x, x, x, (None,) + (1,) * 8, 1.0, None, n),
              lambda n: N.layernorm_backward_workspace_bytes(n, 1, 1), lambda n: N._desc(1, n, 1, x, x, x, 1.0, None)):
        with pytest.raises(ValueError, match="2\\^31"):
            q(many)
        q(1)


def test_python_bindings_refuse_wrong_tensors():
    """Shapes, types and devices are checked before the library is called."""
    import torch
    q, g = torch.zeros(2, 3, 4, 8), torch.zeros(2, 3, 4)
    with pytest.raises(ValueError, match="GPU"):
        L.linattn_forward(q, q, q, g)
    with pytest.raises(ValueError, match="dimensions"):
        L.linattn_forward(q[0], q, q, g)
    with pytest.raises(ValueError, match="dimensions"):
        L.linattn_step(q, q, q, g, torch.zeros(2, 4, 8, 8))
    with pytest.raises(ValueError, match="GPU"):
        N.layernorm_forward(torch.zeros(2, 3, 8))
    with pytest.raises(ValueError, match="dimensions"):
        N.layernorm_forward(torch.zeros(2, 8))


def _code(name):
    src = open(os.path.join(KERNELS, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", src, flags=re.S))


def test_one_mfma_opcode_per_source():
    """As for the recurrences' sources: no accumulator chain mixes shapes, nothing in inline asm, no packed fp32."""
    found = {}
    for name in sorted(os.listdir(KERNELS)):
        code = _code(name)
        assert not re.search(r"\bv_mfma_\w+|__builtin_amdgcn_smfmac_\w+|v_pk_(add|mul|fma)_f32", code), name
        builtins = set(re.findall(r"__builtin_amdgcn_mfma_\w+", code))
        assert len(builtins) <= 1, name
        if builtins:
            found[name] = builtins.pop()
    assert found == {"linattn_bf16.hip": "__builtin_amdgcn_mfma_f32_16x16x32_bf16", "linattn_f32.hip": "__builtin_amdgcn_mfma_f32_16x16x4f32"}
