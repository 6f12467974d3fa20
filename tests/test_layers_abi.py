"""C ABI of the lookup, the layer norm, the router and the weighted sum: exported symbols and refusals on the host,
before any HIP call (CPU only), and the compiled kernels' registers."""
import os
import re
import subprocess

import pytest
import torch

import edge_node_scatter_amd as zs
from edge_node_scatter_amd import build as zs_build
from edge_node_scatter_amd import layers

NULL, SHAPE, UNSUPPORTED, ALIAS, WORKSPACE = -1, -2, -4, -5, -6
# fake device addresses, 64 GiB apart: every call below fails its host checks, so none is used
A, B, C, D, E, F, G, H, I, J = (0x700000000000 + (i << 36) for i in range(10))


@pytest.fixture(scope="module")
def lib():
    return layers.load_layers()


def test_header_symbols_exported(lib):
    text = open(layers.LAYERS_HEADER_PATH).read()
    declared = set(re.findall(r"^\w[\w\s\*]*?\b(zs_\w+)\s*\(", text, flags=re.M))
    assert declared == {"zs_embedding", "zs_embedding_backward_workspace_bytes", "zs_embedding_backward", "zs_layer_norm",
                        "zs_layer_norm_workspace_bytes", "zs_layer_norm_backward", "zs_route", "zs_route_backward", "zs_combine",
                        "zs_combine_backward"}
    out = subprocess.check_output(["nm", "-D", "--defined-only", zs.LIB_PATH], text=True)
    assert declared <= {line.split()[-1] for line in out.splitlines() if " T " in line}


def test_constants_match_the_header():
    text = open(layers.LAYERS_HEADER_PATH).read()
    value = lambda name: int(re.search(rf"#define {name} +(\d+)", text).group(1))  # noqa: E731
    assert value("ZS_MAX_LAYER_WIDTH") == layers.MAX_LAYER_WIDTH and value("ZS_MAX_EXPERTS") == layers.MAX_EXPERTS
    assert value("ZS_MAX_SLOTS") == layers.MAX_SLOTS and value("ZS_MAX_EXPERT_GROUPS") == layers.MAX_EXPERT_GROUPS


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "zs_layers.h"\nint main(void) { return (int)sizeof(zs_router) - 28; }\n')
    exe = tmp_path / "t"
    subprocess.check_call(["gcc", "-std=c11", "-Wall", "-Werror", "-I", zs_build.INCLUDE, str(src), "-o", str(exe)])
    assert subprocess.call([str(exe)]) == 0
    import ctypes
    assert ctypes.sizeof(layers._Router) == 28


def test_embedding_rejects(lib):
    base = dict(t=A, ld=16, idx=B, M=10, V=7, c=16, scale=1.0, dt=0, y=C, s=None)

    def f(**kw):
        return lib.zs_embedding(*{**base, **kw}.values())
    for kw in (dict(M=-1), dict(M=1 << 31), dict(V=0), dict(V=1 << 31), dict(c=0), dict(c=8193), dict(ld=-1), dict(ld=1 << 60)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(t=None), dict(idx=None), dict(y=None)):
        assert f(**kw) == NULL, kw
    for kw in (dict(dt=2), dict(t=A + 2), dict(idx=B + 4), dict(y=C + 1), dict(dt=1, t=A + 1)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(y=A), dict(y=A + 4 * 111), dict(y=B + 72), dict(ld=1000, y=A + 4 * 6015)):
        assert f(**kw) == ALIAS, kw
    assert f(M=0, t=None, idx=None, y=None) == 0


def test_embedding_backward_rejects(lib):
    size = lib.zs_embedding_backward_workspace_bytes
    assert size(-1, 8, 0) == 0 and size(10, 0, 0) == 0 and size(10, 8, 5) == 0 and size(0, 8, 0) == 0 and size(8, 8192, 0) == 0   # one workgroup leaves nothing
    need = size(100000, 16, 0)
    assert need > 0
    base = dict(gy=A, ld=16, idx=B, off=C, perm=D, M=100000, V=7, c=16, scale=1.0, dt=0, g=E, ws=F, nb=need, s=None)

    def f(**kw):
        return lib.zs_embedding_backward(*{**base, **kw}.values())
    for kw in (dict(M=-1), dict(M=1 << 31), dict(V=0), dict(c=0), dict(c=8193), dict(ld=-1), dict(ld=1 << 60)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(gy=None), dict(idx=None), dict(off=None), dict(g=None)):
        assert f(**kw) == NULL, kw
    for kw in (dict(dt=7), dict(gy=A + 2), dict(idx=B + 4), dict(off=C + 1), dict(perm=D + 2), dict(g=E + 3), dict(ws=F + 16)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(ws=None), dict(nb=need - 1)):
        assert f(**kw) == WORKSPACE, kw
    for kw in (dict(g=A), dict(g=C + 28), dict(ws=E), dict(g=F + 256), dict(ws=D + 256)):
        assert f(**kw) == ALIAS, kw


def test_layer_norm_rejects(lib):
    base = dict(x=A, ld=16, w=B, b=C, M=4, c=16, eps=1e-5, dt=0, y=D, s=None)

    def f(**kw):
        return lib.zs_layer_norm(*{**base, **kw}.values())
    for kw in (dict(M=-1), dict(c=0), dict(c=8193), dict(ld=-1), dict(ld=1 << 61), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(w=None), dict(y=None)):
        assert f(**kw) == NULL, kw
    for kw in (dict(dt=9), dict(x=A + 2), dict(w=B + 1), dict(b=C + 2), dict(y=D + 2)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(y=A), dict(y=B + 32), dict(y=C)):
        assert f(**kw) == ALIAS, kw
    assert f(M=0) == 0
    need = lib.zs_layer_norm_workspace_bytes(400, 16)
    assert need > 0 and lib.zs_layer_norm_workspace_bytes(1, 8192) == 0   # one workgroup's sums are the gradients
    assert lib.zs_layer_norm_workspace_bytes(4, 0) == 0 and lib.zs_layer_norm_workspace_bytes(-1, 8) == 0
    back = dict(gy=A, lg=16, x=B, ld=16, w=C, M=400, c=16, eps=1e-5, dt=0, gx=D, gw=E, gb=F, ws=G, nb=need, s=None)

    def g(**kw):
        return lib.zs_layer_norm_backward(*{**back, **kw}.values())
    for kw in (dict(M=-1), dict(c=0), dict(eps=-1.0), dict(lg=-2), dict(ld=-2)):
        assert g(**kw) == SHAPE, kw
    for kw in (dict(gy=None), dict(x=None), dict(w=None), dict(gx=None), dict(gw=None)):
        assert g(**kw) == NULL, kw
    for kw in (dict(dt=3), dict(gy=A + 1), dict(gx=D + 2), dict(gw=E + 2), dict(gb=F + 1), dict(ws=G + 8)):
        assert g(**kw) == UNSUPPORTED, kw
    for kw in (dict(ws=None), dict(nb=need - 1)):
        assert g(**kw) == WORKSPACE, kw
    for kw in (dict(gx=A), dict(gw=C), dict(gb=E + 32), dict(ws=B), dict(ws=D)):
        assert g(**kw) == ALIAS, kw


ROUTER = dict(k=2, sigmoid=0, groups=4, top_groups=2, best=2, renormalise=1, scale=1.0)


def test_route_rejects(lib):
    base = dict(x=A, ld=16, b=B, r=ROUTER, M=10, n=16, dt=0, w=C, e=D, s=None)

    def f(**kw):
        a = {**base, **kw}
        a["r"] = None if a["r"] is None else layers._Router(*{**ROUTER, **a["r"]}.values())
        return lib.zs_route(*a.values())
    for r in (dict(k=0), dict(k=9), dict(k=65), dict(groups=0), dict(groups=3), dict(groups=65), dict(top_groups=0), dict(top_groups=5), dict(best=0), dict(best=3),
              dict(sigmoid=2), dict(renormalise=-1), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert f(r=r) == SHAPE, r
    for kw in (dict(M=-1), dict(M=1 << 31), dict(M=(1 << 31) - 1), dict(n=0), dict(n=1028), dict(ld=-1), dict(ld=1 << 60)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(w=None), dict(e=None), dict(r=None)):
        assert f(**kw) == NULL, kw
    for kw in (dict(dt=2), dict(x=A + 2), dict(b=B + 2), dict(w=C + 1), dict(e=D + 4)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(w=A), dict(e=A + 64), dict(e=C), dict(w=B)):
        assert f(**kw) == ALIAS, kw
    assert f(M=0, x=None, w=None, e=None) == 0
    back = dict(gw=A, x=B, ld=16, e=C, r=ROUTER, M=10, n=16, dt=0, gx=D, s=None)

    def g(**kw):
        a = {**back, **kw}
        a["r"] = None if a["r"] is None else layers._Router(*{**ROUTER, **a["r"]}.values())
        return lib.zs_route_backward(*a.values())
    assert g(r=dict(k=9)) == SHAPE and g(M=-1) == SHAPE and g(ld=-1) == SHAPE
    for kw in (dict(gw=None), dict(x=None), dict(e=None), dict(gx=None), dict(r=None)):
        assert g(**kw) == NULL, kw
    for kw in (dict(dt=2), dict(gw=A + 2), dict(x=B + 1), dict(e=C + 4), dict(gx=D + 2)):
        assert g(**kw) == UNSUPPORTED, kw
    for kw in (dict(gx=A), dict(gx=B + 64), dict(gx=C)):
        assert g(**kw) == ALIAS, kw


def test_combine_rejects(lib):
    base = dict(z=A, ld=16, w=B, M=10, k=2, c=16, dt=0, y=C, s=None)

    def f(**kw):
        return lib.zs_combine(*{**base, **kw}.values())
    for kw in (dict(M=-1), dict(M=1 << 30, k=4), dict(k=0), dict(k=65), dict(c=0), dict(c=8193), dict(ld=-1), dict(ld=1 << 60)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(z=None), dict(w=None), dict(y=None)):
        assert f(**kw) == NULL, kw
    for kw in (dict(dt=2), dict(z=A + 2), dict(w=B + 2), dict(y=C + 1)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(y=A), dict(y=A + 4 * 319), dict(y=B + 4)):
        assert f(**kw) == ALIAS, kw
    assert f(M=0, z=None, w=None, y=None) == 0
    back = dict(gy=A, lg=16, z=B, ld=16, w=C, M=10, k=2, c=16, dt=0, gz=D, gw=E, s=None)

    def g(**kw):
        return lib.zs_combine_backward(*{**back, **kw}.values())
    assert g(k=0) == SHAPE and g(lg=-1) == SHAPE and g(lg=1 << 60) == SHAPE
    for kw in (dict(gy=None), dict(z=None), dict(w=None), dict(gz=None), dict(gw=None)):
        assert g(**kw) == NULL, kw
    for kw in (dict(dt=2), dict(gy=A + 2), dict(z=B + 1), dict(w=C + 2), dict(gz=D + 1), dict(gw=E + 2)):
        assert g(**kw) == UNSUPPORTED, kw
    for kw in (dict(gz=A), dict(gz=B + 4), dict(gw=C), dict(gw=D + 64)):
        assert g(**kw) == ALIAS, kw


def test_router_refusals():
    for kw in (dict(n_experts=0, k=1), dict(n_experts=1025, k=1), dict(n_experts=16, k=0), dict(n_experts=16, k=17), dict(n_experts=128, k=65), dict(n_experts=16, k=2, score="max"),
               dict(n_experts=16, k=2, groups=3), dict(n_experts=16, k=2, groups=4, top_groups=5), dict(n_experts=16, k=2, groups=4, top_groups=0),
               dict(n_experts=16, k=5, groups=4, top_groups=1), dict(n_experts=128, k=1, groups=128), dict(n_experts=16, k=2, best=3), dict(n_experts=16, k=2, scale=float("nan"))):
        with pytest.raises(ValueError):
            zs.Router(**kw)
    zs.Router(1, 1), zs.Router(1024, 64, groups=64, top_groups=64)
    r = zs.Router(16, 2)
    with pytest.raises(AttributeError):   # outputs are sized by what the library was told
        r.k = 4


def test_cpu_tensors_are_refused():
    x, idx, w = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(8)
    r = zs.Router(8, 2)
    for call in (lambda: zs.zs_embedding(x, idx), lambda: zs.zs_embedding_backward(x, idx, 4), lambda: zs.zs_layer_norm(x, w), lambda: zs.zs_layer_norm_backward(x, x, w),
                 lambda: zs.zs_route(x, r), lambda: zs.zs_route_backward(x, x, idx, r), lambda: zs.expert_groups(idx[:, None], 8), lambda: zs.zs_combine(x, w),
                 lambda: zs.zs_combine_backward(x, x, w)):
        with pytest.raises(ValueError):
            call()


def test_kernels_keep_their_values_in_registers(tmp_path):
    """No kernel of these sources spills or uses scratch, and none has packed fp32 instructions or atomics."""
    seen = 0
    for path in zs_build.device_asm(str(tmp_path)):
        if not os.path.basename(path).startswith(("zs_embed", "zs_lnorm", "zs_route", "zs_combine")):
            continue
        text = open(path).read()
        assert not re.search(r"\bv_pk_(?:fma|mul|add)_f32\b", text), path
        assert not re.search(r"\b(?:global|flat|buffer)_atomic", text), path
        for m in re.finditer(r"\.vgpr_spill_count:\s+(\d+)", text):
            seen += 1
            assert m.group(1) == "0", path
        assert not re.search(r"\.private_segment_fixed_size:\s+[1-9]", text), path
    assert seen > 60
