"""C ABI of the grouped products, the residual join and AdamW: exported symbols and refusals on the host, before any
HIP call (CPU only), and the compiled kernels' registers."""
import ctypes
import os
import re
import subprocess

import pytest

import edge_node_scatter_amd as zs
from edge_node_scatter_amd import block
from edge_node_scatter_amd import build as zs_build

NULL, SHAPE, UNSUPPORTED, ALIAS, WORKSPACE = -1, -2, -4, -5, -6
# fake device addresses, 64 GiB apart: every call below fails its host checks, so none is used
A, B, C, D, E, F, G, H, I, J = (0x700000000000 + (i << 36) for i in range(10))


@pytest.fixture(scope="module")
def lib():
    return block.load_block()


def test_header_symbols_exported(lib):
    text = open(block.BLOCK_HEADER_PATH).read()
    declared = set(re.findall(r"^\w[\w\s\*]*?\b(zs_\w+)\s*\(", text, flags=re.M))
    assert declared == {"zs_grouped_mm", "zs_grouped_mm_wgrad_workspace_bytes", "zs_grouped_mm_wgrad", "zs_grouped_mm_backward", "zs_block_join",
                        "zs_block_join_workspace_bytes", "zs_block_join_backward", "zs_adamw_step", "zs_adamw_step8",
                        "zs_adamw_moments8"}
    out = subprocess.check_output(["nm", "-D", "--defined-only", zs.LIB_PATH], text=True)
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert declared <= exported


def test_constants_match_the_header():
    text = open(block.BLOCK_HEADER_PATH).read()
    value = lambda name: int(re.search(rf"#define {name} +(\d+)", text).group(1))  # noqa: E731
    assert value("ZS_MAX_GROUPS") == block.MAX_GROUPS and value("ZS_MAX_WIDTH") == block.MAX_WIDTH
    assert value("ZS_MAX_JOIN_WIDTH") == block.MAX_JOIN_WIDTH and value("ZS_ADAMW_BLOCK") == block.STATE_BLOCK


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "zs_block.h"\nint main(void) { return (int)sizeof(zs_adamw_tensor) - 48; }\n')
    exe = tmp_path / "t"
    subprocess.check_call(["gcc", "-std=c11", "-Wall", "-Werror", "-I", zs_build.INCLUDE, str(src), "-o", str(exe)])
    assert subprocess.call([str(exe)]) == 0
    assert ctypes.sizeof(block._Tensor) == 48


def test_grouped_mm_rejects(lib):
    base = dict(x=A, ldx=8, w=B, wg=64, ldw=8, t=0, off=C, perm=D, M=10, G=3, k=8, n=8, dt=0, y=E, ldy=8, s=None)

    def f(**kw):
        return lib.zs_grouped_mm(*{**base, **kw}.values())
    for kw in (dict(M=-1), dict(M=1 << 31), dict(G=0), dict(G=(1 << 20) + 1), dict(k=0), dict(n=0), dict(k=65537), dict(n=65537),
               dict(ldx=-1), dict(ldy=7), dict(ldw=-8), dict(wg=-1), dict(ldx=1 << 60), dict(ldy=1 << 62), dict(wg=1 << 60)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(w=None), dict(off=None), dict(y=None)):
        assert f(**kw) == NULL, kw
    for kw in (dict(dt=2), dict(dt=-1), dict(x=A + 2), dict(w=B + 1), dict(y=E + 3), dict(off=C + 2), dict(perm=D + 1), dict(dt=1, x=A + 1)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(y=A), dict(y=A + 4 * 72), dict(y=B + 4 * 191), dict(y=C + 12), dict(y=D + 36), dict(ldy=1000, y=A - 4000)):
        assert f(**kw) == ALIAS, kw
    assert f(M=0, x=None, y=None, perm=None) == 0


def test_wgrad_rejects(lib):
    size = lib.zs_grouped_mm_wgrad_workspace_bytes
    assert size(-1, 3, 8, 8, 0) == 0 and size(10, 3, 8, 8, 5) == 0 and size(10, 3, 8, 8, 0) == 0
    need = size(100000, 3, 8, 8, 0)
    assert need > 0
    base = dict(x=A, ldx=8, gy=B, ldg=8, off=C, perm=D, M=100000, G=3, k=8, n=8, dt=0, gw=E, ws=F, nb=need, s=None)

    def f(**kw):
        return lib.zs_grouped_mm_wgrad(*{**base, **kw}.values())
    for kw in (dict(M=-1), dict(G=0), dict(k=0), dict(n=65537), dict(ldx=-1), dict(ldg=-1), dict(ldg=1 << 60)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(gy=None), dict(off=None), dict(gw=None)):
        assert f(**kw) == NULL, kw
    for kw in (dict(dt=3), dict(x=A + 2), dict(gw=E + 1), dict(ws=F + 8)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(ws=None), dict(nb=need - 1), dict(nb=0)):
        assert f(**kw) == WORKSPACE, kw
    for kw in (dict(gw=A), dict(gw=F + 16), dict(ws=B + 256), dict(ws=D)):
        assert f(**kw) == ALIAS, kw


def test_both_gradients_reject(lib):
    need = lib.zs_grouped_mm_wgrad_workspace_bytes(100000, 3, 8, 8, 0)
    base = dict(gy=A, ldg=8, x=B, ldx=8, w=C, wg=64, ldw=8, off=D, perm=E, M=100000, G=3, k=8, n=8, dt=0, gx=F, gw=G, ws=H, nb=need, s=None)

    def f(**kw):
        return lib.zs_grouped_mm_backward(*{**base, **kw}.values())
    for kw in (dict(M=-1), dict(G=0), dict(k=0), dict(n=65537), dict(ldx=-1), dict(ldg=-1), dict(ldw=-1), dict(wg=-1), dict(wg=1 << 60)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(gy=None), dict(w=None), dict(off=None), dict(gx=None), dict(gw=None)):
        assert f(**kw) == NULL, kw
    for kw in (dict(dt=3), dict(x=B + 2), dict(w=C + 1), dict(gx=F + 2), dict(ws=H + 8)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(ws=None), dict(nb=need - 1)):
        assert f(**kw) == WORKSPACE, kw
    for kw in (dict(gw=C), dict(gx=B), dict(gx=A + 32), dict(gw=F + 64), dict(ws=G), dict(gx=E)):
        assert f(**kw) == ALIAS, kw


def test_join_rejects(lib):
    base = dict(x=A, ldx=16, z=B, ldz=16, g=C, ldg=16, gw=16, sc=D, po=D + 256, pr=D + 512, M=4, c=16, eps=1e-6, dt=0, y=E, h=F, s=None)

    def f(**kw):
        return lib.zs_block_join(*{**base, **kw}.values())
    for kw in (dict(M=-1), dict(c=0), dict(c=8193), dict(gw=2), dict(gw=-1), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(ldx=-1), dict(ldz=-4), dict(ldg=-1), dict(ldx=1 << 61)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(g=None), dict(sc=None), dict(po=None), dict(y=None), dict(h=None), dict(z=None, pr=None)):
        assert f(**kw) == NULL, kw
    for kw in (dict(dt=9), dict(x=A + 2), dict(z=B + 1), dict(g=C + 2), dict(sc=D + 1), dict(y=E + 2), dict(h=F + 1)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(y=A), dict(h=E), dict(h=B + 64), dict(y=C), dict(h=D + 512)):
        assert f(**kw) == ALIAS, kw
    assert f(M=0) == 0
    need = lib.zs_block_join_workspace_bytes(4, 16)
    assert need > 0 and lib.zs_block_join_workspace_bytes(4, 0) == 0 and lib.zs_block_join_workspace_bytes(-1, 8) == 0
    back = dict(gy=G, gh=G + 4096, x=A, ldx=16, z=B, ldz=16, g=C, ldg=16, gw=16, sc=D, po=D + 256, pr=D + 512, M=4, c=16, eps=1e-6, dt=0,
                gx=E, gz=F, gg=H, gsc=I, gpo=I + 256, gpr=I + 512, ws=J, nb=need, s=None)

    def b(**kw):
        return lib.zs_block_join_backward(*{**back, **kw}.values())
    assert b(c=0) == SHAPE and b(eps=-1.0) == SHAPE
    for kw in (dict(gx=None), dict(gz=None), dict(gg=None), dict(gsc=None), dict(gpo=None), dict(gpr=None), dict(x=None)):
        assert b(**kw) == NULL, kw
    for kw in (dict(gy=G + 1), dict(gsc=I + 2), dict(ws=J + 4)):
        assert b(**kw) == UNSUPPORTED, kw
    for kw in (dict(ws=None), dict(nb=need - 1)):
        assert b(**kw) == WORKSPACE, kw
    for kw in (dict(gx=G), dict(gz=E + 4), dict(gg=A), dict(gsc=I + 300), dict(ws=G), dict(gx=G + 4096)):
        assert b(**kw) == ALIAS, kw


def test_adamw_rejects(lib):
    def call(tensors, m=A, v=B, total=512, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, step=1, bits=32, none=False):
        t = (block._Tensor * max(1, len(tensors)))(*[block._Tensor(*x) for x in tensors])
        c = block._Config(lr, b1, b2, eps, wd, step)
        t = None if none else t
        if bits == 32:
            return lib.zs_adamw_step(t, len(tensors), c, m, v, total, None)
        return lib.zs_adamw_step8(t, len(tensors), c, m, A + (1 << 20), v, B + (1 << 20), total, 0, None)
    ok = (C, D, E, 100, 0, 0, 0)   # param, grad, copy, n, offset, grad type, reserved
    for kw in (dict(lr=-1.0), dict(lr=float("nan")), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=float("nan")), dict(eps=-1.0),
               dict(wd=-1.0), dict(step=0), dict(total=-1), dict(total=99)):
        assert call([ok], **kw) == SHAPE, kw
    for t in ((C, D, E, -1, 0, 0, 0), (C, D, E, 100, 128, 0, 0), (C, D, E, 100, 512, 0, 0), (C, D, E, 600, 0, 0, 0)):
        assert call([t]) == SHAPE, t
    assert call([ok, (F, G, H, 10, 0, 0, 0)]) == SHAPE            # slices in one another
    assert call([(C, D, E, 10, 256, 0, 0), (F, G, H, 10, 0, 0, 0)]) == SHAPE   # not in order
    assert call([(None, D, E, 100, 0, 0, 0)]) == NULL and call([(C, None, E, 100, 0, 0, 0)]) == NULL
    assert call([ok], m=None) == NULL and call([ok], v=None) == NULL and call([ok], none=True) == NULL
    for t in ((C, D, E, 100, 0, 2, 0), (C, D, E, 100, 0, 0, 1), (C + 2, D, E, 100, 0, 0, 0), (C, D + 2, E, 100, 0, 0, 0), (C, D + 1, E, 100, 0, 1, 0), (C, D, E + 1, 100, 0, 0, 0)):
        assert call([t]) == UNSUPPORTED, t
    assert call([ok], m=A + 4) == UNSUPPORTED
    for t in ((C, C + 16, E, 100, 0, 0, 0), (C, D, C + 8, 100, 0, 0, 0), (C, D, D, 100, 0, 0, 0), (A + 4, D, E, 100, 0, 0, 0), (C, B, E, 100, 0, 0, 0)):
        assert call([t]) == ALIAS, t
    assert call([ok], m=A, v=A + 16) == ALIAS
    assert call([ok], bits=8, total=600) == SHAPE
    assert call([ok], bits=8, m=None) == NULL
    assert call([ok], bits=8, m=A + 2) == UNSUPPORTED
    assert call([(A + (1 << 20), D, E, 100, 0, 0, 0)], bits=8) == ALIAS   # a parameter over the scales
    assert call([(None, None, None, 0, 0, 0, 0)], total=0) == 0 and call([]) == 0
    mom = lib.zs_adamw_moments8
    assert mom(A, B, C, D, 100, E, F, None) == SHAPE and mom(A, B, C, D, -256, E, F, None) == SHAPE
    assert mom(A, B, C, None, 256, E, F, None) == NULL and mom(A, B, C, D, 256, E + 4, F, None) == UNSUPPORTED
    assert mom(A, B, C, D, 256, A, F, None) == ALIAS and mom(A, B, C, D, 256, E, E + 64, None) == ALIAS


def test_kernels_keep_their_values_in_registers(tmp_path):
    """No kernel of the new sources spills, and none has packed fp32 instructions."""
    seen = 0
    for path in zs_build.device_asm(str(tmp_path)):
        if not os.path.basename(path).startswith(("zs_gmm", "zs_wgrad", "zs_join", "zs_adamw")):
            continue
        text = open(path).read()
        assert not re.search(r"\bv_pk_(?:fma|mul|add)_f32\b", text), path
        for m in re.finditer(r"\.vgpr_spill_count:\s+(\d+)", text):
            seen += 1
            assert m.group(1) == "0", path
        assert not re.search(r"\.private_segment_fixed_size:\s+[1-9]", text), path
    assert seen > 20


def test_launches_of_large_grids(tmp_path):
    """launch_ranges: every workgroup once, in order, fewer than 2^32 threads a launch, starts on multiples of 8, and no
    launch after an error."""
    src = tmp_path / "t.cpp"
    src.write_text("""
#include <cstdlib>
#include <initializer_list>
#include "zs_launch.h"
int main() {
    for (int threads : {256, 512, 1024})
        for (int64_t grid : {int64_t(1), (int64_t(1) << 23) - 1, int64_t(1) << 23, (int64_t(1) << 24) - 8, int64_t(1) << 24, (int64_t(1) << 24) + 25, int64_t(0x7fffffff)}) {
            int64_t at = 0;
            int calls = 0;
            const int err = zs::launch_ranges(grid, threads, [&](int64_t first, int64_t count) {
                if (first != at || first % 8 || count < 1 || count * threads >= int64_t(1) << 32) std::abort();
                at += count;
                ++calls;
                return 0;
            });
            if (err || at != grid || (grid * threads < (int64_t(1) << 32) - 8 * threads && calls != 1)) std::abort();
        }
    int calls = 0;
    if (zs::launch_ranges(int64_t(1) << 30, 256, [&](int64_t, int64_t) { return ++calls == 3 ? 7 : 0; }) != 7 || calls != 3) std::abort();
    if (zs::launch_ranges(0, 256, [&](int64_t, int64_t) { return 9; })) std::abort();
    return 0;
}
""")
    exe = tmp_path / "t"
    subprocess.check_call(["g++", "-std=c++17", "-Wall", "-Werror", "-I", zs_build.CSRC, str(src), "-o", str(exe)])
    assert subprocess.call([str(exe)]) == 0


def test_m0_belongs_to_the_loads_to_lds(tmp_path):
    """Inline assembly writes m0 without being able to say so: in kernels with those loads every mention of m0 is its
    write right before a load, and no instruction reads it unnamed."""
    loads = 0
    for path in zs_build.device_asm(str(tmp_path)):
        if not os.path.basename(path).startswith(("zs_gmm", "zs_wgrad")):
            continue
        for body in re.findall(r"^_Z\S+:[^\n]*\n(.*?)^\.Lfunc_end", open(path).read(), flags=re.M | re.S):
            lines = [x.split(";")[0].strip() for x in body.splitlines()]
            lines = [x for x in lines if x and not x.startswith(".")]
            if not any("load_lds" in x for x in lines):
                continue
            for i, x in enumerate(lines):
                if re.search(r"\bm0\b", x):
                    assert x.startswith("s_mov_b32 m0, s") and lines[i + 1] == "s_nop 0" and lines[i + 2].startswith("global_load_lds_dwordx4"), x
                    loads += 1
                assert not re.match(r"(s_movrel|v_movrel|s_set_gpr_idx|s_sendmsg|v_interp|ds_gws|ds_append|ds_consume|ds_ordered|buffer_load\S* .*\blds\b)", x), x
            assert sum(bool(re.search(r"\bm0\b", x)) for x in lines) == sum(x.startswith("global_load_lds") for x in lines)
    assert loads > 100
