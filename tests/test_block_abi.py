"""The C ABI of the operators around a mixing layer without a GPU: bad arguments are refused before
any launch, and empty calls succeed without one.  And the 64-bit references against each other."""
import os
import subprocess

import pytest
import torch

from block_util import ref_pack, ref_unpack
from gated_delta_rule_41_gb300 import block
from gated_delta_rule_41_gb300 import build as kbuild
from gated_delta_rule_41_gb300.block import KdaAddNormDims, KdaGatedNormDims, KdaScanDims

FAKE, ODD = 1 << 20, (1 << 20) + 1      # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return block._lib()


def scan(**kw):
    base = dict(B=2, T=10, C=16, dtype=1, tied=0, x_batch=160, x_token=16, g_batch=160, g_token=16)
    base.update(kw)
    return KdaScanDims(**base)


def fwd(lib, d, cu=None, n=0, x=FAKE, g=FAKE, h0=None, o=FAKE, ht=None, states=None):
    return lib.kda_gated_scan_fwd(d, cu, n, x, g, h0, o, ht, states, None)


def bwd(lib, d, cu=None, n=0, x=FAKE, states=FAKE, do=FAKE, dx=FAKE, dg=FAKE, dht=None):
    return lib.kda_gated_scan_bwd(d, cu, n, x, FAKE, None, states, do, dht, dx, dg, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(B=-1), 2), (dict(T=-1), 2), (dict(C=0), 2),
    (dict(x_token=15), 2), (dict(g_token=0), 2), (dict(x_batch=8), 2), (dict(x_token=-16), 2),
    (dict(B=65536, T=1), 3), (dict(B=1, T=1 << 30), 3), (dict(B=1 << 10, T=1 << 20), 3)])
def test_scan_dims(lib, kw, want):
    d = scan(**kw)
    assert fwd(lib, d) == want and bwd(lib, d) == want


def test_scan_pointers(lib):
    d = scan()
    assert lib.kda_gated_scan_fwd(None, None, 0, *([FAKE] * 6), None) == 1
    assert fwd(lib, d, x=None) == 1 and fwd(lib, d, g=ODD) == 4 and fwd(lib, d, o=ODD) == 4
    assert fwd(lib, d, h0=FAKE + 2) == 4 and fwd(lib, d, ht=FAKE + 2) == 4 and fwd(lib, d, states=ODD) == 4
    assert fwd(lib, scan(dtype=0), x=FAKE + 2) == 4
    assert fwd(lib, d, o=None) == 0                      # nothing asked for, nothing done
    assert fwd(lib, d, cu=FAKE, n=3) == 2                # packed: B == 1
    assert fwd(lib, scan(B=1), cu=FAKE, n=0) == 2 and fwd(lib, scan(B=1), cu=ODD, n=3) == 4
    assert fwd(lib, scan(B=1), cu=FAKE, n=65536) == 3
    for name in ("x", "states", "do", "dx", "dg"):
        assert bwd(lib, d, **{name: None}) == 1 and bwd(lib, d, **{name: ODD}) == 4
    assert bwd(lib, d, dht=FAKE + 1) == 4
    assert fwd(lib, scan(B=0), x=None, g=None, o=None) == 0
    assert bwd(lib, scan(B=0), x=None, states=None, do=None, dx=None, dg=None) == 0
    assert fwd(lib, scan(T=0), x=None, g=None, o=None) == 0

    def step(d, x=FAKE, state=FAKE, new=FAKE, o=FAKE):
        return lib.kda_gated_scan_step(d, x, FAKE, state, new, o, None)

    assert step(scan(x_batch=8)) == 2 and step(d, x=None) == 1 and step(d, state=None) == 1
    assert step(d, new=FAKE + 2) == 4 and step(d, o=ODD) == 4 and step(scan(B=0), x=None) == 0


def gated(**kw):
    base = dict(T=4, H=2, D=64, dtype=1, w_dtype=0, gate=0, eps=1e-5, x_stride=128, gate_stride=128)
    base.update(kw)
    return KdaGatedNormDims(**base)


def gfwd(lib, d, x=FAKE, z=FAKE, w=FAKE, y=FAKE, kept=(None,) * 4):
    return lib.kda_gated_norm_fwd(d, x, z, w, y, *kept, None)


def gbwd(lib, d, x=FAKE, xs=None, z=FAKE, zs=None, w=FAKE, dy=FAKE, dx=FAKE, dz=FAKE, dw=FAKE, ws=FAKE, n=1 << 40):
    return lib.kda_gated_norm_bwd(d, x, xs, z, zs, w, dy, dx, dz, dw, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), 1), (dict(w_dtype=2), 1), (dict(gate=2), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(T=-1), 2), (dict(H=0), 2), (dict(D=0), 2),
    (dict(D=16385), 3), (dict(T=1 << 29, x_stride=1 << 40, gate_stride=1 << 40), 3), (dict(x_stride=127), 2),
    (dict(gate_stride=-128), 2)])
def test_gated_dims(lib, kw, want):
    d = gated(**kw)
    assert gfwd(lib, d) == want and gbwd(lib, d) == want and lib.kda_gated_norm_workspace_bytes(d) == 0


def test_gated_pointers(lib):
    d = gated()
    assert gfwd(lib, d, x=None) == 1 and gfwd(lib, d, z=ODD) == 4 and gfwd(lib, d, y=None) == 1
    assert gfwd(lib, d, w=FAKE + 2) == 4 and gfwd(lib, gated(T=0), x=None, z=None, y=None) == 0
    assert gfwd(lib, d, kept=(FAKE, FAKE, None, None)) == 1
    assert gbwd(lib, d, dy=None) == 1 and gbwd(lib, d, dx=ODD) == 4 and gbwd(lib, d, dw=FAKE + 2) == 4
    assert gbwd(lib, d, xs=FAKE) == 1 and gbwd(lib, d, zs=FAKE) == 1
    assert gbwd(lib, d, x=ODD) == 4
    need = lib.kda_gated_norm_workspace_bytes(d)
    assert need > 0 and need % 256 == 0
    assert gbwd(lib, d, ws=None) == 5 and gbwd(lib, d, n=need - 1) == 5 and gbwd(lib, d, ws=FAKE + 16) == 4
    assert gbwd(lib, gated(T=0), dw=None) == 0


def add(**kw):
    base = dict(T=4, D=64, dtype=1, res_dtype=1, w_dtype=0, eps=1e-5, alpha=1.0, r_stride=64, x_stride=64)
    base.update(kw)
    return KdaAddNormDims(**base)


def afwd(lib, d, r=FAKE, x=FAKE, av=None, w=FAKE, out=FAKE, y=FAKE):
    return lib.kda_add_norm_fwd(d, r, x, av, w, out, y, None)


def abwd(lib, d, r=FAKE, x=FAKE, av=None, w=FAKE, dy=FAKE, dr=FAKE, dres=FAKE, dx=FAKE, dw=FAKE, da=None,
         ws=FAKE, n=1 << 40):
    return lib.kda_add_norm_bwd(d, r, x, av, w, dy, dr, dres, dx, dw, da, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), 1), (dict(res_dtype=9), 1), (dict(w_dtype=2), 1), (dict(eps=0.0), 1),
    (dict(alpha=float("inf")), 1), (dict(T=-1), 2), (dict(D=0), 2), (dict(D=16400), 3), (dict(T=1 << 30), 3),
    (dict(dtype=0), 3), (dict(r_stride=63), 2), (dict(x_stride=0), 2)])
def test_add_dims(lib, kw, want):
    d = add(**kw)
    assert afwd(lib, d) == want and abwd(lib, d) == want and lib.kda_add_norm_workspace_bytes(d) == 0


def test_add_pointers(lib):
    d = add()
    assert afwd(lib, d, r=None) == 1 and afwd(lib, d, y=ODD) == 4 and afwd(lib, d, out=None) == 1
    assert afwd(lib, d, av=FAKE + 2) == 4 and afwd(lib, add(res_dtype=0), out=FAKE + 2) == 4
    assert afwd(lib, add(T=0), r=None, x=None, out=None, y=None) == 0
    assert abwd(lib, d, dres=None) == 1 and abwd(lib, d, dy=None) == 1 and abwd(lib, d, dr=ODD) == 4
    assert abwd(lib, d, x=None, da=FAKE) == 1 and abwd(lib, d, da=FAKE + 2) == 4
    need = lib.kda_add_norm_workspace_bytes(d)
    assert need > 0 and need % 256 == 0
    assert abwd(lib, d, ws=None) == 5 and abwd(lib, d, n=need - 1) == 5 and abwd(lib, d, ws=FAKE + 4) == 4
    assert abwd(lib, add(T=0), dw=None) == 0


def test_pack(lib):
    def pack(x=FAKE, t=1, rows=4, D=64, stride=64, codes=FAKE, scales=FAKE):
        return lib.kda_pack8(x, t, rows, D, stride, codes, scales, None)

    def unpack(codes=FAKE, scales=FAKE, rows=4, D=64, x=FAKE, t=1):
        return lib.kda_unpack8(codes, scales, rows, D, x, t, None)

    assert pack(x=None) == 1 and pack(x=ODD) == 4 and pack(codes=None) == 1 and pack(scales=None) == 1
    assert pack(t=2) == 1 and pack(rows=-1) == 2 and pack(D=0) == 2 and pack(stride=63) == 2
    assert pack(rows=1 << 40) == 3 and pack(rows=0, x=None) == 0
    assert unpack(codes=None) == 1 and unpack(x=ODD) == 4 and unpack(t=7) == 1 and unpack(D=0) == 2
    assert unpack(rows=-1) == 2 and unpack(rows=1 << 40) == 3 and unpack(rows=0, x=None) == 0


def test_sizes_past_32_bits():
    """Refused before they are cut to the C entries' ints; rows that would be longer are not joined."""
    huge = (1 << 31) + 64
    x = torch.empty(1).expand(1, huge, 1)
    for make in (lambda: block._scan_dims(x, x, False), lambda: block._step_dims(x[0], x[0], False),
                 lambda: block._gated_dims(x.transpose(0, 1), x.transpose(0, 1), None, 0, 1e-5, "silu"),
                 lambda: block._add_dims(x[0], None, None, None, 0, 1e-5), lambda: block._rows("x", x[0, :, 0])):
        with pytest.raises(block.KdaError) as e:
            make()
        assert e.value.status == 3
    y = torch.empty(4, 1 << 22, 1024, device="meta")[:, :1 << 21]      # 2^31 elements of 2^32 a row
    assert block._rows("x", y[:, :1 << 20]) == (4, 1 << 30, 1 << 32)
    with pytest.raises(block.KdaError):
        block._rows("x", y)


def test_reference_codes():
    """The trial of exponents and the grid of codes against torch's own 8-bit type."""
    x = torch.randn(50, 64, generator=torch.Generator().manual_seed(1)) * 100
    codes, scales = ref_pack(x)
    s = torch.pow(2.0, scales.double() - 127).repeat_interleave(32, -1)
    assert torch.equal(codes, (x.double() / s).float().to(torch.float8_e4m3fn).double())
    top = codes.unflatten(-1, (-1, 32)).abs().amax(-1)
    assert (top <= 448).all() and (top >= 224).all()
    assert ((ref_unpack(codes, scales) - x.double()).abs() <= x.double().abs() * 2.0 ** -4 + 2.0 ** -10 * s).all()


def test_exchange_arguments(lib):
    def call(ctas=4, turns=5, stall=0, limit=1000, sums=FAKE):
        return lib.kda_selftest_exchange(ctas, turns, -1, 0, stall, limit, sums, None)

    assert call(limit=-1) == 1 and call(limit=1 << 40) == 1 and call(sums=None) == 1
    assert call(stall=-1) == 1 and call(stall=1 << 40) == 1
    assert call(ctas=0) == 2 and call(ctas=17) == 2 and call(turns=-1) == 2 and call(turns=251) == 2
    assert call(sums=ODD) == 4


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    here, out = os.path.dirname(os.path.abspath(__file__)), str(tmp_path_factory.mktemp("model") / "model")
    subprocess.run(["g++", "-O2", "-std=c++17", "-pthread", "-I", kbuild.CSRC,
                    os.path.join(here, "exchange_model.cpp"), "-o", out], check=True)
    return out


@pytest.mark.parametrize("ctas,turns,seeds,rounds", [(1, 5, 20, 1 << 30), (13, 20, 2, 1 << 30), (2, 9, 30, 300),
                                                     (4, 12, 20, 200), (4, 12, 20, 3000), (16, 9, 6, 300),
                                                     (16, 200, 1, 300)])
def test_exchange_of_a_cluster(model, ctas, turns, seeds, rounds):
    """Nothing comes to a CTA that has ended, no barrier gets an arrival too many, and without a lost CTA no
    turn reads another's maps, whichever waits give up (and with waits that do not, none is lost)."""
    r = subprocess.run([model, str(ctas), str(turns), str(seeds), str(rounds)], capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0, r.stdout
    lost = int(r.stdout.split()[-1])
    assert lost == 0 if rounds == 1 << 30 else lost > 0
