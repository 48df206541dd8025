"""Host-side checks of the norm, the short convolution and the selective scan
(no GPU): every refusal of the C ABI and the binding, and a replay of the index
arithmetic that cuts ragged sequences into tiles.
"""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

import gated_delta_rule_104_b200._binding as b

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
A = 0x7f0000000000  # fake, aligned "device" addresses: never dereferenced
INV, UNS = b.DL_ERR_INVALID_ARG, b.DL_ERR_UNSUPPORTED


def addr(i):
    return A + i * (1 << 30)


@pytest.fixture(scope="module")
def lib():
    return b.load()


def error(lib):
    return lib.dl_last_error().decode()


# ------------------------------------------------------------------ norm

def norm(lib, **k):
    v = dict(x=addr(0), xd=b.DL_BF16, xs=256, res=None, ro=None, rd=b.DL_F32, w=addr(3), wd=b.DL_F32, eps=1e-5, y=addr(4),
             yd=b.DL_BF16, scale=None, group=0, rows=4, width=256)
    v.update(k)
    return lib.dl_rms_norm(v["x"], v["xd"], v["xs"], v["res"], v["ro"], v["rd"], v["w"], v["wd"], v["eps"], v["y"], v["yd"],
                           v["scale"], v["group"], v["rows"], v["width"], None)


@pytest.mark.parametrize("bad,status,text", [
    (dict(xd=b.DL_I8), INV, "x dtype"), (dict(wd=7), INV, "weight dtype"), (dict(yd=9), INV, "y dtype"),
    (dict(res=addr(1), ro=addr(2), rd=b.DL_E4M3), INV, "residual dtype"),
    (dict(rows=-1), INV, "negative"), (dict(width=0, xs=0), INV, "width"), (dict(width=32769, xs=32769), UNS, "32768"),
    (dict(rows=1 << 31), UNS, "exceeds"), (dict(eps=-1.0), INV, "eps"), (dict(eps=float("nan")), INV, "eps"),
    (dict(xs=255), INV, "x_stride"), (dict(ro=addr(2)), INV, "without a residual"), (dict(res=addr(1)), INV, "residual_out"),
    (dict(scale=addr(5)), INV, "without an 8-bit"), (dict(yd=b.DL_I8), INV, "scale is a null"),
    (dict(yd=b.DL_E4M3, scale=addr(5), group=64), UNS, "group"), (dict(x=None), INV, "x is a null"),
    (dict(y=None), INV, "y is a null"), (dict(w=None), INV, "weight is a null"), (dict(x=addr(0) + 1), INV, "aligned"),
    (dict(y=addr(0) + 64), INV, "overlaps"), (dict(res=addr(1), ro=addr(1) + 4), INV, "overlaps"),
    (dict(res=addr(1), ro=addr(0)), INV, "overlaps"), (dict(yd=b.DL_I8, scale=addr(4) + 8), INV, "overlaps"),
])
def test_norm_refusals(lib, bad, status, text):
    assert norm(lib, **bad) == status, error(lib)
    assert text in error(lib)


def test_norm_of_no_rows_is_done_at_once(lib):
    assert norm(lib, rows=0, x=None, y=None) == b.DL_OK


def test_rows_from_8bit_refusals(lib):
    def f(c=addr(0), cd=b.DL_I8, s=addr(1), group=0, o=addr(2), od=b.DL_F32, rows=4, width=256):
        return lib.dl_rows_from_8bit(c, cd, s, group, o, od, rows, width, None)

    assert f(cd=b.DL_BF16) == INV and f(od=b.DL_I8) == INV and f(c=None) == INV and f(s=None) == INV and f(o=None) == INV
    assert f(group=100) == UNS and f(width=0) == INV and f(rows=-3) == INV and f(o=addr(0)) == INV and f(s=addr(1) + 2) == INV
    assert f(rows=0, c=None) == b.DL_OK


# ------------------------------------------------------------------ convolution

def conv(lib, prompt=True, cv=None, **k):
    v = dict(w=addr(0), bias=addr(1), channels=256, taps=4, dtype=b.DL_BF16, x=addr(2), xs=256, T=100, start=addr(3), n=3,
             state=addr(4), P=5, slot=addr(5), status=addr(6), y=addr(7))
    v.update(k)
    c = b.dl_conv(v["w"], v["bias"], v["channels"], v["taps"], v["dtype"], 1)
    cp = None if cv == -1 else ctypes.byref(c)
    if prompt:
        return lib.dl_conv_prompt(cp, v["x"], v["xs"], v["T"], v["start"], v["n"], v["state"], v["P"], v["slot"], v["status"],
                                  v["y"], None)
    return lib.dl_conv_step(cp, v["x"], v["xs"], v["n"], v["state"], v["P"], v["slot"], v["status"], v["y"], None)


@pytest.mark.parametrize("prompt", [True, False])
@pytest.mark.parametrize("bad,status,text", [
    (dict(cv=-1), INV, "conv is a null"), (dict(dtype=b.DL_I8), INV, "dtype"), (dict(taps=1), UNS, "taps"),
    (dict(taps=5), UNS, "taps"), (dict(channels=0), INV, "channels"), (dict(xs=255), INV, "x_stride"), (dict(n=0), INV, ">= 1"),
    (dict(n=6), INV, "distinct slots"), (dict(w=None), INV, "conv.w"), (dict(x=None), INV, "x is a null"),
    (dict(state=None), INV, "state is a null"), (dict(y=None), INV, "y is a null"), (dict(y=addr(2)), INV, "overlaps"),
    (dict(state=addr(0)), INV, "overlaps"), (dict(slot=addr(5) + 2), INV, "aligned"), (dict(status=addr(7)), INV, "overlaps"),
    (dict(x=addr(2) + 1), INV, "aligned"),
])
def test_conv_refusals(lib, prompt, bad, status, text):
    assert conv(lib, prompt, **bad) == status, error(lib)
    assert text in error(lib)


def test_conv_prompt_refusals(lib):
    assert conv(lib, start=None) == INV and "seq_start is a null" in error(lib)
    assert conv(lib, T=-1) == INV
    assert conv(lib, T=0, x=None, y=None) == b.DL_OK
    assert conv(lib, T=1 << 30, channels=1 << 20, xs=1 << 20) == UNS


# ------------------------------------------------------------------ scan

def ssm(lib, prompt=True, null_in=False, **k):
    v = dict(S=addr(0), sd=b.DL_F32, P=5, slot=addr(1), status=addr(2), x=addr(3), xs=6 * 128, dt=addr(4), ds=6, bb=addr(5),
             bs=2 * 64, c=addr(6), cs=2 * 64, z=None, zs=0, A=addr(7), D=addr(8), bias=addr(9), dtype=b.DL_BF16, start=addr(10),
             n=3, T=100, y=addr(11), H=6, G=2, dk=64, dv=128, work=addr(12), wb=1 << 30)
    v.update(k)
    m = b.dl_ssm(v["x"], v["xs"], v["dt"], v["ds"], v["bb"], v["bs"], v["c"], v["cs"], v["z"], v["zs"], v["A"], v["D"],
                 v["bias"], v["dtype"])
    mp = None if null_in else ctypes.byref(m)
    if prompt:
        return lib.dl_ssm_prompt(v["S"], v["sd"], v["P"], v["slot"], v["status"], mp, v["start"], v["n"], v["T"], v["y"],
                                 v["H"], v["G"], v["dk"], v["dv"], v["work"], v["wb"], None)
    return lib.dl_ssm_step(v["S"], v["sd"], v["P"], v["slot"], v["status"], mp, v["y"], v["n"], v["H"], v["G"], v["dk"],
                           v["dv"], None)


@pytest.mark.parametrize("prompt", [True, False])
@pytest.mark.parametrize("bad,status,text", [
    (dict(null_in=True), INV, "in is a null"), (dict(n=0), INV, ">= 1"), (dict(n=6), INV, "distinct slots"),
    (dict(H=0), INV, "H=0"), (dict(dk=32), UNS, "d_k"), (dict(dv=96), UNS, "d_v"), (dict(sd=b.DL_I8), UNS, "state"),
    (dict(sd=b.DL_E4M3), INV, "state dtype"), (dict(dtype=b.DL_I8), INV, "input dtype"), (dict(G=4), INV, "G=4"),
    (dict(G=0), INV, "G=0"), (dict(xs=6 * 128 - 1), INV, "x_stride"), (dict(xs=6 * 128 + 1), INV, "16 bytes"),
    (dict(ds=5), INV, "dt_stride"), (dict(bs=127), INV, "b_stride"), (dict(cs=132), INV, "c_stride"),
    (dict(z=addr(13)), INV, "z_stride"), (dict(x=addr(3) + 8), INV, "x is not 16-byte"), (dict(bb=None), INV, "b is a null"),
    (dict(dt=None), INV, "dt is a null"), (dict(A=None), INV, "A is a null"), (dict(S=None), INV, "S is a null"),
    (dict(y=addr(3) + 256), INV, "overlaps"), (dict(S=addr(7) - 64), INV, "overlaps"), (dict(y=addr(0) + 512), INV, "overlaps"),
    (dict(status=addr(11) + 4), INV, "overlaps"),
])
def test_ssm_refusals(lib, prompt, bad, status, text):
    assert ssm(lib, prompt, **bad) == status, error(lib)
    assert text in error(lib)


def test_ssm_prompt_refusals(lib):
    assert ssm(lib, start=None) == INV and ssm(lib, T=-1) == INV
    assert ssm(lib, T=0, x=None, y=None) == b.DL_OK
    need = lib.dl_ssm_work_bytes(1 << 16, 1, 6, 64, 128)
    assert lib.dl_ssm_work_bytes(-1, 1, 6, 64, 128) == 0 and lib.dl_ssm_work_bytes(100, 0, 6, 64, 128) == 0
    if need:
        assert ssm(lib, T=1 << 16, n=1, wb=need - 1) == INV and "work holds" in error(lib)
        assert ssm(lib, T=1 << 16, n=1, work=None) == INV and ssm(lib, T=1 << 16, n=1, work=addr(12) + 8) == INV
        assert ssm(lib, T=1 << 16, n=1, work=addr(0)) == INV and "overlaps" in error(lib)


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 64), torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        b.dl_rms_norm(x, w, 1e-5, torch.zeros(2, 64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        b.dl_conv_step(x, torch.zeros(64, 4), None, torch.zeros(2, 3, 64), None, x)
    S, v = torch.zeros(1, 1, 64, 64), torch.zeros(1, 1, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        b.dl_ssm_step(S, None, v, torch.zeros(1, 1), torch.zeros(1), v, v, v)


# ------------------------------------------------------------------ tiles of ragged sequences

@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("replay") / "seq_index_replay")
    csrc = os.path.join(ROOT, "gated_delta_rule_104_b200", "csrc")
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", f"-I{csrc}", "-o", exe,
                    os.path.join(HERE, "replay", "seq_index_replay.cpp")], check=True)
    return exe


def tiles(exe, cases):
    """([(seq, first, last), ...], [(seq, first, last, place), ...], places) of each (T, len, seq_start): the tiles, those
    that are not a sequence's last with their place in the workspace, and its places."""
    text = "".join(f"{len(s) - 1} {T} {n} {' '.join(map(str, s))}\n" for T, n, s in cases)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=300, check=True).stdout
    got, line, all_ = [], [], None
    for row in out.splitlines():
        if row == "ends":
            all_, line = line, []
        elif row.startswith("end"):
            got.append((all_, line, int(row.split()[1])))
            line = []
        else:
            line.append(tuple(int(v) for v in row.split()))
    assert len(got) == len(cases)
    return got


def test_tiles_cover_every_row_of_every_sequence_once(replay):
    rng = random.Random(7)
    cases = []
    for _ in range(400):
        lens = [rng.choice([0, 1, 2, 31, 32, 33, 63, 64, 65, rng.randrange(500)]) for _ in range(rng.randrange(1, 20))]
        first, start = rng.choice([0, 0, 5, 64]), []
        start = [first]
        for n in lens:
            start.append(start[-1] + n)
        cases.append((start[-1] + rng.choice([0, 1, 77]), rng.choice([32, 64, 96, 512]), start))
    for (T, n, start), (got, ends, places) in zip(cases, tiles(replay, cases)):
        want = [(i, r) for i in range(len(start) - 1) for r in range(start[i], start[i + 1])]
        assert sorted((i, r) for i, a, z in got for r in range(a, z)) == want
        assert all((a - start[i]) % n == 0 and z - a <= n for i, a, z in got)
        assert [e[:3] for e in ends] == sorted(t for t in got if t[2] < start[t[0] + 1])
        # a sequence's places: its tiles' in order, no two sequences' alike, all inside the workspace
        used = [e[3] for e in ends] + [e[3] + 1 for e in ends if e[2] + n >= start[e[0] + 1]]
        assert len(set(used)) == len(used) and all(0 <= u < places for u in used)


def test_bad_sequence_bounds_never_leave_the_rows(replay):
    rng = random.Random(8)
    big = 2 ** 31 - 1
    cases = [(100, 32, [rng.choice([-big, -5, 0, 3, 50, 100, 101, 4000, big]) for _ in range(rng.randrange(2, 9))])
             for _ in range(1000)]
    for (T, _, start), (got, ends, places) in zip(cases, tiles(replay, cases)):
        for i, a, z in got + [e[:3] for e in ends]:
            assert 0 <= start[i] <= a < z <= start[i + 1] <= T
        assert all(0 <= e[3] and e[3] + 1 < places for e in ends)


def test_layout_of_the_tensor_core_scan(tmp_path):
    """Shared and tensor memory of every form of the scan, replayed from the kernel's own layout header."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "ssm_tc_replay")
    csrc = os.path.join(ROOT, "gated_delta_rule_104_b200", "csrc")
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", f"-I{csrc}", "-o", exe,
                    os.path.join(HERE, "replay", "ssm_tc_replay.cpp")], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stdout
