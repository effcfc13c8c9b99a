"""Host side of the serving entry points, without a GPU: refusals, which come before any device work, sizes of
workspaces and prepared factors, and the frequencies of rotary positions against their formulas in 64 bits."""
import ctypes
import math
import struct
from fractions import Fraction

import pytest

import attention_rank_additive_b200 as fb

INVALID, UNSUPPORTED, WORKSPACE = fb.FB_ERR_INVALID_ARG, fb.FB_ERR_UNSUPPORTED, fb.FB_ERR_WORKSPACE
A = 1 << 20  # an aligned address that no refused call reads
ODD = A + 1


def _changed(names, good, changes):
    args = dict(zip(names, good))
    assert set(changes) <= set(names)
    args.update(changes)
    return [args[n] for n in names]


ROPE = ("dt B N d rot interleaved turns factor positions pos_bstride Hq Q q_bstride q_hstride q_nstride Qo qo_bstride "
        "qo_hstride qo_nstride Hk K k_bstride k_hstride k_nstride Ko ko_bstride ko_hstride ko_nstride stream").split()
ROPE_GOOD = [fb.FB_BF16, 2, 3, 64, 64, 0, A, 1.0, A, 3, 2, A, 384, 192, 64, A, 384, 192, 64, 2, A, 384, 192, 64, A, 384,
             192, 64, 0]


ROPE_BAD = [
    (UNSUPPORTED, dict(dt=fb.FB_F16)), (UNSUPPORTED, dict(dt=fb.FB_E4M3)), (UNSUPPORTED, dict(d=4098, rot=64)),
    (UNSUPPORTED, dict(Hq=65537)),
    (INVALID, dict(B=0)), (INVALID, dict(N=0)), (INVALID, dict(Hq=0)), (INVALID, dict(Hk=-1)), (INVALID, dict(rot=0)),
    (INVALID, dict(rot=33)), (INVALID, dict(rot=66)), (INVALID, dict(turns=0)), (INVALID, dict(Q=0)),
    (INVALID, dict(Qo=0)), (INVALID, dict(K=0)), (INVALID, dict(Ko=0)), (INVALID, dict(factor=math.inf)),
    (INVALID, dict(factor=math.nan)), (INVALID, dict(factor=0.0)), (INVALID, dict(q_nstride=-64)),
    (INVALID, dict(ko_bstride=-1)), (INVALID, dict(pos_bstride=-1)), (INVALID, dict(Q=ODD)), (INVALID, dict(Ko=ODD)),
    (INVALID, dict(turns=A + 4)), (INVALID, dict(positions=ODD)), (INVALID, dict(qo_hstride=128)),
]


@pytest.mark.parametrize("status,changes", ROPE_BAD)
def test_rope_refusals(status, changes):
    args = _changed(ROPE, ROPE_GOOD, changes)
    assert fb.fb_rope_fwd(*args) == fb.fb_rope_bwd(*args) == status


WRITE = ("dt cache_dt B H T d K kb kh kt V vb vh vt kp vp ks vs num_pages page table max_pages starts counts "
         "stream").split()
WRITE_GOOD = [fb.FB_BF16, fb.FB_E4M3, 2, 4, 3, 64, A, 768, 192, 64, A, 768, 192, 64, A, A, A, A, 9, 16, A, 4, A, A, 0]
READ = "dt cache_dt B H N d kp vp ks vs num_pages page table max_pages starts counts K V stream".split()
READ_GOOD = [fb.FB_BF16, fb.FB_E4M3, 2, 4, 3, 64, A, A, A, A, 9, 16, A, 4, A, A, A, A, 0]
CACHE = [
    (UNSUPPORTED, dict(dt=fb.FB_F16)), (UNSUPPORTED, dict(dt=fb.FB_E4M3)), (UNSUPPORTED, dict(cache_dt=fb.FB_F32)),
    (UNSUPPORTED, dict(d=8)), (UNSUPPORTED, dict(d=72)), (UNSUPPORTED, dict(d=144)), (UNSUPPORTED, dict(page=24)),
    (UNSUPPORTED, dict(page=8)), (UNSUPPORTED, dict(page=512)),
    (INVALID, dict(B=0)), (INVALID, dict(H=0)), (INVALID, dict(num_pages=0)), (INVALID, dict(max_pages=0)),
    (INVALID, dict(kp=0)), (INVALID, dict(vp=0)), (INVALID, dict(ks=0)), (INVALID, dict(vs=0)), (INVALID, dict(table=0)),
    (INVALID, dict(K=0)), (INVALID, dict(V=0)), (INVALID, dict(kp=A + 8)), (INVALID, dict(K=A + 8)),
    (INVALID, dict(table=ODD)), (INVALID, dict(starts=ODD)), (INVALID, dict(counts=ODD)),
]


WRITE_BAD = CACHE + [
    (INVALID, dict(T=0)), (INVALID, dict(starts=0)), (INVALID, dict(kt=-64)), (UNSUPPORTED, dict(vh=196)),
    (UNSUPPORTED, dict(dt=fb.FB_F32, kb=770)),
]
READ_BAD = CACHE + [(INVALID, dict(N=0))]


@pytest.mark.parametrize("status,changes", WRITE_BAD)
def test_cache_write_refusals(status, changes):
    assert fb.fb_cache_write(*_changed(WRITE, WRITE_GOOD, changes)) == status


@pytest.mark.parametrize("status,changes", READ_BAD)
def test_cache_read_refusals(status, changes):
    assert fb.fb_cache_read(*_changed(READ, READ_GOOD, changes)) == status


def test_cache_bias_sizes_and_refusals():
    assert fb.fb_cache_bias_bytes(4, 2, 100, 3) == 6 * 100 * 16
    assert fb.fb_cache_bias_bytes(1, 1, 10, 17) == 1024 + 20 * 32 * 4
    for bad in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (1, 1, 1, 129)):
        assert fb.fb_cache_bias_bytes(*bad) == 0
    for status, args in (
            (INVALID, (0, 1, 1, 8, A, A, A, 1 << 20, 0)), (INVALID, (1, 1, 1, 0, A, A, A, 1 << 20, 0)),
            (UNSUPPORTED, (1, 1, 1, 129, A, A, A, 1 << 20, 0)), (UNSUPPORTED, (1 << 10, 1, 1 << 30, 8, A, A, A, 1 << 62, 0)),
            (INVALID, (1, 1, 1, 8, 0, A, A, 1 << 20, 0)), (INVALID, (1, 1, 1, 8, A, ODD, A, 1 << 20, 0)),
            (WORKSPACE, (1, 1, 1, 8, A, A, 0, 1 << 20, 0)), (WORKSPACE, (1, 1, 1, 8, A, A, A + 128, 1 << 20, 0)),
            (WORKSPACE, (1, 1, 1, 8, A, A, A, 1024 + 2 * 16 * 4 - 1, 0))):
        assert fb.fb_cache_bias_prepare(*args) == status


ATTN = ("cache_dt B Hq H T d Q kp vp ks vs num_pages page table max_pages prefix counts mask words depths R P fq fk "
        "bias scale O LSE ws ws_bytes stream").split()
ATTN_GOOD = [fb.FB_E4M3, 2, 8, 4, 5, 64, A, A, A, A, A, 9, 16, A, 4, A, A, A, 1, A, 8, 64, 8, 4, A, 0.125, A, A, A, 1 << 40,
             0]


ATTN_BAD = [
    (UNSUPPORTED, dict(cache_dt=fb.FB_F32)), (UNSUPPORTED, dict(d=24)), (UNSUPPORTED, dict(d=144)),
    (UNSUPPORTED, dict(page=48)), (UNSUPPORTED, dict(T=70000, words=4000)), (UNSUPPORTED, dict(Hq=32768)),
    (UNSUPPORTED, dict(B=(1 << 20) + 1)), (UNSUPPORTED, dict(R=129)), (UNSUPPORTED, dict(R=-1)),
    (UNSUPPORTED, dict(max_pages=1 << 27, page=16)),
    (INVALID, dict(B=0)), (INVALID, dict(Hq=0)), (INVALID, dict(H=0)), (INVALID, dict(T=0)), (INVALID, dict(Hq=6)),
    (INVALID, dict(num_pages=0)), (INVALID, dict(max_pages=0)), (INVALID, dict(Q=0)), (INVALID, dict(kp=0)),
    (INVALID, dict(vp=0)), (INVALID, dict(ks=0)), (INVALID, dict(vs=0)), (INVALID, dict(table=0)),
    (INVALID, dict(prefix=0)), (INVALID, dict(O=0)), (INVALID, dict(LSE=0)), (INVALID, dict(Q=A + 8)),
    (INVALID, dict(ks=A + 4)), (INVALID, dict(bias=A + 8)), (INVALID, dict(mask=ODD)), (INVALID, dict(LSE=ODD)),
    (INVALID, dict(words=0)), (INVALID, dict(T=33)), (INVALID, dict(scale=0.0)), (INVALID, dict(scale=-1.0)),
    (INVALID, dict(scale=math.inf)), (INVALID, dict(scale=math.nan)), (INVALID, dict(bias=0)), (INVALID, dict(P=0)),
    (INVALID, dict(fq=2)), (INVALID, dict(fk=8)), (WORKSPACE, dict(ws=0)), (WORKSPACE, dict(ws=A + 128)),
    (WORKSPACE, dict(ws_bytes=4096)),
]


@pytest.mark.parametrize("status,changes", ATTN_BAD)
def test_attn_cache_refusals(status, changes):
    assert fb.fb_attn_cache_fwd(*_changed(ATTN, ATTN_GOOD, changes)) == status


def test_attn_cache_workspace():
    assert fb.fb_attn_cache_workspace_bytes(1, 12, 12, 1, 64) > 0
    assert fb.fb_attn_cache_workspace_bytes(1, 12, 12, 1, 64) == fb.fb_attn_cache_workspace_bytes(64, 12, 12, 1, 64)
    for bad in ((0, 8, 8, 1, 64), (1, 8, 3, 1, 64), (1, 8, 8, 0, 64), (1, 8, 8, 1, 40), (1, 8, 8, 65537, 64)):
        assert fb.fb_attn_cache_workspace_bytes(*bad) == 0


def _packed(names, values):
    return struct.pack("=" + "".join("d" if n in ("factor", "scale") else "q" for n in names), *values)


@pytest.mark.parametrize("entry,names,good,refused", [
    (0, ROPE, ROPE_GOOD, ROPE_BAD), (1, ROPE, ROPE_GOOD, ROPE_BAD), (2, WRITE, WRITE_GOOD, WRITE_BAD),
    (3, READ, READ_GOOD, READ_BAD), (4, ATTN, ATTN_GOOD, ATTN_BAD)])
def test_packed_calls_refuse_what_the_plain_ones_refuse(entry, names, good, refused):
    for status, changes in refused:
        assert fb.fb_call(entry, _packed(names, _changed(names, good, changes)), len(names)) == status, changes
    assert fb.fb_call(entry, _packed(names, good), len(names) - 1) == INVALID
    assert fb.fb_call(entry, None, len(names)) == INVALID


def test_packed_calls_know_their_entries():
    for entry in (-1, 5):
        assert fb.fb_call(entry, _packed(ROPE, ROPE_GOOD), len(ROPE)) == UNSUPPORTED


# ------------------------------------------------------------ frequencies of rotary positions

def _frequencies(*args):
    rot = args[0]
    freq, out = (ctypes.c_double * max(1, rot // 2))(), ctypes.c_double(-1)
    status = fb.fb_rope_frequencies_host(*args, ctypes.addressof(freq), ctypes.addressof(out))
    return status, list(freq), out.value


@pytest.mark.parametrize("rot", [2, 20, 64, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_frequencies(rot, base):
    plain = [base ** (-2.0 * p / rot) for p in range(rot // 2)]
    by, trained, fast, slow = 8.0, 4096.0, 32.0, 1.0

    def close(got, want):
        assert all(math.isclose(a, b, rel_tol=2.0 ** -44) for a, b in zip(got, want)) and len(got) == len(want)

    status, got, out = _frequencies(rot, base, 0, 1.0, trained, fast, slow)
    close(got, plain)
    assert status == fb.FB_OK and out == 1.0
    status, got, out = _frequencies(rot, base, 1, by, trained, fast, slow)
    close(got, [w / by for w in plain])
    if rot > 2:
        status, got, out = _frequencies(rot, base, 2, by, trained, fast, slow)
        close(got, [(base * by ** (rot / (rot - 2))) ** (-2.0 * p / rot) for p in range(rot // 2)])
        assert math.isclose(got[-1], plain[-1] / by, rel_tol=1e-12)  # the slowest pair is stretched by the factor
    status, got, out = _frequencies(rot, base, 3, by, trained, fast, slow)
    assert status == fb.FB_OK and math.isclose(out, 0.1 * math.log(by) + 1.0)
    for w, g in zip(plain, got):
        assert w / by * (1 - 1e-12) <= g <= w * (1 + 1e-12)
    status, got, out = _frequencies(rot, base, 4, by, trained, fast, slow)
    assert status == fb.FB_OK and out == 1.0
    keep = [min(1.0, max(0.0, (trained * w / (2 * math.pi) - slow) / (fast - slow))) for w in plain]
    close(got, [w / by * (1 - k) + w * k for w, k in zip(plain, keep)])


@pytest.mark.parametrize("args", [
    (0, 1e4, 0, 1.0, 0, 0, 0), (3, 1e4, 0, 1.0, 0, 0, 0), (4098, 1e4, 0, 1.0, 0, 0, 0), (64, 1.0, 0, 1.0, 0, 0, 0),
    (64, math.inf, 0, 1.0, 0, 0, 0), (64, 1e4, 1, 0.5, 0, 0, 0), (64, 1e4, 1, math.nan, 0, 0, 0), (2, 1e4, 2, 2.0, 0, 0, 0),
    (64, 1e4, 3, 2.0, 0.0, 32.0, 1.0), (64, 1e4, 3, 2.0, 4096.0, 1.0, 1.0), (64, 1e4, 4, 2.0, 4096.0, 32.0, 0.0),
])
def test_frequencies_refused(args):
    assert _frequencies(*args)[0] == INVALID


def test_frequencies_unknown_scaling():
    assert _frequencies(64, 1e4, 5, 1.0, 4096.0, 32.0, 1.0)[0] == UNSUPPORTED


def test_turns():
    """2^64 w / 2 pi, modulo 2^64, within the roundings of two doubles (2^-52 of the turns)."""
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    freq = [1.0, 0.5, 1e-5, 0.0, 2 * math.pi, 7.0, -0.25, 10000.0 ** -0.97]
    f, t = (ctypes.c_double * len(freq))(*freq), (ctypes.c_uint64 * len(freq))()
    assert fb.fb_rope_turns_host(len(freq), ctypes.addressof(f), ctypes.addressof(t)) == fb.FB_OK
    for w, got in zip(freq, t):
        exact = Fraction(w) / (2 * pi)
        off = (Fraction(int(got), 2 ** 64) - exact) % 1
        assert min(off, 1 - off) <= abs(exact) * Fraction(1, 2 ** 52) + Fraction(2, 2 ** 54)
    f[2] = math.nan
    assert fb.fb_rope_turns_host(len(freq), ctypes.addressof(f), ctypes.addressof(t)) == INVALID
    assert fb.fb_rope_turns_host(0, ctypes.addressof(f), ctypes.addressof(t)) == INVALID
    assert fb.fb_rope_turns_host(2, 0, ctypes.addressof(t)) == INVALID


@pytest.mark.parametrize("rot", [8, 64, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("by,trained,fast,slow", [(8.0, 4096.0, 32.0, 1.0), (16.0, 8192.0, 32.0, 1.0), (2.0, 300.0, 5.0, 0.25)])
def test_yarn_ramp(rot, base, by, trained, fast, slow):
    """Pair p keeps its frequency as far as it makes `fast` turns over the trained length, is divided by `by` from `slow`
    turns down, and in between the share kept falls linearly with p, from the whole pair number below the first border to
    the one above the second (within 0 and rot - 1)."""
    status, got, _ = _frequencies(rot, base, 3, by, trained, fast, slow)
    assert status == fb.FB_OK

    def border(turns):  # base^(-2 p / rot) trained / 2 pi = turns
        return rot / 2 * math.log(trained / (2 * math.pi * turns)) / math.log(base)

    first, last = max(math.floor(border(fast)), 0), min(math.ceil(border(slow)), rot - 1)
    ramped = 0
    for p in range(rot // 2):
        w = base ** (-2.0 * p / rot)
        share = 1.0 if p <= first else (0.0 if p >= last else (last - p) / (last - first))
        assert math.isclose(got[p], w * share + w / by * (1.0 - share), rel_tol=2.0 ** -40)
        ramped += 0.0 < share < 1.0
    assert first < last and (ramped > 0 or rot == 8)
