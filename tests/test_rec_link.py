"""The gated recurrence's decays and the links of its tiles on the CPU: csrc/rec_link.h, which the
kernels call, compiled for the host (rec_link_host.cpp) and called here."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from chunk_wise_weight_chunked_amd import build as hipbuild

HERE = os.path.dirname(os.path.abspath(__file__))
f32 = np.float32

pytestmark = pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"),
                                reason="hipcc not available")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("rec_link") / "librec_link.so")
    cmd = [hipbuild.hipcc(), "-x", "hip", "--cuda-host-only", "--offload-arch=" + hipbuild.ARCH,
           "-O2", "-std=c++17", "-ffp-contract=off", "-fPIC", "-shared", "-pthread",
           os.path.join(HERE, "rec_link_host.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    lib = ctypes.CDLL(out)
    f, u64, i64, vp = ctypes.c_float, ctypes.c_uint64, ctypes.c_int64, ctypes.c_void_p
    for name, res, args in (
            ("rec_log_rate", f, [f]), ("rec_decay_of", f, [f]), ("rec_decay_both", f, [f, f]),
            ("rec_decayed", f, [f, f, f]), ("rec_word_of", u64, [f, f]),
            ("rec_state_word", u64, [f]), ("rec_unset", u64, []), ("rec_group", ctypes.c_int, []),
            ("rec_state_before", f, [vp, i64]),
            ("rec_link_all", ctypes.c_int, [i64, i64, i64, vp, vp, vp, vp, ctypes.c_int, vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


def value(dec):
    """(a, 1 - a) of a decay as the kernels hold it, in 64 bits."""
    dec = np.float64(dec)
    return (1 + dec, -dec) if np.signbit(dec) else (dec, 1 - dec)


def test_rates(lib):
    """Below 0 and NaN: NaN; 0 of either sign: a z of -0, whose decay keeps a state."""
    for r in (0.0, -0.0):
        z = lib.rec_log_rate(r)
        assert z == 0 and np.signbit(z)
        for gate in (0.0, 1e-30, 0.5, 1.0):
            dec = lib.rec_decay_of(float(f32(z) * f32(gate)))
            assert dec == 0 and np.signbit(dec)
            for h in (3.0, -1e30, 0.0):
                assert lib.rec_decayed(dec, h, 0.25) == f32(f32(h) + f32(0.25))
    for r in (-1e-30, -1.0, float("-inf"), float("nan")):
        assert np.isnan(lib.rec_log_rate(r))
    for r in (1e-38, 1e-3, 1.0, 50.0):
        # log2 e and the product, rounded once each
        want = -np.float64(f32(r)) / np.log(2)
        assert abs(lib.rec_log_rate(r) - want) <= 2.0 ** -23 * abs(want)
    for r in (2.0 ** 100, 1e38, float("inf")):
        assert lib.rec_log_rate(r) == lib.rec_log_rate(2.0 ** 100)
        assert lib.rec_decay_of(lib.rec_log_rate(r)) == 0


def test_a_decay(lib):
    """2^z to a few roundings of itself and, where it is near 1, of its distance from 1."""
    rng = np.random.default_rng(1)
    zs = np.concatenate([-10.0 ** rng.uniform(-40, 2, 500), -rng.uniform(0.4, 0.6, 100)])
    for z in zs.astype(f32):
        dec = lib.rec_decay_of(z)
        a, gap = value(dec)
        want, whole = -np.expm1(np.float64(z) * np.log(2)), np.exp2(np.float64(z))
        assert np.signbit(dec) == (z > -0.5)
        # near: the polynomial's 3.3e-8 and six roundings, which shrink with z towards its constant
        # term; far: exp2's two
        if np.signbit(dec):
            assert abs(gap - want) <= (3.3e-8 + 3 * 2.0 ** -24) * want + 2.0 ** -149
        else:
            assert abs(a - whole) <= 2.0 ** -23 * whole + 2.0 ** -149


def test_the_decay_over_two_runs(lib):
    """The product of any two to 2^-22 of itself and, near 1, of its distance from 1."""
    rng = np.random.default_rng(8)
    some = [-0.0, 0.0, 1e-30, 0.7, -0.29, -1e-7, -1e-30]
    some += [-(10.0 ** -e) for e in rng.uniform(0.6, 8, 40)] + list(rng.uniform(0, .7, 40))
    some = [float(f32(x)) for x in some]
    both = lib.rec_decay_both
    for a in some:
        for x, y in ((-0.0, a), (a, -0.0)):
            assert both(x, y) == a and np.signbit(both(x, y)) == np.signbit(a)
        for b in some:
            got = both(a, b)
            (va, ua), (vb, ub) = value(a), value(b)
            assert abs(value(got)[0] - va * vb) <= 2.0 ** -22 * va * vb + 2.0 ** -149
            if np.signbit(got):  # 1 - a b = (1 - a) + (1 - b) - (1 - a)(1 - b)
                want = ua + ub - ua * ub
                assert abs(value(got)[1] - want) <= 2.0 ** -22 * want + 2.0 ** -149
    for a, b in ((np.nan, -0.0), (-0.0, np.nan), (0.5, np.nan), (np.nan, np.nan)):
        assert np.isnan(both(a, b))


def test_no_word_is_taken_for_another(lib):
    """A map is neither unset nor a state, whatever NaN its decay is; a state never unset."""
    nans = np.array([0xffffffff, 0x7fffffff, 0x7fc00000, 0xffc00001], np.uint32).view(f32)
    state = lib.rec_state_word(0.0) >> 32
    for h in list(nans) + [0.0, -0.0, np.inf, 1.5]:
        assert lib.rec_state_word(h) != lib.rec_unset()
        for dec in list(nans) + [0.0, -0.0, -0.29, 0.7, 1.0]:
            w = lib.rec_word_of(dec, h)
            assert w != lib.rec_unset() and w >> 32 != state


def maps(rng, *shape):
    """Decays near 1 and far from it, and states behind from 0."""
    near, far = -np.abs(rng.normal(size=shape)) * 0.1, rng.random(shape) * 0.7
    return (np.where(rng.random(shape) < 0.5, np.maximum(near, -0.29), far).astype(f32),
            rng.normal(size=shape).astype(f32))


def test_the_state_found_does_not_depend_on_what_is_published(lib):
    """From the nearest group whose state is known and the maps behind it, up to six of them in
    all, always the same number to the bit."""
    rng = np.random.default_rng(7)
    n = 30
    dec, h = maps(rng, n)
    states = [f32(rng.normal())]
    for j in range(1, n):
        states.append(lib.rec_decayed(dec[j], states[-1], h[j]))
    for k in range(n):
        for known in range(max(0, k - 5), k + 1):
            for _ in range(5):
                words = []
                for j in range(k + 1):
                    kind = ("state" if j == known else
                            rng.choice(["map", "state"] if j > known else ["unset", "map", "state"]))
                    if j == 0 and kind == "map":
                        kind = "unset"  # the first group's word has no map
                    words.append(lib.rec_unset() if kind == "unset" else
                                 lib.rec_word_of(dec[j], h[j]) if kind == "map" else
                                 lib.rec_state_word(states[j]))
                words = np.array(words, np.uint64)
                assert f32(lib.rec_state_before(words.ctypes.data, k)) == states[k], (k, known)


def link_all(lib, dec, h, first, nap, threads):
    B, tiles, d = dec.shape
    before = np.full_like(dec, 7)
    assert lib.rec_link_all(B, tiles, d, dec.ctypes.data, h.ctypes.data, first.ctypes.data,
                            nap.ctypes.data, threads, before.ctypes.data)
    return before


@pytest.mark.parametrize("B,tiles,d", [(1, 2, 3), (2, 7, 1), (1, 8, 2), (3, 9, 2), (1, 16, 1),
                                       (3, 16, 2), (2, 17, 3), (1, 64, 2), (1, 65, 2), (2, 100, 2)])
def test_tiles_are_linked(lib, B, tiles, d):
    """Each tile's state is that of the chain of maps in 64 bits, and the same to the bit however
    many workers there are and whichever of them are late."""
    rng = np.random.default_rng(tiles)
    dec, h = maps(rng, B, tiles, d)
    first = rng.normal(size=(B, d)).astype(f32)
    late = lambda p: (rng.random(B * tiles) < p).astype(np.uint8)  # noqa: E731
    got = link_all(lib, dec, h, first, late(0), 1)
    s, size = first.astype(np.float64), np.abs(first).astype(np.float64)
    for k in range(tiles):
        # a term goes through its group's map (at most 8 joined, 5 roundings each), 13 groups (2
        # each) and the maps in front of its tile: less than 128 roundings
        assert (np.abs(got[:, k] - s) <= 128 * 2.0 ** -24 * size).all(), k
        a = np.where(np.signbit(dec[:, k]), 1 + dec[:, k].astype(np.float64), dec[:, k])
        s, size = a * s + h[:, k], a * size + np.abs(h[:, k])
    for threads in (2, 5, 16):
        for p in (0, 0.1, 0.5):
            again = link_all(lib, dec, h, first, late(p), threads)
            assert np.array_equal(again.view(np.uint32), got.view(np.uint32)), (threads, p)


def test_links_carry_what_is_not_finite(lib):
    """A NaN or an infinity reaches the tiles behind it in its channel, and no wait goes on."""
    rng = np.random.default_rng(3)
    dec, h = maps(rng, 1, 40, 4)
    first = np.zeros((1, 4), f32)
    dec[0, 5, 1], h[0, 20, 2], first[0, 3] = np.nan, np.inf, np.nan
    for threads in (1, 8):
        got = link_all(lib, dec, h, first, np.zeros(40, np.uint8), threads)
        fine = np.isfinite(got[0])
        assert fine[:, 0].all()
        assert fine[:6, 1].all() and not fine[6:, 1].any()
        assert fine[:21, 2].all() and not fine[21, 2]
        assert not fine[:, 3].any()


def test_links_keep_a_state(lib):
    """A rate of 0 of either sign: the state goes through every tile as it is."""
    dec = np.full((1, 50, 2), lib.rec_decay_of(0.25 * lib.rec_log_rate(-0.0)), f32)
    first = np.array([[3.0, -1e-30]], f32)
    for threads in (1, 4):
        got = link_all(lib, dec, np.zeros_like(dec), first, np.zeros(50, np.uint8), threads)
        assert (got == first[:, None]).all()
