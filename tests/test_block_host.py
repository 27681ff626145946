"""Host-side checks of the block operators' C ABI (no GPU needed): exports, and
every refusal with its documented status before the device is touched.  Invalid
calls use fake (never dereferenced) device addresses.  The 64-bit forms that the
GPU tests compare with are checked here against differences."""
import contextlib
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from chunk_wise_weight_chunked_amd import block
from chunk_wise_weight_chunked_amd import build as hipbuild
from chunk_wise_weight_chunked_amd import ttt_mlp as tm

import _block_ref as ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "ttt_block.h")
A = 1 << 40  # fake addresses, 1 GiB apart


def at(i):
    return A + (i << 30)


def test_exports_every_declared_symbol():
    lib = block._load()
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ttt_[a-z_0-9]+)\s*\(", text)))
    assert set(names) == set(block.EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def refused(call, status, word):
    with pytest.raises(tm.TTTError) as e:
        call()
    assert e.value.status == status, e.value
    assert word in str(e.value), str(e.value)


INVALID, UNSUPPORTED = tm.TTT_ERR_INVALID_ARGUMENT, tm.TTT_ERR_UNSUPPORTED


# ------------------------------------------------------------------- the norm
def norm_desc(**kw):
    base = dict(rows=4, d=256, dtype=torch.bfloat16, res_dtype=None, x_stride=None, y_stride=None,
                eps=1e-6, out=0, scale_group=0)
    base.update(kw)
    return block.make_addnorm_desc(**base)


BAD_NORM = [
    (dict(rows=0), INVALID, "rows"),
    (dict(rows=1 << 31), UNSUPPORTED, "rows"),
    (dict(d=0), INVALID, "d must"),
    (dict(d=100), UNSUPPORTED, "d must"),
    (dict(d=16384 + 8), UNSUPPORTED, "d must"),
    (dict(dtype=5, res_dtype=5), INVALID, "dtype"),
    (dict(dtype=torch.float32, res_dtype=torch.bfloat16), INVALID, "res_dtype"),
    (dict(x_stride=248), INVALID, "x_stride"),
    (dict(x_stride=260), UNSUPPORTED, "x_stride"),
    (dict(y_stride=255), INVALID, "y_stride"),
    (dict(eps=float("nan")), INVALID, "eps"),
    (dict(eps=-1e-6), INVALID, "eps"),
    (dict(out=2), INVALID, "out"),
    (dict(out=1, scale_group=64), INVALID, "scale_group"),
    (dict(scale_group=128), INVALID, "scale_group"),
    (dict(d=200, out=1, scale_group=128), UNSUPPORTED, "scale_group"),
    (dict(rows=1 << 30, x_stride=1 << 40), UNSUPPORTED, "2^56"),
    (dict(rows=1 << 30, y_stride=1 << 30), UNSUPPORTED, "2^56"),
]


@pytest.mark.parametrize("kw,status,word", BAD_NORM)
def test_norm_refuses_descriptors(kw, status, word):
    d = norm_desc(**kw)
    scale = at(5) if kw.get("out") else None
    refused(lambda: block.ttt_addnorm_forward(d, at(1), at(2), at(3), at(4), at(6), scale, 0),
            status, word)


def test_norm_refuses_buffers():
    d = norm_desc()
    fwd = lambda *a: (lambda: block.ttt_addnorm_forward(d, *a, stream=0))  # noqa: E731
    refused(fwd(None, at(2), at(3), at(4), at(5), None), INVALID, "non-NULL")
    refused(fwd(at(1), at(2), None, at(4), at(5), None), INVALID, "non-NULL")
    refused(fwd(at(1), at(2), at(3), at(4), None, None), INVALID, "non-NULL")
    refused(fwd(at(1), at(2), at(3), at(4), at(5), at(6)), INVALID, "y_scale")
    refused(fwd(at(1) + 8, at(2), at(3), at(4), at(5), None), INVALID, "16-byte")
    refused(fwd(at(1), at(2), at(3), at(2) + 256, at(5), None), INVALID, "r overlaps res")
    refused(fwd(at(1), at(2), at(3), at(4), at(1) + 512, None), INVALID, "y overlaps x")
    refused(fwd(at(1), at(2), at(3), at(4), at(4), None), INVALID, "overlaps")
    refused(fwd(at(1), at(2), at(3), at(1), at(5), None), INVALID, "r overlaps x")
    f8 = norm_desc(out=block.TTT_NORM_FP8)
    refused(lambda: block.ttt_addnorm_forward(f8, at(1), None, at(3), None, at(5), None, 0),
            INVALID, "y_scale")
    refused(lambda: block.ttt_addnorm_forward(f8, at(1), None, at(3), None, at(1), at(6), 0),
            INVALID, "y overlaps x")


def test_norm_backward_refusals():
    d = norm_desc(rows=600)
    need = block.ttt_addnorm_backward_workspace_size(d)
    # a wave per row, four to a workgroup: 150 workgroups, one row of d sums each
    assert need == 150 * 256 * 4
    bwd = lambda *a: (lambda: block.ttt_addnorm_backward(d, *a, stream=0))  # noqa: E731
    ok = [at(1), at(2), at(3), at(4), at(5), at(6), at(7)]
    refused(bwd(*ok, None, 0), INVALID, "ws")
    refused(bwd(*ok, at(8) + 16, need), INVALID, "256-byte")
    refused(bwd(*ok, at(8), need - 256), tm.TTT_ERR_WORKSPACE_TOO_SMALL, "needed")
    for i in (0, 1, 2, 4):
        bad = list(ok)
        bad[i] = None
        refused(bwd(*bad, at(8), need), INVALID, "non-NULL")
    bad = list(ok)
    bad[4] = at(2)
    refused(bwd(*bad, at(8), need), INVALID, "dr overlaps r")
    f8 = norm_desc(out=1)
    refused(lambda: block.ttt_addnorm_backward(f8, *ok, at(8), need, 0), INVALID, "NORM_SAME")


def test_norm_reference_against_differences():
    rng = np.random.default_rng(1)
    r, w, dy = rng.normal(size=(3, 16)), rng.normal(size=16), rng.normal(size=(3, 16))
    dx, dw = ref.addnorm_grads(dy, r, w, 1e-3)
    e = 1e-5
    for _ in range(5):
        u, z = rng.normal(size=r.shape), rng.normal(size=16)
        f = lambda s: (dy * ref.addnorm(r + s * u, None, w + s * z, 1e-3)[1]).sum()  # noqa: E731
        assert abs((f(e) - f(-e)) / (2 * e) - ((dx * u).sum() + (dw * z).sum())) < 1e-7


# ---------------------------------------------------------- linear attention
def attn_desc(**kw):
    base = dict(batch=2, seq_len=64, heads=4, kv_heads=2, d_key=64, d_value=64,
                dtype=torch.bfloat16, scale=0.125)
    base.update(kw)
    return block.make_linattn_desc(**base)


BAD_ATTN = [
    (dict(batch=0), INVALID, "batch"),
    (dict(seq_len=0), INVALID, "seq_len"),
    (dict(heads=0), INVALID, "heads"),
    (dict(kv_heads=0), INVALID, "kv_heads"),
    (dict(kv_heads=3), INVALID, "multiple of kv_heads"),
    (dict(heads=65536, kv_heads=1), UNSUPPORTED, "65535"),
    (dict(batch=1 << 23), UNSUPPORTED, "batch * heads"),
    (dict(batch=(1 << 19) + 1), UNSUPPORTED, "batch * heads"),
    (dict(seq_len=1 << 31), UNSUPPORTED, "seq_len"),
    (dict(seq_len=1 << 30, heads=64), UNSUPPORTED, "2^34"),
    (dict(d_key=0), INVALID, "d_key"),
    (dict(d_key=60), UNSUPPORTED, "multiples of 8"),
    (dict(d_value=136), UNSUPPORTED, "at most 128"),
    (dict(dtype=9), INVALID, "dtype"),
    (dict(scale=float("inf")), INVALID, "scale"),
    (dict(q_stride=(64, -8, 64)), INVALID, "strides"),
    (dict(k_stride=(4096, 100, 64)), UNSUPPORTED, "multiples of 8"),
    (dict(v_stride=(1 << 41, 128, 64)), UNSUPPORTED, "2^40"),
    (dict(seq_len=1 << 20, k_stride=(0, 1 << 40, 64)), UNSUPPORTED, "2^56"),
    (dict(q_stride=(64, (1 << 26) + 8, 64)), UNSUPPORTED, "2^27"),
    (dict(dtype=torch.float32, v_stride=(64, (1 << 25) + 8, 64)), UNSUPPORTED, "2^27"),
    (dict(o_stride=(64 * 256, 256, 32)), INVALID, "one place"),
    (dict(o_stride=(0, 256, 64)), INVALID, "one place"),
    (dict(o_stride=(64 * 256, 128, 64)), INVALID, "one place"),
]


@pytest.mark.parametrize("kw,status,word", BAD_ATTN)
def test_attention_refuses_descriptors(kw, status, word):
    d = attn_desc(**kw)
    refused(lambda: block.ttt_linattn_forward(d, at(1), at(2), at(3), at(4), None, None, None,
                                              at(5), at(6), 1 << 29, 0), status, word)
    if word not in ("one place", "2^27"):
        refused(lambda: block.ttt_linattn_workspace_size(d), status, word)


def test_attention_refuses_buffers():
    d = attn_desc()
    fwd = lambda *a, **k: (lambda: block.ttt_linattn_forward(  # noqa: E731
        k.get("d", d), *a, k.get("ws"), k.get("n", 0), 0))
    ok = [at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8)]
    assert block.ttt_linattn_workspace_size(d) == 0
    for i in (0, 1, 2, 3, 7):
        bad = list(ok)
        bad[i] = None
        refused(fwd(*bad), INVALID, "non-NULL")
    for i in (0, 1, 2, 5, 6, 7):
        bad = list(ok)
        bad[i] += 8
        refused(fwd(*bad), INVALID, "16-byte")
    for i in (3, 4):
        bad = list(ok)
        bad[i] += 2
        refused(fwd(*bad), INVALID, "4-byte")
    for i, j, word in ((7, 0, "o overlaps q"), (7, 1, "o overlaps k"), (7, 5, "o overlaps state_in"),
                       (6, 2, "state_out overlaps v"), (7, 3, "o overlaps log_decay"),
                       (6, 4, "state_out overlaps lengths"), (6, 7, "overlaps")):
        bad = list(ok)
        bad[i] = bad[j]
        refused(fwd(*bad), INVALID, word)
    bad = list(ok)
    bad[6] = bad[5] + 256  # in place is the same address or none
    refused(fwd(*bad), INVALID, "state_out overlaps state_in")
    long = attn_desc(seq_len=8192)
    need = block.ttt_linattn_workspace_size(long)
    assert need > 0 and need % (2 * 4 * 64 * 64 * 4) == 0
    refused(fwd(*ok, d=long), INVALID, "ws is NULL")
    refused(fwd(*ok, d=long, ws=at(9) + 64, n=need), INVALID, "256-byte")
    refused(fwd(*ok, d=long, ws=at(9), n=need - 1), tm.TTT_ERR_WORKSPACE_TOO_SMALL, "needed")
    refused(fwd(*ok, d=long, ws=at(8), n=need), INVALID, "overlaps")


def test_attention_backward_refusals():
    d = attn_desc()
    # shared heads: an fp32 gradient for every query head
    assert block.ttt_linattn_backward_workspace_size(d) >= 2 * 64 * 4 * 64 * 4
    assert block.ttt_linattn_backward_workspace_size(attn_desc(kv_heads=4)) == 0
    need = block.ttt_linattn_backward_workspace_size(d)
    # q, k, v, log_decay, lengths, state_in, dO, dstate_out, dq, dk, dv, dstate_in
    ok = [at(i) for i in range(1, 13)]
    bwd = lambda a, ws=at(20), n=need: (lambda: block.ttt_linattn_backward(  # noqa: E731
        d, *a, ws, n, 0))
    for i in (0, 1, 2, 3, 6, 8, 9, 10):
        bad = list(ok)
        bad[i] = None
        refused(bwd(bad), INVALID, "non-NULL")
    refused(bwd(ok, None, 0), INVALID, "ws is NULL")
    refused(bwd(ok, at(20), need - 1), tm.TTT_ERR_WORKSPACE_TOO_SMALL, "needed")
    for i, j in ((8, 0), (9, 1), (10, 6), (11, 5), (8, 9), (10, 3)):
        bad = list(ok)
        bad[i] = bad[j]
        refused(bwd(bad), INVALID, "overlaps")


def test_error_message_is_cleared_by_a_good_call():
    with pytest.raises(tm.TTTError):
        block.ttt_linattn_workspace_size(attn_desc(batch=0))
    assert tm.ttt_last_error()
    block.ttt_linattn_workspace_size(attn_desc())
    assert tm.ttt_last_error() == ""
    assert block._load().ttt_linattn_workspace_size(ctypes.byref(attn_desc()), None) == INVALID


def test_binding_refuses_tensors():
    x = torch.zeros(2, 8, 4, 64)
    lg = torch.zeros(4)
    for bad in (dict(q=x[0]), dict(k=x.bfloat16()), dict(k=x[:, :7]), dict(v=x.transpose(2, 3)),
                dict(q=x[..., :32]), dict(log_decay=lg.double()), dict(log_decay=lg[:3]),
                dict(lengths=torch.zeros(2)), dict(state=torch.zeros(2, 4, 64, 32)),
                dict(state_out=torch.zeros(2, 4, 64, 64, dtype=torch.float64)),
                dict()):  # CPU tensors
        a = dict(q=x, k=x, v=x, log_decay=lg) | bad
        with pytest.raises(ValueError):
            block.linattn_forward(**a)
    with pytest.raises(ValueError):
        block.linattn_backward(x, x, x, lg, x[..., :32])
    w = torch.zeros(64)
    for bad in (dict(x=x.double()), dict(weight=w[:32]), dict(weight=w.bfloat16()),
                dict(res=x[:1]), dict(res=x.bfloat16()), dict(x=x.transpose(0, 1)),
                dict(out_dtype=torch.bfloat16), dict(res=None, r_out=x), dict(x=x[:0], res=None),
                dict(x=x[..., :0], res=None, weight=w[:0]), dict()):
        with pytest.raises(ValueError):
            block.add_rmsnorm(**(dict(x=x, res=x, weight=w) | bad))
    with pytest.raises(ValueError):
        block.add_rmsnorm_backward(x, x, w, dr=x[:1])


def test_attention_reference_against_differences():
    # the operator is linear in each of q, k, v and the state: differences are exact
    rng = np.random.default_rng(2)
    B, T, H, G, dk, dv = 2, 7, 4, 2, 5, 3
    n = rng.normal
    q, k, v = n(size=(B, T, H, dk)), n(size=(B, T, G, dk)), n(size=(B, T, G, dv))
    st, ds, dO = n(size=(B, H, dk, dv)), n(size=(B, H, dk, dv)), n(size=(B, T, H, dv))
    lg, ln = -rng.uniform(0, 1, size=H), [7, 4]
    dO[1, 4:] = 0  # outputs behind the end are constants
    grads = ref.linattn_grads(q, k, v, lg, 0.5, dO, st, ds, ln)

    def f(q, k, v, st):
        o, S = ref.linattn(q, k, v, lg, 0.5, st, ln)
        return (dO * o).sum() + (ds * S).sum()

    for i, g in enumerate(grads):
        a = [q, k, v, st]
        u = n(size=a[i].shape)
        hi, lo = list(a), list(a)
        hi[i], lo[i] = a[i] + u, a[i] - u
        assert abs((f(*hi) - f(*lo)) / 2 - (g * u).sum()) < 1e-9 * max(1, np.abs(g * u).sum())


# --------------------------------------------------- what the C ABI hands to the launches
# block_api.cpp with launches that only take down what they were given
LAUNCHES = r"""
#include <cstdarg>
#include "block.h"
#include "api_common.h"
extern "C" { int64_t seen[64]; int seen_count; }
namespace ttt {
namespace api {
ttt_status_t fail(ttt_status_t code, const char*, ...) { return code; }
ttt_status_t ok() { return TTT_OK; }
ttt_status_t hip_fail(hipError_t, const char*) { return TTT_ERR_HIP; }
Range range(const char* n, const void* p, size_t b) { return {n, (uintptr_t)p, (uintptr_t)p + b}; }
bool overlaps(const Range& x, const Range& y) { return x.lo < y.hi && y.lo < x.hi; }
bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }
}
hipError_t note(const LinArgs& a) {
  for (const LinOperand* o : {&a.q, &a.k, &a.v, &a.w}) if (o->p) seen[seen_count++] = o->st;
  return hipSuccess;
}
hipError_t launch_linattn_chunked(const LinArgs& a, float*, hipStream_t) { return note(a); }
hipError_t launch_linattn_step(const LinArgs& a, hipStream_t) { return note(a); }
hipError_t launch_linattn_starts(const LinArgs*, int, float*, hipStream_t) { return hipSuccess; }
hipError_t launch_linattn_sum_heads(const float*, void*, int64_t, const float*, void*, int64_t,
                                    int64_t, int64_t, int64_t, int64_t, Dtype, hipStream_t) {
  return hipSuccess;
}
bool linattn_square(int64_t dk, int64_t dv) { return (dk <= 64) == (dv <= 64); }
size_t linattn_segment_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, Dtype) { return 0; }
int64_t addnorm_backward_blocks(const NormArgs&) { return 1; }
hipError_t launch_addnorm_forward(const NormArgs&, const void*, const void*, const void*, void*,
                                  void*, float*, hipStream_t) { return hipSuccess; }
hipError_t launch_addnorm_backward(const NormArgs&, const void*, const void*, const void*,
                                   const void*, void*, void*, float*, float*, hipStream_t) {
  return hipSuccess;
}
}
"""


@pytest.fixture(scope="module")
def api(tmp_path_factory):
    d = tmp_path_factory.mktemp("api")
    (d / "launches.cpp").write_text(LAUNCHES)
    cmd = ["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__",
           "-I/opt/rocm/include", "-I" + hipbuild.CSRC, str(d / "launches.cpp"),
           os.path.join(hipbuild.CSRC, "block_api.cpp"), "-o", str(d / "api.so")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    lib, own = ctypes.CDLL(str(d / "api.so")), block._load()
    for name in ("ttt_linattn_forward", "ttt_linattn_backward"):
        getattr(lib, name).argtypes = getattr(own, name).argtypes
    return lib


@pytest.mark.skipif(not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"), reason="no HIP headers")
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d_value", [64, 128])
@pytest.mark.parametrize("st", [0, 64, 1 << 27, 1 << 30, (1 << 32) // 31 // 8 * 8, 1 << 40])
def test_one_tokens_stride_reaches_no_address(api, st, d_value, dtype):
    """The stride between tokens of a call of one token means nothing and may be anything.  The
    chunked kernels put a last chunk's tokens at the end of a tile of 32 and reach its rows by
    32-bit offsets, so a stride that is passed on has to keep 31 rows below 2^32 bytes."""
    d = attn_desc(seq_len=1, d_value=d_value, dtype=dtype, q_stride=(1 << 20, st, 64),
                  k_stride=(1 << 20, st, 64), v_stride=(1 << 20, st, 128),
                  o_stride=(1 << 20, st, 128))
    seen, count = (ctypes.c_int64 * 64).in_dll(api, "seen"), ctypes.c_int.in_dll(api, "seen_count")
    es = 2 if dtype == torch.bfloat16 else 4
    for call, args in ((api.ttt_linattn_forward, [at(1), at(2), at(3), at(4), None, None, None, at(8)]),
                       (api.ttt_linattn_backward, [at(1), at(2), at(3), at(4), None, None, at(7), None,
                                                   at(8), at(9), at(10), None])):
        count.value = 0
        assert call(ctypes.byref(d), *args, at(20), 1 << 29, None) == 0
        assert count.value >= 3
        for i in range(count.value):
            assert (31 * seen[i] + 128) * es < 1 << 32, (seen[i], es)


class FakeTensor(torch.Tensor):
    """Stands for a tensor of another device than the current one."""

    is_cuda = True

    @staticmethod
    def __new__(cls, address):
        t = torch.Tensor._make_subclass(cls, torch.zeros(1))
        t.address = address
        return t

    def data_ptr(self):
        return self.address

    def get_device(self):
        return 1


def test_null_streams_belong_to_their_device(monkeypatch):
    """A null handle is the null stream of the device that is current: a call without a stream, or
    with another device's default stream, makes the tensors' (the stream's) device current."""
    entered, handles = [], []
    device = [0]

    @contextlib.contextmanager
    def on(index):
        device[0] = getattr(index, "index", index)
        entered.append(device[0])
        yield
        device[0] = 0

    monkeypatch.setattr(torch.cuda, "device", on)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: device[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)

    class Lib:
        def __getattr__(self, name):
            return lambda *a: handles.append((device[0], a[-1])) or 0

    monkeypatch.setattr(block, "_load", Lib)
    t = [FakeTensor(at(i)) for i in range(13)]
    d, n = attn_desc(), norm_desc()
    second = FakeStream()
    second.cuda_stream, second.device = 0, torch.device("cuda", 1)
    for stream, want in ((None, (1, 0)), (second, (1, 0)), (0, (0, 0)), (0x5000, (0, 0x5000))):
        block.ttt_addnorm_forward(n, *t[:5], stream=stream)
        block.ttt_addnorm_backward(n, *t[:8], 0, stream=stream)
        block.ttt_linattn_forward(d, *t[:9], 0, stream=stream)
        block.ttt_linattn_backward(d, *t[:13], 0, stream=stream)
        assert handles == [want] * 4 and entered == ([1] * 4 if want[0] else [])
        handles.clear(), entered.clear()


def test_a_workspace_of_another_device_is_refused(monkeypatch):
    looked_at = []
    monkeypatch.setattr(block, "_same_device", lambda like, *t: looked_at.extend(t))
    for name in ("ttt_linattn_forward", "ttt_linattn_backward"):
        monkeypatch.setattr(block, name, lambda *a, **k: None)
    q, lg, ws = torch.zeros(1, 8, 4, 64), torch.zeros(4), torch.zeros(256, dtype=torch.uint8)
    block.linattn_forward(q, q, q, lg, ws=ws)
    assert any(t is ws for t in looked_at)
    looked_at.clear()
    block.linattn_backward(q, q, q, lg, q, ws=ws)
    assert any(t is ws for t in looked_at)


# ---------------------------------------------------------- plans kept between calls
def test_plans_take_the_values_of_scale_and_eps(monkeypatch):
    """A scale or an eps given as a tensor counts with its value at the call: the plans that are
    kept by shapes and values must not be found again by the tensor's identity."""
    seen = []
    for name in ("ttt_addnorm_forward", "ttt_addnorm_backward"):
        monkeypatch.setattr(block, name, lambda desc, *a, **k: seen.append(desc.eps))
    for name in ("ttt_linattn_forward", "ttt_linattn_backward"):
        monkeypatch.setattr(block, name, lambda desc, *a, **k: seen.append(desc.scale))
    x, w, q, lg = torch.zeros(2, 64), torch.zeros(64), torch.zeros(1, 8, 4, 64), torch.zeros(4)
    for call in (lambda t: block.add_rmsnorm(x, x, w, eps=t),
                 lambda t: block.add_rmsnorm_backward(x, x, w, eps=t),
                 lambda t: block.linattn_forward(q, q, q, lg, scale=t),
                 lambda t: block.linattn_backward(q, q, q, lg, q, scale=t)):
        t = torch.tensor(0.5)
        for value in (0.5, 0.25, 2.0):
            t.fill_(value)
            call(t)
            assert seen.pop() == value
        call(0.125)
        assert seen.pop() == 0.125
    block.linattn_forward(q, q, q, lg)
    assert seen.pop() == 0.125  # 64^-0.5


# ------------------------------------------------------------------ streams as arguments
class FakeStream:
    """Stands for torch's streams: one of the pool where no pointer, or a null one, is given."""

    def __init__(self, handle=0, device=None):
        self.cuda_stream = handle or 0xdead00


def test_a_stream_handle_is_the_stream_entered(monkeypatch):
    """A tensor-level call runs on the stream whose raw handle it is given, the null stream's 0
    among them: torch takes a null pointer as none and makes a stream of its own."""
    default = FakeStream()
    default.cuda_stream = 0
    entered = []

    @contextlib.contextmanager
    def stream(s):
        entered.append(s.cuda_stream)
        yield

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: default)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    for name in ("ttt_addnorm_forward", "ttt_addnorm_backward", "ttt_linattn_forward",
                 "ttt_linattn_backward"):
        monkeypatch.setattr(block, name, lambda *a, **k: None)
    x, w, q, lg = torch.zeros(2, 64), torch.zeros(64), torch.zeros(1, 8, 4, 64), torch.zeros(4)
    for s, handle in ((0, 0), (0x5000, 0x5000), (FakeStream(0x7000), 0x7000), (default, 0)):
        for call in (lambda s: block.add_rmsnorm(x, x, w, stream=s),
                     lambda s: block.add_rmsnorm_backward(x, x, w, stream=s),
                     lambda s: block.linattn_forward(q, q, q, lg, stream=s),
                     lambda s: block.linattn_backward(q, q, q, lg, q, stream=s)):
            call(s)
            assert entered.pop() == handle and not entered


# ---------------------------------------------------- the waits of the compiled kernels
VMEM = re.compile(r"^\s*(buffer|global|flat|scratch)_(load|store|atomic)\w*")


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not available")
def test_no_load_into_lds_is_in_flight_at_a_barrier(tmp_path):
    """The chunked kernels fill LDS tiles by direct loads and let other waves read them after a
    barrier: in the gfx950 code that hipcc makes, every barrier of such a kernel has vmcnt(0)
    in front of it with no vector memory operation in between."""
    src = os.path.join(hipbuild.CSRC, "linattn.hip")
    out = tmp_path / "linattn.s"
    cmd = ["/opt/rocm/bin/hipcc", f"--offload-arch={hipbuild.ARCH}", "-O3", "-std=c++17",
           "--cuda-device-only", "-S", "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", src, "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    functions, name = {}, None
    for line in out.read_text().splitlines():
        m = re.match(r"^(_Z\w+):", line)
        if m:
            name = m.group(1)
            functions[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name:
            functions[name].append(line)
    checked = 0
    for name, lines in functions.items():
        if not any("buffer_load" in x and x.rstrip().endswith("lds") for x in lines):
            continue
        assert not any("scratch_" in x for x in lines), name  # nothing spilled either
        for i, x in enumerate(lines):
            if "s_barrier" not in x:
                continue
            j = i - 1
            while not re.search(r"s_waitcnt.*vmcnt\(0\)", lines[j]):
                assert not VMEM.match(lines[j]), (name, lines[j])
                assert not re.match(r"^\.LBB", lines[j]), (name, "no wait in the barrier's block")
                j -= 1
            checked += 1
    assert checked >= 2 * 20, checked


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not available")
def test_the_librarys_own_build_waits_at_barriers(tmp_path):
    """The same of the code that the library is built from: with the compiler and the flags of
    build.py, whatever they become."""
    out = tmp_path / "linattn.s"
    flags = [f for f in hipbuild.HIPCC_FLAGS if f != "-shared"]
    cmd = [hipbuild.hipcc(), *flags, "--cuda-device-only", "-S",
           os.path.join(hipbuild.CSRC, "linattn.hip"), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    kernels = [k for k in re.split(r"^(?=_Z\w+:)", out.read_text(), flags=re.M)
               if re.search(r"buffer_load\w* .*\blds$", k, re.M)]
    barriers = 0
    for k in kernels:
        lines = k.split(".Lfunc_end")[0].splitlines()
        assert not any("scratch_" in x for x in lines), lines[0]
        waited = False  # vmcnt(0) behind the last vector memory operation of this block
        for x in lines:
            if VMEM.match(x) or re.match(r"^\.LBB", x):
                waited = False
            elif re.search(r"s_waitcnt.*vmcnt\(0\)", x):
                waited = True
            elif "s_barrier" in x:
                assert waited, lines[0]
                barriers += 1
    assert len(kernels) >= 20 and barriers >= 2 * len(kernels), (len(kernels), barriers)
