"""Refusals of the paged-cache calls, on the host: C entry points with addresses
that are never dereferenced, and the binding with host tensors.  CPU only."""

import ctypes
import types

import pytest
import torch

import global_attention_swa_b200 as mimo

FAKE = 0x10000
INVALID, UNSUPPORTED, WORKSPACE, OK = (mimo.MIMO_ERR_INVALID_ARG, mimo.MIMO_ERR_UNSUPPORTED,
                                       mimo.MIMO_ERR_WORKSPACE, mimo.MIMO_OK)


def p(x):
    return ctypes.c_void_p(x) if x else None


def _attend(hq=64, hkv=4, dqk=192, q=FAKE, k=FAKE, v=FAKE, table=FAKE, cu=FAKE, lens=FAKE, seqs=2, total=8,
            most=4, pages=16, ps=64, width=4, window=0, sinks=None, out=FAKE, lse=None, ws=FAKE, wsb=1 << 40):
    d = mimo.make_dims(hq, hkv, dqk)
    return mimo.lib.mimo_attn_paged_attention(ctypes.byref(d), p(q), p(k), p(v), p(table), p(cu), p(lens), seqs,
                                              total, most, pages, ps, width, window, p(sinks), p(out), p(lse),
                                              p(ws), wsb, None)


@pytest.mark.parametrize("bad,status", [
    (dict(hq=6, hkv=4), INVALID), (dict(dqk=128), UNSUPPORTED), (dict(hq=129, hkv=1), UNSUPPORTED),
    (dict(window=-1), INVALID), (dict(seqs=-1), INVALID), (dict(total=-1), INVALID), (dict(most=-1), INVALID),
    (dict(most=9), INVALID), (dict(pages=0), INVALID), (dict(ps=0), INVALID), (dict(width=0), INVALID),
    (dict(ps=8), UNSUPPORTED), (dict(ps=40), UNSUPPORTED), (dict(pages=1 << 26), UNSUPPORTED),
    (dict(width=1 << 26), UNSUPPORTED), (dict(pages=(1 << 25) - 1), UNSUPPORTED), (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID),
    (dict(out=0), INVALID), (dict(table=0), INVALID), (dict(cu=0), INVALID), (dict(lens=0), INVALID),
    (dict(q=FAKE + 2), INVALID), (dict(k=FAKE + 8), INVALID), (dict(out=FAKE + 4), INVALID),
    (dict(lse=FAKE + 2), INVALID), (dict(sinks=FAKE + 1), INVALID), (dict(table=FAKE + 2), INVALID),
    (dict(lens=FAKE + 1), INVALID), (dict(cu=FAKE + 3), INVALID),
])
def test_attention_refuses(bad, status):
    assert _attend(**bad) == status
    assert mimo.lib.mimo_attn_last_error().decode()


def test_attention_workspace_contract():
    need = mimo.mimo_attn_paged_attention_workspace_size(64, 4, 2, 8, 4)
    assert need > 0
    assert _attend(ws=0) == WORKSPACE and _attend(wsb=need - 1) == WORKSPACE and _attend(ws=FAKE + 8) == WORKSPACE
    assert "workspace" in mimo.lib.mimo_attn_last_error().decode()
    # more rows to a sequence: twice the rows to a part; a short window: no parts
    assert mimo.mimo_attn_paged_attention_workspace_size(64, 4, 2, 80, 40) > need
    assert mimo.mimo_attn_paged_attention_workspace_size(64, 4, 2, 80, 40, 129) == 0
    assert mimo.mimo_attn_paged_attention_workspace_size(64, 4, 2, 80, 40, 4096) > 0
    assert mimo.mimo_attn_paged_attention_workspace_size(64, 4, 0, 0, 0) == 0


def test_attention_of_nothing_is_a_no_op():
    assert _attend(seqs=0) == OK
    assert _attend(total=0, most=0) == OK
    assert _attend(most=0) == OK


def _append(hq=64, hkv=4, q=FAKE, qo=FAKE, k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, seqs=2, total=8, pages=16, ps=64,
            width=4, theta=1e4, rd=192, lens=FAKE):
    d = mimo.make_dims(hq, hkv)
    return mimo.lib.mimo_attn_paged_append(ctypes.byref(d), p(q), p(qo), p(k), p(v), p(kp), p(vp), p(FAKE), p(FAKE),
                                           p(lens), seqs, total, pages, ps, width, theta, rd, None)


@pytest.mark.parametrize("bad,status", [
    (dict(theta=0.0), INVALID), (dict(theta=float("nan")), INVALID), (dict(theta=float("inf")), INVALID),
    (dict(rd=7), INVALID), (dict(rd=194), INVALID), (dict(rd=-2), INVALID), (dict(q=0), INVALID),
    (dict(qo=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(kp=0), INVALID), (dict(vp=0), INVALID),
    (dict(q=FAKE + 2), INVALID), (dict(vp=FAKE + 8), INVALID), (dict(ps=24), UNSUPPORTED), (dict(lens=0), INVALID),
    (dict(total=-1), INVALID), (dict(hq=6), INVALID),
])
def test_append_refuses(bad, status):
    assert _append(**bad) == status


def test_append_of_nothing_is_a_no_op():
    assert _append(seqs=0) == OK and _append(total=0) == OK


def _hold(refs=FAKE, pages=16, table=FAKE, seqs=2, width=4, ps=64, lens=FAKE, first=None, wf=None, ro=FAKE,
          to=FAKE, moves=FAKE, info=FAKE, ws=FAKE, wsb=1 << 20):
    return mimo.lib.mimo_attn_page_hold(p(refs), pages, p(table), seqs, width, ps, p(lens), p(first), p(wf), p(ro),
                                        p(to), p(moves), p(info), p(ws), wsb, None)


@pytest.mark.parametrize("bad,status", [
    (dict(pages=0), INVALID), (dict(seqs=-1), INVALID), (dict(width=-1), INVALID), (dict(ps=0), INVALID),
    (dict(refs=0), INVALID), (dict(table=0), INVALID), (dict(ro=0), INVALID), (dict(to=0), INVALID),
    (dict(lens=0), INVALID), (dict(moves=0), INVALID), (dict(info=0), INVALID), (dict(ws=0), WORKSPACE),
    (dict(wsb=67), WORKSPACE), (dict(seqs=1 << 16, width=1 << 15), UNSUPPORTED),
    (dict(ps=1 << 30, width=4), UNSUPPORTED), (dict(first=FAKE + 2), INVALID), (dict(wf=FAKE + 1), INVALID),
    (dict(refs=FAKE + 2), INVALID), (dict(to=FAKE + 1), INVALID),
])
def test_hold_refuses(bad, status):
    assert _hold(**bad) == status


def _fork(refs=FAKE, pages=16, table=0x100000, seqs=2, width=4, parent=FAKE, n=2, ro=FAKE, to=0x200000):
    return mimo.lib.mimo_attn_page_fork(p(refs), pages, p(table), seqs, width, p(parent), n, p(ro), p(to), None)


@pytest.mark.parametrize("bad,status", [
    (dict(pages=0), INVALID), (dict(n=-1), INVALID), (dict(refs=0), INVALID), (dict(table=0), INVALID),
    (dict(parent=0), INVALID), (dict(ro=0), INVALID), (dict(to=0), INVALID), (dict(to=0x100000), INVALID),
    (dict(to=0x100000 + 28), INVALID), (dict(table=0x200000 + 28), INVALID), (dict(parent=FAKE + 2), INVALID),
    (dict(n=1 << 16, width=1 << 15), UNSUPPORTED),
])
def test_fork_refuses(bad, status):
    assert _fork(**bad) == status


def _compact(refs=FAKE, pages=16, table=FAKE, most=4, moves=FAKE, info=FAKE, ws=FAKE, wsb=1 << 20):
    return mimo.lib.mimo_attn_page_compact(p(refs), pages, p(table), 2, 4, most, p(FAKE), p(FAKE), p(moves), p(info),
                                           p(ws), wsb, None)


@pytest.mark.parametrize("bad,status", [
    (dict(pages=0), INVALID), (dict(most=-1), INVALID), (dict(moves=0), INVALID), (dict(info=0), INVALID),
    (dict(ws=0), WORKSPACE), (dict(wsb=63), WORKSPACE), (dict(refs=0), INVALID), (dict(table=0), INVALID),
])
def test_compact_refuses(bad, status):
    assert _compact(**bad) == status


def _copy(hkv=4, k=FAKE, v=FAKE, layers=2, pages=16, ps=64, moves=FAKE, n=3):
    d = mimo.make_dims(hkv, hkv)
    return mimo.lib.mimo_attn_page_copy(ctypes.byref(d), p(k), p(v), layers, pages, ps, p(moves), n, None)


@pytest.mark.parametrize("bad,status", [
    (dict(layers=-1), INVALID), (dict(n=-1), INVALID), (dict(pages=0), INVALID), (dict(ps=0), INVALID),
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(moves=0), INVALID), (dict(k=FAKE + 8), INVALID),
    (dict(moves=FAKE + 2), INVALID), (dict(ps=1 << 27), UNSUPPORTED),
])
def test_copy_refuses(bad, status):
    assert _copy(**bad) == status


def test_copy_of_nothing_is_a_no_op():
    assert _copy(n=0) == OK and _copy(layers=0) == OK


class _Recorder:
    """A stand-in library: the workspace sizes, and which calls were made."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return 64 if name.endswith("_workspace_size") else 0
        return fn


@pytest.fixture
def host(monkeypatch):
    """The binding on host tensors, its device check alone bypassed."""
    real = mimo._ptr

    def host_ptr(t, name="tensor", dtype=None):
        if t is None:
            return None
        return real(types.SimpleNamespace(is_cuda=True, is_contiguous=t.is_contiguous, dtype=t.dtype,
                                          data_ptr=t.data_ptr), name, dtype)

    def host_addr(t, name, dtype, shape, dev):
        if t is None:
            return 0
        mimo._shape(t, shape, name)
        mimo._same_device(dev, **{name: t})
        return host_ptr(t, name, dtype).value

    lib = _Recorder()
    monkeypatch.setattr(mimo, "_addr", host_addr)
    monkeypatch.setattr(mimo, "lib", lib)
    monkeypatch.setattr(mimo, "_ptr", host_ptr)
    monkeypatch.setattr(mimo, "_stream", lambda stream, dev: None)
    return lib


BF, I32 = torch.bfloat16, torch.int32


def _inputs():
    z = lambda *s, dt=BF: torch.zeros(s, dtype=dt)  # noqa: E731
    return dict(q=z(10, 8, 192), kp=z(6, 16, 2, 192), vp=z(6, 16, 2, 128), table=z(3, 4, dt=I32), cu=z(4, dt=I32),
                lens=z(3, dt=I32), sinks=torch.zeros(8), k=z(10, 2, 192), v=z(10, 2, 128), refs=z(6, dt=I32))


def _call_attend(x, **kw):
    return mimo.mimo_attn_paged_attention(x["q"], x["kp"], x["vp"], x["table"], x["cu"], x["lens"], 5, 0, x["sinks"], **kw)


def _call_append(x, **kw):
    return mimo.mimo_attn_paged_append(x["q"], x["k"], x["v"], x["kp"], x["vp"], x["table"], x["cu"], x["lens"], 1e4, **kw)


def _call_hold(x, **kw):
    return mimo.mimo_attn_page_hold(x["refs"], x["table"], x["lens"], 16, **kw)


def test_wrappers_accept_their_documented_arguments(host):
    x = _inputs()
    for dt in (BF, torch.float32):
        out, lse = _call_attend(x, out_dtype=dt)
        assert out.shape == (10, 8, 128) and out.dtype == dt and lse.shape == (8, 10)
    assert _call_attend(x, return_lse=False)[1] is None
    assert _call_append(x).shape == x["q"].shape
    assert _call_append(x, q_out=x["q"]) is x["q"]
    refs, table, moves, info = _call_hold(x, first=x["lens"], write_from=x["lens"])
    assert refs.shape == (6,) and table.shape == (3, 4) and moves.shape == (3, 2) and info.shape == (2,)
    refs, table = mimo.mimo_attn_page_fork(x["refs"], x["table"], torch.zeros(5, dtype=I32))
    assert table.shape == (5, 4)
    refs, table, moves, info = mimo.mimo_attn_page_compact(x["refs"], x["table"], 3)
    assert moves.shape == (3, 2)
    mimo.mimo_attn_page_copy(x["kp"], x["vp"], moves)
    mimo.mimo_attn_page_copy(x["kp"][None], x["vp"][None], moves)
    assert {n for n, _ in host.calls if not n.endswith("_size")} == {
        "mimo_attn_paged_attention", "mimo_attn_paged_append", "mimo_attn_page_hold", "mimo_attn_page_fork",
        "mimo_attn_page_compact", "mimo_attn_page_copy"}


@pytest.mark.parametrize("name,change,error,match", [
    ("kp", lambda t: t[:, :, :1], ValueError, "v_pages|k_pages|contiguous"),
    ("kp", lambda t: t[0], ValueError, "k_pages"),
    ("vp", lambda t: t[:5], ValueError, "v_pages"),
    ("table", lambda t: t[:2], ValueError, "cu_seqlens_q"),
    ("table", lambda t: t[0], ValueError, "block_table"),
    ("table", lambda t: t.long(), TypeError, "block_table"),
    ("cu", lambda t: t[:3], ValueError, "cu_seqlens_q"),
    ("cu", lambda t: t.long(), TypeError, "cu_seqlens_q"),
    ("lens", lambda t: t[:2], ValueError, "seqlens"),
    ("sinks", lambda t: t[:4], ValueError, "sinks"),
    ("sinks", lambda t: t.double(), TypeError, "sinks"),
    ("q", lambda t: t.half(), TypeError, "q must be"),
    ("q", lambda t: t.transpose(0, 1).contiguous().transpose(0, 1), ValueError, "contiguous"),
    ("kp", lambda t: t.float(), TypeError, "k_pages"),
    ("vp", lambda t: t.to("meta"), ValueError, "v_pages is on meta"),
])
def test_attention_wrapper_refuses(host, name, change, error, match):
    x = _inputs()
    x[name] = change(x[name])
    with pytest.raises(error, match=match):
        _call_attend(x)
    assert not [n for n, _ in host.calls if not n.endswith("_size")]


def test_other_wrappers_refuse(host):
    x = _inputs()
    with pytest.raises(ValueError, match="k_new"):
        mimo.mimo_attn_paged_append(x["q"], x["k"][:9], x["v"], x["kp"], x["vp"], x["table"], x["cu"], x["lens"], 1e4)
    with pytest.raises(ValueError, match="q_out"):
        _call_append(x, q_out=x["q"][:9])
    for kw in (dict(first=x["lens"][:2]), dict(write_from=x["lens"][:1]), dict(moves=torch.zeros((2, 2), dtype=I32)),
               dict(refs_out=x["refs"][:5]), dict(table_out=x["table"][:, :3]), dict(info=torch.zeros(3, dtype=I32))):
        with pytest.raises(ValueError, match=next(iter(kw))):
            _call_hold(x, **kw)
    with pytest.raises(TypeError, match="page_refs"):
        mimo.mimo_attn_page_hold(x["refs"].long(), x["table"], x["lens"], 16)
    with pytest.raises(ValueError, match="parent"):
        mimo.mimo_attn_page_fork(x["refs"], x["table"], torch.zeros((2, 2), dtype=I32))
    with pytest.raises(ValueError, match="moves"):
        mimo.mimo_attn_page_compact(x["refs"], x["table"], 3, moves=torch.zeros((4, 2), dtype=I32))
    with pytest.raises(ValueError, match="moves"):
        mimo.mimo_attn_page_copy(x["kp"], x["vp"], torch.zeros((4, 3), dtype=I32))
    with pytest.raises(ValueError, match="layer axis"):
        mimo.mimo_attn_page_copy(x["kp"], x["vp"][None], torch.zeros((4, 2), dtype=I32))
    with pytest.raises(ValueError, match="v_pages"):
        mimo.mimo_attn_page_copy(x["kp"], x["vp"][:5], torch.zeros((4, 2), dtype=I32))
    assert not [n for n, _ in host.calls if not n.endswith("_size")]


@pytest.mark.parametrize("big", [2 ** 31, -2 ** 31 - 1, 2 ** 32 + 1, 2 ** 70])
def test_whole_numbers_past_32_bits_are_refused(host, big):
    x = _inputs()
    att = (x["q"], x["kp"], x["vp"], x["table"], x["cu"], x["lens"])
    for call, what in ((lambda: mimo.mimo_attn_paged_attention(*att, big, 0, x["sinks"]), "max_seqlen_q"),
                       (lambda: mimo.mimo_attn_paged_attention(*att, 5, big, x["sinks"]), "window"),
                       (lambda: _call_append(x, rotary_dim=big), "rotary_dim"),
                       (lambda: mimo.mimo_attn_page_hold(x["refs"], x["table"], x["lens"], big), "page_size"),
                       (lambda: mimo.mimo_attn_page_compact(x["refs"], x["table"], big), "max_moves")):
        with pytest.raises(ValueError, match=what):
            call()
    assert not [n for n, _ in host.calls if not n.endswith("_size")]


def test_a_scale_given_as_a_tensor_is_read_at_each_call(host):
    scale = torch.tensor(0.5)
    for want in (0.5, 0.25):
        scale.fill_(want)
        _call_attend(_inputs(), softmax_scale=scale, v_scale=2 * scale)
        dims = host.calls[-1][1][0]._obj
        assert (dims.softmax_scale, dims.v_scale) == (want, 2 * want)


def test_paged_cache_refuses_sizes():
    from global_attention_swa_b200.paged_cache import PagedCache

    for bad in (dict(num_pages=0), dict(page_size=24), dict(window=-1), dict(rollback=-1), dict(num_layers=0)):
        with pytest.raises(ValueError):
            PagedCache(**{**dict(num_layers=1, num_pages=4, page_size=16, num_seqs=2, max_pages=2, device="cpu"), **bad})


def test_native_calls_leave_what_is_not_plain_to_the_binding():
    """Host tensors, wrong counts of arguments and things that are no tensors: the native
    part of the binding says None, and the wrapper goes on to say what is wrong."""
    if mimo._fast is None:
        pytest.skip("the native part of the binding is not built")
    x = _inputs()
    args = (x["q"], x["kp"], x["vp"], x["table"], x["cu"], x["lens"], 5, 0, x["sinks"], None, None, None, False, 0.0,
            1.0, True)
    assert mimo._fast.paged_attention(*args) is None
    assert mimo._fast.paged_attention(*args[:-1]) is None
    assert mimo._fast.paged_attention(None, *args[1:]) is None
    assert mimo._fast.page_hold(x["refs"], x["table"], x["lens"], 16, *[None] * 7) is None
    assert mimo._fast.page_fork(x["refs"], x["table"], x["lens"], None, None) is None
    assert mimo._fast.page_compact(x["refs"], x["table"], 3, *[None] * 5) is None
    assert mimo._fast.page_copy(x["kp"], x["vp"], torch.zeros((1, 2), dtype=I32)) is None
    assert mimo._fast.paged_append(x["q"], x["k"], x["v"], x["kp"], x["vp"], x["table"], x["cu"], x["lens"], 1e4, 192,
                                   None) is None
    with pytest.raises(TypeError):
        mimo._fast.bind(1, 2)
    with pytest.raises(ValueError, match="CUDA"):
        _call_hold(x)
