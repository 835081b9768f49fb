"""What the operators between a hidden state and text refuse, through the C ABI
and the binding, without a device: every check here comes before any launch."""
import ctypes
import threading
import time

import numpy as np
import pytest
import torch

import answers


@pytest.fixture(scope="module")
def bpe():
    import bpe_merge_amd
    return bpe_merge_amd


HOST = (ctypes.c_uint8 * 65536)()
P = ctypes.addressof(HOST)


def _norm(bpe, **change):
    a = dict(x=P, xs=256, r=None, rs=0, w=P, kind=0, rows=2, d=256, eps=1e-5, sum=None, ss=0, q=P, qs=256, s=P)
    a.update(change)
    return bpe._lib.bpe_norm_quant(a["x"], a["xs"], a["r"], a["rs"], a["w"], a["kind"], a["rows"], a["d"], a["eps"],
                                   a["sum"], a["ss"], a["q"], a["qs"], a["s"], None)


@pytest.mark.parametrize("change, word", [
    (dict(kind=3), "type"), (dict(kind=-1), "type"), (dict(d=0), "d = 0"), (dict(d=65537), "65537"),
    (dict(rows=1 << 31), "rows"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(xs=255), "stride"),
    (dict(r=P, rs=255), "stride"), (dict(sum=P + 4, ss=255), "stride"), (dict(qs=255), "stride"),
    (dict(sum=P, ss=512), "in place"), (dict(r=P + 4, rs=256, sum=P + 4, ss=300), "in place"), (dict(x=P + 2), "aligned"),
    (dict(kind=2, w=P + 1), "aligned"), (dict(s=P + 2), "aligned"), (dict(x=None), "x must be non-NULL"),
    (dict(), "device memory")])
def test_norm_quant_refuses(bpe, change, word):
    assert _norm(bpe, **change) == bpe.EINVAL
    assert word in bpe._lib.bpe_last_error().decode()


def test_norm_quant_of_no_rows_needs_no_device(bpe):
    assert _norm(bpe, rows=0, x=None, w=None, q=None, s=None) == bpe.OK


@pytest.mark.parametrize("change", [
    dict(sum=P + 4, ss=256), dict(sum=P + 1024, ss=256), dict(sum=P + 1020, ss=300), dict(x=P + 8192, r=P, rs=256, sum=P + 2044, ss=256),
    dict(sum=P, ss=256, r=P + 512, rs=256)])
def test_norm_quant_refuses_a_sum_over_part_of_its_inputs(bpe, change):
    assert _norm(bpe, **change) == bpe.EINVAL
    assert "share no memory" in bpe._lib.bpe_last_error().decode()


@pytest.mark.parametrize("change", [
    dict(sum=P, ss=256), dict(r=P, rs=256, sum=P, ss=256), dict(x=P + 8192, r=P, rs=256, sum=P, ss=256), dict(sum=P + 2048, ss=256),
    dict(xs=600, sum=P + 1024, ss=600), dict(xs=600, r=P + 1024, rs=600, sum=P + 1024, ss=600), dict(rows=1, sum=P + 1024, ss=256)])
def test_norm_quant_takes_a_sum_in_place_or_beside_its_inputs(bpe, change):
    assert _norm(bpe, **change) == bpe.EINVAL  # host memory, which is looked at last
    assert "device memory" in bpe._lib.bpe_last_error().decode()


def _product(bpe, **change):
    a = dict(a=P, as_=256, sa=P, sas=2, b=P, bs=256, sb=P, sbs=2, m=4, n=8, k=256, out=P, os=8, kind=0)
    a.update(change)
    return bpe._lib.bpe_matmul_scaled(a["a"], a["as_"], a["sa"], a["sas"], a["b"], a["bs"], a["sb"], a["sbs"], a["m"],
                                      a["n"], a["k"], a["out"], a["os"], a["kind"], None)


@pytest.mark.parametrize("change, word", [
    (dict(kind=9), "type"), (dict(k=0), "k = 0"), (dict(m=0x7FFF81), "at most"), (dict(n=0x7FFF81), "at most"),
    (dict(k=0x7FFF81), "at most"), (dict(as_=255), "stride"), (dict(bs=100), "stride"), (dict(os=7), "stride"),
    (dict(sas=1), "stride"), (dict(n=300, os=300, sbs=1), "stride"), (dict(sa=P + 1), "aligned"),
    (dict(out=P + 2), "aligned"), (dict(a=None), "a must be non-NULL"), (dict(), "device memory")])
def test_matmul_scaled_refuses(bpe, change, word):
    assert _product(bpe, **change) == bpe.EINVAL
    assert word in bpe._lib.bpe_last_error().decode()


def test_matmul_scaled_of_nothing_needs_no_device(bpe):
    assert _product(bpe, m=0, a=None, out=None) == bpe.OK
    assert _product(bpe, n=0, b=None, out=None) == bpe.OK


@pytest.mark.parametrize("change, word", [
    (dict(kind=5), "type"), (dict(n=0x7FFF81), "at most"), (dict(ws=10), "stride"), (dict(qs=10), "stride"),
    (dict(w=P + 1), "aligned"), (dict(w=None), "w must be non-NULL"), (dict(), "device memory")])
def test_quant_weight_refuses(bpe, change, word):
    a = dict(w=P, ws=64, kind=0, n=4, k=64, q=P, qs=64, s=P)
    a.update(change)
    assert bpe._lib.bpe_quant_weight(a["w"], a["ws"], a["kind"], a["n"], a["k"], a["q"], a["qs"], a["s"],
                                     None) == bpe.EINVAL
    assert word in bpe._lib.bpe_last_error().decode()


def _sample(bpe, how=None, **change):
    a = dict(x=P, stride=100, kind=0, rows=2, v=100, u=P, ids=P, logp=None)
    s = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    for key in list(change):
        (s if key in s or key.endswith("s") and key[:-1] in s else a)[key] = change[key]
    h = bpe.Sampling(**s)
    return bpe._lib.bpe_sample(a["x"], a["stride"], a["kind"], a["rows"], a["v"], a["u"],
                               None if how == "null" else ctypes.byref(h), a["ids"], a["logp"], None)


@pytest.mark.parametrize("change, word", [
    (dict(kind=3), "type"), (dict(v=0), "vocab"), (dict(v=1048577, stride=1048577), "vocab"), (dict(how="null"), "settings"),
    (dict(temperature=-0.1), "temperature"), (dict(temperature=float("nan")), "temperature"), (dict(top_k=-1), "top_k"),
    (dict(top_p=0.0), "top_p"), (dict(top_p=1.01), "top_p"), (dict(top_p=float("nan")), "top_p"), (dict(min_p=-0.1), "min_p"),
    (dict(min_p=1.1), "min_p"), (dict(min_p=float("nan")), "min_p"), (dict(stride=99), "stride"), (dict(x=P + 1), "aligned"),
    (dict(ids=P + 2), "aligned"), (dict(x=None), "logits must be non-NULL"), (dict(), "device memory")])
def test_sample_refuses(bpe, change, word):
    assert _sample(bpe, **change) == bpe.EINVAL
    assert word in bpe._lib.bpe_last_error().decode()


def test_sample_of_no_rows_needs_no_device(bpe):
    assert _sample(bpe, rows=0, x=None, u=None, ids=None) == bpe.OK


def test_decoder_refuses(bpe):
    lib = bpe._lib
    h = ctypes.c_void_p()
    m = np.array([[97, 98, 5], [256, 300, 4]], dtype=np.uint32)
    assert lib.bpe_decoder_build(None, 1, ctypes.byref(h)) == bpe.EINVAL
    assert lib.bpe_decoder_build(m.ctypes.data, 1, None) == bpe.EINVAL
    assert lib.bpe_decoder_build(m.ctypes.data, 65281, ctypes.byref(h)) == bpe.EIDSPACE
    assert lib.bpe_decoder_build(m.ctypes.data, 2, ctypes.byref(h)) == bpe.EINVAL
    assert "does not exist" in lib.bpe_last_error().decode()
    double = np.array([[97, 97, 1]] + [[255 + i, 255 + i, 1] for i in range(1, 30)], dtype=np.uint32)
    assert lib.bpe_decoder_build(double.ctypes.data, 30, ctypes.byref(h)) == bpe.EINVAL
    assert "string" in lib.bpe_last_error().decode()
    assert not h.value
    n = ctypes.c_size_t(7)
    assert lib.bpe_decoder_decode(None, P, 4, None, P, 100, None, ctypes.byref(n)) == bpe.EINVAL
    assert lib.bpe_decoder_info(None, None, None) == bpe.EINVAL
    lib.bpe_decoder_free(None)


def test_the_binding_refuses_host_tensors_and_wrong_types(bpe):
    x = torch.zeros(4, 256)
    q = torch.zeros(4, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(TypeError, match="CUDA"):
        bpe.norm_quant(x, torch.ones(256))
    with pytest.raises(TypeError, match="CUDA"):
        bpe.quant_weight(x)
    with pytest.raises(TypeError, match="CUDA"):
        bpe.matmul_scaled(q, torch.ones(4, 2), q, torch.ones(1, 2))
    with pytest.raises(TypeError, match="CUDA"):
        bpe.sample(x, torch.zeros(4))


class Recorder:
    """In the library's place: keeps what bpe_sample is called with."""

    def bpe_sample(self, logits, stride, kind, rows, vocab, u, how, ids, logp, stream):
        h = how._obj
        self.top_k = h.top_k
        self.top_ks = list((ctypes.c_int32 * rows).from_address(h.top_ks)) if h.top_ks else None
        return 0


@pytest.fixture
def recorder(bpe, monkeypatch):
    r = Recorder()
    monkeypatch.setattr(bpe, "_lib", r)
    monkeypatch.setattr(bpe, "_cuda", lambda t, name, dtype=None: t)
    monkeypatch.setattr(bpe, "_stream_handle", lambda device: None)
    return r


def test_a_top_k_past_32_bits_is_not_another_one(bpe, recorder):
    x, u = torch.zeros(2, 40), torch.zeros(2)
    for given in (0, 1, 7, 0x7FFFFFFF, 1 << 20):
        bpe.sample(x, u, top_k=given)
        assert recorder.top_k == given
    for given in (1 << 31, (1 << 32) + 1, 1 << 32, 1 << 80):  # all of a row
        bpe.sample(x, u, top_k=given)
        assert recorder.top_k >= bpe.SAMPLE_MAX_VOCAB
    for given in (-1, -(1 << 31) - 1, -(1 << 32) + 5):  # for the library to refuse
        bpe.sample(x, u, top_k=given)
        assert recorder.top_k < 0
    with pytest.raises(TypeError):
        bpe.sample(x, u, top_k=5.0)


def test_row_top_ks_past_32_bits_are_not_other_ones(bpe, recorder):
    x, u = torch.zeros(5, 40), torch.zeros(5)
    bpe.sample(x, u, top_k=torch.tensor([0, 1, -3, 1 << 30, 7], dtype=torch.int32))
    assert recorder.top_ks == [0, 1, -3, 1 << 30, 7]
    bpe.sample(x, u, top_k=torch.tensor([3, (1 << 32) + 1, 1 << 31, -(1 << 32) + 5, 0]))
    k = recorder.top_ks
    assert k[0] == 3 and k[1] >= bpe.SAMPLE_MAX_VOCAB and k[2] >= bpe.SAMPLE_MAX_VOCAB and k[3] <= 0 and k[4] == 0
    for dtype in (torch.uint8, torch.int16):
        bpe.sample(x, u, top_k=torch.tensor([3, 100, 0, 1, 7], dtype=dtype))
        assert recorder.top_ks == [3, 100, 0, 1, 7]
    bpe.sample(x, u, top_k=torch.tensor([3.0, 1e30, 0.0, -1e30, 7.0]))
    k = recorder.top_ks
    assert k[0] == 3 and k[1] >= bpe.SAMPLE_MAX_VOCAB and k[2] == 0 and k[3] <= 0 and k[4] == 7


def test_threads_that_share_a_decoder_take_turns(bpe, monkeypatch):
    """Calls on one decoder must not overlap, nor one with its end; the
    interpreter's lock is not held during a call."""
    class Busy:
        inside = most = calls = freed = 0

        def enter(self):
            self.inside += 1
            self.most = max(self.most, self.inside)
            time.sleep(0.002)
            self.inside -= 1

        def bpe_decoder_decode(self, handle, tokens, n, stream, out, room, places, n_bytes):
            self.calls += 1
            self.enter()
            n_bytes._obj.value = 0
            return 0 if handle.value and not self.freed else bpe.EINVAL

        def bpe_last_error(self):
            return b"freed"

        bpe_strerror = lambda self, status: b"invalid"  # noqa: E731

        def bpe_decoder_free(self, handle):
            self.enter()
            self.freed += 1

        def bpe_decoder_info(self, handle, vocab, longest):
            longest._obj.value = 1
            return 0

        def bpe_decoder_build(self, merges, n, handle):
            handle._obj.value = 1
            return 0

    busy = Busy()
    monkeypatch.setattr(bpe, "_lib", busy)
    monkeypatch.setattr(bpe, "_cuda", lambda t, name, dtype=None: t)
    monkeypatch.setattr(bpe, "_stream_handle", lambda device: None)
    monkeypatch.setattr(bpe, "_merge_list", lambda merges, device: torch.zeros(0, 3, dtype=torch.int32))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    d = bpe.Decoder([])
    tokens, failed = torch.zeros(3, dtype=torch.int32), []

    def work(times):
        try:
            for _ in range(times):
                d.decode(tokens)
                time.sleep(0.0005)
        except Exception as e:
            failed.append(e)
    try:
        threads = [threading.Thread(target=work, args=(10,)) for _ in range(4)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not failed and busy.calls == 40 and busy.most == 1
        late = threading.Thread(target=work, args=(5000,))  # meets free(): the library's error for no decoder
        late.start()
        time.sleep(0.003)
        d.free()
        late.join()
        assert busy.freed == 1 and busy.most == 1
        assert len(failed) == 1 and isinstance(failed[0], bpe.BpeError)
    finally:
        d._h = ctypes.c_void_p(None)  # not the library's to release


# the 64-bit forms themselves

def test_the_plain_draw_by_hand():
    logits = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    ids = [answers.draw(logits, u, 1.0, 0, 1.0, 0.0)[0] for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.69, 0.71, 0.99, 1.0)]
    assert ids == [0, 0, 1, 1, 2, 2, 3, 3, 3]
    assert [answers.draw(logits, u, 1.0, 2, 1.0, 0.0)[0] for u in (0.0, 0.57, 0.58)] == [1, 1, 3]
    assert [answers.draw(logits, u, 1.0, 0, 0.69, 0.0)[0] for u in (0.0, 0.57, 0.58)] == [1, 1, 3]
    assert [answers.draw(logits, u, 1.0, 0, 0.71, 0.0)[0] for u in (0.0, 0.5, 0.99)] == [1, 2, 3]
    assert [answers.draw(logits, u, 1.0, 0, 1.0, 0.6)[0] for u in (0.0, 0.58, 0.99)] == [1, 3, 3]
    assert answers.draw(logits, 0.9, 0.0, 0, 1.0, 0.0) == (1, 0.0)
    assert answers.draw([-np.inf, np.nan], 0.5, 1.0, 0, 1.0, 0.0) == (-1, -np.inf)
    assert answers.draw([1.0, 2.0, 2.0, 2.0], 0.6, 1.0, 2, 1.0, 0.0)[0] == 2  # of equal logits the lowest ids


def test_the_plain_norm_by_hand():
    y, h = answers.norm(torch.tensor([[3.0, 4.0]]), torch.tensor([[0.0, 0.0]]), torch.tensor([2.0, 1.0]), 0.0)
    assert np.allclose(y, [[6 / np.sqrt(12.5), 4 / np.sqrt(12.5)]]) and h.tolist() == [[3.0, 4.0]]
