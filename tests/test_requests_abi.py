"""Argument checks of the adapters' and beam search's calls through the C ABI,
on the host: a refused call launches nothing.  And the references' own pins."""
import ctypes

import numpy as np
import pytest
import torch

import ref_requests as ref
import weight_only_quantized_wql_gb300 as wql

OK, EINVAL, EUNSUPPORTED, ECUDA, EWORKSPACE = 0, 1, 2, 3, 4
A = 0x7F0000100000  # an aligned fake device address: never dereferenced by the checks
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(autouse=True)
def nothing_launched():
    before = wql.wql_launch_count()
    yield
    assert wql.wql_launch_count() == before


@pytest.fixture(scope="module")
def lib():
    return wql.load()


def test_lora_workspace():
    # u in 4 bytes a rank, padded to 16, 32, 64 or 128, and a factor per row
    for m, r, padded in ((1, 8, 16), (256, 64, 64), (3, 128, 128), (7, 40, 64), (1000, 24, 32)):
        size = wql.wql_lora_workspace_size(m, r)
        assert size % 256 == 0 and size >= m * padded * 4 + 4 * m
    for m, r in ((0, 8), (-1, 8), (1, 0), (1, 129), ((1 << 23) + 1, 8)):
        assert wql.wql_lora_workspace_size(m, r) == 0


def test_lora_refusals(lib):
    def call(dt=F16, rank=16, count=4, n=100, k=64, a=A, b=A, s=A, x=A, m=2, ids=A, y=A, out=A,
             ws=A, wsb=1 << 20):
        w = wql._WqlLora(dt, rank, count, n, k, a, b, s)
        return lib.wql_lora_add(ctypes.byref(w), x, m, ids, y, out, ws, wsb, None)

    assert lib.wql_lora_add(None, A, 2, A, A, A, A, 1 << 20, None) == EINVAL
    assert call(m=-1) == EINVAL
    assert call(count=-1) == EINVAL
    assert call(n=-1) == EINVAL
    assert call(k=0) == EINVAL
    assert call(rank=0) == EINVAL
    for name in ("a", "b", "x", "ids", "y", "out"):
        assert call(**{name: None}) == EINVAL, name
    assert call(dt=F32) == EUNSUPPORTED
    assert call(rank=12) == EUNSUPPORTED
    assert call(rank=136) == EUNSUPPORTED
    assert call(k=68) == EUNSUPPORTED
    assert call(k=(1 << 20) + 8) == EUNSUPPORTED
    assert call(n=1 << 31) == EUNSUPPORTED
    assert call(count=1 << 22) == EUNSUPPORTED
    assert call(m=(1 << 23) + 1) == EUNSUPPORTED
    for name, off in (("a", 8), ("b", 8), ("x", 8), ("s", 2), ("ids", 2), ("y", 1), ("out", 1)):
        assert call(**{name: A + off}) == EUNSUPPORTED, name
    assert call(ws=None) == EWORKSPACE
    assert call(ws=A + 16) == EWORKSPACE
    assert call(wsb=wql.wql_lora_workspace_size(2, 16) - 1) == EWORKSPACE
    assert call(m=0, x=None, ids=None, y=None, out=None, ws=None) == OK
    assert call(n=0, b=None, y=None, out=None, ws=None) == OK


def test_lora_out_shares_nothing(lib):
    """out is y, or apart from everything that the call reads."""
    at = {"x": 0x100000, "ids": 0x200000, "y": 0x300000, "out": 0x400000, "a": 0x500000,
          "b": 0x600000, "scale": 0x700000, "ws": 0x800000}
    m, n, k, count, rank = 3, 100, 64, 4, 16
    need = wql.wql_lora_workspace_size(m, rank)
    size = {"x": m * k * 2, "ids": m * 4, "y": m * n * 2, "a": count * rank * k * 2,
            "b": count * rank * n * 2, "scale": count * 4, "ws": need}

    def call(out):
        w = wql._WqlLora(F16, rank, count, n, k, at["a"], at["b"], at["scale"])
        return lib.wql_lora_add(ctypes.byref(w), at["x"], m, at["ids"], at["y"], out, at["ws"],
                                need, None)

    for name, bytes_ in size.items():
        assert call(at[name] + bytes_ - 2) == EINVAL, name
        assert call(at[name] - m * n * 2 + 2) == EINVAL, name
        if name != "y":
            assert call(at[name]) == EINVAL, name


def test_beam_workspace():
    # 8 bytes and a list of keys for every part of a row
    for b, w, n in ((1, 1, 1), (1, 4, 151936), (64, 4, 151936), (3, 32, 1 << 20)):
        size = wql.wql_beam_workspace_size(b, w, n)
        assert size % 256 == 0 and size >= b * w * (8 + 8 * w)
    for b, w, n in ((0, 4, 100), (1, 0, 100), (1, 33, 100), (1, 4, 0), (1, 4, (1 << 20) + 1),
                    (1 << 20, 2, 100)):
        assert wql.wql_beam_workspace_size(b, w, n) == 0


def test_beam_select_refusals(lib):
    def call(l=A, dt=F16, batch=2, beams=4, n=100, s=A, eos=-1, order=0, t=A, p=A, so=A, e=A, ws=A,
             wsb=1 << 20):
        return lib.wql_beam_select(l, dt, batch, beams, n, s, eos, order, t, p, so, e, ws, wsb, None)

    assert call(batch=-1) == EINVAL
    assert call(beams=0) == EINVAL
    assert call(n=0) == EINVAL
    assert call(eos=-2) == EINVAL
    assert call(eos=100) == EINVAL
    assert call(order=2) == EINVAL
    for name in ("l", "s", "t", "p", "so"):
        assert call(**{name: None}) == EINVAL, name
    assert call(dt=3) == EUNSUPPORTED
    assert call(beams=33) == EUNSUPPORTED
    assert call(n=(1 << 20) + 1) == EUNSUPPORTED
    assert call(batch=1 << 19) == EUNSUPPORTED
    assert call(l=A + 1) == EUNSUPPORTED
    assert call(l=A + 2, dt=F32) == EUNSUPPORTED
    for name in ("s", "t", "p", "so", "e"):
        assert call(**{name: A + 2}) == EUNSUPPORTED, name
    assert call(ws=None) == EWORKSPACE
    assert call(ws=A + 8) == EWORKSPACE
    assert call(wsb=wql.wql_beam_workspace_size(2, 4, 100) - 1) == EWORKSPACE
    assert call(batch=0, l=None, s=None, t=None, p=None, so=None, ws=None) == OK


def states(*fields):
    return (wql._WqlState * len(fields))(*(wql._WqlState(*f) for f in fields))


# (data, row stride, blocks, block stride, positions, position stride, position bytes)
def cache(at=A, rows=8, heads=2, length=10, dim=16):
    return (at, heads * length * dim, heads, length * dim, length, dim, dim)


def test_beam_reorder_refusals(lib):
    def call(st, parents=A, batch=2, beams=4, lengths=None, count=None):
        return lib.wql_beam_reorder(st, len(st) if st and count is None else (count or 0), parents,
                                    batch, beams, lengths, None)

    one = states(cache())
    assert call(one, batch=-1) == EINVAL
    assert call(one, beams=0) == EINVAL
    assert call(one, parents=None) == EINVAL
    assert call(None, count=1) == EINVAL
    assert call(one, count=-1) == EINVAL
    for i in range(1, 7):
        f = list(cache())
        f[i] = -1
        assert call(states(f)) == EINVAL, i
    assert call(states(cache(at=None))) == EINVAL
    assert call(one, beams=33) == EUNSUPPORTED
    assert call(one, batch=65536) == EUNSUPPORTED
    assert call(states(*[cache()] * 1025)) == EUNSUPPORTED
    assert call(one, parents=A + 2) == EUNSUPPORTED
    assert call(one, lengths=A + 2) == EUNSUPPORTED
    assert call(states((A, 1 << 40, 1, 0, 1, 16, 16))) == EUNSUPPORTED
    assert call(states((A, 1 << 33, 1 << 16, 1 << 16, 1 << 16, 1, 1))) == EUNSUPPORTED
    # spans that no memory has, and whose arithmetic would not fit
    assert call(states((A, 1 << 39, 1 << 30, 1 << 39, 1, 1, 1))) == EUNSUPPORTED
    assert call(states((A, 1 << 39, 1, 0, 1 << 30, 1 << 39, 1))) == EUNSUPPORTED
    assert call(states((A, 1 << 39, 1, 0, 1, 16, 16)), batch=65535) == EUNSUPPORTED
    assert call(one, count=0) == OK
    assert call(one, batch=0) == OK
    assert call(one, beams=1) == OK                       # nothing can move


def overlapping(lib, *fields):
    st = states(*fields)
    # one beam: a sound call has nothing to launch
    return lib.wql_beam_reorder(st, len(st), A, 8, 1, None, None) == EINVAL


def test_states_that_overlap(lib):
    c = cache()
    end = 8 * c[1]
    assert not overlapping(lib, c)
    assert not overlapping(lib, c, cache(at=A + end))
    assert overlapping(lib, c, c)                                     # the same one twice
    assert overlapping(lib, c, cache(at=A + end - 16))
    assert overlapping(lib, c, cache(at=A + 16))
    # a row that is not as long as what it holds, an expanded one
    assert overlapping(lib, (A, 300, 2, 160, 10, 16, 16))
    assert overlapping(lib, (A, 0, 2, 160, 10, 16, 16))
    assert overlapping(lib, (A, 320, 2, 160, 10, 8, 16))
    # keys and values in one tensor: [rows, 2, heads, length, dim] ...
    kv = (640, 2, 160, 10, 16, 16)
    assert not overlapping(lib, (A, *kv), (A + 320, *kv))
    assert overlapping(lib, (A, *kv), (A + 304, *kv))
    # ... [rows, heads, length, 2, dim], and [rows, heads, 2, length, dim]
    kv = (640, 2, 320, 10, 32, 16)
    assert not overlapping(lib, (A, *kv), (A + 16, *kv))
    assert not overlapping(lib, (A + 16, *kv), (A, *kv))
    assert overlapping(lib, (A, *kv), (A + 8, *kv))
    kv = (640, 2, 320, 10, 16, 16)
    assert not overlapping(lib, (A, *kv), (A + 160, *kv))
    # layers side by side, and a block that reaches into the next repetition
    assert not overlapping(lib, *((A + 64 * i, 256, 1, 0, 1, 64, 64) for i in range(4)))
    assert overlapping(lib, (A, 256, 1, 0, 1, 128, 128), (A + 192, 256, 1, 0, 1, 128, 128))
    # different strides over one span are not told apart
    assert overlapping(lib, (A, 256, 1, 0, 1, 16, 16), (A + 32, 512, 1, 0, 1, 16, 16))
    # rows inside positions: [length, rows, dim]
    assert not overlapping(lib, (A, 16, 1, 0, 10, 16 * 8, 16))
    assert overlapping(lib, (A, 16, 1, 0, 10, 16 * 7, 16))
    # empty ones overlap nothing
    assert not overlapping(lib, c, (A, 0, 0, 0, 10, 16, 16), (A, 0, 1, 0, 0, 16, 16))


def test_overlap_is_brute_force(lib):
    """Small states at random against the sets of their bytes; the check may
    refuse what does not overlap, and does so for a known share only."""
    rng = np.random.default_rng(1)

    def touched(f):
        at, rs, o, os, p, ps, pb = f
        return [at + r * rs + i * os + j * ps + k for r in range(8) for i in range(o)
                for j in range(p) for k in range(pb)]

    wrong = sound = 0
    for _ in range(3000):
        f = []
        for _ in range(2):
            o, p, pb = (int(v) for v in rng.integers(1, 4, 3))
            ps, os, rs = (int(v) for v in rng.choice([1, 2, 4, 8, 12, 24, 48], 3))
            f.append((A + int(rng.integers(0, 60)), rs, o, os, p, ps, pb))
        if rng.random() < 0.7:
            f[1] = (f[1][0], *f[0][1:])
        a, b = touched(f[0]), touched(f[1])
        clash = len(set(a)) < len(a) or len(set(b)) < len(b) or bool(set(a) & set(b))
        said = overlapping(lib, *f)
        assert said or not clash, f
        wrong += said and not clash
        sound += not clash
    assert wrong < 0.7 * sound, (wrong, sound)


@pytest.mark.parametrize("order", [(0, 1, 2, 3), (0, 2, 1, 3), (2, 0, 3, 1), (1, 0, 2, 3), (3, 0, 1, 2)])
def test_layers_of_one_allocation(lib, order):
    """Rows, heads, positions and layers of one tensor in any order: its layers lie apart,
    and two that share a byte are found among many."""
    sizes = (8, 3, 10, 150)
    stride, size = [0] * 4, 16
    for d in reversed(order):
        stride[d] = size
        size *= sizes[d]
    layers = [(A + l * stride[3], stride[0], 3, stride[1], 10, stride[2], 16) for l in range(150)]
    assert not overlapping(lib, *layers)
    assert not overlapping(lib, *layers[::-1])
    for l, by in ((0, 8), (70, -8), (149, 8)):
        moved = list(layers)
        moved[l] = (layers[l][0] + by, *layers[l][1:])
        # (the last layer's last byte has nothing behind it, where layers are outermost)
        if not (l == 149 and by > 0 and order[0] == 3):
            assert overlapping(lib, *moved), (l, by)
    assert overlapping(lib, *layers, layers[33])


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64, dtype=torch.float16)
    ad = wql.LoraAdapters(torch.zeros(1, 8, 64).half(), torch.zeros(1, 10, 8).half())
    for f in (lambda: wql.wql_lora_add(torch.zeros(2, 10).half(), x, ad,
                                       torch.zeros(2, dtype=torch.int32)),
              lambda: wql.wql_beam_select(x, torch.zeros(1, 2)),
              lambda: wql.wql_beam_reorder([x], torch.zeros(1, 2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()
    assert wql.wql_beam_reorder([], torch.zeros(1, 2, dtype=torch.int32)) == []


# ---------------------------------------------------------------------------
# the references
# ---------------------------------------------------------------------------
def test_select_worked():
    """Two beams with uniform rows over 4 tokens: the first beam's tokens 0, 1
    win; the end token 0 of the first beam counts, the second's does not."""
    l = np.zeros((1, 2, 4))
    t, p, s, e, _ = ref.beam_select(l, np.array([[0.0, -1.0]]), -1, False)
    assert t.tolist() == [[0, 1]] and p.tolist() == [[0, 0]]
    np.testing.assert_allclose(s, np.log(0.25))
    t, p, s, e, _ = ref.beam_select(l, np.array([[0.0, -1.0]]), 0, False)
    assert t.tolist() == [[1, 2]] and np.isclose(e[0, 0], np.log(0.25)) and e[0, 1] == -np.inf
    # anchored: both continue beam 1; its best stays there, the other takes slot 0
    t, p, s, e, _ = ref.beam_select(l, np.array([[-1.0, 0.0]]), -1, True)
    assert t.tolist() == [[1, 0]] and p.tolist() == [[1, 1]]
    # a row with infinities, a beam without a score, and not enough to go on
    l = np.array([[[0.0, np.inf, np.inf, np.nan], [1.0, 1.0, 1.0, 1.0], [-np.inf] * 4]])
    t, p, s, e, _ = ref.beam_select(l, np.array([[-2.0, -np.inf, 0.0]]), -1, False)
    assert t.tolist() == [[1, 2, -1]] and p.tolist() == [[0, 0, -1]]
    assert s.tolist() == [[-2.0, -2.0, -np.inf]]


def test_log_softmax_is_torchs():
    l = np.random.default_rng(0).normal(size=(3, 50)) * 5
    np.testing.assert_allclose(ref.log_softmax(l),
                               torch.log_softmax(torch.from_numpy(l), -1).numpy(), rtol=1e-12)


def test_reorder_worked():
    s = np.arange(12).reshape(4, 3)
    got = ref.reorder(s, np.array([[1, 0], [0, 5]]), np.array([2, 3]), 1)
    assert got.tolist() == [[3, 4, 2], [0, 1, 5], [6, 7, 8], [9, 10, 11]]


def test_lora_worked():
    y = np.zeros((3, 2))
    x = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    a = np.array([[[1.0, 1.0]], [[0.0, 1.0]]])                # rank 1
    b = np.array([[[1.0], [2.0]], [[3.0], [-1.0]]])
    out, _, _ = ref.lora(y, x, a, b, np.array([1.0, 0.5]), [0, 1, 2])
    assert out.tolist() == [[3.0, 6.0], [6.0, -2.0], [0.0, 0.0]]
